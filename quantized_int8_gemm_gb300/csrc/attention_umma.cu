// attention_umma.cu -- attention of new tokens over the paged cache on the
// tensor cores of sm_103a (tcgen05), for head widths up to 128.
//
// A unit (attention.cuh) is up to 256 rows of one K/V head, as two tiles of
// 128, over a run of K/V tiles of 128 keys.  For each tile t and key tile j
//   S_t = Q_t K_j^T   (TMEM, fp32)            one UMMA warp
//   P_t = exp2(scale S_t - m), 16 bits, over S_t's columns    softmax warps of t
//   O_t += P_t V_j    (TMEM, fp32; P read from TMEM)          the UMMA warp
// While the softmax warps of one tile work, the tensor core runs the other
// tile's products.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <numeric>

#include "attention.cuh"

namespace mmq {
namespace {

constexpr int kKt = 128;        // keys of a tile
constexpr int kThreads = 384;   // softmax warps 0-3 (tile 0) and 4-7 (tile 1), control warps 8-11
constexpr int kUmmaWarp = 8, kLoadWarp = 9, kTailWarp = 10;
constexpr int kRegsLaunch = 168, kRegsSoftmax = 216, kRegsControl = 72;
static_assert(256 * kRegsSoftmax + 128 * kRegsControl == kThreads * kRegsLaunch,
              "the register split must add up to what the launch holds");
constexpr int kUnits = 2;       // units handed out ahead
constexpr float kSlack = 8.0f;  // the running maximum may lag by 2^8 (see the softmax)

// Shared memory.  A tile of Q, K or V is kDp / 64 images of 128 rows x 128
// bytes with the 128-byte swizzle, 16 KB each.
template <int kDp>
struct Lay {
  static constexpr int kHalves = kDp / 64;
  static constexpr int kTile = kHalves * 16384;
  static constexpr int kStages = kDp == 64 ? 10 : 5;
  static constexpr int kQ = 0;
  static constexpr int kRing = 2 * kTile;
  static constexpr int kBars = kRing + kStages * kTile;
  static constexpr int kNumBars = 3 * kStages + 2 + 8 + 2 * kUnits + 1;
  static constexpr int kUnitsAt = kBars + kNumBars * 8;
  static constexpr int kSlot = kUnitsAt + kUnits * static_cast<int>(sizeof(AttnUnit));
  static constexpr int kBytes = kSlot + 16 + 1024;  // the base is rounded up to 1024
  static_assert(kBytes <= 232448, "shared memory of a CTA");
};

struct Maps {
  CUtensorMap q, k, v;
};

__device__ __forceinline__ void tma_load4(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
// D[tmem] (+)= A[tmem] . B[smem], 16-bit A packed two to a column
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Descriptor of V as the N x K operand: rows of memory are keys (K), 64
// contiguous elements of N a row; 128-byte swizzle.  Leading offset: from one
// 64-wide image to the next; stride offset: from eight keys to the next eight.
__device__ __forceinline__ uint64_t sdesc_nmajor_sw128(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(16384 >> 4) << 16 |
         static_cast<uint64_t>(1024 >> 4) << 32 | static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}
// idesc_f16_f32 with bf16 operands and, for V, B with N contiguous
template <class T>
constexpr uint32_t kFormat = 0;
template <>
constexpr uint32_t kFormat<__nv_bfloat16> = 1u << 7 | 1u << 10;
constexpr uint32_t kBNMajor = 1u << 16;

__device__ __forceinline__ uint32_t pack(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

template <class T, int kDp>
__global__ void __launch_bounds__(kThreads, 1)
    attention_umma_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ Maps maps, int tile_tok, int box) {
  using L = Lay<kDp>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t *smem = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = base + L::kBars;
  auto kv_full = [&](int s) { return bars + 8u * s; };
  auto kv_empty = [&](int s) { return bars + 8u * (L::kStages + s); };
  auto tail = [&](int s) { return bars + 8u * (2 * L::kStages + s); };
  constexpr int kFix = 3 * L::kStages;
  const uint32_t q_full = bars + 8u * kFix, q_empty = bars + 8u * (kFix + 1);
  auto s_full = [&](int t) { return bars + 8u * (kFix + 2 + t); };
  auto p_full = [&](int t) { return bars + 8u * (kFix + 4 + t); };
  auto o_full = [&](int t) { return bars + 8u * (kFix + 6 + t); };
  auto o_empty = [&](int t) { return bars + 8u * (kFix + 8 + t); };
  auto u_full = [&](int i) { return bars + 8u * (kFix + 10 + i); };
  auto u_empty = [&](int i) { return bars + 8u * (kFix + 10 + kUnits + i); };
  const uint32_t done = bars + 8u * (L::kNumBars - 1);
  AttnUnit *units = reinterpret_cast<AttnUnit *>(smem + L::kUnitsAt);
  const WaitCtl &w = a.wait;
  const int half_rows = tile_tok * a.rep;  // rows of one tile (at most 128)

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(kv_full(s), 1);
      mbar_init(kv_empty(s), 1);
      mbar_init(tail(s), 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_full(t), 1);
      mbar_init(p_full(t), 4);
      mbar_init(o_full(t), 1);
      mbar_init(o_empty(t), 4);
    }
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(u_full(i), 1);
      mbar_init(u_empty(i), 10);  // the UMMA warp, the tail warp and eight softmax warps
    }
    mbar_init(done, 1);
    fence_mbar_init();
  }
  if (warp == kUmmaWarp) {
    tmem_alloc(base + L::kSlot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::kSlot);
  auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity, w)) != 0; };
  // The next unit (false: none, or a wait ran out).
  auto take_unit = [&](uint32_t i, AttnUnit &un, bool &ok) {
    const int e = i % kUnits;
    ok = wait(u_full(e), (i / kUnits) & 1);
    if (!ok) return false;
    un = units[e];
    __syncwarp();
    if (lane == 0) mbar_arrive(u_empty(e));
    return un.n > 0;
  };
  auto two_tiles = [&](const AttnUnit &un) { return un.row0 + half_rows < un.n * a.rep; };
  // TMEM columns: S_t (and P_t over it) at 128 t, O_t at 256 + 128 t

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (warp == kLoadWarp) {
      // ---------------------------------------------------------- loads, and the units' order
      AttnSchedule<kKt> sched;
      sched.plan(a, 2 * half_rows, gridDim.x, 4);
      const int boxes = kKt / box;  // of a key tile, each `box` keys of one page
      uint32_t ks = 0, nu = 0, nq = 0;
      uint32_t tails = 0;           // stages whose last load was a tail
      bool ok = true;
      for (int u = blockIdx.x; ok; u += gridDim.x, ++nu) {
        AttnUnit un;
        const bool more = sched.find(a, u, un);
        if (!more) un.n = 0;
        const int e = nu % kUnits;
        ok = wait(u_empty(e), ((nu / kUnits) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) {
          units[e] = un;
          mbar_arrive(u_full(e));
        }
        if (!more) break;
        if (un.t_begin == un.t_end) continue;
        const bool two = two_tiles(un);
        ok = wait(q_empty, (nq & 1) ^ 1);
        if (!ok) break;
        ++nq;
        if (lane == 0) mbar_arrive_expect_tx(q_full, (two ? 2 : 1) * L::kHalves * half_rows * 128);
        __syncwarp();
        if (lane < 2 * L::kHalves) {
          const int t = lane / L::kHalves, h = lane % L::kHalves;
          if (t == 0 || two)
            tma_load4(base + L::kQ + t * L::kTile + h * 16384, &maps.q, h * 64, 0, un.head, un.q0 + un.row0 / a.rep + t * tile_tok, q_full);
        }
        const int32_t *row = a.table + un.b * a.table_stride;
        const int mine = lane / L::kHalves, h = lane % L::kHalves;  // (boxes * halves <= 32)
        auto page_of = [&](int t) {
          const int key = t * kKt + mine * box;
          int id = 0;
          if (mine < boxes && key < un.len && t < un.t_end) {
            id = row[key / a.page_size];
            if (id < 0 || id >= a.pages) {  // out of the cache: past the map's last page, zeros come
              record_index(w.status);
              id = static_cast<int>(a.pages);
            }
          }
          return id;
        };
        int next = page_of(un.t_begin);
        for (int t = un.t_begin; t < un.t_end && ok; ++t) {
          const int id = next, key = t * kKt + mine * box, off = key % a.page_size;
          next = page_of(t + 1);
          const int keys = min(kKt, un.len - t * kKt), n = (keys + box - 1) / box;
          const bool load = mine < n;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++ks) {
            const int s = ks % L::kStages;
            ok = wait(kv_empty(s), ((ks / L::kStages) & 1) ^ 1);
            if (!ok) break;
            // the last keys' V goes through the tail warp
            const bool last = kv == 1 && keys < kKt;
            const uint32_t bar = last ? tail(s) : kv_full(s);
            tails = last ? tails | 1u << s : tails & ~(1u << s);
            if (lane == 0) mbar_arrive_expect_tx(bar, n * L::kHalves * box * 128);
            __syncwarp();
            if (load)
              tma_load4(base + L::kRing + s * L::kTile + h * 16384 + mine * box * 128, kv ? &maps.v : &maps.k, h * 64, off, un.head, id, bar);
          }
        }
      }
      if (!ok) {  // drain this CTA's copies still in flight
        if (nq) mbar_wait(q_full, (nq - 1) & 1, w, false);
        const uint32_t from = ks > L::kStages ? ks - L::kStages : 0;
        for (uint32_t i = from; i < ks; ++i) {
          const int s = i % L::kStages;
          if (!(tails >> s & 1)) mbar_wait(kv_full(s), (i / L::kStages) & 1, w, false);
          else for (int spin = 0; spin < 4096 && !(mbar_try_wait(tail(s), 0) && mbar_try_wait(tail(s), 1)); ++spin) {}
        }
      }
    } else if (warp == kTailWarp) {
      // ---------------------------------------------------------- the last keys' V
      // Rows past the last key, up to the next multiple of 16 (the K of one
      // UMMA), hold what the page holds there, or an earlier tile: zeros, so
      // that 0 * V is 0.
      uint32_t ks = 0, nu = 0, phase = 0;
      bool ok = true;
      AttnUnit un;
      while (take_unit(nu++, un, ok)) {
        const int tiles = un.t_end - un.t_begin;
        if (tiles == 0) continue;
        const int keys = un.len - (un.t_end - 1) * kKt;
        ks += 2 * tiles;
        if (keys >= kKt) continue;
        const int s = (ks - 1) % L::kStages;
        ok = wait(tail(s), phase >> s & 1);
        if (!ok) break;
        phase ^= 1u << s;
        const int zero = ((keys + 15) & ~15) - keys;
        uint8_t *v = smem + L::kRing + s * L::kTile;
        for (int i = lane; i < zero * 8 * L::kHalves; i += 32) {
          const int r = keys + i / (8 * L::kHalves), c = i % (8 * L::kHalves);
          *reinterpret_cast<uint4 *>(v + (c >> 3) * 16384 + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(kv_full(s));
      }
    } else if (warp == kUmmaWarp) {
      // ---------------------------------------------------------- UMMAs
      uint32_t elected;
      asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(elected));
      constexpr uint32_t id_qk = idesc_f16_f32(128, kKt) | kFormat<T>;
      constexpr uint32_t id_pv = idesc_f16_f32(128, kDp) | kFormat<T> | kBNMajor;
      uint32_t ks = 0, nu = 0, nq = 0, np[2] = {0, 0}, no[2] = {0, 0};
      bool ok = true;
      AttnUnit un;
      auto qk = [&](int t, int s) {
        if (elected) {
          const uint64_t qd = sdesc_kmajor_sw128(base + L::kQ + t * L::kTile), kd = sdesc_kmajor_sw128(base + L::kRing + s * L::kTile);
#pragma unroll
          for (int k = 0; k < kDp / 16; ++k) {
            const uint64_t at = (k >> 2) * (16384 >> 4) + (k & 3) * 2;
            umma_f16(tmem + 128 * t, qd + at, kd + at, id_qk, k > 0);
          }
          umma_commit(s_full(t));
        }
        __syncwarp();
      };
      auto pv = [&](int t, int s, int steps, bool fresh) {
        if (elected) {
          const uint64_t vd = sdesc_nmajor_sw128(base + L::kRing + s * L::kTile);
          for (int k = 0; k < steps; ++k)
            umma_ts(tmem + 256 + 128 * t, tmem + 128 * t + 8 * k, vd + k * (2048 >> 4), id_pv, !(fresh && k == 0));
        }
        __syncwarp();
      };
      while (take_unit(nu++, un, ok)) {
        const int tiles = un.t_end - un.t_begin;
        if (tiles == 0) continue;
        const int n_t = two_tiles(un) ? 2 : 1;
        ok = wait(q_full, nq++ & 1) && wait(kv_full(ks % L::kStages), (ks / L::kStages) & 1);
        if (!ok) break;
        tc_fence_after();
        for (int t = 0; t < n_t; ++t) qk(t, ks % L::kStages);
        if (elected) {
          umma_commit(kv_empty(ks % L::kStages));
          if (tiles == 1) umma_commit(q_empty);
        }
        __syncwarp();
        ++ks;
        for (int j = 0; j < tiles && ok; ++j, ks += 2) {
          // ks: V of tile j, ks + 1: K of tile j + 1
          const int sv = ks % L::kStages, sk = (ks + 1) % L::kStages;
          const bool more = j + 1 < tiles;
          const int keys = min(kKt, un.len - (un.t_begin + j) * kKt), steps = (keys + 15) >> 4;
          ok = wait(kv_full(sv), (ks / L::kStages) & 1);
          for (int t = 0; t < n_t && ok; ++t) {
            if (j == 0) ok = wait(o_empty(t), (no[t]++ & 1) ^ 1);
            ok = ok && wait(p_full(t), np[t]++ & 1);
            if (ok && more && t == 0) ok = wait(kv_full(sk), ((ks + 1) / L::kStages) & 1);
            if (!ok) break;
            tc_fence_after();
            pv(t, sv, steps, j == 0);
            if (t == n_t - 1) {
              if (elected) umma_commit(kv_empty(sv));
              __syncwarp();
            }
            if (more) {
              qk(t, sk);
            } else {
              if (elected) umma_commit(o_full(t));
              __syncwarp();
            }
          }
          if (ok && more) {
            if (elected) {
              umma_commit(kv_empty(sk));
              if (j + 2 == tiles) umma_commit(q_empty);  // the unit's last Q K^T
            }
            __syncwarp();
          }
        }
        if (!ok) break;
        --ks;  // the loop counted a K past the unit's last V
      }
      if (elected) umma_commit(done);
      __syncwarp();
      mbar_wait(done, 0, w, false);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ------------------------------------------------------------ softmax: one row a thread
    const int t = warp >> 2, quad = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t ts = tmem + lanes + 128 * t, to = tmem + lanes + 256 + 128 * t;
    const float sc = a.scale_log2;
    uint32_t nu = 0, ns = 0, no = 0;
    bool ok = true;
    AttnUnit un;
    while (take_unit(nu++, un, ok)) {
      if (t == 1 && !two_tiles(un)) continue;
      const int r = quad * 32 + lane, row = un.row0 + t * half_rows + r, tok = row / a.rep;
      const bool valid = r < half_rows && row < un.n * a.rep;
      const bool some = __any_sync(0xffffffffu, valid);
      int lo, hi;
      attn_row_range(a, un.n, un.len, tok, lo, hi);
      float m = -INFINITY, l = 0.0f;
      for (int j = un.t_begin; j < un.t_end; ++j) {
        ok = wait(s_full(t), ns & 1);
        if (!ok) break;
        ++ns;
        tc_fence_after();
        if (some) {
          uint32_t x[2][64];
          tmem_ld_32x32b_x64(ts, x[0]);
          tmem_ld_32x32b_x64(ts + 64, x[1]);
          tmem_wait_ld(x[0]);
          tmem_wait_ld(x[1]);
          const int from = lo - j * kKt, span = hi - lo;
          if (__any_sync(0xffffffffu, valid && (from > 0 || hi < (j + 1) * kKt))) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int c = 0; c < 64; ++c)
                if (span <= 0 || static_cast<uint32_t>(h * 64 + c - from) >= static_cast<uint32_t>(span)) x[h][c] = 0xff800000u;
          }
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < 64; ++c) top[c & 3] = fmaxf(top[c & 3], __uint_as_float(x[h][c]));
          const float tile_top = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
          // The maximum is only a guard against overflow: any m gives the same
          // quotient.  It moves when it would lag by more than 2^8, so that O
          // in TMEM is rescaled a few times a row and not in every tile; the
          // weights then stay below 2^8, within both 16-bit types.  O is at
          // rest here: S_t(j) was issued behind the last P_t V.
          const bool lags = valid && (tile_top - m) * sc > kSlack;  // (also from -inf; NaN: no)
          if (j == un.t_begin) {
            m = tile_top;
          } else if (__any_sync(0xffffffffu, lags)) {
            const float now = lags ? tile_top : m;
            const float f = lags ? exp2_fast((m - now) * sc) : 1.0f;
            m = now;
            l *= f;
#pragma unroll
            for (int c = 0; c < kDp; c += 32) {
              uint32_t y[32];
              tmem_ld_32x32b_x32(to + c, y);
              tmem_wait_ld(y);
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
              tmem_st_32x32b_x32(to + c, y);
            }
          }
          const float off = m == -INFINITY ? 0.0f : m * sc;
          float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t p[32];
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
              const float e0 = exp2_fast(fmaf(__uint_as_float(x[h][c]), sc, -off));
              const float e1 = exp2_fast(fmaf(__uint_as_float(x[h][c + 1]), sc, -off));
              sum[c & 2] += e0;
              sum[(c & 2) + 1] += e1;
              p[c / 2] = pack(e0, e1, T());  // one rounding, to the type of V: the UMMA's operands have one type
            }
            tmem_st_32x32b_x32(ts + 32 * h, p);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(t));
      }
      if (!ok) break;
      // ---- the row's result
      const int head = un.head * a.rep + row - tok * a.rep;
      const int64_t at = static_cast<int64_t>(un.q0 + tok) * a.hq + head;
      const bool none = un.t_begin == un.t_end;
      if (!none) {
        ok = wait(o_full(t), no & 1);
        if (!ok) break;
        ++no;
        tc_fence_after();
      }
      const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;  // (NaN stays)
      if (some) {
        const bool split = un.pieces > 1;
        float *po = a.part_o + (un.piece * a.ntok * a.hq + at) * a.d;
        const int64_t oat = (un.q0 + tok) * a.out_token + head * a.out_head;
#pragma unroll
        for (int c = 0; c < kDp; c += 32) {
          uint32_t y[32];
          if (none) {
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = 0;
          } else {
            tmem_ld_32x32b_x32(to + c, y);
            tmem_wait_ld(y);
          }
          if (!valid) continue;
          // a row without a key in these tiles has P = 0 throughout
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(l == 0.0f ? 0.0f : __uint_as_float(y[i]) * inv);
          if (split || a.out_type == MMQ_DT_F32) {
            float *dst = split ? po : static_cast<float *>(a.out) + oat;
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              if (c + i < a.d) *reinterpret_cast<uint4 *>(dst + c + i) = make_uint4(y[i], y[i + 1], y[i + 2], y[i + 3]);
          } else {
            T *dst = static_cast<T *>(a.out) + oat;
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              if (c + i >= a.d) continue;
              uint4 z;
              z.x = pack(__uint_as_float(y[i]), __uint_as_float(y[i + 1]), T());
              z.y = pack(__uint_as_float(y[i + 2]), __uint_as_float(y[i + 3]), T());
              z.z = pack(__uint_as_float(y[i + 4]), __uint_as_float(y[i + 5]), T());
              z.w = pack(__uint_as_float(y[i + 6]), __uint_as_float(y[i + 7]), T());
              *reinterpret_cast<uint4 *>(dst + c + i) = z;
            }
          }
        }
        if (valid) {
          const float lse2 = l > 0.0f ? fmaf(m, sc, log2f(l)) : l == 0.0f ? -INFINITY : l;
          if (split) {
            a.part_lse[un.piece * a.ntok * a.hq + at] = lse2;
            if (un.piece == 0) a.part_n[at] = un.pieces;
          } else {
            if (a.lse) a.lse[at] = lse2 * kLn2;
            if (a.max_pieces > 1) a.part_n[at] = 1;
          }
        }
      }
      if (!none) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_empty(t));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kUmmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static const EncodeFn fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult got;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &got) != cudaSuccess ||
        got != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// A map of four dimensions (row, and three with strides in elements), boxes of
// 64 elements by b1 x 1 x b3.
bool encode(CUtensorMap *m, int type, const void *p, int64_t d, const int64_t (&n)[3], const int64_t (&stride)[3], int b1, int b3) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(n[0]), static_cast<cuuint64_t>(n[1]),
                              static_cast<cuuint64_t>(n[2])};
  cuuint64_t bytes[3];
  // (a dimension of one element has no stride; the map wants one all the same)
  for (int i = 0; i < 3; ++i) bytes[i] = static_cast<cuuint64_t>(n[i] == 1 ? d : stride[i]) * 2;
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(b1), 1, static_cast<cuuint32_t>(b3)}, one[4] = {1, 1, 1, 1};
  return encoder()(m, type == MMQ_DT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                   const_cast<void *>(p), dims, bytes, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, int kDp>
cudaError_t launch_umma(const AttnArgs &a, const Maps &maps, int tile_tok, int box, int dev, unsigned grid, cudaStream_t s) {
  constexpr auto kern = attention_umma_kernel<T, kDp>;
  static std::atomic<int> ready[64];  // 0 unknown, 1 ready, 2 unusable
  int st = ready[dev].load();
  if (st == 0) {
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<kDp>::kBytes);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    st = fa.numRegs == kRegsLaunch ? 1 : 2;  // (a mismatch would stall setmaxnreg)
    ready[dev].store(st);
  }
  if (st != 1) return cudaErrorInvalidKernelImage;
  attention_umma_kernel<T, kDp><<<grid, kThreads, Lay<kDp>::kBytes, s>>>(a, maps, tile_tok, box);
  return cudaGetLastError();
}

}  // namespace

// The tile shape of the tcgen05 kernel for this problem; false: it does not
// take it.  Pages are copied in boxes of gcd(page_size, 128) keys, at least
// eight, so that a box is whole swizzle groups and a warp's lanes cover a tile.
bool attention_umma_shape(const mmq_paged_cache &c, const mmq_attention &t, int *tile_tok, int *box) {
  const int rep = t.q_heads / c.heads;
  *box = std::gcd(c.page_size, kKt);
  *tile_tok = rep <= 128 ? 128 / rep : 0;
  return c.head_dim <= 128 && rep <= 128 && *box >= 8 && encoder();
}

cudaError_t launch_attention_umma(const AttnArgs &a, const mmq_paged_cache &c, int tile_tok, int box, int dev, unsigned grid,
                                  cudaStream_t s, bool *taken) {
  Maps m;
  *taken = encode(&m.q, c.type, a.q, a.d, {a.rep, a.hkv, a.ntok}, {a.q_head, a.rep * a.q_head, a.q_token}, a.rep, tile_tok) &&
           encode(&m.k, c.type, a.k, a.d, {c.page_size, a.hkv, a.pages}, {a.k_token, a.k_head, a.k_page}, box, 1) &&
           encode(&m.v, c.type, a.v, a.d, {c.page_size, a.hkv, a.pages}, {a.v_token, a.v_head, a.v_page}, box, 1);
  if (!*taken) return cudaSuccess;
  if (c.type == MMQ_DT_F16)
    return a.d <= 64 ? launch_umma<__half, 64>(a, m, tile_tok, box, dev, grid, s) : launch_umma<__half, 128>(a, m, tile_tok, box, dev, grid, s);
  return a.d <= 64 ? launch_umma<__nv_bfloat16, 64>(a, m, tile_tok, box, dev, grid, s)
                   : launch_umma<__nv_bfloat16, 128>(a, m, tile_tok, box, dev, grid, s);
}

}  // namespace mmq
