// attention_umma.cu -- attention of new tokens over the paged cache on the
// tensor cores of sm_103a (tcgen05), for head widths up to 128.
//
// A unit (attention.cuh) is up to 256 rows of one K/V head, as two tiles of
// 128, over tiles of 128 keys.  There are two lanes t of
//   S_t = Q K_j^T   (TMEM, fp32)                            UMMA warp t
//   P_t = exp2(scale S_t - m), 16 bits, into TMEM           softmax warps of t
//   O_t += P_t V_j  (TMEM, fp32; P read from TMEM)          UMMA warp t
// and while the softmax warps of one lane work, the tensor core runs the other
// lane's products.  With two row tiles lane t is row tile t and sees every key
// tile.  With one (decode steps, short chunks) both lanes are that tile: lane t
// takes every second key tile, and their results are joined at the end.
//
// What bounds it (one GB300, calls back to back):
//   long chunks  (4096 tokens over 32097 keys, 28 heads on 4, d 128: 1.09 to
//       1.18 ms by clocks, 1.5 to 1.6 PFLOP/s) the chain of one lane, softmax
//       about 1.7 thousand clocks, P V and Q K^T 0.5 each and the hand-offs: a
//       key tile of both lanes takes about 2.6 thousand clocks, 2.05 of them
//       UMMAs, whose operands also take all of shared memory's bandwidth;
//   heads of 64  (prompts of 301 to 2630 tokens, window 1000: 59 us) the softmax
//       warps, about 2.4 thousand clocks a key tile of both lanes, and what a
//       unit of few tiles costs beside them;
//   decode steps (64 tokens over 97 to 12002 keys, 333 MB: 65 us) HBM while the
//       tiles run, about 51 us; the rest is the first tile's way in (5 us: plan,
//       page ids, copies, first products, code met for the first time), the last
//       one's way out and the join.
// Tried and left out: two softmax threads a row on sixteen warps (77 against
// 66 us for the decode steps, 1283 against 1150 for the chunk), four warps for
// the copies (36 against 34 us for drafted tokens), waits that hand the warp to
// the hardware for longer (no change), a rehearsal of the softmax code while the
// plan is made (4 us more).
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
constexpr int kUmmaWarp = 8, kLoadWarp = 10;  // UMMA warp of lane t: 8 + t; 10: K, 11: V
constexpr int kRegsLaunch = 168, kRegsSoftmax = 208, kRegsControl = 88;
static_assert(256 * kRegsSoftmax + 128 * kRegsControl == kThreads * kRegsLaunch,
              "the register split must add up to what the launch holds");
constexpr int kUnits = 2;       // units handed out ahead
constexpr float kSlack = 8.0f;  // the running maximum may lag by 2^8 (see the softmax)

// Shared memory.  A tile of Q, K or V is kDp / 64 images of 128 rows x 128
// bytes with the 128-byte swizzle, 16 KB each.
template <int kDp>
struct Lay {
  static constexpr int kHalves = kDp / 64;
  // TMEM columns.  S_0, S_1; for heads of 64 there is room for P beside S, so
  // that Q K^T of the next key tile runs while the softmax of this one does.
  static constexpr bool kApart = kDp == 64;
  static constexpr int kO = 256, kP = kApart ? 256 + 2 * kDp : 0, kPStep = kApart ? 64 : 128;
  static constexpr int kTile = kHalves * 16384;
  static constexpr int kStages = kDp == 64 ? 10 : 5;
  static constexpr int kQ = 0;
  static constexpr int kRing = 2 * kTile;
  static constexpr int kBars = kRing + kStages * kTile;
  static constexpr int kNumBars = 3 * kStages + 2 + 18 + 2 * kUnits + 2;
  static constexpr int kStats = kBars + kNumBars * 8;  // [lane][row] maximum and sum
  static constexpr int kUnitsAt = kStats + 2 * 128 * 8;
  static constexpr int kSlot = kUnitsAt + kUnits * static_cast<int>(sizeof(AttnUnit));
  static constexpr int kBytes = kSlot + 16;
  static_assert(kBytes <= 232448, "shared memory of a CTA");
};

__device__ __forceinline__ void tma_load4(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
// (no branch: the warp stays together)
__device__ __forceinline__ void mbar_arrive_if(bool yes, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
      "r"(static_cast<uint32_t>(yes))
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

__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void parts_of(uint64_t p, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 32 lanes x 32 columns, and the largest of each lane's 32 (fp32; NaN is passed over).
__device__ __forceinline__ void tmem_ld_max_x32(uint32_t taddr, uint32_t *r, float &top) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, %32, [%33];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=f"(top)
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Bits [from, to) of 32.
__device__ __forceinline__ uint32_t bits_of(int from, int to) {
  auto below = [](int n) { return n >= 32 ? 0xffffffffu : (1u << max(n, 0)) - 1; };
  return below(to) & ~below(from);
}

template <class T, int kDp>
__global__ void __launch_bounds__(kThreads, 1)
    attention_umma_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ AttnUmma um) {
  using L = Lay<kDp>;
  extern __shared__ __align__(1024) uint8_t smem[];  // (swizzle groups are 1024 bytes)
  const uint32_t base = smem_addr(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = base + L::kBars;
  auto kv_full = [&](int s) { return bars + 8u * s; };
  auto kv_empty = [&](int s) { return bars + 8u * (L::kStages + s); };
  auto tail = [&](int s) { return bars + 8u * (2 * L::kStages + s); };
  constexpr int kFix = 3 * L::kStages;
  const uint32_t q_full = bars + 8u * kFix, q_empty = bars + 8u * (kFix + 1);
  auto s_full = [&](int t) { return bars + 8u * (kFix + 2 + t); };
  auto p_full = [&](int t, int half) { return bars + 8u * (kFix + 4 + 2 * t + half); };
  auto o_full = [&](int t) { return bars + 8u * (kFix + 8 + t); };
  auto o_empty = [&](int t) { return bars + 8u * (kFix + 10 + t); };
  const uint32_t stats_full = bars + 8u * (kFix + 12), stats_empty = bars + 8u * (kFix + 13);
  auto turn = [&](int t) { return bars + 8u * (kFix + 14 + t); };
  auto s_empty = [&](int t) { return bars + 8u * (kFix + 16 + t); };
  auto p_empty = [&](int t) { return bars + 8u * (kFix + 18 + t); };
  auto u_full = [&](int i) { return bars + 8u * (kFix + 20 + i); };
  auto u_empty = [&](int i) { return bars + 8u * (kFix + 20 + kUnits + i); };
  const uint32_t added = bars + 8u * (L::kNumBars - 2), done = bars + 8u * (L::kNumBars - 1);
  AttnUnit *units = reinterpret_cast<AttnUnit *>(smem + L::kUnitsAt);
  const WaitCtl &w = a.wait;
  float2 *stats = reinterpret_cast<float2 *>(smem + L::kStats);
  // More than 32 requests: the softmax warps add up their rooms on the units'
  // line, into the place of the statistics (4096 requests of 301 keys, 8 heads on
  // 1: 187 us, 1024, 28 heads on 4: 167; 291 and 194 by the planning warp alone,
  // when that was changed).
  int *sums = reinterpret_cast<int *>(stats);
  static_assert((kAttnSums + 1) * sizeof(int) <= 2 * 128 * sizeof(float2));
  volatile uint32_t *last = reinterpret_cast<volatile uint32_t *>(smem + L::kSlot + 8);  // the load warps' loads of the ring, at their end
  const int tile_tok = um.tile_tok, box = um.box;
  const int half_rows = tile_tok * a.rep;  // rows of one tile (at most 128)

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(kv_full(s), 1);
      mbar_init(kv_empty(s), 2);  // both UMMA warps
      mbar_init(tail(s), 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_full(t), 1);
      mbar_init(p_full(t, 0), 4);
      mbar_init(p_full(t, 1), 4);
      mbar_init(o_full(t), 1);
      mbar_init(o_empty(t), 8);
      mbar_init(turn(t), 1);
      mbar_init(s_empty(t), 4);
      mbar_init(p_empty(t), 1);
    }
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(u_full(i), 1);
      mbar_init(u_empty(i), 11);  // the UMMA warps, the V warp and eight softmax warps
    }
    mbar_init(stats_full, 8);
    mbar_init(stats_empty, 8);
    mbar_init(done, 2);
    mbar_init(added, 8);
    sums[kAttnSums] = 0;
    fence_mbar_init();
  }
  if (warp == kLoadWarp + 1 && lane < 3) {
    const CUtensorMap *m = lane == 0 ? &um.q : lane == 1 ? &um.k : &um.v;
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
  }
  if (warp == kUmmaWarp) {
    tmem_alloc(base + L::kSlot, 512);
    tmem_relinquish();
  }
  AttnUnit un;
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
    mbar_arrive_if(lane == 0, u_empty(e));
    return un.n > 0;
  };
  auto two_tiles = [&](const AttnUnit &un) { return un.row0 + half_rows < un.n * a.rep; };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    griddep_wait();
    griddep_launch_dependents();  // the next kernel's CTAs come as these leave
    if (warp >= kLoadWarp) {
      // ---------------------------------------------------------- loads: one warp K, and the units' order; one Q and V
      // (a warp issues a copy every 69 clocks whatever its size, and a tile of
      // 16-token pages is 16 copies of 2 KB)
      const int kv = warp - kLoadWarp;
      const int boxes = kKt / box;                                // of a key tile, each `box` keys of one page
      const int mine = lane / L::kHalves, h = lane % L::kHalves;  // (boxes * halves <= 32)
      const CUtensorMap *map = kv ? &um.v : &um.k;
      uint32_t ks = kv, nu = 0, nq = 0;  // ks: this warp's next load of the ring
      uint32_t tails = 0, phase = 0;     // stages whose last load (of this warp) went to tail(), and its phases
      uint32_t open = 0;                 // those that it has not been waited for
      bool ok = true;
      AttnSchedule<kKt, 0> sched;
      if (kv == 0) {
        sched.no_cut(a);
        if (a.nreq > 32) ok = wait(added, 0);
        if (ok) sched.plan(a, sums);
      }
      for (; ok; ++nu) {
        if (kv == 0) {
          if (!sched.next(a, un)) un.n = 0;
          const int e = nu % kUnits;
          ok = wait(u_empty(e), ((nu / kUnits) & 1) ^ 1);
          if (!ok) break;
          if (lane == 0) {
            units[e] = un;
            mbar_arrive(u_full(e));
          }
          if (un.n == 0) break;
        } else if (!take_unit(nu, un, ok)) {
          break;
        }
        if (un.t_begin == un.t_end) continue;
        // page ids are read two tiles ahead and looked at when they are used
        const int32_t *row = a.table + un.b * a.table_stride;
        auto page_of = [&](int t) {
          const int key = t * kKt + mine * box;
          return mine < boxes && key + box > un.from && key < un.len && t < un.t_end ? row[a.by_page(key)] : 0;
        };
        int ahead[2] = {page_of(un.t_begin), page_of(un.t_begin + 1)};
        if (kv) {
          const bool two = two_tiles(un);
          ok = wait(q_empty, (nq & 1) ^ 1);
          if (!ok) break;
          ++nq;
          if (lane == 0) mbar_arrive_expect_tx(q_full, (two ? 2 : 1) * L::kHalves * half_rows * 128);
          __syncwarp();
          if (lane < 2 * L::kHalves) {
            const int t = lane / L::kHalves, g = lane % L::kHalves;
            if (t == 0 || two)
              tma_load4(base + L::kQ + t * L::kTile + g * 16384, &um.q, g * 64, 0, un.head, un.q0 + a.by_rep(un.row0) + t * tile_tok, q_full);
          }
        }
        // V rows before the first key that a window leaves, or past the last
        // one up to the next multiple of 16 (the K of one UMMA), hold what the
        // page holds there, or an earlier tile: zeros, so that 0 * V is 0.
        auto finish = [&](int s, int skip, int keys) {
          if (!wait(tail(s), phase >> s & 1)) return false;
          phase ^= 1u << s;
          open &= ~(1u << s);
          const int behind = -keys & 15;
          uint8_t *v = smem + L::kRing + s * L::kTile;
          for (int i = lane; i < (skip + behind) * 8 * L::kHalves; i += 32) {
            const int x = i / (8 * L::kHalves), c = i % (8 * L::kHalves), r = x < skip ? x : keys + x - skip;
            *reinterpret_cast<uint4 *>(v + (c >> 3) * 16384 + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(kv_full(s));
          return true;
        };
        int held = -1;  // a first tile's V, finished when the next copy is on its way
        for (int t = un.t_begin; t < un.t_end; ++t) {
          int id = ahead[0];
          ahead[0] = ahead[1];
          ahead[1] = page_of(t + 2);
          const int key = t * kKt + mine * box, off = key - a.by_page(key) * a.page_size;
          const int keys = min(kKt, un.len - t * kKt), skip = max(0, un.from - t * kKt);
          const int box_log2 = 31 - __clz(box), n0 = skip >> box_log2, n = (keys + box - 1) >> box_log2;  // (a divisor of 128)
          const int s = ks % L::kStages;
          ok = wait(kv_empty(s), ((ks / L::kStages) & 1) ^ 1);
          if (!ok) break;
          if (id < 0 || id >= a.pages) {  // out of the cache: past the map's last page, zeros come
            record_index(w.status);
            id = static_cast<int>(a.pages);
          }
          const bool edge = kv == 1 && (keys < kKt || skip);  // V with rows that are no keys
          const uint32_t bar = edge ? tail(s) : kv_full(s);
          tails = edge ? tails | 1u << s : tails & ~(1u << s);
          if (edge) open |= 1u << s;
          if (lane == 0) mbar_arrive_expect_tx(bar, (n - n0) * L::kHalves * box * 128);
          __syncwarp();
          if (mine >= n0 && mine < n) tma_load4(base + L::kRing + s * L::kTile + h * 16384 + mine * box * 128, map, h * 64, off, un.head, id, bar);
          ks += 2;  // (also where a wait below runs out: the copy is on its way)
          if (held >= 0) ok = finish(held, un.from - un.t_begin * kKt, kKt);
          held = edge && t + 1 < un.t_end ? s : -1;
          if (ok && edge && held < 0) ok = finish(s, skip, keys);
          if (!ok) break;
        }
        if (!ok) break;
      }
      // No CTA ends with a copy in flight, whoever gave up: both warps have issued
      // their last load here, and each waits for those of its own that may not
      // have landed, the last of a stage.  (All have where no wait ran out.)
      if (lane == 0) last[kv] = ks;
      __syncwarp();
      asm volatile("bar.sync 1, 64;" ::: "memory");  // both load warps
      if (nq) mbar_wait(q_full, (nq - 1) & 1, w, false);
      for (int64_t k = static_cast<int64_t>(ks) - 2; k >= 0 && k + L::kStages + 2 > ks; k -= 2) {
        const int s = static_cast<int>(k % L::kStages);
        // the other warp has loaded the stage again: this load was used (with an even ring it never does)
        if ((L::kStages & 1) && k + L::kStages < last[kv ^ 1]) continue;
        if (!(tails >> s & 1)) mbar_wait(kv_full(s), static_cast<uint32_t>(k / L::kStages) & 1, w, false);
        else if (open >> s & 1) mbar_wait(tail(s), phase >> s & 1, w, false);
      }
    } else {
      // ---------------------------------------------------------- UMMAs of lane t
      // Two warps, as the tensor pipe queues little work: while one waits for
      // its weights or a stage, the other keeps it fed.  S_t, P_t and O_t are
      // this warp's alone, and its UMMAs run in the order they are issued in.
      const int t = warp - kUmmaWarp;
      uint32_t elected;
      asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(elected));
      constexpr uint32_t id_qk = idesc_f16_f32(128, kKt) | kFormat<T>;
      constexpr uint32_t id_pv = idesc_f16_f32(128, kDp) | kFormat<T> | kBNMajor;
      const uint64_t kd0 = sdesc_kmajor_sw128(base + L::kRing), vd0 = sdesc_nmajor_sw128(base + L::kRing);
      const uint32_t d_s = tmem + 128 * t, d_o = tmem + L::kO + kDp * t, d_p = tmem + L::kP + L::kPStep * t;
      uint32_t ks = 0, nu = 0, nq = 0, np = 0, no = 0, nt = 0, ns = 0;
      bool ok = true;
      auto stage = [&](uint32_t k) { return static_cast<int>(k % L::kStages); };
      auto landed = [&](uint32_t k) { return wait(kv_full(stage(k)), (k / L::kStages) & 1); };
      // Both lanes pass every load of the ring in its order, also those only
      // the other one uses: a lane that skipped a stage's load could take the
      // load before it for its own (a phase is told by its parity).
      auto skip = [&](uint32_t k) {
        const bool got = landed(k);
        mbar_arrive_if(got && lane == 0, kv_empty(stage(k)));
        return got;
      };
      // With two row tiles the lanes take turns (P_t V of one key tile and Q K^T
      // of the next are one turn), so that one lane's softmax runs beside the
      // other's UMMAs; left alone they fall into step and the tensor pipe idles
      // while both wait for their weights (3.9 against 3.0 thousand clocks a
      // key tile).
      auto my_turn = [&](bool two) { return L::kApart || !two || wait(turn(t), (nt++ & 1) ^ (t == 0)); };
      // S_t = Q K^T from load k
      auto qk = [&](uint64_t qd, uint32_t k, bool two, bool known) {
        bool got = known || landed(k);
        if (L::kApart && got) got = wait(s_empty(t), (ns++ & 1) ^ 1);
        if (got) {
          tc_fence_after();
          if (elected) {
            const uint64_t kd = kd0 + stage(k) * (L::kTile >> 4);
#pragma unroll
            for (int i = 0; i < kDp / 16; ++i) {
              const uint64_t at = (i >> 2) * (16384 >> 4) + (i & 3) * 2;
              umma_f16(d_s, qd + at, kd + at, id_qk, i > 0);
            }
            if (!L::kApart && two) mbar_arrive(turn(t ^ 1));
            umma_commit(s_full(t));
            umma_commit(kv_empty(stage(k)));
          }
          __syncwarp();
        }
        return got;
      };
      // O_t (+)= P_t V from load k; the first 64 keys' weights may be there before the rest
      auto pv = [&](uint32_t k, int steps, bool fresh, bool two, bool last) {
        bool got = landed(k);
        if (!L::kApart && got && two && !last) got = landed(k + 1);  // (the next key tile's K, so that the turn does not wait for it)
        if (got && fresh) got = wait(o_empty(t), (no++ & 1) ^ 1);
        const uint64_t vd = vd0 + stage(k) * (L::kTile >> 4);
        const uint32_t parity = np++ & 1;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (got) got = wait(p_full(t, half), parity);
          if (got && half == 0) got = my_turn(two);
          if (!got) return false;
          tc_fence_after();
          if (elected) {
#pragma unroll
            for (int i = 4 * half; i < 4 * half + 4; ++i)
              if (i < steps) umma_ts(d_o, d_p + 8 * i, vd + i * (2048 >> 4), id_pv, !(fresh && i == 0));
            if (half) {
              if (!L::kApart && two && last) mbar_arrive(turn(t ^ 1));
              umma_commit(kv_empty(stage(k)));
              if (L::kApart) umma_commit(p_empty(t));
            }
          }
          __syncwarp();
        }
        return true;
      };
      while (take_unit(nu++, un, ok)) {
        const int tiles = un.t_end - un.t_begin;
        if (tiles == 0) continue;
        const bool two = two_tiles(un);
        ok = wait(q_full, nq++ & 1);
        if (!ok) break;
        const uint64_t qd = sdesc_kmajor_sw128(base + L::kQ + (two ? t : 0) * L::kTile);
        const int first = two ? 0 : t, dj = two ? 1 : 2;  // this lane's key tiles
        const uint32_t end = ks + 2 * tiles;              // loads: K of tile j at ks + 2j, then its V
        // the other lane's tile before key tile j, if it has one there
        auto pass = [&](int j) { return two || j < 1 || (skip(ks + 2 * j - 2) && skip(ks + 2 * j - 1)); };
        auto qk_of = [&](int j) {
          ok = pass(j) && qk(qd, ks + 2 * j, two, !L::kApart && two && j != first);
          if (ok && j + dj >= tiles) {  // the lane's last
            if (elected) umma_commit(q_empty);
            __syncwarp();
          }
        };
        if (first < tiles) {
          ok = my_turn(two);
          if (ok) qk_of(first);
        } else if (lane == 0) {
          mbar_arrive(q_empty);
        }
        for (int j = first; j < tiles && ok; j += dj) {
          const bool last = j + dj >= tiles;
          if (L::kApart && !last) qk_of(j + dj);
          ok = ok && pv(ks + 2 * j + 1, (min(kKt, un.len - (un.t_begin + j) * kKt) + 15) >> 4, j == first, two, last);
          if (!L::kApart && ok && !last) qk_of(j + dj);
          if (ok && last) {
            if (elected) umma_commit(o_full(t));
            __syncwarp();
          }
        }
        if (ok && !two && ((tiles - 1) & 1) != t) ok = skip(end - 2) && skip(end - 1);
        if (!ok) break;
        ks = end;
      }
      if (elected) umma_commit(done);
      __syncwarp();
      mbar_wait(done, 0, w, false);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    griddep_wait();
    griddep_launch_dependents();
    if (a.nreq > 32) {
      AttnSchedule<kKt, 0> rooms;
      rooms.add_up(a, warp, kUmmaWarp, sums);
      __syncwarp();
      mbar_arrive_if(lane == 0, added);
    }
    // ------------------------------------------------------------ softmax: one row a thread
    const int t = warp >> 2, quad = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t ts = tmem + lanes + 128 * t, tp = tmem + lanes + L::kP + L::kPStep * t;
    const uint32_t to = tmem + lanes + L::kO + kDp * t, other_o = tmem + lanes + L::kO + kDp * (t ^ 1);
    const float sc = a.scale_log2;
    uint32_t nu = 0, ns = 0, no[2] = {0, 0}, nx = 0;
    bool ok = true;
    while (take_unit(nu++, un, ok)) {
      const bool two = two_tiles(un);
      const int tiles = un.t_end - un.t_begin, q = two ? t : 0;
      const int r = quad * 32 + lane, row = un.row0 + q * half_rows + r, tok = a.by_rep(row);
      const bool valid = r < half_rows && row < un.n * a.rep;
      const bool some = __any_sync(0xffffffffu, valid);
      int lo, hi;
      attn_row_range(a, un.place, un.len, tok, lo, hi);
      float m = -INFINITY, l = 0.0f;
      // 64 weights and their sums.  Eight at a time, the exponentials of one
      // group beside the sums and conversions of the one before: exp2 keeps its
      // unit busy for 4 clocks a warp, the packed FMA, the add and the
      // conversion two each.  The one rounding is to the type of V (a UMMA's
      // operands have one type).
      auto weights = [](const uint32_t (&x)[64], uint32_t (&p)[32], uint64_t sc2, uint64_t off2, uint64_t (&sum)[2]) {
        float e[2][8];
#pragma unroll
        for (int g = 0; g <= 8; ++g)
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            float *now = e[g & 1] + i, *old = e[(g & 1) ^ 1] + i;
            if (g < 8) {
              parts_of(fma2(pair_of(__uint_as_float(x[8 * g + i]), __uint_as_float(x[8 * g + i + 1])), sc2, off2), now[0], now[1]);
              now[0] = exp2_fast(now[0]);
            }
            if (g > 0) sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], pair_of(old[0], old[1]));
            if (g < 8) now[1] = exp2_fast(now[1]);
            if (g > 0) p[4 * (g - 1) + i / 2] = pack(old[0], old[1], T());
          }
      };
      // The maximum is only a guard against overflow: any m gives the same
      // quotient.  It moves when it would lag by more than 2^8, so that O in
      // TMEM is rescaled a few times a row and not in every tile; the weights
      // then stay below 2^8, within both 16-bit types.  O is at rest when this
      // is called: P_t V of the tile before is done (where P lies over S, S_t
      // was issued behind it).
      auto follow = [&](float tile_top, bool first) {
        const bool lags = valid && (tile_top - m) * sc > kSlack;  // (also from -inf; NaN: no)
        if (first) {
          m = tile_top;
        } else if (__any_sync(0xffffffffu, lags)) {
          const float now = lags ? tile_top : m;
          const float f = lags ? exp2_fast((m - now) * sc) : 1.0f;
          m = now;
          l *= f;
#pragma unroll 1
          for (int c = 0; c < kDp; c += 16) {
            uint32_t y[16];
            tmem_ld_x16(to + c, y);
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
            tmem_st_x16(to + c, y);
          }
        }
      };
      const int j0 = un.t_begin + (two ? 0 : t), dj = two ? 1 : 2;
      for (int j = j0; j < un.t_end; j += dj) {
        ok = wait(s_full(t), ns & 1);
        if (!ok) break;
        ++ns;
        tc_fence_after();
        if (some) {
          if constexpr (L::kApart) {
            // Hidden keys: S is set to -inf in TMEM first, 32 columns at a time
            // (small code; few tiles have any).  A row's keys are the bits of a
            // word, so that a column costs one select (compared with both ends: 61
            // against 58 us for the prompts; in registers behind the load 59.5).
            const int from = lo - j * kKt, to_key = hi - j * kKt;
            if (__any_sync(0xffffffffu, valid && (from > 0 || to_key < kKt))) {
#pragma unroll 1
              for (int c = 0; c < kKt; c += 32) {
                const uint32_t seen = bits_of(from - c, to_key - c);
                if (!__any_sync(0xffffffffu, valid && seen != 0xffffffffu)) continue;
                uint32_t y[32];
                tmem_ld_32x32b_x32(ts + c, y);
                tmem_wait_ld(y);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (!(seen >> i & 1)) y[i] = 0xff800000u;
                tmem_st_32x32b_x32(ts + c, y);
              }
              tmem_wait_st();
            }
            uint32_t x[2][64];
            float top[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) tmem_ld_max_x32(ts + 32 * h, x[h >> 1] + 32 * (h & 1), top[h]);
            tmem_wait_ld(x[0]);
            tmem_wait_ld(x[1]);
            asm volatile("" : "+f"(top[0]), "+f"(top[1]), "+f"(top[2]), "+f"(top[3]));
            tc_fence_before();
            __syncwarp();
            mbar_arrive_if(lane == 0, s_empty(t));
            ok = wait(p_empty(t), (ns & 1));  // P_t V of the tile before (ns counts this tile already)
            if (!ok) break;
            tc_fence_after();
            follow(max3(fmaxf(top[0], top[1]), top[2], top[3]), j == j0);
            const float off = m == -INFINITY ? 0.0f : -m * sc;
            const uint64_t sc2 = pair_of(sc, sc), off2 = pair_of(off, off);
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t p[32];
              weights(x[h], p, sc2, off2, sum);
              tmem_st_32x32b_x32(tp + 32 * h, p);
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              mbar_arrive_if(lane == 0, p_full(t, h));
            }
            float s0, s1;
            parts_of(add2(sum[0], sum[1]), s0, s1);
            l += s0 + s1;
          } else {
            // Two passes over S, both in short loops: the tile's code has to stay
            // in the instruction caches of warps that run different parts of it
            // (unrolled over all 128 columns, warps waited for instructions as
            // often as they issued one).  First the maximum.
            const int from = lo - j * kKt, to_key = hi - j * kKt;
            const bool ends = __any_sync(0xffffffffu, valid && (from > 0 || to_key < kKt));
            // (P V stops at the last key: 1024 decode rows over 171 keys 122 us, 134 with both halves)
            const int halves = un.len - j * kKt <= kKt / 2 ? 1 : 2;
            float top[4];
            if (!ends) {
              uint32_t x[4][32];
#pragma unroll
              for (int h = 0; h < 4; ++h) tmem_ld_max_x32(ts + 32 * h, x[h], top[h]);
              tmem_wait_ld();
              asm volatile("" : "+f"(top[0]), "+f"(top[1]), "+f"(top[2]), "+f"(top[3]));
            } else {  // hidden keys (the tiles at a row's ends) become -inf in TMEM
              top[0] = top[1] = top[2] = top[3] = -INFINITY;
#pragma unroll 1
              for (int c = 0; c < 64 * halves; c += 32) {
                const int y0 = from - c, y1 = to_key - c;
                uint32_t y[32];
                tmem_ld_32x32b_x32(ts + c, y);
                tmem_wait_ld(y);
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                  if (i < y0 || i >= y1) y[i] = 0xff800000u;
                  if (i + 1 < y0 || i + 1 >= y1) y[i + 1] = 0xff800000u;
                  top[(i >> 1) & 3] = max3(top[(i >> 1) & 3], __uint_as_float(y[i]), __uint_as_float(y[i + 1]));
                }
                tmem_st_32x32b_x32(ts + c, y);
              }
              tmem_wait_st();
            }
            follow(max3(fmaxf(top[0], top[1]), top[2], top[3]), j == j0);
            const float off = m == -INFINITY ? 0.0f : -m * sc;
            const uint64_t sc2 = pair_of(sc, sc), off2 = pair_of(off, off);
            uint64_t sum[2] = {0, 0};
            // Then the weights, 64 columns at a time (over S: behind what has been read).
#pragma unroll 1
            for (int h = 0; h < halves; ++h) {
              uint32_t x[64], p[32];
              tmem_ld_32x32b_x64(ts + 64 * h, x);
              tmem_wait_ld(x);
              weights(x, p, sc2, off2, sum);
              tmem_st_32x32b_x32(tp + 32 * h, p);
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              mbar_arrive_if(lane == 0, p_full(t, h));
            }
            if (halves == 1) mbar_arrive_if(lane == 0, p_full(t, 1));
            float s0, s1;
            parts_of(add2(sum[0], sum[1]), s0, s1);
            l += s0 + s1;
          }
        } else {
          if (L::kApart) {
            mbar_arrive_if(lane == 0, s_empty(t));
            ok = wait(p_empty(t), (ns & 1));
            if (!ok) break;
          }
          mbar_arrive_if(lane == 0, p_full(t, 0));
          mbar_arrive_if(lane == 0, p_full(t, 1));
        }
      }
      if (!ok) break;
      // ---- the rows' results: of lane t, or of both lanes together, where the
      // warps of each lane write half the columns
      const bool both = !two && tiles > 1;
      if (!two && !both && t == 1) {  // nothing of this unit came here
        if (tiles) ++no[0];
        continue;
      }
      float f0 = 1.0f, f1 = 0.0f;  // of O_t and of the other lane's
      if (tiles) {
        if (both) {
          ok = wait(stats_empty, (nx & 1) ^ 1);
          if (!ok) break;
          stats[128 * t + r] = make_float2(m, l);
          __syncwarp();
          mbar_arrive_if(lane == 0, stats_full);
          ok = wait(stats_full, nx++ & 1) && wait(o_full(t ^ 1), no[t ^ 1] & 1);
          if (!ok) break;
        }
        ok = wait(o_full(t), no[t] & 1);
        if (!ok) break;
        tc_fence_after();
        ++no[0];
        if (two || both) ++no[1];
        if (both) {
          const float2 x = stats[128 * (t ^ 1) + r];
          __syncwarp();
          mbar_arrive_if(lane == 0, stats_empty);
          const float top = fmaxf(m, x.x), off = top == -INFINITY ? 0.0f : top;
          f0 = exp2_fast((m - off) * sc);
          f1 = exp2_fast((x.x - off) * sc);
          m = top;
          l = __fadd_rn(__fmul_rn(l, f0), __fmul_rn(x.y, f1));  // (the same number in both lanes)
        }
      }
      const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;  // (NaN stays)
      f0 *= inv;
      f1 *= inv;
      const int head = un.head * a.rep + row - tok * a.rep;
      const int64_t at = static_cast<int64_t>(un.q0 + tok) * a.hq + head;
      if (some) {
        const bool cut = un.slot >= 0;
        float4 *po = a.part_o + static_cast<int64_t>(un.slot) * (a.d / 4) * (2 * half_rows) + (row - un.row0);
        const int64_t oat = (un.q0 + tok) * a.out_token + head * a.out_head;
        // the row of this lane's pair of lanes that it writes to in the second store
        const int64_t here = valid ? oat : -1, other = __shfl_xor_sync(0xffffffffu, here, 1);
        const bool odd = lane & 1;
        // 16 columns a turn of a short loop: run once a unit, straight code
        // costs about five clocks an instruction, waiting to be fetched.
#pragma unroll 1
        for (int c = both ? kDp / 2 * t : 0; c < (both && t == 0 ? min(a.d, kDp / 2) : a.d); c += 16) {
          uint32_t y[16];
          if (tiles == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = 0;
          } else {
            tmem_ld_x16(to + c, y);
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * f0);
            if (both) {
              uint32_t z[16];
              tmem_ld_x16(other_o + c, z);
#pragma unroll
              for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(fmaf(__uint_as_float(z[i]), f1, __uint_as_float(y[i])));
            }
          }
          const bool full = c + 16 <= a.d;  // (else eight columns)
          if (cut) {
            if (valid) {
              float4 *dst = po + (c / 4) * (2 * half_rows);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (i < 2 || full)
                  dst[i * (2 * half_rows)] = make_float4(__uint_as_float(y[4 * i]), __uint_as_float(y[4 * i + 1]),
                                                         __uint_as_float(y[4 * i + 2]), __uint_as_float(y[4 * i + 3]));
            }
          } else if (a.out_type == MMQ_DT_F32) {
            if (valid) {
              uint4 *dst = reinterpret_cast<uint4 *>(static_cast<float *>(a.out) + oat + c);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (i < 2 || full) dst[i] = make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
            }
          } else {
            // Two lanes swap 16-byte chunks, so that they write 32 bytes of one
            // row together (a store to 32 rows takes the memory pipe 32 clocks).
            uint32_t z[2][4];
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i >> 2][i & 3] = pack(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1]), T());
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t give = odd ? z[0][k] : z[1][k], got = __shfl_xor_sync(0xffffffffu, give, 1);
              if (odd) z[0][k] = got;
              else z[1][k] = got;
            }
            // even lane: chunk 0 of its row, then of the odd lane's; odd lane: chunk 1 of the even lane's, then of its own
            const int64_t r0 = odd ? other : here, r1 = odd ? here : other;
            T *dst = static_cast<T *>(a.out) + c + 8 * odd;
            if (full || !odd) {
              if (r0 >= 0) *reinterpret_cast<uint4 *>(dst + r0) = make_uint4(z[0][0], z[0][1], z[0][2], z[0][3]);
              if (r1 >= 0) *reinterpret_cast<uint4 *>(dst + r1) = make_uint4(z[1][0], z[1][1], z[1][2], z[1][3]);
            }
          }
        }
        if (valid && !(both && t)) {
          const float lse2 = l > 0.0f ? fmaf(m, sc, log2f(l)) : l == 0.0f ? -INFINITY : l;
          if (cut) a.part_lse[un.slot * (2 * half_rows) + row - un.row0] = lse2;
          else if (a.lse) a.lse[at] = lse2 * kLn2;
        }
      }
      if (tiles) {
        tc_fence_before();
        __syncwarp();
        // eight arrivals a lane's O: both lanes' warps once, or its own twice
        mbar_arrive_if(lane == 0, o_empty(t));
        mbar_arrive_if(lane == 0, o_empty(both ? t ^ 1 : t));
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
// 64 elements by b1 x 1 x b3.  128 bytes a request to memory: a head of 64 is no
// longer, and with 256 the next head's row came with it, often for nothing (64
// decode rows of 5001 keys, 8 K/V heads of 64, pages of 16: 111 to 121 us by
// machine, 155 to 161 with 256; heads of 128 alike).
bool encode(CUtensorMap *m, int type, const void *p, int64_t d, const int64_t (&n)[3], const int64_t (&stride)[3], int b1, int b3) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(n[0]), static_cast<cuuint64_t>(n[1]),
                              static_cast<cuuint64_t>(n[2])};
  cuuint64_t bytes[3];
  // (a dimension of one element has no stride; the map wants one all the same)
  for (int i = 0; i < 3; ++i) bytes[i] = static_cast<cuuint64_t>(n[i] == 1 ? d : stride[i]) * 2;
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(b1), 1, static_cast<cuuint32_t>(b3)}, one[4] = {1, 1, 1, 1};
  return encoder()(m, type == MMQ_DT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                   const_cast<void *>(p), dims, bytes, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, int kDp>
cudaError_t launch_umma(const AttnArgs &a, const AttnUmma &u, int dev, unsigned grid, cudaStream_t s) {
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
  return launch_early(attention_umma_kernel<T, kDp>, grid, 1, kThreads, Lay<kDp>::kBytes, s, a, u);
}

}  // namespace

// The tcgen05 kernel takes head widths and groups of query heads up to 128.
// Pages are copied in boxes of gcd(page_size, 128) keys, at least eight, so
// that a box is whole swizzle groups and a warp's lanes cover a tile.
bool attention_umma(const AttnArgs &a, int type, AttnUmma *u) {
  if (a.d > 128 || a.rep > 128) return false;
  u->tile_tok = 128 / a.rep;
  u->box = std::gcd(a.page_size, kKt);
  return u->box >= 8 && encoder() &&
         encode(&u->q, type, a.q, a.d, {a.rep, a.hkv, a.ntok}, {a.q_head, a.rep * a.q_head, a.q_token}, a.rep, u->tile_tok) &&
         encode(&u->k, type, a.k, a.d, {a.page_size, a.hkv, a.pages}, {a.k_token, a.k_head, a.k_page}, u->box, 1) &&
         encode(&u->v, type, a.v, a.d, {a.page_size, a.hkv, a.pages}, {a.v_token, a.v_head, a.v_page}, u->box, 1);
}

cudaError_t launch_attention_umma(const AttnArgs &a, const AttnUmma &u, int type, int dev, unsigned grid, cudaStream_t s) {
  if (type == MMQ_DT_F16) return a.d <= 64 ? launch_umma<__half, 64>(a, u, dev, grid, s) : launch_umma<__half, 128>(a, u, dev, grid, s);
  return a.d <= 64 ? launch_umma<__nv_bfloat16, 64>(a, u, dev, grid, s) : launch_umma<__nv_bfloat16, 128>(a, u, dev, grid, s);
}

}  // namespace mmq
