// lora.cu -- low-rank adapters of many requests beside a shared projection:
// out[t] = y[t] + s_a (x[t] A_a^T) B_a^T with the adapter a of token t's request.
//
// The plan sorts a step's tokens by adapter, once for all its projections, and
// cuts them into tiles of one adapter.  A cluster of eight CTAs takes a tile:
// each multiplies an eighth of x's columns by A, the partial sums are joined
// through the cluster's shared memory, and each writes an eighth of the output
// columns.  So a tile's x, y and out go through once, in one launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace mmq {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// ---------------------------------------------------------------- plan
// Words: [0] tiles, [1] tiles with an adapter (they come first), then ntok
// token rows in the adapters' order, then (adapter, first entry, entries) a tile.
constexpr int kHead = 4;
constexpr int kPlanThreads = 1024, kPlanTokens = 8192;  // tokens of a CTA
constexpr int kRequestBits = 13;                        // kMaxRequests
constexpr uint32_t kEmpty = 0xffffffffu, kNone = 1u << 18;

__device__ __forceinline__ int plan_exclusive(int x, int &total, int *sm, bool largest) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto join = [&](int p, int q) { return largest ? max(p, q) : p + q; };
  int s = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(kAll, s, d);
    if (lane >= d) s = join(s, y);
  }
  if (lane == 31) sm[warp] = s;
  const int up = __shfl_up_sync(kAll, s, 1);
  __syncthreads();
  int all = sm[lane];  // (32 warps)
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(kAll, all, d);
    if (lane >= d) all = join(all, y);
  }
  total = __shfl_sync(kAll, all, 31);
  const int before = __shfl_sync(kAll, all, warp > 0 ? warp - 1 : 0);
  __syncthreads();
  return join(warp > 0 ? before : 0, lane > 0 ? up : 0);
}

// The largest i in [0, n) with sums[i] <= x (sums ascending, sums[0] <= x).
__device__ __forceinline__ int last_not_above(const int *sums, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Keys (adapter, request) are sorted in shared memory, so the order does not
// depend on the threads'.  Every CTA sorts for itself and writes its tokens.
__global__ void __launch_bounds__(kPlanThreads) lora_plan_kernel(const __grid_constant__ LoraPlanArgs a) {
  extern __shared__ uint32_t keys[];  // a.slots (a power of two), then the tokens and the tiles before each key
  __shared__ int s_warp[32];
  __shared__ int s_bad;
  int *tokens_before = reinterpret_cast<int *>(keys + a.slots), *tiles_before = tokens_before + a.slots;
  const int tid = threadIdx.x, nreq = static_cast<int>(a.nreq), ntok = static_cast<int>(a.ntok);
  griddep_wait();
  griddep_launch_dependents();
  if (tid == 0) s_bad = 0;
  __syncthreads();
  auto bounds = [&](int b, int &begin, int &end) {
    begin = a.q_start[b], end = a.q_start[b + 1];
    const bool descends = end < begin || begin < 0;
    begin = min(max(begin, 0), ntok), end = min(max(end, 0), ntok);
    return !descends;
  };
  for (int i = tid; i < a.slots; i += kPlanThreads) {
    uint32_t key = kEmpty;
    if (i < nreq) {
      int begin, end;
      if (!bounds(i, begin, end)) s_bad = 1, record_index(a.status);
      int id = a.adapters[i];
      if (id < -1 || id >= a.nadapters) record_index(a.status), id = -1;
      if (end > begin) key = (id < 0 ? kNone : static_cast<uint32_t>(id)) << kRequestBits | static_cast<uint32_t>(i);
    }
    keys[i] = key;
  }
  __syncthreads();
  for (int size = 2; size <= a.slots; size <<= 1) {
    for (int step = size >> 1; step; step >>= 1) {
      for (int i = tid; i < a.slots >> 1; i += kPlanThreads) {
        const int p = 2 * i - (i & (step - 1)), q = p + step;
        const uint32_t x = keys[p], y = keys[q];
        if ((x > y) == ((p & size) == 0)) keys[p] = y, keys[q] = x;
      }
      __syncthreads();
    }
  }
  // (each thread has the keys from tid * per on)
  const int per = (a.slots + kPlanThreads - 1) / kPlanThreads, i0 = min(tid * per, a.slots), i1 = min(i0 + per, a.slots);
  auto length = [&](int i) {
    if (keys[i] == kEmpty) return 0;
    int begin, end;
    bounds(static_cast<int>(keys[i] & ((1u << kRequestBits) - 1)), begin, end);
    return end - begin;
  };
  auto adapter = [&](int i) { return keys[i] >> kRequestBits; };
  int sum = 0, total, none;
  for (int i = i0; i < i1; ++i) sum += length(i);
  int at = plan_exclusive(sum, total, s_warp, false);
  int first = 0;  // largest begin of a group up to here
  for (int i = i0; i < i1; ++i) {
    tokens_before[i] = at;
    if (i == 0 || adapter(i - 1) != adapter(i)) first = at;
    at += length(i);
  }
  __syncthreads();
  const int before = plan_exclusive(first, none, s_warp, true);
  auto tiles_of = [&](int i, int &start) {  // tiles of the group that ends with key i
    if (i == 0 || adapter(i - 1) != adapter(i)) start = tokens_before[i];
    const int end = i + 1 < a.slots ? tokens_before[i + 1] : total;
    const bool last = keys[i] != kEmpty && (i + 1 == a.slots || adapter(i + 1) != adapter(i));
    return last ? (end - start + a.tile - 1) / a.tile : 0;
  };
  int start = before, tiles = 0, all_tiles;
  for (int i = i0; i < i1; ++i) tiles += tiles_of(i, start);
  int tile = plan_exclusive(tiles, all_tiles, s_warp, false);
  start = before;
  for (int i = i0; i < i1; ++i) {
    tiles_before[i] = tile;
    tile += tiles_of(i, start);
  }
  __syncthreads();
  if (s_bad) total = all_tiles = 0;
  int32_t *order = a.plan + kHead, *list = order + ntok;
  const int p0 = static_cast<int>(blockIdx.x) * kPlanTokens, p1 = min(p0 + kPlanTokens, total);
  for (int p = p0 + tid; p < p1; p += kPlanThreads) {
    const int i = last_not_above(tokens_before, a.slots, p);
    // (keys without tokens stand last, behind every token)
    order[p] = a.q_start[keys[i] & ((1u << kRequestBits) - 1)] + (p - tokens_before[i]);
  }
  for (int k = static_cast<int>(blockIdx.x) * kPlanThreads + tid; k < all_tiles; k += static_cast<int>(gridDim.x) * kPlanThreads) {
    const int i = last_not_above(tiles_before, a.slots, k);
    int g = i;  // the group's first key
    if (i > 0) {
      int lo = -1, hi = i;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (adapter(mid) == adapter(i)) hi = mid;
        else lo = mid;
      }
      g = hi;
    }
    const int end = i + 1 < a.slots ? tokens_before[i + 1] : total;
    const int begin = tokens_before[g] + (k - tiles_before[i]) * a.tile;
    const uint32_t id = adapter(i);
    list[3 * k] = id == kNone ? -1 : static_cast<int>(id);
    list[3 * k + 1] = begin;
    list[3 * k + 2] = min(a.tile, end - begin);
    if (id != kNone && (k + 1 == all_tiles || adapter(last_not_above(tiles_before, a.slots, k + 1)) == kNone)) a.plan[1] = k + 1;
    if (k == 0 && id == kNone) a.plan[1] = 0;
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.plan[0] = all_tiles;
    if (all_tiles == 0) a.plan[1] = 0;
  }
}

// ---------------------------------------------------------------- products
constexpr int kCtas = 8, kThreads = 256, kWarps = kThreads / 32;
constexpr int kRankPass = 64;  // ranks whose sums a warp holds at once

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// D += A B, 16 x 16 by 16 x 8, bf16 in, fp32 sums.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// A pair of numbers as two bf16 terms: x = h + l, off by 2^-18 of x at the most
// (each term is rounded to nearest, 2^-9 of what it stands for).  An infinite or
// NaN number keeps its value in h and has l = 0 or NaN.
struct Terms {
  uint32_t h, l;
};
__device__ __forceinline__ Terms split(float x, float y) {
  Terms t;
  t.h = pack(x, y);
  t.l = pack(x - low(t.h), y - high(t.h));
  return t;
}

// Eight numbers of a row of weights, as bf16: exactly, fp16 weights as two terms.
template <class W>
struct Weights8;
template <>
struct Weights8<__nv_bfloat16> {
  uint32_t h[4];
  __device__ __forceinline__ void set(uint4 r) { h[0] = r.x, h[1] = r.y, h[2] = r.z, h[3] = r.w; }
};
template <>
struct Weights8<__half> {
  uint32_t h[4], l[4];
  __device__ __forceinline__ void set(uint4 r) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
      const Terms t = split(f.x, f.y);
      h[i] = t.h, l[i] = t.l;
    }
  }
};

// The lane's eight columns (two steps of 16) of rows p and q of weights by
// those of eight rows of terms.  Which column is which within the 32 does not matter as
// long as both sides agree: lane quarter c has columns 8c .. 8c + 7, which lie
// together in memory.
template <class W>
__device__ __forceinline__ void product(float (&d)[4], const Weights8<W> &p, const Weights8<W> &q, const Terms (&x)[4]) {
#pragma unroll
  for (int k = 0; k < 4; k += 2) {
    mma(d, p.h[k], q.h[k], p.h[k + 1], q.h[k + 1], x[k].h, x[k + 1].h);
    mma(d, p.h[k], q.h[k], p.h[k + 1], q.h[k + 1], x[k].l, x[k + 1].l);
    if constexpr (sizeof(Weights8<W>) == 32) mma(d, p.l[k], q.l[k], p.l[k + 1], q.l[k + 1], x[k].h, x[k + 1].h);
  }
}

__device__ __forceinline__ uint4 zero4() { return make_uint4(0, 0, 0, 0); }

// Eight numbers of x as terms.
__device__ __forceinline__ void load_x(Terms (&out)[4], const void *row, int x_type, int k, bool there) {
  float v[8] = {};
  if (there) {
    if (x_type == MMQ_DT_F32) {
      const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(row) + k);
      const float4 a = __ldg(p), b = __ldg(p + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      const uint4 r = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(row) + k));
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = x_type == MMQ_DT_F16 ? __half22float2(*reinterpret_cast<const __half2 *>(&w[i])) : make_float2(low(w[i]), high(w[i]));
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = split(v[2 * i], v[2 * i + 1]);
}

// Shared memory: partial sums of the CTA's warps; of the CTA; the joined sums
// as terms, a token's ranks together, rows 16 words from a multiple of 32
// apart (eight lanes of a 16-byte read then touch every bank once).
template <int kTile>
struct Shape {
  static constexpr int kTokens = kTile > 16 ? 16 : kTile;      // tokens of a warp in the first product
  static constexpr int kGroups = kTile / kTokens;              // warps side by side over tokens
  static constexpr int kSplit = kWarps / kGroups;              // and over the columns of x
  static constexpr int kColumns = kTokens / 8;
  __host__ __device__ static constexpr int pitch(int rank) { return (rank + 31) / 32 * 16 % 32 ? (rank + 31) / 32 * 16 : (rank + 31) / 32 * 16 + 16; }
  static size_t bytes(int rank) {
    return 4 * (static_cast<size_t>(kSplit) * kRankPass * kTile + static_cast<size_t>((rank + 15) / 16 * 16) * kTile +
                2 * static_cast<size_t>(kTile) * pitch(rank));
  }
};

template <class W, int kTile>
__global__ void __launch_bounds__(kThreads, 2) __cluster_dims__(kCtas, 1, 1) lora_kernel(const __grid_constant__ LoraArgs a) {
  using S = Shape<kTile>;
  extern __shared__ __align__(16) float smem[];
  __shared__ int s_row[kTile];
  const mmq_lora_args &t = a.t;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int rank = static_cast<int>(cluster_ctarank()), tile = static_cast<int>(blockIdx.x / kCtas);
  griddep_wait();
  griddep_launch_dependents();
  const bool in_place = t.y == t.out;
  if (tile >= t.plan[in_place ? 1 : 0]) return;  // (the whole cluster)
  const int32_t *entry = t.plan + kHead + t.ntok + 3 * static_cast<int64_t>(tile);
  const int adapter = entry[0], first = entry[1], n = entry[2];
  if (tid < kTile) s_row[tid] = tid < n ? t.plan[kHead + first + tid] : -1;
  const int id = static_cast<int>(t.id), od = static_cast<int>(t.od), rmax = t.rank;
  const int r = adapter < 0 ? 0 : t.ranks ? min(max(t.ranks[adapter], 0), rmax) : rmax;
  const int units = (od + 31) / 32, per = (units + kCtas - 1) / kCtas, u1 = min((rank + 1) * per, units);
  __syncthreads();
  if (r == 0) {
    if (in_place) return;
    for (int k = 0; k < n; ++k) {
      const int64_t row = s_row[k];
      for (int o = rank * per * 32 + tid; o < min(u1 * 32, od); o += kThreads) t.out[row * t.out_row + o] = t.y[row * t.y_row + o];
    }
    return;
  }
  const int r16 = (r + 15) / 16 * 16, r32 = (r + 31) / 32 * 32, pitch = S::pitch(rmax);
  float *part = smem, *mine = part + S::kSplit * kRankPass * kTile;  // [split][rank of the pass][token]; [rank][token]
  uint32_t *terms = reinterpret_cast<uint32_t *>(mine + (rmax + 15) / 16 * 16 * kTile);  // [term][token][pitch]
  for (int k = tid; k < 2 * kTile * pitch; k += kThreads) terms[k] = 0;  // (ranks past r)

  // the first product, transposed: ranks x tokens over the CTA's columns
  {
    const int steps = (id + 31) / 32, share = (steps + kCtas - 1) / kCtas, end = min((rank + 1) * share, steps);
    const int tokens0 = warp % S::kGroups * S::kTokens, slot = warp / S::kGroups;
    const W *weights = static_cast<const W *>(t.a) + static_cast<int64_t>(adapter) * rmax * id;
    const size_t x_size = t.x_type == MMQ_DT_F32 ? 4 : 2;
    const unsigned char *row[S::kColumns];
    bool there[S::kColumns];
#pragma unroll
    for (int j = 0; j < S::kColumns; ++j) {
      const int of = s_row[tokens0 + 8 * j + g];
      there[j] = of >= 0;
      row[j] = static_cast<const unsigned char *>(t.x) + static_cast<int64_t>(max(of, 0)) * t.x_row * x_size;
    }
    for (int r0 = 0; r0 < r; r0 += kRankPass) {
      float acc[kRankPass / 16][S::kColumns][4] = {};
      if (tokens0 < n) {
        for (int step = rank * share + slot; step < end; step += S::kSplit) {
          const int k = 32 * step + 8 * c;
          const bool in = k < id;
          Terms x[S::kColumns][4];
          uint4 raw[kRankPass / 16][2];
#pragma unroll
          for (int m = 0; m < kRankPass / 16; ++m) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int of = r0 + 16 * m + 8 * h + g;
              raw[m][h] = in && of < r ? __ldg(reinterpret_cast<const uint4 *>(weights + static_cast<int64_t>(of) * id + k)) : zero4();
            }
          }
#pragma unroll
          for (int j = 0; j < S::kColumns; ++j) load_x(x[j], row[j], t.x_type, k, in && there[j]);
#pragma unroll
          for (int m = 0; m < kRankPass / 16; ++m) {
            if (r0 + 16 * m >= r) break;
            Weights8<W> p, q;
            p.set(raw[m][0]), q.set(raw[m][1]);
#pragma unroll
            for (int j = 0; j < S::kColumns; ++j) product<W>(acc[m][j], p, q, x[j]);
          }
        }
      }
      if (r0) __syncthreads();
#pragma unroll
      for (int m = 0; m < kRankPass / 16; ++m) {
        if (r0 + 16 * m >= r) break;
#pragma unroll
        for (int j = 0; j < S::kColumns; ++j) {
          float *to = part + (slot * kRankPass + 16 * m + g) * kTile + tokens0 + 8 * j + 2 * c;
          *reinterpret_cast<float2 *>(to) = make_float2(acc[m][j][0], acc[m][j][1]);
          *reinterpret_cast<float2 *>(to + 8 * kTile) = make_float2(acc[m][j][2], acc[m][j][3]);
        }
      }
      __syncthreads();
      const int here = min(r16 - r0, kRankPass) * kTile;
      for (int e = tid; e < here; e += kThreads) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < S::kSplit; ++k) s += part[k * kRankPass * kTile + e];
        mine[r0 * kTile + e] = s;
      }
    }
  }
  cluster_sync();
  // joined over the cluster: each CTA adds up a share of the pairs of ranks and
  // sends it to all
  const float scale = t.scales ? t.scales[adapter] : 1.0f;
  for (int e = rank * kThreads + tid; e < r16 / 2 * kTile; e += kCtas * kThreads) {
    const int pair = e / kTile, token = e % kTile;
    float s0 = 0.0f, s1 = 0.0f, v0[kCtas], v1[kCtas];
#pragma unroll
    for (int k = 0; k < kCtas; ++k) {
      const uint32_t from = mapa_shared(smem_addr(mine + 2 * pair * kTile + token), k);
      v0[k] = ld_cluster(from), v1[k] = ld_cluster(from + 4 * kTile);
    }
#pragma unroll
    for (int k = 0; k < kCtas; ++k) s0 += v0[k], s1 += v1[k];
    const Terms sum = split(s0 * scale, s1 * scale);
#pragma unroll
    for (int k = 0; k < kCtas; ++k) {
      const uint32_t to = mapa_shared(smem_addr(terms + token * pitch + pair), k);
      st_cluster(to, sum.h);
      st_cluster(to + 4 * kTile * pitch, sum.l);
    }
  }
  cluster_sync();

  // the second product: 32 output columns of a warp at a time, of which a lane
  // has four that lie together (rows g and g + 8 of two blocks of 16)
  const W *weights = static_cast<const W *>(t.b) + static_cast<int64_t>(adapter) * od * rmax;
  constexpr int kEach = kTile < 32 ? kTile / 8 : 4;  // columns of eight tokens at once
  const int columns = (n + 7) / 8;
  for (int u = rank * per + warp; u < u1; u += kWarps) {
    const int o = 32 * u + 4 * g;
    for (int j0 = 0; j0 < columns; j0 += kEach) {
      float4 y[kEach][2];
      int at[kEach][2];
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = 8 * (j0 + j) + 2 * c + h;
          at[j][h] = k < n ? s_row[k] : -1;
          y[j][h] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (at[j][h] < 0 || o >= od) continue;
          const float *from = t.y + static_cast<int64_t>(at[j][h]) * t.y_row + o;
          if (a.wide) {
            y[j][h] = __ldcs(reinterpret_cast<const float4 *>(from));
          } else {
            y[j][h].x = from[0];
            if (o + 1 < od) y[j][h].y = from[1];
            if (o + 2 < od) y[j][h].z = from[2];
            if (o + 3 < od) y[j][h].w = from[3];
          }
        }
      }
      float acc[2][kEach][4] = {};
      for (int r0 = 0; r0 < r32; r0 += 32) {
        const int k = r0 + 8 * c;
        Weights8<W> w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 raw = zero4();
          if (k < r && o + i < od) raw = __ldg(reinterpret_cast<const uint4 *>(weights + static_cast<int64_t>(o + i) * rmax + k));
          if (k < r && k + 8 > r) {  // columns past the rank
            uint32_t *v = &raw.x;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] &= k + 2 * e + 1 < r ? 0xffffffffu : k + 2 * e < r ? 0xffffu : 0u;
          }
          w[i].set(raw);
        }
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
          const uint32_t *from = terms + (8 * (j0 + j) + g) * pitch + k / 2;
          const uint4 h = *reinterpret_cast<const uint4 *>(from), l = *reinterpret_cast<const uint4 *>(from + kTile * pitch);
          const Terms x[4] = {{h.x, l.x}, {h.y, l.y}, {h.z, l.z}, {h.w, l.w}};
          product<W>(acc[0][j], w[0], w[1], x);
          product<W>(acc[1][j], w[2], w[3], x);
        }
      }
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (at[j][h] < 0 || o >= od) continue;
          const float4 v = make_float4(y[j][h].x + acc[0][j][h], y[j][h].y + acc[0][j][h + 2], y[j][h].z + acc[1][j][h], y[j][h].w + acc[1][j][h + 2]);
          float *to = t.out + static_cast<int64_t>(at[j][h]) * t.out_row + o;
          if (a.wide) {
            *reinterpret_cast<float4 *>(to) = v;
          } else {
            to[0] = v.x;
            if (o + 1 < od) to[1] = v.y;
            if (o + 2 < od) to[2] = v.z;
            if (o + 3 < od) to[3] = v.w;
          }
        }
      }
    }
  }
}

// Tokens of a tile: as many as an adapter has on the average, at the most 64,
// and few enough for two CTAs an SM.
int tile_of(int64_t ntok, int64_t nreq, int64_t nadapters) {
  const int64_t groups = std::max<int64_t>(1, std::min(nreq, nadapters + 1));
  const int64_t want = std::min((ntok + groups - 1) / groups, ntok * kCtas / (2 * 152));
  return want <= 8 ? 8 : want <= 16 ? 16 : want <= 32 ? 32 : 64;
}
int64_t most_tiles(int64_t ntok, int64_t nreq, int64_t nadapters) {
  return std::min(ntok, ntok / tile_of(ntok, nreq, nadapters) + std::min(nreq, nadapters + 1));
}

template <class W, int kTile>
cudaError_t launch_with(const LoraArgs &a, cudaStream_t s) {
  const size_t smem = Shape<kTile>::bytes(a.t.rank);
  const cudaError_t e = cudaFuncSetAttribute(lora_kernel<W, kTile>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int64_t tiles = most_tiles(a.t.ntok, a.t.nreq, a.t.nadapters);
  return launch_early(lora_kernel<W, kTile>, static_cast<unsigned>(tiles * kCtas), 1, kThreads, smem, s, a);
}

template <class W>
cudaError_t launch_of(const LoraArgs &a, cudaStream_t s) {
  switch (tile_of(a.t.ntok, a.t.nreq, a.t.nadapters)) {
    case 8: return launch_with<W, 8>(a, s);
    case 16: return launch_with<W, 16>(a, s);
    case 32: return launch_with<W, 32>(a, s);
    default: return launch_with<W, 64>(a, s);
  }
}

}  // namespace

int64_t lora_plan_words(int64_t ntok, int64_t nreq, int64_t nadapters) { return kHead + ntok + 3 * most_tiles(ntok, nreq, nadapters); }

cudaError_t launch_lora_plan(LoraPlanArgs a, cudaStream_t s) {
  a.tile = tile_of(a.ntok, a.nreq, a.nadapters);
  a.slots = 1;
  while (a.slots < a.nreq) a.slots *= 2;
  const size_t smem = 3 * static_cast<size_t>(a.slots) * 4;
  if (smem > 32 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(lora_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  const int64_t ctas = std::max<int64_t>(1, (a.ntok + kPlanTokens - 1) / kPlanTokens);
  return launch_early(lora_plan_kernel, static_cast<unsigned>(ctas), 1, kPlanThreads, smem, s, a);
}

cudaError_t launch_lora(LoraArgs a, cudaStream_t s) {
  const mmq_lora_args &t = a.t;
  auto whole = [](const void *p, int64_t row) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row % 4 == 0; };
  a.wide = t.od % 4 == 0 && whole(t.y, t.y_row) && whole(t.out, t.out_row);
  return t.type == MMQ_DT_F16 ? launch_of<__half>(a, s) : launch_of<__nv_bfloat16>(a, s);
}

}  // namespace mmq
