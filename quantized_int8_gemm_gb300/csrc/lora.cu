// lora.cu -- low-rank adapters of many requests beside a shared projection:
// out[t] = y[t] + s_a (x[t] A_a^T) B_a^T with the adapter a of token t's request.
//
// The plan sorts a step's tokens by adapter, once for all its projections, and
// cuts them into tiles of one adapter, so that x, y and out go through once and
// an adapter's weights are read once for each tile.
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
constexpr int kPlanTokens = 8192;  // tokens of a CTA
constexpr int kRequestBits = 13;                        // kMaxRequests
constexpr uint32_t kEmpty = 0xffffffffu, kNone = 1u << 18;

template <int kPlanThreads>
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
  int all = lane < kPlanThreads / 32 ? sm[lane] : 0;
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
// Latency bound: two rounds of reads, the sort, four sums over the CTA.
template <int kPlanThreads>
__global__ void __launch_bounds__(kPlanThreads) lora_plan_kernel(const __grid_constant__ LoraPlanArgs a) {
  // a.slots (a power of two) keys, as they come and sorted, then of the sorted ones'
  // the first row and the tokens and tiles before them; one more for the ends
  extern __shared__ __align__(16) uint32_t loaded[];
  __shared__ int s_warp[32];
  __shared__ int s_bad;
  uint32_t *keys = loaded + (a.few ? a.slots : 0);
  int *begins = reinterpret_cast<int *>(keys + a.slots), *tokens_before = begins + a.slots, *tiles_before = tokens_before + a.slots + 1;
  const int tid = threadIdx.x, nreq = static_cast<int>(a.nreq), ntok = static_cast<int>(a.ntok);
  griddep_wait();
  griddep_launch_dependents();
  if (tid == 0) s_bad = 0;
  __syncthreads();
  for (int i = tid; i < a.slots; i += kPlanThreads) {
    uint32_t key = kEmpty;
    if (i < nreq) {
      int begin = a.q_start[i], end = a.q_start[i + 1], id = a.adapters[i];
      if (end < begin || begin < 0) s_bad = 1, record_index(a.status);
      begin = min(max(begin, 0), ntok), end = min(max(end, 0), ntok);
      if (id < -1 || id >= a.nadapters) record_index(a.status), id = -1;
      if (end > begin) key = (id < 0 ? kNone : static_cast<uint32_t>(id)) << kRequestBits | static_cast<uint32_t>(i);
    }
    loaded[i] = key;
  }
  __syncthreads();
  if (a.few) {
    // a key's place is the number of smaller ones (no two are alike but empty
    // ones, which follow in the order that they came)
    if (tid < a.slots) {
      const uint32_t mine = loaded[tid];
      int place = 0;
      if (a.slots < 4) {
        for (int i = 0; i < a.slots; ++i) place += loaded[i] < mine || (loaded[i] == mine && i < tid);
      } else if (mine == kEmpty) {
        for (int i = 0; i < a.slots; ++i) place += loaded[i] < mine || i < tid;
      } else {
        for (int i = 0; i < a.slots; i += 4) {
          const uint4 k = *reinterpret_cast<const uint4 *>(loaded + i);
          place += (k.x < mine) + (k.y < mine) + (k.z < mine) + (k.w < mine);
        }
      }
      keys[place] = mine;
    }
    __syncthreads();
  } else {
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
  }
  // (each thread has the keys from tid * per on)
  const int per = (a.slots + kPlanThreads - 1) / kPlanThreads, i0 = min(tid * per, a.slots), i1 = min(i0 + per, a.slots);
  auto adapter = [&](int i) { return keys[i] >> kRequestBits; };
  int sum = 0, total, none;
  for (int i = i0; i < i1; ++i) {
    int begin = 0, end = 0;
    if (keys[i] != kEmpty) {
      const int b = static_cast<int>(keys[i] & ((1u << kRequestBits) - 1));
      begin = min(max(a.q_start[b], 0), ntok), end = min(max(a.q_start[b + 1], 0), ntok);
    }
    begins[i] = begin, tokens_before[i] = sum;  // (of the thread's, for now)
    sum += end - begin;
  }
  const int at = plan_exclusive<kPlanThreads>(sum, total, s_warp, false);
  int first = 0;  // largest begin of a group up to here
  for (int i = i0; i < i1; ++i) {
    tokens_before[i] += at;
    if (i == 0 || adapter(i - 1) != adapter(i)) first = tokens_before[i];
  }
  if (tid == 0) tokens_before[a.slots] = total;
  const int before = plan_exclusive<kPlanThreads>(first, none, s_warp, true);  // (and the CTA's threads meet)
  auto tiles_of = [&](int i, int &start) {  // tiles of the group that ends with key i
    if (i == 0 || adapter(i - 1) != adapter(i)) start = tokens_before[i];
    const bool last = keys[i] != kEmpty && (i + 1 == a.slots || adapter(i + 1) != adapter(i));
    return last ? (tokens_before[i + 1] - start + a.tile - 1) / a.tile : 0;
  };
  int start = before, tiles = 0, all_tiles;
  for (int i = i0; i < i1; ++i) tiles += tiles_of(i, start);
  int tile = plan_exclusive<kPlanThreads>(tiles, all_tiles, s_warp, false);
  start = before;
  const bool bad = s_bad;
  int32_t *order = a.plan + kHead, *list = order + ntok;
  for (int i = i0; i < i1; ++i) {
    tiles_before[i] = tile;
    const int mine = tiles_of(i, start);
    if (mine && !bad && blockIdx.x == 0) {
      const int id = adapter(i) == kNone ? -1 : static_cast<int>(adapter(i)), end = tokens_before[i + 1];
      if (mine <= 4) {  // (groups of many tiles: by all threads, below)
        for (int k = 0; k < mine; ++k) {
          int32_t *to = list + 3 * (tile + k);
          to[0] = id, to[1] = start + k * a.tile, to[2] = min(a.tile, end - start - k * a.tile);
        }
      }
      if (id < 0) a.plan[1] = tile;  // (the tiles without an adapter stand last)
      else if (tile + mine == all_tiles) a.plan[1] = all_tiles;
    }
    tile += mine;
  }
  if (tid == 0) tiles_before[a.slots] = all_tiles;
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0) {
    a.plan[0] = bad ? 0 : all_tiles;
    if (bad || all_tiles == 0) a.plan[1] = 0;
  }
  if (bad) return;
  const int p0 = static_cast<int>(blockIdx.x) * kPlanTokens, p1 = min(p0 + kPlanTokens, total);
  for (int p = p0 + tid; p < p1; p += kPlanThreads) {
    const int i = last_not_above(tokens_before, a.slots, p);  // (keys without tokens stand last, behind every token)
    order[p] = begins[i] + (p - tokens_before[i]);
  }
  for (int k = static_cast<int>(blockIdx.x) * kPlanThreads + tid; k < all_tiles; k += static_cast<int>(gridDim.x) * kPlanThreads) {
    const int i = last_not_above(tiles_before, a.slots, k);  // the group's last key
    if (tiles_before[i + 1] - tiles_before[i] <= 4) continue;
    int lo = -1, hi = i;  // its first one
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (adapter(mid) == adapter(i)) hi = mid;
      else lo = mid;
    }
    const int begin = tokens_before[hi] + (k - tiles_before[i]) * a.tile;
    list[3 * k] = adapter(i) == kNone ? -1 : static_cast<int>(adapter(i));
    list[3 * k + 1] = begin;
    list[3 * k + 2] = min(a.tile, tokens_before[i + 1] - begin);
  }
}

// ---------------------------------------------------------------- products
constexpr int kCtas = 8, kThreads = 256, kWarps = kThreads / 32;
constexpr int kStages = 3;

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// 16 bytes to shared memory in the background, or 16 zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ float4 lds4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }

// D += A B, 16 x 16 by 16 x 8, bf16 in, fp32 sums.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The tensor cores cut what they add up off at the last bit of the largest: long
// sums go on in fp32 proper, from sums of 32 columns (18944 columns at rank 32:
// 1.6e-6 off in one chain, 2.3e-7 so; fp32 products by a library 6e-7).
__device__ __forceinline__ void add(float (&sum)[4], const float (&x)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] += x[e];
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// x -= a, y -= b, in one instruction (as a product with -1, which is exact).
__device__ __forceinline__ void subtract(float &x, float &y, float a, float b) {
  asm("{\n\t.reg .b64 m, v, d;\n\t"
      "mov.b64 m, {%4, %4};\n\tmov.b64 v, {%2, %3};\n\tmov.b64 d, {%0, %1};\n\t"
      "fma.rn.f32x2 d, v, m, d;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b), "f"(-1.0f));
}

// A pair of numbers as three bf16 terms: each is rounded to nearest, so that
// what is left after it is at most 2^-9 of what it stands for, and after the
// third nothing of an fp32 number's 24 bits.  (With two terms, 2^-18 off, the
// outputs were 1.2 to 2.9e-6 from the 64-bit ones; fp32 sums are 2 to 10e-7 off.)
constexpr int kTerms = 3;
struct Terms {
  uint32_t w[kTerms];
};
__device__ __forceinline__ Terms split(float x, float y) {
  Terms t;
#pragma unroll
  for (int i = 0; i < kTerms; ++i) {
    t.w[i] = pack(x, y);
    if (i + 1 < kTerms) subtract(x, y, low(t.w[i]), high(t.w[i]));
  }
  return t;
}

// Eight numbers of a row of weights, as bf16: exactly, fp16 weights as two terms.
template <class W>
struct Weights8;
template <>
struct Weights8<__nv_bfloat16> {
  static constexpr int kParts = 1;
  uint32_t w[1][4];
  __device__ __forceinline__ void set(uint4 r) { w[0][0] = r.x, w[0][1] = r.y, w[0][2] = r.z, w[0][3] = r.w; }
};
template <>
struct Weights8<__half> {
  static constexpr int kParts = 2;
  uint32_t w[2][4];
  __device__ __forceinline__ void set(uint4 r) {
    const uint32_t v[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v[i]));
      w[0][i] = pack(f.x, f.y);
      w[1][i] = pack(f.x - low(w[0][i]), f.y - high(w[0][i]));
    }
  }
};

// The lane's eight columns (two steps of 16) of rows p and q of weights by
// those of eight rows of terms.  Which column is which within the 32 does not
// matter as long as both sides agree: lane quarter c has columns 8c .. 8c + 7,
// which lie together in memory.  Small products first; those of terms that
// together are below 2^-24 are left out.
template <class W>
__device__ __forceinline__ void product(float (&d)[4], const Weights8<W> &p, const Weights8<W> &q, const Terms (&x)[4]) {
#pragma unroll
  for (int k = 0; k < 4; k += 2) {
#pragma unroll
    for (int order = kTerms - 1; order >= 0; --order) {
#pragma unroll
      for (int i = Weights8<W>::kParts - 1; i >= 0; --i) {
        const int j = order - i;
        if (j < 0) continue;
        mma(d, p.w[i][k], q.w[i][k], p.w[i][k + 1], q.w[i][k + 1], x[k].w[j], x[k + 1].w[j]);
      }
    }
  }
}

// An operand of 16 rows of weights by 16 columns, as the tensor cores take it: a
// lane's pairs of columns of rows p and q, in this order, as bf16 terms.  The
// registers of one have to lie together: where they are those that a 16-byte
// load has filled, each product copied them first (5 moves a product), so
// they are made once.
template <class W>
struct Operand {
  static constexpr int kParts = Weights8<W>::kParts;
  uint32_t w[kParts][4];
  // from pairs as loaded; zero: a 0 that the compiler does not know of
  __device__ __forceinline__ void set(uint32_t p0, uint32_t q0, uint32_t p1, uint32_t q1, uint32_t zero) {
    const uint32_t v[4] = {p0, q0, p1, q1};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kParts == 1) {
        w[0][i] = v[i] ^ zero;
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v[i]));
        w[0][i] = pack(f.x, f.y);
        w[kParts - 1][i] = pack(f.x - low(w[0][i]), f.y - high(w[0][i]));
      }
    }
  }
};
template <class W>
__device__ __forceinline__ void product(float (&d)[4], const Operand<W> &a, const Terms &x0, const Terms &x1) {
#pragma unroll
  for (int order = kTerms - 1; order >= 0; --order) {
#pragma unroll
    for (int i = Operand<W>::kParts - 1; i >= 0; --i)
      if (order - i >= 0) mma(d, a.w[i][0], a.w[i][1], a.w[i][2], a.w[i][3], x0.w[order - i], x1.w[order - i]);
  }
}

__device__ __forceinline__ uint4 zero4() { return make_uint4(0, 0, 0, 0); }

// Eight numbers of x as terms, from 16 or 32 bytes (a and, if fp32, b).
template <bool kFp32>
__device__ __forceinline__ void split8(Terms (&out)[4], uint4 a, uint4 b, int x_type) {
  if constexpr (kFp32) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = split(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    return;
  }
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = x_type == MMQ_DT_F16 ? __half22float2(*reinterpret_cast<const __half2 *>(&w[i])) : make_float2(low(w[i]), high(w[i]));
    out[i] = split(f.x, f.y);
  }
}

// How a CTA's warps share the first product: over groups of tokens and, within
// a piece of x's columns, over 32 columns each.
template <int kTile>
struct Shape {
  static constexpr int kTokens = kTile == 64 ? 16 : 8, kGroups = kTile / kTokens, kSplit = kWarps / kGroups, kColumns = kTokens / 8;
  static constexpr int kPiece = 32 * kSplit;  // columns of a stage
};
// The terms of the joined sums, of a tile: [term][token][pitch] words, a token's
// ranks together, rows 16 words from a multiple of 32 apart (eight lanes of a
// 16-byte read then touch every bank once).
__host__ __device__ constexpr int pitch_of(int rank) { return rank <= 32 ? 16 : rank <= 64 ? 48 : 80; }
__host__ __device__ constexpr int up16(int rank) { return (rank + 15) / 16 * 16; }

__host__ __device__ constexpr int few_front(int rank) {  // bytes of the partial sums or the terms of eight tokens
  const int part = 4 * kWarps * 64 * 8, terms = 4 * kTerms * 8 * pitch_of(rank);
  return part > terms ? part : terms;
}

// A tile of the plan; n = 0 behind the last one (of those with an adapter, if
// only they are wanted), whose entries the plan has room for but nobody wrote.
struct Tile {
  int adapter, first, n, rank;
  float scale;
};
__device__ __forceinline__ Tile tile_at(const mmq_lora_args &t, int tile, bool adapters_only) {
  const int32_t *entry = t.plan + kHead + t.ntok + 3 * static_cast<int64_t>(tile);
  Tile k;
  k.adapter = entry[0], k.first = entry[1], k.n = entry[2];
  if (tile >= t.plan[adapters_only ? 1 : 0]) return {-1, 0, 0, 0, 1.0f};
  k.rank = k.adapter < 0 ? 0 : t.ranks ? min(max(t.ranks[k.adapter], 0), t.rank) : t.rank;
  k.scale = t.scales && k.adapter >= 0 ? t.scales[k.adapter] : 1.0f;
  return k;
}

// Rows of a tile without an adapter (or of rank 0): out = y in columns [o0, o1).
__device__ __forceinline__ void copy_rows(const LoraArgs &a, const int *s_row, int n, int o0, int o1) {
  const mmq_lora_args &t = a.t;
  constexpr int kEach = 8;
  const int width = a.wide ? (o1 - o0) / 4 : o1 - o0, items = n * width;
  for (int i0 = threadIdx.x; i0 < items; i0 += kEach * kThreads) {
    float4 v[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int i = i0 + u * kThreads;
      if (i >= items) continue;
      const float *from = t.y + s_row[i / width] * t.y_row + o0 + (a.wide ? 4 : 1) * (i % width);
      if (a.wide) v[u] = __ldcs(reinterpret_cast<const float4 *>(from));
      else v[u].x = *from;
    }
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int i = i0 + u * kThreads;
      if (i >= items) continue;
      float *to = t.out + s_row[i / width] * t.out_row + o0 + (a.wide ? 4 : 1) * (i % width);
      if (a.wide) *reinterpret_cast<float4 *>(to) = v[u];
      else *to = v[u].x;
    }
  }
}

// Partial sums of the warps of a CTA, [split][rank of the pass][token], added up
// in their order into the CTA's, [rank][token].
template <int kTile, int kPass>
__device__ __forceinline__ void add_up(float *mine, const float *part, int r0, int r16) {
  using S = Shape<kTile>;
  for (int e = threadIdx.x; e < min(r16 - r0, kPass) * kTile; e += kThreads) {
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < S::kSplit; ++k) s += part[k * kPass * kTile + e];
    mine[r0 * kTile + e] = s;
  }
}
template <int kTile, int kPass, int kColumns>
__device__ __forceinline__ void put_part(float *part, const float (&acc)[kPass / 16][kColumns][4], int ranks, int slot, int tokens0) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int m = 0; m < kPass / 16; ++m) {
    if (16 * m >= ranks) break;
#pragma unroll
    for (int j = 0; j < kColumns; ++j) {
      float *to = part + (slot * kPass + 16 * m + g) * kTile + tokens0 + 8 * j + 2 * c;
      *reinterpret_cast<float2 *>(to) = make_float2(acc[m][j][0], acc[m][j][1]);
      *reinterpret_cast<float2 *>(to + 8 * kTile) = make_float2(acc[m][j][2], acc[m][j][3]);
    }
  }
}
// Ranks 2 pair and 2 pair + 1 of a token, joined over the cluster in the CTAs' order.
template <int kTile>
__device__ __forceinline__ Terms joined(const float *mine, int pair, int token, float scale) {
  float s0 = 0.0f, s1 = 0.0f, v0[kCtas], v1[kCtas];
#pragma unroll
  for (int k = 0; k < kCtas; ++k) {
    const uint32_t from = mapa_shared(smem_addr(mine + 2 * pair * kTile + token), k);
    v0[k] = ld_cluster(from), v1[k] = ld_cluster(from + 4 * kTile);
  }
#pragma unroll
  for (int k = 0; k < kCtas; ++k) s0 += v0[k], s1 += v1[k];
  return split(s0 * scale, s1 * scale);
}

// Four output columns o .. o + 3 of a token.
__device__ __forceinline__ float4 load_y(const LoraArgs &a, int row, int o) {
  float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const int od = static_cast<int>(a.t.od);
  if (row < 0 || o >= od) return y;
  const float *from = a.t.y + row * a.t.y_row + o;
  if (a.wide) return __ldcs(reinterpret_cast<const float4 *>(from));
  y.x = from[0];
  if (o + 1 < od) y.y = from[1];
  if (o + 2 < od) y.z = from[2];
  if (o + 3 < od) y.w = from[3];
  return y;
}
__device__ __forceinline__ void store_out(const LoraArgs &a, int row, int o, float4 v) {
  const int od = static_cast<int>(a.t.od);
  if (row < 0 || o >= od) return;
  float *to = a.t.out + row * a.t.out_row + o;
  if (a.wide) {
    *reinterpret_cast<float4 *>(to) = v;
    return;
  }
  to[0] = v.x;
  if (o + 1 < od) to[1] = v.y;
  if (o + 2 < od) to[2] = v.z;
  if (o + 3 < od) to[3] = v.w;
}
template <int kEach>
__device__ __forceinline__ float4 sum_of(const float (&acc)[2][kEach][4], int j, int h, const float4 &y) {
  return make_float4(y.x + acc[0][j][h], y.y + acc[0][j][h + 2], y.z + acc[1][j][h], y.w + acc[1][j][h + 2]);
}

// ---------------------------------------------------------------- few tokens: one kernel
// A cluster takes a tile of eight tokens: each CTA multiplies an eighth of x's
// columns by A, every CTA adds up the eight sums in their order, and each writes
// an eighth of the output columns.  HBM bound by the adapters with many tiles,
// latency bound with few.  Up to rank 32 two pieces of A and what the second
// product needs first are asked for ahead, in 118 registers (127 with fp16 weights; one token, 3584 ->
// 4608, rank 16: 8.4 -> 6.4 us); beyond, three CTAs an SM hide more than reads
// ahead in two do (96 tokens of 50 adapters of rank 64: 22.1 against 24.6 us), and
// B comes to L2 during the first product.  The 80 registers of three CTAs an SM do not
// hold everything: 68 bytes a thread are spilled (36 with fp16 weights).
constexpr int kFew = 8;  // tokens
template <class W, int kPass>  // ranks whose sums a warp holds at once
__global__ void __launch_bounds__(kThreads, kPass == 32 ? 2 : 3) __cluster_dims__(kCtas, 1, 1) lora_few_kernel(const __grid_constant__ LoraArgs a) {
  constexpr int kHold = kPass / 32;  // steps of 32 ranks of the second product
  constexpr bool kAhead = kPass == 32;  // (registers for two)
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int s_row[kFew];
  const mmq_lora_args &t = a.t;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int rank = static_cast<int>(cluster_ctarank()), tile = static_cast<int>(blockIdx.x / kCtas);
  griddep_wait();
  griddep_launch_dependents();
  const bool in_place = t.y == t.out;
  const Tile k_tile = tile_at(t, tile, in_place);
  if (k_tile.n == 0) return;  // (the whole cluster)
  const int n = k_tile.n, r = k_tile.rank;
  if (tid < kFew) s_row[tid] = tid < n ? t.plan[kHead + k_tile.first + tid] : -1;
  const int id = static_cast<int>(t.id), od = static_cast<int>(t.od), rmax = t.rank;
  const int units = (od + 31) / 32, u0 = units * rank / kCtas, u1 = units * (rank + 1) / kCtas;
  if (r == 0) {
    __syncthreads();
    if (!in_place) copy_rows(a, s_row, n, min(32 * u0, od), min(32 * u1, od));
    return;
  }
  const W *down = static_cast<const W *>(t.a) + static_cast<int64_t>(k_tile.adapter) * rmax * id;
  const W *up = static_cast<const W *>(t.b) + static_cast<int64_t>(k_tile.adapter) * od * rmax;
  const int r16 = up16(r), pitch = pitch_of(rmax);
  // partial sums of the warps, later the terms; behind them the CTA's sums
  float *part = reinterpret_cast<float *>(smem), *mine = reinterpret_cast<float *>(smem + few_front(rmax));
  uint32_t *terms = reinterpret_cast<uint32_t *>(smem);
  // The first product: the warps take 32 columns at a time.
  const int steps = (id + 31) / 32, s0 = steps * rank / kCtas + warp, s1 = steps * (rank + 1) / kCtas;
  const int x_size = t.x_type == MMQ_DT_F32 ? 4 : 2;
  struct Piece {
    uint4 w[kPass / 16][2], lo, hi;
  };
  auto fetch_w = [&](Piece &p, int step, int r0) {
    const int k = 32 * step + 8 * c;
#pragma unroll
    for (int m = 0; m < kPass / 16; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = r0 + 16 * m + 8 * h + g;
        p.w[m][h] = k < id && at < r ? __ldg(reinterpret_cast<const uint4 *>(down + static_cast<int64_t>(at) * id + k)) : zero4();
      }
  };
  Piece now;
  if (kAhead && s0 < s1) fetch_w(now, s0, 0);
  if (tid < 32) {
    // the adapter is most of what is read: the second product's part of it comes
    // to L2 during the first
    const char *from = reinterpret_cast<const char *>(up + static_cast<int64_t>(32 * u0) * rmax);
    const int64_t bytes = static_cast<int64_t>(min(32 * u1, od) - 32 * u0) * rmax * 2;
    for (int64_t at = tid * 4096; at < bytes; at += 32 * 4096)
      bulk_prefetch_l2(from + at, static_cast<uint32_t>(min(bytes - at, static_cast<int64_t>(4096))));
  }
  __syncthreads();
  const int of = s_row[g];
  const unsigned char *row = static_cast<const unsigned char *>(t.x) + max(of, 0) * t.x_row * x_size;
  auto fetch_x = [&](Piece &p, int step) {
    const int k = 32 * step + 8 * c;
    p.lo = p.hi = zero4();
    if (k >= id || of < 0) return;
    p.lo = __ldg(reinterpret_cast<const uint4 *>(row + static_cast<int64_t>(k) * x_size));
    if (x_size == 4) p.hi = __ldg(reinterpret_cast<const uint4 *>(row + static_cast<int64_t>(k) * x_size) + 1);
  };
  if (kAhead && s0 < s1) fetch_x(now, s0);
  uint4 ahead[kHold][4];  // of the second product: the weights, and y
  float4 y[2];
  auto fetch_up = [&](uint4 (&w)[4], int u, int r0) {
    const int k = r0 + 8 * c, o = 32 * u + 4 * g;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = k < r && o + i < od ? __ldg(reinterpret_cast<const uint4 *>(up + static_cast<int64_t>(o + i) * rmax + k)) : zero4();
  };
  auto fetch_unit = [&](int u) {
    if (u >= u1) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) y[h] = load_y(a, s_row[2 * c + h], 32 * u + 4 * g);
#pragma unroll
    for (int s = 0; s < kHold; ++s) fetch_up(ahead[s], u, 32 * s);
  };
  for (int r0 = 0; r0 < r; r0 += kPass) {
    const int ranks = min(r - r0, kPass);
    float acc[kPass / 16][1][4] = {};
    auto multiply = [&](const Piece &p) {
      Terms xt[4];
      if (x_size == 4) split8<true>(xt, p.lo, p.hi, t.x_type);
      else split8<false>(xt, p.lo, p.hi, t.x_type);
#pragma unroll
      for (int m = 0; m < kPass / 16; ++m) {
        if (16 * m >= ranks) break;
        Weights8<W> u, v;
        u.set(p.w[m][0]), v.set(p.w[m][1]);
        float here[4] = {};
        product<W>(here, u, v, xt);
        add(acc[m][0], here);
      }
    };
    for (int step = s0; step < s1; step += kWarps) {
      if constexpr (kAhead) {
        Piece next;
        const bool more = step + kWarps < s1;
        if (more) fetch_w(next, step + kWarps, r0), fetch_x(next, step + kWarps);
        multiply(now);
        if (more) now = next;
      } else {
        fetch_w(now, step, r0), fetch_x(now, step);
        multiply(now);
      }
    }
    if (kAhead && r0 + kPass >= r) fetch_unit(u0 + warp);
    if (r0) __syncthreads();
    put_part<kFew, kPass>(part, acc, ranks, warp, 0);
    __syncthreads();
    add_up<kFew, kPass>(mine, part, r0, r16);
  }
  cluster_sync();  // (part makes room, too)
  for (int e = tid; e < r16 / 2 * kFew; e += kThreads) {
    const int pair = e / kFew, token = e % kFew;
    const Terms sum = joined<kFew>(mine, pair, token, k_tile.scale);
#pragma unroll
    for (int i = 0; i < kTerms; ++i) terms[(i * kFew + token) * pitch + pair] = sum.w[i];
  }
  const int left = ((r + 31) / 32 * 32 - r16) / 2;  // pairs of ranks past r, of the last step: 0 or 8
  for (int e = tid; e < kTerms * kFew * left; e += kThreads) terms[e / left * pitch + r16 / 2 + e % left] = 0;
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");  // (a CTA stays until the others have read its sums)
  __syncthreads();
  for (int u = u0 + warp; u < u1; u += kWarps) {
    const int o = 32 * u + 4 * g;
    if (!kAhead) fetch_unit(u);
    float acc[2][1][4] = {};
    auto multiply = [&](uint4 (&raw)[4], int r0) {
      const int k = r0 + 8 * c;
      Weights8<W> w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (k < r && k + 8 > r) {  // columns past the rank
          uint32_t *v = &raw[i].x;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] &= k + 2 * e + 1 < r ? 0xffffffffu : k + 2 * e < r ? 0xffffu : 0u;
        }
        w[i].set(raw[i]);
      }
      Terms x[4];
#pragma unroll
      for (int i = 0; i < kTerms; ++i) {
        const uint4 v = *reinterpret_cast<const uint4 *>(terms + (i * kFew + g) * pitch + k / 2);
        x[0].w[i] = v.x, x[1].w[i] = v.y, x[2].w[i] = v.z, x[3].w[i] = v.w;
      }
      product<W>(acc[0][0], w[0], w[1], x);
      product<W>(acc[1][0], w[2], w[3], x);
    };
#pragma unroll
    for (int s = 0; s < kHold; ++s)
      if (32 * s < r) multiply(ahead[s], 32 * s);
    for (int r0 = 32 * kHold; r0 < r; r0 += 32) {
      uint4 raw[4];
      fetch_up(raw, u, r0);
      multiply(raw, r0);
    }
    float4 out[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) out[h] = sum_of<1>(acc, 0, h, y[h]);
    if (kAhead) fetch_unit(u + kWarps);
#pragma unroll
    for (int h = 0; h < 2; ++h) store_out(a, s_row[2 * c + h], o, out[h]);
  }
  asm volatile("barrier.cluster.wait;" ::: "memory");
}

// ---------------------------------------------------------------- more tokens: two kernels
// With prompts the rows of x, y and out are most of what is read and written,
// and the two products have little in common in their shares: tiles by columns
// of x, joined; tiles by columns of out.  In one kernel (each CTA an eighth of
// both) a tile's CTAs lived 60 us and the last, partly filled wave as long as the
// first (2158 tokens, 3584 to 18944: 128 us).
//
// The first product: a cluster takes a tile, each CTA an eighth of x's columns,
// through stages of shared memory; the sums are joined through the cluster's
// shared memory and left as terms.  (Tiles of 64 with fp32 x up to rank 32 spill 16 bytes a
// thread into 80 registers, 32 with fp16 weights.)
template <class W, int kTile, bool kFp32, int kPass>
__global__ void __launch_bounds__(kThreads, kPass == 32 ? 3 : 2) __cluster_dims__(kCtas, 1, 1) lora_down_kernel(const __grid_constant__ LoraArgs a) {
  using S = Shape<kTile>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int s_row[kTile];
  const mmq_lora_args &t = a.t;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int rank = static_cast<int>(cluster_ctarank()), tile = static_cast<int>(blockIdx.x / kCtas);
  griddep_wait();
  griddep_launch_dependents();
  const Tile k_tile = tile_at(t, tile, true);
  if (k_tile.n == 0) return;  // (the whole cluster)
  const int n = k_tile.n, r = k_tile.rank;
  if (r == 0) return;
  if (tid < kTile) s_row[tid] = tid < n ? t.plan[kHead + k_tile.first + tid] : -1;
  const int id = static_cast<int>(t.id), rmax = t.rank, r16 = up16(r), stage_ranks = min(up16(rmax), kPass);
  constexpr int kSize = kFp32 ? 4 : 2, kXRow = S::kPiece * kSize, kWRow = S::kPiece * 2, kXStage = kTile * kXRow;  // bytes
  const uint32_t stage_bytes = kXStage + stage_ranks * kWRow;
  float *part = reinterpret_cast<float *>(smem), *mine = reinterpret_cast<float *>(smem + a.front);
  const int pieces = (id + S::kPiece - 1) / S::kPiece, p0 = pieces * rank / kCtas, p1 = pieces * (rank + 1) / kCtas;
  const int tokens0 = warp % S::kGroups * S::kTokens, slot = warp / S::kGroups;
  const W *down = static_cast<const W *>(t.a) + static_cast<int64_t>(k_tile.adapter) * rmax * id;
  const unsigned char *x = static_cast<const unsigned char *>(t.x);
  // Pieces of x and of the weights in 16-byte chunks, moved about by their row so
  // that the rows of a read do not meet in a bank.
  auto x_at = [](int row, int chunk) { return static_cast<uint32_t>(row * kXRow + ((chunk ^ (kFp32 ? (row & 3) << 1 : row & 7)) << 4)); };
  auto w_at = [](int row, int chunk) { return static_cast<uint32_t>(kXStage + row * kWRow + ((chunk ^ (row & 7)) << 4)); };
  __syncthreads();
  // This thread's copies of every stage: rows kXRows apart of one chunk of x,
  // rows kWRows apart of one of the weights.
  constexpr int kXChunks = kXRow / 16, kXRows = kThreads / kXChunks, kXCopies = kTile / kXRows;
  constexpr int kWChunks = kWRow / 16, kWRows = kThreads / kWChunks, kWCopies = kPass / kWRows;
  static_assert(kXCopies * kXRows == kTile && kWCopies * kWRows == kPass, "a stage is whole rounds of the threads");
  const int x_row = tid / kXChunks, x_k = tid % kXChunks * (16 / kSize), w_row = tid / kWChunks, w_k = tid % kWChunks * 8;
  const unsigned char *x_from[kXCopies];
  bool x_there[kXCopies];
#pragma unroll
  for (int u = 0; u < kXCopies; ++u) {
    const int of = s_row[x_row + u * kXRows];
    x_there[u] = of >= 0;
    x_from[u] = x + (max(of, 0) * t.x_row + x_k) * kSize;
  }
  const uint32_t base = smem_addr(smem), x_to = base + x_at(x_row, tid % kXChunks), w_to = base + w_at(w_row, tid % kWChunks);
  static_assert(kXRows % (kFp32 ? 4 : 8) == 0 && kWRows % 8 == 0, "a thread's rows are moved about alike");
  // and what it reads of one: of x the pairs of columns 2 c, 2 c + 8, 2 c + 16 and
  // 2 c + 24 of the 32; of the weights a row for the others' operands
  uint32_t x_read[4], w_read[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = (32 * slot + 8 * i + 2 * c) * kSize;
    x_read[i] = base + x_at(tokens0 + g, at >> 4) + (at & 15);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) w_read[i] = base + w_at(lane & 15, 4 * slot + 2 * i + (lane >> 4));
  for (int r0 = 0; r0 < r; r0 += kPass) {
    const int ranks = min(r - r0, kPass), rows = min(r16 - r0, kPass);
    float acc[kPass / 16][S::kColumns][4] = {};
    const W *w_from = down + static_cast<int64_t>(r0 + w_row) * id + w_k;
    auto load = [&](int p, uint32_t stage) {
      const int k0 = p * S::kPiece;
      const bool x_in = k0 + x_k < id, w_in = k0 + w_k < id;
#pragma unroll
      for (int u = 0; u < kXCopies; ++u)
        copy16(x_to + stage + u * kXRows * kXRow, x_from[u] + static_cast<int64_t>(x_in ? k0 : 0) * kSize, x_in && x_there[u]);
#pragma unroll
      for (int u = 0; u < kWCopies; ++u) {
        const int row = w_row + u * kWRows;
        if (row >= rows) break;
        const bool there = w_in && row < ranks;
        copy16(w_to + stage + u * kWRows * kWRow, there ? w_from + static_cast<int64_t>(u * kWRows) * id + k0 : down, there);
      }
    };
    uint32_t to = 0, from = 0;  // stages
#pragma unroll
    for (int p = 0; p < kStages - 1; ++p) {
      if (p0 + p < p1) load(p0 + p, to);
      copies_commit();
      to += stage_bytes;
    }
    for (int p = p0; p < p1; ++p) {
      copies_wait<kStages - 2>();
      __syncthreads();
      if (p + kStages - 1 < p1) load(p + kStages - 1, to);
      copies_commit();
      to = to == (kStages - 1) * stage_bytes ? 0 : to + stage_bytes;
      const uint32_t now = from;
      from = from == (kStages - 1) * stage_bytes ? 0 : from + stage_bytes;
      if (tokens0 >= n) continue;
      Terms xt[S::kColumns][4];
#pragma unroll
      for (int j = 0; j < S::kColumns; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t at = x_read[i] + now + 8 * j * kXRow;
          float2 v;
          if constexpr (kFp32) {
            asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
          } else {
            uint32_t w;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(at) : "memory");
            v = t.x_type == MMQ_DT_F16 ? __half22float2(*reinterpret_cast<const __half2 *>(&w)) : make_float2(low(w), high(w));
          }
          xt[j][i] = split(v.x, v.y);
        }
#pragma unroll
      for (int m = 0; m < kPass / 16; ++m) {
        if (16 * m >= ranks) break;
        float here[S::kColumns][4] = {};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t v[4];
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                       : "r"(w_read[i] + now + 16 * m * kWRow)
                       : "memory");
          Operand<W> w;
          w.set(v[0], v[1], v[2], v[3], 0);
#pragma unroll
          for (int j = 0; j < S::kColumns; ++j) product<W>(here[j], w, xt[j][2 * i], xt[j][2 * i + 1]);
        }
#pragma unroll
        for (int j = 0; j < S::kColumns; ++j) add(acc[m][j], here[j]);
      }
    }
    copies_wait<0>();
    __syncthreads();
    put_part<kTile, kPass>(part, acc, ranks, slot, tokens0);
    __syncthreads();
    add_up<kTile, kPass>(mine, part, r0, r16);
    __syncthreads();  // (part makes room)
  }
  cluster_sync();
  const int pitch = pitch_of(rmax), pairs = (r + 31) / 32 * 16;  // (zeros up to whole steps of the second product)
  uint32_t *to = a.terms + static_cast<int64_t>(tile) * kTerms * kTile * pitch;
  for (int e = rank * kThreads + tid; e < pairs * kTile; e += kCtas * kThreads) {
    const int pair = e % pairs, token = e / pairs;
    Terms sum = {};
    if (2 * pair < r16) sum = joined<kTile>(mine, pair, token, k_tile.scale);
#pragma unroll
    for (int i = 0; i < kTerms; ++i) to[(i * kTile + token) * pitch + pair] = sum.w[i];
  }
  // (a CTA stays until the others have read its sums)
  asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait;" ::: "memory");
}

// The second product: a CTA takes a.columns output columns of a tile, a warp 32 of
// them and 16 tokens at a time, the next ones' y on its way.  The weights of 32
// columns stay in registers for the tile's tokens, up to rank 64 (32 in fp16).
// HBM bound (y in, out out).
// Weights of up to 32 ranks in bf16 leave registers for four CTAs an SM, which hide
// more of each other than longer stretches of a row save (64 tiles of 18944 columns,
// both projections: four CTAs with 256 columns 234 us, 512 240, 768 259; two with
// 512 250, 768 239, 1024 247; three with 512 241); 4 bytes a thread are spilled for it.
template <class W>
__host__ __device__ constexpr int up_ctas(int pitch) { return pitch == 16 && Weights8<W>::kParts == 1 ? 4 : 2; }
__host__ __device__ constexpr int y_pieces(int ctas) { return ctas == 4 ? 2 : 3; }  // of y, on their way or in use
constexpr int kEach = 2;  // columns of eight tokens at once (four gained nothing, and spilled)
template <class W, int kTile, int kPitch>
__global__ void __launch_bounds__(kThreads, up_ctas<W>(kPitch)) lora_up_kernel(const __grid_constant__ LoraArgs a) {
  constexpr int kYPieces = y_pieces(up_ctas<W>(kPitch));
  constexpr int kHold = kPitch == 16 ? 1 : kPitch == 48 && Operand<W>::kParts == 1 ? 2 : 0;  // steps of 32 ranks whose weights stay
  constexpr int kWords = kTerms * kTile * kPitch;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ const char *s_y[kTile];  // a token's row; null: none
  __shared__ char *s_out[kTile];
  __shared__ int s_row[kTile];
  const mmq_lora_args &t = a.t;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int tile = a.by_chunks(static_cast<int>(blockIdx.x)), chunk = static_cast<int>(blockIdx.x) - tile * a.chunks;
  const bool in_place = t.y == t.out;
  // (the first product's kernel lets this one begin when everything before it is
  // done, so that all but the terms may be read before the wait)
  const Tile k_tile = tile_at(t, tile, in_place);
  const bool none = k_tile.n == 0;
  const int n = k_tile.n, r = k_tile.rank, od = static_cast<int>(t.od), rmax = t.rank, ranks = (r + 31) / 32;
  const int o0 = chunk * a.columns, o1 = min(o0 + a.columns, od);
  if (tid < kTile) {
    const int row = tid < n ? t.plan[kHead + k_tile.first + tid] : -1;
    s_row[tid] = row;
    s_y[tid] = row < 0 ? nullptr : reinterpret_cast<const char *>(t.y + row * t.y_row);
    s_out[tid] = row < 0 ? nullptr : reinterpret_cast<char *>(t.out + row * t.out_row);
  }
  __syncthreads();
  // A warp's columns are 32 from o0 + 32 warp on, then every 32 kWarps; its pieces
  // of them 8 kEach tokens.  Each thread copies what it needs of y itself, some
  // pieces ahead, to places that no other reads: [piece in flight][part][thread].
  const int first = o0 + 32 * warp, steps = (n + 8 * kEach - 1) / (8 * kEach);
  const int pieces = first < o1 && r > 0 ? (o1 - first + 32 * kWarps - 1) / (32 * kWarps) * steps : 0;
  constexpr uint32_t kPiece = 2 * kEach * kThreads * 16, kPart = kThreads * 16;
  const uint32_t ring = smem_addr(smem) + 4 * kWords + tid * 16;
  // A piece within the tile and the columns, in 16-byte pieces, needs no checks.
  auto whole = [&](int o, int k0) { return a.wide && k0 + 8 * kEach <= n && o + 32 <= od; };
  int ahead_o = first, ahead_k = 0, ahead = 0;
  uint32_t ahead_at = ring;
  auto fetch_next = [&] {
    if (ahead < pieces) {
      const char *const *rows = s_y + ahead_k + 2 * c;
      const uint32_t column = 4 * (ahead_o + 4 * g);
      if (whole(ahead_o, ahead_k)) {
#pragma unroll
        for (int j = 0; j < kEach; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) copy16(ahead_at + (2 * j + h) * kPart, rows[8 * j + h] + column);
      } else {
#pragma unroll 1
        for (int q = 0; q < 2 * kEach; ++q) {
          const char *row = rows[q / 2 * 8 + q % 2];
          const int left = row ? od - ahead_o - 4 * g : 0;
          if (a.wide) {
            if (left > 0) copy16(ahead_at + q * kPart, row + column);
          } else {
            for (int e = 0; e < min(left, 4); ++e) copy4(ahead_at + q * kPart + 4 * e, row + column + 4 * e);
          }
        }
      }
    }
    copies_commit();
    ++ahead;
    ahead_at = ahead_at == ring + (kYPieces - 1) * kPiece ? ring : ahead_at + kPiece;
    ahead_k += 8 * kEach;
    if (ahead_k >= n) ahead_k = 0, ahead_o += 32 * kWarps;
  };
#pragma unroll
  for (int i = 0; i < kYPieces - 1; ++i) fetch_next();
  // rows o + 4 g + i of the weights, ranks 32 step + 8 c on
  const W *up = static_cast<const W *>(t.b) + (static_cast<int64_t>(max(k_tile.adapter, 0)) * od + 4 * g) * rmax + 8 * c;
  auto weights = [&](uint4 (&w)[4], int o, int step) {
    const int k = 32 * step + 8 * c;
    const W *from = up + static_cast<int64_t>(o) * rmax + 32 * step;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = k < r && o + 4 * g + i < od ? __ldg(reinterpret_cast<const uint4 *>(from + i * rmax)) : zero4();
    if (k < r && k + 8 > r) {  // columns past the rank
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t *v = &w[i].x;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] &= k + 2 * e + 1 < r ? 0xffffffffu : k + 2 * e < r ? 0xffffu : 0u;
      }
    }
  };
  // as operands: blocks of 16 rows (4 g, 4 g + 1; 4 g + 2, 4 g + 3), halves of a step
  struct Step {
    Operand<W> w[2][2];
  };
  auto operands = [&](Step &to, int o, int step) {
    uint4 raw[4];
    weights(raw, o, step);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint4 p = raw[2 * b], q = raw[2 * b + 1];
      to.w[b][0].set(p.x, q.x, p.y, q.y, a.zero), to.w[b][1].set(p.z, q.z, p.w, q.w, a.zero);
    }
  };
  Step hold[kHold ? kHold : 1];
  auto take = [&](int o) {
    if (o < o1)
#pragma unroll
      for (int k = 0; k < kHold; ++k)
        if (k < ranks) operands(hold[k], o, k);
  };
  if (pieces) take(first);
  griddep_wait();
  griddep_launch_dependents();
  if (none) return;
  if (r == 0) {
    if (!in_place) copy_rows(a, s_row, n, o0, o1);
    return;
  }
  {
    const uint32_t *from = a.terms + static_cast<int64_t>(tile) * kWords;
    const int chunks = ranks * 4;  // of 16 bytes, of a row
    for (int i = tid; i < kTerms * kTile * chunks; i += kThreads) {
      const int row = i / chunks, at = row * kPitch + 4 * (i - row * chunks);
      copy16(smem_addr(smem) + 4 * at, from + at);
    }
    copies_commit();
    copies_wait<0>();
    __syncthreads();
  }
  const unsigned char *terms = smem + 4 * (g * kPitch + 4 * c);
  int o = first, k0 = 0;
  uint32_t at = ring;
  for (int i = 0; i < pieces; ++i) {
    fetch_next();
    float acc[2][kEach][4] = {};
    const unsigned char *mine = terms + 4 * k0 * kPitch;
    auto step = [&](const Step &k, int s) {
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        Terms x[4];
#pragma unroll
        for (int q = 0; q < kTerms; ++q) {
          const uint4 v = *reinterpret_cast<const uint4 *>(mine + 4 * ((q * kTile + 8 * j) * kPitch + 16 * s));
          x[0].w[q] = v.x, x[1].w[q] = v.y, x[2].w[q] = v.z, x[3].w[q] = v.w;
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) product<W>(acc[b][j], k.w[b][i], x[2 * i], x[2 * i + 1]);
      }
    };
    if constexpr (kHold > 0) {
#pragma unroll
      for (int s = 0; s < kHold; ++s)
        if (s < ranks) step(hold[s], s);
    } else {
      for (int s = 0; s < ranks; ++s) {
        Step k;
        operands(k, o, s);
        step(k, s);
      }
    }
    copies_wait<kYPieces - 1>();
    char *const *rows = s_out + k0 + 2 * c;
    const uint32_t column = 4 * (o + 4 * g);
    if (whole(o, k0)) {
#pragma unroll
      for (int j = 0; j < kEach; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          __stcs(reinterpret_cast<float4 *>(rows[8 * j + h] + column), sum_of<kEach>(acc, j, h, lds4(at + (2 * j + h) * kPart)));
    } else {
#pragma unroll
      for (int j = 0; j < kEach; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 v = sum_of<kEach>(acc, j, h, lds4(at + (2 * j + h) * kPart));
          float *to = reinterpret_cast<float *>(rows[8 * j + h] + column);
          const int left = rows[8 * j + h] ? od - o - 4 * g : 0;
          if (a.wide) {
            if (left > 0) *reinterpret_cast<float4 *>(to) = v;
            continue;
          }
          if (left > 0) to[0] = v.x;
          if (left > 1) to[1] = v.y;
          if (left > 2) to[2] = v.z;
          if (left > 3) to[3] = v.w;
        }
    }
    at = at == ring + (kYPieces - 1) * kPiece ? ring : at + kPiece;
    k0 += 8 * kEach;
    if (k0 >= n) {
      k0 = 0, o += 32 * kWarps;
      take(o);
    }
  }
  copies_wait<0>();
}

// Tokens of a tile: as many as an adapter has on the average, at the most 64,
// and few enough for two CTAs an SM (3584 -> 3584, rank 32; 16 adapters of 8 tokens:
// tiles of 8 7.4 us, of 16 11.0; of 32: 15.4 and 13.6, tiles of 64 23; one adapter of 2000
// tokens: tiles of 16 42 us, of 64 35).
int tile_of(int64_t ntok, int64_t nreq, int64_t nadapters) {
  const int64_t groups = std::max<int64_t>(1, std::min(nreq, nadapters + 1));
  const int64_t want = std::min((ntok + groups - 1) / groups, ntok * kCtas / (2 * 152));
  return want <= 8 ? 8 : want <= 32 ? 16 : 64;
}
int64_t most_tiles(int64_t ntok, int64_t nreq, int64_t nadapters) {
  return std::min(ntok, ntok / tile_of(ntok, nreq, nadapters) + std::min(nreq, nadapters + 1));
}

// most: bytes of shared memory of the kernel's largest rank, for every call.
template <class K>
cudaError_t allow(K kernel, size_t smem, size_t most) {
  if (smem <= 46 * 1024) return cudaSuccess;  // (beside the static arrays, within the 48 KB that need no leave)
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
}

template <class W>
cudaError_t launch_few(const LoraArgs &a, cudaStream_t s) {
  const size_t smem = few_front(a.t.rank) + 4 * static_cast<size_t>(up16(a.t.rank)) * kFew;
  static_assert(few_front(kMaxRank) + 4 * up16(kMaxRank) * kFew <= 46 * 1024, "within what needs no leave");
  const auto kernel = a.t.rank <= 32 ? lora_few_kernel<W, 32> : lora_few_kernel<W, 64>;
  return launch_early(kernel, static_cast<unsigned>(most_tiles(a.t.ntok, a.t.nreq, a.t.nadapters) * kCtas), 1, kThreads, smem, s, a);
}

template <class W, int kTile>
cudaError_t launch_with(LoraArgs a, const CallContext &ctx, cudaStream_t s) {
  using S = Shape<kTile>;
  const int64_t tiles = most_tiles(a.t.ntok, a.t.nreq, a.t.nadapters), pitch = pitch_of(a.t.rank);
  // columns of a CTA in the second product: 256 with four CTAs an SM; with two more, as
  // what it needs beside y and out comes once, but CTAs for five rounds of the SMs
  const int ctas = up_ctas<W>(static_cast<int>(pitch)), y_copies = y_pieces(ctas);
  const int64_t want = ctas == 4 ? 256 : a.t.od * tiles / (5 * 2 * 152) + 128;
  a.columns = static_cast<int>(std::min<int64_t>(2048, std::max<int64_t>(256, want / 256 * 256)));
  const int64_t chunks = (a.t.od + a.columns - 1) / a.columns;
  if (tiles * chunks > 0x7fffffff) return cudaErrorNotSupported;
  a.chunks = static_cast<int>(chunks), a.by_chunks = FastDiv(a.chunks);
  const int x_size = a.t.x_type == MMQ_DT_F32 ? 4 : 2, pass = a.t.rank <= 32 ? 32 : 64;
  auto front = [&](int rank) { return std::max(kStages * S::kPiece * (kTile * x_size + std::min(up16(rank), pass) * 2), 4 * S::kSplit * pass * kTile); };
  auto down_bytes = [&](int rank) { return front(rank) + 4 * static_cast<size_t>(up16(rank)) * kTile; };
  a.front = front(a.t.rank);
  const size_t down = down_bytes(a.t.rank), left = 4 * kTerms * kTile * pitch, up = left + y_copies * 2 * kEach * 16 * kThreads;
  const auto first = pass == 32 ? (x_size == 4 ? lora_down_kernel<W, kTile, true, 32> : lora_down_kernel<W, kTile, false, 32>)
                                : (x_size == 4 ? lora_down_kernel<W, kTile, true, 64> : lora_down_kernel<W, kTile, false, 64>);
  const auto second = pitch == 16 ? lora_up_kernel<W, kTile, 16> : pitch == 48 ? lora_up_kernel<W, kTile, 48> : lora_up_kernel<W, kTile, 80>;
  cudaError_t e = allow(first, down, down_bytes(pass == 32 ? 32 : kMaxRank));
  if (e == cudaSuccess) e = allow(second, up, up);  // (the kernel's own, for every rank that it takes)
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (e == cudaSuccess) e = cudaStreamIsCapturing(s, &cap);
  if (e != cudaSuccess) return e;
  void *scratch = nullptr;
  e = cap == cudaStreamCaptureStatusActive ? cudaMallocAsync(&scratch, tiles * left, s) : cudaMallocFromPoolAsync(&scratch, tiles * left, ctx.pool, s);
  if (e != cudaSuccess) return e;
  a.terms = static_cast<uint32_t *>(scratch);
  e = launch_early(first, static_cast<unsigned>(tiles * kCtas), 1, kThreads, down, s, a);
  if (e == cudaSuccess) e = launch_early(second, static_cast<unsigned>(tiles * chunks), 1, kThreads, up, s, a);
  const cudaError_t ef = cudaFreeAsync(scratch, s);
  return e != cudaSuccess ? e : ef;
}

template <class W>
cudaError_t launch_of(const LoraArgs &a, const CallContext &ctx, cudaStream_t s) {
  switch (tile_of(a.t.ntok, a.t.nreq, a.t.nadapters)) {
    case 8: return launch_few<W>(a, s);
    case 16: return launch_with<W, 16>(a, ctx, s);
    default: return launch_with<W, 64>(a, ctx, s);
  }
}

}  // namespace

int64_t lora_plan_words(int64_t ntok, int64_t nreq, int64_t nadapters) { return kHead + ntok + 3 * most_tiles(ntok, nreq, nadapters); }

cudaError_t launch_lora_plan(LoraPlanArgs a, cudaStream_t s) {
  a.tile = tile_of(a.ntok, a.nreq, a.nadapters);
  a.slots = 1;
  while (a.slots < a.nreq) a.slots *= 2;
  a.few = a.slots <= 1024;  // (up to 1024 keys are compared with all: 256 reads; sorting them takes 55 steps with barriers)
  const size_t smem = ((a.few ? 5 : 4) * static_cast<size_t>(a.slots) + 2) * 4;
  constexpr int kMost = (4 * kMaxRequests + 2) * 4;
  static_assert((kMaxRequests & (kMaxRequests - 1)) == 0 && kMaxRequests == 1 << kRequestBits, "the slots of the most requests");
  // (few requests of few tokens: fewer warps to meet, one request 3.1 instead of 3.7 us, 96 4.9
  // instead of 5.4)
  if (a.slots <= 128 && a.ntok <= 512) return launch_early(lora_plan_kernel<128>, 1, 1, 128, smem, s, a);
  if (smem > 32 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(lora_plan_kernel<1024>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
  }
  const int64_t ctas = std::max<int64_t>(1, (a.ntok + kPlanTokens - 1) / kPlanTokens);
  return launch_early(lora_plan_kernel<1024>, static_cast<unsigned>(ctas), 1, 1024, smem, s, a);
}

cudaError_t launch_lora(LoraArgs a, const CallContext &ctx, cudaStream_t s) {
  const mmq_lora_args &t = a.t;
  auto whole = [](const void *p, int64_t row) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && row % 4 == 0; };
  a.wide = t.od % 4 == 0 && whole(t.y, t.y_row) && whole(t.out, t.out_row);
  return t.type == MMQ_DT_F16 ? launch_of<__half>(a, ctx, s) : launch_of<__nv_bfloat16>(a, ctx, s);
}

}  // namespace mmq
