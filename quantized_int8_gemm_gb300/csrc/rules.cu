// rules.cu -- logits under each request's rules, and their probabilities: penalties
// by the counts of the request's tokens, sparse biases, a grammar's bits, then
// softmax(x / T).  The softmax keeps a running maximum and sum (Milakov and
// Gimelshein, "Online normalizer calculation for softmax", 2018).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace mmq {
namespace {

constexpr int kMostCtas = 16, kThreads = 256, kWarps = kThreads / 32;
// Elements of a CTA at the most, for which the kernel has barriers: a sixteenth of
// 2^18, or 32 KB of 16 bits.
constexpr int kMostSlice = 16384;
static_assert(kMaxVocab <= kMostSlice * kMostCtas, "the largest vocabulary in as many slices");
constexpr unsigned kAll = 0xffffffffu;
// Of a listed token's count: it is among the prompt's; it has a bias; the row's mask hides it.
constexpr uint32_t kMet = 0x80000000u, kBiased = 0x40000000u, kHidden = 0x20000000u;
static_assert(kMaxSaid < kHidden, "a count does not reach the flags");

// 8 bytes into another CTA's shared memory, counted by a barrier beside them
// (both addresses from mapa_shared): no fence, as a store and a cluster barrier
// would need, and so no wait for this thread's other stores.
__device__ __forceinline__ void send(uint32_t addr, uint64_t v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u64 [%0], %1, [%2];" ::"r"(addr), "l"(v), "r"(bar) : "memory");
}
// (Results below 2^-126 become 0: the instruction that keeps them is four.)
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two numbers at once.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ void unpair(uint64_t v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}
// 2^((v - low) scale) of each.
__device__ __forceinline__ float4 exponentials(const float4 &v, float low, float scale) {
  const uint64_t l = pair(-low, -low), s = pair(scale, scale);
  float4 e;
  unpair(mul2(add2(pair(v.x, v.y), l), s), e.x, e.y);
  unpair(mul2(add2(pair(v.z, v.w), l), s), e.z, e.w);
  return make_float4(exp2_approx(e.x), exp2_approx(e.y), exp2_approx(e.z), exp2_approx(e.w));
}
__device__ __forceinline__ float4 times(const float4 &v, float factor) {
  const uint64_t f = pair(factor, factor);
  float4 p;
  unpair(mul2(pair(v.x, v.y), f), p.x, p.y);
  unpair(mul2(pair(v.z, v.w), f), p.z, p.w);
  return p;
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void store_low(float *p) { *p = -INFINITY; }
__device__ __forceinline__ void store_low(__half *p) { *p = __ushort_as_half(0xfc00); }
__device__ __forceinline__ void store_low(__nv_bfloat16 *p) { *p = __ushort_as_bfloat16(0xff80); }
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// Four elements that begin on their own alignment.
__device__ __forceinline__ float4 load4(const __half *p) {
  const uint2 r = *reinterpret_cast<const uint2 *>(p);
  const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&r.x)), b = __half22float2(*reinterpret_cast<const __half2 *>(&r.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
  const uint2 r = *reinterpret_cast<const uint2 *>(p);
  return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
}
// A CTA's slice of a row on its way to shared memory: whole pieces of 16 bytes by
// bulk copies, the elements in front of and behind them by threads.  Element e
// comes to stage[place + e], place being that of the slice in 16 bytes of memory.
constexpr int kFours = 4;                   // fours of a thread at once
constexpr int kEach = kFours * kThreads;    // and of a copy (each has a barrier; all are waited for before the first four)
template <class T>
struct Slice {
  static constexpr int kPiece = 16 / sizeof(T);
  const T *src;
  int place, head, body, len, fours, chunks;  // elements; fours of them; copies
  __device__ __forceinline__ Slice(const T *p, int n) : src(p), len(n) {
    place = static_cast<int>(reinterpret_cast<uintptr_t>(p) / sizeof(T) & (kPiece - 1));
    head = min((kPiece - place) & (kPiece - 1), n);
    body = (n - head) / kPiece * kPiece;
    fours = ((place & 3) + n + 3) >> 2;
    chunks = (fours + kEach - 1) / kEach;
  }
  // Where chunk k begins in the stage: a piece's begin not before its first four.
  __device__ __forceinline__ int chunk(int k) const {
    const int first = 4 * k * kEach + (place & ~3), at = k == 0 ? 0 : (first + kPiece - 1) & ~(kPiece - 1);
    return min(max(at, place + head), place + head + body);
  }
  __device__ __forceinline__ void copy(T *stage, const uint64_t *bars) const {  // (one thread)
    for (int k = 0; k < chunks; ++k) {
      const int from = chunk(k), to = k + 1 < chunks ? chunk(k + 1) : place + head + body;
      const uint32_t bytes = (to - from) * static_cast<uint32_t>(sizeof(T)), bar = smem_addr(bars + k);
      mbar_arrive_expect_tx(bar, bytes);
      if (bytes)
        asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_addr(stage + from)),
                     "l"(src + (from - place)), "r"(bytes), "r"(bar)
                     : "memory");
    }
  }
  // The element that thread k (of 2 kPiece) brings, -1: none.
  __device__ __forceinline__ int edge(int k) const {
    if (k < kPiece) return k < head ? k : -1;
    return k < 2 * kPiece && head + body + k - kPiece < len ? head + body + k - kPiece : -1;
  }
};
__device__ __forceinline__ void put(void *out, int type, int64_t at, float v) {
  if (type == MMQ_DT_F32) {
    static_cast<float *>(out)[at] = v;
  } else {
    const uint16_t half = __half_as_ushort(__float2half_rn(v)), brain = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    static_cast<uint16_t *>(out)[at] = type == MMQ_DT_F16 ? half : brain;
  }
}
// A slice of a row that is written, each element rounded once.
struct Out {
  void *p;
  int64_t at;       // the slice's first element
  int type, inner0, inners;  // fours that are the slice's alone and lie in memory as they do here: inners of them, from inner0 on
  char *base;       // where four 0 would begin
  __device__ __forceinline__ Out(void *out, int t, int64_t first, int m, int len) : p(out), at(first), type(t) {
    const int size = t == MMQ_DT_F32 ? 4 : 2;
    base = static_cast<char *>(out) + (first - m) * size;
    inner0 = m > 0;
    inners = (reinterpret_cast<uintptr_t>(base) & (4 * size - 1)) == 0 ? ((m + len) >> 2) - inner0 : 0;
  }
  __device__ __forceinline__ void four(int f, int m, int len, const float4 &v) const {
    if (static_cast<unsigned>(f - inner0) < static_cast<unsigned>(max(inners, 0))) {
      if (type == MMQ_DT_F32) {
        __stcs(reinterpret_cast<float4 *>(base) + f, v);
      } else {
        const uint2 half = make_uint2(pack2(v.x, v.y, __half()), pack2(v.z, v.w, __half()));
        const uint2 brain = make_uint2(pack2(v.x, v.y, __nv_bfloat16()), pack2(v.z, v.w, __nv_bfloat16()));
        __stcs(reinterpret_cast<uint2 *>(base) + f, type == MMQ_DT_F16 ? half : brain);
      }
      return;
    }
    const float x[4] = {v.x, v.y, v.z, v.w};
    for (int u = 0; u < 4; ++u) {
      const int e = 4 * f - m + u;
      if (e >= 0 && e < len) put(p, type, at + e, u == 0 ? x[0] : u == 1 ? x[1] : u == 2 ? x[2] : x[3]);
    }
  }
};

__device__ __forceinline__ uint64_t warp_max(uint64_t x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const uint64_t y = __shfl_xor_sync(kAll, x, d);
    x = y > x ? y : x;
  }
  return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(kAll, x, d));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(kAll, x, d);
  return x;
}

// The largest number so far and the sum of 2^((x - largest) scale); without a
// number above -inf the sum is 0, or NaN.
struct Part {
  float top = -INFINITY, sum = 0.0f;
  __device__ __forceinline__ float from() const { return top == -INFINITY ? 0.0f : top; }
  __device__ __forceinline__ void raise(float to, float scale) {
    if (to > top) {
      sum *= exp2_approx((top - to) * scale);
      top = to;
    }
  }
  __device__ __forceinline__ void add(float x, float scale) { sum += exp2_approx((x - from()) * scale); }
};
// Joined over a warp's lanes, in each of them.
__device__ __forceinline__ Part joined(Part p, float scale) {
  Part all;
  all.top = warp_max(p.top);
  all.sum = warp_sum(p.sum * exp2_approx((p.top - all.from()) * scale));
  return all;
}
__device__ __forceinline__ uint64_t as_word(Part p) { return static_cast<uint64_t>(__float_as_uint(p.top)) << 32 | __float_as_uint(p.sum); }
__device__ __forceinline__ Part as_part(uint64_t w) {
  Part p;
  p.top = __uint_as_float(static_cast<uint32_t>(w >> 32)), p.sum = __uint_as_float(static_cast<uint32_t>(w));
  return p;
}
// The better of two candidates for the largest logit is the larger number: the
// logit's bits in ascending order above, the complement of the index below; all
// ones for NaN, 0 for none.
__device__ __forceinline__ uint64_t candidate(float x, int v) {
  const uint32_t w = __float_as_uint(x + 0.0f);  // (-0 as 0)
  if (x != x) return ~uint64_t(0);
  if (x == -INFINITY) return 0;
  return static_cast<uint64_t>(w >> 31 ? ~w : w | 0x80000000u) << 32 | (kAll - static_cast<uint32_t>(v));
}

// ---------------------------------------------------------------- the request's tokens and biases
constexpr int kListThreads = 1024;
static_assert(kMaxBiases + 2 * kListThreads - 1 <= 0x7fffffff, "numbers of biases are ints");
constexpr int kEntries = 4096;           // listed tokens that are worked out at once
constexpr int kDrafted = 32;              // drafted tokens that a row's CTAs keep at hand
constexpr int kStarts = kMostCtas + 2;   // numbers for a request: where each CTA's part of its list begins, the first bias
static_assert(kMaxListed * kStarts <= 0x7fffffff, "b * kStarts is an int");

// Sum of x over the threads before this one, and over all.
__device__ __forceinline__ int block_exclusive(int x, int &total, int *sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(kAll, s, d);
    if (lane >= d) s += y;
  }
  if (lane == 31) sm[warp] = s;
  __syncthreads();
  int all = sm[lane];  // (32 warps)
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(kAll, all, d);
    if (lane >= d) all += y;
  }
  total = __shfl_sync(kAll, all, 31);
  const int before = __shfl_sync(kAll, all, warp > 0 ? warp - 1 : 0);
  __syncthreads();
  return (warp > 0 ? before : 0) + s - x;
}

// Lists a request's distinct tokens (drafted ones and those with a bias among
// them), ascending, with the times they count before any drafted one and the sums of their
// biases.  A CTA a request: the bits in shared memory
// give every token its place in the list (sums of population counts), so
// the list does not depend on the order that the threads came in.  Latency
// bound: a round of reads, two passes over the tokens.  Every row of the
// request goes by this list; counting in each CTA of each row took longer
// than the rows themselves (160 requests of 6 rows of 100277: 327 us).
__global__ void __launch_bounds__(kListThreads) token_list_kernel(const __grid_constant__ RulesArgs a) {
  extern __shared__ __align__(16) uint32_t bits[];  // a bit for each token; listed ones before each word; counts, biases, tokens of a round
  __shared__ int s_sums[32], s_first;
  __shared__ bool s_twice;
  const mmq_token_rules &t = a.t;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x, vocab = static_cast<int>(t.vocab);
  const int words = (vocab + 31) / 32;
  int *before = reinterpret_cast<int *>(bits + words), *list = before + words;
  uint32_t *counts = reinterpret_cast<uint32_t *>(list + kEntries);
  float *biases = reinterpret_cast<float *>(counts + kEntries);
  for (int w = tid; w < words; w += kListThreads) bits[w] = 0;
  if (tid == 0) s_twice = false, s_first = 0;
  griddep_wait();
  griddep_launch_dependents();
  const int width = static_cast<int>(t.tokens_width), drafted = t.draft ? t.rows - 1 : 0, nbias = static_cast<int>(t.nbias);
  const int said = !a.penalties ? 0 : t.token_lens ? t.token_lens[b] : width, prompt = t.prompt_lens ? t.prompt_lens[b] : 0;
  const int32_t *ids = t.tokens + b * t.tokens_stride, *draft = t.draft + b * t.draft_stride;
  // (the first tokens of the row's width, while their number is on its way)
  constexpr int kKept = 4;
  int kept[kKept], bias_id = 0;
  float bias_value = 0.0f;
  auto load = [&](int j0, int end) {
#pragma unroll
    for (int u = 0; u < kKept; ++u)
      if (j0 + u * kListThreads < end) kept[u] = ids[j0 + u * kListThreads];
  };
  load(tid, a.penalties ? width : 0);
  const int n = max(min(said, width), 0);
  __syncthreads();
  int bias0 = 0, bias1 = 0;
  if (t.bias_start) {
    // (begins that descend are raised, so that no two requests' lists overlap)
    const int begin = t.bias_start[b], end = t.bias_start[b + 1];
    for (int j = tid; j <= b; j += kListThreads) {
      const int x = min(t.bias_start[j], nbias);
      if (x > 0) atomicMax(&s_first, x);
    }
    if (tid == 0 && (begin < 0 || end < begin || end > nbias)) record_index(a.status);
    __syncthreads();
    bias0 = s_first, bias1 = max(bias0, min(end, nbias));
  }
  if (tid == 0 && said > width) record_index(a.status);
  if (bias0 + tid < bias1) bias_id = t.bias_ids[bias0 + tid], bias_value = t.bias_values[bias0 + tid];
  auto known = [&](int id) { return id >= 0 && id < vocab; };
  auto set = [&](int id) {
    if (known(id)) atomicOr(&bits[id >> 5], 1u << (id & 31));
    else record_index(a.status);
  };
  for (int j0 = tid; j0 < n; j0 += kKept * kListThreads) {
    if (j0 != tid) load(j0, n);
#pragma unroll
    for (int u = 0; u < kKept; ++u)
      if (j0 + u * kListThreads < n) set(kept[u]);
  }
  const int last = min(drafted, t.n_draft ? max(t.n_draft[b], 0) : drafted);
  if (a.penalties)  // (all of them, so that a row does not depend on the rows behind it)
    for (int j = tid; j < drafted; j += kListThreads)
      if (j < last || known(draft[j])) set(draft[j]);
  for (int j = bias0 + tid; j < bias1; j += kListThreads) set(j < bias0 + kListThreads ? bias_id : t.bias_ids[j]);
  __syncthreads();
  const int per = (words + kListThreads - 1) / kListThreads, w0 = min(tid * per, words), w1 = min(w0 + per, words);
  int mine = 0, listed;
  for (int w = w0; w < w1; ++w) mine += __popc(bits[w]);
  int at = block_exclusive(mine, listed, s_sums);
  for (int w = w0; w < w1; ++w) {
    before[w] = at;
    at += __popc(bits[w]);
  }
  __syncthreads();
  if (tid <= a.ctas) {
    const int w = tid * (a.slice / 32);
    a.starts[b * kStarts + tid] = w < words ? before[w] : listed;
  }
  if (tid == 0) a.starts[b * kStarts + kMostCtas + 1] = bias0;
  const int64_t base = static_cast<int64_t>(b) * (width + drafted) + bias0;
  for (int e0 = 0; e0 < listed; e0 += kEntries) {
    const int here = min(kEntries, listed - e0);
    for (int k = tid; k < here; k += kListThreads) counts[k] = 0, biases[k] = 0.0f;
    __syncthreads();
    auto place = [&](int id) {  // in the round, or -1
      if (!known(id)) return -1;
      const int k = before[id >> 5] + __popc(bits[id >> 5] & ((1u << (id & 31)) - 1)) - e0;
      return k < here ? k : -1;
    };
    for (int j0 = tid; j0 < n; j0 += kKept * kListThreads) {
      if (n > kKept * kListThreads) load(j0, n);
#pragma unroll
      for (int u = 0; u < kKept; ++u) {
        const int j = j0 + u * kListThreads, k = j < n ? place(kept[u]) : -1;
        if (k < 0) continue;
        list[k] = kept[u];
        if (j >= prompt) atomicAdd(&counts[k], 1u);
        else atomicOr(&counts[k], kMet);
      }
    }
    if (a.penalties)
      for (int j = tid; j < drafted; j += kListThreads)
        if (const int k = place(draft[j]); k >= 0) list[k] = draft[j];
    for (int j = bias0 + tid; j < bias1; j += kListThreads) {
      const bool again = j >= bias0 + kListThreads;
      const int id = again ? t.bias_ids[j] : bias_id, k = place(id);
      if (k < 0) continue;
      list[k] = id;
      if (atomicOr(&counts[k], kBiased) & kBiased) s_twice = true;
      else biases[k] = again ? t.bias_values[j] : bias_value;
    }
    __syncthreads();
    if (s_twice) {  // a token twice: one warp adds up, in the list's order
      for (int k = tid; k < here; k += kListThreads) biases[k] = 0.0f;
      __syncthreads();
      if (warp == 0) {
        for (int j0 = bias0; j0 < bias1; j0 += 32) {
          const int j = j0 + lane, k = j < bias1 ? place(t.bias_ids[j]) : -1;
          const unsigned peers = __match_any_sync(kAll, k >= 0 ? k : -1 - lane);
          const int turn = __popc(peers & ((1u << lane) - 1));
          for (int r = 0; __any_sync(kAll, r <= turn); ++r) {
            if (k >= 0 && r == turn) biases[k] += t.bias_values[j];
            __syncwarp();
          }
        }
      }
      __syncthreads();
    }
    for (int k = tid; k < here; k += kListThreads) {
      const int64_t to = base + e0 + k;
      a.list[to] = list[k], a.counts[to] = counts[k], a.biases[to] = biases[k];
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- rows
// A cluster takes a row, each CTA of it a slice, in shared memory.  Elements
// that are listed (above) or that a mask hides are left out of a stream that
// all others go by in: for their exponentials against the largest of those that
// a thread has at once, and when the row's sum is known, to be written.  The
// listed ones, few, are worked out one a thread.
//
// HBM bound with many rows (the row in, the row out), latency bound with few.
template <class T>
__global__ void __launch_bounds__(kThreads, 4) token_probs_kernel(const __grid_constant__ RulesArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr bool kWide = sizeof(T) == 4;
  constexpr int kChunks = kMostSlice / (4 * kEach) + 1;  // (one more for where the slice begins)
  __shared__ __align__(8) uint64_t s_bars[kChunks], s_told;
  __shared__ uint64_t s_warp[kWarps], s_all[kMostCtas], s_word;
  __shared__ int s_draft[kDrafted];
  __shared__ float s_from[kWide ? kChunks : 1][kThreads];  // what each thread's exponentials of a copy are against; -inf where all are 0 (or NaN)
  const mmq_token_rules &t = a.t;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_ctarank()), row = a.by_ctas(static_cast<int>(blockIdx.x)), b = a.by_rows(row), i = row - b * t.rows;
  const int words = a.slice / 32;
  T *stage = reinterpret_cast<T *>(smem);
  uint32_t *skip = reinterpret_cast<uint32_t *>(stage + a.slice + 16);  // a bit for each element that the mask hides, one word in front
  const int s0 = rank * a.slice, vocab = static_cast<int>(t.vocab), len = max(min(a.slice, vocab - s0), 0);
  const bool first_thread = tid == 0 && rank == 0;
  const Slice<T> slice(static_cast<const T *>(t.logits) + b * t.logits_req + i * t.logits_row + s0, len);
  if (tid == 0) {
#pragma unroll
    for (int k = 0; k < kChunks; ++k) mbar_init(smem_addr(s_bars + k), 1);
    mbar_init(smem_addr(&s_told), 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(smem_addr(&s_told), 8u * a.ctas);
  }
  // The lists' kernel lets this one begin when everything before it is done, so
  // what is read before the wait is there; its own lists are, behind it.
  if (!a.sparse) griddep_wait();
  const int drafted = t.n_draft ? t.n_draft[b] : t.rows - 1;
  if (i > max(drafted, 0)) return;  // (the whole cluster)
  if (tid == 0) slice.copy(stage, s_bars);
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");  // (the barriers are there: fence_mbar_init)
  // everything that one number of the request says, in one round of reads
  const float rho = t.repetition ? t.repetition[b] : 1.0f, alpha = t.frequency ? t.frequency[b] : 0.0f;
  const float beta = t.presence ? t.presence[b] : 0.0f, temperature = t.temperature ? t.temperature[b] : 1.0f;
  const int64_t which = !t.mask ? -1 : t.mask_rows ? t.mask_rows[row] : row;
  const bool masked = which >= 0 && which < t.nmasks;
  if (first_thread) {
    if (i == 0 && (drafted < 0 || drafted >= t.rows)) record_index(a.status);
    if (t.mask && !masked && which != -1) record_index(a.status);
  }
  const int32_t *mask = t.mask + which * t.mask_stride + (s0 >> 5);
  if (a.penalties && t.draft && tid < min(i, kDrafted)) s_draft[tid] = t.draft[b * t.draft_stride + tid];
  // what is in front of the slice and behind it, in its first and last four
  const int m = slice.place & 3;
  if (const int e = slice.edge(tid); e >= 0) stage[slice.place + e] = slice.src[e];
  if (tid >= 64 && tid < 64 + m) store_low(stage + slice.place - 1 - (tid - 64));
  if (tid >= 96 && tid < 100) store_low(stage + slice.place + len + (tid - 96));
  if (masked) {
    for (int w = tid; w < words; w += kThreads) skip[1 + w] = 32 * w < len ? ~static_cast<uint32_t>(mask[w]) : 0;
    if (tid == 0) skip[0] = skip[words + 1] = 0;
  }
  const float scale = fmaxf(fminf(__fdiv_rn(1.44269504088896341f, temperature), FLT_MAX), 0x1p-149f);  // log2(e) / T, not 0 or inf
  const bool greedy = !(temperature > 0.0f);
  if (a.sparse) griddep_wait();
  griddep_launch_dependents();
  int list0 = 0, list1 = 0;
  int64_t list_base = 0;
  if (a.sparse) {
    const int32_t *starts = a.starts + b * kStarts;
    list0 = starts[rank], list1 = starts[rank + 1];
    list_base = static_cast<int64_t>(b) * (t.tokens_width + (t.draft ? t.rows - 1 : 0)) + starts[kMostCtas + 1];
  }
  // The listed elements, several of a thread at once: what the list, the logits
  // and the mask have of them, and their adjusted logits.  The reads of a
  // thread's first ones are on their way during the copies, which bring their logits.
  constexpr int kListed = 2, kMore = 4;
  struct Listed {
    int at;  // -1: none
    uint32_t count;
    float bias, logit;
  };
  auto look_up = [&](int k0, auto &l) {
    constexpr int kHere = sizeof(l) / sizeof(Listed);
#pragma unroll
    for (int u = 0; u < kHere; ++u) {
      const int k = k0 + tid + u * kThreads;
      l[u].at = -1;
      if (k < list1) l[u].at = a.list[list_base + k] - s0, l[u].count = a.counts[list_base + k], l[u].bias = a.biases[list_base + k];
    }
#pragma unroll
    for (int u = 0; u < kHere; ++u)
      if (l[u].at >= 0) {
        if (k0 != list0) l[u].logit = to_f32(slice.src[l[u].at]);
        if (masked && !(static_cast<uint32_t>(mask[l[u].at >> 5]) >> (l[u].at & 31) & 1)) l[u].count |= kHidden;
      }
  };
  auto adjust = [&](const Listed &l) {
    float y = l.logit;
    if (a.penalties) {
      uint32_t times = l.count & ~(kMet | kBiased | kHidden);
      if (t.draft)
        for (int j = 0; j < i; ++j) times += (j < kDrafted ? s_draft[j] : t.draft[b * t.draft_stride + j]) == l.at + s0;
      if (times || (l.count & kMet)) y = y > 0.0f ? __fdiv_rn(y, rho) : __fmul_rn(y, rho);
      if (times) y = __fsub_rn(__fsub_rn(y, __fmul_rn(alpha, static_cast<float>(times))), beta);
    }
    if (l.count & kBiased) y = __fadd_rn(y, l.bias);
    return l.count & kHidden ? -INFINITY : y;
  };
  Listed mine[kListed];
  look_up(list0, mine);
  Part part;
  uint64_t key = 0;
  // four f of the slice, elements 4 f - m on: what is not the stream's is -inf
  float4 *const fours = reinterpret_cast<float4 *>(stage + slice.place - m);
  auto plain_four = [&](int f) {
    if constexpr (kWide) return fours[f];
    else return load4(stage + slice.place - m + 4 * f);
  };
  auto four = [&](int f) {  // (what the mask hides is -inf in the slice, too, from then on)
    float4 v = plain_four(f);
    if (masked) {
      const int e = 4 * f - m + 32;
      const uint32_t off = __funnelshift_r(skip[e >> 5], skip[(e >> 5) + 1], e) & 15;
      if (off & 1) v.x = -INFINITY;
      if (off & 2) v.y = -INFINITY;
      if (off & 4) v.z = -INFINITY;
      if (off & 8) v.w = -INFINITY;
      if constexpr (!kWide)
        if (off) *reinterpret_cast<uint2 *>(stage + slice.place - m + 4 * f) = make_uint2(pack2(v.x, v.y, T()), pack2(v.z, v.w, T()));
    }
    return v;
  };

  const Out adjusted(t.adjusted, t.adjusted_type, b * t.adjusted_req + i * t.adjusted_row + s0, m, len);
  const WaitCtl wait = {a.status, a.abort_epoch, a.epoch, a.limit_ns};
  // (one warp asks, the others are at the barrier: asking is an instruction after another)
  if (warp == 0)
    for (int k = 0; k < slice.chunks; ++k)
      if (!mbar_wait(smem_addr(s_bars + k), 0, wait, false)) mbar_wait(smem_addr(s_bars + k), 0, wait, false);
  __syncthreads();
  if (a.sparse) {  // the listed ones leave the stream
#pragma unroll
    for (int u = 0; u < kListed; ++u)
      if (mine[u].at >= 0) {
        T *at = stage + slice.place + mine[u].at;
        mine[u].logit = to_f32(*at);
        store_low(at);
      }
#pragma unroll 4
    for (int k = list0 + tid + kListed * kThreads; k < list1; k += kThreads) store_low(stage + slice.place + a.list[list_base + k] - s0);
    __syncthreads();
  }

  // the stream, kEach fours at a time
  float best = -INFINITY;
  for (int k = 0; k < slice.chunks; ++k) {
    const int f0 = k * kEach + tid;
    float4 x[kFours];
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < kFours; ++u)
      if (f0 + u * kThreads < slice.fours) {
        x[u] = four(f0 + u * kThreads);
        if (t.adjusted && !a.in_place) adjusted.four(f0 + u * kThreads, m, len, x[u]);
        top = fmaxf(top, fmaxf(fmaxf(x[u].x, x[u].y), fmaxf(x[u].z, x[u].w)));
      }
    if (!t.probs) continue;
    if (greedy) {
#pragma unroll
      for (int u = 0; u < kFours; ++u)
        if (f0 + u * kThreads < slice.fours && (x[u].x != x[u].x || x[u].y != x[u].y || x[u].z != x[u].z || x[u].w != x[u].w)) key = ~uint64_t(0);
      if (top > best) {  // only numbers above the largest so far
        best = top;
        int at = 0;
#pragma unroll
        for (int u = kFours - 1; u >= 0; --u)
          if (f0 + u * kThreads < slice.fours) {
            const int e = 4 * (f0 + u * kThreads) - m;
            if (x[u].w == top) at = e + 3;
            if (x[u].z == top) at = e + 2;
            if (x[u].y == top) at = e + 1;
            if (x[u].x == top) at = e;
          }
        const uint64_t c = candidate(top, s0 + at);
        key = c > key ? c : key;
      }
      continue;
    }
    const float low = top == -INFINITY ? 0.0f : top;  // (-inf less -inf is no number)
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < kFours; ++u)
      if (f0 + u * kThreads < slice.fours) {
        const float4 v = exponentials(x[u], low, scale);
        sum += (v.x + v.y) + (v.z + v.w);
        if constexpr (kWide) fours[f0 + u * kThreads] = v;
      }
    if constexpr (kWide) s_from[k][tid] = top;
    // (against top, not low: where there is nothing, 0 or NaN times 2^-inf = 0; 2^(0 - largest)
    // may be infinite)
    part.raise(top, scale);
    part.sum += sum * exp2_approx((top - part.from()) * scale);
  }
  // the listed ones
  float my_y[kListed];
#pragma unroll
  for (int u = 0; u < kListed; ++u)
    if (mine[u].at >= 0) my_y[u] = adjust(mine[u]);
  auto for_listed = [&](auto &&f) {
#pragma unroll
    for (int u = 0; u < kListed; ++u)
      if (mine[u].at >= 0) f(mine[u].at, my_y[u]);
    for (int k0 = list0 + kListed * kThreads; k0 < list1; k0 += kMore * kThreads) {
      Listed l[kMore];
      look_up(k0, l);
#pragma unroll
      for (int u = 0; u < kMore; ++u)
        if (l[u].at >= 0) f(l[u].at, adjust(l[u]));
    }
  };
  if (a.sparse && t.probs)
    for_listed([&](int at, float y) {
      if (greedy) {
        const uint64_t c = candidate(y, s0 + at);
        key = c > key ? c : key;
      } else {
        part.raise(y, scale);
        part.add(y, scale);
      }
    });
  if (t.adjusted && a.in_place && masked) {  // (listed ones stay as they are until the end)
    for (int e = tid; e < len; e += kThreads)
      if (!(static_cast<uint32_t>(mask[e >> 5]) >> (e & 31) & 1)) put(t.adjusted, t.adjusted_type, adjusted.at + e, -INFINITY);
  }
  if (!t.probs) {
    if (a.sparse) {
      __syncthreads();  // (before the listed ones' places are written again)
      for_listed([&](int at, float y) { put(t.adjusted, t.adjusted_type, adjusted.at + at, y); });
    }
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    return;
  }

  // largest number and sum, or candidate: the warp's, the CTA's, the cluster's
  uint64_t word = greedy ? warp_max(key) : as_word(joined(part, scale));
  if (lane == 0) s_warp[warp] = word;
  __syncthreads();
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");  // (every CTA of the cluster runs)
  if (warp == 0) {
    auto join = [&](const uint64_t *words_of, int count) {
      if (greedy) return warp_max(lane < count ? words_of[lane] : 0);
      return as_word(joined(lane < count ? as_part(words_of[lane]) : Part{}, scale));
    };
    word = join(s_warp, kWarps);
    if (lane < a.ctas) send(mapa_shared(smem_addr(s_all + rank), lane), word, mapa_shared(smem_addr(&s_told), lane));
    if (!mbar_wait(smem_addr(&s_told), 0, wait, false)) mbar_wait(smem_addr(&s_told), 0, wait, false);
    word = join(s_all, a.ctas);
    if (lane == 0) s_word = word;
  }
  __syncthreads();
  word = s_word;
  const Part all = as_part(word);
  const bool bad = greedy && word == ~uint64_t(0);
  const int first = greedy && word && !bad ? static_cast<int>(kAll - static_cast<uint32_t>(word)) - s0 : -8;  // greedy: the element that has it all
  const float base = all.from(), factor = all.sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, all.sum);
  auto probability = [&](float y, int e) {
    if (greedy) return bad ? NAN : e == first ? 1.0f : 0.0f;
    return exp2_approx((y - base) * scale) * factor;
  };
  const Out out(t.probs, t.probs_type, b * t.probs_req + i * t.probs_row + s0, m, len);
  if (greedy) {
    for (int f = tid; f < slice.fours; f += kThreads) {
      const int e = 4 * f - m;
      out.four(f, m, len, make_float4(probability(0, e), probability(0, e + 1), probability(0, e + 2), probability(0, e + 3)));
    }
  } else {
    for (int k = 0; k < slice.chunks; ++k) {
      float share = 0.0f;
      if constexpr (kWide) share = exp2_approx((s_from[k][tid] - base) * scale) * factor;
#pragma unroll
      for (int u = 0; u < kFours; ++u) {
        const int f = k * kEach + tid + u * kThreads;
        if (f >= slice.fours) break;
        float4 v;
        if constexpr (kWide) {
          v = times(fours[f], share);
        } else {
          v = times(exponentials(plain_four(f), base, scale), factor);
        }
        out.four(f, m, len, v);
      }
    }
  }
  if (a.sparse) {
    __syncthreads();  // (before the listed ones' places are written again)
    for_listed([&](int at, float y) {
      put(t.probs, t.probs_type, out.at + at, probability(y, at));
      if (t.adjusted) put(t.adjusted, t.adjusted_type, adjusted.at + at, y);
    });
  }
}

// Bytes of shared memory: of a row's CTA with that many elements, of a request's list.
size_t row_bytes(size_t slice, size_t size, bool mask) { return (slice + 16) * size + (mask ? 4 * (slice / 32 + 2) : 0); }
size_t list_bytes(size_t vocab) { return 8 * ((vocab + 31) / 32) + 12 * kEntries; }

template <class T>
cudaError_t launch_with(const RulesArgs &a, size_t smem, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (a.ctas > 8) e = cudaFuncSetAttribute(token_probs_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && smem > 40 * 1024)  // (beside the static arrays, within the 48 KB that need no leave)
    e = cudaFuncSetAttribute(token_probs_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(row_bytes(kMostSlice, sizeof(T), true)));
  if (e != cudaSuccess) return e;
  const unsigned ctas = a.ctas;
  return launch_early(token_probs_kernel<T>, Cluster{ctas}, static_cast<unsigned>(a.t.nreq * a.t.rows) * ctas, 1, kThreads, smem, s, a);
}

}  // namespace

cudaError_t launch_token_probs(RulesArgs a, const CallContext &ctx, cudaStream_t s) {
  // CTAs of a row: slices of up to 50 KB in fp32 (960 rows of 100277: 8 CTAs of a row 189 us,
  // 7 208, 9 196, 10 200, 12 225, 16 275) and of up to 32 KB, the most that the kernel takes,
  // in 16 bits (120 rows of 128256: 8 CTAs 56.3 us, 9 56.8, 10 58.2, 12 58.8, 16 61.8); with few
  // rows more, as long as all run at once and have 2048 elements or more (one row of 32000:
  // 2 CTAs 11.2 us, 4 9.2, 8 8.4, 12 8.3, 15 8.5, 16 8.4)
  const int64_t rows = a.t.nreq * a.t.rows, size = a.t.type == MMQ_DT_F32 ? 4 : 2, most = (size == 4 ? 50 : 32) * 1024;
  const int64_t fit = (a.t.vocab * size + most - 1) / most, few = std::min(4 * 152 / rows, a.t.vocab / 2048);
  const int64_t ctas = std::min<int64_t>(kMostCtas, std::max<int64_t>({fit, few, 1}));
  a.ctas = static_cast<int>(ctas);
  a.by_ctas = FastDiv(a.ctas);
  a.slice = static_cast<int>(((a.t.vocab + ctas - 1) / ctas + 31) / 32 * 32);  // (masks in whole words)
  if (a.slice > kMostSlice) return cudaErrorNotSupported;  // (the rule above gives none such; the kernel would pass its barriers' end)
  a.by_rows = FastDiv(a.t.rows);
  a.sparse = a.penalties || a.t.bias_start;
  void *scratch = nullptr;
  cudaError_t e = cudaSuccess;
  if (a.sparse) {
    const size_t listed = a.t.nreq * (a.t.tokens_width + (a.t.draft ? a.t.rows - 1 : 0)) + a.t.nbias;
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    e = cudaStreamIsCapturing(s, &cap);
    if (e != cudaSuccess) return e;
    const size_t bytes = 4 * (3 * listed + a.t.nreq * kStarts);
    e = cap == cudaStreamCaptureStatusActive ? cudaMallocAsync(&scratch, bytes, s) : cudaMallocFromPoolAsync(&scratch, bytes, ctx.pool, s);
    if (e != cudaSuccess) return e;
    a.starts = static_cast<int32_t *>(scratch);
    a.list = a.starts + a.t.nreq * kStarts;
    a.counts = reinterpret_cast<uint32_t *>(a.list + listed);
    a.biases = reinterpret_cast<float *>(a.counts + listed);
    e = cudaFuncSetAttribute(token_list_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(list_bytes(kMaxVocab)));
    if (e == cudaSuccess) e = launch_early(token_list_kernel, static_cast<unsigned>(a.t.nreq), 1, kListThreads, list_bytes(a.t.vocab), s, a);
  }
  const size_t smem = row_bytes(a.slice, size, a.t.mask);
  if (e == cudaSuccess) {
    if (a.t.type == MMQ_DT_F32) e = launch_with<float>(a, smem, s);
    else e = a.t.type == MMQ_DT_F16 ? launch_with<__half>(a, smem, s) : launch_with<__nv_bfloat16>(a, smem, s);
  }
  if (scratch) {
    const cudaError_t ef = cudaFreeAsync(scratch, s);
    if (e == cudaSuccess) e = ef;
  }
  return e;
}

}  // namespace mmq
