// rules.cu -- logits under each request's rules, and their probabilities.
//
// A row: penalties by the counts of the request's tokens, sparse biases, a
// grammar's bits, then softmax(x / T).  A cluster of eight CTAs takes a row,
// each an eighth of the vocabulary in shared memory, so the logits are read
// once and the probabilities written once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace mmq {
namespace {

constexpr int kCtas = 8, kThreads = 512, kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;
constexpr uint32_t kMet = 0x8000, kTimes = 0x7fff;  // a token's 16 bits: among the prompt's; times behind it

__device__ __forceinline__ void st_cluster(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }
__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// Elements [0, len) of a row's slice from x[m] on; `m` is the slice's place in
// 16 bytes of memory, so that whole 16-byte pieces lie on 16 bytes here too.
__device__ __forceinline__ void load_slice(const float *p, float *x, int m, int len, uint32_t bar) {
  const int head = min((4 - m) & 3, len), body = (len - head) >> 2, tail = head + 4 * body;
  if (threadIdx.x == 0) {
    mbar_arrive_expect_tx(bar, body * 16);
    if (body)
      asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_addr(x + m + head)),
                   "l"(p + head), "r"(body * 16), "r"(bar)
                   : "memory");
  }
  const int t = static_cast<int>(threadIdx.x);
  if (t < head) x[m + t] = p[t];
  else if (t >= 4 && t - 4 < len - tail) x[m + tail + t - 4] = p[tail + t - 4];
}
template <class T>
__device__ __forceinline__ void load_slice(const T *p, float *x, int m, int len, uint32_t) {
  const int head = min((8 - m) & 7, len), body = (len - head) >> 3, tail = head + 8 * body;
  const uint4 *src = reinterpret_cast<const uint4 *>(p + head);
  float4 *dst = reinterpret_cast<float4 *>(x + m + head);
  for (int i0 = threadIdx.x; i0 < body; i0 += 4 * kThreads) {
    uint4 r[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i0 + u * kThreads < body) r[u] = __ldcs(src + i0 + u * kThreads);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i0 + u * kThreads < body) {
        const float2 a = unpack2(r[u].x, T()), b = unpack2(r[u].y, T()), c = unpack2(r[u].z, T()), d = unpack2(r[u].w, T());
        dst[2 * (i0 + u * kThreads)] = make_float4(a.x, a.y, b.x, b.y);
        dst[2 * (i0 + u * kThreads) + 1] = make_float4(c.x, c.y, d.x, d.y);
      }
  }
  const int t = static_cast<int>(threadIdx.x);
  if (t < head) x[m + t] = to_f32(p[t]);
  else if (t >= 8 && t - 8 < len - tail) x[m + tail + t - 8] = to_f32(p[tail + t - 8]);
}

// One element, or four that begin on their own alignment, rounded once.
__device__ __forceinline__ void put(void *p, int type, int64_t at, float v) {
  if (type == MMQ_DT_F32) __stcs(static_cast<float *>(p) + at, v);
  else if (type == MMQ_DT_F16) static_cast<__half *>(p)[at] = __float2half_rn(v);
  else static_cast<__nv_bfloat16 *>(p)[at] = __float2bfloat16_rn(v);
}
__device__ __forceinline__ void put4(void *p, int type, int64_t at, float4 v) {
  if (type == MMQ_DT_F32) {
    __stcs(reinterpret_cast<float4 *>(static_cast<float *>(p) + at), v);
    return;
  }
  uint2 r;
  if (type == MMQ_DT_F16) r = make_uint2(pack2(v.x, v.y, __half()), pack2(v.z, v.w, __half()));
  else r = make_uint2(pack2(v.x, v.y, __nv_bfloat16()), pack2(v.z, v.w, __nv_bfloat16()));
  __stcs(reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + at), r);
}
// Elements of a slice (x[m], ...) to out[at], ...; f gives what is written for
// element e.  Four at a time where their places in memory and here agree.
template <class F>
__device__ __forceinline__ void write_slice(void *out, int type, int64_t at, int m, int len, F &&f) {
  const uint32_t bytes = type == MMQ_DT_F32 ? 4 : 2;
  const int place = static_cast<int>((reinterpret_cast<uintptr_t>(out) / bytes + at) & 3);
  const int t = static_cast<int>(threadIdx.x);
  if (place == (m & 3)) {
    const int head = min((4 - place) & 3, len), body = (len - head) >> 2, tail = head + 4 * body;
    for (int i = t; i < body; i += kThreads) {
      const int e = head + 4 * i;
      put4(out, type, at + e, make_float4(f(e), f(e + 1), f(e + 2), f(e + 3)));
    }
    if (t < head) put(out, type, at + t, f(t));
    else if (t >= 4 && t - 4 < len - tail) put(out, type, at + tail + t - 4, f(tail + t - 4));
    return;
  }
#pragma unroll 4
  for (int e = t; e < len; e += kThreads) put(out, type, at + e, f(e));
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
__device__ __forceinline__ uint64_t warp_max(uint64_t x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const uint64_t y = __shfl_xor_sync(kAll, x, d);
    x = y > x ? y : x;
  }
  return x;
}

// Counts a token of the slice: `answered` ones up to kTimes, the prompt's once.
__device__ __forceinline__ void count(uint32_t *counts, int at, bool answered, bool many) {
  uint32_t *w = counts + (at >> 1);
  const int shift = (at & 1) * 16;
  if (!answered) {
    atomicOr(w, kMet << shift);
  } else if (!many) {
    atomicAdd(w, 1u << shift);
  } else {  // more tokens than kTimes: one of them could go over
    uint32_t old = *w, was;
    do {
      was = old;
      if ((was >> shift & kTimes) == kTimes) return;
      old = atomicCAS(w, was, was + (1u << shift));
    } while (old != was);
  }
}

// HBM bound with many rows (the row in, the row out), latency bound with few.
template <class T>
__global__ void __launch_bounds__(kThreads) __cluster_dims__(kCtas, 1, 1) token_probs_kernel(const __grid_constant__ RulesArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(8) uint64_t s_bar;
  __shared__ float s_max[kWarps], s_sum[kWarps];
  __shared__ uint64_t s_key[kWarps], s_all[kCtas];
  __shared__ int s_bias_id[kThreads];
  __shared__ float s_bias[kThreads];
  const mmq_token_rules &t = a.t;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_ctarank();
  const int row = static_cast<int>(blockIdx.x / kCtas), b = a.by_rows(row), i = row - b * t.rows;
  float *x = reinterpret_cast<float *>(smem);                        // a.slice + 8
  uint32_t *counts = reinterpret_cast<uint32_t *>(x + a.slice + 8);  // 16 bits an element, if there are penalties
  uint32_t *allowed = counts + (a.penalties ? a.slice / 2 + 4 : 0);  // a bit an element, one word in front
  if (tid == 0) {
    mbar_init(smem_addr(&s_bar), 1);
    fence_mbar_init();
  }
  const int s0 = static_cast<int>(rank) * a.slice, vocab = static_cast<int>(t.vocab), len = max(min(a.slice, vocab - s0), 0);
  if (a.penalties)
    for (int e = tid; e < a.slice / 8 + 1; e += kThreads) reinterpret_cast<uint4 *>(counts)[e] = make_uint4(0, 0, 0, 0);
  griddep_wait();
  griddep_launch_dependents();
  if (t.n_draft) {
    const int n = t.n_draft[b];
    if (tid == 0 && rank == 0 && i == 0 && (n < 0 || n >= t.rows)) record_index(a.status);
    if (i > max(n, 0)) return;  // (the whole cluster)
  }
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  __syncthreads();
  constexpr int kPiece = 16 / sizeof(T);
  const T *src = static_cast<const T *>(t.logits) + b * t.logits_req + i * t.logits_row + s0;
  const int m = static_cast<int>(reinterpret_cast<uintptr_t>(src) / sizeof(T) & (kPiece - 1));
  load_slice(src, x, m, len, smem_addr(&s_bar));
  if (a.penalties) {
    const int32_t *ids = t.tokens + b * t.tokens_stride;
    int n = static_cast<int>(t.tokens_width);
    if (t.token_lens) {
      const int said = t.token_lens[b];
      if (tid == 0 && rank == 0 && i == 0 && said > n) record_index(a.status);
      n = max(min(said, n), 0);
    }
    const int prompt = t.prompt_lens ? t.prompt_lens[b] : 0;
    auto meet = [&](int v, bool answered) {
      const int at = v - s0;
      if (at >= 0 && at < len) count(counts, m + at, answered, a.many);
      else if (rank == 0 && (v < 0 || v >= vocab)) record_index(a.status);
    };
    for (int j0 = tid; j0 < n; j0 += 4 * kThreads) {
      int v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (j0 + u * kThreads < n) v[u] = ids[j0 + u * kThreads];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (j0 + u * kThreads < n) meet(v[u], j0 + u * kThreads >= prompt);
    }
    if (t.draft)
      for (int j = tid; j < i; j += kThreads) meet(t.draft[b * t.draft_stride + j], true);
  }
  bool masked = false;
  if (t.mask) {
    const int64_t which = t.mask_rows ? t.mask_rows[row] : row;
    masked = which >= 0 && which < t.nmasks;
    if (tid == 0 && rank == 0 && !masked && which != -1) record_index(a.status);
    if (masked) {
      const int32_t *bits = t.mask + which * t.mask_stride + (s0 >> 5);
      const int words = (len + 31) >> 5;
      for (int w = tid; w < words; w += kThreads) allowed[1 + w] = static_cast<uint32_t>(bits[w]);
      if (tid == 0) allowed[0] = allowed[1 + words] = 0;
    }
  }
  const float rho = t.repetition ? t.repetition[b] : 1.0f, alpha = t.frequency ? t.frequency[b] : 0.0f;
  const float beta = t.presence ? t.presence[b] : 0.0f, temperature = t.temperature ? t.temperature[b] : 1.0f;
  const bool greedy = !(temperature > 0.0f);
  int bias0 = 0, bias1 = 0;
  if (t.bias_start) {
    bias0 = t.bias_start[b], bias1 = t.bias_start[b + 1];
    const int most = static_cast<int>(t.nbias);
    if (tid == 0 && rank == 0 && i == 0 && (bias0 < 0 || bias1 < bias0 || bias1 > most)) record_index(a.status);
    bias0 = max(bias0, 0), bias1 = min(bias1, most);
  }
  __syncthreads();
  if constexpr (sizeof(T) == 4) {
    const WaitCtl wait = {a.status, a.abort_epoch, a.epoch, a.limit_ns};
    mbar_wait(smem_addr(&s_bar), 0, wait, false);
  }
  // elements of x in fours; place q holds those of x[4 q], ..., of which
  // elements [0, len) are this slice's
  const int last = (m + len + 3) >> 2;
  auto penalized = [&](float v, uint32_t c) {
    if (c) {
      v = v > 0.0f ? __fdiv_rn(v, rho) : __fmul_rn(v, rho);
      const uint32_t times = c & kTimes;
      if (times) v = __fsub_rn(__fsub_rn(v, __fmul_rn(alpha, static_cast<float>(times))), beta);
    }
    return v;
  };
  auto penalties = [&](int q, float4 &v) {
    const uint2 c = reinterpret_cast<const uint2 *>(counts)[q];
    if (c.x | c.y) {
      v.x = penalized(v.x, c.x & 0xffff), v.y = penalized(v.y, c.x >> 16);
      v.z = penalized(v.z, c.y & 0xffff), v.w = penalized(v.w, c.y >> 16);
    }
  };
  if (bias1 > bias0) {
    if (a.penalties) {
      for (int q = tid; q < last; q += kThreads) {
        float4 v = reinterpret_cast<float4 *>(x)[q];
        penalties(q, v);
        reinterpret_cast<float4 *>(x)[q] = v;
      }
    }
    for (int j0 = bias0; j0 < bias1; j0 += kThreads) {
      const int n = min(kThreads, bias1 - j0);
      if (tid < n) s_bias_id[tid] = t.bias_ids[j0 + tid], s_bias[tid] = t.bias_values[j0 + tid];
      __syncthreads();
      if (warp == 0) {
        for (int k = 0; k < n; k += 32) {
          const int v = k + lane < n ? s_bias_id[k + lane] : s0, at = v - s0;
          if (rank == 0 && (v < 0 || v >= vocab)) record_index(a.status);
          const bool here = k + lane < n && at >= 0 && at < len;
          // the same token twice: in the list's order
          const unsigned peers = __match_any_sync(kAll, here ? at : -1 - lane);
          const int turn = __popc(peers & ((1u << lane) - 1));
          for (int r = 0; __any_sync(kAll, r <= turn); ++r) {
            if (here && r == turn) x[m + at] = __fadd_rn(x[m + at], s_bias[k + lane]);
            __syncwarp();
          }
        }
      }
      __syncthreads();
    }
  }
  const bool late = bias1 > bias0 || !a.penalties;  // (no penalties to be applied any more)
  float top = -INFINITY;
  bool nan = false;
  uint64_t key = 0;
  for (int q = tid; q < last; q += kThreads) {
    float4 v = reinterpret_cast<float4 *>(x)[q];
    if (!late) penalties(q, v);
    float *e = &v.x;
    const int at = 4 * q - m;
    uint32_t on = 15;
    if (masked) on = __funnelshift_r(allowed[(at + 32) >> 5], allowed[((at + 32) >> 5) + 1], at + 32);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (!(on >> u & 1) || at + u < 0 || at + u >= len) e[u] = -INFINITY;
      if (greedy) {
        nan |= e[u] != e[u];
        const uint32_t w = __float_as_uint(e[u] + 0.0f);  // (-0 as 0)
        const uint64_t mine = static_cast<uint64_t>(w >> 31 ? ~w : w | 0x80000000u) << 32 | (kAll - static_cast<uint32_t>(s0 + at + u));
        if (e[u] > -INFINITY && mine > key) key = mine;
      }
      top = fmaxf(top, e[u]);
    }
    reinterpret_cast<float4 *>(x)[q] = v;
  }
  if (t.adjusted) {
    __syncthreads();
    write_slice(t.adjusted, t.adjusted_type, b * t.adjusted_req + i * t.adjusted_row + s0, m, len, [&](int e) { return x[m + e]; });
    if (!t.probs) {
      asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
      return;
    }
  }
  const int64_t at = b * t.probs_req + i * t.probs_row + s0;
  if (greedy) {
    key = warp_max(key);
    if (__any_sync(kAll, nan)) key = ~uint64_t(0);
    if (lane == 0) s_key[warp] = key;
    __syncthreads();
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    if (warp == 0) {
      key = warp_max(lane < kWarps ? s_key[lane] : 0);
      if (lane < kCtas) st_cluster(mapa_shared(smem_addr(s_all + rank), lane), key);
    }
    cluster_sync();
#pragma unroll
    for (int c = 0; c < kCtas; ++c) key = s_all[c] > key ? s_all[c] : key;
    const int best = key ? static_cast<int>(kAll - static_cast<uint32_t>(key)) - s0 : -1;
    const bool bad = key == ~uint64_t(0);
    write_slice(t.probs, t.probs_type, at, m, len, [&](int e) { return bad ? NAN : e == best ? 1.0f : 0.0f; });
    return;
  }
  top = warp_max(top);
  if (lane == 0) s_max[warp] = top;
  __syncthreads();
  top = warp_max(lane < kWarps ? s_max[lane] : -INFINITY);
  const float from = top == -INFINITY ? 0.0f : top;
  const float scale = fminf(__fdiv_rn(1.44269504088896341f, temperature), FLT_MAX);  // log2(e) / T
  float sum = 0.0f;
  for (int q = tid; q < last; q += kThreads) {
    float4 v = reinterpret_cast<float4 *>(x)[q];
    v.x = exp2_approx((v.x - from) * scale), v.y = exp2_approx((v.y - from) * scale);
    v.z = exp2_approx((v.z - from) * scale), v.w = exp2_approx((v.w - from) * scale);
    sum += (v.x + v.y) + (v.z + v.w);
    reinterpret_cast<float4 *>(x)[q] = v;
  }
  sum = warp_sum(sum);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  if (warp == 0) {
    sum = warp_sum(lane < kWarps ? s_sum[lane] : 0.0f);
    const uint64_t both = static_cast<uint64_t>(__float_as_uint(top)) << 32 | __float_as_uint(sum);
    if (lane < kCtas) st_cluster(mapa_shared(smem_addr(s_all + rank), lane), both);
  }
  cluster_sync();
  float highest = -INFINITY, total = 0.0f;
#pragma unroll
  for (int c = 0; c < kCtas; ++c) highest = fmaxf(highest, __uint_as_float(static_cast<uint32_t>(s_all[c] >> 32)));
  const float base = highest == -INFINITY ? 0.0f : highest;
#pragma unroll
  for (int c = 0; c < kCtas; ++c) {
    const float part = __uint_as_float(static_cast<uint32_t>(s_all[c])), high = __uint_as_float(static_cast<uint32_t>(s_all[c] >> 32));
    total += part * exp2_approx((high - base) * scale);
  }
  const float factor = total == 0.0f ? 0.0f : __fdiv_rn(exp2_approx((top - base) * scale), total);
  write_slice(t.probs, t.probs_type, at, m, len, [&](int e) { return x[m + e] * factor; });
}

template <class T>
cudaError_t launch_with(const RulesArgs &a, size_t smem, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(token_probs_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_early(token_probs_kernel<T>, static_cast<unsigned>(a.t.nreq * a.t.rows * kCtas), 1, kThreads, smem, s, a);
}

}  // namespace

cudaError_t launch_token_probs(RulesArgs a, cudaStream_t s) {
  a.slice = static_cast<int>(((a.t.vocab + kCtas - 1) / kCtas + 31) / 32 * 32);  // (masks in whole words)
  a.by_rows = FastDiv(a.t.rows);
  const size_t smem = (a.slice + 8) * 4 + (a.penalties ? (a.slice / 2 + 4) * 4 : 0) + (a.t.mask ? (a.slice / 32 + 2) * 4 : 0);
  if (a.t.type == MMQ_DT_F32) return launch_with<float>(a, smem, s);
  return a.t.type == MMQ_DT_F16 ? launch_with<__half>(a, smem, s) : launch_with<__nv_bfloat16>(a, smem, s);
}

}  // namespace mmq
