// verify.cu -- drafted tokens against the target's probabilities.
//
// Drafted token x_i of a request is kept while u_i * q_i(x_i) < p_i(x_i), i.e.
// with probability min(1, p/q) for u uniform in [0, 1).  At the first refusal
// the token is drawn from the normalised (p - q)+, after the last drafted
// token from p.  With e_v independent exponential variates, argmax_v w_v / e_v
// draws v with probability w_v / sum w: no sum over the vocabulary is needed,
// and a maximum does not depend on the order it is taken in, so the result is
// the same for every split of the row.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace mmq {
namespace {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// The better of two candidates is the larger number: the key's bits above,
// the complement of the index below (so that ties go to the lowest index).
// 0: no candidate.
__device__ __forceinline__ void consider(uint64_t &best, float w, float e, int64_t v) {
  const float key = w / e;
  if (!(w > 0.0f && key > 0.0f)) return;
  const uint64_t mine = static_cast<uint64_t>(__float_as_uint(key)) << 32 | (0xffffffffu - static_cast<uint32_t>(v));
  if (mine > best) best = mine;
}

// This CTA's part of one row.  Weights: p, less q where there is one, and none
// for entry `skip`.  Loads of single elements, each a whole line of a warp, and
// a batch of them before the first use: rows of an odd vocabulary begin
// anywhere, and three rows of one request differ in it.
//
// Few entries are worth an IEEE division: with a the product of w and the
// approximate reciprocal (off by less than 2^-21), an entry whose a is below
// (1 - 2^-19) of the warp's largest so far cannot win.  So a warp takes the
// largest a of a batch first and divides where a lane is near it; entries
// whose reciprocal leaves the normal range are always divided.
template <class T, int kCtas, int kThreads>
__device__ __forceinline__ uint64_t race(const T *__restrict__ p, const T *__restrict__ q, const float *__restrict__ e,
                                         int64_t n, int64_t skip, uint32_t rank) {
  constexpr int kBatch = kThreads == 512 ? 8 : 6, kStep = kCtas * kThreads;
  const int lane = threadIdx.x & 31;
  uint64_t best = 0;
  float highest = 0.0f;
  auto batch = [&](int64_t v0, auto is_whole) {  // entries v0 + lane + u * kStep (not whole: those below n)
    constexpr bool whole = decltype(is_whole)::value;
    T pv[kBatch], qv[kBatch];
    float w[kBatch], ev[kBatch];
    const T *pb = p + v0 + lane, *qb = q + v0 + lane;
    const float *eb = e + v0 + lane;
    const int64_t left = n - v0 - lane;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const bool in = whole || u * kStep < left;
      if (in) pv[u] = __ldcs(pb + u * kStep);
      if (in && q) qv[u] = __ldcs(qb + u * kStep);
      if (in) ev[u] = __ldcs(eb + u * kStep);
    }
    // 0: no weight; negative: to be divided in any case
    auto near_key = [](float wt, float x) {
      float r;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
      return !(wt > 0.0f) ? 0.0f : x >= 0x1p-125f && x <= 0x1p125f ? wt * r : -1.0f;
    };
    float top = 0.0f, low = 0.0f;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (!whole && u * kStep >= left) {
        w[u] = 0.0f, ev[u] = 1.0f;
        continue;
      }
      w[u] = q ? to_f32(pv[u]) - to_f32(qv[u]) : to_f32(pv[u]);
      if (v0 + lane + u * kStep == skip) w[u] = 0.0f;
      const float x = near_key(w[u], ev[u]);
      top = fmaxf(top, x);
      low = fminf(low, x);
    }
    highest = fmaxf(highest, __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top))));
    const float floor = highest > 1e-30f ? highest * (1.0f - 0x1p-19f) : 0.0f;
    if (low < 0.0f || (top >= floor && top > 0.0f)) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const float x = near_key(w[u], ev[u]);
        if (x < 0.0f || (x > 0.0f && x >= floor)) consider(best, w[u], ev[u], v0 + lane + u * kStep);
      }
    }
  };
  int64_t v0 = static_cast<int64_t>(rank) * kThreads + (threadIdx.x - lane);  // (the warp as one)
  for (; v0 + 31 + (kBatch - 1) * kStep < n; v0 += kBatch * kStep) batch(v0, std::true_type());
  if (v0 < n) batch(v0, std::false_type());
  return best;
}

__device__ __forceinline__ uint64_t warp_max(uint64_t x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const uint64_t y = __shfl_xor_sync(0xffffffffu, x, d);
    x = y > x ? y : x;
  }
  return x;
}

// The cluster's best: each CTA reduces its own and writes it to every CTA.
template <int kCtas, int kThreads>
__device__ __forceinline__ uint64_t cluster_best(uint64_t mine, uint64_t *own, uint64_t *all, uint32_t rank) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  mine = warp_max(mine);
  if (lane == 0) own[warp] = mine;
  __syncthreads();
  if (warp == 0) {
    const uint64_t b = warp_max(lane < kThreads / 32 ? own[lane] : 0);
    if (lane < kCtas)
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa_shared(smem_addr(all + rank), lane)), "l"(b) : "memory");
  }
  cluster_sync();
  uint64_t best = 0;
#pragma unroll
  for (int i = 0; i < kCtas; ++i) best = all[i] > best ? all[i] : best;
  return best;
}

// A cluster of 8 CTAs for each request: the row of the vocabulary is split
// over them and joined through their shared memory, one launch, no scratch.
// HBM bound with many requests, one row each of p, q and e (12 B an entry in
// fp32; 160 requests, 100277 entries, 193 MB: 36 us, 5.4 TB/s); latency bound
// with few (6 requests of 32000: 4.6 us), the drafted tokens' three dependent
// reads and the join.
// Up to 32 requests, whose clusters all run at once, CTAs have 512 threads, two
// an SM, and eight entries a thread in flight (6 requests of 32000 4.6 us, 30:
// 6.2, 10 of 151936: 10.3; the other shape 5.2, 6.8 and 15.1).  Beyond that they
// have 256 threads, five an SM, and six entries: what a CTA waits for at its
// start and end is hidden behind more others (36 us against 47; four an SM and
// eight entries 40, six an SM 36.5, eight an SM and four entries 38, clusters of
// four 37 to 44).
constexpr unsigned kFewRequests = 32;
template <class T, int kCtas, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 5 : 2) __cluster_dims__(kCtas, 1, 1)
    verify_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ uint64_t own[kThreads / 32], all[2][kCtas];
  __shared__ int s_kept;
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t rank = blockIdx.x;  // (a cluster is a row of the grid)
  const int64_t b = blockIdx.y;
  const int k = a.k, lane = threadIdx.x & 31;
  const int n = max(0, min(a.n_draft ? a.n_draft[b] : k, k));
  const T *target = static_cast<const T *>(a.target) + b * a.target_req;
  const T *draft = a.draft ? static_cast<const T *>(a.draft) + b * a.draft_req : nullptr;
  const int32_t *ids = a.tokens + b * a.tokens_stride;
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  if (threadIdx.x < 32) {  // kept drafted tokens
    int kept = n;
    for (int i0 = 0; i0 < k && kept == n; i0 += 32) {
      const int i = i0 + lane;
      bool pass = true;
      if (i < k) {  // (n may still be on its way)
        const int64_t x = ids[i];
        const float u = a.u[b * a.u_stride + i];
        const bool known = x >= 0 && x < a.vocab;
        const int64_t at = known ? x : 0;
        const float p = to_f32(target[i * a.target_row + at]);
        const float q = draft ? to_f32(draft[i * a.draft_row + at]) : 1.0f;
        pass = i >= n || (known && __fmul_rn(u, q) < p);
        if (i < n && !known) record_index(a.status);
      }
      const uint32_t refused = __ballot_sync(0xffffffffu, !pass);
      if (refused) kept = i0 + __ffs(refused) - 1;
    }
    if (lane == 0) s_kept = kept;
  }
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");  // (also the CTA's threads: every CTA of the cluster runs)
  __syncthreads();
  const int kept = s_kept;
  const T *p = target + static_cast<int64_t>(kept) * a.target_row;
  const T *q = draft ? draft + static_cast<int64_t>(kept) * a.draft_row : nullptr;
  const float *e = a.noise + b * a.noise_stride;
  uint64_t best = 0;
  // a draft without probabilities gave its token all of them: p without that token
  if (kept < n) best = cluster_best<kCtas, kThreads>(race<T, kCtas, kThreads>(p, q, e, a.vocab, q ? -1 : static_cast<int64_t>(ids[kept]), rank), own, all[0], rank);
  if (best == 0)  // nothing was refused, or p - q is nowhere positive
    best = cluster_best<kCtas, kThreads>(race<T, kCtas, kThreads>(p, nullptr, e, a.vocab, -1, rank), own, all[1], rank);
  if (rank != 0) return;
  const int drawn = best ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(best)) : -1;
  for (int i = threadIdx.x; i <= k; i += kThreads)
    a.out[b * (k + 1) + i] = i < kept ? ids[i] : i == kept ? drawn : -1;
  if (threadIdx.x == 0) a.accepted[b] = kept;
}

template <class T>
cudaError_t launch_verify_of(const VerifyArgs &a, cudaStream_t s) {
  const unsigned n = static_cast<unsigned>(a.nreq);
  if (n <= kFewRequests) return launch_early(verify_kernel<T, 8, 512>, 8, n, 512, 0, s, a);
  return launch_early(verify_kernel<T, 8, 256>, 8, n, 256, 0, s, a);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t s) {
  if (a.type == MMQ_DT_F32) return launch_verify_of<float>(a, s);
  return a.type == MMQ_DT_F16 ? launch_verify_of<__half>(a, s) : launch_verify_of<__nv_bfloat16>(a, s);
}

}  // namespace mmq
