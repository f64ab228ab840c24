// checks.h -- host-side argument checks shared by the entry points of the
// serving step (serving.cu, requests.cu).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "mmq.h"

namespace mmq {

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
template <class... T>
bool aligned_elements(const T *...p) { return (aligned(p, alignof(T)) && ...); }
inline int cuda_rc(cudaError_t e) {
  if (e == cudaSuccess) return MMQ_OK;
  cudaGetLastError();
  return e == cudaErrorMemoryAllocation ? MMQ_ERR_OOM : e == cudaErrorNotSupported ? MMQ_ERR_UNSUPPORTED : MMQ_ERR_CUDA;
}
constexpr int64_t kInt32 = 0x7fffffff;

inline int check_cache(const mmq_paged_cache *c) {
  if (!c || !c->k || !c->v || c->pages < 1 || c->pages > kInt32 || c->page_size < 1 || c->heads < 1) return MMQ_ERR_ARG;
  if (c->head_dim < 8 || c->head_dim > 256 || c->head_dim % 8) return MMQ_ERR_ARG;
  if (c->type != MMQ_DT_F16 && c->type != MMQ_DT_BF16) return MMQ_ERR_TYPE;
  if (c->k_page < 0 || c->k_token < 0 || c->k_head < 0 || c->v_page < 0 || c->v_token < 0 || c->v_head < 0) return MMQ_ERR_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return MMQ_ERR_ALIGN;
  if ((c->k_page | c->k_token | c->k_head | c->v_page | c->v_token | c->v_head) % 8) return MMQ_ERR_ALIGN;
  return MMQ_OK;
}

// A run of bytes, or `rows` of them `pitch` apart.
struct Run {
  uintptr_t at;
  uint64_t bytes, pitch, rows;
  template <class T>
  Run(const T *p, int64_t n, int64_t stride = 0, int64_t count = 1)
      : at(reinterpret_cast<uintptr_t>(p)), bytes(n * sizeof(T)), pitch(stride * sizeof(T)), rows(count) {}
};
// Whether a (one run) and b share a byte: the first row of b that ends behind a's begin is the one to look at.
inline bool meet(const Run &a, const Run &b) {
  if (!a.bytes || !b.bytes || !b.rows) return false;
  const uint64_t r = a.at < b.at + b.bytes ? 0 : b.pitch ? (a.at - b.at - b.bytes) / b.pitch + 1 : b.rows;
  return r < b.rows && b.at + r * b.pitch < a.at + a.bytes;
}

}  // namespace mmq
