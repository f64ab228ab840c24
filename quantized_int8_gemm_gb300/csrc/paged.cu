// paged.cu -- the bookkeeping of a paged K/V cache: page tables and slot maps
// from request lengths, and the rows of K and V written by those slots.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace mmq {
namespace {

// ---------------------------------------------------------------- page tables
constexpr int kTabThreads = 512;  // and tokens of a CTA

// Sums stop at 2^31 - 1 (for numbers that are not negative the order does not matter).
__device__ __forceinline__ int sat_add(int a, int b) {
  return static_cast<int>(min(static_cast<uint32_t>(a) + static_cast<uint32_t>(b), 0x7fffffffu));
}

// Exclusive sums over the CTA's threads of two values; returns the totals.
__device__ __forceinline__ void block_exclusive(int &a, int &b, int &ta, int &tb, int *sm) {
  constexpr int kWarps = kTabThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int ia = a, ib = b;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int ya = __shfl_up_sync(0xffffffffu, ia, d), yb = __shfl_up_sync(0xffffffffu, ib, d);
    if (lane >= d) ia = sat_add(ia, ya), ib = sat_add(ib, yb);
  }
  if (lane == 31) sm[warp] = ia, sm[kWarps + warp] = ib;
  ia = __shfl_up_sync(0xffffffffu, ia, 1), ib = __shfl_up_sync(0xffffffffu, ib, 1);
  if (lane == 0) ia = ib = 0;
  __syncthreads();
  int pa = 0, pb = 0;
  ta = tb = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int xa = sm[w], xb = sm[kWarps + w];
    if (w < warp) pa = sat_add(pa, xa), pb = sat_add(pb, xb);
    ta = sat_add(ta, xa);
    tb = sat_add(tb, xb);
  }
  a = sat_add(pa, ia);
  b = sat_add(pb, ib);
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

// A request's lengths and pages: `need` pages for cached + fresh tokens, of
// which it takes `more` from the free list; `lost` are beyond its table's row.
struct Pages {
  int cached, fresh, held, more, lost;
};
__device__ __forceinline__ Pages pages_of(const PageTablesArgs &a, int b) {
  Pages p;
  p.cached = max(a.cached[b], 0);
  p.fresh = max(a.fresh[b], 0);
  p.held = max(a.held[b], 0);
  const int width = static_cast<int>(a.table_width);
  // ceil(sum / page_size) in 32 bits: the sum is below 2^32
  const uint32_t sum = static_cast<uint32_t>(p.cached) + static_cast<uint32_t>(p.fresh), size = a.page_size;
  const int need = static_cast<int>(min(sum / size + (sum % size != 0), 0x7fffffffu));
  p.more = max(min(need, width) - p.held, 0);
  p.lost = max(need - max(p.held, width), 0);
  return p;
}

// One launch for everything.  Each CTA sums the requests' lengths by itself
// (nreq numbers, from L2) and so needs nothing from another CTA; it then takes
// its 512 tokens and its share of the new pages and finds each one's request by
// bisection in shared memory.  Latency bound: two rounds of reads from L2, a
// scan and about ten steps of bisection; the 12 B a token that it writes are
// 0.8 MB at 65536 tokens.
__global__ void __launch_bounds__(kTabThreads) page_tables_kernel(const __grid_constant__ PageTablesArgs a) {
  extern __shared__ int sums[];  // [nreq + 1] first token, [nreq + 1] first new page
  __shared__ int warp_sums[2 * kTabThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int n = a.nreq, tid = threadIdx.x;
  int *first_tok = sums, *first_page = sums + n + 1;
  constexpr int kKept = 2;  // requests of a thread that stay in registers
  const int per = (n + kTabThreads - 1) / kTabThreads, b0 = min(tid * per, n), b1 = min(b0 + per, n);
  int tok = 0, page = 0, tok_all, page_all;
  Pages kept[kKept];
#pragma unroll
  for (int i = 0; i < kKept; ++i) {
    kept[i] = Pages{0, 0, 0, 0, 0};
    if (b0 + i < b1) kept[i] = pages_of(a, b0 + i);
  }
#pragma unroll
  for (int i = 0; i < kKept; ++i) tok = sat_add(tok, kept[i].fresh), page = sat_add(page, kept[i].more);
  for (int b = b0 + kKept; b < b1; ++b) {
    const Pages p = pages_of(a, b);
    tok = sat_add(tok, p.fresh);
    page = sat_add(page, p.more);
  }
  block_exclusive(tok, page, tok_all, page_all, warp_sums);
  const int nfree = static_cast<int>(a.nfree);
  int lost = 0;
  auto place = [&](int b, const Pages &p) {
    first_tok[b] = tok;
    first_page[b] = page;
    if (blockIdx.x == 0) {
      a.q_start[b] = tok;
      a.seq_lens[b] = sat_add(p.cached, p.fresh);
      a.held_out[b] = p.held + max(min(p.more, nfree - page), 0);
    }
    tok = sat_add(tok, p.fresh);
    page = sat_add(page, p.more);
    lost = sat_add(lost, p.lost);
  };
#pragma unroll
  for (int i = 0; i < kKept; ++i)
    if (b0 + i < b1) place(b0 + i, kept[i]);
  for (int b = b0 + kKept; b < b1; ++b) place(b, pages_of(a, b));
  if (tid == 0) {
    first_tok[n] = tok_all;
    first_page[n] = page_all;
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    int zero = 0, lost_all, none;
    block_exclusive(lost, zero, lost_all, none, warp_sums);
    if (tid == 0) {
      a.q_start[n] = tok_all;
      a.taken[0] = min(page_all, nfree);
      a.taken[1] = sat_add(max(page_all - nfree, 0), lost_all);
    }
  }
  // tokens
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kTabThreads + tid;
  if (t < a.max_tokens) {
    int64_t slot = -1;
    int position = -1;
    if (t < tok_all) {
      const int b = last_not_above(first_tok, n, static_cast<int>(t));
      const int held = max(a.held[b], 0);
      const int64_t pos = static_cast<int64_t>(max(a.cached[b], 0)) + (static_cast<int>(t) - first_tok[b]);
      const int64_t blk = static_cast<uint32_t>(pos) / static_cast<uint32_t>(a.page_size);  // (pos is below 2^32)
      int id = -1;
      if (blk < a.table_width) {
        if (blk < held) {
          id = a.table[static_cast<int64_t>(b) * a.table_stride + blk];
        } else {
          const int64_t j = first_page[b] + (blk - held);
          if (j < nfree) id = a.free_pages[j];
        }
      }
      position = static_cast<int>(min(pos, static_cast<int64_t>(0x7fffffff)));
      if (id >= 0) slot = static_cast<int64_t>(id) * a.page_size + (pos - blk * a.page_size);
    }
    a.slots[t] = slot;
    a.positions[t] = position;
  }
  // new entries of the tables
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kTabThreads;  // (2^31 with the most token rows)
  for (int64_t j = static_cast<int64_t>(blockIdx.x) * kTabThreads + tid; j < page_all; j += stride) {
    const int b = last_not_above(first_page, n, static_cast<int>(j));
    const int at = max(a.held[b], 0) + (static_cast<int>(j) - first_page[b]);
    a.table[static_cast<int64_t>(b) * a.table_stride + at] = j < nfree ? a.free_pages[j] : -1;
  }
}

// ---------------------------------------------------------------- K and V rows
template <class T>
__device__ __forceinline__ void load8(const void *p, int64_t at, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<float>(const void *p, int64_t at, float (&x)[8]) {
  const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
  const float4 a = __ldcs(s), b = __ldcs(s + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__half>(const void *p, int64_t at, float (&x)[8]) {
  const uint4 r = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const __half *>(p) + at));
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const void *p, int64_t at, float (&x)[8]) {
  const uint4 r = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + at));
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

constexpr int kWriteThreads = 256;

// One thread moves 8 elements of a row at a time: 32 B (16 B) in, 16 B out.
// HBM bound (16384 tokens of 2 x 4 x 128 fp32 to bf16, one in nine padding: 15.8
// us, 5.7 TB/s of what it reads and writes); the one dependent read is the
// token's slot.  Two or four items of a thread in flight were slower (17.5 us,
// one 16.3 then): the CTAs of an SM hide the latency by themselves.  The source
// is read once (streaming loads), the cache rows are left in L2 for the
// attention that follows.
template <class S, class D>
__global__ void __launch_bounds__(kWriteThreads) kv_write_kernel(const __grid_constant__ KvWriteArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int chunks = a.head_dim >> 3, per_tensor = a.heads * chunks, per_tok = 2 * per_tensor;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens_per_cta;
  const int items = static_cast<int>(min(static_cast<int64_t>(a.tokens_per_cta), a.ntok - t0)) * per_tok;
  for (int i = threadIdx.x; i < items; i += kWriteThreads) {
    const int tl = a.by_items(i), r = i - tl * per_tok;
    const bool is_v = r >= per_tensor;
    const int c = is_v ? r - per_tensor : r, head = a.by_chunks(c), col = (c - head * chunks) << 3;
    const int64_t t = t0 + tl, slot = a.slots[t];
    float x[8];
    load8<S>(is_v ? a.v : a.k, is_v ? t * a.v_token + head * a.v_head + col : t * a.k_token + head * a.k_head + col, x);
    if (slot < 0) continue;  // padding
    if (slot >= a.cache.pages * a.cache.page_size) {
      record_index(a.status);
      continue;
    }
    int64_t page, row;
    if (slot <= 0x7fffffff) {
      page = a.by_page(static_cast<int>(slot)), row = static_cast<int>(slot) - static_cast<int>(page) * a.cache.page_size;
    } else {
      page = slot / a.cache.page_size, row = slot - page * a.cache.page_size;
    }
    uint4 o;
    o.x = pack2(x[0], x[1], D());
    o.y = pack2(x[2], x[3], D());
    o.z = pack2(x[4], x[5], D());
    o.w = pack2(x[6], x[7], D());
    D *dst = is_v ? static_cast<D *>(a.cache.v) + page * a.cache.v_page + row * a.cache.v_token + head * a.cache.v_head
                  : static_cast<D *>(a.cache.k) + page * a.cache.k_page + row * a.cache.k_token + head * a.cache.k_head;
    *reinterpret_cast<uint4 *>(dst + col) = o;
  }
}

template <class S>
cudaError_t launch_kv_write_from(const KvWriteArgs &a, unsigned grid, cudaStream_t s) {
  return launch_early(a.cache.type == MMQ_DT_F16 ? kv_write_kernel<S, __half> : kv_write_kernel<S, __nv_bfloat16>, grid, 1, kWriteThreads, 0, s, a);
}

}  // namespace

cudaError_t launch_page_tables(const PageTablesArgs &a, cudaStream_t s) {
  const size_t smem = 2 * (static_cast<size_t>(a.nreq) + 1) * sizeof(int);
  if (smem > 32 * 1024) {  // (beside the static arrays, within the 48 KB that need no leave)
    const cudaError_t e = cudaFuncSetAttribute(page_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * (kMaxRequests + 1) * 4);
    if (e != cudaSuccess) return e;
  }
  const int64_t ctas = (a.max_tokens + kTabThreads - 1) / kTabThreads;
  return launch_early(page_tables_kernel, static_cast<unsigned>(ctas > 0 ? ctas : 1), 1, kTabThreads, smem, s, a);
}

cudaError_t launch_kv_write(KvWriteArgs a, cudaStream_t s) {
  // about two items a thread, one where that would leave SMs idle; at least one token a CTA
  const int per_tok = 2 * a.heads * (a.head_dim >> 3);
  const bool many = a.ntok * per_tok >= static_cast<int64_t>(2 * kWriteThreads) * 152;
  a.tokens_per_cta = std::max(1, (many ? 2 : 1) * kWriteThreads / per_tok);
  a.by_items = FastDiv(per_tok), a.by_chunks = FastDiv(a.head_dim >> 3), a.by_page = FastDiv(a.cache.page_size);
  const int64_t grid = (a.ntok + a.tokens_per_cta - 1) / a.tokens_per_cta;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  if (a.src_type == MMQ_DT_F32) return launch_kv_write_from<float>(a, static_cast<unsigned>(grid), s);
  if (a.src_type == MMQ_DT_F16) return launch_kv_write_from<__half>(a, static_cast<unsigned>(grid), s);
  return launch_kv_write_from<__nv_bfloat16>(a, static_cast<unsigned>(grid), s);
}

}  // namespace mmq
