// pages.cu -- pages of a paged K/V cache shared, given back, moved and copied:
// the plans (which row holds which page, what is free, what has to be copied)
// and the copies.
//
// The plans keep no counts from call to call: what is held is read off the
// page table, as one bit a page.  Each CTA of a cluster sets the bits of its
// rows' pages in its own shared memory, the bits are joined through the
// cluster's, and ranks of pages (the j-th free one) are sums of population
// counts.  So every result follows from the table alone, in the order of the
// page ids and of the rows, whatever order the threads ran in.
#include <climits>

#include "internal.h"
#include "ptx.cuh"

namespace mmq {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kGroup = 8;  // words of bits whose population is summed as one
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_cluster4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void or_cluster(uint32_t addr, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
template <int kCtas>
__device__ __forceinline__ void sync_all() {
  if constexpr (kCtas == 1) __syncthreads();
  else cluster_sync();
}

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
  int mine = sm[lane], before = mine;  // (kWarps == 32)
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(kAll, before, d);
    if (lane >= d) before += y;
  }
  total = __shfl_sync(kAll, before, 31);
  const int up = __shfl_sync(kAll, before, warp > 0 ? warp - 1 : 0);
  __syncthreads();
  return (warp > 0 ? up : 0) + s - x;
}

// A CTA's share of table rows, by pieces of 32 kBatch entries, the rows' first ones
// first (with a warp a row the others waited for those with long rows: 500 rows
// compacted 18.4 us, so 16.1; 8 rows 6.1 and 4.5): f(row's index in the share, j,
// entry j) for this lane's j < limit(row), loaded kBatch at a time, and fill(row, j)
// from there to the width.  Where instead(entry) points to a number, that takes the
// entry's place (again kBatch loads at a time).  Few rows go by pieces of 128 (8 rows
// 4.5 us against 4.8), many by 256 (500 rows 16.1 against 18.2).
template <int kBatch, class N, class L, class I, class F, class E>
__device__ __forceinline__ void for_entries(int count, int width, N &&limit, L &&load, I &&instead, F &&f, E &&fill) {
  constexpr int kPiece = 32 * kBatch;  // (a width is 1023 below 2^31 - 1 at the most, so that j0 + kPiece does not wrap)
  const int lane = threadIdx.x & 31, pieces = (width + kPiece - 1) / kPiece;
  int r = threadIdx.x >> 5, j0 = lane;
  for (int k = 0; k < pieces * count; ++k) {
    while (r >= count) {
      r -= count, j0 += kPiece;
      if (j0 - lane >= width || count == 0) return;
    }
    const int n = limit(r);
    int id[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (j0 + 32 * u < n) id[u] = load(r, j0 + 32 * u);
    const int *from[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) from[u] = j0 + 32 * u < n ? instead(id[u]) : nullptr;
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (from[u]) id[u] = __ldcg(from[u]);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int j = j0 + 32 * u;
      if (j < n) f(r, j, id[u]);
      else if (j < width) fill(r, j);
    }
    r += kWarps;
  }
}

// Bits of pages: words of the whole cache, and those that one CTA of the
// cluster joins and ranks (whole groups).
struct Bits {
  int words, slice;
  __host__ __device__ Bits(int64_t pages, int ctas) {
    words = static_cast<int>((pages + 31) / 32);
    slice = (words + ctas - 1) / ctas;
    slice = (slice + kGroup - 1) / kGroup * kGroup;
  }
};

__device__ __forceinline__ void set_bit(uint32_t *words, int id) { atomicOr(&words[id >> 5], 1u << (id & 31)); }

// The cluster's words of this CTA's slice, joined.
template <int kCtas>
__device__ __forceinline__ uint32_t joined(const uint32_t *own, int at) {
  if constexpr (kCtas == 1) return own[at];
  uint32_t v[kCtas], got = 0;
#pragma unroll
  for (int c = 0; c < kCtas; ++c) v[c] = ld_cluster(mapa_shared(smem_addr(own + at), c));
#pragma unroll
  for (int c = 0; c < kCtas; ++c) got |= v[c];
  return got;
}

// Writes v to entry `rank` of every CTA's array.
template <int kCtas>
__device__ __forceinline__ void tell_all(int *array, int rank, int v) {
  if (threadIdx.x < kCtas) {
    if constexpr (kCtas == 1) array[0] = v;
    else st_cluster(mapa_shared(smem_addr(array + rank), threadIdx.x), v);
  }
}

// Rows of a page table made anew (see mmq.h).  A thread has one row of the new
// table, its warps the entries.  Latency bound: the entries are read and
// written once (2 MB for 700 rows of 9000 tokens in pages of 16), between them
// are six joins of the cluster.
template <int kCtas>
__global__ void __launch_bounds__(kThreads) fork_kernel(const __grid_constant__ ForkArgs a) {
  extern __shared__ __align__(16) uint32_t bits[];
  __shared__ int s_parent[kThreads], s_full[kThreads], s_need[kThreads], s_target[kThreads], s_warp[kWarps];
  __shared__ int s_copies[kCtas], s_free[kCtas];
  const Bits n(a.npages, kCtas);
  uint32_t *own = bits, *full = own + n.words, *held = full + n.slice;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = kCtas == 1 ? 0 : static_cast<int>(cluster_ctarank()), npages = static_cast<int>(a.npages);
  const int width = static_cast<int>(a.table_width), nnew = static_cast<int>(a.nnew);
  const int per = (nnew + kCtas - 1) / kCtas, b0 = min(rank * per, nnew), mine = min(per, nnew - b0), b = b0 + tid;
  for (int i = tid; i < n.words; i += kThreads) own[i] = 0;
  griddep_wait();
  griddep_launch_dependents();
  // my row: w is its writable page, -1 if it has none
  int need = 0, nfull = 0, w = -1, left = 0;
  if (tid < mine) {
    const int p = a.parents[b], length = max(a.lens[b], 0);
    if (p >= 0 && p < a.nold) {
      const int has = min(max(a.held[p], 0), width), whole = length / a.page_size, over = length - whole * a.page_size;
      const int want = whole + (over > 0);
      need = min(want, has), nfull = min(whole, has);
      if (want > has) record_index(a.status);
      if (over > 0 && whole < need) {
        w = a.table[p * a.table_stride + whole];
        left = over;
        if (w < 0 || w >= npages) record_index(a.status), w = -1;
      }
    } else if (p != -1) {
      record_index(a.status);
    }
    if (w >= 0) a.free_pages[w] = INT_MAX;  // lowest row that has this page as its writable one
    s_parent[tid] = p, s_full[tid] = nfull, s_need[tid] = need;
  }
  sync_all<kCtas>();
  if (w >= 0) atomicMin(&a.free_pages[w], b);
  for_entries<kCtas == 1 ? 4 : 8>(
      mine, width, [&](int r) { return s_full[r]; }, [&](int r, int j) { return a.table[s_parent[r] * a.table_stride + j]; },
      [](int) -> const int * { return nullptr; },
      [&](int r, int j, int id) {
        if (id >= 0 && id < npages) set_bit(own, id);
        else record_index(a.status), id = -1;
        a.new_table[(b0 + r) * a.new_stride + j] = id;
      },
      [&](int r, int j) {  // (the writable page: its row's thread writes it)
        if (j >= s_need[r]) a.new_table[(b0 + r) * a.new_stride + j] = -1;
      });
  sync_all<kCtas>();
  const int w0 = min(rank * n.slice, n.words), words = min(n.slice, n.words - w0);
  for (int i = tid; i < n.slice; i += kThreads) full[i] = held[i] = i < words ? joined<kCtas>(own, w0 + i) : 0;
  sync_all<kCtas>();
  bool copy = false;
  if (w >= 0) {
    const int owner = (w >> 5) / n.slice, at = (w >> 5) - owner * n.slice;
    const uint32_t bit = 1u << (w & 31);
    const uint32_t others = kCtas == 1 ? full[at] : ld_cluster(mapa_shared(smem_addr(full + at), owner));
    copy = (others & bit) || __ldcg(&a.free_pages[w]) != b;
    if (!copy) {
      if constexpr (kCtas == 1) atomicOr(&held[at], bit);
      else or_cluster(mapa_shared(smem_addr(held + at), owner), bit);
    }
  }
  int copies_here;
  const int nth = block_exclusive(copy, copies_here, s_warp);
  tell_all<kCtas>(s_copies, rank, copies_here);
  sync_all<kCtas>();
  // free pages of my slice, by groups
  const int groups = n.slice / kGroup;
  auto free_word = [&](int i) {
    const int id0 = (w0 + i) * 32;
    if (i >= words) return 0u;
    return ~held[i] & (npages - id0 >= 32 ? kAll : (1u << (npages - id0)) - 1);
  };
  int free_group = 0, free_here;
  if (tid < groups)
#pragma unroll
    for (int i = 0; i < kGroup; ++i) free_group += __popc(free_word(tid * kGroup + i));
  const int before = block_exclusive(free_group, free_here, s_warp);
  if (tid < groups) full[tid] = before;  // (nobody reads the bits there any more)
  tell_all<kCtas>(s_free, rank, free_here);
  sync_all<kCtas>();
  int base = 0, total = 0, copies = 0;
#pragma unroll
  for (int c = 0; c < kCtas; ++c) {
    base += c < rank ? s_free[c] : 0;
    total += s_free[c], copies += s_copies[c];
  }
  // the lowest free pages go to the copies, the others to the list
  for (int g = warp; g < groups; g += kWarps) {
    int at = base + static_cast<int>(full[g]);
    for (int i = g * kGroup; i < (g + 1) * kGroup; ++i) {
      const uint32_t f = free_word(i);
      const int k = at + __popc(f & ((1u << lane) - 1)), id = (w0 + i) * 32 + lane;
      at += __popc(f);
      if (!(f >> lane & 1)) continue;
      if (k >= copies) {
        a.free_pages[k - copies] = id;
        continue;
      }
      int of = 0, first = 0;  // the CTA whose row takes it
#pragma unroll
      for (int c = 0; c < kCtas - 1; ++c)
        if (k >= first + s_copies[c] && of == c) first += s_copies[c], of = c + 1;
      if constexpr (kCtas == 1) s_target[k] = id;
      else st_cluster(mapa_shared(smem_addr(s_target + (k - first)), of), id);
    }
  }
  const int listed = max(total - copies, 0);
  for (int i = listed + rank * kThreads + tid; i < npages; i += kCtas * kThreads) a.free_pages[i] = -1;
  sync_all<kCtas>();
  if (rank == 0 && tid == 0) a.counts[0] = listed, a.counts[1] = max(copies - total, 0);
  if (tid < mine) {
    int first = 0;
#pragma unroll
    for (int c = 0; c < kCtas; ++c) first += c < rank ? s_copies[c] : 0;
    const int to = copy && first + nth < total ? s_target[nth] : -1;
    if (nfull < need) a.new_table[b * a.new_stride + nfull] = copy ? to : w;
    a.held_out[b] = need;
    a.pairs[2 * b] = to >= 0 ? w : -1, a.pairs[2 * b + 1] = to;
    a.tokens[b] = to >= 0 ? left : 0;
  }
}

// Moves that bring the held pages to the front (see mmq.h), and the table
// after them.  Latency bound: the entries are read twice (the second time from
// L2) and written once.
template <int kCtas>
__global__ void __launch_bounds__(kThreads) compact_kernel(const __grid_constant__ CompactArgs a) {
  extern __shared__ __align__(16) uint32_t bits[];
  __shared__ int s_warp[kWarps], s_held[kCtas], s_below;
  const Bits n(a.npages, kCtas);
  const int all_groups = kCtas * n.slice / kGroup, groups = n.slice / kGroup;
  // bits of the whole cache (first this CTA's rows', later everyone's), of my
  // slice, pages held before each word within its group (up to 224), before each group of my
  // slice, of the whole cache
  uint32_t *own = bits, *held = own + kCtas * n.slice;
  uint8_t *word_before = reinterpret_cast<uint8_t *>(held + n.slice);
  int *mine_before = reinterpret_cast<int *>(word_before + kCtas * n.slice), *all_before = mine_before + groups;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = kCtas == 1 ? 0 : static_cast<int>(cluster_ctarank()), npages = static_cast<int>(a.npages);
  const int width = static_cast<int>(a.table_width), nreq = static_cast<int>(a.nreq);
  for (int i = tid; i < kCtas * n.slice; i += kThreads) own[i] = 0;
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  const int mine = rank < nreq ? (nreq - rank + kCtas - 1) / kCtas : 0;  // rows rank, rank + kCtas, ...
  auto row_of = [&](int r) { return rank + static_cast<int64_t>(r) * kCtas; };
  auto limit = [&](int r) { return min(max(a.held[row_of(r)], 0), width); };
  auto load = [&](int r, int j) { return a.table[row_of(r) * a.table_stride + j]; };
  for_entries<kCtas == 1 ? 4 : 8>(
      mine, width, limit, load, [](int) -> const int * { return nullptr; },
      [&](int, int, int id) {
        if (id >= 0 && id < npages) set_bit(own, id);
        else record_index(a.status);
      },
      [&](int r, int j) { a.new_table[row_of(r) * a.new_stride + j] = -1; });
  sync_all<kCtas>();
  for (int i = tid; i < n.slice; i += kThreads) held[i] = joined<kCtas>(own, rank * n.slice + i);
  __syncthreads();
  int held_group = 0, held_here;
  if (tid < groups)
#pragma unroll
    for (int i = 0; i < kGroup; ++i) held_group += __popc(held[tid * kGroup + i]);
  const int before = block_exclusive(held_group, held_here, s_warp);
  if (tid < groups) mine_before[tid] = before;
  tell_all<kCtas>(s_held, rank, held_here);
  sync_all<kCtas>();
  int base = 0, total = 0;
#pragma unroll
  for (int c = 0; c < kCtas; ++c) base += c < rank ? s_held[c] : 0, total += s_held[c];
  // everyone's bits and sums: two warps take each CTA's
  {
    constexpr int kThreadsEach = kThreads / kCtas;
    const int c = tid / kThreadsEach;
    const uint32_t words_of = kCtas == 1 ? smem_addr(held) : mapa_shared(smem_addr(held), c);
    const uint32_t sums_of = kCtas == 1 ? smem_addr(mine_before) : mapa_shared(smem_addr(mine_before), c);
    int sum = 0;
#pragma unroll
    for (int k = 0; k < kCtas; ++k) sum += k < c ? s_held[k] : 0;
#pragma unroll 2
    for (int g = tid % kThreadsEach; g < groups; g += kThreadsEach) {
      uint4 half[2];
      int first;
      if constexpr (kCtas == 1) {
        half[0] = reinterpret_cast<const uint4 *>(held)[2 * g], half[1] = reinterpret_cast<const uint4 *>(held)[2 * g + 1], first = mine_before[g];
      } else {
        half[0] = ld_cluster4(words_of + 32 * g), half[1] = ld_cluster4(words_of + 32 * g + 16), first = static_cast<int>(ld_cluster(sums_of + 4 * g));
      }
      const int at = c * groups + g;
      uint32_t in_group[2], here = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t w[4] = {half[h].x, half[h].y, half[h].z, half[h].w};
        in_group[h] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) in_group[h] |= here << (8 * i), here += __popc(w[i]);
        reinterpret_cast<uint4 *>(own)[2 * at + h] = half[h];
      }
      reinterpret_cast<uint2 *>(word_before)[at] = make_uint2(in_group[0], in_group[1]);
      all_before[at] = sum + first;
    }
  }
  __syncthreads();
  auto held_before = [&](int id) {  // pages held below id (id <= npages, within the words there are)
    const int word = id >> 5, g = word / kGroup;
    return all_before[g] + word_before[word] + __popc(own[word] & ((1u << (id & 31)) - 1));
  };
  if (tid == 0) s_below = total < kCtas * n.slice * 32 ? held_before(total) : total;
  __syncthreads();
  const int below = s_below, moves = total - below, room = npages / 2;
  for (int g = warp; g < groups; g += kWarps) {
    int at = base + mine_before[g];
    for (int i = g * kGroup; i < (g + 1) * kGroup; ++i) {
      const uint32_t h = held[i];
      const int id = (rank * n.slice + i) * 32 + lane, k = at + __popc(h & ((1u << lane) - 1));
      at += __popc(h);
      if (id >= npages) continue;
      if (h >> lane & 1) {
        if (id >= total) a.pairs[2 * (k - below)] = id;
      } else if (id < total) {
        a.pairs[2 * (id - k) + 1] = id;
      }
    }
  }
  for (int i = moves + rank * kThreads + tid; i < room; i += kCtas * kThreads) reinterpret_cast<int2 *>(a.pairs)[i] = make_int2(-1, -1);
  if (rank == 0 && tid == 0) a.counts[0] = total, a.counts[1] = moves;
  sync_all<kCtas>();
  for_entries<kCtas == 1 ? 4 : 8>(
      mine, width, limit, load,
      [&](int id) -> const int * { return id >= total && id < npages ? &a.pairs[2 * (held_before(id) - below) + 1] : nullptr; },
      [&](int r, int j, int id) { a.new_table[row_of(r) * a.new_stride + j] = id < 0 || id >= npages ? -1 : id; },
      [&](int, int) {});
}

// ---------------------------------------------------------------- copies
constexpr int kCopyThreads = 256, kCopyEach = 4;

// 16 B an item, four items of a thread in flight; the items of a page lie in
// the order of its memory (K's), so that a warp's are neighbours.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ PageCopyArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t pair = a.parts == 1 ? blockIdx.x : blockIdx.x / static_cast<unsigned>(a.parts);
  const int part = static_cast<int>(blockIdx.x - pair * a.parts);
  const int from = a.pairs[2 * pair], to = a.pairs[2 * pair + 1];
  const int tokens = a.tokens ? min(max(a.tokens[pair], 0), a.cache.page_size) : a.cache.page_size;
  if (from < 0 || to < 0) return;
  if (from >= a.cache.pages || to >= a.cache.pages) {
    if (threadIdx.x == 0) record_index(a.status);
    return;
  }
  uint4 x[kCopyEach];
  uint4 *dst[kCopyEach];
#pragma unroll
  for (int u = 0; u < kCopyEach; ++u) {
    int i = (part * kCopyEach + u) * kCopyThreads + static_cast<int>(threadIdx.x);
    const bool is_v = i >= a.per_tensor;
    if (is_v) i -= a.per_tensor;
    dst[u] = nullptr;
    if (i >= a.per_tensor) continue;
    const int outer = a.by_outer(i), rest = i - outer * a.outer_items, inner = a.by_chunks(rest), col = (rest - inner * a.chunks) << 3;
    const int t = a.token_outer ? outer : inner, head = a.token_outer ? inner : outer;
    if (t >= tokens) continue;
    const int64_t in_page = is_v ? t * a.cache.v_token + head * a.cache.v_head + col : t * a.cache.k_token + head * a.cache.k_head + col;
    uint16_t *p = static_cast<uint16_t *>(is_v ? a.cache.v : a.cache.k);
    const int64_t pitch = is_v ? a.cache.v_page : a.cache.k_page;
    x[u] = __ldcs(reinterpret_cast<const uint4 *>(p + from * pitch + in_page));
    dst[u] = reinterpret_cast<uint4 *>(p + to * pitch + in_page);
  }
#pragma unroll
  for (int u = 0; u < kCopyEach; ++u)
    if (dst[u]) *dst[u] = x[u];
}

// most: bytes of shared memory of the largest cache, for every call.
template <class K, class A>
cudaError_t launch_cluster(K kernel, unsigned ctas, size_t smem, size_t most, cudaStream_t s, const A &a) {
  cudaError_t e = cudaSuccess;
  if (ctas > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && smem > 24 * 1024)  // (beside the static arrays, within the 48 KB that need no leave)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
  return e != cudaSuccess ? e : launch_early(kernel, Cluster{ctas}, ctas, 1, kThreads, smem, s, a);
}

// One CTA for few entries of the table, or a cluster of sixteen.  Forks of 64 rows of
// 128 pages take 8.6 us by one and 9.5 by sixteen, of 64 rows of 256 11.2 and 9.8;
// compactions, which go over the entries twice, of 32 rows of 128 6.0 and 7.1, of 64
// rows of 128 9.9 and 7.2.
constexpr int kMany = 16;
constexpr int64_t kForked = 8192, kMoved = 4096;
constexpr int64_t kFewPages = 32768;
bool one_cta(int64_t rows, int64_t width, int64_t npages, int64_t entries) {
  return rows <= kThreads && rows * width <= entries && npages <= kFewPages;
}
constexpr int64_t most_pages(int ctas) { return ctas == 1 ? kFewPages : kMaxPages; }

size_t fork_bytes(int64_t pages, int ctas) {
  const Bits n(pages, ctas);
  return sizeof(uint32_t) * (n.words + 2 * static_cast<size_t>(n.slice));
}
template <int kCtas>
cudaError_t launch_fork_with(const ForkArgs &a, cudaStream_t s) {
  return launch_cluster(fork_kernel<kCtas>, kCtas, fork_bytes(a.npages, kCtas), fork_bytes(most_pages(kCtas), kCtas), s, a);
}

size_t compact_bytes(int64_t pages, int ctas) {
  const Bits n(pages, ctas);
  const size_t groups = n.slice / kGroup;
  return sizeof(uint32_t) * ((ctas + 1) * static_cast<size_t>(n.slice) + (ctas + 1) * groups) + ctas * static_cast<size_t>(n.slice);
}
template <int kCtas>
cudaError_t launch_compact_with(const CompactArgs &a, cudaStream_t s) {
  return launch_cluster(compact_kernel<kCtas>, kCtas, compact_bytes(a.npages, kCtas), compact_bytes(most_pages(kCtas), kCtas), s, a);
}

}  // namespace

cudaError_t launch_page_fork(const ForkArgs &a, cudaStream_t s) {
  return one_cta(a.nnew, a.table_width, a.npages, kForked) ? launch_fork_with<1>(a, s) : launch_fork_with<kMany>(a, s);
}

cudaError_t launch_page_compact(const CompactArgs &a, cudaStream_t s) {
  return one_cta(a.nreq, a.table_width, a.npages, kMoved) ? launch_compact_with<1>(a, s) : launch_compact_with<kMany>(a, s);
}

cudaError_t launch_page_copy(PageCopyArgs a, cudaStream_t s) {
  const mmq_paged_cache &c = a.cache;
  a.chunks = c.head_dim >> 3;
  a.token_outer = c.k_token >= c.k_head;
  a.outer_items = (a.token_outer ? c.heads : c.page_size) * a.chunks;
  a.per_tensor = c.page_size * c.heads * a.chunks;
  a.by_chunks = FastDiv(a.chunks), a.by_outer = FastDiv(a.outer_items);
  constexpr int kPer = kCopyThreads * kCopyEach;
  a.parts = static_cast<int>((2 * static_cast<int64_t>(a.per_tensor) + kPer - 1) / kPer);
  if (a.npairs > 0x7fffffff / a.parts) return cudaErrorNotSupported;
  return launch_early(copy_kernel, static_cast<unsigned>(a.npairs * a.parts), 1, kCopyThreads, 0, s, a);
}

}  // namespace mmq
