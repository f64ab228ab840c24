// attention.cuh -- what the kernels of attention over a paged cache share: the
// arguments, and how the work of all requests is cut into units.
//
// Rows: the query heads that share a K/V head (`rep` of them) are rows of one
// problem, row = token * rep + head within the group, so K and V are read once
// for the whole group.  A unit is one K/V head, a run of `rows` rows of one
// request and a run of its K/V tiles ("piece").  Which units there are follows
// from the lengths, which only the device knows: a warp of every CTA works
// them out for itself and CTA c takes units c, c + grid, ...
#pragma once
#include <cuda_runtime.h>

#include <atomic>

#include "internal.h"
#include "ptx.cuh"

namespace mmq {

struct AttnArgs {
  const void *q, *k, *v;
  void *out;
  float *lse;
  const int32_t *table, *seq_lens, *q_start;
  float *part_o, *part_lse;  // partial results of split rows: [piece][token][q head][d], [piece][token][q head]
  int32_t *part_n;           // pieces of a row: [token][q head]
  int64_t q_token, q_head, out_token, out_head;
  int64_t k_page, k_token, k_head, v_page, v_token, v_head;
  int64_t table_stride, pages, ntok;
  int32_t nreq, table_width, page_size, hq, hkv, rep, d;
  int32_t causal, window, out_type;
  int32_t max_pieces;
  float scale_log2;  // scale * log2(e)
  WaitCtl wait;
};

// The part of one request that does not depend on the unit.
struct AttnRequest {
  int q0, n;       // first token, tokens
  int len;         // keys
  int tiles;       // row tiles
  int t_lo, n_kv;  // first K/V tile that any row sees, K/V tiles from there
};

template <int kKt>
__device__ __forceinline__ AttnRequest attn_request(const AttnArgs &a, int b, int rows) {
  AttnRequest r;
  const int ntok = static_cast<int>(a.ntok);
  r.q0 = max(0, min(a.q_start[b], ntok));
  r.n = max(r.q0, min(a.q_start[b + 1], ntok)) - r.q0;
  const int64_t room = static_cast<int64_t>(a.table_width) * a.page_size;
  int len = max(a.seq_lens[b], 0);
  if (len > room) {
    record_index(a.wait.status);
    len = static_cast<int>(room);
  }
  r.len = len;
  r.tiles = (r.n * a.rep + rows - 1) / rows;
  const int64_t lo = a.window ? max(static_cast<int64_t>(0), static_cast<int64_t>(len) - r.n - a.window + 1) : 0;
  r.t_lo = static_cast<int>(min(lo, static_cast<int64_t>(len))) / kKt;
  r.n_kv = max(0, (len + kKt - 1) / kKt - r.t_lo);
  return r;
}

struct AttnUnit {
  int q0, n, len, b, head;
  int row0;          // first row of the unit within the request
  int piece, pieces;
  int t_begin, t_end;  // K/V tiles (may be none)
};

// A row's keys: [lo, hi).
__device__ __forceinline__ void attn_row_range(const AttnArgs &a, int n, int len, int tok, int &lo, int &hi) {
  const int pos = len - n + tok;
  hi = a.causal ? max(0, min(len, pos + 1)) : len;
  lo = a.window ? max(0, pos - a.window + 1) : 0;
}

// Deals the units out; every lane of one warp calls each function.
template <int kKt>
struct AttnSchedule {
  int rows, cut;   // rows of a unit; K/V tiles of a piece
  int b0, before;  // first request of the lanes' 32, units before it
  int first;       // (lane) units of the lanes' requests before this one
  AttnRequest r;   // (lane)
  int pieces, each;

  // `slots` units run at once; `fixed`: a unit's cost beside its tiles, in tiles.
  // The cut is the one of eight with the least waves * (tiles + fixed).
  __device__ void plan(const AttnArgs &a, int unit_rows, int slots, int fixed) {
    rows = unit_rows;
    cut = 1 << 28;
    b0 = -32;
    before = 0;
    const int lane = threadIdx.x & 31;
    if (a.max_pieces > 1) {
      int64_t work = 0;
      int longest = 0;
      for (int b = lane; b < a.nreq; b += 32) {
        const AttnRequest q = attn_request<kKt>(a, b, rows);
        work += static_cast<int64_t>(q.tiles) * a.hkv * q.n_kv;
        if (q.tiles) longest = max(longest, q.n_kv);
      }
      for (int d = 16; d; d >>= 1) work += __shfl_xor_sync(0xffffffffu, work, d);
      longest = __reduce_max_sync(0xffffffffu, longest);
      const int even = max(1, static_cast<int>(min((work + slots - 1) / slots, static_cast<int64_t>(1) << 24)));
      int cand[8] = {even, even + (even + 7) / 8, even + (even + 3) / 4, even + (even + 1) / 2, 2 * even,
                     max(1, (even + 1) / 2), max(1, (even + 2) / 3), max(1, longest)};
      int units[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      for (int b = lane; b < a.nreq; b += 32) {
        const AttnRequest q = attn_request<kKt>(a, b, rows);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          units[i] += q.tiles * a.hkv * max(1, min(a.max_pieces, (q.n_kv + cand[i] - 1) / cand[i]));
      }
      int64_t least = INT64_MAX;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int u = __reduce_add_sync(0xffffffffu, units[i]);
        const int64_t cost = static_cast<int64_t>((u + slots - 1) / slots) * (min(cand[i], longest) + fixed);
        if (cost < least) least = cost, cut = cand[i];
      }
    }
    load(a, 0);
  }

  __device__ __forceinline__ void load(const AttnArgs &a, int from) {
    const int lane = threadIdx.x & 31;
    b0 = from;
    int units = 0;
    r = AttnRequest{0, 0, 0, 0, 0, 0};
    pieces = each = 1;
    if (b0 + lane < a.nreq) {
      r = attn_request<kKt>(a, b0 + lane, rows);
      if (r.n_kv > 0) {
        const int want = max(1, min(a.max_pieces, (r.n_kv + cut - 1) / cut));
        each = (r.n_kv + want - 1) / want;
        pieces = (r.n_kv + each - 1) / each;
      }
      units = r.tiles * pieces * a.hkv;
    }
    int sum = units;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, d);
      if ((threadIdx.x & 31) >= d) sum += y;
    }
    first = sum - units;
    total = __shfl_sync(0xffffffffu, sum, 31);
  }
  int total;  // units of the lanes' requests

  // Unit u (ascending from call to call); false when there are fewer.
  __device__ bool find(const AttnArgs &a, int u, AttnUnit &o) {
    while (u - before >= total) {
      if (b0 + 32 >= a.nreq) return false;
      before += total;
      load(a, b0 + 32);
    }
    int i = u - before;
    // the last request whose units begin at or before i (one without units begins where the next does)
    const uint32_t here = __ballot_sync(0xffffffffu, first <= i);
    const int l = 31 - __clz(here);
    i -= __shfl_sync(0xffffffffu, first, l);
    o.b = b0 + l;
    o.q0 = __shfl_sync(0xffffffffu, r.q0, l);
    o.n = __shfl_sync(0xffffffffu, r.n, l);
    o.len = __shfl_sync(0xffffffffu, r.len, l);
    o.pieces = __shfl_sync(0xffffffffu, pieces, l);
    const int run = __shfl_sync(0xffffffffu, each, l), tiles = __shfl_sync(0xffffffffu, r.tiles, l);
    const int t_lo = __shfl_sync(0xffffffffu, r.t_lo, l);
    o.head = i % a.hkv;
    i /= a.hkv;
    o.piece = i % o.pieces;
    o.row0 = (tiles - 1 - i / o.pieces) * rows;  // the rows that see most come first
    int lo, hi, none;
    attn_row_range(a, o.n, o.len, o.row0 / a.rep, lo, none);
    attn_row_range(a, o.n, o.len, min(o.n - 1, (o.row0 + rows - 1) / a.rep), none, hi);
    o.t_begin = max(t_lo + o.piece * run, lo / kKt);
    o.t_end = min(t_lo + (o.piece + 1) * run, (hi + kKt - 1) / kKt);
    if (o.t_end < o.t_begin) o.t_end = o.t_begin;
    return true;
  }
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLn2 = 0.693147180559945309f;

// Lets a kernel use `bytes` of dynamic shared memory on device `dev`, once.
template <auto kKernel>
cudaError_t allow_smem(int dev, int bytes) {
  static std::atomic<uint64_t> done{0};
  if (done.load(std::memory_order_relaxed) >> dev & 1) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(uint64_t(1) << dev);
  return e;
}

// The kernels' launches (attention.cu, attention_umma.cu).
cudaError_t launch_attention_rows(const AttnArgs &a, int type, int dev, unsigned grid, cudaStream_t s);
bool attention_umma_shape(const mmq_paged_cache &c, const mmq_attention &t, int *tile_tok, int *box);
cudaError_t launch_attention_umma(const AttnArgs &a, const mmq_paged_cache &c, int tile_tok, int box, int dev, unsigned grid,
                                  cudaStream_t s, bool *taken);

}  // namespace mmq
