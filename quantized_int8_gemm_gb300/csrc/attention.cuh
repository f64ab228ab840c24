// attention.cuh -- what the kernels of attention over a paged cache share: the
// arguments, and how the work of all requests is dealt to the CTAs.
//
// Rows: the query heads that share a K/V head (`rep` of them) are rows of one
// problem, row = token * rep + head within the group, so K and V are read once
// for the whole group.  A unit is a K/V head and a run of `rows` rows of one
// request, over the tiles of keys that its rows see.
//
// Which units there are follows from the lengths, which only the device
// knows.  All units' tiles are laid end to end, with a gap (`kGap` tiles) in
// front of each unit for what a unit costs beside its tiles, and each CTA
// takes an equal stretch of that line: a few long rows and many short ones
// then take every CTA the same time, and a CTA holds at most two pieces of
// units that others share.  A warp of every CTA works its stretch out by
// itself; with more than 32 requests the other warps add their room up first.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "internal.h"
#include "ptx.cuh"

namespace mmq {

// A unit cut into pieces: CTAs c .. last each left a partial result.
struct AttnCut {
  int q0, n, row0, head;
  int last;  // -1: no unit of CTA c is cut behind it
};

struct AttnArgs {
  const void *q, *k, *v;
  void *out;
  float *lse;
  const int32_t *table, *seq_lens, *q_start;
  // Partial results (fp32, normalised) of pieces, two slots a CTA: slot 2c + 1
  // of the unit that begins in CTA c and goes on, slot 2c of one that began
  // before it.  part_o [slot][d / 4][row of the unit] of 4 columns each,
  // part_lse [slot][row of the unit] to base 2, cuts [CTA].  Null: units stay whole.
  float4 *part_o;
  float *part_lse;
  AttnCut *cuts;
  int64_t q_token, q_head, out_token, out_head;
  int64_t k_page, k_token, k_head, v_page, v_token, v_head;
  int64_t table_stride, pages, ntok;
  int32_t nreq, table_width, page_size, hq, hkv, rep, d;
  int32_t causal, window, out_type;
  int32_t unit_tok;  // tokens of a unit (0: units are 64 rows, whatever their tokens)
  FastDiv by_page, by_rep, by_unit_tok, by_grid;
  float scale_log2;  // scale * log2(e)
  WaitCtl wait;
};

// The part of one request that does not depend on the unit.
struct AttnRequest {
  int q0, n;  // first token, tokens that q has rows for
  int place;  // of its first token among the keys (below 0 if it has more new tokens than keys)
  int len;    // keys that its rows see at most
};

struct AttnLengths {
  int from, to, len;
};
__device__ __forceinline__ AttnRequest attn_request(const AttnArgs &a, const AttnLengths &x) {
  AttnRequest r;
  const int ntok = static_cast<int>(a.ntok), from = x.from, to = x.to, len = x.len;
  r.q0 = max(0, min(from, ntok));
  r.n = max(r.q0, min(to, ntok)) - r.q0;
  if (to < from) record_index(a.wait.status);  // (then rows may be two requests', and the line longer than the host allowed for)
  // (a tile's keys are counted past the last one)
  const int64_t room = min(static_cast<int64_t>(a.table_width) * a.page_size, static_cast<int64_t>(0x7fffff00));
  r.len = max(len, 0);
  if (r.len > room) {
    record_index(a.wait.status);
    r.len = static_cast<int>(room);
  }
  // Places go by all of the request's new tokens, also those past q's rows (a
  // step whose tables counted more tokens than it has rows for); the keys end
  // where the last row's do, since nothing wrote those of the tokens behind it.
  r.place = r.len - (max(r.q0, to) - r.q0);
  if (a.causal) r.len = max(0, r.place + r.n);
  return r;
}

struct AttnUnit {
  int q0, n, place, len, b, head;
  int row0;            // first row of the unit within the request
  int from;            // first key that a row of the unit sees
  int t_begin, t_end;  // K/V tiles (may be none)
  int slot;            // of the partial result; -1: the unit is whole
};

// A row's keys: [lo, hi).
__device__ __forceinline__ void attn_row_range(const AttnArgs &a, int place, int len, int tok, int &lo, int &hi) {
  const int pos = place + tok;
  hi = a.causal ? max(0, min(len, pos + 1)) : len;
  lo = a.window && pos >= a.window ? pos - a.window + 1 : 0;  // (pos below 0 less a wide window would wrap)
}

constexpr int kAttnGap = 3;
constexpr int kAttnSums = 511;  // groups of requests at most

// Deals the units out; every lane of one warp calls each function.  kRows: of
// a unit, or 0 where units are whole tokens (AttnArgs::unit_tok).
template <int kKt, int kRows>
struct AttnSchedule {
  static constexpr int kGap = kAttnGap;
  static constexpr int kLeast = 2;  // tiles a CTA takes at least
  int b0;           // first of the 32 requests the lanes hold
  AttnRequest r;    // (lane)
  bool split;
  // Places on the line: 32 bits (the host has checked its length)
  int each;         // a CTA's stretch
  int lo, hi;       // this CTA's
  int pos;          // where the current unit begins
  int b, qt, head;  // the current unit; b >= nreq: none
  AttnRequest cur;  // its request

  // Row tiles of n tokens (worked out where they are wanted: the requests at
  // hand stay in registers beside the attention itself).
  __device__ static __forceinline__ int row_tiles(const AttnArgs &a, int n) {
    return kRows ? (n * a.rep + kRows - 1) / max(kRows, 1) : a.by_unit_tok(n + a.unit_tok - 1);
  }
  // K/V tiles of the rows of row tile q, and the first key that they see.
  __device__ __forceinline__ void tiles_of(const AttnArgs &a, const AttnRequest &x, int q, int &from, int &t0, int &t1) const {
    int to, none;
    const int first = kRows ? a.by_rep(q * kRows) : q * a.unit_tok;
    const int last = min(x.n, kRows ? a.by_rep((q + 1) * kRows - 1) + 1 : first + a.unit_tok) - 1;
    attn_row_range(a, x.place, x.len, first, from, none);
    attn_row_range(a, x.place, x.len, last, none, to);
    t0 = from / kKt;
    t1 = max(t0, (to + kKt - 1) / kKt);
  }
  // Room of one unit on the line.
  __device__ __forceinline__ int room_of(const AttnArgs &a, const AttnRequest &x, int q) const {
    int from, t0, t1;
    tiles_of(a, x, q, from, t0, t1);
    return kGap + max(1, t1 - t0);
  }
  __device__ __forceinline__ AttnRequest lane_request(int l) const {
    return {__shfl_sync(0xffffffffu, r.q0, l), __shfl_sync(0xffffffffu, r.n, l), __shfl_sync(0xffffffffu, r.place, l),
            __shfl_sync(0xffffffffu, r.len, l)};
  }
  __device__ static __forceinline__ AttnLengths lengths(const AttnArgs &a, int from) {
    const int at = from + static_cast<int>(threadIdx.x & 31);
    AttnLengths x{0, 0, 0};
    if (from >= 0 && at < a.nreq) x = {a.q_start[at], a.q_start[at + 1], a.seq_lens[at]};
    return x;
  }
  __device__ __forceinline__ void load(const AttnArgs &a, int from) {
    b0 = from;
    r = attn_request(a, lengths(a, from));
  }
  __device__ static __forceinline__ int inclusive(int x) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (static_cast<int>(threadIdx.x & 31) >= d) x += y;
    }
    return x;
  }
  // Room of the lane's request (all K/V heads), and the longest unit's.
  __device__ __forceinline__ int lane_room(const AttnArgs &a, int &longest) const {
    const int lane = threadIdx.x & 31;
    int sum = 0;
    const int own = row_tiles(a, r.n);
    if (own == 1) {
      sum = room_of(a, r, 0);
      longest = max(longest, sum);
    }
    uint32_t many = __ballot_sync(0xffffffffu, own > 1);
    while (many) {
      const int l = __ffs(many) - 1;
      many &= many - 1;
      const AttnRequest x = lane_request(l);
      const int tiles = __shfl_sync(0xffffffffu, own, l);
      int part = 0;
#pragma unroll 1
      for (int q = lane; q < tiles; q += 32) {
        const int y = room_of(a, x, q);
        part += y;
        longest = max(longest, y);
      }
      part = __reduce_add_sync(0xffffffffu, part);
      if (lane == l) sum = part;
    }
    return sum * a.hkv;
  }

  // Groups of requests whose rooms are added up ahead: 2^log2 requests each, 32 or more.
  __device__ static __forceinline__ int group_log2(const AttnArgs &a) {
    const uint32_t q = (static_cast<uint32_t>(a.nreq) - 1) / (32 * kAttnSums);  // (511 * 2^k >= nreq / 32 where 2^k > q)
    return 5 + (32 - __clz(q));
  }
  // One warp's part of the rooms of all requests, in shared memory: sums[i] of
  // group i = first, first + step, ...; sums[kAttnSums], 0 before, becomes the
  // longest unit's.
  __device__ __forceinline__ void add_up(const AttnArgs &a, int first, int step, int *sums) {
    const int log2 = group_log2(a), groups = ((a.nreq - 1) >> log2) + 1;
    int longest = 0;
    AttnLengths ahead{0, 0, 0};
    if (first < groups) ahead = lengths(a, first << log2);
#pragma unroll 1
    for (int i = first; i < groups; i += step) {
      int sum = 0;
#pragma unroll 1
      for (int j = 0; j < 1 << log2; j += 32) {
        const AttnLengths now = ahead;
        if (j + 32 < 1 << log2) ahead = lengths(a, (i << log2) + j + 32);
        else if (i + step < groups) ahead = lengths(a, (i + step) << log2);
        r = attn_request(a, now);
        sum += lane_room(a, longest);
      }
      sum = __reduce_add_sync(0xffffffffu, sum);
      if ((threadIdx.x & 31) == 0) sums[i] = sum;
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if ((threadIdx.x & 31) == 0) atomicMax(sums + kAttnSums, longest);
  }

  // This CTA's cut unit is none until next() finds one.  The join reads what
  // is told here even where this CTA gives up, so the warp that calls next()
  // comes here first, before anything that it waits for.
  __device__ static __forceinline__ void no_cut(const AttnArgs &a) {
    if (a.cuts && (threadIdx.x & 31) == 0) a.cuts[blockIdx.x].last = -1;
  }

  // Finds this CTA's stretch and the first unit that reaches into it.  With more
  // than 32 requests `sums` is what add_up left.
  __device__ __forceinline__ void plan(const AttnArgs &a, const int *sums) {
    const int lane = threadIdx.x & 31, log2 = group_log2(a), groups = ((a.nreq - 1) >> log2) + 1;
    int total = 0, mine = 0, longest = 0;
    if (groups > 1) {
      for (int i = lane; i < groups; i += 32) total += sums[i];
      longest = sums[kAttnSums];
    } else {
      load(a, 0);
      total = mine = lane_room(a, longest);
    }
    total = __reduce_add_sync(0xffffffffu, total);
    longest = __reduce_max_sync(0xffffffffu, longest);
    each = max(a.by_grid(total + static_cast<int>(gridDim.x) - 1), kLeast);
    // Whole units cost half the longest in balance, pieces their partial
    // results and the join (about four tiles' time).
    split = a.part_o && max(longest, each + longest / 2) > each + 4;
    lo = each * static_cast<int>(blockIdx.x);
    hi = lo + each;
    pos = 0;
    uint32_t past;
    if (groups > 1) {  // the group that reaches past lo
      int i = 0;
      for (;; i += 32) {
        mine = i + lane < groups ? sums[i + lane] : 0;
        const int end = inclusive(mine);
        past = __ballot_sync(0xffffffffu, pos + end > lo);
        if (past) {
          const int l = __ffs(past) - 1;
          pos += __shfl_sync(0xffffffffu, end - mine, l);
          load(a, (i + l) << log2);
          break;
        }
        pos += __shfl_sync(0xffffffffu, end, 31);
        if (i + 32 >= groups) {
          b = a.nreq;
          return;
        }
      }
      mine = lane_room(a, longest);
    }
    int end = inclusive(mine);
    while (!(past = __ballot_sync(0xffffffffu, pos + end > lo))) {
      pos += __shfl_sync(0xffffffffu, end, 31);
      if (b0 + 32 >= a.nreq) {
        b = a.nreq;
        return;
      }
      load(a, b0 + 32);
      mine = lane_room(a, longest);
      end = inclusive(mine);
    }
    int l = __ffs(past) - 1;
    pos += __shfl_sync(0xffffffffu, end - mine, l);
    b = b0 + l;
    cur = lane_request(l);
    qt = 0;
    const int tiles = row_tiles(a, cur.n);
    for (; tiles > 1; qt += 32) {  // (the request reaches past lo, so one of its row tiles does)
      mine = qt + lane < tiles ? room_of(a, cur, qt + lane) * a.hkv : 0;
      end = inclusive(mine);
      past = __ballot_sync(0xffffffffu, mine && pos + end > lo);
      if (past || qt + 32 >= tiles) break;
      pos += __shfl_sync(0xffffffffu, end, 31);
    }
    if (tiles > 1) {
      l = past ? __ffs(past) - 1 : 0;
      pos += __shfl_sync(0xffffffffu, end - mine, l);
      qt += l;
    }
    const int unit = room_of(a, cur, qt);
    head = lo > pos ? min((lo - pos) / unit, a.hkv - 1) : 0;  // (less than hkv anyway, unless row starts descend and places wrap)
    pos += head * unit;
  }

  __device__ __forceinline__ void step(const AttnArgs &a, int unit) {
    pos += unit;
    if (++head < a.hkv) return;
    head = 0;
    if (++qt < row_tiles(a, cur.n)) return;
    qt = 0;
    for (;;) {  // the next request with rows
      const int l = b + 1 - b0;
      const uint32_t rest = __ballot_sync(0xffffffffu, r.n > 0 && static_cast<int>(threadIdx.x & 31) >= l);
      if (rest) {
        b = b0 + __ffs(rest) - 1;
        cur = lane_request(__ffs(rest) - 1);
        return;
      }
      if (b0 + 32 >= a.nreq) {
        b = a.nreq;
        return;
      }
      load(a, b0 + 32);
      b = b0 - 1;
    }
  }

  // This CTA's next unit, or piece of one; false when there are no more.
  __device__ __forceinline__ bool next(const AttnArgs &a, AttnUnit &o) {
    while (b < a.nreq) {
      int from, t0, t1;
      tiles_of(a, cur, qt, from, t0, t1);
      const int unit = kGap + max(1, t1 - t0), first = pos + kGap, end = pos + unit;  // where its tiles lie
      if (first >= hi) break;
      o = {cur.q0, cur.n, cur.place, cur.len, b, head, qt * (kRows ? kRows : a.unit_tok * a.rep), from, t0, t1, -1};
      step(a, unit);
      if (!split) {
        if (first >= lo) return true;
        continue;
      }
      if (end <= lo) continue;
      const int me = blockIdx.x, c0 = first >= lo ? me : first / each, c1 = end <= hi ? me : (end - 1) / each;
      if (c0 == c1) return true;
      o.t_begin = t0 + max(0, lo - first);
      o.t_end = min(t1, t0 + (hi - first));
      const bool begins = c0 == me;
      o.slot = 2 * me + begins;
      if (begins && (threadIdx.x & 31) == 0) a.cuts[me] = {o.q0, o.n, o.row0, o.head, min(c1, static_cast<int>(gridDim.x) - 1)};
      return true;
    }
    return false;
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
// What the tcgen05 kernel needs beside the arguments; false: it does not take the problem.
struct AttnUmma {
  CUtensorMap q, k, v;
  int tile_tok;  // tokens of a row tile
  int box;       // keys of one copy
};
bool attention_umma(const AttnArgs &a, int type, AttnUmma *u);
cudaError_t launch_attention_umma(const AttnArgs &a, const AttnUmma &u, int type, int dev, unsigned grid, cudaStream_t s);

}  // namespace mmq
