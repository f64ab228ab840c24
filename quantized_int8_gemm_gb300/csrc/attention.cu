// attention.cu -- attention of new tokens over the paged cache: the general
// kernel (warp-level MMA, any page size and head width up to 256), the join of
// split rows, and the choice between the kernels.
//
//   S = scale * q . k over the keys a row sees,  out = softmax(S) . v,
//   lse = log(sum exp(S));  a row that sees nothing: out 0, lse -inf.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "attention.cuh"

namespace mmq {
namespace {

template <class T>
struct Pair;
template <>
struct Pair<__half> {
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <>
struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 16 bytes, or (bytes == 0) 16 zeros
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

constexpr int kRows = 64, kKt = 64, kThreads = 128;
constexpr int kSms = 152;

// Byte offset of 16-byte chunk c of row r in a tile of kDp-wide rows; the
// swizzle keeps the eight rows of an ldmatrix on different banks.
template <int kDp>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  return static_cast<uint32_t>(r * kDp * 2 + (((c & ~7) | ((c ^ r) & 7)) << 4));
}

// The general kernel.  A unit: 64 rows, 16 a warp, over K/V tiles of 64 keys,
// double-buffered copies (cp.async, zeros for what lies past the request's
// last key or behind the rows' windows, so that what unwritten or reused memory
// holds never meets the tensor core).
// S and P stay in registers; the running maximum, sum and the output are
// fp32, P is rounded to the cache's type for the second product.  It serves
// the shapes the tcgen05 kernel does not take: heads wider than 128, pages
// without eight keys in a row, groups of more than 128 query heads.  Bound by
// the latency of one warp's products where few rows are at work (16 q heads
// over 4 K/V heads of 256, 32 tokens over 4001 keys: 137 us, 3.8 TB/s) and by
// the warp-level tensor rate beside the softmax in chunks (512 tokens over 4608
// keys: 147 us, 250 TFLOP/s).
template <class T, int kDp>
__global__ void __launch_bounds__(kThreads) attention_rows_kernel(const __grid_constant__ AttnArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ AttnUnit s_unit;
  __shared__ int s_more, s_sums[kAttnSums + 1];
  constexpr int kChunks = kDp / 8;
  constexpr int kTile = kKt * kDp * 2;
  const uint32_t sq = smem_addr(smem), sk = sq + kRows * kDp * 2, sv = sk + 2 * kTile;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  AttnSchedule<kKt, kRows> sched;
  griddep_wait();
  griddep_launch_dependents();
  if (warp == 0) sched.no_cut(a);
  if (a.nreq > 32) {
    if (tid == 0) s_sums[kAttnSums] = 0;
    __syncthreads();
    sched.add_up(a, warp, kThreads / 32, s_sums);
    __syncthreads();
  }
  if (warp == 0) sched.plan(a, s_sums);

  for (;;) {
    if (warp == 0) {
      AttnUnit x;
      const bool more = sched.next(a, x);
      if (lane == 0) {
        s_more = more;
        if (more) s_unit = x;
      }
    }
    __syncthreads();
    if (!s_more) break;
    const AttnUnit un = s_unit;
    const int all_rows = un.n * a.rep;
    const T *q = static_cast<const T *>(a.q);
    for (int i = tid; i < kRows * kChunks; i += kThreads) {
      const int r = i / kChunks, c = i % kChunks, row = un.row0 + r;
      const bool in = row < all_rows && c * 8 < a.d;
      const int tok = a.by_rep(row);
      const T *src = in ? q + (un.q0 + tok) * a.q_token + (un.head * a.rep + row - tok * a.rep) * a.q_head + c * 8 : q;
      cp_async16(sq + tile_at<kDp>(r, c), src, in ? 16 : 0);
    }
    // A warp copies 16 keys of a tile: 16 lanes look their keys' rows up, then
    // each copy takes its row's place from its lane.
    auto load = [&](int t, int buf) {
      const int key = t * kKt + warp * 16 + (lane & 15);
      int64_t k_at = -1, v_at = -1;
      if (key >= un.from && key < un.len) {
        const int blk = a.by_page(key), off = key - blk * a.page_size;
        const int64_t page = a.table[un.b * a.table_stride + blk];
        if (page >= 0 && page < a.pages) {
          k_at = page * a.k_page + off * a.k_token + un.head * a.k_head;
          v_at = page * a.v_page + off * a.v_token + un.head * a.v_head;
        } else {
          record_index(a.wait.status);
        }
      }
      constexpr int kRowsAtOnce = 32 / kChunks;
      const int c = lane % kChunks;
      const T *k = static_cast<const T *>(a.k) + c * 8, *v = static_cast<const T *>(a.v) + c * 8;
#pragma unroll
      for (int i = 0; i < 16; i += kRowsAtOnce) {
        const int at = i + lane / kChunks;
        const int64_t ko = __shfl_sync(0xffffffffu, k_at, at), vo = __shfl_sync(0xffffffffu, v_at, at);
        const bool in = ko >= 0 && c * 8 < a.d;
        const uint32_t to = buf * kTile + tile_at<kDp>(warp * 16 + at, c);
        cp_async16(sk + to, in ? k + ko : a.k, in ? 16 : 0);
        cp_async16(sv + to, in ? v + vo : a.v, in ? 16 : 0);
      }
    };
    if (un.t_begin < un.t_end) load(un.t_begin, 0);
    cp_async_commit();

    float o[kDp / 8][4];
#pragma unroll
    for (int j = 0; j < kDp / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    int lo[2], hi[2];
    // (from shared memory, not from the copy in registers, of which the loop has none to spare: 119.5 against 123.2 us for
    // 512 tokens over 4608 keys, pages of 5)
#pragma unroll
    for (int h = 0; h < 2; ++h) attn_row_range(a, s_unit.place, s_unit.len, a.by_rep(s_unit.row0 + warp * 16 + (lane >> 2) + 8 * h), lo[h], hi[h]);

    for (int t = un.t_begin; t < un.t_end; ++t) {
      const int buf = (t - un.t_begin) & 1;
      if (t + 1 < un.t_end) load(t + 1, buf ^ 1);
      cp_async_commit();
      cp_async_wait<1>();
      __syncthreads();
      float s[kKt / 8][4];
#pragma unroll
      for (int j = 0; j < kKt / 8; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.0f;
#pragma unroll
      for (int kk = 0; kk < kDp / 16; ++kk) {
        uint32_t qa[4];
        ldmatrix_x4(qa, sq + tile_at<kDp>(warp * 16 + (lane & 15), 2 * kk + (lane >> 4)));
#pragma unroll
        for (int j = 0; j < kKt / 16; ++j) {
          uint32_t kb[4];
          ldmatrix_x4(kb, sk + buf * kTile + tile_at<kDp>(j * 16 + (lane & 7) + ((lane >> 4) << 3), 2 * kk + ((lane >> 3) & 1)));
          Pair<T>::mma(s[2 * j], qa, kb[0], kb[1]);
          Pair<T>::mma(s[2 * j + 1], qa, kb[2], kb[3]);
        }
      }
      const int key0 = t * kKt + 2 * (lane & 3);
      float top[2] = {m[0], m[1]};
#pragma unroll
      for (int j = 0; j < kKt / 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = key0 + 8 * j + (i & 1), h = i >> 1;
          if (key < lo[h] || key >= hi[h]) s[j][i] = -INFINITY;
          top[h] = fmaxf(top[h], s[j][i]);
        }
      float base[2], shrink[2], part[2] = {0.0f, 0.0f};  // the tile's sums first: fewer roundings at the size of l
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
        base[h] = top[h] == -INFINITY ? 0.0f : top[h] * a.scale_log2;
        shrink[h] = exp2_fast(fmaf(m[h], a.scale_log2, -base[h]));
        m[h] = top[h];
        l[h] *= shrink[h];
      }
#pragma unroll
      for (int j = 0; j < kKt / 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[j][i] = exp2_fast(fmaf(s[j][i], a.scale_log2, -base[i >> 1]));
          part[i >> 1] += s[j][i];
        }
      l[0] += part[0];
      l[1] += part[1];
#pragma unroll
      for (int j = 0; j < kDp / 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][i] *= shrink[i >> 1];
#pragma unroll
      for (int kk = 0; kk < kKt / 16; ++kk) {
        const uint32_t pa[4] = {Pair<T>::pack(s[2 * kk][0], s[2 * kk][1]), Pair<T>::pack(s[2 * kk][2], s[2 * kk][3]),
                                Pair<T>::pack(s[2 * kk + 1][0], s[2 * kk + 1][1]),
                                Pair<T>::pack(s[2 * kk + 1][2], s[2 * kk + 1][3])};
#pragma unroll
        for (int j = 0; j < kDp / 16; ++j) {
          uint32_t vb[4];
          ldmatrix_x4_trans(vb, sv + buf * kTile + tile_at<kDp>(kk * 16 + (lane & 15), 2 * j + (lane >> 4)));
          Pair<T>::mma(o[2 * j], pa, vb[0], vb[1]);
          Pair<T>::mma(o[2 * j + 1], pa, vb[2], vb[3]);
        }
      }
      __syncthreads();
    }
    cp_async_wait<0>();

#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float sum = l[h];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int row = un.row0 + warp * 16 + (lane >> 2) + 8 * h;
      if (row >= all_rows) continue;
      const int tok = a.by_rep(row), head = un.head * a.rep + row - tok * a.rep;
      const int64_t at = static_cast<int64_t>(un.q0 + tok) * a.hq + head;
      const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;  // (NaN stays)
      const float lse2 = sum > 0.0f ? fmaf(m[h], a.scale_log2, log2f(sum)) : sum == 0.0f ? -INFINITY : sum;
      if (un.slot >= 0) {
        float *dst = reinterpret_cast<float *>(a.part_o + static_cast<int64_t>(un.slot) * (a.d / 4) * kRows) + 4 * (row - un.row0);
#pragma unroll
        for (int j = 0; j < kDp / 8; ++j) {
          const int col = 8 * j + 2 * (lane & 3);
          if (col < a.d)
            *reinterpret_cast<float2 *>(dst + (col >> 2) * (4 * kRows) + (col & 3)) = make_float2(o[j][2 * h] * inv, o[j][2 * h + 1] * inv);
        }
        if ((lane & 3) == 0) a.part_lse[un.slot * kRows + row - un.row0] = lse2;
      } else {
        const int64_t to = (un.q0 + tok) * a.out_token + head * a.out_head;
#pragma unroll
        for (int j = 0; j < kDp / 8; ++j) {
          const int col = 8 * j + 2 * (lane & 3);
          if (col >= a.d) continue;
          const float x = o[j][2 * h] * inv, y = o[j][2 * h + 1] * inv;
          if (a.out_type == MMQ_DT_F32) *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + to + col) = make_float2(x, y);
          else *reinterpret_cast<uint32_t *>(static_cast<T *>(a.out) + to + col) = Pair<T>::pack(x, y);
        }
        if ((lane & 3) == 0 && a.lse) a.lse[at] = lse2 * kLn2;
      }
    }
    __syncthreads();  // the Q tile and s_unit are free
  }
}

// Joins the pieces of a cut unit: with lse_p (base 2) and normalised outputs
// o_p, out = sum 2^(lse_p - top) o_p / sum 2^(lse_p - top), in fp32 and in an
// order that only the pieces' number and the unit's size decide.  Block (c, y):
// rows 16 y .. of the unit that begins in CTA c; a thread eight columns of a
// row, lanes along the rows (as the partial results lie), with a running maximum,
// so that weights and outputs are read in one round.  Latency bound where few
// rows are cut, else L2 bound.
//
// attention_join_split_kernel, for calls of few units: where a unit has more
// than eight pieces and fewer rows than there are blocks for, blocks also take a
// part of its columns each and a block's threads a part of the pieces (one row
// over 30001 keys: 8 heads on 1, 118 pieces, 19 us for the call, 52 with all
// pieces in one thread's turn; 28 heads on 4 24 and 34.5).  With many units it
// costs 0.5 us more than the other one.
constexpr int kJoinRows = 16, kJoinLeast = 8, kJoinPieces = 8;  // (blocks a unit; pieces a thread)
// Eight columns of a joined row, from their sums and that of the weights relative to top.
template <class T>
__device__ __forceinline__ void store_joined(const AttnArgs &a, int64_t tok, int head, int c, const float4 &x, const float4 &y, float top,
                                             float sum) {
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t to = tok * a.out_token + head * a.out_head + 8 * c;
  if (a.out_type == MMQ_DT_F32) {
    float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + to);
    dst[0] = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    dst[1] = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
  } else {
    uint4 z;
    z.x = Pair<T>::pack(x.x * inv, x.y * inv);
    z.y = Pair<T>::pack(x.z * inv, x.w * inv);
    z.z = Pair<T>::pack(y.x * inv, y.y * inv);
    z.w = Pair<T>::pack(y.z * inv, y.w * inv);
    *reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + to) = z;
  }
  if (c == 0 && a.lse) a.lse[tok * a.hq + head] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
}
template <class T>
__device__ __forceinline__ void join_plain(const AttnArgs &a, const AttnCut &u, int unit_rows, int r0, int rows, int c0, int pieces) {
  const int r = threadIdx.x % kJoinRows;
  if (r >= rows) return;
  const int row = u.row0 + r0 + r, rtok = a.by_rep(row), head = u.head * a.rep + row - rtok * a.rep;
  const int64_t tok = u.q0 + rtok;
  for (int c = threadIdx.x / kJoinRows; c < a.d / 8; c += 256 / kJoinRows) {
    float top = -INFINITY, sum = 0.0f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll 4
    for (int p = 0; p < pieces; ++p) {
      const int64_t s = 2 * (c0 + p) + (p == 0);
      const float l = a.part_lse[s * unit_rows + r0 + r];
      const float4 *src = a.part_o + (s * (a.d / 4) + 2 * c) * unit_rows + r0 + r;
      const float4 f = __ldcs(src), g = __ldcs(src + unit_rows);
      if (l == -INFINITY) continue;
      const float high = fmaxf(top, l), keep = top == -INFINITY ? 0.0f : exp2f(top - high), w = exp2f(l - high);
      top = high;
      sum = fmaf(sum, keep, w);
      x.x = fmaf(x.x, keep, w * f.x), x.y = fmaf(x.y, keep, w * f.y), x.z = fmaf(x.z, keep, w * f.z), x.w = fmaf(x.w, keep, w * f.w);
      y.x = fmaf(y.x, keep, w * g.x), y.y = fmaf(y.y, keep, w * g.y), y.z = fmaf(y.z, keep, w * g.z), y.w = fmaf(y.w, keep, w * g.w);
    }
    store_joined<T>(a, tok, head, c, x, y, top, sum);
  }
}
template <class T>
__global__ void __launch_bounds__(256) attention_join_kernel(const __grid_constant__ AttnArgs a, int unit_rows) {
  griddep_wait();
  griddep_launch_dependents();
  const AttnCut u = a.cuts[blockIdx.x];
  const int r0 = blockIdx.y * kJoinRows, rows = min(min(unit_rows, u.n * a.rep - u.row0) - r0, kJoinRows);
  if (u.last < 0 || rows <= 0) return;
  join_plain<T>(a, u, unit_rows, r0, rows, blockIdx.x, u.last - static_cast<int>(blockIdx.x) + 1);
}

template <class T>
__global__ void __launch_bounds__(256) attention_join_split_kernel(const __grid_constant__ AttnArgs a, int unit_rows) {
  __shared__ float s_top[256], s_sum[256];
  __shared__ float4 s_x[256], s_y[256];
  griddep_wait();
  griddep_launch_dependents();
  const AttnCut u = a.cuts[blockIdx.x];
  const int all = min(unit_rows, u.n * a.rep - u.row0);
  if (u.last < 0 || all <= 0) return;
  // row groups, and column groups (a power of two, up to 16)
  const int row_groups = (all + kJoinRows - 1) / kJoinRows;
  const int c0 = blockIdx.x, pieces = u.last - c0 + 1;
  const int cols_log2 = pieces <= kJoinPieces ? 0 : min(min(31 - __clz(static_cast<int>(gridDim.y) / row_groups), 32 - __clz((pieces - 1) / kJoinPieces)), 4);
  const int group = static_cast<int>(blockIdx.y) / row_groups;
  const int r0 = (static_cast<int>(blockIdx.y) - group * row_groups) * kJoinRows, rows = min(all - r0, kJoinRows);
  const int chunks = a.d / 8, mine = (chunks + (1 << cols_log2) - 1) >> cols_log2;
  const int first = group * mine, end = min(chunks, first + mine);
  if (group >> cols_log2 || first >= end) return;
  if (cols_log2 == 0) {
    join_plain<T>(a, u, unit_rows, r0, rows, c0, pieces);
    return;
  }
  // 16 lots of threads: `par` columns' chunks at a time, and as many parts of the pieces as that leaves
  const int par_log2 = min(32 - __clz(mine - 1), 4), par = 1 << par_log2, parts = 16 >> par_log2;
  const int r = threadIdx.x % kJoinRows, lot = threadIdx.x / kJoinRows;
  const int row = u.row0 + r0 + r, rtok = a.by_rep(row), head = u.head * a.rep + row - rtok * a.rep;
  const int64_t tok = u.q0 + rtok;
  for (int base = first; base < end; base += par) {
    const int c = base + (lot & (par - 1)), part = lot >> par_log2;
    const bool in = r < rows && c < end;
    float top = -INFINITY, sum = 0.0f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    auto add = [&](float l, float w_sum, const float4 &f, const float4 &g) {  // (w_sum: of f and g's weights, relative to l)
      const float high = fmaxf(top, l), keep = top == -INFINITY ? 0.0f : exp2f(top - high), w = exp2f(l - high);
      top = high;
      sum = fmaf(sum, keep, w * w_sum);
      x.x = fmaf(x.x, keep, w * f.x), x.y = fmaf(x.y, keep, w * f.y), x.z = fmaf(x.z, keep, w * f.z), x.w = fmaf(x.w, keep, w * f.w);
      y.x = fmaf(y.x, keep, w * g.x), y.y = fmaf(y.y, keep, w * g.y), y.z = fmaf(y.z, keep, w * g.z), y.w = fmaf(y.w, keep, w * g.w);
    };
    if (in) {
#pragma unroll 4
      for (int p = part; p < pieces; p += parts) {
        const int64_t s = 2 * (c0 + p) + (p == 0);
        const float l = a.part_lse[s * unit_rows + r0 + r];
        const float4 *src = a.part_o + (s * (a.d / 4) + 2 * c) * unit_rows + r0 + r;
        const float4 f = __ldcs(src), g = __ldcs(src + unit_rows);
        if (l != -INFINITY) add(l, 1.0f, f, g);
      }
    }
    if (parts > 1) {
      __syncthreads();  // (the chunk before has been read)
      s_top[threadIdx.x] = top, s_sum[threadIdx.x] = sum, s_x[threadIdx.x] = x, s_y[threadIdx.x] = y;
      __syncthreads();
      if (part == 0)
        for (int i = 1; i < parts; ++i) {
          const int o = threadIdx.x + i * par * kJoinRows;
          if (s_sum[o] != 0.0f) add(s_top[o], s_sum[o], s_x[o], s_y[o]);  // (NaN: added)
        }
    }
    if (!in || part) continue;
    store_joined<T>(a, tok, head, c, x, y, top, sum);
  }
}

template <class T, int kDp>
cudaError_t launch_rows(const AttnArgs &a, int dev, unsigned grid, cudaStream_t s) {
  constexpr int smem = (kRows + 4 * kKt) * kDp * 2;
  const cudaError_t e = allow_smem<attention_rows_kernel<T, kDp>>(dev, smem);
  if (e != cudaSuccess) return e;
  return launch_early(attention_rows_kernel<T, kDp>, grid, 1, kThreads, smem, s, a);
}
template <class T>
cudaError_t launch_rows_of(const AttnArgs &a, int dev, unsigned grid, cudaStream_t s) {
  if (a.d <= 64) return launch_rows<T, 64>(a, dev, grid, s);
  if (a.d <= 128) return launch_rows<T, 128>(a, dev, grid, s);
  return launch_rows<T, 256>(a, dev, grid, s);
}

template <class T>
cudaError_t launch_join(const AttnArgs &a, int unit_rows, int64_t units, unsigned grid, cudaStream_t s) {
  // (no unit has more rows than all tokens together)
  const int64_t groups = (std::min<int64_t>(unit_rows, a.ntok * a.rep) + kJoinRows - 1) / kJoinRows;
  if (units * 4 > grid) return launch_early(attention_join_kernel<T>, grid, static_cast<unsigned>(groups), 256, 0, s, a, unit_rows);
  return launch_early(attention_join_split_kernel<T>, grid, static_cast<unsigned>(std::max<int64_t>(groups, kJoinLeast)), 256, 0, s, a,
                      unit_rows);
}

}  // namespace

cudaError_t launch_attention_rows(const AttnArgs &a, int type, int dev, unsigned grid, cudaStream_t s) {
  return type == MMQ_DT_F16 ? launch_rows_of<__half>(a, dev, grid, s) : launch_rows_of<__nv_bfloat16>(a, dev, grid, s);
}

cudaError_t launch_attention(const mmq_paged_cache &c, const mmq_attention &t, const CallContext &ctx, cudaStream_t s) {
  AttnArgs a = {};
  a.q = t.q, a.k = c.k, a.v = c.v, a.out = t.out, a.lse = t.lse;
  a.table = t.table, a.seq_lens = t.seq_lens, a.q_start = t.q_start;
  a.q_token = t.q_token, a.q_head = t.q_head, a.out_token = t.out_token, a.out_head = t.out_head;
  a.k_page = c.k_page, a.k_token = c.k_token, a.k_head = c.k_head;
  a.v_page = c.v_page, a.v_token = c.v_token, a.v_head = c.v_head;
  a.table_stride = t.table_stride, a.pages = c.pages, a.ntok = t.ntok;
  a.nreq = static_cast<int32_t>(t.nreq), a.table_width = t.table_width, a.page_size = c.page_size;
  a.hq = t.q_heads, a.hkv = c.heads, a.rep = t.q_heads / c.heads, a.d = c.head_dim;
  a.causal = t.causal, a.window = t.window, a.out_type = t.out_type;
  a.scale_log2 = t.scale * 1.44269504088896341f;
  a.wait = {&ctx.words->status, &ctx.words->abort_epoch, ctx.epoch, ctx.limit_ns};

  // The tcgen05 kernel (one CTA an SM) takes every shape it can, the general
  // one (two CTAs an SM, one with heads wider than 128) the rest: 32 rows of one
  // token over 4001 keys, 4 K/V heads of 128, take 54 us in the first (pages of 8
  // or 16 keys) and 70 us in the second (pages of 5), 512 tokens over 4608 keys
  // (16 heads on 4) 29 and 74 us.
  AttnUmma um;
  const bool umma = attention_umma(a, c.type, &um);
  const int unit_rows = umma ? 2 * um.tile_tok * a.rep : kRows, kt = umma ? 128 : kKt;
  const unsigned grid = umma || a.d > 128 ? kSms : 2 * kSms;
  a.unit_tok = umma ? 2 * um.tile_tok : 0;
  a.by_page = FastDiv(c.page_size), a.by_rep = FastDiv(a.rep), a.by_grid = FastDiv(grid);
  a.by_unit_tok = FastDiv(umma ? a.unit_tok : 1);
  // The units' line (attention.cuh) is counted in 32 bits.
  const int64_t room = static_cast<int64_t>(t.table_width) * c.page_size;
  const int64_t units = ((t.ntok * a.rep + unit_rows - 1) / unit_rows + std::min(t.nreq, t.ntok)) * c.heads;
  if (units >= (int64_t(1) << 30) / (std::min<int64_t>(room, 0x7fffffff) / kt + 2 + kAttnGap)) return cudaErrorNotSupported;
  // Scratch for the pieces of cut units, unless no row can have keys for it.
  const bool cut = room > 2 * kt;
  void *scratch = nullptr;
  cudaError_t e = cudaSuccess;
  if (cut) {
    const size_t lse_bytes = static_cast<size_t>(2 * grid) * unit_rows * 4, o_bytes = lse_bytes * a.d;
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    e = cudaStreamIsCapturing(s, &cap);
    if (e != cudaSuccess) return e;
    const size_t bytes = o_bytes + lse_bytes + grid * sizeof(AttnCut);
    e = cap == cudaStreamCaptureStatusActive ? cudaMallocAsync(&scratch, bytes, s)
                                             : cudaMallocFromPoolAsync(&scratch, bytes, ctx.pool, s);
    if (e != cudaSuccess) return e;
    a.part_o = static_cast<float4 *>(scratch);
    a.part_lse = reinterpret_cast<float *>(static_cast<uint8_t *>(scratch) + o_bytes);
    a.cuts = reinterpret_cast<AttnCut *>(static_cast<uint8_t *>(scratch) + o_bytes + lse_bytes);
  }
  e = umma ? launch_attention_umma(a, um, c.type, ctx.device, grid, s) : launch_attention_rows(a, c.type, ctx.device, grid, s);
  if (e == cudaSuccess && cut)
    e = c.type == MMQ_DT_F16 ? launch_join<__half>(a, unit_rows, units, grid, s) : launch_join<__nv_bfloat16>(a, unit_rows, units, grid, s);
  if (scratch) {
    const cudaError_t ef = cudaFreeAsync(scratch, s);
    if (e == cudaSuccess) e = ef;
  }
  return e;
}

}  // namespace mmq
