// internal.h -- declarations shared by the translation units of libmmq.so.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "mmq.h"

// A registered weight.  Device memory owned by the handle:
//   bplane  the GEMM's pre-tiled weight plane (tiling.h): per 128-row tile,
//           super-block and half, the fp16 operand image with the sub-block
//           scale folded in and, for q4_K, the integer-min image; then the
//           scale region (d and, for q4_K, dmin rows).  Rows od..od_pad-1
//           are zero.
//   wexp    optional dense centered q6_K plane, int8 [od][id], q - 32
//   rawplane  optional packed bytes of W regrouped per tile (tiling.h), read
//           by the GEMM's raw arm
struct mmq_weights_s {
  int type = 0;
  int device = 0;
  uint32_t flags = 0;
  int64_t od = 0, id = 0, od_pad = 0, nsb = 0, nb32 = 0;
  void *bplane = nullptr;
  int8_t *wexp = nullptr;
  uint8_t *rawplane = nullptr;  // MMQ_REG_RAW: packed bytes regrouped for the raw arm
  // q6_K with a sub-block scale |sc| > 64: sc*(q - 32) needs up to 13 bits, so
  // the operand plane holds B1 = 2*sc*((q-32) >> 1) and this plane, same
  // layout, B0 = sc*((q-32) & 1); both exact in fp16, B1 + B0 = sc*(q - 32)
  uint8_t *b0plane = nullptr;
  size_t bplane_bytes = 0, wexp_bytes = 0, rawplane_bytes = 0, b0plane_bytes = 0;
};

namespace mmq {

struct WaitCtl;

// Per-device status words (device memory), see WaitCtl in ptx.cuh.
struct DevStatus {
  int status;
  unsigned abort_epoch;
};

constexpr int kRowTile = 128;  // od padding granule == GEMM weight tile

cudaError_t launch_quantize_q8_0(const float *X, int64_t nt, int64_t id, uint8_t *Q,
                                 cudaStream_t s);

// Registration: bytes of the tiled weight plane, and the expansion kernels.
// *bad_scale (device int) becomes nonzero if a q6_K sub-block scale |sc| > 64.
size_t bplane_bytes(int type, int64_t od, int64_t id);
size_t bplane_operand_bytes(int type, int64_t od, int64_t id);  // without the scale region
size_t rawplane_bytes(int type, int64_t od, int64_t id);
cudaError_t launch_dequant(int type, const uint8_t *W, int64_t od, int64_t id, void *out,
                           int out_type, cudaStream_t s);
cudaError_t launch_register(const mmq_weights_s *h, const uint8_t *W, int *bad_scale,
                            cudaStream_t s);
// second pass for q6_K handles with |sc| > 64: B1 into the operand plane, B0
// into h->b0plane (allocated by the caller, b0plane_bytes)
cudaError_t launch_register_b0(const mmq_weights_s *h, const uint8_t *W, cudaStream_t s);

// GEMM: scratch bytes for nt tokens, and the launch of the activation
// prepass + GEMM kernel.  With streamk_allowed the GEMM may split tiles
// between CTAs (and then needs more scratch).  ev0/ev1 (optional) are
// recorded around the GEMM kernel with cudaEventRecordWithFlags(ev, s,
// ev_flags).
// raw: stream the handle's raw plane and unpack it in the kernel.
size_t gemm_scratch_bytes(const mmq_weights_s *h, int64_t nt, bool streamk_allowed, bool raw);
// dump (test hook; whole tiles, not the raw arm): also store every chunk's raw
// partial, fp32, at dump[(t * nb32 + chunk) * od_pad + o] (nt_pad x nb32 x od_pad)
cudaError_t launch_gemm(const mmq_weights_s *h, const uint8_t *Q, const float *X, int64_t nt,
                        float *Y, void *scratch, bool streamk_allowed, bool raw, DevStatus *st,
                        unsigned epoch, uint64_t limit_ns, cudaStream_t s, cudaEvent_t ev0,
                        cudaEvent_t ev1, unsigned ev_flags, float *dump = nullptr);

// Split arm (activation scale folded into A as an exact fp16 hi + lo pair):
// scratch bytes, and the prepass + GEMM launch.  pair: the same operands and
// arithmetic on 2-CTA clusters (cta_group::2 UMMAs of 256 weight rows by 128
// tokens; one-plane handles only).
size_t gemm_split_scratch_bytes(const mmq_weights_s *h, int64_t nt, bool pair);
// whether the split arm would run 256-row weight tiles or pieces of tiles for this many tokens
bool gemm_split_wide(const mmq_weights_s *h, int64_t nt);
// whether MMQ_ARM_AUTO takes the pair arm for this many tokens
bool gemm_pair_preferred(const mmq_weights_s *h, int64_t nt);
cudaError_t launch_gemm_split(const mmq_weights_s *h, const uint8_t *Q, const float *X, int64_t nt, float *Y,
                              void *scratch, DevStatus *st, unsigned epoch, uint64_t limit_ns,
                              cudaStream_t s, cudaEvent_t ev0, cudaEvent_t ev1, unsigned ev_flags, bool pair);

cudaError_t launch_wait_selftest(DevStatus *st, unsigned epoch, uint64_t limit_ns,
                                 cudaStream_t s);

// What an entry point needs to launch on the current device: its status words
// and scratch pool, an epoch of its own and the limit of device waits.  Returns
// an MMQ_* code.
struct CallContext {
  int device;
  DevStatus *words;
  cudaMemPool_t pool;
  unsigned epoch;
  uint64_t limit_ns;
};
int call_context(CallContext *out);

// Launches a kernel that may begin while the one before it on the stream ends
// (it calls griddep_wait before it touches memory another kernel may use).
// cluster: CTAs of a cluster, where the kernel does not say itself.
struct Cluster {
  unsigned ctas = 0;
};
template <class... Params, class... Args>
cudaError_t launch_early(void (*kernel)(Params...), Cluster cluster, unsigned grid_x, unsigned grid_y, unsigned threads, size_t smem, cudaStream_t s,
                         const Args &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid_x, grid_y);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster.ctas, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster.ctas ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <class... Params, class... Args>
cudaError_t launch_early(void (*kernel)(Params...), unsigned grid_x, unsigned grid_y, unsigned threads, size_t smem, cudaStream_t s,
                         const Args &...args) {
  return launch_early(kernel, Cluster{}, grid_x, grid_y, threads, smem, s, args...);
}

// Division of 0 <= n < 2^31 by a number the host knows: with l = ceil(log2 d)
// and m = ceil(2^(31 + l) / d), n m / 2^(31 + l) exceeds n / d by less than 1 / d.
struct FastDiv {
  uint32_t m = 0, shift = 0;
  FastDiv() = default;
  explicit FastDiv(uint32_t d) {
    uint32_t l = 0;
    while ((uint64_t(1) << l) < d) ++l;
    shift = 31 + l;
    m = static_cast<uint32_t>(((uint64_t(1) << shift) + d - 1) / d);
  }
  __device__ __forceinline__ int operator()(int n) const {
    return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(n)) * m >> shift);
  }
};

// ---- paged cache and serving step (paged.cu, verify.cu, attention*.cu) ----
constexpr int64_t kMaxRequests = 8192;  // their sums stay in shared memory

struct PageTablesArgs {
  const int32_t *cached, *fresh, *held;
  int32_t *table;
  const int32_t *free_pages;
  int32_t *q_start, *seq_lens, *held_out;
  int64_t *slots;
  int32_t *positions, *taken;
  int64_t table_stride, table_width, nfree, max_tokens;
  int32_t nreq, page_size;
};
cudaError_t launch_page_tables(const PageTablesArgs &a, cudaStream_t s);

struct KvWriteArgs {
  mmq_paged_cache cache;
  const void *k, *v;
  int64_t k_token, k_head, v_token, v_head;
  const int64_t *slots;
  int64_t ntok;
  int32_t heads, head_dim, src_type, tokens_per_cta;
  FastDiv by_items, by_chunks, by_page;  // items of a token, 8-element chunks of a row, page_size
  int *status;
};
cudaError_t launch_kv_write(KvWriteArgs a, cudaStream_t s);

struct VerifyArgs {
  const void *target, *draft;
  const int32_t *tokens, *n_draft;
  const float *u, *noise;
  int32_t *out, *accepted;
  int64_t target_req, target_row, draft_req, draft_row, tokens_stride, u_stride, noise_stride;
  int64_t nreq, vocab;
  int32_t k, type;
  int *status;
};
cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t s);

// ---- what differs from request to request (pages.cu, rules.cu, lora.cu) ----
// The most of each that the entry points take.  How much shared memory a kernel may
// have is a setting of the kernel on its device, not of a call, so it is always that
// of the most, whatever a call needs: set to a call's own, a small call of one thread
// between another's setting and launch made that launch fail.
constexpr int64_t kMaxPages = int64_t(1) << 20, kMaxVocab = int64_t(1) << 18, kMaxAdapters = int64_t(1) << 18;
constexpr int kMaxRank = 128;

struct ForkArgs : mmq_fork {
  int *status;
};
cudaError_t launch_page_fork(const ForkArgs &a, cudaStream_t s);

struct CompactArgs {
  const int32_t *table, *held;
  int32_t *new_table, *pairs, *counts;
  int64_t nreq, table_width, table_stride, new_stride, npages;
  int *status;
};
cudaError_t launch_page_compact(const CompactArgs &a, cudaStream_t s);

struct PageCopyArgs {
  mmq_paged_cache cache;
  const int32_t *pairs, *tokens;
  int64_t npairs;
  int *status;
  int32_t chunks, outer_items, per_tensor, parts;  // 16-byte items: of a row, of an outer index, of a page; CTAs of a pair
  bool token_outer;                                // the order of a page's memory
  FastDiv by_chunks, by_outer;
};
cudaError_t launch_page_copy(PageCopyArgs a, cudaStream_t s);

constexpr int64_t kMaxSaid = (int64_t(1) << 29) - 1;  // tokens of a request, so that a count of them lies below its flags
constexpr int64_t kMaxBiases = 0x7fffffff - 2047;     // so that rounds of 1024 behind the last one stay in 32 bits
constexpr int64_t kMaxListed = 0x7fffffff / 18;  // requests with lists, whose `starts` are counted in 32 bits

struct RulesArgs {
  mmq_token_rules t;
  bool penalties, sparse, in_place;  // tokens are counted; there are lists; adjusted is the logits
  int32_t slice, ctas;               // entries of a CTA; CTAs of a row
  FastDiv by_rows, by_ctas;
  // where each CTA's part of a request's list begins; the listed tokens, their
  // counts and biases
  int32_t *starts, *list;
  uint32_t *counts;
  float *biases;
  int *status;
  unsigned *abort_epoch;
  unsigned epoch;
  uint64_t limit_ns;
};
cudaError_t launch_token_probs(RulesArgs a, const CallContext &ctx, cudaStream_t s);

struct LoraPlanArgs {
  const int32_t *adapters, *q_start;
  int64_t nreq, ntok, nadapters;
  int32_t *plan;
  int *status;
  int32_t tile, slots;  // tokens of a tile; keys that are sorted, a power of two
  bool few;             // keys few enough to be compared with one another
};
cudaError_t launch_lora_plan(LoraPlanArgs a, cudaStream_t s);
int64_t lora_plan_words(int64_t ntok, int64_t nreq, int64_t nadapters);

struct LoraArgs {
  mmq_lora_args t;
  bool wide;              // rows of y and out in 16-byte pieces
  int32_t front;          // bytes of the first product's stages
  int32_t columns, chunks;  // of a CTA in the second product; CTAs of a tile
  FastDiv by_chunks;
  uint32_t *terms;        // what the first leaves for the second
  uint32_t zero = 0;
};
cudaError_t launch_lora(LoraArgs a, const CallContext &ctx, cudaStream_t s);

// Engine-rate microbenchmarks (probe.cu); out[0..4] as mmq_probe_engine_rates.
cudaError_t launch_engine_probes(DevStatus *st, unsigned epoch, uint64_t limit_ns, cudaStream_t s, double *out);

cudaError_t launch_attention(const mmq_paged_cache &cache, const mmq_attention &at, const CallContext &ctx,
                             cudaStream_t s);

// Fixed scratch of mmq_gemm_noalloc (a static device array in gemm.cu).
constexpr size_t kNoallocScratchBytes = size_t(16) << 20;
cudaError_t noalloc_scratch(int dev, void **out);
// Loads, on the handle's device, the scratch array's module and the kernels
// mmq_gemm_noalloc launches for this handle (registration calls it).
cudaError_t prepare_noalloc(const mmq_weights_s *h);

}  // namespace mmq
