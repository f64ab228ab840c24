/*
 * mmq.h -- C ABI of the GB300 (sm_103a) k-quant x q8_0 prefill GEMM library
 * (libmmq.so).
 *
 * The operation is the prefill "MMQ" GEMM of the minfer CUDA optimisation
 * log:   Y[t][o] = sum_k W[o][k] * X[t][k]
 * with W stored as q6_K or q4_K super-blocks and X quantized per token into
 * q8_0 "pad40" blocks.  Three steps, one entry point each:
 *   mmq_quantize_act     X (fp32)            -> Q (q8_0 pad40 blocks)
 *   mmq_register_weights W (packed k-quant)  -> handle (internal planes,
 *                                               optional dense W_exp plane)
 *   mmq_gemm             handle, Q           -> Y (fp32)
 * and mmq_gemm_f32 (handle, X -> Y) for the two steps fused.
 *
 * Conventions for every entry point:
 *   - Pointers named "device" are CUDA device pointers on the current device;
 *     the caller owns them.  Nothing is freed or retained by the library
 *     except inside an mmq_weights_t handle.
 *   - Work is enqueued asynchronously on `stream` (a cudaStream_t; NULL is
 *     the legacy default stream) unless stated otherwise.
 *   - Return value: MMQ_OK (0) or a negative MMQ_ERR_* code.  Argument
 *     checks happen on the host before anything is enqueued; no C++
 *     exception crosses this boundary.
 *   - A device-side bounded wait that expires records a status word read by
 *     mmq_last_device_error(); the kernel then returns instead of hanging.
 */
#ifndef MMQ_H
#define MMQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *mmq_stream_t;   /* same type as cudaStream_t */
typedef struct mmq_weights_s *mmq_weights_t;

/* ---- status codes ------------------------------------------------------ */
#define MMQ_OK 0
#define MMQ_ERR_ARG -1             /* null pointer, bad size, id % 256 != 0, ... */
#define MMQ_ERR_ALIGN -2           /* a pointer misses the alignment stated below */
#define MMQ_ERR_TYPE -3            /* unknown weight type */
#define MMQ_ERR_CUDA -4            /* a CUDA runtime call failed */
#define MMQ_ERR_DEVICE_TIMEOUT -5  /* a bounded device wait expired (see above) */
#define MMQ_ERR_OOM -6             /* device allocation failed */
#define MMQ_ERR_UNSUPPORTED -7     /* valid input this build does not handle */
#define MMQ_ERR_NO_DEVICE -8       /* current device is not a GB300 (sm_103) */
#define MMQ_ERR_SCRATCH_LIMIT -9   /* problem exceeds mmq_gemm_noalloc's fixed scratch */
#define MMQ_ERR_DEVICE_INDEX -10   /* an index in device memory was out of range (mmq_last_device_error) */

/* ---- weight types (ggml numbering) ------------------------------------- */
#define MMQ_Q4_K 12
#define MMQ_Q6_K 14

/* ---- byte layouts (defined once; the library's kernels use these) ------
 * q8_0 pad40 activation block, one per token t per 32-element chunk c of K,
 * block (t, c) at byte (t*nb32 + c)*40, nb32 = id/32.
 * Source: "26 · r21 — Coalesced block-linear A staging", §2.1, and
 * "25 · r20: Split-phase A staging", §3.2.
 *   [0,2)  d    fp16, little-endian;  [2,4) zero
 *   [4,36) qs   32 x int8;            [36,40) ssum int32 = sum of qs        */
#define MMQ_Q8_BLOCK_BYTES 40
#define MMQ_Q8_D_OFF 0
#define MMQ_Q8_QS_OFF 4
#define MMQ_Q8_SSUM_OFF 36
/* block_q6_K, 256 weights in 16 sub-blocks of 16, w = d*sc[e/16]*(q-32).
 * Source: "47 · r44 — W_exp stride mismatch root cause", §2.2; scale bytes
 * at 192: "46 · r43 — PC-sampling attribution", §3.1.                      */
#define MMQ_Q6K_BLOCK_BYTES 210
#define MMQ_Q6K_QL_OFF 0
#define MMQ_Q6K_QH_OFF 128
#define MMQ_Q6K_SC_OFF 192
#define MMQ_Q6K_D_OFF 208
/* block_q4_K, 256 weights in 8 sub-blocks of 32, w = d*sc*q - dmin*m.  Not
 * printed on the pages; the ggml layout is the reading taken.              */
#define MMQ_Q4K_BLOCK_BYTES 144
#define MMQ_Q4K_D_OFF 0
#define MMQ_Q4K_DMIN_OFF 2
#define MMQ_Q4K_SC_OFF 4
#define MMQ_Q4K_QS_OFF 16
/* every GEMM entry point requires id % MMQ_QK == 0 ("the NB-BT launch gate",
 * "47 · r44 — W_exp stride mismatch root cause", §3.1)                     */
#define MMQ_QK 256

/* ---- registration flags ------------------------------------------------ */
#define MMQ_REG_WEXP 0x1u  /* also build the dense int8 W_exp code plane */
#define MMQ_REG_RAW 0x2u   /* also keep the packed bytes, regrouped, for MMQ_ARM_RAW */

/* ---- GEMM arms (flags of mmq_gemm select one; arm_used reports it) ----- */
#define MMQ_ARM_AUTO 0     /* library choice: MMQ_ARM_PAIR above 128 tokens for one-plane
                              operands (q4_K, and q6_K with every |sc| <= 64), except
                              q6_K problems whose 256-row split tiles fill two or more
                              waves of SMs to 85 %; otherwise MMQ_ARM_SPLIT for one-plane
                              q6_K, and for q4_K when the split arm runs 256-row weight
                              tiles (problems with more 128 x 128 output tiles than SMs)
                              or pieces of tiles (problems with at most half as many tiles
                              as SMs); else MMQ_ARM_F16 */
#define MMQ_ARM_F16 1      /* operands from the registered fp16 operand plane (bulk copies) */
#define MMQ_ARM_RAW 2      /* packed weight bytes streamed and unpacked to fp16 in shared
                              memory inside the GEMM ("47 · r44 — W_exp stride mismatch
                              root cause", §3.2: the in-kernel recombination); needs a
                              handle registered with MMQ_REG_RAW whose operand is one
                              plane (q4_K, or q6_K with every |sc| <= 64; otherwise
                              MMQ_ERR_UNSUPPORTED); bit-identical to F16 */
#define MMQ_ARM_SPLIT 3    /* the activation scale folded into the A operand as an exact
                              fp16 pair (hi = rn(da'*qs), lo = rn(da'*qs - hi)), so the
                              tensor core sums a whole 256-K super-block and the scales
                              apply once per super-block: every product exact, fp32
                              summation (results within the GEMM tolerance, not
                              bit-identical to F16); whole tiles of 128 or 256 weight
                              rows per CTA, or -- with at most half as many 128 x 128
                              tiles as SMs -- each tile's super-blocks cut into pieces
                              over several CTAs whose partial sums are added in a fixed
                              order (repeat calls bit-identical) */
#define MMQ_ARM_PAIR 4     /* MMQ_ARM_SPLIT's operands and arithmetic on pairs of SMs: 2-CTA
                              clusters run cta_group::2 UMMAs of 256 weight rows x 128 (112,
                              96) tokens, each SM staging its own 128 weight rows and half
                              of the token rows, so a 64-K stage of the operand ring holds a
                              third less and takes two bulk copies; whole tiles; results
                              within fp32 summation of MMQ_ARM_SPLIT's (the tensor core sums
                              the transposed tile in its own order); handles whose operand
                              is one plane (otherwise MMQ_ERR_UNSUPPORTED) */

/*
 * mmq_quantize_act -- q8_0 quantization of activations.
 * Source: the pad40 block of "26 · r21 — Coalesced block-linear A staging",
 * §2.1; the quantizer itself (d = amax/127, q = round-half-away(x/d)) is the
 * task's workload definition, computed in fp32 with IEEE division.
 *   X   device, fp32, nt x id row-major, 16-byte aligned.
 *   nt  tokens (>= 0; 0 is a no-op).   id  K, a positive multiple of 32.
 *   Q   device, caller-allocated nt*(id/32)*40 bytes, 16-byte aligned;
 *       fully overwritten (pad bytes [2,4) of each block are written as 0).
 * Non-finite X, or |X| large enough that amax/127 overflows fp16, is out of
 * contract (no error is raised; the bytes written are unspecified).
 * Errors: MMQ_ERR_ARG, MMQ_ERR_ALIGN, MMQ_ERR_NO_DEVICE, MMQ_ERR_CUDA.
 */
int mmq_quantize_act(const float *X, int64_t nt, int64_t id, void *Q, mmq_stream_t stream);

/*
 * mmq_register_weights -- one-time expansion of a packed k-quant weight.
 * Source: registration-time expansion and the dense W_exp plane of
 * "46 · r43 — PC-sampling attribution", §3.2, and "47 · r44 — W_exp stride
 * mismatch root cause", §2.1-2.2 (out[j*id + sb*256 + e] = q - 32, row pitch
 * id, super-block pitch 256).
 *   type  MMQ_Q6_K or MMQ_Q4_K.
 *   W     device, od rows of id/256 packed blocks (210 B q6_K, 144 B q4_K),
 *         row pitch (id/256)*block bytes, no alignment requirement.  Read
 *         only during this call; the caller keeps ownership.
 *   od    output rows (> 0).   id  K, a positive multiple of 256.
 *   flags MMQ_REG_WEXP: also keep the dense int8 W_exp code plane (od*id
 *         bytes): q6_K the centered code q - 32, q4_K the code q (the same
 *         plane carried to q4_K); the operand plane is then built by reading
 *         W_exp back with its dense strides.
 *         MMQ_REG_RAW: also keep the packed bytes regrouped for MMQ_ARM_RAW
 *         (od_pad*id*0.56 B q4_K, *0.88 B q6_K).
 *   out   receives a handle owning the internal planes (fp16 operand plane
 *         with sub-block scales folded in, fp32 scale planes, optional
 *         W_exp) until mmq_release_weights.
 * Synchronizes `stream` before returning (registration is a one-time cost).
 * q6_K sub-block scales take the whole int8 range.  While every |sc| <= 64
 * the folded operand sc*(q-32) (|.| <= 2048) is one exact fp16 plane; if any
 * |sc| > 64 (up to 4096, not always exact in fp16) the handle holds two
 * planes, B1 = 2*sc*((q-32) >> 1) and B0 = sc*((q-32) & 1), each exact, whose
 * sum the GEMM forms on the tensor core (twice the operand bytes; see
 * mmq_weights_info).  Errors: MMQ_ERR_ARG, MMQ_ERR_TYPE, MMQ_ERR_OOM,
 * MMQ_ERR_NO_DEVICE, MMQ_ERR_CUDA.
 */
int mmq_register_weights(int type, const void *W, int64_t od, int64_t id, uint32_t flags,
                         mmq_stream_t stream, mmq_weights_t *out);

/* Frees a handle and its device planes (synchronizes the device). NULL is
 * accepted.  Returns MMQ_OK or MMQ_ERR_CUDA. */
int mmq_release_weights(mmq_weights_t h);

/*
 * mmq_weights_wexp -- the dense int8 W_exp plane of a handle registered with
 * MMQ_REG_WEXP ("46 · r43 — PC-sampling attribution", §3.2; q6_K q - 32, q4_K q):
 * element (o, k) at plane[o*row_pitch + k], row_pitch == id, super-block
 * pitch 256.  The pointer is device memory owned by the handle.
 * Errors: MMQ_ERR_ARG (null argument), MMQ_ERR_UNSUPPORTED (no plane).
 */
int mmq_weights_wexp(mmq_weights_t h, const int8_t **plane, int64_t *row_pitch);

/*
 * mmq_dequantize_weights -- the dequantization fallback: packed k-quant rows
 * to a dense od x id plane of real weights, for consumers that do not run
 * the MMQ contraction ("47 · r44 — W_exp stride mismatch root cause", §2.2:
 * the dequant/embedding paths read the raw blocks).  Each weight
 * (q6_K d*sc*(q-32), q4_K d*sc*q - dmin*m) is formed exactly in fp64 and
 * rounded once, to nearest even, to the output type.
 *   type   MMQ_Q6_K or MMQ_Q4_K.   W  device, packed rows as for
 *          mmq_register_weights.   od, id  as there.
 *   out    device, od*id elements of out_type, row-major (row pitch id),
 *          16-byte aligned.
 *   out_type MMQ_OUT_F16 or MMQ_OUT_F32.
 * Errors: MMQ_ERR_ARG, MMQ_ERR_ALIGN, MMQ_ERR_TYPE, MMQ_ERR_NO_DEVICE,
 * MMQ_ERR_CUDA.
 */
#define MMQ_OUT_F16 1
#define MMQ_OUT_F32 2
int mmq_dequantize_weights(int type, const void *W, int64_t od, int64_t id, void *out,
                           int out_type, mmq_stream_t stream);

/* Sizes of a handle's device planes, in bytes (the VRAM side of the
 * registration trade-off, "47 · r44 — W_exp stride mismatch root cause",
 * §2.4).  Any out pointer may be NULL. */
int mmq_weights_info(mmq_weights_t h, int *type, int64_t *od, int64_t *id,
                     int64_t *operand_bytes, int64_t *scale_bytes, int64_t *wexp_bytes);

/*
 * mmq_gemm -- Y = dequant(Q) . dequant(W)^T for a registered weight.
 * Source: the MMQ contraction with per-sub-block integer dot products
 * rescaled by d*sc (q6_K: "47 · r44 — W_exp stride mismatch root cause",
 * §1.1 and §2.1) and the q4_K min correction through ssum.
 *   h     handle from mmq_register_weights (same device).
 *   Q     device, nt*(id/32)*40 bytes of pad40 blocks, 16-byte aligned.
 *   nt    tokens (>= 0; 0 is a no-op).
 *   Y     device, fp32, nt x od row-major, 16-byte aligned; overwritten.
 *   flags MMQ_ARM_AUTO or one MMQ_ARM_*; arm_used (may be NULL) receives
 *         the arm that ran.
 * Allocates its scratch -- the activation operand plane for tokens padded to
 * a multiple of 128 (nt_pad*id*2 bytes for MMQ_ARM_F16 and MMQ_ARM_RAW, plus
 * nt_pad*(id/32)*8 of per-block scales; nt_pad*id*4 of hi + lo images for
 * MMQ_ARM_SPLIT; about 1/16 more for q4_K's min images), and for a stream-K
 * launch of the fp16-plane arm one 64 KB partial tile per CTA (for the split
 * arm's pieces one 64 KB partial per piece and a counter per tile) -- stream-ordered from a
 * library-private memory pool and frees it stream-ordered; while `stream` is
 * being captured into a CUDA graph the scratch becomes a graph memory node
 * (cudaMallocAsync), so the call can be captured and replayed.
 * Errors: MMQ_ERR_ARG, MMQ_ERR_ALIGN, MMQ_ERR_UNSUPPORTED, MMQ_ERR_OOM,
 * MMQ_ERR_NO_DEVICE, MMQ_ERR_CUDA.  A device timeout is reported later by
 * mmq_last_device_error().
 */
int mmq_gemm(mmq_weights_t h, const void *Q, int64_t nt, float *Y, mmq_stream_t stream,
             uint32_t flags, int *arm_used);

/*
 * mmq_gemm_f32 -- the GEMM straight from fp32 activations: each token is
 * quantized to q8_0 exactly as mmq_quantize_act does and fed to the
 * contraction without the pad40 plane being written: the producer emits the
 * quantized operand plane directly, the step after the separate
 * quantize-transpose prepass in "26 · r21 — Coalesced block-linear A
 * staging", §5.  Y is bit-identical to mmq_quantize_act followed by
 * mmq_gemm on the same X.
 *   X     device, fp32, nt x id row-major, 16-byte aligned.
 *   Other arguments, scratch, the out-of-contract inputs of mmq_quantize_act
 *   and the errors as mmq_gemm.
 */
int mmq_gemm_f32(mmq_weights_t h, const float *X, int64_t nt, float *Y, mmq_stream_t stream,
                 uint32_t flags, int *arm_used);

/*
 * mmq_gemm_profiled -- mmq_gemm that also records two caller-created CUDA
 * events (cudaEvent_t, either may be NULL) on `stream` immediately before
 * and after the main GEMM kernel, so the caller can time that kernel alone.
 * Arguments and errors otherwise as mmq_gemm.
 */
int mmq_gemm_profiled(mmq_weights_t h, const void *Q, int64_t nt, float *Y, mmq_stream_t stream,
                      uint32_t flags, int *arm_used, void *ev_start, void *ev_stop);

/* mmq_gemm_f32 with the same two events around its main GEMM kernel. */
int mmq_gemm_f32_profiled(mmq_weights_t h, const float *X, int64_t nt, float *Y,
                          mmq_stream_t stream, uint32_t flags, int *arm_used, void *ev_start,
                          void *ev_stop);

/*
 * mmq_gemm_noalloc -- mmq_gemm for callers that cannot allocate device
 * memory: a caller whose GPU memory is entirely owned by another allocator
 * (for example a framework's caching allocator that reserved the device),
 * or one on a path where cudaMalloc's implicit device synchronization is not
 * acceptable.  The log pages have no counterpart to this entry point.
 * It allocates nothing: its scratch is a fixed 16 MiB device array compiled
 * into the library, which every device that loads the library holds until
 * the process exits.  The caller still passes Q and Y (as for mmq_gemm) and
 * a handle from mmq_register_weights, which must have run on the current
 * device first.
 *   - Problems whose scratch exceeds 16 MiB are rejected with
 *     MMQ_ERR_SCRATCH_LIMIT.  Scratch per token, with nt rounded up to a
 *     multiple of 128: id*2 + (id/32)*4 + 4 bytes, plus (id/256)*32 for q4_K;
 *     e.g. id = 3584 allows up to 2048 (q4_K) or 2176 (q6_K) tokens.
 *   - mmq_register_weights prepares what this entry point launches: it
 *     looks up the array's device address on its device and loads the
 *     GEMM's module and kernels there.  Without that, CUDA's lazy module
 *     loading (the default since CUDA 12.2) would load them -- allocating
 *     the array and the kernels' code -- inside the first call here.  So,
 *     after a registration on the device, no call allocates; the first call
 *     on a device still looks the address up in a host-side table, so make
 *     it before any stream capture.
 *   - Every call shares the one array, which keeps the previous call's
 *     contents; each call rewrites or clears everything it reads.  Calls
 *     that can overlap on the GPU (different streams, no ordering) race on
 *     the array: order them on one stream or with events.
 * Always runs the MMQ_ARM_F16 arm.  Errors: MMQ_ERR_ARG, MMQ_ERR_ALIGN,
 * MMQ_ERR_SCRATCH_LIMIT, MMQ_ERR_NO_DEVICE, MMQ_ERR_CUDA; a device timeout is
 * reported by mmq_last_device_error().
 */
int mmq_gemm_noalloc(mmq_weights_t h, const void *Q, int64_t nt, float *Y, mmq_stream_t stream);

/*
 * mmq_debug_chunk_partials -- test hook for the integer exactness of the
 * fp16-plane arm: runs its GEMM (whole tiles) on Q and writes, for every
 * token t, 32-element chunk c and output row o, the raw partial the tensor
 * core left in TMEM before any float scale was applied:
 *   P[t][c][o] = sum_{k in chunk c} qs[t][k] * B[o][k],
 * B the registered operand (sc*(q-32) for q6_K, sc*q for q4_K; for a
 * two-plane q6_K handle the sum of both planes' UMMAs).  Each is an integer
 * below 2^24 in magnitude, stored exactly in fp32 (the per-sub-block integer
 * dot products of "47 · r44 — W_exp stride mismatch root cause", §1.1,
 * rescaled by sc).
 *   Q   device pad40 blocks as for mmq_gemm, 16-byte aligned.
 *   P   device, fp32, nt x (id/32) x od, 16-byte aligned; overwritten.
 * Takes nt_pad*(id/32)*od_pad*4 bytes of scratch beside the GEMM's (meant
 * for small problems).  Errors as mmq_gemm.
 */
int mmq_debug_chunk_partials(mmq_weights_t h, const void *Q, int64_t nt, float *P, mmq_stream_t stream);

/* ---- the serving step around the projections ---------------------------
 * Four entry points that hand each other their outputs: page tables and slot
 * maps from request lengths, the projections' K and V rows into a paged
 * cache, attention of the new tokens over it, and the verification of drafted
 * tokens, whose accepted counts give the next step's lengths.  Lengths stay
 * on the device: nothing here synchronizes or reads them back, so every call
 * can be captured into a CUDA graph and replayed on other lengths.
 *
 * Element types.  The values of MMQ_OUT_F16 / MMQ_OUT_F32, and bf16. */
#define MMQ_DT_F16 1
#define MMQ_DT_F32 2
#define MMQ_DT_BF16 3

/* A paged cache of keys and values.  Row (page, token, head) of K begins at
 * element page*k_page + token*k_token + head*k_head and holds head_dim
 * contiguous elements; V the same with its own strides.  So both
 * [page][token][head][d] and [page][head][token][d] are strides of this.
 * Slot s is token s % page_size of page s / page_size. */
typedef struct mmq_paged_cache {
  void *k, *v;                      /* device, 16-byte aligned */
  int64_t k_page, k_token, k_head;  /* strides in elements, multiples of 8 */
  int64_t v_page, v_token, v_head;
  int64_t pages;                    /* >= 1 */
  int32_t page_size;                /* >= 1, any size */
  int32_t heads;                    /* K/V heads */
  int32_t head_dim;                 /* a multiple of 8, at most 256 */
  int32_t type;                     /* MMQ_DT_F16 or MMQ_DT_BF16 */
} mmq_paged_cache;

/*
 * mmq_page_tables -- page tables, slot map and row starts of a step, built on
 * the device from the requests' lengths.  Request b has cached[b] tokens in
 * the cache, brings fresh[b] new ones and holds held[b] pages (it may hold
 * more than its tokens fill, after refused drafted tokens).  With
 *   need[b] = ceil((cached[b] + fresh[b]) / page_size)
 * it takes need[b] - held[b] pages, if positive, from free_pages, in the
 * order of the requests; table[b][held[b]..] receives them (the other entries
 * are left as they are).
 *   cached, fresh, held  device, int32, nreq each; negative counts as 0.
 *   table       device, int32, nreq rows of table_width, row pitch
 *               table_stride; read and extended in place.  Running the call
 *               again on the same inputs writes the same.
 *   free_pages  device, int32, nfree page ids (nfree >= 0).
 *   q_start     device, int32, nreq + 1: the new tokens' first rows and their
 *               total.   seq_lens  device, int32, nreq: cached + fresh.
 *   held_out    device, int32, nreq: pages held now.
 *   slots       device, int64, max_tokens: slot of every new token; -1 for a
 *               token that found no page and behind the last token.
 *   positions   device, int32, max_tokens: place of the token in its request;
 *               -1 behind the last token.
 *   taken       device, int32, 2: pages taken from the front of free_pages;
 *               pages missing (free_pages too short or need > table_width;
 *               their table entries are -1).
 * New tokens past max_tokens get no slot.  What is written (table among it)
 * may overlap nothing else of the call: held_out is another buffer than held,
 * seq_lens another than cached (MMQ_ERR_ARG).  nreq in 0..8192 (more:
 * MMQ_ERR_UNSUPPORTED).  One kernel, no scratch.  Errors: MMQ_ERR_ARG,
 * MMQ_ERR_ALIGN (elements off their own alignment), MMQ_ERR_UNSUPPORTED,
 * MMQ_ERR_NO_DEVICE, MMQ_ERR_CUDA.
 */
int mmq_page_tables(const int32_t *cached, const int32_t *fresh, const int32_t *held, int64_t nreq,
                    int32_t *table, int64_t table_width, int64_t table_stride, const int32_t *free_pages,
                    int64_t nfree, int32_t page_size, int64_t max_tokens, int32_t *q_start, int32_t *seq_lens,
                    int32_t *held_out, int64_t *slots, int32_t *positions, int32_t *taken, mmq_stream_t stream);

/*
 * mmq_kv_write -- rows of K and V into their slots of a paged cache.
 *   k, v     device, 16-byte aligned; element (t, head, i) at t*k_token +
 *            head*k_head + i (strides multiples of 8 elements, so K and V may
 *            be columns of a fused projection's output), cache->heads heads.
 *   src_type MMQ_DT_F32, MMQ_DT_F16 or MMQ_DT_BF16; rounded to the cache's
 *            type to nearest even, once.
 *   slots    device, int64, ntok: a negative slot writes nothing; a slot past
 *            the cache writes nothing and is reported by
 *            mmq_last_device_error; a slot twice leaves either row.
 *   ntok     >= 0; 0 is a no-op.
 * Errors: MMQ_ERR_ARG, MMQ_ERR_ALIGN, MMQ_ERR_TYPE, MMQ_ERR_UNSUPPORTED
 * (a token's K and V of more than 2^33 elements), MMQ_ERR_NO_DEVICE,
 * MMQ_ERR_CUDA.
 */
int mmq_kv_write(const mmq_paged_cache *cache, const void *k, int64_t k_token, int64_t k_head, const void *v,
                 int64_t v_token, int64_t v_head, int src_type, const int64_t *slots, int64_t ntok,
                 mmq_stream_t stream);

/* Arguments of mmq_paged_attention. */
typedef struct mmq_attention {
  const void *q;             /* device, 16-byte aligned, the cache's type: (t, head, i) at t*q_token + head*q_head + i */
  void *out;                 /* device, 16-byte aligned: (t, head, i) at t*out_token + head*out_head + i */
  float *lse;                /* device, ntok x q_heads, or NULL */
  const int32_t *table;      /* device, nreq rows of table_width page ids, row pitch table_stride */
  const int32_t *seq_lens;   /* device, nreq: keys of each request, its new tokens among them */
  const int32_t *q_start;    /* device, nreq + 1: first row of each request's new tokens, ascending from 0 */
  int64_t q_token, q_head;   /* strides in elements, multiples of 8 */
  int64_t out_token, out_head;
  int64_t table_stride;
  int64_t nreq, ntok;        /* requests; rows of q (ntok * q_heads below 2^31 - 512) */
  int32_t table_width;
  int32_t q_heads;           /* a multiple of cache->heads: q head h reads K/V head h / (q_heads / heads) */
  int32_t out_type;          /* the cache's type or MMQ_DT_F32 */
  int32_t causal;            /* nonzero: a token sees no later one */
  int32_t window;            /* > 0: a token sees the last `window` keys up to itself; 0: no window */
  float scale;               /* of q . k; positive */
} mmq_attention;

/*
 * mmq_paged_attention -- attention of each request's new tokens over its
 * pages.  Token i of request b is at position p = seq_lens[b] - n + i, n =
 * q_start[b+1] - q_start[b]; it sees keys j < seq_lens[b] with j <= p (causal)
 * and j > p - window (window > 0).  out = softmax(scale q.k) v over them, lse
 * the natural logarithm of their sum of exponentials; a row that sees no key
 * gets out = 0, lse = -inf.  One token a request (a decode step), a few (drafted
 * tokens) or thousands (a prompt's chunk) go through this one call, in any
 * mixture.
 *   Rows of q past q_start[nreq] belong to no request; their out and lse are
 * not written.  Where q_start counts more tokens than q has rows (ntok), the
 * rows that are there keep their positions and the others are left out.
 *   seq_lens[b] = 0 and n = 0 are allowed.  Keys past seq_lens[b]
 * are not used, whatever their memory holds, and table entries past the last
 * key's page are not read; nor, with a window, keys and pages behind that of
 * the request's first new token, so that such pages can be given away.  A non-finite V row that some row of a chunk sees
 * may also make rows of that chunk non-finite that do not see it.
 *   A page id outside the cache, or seq_lens[b] past table_width*page_size, is
 * reported by mmq_last_device_error; that request's rows are then unspecified.
 * So is a q_start that descends; every row is then unspecified.
 *   Products and sums are fp32; the softmax weights are rounded to the
 * cache's type before they multiply V.  The results of one problem do not
 * change from call to call.
 *   Long rows are split over the SMs when there are few of them: partial
 * results (fp32, two for each SM, 40 MB) are stream-ordered scratch as for
 * mmq_gemm.
 * Errors: MMQ_ERR_ARG, MMQ_ERR_ALIGN, MMQ_ERR_TYPE, MMQ_ERR_OOM,
 * MMQ_ERR_UNSUPPORTED (2^30 or more tiles of rows by keys),
 * MMQ_ERR_NO_DEVICE, MMQ_ERR_CUDA.
 */
int mmq_paged_attention(const mmq_paged_cache *cache, const mmq_attention *args, mmq_stream_t stream);

/* Arguments of mmq_verify_draft. */
typedef struct mmq_verification {
  const void *target;        /* device, type: probability of token v after drafted token i (row 0: before the
                                first) at b*target_req + i*target_row + v, k + 1 rows a request */
  const void *draft;         /* device, type: the draft's probabilities, k rows a request; NULL: the draft
                                gave its token probability 1 */
  const int32_t *tokens;     /* device: drafted token i of request b at b*tokens_stride + i */
  const int32_t *n_draft;    /* device, nreq: drafted tokens of each request, 0..k; NULL: k */
  const float *u;            /* device: uniform in [0, 1) at b*u_stride + i */
  const float *noise;        /* device: independent exponential variates at b*noise_stride + v */
  int32_t *out;              /* device, nreq x (k + 1) */
  int32_t *accepted;         /* device, nreq */
  int64_t target_req, target_row, draft_req, draft_row, tokens_stride, u_stride, noise_stride; /* in elements */
  int64_t nreq, vocab;
  int32_t k;                 /* >= 0 */
  int32_t type;              /* of target and draft: MMQ_DT_F32, MMQ_DT_F16 or MMQ_DT_BF16 */
} mmq_verification;

/*
 * mmq_verify_draft -- verification of drafted tokens.  Drafted token x_i is
 * kept while u_i * q_i(x_i) < p_i(x_i) (fp32); accepted[b] is the number kept
 * before the first refusal.  Behind them comes one more token: after a refusal
 * at row i it is argmax_v (p_i - q_i)+(v) / noise(v), or argmax_v p_i(v) /
 * noise(v) where p_i - q_i is nowhere positive; with all kept it is
 * argmax_v p_n(v) / noise(v).  Ties go to the lowest v; weights that are not
 * positive (NaN among them) take no part; -1 if there are none.  With
 * exponential noise that is a draw from the normalised weights.
 *   out[b] = kept tokens, the drawn token, then -1.
 * A drafted token outside [0, vocab) is refused and reported by
 * mmq_last_device_error.  nreq in 0..65535, vocab in 1..2^31-1.  One kernel,
 * no scratch.
 * Errors: MMQ_ERR_ARG, MMQ_ERR_ALIGN (elements off their own alignment),
 * MMQ_ERR_TYPE, MMQ_ERR_NO_DEVICE, MMQ_ERR_CUDA.
 */
int mmq_verify_draft(const mmq_verification *args, mmq_stream_t stream);

/* ---- what differs from request to request in a step ---------------------
 * The pages that requests share, give back or get copies of; the rules that a
 * request puts on its next token; the low-rank adapter that it brings beside
 * the shared projections.  As above nothing synchronizes or reads device
 * memory back.
 *
 * mmq_page_fork -- the rows of a page table made anew from the rows that there
 * are: row b continues old row parents[b] with its first lens[b] tokens.  One
 * call forks a request (two rows with one parent), reorders beams, ends a
 * request (no row continues it), and takes back the pages that refused drafted
 * tokens left (lens[b] shorter).  With
 *   need[b] = min(ceil(lens[b] / page_size), held[parents[b]], table_width)
 * row b gets the first need[b] pages of its parent.  Rows may share pages that
 * are full; the page that the next token goes into (the last one, where
 * lens[b] is no multiple of page_size) is a row's own: of the rows that
 * have it as that page the lowest keeps it, unless another row has it as a
 * full one, and every other row gets a free page in its place and an entry in
 * `pairs`, for mmq_page_copy.  Pages that no new row holds are free.
 *   table, held  device, int32: nold rows of table_width page ids, row pitch
 *                table_stride; pages that each row holds.
 *   parents, lens device, int32, nnew each: old row (-1: an empty row), tokens
 *                (negative counts as 0).
 *   npages       pages of the cache; ids are 0..npages - 1.
 *   new_table    device, int32, nnew rows of table_width, row pitch
 *                new_stride; -1 behind a row's pages.
 *   held_out     device, int32, nnew: need.
 *   pairs        device, int32, nnew x 2: page to copy and the free page that
 *                takes its place, -1 -1 for a row without a copy.
 *   tokens       device, int32, nnew: tokens to copy (0 without a copy).
 *   free_pages   device, int32, npages: ids that no new row holds, ascending,
 *                then -1.  Copies take the lowest ids, in the rows' order.
 *   counts       device, int32, 2: entries of free_pages; copies that found no
 *                free page (their table entries are -1).
 * Pages that are to stay held though no request has them are a row of their
 * own.  An entry of parents or of a row outside its range (the page becomes
 * -1), or lens[b] beyond what its parent holds, is reported by
 * mmq_last_device_error.  What is written may overlap nothing else of the
 * call (MMQ_ERR_ARG).  nold, nnew in 0..8192, npages in 0..2^20, table_width
 * at most 2^31 - 1024 (more: MMQ_ERR_UNSUPPORTED).  One kernel, no scratch.
 * Errors: MMQ_ERR_ARG, MMQ_ERR_ALIGN (elements off their own alignment),
 * MMQ_ERR_UNSUPPORTED, MMQ_ERR_NO_DEVICE, MMQ_ERR_CUDA.
 */
typedef struct mmq_fork {
  const int32_t *table, *held, *parents, *lens;
  int32_t *new_table, *held_out, *pairs, *tokens, *free_pages, *counts;
  int64_t nold, nnew, table_width, table_stride, new_stride, npages;
  int32_t page_size;         /* >= 1 */
} mmq_fork;
int mmq_page_fork(const mmq_fork *args, mmq_stream_t stream);

/*
 * mmq_page_compact -- moves that bring the held pages of a cache to its front:
 * with H pages held by any row, the j-th held id from H on moves to the j-th
 * id below H that is not held.
 *   table, held  device, int32, as for mmq_page_fork, nreq rows.
 *   new_table    device, int32, nreq rows of table_width, row pitch
 *                new_stride: the table after the moves, -1 behind a row's pages.
 *   pairs        device, int32, (npages / 2) x 2: from, to; then -1 -1.  No
 *                page is both.
 *   counts       device, int32, 2: H, moves.
 * After mmq_page_copy(pairs) pages H..npages - 1 are free.  A page id out of
 * range in a row becomes -1 and is reported by mmq_last_device_error.  Limits,
 * overlaps and errors as mmq_page_fork.  One kernel, no scratch.
 */
int mmq_page_compact(const int32_t *table, const int32_t *held, int64_t nreq, int64_t table_width, int64_t table_stride,
                     int64_t npages, int32_t *new_table, int64_t new_stride, int32_t *pairs, int32_t *counts,
                     mmq_stream_t stream);

/*
 * mmq_page_copy -- pages of K and V copied within a cache.
 *   pairs   device, int32, npairs x 2: page from, page to.  A pair with a
 *           negative id copies nothing; an id past the cache copies nothing
 *           and is reported by mmq_last_device_error.
 *   tokens  device, int32, npairs: leading tokens to copy (0..page_size, others
 *           are brought into that range), or NULL: whole pages.
 * All pairs at once: a page that one pair writes and another reads or writes
 * holds either's rows (mmq_page_fork and mmq_page_compact give no such
 * pairs).  npairs >= 0; 0 is a no-op.  Errors: MMQ_ERR_ARG, MMQ_ERR_ALIGN,
 * MMQ_ERR_TYPE, MMQ_ERR_UNSUPPORTED (a page of more than 2^32 elements),
 * MMQ_ERR_NO_DEVICE, MMQ_ERR_CUDA.
 */
int mmq_page_copy(const mmq_paged_cache *cache, const int32_t *pairs, const int32_t *tokens, int64_t npairs,
                  mmq_stream_t stream);

/* Arguments of mmq_token_probs. */
typedef struct mmq_token_rules {
  const void *logits;          /* device, type: token v of row i of request b at b*logits_req + i*logits_row + v */
  void *probs;                 /* device, probs_type, or NULL: b*probs_req + i*probs_row + v */
  void *adjusted;              /* device, adjusted_type, or NULL; may be the logits themselves (same type and strides) */
  const float *temperature;    /* device, nreq; NULL: 1 */
  const int32_t *tokens;       /* device: token j of request b at b*tokens_stride + j; NULL: none */
  const int32_t *token_lens;   /* device, nreq; NULL: tokens_width */
  const int32_t *prompt_lens;  /* device, nreq: leading tokens that are the prompt's; NULL: 0 */
  const int32_t *draft;        /* device: drafted token j of request b at b*draft_stride + j; NULL: none */
  const int32_t *n_draft;      /* device, nreq: rows past row n_draft[b] are not computed or written; NULL: all rows */
  const float *repetition;     /* device, nreq; NULL: 1 */
  const float *frequency;      /* device, nreq; NULL: 0 */
  const float *presence;       /* device, nreq; NULL: 0 */
  const int32_t *bias_start;   /* device, nreq + 1: first bias of each request, ascending; NULL: none */
  const int32_t *bias_ids;     /* device, nbias */
  const float *bias_values;    /* device, nbias */
  const int32_t *mask;         /* device, nmasks rows of mask_stride words: bit v % 32 of word v / 32 allows token v; NULL: none */
  const int32_t *mask_rows;    /* device, nreq x rows: row of mask, -1: no mask; NULL: row b*rows + i */
  int64_t logits_req, logits_row, probs_req, probs_row, adjusted_req, adjusted_row;
  int64_t tokens_stride, tokens_width, draft_stride, nbias, mask_stride, nmasks;
  int64_t nreq, vocab;
  int32_t rows;                /* rows of a request, >= 1: one, and one for each drafted token */
  int32_t type, probs_type, adjusted_type; /* MMQ_DT_F32, MMQ_DT_F16 or MMQ_DT_BF16 */
} mmq_token_rules;

/*
 * mmq_token_probs -- probabilities of the next tokens under each request's
 * rules, as mmq_verify_draft reads them.  Row i of request b stands behind
 * its tokens and its first i drafted ones.  With c(v) the times that token v
 * is among the tokens behind the prompt and those drafted ones, in fp32 and in
 * this order:
 *   x = logits[v];  v among the tokens or drafted ones: x = x > 0 ? x / repetition : x * repetition
 *   x -= frequency * c(v);  c(v) > 0: x -= presence;  x += the sum of v's biases, in their order
 *   v not allowed by the row's mask: x = -inf
 *   adjusted[v] = x;  probs = softmax(x / temperature), over the row
 * temperature not above 0: probability 1 for the largest x (ties: the lowest
 * v).  A row with no token left gets probabilities of 0; a NaN that no mask
 * hides (or, with a temperature, +inf) makes a row's probabilities NaN.
 * Sums are fp32; probs and adjusted are rounded once.  Exponentials are within
 * 2^-20, and 2^-23 times the size of their exponent, of themselves;
 * probabilities below 2^-126 may become 0.  The results of one problem do not
 * change from call to call; a row that begins elsewhere in 16 bytes of memory,
 * or is one of another number of rows, is added up in other groups, so that a
 * request alone and in a batch may differ in the last bits.
 *   Tokens, drafted tokens and biases outside [0, vocab) are left out, a mask
 * row past nmasks is no mask, token_lens past tokens_width, n_draft past
 * rows - 1, bias_start past nbias are cut; all of them are reported by
 * mmq_last_device_error.
 * What is written may overlap nothing else of the call (MMQ_ERR_ARG), but for
 * adjusted in the logits' place.
 * vocab in 1..2^18, tokens_width below 2^29, nbias at most 2^31 - 2048,
 * nreq*rows below 2^27, nreq with penalized tokens or with biases at most
 * 119304647 (more: MMQ_ERR_UNSUPPORTED).  With such tokens or biases each
 * request's are listed first, in stream-ordered scratch as for mmq_gemm (12
 * bytes for each token of the rows' width, drafted token and bias, 72 a
 * request).
 * Errors: MMQ_ERR_ARG, MMQ_ERR_ALIGN (elements off their own alignment),
 * MMQ_ERR_TYPE, MMQ_ERR_OOM, MMQ_ERR_UNSUPPORTED, MMQ_ERR_NO_DEVICE,
 * MMQ_ERR_CUDA.
 */
int mmq_token_probs(const mmq_token_rules *args, mmq_stream_t stream);

/*
 * mmq_lora_plan -- the tokens of a step in the order of their adapters, once
 * for all its projections.
 *   adapters  device, int32, nreq: adapter of each request's tokens, -1: none
 *             (an id outside -1..nadapters - 1 counts as none and is reported
 *             by mmq_last_device_error).
 *   q_start   device, int32, nreq + 1, as for mmq_paged_attention (one that
 *             descends is reported; the plan is then empty).
 *   ntok      token rows; rows behind q_start[nreq] belong to no request.
 *   plan      device, int32, mmq_lora_plan_words(ntok, nreq, nadapters) words, for
 *             mmq_lora with the same ntok, nreq and nadapters.
 * nreq in 0..8192, nadapters in 0..2^18 (more: MMQ_ERR_UNSUPPORTED).  One
 * kernel, no scratch.  Errors: MMQ_ERR_ARG, MMQ_ERR_ALIGN,
 * MMQ_ERR_UNSUPPORTED, MMQ_ERR_NO_DEVICE, MMQ_ERR_CUDA.
 */
int mmq_lora_plan(const int32_t *adapters, const int32_t *q_start, int64_t nreq, int64_t ntok, int64_t nadapters,
                  int32_t *plan, mmq_stream_t stream);
/* int32 words of a plan; -1 for sizes that mmq_lora_plan refuses. */
int64_t mmq_lora_plan_words(int64_t ntok, int64_t nreq, int64_t nadapters);

/* Arguments of mmq_lora. */
typedef struct mmq_lora_args {
  const void *x;            /* device, 16-byte aligned, x_type: (t, i) at t*x_row + i */
  const float *y;           /* device: (t, o) at t*y_row + o */
  float *out;               /* device: (t, o) at t*out_row + o; y itself, or memory that overlaps nothing of the call */
  const void *a, *b;        /* device, 16-byte aligned, type: (adapter, r, i) at (adapter*rank + r)*id + i; (adapter, o, r) at
                               (adapter*od + o)*rank + r */
  const float *scales;      /* device, nadapters; NULL: 1 */
  const int32_t *ranks;     /* device, nadapters: rank of each (0..rank, others are brought into that range); NULL: rank */
  const int32_t *plan;      /* from mmq_lora_plan */
  int64_t x_row, y_row, out_row; /* in elements; x_row * the element's size a multiple of 16 bytes */
  int64_t ntok, nreq, nadapters; /* as in the plan */
  int64_t id, od;           /* id a multiple of 8; both at most 2^28 (more: MMQ_ERR_UNSUPPORTED) */
  int32_t rank;             /* of the arrays a and b: a multiple of 8, at most 128 */
  int32_t type;             /* of a and b: MMQ_DT_F16 or MMQ_DT_BF16 */
  int32_t x_type;           /* MMQ_DT_F32, MMQ_DT_F16 or MMQ_DT_BF16 */
} mmq_lora_args;

/*
 * mmq_lora -- low-rank adapters beside a shared projection:
 *   out[t][o] = y[t][o] + scale * sum_r b[o][r] * (sum_i a[r][i] * x[t][i])
 * with the adapter, and the rank, of token t's request.  Tokens of a request
 * without an adapter get out = y; rows of no request are not written.  Where
 * out is y (the usual call, behind mmq_gemm_f32) only rows with an adapter are
 * touched.  Rows and columns of a and b past an adapter's rank are not used,
 * whatever they hold.
 *   Sums are fp32; x and the inner sums enter the tensor cores as three 16-bit
 * terms, which hold their 24 bits.  An x or an inner sum that is not finite
 * (or that the first term rounds to infinity, from 3.39e38 on) makes its row
 * NaN.  The results of one problem do not change from call to call.
 *   With g = min(nreq, nadapters + 1) groups of tokens (at least one),
 * ceil(ntok / g) above 8 and ntok above 341 the inner sums are stream-ordered
 * scratch as for mmq_gemm: for tiles of 64 tokens (of 16, where ceil(ntok / g)
 * or ntok * 8 / 304 is at most 32), min(ntok, ntok / tile + g) of them, 192
 * bytes a token's place up to rank 32, 576 up to 64, else 960.  Other calls
 * have none.
 * Errors: MMQ_ERR_ARG, MMQ_ERR_ALIGN, MMQ_ERR_TYPE, MMQ_ERR_OOM,
 * MMQ_ERR_UNSUPPORTED, MMQ_ERR_NO_DEVICE, MMQ_ERR_CUDA.
 */
int mmq_lora(const mmq_lora_args *args, mmq_stream_t stream);

/* Synchronizes the current device, then returns and clears the device status
 * word: MMQ_OK, MMQ_ERR_DEVICE_TIMEOUT if a bounded wait expired since
 * the last call, or MMQ_ERR_DEVICE_INDEX if an index was out of range (the
 * first of them, if both). */
int mmq_last_device_error(void);

/* Limit of every device-side wait, in ns (default 2e9).  Host-global. */
void mmq_set_wait_timeout_ns(uint64_t ns);

/* Failure-detection self test: launches one CTA that waits on a barrier
 * nothing arrives at, bounded by timeout_ns, then synchronizes and returns
 * mmq_last_device_error() -- MMQ_ERR_DEVICE_TIMEOUT when the bound works. */
int mmq_selftest_wait_timeout(uint64_t timeout_ns, mmq_stream_t stream);

/*
 * mmq_probe_engine_rates -- measurement hook, not part of the method: the
 * rates of the exact-integer-capable tensor engines on the current device,
 * the numbers behind the choice of tcgen05 kind::f16 for the integer
 * contraction and of the fp16/bf16 peak as the roofline's denominator (the
 * log pages run int8 IMMA; sm_103a has no tcgen05 kind::i8).  Writes
 *   out[0..2]  tcgen05.mma kind::f16, M = 128, K = 16, N = 64 / 128 / 256:
 *              MACs per clock per SM (one issuing warp per SM, back to back)
 *   out[3]     mma.sync m16n8k32 s8 -> s32 over the whole GPU, TOPS (2 ops per MAC)
 *   out[4]     mma.sync m16n8k16 f16 -> f32 over the whole GPU, TFLOP/s
 *   out[5..6]  as out[0..2], N = 96 / 112
 *   out[7..11] tcgen05.mma.cta_group::2 kind::f16 on 2-CTA clusters, M = 256,
 *              K = 16, N = 64 / 96 / 112 / 128 / 256: MACs per clock per SM
 *              of the pair (the pair arm's UMMA shape)
 * (12 doubles.)
 * Synchronizes `stream`; takes well under a second.  Errors: MMQ_ERR_ARG,
 * MMQ_ERR_NO_DEVICE, MMQ_ERR_CUDA, MMQ_ERR_DEVICE_TIMEOUT.
 */
int mmq_probe_engine_rates(double *out, mmq_stream_t stream);

/* Static text for a status code. */
const char *mmq_strerror(int code);

#ifdef __cplusplus
}
#endif
#endif /* MMQ_H */
