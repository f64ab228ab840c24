// serving.cu -- the extern "C" entry points of the serving step around the
// projections (declared in mmq.h): argument checks and launches.
#include <cuda_runtime.h>

#include <cmath>

#include "checks.h"
#include "internal.h"

using mmq::aligned, mmq::aligned_elements, mmq::check_cache, mmq::cuda_rc, mmq::kInt32, mmq::meet, mmq::Run;

extern "C" {

int mmq_page_tables(const int32_t *cached, const int32_t *fresh, const int32_t *held, int64_t nreq, int32_t *table,
                    int64_t table_width, int64_t table_stride, const int32_t *free_pages, int64_t nfree,
                    int32_t page_size, int64_t max_tokens, int32_t *q_start, int32_t *seq_lens, int32_t *held_out,
                    int64_t *slots, int32_t *positions, int32_t *taken, mmq_stream_t stream) {
  if (nreq < 0 || table_width < 0 || table_width > kInt32 || table_stride < table_width || nfree < 0 || nfree > kInt32 ||
      page_size < 1 || max_tokens < 0 || max_tokens > kInt32)
    return MMQ_ERR_ARG;
  if (nreq > mmq::kMaxRequests) return MMQ_ERR_UNSUPPORTED;
  if (!q_start || !taken) return MMQ_ERR_ARG;
  if (nreq && (!cached || !fresh || !held || !seq_lens || !held_out)) return MMQ_ERR_ARG;
  if ((nreq && table_width && !table) || (nfree && !free_pages) || (max_tokens && (!slots || !positions))) return MMQ_ERR_ARG;
  // CTAs read the lengths and the free list again after others have written
  // theirs, so nothing that is written may lie on anything else.
  const Run written[] = {{q_start, nreq + 1}, {seq_lens, nreq}, {held_out, nreq}, {slots, max_tokens}, {positions, max_tokens}, {taken, 2}};
  const Run read[] = {{cached, nreq}, {fresh, nreq}, {held, nreq}, {free_pages, nfree}}, rows(table, table_width, table_stride, nreq);
  for (const Run &w : written) {
    if (meet(w, rows)) return MMQ_ERR_ARG;
    for (const Run &x : written)
      if (&x != &w && meet(w, x)) return MMQ_ERR_ARG;
    for (const Run &x : read)
      if (meet(w, x)) return MMQ_ERR_ARG;
  }
  for (const Run &x : read)
    if (meet(x, rows)) return MMQ_ERR_ARG;
  if (!aligned_elements(cached, fresh, held, table, free_pages, q_start, seq_lens, held_out, slots, positions, taken)) return MMQ_ERR_ALIGN;
  mmq::CallContext ctx;
  if (int rc = mmq::call_context(&ctx)) return rc;
  mmq::PageTablesArgs a;
  a.cached = cached, a.fresh = fresh, a.held = held, a.table = table, a.free_pages = free_pages;
  a.q_start = q_start, a.seq_lens = seq_lens, a.held_out = held_out, a.slots = slots, a.positions = positions;
  a.taken = taken, a.table_stride = table_stride, a.table_width = table_width, a.nfree = nfree;
  a.max_tokens = max_tokens, a.nreq = static_cast<int32_t>(nreq), a.page_size = page_size;
  return cuda_rc(mmq::launch_page_tables(a, reinterpret_cast<cudaStream_t>(stream)));
}

int mmq_kv_write(const mmq_paged_cache *cache, const void *k, int64_t k_token, int64_t k_head, const void *v,
                 int64_t v_token, int64_t v_head, int src_type, const int64_t *slots, int64_t ntok,
                 mmq_stream_t stream) {
  if (int rc = check_cache(cache)) return rc;
  if (src_type != MMQ_DT_F32 && src_type != MMQ_DT_F16 && src_type != MMQ_DT_BF16) return MMQ_ERR_TYPE;
  if (ntok < 0 || ntok > kInt32 || k_token < 0 || k_head < 0 || v_token < 0 || v_head < 0) return MMQ_ERR_ARG;
  if (cache->heads > (int64_t(1) << 30) / (2 * (cache->head_dim / 8))) return MMQ_ERR_UNSUPPORTED;  // a token's chunks, in 32 bits
  if (ntok == 0) return MMQ_OK;
  if (!k || !v || !slots) return MMQ_ERR_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8) || (k_token | k_head | v_token | v_head) % 8) return MMQ_ERR_ALIGN;
  mmq::CallContext ctx;
  if (int rc = mmq::call_context(&ctx)) return rc;
  mmq::KvWriteArgs a;
  a.cache = *cache, a.k = k, a.v = v, a.k_token = k_token, a.k_head = k_head, a.v_token = v_token, a.v_head = v_head;
  a.slots = slots, a.ntok = ntok, a.heads = cache->heads, a.head_dim = cache->head_dim, a.src_type = src_type;
  a.tokens_per_cta = 1, a.status = &ctx.words->status;
  return cuda_rc(mmq::launch_kv_write(a, reinterpret_cast<cudaStream_t>(stream)));
}

int mmq_paged_attention(const mmq_paged_cache *cache, const mmq_attention *args, mmq_stream_t stream) {
  if (int rc = check_cache(cache)) return rc;
  if (!args) return MMQ_ERR_ARG;
  const mmq_attention &t = *args;
  if (t.out_type != cache->type && t.out_type != MMQ_DT_F32) return MMQ_ERR_TYPE;
  if (t.nreq < 0 || t.nreq > kInt32 || t.ntok < 0 || t.table_width < 0 || t.table_stride < t.table_width || t.q_heads < 1 ||
      t.q_heads % cache->heads || t.window < 0)
    return MMQ_ERR_ARG;
  if (!(t.scale > 0.0f) || std::isinf(t.scale)) return MMQ_ERR_ARG;
  if (t.q_token < 0 || t.q_head < 0 || t.out_token < 0 || t.out_head < 0) return MMQ_ERR_ARG;
  if (t.ntok > (kInt32 - 512) / t.q_heads) return MMQ_ERR_ARG;  // rows are counted in 32 bits, a unit's past the last one
  if (t.nreq == 0 || t.ntok == 0) return MMQ_OK;
  if (!t.q || !t.out || !t.seq_lens || !t.q_start || (t.table_width && !t.table)) return MMQ_ERR_ARG;
  if (!aligned_elements(t.lse, t.table, t.seq_lens, t.q_start)) return MMQ_ERR_ALIGN;
  if (!aligned(t.q, 16) || !aligned(t.out, 16) || (t.q_token | t.q_head | t.out_token | t.out_head) % 8) return MMQ_ERR_ALIGN;
  mmq::CallContext ctx;
  if (int rc = mmq::call_context(&ctx)) return rc;
  return cuda_rc(mmq::launch_attention(*cache, t, ctx, reinterpret_cast<cudaStream_t>(stream)));
}

int mmq_verify_draft(const mmq_verification *args, mmq_stream_t stream) {
  if (!args) return MMQ_ERR_ARG;
  const mmq_verification &t = *args;
  if (t.type != MMQ_DT_F32 && t.type != MMQ_DT_F16 && t.type != MMQ_DT_BF16) return MMQ_ERR_TYPE;
  if (t.nreq < 0 || t.nreq > 65535 || t.vocab < 1 || t.vocab > kInt32 || t.k < 0 || t.k == kInt32) return MMQ_ERR_ARG;
  if (t.target_req < 0 || t.target_row < 0 || t.draft_req < 0 || t.draft_row < 0 || t.tokens_stride < 0 || t.u_stride < 0 ||
      t.noise_stride < 0)
    return MMQ_ERR_ARG;
  if (t.nreq == 0) return MMQ_OK;
  if (!t.target || !t.noise || !t.out || !t.accepted || (t.k && (!t.tokens || !t.u))) return MMQ_ERR_ARG;
  const uintptr_t esz = t.type == MMQ_DT_F32 ? 4 : 2;
  if (!aligned(t.target, esz) || !aligned(t.draft, esz)) return MMQ_ERR_ALIGN;
  if (!aligned_elements(t.tokens, t.n_draft, t.u, t.noise, t.out, t.accepted)) return MMQ_ERR_ALIGN;
  mmq::CallContext ctx;
  if (int rc = mmq::call_context(&ctx)) return rc;
  mmq::VerifyArgs a;
  a.target = t.target, a.draft = t.draft, a.tokens = t.tokens, a.n_draft = t.n_draft, a.u = t.u, a.noise = t.noise;
  a.out = t.out, a.accepted = t.accepted, a.target_req = t.target_req, a.target_row = t.target_row;
  a.draft_req = t.draft_req, a.draft_row = t.draft_row, a.tokens_stride = t.tokens_stride, a.u_stride = t.u_stride;
  a.noise_stride = t.noise_stride, a.nreq = t.nreq, a.vocab = t.vocab, a.k = t.k, a.type = t.type;
  a.status = &ctx.words->status;
  return cuda_rc(mmq::launch_verify(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
