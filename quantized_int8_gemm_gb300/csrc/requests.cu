// requests.cu -- the extern "C" entry points of what differs from request to
// request in a serving step (declared in mmq.h): argument checks and launches.
#include <cuda_runtime.h>

#include <algorithm>

#include "checks.h"
#include "internal.h"

using mmq::aligned, mmq::aligned_elements, mmq::check_cache, mmq::cuda_rc, mmq::kInt32, mmq::kMaxAdapters, mmq::kMaxPages, mmq::kMaxRequests,
    mmq::kMaxVocab, mmq::meet, mmq::Run;

namespace {

constexpr int64_t kMaxWidth = kInt32 - 1023;  // of page tables: columns of a round of warps behind the last one stay in 32 bits
constexpr int64_t kMostColumns = int64_t(1) << 28;  // of x and out: bytes in a row stay below 2^31

bool is_type(int t) { return t == MMQ_DT_F32 || t == MMQ_DT_F16 || t == MMQ_DT_BF16; }
int64_t size_of(int t) { return t == MMQ_DT_F32 ? 4 : 2; }

// Whether what is written (the rows of a new table, and runs) lies on nothing
// else of the call.
template <size_t kWritten, size_t kRead>
bool apart(const Run (&written)[kWritten], const Run (&read)[kRead], const Run &old_rows, const Run &new_rows) {
  for (const Run &w : written) {
    if (meet(w, old_rows) || meet(w, new_rows)) return false;
    for (const Run &x : written)
      if (&x != &w && meet(w, x)) return false;
    for (const Run &x : read)
      if (meet(w, x)) return false;
  }
  for (const Run &x : read)
    if (meet(x, new_rows)) return false;
  Run whole = new_rows;  // (rows by rows only where the whole stretches meet: halves of wider rows do)
  whole.bytes += new_rows.rows ? (new_rows.rows - 1) * new_rows.pitch : 0, whole.rows = 1;
  if (!meet(whole, old_rows)) return true;
  for (uint64_t r = 0; r < new_rows.rows; ++r) {
    Run row = new_rows;
    row.at += r * row.pitch, row.rows = 1;
    if (meet(row, old_rows)) return false;
  }
  return true;
}

bool table_fits(int64_t nreq, int64_t width, int64_t stride) {
  return nreq >= 0 && width >= 0 && width <= kInt32 && stride >= width && stride <= (int64_t(1) << 40);
}

// Whether n strides stay below any memory there is.
bool spans(int64_t n, int64_t stride) { return stride >= 0 && stride <= (int64_t(1) << 48) / (n > 0 ? n : 1); }

// Rows of n elements in two strides: blocks of rows, the larger stride between blocks.
struct Rows {
  Run block;  // the first one's
  uint64_t pitch, blocks;
  template <class T>
  Rows(const T *p, int64_t n, int64_t s0, int64_t n0, int64_t s1 = 0, int64_t n1 = 1)
      : block(p, p ? n : 0, std::min(s0, s1), s0 < s1 ? n0 : n1), pitch(std::max(s0, s1) * sizeof(T)), blocks(s0 < s1 ? n1 : n0) {}
  uint64_t block_bytes() const { return (block.rows - 1) * block.pitch + block.bytes; }
};
bool meet(const Run &a, const Rows &b) {
  if (!a.bytes || !b.block.bytes || !b.block.rows || !b.blocks) return false;
  // from the first block that ends behind a's begin to the last that begins in front of its end
  const uint64_t bytes = b.block_bytes(), blocks = b.pitch ? b.blocks : 1;
  Run block = b.block;
  uint64_t k = a.at < block.at + bytes ? 0 : b.pitch ? (a.at - block.at - bytes) / b.pitch + 1 : 1;
  for (block.at += k * b.pitch; k < blocks && block.at < a.at + a.bytes; ++k, block.at += b.pitch)
    if (mmq::meet(a, block)) return true;
  return false;
}
// Row by row only where the whole stretches meet (halves of wider rows do).
bool meet(const Rows &a, const Rows &b) {
  auto whole = [](const Rows &r) {
    Run w = r.block;
    if (w.bytes && r.block.rows && r.blocks) w.bytes = (r.blocks - 1) * r.pitch + r.block_bytes();
    w.rows = 1;
    return w;
  };
  if (!mmq::meet(whole(a), whole(b))) return false;
  for (uint64_t k = 0; k < a.blocks; ++k)
    for (uint64_t i = 0; i < a.block.rows; ++i) {
      Run row = a.block;
      row.at += k * a.pitch + i * a.block.pitch, row.rows = 1;
      if (meet(row, b)) return true;
    }
  return false;
}

}  // namespace

extern "C" {

int mmq_page_fork(const mmq_fork *args, mmq_stream_t stream) {
  if (!args) return MMQ_ERR_ARG;
  const mmq_fork &t = *args;
  if (!table_fits(t.nold, t.table_width, t.table_stride) || !table_fits(t.nnew, t.table_width, t.new_stride) || t.npages < 0 ||
      t.page_size < 1)
    return MMQ_ERR_ARG;
  if (t.nold > kMaxRequests || t.nnew > kMaxRequests || t.npages > kMaxPages || t.table_width > kMaxWidth) return MMQ_ERR_UNSUPPORTED;
  if (!t.counts || (t.npages && !t.free_pages)) return MMQ_ERR_ARG;
  if (t.nold && (!t.held || (t.table_width && !t.table))) return MMQ_ERR_ARG;
  if (t.nnew && (!t.parents || !t.lens || !t.held_out || !t.pairs || !t.tokens || (t.table_width && !t.new_table))) return MMQ_ERR_ARG;
  if (!aligned_elements(t.table, t.held, t.parents, t.lens, t.new_table, t.held_out, t.pairs, t.tokens, t.free_pages, t.counts)) return MMQ_ERR_ALIGN;
  const Run written[] = {{t.held_out, t.nnew}, {t.pairs, 2 * t.nnew}, {t.tokens, t.nnew}, {t.free_pages, t.npages}, {t.counts, 2}};
  const Run read[] = {{t.held, t.nold}, {t.parents, t.nnew}, {t.lens, t.nnew}};
  if (!apart(written, read, Run(t.table, t.table_width, t.table_stride, t.nold), Run(t.new_table, t.table_width, t.new_stride, t.nnew)))
    return MMQ_ERR_ARG;
  mmq::CallContext ctx;
  if (int rc = mmq::call_context(&ctx)) return rc;
  mmq::ForkArgs a;
  static_cast<mmq_fork &>(a) = t;
  a.status = &ctx.words->status;
  return cuda_rc(mmq::launch_page_fork(a, reinterpret_cast<cudaStream_t>(stream)));
}

int mmq_page_compact(const int32_t *table, const int32_t *held, int64_t nreq, int64_t table_width, int64_t table_stride,
                     int64_t npages, int32_t *new_table, int64_t new_stride, int32_t *pairs, int32_t *counts,
                     mmq_stream_t stream) {
  if (!table_fits(nreq, table_width, table_stride) || !table_fits(nreq, table_width, new_stride) || npages < 0) return MMQ_ERR_ARG;
  if (nreq > kMaxRequests || npages > kMaxPages || table_width > kMaxWidth) return MMQ_ERR_UNSUPPORTED;
  if (!counts || (npages > 1 && !pairs) || (nreq && (!held || (table_width && (!table || !new_table))))) return MMQ_ERR_ARG;
  if (!aligned_elements(table, held, new_table, counts) || !aligned(pairs, 8)) return MMQ_ERR_ALIGN;
  const Run written[] = {{pairs, npages / 2 * 2}, {counts, 2}};
  const Run read[] = {{held, nreq}};
  if (!apart(written, read, Run(table, table_width, table_stride, nreq), Run(new_table, table_width, new_stride, nreq))) return MMQ_ERR_ARG;
  mmq::CallContext ctx;
  if (int rc = mmq::call_context(&ctx)) return rc;
  mmq::CompactArgs a;
  a.table = table, a.held = held, a.nreq = nreq, a.table_width = table_width, a.table_stride = table_stride, a.npages = npages;
  a.new_table = new_table, a.new_stride = new_stride, a.pairs = pairs, a.counts = counts, a.status = &ctx.words->status;
  return cuda_rc(mmq::launch_page_compact(a, reinterpret_cast<cudaStream_t>(stream)));
}

int mmq_page_copy(const mmq_paged_cache *cache, const int32_t *pairs, const int32_t *tokens, int64_t npairs, mmq_stream_t stream) {
  if (int rc = check_cache(cache)) return rc;
  if (npairs < 0 || npairs > kInt32) return MMQ_ERR_ARG;
  if (int64_t(cache->page_size) * cache->heads > (int64_t(1) << 29) / (cache->head_dim / 8)) return MMQ_ERR_UNSUPPORTED;  // a page's chunks, in 32 bits
  if (npairs == 0) return MMQ_OK;
  if (!pairs) return MMQ_ERR_ARG;
  if (!aligned_elements(pairs, tokens)) return MMQ_ERR_ALIGN;
  mmq::CallContext ctx;
  if (int rc = mmq::call_context(&ctx)) return rc;
  mmq::PageCopyArgs a;
  a.cache = *cache, a.pairs = pairs, a.tokens = tokens, a.npairs = npairs, a.status = &ctx.words->status;
  return cuda_rc(mmq::launch_page_copy(a, reinterpret_cast<cudaStream_t>(stream)));
}

int mmq_token_probs(const mmq_token_rules *args, mmq_stream_t stream) {
  if (!args) return MMQ_ERR_ARG;
  const mmq_token_rules &t = *args;
  if (!is_type(t.type) || (t.probs && !is_type(t.probs_type)) || (t.adjusted && !is_type(t.adjusted_type))) return MMQ_ERR_TYPE;
  if (t.nreq < 0 || t.rows < 1 || t.vocab < 1 || t.tokens_width < 0 || t.tokens_width > kInt32 || t.nbias < 0 || t.nbias > kInt32 ||
      t.nmasks < 0 || t.nmasks > kInt32)
    return MMQ_ERR_ARG;
  for (int64_t stride : {t.logits_req, t.probs_req, t.adjusted_req, t.tokens_stride, t.draft_stride})
    if (!spans(t.nreq, stride)) return MMQ_ERR_ARG;
  for (int64_t stride : {t.logits_row, t.probs_row, t.adjusted_row})
    if (!spans(t.rows, stride)) return MMQ_ERR_ARG;
  if (!spans(t.nmasks, t.mask_stride)) return MMQ_ERR_ARG;
  if (t.vocab > kMaxVocab || t.tokens_width > mmq::kMaxSaid || t.nbias > mmq::kMaxBiases) return MMQ_ERR_UNSUPPORTED;
  if (t.nreq > ((int64_t(1) << 27) - 1) / t.rows) return MMQ_ERR_UNSUPPORTED;
  if (t.nreq == 0) return MMQ_OK;
  if (!t.logits || (!t.probs && !t.adjusted) || (t.tokens_width && !t.tokens) || (t.nbias && (!t.bias_ids || !t.bias_values))) return MMQ_ERR_ARG;
  if (t.mask && t.mask_stride < (t.vocab + 31) / 32 && t.nmasks > 1) return MMQ_ERR_ARG;
  if (!aligned(t.logits, size_of(t.type)) || !aligned(t.probs, size_of(t.probs_type)) || !aligned(t.adjusted, size_of(t.adjusted_type))) return MMQ_ERR_ALIGN;
  if (!aligned_elements(t.temperature, t.tokens, t.token_lens, t.prompt_lens, t.draft, t.n_draft, t.repetition, t.frequency, t.presence,
                        t.bias_start, t.bias_ids, t.bias_values, t.mask, t.mask_rows))
    return MMQ_ERR_ALIGN;
  // what is written overlaps no row that another cluster reads or writes
  auto rows_of = [&](const void *p, int type, int64_t req, int64_t row) {
    if (type == MMQ_DT_F32) return Rows(static_cast<const float *>(p), t.vocab, req, t.nreq, row, t.rows);
    return Rows(static_cast<const uint16_t *>(p), t.vocab, req, t.nreq, row, t.rows);
  };
  auto rows_apart = [&](int64_t req, int64_t row) {  // rows do not lie on one another
    return (t.rows == 1 || row >= t.vocab) && (t.nreq == 1 || req >= (t.rows - 1) * row + t.vocab || (t.rows > 1 && row >= (t.nreq - 1) * req + t.vocab && req >= t.vocab));
  };
  const Rows logits = rows_of(t.logits, t.type, t.logits_req, t.logits_row), probs = rows_of(t.probs, t.probs_type, t.probs_req, t.probs_row);
  const Rows adjusted = rows_of(t.adjusted, t.adjusted_type, t.adjusted_req, t.adjusted_row);
  const bool same = t.adjusted == t.logits && t.adjusted_type == t.type && t.adjusted_req == t.logits_req && t.adjusted_row == t.logits_row;
  if (t.probs && (!rows_apart(t.probs_req, t.probs_row) || meet(probs, logits) || meet(probs, adjusted))) return MMQ_ERR_ARG;
  if (t.adjusted && (!rows_apart(t.adjusted_req, t.adjusted_row) || (!same && meet(adjusted, logits)))) return MMQ_ERR_ARG;
  auto vector = [](const auto *p, int64_t n) { return Rows(p, n, 0, 1); };
  const Rows read[] = {vector(t.temperature, t.nreq), vector(t.token_lens, t.nreq), vector(t.prompt_lens, t.nreq), vector(t.n_draft, t.nreq),
                       vector(t.repetition, t.nreq), vector(t.frequency, t.nreq), vector(t.presence, t.nreq), vector(t.bias_start, t.nreq + 1),
                       vector(t.bias_ids, t.nbias), vector(t.bias_values, t.nbias), vector(t.mask_rows, t.nreq * t.rows),
                       Rows(t.tokens, t.tokens_width, t.tokens_stride, t.nreq), Rows(t.draft, t.rows - 1, t.draft_stride, t.nreq),
                       Rows(t.mask, (t.vocab + 31) / 32, t.mask_stride, t.nmasks)};
  for (const Rows &r : read)
    if (meet(probs, r) || meet(adjusted, r)) return MMQ_ERR_ARG;
  mmq::RulesArgs a;
  a.t = t;
  if (!t.tokens) a.t.tokens_width = 0;
  if (t.nbias == 0) a.t.bias_start = nullptr;
  a.in_place = same;
  a.penalties = (a.t.tokens_width > 0 || (t.draft && t.rows > 1)) && (t.repetition || t.frequency || t.presence);
  if ((a.penalties || a.t.bias_start) && t.nreq > mmq::kMaxListed) return MMQ_ERR_UNSUPPORTED;
  mmq::CallContext ctx;
  if (int rc = mmq::call_context(&ctx)) return rc;
  a.status = &ctx.words->status, a.abort_epoch = &ctx.words->abort_epoch, a.epoch = ctx.epoch, a.limit_ns = ctx.limit_ns;
  return cuda_rc(mmq::launch_token_probs(a, ctx, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t mmq_lora_plan_words(int64_t ntok, int64_t nreq, int64_t nadapters) {
  if (ntok < 0 || ntok > kInt32 / 64 || nreq < 0 || nreq > kMaxRequests || nadapters < 0 || nadapters > kMaxAdapters) return -1;
  return mmq::lora_plan_words(ntok, nreq, nadapters);
}

int mmq_lora_plan(const int32_t *adapters, const int32_t *q_start, int64_t nreq, int64_t ntok, int64_t nadapters, int32_t *plan,
                  mmq_stream_t stream) {
  if (nreq < 0 || ntok < 0 || nadapters < 0) return MMQ_ERR_ARG;
  if (mmq_lora_plan_words(ntok, nreq, nadapters) < 0) return MMQ_ERR_UNSUPPORTED;
  if (!plan || !q_start || (nreq && !adapters)) return MMQ_ERR_ARG;
  if (!aligned_elements(adapters, q_start, plan)) return MMQ_ERR_ALIGN;
  const Run words(plan, mmq::lora_plan_words(ntok, nreq, nadapters));
  if (meet(words, Run(adapters, nreq)) || meet(words, Run(q_start, nreq + 1))) return MMQ_ERR_ARG;
  mmq::CallContext ctx;
  if (int rc = mmq::call_context(&ctx)) return rc;
  mmq::LoraPlanArgs a;
  a.adapters = adapters, a.q_start = q_start, a.nreq = nreq, a.ntok = ntok, a.nadapters = nadapters, a.plan = plan;
  a.status = &ctx.words->status;
  return cuda_rc(mmq::launch_lora_plan(a, reinterpret_cast<cudaStream_t>(stream)));
}

int mmq_lora(const mmq_lora_args *args, mmq_stream_t stream) {
  if (!args) return MMQ_ERR_ARG;
  const mmq_lora_args &t = *args;
  if ((t.type != MMQ_DT_F16 && t.type != MMQ_DT_BF16) || !is_type(t.x_type)) return MMQ_ERR_TYPE;
  if (t.ntok < 0 || t.nreq < 0 || t.nadapters < 0 || t.id < 8 || t.id % 8 || t.od < 1 || t.rank < 8 || t.rank % 8 || t.rank > mmq::kMaxRank) return MMQ_ERR_ARG;
  for (int64_t stride : {t.x_row, t.y_row, t.out_row})
    if (!spans(t.ntok, stride)) return MMQ_ERR_ARG;
  if (t.id > kMostColumns || t.od > kMostColumns || mmq_lora_plan_words(t.ntok, t.nreq, t.nadapters) < 0) return MMQ_ERR_UNSUPPORTED;
  if (t.ntok == 0 || t.nreq == 0) return MMQ_OK;
  if (!t.x || !t.y || !t.out || !t.plan || (t.nadapters && (!t.a || !t.b))) return MMQ_ERR_ARG;
  if (!aligned(t.x, 16) || !aligned(t.a, 16) || !aligned(t.b, 16) || t.x_row * size_of(t.x_type) % 16) return MMQ_ERR_ALIGN;
  if (!aligned_elements(t.y, t.out, t.scales, t.ranks, t.plan)) return MMQ_ERR_ALIGN;
  if (t.ntok > 1 && t.out_row < t.od) return MMQ_ERR_ARG;  // rows that lie on one another
  if (t.y == t.out) {
    if (t.ntok > 1 && t.y_row != t.out_row) return MMQ_ERR_ARG;
  }
  const Run x(static_cast<const char *>(t.x), t.id * size_of(t.x_type), t.x_row * size_of(t.x_type), t.ntok), y(t.y, t.od, t.y_row, t.ntok);
  const Run rest[] = {{static_cast<const char *>(t.a), 2 * t.nadapters * t.rank * t.id}, {static_cast<const char *>(t.b), 2 * t.nadapters * t.od * t.rank},
                      {t.scales, t.scales ? t.nadapters : 0}, {t.ranks, t.ranks ? t.nadapters : 0},
                      {t.plan, mmq::lora_plan_words(t.ntok, t.nreq, t.nadapters)}};
  Run out(t.out, t.od, t.out_row, t.ntok);
  for (const Run &r : rest)
    if (meet(r, out)) return MMQ_ERR_ARG;
  // rows by rows only where the whole stretches meet (columns of one array do)
  auto span = [](const Run &r) { Run s = r; s.bytes += (r.rows - 1) * r.pitch, s.rows = 1; return s; };
  for (const Run *other : {&x, t.y == t.out ? nullptr : &y}) {
    if (!other || !meet(span(out), span(*other))) continue;
    Run row = out;
    row.rows = 1;
    for (uint64_t k = 0; k < out.rows; ++k, row.at += out.pitch)
      if (meet(row, *other)) return MMQ_ERR_ARG;
  }
  mmq::CallContext ctx;
  if (int rc = mmq::call_context(&ctx)) return rc;
  mmq::LoraArgs a;
  a.t = t;
  if (t.ntok == 1) a.t.x_row = 0, a.t.y_row = 0, a.t.out_row = 0;
  return cuda_rc(mmq::launch_lora(a, ctx, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
