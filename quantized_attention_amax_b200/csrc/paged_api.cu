// paged_api.cu -- the C ABI's entry points on paged caches (include/faq.h): host-side argument
// validation and dispatch.
#include <cuda_runtime.h>

#include "internal.cuh"
#include "sm100.cuh"

namespace faq {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

fa_status from_cuda(cudaError_t e) {
  return e == cudaSuccess ? FA_OK : e == cudaErrorNotSupported ? FA_ERR_UNSUPPORTED : FA_ERR_CUDA;
}

bool per_head(int mode) { return mode == FA_MODE_INT8_PER_HEAD || mode == FA_MODE_FP8_PER_HEAD; }

fa_status check_cache(const fa_paged_cache* c) {
  if (!c) return FA_ERR_INVALID_ARG;
  if (!per_head(c->mode) && c->mode != FA_MODE_INT8_PER_TOKEN && c->mode != FA_MODE_FP8_PER_TOKEN)
    return FA_ERR_UNSUPPORTED;
  if (c->pages < 1 || c->H < 1 || (c->layout != FA_LAYOUT_BNSD && c->layout != FA_LAYOUT_BSND)) return FA_ERR_INVALID_ARG;
  if (c->D != 64 && c->D != 128) return FA_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1))) return FA_ERR_UNSUPPORTED;
  // strides inside a page are kept in 32 bits
  if ((long long)c->H * c->page_size * c->D > 0x7FFFFFFFLL) return FA_ERR_UNSUPPORTED;
  if (!c->k_scales || !c->v_scales || !aligned(c->k_scales, 4) || !aligned(c->v_scales, 4)) return FA_ERR_INVALID_ARG;
  if (!c->k_codes || !c->v_codes || !aligned(c->k_codes, 16) || !aligned(c->v_codes, 16))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

fa_status check_batch(const fa_paged_batch* b) {
  if (!b || b->B < 0 || b->max_pages < 0 || b->max_q < 0) return FA_ERR_INVALID_ARG;
  if (b->B == 0) return FA_OK;
  if (!b->seq_lens || !aligned(b->seq_lens, 4) || !aligned(b->cu_q, 4) || !aligned(b->page_table, 4) ||
      (b->max_pages > 0 && !b->page_table))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

fa_status check_rows(const fa_rows* r, int D) {
  if (!r || r->T < 0 || r->H < 1 || r->D != D) return FA_ERR_INVALID_ARG;
  if (r->stride < (long long)r->H * r->D || r->stride % 8 != 0) return FA_ERR_INVALID_ARG;
  if (r->T > 0 && (!r->data || !aligned(r->data, 16))) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// Do two ranges of bytes share any?
bool overlap(const void* a, long long na, const void* b, long long nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na > 0 && nb > 0 && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

// Do rows share bytes with a dense range?  Row i of r is [x + i s, x + i s + w): is there an i with both x + i s below
// the range's end and its own end above the range's start.
bool overlap(const fa_rows* r, const void* b, long long nb) {
  const long long s = r->stride * 2, w = (long long)r->H * r->D * 2;
  if (r->T < 1 || !overlap(r->data, (r->T - 1) * s + w, b, nb)) return false;
  const long long from = (long long)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(r->data));
  const long long i = from < w ? 0 : (from - w) / s + 1;  // the first row that ends past the range's start
  return i < r->T && i * s < from + nb;
}

// Do two sets of rows?  With one stride, columns side by side of one matrix do not; with two, ranges that cross count.
bool overlap(const fa_rows* a, const fa_rows* b) {
  const long long s = a->stride * 2, wa = (long long)a->H * a->D * 2, wb = (long long)b->H * b->D * 2;
  if (a->T < 1 || b->T < 1) return false;
  if (a->T == 1) return overlap(b, a->data, wa);
  if (b->T == 1) return overlap(a, b->data, wb);
  if (!overlap(a->data, (a->T - 1) * s + wa, b->data, (b->T - 1) * b->stride * 2 + wb)) return false;
  if (a->stride != b->stride) return true;
  const long long d = (long long)(reinterpret_cast<uintptr_t>(b->data) - reinterpret_cast<uintptr_t>(a->data));
  const long long m = ((d % s) + s) % s;  // where a row of b starts in a row of a
  return m < wa || m + wb > s;
}

// Largest cached length is kept in 32 bits: the table's tokens must fit.
bool lengths_fit(const fa_paged_cache* c, const fa_paged_batch* b) {
  return (long long)b->max_pages * c->page_size <= 0x40000000LL;
}

fa_status check_attend(const fa_rows* q, const fa_paged_cache* c, const fa_paged_batch* b) {
  fa_status st;
  if ((st = check_cache(c)) != FA_OK) return st;
  if ((st = check_batch(b)) != FA_OK) return st;
  if ((st = check_rows(q, c->D)) != FA_OK) return st;
  if (q->H % c->H != 0) return FA_ERR_INVALID_ARG;
  if (!b->cu_q && q->T != b->B) return FA_ERR_INVALID_ARG;
  if (!lengths_fit(c, b)) return FA_ERR_UNSUPPORTED;
  if ((long long)q->T * q->H > 0x7FFFFFFFLL) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

}  // namespace
}  // namespace faq

using namespace faq;

extern "C" {

fa_status fa_rope_table(float* table, int positions, int rotary_dim, const double* inv_freq, double factor,
                        fa_stream_t s) {
  if (positions < 0 || rotary_dim < 2 || rotary_dim > 128 || rotary_dim % 2 || !inv_freq) return FA_ERR_INVALID_ARG;
  if (positions == 0) return FA_OK;
  if (!table || !aligned(table, 4)) return FA_ERR_INVALID_ARG;
  return from_cuda(launch_rope_table(table, positions, rotary_dim, inv_freq, factor, reinterpret_cast<cudaStream_t>(s)));
}

fa_status fa_rope_append(const fa_rows* q, const fa_rows* k, const fa_rows* v, const fa_paged_cache* cache,
                         const fa_paged_batch* batch, const float* cos_sin, int table_positions, int rotary_dim,
                         const int* positions, int interleaved, const float* amax_k, const float* amax_v,
                         const fa_rows* q_out, fa_stream_t s) {
  fa_status st;
  if ((st = check_cache(cache)) != FA_OK) return st;
  if ((st = check_batch(batch)) != FA_OK) return st;
  if ((st = check_rows(k, cache->D)) != FA_OK) return st;
  if ((st = check_rows(v, cache->D)) != FA_OK) return st;
  if (k->H != cache->H || v->H != cache->H || v->T != k->T) return FA_ERR_INVALID_ARG;
  if (!q != !q_out) return FA_ERR_INVALID_ARG;
  if (q) {
    if ((st = check_rows(q, cache->D)) != FA_OK) return st;
    if ((st = check_rows(q_out, cache->D)) != FA_OK) return st;
    if (q->T != k->T || q_out->T != q->T || q_out->H != q->H) return FA_ERR_INVALID_ARG;
    if (q->data == q_out->data && q->stride != q_out->stride) return FA_ERR_INVALID_ARG;
    // in place, or apart: other warps read what a row of q_out lies on
    if ((q->data != q_out->data && overlap(q, q_out)) || overlap(k, q_out) || overlap(v, q_out)) return FA_ERR_INVALID_ARG;
  }
  if (!batch->cu_q && k->T != batch->B) return FA_ERR_INVALID_ARG;
  if (rotary_dim < 0 || rotary_dim > cache->D || rotary_dim % 16 != 0 || table_positions < 0) return FA_ERR_INVALID_ARG;
  if (rotary_dim > 0 && (!cos_sin || !aligned(cos_sin, 16))) return FA_ERR_INVALID_ARG;
  if (!aligned(positions, 4)) return FA_ERR_INVALID_ARG;
  if (per_head(cache->mode) && (!amax_k || !amax_v)) return FA_ERR_NO_CALIBRATION;
  if (!lengths_fit(cache, batch)) return FA_ERR_UNSUPPORTED;
  if (k->T == 0 || batch->B == 0) return FA_OK;
  int* status = device_status_ptr();
  if (!status) return FA_ERR_CUDA;
  const RopeAppendArgs a = {q,         k,           v,      cache,  batch, cos_sin, table_positions, rotary_dim,
                            positions, interleaved, amax_k, amax_v, q_out, status};
  return from_cuda(launch_rope_append(a, reinterpret_cast<cudaStream_t>(s)));
}

size_t fa_paged_attention_workspace_size(const fa_rows* q, const fa_paged_cache* cache, const fa_paged_batch* batch) {
  if (check_attend(q, cache, batch) != FA_OK) return 0;
  const PagedAttnArgs a = {q, cache, batch, 0, 0.0f, nullptr, nullptr, nullptr, nullptr, 0, 0};
  return paged_attention_ws(a);
}

fa_status fa_paged_attention(const fa_rows* q, const fa_paged_cache* cache, const fa_paged_batch* batch, int causal,
                             float softmax_scale, void* out, float* lse, void* workspace, size_t ws_bytes,
                             fa_stream_t s) {
  const fa_status st = check_attend(q, cache, batch);
  if (st != FA_OK) return st;
  if (q->T == 0 || batch->B == 0) return FA_OK;
  if (!out || !aligned(out, 16) || !aligned(lse, 4)) return FA_ERR_INVALID_ARG;
  // rows of q are read after others' results are written
  const long long n_out = (long long)q->T * q->H * q->D * 2, n_lse = (long long)q->T * q->H * 4;
  if (overlap(q, out, n_out) || overlap(q, lse, n_lse) || overlap(out, n_out, lse, n_lse)) return FA_ERR_INVALID_ARG;
  PagedAttnArgs a = {q, cache, batch, causal ? 1 : 0, softmax_scale, out, lse, nullptr, nullptr, 0, 0};
  const long long n_ws = (long long)paged_attention_ws(a);
  if (!workspace || ws_bytes < (size_t)n_ws || !aligned(workspace, 256)) return FA_ERR_WORKSPACE;
  if (overlap(q, workspace, n_ws) || overlap(out, n_out, workspace, n_ws) || overlap(lse, n_lse, workspace, n_ws))
    return FA_ERR_INVALID_ARG;
  a.status = device_status_ptr();
  if (!a.status) return FA_ERR_CUDA;
  return from_cuda(launch_paged_attention(a, workspace, reinterpret_cast<cudaStream_t>(s)));
}

fa_status fa_paged_weights(const fa_rows* q, const float* lse, const fa_paged_cache* cache, const fa_paged_batch* batch,
                           int causal, float softmax_scale, float* acc, long long acc_stride, int accumulate,
                           fa_stream_t s) {
  const fa_status st = check_attend(q, cache, batch);
  if (st != FA_OK) return st;
  if (acc_stride < 0) return FA_ERR_INVALID_ARG;
  if (batch->B == 0 || (q->T == 0 && accumulate)) return FA_OK;  // (no new token: the weights are zero)
  if ((q->T > 0 && !lse) || !aligned(lse, 4) || (acc_stride > 0 && !acc) || !aligned(acc, 4)) return FA_ERR_INVALID_ARG;
  const long long n_acc = (long long)batch->B * cache->H * acc_stride * 4;
  if (overlap(q, acc, n_acc) || overlap(lse, (long long)q->T * q->H * 4, acc, n_acc)) return FA_ERR_INVALID_ARG;
  int* status = device_status_ptr();
  if (!status) return FA_ERR_CUDA;
  const PagedAttnArgs a = {q,   cache, batch,      causal ? 1 : 0, softmax_scale, nullptr, const_cast<float*>(lse), status,
                           acc, acc_stride, accumulate ? 1 : 0};
  return from_cuda(launch_paged_weights(a, reinterpret_cast<cudaStream_t>(s)));
}

fa_status fa_paged_evict(const fa_paged_cache* cache, const fa_paged_batch* batch, const float* scores,
                         long long score_stride, int budget, int sink, int recent, int* kept, int* new_lens,
                         float* scores_out, fa_stream_t s) {
  fa_status st;
  if ((st = check_cache(cache)) != FA_OK) return st;
  if ((st = check_batch(batch)) != FA_OK) return st;
  if (score_stride < 0 || budget < 1 || sink < 0 || recent < 0 || (long long)sink + recent > budget)
    return FA_ERR_INVALID_ARG;
  // (a budget near 2^31 would pass 32 bits in the loops over its entries)
  if (!lengths_fit(cache, batch) || budget > 0x40000000) return FA_ERR_UNSUPPORTED;
  if (batch->B == 0) return FA_OK;
  if ((score_stride > 0 && !scores) || !aligned(scores, 4) || !kept || !aligned(kept, 4) || !new_lens ||
      !aligned(new_lens, 4) || !aligned(scores_out, 4))
    return FA_ERR_INVALID_ARG;
  // the outputs lie apart from each other and from what other CTAs still read (new_lens is not seq_lens)
  const long long items = (long long)batch->B * cache->H, n_sc = items * score_stride * 4, n_kept = items * budget * 4;
  const long long n_b = (long long)batch->B * 4, n_tab = n_b * batch->max_pages;
  const void* outs[3] = {scores_out, kept, new_lens};
  const long long n_out[3] = {n_sc, n_kept, n_b};
  for (int i = 0; i < 3; ++i) {
    if (overlap(outs[i], n_out[i], scores, n_sc) || overlap(outs[i], n_out[i], batch->seq_lens, n_b) ||
        overlap(outs[i], n_out[i], batch->page_table, n_tab))
      return FA_ERR_INVALID_ARG;
    for (int k = 0; k < i; ++k)
      if (overlap(outs[i], n_out[i], outs[k], n_out[k])) return FA_ERR_INVALID_ARG;
  }
  int* status = device_status_ptr();
  if (!status) return FA_ERR_CUDA;
  const PagedEvictArgs a = {cache, batch, scores, score_stride, budget, sink, recent, kept, new_lens, scores_out, status};
  return from_cuda(launch_paged_evict(a, reinterpret_cast<cudaStream_t>(s)));
}

}  // extern "C"
