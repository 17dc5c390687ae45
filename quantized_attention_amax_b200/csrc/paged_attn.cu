// paged_attn.cu -- attention over a paged cache: which kernel serves which sequences.
//
// Sequences of up to 16 query rows per kv head (new tokens x the group's query heads) go to the decode kernel, which
// reads the codes as 8-bit MMA operands and is bound by their bytes; those of more to the chunk kernel, whose
// 128-row tiles they fill.
#include <cuda_runtime.h>

#include "paged_sched.cuh"

namespace faq {

size_t paged_attention_ws(const PagedAttnArgs& a) {
  return paged_most_rows(a) <= 16 ? paged_decode_ws(a.q->D) : paged_chunk_ws(a.q->D);
}

cudaError_t launch_paged_attention(const PagedAttnArgs& a, void* ws, cudaStream_t s) {
  const long long rows = paged_most_rows(a);
  // the decode kernel's workspace is the smaller one, and is done with when the chunk kernel starts
  const cudaError_t e = launch_paged_decode(a, rows < 16 ? (int)rows : 16, ws, s);
  return e != cudaSuccess || rows <= 16 ? e : launch_paged_chunk(a, ws, s);
}

}  // namespace faq
