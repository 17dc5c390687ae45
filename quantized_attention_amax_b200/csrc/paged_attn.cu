// paged_attn.cu -- attention over a paged cache: which kernel serves which sequences.
//
// D = 128: sequences of up to 16 query rows per kv head (new tokens x the group's query heads) go to the
// decode kernel, which reads the codes as 8-bit MMA operands and is bound by their bytes; those of more to the chunk
// kernel, whose 128-row tiles they fill.  D = 64: all to the chunk kernel.
#include <cuda_runtime.h>

#include "paged_sched.cuh"

namespace faq {

size_t paged_attention_ws(const PagedAttnArgs& a) {
  const int D = a.q->D;
  if (D == 128 && paged_most_rows(a) <= 16) return paged_decode_ws();
  return paged_chunk_ws(D);
}

cudaError_t launch_paged_attention(const PagedAttnArgs& a, void* ws, cudaStream_t s) {
  const int D = a.q->D;
  const long long rows = paged_most_rows(a);
  if (D == 128) {
    // sequences of up to 16 query rows per kv head, then those of more
    const cudaError_t e = launch_paged_decode(a, rows < 16 ? (int)rows : 16, ws, s);
    if (e != cudaSuccess || rows <= 16) return e;
  }
  return launch_paged_chunk(a, ws, s);
}

}  // namespace faq
