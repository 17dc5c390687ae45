// paged_common.cuh -- what the paged-cache kernels share: the cache and batch as kernels see them,
// the checks of lengths and pages, and the conversions of 8-bit codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "attn_common.cuh"
#include "internal.cuh"
#include "sm100.cuh"

namespace faq {
namespace paged {

// A paged cache with its strides in bytes (codes), so that both layouts share one address rule:
// code row of slot `o` of page `pg`, head h: pg * page_stride + h * head_stride + o * tok_stride.
struct Cache {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  long long page_stride;
  int head_stride, tok_stride;
  int pages, H, page_shift, page_mask;
  int per_token;  // scales [pages, H, page_size], else [H]
  int bnsd;       // pages are [H, page_size, D], else [page_size, H, D]

  __device__ __forceinline__ long long row(int pg, int h, int slot) const {
    return (long long)pg * page_stride + (long long)h * head_stride + (long long)slot * tok_stride;
  }
  __device__ __forceinline__ long long scale(int pg, int h, int slot) const {
    return (((long long)pg * H + h) << page_shift) + slot;
  }
  // FA_DEBUG_BOUNDS builds: `n` bytes of codes from `off`, and the per-token modes' scale `i`
  __device__ __forceinline__ bool holds(long long off, int n, int where) const {
    return in_bounds(off >= 0 && off + n <= (long long)pages * page_stride, where);
  }
  __device__ __forceinline__ bool holds_scale(long long i, int where) const {
    return in_bounds(i >= 0 && i < (long long)pages * H * (page_mask + 1), where);
  }
};

struct Batch {
  const int* table;
  const int* lens;
  const int* cu;  // nullptr: one new token per sequence
  int B, max_pages, max_q, T;
};

// Record a failed check of caller data (a length, page or position) in the status word.
__device__ __forceinline__ void bad(int* status, int where) {
  atomicCAS(status, 0, (where << 8) | kStatusBounds);
}

// Sequence b: its first new-token row, number of new tokens and cached tokens, checked.  A
// sequence that fails a check reads as (0, 0, 0).
struct Seq {
  int q0, m, n;
};
__device__ __forceinline__ Seq load_seq(const Batch& bt, int page_shift, int b, int* status, int where) {
  Seq s;
  if (!in_bounds(b >= 0 && b < bt.B, 162)) return {0, 0, 0};
  s.q0 = bt.cu ? __ldg(bt.cu + b) : b;
  const int q1 = bt.cu ? __ldg(bt.cu + b + 1) : b + 1;
  s.n = __ldg(bt.lens + b);
  s.m = q1 - s.q0;
  const bool ok = s.q0 >= 0 && q1 >= s.q0 && q1 <= bt.T && s.m <= bt.max_q && s.n >= 0 &&
                  s.n <= ((long long)bt.max_pages << page_shift);
  if (!ok) {
    bad(status, where);
    s = {0, 0, 0};
  }
  return s;
}

// Page of cache index j of sequence b, or -1 (recorded) if it is not a page of the cache.
__device__ __forceinline__ int page_of(const Batch& bt, const Cache& c, int b, int j, int* status, int where) {
  if (!in_bounds(b >= 0 && b < bt.B && j >= 0 && (j >> c.page_shift) < bt.max_pages, 161)) return -1;
  const int pg = __ldg(bt.table + (long long)b * bt.max_pages + (j >> c.page_shift));
  if ((unsigned)pg >= (unsigned)c.pages) {
    bad(status, where);
    return -1;
  }
  return pg;
}

// A scale as the kernels use it: one that is NaN or infinite makes what it scales NaN.
__device__ __forceinline__ float finite_or_nan(float s) { return fabsf(s) < INFINITY ? s : __uint_as_float(0x7FC00000u); }

// The E4M3 NaN codes (0x7F and 0xFF) of a word's four: 0x80 in their bytes.
__device__ __forceinline__ uint32_t e4m3_nans(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Where V is no number: in a tile that some rows do not see whole, NaN codes would reach rows that do not see them (0
// times NaN is NaN), so they are cleared, and the lowest key whose element d was one is kept for d here; the
// rows that see that key get their NaN when they are written.
__device__ __forceinline__ void note_nans(uint32_t nans, int d, int key, int* nan_key) {
  for (; nans; nans &= nans - 1) atomicMin(nan_key + d + ((__ffs(nans) - 1) >> 3), key);
}

// Four codes of one word -> two fp16 pairs (bytes 0, 1 and 2, 3), exactly.
template <bool FP8>
__device__ __forceinline__ void codes4_to_h2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FP8) {
    lo = attn::e4m3x2_to_h2((uint16_t)w);
    hi = attn::e4m3x2_to_h2((uint16_t)(w >> 16));
  } else {
    const uint32_t u = w ^ 0x80808080u;
    lo = attn::s8x2_to_h2(u, 0x4140);
    hi = attn::s8x2_to_h2(u, 0x4342);
  }
}

// Power of two 2^e that brings a row's largest |x| = m into [2^14, 2^15) for fp16 (m zero, infinite
// or NaN: 1), and its inverse.  bf16 values times 2^e are exact in fp16 down to 2^-29 of the row's
// largest, and lose at most 2^-39 of it below that.
__device__ __forceinline__ float pow2_to_fp16(float m, float& inv) {
  const int E = (int)((__float_as_uint(m) >> 23) & 0xFFu);
  if (E == 0xFF || m == 0.0f) {
    inv = 1.0f;
    return 1.0f;
  }
  const int e = max(E, 16);  // exponent fields of both factors stay normal (2..240 and 14..252)
  inv = __uint_as_float((uint32_t)(e - 14) << 23);           // 2^(e - 127 - 14)
  return __uint_as_float((uint32_t)(254 - (e - 14)) << 23);  // 2^(127 + 14 - e)
}

}  // namespace paged

// The kernels' view of checked descriptors.
inline paged::Cache paged_cache_of(const fa_paged_cache& c) {
  paged::Cache o = {};
  o.k = static_cast<uint8_t*>(c.k_codes);
  o.v = static_cast<uint8_t*>(c.v_codes);
  o.ks = static_cast<float*>(c.k_scales);
  o.vs = static_cast<float*>(c.v_scales);
  const bool bnsd = c.layout == FA_LAYOUT_BNSD;
  o.page_stride = (long long)c.H * c.page_size * c.D;
  o.head_stride = bnsd ? c.page_size * c.D : c.D;
  o.tok_stride = bnsd ? c.D : c.H * c.D;
  o.pages = c.pages;
  o.H = c.H;
  while ((1 << o.page_shift) < c.page_size) ++o.page_shift;
  o.page_mask = c.page_size - 1;
  o.bnsd = bnsd;
  o.per_token = c.mode == FA_MODE_INT8_PER_TOKEN || c.mode == FA_MODE_FP8_PER_TOKEN;
  return o;
}
inline paged::Batch paged_batch_of(const fa_paged_batch& b, int T) {
  return {b.page_table, b.seq_lens, b.cu_q, b.B, b.max_pages, b.max_q > 0 ? b.max_q : T, T};
}

}  // namespace faq
