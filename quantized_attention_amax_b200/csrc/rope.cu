// rope.cu -- rotary positions, and the append of new tokens into a paged quantized cache.
//
// A pair (a, b) of a head at position p turns by the angle p f: a' = a cos - b sin, b' = b cos + a sin.
// Products and sums are rounded to fp32 one by one (no fused multiply-add), so that the bf16 results
// and the codes made from them are the same wherever the formula is evaluated in fp32.
//
// rope_append_kernel is bound by its rows' bytes: per token (2 Hq + 2 Hkv) D bf16 values and 2 Hkv D
// codes pass once.  A warp takes one token and a run of its heads, so the token's sequence, position
// and angles are found once (its first rows are on their way meanwhile); each lane holds 8 elements (16 bytes)
// of a row, D / 8 lanes a row, and the (i, i + rotary_dim / 2) pairs meet by shuffles.
// Measured: 32768 tokens of 32 query and 8 kv heads of 128 (int8 per token, 757 MB) in 165 us, 4.6 TB/s, 70 % of
// the copy bandwidth (what is left: 74 % of the issue slots are taken by unpacking, rotating and quantizing, and more rows
// in flight cost more in registers than they bring); 16 tokens in 6.5 us, a launch and four dependent loads.
#include <cuda_bf16.h>

#include "paged_common.cuh"
#include "quant_common.cuh"

namespace faq {
namespace {
using namespace paged;

// Rows a lane holds at once, and as many on their way (2 / 4 / 8 measured 66 / 70 / 107 us for 5000 tokens of 40 heads)
constexpr int kRows = 2;

struct InvFreq {
  double f[64];
};

// One thread per (position, pair): the angle, its sine and cosine in 64 bits (positions reach 2^20
// and more, where a 32-bit angle would be off by whole radians), one rounding each.
__global__ void __launch_bounds__(256) rope_table_kernel(float* __restrict__ table, long long n, int half, InvFreq inv,
                                                         double factor) {
  const long long stride = (long long)gridDim.x * blockDim.x;
  for (long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x; idx < n; idx += stride) {
    const long long p = idx / half;
    const int i = (int)(idx - p * half);
    double sn, cs;
    sincos((double)p * inv.f[i], &sn, &cs);
    if (!in_bounds(p * 2 * half + half + i < 2 * n, 167)) continue;
    table[p * 2 * half + i] = (float)(factor * cs);
    table[p * 2 * half + half + i] = (float)(factor * sn);
  }
}

struct Rows {
  const __nv_bfloat16* p;
  long long stride;
  int H;
};

struct AppendArgs {
  Rows q, k, v;
  __nv_bfloat16* qo;
  long long qo_stride;
  Cache c;
  Batch bt;
  const float* cs;
  int table_positions, rd;
  const int* positions;
  const float* amax_k;
  const float* amax_v;
  int parts;     // warps per token
  int per_part;  // head rows per warp
  int* status;
};

// The (first) sequence whose rows hold row t; bt.B if none does.
__device__ __forceinline__ int seq_of_row(const Batch& bt, int t, int lane) {
  if (!bt.cu) return t < bt.B ? t : bt.B;
  for (int b0 = 0; b0 < bt.B; b0 += 32) {
    const int b = b0 + lane;
    const unsigned in = __ballot_sync(0xffffffffu, b < bt.B && __ldg(bt.cu + b) <= t && t < __ldg(bt.cu + b + 1));
    if (in) return b0 + __ffs(in) - 1;
  }
  return bt.B;
}

// a' = a cos - b sin, b' = b cos + a sin
__device__ __forceinline__ float turn_a(float a, float b, float c, float s) {
  return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float turn_b(float a, float b, float c, float s) {
  return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

template <int MODE, int D, bool INTER>
__global__ void __launch_bounds__(256) rope_append_kernel(const AppendArgs a) {
  constexpr int LPR = D / 8;     // lanes per row
  constexpr int RPW = 32 / LPR;  // rows a warp holds at once
  constexpr bool PER_HEAD = MODE == FA_MODE_INT8_PER_HEAD || MODE == FA_MODE_FP8_PER_HEAD;
  constexpr bool INT8 = MODE == FA_MODE_INT8_PER_HEAD || MODE == FA_MODE_INT8_PER_TOKEN;
  constexpr float QMAX = INT8 ? 127.0f : 448.0f;
  const int lane = threadIdx.x & 31;
  const int gl = lane % LPR, sub = lane / LPR;
  const long long w = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (blockIdx.x == 0)  // every sequence's check, of those too that no row leads to
    for (int b = threadIdx.x; b < a.bt.B; b += blockDim.x) load_seq(a.bt, a.c.page_shift, b, a.status, 201);
  if (PER_HEAD && blockIdx.x == 0)
    for (int h = threadIdx.x; h < a.c.H; h += blockDim.x) {
      a.c.ks[h] = __fdiv_rn(__ldg(a.amax_k + h), QMAX);
      a.c.vs[h] = __fdiv_rn(__ldg(a.amax_v + h), QMAX);
    }
  const int t = (int)(w / a.parts), part = (int)(w % a.parts);
  if (t >= a.bt.T) return;
  const int Hq = a.q.H, total = Hq + 2 * a.c.H;
  const int r_end = min(total, (part + 1) * a.per_part);
  // U rows at a time, the next ones on their way; the first are asked for before anything is known of the token
  constexpr int U = kRows;
  uint4 ahead[U];
  auto load = [&](int r0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPW;
      const Rows& x = r < Hq ? a.q : r < Hq + a.c.H ? a.k : a.v;
      const int h = r < Hq ? r : r < Hq + a.c.H ? r - Hq : r - Hq - a.c.H;
      const bool ok = r < r_end && in_bounds(t < a.bt.T && h >= 0 && h < x.H, 163);
      ahead[u] = ok ? *(reinterpret_cast<const uint4*>(x.p + (long long)t * x.stride + (long long)h * D) + gl)
                           : make_uint4(0, 0, 0, 0);
    }
  };
  load(part * a.per_part + sub);
  const int b = seq_of_row(a.bt, t, lane);
  if (b >= a.bt.B) return;  // a padded row
  const Seq s = load_seq(a.bt, a.c.page_shift, b, a.status, 201);
  const int j = s.n - s.m + (t - s.q0);  // cache index
  if (s.m == 0 || t < s.q0 || t >= s.q0 + s.m || j < 0) {
    if (s.m > 0) bad(a.status, 202);  // more new tokens than cached ones, or cu_q that does not ascend
    return;
  }
  // this lane's angles: elements 8 gl .. 8 gl + 7 of a row
  const bool rot = gl * 8 < a.rd;
  float cs[8], sn[8];
  if (a.rd > 0) {
    const int p = a.positions ? __ldg(a.positions + t) : j;
    if ((unsigned)p >= (unsigned)a.table_positions) {
      if (lane == 0) bad(a.status, 203);
      return;
    }
    if (rot) {
      const float* row = a.cs + (long long)p * a.rd;
      // pair indices of the lane: interleaved 4 gl .. 4 gl + 3, else 8 (gl mod half) .. + 7
      const int half8 = a.rd / 16;
      const int i0 = INTER ? gl * 4 : (gl < half8 ? gl : gl - half8) * 8;
#pragma unroll
      for (int q = 0; q < (INTER ? 1 : 2); ++q) {
        *reinterpret_cast<float4*>(&cs[4 * q]) = __ldg(reinterpret_cast<const float4*>(row + i0) + q);
        *reinterpret_cast<float4*>(&sn[4 * q]) = __ldg(reinterpret_cast<const float4*>(row + a.rd / 2 + i0) + q);
      }
    }
  }
  const int pg = page_of(a.bt, a.c, b, j, a.status, 204);
  const int slot = j & a.c.page_mask;
  // lane that holds the other half of this lane's pairs (half layout)
  const int other = INTER ? lane : sub * LPR + (rot ? (gl < a.rd / 16 ? gl + a.rd / 16 : gl - a.rd / 16) : gl);
  const bool first = gl < a.rd / 16;

  for (int r0 = part * a.per_part + sub; r0 - sub < r_end; r0 += U * RPW) {
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = ahead[u];
    load(r0 + U * RPW);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPW;
      const bool live = r < r_end;
      const bool is_q = r < Hq, is_v = r >= Hq + a.c.H;
      float x[8];
      unpack_bf16x8(raw[u], x);
      if (a.rd > 0) {
        float y[8];
        if (!INTER) {
          const uint4 o = make_uint4(__shfl_sync(0xffffffffu, raw[u].x, other), __shfl_sync(0xffffffffu, raw[u].y, other),
                                     __shfl_sync(0xffffffffu, raw[u].z, other), __shfl_sync(0xffffffffu, raw[u].w, other));
          unpack_bf16x8(o, y);
        }
        if (rot && !is_v) {
          if (INTER) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float p = x[2 * i], q = x[2 * i + 1];
              x[2 * i] = turn_a(p, q, cs[i], sn[i]);
              x[2 * i + 1] = turn_b(p, q, cs[i], sn[i]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = first ? turn_a(x[i], y[i], cs[i], sn[i]) : turn_b(y[i], x[i], cs[i], sn[i]);
          }
          uint32_t* rw = &raw[u].x;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 v2 = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            rw[i] = *reinterpret_cast<const uint32_t*>(&v2);
          }
        }
      }
      if (live && is_q && in_bounds(t < a.bt.T && r * D + 8 * gl + 8 <= a.qo_stride, 164))
        *(reinterpret_cast<uint4*>(a.qo + (long long)t * a.qo_stride + (long long)r * D) + gl) = raw[u];
      if (r - sub + RPW <= Hq) continue;  // no K or V row in this warp's rows: the same for every lane
      // ---- quantize the K or V row
      const int h = is_v ? r - Hq - a.c.H : r - Hq;
      const bool kv = live && !is_q;
      float sc = 0.0f;
      if (PER_HEAD) {
        sc = kv ? __fdiv_rn(__ldg((is_v ? a.amax_v : a.amax_k) + h), QMAX) : 0.0f;
      } else {
        uint32_t m2 = bf16x2_absmax_nan(bf16x2_absmax_nan(raw[u].x, raw[u].y), bf16x2_absmax_nan(raw[u].z, raw[u].w));
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1) m2 = bf16x2_absmax_nan(m2, __shfl_xor_sync(0xffffffffu, m2, off));
        m2 &= 0x7FFF7FFFu;
        const float lo = __uint_as_float(m2 << 16), hi = __uint_as_float(m2 & 0xFFFF0000u);
        sc = __fdiv_rn(lo != lo ? lo : hi != hi ? hi : fmaxf(lo, hi), QMAX);
      }
      if (!kv || pg < 0 || !a.c.holds(a.c.row(pg, h, slot) + 8 * gl, 8, 165)) continue;
      unpack_bf16x8(raw[u], x);
      // x / s as IEEE division rounds it where that decides the code (quant_common.cuh)
      if (sc >= kFastDivMin && sc < INFINITY) {
        const float rc = __frcp_rn(sc);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          x[i] = INT8 ? int8_div(x[i], sc, rc) : PER_HEAD ? fp8_div_sat(x[i], sc, rc) : fp8_div(x[i], sc, rc);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = sc > 0.0f ? __fdiv_rn(x[i], sc) : 0.0f;
      }
      const uint2 o = INT8 ? make_uint2(s8x4<true>(x[0], x[1], x[2], x[3]), s8x4<true>(x[4], x[5], x[6], x[7]))
                           : make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
      *(reinterpret_cast<uint2*>((is_v ? a.c.v : a.c.k) + a.c.row(pg, h, slot)) + gl) = o;
      if (!PER_HEAD && gl == 0 && a.c.holds_scale(a.c.scale(pg, h, slot), 166)) (is_v ? a.c.vs : a.c.ks)[a.c.scale(pg, h, slot)] = sc;
    }
  }
}

template <int MODE, int D>
cudaError_t launch_append_d(const AppendArgs& a, bool inter, long long warps, cudaStream_t s) {
  const long long grid = (warps + 7) / 8;
  if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  if (inter)
    rope_append_kernel<MODE, D, true><<<(unsigned)grid, 256, 0, s>>>(a);
  else
    rope_append_kernel<MODE, D, false><<<(unsigned)grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

template <int MODE>
cudaError_t launch_append_mode(const AppendArgs& a, int D, bool inter, long long warps, cudaStream_t s) {
  return D == 128 ? launch_append_d<MODE, 128>(a, inter, warps, s) : launch_append_d<MODE, 64>(a, inter, warps, s);
}

}  // namespace

cudaError_t launch_rope_table(float* table, int positions, int rotary_dim, const double* inv_freq, double factor,
                              cudaStream_t s) {
  InvFreq f = {};
  for (int i = 0; i < rotary_dim / 2; ++i) f.f[i] = inv_freq[i];
  const long long n = (long long)positions * (rotary_dim / 2);
  if (n == 0) return cudaSuccess;
  if (const cudaError_t be = bounds_attach(); be != cudaSuccess) return be;
  const long long want = (n + 255) / 256, cap = 16LL * sm_count();
  rope_table_kernel<<<(unsigned)(want < cap ? want : cap), 256, 0, s>>>(table, n, rotary_dim / 2, f, factor);
  return cudaGetLastError();
}

cudaError_t launch_rope_append(const RopeAppendArgs& r, cudaStream_t s) {
  if (const cudaError_t be = bounds_attach(); be != cudaSuccess) return be;
  AppendArgs a = {};
  if (r.q) a.q = {static_cast<const __nv_bfloat16*>(r.q->data), r.q->stride, r.q->H};
  a.k = {static_cast<const __nv_bfloat16*>(r.k->data), r.k->stride, r.k->H};
  a.v = {static_cast<const __nv_bfloat16*>(r.v->data), r.v->stride, r.v->H};
  if (r.q_out) {
    a.qo = static_cast<__nv_bfloat16*>(r.q_out->data);
    a.qo_stride = r.q_out->stride;
  }
  a.c = paged_cache_of(*r.cache);
  a.bt = paged_batch_of(*r.batch, r.k->T);
  a.cs = r.cos_sin;
  a.table_positions = r.table_positions;
  a.rd = r.rotary_dim;
  a.positions = r.positions;
  a.amax_k = r.amax_k;
  a.amax_v = r.amax_v;
  a.status = r.status;
  const int total = a.q.H + 2 * a.c.H;
  // one warp per token once the tokens alone fill the GPU's warps (64 per SM); fewer tokens split
  // their heads over warps, down to two rounds of loads each
  const int per_round = 2 * kRows * (32 / (r.cache->D / 8));
  const int most = (total + per_round - 1) / per_round;
  const long long fill = (64LL * sm_count() + r.k->T - 1) / r.k->T;
  a.parts = (int)(fill < 1 ? 1 : fill > most ? most : fill);
  a.per_part = ((total + a.parts - 1) / a.parts + per_round - 1) / per_round * per_round;
  a.parts = (total + a.per_part - 1) / a.per_part;
  const long long warps = (long long)r.k->T * a.parts;
  const bool inter = r.interleaved != 0;
  switch (r.cache->mode) {
    case FA_MODE_INT8_PER_HEAD: return launch_append_mode<FA_MODE_INT8_PER_HEAD>(a, r.cache->D, inter, warps, s);
    case FA_MODE_FP8_PER_HEAD: return launch_append_mode<FA_MODE_FP8_PER_HEAD>(a, r.cache->D, inter, warps, s);
    case FA_MODE_INT8_PER_TOKEN: return launch_append_mode<FA_MODE_INT8_PER_TOKEN>(a, r.cache->D, inter, warps, s);
    case FA_MODE_FP8_PER_TOKEN: return launch_append_mode<FA_MODE_FP8_PER_TOKEN>(a, r.cache->D, inter, warps, s);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace faq
