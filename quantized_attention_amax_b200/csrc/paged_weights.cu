// paged_weights.cu -- the attention weight that new tokens give each cached token (column sums of the
// softmax matrix):  w_j = sum over the rows r of a kv head that see j of 2^(x_rj - log2(e) lse_r),
// x_rj = log2(e) softmax_scale s_k(j) q_r . k_j.
//
// With one new token per sequence the K codes' bytes bound it; with a window of tokens the products and
// exponentials do.  The keys are the MMA's 16 rows (they stay in registers, as fp16) and the query rows its
// columns, 8 at a time, from shared memory: a key's weight is then summed along the columns a thread
// holds and over its quad, in a fixed order, and no two threads write one key.  A warp takes 16 keys,
// a unit is 128 keys of one (sequence, kv head), and the CTAs take equal runs of units counted from the lengths
// on the device.
#include <cuda_bf16.h>

#include "paged_common.cuh"

namespace faq {
namespace {
using namespace paged;

constexpr int WW = 8;        // warps per CTA
constexpr int WUK = WW * 16; // keys per unit
constexpr int WR = 64;       // query rows in shared memory at a time

struct WeightP {
  const __nv_bfloat16* q;
  long long q_stride;
  Cache c;
  Batch bt;
  int Hq, G, causal, accumulate;
  float scale_log2;
  const float* lse;
  float* acc;
  long long acc_stride;
  int* status;
};

// A row's constants: x - lse2 is sum * f * s_k - hi - lo; lim: the last key it sees (-1: none).
struct __align__(16) RowC {
  float f, hi, lo;
  int lim;
};

template <int D>
struct WS {
  static constexpr uint32_t QROW = 2 * D + 16;  // bytes per fp16 row; the pad spreads rows over the banks
  static constexpr uint32_t ROWC = WR * QROW;
  static constexpr uint32_t TOTAL = ROWC + WR * 16;
};

__device__ __forceinline__ int weight_units(const WeightP& p, int b, Seq& s) {
  s = load_seq(p.bt, p.c.page_shift, b, p.status, 221);
  if (s.n > p.acc_stride) {
    bad(p.status, 222);
    s = {0, 0, 0};
  }
  return s.m > 0 || !p.accumulate ? (s.n + WUK - 1) / WUK : 0;
}

template <int D, bool FP8, bool TOK>
__global__ void __launch_bounds__(WW * 32) paged_weights_kernel(const WeightP p) {
  using L = WS<D>;
  constexpr int KC = D / 64;
  __shared__ __align__(16) uint8_t smem[L::TOTAL];
  RowC* rowc = reinterpret_cast<RowC*>(smem + L::ROWC);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;

  long long total = 0;
  for (int b = lane; b < p.bt.B; b += 32) {
    Seq s;
    total += weight_units(p, b, s);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  total *= p.c.H;
  const long long u0 = total * blockIdx.x / gridDim.x, u1 = total * (blockIdx.x + 1) / gridDim.x;
  if (u0 >= u1) return;
  // the sequence of unit u0
  int b = -1;
  Seq s = {0, 0, 0};
  int nt = 0;
  long long first = 0;
  {
    long long base = 0;
    for (int b0 = 0; b0 < p.bt.B && b < 0; b0 += 32) {
      Seq x = {0, 0, 0};
      const int n = b0 + lane < p.bt.B ? weight_units(p, b0 + lane, x) : 0;
      const long long mine = (long long)n * p.c.H;
      long long end = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, end, off);
        if (lane >= off) end += o;
      }
      const unsigned after = __ballot_sync(0xffffffffu, base + end > u0);
      if (after) {
        const int src = __ffs(after) - 1;
        b = b0 + src;
        s.q0 = __shfl_sync(0xffffffffu, x.q0, src);
        s.m = __shfl_sync(0xffffffffu, x.m, src);
        s.n = __shfl_sync(0xffffffffu, x.n, src);
        nt = __shfl_sync(0xffffffffu, n, src);
        first = base + __shfl_sync(0xffffffffu, end - mine, src);
      }
      base += __shfl_sync(0xffffffffu, end, 31);
    }
  }
  int hk = (int)((u0 - first) / nt), tile = (int)((u0 - first) % nt);
  int held = -1;  // the (row block of the) item whose Q rows are in shared memory

  for (long long u = u0; u < u1; ++u) {
    const int rows = s.m * p.G;
    const int nblk = (rows + WR - 1) / WR;
    // ---- this warp's 16 keys: rows g and g + 8 of the A fragments
    const int k0 = tile * WUK + warp * 16;
    uint32_t ka[D / 16][4];
    float ksc[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int j = k0 + g + 8 * x;
      const int pg = j < s.n ? page_of(p.bt, p.c, b, j, p.status, 223) : -1;
      const uint8_t* src = p.c.k + (pg >= 0 ? p.c.row(pg, hk, j & p.c.page_mask) : 0);
      ksc[x] = TOK ? (pg >= 0 ? __ldg(p.c.ks + p.c.scale(pg, hk, j & p.c.page_mask)) : 0.0f) : __ldg(p.c.ks + hk);
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const uint4 kw = pg >= 0 ? __ldg(reinterpret_cast<const uint4*>(src) + t + 4 * c) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) codes4_to_h2<FP8>(w[k], ka[4 * c + k][x], ka[4 * c + k][2 + x]);
      }
    }
    float sum[2] = {0.0f, 0.0f};
    for (int blk = 0; blk < nblk; ++blk) {
      // ---- Q rows of the block as fp16, and their constants
      if (held != blk || nblk > 1) {
        __syncthreads();
        for (int r = warp; r < (min(rows - blk * WR, WR) + 7) / 8 * 8; r += WW) {
          const int rr = blk * WR + r;
          const int i = rr / p.G;
          const bool ok = rr < rows;
          const long long row = (long long)(s.q0 + i);
          const int hq = hk * p.G + rr - i * p.G;
          uint32_t w[D / 64];  // D / 32 elements per lane
          const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + row * p.q_stride + (long long)hq * D);
          float m = 0.0f;
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            w[c] = ok ? __ldg(src + lane * (D / 64) + c) : 0u;
            m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[c] << 16)), fabsf(__uint_as_float(w[c] & 0xFFFF0000u))));
          }
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
          float inv;
          const float sc = pow2_to_fp16(m, inv);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const __half2 h = __floats2half2_rn(__uint_as_float(w[c] << 16) * sc, __uint_as_float(w[c] & 0xFFFF0000u) * sc);
            *reinterpret_cast<__half2*>(smem + r * L::QROW + (lane * (D / 64) + c) * 4) = h;
          }
          if (lane == 0) {
            const float lse = ok ? __ldg(p.lse + row * p.Hq + hq) : -INFINITY;
            RowC rc;
            rc.f = p.scale_log2 * inv;
            rc.lim = !ok || lse == -INFINITY ? -1 : p.causal ? min(s.n - 1, s.n - s.m + i) : s.n - 1;
            // log2(e) lse in two terms: log2(e) = 1.4427... as fp32 plus its remainder
            rc.hi = rc.lim < 0 ? 0.0f : lse * 1.44269502f;
            rc.lo = rc.lim < 0 ? 0.0f : fmaf(lse, 1.44269502f, -rc.hi) + lse * 1.92596303e-8f;
            rowc[r] = rc;
          }
        }
        __syncthreads();
        held = blk;
      }
      const int nn = (min(rows - blk * WR, WR) + 7) / 8;
      for (int n = 0; n < nn; ++n) {
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        const uint8_t* qrow = smem + (n * 8 + g) * L::QROW;
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
          for (int y = 0; y < 2; ++y) {  // MMA steps 4 c + 2 y and + 1: dims 16 (t + 4 c) + 8 y .. + 7
            const uint4 qv = *reinterpret_cast<const uint4*>(qrow + (t + 4 * c) * 32 + y * 16);
            mma16816(d, ka[4 * c + 2 * y], qv.x, qv.y);
            mma16816(d, ka[4 * c + 2 * y + 1], qv.z, qv.w);
          }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const RowC rc = rowc[n * 8 + 2 * t + e];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int j = k0 + g + 8 * x;
            const float v = attn::ex2(fmaf(d[2 * x + e] * ksc[x], rc.f, -rc.hi) - rc.lo);
            sum[x] += j <= rc.lim ? v : 0.0f;
          }
        }
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 1);
      sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 2);
    }
    if (t < 2) {
      const int j = k0 + g + 8 * t;
      if (j < s.n) {
        float* dst = p.acc + ((long long)b * p.c.H + hk) * p.acc_stride + j;
        const float w = t ? sum[1] : sum[0];
        *dst = p.accumulate ? *dst + w : w;
      }
    }
    // ---- the next unit
    if (++tile == nt) {
      tile = 0;
      held = -1;
      if (++hk == p.c.H) {
        hk = 0;
        if (u + 1 < u1) {
          do {
            if (++b >= p.bt.B) return;  // cannot be while the lengths stay as they were counted
            nt = weight_units(p, b, s);
          } while (nt == 0);
        }
      }
    }
  }
}

template <int D, bool FP8, bool TOK>
cudaError_t launch_d(const WeightP& p, cudaStream_t s) {
  paged_weights_kernel<D, FP8, TOK><<<2 * sm_count(), WW * 32, 0, s>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_mode(const WeightP& p, int mode, cudaStream_t s) {
  switch (mode) {
    case FA_MODE_INT8_PER_HEAD: return launch_d<D, false, false>(p, s);
    case FA_MODE_FP8_PER_HEAD: return launch_d<D, true, false>(p, s);
    case FA_MODE_INT8_PER_TOKEN: return launch_d<D, false, true>(p, s);
    case FA_MODE_FP8_PER_TOKEN: return launch_d<D, true, true>(p, s);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace

cudaError_t launch_paged_weights(const PagedAttnArgs& a, cudaStream_t s) {
  WeightP p = {};
  p.q = static_cast<const __nv_bfloat16*>(a.q->data);
  p.q_stride = a.q->stride;
  p.c = paged_cache_of(*a.cache);
  p.bt = paged_batch_of(*a.batch, a.q->T);
  p.Hq = a.q->H;
  p.G = a.q->H / a.cache->H;
  p.causal = a.causal;
  p.accumulate = a.accumulate;
  p.scale_log2 = (a.softmax_scale > 0.0f ? a.softmax_scale : 1.0f / sqrtf((float)a.q->D)) * 1.4426950408889634f;
  p.lse = a.lse;
  p.acc = a.acc;
  p.acc_stride = a.acc_stride;
  p.status = a.status;
  return a.q->D == 128 ? launch_mode<128>(p, a.cache->mode, s) : launch_mode<64>(p, a.cache->mode, s);
}

}  // namespace faq
