// paged_attn.cu -- attention of a ragged batch of new tokens over a paged quantized cache, for few
// query rows per kv head (single tokens, drafts): split-KV on register MMAs.
//
//   O_r = sum_j p_rj s_v(j) v_j / sum_j p_rj,   p_rj = 2^(x_rj - m_r),
//   x_rj = log2(e) softmax_scale s_k(j) q_r . k_j   over the keys j that row r sees.
//
// With few rows the cache's bytes bound it: every code is read once, and the arithmetic has to hide
// behind that.  The rows of one kv head -- new tokens times the group's query heads -- fill the 16 rows of an
// m16n8k16 fp16 MMA, so a code serves the whole group; int8 and E4M3 codes are exact in fp16, and Q's
// rows are scaled by powers of two into fp16's range (exact but for values 2^-29 below the row's
// largest).  Work is cut into units of 256 keys of one (sequence, kv head, row block), counted from the lengths
// on the device, and each of the grid's CTAs takes an equal run of consecutive units, whatever the
// lengths: a ragged batch balances, and a captured graph follows lengths that change.  A run that
// covers all of an item writes its output; items cut by a run's border leave (O, m, l) in the
// workspace, which the combine kernel merges.
//
// Each warp streams its own 32-key pieces (K and V codes and their scales) through a ring of shared
// memory stages with cp.async, so no barrier is needed inside an item; a warp keeps its own (m, l, O)
// and the eight are merged at the item's end.
#include <cuda_bf16.h>

#include "paged_sched.cuh"

namespace faq {
namespace {
using namespace paged;

constexpr int AW = 8;         // warps per CTA
constexpr int SK = 32;        // keys per warp piece
constexpr int UK = AW * SK;   // keys per unit
constexpr int NST = 3;        // ring stages per warp
constexpr float kPShift = 14.0f;  // probabilities are held as p 2^14: fp16 keeps 11 bits of them down to 2^-28
constexpr float kPInv = 1.0f / 16384.0f;

using PL = Plan<UK, 16, 1, 0x7FFFFFFF>;

template <int D>
struct AS {
  static constexpr uint32_t K = 0;                   // [32][D]
  static constexpr uint32_t V = SK * D;              // [32][D]
  static constexpr uint32_t SC = 2 * SK * D;         // [32] K scales, [32] V scales
  static constexpr uint32_t STAGE = SC + 2 * SK * 4;
  static constexpr uint32_t WARP = NST * STAGE;
  static constexpr uint32_t RING = AW * WARP;
  static constexpr uint32_t MERGE_O = 0;             // [AW][16][D] floats, over the ring
  static constexpr uint32_t MERGE_ML = RING;         // [AW][16] (m, l), own space
  static constexpr uint32_t TOTAL = MERGE_ML + AW * 16 * 8;
  static_assert(AW * 16 * D * 4 <= RING, "the merge fits the ring");
};

template <int D, bool FP8, bool TOK>
__global__ void __launch_bounds__(AW * 32, 1) paged_attn_kernel(const AttnP p) {
  using L = AS<D>;
  constexpr int CH = D / 16;  // 16-byte chunks per code row
  constexpr int KC = D / 64;  // chunks of a K row per lane of a quad
  constexpr int NV = D / 8;   // output column tiles
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * L::WARP;
  const uint32_t ring_u = smem_u32(ring);

  const long long total = total_units<PL>(p, lane);
  const int runs = run_count(total, gridDim.x);
  if ((int)blockIdx.x >= runs) return;
  const long long u0 = run_start(total, blockIdx.x, runs), u1 = run_start(total, blockIdx.x + 1, runs);
  long long u = u0;
  Item it = find_item<PL>(p, u, lane);

  while (u < u1) {
    const Seq s = it.s;
    const long long item_end = it.first + it.nt;
    const long long seg_end = item_end < u1 ? item_end : u1;
    const int key0 = (int)(u - it.first) * UK;
    const int key1 = min(s.n, (int)(seg_end - it.first) * UK);
    const int rows = s.m * p.G;

    // ---- Q fragments: rows g and g + 8 of the block, the dims that match the K chunks of this lane
    uint32_t qa[D / 16][4];
    float f_row[2];  // log2(e) softmax_scale 2^-e of the row (and s_k, per-head modes)
    int lim[2];      // last key the row sees
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = it.rb * 16 + g + 8 * x;
      const int i = r / p.G;
      const bool ok = r < rows;
      lim[x] = row_limit(p, s, r);
      const __nv_bfloat16* src = p.q + (long long)(s.q0 + i) * p.q_stride + (long long)(it.hk * p.G + r - i * p.G) * D;
      uint4 raw[KC][2];
      float m = 0.0f;
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          raw[c][y] = ok ? __ldg(reinterpret_cast<const uint4*>(src + 16 * (t + 4 * c)) + y) : make_uint4(0, 0, 0, 0);
          const uint32_t* w = &raw[c][y].x;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xFFFF0000u))));
        }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      float inv;
      const float sc = pow2_to_fp16(m, inv);
      f_row[x] = p.scale_log2 * inv * (TOK ? 1.0f : __ldg(p.c.ks + it.hk));
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // MMA step 4 c + k: dims 16 (t + 4 c) + 4 k .. + 3
          const uint32_t w0 = k < 2 ? (k == 0 ? raw[c][0].x : raw[c][0].z) : (k == 2 ? raw[c][1].x : raw[c][1].z);
          const uint32_t w1 = k < 2 ? (k == 0 ? raw[c][0].y : raw[c][0].w) : (k == 2 ? raw[c][1].y : raw[c][1].w);
          const __half2 h0 = __floats2half2_rn(__uint_as_float(w0 << 16) * sc, __uint_as_float(w0 & 0xFFFF0000u) * sc);
          const __half2 h1 = __floats2half2_rn(__uint_as_float(w1 << 16) * sc, __uint_as_float(w1 & 0xFFFF0000u) * sc);
          qa[4 * c + k][x] = *reinterpret_cast<const uint32_t*>(&h0);
          qa[4 * c + k][2 + x] = *reinterpret_cast<const uint32_t*>(&h1);
        }
    }
    const int lim_lo = p.causal ? s.n - s.m : s.n - 1;  // every row sees the keys up to here

    float o[NV][4];
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.0f, 0.0f};
    float r_run[2] = {0.0f, 0.0f};  // TOK: O holds sums of p s_v / r

    // ---- this warp's pieces: keys key0 + 32 (warp + 8 i)
    const int n_keys = key1 - key0;
    const int pieces = n_keys > warp * SK ? (n_keys - warp * SK + UK - 1) / UK : 0;
    auto load = [&](int i) {
      if (i < pieces) {
        const uint32_t st = ring_u + (i % NST) * L::STAGE;
        const int k0 = key0 + (warp + i * AW) * SK;
        // 2 lanes' worth of rows at a time: lane l loads chunk l % CH of rows l / CH + n (32 / CH)
#pragma unroll
        for (int n = 0; n < CH; ++n) {
          const int row = lane / CH + n * (32 / CH), c = lane % CH;
          const int j = k0 + row;
          int pg = -1;
          if (j < key1) pg = page_of(p.bt, p.c, it.b, j, p.status, 212);
          const bool ok = pg >= 0;
          const long long off = ok ? p.c.row(pg, it.hk, j & p.c.page_mask) + c * 16 : 0;
          // chunk swizzles: K rows are read by two neighbouring rows' quads at once, V rows by chunk
          const int ck = D == 128 ? c ^ ((row & 1) << 2) : c;
          const int cv = D == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3);
          cp_async16(st + L::K + row * D + ck * 16, p.c.k + off, ok);
          cp_async16(st + L::V + row * D + cv * 16, p.c.v + off, ok);
        }
        if (TOK) {
          const int j = k0 + lane;
          int pg = -1;
          if (j < key1) pg = page_of(p.bt, p.c, it.b, j, p.status, 212);
          const bool ok = pg >= 0;
          const long long si = ok ? p.c.scale(pg, it.hk, j & p.c.page_mask) : 0;
          cp_async4(st + L::SC + lane * 4, p.c.ks + si, ok);
          cp_async4(st + L::SC + (SK + lane) * 4, p.c.vs + si, ok);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) load(i);

    for (int i = 0; i < pieces; ++i) {
      __syncwarp();  // every lane is done with the stage that the next load overwrites
      load(i + NST - 1);
      cp_async_wait<NST - 1>();
      __syncwarp();
      const uint8_t* st = ring + (i % NST) * L::STAGE;
      const int k0 = key0 + (warp + i * AW) * SK;

      // ---- S = Q K^T: four tiles of 8 keys
      float sc[4][4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
        const int row = n * 8 + g;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          const int ck = D == 128 ? (t + 4 * c) ^ ((row & 1) << 2) : t;
          const uint4 kw = *reinterpret_cast<const uint4*>(st + L::K + row * D + ck * 16);
          const uint32_t w[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t b0, b1;
            codes4_to_h2<FP8>(w[k], b0, b1);
            mma16816(sc[n], qa[4 * c + k], b0, b1);
          }
        }
      }
      // ---- scales and masks: x = log2(e) softmax_scale s_k q . k
      const float* ksc = reinterpret_cast<const float*>(st + L::SC);
      const bool mask = k0 + SK - 1 > lim_lo || k0 + SK > key1;  // rows past the block's last are never written
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        float2 ks2 = make_float2(1.0f, 1.0f);
        if (TOK) ks2 = *reinterpret_cast<const float2*>(ksc + n * 8 + 2 * t);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = sc[n][e] * f_row[e >> 1];
          if (TOK) x *= (e & 1) ? ks2.y : ks2.x;
          if (mask) {
            const int j = k0 + n * 8 + 2 * t + (e & 1);
            if (j > lim[e >> 1] || j >= key1) x = -INFINITY;
          }
          sc[n][e] = x;
          mx[e >> 1] = fmaxf(mx[e >> 1], x);
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
        mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2));
      }
      // ---- p 2^14 against the running maximum, the row's sum, and the fp16 factors of V: p itself, or
      // in the per-token modes p s_v / r.  r is a power of two that follows the largest p s_v of the keys the row
      // sees (not the largest s_v, which a key of no weight, or one the row does not see, may have), so
      // that the factors keep fp16's 11 bits whatever the scales' range.
      float al[2], rinv[2] = {1.0f, 1.0f};
      bool moved = false;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float mn = fmaxf(m_run[x], mx[x]);
        al[x] = mn == m_run[x] ? 1.0f : attn::ex2(m_run[x] - mn);  // 0 from -inf
        moved = moved || mn != m_run[x];
        m_run[x] = mn;
        l_run[x] *= al[x];
      }
      float pv[4][4], wmax[2] = {0.0f, 0.0f};
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        float2 v2 = make_float2(1.0f, 1.0f);
        if (TOK) v2 = *reinterpret_cast<const float2*>(ksc + SK + n * 8 + 2 * t);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float m = m_run[e >> 1];
          const float x = sc[n][e];
          pv[n][e] = attn::ex2(x - (m == -INFINITY ? 0.0f : m) + kPShift);
          l_run[e >> 1] += pv[n][e];
          if (TOK) {
            pv[n][e] = x == -INFINITY ? 0.0f : pv[n][e] * ((e & 1) ? v2.y : v2.x);  // a masked key's scale may be anything
            wmax[e >> 1] = fmaxf(wmax[e >> 1], pv[n][e]);
          }
        }
      }
      if (TOK) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          wmax[x] = fmaxf(wmax[x], __shfl_xor_sync(0xffffffffu, wmax[x], 1));
          wmax[x] = fmaxf(wmax[x], __shfl_xor_sync(0xffffffffu, wmax[x], 2));
          // r: 2^14 r is above both the largest new factor and the largest one so far
          const float top = fmaxf(wmax[x], r_run[x] * al[x] * 8192.0f);
          const int E = max((int)(__float_as_uint(top) >> 23), 15);
          const float r = __uint_as_float((uint32_t)(E - 13) << 23);
          rinv[x] = __uint_as_float((uint32_t)(254 - (E - 13)) << 23);
          moved = moved || r != r_run[x];
          al[x] *= r_run[x] * rinv[x];
          r_run[x] = r;
        }
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][e] *= al[e >> 1];
      }
      uint32_t pa[2][4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const __half2 h0 = TOK ? __floats2half2_rn(pv[n][0] * rinv[0], pv[n][1] * rinv[0]) : __floats2half2_rn(pv[n][0], pv[n][1]);
        const __half2 h1 = TOK ? __floats2half2_rn(pv[n][2] * rinv[1], pv[n][3] * rinv[1]) : __floats2half2_rn(pv[n][2], pv[n][3]);
        pa[n >> 1][(n & 1) * 2] = *reinterpret_cast<const uint32_t*>(&h0);
        pa[n >> 1][(n & 1) * 2 + 1] = *reinterpret_cast<const uint32_t*>(&h1);
      }
      // ---- O += P V: output column tile n holds, at column g, dim (D / 8) g + n
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        uint32_t vw[4][NV / 4];  // the lane's dims (D / 8) g .. of keys 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int row = kk * 16 + 2 * t + (y & 1) + (y >> 1) * 8;
          if (D == 128) {
            const uint4 v4 = *reinterpret_cast<const uint4*>(st + L::V + row * D + ((g ^ (row & 7)) << 4));
            vw[y][0] = v4.x;
            vw[y][1] = v4.y;
            vw[y][2 % (NV / 4)] = v4.z;
            vw[y][3 % (NV / 4)] = v4.w;
          } else {
            const uint2 v2 = *reinterpret_cast<const uint2*>(st + L::V + row * D + (((g >> 1) ^ ((row >> 1) & 3)) << 4) +
                                                             (g & 1) * 8);
            vw[y][0] = v2.x;
            vw[y][1] = v2.y;
          }
        }
#pragma unroll
        for (int c = 0; c < NV / 4; ++c) {
          // interleave the key pairs' bytes: (a0 b0 a1 b1), (a2 b2 a3 b3)
          const uint32_t x0 = __byte_perm(vw[0][c], vw[1][c], 0x5140), x1 = __byte_perm(vw[0][c], vw[1][c], 0x7362);
          const uint32_t y0 = __byte_perm(vw[2][c], vw[3][c], 0x5140), y1 = __byte_perm(vw[2][c], vw[3][c], 0x7362);
          uint32_t b0[4], b1[4];
          codes4_to_h2<FP8>(x0, b0[0], b0[1]);
          codes4_to_h2<FP8>(x1, b0[2], b0[3]);
          codes4_to_h2<FP8>(y0, b1[0], b1[1]);
          codes4_to_h2<FP8>(y1, b1[2], b1[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) mma16816(o[4 * c + e], pa[kk], b0[e], b1[e]);
        }
      }
    }

    // ---- merge the warps: each row's sum over the quad, then (m, l) and O through shared memory
    cp_async_wait<0>();
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l_run[x] += __shfl_xor_sync(0xffffffffu, l_run[x], 1);
      l_run[x] += __shfl_xor_sync(0xffffffffu, l_run[x], 2);
    }
    float2* ml = reinterpret_cast<float2*>(smem + L::MERGE_ML);
    if (t == 0) {
      ml[warp * 16 + g] = make_float2(m_run[0], l_run[0]);
      ml[warp * 16 + g + 8] = make_float2(m_run[1], l_run[1]);
    }
    __syncthreads();  // every warp's ring is idle, and (m, l) are there
    float* mo = reinterpret_cast<float*>(smem + L::MERGE_O);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = g + 8 * x;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < AW; ++w) m = fmaxf(m, ml[w * 16 + r].x);
      const float al = m_run[x] == -INFINITY ? 0.0f : attn::ex2(m_run[x] - m) * (TOK ? r_run[x] : 1.0f);
      float* dst = mo + (warp * 16 + r) * D;
      // columns 2t and 2t + 1 of tile n are dims (D / 8) 2t + n and (D / 8)(2t + 1) + n
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int n = 0; n < NV; n += 4)
          *reinterpret_cast<float4*>(dst + NV * (2 * t + y) + n) =
              make_float4(al == 0.0f ? 0.0f : o[n][2 * x + y] * al, al == 0.0f ? 0.0f : o[n + 1][2 * x + y] * al,
                          al == 0.0f ? 0.0f : o[n + 2][2 * x + y] * al, al == 0.0f ? 0.0f : o[n + 3][2 * x + y] * al);
    }
    __syncthreads();
    const bool whole = u == it.first && seg_end == item_end;
    const int slot = 2 * blockIdx.x + (u == u0 ? 0 : 1);
    for (int idx = threadIdx.x; idx < 16 * D / 4; idx += AW * 32) {
      const int r = idx / (D / 4), c = idx % (D / 4);
      float m = -INFINITY, l = 0.0f;
#pragma unroll
      for (int w = 0; w < AW; ++w) m = fmaxf(m, ml[w * 16 + r].x);
      float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < AW; ++w) {
        const float2 v = ml[w * 16 + r];
        if (v.x > -INFINITY) l += v.y * attn::ex2(v.x - m);
        const float4 x = *reinterpret_cast<const float4*>(mo + (w * 16 + r) * D + c * 4);
        a.x += x.x;
        a.y += x.y;
        a.z += x.z;
        a.w += x.w;
      }
      l *= kPInv;
      a.x *= kPInv;
      a.y *= kPInv;
      a.z *= kPInv;
      a.w *= kPInv;
      if (whole) {
        const int rr = it.rb * 16 + r;
        if (rr < rows) {
          const int i = rr / p.G, hq = it.hk * p.G + rr - i * p.G;
          const float f = row_factor(p, it.hk, l, m, m);
          const long long row = (long long)(s.q0 + i) * p.Hq + hq;
          const __nv_bfloat162 v0 = __floats2bfloat162_rn(a.x * f, a.y * f), v1 = __floats2bfloat162_rn(a.z * f, a.w * f);
          *reinterpret_cast<uint2*>(p.out + row * D + c * 4) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&v0), *reinterpret_cast<const uint32_t*>(&v1));
          if (c == 0 && p.lse) p.lse[row] = row_lse(l, m);
        }
      } else {
        *reinterpret_cast<float4*>(p.part_o + ((long long)slot * 16 + r) * D + c * 4) = a;
        if (c == 0) p.part_ml[(long long)slot * 16 + r] = make_float4(m, l, m, 0.0f);
      }
    }
    __syncthreads();  // the ring is free again

    u = seg_end;
    if (u >= u1) break;
    if (!next_item<PL>(p, it)) return;  // cannot be while the lengths stay as they were counted
  }
}

template <int D, bool FP8, bool TOK>
cudaError_t launch_d(const AttnP& p, int grid, cudaStream_t s) {
  auto kern = paged_attn_kernel<D, FP8, TOK>;
  cudaError_t e;
  if ((e = set_smem_limit(reinterpret_cast<const void*>(kern), AS<D>::TOTAL)) != cudaSuccess) return e;
  kern<<<grid, AW * 32, AS<D>::TOTAL, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  combine_kernel<PL, D><<<grid, 128, 0, s>>>(p, grid);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_mode(const AttnP& p, int mode, int grid, cudaStream_t s) {
  switch (mode) {
    case FA_MODE_INT8_PER_HEAD: return launch_d<D, false, false>(p, grid, s);
    case FA_MODE_FP8_PER_HEAD: return launch_d<D, true, false>(p, grid, s);
    case FA_MODE_INT8_PER_TOKEN: return launch_d<D, false, true>(p, grid, s);
    case FA_MODE_FP8_PER_TOKEN: return launch_d<D, true, true>(p, grid, s);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace

// Query rows per kv head that a sequence of the batch can have.
static long long most_rows(const PagedAttnArgs& a) {
  const int max_q = a.batch->cu_q ? (a.batch->max_q > 0 ? min(a.batch->max_q, a.q->T) : a.q->T) : 1;
  return (long long)max_q * (a.q->H / a.cache->H);
}

size_t paged_attention_ws(const PagedAttnArgs& a) {
  const int D = a.q->D;
  if (D == 128 && most_rows(a) <= 16) return paged_decode_ws();
  return paged_chunk_ws(D);
}

cudaError_t launch_paged_attention(const PagedAttnArgs& a, void* ws, cudaStream_t s) {
  const int D = a.q->D;
  const long long rows = most_rows(a);
  if (D == 128) {
    // sequences of up to 16 query rows per kv head, then those of more
    const cudaError_t e = launch_paged_decode(a, rows < 16 ? (int)rows : 16, ws, s);
    if (e != cudaSuccess || rows <= 16) return e;
  }
  return launch_paged_chunk(a, ws, s);
}

}  // namespace faq
