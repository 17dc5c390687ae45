// paged_sched.cuh -- how the paged attention kernels share out a ragged batch.
//
// The work of one call is a row of units: sequence by sequence, kv head by kv head, row block by row
// block (RB query rows: new tokens x the group's heads), UK keys to a unit.  The units are counted on the device
// from the batch's lengths, and CTA c of `runs` takes the c-th of as many equal runs of consecutive units,
// so a ragged batch balances whatever its lengths, and a captured graph follows lengths that change.  An
// item -- one row block's units -- that a run covers wholly is written out by that CTA; the pieces of items that a
// run's border cuts are left as partial results (O, m, l), at most two a run: the one at the run's
// start in slot 0, any later one in slot 1.
#pragma once

#include "paged_common.cuh"

namespace faq {
namespace paged {

struct AttnP {
  const __nv_bfloat16* q;
  long long q_stride;
  Cache c;
  Batch bt;
  int Hq, G, causal;
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  float* part_o;    // [2 runs][rows of a block][D]: sums of p s_v v in units of 2^mv
  float4* part_ml;  // [2 runs][rows of a block]: m, l (sum of p in units of 2^m), mv
  int* status;
};

// Sequences whose row count lies in [MINR, MAXR] are this kernel's.  TRIM: causal row blocks count only the
// units they see (worth it where blocks are many; their sums have no closed form).
template <int UK_, int RB_, int MINR_, int MAXR_, bool TRIM_ = false>
struct Plan {
  static constexpr int UK = UK_, RB = RB_, MINR = MINR_, MAXR = MAXR_;
  static constexpr bool TRIM = TRIM_;
};

struct Item {
  int b, hk, rb;    // sequence, kv head, row block
  Seq s;
  int nrb, nt;      // the sequence's row blocks, units of this one
  long long first;  // first unit of the item
};

// Sequence b and its row blocks (none if it is not this plan's).
template <typename PL>
__device__ __forceinline__ void seq_blocks(const AttnP& p, int b, Seq& s, int& nrb) {
  s = load_seq(p.bt, p.c.page_shift, b, p.status, 211);
  const long long rows = (long long)s.m * p.G;
  nrb = rows >= PL::MINR && rows <= PL::MAXR ? (int)((rows + PL::RB - 1) / PL::RB) : 0;
}

// Units of row block rb: at least one, since rows that see no key are written too.
template <typename PL>
__device__ __forceinline__ int block_units(const AttnP& p, const Seq& s, int rb) {
  int end = s.n;
  if (PL::TRIM && p.causal) {
    const int last = min((rb + 1) * PL::RB, s.m * p.G) - 1;
    end = min(s.n, s.n - s.m + last / p.G + 1);
  }
  return max(1, (end + PL::UK - 1) / PL::UK);
}

// Units of one kv head of each lane's sequence (a warp's work).
template <typename PL>
__device__ __forceinline__ long long head_units(const AttnP& p, const Seq& s, int nrb, int lane) {
  if (!PL::TRIM || !p.causal) return nrb ? (long long)nrb * block_units<PL>(p, s, 0) : 0;
  long long w = 0;
  if (nrb <= 4)
    for (int k = 0; k < nrb; ++k) w += block_units<PL>(p, s, k);
  for (unsigned big = __ballot_sync(0xffffffffu, nrb > 4); big; big &= big - 1) {
    const int src = __ffs(big) - 1;
    const Seq o = {0, __shfl_sync(0xffffffffu, s.m, src), __shfl_sync(0xffffffffu, s.n, src)};
    const int no = __shfl_sync(0xffffffffu, nrb, src);
    long long v = 0;
    for (int k = lane; k < no; k += 32) v += block_units<PL>(p, o, k);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (lane == src) w = v;
  }
  return w;
}

// All units of the batch (every lane of the warp gets the sum).
template <typename PL>
__device__ __forceinline__ long long total_units(const AttnP& p, int lane) {
  long long w = 0;
  for (int b0 = 0; b0 < p.bt.B; b0 += 32) {
    Seq s = {0, 0, 0};
    int nrb = 0;
    if (b0 + lane < p.bt.B) seq_blocks<PL>(p, b0 + lane, s, nrb);
    w += head_units<PL>(p, s, nrb, lane);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) w += __shfl_xor_sync(0xffffffffu, w, off);
  return w * p.c.H;
}

__device__ __forceinline__ long long lanes_before(long long v, int lane) {  // sum over the lanes up to this one
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += o;
  }
  return v;
}

// The item that holds unit u < total (a warp's work).
template <typename PL>
__device__ __forceinline__ Item find_item(const AttnP& p, long long u, int lane) {
  long long base = 0;
  Item it = {};
  for (int b0 = 0; b0 < p.bt.B; b0 += 32) {
    Seq s = {0, 0, 0};
    int nrb = 0;
    if (b0 + lane < p.bt.B) seq_blocks<PL>(p, b0 + lane, s, nrb);
    const long long head = head_units<PL>(p, s, nrb, lane), mine = head * p.c.H;
    const long long end = base + lanes_before(mine, lane);
    const unsigned after = __ballot_sync(0xffffffffu, end > u);
    if (!after) {
      base = __shfl_sync(0xffffffffu, end, 31);
      continue;
    }
    const int src = __ffs(after) - 1;
    it.b = b0 + src;
    it.s.q0 = __shfl_sync(0xffffffffu, s.q0, src);
    it.s.m = __shfl_sync(0xffffffffu, s.m, src);
    it.s.n = __shfl_sync(0xffffffffu, s.n, src);
    it.nrb = __shfl_sync(0xffffffffu, nrb, src);
    const long long start = __shfl_sync(0xffffffffu, end - mine, src), per = __shfl_sync(0xffffffffu, head, src);
    it.hk = (int)((u - start) / per);
    it.first = start + it.hk * per;
    if (!PL::TRIM || !p.causal) {
      it.nt = block_units<PL>(p, it.s, 0);
      it.rb = (int)((u - it.first) / it.nt);
      it.first += (long long)it.rb * it.nt;
      return it;
    }
    for (int k0 = 0; k0 < it.nrb; k0 += 32) {
      const int n = k0 + lane < it.nrb ? block_units<PL>(p, it.s, k0 + lane) : 0;
      const long long e = it.first + lanes_before(n, lane);
      const unsigned in = __ballot_sync(0xffffffffu, e > u);
      if (in) {
        const int k = __ffs(in) - 1;
        it.rb = k0 + k;
        it.nt = __shfl_sync(0xffffffffu, n, k);
        it.first = __shfl_sync(0xffffffffu, e, k) - it.nt;
        return it;
      }
      it.first = __shfl_sync(0xffffffffu, e, 31);
    }
  }
  it.b = p.bt.B;
  return it;
}

// The item after `it`: next row block, kv head, or sequence with units.  False past the last.
template <typename PL>
__device__ __forceinline__ bool next_item(const AttnP& p, Item& it) {
  it.first += it.nt;
  if (++it.rb == it.nrb) {
    it.rb = 0;
    if (++it.hk == p.c.H) {
      it.hk = 0;
      do {
        if (++it.b >= p.bt.B) return false;
        seq_blocks<PL>(p, it.b, it.s, it.nrb);
      } while (it.nrb == 0);
    }
  }
  it.nt = block_units<PL>(p, it.s, it.rb);
  return true;
}

// Run c of `runs` equal ones; a grid larger than the units leaves its last CTAs idle, so no run is empty.
__device__ __forceinline__ long long run_start(long long total, int c, int runs) { return total * c / runs; }
__device__ __forceinline__ int run_count(long long total, int grid) { return total < grid ? (int)total : grid; }

// The last key that row r of the item's sequence sees (-1: none; rows past the sequence's: -1).
__device__ __forceinline__ int row_limit(const AttnP& p, const Seq& s, int r) {
  const int i = r / p.G;
  return i >= s.m ? -1 : p.causal ? min(s.n - 1, s.n - s.m + i) : s.n - 1;
}

// One row's result from its merged sums: bf16 values a f, and the LSE.
__device__ __forceinline__ float row_factor(const AttnP& p, int hk, float l, float m, float mv) {
  if (!(l > 0.0f) && l == l) return 0.0f;  // no key seen
  return (p.c.per_token ? attn::ex2(mv - m) : finite_or_nan(__ldg(p.c.vs + hk))) / l;
}
// FA_DEBUG_BOUNDS builds: row r of kv head hk of the sequence is a row of q
__device__ __forceinline__ bool q_row_ok(const AttnP& p, const Seq& s, int hk, int r, int where) {
  const int i = r / p.G, hq = hk * p.G + r - i * p.G;
  return in_bounds(s.q0 >= 0 && i >= 0 && s.q0 + i < p.bt.T && hq >= 0 && hq < p.Hq, where);
}
__device__ __forceinline__ float row_lse(float l, float m) { return (m + log2f(l)) * 0.69314718055994530942f; }

// Programmatic dependent launch: a kernel lets the one behind it start (its launch and prologue then overlap), which
// waits for it before reading what it wrote.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The merge of the items that a run's border cuts: CTA c takes the item that starts in run c and
// ends past it, whose pieces lie in run c's slot and in slot 0 of the runs after it; blockIdx.y takes 16 of the
// block's rows.  A thread holds four dims of one or two rows.  The pieces' (m, l, mv) come through shared memory,
// CB at a time, so that the loads of the accumulators do not wait for one another (one piece after
// another took 32 us for the 38 pieces of a 131071-token item; this 5).
constexpr int CB = 64;
template <typename PL, int D>
__global__ void __launch_bounds__(256) combine_kernel(const AttnP p, int grid) {
  const int lane = threadIdx.x & 31;
  const int c = blockIdx.x;
  const long long total = total_units<PL>(p, lane);
  const int runs = run_count(total, grid);
  Item it = {};
  long long item_end = 0;
  int rows = 0, slot0 = 0;
  const int row0 = blockIdx.y * 16;
  if (c < runs) {
    const long long u0 = run_start(total, c, runs), u1 = run_start(total, c + 1, runs);
    if (u1 < total) {
      it = find_item<PL>(p, u1 - 1, lane);
      item_end = it.first + it.nt;
      if (item_end > u1 && it.first >= u0) rows = min(it.s.m * p.G - it.rb * PL::RB, PL::RB);
      slot0 = 2 * c + (it.first == u0 ? 0 : 1);
    }
  }
  // Every CTA waits, those without work too: what follows this kernel in the stream then follows the one before it.
  wait_for_previous();
  if (row0 >= rows) return;
  // the run that holds the item's last unit u: the largest k with floor(total k / runs) <= u
  const int last = (int)((item_end * runs - 1) / total);
  const int pieces = last - c + 1;
  constexpr int CPR = D / 4, RT = 256 / CPR, NR = 16 / RT;  // chunks a row, rows side by side, rows a thread
  const int ch = threadIdx.x % CPR, rid = threadIdx.x / CPR;
  // few rows: the threads that would have none share the pieces out
  const int left = rows - row0;
  const int across = left > 4 ? RT : left > 2 ? min(4, RT) : left > 1 ? 2 : 1, splits = RT / across;
  const int r0 = rid % across, part = rid / across;
  __shared__ float4 ml[CB][16];
  __shared__ float4 sum[256];
  __shared__ float sum_l[256];
  float m[NR], mv[NR], l[NR];
  float4 acc[NR];
#pragma unroll
  for (int y = 0; y < NR; ++y) {
    m[y] = mv[y] = -INFINITY;
    l[y] = 0.0f;
    acc[y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  auto row_of = [&](int k, int r) { return (long long)(k == 0 ? slot0 : 2 * (c + k)) * PL::RB + row0 + r; };
  for (int k0 = 0; k0 < pieces; k0 += CB) {
    const int n = min(CB, pieces - k0);
    __syncthreads();
    for (int i = threadIdx.x; i < n * 16; i += 256)
      if (in_bounds(row_of(k0 + i / 16, i % 16) < 2LL * grid * PL::RB, 171)) ml[i / 16][i % 16] = p.part_ml[row_of(k0 + i / 16, i % 16)];
    __syncthreads();
#pragma unroll
    for (int y = 0; y < NR; ++y) {
      const int r = r0 + y * RT;
      if (row0 + r >= rows || (y > 0 && splits > 1)) continue;
      float mn = m[y], mvn = mv[y];
      for (int k = 0; k < n; ++k) {
        mn = fmaxf(mn, ml[k][r].x);
        mvn = fmaxf(mvn, ml[k][r].z);
      }
      const float wl = mn == m[y] ? 1.0f : attn::ex2(m[y] - mn), wo = mvn == mv[y] ? 1.0f : attn::ex2(mv[y] - mvn);
      l[y] *= wl;  // (every part sees every piece's maxima)
      acc[y] = make_float4(acc[y].x * wo, acc[y].y * wo, acc[y].z * wo, acc[y].w * wo);
      m[y] = mn;
      mv[y] = mvn;
#pragma unroll 8
      for (int k = part; k < n; k += splits) {
        const float4 v = ml[k][r];
        if (!in_bounds(row_of(k0 + k, r) < 2LL * grid * PL::RB, 172)) continue;
        const float4 x = *(reinterpret_cast<const float4*>(p.part_o + row_of(k0 + k, r) * D) + ch);
        // maxima pass over NaN, so a piece whose scores are all NaN has m = -inf, as one without keys has: its sum
        // tells them apart (NaN or 0) and enters as it is, and so do sums of p v (0, or NaN)
        l[y] += v.x > -INFINITY ? attn::ex2(v.x - mn) * v.y : v.y;
        const float w = v.z > -INFINITY ? attn::ex2(v.z - mvn) : 0.0f;
        acc[y].x += w * x.x;
        acc[y].y += w * x.y;
        acc[y].z += w * x.z;
        acc[y].w += w * x.w;
      }
    }
  }
  if (splits > 1) {
    sum[threadIdx.x] = acc[0];
    sum_l[threadIdx.x] = l[0];
    __syncthreads();
    if (part > 0) return;
    for (int q = 1; q < splits; ++q) {
      const int t = threadIdx.x + q * across * CPR;
      const float4 x = sum[t];
      acc[0].x += x.x;
      acc[0].y += x.y;
      acc[0].z += x.z;
      acc[0].w += x.w;
      l[0] += sum_l[t];
    }
  }
#pragma unroll
  for (int y = 0; y < NR; ++y) {
    const int r = r0 + y * RT;
    if (row0 + r >= rows || (y > 0 && splits > 1)) continue;
    const int rr = it.rb * PL::RB + row0 + r;
    const int i = rr / p.G, hq = it.hk * p.G + rr - i * p.G;
    const float f = row_factor(p, it.hk, l[y], m[y], mv[y]);
    const long long row = (long long)(it.s.q0 + i) * p.Hq + hq;
    if (!in_bounds(row >= 0 && row < (long long)p.bt.T * p.Hq, 173)) continue;
    const __nv_bfloat162 v0 = __floats2bfloat162_rn(acc[y].x * f, acc[y].y * f), v1 = __floats2bfloat162_rn(acc[y].z * f, acc[y].w * f);
    *reinterpret_cast<uint2*>(p.out + row * D + ch * 4) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&v0), *reinterpret_cast<const uint32_t*>(&v1));
    if (ch == 0 && p.lse) p.lse[row] = row_lse(l[y], m[y]);
  }
}

// The combine kernel behind a kernel of that plan that let it start.
template <typename PL, int D>
inline cudaError_t launch_combine(const AttnP& p, int grid, cudaStream_t s) {
  if (const cudaError_t be = bounds_attach(); be != cudaSuccess) return be;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, PL::RB / 16);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, combine_kernel<PL, D>, p, grid);
}

// Workspace of a kernel of that plan with `grid` CTAs.
template <typename PL>
inline size_t plan_ws(int D, int grid) {
  return (size_t)2 * grid * PL::RB * ((size_t)D * 4 + 16);
}
template <typename PL>
inline void plan_carve(AttnP& p, void* ws, int D, int grid) {
  p.part_o = static_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float4*>(p.part_o + (size_t)2 * grid * PL::RB * D);
}

}  // namespace paged

// A call's parameters but for the workspace.
inline paged::AttnP paged_attn_params(const PagedAttnArgs& a) {
  paged::AttnP p = {};
  p.q = static_cast<const __nv_bfloat16*>(a.q->data);
  p.q_stride = a.q->stride;
  p.c = paged_cache_of(*a.cache);
  p.bt = paged_batch_of(*a.batch, a.q->T);
  p.Hq = a.q->H;
  p.G = a.q->H / a.cache->H;
  p.causal = a.causal;
  p.scale_log2 = (a.softmax_scale > 0.0f ? a.softmax_scale : 1.0f / sqrtf((float)a.q->D)) * 1.4426950408889634f;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.status = a.status;
  return p;
}

// Query rows per kv head that a sequence of the batch can have.
inline long long paged_most_rows(const PagedAttnArgs& a) {
  const int T = a.q->T, max_q = a.batch->max_q > 0 && a.batch->max_q < T ? a.batch->max_q : T;
  return (long long)(a.batch->cu_q ? max_q : 1) * (a.q->H / a.cache->H);
}

// Tensor map over a cache's codes: boxes of one page's (at most `keys`) rows of one head, with the swizzle of
// MMA operands of that row length (128 or 64 bytes) or rows one behind the other.  A page index past the pool
// reads zeros.
inline cudaError_t make_page_map(CUtensorMap* map, const void* base, const fa_paged_cache& c, int keys, bool swizzle) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return cudaErrorNotSupported;
  const bool bnsd = c.layout == FA_LAYOUT_BNSD;
  const cuuint64_t D = c.D, H = c.H, P = c.page_size;
  const cuuint32_t rows = c.page_size < keys ? c.page_size : keys;
  const cuuint64_t dims[4] = {D, bnsd ? P : H, bnsd ? H : P, (cuuint64_t)c.pages};
  const cuuint64_t strides[3] = {D, (bnsd ? P : H) * D, H * P * D};
  const cuuint32_t box[4] = {(cuuint32_t)D, bnsd ? rows : 1, bnsd ? 1 : rows, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const CUtensorMapSwizzle swz = !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE : D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace faq
