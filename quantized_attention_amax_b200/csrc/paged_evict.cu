// paged_evict.cu -- eviction from a paged cache: keep the first `sink`, the last `recent` and the
// highest-scored of the other tokens of each (sequence, kv head), and move the kept rows to the front.
//
// One cluster of CTAs per (sequence, kv head), in one launch:
//   1. the score that the last kept candidate has, by radix selection on the scores' bits (11, 11
//      and 10 of them, highest first): each CTA counts its slice's digits in shared memory, the counts
//      of the cluster's CTAs are added through distributed shared memory;
//   2. the kept indices in order: each warp counts its part's scores above the threshold and equal to
//      it, the counts before it give its places, and of the equal ones the lowest indices are taken;
//   3. the rows, in rounds: every CTA of the cluster brings its share of the round's kept rows into
//      registers (8 chunks a thread, all on their way at once), a cluster barrier, then all are written.  A row's new index is never above its
//      old one, so what a round writes lies below every row that later rounds read: the barrier between a
//      round's reads and its writes is all the order that moving in place needs.
// The scores (once) and the kept rows (read and written once) bound it; slices are kept in shared
// memory between the passes.  The cluster is as large as the GPU's SMs allow for the number of
// (sequence, head) pairs, up to 8 CTAs.
// Measured: 8 sequences of up to 32768 tokens, 8 heads of 128, cut to 4096 (fp8 per token): 91 us, of which the moved rows'
// bytes are 22 at the copy bandwidth: the passes follow one another, each with a cluster barrier, and 64 clusters of two
// leave 20 SMs idle.  One sequence of 2000 cut to 512: 28 us, the chain of passes and barriers alone.
#include <cooperative_groups.h>

#include "paged_common.cuh"

namespace cg = cooperative_groups;

namespace faq {
namespace {
using namespace paged;

constexpr int ET = 1024;            // threads per CTA
constexpr int EW = ET / 32;
constexpr int BINS = 2048;
constexpr int KEY_BYTES = 144 * 1024;  // score bits of the slice
constexpr int RU = 8;               // rows a thread holds in a round

struct EvictP {
  Cache c;
  Batch bt;
  const float* scores;
  long long score_stride;
  int budget, sink, recent;
  int* kept;
  int* new_lens;
  float* scores_out;
  int* status;
};

// Order-preserving bits: NaN lowest, then -inf .. +inf, the two zeros equal.
__device__ __forceinline__ uint32_t score_bits(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.0f ? 0.0f : x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct __align__(16) EvictSmem {
  uint32_t hist[2][BINS];
  uint32_t warp_sum[EW];
  uint32_t warp_gt[EW], warp_eq[EW];
  uint32_t cta_gt, cta_eq;
  uint32_t digit, above;  // the digit holding the threshold, and how many lie above it
};

template <int D>
__global__ void __launch_bounds__(ET, 1) paged_evict_kernel(const EvictP p) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ EvictSmem sm;
  cg::cluster_group cl = cg::this_cluster();
  const int cs = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = blockIdx.x / cs;
  const int b = bh / p.c.H, h = bh - b * p.c.H;
  const int n = __ldg(p.bt.lens + b);
  if (n < 0 || n > ((long long)p.bt.max_pages << p.c.page_shift) || n > p.score_stride) {  // uniform in the cluster
    if (tid == 0) bad(p.status, 231);
    return;
  }
  const float* sc = p.scores + (long long)bh * p.score_stride;
  int* kept = p.kept + (long long)bh * p.budget;
  float* so = p.scores_out ? p.scores_out + (long long)bh * p.score_stride : nullptr;
  const int keep = min(n, p.budget);
  const int gt0 = rank * ET + tid, gts = cs * ET;  // the thread among the cluster's
  if (h == 0 && gt0 == 0) p.new_lens[b] = keep;
  // the extents of this item's lists (FA_DEBUG_BOUNDS builds)
  auto kept_ok = [&](long long i) { return in_bounds(i >= 0 && i < p.budget, 194); };
  auto score_ok = [&](long long i) { return in_bounds(i >= 0 && i < p.score_stride, 195); };
  for (int i = keep + gt0; i < p.budget; i += gts)
    if (kept_ok(i)) kept[i] = -1;
  if (so)
    for (long long i = keep + gt0; i < p.score_stride; i += gts)
      if (score_ok(i)) so[i] = 0.0f;
  if (n <= p.budget) {
    for (int i = gt0; i < n; i += gts) {
      if (!kept_ok(i) || !score_ok(i)) continue;
      kept[i] = i;
      if (so) so[i] = __ldg(sc + i);
    }
    return;
  }

  // ---- 1. the threshold: the need-th highest of the candidates [sink, n - recent)
  const int cand = n - p.recent - p.sink;
  int need = p.budget - p.sink - p.recent;  // 0 <= need < cand
  const int chunk = (cand + cs - 1) / cs;
  const int lo = min(cand, rank * chunk), cnt = min(cand, lo + chunk) - lo;
  const float* mine = sc + p.sink + lo;
  constexpr int CAP = KEY_BYTES / 4;
  const int cached = min(cnt, CAP);
  for (int i0 = 0; i0 < cached; i0 += 8 * ET) {  // eight loads on their way at once
    float x[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int i = i0 + q * ET + tid;
      x[q] = i < cached && score_ok(p.sink + lo + i) ? __ldg(mine + i) : 0.0f;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int i = i0 + q * ET + tid;
      if (i < cached) keys[i] = score_bits(x[q]);
    }
  }
  auto key = [&](int i) { return i < CAP ? keys[i] : score_ok(p.sink + lo + i) ? score_bits(__ldg(mine + i)) : 0u; };

  uint32_t thr = 0;
  if (need > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t mask = pass == 2 ? 1023u : 2047u;
      uint32_t* hist = sm.hist[pass & 1];
      for (int i = tid; i < BINS; i += ET) hist[i] = 0;
      __syncthreads();
      const uint32_t hi_mask = pass == 0 ? 0u : pass == 1 ? 0xFFE00000u : 0xFFFFFC00u;
#pragma unroll 4
      for (int i = tid; i < cnt; i += ET) {
        const uint32_t k = key(i);
        if ((k & hi_mask) == thr) atomicAdd(&hist[(k >> shift) & mask], 1u);
      }
      cl.sync();
      // this thread's two bins, the higher first, summed over the cluster
      static_assert(BINS == 2 * ET, "two bins a thread");
      uint32_t mybin[2] = {0, 0};
      const int top = BINS - 1 - 2 * tid;
#pragma unroll 8
      for (int r = 0; r < cs; ++r) {
        const uint2 h = *reinterpret_cast<const uint2*>(cl.map_shared_rank(hist, r) + top - 1);
        mybin[0] += h.y;
        mybin[1] += h.x;
      }
      const uint32_t sum = mybin[0] + mybin[1];
      uint32_t incl = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
      }
      if (lane == 31) sm.warp_sum[warp] = incl;
      __syncthreads();
      uint32_t before = incl - sum;
      for (int w = 0; w < warp; ++w) before += sm.warp_sum[w];
      if (before < (uint32_t)need && before + sum >= (uint32_t)need) {  // one thread of the CTA
        int q = 0;
        while (before + mybin[q] < (uint32_t)need) before += mybin[q++];
        sm.digit = (uint32_t)(top - q);
        sm.above = before;
      }
      __syncthreads();
      thr |= sm.digit << shift;
      need -= (int)sm.above;
      __syncthreads();  // digit, above and warp_sum are read
    }
  }
  // need: how many of the scores equal to thr are kept (with need == 0 from the start: none at all)
  const bool none = p.budget - p.sink - p.recent == 0;

  // ---- 2. the kept indices, in order
  const int per = ((cnt + EW - 1) / EW + 31) / 32 * 32;
  const int w0 = min(cnt, warp * per), w1 = min(cnt, w0 + per);
  uint32_t gt = 0, eq = 0;
  __syncthreads();
  if (!none)
    for (int i = w0 + lane; i - lane < w1; i += 32) {
      const uint32_t k = i < w1 ? key(i) : 0;
      gt += __popc(__ballot_sync(0xffffffffu, i < w1 && k > thr));
      eq += __popc(__ballot_sync(0xffffffffu, i < w1 && k == thr));
    }
  if (lane == 0) {
    sm.warp_gt[warp] = gt;
    sm.warp_eq[warp] = eq;
  }
  __syncthreads();
  if (tid == 0) {
    uint32_t a = 0, e = 0;
    for (int w = 0; w < EW; ++w) {
      a += sm.warp_gt[w];
      e += sm.warp_eq[w];
    }
    sm.cta_gt = a;
    sm.cta_eq = e;
  }
  cl.sync();
  uint32_t gt_before = 0, eq_before = 0;
  for (int r = 0; r < rank; ++r) {
    gt_before += *cl.map_shared_rank(&sm.cta_gt, r);
    eq_before += *cl.map_shared_rank(&sm.cta_eq, r);
  }
  for (int w = 0; w < warp; ++w) {
    gt_before += sm.warp_gt[w];
    eq_before += sm.warp_eq[w];
  }
  const unsigned below = (1u << lane) - 1u;
  if (!none)
    for (int i = w0 + lane; i - lane < w1; i += 32) {
      const uint32_t k = i < w1 ? key(i) : 0;
      const bool is_gt = i < w1 && k > thr, is_eq = i < w1 && k == thr;
      const unsigned bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
      const uint32_t e = eq_before + __popc(be & below);  // equal scores before this one
      if (is_gt || (is_eq && e < (uint32_t)need)) {
        const uint32_t place = gt_before + __popc(bg & below) + min(e, (uint32_t)need);
        if (kept_ok((long long)p.sink + place)) kept[p.sink + place] = p.sink + lo + i;
      }
      gt_before += __popc(bg);
      eq_before += __popc(be);
    }
  for (int i = gt0; i < p.sink; i += gts)
    if (kept_ok(i)) kept[i] = i;
  for (int i = gt0; i < p.recent; i += gts)
    if (kept_ok(p.budget - p.recent + i)) kept[p.budget - p.recent + i] = n - p.recent + i;
  cl.sync();  // the list is written; the slices' keys are read

  if (so)  // the kept tokens' scores
#pragma unroll 4
    for (int i = gt0; i < keep; i += gts)
      if (score_ok(i) && score_ok(__ldcg(kept + i))) so[i] = __ldg(sc + __ldcg(kept + i));

  // ---- 3. the rows
  constexpr int CH = D / 16;               // 16-byte chunks per code row
  constexpr int RS = ET / (2 * CH);        // rows side by side: 2 CH threads a row, K's chunks, then V's
  constexpr int R = RU * RS;               // rows per CTA and round
  const int c = tid % (2 * CH), r0 = tid / (2 * CH), cc = c % CH;
  uint8_t* codes = c < CH ? p.c.k : p.c.v;
  float* scales = p.c.per_token ? (c < CH ? p.c.ks : p.c.vs) : nullptr;  // moved by the first of K's and of V's threads
  const int* table = p.bt.table + (long long)b * p.bt.max_pages;
  for (int base = 0; base < keep; base += cs * R) {
    const int d0 = base + rank * R + r0;
    int f[RU];
    uint4 row[RU];
    float scale[RU];
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      const int d = d0 + u * RS;
      f[u] = d < keep ? __ldcg(kept + d) : -1;
      if (f[u] == d) f[u] = -1;  // stays where it is
    }
    int pg[RU];
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      if (!in_bounds(f[u] < n && ((d0 + u * RS) >> p.c.page_shift) >= 0, 196)) f[u] = -1;
      pg[u] = f[u] >= 0 ? __ldg(table + (f[u] >> p.c.page_shift)) : -1;
    }
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      if (f[u] >= 0 && (unsigned)pg[u] >= (unsigned)p.c.pages) {
        bad(p.status, 232);
        f[u] = -1;
      }
      if (f[u] >= 0) {
        const int slot = f[u] & p.c.page_mask;
        if (!p.c.holds(p.c.row(pg[u], h, slot) + 16 * cc, 16, 197) || !p.c.holds_scale(p.c.scale(pg[u], h, slot), 198)) {
          f[u] = -1;
          continue;
        }
        row[u] = __ldcg(reinterpret_cast<const uint4*>(codes + p.c.row(pg[u], h, slot)) + cc);
        if (scales && cc == 0) scale[u] = __ldcg(scales + p.c.scale(pg[u], h, slot));
      }
    }
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      const int d = d0 + u * RS;
      pg[u] = f[u] >= 0 ? __ldg(table + (d >> p.c.page_shift)) : -1;
    }
    cl.sync();  // every row of the round is read
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      if (f[u] < 0) continue;
      if ((unsigned)pg[u] >= (unsigned)p.c.pages) {
        bad(p.status, 232);
        continue;
      }
      const int slot = (d0 + u * RS) & p.c.page_mask;
      if (!p.c.holds(p.c.row(pg[u], h, slot) + 16 * cc, 16, 197) || !p.c.holds_scale(p.c.scale(pg[u], h, slot), 198)) continue;
      reinterpret_cast<uint4*>(codes + p.c.row(pg[u], h, slot))[cc] = row[u];
      if (scales && cc == 0) scales[p.c.scale(pg[u], h, slot)] = scale[u];
    }
  }
}

template <int D>
cudaError_t launch_d(const EvictP& p, cudaStream_t s) {
  auto kern = paged_evict_kernel<D>;
  cudaError_t e;
  if ((e = set_smem_limit(reinterpret_cast<const void*>(kern), KEY_BYTES)) != cudaSuccess) return e;
  const long long items = (long long)p.bt.B * p.c.H;
  int cs = 8;
  while (cs > 1 && items * cs > sm_count()) cs >>= 1;
  if (items * cs > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * cs));
  cfg.blockDim = dim3(ET);
  cfg.dynamicSmemBytes = KEY_BYTES;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = cs;
  at.val.clusterDim.y = 1;
  at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_paged_evict(const PagedEvictArgs& a, cudaStream_t s) {
  if (const cudaError_t be = bounds_attach(); be != cudaSuccess) return be;
  EvictP p = {};
  p.c = paged_cache_of(*a.cache);
  p.bt = paged_batch_of(*a.batch, 0);
  p.scores = a.scores;
  p.score_stride = a.score_stride;
  p.budget = a.budget;
  p.sink = a.sink;
  p.recent = a.recent;
  p.kept = a.kept;
  p.new_lens = a.new_lens;
  p.scores_out = a.scores_out;
  p.status = a.status;
  return a.cache->D == 128 ? launch_d<128>(p, s) : launch_d<64>(p, s);
}

}  // namespace faq
