// paged_weights.cu -- the attention weight that new tokens give each cached token (column sums of the
// softmax matrix):  w_j = sum over the rows r of a kv head that see j of 2^(x_rj - log2(e) lse_r),
// x_rj = log2(e) softmax_scale s_k(j) q_r . k_j.
//
// With one new token per sequence the K codes' bytes bound it; with a window of tokens the exponentials and what
// surrounds them do.  As in the decode kernel the codes are MMA operands as TMA leaves them and the query
// rows enter as three 8-bit digits each (paged_digits.cuh):  S^T [128 keys x 3 rows] = K . Q^T.  A thread owns a
// key: it joins the digits' sums, takes the exponential and adds up along its rows, so a key's weight is summed in a
// fixed order by one thread, and no two threads write one key.  Up to 256 rows stay in shared memory; a
// sequence with more is walked once per 256 rows, adding to what the walk before left.  Two warpgroups take the key
// tiles in turn (64 rows of one tile at a time each), so one's MMAs run under the other's exponentials.
// Units are 128 keys of one (sequence, kv head); the CTAs take equal runs of them, counted from the lengths on
// the device.
// Measured: one token to each of 16 sequences of up to 16384 (int8 per head, 212 MB): 47 us, 4.5 TB/s; 64 tokens to two of
// up to 32768 (fp8 per token): 101 us, the exponentials' loops of eight warps (four warpgroups with 32 rows a step
// spill registers and take as long, with 16 rows a step 142 us).
#include "paged_digits.cuh"
#include "paged_sched.cuh"

namespace faq {
namespace {
using namespace paged;

constexpr int TK = 128;      // keys per tile
constexpr int NKS = 4;       // K tiles in flight
constexpr int QR = 256;      // query rows in shared memory
constexpr int WT = 384;      // warp 0 loads, warp 1 MMAs, warps 4-7 and 8-11 the weights

struct WeightP {
  AttnP a;
  int accumulate;
  float* acc;
  long long acc_stride;
};

// A row's constants: x - lse2 is sum * s_k * f - hi - lo; lim: the last key it sees.
struct __align__(16) RowC {
  float f, hi, lo;
  int lim;
};

// R rows to a group of 3 R columns: digit k of row r of the group is column k R + r.  Groups of 16 rows come in
// steps of up to four (N = 48 .. 192 columns); up to 4 rows in all take one group of 4 (N = 16).
template <int D, int R>
struct WL {
  static constexpr int GC = R == 4 ? 16 : 48;          // columns of a group
  static constexpr int GS = R == 4 ? 1 : 4;            // groups of a step
  static constexpr int ROWS = R == 4 ? 4 : QR;
  static constexpr uint32_t TILE = TK * D;
  static constexpr uint32_t Q = 0;                     // [ROWS / R groups][GC][D] digits, swizzled
  static constexpr uint32_t K = (ROWS / R * GC * D + 1023) & ~1023u;
  static constexpr uint32_t ROW = K + NKS * TILE;
  static constexpr uint32_t BAR = ROW + ROWS * 16;
  static constexpr uint32_t TOTAL = BAR + 256;
  static constexpr uint32_t ALLOC = TOTAL + 1024;
};

enum { W_KF = 0, W_KE = W_KF + NKS, W_Q = W_KE + NKS, W_QD, W_SF, W_SE = W_SF + 2, W_FIN = W_SE + 2, W_COUNT };

__device__ __forceinline__ int weight_units(const WeightP& p, int b, Seq& s) {
  s = load_seq(p.a.bt, p.a.c.page_shift, b, p.a.status, 221);
  if (s.n > p.acc_stride) {
    bad(p.a.status, 222);
    s = {0, 0, 0};
  }
  return s.m > 0 || !p.accumulate ? (s.n + TK - 1) / TK : 0;
}

// The CTA's run, piece by piece: key tiles [t0, t1) of one (sequence, kv head).
struct WRun {
  int b, hk, nt, t0, t1;
  Seq s;
  long long left;  // units of the run from t0 on
  __device__ __forceinline__ void piece() { t1 = (int)(left < nt - t0 ? t0 + left : nt); }
  __device__ __forceinline__ bool next(const WeightP& p) {
    left -= t1 - t0;
    if (left <= 0) return false;
    t0 = 0;
    if (++hk == p.a.c.H) {
      hk = 0;
      do {
        if (++b >= p.a.bt.B) return false;  // cannot be while the lengths stay as they were counted
        nt = weight_units(p, b, s);
      } while (nt == 0);
    }
    piece();
    return true;
  }
};

template <int D, bool FP8, bool TOK, int R>
__global__ void __launch_bounds__(WT, 1) paged_weights_kernel(const __grid_constant__ CUtensorMap tmk, const WeightP wp) {
  using L = WL<D, R>;
  constexpr uint32_t SW = D == 128 ? kSwz128 : kSwz64, SBO = 8 * D;
  const AttnP& p = wp.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + W_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* out_rows = reinterpret_cast<int*>(tmem_slot + 2);  // [2]: a walk's rows hold one that gives nothing
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // ---- the run: units [total c / grid, total (c + 1) / grid)
  long long total = 0;
  for (int b = lane; b < p.bt.B; b += 32) {
    Seq s;
    total += weight_units(wp, b, s);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  total *= p.c.H;
  const long long u0 = total * blockIdx.x / gridDim.x, u1 = total * (blockIdx.x + 1) / gridDim.x;
  if (u0 >= u1) return;
  WRun run = {};
  run.b = -1;
  {
    long long base = 0;
    for (int b0 = 0; b0 < p.bt.B && run.b < 0; b0 += 32) {
      Seq x = {0, 0, 0};
      const int n = b0 + lane < p.bt.B ? weight_units(wp, b0 + lane, x) : 0;
      const long long mine = (long long)n * p.c.H, end = base + lanes_before(mine, lane);
      const unsigned after = __ballot_sync(0xffffffffu, end > u0);
      if (after) {
        const int src = __ffs(after) - 1;
        run.b = b0 + src;
        run.s.q0 = __shfl_sync(0xffffffffu, x.q0, src);
        run.s.m = __shfl_sync(0xffffffffu, x.m, src);
        run.s.n = __shfl_sync(0xffffffffu, x.n, src);
        run.nt = __shfl_sync(0xffffffffu, n, src);
        const long long at = u0 - __shfl_sync(0xffffffffu, end - mine, src);
        run.hk = (int)(at / run.nt);
        run.t0 = (int)(at - (long long)run.hk * run.nt);
      }
      base = __shfl_sync(0xffffffffu, end, 31);
    }
  }
  run.left = u1 - u0;
  run.piece();

  if (tid == 0) {
    for (int i = 0; i < NKS; ++i) {
      mbar_init(&bar[W_KF + i], 1);
      mbar_init(&bar[W_KE + i], 1);
    }
    mbar_init(&bar[W_Q], 256);
    mbar_init(&bar[W_QD], 256);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar[W_SF + i], 1);
      mbar_init(&bar[W_SE + i], 4);
    }
    mbar_init(&bar[W_FIN], 1);
    *abort_flag = 0;
    out_rows[0] = out_rows[1] = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  auto walks = [&]() { return (run.s.m * p.G + L::ROWS - 1) / L::ROWS; };  // of the piece's tiles
  auto wait = [&](int which, int phase, int where) { return mbar_wait(&bar[which], phase & 1, abort_flag, p.status, where); };
  auto wwait = [&](int which, int phase, int where) { return __all_sync(0xffffffffu, wait(which, phase, where)); };

  if (warp == 0) {
    // ------------------------------------------------------------------ loads
    const int box = min(TK, p.c.page_mask + 1), nbox = TK / box;
    if (lane == 0) tma_prefetch_desc(&tmk);
    int j = 0;
    bool ok = true;
    do {
      const int b = run.b, hk = run.hk, n = run.s.n;
      auto page = [&](int t) {
        const int k0 = t * TK + lane * box;
        int pg = p.c.pages;  // past the end, or not a page of the cache: one past the pool, read as zeros
        if (t < run.t1 && lane < nbox && k0 < n) {
          pg = page_of(p.bt, p.c, b, k0, p.status, 223);
          if (pg < 0) pg = p.c.pages;
        }
        return pg;
      };
      const int nw = walks();
      for (int w = 0; w < nw && ok; ++w) {
        int pg = page(run.t0);
        for (int t = run.t0; t < run.t1 && ok; ++t, ++j) {
          const int next = page(t + 1), s = j % NKS;
          const int off = (t * TK + lane * box) & p.c.page_mask;
          if (j >= NKS && !(ok = wwait(W_KE + s, j / NKS - 1, 261))) break;
          if (lane == 0) mbar_arrive_expect_tx(&bar[W_KF + s], L::TILE);
          __syncwarp();
          if (lane < nbox)
            tma_load_4d(smem + L::K + s * L::TILE + lane * box * D, &tmk, &bar[W_KF + s], 0, p.c.bnsd ? off : hk,
                        p.c.bnsd ? hk : off, pg);
          pg = next;
        }
      }
    } while (ok && run.next(wp));
    if (*abort_flag)
      for (int t = max(0, j - NKS); t < j; ++t) mbar_drain(&bar[W_KF + t % NKS], (t / NKS) & 1);
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------- MMAs
    if (lane == 0) {
      const uint32_t sQ = smem_u32(smem + L::Q), sK = smem_u32(smem + L::K);
      int j = 0, nq = 0, steps[2] = {0, 0};
      bool ok = true;
      do {
        const int rows = run.s.m * p.G, nw = walks();
        for (int w = 0; w < nw && ok; ++w, ++nq) {
          if (!(ok = wait(W_Q, nq, 262))) break;
          tc_fence_after();
          const int groups = (min(rows - w * L::ROWS, L::ROWS) + R - 1) / R;
          // two tiles at a time, one to a warpgroup, their steps in turn
          for (int t = run.t0; t < run.t1 && ok; t += 2, j += 2) {
            const int n = min(2, run.t1 - t);
            for (int g = 0; g < groups && ok; g += L::GS) {
              const int gn = min(L::GS, groups - g);
              const uint32_t idesc = FP8 ? make_idesc(kAccF32, kFmtE4M3, kFmtE4M3, 0, 0, gn * L::GC, 128)
                                         : make_idesc(kAccS32, kFmtS8, kFmtS8, 0, 0, gn * L::GC, 128);
              for (int x = 0; x < n && ok; ++x) {
                const int s = (j + x) % NKS;
                if (g == 0) ok = wait(W_KF + s, (j + x) / NKS, 263);
                if (ok && steps[x] > 0) ok = wait(W_SE + x, steps[x] - 1, 264);
                if (!ok) break;
                ++steps[x];
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk) {
                  const uint64_t da = make_sdesc(sK + s * L::TILE + kk * 32, 16, SBO, SW);
                  const uint64_t db = make_sdesc(sQ + g * L::GC * D + kk * 32, 16, SBO, SW);
                  if (FP8)
                    mma_f8f6f4(tbase + x * 256, da, db, idesc, kk > 0);
                  else
                    mma_i8(tbase + x * 256, da, db, idesc, kk > 0);
                }
                mma_commit(&bar[W_SF + x]);
                if (g + L::GS >= groups) mma_commit(&bar[W_KE + s]);
              }
            }
            if (n == 1) --j;  // an odd last tile
          }
        }
      } while (ok && run.next(wp));
      mma_commit(&bar[W_FIN]);
      mbar_drain(&bar[W_FIN], 0);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- weights
    const int x = (warp - 4) >> 2;             // warpgroup: the tiles of its turn
    const int wt = tid - 128;                  // of the 256 threads
    const int i = (warp & 3) * 32 + lane;      // key of the tile, TMEM lane
    const uint32_t loff = (uint32_t)((warp & 3) * 32) << 16;
    RowC* rowc = reinterpret_cast<RowC*>(smem + L::ROW);
    int nq = 0, steps = 0;
    bool ok = true;
    do {
      const Seq s = run.s;
      const int hk = run.hk, b = run.b, rows = s.m * p.G, nw = walks();
      float* acc = wp.acc + ((long long)b * p.c.H + hk) * wp.acc_stride;
      auto acc_ok = [&](int j) { return in_bounds(j >= 0 && j < wp.acc_stride && b >= 0 && b < p.bt.B && hk >= 0 && hk < p.c.H, 192); };
      if (nw == 0)  // no new token, not accumulating: zeros
        for (int j = run.t0 * TK + wt; j < min(run.t1 * TK, s.n); j += 256)
          if (acc_ok(j)) acc[j] = 0.0f;
      for (int w = 0; w < nw && ok; ++w, ++nq) {
        // ---- Q digits and the rows' constants, D / 16 lanes a row, once the MMAs of the walk before are done
        if (nq > 0) {
          mbar_arrive(&bar[W_QD]);
          if (!(ok = wwait(W_QD, nq - 1, 265))) break;
        }
        constexpr int LPR = D / 16;
        const int here = min(rows - w * L::ROWS, L::ROWS), groups = (here + R - 1) / R;
        for (int idx = wt; idx - lane < groups * R * LPR; idx += 256) {
          const int rl = idx / LPR, c = idx % LPR, r = w * L::ROWS + rl, ii = r / p.G;
          const bool in = idx < groups * R * LPR, mine = in && r < rows && q_row_ok(p, s, hk, r, 191);
          const int hq = hk * p.G + r - ii * p.G;
          // a row whose LSE is not finite gives nothing, whatever its query and the keys hold
          const float lse = mine ? __ldg(p.lse + (long long)(s.q0 + ii) * p.Hq + hq) : -INFINITY;
          const bool live = fabsf(lse) < INFINITY;
          const uint4* src = reinterpret_cast<const uint4*>(p.q + (long long)(s.q0 + ii) * p.q_stride + (long long)hq * D + c * 16);
          uint4 raw[2];
          raw[0] = live ? __ldg(src) : make_uint4(0, 0, 0, 0);
          raw[1] = live ? __ldg(src + 1) : make_uint4(0, 0, 0, 0);
          const uint32_t* wv = &raw[0].x;
          float m = 0.0f;
          bool bad_value = false;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float y0 = fabsf(__uint_as_float(wv[e] << 16)), y1 = fabsf(__uint_as_float(wv[e] & 0xFFFF0000u));
            bad_value = bad_value || y0 != y0 || y1 != y1;
            m = fmaxf(m, fmaxf(y0, y1));
          }
          if (bad_value) m = INFINITY;
#pragma unroll
          for (int off = LPR / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
          float inv;
          const float sc = digit_scale<FP8>(m, inv);
          uint32_t dw[3][4] = {};
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            uint32_t d[3];
            const float y = __uint_as_float((e & 1) ? wv[e >> 1] & 0xFFFF0000u : wv[e >> 1] << 16);
            q_digits<FP8>(sc == 0.0f ? 0.0f : y, sc, d);
#pragma unroll
            for (int k = 0; k < 3; ++k) dw[k][e >> 2] |= d[k] << (8 * (e & 3));
          }
          if (!in) continue;
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const uint32_t col = rl / R * L::GC + k * R + rl % R;
            *reinterpret_cast<uint4*>(smem + L::Q + (D == 128 ? swz128_offset(col, c) : swz64_offset(col, c))) =
                make_uint4(dw[k][0], dw[k][1], dw[k][2], dw[k][3]);
          }
          if (c == 0) {
            RowC rc;
            rc.f = p.scale_log2 * inv;
            rc.lim = live ? row_limit(p, s, r) : -1;
            if (mine && rc.lim < 0) out_rows[nq & 1] = 1;
            // log2(e) lse in two terms: log2(e) is 1.442695... as fp32 plus its remainder; rows that give
            // nothing: so far down that every exponential is 0
            rc.hi = rc.lim < 0 ? 1e30f : lse * 1.44269502f;
            rc.lo = rc.lim < 0 ? 0.0f : fmaf(lse, 1.44269502f, -rc.hi) + lse * 1.92596303e-8f;
            rowc[rl] = rc;
          }
        }
        fence_async_smem();
        mbar_arrive(&bar[W_Q]);
        if (!(ok = wwait(W_Q, nq, 266))) break;
        const bool some_out = out_rows[nq & 1] != 0;
        if (wt == 0) out_rows[(nq + 1) & 1] = 0;  // read in the walk before, written in the next
        const int lim_lo = p.causal ? s.n - s.m + w * L::ROWS / p.G : s.n - 1;  // every row of the walk sees the keys up to here
        // ---- this warpgroup's tiles
        float sk_next = 0.0f;
        auto load_scale = [&](int t) {
          const int key = t * TK + i;
          if (!TOK) return __ldg(p.c.ks + hk);
          if (t >= run.t1 || key >= s.n) return 0.0f;
          const int pg = page_of(p.bt, p.c, b, key, p.status, 223);
          const long long si = p.c.scale(pg, hk, key & p.c.page_mask);
          return pg >= 0 && p.c.holds_scale(si, 193) ? __ldg(p.c.ks + si) : 0.0f;
        };
        if (run.t0 + x < run.t1) sk_next = load_scale(run.t0 + x);
        for (int t = run.t0 + x; t < run.t1 && ok; t += 2) {
          const int key = t * TK + i;
          const float sk = sk_next;
          sk_next = TOK ? load_scale(t + 2) : sk;
          const bool add = wp.accumulate || w > 0;
          const float old = add && key < s.n && acc_ok(key) ? acc[key] : 0.0f;
          // (rows that pad a group need no mask of their own: a key that makes them NaN makes a row that sees it NaN)
          const bool masked = some_out || t * TK + TK - 1 > lim_lo;
          float sum[2] = {0.0f, 0.0f};
          for (int g = 0; g < groups && ok; g += L::GS, ++steps) {
            if (!(ok = wwait(W_SF + x, steps, 267))) break;
            tc_fence_after();
            const int gn = min(L::GS, groups - g);
#pragma unroll 1
            for (int q = 0; q < gn; ++q) {
              uint32_t a[L::GC];
#pragma unroll
              for (int c = 0; c < L::GC / 16; ++c)
                tmem_ld16(tbase + x * 256 + q * L::GC + c * 16 + loff, *reinterpret_cast<uint32_t(*)[16]>(&a[16 * c]));
              tmem_ld_wait();
              const RowC* rq = rowc + (g + q) * R;
#pragma unroll
              for (int r = 0; r < R; ++r) {
                const RowC rc = rq[r];
                const float y = join_digits<FP8>(a[r], a[R + r], a[2 * R + r]) * sk;
                float e = attn::ex2(fmaf(y, rc.f, -rc.hi) - rc.lo);
                if (masked) e = key <= rc.lim ? e : 0.0f;
                sum[r & 1] += e;
              }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[W_SE + x]);
          }
          if (ok && key < s.n && acc_ok(key)) acc[key] = old + (sum[0] + sum[1]);
        }
      }
    } while (ok && run.next(wp));
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int D, bool FP8, bool TOK, int R>
cudaError_t launch_r(const CUtensorMap& mk, const WeightP& p, cudaStream_t s) {
  using L = WL<D, R>;
  static_assert(L::ALLOC <= 227 * 1024, "shared memory per CTA");
  auto kern = paged_weights_kernel<D, FP8, TOK, R>;
  cudaError_t e;
  if ((e = set_smem_limit(reinterpret_cast<const void*>(kern), L::ALLOC)) != cudaSuccess) return e;
  kern<<<sm_count(), WT, L::ALLOC, s>>>(mk, p);
  return cudaGetLastError();
}

template <int D, bool FP8, bool TOK>
cudaError_t launch_d(const CUtensorMap& mk, const WeightP& p, long long rows, cudaStream_t s) {
  return rows <= 4 ? launch_r<D, FP8, TOK, 4>(mk, p, s) : launch_r<D, FP8, TOK, 16>(mk, p, s);
}

template <int D>
cudaError_t launch_mode(const CUtensorMap& mk, const WeightP& p, int mode, long long rows, cudaStream_t s) {
  switch (mode) {
    case FA_MODE_INT8_PER_HEAD: return launch_d<D, false, false>(mk, p, rows, s);
    case FA_MODE_FP8_PER_HEAD: return launch_d<D, true, false>(mk, p, rows, s);
    case FA_MODE_INT8_PER_TOKEN: return launch_d<D, false, true>(mk, p, rows, s);
    case FA_MODE_FP8_PER_TOKEN: return launch_d<D, true, true>(mk, p, rows, s);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace

cudaError_t launch_paged_weights(const PagedAttnArgs& a, cudaStream_t s) {
  WeightP p = {};
  p.a = paged_attn_params(a);
  p.accumulate = a.accumulate;
  p.acc = a.acc;
  p.acc_stride = a.acc_stride;
  if (const cudaError_t be = bounds_attach(); be != cudaSuccess) return be;
  CUtensorMap mk;
  const cudaError_t e = make_page_map(&mk, a.cache->k_codes, *a.cache, TK, true);
  if (e != cudaSuccess) return e;
  const long long rows = paged_most_rows(a);
  return a.q->D == 128 ? launch_mode<128>(mk, p, a.cache->mode, rows, s) : launch_mode<64>(mk, p, a.cache->mode, rows, s);
}

}  // namespace faq
