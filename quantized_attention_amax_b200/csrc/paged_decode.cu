// paged_decode.cu -- attention of at most 16 query rows per kv head (single tokens, drafts) over a paged
// 8-bit cache, on the tensor cores' 8-bit kinds.
//
// The cache's bytes bound it (2 n Hkv D of them per sequence; with 16 rows the softmax threads do, which hold all of a
// key's rows), so nothing but the tensor core touches the
// codes: TMA brings 128-key tiles of K and V, page by page, into swizzled shared memory, and they are MMA
// operands as they are.  The query rows and the probabilities enter as three 8-bit digits each
// (paged_digits.cuh), three MMA columns per row:
//   S^T [128 keys x N] = K . Q^T       A = K codes, B = Q digits,        N >= 3 R (R rows)
//   O^T [128 dims x N] = V^T . P^T     A = V codes (MN-major), B = P digits
// With D = 64 the second product's 128 rows are the 64 dims over the tile's first 64 keys, then over its last
// 64 (V's two halves as two operand atoms); its columns are doubled likewise, and of the four blocks the two that
// pair a half with itself count.
// A softmax thread owns a key of S^T and a dim of O^T (D = 64: of one half's).  Per tile: join the digits' sums into scores, the rows'
// maxima over the 128 keys (warp reductions, then the four warps through shared memory), p = 2^(x - m) into the row
// sums, and the digits of w = s_v 2^(x - u) for the second product (per-head modes: w = p, without s_v), 2^u the row's
// largest weight so far, halved until it is less than twice the tile's own largest: w is at most 1 whatever the scales'
// range, and the digits' fixed step stays small beside a tile's weights, however far these lie below the row's
// largest (a long history's many small weights would otherwise count in the row sum alone).  O is kept in registers,
// rescaled from tile to tile, by whole powers of two while the maximum stays.  Two CTAs per SM cover each other's chains; K / V rings of three tiles keep about 100 KB per CTA
// in flight.  Work is shared out as paged_sched.cuh says; a CTA's rings run on across its items.
// Measured (combine included): 16 sequences of up to 32768 tokens, 32 / 8 heads of 128, int8 per head (760 MB): 127 to
// 130 us, 5.8 to 6.0 TB/s, 89 to 91 % of the copy bandwidth (with warp-level 16-bit MMAs on converted codes: 221), fp8 per token
// 136; one of 131071, fp8 per token: 62 us (42 at the copy bandwidth; the runs' starts and the combine are the rest); one
// of 1000: 12.6 us, the two launches and one chain; four tokens to each of 8 sequences of 32768: 138 us int8 per head, 183 fp8 per
// token (182 and 350 when every thread kept every row's units in registers, which spilled).
#include "paged_digits.cuh"
#include "paged_sched.cuh"

namespace faq {
namespace {
using namespace paged;

constexpr int TK = 128;     // keys per tile
constexpr int NST = 3;      // K / V stages
constexpr int DT = 192;     // warp 0 loads, warp 1 MMAs, warps 2-5 softmax
// How far (powers of two) a tile's unit may lie below the largest weight: fp32 holds O in the lower one, and what 2^24 below it is
// lost weighs 2^-84 of the largest weight.
constexpr float kFall = 60.0f;

using DPL = Plan<TK, 16, 1, 16>;

template <int D, int R>
struct DL {
  static constexpr int N = R == 4 ? 16 : R == 8 ? 32 : 48;  // 3 R columns, a multiple of 16
  static constexpr int NO = D == 128 ? N : 2 * N;           // columns of O^T
  static constexpr int NP = R == 16 ? 1 : 2;                // P buffers (16 rows leave room for one)
  static constexpr int NS = D == 64 && R == 16 ? 1 : 2;     // S buffers (two CTAs share 512 TMEM columns)
  static constexpr uint32_t TILE = TK * D;
  static constexpr uint32_t K = 0;
  static constexpr uint32_t V = K + NST * TILE;
  static constexpr uint32_t Q = V + NST * TILE;             // [N][D] digits, swizzled
  static constexpr uint32_t P = Q + N * 128;                // NP x [N][128 keys] (D = 64: [2 N][64 keys])
  static constexpr uint32_t RED = P + NP * N * 128;         // 2 x [4 warps][2 R] maxima
  static constexpr uint32_t SUM = RED + 2 * 4 * 2 * R * 4;  // [4 warps][R] sums
  static constexpr uint32_t ROW = SUM + 4 * R * 4;          // [R] factors, [R] limits
  static constexpr uint32_t NAN_KEY = ROW + 2 * R * 4;      // per dim (D = 64: of each half), and of each warp's V scales: the lowest key that is no number
  static constexpr uint32_t UNIT = NAN_KEY + 132 * 4;       // [4 warps][R] the tile's units, then 2 x [4][R] what O's changes by
  static constexpr uint32_t BAR = UNIT + 4 * R * 16 + 2 * 4 * R * 4;
  static constexpr uint32_t TOTAL = BAR + 256;
  static constexpr uint32_t ALLOC = TOTAL + 1024;
  static constexpr uint32_t TO = NS * N;                    // TMEM: S^T buffers, then two of O^T
  static constexpr uint32_t COLS = TO + 2 * NO <= 64 ? 64 : TO + 2 * NO <= 128 ? 128 : 256;
  static_assert(TO + 2 * NO <= COLS, "TMEM columns");
  static_assert(Q % 1024 == 0 && (N * 128) % 1024 == 0, "operands keep the swizzle's alignment");
  static_assert(2 * (ALLOC + 1024) <= 228 * 1024, "two CTAs per SM");
  static_assert(D == 128 || 64 * R * 4 <= N * 128, "the halves' exchange fits a P buffer");
};

enum {
  B_KF = 0,            // [NST] K tile landed
  B_KE = B_KF + NST,   // [NST] K stage free
  B_VF = B_KE + NST,   // [NST]
  B_VE = B_VF + NST,   // [NST]
  B_Q = B_VE + NST,    // Q digits of an item's piece written
  B_SF = B_Q + 1,      // [2] S^T done
  B_SE = B_SF + 2,     // [2] S^T read
  B_PF = B_SE + 2,     // [2] P digits written
  B_OF = B_PF + 2,     // [2] O^T done (and P read)
  B_OE = B_OF + 2,     // [2] O^T read
  B_RED = B_OE + 2,    // [2] the four warps' maxima written
  B_SUM = B_RED + 2,   // the four warps' sums written
  B_FIN = B_SUM + 1,
  B_COUNT = B_FIN + 1
};
static_assert(B_COUNT * 8 + 8 <= 256, "barriers fit their region");

// 32 lanes' maximum (NaN ignored), one instruction.
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Row i of a swizzled V tile: all of it past the sequence's end, else its E4M3 NaN codes, cleared, and these noted for their
// dims.  A call: its loops inlined cost the tiles that never come here 20 % (137 -> 165 us for 16 sequences of up to 32768
// tokens, fp8 per token).
template <int D>
__device__ __noinline__ void clear_nans(uint8_t* tile, int i, bool past, int key, int* nan_key) {
#pragma unroll 1
  for (int c = 0; c < D / 16; ++c) {
    uint32_t* at = reinterpret_cast<uint32_t*>(tile + (D == 128 ? swz128_offset(i, c) : swz64_offset(i, c)));
    const uint4 x = *reinterpret_cast<const uint4*>(at);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if (past) {
      *reinterpret_cast<uint4*>(at) = make_uint4(0, 0, 0, 0);
    } else if (e4m3_nans(w[0]) | e4m3_nans(w[1]) | e4m3_nans(w[2]) | e4m3_nans(w[3])) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t nans = e4m3_nans(w[e]);
        note_nans(nans, (D == 128 ? 0 : i & 64) + 16 * c + 4 * e, key, nan_key);
        at[e] = w[e] & ~((nans >> 7) * 0xFFu);
      }
    }
  }
}

// The CTA's run of units, piece by piece: an item's tiles [t0, t1).
struct Run {
  Item it;
  long long u, u1, u0;
  int t0, t1;  // key tiles of the piece
  __device__ __forceinline__ void piece() {
    const long long e = it.first + it.nt < u1 ? it.first + it.nt : u1;
    const int tiles = (it.s.n + TK - 1) / TK;
    t0 = (int)(u - it.first);
    t1 = min((int)(e - it.first), tiles);
  }
  __device__ __forceinline__ bool next(const AttnP& p) {
    u = it.first + it.nt;
    if (u >= u1 || !next_item<DPL>(p, it)) return false;
    piece();
    return true;
  }
};

template <int HD, bool FP8, bool TOK, int R>
__global__ void __launch_bounds__(DT, 2)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const AttnP p) {
  using L = DL<HD, R>;
  constexpr int N = L::N, NO = L::NO, NS = L::NS;
  constexpr int JOBS = TOK ? 2 * R : R;  // a tile's maxima: of x, and (per-token modes) of x + log2 s_v
  constexpr uint32_t TILE = L::TILE, SW = HD == 128 ? kSwz128 : kSwz64, SBO = 8 * HD;
  auto swz = [](uint32_t row, uint32_t chunk) { return HD == 128 ? swz128_offset(row, chunk) : swz64_offset(row, chunk); };
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + B_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bar + B_COUNT + 1) ;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const long long total = total_units<DPL>(p, lane);
  const int runs = run_count(total, gridDim.x);
  if ((int)blockIdx.x >= runs) return;
  Run run;
  run.u0 = run.u = run_start(total, blockIdx.x, runs);
  run.u1 = run_start(total, blockIdx.x + 1, runs);
  run.it = find_item<DPL>(p, run.u, lane);
  run.piece();

  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&bar[B_KF + i], 1);
      mbar_init(&bar[B_KE + i], 1);
      mbar_init(&bar[B_VF + i], 1);
      mbar_init(&bar[B_VE + i], 1);
    }
    mbar_init(&bar[B_Q], 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar[B_SF + i], 1);
      mbar_init(&bar[B_SE + i], 4);
      mbar_init(&bar[B_PF + i], 4);
      mbar_init(&bar[B_OF + i], 1);
      mbar_init(&bar[B_OE + i], 4);
      mbar_init(&bar[B_RED + i], 128);
    }
    mbar_init(&bar[B_SUM], 128);
    mbar_init(&bar[B_FIN], 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::COLS);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  let_next_start();

  if (warp == 0) {
    // ------------------------------------------------------------------ loads
    // a tile is 128 / page boxes (one for pages of 128 keys and more): lane l loads box l's K and V
    const int box = min(TK, p.c.page_mask + 1), nbox = TK / box;
    const bool bnsd = p.c.bnsd;
    if (lane == 0) {
      tma_prefetch_desc(&tmk);
      tma_prefetch_desc(&tmv);
    }
    int j = 0, nk = 0;  // tiles issued over the whole run (K's count leads V's inside the loop)
    bool ok = true;
    do {
      const int b = run.it.b, hk = run.it.hk, n = run.it.s.n;
      // page of box `lane` of tile t; past the sequence's end, or not a page of the cache: one past the
      // pool, which TMA reads as zeros
      auto page = [&](int t) {
        const int k0 = t * TK + lane * box;
        int pg = p.c.pages;
        if (lane < nbox && k0 < n) {
          pg = page_of(p.bt, p.c, b, k0, p.status, 212);
          if (pg < 0) pg = p.c.pages;
        }
        return pg;
      };
      int pg = run.t0 < run.t1 ? page(run.t0) : 0;
      for (int t = run.t0; t < run.t1 && ok; ++t, ++j) {
        const int nxt = t + 1 < run.t1 ? page(t + 1) : 0;  // its latency passes while this tile waits
        const int s = j % NST;
        const int off = (t * TK + lane * box) & p.c.page_mask;
        if (j >= NST) ok = __all_sync(0xffffffffu, mbar_wait(&bar[B_KE + s], ((j / NST) - 1) & 1, abort_flag, p.status, 213));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&bar[B_KF + s], TILE);
        __syncwarp();
        if (lane < nbox)
          tma_load_4d(smem + L::K + s * TILE + lane * box * HD, &tmk, &bar[B_KF + s], 0, bnsd ? off : hk, bnsd ? hk : off, pg);
        nk = j + 1;
        if (j >= NST) ok = __all_sync(0xffffffffu, mbar_wait(&bar[B_VE + s], ((j / NST) - 1) & 1, abort_flag, p.status, 214));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&bar[B_VF + s], TILE);
        __syncwarp();
        if (lane < nbox)
          tma_load_4d(smem + L::V + s * TILE + lane * box * HD, &tmv, &bar[B_VF + s], 0, bnsd ? off : hk, bnsd ? hk : off, pg);
        pg = nxt;
      }
    } while (ok && run.next(p));
    if (*abort_flag) {
      // let the issued loads land before the CTA can leave
      for (int t = max(0, nk - NST); t < nk; ++t) mbar_drain(&bar[B_KF + t % NST], (t / NST) & 1);
      for (int t = max(0, j - NST); t < j; ++t) mbar_drain(&bar[B_VF + t % NST], (t / NST) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------- MMAs
    if (lane == 0) {
      constexpr uint32_t id_qk = FP8 ? make_idesc(kAccF32, kFmtE4M3, kFmtE4M3, 0, 0, N, 128)
                                     : make_idesc(kAccS32, kFmtS8, kFmtS8, 0, 0, N, 128);
      constexpr uint32_t id_pv = FP8 ? make_idesc(kAccF32, kFmtE4M3, kFmtE4M3, 1, 0, NO, 128)
                                     : make_idesc(kAccS32, kFmtS8, kFmtU8, 1, 0, NO, 128);
      const uint32_t sQ = smem_u32(smem + L::Q), sK = smem_u32(smem + L::K), sV = smem_u32(smem + L::V), sP = smem_u32(smem + L::P);
      auto mma = [](uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
        if (FP8)
          mma_f8f6f4(d, a, b, id, acc);
        else
          mma_i8(d, a, b, id, acc);
      };
      auto pv = [&](int j) {  // O^T of tile j
        const int s = j % NST, bb = j & 1;
        if (!mbar_wait(&bar[B_PF + bb], (j >> 1) & 1, abort_flag, p.status, 215)) return false;
        if (!mbar_wait(&bar[B_VF + s], (j / NST) & 1, abort_flag, p.status, 216)) return false;
        if (j >= 2 && !mbar_wait(&bar[B_OE + bb], ((j >> 1) - 1) & 1, abort_flag, p.status, 217)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < HD / 32; ++kk)  // 128 keys, or 64 of both halves (the second operand atom: 64 rows on)
          mma(tbase + L::TO + bb * NO, make_sdesc(sV + s * TILE + kk * 32 * HD, 64 * HD, SBO, SW),
              make_sdesc(sP + (L::NP == 2 ? bb : 0) * N * 128 + kk * 32, 16, SBO, SW), id_pv, kk > 0);
        mma_commit(&bar[B_VE + s]);
        mma_commit(&bar[B_OF + bb]);
        return true;
      };
      int j = 0, piece = 0;
      bool ok = true;
      do {
        if (run.t0 < run.t1) ok = mbar_wait(&bar[B_Q], piece++ & 1, abort_flag, p.status, 218);
        for (int t = run.t0; t < run.t1 && ok; ++t, ++j) {
          const int s = j % NST, bb = j % NS;
          ok = mbar_wait(&bar[B_KF + s], (j / NST) & 1, abort_flag, p.status, 219) &&
               (j < NS || mbar_wait(&bar[B_SE + bb], (j / NS - 1) & 1, abort_flag, p.status, 220));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < HD / 32; ++kk)
            mma(tbase + bb * N, make_sdesc(sK + s * TILE + kk * 32, 16, SBO, SW), make_sdesc(sQ + kk * 32, 16, SBO, SW),
                id_qk, kk > 0);
          mma_commit(&bar[B_KE + s]);
          mma_commit(&bar[B_SF + bb]);
          // the piece's first tile has no P V of its own piece before it
          if (t > run.t0) ok = pv(j - 1);
        }
        if (ok && run.t0 < run.t1) ok = pv(j - 1);
      } while (ok && run.next(p));
      mma_commit(&bar[B_FIN]);
      mbar_drain(&bar[B_FIN], 0);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax
    const int wg = warp & 3;          // TMEM lanes 32 wg .. + 31
    const int i = wg * 32 + lane;     // key of S^T, row of O^T: dim i, or (D = 64) dim i % 64 over half i / 64 of the keys
    const int half = HD == 128 ? 0 : wg >> 1;
    const uint32_t loff = (uint32_t)(wg * 32) << 16;
    float* red = reinterpret_cast<float*>(smem + L::RED);
    float* sums = reinterpret_cast<float*>(smem + L::SUM);
    float* halves = reinterpret_cast<float*>(smem + L::P);  // at a piece's end, when no P is in use
    float* rowf = reinterpret_cast<float*>(smem + L::ROW);
    int* rowl = reinterpret_cast<int*>(smem + L::ROW) + R;
    int* nan_key = reinterpret_cast<int*>(smem + L::NAN_KEY);
    float4* units = reinterpret_cast<float4*>(smem + L::UNIT);
    float* alb = reinterpret_cast<float*>(units + 4 * R);
    auto wait = [&](int which, int phase, int where) {
      return __all_sync(0xffffffffu, mbar_wait(&bar[which], phase & 1, abort_flag, p.status, where));
    };
    int j = 0, piece = 0;
    bool ok = true;
    do {
      const Seq s = run.it.s;
      const int hk = run.it.hk, b = run.it.b, rows = s.m * p.G;
      // o is in units of 2^(top - down) (l too, in the per-head modes), top the running maximum, down whole.  Lane r of every
      // warp keeps row r's; in the per-token modes lane R + r does, and lane r the maximum of x, which is l's unit.
      float top = -INFINITY, down = 0.0f;
      const bool unit_lane = !TOK || lane >= R;
      float l_run[R], o[R];
#pragma unroll
      for (int r = 0; r < R; ++r) l_run[r] = o[r] = 0.0f;
      if (run.t0 < run.t1) {
        // ---- Q digits: D / 16 lanes a row, 16 values each
        constexpr int LPR = HD / 16;
        for (int idx = i; idx - lane < R * LPR; idx += 128) {
          const int r = idx / LPR, c = idx % LPR, ii = r / p.G;
          const bool live = r < R && r < rows && q_row_ok(p, s, hk, r, 174);
          const uint4* src = reinterpret_cast<const uint4*>(p.q + (long long)(s.q0 + ii) * p.q_stride +
                                                            (long long)(hk * p.G + r - ii * p.G) * HD + c * 16);
          uint4 raw[2];
          raw[0] = live ? __ldg(src) : make_uint4(0, 0, 0, 0);
          raw[1] = live ? __ldg(src + 1) : make_uint4(0, 0, 0, 0);
          const uint32_t* w = &raw[0].x;
          float m = 0.0f;
          bool bad_value = false;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float x0 = fabsf(__uint_as_float(w[e] << 16)), x1 = fabsf(__uint_as_float(w[e] & 0xFFFF0000u));
            bad_value = bad_value || x0 != x0 || x1 != x1;
            m = fmaxf(m, fmaxf(x0, x1));
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
            const uint32_t ww = w[e >> 1];
            const float x = __uint_as_float((e & 1) ? ww & 0xFFFF0000u : ww << 16);
            q_digits<FP8>(sc == 0.0f ? 0.0f : x, sc, d);
#pragma unroll
            for (int k = 0; k < 3; ++k) dw[k][e >> 2] |= d[k] << (8 * (e & 3));
          }
          if (r >= R) continue;
#pragma unroll
          for (int k = 0; k < 3; ++k)
            *reinterpret_cast<uint4*>(smem + L::Q + swz(k * R + r, c)) =
                make_uint4(dw[k][0], dw[k][1], dw[k][2], dw[k][3]);
          if (c == 0) {
            rowf[r] = p.scale_log2 * inv * (TOK ? 1.0f : finite_or_nan(__ldg(p.c.ks + hk)));
            rowl[r] = row_limit(p, s, r);
          }
        }
        if (FP8) nan_key[i] = 0x7FFFFFFF;
        fence_async_smem();
        mbar_arrive(&bar[B_Q]);
        ok = wait(B_Q, piece, 221);
      }
      const int lim_lo = p.causal ? s.n - s.m : s.n - 1;  // every row sees the keys up to here
      // per-token scales of this thread's key, one tile ahead; its page two tiles ahead
      float sk = 0.0f, sv = 0.0f, sk_n = 0.0f, sv_n = 0.0f;
      int bad_key = 0x7FFFFFFF;  // this thread's lowest key whose V scale is no number
      int pg_n = -1;
      auto load_page = [&](int t) {
        const int key = t * TK + i;
        return key < s.n && t < run.t1 ? page_of(p.bt, p.c, b, key, p.status, 212) : -1;
      };
      auto load_scales = [&](int t, int pg, float& k, float& v) {
        const long long si = p.c.scale(pg, hk, (t * TK + i) & p.c.page_mask);
        if (pg >= 0 && !p.c.holds_scale(si, 175)) pg = -1;
        k = pg >= 0 ? __ldg(p.c.ks + si) : 0.0f;
        v = pg >= 0 ? __ldg(p.c.vs + si) : 0.0f;
      };
      if (TOK && run.t0 < run.t1) {
        load_scales(run.t0, load_page(run.t0), sk_n, sv_n);
        pg_n = load_page(run.t0 + 1);
      }
      for (int t = run.t0; t < run.t1 && ok; ++t, ++j) {
        const int bb = j & 1, sb = j % NS;
        const int key = t * TK + i;
        const bool masked = t * TK + TK - 1 > lim_lo;
        if (TOK) {
          sk = sk_n;
          sv = sv_n;
          if (t + 1 < run.t1) {
            load_scales(t + 1, pg_n, sk_n, sv_n);
            pg_n = load_page(t + 2);
          }
        }
        if (FP8 && masked) {
          // V codes that not every row sees must be finite: rows past the end are cleared, and NaN codes
          if (!(ok = wait(B_VF + j % NST, j / NST, 222))) break;
          clear_nans<HD>(smem + L::V + (j % NST) * TILE, i, key >= s.n, key, nan_key);
        }
        if (!(ok = wait(B_SF + sb, j / NS, 223))) break;
        tc_fence_after();
        uint32_t a[N];
#pragma unroll
        for (int c = 0; c < N / 16; ++c) tmem_ld16(tbase + sb * N + c * 16 + loff, *reinterpret_cast<uint32_t(*)[16]>(&a[16 * c]));
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[B_SE + sb]);
        // ---- scores and the rows' maxima
        const bool v_bad = TOK && !(fabsf(sv) < INFINITY);  // a NaN or infinite V scale: rows that see the key are NaN
        bad_key = min(bad_key, v_bad ? key : 0x7FFFFFFF);
        if (TOK) sk = finite_or_nan(sk);
        float x[R];
        const float lsv = TOK ? log2f(v_bad ? 0.0f : sv) : 0.0f;
        float mx = -INFINITY;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          x[r] = join_digits<FP8>(a[r], a[R + r], a[2 * R + r]) * rowf[r];
          if (TOK) x[r] *= sk;
          if (masked && key > rowl[r]) x[r] = -INFINITY;
          const float m = warp_max(x[r]);
          if (lane == r) mx = m;
          if (TOK) {
            const float m2 = warp_max(x[r] + lsv);
            if (lane == R + r) mx = m2;
          }
        }
        if (lane < JOBS) red[(bb * 4 + wg) * JOBS + lane] = mx;
        mbar_arrive(&bar[B_RED + bb]);
        if (!(ok = wait(B_RED + bb, j >> 1, 224))) break;
        // ---- p into the sums, the digits of w = s_v 2^(x - unit)
        if (L::NP == 1 || j >= 2) {
          // the P buffer is free once the P V that read it is done
          const int jp = L::NP == 1 ? j - 1 : j - 2;
          if (jp >= 0 && !(ok = wait(B_OF + (jp & 1), jp >> 1, 225))) break;
        }
        uint8_t* sp = smem + L::P + (L::NP == 2 ? bb : 0) * N * 128;
        if (lane < JOBS) {
          // the tile's unit: the largest weight so far, or the last of its halves that is not below the tile's own largest
          const float* rd = red + bb * 4 * JOBS + lane;
          const float c = fmaxf(fmaxf(fmaxf(rd[0], rd[JOBS]), fmaxf(rd[2 * JOBS], rd[3 * JOBS])), -INFINITY);
          const float mx_new = fmaxf(top, c);
          const float d = unit_lane ? fminf(floorf(mx_new - c), kFall) : 0.0f;
          const bool none = mx_new == -INFINITY;
          const float base = none ? 0.0f : mx_new - d;
          const float al = none ? 0.0f : attn::ex2((top - mx_new) + (d - down));  // a whole power while the maximum stays; 0 from -inf
          top = mx_new;
          down = d;
          if (unit_lane) alb[(bb * 4 + wg) * R + lane % R] = al;
          reinterpret_cast<float2*>(units + wg * R + lane % R)[TOK && !unit_lane] = make_float2(base, al);
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float4 u = units[wg * R + r];
          float w = attn::ex2((TOK ? x[r] + lsv : x[r]) - u.x);
          if (TOK) {
            l_run[r] = l_run[r] * u.w + attn::ex2(x[r] - u.z);
            // not p s_v: p may vanish where s_v is large; a masked key, or one whose s_v is no number, has weight 0 here
            if (!(x[r] > -INFINITY) || v_bad) w = 0.0f;
          } else {
            l_run[r] = l_run[r] * u.y + w;
          }
          uint32_t d[3];
          p_digits<FP8>(w, d);
#pragma unroll
          for (int k = 0; k < 3; ++k) sp[swz((HD == 128 ? 0 : (i >> 6) * N) + k * R + r, (HD == 128 ? i : i & 63) >> 4) + (i & 15)] = (uint8_t)d[k];
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[B_PF + bb]);
        // ---- O^T of the tile before
        if (t > run.t0) {
          const int jb = (j - 1) & 1;
          if (!(ok = wait(B_OF + jb, (j - 1) >> 1, 226))) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < N / 16; ++c)
            tmem_ld16(tbase + L::TO + jb * NO + half * N + c * 16 + loff, *reinterpret_cast<uint32_t(*)[16]>(&a[16 * c]));
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar[B_OE + jb]);
#pragma unroll
          for (int r = 0; r < R; ++r) o[r] = o[r] * alb[(jb * 4 + wg) * R + r] + join_digits<FP8>(a[r], a[R + r], a[2 * R + r]);
        }
      }
      if (!ok) break;
      // ---- the piece's end: its last O^T, the row sums, the result
      if (run.t0 < run.t1) {
        const int jb = (j - 1) & 1;
        if (!(ok = wait(B_OF + jb, (j - 1) >> 1, 227))) break;
        tc_fence_after();
        uint32_t a[N];
#pragma unroll
        for (int c = 0; c < N / 16; ++c)
          tmem_ld16(tbase + L::TO + jb * NO + half * N + c * 16 + loff, *reinterpret_cast<uint32_t(*)[16]>(&a[16 * c]));
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar[B_OE + jb]);
        int lim[R];
        if (TOK) {
          bad_key = __reduce_min_sync(0xffffffffu, bad_key);
          if (lane == 0) nan_key[128 + wg] = bad_key;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          o[r] = o[r] * alb[(jb * 4 + wg) * R + r] + join_digits<FP8>(a[r], a[R + r], a[2 * R + r]);
          // every key's thread has noted its NaN codes before the last tile's maxima
          if (FP8 && nan_key[i] <= rowl[r]) o[r] = __uint_as_float(0x7FC00000u);
          if (TOK) lim[r] = rowl[r];  // (read before B_SUM: the next piece's limits come after it)
          float l = l_run[r];
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
          if (lane == 0) sums[wg * R + r] = l;
          if (HD == 64 && half) halves[r * 64 + (i & 63)] = o[r];
        }
        mbar_arrive(&bar[B_SUM]);
        if (!(ok = wait(B_SUM, piece, 228))) break;
        ++piece;
        if (TOK) bad_key = min(min(nan_key[128], nan_key[129]), min(nan_key[130], nan_key[131]));
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if (TOK && bad_key <= lim[r]) o[r] = __uint_as_float(0x7FC00000u);
          if (HD == 64 && !half) o[r] += halves[r * 64 + i];
          l_run[r] = (sums[r] + sums[R + r]) + (sums[2 * R + r] + sums[3 * R + r]);
        }
      }
      // (mv, o's factor) and, in the per-token modes, (m, 1): o and the per-head l in units of 2^mv
      if (lane < JOBS)
        reinterpret_cast<float2*>(units + wg * R + lane % R)[TOK && !unit_lane] =
            make_float2(top, top == -INFINITY ? 1.0f : attn::ex2(-down));
      __syncwarp();
      const bool whole = run.u == run.it.first && run.it.first + run.it.nt <= run.u1;
      const int slot = 2 * blockIdx.x + (run.u == run.u0 ? 0 : 1);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r >= rows || half) break;
        const float4 u = units[wg * R + r];
        const float val = o[r] * u.y * kPUnit<FP8>, m = TOK ? u.z : u.x, l = TOK ? l_run[r] : l_run[r] * u.y;
        if (whole) {
          const int ii = r / p.G;
          const long long row = (long long)(s.q0 + ii) * p.Hq + hk * p.G + r - ii * p.G;
          if (!q_row_ok(p, s, hk, r, 176)) continue;
          p.out[row * HD + i] = __float2bfloat16(val * row_factor(p, hk, l, m, u.x));
          if (i == 0 && p.lse) p.lse[row] = row_lse(l, m);
        } else if (in_bounds(slot < 2 * (int)gridDim.x && r < DPL::RB, 177)) {
          p.part_o[((long long)slot * DPL::RB + r) * HD + i] = val;
          if (i == 0) p.part_ml[(long long)slot * DPL::RB + r] = make_float4(m, l, u.x, 0.0f);
        }
      }
    } while (ok && run.next(p));
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, L::COLS);
  }
}

template <int D, bool FP8, bool TOK, int R>
cudaError_t launch_r(const CUtensorMap& mk, const CUtensorMap& mv, const AttnP& p, int grid, cudaStream_t s) {
  auto kern = paged_decode_kernel<D, FP8, TOK, R>;
  cudaError_t e;
  if ((e = set_smem_limit(reinterpret_cast<const void*>(kern), DL<D, R>::ALLOC)) != cudaSuccess) return e;
  kern<<<grid, DT, DL<D, R>::ALLOC, s>>>(mk, mv, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_combine<DPL, D>(p, grid, s);
}

template <int D, bool FP8, bool TOK>
cudaError_t launch_rows(const CUtensorMap& mk, const CUtensorMap& mv, const AttnP& p, int rows, int grid, cudaStream_t s) {
  if (rows <= 4) return launch_r<D, FP8, TOK, 4>(mk, mv, p, grid, s);
  if (rows <= 8) return launch_r<D, FP8, TOK, 8>(mk, mv, p, grid, s);
  return launch_r<D, FP8, TOK, 16>(mk, mv, p, grid, s);
}

template <int D>
cudaError_t launch_mode(const CUtensorMap& mk, const CUtensorMap& mv, const AttnP& p, int mode, int rows, int grid,
                        cudaStream_t s) {
  switch (mode) {
    case FA_MODE_INT8_PER_HEAD: return launch_rows<D, false, false>(mk, mv, p, rows, grid, s);
    case FA_MODE_FP8_PER_HEAD: return launch_rows<D, true, false>(mk, mv, p, rows, grid, s);
    case FA_MODE_INT8_PER_TOKEN: return launch_rows<D, false, true>(mk, mv, p, rows, grid, s);
    case FA_MODE_FP8_PER_TOKEN: return launch_rows<D, true, true>(mk, mv, p, rows, grid, s);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace

size_t paged_decode_ws(int D) { return plan_ws<DPL>(D, 2 * sm_count()); }

cudaError_t launch_paged_decode(const PagedAttnArgs& a, int rows, void* ws, cudaStream_t s) {
  AttnP p = paged_attn_params(a);
  if (const cudaError_t be = bounds_attach(); be != cudaSuccess) return be;
  const int D = a.q->D, grid = 2 * sm_count();
  plan_carve<DPL>(p, ws, D, grid);
  CUtensorMap mk, mv;
  cudaError_t e;
  if ((e = make_page_map(&mk, a.cache->k_codes, *a.cache, TK, true)) != cudaSuccess) return e;
  if ((e = make_page_map(&mv, a.cache->v_codes, *a.cache, TK, true)) != cudaSuccess) return e;
  return D == 128 ? launch_mode<128>(mk, mv, p, a.cache->mode, rows, grid, s)
                  : launch_mode<64>(mk, mv, p, a.cache->mode, rows, grid, s);
}

}  // namespace faq
