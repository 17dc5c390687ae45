// paged_chunk.cu -- attention of many query rows per kv head (chunks of prompts, drafts) over a paged
// 8-bit cache, on the tensor cores' 16-bit kind.
//
// Long chunks are bound by the two products, 4 D flops per (row, key).  One CTA owns a block of 256 query rows
// of one kv head (new tokens x the group's heads, so that every row of the block reads the same keys) as two
// 128-row tiles, A and B, with one S and one O accumulator each in TMEM.  The MMA thread alternates the tiles
//   QK_A(0) QK_B(0) | PV_A(0) QK_A(1) PV_B(0) QK_B(1) | PV_A(1) ...
// so that the tensor pipe works on one tile while the other's softmax runs.  Blocks of at most 128 rows have
// both tiles hold the same rows, A for the even and B for the odd key tiles: the two chains overlap as before,
// and the merge of the two is done on the accumulators at the end.
//
// Codes are exact in fp16, and so are Q's rows scaled by powers of two (but for values 2^-29 below the row's
// largest).  TMA brings the codes page by page to a staging ring, four warps convert them and write the swizzled
// MMA operands (about 2000 warp instructions a tile, which fit beside the softmax of 256 rows: the cache needs
// no conversion pass of its own).  P (fp16, up to 2^15) overwrites S in TMEM and is the A operand of
// P V.  Scales: per head at the ends.  Per token: s_k on the scores, s_v on P; a row's factors are held against
// the largest of them, whatever the scales' range: w_j = s_v(j) 2^(x_j - mv), mv the running maximum of
// x + log2 s_v, and the sum of p is that of 2^(x_j - mv).
// Work is shared out as paged_sched.cuh says: a causal block counts the key tiles it sees.
// Measured: two chunks of up to 1500 tokens behind up to 32768, 32 / 8 heads of 128: int8 per head 1.60 ms (810 TFLOP/s,
// 50 % of the library GEMM's rate), fp8 per head 1.58, fp8 per token 3.06 ms (426 TFLOP/s; 11.2 ms with warp-level MMAs).
// Per head, a step of both tiles takes about 4000 cycles where the exponentials alone take 2048: the chain from one
// product through a softmax to the next.  Per token the softmax is the longer side (3100 to 4500 cycles): both scales of
// every key come from shared memory for every row, and their latency shows with two warps to a scheduler.
#include "paged_sched.cuh"

namespace faq {
namespace {
using namespace paged;

constexpr int BM = 128;       // rows per tile
constexpr int TN = 128;       // keys per tile
constexpr int NSG = 2;        // K and V stages
constexpr int NSC = 3;        // scale stages (per-token modes)
constexpr int CT = 512;       // warpgroups: pieces + loads, MMAs; converters; softmax A; softmax B
constexpr int NU = 3;         // load units in the staging ring (one is converted, two are on their way)
constexpr int R0 = 88, RC = 88, RS = 168;  // the warpgroups' registers
static_assert(128 * (R0 + RC + 2 * RS) <= CT * 128, "register split exceeds the launch");
static_assert(R0 <= 128 && RC <= 128 && RS >= 128, "launched with 128 registers a thread: the first two warpgroups give some back");
constexpr float kShift = 7.0f;  // P is held as p 2^7: fp16 keeps 11 bits of it down to 2^-21, and the running maximum may lag by 2^8
// V scales below this are brought up to it, and their codes (exact otherwise) scaled down: 2^(x - mv) stays finite
constexpr float kMinScale = 0x1p-90f;

using CPL = Plan<TN, 2 * BM, 17, 0x7FFFFFFF, true>;

template <int D>
struct CL {
  static constexpr int NA = D / 64;                    // 128-byte atoms per fp16 row
  static constexpr uint32_t ATOM = 128 * 128;          // bytes of one atom of 128 rows
  static constexpr uint32_t TILE = NA * ATOM;
  static constexpr uint32_t Q = 0;                     // two tiles
  static constexpr uint32_t K = Q + 2 * TILE;          // NSG stages
  static constexpr uint32_t V = K + NSG * TILE;        // NSG stages
  static constexpr uint32_t SC = V + NSG * TILE;       // NSC x ([128] s_k, [128] s_v, [128] factors of V codes, [4] warps that have one, [4] largest s_v)
  static constexpr uint32_t SCB = 3 * TN * 4 + 64;
  static constexpr uint32_t ML = SC + NSC * SCB;       // [128] (m, l) of tile B (blocks of at most 128 rows)
  static constexpr uint32_t PC = ML + BM * 8;          // NPC pieces
  static constexpr uint32_t NAN_KEY = PC + 4 * 64;     // NPC x ([128] per dim, [4]: of the V scales): the lowest key that is no number
  static constexpr uint32_t BAR = NAN_KEY + 4 * 132 * 4;
  static constexpr int UR = 8192 / D;                  // keys of a load unit
  static constexpr int UT = TN / UR;                   // units of a tile of one operand
  static constexpr uint32_t UNIT = UR * D;             // raw codes: 8 KB
  static constexpr uint32_t RAW = (BAR + 384 + 127) & ~127u;  // NU units on their way
  static constexpr uint32_t TOTAL = RAW + NU * UNIT;
  static constexpr uint32_t ALLOC = TOTAL + 1024;
  static_assert(ALLOC <= 227 * 1024, "shared memory per CTA");
  static constexpr uint32_t TS0 = 0, TO0 = 256, TO1 = 256 + D;  // TMEM columns: S_A, S_B at 0, 128
};

enum {
  C_Q = 0,             // Q tiles written, and O free
  C_KF = 1,            // [NSG]
  C_KE = C_KF + NSG,
  C_VF = C_KE + NSG,
  C_VE = C_VF + NSG,
  C_SF = C_VE + NSG,   // [2] S_A / S_B done
  C_PF = C_SF + 2,     // [2] P stored
  C_PV = C_PF + 2,     // [2] P V done
  C_SCF = C_PV + 2,    // [NSC]
  C_SCE = C_SCF + NSC, // [NSC]
  C_ML = C_SCE + NSC,  // tile B's (m, l) written
  C_FIN = C_ML + 1,
  C_PCF = C_FIN + 1,   // [NPC] piece written
  C_PCE = C_PCF + 4,   // [NPC] piece done with
  C_RF = C_PCE + 4,    // [NU] staged unit landed
  C_RE = C_RF + NU,    // [NU] staging slot free
  C_COUNT = C_RE + NU
};
static_assert(C_COUNT * 8 + 8 <= 384, "barriers fit their region");

template <int R>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// Four floats from shared memory, read here and now: the compiler would otherwise keep a tile's scales in
// registers from one use to the next, and spill the scores for them.
__device__ __forceinline__ float4 lds4(const float* p) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(smem_u32(p)) : "memory");
  return v;
}

template <bool V>
struct Bool {
  static constexpr bool value = V;
};

// One piece of the CTA's run: key tiles [t0, t1) of a row block.  Warp 0 walks the run and leaves the
// pieces in a ring in shared memory, so that the other warps spend no registers on the walk.
struct Piece {
  int b, hk, q0, m, n;  // the sequence and kv head
  int row0;             // the block's first row
  int t0, t1_last;      // (t1 << 1) + (no piece follows): one word, so that a reader that has t1 has the flag
  int kt[2];            // key tiles that the rows of tile A / B see
  int dual;             // both tiles hold the block's rows (at most 128), and share the key tiles out
  int whole;            // the piece is the whole item
  int slot;             // of its partial result
  int pad[3];
};
constexpr int NPC = 4;  // pieces in the ring

// Does tile x (A or B) have key tile t, and how many tiles has it?
__device__ __forceinline__ bool has_tile(int t0, int t1, int kt, int dual, int x, int t) {
  return t >= t0 && t < t1 && t < kt && (!dual || ((t - t0) & 1) == x);
}
__device__ __forceinline__ int tile_count(int t0, int t1, int kt, int dual, int x) {
  const int n = min(t1, kt) - t0;
  return n <= 0 ? 0 : dual ? (n + 1 - x) / 2 : n;
}

template <typename PL>
__device__ __forceinline__ Piece make_piece(const AttnP& p, const Item& it, long long u, long long u0, long long u1) {
  Piece o = {};
  const Seq& s = it.s;
  o.b = it.b;
  o.hk = it.hk;
  o.q0 = s.q0;
  o.m = s.m;
  o.n = s.n;
  o.row0 = it.rb * PL::RB;
  const int rows = min(s.m * p.G - o.row0, PL::RB);
  o.dual = rows <= BM;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int end_row = o.row0 + (o.dual || x ? rows : BM) - 1;
    const int end = p.causal ? min(s.n, s.n - s.m + end_row / p.G + 1) : s.n;
    o.kt[x] = end > 0 ? (end + TN - 1) / TN : 0;
  }
  const long long item_end = it.first + it.nt, e = item_end < u1 ? item_end : u1;
  o.t0 = (int)(u - it.first);
  o.t1_last = max(o.t0, min((int)(e - it.first), max(o.kt[0], o.kt[1]))) * 2 + (item_end >= u1);
  o.whole = u == it.first && item_end <= u1;
  o.slot = 2 * blockIdx.x + (u == u0 ? 0 : 1);
  return o;
}

template <int D, bool FP8, bool TOK>
__global__ void __launch_bounds__(CT, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const AttnP p) {
  using L = CL<D>;
  using PL = CPL;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + C_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const long long total = total_units<PL>(p, lane);
  const int runs = run_count(total, gridDim.x);
  if ((int)blockIdx.x >= runs) return;
  if (tid == 0) {
    mbar_init(&bar[C_Q], 256);
    for (int i = 0; i < NSG; ++i) {
      mbar_init(&bar[C_KF + i], 4);
      mbar_init(&bar[C_KE + i], 1);
      mbar_init(&bar[C_VF + i], 4);
      mbar_init(&bar[C_VE + i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar[C_SF + i], 1);
      mbar_init(&bar[C_PF + i], 4);
      mbar_init(&bar[C_PV + i], 1);
    }
    for (int i = 0; i < NSC; ++i) {
      mbar_init(&bar[C_SCF + i], 4);
      mbar_init(&bar[C_SCE + i], 8);
    }
    mbar_init(&bar[C_ML], 128);
    mbar_init(&bar[C_FIN], 1);
    for (int i = 0; i < NPC; ++i) {
      mbar_init(&bar[C_PCF + i], 1);
      mbar_init(&bar[C_PCE + i], 13);  // the MMA thread, four converter warps, eight softmax warps
    }
    for (int i = 0; i < NU; ++i) {
      mbar_init(&bar[C_RF + i], 1);
      mbar_init(&bar[C_RE + i], 4);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  let_next_start();
  auto wait = [&](int which, int phase, int where) { return mbar_wait(&bar[which], phase & 1, abort_flag, p.status, where); };
  auto wwait = [&](int which, int phase, int where) { return __all_sync(0xffffffffu, wait(which, phase, where)); };
  Piece* pieces = reinterpret_cast<Piece*>(smem + L::PC);
  int* nan_keys = reinterpret_cast<int*>(smem + L::NAN_KEY);

  if (warp < 4) {
    regs_dec<R0>();
    if (warp == 0) {
      // ------------------------------------------ the run's pieces, and their loads
      const long long u0 = run_start(total, blockIdx.x, runs), u1 = run_start(total, blockIdx.x + 1, runs);
      Item it = find_item<PL>(p, u0, lane);
      const int box = min(L::UR, p.c.page_mask + 1), nbox = L::UR / box;  // lane l < nbox loads a unit's l-th box
      const bool bnsd = p.c.bnsd;
      if (lane == 0) {
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
      }
      long long u = u0;
      int g = 0;  // units issued
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (k >= NPC && !(ok = wwait(C_PCE + k % NPC, k / NPC - 1, 240))) break;
        Piece pc = make_piece<PL>(p, it, u, u0, u1);
        u = it.first + it.nt;
        // (no next item cannot be while the lengths stay as they were counted)
        if (!(pc.t1_last & 1) && !next_item<PL>(p, it)) pc.t1_last |= 1;
        const int t1 = pc.t1_last >> 1;
        if (FP8 || TOK)
          for (int d = lane; d < 132; d += 32) nan_keys[(k % NPC) * 132 + d] = 0x7FFFFFFF;
        __syncwarp();
        if (lane == 0) {
          pieces[k % NPC] = pc;
          mbar_arrive(&bar[C_PCF + k % NPC]);
        }
        // lane l < 8: the page of a tile's l-th 16 keys; past the end, or not a page: one past the pool, read as zeros
        auto page = [&](int t) {
          const int key = t * TN + (lane & 7) * 16;
          int pg = p.c.pages;
          if (t < t1 && key < pc.n) {
            pg = page_of(p.bt, p.c, pc.b, key, p.status, 212);
            if (pg < 0) pg = p.c.pages;
          }
          return pg;
        };
        int pages = pc.t0 < t1 ? page(pc.t0) : 0;
        for (int t = pc.t0; t < t1 && ok; ++t) {
          const int next = page(t + 1);  // its latency passes while this tile's units wait
#pragma unroll 1
          for (int q = 0; q < 2 * L::UT; ++q, ++g) {
            const int sl = g % NU, row = (q % L::UT) * L::UR + lane * box;  // this lane's box
            const int pg = __shfl_sync(0xffffffffu, pages, (row >> 4) & 7);
            if (g >= NU && !(ok = wwait(C_RE + sl, g / NU - 1, 238))) break;
            if (lane == 0) mbar_arrive_expect_tx(&bar[C_RF + sl], L::UNIT);
            __syncwarp();
            if (lane < nbox) {
              const int off = (t * TN + row) & p.c.page_mask;
              tma_load_4d(smem + L::RAW + sl * L::UNIT + lane * box * D, q < L::UT ? &tmk : &tmv, &bar[C_RF + sl], 0,
                          bnsd ? off : pc.hk, bnsd ? pc.hk : off, pg);
            }
          }
          pages = next;
        }
        if (pc.t1_last & 1) break;
      }
      if (*abort_flag)  // let the issued loads land before the CTA can leave
        for (int t = max(0, g - NU); t < g; ++t) mbar_drain(&bar[C_RF + t % NU], (t / NU) & 1);
      __syncwarp();
    } else if (warp == 1) {
      // ----------------------------------------------------------------- MMAs
      if (lane == 0) {
        constexpr uint32_t id_qk = make_idesc(kAccF32, kFmtF16, kFmtF16, 0, 0, TN, BM);
        constexpr uint32_t id_pv = make_idesc(kAccF32, kFmtF16, kFmtF16, 0, 1, D, BM);
        const uint64_t dq = make_sdesc(smem_u32(smem + L::Q), 16, 1024, kSwz128);
        const uint64_t dk = make_sdesc(smem_u32(smem + L::K), 16, 1024, kSwz128);
        const uint64_t dv = make_sdesc(smem_u32(smem + L::V), L::ATOM, 1024, kSwz128);
        const uint32_t k_hi = (uint32_t)(dk >> 32), v_hi = (uint32_t)(dv >> 32);
        int base = 0, nq = 0;   // tiles of the pieces before this one, pieces with tiles
        int done[2] = {0, 0};   // tiles of A / B so far
        bool ok = true, more = true;
        for (int k = 0; ok && more; ++k) {
          if (!(ok = wait(C_PCF + k % NPC, k / NPC, 239))) break;
          const Piece& pc = pieces[k % NPC];
          const int t0 = pc.t0, t1 = pc.t1_last >> 1, kt0 = pc.kt[0], kt1 = pc.kt[1], dual = pc.dual;
          more = !(pc.t1_last & 1);
          if (t0 >= t1) {
            mbar_arrive(&bar[C_PCE + k % NPC]);
            continue;
          }
          if (!(ok = wait(C_Q, nq++, 241))) break;
          tc_fence_after();
          const int step = dual ? 2 : 1;
          auto has = [&](int x, int t) { return has_tile(t0, t1, x ? kt1 : kt0, dual, x, t); };
          auto qk = [&](int x, int t) {
            const int j = base + t - t0;
            if (!wait(C_KF + j % NSG, j / NSG, 242)) return false;
            tc_fence_after();
            const uint32_t ql = (uint32_t)dq + x * (L::TILE >> 4), kl = (uint32_t)dk + (j % NSG) * (L::TILE >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk / 4) * L::ATOM + (kk % 4) * 32) >> 4;
              mma_f16_lh(tbase + L::TS0 + x * 128, ql + off, k_hi, kl + off, k_hi, id_qk, kk > 0);
            }
            mma_commit(&bar[C_SF + x]);
            if (x == 1 || !has(1, t)) mma_commit(&bar[C_KE + j % NSG]);  // the tile's last reader
            return true;
          };
          auto pv = [&](int x, int t) {
            const int j = base + t - t0;
            if (!mbar_wait_spin(&bar[C_PF + x], done[x] & 1, abort_flag, p.status, 243)) return false;
            if (!wait(C_VF + j % NSG, j / NSG, 244)) return false;
            tc_fence_after();
            const uint32_t vl = (uint32_t)dv + (j % NSG) * (L::TILE >> 4);
#pragma unroll
            for (int ks = 0; ks < TN / 16; ++ks)
              mma_f16_ts_lh(tbase + (x ? L::TO1 : L::TO0), tbase + L::TS0 + x * 128 + ks * 8, vl + ((ks * 16 * 128) >> 4), v_hi,
                            id_pv, (t >= t0 + step || ks > 0) ? 1u : 0u);
            mma_commit(&bar[C_PV + x]);
            if (x == 1 || !has(1, t)) mma_commit(&bar[C_VE + j % NSG]);
            ++done[x];
            return true;
          };
          // step r: P V of the tiles' r-th key tiles, each followed by its next Q K^T; r = -1: the first Q K^T
#pragma unroll 1
          for (int r = -step; ok && t0 + r < t1; r += step) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int t = t0 + r + (dual ? x : 0);
              if (ok && r >= 0 && has(x, t)) ok = pv(x, t);
              if (ok && has(x, t + step)) ok = qk(x, t + step);
            }
          }
          base += t1 - t0;
          mbar_arrive(&bar[C_PCE + k % NPC]);
        }
        mma_commit(&bar[C_FIN]);
        mbar_drain(&bar[C_FIN], 0);
      }
      __syncwarp();
    }
  } else if (warp < 8) {
    regs_dec<RC>();
    // ------------------------------------------- codes -> fp16 operand tiles
    // A tile comes in 2 UT units, K first.  Thread: chunk c (16 codes, 32 bytes of fp16; D / 16 lanes a row) of every
    // RPP-th row.  Its key's scales come a tile ahead.
    constexpr int UT = L::UT, UR = L::UR;
    constexpr int LPR = D / 16, RPP = 128 / LPR, NP = UR / RPP;  // lanes per row, rows per pass, passes per unit
    const int ct = tid - 128, c = ct % LPR, r0 = ct / LPR;
    // the two 16-byte chunks of a row: lanes of the row's halves (D = 64: of odd rows) write them in turn, so that
    // eight lanes cover the eight chunk positions of the banks
    const int odd = (D == 128 ? c >> 2 : r0) & 1;
    const uint32_t at0 = (c >> 2) * L::ATOM + swz128_offset(r0, 2 * (c & 3) + odd);
    const uint32_t at1 = (c >> 2) * L::ATOM + swz128_offset(r0, 2 * (c & 3) + 1 - odd);
    static_assert(RPP % 8 == 0, "passes keep the swizzle phase of the thread's first row");
    int base = 0, g = 0;
    bool ok = true, more = true;
    for (int k = 0; ok && more; ++k) {
      if (!(ok = wwait(C_PCF + k % NPC, k / NPC, 239))) break;
      const Piece& pc = pieces[k % NPC];
      const int hk = pc.hk, b = pc.b, n = pc.n, t0 = pc.t0, t1 = pc.t1_last >> 1;
      const int lim_lo = p.causal ? n - pc.m : n - 1;
      int* nan_key = nan_keys + (k % NPC) * 132;
      more = !(pc.t1_last & 1);
      float sk = 0.0f, sv = 0.0f;  // this thread's key of the coming tile
      int raw_page = -1;           // its page in the tile after that, as it lies in the table
      auto load_page = [&](int t) {
        const int key = t * TN + ct;
        return t < t1 && key < n && in_bounds(key >= 0 && (key >> p.c.page_shift) < p.bt.max_pages, 181) ? __ldg(p.bt.table + (long long)b * p.bt.max_pages + (key >> p.c.page_shift)) : -1;
      };
      auto load_scales = [&](int t, int pg) {
        sk = sv = 0.0f;
        if ((unsigned)pg < (unsigned)p.c.pages) {
          const long long si = p.c.scale(pg, hk, (t * TN + ct) & p.c.page_mask);
          if (!p.c.holds_scale(si, 182)) return;
          sk = __ldg(p.c.ks + si);
          sv = __ldg(p.c.vs + si);
        }
      };
      if (TOK && t0 < t1) {
        load_scales(t0, load_page(t0));
        raw_page = load_page(t0 + 1);
      }
      for (int t = t0; t < t1 && ok; ++t) {
        const int j = base + t - t0, st = j % NSG, ss = j % NSC;
        float* sc = reinterpret_cast<float*>(smem + L::SC + ss * L::SCB);
        if (TOK) {
          // s_k, s_v and the factor of the V codes (1 but for tiny scales).  The rows that see a key whose s_v is NaN or
          // infinite get their NaN when they are written.
          float f = 1.0f;
          if (!(fabsf(sv) < INFINITY)) {
            atomicMin(nan_key + 128, t * TN + ct);
            f = 0.0f;
            sv = kMinScale;
          } else if (sv < kMinScale) {
            f = sv * (1.0f / kMinScale);
            sv = kMinScale;
          }
          if (j >= NSC && !(ok = wwait(C_SCE + ss, j / NSC - 1, 245))) break;
          sc[ct] = finite_or_nan(sk);
          sc[TN + ct] = sv;
          sc[2 * TN + ct] = f;
          const bool any_f = __any_sync(0xffffffffu, f != 1.0f);
          const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(sv));
          __syncwarp();
          if (lane == 0) {
            sc[3 * TN + (warp & 3)] = any_f ? 1.0f : 0.0f;
            sc[3 * TN + 4 + (warp & 3)] = __uint_as_float(top);
            mbar_arrive(&bar[C_SCF + ss]);
          }
          load_scales(t + 1, raw_page);
          raw_page = load_page(t + 2);
        }
        // in a tile that not every row sees whole, V rows past the end are cleared, and NaN codes
        const bool edge = FP8 && t * TN + TN - 1 > lim_lo;
#pragma unroll 1
        for (int u = 0; u < 2 * UT; ++u, ++g) {
          const int sl = g % NU;
          if (!(ok = wwait(C_RF + sl, g / NU, 237))) break;
          if (u == 0 && j >= NSG && !(ok = wwait(C_KE + st, j / NSG - 1, 246))) break;
          if (u == UT && j >= NSG && !(ok = wwait(C_VE + st, j / NSG - 1, 247))) break;
          if (u == UT && TOK && !(ok = wwait(C_SCF + ss, j / NSC, 255))) break;  // the other warps' factors
          if (FP8 && edge && u >= UT) {  // this thread's chunks, in the staging slot
#pragma unroll 1
            for (int q = 0; q < NP; ++q) {
              const int key = t * TN + (u - UT) * UR + r0 + q * RPP;
              uint32_t* at = reinterpret_cast<uint32_t*>(smem + L::RAW + sl * L::UNIT + ct * 16 + q * 2048);
              const uint4 x = *reinterpret_cast<const uint4*>(at);
              if (key >= n) {
                *reinterpret_cast<uint4*>(at) = make_uint4(0, 0, 0, 0);
              } else if (e4m3_nans(x.x) | e4m3_nans(x.y) | e4m3_nans(x.z) | e4m3_nans(x.w)) {
#pragma unroll 1
                for (int e = 0; e < 4; ++e) {
                  const uint32_t nans = e4m3_nans(at[e]);
                  note_nans(nans, 16 * c + 4 * e, key, nan_key);
                  at[e] &= ~((nans >> 7) * 0xFFu);
                }
              }
            }
            fence_async_smem();  // the slot's next bytes come by TMA
          }
          uint8_t* tile = smem + (u < UT ? L::K : L::V) + st * L::TILE + (u % UT) * UR * 128;
          const uint8_t* raw = smem + L::RAW + sl * L::UNIT + ct * 16;
          bool scaled = false;
          if (TOK && u >= UT) {
            const float4 y = *reinterpret_cast<const float4*>(sc + 3 * TN);
            scaled = y.x + y.y + y.z + y.w != 0.0f;
          }
          uint4 xs[NP];
#pragma unroll
          for (int q = 0; q < NP; ++q) xs[q] = *reinterpret_cast<const uint4*>(raw + q * 2048);
#pragma unroll
          for (int q = 0; q < NP; ++q) {
            const uint32_t w[4] = {xs[q].x, xs[q].y, xs[q].z, xs[q].w};
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) codes4_to_h2<FP8>(w[e], h[2 * e], h[2 * e + 1]);
            if (scaled) {
              const __half2 f2 = __float2half2_rn(sc[2 * TN + (u - UT) * UR + r0 + q * RPP]);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&h[e]), f2);
                h[e] = *reinterpret_cast<const uint32_t*>(&y);
              }
            }
            const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
            *reinterpret_cast<uint4*>(tile + at0 + q * RPP * 128) = odd ? hi : lo;
            *reinterpret_cast<uint4*>(tile + at1 + q * RPP * 128) = odd ? lo : hi;
          }
          // the slot is given back once its values have been used: an arrive behind loads that are still on their way lets
          // the next unit land under them
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar[C_RE + sl]);
          if (u % UT == UT - 1) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[(u < UT ? C_KF : C_VF) + st]);
          }
        }
      }
      base += t1 - t0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[C_PCE + k % NPC]);
    }
  } else {
    regs_inc<RS>();
    // ---------------------------------------------------------------- softmax
    const int x = (warp - 8) >> 2;
    const int i = tid - 256 - x * 128;  // row of the tile, TMEM lane
    const uint32_t loff = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + L::TS0 + x * 128;
    const uint32_t tO = tbase + (x ? L::TO1 : L::TO0);
    float2* ml = reinterpret_cast<float2*>(smem + L::ML);
    int base = 0, n_done = 0, n_dual = 0, nq = 0;
    int done_b = 0;  // tile A's view of tile B's count (blocks of at most 128 rows)
    bool ok = true, more = true;
    for (int k = 0; ok && more; ++k) {
      if (!(ok = wwait(C_PCF + k % NPC, k / NPC, 239))) break;
      const Piece& pc = pieces[k % NPC];  // kept until the piece is done
      const int t0 = pc.t0, t1 = pc.t1_last >> 1, kt = pc.kt[x], dual = pc.dual;
      more = !(pc.t1_last & 1);
      int lim = -1;
      float f = 0.0f;
      bool warp_live = false;
      if (t0 < t1) {  // (a piece without keys has no products, and is not waited for)
        // ---- this thread's Q row as fp16, scaled by a power of two
        const Seq s = {pc.q0, pc.m, pc.n};
        const int hk = pc.hk, r = pc.row0 + i + (dual ? 0 : x * BM), ii = r / p.G;
        const bool live = r < s.m * p.G && q_row_ok(p, s, hk, r, 183);
        lim = live ? row_limit(p, s, r) : -1;
        warp_live = __any_sync(0xffffffffu, live);
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (long long)(s.q0 + ii) * p.q_stride +
                                                          (long long)(hk * p.G + r - ii * p.G) * D);
        float m = 0.0f;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = live ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xFFFF0000u))));
        }
        const float head_scale = TOK ? 1.0f : __ldg(p.c.ks + hk);
        float inv;
        float sc = pow2_to_fp16(m, inv);
        // a query or K scale that is no number: NaN in the row's operand, so that the keys it does not see stay masked
        if (!(m < INFINITY) || !(fabsf(head_scale) < INFINITY)) sc = __uint_as_float(0x7FC00000u);
        uint8_t* qt = smem + L::Q + x * L::TILE;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = live ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __half2 hv = __floats2half2_rn(__uint_as_float(w[e] << 16) * sc, __uint_as_float(w[e] & 0xFFFF0000u) * sc);
            h[e] = *reinterpret_cast<const uint32_t*>(&hv);
          }
          *reinterpret_cast<uint4*>(qt + (c >> 3) * L::ATOM + swz128_offset(i, c & 7)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
        f = p.scale_log2 * inv * head_scale;
        if (f == 0.0f || sc != sc) f = 1e-37f;  // a zero K scale: scores vanish, and hidden keys stay at -inf
        fence_async_smem();
        tc_fence_before();
        mbar_arrive(&bar[C_Q]);
        // both warpgroups: none runs a piece ahead of the other (the merge of the two goes through ml)
        if (!(ok = wwait(C_Q, nq++, 254))) break;
      }
      const int lim_lo = p.causal ? pc.n - pc.m + pc.row0 / p.G : pc.n - 1;  // every row of the block sees the keys up to here
      // factors of V: 2^(x - m_run + 7), times s_v in the per-token modes, whose m_run is that of x + log2 s_v;
      // m_raw: m_run before f
      float m_run = -INFINITY, m_raw = 0.0f, l_run = 0.0f;
      bool first = true;
      for (int t = t0; t < t1 && ok; ++t) {
        const int j = base + t - t0, ss = j % NSC;
        const float* sc = reinterpret_cast<const float*>(smem + L::SC + ss * L::SCB);
        if (TOK && !(ok = wwait(C_SCF + ss, j / NSC, 248))) break;
        if (!has_tile(t0, t1, kt, dual, x, t)) {
          if (TOK) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[C_SCE + ss]);
          }
          continue;
        }
        if (!(ok = wwait(C_SF + x, n_done, 249))) break;
        tc_fence_after();
        if (!warp_live) {  // no row of this warp is the sequence's: whatever its P and O are, nothing reads them
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&bar[C_PF + x]);
            if (TOK) mbar_arrive(&bar[C_SCE + ss]);
          }
          ++n_done;
          first = false;
          continue;
        }
        const bool masked = t * TN + TN - 1 > lim_lo;
        // The row's scores, CW at a time (all 128 at once spill), times s_k in the per-token modes, masked.
        constexpr int CW = 64;
        auto scores = [&](auto&& use, auto fresh) {
#pragma unroll
          for (int c = 0; c < TN; c += CW) {
            uint32_t tr[CW];
#pragma unroll
            for (int q = 0; q < CW; q += 32) tmem_ld32(tS + loff + c + q, *reinterpret_cast<uint32_t(*)[32]>(&tr[q]));
            tmem_ld_wait();
            float v[CW];
#pragma unroll
            for (int k = 0; k < CW; ++k) v[k] = __uint_as_float(tr[k]);
            if (TOK) {
              // the scales of 16 keys at a time: their loads' latencies pass together
#pragma unroll
              for (int k = 0; k < CW; k += 16) {
                float4 ks[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) ks[e] = decltype(fresh)::value ? lds4(sc + c + k + 4 * e) : *reinterpret_cast<const float4*>(sc + c + k + 4 * e);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  attn::fmul2(v[k + 4 * e], v[k + 4 * e + 1], ks[e].x, ks[e].y);
                  attn::fmul2(v[k + 4 * e + 2], v[k + 4 * e + 3], ks[e].z, ks[e].w);
                }
              }
            }
            if (masked) {
#pragma unroll
              for (int k = 0; k < CW; ++k)
                if (t * TN + c + k > lim) v[k] = -INFINITY;
            }
            use(v, c);
          }
        };
        // After a row's first tile the maximum rarely moves: the factors are taken against the old one, and
        // their sum tells whether that was safe (below 2^15 every one fits fp16).  Otherwise, and on a row's first
        // tile, the tile's maximum is taken first, and O rescaled if it moves.
        float l_tile = 0.0f;
        float sv_top = 1.0f;
        if (TOK) {
          const float4 y = *reinterpret_cast<const float4*>(sc + 3 * TN + 4);
          sv_top = fmaxf(fmaxf(y.x, y.y), fmaxf(y.z, y.w));
        }
        uint32_t hp[TN / 2];
        bool exact = __any_sync(0xffffffffu, m_run == -INFINITY);
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
          if (exact) {
            float mx[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) mx[e] = -INFINITY;
            scores([&](float(&v)[CW], int c) {
              if (TOK) {
#pragma unroll
                for (int k = 0; k < CW; ++k) v[k] = fmaf(v[k], f, __log2f(sc[TN + c + k]));
              }
#pragma unroll
              for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int q = 0; q < CW / 8; q += 2) mx[e] = attn::fmax3(mx[e], v[e + 8 * q], v[e + 8 * q + 8]);
            }, Bool<true>{});
            const float mt = attn::fmax3(attn::fmax3(mx[0], mx[1], mx[2]), attn::fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
            const float mts = TOK || mt == -INFINITY ? mt : mt * f;
            const float m_new = mts > m_run + 8.0f ? mts : m_run;
            const float alpha = m_new == m_run ? 1.0f : attn::ex2(m_run - m_new);  // 0 from -inf
            if (!first && __any_sync(0xffffffffu, alpha != 1.0f)) {
              if (!(ok = wwait(C_PV + x, n_done - 1, 250))) break;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                tmem_ld16(tO + loff + c * 16, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st16(tO + loff + c * 16, o);
              }
              tmem_st_wait();
            }
            l_run *= alpha;
            if (m_new != m_run) m_raw = mt;
            m_run = m_new;
          }
          // scores past 2^20: v f and the rounded maximum would differ by more than an exponent can bear, so
          // the maximum is taken off before f
          const bool far = __any_sync(0xffffffffu, m_run > -INFINITY && fabsf(m_run) > 0x1p20f);
          // (per-token modes: after f's own rounding, which the maximum has had too)
          const float fe = TOK && far ? 1.0f : f;
          const float nb = m_run == -INFINITY ? 0.0f : kShift - (far && !TOK ? 0.0f : m_run);
          float ls[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          scores([&](float(&v)[CW], int c) {
            if (far) {
#pragma unroll
              for (int k = 0; k < CW; ++k) v[k] = TOK ? v[k] * f : v[k] - m_raw;
            }
#pragma unroll
            for (int k = 0; k < CW; k += 16) {
              float4 vs[4];
              if (TOK) {
#pragma unroll
                for (int e = 0; e < 4; ++e) vs[e] = *reinterpret_cast<const float4*>(sc + TN + c + k + 4 * e);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float* o = &v[k + 4 * e];
                attn::ffma2(o[0], o[1], fe, fe, nb, nb);
                attn::ffma2(o[2], o[3], fe, fe, nb, nb);
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4) o[i4] = attn::ex2(o[i4]);
                attn::fadd2(ls[0], ls[1], o[0], o[1]);
                attn::fadd2(ls[2], ls[3], o[2], o[3]);
                if (TOK) {
                  attn::fmul2(o[0], o[1], vs[e].x, vs[e].y);
                  attn::fmul2(o[2], o[3], vs[e].z, vs[e].w);
                }
                const __half2 h0 = __floats2half2_rn(o[0], o[1]), h1 = __floats2half2_rn(o[2], o[3]);
                hp[(c + k) / 2 + 2 * e] = *reinterpret_cast<const uint32_t*>(&h0);
                hp[(c + k) / 2 + 2 * e + 1] = *reinterpret_cast<const uint32_t*>(&h1);
              }
            }
          }, Bool<false>{});
          l_tile = (ls[0] + ls[1]) + (ls[2] + ls[3]);
          // the sum (times the tile's largest s_v) is above every factor
          const float w = TOK ? l_tile * sv_top : l_tile;
          if (exact || !__any_sync(0xffffffffu, !(w < 32768.0f))) break;
          exact = true;
        }
        if (!ok) break;
        // ---- P: the factors as fp16, over S
        tmem_st32(tS + loff, *reinterpret_cast<uint32_t(*)[32]>(&hp[0]));
        tmem_st32(tS + loff + 32, *reinterpret_cast<uint32_t(*)[32]>(&hp[32]));
        tmem_st_wait();
        l_run += l_tile;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bar[C_PF + x]);
          if (TOK) mbar_arrive(&bar[C_SCE + ss]);
        }
        ++n_done;
        first = false;
      }
      base += t1 - t0;
      if (!ok) break;
      // -------------------------------------------------------------- results
      const bool any = tile_count(t0, t1, kt, dual, x) > 0;
      const int n_b = tile_count(t0, t1, pc.kt[1], dual, 1);
      if (any && !(ok = wwait(C_PV + x, n_done - 1, 251))) break;
      tc_fence_after();
      float m_ref = m_run == -INFINITY ? -INFINITY : m_run - kShift;  // l and O are in units of 2^m_ref
      float wa = 1.0f, wb = 0.0f;
      if (dual && t0 < t1) {
        if (x == 1) {
          ml[i] = make_float2(m_ref, l_run);
          mbar_arrive(&bar[C_ML]);
        } else {
          if (!(ok = wwait(C_ML, n_dual, 252))) break;
          done_b += n_b;
          if (n_b > 0 && !(ok = wwait(C_PV + 1, done_b - 1, 253))) break;
          tc_fence_after();
          const float2 o = ml[i];
          const float m = fmaxf(m_ref, o.x);
          wa = m_ref == -INFINITY ? 0.0f : attn::ex2(m_ref - m);
          wb = o.x == -INFINITY ? 0.0f : attn::ex2(o.x - m);
          l_run = l_run * wa + o.y * wb;
          m_ref = m;
        }
        ++n_dual;
      } else {
        done_b += n_b;
      }
      if (!(dual && x == 1)) {
        const bool any_b = dual && n_b > 0;
        const bool whole = pc.whole;
        const int hk = pc.hk, r = pc.row0 + i + (dual ? 0 : x * BM), ii = r / p.G;
        const bool live = r < pc.m * p.G && q_row_ok(p, {pc.q0, pc.m, pc.n}, hk, r, 184) &&
                          (whole || in_bounds(pc.slot < 2 * (int)gridDim.x && r - pc.row0 >= 0 && r - pc.row0 < PL::RB, 185));
        const long long slot_row = (long long)pc.slot * PL::RB + (r - pc.row0);
        const long long out_row = (long long)(pc.q0 + ii) * p.Hq + hk * p.G + r - ii * p.G;
        const float fac = whole ? row_factor(p, hk, l_run, m_ref, m_ref) : 1.0f;
        const int* nan_key = nan_keys + (k % NPC) * 132;
        const bool all_nan = TOK && nan_key[128] <= lim;
        if (live) {
          if (whole) {
            if (p.lse) p.lse[out_row] = row_lse(l_run, m_ref);
          } else {
            p.part_ml[slot_row] = make_float4(m_ref, l_run, m_ref, 0.0f);
          }
        }
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t o[16], ob[16];
          if (any) tmem_ld16(tO + loff + c * 16, o);
          if (any_b) tmem_ld16(tbase + L::TO1 + loff + c * 16, ob);
          tmem_ld_wait();
          float y[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            y[k] = any ? __uint_as_float(o[k]) * wa : 0.0f;
            if (any_b) y[k] += __uint_as_float(ob[k]) * wb;
            y[k] *= fac;
            if (all_nan || (FP8 && nan_key[c * 16 + k] <= lim)) y[k] = __uint_as_float(0x7FC00000u);
          }
          if (live && whole) {
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const __nv_bfloat162 v2 = __floats2bfloat162_rn(y[2 * e], y[2 * e + 1]);
              h[e] = *reinterpret_cast<const uint32_t*>(&v2);
            }
            uint4* dst = reinterpret_cast<uint4*>(p.out + out_row * D + c * 16);
            dst[0] = make_uint4(h[0], h[1], h[2], h[3]);
            dst[1] = make_uint4(h[4], h[5], h[6], h[7]);
          } else if (live) {
            float4* dst = reinterpret_cast<float4*>(p.part_o + slot_row * D + c * 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[e] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
          }
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[C_PCE + k % NPC]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int D, bool FP8, bool TOK>
cudaError_t launch_a(const CUtensorMap& mk, const CUtensorMap& mv, const AttnP& p, int grid, cudaStream_t s) {
  auto kern = paged_chunk_kernel<D, FP8, TOK>;
  cudaError_t e;
  if ((e = set_smem_limit(reinterpret_cast<const void*>(kern), CL<D>::ALLOC)) != cudaSuccess) return e;
  kern<<<grid, CT, CL<D>::ALLOC, s>>>(mk, mv, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_combine<CPL, D>(p, grid, s);
}

template <int D>
cudaError_t launch_mode(const CUtensorMap& mk, const CUtensorMap& mv, const AttnP& p, int mode, int grid, cudaStream_t s) {
  switch (mode) {
    case FA_MODE_INT8_PER_HEAD: return launch_a<D, false, false>(mk, mv, p, grid, s);
    case FA_MODE_FP8_PER_HEAD: return launch_a<D, true, false>(mk, mv, p, grid, s);
    case FA_MODE_INT8_PER_TOKEN: return launch_a<D, false, true>(mk, mv, p, grid, s);
    case FA_MODE_FP8_PER_TOKEN: return launch_a<D, true, true>(mk, mv, p, grid, s);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace

size_t paged_chunk_ws(int D) { return plan_ws<CPL>(D, sm_count()); }

cudaError_t launch_paged_chunk(const PagedAttnArgs& a, void* ws, cudaStream_t s) {
  AttnP p = paged_attn_params(a);
  if (const cudaError_t be = bounds_attach(); be != cudaSuccess) return be;
  const int D = a.q->D, grid = sm_count();
  plan_carve<CPL>(p, ws, D, grid);
  CUtensorMap mk, mv;
  cudaError_t e;
  if ((e = make_page_map(&mk, a.cache->k_codes, *a.cache, 8192 / D, false)) != cudaSuccess) return e;
  if ((e = make_page_map(&mv, a.cache->v_codes, *a.cache, 8192 / D, false)) != cudaSuccess) return e;
  return D == 128 ? launch_mode<128>(mk, mv, p, a.cache->mode, grid, s)
                  : launch_mode<64>(mk, mv, p, a.cache->mode, grid, s);
}

}  // namespace faq
