// Linear attention with a decay per head on the tensor cores: one pass of
// the recurrence in decay.h (the forward, or one gradient) for bf16 inputs.
//
// A CTA walks one segment of one head in chunks of 128 rows, the state S
// (D x D, fp32) carried from chunk to chunk in registers.  Per chunk, with
// rows t, s and lambda = exp(g):
//
//   M   = X Y^T                                   fp32, tensor memory
//   P   = M lambda^|t-s| where s is not after t   bf16, over M
//   O   = si lambda^(t+1) (X S) + so (P Z)        two products, one accumulator region
//   U   = Y'^T Z,  y'_s = lambda^(n-1-s) y_s
//   S  <- lambda^n S + us U
//
// Roundings to bf16: P, and the copy of S that X is multiplied with (once
// each; outputs are bf16 as well, and all three come to 0.0023 of the norm
// where the output's alone is 0.0017; second parts would cost a product each
// and columns of tensor memory that are not there).  A state that is handed
// out loses nothing:
// y' is an fp32 number, taken apart into three bf16 parts of eight bits, and U
// is the sum of three products, as exact as an fp32 sum.  Where the state is
// only multiplied with, rounded to bf16 (2^-9), and for rows that weigh less
// than 1/16 in the state handed out, two parts do (2^-16): a third of the
// instructions, two thirds of the products.
//
// Roles (18 warps):
//   warps 0-7   thread = row t, half of the columns each: M to P, X S scaled,
//               O out
//   warps 8-15  32 features of y, half of the rows each: y' into tensor
//               memory (transposed, as U's A operand); thread = row of the
//               state, half of the columns each
//   warp 16     TMA loads of X, Y, Z (two stages) and stores of O, which is
//               staged over its chunk's X
//   warp 17     the MMAs, one elected lane issuing
//
// Tensor memory (512 columns): M 128 (P over its columns 0-31 and 64-95, the
// third part of y' over 32-63 and 96-127), O 128, U 128, y' parts one and
// two 64 each; at D = 64 half of O's and U's are free.  Shared memory: two
// stages of X, Y, Z (192 KB at D = 128) and S as bf16 (32 KB).
//
// What bounds it: a chunk's chain of steps.  With two parts a chunk takes 2.65
// us, about 5300 clk, on 128 SMs at once (2.5 us on one SM alone), of which the
// tensor pipe works 2560 at D = 128; with three 4.0 us, about 8000 clk, of which
// it works 512 more; at D = 64 1.9 and 2.7 us (all from the difference of 33, 17
// and 9 chunks).
// Of it y' is 1700 to 1900 clk (two parts), U 1024 and about 900 of queueing,
// commit and hand-over, the state 1050, one after the other: there is one y'
// and one U, and at D = 128 no tensor memory for a second.  16 heads of 32768
// rows, each launch by itself: outputs 89 us (6.0 TB/s), sums 44 (two parts)
// and 54 (three for the weakest decays), all gradients 263 (1.3 GB of DRAM
// traffic).
//
// At D = 64 U's A operand has 64 of 128 lanes: the others hold whatever the
// tensor memory did, and the rows of U that come of them are not read.
#include <cuda.h>

#include <type_traits>

#include "common.cuh"
#include "decay.h"
#include "host_common.h"
#include "launch_util.h"
#include "mma4.cuh"
#include "ptx.cuh"
#include "tmap.h"

namespace sca {
namespace decay_tc {

constexpr int kSub = kDecaySub;
constexpr int kThreads = 640;               // five warpgroups
constexpr int kConv = 256;                  // threads of a converter group
constexpr int kConvWarps = kConv / 32;      // arrivals of one on a barrier
constexpr int kProdWarp = 16, kMmaWarp = 17;
constexpr int PANEL = kSub * 128;           // 128 rows x 64 bf16, 128-byte swizzle
// Registers a thread: the launch gives 640 x 96 = 61440; the row group gives
// up 24, the role warps 16, and the feature group, which holds the state,
// takes 32: 256 x 72 + 256 x 128 + 128 x 80 = 61440.
constexpr int kRegRows = 72, kRegFeatures = 128, kRegRoles = 80;
static_assert(256 * kRegRows + 256 * kRegFeatures + 128 * kRegRoles <= kThreads * 96, "register split");

struct Bars {
  uint64_t yz_full[3], x_full[2], yz_free[3], out_staged[2];
  uint64_t m_full, m_read;      // M in tensor memory; read out of it (chunks of three parts)
  uint64_t s_full;              // the chunk's start state (bf16) in shared memory
  uint64_t o1_full, o2_full;    // X S done; P Z done
  uint64_t o_free;              // P Z read
  uint64_t p_full;              // P in tensor memory and X S read
  uint64_t k_full;              // y' in tensor memory, rows of Z behind the sequence zeroed
  uint64_t z_full;              // these rows zeroed (a pass has one ragged chunk at most)
  uint64_t u_full;
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

template <int D>
struct Layout {
  static constexpr int TILE = D / 64 * PANEL;
  static constexpr int STAGE = 3 * TILE;                  // X, Y, Z
  static constexpr int S_OFF = 2 * STAGE;                 // S: D rows of D bf16, panels of 64 columns
  static constexpr int SPANEL = D * 128;
  static constexpr int TAB_OFF = S_OFF + D / 64 * SPANEL; // lambda^d at [128 + d], d in [-128, 128]; 0 below 0
  static constexpr int W_OFF = TAB_OFF + 260 * 4;         // weights of a full chunk's pairs of rows, two bf16 parts
  static constexpr int C_OFF = W_OFF + kSub / 2 * 8;      // column factors of 32 columns
  static constexpr int BAR_OFF = C_OFF + 32 * 4;
  static constexpr int SMEM = BAR_OFF + static_cast<int>(sizeof(Bars)) + 1024;
  static_assert(SMEM <= 232448, "one CTA's shared memory");
};

struct Args {
  CUtensorMap mx, my, mz, mo;
  DecayPass p;
};

// Four 8 x 8 bf16 blocks of a row-major tile, transposed: lane i gets, of
// each, column i / 4 of rows 2 (i % 4) and 2 (i % 4) + 1, as a pair.
SCA_INLINE void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// 16 lanes x 8 columns of tensor memory: lane i of the warp holds lanes i / 4
// (r0, r2) and i / 4 + 8 (r1, r3), columns i % 4 (r0, r1) and 4 + i % 4.
SCA_INLINE void tmem_st_16x128b_x2(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}

SCA_INLINE float2 unpack_bf16x2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// a pair as bf16, infinities as the largest finite numbers
SCA_INLINE uint32_t pack_sat_bf16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// a pair as three bf16 parts each: x = hi + mid + lo up to 2^-24 x.  Of an
// infinity the first two are the largest finite number and the last is the
// infinity: rounded to itself, the first would leave inf - inf to the others.
SCA_INLINE void split3(float2 x, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = pack_sat_bf16x2(x.x, x.y);
  x = fsub2(x, unpack_bf16x2(hi));
  mid = pack_sat_bf16x2(x.x, x.y);
  x = fsub2(x, unpack_bf16x2(mid));
  lo = pack_bf16x2(x.x, x.y);
}

// bf16 arithmetic on pairs, each operation rounded once
SCA_INLINE uint32_t bmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
SCA_INLINE uint32_t bfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// infinities as the largest finite numbers
SCA_INLINE uint32_t finite2(uint32_t a) {
  uint32_t d;
  asm("min.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(0x7f7f7f7fu));
  return d;
}

template <int D, bool kStates, bool kRev, bool k3>
SCA_INLINE void pass(const Args& ka, const int seg, const int bh) {
  using L = Layout<D>;
  const DecayPass& p = ka.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + L::BAR_OFF);
  float* tab = reinterpret_cast<float*>(smem + L::TAB_OFF);
  uint2* w2 = reinterpret_cast<uint2*>(smem + L::W_OFF);
  float* wcol = reinterpret_cast<float*>(smem + L::C_OFF);

  // Stages: X, Y, Z each in two; sums alone have Y and Z in three
  constexpr int kSt = kStates ? 3 : 2, kStage = kStates ? 2 * L::TILE : L::STAGE, kYoff = kStates ? 0 : L::TILE;
  auto stage_of = [](int c) { return kStates ? c % 3 : c & 1; };
  auto phase_of = [](int c) { return (kStates ? c / 3 : c >> 1) & 1; };
  const int b = bh / p.H, h = bh % p.H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool loads = threadIdx.x == 32 * kProdWarp;   // the thread that issues them
  if (loads) {
    for (int i = 0; i < kSt; ++i) {
      mbar_init(&bars->yz_full[i], 1);
      mbar_init(&bars->yz_free[i], kStates ? 1 : 2);   // U done; P Z done
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->x_full[i], 1);
      mbar_init(&bars->out_staged[i], kConvWarps);
    }
    mbar_init(&bars->m_full, 1);
    mbar_init(&bars->m_read, kConvWarps);
    mbar_init(&bars->s_full, kConvWarps);
    mbar_init(&bars->o1_full, 1);
    mbar_init(&bars->o2_full, 1);
    mbar_init(&bars->o_free, kConvWarps);
    mbar_init(&bars->p_full, kConvWarps);
    mbar_init(&bars->k_full, kConvWarps);
    mbar_init(&bars->z_full, kConvWarps);
    mbar_init(&bars->u_full, 1);
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    fence_mbar_init();
    tma_prefetch_map(&ka.my);
    tma_prefetch_map(&ka.mz);
    if (!kStates) {
      tma_prefetch_map(&ka.mx);
      tma_prefetch_map(&ka.mo);
    }
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  wait_for_previous();   // the lengths may be an earlier kernel's as well
  const float g = p.log_decay[h];
  const int64_t len = decay_len(p, b);
  const DecayRows rows = decay_rows(p, seg, len);
  const int row_lo = static_cast<int>(rows.lo), row_hi = static_cast<int>(rows.hi);   // S < 2^24
  const int nchunk = (row_hi - row_lo + kSub - 1) / kSub;
  const bool want_end = kStates || (p.end != nullptr && seg == p.nseg - 1);
  // first row and number of rows of chunk c (processing order)
  auto row_of = [&](int c) { return row_lo + (kRev ? nchunk - 1 - c : c) * kSub; };
  auto n_of = [&](int c) { return min(kSub, row_hi - row_of(c)); };
  // Does chunk c take three parts?  Where the state is handed out, and its rows
  // still weigh more than 1/16 there: with two parts an earlier chunk leaves
  // less than 2^-16 / 16 of its own weight.
  int exact_rows = 0;   // rows from the end that do
  if (k3 && p.exact) exact_rows = g < -1e-6f ? static_cast<int>(2.7725887f / -g) + 1 : 1 << 24;   // lambda^rows = 1/16
  const int end_row = kRev ? 0 : static_cast<int>(len);
  auto exact_of = [&](int c) {
    if (!k3) return false;
    const int after = kRev ? row_of(c) - end_row : end_row - (row_of(c) + n_of(c));   // rows behind the chunk
    return after < exact_rows;
  };
  const int delta0 = kRev && !kStates && rows.s1 >= len ? 1 : 0;   // power taken off in the first chunk

  auto load = [&](uint64_t* bar, uint8_t* to, const CUtensorMap* m, int row) {
    for (int k = 0; k < D / 64; ++k) tma_load_4d(to + k * PANEL, m, bar, 64 * k, row, h, b);
  };
  auto load_yz = [&](int c) {
    const int s = stage_of(c);
    uint8_t* st = smem + s * kStage + kYoff;
    mbar_arrive_expect_tx(&bars->yz_full[s], 2 * L::TILE);
    load(&bars->yz_full[s], st, &ka.my, row_of(c));
    load(&bars->yz_full[s], st + L::TILE, &ka.mz, row_of(c));
  };
  auto load_x = [&](int c) {
    mbar_arrive_expect_tx(&bars->x_full[c & 1], L::TILE);
    load(&bars->x_full[c & 1], smem + (c & 1) * kStage, &ka.mx, row_of(c));
  };
  if (loads && nchunk > 0) {   // the first chunk's, while the others make the tables
    load_yz(0);
    if (!kStates) load_x(0);
  }

  if (threadIdx.x < 129) {
    const int d = threadIdx.x;
    const float w = decay_pow(g, d);
    tab[128 + d] = w;
    if (d < 128) {
      tab[d] = 0.f;
      const float us = p.us * w;
      const __nv_bfloat16 wh = __float2bfloat16_rn(us), wl = __float2bfloat16_rn(us - __bfloat162float(wh));
      const int r = kRev ? d : 127 - d;   // row r's halves of its pair's words
      __nv_bfloat16* at = reinterpret_cast<__nv_bfloat16*>(w2 + (r >> 1)) + (r & 1);
      at[0] = wh;
      at[2] = wl;
    }
    if (kRev ? d < 32 : d >= 1 && d <= 32) wcol[kRev ? d : 32 - d] = w;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const uint32_t tM = tmem, tO = tmem + 128, tU = tmem + 256, tK = tmem + 384;
  // chunk c's parts of y', 64 columns each (the third in two halves of 32
  // where M is); sums alone have two sets
  auto t_hi = [&](int c) { return kStates && (c & 1) ? tM + 64 : tK; };
  auto t_mid = [&](int c) { return kStates && (c & 1) ? tO : tK + 64; };
  auto t_lo = [&](int c) { return !kStates ? tM + 32 : ((c & 1) ? tO + 64 : tM); };
  volatile int* abort = &bars->abort;
  const uint32_t s0 = smem_u32(smem);
  auto wait_all = [&](uint64_t* bar, uint32_t par) { return wait_all_or_abort(bar, par, abort); };

  if (warp >= kProdWarp) {
    reg_dec<kRegRoles>();
  if (warp == kProdWarp) {
    // ------------------------------------------------ loads and stores
    if (lane == 0) {
      // chunk c's outputs, staged over its X, and X's stage free again
      auto store = [&](int c) -> bool {
        if (!wait_or_abort(&bars->out_staged[c & 1], (c >> 1) & 1, abort)) return false;
        for (int k = 0; k < D / 64; ++k)
          tma_store_4d(&ka.mo, smem + (c & 1) * L::STAGE + k * PANEL, 64 * k, row_of(c), h, b);
        bulk_commit();
        bulk_wait_read<0>();
        return true;
      };
      int c = nchunk > 0, nx = kStates ? 0 : c;   // chunks whose Y, Z and whose X were asked for
      for (; c < nchunk; ++c) {
        if (c >= kSt && !wait_or_abort(&bars->yz_free[stage_of(c)], phase_of(c) ^ 1, abort)) break;
        load_yz(c);
        if (!kStates) {
          if (c >= 2 && !store(c - 2)) {
            ++c;
            break;
          }
          load_x(c);
          ++nx;
        }
      }
      if (!kStates && !*abort)
        for (int j = nchunk > 2 ? nchunk - 2 : 0; j < nchunk; ++j)
          if (!store(j)) break;
      if (*abort) {   // let the copies in flight land before the CTA goes away
        for (int j = (c > kSt ? c - kSt : 0); j < c; ++j) mbar_wait_drain(&bars->yz_full[stage_of(j)], phase_of(j));
        for (int j = (nx > 2 ? nx - 2 : 0); j < nx; ++j) mbar_wait_drain(&bars->x_full[j & 1], (j >> 1) & 1);
      }
      if (!kStates) bulk_wait_all();
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------- MMAs
    constexpr uint32_t id_m = idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t id_o = idesc_bf16_f32(128, D, false, true);   // X S, P Z and U alike: B with N along the row
    bool ok = true;
    for (int c = 0; ok && c < nchunk; ++c) {
      const int s = stage_of(c);
      const bool need_u = want_end || c + 1 < nchunk;
      const uint32_t sX = s0 + s * kStage, sY = sX + kYoff, sZ = sY + L::TILE;
      const uint64_t zd = sdesc_sw128(sZ, PANEL, 1024);
      if (!(ok = wait_all(&bars->yz_full[s], phase_of(c)))) break;
      if (kStates) {
        if (!(ok = wait_all(&bars->s_full, c & 1))) break;   // U of the chunk before has been read
      } else {
        if (!(ok = wait_all(&bars->x_full[s], (c >> 1) & 1))) break;
        tc_fence_after();
        const uint64_t xd = sdesc_sw128(sX, 16, 1024), yd = sdesc_sw128(sY, 16, 1024);
#pragma unroll
        for (int k = 0; k < D / 64; ++k)   // panels of 64 columns: 32 bytes a step along the row
          umma4_ss<2, 2>(tM, sdesc_step(xd, k * PANEL), sdesc_step(yd, k * PANEL), id_m, k);
        umma_commit_w(&bars->m_full);
        if (!(ok = wait_all(&bars->s_full, c & 1))) break;
        if (c > 0 && !(ok = wait_all(&bars->o_free, (c - 1) & 1))) break;
        tc_fence_after();
        const uint64_t sd = sdesc_sw128(s0 + L::S_OFF, L::SPANEL, 1024);
#pragma unroll
        for (int k = 0; k < D / 64; ++k)   // S: 16 rows (2048 bytes) a step
          umma4_ss<2, 128>(tO, sdesc_step(xd, k * PANEL), sdesc_step(sd, k * 8192), id_o, k);
        umma_commit_w(&bars->o1_full);
      }
      // U and P Z, whichever is ready first
      bool u_left = true, p_left = !kStates;
      while (ok && (u_left || p_left)) {
        bool take_u = u_left;
        if (u_left && p_left) {
          const uint32_t since = globaltimer_lo();
          for (uint32_t turn = 1;; ++turn) {
            if (__any_sync(0xffffffffu, mbar_test(&bars->p_full, c & 1))) {
              take_u = false;
              break;
            }
            if (__any_sync(0xffffffffu, mbar_test(&bars->k_full, c & 1))) break;
            // the bounded wait below records what gave up
            if (turn % 64 == 0 &&
                __any_sync(0xffffffffu, *abort || globaltimer_lo() - since > static_cast<uint32_t>(kWaitLimitNs)))
              break;
          }
        }
        if (!(ok = wait_all(take_u ? &bars->k_full : &bars->p_full, c & 1))) break;
        if (!take_u && n_of(c) < kSub && !(ok = wait_all(&bars->z_full, 0))) break;
        tc_fence_after();
        if (take_u) {
          u_left = false;
          if (need_u) {
            const bool e3 = exact_of(c);
            // 64 rows of y' at a time: 32 columns of each part
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint64_t z = sdesc_step(zd, k * 8192);
              umma4_ts<128>(tU, t_hi(c) + 32 * k, z, id_o, k);
              umma4_ts<128>(tU, t_mid(c) + 32 * k, z, id_o, 1);
              if (k3 && e3) umma4_ts<128>(tU, t_lo(c) + (kStates ? 32 : 64) * k, z, id_o, 1);
            }
            umma_commit_w(&bars->u_full);
          }
        } else {
          p_left = false;
#pragma unroll
          for (int k = 0; k < 2; ++k) umma4_ts<128>(tO, tM + 64 * k, sdesc_step(zd, k * 8192), id_o, 1);
          umma_commit_w(&bars->o2_full);
        }
      }
      if (!ok) break;
    }
    if (!ok || *abort) {   // every MMA issued has finished before the memory goes
      umma_commit_w(&bars->drain);
      mbar_wait_drain(&bars->drain, 0);
    }
  }
  } else if (warp < 8) {
    // ------------------------------------------- rows: M to P, outputs
    reg_dec<kRegRows>();
    if (!kStates) {
      const int q4 = warp & 3, half = warp >> 2;
      const int t = q4 * 32 + lane;
      const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
      bool ok = true;
      for (int c = 0; ok && c < nchunk; ++c) {
        const int n = n_of(c), delta = c == 0 ? delta0 : 0;
        const bool e3 = exact_of(c) && (want_end || c + 1 < nchunk);
        if (!(ok = wait_all(&bars->m_full, c & 1))) break;
        tc_fence_after();
        {
          // A piece of 32 columns [c0, c0 + 32) for the warp's 32 rows is
          // masked whole, or lies clear of the diagonal, where the power
          // splits into a row's and a column's (both at most 1):
          // lambda^(t - s) = lambda^(t - c0 - 32) lambda^(c0 + 32 - s);
          // the diagonal piece, and every piece of a ragged chunk in reverse
          // (columns behind the sequence may hold NaN), goes element by
          // element.
          // The second piece first: the third part of y' waits for its
          // columns.  Its P goes where the first piece still is, so it is
          // held until that one is read.
          uint32_t held[16];
#pragma unroll 1
          for (int k = 1; k >= 0; --k) {
            const int c0 = 64 * half + 32 * k;
            uint32_t v[32], pk[16];
            tmem_ld32(tM + lane_off + c0, v);
            tmem_wait_ld32(v);
            if (k == 1) {
              tc_fence_before();
              if (e3) warp_arrive(&bars->m_read, lane);
            } else {
              tmem_st16(tM + lane_off + 64 * half + 16, held);
            }
            if (kRev ? c0 < 32 * q4 : c0 > 32 * q4) {
#pragma unroll
              for (int i = 0; i < 16; ++i) pk[i] = 0u;
            } else if (c0 != 32 * q4 && (!kRev || n == kSub)) {
              const float fr = p.so * tab[128 + (kRev ? c0 - t : t - c0 - 32)];
              const float2 f2 = make_float2(fr, fr);
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                const float4 w = *reinterpret_cast<const float4*>(wcol + 2 * i);
                const uint32_t* m = v + 2 * i;
                const float2 x = fmul2(fmul2(make_float2(__uint_as_float(m[0]), __uint_as_float(m[1])), f2),
                                       make_float2(w.x, w.y));
                const float2 y = fmul2(fmul2(make_float2(__uint_as_float(m[2]), __uint_as_float(m[3])), f2),
                                       make_float2(w.z, w.w));
                pk[i] = pack_bf16x2(x.x, x.y);
                pk[i + 1] = pack_bf16x2(y.x, y.y);
              }
            } else {
              // column j is row s = c0 + j: kept for j in [j0, j1)
              const int at = t - c0;
              const int j0 = kRev ? at : 0, j1 = kRev ? n - c0 : at + 1;
              const float* w = tab + 128 + (kRev ? -at : at);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float x[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int j = 2 * i + e;
                  const float y = p.so * __uint_as_float(v[j]) * w[kRev ? j : -j];
                  x[e] = j >= j0 && j < j1 ? y : 0.f;
                }
                pk[i] = pack_bf16x2(x[0], x[1]);
              }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) held[i] = pk[i];
          }
          tmem_st16(tM + lane_off + 64 * half, held);
        }
        // X S by the rows' powers, in place: P Z is added to it
        const int rho = kRev ? n - 1 - t : t;
        const bool live = t < n;
        const float f = live ? p.si * tab[128 + rho + 1 - delta] : 0.f;
        if (!(ok = wait_all(&bars->o1_full, c & 1))) break;
        tc_fence_after();
        const uint32_t to = tO + lane_off + (D / 2) * half;
#pragma unroll 1
        for (int k = 0; k < D / 2; k += 32) {
          uint32_t v[32];
          tmem_ld32(to + k, v);
          tmem_wait_ld32(v);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(f * __uint_as_float(v[i]));
          tmem_st32(to + k, v);
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&bars->p_full, lane);
        if (!(ok = wait_all(&bars->o2_full, c & 1))) break;
        tc_fence_after();
        if (threadIdx.x == 0) mbar_arrive(&bars->yz_free[c & 1]);
        uint8_t* dst = smem + (c & 1) * L::STAGE + t * 128;
#pragma unroll 1
        for (int k = 0; k < D / 2; k += 32) {
          uint32_t v[32];
          tmem_ld32(to + k, v);
          tmem_wait_ld32(v);
          if (k + 32 == D / 2) {
            tc_fence_before();
            warp_arrive(&bars->o_free, lane);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {   // eight columns: one 16-byte chunk of the swizzled row
            uint32_t r[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              r[e] = live ? pack_bf16x2(__uint_as_float(v[8 * q + 2 * e]), __uint_as_float(v[8 * q + 2 * e + 1])) : 0u;
            const int col = (D / 2) * half + k + 8 * q;
            *reinterpret_cast<uint4*>(dst + (col >> 6) * PANEL + ((((col & 63) >> 3) ^ (t & 7)) << 4)) =
                make_uint4(r[0], r[1], r[2], r[3]);
          }
        }
        fence_async_smem();
        warp_arrive(&bars->out_staged[c & 1], lane);
      }
      // rows of whole tiles behind the sequence
      const int64_t z0 = rows.lo + static_cast<int64_t>(nchunk) * kSub;
      if (z0 < rows.s1) {
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + b * p.ov.b + h * p.ov.h;
        for (int64_t e = threadIdx.x; e < (rows.s1 - z0) * (D / 8); e += kConv)
          *reinterpret_cast<uint4*>(out + (z0 + e / (D / 8)) * p.ov.s + 8 * (e % (D / 8))) = make_uint4(0, 0, 0, 0);
      }
    }
  } else {
    // ------------------------------- features: y' and the running state
    reg_inc<kRegFeatures>();
    const int q4 = warp & 3, half = (warp >> 2) & 1;
    const int f = q4 * 32 + lane;      // feature of y: row of the state
    const bool has = D == 128 || f < D;   // warp-uniform
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    const int tid = threadIdx.x - 256;
    const uint32_t tu = tU + lane_off + (D / 2) * half;
    float run[D / 2];                  // S[f][(D/2) half + u]
    const float* from = nullptr;
    if (!kStates) from = p.seg ? p.seg + (static_cast<int64_t>(bh) * p.nseg + seg) * D * D
                               : (p.init ? p.init + b * p.init_b + static_cast<int64_t>(h) * D * D : nullptr);
#pragma unroll
    for (int u = 0; u < D / 2; ++u) run[u] = 0.f;
    // the first chunk takes its state as it takes every U: from zeros, by a carry of one
    if (has) {
#pragma unroll
      for (int k = 0; k < D / 2; k += 32) tmem_st32(tu + k, reinterpret_cast<const uint32_t*>(run) + k);
      tmem_wait_st();
    }
    if (from && has) {
      if (p.transposed) {
#pragma unroll
        for (int u = 0; u < D / 2; ++u) run[u] = from[((D / 2) * half + u) * D + f];
      } else {
#pragma unroll
        for (int u = 0; u < D / 2; u += 4) {
          const float4 v = *reinterpret_cast<const float4*>(from + f * D + (D / 2) * half + u);
          run[u] = v.x;
          run[u + 1] = v.y;
          run[u + 2] = v.z;
          run[u + 3] = v.w;
        }
      }
    }
    float carry = 1.f;
    int n_exact = 0;   // chunks of three parts so far
    // S = carry S + U, and S as bf16 for X S
    auto take_u = [&]() {
      if (has) {
        uint8_t* dst = smem + L::S_OFF + f * 128;
#pragma unroll
        for (int k = 0; k < D / 2; k += 32) {
          uint32_t v[32];
          tmem_ld32(tu + k, v);
          tmem_wait_ld32(v);
#pragma unroll
          for (int u = 0; u < 32; u += 2) {
            const float2 r = ffma2(make_float2(carry, carry), make_float2(run[k + u], run[k + u + 1]),
                                   make_float2(__uint_as_float(v[u]), __uint_as_float(v[u + 1])));
            run[k + u] = r.x;
            run[k + u + 1] = r.y;
          }
          if (!kStates) {
#pragma unroll
            for (int u = k; u < k + 32; u += 8) {
              const int col = (D / 2) * half + u;
              *reinterpret_cast<uint4*>(dst + (col >> 6) * L::SPANEL + ((((col & 63) >> 3) ^ (f & 7)) << 4)) =
                  make_uint4(pack_bf16x2(run[u], run[u + 1]), pack_bf16x2(run[u + 2], run[u + 3]),
                             pack_bf16x2(run[u + 4], run[u + 5]), pack_bf16x2(run[u + 6], run[u + 7]));
            }
          }
        }
      }
      tc_fence_before();
    };
    bool ok = true;
    for (int c = 0; ok && c < nchunk; ++c) {
      const int s = stage_of(c), n = n_of(c), delta = c == 0 ? delta0 : 0;
      const bool need_u = want_end || c + 1 < nchunk, e3 = exact_of(c);
      auto take_state = [&]() -> bool {   // the state before the chunk
        if (c > 0) {
          if (!wait_all(&bars->u_full, (c - 1) & 1)) return false;
          tc_fence_after();
          if (tid == 0) mbar_arrive(&bars->yz_free[stage_of(c - 1)]);
        }
        take_u();
        if (!kStates) fence_async_smem();
        warp_arrive(&bars->s_full, lane);
        carry = tab[128 + n - delta];
        return true;
      };
      if (!kStates && !(ok = take_state())) break;
      if (!(ok = wait_all(&bars->yz_full[s], phase_of(c)))) break;
      uint8_t* sY = smem + s * kStage + kYoff;
      if (n < kSub) {   // rows of Z behind the sequence may hold anything
        uint8_t* sZ = sY + L::TILE;
        for (int e = tid; e < (kSub - n) * (D / 8); e += kConv) {
          const int r = n + e / (D / 8), q = e % (D / 8);
          *reinterpret_cast<uint4*>(sZ + (q >> 3) * PANEL + r * 128 + (q & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
        if (!kStates) warp_arrive(&bars->z_full, lane);
      }
      if (need_u && has) {
        // Two blocks of 16 features, 16 rows at a time: transposed 8 x 8
        // blocks are, lane by lane, what the 16 x 128-bit stores take.
        const uint32_t yb = smem_u32(sY) + (64 * half + (lane & 7) + ((lane >> 4) & 1) * 8) * 128;
        uint32_t ya[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int ch = 4 * q4 + 2 * k + ((lane >> 3) & 1);   // 16-byte chunk of the row
          ya[k] = yb + (ch >> 3) * PANEL + (((ch & 7) ^ (lane & 7)) << 4);
        }
        const int rw = 64 * half + 2 * (lane & 3);             // this lane's pairs start at rows rw + 8 i
        // rows r, r + 1 of a chunk of n: their weights
        auto weights = [&](int r) {
          return make_float2(r < n ? p.us * tab[128 + (kRev ? r : n - 1 - r)] : 0.f,
                             r + 1 < n ? p.us * tab[128 + (kRev ? r + 1 : n - 2 - r)] : 0.f);
        };
        if (!e3) {
          // two parts, in bf16 arithmetic from the weight's own two (wh + wl,
          // 16 bits): hi = y wh rounded, mid = (y wh - hi, exact) + y wl.  Of
          // an infinity, as in split3, hi stays finite and mid is infinite:
          // one more operation a pair, 0.2% of a long prompt's time and 0.7%
          // of training's (made again where found instead: 1.3 to 6%).
          auto conv2 = [&](auto ragged) {
            constexpr bool kRagged = decltype(ragged)::value;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              uint32_t wh[2], wl[2], keep[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int r = rw + 16 * q + 8 * i;
                if (kRagged) {
                  const float2 w = weights(r);
                  wh[i] = pack_bf16x2(w.x, w.y);
                  const float2 l = fsub2(w, unpack_bf16x2(wh[i]));
                  wl[i] = pack_bf16x2(l.x, l.y);
                  // what lies behind the sequence may be NaN
                  keep[i] = (r < n ? 0xffffu : 0u) | (r + 1 < n ? 0xffff0000u : 0u);
                } else {
                  const uint2 v = w2[r >> 1];
                  wh[i] = v.x;
                  wl[i] = v.y;
                }
              }
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t y[4], hi[4], mid[4];
                ldsm4_t(ya[k] + q * 2048, y);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  if (kRagged) y[i] &= keep[i >> 1];
                  const uint32_t yf = finite2(y[i]);
                  hi[i] = bmul2(yf, wh[i >> 1]);
                  mid[i] = bfma2(yf, wl[i >> 1], bfma2(y[i], wh[i >> 1], hi[i] ^ 0x80008000u));
                }
                const uint32_t at = lane_off + (static_cast<uint32_t>(16 * k) << 16) + 32 * half + 8 * q;
                tmem_st_16x128b_x2(t_hi(c) + at, hi);
                tmem_st_16x128b_x2(t_mid(c) + at, mid);
              }
            }
          };
          if (n == kSub) conv2(std::false_type{});
          else conv2(std::true_type{});
        } else {
          // three parts of the fp32 product
#pragma unroll 1
          for (int g = 0; g < 2; ++g) {   // 32 rows at a time
            uint32_t lo[2][2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int q = 2 * g + j;
              float2 w[2];
              uint32_t keep[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int r = rw + 16 * q + 8 * i;
                w[i] = weights(r);
                keep[i] = (r < n ? 0xffffu : 0u) | (r + 1 < n ? 0xffff0000u : 0u);
              }
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t y[4], hi[4], mid[4];
                ldsm4_t(ya[k] + q * 2048, y);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  split3(fmul2(unpack_bf16x2(y[i] & keep[i >> 1]), w[i >> 1]), hi[i], mid[i], lo[j][k][i]);
                const uint32_t at = lane_off + (static_cast<uint32_t>(16 * k) << 16) + 32 * half + 8 * q;
                tmem_st_16x128b_x2(t_hi(c) + at, hi);
                tmem_st_16x128b_x2(t_mid(c) + at, mid);
              }
            }
            // the third part goes between the columns of P: once M, which
            // follows the U of the chunk before, has been read there
            if (!kStates && g == 0) {
              if (!(ok = wait_all(&bars->m_read, n_exact & 1))) break;
              ++n_exact;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int k = 0; k < 2; ++k)
                tmem_st_16x128b_x2(t_lo(c) + lane_off + (static_cast<uint32_t>(16 * k) << 16) +
                                       (kStates ? 32 : 64) * half + 8 * (2 * g + j),
                                   lo[j][k]);
          }
        }
        if (!ok) break;
        tmem_wait_st();
      }
      tc_fence_before();
      warp_arrive(&bars->k_full, lane);
      // sums alone have y' of two chunks in tensor memory: this one's is made
      // while U of the one before runs
      if (kStates && !(ok = take_state())) break;
    }
    if (ok && want_end) {
      if (nchunk > 0) {
        ok = wait_all(&bars->u_full, (nchunk - 1) & 1);
        tc_fence_after();
      }
      if (ok) take_u();
      if (ok && has) {
        float* to = kStates ? p.seg + (static_cast<int64_t>(bh) * p.nseg + seg) * D * D
                            : p.end + static_cast<int64_t>(bh) * D * D;
        const float mul = !kStates && kRev && len > 0 ? tab[129] : 1.f;
#pragma unroll
        for (int u = 0; u < D / 2; u += 4)
          *reinterpret_cast<float4*>(to + f * D + (D / 2) * half + u) =
              make_float4(mul * run[u], mul * run[u + 1], mul * run[u + 2], mul * run[u + 3]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  report_abort(abort, p.status);
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool kStates, bool kRev, bool k3>
__global__ void __launch_bounds__(kThreads, 1) pass_kernel(const __grid_constant__ Args ka) {
  pass<D, kStates, kRev, k3>(ka, blockIdx.x, blockIdx.y);
}

// The three gradients in one launch: by themselves short or few sequences
// would leave most SMs idle three times over.  First every segment's dq, then
// dv and dk of a segment side by side: they read the same q and dO within
// microseconds, from L2, and run the same code.  (All three side by side were
// slower by a third: neighbouring SMs share instruction caches, and two
// directions' code do not fit.)
struct Args3 {
  Args dq, dv, dk;
};
template <int D, bool k3>
__global__ void __launch_bounds__(kThreads, 1) bwd_kernel(const __grid_constant__ Args3 a) {
  const int nseg = a.dq.p.nseg, n = nseg * a.dq.p.B * a.dq.p.H, i = blockIdx.x;
  if (i < n) {
    pass<D, false, false, false>(a.dq, i % nseg, i / nseg);
  } else {
    const int j = (i - n) >> 1;
    pass<D, false, true, k3>((i - n) & 1 ? a.dk : a.dv, j % nseg, j / nseg);
  }
}

template <int D, bool kStates, bool kRev, bool k3>
static int launch(const Args& a, cudaStream_t st) {
  constexpr int smem = Layout<D>::SMEM;
  static std::atomic<bool> done[kMaxCachedDevices];
  cudaError_t e = allow_smem(pass_kernel<D, kStates, kRev, k3>, smem, done);
  if (e != cudaSuccess) return cuda_status(e, "decay_attn (tensor cores)");
  const dim3 grid(a.p.nseg - (kStates && !a.p.end ? 1 : 0), a.p.B * a.p.H);
  e = launch_early(pass_kernel<D, kStates, kRev, k3>, grid, kThreads, smem, st, a);
  return cuda_status(e, "decay_attn (tensor cores) launch");
}

// Sums of a forward pass are exact ones always (the forward hands its state
// out, and a backward makes the same bits again), outputs by themselves a
// forward's always.
template <int D>
static int sums(const Args& a, cudaStream_t st) {
  if (!a.p.reverse) return launch<D, true, false, true>(a, st);
  return a.p.exact ? launch<D, true, true, true>(a, st) : launch<D, true, true, false>(a, st);
}
template <int D>
static int outputs(const Args& a, cudaStream_t st) {
  return a.p.exact ? launch<D, false, false, true>(a, st) : launch<D, false, false, false>(a, st);
}

template <int D, bool k3>
static int launch3(const Args3& a, cudaStream_t st) {
  constexpr int smem = Layout<D>::SMEM;
  static std::atomic<bool> done[kMaxCachedDevices];
  cudaError_t e = allow_smem(bwd_kernel<D, k3>, smem, done);
  if (e != cudaSuccess) return cuda_status(e, "decay_attn_bwd (tensor cores)");
  const int grid = 3 * a.dq.p.nseg * a.dq.p.B * a.dq.p.H;
  e = launch_early(bwd_kernel<D, k3>, dim3(grid), kThreads, smem, st, a);
  return cuda_status(e, "decay_attn_bwd (tensor cores) launch");
}

static int make_args(Args& a, const DecayPass& p, int D, bool states) {
  a.p = p;
  cudaError_t e = make_tmap_bf16(&a.my, p.y, D, p.S, p.H, p.B, p.yv, 64, kSub);
  if (e == cudaSuccess) e = make_tmap_bf16(&a.mz, p.z, D, p.S, p.H, p.B, p.zv, 64, kSub);
  if (e == cudaSuccess && !states) e = make_tmap_bf16(&a.mx, p.x, D, p.S, p.H, p.B, p.xv, 64, kSub);
  if (e == cudaSuccess && !states) e = make_tmap_bf16(&a.mo, p.out, D, p.S, p.H, p.B, p.ov, 64, kSub);
  SCA_REQUIRE(e == cudaSuccess, SCA_ERR_ALIGN, "decay_attn: layout not expressible as a TMA tensor map");
  return SCA_OK;
}

}  // namespace decay_tc

using namespace decay_tc;

int decay_tc_pass(const DecayPass& p, int D, bool states, cudaStream_t stream) {
  Args a;
  const int rc = make_args(a, p, D, states);
  if (rc != SCA_OK) return rc;
  if (states) return D == 64 ? sums<64>(a, stream) : sums<128>(a, stream);
  return D == 64 ? outputs<64>(a, stream) : outputs<128>(a, stream);
}

int decay_tc_backward(const DecayPass& dq, const DecayPass& dv, const DecayPass& dk, int D, cudaStream_t stream) {
  Args3 a;
  int rc;
  if ((rc = make_args(a.dq, dq, D, false)) != SCA_OK || (rc = make_args(a.dv, dv, D, false)) != SCA_OK ||
      (rc = make_args(a.dk, dk, D, false)) != SCA_OK)
    return rc;
  if (dv.exact) return D == 64 ? launch3<64, true>(a, stream) : launch3<128, true>(a, stream);
  return D == 64 ? launch3<64, false>(a, stream) : launch3<128, false>(a, stream);
}

}  // namespace sca
