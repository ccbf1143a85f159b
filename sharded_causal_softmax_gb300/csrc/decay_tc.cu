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
// each; outputs are bf16 as well).  The state itself loses nothing: y' is an
// fp32 number, taken apart into three bf16 parts of eight bits, and U is the
// sum of three products, as exact as an fp32 sum.  (Two parts leave 2.6e-6 of
// it, ten times what fp32 sums do.)
//
// Roles (18 warps):
//   warps 0-7   thread = row t, half of the columns each: M to P, O out
//   warps 8-15  thread = feature of y, half of the columns each: y' into
//               tensor memory (transposed, as U's A operand), the state
//   warp 16     TMA loads of X, Y, Z (two stages) and stores of O, which is
//               staged over its chunk's X
//   warp 17     the MMAs, one elected lane issuing
//
// Tensor memory (512 columns): M 128 (P over its columns 0-31 and 64-95, the
// third part of y' over 32-63 and 96-127), O 128, U 128, y' parts one and
// two 64 each.  Shared memory: two stages of X, Y, Z (192 KB at D = 128) and
// S as bf16 (32 KB).
//
// At D = 64 U's A operand has 64 of 128 lanes: the others hold whatever the
// tensor memory did, and the rows of U that come of them are not read.
#include <cuda.h>

#include <type_traits>

#include "common.cuh"
#include "decay.h"
#include "host_common.h"
#include "ptx.cuh"
#include "tmap.h"

namespace sca {
namespace decay_tc {

constexpr int kSub = kDecaySub;
constexpr int kThreads = 576;
constexpr int kConv = 256;                  // threads of a converter group
constexpr int kProdWarp = 16, kMmaWarp = 17;
constexpr int PANEL = kSub * 128;           // 128 rows x 64 bf16, 128-byte swizzle

struct Bars {
  uint64_t yz_full[2], x_full[2], yz_free[2], out_staged[2];
  uint64_t m_full, m_read;      // M in tensor memory; read out of it
  uint64_t s_full;              // the chunk's start state (bf16) in shared memory
  uint64_t o1_full, o2_full;    // X S done; P Z done
  uint64_t o_free;              // P Z read
  uint64_t p_full;              // P in tensor memory and X S read
  uint64_t k_full;              // y' in tensor memory, rows of Z behind the sequence zeroed
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
  static constexpr int W_OFF = TAB_OFF + 260 * 4;         // weights of a full chunk's rows
  static constexpr int BAR_OFF = W_OFF + kSub * 4;
  static constexpr int SMEM = BAR_OFF + static_cast<int>(sizeof(Bars)) + 1024;
  static_assert(SMEM <= 232448, "one CTA's shared memory");
};

struct Args {
  CUtensorMap mx, my, mz, mo;
  DecayPass p;
};

SCA_INLINE void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

SCA_INLINE void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               SCA_I8(r, 0)
               : "memory");
}

// a pair as three bf16 parts each: x = hi + mid + lo up to 2^-24 x
SCA_INLINE void split3(float x0, float x1, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = pack_bf16x2(x0, x1);
  x0 -= __uint_as_float(hi << 16);
  x1 -= __uint_as_float(hi & 0xffff0000u);
  mid = pack_bf16x2(x0, x1);
  x0 -= __uint_as_float(mid << 16);
  x1 -= __uint_as_float(mid & 0xffff0000u);
  lo = pack_bf16x2(x0, x1);
}

template <int D, bool kStates, bool kRev>
__global__ void __launch_bounds__(kThreads, 1) pass_kernel(const __grid_constant__ Args ka) {
  using L = Layout<D>;
  const DecayPass& p = ka.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + L::BAR_OFF);
  float* tab = reinterpret_cast<float*>(smem + L::TAB_OFF);
  float* wfull = reinterpret_cast<float*>(smem + L::W_OFF);

  const int seg = blockIdx.x, bh = blockIdx.y, b = bh / p.H, h = bh % p.H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float g = p.log_decay[h];
  const int64_t len = decay_len(p, b);
  const DecayRows rows = decay_rows(p, seg, len);
  const int nchunk = static_cast<int>((rows.hi - rows.lo + kSub - 1) / kSub);
  const bool want_end = kStates || (p.end != nullptr && seg == p.nseg - 1);
  // first row and number of rows of chunk c (processing order)
  auto row_of = [&](int c) { return static_cast<int>(rows.lo) + (kRev ? nchunk - 1 - c : c) * kSub; };
  auto n_of = [&](int c) { return static_cast<int>(min64(kSub, rows.hi - row_of(c))); };
  const int delta0 = kRev && !kStates && rows.s1 >= len ? 1 : 0;   // power taken off in the first chunk

  if (threadIdx.x < 129) {
    const int d = threadIdx.x;
    const float w = decay_pow(g, d);
    tab[128 + d] = w;
    if (d < 128) {
      tab[d] = 0.f;
      wfull[kRev ? d : 127 - d] = w;
    }
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->yz_full[i], 1);
      mbar_init(&bars->x_full[i], 1);
      mbar_init(&bars->yz_free[i], 1);
      mbar_init(&bars->out_staged[i], kConv);
    }
    mbar_init(&bars->m_full, 1);
    mbar_init(&bars->m_read, kConv);
    mbar_init(&bars->s_full, kConv);
    mbar_init(&bars->o1_full, 1);
    mbar_init(&bars->o2_full, 1);
    mbar_init(&bars->o_free, kConv);
    mbar_init(&bars->p_full, kConv);
    mbar_init(&bars->k_full, kConv);
    mbar_init(&bars->u_full, 1);
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const uint32_t tM = tmem, tO = tmem + 128, tU = tmem + 256, tK0 = tmem + 384, tK1 = tmem + 448;
  volatile int* abort = &bars->abort;
  int* status = p.status;
  const uint32_t s0 = smem_u32(smem);
  auto wait_all = [&](uint64_t* bar, uint32_t par) {
    return __all_sync(0xffffffffu, mbar_wait(bar, par, abort, status));
  };

  if (warp == kProdWarp) {
    // ------------------------------------------------ loads and stores
    if (lane == 0) {
      tma_prefetch_map(&ka.my);
      tma_prefetch_map(&ka.mz);
      if (!kStates) {
        tma_prefetch_map(&ka.mx);
        tma_prefetch_map(&ka.mo);
      }
      auto load = [&](uint64_t* bar, uint8_t* to, const CUtensorMap* m, int row) {
        for (int k = 0; k < D / 64; ++k) tma_load_4d(to + k * PANEL, m, bar, 64 * k, row, h, b);
      };
      // chunk c's outputs, staged over its X, and X's stage free again
      auto store = [&](int c) -> bool {
        if (!mbar_wait(&bars->out_staged[c & 1], (c >> 1) & 1, abort, status)) return false;
        for (int k = 0; k < D / 64; ++k)
          tma_store_4d(&ka.mo, smem + (c & 1) * L::STAGE + k * PANEL, 64 * k, row_of(c), h, b);
        bulk_commit();
        bulk_wait_read<0>();
        return true;
      };
      int c = 0, nx = 0;   // chunks whose Y, Z and whose X were asked for
      for (; c < nchunk; ++c) {
        const int s = c & 1;
        uint8_t* st = smem + s * L::STAGE;
        if (c >= 2 && !mbar_wait(&bars->yz_free[s], ((c >> 1) + 1) & 1, abort, status)) break;
        mbar_arrive_expect_tx(&bars->yz_full[s], 2 * L::TILE);
        load(&bars->yz_full[s], st + L::TILE, &ka.my, row_of(c));
        load(&bars->yz_full[s], st + 2 * L::TILE, &ka.mz, row_of(c));
        if (!kStates) {
          if (c >= 2 && !store(c - 2)) {
            ++c;
            break;
          }
          mbar_arrive_expect_tx(&bars->x_full[s], L::TILE);
          load(&bars->x_full[s], st, &ka.mx, row_of(c));
          ++nx;
        }
      }
      if (!kStates && !*abort)
        for (int j = nchunk > 2 ? nchunk - 2 : 0; j < nchunk; ++j)
          if (!store(j)) break;
      if (*abort) {   // let the copies in flight land before the CTA goes away
        for (int j = (c > 2 ? c - 2 : 0); j < c; ++j) mbar_wait_drain(&bars->yz_full[j & 1], (j >> 1) & 1);
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
      const int s = c & 1;
      const bool need_u = want_end || c + 1 < nchunk;
      const uint32_t sX = s0 + s * L::STAGE, sY = sX + L::TILE, sZ = sY + L::TILE;
      const uint64_t zd = sdesc_sw128(sZ, PANEL, 1024);
      if (!(ok = wait_all(&bars->yz_full[s], (c >> 1) & 1))) break;
      auto issue_u = [&]() -> bool {
        if (!wait_all(&bars->k_full, c & 1)) return false;
        tc_fence_after();
        if (need_u) {
          // rows [16 kk, 16 kk + 16) of y': eight columns of each part
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) umma_ts_w(tU, tK0 + 8 * kk, sdesc_step(zd, kk * 2048), id_o, kk > 0 ? 1u : 0u);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) umma_ts_w(tU, tK1 + 8 * kk, sdesc_step(zd, kk * 2048), id_o, 1u);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_ts_w(tU, tM + 32 + 64 * (kk >> 2) + 8 * (kk & 3), sdesc_step(zd, kk * 2048), id_o, 1u);
          umma_commit_w(&bars->u_full);
        }
        return true;
      };
      if (kStates) {
        if (!(ok = issue_u())) break;
        if (c + 2 < nchunk) umma_commit_w(&bars->yz_free[s]);
        continue;
      }
      if (!(ok = wait_all(&bars->x_full[s], (c >> 1) & 1))) break;
      tc_fence_after();
      {
        const uint64_t xd = sdesc_sw128(sX, 16, 1024), yd = sdesc_sw128(sY, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * PANEL + (kk & 3) * 32;
          umma_ss_w(tM, sdesc_step(xd, off), sdesc_step(yd, off), id_m, kk > 0 ? 1u : 0u);
        }
        umma_commit_w(&bars->m_full);
        if (!(ok = wait_all(&bars->s_full, c & 1))) break;
        if (c > 0 && !(ok = wait_all(&bars->o_free, (c - 1) & 1))) break;
        tc_fence_after();
        const uint64_t sd = sdesc_sw128(s0 + L::S_OFF, L::SPANEL, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * PANEL + (kk & 3) * 32;
          umma_ss_w(tO, sdesc_step(xd, off), sdesc_step(sd, kk * 2048), id_o, kk > 0 ? 1u : 0u);
        }
        umma_commit_w(&bars->o1_full);
      }
      // U or P Z, whichever is ready first; behind a ragged chunk's zeroing of Z, U's wait comes first
      const bool u_first = n_of(c) < kSub || __all_sync(0xffffffffu, mbar_try_wait(&bars->k_full, c & 1));
      if (u_first && !(ok = issue_u())) break;
      if (!(ok = wait_all(&bars->p_full, c & 1))) break;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        umma_ts_w(tO, tM + 64 * (kk >> 2) + 8 * (kk & 3), sdesc_step(zd, kk * 2048), id_o, kk > 0 ? 1u : 0u);
      umma_commit_w(&bars->o2_full);
      if (!u_first && !(ok = issue_u())) break;
      // nobody waits for the last two: an arrival must not outlive the CTA
      if (c + 2 < nchunk) umma_commit_w(&bars->yz_free[s]);
    }
    if (!ok || *abort) {   // every MMA issued has finished before the memory goes
      umma_commit_w(&bars->drain);
      mbar_wait_drain(&bars->drain, 0);
    }
  } else if (warp < 8) {
    // ------------------------------------------- rows: M to P, outputs
    if (!kStates) {
      const int q4 = warp & 3, half = warp >> 2;
      const int t = q4 * 32 + lane;
      const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
      bool ok = true;
      for (int c = 0; ok && c < nchunk; ++c) {
        const int n = n_of(c), delta = c == 0 ? delta0 : 0;
        if (!(ok = wait_all(&bars->m_full, c & 1))) break;
        tc_fence_after();
        {
          uint32_t v[64], pk[32];
          tmem_ld32(tM + lane_off + 64 * half, v);
          tmem_ld32(tM + lane_off + 64 * half + 32, v + 32);
          tmem_wait_ld32(v);
          tmem_wait_ld32(v + 32);
          tc_fence_before();
          mbar_arrive(&bars->m_read);
          // column j is row s = 64 half + j: kept for j in [j0, j1)
          const int at = t - 64 * half;
          const int j0 = kRev ? at : 0, j1 = kRev ? n - 64 * half : at + 1;
          const float* w = tab + 128 + (kRev ? -at : at);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float x[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int j = 2 * i + e;
              const float y = __uint_as_float(v[j]) * w[kRev ? j : -j];
              x[e] = j >= j0 && j < j1 ? y : 0.f;
            }
            pk[i] = pack_bf16x2(x[0], x[1]);
          }
          tmem_st32(tM + lane_off + 64 * half, pk);
        }
        const int rho = kRev ? n - 1 - t : t;
        const bool live = t < n;
        const float f = live ? p.si * tab[128 + rho + 1 - delta] : 0.f;
        if (!(ok = wait_all(&bars->o1_full, c & 1))) break;
        tc_fence_after();
        uint32_t o1[D / 2];
#pragma unroll
        for (int k = 0; k < D / 2; k += 32) tmem_ld32(tO + lane_off + (D / 2) * half + k, o1 + k);
#pragma unroll
        for (int k = 0; k < D / 2; k += 32) tmem_wait_ld32(o1 + k);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars->p_full);
        if (!(ok = wait_all(&bars->o2_full, c & 1))) break;
        tc_fence_after();
        uint8_t* dst = smem + (c & 1) * L::STAGE + t * 128;
#pragma unroll
        for (int k = 0; k < D / 2; k += 32) {
          uint32_t o2[32];
          tmem_ld32(tO + lane_off + (D / 2) * half + k, o2);
          tmem_wait_ld32(o2);
          if (k + 32 == D / 2) {
            tc_fence_before();
            mbar_arrive(&bars->o_free);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {   // eight columns: one 16-byte chunk of the swizzled row
            uint32_t r[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i = 8 * q + 2 * e;
              const float x0 = fmaf(f, __uint_as_float(o1[k + i]), p.so * __uint_as_float(o2[i]));
              const float x1 = fmaf(f, __uint_as_float(o1[k + i + 1]), p.so * __uint_as_float(o2[i + 1]));
              r[e] = live ? pack_bf16x2(x0, x1) : 0u;
            }
            const int col = (D / 2) * half + k + 8 * q;
            *reinterpret_cast<uint4*>(dst + (col >> 6) * PANEL + ((((col & 63) >> 3) ^ (t & 7)) << 4)) =
                make_uint4(r[0], r[1], r[2], r[3]);
          }
        }
        fence_async_smem();
        mbar_arrive(&bars->out_staged[c & 1]);
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
    const int q4 = warp & 3, half = (warp >> 2) & 1;
    const int f = q4 * 32 + lane;      // feature of y: row of the state
    const bool has = f < D;            // warp-uniform
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    const int tid = threadIdx.x - 256;
    float run[D / 2];                  // S[f][(D/2) half + u]
    const float* from = nullptr;
    if (!kStates) from = p.seg ? p.seg + (static_cast<int64_t>(bh) * p.nseg + seg) * D * D
                               : (p.init ? p.init + b * p.init_b + static_cast<int64_t>(h) * D * D : nullptr);
#pragma unroll
    for (int u = 0; u < D / 2; ++u) run[u] = 0.f;
    if (from && has) {
      if (p.transposed) {
#pragma unroll
        for (int u = 0; u < D / 2; ++u) run[u] = from[((D / 2) * half + u) * D + f];
      } else {
#pragma unroll
        for (int u = 0; u < D / 2; u += 4) {
          const float4 v = *reinterpret_cast<const float4*>(from + f * D + (D / 2) * half + u);
          run[u] = v.x; run[u + 1] = v.y; run[u + 2] = v.z; run[u + 3] = v.w;
        }
      }
    }
    // S as bf16 for X S
    auto put_state = [&]() {
      if (has) {
        uint8_t* dst = smem + L::S_OFF + f * 128;
#pragma unroll
        for (int u = 0; u < D / 2; u += 8) {
          const int col = (D / 2) * half + u;
          *reinterpret_cast<uint4*>(dst + (col >> 6) * L::SPANEL + ((((col & 63) >> 3) ^ (f & 7)) << 4)) =
              make_uint4(pack_bf16x2(run[u], run[u + 1]), pack_bf16x2(run[u + 2], run[u + 3]),
                         pack_bf16x2(run[u + 4], run[u + 5]), pack_bf16x2(run[u + 6], run[u + 7]));
        }
      }
      fence_async_smem();
      mbar_arrive(&bars->s_full);
    };
    bool ok = true;
    for (int c = 0; ok && c < nchunk; ++c) {
      const int s = c & 1, n = n_of(c), delta = c == 0 ? delta0 : 0;
      const bool need_u = want_end || c + 1 < nchunk;
      if (!kStates) put_state();
      if (!(ok = wait_all(&bars->yz_full[s], (c >> 1) & 1))) break;
      uint8_t* sY = smem + s * L::STAGE + L::TILE;
      if (n < kSub) {   // rows of Z behind the sequence may hold anything
        uint8_t* sZ = sY + L::TILE;
        for (int e = tid; e < (kSub - n) * (D / 8); e += kConv) {
          const int r = n + e / (D / 8), q = e % (D / 8);
          *reinterpret_cast<uint4*>(sZ + (q >> 3) * PANEL + r * 128 + (q & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
      }
      if (!kStates && !(ok = wait_all(&bars->m_read, c & 1))) break;
      if (need_u && has) {
        const uint8_t* yb = sY + (f >> 6) * PANEL + (f & 7) * 2;
        int off[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) off[k] = (((f & 63) >> 3) ^ k) << 4;
        auto conv = [&](auto ragged) {
          constexpr bool kRagged = decltype(ragged)::value;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t hi[8], mid[8], lo[8];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const int r0 = 64 * half + 16 * q + 2 * i;   // rows r0 .. r0 + 3
              float w[4];
              if (!kRagged) {
                const float4 v = *reinterpret_cast<const float4*>(wfull + r0);
                w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
              }
              float x[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int r = r0 + e;
                const uint32_t y = *reinterpret_cast<const uint16_t*>(yb + r * 128 + off[(2 * i + e) & 7]);
                if (kRagged) x[e] = r < n ? __uint_as_float(y << 16) * tab[128 + (kRev ? r : n - 1 - r)] : 0.f;
                else x[e] = __uint_as_float(y << 16) * w[e];
              }
              split3(x[0], x[1], hi[i], mid[i], lo[i]);
              split3(x[2], x[3], hi[i + 1], mid[i + 1], lo[i + 1]);
            }
            tmem_st8(tK0 + lane_off + 32 * half + 8 * q, hi);
            tmem_st8(tK1 + lane_off + 32 * half + 8 * q, mid);
            tmem_st8(tM + lane_off + 32 + 64 * half + 8 * q, lo);
          }
        };
        if (n == kSub) conv(std::false_type{});
        else conv(std::true_type{});
        tmem_wait_st();
      }
      tc_fence_before();
      mbar_arrive(&bars->k_full);
      if (need_u) {
        if (!(ok = wait_all(&bars->u_full, c & 1))) break;
        tc_fence_after();
        const float carry = tab[128 + n - delta];
        if (has) {
#pragma unroll
          for (int k = 0; k < D / 2; k += 32) {
            uint32_t v[32];
            tmem_ld32(tU + lane_off + (D / 2) * half + k, v);
            tmem_wait_ld32(v);
#pragma unroll
            for (int u = 0; u < 32; ++u) run[k + u] = fmaf(carry, run[k + u], p.us * __uint_as_float(v[u]));
          }
        }
        tc_fence_before();
      }
    }
    if (ok && want_end && has) {
      float* to = kStates ? p.seg + (static_cast<int64_t>(bh) * p.nseg + seg) * D * D
                          : p.end + static_cast<int64_t>(bh) * D * D;
      const float mul = !kStates && kRev && len > 0 ? tab[129] : 1.f;
      if (!kStates && p.transposed) {
#pragma unroll
        for (int u = 0; u < D / 2; ++u) to[((D / 2) * half + u) * D + f] = mul * run[u];
      } else {
#pragma unroll
        for (int u = 0; u < D / 2; u += 4)
          *reinterpret_cast<float4*>(to + f * D + (D / 2) * half + u) =
              make_float4(mul * run[u], mul * run[u + 1], mul * run[u + 2], mul * run[u + 3]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool kStates, bool kRev>
static int launch(const Args& a, cudaStream_t st) {
  constexpr int smem = Layout<D>::SMEM;
  cudaError_t e = cudaFuncSetAttribute(pass_kernel<D, kStates, kRev>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_status(e, "decay_attn (tensor cores)");
  const dim3 grid(a.p.nseg - (kStates ? 1 : 0), a.p.B * a.p.H);
  pass_kernel<D, kStates, kRev><<<grid, kThreads, smem, st>>>(a);
  return cuda_status(cudaGetLastError(), "decay_attn (tensor cores) launch");
}

template <int D>
static int by_kind(const Args& a, bool states, cudaStream_t st) {
  if (states) return a.p.reverse ? launch<D, true, true>(a, st) : launch<D, true, false>(a, st);
  return a.p.reverse ? launch<D, false, true>(a, st) : launch<D, false, false>(a, st);
}

}  // namespace decay_tc

int decay_tc_pass(const DecayPass& p, int D, bool states, cudaStream_t stream) {
  using namespace decay_tc;
  Args a;
  a.p = p;
  cudaError_t e = make_tmap_bf16(&a.my, p.y, D, p.S, p.H, p.B, p.yv, 64, kSub);
  if (e == cudaSuccess) e = make_tmap_bf16(&a.mz, p.z, D, p.S, p.H, p.B, p.zv, 64, kSub);
  if (e == cudaSuccess && !states) e = make_tmap_bf16(&a.mx, p.x, D, p.S, p.H, p.B, p.xv, 64, kSub);
  if (e == cudaSuccess && !states) e = make_tmap_bf16(&a.mo, p.out, D, p.S, p.H, p.B, p.ov, 64, kSub);
  SCA_REQUIRE(e == cudaSuccess, SCA_ERR_ALIGN, "decay_attn: layout not expressible as a TMA tensor map");
  return D == 64 ? by_kind<64>(a, states, stream) : by_kind<128>(a, states, stream);
}

}  // namespace sca
