// Decode attention over a shared prefix and each request's own suffix on the
// tensor cores (bf16).
//
// The keys are cut into tiles of 128.  A unit is what reads one key/value
// head's keys for the same query rows: the prefix for up to two row tiles of
// 128 (the rows of floor(128 / R) whole requests each), or one request's
// suffix for its R rows.  All units' tiles lie on one line, weighted by what
// they cost, and CTA i of G takes the i-th part of it, whatever the lengths:
// a part is a few pieces of units.  Every piece leaves (o, lse) partials,
// merge_kernel finds them by the same arithmetic and joins them.
//
// Two streams of (query rows, S, O) take turns on the tensor cores, each with
// its own softmax warpgroup, so that one's exponentials run under the other's
// products:
//   two row tiles of the prefix: both streams read the same key tiles (each
//     loaded once for 256 rows), stream = row tile;
//   one row tile, or a suffix: the same rows, stream 0 takes the even tiles
//     and stream 1 the odd ones, as partials of their own.
//
//   warps 4-7, 8-11 softmax of streams 0 and 1: thread = query row, all 128
//                   columns of S in one pass, P (bf16) over S in tensor
//                   memory; O rescaled when the row maximum grows by more
//                   than 2^8; warps whose rows are all unused only arrive
//   warp 0          TMA: Q (two buffers), and K, V in the order the MMAs use
//                   them through one ring of five 128-row tiles
//   warp 1          the MMAs: S(0) S(1) | P V(m) S(m + 2) ...
//
// What bounds it: a key tile for two row tiles takes 1.8 us, about 3600 clk, of
// which the tensor pipe works 2048 at D = 128: a stream's scores, softmax (1750
// clk), hand-over (200 to 500: the softmax warps that share a scheduler with
// warp 1 come last) and product follow one another, and at D = 128 tensor
// memory has no room for a second S (at D = 64, 1.5 us a tile, O0 and O1 leave
// 128 columns free).  For one row tile 1.35 us, 7.4 TB/s of keys, as fast as
// they can be read.  64 requests behind 131072 keys, 32 heads on 8, suffixes to 2048: 165
// us, 115 being what the bytes take; 4 requests behind 500 keys 9.7 us in a
// captured graph (otherwise the host bounds it: 10.6 to 12.7 a call).
//
// P is rounded to bf16 for its product with V, as in the framework's causal
// attention: a second part would double that product, half of the tensor
// pipe's work, for errors of 0.0023 of the norm instead of 0.0017.
//
// S(m + 2) is issued after P V(m), and MMAs run in order: when S of a stream
// is there, so is everything that was added to its O before, and the tiles
// that those products read are free.  So one commit serves P V(m) and S(m + 2)
// together, and the softmax warps that see S give the tiles back: a commit
// holds the tensor pipe for about 110 clk (8 MMAs, 512 clk, and one commit
// took 623 in a loop, and two commits 687).
// Tensor memory: S0, S1 (128 columns each), O0, O1 (D each).
#include <cuda.h>

#include "common.cuh"
#include "host_common.h"
#include "launch_util.h"
#include "mma4.cuh"
#include "overlap.cuh"
#include "prefix.h"
#include "ptx.cuh"
#include "tmap.h"

namespace sca {
namespace prefix_tc {

constexpr int BN = 128;
constexpr int kThreads = 384;
constexpr int kProd = 0, kMma = 1;       // the softmax warps are 4 to 11
constexpr int PANEL = 128 * 128;          // 128 rows x 64 bf16, 128-byte swizzle
constexpr int RING = 5;
constexpr float kRescaleLog2 = 8.0f;
// registers: 384 x 168 at launch = 256 x 208 + 128 x 88
constexpr int kRegSoftmax = 208, kRegRoles = 88;
static_assert(256 * kRegSoftmax + 128 * kRegRoles <= kThreads * 168, "register split");
constexpr int kMaxCtas = 160;             // G at most: the merge's tables
// What a tile of one or two row tiles costs, and the start and end of a unit,
// in about 450 clk.  On one box 64 requests behind 131072 keys took 161 us,
// with 6, 8 and 13 (measured before a unit's start was shortened) 164, with 6,
// 9 and 14 163; 13 requests behind 8191 keys 21.4, 21.9 and 22.2.
constexpr int kCostOne = 5, kCostTwo = 8, kCostUnit = 10;

struct Args {
  CUtensorMap mq, mq1, mkp, mvp, mks, mvs;   // queries of nb requests, of one
  PrefixArgs a;
  int32_t nb;          // requests per row tile
  int32_t row_tiles;
  int32_t pairs;       // units per key/value head: pairs of row tiles
  int32_t n_pu, n_su;  // prefix and suffix units
  int32_t tp;          // prefix tiles
  int32_t G;
};

// ---- the line of tiles ----------------------------------------------------
// Places on the line are 32-bit numbers (the host refuses more): a 64-bit
// division is a hundred instructions, and every role does a few.

__host__ __device__ __forceinline__ int head_cost(const Args& k) {   // the prefix's, of one key/value head
  return k.tp * ((k.row_tiles / 2) * kCostTwo + (k.row_tiles & 1) * kCostOne) + k.pairs * kCostUnit;
}
__device__ __forceinline__ int pair_cost(const Args& k) { return k.tp * kCostTwo + kCostUnit; }
// of a request's suffix of T tiles, for one key/value head
__host__ __device__ __forceinline__ int suffix_cost(int T) { return T ? T * kCostOne + kCostUnit : 0; }
__device__ __forceinline__ int suffix_tiles(const Args& k, int b) {
  return (static_cast<int>(suffix_len(k.a, b)) + BN - 1) / BN;
}

// CTA i of G takes [start(i), start(i + 1)) of a line W long.
struct Line {
  int W, G, q, r;
  __device__ __forceinline__ Line(int W_, int G_) : W(W_), G(G_), q(W_ / G_), r(W_ % G_) {}
  __device__ __forceinline__ int start(int i) const { return q * i + r * i / G; }
  // whose part holds `pos`
  __device__ __forceinline__ int cta_of(int pos) const {
    int i = static_cast<int>(__fdividef(static_cast<float>(pos) * static_cast<float>(G), static_cast<float>(W)));
    i = i < G ? i : G - 1;
    while (i + 1 < G && start(i + 1) <= pos) ++i;
    while (i > 0 && start(i) > pos) --i;
    return i;
  }
};
// The tiles [j0, j1) of a unit of T tiles at `at` whose place is in [lo, hi):
// tile j lies at `at` + kCostUnit + j w, the unit's own cost before the first.
__device__ __forceinline__ void part_tiles(int at, int T, bool two, int lo, int hi, int& j0, int& j1) {
  const int first = at + kCostUnit, w = (two ? kCostTwo : kCostOne) - 1;
  const int a = max(lo - first, 0) + w, e = max(hi - first, 0) + w;
  j0 = two ? a / kCostTwo : a / kCostOne;
  j1 = min(T, two ? e / kCostTwo : e / kCostOne);
}

struct Piece {
  int u, b, hk, rt;      // unit, request (suffix), key/value head, first row tile (prefix)
  int j0, nt;            // tiles [j0, j0 + nt)
  bool suffix, two;
};

struct Cursor {
  int lo, hi, at;        // this CTA's part of the line; where unit u starts
  int u;
  __device__ __forceinline__ bool next(const Args& k, Piece& p) {
    const int n = k.n_pu + k.n_su;
    while (at < hi && u < n) {
      p.u = u;
      p.suffix = u >= k.n_pu;
      int T;
      if (p.suffix) {
        p.b = (u - k.n_pu) / k.a.Hkv;
        p.hk = (u - k.n_pu) - p.b * k.a.Hkv;
        p.rt = 0;
        p.two = false;
        T = suffix_tiles(k, p.b);
      } else {
        p.b = 0;
        p.hk = u / k.pairs;
        p.rt = 2 * (u - p.hk * k.pairs);
        p.two = p.rt + 1 < k.row_tiles;
        T = k.tp;
      }
      int a, e;
      part_tiles(at, T, p.two, lo, hi, a, e);
      if (T) at += T * (p.two ? kCostTwo : kCostOne) + kCostUnit;
      ++u;
      if (e > a) {
        p.j0 = a;
        p.nt = e - a;
        return true;
      }
    }
    return false;
  }
};

// Row of the partials of CTA i's piece of unit u, stream s, query row r of
// the stream: unit + CTA counts the pieces in order, so it names one.
__device__ __forceinline__ int64_t part_row(const Args& k, int u, int i, int s, int r) {
  if (u < k.n_pu) return (static_cast<int64_t>(u + i) * 2 + s) * 128 + r;
  const int64_t first = k.n_pu ? static_cast<int64_t>(k.n_pu + k.G) * 256 : 0;
  return first + (static_cast<int64_t>(u - k.n_pu + i) * 2 + s) * k.a.R + r;
}

static int64_t part_rows(int64_t n_pu, int64_t n_su, int64_t G, int64_t R) {
  return (n_pu ? (n_pu + G) * 256 : 0) + (n_su ? (n_su + G) * 2 * R : 0);
}

// ---- partials -------------------------------------------------------------

struct Bars {
  uint64_t q_full[2], q_free[2];
  uint64_t full[RING], free[RING];
  uint64_t s_full[2], p_full[2], o_full[2], o_free[2];
  uint64_t drain;
  Cursor cur;            // behind the first piece
  Piece first;
  int any;               // is there one?
  uint32_t tmem_base;
  int abort;
};

template <int D>
struct Layout {
  static constexpr int TILE = D / 64 * PANEL;
  static constexpr int Q_OFF = 0;
  static constexpr int RING_OFF = 2 * TILE;
  static constexpr int BAR_OFF = RING_OFF + RING * TILE;
  static constexpr int USED = BAR_OFF + static_cast<int>(sizeof(Bars)) + 1024;
  // one CTA per SM (tensor memory is allocated whole)
  static constexpr int SMEM = USED > 120 * 1024 ? USED : 120 * 1024;
  static_assert(SMEM <= 232448, "one CTA's shared memory");
};

// this CTA's part of the line and the unit it starts in (one warp)
SCA_INLINE Cursor find_part(const Args& k, int lane) {
  const int hc = head_cost(k), wp = k.n_pu ? hc * k.a.Hkv : 0;
  int cost = 0;
  if (k.n_su)
    for (int b = lane; b < k.a.B; b += 32) cost += suffix_cost(suffix_tiles(k, b));
  for (int o = 16; o; o >>= 1) cost += __shfl_xor_sync(0xffffffffu, cost, o);
  const Line line(wp + cost * k.a.Hkv, k.G);
  const int lo = line.start(blockIdx.x), hi = line.start(blockIdx.x + 1);
  int u = 0, at = 0;
  if (lo < wp) {
    const int hk = lo / hc, rem = lo - hk * hc, two = pair_cost(k);
    const int rp = min(rem / two, k.pairs - 1);
    u = hk * k.pairs + rp;
    at = hk * hc + rp * two;
  } else {
    u = k.n_pu;
    at = wp;
    for (int b0 = 0; k.n_su && b0 < k.a.B; b0 += 32) {   // requests before the one that holds lo
      const int b = b0 + lane;
      int cum = b < k.a.B ? suffix_cost(suffix_tiles(k, b)) * k.a.Hkv : 0;
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, cum, o);
        if (lane >= o) cum += v;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, at + cum > lo);
      const int cnt = past ? __ffs(past) - 1 : 32;        // lanes wholly before lo
      const int skipped = __shfl_sync(0xffffffffu, cum, cnt ? cnt - 1 : 0);
      if (cnt) at += skipped;
      u = k.n_pu + (b0 + cnt < k.a.B ? b0 + cnt : k.a.B) * k.a.Hkv;
      if (past) break;
    }
  }
  return Cursor{lo, hi, at, u};
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) partials_kernel(const __grid_constant__ Args ka) {
  using L = Layout<D>;
  const PrefixArgs& a = ka.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + L::BAR_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 32 * kProd) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->q_free[i], 1);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_full[i], 4);
      mbar_init(&bars->o_full[i], 1);
      mbar_init(&bars->o_free[i], 4);
    }
    for (int i = 0; i < RING; ++i) {
      mbar_init(&bars->full[i], 1);
      mbar_init(&bars->free[i], 1);
    }
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == kProd) {
    __syncwarp();
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 64 && ka.n_pu) {
    tma_prefetch_map(&ka.mq);
    tma_prefetch_map(&ka.mkp);
    tma_prefetch_map(&ka.mvp);
  }
  if (threadIdx.x == 96 && ka.n_su) {
    tma_prefetch_map(&ka.mq1);
    tma_prefetch_map(&ka.mks);
    tma_prefetch_map(&ka.mvs);
  }
  wait_for_previous();     // the lengths may be an earlier kernel's as well
  // The merge's CTAs may start on SMs that are done, and find their pieces: not
  // earlier, since they read the lengths before they wait for this grid.
  let_next_start();
  volatile int* abort = &bars->abort;
  // loads (one thread of warp kProd): so far, and a piece's queries and first keys
  int it = 0, nq[2] = {0, 0}, turn = 0;
  auto load_q = [&](int buf, const CUtensorMap* m, int n, int b0, int hk) {
    if (nq[buf] > 0 && !wait_or_abort(&bars->q_free[buf], (nq[buf] - 1) & 1, abort)) return false;
    mbar_arrive_expect_tx(&bars->q_full[buf], D / 64 * a.R * 128 * n);
    for (int c = 0; c < D / 64; ++c)
      tma_load_4d(smem + L::Q_OFF + buf * L::TILE + c * PANEL, m, &bars->q_full[buf], 64 * c, 0, b0, hk);
    ++nq[buf];
    return true;
  };
  auto load = [&](const CUtensorMap* m, int tile, int hk, int b) {
    const int st = it % RING;
    if (it >= RING && !wait_or_abort(&bars->free[st], (it / RING - 1) & 1, abort)) return false;
    mbar_arrive_expect_tx(&bars->full[st], L::TILE);
    for (int c = 0; c < D / 64; ++c)
      tma_load_4d(smem + L::RING_OFF + st * L::TILE + c * PANEL, m, &bars->full[st], 64 * c, tile * BN, hk, b);
    ++it;
    return true;
  };
  auto begin = [&](const Piece& p) {
    bool ok;
    if (p.two) {
      ok = load_q(0, &ka.mq, ka.nb, p.rt * ka.nb, p.hk) && load_q(1, &ka.mq, ka.nb, (p.rt + 1) * ka.nb, p.hk);
    } else {
      ok = p.suffix ? load_q(turn, &ka.mq1, 1, p.b, p.hk) : load_q(turn, &ka.mq, ka.nb, p.rt * ka.nb, p.hk);
      turn ^= 1;
    }
    return ok && load(p.suffix ? &ka.mks : &ka.mkp, p.j0, p.hk, p.b);
  };
  if (warp == kProd) {
    // the first piece, found once for all roles, and its loads on their way
    // before anything else: a short call waits for little but this
    Cursor c = find_part(ka, lane);
    if (lane == 0) {
      Piece f = {};
      const bool any = c.next(ka, f);
      bars->cur = c;
      bars->first = f;
      bars->any = any;
      if (any) begin(f);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const uint32_t s0 = smem_u32(smem);
  Cursor cur = bars->cur;
  Piece p = bars->first;
  bool more = bars->any;
  auto wait_all = [&](uint64_t* bar, uint32_t par) { return wait_all_or_abort(bar, par, abort); };

  if (warp < 4) {
    reg_dec<kRegRoles>();
    if (warp == kProd) {
      // ------------------------------------------------------- loads
      if (lane == 0) {
        bool ok = true;
        for (bool begun = true; ok && more; begun = false, more = ok && cur.next(ka, p)) {
          const CUtensorMap *mk = p.suffix ? &ka.mks : &ka.mkp, *mv = p.suffix ? &ka.mvs : &ka.mvp;
          // two row tiles: K0 V0 K1 V1 ...; one: K0 K1 V0 K2 V1 ...
          ok = begun || begin(p);
          for (int j = 0; ok && j < p.nt; ++j) {
            if (p.two) ok = load(mv, p.j0 + j, p.hk, p.b) && (j + 1 == p.nt || load(mk, p.j0 + j + 1, p.hk, p.b));
            else ok = (j + 1 == p.nt || load(mk, p.j0 + j + 1, p.hk, p.b)) && load(mv, p.j0 + j, p.hk, p.b);
          }
        }
        if (*abort) {   // let the copies in flight land before the CTA goes away
          for (int j = it > RING ? it - RING : 0; j < it; ++j) mbar_wait_drain(&bars->full[j % RING], (j / RING) & 1);
          for (int j = 0; j < 2; ++j)
            if (nq[j]) mbar_wait_drain(&bars->q_full[j], (nq[j] - 1) & 1);
        }
      }
    } else if (warp == kMma) {
      // -------------------------------------------------------- MMAs
      constexpr uint32_t id_s = idesc_bf16_f32(128, BN, false, false);
      constexpr uint32_t id_o = idesc_bf16_f32(128, D, false, true);
      int it = 0;                                  // ring place of the piece
      auto advance = [](int& st, int& ph, int n) {   // a place of the ring and its phase, n on
        st += n;
        if (st >= RING) {
          st -= RING;
          ph ^= 1;
        }
      };
      int q_ph = 0, p_ph = 0, o_ph = 3, turn = 0;   // phases, bit s or buffer
      bool ok = true;
      Piece pn;
      while (ok && more) {
        const int M = p.two ? 2 * p.nt : p.nt, qb = p.two ? 0 : turn;
        if (!p.two) turn ^= 1;
        ok = wait_all(&bars->q_full[qb], (q_ph >> qb) & 1) && (!p.two || wait_all(&bars->q_full[1], (q_ph >> 1) & 1));
        q_ph ^= p.two ? 3 : 1 << qb;
        // the places that are next for S and for P V
        int kst = it % RING, kph = (it / RING) & 1, vst = kst, vph = kph;
        advance(vst, vph, p.two || p.nt == 1 ? 1 : 2);
        for (int m = -2; ok && m < M; ++m) {
          const int s = m & 1;
          const uint32_t tS = tmem + 128 * s, tO = tS + 256;
          if (m == 0) more = cur.next(ka, pn);   // its loads' latency under the first softmax
          // P comes last: what is waited for before it costs nothing then
          if (m + 2 < M && !(ok = wait_all(&bars->full[kst], kph))) break;
          if (m >= 0) {
            if (!(ok = wait_all(&bars->full[vst], vph))) break;
            if (m < 2) {   // the stream's O of the piece before has been read
              if (!(ok = wait_all(&bars->o_free[s], (o_ph >> s) & 1))) break;
              o_ph ^= 1 << s;
            }
            const uint64_t vd = sdesc_sw128(s0 + L::RING_OFF + vst * L::TILE, PANEL, 1024);
            if (!p.two) advance(vst, vph, m + 2 == M ? 1 : 2);
            else if (s == 1) advance(vst, vph, 2);
            if (!(ok = wait_all(&bars->p_full[s], (p_ph >> s) & 1))) break;
            p_ph ^= 1 << s;
            tc_fence_after();
            umma4_ts<128>(tO, tS, vd, id_o, m >= 2);
            umma4_ts<128>(tO, tS + 32, sdesc_step(vd, 8192), id_o, 1);
            if (m + 2 >= M) umma_commit_w(&bars->o_full[s]);
          }
          if (m + 2 < M) {
            tc_fence_after();
            const uint64_t qd = sdesc_sw128(s0 + L::Q_OFF + (p.two ? s : qb) * L::TILE, 16, 1024);
            const uint64_t kd = sdesc_sw128(s0 + L::RING_OFF + kst * L::TILE, 16, 1024);
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              umma4_ss<2, 2>(tS, sdesc_step(qd, c * PANEL), sdesc_step(kd, c * PANEL), id_s, c);
            umma_commit_w(&bars->s_full[s]);
            if (!p.two) advance(kst, kph, m < -1 ? 1 : 2);
            else if (s == 1) advance(kst, kph, 2);
          }
        }
        it += 2 * p.nt;
        p = pn;
      }
      // every MMA, and every arrival that goes with one, before the memory goes
      umma_commit_w(&bars->drain);
      mbar_wait_drain(&bars->drain, 0);
    }
  } else {
    // -------------------------------------------------------- softmax
    reg_inc<kRegSoftmax>();
    const int s = (warp >> 2) - 1, row = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + 128 * s + lane_off, tO = tmem + 256 + 128 * s + lane_off;
    const float sl2 = a.scale_log2;
    int it = 0, ns = 0, np = 0;   // ring place of the piece, tiles and pieces of this stream so far
    int turn = 0;                 // query buffer of the next piece of one row tile
    const bool gives = (warp & 3) == 0 && lane == 0;   // gives tiles back to the producer
    bool ok = true;
    Piece pn;
    while (ok && more) {
      const int cnt = p.two ? p.nt : (p.nt + 1 - s) / 2;
      // the row's keys are [0, seen)
      const int len = static_cast<int>(p.suffix ? suffix_len(a, p.b) : a.prefix_len);
      const int rt = p.rt + (p.two ? s : 0);
      const int b = p.suffix ? p.b : rt * ka.nb + row / a.R;
      const bool valid = row < (p.suffix ? a.R : a.R * ka.nb) && b < a.B;
      const bool some = __any_sync(0xffffffffu, valid);
      const int seen = p.suffix ? len - (a.T - 1 - (row % a.R) % a.T) : len;
      float m_used = -INFINITY, l = 0.f;
      const int M = p.two ? 2 * p.nt : p.nt, qb = turn;
      if (!p.two) turn ^= 1;
      // ring places of the next K and V to give back: every second one, or of
      // one row tile (K0 K1 V0 K2 V1 ... V) every fourth, the first K before
      const int first = it % RING;
      auto wrap = [](int st) { return st >= RING ? st - RING : st; };
      int fk = wrap(first + (p.two ? 0 : s)), fv = wrap(first + (p.two ? 1 : 2 + 2 * s));
      for (int k = 0; k < cnt; ++k, ++ns) {
        const int j = p.j0 + (p.two ? k : 2 * k + s);
        const int k0 = j * BN;
        if (!(ok = wait_all(&bars->s_full[s], ns & 1))) break;
        tc_fence_after();
        if (gives && (!p.two || s == 1)) {   // of two row tiles, stream 1 comes second
          const int m = 2 * k + s;
          mbar_arrive(&bars->free[fk]);
          fk = wrap(fk + (p.two ? 2 : (m == 0 ? 3 : 4)));
          if (k > 0) {
            mbar_arrive(&bars->free[fv]);
            fv = wrap(fv + (p.two ? 2 : 4));
          }
          if (m == M - 1) {                  // the piece's last use of its queries
            if (p.two || qb == 0) mbar_arrive(&bars->q_free[0]);
            if (p.two || qb == 1) mbar_arrive(&bars->q_free[1]);
          }
        }
        if (some) {
          const int left = seen - k0;   // columns that the row sees, at most 0 for none
          // columns [n, 32) of 32 to -inf
          auto mask = [](uint32_t (&y)[32], int n) {
            const uint32_t bits = n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(bits & (1u << c))) y[c] = 0xff800000u;
          };
          float2 l0 = make_float2(0.f, 0.f), l1 = make_float2(0.f, 0.f);
          // One pass, 32 columns at a time in a short loop (held in registers
          // all at once they would be four times the code, and fetching code
          // is what a short call waits for).  A row's numbers are relative to
          // 2^m_used, which follows its maximum only when that has grown by
          // more than 2^kRescaleLog2: fp32 sums and bf16 P keep their
          // relative precision at any power of two.
#pragma unroll 1
          for (int h = 0; h < 4; ++h) {
            uint32_t y[32], pk[16];
            tmem_ld32(tS + 32 * h, y);
            tmem_wait_ld32(y);
            if (left < BN) mask(y, left - 32 * h);
            float m0 = __uint_as_float(y[0]), m1 = __uint_as_float(y[1]), m2 = __uint_as_float(y[2]), m3 = __uint_as_float(y[3]);
#pragma unroll
            for (int c = 4; c < 32; c += 4) {
              m0 = fmaxf(m0, __uint_as_float(y[c]));
              m1 = fmaxf(m1, __uint_as_float(y[c + 1]));
              m2 = fmaxf(m2, __uint_as_float(y[c + 2]));
              m3 = fmaxf(m3, __uint_as_float(y[c + 3]));
            }
            const float top = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * sl2;
            const bool need = top > m_used + kRescaleLog2;
            if (__any_sync(0xffffffffu, need)) {
              // (a key that outweighs all others by that much gets P = 1, unrounded)
              const float m_new = need ? top : m_used;
              const float alpha = need ? ex2(m_used - m_new) : 1.f;   // m_used = -inf gives 0
              m_used = m_new;
              l *= alpha;
              const float2 al = make_float2(alpha, alpha), zero = make_float2(0.f, 0.f);
              l0 = ffma2(l0, al, zero);
              l1 = ffma2(l1, al, zero);
              // what is read back below may have been stored by this loop:
              // P, and O at a growth in the 32 columns before
              tmem_wait_st();
              if (k > 0) {
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                  uint32_t r[32];
                  tmem_ld32(tO + c, r);
                  tmem_wait_ld32(r);
#pragma unroll
                  for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
                  tmem_st32(tO + c, r);
                }
              }
              if (h > 0) {   // P so far: rounded once more, at less than 2^-8 of the row's weight
#pragma unroll 1
                for (int c = 0; c < 16 * h; c += 32) {   // (and S that has been read)
                  uint32_t r[32];
                  tmem_ld32(tS + c, r);
                  tmem_wait_ld32(r);
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    r[e] = pack_bf16x2(__uint_as_float(r[e] << 16) * alpha, __uint_as_float(r[e] & 0xffff0000u) * alpha);
                  tmem_st32(tS + c, r);
                }
                tmem_wait_st();   // of an odd number of 16 columns, the next are stored again below
              }
            }
            const float msub = m_used == -INFINITY ? 0.f : m_used;
            const float2 sc2 = make_float2(sl2, sl2), nm2 = make_float2(-msub, -msub);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float2 u = ffma2(make_float2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1])), sc2, nm2);
              const float2 v = ffma2(make_float2(__uint_as_float(y[2 * i + 2]), __uint_as_float(y[2 * i + 3])), sc2, nm2);
              const float2 pu = make_float2(ex2(u.x), ex2(u.y)), pv = make_float2(ex2(v.x), ex2(v.y));
              l0 = fadd2(l0, pu);
              l1 = fadd2(l1, pv);
              pk[i] = pack_bf16x2(pu.x, pu.y);
              pk[i + 1] = pack_bf16x2(pv.x, pv.y);
            }
            tmem_st16(tS + 16 * h, pk);   // over columns that have been read
          }
          const float2 ls = fadd2(l0, l1);
          l += ls.x + ls.y;
          tmem_wait_st();
        }
        if (p.suffix && len - k0 < BN) {
          // the suffix's last tile, and so the piece's: rows of V behind it may hold anything
          const int i = it + 2 * p.nt - 1, st = i % RING, n = len - k0;
          if (!(ok = wait_all(&bars->full[st], (i / RING) & 1))) break;
          uint8_t* v = smem + L::RING_OFF + st * L::TILE;
          for (int e = row; e < (BN - n) * (D / 8); e += 128) {
            const int r = n + e / (D / 8), q = e % (D / 8);
            *reinterpret_cast<uint4*>(v + (q >> 3) * PANEL + r * 128 + (q & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_async_smem();
        }
        tc_fence_before();
        warp_arrive(&bars->p_full[s], lane);
        if (k == 0) more = cur.next(ka, pn);
      }
      if (!ok) break;
      if (cnt == 0) more = cur.next(ka, pn);
      if (cnt > 0) {
        if (!(ok = wait_all(&bars->o_full[s], np & 1))) break;
        ++np;
        tc_fence_after();
        // one row tile's last V comes right behind its K
        if (gives && (!p.two || s == 1))
          mbar_arrive(&bars->free[!p.two && 2 * (cnt - 1) + s == M - 1 ? wrap(fv + RING - 1) : fv]);
        if (some) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          const int64_t at = part_row(ka, p.u, blockIdx.x, s, row);
          float* po = a.part_o + at * D;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t r[32];
            tmem_ld32(tO + c, r);
            tmem_wait_ld32(r);
            if (valid) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(po + c + e) =
                    make_float4(__uint_as_float(r[e]) * inv, __uint_as_float(r[e + 1]) * inv,
                                __uint_as_float(r[e + 2]) * inv, __uint_as_float(r[e + 3]) * inv);
            }
          }
          if (valid) a.part_lse[at] = l == 0.f ? -INFINITY : m_used + log2f(l);
        }
        tc_fence_before();
        warp_arrive(&bars->o_free[s], lane);
      }
      it += 2 * p.nt;
      p = pn;
    }
  }

  tc_fence_before();
  __syncthreads();
  report_abort(abort, a.status);
  if (warp == kProd) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---- merge ----------------------------------------------------------------

// A query row's partials are those of the pieces that its prefix unit and its
// suffix unit were cut into, the same list for all rows of a request and
// key/value head.  A CTA joins ROWS of them, 4 / ROWS warps each: four where
// rows are many and making their lists would take longest; one where they are
// few and reading the partials one after the other would.
template <int D, int ROWS>
__global__ void __launch_bounds__(128) merge_kernel(const __grid_constant__ Args k) {
  constexpr int W4 = D / 4, WPR = 4 / ROWS, NG = WPR * (32 / W4);   // threads, warps and groups of threads a row
  __shared__ float sw[ROWS][4 * kMaxCtas];
  __shared__ int64_t srow[4 * kMaxCtas];   // the first row's; -1: that piece has no such partial
  __shared__ float4 so[ROWS][NG][W4];
  __shared__ float red[4], red2[4];
  __shared__ int tot[4], before[4];
  const PrefixArgs& a = k.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (a.R + ROWS - 1) / ROWS, bh = static_cast<int>(blockIdx.x) / per;
  const int r0 = (static_cast<int>(blockIdx.x) - bh * per) * ROWS;
  const int b = bh / a.Hkv, hk = bh - b * a.Hkv;
  int t_all = 0, t_before = 0;   // costs of all suffixes, and of those before this request's
  if (k.n_su)
    for (int i = tid; i < a.B; i += 128) {
      const int t = suffix_cost(suffix_tiles(k, i));
      t_all += t;
      if (i < b) t_before += t;
    }
  for (int o = 16; o; o >>= 1) {
    t_all += __shfl_xor_sync(0xffffffffu, t_all, o);
    t_before += __shfl_xor_sync(0xffffffffu, t_before, o);
  }
  if (lane == 0) {
    tot[warp] = t_all;
    before[warp] = t_before;
  }
  __syncthreads();
  t_all = tot[0] + tot[1] + tot[2] + tot[3];
  t_before = before[0] + before[1] + before[2] + before[3];
  const int hc = head_cost(k), wp = k.n_pu ? hc * a.Hkv : 0;
  const Line line(max(wp + t_all * a.Hkv, 1), k.G);
  let_next_start();
  int n = 0;   // entries so far
  auto list = [&](int u, int at, int T, bool two, int s_two, int pr) {
    if (T == 0) return;
    const int first = at + kCostUnit;
    const int i0 = line.cta_of(first), i1 = line.cta_of(first + (T - 1) * (two ? kCostTwo : kCostOne));
    const int cnt = (i1 - i0 + 1) * (two ? 1 : 2);
    for (int e = tid; e < cnt; e += 128) {
      const int i = i0 + (two ? e : e >> 1), s = two ? s_two : e & 1;
      int j0, j1;
      part_tiles(at, T, two, line.start(i), line.start(i + 1), j0, j1);
      const bool has = j1 - j0 > (two ? 0 : s);   // stream 1 of a single tile has none
      srow[n + e] = has ? part_row(k, u, i, s, pr) : -1;
    }
    n += cnt;
  };
  if (k.n_pu) {
    const int rt = b / k.nb, rp = rt / 2;
    const bool two = 2 * rp + 1 < k.row_tiles;
    list(hk * k.pairs + rp, hk * hc + rp * pair_cost(k), k.tp, two, rt & 1, (b % k.nb) * a.R + r0);
  }
  if (k.n_su) {
    const int T = suffix_tiles(k, b);
    list(k.n_pu + b * a.Hkv + hk, wp + t_before * a.Hkv + hk * suffix_cost(T), T, false, 0, r0);
  }
  __syncthreads();
  wait_for_previous();   // the partials are there
  const int rw = warp / WPR, part = warp % WPR;
  const bool valid = r0 + rw < a.R;
  // one number a warp, joined over the row's warps in a fixed order
  auto join = [&](float v, float* to, auto f) {
    for (int o = 16; o; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (WPR == 1) {
      __syncwarp();
      return v;
    }
    if (lane == 0) to[warp] = v;
    __syncthreads();
    v = to[rw * WPR];
    for (int i = 1; i < WPR; ++i) v = f(v, to[rw * WPR + i]);
    return v;
  };
  float m = -INFINITY;
  for (int e = 32 * part + lane; e < n; e += 32 * WPR) {
    const float v = valid && srow[e] >= 0 ? a.part_lse[srow[e] + rw] : -INFINITY;
    sw[rw][e] = v;
    m = fmaxf(m, v);
  }
  m = join(m, red, [](float x, float y) { return fmaxf(x, y); });
  const float mm = m == -INFINITY ? 0.f : m;
  float total = 0.f;
  for (int e = 32 * part + lane; e < n; e += 32 * WPR) {
    const float w = ex2(sw[rw][e] - mm);   // 0 where a piece has nothing for the row
    total += w;
    sw[rw][e] = w;
  }
  total = join(total, red2, [](float x, float y) { return x + y; });
  const int g = part * (32 / W4) + lane / W4, c = lane % W4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int e = g; e < n; e += NG) {
    const float w = sw[rw][e];
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (w != 0.f) v = reinterpret_cast<const float4*>(a.part_o + (srow[e] + rw) * D)[c];
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
  }
  if (NG > 1) {
    so[rw][g][c] = acc;
    if (WPR > 1) __syncthreads();
    else __syncwarp();
  }
  if (g != 0 || !valid) return;
#pragma unroll
  for (int i = 1; i < NG; ++i) {
    const float4 v = so[rw][i][c];
    acc.x += v.x;
    acc.y += v.y;
    acc.z += v.z;
    acc.w += v.w;
  }
  const float inv = total == 0.f ? 0.f : 1.f / total;
  uint2 out;
  out.x = pack_bf16x2(acc.x * inv, acc.y * inv);
  out.y = pack_bf16x2(acc.z * inv, acc.w * inv);
  const int64_t row = static_cast<int64_t>(bh) * a.R + r0 + rw;
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + row * D + 4 * c) = out;
  if (c == 0) a.lse[row] = total == 0.f ? -INFINITY : (mm + log2f(total)) * kLn2;
}

template <int D>
static cudaError_t launch(const Args& k, cudaStream_t st) {
  using L = Layout<D>;
  static std::atomic<bool> done[kMaxCachedDevices];
  cudaError_t e = allow_smem(partials_kernel<D>, L::SMEM, done);
  if (e != cudaSuccess) return e;
  if ((e = launch_early(partials_kernel<D>, dim3(k.G), kThreads, L::SMEM, st, k)) != cudaSuccess) return e;
  // Four rows a CTA where rows are many (eight times the CTAs of the partials;
  // then few pieces are a row's): 2048 rows of 20 pieces 167 us instead of
  // 170, 780 rows 26.2 instead of 21.8.
  const int bh = k.a.B * k.a.Hkv;
  if (k.a.R > 1 && bh * k.a.R >= 8 * k.G)
    return launch_early(merge_kernel<D, 4>, dim3(static_cast<unsigned>(bh * ((k.a.R + 3) / 4))), 128, 0, st, k);
  return launch_early(merge_kernel<D, 1>, dim3(static_cast<unsigned>(bh * k.a.R)), 128, 0, st, k);
}

}  // namespace prefix_tc

using namespace prefix_tc;

static Args units(int B, int Hkv, int R, int64_t prefix_len, int64_t suffix_cap, int sms) {
  Args k = {};
  k.nb = 128 / R;
  k.row_tiles = (B + k.nb - 1) / k.nb;
  k.pairs = (k.row_tiles + 1) / 2;
  k.tp = static_cast<int>((prefix_len + BN - 1) / BN);
  k.n_pu = k.tp ? Hkv * k.pairs : 0;
  k.n_su = suffix_cap ? B * Hkv : 0;
  const int64_t tiles = static_cast<int64_t>(k.n_pu) * k.tp + static_cast<int64_t>(k.n_su) * ((suffix_cap + BN - 1) / BN);
  const int64_t most = sms < kMaxCtas ? sms : kMaxCtas;
  // a CTA a tile at most: half as many took 15.2 us a call instead of 12.7 for
  // 4 requests behind 500 keys (64 tiles), three times as many 15.2 as well
  k.G = static_cast<int>(tiles < most ? (tiles < 1 ? 1 : tiles) : most);
  return k;
}

int64_t prefix_tc_workspace(int B, int Hkv, int R, int D, int64_t prefix_len, int64_t suffix_cap, int sms) {
  const Args k = units(B, Hkv, R, prefix_len, suffix_cap, sms);
  return part_rows(k.n_pu, k.n_su, k.G, R) * (D + 1) * 4;
}

int prefix_tc_decode(const PrefixArgs& a, int D, int sms, float* ws, cudaStream_t stream) {
  Args k = units(a.B, a.Hkv, a.R, a.prefix_len, a.suffix_cap, sms);
  const double line = static_cast<double>(k.n_pu) * (static_cast<double>(k.tp) * kCostTwo + kCostUnit) +
                      static_cast<double>(k.n_su) * (a.suffix_cap / 128.0 * kCostOne + kCostOne + kCostUnit);
  SCA_REQUIRE(line < 2e9, SCA_ERR_UNSUPPORTED, "prefix_attn_decode: more than about 2^28 tiles of 128 keys");
  k.a = a;
  k.a.n_suffix = k.n_su;   // suffix_len: whether there are lengths
  k.a.part_o = ws;
  k.a.part_lse = ws + part_rows(k.n_pu, k.n_su, k.G, a.R) * D;
  const View q{static_cast<int64_t>(a.R) * D, a.q_b, D};   // rows, then requests, then key/value heads
  cudaError_t e = make_tmap_bf16_box(&k.mq, a.q, D, a.R, a.B, a.Hkv, q, 64, a.R, k.nb);
  if (e == cudaSuccess) e = make_tmap_bf16_box(&k.mq1, a.q, D, a.R, a.B, a.Hkv, q, 64, a.R, 1);
  if (e == cudaSuccess && k.n_pu) {
    e = make_tmap_bf16(&k.mkp, a.kp, D, a.prefix_len, a.Hkv, 1, a.pv, 64, BN);
    if (e == cudaSuccess) e = make_tmap_bf16(&k.mvp, a.vp, D, a.prefix_len, a.Hkv, 1, a.pv, 64, BN);
  }
  if (e == cudaSuccess && k.n_su) {
    e = make_tmap_bf16(&k.mks, a.ks, D, a.suffix_cap, a.Hkv, a.B, a.sv, 64, BN);
    if (e == cudaSuccess) e = make_tmap_bf16(&k.mvs, a.vs, D, a.suffix_cap, a.Hkv, a.B, a.sv, 64, BN);
  }
  SCA_REQUIRE(e == cudaSuccess, SCA_ERR_ALIGN, "prefix_attn_decode: layout not expressible as a TMA tensor map");
  return cuda_status(D == 64 ? launch<64>(k, stream) : launch<128>(k, stream), "prefix_attn_decode (tensor cores)");
}

}  // namespace sca
