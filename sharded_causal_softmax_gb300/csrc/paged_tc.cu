// Attention of newest tokens over a paged cache on the tensor cores (bf16).
//
// A unit is what reads one request's rows of one key/value head for the same
// query rows: up to two row tiles of 128.  Keys go in tiles of 128 rows, page
// by page (one TMA box each) into shared memory.  All units' tiles lie on one
// line, weighted by what they cost, and CTA i of G takes the i-th part of it,
// whatever the lengths.  A piece of a unit that is the whole of it gives o and
// lse; pieces of one that was cut leave (o, lse) partials, which are joined by
// columns and in a fixed order at the unit's end.  A CTA has at most one piece at the start of a unit
// that is cut and one further on in a unit, so the partials take four row tiles
// a CTA whatever the sizes.
//
// Two streams of (query rows, S, O) take turns on the tensor cores, each with
// its own softmax warpgroup, so that one's exponentials run under the other's
// products:
//   two row tiles: both streams read the same key tiles, stream = row tile;
//   one row tile:  the same rows, stream 0 takes the even tiles and stream 1
//                  the odd ones; at the piece's end the two join, each thread
//                  half the columns of its row.
//
//   warps 4-7, 8-11 softmax of streams 0 and 1: thread = query row
//   warps 0, 2      TMA: Q (two buffers) and K, and V, in the order the MMAs use
//                   them through one ring of 128-row tiles; a lane a page
//   warp 1          the MMAs: S(0) S(1) | P V(m) S(m + 2) ...
//
// P is rounded to bf16 for its product with V, as in the framework's causal
// attention (sums, maxima and partials stay fp32; against 64 bits 0.0023 of the
// norm, where P in fp32 has 0.0017, the output's own rounding).  S(m + 2) is issued
// after P V(m), and MMAs run in order: when S of a stream is there, so is
// everything that was added to its O before, and the tiles that those products
// read are free.
// Tensor memory: S0, S1 (128 columns each), O0, O1 (D each).
//
// What bounds it: a row's products with a key and a value are 4 D operations, and
// its keys and values come once a unit, so from about 100 rows on the tensor pipe
// would.  Measured, 16 requests of 32 heads on 8 of 128, 64 tokens, 16384 rows: 217
// us, 1.27 PFLOP/s, 0.65 of the cuBLAS rate.  A stream's steps follow one another:
// softmax of a tile 1550 clk, then 1600 until its next scores are there (of which 1024
// are the two streams' MMAs, the rest hand-overs); a third buffer of scores that could
// hide them does not fit tensor memory beside O at D = 128.  A call of less work is
// its start (4.7 us), its tiles (1.95 us for two row tiles, 1.5 for one) and the join
// (3 to 6): 13 requests of up to 8191 rows, 20 heads on 4, 24 tokens, 31 us, where the
// bytes alone take 13.  Its tiles run at the memory's rate (64 KB in 1.5 us on every SM,
// 6.6 TB/s); start and join are what is lost.  Pieces of prompts: 8 heads' 32768 rows of
// 128 1.62 ms, 1.36 PFLOP/s, 8192 rows of 8 heads on 2 169 us, 512 rows of 32 on 8 behind
// 4096, four requests, 134 us (1.09).
#include <cuda.h>

#include <type_traits>

#include "common.cuh"
#include "host_common.h"
#include "launch_util.h"
#include "mma4.cuh"
#include "overlap.cuh"
#include "paged.h"
#include "paged_line.cuh"
#include "ptx.cuh"
#include "row_softmax.cuh"
#include "tmap.h"

namespace sca {
namespace paged_tc {

using namespace paged_line;

constexpr int kThreads = 384;
constexpr int kProd = 0, kMma = 1, kValues = 2;   // the softmax warps are 4 to 11
constexpr int PANEL = 128 * 128;          // 128 rows x 64 bf16, 128-byte swizzle
// registers: 384 x 168 at launch = 256 x 208 + 128 x 88
constexpr int kRegSoftmax = 208, kRegRoles = 88;
static_assert(256 * kRegSoftmax + 128 * kRegRoles <= kThreads * 168, "register split");
// Up to how many pieces their last CTA joins alone; how long a CTA without further
// work waits for the other pieces of its unit, in clk.
constexpr int kAlone = 4, kPatience = 40000;
constexpr int64_t kLseRows = kMaxCtas * 512;
// What a tile of one or two row tiles costs and the start and end of a unit, in
// about 450 clk; what is not cut.  Units at 22 and 45 left 64 requests of 700 rows, 32
// tokens, at 28.6 us (here 18.1) and 32 requests of 2048 rows, 8 tokens, at 33.0 (31.3);
// at 40 and 80, 50 and 90 the other cases gain or lose 2%.
constexpr int kCostOne = 5, kCostTwo = 8, kCostUnit = 30, kCostWhole = 70;
// Tiles of a CTA, at least, for one unit or two, since every further piece is joined:
// one request's 24 rows of one head behind 38149 rows 27.6 us, with one tile 32.6, 64 rows
// behind 20000 of 64 18.2 and 27.7; 12 units behind 2000 rows 23.1 and 19.3.
constexpr int kLeast = 3;

struct Args {
  CUtensorMap mq, mk, mv;
  Units u;
  int32_t q_rows;             // rows of a query box
  int32_t box_log2;           // rows of a page's box
  int32_t* counters;          // [3][kMaxCtas] of the cut unit that starts in CTA i; zero between calls
  // [CTA][2][256] rows: of a piece that is not its unit's first, of one that is;
  // part_o [CTA][2][2][D][128]
  float *part_o, *part_lse;
};

// Row rr of the unit in CTA i's partials: of a piece at its unit's start, or of one further on.
SCA_INLINE int64_t part_row(int i, bool starts, int rr) { return static_cast<int64_t>((i * 2 + starts) * 256 + rr); }

// ---- the kernel -----------------------------------------------------------

template <int RING>
struct Bars {
  uint64_t q_full[2], q_free[2];
  uint64_t full[RING], free[RING];
  uint64_t s_full[2], p_full[2], o_full[2], o_free[2];
  uint64_t stats, stored, joined;   // between the softmax warps: both streams' ends, a partial written, who joins
  uint64_t drain;
  Cursor cur;            // behind the first piece
  Piece first;
  Line line;
  int any;               // is there one?
  int slice[2];          // of the columns to join; behind the last: none (by the phase of `joined`)
  uint32_t tmem_base;
  int abort;
};

template <int D>
struct Layout {
  static constexpr int RING = D == 64 ? 11 : 5;
  static constexpr int TILE = D / 64 * PANEL;
  static constexpr int Q_OFF = 0;
  static constexpr int RING_OFF = 2 * TILE;
  static constexpr int STAT_OFF = RING_OFF + RING * TILE;   // (maximum, sum) of both streams' rows
  static constexpr int BAR_OFF = STAT_OFF + 2 * 128 * 8;
  static constexpr int SMEM = BAR_OFF + static_cast<int>(sizeof(Bars<RING>));
  // one CTA per SM (tensor memory is allocated whole)
  static_assert(SMEM > 120 * 1024 && SMEM <= 232448, "one CTA's shared memory");
};

// kUneven: long pieces of prompts, whose rows see different numbers of rows
template <int D, bool kUneven>
__global__ void __launch_bounds__(kThreads, 1) attend_kernel(const __grid_constant__ Args ka) {
  using L = Layout<D>;
  constexpr int RING = L::RING, NP = D / 64;
  const PagedArgs& a = ka.u.a;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars<RING>* bars = reinterpret_cast<Bars<RING>*>(smem + L::BAR_OFF);
  float2* stat = reinterpret_cast<float2*>(smem + L::STAT_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (smem_u32(smem) & 1023) {   // the swizzle needs it (the whole CTA returns)
    report(a.status, SCA_ERR_ALIGN);
    return;
  }
  if (threadIdx.x == 32 * kProd) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->q_free[i], 1);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_full[i], 4);
      mbar_init(&bars->o_full[i], 1);
      mbar_init(&bars->o_free[i], 8);
    }
    for (int i = 0; i < RING; ++i) {
      mbar_init(&bars->full[i], 1);
      mbar_init(&bars->free[i], 1);
    }
    mbar_init(&bars->stats, 8);
    mbar_init(&bars->stored, 8);
    mbar_init(&bars->joined, 8);
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == kProd) {
    __syncwarp();
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 64) {
    tma_prefetch_map(&ka.mq);
    tma_prefetch_map(&ka.mk);
    tma_prefetch_map(&ka.mv);
  }
  wait_for_previous();
  volatile int* abort = &bars->abort;
  // ---- loads, by all lanes of their warp, each the box of its page
  int nq[2] = {0, 0}, turn = 0;   // warp kProd: queries so far, the next buffer
  const int bi = lane / NP, panel = lane - bi * NP, box_row = bi << ka.box_log2;
  auto load_q = [&](int buf, int rt, const Piece& p) {
    if (nq[buf] > 0 && !wait_all_or_abort(&bars->q_free[buf], (nq[buf] - 1) & 1, abort)) return false;
    if (lane == 0) {
      mbar_arrive_expect_tx(&bars->q_full[buf], NP * ka.q_rows * 128);
      for (int c = 0; c < NP; ++c)
        tma_load_4d(smem + L::Q_OFF + buf * L::TILE + c * PANEL, &ka.mq, &bars->q_full[buf], 64 * c, rt * 128, p.hk, p.b);
    }
    ++nq[buf];
    return true;
  };
  // This lane's entry of the table.  Looked up a tile ahead and looked at only
  // where it is used, so that its latency runs under the load before.
  auto entry_of = [&](const Piece& p, int j) {
    const int row = (p.j0 + j) * BN + box_row;
    return j < p.nt && box_row < BN && row < p.rows ? a.table[p.b * a.table_b + (row >> a.page_log2)] : 0;
  };
  // a tile to its place in the ring; an entry outside the pool becomes `pages`, where all is zero
  auto load = [&](const CUtensorMap* m, int place, const Piece& p, int j, int entry) {
    const int st = place % RING, row = (p.j0 + j) * BN + box_row;
    const bool has = box_row < BN && row < p.rows;
    if (has && (entry < 0 || entry >= a.pages)) {
      report(a.status, SCA_ERR_RANGE);
      entry = static_cast<int>(a.pages);
    }
    if (place >= RING && !wait_all_or_abort(&bars->free[st], (place / RING - 1) & 1, abort)) return false;
    const int boxes = __popc(__ballot_sync(0xffffffffu, has));
    if (lane == 0) mbar_arrive_expect_tx(&bars->full[st], boxes << (ka.box_log2 + 7));
    __syncwarp();
    if (has)
      tma_load_4d(smem + L::RING_OFF + st * L::TILE + panel * PANEL + (box_row << 7), m, &bars->full[st], 64 * panel,
                  row & ((1 << a.page_log2) - 1), p.hk, entry);
    return true;
  };
  // Places of a piece's tiles, its first at `it`.  Two row tiles: K0 V0 K1 V1 ...;
  // one: K0 K1 V0 K2 V1 ... V.
  auto place_k = [](int it, const Piece& p, int j) { return it + (p.two ? 2 * j : (j ? 2 * j - 1 : 0)); };
  auto place_v = [](int it, const Piece& p, int j) { return it + 2 * j + (p.two || j + 1 == p.nt ? 1 : 2); };
  // on the abort path, let the copies in flight land before the CTA goes away
  // (a place of the other warp's is waited for as well, or in vain for a while)
  auto land = [&](int last) {
    if (*abort && lane == 0)
      for (int x = last; x >= 0 && x > last - RING; --x) mbar_wait_drain(&bars->full[x % RING], (x / RING) & 1);
  };
  auto load_queries = [&](const Piece& p) {
    if (p.two) return load_q(0, p.rt, p) && load_q(1, p.rt + 1, p);
    turn ^= 1;
    return load_q(turn ^ 1, p.rt, p);
  };
  if (warp == kProd) {
    // the first piece, found once for all roles, and its loads on their way
    // before anything else: a short call waits for little but this
    Line line;
    Cursor c = find_part<kUneven>(ka.u, lane, line);
    Piece f = {};
    const bool any = c.next<kUneven>(ka.u, f);
    if (lane == 0) {
      bars->cur = c;
      bars->first = f;
      bars->line = line;
      bars->any = any;
    }
    if (blockIdx.x == 0)
      for (int b = lane; b < a.B; b += 32) report_beyond(a, b);
    if (any && f.nt > 0) {
      const int entry = entry_of(f, 0);
      load_queries(f);
      load(&ka.mk, 0, f, 0, entry);
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
      // --------------------------------------------------- Q and K
      int it = 0, last = 0;
      bool ok = true;
      for (bool begun = true; ok && more; begun = false, more = ok && cur.next<kUneven>(ka.u, p)) {
        if (p.nt == 0) continue;
        int next = entry_of(p, begun ? 1 : 0);
        ok = begun || load_queries(p);
        for (int j = begun ? 1 : 0; ok && j < p.nt; ++j) {
          const int now = next;
          next = entry_of(p, j + 1);
          ok = load(&ka.mk, last = place_k(it, p, j), p, j, now);
        }
        it += 2 * p.nt;
      }
      land(last);
      if (*abort && lane == 0)
        for (int j = 0; j < 2; ++j)
          if (nq[j]) mbar_wait_drain(&bars->q_full[j], (nq[j] - 1) & 1);
    } else if (warp == kValues) {
      // --------------------------------------------------------- V
      int it = 0, last = -1;
      for (bool ok = true; ok && more; more = ok && cur.next<kUneven>(ka.u, p)) {
        int next = entry_of(p, 0);
        for (int j = 0; ok && j < p.nt; ++j) {
          const int now = next;
          next = entry_of(p, j + 1);
          ok = load(&ka.mv, last = place_v(it, p, j), p, j, now);
        }
        it += 2 * p.nt;
      }
      land(last);
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
        if (p.nt == 0) {
          more = cur.next<kUneven>(ka.u, p);
          continue;
        }
        const int M = p.two ? 2 * p.nt : p.nt, qb = p.two ? 0 : turn;
        if (!p.two) turn ^= 1;
        ok = wait_all(&bars->q_full[qb], (q_ph >> qb) & 1) && (!p.two || wait_all(&bars->q_full[1], (q_ph >> 1) & 1));
        q_ph ^= p.two ? 3 : 1 << qb;
        // the places that are next for S and for P V
        int kst = it % RING, kph = (it / RING) & 1, vst = kst, vph = kph;
        advance(vst, vph, p.two || p.nt == 1 ? 1 : 2);
        // A wait takes about 200 clk even where all is there, and the tensor pipe has
        // only a few MMAs in hand: waits come between MMAs that it still works on, and
        // what both streams read is waited for once (wide trees 228 -> 224 us).
        bool v_there = false;
        for (int m = -2; ok && m < M; ++m) {
          const int s = m & 1;
          const uint32_t tS = tmem + 128 * s, tO = tS + 256;
          const bool again = p.two && s == 1;        // the same K and V as the step before
          if (m == 0) more = cur.next<kUneven>(ka.u, pn);     // its loads' latency under the first softmax
          if (m >= 0) {
            if (!v_there && !(ok = wait_all(&bars->full[vst], vph))) break;
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
            if (m + 2 < M && !again && !(ok = wait_all(&bars->full[kst], kph))) break;
            umma4_ts<128>(tO, tS + 32, sdesc_step(vd, 8192), id_o, 1);
            if (m + 2 >= M) umma_commit_w(&bars->o_full[s]);
          } else if (m + 2 < M && !again && !(ok = wait_all(&bars->full[kst], kph))) {
            break;
          }
          if (m + 2 < M) {
            tc_fence_after();
            const uint64_t qd = sdesc_sw128(s0 + L::Q_OFF + (p.two ? s : qb) * L::TILE, 16, 1024);
            const uint64_t kd = sdesc_sw128(s0 + L::RING_OFF + kst * L::TILE, 16, 1024);
#pragma unroll
            for (int c = 0; c < NP; ++c)
              umma4_ss<2, 2>(tS, sdesc_step(qd, c * PANEL), sdesc_step(kd, c * PANEL), id_s, c);
            umma_commit_w(&bars->s_full[s]);
            if (!p.two) advance(kst, kph, m < -1 ? 1 : 2);
            else if (s == 1) advance(kst, kph, 2);
          }
          v_there = m >= 0 && m + 1 < M;
          if (v_there && !(p.two && s == 0)) ok = wait_all(&bars->full[vst], vph);
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
    const uint32_t tS = tmem + 128 * s + lane_off, tO0 = tmem + 256 + lane_off, tO = tO0 + 128 * s;
    const float sl2 = a.scale_log2;
    int it = 0, ns = 0;           // ring place of the piece; tiles of this stream so far
    int o_ph = 0, x_ph = 0, y_ph = 0, j_ph = 0;   // phases of o_full (bit s), stats, stored, joined
    int turn = 0;                 // query buffer of the next piece of one row tile
    const bool gives = (warp & 3) == 0 && lane == 0;   // gives tiles back to the producer
    __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(a.o);
    bool ok = true;
    Piece pn;
    while (ok && more) {
      const int64_t head_row = (static_cast<int64_t>(p.b) * a.Hkv + p.hk) * a.R;   // of o and lse
      if (p.nt == 0) {   // nothing to see
        const int n = min(p.two ? 256 : 128, a.R - 128 * p.rt);
        for (int e = threadIdx.x - 128; e < n * (D / 8); e += 256)
          reinterpret_cast<uint4*>(out + (head_row + 128 * p.rt) * D)[e] = make_uint4(0, 0, 0, 0);
        for (int e = threadIdx.x - 128; e < n; e += 256) a.lse[head_row + 128 * p.rt + e] = -INFINITY;
        more = cur.next<kUneven>(ka.u, p);
        continue;
      }
      const int cnt = p.two ? p.nt : (p.nt + 1 - s) / 2;
      const int r = (p.rt + (p.two ? s : 0)) * 128 + row;   // query row of the request and head
      const bool valid = r < a.R;
      const bool some = __any_sync(0xffffffffu, valid);
      const Sight sees = valid ? sight(a, p.b, r % a.T, Held{p.len, p.cnt}, p.rows) : Sight{0, 0};
      // the pieces of the unit, by CTAs i0, i0 + 1, ...
      const bool whole = p.whole();
      int i0 = blockIdx.x, n = 1;
      if (!whole) {
        const Line line = bars->line;
        if (p.j0) i0 = line.cta_of(p.at + ka.u.cost_unit);
        n = pieces_of(ka.u, line, p, i0);
      }
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
        if (some)
          softmax_tile<D>(tS, tO, k > 0, sl2, m_used, l, [&](uint32_t (&y)[32], int h) {
            if (k0 + BN > sees.full) mask_columns(y, seen_bits(sees, p.len, k0 + 32 * h));
          });
        if (k0 + BN > p.rows) {
          // the request's last tile, and so the piece's: rows of V behind it may hold anything
          const int i = it + 2 * p.nt - 1, st = i % RING, n = p.rows - k0;
          if (!(ok = wait_all(&bars->full[st], (i / RING) & 1))) break;
          uint8_t* v = smem + L::RING_OFF + st * L::TILE;
          for (int e = row; e < (BN - n) * (D / 8); e += 128) {
            const int vr = n + e / (D / 8), q = e % (D / 8);
            *reinterpret_cast<uint4*>(v + (q >> 3) * PANEL + vr * 128 + (q & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_async_smem();
        }
        tc_fence_before();
        warp_arrive(&bars->p_full[s], lane);
        if (k == 0) more = cur.next<kUneven>(ka.u, pn);
      }
      if (!ok) break;
      if (cnt == 0) more = cur.next<kUneven>(ka.u, pn);
      // ---- the piece's end
      const bool both = !p.two && p.nt > 1;   // two streams' sums of the same rows
      const bool tells = p.two || s == 0;     // whether this thread writes the row's lse
      const int mine = p.two ? 1 << s : (both ? 3 : 1);
      const int me = blockIdx.x - i0, unit_row = row + (p.two ? 128 * s : 0);   // of the unit's 256
      // Where few others are there already, this one need not be written down;
      // looked up under the last product.
      const bool ask = !whole && n <= kAlone;
      if (ask && threadIdx.x == 128) {
        const bool all = load_acquire(ka.counters + i0) == n - 1;
        bars->slice[j_ph] = all ? 0 : 1;
        if (all) {   // nothing is left for those that wait
          atomicAdd(ka.counters + i0 + kMaxCtas, D);
          add_acq_rel(ka.counters + i0, 1);
        }
      }
      for (int i = 0; ok && i < 2; ++i)
        if (mine >> i & 1) ok = wait_all(&bars->o_full[i], (o_ph >> i) & 1);
      if (!ok) break;
      o_ph ^= p.two ? 3 : mine;   // the other stream's O of two row tiles is done before this one's next piece
      tc_fence_after();
      // one row tile's last V comes right behind its K
      if (gives && (p.two ? s == 1 : cnt > 0))
        mbar_arrive(&bars->free[!p.two && 2 * (cnt - 1) + s == M - 1 ? wrap(fv + RING - 1) : fv]);
      float m0 = m_used, l0 = l, m1 = -INFINITY, l1 = 0.f;   // of O0 and O1 (two row tiles: of this stream's O)
      if (!p.two) {
        if (cnt > 0) stat[128 * s + row] = make_float2(m_used, l);
        warp_arrive(&bars->stats, lane);
        if (!(ok = wait_all(&bars->stats, x_ph))) break;
        x_ph ^= 1;
        const float2 st0 = stat[row], st1 = both ? stat[128 + row] : make_float2(-INFINITY, 0.f);
        m0 = st0.x, l0 = st0.y, m1 = st1.x, l1 = st1.y;
      }
      const float top = fmaxf(m0, m1), sub = top == -INFINITY ? 0.f : top;
      float w0 = ex2(m0 - sub), w1 = ex2(m1 - sub);
      const float total = w0 * l0 + w1 * l1, inv = total == 0.f ? 0.f : 1.f / total;
      const float lse2 = total == 0.f ? -INFINITY : sub + log2f(total);
      w0 *= inv;
      w1 *= inv;
      // columns [c0, c1) of the row: half of them where the streams share it
      const int c0 = p.two ? 0 : s * (D / 2), c1 = p.two ? D : c0 + D / 2;
      // Columns go sixteen at a time: the code runs once or twice a launch, and
      // fetching it takes longer than the work.  Partials lie with rows side by
      // side, a warp's store in one line (with a row's 16 bytes a lane, 32 lines a
      // store, 256 rows took 4.8 us to write, now 1.8).
      auto part_at = [&](int cta, int c) {
        return ka.part_o + (part_row(cta, cta == i0, unit_row) - row) * D + static_cast<int64_t>(c) * 128 + row;
      };
      auto put_out = [&](const float (&x)[16], int c) {
        __nv_bfloat16* po = out + (head_row + r) * D + c;
#pragma unroll
        for (int e = 0; e < 16; e += 8)
          *reinterpret_cast<uint4*>(po + e) = make_uint4(pack_bf16x2(x[e], x[e + 1]), pack_bf16x2(x[e + 2], x[e + 3]),
                                                         pack_bf16x2(x[e + 4], x[e + 5]), pack_bf16x2(x[e + 6], x[e + 7]));
      };
      // what thread 128 found out, told to all softmax warps
      auto told = [&] {
        warp_arrive(&bars->joined, lane);
        if (!(ok = wait_all(&bars->joined, j_ph))) return -1;
        j_ph ^= 1;
        return bars->slice[j_ph ^ 1];
      };
      bool alone = false;
      if (ask) {
        alone = told() == 0;
        if (!ok) break;
      }
      auto lse_of = [&](int t) { return t < n ? __ldcg(ka.part_lse + part_row(i0 + t, t == 0, unit_row)) : -INFINITY; };
      float base = 0.f;         // of the weights: the largest lse of the row's pieces
      auto find_base = [&](int own) {
        float most = own >= 0 ? lse2 : -INFINITY;
#pragma unroll 1
        for (int t0 = 0; t0 < n; t0 += 16) {
          float e[16];
#pragma unroll
          for (int t = 0; t < 16; ++t) e[t] = t0 + t == own ? lse2 : lse_of(t0 + t);
#pragma unroll
          for (int t = 0; t < 16; ++t) most = fmaxf(most, e[t]);
        }
        base = most == -INFINITY ? 0.f : most;
      };
      // x becomes the weighted mean of columns c, c + 1, ... of all pieces, P pieces'
      // loads together; piece `own` (-1: none) is in x.  Returns the row's lse.
      auto join = [&](auto& x, auto pieces, int own, int c) {
        constexpr int P = decltype(pieces)::value, C = sizeof(x) / 4;
        float acc[C] = {}, sum = 0.f;
#pragma unroll 1
        for (int t0 = 0; t0 < n; t0 += P) {
          float f[P], y[P][C];
#pragma unroll
          for (int t = 0; t < P; ++t) {
            const bool there = t0 + t < n && t0 + t != own;
            const float* const po = part_at(there ? i0 + t0 + t : i0, c);
            f[t] = t0 + t == own ? lse2 : lse_of(t0 + t);
#pragma unroll
            for (int e = 0; e < C; ++e) y[t][e] = there ? __ldcg(po + e * 128) : (t0 + t == own ? x[e] : 0.f);
          }
#pragma unroll
          for (int t = 0; t < P; ++t) {
            f[t] = ex2(f[t] - base);
            sum += f[t];
#pragma unroll
            for (int e = 0; e < C; ++e) acc[e] = fmaf(f[t], y[t][e], acc[e]);
          }
        }
        const float f = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int e = 0; e < C; ++e) x[e] = acc[e] * f;
        return sum == 0.f ? -INFINITY : base + log2f(sum);
      };
      using Four = std::integral_constant<int, 4>;
      using Eight = std::integral_constant<int, 8>;
      using Sixteen = std::integral_constant<int, 16>;
      if (some) {
        const uint32_t tA = p.two ? tO : tO0;
        float row_lse = lse2;
        if (alone && valid) find_base(me);
#pragma unroll 1
        for (int c = c0; c < c1; c += 16) {
          uint32_t u[16];
          float x[16];
          __syncwarp();
          tmem_row(tA + c, u);
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(u[e]) * w0;
          if (both) {
            tmem_row(tO0 + 128 + c, u);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = fmaf(__uint_as_float(u[e]), w1, x[e]);
          }
          if (valid) {
            if (total == 0.f) {   // no weight: nothing of what the products made of it
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = 0.f;
            }
            if (alone) row_lse = join(x, Four(), me, c);
            if (whole || alone) {
              put_out(x, c);
            } else {
              float* const po = part_at(blockIdx.x, c);
#pragma unroll
              for (int e = 0; e < 16; ++e) po[e * 128] = x[e];
            }
          }
        }
        if (valid && tells) {
          if (whole || alone) a.lse[head_row + r] = row_lse * kLn2;
          else ka.part_lse[part_row(blockIdx.x, me == 0, unit_row)] = lse2;
        }
      }
      // O has been read: eight arrivals a stream, four of them twice where a stream is one warpgroup's
      tc_fence_before();
      __syncwarp();
      if (lane == 0)
        for (int i = 0; i < 2; ++i)
          if (mine >> i & 1) {
            mbar_arrive(&bars->o_free[i]);
            if (p.two) mbar_arrive(&bars->o_free[i]);
          }
      if (!whole) {
        // ---- a cut unit: its pieces are joined by columns, by all CTAs that are still
        // there when the last has come (by the last one alone, with 13 pieces of 216
        // rows, 35 us instead of 24).  Nobody depends on another's waiting: who comes
        // last goes on until all columns are taken.
        int32_t* const arrived = ka.counters + i0;
        int32_t* const taken = arrived + kMaxCtas;
        int32_t* const left = taken + kMaxCtas;
        if (!alone) {
          // A slice is 16 columns, or fewer of more pieces; of one row tile each stream
          // takes half of it.  64 loads of a thread are in flight together.
          const bool long_line = n > 32;
          const int width = p.two ? (long_line ? 4 : n > 16 ? 8 : 16) : (long_line ? 8 : 16), slices = D / width, take = (slices + n - 1) / n;
          warp_arrive(&bars->stored, lane);   // partials are written
          if (!(ok = wait_all(&bars->stored, y_ph))) break;
          y_ph ^= 1;
          bool all = false;
          if (threadIdx.x == 128) {
            all = add_acq_rel(arrived, 1) == n - 1;
            if (!all && !more) {
              const long long t0 = clock64();
              do all = load_acquire(arrived) == n;
              while (!all && clock64() - t0 < kPatience);
            }
          }
          bool begun = false;
          while (true) {
            if (threadIdx.x == 128) bars->slice[j_ph] = all ? atomicAdd(taken, take) : slices;
            const int slice = told();
            if (!ok || slice >= slices) break;
            if (valid && !begun) find_base(-1);
            begun = true;
            const int end = min(slice + take, slices);
#pragma unroll 1
            for (int i = slice; i < end; ++i) {
              if (!valid) continue;
              float row_lse;
              if (long_line) {
                const int c = i * width + (p.two ? 0 : 4 * s);
                float x[4];
                row_lse = join(x, Sixteen(), -1, c);
                *reinterpret_cast<uint2*>(out + (head_row + r) * D + c) =
                    make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
              } else if (width == 16 && p.two) {
                float x[16];
                row_lse = join(x, Four(), -1, 16 * i);
                put_out(x, 16 * i);
              } else {
                const int c = i * width + (p.two ? 0 : 8 * s);
                float x[8];
                row_lse = join(x, Eight(), -1, c);
                *reinterpret_cast<uint4*>(out + (head_row + r) * D + c) = make_uint4(
                    pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
              }
              if (i == 0 && (p.two || s == 0)) a.lse[head_row + r] = row_lse * kLn2;
            }
          }
          if (!ok) break;
        }
        // who leaves last leaves zeros
        if (threadIdx.x == 128 && atomicAdd(left, 1) == n - 1) *arrived = *taken = *left = 0;
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

template <int D, bool kUneven>
static cudaError_t launch(const Args& k, cudaStream_t st) {
  using L = Layout<D>;
  static std::atomic<bool> done[kMaxCachedDevices];
  const cudaError_t e = allow_smem(attend_kernel<D, kUneven>, L::SMEM, done);
  if (e != cudaSuccess) return e;
  return launch_early(attend_kernel<D, kUneven>, dim3(k.u.G), kThreads, L::SMEM, st, k);
}

constexpr int64_t kHeadFloats = 1024;   // the counters, in front of the partials
static_assert(3 * kMaxCtas <= kHeadFloats, "counters");

}  // namespace paged_tc

using namespace paged_tc;

int64_t paged_tc_workspace(int D, int sms) {
  return (kHeadFloats + kLseRows + static_cast<int64_t>(sms < kMaxCtas ? sms : kMaxCtas) * 512 * D) * 4;
}

int paged_tc_attend(const PagedArgs& a, int D, int sms, float* ws, cudaStream_t stream) {
  Args k = {};
  const int64_t units = static_cast<int64_t>(a.B) * a.Hkv * ((a.R + 255) / 256);
  SCA_REQUIRE(make_units(k.u, a, sms, kCostOne, kCostTwo, kCostUnit, kCostWhole, units <= 2 ? kLeast : 1), SCA_ERR_UNSUPPORTED,
              "paged_tree_attend: more than about 2^28 tiles of 128 rows");
  k.q_rows = a.R < 128 ? a.R : 128;
  k.box_log2 = a.page_log2 < 7 ? a.page_log2 : 7;
  k.counters = reinterpret_cast<int32_t*>(ws);
  k.part_lse = ws + kHeadFloats;
  k.part_o = k.part_lse + kLseRows;
  const int page = 1 << a.page_log2;
  const View q{a.q_b, static_cast<int64_t>(a.R) * D, D};
  cudaError_t e = make_tmap_bf16(&k.mq, a.q, D, a.R, a.Hkv, a.B, q, 64, k.q_rows);
  if (e == cudaSuccess)
    e = make_tmap_bf16(&k.mk, a.kp, D, page, a.Hkv, static_cast<int>(a.pages), a.pool, 64, 1 << k.box_log2);
  if (e == cudaSuccess)
    e = make_tmap_bf16(&k.mv, a.vp, D, page, a.Hkv, static_cast<int>(a.pages), a.pool, 64, 1 << k.box_log2);
  SCA_REQUIRE(e == cudaSuccess, SCA_ERR_ALIGN, "paged_tree_attend: layout not expressible as a TMA tensor map");
  if (uneven(k.u)) e = D == 64 ? launch<64, true>(k, stream) : launch<128, true>(k, stream);
  else e = D == 64 ? launch<64, false>(k, stream) : launch<128, false>(k, stream);
  return cuda_status(e, "paged_tree_attend (tensor cores)");
}

}  // namespace sca
