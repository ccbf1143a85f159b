// Attention of newest tokens over a paged cache on the tensor cores, few query
// rows a key/value head (decoding, small trees): both products turned round, so
// that the 128 rows of an MMA are keys, then features, and up to 16 query rows are
// its columns.
//
//   S^T = K Q^T         128 keys x 16 rows, in tensor memory
//   P^T = exp(S^T - m)  a thread a key: 4, 8 or 16 numbers, not 128
//   O^T += V^T P^T      D features x 16 rows, in tensor memory
//
// The work is shared out as in paged_tc.cu: units' tiles on one line, a part of it
// a CTA.  Two softmax warpgroups take a piece's tiles in turn, each with S, P, O
// and maxima of its own, and meet at the piece's end: a tile's chain of hand-overs
// (about 1300 clk for 4 rows, half of it barriers) takes longer than its keys take
// to arrive with D = 64.  A thread adds up its own keys' weights, which meet at the
// end too; only the row maxima meet tile by tile (they are followed when they
// grow by more than 2^8, as in row_softmax.cuh).  O has two buffers, so that a
// piece's end runs under the start of the next piece.
//
//   warps 0, 2  TMA: Q (two buffers) and K, and V, through one ring of 128-row
//              tiles, in the order of their use: K0 K1 V0 K2 V1 ...; a lane a page (by
//              one warp a tile's two loads took 1900 clk, its rows 700 with D = 64)
//   warp 1     the MMAs: S(0) | S(i + 1) P V(i) ..., pieces one after the other
//   warps 4-7, 8-11  softmax of even and of odd tiles: thread = key, then feature
// Tensor memory: S and, for even and odd pieces, O of both (16 columns each).
//
// What bounds it: 2 D operations a key, value and row are little beside their bytes,
// so HBM, where caches are long: 32 requests of 32768 rows, 8 heads of 128, 605 us, 7.1
// TB/s (the copy rate is 6.8).  With D = 64 the warp that issues the MMAs is: about 1600
// clk a tile, 45 requests x 6 heads x 5903 rows of 64 in 72 us where the bytes
// take 60.  Short calls are a chain: launch and start 4 us, a page number and its
// rows 1.5, the tile 1, the join 2.
#include <cuda.h>

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
namespace paged_few {

using namespace paged_line;

constexpr int kThreads = 384;
constexpr int kProd = 0, kMma = 1, kValues = 2;
constexpr int PANEL = 128 * 128;          // 128 rows x 64 bf16, 128-byte swizzle
constexpr int NR = 16;                    // columns of the MMAs, the fewest that they take
constexpr int kColumns = 128;             // of tensor memory: 2 of S, 4 of O, a power of two
static_assert(NR == kPagedFewRows && 6 * NR <= kColumns, "rows");
// What a tile of D features and the start and end of a unit cost; what is not
// cut.  Units at 12 and 52 left 64 requests of 500 rows at 23.6 us (here 19.8), at 30
// and 70 at 23.3; longer caches are within 1% with either.
constexpr int kCost128 = 10, kCost64 = 6, kCostUnit = 18, kCostWhole = 58;

struct Args {
  CUtensorMap mq, mk, mv;
  Units u;
  int32_t box_log2;           // rows of a page's box
  int32_t* counters;          // [kMaxCtas] pieces done of the cut unit that starts in CTA i; zero between calls
  float *part_o, *part_lse;   // [CTA][2][NR] rows: of a piece that is not its unit's first, of one that is
};

// A piece as the producer hands it on, with its queries; behind the last: no tiles.
struct Job {
  int b, hk, len, cnt, rows, j0, nt;
  int i0, n;             // the unit's n pieces are those of CTAs i0, i0 + 1, ...
};

// Queries have two buffers, jobs eight places: a buffer of queries is given back
// when its piece's last scores are made, and a group that has no tile in a piece
// may look at its job later, but before anyone is two pieces further.
constexpr int kJobs = 8;

template <int RING>
struct Bars {
  uint64_t q_full[2], q_free[2];   // (q_full: for the MMAs, and the job)
  uint64_t job_full[kJobs];        // for the softmax
  uint64_t full[RING], free[RING];
  uint64_t s_full[2], p_full[2], o_full[2], o_free[2];
  uint64_t meet[2], both;          // the warps of a softmax group; all of them
  uint64_t drain;
  Job jobs[kJobs];
  int last;              // this CTA joins the unit
  uint32_t tmem_base;
  int abort;
};

template <int D>
struct Layout {
  static constexpr int TILE = D / 64 * PANEL;
  static constexpr int RING = D == 64 ? 10 : 6;
  static constexpr int QB = NR * D * 2, PB = NR * 256;      // a buffer of queries; of weights
  static constexpr int Q_OFF = RING * TILE;
  static constexpr int P_OFF = Q_OFF + 2 * QB;
  // of both groups:
  static constexpr int MAX_OFF = P_OFF + 2 * PB;            // [2][2][4][NR] a warp's maxima of a tile
  static constexpr int SUM_OFF = MAX_OFF + 4 * 4 * NR * 4;  // [2][4][NR] a warp's sums of a piece
  // [2][2][NR] a row's maximum, then its O's weight, of even and of odd pieces: a
  // warp may still read a piece's when another, without a tile in the next, has
  // got to that one's end
  static constexpr int TOP_OFF = SUM_OFF + 2 * 4 * NR * 4;
  static constexpr int SEE_OFF = TOP_OFF + 4 * NR * 4;      // [2][NR] what a row sees
  static constexpr int BAR_OFF = SEE_OFF + 2 * NR * 16;
  static constexpr int USED = BAR_OFF + static_cast<int>(sizeof(Bars<RING>));
  // With D = 64 the MMA's upper 64 rows are features that are not there: it reads
  // on behind the tile (and nothing reads what it makes of that).
  static constexpr int SMEM = USED > (RING + 1) * PANEL || D == 128 ? USED : (RING + 1) * PANEL;
  static_assert(SMEM > 120 * 1024 && SMEM <= 232448 && QB / (D / 64) % 1024 == 0, "one CTA's shared memory");
};

// x[r] of all lanes for N rows, combined by f: lane i gets row i % N.
template <int N, typename F>
SCA_INLINE float across(float (&x)[N], int lane, const F& f) {
#pragma unroll
  for (int w = N / 2; w; w >>= 1)
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      if (i < w) {
        const float give = lane & w ? x[i] : x[i + w];
        x[i] = f(lane & w ? x[i + w] : x[i], __shfl_xor_sync(0xffffffffu, give, w));
      }
#pragma unroll
  for (int w = N; w < 32; w <<= 1) x[0] = f(x[0], __shfl_xor_sync(0xffffffffu, x[0], w));
  return x[0];
}

// NQ: the rows that softmax looks at; those behind them stay zero
template <int D, int NQ>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(const __grid_constant__ Args ka) {
  using L = Layout<D>;
  constexpr int RING = L::RING, NP = D / 64;
  const PagedArgs& a = ka.u.a;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars<RING>* bars = reinterpret_cast<Bars<RING>*>(smem + L::BAR_OFF);
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
      mbar_init(&bars->meet[i], 4);
    }
    for (int i = 0; i < RING; ++i) {
      mbar_init(&bars->full[i], 1);
      mbar_init(&bars->free[i], 1);
    }
    for (int i = 0; i < kJobs; ++i) mbar_init(&bars->job_full[i], 1);
    mbar_init(&bars->both, 8);
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == kMma) {
    tmem_alloc(&bars->tmem_base, kColumns);
    tmem_relinquish();
  }
  if (threadIdx.x == 96) {
    tma_prefetch_map(&ka.mq);
    tma_prefetch_map(&ka.mk);
    tma_prefetch_map(&ka.mv);
  }
  if (warp == kProd) {   // queries and weights of rows that are not there
    for (int e = lane; e < 2 * (L::QB + L::PB) / 16; e += 32) reinterpret_cast<uint4*>(smem + L::Q_OFF)[e] = make_uint4(0, 0, 0, 0);
    fence_async_smem();
    __syncwarp();
  }
  wait_for_previous();
  volatile int* abort = &bars->abort;
  auto wait_all = [&](uint64_t* bar, uint32_t par) { return wait_all_or_abort(bar, par, abort); };
  // ---- loads, by all lanes of their warp, each the box of its page
  const int bi = lane / NP, panel = lane - bi * NP, box_row = bi << ka.box_log2;
  // This lane's entry of the table.  Looked up a tile ahead and looked at only
  // where it is used, so that its latency runs under the load before.
  auto entry_of = [&](int b, int rows, int tile) {
    const int row = tile * BN + box_row;
    return box_row < BN && row < rows ? a.table[b * a.table_b + (row >> a.page_log2)] : 0;
  };
  // the tile to its place in the ring; an entry outside the pool becomes `pages`, where all is zero
  auto load = [&](const CUtensorMap* m, int place, int hk, int rows, int tile, int entry) {
    const int st = place % RING, row = tile * BN + box_row;
    const bool has = box_row < BN && row < rows;
    if (has && (entry < 0 || entry >= a.pages)) {
      report(a.status, SCA_ERR_RANGE);
      entry = static_cast<int>(a.pages);
    }
    if (place >= RING && !wait_all(&bars->free[st], (place / RING - 1) & 1)) return false;
    const int boxes = __popc(__ballot_sync(0xffffffffu, has));
    if (lane == 0) mbar_arrive_expect_tx(&bars->full[st], boxes << (ka.box_log2 + 7));
    __syncwarp();
    if (has)
      tma_load_4d(smem + st * L::TILE + panel * PANEL + (box_row << 7), m, &bars->full[st], 64 * panel,
                  row & ((1 << a.page_log2) - 1), hk, entry);
    return true;
  };
  // on the abort path, let the copies in flight (K's at 0 and odd places, V's at the
  // others, up to the last) land before the CTA goes away
  auto land = [&](bool keys, int last) {
    if (*abort && lane == 0)
      for (int x = last; x >= 0 && x > last - RING; --x)
        if (keys == (x == 0 || x % 2 == 1)) mbar_wait_drain(&bars->full[x % RING], (x / RING) & 1);
  };
  // K's and V's places; K(0) alone comes first
  auto place_k = [](int i) { return i == 0 ? 0 : 2 * i - 1; };
  auto place_v = [](int i) { return 2 * i + 2; };
  int it = 0, nq = 0, entry = 0;   // warp kProd: tiles and pieces so far; the next tile's entry
  Cursor cur;
  Line line;
  // the next piece with tiles, told to the other roles with its queries; rows
  // that see nothing are written here
  auto begin = [&](Piece& p) {
    bool more;
    while ((more = cur.next(ka.u, p)) && p.nt == 0) {
      const int64_t row = (static_cast<int64_t>(p.b) * a.Hkv + p.hk) * a.R;
      for (int e = lane; e < a.R * (D / 8); e += 32)
        reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + row * D)[e] = make_uint4(0, 0, 0, 0);
      if (lane < a.R) a.lse[row + lane] = -INFINITY;
    }
    const int buf = nq & 1;
    if (nq >= 2 && !wait_all(&bars->q_free[buf], (nq / 2 - 1) & 1)) return false;
    Job& j = bars->jobs[nq % kJobs];
    uint64_t* const job_full = &bars->job_full[nq % kJobs];
    ++nq;
    if (!more) {
      if (lane == 0) {
        j.nt = 0;
        mbar_arrive(job_full);
        mbar_arrive(&bars->q_full[buf]);
      }
      return false;
    }
    entry = entry_of(p.b, p.rows, p.j0);
    if (lane == 0) {
      int i0 = blockIdx.x, n = 1;
      if (!p.whole()) {
        if (p.j0) i0 = line.cta_of(p.at + ka.u.cost_unit);
        n = pieces_of(ka.u, line, p, i0);
      }
      j = {p.b, p.hk, p.len, p.cnt, p.rows, p.j0, p.nt, i0, n};
      mbar_arrive(job_full);
      mbar_arrive_expect_tx(&bars->q_full[buf], a.R * D * 2);
      for (int c = 0; c < NP; ++c)
        tma_load_4d(smem + L::Q_OFF + buf * L::QB + c * NR * 128, &ka.mq, &bars->q_full[buf], 64 * c, 0, p.hk, p.b);
    }
    __syncwarp();
    const int first = entry;
    entry = p.nt > 1 ? entry_of(p.b, p.rows, p.j0 + 1) : 0;
    return load(&ka.mk, place_k(it++), p.hk, p.rows, p.j0, first);
  };
  Piece p;
  bool more = false;
  if (warp == kProd) {
    // the first piece, and its loads on their way before anything else: a short
    // call waits for little but this
    cur = find_part(ka.u, lane, line);
    more = begin(p);
    if (blockIdx.x == 0)
      for (int b = lane; b < a.B; b += 32) report_beyond(a, b);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const uint32_t s0 = smem_u32(smem);

  if (warp == kProd) {
    // --------------------------------------------------- Q, K, jobs
    for (bool ok = more; ok; ok = ok && begin(p))
      for (int j = 1; ok && j < p.nt; ++j) {
        const int now = entry;
        if (j + 1 < p.nt) entry = entry_of(p.b, p.rows, p.j0 + j + 1);
        ok = load(&ka.mk, place_k(it++), p.hk, p.rows, p.j0 + j, now);
      }
    land(true, it ? place_k(it - 1) : -1);
    if (*abort && lane == 0)
      for (int j = nq > 2 ? nq - 2 : 0; j < nq; ++j) mbar_wait_drain(&bars->q_full[j & 1], (j / 2) & 1);
  } else if (warp == kValues) {
    // ------------------------------------------------------------- V
    int i = 0;
    bool ok = true;
    for (int np = 0; ok; ++np) {
      if (!(ok = wait_all(&bars->job_full[np % kJobs], (np / kJobs) & 1))) break;
      const Job p = bars->jobs[np % kJobs];
      if (p.nt == 0) break;
      int next = entry_of(p.b, p.rows, p.j0);
      for (int j = 0; ok && j < p.nt; ++j, ++i) {
        const int now = next;
        if (j + 1 < p.nt) next = entry_of(p.b, p.rows, p.j0 + j + 1);
        ok = load(&ka.mv, place_v(i), p.hk, p.rows, p.j0 + j, now);
      }
    }
    land(false, i ? place_v(i - 1) : -1);
  } else if (warp == kMma) {
    // ---------------------------------------------------------- MMAs
    constexpr uint32_t id_s = idesc_bf16_f32(128, NR, false, false);
    constexpr uint32_t id_o = idesc_bf16_f32(128, NR, true, false);
    bool ok = true;
    int j = 0, nt = 0, np = -1, i = 0, o_ph = 3;   // the tile whose S comes next: j of nt of piece np, the i-th of all
    // the piece after np; none: nt = 0
    auto next_piece = [&] {
      ++np;
      j = nt = 0;
      if ((ok = wait_all(&bars->q_full[np & 1], (np / 2) & 1))) nt = bars->jobs[np % kJobs].nt;
    };
    auto scores = [&] {
      const int place = place_k(i), st = place % RING, qb = np & 1;
      if (!wait_all(&bars->full[st], (place / RING) & 1)) return false;
      tc_fence_after();
      const uint64_t kd = sdesc_sw128(s0 + st * L::TILE, 16, 1024);
      const uint64_t qd = sdesc_sw128(s0 + L::Q_OFF + qb * L::QB, 16, 1024);
#pragma unroll
      for (int c = 0; c < NP; ++c)
        umma4_ss<2, 2>(tmem + NR * (i & 1), sdesc_step(kd, c * PANEL), sdesc_step(qd, c * NR * 128), id_s, c);
      umma_commit_w(&bars->s_full[i & 1]);
      return true;
    };
    next_piece();
    if (ok && nt) ok = scores();
    while (ok && nt) {
      // S of the next tile, perhaps of the next piece, and then P V of this one
      const bool first = j == 0, starts = j < 2;   // of the piece; of its group's O
      const int ob = np & 1, now = i;
      const bool last = ++j == nt;
      ++i;
      if (last) {
        next_piece();
        if (!ok) break;
      }
      if (nt && !(ok = scores())) break;
      const int place = place_v(now), st = place % RING;
      if (!(ok = wait_all(&bars->full[st], (place / RING) & 1))) break;
      if (first) {   // the O of two pieces before has been read
        if (!(ok = wait_all(&bars->o_free[ob], (o_ph >> ob) & 1))) break;
        o_ph ^= 1 << ob;
      }
      if (!(ok = wait_all(&bars->p_full[now & 1], (now / 2) & 1))) break;
      tc_fence_after();
      const uint64_t vd = sdesc_sw128(s0 + st * L::TILE, PANEL, 1024);
      const uint64_t pd = sdesc_sw128(s0 + L::P_OFF + (now & 1) * L::PB, 16, 1024);
      const uint32_t tO = tmem + NR * (2 + 2 * ob + (now & 1));
      umma4_ss<128, 2>(tO, vd, pd, id_o, !starts);
      umma4_ss<128, 2>(tO, sdesc_step(vd, 8192), sdesc_step(pd, NR * 128), id_o, 1);
      if (last) umma_commit_w(&bars->o_full[ob]);
    }
    // every MMA, and every arrival that goes with one, before the memory goes
    umma_commit_w(&bars->drain);
    mbar_wait_drain(&bars->drain, 0);
  } else if (warp >= 4) {
    // ------------------------------------------------------- softmax
    const int group = (warp >> 2) - 1, quad = warp & 3, key = quad * 32 + lane, st = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    float* const wmax = reinterpret_cast<float*>(smem + L::MAX_OFF) + group * 8 * NR;
    float* const wsum = reinterpret_cast<float*>(smem + L::SUM_OFF);
    Sight* const sees = reinterpret_cast<Sight*>(smem + L::SEE_OFF) + group * NR;
    __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(a.o);
    const float sl2 = a.scale_log2;
    int i = 0, np = 0, meet_ph = 0, both_ph = 0;   // tiles and pieces so far
    bool ok = true;
    auto meet = [&] {   // of the group's warps
      warp_arrive(&bars->meet[group], lane);
      ok = wait_all(&bars->meet[group], meet_ph);
      meet_ph ^= 1;
      return ok;
    };
    auto both = [&] {   // of both groups'
      warp_arrive(&bars->both, lane);
      ok = wait_all(&bars->both, both_ph);
      both_ph ^= 1;
      return ok;
    };
    while (true) {
      if (!(ok = wait_all(&bars->job_full[np % kJobs], (np / kJobs) & 1))) break;
      const Job p = bars->jobs[np % kJobs];
      if (p.nt == 0) break;
      const int64_t head_row = (static_cast<int64_t>(p.b) * a.Hkv + p.hk) * a.R;   // of o and lse
      const int i0 = p.i0, n = p.n;
      const bool whole = n == 1;
      if (st < NQ) sees[st] = st < a.R ? sight(a, p.b, st % a.T, Held{p.len, p.cnt}, p.rows) : Sight{0, 0};
      float m[NQ], l[NQ];
#pragma unroll
      for (int r = 0; r < NQ; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
      }
      const uint32_t tO0 = tmem + NR * (2 + 2 * (np & 1)) + lane_off, tO = tO0 + NR * group;
      const int begin = (i ^ group) & 1, end = i + p.nt;   // this group's first tile; behind the last of all
      i += begin;
      for (int k = begin; k < p.nt; k += 2, i += 2) {
        const int k0 = (p.j0 + k) * BN;
        if (!(ok = wait_all(&bars->s_full[i & 1], (i / 2) & 1))) break;
        tc_fence_after();
        if (st == 0) {   // S came behind P V of the group's tile before: what they read is free
          mbar_arrive(&bars->free[place_k(i) % RING]);
          if (i >= 2) mbar_arrive(&bars->free[place_v(i - 2) % RING]);
          if (k == p.nt - 1) mbar_arrive(&bars->q_free[np & 1]);
        }
        uint32_t y[NQ];
        tmem_row(tmem + NR * (i & 1) + lane_off, y);
        float x[NQ];
#pragma unroll
        for (int r = 0; r < NQ; ++r) x[r] = __uint_as_float(y[r]) * sl2;
        if (k0 + BN > p.len) {
          const int off = k0 + key - p.len;   // which of the newest tokens' rows it is
          if (k == begin && !meet()) break;   // what rows see is there
#pragma unroll
          for (int r = 0; r < NQ; ++r) {
            const Sight v = sees[r];
            const bool seen = k0 + key < v.full || (off >= 0 && off < 64 && (v.word >> off & 1));
            if (!seen) x[r] = -INFINITY;
          }
        }
        // the tile's maxima of all rows, by all threads alike
        float t[NQ];
#pragma unroll
        for (int r = 0; r < NQ; ++r) t[r] = x[r];
        const float mine = across<NQ>(t, lane, [](float u, float v) { return fmaxf(u, v); });
        float* const wm = wmax + (i >> 1 & 1) * 4 * NR;
        if (lane < NQ) wm[quad * NR + lane] = mine;
        if (!meet()) break;
        bool grows = false;
#pragma unroll
        for (int r = 0; r < NQ; r += 4) {
          const float4 u = *reinterpret_cast<const float4*>(wm + r), v = *reinterpret_cast<const float4*>(wm + NR + r);
          const float4 w = *reinterpret_cast<const float4*>(wm + 2 * NR + r), z = *reinterpret_cast<const float4*>(wm + 3 * NR + r);
          t[r] = fmaxf(fmaxf(u.x, v.x), fmaxf(w.x, z.x));
          t[r + 1] = fmaxf(fmaxf(u.y, v.y), fmaxf(w.y, z.y));
          t[r + 2] = fmaxf(fmaxf(u.z, v.z), fmaxf(w.z, z.z));
          t[r + 3] = fmaxf(fmaxf(u.w, v.w), fmaxf(w.w, z.w));
        }
#pragma unroll
        for (int r = 0; r < NQ; ++r) grows |= t[r] > m[r] + kRescaleLog2;
        if (grows) {
#pragma unroll
          for (int r = 0; r < NQ; ++r) {
            const bool up = t[r] > m[r] + kRescaleLog2;
            const float f = up ? ex2(m[r] - t[r]) : 1.f;   // m = -inf gives 0
            m[r] = up ? t[r] : m[r];
            l[r] *= f;
            t[r] = f;
          }
          if (k != begin) {
            uint32_t o[NQ];
            tmem_row(tO, o);
#pragma unroll
            for (int r = 0; r < NQ; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * t[r]);
            tmem_put_row(tO, o);
            tmem_wait_st();
          }
        }
        // Weights, by rows of 128 keys: two panels, swizzled.  bf16 for the product with V, which
        // the MMA takes no other way beside bf16 values; their sum is of the fp32 ones.
        uint8_t* const ps = smem + L::P_OFF + (i & 1) * L::PB + (key >> 6) * (NR * 128) + (key & 7) * 2;
#pragma unroll
        for (int r = 0; r < NQ; ++r) {
          const float w = ex2(x[r] - (m[r] == -INFINITY ? 0.f : m[r]));
          l[r] += w;
          *reinterpret_cast<__nv_bfloat16*>(ps + r * 128 + ((((key & 63) >> 3) ^ (r & 7)) << 4)) = __float2bfloat16_rn(w);
        }
        if (k0 + BN > p.rows) {
          // the request's last tile: rows of V behind it may hold anything
          const int place = place_v(i), slot = place % RING, left = p.rows - k0;
          if (!(ok = wait_all(&bars->full[slot], (place / RING) & 1))) break;
          uint8_t* v = smem + slot * L::TILE;
          for (int e = st; e < (BN - left) * (D / 8); e += 128) {
            const int vr = left + e / (D / 8), q = e % (D / 8);
            *reinterpret_cast<uint4*>(v + (q >> 3) * PANEL + vr * 128 + (q & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_async_smem();
        tc_fence_before();
        warp_arrive(&bars->p_full[i & 1], lane);
      }
      if (!ok) break;
      i = end;
      // ---- the piece's end: sums of all keys; thread = feature from here on
      float* const tops = reinterpret_cast<float*>(smem + L::TOP_OFF) + (np & 1) * 2 * NR;
      const float part = across<NQ>(l, lane, [](float u, float v) { return u + v; });
      if (lane < NQ) wsum[(4 * group + quad) * NR + lane] = part;
      if (st == 0)
#pragma unroll
        for (int r = 0; r < NQ; ++r) tops[group * NR + r] = m[r];
      if (!both()) break;
      const int at = (blockIdx.x * 2 + (p.j0 == 0)) * NR;   // of this piece's partials
      if (group == 0 && st < a.R) {
        const Sight v = sees[st];
        float sum[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float* const w = wsum + 4 * g * NR + st;
          sum[g] = (w[0] + w[NR]) + (w[2 * NR] + w[3 * NR]);
        }
        const float m0 = tops[st], m1 = tops[NR + st], top = fmaxf(m0, m1), base = top == -INFINITY ? 0.f : top;
        const float w0 = ex2(m0 - base), w1 = ex2(m1 - base), total = w0 * sum[0] + w1 * sum[1];
        const bool none = total == 0.f || (v.full == 0 && v.word == 0);
        const float lse2 = none ? -INFINITY : base + log2f(total), f = none ? 0.f : 1.f / total;
        if (whole) a.lse[head_row + st] = lse2 * kLn2;
        else ka.part_lse[at + st] = lse2;
        // 0: nothing of what is in that O.  (Padding's sums hold keys that it does not see: with an
        // infinite score w0 is NaN.)
        tops[st] = none ? 0.f : w0 * f;
        tops[NR + st] = none ? 0.f : w1 * f;
      }
      if (!(ok = wait_all(&bars->o_full[np & 1], (np / 2) & 1))) break;
      if (!both()) break;
      tc_fence_after();
#pragma unroll 1
      for (int r0 = 4 * group; r0 < a.R; r0 += 8) {   // (in a loop: its code is fetched for every few calls)
        uint32_t o0[4], o1[4];
        tmem_row(tO0 + r0, o0);
        tmem_row(tO0 + NR + r0, o1);
        const float4 f0 = *reinterpret_cast<const float4*>(tops + r0), f1 = *reinterpret_cast<const float4*>(tops + NR + r0);
        const float u[4] = {f0.x, f0.y, f0.z, f0.w}, v[4] = {f1.x, f1.y, f1.z, f1.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = (u[e] == 0.f ? 0.f : __uint_as_float(o0[e]) * u[e]) + (v[e] == 0.f ? 0.f : __uint_as_float(o1[e]) * v[e]);
          if (r0 + e < a.R && (D == 128 || key < D)) {
            if (whole) out[(head_row + r0 + e) * D + key] = __float2bfloat16_rn(x);
            else ka.part_o[static_cast<int64_t>(at + r0 + e) * D + key] = x;
          }
        }
      }
      tc_fence_before();
      warp_arrive(&bars->o_free[np & 1], lane);
      ++np;
      if (!whole) {
        // ---- a cut unit: its last CTA joins the pieces, a warp a row
        if (!both()) break;   // partials are written
        if (threadIdx.x == 128) {
          const bool all = add_acq_rel(&ka.counters[i0], 1) == n - 1;
          if (all) ka.counters[i0] = 0;
          bars->last = all;
        }
        if (!both()) break;
        if (bars->last) {
          // a warp a row, or two rows at once; what goes first is read with the lse,
          // not behind it
          constexpr int W4 = D / 4, PER = 32 / W4, Q = (kMaxCtas + 31) / 32;   // pieces that a load brings
          constexpr int N2 = NQ > 8 ? 2 : 1, V = 8 / N2;
          const int c = lane % W4, half = lane / W4, r0 = 4 * group + quad;
          auto at_of = [&](int t, int r) { return ((i0 + t) * 2 + (t == 0)) * NR + r; };
          float4 v[N2][V];
          auto get = [&](int t0) {
#pragma unroll
            for (int i = 0; i < N2; ++i)
#pragma unroll
              for (int e = 0; e < V; ++e) {
                const int t = t0 + e * PER + half, r = r0 + 8 * i;
                v[i][e] = t < n && r < a.R
                              ? __ldcg(reinterpret_cast<const float4*>(ka.part_o + static_cast<int64_t>(at_of(t, r)) * D) + c)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
              }
          };
          get(0);
          float w[N2][Q], base[N2], sum[N2];
          float4 acc[N2];
#pragma unroll
          for (int i = 0; i < N2; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
              const int t = 32 * q + lane, r = r0 + 8 * i;
              w[i][q] = t < n && r < a.R ? __ldcg(ka.part_lse + at_of(t, r)) : -INFINITY;
              mx = fmaxf(mx, w[i][q]);
            }
            for (int o2 = 16; o2; o2 >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o2));
            base[i] = mx == -INFINITY ? 0.f : mx;
            sum[i] = 0.f;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
              w[i][q] = ex2(w[i][q] - base[i]);
              sum[i] += w[i][q];
            }
            for (int o2 = 16; o2; o2 >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o2);
            acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          }
#pragma unroll
          for (int q = 0; q < Q; ++q)
            for (int t0 = 32 * q; t0 < min(n, 32 * q + 32); t0 += V * PER) {
              if (t0) get(t0);
#pragma unroll
              for (int i = 0; i < N2; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                  const float f = __shfl_sync(0xffffffffu, w[i][q], (t0 + e * PER + half) & 31);
                  acc[i].x = fmaf(f, v[i][e].x, acc[i].x);
                  acc[i].y = fmaf(f, v[i][e].y, acc[i].y);
                  acc[i].z = fmaf(f, v[i][e].z, acc[i].z);
                  acc[i].w = fmaf(f, v[i][e].w, acc[i].w);
                }
            }
#pragma unroll
          for (int i = 0; i < N2; ++i) {
            const int r = r0 + 8 * i;
            if (PER == 2) {
              acc[i].x += __shfl_xor_sync(0xffffffffu, acc[i].x, 16);
              acc[i].y += __shfl_xor_sync(0xffffffffu, acc[i].y, 16);
              acc[i].z += __shfl_xor_sync(0xffffffffu, acc[i].z, 16);
              acc[i].w += __shfl_xor_sync(0xffffffffu, acc[i].w, 16);
            }
            const float f = sum[i] == 0.f ? 0.f : 1.f / sum[i];
            if (half == 0 && r < a.R)
              *reinterpret_cast<uint2*>(out + (head_row + r) * D + 4 * c) =
                  make_uint2(pack_bf16x2(acc[i].x * f, acc[i].y * f), pack_bf16x2(acc[i].z * f, acc[i].w * f));
            if (lane == 0 && r < a.R) a.lse[head_row + r] = sum[i] == 0.f ? -INFINITY : (base[i] + log2f(sum[i])) * kLn2;
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  report_abort(abort, a.status);
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kColumns);
  }
}

template <int D, int NQ>
static cudaError_t launch(const Args& k, cudaStream_t st) {
  constexpr int smem = Layout<D>::SMEM;
  static std::atomic<bool> done[kMaxCachedDevices];
  const cudaError_t e = allow_smem(few_kernel<D, NQ>, smem, done);
  if (e != cudaSuccess) return e;
  return launch_early(few_kernel<D, NQ>, dim3(k.u.G), kThreads, smem, st, k);
}
template <int D>
static cudaError_t launch_rows_of(const Args& k, cudaStream_t st) {
  const int R = k.u.a.R;
  return R <= 4 ? launch<D, 4>(k, st) : R <= 8 ? launch<D, 8>(k, st) : launch<D, 16>(k, st);
}

constexpr int64_t kHeadFloats = 1024;   // the counters, in front of the partials
static_assert(kMaxCtas <= kHeadFloats, "counters");

}  // namespace paged_few

using namespace paged_few;

int64_t paged_few_workspace(int D) {
  return (kHeadFloats + static_cast<int64_t>(kMaxCtas) * 2 * kPagedFewRows * (D + 1)) * 4;
}

int paged_few_attend(const PagedArgs& a, int D, int sms, float* ws, cudaStream_t stream) {
  Args k = {};
  const int tile = D == 128 ? kCost128 : kCost64;
  SCA_REQUIRE(make_units(k.u, a, sms, tile, tile, kCostUnit, kCostWhole, 1), SCA_ERR_UNSUPPORTED,
              "paged_tree_attend: more than about 2^28 tiles of 128 rows");
  k.box_log2 = a.page_log2 < 7 ? a.page_log2 : 7;
  k.counters = reinterpret_cast<int32_t*>(ws);
  k.part_lse = ws + kHeadFloats;
  k.part_o = k.part_lse + kMaxCtas * 2 * kPagedFewRows;
  const int page = 1 << a.page_log2;
  const View q{a.q_b, static_cast<int64_t>(a.R) * D, D};
  cudaError_t e = make_tmap_bf16(&k.mq, a.q, D, a.R, a.Hkv, a.B, q, 64, a.R);
  if (e == cudaSuccess)
    e = make_tmap_bf16(&k.mk, a.kp, D, page, a.Hkv, static_cast<int>(a.pages), a.pool, 64, 1 << k.box_log2);
  if (e == cudaSuccess)
    e = make_tmap_bf16(&k.mv, a.vp, D, page, a.Hkv, static_cast<int>(a.pages), a.pool, 64, 1 << k.box_log2);
  SCA_REQUIRE(e == cudaSuccess, SCA_ERR_ALIGN, "paged_tree_attend: layout not expressible as a TMA tensor map");
  e = D == 64 ? launch_rows_of<64>(k, stream) : launch_rows_of<128>(k, stream);
  return cuda_status(e, "paged_tree_attend (tensor cores, few rows)");
}

}  // namespace sca
