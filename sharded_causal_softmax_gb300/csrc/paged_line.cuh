// How the tensor-core kernels of the paged cache share out their work: all units'
// tiles of 128 rows on one line, weighted by what they cost, of which every CTA
// takes a part, whatever the lengths.  A unit is what reads one request's rows of
// one key/value head for the same query rows: up to two row tiles of 128.
#pragma once

#include "paged.h"

namespace sca {
namespace paged_line {

constexpr int BN = 128;
constexpr int kMaxCtas = 160;

struct Units {
  PagedArgs a;
  int32_t row_tiles, pairs;   // of a request and key/value head
  int32_t G;                  // CTAs
  // What a tile of one and of two row tiles costs, and a unit's start and end
  // (the last, writing and joining partials in it); units of up to cost_whole
  // are not cut.
  int32_t cost_one, cost_two, cost_unit, cost_whole;
  int32_t least;              // tiles of a CTA, where there is less work than for all of them
};

// Places are 32-bit numbers (the host refuses more).

SCA_INLINE int unit_cost(const Units& k, int T, bool two) { return T * (two ? k.cost_two : k.cost_one) + k.cost_unit; }
// of a request that holds T tiles, over its key/value heads
SCA_INLINE int request_cost(const Units& k, int T) {
  return k.a.Hkv * ((k.row_tiles / 2) * unit_cost(k, T, true) + (k.row_tiles & 1) * unit_cost(k, T, false));
}
SCA_INLINE int tiles_of(const Units& k, int b) {
  const Held h = held(k.a, b);
  return h.cnt ? (rows_of(k.a, h) + BN - 1) / BN : 0;
}

// Tokens in a row see no further than the last of them, so that the later pairs of
// a long prompt see up to all of it and the first ones little: each has places on the
// line for what it sees (all places alike, and those of unseen tiles empty, a prompt of
// 32768 rows took 2.9 ms instead of 1.6).
SCA_INLINE int seen_tiles(const Units& k, int len, int cnt, int rows, int rp) {
  const int r0 = rp * 256, r1 = min(r0 + 256, k.a.R) - 1;
  const int t0 = r0 % k.a.T, t1 = r0 / k.a.T == r1 / k.a.T ? r1 % k.a.T : k.a.T - 1;
  const int see = r0 / k.a.T == r1 / k.a.T && t0 >= cnt ? 0 : min(rows, len + t1 + 1);
  return (see + BN - 1) / BN;
}
// The cost of a head's pairs, up to where it passes `upto`; `rp`: that pair.  (In kernels
// of their own, kUneven: in all, it cost calls of few rows 1 to 5 us.)
SCA_INLINE int uneven_cost(const Units& k, int b, int upto, int* rp) {
  const Held h = held(k.a, b);
  const int rows = h.cnt ? rows_of(k.a, h) : 0;
  int sum = 0, i = 0;
  for (; i < k.pairs; ++i) {
    const int cost = unit_cost(k, seen_tiles(k, h.len, h.cnt, rows, i), 2 * i + 1 < k.row_tiles);
    if (sum + cost > upto) break;
    sum += cost;
  }
  *rp = i;
  return sum;
}

// CTA i of G takes [start(i), start(i + 1)) of a line W long.
struct Line {
  int W, G, q, r;
  SCA_INLINE Line() : W(0), G(1), q(0), r(0) {}
  SCA_INLINE Line(int W_, int G_) : W(W_), G(G_), q(W_ / G_), r(W_ % G_) {}
  SCA_INLINE int start(int i) const { return i >= G ? W : q * i + r * i / G; }
  // whose part holds `pos`
  SCA_INLINE int cta_of(int pos) const {
    int i = static_cast<int>(__fdividef(static_cast<float>(pos) * static_cast<float>(G), static_cast<float>(W)));
    i = i < G ? i : G - 1;
    while (i + 1 < G && start(i + 1) <= pos) ++i;
    while (i > 0 && start(i) > pos) --i;
    return i;
  }
};

struct Piece {
  int b, hk, rt;           // request, key/value head, first row tile
  int len, cnt, rows;      // what the request holds
  int j0, nt;              // tiles [j0, j0 + nt); none: the unit's rows see nothing
  int at, tiles;           // of its unit: where it starts on the line, its tiles
  bool two;
  SCA_INLINE bool whole() const { return nt == tiles; }
};

// Walks the units from (b, hk, rp) on: a request's numbers are found once for all
// of its units.
struct Cursor {
  int lo, hi, at;          // this CTA's part of the line; where the unit starts
  int b, hk, rp;           // request, key/value head, pair of row tiles
  int len, cnt, rows;      // what the request holds, once `known`
  bool known;
  template <bool kUneven = false>
  SCA_INLINE bool next(const Units& k, Piece& p) {
    while (at < hi && b < k.a.B) {
      if (!known) {
        const Held h = held(k.a, b);
        len = h.len;
        cnt = h.cnt;
        rows = h.cnt ? rows_of(k.a, h) : 0;
        known = true;
      }
      p.b = b;
      p.hk = hk;
      p.rt = 2 * rp;
      p.two = p.rt + 1 < k.row_tiles;
      p.len = len;
      p.cnt = cnt;
      p.rows = rows;
      const int T = (rows + BN - 1) / BN, w = p.two ? k.cost_two : k.cost_one, first = at + k.cost_unit;
      p.at = at;
      // Rows of tokens in a row see no further than their last; of few rows the tiles
      // behind that have places on the line, but nobody takes them.
      p.tiles = k.a.tree == nullptr && k.a.T > 1 ? seen_tiles(k, len, cnt, rows, rp) : T;
      const int cost = unit_cost(k, kUneven ? p.tiles : T, p.two), mid = at + cost / 2;
      const bool mine = mid >= lo && mid < hi;   // of one that is not cut
      at += cost;
      if (++rp == k.pairs) {
        rp = 0;
        if (++hk == k.a.Hkv) {
          hk = 0;
          ++b;
          known = false;
        }
      }
      if (cost <= k.cost_whole || p.tiles == 0) {
        p.j0 = 0;
        p.nt = p.tiles;
        if (mine) return true;
        continue;
      }
      p.j0 = (max(lo - first, 0) + w - 1) / w;
      p.nt = min(p.tiles, (max(hi - first, 0) + w - 1) / w) - p.j0;
      if (p.nt > 0) return true;
    }
    return false;
  }
};

// Pieces of a cut unit, by CTAs i0, i0 + 1, ...
SCA_INLINE int pieces_of(const Units& k, const Line& line, const Piece& p, int i0) {
  return line.cta_of(p.at + k.cost_unit + (p.tiles - 1) * (p.two ? k.cost_two : k.cost_one)) - i0 + 1;
}
// One thread speaks for its CTA: what the others wrote before a barrier that it
// waited for is released with its own, and what it acquires they may read (past
// the L1 cache) behind the next.
SCA_INLINE int load_acquire(const int32_t* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
SCA_INLINE int add_acq_rel(int32_t* p, int x) {
  int v;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;" : "=r"(v) : "l"(p), "r"(x) : "memory");
  return v;
}

// this CTA's part of the line and the unit it starts in (one warp)
template <bool kUneven = false>
SCA_INLINE Cursor find_part(const Units& k, int lane, Line& line) {
  const int each = (k.a.B + 31) / 32;   // requests of a lane
  auto scan = [&](int x) {              // this lane's and those before it
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += v;
    }
    return x;
  };
  auto cost_of = [&](int b) {
    if (b >= k.a.B) return 0;
    int rp;
    return kUneven ? k.a.Hkv * uneven_cost(k, b, 0x7fffffff, &rp) : request_cost(k, tiles_of(k, b));
  };
  int cost = 0;
#pragma unroll 4
  for (int i = 0; i < each; ++i) cost += cost_of(lane * each + i);
  int sums = scan(cost);
  // No part is shorter than a tile, so that a unit's pieces are consecutive CTAs'.
  const int all = __shfl_sync(0xffffffffu, sums, 31), w = k.row_tiles > 1 ? k.cost_two : k.cost_one;
  line = Line(all, max(1, min(k.G, all / (w * k.least))));
  const int i = blockIdx.x, lo = line.start(i), hi = line.start(i + 1);
  // requests before the one that holds lo: whole lanes, then those of one lane
  int at = 0, b = 0;
  auto skip = [&](int upto, int step) {
    const uint32_t past = __ballot_sync(0xffffffffu, at + upto > lo);
    const int cnt = past ? __ffs(past) - 1 : 32;
    const int skipped = __shfl_sync(0xffffffffu, upto, cnt ? cnt - 1 : 0);
    if (cnt) at += skipped;
    b += cnt * step;
    return past != 0;
  };
  if (skip(sums, each) && each > 1) {
    const int end = b + each;
    while (true) {
      const int at_lane = b + lane;
      if (skip(scan(at_lane < end ? cost_of(at_lane) : 0), 1) || b >= end) break;
    }
  }
  int hk = 0, rp = 0;
  if (b < k.a.B) {   // units of that request before the one that holds lo
    if (kUneven) {
      const int head = uneven_cost(k, b, 0x7fffffff, &rp);
      hk = (lo - at) / head;
      at += hk * head;
      at += uneven_cost(k, b, lo - at, &rp);
    } else {
      const int T = tiles_of(k, b), head = request_cost(k, T) / k.a.Hkv, two = unit_cost(k, T, true);
      const int rem = lo - at;
      hk = rem / head;
      rp = min((rem - hk * head) / two, k.pairs - 1);
      at += hk * head + rp * two;
    }
  }
  return Cursor{lo, hi, at, b, hk, rp, 0, 0, 0, false};
}

// whether the pairs of a request see different numbers of rows
inline bool uneven(const Units& k) { return k.a.tree == nullptr && k.a.T > 1 && k.pairs > 1; }

// The host's side: units of R query rows; false: places pass 32 bits.
inline bool make_units(Units& k, const PagedArgs& a, int sms, int one, int two, int unit, int whole, int least) {
  k.a = a;
  k.row_tiles = (a.R + 127) / 128;
  k.pairs = (k.row_tiles + 1) / 2;
  k.G = sms < kMaxCtas ? sms : kMaxCtas;
  k.cost_one = one;
  k.cost_two = two;
  k.cost_unit = unit;
  k.cost_whole = whole;
  k.least = least;
  const double tiles = static_cast<double>((static_cast<int64_t>(a.table_n) << a.page_log2) / BN + 1);
  return static_cast<double>(a.B) * a.Hkv * k.pairs * (tiles * two + unit) < 2e9;
}

}  // namespace paged_line
}  // namespace sca
