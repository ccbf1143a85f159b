// A cache of keys and values in pages, and attention of drafted tokens over
// it: the arguments of its kernels (paged.cu: checks, acceptance, fp32
// arithmetic; paged_f32.cu: that of many rows; paged_tc.cu, paged_few.cu: tensor
// cores).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace sca {

// The query rows of one request and key/value head are R = group * T rows (head
// within the group, then token) that lie one after the other: row r of request
// b and key/value head hk is row (b Hkv + hk) R + r of o and lse, and of q but
// for q's own batch stride.
struct PagedArgs {
  const void *q, *kp, *vp;
  const int32_t *table, *lengths, *counts;   // counts NULL: T
  const uint64_t* tree;                      // NULL: each token sees those up to itself
  void* o;
  float* lse;
  int64_t q_b, table_b, tree_b, pages;
  View pool;                                 // page, head, row
  int32_t B, Hkv, R, T, page_log2, table_n;
  float scale_log2;
  int* status;
};

// What a request holds: `len` rows that every token sees, `cnt` newest tokens'
// behind them, no more than its table reaches.
struct Held {
  int32_t len, cnt;
};
SCA_INLINE Held held(const PagedArgs& a, int b) {
  const int64_t cap = static_cast<int64_t>(a.table_n) << a.page_log2;
  int64_t n = a.lengths[b], c = a.counts ? a.counts[b] : a.T;
  n = n < 0 ? 0 : min64(n, cap);
  c = c < 0 ? 0 : min64(c, a.T);
  return {static_cast<int32_t>(n), static_cast<int32_t>(c)};
}
// the rows that are there (fewer than len + cnt behind a table's end)
SCA_INLINE int32_t rows_of(const PagedArgs& a, Held h) {
  return static_cast<int32_t>(min64(static_cast<int64_t>(h.len) + h.cnt, static_cast<int64_t>(a.table_n) << a.page_log2));
}

// records a request whose rows do not fit its table
SCA_INLINE void report_beyond(const PagedArgs& a, int b) {
  const int64_t c = a.counts ? a.counts[b] : a.T;
  if (max(a.lengths[b], 0) + (c < 0 ? 0 : min64(c, a.T)) > static_cast<int64_t>(a.table_n) << a.page_log2)
    report(a.status, SCA_ERR_RANGE);
}

// Which rows token t of a request sees: the first `full` and, of the 64 from
// `len` on, those in `word`.
struct Sight {
  int32_t full;
  uint64_t word;
};
SCA_INLINE Sight sight(const PagedArgs& a, int b, int t, Held h, int32_t rows) {
  if (t >= h.cnt) return {0, 0};
  if (a.tree == nullptr) return {static_cast<int32_t>(min64(rows, static_cast<int64_t>(h.len) + t + 1)), 0};
  const int32_t n = rows - h.len;   // the newest rows that are there, at most 64
  return {h.len, a.tree[b * a.tree_b + t] & (n >= 64 ? ~0ull : (1ull << n) - 1)};
}
// bit c: row s0 + c is seen (c < 32)
SCA_INLINE uint32_t seen_bits(Sight v, int32_t len, int32_t s0) {
  const int32_t n = v.full - s0, off = s0 - len;
  uint32_t bits = n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1);
  if (v.word) {
    if (off >= 0) bits |= off < 64 ? static_cast<uint32_t>(v.word >> off) : 0u;
    else if (off > -32) bits |= static_cast<uint32_t>(v.word) << -off;
  }
  return bits;
}

// fp32 arithmetic: rows in tiles, keys in `splits` pieces (in turn: tile, tile +
// splits, ...; with clusters, each of `cluster` CTAs), whose partials a launch of
// its own joins.
struct PagedSplit {
  PagedArgs a;
  float* part_o;      // [rows of all][splits][D] normalised partial outputs
  float* part_lse;    // [rows of all][splits] their lse, base 2
  int32_t cluster, splits, row_tiles;
};
constexpr int kPagedSplits = 64;   // at most

// Of many query rows a head (paged_f32.cu).  `most`: pieces that no shorter table has more of.
PagedSplit paged_f32_cut(const PagedArgs& a, int sms, int* most);
cudaError_t paged_f32_launch(const PagedSplit& k, int D, cudaStream_t stream);

// Tensor-core paths: bytes of workspace, and the step.  Of up to kPagedFewRows
// query rows a key/value head (paged_few.cu), and of any number (paged_tc.cu).
constexpr int kPagedFewRows = 16;
int64_t paged_few_workspace(int D);
int paged_few_attend(const PagedArgs& a, int D, int sms, float* ws, cudaStream_t stream);
int64_t paged_tc_workspace(int D, int sms);
int paged_tc_attend(const PagedArgs& a, int D, int sms, float* ws, cudaStream_t stream);

}  // namespace sca
