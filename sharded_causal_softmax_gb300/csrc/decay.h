// Linear attention with a decay per head: the one recurrence that the
// forward and every gradient are passes of, and the launchers of its kernels
// (decay.cu: fp32 arithmetic; decay_tc.cu: tensor cores).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "overlap.cuh"

namespace sca {

// One pass over a batch of sequences.  With n rows in processing order
// (rising row numbers, or falling ones when `reverse`) and lambda = exp(g_h):
//
//   S_t   = lambda S_{t-1} + us y_t^T z_t
//   out_t = si lambda x_t S_{t-1} + so (x_t . y_t) z_t + ...
//         = so sum_{s <= t} lambda^(t-s) (x_t . y_s) z_s + si lambda^(t+1) x_t S_0
//
//   pass   x   y   z   direction  state (row, column)     so     si     us
//   o      q   k   v   forward    k, v                    scale  scale  1
//   dq     dO  v   k   forward    v, k: transposed        scale  scale  1
//   dk     v   dO  q   reverse    dO, q: transposed       scale  1      scale
//   dv     k   q   dO  reverse    q, dO                   scale  1      scale
//
// A gradient of the state after the last row enters a reverse pass at that
// row itself, not one row before it: its power is one lower (`delta` in the
// kernels) until the first row has been taken.
struct DecayPass {
  const void *x, *y, *z;
  void* out;
  View xv, yv, zv, ov;
  const float* log_decay;     // [H], <= 0
  const int32_t* lengths;     // [B] or NULL (every row)
  const float* init;          // [.][H][D][D] state before the first row, or NULL (zero)
  int64_t init_b;             // its batch stride (0: shared by the batch)
  float* seg;                 // [BH][nseg][D][D] state before each segment, in processing order; NULL when nseg = 1
  float* end;                 // [B][H][D][D] state after the last row (reverse: times lambda), or NULL
  int64_t S, seg_rows;
  int32_t B, H, nseg;
  int32_t reverse;
  int32_t exact;              // the state is handed out: keep it fp32 throughout
  int32_t transposed;         // init and seg hold the transpose of this pass's state (no sums, no end then)
  float so, si, us;
  int* status;
};

constexpr int kDecaySub = 128;   // rows of a chunk of the tensor-core kernels
constexpr int kDecayBlk = 64;    // rows of a chunk of the fp32 kernels

// exp(g n): the product's rounding error is put back, so that the power is
// within a few units of the last place of fp32 also where |g n| is large.
// g = -inf (a decay of zero) gives 1 for n = 0 and 0 otherwise.
SCA_INLINE float decay_pow(float g, int64_t n) {
  if (n == 0) return 1.f;
  const float fn = static_cast<float>(n);   // n < 2^24 for every use
  const float p = g * fn;
  if (p < -104.f) return 0.f;               // below the smallest fp32
  return expf(p) * (1.f + fmaf(g, fn, -p));
}

// Rows [lo, hi) of segment i (processing order) that belong to a sequence of
// `len` rows, and the segment's end s1 among the padded rows.
struct DecayRows {
  int64_t lo, hi, s1;
};
__host__ __device__ __forceinline__ DecayRows decay_rows(const DecayPass& p, int i, int64_t len) {
  const int64_t j = p.reverse ? p.nseg - 1 - i : i;
  DecayRows r;
  r.lo = j * p.seg_rows;
  r.s1 = min64(p.S, r.lo + p.seg_rows);
  r.hi = min64(r.s1, len);
  if (r.hi < r.lo) r.hi = r.lo;
  return r;
}

__device__ __forceinline__ int64_t decay_len(const DecayPass& p, int b) {
  if (!p.lengths) return p.S;
  const int64_t n = p.lengths[b];
  return n < 0 ? 0 : min64(n, p.S);
}

// Tensor-core passes (bf16, decay_tc.cu).  states: the segments' own sums
// into p.seg (processing order, the last one skipped where nobody asks for the
// end); else a forward's whole pass.
int decay_tc_pass(const DecayPass& p, int D, bool states, cudaStream_t stream);
// the three gradients' passes (their states before the segments summed)
int decay_tc_backward(const DecayPass& dq, const DecayPass& dv, const DecayPass& dk, int D, cudaStream_t stream);

}  // namespace sca
