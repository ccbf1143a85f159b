// Decode attention over a shared prefix and each request's own suffix: the
// arguments of its kernels (prefix.cu: fp32 arithmetic and the merge;
// prefix_tc.cu: tensor cores).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace sca {

// The query rows of one request and key/value head are R = group * T rows
// (head within the group, then token) that lie one after the other, so row r
// of request b and key/value head hk is row (b Hkv + hk) R + r of o and lse,
// and of q but for q's own batch stride.  Keys go in pieces of `piece` rows;
// slot p < n_prefix of a row's partials is prefix piece p, slot n_prefix + s
// piece s of the request's suffix (written only if it starts below the
// suffix's length).
struct PrefixArgs {
  const void *q, *kp, *vp, *ks, *vs;
  const int32_t* lengths;
  void* o;
  float* lse;
  float* part_o;       // [rows][slots][D] normalised partial outputs
  float* part_lse;     // [rows][slots] their lse, base 2
  int64_t q_b;
  View pv, sv;         // prefix (b unused) and suffix views
  int64_t prefix_len, suffix_cap, piece;
  int32_t B, Hkv, R, T;
  int32_t n_prefix, n_suffix, slots;
  float scale_log2;
  int* status;
};

__device__ __forceinline__ int64_t suffix_len(const PrefixArgs& a, int b) {
  const int64_t n = a.n_suffix ? a.lengths[b] : 0;
  return n < 0 ? 0 : min64(n, a.suffix_cap);
}

// Tensor-core path (prefix_tc.cu), with a cut of its own: bytes of workspace,
// and the step (part_o, part_lse, piece and the slot counts of `a` unused).
int64_t prefix_tc_workspace(int B, int Hkv, int R, int D, int64_t prefix_len, int64_t suffix_cap, int sms);
int prefix_tc_decode(const PrefixArgs& a, int D, int sms, float* ws, cudaStream_t stream);

}  // namespace sca
