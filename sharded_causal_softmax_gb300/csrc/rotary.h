// Rows turned to their positions, in place of themselves or into the pages of
// a cache: the arguments of its kernel (rotary.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "disjoint.h"
#include "sca.h"

namespace sca {

// Tensors 0 and 1 are turned, 2 is copied; the heads of all three are numbered
// one after the other.  With a table, tensors 1 and 2 go to a pool's pages
// (`out` strides: page, head, row) and rows at or past counts are padding.
struct RowsArgs {
  const void* in[3];
  void* out[3];
  View iv[3], ov[3];
  int32_t heads[3];
  int64_t B, S;
  int32_t D, rd, interleaved;
  float amplitude, sign;       // sign -1: the transposed matrix
  const uint64_t* turns;
  const int32_t* positions;    // NULL: the row's own place
  int64_t pos_b;
  const int32_t *table, *lengths, *counts;
  int64_t table_b, pages;
  int32_t table_n, page_log2;
  int32_t chunk;               // heads of a CTA
  int* status;
};

// The rows of a [B, H, S, D] view at x, for share_bytes.
inline Rows row_set(const void* x, const sca_view& v, int64_t B, int64_t H, int64_t S, int64_t D, int64_t eb) {
  return {x, D * eb, {v.b * eb, v.h * eb, v.s * eb}, {B, H, S}};
}

// Launches over all rows and heads (fills in chunk); dtype: sca_dtype.
cudaError_t launch_rows(RowsArgs a, int dtype, cudaStream_t st);

}  // namespace sca
