// One tile of an online softmax in tensor memory: a thread holds a query row,
// whose scores become P (bf16) where they lie.
#pragma once

#include "ptx.cuh"

namespace sca {

// A row's maximum is followed when it has grown by more than 2^this.
constexpr float kRescaleLog2 = 8.0f;

// columns whose bit of `bits` is clear to -inf
SCA_INLINE void mask_columns(uint32_t (&y)[32], uint32_t bits) {
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (!(bits & (1u << c))) y[c] = 0xff800000u;
}

// The 128 scores of this thread's row at tS (tensor memory) to P = exp(scale
// s - 2^m), rounded to bf16, over them; m and l the row's running maximum (base
// 2) and sum; O at tO (D columns) is rescaled with them where `has_o`.  mask(y,
// h) hides columns of the 32 from 32 h on.  All 32 lanes of the warp call it.
//
// One pass, 32 columns at a time in a short loop (held in registers all at once
// they would be four times the code, and fetching code is what a short call
// waits for).  A row's numbers are relative to 2^m, which follows its maximum
// only when that has grown by more than 2^kRescaleLog2: fp32 sums and bf16 P
// keep their relative precision at any power of two.
template <int D, typename Mask>
SCA_INLINE void softmax_tile(uint32_t tS, uint32_t tO, bool has_o, float sl2, float& m, float& l, const Mask& mask) {
  float2 l0 = make_float2(0.f, 0.f), l1 = make_float2(0.f, 0.f);
#pragma unroll 1
  for (int h = 0; h < 4; ++h) {
    uint32_t y[32], pk[16];
    tmem_ld32(tS + 32 * h, y);
    tmem_wait_ld32(y);
    mask(y, h);
    float m0 = __uint_as_float(y[0]), m1 = __uint_as_float(y[1]), m2 = __uint_as_float(y[2]), m3 = __uint_as_float(y[3]);
#pragma unroll
    for (int c = 4; c < 32; c += 4) {
      m0 = fmaxf(m0, __uint_as_float(y[c]));
      m1 = fmaxf(m1, __uint_as_float(y[c + 1]));
      m2 = fmaxf(m2, __uint_as_float(y[c + 2]));
      m3 = fmaxf(m3, __uint_as_float(y[c + 3]));
    }
    const float top = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * sl2;
    const bool need = top > m + kRescaleLog2;
    if (__any_sync(0xffffffffu, need)) {
      // (a key that outweighs all others by that much gets P = 1, unrounded)
      const float m_new = need ? top : m;
      const float alpha = need ? ex2(m - m_new) : 1.f;   // m = -inf gives 0
      m = m_new;
      l *= alpha;
      const float2 al = make_float2(alpha, alpha), zero = make_float2(0.f, 0.f);
      l0 = ffma2(l0, al, zero);
      l1 = ffma2(l1, al, zero);
      // what is read back below may have been stored by this loop:
      // P, and O at a growth in the 32 columns before
      tmem_wait_st();
      if (has_o) {
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
    const float msub = m == -INFINITY ? 0.f : m;
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

}  // namespace sca
