// Rotary positions: pairs of features turned by position times frequency, of
// whole tensors (rotary_apply) or on the way into a paged cache
// (paged_kv_append in paged.cu).
//
//   y_a = m (x_a cos t - x_b sin t),  y_b = m (x_a sin t + x_b cos t),  t = p f_i
//
// Angles.  f_i comes as a 64-bit fraction of a turn, so that p f_i mod 2^64 is
// one integer product and exact at any position; the nearest quarter is taken
// off as an integer too, and what is left, at most an eighth of a turn, goes to
// sincospif rounded to fp32 (within 1.5 2^-24 of it, however small).  No table of
// cosines: at 32K rows of 128 features it would be 16 MB to read beside the rows.
//
// Every row is read and written once, 3 FMAs a feature: HBM bounds it.  A
// thread owns two vectors of 16 bytes of a row, half the turned features apart
// (or half the others), and walks the heads with them, so the angles of a row
// are computed once for `chunk` heads.
//
// A small call (captured: 512 drafted rows of 48 heads 4.6 us, its bytes 1.9) is a chain:
// lengths, page number, angles, and only then the rows' loads.  Only the stores need
// the pages and only the arithmetic the angles; the loads stand behind them because
// the code was written so, and that is not measured the other way round.
#include <cmath>
#include <utility>

#include "disjoint.h"
#include "host_common.h"
#include "launch_util.h"
#include "overlap.cuh"
#include "rotary.h"

namespace sca {
namespace rotary {

constexpr int kThreads = 128;
constexpr int kHeads = 4;   // heads whose loads are in flight together

// V elements of T, moved at once (16 bytes, or one element)
template <typename T, int V>
struct Vec;
template <>
struct Vec<__nv_bfloat16, 8> {
  using raw = uint4;
  static SCA_INLINE void unpack(const uint4& r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static SCA_INLINE uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<float, 4> {
  using raw = float4;
  static SCA_INLINE void unpack(const float4& r, float (&x)[4]) {
    x[0] = r.x;
    x[1] = r.y;
    x[2] = r.z;
    x[3] = r.w;
  }
  static SCA_INLINE float4 pack(const float (&x)[4]) { return make_float4(x[0], x[1], x[2], x[3]); }
};
template <>
struct Vec<__nv_bfloat16, 1> {
  using raw = __nv_bfloat16;
  static SCA_INLINE void unpack(raw r, float (&x)[1]) { x[0] = __bfloat162float(r); }
  static SCA_INLINE raw pack(const float (&x)[1]) { return __float2bfloat16_rn(x[0]); }
};
template <>
struct Vec<float, 1> {
  using raw = float;
  static SCA_INLINE void unpack(raw r, float (&x)[1]) { x[0] = r; }
  static SCA_INLINE raw pack(const float (&x)[1]) { return x[0]; }
};

// cos and sin of p times f 2^-64 turns
SCA_INLINE void turn(uint64_t f, int64_t p, float& c, float& s) {
  const uint64_t t = f * static_cast<uint64_t>(p);
  const uint32_t quarter = static_cast<uint32_t>((t + (1ull << 61)) >> 62);
  // what is left, in two signed words: its upper 32 bits alone would lose up to 2^-32 turns, 1e-3 of a
  // slow pair's sine.  (A conversion of 64 bits took 0.2 to 0.5 us of a short call.)
  const int32_t lo = static_cast<int32_t>(static_cast<uint32_t>(t));
  const int32_t hi = static_cast<int32_t>(static_cast<uint32_t>(t >> 32) - (quarter << 30)) + (lo < 0);
  float cr, sr;
  sincospif(fmaf(static_cast<float>(lo), 0x1p-63f, static_cast<float>(hi) * 0x1p-31f), &sr, &cr);
  const float a = quarter & 1 ? sr : cr, b = quarter & 1 ? cr : sr;
  c = quarter == 1 || quarter == 2 ? -a : a;
  s = quarter >= 2 ? -b : b;
}

template <typename T, int V, bool kPaged>
__global__ void __launch_bounds__(kThreads) rows_kernel(const __grid_constant__ RowsArgs a) {
  using X = Vec<T, V>;
  using raw = typename X::raw;
  wait_for_previous();
  const int units = a.D / (2 * V);
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t row = at / units;
  const int u = static_cast<int>(at - row * units);
  if (row >= a.B * a.S) return;
  const int64_t b = row / a.S, s = row - b * a.S;
  int64_t slot = s, to = 0;
  bool live = true, placed = true;
  if (kPaged) {
    const int len = a.lengths[b];
    slot += len > 0 ? len : 0;
    live = a.counts == nullptr || s < a.counts[b];
    const int64_t entry = slot >> a.page_log2;
    int64_t page = -1;
    if (live && entry < a.table_n) page = a.table[b * a.table_b + entry];
    placed = page >= 0 && page < a.pages;
    if (live && !placed) report(a.status, SCA_ERR_RANGE);
    to = page * a.ov[1].b + (slot & ((1ll << a.page_log2) - 1)) * a.ov[1].s;
  }
  // the two vectors of this thread, and the pairs in them
  const int turned = a.rd / (2 * V);
  const bool turns = u < turned;
  const bool next_to = V == 1 && turns && a.interleaved;   // single elements are one pair
  const int e0 = next_to ? 2 * u : (turns ? u * V : a.rd + (u - turned) * V);
  const int e1 = next_to ? e0 + 1 : e0 + (turns ? a.rd : a.D - a.rd) / 2;
  float c[V], sn[V];
  if (turns) {
    const int64_t p = a.positions ? a.positions[b * a.pos_b + s] : slot;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      // interleaved vectors hold whole pairs: half of these in either
      const int i = V == 1 || !a.interleaved ? u * V + e : u * (V / 2) + (e < V / 2 ? e : a.rd / 4 + e - V / 2);
      turn(a.turns[i], p, c[e], sn[e]);
      c[e] *= a.amplitude;
      sn[e] *= a.amplitude * a.sign;
    }
  }
  const int h0 = blockIdx.y * a.chunk, n0 = a.heads[0], n1 = n0 + a.heads[1], n2 = n1 + a.heads[2];
  const int h1 = min(h0 + a.chunk, n2);
  // kHeads at a time: their loads go out together, before the first store
  // (which, for all the compiler knows, might write what the next one reads)
#pragma unroll 1
  for (int h = h0; h < h1; h += kHeads) {
    raw r0[kHeads], r1[kHeads];
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      if (h + j >= h1 || !live) continue;
      const int i = h + j < n0 ? 0 : (h + j < n1 ? 1 : 2), hh = h + j - (i == 0 ? 0 : (i == 1 ? n0 : n1));
      const T* in = static_cast<const T*>(a.in[i]) + b * a.iv[i].b + hh * a.iv[i].h + s * a.iv[i].s;
      r0[j] = *reinterpret_cast<const raw*>(in + e0);
      r1[j] = *reinterpret_cast<const raw*>(in + e1);
    }
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      if (h + j >= h1) continue;
      const int i = h + j < n0 ? 0 : (h + j < n1 ? 1 : 2), hh = h + j - (i == 0 ? 0 : (i == 1 ? n0 : n1));
      const bool to_page = kPaged && i > 0;
      if (to_page && !placed) continue;
      if (!live) {
        float zero[V] = {};
        r0[j] = r1[j] = X::pack(zero);
      } else if (turns && i < 2) {
        float x0[V], x1[V];
        X::unpack(r0[j], x0);
        X::unpack(r1[j], x1);
        if (V == 1 || !a.interleaved) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float x = x0[e], y = x1[e];
            x0[e] = fmaf(x, c[e], -y * sn[e]);
            x1[e] = fmaf(x, sn[e], y * c[e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            const float x = x0[2 * e], y = x0[2 * e + 1], z = x1[2 * e], w = x1[2 * e + 1];
            x0[2 * e] = fmaf(x, c[e], -y * sn[e]);
            x0[2 * e + 1] = fmaf(x, sn[e], y * c[e]);
            x1[2 * e] = fmaf(z, c[V / 2 + e], -w * sn[V / 2 + e]);
            x1[2 * e + 1] = fmaf(z, sn[V / 2 + e], w * c[V / 2 + e]);
          }
        }
        r0[j] = X::pack(x0);
        r1[j] = X::pack(x1);
      }
      T* out = static_cast<T*>(a.out[i]) + hh * a.ov[i].h + (to_page ? to : b * a.ov[i].b + s * a.ov[i].s);
      *reinterpret_cast<raw*>(out + e0) = r0[j];
      *reinterpret_cast<raw*>(out + e1) = r1[j];
    }
  }
}

template <typename T, int V>
static cudaError_t launch(RowsArgs& a, cudaStream_t st) {
  const int64_t blocks = (a.B * a.S * (a.D / (2 * V)) + kThreads - 1) / kThreads;
  const int heads = a.heads[0] + a.heads[1] + a.heads[2];
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  // As many heads a CTA as leave every SM two CTAs, 8 at most.  Eight CTAs an SM
  // compute their angles for too few heads (captured: 512 drafted rows of 48 heads 7.6 us
  // instead of 4.6, 3 x 1001 rows, 12 + 4 heads of 64, fp32, there and back 12.0 instead of
  // 11.3; a caller who does not capture waits for the host either way), 16 heads leave
  // too few rows in flight (32K rows of 32 heads 164 instead of 161 us), 4 compute
  // angles too often (171).
  const int64_t most = blocks * heads / (2 * sm_count());
  a.chunk = 8;
  while (a.chunk > 1 && a.chunk > most) a.chunk /= 2;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((heads + a.chunk - 1) / a.chunk));
  return a.table ? launch_early(rows_kernel<T, V, true>, grid, kThreads, 0, st, a)
                 : launch_early(rows_kernel<T, V, false>, grid, kThreads, 0, st, a);
}

// whether every address and stride allows vectors of 16 bytes
static bool wide(const RowsArgs& a, int eb) {
  const int V = 16 / eb;
  if (a.D % (2 * V) || a.rd % (2 * V)) return false;
  for (int i = 0; i < 3; ++i) {
    if (!a.heads[i]) continue;
    const View& x = a.iv[i];
    const View& y = a.ov[i];
    if (!aligned(a.in[i], 16) || !aligned(a.out[i], 16) || x.b % V || x.h % V || x.s % V || y.b % V || y.h % V || y.s % V)
      return false;
  }
  return true;
}

}  // namespace rotary

cudaError_t launch_rows(RowsArgs a, int dtype, cudaStream_t st) {
  using namespace rotary;
  if (dtype == SCA_BF16)
    return wide(a, 2) ? launch<__nv_bfloat16, 8>(a, st) : launch<__nv_bfloat16, 1>(a, st);
  return wide(a, 4) ? launch<float, 4>(a, st) : launch<float, 1>(a, st);
}

namespace rotary {

constexpr int64_t kMostStride = 1LL << 40;

// whether a view's rows lie apart: each axis steps over all of those of
// smaller strides
static bool apart(const sca_view& v, int64_t B, int64_t H, int64_t S, int64_t D) {
  int64_t st[3] = {v.b, v.h, v.s}, n[3] = {B, H, S}, e = D;
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      if (st[j] > st[j + 1]) {
        std::swap(st[j], st[j + 1]);
        std::swap(n[j], n[j + 1]);
      }
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) continue;
    if (st[i] < e) return false;
    e += (n[i] - 1) * st[i];
  }
  return true;
}

static int check(const char* what, const sca_view& in, const sca_view& out, const void* x, const void* y, int64_t B,
                 int64_t H, int64_t S, int64_t D, int eb) {
  SCA_REQUIRE(x && y, SCA_ERR_ARG, "rotary_apply: NULL %s", what);
  for (const int64_t x : {in.b, in.h, in.s, out.b, out.h, out.s})
    SCA_REQUIRE(x >= 0 && x < kMostStride, SCA_ERR_ARG, "rotary_apply: strides of %s negative or above 2^40", what);
  SCA_REQUIRE(aligned(x, eb) && aligned(y, eb), SCA_ERR_ALIGN, "rotary_apply: %s off its element size", what);
  SCA_REQUIRE(apart(out, B, H, S, D), SCA_ERR_ARG, "rotary_apply: rows of the output of %s overlap", what);
  const bool same = x == y && (B == 1 || in.b == out.b) && (H == 1 || in.h == out.h) && (S == 1 || in.s == out.s);
  SCA_REQUIRE(same || !share_bytes(row_set(x, in, B, H, S, D, eb), row_set(y, out, B, H, S, D, eb)), SCA_ERR_ARG,
              "rotary_apply: %s and its output overlap without being the same", what);
  return SCA_OK;
}

}  // namespace rotary
}  // namespace sca

using namespace sca;

extern "C" int rotary_apply(const sca_rotary_dims* d, const void* q, const void* k, const uint64_t* turns,
                            const int32_t* positions, void* qo, void* ko, void* stream) {
  SCA_REQUIRE(d != nullptr, SCA_ERR_ARG, "rotary_apply: dims is NULL");
  SCA_REQUIRE(d->B >= 1 && d->H >= 1 && d->Hkv >= 0 && static_cast<int64_t>(d->H) + d->Hkv <= 65535, SCA_ERR_ARG,
              "rotary_apply: B=%d, H=%d, Hkv=%d", d->B, d->H, d->Hkv);
  SCA_REQUIRE(d->S >= 1 && d->S < 1LL << 31 && d->B * d->S < 1LL << 36, SCA_ERR_ARG, "rotary_apply: B=%d, S=%lld",
              d->B, static_cast<long long>(d->S));
  SCA_REQUIRE(d->D >= 2 && d->D <= 1024 && d->D % 2 == 0, SCA_ERR_ARG, "rotary_apply: D=%d: even, up to 1024", d->D);
  SCA_REQUIRE(d->rotary_dim >= 0 && d->rotary_dim <= d->D && d->rotary_dim % 2 == 0, SCA_ERR_ARG,
              "rotary_apply: rotary_dim=%d of D=%d", d->rotary_dim, d->D);
  SCA_REQUIRE(d->dtype == SCA_BF16 || d->dtype == SCA_F32, SCA_ERR_ARG, "rotary_apply: dtype=%d unknown", d->dtype);
  SCA_REQUIRE(std::isfinite(d->amplitude), SCA_ERR_ARG, "rotary_apply: amplitude is not finite");
  SCA_REQUIRE(d->rotary_dim == 0 || turns, SCA_ERR_ARG, "rotary_apply: NULL turns");
  SCA_REQUIRE(aligned(turns, 8) && aligned(positions, 4), SCA_ERR_ALIGN, "rotary_apply: turns or positions misaligned");
  SCA_REQUIRE(d->pos_b >= 0, SCA_ERR_ARG, "rotary_apply: negative stride of positions");
  const int eb = d->dtype == SCA_BF16 ? 2 : 4;
  int rc = rotary::check("q", d->q, d->qo, q, qo, d->B, d->H, d->S, d->D, eb);
  if (rc == SCA_OK && d->Hkv) rc = rotary::check("k", d->k, d->ko, k, ko, d->B, d->Hkv, d->S, d->D, eb);
  if (rc != SCA_OK) return rc;
  if (d->Hkv) {   // (heads of both are turned at once, in no order)
    const Rows r[4] = {row_set(q, d->q, d->B, d->H, d->S, d->D, eb), row_set(qo, d->qo, d->B, d->H, d->S, d->D, eb),
                       row_set(k, d->k, d->B, d->Hkv, d->S, d->D, eb), row_set(ko, d->ko, d->B, d->Hkv, d->S, d->D, eb)};
    SCA_REQUIRE(!share_bytes(r[1], r[2]) && !share_bytes(r[3], r[0]) && !share_bytes(r[1], r[3]), SCA_ERR_ARG,
                "rotary_apply: an output overlaps the other input or output");
  }
  RowsArgs a = {};
  a.in[0] = q;
  a.in[1] = k;
  a.out[0] = qo;
  a.out[1] = ko;
  a.iv[0] = {d->q.b, d->q.h, d->q.s};
  a.iv[1] = {d->k.b, d->k.h, d->k.s};
  a.ov[0] = {d->qo.b, d->qo.h, d->qo.s};
  a.ov[1] = {d->ko.b, d->ko.h, d->ko.s};
  a.heads[0] = d->H;
  a.heads[1] = d->Hkv;
  a.B = d->B;
  a.S = d->S;
  a.D = d->D;
  a.rd = d->rotary_dim;
  a.interleaved = d->interleaved != 0;
  a.amplitude = d->amplitude;
  a.sign = d->transposed ? -1.f : 1.f;
  a.turns = turns;
  a.positions = positions;
  a.pos_b = d->pos_b;
  return cuda_status(launch_rows(a, d->dtype, as_stream(stream)), "rotary_apply");
}
