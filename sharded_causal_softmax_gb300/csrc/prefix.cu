// Attention of a decode step for a batch that shares a long prefix: C-ABI
// entry points, the partials in fp32 arithmetic (fp32 inputs, and the
// cross-check of the tensor-core kernel in prefix_tc.cu) and the merge.
//
//   partial over a piece of keys J:  lse_J = ln sum_j exp(s_j),  o_J = sum_j exp(s_j - lse_J) v_j
//   o = sum_J w_J o_J / sum_J w_J,  w_J = exp(lse_J - max lse),  lse = max + ln sum_J w_J
//
// The prefix's keys are walked once for the rows of all requests, a
// request's suffix keys for its own rows.
#include <cmath>

#include "common.cuh"
#include "host_common.h"
#include "launch_util.h"
#include "prefix.h"

namespace sca {
namespace prefix {

constexpr int kThreads = 128;
constexpr int kRows = 32;    // rows of a CTA, four threads each
constexpr int kKeys = 32;    // keys of a shared-memory tile

SCA_INLINE float4 get4(const float* p) { return *reinterpret_cast<const float4*>(p); }
SCA_INLINE float4 get4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}

// The shared-memory reads that feed the FMAs bound it, one 16-byte vector for
// four: 64 requests behind 131072 keys (32 heads on 8, bf16) take 9640 us, 14
// TFLOP/s of about 76 (the tensor cores 165 us); fp32, 16 requests behind 8192
// keys, suffixes of 512, 32 heads on 8: 290 us, 7.9 TFLOP/s; 4 requests behind
// 500 keys, 8 heads of 64: 32 us, 26 captured.
// One CTA: a piece of the prefix (kSuffix = false: grid y is the key/value
// head, rows run over all requests) or of one request's suffix (grid y is
// request x key/value head), for kRows query rows.  Blocks of rows go with the
// pieces, which come first, on grid x: up to 262140 of the prefix's, more than
// another axis holds.  Thread ql of a row's four holds the float4 columns ql,
// ql + 4, ...
template <int D, typename T, bool kSuffix>
__global__ void __launch_bounds__(kThreads) simt_partials(const __grid_constant__ PrefixArgs a) {
  constexpr int NF = D / 16;
  __shared__ float4 Ks[kKeys][D / 4];
  __shared__ float4 Vs[kKeys][D / 4];
  const int hk = kSuffix ? blockIdx.y % a.Hkv : blockIdx.y;
  const int pieces = kSuffix ? a.n_suffix : a.n_prefix, piece = blockIdx.x % pieces;
  const int rows = kSuffix ? a.R : a.B * a.R;
  const int ql = threadIdx.x & 3, row = blockIdx.x / pieces * kRows + (threadIdx.x >> 2);
  const bool valid = row < rows;
  const int b = kSuffix ? blockIdx.y / a.Hkv : (valid ? row / a.R : 0), r = kSuffix ? row : row % a.R;
  const int64_t len = kSuffix ? suffix_len(a, b) : a.prefix_len;
  const int64_t k0 = piece * a.piece, k1 = min64(len, k0 + a.piece);
  if (k0 >= k1) return;
  const int64_t seen = kSuffix ? len - (a.T - 1 - r % a.T) : len;   // this row's keys are [0, seen)
  const View& kv = kSuffix ? a.sv : a.pv;
  const T* kb = static_cast<const T*>(kSuffix ? a.ks : a.kp) + (kSuffix ? b * kv.b : 0) + hk * kv.h;
  const T* vb = static_cast<const T*>(kSuffix ? a.vs : a.vp) + (kSuffix ? b * kv.b : 0) + hk * kv.h;
  const T* qp = static_cast<const T*>(a.q) + (valid ? b * a.q_b + (static_cast<int64_t>(hk) * a.R + r) * D : 0);
  float4 qv[NF], acc[NF];
#pragma unroll
  for (int t = 0; t < NF; ++t) {
    qv[t] = get4(qp + 4 * (ql + 4 * t));
    acc[t] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float m = -INFINITY, l = 0.f;
  for (int64_t t0 = k0; t0 < k1; t0 += kKeys) {
    const int nk = static_cast<int>(min64(kKeys, k1 - t0));
    __syncthreads();
    for (int e = threadIdx.x; e < kKeys * (D / 4); e += kThreads) {
      const int j = e / (D / 4), f = e % (D / 4);
      const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
      Ks[j][f] = j < nk ? get4(kb + (t0 + j) * kv.s + 4 * f) : zero;
      Vs[j][f] = j < nk ? get4(vb + (t0 + j) * kv.s + 4 * f) : zero;
    }
    __syncthreads();
#pragma unroll 1
    for (int j0 = 0; j0 < kKeys; j0 += 8) {
      float s[8], mx = -INFINITY;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        float d = 0.f;
#pragma unroll
        for (int t = 0; t < NF; ++t) {
          const float4 k = Ks[j0 + u][ql + 4 * t];
          d = fmaf(qv[t].x, k.x, fmaf(qv[t].y, k.y, fmaf(qv[t].z, k.z, fmaf(qv[t].w, k.w, d))));
        }
        d += __shfl_xor_sync(0xffffffffu, d, 1);
        d += __shfl_xor_sync(0xffffffffu, d, 2);
        s[u] = t0 + j0 + u < k1 && t0 + j0 + u < seen ? d * a.scale_log2 : -INFINITY;
        mx = fmaxf(mx, s[u]);
      }
      const float m_new = fmaxf(m, mx), sub = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = exp2f(m - sub);
      m = m_new;
      l *= alpha;
#pragma unroll
      for (int t = 0; t < NF; ++t) {
        acc[t].x *= alpha;
        acc[t].y *= alpha;
        acc[t].z *= alpha;
        acc[t].w *= alpha;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float p = exp2f(s[u] - sub);
        l += p;
#pragma unroll
        for (int t = 0; t < NF; ++t) {
          const float4 v = Vs[j0 + u][ql + 4 * t];
          acc[t].x = fmaf(p, v.x, acc[t].x);
          acc[t].y = fmaf(p, v.y, acc[t].y);
          acc[t].z = fmaf(p, v.z, acc[t].z);
          acc[t].w = fmaf(p, v.w, acc[t].w);
        }
      }
    }
  }
  if (!valid) return;
  const int64_t at = ((static_cast<int64_t>(b) * a.Hkv + hk) * a.R + r) * a.slots + (kSuffix ? a.n_prefix : 0) + piece;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  float* po = a.part_o + at * D;
#pragma unroll
  for (int t = 0; t < NF; ++t)
    *reinterpret_cast<float4*>(po + 4 * (ql + 4 * t)) =
        make_float4(acc[t].x * inv, acc[t].y * inv, acc[t].z * inv, acc[t].w * inv);
  if (ql == 0) a.part_lse[at] = l == 0.f ? -INFINITY : m + log2f(l);
}

SCA_INLINE void put4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
SCA_INLINE void put4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  uint2 u;
  u.x = *reinterpret_cast<const uint32_t*>(&a);
  u.y = *reinterpret_cast<const uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = u;
}

// One CTA of four groups of D/4 threads per query row: the groups take the
// row's partials in turn, their sums meet in shared memory in a fixed order.
template <int D, typename T>
__global__ void __launch_bounds__(D) merge_kernel(const __grid_constant__ PrefixArgs a) {
  constexpr int W = D / 4;
  __shared__ float4 so[4][W];
  __shared__ float sw[4];
  const int64_t row = blockIdx.x;
  const int b = static_cast<int>(row / (static_cast<int64_t>(a.Hkv) * a.R));
  const int64_t len = suffix_len(a, b);
  const int n = a.n_prefix + static_cast<int>((len + a.piece - 1) / a.piece);
  const float* lp = a.part_lse + row * a.slots;
  const float4* op = reinterpret_cast<const float4*>(a.part_o + row * a.slots * D);
  const int g = threadIdx.x / W, c = threadIdx.x % W;
  float m = -INFINITY;
  for (int i = 0; i < n; ++i) m = fmaxf(m, lp[i]);
  const float mm = m == -INFINITY ? 0.f : m;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float w = 0.f;
#pragma unroll 4
  for (int i = g; i < n; i += 4) {
    const float wi = exp2f(lp[i] - mm);
    const float4 v = op[static_cast<int64_t>(i) * W + c];
    w += wi;
    acc.x = fmaf(wi, v.x, acc.x);
    acc.y = fmaf(wi, v.y, acc.y);
    acc.z = fmaf(wi, v.z, acc.z);
    acc.w = fmaf(wi, v.w, acc.w);
  }
  so[g][c] = acc;
  if (c == 0) sw[g] = w;
  __syncthreads();
  if (g != 0) return;
  const float total = (sw[0] + sw[1]) + (sw[2] + sw[3]);
  const float inv = total == 0.f ? 0.f : 1.f / total;
  const float4 p = so[0][c], q = so[1][c], r = so[2][c], s = so[3][c];
  put4(static_cast<T*>(a.o) + row * D + 4 * c,
       make_float4(((p.x + q.x) + (r.x + s.x)) * inv, ((p.y + q.y) + (r.y + s.y)) * inv,
                   ((p.z + q.z) + (r.z + s.z)) * inv, ((p.w + q.w) + (r.w + s.w)) * inv));
  if (c == 0) a.lse[row] = total == 0.f ? -INFINITY : (mm + log2f(total)) * kLn2;
}

template <int D, typename T>
static cudaError_t simt(const PrefixArgs& a, cudaStream_t st) {
  if (a.n_prefix) {
    simt_partials<D, T, false><<<dim3((a.B * a.R + kRows - 1) / kRows * a.n_prefix, a.Hkv), kThreads, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (a.n_suffix)
    simt_partials<D, T, true><<<dim3((a.R + kRows - 1) / kRows * a.n_suffix, a.B * a.Hkv), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

// Keys go in tiles of 128.  A work item is one piece of keys for one tile of
// rows; a piece is as many tiles as give each SM two items or more, at most
// one piece per prefix or suffix.
struct Pieces {
  int64_t tiles;       // per piece
  int64_t n_prefix, n_suffix;
};
static int64_t units_prefix(const sca_prefix_dims* d) {
  const int R = d->H / d->Hkv * d->T, nb = 128 / R;
  return static_cast<int64_t>(d->Hkv) * ((d->B + nb - 1) / nb);
}
static Pieces pieces(const sca_prefix_dims* d) {
  const int64_t tp = (d->prefix_len + 127) / 128, ts = (d->suffix_cap + 127) / 128;
  const int64_t steps = units_prefix(d) * tp + static_cast<int64_t>(d->B) * d->Hkv * ts;
  Pieces p;
  const int64_t slots = 2 * static_cast<int64_t>(sm_count());
  p.tiles = (steps + slots - 1) / slots;
  if (p.tiles < 1) p.tiles = 1;
  p.n_prefix = (tp + p.tiles - 1) / p.tiles;
  p.n_suffix = (ts + p.tiles - 1) / p.tiles;
  return p;
}
// the most partials of a row at these sizes or smaller keys: pieces() gives
// at most 2 SMs' worth of items over all units, plus a rounding each
static int64_t most_slots(const sca_prefix_dims* d) {
  const int64_t tp = (d->prefix_len + 127) / 128, ts = (d->suffix_cap + 127) / 128;
  const int64_t items = 2 * static_cast<int64_t>(sm_count());
  const int64_t a = min64(tp, items / units_prefix(d) + 1);
  const int64_t b = min64(ts, items / (static_cast<int64_t>(d->B) * d->Hkv) + 1);
  return a + b;
}

static bool use_tc(const sca_prefix_dims* d) { return d->dtype == SCA_BF16 && d->algo != SCA_ALGO_SIMT; }

static int check_view(const sca_view& v, int mult, int D, const char* what) {
  SCA_REQUIRE(v.b >= 0 && v.h >= 0 && v.s >= D, SCA_ERR_ARG,
              "prefix_attn: %s strides must be >= 0 and the row stride >= D", what);
  SCA_REQUIRE(v.b % mult == 0 && v.h % mult == 0 && v.s % mult == 0, SCA_ERR_ALIGN,
              "prefix_attn: %s strides must be multiples of %d elements", what, mult);
  return SCA_OK;
}

static int check_dims(const sca_prefix_dims* d) {
  SCA_REQUIRE(d != nullptr, SCA_ERR_ARG, "prefix_attn: dims is NULL");
  SCA_REQUIRE(d->B >= 1 && d->H >= 1 && d->Hkv >= 1 && d->T >= 1 && d->H % d->Hkv == 0 &&
                  static_cast<int64_t>(d->B) * d->H <= 65535,
              SCA_ERR_ARG, "prefix_attn: B=%d, H=%d, Hkv=%d, T=%d: need positive sizes, Hkv dividing H, B*H <= 65535",
              d->B, d->H, d->Hkv, d->T);
  SCA_REQUIRE(static_cast<int64_t>(d->H / d->Hkv) * d->T <= 128, SCA_ERR_UNSUPPORTED,
              "prefix_attn: %d heads a key/value head x %d tokens: at most 128 query rows", d->H / d->Hkv, d->T);
  SCA_REQUIRE(d->D == 64 || d->D == 128, SCA_ERR_UNSUPPORTED, "prefix_attn: D=%d: only 64 and 128", d->D);
  SCA_REQUIRE(d->dtype == SCA_BF16 || d->dtype == SCA_F32, SCA_ERR_ARG, "prefix_attn: dtype=%d unknown", d->dtype);
  SCA_REQUIRE(d->algo >= SCA_ALGO_AUTO && d->algo <= SCA_ALGO_TC, SCA_ERR_ARG, "prefix_attn: algo=%d unknown", d->algo);
  SCA_REQUIRE(d->dtype == SCA_BF16 || d->algo != SCA_ALGO_TC, SCA_ERR_UNSUPPORTED,
              "prefix_attn: the tensor-core kernel takes bf16 inputs only");
  SCA_REQUIRE(std::isfinite(d->scale) && d->scale > 0.f, SCA_ERR_ARG, "prefix_attn: scale must be finite and positive");
  SCA_REQUIRE(d->prefix_len >= 0 && d->prefix_len < (1LL << 31) - 128 && d->suffix_cap >= 0 &&
                  d->suffix_cap < (1LL << 31) - 128,
              SCA_ERR_ARG, "prefix_attn: prefix_len or suffix_cap out of range");
  const int mult = d->dtype == SCA_BF16 ? 8 : 4;
  SCA_REQUIRE(d->q_b >= 0 && (d->B == 1 || d->q_b >= static_cast<int64_t>(d->H) * d->T * d->D), SCA_ERR_ARG,
              "prefix_attn: q batch stride below H*T*D");
  SCA_REQUIRE(d->q_b % mult == 0, SCA_ERR_ALIGN, "prefix_attn: q batch stride must be a multiple of %d elements", mult);
  int rc;
  if (d->prefix_len && (rc = check_view(d->prefix, mult, d->D, "prefix")) != SCA_OK) return rc;
  if (d->suffix_cap && (rc = check_view(d->suffix, mult, d->D, "suffix")) != SCA_OK) return rc;
  return SCA_OK;
}

}  // namespace prefix
}  // namespace sca

using namespace sca;
using namespace sca::prefix;

extern "C" int prefix_attn_workspace(const sca_prefix_dims* d, int64_t* bytes) {
  int rc;
  if ((rc = check_dims(d)) != SCA_OK) return rc;
  SCA_REQUIRE(bytes != nullptr, SCA_ERR_ARG, "prefix_attn_workspace: bytes is NULL");
  *bytes = use_tc(d) ? prefix_tc_workspace(d->B, d->Hkv, d->H / d->Hkv * d->T, d->D, d->prefix_len, d->suffix_cap,
                                           sm_count())
                     : static_cast<int64_t>(d->B) * d->H * d->T * most_slots(d) * (d->D + 1) * 4;
  return SCA_OK;
}

extern "C" int prefix_attn_decode(const sca_prefix_dims* d, const void* q, const void* k_prefix,
                                  const void* v_prefix, const void* k_suffix, const void* v_suffix,
                                  const int32_t* lengths, void* o, float* lse, float* ws, int64_t ws_bytes,
                                  int* dev_status, void* stream) {
  int rc;
  if ((rc = check_dims(d)) != SCA_OK) return rc;
  SCA_REQUIRE(q && o && lse, SCA_ERR_ARG, "prefix_attn_decode: NULL pointer");
  SCA_REQUIRE(d->prefix_len == 0 || (k_prefix && v_prefix), SCA_ERR_ARG, "prefix_attn_decode: NULL prefix");
  SCA_REQUIRE(d->suffix_cap == 0 || (k_suffix && v_suffix && lengths), SCA_ERR_ARG,
              "prefix_attn_decode: NULL suffix or lengths");
  SCA_REQUIRE(aligned(q, 16) && aligned(k_prefix, 16) && aligned(v_prefix, 16) && aligned(k_suffix, 16) &&
                  aligned(v_suffix, 16) && aligned(o, 16) && aligned(lse, 4) && aligned(ws, 16) &&
                  aligned(lengths, 4),
              SCA_ERR_ALIGN, "prefix_attn_decode: tensors must be 16-byte aligned, lse and lengths 4-byte");
  const bool tc = use_tc(d);
  const int sms = sm_count();
  const Pieces p = pieces(d);
  const int64_t rows = static_cast<int64_t>(d->B) * d->H * d->T, slots = p.n_prefix + p.n_suffix;
  const int64_t need = tc ? prefix_tc_workspace(d->B, d->Hkv, d->H / d->Hkv * d->T, d->D, d->prefix_len,
                                                d->suffix_cap, sms)
                          : rows * slots * (d->D + 1) * 4;
  SCA_REQUIRE(need == 0 || (ws && ws_bytes >= need), SCA_ERR_ARG,
              "prefix_attn_decode: workspace of %lld bytes, %lld needed", static_cast<long long>(ws ? ws_bytes : 0),
              static_cast<long long>(need));
  PrefixArgs a = {};
  a.q = q;
  a.kp = k_prefix;
  a.vp = v_prefix;
  a.ks = k_suffix;
  a.vs = v_suffix;
  a.lengths = lengths;
  a.o = o;
  a.lse = lse;
  a.part_o = ws;
  a.part_lse = ws + rows * slots * d->D;
  a.q_b = d->q_b;
  a.pv = {0, d->prefix.h, d->prefix.s};
  a.sv = {d->suffix.b, d->suffix.h, d->suffix.s};
  a.prefix_len = d->prefix_len;
  a.suffix_cap = d->suffix_cap;
  a.piece = p.tiles * 128;
  a.B = d->B;
  a.Hkv = d->Hkv;
  a.R = d->H / d->Hkv * d->T;
  a.T = d->T;
  a.n_prefix = static_cast<int>(p.n_prefix);
  a.n_suffix = static_cast<int>(p.n_suffix);
  a.slots = static_cast<int>(slots);
  a.scale_log2 = d->scale * kLog2e;
  a.status = dev_status;
  cudaStream_t st = as_stream(stream);
  if (tc) return prefix_tc_decode(a, d->D, sms, ws, st);
  const bool bf16 = d->dtype == SCA_BF16;
  if (slots) {
    cudaError_t e;
    if (d->D == 64) e = bf16 ? simt<64, __nv_bfloat16>(a, st) : simt<64, float>(a, st);
    else e = bf16 ? simt<128, __nv_bfloat16>(a, st) : simt<128, float>(a, st);
    if (e != cudaSuccess) return cuda_status(e, "prefix_attn_decode");
  }
  const unsigned grid = static_cast<unsigned>(rows);
  if (d->D == 64 && bf16) merge_kernel<64, __nv_bfloat16><<<grid, 64, 0, st>>>(a);
  else if (d->D == 64) merge_kernel<64, float><<<grid, 64, 0, st>>>(a);
  else if (bf16) merge_kernel<128, __nv_bfloat16><<<grid, 128, 0, st>>>(a);
  else merge_kernel<128, float><<<grid, 128, 0, st>>>(a);
  return cuda_status(cudaGetLastError(), "prefix_attn_decode");
}
