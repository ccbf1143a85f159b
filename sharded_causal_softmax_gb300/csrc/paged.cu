// A cache of keys and values in pages: C-ABI entry points (append, attention of
// drafted tokens, acceptance), the acceptance kernel, and the attention in
// fp32 arithmetic (fp32 inputs, and the cross-check of the tensor-core kernel
// in paged_tc.cu).  The rows of an append go through rotary.cu.
//
//   partial over a piece of rows J:  lse_J = ln sum_j exp(s_j),  o_J = sum_j exp(s_j - lse_J) v_j
//   o = sum_J w_J o_J / sum_J w_J,  w_J = exp(lse_J - max lse),  lse = max + ln sum_J w_J
#include <cmath>

#include "host_common.h"
#include "launch_util.h"
#include "overlap.cuh"
#include "paged.h"
#include "rotary.h"

namespace sca {
namespace paged {

constexpr int kThreads = 128;
constexpr int kKeys = 32;    // keys of a shared-memory tile

SCA_INLINE float4 get4(const float* p) { return *reinterpret_cast<const float4*>(p); }
SCA_INLINE float4 get4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}
SCA_INLINE void put4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
SCA_INLINE void put4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  uint2 u;
  u.x = *reinterpret_cast<const uint32_t*>(&a);
  u.y = *reinterpret_cast<const uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = u;
}
SCA_INLINE float4 scaled(float4 v, float w) { return make_float4(v.x * w, v.y * w, v.z * w, v.w * w); }
SCA_INLINE float4 added(float4 v, float w, float4 to) {
  return make_float4(fmaf(w, v.x, to.x), fmaf(w, v.y, to.y), fmaf(w, v.z, to.z), fmaf(w, v.w, to.w));
}

struct SimtArgs {
  PagedArgs a;
  float* part_o;      // [rows of all][pieces][D] normalised partial outputs
  float* part_lse;    // [rows of all][pieces] their lse, base 2
  int32_t pieces, row_tiles;
};

// rows of a piece of a request that holds `rows`: equal parts, in whole tiles
SCA_INLINE int piece_rows(int rows, int pieces) {
  const int tiles = (rows + kKeys - 1) / kKeys;
  return (tiles + pieces - 1) / pieces * kKeys;
}

// One CTA: a piece of one request's rows of one key/value head (grid y) for RP
// query rows.  Four threads hold a row, thread ql of them the float4 columns
// ql, ql + 4, ...; 32 / RP of them share a row, each with keys of its own.
template <int D, typename T, int RP>
__global__ void __launch_bounds__(kThreads) simt_partials(const __grid_constant__ SimtArgs k) {
  constexpr int NF = D / 16, PH = 32 / RP, KG = kKeys / PH < 8 ? kKeys / PH : 8;
  __shared__ float4 Ks[kKeys][D / 4];
  __shared__ float4 Vs[kKeys][D / 4];
  __shared__ float sm[32], sl[32];
  const PagedArgs& a = k.a;
  wait_for_previous();
  const int b = blockIdx.y / a.Hkv, hk = blockIdx.y - b * a.Hkv;
  const int rt = blockIdx.x / k.pieces, piece = blockIdx.x - rt * k.pieces;
  const Held held_rows = held(a, b);
  const int rows = held_rows.cnt ? rows_of(a, held_rows) : 0, per = piece_rows(rows, k.pieces);
  if (threadIdx.x == 0) report_beyond(a, b);
  const int k0 = min(piece * per, rows), k1 = min(k0 + per, rows);
  if (k0 >= k1) return;
  const int ql = threadIdx.x & 3, slot = threadIdx.x >> 2, ph = slot / RP, r = rt * RP + slot % RP;
  const bool valid = r < a.R;
  const Sight sees = valid ? sight(a, b, r % a.T, held_rows, rows) : Sight{0, 0};
  const T* qp = static_cast<const T*>(a.q) + b * a.q_b + (static_cast<int64_t>(hk) * a.R + (valid ? r : 0)) * D;
  float4 qv[NF], acc[NF];
#pragma unroll
  for (int t = 0; t < NF; ++t) {
    qv[t] = get4(qp + 4 * (ql + 4 * t));
    acc[t] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const T *kb = static_cast<const T*>(a.kp) + hk * a.pool.h, *vb = static_cast<const T*>(a.vp) + hk * a.pool.h;
  const int32_t* table = a.table + b * a.table_b;
  float m = -INFINITY, l = 0.f;
  for (int t0 = k0; t0 < k1; t0 += kKeys) {
    const int nk = min(kKeys, k1 - t0);
    __syncthreads();
    for (int e = threadIdx.x; e < kKeys * (D / 4); e += kThreads) {
      const int j = e / (D / 4), f = e % (D / 4), row = t0 + j;
      float4 kx = make_float4(0.f, 0.f, 0.f, 0.f), vx = kx;
      if (j < nk) {
        const int64_t page = table[row >> a.page_log2];
        if (page >= 0 && page < a.pages) {
          const int64_t at = page * a.pool.b + (row & ((1 << a.page_log2) - 1)) * a.pool.s + 4 * f;
          kx = get4(kb + at);
          vx = get4(vb + at);
        } else {
          report(a.status, SCA_ERR_RANGE);
        }
      }
      Ks[j][f] = kx;
      Vs[j][f] = vx;
    }
    __syncthreads();
    const uint32_t bits = t0 + kKeys <= sees.full ? 0xffffffffu : seen_bits(sees, held_rows.len, t0);
#pragma unroll 1
    for (int j0 = 0; j0 < kKeys; j0 += KG * PH) {
      float s[KG], mx = -INFINITY;
#pragma unroll
      for (int u = 0; u < KG; ++u) {
        const int j = j0 + u * PH + ph;
        float d = 0.f;
#pragma unroll
        for (int t = 0; t < NF; ++t) {
          const float4 x = Ks[j][ql + 4 * t];
          d = fmaf(qv[t].x, x.x, fmaf(qv[t].y, x.y, fmaf(qv[t].z, x.z, fmaf(qv[t].w, x.w, d))));
        }
        d += __shfl_xor_sync(0xffffffffu, d, 1);
        d += __shfl_xor_sync(0xffffffffu, d, 2);
        s[u] = (bits >> j) & 1 && j < nk ? d * a.scale_log2 : -INFINITY;
        mx = fmaxf(mx, s[u]);
      }
      const float m_new = fmaxf(m, mx), sub = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = exp2f(m - sub);
      m = m_new;
      l *= alpha;
#pragma unroll
      for (int t = 0; t < NF; ++t) acc[t] = scaled(acc[t], alpha);
#pragma unroll
      for (int u = 0; u < KG; ++u) {
        const float p = exp2f(s[u] - sub);
        l += p;
#pragma unroll
        for (int t = 0; t < NF; ++t) acc[t] = added(Vs[j0 + u * PH + ph][ql + 4 * t], p, acc[t]);
      }
    }
  }
  if (PH > 1) {   // the row's sums over its phases' keys, in shared memory in a fixed order
    float4* so = &Ks[0][0];   // [32][D / 4]
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NF; ++t) so[slot * (D / 4) + ql + 4 * t] = acc[t];
    if (ql == 0) {
      sm[slot] = m;
      sl[slot] = l;
    }
    __syncthreads();
    if (ph != 0) return;
    float top = -INFINITY;
    for (int p = 0; p < PH; ++p) top = fmaxf(top, sm[p * RP + slot]);
    const float sub = top == -INFINITY ? 0.f : top;
    m = top;
    l = 0.f;
#pragma unroll
    for (int t = 0; t < NF; ++t) acc[t] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p = 0; p < PH; ++p) {
      const float w = exp2f(sm[p * RP + slot] - sub);
      l = fmaf(w, sl[p * RP + slot], l);
#pragma unroll
      for (int t = 0; t < NF; ++t) acc[t] = added(so[(p * RP + slot) * (D / 4) + ql + 4 * t], w, acc[t]);
    }
  }
  if (!valid) return;
  const int64_t at = (static_cast<int64_t>(blockIdx.y) * a.R + r) * k.pieces + piece;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  float* po = k.part_o + at * D;
#pragma unroll
  for (int t = 0; t < NF; ++t) put4(po + 4 * (ql + 4 * t), scaled(acc[t], inv));
  if (ql == 0) k.part_lse[at] = l == 0.f ? -INFINITY : m + log2f(l);
}

// One CTA of four groups of D/4 threads per query row: the groups take the
// row's partials in turn, their sums meet in shared memory in a fixed order.
template <int D, typename T>
__global__ void __launch_bounds__(D) merge_kernel(const __grid_constant__ SimtArgs k) {
  constexpr int W = D / 4;
  __shared__ float4 so[4][W];
  __shared__ float sw[4];
  const PagedArgs& a = k.a;
  wait_for_previous();
  const int64_t row = blockIdx.x;
  const int b = static_cast<int>(row / (static_cast<int64_t>(a.Hkv) * a.R));
  const Held h = held(a, b);
  const int rows = h.cnt ? rows_of(a, h) : 0, per = piece_rows(rows, k.pieces), n = per ? (rows + per - 1) / per : 0;
  const float* lp = k.part_lse + row * k.pieces;
  const float4* op = reinterpret_cast<const float4*>(k.part_o + row * k.pieces * D);
  const int g = threadIdx.x / W, c = threadIdx.x % W;
  float m = -INFINITY;
  for (int i = 0; i < n; ++i) m = fmaxf(m, lp[i]);
  const float mm = m == -INFINITY ? 0.f : m;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float w = 0.f;
#pragma unroll 4
  for (int i = g; i < n; i += 4) {
    const float wi = exp2f(lp[i] - mm);
    w += wi;
    acc = added(op[static_cast<int64_t>(i) * W + c], wi, acc);
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

// few rows leave most of a CTA's threads to share them
static int rows_per_cta(int R) { return R <= 4 ? 4 : (R <= 8 ? 8 : (R <= 16 ? 16 : 32)); }

static SimtArgs simt_cut(const PagedArgs& a, int sms) {
  SimtArgs k = {};
  k.a = a;
  const int rp = rows_per_cta(a.R);
  k.row_tiles = (a.R + rp - 1) / rp;
  const int64_t units = static_cast<int64_t>(a.B) * a.Hkv * k.row_tiles;
  const int64_t cap = ((static_cast<int64_t>(a.table_n) << a.page_log2) + kKeys - 1) / kKeys;
  int64_t n = (4ll * sms + units - 1) / units;   // four CTAs an SM
  n = n > 256 ? 256 : n;
  n = n > cap ? cap : n;
  k.pieces = static_cast<int>(n < 1 ? 1 : n);
  return k;
}
static int64_t simt_workspace(const SimtArgs& k, int D) {
  return static_cast<int64_t>(k.a.B) * k.a.Hkv * k.a.R * k.pieces * (D + 1) * 4;
}

template <int D, typename T>
static cudaError_t simt(const SimtArgs& k, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(k.row_tiles) * k.pieces, static_cast<unsigned>(k.a.B) * k.a.Hkv);
  cudaError_t e;
  switch (rows_per_cta(k.a.R)) {
    case 4: e = launch_early(simt_partials<D, T, 4>, grid, kThreads, 0, st, k); break;
    case 8: e = launch_early(simt_partials<D, T, 8>, grid, kThreads, 0, st, k); break;
    case 16: e = launch_early(simt_partials<D, T, 16>, grid, kThreads, 0, st, k); break;
    default: e = launch_early(simt_partials<D, T, 32>, grid, kThreads, 0, st, k);
  }
  if (e != cudaSuccess) return e;
  const unsigned rows = static_cast<unsigned>(static_cast<int64_t>(k.a.B) * k.a.Hkv * k.a.R);
  return launch_early(merge_kernel<D, T>, dim3(rows), D, 0, st, k);
}

// ---- acceptance -----------------------------------------------------------

struct AcceptArgs {
  void *kp, *vp;
  const int32_t *table, *lengths, *path, *accepted;
  int32_t* lengths_out;
  int64_t table_b, pages, pool_b, pool_h, pool_s;   // bytes
  int32_t Hkv, T, table_n, page_log2, vecs;         // 16-byte vectors of a row
  int* status;
};

constexpr int kAcceptThreads = 256;
constexpr int kNodes = 64;   // rows whose places are in shared memory together

// One CTA a request.  A thread owns 16-byte columns (of K or V, a head, a
// vector) and moves them row by row.  The path rises, so the row that goes to
// place i comes from i or further back, and no row is overwritten before it
// has been read; four are read at a time.
__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(const __grid_constant__ AcceptArgs a) {
  __shared__ int64_t src[kNodes], dst[kNodes];
  wait_for_previous();
  const int b = blockIdx.x;
  const int len = max(a.lengths[b], 0), n = min(max(a.accepted[b], 0), a.T);
  const int32_t* path = a.path + static_cast<int64_t>(b) * a.T;
  const int32_t* table = a.table + b * a.table_b;
  auto place = [&](int64_t row) -> int64_t {   // -1: nowhere
    const int64_t entry = row >> a.page_log2;
    const int64_t page = entry < a.table_n ? table[entry] : -1;
    return page < 0 || page >= a.pages ? -1 : page * a.pool_b + (row & ((1ll << a.page_log2) - 1)) * a.pool_s;
  };
  bool bad = false;
  for (int i = threadIdx.x; i < n; i += kAcceptThreads) {
    const int p = path[i];
    bad |= p < 0 || p >= a.T || (i > 0 && p <= path[i - 1]);
    if (!bad) bad = place(static_cast<int64_t>(len) + i) < 0 || place(static_cast<int64_t>(len) + p) < 0;
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) {
    if (bad) report(a.status, SCA_ERR_RANGE);
    a.lengths_out[b] = bad ? a.lengths[b] : len + n;
  }
  if (bad) return;
  const int columns = 2 * a.Hkv * a.vecs;
  for (int i0 = 0; i0 < n; i0 += kNodes) {
    const int cnt = min(kNodes, n - i0);
    __syncthreads();
    for (int i = threadIdx.x; i < cnt; i += kAcceptThreads) {
      dst[i] = place(static_cast<int64_t>(len) + i0 + i);
      src[i] = place(static_cast<int64_t>(len) + path[i0 + i]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < columns; c += kAcceptThreads) {
      const int v = c % a.vecs, h = c / a.vecs % a.Hkv;
      char* base = static_cast<char*>(c < a.Hkv * a.vecs ? a.kp : a.vp) + h * a.pool_h + 16 * v;
      for (int i = 0; i < cnt; i += 4) {
        uint4 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i + j < cnt && src[i + j] != dst[i + j]) x[j] = *reinterpret_cast<const uint4*>(base + src[i + j]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i + j < cnt && src[i + j] != dst[i + j]) *reinterpret_cast<uint4*>(base + dst[i + j]) = x[j];
      }
    }
  }
}

// ---- checks ---------------------------------------------------------------

constexpr int64_t kMostStride = 1LL << 40;

static int check_cache(const char* what, const sca_paged_dims* d) {
  SCA_REQUIRE(d != nullptr, SCA_ERR_ARG, "%s: dims is NULL", what);
  SCA_REQUIRE(d->B >= 1 && d->Hkv >= 1 && d->T >= 1 && d->T < 1 << 24 && static_cast<int64_t>(d->B) * d->Hkv <= 65535,
              SCA_ERR_ARG, "%s: B=%d, Hkv=%d, T=%d: need positive sizes, B*Hkv <= 65535, T < 2^24", what, d->B, d->Hkv,
              d->T);
  SCA_REQUIRE(d->dtype == SCA_BF16 || d->dtype == SCA_F32, SCA_ERR_ARG, "%s: dtype=%d unknown", what, d->dtype);
  const int mult = d->dtype == SCA_BF16 ? 8 : 4;
  SCA_REQUIRE(d->D >= mult && d->D <= 1024 && d->D % mult == 0, SCA_ERR_ARG,
              "%s: D=%d: a multiple of 16 bytes, up to 1024", what, d->D);
  SCA_REQUIRE(d->page >= 16 && d->page <= 1024 && (d->page & (d->page - 1)) == 0, SCA_ERR_ARG,
              "%s: page=%d: 16, 32, ... 1024 rows", what, d->page);
  SCA_REQUIRE(d->pages >= 1 && d->pages < 1LL << 31 && d->table_n >= 1 &&
                  static_cast<int64_t>(d->table_n) * d->page < (1LL << 31) - (1LL << 20) && d->table_b >= 0 &&
                  d->table_b < kMostStride,
              SCA_ERR_ARG, "%s: pages=%lld, table_n=%d, table_b=%lld", what, static_cast<long long>(d->pages), d->table_n,
              static_cast<long long>(d->table_b));
  const sca_view& p = d->pool;
  SCA_REQUIRE(p.b >= 0 && p.h >= 0 && p.b < kMostStride && p.h < kMostStride && p.s >= d->D && p.s < kMostStride,
              SCA_ERR_ARG, "%s: strides of the pool must be >= 0, of its rows >= D", what);
  SCA_REQUIRE(p.b % mult == 0 && p.h % mult == 0 && p.s % mult == 0, SCA_ERR_ALIGN,
              "%s: strides of the pool must be multiples of %d elements", what, mult);
  return SCA_OK;
}

// a pool that is written: no row may be another's
static bool apart(const sca_paged_dims* d) {
  int64_t st[3] = {d->pool.b, d->pool.h, d->pool.s}, n[3] = {d->pages, d->Hkv, d->page}, e = d->D;
  for (int i = 0; i < 3; ++i) {
    int at = -1;
    for (int j = 0; j < 3; ++j)
      if (n[j] > 1 && (at < 0 || st[j] < st[at])) at = j;
    if (at < 0) break;
    if (st[at] < e) return false;
    e += (n[at] - 1) * st[at];
    n[at] = 1;
  }
  return true;
}

static int page_log2(const sca_paged_dims* d) {
  int n = 4;
  while (1 << n < d->page) ++n;
  return n;
}

static int check_attend(const sca_paged_dims* d) {
  int rc;
  if ((rc = check_cache("paged_tree", d)) != SCA_OK) return rc;
  SCA_REQUIRE(d->H >= 1 && d->H % d->Hkv == 0 && static_cast<int64_t>(d->B) * d->H <= 65535 &&
                  static_cast<int64_t>(d->B) * d->H * d->T < 1LL << 31,
              SCA_ERR_ARG, "paged_tree: B=%d, H=%d, Hkv=%d, T=%d: Hkv must divide H, B*H be at most 65535, B*H*T below 2^31",
              d->B, d->H, d->Hkv, d->T);
  SCA_REQUIRE(d->D == 64 || d->D == 128, SCA_ERR_UNSUPPORTED, "paged_tree: D=%d: only 64 and 128", d->D);
  SCA_REQUIRE(static_cast<int64_t>(d->H / d->Hkv) * d->T <= 65536, SCA_ERR_UNSUPPORTED,
              "paged_tree: %d heads a key/value head x %d tokens: at most 65536 query rows", d->H / d->Hkv, d->T);
  SCA_REQUIRE(d->algo >= SCA_ALGO_AUTO && d->algo <= SCA_ALGO_TC, SCA_ERR_ARG, "paged_tree: algo=%d unknown", d->algo);
  SCA_REQUIRE(d->dtype == SCA_BF16 || d->algo != SCA_ALGO_TC, SCA_ERR_UNSUPPORTED,
              "paged_tree: the tensor-core kernel takes bf16 inputs only");
  SCA_REQUIRE(std::isfinite(d->scale) && d->scale > 0.f, SCA_ERR_ARG, "paged_tree: scale must be finite and positive");
  const int mult = d->dtype == SCA_BF16 ? 8 : 4;
  SCA_REQUIRE(d->q.b >= 0 && d->q.b < kMostStride && (d->B == 1 || d->q.b >= static_cast<int64_t>(d->H) * d->T * d->D),
              SCA_ERR_ARG, "paged_tree: q batch stride below H*T*D");
  SCA_REQUIRE(d->q.b % mult == 0, SCA_ERR_ALIGN, "paged_tree: q batch stride must be a multiple of %d elements", mult);
  SCA_REQUIRE(d->tree_b >= 0 && d->tree_b < kMostStride, SCA_ERR_ARG, "paged_tree: negative stride of tree");
  return SCA_OK;
}

static bool use_tc(const sca_paged_dims* d) { return d->dtype == SCA_BF16 && d->algo != SCA_ALGO_SIMT; }

static PagedArgs make_args(const sca_paged_dims* d) {
  PagedArgs a = {};
  a.q_b = d->q.b;
  a.table_b = d->table_b;
  a.tree_b = d->tree_b;
  a.pages = d->pages;
  a.pool = {d->pool.b, d->pool.h, d->pool.s};
  a.B = d->B;
  a.Hkv = d->Hkv;
  a.R = d->H / d->Hkv * d->T;
  a.T = d->T;
  a.page_log2 = page_log2(d);
  a.table_n = d->table_n;
  a.scale_log2 = d->scale * kLog2e;
  return a;
}

static int64_t workspace(const sca_paged_dims* d) {
  const int sms = sm_count();
  return use_tc(d) ? paged_tc_workspace(d->D, sms) : simt_workspace(simt_cut(make_args(d), sms), d->D);
}

}  // namespace paged
}  // namespace sca

using namespace sca;
using namespace sca::paged;

extern "C" int paged_tree_workspace(const sca_paged_dims* d, int64_t* bytes) {
  int rc;
  if ((rc = check_attend(d)) != SCA_OK) return rc;
  SCA_REQUIRE(bytes != nullptr, SCA_ERR_ARG, "paged_tree_workspace: bytes is NULL");
  *bytes = workspace(d);
  return SCA_OK;
}

extern "C" int paged_tree_attend(const sca_paged_dims* d, const void* q, const void* k_pages, const void* v_pages,
                                 const int32_t* table, const int32_t* lengths, const int32_t* counts,
                                 const uint64_t* tree, void* o, float* lse, float* ws, int64_t ws_bytes,
                                 int* dev_status, void* stream) {
  int rc;
  if ((rc = check_attend(d)) != SCA_OK) return rc;
  SCA_REQUIRE(q && k_pages && v_pages && table && lengths && o && lse, SCA_ERR_ARG, "paged_tree_attend: NULL pointer");
  SCA_REQUIRE(tree == nullptr || d->T <= 64, SCA_ERR_UNSUPPORTED, "paged_tree_attend: a tree of %d tokens: at most 64",
              d->T);
  SCA_REQUIRE(aligned(q, 16) && aligned(k_pages, 16) && aligned(v_pages, 16) && aligned(o, 16) && aligned(ws, 16) &&
                  aligned(lse, 4) && aligned(table, 4) && aligned(lengths, 4) && aligned(counts, 4) && aligned(tree, 8),
              SCA_ERR_ALIGN, "paged_tree_attend: tensors must be 16-byte aligned, tree 8-byte, the others 4-byte");
  const int64_t need = workspace(d);
  SCA_REQUIRE(ws && ws_bytes >= need, SCA_ERR_ARG, "paged_tree_attend: workspace of %lld bytes, %lld needed",
              static_cast<long long>(ws ? ws_bytes : 0), static_cast<long long>(need));
  PagedArgs a = make_args(d);
  a.q = q;
  a.kp = k_pages;
  a.vp = v_pages;
  a.table = table;
  a.lengths = lengths;
  a.counts = counts;
  a.tree = tree;
  a.o = o;
  a.lse = lse;
  a.status = dev_status;
  cudaStream_t st = as_stream(stream);
  const int sms = sm_count();
  if (use_tc(d)) return paged_tc_attend(a, d->D, sms, ws, st);
  SimtArgs k = simt_cut(a, sms);
  k.part_o = ws;
  k.part_lse = ws + static_cast<int64_t>(a.B) * a.Hkv * a.R * k.pieces * d->D;
  const bool bf16 = d->dtype == SCA_BF16;
  cudaError_t e;
  if (d->D == 64) e = bf16 ? simt<64, __nv_bfloat16>(k, st) : simt<64, float>(k, st);
  else e = bf16 ? simt<128, __nv_bfloat16>(k, st) : simt<128, float>(k, st);
  return cuda_status(e, "paged_tree_attend");
}

extern "C" int paged_kv_append(const sca_paged_dims* d, const void* q, const void* k, const void* v,
                               const int32_t* table, const int32_t* lengths, const int32_t* counts,
                               const int32_t* positions, const uint64_t* turns, void* k_pages, void* v_pages,
                               void* q_out, int* dev_status, void* stream) {
  int rc;
  if ((rc = check_cache("paged_kv_append", d)) != SCA_OK) return rc;
  SCA_REQUIRE(k && v && table && lengths && k_pages && v_pages, SCA_ERR_ARG, "paged_kv_append: NULL pointer");
  SCA_REQUIRE((q == nullptr) == (q_out == nullptr), SCA_ERR_ARG, "paged_kv_append: q and q_out go together");
  SCA_REQUIRE(q == nullptr || (d->H >= 1 && static_cast<int64_t>(d->B) * d->H <= 65535), SCA_ERR_ARG,
              "paged_kv_append: B=%d, H=%d", d->B, d->H);
  SCA_REQUIRE(d->rotary_dim >= 0 && d->rotary_dim <= d->D && d->rotary_dim % 2 == 0, SCA_ERR_ARG,
              "paged_kv_append: rotary_dim=%d of D=%d", d->rotary_dim, d->D);
  SCA_REQUIRE(d->rotary_dim == 0 || turns, SCA_ERR_ARG, "paged_kv_append: NULL turns");
  SCA_REQUIRE(std::isfinite(d->amplitude), SCA_ERR_ARG, "paged_kv_append: amplitude is not finite");
  SCA_REQUIRE(d->pos_b >= 0 && d->pos_b < kMostStride, SCA_ERR_ARG, "paged_kv_append: stride of positions");
  SCA_REQUIRE(apart(d), SCA_ERR_ARG, "paged_kv_append: rows of the pool overlap");
  const int eb = d->dtype == SCA_BF16 ? 2 : 4;
  for (const sca_view* x : {&d->q, &d->k, &d->v}) {
    if (x == &d->q && q == nullptr) continue;
    for (const int64_t s : {x->b, x->h, x->s})
      SCA_REQUIRE(s >= 0 && s < kMostStride, SCA_ERR_ARG, "paged_kv_append: strides of q, k or v negative or above 2^40");
  }
  SCA_REQUIRE(aligned(k_pages, 16) && aligned(v_pages, 16) && aligned(q_out, 16) && aligned(q, eb) && aligned(k, eb) &&
                  aligned(v, eb) && aligned(turns, 8) && aligned(table, 4) && aligned(lengths, 4) && aligned(counts, 4) &&
                  aligned(positions, 4),
              SCA_ERR_ALIGN, "paged_kv_append: pools and q_out must be 16-byte aligned, the others to their elements");
  RowsArgs a = {};
  a.in[0] = q;
  a.in[1] = k;
  a.in[2] = v;
  a.out[0] = q_out;
  a.out[1] = k_pages;
  a.out[2] = v_pages;
  a.iv[0] = {d->q.b, d->q.h, d->q.s};
  a.iv[1] = {d->k.b, d->k.h, d->k.s};
  a.iv[2] = {d->v.b, d->v.h, d->v.s};
  a.heads[0] = q ? d->H : 0;
  a.heads[1] = a.heads[2] = d->Hkv;
  a.ov[0] = {static_cast<int64_t>(a.heads[0]) * d->T * d->D, static_cast<int64_t>(d->T) * d->D, d->D};
  a.ov[1] = a.ov[2] = {d->pool.b, d->pool.h, d->pool.s};
  a.B = d->B;
  a.S = d->T;
  a.D = d->D;
  a.rd = d->rotary_dim;
  a.interleaved = d->interleaved != 0;
  a.amplitude = d->amplitude;
  a.sign = 1.f;
  a.turns = turns;
  a.positions = positions;
  a.pos_b = d->pos_b;
  a.table = table;
  a.lengths = lengths;
  a.counts = counts;
  a.table_b = d->table_b;
  a.pages = d->pages;
  a.table_n = d->table_n;
  a.page_log2 = page_log2(d);
  a.status = dev_status;
  return cuda_status(launch_rows(a, d->dtype, as_stream(stream)), "paged_kv_append");
}

extern "C" int paged_kv_accept(const sca_paged_dims* d, void* k_pages, void* v_pages, const int32_t* table,
                               const int32_t* lengths, const int32_t* path, const int32_t* accepted,
                               int32_t* lengths_out, int* dev_status, void* stream) {
  int rc;
  if ((rc = check_cache("paged_kv_accept", d)) != SCA_OK) return rc;
  SCA_REQUIRE(k_pages && v_pages && table && lengths && path && accepted && lengths_out, SCA_ERR_ARG,
              "paged_kv_accept: NULL pointer");
  SCA_REQUIRE(apart(d), SCA_ERR_ARG, "paged_kv_accept: rows of the pool overlap");
  SCA_REQUIRE(aligned(k_pages, 16) && aligned(v_pages, 16) && aligned(table, 4) && aligned(lengths, 4) &&
                  aligned(path, 4) && aligned(accepted, 4) && aligned(lengths_out, 4),
              SCA_ERR_ALIGN, "paged_kv_accept: pools must be 16-byte aligned, the others 4-byte");
  const int eb = d->dtype == SCA_BF16 ? 2 : 4;
  AcceptArgs a = {};
  a.kp = k_pages;
  a.vp = v_pages;
  a.table = table;
  a.lengths = lengths;
  a.path = path;
  a.accepted = accepted;
  a.lengths_out = lengths_out;
  a.table_b = d->table_b;
  a.pages = d->pages;
  a.pool_b = d->pool.b * eb;
  a.pool_h = d->pool.h * eb;
  a.pool_s = d->pool.s * eb;
  a.Hkv = d->Hkv;
  a.T = d->T;
  a.table_n = d->table_n;
  a.page_log2 = page_log2(d);
  a.vecs = d->D * eb / 16;
  a.status = dev_status;
  return cuda_status(launch_early(accept_kernel, dim3(d->B), kAcceptThreads, 0, as_stream(stream), a), "paged_kv_accept");
}
