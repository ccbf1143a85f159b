// A cache of keys and values in pages: C-ABI entry points (append, attention of
// drafted tokens, acceptance), the acceptance kernel, and the attention in
// fp32 arithmetic (fp32 inputs, and the cross-check of the tensor-core kernel
// in paged_tc.cu).  The rows of an append go through rotary.cu.
//
//   partial over a piece of rows J:  lse_J = ln sum_j exp(s_j),  o_J = sum_j exp(s_j - lse_J) v_j
//   o = sum_J w_J o_J / sum_J w_J,  w_J = exp(lse_J - max lse),  lse = max + ln sum_J w_J
#include <cooperative_groups.h>

#include <cmath>

#include "host_common.h"
#include "launch_util.h"
#include "overlap.cuh"
#include "paged.h"
#include "rotary.h"

namespace sca {
namespace paged {

namespace cg = cooperative_groups;

SCA_INLINE float4 get4(const float* p) { return *reinterpret_cast<const float4*>(p); }
SCA_INLINE void put4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
SCA_INLINE void put4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  uint2 u;
  u.x = *reinterpret_cast<const uint32_t*>(&a);
  u.y = *reinterpret_cast<const uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = u;
}
SCA_INLINE void put1(float* p, float v) { *p = v; }
SCA_INLINE void put1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Elements of a row that one load brings: 16 bytes of a key, four values.
template <typename T>
struct Row;
template <>
struct Row<float> {
  using Key = float4;
  using Value = float4;
  static constexpr int N = 4;
  static SCA_INLINE void key(const float4& r, float* x) {
    x[0] = r.x;
    x[1] = r.y;
    x[2] = r.z;
    x[3] = r.w;
  }
  static SCA_INLINE float4 value(const float4& r) { return r; }
  static SCA_INLINE float4 none4() { return make_float4(0.f, 0.f, 0.f, 0.f); }
  static SCA_INLINE float4 no_value() { return none4(); }
};
template <>
struct Row<__nv_bfloat16> {
  using Key = uint4;
  using Value = uint2;
  static constexpr int N = 8;
  static SCA_INLINE void key(const uint4& r, float* x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static SCA_INLINE float4 value(const uint2& r) {
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xffff0000u));
  }
  static SCA_INLINE uint4 none4() { return make_uint4(0, 0, 0, 0); }
  static SCA_INLINE uint2 no_value() { return make_uint2(0, 0); }
};

constexpr int kThreads = 256;
constexpr int kCluster = 16, kSplits = kPagedSplits;   // at most

// RT query rows of one request and key/value head (grid y) over every n-th tile
// of its rows, n = cluster * splits; the CTAs of a cluster then join their sums
// through each other's shared memory.
//
// Keys and values go straight from global memory to registers, once: eight
// threads hold a key (16 bytes of it at a time, next to one another's), NK keys a
// thread, and take the products of all rows with them; for the output a warp
// (D = 64: half of one) holds a value row, and each thread four columns of all RT
// rows.  A tile's loads go out as soon as the registers of the tile before are
// free, and pages are looked up a tile ahead.  Queries and weights come from
// shared memory, a vector of 16 bytes for 4 NK FMAs.
//
// What bounds it: HBM for few rows and long caches (8 requests x 8 heads x 28844 rows
// of 128, fp32, 3 rows a head: 303 us, 6.2 TB/s); for more rows the chain of a tile's
// steps, two CTAs an SM: 12 to 19 TFLOP/s (93 rows of 18 x 3 heads, 980 keys: 154 us)
// where FMAs could do 70; small calls launch, loads and the cluster's join: 40
// units of 9 rows, up to 1012 keys of 64, 10.5 us.
template <int D, typename T, int RT>
struct Simt {
  static constexpr int NK = 256 / D;               // keys a thread
  static constexpr int KT = kThreads / 8 * NK;     // keys of a tile
  static constexpr int NV = D / Row<T>::N / 8;     // 16-byte vectors of a key a thread
  static constexpr int C4 = D / 4;                 // threads of a value row
  static constexpr int PH = kThreads / C4;         // value rows at a time
  static constexpr int VK = KT / PH;               // of a thread
  static constexpr int N = RT * NK;                // products of a thread
};

template <int D, typename T, int RT>
__global__ void __launch_bounds__(kThreads, 2) simt_kernel(const __grid_constant__ PagedSplit k) {
  using S = Simt<D, T, RT>;
  using L = Row<T>;
  constexpr int NK = S::NK, KT = S::KT, NV = S::NV, C4 = S::C4, PH = S::PH, VK = S::VK;
  __shared__ alignas(16) float qs[RT][D];
  __shared__ float sc[RT][KT + 1];                 // scores
  __shared__ alignas(16) float ps[KT][RT];         // their weights
  __shared__ int64_t at[2][KT];                    // where a tile's rows lie; -1: nowhere
  __shared__ alignas(16) float red[PH / 2][RT][D];
  __shared__ alignas(16) float os[RT][D];          // this CTA's sums, for the cluster
  __shared__ float ms[RT], ls[RT], al[RT];
  __shared__ Sight sees[RT];
  const PagedArgs& a = k.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.y / a.Hkv, hk = blockIdx.y - b * a.Hkv;
  const int n = k.cluster * k.splits, rt = blockIdx.x / n, piece = blockIdx.x - rt * n, r0 = rt * RT;
  wait_for_previous();
  const int32_t* table = a.table + b * a.table_b;
  // where row tid of a tile lies, given its entry of the table
  auto place = [&](int row, int entry) -> int64_t {
    if (entry >= 0 && entry < a.pages)
      return static_cast<int64_t>(entry) * a.pool.b + (row & ((1 << a.page_log2) - 1)) * a.pool.s;
    report(a.status, SCA_ERR_RANGE);
    return -1;
  };
  // The first tile's entries and the queries come with the lengths, not behind
  // them; an entry that turns out to be no row's is not used.
  const int row0 = piece * KT + tid, entry0 = row0 >> a.page_log2;
  const int first_page = tid < KT && entry0 < a.table_n ? table[entry0] : -1;
  const T* qp = static_cast<const T*>(a.q) + b * a.q_b + static_cast<int64_t>(hk) * a.R * D;
  for (int e = tid; e < RT * (D / 4); e += kThreads) {
    const int r = e / (D / 4), c = e % (D / 4);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r < a.R) v = L::value(reinterpret_cast<const typename L::Value*>(qp + static_cast<int64_t>(r0 + r) * D)[c]);
    put4(&qs[r][4 * c], v);
  }
  const Held h = held(a, b);
  const int rows = h.cnt ? rows_of(a, h) : 0, tiles = (rows + KT - 1) / KT;
  auto look_up = [&](int tile) {
    const int row = tile * KT + tid;
    return tid < KT && row < rows ? place(row, table[row >> a.page_log2]) : static_cast<int64_t>(-1);
  };
  if (tid < KT) at[0][tid] = row0 < rows ? place(row0, first_page) : -1;
  if (tid < RT) {
    ms[tid] = -INFINITY;
    ls[tid] = 0.f;
    sees[tid] = r0 + tid < a.R ? sight(a, b, (r0 + tid) % a.T, h, rows) : Sight{0, 0};
  }
  if (blockIdx.x == 0 && hk == 0 && tid == 0) report_beyond(a, b);
  __syncthreads();
  const T *kb = static_cast<const T*>(a.kp) + hk * a.pool.h, *vb = static_cast<const T*>(a.vp) + hk * a.pool.h;
  const int l8 = tid & 7, kg = tid >> 3, c4 = tid % C4, ph = tid / C4;
  typename L::Key kr[NK][NV];
  typename L::Value vr[VK];
  auto load_keys = [&](int buf) {
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const int64_t x = at[buf][kg + 32 * i];
#pragma unroll
      for (int v = 0; v < NV; ++v)
        kr[i][v] = x < 0 ? L::none4() : reinterpret_cast<const typename L::Key*>(kb + x)[l8 + 8 * v];
    }
  };
  auto load_values = [&](int buf) {
#pragma unroll
    for (int i = 0; i < VK; ++i) {
      const int64_t x = at[buf][ph + PH * i];
      vr[i] = x < 0 ? L::no_value() : reinterpret_cast<const typename L::Value*>(vb + x)[c4];
    }
  };
  load_keys(0);
  load_values(0);
  float4 acc[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
  int buf = 0;
#pragma unroll 1
  for (int tile = piece; tile < tiles; tile += n, buf ^= 1) {
    const bool more = tile + n < tiles;
    if (more && tid < KT) at[buf ^ 1][tid] = look_up(tile + n);
    // ---- scores: NK keys of this thread's eighth of D with every row
    float s[S::N];
#pragma unroll
    for (int i = 0; i < S::N; ++i) s[i] = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float x[NK][L::N];
#pragma unroll
      for (int i = 0; i < NK; ++i) L::key(kr[i][v], x[i]);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int e = 0; e < L::N; e += 4) {
          const float4 q = get4(&qs[r][(l8 + 8 * v) * L::N + e]);
#pragma unroll
          for (int i = 0; i < NK; ++i)
            s[r * NK + i] = fmaf(q.x, x[i][e], fmaf(q.y, x[i][e + 1], fmaf(q.z, x[i][e + 2], fmaf(q.w, x[i][e + 3], s[r * NK + i]))));
        }
    }
    // the eight threads of a key add up: each hands half of its sums over at every step
#pragma unroll
    for (int w = S::N / 2, o = 4; o; w >>= 1, o >>= 1)
#pragma unroll
      for (int i = 0; i < S::N / 2; ++i)
        if (i < w) {
          const float give = l8 & o ? s[i] : s[i + w];
          s[i] = (l8 & o ? s[i + w] : s[i]) + __shfl_xor_sync(0xffffffffu, give, o);
        }
    const int first = (l8 & 4 ? S::N / 2 : 0) + (l8 & 2 ? S::N / 4 : 0) + (l8 & 1 ? S::N / 8 : 0);
#pragma unroll
    for (int i = 0; i < S::N / 8; ++i) sc[(first + i) / NK][kg + 32 * ((first + i) % NK)] = s[i] * a.scale_log2;
    __syncthreads();
    if (more) load_keys(buf ^ 1);
    // ---- weights: a warp a row
    for (int r = warp; r < RT; r += kThreads / 32) {
      float x[KT / 32], mx = -INFINITY;
      const Sight sr = sees[r];
#pragma unroll
      for (int i = 0; i < KT / 32; ++i) {
        const int j = tile * KT + 32 * i;
        const uint32_t bits = seen_bits(sr, h.len, j);
        x[i] = (bits >> lane) & 1 && j + lane < rows ? sc[r][32 * i + lane] : -INFINITY;
        mx = fmaxf(mx, x[i]);
      }
      for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float old = ms[r], m = fmaxf(old, mx), sub = m == -INFINITY ? 0.f : m;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < KT / 32; ++i) {
        x[i] = exp2f(x[i] - sub);
        sum += x[i];
        ps[32 * i + lane][r] = x[i];
      }
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      __syncwarp();
      if (lane == 0) {
        const float f = exp2f(old - sub);
        ms[r] = m;
        ls[r] = fmaf(ls[r], f, sum);
        al[r] = f;
      }
    }
    __syncthreads();
    // ---- output: four columns of every row over this thread's value rows
    if (tile != piece) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float f = al[r];
        acc[r] = make_float4(acc[r].x * f, acc[r].y * f, acc[r].z * f, acc[r].w * f);
      }
    }
#pragma unroll
    for (int i = 0; i < VK; ++i) {
      const float4 v = L::value(vr[i]);
#pragma unroll
      for (int r4 = 0; r4 < RT; r4 += 4) {
        const float4 w = get4(&ps[ph + PH * i][r4]);
        const float w4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          acc[r4 + r].x = fmaf(w4[r], v.x, acc[r4 + r].x);
          acc[r4 + r].y = fmaf(w4[r], v.y, acc[r4 + r].y);
          acc[r4 + r].z = fmaf(w4[r], v.z, acc[r4 + r].z);
          acc[r4 + r].w = fmaf(w4[r], v.w, acc[r4 + r].w);
        }
      }
    }
    if (more) load_values(buf ^ 1);
  }
  // ---- the value rows' sums, in a fixed order: the upper half of them, then all
  if (ph >= PH / 2) {
#pragma unroll
    for (int r = 0; r < RT; ++r) put4(&red[ph - PH / 2][r][4 * c4], acc[r]);
  }
  __syncthreads();
  if (ph < PH / 2) {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const float4 v = get4(&red[ph][r][4 * c4]);
      put4(&red[ph][r][4 * c4], make_float4(acc[r].x + v.x, acc[r].y + v.y, acc[r].z + v.z, acc[r].w + v.w));
    }
  }
  __syncthreads();
  for (int e = tid; e < RT * D; e += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < PH / 2; ++i) v += (&red[i][0][0])[e];
    (&os[0][0])[e] = v;
  }
  // ---- the cluster's CTAs: each takes every n-th number of the rows
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = k.cluster, rank = static_cast<int>(cluster.block_rank()), split = piece / nc;
  cluster.sync();
  const int per = RT * D / nc;
  for (int e = rank * per + tid; e < (rank + 1) * per; e += kThreads) {
    const int r = e / D, c = e % D;
    if (r0 + r >= a.R) break;
    float m[8], mx = -INFINITY, sum = 0.f, o = 0.f;
    auto maxima = [&](int i0) {   // of eight CTAs
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m[i] = i0 + i < nc ? *cluster.map_shared_rank(&ms[r], i0 + i) : -INFINITY;
        mx = fmaxf(mx, m[i]);
      }
    };
    maxima(0);
    if (nc > 8) maxima(8);
    const float sub = mx == -INFINITY ? 0.f : mx;
    auto sums = [&](int i0) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i0 + i < nc) {
          const float w = exp2f(m[i] - sub);
          sum = fmaf(w, *cluster.map_shared_rank(&ls[r], i0 + i), sum);
          o = fmaf(w, *cluster.map_shared_rank(&os[r][c], i0 + i), o);
        }
    };
    if (nc > 8) {   // (the maxima at hand are those of the upper eight)
      sums(8);
      maxima(0);
    }
    sums(0);
    o = sum == 0.f ? 0.f : o / sum;
    const float lse2 = sum == 0.f ? -INFINITY : sub + log2f(sum);
    const int64_t row = static_cast<int64_t>(blockIdx.y) * a.R + r0 + r;
    if (k.splits == 1) {
      put1(static_cast<T*>(a.o) + row * D + c, o);
      if (c == 0) a.lse[row] = lse2 * kLn2;
    } else {
      k.part_o[(row * k.splits + split) * D + c] = o;
      if (c == 0) k.part_lse[row * k.splits + split] = lse2;
    }
  }
  cluster.sync();   // nobody's shared memory goes before all have read it
}

// One CTA of four groups of D/4 threads per query row: the groups take the
// row's partials in turn, their sums meet in shared memory in a fixed order.
template <int D, typename T>
__global__ void __launch_bounds__(D) merge_kernel(const __grid_constant__ PagedSplit k) {
  constexpr int W = D / 4;
  __shared__ float4 so[4][W];
  __shared__ float sw[kSplits];
  const PagedArgs& a = k.a;
  wait_for_previous();
  const int64_t row = blockIdx.x;
  const int n = k.splits, g = threadIdx.x / W, c = threadIdx.x % W;
  const float4* op = reinterpret_cast<const float4*>(k.part_o + row * n * D);
  static_assert(kSplits <= 64 && D >= 64, "a thread a partial");
  if (threadIdx.x < n) sw[threadIdx.x] = k.part_lse[row * n + threadIdx.x];
  __syncthreads();
  float m = -INFINITY, total = 0.f;
  for (int i = 0; i < n; ++i) m = fmaxf(m, sw[i]);
  const float mm = m == -INFINITY ? 0.f : m;
  for (int i = 0; i < n; ++i) total += exp2f(sw[i] - mm);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = g; i0 < n; i0 += 32) {   // eight partials' loads together
    float4 v[8];
#pragma unroll
    for (int t = 0; t < 8; ++t)
      v[t] = i0 + 4 * t < n ? op[static_cast<int64_t>(i0 + 4 * t) * W + c] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const float w = i0 + 4 * t < n ? exp2f(sw[i0 + 4 * t] - mm) : 0.f;
      acc.x = fmaf(w, v[t].x, acc.x);
      acc.y = fmaf(w, v[t].y, acc.y);
      acc.z = fmaf(w, v[t].z, acc.z);
      acc.w = fmaf(w, v[t].w, acc.w);
    }
  }
  so[g][c] = acc;
  __syncthreads();
  if (g != 0) return;
  const float inv = total == 0.f ? 0.f : 1.f / total;
  const float4 p = so[0][c], q = so[1][c], r = so[2][c], s = so[3][c];
  put4(static_cast<T*>(a.o) + row * D + 4 * c,
       make_float4(((p.x + q.x) + (r.x + s.x)) * inv, ((p.y + q.y) + (r.y + s.y)) * inv,
                   ((p.z + q.z) + (r.z + s.z)) * inv, ((p.w + q.w) + (r.w + s.w)) * inv));
  if (c == 0) a.lse[row] = total == 0.f ? -INFINITY : (mm + log2f(total)) * kLn2;
}

// rows of a CTA: eight, or four where that leaves fewer without use
static int rows_per_cta(int R) { return (R + 7) / 8 * 8 > (R + 3) / 4 * 4 ? 4 : 8; }

static PagedSplit simt_cut(const PagedArgs& a, int D, int sms) {
  PagedSplit k = {};
  k.a = a;
  const int rt = rows_per_cta(a.R), KT = kThreads / 8 * (256 / D);
  k.row_tiles = (a.R + rt - 1) / rt;
  const int64_t units = static_cast<int64_t>(a.B) * a.Hkv * k.row_tiles;
  const int64_t tiles = ((static_cast<int64_t>(a.table_n) << a.page_log2) + KT - 1) / KT;
  // a CTA an SM at least (two: 4 x 8 x 4 rows x 200 keys of 128, bf16, 16.6 us instead of 13.2)
  // Clusters of sixteen, for which the SMs of one part of the chip must be free, only for
  // up to two tiles a CTA and few units, or where eight CTAs would need a second
  // cluster: one head, 8 rows x 1000 keys 8.9 -> 7.5 us, 2 heads, one row x 3000 of 64 8.2
  // -> 7.7, 8 heads, 4 rows x 2000 10.7 -> 9.6; but 8 units x 1000 keys 6.8 -> 7.2.
  const bool wide = tiles <= 2 * kCluster && (units <= 4 || (units * kCluster <= sms && tiles > kCluster));
  const int most_ctas = wide ? kCluster : 8;
  k.cluster = 1;
  while (k.cluster < most_ctas && k.cluster < tiles && units * k.cluster < sms) k.cluster *= 2;
  // Several clusters a unit fill the SMs twice, but not for fewer than two tiles
  // a CTA: their join is a launch of its own (one token behind 1000 keys 8.4 us
  // instead of 7.1; behind 4000 keys 11.1, and 15.3 with one cluster).
  int64_t n = 2ll * sms / (units * k.cluster), most = tiles / k.cluster / 2;
  n = n > kSplits ? kSplits : n;
  n = n > most ? most : n;
  k.splits = static_cast<int>(n < 1 ? 1 : n);
  return k;
}
// Partials lie behind the counters of the tensor-core kernels, which may get the
// same workspace: a plan's call with a short table is a small one.
constexpr int64_t kHeadFloats = 1024;
static int64_t simt_workspace(const PagedArgs& a, int splits, int D) {
  return splits == 1 ? 0 : (kHeadFloats + static_cast<int64_t>(a.B) * a.Hkv * a.R * splits * (D + 1)) * 4;
}

template <int D, typename T, int RT>
static cudaError_t launch_simt(const PagedSplit& k, cudaStream_t st) {
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(k.cluster);
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(k.row_tiles) * k.cluster * k.splits, static_cast<unsigned>(k.a.B) * k.a.Hkv);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  static std::atomic<bool> done[kMaxCachedDevices];
  if (k.cluster > 8) {
    const cudaError_t e =
        allow_attribute(simt_kernel<D, T, RT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1, done);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, simt_kernel<D, T, RT>, k);
}

template <int D, typename T>
static cudaError_t simt(const PagedSplit& k, cudaStream_t st) {
  cudaError_t e;
  if (k.cluster == 0) e = paged_f32_launch(k, D, st);   // (fp32 alone)
  else e = rows_per_cta(k.a.R) == 4 ? launch_simt<D, T, 4>(k, st) : launch_simt<D, T, 8>(k, st);
  if (e != cudaSuccess || k.splits == 1) return e;
  return launch_early(merge_kernel<D, T>, dim3(static_cast<unsigned>(static_cast<int64_t>(k.a.B) * k.a.Hkv * k.a.R)), D, 0,
                      st, k);
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
// has been read; four are read at a time.  Trips to memory one after the other bound
// it: accepted, path, pages, then each four rows behind the stores of those before
// (captured, one request 2.4 us, 256 requests, up to 20 rows of 64 moved, 8 heads of 128,
// 5.2 us, where the rows' bytes take 1).  Not all of that order is forced: the path could be
// read beside the lengths, and more rows at a time.  Neither is measured.
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
    bool wrong = p < 0 || p >= a.T || (i > 0 && p <= path[i - 1]);
    if (!wrong) {
      const int64_t to = place(static_cast<int64_t>(len) + i), from = place(static_cast<int64_t>(len) + p);
      wrong = to < 0 || from < 0;
      if (i < kNodes) {
        dst[i] = to;
        src[i] = from;
      }
    }
    bad |= wrong;
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
    if (i0 > 0) {   // (the first places are there)
      __syncthreads();
      for (int i = threadIdx.x; i < cnt; i += kAcceptThreads) {
        dst[i] = place(static_cast<int64_t>(len) + i0 + i);
        src[i] = place(static_cast<int64_t>(len) + path[i0 + i]);
      }
      __syncthreads();
    }
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

static bool few_rows(const sca_paged_dims* d) { return static_cast<int64_t>(d->H / d->Hkv) * d->T <= kPagedFewRows; }

// Tensor cores for bf16, unless the whole cache of the call's requests is small:
// their kernels' start, one-off code and joins take longer than the work in fp32
// then.  Rows and keys count by whole tiles of the fp32 kernel.  32 heads on 8 of 128,
// one token: behind 1000 rows (17 MFLOP) 7.1 us in fp32 and 9.4, behind 4000 (67) 13.8
// and 11.6, four requests behind 1000 9.4 and 10.7; 8 heads of their own, 16 requests
// behind 500 (134) 13.8 and 9.5; more rows, 64 of one head, 23 requests behind 29 rows
// (48) 11.5 and 8.6, but 6 heads' 22, two requests behind 525 (48) 7.8 and 11.9: few
// tiles of rows leave room for clusters.  The table's width stands for the lengths,
// which only the device knows: the token behind 1000 rows takes 6.6 us with a table of
// their size, 8.3 and 9.7 with one for 4096 and 32768 rows.
static bool use_tc(const sca_paged_dims* d) {
  if (d->dtype != SCA_BF16 || d->algo != SCA_ALGO_AUTO) return d->algo == SCA_ALGO_TC;
  const int64_t KT = kThreads / 8 * (256 / d->D), keys = (static_cast<int64_t>(d->table_n) * d->page + KT - 1) / KT * KT;
  const int R = d->H / d->Hkv * d->T, rt = rows_per_cta(R);
  const double row_tiles = static_cast<double>(d->B) * d->Hkv * ((R + rt - 1) / rt);
  return row_tiles * rt * 4 * d->D * keys > (few_rows(d) ? 70e6 : row_tiles <= 100 ? 100e6 : 40e6);
}

// fp32 rows in tiles of 64 (paged_f32.cu), where those are full enough and the keys
// long enough: a full one takes 0.62 of the time of its rows by eights (32 requests' x
// 8 heads' 32 rows, 1000 keys of 128: 267 us instead of 214; 54 heads' 93 rows 115
// instead of 154; 1 x 8 heads' 64 rows, 4000 keys 38 instead of 58), but starts more
// slowly (16 heads' 112 rows, 128 keys 19.5 us instead of 13.2).
static bool many_f32_rows(const sca_paged_dims* d) {
  const int64_t R = d->H / d->Hkv * d->T;
  return d->dtype == SCA_F32 && (R + 63) / 64 * 64 * 62 < (R + 7) / 8 * 8 * 100 &&
         static_cast<int64_t>(d->table_n) * d->page >= 512;
}

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
  if (use_tc(d)) return few_rows(d) ? paged_few_workspace(d->D) : paged_tc_workspace(d->D, sms);
  const PagedArgs a = make_args(d);
  int splits;
  if (many_f32_rows(d)) paged_f32_cut(a, sms, &splits);
  else splits = simt_cut(a, d->D, sms).splits;
  return simt_workspace(a, splits, d->D);
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
  SCA_REQUIRE(need == 0 || (ws && ws_bytes >= need), SCA_ERR_ARG, "paged_tree_attend: workspace of %lld bytes, %lld needed",
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
  if (use_tc(d)) return few_rows(d) ? paged_few_attend(a, d->D, sms, ws, st) : paged_tc_attend(a, d->D, sms, ws, st);
  int most;
  PagedSplit k = many_f32_rows(d) ? paged_f32_cut(a, sms, &most) : simt_cut(a, d->D, sms);
  k.part_o = ws + kHeadFloats;
  k.part_lse = k.part_o + static_cast<int64_t>(a.B) * a.Hkv * a.R * k.splits * d->D;
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
  // Rows are read and written in no order: what is written must be nothing else.  Queries
  // may be turned in place, where every thread writes what it has read.
  const int64_t one = static_cast<int64_t>(d->T) * d->D;
  const int H = q ? d->H : 0;
  const sca_view out = {H * one, one, d->D};
  const Rows to[3] = {row_set(k_pages, d->pool, d->pages, d->Hkv, d->page, d->D, eb),
                      row_set(v_pages, d->pool, d->pages, d->Hkv, d->page, d->D, eb),
                      row_set(q_out, out, d->B, H, d->T, d->D, eb)};
  const Rows from[3] = {row_set(k, d->k, d->B, d->Hkv, d->T, d->D, eb), row_set(v, d->v, d->B, d->Hkv, d->T, d->D, eb),
                        row_set(q, d->q, d->B, H, d->T, d->D, eb)};
  const bool in_place = q == q_out && (d->B == 1 || d->q.b == out.b) && (H == 1 || d->q.h == out.h) &&
                        (d->T == 1 || d->q.s == out.s);
  const int n = q ? 3 : 2;
  for (int i = 0; i < n; ++i) {
    for (int j = 0; j < n; ++j)
      SCA_REQUIRE((i == 2 && j == 2 && in_place) || !share_bytes(to[i], from[j]), SCA_ERR_ARG,
                  "paged_kv_append: q, k or v overlaps the pools or q_out");
    for (int j = 0; j < i; ++j)
      SCA_REQUIRE(!share_bytes(to[i], to[j]), SCA_ERR_ARG, "paged_kv_append: the pools and q_out overlap");
  }
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
  a.heads[0] = H;
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
  SCA_REQUIRE(!share_bytes(row_set(k_pages, d->pool, d->pages, d->Hkv, d->page, d->D, eb),
                           row_set(v_pages, d->pool, d->pages, d->Hkv, d->page, d->D, eb)),
              SCA_ERR_ARG, "paged_kv_accept: the pools overlap");
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
