// Causal linear attention with a decay per head: C-ABI entry points, the
// cut of long sequences into segments, the kernels in fp32 arithmetic (fp32
// inputs, and the cross-check of the tensor-core kernels in decay_tc.cu) and
// the single-token step.
//
//   S_t = exp(g_h) S_{t-1} + k_t^T v_t,   o_t = scale q_t S_t
//
// Every direction is a pass of one recurrence (decay.h).  A sequence is cut
// into nseg segments so that heads x batch x segments fill the SMs; then
// three launches do a pass: each segment's own sum (simt_pass<kStates>), the
// state before each segment and behind the last (seg_scan_kernel), the
// outputs (simt_pass).
#include <cmath>

#include "common.cuh"
#include "decay.h"
#include "host_common.h"
#include "launch_util.h"

namespace sca {
namespace decay {

constexpr int kBlk = kDecayBlk;
constexpr int kThreads = 256;

// acc[i][u] += sum_k A(m0 + i, k) * B(k, n), A and B in shared memory, each
// read row-major or transposed (AT: A[k][m], BT: B[n][k]), K a multiple of 4.
// Columns n = RN tj + u, or tj + 16 u where B is transposed (then 16 threads
// read 16 rows, which the row stride of 4 mod 32 words spreads over the
// banks).  Reads are 16 bytes wide: with scalar ones the loop waited for them
// twice as long as for its FMAs.
template <int RM, int RN, bool AT, bool BT>
SCA_INLINE void mm(float (&acc)[RM][RN], const float* A, int lda, const float* B, int ldb, int K, int m0, int tj) {
  static_assert(RM % 4 == 0 && RN % 4 == 0, "whole vectors");
#pragma unroll 2
  for (int k = 0; k < K; k += 4) {
    float a[4][RM], b[4][RN];   // [k][.]
#pragma unroll
    for (int i = 0; i < RM; i += AT ? 4 : 1)
      if (AT) {
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<float4*>(&a[e][i]) = *reinterpret_cast<const float4*>(A + (k + e) * lda + m0 + i);
      } else {
        const float4 v = *reinterpret_cast<const float4*>(A + (m0 + i) * lda + k);
        a[0][i] = v.x; a[1][i] = v.y; a[2][i] = v.z; a[3][i] = v.w;
      }
#pragma unroll
    for (int u = 0; u < RN; u += BT ? 1 : 4)
      if (BT) {
        const float4 v = *reinterpret_cast<const float4*>(B + (tj + 16 * u) * ldb + k);
        b[0][u] = v.x; b[1][u] = v.y; b[2][u] = v.z; b[3][u] = v.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<float4*>(&b[e][u]) = *reinterpret_cast<const float4*>(B + (k + e) * ldb + RN * tj + u);
      }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int u = 0; u < RN; ++u) acc[i][u] = fmaf(a[e][i], b[e][u], acc[i][u]);
  }
}

SCA_INLINE void put(float* p, float x) { *p = x; }
SCA_INLINE void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
SCA_INLINE void put4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
SCA_INLINE void put4(__nv_bfloat16* p, float a, float b, float c, float d) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b), y = __floats2bfloat162_rn(c, d);
  uint2 u;
  u.x = *reinterpret_cast<const uint32_t*>(&x);
  u.y = *reinterpret_cast<const uint32_t*>(&y);
  *reinterpret_cast<uint2*>(p) = u;
}
SCA_INLINE float4 get4(const float* p) { return *reinterpret_cast<const float4*>(p); }
SCA_INLINE float4 get4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}

template <int D>
struct Smem {
  static constexpr int LD = D + 4;      // rows on 16 bytes, 4 words apart modulo the banks
  static constexpr int LM = kBlk + 4;
  static constexpr int S = 0;
  static constexpr int X = S + D * LD;
  static constexpr int Y = X + kBlk * LD;
  static constexpr int Z = Y + kBlk * LD;
  static constexpr int M = X;           // once both products with X are made
  static constexpr int W = Z + kBlk * LD;
  static constexpr int BYTES = (W + kBlk + 1) * 4;
};

// fp32 FMAs bound it: 64 rows of 64 features are 8192 clk of them a chunk and
// SM.  Training on 8 heads x 1000 rows of 64 takes 45.8 us in a loop, 16.8 of
// them forward.  Its launches one at a time, with cold caches, are longer: 8.5
// (sums), 4.6 (scan) and 14.2 us (outputs) forward, 7.6, 4.4 and 24.4 (the
// three gradients, as one) backward.  A prompt of 16 heads x 32768 rows of 128:
// 2021 us, 25 TFLOP/s of about 76.
//
// One CTA per (segment, batch x head): chunks of kBlk rows in processing
// order, the state in shared memory.  kStates: only the segment's own sum
// (from a zero state), into p.seg.
// grid z: which of up to three passes (a backward's).
struct Passes {
  DecayPass p[3];
};
template <int D, typename T, bool kStates>
__global__ void __launch_bounds__(kThreads, D == 64 ? 3 : 1) simt_pass(const __grid_constant__ Passes ps) {
  const DecayPass& p = ps.p[blockIdx.z];
  using L = Smem<D>;
  constexpr int LD = L::LD, LM = L::LM, R = D / 16;
  extern __shared__ float sm[];
  float *Ss = sm + L::S, *Xs = sm + L::X, *Ys = sm + L::Y, *Zs = sm + L::Z, *Ms = sm + L::M, *W = sm + L::W;
  const int i = blockIdx.x, bh = blockIdx.y, b = bh / p.H, h = bh % p.H;
  const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
  wait_for_previous();   // the lengths may be an earlier kernel's as well
  const float g = p.log_decay[h];
  const int64_t len = decay_len(p, b);
  const DecayRows rows = decay_rows(p, i, len);
  const bool rev = p.reverse != 0;
  const T* x = static_cast<const T*>(p.x) + b * p.xv.b + h * p.xv.h;
  const T* y = static_cast<const T*>(p.y) + b * p.yv.b + h * p.yv.h;
  const T* z = static_cast<const T*>(p.z) + b * p.zv.b + h * p.zv.h;
  T* out = kStates ? nullptr : static_cast<T*>(p.out) + b * p.ov.b + h * p.ov.h;

  for (int e = threadIdx.x; e <= kBlk; e += kThreads) W[e] = decay_pow(g, e);
  const float* from = nullptr;
  if (!kStates) from = p.seg ? p.seg + (static_cast<int64_t>(bh) * p.nseg + i) * D * D
                             : (p.init ? p.init + b * p.init_b + static_cast<int64_t>(h) * D * D : nullptr);
#pragma unroll 4
  for (int e = threadIdx.x; e < D * (D / 4); e += kThreads) {
    const int r = e / (D / 4), c = 4 * (e % (D / 4));
    const float4 v = from ? *reinterpret_cast<const float4*>(from + r * D + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    if (!p.transposed) {
      *reinterpret_cast<float4*>(Ss + r * LD + c) = v;
    } else {
      Ss[c * LD + r] = v.x;
      Ss[(c + 1) * LD + r] = v.y;
      Ss[(c + 2) * LD + r] = v.z;
      Ss[(c + 3) * LD + r] = v.w;
    }
  }
  // rows behind the sequence: zeros
  if (!kStates)
    for (int64_t e = threadIdx.x; e < (rows.s1 - rows.hi) * D; e += kThreads)
      put(out + (rows.hi + e / D) * p.ov.s + e % D, 0.f);
  int delta = rev && !kStates && rows.s1 >= len ? 1 : 0;
  const int nchunk = static_cast<int>((rows.hi - rows.lo + kBlk - 1) / kBlk);
  const bool want_end = kStates || (p.end && i == p.nseg - 1);
  for (int ci = 0; ci < nchunk; ++ci) {
    const int64_t c0 = rows.lo + static_cast<int64_t>(rev ? nchunk - 1 - ci : ci) * kBlk;
    const int n = static_cast<int>(min64(kBlk, rows.hi - c0));
    __syncthreads();
#pragma unroll 4
    for (int e = threadIdx.x; e < kBlk * (D / 4); e += kThreads) {
      const int r = e / (D / 4), c = 4 * (e % (D / 4));
      const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
      const bool in = r < n;
      if (!kStates) *reinterpret_cast<float4*>(Xs + r * LD + c) = in ? get4(x + (c0 + r) * p.xv.s + c) : zero;
      *reinterpret_cast<float4*>(Ys + r * LD + c) = in ? get4(y + (c0 + r) * p.yv.s + c) : zero;
      *reinterpret_cast<float4*>(Zs + r * LD + c) = in ? get4(z + (c0 + r) * p.zv.s + c) : zero;
    }
    __syncthreads();
    if (!kStates) {
      float acc[4][R] = {}, m[4][4] = {};
      mm<4, R, false, false>(acc, Xs, LD, Ss, LD, D, 4 * ti, tj);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int t = 4 * ti + a, rho = rev ? n - 1 - t : t;     // place in processing order
        const float f = t < n ? p.si * W[rho + 1 - delta] : 0.f;
#pragma unroll
        for (int u = 0; u < R; ++u) acc[a][u] *= f;
      }
      mm<4, 4, false, true>(m, Xs, LD, Ys, LD, D, 4 * ti, tj);
      __syncthreads();
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int t = 4 * ti + a, s = tj + 16 * u, d = rev ? s - t : t - s;
          Ms[t * LM + s] = d >= 0 && s < n && t < n ? p.so * W[d] * m[a][u] : 0.f;
        }
      __syncthreads();
      mm<4, R, false, false>(acc, Ms, LM, Zs, LD, kBlk, 4 * ti, tj);
#pragma unroll
      for (int a = 0; a < 4; ++a)
        if (4 * ti + a < n)
#pragma unroll
          for (int u = 0; u < R; u += 4)
            put4(out + (c0 + 4 * ti + a) * p.ov.s + R * tj + u, acc[a][u], acc[a][u + 1], acc[a][u + 2], acc[a][u + 3]);
    }
    if (!want_end && ci + 1 == nchunk) break;   // nobody asks for the state after the last rows
    // S = lambda^(n - delta) S + us sum_s lambda^(n - 1 - rho_s) y_s^T z_s
    for (int e = threadIdx.x; e < n * D; e += kThreads) {
      const int r = e / D, c = e % D;
      Ys[r * LD + c] *= W[rev ? r : n - 1 - r];
    }
    __syncthreads();
    float u2[R][R] = {};
    mm<R, R, true, false>(u2, Ys, LD, Zs, LD, kBlk, R * ti, tj);
    const float carry = W[n - delta];
#pragma unroll
    for (int a = 0; a < R; ++a)
#pragma unroll
      for (int u = 0; u < R; ++u) {
        float* s = Ss + (R * ti + a) * LD + R * tj + u;
        *s = fmaf(carry, *s, p.us * u2[a][u]);
      }
    delta = 0;
  }
  __syncthreads();
  float* to = nullptr;
  float mul = 1.f;
  if (kStates) to = p.seg + (static_cast<int64_t>(bh) * p.nseg + i) * D * D;
  else if (want_end) {
    to = p.end + static_cast<int64_t>(bh) * D * D;
    if (rev && len > 0) mul = decay_pow(g, 1);
  }
  if (to)
    for (int e = threadIdx.x; e < D * D; e += kThreads) {
      const int r = e / D, c = e % D;
      to[e] = mul * Ss[r * LD + c];
    }
}

// The segments' own sums (processing order) become the state before each
// segment: start_0 = init, start_(i+1) = lambda^(n_i - delta) start_i + own_i;
// the one behind the last segment is the end state, where `end` wants it (in
// reverse times lambda, if there were rows; the last segment has a sum only
// then).  An entry a thread, all loads of a group of segments in flight before
// the first is used; the powers are made once, by the first warp.  9 segments
// of 16 heads (9.4 MB, in L2): 6.5 us, most of it two round trips and the
// launch.
constexpr int kScanGroup = 16;
__global__ void __launch_bounds__(256) seg_scan_kernel(const __grid_constant__ DecayPass p) {
  __shared__ float pw[kScanGroup];
  const int e = blockIdx.x * 256 + threadIdx.x;
  const int bh = blockIdx.y, b = bh / p.H, h = bh % p.H;
  const int DD = gridDim.x * 256;
  wait_for_previous();
  float* base = p.seg + static_cast<int64_t>(bh) * p.nseg * DD + e;
  const int n_own = p.end ? p.nseg : p.nseg - 1;
  float run = p.init ? p.init[b * p.init_b + static_cast<int64_t>(h) * DD + e] : 0.f;
  for (int i0 = 0; i0 < p.nseg; i0 += kScanGroup) {
    float v[kScanGroup];
#pragma unroll
    for (int u = 0; u < kScanGroup; ++u) v[u] = i0 + u < n_own ? base[static_cast<int64_t>(i0 + u) * DD] : 0.f;
    __syncthreads();
    if (threadIdx.x < kScanGroup && i0 + threadIdx.x < p.nseg) {
      const int64_t len = decay_len(p, b);
      const DecayRows r = decay_rows(p, i0 + threadIdx.x, len);
      const int64_t n = r.hi - r.lo;
      pw[threadIdx.x] = n > 0 ? decay_pow(p.log_decay[h], n - (p.reverse && r.s1 >= len ? 1 : 0)) : 1.f;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kScanGroup; ++u)
      if (i0 + u < p.nseg) {
        base[static_cast<int64_t>(i0 + u) * DD] = run;
        run = fmaf(pw[u], run, v[u]);   // a segment without rows has a sum of zero
      }
  }
  if (p.end) {
    const bool back = p.reverse && decay_len(p, b) > 0;
    p.end[static_cast<int64_t>(bh) * DD + e] = back ? decay_pow(p.log_decay[h], 1) * run : run;
  }
}

// One token of every sequence: S <- lambda S + k^T v in place, o = scale q S.
// It reads and writes the states (2 x 4 D^2 bytes a head) and nothing else of
// size, so bytes bound it.  A CTA takes COLS columns of one state: a thread
// holds the same four columns of D / RG rows, all of whose loads are in
// flight before the first is used; the sum over rows ends in shared memory,
// in a fixed order.  256 x 16 heads of 128: 79.8 us, 6.7 TB/s.
struct StepArgs {
  const void *q, *k, *v;
  View qv, kv, vv;
  const float* log_decay;
  float* state;
  int64_t state_b;
  void* o;
  int32_t H;
  float scale;
};
template <int D, typename T, int COLS>
__global__ void __launch_bounds__(256) step_kernel(const __grid_constant__ StepArgs a) {
  constexpr int CG = COLS / 4, RG = 256 / CG, NR = D / RG;
  static_assert(RG <= D, "a row group has a row");
  __shared__ float qs[D], ks[D];
  __shared__ float4 red[RG][CG];
  wait_for_previous();
  const int bh = blockIdx.y, b = bh / a.H, h = bh - b * a.H;
  const int cg = threadIdx.x % CG, rg = threadIdx.x / CG, c0 = blockIdx.x * COLS;
  float4* S = reinterpret_cast<float4*>(a.state + b * a.state_b + static_cast<int64_t>(h) * D * D + c0) + cg;
  float4 s[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) s[i] = S[(rg + i * RG) * (D / 4)];
  if (threadIdx.x < D) qs[threadIdx.x] = to_f32(static_cast<const T*>(a.q)[b * a.qv.b + h * a.qv.h + threadIdx.x]);
  if (threadIdx.x >= 256 - D) ks[threadIdx.x - (256 - D)] = to_f32(static_cast<const T*>(a.k)[b * a.kv.b + h * a.kv.h + threadIdx.x - (256 - D)]);
  const T* vp = static_cast<const T*>(a.v) + b * a.vv.b + h * a.vv.h + c0 + 4 * cg;
  const float4 vr = make_float4(to_f32(vp[0]), to_f32(vp[1]), to_f32(vp[2]), to_f32(vp[3]));
  const float lam = decay_pow(a.log_decay[h], 1);
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int r = rg + i * RG;
    const float kr = ks[r], qr = qs[r];
    s[i].x = fmaf(lam, s[i].x, kr * vr.x);
    s[i].y = fmaf(lam, s[i].y, kr * vr.y);
    s[i].z = fmaf(lam, s[i].z, kr * vr.z);
    s[i].w = fmaf(lam, s[i].w, kr * vr.w);
    S[r * (D / 4)] = s[i];
    acc.x = fmaf(qr, s[i].x, acc.x);
    acc.y = fmaf(qr, s[i].y, acc.y);
    acc.z = fmaf(qr, s[i].z, acc.z);
    acc.w = fmaf(qr, s[i].w, acc.w);
  }
  red[rg][cg] = acc;
  __syncthreads();
  if (threadIdx.x < COLS) {
    const float* r = reinterpret_cast<const float*>(red) + threadIdx.x;
    float sum = 0.f;
#pragma unroll 8
    for (int i = 0; i < RG; ++i) sum += r[i * COLS];
    put(static_cast<T*>(a.o) + static_cast<int64_t>(bh) * D + c0 + threadIdx.x, a.scale * sum);
  }
}

template <int D, typename T, bool kStates>
static cudaError_t launch_simt(const Passes& ps, int n, cudaStream_t st) {
  static std::atomic<bool> done[kMaxCachedDevices];
  cudaError_t e = allow_smem(simt_pass<D, T, kStates>, Smem<D>::BYTES, done);
  if (e != cudaSuccess) return e;
  const dim3 grid(ps.p[0].nseg - (kStates && !ps.p[0].end ? 1 : 0), ps.p[0].B * ps.p[0].H, n);
  return launch_early(simt_pass<D, T, kStates>, grid, kThreads, Smem<D>::BYTES, st, ps);
}

template <bool kStates>
static cudaError_t simt(const Passes& p, int n, int D, int dtype, cudaStream_t st) {
  if (D == 64)
    return dtype == SCA_BF16 ? launch_simt<64, __nv_bfloat16, kStates>(p, n, st) : launch_simt<64, float, kStates>(p, n, st);
  return dtype == SCA_BF16 ? launch_simt<128, __nv_bfloat16, kStates>(p, n, st)
                           : launch_simt<128, float, kStates>(p, n, st);
}

// Segments per sequence.  A CTA takes one segment and one CTA runs per SM (in
// fp32 arithmetic at D = 64 three fit; the rule does not count on that).
// In units of one chunk of the main pass, a wave of CTAs takes its chunks and
// about two for its start and end; with more than one segment the sums take
// 0.6 a chunk and 1.5 a wave before that, and the scan 1.5 and 0.1 a segment.
// The number of segments with the least such time is taken, up to two CTAs
// per SM.
static int64_t most_segments(int64_t BH, int64_t S, int blk, int sms) {
  const int64_t chunks = (S + blk - 1) / blk, fill = 2 * sms / BH;
  return chunks < fill ? chunks : (fill < 1 ? 1 : fill);
}
static int segments(int64_t BH, int64_t S, int blk, int sms) {
  const int64_t chunks = (S + blk - 1) / blk, most = most_segments(BH, S, blk, sms);
  int best = 1;
  double best_t = 0;
  for (int64_t want = 1; want <= most; ++want) {
    const int64_t per = (chunks + want - 1) / want;
    if ((chunks + per - 1) / per != want) continue;      // the last would be empty
    double t = static_cast<double>((BH * want + sms - 1) / sms) * (per + 2.0);
    if (want > 1) t += static_cast<double>((BH * want + sms - 1) / sms) * (0.6 * per + 1.5) + 1.5 + 0.1 * want;
    if (want == 1 || t < best_t) {
      best_t = t;
      best = static_cast<int>(want);
    }
  }
  return best;
}

struct Cut {
  int nseg;
  int64_t seg_rows;
};
static bool use_tc(const sca_decay_dims* d) {
  return d->dtype == SCA_BF16 && d->algo != SCA_ALGO_SIMT;
}
static Cut cut(const sca_decay_dims* d) {
  const int blk = use_tc(d) ? kDecaySub : kBlk;
  const int64_t chunks = (d->S + blk - 1) / blk;
  Cut c;
  c.nseg = segments(static_cast<int64_t>(d->B) * d->H, d->S, blk, sm_count());
  c.seg_rows = (chunks + c.nseg - 1) / c.nseg * blk;
  return c;
}

static int64_t seg_floats(const sca_decay_dims* d, const Cut& c) {
  return c.nseg == 1 ? 0 : static_cast<int64_t>(d->B) * d->H * c.nseg * d->D * d->D;
}

static int check_view(const sca_view& v, int mult, int D, const char* who, const char* what) {
  SCA_REQUIRE(v.b >= 0 && v.h >= 0 && v.s >= D, SCA_ERR_ARG, "%s: %s strides must be >= 0 and the row stride >= D", who,
              what);
  SCA_REQUIRE(v.b % mult == 0 && v.h % mult == 0 && v.s % mult == 0, SCA_ERR_ALIGN,
              "%s: %s strides must be multiples of %d elements", who, what, mult);
  return SCA_OK;
}

static int check_dims(const sca_decay_dims* d, bool rows, const char* who) {
  SCA_REQUIRE(d != nullptr, SCA_ERR_ARG, "%s: dims is NULL", who);
  SCA_REQUIRE(d->B >= 1 && d->H >= 1 && static_cast<int64_t>(d->B) * d->H <= 65535, SCA_ERR_ARG,
              "%s: B=%d, H=%d: need B, H >= 1 and B*H <= 65535", who, d->B, d->H);
  SCA_REQUIRE(d->D == 64 || d->D == 128, SCA_ERR_UNSUPPORTED, "%s: D=%d: only 64 and 128", who, d->D);
  SCA_REQUIRE(d->dtype == SCA_BF16 || d->dtype == SCA_F32, SCA_ERR_ARG, "%s: dtype=%d unknown", who, d->dtype);
  SCA_REQUIRE(d->algo >= SCA_ALGO_AUTO && d->algo <= SCA_ALGO_TC, SCA_ERR_ARG, "%s: algo=%d unknown", who, d->algo);
  SCA_REQUIRE(d->dtype == SCA_BF16 || d->algo != SCA_ALGO_TC, SCA_ERR_UNSUPPORTED,
              "%s: the tensor-core kernels take bf16 inputs only", who);
  SCA_REQUIRE(std::isfinite(d->scale), SCA_ERR_ARG, "%s: scale is not finite", who);
  const int mult = d->dtype == SCA_BF16 ? 8 : 4;
  int rc;
  sca_view q = d->q, k = d->k, v = d->v;
  if (!rows) q.s = k.s = v.s = d->D;   // a step's tensors have no row axis
  if ((rc = check_view(q, mult, d->D, who, "q")) != SCA_OK) return rc;
  if ((rc = check_view(k, mult, d->D, who, "k")) != SCA_OK) return rc;
  if ((rc = check_view(v, mult, d->D, who, "v")) != SCA_OK) return rc;
  if (!rows) return SCA_OK;
  SCA_REQUIRE(d->S >= 1 && d->S < (1LL << 24), SCA_ERR_ARG, "%s: S=%lld outside [1, 2^24)", who,
              static_cast<long long>(d->S));
  return check_view(d->o, mult, d->D, who, "o");
}

static bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uintptr_t>(bn) && y < x + static_cast<uintptr_t>(an);
}

static DecayPass common(const sca_decay_dims* d, const Cut& c, const float* log_decay, const int32_t* lengths,
                        int* status) {
  DecayPass p = {};
  p.log_decay = log_decay;
  p.lengths = lengths;
  p.S = d->S;
  p.B = d->B;
  p.H = d->H;
  p.nseg = c.nseg;
  p.seg_rows = c.seg_rows;
  p.ov = {d->o.b, d->o.h, d->o.s};
  p.so = d->scale;
  p.status = status;
  return p;
}

static View view_of(const sca_view& v) { return {v.b, v.h, v.s}; }

static int one_pass(const DecayPass& p, const sca_decay_dims* d, bool states, cudaStream_t st, const char* who) {
  if (use_tc(d)) return decay_tc_pass(p, d->D, states, st);
  Passes one = {};
  one.p[0] = p;
  return cuda_status(states ? simt<true>(one, 1, d->D, d->dtype, st) : simt<false>(one, 1, d->D, d->dtype, st), who);
}

// the states before the segments of pass p, into p.seg
static int seg_states(const DecayPass& p, const sca_decay_dims* d, cudaStream_t st, const char* who) {
  const int rc = one_pass(p, d, true, st, who);
  if (rc != SCA_OK) return rc;
  return cuda_status(launch_early(seg_scan_kernel, dim3(d->D * d->D / 256, p.B * p.H), 256, 0, st, p), who);
}

static DecayPass forward_pass(const sca_decay_dims* d, const Cut& c, const void* q, const void* k, const void* v,
                              const float* log_decay, const int32_t* lengths, const float* state_in,
                              int64_t state_in_b, float* ws, int* status) {
  DecayPass p = common(d, c, log_decay, lengths, status);
  p.x = q;
  p.y = k;
  p.z = v;
  p.xv = view_of(d->q);
  p.yv = view_of(d->k);
  p.zv = view_of(d->v);
  p.init = state_in;
  p.init_b = state_in_b;
  p.seg = c.nseg > 1 ? ws : nullptr;
  p.si = d->scale;
  p.us = 1.f;
  p.exact = 1;
  return p;
}

static int check_state(const float* s, int64_t b, const sca_decay_dims* d, const char* who, const char* what) {
  SCA_REQUIRE(aligned(s, 16), SCA_ERR_ALIGN, "%s: %s must be 16-byte aligned", who, what);
  const int64_t one = static_cast<int64_t>(d->H) * d->D * d->D;
  SCA_REQUIRE(!s || b == 0 || b >= one, SCA_ERR_ARG,
              "%s: %s batch stride must be 0 (one state for the batch) or at least H*D*D", who, what);
  SCA_REQUIRE(b % 4 == 0, SCA_ERR_ALIGN, "%s: %s batch stride must be a multiple of 4", who, what);
  return SCA_OK;
}

}  // namespace decay
}  // namespace sca

using namespace sca;
using namespace sca::decay;

extern "C" int decay_attn_workspace(const sca_decay_dims* d, int backward, int64_t* bytes) {
  int rc;
  if ((rc = check_dims(d, true, "decay_attn_workspace")) != SCA_OK) return rc;
  SCA_REQUIRE(bytes != nullptr, SCA_ERR_ARG, "decay_attn_workspace: bytes is NULL");
  // for any number of rows up to S: fewer may be cut into more segments
  Cut c;
  c.nseg = static_cast<int>(most_segments(static_cast<int64_t>(d->B) * d->H, d->S, use_tc(d) ? kDecaySub : kBlk,
                                          sm_count()));
  *bytes = seg_floats(d, c) * 4 * (backward ? 2 : 1);
  return SCA_OK;
}

extern "C" int decay_attn_fwd(const sca_decay_dims* d, const void* q, const void* k, const void* v,
                              const float* log_decay, const int32_t* lengths, const float* state_in,
                              int64_t state_in_b, void* o, float* state_out, float* ws, int64_t ws_bytes,
                              int* dev_status, void* stream) {
  const char* who = "decay_attn_fwd";
  int rc;
  if ((rc = check_dims(d, true, who)) != SCA_OK) return rc;
  SCA_REQUIRE(q && k && v && log_decay && o && state_out, SCA_ERR_ARG, "%s: NULL pointer", who);
  SCA_REQUIRE(aligned(q, 16) && aligned(k, 16) && aligned(v, 16) && aligned(o, 16) && aligned(state_out, 16) &&
                  aligned(ws, 16),
              SCA_ERR_ALIGN, "%s: tensors must be 16-byte aligned", who);
  if ((rc = check_state(state_in, state_in_b, d, who, "state_in")) != SCA_OK) return rc;
  const Cut c = cut(d);
  const int64_t need = seg_floats(d, c) * 4;
  SCA_REQUIRE(need == 0 || (ws && ws_bytes >= need), SCA_ERR_ARG, "%s: workspace of %lld bytes, %lld needed", who,
              static_cast<long long>(ws ? ws_bytes : 0), static_cast<long long>(need));
  // in place (state_out is state_in, one state per sequence) every state is
  // read before it is written; any other overlap is not
  const int64_t one = static_cast<int64_t>(d->H) * d->D * d->D;
  const bool in_place = state_in == state_out && state_in_b == one;
  SCA_REQUIRE(!state_in || in_place ||
                  !overlap(state_in, ((d->B - 1) * state_in_b + one) * 4, state_out, d->B * one * 4),
              SCA_ERR_ARG, "%s: state_out overlaps state_in without being the same states", who);
  DecayPass p = forward_pass(d, c, q, k, v, log_decay, lengths, state_in, state_in_b, ws, dev_status);
  cudaStream_t st = as_stream(stream);
  p.end = state_out;
  if (p.seg) {
    if ((rc = seg_states(p, d, st, who)) != SCA_OK) return rc;
    p.end = nullptr;   // the scan has written it
    p.exact = 0;
  }
  p.out = o;
  return one_pass(p, d, false, st, who);
}

extern "C" int decay_attn_bwd(const sca_decay_dims* d, const void* q, const void* k, const void* v, const void* dout,
                              const sca_view* dout_view, const float* log_decay, const int32_t* lengths,
                              const float* state_in, int64_t state_in_b, const float* dstate_out,
                              int64_t dstate_out_b, void* dq, void* dk, void* dv, float* dstate_in, float* ws,
                              int64_t ws_bytes, int ws_holds_forward, int* dev_status, void* stream) {
  const char* who = "decay_attn_bwd";
  int rc;
  if ((rc = check_dims(d, true, who)) != SCA_OK) return rc;
  SCA_REQUIRE(q && k && v && dout && dout_view && log_decay && dq && dk && dv, SCA_ERR_ARG, "%s: NULL pointer", who);
  SCA_REQUIRE(aligned(q, 16) && aligned(k, 16) && aligned(v, 16) && aligned(dout, 16) && aligned(dq, 16) &&
                  aligned(dk, 16) && aligned(dv, 16) && aligned(dstate_in, 16) && aligned(ws, 16),
              SCA_ERR_ALIGN, "%s: tensors must be 16-byte aligned", who);
  if ((rc = check_view(*dout_view, d->dtype == SCA_BF16 ? 8 : 4, d->D, who, "dout")) != SCA_OK) return rc;
  if ((rc = check_state(state_in, state_in_b, d, who, "state_in")) != SCA_OK) return rc;
  if ((rc = check_state(dstate_out, dstate_out_b, d, who, "dstate_out")) != SCA_OK) return rc;
  const int64_t one = static_cast<int64_t>(d->H) * d->D * d->D;
  SCA_REQUIRE(!dstate_out || !dstate_in ||
                  !overlap(dstate_out, ((d->B - 1) * dstate_out_b + one) * 4, dstate_in, d->B * one * 4),
              SCA_ERR_ARG, "%s: dstate_in overlaps dstate_out", who);
  SCA_REQUIRE(!state_in || !dstate_in ||
                  !overlap(state_in, ((d->B - 1) * state_in_b + one) * 4, dstate_in, d->B * one * 4),
              SCA_ERR_ARG, "%s: dstate_in overlaps state_in", who);
  const Cut c = cut(d);
  const int64_t half = seg_floats(d, c);
  SCA_REQUIRE(half == 0 || (ws && ws_bytes >= 2 * half * 4), SCA_ERR_ARG, "%s: workspace of %lld bytes, %lld needed",
              who, static_cast<long long>(ws ? ws_bytes : 0), static_cast<long long>(2 * half * 4));
  cudaStream_t st = as_stream(stream);
  const View dov = view_of(*dout_view);
  // dq: the forward's states, transposed
  DecayPass p = forward_pass(d, c, q, k, v, log_decay, lengths, state_in, state_in_b, ws, dev_status);
  if (p.seg && !ws_holds_forward && (rc = seg_states(p, d, st, who)) != SCA_OK) return rc;
  p.x = dout;
  p.xv = dov;
  p.y = v;
  p.yv = view_of(d->v);
  p.z = k;
  p.zv = view_of(d->k);
  p.transposed = 1;
  p.exact = 0;
  p.out = dq;
  // dv, and the state's gradient back to the first row
  DecayPass r = common(d, c, log_decay, lengths, dev_status);
  r.reverse = 1;
  r.si = 1.f;
  r.us = d->scale;
  r.exact = dstate_in != nullptr;
  r.init = dstate_out;
  r.init_b = dstate_out_b;
  r.seg = c.nseg > 1 ? ws + half : nullptr;
  r.x = k;
  r.xv = view_of(d->k);
  r.y = q;
  r.yv = view_of(d->q);
  r.z = dout;
  r.zv = dov;
  r.end = dstate_in;
  if (r.seg) {
    if ((rc = seg_states(r, d, st, who)) != SCA_OK) return rc;
    r.end = nullptr;   // the scan has written it
    r.exact = 0;
  }
  r.out = dv;
  // dk: the same states, transposed
  DecayPass t = r;
  t.x = v;
  t.xv = view_of(d->v);
  t.y = dout;
  t.yv = dov;
  t.z = q;
  t.zv = view_of(d->q);
  t.transposed = 1;
  t.exact = 0;
  t.out = dk;
  t.end = nullptr;
  if (use_tc(d)) return decay_tc_backward(p, r, t, d->D, st);
  const Passes all = {{p, r, t}};
  return cuda_status(simt<false>(all, 3, d->D, d->dtype, st), who);
}

extern "C" int decay_attn_step(const sca_decay_dims* d, const void* q, const void* k, const void* v,
                               const float* log_decay, float* state, int64_t state_b, void* o, void* stream) {
  const char* who = "decay_attn_step";
  int rc;
  if ((rc = check_dims(d, false, who)) != SCA_OK) return rc;
  SCA_REQUIRE(q && k && v && log_decay && state && o, SCA_ERR_ARG, "%s: NULL pointer", who);
  SCA_REQUIRE(aligned(q, 16) && aligned(k, 16) && aligned(v, 16) && aligned(o, 16), SCA_ERR_ALIGN,
              "%s: tensors must be 16-byte aligned", who);
  SCA_REQUIRE(d->B == 1 || state_b != 0, SCA_ERR_ARG, "%s: every sequence needs a state of its own (batch stride 0)", who);
  if ((rc = check_state(state, state_b, d, who, "state")) != SCA_OK) return rc;
  const int64_t BH = static_cast<int64_t>(d->B) * d->H;
  // whole states where they fill the SMs by themselves, else slices of 32
  // columns: four CTAs a state (two at D = 64)
  const bool whole = BH >= 2 * sm_count();
  const StepArgs a{q, k, v, view_of(d->q), view_of(d->k), view_of(d->v), log_decay, state, state_b, o, d->H, d->scale};
  cudaStream_t st = as_stream(stream);
  cudaError_t e;
#define SCA_STEP(DD, TT)                                                                            \
  e = whole ? launch_early(step_kernel<DD, TT, DD>, dim3(1, static_cast<unsigned>(BH)), 256, 0, st, a) \
            : launch_early(step_kernel<DD, TT, 32>, dim3(DD / 32, static_cast<unsigned>(BH)), 256, 0, st, a)
  if (d->D == 64 && d->dtype == SCA_BF16) SCA_STEP(64, __nv_bfloat16);
  else if (d->D == 64) SCA_STEP(64, float);
  else if (d->dtype == SCA_BF16) SCA_STEP(128, __nv_bfloat16);
  else SCA_STEP(128, float);
#undef SCA_STEP
  return cuda_status(e, who);
}
