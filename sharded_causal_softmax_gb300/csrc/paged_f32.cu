// Attention of many query rows over a paged cache in fp32: both products from
// shared memory, 64 rows x 64 keys at a time.
//
// 4 D operations a key and row: with more than a dozen rows a head the FMAs bound
// it, not HBM.  A thread holds four rows x four keys of the scores and, of the same
// rows, D / 16 columns of the output: two numbers from shared memory feed
// four FMAs.  The 16 threads of a row are half a warp, so that maxima are
// shuffles and the weights stay in their warp.  Keys and values have two buffers
// each, filled by asynchronous copies a tile ahead, and page numbers are looked up a
// tile before that: one barrier a tile.
//
// Measured: 32 heads' 256 rows, 2000 keys of 128: 261 us, 32 TFLOP/s of about 76 (by
// eights, as in paged.cu, 408), on the 128 SMs that its CTAs fill.  Shared memory bounds
// it: a warp's read of 16 bytes takes three turns there on average, ten reads for 96
// FMAs, 0.73 of its turns and 0.53 of the FMAs'.  Eight rows x four keys a thread
// (64 rows x 128 keys, one buffer each of keys and values) would need twelve reads for 128
// FMAs of the scores instead of eight for 64; not built.
#include "common.cuh"
#include "host_common.h"
#include "launch_util.h"
#include "overlap.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace sca {
namespace paged_f32 {

constexpr int kThreads = 256, MR = 64, KT = 64;

template <int D>
struct Layout {   // in floats
  static constexpr int KS = D + 4, PS = KT + 4;   // rows of queries and keys, and of weights: no two of eight in one bank
  static constexpr int K_OFF = MR * KS;
  static constexpr int V_OFF = K_OFF + 2 * KT * KS;
  static constexpr int P_OFF = V_OFF + 2 * KT * D;
  static constexpr int AT_OFF = P_OFF + MR * PS;          // int64 [2][KT]: where a tile's rows lie, -1: nowhere
  static constexpr int SEE_OFF = AT_OFF + 2 * 2 * KT;     // [MR] what a row sees
  static constexpr int SMEM = (SEE_OFF + 4 * MR) * 4;
  static_assert(SMEM <= 232448 && AT_OFF % 4 == 0, "shared memory");
};

SCA_INLINE void copy16(float* dst, const float* src, bool there) {   // zeros where nothing is
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0)
               : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) rows_f32_kernel(const __grid_constant__ PagedSplit k) {
  using L = Layout<D>;
  constexpr int KS = L::KS, PS = L::PS, V4 = D / 4, C = D / 64;   // C: float4 of output columns a thread
  extern __shared__ __align__(16) float sm[];
  int64_t* const at = reinterpret_cast<int64_t*>(sm + L::AT_OFF);
  Sight* const sees = reinterpret_cast<Sight*>(sm + L::SEE_OFF);
  const PagedArgs& a = k.a;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int b = blockIdx.y / a.Hkv, hk = blockIdx.y - b * a.Hkv;
  const int n = k.splits, rt = blockIdx.x / n, piece = blockIdx.x - rt * n, r0 = rt * MR;
  wait_for_previous();
  const float* const q = static_cast<const float*>(a.q) + b * a.q_b + static_cast<int64_t>(hk) * a.R * D;
  for (int e = tid; e < MR * V4; e += kThreads) {
    const int r = e / V4, c = e % V4;
    const bool there = r0 + r < a.R;
    copy16(sm + r * KS + 4 * c, q + static_cast<int64_t>(there ? r0 + r : 0) * D + 4 * c, there);
  }
  const Held h = held(a, b);
  const int rows = h.cnt ? rows_of(a, h) : 0;
  // tokens in a row see no further than the last of them
  const int last = min(r0 + MR, a.R) - 1;
  const int see = a.tree == nullptr && r0 / a.T == last / a.T ? min(rows, h.len + last % a.T + 1) : rows;
  const int tiles = (see + KT - 1) / KT;
  if (blockIdx.x == 0 && hk == 0 && tid == 0) report_beyond(a, b);
  const int32_t* const table = a.table + b * a.table_b;
  auto entry_of = [&](int tile) {
    const int row = tile * KT + tid;
    return tid < KT && row < rows ? table[row >> a.page_log2] : 0;
  };
  auto put_place = [&](int buf, int tile, int entry) {
    if (tid >= KT) return;
    const int row = tile * KT + tid;
    int64_t x = -1;
    if (row < rows) {
      if (entry >= 0 && entry < a.pages)
        x = static_cast<int64_t>(entry) * a.pool.b + (row & ((1 << a.page_log2) - 1)) * a.pool.s;
      else
        report(a.status, SCA_ERR_RANGE);
    }
    at[buf * KT + tid] = x;
  };
  const float *const kb = static_cast<const float*>(a.kp) + hk * a.pool.h,
              *const vb = static_cast<const float*>(a.vp) + hk * a.pool.h;
  auto load = [&](int buf) {
#pragma unroll
    for (int e = tid; e < KT * V4; e += kThreads) {
      const int r = e / V4, c = 4 * (e % V4);
      const int64_t x = at[buf * KT + r];
      copy16(sm + L::K_OFF + (buf * KT + r) * KS + c, kb + (x < 0 ? 0 : x) + c, x >= 0);
      copy16(sm + L::V_OFF + (buf * KT + r) * D + c, vb + (x < 0 ? 0 : x) + c, x >= 0);
    }
  };
  put_place(0, piece, entry_of(piece));
  put_place(1, piece + n, entry_of(piece + n));
  for (int r = tid; r < MR; r += kThreads) sees[r] = r0 + r < a.R ? sight(a, b, (r0 + r) % a.T, h, rows) : Sight{0, 0};
  __syncthreads();
  if (piece < tiles) load(0);
  float m[4], l[4];
  float4 acc[4][C];
  int least = 0x7fffffff;   // what all rows of this thread see
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
    least = min(least, sees[ty + 16 * i].full);
#pragma unroll
    for (int c = 0; c < C; ++c) acc[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float* const ps = sm + L::P_OFF + ty * PS;
  int buf = 0;
#pragma unroll 1
  for (int tile = piece; tile < tiles; tile += n, buf ^= 1) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();   // the tile is there; nobody uses the other buffers any more
    if (tile + n < tiles) load(buf ^ 1);
    const int entry = entry_of(tile + 2 * n);
    // ---- scores
    float s[4][4] = {};
    const float *const qs = sm + ty * KS, *const ks = sm + L::K_OFF + (buf * KT + tx) * KS;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      float4 x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(qs + 16 * i * KS + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(ks + 16 * j * KS + d);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, s[i][j]))));
    }
    // ---- weights
    const int k0 = tile * KT;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] *= a.scale_log2;
      if (k0 + KT > least) {
        const Sight v = sees[ty + 16 * i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = k0 + tx + 16 * j, off = key - h.len;
          if (!(key < v.full || (off >= 0 && off < 64 && (v.word >> off & 1)))) s[i][j] = -INFINITY;
        }
      }
      float top = fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]));
#pragma unroll
      for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      top = fmaxf(top, m[i]);
      const float sub = top == -INFINITY ? 0.f : top, f = exp2f(m[i] - sub);
      m[i] = top;
      l[i] *= f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float w = exp2f(s[i][j] - sub);
        l[i] += w;
        ps[16 * i * PS + tx + 16 * j] = w;
      }
#pragma unroll
      for (int c = 0; c < C; ++c)
        acc[i][c] = make_float4(acc[i][c].x * f, acc[i][c].y * f, acc[i][c].z * f, acc[i][c].w * f);
    }
    __syncwarp();
    // ---- output
    const float* const vs = sm + L::V_OFF + buf * KT * D + 4 * tx;
#pragma unroll 2
    for (int j = 0; j < KT; j += 4) {
      float w[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(ps + 16 * i * PS + j);
        w[i][0] = x.x;
        w[i][1] = x.y;
        w[i][2] = x.z;
        w[i][3] = x.w;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const float4 v = *reinterpret_cast<const float4*>(vs + (j + e) * D + 64 * c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[i][c].x = fmaf(w[i][e], v.x, acc[i][c].x);
            acc[i][c].y = fmaf(w[i][e], v.y, acc[i][c].y);
            acc[i][c].z = fmaf(w[i][e], v.z, acc[i][c].z);
            acc[i][c].w = fmaf(w[i][e], v.w, acc[i][c].w);
          }
        }
    }
    put_place(buf, tile + 2 * n, entry);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float sum = l[i];
#pragma unroll
    for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int r = r0 + ty + 16 * i;
    if (r >= a.R) continue;
    // no weight: zeros, not 0 times what acc holds (hidden values that are not finite leave NaN there)
    const bool none = sum == 0.f;
    const float f = none ? 0.f : 1.f / sum, lse2 = none ? -INFINITY : m[i] + log2f(sum);
    const int64_t row = static_cast<int64_t>(blockIdx.y) * a.R + r, at_row = n == 1 ? row : row * n + piece;
    float* const o = (n == 1 ? static_cast<float*>(a.o) : k.part_o) + at_row * D + 4 * tx;
#pragma unroll
    for (int c = 0; c < C; ++c)
      *reinterpret_cast<float4*>(o + 64 * c) =
          none ? make_float4(0.f, 0.f, 0.f, 0.f)
               : make_float4(acc[i][c].x * f, acc[i][c].y * f, acc[i][c].z * f, acc[i][c].w * f);
    if (tx == 0) (n == 1 ? a.lse : k.part_lse)[at_row] = n == 1 ? lse2 * kLn2 : lse2;
  }
}

template <int D>
static cudaError_t launch(const PagedSplit& k, cudaStream_t st) {
  static std::atomic<bool> done[kMaxCachedDevices];
  const cudaError_t e = allow_smem(rows_f32_kernel<D>, Layout<D>::SMEM, done);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(k.row_tiles) * k.splits, static_cast<unsigned>(k.a.B) * k.a.Hkv);
  return launch_early(rows_f32_kernel<D>, grid, kThreads, Layout<D>::SMEM, st, k);
}

}  // namespace paged_f32

using namespace paged_f32;

// Pieces of a unit's keys: the number that takes the fewest tiles one after the
// other, of those on the SMs at once and the join's, about two tiles.
PagedSplit paged_f32_cut(const PagedArgs& a, int sms, int* most) {
  PagedSplit k = {};
  k.a = a;
  k.row_tiles = (a.R + MR - 1) / MR;
  const int64_t units = static_cast<int64_t>(a.B) * a.Hkv * k.row_tiles;
  const int64_t tiles = ((static_cast<int64_t>(a.table_n) << a.page_log2) + KT - 1) / KT;
  int64_t n_most = 4ll * sms / units;
  n_most = n_most > kPagedSplits ? kPagedSplits : n_most;
  n_most = n_most > tiles ? tiles : n_most;
  k.splits = 1;
  int64_t best = 0;
  for (int n = 1; n <= n_most || n == 1; ++n) {
    const int64_t cost = (units * n + sms - 1) / sms * ((tiles + n - 1) / n) + (n > 1 ? 2 : 0);
    if (n == 1 || cost < best) {
      best = cost;
      k.splits = n;
    }
  }
  *most = static_cast<int>(n_most < 1 ? 1 : n_most);
  return k;
}

cudaError_t paged_f32_launch(const PagedSplit& k, int D, cudaStream_t st) {
  return D == 64 ? launch<64>(k, st) : launch<128>(k, st);
}

}  // namespace sca
