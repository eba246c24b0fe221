// Root-mean-square norm with the residual's addition, also quantized to
// MXFP8, and its backward pass: what stands in front of every MoE layer.
//
// Forward, row by row (d values):
//   r    = x + res, rounded to the layer dtype (the residual stream as the
//          next block reads it); r = x without res
//   rstd = 1 / sqrt(mean(r^2) + eps), from the rounded r, so that a backward
//          pass that reads r differentiates what was computed
//   y    = r * gamma * rstd in fp32, rounded once to the layer dtype
//   codes, scales = MXFP8 of the rounded y: bit for bit what the FP8 expert
//          kernels' own quantizer makes of y.
// Backward, with a = dy * gamma and n = r * rstd:
//   dr     = rstd * (a - n * mean(a n)) + dres, rounded once
//   dgamma = sum over rows of dy * n (fp32 partials of up to 512 workgroups,
//          joined in binary64 in a fixed order, rounded once).
//
// Both passes are bound by HBM: a row is read once, kept in registers and
// written once.  A short row belongs to one wavefront (no LDS, no barrier), a
// longer one to a workgroup of 256 or 1024 threads (norm_shape).  Measured
// (three input sets in turn): forward with MXFP8 output, bf16, 16384 x 6144, 165 to
// 168 us for 909 MB, 5.4 TB/s, where a large copy moves 4.8, fp32, 16384 x 2048, 90 us,
// 5.9 TB/s; backward, bf16, 8192 x 2048, 28 + 5 us for 134 MB.  Calls of a few rows are
// bound by the launch: 1 x 6144 takes 5 us on the card, 7 us to issue.
#include "zc_common.h"

namespace zc {
namespace {

// Sum over the TPR threads of a row; every thread gets it.  Wave butterflies,
// then the wave sums in wave order.
template <int TPR, typename S>
__device__ __forceinline__ S row_sum(S v, S* s_red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  if constexpr (TPR > 64) {
    __syncthreads();  // the previous sum has been read
    if ((threadIdx.x & 63) == 0) s_red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s_red[0];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w) v += s_red[w];
  }
  return v;
}

// m^-1/2 (m > 0): the hardware's fp32 estimate and one Newton step in binary64.
// Every value of the row is scaled by it, so the threads' fp32 sums are joined
// in binary64 too.  m beyond fp32 gives 0, NaN stays NaN; where fp32 would be
// subnormal (eps and the row both next to nothing) all of it runs in binary64.
__device__ __forceinline__ double rsqrt_f64(double m) {
  if (m < 1e-36) return 1.0 / sqrt(m);
  const float e = __frsqrt_rn(static_cast<float>(m));
  if (!(e > 0.f) || isinf(e)) return e;
  const double y = e;
  return y * (1.5 - 0.5 * m * y * y);
}

// MXFP8 of one thread's 8 values of a block of 32 held by 4 consecutive
// lanes.
__device__ __forceinline__ uint64_t mx_quad(const float* f, int& S) {
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[e]));
  amax = fmaxf(amax, __shfl_xor(amax, 1));
  amax = fmaxf(amax, __shfl_xor(amax, 2));
  S = mx_scale(amax);
  uint64_t q = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    q |= static_cast<uint64_t>(mx_code(f[e], S)) << (8 * e);
  }
  return q;
}

template <typename T, int NV, int TPR, bool MX>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_fwd_kernel(
    const T* x, const T* res, const T* __restrict__ gamma, T* r, T* y, float* __restrict__ rstd,
    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t Tn, int d, double inv_d,
    double eps) {
  constexpr int V = V16<T>::n;
  constexpr int RPB = (TPR < 256 ? 256 : TPR) / TPR;
  __shared__ double s_red[TPR / 64];
  const int tid = threadIdx.x % TPR;
  // (beyond kNormGrid workgroups the grid goes round again)
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * RPB + threadIdx.x / TPR; row < Tn;
       row += static_cast<int64_t>(gridDim.x) * RPB) {
  const int64_t base = row * d;
  // all loads of the row first; a vector past its end counts as zeros
  typename V16<T>::raw_t wx[NV], wr[NV], wg[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = (tid + i * TPR) * V;
    wx[i] = j < d ? V16<T>::ld_raw(x + base + j) : typename V16<T>::raw_t{};
  }
  if (res) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = (tid + i * TPR) * V;
      wr[i] = j < d ? V16<T>::ld_raw(res + base + j) : typename V16<T>::raw_t{};
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = (tid + i * TPR) * V;
    wg[i] = j < d ? V16<T>::ld_raw(gamma + j) : typename V16<T>::raw_t{};
  }
  float f[NV][V];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    V16<T>::unpack(wx[i], f[i]);
    if (res) {
      float g[V];
      V16<T>::unpack(wr[i], g);
#pragma unroll
      for (int e = 0; e < V; ++e) f[i][e] = V16<T>::round(f[i][e] + g[e]);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) ss += f[i][e] * f[i][e];
  }
  // r * gamma is exact in fp32 for bf16 rows; times rstd as a sum of two fp32
  // (hi + lo), so that y is rounded once to fp32 and once to its type: a bf16
  // y next to a rounding border, and the codes made of it, seldom cross it.
  // Where r * gamma or y leave fp32 the sum could be inf - inf: there rstd comes
  // first, which gives an infinity, or y where only r * gamma is too large
  const double rd = rsqrt_f64(row_sum<TPR>(static_cast<double>(ss), s_red) * inv_d + eps);
  const float rs = static_cast<float>(rd), rs_lo = static_cast<float>(rd - rs);
  if (rstd && tid == 0) rstd[row] = rs;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = (tid + i * TPR) * V;
    if (j >= d) break;
    float g[V];
    V16<T>::unpack(wg[i], g);
    if (r) V16<T>::store(r + base + j, f[i]);
    float v[V], finite = 0.f;  // NaN with a NaN or an infinity among v
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float p = f[i][e] * g[e];
      v[e] = __builtin_fmaf(p, rs, p * rs_lo);
      finite = __builtin_fmaf(v[e], 0.f, finite);
    }
    if (finite != finite) {  // (16384 x 6144: 166.4 -> 167.9 us; chosen value by value, 171)
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (!(fabsf(v[e]) <= 3.402823466e38f)) v[e] = (f[i][e] * rs) * g[e];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) f[i][e] = V16<T>::round(v[e]);
    V16<T>::store(y + base + j, f[i]);
    if constexpr (MX) {
      int S;
      *reinterpret_cast<uint64_t*>(codes + base + j) = mx_quad(f[i], S);
      // block b of the row; the four scales of 128 values in the order 0 2 1 3
      const int b = j / 32, k = b & 3;
      if ((tid & 3) == 0) scales[base / 32 + (b & ~3) + ((k & 1) << 1 | k >> 1)] = static_cast<uint8_t>(S);
    }
  }
  }
}

// Rows are dealt to nblk workgroups (nblk by T and d alone): workgroup b
// takes rows b * RPB + sub, then every nblk * RPB further, and keeps the
// dgamma sums of its columns in registers.
template <typename T, int NV, int TPR>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_bwd_kernel(
    const T* dy, const T* r, const T* __restrict__ gamma,
    const float* __restrict__ rstd, const T* dres, T* dr, float* __restrict__ part, int64_t Tn,
    int d) {
  constexpr int V = V16<T>::n;
  constexpr int RPB = (TPR < 256 ? 256 : TPR) / TPR;
  __shared__ float s_red[TPR / 64];
  const int tid = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  float acc[NV][V], gm[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = (tid + i * TPR) * V;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[i][e] = 0.f;
    V16<T>::unpack(j < d ? V16<T>::ld_raw(gamma + j) : typename V16<T>::raw_t{}, gm[i]);
  }
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * RPB + sub; row < Tn;
       row += static_cast<int64_t>(gridDim.x) * RPB) {
    const int64_t base = row * d;
    const float rs = rstd[row];
    typename V16<T>::raw_t wa[NV], wn[NV], wg[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = (tid + i * TPR) * V;
      wa[i] = j < d ? V16<T>::ld_raw(dy + base + j) : typename V16<T>::raw_t{};
      wn[i] = j < d ? V16<T>::ld_raw(r + base + j) : typename V16<T>::raw_t{};
      wg[i] = dres && j < d ? V16<T>::ld_raw(dres + base + j) : typename V16<T>::raw_t{};
    }
    float a[NV][V], n[NV][V], s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      V16<T>::unpack(wa[i], a[i]);
      V16<T>::unpack(wn[i], n[i]);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        n[i][e] *= rs;
        acc[i][e] += a[i][e] * n[i][e];
        a[i][e] *= gm[i][e];
        s += a[i][e] * n[i][e];
      }
    }
    const float c = row_sum<TPR>(s, s_red) / static_cast<float>(d);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = (tid + i * TPR) * V;
      if (j >= d) break;
      float g[V];
      V16<T>::unpack(wg[i], g);
#pragma unroll
      for (int e = 0; e < V; ++e) a[i][e] = rs * (a[i][e] - n[i][e] * c) + g[e];
      V16<T>::store(dr + base + j, a[i]);
    }
  }
  if constexpr (RPB > 1) {
    // the workgroup's wavefronts, added in order
    __shared__ float s_acc[RPB - 1][NV * TPR * V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (sub > 0) s_acc[sub - 1][(i * V + e) * TPR + tid] = acc[i][e];
    __syncthreads();
    if (sub > 0) return;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e)
#pragma unroll
        for (int w = 0; w < RPB - 1; ++w) acc[i][e] += s_acc[w][(i * V + e) * TPR + tid];
  }
  float* p = part + static_cast<int64_t>(blockIdx.x) * d;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = (tid + i * TPR) * V;
    if (j >= d) break;
#pragma unroll
    for (int q = 0; q < V / 4; ++q)
      reinterpret_cast<f32x4_t*>(p + j)[q] =
          f32x4_t{acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3]};
  }
}

// dgamma[j] = the np partial rows' column j: 32 groups of consecutive rows,
// each summed ascending, added in group order, all in binary64 (in fp32 the join
// of up to 512 rows costs more than the partials' own sums; it is bound by
// the latency of its loads either way).  32 columns a workgroup, and 16 loads go
// out at once a thread.
constexpr int kRedCols = 32, kRedGroups = 32;
template <typename T>
__global__ __launch_bounds__(kRedCols * kRedGroups) void norm_dgamma_kernel(
    const float* __restrict__ part, int np, int d, T* __restrict__ dgamma) {
  __shared__ double s_p[kRedGroups][kRedCols];
  const int c = threadIdx.x % kRedCols, g = threadIdx.x / kRedCols;
  const int j = blockIdx.x * kRedCols + c;
  const int per = (np + kRedGroups - 1) / kRedGroups;
  const int hi = j < d ? min(np, (g + 1) * per) : 0;
  double v = 0.0;
  for (int b0 = g * per; b0 < hi; b0 += 16) {
    // (past the group its last row again, and not added: with a load behind a
    // branch the compiler widens the value there, and waits for each)
    float w[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) w[u] = part[static_cast<int64_t>(min(b0 + u, hi - 1)) * d + j];
#pragma unroll
    for (int u = 0; u < 16; ++u) v += b0 + u < hi ? static_cast<double>(w[u]) : 0.0;
  }
  s_p[g][c] = v;
  __syncthreads();
  if (g == 0 && j < d) {
#pragma unroll
    for (int k = 1; k < kRedGroups; ++k) v += s_p[k][c];
    Elem<T>::st(dgamma + j, static_cast<float>(v));
  }
}

// A launch holds fewer than 2^32 threads.
constexpr int64_t kNormGrid = int64_t(1) << 20;

// Partial rows of the dgamma sum at most (a call on 8192 rows of 2048 and of 6144,
// three input sets in turn, us: 256 38 and 103, 512 31 and 81, 1024 35 and 91).
constexpr int kNormBlocks = 512;

// One row's threads and vectors per thread: f(NV, TPR) with NV * TPR
// vectors covering the row (d <= kNormMaxD).  By d alone: a row's result does not
// depend on how many others the call has.  Measured, bf16, us; 8192 rows and more as
// calls on three input sets in turn, so that a set is not in the caches from the
// call before, 16 rows and fewer as calls in a graph:
//  - 768 columns on a wavefront against 256 threads: 16 rows 4.4 and 3.6, 8192 rows
//    14.9 and 20.8 (1024 columns 17.6 and 21.4, backward 19.0 and 30.4).
//  - 2048 columns: forward, 16 rows 6.3 and 3.7, 8192 rows 30.0 and 28.2 (1544
//    columns, 32768 rows: 80 and 86); backward, 16 rows 7.2 and 5.3, 8192 rows 30.8
//    and 33.6.  So the forward's wavefronts end at 128 vectors, the backward's,
//    which would join as many more partial rows, at 256.
//  - 4096 columns on 256 threads against a wavefront: 8192 rows, forward 49.7 and
//    67.8, backward 54.2 and 77.1.
//  - 6144 columns (forward with MXFP8) on 256 threads against 512: one row 6.7 and
//    5.6, 16384 rows 165 and 184; against 1024: 6.5 and 5.2, 165 and 184.
template <typename T, bool BWD, typename F>
hipError_t norm_shape(int d, F&& f) {
  const int vecs = (d + V16<T>::n - 1) / V16<T>::n;
  using std::integral_constant;
  if (vecs <= 64) return f(integral_constant<int, 1>{}, integral_constant<int, 64>{});
  if (vecs <= 128) return f(integral_constant<int, 2>{}, integral_constant<int, 64>{});
  if (vecs <= 256) {
    if constexpr (BWD) return f(integral_constant<int, 4>{}, integral_constant<int, 64>{});
    else return f(integral_constant<int, 1>{}, integral_constant<int, 256>{});
  }
  if (vecs <= 512) return f(integral_constant<int, 2>{}, integral_constant<int, 256>{});
  if (vecs <= 768) return f(integral_constant<int, 3>{}, integral_constant<int, 256>{});
  if (vecs <= 1024) return f(integral_constant<int, 4>{}, integral_constant<int, 256>{});
  if (vecs <= 2048) return f(integral_constant<int, 2>{}, integral_constant<int, 1024>{});
  if constexpr (kNormMaxD > 4096 * V16<T>::n)  // (fp32 rows)
    if (vecs > 4096) return f(integral_constant<int, 8>{}, integral_constant<int, 1024>{});
  return f(integral_constant<int, 4>{}, integral_constant<int, 1024>{});
}

int64_t norm_bwd_blocks(int64_t Tn, int rpb) {
  const int64_t b = (Tn + rpb - 1) / rpb;
  return b < kNormBlocks ? b : kNormBlocks;
}

template <typename T>
int norm_rows_per_block(int d) {
  return (d + V16<T>::n - 1) / V16<T>::n <= 256 ? 4 : 1;
}

}  // namespace

template <typename T>
hipError_t launch_norm_fwd(const T* x, const T* res, const T* gamma, T* r, T* y, float* rstd,
                           uint8_t* codes, uint8_t* scales, int64_t Tn, int d, float eps,
                           hipStream_t s) {
  if (Tn == 0) return hipSuccess;
  return norm_shape<T, false>(d, [&](auto nv, auto tpr) {
    constexpr int NV = decltype(nv)::value, TPR = decltype(tpr)::value;
    constexpr int NT = TPR < 256 ? 256 : TPR, RPB = NT / TPR;
    const int64_t blocks = (Tn + RPB - 1) / RPB;
    const dim3 grid(static_cast<unsigned>(blocks < kNormGrid ? blocks : kNormGrid)), block(NT);
    if constexpr (std::is_same<T, bf16_t>::value) {
      if (codes) {
        hipLaunchKernelGGL((norm_fwd_kernel<T, NV, TPR, true>), grid, block, 0, s, x, res, gamma, r,
                           y, rstd, codes, scales, Tn, d, 1.0 / d, static_cast<double>(eps));
        return hipGetLastError();
      }
    }
    hipLaunchKernelGGL((norm_fwd_kernel<T, NV, TPR, false>), grid, block, 0, s, x, res, gamma, r, y,
                       rstd, codes, scales, Tn, d, 1.0 / d, static_cast<double>(eps));
    return hipGetLastError();
  });
}

template <typename T>
int64_t norm_bwd_parts(int64_t Tn, int d) {
  return norm_bwd_blocks(Tn, norm_rows_per_block<T>(d));
}

template <typename T>
hipError_t launch_norm_bwd(const T* dy, const T* r, const T* gamma, const float* rstd,
                           const T* dres, T* dr, T* dgamma, float* part, int64_t Tn, int d,
                           hipStream_t s) {
  const int np = static_cast<int>(norm_bwd_parts<T>(Tn, d));
  if (Tn > 0) {
    const hipError_t e = norm_shape<T, true>(d, [&](auto nv, auto tpr) {
      constexpr int NV = decltype(nv)::value, TPR = decltype(tpr)::value;
      constexpr int NT = TPR < 256 ? 256 : TPR, RPB = NT / TPR;
      hipLaunchKernelGGL((norm_bwd_kernel<T, NV, TPR>),
                         dim3(static_cast<unsigned>(norm_bwd_blocks(Tn, RPB))), dim3(NT), 0, s, dy,
                         r, gamma, rstd, dres, dr, part, Tn, d);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(norm_dgamma_kernel<T>, dim3((d + kRedCols - 1) / kRedCols),
                     dim3(kRedCols * kRedGroups), 0, s, part, np, d, dgamma);
  return hipGetLastError();
}

#define ZC_INST(T)                                                                              \
  template hipError_t launch_norm_fwd<T>(const T*, const T*, const T*, T*, T*, float*, uint8_t*, \
                                         uint8_t*, int64_t, int, float, hipStream_t);           \
  template int64_t norm_bwd_parts<T>(int64_t, int);                                             \
  template hipError_t launch_norm_bwd<T>(const T*, const T*, const T*, const float*, const T*,  \
                                         T*, T*, float*, int64_t, int, hipStream_t);
ZC_INST(bf16_t)
ZC_INST(float)
#undef ZC_INST

}  // namespace zc
