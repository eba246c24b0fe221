// What follows a backward pass: the norm of all gradients with the factor that
// clips them, and an AdamW step over many tensors, states in 32 or in 8 bits.
//
//   norm   = sqrt(sum of g^2), factor = min(1, max_norm / norm)
//   g'     = factor g
//   m      = b1 m + (1 - b1) g'            v = b2 v + (1 - b2) g'^2
//   p      = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
// all in fp32 (the sum of squares in binary64), each result rounded once to where
// it is kept.
//
// 8-bit states: 128 values share an fp32 scale s = max / 448 (max times 1 / 448 in
// fp32), and a state is an E4M3 code times s; for v the codes are of sqrt(v), which halves the range of
// exponents they have to span, and no positive v becomes 0 (the smallest code
// instead: m / sqrt(v) would leave all bounds).  Rounded to nearest a state moves
// only where a step changes it by half a code's distance, 3 to 6 %, which at b2
// near 1 it hardly ever does; rounded stochastically (down after adding a random
// part of a code's distance) it follows on average.  bf16 weights without an fp32
// copy lose small steps alike and are rounded alike.  The random bits are a
// function of seed, step, tensor and element.
//
// Both are bound by HBM: every array goes through once, nothing is reused.
#include "zc_common.h"

namespace zc {
namespace {

constexpr int kThreads = 256;

// Tensors of one launch, passed by value: nothing has to be copied to the device
// before it, and a captured launch holds them.  As many as the 4 KB of kernel
// arguments take; short lists have a kernel whose arguments are short (the host
// writes all of them: a step of 5 tensors keeps it 6.2 us, with long arguments 7.2).
constexpr int kFew = 8;
constexpr int kArgBytes = 4096;

template <int CAP>
struct NormArgs {
  const void* g[CAP];
  int64_t n[CAP];
  int32_t first[CAP + 1];  // first chunk of each
  int32_t count;
  int32_t chunk;           // elements of a chunk
  double* part;            // a sum for each chunk
};
constexpr int kNormTensors = (kArgBytes - 32) / 20;

// A tensor's pointers: p, g, m, v, with 8-bit states their scales, and the fp32 copy.
enum { T_P = 0, T_G, T_M, T_V, T_MS, T_VS };
template <int NP, int CAP>
struct AdamArgs {
  void* ptr[CAP][NP];
  int64_t n[CAP];
  float decay[CAP];
  int32_t first[CAP + 1];  // first chunk of each
  int32_t count;
  int32_t passes;  // rounds of kThreads vectors in a chunk
  int32_t base;    // number of the first tensor in the whole list
  AdamwScalars s;
};
template <int NP>
constexpr int kAdamTensors = (kArgBytes - 32 - int(sizeof(AdamwScalars))) / (8 * NP + 16);
static_assert(sizeof(NormArgs<kNormTensors>) <= kArgBytes &&
              sizeof(AdamArgs<4, kAdamTensors<4>>) <= kArgBytes &&
              sizeof(AdamArgs<7, kAdamTensors<7>>) <= kArgBytes, "kernel arguments");

// The tensor that chunk b belongs to: the last whose first chunk is not behind b.
template <int CAP>
__device__ __forceinline__ int tensor_of(const int32_t (&first)[CAP], int count, int b) {
  if constexpr (CAP <= kFew + 1) {
    int i = 0;
#pragma unroll
    for (int k = 1; k < CAP - 1; ++k) i += k < count && first[k] <= b;
    return i;
  }
  // (all of them at once: a search would wait for one load after the other, 0.6 us of
  // the 19 us of 4.8 M weights in 61 tensors)
  int i = -1;
#pragma unroll
  for (int k0 = 0; k0 < CAP - 1; k0 += 64) {
    const int k = k0 + (threadIdx.x & 63);
    i += __popcll(__ballot(k < count && first[k < CAP - 1 ? k : 0] <= b));
  }
  return i;
}

// ------------------------------------------------------------------ norm
// Sum over the threads of a workgroup in a fixed order (thread 0 gets it).
template <int NT>
__device__ __forceinline__ double block_sum(double v, double* s_red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) s_red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = s_red[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) v += s_red[w];
  return v;
}

template <typename T, int CAP>
__global__ __launch_bounds__(kThreads) void sqsum_kernel(NormArgs<CAP> a) {
  constexpr int V = V16<T>::n;
  __shared__ double s_red[kThreads / 64];
  const int i = tensor_of(a.first, a.count, blockIdx.x);
  const T* g = static_cast<const T*>(a.g[i]);
  const int64_t n = a.n[i];
  const int64_t begin = static_cast<int64_t>(blockIdx.x - a.first[i]) * a.chunk;
  const int64_t end = begin + a.chunk < n ? begin + a.chunk : n;
  double sum = 0.0;
  int64_t j = begin + threadIdx.x * V;
  for (; j + 3 * kThreads * V + V <= end; j += 4 * kThreads * V) {
    typename V16<T>::raw_t w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) w[u] = V16<T>::ld_raw_once(g + j + u * kThreads * V);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float f[V];
      V16<T>::unpack(w[u], f);
#pragma unroll
      for (int e = 0; e < V; ++e) sum = fma(static_cast<double>(f[e]), static_cast<double>(f[e]), sum);
    }
  }
  for (; j < end; j += kThreads * V) {
    for (int e = 0; e < V && j + e < end; ++e) {
      const double f = Elem<T>::ld(g + j + e);
      sum = fma(f, f, sum);
    }
  }
  sum = block_sum<kThreads>(sum, s_red);
  if (threadIdx.x == 0) a.part[blockIdx.x] = sum;
}

// out = [norm, factor]; one more step where the norm is finite.
__global__ __launch_bounds__(1024) void norm_finish_kernel(const double* __restrict__ part,
                                                           int64_t n, double max_norm,
                                                           float* __restrict__ out,
                                                           int64_t* __restrict__ step) {
  __shared__ double s_red[1024 / 64];
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 1024) sum += part[i];
  sum = block_sum<1024>(sum, s_red);
  if (threadIdx.x != 0) return;
  const double norm = sqrt(sum);
  const bool fine = norm <= 1.7976931348623157e308;
  out[0] = static_cast<float>(norm);
  // (0 stands for a norm that is not finite, not for a small quotient)
  out[1] = !fine ? 0.f : norm > max_norm ? fmaxf(static_cast<float>(max_norm / norm), 0x1p-149f) : 1.f;
  if (step && fine) *step += 1;
}

// ----------------------------------------------------------------- AdamW
// Random bits of a number.  The multipliers here and of the keys are odd constants
// known to spread bits well: the 32-bit primes of the xxHash algorithm, and 2^32 over
// the golden ratio.
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x *= 0x9E3779B1u;
  x ^= x >> 15;
  x *= 0x85EBCA77u;
  return x ^ (x >> 13);
}

// Largest of the 16 lanes of a row (a block of 128 values), in every lane.
__device__ __forceinline__ float row_max(float v) {
  auto turn = [](float f, auto c) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(f), decltype(c)::value, 0xf,
                                                       0xf, true));
  };
  v = fmaxf(v, turn(v, std::integral_constant<int, 0x128>{}));  // row_ror 8, 4, 2, 1
  v = fmaxf(v, turn(v, std::integral_constant<int, 0x124>{}));
  v = fmaxf(v, turn(v, std::integral_constant<int, 0x122>{}));
  return fmaxf(v, turn(v, std::integral_constant<int, 0x121>{}));
}

// a / b with the reciprocal r of b, rounded to nearest, and the remainder of the
// quotient.  a * r is off by 2^-23 of it at most, which the remainder takes away but
// for 2^-46: the nearest number unless a / b lies that close to the middle between two
// (none of 3.5e10 quotients measured was another).
__device__ __forceinline__ float quotient(float a, float b, float r) {
  const float t = a * r;
  return fmaf(fmaf(-t, b, a), r, t);
}

// Square roots of N values, rounded to nearest: from the hardware's estimate of the
// reciprocal root and the root's remainder, sqrt(x) = s + (x - s^2) / (2 s), where
// all x are far from the ends of the exponents (measured for every number there: all
// are the nearest; 8 operations each, where the general
// routine takes some 19: 227 us -> 205 us of 100.7 M weights with 8-bit states).
template <int N>
__device__ __forceinline__ void roots(const float* x, float* r) {
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int e = 1; e < N; ++e) {
    lo = fminf(lo, x[e]);
    hi = fmaxf(hi, x[e]);
  }
  if (__all(lo >= 0x1p-96f && hi <= 0x1p120f)) {  // (a branch of the wavefront's)
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float y = __builtin_amdgcn_rsqf(x[e]), s = x[e] * y;
      r[e] = fmaf(fmaf(-s, s, x[e]), 0.5f * y, s);
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) r[e] = sqrtf(x[e]);
  }
}

// Eight values of a block as codes and the block's scale.  Rounded stochastically
// a value goes down after 16 random bits' part of its distance is added: what the
// hardware's conversion does with them as the upper bits of its operand (measured:
// the same for every exponent, subnormal codes too).  The quotient of the largest
// may be a rounding above 448, 2^-20 of the distance to the next code: less than
// what the random bits lack of 1, and nothing to a rounding to nearest.  ROOT: none
// is negative, and no positive one becomes 0.
template <bool SR, bool ROOT>
__device__ __forceinline__ uint2 encode(const float* f, const uint32_t* noise, float& scale) {
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, ROOT ? f[e] : fabsf(f[e]));
  scale = fmaxf(row_max(amax) * (1.f / 448.f), 0x1p-120f);
  const float inv = 1.f / scale;
  int w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = quotient(f[4 * i + e], scale, inv);
    if constexpr (SR) {
      const uint32_t* z = noise + 4 * i;
      auto bits = [](uint32_t n) { return static_cast<int>(ROOT ? n & 0xffff0000u : n << 16); };
      w[i] = __builtin_amdgcn_cvt_sr_fp8_f32(q[0], bits(z[0]), w[i], 0);
      w[i] = __builtin_amdgcn_cvt_sr_fp8_f32(q[1], bits(z[1]), w[i], 1);
      w[i] = __builtin_amdgcn_cvt_sr_fp8_f32(q[2], bits(z[2]), w[i], 2);
      w[i] = __builtin_amdgcn_cvt_sr_fp8_f32(q[3], bits(z[3]), w[i], 3);
    } else {
      w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
      w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w[i], true);
    }
    // (a byte of zeros somewhere: few blocks, or all zeros)
    if (ROOT && __any(((w[i] - 0x01010101) & ~w[i] & 0x80808080) != 0)) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((w[i] >> (8 * e) & 0xff) == 0 && f[4 * i + e] > 0.f) w[i] |= 1 << (8 * e);
    }
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void decode(uint2 w, float scale, float* f) {
  const uint32_t v[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(v[i], false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(v[i], true);
    f[4 * i] = lo[0] * scale;
    f[4 * i + 1] = lo[1] * scale;
    f[4 * i + 2] = hi[0] * scale;
    f[4 * i + 3] = hi[1] * scale;
  }
}

// W consecutive elements, or the first `left` of them.
template <typename T, int W>
__device__ __forceinline__ void load(const T* p, int left, float* f) {
  if (left >= W) {
    if constexpr (sizeof(T) == 2 && W == 4) {
      const uint2 w = *reinterpret_cast<const uint2*>(p);
      f[0] = __uint_as_float(w.x << 16);
      f[1] = __uint_as_float(w.x & 0xffff0000u);
      f[2] = __uint_as_float(w.y << 16);
      f[3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
#pragma unroll
      for (int i = 0; i < W / V16<T>::n; ++i)
        V16<T>::unpack(V16<T>::ld_raw_once(p + i * V16<T>::n), f + i * V16<T>::n);
    }
  } else {
#pragma unroll
    for (int e = 0; e < W; ++e) f[e] = e < left ? Elem<T>::ld(p + e) : 0.f;
  }
}
// (Nothing that a step writes is read again soon: non-temporal stores, 514 us -> 459 us
// of 100.7 M weights with fp32 copies and states, 213 us -> 205 us with 8-bit ones.)
template <typename T, int W>
__device__ __forceinline__ void store(T* p, int left, const float* f) {
  if (left >= W) {
    if constexpr (sizeof(T) == 2) {
      // (the vector type: the hardware converts two at a time)
      typedef __bf16 bf16w_t __attribute__((ext_vector_type(W)));
      bf16w_t v;
#pragma unroll
      for (int e = 0; e < W; ++e) v[e] = static_cast<__bf16>(f[e]);
      __builtin_nontemporal_store(v, reinterpret_cast<bf16w_t*>(p));
    } else {
#pragma unroll
      for (int i = 0; i < W; i += 4)
        __builtin_nontemporal_store(f32x4_t{f[i], f[i + 1], f[i + 2], f[i + 3]},
                                    reinterpret_cast<f32x4_t*>(p + i));
    }
  } else {
#pragma unroll
    for (int e = 0; e < W; ++e)
      if (e < left) Elem<T>::st(p + e, f[e]);
  }
}
// bf16 weights rounded down after 16 random bits' part of their distance is added:
// the upper half of the sum.  An infinity stays one; a NaN, whose lower bits may be
// set too and carry out of the sum, becomes the one without them.
template <int W>
__device__ __forceinline__ void store_bits(bf16_t* p, int left, const float* f, const uint32_t* add) {
  uint32_t u[W];
#pragma unroll
  for (int e = 0; e < W; ++e) u[e] = __float_as_uint(f[e]) + add[e];
  bool nan = false;
#pragma unroll
  for (int e = 0; e < W; e += 2) nan |= __builtin_isunordered(f[e], f[e + 1]);
  if (__any(nan)) {  // (a branch of the wavefront's)
#pragma unroll
    for (int e = 0; e < W; ++e)
      if (f[e] != f[e]) u[e] = 0x7fc00000u;
  }
  if (left >= W) {
    typedef uint32_t words_t __attribute__((ext_vector_type(W / 2)));
    words_t w;
#pragma unroll
    for (int e = 0; e < W / 2; ++e) w[e] = __builtin_amdgcn_perm(u[2 * e + 1], u[2 * e], 0x07060302u);
    __builtin_nontemporal_store(w, reinterpret_cast<words_t*>(p));
  } else {
#pragma unroll
    for (int e = 0; e < W; ++e)
      if (e < left) p[e] = static_cast<bf16_t>(u[e] >> 16);
  }
}
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int left) {
  if (left >= 8) return *reinterpret_cast<const uint2*>(p);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) w[e / 4] |= static_cast<uint32_t>(p[e]) << (8 * (e % 4));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(uint8_t* p, int left, uint2 c) {
  if (left >= 8) {
    typedef uint32_t words_t __attribute__((ext_vector_type(2)));
    __builtin_nontemporal_store(words_t{c.x, c.y}, reinterpret_cast<words_t*>(p));
    return;
  }
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) p[e] = static_cast<uint8_t>(w[e / 4] >> (8 * (e % 4)));
}

// P weights, G gradients; MASTER: fp32 weights with bf16 copies; B8: 8-bit
// states; SR: stochastic rounding of what has fewer than 32 bits.
template <typename P, typename G, bool MASTER, bool B8, bool SR, int CAP>
__global__ __launch_bounds__(kThreads) void adamw_kernel(
    AdamArgs<(B8 ? 6 : 4) + MASTER, CAP> a) {
  constexpr int W = B8 ? 8 : 4;  // elements of a thread and pass
  constexpr int NP = (B8 ? 6 : 4) + MASTER;
  const AdamwScalars& s = a.s;
  const float factor = s.factor ? *s.factor : 1.f;
  if (factor == 0.f) return;
  const int64_t t = s.step_ptr ? *s.step_ptr : s.step;
  const float lr = s.lr_ptr ? *s.lr_ptr : s.lr;
  // 1 - b^t = -expm1(t log b); the argument in binary64, as t may be large
  const double steps = static_cast<double>(t > 1 ? t : 1);
  const float rate = lr / -expm1f(static_cast<float>(steps * s.log_beta1));
  const float root = 1.f / sqrtf(-expm1f(static_cast<float>(steps * s.log_beta2)));
  const float b1 = s.beta1, c1 = s.rest1, b2 = s.beta2, c2 = s.rest2, eps = s.eps;

  const int i = tensor_of(a.first, a.count, blockIdx.x);
  void* const* ptr = a.ptr[i];
  P* const xp = static_cast<P*>(ptr[T_P]);
  float* const xmaster = MASTER ? static_cast<float*>(ptr[NP - 1]) : nullptr;
  const float keep = 1.f - lr * a.decay[i];
  const int64_t n = a.n[i];
  int64_t j = (static_cast<int64_t>(blockIdx.x - a.first[i]) * a.passes * kThreads + threadIdx.x) * W;
  const uint32_t key0 = (s.seed + 0x9E3779B9u * static_cast<uint32_t>(a.base + i)) ^
                        static_cast<uint32_t>(t) * 0x85EBCA77u;
  for (int pass = 0; pass < a.passes; ++pass, j += kThreads * W) {
    // (a block of 8-bit states lies in one row of lanes: all of it is here, or none)
    if (j >= n && (!B8 || (j & ~int64_t(127)) >= n)) break;
    const int left = j >= n ? 0 : n - j < W ? static_cast<int>(n - j) : W;
    float g[W], p[W], m[W], v[W];
    load<G, W>(static_cast<const G*>(ptr[T_G]) + j, left, g);
    if constexpr (MASTER)
      load<float, W>(xmaster + j, left, p);
    else
      load<P, W>(xp + j, left, p);
    if constexpr (B8) {
      const int64_t blk = j >> 7;
      decode(load_codes(static_cast<const uint8_t*>(ptr[T_M]) + j, left), static_cast<const float*>(ptr[T_MS])[blk], m);
      decode(load_codes(static_cast<const uint8_t*>(ptr[T_V]) + j, left), static_cast<const float*>(ptr[T_VS])[blk], v);
#pragma unroll
      for (int e = 0; e < W; ++e) v[e] *= v[e];
    } else {
      load<float, W>(static_cast<const float*>(ptr[T_M]) + j, left, m);
      load<float, W>(static_cast<const float*>(ptr[T_V]) + j, left, v);
    }
#pragma unroll
    for (int e = 0; e < W; ++e) {
      // (each operation rounded by itself, so that a state does not depend on what
      // the compiler fuses: the codes of two builds are the same)
#pragma clang fp contract(off)
      g[e] *= factor;
      m[e] = b1 * m[e] + c1 * g[e];
      v[e] = b2 * v[e] + c2 * (g[e] * g[e]);
    }
    float r[W];
    roots<W>(v, r);
    // (the hardware's reciprocal, 1 ulp: a rounding or two of the step, which is small
    // beside p)
#pragma unroll
    for (int e = 0; e < W; ++e) {
      const float q = m[e] * __builtin_amdgcn_rcpf(fmaf(r[e], root, eps));
      p[e] = fmaf(-rate, q, p[e] * keep);
    }
    uint32_t noise[W];
    if constexpr (SR) {
      const uint32_t key = key0 + 0xC2B2AE3Du * static_cast<uint32_t>(j >> 32);
#pragma unroll
      for (int e = 0; e < W; ++e) noise[e] = mix((static_cast<uint32_t>(j) ^ key) ^ e);  // j + e = j ^ e
    }
    if constexpr (MASTER) store<float, W>(xmaster + j, left, p);
    if constexpr (SR && sizeof(P) == 2 && !MASTER) {
      uint32_t add[W];
#pragma unroll
      for (int e = 0; e < W; ++e) add[e] = (noise[e] * 0xC2B2AE3Du) >> 16;
      store_bits<W>(xp + j, left, p, add);
    } else {
      store<P, W>(xp + j, left, p);
    }
    if constexpr (B8) {
      const int64_t blk = j >> 7;
      float sm, sv;
      const uint2 cm = encode<SR, false>(m, noise, sm), cv = encode<SR, true>(r, noise, sv);
      store_codes(static_cast<uint8_t*>(ptr[T_M]) + j, left, cm);
      store_codes(static_cast<uint8_t*>(ptr[T_V]) + j, left, cv);
      if ((j & 127) == 0) {
        static_cast<float*>(ptr[T_MS])[blk] = sm;
        static_cast<float*>(ptr[T_VS])[blk] = sv;
      }
    } else {
      store<float, W>(static_cast<float*>(ptr[T_M]) + j, left, m);
      store<float, W>(static_cast<float*>(ptr[T_V]) + j, left, v);
    }
  }
}

// Elements of a chunk of the norm: large ones where there are enough of them for
// the card.
int norm_chunk(int64_t total, bool bf16) {
  const int step = 4 * kThreads * (bf16 ? 8 : 4);
  int c = step;
  while (c < 32 * step && total / (2 * c) >= 2048) c *= 2;
  return c;
}

// Chunks of a launch at most (a launch holds fewer than 2^32 threads).
constexpr int64_t kMaxChunks = int64_t(1) << 23;

// Deals tensors 0 .. count - 1 of n(i) elements to launches: put(k, i) enters tensor
// i as the launch's k-th, go(k) launches k of them.
template <int CAP, typename A, typename N, typename Put, typename Go>
hipError_t deal(A& a, int64_t count, int64_t chunk, N n, Put put, Go go) {
  int k = 0;
  a.first[0] = 0;
  for (int64_t i = 0; i < count; ++i) {
    const int64_t blocks = (n(i) + chunk - 1) / chunk;
    if (k == CAP || (k && a.first[k] + blocks > kMaxChunks)) {
      const hipError_t e = go(k);
      if (e != hipSuccess) return e;
      k = 0;
    }
    put(k, i);
    a.first[k + 1] = static_cast<int32_t>(a.first[k] + blocks);
    ++k;
  }
  return k ? go(k) : hipSuccess;
}

template <typename T, int CAP>
hipError_t norm_parts(const void* const* g, const int64_t* n, int64_t count, int chunk, double* part,
                      int64_t* parts, hipStream_t s) {
  NormArgs<CAP> a;
  a.chunk = chunk;
  *parts = 0;
  return deal<CAP>(
      a, count, chunk, [&](int64_t i) { return n[i]; },
      [&](int k, int64_t i) {
        a.g[k] = g[i];
        a.n[k] = n[i];
      },
      [&](int k) {
        if (a.first[k] == 0) return hipSuccess;
        a.count = k;
        a.part = part + *parts;
        *parts += a.first[k];
        hipLaunchKernelGGL((sqsum_kernel<T, CAP>), dim3(a.first[k]), dim3(kThreads), 0, s, a);
        return hipGetLastError();
      });
}

template <typename P, typename G, bool MASTER, bool B8, bool SR, int CAP>
hipError_t adamw_deal(const AdamwTensor* t, int64_t count, const AdamwScalars& scalars, hipStream_t s) {
  constexpr int NP = (B8 ? 6 : 4) + MASTER, W = B8 ? 8 : 4;
  AdamArgs<NP, CAP> a;
  a.s = scalars;
  int64_t total = 0, most = 0;
  for (int64_t i = 0; i < count; ++i) {
    total += t[i].n;
    most = t[i].n > most ? t[i].n : most;
  }
  // Rounds a workgroup.  32-bit states: one, the loads of many short workgroups overlap
  // best (100.7 M weights with fp32 copies: 458 us; two rounds 496, four 511).  8-bit
  // ones, where the scalars of the step cost as much as a round's loads: up to four while
  // that leaves enough workgroups (205 us; two 214, one 234).  More where a tensor has too many.
  int64_t passes = 1;
  while (B8 && passes < 4 && total / (2 * passes * kThreads * W) >= 4096) passes *= 2;
  while (most / (passes * kThreads * W) >= kMaxChunks) passes *= 2;
  a.passes = static_cast<int32_t>(passes);
  return deal<CAP>(
      a, count, passes * kThreads * W, [&](int64_t i) { return t[i].n; },
      [&](int k, int64_t i) {
        if (k == 0) a.base = static_cast<int32_t>(i);
        void** ptr = a.ptr[k];
        ptr[T_P] = t[i].p;
        ptr[T_G] = const_cast<void*>(t[i].g);
        ptr[T_M] = t[i].m;
        ptr[T_V] = t[i].v;
        if constexpr (B8) {
          ptr[T_MS] = t[i].m_scale;
          ptr[T_VS] = t[i].v_scale;
        }
        if constexpr (MASTER) ptr[NP - 1] = t[i].master;
        a.n[k] = t[i].n;
        a.decay[k] = static_cast<float>(t[i].weight_decay);
      },
      [&](int k) {
        if (a.first[k] == 0) return hipSuccess;
        a.count = k;
        hipLaunchKernelGGL((adamw_kernel<P, G, MASTER, B8, SR, CAP>), dim3(a.first[k]), dim3(kThreads),
                           0, s, a);
        return hipGetLastError();
      });
}
template <typename P, typename G, bool MASTER, bool B8, bool SR>
hipError_t adamw_list(const AdamwTensor* t, int64_t count, const AdamwScalars& c, hipStream_t s) {
  if (count <= kFew) return adamw_deal<P, G, MASTER, B8, SR, kFew>(t, count, c, s);
  return adamw_deal<P, G, MASTER, B8, SR, kAdamTensors<(B8 ? 6 : 4) + MASTER>>(t, count, c, s);
}
template <typename P, typename G, bool MASTER>
hipError_t adamw_kind(bool b8, bool sr, const AdamwTensor* t, int64_t count, const AdamwScalars& c,
                      hipStream_t s) {
  if (b8)
    return sr ? adamw_list<P, G, MASTER, true, true>(t, count, c, s)
              : adamw_list<P, G, MASTER, true, false>(t, count, c, s);
  if constexpr (sizeof(P) == 2 && !MASTER) {
    if (sr) return adamw_list<P, G, MASTER, false, true>(t, count, c, s);
  }  // (else there is nothing to round stochastically)
  return adamw_list<P, G, MASTER, false, false>(t, count, c, s);
}

}  // namespace

int64_t grad_norm_parts(const int64_t* n, int64_t count, bool bf16) {
  int64_t total = 0, parts = 0;
  for (int64_t i = 0; i < count; ++i) total += n[i];
  const int64_t chunk = norm_chunk(total, bf16);
  for (int64_t i = 0; i < count; ++i) parts += (n[i] + chunk - 1) / chunk;
  return parts;
}

hipError_t launch_grad_norm(const void* const* g, const int64_t* n, int64_t count, bool bf16,
                            double max_norm, double* part, float* out, int64_t* step,
                            hipStream_t s) {
  int64_t total = 0, parts = 0;
  for (int64_t i = 0; i < count; ++i) total += n[i];
  const int chunk = norm_chunk(total, bf16);
  hipError_t e;
  if (count <= kFew)
    e = bf16 ? norm_parts<bf16_t, kFew>(g, n, count, chunk, part, &parts, s)
             : norm_parts<float, kFew>(g, n, count, chunk, part, &parts, s);
  else
    e = bf16 ? norm_parts<bf16_t, kNormTensors>(g, n, count, chunk, part, &parts, s)
             : norm_parts<float, kNormTensors>(g, n, count, chunk, part, &parts, s);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(norm_finish_kernel, dim3(1), dim3(1024), 0, s, part, parts, max_norm, out, step);
  return hipGetLastError();
}

hipError_t launch_adamw(const AdamwTensor* t, int64_t count, bool bf16, bool g_bf16, bool master,
                        bool b8, bool sr, const AdamwScalars& c, hipStream_t s) {
  if (!bf16) return adamw_kind<float, float, false>(b8, sr, t, count, c, s);
  if (g_bf16 && master) return adamw_kind<bf16_t, bf16_t, true>(b8, sr, t, count, c, s);
  if (g_bf16) return adamw_kind<bf16_t, bf16_t, false>(b8, sr, t, count, c, s);
  if (master) return adamw_kind<bf16_t, float, true>(b8, sr, t, count, c, s);
  return adamw_kind<bf16_t, float, false>(b8, sr, t, count, c, s);
}

}  // namespace zc
