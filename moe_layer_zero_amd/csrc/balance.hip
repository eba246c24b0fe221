// Balance loss of packed sequences, their per-expert counts and the gradient
// of the router scores.
//
// "LongCat-Flash Technical Report", section 2.1.2, applied to each sequence
// by itself: with T_s the valid tokens of sequence s and c_se its picks of
// expert e among them,
//   f_sg = D / (K_e T_s) * picks in group g       (FFN groups, g < D)
//        = 1 / ((K - K_e) T_s) * picks            (zero-computation experts)
//   L_s  = alpha sum_g f_sg P_sg,  P_sg = mean over valid tokens of the
//          group's softmax mass,
//   L    = mean of L_s over the S' sequences with a valid token.
// f counts discrete picks and has no gradient, so with
//   k_sj = alpha f_sg(j) / (S' T_s)   and   q_t = sum_j p_tj k_sj
// the gradient is dL/dl_tj = p_tj (k_sj - q_t), and the loss itself is
// L = sum_t q_t, L_s = S' sum of q_t over the sequence: one number a token
// that the gradient needs anyway.  No column sums of the softmax, and one
// pass over the scores for loss and gradient together.
//
// k_sj - q_t is a difference of nearly equal numbers in every sequence that is
// close to balance, which is where the loss drives them, and zero in one that
// is balanced.  So what is kept of k is k_sj - k_s0, the difference taken of
// the counts in binary64 (0 exactly where they agree), and the sums over a
// token's scores run in binary64 too:
//   u_t = sum_j e_tj (k_sj - k_s0) / sum_j e_tj,   q_t = k_s0 + u_t,
//   dL/dl_tj = p_tj ((k_sj - k_s0) - u_t).
// The error is then that of the fp32 exponentials e, relative to
// |k_sj - q_t| and the spread of k about q_t: in an emulation of E = 192 scores
// 6e-8 of the gradient at any imbalance, where fp32 k and sums lose 6e-7 at 10%
// and 1e-3 at 0.01%.
//
// Passes: picks counted (integer sums, so their order is free), k from the
// counts, the scores' pass, the tokens' q summed in a fixed order.  The
// scores' pass is bound by HBM (4 bytes read and 4 written a score).  Measured:
// 16381 tokens of 768 scores in 37 sequences, masked: that pass 25 us, 4.0 TB/s
// (the call 40.3 us, 39.2 with k and its sums in fp32), the counts, k and loss 5 to
// 6 us each; at 64 tokens of 12 scores three kernels of 2 to 4 us, less than their
// launches cost the host.
#include "zc_common.h"

namespace zc {
namespace {

constexpr int kWaves = 4;           // wavefronts of the scores' pass
constexpr int kCountThreads = 1024;

struct Seqs {
  const int32_t* cu;    // [S+1], NULL: one sequence of all tokens
  const uint8_t* mask;  // [T], NULL: all valid
  int S, T;
};

// Token range of sequence s; offsets outside [0, T] or descending stay in
// bounds.
__device__ __forceinline__ void seq_range(const Seqs& q, int s, int& lo, int& hi) {
  lo = q.cu ? min(max(q.cu[s], 0), q.T) : 0;
  hi = q.cu ? min(max(q.cu[s + 1], lo), q.T) : q.T;
}

struct LossCfg {
  int N, E, K, D;
  // f = ffn / (den T_s) picks of an FFN group, zero / (den T_s) of the others
  double ffn, zero, den;
  double alpha;
};

// k_sj - k_s0 and k_s0 of one sequence from its counts (s_hist, in LDS), by the
// workgroup.  With Z > 0 both groups' f are brought to the denominator K_e (K -
// K_e) T_s first, so that equal f (of a K_e with few bits) differ by 0.
__device__ __forceinline__ void write_coef(const LossCfg& c, const int* s_hist, int* s_group,
                                           int ts, int used, double* __restrict__ coef,
                                           double* __restrict__ k0) {
#pragma clang fp contract(off)  // (a fused product would differ from the rounded one it is taken from)
  const int G = c.N / c.D;
  for (int g = threadIdx.x; g <= c.D; g += blockDim.x) s_group[g] = 0;
  __syncthreads();
  for (int j = threadIdx.x; j < c.E; j += blockDim.x)
    if (s_hist[j]) atomicAdd(s_group + (j < c.N ? j / G : c.D), s_hist[j]);
  __syncthreads();
  const double t = static_cast<double>(ts);
  const double first = c.ffn * static_cast<double>(s_group[0]);
  const double scale = ts > 0 ? c.alpha / (c.den * static_cast<double>(used) * t * t) : 0.0;
  for (int j = threadIdx.x; j < c.E; j += blockDim.x) {
    const int g = j < c.N ? j / G : c.D;
    coef[j] = scale * ((g < c.D ? c.ffn : c.zero) * static_cast<double>(s_group[g]) - first);
  }
  if (threadIdx.x == 0) *k0 = scale * first;
}

// Integer sum over the workgroup; every thread gets it.
__device__ __forceinline__ int block_sum(int v, int* s_red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s_red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x) / 64; ++w) v += s_red[w];
  return v;
}

__device__ __forceinline__ int valid_tokens(const Seqs& q, int lo, int hi, int* s_red) {
  if (!q.mask) return hi - lo;
  int n = 0;
  for (int t = lo + threadIdx.x; t < hi; t += blockDim.x) n += q.mask[t] != 0;
  return block_sum(n, s_red);
}

// Picks of the tokens [lo, hi) into hist (LDS or global), valid ones only.
// A thread's loads of eight rounds go out together: the pass is otherwise
// one round trip of a pick and its mask byte after another.
__device__ __forceinline__ void count_picks(const Seqs& q, const int32_t* __restrict__ idx, int K,
                                            int E, int lo, int hi, int* hist) {
  const int32_t* row = idx + static_cast<int64_t>(lo) * K;
  const int n = (hi - lo) * K;  // T * K < 2^31
  for (int64_t i0 = threadIdx.x; i0 < n; i0 += 8 * static_cast<int64_t>(blockDim.x)) {
    int e[8], m[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t i = i0 + u * static_cast<int64_t>(blockDim.x);
      e[u] = i < n ? row[i] : -1;
      m[u] = i < n && q.mask ? q.mask[lo + static_cast<uint32_t>(i) / static_cast<uint32_t>(K)] : 1;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (m[u] && e[u] >= 0 && e[u] < E) atomicAdd(hist + e[u], 1);
  }
}

// First sequence whose end lies behind token t, S if none: the number of
// leading ends <= t, searched 64 at a time by the wavefront.
__device__ __forceinline__ int find_seq(const Seqs& q, int t, int lane) {
  if (!q.cu) return 0;
  int lo = 0, hi = q.S;
  while (lo < hi) {
    const int step = (hi - lo + 63) / 64;
    const int i = lo + lane * step;
    const bool before = i < hi && q.cu[min(i, q.S - 1) + 1] <= t;
    const int n = __popcll(__ballot(before));
    if (n == 0) return lo;
    hi = min(lo + n * step, hi);
    lo = lo + (n - 1) * step + 1;
  }
  return lo;
}

// Part p of P of sequence s (workgroup s P + p): its picks of each expert and
// its valid tokens, as a row of their own, so nothing has to be zero before.
__global__ __launch_bounds__(kCountThreads) void balance_count_kernel(
    Seqs q, const int32_t* __restrict__ idx, int K, int E, int P, int32_t* __restrict__ part,
    int* __restrict__ ts) {
  __shared__ int s_hist[kMaxExperts], s_red[kCountThreads / 64];
  const int s = blockIdx.x / P, p = blockIdx.x % P;
  int lo, hi;
  seq_range(q, s, lo, hi);
  const int64_t len = hi - lo;
  hi = lo + static_cast<int>(len * (p + 1) / P);
  lo = lo + static_cast<int>(len * p / P);
  for (int j = threadIdx.x; j < E; j += blockDim.x) s_hist[j] = 0;
  __syncthreads();
  const int live = valid_tokens(q, lo, hi, s_red);
  if (live) count_picks(q, idx, K, E, lo, hi, s_hist);
  __syncthreads();
  for (int j = threadIdx.x; j < E; j += blockDim.x)
    part[static_cast<int64_t>(blockIdx.x) * E + j] = s_hist[j];
  if (threadIdx.x == 0) ts[blockIdx.x] = live;
}

// Sequences among [0, S) with a valid token, and those of sequence mine, from
// the parts' token counts (P > 1 only with S <= kMaxSplit).
constexpr int kMaxSplit = 128;
__device__ __forceinline__ int count_used(const int* ts, int S, int P, int mine, int* s_red,
                                          int& live) {
  __shared__ int s_live[kMaxSplit];
  int n = 0;
  if (P == 1) {
    for (int s = threadIdx.x; s < S; s += blockDim.x) n += ts[s] != 0;
    live = ts[mine];
    return block_sum(n, s_red);
  }
  if (threadIdx.x < kMaxSplit) s_live[threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < S * P; i += blockDim.x) atomicAdd(s_live + i / P, ts[i]);
  __syncthreads();
  live = s_live[mine];
  return block_sum(threadIdx.x < static_cast<unsigned>(S) && s_live[threadIdx.x] != 0, s_red);
}
__global__ __launch_bounds__(kCountThreads) void balance_used_kernel(const int* ts, int S,
                                                                     int* used) {
  __shared__ int s_red[kCountThreads / 64];
  int live;
  const int n = count_used(ts, S, 1, 0, s_red, live);
  if (threadIdx.x == 0) *used = n;
}

// Counts and k of a sequence from its parts.  n_used: the sequences with a
// valid token, NULL to count them here.
__global__ __launch_bounds__(kCountThreads) void balance_coef_kernel(
    LossCfg c, int S, int P, const int32_t* __restrict__ part, const int* __restrict__ ts,
    const int* __restrict__ n_used, int32_t* __restrict__ counts, double* __restrict__ coef,
    double* __restrict__ k0, float* __restrict__ seq_scale) {
  __shared__ int s_hist[kMaxExperts], s_group[kMaxExperts + 1], s_red[kCountThreads / 64];
  const int s = blockIdx.x;
  int live, used;
  if (n_used) {
    used = *n_used;
    live = ts[s];  // P == 1
  } else {
    used = count_used(ts, S, P, s, s_red, live);
  }
  const int64_t row = static_cast<int64_t>(s) * P * c.E;
  for (int j = threadIdx.x; j < c.E; j += blockDim.x) {
    int n = 0;
    for (int p0 = 0; p0 < P; p0 += 16) {
      int w[16];
#pragma unroll
      for (int u = 0; u < 16; ++u)
        w[u] = p0 + u < P ? part[row + static_cast<int64_t>(p0 + u) * c.E + j] : 0;
#pragma unroll
      for (int u = 0; u < 16; ++u) n += w[u];
    }
    s_hist[j] = n;
    counts[static_cast<int64_t>(s) * c.E + j] = n;
  }
  __syncthreads();
  write_coef(c, s_hist, s_group, live, used, coef + static_cast<int64_t>(s) * c.E, k0 + s);
  if (threadIdx.x == 0) seq_scale[s] = static_cast<float>(used);
}

// Small batches: a workgroup counts its whole sequence and writes its counts
// and k at once.  The number of sequences with a valid token is counted by
// every workgroup again.
__global__ __launch_bounds__(kCountThreads) void balance_count_coef_kernel(
    LossCfg c, Seqs q, const int32_t* __restrict__ idx, int32_t* counts, double* coef, double* k0,
    float* seq_scale) {
  __shared__ int s_hist[kMaxExperts], s_group[kMaxExperts + 1], s_red[kCountThreads / 64], s_used;
  const int s = blockIdx.x, lane = threadIdx.x & 63;
  if (threadIdx.x == 0) s_used = 0;
  for (int j = threadIdx.x; j < c.E; j += blockDim.x) s_hist[j] = 0;
  __syncthreads();
  // wavefronts share the sequences out
  int mine = 0;
  for (int o = threadIdx.x >> 6; o < q.S; o += kCountThreads / 64) {
    int lo, hi;
    seq_range(q, o, lo, hi);
    bool any = !q.mask && hi > lo;
    for (int t = lo; q.mask && t < hi && !any; t += 64)
      any = __any(t + lane < hi && q.mask[min(t + lane, q.T - 1)] != 0);
    mine += any;
  }
  if (lane == 0 && mine) atomicAdd(&s_used, mine);
  int lo, hi;
  seq_range(q, s, lo, hi);
  const int ts = valid_tokens(q, lo, hi, s_red);
  count_picks(q, idx, c.K, c.E, lo, hi, s_hist);
  __syncthreads();
  write_coef(c, s_hist, s_group, ts, s_used, coef + static_cast<int64_t>(s) * c.E, k0 + s);
  for (int j = threadIdx.x; j < c.E; j += blockDim.x)
    counts[static_cast<int64_t>(s) * c.E + j] = s_hist[j];
  if (threadIdx.x == 0) seq_scale[s] = static_cast<float>(s_used);
}

// The scores' pass: a wavefront per token, NV pieces of VEC scores a lane
// (E <= 64 NV VEC, E a multiple of VEC).  The row's loads go out before its
// sequence is looked up.  A token that is masked or behind the last sequence
// gets zeros, whatever it holds.
template <int NV, int VEC>
__global__ __launch_bounds__(64 * kWaves) void balance_scores_kernel(
    Seqs q, const float* __restrict__ logits, int E, const double* __restrict__ coef,
    const double* __restrict__ k0, float* __restrict__ dot, float* __restrict__ dl) {
  typedef float vec_t __attribute__((ext_vector_type(VEC)));
  typedef double dvec_t __attribute__((ext_vector_type(VEC)));
  const int lane = threadIdx.x & 63;
  const int64_t tt = static_cast<int64_t>(blockIdx.x) * kWaves + (threadIdx.x >> 6);
  if (tt >= q.T) return;
  const int t = static_cast<int>(tt), n = E / VEC;
  const vec_t* row = reinterpret_cast<const vec_t*>(logits + tt * E);
  vec_t* out = reinterpret_cast<vec_t*>(dl + tt * E);
  vec_t p[NV];
  dvec_t k[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = lane + 64 * i;
    p[i] = j < n ? row[j] : vec_t(-INFINITY);
  }
  const bool valid = !q.mask || q.mask[t];
  const int s = find_seq(q, t, lane);
  if (!valid || s >= q.S || (q.cu && q.cu[s] > t)) {
    if (dl)
      for (int j = lane; j < n; j += 64) out[j] = vec_t(0.f);
    if (lane == 0) dot[t] = 0.f;
    return;
  }
  const dvec_t* kr = reinterpret_cast<const dvec_t*>(coef + static_cast<int64_t>(s) * E);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = lane + 64 * i;
    k[i] = j < n ? kr[j] : dvec_t(0.0);
  }
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) m = fmaxf(m, p[i][e]);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  double sum = 0.0, sk = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      p[i][e] = lane + 64 * i < n ? expf(p[i][e] - m) : 0.f;
      sum += static_cast<double>(p[i][e]);
      sk += static_cast<double>(p[i][e]) * k[i][e];
    }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    sum += __shfl_xor(sum, o);
    sk += __shfl_xor(sk, o);
  }
  const float inv = 1.0f / static_cast<float>(sum);
  const double u = sk / sum;
  if (lane == 0) dot[t] = static_cast<float>(k0[s] + u);
  if (dl) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = lane + 64 * i;
      vec_t v;
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = (p[i][e] * inv) * static_cast<float>(k[i][e] - u);
      if (j < n) out[j] = v;
    }
  }
}

// Workgroup s: L_s = S' sum of q_t over its sequence; workgroup S: L, the sum
// over all tokens (q_t is 0 where none counts).  Binary64, each thread its
// tokens ascending, eight loads at a time, then a fixed tree.
__global__ __launch_bounds__(kCountThreads) void balance_loss_kernel(
    Seqs q, const float* __restrict__ dot, const float* __restrict__ seq_scale,
    float* __restrict__ loss) {
  __shared__ double s_red[kCountThreads / 64];
  const int s = blockIdx.x;
  int lo = 0, hi = q.T;
  double scale = 1.0;
  if (s < q.S) {
    seq_range(q, s, lo, hi);
    scale = static_cast<double>(seq_scale[s]);
  }
  double v = 0.0;
  for (int64_t t0 = lo + static_cast<int64_t>(threadIdx.x); t0 < hi; t0 += 8 * kCountThreads) {
    float w[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) w[u] = t0 + u * kCountThreads < hi ? dot[t0 + u * kCountThreads] : 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) v += static_cast<double>(w[u]);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) s_red[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x != 0) return;
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kCountThreads / 64; ++w) v += s_red[w];
  loss[s < q.S ? 1 + s : 0] = static_cast<float>(v * scale);
}

int64_t up256(int64_t b) { return (b + 255) & ~int64_t(255); }

// Parts a sequence is counted in: about 256 workgroups in all, at most 64 a
// sequence (their rows are added by one workgroup) and at least 8192 picks each,
// if every sequence were the average one (one sequence of 1024 tokens, K = 8:
// 9.5 us, with parts of 1024 picks 12.8; 16384 tokens, K = 12: 35 and 36, 55 in
// one part).  But enough that a sequence which holds the whole batch, the
// others empty, is counted in parts of at most 32768
// (16381 tokens in 37 ragged sequences, K = 12, the call: 39.1 us, with 65536 41.2).
int count_parts(int64_t Tn, int64_t K, int64_t S) {
  if (S > kMaxSplit) return 1;
  const int64_t even = Tn * K / (8192 * S), least = (Tn * K + 32767) / 32768;
  int64_t p = 256 / S < even ? 256 / S : even;
  if (p < least) p = least;
  return p < 1 ? 1 : p > 64 ? 64 : static_cast<int>(p);
}

}  // namespace

// coef [S][E] and k_s0 [S] (binary64), scale [S], parts' counts [S][P][E] and
// tokens [S][P], the number of used sequences, dot [T]
size_t seq_balance_scratch_bytes(int64_t Tn, int64_t E, int64_t K, int64_t S) {
  const int64_t P = count_parts(Tn, K, S);
  return static_cast<size_t>(up256(8 * S * E) + up256(8 * S) + up256(4 * S) +
                             up256(4 * S * P * E) + up256(4 * S * P + 4) + up256(4 * Tn));
}

hipError_t launch_seq_balance(const float* logits, const int32_t* topk_idx, int Tn, int N, int E,
                              int K, int D, double K_e, double alpha, int S, const int32_t* cu,
                              const uint8_t* mask, float* loss, int32_t* counts, float* dlogits,
                              void* scratch, hipStream_t s) {
  const int P = count_parts(Tn, K, S);
  const int64_t rows = static_cast<int64_t>(S) * P;
  char* p = static_cast<char*>(scratch);
  auto take = [&p](int64_t b) {
    char* r = p;
    p += up256(b);
    return r;
  };
  double* coef = reinterpret_cast<double*>(take(8 * static_cast<int64_t>(S) * E));
  double* k0 = reinterpret_cast<double*>(take(8 * static_cast<int64_t>(S)));
  float* scale = reinterpret_cast<float*>(take(4 * static_cast<int64_t>(S)));
  int32_t* part = reinterpret_cast<int32_t*>(take(4 * rows * E));
  int* ts = reinterpret_cast<int*>(take(4 * rows + 4));
  int* used = ts + rows;
  float* dot = reinterpret_cast<float*>(take(4 * static_cast<int64_t>(Tn)));
  const Seqs q{cu, mask, S, Tn};
  const bool z = E > N;
  const LossCfg c{N, E, K, D, z ? D * (K - K_e) : D, z ? K_e : 0.0, z ? K_e * (K - K_e) : K_e, alpha};
  hipError_t e;
  // Sequences not split: one workgroup each counts the picks and writes k at once
  // (1024 tokens, 32 sequences: 9.7 us, two launches 12.8; 256 sequences 13.5 and
  // 14.7; 1024, each looking through all: 45 and 27).
  if (P == 1 && S <= 256) {
    hipLaunchKernelGGL(balance_count_coef_kernel, dim3(S), dim3(kCountThreads), 0, s, c, q,
                       topk_idx, counts, coef, k0, scale);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  } else {
    hipLaunchKernelGGL(balance_count_kernel, dim3(static_cast<unsigned>(rows)),
                       dim3(kCountThreads), 0, s, q, topk_idx, K, E, P, part, ts);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    // from 1024 sequences on a workgroup's own count of the used ones costs more
    // than a launch (512: 19.3 us, apart 20.1; 1024: 27.0 and 26.5; 4096: 80 and 68)
    const bool apart = S >= 1024;
    if (apart) {
      hipLaunchKernelGGL(balance_used_kernel, dim3(1), dim3(kCountThreads), 0, s, ts, S, used);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    hipLaunchKernelGGL(balance_coef_kernel, dim3(S), dim3(kCountThreads), 0, s, c, S, P, part, ts,
                       apart ? used : nullptr, counts, coef, k0, scale);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (Tn > 0) {
    const dim3 grid((Tn + kWaves - 1) / kWaves), block(64 * kWaves);
#define ZC_BAL(NV, VEC)                                                                            \
  hipLaunchKernelGGL((balance_scores_kernel<NV, VEC>), grid, block, 0, s, q, logits, E, coef, k0, \
                     dot, dlogits)
    if (E % 4 == 0) {
      if (E <= 256) ZC_BAL(1, 4);
      else if (E <= 512) ZC_BAL(2, 4);
      else if (E <= 768) ZC_BAL(3, 4);
      else ZC_BAL(4, 4);
    } else {
      if (E <= 64) ZC_BAL(1, 1);
      else if (E <= 128) ZC_BAL(2, 1);
      else if (E <= 256) ZC_BAL(4, 1);
      else if (E <= 512) ZC_BAL(8, 1);
      else ZC_BAL(16, 1);
    }
#undef ZC_BAL
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  hipLaunchKernelGGL(balance_loss_kernel, dim3(S + 1), dim3(kCountThreads), 0, s, q, dot, scale,
                     loss);
  return hipGetLastError();
}

}  // namespace zc
