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
// Passes: picks counted (integer sums, so their order is free), k from the
// counts, the scores' pass, the tokens' q summed in a fixed order.  The
// scores' pass is bound by HBM (4 bytes read and 4 written a score).
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
  double ffn;    // D / K_e
  double zero;   // 1 / (K - K_e), 0 without zero-computation experts
  double alpha;
};

// k_sj of one sequence from its counts (s_hist, in LDS), by the workgroup.
__device__ __forceinline__ void write_coef(const LossCfg& c, const int* s_hist, int* s_group,
                                           int ts, int used, float* __restrict__ coef) {
  const int G = c.N / c.D;
  for (int g = threadIdx.x; g <= c.D; g += blockDim.x) s_group[g] = 0;
  __syncthreads();
  for (int j = threadIdx.x; j < c.E; j += blockDim.x)
    if (s_hist[j]) atomicAdd(s_group + (j < c.N ? j / G : c.D), s_hist[j]);
  __syncthreads();
  const double t = static_cast<double>(ts);
  for (int j = threadIdx.x; j < c.E; j += blockDim.x) {
    double k = 0.0;
    if (ts > 0) {
      const int g = j < c.N ? j / G : c.D;
      const double f = (g < c.D ? c.ffn : c.zero) * static_cast<double>(s_group[g]) / t;
      k = c.alpha * f / (static_cast<double>(used) * t);
    }
    coef[j] = static_cast<float>(k);
  }
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

// Picks of the tokens [lo, hi) into s_hist (LDS or global), valid ones only.
__device__ __forceinline__ void count_picks(const Seqs& q, const int32_t* __restrict__ idx, int K,
                                            int E, int lo, int hi, int* hist) {
  const int64_t b = static_cast<int64_t>(lo) * K;
  const int n = (hi - lo) * K;  // T * K < 2^31
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    if (q.mask && !q.mask[lo + i / K]) continue;
    const int e = idx[b + i];
    if (e >= 0 && e < E) atomicAdd(hist + e, 1);
  }
}

// counts, ts and the two counters behind it to zero (a kernel: a memset node in a
// captured graph would not do)
__global__ void balance_zero_kernel(int32_t* counts, int64_t n, int* ts, int S) {
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = i0; i < n; i += step) counts[i] = 0;
  for (int64_t i = i0; i < S + 2; i += step) ts[i] = 0;
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

// One workgroup counts kChunk tokens: a run of one sequence's tokens in LDS,
// then added to the sequence's counts; a short run straight into them.
// Whoever counts a sequence's first valid token counts the sequence as used.
constexpr int kChunk = 256, kShortRun = 32;
__global__ __launch_bounds__(256) void balance_count_kernel(Seqs q, const int32_t* __restrict__ idx,
                                                            int K, int E, int32_t* counts,
                                                            int* ts, int* used) {
  __shared__ int s_hist[kMaxExperts];
  __shared__ int s_red[4];
  const int c0 = blockIdx.x * kChunk, c1 = min(c0 + kChunk, q.T);
  for (int pos = c0; pos < c1;) {
    const int s = find_seq(q, pos, threadIdx.x & 63);
    if (s >= q.S) break;
    int lo, hi;
    seq_range(q, s, lo, hi);
    lo = max(lo, pos);
    hi = min(hi, c1);
    pos = max(pos + 1, hi);
    if (lo >= hi) continue;
    const int live = valid_tokens(q, lo, hi, s_red);
    if (live == 0) continue;
    if (threadIdx.x == 0 && atomicAdd(ts + s, live) == 0) atomicAdd(used, 1);
    int32_t* row = counts + static_cast<int64_t>(s) * E;
    if (hi - lo < kShortRun) {
      count_picks(q, idx, K, E, lo, hi, row);
      continue;
    }
    __syncthreads();
    for (int j = threadIdx.x; j < E; j += blockDim.x) s_hist[j] = 0;
    __syncthreads();
    count_picks(q, idx, K, E, lo, hi, s_hist);
    __syncthreads();
    for (int j = threadIdx.x; j < E; j += blockDim.x)
      if (s_hist[j]) atomicAdd(row + j, s_hist[j]);
  }
}

__global__ __launch_bounds__(256) void balance_coef_kernel(LossCfg c, const int32_t* counts,
                                                           const int* ts, const int* n_used,
                                                           float* coef, float* seq_scale) {
  __shared__ int s_hist[kMaxExperts], s_group[kMaxExperts + 1];
  const int s = blockIdx.x;
  const int used = *n_used;
  for (int j = threadIdx.x; j < c.E; j += blockDim.x)
    s_hist[j] = counts[static_cast<int64_t>(s) * c.E + j];
  __syncthreads();
  write_coef(c, s_hist, s_group, ts[s], used, coef + static_cast<int64_t>(s) * c.E);
  if (threadIdx.x == 0) seq_scale[s] = static_cast<float>(used);
}

// Small batches: a workgroup counts its whole sequence and writes its counts
// and k at once.  The number of sequences with a valid token is counted by
// every workgroup again.
__global__ __launch_bounds__(kCountThreads) void balance_count_coef_kernel(
    LossCfg c, Seqs q, const int32_t* __restrict__ idx, int32_t* counts, float* coef,
    float* seq_scale, int* arrived) {
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
  write_coef(c, s_hist, s_group, ts, s_used, coef + static_cast<int64_t>(s) * c.E);
  for (int j = threadIdx.x; j < c.E; j += blockDim.x)
    counts[static_cast<int64_t>(s) * c.E + j] = s_hist[j];
  if (threadIdx.x == 0) {
    seq_scale[s] = static_cast<float>(s_used);
    if (s == 0) *arrived = 0;
  }
}

// The scores' pass: a wavefront takes kRun consecutive tokens and keeps its
// sequence's k in registers, NPER slots a lane (E <= 64 NPER).  A token
// that is masked or behind the last sequence gets zeros, whatever it holds.
constexpr int kRun = 4;
template <int NPER>
__global__ __launch_bounds__(64 * kWaves) void balance_scores_kernel(
    Seqs q, const float* __restrict__ logits, int E, const float* __restrict__ coef,
    float* __restrict__ dot, float* __restrict__ dl) {
  const int lane = threadIdx.x & 63;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWaves + (threadIdx.x >> 6)) * kRun;
  if (t0 >= q.T) return;
  const int t1 = static_cast<int>(min(t0 + kRun, static_cast<int64_t>(q.T)));
  int s = find_seq(q, static_cast<int>(t0), lane), have = -1;
  float k[NPER];
  for (int t = static_cast<int>(t0); t < t1; ++t) {
    if (s < q.S && q.cu && q.cu[s + 1] <= t) s = find_seq(q, t, lane);
    const bool live = s < q.S && (!q.cu || q.cu[s] <= t) && (!q.mask || q.mask[t]);
    const int64_t b = static_cast<int64_t>(t) * E;
    if (!live) {
      if (dl)
        for (int j = lane; j < E; j += 64) dl[b + j] = 0.f;
      if (lane == 0) dot[t] = 0.f;
      continue;
    }
    if (s != have) {
#pragma unroll
      for (int i = 0; i < NPER; ++i) {
        const int j = lane + 64 * i;
        k[i] = j < E ? coef[static_cast<int64_t>(s) * E + j] : 0.f;
      }
      have = s;
    }
    float p[NPER], m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      const int j = lane + 64 * i;
      p[i] = j < E ? logits[b + j] : -INFINITY;
      m = fmaxf(m, p[i]);
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    float sum = 0.f, sk = 0.f;
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      const int j = lane + 64 * i;
      p[i] = j < E ? expf(p[i] - m) : 0.f;
      sum += p[i];
      sk += p[i] * k[i];
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      sum += __shfl_xor(sum, o);
      sk += __shfl_xor(sk, o);
    }
    const float inv = 1.0f / sum, qt = sk * inv;
    if (lane == 0) dot[t] = qt;
    if (dl) {
#pragma unroll
      for (int i = 0; i < NPER; ++i) {
        const int j = lane + 64 * i;
        if (j < E) dl[b + j] = (p[i] * inv) * (k[i] - qt);
      }
    }
  }
}

// L_s = S' sum of q_t over the sequence, a workgroup each, in binary64; the
// last workgroup to arrive adds the sequences' sums in order for L.
__global__ __launch_bounds__(kCountThreads) void balance_loss_kernel(
    Seqs q, const float* __restrict__ dot, const float* __restrict__ seq_scale, double* sums,
    int* arrived, float* __restrict__ loss) {
  __shared__ double s_red[kCountThreads / 64];
  __shared__ int s_last;
  const int s = blockIdx.x;
  int lo, hi;
  seq_range(q, s, lo, hi);
  auto total = [&](double v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s_red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
    for (int w = 0; w < kCountThreads / 64; ++w) v += s_red[w];
    return v;
  };
  double v = 0.0;
  for (int t = lo + threadIdx.x; t < hi; t += kCountThreads) v += static_cast<double>(dot[t]);
  v = total(v);
  if (threadIdx.x == 0) {
    loss[1 + s] = static_cast<float>(v * static_cast<double>(seq_scale[s]));
    __hip_atomic_store(sums + s, v, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT);
    s_last = __hip_atomic_fetch_add(arrived, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
             static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (!s_last) return;
  v = 0.0;
  for (int o = threadIdx.x; o < q.S; o += kCountThreads)
    v += __hip_atomic_load(sums + o, __ATOMIC_ACQUIRE, __HIP_MEMORY_SCOPE_AGENT);
  v = total(v);
  if (threadIdx.x == 0) loss[0] = static_cast<float>(v);
}

int64_t up256(int64_t b) { return (b + 255) & ~int64_t(255); }

}  // namespace

// coef [S][E], scale [S], sums [S] (binary64), ts [S] and two counters, dot [T]
size_t seq_balance_scratch_bytes(int64_t Tn, int64_t E, int64_t S) {
  return static_cast<size_t>(up256(4 * S * E) + up256(4 * S) + up256(8 * S) + up256(4 * S + 8) +
                             up256(4 * Tn));
}

hipError_t launch_seq_balance(const float* logits, const int32_t* topk_idx, int Tn, int N, int E,
                              int K, int D, double K_e, double alpha, int S, const int32_t* cu,
                              const uint8_t* mask, float* loss, int32_t* counts, float* dlogits,
                              void* scratch, hipStream_t s) {
  char* p = static_cast<char*>(scratch);
  auto take = [&p](int64_t b) {
    char* r = p;
    p += up256(b);
    return r;
  };
  float* coef = reinterpret_cast<float*>(take(4 * static_cast<int64_t>(S) * E));
  float* scale = reinterpret_cast<float*>(take(4 * static_cast<int64_t>(S)));
  double* sums = reinterpret_cast<double*>(take(8 * static_cast<int64_t>(S)));
  int* ts = reinterpret_cast<int*>(take(4 * static_cast<int64_t>(S) + 8));
  int *used = ts + S, *arrived = used + 1;
  float* dot = reinterpret_cast<float*>(take(4 * static_cast<int64_t>(Tn)));
  const Seqs q{cu, mask, S, Tn};
  const LossCfg c{N, E, K, D, D / K_e, E > N ? 1.0 / (K - K_e) : 0.0, alpha};
  hipError_t e;
  // Few picks: one workgroup a sequence counts them all (at most 64 a thread)
  // and one launch does for three.
  if (static_cast<int64_t>(Tn) * K <= 65536 && S <= 256) {
    hipLaunchKernelGGL(balance_count_coef_kernel, dim3(S), dim3(kCountThreads), 0, s, c, q,
                       topk_idx, counts, coef, scale, arrived);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  } else {
    const int64_t n = static_cast<int64_t>(S) * E;
    const int64_t zb = (n + 1023) / 1024;
    hipLaunchKernelGGL(balance_zero_kernel, dim3(static_cast<unsigned>(zb < 1024 ? zb : 1024)),
                       dim3(256), 0, s, counts, n, ts, S);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(balance_count_kernel, dim3((Tn + kChunk - 1) / kChunk), dim3(256), 0, s, q,
                       topk_idx, K, E, counts, ts, used);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(balance_coef_kernel, dim3(S), dim3(256), 0, s, c, counts, ts, used, coef,
                       scale);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (Tn > 0) {
    const dim3 grid((Tn + kWaves * kRun - 1) / (kWaves * kRun)), block(64 * kWaves);
    const int nper = (E + 63) / 64;
#define ZC_BAL(NP) \
  hipLaunchKernelGGL((balance_scores_kernel<NP>), grid, block, 0, s, q, logits, E, coef, dot, dlogits)
    if (nper <= 1) ZC_BAL(1);
    else if (nper <= 2) ZC_BAL(2);
    else if (nper <= 3) ZC_BAL(3);
    else if (nper <= 4) ZC_BAL(4);
    else if (nper <= 8) ZC_BAL(8);
    else if (nper <= 12) ZC_BAL(12);
    else ZC_BAL(16);
#undef ZC_BAL
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  hipLaunchKernelGGL(balance_loss_kernel, dim3(S), dim3(kCountThreads), 0, s, q, dot, scale, sums,
                     arrived, loss);
  return hipGetLastError();
}

}  // namespace zc
