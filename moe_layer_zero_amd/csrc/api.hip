// C ABI of libzcmoe: argument checks, workspace carving and the launch
// sequence of each entry point.  See include/zc_moe.h for the contract.
#include <algorithm>
#include <atomic>
#include <cstdarg>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>
#include <type_traits>
#include <vector>

#include "../../include/zc_moe.h"
#include "zc_common.h"

using zc::bf16_t;

namespace {

thread_local std::string g_last_error;

zc_status fail(zc_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
zc_status fail(zc_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return s;
}

zc_status hip_fail(hipError_t e, const char* what) {
  return fail(ZC_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

#define ZC_HIP(call, what)                           \
  do {                                               \
    hipError_t e_ = (call);                          \
    if (e_ != hipSuccess) return hip_fail(e_, what); \
  } while (0)

// ---- optional per-phase kernel timing (zc_moe_profile)
struct PhaseRec {
  int phase;
  hipEvent_t a, b;
};
std::mutex g_prof_mu;
std::atomic<bool> g_prof_on{false};
std::vector<PhaseRec> g_prof_recs;

// Set while the calling thread runs the allocation-free forward: its
// launches record no timing events (creating an event may allocate).
thread_local bool t_no_events = false;

// Records a start event on construction and an end event in done(), on the
// stream of the launch, when profiling is on.
class PhaseScope {
 public:
  PhaseScope(int phase, hipStream_t s) : phase_(phase), s_(s) {
    if (!t_no_events && g_prof_on.load(std::memory_order_relaxed) &&
        hipEventCreate(&a_) == hipSuccess)
      (void)hipEventRecord(a_, s_);
    else
      a_ = nullptr;
  }
  void done() {
    if (!a_) return;
    hipEvent_t b = nullptr;
    if (hipEventCreate(&b) != hipSuccess) {
      (void)hipEventDestroy(a_);
      return;
    }
    (void)hipEventRecord(b, s_);
    std::lock_guard<std::mutex> lk(g_prof_mu);
    g_prof_recs.push_back(PhaseRec{phase_, a_, b});
  }

 private:
  int phase_;
  hipStream_t s_;
  hipEvent_t a_;
};

#define ZC_LAUNCH(phase, call, what)                 \
  do {                                               \
    PhaseScope ps_((phase), s);                      \
    hipError_t e_ = (call);                          \
    ps_.done();                                      \
    if (e_ != hipSuccess) return hip_fail(e_, what); \
  } while (0)

void drop_records() {
  for (auto& r : g_prof_recs) {
    (void)hipEventDestroy(r.a);
    (void)hipEventDestroy(r.b);
  }
  g_prof_recs.clear();
}

// Compute-unit count of the current device, cached per device.
std::atomic<int> g_cu[64];

int cu_count() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) dev = 0;
  if (dev < 64) {
    int v = g_cu[dev].load(std::memory_order_relaxed);
    if (v > 0) return v;
  }
  int n = 0;
  if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
    n = 256;
  // the persistent grids deal their tiles to the 8 XCDs in equal shares
  n = n < 8 ? 8 : n / 8 * 8;
  if (dev < 64) g_cu[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Compute units the persistent grids of a call are sized for.
int cus(const zc_moe_desc* d) {
  const int n = cu_count();
  return d->cu_limit > 0 && d->cu_limit < n ? d->cu_limit : n;
}

int64_t a256(int64_t b) { return (b + 255) & ~int64_t(255); }
int64_t esize(const zc_moe_desc* d) { return d->dtype == ZC_F32 ? 4 : 2; }
int64_t ldl_of(int64_t E) { return (E + 7) / 8 * 8; }

#define ZC_CHECK(x)                   \
  do {                                \
    zc_status s_ = (x);               \
    if (s_ != ZC_OK) return s_;       \
  } while (0)

// Shapes the packed layout and its forward kernels handle: bf16, d and I
// multiples of 256, activation buffers (x [T][d], h [T*K][I]) addressable
// with 32-bit byte offsets.
zc_status check_packable(const zc_moe_desc* d) {
  if (d->dtype != ZC_BF16) return fail(ZC_ERR_UNSUPPORTED, "packed weights need a bf16 layer");
  if (d->d % 256 || d->I % 256)
    return fail(ZC_ERR_UNSUPPORTED, "packed weights need d and I multiples of 256 (d=%lld I=%lld)",
                (long long)d->d, (long long)d->I);
  if (d->T * d->d * 2 >= (int64_t(1) << 31) || d->T * d->K * d->I * 2 >= (int64_t(1) << 31))
    return fail(ZC_ERR_UNSUPPORTED, "packed-weight forward needs T*d and T*K*I below 2^30");
  return ZC_OK;
}

// Shapes the MXFP8 forward handles: bf16 layer, d and I multiples of 512
// (whole groups of four 128-step slabs), 32-bit byte offsets into x' and h'.
zc_status check_mxfp8(const zc_moe_desc* d) {
  if (d->dtype != ZC_BF16) return fail(ZC_ERR_UNSUPPORTED, "MXFP8 weights need a bf16 layer");
  if (d->d % 512 || d->I % 512)
    return fail(ZC_ERR_UNSUPPORTED, "MXFP8 weights need d and I multiples of 512 (d=%lld I=%lld)",
                (long long)d->d, (long long)d->I);
  if (d->T * d->d >= (int64_t(1) << 31) || d->T * d->K * d->I >= (int64_t(1) << 31))
    return fail(ZC_ERR_UNSUPPORTED, "MXFP8 forward needs T*d and T*K*I below 2^31");
  return ZC_OK;
}

// Group size of a 4-bit weight layout, 0 for the other layouts.
int int4_group(const zc_moe_desc* d) {
  switch (d->weight_layout) {
    case ZC_WEIGHTS_INT4_G32: return 32;
    case ZC_WEIGHTS_INT4_G64: return 64;
    case ZC_WEIGHTS_INT4_G128: return 128;
    default: return 0;
  }
}

zc_status check_int4(const zc_moe_desc* d) {
  if (d->dtype != ZC_BF16) return fail(ZC_ERR_UNSUPPORTED, "4-bit weights need a bf16 layer");
  if (d->d % 128 || d->I % 128)
    return fail(ZC_ERR_UNSUPPORTED, "4-bit weights need d and I multiples of 128 (d=%lld I=%lld)",
                (long long)d->d, (long long)d->I);
  return ZC_OK;
}

// MXFP4 weights; their rows are MXFP4 too (A4) or MXFP8 (A8).
bool mxfp4(const zc_moe_desc* d) {
  return d->weight_layout == ZC_WEIGHTS_MXFP4_A8 || d->weight_layout == ZC_WEIGHTS_MXFP4_A4;
}
bool mxfp4_a4(const zc_moe_desc* d) { return d->weight_layout == ZC_WEIGHTS_MXFP4_A4; }
zc_status check_mxfp4(const zc_moe_desc* d) {
  if (d->dtype != ZC_BF16) return fail(ZC_ERR_UNSUPPORTED, "MXFP4 weights need a bf16 layer");
  if (d->d % 128 || d->I % 128)
    return fail(ZC_ERR_UNSUPPORTED, "MXFP4 weights need d and I multiples of 128 (d=%lld I=%lld)",
                (long long)d->d, (long long)d->I);
  return ZC_OK;
}
// Layers whose row tiles the experts' kernels list themselves.
bool own_tiles(const zc_moe_desc* d) { return int4_group(d) || mxfp4(d); }

zc_status check_desc(const zc_moe_desc* d) {
  if (!d) return fail(ZC_ERR_INVALID, "desc is NULL");
  const int64_t E = d->N + d->Z;
  if (d->T < 0 || d->d < 1 || d->N < 0 || d->Z < 0 || d->I < 1)
    return fail(ZC_ERR_INVALID, "bad sizes T=%lld d=%lld N=%lld Z=%lld I=%lld", (long long)d->T,
                (long long)d->d, (long long)d->N, (long long)d->Z, (long long)d->I);
  if (E < 1 || E > 1024) return fail(ZC_ERR_INVALID, "N+Z=%lld outside 1..1024", (long long)E);
  if (d->K < 1 || d->K > E || d->K > 32)
    return fail(ZC_ERR_INVALID, "K=%lld outside 1..min(N+Z, 32)", (long long)d->K);
  if (d->dtype != ZC_F32 && d->dtype != ZC_BF16)
    return fail(ZC_ERR_INVALID, "dtype %d is neither ZC_F32 nor ZC_BF16", d->dtype);
  if (d->gate_norm != 0 && d->gate_norm != 1)
    return fail(ZC_ERR_INVALID, "gate_norm %d is neither 0 nor 1", d->gate_norm);
  if (!std::isfinite(d->out_scale)) return fail(ZC_ERR_INVALID, "out_scale is not finite");
  if (d->weight_layout != ZC_WEIGHTS_ROWMAJOR && d->weight_layout != ZC_WEIGHTS_PACKED &&
      d->weight_layout != ZC_WEIGHTS_MXFP8 && !int4_group(d) && !mxfp4(d))
    return fail(ZC_ERR_INVALID, "weight_layout %d is not ROWMAJOR, PACKED, MXFP8, INT4 or MXFP4",
                d->weight_layout);
  if (d->cu_limit < 0 || d->cu_limit % 8)
    return fail(ZC_ERR_INVALID, "cu_limit %d is neither 0 nor a positive multiple of 8",
                d->cu_limit);
  if (d->T * d->K >= (int64_t(1) << 31) || d->d >= (int64_t(1) << 24) || d->I >= (int64_t(1) << 24))
    return fail(ZC_ERR_UNSUPPORTED, "T*K, d or I too large for 32-bit indexing");
  const int64_t mult = d->dtype == ZC_BF16 ? 64 : 32;
  if (d->d % mult || d->I % mult)
    return fail(ZC_ERR_UNSUPPORTED, "%s layers need d and I multiples of %lld (d=%lld I=%lld)",
                d->dtype == ZC_BF16 ? "bf16" : "fp32", (long long)mult, (long long)d->d,
                (long long)d->I);
  if (d->weight_layout == ZC_WEIGHTS_PACKED) ZC_CHECK(check_packable(d));
  if (d->weight_layout == ZC_WEIGHTS_MXFP8) ZC_CHECK(check_mxfp8(d));
  if (int4_group(d)) ZC_CHECK(check_int4(d));
  if (mxfp4(d)) ZC_CHECK(check_mxfp4(d));
  return ZC_OK;
}

bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

zc_status check_ptr(const void* p, const char* name, bool nullable = false) {
  if (!p) return nullable ? ZC_OK : fail(ZC_ERR_INVALID, "%s is NULL", name);
  if (!aligned(p)) return fail(ZC_ERR_INVALID, "%s is not 16-byte aligned", name);
  return ZC_OK;
}

// Per-token buffers may be NULL when there are no tokens (T == 0).
zc_status check_route(const zc_route_buf* r, bool no_tokens) {
  if (!r) return fail(ZC_ERR_INVALID, "route buffer is NULL");
  ZC_CHECK(check_ptr(r->logits, "r->logits", no_tokens));
  ZC_CHECK(check_ptr(r->topk_idx, "r->topk_idx", no_tokens));
  ZC_CHECK(check_ptr(r->topk_gate, "r->topk_gate", no_tokens));
  ZC_CHECK(check_ptr(r->counts, "r->counts"));
  ZC_CHECK(check_ptr(r->offsets, "r->offsets"));
  ZC_CHECK(check_ptr(r->perm, "r->perm", no_tokens));
  ZC_CHECK(check_ptr(r->inv, "r->inv", no_tokens));
  return ZC_OK;
}

// ---- workspace layouts (all pieces 256-byte aligned)
struct RouteWs {
  int32_t* tile_off;   // row-tile prefix for the generic grouped GEMM
  int32_t* tile_off2;  // row-tile prefix for the bf16 forward expert GEMMs
  int32_t* tile_exp;   // expert of each of those row tiles
  int32_t* tile_exp1;  // expert of each row tile of the first prefix
  int32_t* sched;      // tile counters of the packed-weight GEMMs
  float* rpart;        // fp32 partials of a split router GEMM (nullptr: unsplit)
  void* dispatch;
};
// Row tiles of the second prefix, at most: every FFN pick in a tile of its
// own expert, tiles at least 32 rows high.
int64_t max_tiles2(const zc_moe_desc* d) { return d->T * d->K / 32 + d->N + 1; }
int64_t rpart_bytes(const zc_moe_desc* d) {
  const int64_t E = d->N + d->Z;
  const int s = zc::router_gemm_splits(d->T, E, d->d);
  return s > 1 ? 4 * s * d->T * E : 0;
}
int64_t route_ws_bytes(const zc_moe_desc* d) {
  return 2 * a256(4 * (d->N + 1)) + 2 * a256(4 * max_tiles2(d)) + a256(4 * zc::kSchedInts) +
         a256(rpart_bytes(d)) + a256(zc::dispatch_scratch_bytes(d->T, d->N + d->Z, d->N));
}
RouteWs carve_route(char* p, const zc_moe_desc* d) {
  RouteWs w;
  w.tile_off = reinterpret_cast<int32_t*>(p);
  w.tile_off2 = reinterpret_cast<int32_t*>(p + a256(4 * (d->N + 1)));
  char* q = p + 2 * a256(4 * (d->N + 1));
  w.tile_exp = reinterpret_cast<int32_t*>(q);
  q += a256(4 * max_tiles2(d));
  w.tile_exp1 = reinterpret_cast<int32_t*>(q);
  q += a256(4 * max_tiles2(d));
  w.sched = reinterpret_cast<int32_t*>(q);
  q += a256(4 * zc::kSchedInts);
  w.rpart = rpart_bytes(d) > 0 ? reinterpret_cast<float*>(q) : nullptr;
  q += a256(rpart_bytes(d));
  w.dispatch = q;
  return w;
}

// Saved activations: a, u, h of every FFN pick in fp32 (what the backward
// differentiates through, unrounded) and the expert outputs y in the layer
// dtype (what the combine used).
struct Saved {
  float *a, *u, *h;
  void* y;
};
int64_t saved_bytes(const zc_moe_desc* d) {
  const int64_t rows = d->T * d->K, es = esize(d);
  return 3 * a256(rows * d->I * 4) + a256(rows * d->d * es);
}
Saved carve_saved(char* p, const zc_moe_desc* d) {
  const int64_t rows = d->T * d->K;
  const int64_t hi = a256(rows * d->I * 4);
  return Saved{reinterpret_cast<float*>(p), reinterpret_cast<float*>(p + hi),
               reinterpret_cast<float*>(p + 2 * hi), p + 3 * hi};
}

// Forward scratch: routing scratch, h in the layer dtype (operand of the
// down GEMM) or its codes and scales, and y when no saved buffer takes it.
// MXFP8 and MXFP4 layers add x' (codes and scales).  Layers that list their own
// row tiles add the list.
zc::Mx4Plan mxfp4_plan(const zc_moe_desc* d) {
  return zc::mx4_plan(mxfp4_a4(d), d->T, d->T * d->K, d->N + d->Z, d->d, d->I);
}
bool fp32_y(const zc_moe_desc* d) {
  return int4_group(d) || (mxfp4(d) && !mxfp4_plan(d).wide);
}
bool mx_rows(const zc_moe_desc* d) { return d->weight_layout == ZC_WEIGHTS_MXFP8 || mxfp4(d); }
// n values of x or h as codes; their scales, n / 32 bytes, lie behind them.
int64_t mx_code_bytes(const zc_moe_desc* d, int64_t n) { return a256(mxfp4_a4(d) ? n / 2 : n); }
int64_t mx_bytes(const zc_moe_desc* d, int64_t n) { return mx_code_bytes(d, n) + a256(n / 32); }
// (codes and scales take no more than h in bf16, but for the 128 values of one row of
// I = 128: 256 bytes each)
int64_t h_bytes(const zc_moe_desc* d) {
  const int64_t n = d->T * d->K * d->I, b = a256(n * esize(d));
  return mx_rows(d) ? std::max(b, mx_bytes(d, n)) : b;
}
int64_t fwd_ws_bytes(const zc_moe_desc* d) {
  const int64_t rows = d->T * d->K;
  // y is fp32 with 4-bit weights (but for many rows of MXFP4 ones)
  const int64_t ys = fp32_y(d) ? 4 : esize(d);
  int64_t b = route_ws_bytes(d) + h_bytes(d) + a256(rows * d->d * ys);
  if (mx_rows(d)) b += mx_bytes(d, d->T * d->d);
  if (own_tiles(d)) b += a256(zc::row_tiles_bytes(rows, d->N));
  return b;
}

struct BwdWs {
  int32_t* tile_off;
  // dadu: da, du [P][2I] on the generic path; dh [P][I] on the packed-weight
  // path (its SwiGLU backward then writes the hi/lo pairs below)
  float *gs, *dg, *dl, *dadu, *dxp, *dxr, *rdw, *lbc;
  // matrix-core backward (use_bwdp): tile prefix and experts, counters,
  // exact bf16 hi/lo pairs of da, du and g h, and x and dout rows in
  // dispatch order
  int32_t *mt2, *texp2, *sched;
  bf16_t *hilo, *ghlo, *xd, *doutd;
};
constexpr int kBwdSched = 48;  // dh, dx, dW_d, dW_g, dW_u: 8 counters each
// The backward's dh and expert-dx GEMMs read the row-major weights directly
// (gemm_rmw.hip), and its expert weight gradients run on operands gathered
// into dispatch order, for bf16 layers with d and I multiples of 256 whose
// byte offsets into dout, x, the hi/lo pairs and the weights fit 31 bits
// (the weight-gradient loads run up to 64 rows past an expert's).
bool use_bwdp(const zc_moe_desc* d) {
  if (d->dtype != ZC_BF16 || d->N == 0 || d->d % 256 || d->I % 256) return false;
  return zc::rmw_supported(d->T * d->K, d->T, d->d, d->I);
}
// Row-tile height of the dh and dx GEMMs: the average rows per FFN expert
// rounded up to 64 or 128.
int bwdp_rows_per_tile(const zc_moe_desc* d) {
  return d->T * d->K / d->N <= 64 ? 64 : zc::kGemmBM;
}
int64_t bwdp_bytes(const zc_moe_desc* d) {
  if (!use_bwdp(d)) return 0;
  const int64_t rows = d->T * d->K;
  return a256(4 * (d->N + 1)) + a256(4 * max_tiles2(d)) + a256(4 * kBwdSched) +
         a256(rows * 4 * d->I * 2) + a256(rows * 2 * d->I * 2) + 2 * a256(rows * d->d * 2);
}
// fp32 partials of the router weight gradient (token chunks), 0 when unsplit
int64_t rdw_bytes(const zc_moe_desc* d) {
  const int64_t E = d->N + d->Z;
  const int s = zc::router_dw_splits(d->T, E, d->d);
  return s > 1 ? 4 * s * E * d->d : 0;
}
int64_t bwd_ws_bytes(const zc_moe_desc* d) {
  const int64_t rows = d->T * d->K, E = d->N + d->Z;
  return a256(4 * (d->N + 1)) + a256(4 * rows) + a256(4 * d->T * d->K) +
         a256(4 * d->T * ldl_of(E)) + a256(4 * rows * 2 * d->I) + a256(4 * rows * d->d) +
         a256(4 * d->T * d->d) + a256(rdw_bytes(d)) + a256(4 * E) + bwdp_bytes(d);
}
BwdWs carve_bwd(char* p, const zc_moe_desc* d) {
  const int64_t rows = d->T * d->K, E = d->N + d->Z;
  BwdWs w;
  w.tile_off = reinterpret_cast<int32_t*>(p);
  p += a256(4 * (d->N + 1));
  auto take = [&p](int64_t bytes) {
    float* q = reinterpret_cast<float*>(p);
    p += a256(bytes);
    return q;
  };
  w.gs = take(4 * rows);
  w.dg = take(4 * d->T * d->K);
  w.dl = take(4 * d->T * ldl_of(E));
  w.dadu = take(4 * rows * 2 * d->I);
  w.dxp = take(4 * rows * d->d);
  w.dxr = take(4 * d->T * d->d);
  w.rdw = rdw_bytes(d) > 0 ? take(rdw_bytes(d)) : nullptr;
  w.lbc = take(4 * E);
  w.mt2 = w.texp2 = w.sched = nullptr;
  w.hilo = w.ghlo = w.xd = w.doutd = nullptr;
  if (use_bwdp(d)) {
    auto takeb = [&p](int64_t bytes) {
      char* q = p;
      p += a256(bytes);
      return q;
    };
    w.mt2 = reinterpret_cast<int32_t*>(takeb(4 * (d->N + 1)));
    w.texp2 = reinterpret_cast<int32_t*>(takeb(4 * max_tiles2(d)));
    w.sched = reinterpret_cast<int32_t*>(takeb(4 * kBwdSched));
    w.hilo = reinterpret_cast<bf16_t*>(takeb(rows * 4 * d->I * 2));
    w.ghlo = reinterpret_cast<bf16_t*>(takeb(rows * 2 * d->I * 2));
    w.xd = reinterpret_cast<bf16_t*>(takeb(rows * d->d * 2));
    w.doutd = reinterpret_cast<bf16_t*>(takeb(rows * d->d * 2));
  }
  return w;
}

zc_status check_ws(const void* ws, size_t ws_bytes, int64_t need) {
  if (need > 0 && (!ws || ws_bytes < static_cast<size_t>(need)))
    return fail(ZC_ERR_WORKSPACE, "workspace of %zu bytes at %p, %lld needed", ws_bytes, ws,
                (long long)need);
  if (ws && (reinterpret_cast<uintptr_t>(ws) & 255u))
    return fail(ZC_ERR_INVALID, "workspace is not 256-byte aligned");
  return ZC_OK;
}

// Load-balance loss settings against the layer: D groups of N/D FFN
// experts, 0 < K_e <= K (K_e < K when there are zero-computation experts,
// whose pick frequency divides by K - K_e), finite alpha.
zc_status check_lb(const zc_moe_desc* d, const zc_lb_cfg* lb) {
  if (!lb) return fail(ZC_ERR_INVALID, "load-balance settings are NULL");
  if (d->N < 1) return fail(ZC_ERR_INVALID, "the load-balance loss needs FFN experts (N >= 1)");
  if (lb->D < 1 || lb->D > d->N || d->N % lb->D)
    return fail(ZC_ERR_INVALID, "D=%lld does not split N=%lld into equal groups",
                (long long)lb->D, (long long)d->N);
  if (!std::isfinite(lb->K_e) || !(lb->K_e > 0.0) || lb->K_e > static_cast<double>(d->K) ||
      (d->Z > 0 && !(lb->K_e < static_cast<double>(d->K))))
    return fail(ZC_ERR_INVALID, "K_e=%g outside (0, K=%lld%s", lb->K_e, (long long)d->K,
                d->Z > 0 ? ")" : "]");
  if (!std::isfinite(lb->alpha)) return fail(ZC_ERR_INVALID, "alpha is not finite");
  return ZC_OK;
}
int64_t stats_ws_bytes(const zc_moe_desc* d) {
  return a256(static_cast<int64_t>(zc::stats_scratch_bytes(d->T, d->K)));
}
int64_t lb_ws_bytes(const zc_moe_desc* d) {
  return a256(static_cast<int64_t>(zc::lb_scratch_bytes(d->T, d->N + d->Z)));
}

// The 256 x 256 forward kernels: bf16 layers with row-major weights (with a
// saved buffer the gate/up epilogue also writes a, u, h in fp32 for the
// backward), 32-bit element offsets (rows * columns < 2^31), and on
// average at least 64 rows per FFN expert (T*K/N, known on the host without
// reading the counts back); decode-sized batches keep the 128 x 128 kernel,
// whose larger grid streams a few rows' worth of weights per expert better.
template <typename T>
bool use_fwd_kernels(const zc_moe_desc* d) {
  if (!std::is_same<T, bf16_t>::value) return false;
  if (d->N == 0 || d->T * d->K < 64 * d->N) return false;
  const int64_t rows = d->T * d->K, cols = d->I > d->d ? d->I : d->d;
  return rows * cols < (int64_t(1) << 31) && d->T * d->d < (int64_t(1) << 31);
}

// The row-major weight kernels of gemm_rmw.hip (forward, with or without
// saved activations): bf16 layers with d and I multiples of 256 whose byte
// offsets fit 31 bits.
bool rmw_layer(const zc_moe_desc* d) {
  return d->dtype == ZC_BF16 && d->N > 0 && d->weight_layout == ZC_WEIGHTS_ROWMAJOR &&
         zc::rmw_fwd_supported(d->T * d->K, d->T, d->d, d->I);
}
template <typename T>
bool use_rmw(const zc_moe_desc* d) {
  return std::is_same<T, bf16_t>::value && rmw_layer(d);
}

// Router scores on the 256 x 256-tile kernel: bf16 layers with E a multiple
// of 256 and at least 128 such tiles (T * E >= 2^23); smaller batches keep
// the generic kernel, which splits the hidden dimension to fill the GPU.
template <typename T>
bool use_dense_router(const zc_moe_desc* d) {
  const int64_t E = d->N + d->Z;
  return std::is_same<T, bf16_t>::value && d->T * E >= (int64_t(1) << 23) &&
         zc::rmw_dense_supported(d->T, E, d->d);
}

// Router + dispatch on an already validated call.
// Row-tile height of the second tile prefix (tile_off2): the packed-weight
// forward picks it from the average rows per FFN expert, the row-major
// kernels of gemm_rmw.hip likewise but at least 64 rows, the other row-major
// bf16 forward kernels use 256.
int fwd_rows_per_tile(const zc_moe_desc* d) {
  if (d->N == 0 || own_tiles(d)) return zc::kFwdBM;  // (4-bit layers list their own tiles)
  const int tm = zc::fwdp_rows_per_tile(d->T * d->K / d->N);
  if (d->weight_layout != ZC_WEIGHTS_ROWMAJOR) return tm;
  return rmw_layer(d) ? (tm < 64 ? 64 : tm) : zc::kFwdBM;
}

template <typename T>
zc_status do_route(const zc_moe_desc* d, const T* x, const T* wr, const float* bias,
                   zc_route_buf* r, const RouteWs& w, hipStream_t s) {
  const int Tn = static_cast<int>(d->T), E = static_cast<int>(d->N + d->Z);
  const int N = static_cast<int>(d->N), K = static_cast<int>(d->K);
  if (x && Tn > 0) {
    if (use_dense_router<T>(d))
      ZC_LAUNCH(ZC_PH_ROUTER_GEMM,
                zc::launch_rmw_dense(reinterpret_cast<const bf16_t*>(x), Tn,
                                     reinterpret_cast<const bf16_t*>(wr), E,
                                     static_cast<int>(d->d), r->logits, cus(d), s),
                "router GEMM launch");
    else
      ZC_LAUNCH(ZC_PH_ROUTER_GEMM,
                zc::launch_router_gemm<T>(x, wr, r->logits, Tn, E, static_cast<int>(d->d),
                                          w.rpart, cus(d), s),
                "router GEMM launch");
  }
  ZC_LAUNCH(ZC_PH_TOPK, zc::launch_topk(r->logits, bias, Tn, E, K, d->gate_norm, r->topk_idx, r->topk_gate, s),
         "top-K launch");
  ZC_LAUNCH(ZC_PH_DISPATCH, zc::launch_dispatch(r->topk_idx, Tn, E, N, K, zc::kGemmBM,
                                                fwd_rows_per_tile(d),
                                                r->counts, r->offsets, r->perm, r->inv, w.tile_off,
                                                w.tile_off2, w.tile_exp, w.tile_exp1, w.sched,
                                                w.dispatch, s),
         "dispatch launch");
  return ZC_OK;
}

// The experts and the combine of a routed batch whose tile tables are in ws
// (rw).  mxq, mxs: x as MXFP8 rows, NULL to quantize it here (MXFP8 layers).
template <typename T>
zc_status do_experts(const zc_moe_desc* d, const T* x, const T* wg, const T* wu, const T* wd,
                     T* out, const zc_route_buf* r, void* saved, const uint8_t* mxq,
                     const uint8_t* mxs, const RouteWs& rw, char* ws, hipStream_t s) {
  const int Tn = static_cast<int>(d->T), N = static_cast<int>(d->N), K = static_cast<int>(d->K);
  const int dd = static_cast<int>(d->d), I = static_cast<int>(d->I);
  const int64_t rows = d->T * d->K;
  char* p = ws + route_ws_bytes(d);
  T* h = reinterpret_cast<T*>(p);
  T* y = reinterpret_cast<T*>(p + h_bytes(d));
  float *sa = nullptr, *su = nullptr, *sh = nullptr;
  if (saved) {
    Saved sv = carve_saved(static_cast<char*>(saved), d);
    sa = sv.a;
    su = sv.u;
    sh = sv.h;
    y = static_cast<T*>(sv.y);
  }
  if (N > 0 && Tn > 0) {
    const int cu = cus(d);
    if (d->weight_layout == ZC_WEIGHTS_MXFP8) {
      // MXFP8 inference: x quantized once, h quantized in the gate/up
      // epilogue (validated: bf16, no saved buffer)
      uint8_t* xq = reinterpret_cast<uint8_t*>(ws + fwd_ws_bytes(d) - mx_bytes(d, d->T * d->d));
      uint8_t* xs = xq + mx_code_bytes(d, d->T * d->d);
      uint8_t* hq = reinterpret_cast<uint8_t*>(h);
      uint8_t* hs = hq + mx_code_bytes(d, rows * d->I);
      if (!mxq)
        ZC_LAUNCH(ZC_PH_QUANTIZE,
                  zc::launch_mxq_rows(reinterpret_cast<const bf16_t*>(x), d->T, dd, xq, xs, s),
                  "activation quantization launch");
      ZC_LAUNCH(ZC_PH_GATE_UP,
                zc::launch_fwdq_gateup(mxq ? mxq : xq, mxq ? mxs : xs, d->T, reinterpret_cast<const uint8_t*>(wg),
                                       reinterpret_cast<const uint8_t*>(wu), r->offsets, r->perm,
                                       rw.tile_off2, rw.tile_exp, rw.sched, fwd_rows_per_tile(d), N,
                                       I, dd, K, hq, hs, cu, s),
                "gate/up GEMM launch");
      ZC_LAUNCH(ZC_PH_DOWN,
                zc::launch_fwdq_down(hq, hs, rows, reinterpret_cast<const uint8_t*>(wd), r->offsets,
                                     rw.tile_off2, rw.tile_exp, rw.sched + 8,
                                     fwd_rows_per_tile(d), N, I, dd,
                                     reinterpret_cast<bf16_t*>(y), cu, s),
                "down GEMM launch");
    } else if (const int G = int4_group(d)) {
      // 4-bit weights (validated: bf16, no saved buffer); y is fp32
      float* yf = reinterpret_cast<float*>(y);
      void* tiles = ws + fwd_ws_bytes(d) - a256(zc::row_tiles_bytes(rows, N));
      // (picks spread over all N + Z experts)
      const int tm = zc::int4_rows_per_tile(rows / (d->N + d->Z), d->T, rows, d->d, d->I);
      ZC_LAUNCH(ZC_PH_TILE_OFFSETS, zc::launch_row_tiles(r->offsets, N, tm, tiles, s),
                "tile list launch");
      ZC_LAUNCH(ZC_PH_GATE_UP,
                zc::launch_int4_gateup(reinterpret_cast<const bf16_t*>(x), d->T,
                                       reinterpret_cast<const uint8_t*>(wg),
                                       reinterpret_cast<const uint8_t*>(wu), G, tiles, r->perm, tm,
                                       rows, N, I, dd, K, reinterpret_cast<bf16_t*>(h), s),
                "gate/up GEMM launch");
      ZC_LAUNCH(ZC_PH_DOWN,
                zc::launch_int4_down(reinterpret_cast<const bf16_t*>(h),
                                     reinterpret_cast<const uint8_t*>(wd), G, tiles, tm, rows, N, I,
                                     dd, yf, s),
                "down GEMM launch");
    } else if (mxfp4(d)) {
      // MXFP4 weights (validated: bf16, no saved buffer)
      const bool a4 = mxfp4_a4(d);
      char* tiles = ws + fwd_ws_bytes(d) - a256(zc::row_tiles_bytes(rows, N));
      uint8_t* xq = reinterpret_cast<uint8_t*>(tiles - mx_bytes(d, d->T * d->d));
      uint8_t* xs = xq + mx_code_bytes(d, d->T * d->d);
      uint8_t* hq = reinterpret_cast<uint8_t*>(h);
      uint8_t* hs = hq + mx_code_bytes(d, rows * d->I);
      const zc::Mx4Plan plan = mxfp4_plan(d);
      if (mxq)
        ZC_LAUNCH(ZC_PH_TILE_OFFSETS, zc::launch_row_tiles(r->offsets, N, plan.tm, tiles, s),
                  "tile list launch");
      else
        ZC_LAUNCH(ZC_PH_QUANTIZE,
                  zc::launch_mx4_start(a4, r->offsets, N, plan.tm, tiles,
                                       reinterpret_cast<const bf16_t*>(x), d->T, dd, xq, xs, s),
                  "tile list and activation quantization launch");
      ZC_LAUNCH(ZC_PH_GATE_UP,
                zc::launch_mx4_gateup(a4, mxq ? mxq : xq, mxq ? mxs : xs, d->T,
                                      reinterpret_cast<const uint8_t*>(wg),
                                      reinterpret_cast<const uint8_t*>(wu), tiles, r->perm, plan, rows,
                                      N, I, dd, K, hq, hs, s),
                "gate/up GEMM launch");
      ZC_LAUNCH(ZC_PH_DOWN,
                zc::launch_mx4_down(a4, hq, hs, reinterpret_cast<const uint8_t*>(wd), tiles, plan, rows,
                                    N, I, dd, y, s),
                "down GEMM launch");
    } else if (d->weight_layout == ZC_WEIGHTS_PACKED) {
      // bf16 inference on packed weights (validated: bf16, no saved buffer)
      const bf16_t* hx = reinterpret_cast<const bf16_t*>(x);
      bf16_t* hh = reinterpret_cast<bf16_t*>(h);
      ZC_LAUNCH(ZC_PH_GATE_UP,
                zc::launch_fwdp_gateup(hx, d->T * d->d, reinterpret_cast<const bf16_t*>(wg),
                                       reinterpret_cast<const bf16_t*>(wu), r->offsets, r->perm,
                                       rw.tile_off2, rw.tile_exp, rw.sched, fwd_rows_per_tile(d), N,
                                       I, dd, K, hh, cu, s),
                "gate/up GEMM launch");
      ZC_LAUNCH(ZC_PH_DOWN,
                zc::launch_fwdp_down(hh, rows * d->I, reinterpret_cast<const bf16_t*>(wd),
                                     r->offsets, rw.tile_off2, rw.tile_exp, rw.sched + 8,
                                     fwd_rows_per_tile(d), N, I, dd, reinterpret_cast<bf16_t*>(y),
                                     cu, s),
                "down GEMM launch");
    } else if (use_rmw<T>(d)) {
      // bf16 on row-major weights; with a saved buffer (training) a, u, h
      // are also kept in fp32
      ZC_LAUNCH(ZC_PH_GATE_UP,
                zc::launch_rmw_gateup(reinterpret_cast<const bf16_t*>(x), d->T,
                                      reinterpret_cast<const bf16_t*>(wg),
                                      reinterpret_cast<const bf16_t*>(wu), r->offsets, r->perm,
                                      rw.tile_off2, rw.tile_exp, rw.sched, fwd_rows_per_tile(d), N,
                                      I, dd, K, reinterpret_cast<bf16_t*>(h), sa, su, sh, cu, s),
                "gate/up GEMM launch");
      ZC_LAUNCH(ZC_PH_DOWN,
                zc::launch_rmw_down(reinterpret_cast<const bf16_t*>(h), rows,
                                    reinterpret_cast<const bf16_t*>(wd), r->offsets, rw.tile_off2,
                                    rw.tile_exp, rw.sched + 8, fwd_rows_per_tile(d), N, I, dd,
                                    reinterpret_cast<bf16_t*>(y), cu, s),
                "down GEMM launch");
    } else if (use_fwd_kernels<T>(d)) {
      // bf16 on row-major weights whose d or I is not a multiple of 256:
      // 256 x 256 tiles, weights streamed once per expert; with a saved
      // buffer the gate/up epilogue also keeps a, u, h
      ZC_LAUNCH(ZC_PH_GATE_UP,
                zc::launch_fwd_gateup(reinterpret_cast<const bf16_t*>(x),
                                      reinterpret_cast<const bf16_t*>(wg),
                                      reinterpret_cast<const bf16_t*>(wu), r->offsets, r->perm,
                                      rw.tile_off2, N, I, dd, K, reinterpret_cast<bf16_t*>(h),
                                      sa, su, sh, cu, s),
                "gate/up GEMM launch");
      ZC_LAUNCH(ZC_PH_DOWN,
                zc::launch_fwd_down(reinterpret_cast<const bf16_t*>(h),
                                    reinterpret_cast<const bf16_t*>(wd), r->offsets, rw.tile_off2, N,
                                    I, dd, reinterpret_cast<bf16_t*>(y), cu, s),
                "down GEMM launch");
    } else {
      ZC_LAUNCH(ZC_PH_GATE_UP, zc::launch_ffn_gateup<T>(x, wg, wu, r->offsets, r->perm, rw.tile_off,
                                                        N, I, dd, K, rows, h, sa, su, sh, cu, s),
                "gate/up GEMM launch");
      ZC_LAUNCH(ZC_PH_DOWN, zc::launch_ffn_down<T>(h, wd, r->offsets, rw.tile_off, N, I, dd, rows,
                                                   y, cu, s),
                "down GEMM launch");
    }
  }
  if constexpr (std::is_same<T, bf16_t>::value) {
    if (fp32_y(d)) {
      ZC_LAUNCH(ZC_PH_COMBINE,
                (zc::launch_combine<T, float>(x, reinterpret_cast<const float*>(y), r->topk_idx,
                                              r->topk_gate, r->inv, Tn, dd, N, K, d->out_scale, out,
                                              s)),
                "combine launch");
      return ZC_OK;
    }
  }
  ZC_LAUNCH(ZC_PH_COMBINE, (zc::launch_combine<T, T>(x, y, r->topk_idx, r->topk_gate, r->inv, Tn, dd, N, K, d->out_scale,
                               out, s)),
         "combine launch");
  return ZC_OK;
}

template <typename T>
zc_status do_forward(const zc_moe_desc* d, const T* x, const T* wr, const float* bias,
                     const T* wg, const T* wu, const T* wd, T* out, zc_route_buf* r, void* saved,
                     char* ws, hipStream_t s) {
  RouteWs rw = carve_route(ws, d);
  ZC_CHECK(do_route<T>(d, x, wr, bias, r, rw, s));
  return do_experts<T>(d, x, wg, wu, wd, out, r, saved, nullptr, nullptr, rw, ws, s);
}

// The same on routing that an earlier call left in r.
template <typename T>
zc_status do_routed_experts(const zc_moe_desc* d, const T* x, const T* wg, const T* wu, const T* wd,
                            T* out, const zc_route_buf* r, const uint8_t* mxq, const uint8_t* mxs,
                            char* ws, hipStream_t s) {
  const RouteWs rw = carve_route(ws, d);
  const int N = static_cast<int>(d->N);
  if (N > 0 && d->T > 0 && !own_tiles(d))
    ZC_LAUNCH(ZC_PH_TILE_OFFSETS,
              zc::launch_tile_offsets2(r->offsets, N, zc::kGemmBM, rw.tile_off,
                                       fwd_rows_per_tile(d), rw.tile_off2, rw.tile_exp, rw.sched,
                                       zc::kSchedInts, s),
              "tile offsets");
  return do_experts<T>(d, x, wg, wu, wd, out, r, nullptr, mxq, mxs, rw, ws, s);
}

template <typename T>
zc_status do_backward(const zc_moe_desc* d, const T* x, const T* wr, const T* wg, const T* wu,
                      const T* wd, const zc_route_buf* r, const void* saved, const T* dout, T* dx,
                      T* dwr, T* dwg, T* dwu, T* dwd, const zc_lb_cfg* lb, const float* dlogits,
                      char* ws, hipStream_t s) {
  const int Tn = static_cast<int>(d->T), N = static_cast<int>(d->N), K = static_cast<int>(d->K);
  const int E = static_cast<int>(d->N + d->Z), dd = static_cast<int>(d->d);
  const int I = static_cast<int>(d->I), ldl = static_cast<int>(ldl_of(E));
  const int64_t rows = d->T * d->K;
  const int cu = cus(d);
  BwdWs w = carve_bwd(ws, d);
  Saved sv = carve_saved(const_cast<char*>(static_cast<const char*>(saved)), d);
  const T* y = static_cast<const T*>(sv.y);
  const bool bwdp = std::is_same<T, bf16_t>::value && use_bwdp(d);
  const int tmb = bwdp ? bwdp_rows_per_tile(d) : 0;
  if (N > 0) {
    if (bwdp) {
      ZC_LAUNCH(ZC_PH_TILE_OFFSETS,
                zc::launch_tile_offsets2(r->offsets, N, zc::kGemmBM, w.tile_off, tmb, w.mt2,
                                         w.texp2, w.sched, kBwdSched, s),
                "tile offsets");
    } else {
      ZC_LAUNCH(ZC_PH_TILE_OFFSETS,
                zc::launch_tile_offsets(r->offsets, N, zc::kGemmBM, w.tile_off, s), "tile offsets");
    }
  }
  if (lb)
    ZC_LAUNCH(ZC_PH_LB_COEF,
              zc::launch_lb_coef(r->counts, Tn, N, E, K, static_cast<int>(lb->D), lb->K_e,
                                 lb->alpha, w.lbc, s),
              "load-balance coefficient launch");
  ZC_LAUNCH(ZC_PH_BWD_COMBINE,
            zc::launch_combine_bwd<T>(x, y, dout, r->logits, r->topk_idx, r->topk_gate, r->inv, Tn,
                                      dd, N, E, K, d->gate_norm, d->out_scale,
                                      lb ? w.lbc : nullptr, dlogits, w.gs, w.dg, w.dl, ldl, s),
            "combine backward launch");
  if (N > 0) {
    if (Tn > 0 && bwdp) {
      ZC_LAUNCH(ZC_PH_BWD_GATHER,
                zc::launch_gather_rows(reinterpret_cast<const bf16_t*>(dout), r->perm, r->offsets,
                                       N, K, dd, rows, w.doutd, s),
                "row gather launch");
      ZC_LAUNCH(ZC_PH_BWD_GATHER,
                zc::launch_gather_rows(reinterpret_cast<const bf16_t*>(x), r->perm, r->offsets, N,
                                       K, dd, rows, w.xd, s),
                "row gather launch");
      ZC_LAUNCH(ZC_PH_BWD_DOWN_DH,
                zc::launch_rmw_dh(w.doutd, rows, reinterpret_cast<const bf16_t*>(wd), r->offsets,
                                  w.mt2, w.texp2, w.sched, tmb, N, I, dd, w.gs, w.dadu, cu, s),
                "down backward (dh) launch");
      ZC_LAUNCH(ZC_PH_BWD_DOWN_DH,
                zc::launch_swiglu_bwd(w.dadu, w.gs, sv.a, sv.u, sv.h, r->offsets, N, I, rows,
                                      w.hilo, w.ghlo, s),
                "SwiGLU backward launch");
    } else if (Tn > 0) {
      ZC_LAUNCH(ZC_PH_BWD_DOWN_DH,
                zc::launch_bwd_down_dh<T>(dout, r->perm, K, w.gs, wd, sv.a, sv.u, r->offsets,
                                          w.tile_off, N, I, dd, rows, w.dadu, cu, s),
                "down backward (dh) launch");
    }
    if (bwdp)
      ZC_LAUNCH(ZC_PH_BWD_DOWN_DW,
                zc::launch_dw(true, N, I, dd, r->offsets, w.sched + 16, w.ghlo, w.ghlo + I, 2 * I,
                              w.doutd, dd, rows, reinterpret_cast<bf16_t*>(dwd), cu, s),
                "down weight-gradient launch");
    else
      ZC_LAUNCH(ZC_PH_BWD_DOWN_DW,
                zc::launch_bwd_down_dw<T>(dout, r->perm, K, sv.h, w.gs, r->offsets, N, I, dd, dwd,
                                          cu, s),
                "down weight-gradient launch");
    if (Tn > 0 && bwdp) {
      ZC_LAUNCH(ZC_PH_BWD_GATE_UP_DX,
                zc::launch_rmw_dx(w.hilo, rows, reinterpret_cast<const bf16_t*>(wg),
                                  reinterpret_cast<const bf16_t*>(wu), r->offsets, w.mt2, w.texp2,
                                  w.sched + 8, tmb, N, I, dd, w.dxp, cu, s),
                "gate/up backward (dx) launch");
    } else if (Tn > 0) {
      ZC_LAUNCH(ZC_PH_BWD_GATE_UP_DX,
                zc::launch_bwd_gateup_dx<T>(w.dadu, wg, wu, r->offsets, w.tile_off, N, I, dd, rows,
                                            w.dxp, cu, s),
                "gate/up backward (dx) launch");
    }
    if (bwdp) {
      ZC_LAUNCH(ZC_PH_BWD_GATE_UP_DW,
                zc::launch_dw(false, N, I, dd, r->offsets, w.sched + 24, w.hilo, w.hilo + I, 4 * I,
                              w.xd, dd, rows, reinterpret_cast<bf16_t*>(dwg), cu, s),
                "gate/up weight-gradient launch");
      ZC_LAUNCH(ZC_PH_BWD_GATE_UP_DW,
                zc::launch_dw(false, N, I, dd, r->offsets, w.sched + 32, w.hilo + 2 * I,
                              w.hilo + 3 * I, 4 * I, w.xd, dd, rows, reinterpret_cast<bf16_t*>(dwu),
                              cu, s),
                "gate/up weight-gradient launch");
    } else {
      ZC_LAUNCH(ZC_PH_BWD_GATE_UP_DW,
                zc::launch_bwd_gateup_dw<T>(w.dadu, x, r->offsets, r->perm, N, I, dd, K, dwg, dwu,
                                            cu, s),
                "gate/up weight-gradient launch");
    }
  }
  ZC_LAUNCH(ZC_PH_BWD_ROUTER_DW, zc::launch_router_dw<T>(w.dl, ldl, x, Tn, E, dd, dwr, w.rdw, cu, s),
            "router weight-gradient launch");
  if (Tn > 0) {
    ZC_LAUNCH(ZC_PH_BWD_ROUTER_DX, zc::launch_router_dx<T>(w.dl, ldl, wr, Tn, E, dd, w.dxr, cu, s),
              "router dx launch");
    ZC_LAUNCH(ZC_PH_BWD_DX_GATHER,
              zc::launch_dx_gather<T>(dout, w.dxp, w.dxr, r->topk_idx, r->topk_gate, r->inv, Tn, dd,
                                      N, K, d->out_scale, dx, s),
              "dx gather launch");
  }
  return ZC_OK;
}

// ---- scratch of the allocation-free forward (zc_moe_forward_noalloc)
// A file-scope device array: every GPU the library runs on holds its own
// copy, at its own address, until the process ends.  Host code never uses
// the array's name as a device address: scratch_ptr() looks each device's
// copy up once (hipGetSymbolAddress, with that device current) and keeps it.
constexpr size_t kNoAllocScratch = size_t(64) << 20;  // ZC_NOALLOC_SCRATCH_BYTES
static __device__ __align__(256) char scratch[kNoAllocScratch];
static_assert(kNoAllocScratch == ZC_NOALLOC_SCRATCH_BYTES, "header and library disagree");

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices];

zc_status scratch_ptr(void** out) {
  int dev = -1;
  ZC_HIP(hipGetDevice(&dev), "hipGetDevice");
  if (dev < 0 || dev >= kMaxDevices)
    return fail(ZC_ERR_UNSUPPORTED, "device %d: the allocation-free forward tracks devices 0..%d",
                dev, kMaxDevices - 1);
  std::lock_guard<std::mutex> lk(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* p = nullptr;
    ZC_HIP(hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)), "hipGetSymbolAddress(scratch)");
    if (!p || (reinterpret_cast<uintptr_t>(p) & 255u))
      return fail(ZC_ERR_HIP, "scratch of device %d at %p is not 256-byte aligned", dev, p);
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return ZC_OK;
}

// Two ranges share bytes.
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const char *p = static_cast<const char*>(a), *q = static_cast<const char*>(b);
  return p && q && na > 0 && nb > 0 && p < q + nb && q < p + na;
}

// A buffer a call reads or writes; outputs may be the very buffer of an
// input where the call allows it (in place), and overlap nothing else.
struct Range {
  const void* p;
  int64_t bytes;
  const char* name;
  bool inplace;  // input: an output may take its place
};
zc_status check_overlap(const Range* out, int nout, const Range* in, int nin) {
  for (int i = 0; i < nout; ++i) {
    for (int j = 0; j < nin; ++j)
      if (overlap(out[i].p, out[i].bytes, in[j].p, in[j].bytes) &&
          !(out[i].inplace && in[j].inplace && out[i].p == in[j].p && out[i].bytes == in[j].bytes))
        return fail(ZC_ERR_INVALID, "%s overlaps %s", out[i].name, in[j].name);
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
        return fail(ZC_ERR_INVALID, "%s overlaps %s", out[i].name, out[j].name);
  }
  return ZC_OK;
}

// Sequences of a packed batch.
zc_status check_seqs(const zc_moe_desc* d, int64_t S) {
  if (S < 1 || S > (int64_t(1) << 20))
    return fail(ZC_ERR_INVALID, "S=%lld sequences outside 1..2^20", (long long)S);
  if (d->T > (int64_t(1) << 25))
    return fail(ZC_ERR_UNSUPPORTED, "T=%lld tokens above 2^25", (long long)d->T);
  return ZC_OK;
}

zc_status check_norm(const zc_norm_desc* d) {
  if (!d) return fail(ZC_ERR_INVALID, "desc is NULL");
  if (d->T < 0 || d->d < 1)
    return fail(ZC_ERR_INVALID, "bad sizes T=%lld d=%lld", (long long)d->T, (long long)d->d);
  if (d->dtype != ZC_F32 && d->dtype != ZC_BF16)
    return fail(ZC_ERR_INVALID, "dtype %d is neither ZC_F32 nor ZC_BF16", d->dtype);
  if (!std::isfinite(d->eps) || !(d->eps > 0.f))
    return fail(ZC_ERR_INVALID, "eps is not a positive number");
  const int mult = d->dtype == ZC_BF16 ? 8 : 4;
  if (d->d % mult || d->d > zc::kNormMaxD)
    return fail(ZC_ERR_UNSUPPORTED, "%s rows need d a multiple of %d and at most %d (d=%lld)",
                d->dtype == ZC_BF16 ? "bf16" : "fp32", mult, zc::kNormMaxD, (long long)d->d);
  if (d->T >= (int64_t(1) << 31)) return fail(ZC_ERR_UNSUPPORTED, "T too large for one grid");
  return ZC_OK;
}
int64_t norm_esize(const zc_norm_desc* d) { return d->dtype == ZC_F32 ? 4 : 2; }
int64_t norm_ws_bytes(const zc_norm_desc* d) {
  const int n = static_cast<int>(d->d);
  const int64_t np = d->dtype == ZC_BF16 ? zc::norm_bwd_parts<bf16_t>(d->T, n)
                                         : zc::norm_bwd_parts<float>(d->T, n);
  return a256(np * d->d * 4);
}

// ---- lists of tensors (gradient norm, AdamW)
constexpr int64_t kMaxTensors = int64_t(1) << 20, kMaxElems = int64_t(1) << 36;
int64_t dtype_size(int dtype) { return dtype == ZC_F32 ? 4 : 2; }
zc_status check_dtype(int dtype, const char* name) {
  if (dtype != ZC_F32 && dtype != ZC_BF16)
    return fail(ZC_ERR_INVALID, "%s %d is neither ZC_F32 nor ZC_BF16", name, dtype);
  return ZC_OK;
}
zc_status check_elems(int64_t n, int64_t i) {
  if (n < 0) return fail(ZC_ERR_INVALID, "tensor %lld has n=%lld", (long long)i, (long long)n);
  if (n >= kMaxElems)
    return fail(ZC_ERR_UNSUPPORTED, "tensor %lld: n=%lld is not below 2^36", (long long)i, (long long)n);
  return ZC_OK;
}
zc_status check_count(const void* tensors, int64_t count) {
  if (count < 0 || count > kMaxTensors)
    return fail(ZC_ERR_INVALID, "count=%lld outside 0..2^20", (long long)count);
  if (count && !tensors) return fail(ZC_ERR_INVALID, "tensors is NULL");
  return ZC_OK;
}

// The buffers of a list: no written one may share bytes with any other.
struct Span {
  uintptr_t begin, end;
  int64_t tensor;
  const char* name;
  bool written;
};
zc_status check_spans(std::vector<Span>& v) {
  std::sort(v.begin(), v.end(), [](const Span& a, const Span& b) { return a.begin < b.begin; });
  const Span *far = nullptr, *far_written = nullptr;  // the one that ends last so far
  for (const Span& x : v) {
    const Span* hit = x.written ? far : far_written;
    if (hit && x.begin < hit->end)
      return fail(ZC_ERR_INVALID, "%s of tensor %lld overlaps %s of tensor %lld", x.name,
                  (long long)x.tensor, hit->name, (long long)hit->tensor);
    if (!far || x.end > far->end) far = &x;
    if (x.written && (!far_written || x.end > far_written->end)) far_written = &x;
  }
  return ZC_OK;
}
void add_span(std::vector<Span>& v, const void* p, int64_t bytes, int64_t tensor, const char* name,
              bool written) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  if (p && bytes > 0) v.push_back(Span{b, b + static_cast<uintptr_t>(bytes), tensor, name, written});
}

// Read and written one by one: aligned like an element.
zc_status check_scalar(const void* p, size_t align, const char* name) {
  if (reinterpret_cast<uintptr_t>(p) % align)
    return fail(ZC_ERR_INVALID, "%s is not %zu-byte aligned", name, align);
  return ZC_OK;
}

zc_status check_grads(const zc_grad_tensor* t, int64_t count, int g_dtype) {
  ZC_CHECK(check_dtype(g_dtype, "g_dtype"));
  ZC_CHECK(check_count(t, count));
  for (int64_t i = 0; i < count; ++i) {
    ZC_CHECK(check_elems(t[i].n, i));
    ZC_CHECK(check_ptr(t[i].g, "g", t[i].n == 0));
  }
  return ZC_OK;
}
// The list as two arrays, and the workspace it takes.
struct Grads {
  std::vector<const void*> g;
  std::vector<int64_t> n;
  int64_t ws_bytes;
  Grads(const zc_grad_tensor* t, int64_t count, bool bf16) {
    for (int64_t i = 0; i < count; ++i) {
      g.push_back(t[i].g);
      n.push_back(t[i].n);
    }
    ws_bytes = a256(8 * zc::grad_norm_parts(n.data(), count, bf16));
  }
};

zc_status do_grad_norm(const zc_grad_tensor* t, int64_t count, int g_dtype, double max_norm,
                       float* out, int64_t* step, void* ws, size_t ws_bytes, hipStream_t s) {
  const bool bf16 = g_dtype == ZC_BF16;
  const Grads l(t, count, bf16);
  ZC_CHECK(check_ws(ws, ws_bytes, l.ws_bytes));
  std::vector<Span> spans;
  for (int64_t i = 0; i < count; ++i)
    add_span(spans, t[i].g, t[i].n * dtype_size(g_dtype), i, "g", false);
  add_span(spans, out, 8, -1, "out", true);
  add_span(spans, step, 8, -1, "step", true);
  add_span(spans, ws, l.ws_bytes, -1, "ws", true);
  ZC_CHECK(check_spans(spans));
  ZC_LAUNCH(ZC_PH_GRAD_NORM,
            zc::launch_grad_norm(l.g.data(), l.n.data(), count, bf16, max_norm,
                                 static_cast<double*>(ws), out, step, s),
            "gradient norm launch");
  return ZC_OK;
}

zc_status check_adamw(const zc_adamw_cfg* c, bool device_step) {
  if (!c) return fail(ZC_ERR_INVALID, "cfg is NULL");
  ZC_CHECK(check_dtype(c->p_dtype, "p_dtype"));
  ZC_CHECK(check_dtype(c->g_dtype, "g_dtype"));
  if (c->g_dtype != c->p_dtype && c->g_dtype != ZC_F32)
    return fail(ZC_ERR_UNSUPPORTED, "bf16 gradients of fp32 weights");
  if (c->state != ZC_STATE_F32 && c->state != ZC_STATE_8BIT)
    return fail(ZC_ERR_INVALID, "state %d is neither ZC_STATE_F32 nor ZC_STATE_8BIT", c->state);
  if (c->rounding != ZC_ROUND_NEAREST && c->rounding != ZC_ROUND_STOCHASTIC)
    return fail(ZC_ERR_INVALID, "rounding %d is neither ZC_ROUND_NEAREST nor ZC_ROUND_STOCHASTIC",
                c->rounding);
  if (!std::isfinite(static_cast<float>(c->lr)) || c->lr < 0.0)
    return fail(ZC_ERR_INVALID, "lr=%g", c->lr);
  if (!(c->beta1 >= 0.0 && c->beta1 < 1.0) || !(c->beta2 >= 0.0 && c->beta2 < 1.0))
    return fail(ZC_ERR_INVALID, "beta1=%g beta2=%g outside [0, 1)", c->beta1, c->beta2);
  const float eps = static_cast<float>(c->eps);
  if (!std::isfinite(eps) || !(eps >= 1.17549435e-38f))
    return fail(ZC_ERR_INVALID, "eps=%g is no positive fp32 number", c->eps);
  if (!device_step && c->step < 1)
    return fail(ZC_ERR_INVALID, "step=%lld, counted from 1", (long long)c->step);
  return ZC_OK;
}

zc_status do_adamw(const zc_adamw_cfg* c, const zc_adamw_tensor* t, int64_t count,
                   const float* factor, const float* lr, const int64_t* step, hipStream_t s) {
  const bool b8 = c->state == ZC_STATE_8BIT;
  // (a tensor without elements may have no pointers)
  const zc_adamw_tensor* some = std::find_if(t, t + count, [](const zc_adamw_tensor& x) { return x.n > 0; });
  const bool master = some != t + count && some->master != nullptr;
  if (master && c->p_dtype != ZC_BF16)
    return fail(ZC_ERR_INVALID, "master weights go with bf16 weights");
  std::vector<zc::AdamwTensor> list(static_cast<size_t>(count));
  std::vector<Span> spans;
  spans.reserve(static_cast<size_t>(count) * (b8 ? 7 : 5) + 3);
  const int64_t ss = b8 ? 1 : 4;
  for (int64_t i = 0; i < count; ++i) {
    const zc_adamw_tensor& x = t[i];
    const bool none = x.n == 0;
    ZC_CHECK(check_elems(x.n, i));
    if (!std::isfinite(x.weight_decay))
      return fail(ZC_ERR_INVALID, "weight_decay of tensor %lld is not finite", (long long)i);
    if ((x.master != nullptr) != master && !none)
      return fail(ZC_ERR_INVALID, "tensor %lld: master weights are for all tensors or none", (long long)i);
    ZC_CHECK(check_ptr(x.p, "p", none));
    ZC_CHECK(check_ptr(x.g, "g", none));
    ZC_CHECK(check_ptr(x.master, "master", true));
    ZC_CHECK(check_ptr(x.m, "m", none));
    ZC_CHECK(check_ptr(x.v, "v", none));
    if (b8 && !none && (!x.m_scale || !x.v_scale))
      return fail(ZC_ERR_INVALID, "tensor %lld: 8-bit states without scales", (long long)i);
    ZC_CHECK(check_scalar(x.m_scale, 4, "m_scale"));
    ZC_CHECK(check_scalar(x.v_scale, 4, "v_scale"));
    if (!b8 && (x.m_scale || x.v_scale))
      return fail(ZC_ERR_INVALID, "tensor %lld: scales go with 8-bit states", (long long)i);
    list[static_cast<size_t>(i)] = zc::AdamwTensor{x.p, x.g, x.master, x.m, x.v, x.m_scale, x.v_scale,
                                                   x.n, x.weight_decay};
    const int64_t blocks = (x.n + 127) / 128 * 4;
    add_span(spans, x.p, x.n * dtype_size(c->p_dtype), i, "p", true);
    add_span(spans, x.g, x.n * dtype_size(c->g_dtype), i, "g", false);
    add_span(spans, x.master, x.n * 4, i, "master", true);
    add_span(spans, x.m, x.n * ss, i, "m", true);
    add_span(spans, x.v, x.n * ss, i, "v", true);
    add_span(spans, x.m_scale, blocks, i, "m_scale", true);
    add_span(spans, x.v_scale, blocks, i, "v_scale", true);
  }
  add_span(spans, factor, 4, -1, "factor", false);
  add_span(spans, lr, 4, -1, "lr", false);
  add_span(spans, step, 8, -1, "step", false);
  ZC_CHECK(check_spans(spans));
  auto f = [](double v) { return static_cast<float>(v); };
  const zc::AdamwScalars sc{std::log(c->beta1), std::log(c->beta2), c->step, factor, lr, step,
                            f(c->lr), f(c->beta1), f(1.0 - c->beta1), f(c->beta2), f(1.0 - c->beta2),
                            f(c->eps), c->seed};
  ZC_LAUNCH(ZC_PH_ADAMW,
            zc::launch_adamw(list.data(), count, c->p_dtype == ZC_BF16, c->g_dtype == ZC_BF16, master,
                             b8, c->rounding == ZC_ROUND_STOCHASTIC, sc, s),
            "AdamW launch");
  return ZC_OK;
}

// A list too long for the host's memory is refused, not thrown through C.
template <typename F>
zc_status no_throw(F&& f) {
  try {
    return f();
  } catch (...) {
    return fail(ZC_ERR_INVALID, "no host memory for a list of tensors");
  }
}

// Bytes of one set of expert weights in the layer's layout.
int64_t weight_set_bytes(const zc_moe_desc* d, int which) {
  const int64_t n = d->N * d->I * d->d;
  if (mxfp4(d))
    return which == ZC_PACK_GATE_UP ? zc::mx4_weight_bytes(d->N, d->I, d->d)
                                    : zc::mx4_weight_bytes(d->N, d->d, d->I);
  if (const int G = int4_group(d)) return n / 2 + n / G * 2;
  return d->weight_layout == ZC_WEIGHTS_MXFP8 ? n + n / 32 : n * esize(d);
}

zc_status check_weights(const zc_moe_desc* d, const void* wg, const void* wu, const void* wd) {
  const bool opt = d->N == 0;
  ZC_CHECK(check_ptr(wg, "w_gate", opt));
  ZC_CHECK(check_ptr(wu, "w_up", opt));
  ZC_CHECK(check_ptr(wd, "w_down", opt));
  return ZC_OK;
}

}  // namespace

extern "C" {

size_t zc_moe_workspace_size(const zc_moe_desc* desc, int op) {
  if (check_desc(desc) != ZC_OK) return 0;
  switch (op) {
    case ZC_OP_ROUTE: return static_cast<size_t>(route_ws_bytes(desc));
    case ZC_OP_FORWARD: return static_cast<size_t>(fwd_ws_bytes(desc));
    case ZC_OP_BACKWARD: return static_cast<size_t>(bwd_ws_bytes(desc));
    case ZC_OP_LB_LOSS: return static_cast<size_t>(lb_ws_bytes(desc));
    case ZC_OP_ROUTE_STATS: return static_cast<size_t>(stats_ws_bytes(desc));
    case ZC_OP_EXPERTS: return static_cast<size_t>(fwd_ws_bytes(desc));
    default: return 0;
  }
}

size_t zc_moe_saved_size(const zc_moe_desc* desc) {
  if (check_desc(desc) != ZC_OK) return 0;
  return static_cast<size_t>(saved_bytes(desc));
}

zc_status zc_moe_route(const zc_moe_desc* desc, const void* x, const void* w_router,
                       const float* bias, zc_route_buf* r, void* ws, size_t ws_bytes,
                       void* stream) {
  ZC_CHECK(check_desc(desc));
  ZC_CHECK(check_route(r, desc->T == 0));
  ZC_CHECK(check_ptr(bias, "bias"));
  if ((x == nullptr) != (w_router == nullptr) && desc->T > 0)
    return fail(ZC_ERR_INVALID, "x and w_router must both be set or both be NULL");
  ZC_CHECK(check_ptr(x, "x", true));
  ZC_CHECK(check_ptr(w_router, "w_router", true));
  ZC_CHECK(check_ws(ws, ws_bytes, route_ws_bytes(desc)));
  RouteWs w = carve_route(static_cast<char*>(ws), desc);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (desc->dtype == ZC_BF16)
    return do_route<bf16_t>(desc, static_cast<const bf16_t*>(x),
                            static_cast<const bf16_t*>(w_router), bias, r, w, s);
  return do_route<float>(desc, static_cast<const float*>(x), static_cast<const float*>(w_router),
                         bias, r, w, s);
}

zc_status zc_moe_forward(const zc_moe_desc* desc, const void* x, const void* w_router,
                         const float* bias, const void* w_gate, const void* w_up,
                         const void* w_down, void* out, zc_route_buf* r, void* saved, void* ws,
                         size_t ws_bytes, void* stream) {
  ZC_CHECK(check_desc(desc));
  const bool none = desc->T == 0;
  ZC_CHECK(check_route(r, none));
  ZC_CHECK(check_ptr(x, "x", none));
  ZC_CHECK(check_ptr(w_router, "w_router"));
  ZC_CHECK(check_ptr(bias, "bias"));
  ZC_CHECK(check_weights(desc, w_gate, w_up, w_down));
  ZC_CHECK(check_ptr(out, "out", none));
  ZC_CHECK(check_ptr(saved, "saved", true));
  if (saved && desc->weight_layout != ZC_WEIGHTS_ROWMAJOR)
    return fail(ZC_ERR_UNSUPPORTED, "a forward that saves activations needs row-major weights");
  ZC_CHECK(check_ws(ws, ws_bytes, fwd_ws_bytes(desc)));
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* w = static_cast<char*>(ws);
  if (desc->dtype == ZC_BF16)
    return do_forward<bf16_t>(desc, static_cast<const bf16_t*>(x),
                              static_cast<const bf16_t*>(w_router), bias,
                              static_cast<const bf16_t*>(w_gate), static_cast<const bf16_t*>(w_up),
                              static_cast<const bf16_t*>(w_down), static_cast<bf16_t*>(out), r,
                              saved, w, s);
  return do_forward<float>(desc, static_cast<const float*>(x), static_cast<const float*>(w_router),
                           bias, static_cast<const float*>(w_gate),
                           static_cast<const float*>(w_up), static_cast<const float*>(w_down),
                           static_cast<float*>(out), r, saved, w, s);
}

zc_status zc_moe_experts(const zc_moe_desc* desc, const void* x, const zc_route_buf* r,
                         const void* w_gate, const void* w_up, const void* w_down,
                         const uint8_t* x_codes, const uint8_t* x_scales, void* out, void* ws,
                         size_t ws_bytes, void* stream) {
  ZC_CHECK(check_desc(desc));
  const bool none = desc->T == 0;
  if (!r) return fail(ZC_ERR_INVALID, "route buffer is NULL");
  ZC_CHECK(check_ptr(r->topk_idx, "r->topk_idx", none));
  ZC_CHECK(check_ptr(r->topk_gate, "r->topk_gate", none));
  ZC_CHECK(check_ptr(r->offsets, "r->offsets"));
  ZC_CHECK(check_ptr(r->perm, "r->perm", none));
  ZC_CHECK(check_ptr(r->inv, "r->inv", none));
  ZC_CHECK(check_ptr(x, "x", none));
  ZC_CHECK(check_weights(desc, w_gate, w_up, w_down));
  ZC_CHECK(check_ptr(x_codes, "x_codes", true));
  ZC_CHECK(check_ptr(x_scales, "x_scales", true));
  if ((x_codes == nullptr) != (x_scales == nullptr))
    return fail(ZC_ERR_INVALID, "x_codes and x_scales must both be set or both be NULL");
  if (x_codes && desc->weight_layout != ZC_WEIGHTS_MXFP8 && !mxfp4(desc))
    return fail(ZC_ERR_INVALID, "x_codes go with MXFP8 or MXFP4 weights");
  ZC_CHECK(check_ptr(out, "out", none));
  const int64_t need = fwd_ws_bytes(desc);
  ZC_CHECK(check_ws(ws, ws_bytes, need));
  const int64_t n = desc->T * desc->d, b = n * esize(desc), k = desc->T * desc->K;
  const int64_t wb = weight_set_bytes(desc, ZC_PACK_GATE_UP);
  const Range in[] = {{w_gate, wb, "w_gate", false}, {w_up, wb, "w_up", false},
                      {w_down, weight_set_bytes(desc, ZC_PACK_DOWN), "w_down", false},
                      {x, b, "x", false}, {x_codes, mxfp4_a4(desc) ? n / 2 : n, "x_codes", false},
                      {x_scales, n / 32, "x_scales", false}, {r->topk_idx, 4 * k, "r->topk_idx", false},
                      {r->topk_gate, 4 * k, "r->topk_gate", false},
                      {r->offsets, 4 * (desc->N + 1), "r->offsets", false},
                      {r->perm, 4 * k, "r->perm", false}, {r->inv, 4 * k, "r->inv", false}};
  const Range outs[] = {{out, b, "out", false}, {ws, need, "ws", false}};
  ZC_CHECK(check_overlap(outs, 2, in, 11));
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* w = static_cast<char*>(ws);
  if (desc->dtype == ZC_BF16)
    return do_routed_experts<bf16_t>(
        desc, static_cast<const bf16_t*>(x), static_cast<const bf16_t*>(w_gate),
        static_cast<const bf16_t*>(w_up), static_cast<const bf16_t*>(w_down),
        static_cast<bf16_t*>(out), r, x_codes, x_scales, w, s);
  return do_routed_experts<float>(desc, static_cast<const float*>(x),
                                  static_cast<const float*>(w_gate),
                                  static_cast<const float*>(w_up),
                                  static_cast<const float*>(w_down), static_cast<float*>(out), r,
                                  nullptr, nullptr, w, s);
}

zc_status zc_moe_forward_noalloc(const zc_moe_desc* desc, const void* x, const void* w_router,
                                 const float* bias, const void* w_gate, const void* w_up,
                                 const void* w_down, void* out, zc_route_buf* r, void* stream) {
  ZC_CHECK(check_desc(desc));
  const int64_t need = fwd_ws_bytes(desc);
  if (need > static_cast<int64_t>(kNoAllocScratch))
    return fail(ZC_ERR_WORKSPACE,
                "the allocation-free forward holds %zu bytes of scratch per device; this layer "
                "needs %lld (zc_moe_workspace_size(desc, ZC_OP_FORWARD))",
                kNoAllocScratch, (long long)need);
  void* ws = nullptr;
  ZC_CHECK(scratch_ptr(&ws));
  t_no_events = true;
  const zc_status st = zc_moe_forward(desc, x, w_router, bias, w_gate, w_up, w_down, out, r,
                                      nullptr, ws, kNoAllocScratch, stream);
  t_no_events = false;
  return st;
}

zc_status zc_moe_backward(const zc_moe_desc* desc, const void* x, const void* w_router,
                          const void* w_gate, const void* w_up, const void* w_down,
                          const zc_route_buf* r, const void* saved, const void* dout, void* dx,
                          void* dw_router, void* dw_gate, void* dw_up, void* dw_down,
                          const zc_lb_cfg* lb, void* ws, size_t ws_bytes, void* stream) {
  return zc_moe_backward_scores(desc, x, w_router, w_gate, w_up, w_down, r, saved, dout, dx,
                                dw_router, dw_gate, dw_up, dw_down, lb, nullptr, ws, ws_bytes,
                                stream);
}

zc_status zc_moe_backward_scores(const zc_moe_desc* desc, const void* x, const void* w_router,
                                 const void* w_gate, const void* w_up, const void* w_down,
                                 const zc_route_buf* r, const void* saved, const void* dout,
                                 void* dx, void* dw_router, void* dw_gate, void* dw_up,
                                 void* dw_down, const zc_lb_cfg* lb, const float* dlogits,
                                 void* ws, size_t ws_bytes, void* stream) {
  ZC_CHECK(check_desc(desc));
  if (desc->weight_layout != ZC_WEIGHTS_ROWMAJOR)
    return fail(ZC_ERR_UNSUPPORTED, "the backward needs row-major weights");
  const bool none = desc->T == 0;
  ZC_CHECK(check_route(r, none));
  ZC_CHECK(check_ptr(x, "x", none));
  ZC_CHECK(check_ptr(w_router, "w_router"));
  ZC_CHECK(check_weights(desc, w_gate, w_up, w_down));
  ZC_CHECK(check_ptr(saved, "saved", none));
  ZC_CHECK(check_ptr(dout, "dout", none));
  ZC_CHECK(check_ptr(dx, "dx", none));
  ZC_CHECK(check_ptr(dw_router, "dw_router"));
  ZC_CHECK(check_weights(desc, dw_gate, dw_up, dw_down));
  if (lb) ZC_CHECK(check_lb(desc, lb));
  ZC_CHECK(check_ptr(dlogits, "dlogits", true));
  ZC_CHECK(check_ws(ws, ws_bytes, bwd_ws_bytes(desc)));
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* w = static_cast<char*>(ws);
  if (desc->dtype == ZC_BF16)
    return do_backward<bf16_t>(
        desc, static_cast<const bf16_t*>(x), static_cast<const bf16_t*>(w_router),
        static_cast<const bf16_t*>(w_gate), static_cast<const bf16_t*>(w_up),
        static_cast<const bf16_t*>(w_down), r, saved, static_cast<const bf16_t*>(dout),
        static_cast<bf16_t*>(dx), static_cast<bf16_t*>(dw_router), static_cast<bf16_t*>(dw_gate),
        static_cast<bf16_t*>(dw_up), static_cast<bf16_t*>(dw_down), lb, dlogits, w, s);
  return do_backward<float>(desc, static_cast<const float*>(x), static_cast<const float*>(w_router),
                            static_cast<const float*>(w_gate), static_cast<const float*>(w_up),
                            static_cast<const float*>(w_down), r, saved,
                            static_cast<const float*>(dout), static_cast<float*>(dx),
                            static_cast<float*>(dw_router), static_cast<float*>(dw_gate),
                            static_cast<float*>(dw_up), static_cast<float*>(dw_down), lb, dlogits, w, s);
}

zc_status zc_moe_lb_loss(const zc_moe_desc* desc, const zc_lb_cfg* lb, const zc_route_buf* r,
                         double* out, void* ws, size_t ws_bytes, void* stream) {
  ZC_CHECK(check_desc(desc));
  ZC_CHECK(check_lb(desc, lb));
  if (!r) return fail(ZC_ERR_INVALID, "route buffer is NULL");
  ZC_CHECK(check_ptr(r->logits, "r->logits", desc->T == 0));
  ZC_CHECK(check_ptr(r->counts, "r->counts"));
  ZC_CHECK(check_ptr(out, "out"));
  ZC_CHECK(check_ws(ws, ws_bytes, lb_ws_bytes(desc)));
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int E = static_cast<int>(desc->N + desc->Z);
  ZC_LAUNCH(ZC_PH_LB_LOSS,
            zc::launch_lb_loss(r->logits, r->counts, static_cast<int>(desc->T),
                               static_cast<int>(desc->N), E, static_cast<int>(desc->K),
                               static_cast<int>(lb->D), lb->K_e, lb->alpha, out, ws, s),
            "load-balance loss launch");
  return ZC_OK;
}

size_t zc_moe_seq_balance_workspace_size(const zc_moe_desc* desc, int64_t S) {
  if (check_desc(desc) != ZC_OK || check_seqs(desc, S) != ZC_OK) return 0;
  return zc::seq_balance_scratch_bytes(desc->T, desc->N + desc->Z, desc->K, S);
}

zc_status zc_moe_seq_balance(const zc_moe_desc* desc, const zc_lb_cfg* lb, const zc_route_buf* r,
                             int64_t S, const int32_t* cu_seqlens, const uint8_t* mask,
                             float* loss, int32_t* counts, float* dlogits, void* ws,
                             size_t ws_bytes, void* stream) {
  ZC_CHECK(check_desc(desc));
  ZC_CHECK(check_lb(desc, lb));
  ZC_CHECK(check_seqs(desc, S));
  const bool none = desc->T == 0;
  if (!r) return fail(ZC_ERR_INVALID, "route buffer is NULL");
  ZC_CHECK(check_ptr(r->logits, "r->logits", none));
  ZC_CHECK(check_ptr(r->topk_idx, "r->topk_idx", none));
  if (!cu_seqlens && S != 1)
    return fail(ZC_ERR_INVALID, "S=%lld sequences need cu_seqlens", (long long)S);
  ZC_CHECK(check_ptr(cu_seqlens, "cu_seqlens", true));
  ZC_CHECK(check_ptr(mask, "mask", true));
  ZC_CHECK(check_ptr(loss, "loss"));
  ZC_CHECK(check_ptr(counts, "counts"));
  ZC_CHECK(check_ptr(dlogits, "dlogits", true));
  const int64_t E = desc->N + desc->Z, T = desc->T;
  const int64_t need = static_cast<int64_t>(zc::seq_balance_scratch_bytes(T, E, desc->K, S));
  ZC_CHECK(check_ws(ws, ws_bytes, need));
  const Range in[] = {{r->logits, 4 * T * E, "r->logits", false},
                      {r->topk_idx, 4 * T * desc->K, "r->topk_idx", false},
                      {cu_seqlens, 4 * (S + 1), "cu_seqlens", false}, {mask, T, "mask", false}};
  const Range out[] = {{loss, 4 * (S + 1), "loss", false}, {counts, 4 * S * E, "counts", false},
                       {dlogits, 4 * T * E, "dlogits", false}, {ws, need, "ws", false}};
  ZC_CHECK(check_overlap(out, 4, in, 4));
  hipStream_t s = static_cast<hipStream_t>(stream);
  ZC_LAUNCH(ZC_PH_SEQ_BALANCE,
            zc::launch_seq_balance(r->logits, r->topk_idx, static_cast<int>(T),
                                   static_cast<int>(desc->N), static_cast<int>(E),
                                   static_cast<int>(desc->K), static_cast<int>(lb->D), lb->K_e,
                                   lb->alpha, static_cast<int>(S), cu_seqlens, mask, loss, counts,
                                   dlogits, ws, s),
            "balance loss launch");
  return ZC_OK;
}

zc_status zc_moe_route_stats(const zc_moe_desc* desc, const zc_route_buf* r, int32_t* hist,
                             double* moments, void* ws, size_t ws_bytes, void* stream) {
  ZC_CHECK(check_desc(desc));
  if (!r) return fail(ZC_ERR_INVALID, "route buffer is NULL");
  ZC_CHECK(check_ptr(r->topk_idx, "r->topk_idx", desc->T == 0));
  ZC_CHECK(check_ptr(hist, "hist"));
  ZC_CHECK(check_ptr(moments, "moments"));
  ZC_CHECK(check_ws(ws, ws_bytes, stats_ws_bytes(desc)));
  hipStream_t s = static_cast<hipStream_t>(stream);
  ZC_LAUNCH(ZC_PH_ROUTE_STATS,
            zc::launch_route_stats(r->topk_idx, static_cast<int>(desc->T),
                                   static_cast<int>(desc->N), static_cast<int>(desc->K), hist,
                                   moments, ws, s),
            "routing statistics launch");
  return ZC_OK;
}

zc_status zc_moe_accumulate_counts(int64_t E, const int32_t* counts, int32_t* acc, void* stream) {
  if (E < 1 || E > 1024) return fail(ZC_ERR_INVALID, "E=%lld outside 1..1024", (long long)E);
  ZC_CHECK(check_ptr(counts, "counts"));
  ZC_CHECK(check_ptr(acc, "acc"));
  if (counts == acc) return fail(ZC_ERR_INVALID, "counts and acc are the same buffer");
  hipStream_t s = static_cast<hipStream_t>(stream);
  ZC_LAUNCH(ZC_PH_ACCUMULATE, zc::launch_accumulate_counts(counts, static_cast<int>(E), acc, s),
            "count accumulation launch");
  return ZC_OK;
}

zc_status zc_moe_pack_weights(const zc_moe_desc* desc, int which, const void* src, void* dst,
                              void* stream) {
  ZC_CHECK(check_desc(desc));
  if (desc->dtype != ZC_BF16) return fail(ZC_ERR_UNSUPPORTED, "packed weights need a bf16 layer");
  if (desc->d % 256 || desc->I % 256)
    return fail(ZC_ERR_UNSUPPORTED, "packed weights need d and I multiples of 256 (d=%lld I=%lld)",
                (long long)desc->d, (long long)desc->I);
  if (which != ZC_PACK_GATE_UP && which != ZC_PACK_DOWN)
    return fail(ZC_ERR_INVALID, "which=%d is neither ZC_PACK_GATE_UP nor ZC_PACK_DOWN", which);
  const bool opt = desc->N == 0;
  ZC_CHECK(check_ptr(src, "src", opt));
  ZC_CHECK(check_ptr(dst, "dst", opt));
  const int64_t bytes = desc->N * desc->I * desc->d * 2;
  const char* a = static_cast<const char*>(src);
  const char* b = static_cast<const char*>(dst);
  if (bytes > 0 && a < b + bytes && b < a + bytes)
    return fail(ZC_ERR_INVALID, "src and dst overlap");
  if (desc->N == 0) return ZC_OK;
  const int R = static_cast<int>(which == ZC_PACK_GATE_UP ? desc->I : desc->d);
  const int C = static_cast<int>(which == ZC_PACK_GATE_UP ? desc->d : desc->I);
  hipError_t e = zc::launch_pack_weights(static_cast<const bf16_t*>(src), static_cast<bf16_t*>(dst),
                                         desc->N, R, C, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "weight packing launch");
  return ZC_OK;
}

size_t zc_moe_quantized_weight_bytes(const zc_moe_desc* desc) {
  if (check_desc(desc) != ZC_OK) return 0;
  const int64_t n = desc->N * desc->I * desc->d;
  return static_cast<size_t>(n + n / 32);
}

zc_status zc_moe_quantize_weights(const zc_moe_desc* desc, int which, const void* src, void* dst,
                                  void* stream) {
  ZC_CHECK(check_desc(desc));
  ZC_CHECK(check_mxfp8(desc));
  if (which != ZC_PACK_GATE_UP && which != ZC_PACK_DOWN)
    return fail(ZC_ERR_INVALID, "which=%d is neither ZC_PACK_GATE_UP nor ZC_PACK_DOWN", which);
  const bool opt = desc->N == 0;
  ZC_CHECK(check_ptr(src, "src", opt));
  ZC_CHECK(check_ptr(dst, "dst", opt));
  const int64_t sbytes = desc->N * desc->I * desc->d * 2;
  const int64_t dbytes = static_cast<int64_t>(zc_moe_quantized_weight_bytes(desc));
  const char* a = static_cast<const char*>(src);
  const char* b = static_cast<const char*>(dst);
  if (sbytes > 0 && a < b + dbytes && b < a + sbytes)
    return fail(ZC_ERR_INVALID, "src and dst overlap");
  if (desc->N == 0) return ZC_OK;
  const int R = static_cast<int>(which == ZC_PACK_GATE_UP ? desc->I : desc->d);
  const int C = static_cast<int>(which == ZC_PACK_GATE_UP ? desc->d : desc->I);
  hipError_t e = zc::launch_mxq_weights(static_cast<const bf16_t*>(src), static_cast<uint8_t*>(dst),
                                        desc->N, R, C, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "weight quantization launch");
  return ZC_OK;
}

size_t zc_moe_int4_weight_bytes(const zc_moe_desc* desc) {
  if (check_desc(desc) != ZC_OK || !int4_group(desc)) return 0;
  return static_cast<size_t>(weight_set_bytes(desc, ZC_PACK_GATE_UP));
}

namespace {
// A call on one set of 4-bit weights: its sizes R, C and G.
zc_status int4_set(const zc_moe_desc* d, int which, int* R, int* C, int* G) {
  ZC_CHECK(check_desc(d));
  *G = int4_group(d);
  if (!*G) return fail(ZC_ERR_INVALID, "weight_layout %d is no INT4 layout", d->weight_layout);
  if (which != ZC_PACK_GATE_UP && which != ZC_PACK_DOWN)
    return fail(ZC_ERR_INVALID, "which=%d is neither ZC_PACK_GATE_UP nor ZC_PACK_DOWN", which);
  *R = static_cast<int>(which == ZC_PACK_GATE_UP ? d->I : d->d);
  *C = static_cast<int>(which == ZC_PACK_GATE_UP ? d->d : d->I);
  return ZC_OK;
}
}  // namespace

zc_status zc_moe_int4_quantize(const zc_moe_desc* desc, int which, const void* src, uint8_t* codes,
                               void* scales, void* stream) {
  int R, C, G;
  ZC_CHECK(int4_set(desc, which, &R, &C, &G));
  const bool opt = desc->N == 0;
  ZC_CHECK(check_ptr(src, "src", opt));
  ZC_CHECK(check_ptr(codes, "codes", opt));
  ZC_CHECK(check_ptr(scales, "scales", opt));
  const int64_t n = desc->N * desc->I * desc->d;
  const Range in[] = {{src, 2 * n, "src", false}};
  const Range out[] = {{codes, n / 2, "codes", false}, {scales, n / G * 2, "scales", false}};
  ZC_CHECK(check_overlap(out, 2, in, 1));
  if (opt) return ZC_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  ZC_LAUNCH(ZC_PH_QUANTIZE,
            zc::launch_int4_quantize(static_cast<const bf16_t*>(src), codes,
                                     static_cast<bf16_t*>(scales), desc->N, R, C, G, s),
            "4-bit quantization launch");
  return ZC_OK;
}

zc_status zc_moe_int4_pack(const zc_moe_desc* desc, int which, const uint8_t* codes,
                           const void* scales, void* dst, void* stream) {
  int R, C, G;
  ZC_CHECK(int4_set(desc, which, &R, &C, &G));
  const bool opt = desc->N == 0;
  ZC_CHECK(check_ptr(codes, "codes", opt));
  ZC_CHECK(check_ptr(scales, "scales", opt));
  ZC_CHECK(check_ptr(dst, "dst", opt));
  const int64_t n = desc->N * desc->I * desc->d;
  const Range in[] = {{codes, n / 2, "codes", false}, {scales, n / G * 2, "scales", false}};
  const Range out[] = {{dst, n / 2 + n / G * 2, "dst", false}};
  ZC_CHECK(check_overlap(out, 1, in, 2));
  if (opt) return ZC_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  ZC_LAUNCH(ZC_PH_QUANTIZE,
            zc::launch_int4_pack(codes, static_cast<const bf16_t*>(scales),
                                 static_cast<uint8_t*>(dst), desc->N, R, C, G, s),
            "4-bit packing launch");
  return ZC_OK;
}

zc_status zc_mxfp4_quantize(int64_t R, int64_t C, int dtype, const void* src, uint8_t* codes,
                            uint8_t* scales, void* values, void* stream) {
  ZC_CHECK(check_dtype(dtype, "dtype"));
  if (R < 0 || C < 1) return fail(ZC_ERR_INVALID, "bad sizes R=%lld C=%lld", (long long)R, (long long)C);
  if (C % 32 || C >= (int64_t(1) << 31) || R >= (int64_t(1) << 40) / C)
    return fail(ZC_ERR_UNSUPPORTED, "MXFP4 rows need C a multiple of 32 and R*C below 2^40 (R=%lld C=%lld)",
                (long long)R, (long long)C);
  const bool none = R == 0;
  ZC_CHECK(check_ptr(src, "src", none));
  ZC_CHECK(check_ptr(codes, "codes", none));
  ZC_CHECK(check_ptr(scales, "scales", none));
  ZC_CHECK(check_ptr(values, "values", true));
  const int64_t n = R * C, b = n * dtype_size(dtype);
  const Range in[] = {{src, b, "src", true}};
  const Range out[] = {{codes, n / 2, "codes", false}, {scales, n / 32, "scales", false},
                       {values, b, "values", true}};
  ZC_CHECK(check_overlap(out, 3, in, 1));
  hipStream_t s = static_cast<hipStream_t>(stream);
  ZC_LAUNCH(ZC_PH_QUANTIZE,
            dtype == ZC_BF16
                ? zc::launch_mx4_rows(static_cast<const bf16_t*>(src), R, C, codes, scales,
                                      static_cast<bf16_t*>(values), s)
                : zc::launch_mx4_rows(static_cast<const float*>(src), R, C, codes, scales,
                                      static_cast<float*>(values), s),
            "MXFP4 quantization launch");
  return ZC_OK;
}

size_t zc_moe_mxfp4_weight_bytes(const zc_moe_desc* desc, int which) {
  if (check_desc(desc) != ZC_OK || !mxfp4(desc) || (which != ZC_PACK_GATE_UP && which != ZC_PACK_DOWN))
    return 0;
  return static_cast<size_t>(weight_set_bytes(desc, which));
}

zc_status zc_moe_mxfp4_pack(const zc_moe_desc* desc, int which, const uint8_t* codes,
                            const uint8_t* scales, void* dst, void* stream) {
  ZC_CHECK(check_desc(desc));
  if (!mxfp4(desc)) return fail(ZC_ERR_INVALID, "weight_layout %d is no MXFP4 layout", desc->weight_layout);
  if (which != ZC_PACK_GATE_UP && which != ZC_PACK_DOWN)
    return fail(ZC_ERR_INVALID, "which=%d is neither ZC_PACK_GATE_UP nor ZC_PACK_DOWN", which);
  const bool opt = desc->N == 0;
  ZC_CHECK(check_ptr(codes, "codes", opt));
  ZC_CHECK(check_ptr(scales, "scales", opt));
  ZC_CHECK(check_ptr(dst, "dst", opt));
  const int64_t n = desc->N * desc->I * desc->d;
  const Range in[] = {{codes, n / 2, "codes", false}, {scales, n / 32, "scales", false}};
  const Range out[] = {{dst, weight_set_bytes(desc, which), "dst", false}};
  ZC_CHECK(check_overlap(out, 1, in, 2));
  if (opt) return ZC_OK;
  const int R = static_cast<int>(which == ZC_PACK_GATE_UP ? desc->I : desc->d);
  const int C = static_cast<int>(which == ZC_PACK_GATE_UP ? desc->d : desc->I);
  hipStream_t s = static_cast<hipStream_t>(stream);
  ZC_LAUNCH(ZC_PH_QUANTIZE,
            zc::launch_mx4_pack(which == ZC_PACK_DOWN, codes, scales, static_cast<uint8_t*>(dst), desc->N, R, C, s),
            "MXFP4 packing launch");
  return ZC_OK;
}

zc_status zc_moe_pid_update(int64_t N, int64_t Z, int64_t K, const int32_t* counts, int64_t T_all,
                            double mu, double K_e, float* bias, void* stream) {
  if (N < 0 || Z < 0 || N + Z < 1 || N + Z > 1024)
    return fail(ZC_ERR_INVALID, "N=%lld Z=%lld: need N, Z >= 0 and 1 <= N+Z <= 1024",
                (long long)N, (long long)Z);
  if (K < 1 || T_all < 1) return fail(ZC_ERR_INVALID, "K and T_all must be >= 1");
  if (!std::isfinite(mu) || !std::isfinite(K_e)) return fail(ZC_ERR_INVALID, "mu or K_e not finite");
  ZC_CHECK(check_ptr(counts, "counts"));
  ZC_CHECK(check_ptr(bias, "bias"));
  hipStream_t s = static_cast<hipStream_t>(stream);
  ZC_LAUNCH(ZC_PH_BIAS_UPDATE, zc::launch_pid(static_cast<int>(N), static_cast<int>(K), counts, T_all, mu, K_e, bias, s),
         "bias update launch");
  return ZC_OK;
}

zc_status zc_rmsnorm_forward(const zc_norm_desc* desc, const void* x, const void* res,
                             const void* gamma, void* r, void* y, float* rstd, uint8_t* codes,
                             uint8_t* scales, void* stream) {
  ZC_CHECK(check_norm(desc));
  const bool none = desc->T == 0;
  ZC_CHECK(check_ptr(x, "x", none));
  ZC_CHECK(check_ptr(res, "res", true));
  ZC_CHECK(check_ptr(gamma, "gamma"));
  ZC_CHECK(check_ptr(r, "r", true));
  ZC_CHECK(check_ptr(y, "y", none));
  ZC_CHECK(check_ptr(rstd, "rstd", true));
  ZC_CHECK(check_ptr(codes, "codes", true));
  ZC_CHECK(check_ptr(scales, "scales", true));
  if ((codes == nullptr) != (scales == nullptr))
    return fail(ZC_ERR_INVALID, "codes and scales must both be set or both be NULL");
  if (codes && (desc->dtype != ZC_BF16 || desc->d % 128))
    return fail(ZC_ERR_UNSUPPORTED, "MXFP8 output needs bf16 rows and d a multiple of 128 (d=%lld)",
                (long long)desc->d);
  const int64_t n = desc->T * desc->d, b = n * norm_esize(desc);
  const Range in[] = {{x, b, "x", true}, {res, b, "res", true},
                      {gamma, desc->d * norm_esize(desc), "gamma", false}};
  const Range out[] = {{r, b, "r", true}, {y, b, "y", true}, {rstd, 4 * desc->T, "rstd", false},
                       {codes, n, "codes", false}, {scales, n / 32, "scales", false}};
  ZC_CHECK(check_overlap(out, 5, in, 3));
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int d = static_cast<int>(desc->d);
  if (desc->dtype == ZC_BF16)
    ZC_LAUNCH(ZC_PH_NORM,
              zc::launch_norm_fwd(static_cast<const bf16_t*>(x), static_cast<const bf16_t*>(res),
                                  static_cast<const bf16_t*>(gamma), static_cast<bf16_t*>(r),
                                  static_cast<bf16_t*>(y), rstd, codes, scales, desc->T, d,
                                  desc->eps, s),
              "norm launch");
  else
    ZC_LAUNCH(ZC_PH_NORM,
              zc::launch_norm_fwd(static_cast<const float*>(x), static_cast<const float*>(res),
                                  static_cast<const float*>(gamma), static_cast<float*>(r),
                                  static_cast<float*>(y), rstd, codes, scales, desc->T, d,
                                  desc->eps, s),
              "norm launch");
  return ZC_OK;
}

size_t zc_rmsnorm_workspace_size(const zc_norm_desc* desc) {
  if (check_norm(desc) != ZC_OK) return 0;
  return static_cast<size_t>(norm_ws_bytes(desc));
}

zc_status zc_rmsnorm_backward(const zc_norm_desc* desc, const void* dy, const void* r,
                              const void* gamma, const float* rstd, const void* dres, void* dr,
                              void* dgamma, void* ws, size_t ws_bytes, void* stream) {
  ZC_CHECK(check_norm(desc));
  const bool none = desc->T == 0;
  ZC_CHECK(check_ptr(dy, "dy", none));
  ZC_CHECK(check_ptr(r, "r", none));
  ZC_CHECK(check_ptr(gamma, "gamma"));
  ZC_CHECK(check_ptr(rstd, "rstd", none));
  ZC_CHECK(check_ptr(dres, "dres", true));
  ZC_CHECK(check_ptr(dr, "dr", none));
  ZC_CHECK(check_ptr(dgamma, "dgamma"));
  ZC_CHECK(check_ws(ws, ws_bytes, norm_ws_bytes(desc)));
  const int64_t es = norm_esize(desc), b = desc->T * desc->d * es;
  const Range in[] = {{dy, b, "dy", true}, {r, b, "r", true}, {dres, b, "dres", true},
                      {gamma, desc->d * es, "gamma", false}, {rstd, 4 * desc->T, "rstd", false}};
  const Range out[] = {{dr, b, "dr", true}, {dgamma, desc->d * es, "dgamma", false},
                       {ws, norm_ws_bytes(desc), "ws", false}};
  ZC_CHECK(check_overlap(out, 3, in, 5));
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int d = static_cast<int>(desc->d);
  float* part = static_cast<float*>(ws);
  if (desc->dtype == ZC_BF16)
    ZC_LAUNCH(ZC_PH_NORM_BWD,
              zc::launch_norm_bwd(static_cast<const bf16_t*>(dy), static_cast<const bf16_t*>(r),
                                  static_cast<const bf16_t*>(gamma), rstd,
                                  static_cast<const bf16_t*>(dres), static_cast<bf16_t*>(dr),
                                  static_cast<bf16_t*>(dgamma), part, desc->T, d, s),
              "norm backward launch");
  else
    ZC_LAUNCH(ZC_PH_NORM_BWD,
              zc::launch_norm_bwd(static_cast<const float*>(dy), static_cast<const float*>(r),
                                  static_cast<const float*>(gamma), rstd,
                                  static_cast<const float*>(dres), static_cast<float*>(dr),
                                  static_cast<float*>(dgamma), part, desc->T, d, s),
              "norm backward launch");
  return ZC_OK;
}

size_t zc_grad_norm_workspace_size(const zc_grad_tensor* tensors, int64_t count, int g_dtype) {
  size_t bytes = 0;
  no_throw([&]() -> zc_status {
    ZC_CHECK(check_dtype(g_dtype, "g_dtype"));
    ZC_CHECK(check_count(tensors, count));
    for (int64_t i = 0; i < count; ++i) ZC_CHECK(check_elems(tensors[i].n, i));
    bytes = static_cast<size_t>(Grads(tensors, count, g_dtype == ZC_BF16).ws_bytes);
    return ZC_OK;
  });
  return bytes;
}

zc_status zc_grad_norm(const zc_grad_tensor* tensors, int64_t count, int g_dtype, double max_norm,
                       float* out, int64_t* step, void* ws, size_t ws_bytes, void* stream) {
  ZC_CHECK(check_grads(tensors, count, g_dtype));
  if (!(max_norm > 0.0)) return fail(ZC_ERR_INVALID, "max_norm=%g is not positive", max_norm);
  if (!out) return fail(ZC_ERR_INVALID, "out is NULL");
  ZC_CHECK(check_scalar(out, 4, "out"));
  ZC_CHECK(check_scalar(step, 8, "step"));
  return no_throw([&] {
    return do_grad_norm(tensors, count, g_dtype, max_norm, out, step, ws, ws_bytes,
                        static_cast<hipStream_t>(stream));
  });
}

zc_status zc_adamw_step(const zc_adamw_cfg* cfg, const zc_adamw_tensor* tensors, int64_t count,
                        const float* factor, const float* lr, const int64_t* step, void* stream) {
  ZC_CHECK(check_adamw(cfg, step != nullptr));
  ZC_CHECK(check_count(tensors, count));
  ZC_CHECK(check_scalar(factor, 4, "factor"));
  ZC_CHECK(check_scalar(lr, 4, "lr"));
  ZC_CHECK(check_scalar(step, 8, "step"));
  return no_throw([&] {
    return do_adamw(cfg, tensors, count, factor, lr, step, static_cast<hipStream_t>(stream));
  });
}

zc_status zc_moe_profile(int on) {
  std::lock_guard<std::mutex> lk(g_prof_mu);
  if (!on) drop_records();
  g_prof_on.store(on != 0);
  return ZC_OK;
}

zc_status zc_moe_profile_read(double* total_ms, int32_t* count) {
  if (!total_ms || !count) return fail(ZC_ERR_INVALID, "total_ms and count must be host arrays");
  for (int i = 0; i < ZC_NUM_PHASES; ++i) {
    total_ms[i] = 0.0;
    count[i] = 0;
  }
  std::lock_guard<std::mutex> lk(g_prof_mu);
  zc_status st = ZC_OK;
  for (auto& r : g_prof_recs) {
    float ms = 0.f;
    hipError_t e = hipEventSynchronize(r.b);
    if (e == hipSuccess) e = hipEventElapsedTime(&ms, r.a, r.b);
    if (e != hipSuccess) {
      st = hip_fail(e, "reading kernel timing events");
      continue;
    }
    total_ms[r.phase] += ms;
    count[r.phase] += 1;
  }
  drop_records();
  return st;
}

const char* zc_moe_phase_name(int phase) {
  static const char* names[ZC_NUM_PHASES] = {
      "router_gemm", "topk", "dispatch", "gate_up_gemm", "down_gemm", "combine",
      "bwd_combine", "bwd_down_dh", "bwd_down_dw", "bwd_gate_up_dx", "bwd_gate_up_dw",
      "bwd_router_dw", "bwd_router_dx", "bwd_dx_gather", "bias_update", "tile_offsets",
      "lb_loss", "lb_coef", "route_stats", "accumulate_counts", "quantize", "bwd_gather",
      "norm", "norm_bwd", "seq_balance", "grad_norm", "adamw"};
  return (phase >= 0 && phase < ZC_NUM_PHASES) ? names[phase] : "";
}

const char* zc_status_string(zc_status s) {
  // callers from C or Python may pass any int: read it as one, never as an
  // out-of-range value of the enum type
  int v = 0;
  static_assert(sizeof v == sizeof s, "zc_status is an int");
  std::memcpy(&v, &s, sizeof v);
  switch (v) {
    case ZC_OK: return "ok";
    case ZC_ERR_INVALID: return "invalid argument";
    case ZC_ERR_UNSUPPORTED: return "unsupported shape";
    case ZC_ERR_WORKSPACE: return "workspace too small";
    case ZC_ERR_HIP: return "HIP error";
  }
  return "unknown status";
}

const char* zc_last_error(void) { return g_last_error.c_str(); }

}  // extern "C"
