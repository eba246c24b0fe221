// Forward expert GEMMs on MXFP4 weights, and the MXFP4 quantizer.
//
//   gate/up: h[p][n] = silu(x[tok(p)] . W_g[e][n]) * (x[tok(p)] . W_u[e][n])
//   down:    y[p][n] = h[p] . W_d[e][n]
// for the rows p of expert e's segment of the dispatch order.  A weight is an E2M1
// code (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign) times a power of two that 32
// reduction steps share (E8M0): the OCP Microscaling format MXFP4.  x and h are
// MXFP8 or MXFP4 rows; h is quantized from its fp32 values where they are made.
// The matrix cores take all of it as it is (v_mfma_scale_f32_16x16x128_f8f6f4:
// products and sums exact or in fp32, scales applied inside), so a weight costs no
// vector instruction, and two 4-bit operands run at twice the rate of 8-bit ones.
//
// Operands of a 16x16x128 step (measured on MI355X): lane l holds row (column) l %
// 16; with g = l / 16, a 4-bit operand's 16 bytes are steps 32 g .. 32 g + 31, low
// half of a byte first; an 8-bit operand's bytes 0..15 are steps 16 g .. and its
// bytes 16..31 steps 64 + 16 g ..; in both the lane's scale is that of block g (steps
// 32 g ..) of its row.
//
// Weights of one set (N matrices [R][C]): codes [N][R/16][C/128][lane][16 bytes]:
// 1 KB holds 16 output columns and 128 reduction steps, a wave's operand as it lies;
// then scales [N][R/16][ceil(C/512)][lane][4 blocks of 128 steps], E8M0: a lane's
// four scales of 512 steps in one word.  Of 32 output columns the even ones are the
// first 16, the odd ones the next: a lane then ends with two neighbours, which make a
// byte of two 4-bit codes.
#include "zc_common.h"

namespace zc {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 128;  // reduction steps of a code block

enum { MX_SWIGLU = 0, MX_STORE = 1 };

typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));

struct Mx4Params {
  int N, ncols, K;          // experts, output columns (I or d), reduction length (d or I)
  const int32_t* total;     // number of row tiles
  const RowTile* tiles;     // one of each (as many as the grid has row tiles)
  const uint8_t* A;         // codes: x' [T][...] gathered through perm, or h' [P][...]
  const uint8_t* As;        // their scales, [rows][K/32]
  const int32_t* perm;      // gate/up only
  int kdiv;                 // K of the layer (slot -> token)
  const uint8_t* B;         // W_g or W_d
  const uint8_t* B2;        // W_u (gate/up)
  uint8_t* hq;              // gate/up output: codes [P][I] or [P][I/2] ...
  uint8_t* hs;              // ... and scales [P][I/32]
  float* y;                 // down output [P][d]
  int64_t per_xcd;          // tiles of an XCD, at most
  int log_run;              // runs of consecutive tiles on one XCD
};

// silu(a) = a / (1 + e^-a) with the hardware reciprocal (about 1 ulp): the result
// is rounded to 8 or 4 bits right after.
__device__ __forceinline__ float silu_f(float a) {
  return a * __builtin_amdgcn_rcpf(1.0f + __expf(-a));
}

// The lane number, taken anew for each tile: what is computed from it would
// otherwise be moved out of the tile loop, and fill the registers for good.
__device__ __forceinline__ int tile_lane() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}

// E8M0 scale of a block of 4-bit codes from the bits of its largest magnitude:
// 2^(floor(log2 max) - 2), so that the largest lies in [4, 8); 255 (NaN) where a
// value is one.
__device__ __forceinline__ int mx4_scale(uint32_t amax) {
  if (amax > 0x7f800000u) return 255;
  const int be = static_cast<int>(amax >> 23);
  return be > 2 ? be - 2 : 0;
}
// 2^(S - 127)
__device__ __forceinline__ float e8m0_f32(int S) {
  return S ? __uint_as_float(static_cast<uint32_t>(S) << 23) : 0x1p-127f;
}
// Two codes (a in the low half) of a and b over 2^(S - 127): nearest, ties to even,
// 6 at most; zeros in a block whose scale is NaN.
template <int BYTE>
__device__ __forceinline__ uint32_t mx4_codes(uint32_t old, float a, float b, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, scale, BYTE);
}

// Largest of the 16 lanes of a row, in every lane.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x128, 0xf, 0xf, true)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x124, 0xf, 0xf, true)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x122, 0xf, 0xf, true)));
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x121, 0xf, 0xf, true)));
}

// A lane's two neighbouring columns 2 l16, 2 l16 + 1 of a 32-column block of h in
// row `row`: codes and the block's scale.  The 16 lanes of the row hold the block.
template <bool A4>
__device__ __forceinline__ void store_h(const Mx4Params& p, int64_t row, int block, int l16,
                                        float h0, float h1) {
  const int64_t at = row * p.ncols + 32 * block + 2 * l16;
  if constexpr (A4) {
    const uint32_t amax = row_max(max(__float_as_uint(h0) & 0x7fffffffu, __float_as_uint(h1) & 0x7fffffffu));
    const int S = mx4_scale(amax);
    const uint32_t c = S == 255 ? 0u : mx4_codes<0>(0u, h0, h1, e8m0_f32(S));
    p.hq[at >> 1] = static_cast<uint8_t>(c);
    if (l16 == 0) p.hs[row * (p.ncols / 32) + block] = static_cast<uint8_t>(S);
  } else {
    // (a NaN does not count in the maximum)
    const float m0 = h0 != h0 ? 0.f : fabsf(h0), m1 = h1 != h1 ? 0.f : fabsf(h1);
    const int S = mx_scale(__uint_as_float(row_max(__float_as_uint(fmaxf(m0, m1)))));
    const uint32_t c = mx_code(h0, S) | mx_code(h1, S) << 8;
    *reinterpret_cast<uint16_t*>(p.hq + at) = static_cast<uint16_t>(c);
    if (l16 == 0)
      p.hs[row * (p.ncols / 32) + (block & ~3) + 2 * (block & 1) + ((block >> 1) & 1)] =
          static_cast<uint8_t>(S);
  }
}

// RB blocks of 16 rows and NB blocks of 16 weight columns a workgroup (gate/up: the
// first half of them gate, the second the matching up columns).  The four wavefronts
// split the reduction and add their sums through LDS in order, so few rows still
// give many workgroups with many loads in flight, and there is no barrier in the loop.
template <int EPI, int RB, int NB, bool A4>
__global__ __launch_bounds__(kThreads, 2) void mx4_kernel(Mx4Params p) {
  constexpr int OUT = (EPI == MX_SWIGLU ? NB / 2 : NB) * 16;  // output columns a workgroup
  constexpr int TM = 16 * RB;
  constexpr int ABYTES = A4 ? kStep / 2 : kStep;  // of a row in a code block
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  const int NT = p.ncols / OUT;
  const int64_t total = static_cast<int64_t>(ld_scalar(p.total)) * NT;
  __shared__ float s_acc[kWaves][RB * NB * 4][64];
  for (int64_t in = blockIdx.x / 8;; in += gridDim.x / 8) {
    const int64_t L = tile_of(blockIdx.x % 8, in, p.log_run);
    if (in >= p.per_xcd) break;
    const RowTile tile = ld_tile(p.tiles + L / NT);
    if (L >= total) break;
    const int lane = tile_lane(), l16 = lane & 15, lq = lane >> 4;
    const int e = tile.e;
    const int q = static_cast<int>(L - static_cast<int64_t>(tile.mt0) * NT);
    const int nt = q / tile.mte;
    const int m0 = tile.seg0 + TM * (q % tile.mte);
    const int mcount = min(TM, tile.seg1 - m0);

    // this lane's rows; rows past the tile read its last row again
    int src[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      src[rb] = m0 + min(16 * rb + l16, mcount - 1);
      if (EPI == MX_SWIGLU) src[rb] = p.perm[src[rb]];
    }
    const int nkb = p.K / kStep, nq = (nkb + 3) / 4;
    const int64_t cmat = static_cast<int64_t>(p.ncols) * p.K / 2;           // codes of one matrix
    const int64_t smat = static_cast<int64_t>(p.ncols / 16) * nq * 256;     // and its scales
    const uint8_t* code[NB];  // wave-uniform
    const uint8_t* scale[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const bool up = EPI == MX_SWIGLU && nb >= NB / 2;
      const uint8_t* base = up ? p.B2 : p.B;
      const int cb = nt * (OUT / 16) + (up ? nb - NB / 2 : nb);
      code[nb] = base + e * cmat + static_cast<int64_t>(cb) * nkb * 1024;
      scale[nb] = base + p.N * cmat + e * smat + static_cast<int64_t>(cb) * nq * 256;
    }
    const uint32_t code_lane = lane * 16, scale_lane = lane * 4;

    struct Buf {
      i32x4_t b[NB];
      int sb[NB];
      i32x4_t a[RB][A4 ? 1 : 2];
      int sa[RB];
    };
    const uint8_t* arow[RB];
    const uint8_t* srow[RB];
    auto load_weights = [&](int kb, Buf& f) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        f.b[nb] = __builtin_nontemporal_load(
            reinterpret_cast<const i32x4_t*>(code[nb] + kb * 1024 + code_lane));
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        f.sb[nb] = scale[nb][(kb >> 2) * 256 + (kb & 3) + scale_lane];
    };
    auto load_rows = [&](int kb, Buf& f) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
#pragma unroll
        for (int i = 0; i < (A4 ? 1 : 2); ++i)
          f.a[rb][i] = *reinterpret_cast<const i32x4_t*>(arow[rb] + kb * ABYTES + 64 * i);
        f.sa[rb] = srow[rb][kb * 4];
      }
    };

    f32x4_t acc[RB][NB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) acc[rb][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](const Buf& f) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        i32x8_t a = {};
        a.lo = f.a[rb][0];
        if constexpr (!A4) a.hi = f.a[rb][1];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          i32x8_t b = {};
          b.lo = f.b[nb];
          acc[rb][nb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              a, b, acc[rb][nb], A4 ? 4 : 0, 4, 0, f.sa[rb], 0, f.sb[nb]);
        }
      }
    };

    // this wavefront's share of the reduction, one block ahead in registers
    const int kb0 = nkb * wave / kWaves, kb1 = nkb * (wave + 1) / kWaves;
    if (kb0 < kb1) {
      Buf f0, f1;
      // the first codes are under way before the rows' tokens are known
      load_weights(kb0, f0);
      asm volatile("" ::: "memory");
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        const int64_t r = EPI == MX_SWIGLU ? src[rb] / p.kdiv : src[rb];
        arow[rb] = p.A + r * (A4 ? p.K / 2 : p.K) + 16 * lq;
        // (MXFP8 rows keep a slab's four scales in the order 0, 2, 1, 3)
        srow[rb] = p.As + r * (p.K / 32) + (A4 ? lq : 2 * (lq & 1) + (lq >> 1));
      }
      load_rows(kb0, f0);
      int kb = kb0;
      for (; kb + 2 <= kb1; kb += 2) {
        load_weights(kb + 1, f1);
        load_rows(kb + 1, f1);
        compute(f0);
        if (kb + 2 < kb1) {
          load_weights(kb + 2, f0);
          load_rows(kb + 2, f0);
        }
        compute(f1);
      }
      if (kb < kb1) compute(f0);
    }

    // the wavefronts' sums, added in order; wavefront w finishes its share of the
    // tile: register v = w of every block, row 16 rb + 4 (lane / 16) + w, columns 2
    // (lane % 16) (even blocks) and the next (odd ones)
    __syncthreads();  // the previous tile's sums have been read
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int v = 0; v < 4; ++v) s_acc[wave][(rb * NB + nb) * 4 + v][lane] = acc[rb][nb][v];
    __syncthreads();
    auto sum = [&](int rb, int nb) {
      const int i = (rb * NB + nb) * 4 + wave;
      return ((s_acc[0][i][lane] + s_acc[1][i][lane]) + s_acc[2][i][lane]) + s_acc[3][i][lane];
    };
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int r = 16 * rb + 4 * lq + wave;
      if (r >= mcount) continue;  // (the 16 lanes of a row alike)
      const int64_t row = static_cast<int64_t>(m0) + r;
      if constexpr (EPI == MX_SWIGLU) {
#pragma unroll
        for (int j = 0; j < NB / 4; ++j) {
          const float h0 = silu_f(sum(rb, 2 * j)) * sum(rb, 2 * j + NB / 2);
          const float h1 = silu_f(sum(rb, 2 * j + 1)) * sum(rb, 2 * j + 1 + NB / 2);
          store_h<A4>(p, row, nt * (OUT / 32) + j, l16, h0, h1);
        }
      } else {
#pragma unroll
        for (int j = 0; j < NB / 2; ++j)
          *reinterpret_cast<float2*>(p.y + row * p.ncols + nt * OUT + 32 * j + 2 * l16) =
              make_float2(sum(rb, 2 * j), sum(rb, 2 * j + 1));
      }
    }
  }
}

// At most this many column tiles of OUT columns by row tiles of height 16 RB.
template <int EPI, int RB, int NB>
hipError_t launch_mx4(bool a4, Mx4Params p, int64_t rows, hipStream_t s) {
  const int OUT = (EPI == MX_SWIGLU ? NB / 2 : NB) * 16;
  deal_tiles(max_row_tiles(rows, p.N, 16 * RB) * (p.ncols / OUT), &p.per_xcd, &p.log_run);
  const dim3 grid(grid_of(p.per_xcd * 8)), block(kThreads);
  if (a4)
    hipLaunchKernelGGL((mx4_kernel<EPI, RB, NB, true>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((mx4_kernel<EPI, RB, NB, false>), grid, block, 0, s, p);
  return hipGetLastError();
}

// Natural codes (two a byte, the even step in the low half) and scales -> the layout
// above.  One thread per 16 bytes of codes, then one per scale.
__global__ __launch_bounds__(256) void mx4_pack_kernel(const u32x4_t* __restrict__ codes,
                                                       const uint8_t* __restrict__ scales,
                                                       uint8_t* __restrict__ dst, int64_t nmat,
                                                       int R, int C) {
  const int nkb = C / kStep, nq = (nkb + 3) / 4;
  const int64_t pieces = nmat * R * (C / 32);
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  // column of lane l16 of a 16-column block of the matrices' R rows
  auto column = [](int64_t blk, int l16) { return (blk >> 1) * 32 + 2 * l16 + (blk & 1); };
  for (int64_t i = i0; i < pieces; i += step) {
    // i = ((mat R/16 + cb) nkb + kb) 64 + lane
    const int lane = i & 63;
    const int64_t blk = i >> 6;
    const int kb = static_cast<int>(blk % nkb);
    const int64_t row = column(blk / nkb, lane & 15);
    reinterpret_cast<u32x4_t*>(dst)[i] = codes[row * (C / 32) + kb * 4 + (lane >> 4)];
  }
  const int64_t ns = nmat * (R / 16) * nq * 256;
  for (int64_t i = i0; i < ns; i += step) {
    // i = (((mat R/16 + cb) nq + quad) 64 + lane) 4 + block of 128 steps
    const int lane = (i >> 2) & 63;
    const int64_t blk = i >> 8;
    const int kb = static_cast<int>(blk % nq) * 4 + static_cast<int>(i & 3);
    const int64_t row = column(blk / nq, lane & 15);
    dst[pieces * 16 + i] = kb < nkb ? scales[row * (C / 32) + kb * 4 + (lane >> 4)] : 0;
  }
}

// Rows -> natural codes and scales, and the values they stand for.  Eight values a
// thread, four lanes a block.
template <typename T>
__global__ __launch_bounds__(256) void mx4_rows_kernel(const T* src, int64_t pieces,
                                                       uint32_t* __restrict__ codes,
                                                       uint8_t* __restrict__ scales, T* values) {
  // (a block's four lanes take the same rounds)
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < pieces;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    float f[8];
#pragma unroll
    for (int j = 0; j < 8 / V16<T>::n; ++j)
      V16<T>::load(src + i * 8 + j * V16<T>::n, f + j * V16<T>::n);
    uint32_t amax = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max(amax, __float_as_uint(f[e]) & 0x7fffffffu);
    amax = max(amax, static_cast<uint32_t>(__shfl_xor(static_cast<int>(amax), 1)));
    amax = max(amax, static_cast<uint32_t>(__shfl_xor(static_cast<int>(amax), 2)));
    const int S = mx4_scale(amax);
    const float scale = e8m0_f32(S);
    uint32_t w = mx4_codes<0>(0u, f[0], f[1], scale);
    w = mx4_codes<1>(w, f[2], f[3], scale);
    w = mx4_codes<2>(w, f[4], f[5], scale);
    w = mx4_codes<3>(w, f[6], f[7], scale);
    if (S == 255) w = 0u;
    codes[i] = w;
    if ((i & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(S);
    if (values) {
      const float sv = S == 255 ? __uint_as_float(0x7fc00000u) : scale;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // E2M1 as a multiple of 1/2: 0 1 2 3 4 6 8 12, a nibble each
        const uint32_t c = w >> (4 * e) & 15u;
        const float h = 0.5f * static_cast<float>(0xC8643210u >> (4 * (c & 7u)) & 15u);
        f[e] = __builtin_copysignf(h, c & 8u ? -1.f : 1.f) * sv;
      }
#pragma unroll
      for (int j = 0; j < 8 / V16<T>::n; ++j)
        V16<T>::store(values + i * 8 + j * V16<T>::n, f + j * V16<T>::n);
    }
  }
}

}  // namespace

int mx4_rows_per_tile(int64_t avg_rows) { return avg_rows <= 13 ? 16 : avg_rows <= 20 ? 32 : 64; }

hipError_t launch_mx4_gateup(bool a4, const uint8_t* xq, const uint8_t* xs, const uint8_t* wg,
                             const uint8_t* wu, const void* tiles, const int32_t* perm, int tm,
                             int64_t rows, int N, int I, int d, int K, uint8_t* hq, uint8_t* hs,
                             hipStream_t s) {
  Mx4Params p{};
  p.N = N; p.ncols = I; p.K = d;
  p.total = static_cast<const int32_t*>(tiles);
  p.tiles = static_cast<const RowTile*>(tiles) + 1;
  p.A = xq; p.As = xs; p.perm = perm; p.kdiv = K;
  p.B = wg; p.B2 = wu; p.hq = hq; p.hs = hs;
  if (tm == 16) return launch_mx4<MX_SWIGLU, 1, 4>(a4, p, rows, s);
  if (tm == 32) return launch_mx4<MX_SWIGLU, 2, 4>(a4, p, rows, s);
  return launch_mx4<MX_SWIGLU, 4, 4>(a4, p, rows, s);
}

hipError_t launch_mx4_down(bool a4, const uint8_t* hq, const uint8_t* hs, const uint8_t* wd,
                           const void* tiles, int tm, int64_t rows, int N, int I, int d, float* y,
                           hipStream_t s) {
  Mx4Params p{};
  p.N = N; p.ncols = d; p.K = I;
  p.total = static_cast<const int32_t*>(tiles);
  p.tiles = static_cast<const RowTile*>(tiles) + 1;
  p.A = hq; p.As = hs; p.kdiv = 1; p.B = wd; p.y = y;
  if (tm == 16) return launch_mx4<MX_STORE, 1, 4>(a4, p, rows, s);
  if (tm == 32) return launch_mx4<MX_STORE, 2, 4>(a4, p, rows, s);
  return launch_mx4<MX_STORE, 4, 4>(a4, p, rows, s);
}

int64_t mx4_weight_bytes(int64_t nmat, int64_t R, int64_t C) {
  return nmat * R * (C / 2) + nmat * (R / 16) * ((C / kStep + 3) / 4) * 256;
}

hipError_t launch_mx4_pack(const uint8_t* codes, const uint8_t* scales, uint8_t* dst, int64_t nmat,
                           int R, int C, hipStream_t s) {
  const int64_t n = mx4_weight_bytes(nmat, R, C) / 16;
  hipLaunchKernelGGL(mx4_pack_kernel, dim3(grid_of((n + 255) / 256)), dim3(256), 0, s,
                     reinterpret_cast<const u32x4_t*>(codes), scales, dst, nmat, R, C);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_mx4_rows(const T* src, int64_t R, int64_t C, uint8_t* codes, uint8_t* scales,
                           T* values, hipStream_t s) {
  const int64_t pieces = R * (C / 8);
  if (pieces == 0) return hipSuccess;
  hipLaunchKernelGGL(mx4_rows_kernel<T>, dim3(grid_of((pieces + 255) / 256)), dim3(256), 0, s, src,
                     pieces, reinterpret_cast<uint32_t*>(codes), scales, values);
  return hipGetLastError();
}
template hipError_t launch_mx4_rows<bf16_t>(const bf16_t*, int64_t, int64_t, uint8_t*, uint8_t*,
                                            bf16_t*, hipStream_t);
template hipError_t launch_mx4_rows<float>(const float*, int64_t, int64_t, uint8_t*, uint8_t*,
                                           float*, hipStream_t);

}  // namespace zc
