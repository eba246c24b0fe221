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
// Weights of one set (N matrices [R][C]), columns in groups of G = 2 (gate, up) or 4
// (down) blocks of 16: codes [N][R/16/G][C/128][G][lane][16 bytes]: 1 KB holds 16
// output columns and 128 reduction steps, a wave's operand as it lies, and a group's
// pieces of a step lie side by side; then scales [N][R/16/G][ceil(C/512)][lane][G][4
// code blocks], E8M0: a lane's scales of 512 steps and a group in one load.  A group's columns
// are dealt to its blocks in turn, so that a lane ends with G neighbours: two 4-bit
// codes of h, a byte; 8 or 16 bytes of y.
#include "row_split.h"
#include "zc_common.h"

namespace zc {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 128;  // reduction steps of a code block

enum { MX_SWIGLU = 0, MX_STORE = 1 };
// Blocks of 16 columns that lie side by side.
template <int EPI>
constexpr int kGroup = EPI == MX_SWIGLU ? 2 : 4;

typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

struct Mx4Params {
  int N, ncols, K;          // experts, output columns (I or d), reduction length (d or I)
  const int32_t* total;     // number of row tiles
  const RowTile* tiles;     // one of each (as many as the grid has row tiles)
  const uint8_t* A;         // codes: x' [T][...] gathered through perm, or h' [P][...]
  const uint8_t* As;        // their scales, [rows][K/32]
  const int32_t* perm;      // gate/up only
  int kdiv;                 // K of the layer (slot -> token)
  uint32_t kdiv_inv;        // many rows: 2^31 / K, rounded up: divides slots below 2^31 / K
                            // (K <= 32, and fewer than 2^22 slots there)
  const uint8_t* B;         // W_g or W_d
  const uint8_t* B2;        // W_u (gate/up)
  uint8_t* hq;              // gate/up output: codes [P][I] or [P][I/2] ...
  uint8_t* hs;              // ... and scales [P][I/32]
  float* y;                 // down output [P][d]
  bf16_t* yb;               // the same of many rows' kernel
  uint32_t a_bytes, as_bytes;  // sizes of A and As where 31 bits hold them
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

// Largest of the 16 lanes of a row, in every lane, of R values.
template <int R>
__device__ __forceinline__ void row_max(uint32_t (&v)[R]) {
#define ZC_ROR_MAX(N)                                                                   \
  _Pragma("unroll") for (int r = 0; r < R; ++r) v[r] = max(                             \
      v[r], static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(v[r], 0x120 + N, 0xf, 0xf, true)))
  ZC_ROR_MAX(8);
  ZC_ROR_MAX(4);
  ZC_ROR_MAX(2);
  ZC_ROR_MAX(1);
#undef ZC_ROR_MAX
}

// Codes of a lane's two neighbouring columns of a 32-column block of h, a row's 16
// lanes holding the block, and the block's scale S, for R rows at once: what waits for
// another lane's value finds the other rows' work to do.  A NaN makes its block's scale
// one, with 8-bit codes too: all of the row's y are NaN either way.
template <bool A4, int R>
__device__ __forceinline__ void codes_h(const float (&h)[R][2], uint32_t (&c)[R], int (&S)[R]) {
  uint32_t top[R];
#pragma unroll
  for (int r = 0; r < R; ++r)
    top[r] = max(__float_as_uint(h[r][0]) & 0x7fffffffu, __float_as_uint(h[r][1]) & 0x7fffffffu);
  row_max(top);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    // the scale's bits as a float: 2^(floor(log2 top) - 2 or 8), 0 for 2^-127
    constexpr uint32_t kDown = (A4 ? 2u : 8u) << 23;
    const uint32_t bits = max(top[r] & 0x7f800000u, kDown) - kDown;
    const int s = static_cast<int>(bits >> 23);
    S[r] = top[r] > 0x7f800000u ? 255 : s;
    if constexpr (A4) {
      c[r] = mx4_codes<0>(0u, h[r][0], h[r][1], __uint_as_float(max(bits, 0x00400000u)));
    } else {
      float q[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        q[i] = fminf(fmaxf(__builtin_ldexpf(h[r][i], 127 - s), -448.f), 448.f);
      c[r] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false)) & 0xffffu;
    }
  }
}

// bf16 of a (low half) and b, nearest, ties to even, in one instruction.
__device__ __forceinline__ uint32_t pk_bf16(float a, float b) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), bf16x2_t));
}

// RB blocks of 16 rows and NB blocks of 16 weight columns a workgroup (gate/up: the
// first half of them gate, the second the matching up columns).  The four wavefronts
// split the reduction and add their sums through LDS in order, so few rows still
// give many workgroups with many loads in flight, and there is no barrier in the loop.
// Bound by HBM: 256 tokens (d 6144, I 2048, 512 experts, MXFP8 rows) read 10.1 GB in 1.58
// ms, 6.4 TB/s; one token 105 MB of gate and up in 19.5 us, 5.4 TB/s (three or four slabs
// in registers in place of two: the same, both).  y is fp32.
template <int EPI, int RB, int NB, bool A4>
__global__ __launch_bounds__(kThreads, 2) void mx4_kernel(Mx4Params p) {
  constexpr int OUT = (EPI == MX_SWIGLU ? NB / 2 : NB) * 16;  // output columns a workgroup
  constexpr int TM = 16 * RB;
  constexpr int ABYTES = A4 ? kStep / 2 : kStep;  // of a row in a code block
  constexpr int G = kGroup<EPI>;
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
      code[nb] = base + e * cmat + (static_cast<int64_t>(cb / G) * nkb * G + cb % G) * 1024;
      scale[nb] = base + p.N * cmat + e * smat + static_cast<int64_t>(cb / G) * nq * G * 256 + cb % G * 4;
    }
    const uint32_t code_lane = lane * 16, scale_lane = lane * 4 * G;

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
            reinterpret_cast<const i32x4_t*>(code[nb] + kb * (1024 * G) + code_lane));
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        f.sb[nb] = scale[nb][(kb >> 2) * (256 * G) + (kb & 3) + scale_lane];
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
    // tile: register v = w of every block, row 16 rb + 4 (lane / 16) + w, and of 2 or 4
    // blocks as many neighbouring columns
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
          const int block = nt * (OUT / 32) + j;
          const float h[1][2] = {{h0, h1}};
          int S[1];
          uint32_t c[1];
          codes_h<A4>(h, c, S);
          if constexpr (A4)
            p.hq[(row * p.ncols + 32 * block) / 2 + l16] = static_cast<uint8_t>(c[0]);
          else
            *reinterpret_cast<uint16_t*>(p.hq + row * p.ncols + 32 * block + 2 * l16) = static_cast<uint16_t>(c[0]);
          if (l16 == 0)
            p.hs[row * (p.ncols / 32) +
                 (A4 ? block : (block & ~3) + 2 * (block & 1) + ((block >> 1) & 1))] = static_cast<uint8_t>(S[0]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < NB / 4; ++j)
          *reinterpret_cast<f32x4_t*>(p.y + row * p.ncols + nt * OUT + 64 * j + 4 * l16) =
              f32x4_t{sum(rb, 4 * j), sum(rb, 4 * j + 1), sum(rb, 4 * j + 2), sum(rb, 4 * j + 3)};
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

// ------------------------------------------------------------- many rows
typedef __attribute__((address_space(3))) void lds_void;
// (Buffer loads: the compiler would have every LDS read wait for all copies in
// flight if they were global loads into LDS.)
__device__ __forceinline__ void copy_to_lds16(__amdgpu_buffer_rsrc_t r, lds_void* dst,
                                              uint32_t voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, dst, 16, voff, soff, 0, 0);
}
// s_waitcnt immediate for "vmcnt <= n" (expcnt and lgkmcnt not waited)
constexpr int vmcnt_imm(int n) { return 0x0f70 | (n & 15) | ((n >> 4) << 14); }
// Barrier for LDS alone: loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// TM rows by 256 weight columns a workgroup (gate/up: 128 gate and the matching up
// columns), 64 columns a wavefront: each weight goes from memory to the registers of
// the one wavefront that multiplies with it, the rows through LDS to all four.  Two
// workgroups a CU.  While a slab of 128 steps is multiplied, two or three slabs of rows
// are under way, copied straight into a ring of three or four LDS slots, and one to three
// of weights in registers.  A slot holds 128 bytes of a row, a cache line: of MXFP4
// rows two slabs (one a slot, half lines: gate/up 2.25 ms, two 2.07), and rows' scales
// come 64 bytes at a time (16 bytes: 2.05 ms, 64: 2.00).  Tiles of 160 rows leave room for
// two slabs of weights in place of four, 2% of the time, and read them for fewer row
// tiles.
//
// What bounds it (16384 tokens, d 6144, I 2048, 512 experts, MXFP4 rows; gate/up 1.89
// ms, 5.2 PFLOP/s; down 1.18 ms).  Products alone would take 0.92 ms at the 7.2 PFLOP/s
// that the instruction reaches, HBM 1.1 ms.  With tiles of 128 rows (1.98 ms), in copies whose weights all came from the
// first-level cache gate/up took 1.50 ms: products, the loads' way through the address
// unit (busy 83% of the time) and the tiles' ends; from the L2s 1.65; the rest is HBM, each
// weight for 2.5 row tiles an expert.  With parts left out: without the weights' loads
// 1.39 ms, the rows' copies 1.78, the products 1.86, the results 1.84.  The same time:
// weights two slabs ahead in place of three, a barrier once in four slabs.  Slower: row
// tiles of an expert some slabs apart (2.03 to 2.4 ms), and, before the step to whole
// lines (2.25 ms then), 256 rows by eight wavefronts (2.52 ms), 256 rows by four with
// 512 registers and seven slabs ahead (4.18 ms: the sums alone fill the accumulation
// registers), weights read non-temporally (2.70 ms: the other row tiles of an expert
// find them in the L2).  With one row tile an expert (2048 tokens) it reads its weights
// at 6 TB/s, in 1.14 ms.  MXFP8 rows, with products of 4.4 PFLOP/s, in many small tiles
// (4093 tokens, d 1024, I 512, 64 experts: gate/up 30 us, down 18) are bound by a
// tile's start and end: 8 and 4 slabs between them, 640 tiles on 512 places.
//
// An expert's rows are spread evenly over its tiles in blocks of 16, and a tile's sums
// are those of 2, 4, 6, 8 or 10 blocks.  y goes out in bf16: it would be twice the bytes
// in fp32 (1.6 of 10.7 GB here), and costs up to 2^-8 of each of K terms: the result's
// error to 64 bits is 1.9e-3 of its norm, with y in fp32 (256 tokens) 1.7e-3, most of it
// out's own rounding.
template <int EPI, bool A4, int TM>
__global__ __launch_bounds__(kThreads, 2) void mx4_wide_kernel(Mx4Params p) {
  constexpr int CB = 128;                      // bytes of a row in a ring slot: a cache line
  constexpr int SPS = A4 ? 2 : 1;              // slabs of 128 steps in a slot
  constexpr int SLOTS = TM > 128 ? 3 : 4;
  constexpr int SLOT = TM * CB;                // bytes of a slot
  constexpr int CP = SLOT / 1024 / kWaves;     // copies a wavefront and slot
  constexpr int RPC = 1024 / CB;               // rows of a copy
  constexpr int SC = TM * 64;                  // bytes of the rows' scales of 2048 steps
  constexpr int SCP = (SC / 1024 + kWaves - 1) / kWaves;  // copies a wavefront of them
  constexpr int OUT = EPI == MX_SWIGLU ? 128 : 256;
  constexpr int G = kGroup<EPI>;
  constexpr int CSC = 4 / G;                   // loads of the columns' scales of 512 steps
  constexpr int NSC = CSC + 1;                 // and with them of the rows'
  // Copies of rows that go out in a slab (MXFP4: a slot's in two slabs).
  constexpr int CEVEN = (CP + SPS - 1) / SPS, CODD = A4 ? CP / 2 : CP;
  // Slabs of weights in registers: four where the sums and rows leave room for them, their
  // loads between the multiplications; else two, loaded at a slab's end.
  constexpr int NBUF = A4 && TM == 128 ? 4 : 2;
  // Loads that may be in flight when slab `slot` of four is needed: those of the two
  // slabs before it, or of the one before it (rows are older).
  constexpr auto wait_of = [](int slot) constexpr {
    return NBUF == 4 ? CEVEN + CODD + 8 + (slot == 1 || slot == 2 ? NSC : 0)
                     : (slot % 2 ? CEVEN : CODD) + 4 + (slot == 1 ? NSC : 0);
  };
  __shared__ __align__(16) uint8_t ring[SLOTS * SLOT + 2 * SC];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nkb = p.K / kStep, nq = nkb / 4;
  const int NT = p.ncols / OUT;
  const __amdgpu_buffer_rsrc_t rows = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.A), (short)0, p.a_bytes, 0x00020000);
  const __amdgpu_buffer_rsrc_t rscale = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.As), (short)0, p.as_bytes, 0x00020000);
  const int64_t total = static_cast<int64_t>(ld_scalar(p.total)) * NT;
  for (int64_t in = blockIdx.x / 8;; in += gridDim.x / 8) {
    const int64_t L = tile_of(blockIdx.x % 8, in, p.log_run);
    if (in >= p.per_xcd) break;
    const RowTile tile = ld_tile(p.tiles + L / NT);
    if (L >= total) break;
    const int lane = tile_lane(), l16 = lane & 15, lq = lane >> 4;
    const int e = tile.e;
    const int q = static_cast<int>(L - static_cast<int64_t>(tile.mt0) * NT);
    const int nt = q / tile.mte, mt = q % tile.mte;
    // the expert's blocks of 16 rows spread evenly over its row tiles
    const int nbe = (tile.seg1 - tile.seg0 + 15) >> 4;
    const int blo = first_block(nbe, mt, tile.mte), bhi = first_block(nbe, mt + 1, tile.mte);
    const int m0 = tile.seg0 + 16 * blo;
    const int mcount = min(tile.seg0 + 16 * bhi, tile.seg1) - m0;

    // the i-th block of 16 rows whose scales this wavefront copies (where there are too
    // few blocks for all wavefronts, the last ones again)
    auto scale_rows = [&](int i) { return wave + kWaves * i < TM / 16 ? wave + kWaves * i : wave + kWaves * (i - 1); };
    // Rows that this lane copies, and those whose scales: first the slots, which are
    // under way while the first weights are asked for.
    int slot_of[CP + SCP];
#pragma unroll
    for (int i = 0; i < CP + SCP; ++i) {
      const int r = i < CP ? (CP * wave + i) * RPC + lane / (CB / 16) : 16 * scale_rows(i - CP) + (lane >> 2);
      slot_of[i] = m0 + min(r, mcount - 1);
      if (EPI == MX_SWIGLU) slot_of[i] = p.perm[slot_of[i]];
    }
    // first of the at-th four (a row's last four end with it)
    auto sfirst = [&](int at) { return max(min(4 * at, nq - 4), 0); };

    const int64_t cmat = static_cast<int64_t>(p.ncols) * p.K / 2, smat = cmat / 16;
    __amdgpu_buffer_rsrc_t codes[2], scales[2];  // gate (or down) and up
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      uint8_t* base = const_cast<uint8_t*>(EPI == MX_SWIGLU && m ? p.B2 : p.B);
      codes[m] = __builtin_amdgcn_make_buffer_rsrc(base + e * cmat, (short)0,
                                                   static_cast<uint32_t>(cmat), 0x00020000);
      scales[m] = __builtin_amdgcn_make_buffer_rsrc(base + p.N * cmat + e * smat, (short)0,
                                                    static_cast<uint32_t>(smat), 0x00020000);
    }
    const int grp = nt * 4 + wave;  // the wavefront's group of column blocks
    const uint32_t code_lane = lane * 16, scale_lane = lane * 4 * G;

    auto run = [&](auto nrb_c) {
      constexpr int NRB = decltype(nrb_c)::value;
      // (what the variants have in common would otherwise move in front of the switch,
      // and the loops' registers with it)
      asm volatile("; %0 blocks of rows" ::"n"(NRB));
      uint32_t src[CP], ssrc[SCP];
      i32x4_t b[NBUF][4];  // [slab % NBUF][column block]
      int sb[4], sbn[4];   // scales of these four slabs, and of the next four
      // one load each: the i-th copy of a slot's rows, `at` slots' worth into the row;
      // the weights' column block nb of slab kb; of the rows' scales of 2048 steps, and
      // the columns' of 512
      auto issue_row = [&](int at, int slot, int i) {
        copy_to_lds16(rows, (lds_void*)(ring + slot * SLOT + (CP * wave + i) * 1024), src[i], at * CB);
      };
      auto issue_weight = [&](int kb, int slot, int nb) {
        b[slot % NBUF][nb] = __builtin_bit_cast(
            i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(codes[EPI == MX_SWIGLU ? nb / 2 : 0],
                                                           code_lane, ((grp * nkb + kb) * G + nb % G) * 1024, 0));
      };
      auto issue_row_scale = [&](int at, int i) {
        copy_to_lds16(rscale, (lds_void*)(ring + SLOTS * SLOT + (at & 1) * SC + scale_rows(i) * 1024),
                      i == 0 ? ssrc[0] : i == 1 ? ssrc[1] : ssrc[SCP - 1], sfirst(at) * 16);
      };
      auto issue_scale = [&](int quad, int* sc, int i) {
        const int at = (grp * nq + quad) * G * 256;
        if constexpr (G == 4) {
          const auto w = __builtin_amdgcn_raw_buffer_load_b128(scales[0], scale_lane, at, 0);
#pragma unroll
          for (int nb = 0; nb < 4; ++nb) sc[nb] = w[nb];
        } else {
          const auto w = __builtin_amdgcn_raw_buffer_load_b64(scales[i], scale_lane, at, 0);
          sc[2 * i] = w[0];
          sc[2 * i + 1] = w[1];
        }
      };

      f32x4_t acc[NRB][4];
#pragma unroll
      for (int rb = 0; rb < NRB; ++rb)
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) acc[rb][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      // where this lane's row of a block lies in a slot: chunk lq, and 4 + lq (MXFP8: of
      // the same slab, MXFP4: of the slot's second one)
      const int frag_at = l16 * CB + 16 * (lq ^ (l16 >> 1));
      // MXFP4: the slot of these four slabs' first half
      int first = 0;
      auto after = [](int s, int n) { return s + n < SLOTS ? s + n : s + n - SLOTS; };
      // and its scale of a slab
      int scale_at = SLOTS * SLOT + l16 * 64 + 16 * (l16 >> 2) + (A4 ? lq : 2 * (lq & 1) + (lq >> 1));

      // Fragments are read AHEAD of their multiplications (of 64 or 128 cycles).
      constexpr int AHEAD = !A4 ? 1 : NRB > 8 ? 2 : 3 < NRB ? 3 : NRB;
      const int last = nkb - 1;
      // One slab: wait for it, meet, multiply, and between the multiplications issue,
      // one by one, the loads of rows three slabs ahead or more, of weights and (with the
      // first of four slabs) of the next four's scales: issued at once they would
      // hold the wavefront up until the address unit has taken them all.  No branch: past the end the
      // last slab is loaded again, so that the number of loads in flight is known.
      auto slab = [&](int kb, int q4, auto slot_c) {
        constexpr int slot = decltype(slot_c)::value;
        constexpr int NR = slot % 2 ? CODD : CEVEN, NW = NR + (NBUF == 4 ? 4 : 0);  // rows, weights
        constexpr int NL = NW + (slot == 0 ? NSC : 0);
        const uint8_t* at = ring + (A4 ? after(first, slot / 2) * SLOT : slot * SLOT);
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(wait_of(slot)));
        lds_barrier();
        i32x8_t a[AHEAD + 1] = {};
        int sa[AHEAD + 1];
        auto frag = [&](int rb) {
          i32x8_t& f = a[rb % (AHEAD + 1)];
          f.lo = *reinterpret_cast<const i32x4_t*>(at + (frag_at ^ (slot % SPS * 64)) + rb * 16 * CB);
          if constexpr (!A4) f.hi = *reinterpret_cast<const i32x4_t*>(at + (frag_at ^ 64) + rb * 16 * CB);
          sa[rb % (AHEAD + 1)] = ring[rb * 1024 + slot * 4 + scale_at];
        };
#pragma unroll
        for (int rb = 0; rb < AHEAD; ++rb) frag(rb);
#pragma unroll
        for (int rb = 0; rb < NRB; ++rb) {
          if (rb + AHEAD < NRB) frag(rb + AHEAD);
#pragma unroll
          for (int i = NL * rb / NRB; i < NL * (rb + 1) / NRB; ++i) {
            if (i < NR && A4)
              issue_row(min(2 * q4 + slot / 2 + 2, last / 2), after(first, 2 + slot / 2),
                        slot % 2 * CEVEN + i);
            else if (i < NR)
              issue_row(min(kb + 3, last), (slot + 3) & 3, i);
            else if (i < NW)
              issue_weight(min(kb + 3, last), (slot + 3) & 3, i - NR);
            else if (i < NL - 1)
              issue_scale(min(q4 + 1, nq - 1), sbn, i - NW);
            else  // (some of them twice in the four quarters: so the number of loads is known)
              issue_row_scale(q4 / 4 + 1, min(q4 & 3, SCP - 1));
          }
#pragma unroll
          for (int nb = 0; nb < 4; ++nb) {
            i32x8_t w = {};
            w.lo = b[slot % NBUF][nb];
            acc[rb][nb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                a[rb % (AHEAD + 1)], w, acc[rb][nb], A4 ? 4 : 0, 4, 0, sa[rb % (AHEAD + 1)], slot,
                sb[nb]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (NBUF == 2) {
#pragma unroll
          for (int nb = 0; nb < 4; ++nb) issue_weight(min(kb + 2, last), slot, nb);
          __builtin_amdgcn_sched_barrier(0);
        }
      };

      using C0 = std::integral_constant<int, 0>;
      using C1 = std::integral_constant<int, 1>;
      using C2 = std::integral_constant<int, 2>;
      using C3 = std::integral_constant<int, 3>;
#pragma unroll
      for (int i = 0; i < CSC; ++i) issue_scale(0, sb, i);
#pragma unroll
      for (int kb = 0; kb < (NBUF == 4 ? 3 : 2); ++kb)
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) issue_weight(kb, kb, nb);
      __builtin_amdgcn_sched_barrier(0);
      // rows past the tile's end are copied from past the buffer's: no data moves
#pragma unroll
      for (int i = 0; i < CP; ++i) {
        const int r = (CP * wave + i) * RPC + lane / (CB / 16);
        const uint32_t tok = EPI == MX_SWIGLU ? __umulhi(2 * slot_of[i], p.kdiv_inv) : slot_of[i];
        src[i] = tok * static_cast<uint32_t>(A4 ? p.K / 2 : p.K) + 16 * ((lane & 7) ^ ((r >> 1) & 7));
        src[i] = r < mcount ? src[i] : p.a_bytes;
      }
      // Rows' scales, 64 bytes (four times 512 steps) at a time; which of the four this
      // lane copies depends on the row (the same ones of all rows would lie in the same
      // LDS banks).
      const int schunk = (lane & 3) ^ (lane >> 4);
#pragma unroll
      for (int i = 0; i < SCP; ++i) {
        const int r = 16 * scale_rows(i) + (lane >> 2);
        const uint32_t tok = EPI == MX_SWIGLU ? __umulhi(2 * slot_of[CP + i], p.kdiv_inv) : slot_of[CP + i];
        ssrc[i] = tok * static_cast<uint32_t>(p.K / 32) + 16 * schunk;
        ssrc[i] = r < mcount && schunk < nq ? ssrc[i] : p.as_bytes;
      }
      lds_barrier();  // the ring is free: the previous tile's reads are done
#pragma unroll
      for (int i = 0; i < SCP; ++i) issue_row_scale(0, i);
#pragma unroll
      for (int at = 0; at < (A4 ? 2 : 3); ++at) {
#pragma unroll
        for (int i = 0; i < CP; ++i) issue_row(at, at, i);
        __builtin_amdgcn_sched_barrier(0);
      }
      // (the waits in the loop count on rows and weights in turn: here the first rows)
      __builtin_amdgcn_s_waitcnt(vmcnt_imm((A4 ? 1 : 2) * CP));
      for (int q4 = 0; q4 < nq; ++q4) {
        slab(4 * q4, q4, C0{});
        slab(4 * q4 + 1, q4, C1{});
        slab(4 * q4 + 2, q4, C2{});
        slab(4 * q4 + 3, q4, C3{});
        scale_at ^= 16 * ((q4 - sfirst(q4 / 4)) ^ (q4 + 1 - sfirst((q4 + 1) / 4)));
        scale_at += (q4 & 3) < 3 ? 0 : q4 & 4 ? -SC : SC;
        first = after(first, 2);
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) sb[nb] = sbn[nb];
      }
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // no copy of this tile lands in the next one's ring

      // Results go out through resources that end with the tile's rows: no branch.
      if constexpr (EPI == MX_SWIGLU) {
        const int pitch = A4 ? p.ncols / 2 : p.ncols, sp = p.ncols / 32, block = nt * 4 + wave;
        const __amdgpu_buffer_rsrc_t hq = __builtin_amdgcn_make_buffer_rsrc(
            p.hq + static_cast<int64_t>(m0) * pitch, (short)0, mcount * pitch, 0x00020000);
        const __amdgpu_buffer_rsrc_t hs = __builtin_amdgcn_make_buffer_rsrc(
            p.hs + static_cast<int64_t>(m0) * sp, (short)0, mcount * sp, 0x00020000);
        const int at = 4 * lq * pitch + (A4 ? 16 * block + l16 : 32 * block + 2 * l16);
        // the first lane of a row writes its scale
        const int sat = l16 ? 0x70000000
                            : 4 * lq * sp + (A4 ? block : (block & ~3) + 2 * (block & 1) + ((block >> 1) & 1));
#pragma unroll
        for (int rb = 0; rb < NRB; ++rb) {
          float h[4][2];
          uint32_t c[4];
          int S[4];
#pragma unroll
          for (int v = 0; v < 4; ++v)
#pragma unroll
            for (int i = 0; i < 2; ++i) h[v][i] = silu_f(acc[rb][i][v]) * acc[rb][2 + i][v];
          codes_h<A4>(h, c, S);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            if constexpr (A4)
              __builtin_amdgcn_raw_buffer_store_b8(static_cast<uint8_t>(c[v]), hq, at + (16 * rb + v) * pitch, 0, 0);
            else
              __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(c[v]), hq, at + (16 * rb + v) * pitch, 0, 0);
            __builtin_amdgcn_raw_buffer_store_b8(static_cast<uint8_t>(S[v]), hs, sat + (16 * rb + v) * sp, 0, 0);
          }
        }
      } else {
        const __amdgpu_buffer_rsrc_t y = __builtin_amdgcn_make_buffer_rsrc(
            p.yb + static_cast<int64_t>(m0) * p.ncols, (short)0, mcount * p.ncols * 2, 0x00020000);
        const int at = (4 * lq * p.ncols + nt * OUT + 64 * wave + 4 * l16) * 2;
#pragma unroll
        for (int rb = 0; rb < NRB; ++rb)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            u32x2_t w;
#pragma unroll
            for (int j = 0; j < 2; ++j)
              w[j] = pk_bf16(acc[rb][2 * j][v], acc[rb][2 * j + 1][v]);
            // (non-temporal: down of 4093 tokens of the small layer 20.5 -> 18.3 us)
            __builtin_amdgcn_raw_buffer_store_b64(w, y, at + (16 * rb + v) * p.ncols * 2, 0, 2);
          }
      }
    };
    switch ((bhi - blo + 1) >> 1) {
      case 1: run(std::integral_constant<int, 2>{}); break;
      case 2: run(std::integral_constant<int, 4>{}); break;
      case 3: run(std::integral_constant<int, 6>{}); break;
      case 4:
        if constexpr (TM > 128) {
          run(std::integral_constant<int, 8>{});
          break;
        }
      default: run(std::integral_constant<int, TM / 16>{}); break;
    }
  }
}

template <int EPI>
hipError_t launch_mx4_wide(bool a4, Mx4Params p, int64_t rows, int tm, hipStream_t s) {
  const int OUT = EPI == MX_SWIGLU ? 128 : 256;
  deal_tiles(max_row_tiles(rows, p.N, tm) * (p.ncols / OUT), &p.per_xcd, &p.log_run);
  const dim3 grid(grid_of(p.per_xcd * 8)), block(kThreads);
  if (!a4)
    hipLaunchKernelGGL((mx4_wide_kernel<EPI, false, 128>), grid, block, 0, s, p);
  else if (tm == 128)
    hipLaunchKernelGGL((mx4_wide_kernel<EPI, true, 128>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((mx4_wide_kernel<EPI, true, 160>), grid, block, 0, s, p);
  return hipGetLastError();
}

// Natural codes (two a byte, the even step in the low half) and scales -> the layout
// above.  One thread per 16 bytes of codes, then one per scale.
__global__ __launch_bounds__(256) void mx4_pack_kernel(const u32x4_t* __restrict__ codes,
                                                       const uint8_t* __restrict__ scales,
                                                       uint8_t* __restrict__ dst, int64_t nmat,
                                                       int R, int C, int log_group) {
  const int nkb = C / kStep, nq = (nkb + 3) / 4;
  const int64_t pieces = nmat * R * (C / 32);
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  // column of lane l16 of a 16-column block of the matrices' R rows
  const int G = 1 << log_group;
  auto column = [=](int64_t group, int j, int l16) { return ((group * 16 + l16) << log_group) + j; };
  for (int64_t i = i0; i < pieces; i += step) {
    // i = (((mat R/16/G + group) nkb + kb) G + block) 64 + lane
    const int lane = i & 63, j = (i >> 6) & (G - 1);
    const int64_t blk = i >> (6 + log_group);
    const int kb = static_cast<int>(blk % nkb);
    const int64_t row = column(blk / nkb, j, lane & 15);
    reinterpret_cast<u32x4_t*>(dst)[i] = codes[row * (C / 32) + kb * 4 + (lane >> 4)];
  }
  const int64_t ns = nmat * (R / 16) * nq * 256;
  for (int64_t i = i0; i < ns; i += step) {
    // i = ((((mat R/16/G + group) nq + quad) 64 + lane) G + block) 4 + code block
    const int lane = (i >> (2 + log_group)) & 63, j = (i >> 2) & (G - 1);
    const int64_t blk = i >> (8 + log_group);
    const int kb = static_cast<int>(blk % nq) * 4 + static_cast<int>(i & 3);
    const int64_t row = column(blk / nq, j, lane & 15);
    dst[pieces * 16 + i] = kb < nkb ? scales[row * (C / 32) + kb * 4 + (lane >> 4)] : 0;
  }
}

// MXFP4 of one thread's 8 values of a block of 32 held by 4 consecutive lanes: the
// codes, and the block's scale S.
__device__ __forceinline__ uint32_t mx4_quad(const float* f, int& S) {
  uint32_t amax = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = max(amax, __float_as_uint(f[e]) & 0x7fffffffu);
  amax = max(amax, static_cast<uint32_t>(__shfl_xor(static_cast<int>(amax), 1)));
  amax = max(amax, static_cast<uint32_t>(__shfl_xor(static_cast<int>(amax), 2)));
  S = mx4_scale(amax);
  const float scale = e8m0_f32(S);
  uint32_t w = mx4_codes<0>(0u, f[0], f[1], scale);
  w = mx4_codes<1>(w, f[2], f[3], scale);
  w = mx4_codes<2>(w, f[4], f[5], scale);
  w = mx4_codes<3>(w, f[6], f[7], scale);
  return S == 255 ? 0u : w;
}

// Rows -> natural codes and scales, and the values they stand for.  Eight values a
// thread.  Bound by HBM: 16384 x 6144 values in bf16 with their values back, 456 MB, in
// 81 us, 5.6 TB/s, a copy's rate (non-temporal loads or stores: the same).
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
    int S;
    const uint32_t w = mx4_quad(f, S);
    codes[i] = w;
    if ((i & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(S);
    if (values) {
      const float sv = S == 255 ? __uint_as_float(0x7fc00000u) : e8m0_f32(S);
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

// The first workgroup lists the row tiles, the others quantize x: both have to be
// there before the products, and neither needs the other (one launch less: 2 us of
// a call on one token).
template <bool A4>
__global__ __launch_bounds__(kMaxExperts) void mx4_start_kernel(
    const int32_t* __restrict__ offsets, int N, int tm, int32_t* __restrict__ total,
    RowTile* __restrict__ tiles, const bf16_t* __restrict__ x, int64_t pieces,
    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  if (blockIdx.x == 0) {
    list_row_tiles(offsets, N, tm, total, tiles);
    return;
  }
  for (int64_t i = static_cast<int64_t>(blockIdx.x - 1) * kMaxExperts + threadIdx.x; i < pieces;
       i += static_cast<int64_t>(gridDim.x - 1) * kMaxExperts) {
    float f[8];
    V16<bf16_t>::load(x + i * 8, f);
    int S;
    if constexpr (A4) {
      reinterpret_cast<uint32_t*>(codes)[i] = mx4_quad(f, S);
      if ((i & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(S);
    } else {
      reinterpret_cast<uint64_t*>(codes)[i] = mx_quad(f, S);
      const int64_t b = i >> 2;  // (rows are whole slabs of 4 blocks: the order 0, 2, 1, 3)
      if ((i & 3) == 0) scales[(b & ~int64_t(3)) + 2 * (b & 1) + ((b >> 1) & 1)] = static_cast<uint8_t>(S);
    }
  }
}

}  // namespace

// Row tiles by the rows an expert has on average.  Few rows: each weight is read once
// and done with, by tiles of 16; from some 10 rows on by the kernel of many rows
// (gate/up, down and combine with MXFP8 rows, us, tiles of 16 / of 32 / many rows):
//   d 6144, I 2048, 512 experts:  8 rows 1782 / 1881 / 1801, 12 rows 2088 / 1996 / 1828,
//     20 rows 3413 / 2287 / 1878
//   d 1024, I 512, 64 experts:    8 rows 26.2 / 29.8 / 28.6, 12 rows 28.5 / 31.4 / 28.7,
//     20 rows 34.7 / 36.1 / 29.7, 64 rows 58.4 / 60.1 / 33.6
// With MXFP4 rows its tiles have up to 160 rows from 110 rows an expert on: that gains
// where it saves tiles, and loses up to 4.5% where it does not (the large layer's
// gate/up, tiles of 128 / of 160): 101 rows 1258 / 1274, 128 rows 1452 / 1334, 187 rows (two
// tiles either way) 1685 / 1760, 256 rows 2007 / 1906, 375 rows 2587 / 2605; the small
// one's at 128 rows 18.6 / 15.8, 255 rows 24.5 / 22.2.
// That kernel takes whole groups of 512 steps, and byte offsets of 31 bits into x, h and
// a matrix: other layers have tiles of 16, 32 or 64.
Mx4Plan mx4_plan(bool a4, int64_t Tn, int64_t rows, int64_t E, int64_t d, int64_t I) {
  const int64_t avg = rows / E, limit = int64_t(1) << 31;
  if (avg <= 10) return {16, false};
  if (d % 512 == 0 && I % 512 == 0 && Tn * d < limit && rows * I < limit && d * I < limit)
    return {a4 && avg >= 110 ? 160 : 128, true};
  return {avg <= 13 ? 16 : avg <= 20 ? 32 : 64, false};
}

hipError_t launch_mx4_start(bool a4, const int32_t* offsets, int N, int tm, void* tiles,
                            const bf16_t* x, int64_t Tn, int d, uint8_t* xq, uint8_t* xs,
                            hipStream_t s) {
  const int64_t pieces = Tn * (d / 8);
  const dim3 grid(1 + grid_of((pieces + kMaxExperts - 1) / kMaxExperts)), block(kMaxExperts);
  int32_t* total = static_cast<int32_t*>(tiles);
  RowTile* list = static_cast<RowTile*>(tiles) + 1;
  if (a4)
    hipLaunchKernelGGL(mx4_start_kernel<true>, grid, block, 0, s, offsets, N, tm, total, list, x,
                       pieces, xq, xs);
  else
    hipLaunchKernelGGL(mx4_start_kernel<false>, grid, block, 0, s, offsets, N, tm, total, list, x,
                       pieces, xq, xs);
  return hipGetLastError();
}

hipError_t launch_mx4_gateup(bool a4, const uint8_t* xq, const uint8_t* xs, int64_t Tn, const uint8_t* wg,
                             const uint8_t* wu, const void* tiles, const int32_t* perm, Mx4Plan plan,
                             int64_t rows, int N, int I, int d, int K, uint8_t* hq, uint8_t* hs,
                             hipStream_t s) {
  Mx4Params p{};
  p.N = N; p.ncols = I; p.K = d;
  p.total = static_cast<const int32_t*>(tiles);
  p.tiles = static_cast<const RowTile*>(tiles) + 1;
  p.A = xq; p.As = xs; p.perm = perm; p.kdiv = K;
  p.B = wg; p.B2 = wu; p.hq = hq; p.hs = hs;
  if (plan.wide) {
    p.a_bytes = static_cast<uint32_t>(a4 ? Tn * d / 2 : Tn * d);
    p.as_bytes = static_cast<uint32_t>(Tn * (d / 32));
    p.kdiv_inv = static_cast<uint32_t>(((int64_t(1) << 31) + K - 1) / K);
    return launch_mx4_wide<MX_SWIGLU>(a4, p, rows, plan.tm, s);
  }
  if (plan.tm == 16) return launch_mx4<MX_SWIGLU, 1, 4>(a4, p, rows, s);
  if (plan.tm == 32) return launch_mx4<MX_SWIGLU, 2, 4>(a4, p, rows, s);
  return launch_mx4<MX_SWIGLU, 4, 4>(a4, p, rows, s);
}

hipError_t launch_mx4_down(bool a4, const uint8_t* hq, const uint8_t* hs, const uint8_t* wd,
                           const void* tiles, Mx4Plan plan, int64_t rows, int N, int I, int d, void* y,
                           hipStream_t s) {
  Mx4Params p{};
  p.N = N; p.ncols = d; p.K = I;
  p.total = static_cast<const int32_t*>(tiles);
  p.tiles = static_cast<const RowTile*>(tiles) + 1;
  p.A = hq; p.As = hs; p.kdiv = 1; p.B = wd;
  if (plan.wide) {
    p.yb = static_cast<bf16_t*>(y);
    p.a_bytes = static_cast<uint32_t>(a4 ? rows * I / 2 : rows * I);
    p.as_bytes = static_cast<uint32_t>(rows * (I / 32));
    return launch_mx4_wide<MX_STORE>(a4, p, rows, plan.tm, s);
  }
  p.y = static_cast<float*>(y);
  if (plan.tm == 16) return launch_mx4<MX_STORE, 1, 4>(a4, p, rows, s);
  if (plan.tm == 32) return launch_mx4<MX_STORE, 2, 4>(a4, p, rows, s);
  return launch_mx4<MX_STORE, 4, 4>(a4, p, rows, s);
}

int64_t mx4_weight_bytes(int64_t nmat, int64_t R, int64_t C) {
  return nmat * R * (C / 2) + nmat * (R / 16) * ((C / kStep + 3) / 4) * 256;
}

hipError_t launch_mx4_pack(bool down, const uint8_t* codes, const uint8_t* scales, uint8_t* dst,
                           int64_t nmat, int R, int C, hipStream_t s) {
  const int64_t n = mx4_weight_bytes(nmat, R, C) / 16;
  hipLaunchKernelGGL(mx4_pack_kernel, dim3(grid_of((n + 255) / 256)), dim3(256), 0, s,
                     reinterpret_cast<const u32x4_t*>(codes), scales, dst, nmat, R, C, down ? 2 : 1);
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
