// Forward expert GEMMs on 4-bit weights with group scales.
//
//   W[r][c] = s[r][c / G] (q[r][c] - 8),  q in 0..15,  G = 32, 64 or 128
//   gate/up: h[p][n] = silu(x[tok(p)] . W_g[e][n]) * (x[tok(p)] . W_u[e][n])
//   down:    y[p][n] = h[p] . W_d[e][n]
// for the rows p of expert e's segment of the dispatch order; x and h in
// bf16, every sum in fp32, h rounded to bf16 (the operand of the next
// product), y kept in fp32 for the combine.
//
// A decode step gives an expert a handful of rows, so it is bound by the
// weights' bytes, a quarter of bf16's: the kernel is built to stream them.
//  - The codes lie in the order in which a wavefront feeds them to the matrix
//    cores: 1 KB holds 16 output columns and 128 reduction steps, lane l's 16
//    bytes are column l % 16, steps 32 t + 8 (l / 16) .. + 7 of t = 0..3: the
//    B operands of four v_mfma_f32_16x16x32_bf16.  One load a lane, no LDS.
//  - A code becomes a bf16 without a conversion: 0x4300 | q is 128 + q
//    exactly, so 8 codes cost 7 integer operations.  The offset is taken
//    out by the matrix cores as well: the sum of -136 x over the group (one
//    more step per row block, shared by all columns) is where each column's
//    sum starts, which leaves sum of x (q - 8) of the group.  Intermediate
//    sums are up to 136 |x| large, so a group's sum carries an error of about
//    136 * 2^-24 sum |x|, 2^-9 of a bf16 half step of x itself.  An
//    infinity in a row gives NaN.
//  - The scale multiplies the group's fp32 sum, not each weight.
//  - The four wavefronts of a workgroup split the reduction and add their
//    sums through LDS in order, so few rows still give many workgroups with
//    many loads in flight, and there is no barrier in the loop.
// Measured at 256 tokens of the layer d = 6144, N = 512, I = 2048, K = 12 (G =
// 128): gate/up 0.99 ms, its 6.5 GB read once at 6.6 TB/s; down 0.55 ms, 5.9 TB/s.
// One token: 21 us (104 MB, 5.0 TB/s) and 11 us.
//
// Weights of one set (N matrices [R][C]): codes [N][R/16][C/128][1 KB], then
// scales [N][R/16][C/128][16 columns][128/G] in bf16.  In a lane's 4 bytes of
// a step t, the code of step 2 p is at bit 4 p, that of 2 p + 1 at 16 + 4 p:
// (word >> 4 p) & 0x000f000f is register p of the operand.
#include "zc_common.h"

namespace zc {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 128;  // reduction steps of a code block

enum { I4_SWIGLU = 0, I4_STORE = 1 };

// What a workgroup has to know of its row tile, in one load: the expert, the
// first of the expert's row tiles and their number, its first row and the end
// of its rows.
struct __align__(32) Tile {
  int32_t e, mt0, mte, seg0, seg1, pad[3];
};
static_assert(sizeof(Tile) == kInt4TileBytes, "the workspace holds them");

struct I4Params {
  int N, ncols, K;          // experts, output columns (I or d), reduction length (d or I)
  const int32_t* total;     // number of row tiles
  const Tile* tiles;        // one of each (as many as the grid has row tiles)
  const bf16_t* A;          // x [T][d] gathered through perm, or h [P][I]
  uint32_t a_bytes;         // its size where 31 bits hold it
  const int32_t* perm;      // gate/up only
  int kdiv;                 // K of the layer (slot -> token)
  const uint8_t* B;         // W_g or W_d
  const uint8_t* B2;        // W_u (gate/up)
  bf16_t* h;                // gate/up output [P][I]
  float* y;                 // down output [P][d]
  int64_t per_xcd;          // tiles of an XCD, at most
  int log_run;              // runs of consecutive tiles on one XCD
};

__device__ __forceinline__ float silu_f(float a) {
  return a * __builtin_amdgcn_rcpf(1.0f + __expf(-a));
}

// Keeps memory reads in the order written (the LDS reads of one matrix step
// behind the step before: hoisted together, a slab's fragments do not fit the
// registers).
__device__ __forceinline__ void step_end() { asm volatile("" ::: "memory"); }

// The lane number, taken anew for each tile: what is computed from it would
// otherwise be moved out of the tile loop, and fill the registers for good.
__device__ __forceinline__ int tile_lane() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t voff, int soff) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0);
}

// The bf16 scales of one column's NG groups of a code block, in whole registers:
// with one group a lane loads the word that holds its column's scale and its
// neighbour's (a 16-bit load is widened where it lands, so it would be waited
// for a slab early).
template <int NG>
struct Scales {
  uint32_t w[(NG + 1) / 2];
  static __device__ __forceinline__ uint32_t lane_offset(int column) {
    return NG == 1 ? (column & ~1) * 2 : column * NG * 2;
  }
  __device__ __forceinline__ void load(const uint8_t* p) {
    constexpr int n = NG == 1 ? 4 : 2 * NG;
    __builtin_memcpy(w, __builtin_assume_aligned(p, n), n);
  }
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t voff, int soff) {
    if constexpr (NG == 4) {
      const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(r, voff, soff, 0);
      w[0] = v[0];
      w[1] = v[1];
    } else {
      w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, voff, soff, 0);
    }
  }
  // upper: 16 where the lane's column is even, else 0 (one group)
  __device__ __forceinline__ float get(int g, int upper) const {
    const uint32_t v = NG == 1 ? w[0] << upper : g & 1 ? w[g / 2] : w[g / 2] << 16;
    return __uint_as_float(v & 0xffff0000u);
  }
};

// Keeps the scaling of a group's sums where it is written: moved behind the
// next loads, the sums of every column and group are live at once.
__device__ __forceinline__ void settle(f32x4_t& v) { asm volatile("" : "+v"(v)); }

// A wave-uniform read of a table written before this kernel, as scalar loads.
__device__ __forceinline__ Tile ld_tile(const Tile* t) {
  typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));
  const i32x8_t v = *(const __attribute__((address_space(4))) i32x8_t*)t;
  return Tile{v[0], v[1], v[2], v[3], v[4], {0, 0, 0}};
}

// Tile number of the in-th tile of XCD x: runs of 2^log_run consecutive tiles
// are dealt to the 8 XCDs (workgroup b runs on XCD b mod 8), so that the row
// tiles of a weight panel, next to each other, read it from one L2.  (Without
// the number of tiles: a workgroup's record and that number are loaded
// together.)
constexpr int kMaxLogRun = 6;
__device__ __forceinline__ int64_t tile_of(int x, int64_t in, int log_run) {
  return (((in >> log_run) * 8 + x) << log_run) + (in & ((1 << log_run) - 1));
}

// Eight codes -> 128 + q in bf16.
// (The two constants come in registers, one of them a vector one, so that
// each pair is a shift and one and-or.)
__device__ __forceinline__ bf16x8_t codes_bf16(uint32_t w, uint32_t mask, uint32_t exponent) {
  u32x4_t r;
#pragma unroll
  for (int p = 0; p < 4; ++p) r[p] = ((w >> (4 * p)) & mask) | exponent;
  return __builtin_bit_cast(bf16x8_t, r);
}

// RB blocks of 16 rows and NB blocks of 16 weight columns a workgroup (gate/up:
// the first half of them gate, the second the matching up columns).
template <int EPI, int RB, int NB, int G>
__global__ __launch_bounds__(kThreads, 2) void int4_kernel(I4Params p) {
  constexpr int NG = kStep / G;                             // groups of a code block
  constexpr int TG = 4 / NG;                                // MFMA steps of a group
  constexpr int OUT = (EPI == I4_SWIGLU ? NB / 2 : NB) * 16;  // output columns a workgroup
  constexpr int TM = 16 * RB;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  const int NT = p.ncols / OUT;
  const int64_t total = static_cast<int64_t>(ld_scalar(p.total)) * NT;
  __shared__ float s_acc[kWaves][RB * NB * 4][64];
  for (int64_t in = blockIdx.x / 8;; in += gridDim.x / 8) {
  const int64_t L = tile_of(blockIdx.x % 8, in, p.log_run);
  if (in >= p.per_xcd) break;
  const Tile tile = ld_tile(p.tiles + L / NT);
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
    if (EPI == I4_SWIGLU) src[rb] = p.perm[src[rb]];
  }
  const int nkb = p.K / kStep;
  const int64_t mat = static_cast<int64_t>(p.ncols) * p.K;  // weights of one matrix
  const uint8_t* code[NB];  // wave-uniform
  const uint8_t* scale[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const bool up = EPI == I4_SWIGLU && nb >= NB / 2;
    const uint8_t* base = up ? p.B2 : p.B;
    const int cb = nt * (OUT / 16) + (up ? nb - NB / 2 : nb);
    code[nb] = base + e * (mat / 2) + static_cast<int64_t>(cb) * nkb * 1024;
    scale[nb] = base + p.N * (mat / 2) + (e * (mat / G) + static_cast<int64_t>(cb) * nkb * 16 * NG) * 2;
  }
  const uint32_t code_lane = lane * 16, scale_lane = Scales<NG>::lane_offset(l16);
  const int upper = l16 & 1 ? 0 : 16;

  struct Buf {
    u32x4_t b[NB];
    Scales<NG> s[NB];
    bf16x8_t a[RB][4];
  };
  const bf16_t* arow[RB];
  auto load_codes = [&](int kb, Buf& f) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
      f.b[nb] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4_t*>(code[nb] + kb * 1024 + code_lane));
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
      f.s[nb].load(scale[nb] + kb * (32 * NG) + scale_lane);
  };
  auto load_rows = [&](int kb, Buf& f) {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        f.a[rb][t] = *reinterpret_cast<const bf16x8_t*>(arow[rb] + kb * kStep + 32 * t);
  };
  auto load = [&](int kb, Buf& f) {
    load_codes(kb, f);
    load_rows(kb, f);
  };

  f32x4_t acc[RB][NB];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[rb][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const u32x4_t off_bits = {0xc308c308u, 0xc308c308u, 0xc308c308u, 0xc308c308u};  // -136
  const bf16x8_t off = __builtin_bit_cast(bf16x8_t, off_bits);
  uint32_t mask = 0x000f000fu, exponent = 0x43004300u;
  asm volatile("" : "+s"(mask), "+v"(exponent));

  auto compute = [&](const Buf& f) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      f32x4_t start[RB];
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        start[rb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = g * TG; t < (g + 1) * TG; ++t)
          start[rb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.a[rb][t], off, start[rb], 0, 0, 0);
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        f32x4_t part[RB];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) part[rb] = start[rb];
#pragma unroll
        for (int t = g * TG; t < (g + 1) * TG; ++t) {
          const bf16x8_t w = codes_bf16(f.b[nb][t], mask, exponent);
#pragma unroll
          for (int rb = 0; rb < RB; ++rb)
            part[rb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.a[rb][t], w, part[rb], 0, 0, 0);
        }
        const float s = f.s[nb].get(g, upper);
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[rb][nb][v] += s * part[rb][v];
      }
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) settle(acc[rb][nb]);
    }
  };

  // this wavefront's share of the reduction, one block ahead in registers
  const int kb0 = nkb * wave / kWaves, kb1 = nkb * (wave + 1) / kWaves;
  if (kb0 < kb1) {
    Buf f0, f1;
    // the first codes are under way before the rows' tokens are known
    load_codes(kb0, f0);
    step_end();
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
      arow[rb] = p.A + static_cast<int64_t>(EPI == I4_SWIGLU ? src[rb] / p.kdiv : src[rb]) * p.K + 8 * lq;
    load_rows(kb0, f0);
    int kb = kb0;
    for (; kb + 2 <= kb1; kb += 2) {
      load(kb + 1, f1);
      compute(f0);
      if (kb + 2 < kb1) load(kb + 2, f0);
      compute(f1);
    }
    if (kb < kb1) compute(f0);
  }

  // the wavefronts' sums, added in order; wavefront w finishes its share of
  // the tile.  Register v of block (rb, nb): row 16 rb + 4 (lane / 16) + v,
  // column 16 nb + lane % 16.
  __syncthreads();  // the previous tile's sums have been read
#pragma unroll
  for (int rb = 0; rb < RB; ++rb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int v = 0; v < 4; ++v) s_acc[wave][(rb * NB + nb) * 4 + v][lane] = acc[rb][nb][v];
  __syncthreads();
  auto sum = [&](int rb, int nb, int v) {
    const int i = (rb * NB + nb) * 4 + v;
    return ((s_acc[0][i][lane] + s_acc[1][i][lane]) + s_acc[2][i][lane]) + s_acc[3][i][lane];
  };
  // wavefront w takes register v = w of every block
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const int r = 16 * rb + 4 * lq + wave;
    if (r >= mcount) continue;
    const int64_t row = (static_cast<int64_t>(m0) + r) * p.ncols + nt * OUT + l16;
    if constexpr (EPI == I4_SWIGLU) {
#pragma unroll
      for (int nb = 0; nb < NB / 2; ++nb)
        p.h[row + 16 * nb] = f2bf(silu_f(sum(rb, nb, wave)) * sum(rb, nb + NB / 2, wave));
    } else {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) p.y[row + 16 * nb] = sum(rb, nb, wave);
    }
  }
  }
}

// ------------------------------------------------------------- many rows
// With more than some 20 rows an expert (int4_rows_per_tile) each decoded weight
// has to feed many rows, and what bounds the products is the matrix cores and the
// vector work beside them: 16384 tokens of that layer take 7.0 to 7.4 ms in gate/up,
// 0.9 PFLOP/s, and 3.8 to 4.0 in down; 4096 tokens of d = 1024, N = 64, I = 512 (G = 64)
// 63 and 40 us, matrix cores busy 36% and 30%, vector issue 57% and 44%.  A workgroup then
// takes 64 rows and 256 weight columns over the whole reduction, a
// wavefront 64 rows and 64 columns (gate/up: 32 gate and the matching 32 up
// columns); 64 x 64 sums and as many of the group at hand fill half of a
// SIMD's registers, so two workgroups share a CU and one's vector work (codes
// decoded, sums scaled), copies and stores run under the other's matrix steps.
//  - The rows' 128-step slabs come through a ring of four LDS slots, copied
//    by the loads themselves (16 bytes a lane, gathered rows); chunk c
//    (16 bytes) of row r lies at chunk c ^ (r & 15), so the 16 lanes of a
//    read phase hit 16 different bank groups.
//  - The sums of -136 x that start each column's sum are shared out: a
//    wavefront makes those of one row block for the next slab and leaves them
//    in LDS, 1 matrix step beside 16.
//  - A group's sums are scaled into the accumulators column block by column
//    block, behind the matrix steps of the next one.
// Each slab issues the copies of the slab three ahead and the codes of the next.
// Loads return in issue order, so where slab k waits until only the issues of
// slab k - 1 are in flight, the rows of slab k + 1 have landed; the barrier
// then shows them to every wavefront, and frees the slot of slab k - 1 for
// slab k + 3.
typedef __attribute__((address_space(3))) void lds_void;
// (A buffer load: the compiler would have every LDS read wait for all copies in
// flight if they were global loads into LDS.)
__device__ __forceinline__ void copy_to_lds16(__amdgpu_buffer_rsrc_t r, lds_void* dst,
                                              uint32_t voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, dst, 16, voff, soff, 0, 0);
}
// s_waitcnt immediate for "vmcnt <= n" (expcnt and lgkmcnt not waited)
constexpr int vmcnt_imm(int n) { return 0x0f70 | (n & 15) | ((n >> 4) << 14); }
constexpr int kAllLoads = vmcnt_imm(0);
// Barrier for LDS alone: loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int EPI, int G>
__global__ __launch_bounds__(kThreads, 2) void int4_wide_kernel(I4Params p) {
  constexpr int RB = 4, NB = 4, NG = kStep / G, TG = 4 / NG;
  constexpr int TM = 16 * RB;
  constexpr int SLOT = TM * kStep;  // bf16 of a ring slot
  constexpr int OUT = EPI == I4_SWIGLU ? 128 : 256;
  constexpr int CP = 4;             // copies a wavefront and slab: 4 rows each
  // the ring, then the starts [slab parity][group][row / 4] (one LDS object: with
  // two, the compiler has LDS reads wait for copies in flight)
  constexpr int kStartWords = 2 * NG * (TM / 4) * 8;  // bf16 of LDS they take
  __shared__ __align__(16) bf16_t ring[4 * SLOT + 2 * kStartWords + 256 * 8];
  f32x4_t* const s_start = reinterpret_cast<f32x4_t*>(ring + 4 * SLOT);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nkb = p.K / kStep;
  const int NT = (p.ncols + OUT - 1) / OUT;
  const __amdgpu_buffer_rsrc_t rows = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<bf16_t*>(p.A), (short)0, p.a_bytes, 0x00020000);
  const int64_t total = static_cast<int64_t>(ld_scalar(p.total)) * NT;
  for (int64_t in = blockIdx.x / 8;; in += gridDim.x / 8) {
    const int64_t L = tile_of(blockIdx.x % 8, in, p.log_run);
    if (in >= p.per_xcd) break;
    const Tile tile = ld_tile(p.tiles + L / NT);
    if (L >= total) break;
    const int lane = tile_lane(), l16 = lane & 15, lq = lane >> 4;
    const int e = tile.e;
    const int q = static_cast<int>(L - static_cast<int64_t>(tile.mt0) * NT);
    const int nt = q / tile.mte;
    const int m0 = tile.seg0 + TM * (q % tile.mte);
    const int mcount = min(TM, tile.seg1 - m0);

    // copies: instruction i of this wavefront fills rows 4 (CP wave + i) + lq
    // (rows past the tile with its last row); byte offsets fit 31 bits, the
    // launch made sure
    uint32_t src[CP];
#pragma unroll
    for (int i = 0; i < CP; ++i) {
      const int r = 4 * (CP * wave + i) + lq;
      const int row = m0 + min(r, mcount - 1);
      const int tok = EPI == I4_SWIGLU ? p.perm[row] / p.kdiv : row;
      src[i] = (static_cast<uint32_t>(tok) * static_cast<uint32_t>(p.K) + 8 * (l16 ^ (r & 15))) * 2;
    }
    auto copy = [&](int kb, int slot) {
#pragma unroll
      for (int i = 0; i < CP; ++i)
        copy_to_lds16(rows, (lds_void*)(ring + (slot & 3) * SLOT + 4 * (CP * wave + i) * kStep),
                      src[i], kb * (2 * kStep));
    };

    // this wavefront's columns; past the matrix (the last tile of a width that
    // is no multiple of 256) its last ones again, not stored.  Loaded through
    // buffer resources: a base, a scalar offset and one lane offset, where
    // eight pairs of address registers would not fit.
    const int64_t mat = static_cast<int64_t>(p.ncols) * p.K;
    __amdgpu_buffer_rsrc_t codes[2], scales[2];  // gate (or down) and up
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      uint8_t* base = const_cast<uint8_t*>(EPI == I4_SWIGLU && m ? p.B2 : p.B);
      codes[m] = __builtin_amdgcn_make_buffer_rsrc(base + e * (mat / 2), (short)0, 0xffffffffu,
                                                   0x00020000);
      scales[m] = __builtin_amdgcn_make_buffer_rsrc(base + p.N * (mat / 2) + e * (mat / G) * 2,
                                                    (short)0, 0xffffffffu, 0x00020000);
    }
    uint32_t col[NB];  // first code block of each column block
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
      col[nb] = (EPI == I4_SWIGLU ? nt * 8 + 2 * wave + (nb & 1)
                                  : min(nt * 16 + 4 * wave + nb, p.ncols / 16 - 1)) * nkb;
    const uint32_t code_lane = lane * 16, scale_lane = Scales<NG>::lane_offset(l16);
    const int upper = l16 & 1 ? 0 : 16;
    struct Buf {
      u32x4_t b[NB];
      Scales<NG> s[NB];
    };
    auto load = [&](int kb, Buf& f) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        f.b[nb] = load16(codes[EPI == I4_SWIGLU ? nb / 2 : 0], code_lane, (col[nb] + kb) * 1024);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
        f.s[nb].load(scales[EPI == I4_SWIGLU ? nb / 2 : 0], scale_lane, (col[nb] + kb) * (32 * NG));
    };

    const u32x4_t off_bits = {0xc308c308u, 0xc308c308u, 0xc308c308u, 0xc308c308u};  // -136
    const bf16x8_t off = __builtin_bit_cast(bf16x8_t, off_bits);
    uint32_t mask = 0x000f000fu, exponent = 0x43004300u;
    asm volatile("" : "+s"(mask), "+v"(exponent));
    auto frag = [&](int kb, int rb, int t) {  // row block rb of the whole tile
      return *reinterpret_cast<const bf16x8_t*>(ring + (kb & 3) * SLOT + (16 * rb + l16) * kStep +
                                                8 * ((4 * t + lq) ^ l16));
    };
    // Sums of -136 x over slab kb's groups, of row block `wave` of the tile (past
    // the last slab: of what the slot holds, and unused).  The 16 lanes of a
    // row quad hold the same sums: the first leaves them in LDS, the others write
    // to a place of their own that nobody reads (no branch).
    bf16_t* const start_out =
        ring + 4 * SLOT + 8 * (l16 == 0 ? 4 * wave + lq : kStartWords / 8 + (threadIdx.x & 255));
    auto starts = [&](int kb) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = g * TG; t < (g + 1) * TG; ++t)
          v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(kb, wave, t), off, v, 0, 0, 0);
        *reinterpret_cast<f32x4_t*>(start_out + ((kb & 1) * NG + g) * (TM / 4) * 8) = v;
      }
    };

    f32x4_t acc[RB][NB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) acc[rb][nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // Slab kb.  A column block's group sums are scaled into the accumulators
    // behind the last matrix steps of the next column block.
    auto compute = [&](int kb, const Buf& f) {
      f32x4_t part[RB][NB];
      auto fold = [&](int nb, int g) {
        const float s = f.s[nb].get(g, upper);
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[rb][nb][v] += s * part[rb][nb][v];
          settle(acc[rb][nb]);
        }
      };
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int g = t / TG;
        const bool first = t % TG == 0, last = t % TG == TG - 1;
        bf16x8_t a[RB];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) a[rb] = frag(kb, rb, t);
        f32x4_t st[RB];
        if (first) {
#pragma unroll
          for (int rb = 0; rb < RB; ++rb)
            st[rb] = s_start[((kb & 1) * NG + g) * (TM / 4) + 4 * rb + lq];
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const bf16x8_t w = codes_bf16(f.b[nb][t], mask, exponent);
#pragma unroll
          for (int rb = 0; rb < RB; ++rb)
            part[rb][nb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                a[rb], w, first ? st[rb] : part[rb][nb], 0, 0, 0);
          if (last && nb > 0) fold(nb - 1, g);
        }
        if (last) fold(NB - 1, g);
        step_end();
      }
    };

    Buf f0, f1;
    lds_barrier();  // the ring is free: the previous tile's reads are done
    const int last = nkb - 1;
    copy(0, 0);
    copy(min(1, last), 1);
    copy(min(2, last), 2);
    load(0, f0);
    __builtin_amdgcn_s_waitcnt(kAllLoads);
    lds_barrier();
    starts(0);
    // Slab kb.  No branch in it: past the end the last slab is copied and
    // loaded again, so that the number of loads in flight is known.
    auto slab = [&](int kb, const Buf& cur, Buf& next) {
      // slab kb + 1 has landed: younger are only the copies and loads of the slab
      // before this one
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(CP + 2 * NB));
      lds_barrier();
      copy(min(kb + 3, last), kb + 3);
      load(min(kb + 1, last), next);
      __builtin_amdgcn_sched_barrier(0);
      starts(kb + 1);
      compute(kb, cur);
    };
    int kb = 0;
    for (; kb + 2 <= nkb; kb += 2) {
      slab(kb, f0, f1);
      slab(kb + 1, f1, f0);
    }
    if (kb < nkb) slab(kb, f0, f1);
    __builtin_amdgcn_s_waitcnt(kAllLoads);  // no copy of this tile lands in the next one's ring

#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int r = 16 * rb + 4 * lq + v;
        if (r >= mcount) continue;
        const int64_t row = (static_cast<int64_t>(m0) + r) * p.ncols + nt * OUT + l16;
        if constexpr (EPI == I4_SWIGLU) {
#pragma unroll
          for (int nb = 0; nb < 2; ++nb)
            p.h[row + 32 * wave + 16 * nb] = f2bf(silu_f(acc[rb][nb][v]) * acc[rb][nb + 2][v]);
        } else if (nt * OUT + 64 * wave < p.ncols) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) p.y[row + 64 * wave + 16 * nb] = acc[rb][nb][v];
        }
      }
  }
}

// Natural layout (two codes a byte, the even step in the low half; scales
// [R][C/G]) -> the layout above.  One thread per 8 codes.
__global__ __launch_bounds__(256) void int4_pack_kernel(const uint32_t* __restrict__ codes,
                                                        const bf16_t* __restrict__ scales,
                                                        uint8_t* __restrict__ dst, int64_t nmat,
                                                        int R, int C, int G) {
  const int64_t words = nmat * R * (C / 8);
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = i0; i < words; i += step) {
    // i = (((mat R/16 + rb) C/128 + kb) 64 + lane) 4 + t
    const int t = i & 3, lane = (i >> 2) & 63;
    const int64_t blk = i >> 8;
    const int kb = static_cast<int>(blk % (C / kStep));
    const int64_t row = blk / (C / kStep) * 16 + (lane & 15);
    const uint32_t w = codes[row * (C / 8) + kb * 16 + t * 4 + (lane >> 4)];
    uint32_t v = 0;
#pragma unroll
    for (int p = 0; p < 4; ++p)
      v |= ((w >> (8 * p)) & 0xfu) << (4 * p) | ((w >> (8 * p + 4)) & 0xfu) << (16 + 4 * p);
    reinterpret_cast<uint32_t*>(dst)[i] = v;
  }
  const int64_t ns = nmat * R * (C / G);
  for (int64_t i = i0; i < ns; i += step) {
    // i = ((mat R/16 + rb) C/128 + kb) 16 NG + column NG + g
    const int NG = kStep / G, g = static_cast<int>(i % NG);
    const int64_t j = i / NG;
    const int64_t blk = j >> 4;
    const int kb = static_cast<int>(blk % (C / kStep));
    const int64_t row = blk / (C / kStep) * 16 + (j & 15);
    reinterpret_cast<bf16_t*>(dst + words * 4)[i] = scales[row * (C / G) + kb * NG + g];
  }
}

// bf16 rows -> codes and scales in the natural layout: s = bf16(max|w| / 7),
// q = nearest of w / s (ties to even) clamped to -8..7, plus 8; a group of
// zeros (or whose scale rounds to 0) has s = 0 and q = 8, a group with a NaN
// or an infinity the scale NaN.  One thread per 8 values.
__global__ __launch_bounds__(256) void int4_quantize_kernel(const bf16_t* __restrict__ src,
                                                            int64_t groups8, int G,
                                                            uint32_t* __restrict__ codes,
                                                            bf16_t* __restrict__ scales) {
  // (a group's lanes take the same rounds: C is a multiple of 128)
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < groups8;
       i += static_cast<int64_t>(gridDim.x) * 256) {
  float f[8];
  V16<bf16_t>::load(src + i * 8, f);
  float m = 0.f;
  bool bad = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    bad |= !(fabsf(f[e]) <= 3.402823466e38f);
    m = fmaxf(m, fabsf(f[e]));
  }
  int b = bad;
  for (int o = 1; o < G / 8; o <<= 1) {
    m = fmaxf(m, __shfl_xor(m, o));
    b |= __shfl_xor(b, o);
  }
  const bf16_t sb = b ? static_cast<bf16_t>(0x7fc0) : f2bf(m / 7.0f);
  const float s = bf2f(sb);
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    int q = 8;
    if (!b && s > 0.f) q = static_cast<int>(fminf(fmaxf(rintf(f[e] / s), -8.f), 7.f)) + 8;
    w |= static_cast<uint32_t>(q) << (4 * e);
  }
  codes[i] = w;
  if (i % (G / 8) == 0) scales[i / (G / 8)] = sb;
  }
}

// Grids beyond this many workgroups go round again (a launch holds fewer than
// 2^32 threads).
constexpr int64_t kMaxGrid = int64_t(1) << 20;
unsigned grid_of(int64_t blocks) {
  return static_cast<unsigned>(blocks < kMaxGrid ? blocks : kMaxGrid);
}

// The records of the row tiles of height tm, in expert order, and their number.
// One workgroup: inclusive scan of the experts' tile counts by wavefront, then
// over the 16 wavefronts' sums.
__global__ __launch_bounds__(kMaxExperts) void int4_tiles_kernel(
    const int32_t* __restrict__ offsets, int N, int tm, int32_t* __restrict__ total,
    Tile* __restrict__ tiles) {
  __shared__ int32_t s_sum[kMaxExperts / 64];
  const int e = threadIdx.x, lane = e & 63, wave = e >> 6;
  const int lo = e < N ? offsets[e] : 0, hi = e < N ? offsets[e + 1] : 0;
  const int n = (hi - lo + tm - 1) / tm;
  int scan = n;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 63) s_sum[wave] = scan;
  __syncthreads();
  int first = scan - n;
  for (int w = 0; w < wave; ++w) first += s_sum[w];
  if (e == kMaxExperts - 1) *total = first + n;
  Tile t{e, first, n, lo, hi, {0, 0, 0}};
  for (int i = 0; i < n; ++i) tiles[first + i] = t;
}

// At most this many column tiles of OUT columns by row tiles of height tm; the
// row tiles rounded up so that the runs of tile_of stay inside the records.
template <typename K>
hipError_t launch_tiles(K kernel32, K kernel64, K kernel128, I4Params p, int G, int64_t rows, int tm,
                        int OUT, hipStream_t s) {
  const int64_t NT = (p.ncols + OUT - 1) / OUT;
  const int64_t most = int4_max_tiles(rows, p.N, tm) * NT;
  // runs of 8 tiles, longer ones while every XCD has at least 32 of them
  p.log_run = 3;
  while (p.log_run < kMaxLogRun && (most >> p.log_run) >= 8 * 64) ++p.log_run;
  const int64_t round = int64_t(8) << p.log_run;
  p.per_xcd = (most + round - 1) / round << p.log_run;
  const dim3 grid(grid_of(p.per_xcd * 8)), block(kThreads);
  hipLaunchKernelGGL(G == 32 ? kernel32 : G == 64 ? kernel64 : kernel128, grid, block, 0, s, p);
  return hipGetLastError();
}
template <int EPI, int RB, int NB>
hipError_t launch_int4(const I4Params& p, int G, int64_t rows, hipStream_t s) {
  return launch_tiles(int4_kernel<EPI, RB, NB, 32>, int4_kernel<EPI, RB, NB, 64>,
                      int4_kernel<EPI, RB, NB, 128>, p, G, rows, 16 * RB,
                      (EPI == I4_SWIGLU ? NB / 2 : NB) * 16, s);
}
template <int EPI>
hipError_t launch_int4_wide(const I4Params& p, int G, int64_t rows, hipStream_t s) {
  return launch_tiles(int4_wide_kernel<EPI, 32>, int4_wide_kernel<EPI, 64>,
                      int4_wide_kernel<EPI, 128>, p, G, rows, 64, EPI == I4_SWIGLU ? 128 : 256, s);
}

}  // namespace

// Measured at d = 6144, I = 2048, G = 128, gate/up and down together: 12 rows an
// expert 1.97 ms with 16-row tiles, 2.20 with 32, 2.44 with 64; 16 rows 2.58,
// 2.33, 2.48; 24 rows 3.47, 2.69, 2.54; 48 rows 5.6, 5.4, 2.7.
int int4_rows_per_tile(int64_t avg_rows, int64_t Tn, int64_t rows, int64_t d, int64_t I) {
  if (avg_rows <= 13) return 16;
  // (the 64-row kernel takes byte offsets of 31 bits into x, h and a matrix)
  const int64_t limit = int64_t(1) << 30;
  if (avg_rows <= 20 || Tn * d >= limit || rows * I >= limit || d * I >= limit) return 32;
  return 64;
}

// Row tiles of height tm at most: every one of the rows' experts has one ragged
// tile.
int64_t int4_max_tiles(int64_t rows, int64_t N, int tm) {
  return rows / tm + (rows < N ? rows : N);
}
// Bytes of their records and count.  tile_of reaches fewer than 8 runs of column
// tiles, so fewer row tiles than that, past the last.
int64_t int4_tiles_bytes(int64_t rows, int64_t N) {
  return kInt4TileBytes * (1 + int4_max_tiles(rows, N, 16) + (8 << kMaxLogRun));
}

hipError_t launch_int4_tiles(const int32_t* offsets, int N, int tm, void* tiles, hipStream_t s) {
  hipLaunchKernelGGL(int4_tiles_kernel, dim3(1), dim3(kMaxExperts), 0, s, offsets, N, tm,
                     static_cast<int32_t*>(tiles), static_cast<Tile*>(tiles) + 1);
  return hipGetLastError();
}

hipError_t launch_int4_gateup(const bf16_t* x, int64_t Tn, const uint8_t* wg, const uint8_t* wu,
                              int G, const void* tiles, const int32_t* perm, int tm, int64_t rows,
                              int N, int I, int d, int K, bf16_t* h, hipStream_t s) {
  I4Params p{};
  p.N = N; p.ncols = I; p.K = d;
  p.total = static_cast<const int32_t*>(tiles);
  p.tiles = static_cast<const Tile*>(tiles) + 1;
  p.A = x; p.a_bytes = static_cast<uint32_t>(Tn * d * 2); p.perm = perm; p.kdiv = K;
  p.B = wg; p.B2 = wu; p.h = h;
  // 16-row tiles: 32 columns of h a workgroup; 16 where that gives too few
  // workgroups to fill the card (one token of d = 6144, I = 2048, K = 12: 18 us
  // against 20); 64 where tiles are so full that their rows' loads count
  // (512 tokens of N = 512: 1.02 ms against 1.09; 64 tokens: 0.63 against 0.59)
  if (tm == 16 && int4_max_tiles(rows, N, 16) * (I / 32) < 1024)
    return launch_int4<I4_SWIGLU, 1, 2>(p, G, rows, s);
  if (tm == 16 && rows > 8 * N) return launch_int4<I4_SWIGLU, 1, 8>(p, G, rows, s);
  if (tm == 16) return launch_int4<I4_SWIGLU, 1, 4>(p, G, rows, s);
  if (tm == 32) return launch_int4<I4_SWIGLU, 2, 4>(p, G, rows, s);
  return launch_int4_wide<I4_SWIGLU>(p, G, rows, s);
}

hipError_t launch_int4_down(const bf16_t* h, const uint8_t* wd, int G, const void* tiles, int tm,
                            int64_t rows, int N, int I, int d, float* y, hipStream_t s) {
  I4Params p{};
  p.N = N; p.ncols = d; p.K = I;
  p.total = static_cast<const int32_t*>(tiles);
  p.tiles = static_cast<const Tile*>(tiles) + 1;
  p.A = h; p.a_bytes = static_cast<uint32_t>(rows * I * 2); p.kdiv = 1; p.B = wd; p.y = y;
  // 16-row tiles: 128 columns of y a workgroup, 64 where that gives too few (one
  // token: 11 us against 15; 256 tokens: 0.57 ms against 0.54)
  if (tm == 16 && int4_max_tiles(rows, N, 16) * (d / 128) < 4096)
    return launch_int4<I4_STORE, 1, 4>(p, G, rows, s);
  if (tm == 16) return launch_int4<I4_STORE, 1, 8>(p, G, rows, s);
  if (tm == 32) return launch_int4<I4_STORE, 2, 4>(p, G, rows, s);
  return launch_int4_wide<I4_STORE>(p, G, rows, s);
}

hipError_t launch_int4_pack(const uint8_t* codes, const bf16_t* scales, uint8_t* dst, int64_t nmat,
                            int R, int C, int G, hipStream_t s) {
  const int64_t words = nmat * R * (C / 8);  // at least the scales: G >= 32
  hipLaunchKernelGGL(int4_pack_kernel, dim3(grid_of((words + 255) / 256)), dim3(256),
                     0, s, reinterpret_cast<const uint32_t*>(codes), scales, dst, nmat, R, C, G);
  return hipGetLastError();
}

hipError_t launch_int4_quantize(const bf16_t* src, uint8_t* codes, bf16_t* scales, int64_t nmat,
                                int R, int C, int G, hipStream_t s) {
  const int64_t n = nmat * R * (C / 8);
  hipLaunchKernelGGL(int4_quantize_kernel, dim3(grid_of((n + 255) / 256)), dim3(256),
                     0, s, src, n, G, reinterpret_cast<uint32_t*>(codes), scales);
  return hipGetLastError();
}

}  // namespace zc
