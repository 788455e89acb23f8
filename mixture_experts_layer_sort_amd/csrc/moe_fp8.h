// Products on block-128 fp8 weights (e4m3 codes, one fp32 scale per 128 x 128
// block), dense and grouped over experts: the arguments of one launch, the
// activation quantiser shared by the kernels, and the launchers.
//
//   y[r, n] = sum_b s_x[r, b] s_w[n / 128, b] sum_{k in block b} c_x[r, k] c_w[n, k]
//
// The inner sum over one block of 128 is exactly one fp8 matrix instruction
// of shape 16 x 16 x 128 (weights as the 16 rows, tokens as the 16 columns),
// started from zero; its four results per lane belong to one token, so the
// block's scale s_x s_w is one fp32 number per lane and is applied by one fp32
// multiply-add per result.  Scales that are not powers of two cannot go through
// the instruction's own e8m0 scale operands without rounding them.
//
// Precision, measured on MI355X: the instruction adds products in groups of 8
// consecutive K, each cut (towards zero) to 13 bits below the exponent of the
// group's largest product; the groups' sums lose nothing more.  7168-long sums
// of quantised normal values have a relative L2 error of 1.3e-5, the same for
// every fp8 instruction shape, far below the rounding of the bf16 outputs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_device.h"

namespace moe {

constexpr int kFp8Blk = 128;           // elements per activation scale, rows and columns per weight scale
constexpr float kFp8Max = 448.f;       // largest e4m3 magnitude
constexpr float kFp8Tiny = 7.8886090522101181e-31f;  // 2^-100: smallest magnitude that sets a block's scale

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

enum Fp8Mode { FP8_DENSE = 0, FP8_GATE_UP = 1, FP8_DOWN = 2 };

// One product.  DENSE: one matrix, `rows` token rows.  GATE_UP / DOWN: expert
// e owns the sorted rows [offsets[e], offsets[e + 1]); GATE_UP reads source row
// pairs[r] / k and writes the activated row r, DOWN reads row r and writes row
// pairs[r].
struct Fp8Args {
  const uint8_t* w;      // codes [E][N][K] (GATE_UP: N = 2 I, gate rows first)
  const float* wsc;      // scales [E][ceil(N / 128)][ceil(K / 128)]
  const uint16_t* x;     // bf16 rows, leading dimension ldx (kernels that quantise themselves)
  long long ldx;
  const uint8_t* xq;     // codes [.][K rounded up to 128] (kernels that read codes)
  const float* xs;       // scales [ceil(K / 128)][xrows]
  int xrows;             // rows of xq
  const int* offsets;    // [E + 1] on the device; unused by DENSE
  const int* pairs;      // sorted pairs; unused by DENSE
  const int4* tiles;     // tile kernel: each token tile's expert, first row, and the first and number of its group
  const int* ntiles;     // their number
  uint16_t* out;         // bf16 (DENSE: [rows, ldo]; GATE_UP: h [rows, I]; DOWN: y [rows, N])
  long long ldo;
  float* part;           // streaming kernel, DENSE without codes: sums of each of `splits` runs of K blocks
  int splits;
  uint8_t* hq;           // tile kernel, GATE_UP: codes [rows, I] and scales [I / 128][rows]
  float* hs;
  int rows, E, N, K, k;
  int cap;               // streaming kernel, grouped: rows per tile (<= 16) where the block quantises them, 0: the waves do
  float limit;           // SwiGLU clamp, 0: none
};

// ------------------------------------------------------------------ exchanges between 16-lane rows

// Maximum over the lanes l, l ^ 16, l ^ 32, l ^ 48: the row swaps of gfx950
// put the other row's (other half's) value beside one's own without LDS.
__device__ __forceinline__ float max_rows(float v) {
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
// Inside each row of 16: rotations by 8, 4, 2, 1.
template <int N>
__device__ __forceinline__ float row_ror(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), 0x120 + N, 0xF, 0xF, true));
}
__device__ __forceinline__ float max_row16(float v) {
  v = fmaxf(v, row_ror<8>(v));
  v = fmaxf(v, row_ror<4>(v));
  v = fmaxf(v, row_ror<2>(v));
  return fmaxf(v, row_ror<1>(v));
}

// Four wave reductions at once: the row swaps put two values' halves (rows) beside each other, so every exchange
// serves all of them, 11 instructions instead of 4 x 10.  The result of value u is in row row4(u) of 16 lanes.
__device__ __forceinline__ constexpr int row4(int u) { return u == 1 ? 2 : u == 2 ? 1 : u; }  // its own inverse
template <class Op>
__device__ __forceinline__ float reduce4(const float (&x)[4], Op op) {
  auto swap = [&](auto r) { return op(__uint_as_float(r[0]), __uint_as_float(r[1])); };
  const float a = swap(__builtin_amdgcn_permlane32_swap(__float_as_uint(x[0]), __float_as_uint(x[1]), false, false));
  const float b = swap(__builtin_amdgcn_permlane32_swap(__float_as_uint(x[2]), __float_as_uint(x[3]), false, false));
  float v = swap(__builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false));
  v = op(v, row_ror<8>(v));
  v = op(v, row_ror<4>(v));
  v = op(v, row_ror<2>(v));
  return op(v, row_ror<1>(v));
}
__device__ __forceinline__ float of_row(float v, int u) {  // the value of u, the same for all lanes
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 16 * row4(u)));
}

// ------------------------------------------------------------------ activation quantiser

// Codes of four fp32 values with |v| <= 448 (1 + 2^-23): nearest, ties to even
// (values this close above 448 round to 448); NaN gives a NaN code.
__device__ __forceinline__ uint32_t fp8_codes4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// Largest magnitudes of the two halves of packed bf16 values, on their bits (magnitudes order like their bits; a NaN
// is larger than everything and stays).
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
constexpr uint32_t kFp8TinyBits = 0x0D800D80u;  // 2^-100 in both halves
__device__ __forceinline__ uint32_t bf16x2_amax(uint32_t v, uint32_t m) {
  u16x2 a, b;
  v &= 0x7FFF7FFFu;
  __builtin_memcpy(&a, &v, 4);
  __builtin_memcpy(&b, &m, 4);
  const u16x2 c = __builtin_elementwise_max(a, b);
  uint32_t o;
  __builtin_memcpy(&o, &c, 4);
  return o;
}
__device__ __forceinline__ uint32_t fp8_amax8(const u32x4& v, uint32_t m) {
#pragma unroll
  for (int i = 0; i < 4; ++i) m = bf16x2_amax(v[i], m);
  return m;
}
__device__ __forceinline__ float bf16x2_max(uint32_t m) { return fmaxf(bf16_lo(m), bf16_hi(m)); }  // of packed magnitudes

// Factor fp32(448 / m) and scale fp32(m / 448) of a block whose largest magnitude m is a bf16 value >= 2^-100: an
// approximate quotient and one correction by its remainder.  The remainder is exact, so the corrected quotient is off
// by 2^-46 relative before its rounding; m has 8 significant bits, so the true quotients are exact or at least 2^-9
// of an ulp away from a rounding border, and both results are the correctly rounded ones.  (m is scaled down by 2^16
// for the reciprocal, which is denormal otherwise near the top of the range.)  Infinite or NaN m: both are NaN.
__device__ __forceinline__ void fp8_factor(float m, float& f, float& s) {
  const float d = m * 0x1p-16f, r = __builtin_amdgcn_rcpf(d);
  constexpr float kNum = kFp8Max * 0x1p-16f, kInv = 1.f / kFp8Max;
  const float f0 = kNum * r;
  f = fmaf(fmaf(-f0, d, kNum), r, f0);
  const float s0 = m * kInv;
  s = fmaf(fmaf(-s0, kFp8Max, m), kInv, s0);
}

// Codes of the 8 bf16 values of v under the factor f = fp32(448 / amax).
__device__ __forceinline__ uint2 fp8_codes8(const u32x4& v, float f) {
  return make_uint2(fp8_codes4(bf16_lo(v[0]) * f, bf16_hi(v[0]) * f, bf16_lo(v[1]) * f, bf16_hi(v[1]) * f),
                    fp8_codes4(bf16_lo(v[2]) * f, bf16_hi(v[2]) * f, bf16_lo(v[3]) * f, bf16_hi(v[3]) * f));
}

__device__ __forceinline__ float swiglu(float g, float u, float limit) {
  if (limit > 0.f) {  // by comparisons, which leave a NaN as it is
    g = g > limit ? limit : g;
    u = u > limit ? limit : u < -limit ? -limit : u;
  }
  return g / (1.f + __expf(-g)) * u;
}

__device__ __forceinline__ f32x4 fp8_mfma(const i32x8& a, const i32x8& b) {
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}

// The same product from the codes as bf16 values (exact, and so are their products): four instructions, each of 8 of a
// lane's 32 values.
struct Bf16Frag {
  bf16x8 v[4];
};
__device__ __forceinline__ Bf16Frag bf16_frag(const i32x8& c) {
  Bf16Frag o;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    union {
      bf16x2 p[4];
      bf16x8 v;
    } u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      u.p[2 * i] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[2 * j + i], 1.f, false);
      u.p[2 * i + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[2 * j + i], 1.f, true);
    }
    o.v[j] = u.v;
  }
  return o;
}
__device__ __forceinline__ f32x4 bf16_mfma(const Bf16Frag& a, const Bf16Frag& b) {
  f32x4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 4; ++j) z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[j], b.v[j], z, 0, 0, 0);
  return z;
}

// ------------------------------------------------------------------ launchers

hipError_t launch_fp8_quantize_weights(int count, int rows, int K, const float* w, uint8_t* codes, float* scales,
                                       hipStream_t s);
// xq [M][Kp], xs [Kp / 128][M] of x's M rows, Kp = K rounded up to 128 (columns past K: zero codes)
hipError_t launch_fp8_quantize_rows(int M, int K, const uint16_t* x, long long ldx, uint8_t* xq, float* xs,
                                    hipStream_t s);
// The same, and beside it the token tiles of `tile` sorted rows of every expert, in groups of up to kFp8TileGroup tiles
// of one expert: tiles[i] = (expert, first row, first tile of the group, tiles in it).
hipError_t launch_fp8_quantize_tokens(int T, int K, const uint16_t* x, uint8_t* xq, float* xs, const int* offsets,
                                      int E, int tile, int4* tiles, int* ntiles, hipStream_t s);
// The tiled kernel (reads codes).  Grouped modes: `tile` sorted rows per token tile, token_tiles: at least their number.
hipError_t launch_fp8_tile(Fp8Mode mode, const Fp8Args& a, int tile, long long token_tiles, int cus,
                           hipStream_t s);
int fp8_tile_tokens(long long rows, int experts);  // sorted rows per tile of the grouped modes
constexpr int kFp8TileTokensMin = 64;
constexpr int kFp8TileGroup = 4;  // tiles of an expert that share a weight slab next to each other (8192 tokens: 4.26 -> 4.22 ms)
// The streaming kernel (few token rows per weight matrix).  DENSE: reads codes (xq, xs), or with xq null and
// fp8_decode_fits() quantises x itself; the grouped modes quantise x themselves.
bool fp8_decode_fits(int M, int K);
// Small dense products: K over `splits` (> 1) runs of blocks, whose sums part [splits][M][N rounded up to 16] a second
// launch adds; 1: not this way.
int fp8_splits(int M, int N, int K);
size_t fp8_split_bytes(int max_M, int N, int K);  // of part for any M <= max_M
int fp8_block_rows(int T, int K);  // Fp8Args::cap of grouped products of T tokens, 0: they do not fit
hipError_t launch_fp8_split(const Fp8Args& a, hipStream_t s);
hipError_t launch_fp8_stream(Fp8Mode mode, const Fp8Args& a, int cus, hipStream_t s);

}  // namespace moe
