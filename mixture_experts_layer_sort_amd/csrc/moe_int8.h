// Products on 8-bit integer weights with one fp32 scale per output channel, dense
// and grouped over experts: the arguments of one launch and the launchers.
//
//   y[r, n] = s_x[r] s_w[n] sum_k c_x[r, k] c_w[n, k]
//
// Rows are quantised with one scale each: amax = max(max |x|, 2^-100), s_x =
// fp32(amax / 127), c = round(fp32(x fp32(127 / amax))), ties to even.  The sums
// are integers of 32 bits and exact (|c_w c_x| <= 128 127, K <= 2^17), so they do
// not depend on how a kernel cuts them up: every kernel gives the same bits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_device.h"
#include "moe_fp8.h"  // u32x4, f32x4, packed magnitudes, swiglu

namespace moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr float kInt8Max = 127.f;
constexpr int kInt8Pad = 128;  // code rows are this many bytes, rounded up; the rest is zero

enum Int8Mode { INT8_DENSE = 0, INT8_GATE_UP = 1, INT8_DOWN = 2 };

// One product.  DENSE: one matrix, `rows` token rows.  GATE_UP / DOWN: expert e owns the sorted rows [offsets[e],
// offsets[e + 1]); GATE_UP reads source row pairs[r] / k and writes the activated row r, DOWN reads row r and writes row
// pairs[r].
struct Int8Args {
  const int8_t* w;      // codes [E][N][K] (GATE_UP: N = 2 I, gate rows first)
  const float* wsc;     // scales [E][N]
  const uint16_t* x;    // bf16 rows, ldx apart (kernels that quantise themselves)
  long long ldx;
  const int8_t* xq;     // codes [xrows][K rounded up to 128] (kernels that read codes)
  const float* xs;      // scales [xrows]
  int xrows;
  const int* offsets;   // [E + 1] on the device; unused by DENSE
  const int* pairs;     // sorted pairs; unused by DENSE
  const int4* tiles;    // tiled kernel: token tiles
  const int* ntiles;
  int* sums;            // tiled kernel, DENSE with splits > 1: [splits][rows][int8_sums_ld(N)]
  int splits;           // runs of K blocks, of different blocks of the launch (0, 1: one)
  uint16_t* out;        // bf16 rows, ldo apart (GATE_UP: the intermediate)
  long long ldo;
  int rows, E, N, K, k;
  int cap;              // streaming kernel, grouped: rows per tile (<= 16) where the block quantises them, 0: codes
  float limit;          // SwiGLU clamp, 0: none
};

__host__ __device__ __forceinline__ int int8_pad(int K) { return (K + kInt8Pad - 1) / kInt8Pad * kInt8Pad; }

// Factor fp32(127 / m) and scale fp32(m / 127) of a row of bf16 values whose largest magnitude is m >= 2^-100, both by
// correctly rounded divisions.  Infinite or NaN m: scale NaN (every output of the row is), factor 0 (codes 0).
__device__ __forceinline__ void int8_factor(float m, float& f, float& s) {
  const bool ok = m < INFINITY;
  f = ok ? kInt8Max / m : 0.f;
  s = ok ? m / kInt8Max : __uint_as_float(0x7FC00000u);
}

// Codes of 4 and 8 values under the factor f: magnitudes are at most 127 (1 + 2^-23), which rounds to 127.  Added to 1.5
// 2^23 a value is rounded to its integer (ties to even), which is the sum's last byte then.  A value that is not finite
// has f = 0: its product is the quiet NaN, whose last byte is 0.
__device__ __forceinline__ uint32_t int8_codes4(float a, float b, float c, float d) {
#pragma clang fp contract(off)  // a value is rounded before the addition: not one fused operation with the product
  constexpr float kRound = 12582912.f;
  auto bits = [](float v) {
#pragma clang fp contract(off)
    return __float_as_uint(v + kRound);
  };
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(bits(d), bits(c), 0x0C0C0400u),
                               __builtin_amdgcn_perm(bits(b), bits(a), 0x0C0C0400u), 0x05040100u);
}
__device__ __forceinline__ uint2 int8_codes8(const u32x4& v, float f) {
  return make_uint2(int8_codes4(bf16_lo(v[0]) * f, bf16_hi(v[0]) * f, bf16_lo(v[1]) * f, bf16_hi(v[1]) * f),
                    int8_codes4(bf16_lo(v[2]) * f, bf16_hi(v[2]) * f, bf16_lo(v[3]) * f, bf16_hi(v[3]) * f));
}

// 16 x 16 x 64: lane r + 16 q holds bytes [16 q, 16 q + 16) of weight row r and of token r; element i of its result is
// weight row 4 q + i, token r.
__device__ __forceinline__ i32x4 int8_mfma(const u32x4& a, const u32x4& b, const i32x4& c) {
  i32x4 x, y;
  __builtin_memcpy(&x, &a, 16);
  __builtin_memcpy(&y, &b, 16);
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(x, y, c, 0, 0, 0);
}

// ------------------------------------------------------------------ launchers

hipError_t launch_int8_quantize_weights(int count, int rows, int K, const float* w, int8_t* codes, float* scales,
                                        hipStream_t s);
// xq [M][Kp], xs [M] of x's M rows, Kp = K rounded up to 128 (bytes past K: zero)
hipError_t launch_int8_quantize_rows(int M, int K, const uint16_t* x, long long ldx, int8_t* xq, float* xs,
                                     hipStream_t s);
// The same, and beside it the token tiles of `tile` sorted rows of every expert.
hipError_t launch_int8_quantize_tokens(int T, int K, const uint16_t* x, int8_t* xq, float* xs, const int* offsets,
                                       int E, int tile, int4* tiles, int* ntiles, hipStream_t s);
// The streaming kernel (few token rows per weight matrix): reads codes, or where a.cap > 0 (grouped) and
// int8_decode_fits() (DENSE with xq null) quantises the rows itself.
bool int8_decode_fits(int M, int K);
int int8_block_rows(Int8Mode mode, const Int8Args& a, int T, int cus);  // Int8Args::cap of T tokens, 0: codes
hipError_t launch_int8_stream(Int8Mode mode, const Int8Args& a, int cus, hipStream_t s);
// The tiled kernel (reads codes).  Grouped modes: `tile` sorted rows per token tile, token_tiles: at least their number.
hipError_t launch_int8_tile(Int8Mode mode, const Int8Args& a, int tile, long long token_tiles, int cus, hipStream_t s);
// Dense products of few tiles and a long K: K in this many runs (> 1), whose sums a second launch adds; 1: not this way.
int int8_splits(int M, int N, int K);
size_t int8_split_bytes(int max_M, int N, int K);  // of the sums for any M <= max_M
__host__ __device__ inline int int8_sums_ld(int N) { return (N + 3) / 4 * 4; }
int int8_tile_tokens(long long rows, int experts);  // sorted rows per tile of the grouped modes
constexpr int kInt8TileTokensMin = 64;
constexpr int kInt8TileGroup = 4;  // tiles of an expert that share a weight slab next to each other

}  // namespace moe
