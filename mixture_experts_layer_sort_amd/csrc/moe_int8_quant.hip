// Quantisers of the 8-bit integer products, bound by memory: 8192 rows of 7168 28.7 us
// (176 MB, 6.1 TB/s; a large copy reaches 5.05 to 5.2), 33 rows of 4096 2.8 (a launch).
// Weights: 4096 x 7168 37 us (147 MB, 4.0 TB/s), 32 such 1167 (4.7 GB, 4.0 TB/s): a matrix is read twice.
#include "moe_int8.h"
#include "moe_tiles.h"

namespace moe {
namespace {

// Largest value of a wave, then of the block's waves (WPR waves per row: 1 or 4), in all of their threads.
template <int WPR>
__device__ __forceinline__ float row_max(float m, float* part) {
  m = max_rows(max_row16(m));
  if constexpr (WPR == 1) return m;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  return fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
}

// One block per weight row: its largest magnitude (not below 2^-100), scale = fp32(amax / 127), code =
// round(fp32(w fp32(127 / amax))).  A row with an infinity or a NaN: scale NaN, codes 0.  Load-time work, bound by memory.
__global__ __launch_bounds__(256) void int8_quantize_weights_kernel(int K, const float* w, int8_t* codes,
                                                                    float* scales) {
  __shared__ float part[4];
  __shared__ int bad[4];
  const float* src = w + (size_t)blockIdx.x * K;
  float m = kFp8Tiny;
  bool fine = true;
  for (int c = 4 * threadIdx.x; c < K; c += 1024) {
    const float4 v = *reinterpret_cast<const float4*>(src + c);
    const float a = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
    fine = fine && fabsf(v.x) < INFINITY && fabsf(v.y) < INFINITY && fabsf(v.z) < INFINITY && fabsf(v.w) < INFINITY;
    m = fmaxf(m, a);
  }
  const uint64_t all = __ballot(!fine);
  if ((threadIdx.x & 63) == 0) bad[threadIdx.x >> 6] = all != 0;
  m = row_max<4>(m, part);
  if (bad[0] | bad[1] | bad[2] | bad[3]) m = INFINITY;
  float f, s;
  int8_factor(m, f, s);
  for (int c = 4 * threadIdx.x; c < K; c += 1024) {
    const float4 v = *reinterpret_cast<const float4*>(src + c);
    *reinterpret_cast<uint32_t*>(codes + (size_t)blockIdx.x * K + c) = int8_codes4(v.x * f, v.y * f, v.z * f, v.w * f);
  }
  if (threadIdx.x == 0) scales[blockIdx.x] = s;
}

// Rows of x: a wave (WPR = 1, four rows per block) or a block (WPR = 4) per row, which stays in registers between its
// maximum and its codes up to kHeld chunks of 8 values per lane; longer rows are read again.  Bound by memory: 2 bytes in,
// 1 out per value.  The last block of a grouped launch writes the token tiles instead.
template <int WPR, int kHeld>
__global__ __launch_bounds__(256) void int8_quantize_rows_kernel(int M, int K, const uint16_t* x, long long ldx,
                                                                 int8_t* xq, float* xs, TileList list) {
  __shared__ float part[4];
  if (list.tiles && blockIdx.x == gridDim.x - 1) {
    write_tiles<kInt8TileGroup>(list);
    return;
  }
  const int Kp = int8_pad(K), at = WPR == 1 ? threadIdx.x & 63 : threadIdx.x;
  constexpr int kStep = 64 * WPR * 8;
  const long long row = WPR == 1 ? (long long)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  const uint16_t* src = x + min(row, (long long)M - 1) * ldx;
  const u32x4 none = {0, 0, 0, 0};
  u32x4 v[kHeld];
  uint32_t top = kFp8TinyBits;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int c = 8 * at + i * kStep;
    v[i] = c < K ? *reinterpret_cast<const u32x4*>(src + c) : none;
  }
#pragma unroll
  for (int i = 0; i < kHeld; ++i) top = fp8_amax8(v[i], top);
  for (int c = 8 * at + kHeld * kStep; c < K; c += kStep) top = fp8_amax8(*reinterpret_cast<const u32x4*>(src + c), top);
  float f, s;
  // on the bits: a NaN is larger than everything and stays
  const float m = bf16x2_max(top);
  const float worst = m == m && !(bf16_lo(top) != bf16_lo(top)) && !(bf16_hi(top) != bf16_hi(top)) ? m : INFINITY;
  int8_factor(row_max<WPR>(worst, part), f, s);
  if (row >= M) return;
  int8_t* dst = xq + row * Kp;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int c = 8 * at + i * kStep;
    if (c < Kp) *reinterpret_cast<uint2*>(dst + c) = int8_codes8(v[i], f);
  }
  for (int c = 8 * at + kHeld * kStep; c < Kp; c += kStep)
    *reinterpret_cast<uint2*>(dst + c) = c < K ? int8_codes8(*reinterpret_cast<const u32x4*>(src + c), f) : make_uint2(0, 0);
  if (at == 0) xs[row] = s;
}

hipError_t launch_rows(int M, int K, const uint16_t* x, long long ldx, int8_t* xq, float* xs, const TileList& list,
                       hipStream_t s) {
  const bool wave = M >= 1024 && K <= 64 * 8 * 16;
  const long long blocks = (wave ? ((long long)M + 3) / 4 : M) + (list.tiles ? 1 : 0);
  if (blocks >= 1LL << 24) return hipErrorInvalidValue;
  const dim3 grid((unsigned)blocks), block(256);
  if (wave) int8_quantize_rows_kernel<1, 16><<<grid, block, 0, s>>>(M, K, x, ldx, xq, xs, list);
  else if (K <= 256 * 8 * 2) int8_quantize_rows_kernel<4, 2><<<grid, block, 0, s>>>(M, K, x, ldx, xq, xs, list);
  else if (K <= 256 * 8 * 4) int8_quantize_rows_kernel<4, 4><<<grid, block, 0, s>>>(M, K, x, ldx, xq, xs, list);
  else int8_quantize_rows_kernel<4, 16><<<grid, block, 0, s>>>(M, K, x, ldx, xq, xs, list);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_quantize_rows(int M, int K, const uint16_t* x, long long ldx, int8_t* xq, float* xs,
                                     hipStream_t s) {
  return launch_rows(M, K, x, ldx, xq, xs, TileList{}, s);
}

hipError_t launch_int8_quantize_tokens(int T, int K, const uint16_t* x, int8_t* xq, float* xs, const int* offsets,
                                       int E, int tile, int4* tiles, int* ntiles, hipStream_t s) {
  return launch_rows(T, K, x, K, xq, xs, TileList{offsets, E, tile, tiles, ntiles}, s);
}

hipError_t launch_int8_quantize_weights(int count, int rows, int K, const float* w, int8_t* codes, float* scales,
                                        hipStream_t s) {
  int8_quantize_weights_kernel<<<dim3((unsigned)((size_t)count * rows)), dim3(256), 0, s>>>(K, w, codes, scales);
  return hipGetLastError();
}

}  // namespace moe
