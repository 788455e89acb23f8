// Quantisers of the block-128 fp8 products.
#include "moe_fp8.h"
#include "moe_tiles.h"

namespace moe {
namespace {

// One block per 128 x 128 weight block: its largest magnitude (not below
// 2^-100), scale = fp32(amax / 448), code = e4m3(fp32(w * fp32(448 / amax))).
// Load-time work, bound by memory: 4096 x 7168 in 38 us, 32 of them in 1180 (3.9 TB/s of 4 bytes in and 1 out; a large
// copy reaches 5.2; the second pass over a block reads the caches).
__global__ __launch_bounds__(256) void fp8_quantize_weights_kernel(int rows, int K, const float* w, uint8_t* codes,
                                                                   float* scales) {
  __shared__ float part[4];
  const int NB = (rows + kFp8Blk - 1) / kFp8Blk, KB = (K + kFp8Blk - 1) / kFp8Blk;
  const int kb = blockIdx.x % KB, nb = blockIdx.x / KB % NB;
  const size_t c = blockIdx.x / ((size_t)KB * NB);
  const int tid = threadIdx.x, col = kb * kFp8Blk + 4 * (tid & 31), row0 = nb * kFp8Blk + (tid >> 5);
  const int nrow = min(kFp8Blk, rows - nb * kFp8Blk);
  const float* src = w + (c * rows + row0) * K + col;  // K % 16 == 0: columns come in fours
  float m = kFp8Tiny;
  if (col < K)
    for (int r = tid >> 5; r < nrow; r += 8) {
      const float4 v = *reinterpret_cast<const float4*>(src + (size_t)(r - (tid >> 5)) * K);
      m = fmaxf(fmaxf(m, fmaxf(fabsf(v.x), fabsf(v.y))), fmaxf(fabsf(v.z), fabsf(v.w)));
    }
  for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
  if ((tid & 63) == 0) part[tid >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  const float f = kFp8Max / m;
  if (col < K)
    for (int r = tid >> 5; r < nrow; r += 8) {
      const float4 v = *reinterpret_cast<const float4*>(src + (size_t)(r - (tid >> 5)) * K);
      *reinterpret_cast<uint32_t*>(codes + (c * rows + nb * kFp8Blk + r) * K + col) =
          fp8_codes4(v.x * f, v.y * f, v.z * f, v.w * f);
    }
  if (tid == 0) scales[blockIdx.x] = m / kFp8Max;
}

// Rows of x quantised per 128 columns.  A block takes ROWS (64, or 8 where few rows
// would leave most of the GPU idle) rows x 512 columns: a
// wave one row of them at a time (16 lanes per 128-column block, 16 bytes
// each), ROWS / 4 rows in turn; the 4 x ROWS scales go out through LDS as runs
// (scales are stored column-block-major, so a tile's tokens read them in one
// piece).  Bound by memory: 2 bytes in, 1 out per value.  The last block of a
// grouped launch writes the token tiles instead.
constexpr int kQCols = 512;

template <int kQRows>
__global__ __launch_bounds__(256) void fp8_quantize_rows_kernel(int M, int K, const uint16_t* x, long long ldx,
                                                                uint8_t* xq, float* xs, TileList list) {
  __shared__ float sc[4][kQRows];
  const int KB = (K + kFp8Blk - 1) / kFp8Blk, Kp = KB * kFp8Blk, CB = (Kp + kQCols - 1) / kQCols;
  if (list.tiles && blockIdx.x == gridDim.x - 1) {
    write_tiles<kFp8TileGroup>(list);
    return;
  }
  const int cb = blockIdx.x % CB, m0 = blockIdx.x / CB * kQRows;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int col = cb * kQCols + 8 * lane;
  constexpr int kPer = kQRows / 4, U = kPer < 8 ? kPer : 8;
  const u32x4 none = {0, 0, 0, 0};
  for (int i0 = 0; i0 < kPer; i0 += U) {
    u32x4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int m = min(m0 + wv * kPer + i0 + u, M - 1);
      v[u] = col < K ? *reinterpret_cast<const u32x4*>(x + (size_t)m * ldx + col) : none;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = wv * kPer + i0 + u;
      float f, s;
      fp8_factor(max_row16(bf16x2_max(fp8_amax8(v[u], kFp8TinyBits))), f, s);
      const uint2 c = fp8_codes8(v[u], f);
      if ((lane & 15) == 0) sc[lane >> 4][row] = s;
      if (m0 + row < M && col < Kp) *reinterpret_cast<uint2*>(xq + (size_t)(m0 + row) * Kp + col) = c;
    }
  }
  __syncthreads();
  const int b = cb * 4 + wv;
  if (b < KB && lane < kQRows && m0 + lane < M) xs[(size_t)b * M + m0 + lane] = sc[wv][lane];
}

hipError_t launch_rows(int M, int K, const uint16_t* x, long long ldx, uint8_t* xq, float* xs, const TileList& list,
                       hipStream_t s) {
  const long long KB = (K + kFp8Blk - 1) / kFp8Blk, CB = (KB * kFp8Blk + kQCols - 1) / kQCols;
  const int rows = M <= 1024 ? 8 : 64;
  const long long blocks = (M + rows - 1) / rows * CB + (list.tiles ? 1 : 0);
  if (rows == 8) fp8_quantize_rows_kernel<8><<<dim3((unsigned)blocks), dim3(256), 0, s>>>(M, K, x, ldx, xq, xs, list);
  else fp8_quantize_rows_kernel<64><<<dim3((unsigned)blocks), dim3(256), 0, s>>>(M, K, x, ldx, xq, xs, list);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_quantize_rows(int M, int K, const uint16_t* x, long long ldx, uint8_t* xq, float* xs,
                                    hipStream_t s) {
  return launch_rows(M, K, x, ldx, xq, xs, TileList{}, s);
}

hipError_t launch_fp8_quantize_tokens(int T, int K, const uint16_t* x, uint8_t* xq, float* xs, const int* offsets,
                                      int E, int tile, int4* tiles, int* ntiles, hipStream_t s) {
  return launch_rows(T, K, x, K, xq, xs, TileList{offsets, E, tile, tiles, ntiles}, s);
}

hipError_t launch_fp8_quantize_weights(int count, int rows, int K, const float* w, uint8_t* codes, float* scales,
                                       hipStream_t s) {
  const size_t blocks = (size_t)count * ((rows + kFp8Blk - 1) / kFp8Blk) * ((K + kFp8Blk - 1) / kFp8Blk);
  fp8_quantize_weights_kernel<<<dim3((unsigned)blocks), dim3(256), 0, s>>>(rows, K, w, codes, scales);
  return hipGetLastError();
}

}  // namespace moe
