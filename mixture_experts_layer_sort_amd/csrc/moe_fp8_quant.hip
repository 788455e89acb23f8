// Quantisers of the block-128 fp8 products.
#include "moe_fp8.h"

namespace moe {
namespace {

// One block per 128 x 128 weight block: its largest magnitude (not below
// 2^-100), scale = fp32(amax / 448), code = e4m3(fp32(w * fp32(448 / amax))).
// Load-time work, bound by reading the fp32 masters.
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

}  // namespace

hipError_t launch_fp8_quantize_weights(int count, int rows, int K, const float* w, uint8_t* codes, float* scales,
                                       hipStream_t s) {
  const size_t blocks = (size_t)count * ((rows + kFp8Blk - 1) / kFp8Blk) * ((K + kFp8Blk - 1) / kFp8Blk);
  fp8_quantize_weights_kernel<<<dim3((unsigned)blocks), dim3(256), 0, s>>>(rows, K, w, codes, scales);
  return hipGetLastError();
}

}  // namespace moe
