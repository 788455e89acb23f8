// Exchanges between the lanes of one wave, without LDS: over rows of 16 lanes,
// or over all 64.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Two values as bf16, nearest even, by one instruction (converted one by one they take three).
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 b = __builtin_convertvector((f32x2{lo, hi}), bf16x2);
  uint32_t u;
  __builtin_memcpy(&u, &b, 4);
  return u;
}

// Between LDS accesses of one wave's lanes to each other's places.  The hardware does a wave's LDS operations in order;
// this keeps the compiler from moving or forwarding a lane's own accesses across.
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int N>
__device__ __forceinline__ uint32_t ror16(uint32_t v) {  // the value of lane l - N of the same row of 16, round
  return __builtin_amdgcn_update_dpp(0u, v, 0x120 + N, 0xF, 0xF, true);
}
template <int N>
__device__ __forceinline__ float ror16(float v) {
  return __uint_as_float(ror16<N>(__float_as_uint(v)));
}
template <int N>
__device__ __forceinline__ double ror16(double v) {
  return __hiloint2double((int)ror16<N>((uint32_t)__double2hiint(v)), (int)ror16<N>((uint32_t)__double2loint(v)));
}

// op over the 16 lanes of a row (L = 16) or all lanes (L = 64), the result in every lane.  Each step joins a lane's value
// with its counterpart's, so for a commutative op all lanes hold the same bits.
template <int L>
__device__ __forceinline__ uint32_t max_lanes(uint32_t v) {
  v = max(v, ror16<8>(v));
  v = max(v, ror16<4>(v));
  v = max(v, ror16<2>(v));
  v = max(v, ror16<1>(v));
  if constexpr (L == 64) {
    auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(a[0], a[1]);
    auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max(b[0], b[1]);
  }
  return v;
}
template <int L>
__device__ __forceinline__ float max_lanes(float v) {
  v = fmaxf(v, ror16<8>(v));
  v = fmaxf(v, ror16<4>(v));
  v = fmaxf(v, ror16<2>(v));
  v = fmaxf(v, ror16<1>(v));
  if constexpr (L == 64) {
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
  }
  return v;
}
template <int L>
__device__ __forceinline__ double sum_lanes(double v) {
  v += ror16<8>(v);
  v += ror16<4>(v);
  v += ror16<2>(v);
  v += ror16<1>(v);
  if constexpr (L == 64) {
    auto h = __builtin_amdgcn_permlane16_swap((uint32_t)__double2hiint(v), (uint32_t)__double2hiint(v), false, false);
    auto l = __builtin_amdgcn_permlane16_swap((uint32_t)__double2loint(v), (uint32_t)__double2loint(v), false, false);
    v = __hiloint2double((int)h[0], (int)l[0]) + __hiloint2double((int)h[1], (int)l[1]);
    h = __builtin_amdgcn_permlane32_swap((uint32_t)__double2hiint(v), (uint32_t)__double2hiint(v), false, false);
    l = __builtin_amdgcn_permlane32_swap((uint32_t)__double2loint(v), (uint32_t)__double2loint(v), false, false);
    v = __hiloint2double((int)h[0], (int)l[0]) + __hiloint2double((int)h[1], (int)l[1]);
  }
  return v;
}
template <int L>
__device__ __forceinline__ float sum_lanes(float v) {
  v += ror16<8>(v);
  v += ror16<4>(v);
  v += ror16<2>(v);
  v += ror16<1>(v);
  if constexpr (L == 64) {
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(b[0]) + __uint_as_float(b[1]);
  }
  return v;
}

}  // namespace moe
