// The end of an expert block, and its gradients.  For every token, in fp32:
//
//   m = sum_j w_j y_j + gate shared
//   n = post ? m q1 post : m,           q1 = 1 / sqrt(mean m^2 + eps)
//   r = residual + scale n
//   normed = r q2 next,                 q2 = 1 / sqrt(mean r^2 + eps)
//
// Backwards (out = r as it was stored; <.> is the mean over the row):
//
//   a = d_normed next,  d_next = sum_t d_normed r q2
//   d = d_out + q2 (a - r q2^2 <a r>),  d_residual = d
//   b = scale d,  d_post = sum_t b m q1,  c = b post
//   dm = post ? q1 (c - m q1^2 <c m>) : b
//   d_y_j = w_j dm,  d_w_j = sum dm y_j,  d_shared = gate dm,  d_gate = sum dm shared
//
// Both are bound by memory: every row is read once and written once.  A block
// takes a token, a thread 8 NC consecutive-by-8 columns of it in registers, so
// that a row's norm needs one exchange over the block and no second read.  The
// weights' gradients are sums over tokens: a block adds those of its tokens (every
// grid-th) in registers, a second launch adds the blocks' in order (the same bits
// every run).
#include "moe_norm.h"

#include "moe_device.h"
#include "moe_fp8.h"  // u32x4, bf16_lo, bf16_hi
#include "moe_wave.h"

namespace moe {
namespace {

__device__ __forceinline__ void unpack(const u32x4& v, float (&o)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) o[2 * i] = bf16_lo(v[i]), o[2 * i + 1] = bf16_hi(v[i]);
}
__device__ __forceinline__ u32x4 pack(const float (&v)[8]) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = f32_to_bf16(v[2 * i]) | (uint32_t)f32_to_bf16(v[2 * i + 1]) << 16;
  return o;
}
__device__ __forceinline__ u32x4 load8(const uint16_t* p) { return *reinterpret_cast<const u32x4*>(p); }
__device__ __forceinline__ void store8(uint16_t* p, const u32x4& v) { *reinterpret_cast<u32x4*>(p) = v; }

// Sums over the block of N values of each thread, in every thread; `part`: [16][N], free again after the next barrier
// of the block.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* part, int waves) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = sum_lanes<64>(v[i]);
  if (waves == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) part[wv * N + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  for (int w = 0; w < waves; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += part[w * N + i];
}

// m += rows j .. j + N - 1 of the token, in slot order.
template <int N, int NC>
__device__ __forceinline__ void add_rows(const NormArgs& a, size_t t, int j, const int (&col)[NC], float (&m)[NC][8]) {
  u32x4 v[N][NC];
  float w[N];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    w[u] = a.w[t * a.k + j + u];
#pragma unroll
    for (int i = 0; i < NC; ++i) v[u][i] = load8(a.y + (t * a.k + j + u) * a.H + col[i]);
  }
#pragma unroll
  for (int u = 0; u < N; ++u)
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float x[8];
      unpack(v[u][i], x);
#pragma unroll
      for (int c = 0; c < 8; ++c) m[i][c] = fmaf(w[u], x[c], m[i][c]);
    }
}

// Columns of this thread: chunks of 8, a block's width apart; past the row's end the last chunk again (`live`: not).
template <int NC>
__device__ __forceinline__ void columns(int H, int (&col)[NC], bool (&live)[NC]) {
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = 8 * (threadIdx.x + i * blockDim.x);
    live[i] = c < H;
    col[i] = live[i] ? c : H - 8;
  }
}

template <int NC>
__global__ __launch_bounds__(1024) void combine_norm_kernel(NormArgs a) {
  __shared__ float part[2][16];
  const int waves = blockDim.x >> 6;
  int col[NC];
  bool live[NC];
  columns<NC>(a.H, col, live);
  for (size_t t = blockIdx.x; t < (size_t)a.T; t += gridDim.x) {
  u32x4 sh[NC], rs[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (a.residual) rs[i] = load8(a.residual + t * a.H + col[i]);
    if (a.shared) sh[i] = load8(a.shared + t * a.H + col[i]);
  }
  float m[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int c = 0; c < 8; ++c) m[i][c] = 0.f;
  int j = 0;
  for (; j + 4 <= a.k; j += 4) add_rows<4, NC>(a, t, j, col, m);
  if (a.k & 2) add_rows<2, NC>(a, t, j, col, m), j += 2;
  if (a.k & 1) add_rows<1, NC>(a, t, j, col, m);
  if (a.shared) {
    const float g = a.gate ? a.gate[t] : 1.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float x[8];
      unpack(sh[i], x);
#pragma unroll
      for (int c = 0; c < 8; ++c) m[i][c] = fmaf(g, x[c], m[i][c]);
    }
  }
  auto mean_square = [&](int n) {
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int c = 0; c < 8; ++c) s[0] += live[i] ? m[i][c] * m[i][c] : 0.f;
    block_sum<1>(s, part[n], waves);
    return 1.f / sqrtf(s[0] / (float)a.H + a.eps);
  };
  if (a.post) {
    const float q = mean_square(0);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float x[8];
      unpack(load8(a.post + col[i]), x);
#pragma unroll
      for (int c = 0; c < 8; ++c) m[i][c] *= q * x[c];
    }
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (a.residual) unpack(rs[i], x);
#pragma unroll
    for (int c = 0; c < 8; ++c) m[i][c] = fmaf(a.scale, m[i][c], x[c]);
    if (live[i]) store8(a.out + t * a.H + col[i], pack(m[i]));
  }
  if (a.next) {
    const float q = mean_square(1);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float x[8];
      unpack(load8(a.next + col[i]), x);
#pragma unroll
      for (int c = 0; c < 8; ++c) m[i][c] *= q * x[c];
      if (live[i]) store8(a.normed + t * a.H + col[i], pack(m[i]));
    }
  }
  __syncthreads();  // the sums are read before the next token's overwrite them
  }
}

// KR >= k: the token's rows stay in registers between the sum and its gradient; KR = 0: they are read again.
template <int NC, int KR>
__global__ __launch_bounds__(1024) void combine_norm_backward_kernel(NormArgs a) {
  __shared__ float part[2][2 * 16];
  __shared__ float dots[16][36];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, waves = blockDim.x >> 6;
  const float rH = 1.f / (float)a.H;
  int col[NC];
  bool live[NC];
  columns<NC>(a.H, col, live);
  float dpost[NC][8], dnext[NC][8];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int c = 0; c < 8; ++c) dpost[i][c] = dnext[i][c] = 0.f;

  for (size_t t = blockIdx.x; t < (size_t)a.T; t += gridDim.x) {
    u32x4 y[KR ? KR : 1][NC], sh[NC];
    float d[NC][8];
    // everything that the token needs is on its way before the first sum
    u32x4 vo[NC], vd[NC], vn[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const size_t at = t * a.H + col[i];
      vd[i] = u32x4{0, 0, 0, 0};
      if (a.d_out) vd[i] = load8(a.d_out + at);
      if (a.next) vo[i] = load8(a.out + at), vn[i] = load8(a.d_normed + at);
      if (a.shared) sh[i] = load8(a.shared + at);
    }
    if constexpr (KR > 0) {
#pragma unroll
      for (int j = 0; j < KR; ++j)
#pragma unroll
        for (int i = 0; i < NC; ++i) y[j][i] = load8(a.y + (t * a.k + min(j, a.k - 1)) * a.H + col[i]);
    }
    const float gate = a.gate ? a.gate[t] : 1.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) unpack(vd[i], d[i]);
    if (a.next) {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float r[8], n[8], g[8];
        unpack(vo[i], r);
        unpack(vn[i], n);
        unpack(load8(a.next + col[i]), g);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          s[0] += live[i] ? r[c] * r[c] : 0.f;
          s[1] += live[i] ? n[c] * g[c] * r[c] : 0.f;
        }
      }
      block_sum<2>(s, part[0], waves);
      const float q = 1.f / sqrtf(s[0] * rH + a.eps), f = q * q * (s[1] * rH);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float r[8], n[8], g[8];
        unpack(vo[i], r);
        unpack(vn[i], n);
        unpack(load8(a.next + col[i]), g);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          dnext[i][c] = fmaf(n[c], r[c] * q, dnext[i][c]);
          d[i][c] = fmaf(q, n[c] * g[c] - r[c] * f, d[i][c]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (a.d_residual && live[i]) store8(a.d_residual + t * a.H + col[i], pack(d[i]));
#pragma unroll
      for (int c = 0; c < 8; ++c) d[i][c] *= a.scale;
    }
    if (a.post) {
      float m[NC][8];
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) m[i][c] = 0.f;
      auto add = [&](const u32x4 (&v)[NC], float w) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          float x[8];
          unpack(v[i], x);
#pragma unroll
          for (int c = 0; c < 8; ++c) m[i][c] = fmaf(w, x[c], m[i][c]);
        }
      };
      if constexpr (KR > 0) {
#pragma unroll
        for (int j = 0; j < KR; ++j)
          if (j < a.k) add(y[j], a.w[t * a.k + j]);
      } else {
        for (int j = 0; j < a.k; ++j) add_rows<1, NC>(a, t, j, col, m);
      }
      if (a.shared) add(sh, gate);
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float g[8];
        unpack(load8(a.post + col[i]), g);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          s[0] += live[i] ? m[i][c] * m[i][c] : 0.f;
          s[1] += live[i] ? d[i][c] * g[c] * m[i][c] : 0.f;
        }
      }
      block_sum<2>(s, part[1], waves);
      const float q = 1.f / sqrtf(s[0] * rH + a.eps), f = q * q * (s[1] * rH);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float g[8];
        unpack(load8(a.post + col[i]), g);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          dpost[i][c] = fmaf(d[i][c], m[i][c] * q, dpost[i][c]);
          d[i][c] = q * (d[i][c] * g[c] - m[i][c] * f);
        }
      }
    }
    // this wave's parts of the sums over the row (slot k: the shared expert's)
    auto row = [&](const u32x4 (&v)[NC], int j, float w, uint16_t* to) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float x[8], o[8];
        unpack(v[i], x);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          s += live[i] ? d[i][c] * x[c] : 0.f;
          o[c] = w * d[i][c];
        }
        if (to && live[i]) store8(to + col[i], pack(o));
      }
      s = sum_lanes<64>(s);
      if (lane == 0) dots[wv][j] = s;
    };
    if constexpr (KR > 0) {
#pragma unroll
      for (int j = 0; j < KR; ++j)
        if (j < a.k) row(y[j], j, a.w[t * a.k + j], a.d_y ? a.d_y + (t * a.k + j) * a.H : nullptr);
    } else {
      for (int j = 0; j < a.k; ++j) {
        u32x4 v[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) v[i] = load8(a.y + (t * a.k + j) * a.H + col[i]);
        row(v, j, a.w[t * a.k + j], a.d_y ? a.d_y + (t * a.k + j) * a.H : nullptr);
      }
    }
    if (a.shared) row(sh, a.k, gate, a.d_shared ? a.d_shared + t * a.H : nullptr);
    __syncthreads();
    if (tid <= a.k && (tid < a.k || a.shared)) {
      float s = 0.f;
      for (int w = 0; w < waves; ++w) s += dots[w][tid];
      if (tid == a.k) {
        if (a.d_gate) a.d_gate[t] = s;
      } else if (a.d_w) {
        a.d_w[t * a.k + tid] = s;
      }
    }
    __syncthreads();
  }
  float* to = a.part + (size_t)blockIdx.x * 2 * a.H;
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (live[i]) {
      if (a.post) {
#pragma unroll
        for (int c = 0; c < 8; c += 4)
          *reinterpret_cast<float4*>(to + col[i] + c) = make_float4(dpost[i][c], dpost[i][c + 1], dpost[i][c + 2], dpost[i][c + 3]);
      }
      if (a.next) {
#pragma unroll
        for (int c = 0; c < 8; c += 4)
          *reinterpret_cast<float4*>(to + a.H + col[i] + c) =
              make_float4(dnext[i][c], dnext[i][c + 1], dnext[i][c + 2], dnext[i][c + 3]);
      }
    }
}

// The blocks' parts: 64 columns by a block, its 16 waves every 16th part, then the waves' sums in order.
__global__ __launch_bounds__(1024) void norm_weights_kernel(NormArgs a, int blocks) {
  __shared__ float sum[16][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, per = (a.H + 63) / 64;
  const int which = a.post && (int)blockIdx.x < per ? 0 : 1, c = ((int)blockIdx.x % per) * 64 + lane;
  const float* p = a.part + (which ? a.H : 0) + min(c, a.H - 1);
  float s = 0.f;
#pragma unroll 4
  for (int b = wv; b < blocks; b += 16) s += p[(size_t)b * 2 * a.H];
  sum[wv][lane] = s;
  __syncthreads();
  if (wv) return;
  for (int w = 1; w < 16; ++w) s += sum[w][lane];
  if (c < a.H) (which ? a.d_next : a.d_post)[c] = s;
}

constexpr int kForwardBlocks = 1 << 20;  // a launch has fewer than 2^32 threads

int threads_of(int H, int nc) { return ((H / 8 + nc - 1) / nc + 63) / 64 * 64; }

template <int NC>
void launch_backward(const NormArgs& a, int blocks, hipStream_t s) {
  const dim3 grid((unsigned)blocks), block(threads_of(a.H, NC));
  if (a.k == 0 || a.k > 8) combine_norm_backward_kernel<NC, 0><<<grid, block, 0, s>>>(a);
  else if (a.k <= 2) combine_norm_backward_kernel<NC, 2><<<grid, block, 0, s>>>(a);
  else if (a.k <= 4) combine_norm_backward_kernel<NC, 4><<<grid, block, 0, s>>>(a);
  else if (a.k <= 6) combine_norm_backward_kernel<NC, 6><<<grid, block, 0, s>>>(a);
  else combine_norm_backward_kernel<NC, 8><<<grid, block, 0, s>>>(a);
}

}  // namespace

hipError_t launch_combine_norm(const NormArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.T < kForwardBlocks ? a.T : kForwardBlocks));
  if (a.H <= 2048) combine_norm_kernel<1><<<grid, dim3(threads_of(a.H, 1)), 0, s>>>(a);
  else combine_norm_kernel<2><<<grid, dim3(threads_of(a.H, 2)), 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_combine_norm_backward(const NormArgs& a, hipStream_t s) {
  const int blocks = a.T < kNormBlocks ? a.T : kNormBlocks;
  if (a.H <= 2048) launch_backward<1>(a, blocks, s);
  else launch_backward<2>(a, blocks, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!a.post && !a.next)) return e;
  const int per = (a.H + 63) / 64;
  norm_weights_kernel<<<dim3(per * ((a.post ? 1 : 0) + (a.next ? 1 : 0))), dim3(1024), 0, s>>>(a, blocks);
  return hipGetLastError();
}

}  // namespace moe
