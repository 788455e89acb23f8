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
// Both are bound by memory: every row is read once and written once (gradients of more
// than 10 rows or more than 8192 columns with a norm of the sum: twice), with stores
// that do not stay in the caches (non-temporal: forward 262 -> 242 us at 8192 x
// 7168, top-8).  A block takes a token, a thread 8 NC columns of it in registers, so
// that a row's norm needs one exchange over the block and no second read.
//
// Gradients: up to 10 rows of up to 8192 columns stay in registers from the sum to its
// gradient, a register that is done with takes a row of the next token, and PF rows of
// it have registers of their own, so that loads are in flight through every exchange.
// Beyond that there are no registers for them: rows are loaded one by one, with a norm
// of the sum twice.
// Nothing else may wait for vector loads in between: the norms' weights are in LDS,
// the rows' weights go through the scalar cache (as vector loads they cost 600 us
// against 493).  The norm weights' gradients are sums over tokens: a block adds those
// of its tokens (every grid-th) in LDS, where a thread has its own columns, a second
// launch adds the blocks' in order (the same bits every run); a single block stores
// them itself (one token of 7168, top-8: 11.5 us, with a second launch 16.6; two tokens
// by one block, 512 columns, 5.9 against 7.8, but 4096 columns 14.7 against 12.1).
// A token's rows cost a block of their own 6 us of arithmetic, two waves per SIMD: so
// the sums of all rows are exchanged together at the end and values converted in pairs
// (100 tokens of 7168 12.6 -> 11.7 us).
//
// Measured, with a gated shared expert and both norms: 8192 x 7168, top-8: forward
// 242 us (1.41 GB, 5.8 TB/s), gradients 489 + 5 us (2.58 GB, 5.3 TB/s; a large copy
// reaches 5.2); 8192 x 4096, top-6 without a shared expert: gradients 207 + 5 us.  Rows
// loaded one by one: 4096 x 4096, top-16 231 us without a norm of the sum (1.28 GB, 5.5
// TB/s) and 291 with it, 4096 x 12288, top-8 411 (2.2 GB, 5.4 TB/s) and 497.
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
  for (int i = 0; i < 4; ++i) o[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
  return o;
}
// 8 values at a row (the same for all lanes) and a column of this lane: a scalar base and 32 bits of offset.
__device__ __forceinline__ u32x4 load8(const uint16_t* row, uint32_t col) {
  return *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint8_t*>(row) + 2u * col);
}
__device__ __forceinline__ void store8(uint16_t* row, uint32_t col, const u32x4& v) {
  __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(reinterpret_cast<uint8_t*>(row) + 2u * col));
}

// A value that is the same for all lanes, through the scalar cache (it is an input that nothing in the launch writes).  As
// a vector load its wait would be one for every row in flight.
__device__ __forceinline__ float scalar(const float* p) {
  return *reinterpret_cast<const __attribute__((address_space(4))) float*>(reinterpret_cast<uintptr_t>(p));
}

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
__device__ __forceinline__ void add_rows(const NormArgs& a, size_t t, int j, const uint32_t (&col)[NC], float (&m)[NC][8]) {
  u32x4 v[N][NC];
  float w[N];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    w[u] = scalar(a.w + t * a.k + j + u);
#pragma unroll
    for (int i = 0; i < NC; ++i) v[u][i] = load8(a.y + (t * a.k + j + u) * a.H, col[i]);
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

// Columns of this thread: chunks of 8, a block's width apart; past the row's end the last chunk again (`live`: not).  Sums
// leave those out whole: with factors of zero an infinity in the last chunk would give them a NaN.
template <int NC>
__device__ __forceinline__ void columns(int H, uint32_t (&col)[NC], bool (&live)[NC]) {
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
  uint32_t col[NC];
  bool live[NC];
  columns<NC>(a.H, col, live);
  for (size_t t = blockIdx.x; t < (size_t)a.T; t += gridDim.x) {
  u32x4 sh[NC], rs[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (a.residual) rs[i] = load8(a.residual + t * a.H, col[i]);
    if (a.shared) sh[i] = load8(a.shared + t * a.H, col[i]);
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
    const float g = a.gate ? scalar(a.gate + t) : 1.f;
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
      for (int c = 0; c < 8; ++c) {
        const float v = live[i] ? m[i][c] : 0.f;
        s[0] = fmaf(v, v, s[0]);
      }
    block_sum<1>(s, part[n], waves);
    return 1.f / sqrtf(s[0] / (float)a.H + a.eps);
  };
  if (a.post) {
    const float q = mean_square(0);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float x[8];
      unpack(load8(a.post, col[i]), x);
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
    if (live[i]) store8(a.out + t * a.H, col[i], pack(m[i]));
  }
  if (a.next) {
    const float q = mean_square(1);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float x[8];
      unpack(load8(a.next, col[i]), x);
#pragma unroll
      for (int c = 0; c < 8; ++c) m[i][c] *= q * x[c];
      if (live[i]) store8(a.normed + t * a.H, col[i], pack(m[i]));
    }
  }
  __syncthreads();  // the sums are read before the next token's overwrite them
  }
}

// KR >= k: the token's rows stay in registers between the sum and its gradient, and as soon as a register is free the
// next token's row is on its way into it, so that loads are in flight through every sum over the block.  KR = 0 (more
// rows, or rows too long for that): rows are read again.
template <int NC, int KR, int PF>
__global__ __launch_bounds__(512) void combine_norm_backward_kernel(NormArgs a) {
  extern __shared__ __align__(16) float4 shared[];
  __shared__ float part[2][2 * 8];
  __shared__ float dots[2][8][36];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, waves = blockDim.x >> 6;
  const float rH = 1.f / (float)a.H;
  uint32_t col[NC];
  bool live[NC];
  columns<NC>(a.H, col, live);
  const int chunks = a.H / 8;
  float4* dpost = shared;  // [2][chunks]: the first and the second four of each chunk
  float4* dnext = shared + (a.post ? 2 * chunks : 0);
  // NC < 4: the norms' weights beside them (from memory, a wait for them would be one for all loads in flight)
  u32x4* gpost = reinterpret_cast<u32x4*>(dnext + (a.next ? 2 * chunks : 0));
  u32x4* gnext = gpost + (a.post ? chunks : 0);
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (live[i]) {
      if (a.post) dpost[col[i] >> 3] = dpost[chunks + (col[i] >> 3)] = zero;
      if (a.next) dnext[col[i] >> 3] = dnext[chunks + (col[i] >> 3)] = zero;
    }
  auto weight = [&](const uint16_t* w, const u32x4* held, int i) { return NC < 4 ? held[col[i] >> 3] : load8(w, col[i]); };
  auto add_to = [&](float4* to, int i, const float (&v)[8]) {
    if (!live[i]) return;
    float4 &lo = to[col[i] >> 3], &hi = to[chunks + (col[i] >> 3)];
    lo = make_float4(lo.x + v[0], lo.y + v[1], lo.z + v[2], lo.w + v[3]);
    hi = make_float4(hi.x + v[4], hi.y + v[5], hi.z + v[6], hi.w + v[7]);
  };

  u32x4 y[KR ? KR : 1][NC], z[PF ? PF : 1][NC], sh[NC], vo[NC], vd[NC], vn[NC];
  auto load_row = [&](u32x4 (&v)[NC], const uint16_t* row) {
#pragma unroll
    for (int i = 0; i < NC; ++i) v[i] = load8(row, col[i]);
  };
  auto load_first = [&](size_t t) {  // what the next norm's gradient reads
    if (a.d_out) load_row(vd, a.d_out + t * a.H);
    if (a.next) load_row(vo, a.out + t * a.H), load_row(vn, a.d_normed + t * a.H);
  };
  auto row_of = [&](size_t t, int j) { return a.y + (t * a.k + j) * a.H; };
  size_t t = blockIdx.x;
  u32x4 w1[NC], w2[NC];
  if constexpr (NC < 4) {
    if (a.post) load_row(w1, a.post);
    if (a.next) load_row(w2, a.next);
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) vd[i] = u32x4{0, 0, 0, 0};
  load_first(t);
  if constexpr (KR > 0) {
#pragma unroll
    for (int j = 0; j < KR; ++j) load_row(y[j], row_of(t, min(j, a.k - 1)));
  }
  if (a.shared) load_row(sh, a.shared + t * a.H);
  if constexpr (NC < 4) {  // every lane reads what it has written (a dead one the last chunk's values, the same ones)
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (a.post) gpost[col[i] >> 3] = w1[i];
      if (a.next) gnext[col[i] >> 3] = w2[i];
    }
  }

  for (int turn = 0;; turn ^= 1) {
    const size_t next = t + gridDim.x < (size_t)a.T ? t + gridDim.x : t;  // the last one again: loaded, not used
    const float gate = a.gate ? scalar(a.gate + t) : 1.f;
#pragma unroll
    for (int j = 0; j < PF; ++j) load_row(z[j], row_of(next, min(j, a.k - 1)));
    float d[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) unpack(vd[i], d[i]);
    if (a.next) {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float r[8], n[8], g[8];
        unpack(vo[i], r);
        unpack(vn[i], n);
        unpack(weight(a.next, gnext, i), g);
        float u0 = s[0], u1 = s[1];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          u0 = fmaf(r[c], r[c], u0);
          u1 = fmaf(n[c] * g[c], r[c], u1);
        }
        s[0] = live[i] ? u0 : s[0];
        s[1] = live[i] ? u1 : s[1];
      }
      block_sum<2>(s, part[0], waves);
      const float q = 1.f / sqrtf(s[0] * rH + a.eps), f = q * q * (s[1] * rH);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float r[8], n[8], g[8];
        unpack(vo[i], r);
        unpack(vn[i], n);
        unpack(weight(a.next, gnext, i), g);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          d[i][c] = fmaf(q, n[c] * g[c] - r[c] * f, d[i][c]);
          r[c] *= n[c] * q;
        }
        add_to(dnext, i, r);
      }
    }
    load_first(next);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (a.d_residual && live[i]) store8(a.d_residual + t * a.H, col[i], pack(d[i]));
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
          if (j < a.k) add(y[j], scalar(a.w + t * a.k + j));
      } else {
        for (int j = 0; j < a.k; ++j) add_rows<1, NC>(a, t, j, col, m);
      }
      if (a.shared) add(sh, gate);
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float g[8];
        unpack(weight(a.post, gpost, i), g);
        float u0 = s[0], u1 = s[1];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          u0 = fmaf(m[i][c], m[i][c], u0);
          u1 = fmaf(d[i][c] * g[c], m[i][c], u1);
        }
        s[0] = live[i] ? u0 : s[0];
        s[1] = live[i] ? u1 : s[1];
      }
      block_sum<2>(s, part[1], waves);
      const float q = 1.f / sqrtf(s[0] * rH + a.eps), f = q * q * (s[1] * rH);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float g[8], p[8];
        unpack(weight(a.post, gpost, i), g);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          p[c] = d[i][c] * m[i][c] * q;
          d[i][c] = q * (d[i][c] * g[c] - m[i][c] * f);
        }
        add_to(dpost, i, p);
      }
    }
    // this lane's part of the sum over the row
    auto row = [&](const u32x4 (&v)[NC], float w, uint16_t* to) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        float x[8], o[8];
        unpack(v[i], x);
        float u = s;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          u = fmaf(d[i][c], x[c], u);
          o[c] = w * d[i][c];
        }
        s = live[i] ? u : s;
        if (to && live[i]) store8(to, col[i], pack(o));
      }
      return s;
    };
    auto add_row = [&](int j, float s) {  // this wave's (slot k: the shared expert's)
      s = sum_lanes<64>(s);
      if (lane == 0) dots[turn][wv][j] = s;
    };
    if constexpr (KR > 0) {
      float s[KR];  // the exchanges of all rows together, so that none waits for another's
#pragma unroll
      for (int j = 0; j < KR; ++j) {
        s[j] = 0.f;
        if (j < a.k) s[j] = row(y[j], scalar(a.w + t * a.k + j), a.d_y ? a.d_y + (t * a.k + j) * a.H : nullptr);
        if (j >= PF) {
          load_row(y[j], row_of(next, min(j, a.k - 1)));
        } else {
#pragma unroll
          for (int i = 0; i < NC; ++i) y[j][i] = z[j][i];
        }
      }
#pragma unroll
      for (int j = 0; j < KR; ++j) add_row(j, s[j]);
    } else {
      for (int j = 0; j < a.k; ++j) {
        load_row(y[0], row_of(t, j));
        add_row(j, row(y[0], scalar(a.w + t * a.k + j), a.d_y ? a.d_y + (t * a.k + j) * a.H : nullptr));
      }
    }
    if (a.shared) {
      add_row(a.k, row(sh, gate, a.d_shared ? a.d_shared + t * a.H : nullptr));
      load_row(sh, a.shared + next * a.H);
    }
    __syncthreads();
    if (tid <= a.k && (tid < a.k || a.shared)) {
      float s = 0.f;
      for (int w = 0; w < waves; ++w) s += dots[turn][w][tid];
      if (tid == a.k) {
        if (a.d_gate) a.d_gate[t] = s;
      } else if (a.d_w) {
        a.d_w[t * a.k + tid] = s;
      }
    }
    if (t + gridDim.x >= (size_t)a.T) break;
    t = next;
  }
  float4* to = reinterpret_cast<float4*>(a.part + (size_t)blockIdx.x * 2 * a.H);
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (live[i]) {
      const int c = col[i] >> 3;
      if (gridDim.x == 1) {  // these are the sums (and the gradients aligned to 4 bytes only)
        auto put = [&](float* d, const float4& lo, const float4& hi) {
          d += col[i];
          d[0] = lo.x, d[1] = lo.y, d[2] = lo.z, d[3] = lo.w;
          d[4] = hi.x, d[5] = hi.y, d[6] = hi.z, d[7] = hi.w;
        };
        if (a.post) put(a.d_post, dpost[c], dpost[chunks + c]);
        if (a.next) put(a.d_next, dnext[c], dnext[chunks + c]);
        continue;
      }
      if (a.post) to[2 * c] = dpost[c], to[2 * c + 1] = dpost[chunks + c];
      if (a.next) to[a.H / 4 + 2 * c] = dnext[c], to[a.H / 4 + 2 * c + 1] = dnext[chunks + c];
    }
}

// The blocks' parts: C columns by a block, its 1024 / C rows of threads every so many-th part, then the rows' sums in
// order.
template <int C>
__global__ __launch_bounds__(1024) void norm_weights_kernel(NormArgs a, int blocks) {
  constexpr int R = 1024 / C;
  __shared__ float sum[R][C];
  const int at = threadIdx.x % C, row = threadIdx.x / C, per = (a.H + C - 1) / C;
  const int which = a.post && (int)blockIdx.x < per ? 0 : 1, c = ((int)blockIdx.x % per) * C + at;
  const float* p = a.part + (which ? a.H : 0) + min(c, a.H - 1);
  float s = 0.f;
#pragma unroll 8
  for (int b = row; b < blocks; b += R) s += p[(size_t)b * 2 * a.H];
  sum[row][at] = s;
  __syncthreads();
  if (row) return;
#pragma unroll 8
  for (int r = 1; r < R; ++r) s += sum[r][at];
  if (c < a.H) (which ? a.d_next : a.d_post)[c] = s;
}

template <int C>
void launch_weights(const NormArgs& a, int blocks, hipStream_t s) {
  const int grid = (a.H + C - 1) / C * ((a.post ? 1 : 0) + (a.next ? 1 : 0));
  norm_weights_kernel<C><<<dim3(grid), dim3(1024), 0, s>>>(a, blocks);
}

constexpr int kForwardBlocks = 1 << 20;  // a launch has fewer than 2^32 threads

int threads_of(int H, int nc) { return ((H / 8 + nc - 1) / nc + 63) / 64 * 64; }

template <int NC, int KR, int PF>
hipError_t launch_backward_rows(const NormArgs& a, int blocks, hipStream_t s) {
  // more dynamic LDS than the default limit, asked for on every call (a host-side attribute, the same number always)
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&combine_norm_backward_kernel<NC, KR, PF>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize,
                                           NC < 4 ? 2 * 8192 * 6 : 2 * 16384 * 4);
  if (e != hipSuccess) return e;
  const size_t lds = (size_t)((a.post ? 1 : 0) + (a.next ? 1 : 0)) * a.H * (NC < 4 ? 6 : 4);
  combine_norm_backward_kernel<NC, KR, PF><<<dim3((unsigned)blocks), dim3(threads_of(a.H, NC)), lds, s>>>(a);
  return hipGetLastError();
}
template <int NC>
hipError_t launch_backward(const NormArgs& a, int blocks, hipStream_t s) {
  if (a.k == 0 || a.k > 10) return launch_backward_rows<NC, 0, 0>(a, blocks, s);
  if (a.k <= 2) return launch_backward_rows<NC, 2, 1>(a, blocks, s);
  if (a.k <= 4) return launch_backward_rows<NC, 4, 2>(a, blocks, s);
  if (a.k <= 6) return launch_backward_rows<NC, 6, 3>(a, blocks, s);
  if (a.k <= 8) return launch_backward_rows<NC, 8, 4>(a, blocks, s);
  return launch_backward_rows<NC, 10, 3>(a, blocks, s);
}

}  // namespace

hipError_t launch_combine_norm(const NormArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.T < kForwardBlocks ? a.T : kForwardBlocks));
  if (a.H <= 2048) combine_norm_kernel<1><<<grid, dim3(threads_of(a.H, 1)), 0, s>>>(a);
  else combine_norm_kernel<2><<<grid, dim3(threads_of(a.H, 2)), 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_combine_norm_backward(const NormArgs& a, hipStream_t s) {
  const int blocks = norm_blocks(a.T, a.H);
  const hipError_t e = a.H > 8192  ? launch_backward_rows<4, 0, 0>(a, blocks, s)  // no registers for the rows
                       : a.H > 512 ? launch_backward<2>(a, blocks, s)
                                   : launch_backward<1>(a, blocks, s);
  if (e != hipSuccess || (!a.post && !a.next) || blocks == 1) return e;
  if (a.H <= 2048) launch_weights<16>(a, blocks, s);  // few columns and many parts: 1024 columns of 2048 parts 14 -> 7.4 us
  else launch_weights<64>(a, blocks, s);
  return hipGetLastError();
}

}  // namespace moe
