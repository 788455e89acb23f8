// Balance loss, router z-loss and per-expert counts of a batch of sequences,
// and the gradient of the router's logits.
//
//   p_t = softmax(logits_t), lse_t = log sum exp(logits_t)
//   per sequence s with n_s valid tokens and c_{s,e} picks of expert e:
//     f_{s,e} = E c_{s,e} / (k n_s),  P_{s,e} = mean_t p_{t,e}
//   loss[0] = coef / S sum_s sum_e f_{s,e} P_{s,e},  loss[1] = z_coef / S sum_s mean_t lse_t^2
//
// Both passes read the logits once (4 T E bytes) and are bound by that read
// (and the gradient's write).
//
// Forward, two launches.  (1) A block takes a chunk of consecutive tokens and,
// for each sequence that the chunk meets, adds the probabilities of its tokens
// in registers (a lane owns the same experts for every token), counts picks in
// LDS and writes one partial record.  Chunk c and sequence s meet along a
// staircase, so slot c + s names the record without a list.  (2) Blocks of
// (sequence, 32 experts) add the sequence's records in chunk order, in 64 bits;
// the last block to finish adds the blocks' parts of the loss in a fixed order.
// No floating-point atomics: the same bits every run.
#include "moe_balance.h"

#include "moe_fp8.h"  // wave reductions

namespace moe {
namespace {

// Row values of one lane: v[i][j] = row[(64 i + lane) VEC + j], `fill` past E.
template <int VEC, int NC>
__device__ __forceinline__ void load_row(float (&v)[NC][VEC], const float* row, int E, int lane, float fill) {
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int e = (64 * i + lane) * VEC;
    if constexpr (VEC == 4) {
      float4 x = make_float4(fill, fill, fill, fill);
      if (e < E) x = *reinterpret_cast<const float4*>(row + e);  // E % 4 == 0
      v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
    } else {
      v[i][0] = e < E ? row[e] : fill;
    }
  }
}

// v := exp(v - max); returns 1 / sum and the log-sum-exp.
template <int VEC, int NC>
__device__ __forceinline__ float softmax_row(float (&v)[NC][VEC], float& lse) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) m = fmaxf(m, v[i][j]);
  m = max_wave(m);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      v[i][j] = __expf(v[i][j] - m);
      s += v[i][j];
    }
  s = sum_wave(s);
  lse = m + logf(s);
  return 1.f / s;
}

__device__ __forceinline__ int seq_bound(const BalanceArgs& a, int s) {  // first token of sequence s
  if (!a.seq) return s == 0 ? 0 : a.T;
  return min(max(a.seq[s], 0), a.T);
}

// The last sequence that begins at or before token t (-1: none; S: t is behind the last one).
__device__ __forceinline__ int seq_of(const BalanceArgs& a, int t) {
  int lo = 0, hi = a.S + 1;  // first s in [0, S] that begins after t (S: the end of the last; S + 1: none)
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (seq_bound(a, mid) > t) hi = mid;
    else lo = mid + 1;
  }
  return lo - 1;
}

template <int VEC, int NC>
__global__ __launch_bounds__(256) void balance_chunk_kernel(BalanceArgs a, int chunk, float* prob, int* count,
                                                            float2* zn, unsigned* ticket) {
  extern __shared__ float lds[];  // [4][E] probabilities of the waves, [E] counts, [4] z, [4] tokens
  float* lp = lds;
  int* lc = reinterpret_cast<int*>(lds + 4 * a.E);
  float* lz = lds + 5 * a.E;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  if (blockIdx.x == 0 && tid == 0) *ticket = 0;
  const int t0 = blockIdx.x * chunk, t1 = min(a.T, t0 + chunk);
  int s = max(0, seq_of(a, t0));
  for (; s < a.S; ++s) {
    const int lo = max(t0, seq_bound(a, s)), hi = min(t1, seq_bound(a, s + 1));
    if (seq_bound(a, s) >= t1) break;
    if (lo >= hi) continue;
    for (int e = tid; e < a.E; e += 256) lc[e] = 0;
    float acc[NC][VEC];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[i][j] = 0.f;
    float z = 0.f;
    int n = 0;
    __syncthreads();
    // picks: all (token, slot) pairs of this part
    for (int p = tid; p < (hi - lo) * a.k; p += 256) {
      const int t = lo + p / a.k;
      const int id = a.ids[(size_t)lo * a.k + p];
      if ((!a.mask || a.mask[t]) && (unsigned)id < (unsigned)a.E) atomicAdd(&lc[id], 1);
    }
    constexpr int U = NC * VEC <= 4 ? 4 : 2;  // tokens in flight per wave
    for (int t = lo + wv; t < hi; t += 4 * U) {
      float v[U][NC][VEC];
      bool ok[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int tu = t + 4 * u;
        ok[u] = tu < hi && (!a.mask || a.mask[tu]);
        if (ok[u]) load_row<VEC, NC>(v[u], a.logits + (size_t)tu * a.E, a.E, lane, -INFINITY);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (ok[u]) {
          float lse;
          const float inv = softmax_row<VEC, NC>(v[u], lse);
#pragma unroll
          for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) acc[i][j] += v[u][i][j] * inv;
          z += lse * lse;
          ++n;
        }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int e = (64 * i + lane) * VEC + j;
        if (e < a.E) lp[wv * a.E + e] = acc[i][j];
      }
    if (lane == 0) {
      lz[wv] = z;
      lz[4 + wv] = (float)n;  // at most 2^24 tokens in all: exact
    }
    __syncthreads();
    const size_t slot = (size_t)blockIdx.x + s;
    for (int e = tid; e < a.E; e += 256) {
      prob[slot * a.E + e] = lp[e] + lp[a.E + e] + lp[2 * a.E + e] + lp[3 * a.E + e];
      count[slot * a.E + e] = lc[e];
    }
    if (tid == 0) zn[slot] = make_float2(lz[0] + lz[1] + lz[2] + lz[3], lz[4] + lz[5] + lz[6] + lz[7]);
    __syncthreads();
  }
}

__device__ __forceinline__ double sum_wave_f64(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// Block (sequence s, slice of 32 experts): 16 waves, each half wave adds the
// records of every 32nd chunk of the sequence.
__global__ __launch_bounds__(1024) void balance_reduce_kernel(BalanceArgs a, int chunk, const float* prob,
                                                              const int* count, const float2* zn, double* part,
                                                              unsigned* ticket) {
  __shared__ double lp[32][kBalanceSlice];
  __shared__ int lc[32][kBalanceSlice];
  __shared__ double lz[16][2];
  __shared__ bool last;
  const int slices = gridDim.x / a.S, s = blockIdx.x / slices, sl = blockIdx.x % slices;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, row = tid >> 5, ex = tid & 31;
  const int lo = seq_bound(a, s), hi = seq_bound(a, s + 1);
  const int c0 = lo / chunk, c1 = hi > lo ? (hi - 1) / chunk + 1 : c0;
  const int e = sl * kBalanceSlice + ex;
  double p = 0.0, z = 0.0, n = 0.0;
  int c = 0;
  if (e < a.E)
    for (int i = c0 + row; i < c1; i += 32) {
      const size_t at = (size_t)(i + s) * a.E + e;
      p += prob[at];
      c += count[at];
    }
  for (int i = c0 + tid; i < c1; i += 1024) {
    const float2 r = zn[i + s];
    z += r.x;
    n += r.y;
  }
  lp[row][ex] = p;
  lc[row][ex] = c;
  z = sum_wave_f64(z);
  n = sum_wave_f64(n);
  if (lane == 0) lz[wv][0] = z, lz[wv][1] = n;
  __syncthreads();
  if (wv == 0) {
    z = n = 0.0;
    for (int i = 0; i < 16; ++i) z += lz[i][0], n += lz[i][1];
    p = 0.0;
    c = 0;
    if (lane < kBalanceSlice) {
      for (int i = 0; i < 32; ++i) p += lp[i][lane], c += lc[i][lane];
      if (e < a.E) a.counts[(size_t)s * a.E + e] = c;
    }
    const double d = n > 0.0 ? n : 1.0;
    const double dot = sum_wave_f64(lane < kBalanceSlice ? p * c : 0.0) * a.E / ((double)a.k * d * d);
    if (lane == 0) {
      part[(size_t)s * (slices + 1) + sl] = dot;
      if (sl == 0) {
        part[(size_t)s * (slices + 1) + slices] = z / d;
        a.tokens[s] = (int)n;
      }
      __threadfence();
      last = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!last || wv != 0) return;
  __threadfence();
  double b = 0.0;
  z = 0.0;
  for (int i = lane; i < a.S * (slices + 1); i += 64) {
    const double v = __hip_atomic_load(part + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (i % (slices + 1) == slices) z += v;
    else b += v;
  }
  b = sum_wave_f64(b);
  z = sum_wave_f64(z);
  if (lane == 0) {
    a.loss[0] = (float)(a.coef / a.S * b);
    a.loss[1] = (float)(a.z_coef / a.S * z);
  }
}

// d logits of one token per wave step:
//   p_e (A_e - sum p A) + Z lse p_e + [e = id_j] w_j (dw_j - sum_i w_i dw_i),
//   A_e = g0 coef / (S k n^2) (E c_e - k n)   (k n, the mean of E c_e, does not change the gradient: subtracted, the
//   difference A_e - sum p A keeps its digits), Z = 2 g1 z_coef / (S n).
template <int VEC, int NC>
__global__ __launch_bounds__(256) void route_backward_kernel(BalanceArgs a, int per_wave) {
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const int t0 = w * per_wave, t1 = min(a.T, t0 + per_wave);
  if (t0 >= t1) return;
  const float g0 = a.d_loss ? a.d_loss[0] * a.coef : 0.f, g1 = a.d_loss ? a.d_loss[1] * a.z_coef : 0.f;
  int s = -2, end = t0;  // sequence of the current token; its end
  float A[NC][VEC], Z = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) A[i][j] = 0.f;
  for (int t = t0; t < t1; ++t) {
    float v[NC][VEC];
    const bool ok = !a.mask || a.mask[t];
    if (ok) load_row<VEC, NC>(v, a.logits + (size_t)t * a.E, a.E, lane, -INFINITY);
    if (a.d_loss && (s == -2 || t >= end)) {
      s = seq_of(a, t);
      end = s + 1 <= a.S ? seq_bound(a, s + 1) : a.T;
      const bool in = s >= 0 && s < a.S;
      if (!in) end = s < 0 ? seq_bound(a, 0) : a.T;
      const float n = in ? (float)max(1, a.tokens[s]) : 1.f;
      const float sc = g0 / ((float)a.S * (float)a.k * n * n);
      const long long mean = in ? (long long)a.k * a.tokens[s] : 0;  // whole numbers: the difference is exact
      Z = in ? 2.f * g1 / ((float)a.S * n) : 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const int e = (64 * i + lane) * VEC + j;
          A[i][j] = in && e < a.E ? sc * (float)((long long)a.E * a.counts[(size_t)s * a.E + e] - mean) : 0.f;
        }
    }
    float d[NC][VEC];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) d[i][j] = 0.f;
    if (ok) {
      if (a.d_loss) {
        float lse;
        const float inv = softmax_row<VEC, NC>(v, lse);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            v[i][j] *= inv;
            dot += v[i][j] * A[i][j];
          }
        const float sub = Z * lse - sum_wave(dot);
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int j = 0; j < VEC; ++j) d[i][j] = v[i][j] * (A[i][j] + sub);
      }
      if (a.d_topk_w) {
        int id = -1;
        float wt = 0.f, dw = 0.f;
        if (lane < a.k) {
          id = a.ids[(size_t)t * a.k + lane];
          wt = a.topk_w[(size_t)t * a.k + lane];
          dw = a.d_topk_w[(size_t)t * a.k + lane];
        }
        const float val = wt * (dw - sum_wave(wt * dw));
        for (int j = 0; j < a.k; ++j) {
          const int idj = __builtin_amdgcn_readlane(id, j);
          const float vj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(val), j));
#pragma unroll
          for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int jj = 0; jj < VEC; ++jj) d[i][jj] += (64 * i + lane) * VEC + jj == idj ? vj : 0.f;
        }
      }
    }
    float* o = a.d_logits + (size_t)t * a.E;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int e = (64 * i + lane) * VEC;
      if (e < a.E) {
        if constexpr (VEC == 4) *reinterpret_cast<float4*>(o + e) = make_float4(d[i][0], d[i][1], d[i][2], d[i][3]);
        else o[e] = d[i][0];
      }
    }
  }
}

// Four consecutive experts per lane where rows allow 16-byte accesses and fill
// the wave's lanes at least by half; else one.
template <class F>
hipError_t dispatch(const BalanceArgs& a, bool vec, F&& f) {
  auto c = [](auto v) { return v; };
  using std::integral_constant;
  if (vec) {
    if (a.E <= 256) return f(c(integral_constant<int, 4>{}), c(integral_constant<int, 1>{}));
    if (a.E <= 512) return f(c(integral_constant<int, 4>{}), c(integral_constant<int, 2>{}));
    return f(c(integral_constant<int, 4>{}), c(integral_constant<int, 4>{}));
  }
  if (a.E <= 64) return f(c(integral_constant<int, 1>{}), c(integral_constant<int, 1>{}));
  if (a.E <= 128) return f(c(integral_constant<int, 1>{}), c(integral_constant<int, 2>{}));
  if (a.E <= 256) return f(c(integral_constant<int, 1>{}), c(integral_constant<int, 4>{}));
  if (a.E <= 512) return f(c(integral_constant<int, 1>{}), c(integral_constant<int, 8>{}));
  return f(c(integral_constant<int, 1>{}), c(integral_constant<int, 16>{}));
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace

hipError_t launch_balance_loss(const BalanceArgs& a, uint8_t* ws, hipStream_t s) {
  const BalanceWorkspace w = balance_workspace(a.T, a.E, a.S);
  const int chunk = balance_chunk(a.T), chunks = balance_chunks(a.T);
  float* prob = reinterpret_cast<float*>(ws + w.prob);
  int* count = reinterpret_cast<int*>(ws + w.count);
  float2* zn = reinterpret_cast<float2*>(ws + w.zn);
  double* part = reinterpret_cast<double*>(ws + w.part);
  unsigned* ticket = reinterpret_cast<unsigned*>(ws + w.ticket);
  const bool vec = a.E % 4 == 0 && a.E > 128 && aligned16(a.logits);
  hipError_t e = dispatch(a, vec, [&](auto v, auto n) {
    balance_chunk_kernel<decltype(v)::value, decltype(n)::value>
        <<<dim3(chunks), dim3(256), (5 * a.E + 8) * sizeof(float), s>>>(a, chunk, prob, count, zn, ticket);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  balance_reduce_kernel<<<dim3(a.S * balance_slices(a.E)), dim3(1024), 0, s>>>(a, chunk, prob, count, zn, part, ticket);
  return hipGetLastError();
}

hipError_t launch_route_backward(const BalanceArgs& a, int cus, hipStream_t s) {
  // consecutive tokens per wave: enough waves to fill the GPU first, then up to 16 to share a sequence's factors
  const long long waves = 32LL * cus;
  int per = (int)((a.T + waves - 1) / waves);
  per = per < 1 ? 1 : per > 16 ? 16 : per;
  const int blocks = (a.T + 4 * per - 1) / (4 * per);
  const bool vec = a.E % 4 == 0 && a.E > 128 && aligned16(a.logits) && aligned16(a.d_logits);
  return dispatch(a, vec, [&](auto v, auto n) {
    route_backward_kernel<decltype(v)::value, decltype(n)::value><<<dim3(blocks), dim3(256), 0, s>>>(a, per);
    return hipGetLastError();
  });
}

}  // namespace moe
