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
// Forward.  A block takes a chunk of consecutive tokens and, for each sequence
// that the chunk meets, adds the probabilities of its tokens in registers (a lane
// owns the same experts for every token), counts picks in LDS and writes one
// record.  Chunk c and sequence s meet along a staircase, so slot c + s names the
// record without a list.  Then the records of a sequence are added in chunk
// order, in 64 bits: in a second launch by blocks of (sequence, 32 experts), of
// which the last to finish adds their parts of the loss in a fixed order; or, for
// small batches, in the same block with the records in LDS.  No floating-point
// atomics: the same bits every run.
//
// Four tokens at once per wave: reductions of four rows share their steps
// (reduce4: 7 exchanges, where each row alone takes 6), so that the vector units,
// which bounded one row at a time, keep up with the reads.  65536 tokens, 256
// experts: forward 34 -> 24 us in one sequence (67 MB, 2.8 TB/s), 26.5 in 16;
// gradient 43 -> 36 us (141 MB, 3.9 TB/s).  A large copy reaches 5.2 TB/s.  Made for up to some tens of sequences: the
// second launch has a block per sequence and 32 experts, and its last one adds their parts in one wave (65536 x 256 in
// 1000 sequences 343 us, in 10000 3.6 ms; the gradient 33 and 46).
#include "moe_balance.h"

#include "moe_fp8.h"  // wave reductions

namespace moe {
namespace {

// Between LDS accesses of one wave's lanes to each other's places.  The hardware does a wave's LDS operations in order;
// this keeps the compiler from moving or forwarding a lane's own accesses across.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

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

// Four rows at once: v := exp(v - max); the rows' sums and log-sum-exps are in the rows of `sum` and `lse` that of_row
// reads.  The difference comes first: logits up to the type's largest and lowest values stay finite.
template <int VEC, int NC>
__device__ __forceinline__ void softmax_rows(float (&v)[4][NC][VEC], float& sum, float& lse) {
  constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
  float m[4], s[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    m[u] = v[u][0][0];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) m[u] = fmaxf(m[u], v[u][i][j]);
  }
  const float top = reduce4(m, [](float a, float b) { return fmaxf(a, b); });
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float mu = of_row(top, u);
    s[u] = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        v[u][i][j] = __builtin_amdgcn_exp2f((v[u][i][j] - mu) * kLog2e);
        s[u] += v[u][i][j];
      }
  }
  sum = reduce4(s, [](float a, float b) { return a + b; });
  lse = fmaf(__builtin_amdgcn_logf(sum), kLn2, top);  // v_log_f32: base 2
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

// Sums over the tokens [t, t + 4), [t + step, t + step + 4), .. below hi: probabilities of the lane's experts, squared
// log-sum-exps, valid tokens.
template <int VEC, int NC>
__device__ __forceinline__ void add_tokens(const BalanceArgs& a, int t, int hi, int step, float (&acc)[NC][VEC],
                                           float& z, int& n, int lane) {
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc[i][j] = 0.f;
  z = 0.f;
  n = 0;
  for (; t < hi; t += step) {
    float v[4][NC][VEC], keep[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int tu = min(t + u, hi - 1);
      keep[u] = t + u < hi && (!a.mask || a.mask[tu]) ? 1.f : 0.f;
      load_row<VEC, NC>(v[u], a.logits + (size_t)tu * a.E, a.E, lane, -INFINITY);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (keep[u] == 0.f) {  // whatever the row holds
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int j = 0; j < VEC; ++j) v[u][i][j] = 0.f;
      }
    float sum, lse;
    softmax_rows<VEC, NC>(v, sum, lse);
    const float inv = __builtin_amdgcn_rcpf(sum), sq = lse * lse;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float f = of_row(inv, u) * keep[u];
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[i][j] = fmaf(v[u][i][j], f, acc[i][j]);
      z = fmaf(of_row(sq, u), keep[u], z);
      n += keep[u] != 0.f;
    }
  }
}

// Adds the picks of the tokens [lo, hi) to the counters; thread `at` of `num`.
__device__ __forceinline__ void add_picks(const BalanceArgs& a, int lo, int hi, int* counters, int at, int num) {
  for (int p = at; p < (hi - lo) * a.k; p += num) {
    const int id = a.ids[(size_t)lo * a.k + p];
    if ((!a.mask || a.mask[lo + p / a.k]) && (unsigned)id < (unsigned)a.E) atomicAdd(&counters[id], 1);
  }
}

// Calls f(s, lo, hi) for each sequence s of which tokens [lo, hi) lie in [t0, t1).
template <class F>
__device__ __forceinline__ void each_sequence(const BalanceArgs& a, int t0, int t1, F&& f) {
  int s = t0 < t1 ? max(0, seq_of(a, t0)) : a.S;
  for (; s < a.S; ++s) {
    const int first = seq_bound(a, s), lo = max(t0, first), hi = min(t1, seq_bound(a, s + 1));
    if (first >= t1) break;
    if (lo < hi) f(s, lo, hi);
  }
}

// Records of a chunk of tokens: prob / count [slot][E], zn [slot], slot = chunk + sequence.
template <int VEC, int NC>
__global__ __launch_bounds__(64 * kBalanceWaves) void balance_chunk_kernel(BalanceArgs a, int chunk, float* prob,
                                                                           int* count, float2* zn, unsigned* ticket) {
  constexpr int W = kBalanceWaves;
  extern __shared__ __align__(16) uint8_t shared[];
  int* counters = reinterpret_cast<int*>(shared);        // [E]
  float* lp = reinterpret_cast<float*>(counters + a.E);  // [W][E]
  float* lz = lp + W * a.E;                              // [W][2]
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (blockIdx.x == 0 && tid == 0) *ticket = 0;
  const int t0 = min(a.T, (int)blockIdx.x * chunk);
  each_sequence(a, t0, min(a.T, t0 + chunk), [&](int s, int lo, int hi) {
    for (int e = tid; e < a.E; e += 64 * W) counters[e] = 0;
    __syncthreads();
    add_picks(a, lo, hi, counters, tid, 64 * W);
    float acc[NC][VEC], z;
    int n;
    add_tokens<VEC, NC>(a, lo + 4 * wv, hi, 4 * W, acc, z, n, lane);
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int e = (64 * i + lane) * VEC + j;
        if (e < a.E) lp[wv * a.E + e] = acc[i][j];
      }
    if (lane == 0) lz[2 * wv] = z, lz[2 * wv + 1] = (float)n;  // at most 2^24 tokens in all: exact
    __syncthreads();
    const size_t slot = (size_t)blockIdx.x + s;
    for (int e = tid; e < a.E; e += 64 * W) {
      float p = lp[e];
#pragma unroll
      for (int w = 1; w < W; ++w) p += lp[w * a.E + e];
      prob[slot * a.E + e] = p;
      count[slot * a.E + e] = counters[e];
    }
    if (tid == 0) {
      float sz = 0.f, sn = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) sz += lz[2 * w], sn += lz[2 * w + 1];
      zn[slot] = make_float2(sz, sn);
    }
    __syncthreads();
  });
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
  const int e = sl * kBalanceSlice + ex;
  const int c0 = lo / chunk, c1 = hi > lo ? (hi - 1) / chunk + 1 : c0;
  double p = 0.0, z = 0.0, n = 0.0;
  int c = 0;
  if (e < a.E) {
#pragma unroll 4
    for (int i = c0 + row; i < c1; i += 32) {
      const size_t at = (size_t)(i + s) * a.E + e;
      p += prob[at];
      c += count[at];
    }
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
    a.loss[1] = a.z_coef == 0.f ? 0.f : (float)(a.z_coef / a.S * z);  // the sum itself may be infinite
  }
}

// Small batches in one block of 16 waves: records in LDS, then a wave per (sequence, 64 experts).
template <int VEC, int NC>
__global__ __launch_bounds__(1024) void balance_small_kernel(BalanceArgs a, int chunk) {
  extern __shared__ __align__(16) uint8_t lds[];
  const int slots = 16 + a.S, slices = (a.E + 63) / 64;
  double* part = reinterpret_cast<double*>(lds);                            // [S][slices + 1]
  float2* zn = reinterpret_cast<float2*>(part + a.S * (slices + 1));        // [slots]
  float* prob = reinterpret_cast<float*>(zn + slots);                       // [slots][E]
  int* count = reinterpret_cast<int*>(prob + (size_t)slots * a.E);          // [slots][E]
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t0 = min(a.T, wv * chunk);
  each_sequence(a, t0, min(a.T, t0 + chunk), [&](int s, int lo, int hi) {
    const int slot = wv + s;
    for (int e = lane; e < a.E; e += 64) count[slot * a.E + e] = 0;  // slots of one wave: no barrier
    wave_sync();
    add_picks(a, lo, hi, count + slot * a.E, lane, 64);
    float acc[NC][VEC], z;
    int n;
    add_tokens<VEC, NC>(a, lo, hi, 4, acc, z, n, lane);
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int e = (64 * i + lane) * VEC + j;
        if (e < a.E) prob[slot * a.E + e] = acc[i][j];
      }
    if (lane == 0) zn[slot] = make_float2(z, (float)n);
  });
  __syncthreads();
  for (int task = wv; task < a.S * slices; task += 16) {
    const int s = task / slices, sl = task % slices, e = sl * 64 + lane;
    const int lo = seq_bound(a, s), hi = seq_bound(a, s + 1);
    const int c0 = lo / chunk, c1 = hi > lo ? (hi - 1) / chunk + 1 : c0;
    double p = 0.0, z = 0.0, n = 0.0;
    int c = 0;
    for (int i = c0; i < c1; ++i) {
      if (e < a.E) {
        p += prob[(i + s) * a.E + e];
        c += count[(i + s) * a.E + e];
      }
      z += zn[i + s].x;
      n += zn[i + s].y;
    }
    if (e < a.E) a.counts[(size_t)s * a.E + e] = c;
    const double d = n > 0.0 ? n : 1.0;
    const double dot = sum_wave_f64(p * c) * a.E / ((double)a.k * d * d);
    if (lane == 0) {
      part[s * (slices + 1) + sl] = dot;
      if (sl == 0) {
        part[s * (slices + 1) + slices] = z / d;
        a.tokens[s] = (int)n;
      }
    }
  }
  __syncthreads();
  if (wv == 0) {
    double b = 0.0, z = 0.0;
    for (int i = lane; i < a.S * (slices + 1); i += 64) {
      if (i % (slices + 1) == slices) z += part[i];
      else b += part[i];
    }
    b = sum_wave_f64(b);
    z = sum_wave_f64(z);
    if (lane == 0) {
      a.loss[0] = (float)(a.coef / a.S * b);
      a.loss[1] = a.z_coef == 0.f ? 0.f : (float)(a.z_coef / a.S * z);  // the sum itself may be infinite
    }
  }
}

// d logits of one token per wave step:
//   p_e (A_e - sum p A) + Z lse p_e + [e = id_j] w_j (dw_j - sum_i w_i dw_i),
//   A_e = g0 coef / (S k n^2) (E c_e - k n)   (k n, the mean of E c_e, does not change the gradient: subtracted, the
//   difference A_e - sum p A keeps its digits), Z = 2 g1 z_coef / (S n).
template <int VEC, int NC>
__global__ __launch_bounds__(256) void route_backward_kernel(BalanceArgs a, int per_wave) {
  __shared__ float lds[4 * 4 * 64 * NC * VEC];  // 4 rows of each wave
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w = blockIdx.x * 4 + wv, t0 = w * per_wave, t1 = min(a.T, t0 + per_wave);
  if (t0 >= t1) return;
  constexpr int kRow = 64 * NC * VEC;
  float* rows = lds + wv * 4 * kRow;
  const float g0 = a.d_loss ? a.d_loss[0] * a.coef : 0.f, g1 = a.d_loss ? a.d_loss[1] * a.z_coef : 0.f;
  int s = -2, end = t0;  // sequence of the current token; its end
  bool in = false;       // the token is in a sequence: the losses have a part (never without d_loss)
  float A[NC][VEC], Z = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) A[i][j] = 0.f;
  // four tokens at once, all of one sequence
  for (int tb = t0; tb < t1;) {
    if (a.d_loss && tb >= end) {
      s = seq_of(a, tb);
      in = s >= 0 && s < a.S;
      end = in ? seq_bound(a, s + 1) : s < 0 ? seq_bound(a, 0) : a.T;
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
    const int te = a.d_loss ? min(t1, end) : t1, num = min(4, te - tb);
    float v[4][NC][VEC], keep[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int t = min(tb + u, te - 1);
      keep[u] = !a.mask || a.mask[t] ? 1.f : 0.f;
      if (a.d_loss) load_row<VEC, NC>(v[u], a.logits + (size_t)t * a.E, a.E, lane, -INFINITY);
    }
    // picks: row r of 16 lanes has those of token row4(r), 16 at a time
    int id[2] = {-1, -1};
    float wt[2] = {0.f, 0.f}, dw[2] = {0.f, 0.f};
    const int mine = row4(lane >> 4);
    const bool live = mine < num && (!a.mask || a.mask[min(tb + mine, te - 1)]);
    if (a.d_topk_w) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = 16 * h + (lane & 15);
        if (live && j < a.k) {
          const size_t at = (size_t)(tb + mine) * a.k + j;
          id[h] = a.ids[at];
          wt[h] = a.topk_w[at];
          dw[h] = a.d_topk_w[at];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (!in || keep[u] == 0.f) {  // whatever the row holds
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int j = 0; j < VEC; ++j) v[u][i][j] = 0.f;
      }
    if (a.d_loss) {
      float sum, lse, dot[4];
      softmax_rows<VEC, NC>(v, sum, lse);
      const float inv = __builtin_amdgcn_rcpf(sum);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float f = of_row(inv, u) * keep[u];
        dot[u] = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            v[u][i][j] *= f;
            dot[u] = fmaf(v[u][i][j], A[i][j], dot[u]);
          }
      }
      const float sub = fmaf(Z, lse, -reduce4(dot, [](float x, float y) { return x + y; }));
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float su = of_row(sub, u);
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int j = 0; j < VEC; ++j) v[u][i][j] *= A[i][j] + su;
      }
    }
    if (a.d_topk_w) {
      // the picks' parts are added to the rows in LDS: one wave's adds, in lane order
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int j = 0; j < VEC; ++j) rows[u * kRow + (64 * i + lane) * VEC + j] = v[u][i][j];
      wave_sync();
      float x = wt[0] * dw[0] + wt[1] * dw[1];
      x += row_ror<8>(x);
      x += row_ror<4>(x);
      x += row_ror<2>(x);
      x += row_ror<1>(x);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if ((unsigned)id[h] < (unsigned)a.E) atomicAdd(&rows[mine * kRow + id[h]], wt[h] * (dw[h] - x));
      wave_sync();
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int j = 0; j < VEC; ++j) v[u][i][j] = rows[u * kRow + (64 * i + lane) * VEC + j];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (u >= num) break;
      float* o = a.d_logits + (size_t)(tb + u) * a.E;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int e = (64 * i + lane) * VEC;
        if (e < a.E) {
          if constexpr (VEC == 4)
            *reinterpret_cast<float4*>(o + e) = make_float4(v[u][i][0], v[u][i][1], v[u][i][2], v[u][i][3]);
          else o[e] = v[u][i][0];
        }
      }
    }
    tb += num;
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

// One block does it all while its 16 waves have two batches of four tokens at most, and their records fit LDS (40 tokens
// of 24 sequences, 64 experts: 8.5 us against 15.4; 500 tokens: 15.1 against 11.0).
constexpr int kSmallLds = 128 * 1024;
size_t small_lds(const BalanceArgs& a) {
  const size_t slots = 16 + a.S, slices = (a.E + 63) / 64;
  return a.S * (slices + 1) * 8 + slots * 8 + slots * a.E * 8;
}

hipError_t launch_balance_loss(const BalanceArgs& a, uint8_t* ws, hipStream_t s) {
  const bool vec = a.E % 4 == 0 && a.E > 128 && aligned16(a.logits);
  if (a.T <= 128 && small_lds(a) <= kSmallLds) {
    const int bytes = (int)small_lds(a), chunk = (a.T + 15) / 16;
    return dispatch(a, vec, [&](auto v, auto n) {
      const hipError_t e = hipFuncSetAttribute(
          reinterpret_cast<const void*>(&balance_small_kernel<decltype(v)::value, decltype(n)::value>),
          hipFuncAttributeMaxDynamicSharedMemorySize, kSmallLds);
      if (e != hipSuccess) return e;
      balance_small_kernel<decltype(v)::value, decltype(n)::value><<<dim3(1), dim3(1024), bytes, s>>>(a, chunk);
      return hipGetLastError();
    });
  }
  const BalanceWorkspace w = balance_workspace(a.T, a.E, a.S);
  const int chunk = balance_chunk(a.T), chunks = balance_chunks(a.T);
  float* prob = reinterpret_cast<float*>(ws + w.prob);
  int* count = reinterpret_cast<int*>(ws + w.count);
  float2* zn = reinterpret_cast<float2*>(ws + w.zn);
  double* part = reinterpret_cast<double*>(ws + w.part);
  unsigned* ticket = reinterpret_cast<unsigned*>(ws + w.ticket);
  hipError_t e = dispatch(a, vec, [&](auto v, auto n) {
    balance_chunk_kernel<decltype(v)::value, decltype(n)::value>
        <<<dim3(chunks), dim3(64 * kBalanceWaves),
           ((kBalanceWaves + 1) * a.E + 2 * kBalanceWaves) * sizeof(float), s>>>(a, chunk, prob, count, zn, ticket);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  balance_reduce_kernel<<<dim3(a.S * balance_slices(a.E)), dim3(1024), 0, s>>>(a, chunk, prob, count, zn, part, ticket);
  return hipGetLastError();
}

hipError_t launch_route_backward(const BalanceArgs& a, int cus, hipStream_t s) {
  // Consecutive tokens per wave: one while that is at most 8 waves per CU (500 tokens, 64 experts: 4.0 us, at four
  // 5.3), else four at once (8192 tokens, 256 experts: 7.8 us, at one 10.2), more where that still leaves 32 waves per
  // CU, up to 16, to share a sequence's factors (65536 tokens: 36 us at eight, 41 at 16).
  const long long waves = 32LL * cus;
  int per = (int)((a.T + waves - 1) / waves);
  per = a.T <= 8 * cus ? 1 : per < 4 ? 4 : per > 16 ? 16 : per;
  const int blocks = (a.T + 4 * per - 1) / (4 * per);
  const bool vec = a.E % 4 == 0 && a.E > 128 && aligned16(a.logits) && aligned16(a.d_logits);
  return dispatch(a, vec, [&](auto v, auto n) {
    route_backward_kernel<decltype(v)::value, decltype(n)::value><<<dim3(blocks), dim3(256), 0, s>>>(a, per);
    return hipGetLastError();
  });
}

}  // namespace moe
