// Scored routing: experts of a token by softmax or sigmoid scores, a choice
// bias, groups, renormalised weights; and the gradient of the logits.
//
//   s_e = sigmoid(l_e) or softmax(l)_e,   c_e = fp32(fp32(s_e) + b_e), -inf where l_e is
//   group score: its largest c, or fp32(largest + second); KG groups are kept
//   picks: the k largest c of the kept groups (equal ones: the lower id first)
//   w_j = scale s_j / (sum_i s_i or 1)
//
// Which of two experts is picked can hang on the last bit of a score, so scores
// are computed in 64 bits (relative error below 1e-14) and rounded once to the
// 32 bits that the definition names: picks are the same whatever computes them.
//
// A token has L lanes, a lane V consecutive experts, so that positions order
// like ids and equal choices need no ids to be compared: a round takes the
// maximum of the lanes' maxima, and the first lane that has it takes its first
// expert that has it.  L = 16 (four tokens per wave share every exchange) where
// there are tokens enough to fill the GPU, L = 64 for few tokens or many experts.
#include "moe_router.h"

#include "moe_wave.h"

namespace moe {
namespace {

constexpr int kWaves = 4;
constexpr int kMaxK = 32;
constexpr uint32_t kOff = 0x007FFFFFu;  // key of -inf: still before 0, an expert that cannot be picked

// exp(x) for x <= 709.78, to 1e-14: 2^n times the Taylor sum of the rest, |rest| <= ln 2 / 2 (12th term: 6e-15).
__device__ __forceinline__ double exp64(double x) {
  if (x < -745.0) return 0.0;  // NaN goes on
  const double n = rint(x * 1.4426950408889634074);
  const double f = fma(n, -1.9082149292705877e-10, fma(n, -0.69314718036912381649, x));  // ln 2 in two parts
  double p = 1.0 / 39916800.0;
  p = fma(p, f, 1.0 / 3628800.0);
  p = fma(p, f, 1.0 / 362880.0);
  p = fma(p, f, 1.0 / 40320.0);
  p = fma(p, f, 1.0 / 5040.0);
  p = fma(p, f, 1.0 / 720.0);
  p = fma(p, f, 1.0 / 120.0);
  p = fma(p, f, 1.0 / 24.0);
  p = fma(p, f, 1.0 / 6.0);
  p = fma(p, f, 0.5);
  p = fma(p, f, 1.0);
  p = fma(p, f, 1.0);
  return ldexp(p, (int)n);
}

// 1 / d, d a normal number: the hardware's estimate and two Newton steps.
__device__ __forceinline__ double rcp64(double d) {
  double r = __builtin_amdgcn_rcp(d);
  r = fma(fma(-d, r, 1.0), r, r);
  return fma(fma(-d, r, 1.0), r, r);
}

// Keys in LDS: a word is left out after every 32, so that groups of 32 begin in different banks.
__host__ __device__ constexpr int key_at(int e) { return e + (e >> 5); }

// 0 below -709, where exp(-l) ends.
__device__ __forceinline__ double sigmoid64(float l) {
  if (l < -709.f) return 0.0;
  return rcp64(1.0 + exp64(-(double)l));
}

// Order of fp32 values as unsigned numbers (-0 is 0); NaN is with -inf.
__device__ __forceinline__ uint32_t order_key(float c) {
  const uint32_t b = __float_as_uint(c + 0.f);
  const uint32_t k = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return c == c ? k : kOff;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

template <int L, int V, bool SOFTMAX, bool VEC>
__global__ __launch_bounds__(64 * kWaves) void route_scores_kernel(RouterArgs a) {
  constexpr int TW = 64 / L;  // tokens of a wave
  extern __shared__ __align__(16) uint32_t shared[];  // groups: keys [wave][TW][key_words], scores [wave][TW][G]
  __shared__ int picks[kWaves][TW][kMaxK];
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int sub = lane & (L - 1), slot = lane / L;
  const long long t = ((long long)blockIdx.x * kWaves + wv) * TW + slot;
  const float* row = a.logits + min(t, (long long)a.T - 1) * a.ldl;
  const int e0 = sub * V;

  float l[V];
#pragma unroll
  for (int i = 0; i < V; ++i) l[i] = -INFINITY;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      if (e0 + i < a.E) {
        const float4 v = *reinterpret_cast<const float4*>(row + e0 + i);
        l[i] = v.x, l[i + 1] = v.y, l[i + 2] = v.z, l[i + 3] = v.w;
      }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i < a.E) l[i] = row[e0 + i];
  }

  double top = 0.0, inv = 1.0;  // softmax: largest logit, 1 / sum
  uint32_t key[V];
  if constexpr (SOFTMAX) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
    m = max_lanes<L>(m);
    top = m == -INFINITY ? 0.0 : (double)m;  // every expert is off: all scores are 0
    double ex[V], sum = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += ex[i] = exp64((double)l[i] - top);
    sum = sum_lanes<L>(sum);
    inv = sum == 0.0 ? 0.0 : rcp64(sum);
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = __float_as_uint((float)(ex[i] * inv));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = __float_as_uint((float)sigmoid64(l[i]));
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = e0 + i;
    const float b = a.bias ? a.bias[min(e, a.E - 1)] : 0.f;
    const uint32_t k = l[i] == -INFINITY ? kOff : order_key(__uint_as_float(key[i]) + b);
    key[i] = e < a.E ? k : 0u;
  }

  if (a.KG < a.G) {  // experts of groups that are not kept: 0
    const int per = a.E / a.G;
    const int words = key_at(a.E);
    uint32_t* keys = shared + (wv * TW + slot) * words;
    uint32_t* score = shared + kWaves * TW * words + (wv * TW + slot) * a.G;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i < a.E) keys[key_at(e0 + i)] = key[i];
    wave_lds_sync();
    for (int g = sub; g < a.G; g += L) {
      uint32_t b1 = 0, b2 = 0;
      for (int i = 0; i < per; ++i) {
        const uint32_t k = keys[key_at(g * per + i)];
        b2 = max(b2, min(b1, k));
        b1 = max(b1, k);
      }
      score[g] = a.top == 1 ? b1 : order_key(of_key(b1) + of_key(b2));
    }
    wave_lds_sync();
    for (int g = sub; g < a.G; g += L) {
      const uint32_t mine = score[g];
      int before = 0;
      for (int h = 0; h < a.G; ++h) {
        const uint32_t other = score[h];
        before += other > mine || (other == mine && h < g);
      }
      if (before >= a.KG)
        for (int i = 0; i < per; ++i) keys[key_at(g * per + i)] = 0u;
    }
    wave_lds_sync();
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = e0 + i < a.E ? keys[key_at(e0 + i)] : 0u;
  }

  for (int j = 0; j < a.k; ++j) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = max(m, key[i]);
    const uint32_t best = max_lanes<L>(m);
    const uint64_t same = __ballot(m == best);
    int first;
    if constexpr (L == 64) first = __ffsll((unsigned long long)same) - 1;
    else first = __ffs((uint32_t)(same >> (lane & 48)) & 0xFFFFu) - 1;
    int at = 0;
    bool open = sub == first;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool hit = open && key[i] == best;
      at = hit ? i : at;
      key[i] = hit ? 0u : key[i];
      open = open && !hit;
    }
    if (sub == first) picks[wv][slot][j] = e0 + at;
  }
  wave_lds_sync();

  const bool mine = sub < a.k;
  const int id = mine ? picks[wv][slot][sub] : 0;
  double s = 0.0;
  if (mine) {
    const float z = row[id];
    s = SOFTMAX ? exp64((double)z - top) * inv : sigmoid64(z);
  }
  if (a.renorm) {
    const double sum = sum_lanes<L>(s);
    s = sum == 0.0 ? 0.0 : s / sum;
  }
  if (mine && t < a.T) {
    a.ids[t * a.k + sub] = id;
    a.w[t * a.k + sub] = (float)((double)a.scale * s);
  }
}

// Gradient.  L lanes per token; lane j has pick j and its part of the gradient in 64 bits; the parts meet the row's
// other values in LDS, where a lane has the experts 4 (l + L i) .. + 3 (or l + L i), so that rows are stored in one run.
// Only softmax scores that are not renormalised give every expert a gradient; else the logits are read at the picks only.
template <int L, bool VEC>
__global__ __launch_bounds__(64 * kWaves) void route_scores_backward_kernel(RouterArgs a) {
  constexpr int TW = 64 / L;
  extern __shared__ __align__(16) float rows[];  // [wave][TW][E rounded up to 4]
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int sub = lane & (L - 1), slot = lane / L;
  const long long t = ((long long)blockIdx.x * kWaves + wv) * TW + slot;
  const long long tt = min(t, (long long)a.T - 1);
  const float* row = a.logits + tt * a.ldl;
  float* mine = rows + (size_t)(wv * TW + slot) * ((a.E + 3) / 4 * 4);
  const bool keep = t < a.T && (!a.mask || a.mask[tt]);
  const bool dense = a.softmax && !a.renorm;

  // picks (an id outside [0, E) has no part)
  int id = -1;
  double g = 0.0;
  float z = 0.f;
  if (sub < a.k) {
    id = a.ids[tt * a.k + sub];
    if ((unsigned)id >= (unsigned)a.E) id = -1;
    if (id >= 0) {
      z = row[id];
      g = (double)a.scale * a.d_w[tt * a.k + sub];
    }
  }
  float m = id >= 0 ? z : -INFINITY;
  float dot = 0.f, inv = 0.f;
  if (dense) {
    for (int e = sub; e < a.E; e += L) m = fmaxf(m, row[e]);
  }
  m = max_lanes<L>(m);
  if (m == -INFINITY) m = 0.f;
  double s = 0.0, ds = 0.0;  // score, and its derivative by its own logit (softmax: the first term)
  if (id >= 0) {
    if (a.softmax) {
      ds = s = exp64((double)z - m);
    } else {
      const double e = exp64(-fabs((double)z)), r = rcp64(1.0 + e);
      s = z < 0.f ? e * r : r;
      ds = e * r * r;
    }
  }
  double part;
  if (dense) {
    // sum of all experts' exponentials in the order of the lanes; the row's own terms below in 32 bits
    double sum = 0.0;
    for (int e = sub; e < a.E; e += L) sum += exp64((double)row[e] - m);
    sum = sum_lanes<L>(sum);
    const double is = sum == 0.0 ? 0.0 : rcp64(sum);
    s *= is;
    dot = (float)sum_lanes<L>(g * s);
    inv = (float)is;
    part = g * s;
  } else {
    if (a.renorm) {
      const double sum = sum_lanes<L>(s);
      const double is = sum == 0.0 ? 0.0 : 1.0 / sum;
      g = (g - sum_lanes<L>(g * s) * is) * is;
    }
    part = g * ds;
  }

  for (int e = sub; e < a.E; e += L)
    mine[e] = dense ? -dot * inv * (float)exp64((double)row[e] - m) : 0.f;
  wave_lds_sync();
  if (id >= 0) atomicAdd(&mine[id], (float)part);
  wave_lds_sync();
  if (t >= a.T) return;
  float* out = a.d_logits + t * a.ldd;
  if constexpr (VEC) {
    for (int e = 4 * sub; e < a.E; e += 4 * L) {
      float4 v = keep ? *reinterpret_cast<const float4*>(mine + e) : make_float4(0.f, 0.f, 0.f, 0.f);
      if (a.accumulate) {
        const float4 o = *reinterpret_cast<const float4*>(out + e);
        v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
      }
      *reinterpret_cast<float4*>(out + e) = v;
    }
  } else {
    for (int e = sub; e < a.E; e += L) {
      const float v = keep ? mine[e] : 0.f;
      out[e] = a.accumulate ? out[e] + v : v;
    }
  }
}

bool vec4(const void* p, long long ld, int E) { return E % 4 == 0 && ld % 4 == 0 && ((uintptr_t)p & 15) == 0; }

template <int L, int V>
hipError_t launch_forward(const RouterArgs& a, hipStream_t s) {
  constexpr int per = kWaves * (64 / L);
  const dim3 grid((unsigned)(((long long)a.T + per - 1) / per)), block(64 * kWaves);
  const size_t lds = a.KG < a.G ? (size_t)per * (key_at(a.E) + a.G) * 4 : 0;
  const bool vec = V % 4 == 0 && vec4(a.logits, a.ldl, a.E);
  if constexpr (V % 4 == 0) {
    if (vec) {
      if (a.softmax) route_scores_kernel<L, V, true, true><<<grid, block, lds, s>>>(a);
      else route_scores_kernel<L, V, false, true><<<grid, block, lds, s>>>(a);
      return hipGetLastError();
    }
  }
  if (a.softmax) route_scores_kernel<L, V, true, false><<<grid, block, lds, s>>>(a);
  else route_scores_kernel<L, V, false, false><<<grid, block, lds, s>>>(a);
  return hipGetLastError();
}

template <int L>
hipError_t launch_backward(const RouterArgs& a, hipStream_t s) {
  constexpr int per = kWaves * (64 / L);
  const dim3 grid((unsigned)(((long long)a.T + per - 1) / per)), block(64 * kWaves);
  const size_t lds = (size_t)per * ((a.E + 3) / 4 * 4) * 4;
  if (vec4(a.d_logits, a.ldd, a.E)) route_scores_backward_kernel<L, true><<<grid, block, lds, s>>>(a);
  else route_scores_backward_kernel<L, false><<<grid, block, lds, s>>>(a);
  return hipGetLastError();
}

// Few tokens: a wave each, for the shorter chain; more than there are waves for: 16 lanes each.  16 lanes hold up to
// 256 experts and 16 picks.
bool sixteen(const RouterArgs& a) { return a.T > 2048 && a.E <= 256 && a.k <= 16; }

}  // namespace

hipError_t launch_route_scores(const RouterArgs& a, hipStream_t s) {
  if (sixteen(a)) {
    if (a.E <= 64) return launch_forward<16, 4>(a, s);
    if (a.E <= 128) return launch_forward<16, 8>(a, s);
    return launch_forward<16, 16>(a, s);
  }
  if (a.E <= 64) return launch_forward<64, 1>(a, s);
  if (a.E <= 128) return launch_forward<64, 2>(a, s);
  if (a.E <= 256) return launch_forward<64, 4>(a, s);
  if (a.E <= 512) return launch_forward<64, 8>(a, s);
  return launch_forward<64, 16>(a, s);
}

hipError_t launch_route_scores_backward(const RouterArgs& a, hipStream_t s) {
  return sixteen(a) ? launch_backward<16>(a, s) : launch_backward<64>(a, s);
}

}  // namespace moe
