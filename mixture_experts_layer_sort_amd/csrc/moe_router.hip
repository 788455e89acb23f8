// Scored routing: experts of a token by softmax or sigmoid scores, a choice
// bias, groups, renormalised weights; and the gradient of the logits.
//
//   s_e = sigmoid(l_e) or softmax(l)_e,   c_e = fp32(fp32(s_e) + b_e), -inf where l_e is
//   group score: its largest c, or fp32(largest + second); KG groups are kept
//   picks: the k largest c of the kept groups (equal ones: the lower id first)
//   w_j = scale s_j / (sum_i s_i or 1)
//
// Which of two experts is picked can hang on the last bit of a score, so scores
// are computed in 64 bits (relative error below 3e-14) and rounded once to the
// 32 bits that the definition names: picks are the same whatever computes them (unless
// a score is that near to a border between two 32-bit numbers).
// (On this GPU a 64-bit multiply-add issues like a 32-bit one.)
//
// A token has L lanes, a lane V consecutive experts, so that positions order
// like ids and equal choices need no ids to be compared.  A lane sorts its largest
// KEEP >= min(k, V) choices (keys alone, by a network); a round takes the maximum of
// the lanes' first keys, and the first lane that has it moves its list up by one.
// Which expert of the lane it was is looked up at the end for all picks at once,
// in the keys as they were (picks of one lane with one value follow each other, the
// n-th is the n-th such expert).  L = 16 (four tokens per wave share every exchange)
// where there are tokens enough to fill the GPU, L = 64 for few tokens or many experts.
//
// Bound by arithmetic: 16384 x 256, sigmoid, 8 groups, top-8: 12.2 us, of which the 64-bit
// scores are 4, the rounds 1.3, the sort 0.6 and the bytes (17.8 MB) 3.5; one token 3.7.
// Softmax without groups: 16384 x 64 5.9 us, x 128 7.5, x 256 11.3, x 384 and x 512 (64
// lanes a token) 23; one token of 1024 experts 5.4.
// Gradient: 32768 x 256, sigmoid 10.5 us (34 MB written), bound by memory; softmax that is
// not renormalised 16.1 (67 MB, 4.2 TB/s), bound by its 64-bit exponentials: in 32 bits, and
// the terms rounded before they cancel, it takes 14.1 and loses all digits of a pick whose
// probability is near 1.
#include "moe_router.h"

#include "moe_wave.h"

namespace moe {
namespace {

constexpr int kWaves = 4;
constexpr uint32_t kOff = 0x007FFFFFu;  // key of -inf: still before 0, an expert that cannot be picked

// exp(x), |x| <= 709: 2^n times a polynomial of the rest f, |f| <= ln 2 / 2 (interpolated at the 10 Chebyshev nodes, off
// by 2e-14 relative; with ln 2 in one part another 1e-16 |n| / 2).
// Constants come from scalar registers (one instruction a step; as literals each would be moved into place first), n by
// an addition that leaves it in the low bits of 1.5 2^52 + n, and 2^n by an addition to the exponent.
struct Exp64 {
  double c[10], log2e, ln2, round;
  __device__ __forceinline__ Exp64()
      : c{1.0000000000000135,    1.0000000000000013,    0.4999999999943859,     0.16666666666615648,    0.04166666704055213,
          0.008333333367311624,  0.0013888801749621653, 0.00019841190647512536, 2.4884459768350122e-05, 2.763264069051338e-06},
        log2e(1.4426950408889634074), ln2(-0.69314718055994530942), round(0x1.8p52) {
#pragma unroll
    for (int i = 0; i < 10; ++i) asm("" : "+s"(c[i]));
    asm("" : "+s"(log2e), "+s"(ln2), "+s"(round));
  }
  __device__ __forceinline__ double operator()(double x) const {
    const double y = fma(x, log2e, round), f = fma(y - round, ln2, x);
    double p = c[9];
#pragma unroll
    for (int i = 8; i >= 0; --i) p = fma(p, f, c[i]);
    return __hiloint2double(__double2hiint(p) + (__double2loint(y) << 20), __double2loint(p));
  }
};
// exp(x), x <= 709; 0 below -700.  NaN goes on: the sum of exponents leaves one as it is or makes a number of it.
__device__ __forceinline__ double exp64(double x, const Exp64& e) { return x < -700.0 ? 0.0 : x == x ? e(x) : x; }

// 1 / d, d a normal number: the hardware's estimate r and its error's series, r (1 + e + e^2), e = 1 - d r.
__device__ __forceinline__ double rcp64(double d) {
  const double r = __builtin_amdgcn_rcp(d), e = fma(-d, r, 1.0);
  return fma(r, fma(e, e, e), r);
}

// A pick's score but for a factor exp(base) that all picks of the token share, and the score's derivative by its logit over
// the score (softmax: but for the sum's part).
struct Share {
  double s, rest;
};
// The base of picks whose largest logit is m.  A softmax has it for its sum.  Sigmoids have one where all of them are far
// below 0: there they are exp(l) (1 + exp(l) is 1 in 64 bits), and renormalised weights, which are ratios, stay those of
// the formula where exp(l) itself is too small for 64 bits.
template <bool SOFTMAX>
__device__ __forceinline__ double share_base(float m) {
  return m == -INFINITY ? 0.0 : SOFTMAX || m < -40.f ? (double)m : 0.0;
}
template <bool SOFTMAX>
__device__ __forceinline__ Share share_of(float l, double base, const Exp64& ex) {
  const bool plain = SOFTMAX || base != 0.0;
  const double e = exp64(plain ? (double)l - base : -fabs((double)l), ex);
  if (plain) return {e, 1.0};
  const double r = rcp64(1.0 + e);
  return l < 0.f ? Share{e * r, r} : Share{r, e * r};
}

// sigmoid(l) rounded to 32 bits (0 below -104); l = NaN: unspecified.
__device__ __forceinline__ float sigmoid32(float l, const Exp64& e) {
  return (float)rcp64(1.0 + e((double)fminf(fmaxf(-l, -700.f), 700.f)));
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

// ------------------------------------------------------------------ sorting a lane's keys, largest first

template <int N>
__device__ __forceinline__ void exchange(uint32_t (&v)[N], int i, int j) {
  const uint32_t a = v[i], b = v[j];
  v[i] = max(a, b);
  v[j] = min(a, b);
}
// Merge exchange sort (Batcher) of v[lo .. lo + n), n a power of two, by its loops over p, q, r, d.
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t (&v)[N], int lo, int n) {
#pragma unroll
  for (int p = 1; p < n; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < n; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < n && (i + j) / (2 * p) == (i + j + k) / (2 * p)) exchange(v, lo + i + j, lo + i + j + k);
}
// The largest KEEP of key, sorted.
template <int V, int KEEP>
__device__ __forceinline__ void sort_list(const uint32_t (&key)[V], uint32_t (&list)[KEEP]) {
  uint32_t v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = key[i];
  if constexpr (KEEP == V) {
    sort_keys<V>(v, 0, V);
  } else {  // both halves, the larger of opposite places (the largest half, first rising, then falling), and its merge
    static_assert(2 * KEEP == V, "half");
    sort_keys<V>(v, 0, KEEP);
    sort_keys<V>(v, KEEP, KEEP);
#pragma unroll
    for (int i = 0; i < KEEP; ++i) v[i] = max(v[i], v[V - 1 - i]);
#pragma unroll
    for (int d = KEEP / 2; d >= 1; d /= 2)
#pragma unroll
      for (int i = 0; i < KEEP; ++i)
        if ((i & d) == 0) exchange(v, i, i + d);
  }
#pragma unroll
  for (int i = 0; i < KEEP; ++i) list[i] = v[i];
}

// ------------------------------------------------------------------ groups

// The two largest keys of a group that has its LG lanes in a row (LG a power of two up to 16), in each of them.
template <int D>
__device__ __forceinline__ void join_two(uint32_t& b1, uint32_t& b2) {
  uint32_t o1, o2;
  if constexpr (D == 1) {         // lane ^ 1, ^ 2: within four lanes
    o1 = __builtin_amdgcn_update_dpp(0u, b1, 0xB1, 0xF, 0xF, true);
    o2 = __builtin_amdgcn_update_dpp(0u, b2, 0xB1, 0xF, 0xF, true);
  } else if constexpr (D == 2) {
    o1 = __builtin_amdgcn_update_dpp(0u, b1, 0x4E, 0xF, 0xF, true);
    o2 = __builtin_amdgcn_update_dpp(0u, b2, 0x4E, 0xF, 0xF, true);
  } else if constexpr (D == 4) {  // mirrored in eight: fours are equal by now
    o1 = __builtin_amdgcn_update_dpp(0u, b1, 0x141, 0xF, 0xF, true);
    o2 = __builtin_amdgcn_update_dpp(0u, b2, 0x141, 0xF, 0xF, true);
  } else {
    o1 = ror16<8>(b1);
    o2 = ror16<8>(b2);
  }
  b2 = max(min(b1, o1), max(b2, o2));
  b1 = max(b1, o1);
}

// Groups of LG whole lanes before this lane's (with a larger score, or as large and lower).
template <int R>
__device__ __forceinline__ void count_before(uint32_t score, int sub, int LG, int& before) {
  if constexpr (R < 16) {
    if ((R & (LG - 1)) == 0) {  // rotated by whole groups: a lower one comes from R lanes below, if there are any
      const uint32_t other = ror16<R>(score);
      before += other > score || (other == score && sub >= R);
    }
    count_before<R + 1>(score, sub, LG, before);
  }
}

template <int L, int V, int KEEP, bool SOFTMAX, bool VEC>
__global__ __launch_bounds__(64 * kWaves) void route_scores_kernel(RouterArgs a) {
  constexpr int TW = 64 / L;  // tokens of a wave
  __shared__ uint32_t shared[kWaves * TW][V * L];  // keys: expert sub V + i at i L + sub
  extern __shared__ uint32_t scores[];             // groups that are not whole lanes: [wave][TW][G]
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int sub = lane & (L - 1), slot = lane / L;
  const long long t = ((long long)blockIdx.x * kWaves + wv) * TW + slot;
  const float* row = a.logits + min(t, (long long)a.T - 1) * a.ldl;
  uint32_t* keys = shared[wv * TW + slot];
  const int e0 = sub * V;

  float l[V], b[V];
#pragma unroll
  for (int i = 0; i < V; ++i) l[i] = -INFINITY, b[i] = 0.f;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      if (e0 + i < a.E) {
        const float4 v = *reinterpret_cast<const float4*>(row + e0 + i);
        l[i] = v.x, l[i + 1] = v.y, l[i + 2] = v.z, l[i + 3] = v.w;
        if (a.bias) {
          const float4 c = *reinterpret_cast<const float4*>(a.bias + e0 + i);
          b[i] = c.x, b[i + 1] = c.y, b[i + 2] = c.z, b[i + 3] = c.w;
        }
      }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i < a.E) {
        l[i] = row[e0 + i];
        if (a.bias) b[i] = a.bias[e0 + i];
      }
  }

  const Exp64 ex64;
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
    for (int i = 0; i < V; ++i) sum += ex[i] = exp64((double)l[i] - top, ex64);
    sum = sum_lanes<L>(sum);
    inv = sum == 0.0 ? 0.0 : rcp64(sum);
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = __float_as_uint((float)(ex[i] * inv));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = __float_as_uint(sigmoid32(l[i], ex64));
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    asm("" : "+v"(key[i]));  // computed for all: not sunk behind a branch for experts that are off, one by one
    const uint32_t k = l[i] == -INFINITY ? kOff : order_key(__uint_as_float(key[i]) + b[i]);
    key[i] = e0 + i < a.E ? k : 0u;
    keys[i * L + sub] = key[i];
  }
  uint32_t list[KEEP];
  sort_list<V, KEEP>(key, list);

  if (a.KG < a.G) {  // lists of experts of groups that are not kept: 0
    const int per = a.E / a.G, LG = per / V;
    if (LG * V == per && LG <= 16 && (LG & (LG - 1)) == 0) {
      uint32_t b1 = list[0], b2 = KEEP > 1 ? list[KEEP > 1 ? 1 : 0] : 0u;
      if (LG > 1) join_two<1>(b1, b2);
      if (LG > 2) join_two<2>(b1, b2);
      if (LG > 4) join_two<4>(b1, b2);
      if (LG > 8) join_two<8>(b1, b2);
      uint32_t score = a.top == 1 ? b1 : order_key(of_key(b1) + of_key(b2));
      int before = 0;
      if constexpr (L == 16) {
        score = e0 < a.E ? score : 0u;  // lanes behind the last expert: behind every group
        count_before<1>(score, sub, LG, before);
      } else {
        for (int g = 0; g < a.G; ++g) {
          const uint32_t other = __builtin_amdgcn_readlane(score, g * LG);
          before += other > score || (other == score && g * LG < (sub & -LG));
        }
      }
#pragma unroll
      for (int i = 0; i < KEEP; ++i) list[i] = before < a.KG ? list[i] : 0u;
    } else {
      uint32_t* score = scores + (wv * TW + slot) * a.G;
      wave_lds_sync();
      for (int g = sub; g < a.G; g += L) {
        uint32_t b1 = 0, b2 = 0;
        for (int e = g * per; e < (g + 1) * per; ++e) {
          const uint32_t k = keys[e % V * L + e / V];
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
          for (int e = g * per; e < (g + 1) * per; ++e) keys[e % V * L + e / V] = 0u;
      }
      wave_lds_sync();
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = keys[i * L + sub];
      sort_list<V, KEEP>(key, list);
    }
  }

  // round j: its value, lane, and how many before it had both
  uint32_t value = 0, last = 0;
  int from = 0, nth = 0, last_lane = -1, run = 0;
  for (int j = 0; j < a.k; ++j) {
    const uint32_t best = max_lanes<L>(list[0]);
    const uint64_t same = __ballot(list[0] == best);
    int first;
    if constexpr (L == 64) first = __ffsll((unsigned long long)same) - 1;
    else first = __ffs((uint32_t)(same >> (lane & 48)) & 0xFFFFu) - 1;
    run = best == last && first == last_lane ? run + 1 : 0;
    last = best;
    last_lane = first;
    value = sub == j ? best : value;
    from = sub == j ? first : from;
    nth = sub == j ? run : nth;
    // by a bit mask (as a choice of values it compiles to selects among all places)
    const uint32_t move = sub == first ? ~0u : 0u;
#pragma unroll
    for (int i = 0; i < KEEP; ++i) list[i] ^= (list[i] ^ (i + 1 < KEEP ? list[i + 1 < KEEP ? i + 1 : i] : 0u)) & move;
  }
  wave_lds_sync();
  int at = 0;
#pragma unroll
  for (int i = V - 1; i >= 0; --i) at = keys[i * L + from] == value ? i : at;  // the first one
  if (nth > 0) {
    int seen = 0;
    for (int i = 0; i < V; ++i)
      if (keys[i * L + from] == value && seen++ == nth) at = i;
  }

  const bool mine = sub < a.k;
  const int id = mine ? from * V + at : 0;
  const float z = mine ? row[id] : -INFINITY;
  double s;
  if (a.renorm) {
    s = share_of<SOFTMAX>(z, share_base<SOFTMAX>(max_lanes<L>(z)), ex64).s;
    const double sum = sum_lanes<L>(s);
    s = sum == 0.0 ? 0.0 : s / sum;
    if (SOFTMAX && inv != inv) s = inv;  // a NaN anywhere in the row
  } else {
    s = SOFTMAX ? exp64((double)z - top, ex64) * inv : share_of<false>(z, 0.0, ex64).s;
  }
  if (mine && t < a.T) {
    a.ids[t * a.k + sub] = id;
    a.w[t * a.k + sub] = (float)((double)a.scale * s);
  }
}

// Gradient.  L lanes per token; lane j has pick j and its part of the gradient; the picks' values meet the row's others
// in LDS, where a lane has 16 experts in fours (4 (l + L i) .. + 3) or, unaligned, every L-th, so that rows are stored in
// one run.  DENSE: softmax scores that are not renormalised, which give every expert a gradient; else the logits are
// read at the picks only, and the rest of a row is zero.
// Every value is 64 bits up to one rounding: of a dominant pick g s (1 - s) is left of two terms that cancel, and the
// parts of an id that a row holds twice may.  So one lane of those with an id has
// its whole value, which no other adds to.
template <int L, bool DENSE, bool VEC>
__global__ __launch_bounds__(64 * kWaves) void route_scores_backward_kernel(RouterArgs a) {
  constexpr int TW = 64 / L, N = 16;
  extern __shared__ __align__(16) float rows[];  // [wave][TW][E rounded up to 4]
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int sub = lane & (L - 1), slot = lane / L;
  const long long t = ((long long)blockIdx.x * kWaves + wv) * TW + slot;
  const long long tt = min(t, (long long)a.T - 1);
  const float* row = a.logits + tt * a.ldl;
  float* mine = rows + (size_t)(wv * TW + slot) * ((a.E + 3) / 4 * 4);
  const bool keep = t < a.T && (!a.mask || a.mask[tt]);
  auto expert = [&](int i) { return VEC ? 4 * (sub + L * (i / 4)) + i % 4 : sub + L * i; };

  float p[N];  // DENSE: logits, then the row's values
  if constexpr (DENSE) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      if constexpr (VEC) {
        float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (expert(i) < a.E) v = *reinterpret_cast<const float4*>(row + expert(i));
        p[i] = v.x, p[i + 1] = v.y, p[i + 2] = v.z, p[i + 3] = v.w;
      } else {
#pragma unroll
        for (int c = i; c < i + 4; ++c) p[c] = expert(c) < a.E ? row[expert(c)] : -INFINITY;
      }
    }
  }

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
      mine[id] = __uint_as_float(sub);
    }
  }
  wave_lds_sync();
  const bool owner = id >= 0 && __float_as_uint(mine[id]) == (uint32_t)sub;  // one of the lanes that have this id
  wave_lds_sync();
  float m = id >= 0 ? z : -INFINITY;
  if constexpr (DENSE) {
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, p[i]);
  }
  m = max_lanes<L>(m);
  if (m == -INFINITY) m = 0.f;
  const Exp64 ex64;
  Share h = {0.0, 0.0};
  if (id >= 0) {
    if (DENSE || a.softmax) h = share_of<true>(z, m, ex64);  // m: of all experts (DENSE) or of the picks
    else h = share_of<false>(z, a.renorm ? share_base<false>(m) : 0.0, ex64);
  }
  double part, rest = 0.0;  // of the pick, and what every expert's score takes off it
  if constexpr (DENSE) {
    double ex[N], sum = 0.0;
#pragma unroll
    for (int i = 0; i < N; ++i) sum += ex[i] = exp64((double)p[i] - m, ex64);
    sum = sum_lanes<L>(sum);
    const double is = sum == 0.0 ? 0.0 : rcp64(sum);
    part = g * h.s * is;
    const double f = -sum_lanes<L>(part) * is;
    rest = h.s * f;
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = (float)(ex[i] * f);
  } else {
    if (a.renorm) {
      const double sum = sum_lanes<L>(h.s);
      h.s = sum == 0.0 ? 0.0 : h.s / sum;  // the pick's weight
      g -= sum_lanes<L>(g * h.s);
    }
    part = g * h.s * h.rest;
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = 0.f;
  }
  if (__ballot(id >= 0 && !owner)) {  // an id twice: all of its parts, in the order of the picks
    double all = 0.0;
    for (int j = 0; j < a.k; ++j) {
      const int other = __shfl(id, j, L);
      const double v = __shfl(part, j, L);
      all += other == id ? v : 0.0;
    }
    part = all;
  }

#pragma unroll
  for (int i = 0; i < N; i += 4) {
    if constexpr (VEC) {
      if (expert(i) < a.E) *reinterpret_cast<float4*>(mine + expert(i)) = make_float4(p[i], p[i + 1], p[i + 2], p[i + 3]);
    } else {
#pragma unroll
      for (int c = i; c < i + 4; ++c)
        if (expert(c) < a.E) mine[expert(c)] = p[c];
    }
  }
  wave_lds_sync();
  if (owner) mine[id] = (float)(part + rest);
  wave_lds_sync();
  if (t >= a.T || (a.accumulate && !keep)) return;  // a masked row stays as it is
  float* out = a.d_logits + t * a.ldd;
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    if constexpr (VEC) {
      const int e = expert(i);
      if (e >= a.E) break;
      float4 v = keep ? *reinterpret_cast<const float4*>(mine + e) : make_float4(0.f, 0.f, 0.f, 0.f);
      if (a.accumulate) {
        const float4 o = *reinterpret_cast<const float4*>(out + e);
        v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
      }
      *reinterpret_cast<float4*>(out + e) = v;
    } else {
#pragma unroll
      for (int c = i; c < i + 4; ++c) {
        const int e = expert(c);
        if (e >= a.E) break;
        const float v = keep ? mine[e] : 0.f;
        out[e] = a.accumulate ? out[e] + v : v;
      }
    }
  }
}

bool vec4(const void* p, long long ld, int E) { return E % 4 == 0 && ld % 4 == 0 && ((uintptr_t)p & 15) == 0; }

template <int L, int V, int KEEP>
hipError_t launch_lists(const RouterArgs& a, hipStream_t s) {
  constexpr int per = kWaves * (64 / L);
  const dim3 grid((unsigned)(((long long)a.T + per - 1) / per)), block(64 * kWaves);
  const size_t lds = a.KG < a.G ? (size_t)per * a.G * 4 : 0;
  if constexpr (V % 4 == 0) {
    if (vec4(a.logits, a.ldl, a.E) && ((uintptr_t)a.bias & 15) == 0) {
      if (a.softmax) route_scores_kernel<L, V, KEEP, true, true><<<grid, block, lds, s>>>(a);
      else route_scores_kernel<L, V, KEEP, false, true><<<grid, block, lds, s>>>(a);
      return hipGetLastError();
    }
  }
  if (a.softmax) route_scores_kernel<L, V, KEEP, true, false><<<grid, block, lds, s>>>(a);
  else route_scores_kernel<L, V, KEEP, false, false><<<grid, block, lds, s>>>(a);
  return hipGetLastError();
}
template <int L, int V>
hipError_t launch_forward(const RouterArgs& a, hipStream_t s) {
  if constexpr (V == 16) {
    if (a.k <= 8) return launch_lists<L, 16, 8>(a, s);
  }
  return launch_lists<L, V, V>(a, s);
}

template <int L, bool DENSE>
hipError_t launch_rows(const RouterArgs& a, hipStream_t s) {
  constexpr int per = kWaves * (64 / L);
  const dim3 grid((unsigned)(((long long)a.T + per - 1) / per)), block(64 * kWaves);
  const size_t lds = (size_t)per * ((a.E + 3) / 4 * 4) * 4;
  if (vec4(a.d_logits, a.ldd, a.E) && (!DENSE || vec4(a.logits, a.ldl, a.E)))
    route_scores_backward_kernel<L, DENSE, true><<<grid, block, lds, s>>>(a);
  else
    route_scores_backward_kernel<L, DENSE, false><<<grid, block, lds, s>>>(a);
  return hipGetLastError();
}
template <int L>
hipError_t launch_backward(const RouterArgs& a, hipStream_t s) {
  return a.softmax && !a.renorm ? launch_rows<L, true>(a, s) : launch_rows<L, false>(a, s);
}

// A wave for each of few tokens, for the shorter chain; 16 lanes where tokens fill the GPU that way (sigmoid, top-8, us
// with 64 / 16 lanes: 256 experts, 2048 tokens 5.2 / 6.4, 4096 6.6 / 6.5, 16384 17.9 / 12.2; 64 experts, 2048 tokens
// 3.4 / 3.6, 4096 4.1 / 3.7).  16 lanes hold up to 256 experts and 16 picks.
bool sixteen(const RouterArgs& a) { return a.T > (a.E > 128 ? 4096 : 2048) && a.E <= 256 && a.k <= 16; }

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
