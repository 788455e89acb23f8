// Streaming product on block-128 fp8 weights: few token rows per weight
// matrix (decoding), so the time is that of reading the weights once.
//
// Item = (token tile of 16 NT rows, R fragments of 16 weight rows).  The
// block's KS waves take the 128-wide K blocks in turn; a wave reads its weight
// fragment straight from the row-major codes into the operand registers (lane
// r + 16 q: row r, bytes [16 q, 16 q + 16) and [64 + 16 q, + 16) of the block:
// two loads that together use whole 128-byte lines; which 32 of the 128 bytes
// a lane holds does not matter, since tokens use the same order) and quantises
// the tokens' bf16 values of the same block itself: the four lanes of a token
// share its 128 values, so the block maximum is two exchanges away.  Partial
// sums of the waves meet in LDS in wave order (the same bits every run).
#include "moe_fp8.h"

namespace moe {
namespace {

template <int NT, int R, int KS, Fp8Mode MODE>
__global__ __launch_bounds__(64 * KS) void fp8_stream_kernel(Fp8Args a) {
  constexpr int kRows = 16 * NT;
  __shared__ f32x4 red[KS][R * NT][64];
  __shared__ int cum[1025];
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int KB = (a.K + kFp8Blk - 1) / kFp8Blk;
  const int NB = (a.N + kFp8Blk - 1) / kFp8Blk;
  // weight rows of one item: DENSE / DOWN 16 R consecutive ones; GATE_UP 8 R gate rows and the 8 R up rows
  constexpr int kItemN = MODE == FP8_GATE_UP ? 8 * R : 16 * R;
  const int nspan = MODE == FP8_GATE_UP ? a.N / 2 : a.N;
  const int nitems = (nspan + kItemN - 1) / kItemN;

  int total;  // token tiles
  if constexpr (MODE == FP8_DENSE) {
    total = (a.rows + kRows - 1) / kRows;
  } else {
    // prefix of the experts' token tiles: one pass of a scan over chunks of the block's size
    int base = 0;
    if (tid == 0) cum[0] = 0;
    int* part = reinterpret_cast<int*>(&red[0][0][0]);
    for (int e0 = 0; e0 < a.E; e0 += 64 * KS) {
      const int e = e0 + tid;
      int c = 0;
      if (e < a.E) c = (max(0, a.offsets[e + 1] - a.offsets[e]) + kRows - 1) / kRows;
      int s = c;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(s, d, 64);
        if (lane >= d) s += o;
      }
      if (lane == 63) part[wv] = s;
      __syncthreads();
      int before = base, all = 0;
      for (int i = 0; i < KS; ++i) {
        if (i < wv) before += part[i];
        all += part[i];
      }
      if (e < a.E) cum[e + 1] = before + s;
      base += all;
      __syncthreads();
    }
    total = base;
  }

  const long long items = (long long)total * nitems;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    // tiles of one weight slab run next to each other on one XCD (blocks go round the 8 XCDs)
    int tile, slab;
    {
      const long long per = 8LL * total;
      const long long g = it / per;
      const int left = min(8LL, nitems - 8 * g);  // slabs of this group
      const long long o = it - g * per;
      slab = (int)(8 * g + o % left);
      tile = (int)(o / left);
    }
    int e = 0, r0, rend;
    if constexpr (MODE == FP8_DENSE) {
      r0 = tile * kRows;
      rend = a.rows;
    } else {
      int lo = 0, hi = a.E - 1;  // the expert with cum[e] <= tile < cum[e + 1]
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid + 1] > tile) hi = mid;
        else lo = mid + 1;
      }
      e = lo;
      r0 = max(0, a.offsets[e]) + (tile - cum[e]) * kRows;
      rend = min(a.offsets[e + 1], a.rows);
    }
    // weight fragments of this lane; rows past the end repeat the last one (results dropped)
    const uint8_t* wrow[R];
    const float* wsc[R];
#pragma unroll
    for (int f = 0; f < R; ++f) {
      int first;
      if constexpr (MODE == FP8_GATE_UP) first = (f < R / 2 ? 0 : nspan) + slab * kItemN + 16 * (f % (R / 2));
      else first = slab * kItemN + 16 * f;
      const int n = min(first + r, a.N - 1);
      wrow[f] = a.w + ((size_t)e * a.N + n) * a.K + 16 * q;
      wsc[f] = a.wsc + ((size_t)e * NB + min(first, a.N - 1) / kFp8Blk) * KB;
    }
    // token rows of this lane
    const uint16_t* xrow[NT];
    bool live[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int row = r0 + 16 * t + r;
      live[t] = row < rend;
      int src = min(row, rend - 1);
      if constexpr (MODE == FP8_GATE_UP) src = a.pairs[src] / a.k;
      xrow[t] = a.x + (size_t)src * a.ldx + 16 * q;
    }
    f32x4 acc[R][NT];
#pragma unroll
    for (int f = 0; f < R; ++f)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[f][t] = f32x4{0.f, 0.f, 0.f, 0.f};

    struct Step {
      u32x4 w[R][2];
      u32x4 x[NT][4];
      float s[R];
    };
    const u32x4 none = {0, 0, 0, 0};
    auto load = [&](Step& st, int kb) {
      const bool lo = kb * kFp8Blk + 16 * q < a.K, hi = kb * kFp8Blk + 64 + 16 * q < a.K;
#pragma unroll
      for (int f = 0; f < R; ++f) {
        const uint8_t* p = wrow[f] + (size_t)kb * kFp8Blk;
        st.w[f][0] = lo ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)) : none;
        st.w[f][1] = hi ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + 64)) : none;
        st.s[f] = wsc[f][kb];
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const u32x4* p = reinterpret_cast<const u32x4*>(xrow[t] + (size_t)kb * kFp8Blk);
        st.x[t][0] = live[t] && lo ? p[0] : none;
        st.x[t][1] = live[t] && lo ? p[1] : none;
        st.x[t][2] = live[t] && hi ? p[8] : none;
        st.x[t][3] = live[t] && hi ? p[9] : none;
      }
    };
    auto compute = [&](const Step& st) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float m = kFp8Tiny;
#pragma unroll
        for (int j = 0; j < 4; ++j) m = fp8_amax8(st.x[t][j], m);
        m = max_rows(m);
        const float f = kFp8Max / m, sx = m / kFp8Max;
        i32x8 b;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint2 c = fp8_codes8(st.x[t][j], f);
          b[2 * j] = (int)c.x;
          b[2 * j + 1] = (int)c.y;
        }
#pragma unroll
        for (int fr = 0; fr < R; ++fr) {
          const u32x4 lo = st.w[fr][0], hi = st.w[fr][1];
          const i32x8 aw = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
          const f32x4 z = fp8_mfma(aw, b);
          const float sc = sx * st.s[fr];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[fr][t][i] = fmaf(z[i], sc, acc[fr][t][i]);
        }
      }
    };
    if (wv < KB) {
      Step s0, s1;
      load(s0, wv);
      int kb = wv;
      while (true) {
        const bool more = kb + KS < KB;
        if (more) load(s1, kb + KS);
        compute(s0);
        if (!more) break;
        const bool more2 = kb + 2 * KS < KB;
        if (more2) load(s0, kb + 2 * KS);
        compute(s1);
        if (!more2) break;
        kb += 2 * KS;
      }
    }
    // waves' partial sums, in wave order; accumulator (f, t) element i of lane r + 16 q is weight row
    // 16 f + 4 q + i, token 16 t + r
#pragma unroll
    for (int f = 0; f < R; ++f)
#pragma unroll
      for (int t = 0; t < NT; ++t) red[wv][f * NT + t][lane] = acc[f][t];
    __syncthreads();
    constexpr int kUnits = MODE == FP8_GATE_UP ? R / 2 * NT : R * NT;
    for (int u = wv; u < kUnits; u += KS) {
      auto sum = [&](int j) {
        f32x4 v = red[0][j][lane];
#pragma unroll
        for (int i = 1; i < KS; ++i) v += red[i][j][lane];
        return v;
      };
      const int f = u / NT, t = u % NT;
      f32x4 v = sum(u);
      const int row = r0 + 16 * t + r;
      if constexpr (MODE == FP8_GATE_UP) {
        const f32x4 up = sum(u + R / 2 * NT);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = swiglu(v[i], up[i], a.limit);
      }
      if (row < rend) {
        const int n = slab * kItemN + 16 * f + 4 * q;
        const size_t orow = MODE == FP8_DOWN ? a.pairs[row] : row;
        uint16_t* o = a.out + orow * (size_t)a.ldo + n;
        const uint32_t b0 = f32_to_bf16(v[0]), b1 = f32_to_bf16(v[1]), b2 = f32_to_bf16(v[2]), b3 = f32_to_bf16(v[3]);
        if (n + 4 <= nspan && ((uintptr_t)o & 7) == 0) {
          *reinterpret_cast<uint2*>(o) = make_uint2(b0 | b1 << 16, b2 | b3 << 16);
        } else {
          if (n < nspan) o[0] = (uint16_t)b0;
          if (n + 1 < nspan) o[1] = (uint16_t)b1;
          if (n + 2 < nspan) o[2] = (uint16_t)b2;
          if (n + 3 < nspan) o[3] = (uint16_t)b3;
        }
      }
    }
    __syncthreads();  // the sums are read before the next item's overwrite them
  }
}

template <Fp8Mode MODE>
hipError_t launch_mode(const Fp8Args& a, int cus, hipStream_t s) {
  constexpr int R = 4, KS = 4;
  const int span = MODE == FP8_GATE_UP ? a.N / 2 : a.N, per = MODE == FP8_GATE_UP ? 8 * R : 16 * R;
  const long long slabs = (span + per - 1) / per;
  const bool one = MODE == FP8_DENSE ? a.rows <= 16 : a.rows <= 16LL * a.E;
  const int tile = one ? 16 : 32;
  const long long tiles = (a.rows + tile - 1) / tile + (MODE == FP8_DENSE ? 0 : (a.rows < a.E ? a.rows : a.E));
  long long grid = tiles * slabs;
  if (grid > 3LL * cus) grid = 3LL * cus;
  if (one) fp8_stream_kernel<1, R, KS, MODE><<<dim3((unsigned)grid), dim3(64 * KS), 0, s>>>(a);
  else fp8_stream_kernel<2, R, KS, MODE><<<dim3((unsigned)grid), dim3(64 * KS), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_stream(Fp8Mode mode, const Fp8Args& a, int cus, hipStream_t s) {
  switch (mode) {
    case FP8_DENSE: return launch_mode<FP8_DENSE>(a, cus, s);
    case FP8_GATE_UP: return launch_mode<FP8_GATE_UP>(a, cus, s);
    default: return launch_mode<FP8_DOWN>(a, cus, s);
  }
}

}  // namespace moe
