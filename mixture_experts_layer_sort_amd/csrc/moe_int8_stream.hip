// Streaming product on 8-bit integer weights: few token rows per weight matrix
// (decoding), so the time is that of reading the weights once.
//
// Item = (token tile, R fragments of 16 weight rows).  The block's KS waves take
// the 128-wide K steps in turn; a wave reads its weight fragment straight from the
// row-major codes into the operand registers (lane r + 16 q: row r, bytes [16 q,
// 16 q + 16) and [64 + 16 q, + 16) of the step; which 32 of the 128 bytes a lane
// holds does not matter, since tokens use the same order), D steps ahead.  The
// waves' integer sums meet in LDS.
//
// Bound by reading the weights: one token of 8 of 256 experts of 7168 x 2048, gate / up
// 46.6 us (235 MB, 5.0 TB/s), down 24.7 (117 MB, 4.8) behind 4.8 for the intermediate's
// codes; 24 tokens 592 and 307.
#include "moe_int8.h"
#include "moe_wave.h"

namespace moe {
namespace {

// fp32 value of a sum: the same two products in every kernel.
__device__ __forceinline__ float value(int acc, float sx, float sw) { return (float)acc * sx * sw; }

// Columns n .. n + 3 of an output row that ends at N.
__device__ __forceinline__ void store4(uint16_t* row, int n, int N, const f32x4& v) {
  uint16_t* o = row + n;
  const uint32_t lo = bf16_pair(v[0], v[1]), hi = bf16_pair(v[2], v[3]);
  if (n + 4 <= N && ((uintptr_t)o & 7) == 0) {
    *reinterpret_cast<uint2*>(o) = make_uint2(lo, hi);
  } else {
    if (n < N) o[0] = (uint16_t)lo;
    if (n + 1 < N) o[1] = (uint16_t)(lo >> 16);
    if (n + 2 < N) o[2] = (uint16_t)hi;
    if (n + 3 < N) o[3] = (uint16_t)(hi >> 16);
  }
}

// Dynamic LDS of the kernels that quantise into it, at most: the limit asked for on every call (the same number, whatever
// other threads launch meanwhile).
constexpr int kBlockLds = 64 * 1024;
__host__ __device__ inline size_t block_lds(int rows, int K) { return (size_t)rows * (int8_pad(K) + 16); }

// Rows `row(i)`, i < rows <= 16, of K bf16 values into LDS: codes [rows][Kp + 16] (the 16 rows of a fragment read start 4
// banks apart), scales [rows].  G waves share a row (all KS of them one row, one each of KS or more).  A thread's first
// HELD pieces of 8 values are loaded by load() (before the weights, since loads return in order) and stay in registers
// between the maximum and the codes, the others are read again.
template <int KS, int HELD, class F>
struct BlockQuantizer {
  int rows, K, G, wv, lane;
  F row;
  u32x4 v[HELD];

  __device__ __forceinline__ BlockQuantizer(int rows_, int K_, int wv_, int lane_, F row_)
      : rows(rows_), K(K_), G(KS), wv(wv_), lane(lane_), row(row_) {
    while (G > 1 && KS / G < rows) G /= 2;
  }
  __device__ __forceinline__ int first() const { return 8 * (lane + 64 * (wv & (G - 1))); }
  __device__ __forceinline__ u32x4 piece(int i, int c) const {
    return c < K ? *reinterpret_cast<const u32x4*>(row(i) + c) : u32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void load() {
    const int i = min(wv / G, rows - 1);
#pragma unroll
    for (int u = 0; u < HELD; ++u) v[u] = piece(i, first() + u * 512 * G);
  }
  __device__ __forceinline__ void store(uint8_t* codes, float* scales, uint32_t* part) {
    const int Kp = int8_pad(K), step = 512 * G;
    for (int i = wv / G; i < rows || G > 1; i += KS / G) {  // G > 1: every wave once
      const bool held = i == wv / G && i < rows;
      uint32_t m = kFp8TinyBits;
      if (held) {
#pragma unroll
        for (int u = 0; u < HELD; ++u) m = fp8_amax8(v[u], m);
      }
      for (int c = first() + (held ? HELD * step : 0); c < K && i < rows; c += step) m = fp8_amax8(piece(i, c), m);
      // magnitudes on their bits, so that a NaN, above everything, stays
      uint32_t b = max_lanes<64>(max(m << 16, m & 0xFFFF0000u));
      if (G > 1) {
        if (lane == 0) part[wv] = b;
        __syncthreads();
        for (int w = 0; w < G; ++w) b = max(b, part[(wv & -G) + w]);
      }
      if (i < rows) {
        float f, s;
        int8_factor(__uint_as_float(b), f, s);
        uint8_t* to = codes + i * (Kp + 16);
        if (held) {
#pragma unroll
          for (int u = 0; u < HELD; ++u)
            if (first() + u * step < Kp) *reinterpret_cast<uint2*>(to + first() + u * step) = int8_codes8(v[u], f);
        }
        for (int c = first() + (held ? HELD * step : 0); c < Kp; c += step)
          *reinterpret_cast<uint2*>(to + c) = int8_codes8(piece(i, c), f);
        if (lane == 0 && (wv & (G - 1)) == 0) scales[i] = s;
      }
      if (G > 1) break;
    }
    __syncthreads();
  }
};

template <int NT, int R, int KS, int D, Int8Mode MODE, bool BLOCK>
__global__ __launch_bounds__(64 * KS) void int8_stream_kernel(Int8Args a) {
  static_assert(!BLOCK || NT == 1, "one token fragment");
  extern __shared__ __align__(16) uint8_t quantized[];  // BLOCK
  __shared__ float qscale[16];
  __shared__ uint32_t qmax[16];
  __shared__ i32x4 red[KS][R * NT][64];
  __shared__ int cum[MODE == INT8_DENSE ? 1 : 1025];
  const int kRows = BLOCK ? a.cap : 16 * NT;
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int Kp = int8_pad(a.K), KB = Kp / 128;
  // weight rows of one item: DENSE / DOWN 16 R consecutive ones; GATE_UP 8 R gate rows and the 8 R up rows
  constexpr int kItemN = MODE == INT8_GATE_UP ? 8 * R : 16 * R;
  const int nspan = MODE == INT8_GATE_UP ? a.N / 2 : a.N;
  const int nitems = (nspan + kItemN - 1) / kItemN;

  int total;  // token tiles
  if constexpr (MODE == INT8_DENSE) {
    total = (a.rows + kRows - 1) / kRows;
  } else {
    // prefix of the experts' token tiles: a scan over chunks of the block's size
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
    if constexpr (MODE == INT8_DENSE) {
      r0 = tile * kRows;
      rend = min(a.rows, r0 + kRows);
    } else {
      int lo = 0, hi = a.E - 1;  // the expert with cum[e] <= tile < cum[e + 1]
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid + 1] > tile) hi = mid;
        else lo = mid + 1;
      }
      e = lo;
      r0 = max(0, a.offsets[e]) + (tile - cum[e]) * kRows;
      rend = min(min(a.offsets[e + 1], a.rows), r0 + kRows);
    }
    auto source = [&](int row) { return MODE == INT8_GATE_UP ? a.pairs[row] / a.k : row; };
    // weight fragments of this lane; rows past the end repeat the last one (results dropped)
    auto first_row = [&](int f) {
      return MODE == INT8_GATE_UP ? (f < R / 2 ? 0 : nspan) + slab * kItemN + 16 * (f % (R / 2)) : slab * kItemN + 16 * f;
    };
    const int8_t* wrow[R];
#pragma unroll
    for (int f = 0; f < R; ++f) wrow[f] = a.w + ((size_t)e * a.N + min(first_row(f) + r, a.N - 1)) * a.K + 16 * q;
    const int8_t* qrow[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if constexpr (BLOCK) qrow[t] = reinterpret_cast<const int8_t*>(quantized) + min(r, rend - r0 - 1) * (Kp + 16) + 16 * q;
      else qrow[t] = a.xq + (size_t)source(min(r0 + 16 * t + r, rend - 1)) * Kp + 16 * q;
    }
    i32x4 acc[R][NT];
#pragma unroll
    for (int f = 0; f < R; ++f)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[f][t] = i32x4{0, 0, 0, 0};

    struct Step {
      u32x4 w[R][2];
      u32x4 x[BLOCK ? 1 : NT][2];
    };
    // Loads without branches around them (each would end in a wait for everything in flight): steps past the last one
    // repeat it, and pieces past the end of a ragged K are the step's first (their tokens' codes are zero).
    auto load = [&](Step& st, int step) {
      const int kb = min(step, KB - 1);
      const int lo = kb * 128 + 16 * q < a.K ? 0 : -16 * q, hi = kb * 128 + 64 + 16 * q < a.K ? 64 : -16 * q;
#pragma unroll
      for (int f = 0; f < R; ++f) {
        const int8_t* p = wrow[f] + (size_t)kb * 128;
        st.w[f][0] = *reinterpret_cast<const u32x4*>(p + lo);
        st.w[f][1] = *reinterpret_cast<const u32x4*>(p + hi);
      }
      if constexpr (!BLOCK) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const u32x4* p = reinterpret_cast<const u32x4*>(qrow[t] + (size_t)kb * 128);
          st.x[t][0] = p[0];
          st.x[t][1] = p[4];
        }
      }
    };
    auto compute = [&](const Step& st, int kb) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        u32x4 lo, hi;
        if constexpr (BLOCK) {
          lo = *reinterpret_cast<const u32x4*>(qrow[t] + kb * 128);
          hi = *reinterpret_cast<const u32x4*>(qrow[t] + kb * 128 + 64);
        } else {
          lo = st.x[t][0], hi = st.x[t][1];
        }
#pragma unroll
        for (int f = 0; f < R; ++f) {
          acc[f][t] = int8_mfma(st.w[f][0], lo, acc[f][t]);
          acc[f][t] = int8_mfma(st.w[f][1], hi, acc[f][t]);
        }
      }
    };
    auto rows_of = [&](int i) { return a.x + (size_t)source(r0 + i) * a.ldx; };
    BlockQuantizer<KS, BLOCK ? 4 : 1, decltype(rows_of)> quantizer(rend - r0, a.K, wv, lane, rows_of);
    if constexpr (BLOCK) {
      quantizer.load();
      asm volatile("" ::: "memory");  // before the weights
    }
    // this wave's steps wv, wv + KS, ...: D of them in flight
    const int n = wv < KB ? (KB - wv + KS - 1) / KS : 0;
    Step st[D];
    if (n > 0) {
#pragma unroll
      for (int u = 0; u < D; ++u)
        if (u == 0 || u < n) load(st[u], wv + u * KS);
    }
    if constexpr (BLOCK) quantizer.store(quantized, qscale, qmax);  // while the first weights are on their way
    if (n > 0) {
      int i = 0;
      for (; i + 2 * D <= n; i += D) {
#pragma unroll
        for (int u = 0; u < D; ++u) {
          compute(st[u], wv + (i + u) * KS);
          load(st[u], wv + (i + u + D) * KS);
        }
      }
      // fewer than 2 D steps are left, the first D of them loaded
#pragma unroll
      for (int u = 0; u < D; ++u)
        if (i + u < n) {
          compute(st[u], wv + (i + u) * KS);
          if (i + u + D < n) load(st[u], wv + (i + u + D) * KS);
        }
#pragma unroll
      for (int u = 0; u < D - 1; ++u)
        if (i + u + D < n) compute(st[u], wv + (i + u + D) * KS);
    }
    // accumulator (f, t) element i of lane r + 16 q is weight row 16 f + 4 q + i, token 16 t + r
#pragma unroll
    for (int f = 0; f < R; ++f)
#pragma unroll
      for (int t = 0; t < NT; ++t) red[wv][f * NT + t][lane] = acc[f][t];
    __syncthreads();
    constexpr int kUnits = MODE == INT8_GATE_UP ? R / 2 * NT : R * NT;
    for (int u = wv; u < kUnits; u += KS) {
      auto sum = [&](int j) {
        i32x4 v = red[0][j][lane];
#pragma unroll
        for (int i = 1; i < KS; ++i) v += red[i][j][lane];
        return v;
      };
      const int f = u / NT, t = u % NT, row = r0 + 16 * t + r;
      if (row < rend) {
        float sx;
        if constexpr (BLOCK) sx = qscale[r];
        else sx = a.xs[source(row)];
        auto values = [&](int j, int n0) {
          const i32x4 c = sum(j);
          f32x4 v;
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = value(c[i], sx, a.wsc[(size_t)e * a.N + min(n0 + 4 * q + i, a.N - 1)]);
          return v;
        };
        f32x4 v = values(u, first_row(f));
        if constexpr (MODE == INT8_GATE_UP) {
          const f32x4 up = values(u + R / 2 * NT, first_row(f + R / 2));
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = swiglu(v[i], up[i], a.limit);
        }
        const size_t orow = MODE == INT8_DOWN ? a.pairs[row] : row;
        store4(a.out + orow * (size_t)a.ldo, slab * kItemN + 16 * f + 4 * q, nspan, v);
      }
    }
    __syncthreads();  // the sums are read before the next item's overwrite them
  }
}

// Grouped token tiles of `per` rows, at most: an expert's last one need not be full.
long long most_tiles(const Int8Args& a, int per) {
  return min((long long)a.rows, (long long)(a.rows + per - 1) / per + min(a.rows, a.E));
}

template <int NT, int R, int KS, int D, Int8Mode MODE, bool BLOCK>
hipError_t launch_one(const Int8Args& a, int cus, hipStream_t s) {
  const int span = MODE == INT8_GATE_UP ? a.N / 2 : a.N, per = MODE == INT8_GATE_UP ? 8 * R : 16 * R;
  const long long slabs = (span + per - 1) / per;
  const int kRows = BLOCK ? a.cap : 16 * NT;
  const long long tiles = MODE == INT8_DENSE ? (a.rows + kRows - 1) / kRows : most_tiles(a, kRows);
  long long grid = tiles * slabs;
  // grouped (the number of items is known on the device only): as many as run at once
  const long long most = MODE != INT8_DENSE ? 3LL * cus : 1LL << 20;
  if (grid > most) grid = most;
  size_t bytes = 0;
  if constexpr (BLOCK) {
    bytes = block_lds(a.cap, a.K);
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&int8_stream_kernel<NT, R, KS, D, MODE, BLOCK>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, kBlockLds);
    if (e != hipSuccess) return e;
  }
  int8_stream_kernel<NT, R, KS, D, MODE, BLOCK><<<dim3((unsigned)grid), dim3(64 * KS), bytes, s>>>(a);
  return hipGetLastError();
}

// Items of 64 weight rows of a grouped product whose tiles hold `per` rows, at most.
long long items64(Int8Mode mode, const Int8Args& a, int per) {
  return most_tiles(a, per) * (mode == INT8_GATE_UP ? (a.N / 2 + 31) / 32 : (a.N + 63) / 64);
}

template <Int8Mode MODE>
hipError_t launch_grouped(const Int8Args& a, int cus, hipStream_t s) {
  // quantising: items of 32 weight rows and more steps in flight while there are few
  if (a.cap > 0)
    return items64(MODE, a, a.cap) <= 3LL * cus / 2 ? launch_one<1, 2, 4, 4, MODE, true>(a, cus, s)
                                                    : launch_one<1, 4, 4, 3, MODE, true>(a, cus, s);
  return a.rows <= 16LL * a.E ? launch_one<1, 4, 4, 2, MODE, false>(a, cus, s) : launch_one<2, 4, 4, 2, MODE, false>(a, cus, s);
}

}  // namespace

// Dense: quantising in every block of the product pays while it is little work (4 rows of 2816 x 4096 6.4 us, codes 5.7
// behind a launch of 3.5; 8 rows 6.0 behind it).
bool int8_decode_fits(int M, int K) { return M <= 16 && M * (int8_pad(K) / 128) <= 224; }

// Grouped: up to 3 items a compute unit.  Blocks that quantise run two at a time there (211 registers), those that read
// codes three, so past 2 items the first have a second round, whose rows are quantised with no weights on their way beside
// it; the launch for the codes costs about as much (us, quantising against codes and their launch: gate / up of H 7168, I
// 2048, one token, top-8, 512 items 46.6 and 42.3 + 4.6, top-9, 576 items 62.3 and 56.1 + 4.7, top-12, 768 items 67.3 and
// 61.1 + 4.8, two tokens, 1024 items 101 and 80.7; of H 4096, I 1408, top-6, two tokens, 528 items 33.3 and 30.3 + 4.7;
// down of the first, top-6, 672 items 21.9 and 18.2 + 4.7, of the second, 768 items 17.7 and 13.9 + 4.7).  While an
// expert's rows are little work (gate / up of H 4096 and 2 experts of I 1024, 8 tokens 13.5 against 12.6 and 2.7, 14 tokens
// 20.4 against 12.6 and 3.0; one of I 4096, 9 tokens 23.8 against 12.6 and 8.0).  And while the codes take 64 KB (two
// blocks' fit a CU's LDS up to 59, beside the sums and offsets).  0: codes.
int int8_block_rows(Int8Mode mode, const Int8Args& a, int T, int cus) {
  const int cap = min(T, 16), rows = min(cap, a.rows / a.E + 1);
  const bool little = rows * (int8_pad(a.K) / 128) < 200;
  return little && block_lds(cap, a.K) <= kBlockLds && items64(mode, a, cap) <= 3LL * cus ? cap : 0;
}

hipError_t launch_int8_stream(Int8Mode mode, const Int8Args& a, int cus, hipStream_t s) {
  switch (mode) {
    case INT8_DENSE:
      if (!a.xq) return launch_one<1, 1, 8, 2, INT8_DENSE, true>(a, cus, s);
      if (a.rows > 16) return launch_one<2, 1, 16, 2, INT8_DENSE, false>(a, cus, s);
      return a.K >= 32 * 128 ? launch_one<1, 1, 16, 2, INT8_DENSE, false>(a, cus, s)
                             : launch_one<1, 2, 8, 2, INT8_DENSE, false>(a, cus, s);
    case INT8_GATE_UP: return launch_grouped<INT8_GATE_UP>(a, cus, s);
    default: return launch_grouped<INT8_DOWN>(a, cus, s);
  }
}

}  // namespace moe
