// Streaming product on block-128 fp8 weights: few token rows per weight
// matrix (decoding), so the time is that of reading the weights once.
//
// Item = (token tile, R fragments of 16 weight rows).  The block's KS waves
// take the 128-wide K blocks in turn; a wave reads its weight fragment straight
// from the row-major codes into the operand registers (lane r + 16 q: row r,
// bytes [16 q, 16 q + 16) and [64 + 16 q, + 16) of the block; which 32 of the
// 128 bytes a lane holds does not matter, since tokens use the same order).
// The two loads of a line are ordinary ones: as non-temporal ones they fetched
// the line's halves one by one (T = 1 experts, H 7168, I 2048: 76.5 us against
// 72.2; M = 1, 18432 x 7168: 28.6 against 25.2, 5.2 TB/s).  Partial sums of the
// waves meet in LDS in wave order (the same bits every run).  More bytes in
// flight than here (more waves, or more steps per wave) made it slower.
#include "moe_fp8.h"

namespace moe {
namespace {

// Columns n .. n + 3 of an output row that ends at N.
__device__ __forceinline__ void store4(uint16_t* row, int n, int N, const f32x4& v) {
  uint16_t* o = row + n;
  const uint32_t b0 = f32_to_bf16(v[0]), b1 = f32_to_bf16(v[1]), b2 = f32_to_bf16(v[2]), b3 = f32_to_bf16(v[3]);
  if (n + 4 <= N && ((uintptr_t)o & 7) == 0) {
    *reinterpret_cast<uint2*>(o) = make_uint2(b0 | b1 << 16, b2 | b3 << 16);
  } else {
    if (n < N) o[0] = (uint16_t)b0;
    if (n + 1 < N) o[1] = (uint16_t)b1;
    if (n + 2 < N) o[2] = (uint16_t)b2;
    if (n + 3 < N) o[3] = (uint16_t)b3;
  }
}

// Where a token's codes come from.  SELF: every wave quantises what it multiplies (the four lanes of a token share a
// block's 128 values, so the maximum is two exchanges away).  CODES: from memory.  BLOCK: the block quantises its item's
// rows into LDS while the first weights are on their way (NT = 1, `cap` <= 16 rows per tile; dynamic LDS of
// block_lds()): the waves' steps are then little more than loads and products (T = 1 experts: 84 -> 77 us).
enum Fp8Source { SELF, CODES, BLOCK };

// Dynamic LDS of the kernels that quantise into it, at most: the limit asked for on every call (the same number, whatever
// other threads launch meanwhile).  fp8_decode_fits() and fp8_block_rows() stay below it.
constexpr int kBlockLds = 64 * 1024;
__host__ __device__ inline size_t block_lds(int rows, int KB) { return (size_t)KB * 64 + (size_t)rows * (KB * kFp8Blk + 16); }

// Rows `row(i)`, i < rows, of K bf16 values: codes [rows][KB 128 + 16] (row stride K + 16 bytes: the 16 rows of a fragment
// read start 4 banks apart) and scales [KB][16].  Pieces of 8 values: 16 consecutive lanes have one block of one row.
template <class F>
__device__ __forceinline__ void quantize_block(uint8_t* codes, float* scales, int rows, int KB, int K, int tid, int threads,
                                               F&& row) {
  const int stride = KB * kFp8Blk + 16;
  for (int c = tid; c < rows * KB * 16; c += threads) {
    const int blk = c >> 4, i = blk / KB, kb = blk - i * KB, col = kb * kFp8Blk + 8 * (c & 15);
    u32x4 v = {0, 0, 0, 0};
    if (col < K) v = *reinterpret_cast<const u32x4*>(row(i) + col);
    float f, s;
    fp8_factor(max_row16(bf16x2_max(fp8_amax8(v, kFp8TinyBits))), f, s);
    *reinterpret_cast<uint2*>(codes + i * stride + col) = fp8_codes8(v, f);
    if ((c & 15) == 0) scales[kb * 16 + i] = s;
  }
}

template <int NT, int R, int KS, int D, Fp8Mode MODE, Fp8Source SRC>
__global__ __launch_bounds__(64 * KS) void fp8_stream_kernel(Fp8Args a) {
  static_assert(SRC != BLOCK || NT == 1, "one token fragment");
  extern __shared__ __align__(16) uint8_t quantized[];  // BLOCK
  const int kRows = SRC == BLOCK ? a.cap : 16 * NT;
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

  constexpr bool kSplit = MODE == FP8_DENSE && SRC == SELF;  // blockIdx.y: the run of K blocks
  const int run = kSplit ? (KB + a.splits - 1) / a.splits : KB, k0 = kSplit ? blockIdx.y * run : 0;
  const int k1 = min(KB, k0 + run);
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
      rend = min(min(a.offsets[e + 1], a.rows), r0 + kRows);
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
    const uint8_t* qrow[NT];  // CODES, BLOCK
    const float* srow[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if constexpr (SRC == BLOCK) {
        const int i = min(r, rend - r0 - 1);
        qrow[t] = quantized + KB * 64 + i * (KB * kFp8Blk + 16) + 16 * q;
        srow[t] = reinterpret_cast<const float*>(quantized) + i;
        break;
      }
      const int row = r0 + 16 * t + r;
      int src = min(row, rend - 1);
      if constexpr (MODE == FP8_GATE_UP) src = a.pairs[src] / a.k;
      if constexpr (SRC == CODES) {
        qrow[t] = a.xq + (size_t)src * ((size_t)KB * kFp8Blk) + 16 * q;
        srow[t] = a.xs + src;
      } else {
        xrow[t] = a.x + (size_t)src * a.ldx + 16 * q;
      }
    }
    f32x4 acc[R][NT];
#pragma unroll
    for (int f = 0; f < R; ++f)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[f][t] = f32x4{0.f, 0.f, 0.f, 0.f};

    struct Step {
      u32x4 w[R][2];
      u32x4 x[NT][SRC == SELF ? 4 : SRC == CODES ? 2 : 1];
      float s[R], sx[NT];
    };
    // Loads without branches around them (each would end in a wait for everything in flight): rows past the end
    // repeat the last one, steps past the last one the last one, and pieces past the end of a ragged K the first
    // piece of the block, cleared in the tokens before they count.
    auto load = [&](Step& st, int step) {
      const int kb = min(step, KB - 1);
      const int lo = kb * kFp8Blk + 16 * q < a.K ? 0 : -16 * q, hi = kb * kFp8Blk + 64 + 16 * q < a.K ? 64 : -16 * q;
#pragma unroll
      for (int f = 0; f < R; ++f) {
        const uint8_t* p = wrow[f] + (size_t)kb * kFp8Blk;
        st.w[f][0] = *reinterpret_cast<const u32x4*>(p + lo);
        st.w[f][1] = *reinterpret_cast<const u32x4*>(p + hi);
        st.s[f] = wsc[f][kb];
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if constexpr (SRC == CODES) {
          const u32x4* p = reinterpret_cast<const u32x4*>(qrow[t] + (size_t)kb * kFp8Blk);
          st.x[t][0] = p[0];
          st.x[t][1] = p[4];
          st.sx[t] = srow[t][(size_t)kb * a.xrows];
        } else if constexpr (SRC == SELF) {
          const u32x4* p = reinterpret_cast<const u32x4*>(xrow[t] + (size_t)kb * kFp8Blk + lo);
          const u32x4* p2 = reinterpret_cast<const u32x4*>(xrow[t] + (size_t)kb * kFp8Blk + hi);
          st.x[t][0] = p[0];
          st.x[t][1] = p[1];
          st.x[t][2] = p2[0];
          st.x[t][3] = p2[1];
        }
      }
    };
    auto clear_ragged = [&](Step& st, int kb) {
      const bool lo = kb * kFp8Blk + 16 * q < a.K, hi = kb * kFp8Blk + 64 + 16 * q < a.K;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if constexpr (SRC == SELF) st.x[t][j][i] = (j < 2 ? lo : hi) ? st.x[t][j][i] : 0u;
    };
    auto compute = [&](Step& st, int kb) {
      if (SRC == SELF && kb * kFp8Blk + kFp8Blk > a.K) clear_ragged(st, kb);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        i32x8 b;
        float sx;
        if constexpr (SRC == BLOCK) {
          const u32x4 lo = *reinterpret_cast<const u32x4*>(qrow[t] + kb * kFp8Blk);
          const u32x4 hi = *reinterpret_cast<const u32x4*>(qrow[t] + kb * kFp8Blk + 64);
          b = i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
          sx = srow[t][kb * 16];
        } else if constexpr (SRC == CODES) {
          const u32x4 lo = st.x[t][0], hi = st.x[t][1];
          b = i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
          sx = st.sx[t];
        } else {
          uint32_t m = kFp8TinyBits;
#pragma unroll
          for (int j = 0; j < 4; ++j) m = fp8_amax8(st.x[t][j], m);
          float f;
          fp8_factor(max_rows(bf16x2_max(m)), f, sx);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint2 c = fp8_codes8(st.x[t][j], f);
            b[2 * j] = (int)c.x;
            b[2 * j + 1] = (int)c.y;
          }
        }
        // The gate and up sums meet the next quantiser, where an error moves values over borders between codes and, in a
        // block's largest value, the whole block; the fp8 instruction cuts products (13 bits below the largest of 8),
        // bf16 products do not, and there is time for them (T = 1, H 4096: an error of 3.5e-3 against 64 bits down to
        // 1.7e-3, that of the output's rounding; T = 1 of 256 experts 72.4 us against 72.6).
        constexpr bool kExact = MODE == FP8_GATE_UP;
        Bf16Frag bx;
        if constexpr (kExact) bx = bf16_frag(b);
#pragma unroll
        for (int fr = 0; fr < R; ++fr) {
          const u32x4 lo = st.w[fr][0], hi = st.w[fr][1];
          const i32x8 aw = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
          const f32x4 z = kExact ? bf16_mfma(bf16_frag(aw), bx) : fp8_mfma(aw, b);
          const float sc = sx * st.s[fr];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[fr][t][i] = fmaf(z[i], sc, acc[fr][t][i]);
        }
      }
    };
    // this wave's steps k0 + wv, k0 + wv + KS, ...: D of them in flight
    const int n = wv < k1 - k0 ? (k1 - k0 - wv + KS - 1) / KS : 0, at = k0 + wv;
    Step st[D];
    if (n > 0) {
#pragma unroll
      for (int u = 0; u < D; ++u)
        if (u == 0 || u < n) load(st[u], at + u * KS);
    }
    if constexpr (SRC == BLOCK) {  // while the first weights are on their way
      quantize_block(quantized + KB * 64, reinterpret_cast<float*>(quantized), rend - r0, KB, a.K, tid, 64 * KS,
                     [&](int i) {
                       const int src = MODE == FP8_GATE_UP ? a.pairs[r0 + i] / a.k : r0 + i;
                       return a.x + (size_t)src * a.ldx;
                     });
      __syncthreads();
    }
    if (n > 0) {
      int i = 0;
      for (; i + 2 * D <= n; i += D) {
#pragma unroll
        for (int u = 0; u < D; ++u) {
          compute(st[u], at + (i + u) * KS);
          load(st[u], at + (i + u + D) * KS);
        }
      }
      // fewer than 2 D steps are left, the first D of them loaded
#pragma unroll
      for (int u = 0; u < D; ++u)
        if (i + u < n) {
          compute(st[u], at + (i + u) * KS);
          if (i + u + D < n) load(st[u], at + (i + u + D) * KS);
        }
#pragma unroll
      for (int u = 0; u < D - 1; ++u)
        if (i + u + D < n) compute(st[u], at + (i + u + D) * KS);
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
        if constexpr (kSplit) {
          const int ldp = (a.N + 15) / 16 * 16;
          *reinterpret_cast<f32x4*>(a.part + ((size_t)blockIdx.y * a.rows + row) * ldp + slab * kItemN + 16 * f + 4 * q) = v;
          continue;
        }
        const size_t orow = MODE == FP8_DOWN ? a.pairs[row] : row;
        store4(a.out + orow * (size_t)a.ldo, slab * kItemN + 16 * f + 4 * q, nspan, v);
      }
    }
    __syncthreads();  // the sums are read before the next item's overwrite them
  }
}

// Decoding through one matrix: up to 16 token rows, weights read once, all rows quantised into LDS by every block.
// Bound by the latency of a launch and of one trip to memory (1 x 7168 x 2048: 5.0 us, 6.0 a call).
template <int R, int KS, int D>
__global__ __launch_bounds__(64 * KS) void fp8_decode_kernel(Fp8Args a) {
  extern __shared__ __align__(16) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int KB = (a.K + kFp8Blk - 1) / kFp8Blk, stride = KB * kFp8Blk + 16;
  float* scales = reinterpret_cast<float*>(lds);                    // [KB][16]
  uint8_t* codes = lds + KB * 64;                                   // [rows][stride]
  f32x4* red = reinterpret_cast<f32x4*>(codes + (size_t)a.rows * stride);  // [KS][R][64]
  const int first = blockIdx.x * 16 * R;
  const uint8_t* wrow[R];
  const float* wsc[R];
#pragma unroll
  for (int f = 0; f < R; ++f) {
    wrow[f] = a.w + (size_t)min(first + 16 * f + r, a.N - 1) * a.K + 16 * q;
    wsc[f] = a.wsc + (size_t)(min(first + 16 * f, a.N - 1) / kFp8Blk) * KB;
  }
  struct Step {
    u32x4 w[R][2];
    float s[R];
  };
  auto load = [&](Step& st, int step) {
    const int kb = min(step, KB - 1);
    const int lo = kb * kFp8Blk + 16 * q < a.K ? 0 : -16 * q, hi = kb * kFp8Blk + 64 + 16 * q < a.K ? 64 : -16 * q;
#pragma unroll
    for (int f = 0; f < R; ++f) {
      const uint8_t* p = wrow[f] + (size_t)kb * kFp8Blk;
      st.w[f][0] = *reinterpret_cast<const u32x4*>(p + lo);
      st.w[f][1] = *reinterpret_cast<const u32x4*>(p + hi);
      st.s[f] = wsc[f][kb];
    }
  };
  const int n = wv < KB ? (KB - wv + KS - 1) / KS : 0;
  Step st[D];
#pragma unroll
  for (int u = 0; u < D; ++u) load(st[u], wv + u * KS);
  quantize_block(codes, scales, a.rows, KB, a.K, tid, 64 * KS, [&](int i) { return a.x + (size_t)i * a.ldx; });
  __syncthreads();
  f32x4 acc[R];
#pragma unroll
  for (int f = 0; f < R; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int rr = min(r, a.rows - 1);
  const uint8_t* xrow = codes + rr * stride + 16 * q;
  auto compute = [&](const Step& s, int kb) {
    const u32x4 lo = *reinterpret_cast<const u32x4*>(xrow + kb * kFp8Blk);
    const u32x4 hi = *reinterpret_cast<const u32x4*>(xrow + kb * kFp8Blk + 64);
    const float sx = scales[kb * 16 + rr];
    const i32x8 b = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
#pragma unroll
    for (int f = 0; f < R; ++f) {
      const u32x4 wl = s.w[f][0], wh = s.w[f][1];
      const i32x8 aw = {(int)wl.x, (int)wl.y, (int)wl.z, (int)wl.w, (int)wh.x, (int)wh.y, (int)wh.z, (int)wh.w};
      const f32x4 z = fp8_mfma(aw, b);
      const float sc = sx * s.s[f];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[f][i] = fmaf(z[i], sc, acc[f][i]);
    }
  };
  int i = 0;
  for (; i + 2 * D <= n; i += D) {
#pragma unroll
    for (int u = 0; u < D; ++u) {
      compute(st[u], wv + (i + u) * KS);
      load(st[u], wv + (i + u + D) * KS);
    }
  }
#pragma unroll
  for (int u = 0; u < D; ++u)
    if (i + u < n) {
      compute(st[u], wv + (i + u) * KS);
      if (i + u + D < n) load(st[u], wv + (i + u + D) * KS);
    }
#pragma unroll
  for (int u = 0; u < D - 1; ++u)
    if (i + u + D < n) compute(st[u], wv + (i + u + D) * KS);
#pragma unroll
  for (int f = 0; f < R; ++f) red[(wv * R + f) * 64 + lane] = acc[f];
  __syncthreads();
  if (wv < R) {
    f32x4 v = red[wv * 64 + lane];
#pragma unroll
    for (int j = 1; j < KS; ++j) v += red[(j * R + wv) * 64 + lane];
    if (r < a.rows) store4(a.out + (size_t)r * a.ldo, first + 16 * wv + 4 * q, a.N, v);
  }
}

// out = the runs' sums, added in order: a thread per four columns.
__global__ __launch_bounds__(256) void fp8_join_kernel(Fp8Args a) {
  const int quads = (a.N + 15) / 16 * 4, c = blockIdx.x * 256 + threadIdx.x, row = c / quads, n = 4 * (c - row * quads);
  if (row >= a.rows) return;
  const f32x4* p = reinterpret_cast<const f32x4*>(a.part) + c;
  f32x4 v = p[0];
#pragma unroll 8
  for (int i = 1; i < a.splits; ++i) v += p[(size_t)i * a.rows * quads];
  store4(a.out + (size_t)row * a.ldo, n, a.N, v);
}

// Grouped token tiles of `per` rows, at most: an expert's last one need not be full.
long long most_tiles(const Fp8Args& a, int per) {
  return min((long long)a.rows, (long long)(a.rows + per - 1) / per + min(a.rows, a.E));
}

template <int NT, int R, int KS, int D, Fp8Mode MODE, Fp8Source SRC>
hipError_t launch_one(const Fp8Args& a, int cus, hipStream_t s) {
  const int span = MODE == FP8_GATE_UP ? a.N / 2 : a.N, per = MODE == FP8_GATE_UP ? 8 * R : 16 * R;
  const long long slabs = (span + per - 1) / per;
  const int kRows = SRC == BLOCK ? a.cap : 16 * NT;
  const long long tiles = MODE == FP8_DENSE ? (a.rows + kRows - 1) / kRows : most_tiles(a, kRows);
  long long grid = tiles * slabs;
  // dense: a block per item; grouped (the number of items is known on the device only): as many as run at once
  if (MODE != FP8_DENSE && grid > 3LL * cus) grid = 3LL * cus;
  const int runs = MODE == FP8_DENSE && SRC == SELF ? a.splits : 1;
  size_t bytes = 0;
  if constexpr (SRC == BLOCK) {
    bytes = block_lds(a.cap, (a.K + kFp8Blk - 1) / kFp8Blk);
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&fp8_stream_kernel<NT, R, KS, D, MODE, SRC>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, kBlockLds);
    if (e != hipSuccess) return e;
  }
  fp8_stream_kernel<NT, R, KS, D, MODE, SRC><<<dim3((unsigned)grid, runs), dim3(64 * KS), bytes, s>>>(a);
  return hipGetLastError();
}

template <int R, int KS>
size_t decode_lds(int M, int K) {
  const size_t KB = (K + kFp8Blk - 1) / kFp8Blk;
  return KB * 64 + M * (KB * kFp8Blk + 16) + KS * R * 1024;
}
template <int R, int KS, int D>
hipError_t launch_decode(const Fp8Args& a, hipStream_t s) {
  const size_t bytes = decode_lds<R, KS>(a.rows, a.K);
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&fp8_decode_kernel<R, KS, D>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, kBlockLds);
  if (e != hipSuccess) return e;
  fp8_decode_kernel<R, KS, D><<<dim3((a.N + 16 * R - 1) / (16 * R)), dim3(64 * KS), bytes, s>>>(a);
  return hipGetLastError();
}

template <Fp8Mode MODE>
hipError_t launch_grouped(const Fp8Args& a, int cus, hipStream_t s) {
  // Items of 64 weight rows; GATE_UP, whose fragments as bf16 take their registers, of 32 (4 tokens, H 7168, I 2048, 256
  // experts, top-8: 253 us against 281).  While there are few items, all of 32 and more steps in flight: a long K needs
  // it (one token, without / with: H 4096, I 14336, top-2 78 / 70 us; H 2048, I 8192, top-1 31 / 24.5; H 1024, I 4096,
  // top-2 19.8 / 16.4), a short one loses a little (H 4096, I 1408, top-6 30.1 / 30.4; I 1536, top-8 36.9 / 40.1; 4
  // tokens of H 7168, I 256, top-8 42.5 / 44.2).
  constexpr int R = MODE == FP8_GATE_UP ? 2 : 4;
  if (a.cap > 0) {
    const long long slabs = MODE == FP8_GATE_UP ? (a.N / 2 + 31) / 32 : (a.N + 63) / 64;  // of 64 rows
    return most_tiles(a, a.cap) * slabs <= 3LL * cus / 2 ? launch_one<1, 2, 4, 4, MODE, BLOCK>(a, cus, s)
                                                         : launch_one<1, R, 4, 2, MODE, BLOCK>(a, cus, s);
  }
  return a.rows <= 16LL * a.E ? launch_one<1, R, 4, 2, MODE, SELF>(a, cus, s) : launch_one<2, R, 4, 2, MODE, SELF>(a, cus, s);
}

}  // namespace

// Quantising in every block of the product pays while it is little work (and the launch before it is not): 4 rows of
// 4096 x 7168 take 11.2 us this way and 11.4 us in two launches, 8 rows 14.5 and 12.3; 8 rows of 7168 x 2048 8.0 and 8.5.
bool fp8_decode_fits(int M, int K) { return M <= 16 && M * ((K + kFp8Blk - 1) / kFp8Blk) <= 224; }

// Few weight rows and a long K (a low-rank projection): one block per 16 weight rows leaves most of the GPU idle and
// every wave several trips to memory.  Then K is split over blocks too, runs of at least 8 blocks of 128 (one per wave),
// as many as fill the compute units; the tokens are quantised where they are used, and a second launch joins the runs
// (17 rows of 576 x 7168: 8.6 us against 13.3 for quantiser and one block per slab; 64 rows 12.9 against 16.1 for the
// tiled kernel; 24 of 1024 x 4096 8.1 against 10.3).  One row is faster in one launch (1 x 1024 x 4096: 5.7 us against 6.5).
constexpr int kSplitRows = 128, kSplitRun = 8, kSplitBlocks = 256;

int fp8_splits(int M, int N, int K) {
  const int KB = (K + kFp8Blk - 1) / kFp8Blk, most = (KB + kSplitRun - 1) / kSplitRun;
  if (M > kSplitRows || M * KB <= 64) return 1;
  const int blocks = (N + 15) / 16 * ((M + 31) / 32);
  const int n = min(most, kSplitBlocks / blocks);
  if (n < 2) return 1;
  const int run = (KB + n - 1) / n;
  return (KB + run - 1) / run;  // no empty run
}

size_t fp8_split_bytes(int max_M, int N, int K) {
  size_t n = 0;
  for (int M = 32; M < max_M + 32 && M <= kSplitRows; M += 32) {  // fewer rows of as many token tiles need less
    const int rows = min(M, max_M), splits = fp8_splits(rows, N, K);
    if (splits > 1) n = max(n, (size_t)splits * rows * ((N + 15) / 16 * 16) * sizeof(float));
  }
  return n;
}

// A tile holds an expert's rows of up to 16 tokens where two blocks' codes fit a CU's LDS.
int fp8_block_rows(int T, int K) {
  const int cap = min(T, 16);
  return block_lds(cap, (K + kFp8Blk - 1) / kFp8Blk) <= kBlockLds ? cap : 0;
}

hipError_t launch_fp8_split(const Fp8Args& a, hipStream_t s) {
  const hipError_t e = a.rows <= 16 ? launch_one<1, 1, 8, 2, FP8_DENSE, SELF>(a, 0, s)
                                    : launch_one<2, 1, 8, 2, FP8_DENSE, SELF>(a, 0, s);
  if (e != hipSuccess) return e;
  const long long quads = (long long)a.rows * ((a.N + 15) / 16 * 4);
  fp8_join_kernel<<<dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_fp8_stream(Fp8Mode mode, const Fp8Args& a, int cus, hipStream_t s) {
  switch (mode) {
    case FP8_DENSE:
      if (!a.xq) return launch_decode<1, 8, 2>(a, s);
      // codes, up to 32 rows: 16 waves share a long K (16 x 4096 x 7168: 13.8 us, 8 waves on 32 rows of weights
      // 17.9), 8 a short one (16 x 7168 x 2048: 8.7 us against 10.8)
      if (a.rows > 16) return launch_one<2, 1, 16, 2, FP8_DENSE, CODES>(a, cus, s);
      return a.K >= 32 * kFp8Blk ? launch_one<1, 1, 16, 2, FP8_DENSE, CODES>(a, cus, s)
                                 : launch_one<1, 2, 8, 2, FP8_DENSE, CODES>(a, cus, s);
    case FP8_GATE_UP: return launch_grouped<FP8_GATE_UP>(a, cus, s);
    default: return launch_grouped<FP8_DOWN>(a, cus, s);
  }
}

}  // namespace moe
