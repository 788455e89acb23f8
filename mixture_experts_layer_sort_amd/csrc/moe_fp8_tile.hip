// Tiled product on block-128 fp8 weights: many token rows per weight matrix
// (prompts), bound by the matrix unit.
//
// Block tile = BN = 16 RF WR weight rows x BT = 16 TF WT tokens, by WR x WT
// waves of RF x TF fragments each; step = one K block of 128, which is one
// 16 x 16 x 128 matrix instruction per fragment, started from zero and added
// to the fp32 accumulator with the block's scale (one number per lane: a lane's
// four results belong to one token).  The multiply-adds (4 per instruction, half
// of its issue time) run while another wave of the same SIMD feeds the matrix
// unit: two waves per SIMD.
//
// Both operands reach LDS by 16-byte direct global->LDS loads (buffer form),
// NS stages of 128-byte rows; piece p of row r lies at slot p ^ (r & 7), which
// makes the fragment reads (16 rows, one 16-byte piece each per quarter wave)
// conflict-free.  One barrier per step: a wave waits for its own loads of the
// step, the barrier says that everyone's have landed and that the stage before
// is free, then the next loads are issued and the step is computed.
#include "moe_fp8.h"

namespace moe {
namespace {

template <int WR_, int WT_, int RF_, int TF_, int NS_>
struct TileShape {
  static constexpr int WR = WR_, WT = WT_, RF = RF_, TF = TF_, NS = NS_;
  static constexpr int NW = WR * WT, BN = 16 * RF * WR, BT = 16 * TF * WT;
  static constexpr int kA = BN * 128, kB = BT * 128, kS = BT * 4, kStage = kA + kB + kS;
  static constexpr int LA = BN / 8 / NW, LB = BT / 8 / NW;  // 16-byte loads per wave and stage
  static constexpr int kOutBytes = BT * BN * 2;             // bf16 output tile (shares the stages' memory)
  static constexpr int kLds = NS * kStage > kOutBytes ? NS * kStage : kOutBytes;
  static_assert(BN / 8 % NW == 0 && BT / 8 % NW == 0 && BT / NW <= 64, "loads are dealt evenly");
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, 0x7FFFFFFF, 0x00020000);
}
__device__ __forceinline__ void load_lds16(const void* base, uint32_t off, void* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc_of(base), (__attribute__((address_space(3))) void*)lds, 16, off, 0, 0,
                                           0);
}
__device__ __forceinline__ void load_lds4(const void* base, uint32_t off, void* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc_of(base), (__attribute__((address_space(3))) void*)lds, 4, off, 0, 0,
                                           0);
}

// Wait until at most N of this wave's vector-memory operations are
// outstanding (and its LDS operations are done), then the block's barrier.
template <int N>
__device__ __forceinline__ void wait_barrier() {
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0x0 << 8));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <class S, Fp8Mode MODE>
__global__ __launch_bounds__(64 * S::NW) void fp8_tile_kernel(Fp8Args a, int band) {
  extern __shared__ __align__(256) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int wr = wv % S::WR, wt = wv / S::WR;
  const int KB = (a.K + kFp8Blk - 1) / kFp8Blk, Kp = KB * kFp8Blk;
  const int nspan = MODE == FP8_GATE_UP ? a.N / 2 : a.N;                // output columns
  constexpr int kSpan = MODE == FP8_GATE_UP ? S::BN / 2 : S::BN;        // per tile
  const int NB = (nspan + kSpan - 1) / kSpan;
  const int MT = MODE == FP8_DENSE ? (a.rows + S::BT - 1) / S::BT : *a.ntiles;

  // Blocks go round the 8 XCDs: XCD x takes a contiguous share of the tile
  // order (bands of token tiles, weight-block-major inside a band), so the
  // tiles that run together on one L2 share their operands.
  const int total = MT * NB, share = (total + 7) / 8;
  const int at = (blockIdx.x & 7) * share + (blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= share || at >= total) return;
  const int bi = at / (band * NB), inb = min(band, MT - bi * band), o = at - bi * band * NB;
  const int nb = o / inb, mt = bi * band + o % inb;

  int e = 0, r0, rend;
  if constexpr (MODE == FP8_DENSE) {
    r0 = mt * S::BT;
    rend = a.rows;
  } else {
    const int2 t = a.tiles[mt];
    e = t.x;
    r0 = t.y;
    rend = a.offsets[e + 1];
  }
  const int n0 = nb * kSpan;
  // token fragments go round the WT waves, so a partly filled tile stays even: fragment tf of wave wt is
  // tokens 16 (tf WT + wt) ..; `live` of them hold tokens
  const int frags = (min(rend - r0, S::BT) + 15) >> 4;
  const int live = (frags - wt + S::WT - 1) / S::WT;

  // this lane's part of the loads: 8 rows of 8 pieces per instruction, row lane / 8, slot lane % 8
  const int lrow = lane >> 3, piece = (lane & 7) ^ lrow;
  const uint8_t* wbase;  // GATE_UP: rows [0, BN / 2) of the tile are gate rows, the rest the matching up rows
  uint32_t woff[S::LA], xoff[S::LB], soff;
  if constexpr (MODE == FP8_GATE_UP) wbase = a.w + (size_t)e * a.N * a.K;
  else wbase = a.w + ((size_t)e * a.N + n0) * a.K;
#pragma unroll
  for (int j = 0; j < S::LA; ++j) {
    const int row = 8 * (wv * S::LA + j) + lrow;
    if constexpr (MODE == FP8_GATE_UP) {
      const int n = min(n0 + row % kSpan, nspan - 1) + (row / kSpan) * nspan;
      woff[j] = (uint32_t)n * (uint32_t)a.K;
    } else {
      woff[j] = (uint32_t)min(row, a.N - 1 - n0) * (uint32_t)a.K;
    }
  }
  // GATE_UP gathers rows of xq through the pairs; the others read consecutive rows
  const uint8_t* xbase = MODE == FP8_GATE_UP ? a.xq : a.xq + (size_t)r0 * Kp;
  const float* sbase = MODE == FP8_GATE_UP ? a.xs : a.xs + r0;
#pragma unroll
  for (int j = 0; j < S::LB; ++j) {
    const int row = min(r0 + 8 * (wv * S::LB + j) + lrow, rend - 1);
    const uint32_t src = MODE == FP8_GATE_UP ? (uint32_t)(a.pairs[row] / a.k) : (uint32_t)(row - r0);
    xoff[j] = src * (uint32_t)Kp + 16 * piece;
  }
  {
    const int row = min(r0 + wv * (S::BT / S::NW) + min(lane, S::BT / S::NW - 1), rend - 1);
    soff = 4u * (MODE == FP8_GATE_UP ? (uint32_t)(a.pairs[row] / a.k) : (uint32_t)(row - r0));
  }
  auto issue = [&](int kb) {
    uint8_t* st = lds + (kb % S::NS) * S::kStage;
    // pieces past the end of a weight row (K not a multiple of 128) load the block's first piece; they are
    // cleared in the fragments
    const uint32_t wp = kb * kFp8Blk + 16 * piece < a.K ? 16u * piece : 0u;
#pragma unroll
    for (int j = 0; j < S::LA; ++j)
      load_lds16(wbase + (size_t)kb * kFp8Blk, woff[j] + wp, st + (wv * S::LA + j) * 1024);
#pragma unroll
    for (int j = 0; j < S::LB; ++j)
      load_lds16(xbase + (size_t)kb * kFp8Blk, xoff[j], st + S::kA + (wv * S::LB + j) * 1024);
    if (lane < S::BT / S::NW)
      load_lds4(sbase + (size_t)kb * a.xrows, soff, st + S::kA + S::kB + wv * (S::BT / S::NW) * 4);
  };

  // weight fragments of this wave: rows of the tile, and their scale rows
  auto frag_row = [&](int f) {
    if constexpr (MODE == FP8_GATE_UP) return (f / (S::RF / 2)) * kSpan + wr * (8 * S::RF) + 16 * (f % (S::RF / 2));
    else return wr * (16 * S::RF) + 16 * f;
  };
  const int nbk = (a.N + kFp8Blk - 1) / kFp8Blk;
  // (constant address space: scalar loads, which do not wait behind the vector loads in flight)
  typedef const __attribute__((address_space(4))) float* cfloat_p;
  cfloat_p wsc[2];  // GATE_UP: gate and up block; else both the same
  {
    const int first = min(n0 + (MODE == FP8_GATE_UP ? wr * 8 * S::RF : wr * 16 * S::RF), nspan - 1);
    wsc[0] = (cfloat_p)(uintptr_t)(a.wsc + ((size_t)e * nbk + first / kFp8Blk) * KB);
    wsc[1] = MODE == FP8_GATE_UP ? (cfloat_p)(uintptr_t)(a.wsc + ((size_t)e * nbk + (nspan + first) / kFp8Blk) * KB)
                                 : wsc[0];
  }

  f32x4 acc[S::RF][S::TF];
#pragma unroll
  for (int f = 0; f < S::RF; ++f)
#pragma unroll
    for (int t = 0; t < S::TF; ++t) acc[f][t] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int slot0 = (q ^ (r & 7)) * 16, slot1 = slot0 ^ 64;  // pieces q and q + 4 of a row with row % 8 == r % 8
  const int aoff = (frag_row(0) + r) * 128, boff = S::kA + (16 * wt + r) * 128, xoffs = S::kA + S::kB + (16 * wt + r) * 4;
  auto compute = [&](int kb, float s0, float s1, auto nt) {
    constexpr int NT = decltype(nt)::value;
    const uint8_t* st = lds + (kb % S::NS) * S::kStage;
    const uint8_t *pa0 = st + aoff + slot0, *pa1 = st + aoff + slot1;
    const uint8_t *pb0 = st + boff + slot0, *pb1 = st + boff + slot1, *px = st + xoffs;
    auto frag = [](const uint8_t* p0, const uint8_t* p1) {
      const u32x4 lo = *reinterpret_cast<const u32x4*>(p0), hi = *reinterpret_cast<const u32x4*>(p1);
      return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };
    i32x8 A[S::RF], B[NT];
    float sx[NT];
    f32x4 z[NT][S::RF];
    constexpr int kUp = MODE == FP8_GATE_UP ? kSpan * 128 : 0;  // bytes from a gate row to its up row
#pragma unroll
    for (int f = 0; f < S::RF; ++f) {
      const int o = MODE == FP8_GATE_UP ? (f / (S::RF / 2)) * kUp + (f % (S::RF / 2)) * 2048 : f * 2048;
      A[f] = frag(pa0 + o, pa1 + o);
    }
    if (kb * kFp8Blk + kFp8Blk > a.K) {  // the last block of a K that ends inside it
      const bool lo = kb * kFp8Blk + 16 * q < a.K, hi = kb * kFp8Blk + 64 + 16 * q < a.K;
#pragma unroll
      for (int f = 0; f < S::RF; ++f)
#pragma unroll
        for (int i = 0; i < 8; ++i) A[f][i] = (i < 4 ? lo : hi) ? A[f][i] : 0;
    }
    // Pipeline over token fragments: fragment t + 1 is read and fragment t - 1 is added while the matrix
    // instructions of fragment t run.  The scheduling groups keep that order.
    B[0] = frag(pb0, pb1);
    sx[0] = *reinterpret_cast<const float*>(px);
#pragma unroll
    for (int t = 0; t <= NT; ++t) {
      if (t + 1 < NT) {
        B[t + 1] = frag(pb0 + (t + 1) * S::WT * 2048, pb1 + (t + 1) * S::WT * 2048);
        sx[t + 1] = *reinterpret_cast<const float*>(px + (t + 1) * S::WT * 64);
        __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
      }
#pragma unroll
      for (int f = 0; f < S::RF; ++f) {
        if (t < NT) {
          z[t][f] = fp8_mfma(A[f], B[t]);
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
        if (t > 0) {
          const float sc = sx[t - 1] * (f < S::RF / 2 ? s0 : s1);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[f][t - 1][i] = fmaf(z[t - 1][f][i], sc, acc[f][t - 1][i]);
          __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
        }
      }
    }
  };

  constexpr int kOps = S::LA + S::LB + 1;  // vector-memory operations of one stage, per wave
#pragma unroll
  for (int i = 0; i < S::NS - 1; ++i)
    if (i < KB) issue(i);
  // one loop per number of token fragments computed (the wave's live ones, rounded up to 1 / 4 of the tile): a
  // bound known at compile time keeps the accumulators in registers
  auto loop = [&](auto nt) {
    float s0 = wsc[0][0], s1 = wsc[1][0];
    for (int kb = 0; kb < KB; ++kb) {
      // the loads of this step have landed; those of later steps may be in flight
      if (S::NS > 2 && kb + S::NS - 2 < KB) wait_barrier<(S::NS - 2) * kOps>();
      else wait_barrier<0>();
      if (kb + S::NS - 1 < KB) issue(kb + S::NS - 1);
      const int next = min(kb + 1, KB - 1);
      const float n0s = wsc[0][next], n1s = wsc[1][next];
      compute(kb, s0, s1, nt);
      s0 = n0s;
      s1 = n1s;
    }
  };
  using std::integral_constant;
  constexpr int kQuarter = S::TF / 4;
  if (live > 3 * kQuarter) loop(integral_constant<int, S::TF>{});
  else if (live > 2 * kQuarter) loop(integral_constant<int, 3 * kQuarter>{});
  else if (live > kQuarter) loop(integral_constant<int, 2 * kQuarter>{});
  else loop(integral_constant<int, kQuarter>{});
  wait_barrier<0>();  // the stages are free

  // accumulator (f, t) element i of lane r + 16 q: tile row frag_row(f) + 4 q + i, token 16 (t WT + wt) + r
  if constexpr (MODE == FP8_GATE_UP) {
    // h of this tile's 128 columns: one activation block, so the tile holds whole scales
    static_assert(S::BN == 256 || MODE != FP8_GATE_UP, "one activation block per tile");
    float* amax = reinterpret_cast<float*>(lds);               // [WR][BT]
    uint8_t* codes = lds + S::WR * S::BT * 4;                  // [BT][128], 16-byte pieces at p ^ (token & 7)
#pragma unroll
    for (int t = 0; t < S::TF; ++t) {
      float m = kFp8Tiny;
#pragma unroll
      for (int f = 0; f < S::RF / 2; ++f)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // rounded to bf16 first: the intermediate's definition
          const float h = __uint_as_float((uint32_t)f32_to_bf16(swiglu(acc[f][t][i], acc[f + S::RF / 2][t][i],
                                                                       a.limit)) << 16);
          acc[f][t][i] = h;
          m = fmaxf(m, fabsf(h));
        }
      m = max_rows(m);
      if (q == 0) amax[wr * S::BT + 16 * (t * S::WT + wt) + r] = m;
    }
    wait_barrier<0>();
#pragma unroll
    for (int t = 0; t < S::TF; ++t) {
      const int tok = 16 * (t * S::WT + wt) + r;
      float m = amax[tok];
#pragma unroll
      for (int w = 1; w < S::WR; ++w) m = fmaxf(m, amax[w * S::BT + tok]);
      const float f = kFp8Max / m;
      if (wr == 0 && q == 0 && r0 + tok < rend) a.hs[(size_t)(n0 / kFp8Blk) * a.rows + r0 + tok] = m / kFp8Max;
#pragma unroll
      for (int fr = 0; fr < S::RF / 2; ++fr) {
        const int col = wr * (8 * S::RF) + 16 * fr + 4 * q;
        *reinterpret_cast<uint32_t*>(codes + tok * 128 + (((col >> 4) ^ (tok & 7)) << 4) + (col & 15)) =
            fp8_codes4(acc[fr][t][0] * f, acc[fr][t][1] * f, acc[fr][t][2] * f, acc[fr][t][3] * f);
      }
    }
    wait_barrier<0>();
    for (int c = tid; c < S::BT * 8; c += 64 * S::NW) {
      const int tok = c >> 3, p = c & 7;
      if (r0 + tok < rend)
        *reinterpret_cast<u32x4*>(a.hq + (size_t)(r0 + tok) * nspan + n0 + 16 * p) =
            *reinterpret_cast<const u32x4*>(codes + tok * 128 + ((p ^ (tok & 7)) << 4));
    }
  } else {
    // through LDS, so that whole token rows are stored: row of BN values, 16-byte pieces at c ^ (token % pieces)
    constexpr int kPieces = S::BN / 8;
#pragma unroll
    for (int t = 0; t < S::TF; ++t) {
      const int tok = 16 * (t * S::WT + wt) + r;
#pragma unroll
      for (int f = 0; f < S::RF; ++f) {
        const int col = frag_row(f) + 4 * q;
        const f32x4 v = acc[f][t];
        *reinterpret_cast<uint2*>(lds + tok * (S::BN * 2) + (((col >> 3) ^ (tok & (kPieces - 1))) << 4) + (col & 4) * 2) =
            make_uint2(f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16,
                       f32_to_bf16(v[2]) | (uint32_t)f32_to_bf16(v[3]) << 16);
      }
    }
    wait_barrier<0>();
    const bool vec = a.ldo % 8 == 0 && ((uintptr_t)a.out & 15) == 0;
    for (int c = tid; c < S::BT * kPieces; c += 64 * S::NW) {
      const int tok = c / kPieces, p = c % kPieces, n = n0 + 8 * p;
      if (r0 + tok >= rend || n >= a.N) continue;
      const u32x4 v = *reinterpret_cast<const u32x4*>(lds + tok * (S::BN * 2) + ((p ^ (tok & (kPieces - 1))) << 4));
      const size_t row = MODE == FP8_DOWN ? (size_t)a.pairs[r0 + tok] : (size_t)(r0 + tok);
      uint16_t* out = a.out + row * (size_t)a.ldo + n;
      if (vec && n + 8 <= a.N) {
        *reinterpret_cast<u32x4*>(out) = v;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (n + i < a.N) out[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
      }
    }
  }
}

template <class S, Fp8Mode MODE>
hipError_t launch_tile(const Fp8Args& a, long long token_tiles, int band, hipStream_t s) {
  const int nspan = MODE == FP8_GATE_UP ? a.N / 2 : a.N, span = MODE == FP8_GATE_UP ? S::BN / 2 : S::BN;
  const long long total = token_tiles * ((nspan + span - 1) / span);
  const long long grid = (total + 7) / 8 * 8;
  // more dynamic LDS than the default limit: asked for on every call (a host-side attribute, no device work)
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&fp8_tile_kernel<S, MODE>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, S::kLds);
  if (e != hipSuccess) return e;
  fp8_tile_kernel<S, MODE><<<dim3((unsigned)grid), dim3(64 * S::NW), S::kLds, s>>>(a, band);
  return hipGetLastError();
}

using Big = TileShape<4, 2, 4, 8, 2>;  // 256 x 256

}  // namespace

int fp8_tile_tokens() { return Big::BT; }

hipError_t launch_fp8_tile(Fp8Mode mode, const Fp8Args& a, long long token_tiles, hipStream_t s) {
  switch (mode) {
    case FP8_DENSE: return launch_tile<Big, FP8_DENSE>(a, (a.rows + Big::BT - 1) / Big::BT, 4, s);
    case FP8_GATE_UP: return launch_tile<Big, FP8_GATE_UP>(a, token_tiles, 1, s);
    default: return launch_tile<Big, FP8_DOWN>(a, token_tiles, 1, s);
  }
}

}  // namespace moe
