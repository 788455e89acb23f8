// Tiled product on 8-bit integer weights: many token rows per weight matrix
// (prompts).
//
// Block tile = BN = 16 RF WR weight rows x BT = 16 TF WT tokens, by WR x WT
// waves of RF x TF fragments each; step = 128 of K, two 16 x 16 x 64 matrix
// instructions per fragment, added to its 32-bit integers.
//
// Both operands reach LDS by 16-byte direct global->LDS loads (buffer form), a
// ring of NS stages of 128-byte rows; piece p of row r lies at slot p ^ (r & 7),
// which makes the fragment reads (16 rows, one 16-byte piece each per quarter
// wave) conflict-free.  A step's barrier comes two fragments before its end: by
// then everything of the stage is in registers, so it says both that the next
// stage has landed and that this one may be refilled, and matrix instructions
// run on while the next fragments are read.  Loads are issued one by one between
// matrix instructions.
//
// The 256 x 256 tile has room for two stages only, and its loads, when they come
// from memory, take longer than a step.  There a stage is refilled in two parts
// as soon as they are free: X = the weights and the first half of the tokens, free
// in the middle of the step (the weights are in registers by then), Y = the second
// half, free at its end:
//   start(kb): X(kb) has landed, everyone is done with stage kb - 1; Y(kb + 1) is issued
//   mid(kb):   Y(kb) has landed, everyone is done with X(kb);        X(kb + 2) is issued
//
// K that ends inside a step: the tokens' codes are zero from there on, and whatever
// integers the weights' pieces hold, their products are.
//
// Bound by operand movement (LDS reads of both operands once per fragment, direct
// loads) and, on long runs, by power: 8192 rows of 4096 x 7168 take 167 us on a cool
// GPU and 196 to 210 at the median (2.9 and 2.3 to 2.5 POP/s; matrix instructions alone reach 3.3 to
// 3.9 on random bits, a library's 8-bit product 2.0 at this shape), 148 with zeros for
// operands; without the matrix instructions the rest took 128 us of 133.  256 experts of
// 7168 x 2048 with 8192 tokens, top-8: gate / up 2160 to 2230 us, down 1300 to 1340 (1.6
// to 1.7 POP/s: an expert's tiles of 256 rows are two thirds full).  33 rows of 2816 x 4096: 8.6 us, of
// which the weights' 12 MB are 2.4.
//
// At 8192 rows, us, against 176 of that time: four waves of 128 x 128 with accumulators
// among the accumulation registers 212 (copies), fragments read in pairs 185 to 192,
// waves that load apart from waves that compute on three weight stages the same, weights
// stored tile by tile the same.  Weight fragments in two sets of registers spill, and a
// spill's memory operations break the counts of the waits below.
#include "moe_int8.h"
#include "moe_wave.h"

namespace moe {
namespace {

template <int WR_, int WT_, int RF_, int TF_, int NS_, int KG_ = 1>
struct TileShape {
  static constexpr int WR = WR_, WT = WT_, RF = RF_, TF = TF_, NS = NS_, KG = KG_;
  static constexpr int NW = WR * WT, BN = 16 * RF * WR, BT = 16 * TF * WT;
  static constexpr int kA = BN * 128, kB = BT * 128, kStage = kA + kB;
  static constexpr int LA = BN / 8 / NW, LB = BT / 8 / NW;  // 16-byte loads per wave and stage
  static constexpr int kOutBytes = BT * BN * 2;             // bf16 output tile (shares the stages' memory)
  static constexpr int kRing = NS * kStage, kLds = KG * kRing > kOutBytes ? KG * kRing : kOutBytes;
  static constexpr bool kTwo = NS == 2;  // refilled in two parts
  static constexpr int kX = kTwo ? LA + LB / 2 : LA + LB, kY = kTwo ? LB / 2 : 0;  // loads per wave of the two parts
  static_assert(BN / 8 % NW == 0 && BT / 16 % NW == 0, "loads are dealt evenly");
  static_assert((KG - 1) * BN * BT * 4 <= KG * kRing, "the groups' sums fit the stages");
  static_assert(TF == 8 || TF == 4, "loops for these");
};

// Direct global->LDS loads of 16 bytes per lane, at base + off.  `bytes` from base on are inside the buffer: a lane with
// off >= bytes reads nothing (rows past the end of a tile; their results are dropped).  The range check is promised for
// the lane's own offset only, not for the instruction's scalar one, so that one stays 0.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, bytes, 0x00020000);
}
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, uint32_t off, void* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, off, 0, 0, 0);
}

// Wait until at most N of this wave's vector-memory operations are outstanding (and its LDS operations are done), then
// the block's barrier.
template <int N>
__device__ __forceinline__ void wait_barrier() {
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0x0 << 8));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// fp32 value of a sum: the same two products in every kernel.
__device__ __forceinline__ float value(int acc, float sx, float sw) { return (float)acc * sx * sw; }

// Grouped products of few rows bound the number of tiles far above what there is: a block per compute unit (one fits)
// takes tiles in turn.  Elsewhere a block per tile, which evens out tiles of unequal cost.
template <class S, Int8Mode MODE>
constexpr bool takes_turns() {
  return S::BT == 64 && MODE != INT8_DENSE;
}

// One tile: weight rows from n0 on (GATE_UP: gate rows, and their up rows) by up to BT token rows from r0 on, of expert e's
// that end at rend.  SPLIT: K blocks [kb0, kb1) of them, whose sums are stored.
template <class S, Int8Mode MODE, bool SPLIT = false>
__device__ __forceinline__ void run_tile(const Int8Args& a, uint8_t* shared, int e, int r0, int rend, int n0, int kb0 = 0,
                                         int kb1 = 0) {
  const int tid = threadIdx.x, lane = tid & 63, gw = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kg = S::KG > 1 ? gw / S::NW : 0, wv = S::KG > 1 ? gw % S::NW : gw;  // K group, wave in it
  const int r = lane & 15, q = lane >> 4;
  const int wr = wv % S::WR, wt = wv / S::WR;
  const int Kp = int8_pad(a.K), KB = SPLIT ? kb1 : Kp / 128;
  const int steps = ((SPLIT ? kb1 - kb0 : KB) + S::KG - 1) / S::KG;  // step s of group g: K block kb0 + s KG + g
  const int nspan = MODE == INT8_GATE_UP ? a.N / 2 : a.N;          // output columns
  constexpr int kSpan = MODE == INT8_GATE_UP ? S::BN / 2 : S::BN;  // per tile
  uint8_t* lds = shared + kg * S::kRing;
  // token fragments go round the WT waves, so a partly filled tile stays even: fragment tf of wave wt is
  // tokens 16 (tf WT + wt) ..; `live` of them hold tokens
  const int frags = (min(rend - r0, S::BT) + 15) >> 4;
  const int live = (frags - wt + S::WT - 1) / S::WT;
  auto source = [&](int row) { return MODE == INT8_GATE_UP ? a.pairs[row] / a.k : row; };

  // Loads.  This lane's part of an instruction: 8 rows of 8 pieces, row lane / 8, slot lane % 8.  Each load of a step
  // has its lane offsets in a register; the K block is in the buffer's base, made once a step.
  const int lrow = lane >> 3, piece = (lane & 7) ^ lrow;
  // first token row of load j: half of each wave's loads fill the first half of the tile's tokens
  auto tok_row = [&](int j) { return j / (S::LB / 2) * (S::BT / 2) + 8 * (wv * (S::LB / 2) + j % (S::LB / 2)); };
  uint32_t woff[S::LA], xoff[S::LB];
#pragma unroll
  for (int i = 0; i < S::LA; ++i) woff[i] = (uint32_t)(8 * i + lrow) * (uint32_t)a.K + 16 * piece;
#pragma unroll
  for (int j = 0; j < S::LB; ++j) {
    const int row = tok_row(j) + lrow;
    if constexpr (MODE == INT8_GATE_UP)
      xoff[j] = r0 + row < rend ? (uint32_t)source(r0 + row) * (uint32_t)Kp + 16 * piece
                                : 0xFFFFFF00u;  // behind the buffer's end: not read
    else
      xoff[j] = (uint32_t)row * (uint32_t)Kp + 16 * piece;
  }
  // this wave's weight rows of the tile: 8 LA from row 8 LA wv on (GATE_UP: all gate rows or all up rows)
  const int wfirst = 8 * S::LA * wv;
  static_assert(MODE != INT8_GATE_UP || kSpan % (8 * S::LA) == 0, "a wave loads gate rows or up rows");
  const int wn = MODE == INT8_GATE_UP ? n0 + wfirst % kSpan + wfirst / kSpan * nspan : n0 + wfirst;
  const int8_t* wbase = a.w + ((size_t)e * a.N + min(wn, a.N - 1)) * a.K;
  const int wbytes = min(a.N - wn, 8 * S::LA) * a.K;  // may be negative: no rows
  const int8_t* xbase = MODE == INT8_GATE_UP ? a.xq : a.xq + (size_t)r0 * Kp;
  const int xbytes = (MODE == INT8_GATE_UP ? a.xrows : min(rend - r0, S::BT)) * Kp;
  // The loads of one step, one by one (X: LA of weights, LB / 2 of tokens; Y: LB / 2).  Steps past the last one load the
  // last one again (into a stage that is not read any more), so that the counts of the waits hold to the end.
  auto stage = [&](int step) { return lds + (S::kTwo ? step & 1 : step % S::NS) * S::kStage; };
  auto k_of = [&](int step) { return min((SPLIT ? kb0 : 0) + step * S::KG + kg, KB - 1) * 128; };
  auto load_tokens = [&](int step, int j) {
    const int k = k_of(step);
    load_lds16(rsrc_of(xbase + k, xbytes - k), xoff[j], stage(step) + S::kA + tok_row(j) * 128);
  };
  auto issue_x = [&](int step, int i) {
    if (i < S::LA) {
      const int k = k_of(step);
      load_lds16(rsrc_of(wbase + k, max(wbytes - k, 0)), woff[i], stage(step) + (wfirst + 8 * i) * 128);
    } else {
      load_tokens(step, i - S::LA);
    }
  };
  auto issue_y = [&](int step, int i) { load_tokens(step, S::LB / 2 + i); };

  // weight fragments of this wave: rows of the tile
  auto frag_row = [&](int f) {
    if constexpr (MODE == INT8_GATE_UP) return (f / (S::RF / 2)) * kSpan + wr * (8 * S::RF) + 16 * (f % (S::RF / 2));
    else return wr * (16 * S::RF) + 16 * f;
  };
  i32x4 acc[S::RF][S::TF];
#pragma unroll
  for (int f = 0; f < S::RF; ++f)
#pragma unroll
    for (int t = 0; t < S::TF; ++t) acc[f][t] = i32x4{0, 0, 0, 0};

  const int slot0 = (q ^ (r & 7)) * 16, slot1 = slot0 ^ 64;  // pieces q and q + 4 of a row with row % 8 == r % 8
  const int aoff = (frag_row(0) + r) * 128, boff = S::kA + (16 * wt + r) * 128;
  struct Frag {
    u32x4 lo, hi;
  };
  auto frag = [&](const uint8_t* p) {
    return Frag{*reinterpret_cast<const u32x4*>(p + slot0), *reinterpret_cast<const u32x4*>(p + slot1)};
  };
  constexpr int kUp = MODE == INT8_GATE_UP ? kSpan * 128 : 0;  // bytes from a gate row to its up row
  constexpr int kHalfF = S::RF / 2;
  auto a_at = [&](int f) { return aoff + (MODE == INT8_GATE_UP ? f / kHalfF * kUp + f % kHalfF * 2048 : f * 2048); };

  // One loop per number NT of token fragments computed (the wave's live ones, rounded up to a quarter of the tile's):
  // a bound known at compile time keeps the accumulators in registers.  Every loop has the same barriers.
  auto loop = [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    constexpr int kStart = NT - 2;  // the slots that the barriers come before
    constexpr int kMid = !S::kTwo ? 0 : NT > S::TF / 2 ? S::TF / 2 - 2 : kStart;
    Frag A[S::RF], B[2];
    constexpr int kLead = S::kTwo ? 2 : S::NS - 1;  // steps that X is issued ahead
#pragma unroll
    for (int n = 0; n < kLead; ++n) {
#pragma unroll
      for (int i = 0; i < S::kX; ++i) issue_x(n, i);
#pragma unroll
      for (int i = 0; i < S::kY; ++i)
        if (n == 0) issue_y(0, i);
    }
    constexpr int kInFlight = (kLead - 1) * S::kX + S::kY;  // operations that may be outstanding at a barrier
    wait_barrier<kInFlight>();  // start(0)
#pragma unroll
    for (int f = 0; f < S::RF; ++f) A[f] = frag(lds + a_at(f));
#pragma unroll
    for (int i = 0; i < 2; ++i) B[i] = frag(lds + boff + i * S::WT * 2048);
#pragma unroll 1
    for (int step = 0; step < steps; ++step) {
      const uint8_t *st = stage(step), *sn = stage(step + 1);
      if (S::KG > 1 && (SPLIT ? kb0 : 0) + step * S::KG + kg >= KB) {  // a group that has run out: its weights count as zero
#pragma unroll
        for (int f = 0; f < S::RF; ++f) A[f].lo = A[f].hi = u32x4{0, 0, 0, 0};
      }
      // slot t: matrix instructions of fragment t, reads of fragment t + 2
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (t == kMid) {
          if (kMid == 0) {
#pragma unroll
            for (int i = 0; i < S::kY; ++i) issue_y(step + 1, i);
          }
          if (S::kTwo) wait_barrier<kInFlight>();  // mid(kb)
          if (kMid == kStart) {
#pragma unroll
            for (int i = 0; i < S::kX; ++i) issue_x(step + kLead, i);
          }
        }
        if (t == kStart) wait_barrier<kInFlight>();  // start(kb + 1)
        __builtin_amdgcn_sched_barrier(0);
        const int tn = t >= kStart ? t - kStart : t + 2;
        const Frag Bn = frag((t >= kStart ? sn : st) + boff + tn * S::WT * 2048);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
        for (int f = 0; f < S::RF; ++f) {
          acc[f][t] = int8_mfma(A[f].lo, B[t & 1].lo, acc[f][t]);
          acc[f][t] = int8_mfma(A[f].hi, B[t & 1].hi, acc[f][t]);
          __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
          // The loads go between matrix instructions: Y over the slots before the mid barrier, X over those between
          // it and the start barrier.
          if (f == (S::RF > 1 ? 1 : 0) && t < kStart) {
            const int slots = t < kMid ? kMid : kStart - kMid, at = t < kMid ? t : t - kMid;
            const int ops = t < kMid ? S::kY : S::kX;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = at * ops / slots; i < (at + 1) * ops / slots; ++i) {
              if (t < kMid) issue_y(step + 1, i);
              else issue_x(step + kLead, i);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
          if (t == NT - 1) {  // this fragment's weights of the next step
            A[f] = frag(sn + a_at(f));
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
          }
        }
        B[t & 1] = Bn;
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  using std::integral_constant;
  if constexpr (S::TF == 8) {
    if (live > 6) loop(integral_constant<int, 8>{});
    else if (live > 4) loop(integral_constant<int, 6>{});
    else if (live > 2) loop(integral_constant<int, 4>{});
    else loop(integral_constant<int, 2>{});
  } else {
    if (live > 2) loop(integral_constant<int, 4>{});
    else loop(integral_constant<int, 2>{});
  }
  wait_barrier<0>();  // the stages are free
  if constexpr (S::KG > 1) {  // the groups' sums
    int* part = reinterpret_cast<int*>(shared);
    if (kg > 0) {
#pragma unroll
      for (int t = 0; t < S::TF; ++t)
#pragma unroll
        for (int f = 0; f < S::RF; ++f)
          *reinterpret_cast<i32x4*>(part + ((((kg - 1) * S::TF + t) * S::RF + f) * S::NW + wv) * 256 + lane * 4) = acc[f][t];
    }
    wait_barrier<0>();
    if (kg == 0) {
      for (int g = 0; g < S::KG - 1; ++g)
#pragma unroll
        for (int t = 0; t < S::TF; ++t)
#pragma unroll
          for (int f = 0; f < S::RF; ++f)
            acc[f][t] += *reinterpret_cast<const i32x4*>(part + (((g * S::TF + t) * S::RF + f) * S::NW + wv) * 256 + lane * 4);
    }
    wait_barrier<0>();
  }
  lds = shared;
  if constexpr (SPLIT) {  // this run's sums, as they lie: a lane's four weight rows are neighbours
    static_assert(MODE == INT8_DENSE, "runs of dense tiles");
    if (kg > 0) return;
    const int ld = int8_sums_ld(a.N);
    int* sums = a.sums + (size_t)blockIdx.y * a.rows * ld;
#pragma unroll
    for (int t = 0; t < S::TF; ++t) {
      const int row = r0 + 16 * (t * S::WT + wt) + r;
#pragma unroll
      for (int f = 0; f < S::RF; ++f) {
        const int n = n0 + frag_row(f) + 4 * q;
        if (row < rend && n < ld) *reinterpret_cast<i32x4*>(sums + (size_t)row * ld + n) = acc[f][t];
      }
    }
    return;
  }

  // accumulator (f, t) element i of lane r + 16 q: tile row frag_row(f) + 4 q + i, token 16 (t WT + wt) + r.  Through
  // LDS, so that whole rows are stored: rows of kSpan values, 16-byte pieces at c ^ (token % pieces).
  constexpr int kPieces = kSpan / 8, kOutF = MODE == INT8_GATE_UP ? S::RF / 2 : S::RF;
  static_assert((kPieces & (kPieces - 1)) == 0, "pieces are exchanged by exclusive or");
  if (kg == 0) {
    const float* wsc = a.wsc + (size_t)e * a.N;
    float sw[S::RF][4];
#pragma unroll
    for (int f = 0; f < S::RF; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = frag_row(f) + 4 * q + i;
        const int n = MODE == INT8_GATE_UP ? n0 + row % kSpan + row / kSpan * nspan : n0 + row;
        sw[f][i] = wsc[min(n, a.N - 1)];
      }
#pragma unroll
    for (int t = 0; t < S::TF; ++t) {
      const int tok = 16 * (t * S::WT + wt) + r;
      const float sx = a.xs[source(min(r0 + tok, rend - 1))];
#pragma unroll
      for (int f = 0; f < kOutF; ++f) {
        const int col = MODE == INT8_GATE_UP ? wr * (8 * S::RF) + 16 * f + 4 * q : frag_row(f) + 4 * q;
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = value(acc[f][t][i], sx, sw[f][i]);
          if constexpr (MODE == INT8_GATE_UP)
            v[i] = swiglu(v[i], value(acc[f + S::RF / 2][t][i], sx, sw[f + S::RF / 2][i]), a.limit);
        }
        *reinterpret_cast<uint2*>(lds + tok * (kSpan * 2) + (((col >> 3) ^ (tok & (kPieces - 1))) << 4) + (col & 4) * 2) =
            make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
      }
    }
  }
  wait_barrier<0>();
  auto out_row = [&](int tok) {
    return a.out + (MODE == INT8_DOWN ? (size_t)a.pairs[r0 + tok] : (size_t)(r0 + tok)) * (size_t)a.ldo;
  };
  if (a.ldo % 8 == 0 && ((uintptr_t)a.out & 15) == 0) {
    for (int c = tid; c < S::BT * kPieces; c += 64 * S::NW * S::KG) {
      const int tok = c / kPieces, p = c % kPieces, n = n0 + 8 * p;
      if (r0 + tok >= rend || n >= nspan) continue;
      const u32x4 v = *reinterpret_cast<const u32x4*>(lds + tok * (kSpan * 2) + ((p ^ (tok & (kPieces - 1))) << 4));
      uint16_t* out = out_row(tok) + n;
      if (n + 8 <= nspan) {
        *reinterpret_cast<u32x4*>(out) = v;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (n + i < nspan) out[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
      }
    }
  } else {  // rows at any alignment: a value per lane, so that a wave's lanes write one run
    for (int c = tid; c < S::BT * kSpan; c += 64 * S::NW * S::KG) {
      const int tok = c / kSpan, col = c % kSpan;
      if (r0 + tok >= rend || n0 + col >= nspan) continue;
      out_row(tok)[n0 + col] = *reinterpret_cast<const uint16_t*>(
          lds + tok * (kSpan * 2) + (((col >> 3) ^ (tok & (kPieces - 1))) << 4) + (col & 7) * 2);
    }
  }
}

using Big = TileShape<4, 2, 4, 8, 2>;  // 256 weight rows x 256 tokens
using Mid = TileShape<4, 2, 4, 4, 3>;  // 256 x 128, three stages
using Few = TileShape<4, 1, 4, 4, 3>;  // 256 x 64, three stages: bound by the weights' stream

template <class S, Int8Mode MODE>
__global__ __launch_bounds__(64 * S::NW * S::KG) void int8_tile_kernel(Int8Args a, int band) {
  extern __shared__ __align__(256) uint8_t shared[];
  const int nspan = MODE == INT8_GATE_UP ? a.N / 2 : a.N;
  constexpr int kSpan = MODE == INT8_GATE_UP ? S::BN / 2 : S::BN;
  const int NB = (nspan + kSpan - 1) / kSpan;
  const int MT = MODE == INT8_DENSE ? (a.rows + S::BT - 1) / S::BT : *a.ntiles;

  // Blocks go round the 8 XCDs: XCD x takes a contiguous share of the tile
  // order (bands of token tiles, weight-block-major inside a band), so the
  // tiles that run together on one L2 share their operands.
  const int total = MT * NB, share = (total + 7) / 8;
  auto tile = [&](int i) {
    const int at = (blockIdx.x & 7) * share + i;
    if (at >= total) return;
    if constexpr (MODE == INT8_DENSE) {
      const int bi = at / (band * NB), inb = min(band, MT - bi * band), o = at - bi * band * NB;
      run_tile<S, MODE>(a, shared, 0, (bi * band + o % inb) * S::BT, a.rows, o / inb * kSpan);
    } else {
      const int4 g = a.tiles[at / NB];  // any tile of the group
      const int o = at - g.z * NB, n0 = o / g.w * kSpan;
      const int4 t = a.tiles[g.z + o % g.w];
      const int rend = a.offsets[t.x + 1];
      // a tile that is half full or less: three whole stages of it fit (8192 tokens, 256 experts: 3.58 -> 3.50 ms)
      if (S::BT == Big::BT && rend - t.y <= Mid::BT) run_tile<Mid, MODE>(a, shared, t.x, t.y, rend, n0);
      else run_tile<S, MODE>(a, shared, t.x, t.y, rend, n0);
    }
  };
  if constexpr (takes_turns<S, MODE>()) {
    for (int i = blockIdx.x >> 3; i < share; i += gridDim.x >> 3) {
      tile(i);
      wait_barrier<63>();  // the output tile in LDS is read before the next loads refill the stages
    }
  } else {
    if ((int)(blockIdx.x >> 3) < share) tile(blockIdx.x >> 3);
  }
}

template <class S, Int8Mode MODE>
hipError_t launch_tile(const Int8Args& a, long long token_tiles, int band, int cus, hipStream_t s) {
  const int nspan = MODE == INT8_GATE_UP ? a.N / 2 : a.N, span = MODE == INT8_GATE_UP ? S::BN / 2 : S::BN;
  const long long total = token_tiles * ((nspan + span - 1) / span);
  long long grid = (total + 7) / 8 * 8;
  if (takes_turns<S, MODE>() && grid > cus / 8 * 8) grid = cus / 8 * 8;
  constexpr int kLds = S::BT == Big::BT && MODE != INT8_DENSE && Mid::kLds > S::kLds ? Mid::kLds : S::kLds;
  // more dynamic LDS than the default limit: asked for on every call (a host-side attribute, no device work)
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&int8_tile_kernel<S, MODE>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (e != hipSuccess) return e;
  int8_tile_kernel<S, MODE><<<dim3((unsigned)grid), dim3(64 * S::NW * S::KG), kLds, s>>>(a, band);
  return hipGetLastError();
}

// Dense products of few tiles and a long K: blockIdx.y is a run of K blocks; a second launch joins the runs.
template <class S>
__global__ __launch_bounds__(64 * S::NW * S::KG) void int8_split_kernel(Int8Args a) {
  extern __shared__ __align__(256) uint8_t shared[];
  const int NB = (a.N + S::BN - 1) / S::BN, KB = int8_pad(a.K) / 128, run = (KB + a.splits - 1) / a.splits;
  const int tile = blockIdx.x, kb0 = blockIdx.y * run;
  run_tile<S, INT8_DENSE, true>(a, shared, 0, tile / NB * S::BT, a.rows, tile % NB * S::BN, kb0, min(KB, kb0 + run));
}

__global__ __launch_bounds__(256) void int8_join_kernel(Int8Args a) {  // a thread per four columns
  const int ld = int8_sums_ld(a.N), c = blockIdx.x * 256 + threadIdx.x, row = c / (ld / 4), n = 4 * (c - row * (ld / 4));
  if (row >= a.rows) return;
  const i32x4* p = reinterpret_cast<const i32x4*>(a.sums) + c;
  i32x4 v = p[0];
#pragma unroll 8
  for (int i = 1; i < a.splits; ++i) v += p[(size_t)i * a.rows * (ld / 4)];
  const float sx = a.xs[row];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < a.N) a.out[(size_t)row * a.ldo + n + i] = f32_to_bf16(value(v[i], sx, a.wsc[n + i]));
}

using Split = TileShape<2, 1, 1, 4, 3, 4>;  // 32 x 64, K over 4 groups of waves

hipError_t launch_split(const Int8Args& a, hipStream_t s) {
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&int8_split_kernel<Split>),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, Split::kLds);
  if (e != hipSuccess) return e;
  const int tiles = ((a.rows + Split::BT - 1) / Split::BT) * ((a.N + Split::BN - 1) / Split::BN);
  int8_split_kernel<Split><<<dim3(tiles, a.splits), dim3(64 * Split::NW * Split::KG), Split::kLds, s>>>(a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  int8_join_kernel<<<dim3((a.rows * (int8_sums_ld(a.N) / 4) + 255) / 256), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

// Nanoseconds of a dense product: rounds of its tiles on `cus` compute units (one block each) x (first loads and
// epilogue + K blocks x step).
template <class S>
long long dense_cost(const Int8Args& a, int cus, int fixed, int step) {
  const long long tiles = (long long)((a.rows + S::BT - 1) / S::BT) * ((a.N + S::BN - 1) / S::BN);
  return (tiles + cus - 1) / cus * (fixed + (long long)(int8_pad(a.K) / 128) * step);
}

// Large tiles have the fewest operand bytes per product, small ones fill the GPU when there are few, and share K over
// groups of waves.  The shape with the least cost is taken; its two numbers are fitted to 17 to 4096 rows of 576 x 7168,
// 2816 x 4096, 4096 x 7168, 7168 x 2048, 18432 x 7168 and 1000 x 2000, where every choice is within a tenth of the best.
hipError_t launch_dense(const Int8Args& a, int cus, hipStream_t s) {
  if (a.splits > 1) return launch_split(a, s);
  using T0 = Split;                        // 32 x 64, K over 4 groups of waves
  using T1 = TileShape<4, 1, 1, 4, 4, 2>;  // 64 x 64, K over 2
  using T2 = TileShape<4, 1, 2, 4, 3, 2>;  // 128 x 64, K over 2
  using T3 = TileShape<4, 2, 2, 4, 4>;     // 128 x 128
  const long long cost[5] = {dense_cost<T0>(a, cus, 3100, 158), dense_cost<T1>(a, cus, 3700, 190),
                             dense_cost<T2>(a, cus, 4300, 270), dense_cost<T3>(a, cus, 8000, 300),
                             dense_cost<Big>(a, cus, 12000, 950)};
  int best = 4;
  for (int i = 3; i >= 0; --i)
    if (cost[i] < cost[best]) best = i;
  switch (best) {
    case 0: return launch_tile<T0, INT8_DENSE>(a, (a.rows + T0::BT - 1) / T0::BT, 4, cus, s);
    case 1: return launch_tile<T1, INT8_DENSE>(a, (a.rows + T1::BT - 1) / T1::BT, 4, cus, s);
    case 2: return launch_tile<T2, INT8_DENSE>(a, (a.rows + T2::BT - 1) / T2::BT, 4, cus, s);
    case 3: return launch_tile<T3, INT8_DENSE>(a, (a.rows + T3::BT - 1) / T3::BT, 4, cus, s);
    default: return launch_tile<Big, INT8_DENSE>(a, (a.rows + Big::BT - 1) / Big::BT, 4, cus, s);
  }
}

template <Int8Mode MODE>
hipError_t launch_grouped(const Int8Args& a, int tile, long long token_tiles, int cus, hipStream_t s) {
  if (tile == Few::BT) return launch_tile<Few, MODE>(a, token_tiles, 1, cus, s);
  if (tile == Mid::BT) return launch_tile<Mid, MODE>(a, token_tiles, 1, cus, s);
  return launch_tile<Big, MODE>(a, token_tiles, 1, cus, s);
}

}  // namespace

// Runs of at least 8 blocks of 128 (two steps of the kernel's four groups), as many as fill 256 compute units, where that
// saves more steps (158 ns each) than the second launch costs (quantiser, runs and join, us, against quantiser and one
// launch: 33 rows of 576 x 7168 12.3 and 15.0, of 200 x 7008 12.6 and 14.9; 16 rows 12.3 and 12.1; in two runs 64 rows of
// 4096 x 7168 16.5 and 15.5).  Joining by atomic additions in one launch took 18 us for its runs alone.
constexpr int kSplitRows = 128, kSplitRun = 8, kSplitBlocks = 256, kSplitSaves = 22;

int int8_splits(int M, int N, int K) {
  const int KB = int8_pad(K) / 128;
  if (M <= 16 || M > kSplitRows || N > kSplitBlocks / 2 * Split::BN) return 1;
  const int tiles = (M + Split::BT - 1) / Split::BT * ((N + Split::BN - 1) / Split::BN);
  const int n = min(KB / kSplitRun, kSplitBlocks / tiles);
  if (n < 3) return 1;
  const int run = (KB + n - 1) / n;
  return KB - run >= kSplitSaves ? (KB + run - 1) / run : 1;  // no empty run
}

size_t int8_split_bytes(int max_M, int N, int K) {
  size_t n = 0;
  for (int M = Split::BT; M < max_M + Split::BT && M <= kSplitRows; M += Split::BT) {  // fewer rows of as many tiles need less
    const int rows = min(M, max_M), splits = int8_splits(rows, N, K);
    if (splits > 1) n = max(n, (size_t)splits * rows * int8_sums_ld(N) * sizeof(int));
  }
  return n;
}

int int8_tile_tokens(long long rows, int experts) {
  return rows < 48 * experts ? Few::BT : rows < 160 * experts ? Mid::BT : Big::BT;
}

hipError_t launch_int8_tile(Int8Mode mode, const Int8Args& a, int tile, long long token_tiles, int cus, hipStream_t s) {
  switch (mode) {
    case INT8_DENSE: return launch_dense(a, cus, s);
    case INT8_GATE_UP: return launch_grouped<INT8_GATE_UP>(a, tile, token_tiles, cus, s);
    default: return launch_grouped<INT8_DOWN>(a, tile, token_tiles, cus, s);
  }
}

}  // namespace moe
