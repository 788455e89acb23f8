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
// Both operands reach LDS by 16-byte direct global->LDS loads (buffer form), a
// ring of NS stages of 128-byte rows; piece p of row r lies at slot p ^ (r & 7),
// which makes the fragment reads (16 rows, one 16-byte piece each per quarter
// wave) conflict-free.  A step's barrier comes two fragments before its end: by
// then everything of the stage is in registers, so it says both that the next
// stage has landed and that this one may be refilled, and matrix instructions
// run on while the next fragments are read.  Loads are issued one by one
// between matrix instructions (in one run they held the waves up).
//
// The 256 x 256 tile has room for two stages only (130 of 160 KB), and its
// loads, when they come from memory, take longer than a step.  There a stage is
// refilled in two parts as soon as they are free: X = the weights and the first
// half of the tokens, free in the middle of the step (the weights are in
// registers by then), Y = the second half, free at its end.  Either part is
// issued one and a half steps before its first use, at the price of a second
// barrier per step:
//   start(kb): X(kb) has landed, everyone is done with stage kb - 1; Y(kb + 1) is issued
//   mid(kb):   Y(kb) has landed, everyone is done with X(kb);        X(kb + 2) is issued
//
// Measured (calls in runs of many, which hold the clock up; a launch by itself under a trace: median of 20):
// 8192 x 4096 x 7168 in 226-239 us with the quantiser's 31 (2.1 PFLOP/s; product by itself 233, at best 200);
// 500 x 2816 x 4096 in 19-20 us with the quantiser (product by itself 18.6); experts of 8192 tokens (256 experts, top-8,
// H 7168, I 2048) 4.0-4.1 ms, 2.57 gate / up and 1.39 down (1.4 PFLOP/s: the tiles are two thirds full); of 333 tokens (64
// experts, top-6, H 4096, I 1408) 255-268 us, 4.1-4.4 TB/s of weights.
#include "moe_fp8.h"

namespace moe {
namespace {

template <int WR_, int WT_, int RF_, int TF_, int NS_, int KG_ = 1>
struct TileShape {
  static constexpr int WR = WR_, WT = WT_, RF = RF_, TF = TF_, NS = NS_, KG = KG_;
  static constexpr int NW = WR * WT, BN = 16 * RF * WR, BT = 16 * TF * WT;
  static constexpr int kA = BN * 128, kB = BT * 128, kS = NW * 2 * 256, kStage = kA + kB + kS;
  static constexpr int LA = BN / 8 / NW, LB = BT / 8 / NW;  // 16-byte loads per wave and stage
  static constexpr int kOutBytes = BT * BN * 2;             // bf16 output tile (shares the stages' memory)
  static constexpr int kRing = NS * kStage, kLds = KG * kRing > kOutBytes ? KG * kRing : kOutBytes;
  static constexpr bool kTwo = NS == 2;                          // refilled in two parts
  // vector-memory operations per wave of the two parts (one part: all of them, and none)
  static constexpr int kX = kTwo ? LA + LB / 2 + 1 : LA + LB + 2, kY = kTwo ? LB / 2 + 1 : 0;
  static_assert(BN / 8 % NW == 0 && BT / 16 % NW == 0, "loads are dealt evenly");
  static_assert((KG - 1) * BN * BT * 4 <= KG * kRing, "the groups' sums fit the stages");
  static_assert(TF == 8 || TF == 4, "a half's scales fit a wave");
};

// Direct global->LDS loads of 16 and 4 bytes per lane, at base + off.  `bytes` from base on are inside the buffer: a
// lane with off >= bytes reads nothing (rows past the end of a tile; their results are dropped).  The range check is
// promised for the lane's own offset only, not for the instruction's scalar one, so that one stays 0.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, bytes, 0x00020000);
}
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, uint32_t off, void* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, off, 0, 0, 0);
}
__device__ __forceinline__ void load_lds4(__amdgpu_buffer_rsrc_t r, uint32_t off, void* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 4, off, 0, 0, 0);
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

// Grouped products of few rows bound the number of tiles far above what there is: a block per compute unit (one fits)
// takes tiles in turn.  Elsewhere a block per tile, which evens out tiles of unequal cost and leaves the loop's
// registers to the tile (experts, 8192 tokens: 4.19 ms against 4.33).
template <class S, Fp8Mode MODE>
constexpr bool takes_turns() {
  return S::BT == 64 && MODE != FP8_DENSE;
}

template <class S, Fp8Mode MODE>
__global__ __launch_bounds__(64 * S::NW * S::KG) void fp8_tile_kernel(Fp8Args a, int band) {
  extern __shared__ __align__(256) uint8_t shared[];
  const int tid = threadIdx.x, lane = tid & 63, gw = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kg = S::KG > 1 ? gw / S::NW : 0, wv = S::KG > 1 ? gw % S::NW : gw;  // K group, wave in it
  const int r = lane & 15, q = lane >> 4;
  const int wr = wv % S::WR, wt = wv / S::WR;
  const int KB = (a.K + kFp8Blk - 1) / kFp8Blk, Kp = KB * kFp8Blk;
  const int steps = (KB + S::KG - 1) / S::KG;  // step s of group g: K block s KG + g
  const int nspan = MODE == FP8_GATE_UP ? a.N / 2 : a.N;                // output columns
  constexpr int kSpan = MODE == FP8_GATE_UP ? S::BN / 2 : S::BN;        // per tile
  const int NB = (nspan + kSpan - 1) / kSpan;
  const int MT = MODE == FP8_DENSE ? (a.rows + S::BT - 1) / S::BT : *a.ntiles;

  // Blocks go round the 8 XCDs: XCD x takes a contiguous share of the tile
  // order (bands of token tiles, weight-block-major inside a band), so the
  // tiles that run together on one L2 share their operands.
  const int total = MT * NB, share = (total + 7) / 8;
  auto run_tile = [&](int i) {
  const int at = (blockIdx.x & 7) * share + i;
  if (at >= total) return;
  uint8_t* lds = shared + kg * S::kRing;
  int e = 0, r0, rend, nb;
  if constexpr (MODE == FP8_DENSE) {
    const int bi = at / (band * NB), inb = min(band, MT - bi * band), o = at - bi * band * NB;
    nb = o / inb;
    r0 = (bi * band + o % inb) * S::BT;
    rend = a.rows;
  } else {
    const int4 g = a.tiles[at / NB];  // any tile of the group
    const int o = at - g.z * NB;
    nb = o / g.w;
    const int4 t = a.tiles[g.z + o % g.w];
    e = t.x;
    r0 = t.y;
    rend = a.offsets[e + 1];
  }
  const int n0 = nb * kSpan;
  // token fragments go round the WT waves, so a partly filled tile stays even: fragment tf of wave wt is
  // tokens 16 (tf WT + wt) ..; `live` of them hold tokens
  const int frags = (min(rend - r0, S::BT) + 15) >> 4;
  const int live = (frags - wt + S::WT - 1) / S::WT;

  // Loads.  This lane's part of an instruction: 8 rows of 8 pieces, row lane / 8, slot lane % 8.  Each load of a step
  // has its lane offsets in a register; the K block is in the buffer's base, made once a step.  (Offsets added up per
  // load: 8192 x 4096 x 7168 7 % slower.)
  const int lrow = lane >> 3, piece = (lane & 7) ^ lrow;
  // first token row of load j: half of each wave's loads fill the first half of the tile's tokens
  auto tok_row = [&](int j) { return j / (S::LB / 2) * (S::BT / 2) + 8 * (wv * (S::LB / 2) + j % (S::LB / 2)); };
  // A wave loads the scales of its own tokens: lane l that of fragment (h TF / 2 + l / 16), token l % 16, of half h
  // (TF = 4 needs 32 of them; the other lanes repeat them into slots of their own)
  auto scale_row = [&](int h) { return 16 * ((h * (S::TF / 2) + (lane >> 4) % (S::TF / 2)) * S::WT + wt) + (lane & 15); };
  uint32_t woff[S::LA], xoff[S::LB], soff[2];
#pragma unroll
  for (int i = 0; i < S::LA; ++i) woff[i] = (uint32_t)(8 * i + lrow) * (uint32_t)a.K + 16 * piece;
  if constexpr (MODE == FP8_GATE_UP) {
#pragma unroll
    for (int j = 0; j < S::LB; ++j)
      xoff[j] = r0 + tok_row(j) + lrow < rend
                    ? (uint32_t)(a.pairs[r0 + tok_row(j) + lrow] / a.k) * (uint32_t)Kp + 16 * piece
                    : 0xFFFFFF00u;  // behind the buffer's end: not read
#pragma unroll
    for (int h = 0; h < 2; ++h)
      soff[h] = 4u * (uint32_t)(a.pairs[min(r0 + scale_row(h), rend - 1)] / a.k);
  } else {
#pragma unroll
    for (int j = 0; j < S::LB; ++j) xoff[j] = (uint32_t)(tok_row(j) + lrow) * (uint32_t)Kp + 16 * piece;
#pragma unroll
    for (int h = 0; h < 2; ++h) soff[h] = 4 * scale_row(h);
  }
  // this wave's weight rows of the tile: 8 LA from row 8 LA wv on (GATE_UP: all gate rows or all up rows)
  const int wfirst = 8 * S::LA * wv;
  static_assert(MODE != FP8_GATE_UP || kSpan % (8 * S::LA) == 0, "a wave loads gate rows or up rows");
  const int wn = MODE == FP8_GATE_UP ? n0 + wfirst % kSpan + wfirst / kSpan * nspan : n0 + wfirst;
  const uint8_t* wbase = a.w + ((size_t)e * a.N + min(wn, a.N - 1)) * a.K;
  const int wbytes = min(a.N - wn, 8 * S::LA) * a.K;  // may be negative: no rows
  const uint8_t* xbase = MODE == FP8_GATE_UP ? a.xq : a.xq + (size_t)r0 * Kp;
  const float* sbase = MODE == FP8_GATE_UP ? a.xs : a.xs + r0;
  const int xrows = MODE == FP8_GATE_UP ? a.xrows : min(rend - r0, S::BT);
  // The loads of one step, one by one (X: LA of weights, LB / 2 of tokens, 1 of scales; Y: LB / 2 and 1).  Steps past
  // the last one load the last one again (into a stage that is not read any more), so that the counts of the waits
  // hold to the end.
  auto stage = [&](int step) { return lds + (S::kTwo ? step & 1 : step % S::NS) * S::kStage; };
  auto load_tokens = [&](int step, int j) {
    const int kb = min(step * S::KG + kg, KB - 1);
    load_lds16(rsrc_of(xbase + kb * kFp8Blk, xrows * Kp - kb * kFp8Blk), xoff[j], stage(step) + S::kA + tok_row(j) * 128);
  };
  auto load_scales = [&](int step, int h) {
    const int kb = min(step * S::KG + kg, KB - 1);
    load_lds4(rsrc_of(sbase + (size_t)kb * a.xrows, xrows * 4), soff[h], stage(step) + S::kA + S::kB + (wv * 2 + h) * 256);
  };
  auto issue_x = [&](int step, int i) {
    if (i < S::LA) {
      const int kb = min(step * S::KG + kg, KB - 1);
      // pieces past the end of a weight row (K not a multiple of 128) load from the next row, or lie behind the buffer's
      // end; they are cleared in the fragments
      load_lds16(rsrc_of(wbase + kb * kFp8Blk, max(wbytes - kb * kFp8Blk, 0)), woff[i],
                 stage(step) + (wfirst + 8 * i) * 128);
    } else if (i < S::LA + S::LB / 2) {
      load_tokens(step, i - S::LA);
    } else if (i == S::LA + S::LB / 2) {
      load_scales(step, 0);
    } else {  // one part only
      if (i < S::kX - 1) load_tokens(step, i - S::LA - 1);
      else load_scales(step, 1);
    }
  };
  auto issue_y = [&](int step, int i) {
    if (i < S::kY - 1) load_tokens(step, S::LB / 2 + i);
    else load_scales(step, 1);
  };

  // weight fragments of this wave: rows of the tile, and their scale rows
  auto frag_row = [&](int f) {
    if constexpr (MODE == FP8_GATE_UP) return (f / (S::RF / 2)) * kSpan + wr * (8 * S::RF) + 16 * (f % (S::RF / 2));
    else return wr * (16 * S::RF) + 16 * f;
  };
  const int nbk = (a.N + kFp8Blk - 1) / kFp8Blk;
  // the scales of 64 K blocks at a time in one register, a lane each: a step takes its own by readlane (a load per
  // step would wait behind the direct-to-LDS loads, a scalar load behind every LDS read)
  const float* wsc[2];  // GATE_UP: gate and up block; else both the same
  {
    const int first = min(n0 + (MODE == FP8_GATE_UP ? wr * 8 * S::RF : wr * 16 * S::RF), nspan - 1);
    wsc[0] = a.wsc + ((size_t)e * nbk + first / kFp8Blk) * KB;
    wsc[1] = MODE == FP8_GATE_UP ? a.wsc + ((size_t)e * nbk + (nspan + first) / kFp8Blk) * KB : wsc[0];
  }

  f32x4 acc[S::RF][S::TF];
#pragma unroll
  for (int f = 0; f < S::RF; ++f)
#pragma unroll
    for (int t = 0; t < S::TF; ++t) acc[f][t] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int slot0 = (q ^ (r & 7)) * 16, slot1 = slot0 ^ 64;  // pieces q and q + 4 of a row with row % 8 == r % 8
  const int aoff = (frag_row(0) + r) * 128, boff = S::kA + (16 * wt + r) * 128, xoffs = S::kA + S::kB + wv * 512 + r * 4;
  auto frag = [](const uint8_t* p0, const uint8_t* p1) {
    const u32x4 lo = *reinterpret_cast<const u32x4*>(p0), hi = *reinterpret_cast<const u32x4*>(p1);
    return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  };
  constexpr int kUp = MODE == FP8_GATE_UP ? kSpan * 128 : 0;  // bytes from a gate row to its up row
  constexpr int kHalfF = S::RF / 2;

  // One loop per number NT of token fragments computed (the wave's live ones, rounded up to a quarter of the tile's):
  // a bound known at compile time keeps the accumulators in registers.  Every loop has the same barriers.
  auto loop = [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    constexpr int kStart = NT - 2;                                 // the slots that the barriers come before
    constexpr int kMid = !S::kTwo ? 0 : NT > S::TF / 2 ? S::TF / 2 - 2 : kStart;
    i32x8 A[S::RF], B[2];
    float sx[2];
    float v0, v1;
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
    {
      const uint8_t* st = lds;
#pragma unroll
      for (int f = 0; f < S::RF; ++f) {
        const int o = MODE == FP8_GATE_UP ? f / kHalfF * kUp + f % kHalfF * 2048 : f * 2048;
        A[f] = frag(st + aoff + slot0 + o, st + aoff + slot1 + o);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        B[i] = frag(st + boff + slot0 + i * S::WT * 2048, st + boff + slot1 + i * S::WT * 2048);
        sx[i] = *reinterpret_cast<const float*>(st + xoffs + i * 64);
      }
    }
#pragma unroll 1
    for (int step = 0; step < steps; ++step) {
      const uint8_t *st = stage(step), *sn = stage(step + 1);
      const int kb = step * S::KG + kg;
      // (every branch of the step stands before its additions: the compiler would sink them all behind a later one)
      if ((step & 63) == 0) {  // lane l: the scales of step + l; zero behind the last block (a group may run out first)
        const int i = (step + lane) * S::KG + kg;
        v0 = i < KB ? wsc[0][min(i, KB - 1)] : 0.f;
        v1 = MODE == FP8_GATE_UP ? (i < KB ? wsc[1][min(i, KB - 1)] : 0.f) : v0;
        asm volatile("" : "+v"(v0), "+v"(v1));  // waited for here, not (behind every load in flight) in each step
      }
      const float s0 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v0), step & 63));
      const float s1 = MODE == FP8_GATE_UP ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v1), step & 63)) : s0;
      if (min(kb, KB - 1) * kFp8Blk + kFp8Blk > a.K) {  // the last block of a K that ends inside it
        const int k0 = min(kb, KB - 1) * kFp8Blk;
        const bool lo = k0 + 16 * q < a.K, hi = k0 + 64 + 16 * q < a.K;
#pragma unroll
        for (int f = 0; f < S::RF; ++f)
#pragma unroll
          for (int i = 0; i < 8; ++i) A[f][i] = (i < 4 ? lo : hi) ? A[f][i] : 0;
      }
      f32x4 z[NT][S::RF];
      float scl0 = 0.f, scl1 = 0.f;
      // slot t: matrix instructions of fragment t, additions of fragment t - 1, reads of fragment t + 2
#pragma unroll
      for (int t = 0; t <= NT; ++t) {
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
        i32x8 Bn;
        float sxn = 0.f;
        if (t < NT) {
          const uint8_t *sb = t >= kStart ? sn : st;
          const int tn = t >= kStart ? t - kStart : t + 2;
          Bn = frag(sb + boff + slot0 + tn * S::WT * 2048, sb + boff + slot1 + tn * S::WT * 2048);
          sxn = *reinterpret_cast<const float*>(sb + xoffs + tn / (S::TF / 2) * 256 + tn % (S::TF / 2) * 64);
          __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
        }
#pragma unroll
        for (int f = 0; f < S::RF; ++f) {
          if (t < NT) {
            z[t][f] = fp8_mfma(A[f], B[t & 1]);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          }
          if (t > 0) {
            const float sc = f < kHalfF ? scl0 : scl1;
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[f][t - 1][i] = fmaf(z[t - 1][f][i], sc, acc[f][t - 1][i]);
            __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
          }
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
            const int o = MODE == FP8_GATE_UP ? f / kHalfF * kUp + f % kHalfF * 2048 : f * 2048;
            A[f] = frag(sn + aoff + slot0 + o, sn + aoff + slot1 + o);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
          }
        }
        if (t < NT) {
          scl0 = sx[t & 1] * s0;
          scl1 = MODE == FP8_GATE_UP ? sx[t & 1] * s1 : scl0;
          B[t & 1] = Bn;
          sx[t & 1] = sxn;
        }
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
  if constexpr (S::KG > 1) {  // the groups' sums, in group order
    float* part = reinterpret_cast<float*>(shared);
    if (kg > 0) {
#pragma unroll
      for (int t = 0; t < S::TF; ++t)
#pragma unroll
        for (int f = 0; f < S::RF; ++f)
          *reinterpret_cast<f32x4*>(part + ((((kg - 1) * S::TF + t) * S::RF + f) * S::NW + wv) * 256 + lane * 4) = acc[f][t];
    }
    wait_barrier<0>();
    if (kg == 0) {
      for (int g = 0; g < S::KG - 1; ++g)
#pragma unroll
        for (int t = 0; t < S::TF; ++t)
#pragma unroll
          for (int f = 0; f < S::RF; ++f)
            acc[f][t] += *reinterpret_cast<const f32x4*>(part + (((g * S::TF + t) * S::RF + f) * S::NW + wv) * 256 + lane * 4);
    }
    wait_barrier<0>();
  }
  lds = shared;

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
      float f, s;
      fp8_factor(m, f, s);
      if (wr == 0 && q == 0 && r0 + tok < rend) a.hs[(size_t)(n0 / kFp8Blk) * a.rows + r0 + tok] = s;
#pragma unroll
      for (int fr = 0; fr < S::RF / 2; ++fr) {
        const int col = wr * (8 * S::RF) + 16 * fr + 4 * q;
        *reinterpret_cast<uint32_t*>(codes + tok * 128 + (((col >> 4) ^ (tok & 7)) << 4) + (col & 15)) =
            fp8_codes4(acc[fr][t][0] * f, acc[fr][t][1] * f, acc[fr][t][2] * f, acc[fr][t][3] * f);
      }
    }
    wait_barrier<0>();
    for (int c = tid; c < S::BT * 8; c += 64 * S::NW * S::KG) {
      const int tok = c >> 3, p = c & 7;
      if (r0 + tok < rend)
        *reinterpret_cast<u32x4*>(a.hq + (size_t)(r0 + tok) * nspan + n0 + 16 * p) =
            *reinterpret_cast<const u32x4*>(codes + tok * 128 + ((p ^ (tok & 7)) << 4));
    }
  } else {
    // through LDS, so that whole token rows are stored: row of BN values, 16-byte pieces at c ^ (token % pieces)
    constexpr int kPieces = S::BN / 8;
    if (kg == 0)
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
    auto out_row = [&](int tok) {
      return a.out + (MODE == FP8_DOWN ? (size_t)a.pairs[r0 + tok] : (size_t)(r0 + tok)) * (size_t)a.ldo;
    };
    if (a.ldo % 8 == 0 && ((uintptr_t)a.out & 15) == 0) {
      for (int c = tid; c < S::BT * kPieces; c += 64 * S::NW * S::KG) {
        const int tok = c / kPieces, p = c % kPieces, n = n0 + 8 * p;
        if (r0 + tok >= rend || n >= a.N) continue;
        const u32x4 v = *reinterpret_cast<const u32x4*>(lds + tok * (S::BN * 2) + ((p ^ (tok & (kPieces - 1))) << 4));
        uint16_t* out = out_row(tok) + n;
        if (n + 8 <= a.N) {
          *reinterpret_cast<u32x4*>(out) = v;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (n + i < a.N) out[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
        }
      }
    } else {  // rows at any alignment: a value per lane, so that a wave's lanes write one run (5570 x 3551 x 144: 57
      for (int c = tid; c < S::BT * S::BN; c += 64 * S::NW * S::KG) {  // -> 45 us; 3552 columns: 28)
        const int tok = c / S::BN, col = c % S::BN;
        if (r0 + tok >= rend || n0 + col >= a.N) continue;
        out_row(tok)[n0 + col] = *reinterpret_cast<const uint16_t*>(
            lds + tok * (S::BN * 2) + (((col >> 3) ^ (tok & (kPieces - 1))) << 4) + (col & 7) * 2);
      }
    }
  }
  };
  if constexpr (takes_turns<S, MODE>()) {
    for (int i = blockIdx.x >> 3; i < share; i += gridDim.x >> 3) {
      run_tile(i);
      wait_barrier<63>();  // the output tile in LDS is read before the next loads refill the stages
    }
  } else {
    if ((int)(blockIdx.x >> 3) < share) run_tile(blockIdx.x >> 3);
  }
}

template <class S, Fp8Mode MODE>
hipError_t launch_tile(const Fp8Args& a, long long token_tiles, int band, int cus, hipStream_t s) {
  const int nspan = MODE == FP8_GATE_UP ? a.N / 2 : a.N, span = MODE == FP8_GATE_UP ? S::BN / 2 : S::BN;
  const long long total = token_tiles * ((nspan + span - 1) / span);
  long long grid = (total + 7) / 8 * 8;
  if (takes_turns<S, MODE>() && grid > cus / 8 * 8) grid = cus / 8 * 8;
  // more dynamic LDS than the default limit: asked for on every call (a host-side attribute, no device work)
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&fp8_tile_kernel<S, MODE>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, S::kLds);
  if (e != hipSuccess) return e;
  fp8_tile_kernel<S, MODE><<<dim3((unsigned)grid), dim3(64 * S::NW * S::KG), S::kLds, s>>>(a, band);
  return hipGetLastError();
}

using Big = TileShape<4, 2, 4, 8, 2>;  // 256 weight rows x 256 tokens

// Tile count of a dense product, rounds of it on `cus` compute units (one block each), and the time of a step
// (one K block) measured with one round or less.
template <class S>
long long dense_cost(const Fp8Args& a, int cus, int ns_per_block) {
  const long long tiles = (long long)((a.rows + S::BT - 1) / S::BT) * ((a.N + S::BN - 1) / S::BN);
  return (tiles + cus - 1) / cus * ns_per_block;
}

// Dense products: large tiles have the fewest operand bytes per product, small ones fill the GPU when there are few,
// and share K over groups of waves.  The shape with the least rounds x step time is taken (the step times are those
// of one block per compute unit; measured with 48 x 4096 x 7168 and confirmed within a fifth on 100 x 7168 x 7168,
// 500 and 1000 x 2816 x 4096, 1000 x 7168 x 7168, 2000 x 1000 x 2000).
hipError_t launch_dense(const Fp8Args& a, int cus, hipStream_t s) {
  using T0 = TileShape<2, 1, 1, 4, 3, 4>;  // 32 x 64, K over 4 groups of waves
  using T1 = TileShape<4, 1, 1, 4, 4, 2>;  // 64 x 64, K over 2
  using T2 = TileShape<4, 1, 2, 4, 3, 2>;  // 128 x 64, K over 2
  using T3 = TileShape<4, 2, 2, 4, 4>;     // 128 x 128
  const long long cost[5] = {dense_cost<T0>(a, cus, 168), dense_cost<T1>(a, cus, 246), dense_cost<T2>(a, cus, 366),
                             dense_cost<T3>(a, cus, 500), dense_cost<Big>(a, cus, 980)};
  int best = 4;
  for (int i = 3; i >= 0; --i)
    if (cost[i] < cost[best]) best = i;
  switch (best) {
    case 0: return launch_tile<T0, FP8_DENSE>(a, (a.rows + T0::BT - 1) / T0::BT, 4, cus, s);
    case 1: return launch_tile<T1, FP8_DENSE>(a, (a.rows + T1::BT - 1) / T1::BT, 4, cus, s);
    case 2: return launch_tile<T2, FP8_DENSE>(a, (a.rows + T2::BT - 1) / T2::BT, 4, cus, s);
    case 3: return launch_tile<T3, FP8_DENSE>(a, (a.rows + T3::BT - 1) / T3::BT, 4, cus, s);
    default: return launch_tile<Big, FP8_DENSE>(a, (a.rows + Big::BT - 1) / Big::BT, 4, cus, s);
  }
}

using Few = TileShape<4, 1, 4, 4, 3>;  // 256 weight rows x 64 tokens, three stages: bound by the weights' stream
using Mid = TileShape<4, 2, 4, 4, 3>;  // 256 x 128, three stages

template <Fp8Mode MODE>
hipError_t launch_grouped(const Fp8Args& a, int tile, long long token_tiles, int cus, hipStream_t s) {
  if (tile == Few::BT) return launch_tile<Few, MODE>(a, token_tiles, 1, cus, s);
  if (tile == Mid::BT) return launch_tile<Mid, MODE>(a, token_tiles, 1, cus, s);
  return launch_tile<Big, MODE>(a, token_tiles, 1, cus, s);
}
}  // namespace

// Sorted rows per tile of the grouped products, by the rows that an expert has on average (64 experts, top-6, H 4096, I
// 1408, us with tiles of 64 / 128 / 256 rows: 47 rows 286 / 285 / -, 94 rows 377 / 327 / 364, 141 rows 496 / 384 / 408,
// 188 rows 597 / 449 / 438).
int fp8_tile_tokens(long long rows, int experts) {
  return rows < 48 * experts ? Few::BT : rows < 160 * experts ? Mid::BT : Big::BT;
}

hipError_t launch_fp8_tile(Fp8Mode mode, const Fp8Args& a, int tile, long long token_tiles, int cus, hipStream_t s) {
  switch (mode) {
    case FP8_DENSE: return launch_dense(a, cus, s);
    case FP8_GATE_UP: return launch_grouped<FP8_GATE_UP>(a, tile, token_tiles, cus, s);
    default: return launch_grouped<FP8_DOWN>(a, tile, token_tiles, cus, s);
  }
}

}  // namespace moe
