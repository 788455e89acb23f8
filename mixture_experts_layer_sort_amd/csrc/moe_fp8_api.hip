// C ABI entry points of the block-128 fp8 products and of the router's
// training operators: host-side argument checks, then launches on the caller's
// stream.  Nothing here allocates device memory, synchronises or reads device
// data.
#include <algorithm>
#include <atomic>

#include "../../include/moe.h"
#include "moe_balance.h"
#include "moe_fp8.h"

using namespace moe;

namespace {

constexpr int kMaxDevices = 64;
std::atomic<int> g_cus[kMaxDevices];  // compute units per device

int cu_count() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return 256;
  int v = g_cus[dev].load(std::memory_order_relaxed);
  if (v > 0) return v;
  if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v <= 0) v = 256;
  g_cus[dev].store(v, std::memory_order_relaxed);
  return v;
}

moe_status launched(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }
bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
template <class... P>
bool aligned4(const P*... p) {  // null is
  return (aligned(p, 4) && ...);
}
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// rows and columns of one weight matrix
bool fp8_shape_ok(int32_t N, int32_t K) {
  return N >= 1 && N <= (1 << 20) && K >= 16 && K % 16 == 0 && K <= (1 << 20);
}

struct LinearWorkspace {
  size_t xq, xs, total;  // or the sums of fp8_splits() at 0
};
LinearWorkspace linear_workspace(size_t M, size_t N, size_t K) {
  const size_t kb = (K + kFp8Blk - 1) / kFp8Blk;
  LinearWorkspace w;
  w.xq = 0;
  w.xs = up256(M * kb * kFp8Blk);
  w.total = std::max(w.xs + up256(M * kb * sizeof(float)), up256(fp8_split_bytes((int)M, (int)N, (int)K)));
  return w;
}

// experts: codes and scales of x, the intermediate (bf16 rows of the streaming kernel; codes and scales of the tiled
// one: I + I / 32 bytes a row, less than the 2 I of bf16), and the token tiles
struct ExpertsWorkspace {
  size_t xq, xs, h, hs, tiles, ntiles, total;
};
// token tiles of `pairs` sorted rows, at most: every expert that has rows may end inside one
size_t max_tiles(const moe_shape* s, size_t pairs, int tile) {
  const size_t E = s->num_experts;
  return pairs / tile + (pairs < E ? pairs : E);
}
ExpertsWorkspace experts_workspace(const moe_shape* s) {
  const size_t T = s->max_tokens, H = s->hidden, P = T * s->top_k, I = s->inter;
  ExpertsWorkspace w;
  w.xq = 0;
  w.xs = up256(T * H);
  w.h = w.xs + up256(T * (H / kFp8Blk) * sizeof(float));
  w.hs = w.h + up256(P * I);
  w.tiles = w.h + up256(P * I) + up256(P * I);
  w.ntiles = w.tiles + up256(max_tiles(s, P, kFp8TileTokensMin) * sizeof(int4));
  w.total = w.ntiles + 256;
  return w;
}

moe_status check_experts(const moe_shape* s) {
  const moe_status st = moe_check_shape(s);
  if (st != MOE_OK) return st;
  return s->dtype == MOE_BF16 && s->activation == MOE_SWIGLU ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

moe_status check_router(int32_t T, int32_t E, int32_t k, const uint8_t*, int32_t num_seqs, const int32_t* seq_offsets,
                        float coef, float z_coef) {
  if (T < 0) return MOE_ERR_INVALID_ARG;
  if (E < 1 || E > 1024 || k < 1 || k > 32 || k > E) return MOE_ERR_UNSUPPORTED;
  if ((long long)T * k > (1LL << 24) || num_seqs > 65536) return MOE_ERR_UNSUPPORTED;
  if (num_seqs < 1 || (num_seqs > 1 && !seq_offsets)) return MOE_ERR_INVALID_ARG;
  if (!(coef >= -3.0e38f && coef <= 3.0e38f && z_coef >= -3.0e38f && z_coef <= 3.0e38f)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_fp8_quantize_weights(int32_t count, int32_t rows, int32_t K, const float* w, void* codes,
                                    float* scales, hipStream_t stream) {
  if (count < 0) return MOE_ERR_INVALID_ARG;
  if (!fp8_shape_ok(rows, K)) return MOE_ERR_UNSUPPORTED;
  const long long blocks = (long long)count * ((rows + 127) / 128) * ((K + 127) / 128);
  if (blocks >= 1LL << 24) return MOE_ERR_UNSUPPORTED;  // a launch has fewer than 2^32 threads; 256 per block here
  if (count == 0) return MOE_OK;
  if (!w || !codes || !scales || !aligned(w, 16) || !aligned(codes, 4) || !aligned(scales, 4))
    return MOE_ERR_INVALID_ARG;
  return launched(launch_fp8_quantize_weights(count, rows, K, w, (uint8_t*)codes, scales, stream));
}

size_t moe_fp8_linear_workspace_bytes(int32_t max_M, int32_t N, int32_t K) {
  if (max_M < 1 || max_M > (1 << 24) || !fp8_shape_ok(N, K)) return 0;
  return linear_workspace(max_M, N, K).total;
}

moe_status moe_fp8_linear(int32_t M, int32_t N, int32_t K, const void* codes, const float* scales, const uint16_t* x,
                          int64_t x_stride, uint16_t* out, int64_t out_stride, void* ws, size_t ws_bytes,
                          hipStream_t stream) {
  if (!fp8_shape_ok(N, K)) return MOE_ERR_UNSUPPORTED;
  if (M < 0 || M > (1 << 24)) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  if (!codes || !scales || !x || !out || !ws) return MOE_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(scales, 4) || !aligned(x, 16) || !aligned(out, 2) || !aligned(ws, 256))
    return MOE_ERR_INVALID_ARG;
  if (x_stride < K || x_stride % 8 || out_stride < N) return MOE_ERR_INVALID_ARG;
  if (x_stride > (1LL << 32) || out_stride > (1LL << 32)) return MOE_ERR_UNSUPPORTED;
  if (ws_bytes < linear_workspace(M, N, K).total) return MOE_ERR_WORKSPACE;
  Fp8Args a = {};
  a.w = (const uint8_t*)codes;
  a.wsc = scales;
  a.x = x;
  a.ldx = x_stride;
  a.out = out;
  a.ldo = out_stride;
  a.rows = M, a.E = 1, a.N = N, a.K = K, a.k = 1;
  a.splits = fp8_splits(M, N, K);
  if (a.splits > 1) {
    a.part = (float*)ws;
    return launched(launch_fp8_split(a, stream));
  }
  if (fp8_decode_fits(M, K)) return launched(launch_fp8_stream(FP8_DENSE, a, cu_count(), stream));
  const LinearWorkspace W = linear_workspace(M, N, K);
  uint8_t* xq = (uint8_t*)ws + W.xq;
  float* xs = (float*)((uint8_t*)ws + W.xs);
  hipError_t e = launch_fp8_quantize_rows(M, K, x, x_stride, xq, xs, stream);
  if (e != hipSuccess) return MOE_ERR_LAUNCH;
  a.xq = xq;
  a.xs = xs;
  a.xrows = M;
  if (M <= 32) return launched(launch_fp8_stream(FP8_DENSE, a, cu_count(), stream));
  return launched(launch_fp8_tile(FP8_DENSE, a, 0, 0, cu_count(), stream));
}

size_t moe_fp8_experts_workspace_bytes(const moe_shape* shape) {
  return check_experts(shape) == MOE_OK ? experts_workspace(shape).total : 0;
}

moe_status moe_fp8_experts(const moe_shape* s, int32_t T, const void* w13_codes, const float* w13_scales,
                           const void* w2_codes, const float* w2_scales, const int32_t* offsets,
                           const int32_t* sorted_pairs, const uint16_t* x, uint16_t* y, void* ws, size_t ws_bytes,
                           hipStream_t stream) {
  const moe_status st = check_experts(s);
  if (st != MOE_OK) return st;
  if (T < 0 || T > s->max_tokens) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!w13_codes || !w13_scales || !w2_codes || !w2_scales || !offsets || !sorted_pairs || !x || !y || !ws)
    return MOE_ERR_INVALID_ARG;
  if (!aligned(w13_codes, 16) || !aligned(w2_codes, 16) || !aligned(x, 16) || !aligned(y, 16) || !aligned(ws, 256))
    return MOE_ERR_INVALID_ARG;
  if (!aligned4(w13_scales, w2_scales, offsets, sorted_pairs)) return MOE_ERR_INVALID_ARG;
  const ExpertsWorkspace W = experts_workspace(s);
  if (ws_bytes < W.total) return MOE_ERR_WORKSPACE;
  uint8_t* base = (uint8_t*)ws;
  const int cus = cu_count();
  Fp8Args a = {};
  a.w = (const uint8_t*)w13_codes;
  a.wsc = w13_scales;
  a.x = x;
  a.ldx = s->hidden;
  a.offsets = offsets;
  a.pairs = sorted_pairs;
  a.out = (uint16_t*)(base + W.h);
  a.ldo = s->inter;
  a.rows = T * s->top_k, a.E = s->num_experts, a.N = 2 * s->inter, a.K = s->hidden, a.k = s->top_k;
  a.limit = s->gate_up_limit;
  hipError_t e;
  // The tiled kernel; the streaming one for up to 8 tokens of 48 rows (H 4096, I 1408, 64 experts, top-6, T = 8: 125 us
  // against 146; H 7168, I 2048, 256 experts, top-8, T = 4: 254 against 258, T = 8: 460 against 413; at T = 16 and uneven
  // experts 102 against 77), where the tiles (128 intermediate columns each) would leave half of the compute units idle,
  // and for gathered rows beyond the tiled kernel's 32-bit addresses.
  const long long P = (long long)T * s->top_k;
  if ((T > 8 || P > 48) && P * (s->inter / 128) > cus / 2 && (long long)T * s->hidden < (1LL << 31)) {
    const int tile = fp8_tile_tokens(P, s->num_experts);
    const long long ntok = (long long)max_tiles(s, P, tile);
    float* xs = (float*)(base + W.xs);
    int4* tiles = (int4*)(base + W.tiles);
    int* ntiles = (int*)(base + W.ntiles);
    e = launch_fp8_quantize_tokens(T, s->hidden, x, base + W.xq, xs, offsets, s->num_experts, tile, tiles,
                                   ntiles, stream);
    if (e != hipSuccess) return MOE_ERR_LAUNCH;
    a.xq = base + W.xq;
    a.xs = xs;
    a.xrows = T;
    a.tiles = tiles;
    a.ntiles = ntiles;
    a.hq = base + W.h;
    a.hs = (float*)(base + W.hs);
    e = launch_fp8_tile(FP8_GATE_UP, a, tile, ntok, cus, stream);
    if (e != hipSuccess) return MOE_ERR_LAUNCH;
    a.w = (const uint8_t*)w2_codes;
    a.wsc = w2_scales;
    a.xq = a.hq;
    a.xs = a.hs;
    a.xrows = a.rows;
    a.out = y;
    a.ldo = s->hidden;
    a.N = s->hidden, a.K = s->inter;
    return launched(launch_fp8_tile(FP8_DOWN, a, tile, ntok, cus, stream));
  }
  a.cap = fp8_block_rows(T, a.K);
  e = launch_fp8_stream(FP8_GATE_UP, a, cus, stream);
  if (e != hipSuccess) return MOE_ERR_LAUNCH;
  a.w = (const uint8_t*)w2_codes;
  a.wsc = w2_scales;
  a.x = a.out;
  a.ldx = s->inter;
  a.out = y;
  a.ldo = s->hidden;
  a.N = s->hidden, a.K = s->inter;
  a.cap = fp8_block_rows(T, a.K);
  return launched(launch_fp8_stream(FP8_DOWN, a, cus, stream));
}

size_t moe_balance_loss_workspace_bytes(int32_t T, int32_t E, int32_t num_seqs) {
  if (T < 1 || T > (1 << 24) || E < 1 || E > 1024 || num_seqs < 1 || num_seqs > 65536) return 0;
  return balance_workspace(T, E, num_seqs).total;
}

moe_status moe_balance_loss(int32_t T, int32_t E, int32_t k, const float* logits, const int32_t* topk_ids,
                            const uint8_t* token_mask, int32_t num_seqs, const int32_t* seq_offsets,
                            float balance_coef, float z_coef, float* loss, int32_t* counts, int32_t* tokens, void* ws,
                            size_t ws_bytes, hipStream_t stream) {
  const moe_status st = check_router(T, E, k, token_mask, num_seqs, seq_offsets, balance_coef, z_coef);
  if (st != MOE_OK || T == 0) return st;
  if (!logits || !topk_ids || !loss || !counts || !tokens || !ws || !aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  if (!aligned4(logits, topk_ids, seq_offsets, loss, counts, tokens)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < balance_workspace(T, E, num_seqs).total) return MOE_ERR_WORKSPACE;
  BalanceArgs a = {};
  a.logits = logits, a.ids = topk_ids, a.mask = token_mask, a.seq = seq_offsets;
  a.T = T, a.E = E, a.k = k, a.S = num_seqs;
  a.coef = balance_coef, a.z_coef = z_coef;
  a.loss = loss, a.counts = counts, a.tokens = tokens;
  return launched(launch_balance_loss(a, (uint8_t*)ws, stream));
}

moe_status moe_route_backward(int32_t T, int32_t E, int32_t k, const float* logits, const int32_t* topk_ids,
                              const float* topk_w, const float* d_topk_w, const uint8_t* token_mask, int32_t num_seqs,
                              const int32_t* seq_offsets, float balance_coef, float z_coef, const int32_t* counts,
                              const int32_t* tokens, const float* d_loss, float* d_logits, hipStream_t stream) {
  const moe_status st = check_router(T, E, k, token_mask, num_seqs, seq_offsets, balance_coef, z_coef);
  if (st != MOE_OK || T == 0) return st;
  if (!logits || !d_logits || (!d_topk_w && !d_loss)) return MOE_ERR_INVALID_ARG;
  if (d_topk_w && (!topk_w || !topk_ids)) return MOE_ERR_INVALID_ARG;
  if (d_loss && (!counts || !tokens)) return MOE_ERR_INVALID_ARG;
  if (!aligned4(logits, topk_ids, topk_w, d_topk_w, seq_offsets, counts, tokens, d_loss, d_logits))
    return MOE_ERR_INVALID_ARG;
  BalanceArgs a = {};
  a.logits = logits, a.ids = topk_ids, a.mask = token_mask, a.seq = seq_offsets;
  a.T = T, a.E = E, a.k = k, a.S = num_seqs;
  a.coef = balance_coef, a.z_coef = z_coef;
  a.counts = const_cast<int*>(counts), a.tokens = const_cast<int*>(tokens);
  a.topk_w = topk_w, a.d_topk_w = d_topk_w, a.d_loss = d_loss, a.d_logits = d_logits;
  return launched(launch_route_backward(a, cu_count(), stream));
}

}  // extern "C"
