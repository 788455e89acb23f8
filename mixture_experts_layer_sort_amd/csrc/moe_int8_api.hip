// C ABI entry points of the products on 8-bit integer weights: host-side
// argument checks, then launches on the caller's stream.  Nothing here allocates
// device memory, synchronises or reads device data.
#include <algorithm>
#include <atomic>

#include "../../include/moe.h"
#include "moe_int8.h"

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

// Rows and columns of one weight matrix; 128 127 2^17 < 2^31: sums fit 32 bits.
bool int8_shape_ok(int32_t N, int32_t K) {
  return N >= 1 && N <= (1 << 20) && K >= 16 && K % 16 == 0 && K <= (1 << 17);
}

struct LinearWorkspace {
  size_t xq, xs, sums, total;
};
LinearWorkspace linear_workspace(size_t M, int N, int K) {
  LinearWorkspace w;
  w.xq = 0;
  w.xs = up256(M * int8_pad(K));
  w.sums = w.xs + up256(M * sizeof(float));
  w.total = w.sums + up256(int8_split_bytes((int)M, N, K));
  return w;
}

// Codes and scales of x, the intermediate as bf16 and as codes and scales, and the token tiles.
struct ExpertsWorkspace {
  size_t xq, xs, h, hq, hs, tiles, ntiles, total;
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
  w.h = w.xs + up256(T * sizeof(float));
  w.hq = w.h + up256(P * I * 2);
  w.hs = w.hq + up256(P * I);
  w.tiles = w.hs + up256(P * sizeof(float));
  w.ntiles = w.tiles + up256(max_tiles(s, P, kInt8TileTokensMin) * sizeof(int4));
  w.total = w.ntiles + 256;
  return w;
}

// Experts by the streaming kernel: up to 8 rows an expert while the tiles (128 intermediate columns of an expert that has
// rows) are fewer than 12 rounds of the GPU, and up to 32 rows while they are a quarter of one round.  Us, streaming / tiled:
// 256 experts of 7168 x 2048, top-8, 16 tokens 734 / 765, 24 893 / 922, 96 1744 / 1706; 64 of 4096 x 1408, top-6, 8 tokens
// 130 / 150, 24 184 / 215, 64 221 / 229, 128 243 / 231; 8 of 4096 x 7168, top-2, 32 tokens 137 / 160, 64 174 / 161; 2 of 4096
// x 1024, 64 tokens 28 / 40.
bool int8_streams(int P, int E, int I, int cus) {
  const long long columns = I / 128;
  return (P <= 8LL * E && (P < E ? P : E) * columns < 12LL * cus) || (P <= 32LL * E && E * columns <= cus / 4);
}

moe_status check_experts(const moe_shape* s) {
  const moe_status st = moe_check_shape(s);
  if (st != MOE_OK) return st;
  if (s->hidden > (1 << 17) || s->inter > (1 << 17)) return MOE_ERR_UNSUPPORTED;
  return s->dtype == MOE_BF16 && s->activation == MOE_SWIGLU ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

moe_status moe_int8_quantize_weights(int32_t count, int32_t rows, int32_t K, const float* w, void* codes,
                                     float* scales, hipStream_t stream) {
  if (count < 0) return MOE_ERR_INVALID_ARG;
  if (!int8_shape_ok(rows, K)) return MOE_ERR_UNSUPPORTED;
  if ((long long)count * rows >= 1LL << 24) return MOE_ERR_UNSUPPORTED;  // a launch has fewer than 2^32 threads
  if (count == 0) return MOE_OK;
  if (!w || !codes || !scales || !aligned(w, 16) || !aligned(codes, 4) || !aligned(scales, 4))
    return MOE_ERR_INVALID_ARG;
  return launched(launch_int8_quantize_weights(count, rows, K, w, (int8_t*)codes, scales, stream));
}

size_t moe_int8_linear_workspace_bytes(int32_t max_M, int32_t N, int32_t K) {
  if (max_M < 1 || max_M > (1 << 24) || !int8_shape_ok(N, K)) return 0;
  return linear_workspace(max_M, N, K).total;
}

moe_status moe_int8_linear(int32_t M, int32_t N, int32_t K, const void* codes, const float* scales, const uint16_t* x,
                           int64_t x_stride, uint16_t* out, int64_t out_stride, void* ws, size_t ws_bytes,
                           hipStream_t stream) {
  if (!int8_shape_ok(N, K)) return MOE_ERR_UNSUPPORTED;
  if (M < 0 || M > (1 << 24)) return MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  if (!codes || !scales || !x || !out || !ws) return MOE_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(scales, 4) || !aligned(x, 16) || !aligned(out, 2) || !aligned(ws, 256))
    return MOE_ERR_INVALID_ARG;
  if (x_stride < K || x_stride % 8 || out_stride < N) return MOE_ERR_INVALID_ARG;
  if (x_stride > (1LL << 32) || out_stride > (1LL << 32)) return MOE_ERR_UNSUPPORTED;
  const LinearWorkspace W = linear_workspace(M, N, K);
  if (ws_bytes < W.total) return MOE_ERR_WORKSPACE;
  Int8Args a = {};
  a.w = (const int8_t*)codes;
  a.wsc = scales;
  a.x = x;
  a.ldx = x_stride;
  a.out = out;
  a.ldo = out_stride;
  a.rows = M, a.E = 1, a.N = N, a.K = K, a.k = 1;
  if (int8_decode_fits(M, K)) {
    a.cap = M;
    return launched(launch_int8_stream(INT8_DENSE, a, cu_count(), stream));
  }
  int8_t* xq = (int8_t*)ws + W.xq;
  float* xs = (float*)((uint8_t*)ws + W.xs);
  a.splits = int8_splits(M, N, K);
  a.sums = (int*)((uint8_t*)ws + W.sums);
  const hipError_t e = launch_int8_quantize_rows(M, K, x, x_stride, xq, xs, stream);
  if (e != hipSuccess) return MOE_ERR_LAUNCH;
  a.xq = xq;
  a.xs = xs;
  a.xrows = M;
  // 17 to 32 rows: the streaming kernel while it is one round of blocks of 16 weight rows (17 rows of 2816 x 4096 10.1 us,
  // tiled 11.4; of 7168 x 2048 11.1 and 9.4; of 18432 x 7168 46 and 26)
  if (a.splits <= 1 && (M <= 16 || (M <= 32 && N <= 16 * cu_count()))) return launched(launch_int8_stream(INT8_DENSE, a, cu_count(), stream));
  return launched(launch_int8_tile(INT8_DENSE, a, 0, 0, cu_count(), stream));
}

size_t moe_int8_experts_workspace_bytes(const moe_shape* shape) {
  return check_experts(shape) == MOE_OK ? experts_workspace(shape).total : 0;
}

moe_status moe_int8_experts(const moe_shape* s, int32_t T, const void* w13_codes, const float* w13_scales,
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
  const int cus = cu_count(), H = s->hidden, I = s->inter, P = T * s->top_k;
  int8_t *xq = (int8_t*)base + W.xq, *hq = (int8_t*)base + W.hq;
  float *xs = (float*)(base + W.xs), *hs = (float*)(base + W.hs);
  uint16_t* h = (uint16_t*)(base + W.h);

  Int8Args up = {};  // gate / up product
  up.w = (const int8_t*)w13_codes;
  up.wsc = w13_scales;
  up.x = x;
  up.ldx = H;
  up.xq = xq;
  up.xs = xs;
  up.xrows = T;
  up.offsets = offsets;
  up.pairs = sorted_pairs;
  up.tiles = (int4*)(base + W.tiles);
  up.ntiles = (int*)(base + W.ntiles);
  up.out = h;
  up.ldo = I;
  up.rows = P, up.E = s->num_experts, up.N = 2 * I, up.K = H, up.k = s->top_k;
  up.limit = s->gate_up_limit;
  Int8Args down = up;
  down.w = (const int8_t*)w2_codes;
  down.wsc = w2_scales;
  down.x = h;
  down.ldx = I;
  down.xq = hq;
  down.xs = hs;
  down.xrows = P;
  down.out = y;
  down.ldo = H;
  down.N = H, down.K = I;

  if (!int8_streams(P, s->num_experts, I, cus) && (long long)T * H < (1LL << 31)) {  // 32-bit offsets of gathered rows
    const int tile = int8_tile_tokens(P, s->num_experts);
    const long long ntok = (long long)max_tiles(s, P, tile);
    if (launch_int8_quantize_tokens(T, H, x, xq, xs, offsets, s->num_experts, tile, (int4*)(base + W.tiles),
                                    (int*)(base + W.ntiles), stream) != hipSuccess ||
        launch_int8_tile(INT8_GATE_UP, up, tile, ntok, cus, stream) != hipSuccess ||
        launch_int8_quantize_rows(P, I, h, I, hq, hs, stream) != hipSuccess)
      return MOE_ERR_LAUNCH;
    return launched(launch_int8_tile(INT8_DOWN, down, tile, ntok, cus, stream));
  }
  up.cap = int8_block_rows(INT8_GATE_UP, up, T, cus);
  if (up.cap == 0 && launch_int8_quantize_rows(T, H, x, H, xq, xs, stream) != hipSuccess) return MOE_ERR_LAUNCH;
  if (launch_int8_stream(INT8_GATE_UP, up, cus, stream) != hipSuccess) return MOE_ERR_LAUNCH;
  down.cap = int8_block_rows(INT8_DOWN, down, T, cus);
  if (down.cap == 0 && launch_int8_quantize_rows(P, I, h, I, hq, hs, stream) != hipSuccess) return MOE_ERR_LAUNCH;
  return launched(launch_int8_stream(INT8_DOWN, down, cus, stream));
}

}  // extern "C"
