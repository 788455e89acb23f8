// Router training: the arguments and launchers of the balance loss and of the
// router's gradient.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

struct BalanceArgs {
  const float* logits;         // [T, E]
  const int* ids;              // [T, k]
  const uint8_t* mask;         // [T] or null: every token is valid
  const int* seq;              // [S + 1] or null: one sequence of all T tokens
  int T, E, k, S;
  float coef, z_coef;
  // forward
  float* loss;                 // [2]
  int* counts;                 // [S, E]
  int* tokens;                 // [S]
  // backward (counts and tokens are inputs there)
  const float* topk_w;         // [T, k], null with d_topk_w
  const float* d_topk_w;       // [T, k] or null
  const float* d_loss;         // [2] or null
  float* d_logits;             // [T, E]
};

// Workspace of the forward pass (bytes into it).  Its size grows with T, E and S, so that of the largest batch serves
// all: records for the most chunks that T tokens or fewer can have (the number itself falls where the chunks grow).
struct BalanceWorkspace {
  size_t prob, count, zn, part, ticket, total;
};

constexpr int kBalanceWaves = 4;      // waves per block of the forward pass
constexpr int kBalanceChunks = 1024;  // token chunks (blocks), at most
inline int balance_chunk(int T) {     // tokens per chunk: four per wave at least
  const int c = (T + kBalanceChunks - 1) / kBalanceChunks;
  return c < 4 * kBalanceWaves ? 4 * kBalanceWaves : c;
}
inline int balance_chunks(int T) { return (T + balance_chunk(T) - 1) / balance_chunk(T); }
constexpr int kBalanceSlice = 32;     // experts per block of the reduction
inline int balance_slices(int E) { return (E + kBalanceSlice - 1) / kBalanceSlice; }

inline BalanceWorkspace balance_workspace(int T, int E, int S) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  const size_t most = ((size_t)T + 4 * kBalanceWaves - 1) / (4 * kBalanceWaves);
  const size_t slots = (most < kBalanceChunks ? most : kBalanceChunks) + S;
  BalanceWorkspace w;
  w.prob = 0;
  w.count = w.prob + up(slots * E * 4);
  w.zn = w.count + up(slots * E * 4);
  w.part = w.zn + up(slots * 8);
  w.ticket = w.part + up((size_t)S * (balance_slices(E) + 1) * 8);
  w.total = w.ticket + 256;
  return w;
}

hipError_t launch_balance_loss(const BalanceArgs& a, uint8_t* ws, hipStream_t s);
hipError_t launch_route_backward(const BalanceArgs& a, int cus, hipStream_t s);

}  // namespace moe
