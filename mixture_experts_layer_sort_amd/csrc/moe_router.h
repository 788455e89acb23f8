// Scored routing and its gradient: arguments and launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

struct RouterArgs {
  const float* logits;  // [T, E], rows ldl apart
  long long ldl;
  int T, E, k;
  bool softmax, renorm;
  float scale;
  // choice
  const float* bias;    // [E] or null
  int G, KG, top;       // groups, kept ones, choices of a group that count
  int* ids;             // [T, k]; an input of the gradient
  float* w;             // [T, k]
  // gradient
  const float* d_w;     // [T, k]
  const uint8_t* mask;  // [T] or null
  bool accumulate;
  float* d_logits;      // [T, E], rows ldd apart
  long long ldd;
};

hipError_t launch_route_scores(const RouterArgs& a, hipStream_t s);
hipError_t launch_route_scores_backward(const RouterArgs& a, hipStream_t s);

}  // namespace moe
