// The end of an expert block: weighted sum, shared expert, norms and residual;
// and its gradients.  Arguments and launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

struct NormArgs {
  int T, H, k;
  const uint16_t* y;         // [T k, H], null with k == 0
  const float* w;            // [T, k]
  const uint16_t* shared;    // [T, H] or null
  const float* gate;         // [T] or null: 1
  const uint16_t* residual;  // [T, H] or null: 0
  const uint16_t* post;      // [H] or null: no norm of the sum
  const uint16_t* next;      // [H] or null: no next norm
  float eps, scale;
  uint16_t* out;             // [T, H]; an input of the gradient (null without next)
  uint16_t* normed;          // [T, H] with next
  // gradient
  const uint16_t* d_out;     // [T, H] or null: 0
  const uint16_t* d_normed;  // [T, H] with next
  uint16_t* d_residual;      // [T, H] or null
  uint16_t* d_y;             // [T k, H] or null
  float* d_w;                // [T, k] or null
  uint16_t* d_shared;        // [T, H] or null
  float* d_gate;             // [T] or null
  float* d_post;             // [H] with post
  float* d_next;             // [H] with next
  float* part;               // workspace: [blocks][2][H]
};

// Blocks of the gradient's first launch, each of which adds its tokens' parts of the weights' gradients: as many as run
// at once on 256 compute units of 8 waves (16 columns a thread).
inline int norm_blocks(int T, int H) {
  const int waves = (H + 1023) / 1024, most = 256 * (waves < 8 ? 8 / waves : 1);
  return T < most ? T : most;
}
inline size_t norm_backward_bytes(int T, int H) {
  const size_t n = (size_t)norm_blocks(T, H) * 2 * H * sizeof(float);
  return (n + 255) / 256 * 256;
}

hipError_t launch_combine_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_combine_norm_backward(const NormArgs& a, hipStream_t s);

}  // namespace moe
