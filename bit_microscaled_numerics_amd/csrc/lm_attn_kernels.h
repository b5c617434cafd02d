// lm_attn_kernels.h -- launch functions of the query / key norm and rotation and of the
// attention kernels (internal to libnvfp4.so; the public interface is include/nvfp4.h).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "../../include/nvfp4.h"

namespace nvfp4 {

// in: q, k and, in the gradient, the incoming dq, dk; out: their results.
struct RopeCall {
  nvfp4_rope r;
  nvfp4_heads q, k, dq, dk, q_out, k_out;
  void* dq_weight;
  void* dk_weight;
  bool grad;
  void* ws;
};
int64_t rope_workspace_bytes(int64_t T, int64_t Hq, int64_t Hkv, int64_t D);
hipError_t launch_rope(const RopeCall& c, hipStream_t s);

struct AttnCall {
  nvfp4_attn a;
  nvfp4_heads q, k, v, out, dout, dq, dk, dv;
  float* lse;   // written by the forward call, read by the gradient
  void* ws;
};
int64_t attn_workspace_bytes(const nvfp4_attn& a, bool grad);
hipError_t launch_attn(const AttnCall& c, hipStream_t s);
hipError_t launch_attn_grad(const AttnCall& c, hipStream_t s);

}  // namespace nvfp4
