// lm_kernels.h -- launch functions of the embedding, gradient-clipping and
// cross-entropy kernels (internal to libnvfp4.so; the public interface is
// include/nvfp4.h).  Types are the public NVFP4_TYPE_* values.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "../../include/nvfp4.h"

namespace nvfp4 {

int num_cus();  // compute units of the current device

struct EmbedArgs {
  const void* ids;
  int ids_type;
  int64_t n, vocab, dim;
  float scale;
};

hipError_t launch_embed(const EmbedArgs& a, const void* w, int w_type, int64_t ldw, void* out,
                        int out_type, int64_t ldo, hipStream_t s);

int64_t embed_grad_workspace_bytes(int64_t n, int64_t vocab, int64_t dim);
hipError_t launch_embed_grad(const EmbedArgs& a, const void* dy, int dy_type, int64_t ld_dy,
                             void* dw, int dw_type, int64_t ld_dw, bool accumulate, void* ws,
                             hipStream_t s);

hipError_t launch_grad_sumsq(const nvfp4_grad* list, int64_t count, double* partials,
                             hipStream_t s);
hipError_t launch_grad_clip(const nvfp4_grad* list, int64_t count, const double* partials,
                            double max_norm, float* norm_out, hipStream_t s);

hipError_t launch_grad_scale(const nvfp4_grad* list, int64_t count, const float* factor,
                             hipStream_t s);

// Softmax cross entropy of a head: loss (and lse) of every token; grad: dh and
// dw as well.  piece: tokens per piece of the gradient (0: chosen here).
struct CeCall {
  const void* h;
  const void* w;
  int64_t ldh, ldw, T, V, D;
  const void* targets;
  int targets_type;
  const float* row_weight;
  int64_t piece;
  float* loss;
  float* lse;
  void* dh;
  void* dw;
  int64_t ld_dh, ld_dw;
  bool grad;
  void* ws;
};
int64_t ce_workspace_bytes(int64_t T, int64_t V, int64_t D, bool grad, int64_t piece);
hipError_t launch_ce(const CeCall& c, hipStream_t s);

}  // namespace nvfp4
