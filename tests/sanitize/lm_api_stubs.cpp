// lm_api_stubs.cpp -- host stand-ins for what lm_api.cpp calls below it: the
// launchers and workspace queries of the embedding, cross-entropy and
// gradient-list kernels, and one HIP runtime function.  Each launcher counts
// its calls and reads the whole list it is given, as the real ones do.
#include <hip/hip_runtime_api.h>

#include <cstdint>

#include "api_common.h"
#include "lm_kernels.h"

int g_launches = 0;
int64_t g_elements = 0;

extern "C" const char* hipGetErrorString(hipError_t) { return "stub"; }
extern "C" const char* nvfp4_last_error(void) { return nvfp4::api::g_last_error; }

namespace nvfp4 {
static hipError_t ok() {
  ++g_launches;
  return hipSuccess;
}
static hipError_t walk(const nvfp4_grad* list, int64_t count) {
  for (int64_t i = 0; i < count; ++i) g_elements += list[i].numel;
  return ok();
}
hipError_t launch_embed(const EmbedArgs&, const void*, int, int64_t, void*, int, int64_t,
                        hipStream_t) {
  return ok();
}
int64_t embed_grad_workspace_bytes(int64_t n, int64_t, int64_t dim) { return n * 8 + n / 64 * dim * 4; }
hipError_t launch_embed_grad(const EmbedArgs&, const void*, int, int64_t, void*, int, int64_t, bool,
                             void*, hipStream_t) {
  return ok();
}
hipError_t launch_grad_sumsq(const nvfp4_grad* l, int64_t n, double*, hipStream_t) { return walk(l, n); }
hipError_t launch_grad_clip(const nvfp4_grad* l, int64_t n, const double*, double, float*,
                            hipStream_t) {
  return walk(l, n);
}
hipError_t launch_grad_scale(const nvfp4_grad* l, int64_t n, const float*, hipStream_t) {
  return walk(l, n);
}
int64_t ce_workspace_bytes(int64_t T, int64_t, int64_t, bool grad, int64_t) {
  return 256 + (grad ? T * 4 : 0);
}
hipError_t launch_ce(const CeCall&, hipStream_t) { return ok(); }
}  // namespace nvfp4
