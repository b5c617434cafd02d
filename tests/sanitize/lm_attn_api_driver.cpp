// lm_attn_api_driver.cpp -- drives the norm, rotation and attention entry points on the host
// (their launchers are the stubs at the end) with valid, invalid and extreme arguments under
// AddressSanitizer and UndefinedBehaviorSanitizer: validation returns the documented status
// and overflows no size.
#include <cstdint>
#include <cstdio>

#include "api_common.h"
#include "lm_attn_kernels.h"
#include "nvfp4.h"

static int failures = 0, launches = 0;
#define EXPECT(call, want)                                                                  \
  do {                                                                                      \
    const long long got_ = (long long)(call);                                               \
    if (got_ != (long long)(want)) {                                                        \
      std::fprintf(stderr, "line %d: %s returned %lld, expected %lld (%s)\n", __LINE__, #call, \
                   got_, (long long)(want), nvfp4_last_error());                            \
      ++failures;                                                                           \
    }                                                                                       \
  } while (0)

alignas(256) static unsigned char dev[1 << 12];   // stands in for device memory

int main() {
  void* P = dev;
  float* F = reinterpret_cast<float*>(dev);
  const int OK = NVFP4_OK, S = NVFP4_ERR_SHAPE;
  const int64_t wild[] = {INT64_MIN, -1, INT64_MAX, int64_t(1) << 62, (int64_t(1) << 40) + 1};
  const nvfp4_rope r{5, 2, 1, 16, 8, NVFP4_TYPE_BF16, NVFP4_TYPE_F32, NVFP4_TYPE_I32, 0, 1, 1e-6f, P, P, P, F};
  const nvfp4_heads x{P, 0, 32, 16}, y{P, 0, 16, 16};
  EXPECT(nvfp4_qk_norm_rope(&r, &x, &y, &x, &y, nullptr), OK);
  EXPECT(nvfp4_qk_norm_rope_grad(&r, &x, &y, &x, &y, &x, &y, P, nullptr, P, 4096, nullptr), OK);
  for (int64_t w : wild) {
    for (int64_t nvfp4_rope::*f : {&nvfp4_rope::T, &nvfp4_rope::Hq, &nvfp4_rope::Hkv, &nvfp4_rope::D,
                                   &nvfp4_rope::rot}) {
      nvfp4_rope b = r;
      b.*f = w;
      EXPECT(nvfp4_qk_norm_rope(&b, &x, &y, &x, &y, nullptr), S);
    }
    for (int64_t nvfp4_heads::*f : {&nvfp4_heads::token, &nvfp4_heads::head}) {
      nvfp4_heads b = x;
      b.*f = w;
      EXPECT(nvfp4_qk_norm_rope(&r, &b, &y, &x, &y, nullptr), S);
    }
    EXPECT(nvfp4_qk_norm_rope_grad_workspace_bytes(w, 1, 1, 8), S);
    EXPECT(nvfp4_qk_norm_rope_grad_workspace_bytes(4, w, 1, 8), S);
    EXPECT(nvfp4_qk_norm_rope_grad_workspace_bytes(4, 1, 1, w), S);
  }
  const nvfp4_attn a{2, 4, 6, 4, 2, 16, nullptr, nullptr, 0, 1, 0, 0.25f};
  const nvfp4_heads q{P, 256, 64, 16}, k{P, 192, 32, 16}, o{dev + 1024, 256, 64, 16}, gq{dev + 2048, 256, 64, 16};
  const nvfp4_heads gk{dev + 3088, 192, 32, 16}, gv{dev + 3600, 192, 32, 16};
  EXPECT(nvfp4_attention(&a, &q, &k, &k, &o, F, P, 4096, nullptr), OK);
  EXPECT(nvfp4_attention_grad(&a, &q, &q, &k, &k, &o, F, &gq, &gk, &gv, P, 4096, nullptr), OK);
  for (int64_t w : wild) {
    for (int64_t nvfp4_attn::*f : {&nvfp4_attn::batch, &nvfp4_attn::Tq, &nvfp4_attn::Tk, &nvfp4_attn::Hq,
                                   &nvfp4_attn::Hkv, &nvfp4_attn::D}) {
      nvfp4_attn b = a;
      b.*f = w;
      EXPECT(nvfp4_attention(&b, &q, &k, &k, &o, F, P, 4096, nullptr), S);
      EXPECT(nvfp4_attention_workspace_bytes(&b, 1), S);
    }
    for (int64_t nvfp4_heads::*f : {&nvfp4_heads::batch, &nvfp4_heads::token, &nvfp4_heads::head}) {
      nvfp4_heads b = q;
      b.*f = w;
      EXPECT(nvfp4_attention(&a, &b, &k, &k, &o, F, P, 4096, nullptr), S);
      b = k;
      b.*f = w;
      EXPECT(nvfp4_attention_grad(&a, &q, &q, &k, &k, &o, F, &gq, &gk, &b, P, 4096, nullptr), S);
    }
  }
  nvfp4_attn b = a;
  b.window = INT64_MAX;
  EXPECT(nvfp4_attention(&b, &q, &k, &k, &o, F, P, 4096, nullptr), OK);
  std::printf("unexpected statuses: %d, launches %d\n", failures, launches);
  return failures != 0;
}

extern "C" const char* hipGetErrorString(hipError_t) { return "stub"; }
extern "C" const char* nvfp4_last_error(void) { return nvfp4::api::g_last_error; }

namespace nvfp4 {
static hipError_t ok() {
  ++launches;
  return hipSuccess;
}
int64_t rope_workspace_bytes(int64_t T, int64_t, int64_t, int64_t D) { return T * D; }
hipError_t launch_rope(const RopeCall&, hipStream_t) { return ok(); }
int64_t attn_workspace_bytes(const nvfp4_attn& a, bool) { return a.Tq * a.Hq; }
hipError_t launch_attn(const AttnCall&, hipStream_t) { return ok(); }
hipError_t launch_attn_grad(const AttnCall&, hipStream_t) { return ok(); }
}  // namespace nvfp4
