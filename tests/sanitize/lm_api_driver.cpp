// lm_api_driver.cpp -- drives the embedding, cross-entropy and gradient-list
// entry points on the host (launchers are stubs, lm_api_stubs.cpp) with valid,
// invalid and extreme arguments under AddressSanitizer and
// UndefinedBehaviorSanitizer: validation returns the documented status, reads
// nothing outside the list it is given and overflows no size.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "nvfp4.h"

extern int g_launches;
extern int64_t g_elements;

static int failures = 0;
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
  double* Q = reinterpret_cast<double*>(dev);
  const int BF = NVFP4_TYPE_BF16, F32 = NVFP4_TYPE_F32, I4 = NVFP4_TYPE_I32, I8 = NVFP4_TYPE_I64;
  const int OK = NVFP4_OK, S = NVFP4_ERR_SHAPE, N = NVFP4_ERR_NULL, G = NVFP4_ERR_ARG;
  const int64_t wild[] = {INT64_MIN, -1, INT64_MAX, int64_t(1) << 62, (int64_t(1) << 40) + 1};

  EXPECT(nvfp4_embed(P, I4, 5, P, BF, 9, 3, 3, 1.f, P, F32, 4, nullptr), OK);
  EXPECT(nvfp4_embed(nullptr, I4, 0, P, BF, 9, 3, 3, 1.f, nullptr, F32, 4, nullptr), OK);
  EXPECT(nvfp4_embed_grad(P, I8, 5, P, F32, 3, 9, 3, 1.f, P, BF, 3, 1, P, 1 << 12, nullptr), OK);
  EXPECT(nvfp4_embed_grad(nullptr, I8, 0, nullptr, F32, 3, 9, 3, 1.f, P, BF, 3, 0, nullptr, 0, nullptr),
         OK);
  EXPECT(nvfp4_linear_ce(P, 8, P, 8, 5, 9, 8, P, I4, F, nullptr, P, 256, nullptr), OK);
  EXPECT(nvfp4_linear_ce_grad(P, 8, P, 8, 5, 9, 8, P, I4, nullptr, 0, F, F, P, 8, P, 8, P, 1 << 12,
                              nullptr),
         OK);
  for (int64_t w : wild) {
    EXPECT(nvfp4_embed(P, I4, w, P, BF, 9, 3, 3, 1.f, P, F32, 4, nullptr), S);
    EXPECT(nvfp4_embed(P, I4, 5, P, BF, w, 3, 3, 1.f, P, F32, 4, nullptr), S);
    EXPECT(nvfp4_embed(P, I4, 5, P, BF, 9, w, w, 1.f, P, F32, w, nullptr), S);
    EXPECT(nvfp4_embed(P, I4, 5, P, BF, 9, 3, w, 1.f, P, F32, 4, nullptr), S);
    EXPECT(nvfp4_embed(P, I4, 5, P, BF, 9, 3, 3, 1.f, P, F32, w, nullptr), S);
    EXPECT(nvfp4_embed_grad(P, I8, w, P, F32, 3, 9, 3, 1.f, P, BF, 3, 1, P, w, nullptr), S);
    EXPECT(nvfp4_embed_grad(P, I8, 5, P, F32, w, 9, 3, 1.f, P, BF, 3, 1, P, w, nullptr), S);
    EXPECT(nvfp4_embed_grad_workspace_bytes(w, 9, 3), S);
    EXPECT(nvfp4_embed_grad_workspace_bytes(5, w, 3), S);
    EXPECT(nvfp4_embed_grad_workspace_bytes(5, 9, w), S);
    for (int grad = 0; grad < 2; ++grad) {
      EXPECT(nvfp4_linear_ce_workspace_bytes(w, 9, 8, grad, 0), S);
      EXPECT(nvfp4_linear_ce_workspace_bytes(5, w, 8, grad, 0), S);
      EXPECT(nvfp4_linear_ce_workspace_bytes(5, 9, w, grad, 0), S);
    }
    EXPECT(nvfp4_linear_ce(P, w, P, 8, 5, 9, 8, P, I4, F, nullptr, P, 256, nullptr), S);
    EXPECT(nvfp4_linear_ce(P, 8, P, w, 5, 9, 8, P, I4, F, nullptr, P, 256, nullptr), S);
    EXPECT(nvfp4_linear_ce_grad(P, 8, P, 8, 5, 9, 8, P, I4, nullptr, 0, F, F, P, w, P, 8, P, 1 << 12,
                                nullptr),
           S);
    EXPECT(nvfp4_grad_sumsq(nullptr, w < 0 ? w : -1, Q, nullptr), S);
    nvfp4_grad g{P, P, w, BF, BF};
    EXPECT(nvfp4_grad_sumsq(&g, 1, Q, nullptr), S);
  }
  EXPECT(nvfp4_linear_ce_workspace_bytes(5, 9, 8, 1, -3), S);
  EXPECT(nvfp4_linear_ce_workspace_bytes(5, 9, 8, 7, 0), G);
  EXPECT(nvfp4_linear_ce_workspace_bytes(int64_t(1) << 30, int64_t(1) << 21, 8, 1, 0), S);

  // lists on the heap of exactly their size: nothing past the end is read
  for (int64_t count : {0, 1, 95, 96, 97, 1000}) {
    std::vector<nvfp4_grad> list(count, nvfp4_grad{P, P, 3, F32, F32});
    g_elements = 0;
    EXPECT(nvfp4_grad_sumsq(list.data(), count, Q, nullptr), OK);
    EXPECT(nvfp4_grad_clip(list.data(), count, Q, 1.0, nullptr, nullptr), OK);
    EXPECT(nvfp4_grad_scale(list.data(), count, F, nullptr), OK);
    EXPECT(g_elements, 9 * count);
    if (count > 0) {
      list.back().in = nullptr;
      const int before = g_launches;
      EXPECT(nvfp4_grad_sumsq(list.data(), count, Q, nullptr), N);
      EXPECT(nvfp4_grad_clip(list.data(), count, Q, 1.0, nullptr, nullptr), N);
      EXPECT(nvfp4_grad_scale(list.data(), count, F, nullptr), N);
      EXPECT(g_launches, before);
    }
  }
  std::printf("unexpected statuses: %d, launches %d\n", failures, g_launches);
  return failures != 0;
}
