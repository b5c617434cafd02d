// lm_api.cpp -- the C ABI of the embedding, gradient-clipping and
// cross-entropy operators (declared in include/nvfp4.h): argument validation,
// then kernel launches on the caller's stream.  Nothing here allocates, frees
// or synchronises.
#include "../../include/nvfp4.h"

#include "api_common.h"
#include "lm_kernels.h"

using namespace nvfp4::api;

namespace {

bool float_type(int t) { return t == NVFP4_TYPE_BF16 || t == NVFP4_TYPE_F32; }
bool index_type(int t) { return t == NVFP4_TYPE_I32 || t == NVFP4_TYPE_I64; }
int64_t type_bytes(int t) {
  return t == NVFP4_TYPE_BF16 ? 2 : t == NVFP4_TYPE_I64 ? 8 : 4;
}

// A matrix [rows][cols] with row pitch ld, natural alignment; NULL is fine
// where there are no rows.
int check_matrix(const void* p, int type, int64_t rows, int64_t cols, int64_t ld,
                 const char* name) {
  if (!float_type(type)) return fail(NVFP4_ERR_ARG, "%s: type %d is not BF16 or F32", name, type);
  if (ld < cols)
    return fail(NVFP4_ERR_SHAPE, "%s: row pitch %lld < %lld columns", name, (long long)ld,
                (long long)cols);
  if (ld > kMaxElems || (rows > 0 && ld > kMaxElems / rows))
    return fail(NVFP4_ERR_SHAPE, "%s: rows*pitch exceeds 2^40 elements", name);
  if (rows == 0) return NVFP4_OK;
  if (p == nullptr) return fail(NVFP4_ERR_NULL, "%s is NULL", name);
  if (!aligned(p, (uintptr_t)type_bytes(type)))
    return fail(NVFP4_ERR_ALIGN, "%s must be aligned to its elements", name);
  return NVFP4_OK;
}

int check_ids(const void* ids, int type, int64_t n, const char* name) {
  if (!index_type(type)) return fail(NVFP4_ERR_ARG, "%s: type %d is not I32 or I64", name, type);
  if (n == 0) return NVFP4_OK;
  if (ids == nullptr) return fail(NVFP4_ERR_NULL, "%s is NULL", name);
  if (!aligned(ids, (uintptr_t)type_bytes(type)))
    return fail(NVFP4_ERR_ALIGN, "%s must be aligned to its elements", name);
  return NVFP4_OK;
}

// Tokens are numbered and words are keyed in 32 bits; one grid dimension
// counts tokens or words, the other column ranges of 512 (at most 65535).
constexpr int64_t kMaxCount = (int64_t(1) << 31) - 1, kMaxDim = int64_t(1) << 24;

int check_embed_sizes(int64_t n, int64_t vocab, int64_t dim) {
  if (n < 0 || n > kMaxCount)
    return fail(NVFP4_ERR_SHAPE, "n=%lld must be 0 .. 2^31 - 1", (long long)n);
  if (vocab < 1 || vocab >= kMaxCount)
    return fail(NVFP4_ERR_SHAPE, "vocab=%lld must be 1 .. 2^31 - 2", (long long)vocab);
  if (dim < 1 || dim > kMaxDim)
    return fail(NVFP4_ERR_SHAPE, "dim=%lld must be 1 .. 2^24", (long long)dim);
  return NVFP4_OK;
}

int check_workspace(const void* ws, int64_t bytes, int64_t need, const char* query) {
  if (need == 0) return NVFP4_OK;
  if (ws == nullptr) return fail(NVFP4_ERR_NULL, "workspace is NULL (%lld bytes needed)", (long long)need);
  if (!aligned(ws, 256)) return fail(NVFP4_ERR_ALIGN, "workspace must be 256-byte aligned");
  if (bytes < need)
    return fail(NVFP4_ERR_ARG, "workspace_bytes=%lld < %lld (%s)", (long long)bytes,
                (long long)need, query);
  return NVFP4_OK;
}

int check_grads(const nvfp4_grad* list, int64_t count, bool outputs) {
  if (count < 0 || count > kMaxCount)
    return fail(NVFP4_ERR_SHAPE, "count=%lld must be 0 .. 2^31 - 1", (long long)count);
  if (count > 0 && list == nullptr) return fail(NVFP4_ERR_NULL, "list is NULL");
  for (int64_t i = 0; i < count; ++i) {
    const nvfp4_grad& g = list[i];
    if (g.numel < 0 || g.numel > kMaxElems)
      return fail(NVFP4_ERR_SHAPE, "gradient %lld: numel=%lld must be 0 .. 2^40", (long long)i,
                  (long long)g.numel);
    if (!float_type(g.in_type) || (outputs && !float_type(g.out_type)))
      return fail(NVFP4_ERR_ARG, "gradient %lld: types must be BF16 or F32", (long long)i);
    if (g.numel == 0) continue;
    if (g.in == nullptr || (outputs && g.out == nullptr))
      return fail(NVFP4_ERR_NULL, "gradient %lld: in / out is NULL", (long long)i);
    if (!aligned(g.in, (uintptr_t)type_bytes(g.in_type)) ||
        (outputs && !aligned(g.out, (uintptr_t)type_bytes(g.out_type))))
      return fail(NVFP4_ERR_ALIGN, "gradient %lld must be aligned to its elements", (long long)i);
    if (outputs && g.in == g.out && g.in_type != g.out_type)
      return fail(NVFP4_ERR_ARG, "gradient %lld: in place needs one type", (long long)i);
  }
  return NVFP4_OK;
}

int check_partials(const double* partials) {
  if (partials == nullptr) return fail(NVFP4_ERR_NULL, "partials is NULL");
  if (!aligned(partials, 8)) return fail(NVFP4_ERR_ALIGN, "partials must be 8-byte aligned");
  return NVFP4_OK;
}

}  // namespace

extern "C" {

int nvfp4_embed(const void* ids, int ids_type, int64_t n, const void* w, int w_type, int64_t vocab,
                int64_t dim, int64_t ldw, float scale, void* out, int out_type, int64_t ldo,
                void* stream) {
  int st = check_embed_sizes(n, vocab, dim);
  if (st) return st;
  if ((st = check_ids(ids, ids_type, n, "ids"))) return st;
  if ((st = check_matrix(w, w_type, vocab, dim, ldw, "w"))) return st;
  if ((st = check_matrix(out, out_type, n, dim, ldo, "out"))) return st;
  return launched(nvfp4::launch_embed(nvfp4::EmbedArgs{ids, ids_type, n, vocab, dim, scale}, w,
                                      w_type, ldw, out, out_type, ldo, as_stream(stream)));
}

int64_t nvfp4_embed_grad_workspace_bytes(int64_t n, int64_t vocab, int64_t dim) {
  const int st = check_embed_sizes(n, vocab, dim);
  return st ? st : nvfp4::embed_grad_workspace_bytes(n, vocab, dim);
}

int nvfp4_embed_grad(const void* ids, int ids_type, int64_t n, const void* dy, int dy_type,
                     int64_t ld_dy, int64_t vocab, int64_t dim, float scale, void* dw, int dw_type,
                     int64_t ld_dw, int accumulate, void* workspace, int64_t workspace_bytes,
                     void* stream) {
  int st = check_embed_sizes(n, vocab, dim);
  if (st) return st;
  if ((st = check_ids(ids, ids_type, n, "ids"))) return st;
  if ((st = check_matrix(dy, dy_type, n, dim, ld_dy, "dy"))) return st;
  if ((st = check_matrix(dw, dw_type, vocab, dim, ld_dw, "dw"))) return st;
  if (accumulate != 0 && accumulate != 1)
    return fail(NVFP4_ERR_ARG, "accumulate=%d must be 0 or 1", accumulate);
  if ((st = check_workspace(workspace, workspace_bytes,
                            nvfp4::embed_grad_workspace_bytes(n, vocab, dim),
                            "nvfp4_embed_grad_workspace_bytes")))
    return st;
  return launched(nvfp4::launch_embed_grad(nvfp4::EmbedArgs{ids, ids_type, n, vocab, dim, scale},
                                           dy, dy_type, ld_dy, dw, dw_type, ld_dw,
                                           accumulate == 1, workspace, as_stream(stream)));
}

int nvfp4_grad_sumsq(const nvfp4_grad* list, int64_t count, double* partials, void* stream) {
  int st = check_grads(list, count, false);
  if (st) return st;
  if ((st = check_partials(partials))) return st;
  return launched(nvfp4::launch_grad_sumsq(list, count, partials, as_stream(stream)));
}

int nvfp4_grad_clip(const nvfp4_grad* list, int64_t count, const double* partials, double max_norm,
                    float* norm_out, void* stream) {
  int st = check_grads(list, count, true);
  if (st) return st;
  if ((st = check_partials(partials))) return st;
  if (!(max_norm >= 0.0)) return fail(NVFP4_ERR_ARG, "max_norm=%g must be 0 or more", max_norm);
  if (norm_out != nullptr && !aligned(norm_out, 4))
    return fail(NVFP4_ERR_ALIGN, "norm_out must be 4-byte aligned");
  return launched(nvfp4::launch_grad_clip(list, count, partials, max_norm, norm_out,
                                          as_stream(stream)));
}

}  // extern "C"
