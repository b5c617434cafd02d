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

// The cross-entropy sizes: offsets inside a tile are 32-bit bytes (256 rows of a
// pitch below 2^22 elements), token and word numbers 32-bit.
constexpr int64_t kMaxPitch = (int64_t(1) << 22) - 8;

int check_ce_sizes(int64_t T, int64_t V, int64_t D, int grad, int64_t piece) {
  if (T < 0 || T > kMaxCount - 512)
    return fail(NVFP4_ERR_SHAPE, "T=%lld must be 0 .. 2^31 - 513", (long long)T);
  // the code rows of a piece are an operand too: V bounded like a pitch there
  const int64_t most = grad ? kMaxPitch - 128 : kMaxCount - 512;
  if (V < 1 || V > most)
    return fail(NVFP4_ERR_SHAPE, "V=%lld must be 1 .. %lld", (long long)V, (long long)most);
  if (D < 8 || D % 8 || D > kMaxPitch)
    return fail(NVFP4_ERR_SHAPE, "D=%lld must be a positive multiple of 8 below 2^22", (long long)D);
  if (grad != 0 && grad != 1) return fail(NVFP4_ERR_ARG, "grad=%d must be 0 or 1", grad);
  if (piece < 0)
    return fail(NVFP4_ERR_SHAPE, "piece_tokens=%lld must be 0 or more", (long long)piece);
  if (T > 0 && (V > kMaxElems / T || D > kMaxElems / T))
    return fail(NVFP4_ERR_SHAPE, "T*V or T*D exceeds 2^40");
  return NVFP4_OK;
}

// A BF16 operand or result of the products: 16-byte rows.
int check_rows16(const void* p, int64_t rows, int64_t cols, int64_t ld, const char* name) {
  int st = check_matrix(p, NVFP4_TYPE_BF16, rows, cols, ld, name);
  if (st) return st;
  if (ld > kMaxPitch)
    return fail(NVFP4_ERR_SHAPE, "%s: row pitch %lld must be below 2^22", name, (long long)ld);
  if (ld % 8 || (rows > 0 && !aligned(p, 16)))
    return fail(NVFP4_ERR_ALIGN, "%s: row pitch %lld must be a multiple of 8, the base 16-byte "
                "aligned", name, (long long)ld);
  return NVFP4_OK;
}

int check_ce(const void* h, int64_t ldh, const void* w, int64_t ldw, int64_t T, int64_t V,
             int64_t D, const void* targets, int targets_type, const float* loss,
             const float* lse) {
  int st = check_rows16(h, T, D, ldh, "h");
  if (st) return st;
  if ((st = check_rows16(w, V, D, ldw, "w"))) return st;
  if ((st = check_ids(targets, targets_type, T, "targets"))) return st;
  if (T > 0 && loss == nullptr) return fail(NVFP4_ERR_NULL, "loss is NULL");
  if (!aligned(loss, 4) || !aligned(lse, 4))
    return fail(NVFP4_ERR_ALIGN, "loss and lse must be 4-byte aligned");
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

int64_t nvfp4_linear_ce_workspace_bytes(int64_t T, int64_t V, int64_t D, int grad,
                                        int64_t piece_tokens) {
  const int st = check_ce_sizes(T, V, D, grad, piece_tokens);
  return st ? st : nvfp4::ce_workspace_bytes(T, V, D, grad == 1, piece_tokens);
}

int nvfp4_linear_ce(const void* h, int64_t ldh, const void* w, int64_t ldw, int64_t T, int64_t V,
                    int64_t D, const void* targets, int targets_type, float* loss, float* lse,
                    void* workspace, int64_t workspace_bytes, void* stream) {
  int st = check_ce_sizes(T, V, D, 0, 0);
  if (st) return st;
  if ((st = check_ce(h, ldh, w, ldw, T, V, D, targets, targets_type, loss, lse))) return st;
  if ((st = check_workspace(workspace, workspace_bytes,
                            nvfp4::ce_workspace_bytes(T, V, D, false, 0),
                            "nvfp4_linear_ce_workspace_bytes")))
    return st;
  nvfp4::CeCall c{};
  c.h = h;
  c.w = w;
  c.ldh = ldh;
  c.ldw = ldw;
  c.T = T;
  c.V = V;
  c.D = D;
  c.targets = targets;
  c.targets_type = targets_type;
  c.loss = loss;
  c.lse = lse;
  c.ws = workspace;
  return launched(nvfp4::launch_ce(c, as_stream(stream)));
}

int nvfp4_linear_ce_grad(const void* h, int64_t ldh, const void* w, int64_t ldw, int64_t T,
                         int64_t V, int64_t D, const void* targets, int targets_type,
                         const float* row_weight, int64_t piece_tokens, float* loss, float* lse,
                         void* dh, int64_t ld_dh, void* dw, int64_t ld_dw, void* workspace,
                         int64_t workspace_bytes, void* stream) {
  int st = check_ce_sizes(T, V, D, 1, piece_tokens);
  if (st) return st;
  if ((st = check_ce(h, ldh, w, ldw, T, V, D, targets, targets_type, loss, lse))) return st;
  if (!aligned(row_weight, 4)) return fail(NVFP4_ERR_ALIGN, "row_weight must be 4-byte aligned");
  if ((st = check_rows16(dh, T, D, ld_dh, "dh"))) return st;
  if ((st = check_rows16(dw, V, D, ld_dw, "dw"))) return st;
  if ((st = check_workspace(workspace, workspace_bytes,
                            nvfp4::ce_workspace_bytes(T, V, D, true, piece_tokens),
                            "nvfp4_linear_ce_workspace_bytes")))
    return st;
  nvfp4::CeCall c{};
  c.h = h;
  c.w = w;
  c.ldh = ldh;
  c.ldw = ldw;
  c.T = T;
  c.V = V;
  c.D = D;
  c.targets = targets;
  c.targets_type = targets_type;
  c.row_weight = row_weight;
  c.piece = piece_tokens;
  c.loss = loss;
  c.lse = lse;
  c.dh = dh;
  c.dw = dw;
  c.ld_dh = ld_dh;
  c.ld_dw = ld_dw;
  c.grad = true;
  c.ws = workspace;
  return launched(nvfp4::launch_ce(c, as_stream(stream)));
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

int nvfp4_grad_scale(const nvfp4_grad* list, int64_t count, const float* factor, void* stream) {
  int st = check_grads(list, count, true);
  if (st) return st;
  if (factor == nullptr) return fail(NVFP4_ERR_NULL, "factor is NULL");
  if (!aligned(factor, 4)) return fail(NVFP4_ERR_ALIGN, "factor must be 4-byte aligned");
  return launched(nvfp4::launch_grad_scale(list, count, factor, as_stream(stream)));
}

}  // extern "C"
