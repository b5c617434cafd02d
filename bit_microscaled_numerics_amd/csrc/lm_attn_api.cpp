// lm_attn_api.cpp -- the C ABI of the query / key norm and rotation and of attention
// (declared in include/nvfp4.h): argument validation, then kernel launches on the
// caller's stream.  Nothing here allocates, frees or synchronises.
#include "../../include/nvfp4.h"

#include <cmath>
#include <utility>

#include "api_common.h"
#include "lm_attn_kernels.h"

using namespace nvfp4::api;

namespace {

// Rows are numbered in 32 bits.
constexpr int64_t kMaxCount = (int64_t(1) << 31) - 513, kMaxHeads = 65536;

bool float_type(int t) { return t == NVFP4_TYPE_BF16 || t == NVFP4_TYPE_F32; }
bool index_type(int t) { return t == NVFP4_TYPE_I32 || t == NVFP4_TYPE_I64; }
uintptr_t type_bytes(int t) { return t == NVFP4_TYPE_BF16 ? 2 : t == NVFP4_TYPE_I64 ? 8 : 4; }

// An operand of n x T x H rows of D: its elements span less than 2^40, its rows lie apart.
int check_heads(const nvfp4_heads* x, int64_t n, int64_t T, int64_t H, int64_t D, uintptr_t align,
                const char* name) {
  if (x == nullptr) return fail(NVFP4_ERR_NULL, "%s is NULL", name);
  if (n == 0 || T == 0 || H == 0) return NVFP4_OK;
  if (x->p == nullptr) return fail(NVFP4_ERR_NULL, "%s: p is NULL", name);
  if (!aligned(x->p, align))
    return fail(NVFP4_ERR_ALIGN, "%s must be aligned to %d bytes", name, (int)align);
  struct Dim { int64_t stride, count; } d[3] = {{x->batch, n}, {x->token, T}, {x->head, H}};
  for (int i = 0; i < 2; ++i)   // ascending strides
    for (int j = 0; j < 2; ++j)
      if (d[j].stride > d[j + 1].stride) std::swap(d[j], d[j + 1]);
  int64_t span = D;
  for (const Dim& e : d) {
    if (e.count == 1) continue;   // its stride is not used
    if (e.stride < span)
      return fail(NVFP4_ERR_SHAPE, "%s: rows overlap (stride %lld, %lld elements within)", name,
                  (long long)e.stride, (long long)span);
    if (e.stride > (kMaxElems - span) / (e.count - 1))
      return fail(NVFP4_ERR_SHAPE, "%s spans more than 2^40 elements", name);
    if (align == 16 && e.stride % 8)
      return fail(NVFP4_ERR_ALIGN, "%s: strides must be multiples of 8", name);
    span += e.stride * (e.count - 1);
  }
  return NVFP4_OK;
}

// The operand as the kernels take it: 0 where a stride is not used.
nvfp4_heads used(const nvfp4_heads* x, int64_t n, int64_t T, int64_t H) {
  return nvfp4_heads{x->p, n > 1 ? x->batch : 0, T > 1 ? x->token : 0, H > 1 ? x->head : 0};
}

int check_workspace(const void* ws, int64_t bytes, int64_t need, const char* query) {
  if (need == 0) return NVFP4_OK;
  if (ws == nullptr)
    return fail(NVFP4_ERR_NULL, "workspace is NULL (%lld bytes needed)", (long long)need);
  if (!aligned(ws, 256)) return fail(NVFP4_ERR_ALIGN, "workspace must be 256-byte aligned");
  if (bytes < need)
    return fail(NVFP4_ERR_ARG, "workspace_bytes=%lld < %lld (%s)", (long long)bytes,
                (long long)need, query);
  return NVFP4_OK;
}

int check_rope_sizes(int64_t T, int64_t Hq, int64_t Hkv, int64_t D) {
  if (T < 0 || T > kMaxCount)
    return fail(NVFP4_ERR_SHAPE, "T=%lld must be 0 .. 2^31 - 513", (long long)T);
  if (Hq < 0 || Hkv < 0 || Hq > kMaxHeads || Hkv > kMaxHeads)
    return fail(NVFP4_ERR_SHAPE, "Hq=%lld, Hkv=%lld must be 0 .. 65536", (long long)Hq, (long long)Hkv);
  if (D < 2 || D % 2 || D > 512)
    return fail(NVFP4_ERR_SHAPE, "D=%lld must be even, 2 .. 512", (long long)D);
  return NVFP4_OK;
}

int check_rope(const nvfp4_rope* r) {
  if (r == nullptr) return fail(NVFP4_ERR_NULL, "r is NULL");
  int st = check_rope_sizes(r->T, r->Hq, r->Hkv, r->D);
  if (st) return st;
  if (r->rot < 0 || r->rot % 2 || r->rot > r->D)
    return fail(NVFP4_ERR_SHAPE, "rot=%lld must be even, 0 .. D", (long long)r->rot);
  if (!float_type(r->type) || !float_type(r->weight_type))
    return fail(NVFP4_ERR_ARG, "type and weight_type must be BF16 or F32");
  if (!index_type(r->positions_type))
    return fail(NVFP4_ERR_ARG, "positions: type %d is not I32 or I64", r->positions_type);
  if ((r->interleaved != 0 && r->interleaved != 1) || (r->norm != 0 && r->norm != 1))
    return fail(NVFP4_ERR_ARG, "interleaved and norm must be 0 or 1");
  if (!(r->eps >= 0.f) || std::isinf(r->eps))
    return fail(NVFP4_ERR_ARG, "eps=%g must be 0 or more and finite", (double)r->eps);
  if (!r->norm && (r->q_weight != nullptr || r->k_weight != nullptr))
    return fail(NVFP4_ERR_ARG, "weights go with norm = 1");
  if (!aligned(r->q_weight, type_bytes(r->weight_type)) ||
      !aligned(r->k_weight, type_bytes(r->weight_type)))
    return fail(NVFP4_ERR_ALIGN, "weights must be aligned to their elements");
  if (r->T > 0 && r->rot > 0) {
    if (r->positions == nullptr || r->inv_freq == nullptr)
      return fail(NVFP4_ERR_NULL, "positions / inv_freq is NULL");
    if (!aligned(r->positions, type_bytes(r->positions_type)) || !aligned(r->inv_freq, 4))
      return fail(NVFP4_ERR_ALIGN, "positions and inv_freq must be aligned to their elements");
  }
  return NVFP4_OK;
}

// In place only with the same strides.
int check_in_place(const nvfp4_heads& in, const nvfp4_heads& out, const char* name) {
  if (in.p != nullptr && in.p == out.p && (in.token != out.token || in.head != out.head))
    return fail(NVFP4_ERR_ARG, "%s: in place needs the same strides", name);
  return NVFP4_OK;
}

int check_attn_sizes(const nvfp4_attn* a) {
  if (a == nullptr) return fail(NVFP4_ERR_NULL, "a is NULL");
  if (a->batch < 0 || a->Tq < 0 || a->Tk < 0 || a->batch > kMaxCount || a->Tq > kMaxCount ||
      a->Tk > kMaxCount)
    return fail(NVFP4_ERR_SHAPE, "batch=%lld, Tq=%lld, Tk=%lld must be 0 .. 2^31 - 513",
                (long long)a->batch, (long long)a->Tq, (long long)a->Tk);
  if (a->Hkv < 1 || a->Hq < 1 || a->Hq > kMaxHeads || a->Hq % a->Hkv)
    return fail(NVFP4_ERR_SHAPE, "Hq=%lld must be a positive multiple of Hkv=%lld, at most 65536",
                (long long)a->Hq, (long long)a->Hkv);
  if (a->D < 8 || a->D % 8 || a->D > 128)
    return fail(NVFP4_ERR_SHAPE, "D=%lld must be a multiple of 8, 8 .. 128", (long long)a->D);
  if ((a->cu_q == nullptr) != (a->cu_k == nullptr))
    return fail(NVFP4_ERR_ARG, "cu_q and cu_k go together");
  const int64_t n = a->cu_q == nullptr ? a->batch : 1;
  if (a->Tq > 0 && (n > kMaxCount / a->Tq || n * a->Tq > kMaxCount / a->Hq))
    return fail(NVFP4_ERR_SHAPE, "queries * Hq must be below 2^31 - 512");
  if (a->Tk > 0 && (n > kMaxCount / a->Tk || n * a->Tk > kMaxCount / a->Hkv))
    return fail(NVFP4_ERR_SHAPE, "keys * Hkv must be below 2^31 - 512");
  if (n > kMaxCount / a->Hq) return fail(NVFP4_ERR_SHAPE, "batch * Hq must be below 2^31 - 512");
  return NVFP4_OK;
}

int check_attn(const nvfp4_attn* a) {
  int st = check_attn_sizes(a);
  if (st) return st;
  if (a->causal != 0 && a->causal != 1)
    return fail(NVFP4_ERR_ARG, "causal=%d must be 0 or 1", a->causal);
  if (a->window < 0 || (a->window > 0 && !a->causal))
    return fail(NVFP4_ERR_ARG, "window=%lld must be 0, or positive and causal", (long long)a->window);
  // the gradient holds lse / scale, which stays in FP32's range between these
  if (!(a->scale >= 0x1p-64f && a->scale <= 0x1p64f))
    return fail(NVFP4_ERR_ARG, "scale=%g must lie within 2^-64 .. 2^64", (double)a->scale);
  if (a->cu_q != nullptr) {
    if (!index_type(a->cu_type))
      return fail(NVFP4_ERR_ARG, "cu_q, cu_k: type %d is not I32 or I64", a->cu_type);
    if (!aligned(a->cu_q, type_bytes(a->cu_type)) || !aligned(a->cu_k, type_bytes(a->cu_type)))
      return fail(NVFP4_ERR_ALIGN, "cu_q and cu_k must be aligned to their elements");
  }
  return NVFP4_OK;
}

// Offsets inside a tile are 32-bit bytes: 128 tokens and the heads of a group.
int check_tile(const nvfp4_heads* x, int64_t T, int64_t G, const char* name) {
  const int64_t most = (int64_t(1) << 22) - 8;
  if ((T > 1 && x->token > most) || (G > 1 && x->head > (int64_t(1) << 29) / (G - 1)))
    return fail(NVFP4_ERR_SHAPE, "%s: token strides must be below 2^22 elements, the heads of a "
                "group within 2^29", name);
  return NVFP4_OK;
}

// Checks an operand and leaves it in *to.
int take_q_side(const nvfp4_attn* a, const nvfp4_heads* x, nvfp4_heads* to, const char* name) {
  const int64_t n = a->cu_q == nullptr ? a->batch : 1;
  int st = check_heads(x, n, a->Tq, a->Hq, a->D, 16, name);
  if (st) return st;
  *to = used(x, n, a->Tq, a->Hq);
  return check_tile(to, a->Tq, a->Hq / a->Hkv, name);
}

int take_k_side(const nvfp4_attn* a, const nvfp4_heads* x, nvfp4_heads* to, const char* name) {
  const int64_t n = a->cu_q == nullptr ? a->batch : 1;
  int st = check_heads(x, n, a->Tk, a->Hkv, a->D, 16, name);
  if (st) return st;
  *to = used(x, n, a->Tk, a->Hkv);
  return check_tile(to, a->Tk, 1, name);
}

// Results are written while operands are still read.
int check_apart(const nvfp4_heads* results, int n, const nvfp4_heads* operands, int m) {
  for (int i = 0; i < n; ++i) {
    for (int j = 0; j < m; ++j)
      if (results[i].p != nullptr && results[i].p == operands[j].p)
        return fail(NVFP4_ERR_ARG, "a result may not be an operand (no attention in place)");
    for (int j = 0; j < i; ++j)
      if (results[i].p != nullptr && results[i].p == results[j].p)
        return fail(NVFP4_ERR_ARG, "two results at one place");
  }
  return NVFP4_OK;
}

int check_lse(const nvfp4_attn* a, const float* lse) {
  const int64_t n = a->cu_q == nullptr ? a->batch : 1;
  if (n * a->Tq > 0 && lse == nullptr) return fail(NVFP4_ERR_NULL, "lse is NULL");
  if (!aligned(lse, 4)) return fail(NVFP4_ERR_ALIGN, "lse must be 4-byte aligned");
  return NVFP4_OK;
}

}  // namespace

extern "C" {

int nvfp4_qk_norm_rope(const nvfp4_rope* r, const nvfp4_heads* q, const nvfp4_heads* k,
                       const nvfp4_heads* q_out, const nvfp4_heads* k_out, void* stream) {
  int st = check_rope(r);
  if (st) return st;
  const uintptr_t el = type_bytes(r->type);
  if ((st = check_heads(q, 1, r->T, r->Hq, r->D, el, "q"))) return st;
  if ((st = check_heads(k, 1, r->T, r->Hkv, r->D, el, "k"))) return st;
  if ((st = check_heads(q_out, 1, r->T, r->Hq, r->D, el, "q_out"))) return st;
  if ((st = check_heads(k_out, 1, r->T, r->Hkv, r->D, el, "k_out"))) return st;
  nvfp4::RopeCall c{};
  c.r = *r;
  c.q = used(q, 1, r->T, r->Hq);
  c.k = used(k, 1, r->T, r->Hkv);
  c.q_out = used(q_out, 1, r->T, r->Hq);
  c.k_out = used(k_out, 1, r->T, r->Hkv);
  if ((st = check_in_place(c.q, c.q_out, "q_out"))) return st;
  if ((st = check_in_place(c.k, c.k_out, "k_out"))) return st;
  return launched(nvfp4::launch_rope(c, as_stream(stream)));
}

int64_t nvfp4_qk_norm_rope_grad_workspace_bytes(int64_t T, int64_t Hq, int64_t Hkv, int64_t D) {
  const int st = check_rope_sizes(T, Hq, Hkv, D);
  return st ? st : nvfp4::rope_workspace_bytes(T, Hq, Hkv, D);
}

int nvfp4_qk_norm_rope_grad(const nvfp4_rope* r, const nvfp4_heads* dq, const nvfp4_heads* dk,
                            const nvfp4_heads* q, const nvfp4_heads* k, const nvfp4_heads* dq_in,
                            const nvfp4_heads* dk_in, void* dq_weight, void* dk_weight,
                            void* workspace, int64_t workspace_bytes, void* stream) {
  int st = check_rope(r);
  if (st) return st;
  const uintptr_t el = type_bytes(r->type);
  if ((st = check_heads(dq, 1, r->T, r->Hq, r->D, el, "dq"))) return st;
  if ((st = check_heads(dk, 1, r->T, r->Hkv, r->D, el, "dk"))) return st;
  if ((st = check_heads(q, 1, r->T, r->Hq, r->D, el, "q"))) return st;
  if ((st = check_heads(k, 1, r->T, r->Hkv, r->D, el, "k"))) return st;
  if ((st = check_heads(dq_in, 1, r->T, r->Hq, r->D, el, "dq_in"))) return st;
  if ((st = check_heads(dk_in, 1, r->T, r->Hkv, r->D, el, "dk_in"))) return st;
  if ((r->q_weight == nullptr && dq_weight != nullptr) ||
      (r->k_weight == nullptr && dk_weight != nullptr))
    return fail(NVFP4_ERR_ARG, "a weight's gradient without its weight");
  if (!aligned(dq_weight, type_bytes(r->weight_type)) ||
      !aligned(dk_weight, type_bytes(r->weight_type)))
    return fail(NVFP4_ERR_ALIGN, "the weights' gradients must be aligned to their elements");
  if ((st = check_workspace(workspace, workspace_bytes,
                            nvfp4::rope_workspace_bytes(r->T, r->Hq, r->Hkv, r->D),
                            "nvfp4_qk_norm_rope_grad_workspace_bytes")))
    return st;
  nvfp4::RopeCall c{};
  c.r = *r;
  c.q = used(q, 1, r->T, r->Hq);
  c.k = used(k, 1, r->T, r->Hkv);
  c.dq = used(dq, 1, r->T, r->Hq);
  c.dk = used(dk, 1, r->T, r->Hkv);
  c.q_out = used(dq_in, 1, r->T, r->Hq);
  c.k_out = used(dk_in, 1, r->T, r->Hkv);
  if ((st = check_in_place(c.dq, c.q_out, "dq_in"))) return st;
  if ((st = check_in_place(c.dk, c.k_out, "dk_in"))) return st;
  c.dq_weight = dq_weight;
  c.dk_weight = dk_weight;
  c.grad = true;
  c.ws = workspace;
  return launched(nvfp4::launch_rope(c, as_stream(stream)));
}

int64_t nvfp4_attention_workspace_bytes(const nvfp4_attn* a, int grad) {
  const int st = check_attn_sizes(a);
  if (st) return st;
  if (grad != 0 && grad != 1) return fail(NVFP4_ERR_ARG, "grad=%d must be 0 or 1", grad);
  return nvfp4::attn_workspace_bytes(*a, grad == 1);
}

int nvfp4_attention(const nvfp4_attn* a, const nvfp4_heads* q, const nvfp4_heads* k,
                    const nvfp4_heads* v, const nvfp4_heads* out, float* lse, void* workspace,
                    int64_t workspace_bytes, void* stream) {
  int st = check_attn(a);
  if (st) return st;
  nvfp4::AttnCall c{};
  if ((st = take_q_side(a, q, &c.q, "q"))) return st;
  if ((st = take_k_side(a, k, &c.k, "k"))) return st;
  if ((st = take_k_side(a, v, &c.v, "v"))) return st;
  if ((st = take_q_side(a, out, &c.out, "out"))) return st;
  if ((st = check_lse(a, lse))) return st;
  const nvfp4_heads operands[] = {c.q, c.k, c.v};
  if ((st = check_apart(&c.out, 1, operands, 3))) return st;
  if ((st = check_workspace(workspace, workspace_bytes, nvfp4::attn_workspace_bytes(*a, false),
                            "nvfp4_attention_workspace_bytes")))
    return st;
  c.a = *a;
  c.lse = lse;
  c.ws = workspace;
  return launched(nvfp4::launch_attn(c, as_stream(stream)));
}

int nvfp4_attention_grad(const nvfp4_attn* a, const nvfp4_heads* dout, const nvfp4_heads* q,
                         const nvfp4_heads* k, const nvfp4_heads* v, const nvfp4_heads* out,
                         const float* lse, const nvfp4_heads* dq, const nvfp4_heads* dk,
                         const nvfp4_heads* dv, void* workspace, int64_t workspace_bytes,
                         void* stream) {
  int st = check_attn(a);
  if (st) return st;
  nvfp4::AttnCall c{};
  if ((st = take_q_side(a, dout, &c.dout, "dout"))) return st;
  if ((st = take_q_side(a, q, &c.q, "q"))) return st;
  if ((st = take_k_side(a, k, &c.k, "k"))) return st;
  if ((st = take_k_side(a, v, &c.v, "v"))) return st;
  if ((st = take_q_side(a, out, &c.out, "out"))) return st;
  if ((st = check_lse(a, lse))) return st;
  if ((st = take_q_side(a, dq, &c.dq, "dq"))) return st;
  if ((st = take_k_side(a, dk, &c.dk, "dk"))) return st;
  if ((st = take_k_side(a, dv, &c.dv, "dv"))) return st;
  const nvfp4_heads operands[] = {c.q, c.k, c.v, c.out, c.dout}, results[] = {c.dq, c.dk, c.dv};
  if ((st = check_apart(results, 3, operands, 5))) return st;
  if ((st = check_workspace(workspace, workspace_bytes, nvfp4::attn_workspace_bytes(*a, true),
                            "nvfp4_attention_workspace_bytes")))
    return st;
  c.a = *a;
  c.lse = const_cast<float*>(lse);
  c.ws = workspace;
  return launched(nvfp4::launch_attn_grad(c, as_stream(stream)));
}

}  // extern "C"
