// lm_attn.hip -- softmax attention and its gradient (internal to libnvfp4.so).
//
// One wave a row: right for every case, bound by the vector units.
#include <hip/hip_runtime.h>

#include "lm_attn.h"

namespace nvfp4 {
namespace attn {

constexpr int64_t kWindowMost = int64_t(1) << 32;   // more than any sequence

Args make_args(const AttnCall& c) {
  const nvfp4_attn& n = c.a;
  auto rows = [](const nvfp4_heads& x) {
    return Rows{static_cast<const uint16_t*>(x.p), x.batch, x.token, x.head};
  };
  Args a{};
  a.q = rows(c.q);
  a.k = rows(c.k);
  a.v = rows(c.v);
  a.out = rows(c.out);
  a.dout = rows(c.dout);
  a.dq = rows(c.dq);
  a.dk = rows(c.dk);
  a.dv = rows(c.dv);
  a.lse = c.lse;
  a.delta = static_cast<float*>(c.ws);
  a.cu_q = n.cu_q;
  a.cu_k = n.cu_k;
  a.wide_cu = n.cu_type == NVFP4_TYPE_I64;
  a.causal = n.causal;
  a.batch = (int)n.batch;
  a.Tq = (int)n.Tq;
  a.Tk = (int)n.Tk;
  a.Hq = (int)n.Hq;
  a.Hkv = (int)n.Hkv;
  a.G = (int)(n.Hq / n.Hkv);
  a.D = (int)n.D;
  a.window = n.window < kWindowMost ? n.window : kWindowMost;   // its sums stay in int64
  a.scale = n.scale;
  a.scale2 = n.scale * 1.4426950408889634f;
  return a;
}

namespace {

constexpr int kWaves = 4;

__global__ __launch_bounds__(kWaves * 64) void k_attn_rows(Args a, int64_t rows) {
  const int64_t r = block_xz() * kWaves + (threadIdx.x >> 6);
  if (r >= rows) return;
  const int h = (int)(r % a.Hq), t = (int)(r / a.Hq % a.Tq), b = (int)(r / a.Hq / a.Tq);
  const Range k = keys_of(a, t);
  const Soft s = row_forward(a, b, t, h, k.lo, k.hi);
  const bool any = k.lo < k.hi;
  s.o.store(row_of_out(a.out, b, t, h), a.D, any ? 1.0f / s.l : 0.0f);
  if ((threadIdx.x & 63) == 0)
    a.lse[stat_at(a, b, t, h)] = any ? (s.m + log2f(s.l)) * 0.6931471805599453f : -INFINITY;
}

__global__ __launch_bounds__(kWaves * 64) void k_attn_delta(Args a, int64_t rows) {
  const int64_t r = block_xz() * kWaves + (threadIdx.x >> 6);
  if (r >= rows) return;
  const int h = (int)(r % a.Hq), t = (int)(r / a.Hq % a.Tq), b = (int)(r / a.Hq / a.Tq);
  const bf16_t* o = row_of(a.out, b, t, h);
  const bf16_t* d = row_of(a.dout, b, t, h);
  float s = 0.0f;
  for (int i = threadIdx.x & 63; i < a.D; i += 64) s += load1(o + i) * load1(d + i);
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) a.delta[r] = s;
}

__global__ __launch_bounds__(kWaves * 64) void k_attn_dq_rows(Args a, int64_t rows) {
  const int64_t r = block_xz() * kWaves + (threadIdx.x >> 6);
  if (r >= rows) return;
  row_dq(a, (int)(r / a.Hq / a.Tq), (int)(r / a.Hq % a.Tq), (int)(r % a.Hq));
}

__global__ __launch_bounds__(kWaves * 64) void k_attn_dkv_rows(Args a, int64_t rows) {
  const int64_t r = block_xz() * kWaves + (threadIdx.x >> 6);
  if (r >= rows) return;
  const int h = (int)(r % a.Hkv), j = (int)(r / a.Hkv % a.Tk), b = (int)(r / a.Hkv / a.Tk);
  const Range t = queries_of(a, j);
  RowSum dk, dv;
  row_dkv(a, b, j, h, (int64_t)t.lo * a.G, (int64_t)t.hi * a.G, dk, dv);
  dk.store(row_of_out(a.dk, b, j, h), a.D, a.scale);
  dv.store(row_of_out(a.dv, b, j, h), a.D, 1.0f);
}

int64_t sequences(const nvfp4_attn& a) { return a.cu_q == nullptr ? a.batch : 1; }
int64_t blocks(int64_t rows) { return (rows + kWaves - 1) / kWaves; }

}  // namespace
}  // namespace attn

using namespace attn;

int64_t attn_workspace_bytes(const nvfp4_attn& a, bool grad) {
  return grad ? sequences(a) * a.Tq * a.Hq * 4 : 0;
}

hipError_t launch_attn(const AttnCall& c, hipStream_t s) {
  const int64_t rows = sequences(c.a) * c.a.Tq * c.a.Hq;
  if (rows == 0) return hipSuccess;
  k_attn_rows<<<grid_xz(blocks(rows)), kWaves * 64, 0, s>>>(make_args(c), rows);
  return hipGetLastError();
}

hipError_t launch_attn_grad(const AttnCall& c, hipStream_t s) {
  const int64_t rows = sequences(c.a) * c.a.Tq * c.a.Hq, keys = sequences(c.a) * c.a.Tk * c.a.Hkv;
  const Args a = make_args(c);
  if (rows > 0) {
    k_attn_delta<<<grid_xz(blocks(rows)), kWaves * 64, 0, s>>>(a, rows);
    k_attn_dq_rows<<<grid_xz(blocks(rows)), kWaves * 64, 0, s>>>(a, rows);
  }
  if (keys > 0) k_attn_dkv_rows<<<grid_xz(blocks(keys)), kWaves * 64, 0, s>>>(a, keys);
  return hipGetLastError();
}

}  // namespace nvfp4
