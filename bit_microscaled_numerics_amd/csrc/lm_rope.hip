// lm_rope.hip -- norms of queries and keys for each head with the position rotation in
// the same pass, and the gradient (internal to libnvfp4.so).
//
// A row of D values is taken as D/2 pairs: the rot/2 rotated ones, then the rest of the
// row as the pairs of its halves, which are not rotated.  A lane owns 8 pairs; 1 .. 32
// lanes make a row, so that a rotation needs no exchange and a norm a few shuffles.
// A wave takes all heads of a token (several tokens, where they are few): the
// sines and cosines of a lane's pairs are formed once for all of them.
//
// Bound by HBM: 4 bytes per value (BF16), 6 in the gradient.
#include <hip/hip_runtime.h>

#include "lm_attn_kernels.h"
#include "lm_device.h"
#include "lm_kernels.h"

namespace nvfp4 {
namespace {

constexpr int kWaves = 4;        // waves of a workgroup
constexpr int kPartials = 1024;  // most workgroups of the gradient, each with sums of dw

struct Side {   // queries or keys
  const uint8_t* x;
  const uint8_t* dy;
  uint8_t* out;
  const void* w;
  int64_t x_token, x_head, dy_token, dy_head, out_token, out_head;   // bytes
};

struct Args {
  Side side[2];
  const void* positions;
  const float* inv_freq;
  float* partials;   // gradient: [workgroup][side][D]
  int64_t T;
  int Hq, H, D, np, nr;     // np rotated pairs, nr others
  int lanes;                // per row, a power of two
  int spread, steps, per;   // heads of a token side by side; rounds of them, and per wave
  int tokens;               // tokens of a wave side by side
  int wide_ids, wide_w, norm;
  float eps;
};

struct Pairs {
  v8f a, b;
};

__device__ __forceinline__ int lane_reduce_steps(int lanes) { return __builtin_ctz(lanes); }

__device__ __forceinline__ float row_sum(float x, int lanes) {
  for (int m = 1; m < lanes; m <<= 1) x += __shfl_xor(x, m);
  return x;
}

// Where pair s of a row lies.
template <bool IL>
__device__ __forceinline__ void place(const Args& k, int s, int& a, int& b) {
  if (s >= k.np) {
    a = 2 * k.np + (s - k.np);
    b = a + k.nr;
  } else if (IL) {
    a = 2 * s;
    b = a + 1;
  } else {
    a = s;
    b = s + k.np;
  }
}

// A lane's pairs: 8 consecutive ones (VEC: all rotated or none, 16-byte pieces of the
// row), or 8 that lie a row's lanes apart.
template <class T, bool IL, bool VEC>
struct Lane {
  const Args& k;
  int first, live;
  __device__ __forceinline__ Lane(const Args& args, int in_row) : k(args) {
    first = VEC ? in_row * 8 : in_row;
    live = (k.np + k.nr) - first;   // pairs from here on
  }
  __device__ __forceinline__ bool has(int i) const { return (VEC ? i : i * k.lanes) < live; }
  __device__ __forceinline__ int pair(int i) const { return first + (VEC ? i : i * k.lanes); }

  template <class U>
  __device__ __forceinline__ Pairs load(const U* row) const {
    Pairs p{};
    if constexpr (VEC) {
      if (live > 0) {
        if (IL && first < k.np) {
          const v8f lo = load8(row + 2 * first), hi = load8(row + 2 * first + 8);
          p.a = __builtin_shufflevector(lo, hi, 0, 2, 4, 6, 8, 10, 12, 14);
          p.b = __builtin_shufflevector(lo, hi, 1, 3, 5, 7, 9, 11, 13, 15);
        } else {
          int a, b;
          place<false>(k, first, a, b);
          p.a = load8(row + a);
          p.b = load8(row + b);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (has(i)) {
          int a, b;
          place<IL>(k, pair(i), a, b);
          p.a[i] = load1(row + a);
          p.b[i] = load1(row + b);
        }
    }
    return p;
  }
  template <class U>
  __device__ __forceinline__ void store(U* row, const Pairs& p) const {
    if constexpr (VEC) {
      if (live > 0) {
        if (IL && first < k.np) {
          store8(row + 2 * first, __builtin_shufflevector(p.a, p.b, 0, 8, 1, 9, 2, 10, 3, 11));
          store8(row + 2 * first + 8, __builtin_shufflevector(p.a, p.b, 4, 12, 5, 13, 6, 14, 7, 15));
        } else {
          int a, b;
          place<false>(k, first, a, b);
          store8(row + a, p.a);
          store8(row + b, p.b);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (has(i)) {
          int a, b;
          place<IL>(k, pair(i), a, b);
          store1(row + a, p.a[i]);
          store1(row + b, p.b[i]);
        }
    }
  }
  __device__ __forceinline__ Pairs weights(const void* w) const {
    if (w == nullptr) {
      Pairs p;
      p.a = p.b = 1.0f;
      return p;
    }
    return k.wide_w ? load(static_cast<const float*>(w)) : load(static_cast<const bf16_t*>(w));
  }
};

// cos and sin of a lane's pairs.  The angle in turns: position * inv_freq in FP64
// (exact up to positions of 2^29), times 1/(2 pi) in two parts with the whole turns
// taken off by a fused multiply-add, so a far position costs no accuracy.
template <class L>
__device__ __forceinline__ void turns(const Args& k, const L& at, double pos, v8f& c, v8f& s) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591011e-18;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] = 1.0f;
    s[i] = 0.0f;
    if (at.has(i) && at.pair(i) < k.np) {
      const double u = pos * (double)k.inv_freq[at.pair(i)];
      const double whole = __builtin_rint(u * kHi);
      const double f = __builtin_fma(u, kLo, __builtin_fma(u, kHi, -whole));
      float si, co;
      sincospif((float)(2.0 * f), &si, &co);
      c[i] = co;
      s[i] = si;
    }
  }
}

__device__ __forceinline__ double position(const Args& k, int64_t t) {
  return k.wide_ids ? (double)static_cast<const int64_t*>(k.positions)[t]
                    : (double)static_cast<const int32_t*>(k.positions)[t];
}

// Who a wave's lanes are: lane group `group` of a row's lanes takes heads head0,
// head0 + spread, .. of token t0 + token.
struct Place {
  int in_row, token, head0;
  bool on;
  __device__ __forceinline__ Place(const Args& k) {
    const int lane = threadIdx.x & 63, group = lane / k.lanes;
    in_row = lane & (k.lanes - 1);
    token = group / k.spread;
    head0 = group - token * k.spread;
    on = token < k.tokens;
  }
};

template <class T, bool IL, bool VEC>
__global__ __launch_bounds__(kWaves * 64) void k_rope(Args k) {
  const Place at(k);
  const int wave = threadIdx.x >> 6;
  const int64_t t = (block_xz() * kWaves + wave) * k.tokens + at.token;
  if (!at.on || t >= k.T) return;
  const Lane<T, IL, VEC> lane(k, at.in_row);
  const int step0 = blockIdx.y * k.per, step1 = min(step0 + k.per, k.steps);
  const Pairs wq = lane.weights(k.side[0].w), wk = lane.weights(k.side[1].w);
  v8f c, s;
  turns(k, lane, k.np ? position(k, t) : 0.0, c, s);
  for (int step = step0; step < step1; ++step) {
    const int h = at.head0 + step * k.spread;
    if (h >= k.H) break;
    const bool key = h >= k.Hq;
    const Side& side = k.side[key];
    const int64_t hh = key ? h - k.Hq : h;
    Pairs x = lane.load(reinterpret_cast<const T*>(side.x + t * side.x_token + hh * side.x_head));
    if (k.norm) {
      float q = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) q += x.a[i] * x.a[i] + x.b[i] * x.b[i];
      const float r = 1.0f / sqrtf(row_sum(q, k.lanes) / (float)k.D + k.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x.a[i] *= r * (key ? wk.a[i] : wq.a[i]);
        x.b[i] *= r * (key ? wk.b[i] : wq.b[i]);
      }
    }
    Pairs y;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y.a[i] = x.a[i] * c[i] - x.b[i] * s[i];
      y.b[i] = x.b[i] * c[i] + x.a[i] * s[i];
    }
    lane.store(reinterpret_cast<T*>(side.out + t * side.out_token + hh * side.out_head), y);
  }
}

// Gradient.  The sums of dw stay in registers over a wave's tokens and heads; a
// workgroup adds its waves and lane groups in LDS, in order, and leaves one row per
// side, which k_rope_dw adds up.
template <class T, bool IL, bool VEC>
__global__ __launch_bounds__(kWaves * 64) void k_rope_grad(Args k) {
  __shared__ float sums[2][512];
  const Place at(k);
  const int wave = threadIdx.x >> 6;
  const Lane<T, IL, VEC> lane(k, at.in_row);
  const Pairs wq = lane.weights(k.side[0].w), wk = lane.weights(k.side[1].w);
  Pairs dw[2] = {};
  const int64_t stride = (int64_t)gridDim.x * kWaves * k.tokens;
  const float inv_d = 1.0f / (float)k.D;
  if (at.on)
    for (int64_t t = ((int64_t)blockIdx.x * kWaves + wave) * k.tokens + at.token; t < k.T; t += stride) {
      v8f c, s;
      turns(k, lane, k.np ? position(k, t) : 0.0, c, s);
      for (int h = at.head0; h < k.H; h += k.spread) {
        const bool key = h >= k.Hq;
        const Side& side = k.side[key];
        const int64_t hh = key ? h - k.Hq : h;
        const Pairs dy =
            lane.load(reinterpret_cast<const T*>(side.dy + t * side.dy_token + hh * side.dy_head));
        Pairs x{};
        if (k.norm)
          x = lane.load(reinterpret_cast<const T*>(side.x + t * side.x_token + hh * side.x_head));
        Pairs g;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          g.a[i] = dy.a[i] * c[i] + dy.b[i] * s[i];
          g.b[i] = dy.b[i] * c[i] - dy.a[i] * s[i];
        }
        if (k.norm) {
          float q = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) q += x.a[i] * x.a[i] + x.b[i] * x.b[i];
          const float r = 1.0f / sqrtf(row_sum(q, k.lanes) * inv_d + k.eps);
          float m = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x.a[i] *= r;
            x.b[i] *= r;
            const float da = g.a[i] * x.a[i], db = g.b[i] * x.b[i];
            dw[0].a[i] += key ? 0.0f : da;
            dw[0].b[i] += key ? 0.0f : db;
            dw[1].a[i] += key ? da : 0.0f;
            dw[1].b[i] += key ? db : 0.0f;
            g.a[i] *= key ? wk.a[i] : wq.a[i];
            g.b[i] *= key ? wk.b[i] : wq.b[i];
            m += g.a[i] * x.a[i] + g.b[i] * x.b[i];
          }
          m = row_sum(m, k.lanes) * inv_d;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            g.a[i] = r * (g.a[i] - x.a[i] * m);
            g.b[i] = r * (g.b[i] - x.b[i] * m);
          }
        }
        lane.store(reinterpret_cast<T*>(side.out + t * side.out_token + hh * side.out_head), g);
      }
    }
  if (k.partials == nullptr) return;
  // lane groups of a wave, then the waves one after the other
  for (int m = k.lanes; m < 64; m <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        dw[j].a[i] += __shfl_xor(dw[j].a[i], m);
        dw[j].b[i] += __shfl_xor(dw[j].b[i], m);
      }
  for (int w = 0; w < kWaves; ++w) {
    if (wave == w && (int)(threadIdx.x & 63) < k.lanes)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (lane.has(i)) {
          int a, b;
          place<IL>(k, lane.pair(i), a, b);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            sums[j][a] = (w ? sums[j][a] : 0.0f) + dw[j].a[i];
            sums[j][b] = (w ? sums[j][b] : 0.0f) + dw[j].b[i];
          }
        }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < 2 * k.D; i += kWaves * 64) {
    const int j = i >= k.D;
    k.partials[(int64_t)blockIdx.x * 2 * k.D + i] = sums[j][i - j * k.D];
  }
}

// dw of both sides: 32 columns a workgroup, its 32 groups of lanes take the rows in
// turn; joined in FP64.
__global__ __launch_bounds__(1024) void k_rope_dw(const float* partials, int rows, int D, void* dwq,
                                                  void* dwk, int wide_w) {
  __shared__ double part[32][33];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), group = threadIdx.x >> 5;
  double sum = 0.0;
  if (col < 2 * D) {
#pragma unroll 8
    for (int r = group; r < rows; r += 32) sum += (double)partials[(int64_t)r * 2 * D + col];
  }
  part[group][threadIdx.x & 31] = sum;
  __syncthreads();
  if (group != 0 || col >= 2 * D) return;
  for (int g = 1; g < 32; ++g) sum += part[g][threadIdx.x & 31];
  void* to = col < D ? dwq : dwk;
  const int at = col < D ? col : col - D;
  if (to == nullptr) return;
  if (wide_w)
    store1(static_cast<float*>(to) + at, (float)sum);
  else
    store1(static_cast<bf16_t*>(to) + at, (float)sum);
}

int row_lanes(int64_t D) {
  int n = 1;
  while (n * 16 < D) n *= 2;
  return n;
}

// Heads of a token side by side in a wave, rounds of them, tokens side by side.
void spread(int64_t H, int64_t D, int* lanes, int* width, int* steps, int* tokens) {
  *lanes = row_lanes(D);
  const int groups = 64 / *lanes;
  *steps = (int)((H + groups - 1) / groups);
  *width = (int)((H + *steps - 1) / *steps);
  *tokens = groups / *width;
}

int64_t grad_blocks(int64_t T, int tokens) {
  const int64_t n = (T + (int64_t)kWaves * tokens - 1) / ((int64_t)kWaves * tokens);
  return n < kPartials ? n : kPartials;
}

template <class T, bool IL, bool VEC>
void launch(const Args& k, bool grad, int64_t blocks, int y, hipStream_t s) {
  if (grad)
    k_rope_grad<T, IL, VEC><<<dim3((uint32_t)blocks), kWaves * 64, 0, s>>>(k);
  else
    k_rope<T, IL, VEC><<<grid_xz(blocks, y), kWaves * 64, 0, s>>>(k);
}

template <class T>
void launch(const Args& k, bool il, bool vec, bool grad, int64_t blocks, int y, hipStream_t s) {
  if (il)
    vec ? launch<T, true, true>(k, grad, blocks, y, s) : launch<T, true, false>(k, grad, blocks, y, s);
  else
    vec ? launch<T, false, true>(k, grad, blocks, y, s) : launch<T, false, false>(k, grad, blocks, y, s);
}

}  // namespace

int64_t rope_workspace_bytes(int64_t T, int64_t Hq, int64_t Hkv, int64_t D) {
  if (T == 0 || Hq + Hkv == 0) return 0;
  int lanes, width, steps, tokens;
  spread(Hq + Hkv, D, &lanes, &width, &steps, &tokens);
  return grad_blocks(T, tokens) * 2 * D * 4;
}

hipError_t launch_rope(const RopeCall& c, hipStream_t s) {
  const nvfp4_rope& r = c.r;
  const int64_t el = r.type == NVFP4_TYPE_BF16 ? 2 : 4;
  const bool sums = c.grad && (c.dq_weight != nullptr || c.dk_weight != nullptr);
  const bool rows = r.T > 0 && r.Hq + r.Hkv > 0;
  Args k{};
  int64_t blocks = 0;
  if (rows) {
    auto side = [&](const nvfp4_heads& x, const nvfp4_heads& dy, const nvfp4_heads& out, const void* w) {
      return Side{static_cast<const uint8_t*>(x.p), static_cast<const uint8_t*>(dy.p),
                  static_cast<uint8_t*>(const_cast<void*>(out.p)), w, x.token * el, x.head * el,
                  dy.token * el, dy.head * el, out.token * el, out.head * el};
    };
    k.side[0] = side(c.q, c.dq, c.q_out, r.q_weight);
    k.side[1] = side(c.k, c.dk, c.k_out, r.k_weight);
    k.positions = r.positions;
    k.inv_freq = r.inv_freq;
    k.partials = sums ? static_cast<float*>(c.ws) : nullptr;
    k.T = r.T;
    k.Hq = (int)r.Hq;
    k.H = (int)(r.Hq + r.Hkv);
    k.D = (int)r.D;
    k.np = (int)(r.rot / 2);
    k.nr = (int)((r.D - r.rot) / 2);
    spread(k.H, r.D, &k.lanes, &k.spread, &k.steps, &k.tokens);
    k.wide_ids = r.positions_type == NVFP4_TYPE_I64;
    k.wide_w = r.weight_type == NVFP4_TYPE_F32;
    k.norm = r.norm;
    k.eps = r.eps;
    const bool vec = k.np % 8 == 0 && k.nr % 8 == 0, il = r.interleaved;
    int y = 1;
    if (c.grad) {
      blocks = grad_blocks(r.T, k.tokens);
    } else {
      blocks = (r.T + (int64_t)kWaves * k.tokens - 1) / ((int64_t)kWaves * k.tokens);
      // few tokens: their heads are shared out among waves
      k.per = k.steps;
      while (k.per > 1 && blocks * ((k.steps + k.per - 1) / k.per) < 2 * num_cus()) k.per = (k.per + 1) / 2;
      y = (k.steps + k.per - 1) / k.per;
    }
    if (el == 2)
      launch<bf16_t>(k, il, vec, c.grad, blocks, y, s);
    else
      launch<float>(k, il, vec, c.grad, blocks, y, s);
  }
  if (sums)
    k_rope_dw<<<(uint32_t)((2 * r.D + 31) / 32), 1024, 0, s>>>(
        static_cast<const float*>(c.ws), (int)blocks, (int)r.D, c.dq_weight, c.dk_weight,
        r.weight_type == NVFP4_TYPE_F32);
  return hipGetLastError();
}

}  // namespace nvfp4
