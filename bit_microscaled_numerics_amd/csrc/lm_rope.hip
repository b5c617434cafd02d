// lm_rope.hip -- norms of queries and keys for each head with the position rotation in
// the same pass, and the gradient (internal to libnvfp4.so).
//
// A row of D values is taken as D/2 pairs: the rot/2 rotated ones, then the rest of the
// row as the pairs of its halves, which are not rotated.  A lane owns 8 pairs, in the
// gradient 4; 1 .. 64 lanes make a row, so that a rotation needs no exchange and a norm a few shuffles.
// A wave takes all heads of a token (several tokens, where they are few): the
// sines and cosines of a lane's pairs are formed once for all of them.
//
// Bound by HBM: 4 bytes per value (BF16), 6 in the gradient; there the vector units are as busy (71%) as in the
// forward kernel, and two dependent sums a row leave the waves waiting for 56% of their time (forward 48%): 4.5
// TB/s of 5.9, where the forward kernel has 5.5.  Widths whose pairs are no multiple of 8 (4 in the gradient)
// load value by value: 8192 tokens of 48 heads of 72, 53 us where the bytes take 19.
#include <hip/hip_runtime.h>

#include "lm_attn_kernels.h"
#include "lm_device.h"
#include "lm_kernels.h"

namespace nvfp4 {
namespace {

constexpr int kWaves = 4;        // waves of a workgroup
constexpr int kPartials = 4096;  // most workgroups of the gradient, each with a row of sums of dw

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
  float* partials;   // gradient: [workgroup][D]
  int64_t T;
  int Hq, H, D, np, nr;     // np rotated pairs, nr others
  int lanes;                // per row, a power of two
  int spread[2], tokens[2]; // heads of a token, and tokens, that lie side by side in a wave
  int steps, per;           // rounds of heads, and per wave
  int blocks[2];            // gradient: workgroups of each side
  int wide_ids, wide_w, norm;
  float eps;
};

// Four consecutive elements as binary32, at any element alignment.
typedef uint32_t v2u_any2 __attribute__((ext_vector_type(2), aligned(2)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void store4(bf16_t* p, v4f v) {
  *reinterpret_cast<v2u_any2*>(p) = __builtin_bit_cast(v2u_any2, __builtin_convertvector(v, v4bf));
}
__device__ __forceinline__ void store4(float* p, v4f v) {
  *reinterpret_cast<v4u_any4*>(p) = __builtin_bit_cast(v4u, v);
}

// N consecutive elements as they lie in memory, at any element alignment, and as binary32.
// Rows are loaded ahead of their use and kept as they lie: unpacked at once they would be waited
// for at once.
template <class T, int N> struct Vec;
template <> struct Vec<bf16_t, 4> {
  typedef v4f type;
  typedef v2u_any2 raw;
  static __device__ __forceinline__ v4f unpack(raw w) { return v4f{bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])}; }
};
template <> struct Vec<bf16_t, 8> {
  typedef v8f type;
  typedef v4u_any2 raw;
  static __device__ __forceinline__ v8f unpack(raw w) { return unpack8(w); }
};
template <> struct Vec<float, 4> {
  typedef v4f type;
  typedef v4u_any4 raw;
  static __device__ __forceinline__ v4f unpack(raw w) { return __builtin_bit_cast(v4f, (v4u)w); }
};
template <> struct Vec<float, 8> {
  typedef v8f type;
  struct raw { v4u_any4 lo, hi; };
  static __device__ __forceinline__ v8f unpack(raw w) {
    return __builtin_shufflevector(__builtin_bit_cast(v4f, (v4u)w.lo), __builtin_bit_cast(v4f, (v4u)w.hi), 0, 1, 2, 3, 4, 5, 6, 7);
  }
};
template <int N> using vfloat = typename Vec<float, N>::type;
template <class T> __device__ __forceinline__ void storev(T* p, v4f v) { store4(p, v); }
template <class T> __device__ __forceinline__ void storev(T* p, v8f v) { store8(p, v); }

// N pairs of a row.
template <int N>
struct Pairs {
  vfloat<N> a, b;
};

// The sum over a row's lanes, in every one of them.
__device__ __forceinline__ float row_sum(float x, int lanes) {
#define MOVED(how) __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), how, 15, 15, true))
  if (lanes > 1) x += MOVED(0xB1);    // the other one of two
  if (lanes > 2) x += MOVED(0x4E);    // the other two of four
  if (lanes > 4) x += MOVED(0x141);   // mirrored within 8
  if (lanes > 8) x += MOVED(0x140);   // mirrored within 16
#undef MOVED
  if (lanes > 16) x += __shfl_xor(x, 16);
  if (lanes > 32) x += __shfl_xor(x, 32);
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

// A lane's N pairs: consecutive ones (VEC: all rotated or none, pieces of 2 N bytes of a BF16
// row), or such that lie a row's lanes apart.
template <bool IL, bool VEC, int N>
struct Lane {
  const Args& k;
  int first, live;
  __device__ __forceinline__ Lane(const Args& args, int in_row) : k(args) {
    first = VEC ? in_row * N : in_row;
    live = (k.np + k.nr) - first;   // pairs from here on
  }
  __device__ __forceinline__ bool has(int i) const { return (VEC ? i : i * k.lanes) < live; }
  __device__ __forceinline__ int pair(int i) const { return first + (VEC ? i : i * k.lanes); }
  __device__ __forceinline__ bool together() const { return IL && first < k.np; }   // VEC: pairs side by side
  // VEC: where the lane's two pieces of N begin.
  __device__ __forceinline__ void pieces(int& a, int& b) const {
    if (together()) {
      a = 2 * first;
      b = a + N;
    } else {
      place<false>(k, first, a, b);
    }
  }

  template <class T, bool V> struct RawOf { struct type { typename Vec<T, N>::raw a, b; }; };
  template <class T> struct RawOf<T, false> { typedef Pairs<N> type; };
  template <class T> using Raw = typename RawOf<T, VEC>::type;

  template <class T>
  __device__ __forceinline__ Raw<T> load(const T* row) const {
    Raw<T> p{};
    if constexpr (VEC) {
      if (live > 0) {
        int a, b;
        pieces(a, b);
        p.a = *reinterpret_cast<const typename Vec<T, N>::raw*>(row + a);
        p.b = *reinterpret_cast<const typename Vec<T, N>::raw*>(row + b);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (has(i)) {
          int a, b;
          place<IL>(k, pair(i), a, b);
          p.a[i] = load1(row + a);
          p.b[i] = load1(row + b);
        }
    }
    return p;
  }
  template <class T>
  __device__ __forceinline__ Pairs<N> unpack(const Raw<T>& w) const {
    if constexpr (VEC) {
      const Pairs<N> x{Vec<T, N>::unpack(w.a), Vec<T, N>::unpack(w.b)};
      if (!together()) return x;
      Pairs<N> p;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        p.a[i] = i < N / 2 ? x.a[2 * i] : x.b[2 * i - N];
        p.b[i] = i < N / 2 ? x.a[2 * i + 1] : x.b[2 * i + 1 - N];
      }
      return p;
    } else {
      return w;
    }
  }
  template <class T>
  __device__ __forceinline__ void store(T* row, Pairs<N> p) const {
    if constexpr (VEC) {
      if (live > 0) {
        int a, b;
        pieces(a, b);
        if (together()) {
          Pairs<N> q;   // as they lie
#pragma unroll
          for (int i = 0; i < N; ++i) {
            q.a[i] = i & 1 ? p.b[i / 2] : p.a[i / 2];
            q.b[i] = i & 1 ? p.b[(i + N) / 2] : p.a[(i + N) / 2];
          }
          p = q;
        }
        storev(row + a, p.a);
        storev(row + b, p.b);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (has(i)) {
          int a, b;
          place<IL>(k, pair(i), a, b);
          store1(row + a, p.a[i]);
          store1(row + b, p.b[i]);
        }
    }
  }
  __device__ __forceinline__ Pairs<N> weights(const void* w) const {
    if (w == nullptr) {
      Pairs<N> p;
      p.a = p.b = 1.0f;
      return p;
    }
    return k.wide_w ? unpack<float>(load(static_cast<const float*>(w)))
                    : unpack<bf16_t>(load(static_cast<const bf16_t*>(w)));
  }
};

// cos and sin of a lane's pairs.  The angle in turns: position * inv_freq in FP64
// (exact up to positions of 2^29), times 1/(2 pi) in two parts with the whole turns
// taken off by a fused multiply-add, so a far position costs no accuracy.
template <bool IL, bool VEC, int N>
__device__ __forceinline__ void turns(const Args& k, const Lane<IL, VEC, N>& at, double pos, vfloat<N>& c,
                                      vfloat<N>& s) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591011e-18;
#pragma unroll
  for (int i = 0; i < N; ++i) {
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
  __device__ __forceinline__ Place(const Args& k, int side) {
    const int lane = threadIdx.x & 63, group = lane >> __builtin_ctz(k.lanes);
    in_row = lane & (k.lanes - 1);
    token = group / k.spread[side];
    head0 = group - token * k.spread[side];
    on = token < k.tokens[side];
  }
};

// One row's norm, weight and rotation.
template <int N, class V>
__device__ __forceinline__ Pairs<N> forward_row(const Args& k, Pairs<N> x, const Pairs<N>& w, const V& c, const V& s) {
  if (k.norm) {
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) q += x.a[i] * x.a[i] + x.b[i] * x.b[i];
    const float r = 1.0f / sqrtf(row_sum(q, k.lanes) / (float)k.D + k.eps);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x.a[i] *= r * w.a[i];
      x.b[i] *= r * w.b[i];
    }
  }
  Pairs<N> y;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    y.a[i] = x.a[i] * c[i] - x.b[i] * s[i];
    y.b[i] = x.b[i] * c[i] + x.a[i] * s[i];
  }
  return y;
}

// Queries and keys of a token by one wave; the next row is loaded before one is worked on.
template <class T, bool IL, bool VEC, int N>
__global__ __launch_bounds__(kWaves * 64) void k_rope(Args k) {
  const Place at(k, 0);
  const int wave = threadIdx.x >> 6;
  const int64_t t = (block_xz() * kWaves + wave) * k.tokens[0] + at.token;
  if (!at.on || t >= k.T) return;
  const Lane<IL, VEC, N> lane(k, at.in_row);
  const int end = min(k.H, at.head0 + min((int)(blockIdx.y + 1) * k.per, k.steps) * k.spread[0]);
  int h = at.head0 + blockIdx.y * k.per * k.spread[0];
  auto row = [&](int h) {
    const bool key = h >= k.Hq;
    const Side& side = k.side[key];
    return lane.load(reinterpret_cast<const T*>(side.x + t * side.x_token + (int64_t)(key ? h - k.Hq : h) * side.x_head));
  };
  if (h >= end) return;
  auto x = row(h);
  const Pairs<N> wq = lane.weights(k.side[0].w), wk = lane.weights(k.side[1].w);
  vfloat<N> c, s;
  turns(k, lane, k.np ? position(k, t) : 0.0, c, s);
  while (h < end) {
    const int next = h + k.spread[0];
    decltype(x) nx{};
    if (next < end) nx = row(next);
    const bool key = h >= k.Hq;
    const Side& side = k.side[key];
    Pairs<N> w;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      w.a[i] = key ? wk.a[i] : wq.a[i];
      w.b[i] = key ? wk.b[i] : wq.b[i];
    }
    lane.store(reinterpret_cast<T*>(side.out + t * side.out_token + (int64_t)(key ? h - k.Hq : h) * side.out_head),
               forward_row(k, lane.template unpack<T>(x), w, c, s));
    x = nx;
    h = next;
  }
}

// Gradient; queries and keys by workgroups of their own.  The sums of dw stay in registers
// over a wave's tokens and heads; a workgroup adds its lane groups and waves in LDS, in order,
// and leaves one row, which k_rope_dw adds up.
template <class T, bool IL, bool VEC, int N>
__global__ __launch_bounds__(kWaves * 64) void k_rope_grad(Args k) {
  __shared__ float sums[512];
  const int j = (int)blockIdx.x >= k.blocks[0], block = blockIdx.x - (j ? k.blocks[0] : 0);
  const Side& side = k.side[j];
  const int H = j ? k.H - k.Hq : k.Hq;
  const Place at(k, j);
  const int wave = threadIdx.x >> 6;
  const Lane<IL, VEC, N> lane(k, at.in_row);
  const Pairs<N> w = lane.weights(side.w);
  Pairs<N> dw{};
  const int64_t stride = (int64_t)k.blocks[j] * kWaves * k.tokens[j];
  const float inv_d = 1.0f / (float)k.D;
  int64_t t = ((int64_t)block * kWaves + wave) * k.tokens[j] + at.token;
  if (at.on && at.head0 < H) {
    struct Row {
      typename Lane<IL, VEC, N>::template Raw<T> dy, x;
    };
    int64_t ahead_t = t;
    int ahead_h = at.head0;
    auto fetch = [&]() {   // the row that is two on
      Row r{};
      if (ahead_t >= k.T) return r;
      r.dy = lane.load(reinterpret_cast<const T*>(side.dy + ahead_t * side.dy_token + ahead_h * side.dy_head));
      if (k.norm) r.x = lane.load(reinterpret_cast<const T*>(side.x + ahead_t * side.x_token + ahead_h * side.x_head));
      ahead_h += k.spread[j];
      if (ahead_h >= H) ahead_h = at.head0, ahead_t += stride;
      return r;
    };
    Row first = fetch(), second = fetch();
    double pos = k.np && t < k.T ? position(k, t) : 0.0;
    for (; t < k.T; t += stride) {
      vfloat<N> c, s;
      turns(k, lane, pos, c, s);
      if (k.np && t + stride < k.T) pos = position(k, t + stride);
      for (int h = at.head0; h < H; h += k.spread[j]) {
        const Pairs<N> dy = lane.template unpack<T>(first.dy);
        Pairs<N> g, n = lane.template unpack<T>(first.x);
        first = second;
        second = fetch();
#pragma unroll
        for (int i = 0; i < N; ++i) {
          g.a[i] = dy.a[i] * c[i] + dy.b[i] * s[i];
          g.b[i] = dy.b[i] * c[i] - dy.a[i] * s[i];
        }
        if (k.norm) {
          float q = 0.0f;
#pragma unroll
          for (int i = 0; i < N; ++i) q += n.a[i] * n.a[i] + n.b[i] * n.b[i];
          float r = 1.0f / sqrtf(row_sum(q, k.lanes) * inv_d + k.eps), m = 0.0f;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            n.a[i] *= r;
            n.b[i] *= r;
            m += g.a[i] * n.a[i] * w.a[i] + g.b[i] * n.b[i] * w.b[i];
          }
          m = row_sum(m, k.lanes) * inv_d;
          // A row that takes no gradient (a token of no sequence) adds nothing, whatever it holds: 0
          // times NaN would reach dw through it.  m is the row's, so all its lanes are here or none.
          if (m != m) {
            float some = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) some += (g.a[i] != 0.0f || g.b[i] != 0.0f) ? 1.0f : 0.0f;
            if (row_sum(some, k.lanes) == 0.0f) {
              n.a = n.b = 0.0f;
              m = r = 0.0f;
            }
          }
#pragma unroll
          for (int i = 0; i < N; ++i) {
            dw.a[i] += g.a[i] * n.a[i];
            dw.b[i] += g.b[i] * n.b[i];
            g.a[i] = r * (g.a[i] * w.a[i] - n.a[i] * m);
            g.b[i] = r * (g.b[i] * w.b[i] - n.b[i] * m);
          }
        }
        lane.store(reinterpret_cast<T*>(side.out + t * side.out_token + h * side.out_head), g);
      }
    }
  }
  if (k.partials == nullptr) return;
  // lane groups of a wave, then the waves one after the other
  for (int m = k.lanes; m < 64; m <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      dw.a[i] += __shfl_xor(dw.a[i], m);
      dw.b[i] += __shfl_xor(dw.b[i], m);
    }
  for (int v = 0; v < kWaves; ++v) {
    if (wave == v && (int)(threadIdx.x & 63) < k.lanes)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (lane.has(i)) {
          int a, b;
          place<IL>(k, lane.pair(i), a, b);
          sums[a] = (v ? sums[a] : 0.0f) + dw.a[i];
          sums[b] = (v ? sums[b] : 0.0f) + dw.b[i];
        }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < k.D; i += kWaves * 64) k.partials[(int64_t)blockIdx.x * k.D + i] = sums[i];
}

// dw of both sides (along y): 32 columns a workgroup, its 32 groups of lanes take the
// side's rows in turn; joined in FP64.
__global__ __launch_bounds__(1024) void k_rope_dw(const float* partials, int rows_q, int rows_k, int D, void* dwq,
                                                  void* dwk, int wide_w) {
  __shared__ double part[32][33];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), group = threadIdx.x >> 5;
  const int first = blockIdx.y ? rows_q : 0, end = blockIdx.y ? rows_q + rows_k : rows_q;
  double sum = 0.0;
  if (col < D) {
#pragma unroll 8
    for (int r = first + group; r < end; r += 32) sum += (double)partials[(int64_t)r * D + col];
  }
  part[group][threadIdx.x & 31] = sum;
  __syncthreads();
  void* to = blockIdx.y ? dwk : dwq;
  if (group != 0 || col >= D || to == nullptr) return;
  for (int g = 1; g < 32; ++g) sum += part[g][threadIdx.x & 31];
  if (wide_w)
    store1(static_cast<float*>(to) + col, (float)sum);
  else
    store1(static_cast<bf16_t*>(to) + col, (float)sum);
}

// Pairs of a lane.  Forward 8, 16-byte loads of BF16 (kernel of 8192 tokens of 48 heads of 128: 36.7 us, 38.0 with
// 4); the gradient, which holds three times the registers, 4 (67.2 us, 78.4 with 8).
constexpr int kForward = 8, kGradient = 4;

// Lanes of a row; heads of a token side by side in a wave, and tokens side by side.
void spread(int64_t H, int64_t D, int pairs, int* lanes, int* width, int* tokens) {
  *lanes = 1;
  while (*lanes * 2 * pairs < D) *lanes *= 2;
  const int64_t groups = 64 / *lanes, steps = H > 0 ? (H + groups - 1) / groups : 1;
  *width = H > 0 ? (int)((H + steps - 1) / steps) : 1;
  *tokens = (int)(groups / *width);
}

int64_t token_blocks(int64_t T, int tokens) {
  return (T + (int64_t)kWaves * tokens - 1) / ((int64_t)kWaves * tokens);
}

// Workgroups of the gradient for queries and keys: at most kPartials, shared out by rows.
void grad_blocks(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, Args* k) {
  spread(Hq, D, kGradient, &k->lanes, &k->spread[0], &k->tokens[0]);
  spread(Hkv, D, kGradient, &k->lanes, &k->spread[1], &k->tokens[1]);
  const int64_t share = Hq + Hkv > 0 ? (kPartials * Hkv + Hq + Hkv - 1) / (Hq + Hkv) : 0;
  const int64_t heads[2] = {Hq, Hkv}, most[2] = {kPartials - share > 1 ? kPartials - share : 1, share > 1 ? share : 1};
  for (int j = 0; j < 2; ++j) {
    const int64_t n = heads[j] > 0 ? token_blocks(T, k->tokens[j]) : 0;
    const int64_t rounds = n == 0 ? 1 : (n + most[j] - 1) / most[j];
    k->blocks[j] = (int)((n + rounds - 1) / rounds);   // as many tokens for each
  }
}

template <class T, bool IL, bool VEC>
void launch(const Args& k, bool grad, int64_t blocks, int y, hipStream_t s) {
  if (grad)
    k_rope_grad<T, IL, VEC, kGradient><<<dim3((uint32_t)blocks), kWaves * 64, 0, s>>>(k);
  else
    k_rope<T, IL, VEC, kForward><<<grid_xz(blocks, y), kWaves * 64, 0, s>>>(k);
}

template <class T>
void launch(const Args& k, bool grad, int64_t blocks, int y, bool il, bool vec, hipStream_t s) {
  if (il)
    vec ? launch<T, true, true>(k, grad, blocks, y, s) : launch<T, true, false>(k, grad, blocks, y, s);
  else
    vec ? launch<T, false, true>(k, grad, blocks, y, s) : launch<T, false, false>(k, grad, blocks, y, s);
}

}  // namespace

int64_t rope_workspace_bytes(int64_t T, int64_t Hq, int64_t Hkv, int64_t D) {
  Args k{};
  grad_blocks(T, Hq, Hkv, D, &k);
  return (int64_t)(k.blocks[0] + k.blocks[1]) * D * 4;
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
    k.wide_ids = r.positions_type == NVFP4_TYPE_I64;
    k.wide_w = r.weight_type == NVFP4_TYPE_F32;
    k.norm = r.norm;
    k.eps = r.eps;
    const int pairs = c.grad ? kGradient : kForward;
    const bool vec = k.np % pairs == 0 && k.nr % pairs == 0, il = r.interleaved;
    int y = 1;
    if (c.grad) {
      grad_blocks(r.T, r.Hq, r.Hkv, r.D, &k);
      blocks = k.blocks[0] + k.blocks[1];
    } else {
      spread(k.H, r.D, kForward, &k.lanes, &k.spread[0], &k.tokens[0]);
      k.steps = (k.H + k.spread[0] - 1) / k.spread[0];
      blocks = token_blocks(r.T, k.tokens[0]);
      // few tokens: their heads are shared out among waves
      k.per = k.steps;
      while (k.per > 1 && blocks * ((k.steps + k.per - 1) / k.per) < 2 * num_cus()) k.per = (k.per + 1) / 2;
      y = (k.steps + k.per - 1) / k.per;
    }
    if (el == 2)
      launch<bf16_t>(k, c.grad, blocks, y, il, vec, s);
    else
      launch<float>(k, c.grad, blocks, y, il, vec, s);
  }
  if (sums)
    k_rope_dw<<<dim3((uint32_t)((r.D + 31) / 32), 2), 1024, 0, s>>>(
        static_cast<const float*>(c.ws), k.blocks[0], k.blocks[1], (int)r.D, c.dq_weight, c.dk_weight,
        r.weight_type == NVFP4_TYPE_F32);
  return hipGetLastError();
}

}  // namespace nvfp4
