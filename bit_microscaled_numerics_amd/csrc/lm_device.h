// lm_device.h -- device helpers shared by the embedding, cross-entropy and
// gradient-clipping kernels (internal to libnvfp4.so).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nvfp4_device.h"

namespace nvfp4 {

typedef float v8f __attribute__((ext_vector_type(8)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// 16-byte vectors at any element alignment.  Rows of these operators may
// start anywhere (odd widths, strides, pieces of a flat buffer); gfx950 takes
// unaligned 16-byte global accesses, so one path serves every layout.
typedef uint32_t v4u_any2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t v4u_any4 __attribute__((ext_vector_type(4), aligned(4)));

struct bf16_t { uint16_t bits; };

__device__ __forceinline__ v8f unpack8(v4u w) {
  v8f r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[2 * i] = bf16_lo(w[i]);
    r[2 * i + 1] = bf16_hi(w[i]);
  }
  return r;
}

// Round to nearest even; NaN stays NaN (v_cvt_pk_bf16_f32).
__device__ __forceinline__ v4u pack8(v8f v) {
  return __builtin_bit_cast(v4u, __builtin_convertvector(v, v8bf));
}

__device__ __forceinline__ float load1(const bf16_t* p) {
  return __uint_as_float((uint32_t)p->bits << 16);
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(bf16_t* p, float v) {
  p->bits = __builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// Eight consecutive elements as binary32.
__device__ __forceinline__ v8f load8(const bf16_t* p) {
  return unpack8(*reinterpret_cast<const v4u_any2*>(p));
}
__device__ __forceinline__ v8f load8(const float* p) {
  const v4f a = __builtin_bit_cast(v4f, (v4u)*reinterpret_cast<const v4u_any4*>(p));
  const v4f b = __builtin_bit_cast(v4f, (v4u)*reinterpret_cast<const v4u_any4*>(p + 4));
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ void store8(bf16_t* p, v8f v) {
  *reinterpret_cast<v4u_any2*>(p) = pack8(v);
}
__device__ __forceinline__ void store8(float* p, v8f v) {
  *reinterpret_cast<v4u_any4*>(p) =
      __builtin_bit_cast(v4u, __builtin_shufflevector(v, v, 0, 1, 2, 3));
  *reinterpret_cast<v4u_any4*>(p + 4) =
      __builtin_bit_cast(v4u, __builtin_shufflevector(v, v, 4, 5, 6, 7));
}

// Eight columns of a row for the thread whose own begin at c: at the end of a row
// whose width is no multiple of 8 they are the row's last eight, of which the first
// `skip` belong to the thread before.  (A loop over the few columns left would put
// the latency of a whole sum behind each.)  Needs dim >= 8.
struct Cols {
  int64_t at;
  int skip;
  __device__ __forceinline__ Cols(int64_t c, int64_t dim)
      : at(c + 8 <= dim ? c : dim - 8), skip((int)(c - (c + 8 <= dim ? c : dim - 8))) {}
};

// The eight values to the row, without the first `skip`.
template <class T>
__device__ __forceinline__ void store8_from(T* row, Cols k, v8f v) {
  if (k.skip == 0) {
    store8(row + k.at, v);
    return;
  }
#pragma unroll
  for (int i = 1; i < 8; ++i)
    if (i >= k.skip) store1(row + k.at + i, v[i]);
}

// One dimension of a launch holds fewer than 2^32 threads; a grid past that is taken
// modulo 2^32 without an error.  Workgroups that are counted by tokens therefore lie
// along x up to kGridX and go on along z.
constexpr int64_t kGridX = int64_t(1) << 21;

inline dim3 grid_xz(int64_t blocks, int64_t y = 1) {
  return dim3((uint32_t)(blocks < kGridX ? blocks : kGridX), (uint32_t)y,
              (uint32_t)((blocks + kGridX - 1) / kGridX));
}
__device__ __forceinline__ int64_t block_xz() { return (int64_t)blockIdx.z * kGridX + blockIdx.x; }

// A wave-uniform value moved to a scalar register.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform64(int64_t x) {
  const uint32_t lo = (uint32_t)uniform((int)(uint32_t)x);
  const uint32_t hi = (uint32_t)uniform((int)(uint32_t)((uint64_t)x >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// The lane number, opaque: addresses derived from it are formed where they are
// used.  In a loop over tiles the compiler otherwise keeps them all across the
// loop; where the products need every register, in scratch memory, and reloads
// them one by one (8000 to 15000 cycles a tile).
__device__ __forceinline__ int fresh_lane() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}

}  // namespace nvfp4
