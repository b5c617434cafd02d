// lm_clip.hip -- the global norm of many gradient tensors, and clipping.
//
//   n = sqrt(sum over all tensors of g^2),  c = min(1, max_norm / (n + 1e-6)),
//   out = c * g
//
// Two passes over the gradients, both bound by HBM: of 629M BF16 values the sums take
// 203 us (6.2 TB/s), the products 443 us (5.7 TB/s).  The tensors come as a
// table in the kernel arguments (up to kBatch per launch): nothing is copied
// to the device, so a call can be captured and needs no plan.
//
// Squares are summed in binary64: the square of a binary32 value is exact
// there to 48 bits and cannot overflow, so the norm is right for gradients of
// any size and its value does not depend on how the work was split (to about
// 2^-50).  Each workgroup leaves its sum in its own word of `partials`; the
// total is the sum of the words, taken in a fixed order by every workgroup of
// the second pass, so no atomics and no third launch are needed, and partial
// sums of several processes can be added word by word.
#include "lm_device.h"
#include "lm_kernels.h"

namespace nvfp4 {

namespace {

// The results are not read again here: stored without a place in the 256 MB cache,
// they leave it to the gradients, and their writes do not trail into the next pass.
__device__ __forceinline__ void store8_once(bf16_t* p, v8f v) {
  __builtin_nontemporal_store((v4u_any2)pack8(v), reinterpret_cast<v4u_any2*>(p));
}
__device__ __forceinline__ void store8_once(float* p, v8f v) {
  const v4u lo = __builtin_bit_cast(v4u, __builtin_shufflevector(v, v, 0, 1, 2, 3));
  const v4u hi = __builtin_bit_cast(v4u, __builtin_shufflevector(v, v, 4, 5, 6, 7));
  __builtin_nontemporal_store((v4u_any4)lo, reinterpret_cast<v4u_any4*>(p));
  __builtin_nontemporal_store((v4u_any4)hi, reinterpret_cast<v4u_any4*>(p + 4));
}

constexpr int kThreads = 256;
constexpr int kWords = NVFP4_SUMSQ_WORDS;     // = workgroups of a launch
constexpr int kVecs = 8;                      // 16-byte vectors per thread and chunk
constexpr int64_t kChunkBytes = 16 * kVecs * kThreads;   // 32 KiB of input
constexpr int kBatch = 96;                    // tensors per launch (kernel arguments stay below 4 KiB)

struct Table {
  const void* in[kBatch];
  void* out[kBatch];
  int64_t numel[kBatch];
  uint32_t first_chunk[kBatch + 1];   // of each tensor, in this launch
  uint8_t types[kBatch];              // bit 0: input FP32, bit 1: output FP32
  int count;
};

__device__ __forceinline__ double sumsq8(v8f v) {
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = __builtin_fma((double)v[i], (double)v[i], s);
  return s;
}

// The squares of elements [i0, i1) of one tensor.
template <class T>
__device__ __forceinline__ double chunk_sumsq(const T* __restrict__ x, int64_t i0, int64_t i1) {
  constexpr int kPer = kChunkBytes / sizeof(T) / (8 * kThreads);   // 8-element vectors per thread
  double s = 0.0;
  if (i1 - i0 == (int64_t)(kChunkBytes / sizeof(T))) {
    v8f v[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) v[u] = load8(x + i0 + 8 * (u * kThreads + threadIdx.x));
#pragma unroll
    for (int u = 0; u < kPer; ++u) s += sumsq8(v[u]);
    return s;
  }
  for (int64_t i = i0 + 8 * threadIdx.x; i < i1; i += 8 * kThreads) {
    if (i + 8 <= i1) {
      s += sumsq8(load8(x + i));
    } else {
      for (int64_t k = i; k < i1; ++k) {
        const double d = load1(x + k);
        s = __builtin_fma(d, d, s);
      }
    }
  }
  return s;
}

// Sum over the workgroup in a fixed order; the result in every thread.
__device__ __forceinline__ double block_sum(double v, double* scratch) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) s += scratch[w];
  return s;
}

// add: a later batch of the same list adds to the words of the earlier ones.
__global__ __launch_bounds__(kThreads) void k_grad_sumsq(Table t, double* __restrict__ partials,
                                                         int add) {
  __shared__ double scratch[kThreads / 64];
  double s = 0.0;
  int k = 0;
  for (uint32_t c = blockIdx.x; c < t.first_chunk[t.count]; c += gridDim.x) {
    while (c >= t.first_chunk[k + 1]) ++k;
    const int64_t per = kChunkBytes / ((t.types[k] & 1) ? 4 : 2);
    const int64_t i0 = (int64_t)(c - t.first_chunk[k]) * per;
    const int64_t i1 = i0 + per < t.numel[k] ? i0 + per : t.numel[k];
    s += (t.types[k] & 1) ? chunk_sumsq(reinterpret_cast<const float*>(t.in[k]), i0, i1)
                          : chunk_sumsq(reinterpret_cast<const bf16_t*>(t.in[k]), i0, i1);
  }
  s = block_sum(s, scratch);
  if (threadIdx.x == 0) partials[blockIdx.x] = add ? partials[blockIdx.x] + s : s;
}

template <class T, class O>
__device__ __forceinline__ void chunk_scale(const T* x, O* out, int64_t i0, int64_t i1, float c) {
  constexpr int kPer = kChunkBytes / sizeof(T) / (8 * kThreads);
  if (i1 - i0 == (int64_t)(kChunkBytes / sizeof(T))) {
    v8f v[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) v[u] = load8(x + i0 + 8 * (u * kThreads + threadIdx.x));
#pragma unroll
    for (int u = 0; u < kPer; ++u) store8_once(out + i0 + 8 * (u * kThreads + threadIdx.x), v[u] * c);
    return;
  }
  for (int64_t i = i0 + 8 * threadIdx.x; i < i1; i += 8 * kThreads) {
    if (i + 8 <= i1) {
      store8(out + i, load8(x + i) * c);
    } else {
      for (int64_t k = i; k < i1; ++k) store1(out + k, load1(x + k) * c);
    }
  }
}

// out = coef * in over the whole table, whose tensors are in reverse order; the
// chunks of each are taken last first as well: the pass before ended there, and
// what it read last is still in the 256 MB cache.  100M FP32 values into BF16:
// 172 us first to last, 160 us so (183 us with ordinary stores too); 629M BF16
// values 671 and 649 us (685 us).
__device__ __forceinline__ void scale_table(const Table& t, float coef) {
  int k = 0;
  for (uint32_t c = blockIdx.x; c < t.first_chunk[t.count]; c += gridDim.x) {
    while (c >= t.first_chunk[k + 1]) ++k;
    if (coef == 1.0f && t.in[k] == t.out[k]) continue;   // in place, nothing to change
    const int64_t per = kChunkBytes / ((t.types[k] & 1) ? 4 : 2);
    const int64_t i0 = (int64_t)(t.first_chunk[k + 1] - 1 - c) * per;
    const int64_t i1 = i0 + per < t.numel[k] ? i0 + per : t.numel[k];
    const auto* xb = reinterpret_cast<const bf16_t*>(t.in[k]);
    const auto* xf = reinterpret_cast<const float*>(t.in[k]);
    auto* ob = reinterpret_cast<bf16_t*>(t.out[k]);
    auto* of = reinterpret_cast<float*>(t.out[k]);
    switch (t.types[k]) {
      case 0: chunk_scale(xb, ob, i0, i1, coef); break;
      case 1: chunk_scale(xf, ob, i0, i1, coef); break;
      case 2: chunk_scale(xb, of, i0, i1, coef); break;
      default: chunk_scale(xf, of, i0, i1, coef); break;
    }
  }
}

__global__ __launch_bounds__(kThreads) void k_grad_clip(Table t, const double* __restrict__ partials,
                                                        double max_norm, float* norm_out) {
  __shared__ double scratch[kThreads / 64];
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kWords / kThreads; ++i) s += partials[i * kThreads + threadIdx.x];
  const double norm = __builtin_sqrt(block_sum(s, scratch));
  const double ratio = max_norm / (norm + 1e-6);
  const float coef = ratio > 1.0 ? 1.0f : (float)ratio;   // a NaN norm stays NaN
  if (norm_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  scale_table(t, coef);
}

__global__ __launch_bounds__(kThreads) void k_grad_scale(Table t, const float* __restrict__ factor) {
  scale_table(t, *factor);
}

// Put a gradient at the end of the table; false: the table is full, or its chunk
// count would pass 31 bits (one tensor alone has at most 2^27 chunks).
bool put(Table& t, const nvfp4_grad& g) {
  if (g.numel == 0) return true;
  const int in32 = g.in_type == NVFP4_TYPE_F32, out32 = g.out_type == NVFP4_TYPE_F32;
  const int64_t per = kChunkBytes / (in32 ? 4 : 2), n = (g.numel + per - 1) / per;
  const int64_t chunks = t.first_chunk[t.count] + n;
  if (t.count == kBatch || chunks > (int64_t(1) << 31) - 1) return false;
  t.in[t.count] = g.in;
  t.out[t.count] = g.out;
  t.numel[t.count] = g.numel;
  t.types[t.count] = (uint8_t)(in32 | out32 << 1);
  t.first_chunk[++t.count] = (uint32_t)chunks;
  return true;
}

// The batch of the list that starts at `at`; returns its end.
int64_t batch_from(const nvfp4_grad* list, int64_t count, int64_t at, Table& t) {
  t.count = 0;
  t.first_chunk[0] = 0;
  while (at < count && put(t, list[at])) ++at;
  return at;
}

// The batch that ends before `end`, last gradient first; returns its start.
int64_t batch_before(const nvfp4_grad* list, int64_t end, Table& t) {
  t.count = 0;
  t.first_chunk[0] = 0;
  while (end > 0 && put(t, list[end - 1])) --end;
  return end;
}

}  // namespace

hipError_t launch_grad_sumsq(const nvfp4_grad* list, int64_t count, double* partials,
                             hipStream_t s) {
  static_assert(sizeof(Table) + 32 < 4096, "kernel arguments");
  Table t;
  int64_t at = 0;
  int add = 0;
  do {   // at least once: an empty list leaves zeros
    at = batch_from(list, count, at, t);
    hipLaunchKernelGGL(k_grad_sumsq, dim3(kWords), dim3(kThreads), 0, s, t, partials, add);
    add = 1;
  } while (at < count);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const nvfp4_grad* list, int64_t count, const double* partials,
                            double max_norm, float* norm_out, hipStream_t s) {
  Table t;
  int64_t end = count;
  do {   // at least once, for the norm
    end = batch_before(list, end, t);
    hipLaunchKernelGGL(k_grad_clip, dim3(kWords), dim3(kThreads), 0, s, t, partials, max_norm,
                       norm_out);
    norm_out = nullptr;
  } while (end > 0);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const nvfp4_grad* list, int64_t count, const float* factor,
                             hipStream_t s) {
  Table t;
  for (int64_t end = count; end > 0;) {
    end = batch_before(list, end, t);
    hipLaunchKernelGGL(k_grad_scale, dim3(kWords), dim3(kThreads), 0, s, t, factor);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
