// lm_embed.hip -- token embedding with scaling, and its gradient.
//
//   forward   y[t] = scale * W[id_t]                       (a row of zeros where
//                                                           id_t is outside [0, V))
//   gradient  dW[v] = scale * sum over {t : id_t = v} dY[t]
//
// Both are bound by HBM: the forward moves T * D elements in and out, the
// gradient reads T * D and writes all V * D.  The gradient is deterministic:
// a stable sort of the tokens by id puts the rows of one word side by side in
// ascending t, and every dW row is one FP32 sum in that order, written once
// (no atomics, no zeroing pass).
#include "lm_device.h"
#include "lm_kernels.h"

namespace nvfp4 {

namespace {

constexpr uint32_t kNoKey = 0xFFFFFFFFu;

__device__ __forceinline__ int64_t load_id(const void* ids, bool wide, int64_t t) {
  return wide ? reinterpret_cast<const int64_t*>(ids)[t]
              : (int64_t) reinterpret_cast<const int32_t*>(ids)[t];
}

// ------------------------------------------------------------------ forward
// One wave per token and column range: the id is loaded once into a scalar
// register, so the row base is scalar and each lane moves 16 bytes of BF16
// (32 of FP32) per vector, up to four vectors in flight.  blockIdx.y cuts the
// columns when there are too few tokens to fill the chip.
constexpr int kEmbedWaves = 4, kVec = 8, kWaveCols = 64 * kVec;

template <class W, class O>
__global__ __launch_bounds__(64 * kEmbedWaves) void k_embed(EmbedArgs a, const W* __restrict__ w,
                                                            int64_t ldw, O* __restrict__ out,
                                                            int64_t ldo, int64_t cols_per) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * kEmbedWaves + uniform(threadIdx.x >> 6);
  if (t >= a.n) return;
  const int64_t id = uniform64(load_id(a.ids, a.ids_type == NVFP4_TYPE_I64, t));
  const bool live = id >= 0 && id < a.vocab;
  const W* src = w + (live ? id : 0) * ldw;
  O* dst = out + t * ldo;
  const int64_t c0 = blockIdx.y * cols_per;
  const int64_t c1 = c0 + cols_per < a.dim ? c0 + cols_per : a.dim;
  for (int64_t c = c0 + lane * kVec; c < c1; c += 4 * kWaveCols) {
    v8f v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (c + u * kWaveCols + kVec <= c1) v[u] = live ? load8(src + c + u * kWaveCols) : v8f{};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t cu = c + u * kWaveCols;
      if (cu + kVec <= c1) {
        v[u] *= a.scale;
        if (!live) v[u] = v8f{};
        store8(dst + cu, v[u]);
      } else {
        for (int64_t e = cu; e < c1; ++e) store1(dst + e, live ? load1(src + e) * a.scale : 0.0f);
      }
    }
  }
}

// --------------------------------------------------------------- token sort
// Stable least-significant-digit radix sort of (id, t) by id; ids outside
// [0, V) get the key V and end up last.  Digits have at most 9 bits, so a
// vocabulary below 2^18 takes two passes.  A wave ranks 64 keys at a time:
// one ballot per digit bit gives every lane the mask of the lanes that share
// its digit; the lowest of them adds the count to the wave's LDS counter.
constexpr int kDigitMax = 9, kBinsMax = 1 << kDigitMax;
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kSmallSort = 16 * kSortThreads;   // tokens one workgroup sorts in LDS
constexpr int kTileSteps = 4, kTileKeys = kTileSteps * kSortThreads;

__device__ __forceinline__ uint32_t key_of(const void* ids, bool wide, int64_t t, int64_t n,
                                           int64_t vocab) {
  if (t >= n) return kNoKey;
  const int64_t id = load_id(ids, wide, t);
  return id >= 0 && id < vocab ? (uint32_t)id : (uint32_t)vocab;
}

// Rank of this lane's key among the wave's earlier keys with the same digit.
// `counts` are this wave's own.
__device__ __forceinline__ uint32_t wave_rank(uint32_t digit, int bits, uint32_t* counts) {
  const int lane = threadIdx.x & 63;
  uint64_t peers = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const uint64_t m = __ballot((digit >> b) & 1u);
    peers &= ((digit >> b) & 1u) ? m : ~m;
  }
  const uint32_t before = (uint32_t)__popcll(peers & ((1ull << lane) - 1ull));
  const int first = __ffsll((unsigned long long)peers) - 1;
  uint32_t base = 0;
  if (lane == first) base = atomicAdd(&counts[digit], (uint32_t)__popcll(peers));
  return (uint32_t)__shfl((int)base, first, 64) + before;
}

// Exclusive sum over the workgroup of one value per thread; `scratch` holds
// one word per wave.  Ends with a barrier.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t* scratch, uint32_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t inc = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t o = (uint32_t)__shfl_up((int)inc, off, 64);
    if (lane >= off) inc += o;
  }
  if (lane == 63) scratch[wave] = inc;
  __syncthreads();
  uint32_t base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    const uint32_t s = scratch[w];
    base += w < wave ? s : 0u;
    all += s;
  }
  __syncthreads();
  *total = all;
  return base + inc - v;
}

// The wave counters [wave][bin] turned into exclusive sums over the waves;
// returns this thread's bin total (0 past the bins).
__device__ __forceinline__ uint32_t scan_waves(uint32_t* counts, int bins) {
  uint32_t run = 0;
  if ((int)threadIdx.x < bins)
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = counts[w * kBinsMax + threadIdx.x];
      counts[w * kBinsMax + threadIdx.x] = run;
      run += c;
    }
  return run;
}

// All passes in one workgroup, keys and token numbers in LDS between passes
// (at most 16384 tokens: 128 KiB).  One launch instead of three per pass,
// which is what a sort of this size costs.
template <int STEPS>
__global__ __launch_bounds__(kSortThreads) void k_sort_small(EmbedArgs a, int bits, int passes,
                                                             uint32_t* __restrict__ keys_out,
                                                             uint32_t* __restrict__ idx_out) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  uint32_t* counts = reinterpret_cast<uint32_t*>(smem);           // [waves][bins]
  uint32_t* bin_base = counts + kSortWaves * kBinsMax;            // [bins]
  uint32_t* scratch = bin_base + kBinsMax;                        // [waves]
  uint32_t* keys = scratch + kSortWaves;                          // [STEPS * threads]
  uint16_t* idx = reinterpret_cast<uint16_t*>(keys + STEPS * kSortThreads);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool wide = a.ids_type == NVFP4_TYPE_I64;
  const int first = wave * 64 * STEPS + lane;
  uint32_t key[STEPS], at[STEPS], rank[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    at[s] = first + 64 * s;
    key[s] = key_of(a.ids, wide, at[s], a.n, a.vocab);
  }
  const int bins = 1 << bits;
  for (int p = 0; p < passes; ++p) {
    for (int i = threadIdx.x; i < kSortWaves * kBinsMax; i += kSortThreads) counts[i] = 0;
    __syncthreads();
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
      rank[s] = wave_rank((key[s] >> (p * bits)) & (bins - 1), bits, counts + wave * kBinsMax);
    __syncthreads();
    uint32_t total;
    const uint32_t mine = scan_waves(counts, bins);
    const uint32_t base = block_exclusive(mine, scratch, &total);
    if ((int)threadIdx.x < bins) bin_base[threadIdx.x] = base;
    __syncthreads();
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const uint32_t d = (key[s] >> (p * bits)) & (bins - 1);
      const uint32_t pos = bin_base[d] + counts[wave * kBinsMax + d] + rank[s];
      keys[pos] = key[s];
      idx[pos] = (uint16_t)at[s];
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      key[s] = keys[first + 64 * s];
      at[s] = idx[first + 64 * s];
    }
    __syncthreads();
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s)
    if (first + 64 * s < a.n) {
      keys_out[first + 64 * s] = key[s];
      idx_out[first + 64 * s] = at[s];
    }
}

// One pass over tiles of 4096 keys: count, scan over [bin][tile], move.  The
// first pass reads the ids (keys_in is null).
struct SortPass {
  EmbedArgs a;
  const uint32_t* keys_in;
  const uint32_t* idx_in;
  uint32_t* keys_out;
  uint32_t* idx_out;
  uint32_t* hist;   // [bins][tiles]
  int64_t tiles;
  int shift, bits;
};

__device__ __forceinline__ uint32_t tile_key(const SortPass& p, int64_t i) {
  if (p.keys_in == nullptr)
    return key_of(p.a.ids, p.a.ids_type == NVFP4_TYPE_I64, i, p.a.n, p.a.vocab);
  return i < p.a.n ? p.keys_in[i] : kNoKey;
}

__global__ __launch_bounds__(kSortThreads) void k_sort_count(SortPass p) {
  __shared__ uint32_t bin[kBinsMax];
  const int bins = 1 << p.bits;
  for (int i = threadIdx.x; i < bins; i += kSortThreads) bin[i] = 0;
  __syncthreads();
#pragma unroll
  for (int s = 0; s < kTileSteps; ++s) {
    const int64_t i = (int64_t)blockIdx.x * kTileKeys + s * kSortThreads + threadIdx.x;
    if (i < p.a.n) atomicAdd(&bin[(tile_key(p, i) >> p.shift) & (bins - 1)], 1u);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < bins; i += kSortThreads)
    p.hist[(int64_t)i * p.tiles + blockIdx.x] = bin[i];
}

__global__ __launch_bounds__(kSortThreads) void k_sort_scan(uint32_t* hist, int64_t n) {
  __shared__ uint32_t scratch[kSortWaves];
  uint32_t carry = 0;
  for (int64_t i0 = 0; i0 < n; i0 += 4 * kSortThreads) {
    const int64_t i = i0 + 4 * threadIdx.x;
    uint32_t v[4], sum = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = i + k < n ? hist[i + k] : 0u;
      sum += v[k];
    }
    uint32_t total;
    uint32_t run = carry + block_exclusive(sum, scratch, &total);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < n) {
        hist[i + k] = run;
        run += v[k];
      }
    carry += total;
  }
}

__global__ __launch_bounds__(kSortThreads) void k_sort_move(SortPass p) {
  __shared__ uint32_t counts[kSortWaves * kBinsMax];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int bins = 1 << p.bits;
  for (int i = threadIdx.x; i < kSortWaves * kBinsMax; i += kSortThreads) counts[i] = 0;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * kTileKeys + wave * 64 * kTileSteps + lane;
  uint32_t key[kTileSteps], rank[kTileSteps];
#pragma unroll
  for (int s = 0; s < kTileSteps; ++s) {
    key[s] = tile_key(p, first + 64 * s);
    rank[s] = wave_rank((key[s] >> p.shift) & (bins - 1), p.bits, counts + wave * kBinsMax);
  }
  __syncthreads();
  scan_waves(counts, bins);
  __syncthreads();
#pragma unroll
  for (int s = 0; s < kTileSteps; ++s) {
    const int64_t i = first + 64 * s;
    if (i < p.a.n) {
      // keys past the end come after every real key of the last tile, so
      // their ranks shift nothing
      const uint32_t d = (key[s] >> p.shift) & (bins - 1);
      const uint32_t pos = p.hist[(int64_t)d * p.tiles + blockIdx.x] +
                           counts[wave * kBinsMax + d] + rank[s];
      p.keys_out[pos] = key[s];
      p.idx_out[pos] = p.idx_in == nullptr ? (uint32_t)i : p.idx_in[i];
    }
  }
}

// ----------------------------------------------------------------- gradient
// A frequent word owns a long run of the sorted tokens.  Aligned windows of
// 64 sorted tokens that lie wholly inside one run are summed first, each by
// its own wave into an FP32 partial row; the row kernel then adds at most 63
// single rows before, the partials, and at most 63 rows after.
constexpr int kWindow = 64;

// The sum of dY rows idx[0 .. count) at columns c .. c + 7 added to acc, in
// order.  idx and count are the same for the whole wave (scalar loads).
template <class Y>
__device__ __forceinline__ void add_rows(v8f& acc, const Y* __restrict__ dy, int64_t ld, int64_t c,
                                         int64_t count, const uint32_t* __restrict__ idx) {
  int64_t j = 0;
  for (; j + 4 <= count; j += 4) {
    v8f v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = load8(dy + (int64_t)idx[j + u] * ld + c);
#pragma unroll
    for (int u = 0; u < 4; ++u) acc += v[u];
  }
  for (; j < count; ++j) acc += load8(dy + (int64_t)idx[j] * ld + c);
}

// The same at one column (the fewer than 8 at the end of a row).
template <class Y>
__device__ __forceinline__ void add_rows(float& acc, const Y* __restrict__ dy, int64_t ld,
                                         int64_t c, int64_t count,
                                         const uint32_t* __restrict__ idx) {
  for (int64_t j = 0; j < count; ++j) acc += load1(dy + (int64_t)idx[j] * ld + c);
}

template <class Y>
__global__ __launch_bounds__(64) void k_embed_window(const uint32_t* __restrict__ keys,
                                                     const uint32_t* __restrict__ idx,
                                                     int64_t vocab, int64_t dim,
                                                     const Y* __restrict__ dy, int64_t ld,
                                                     float* __restrict__ partial) {
  const int64_t win = blockIdx.x, s = win * kWindow;
  const uint32_t k0 = keys[s], k1 = keys[s + kWindow - 1];
  if (k0 != k1 || k0 >= (uint32_t)vocab) return;
  float* dst = partial + win * dim;
  const int64_t c = (int64_t)blockIdx.y * kWaveCols + threadIdx.x * kVec;
  if (c + kVec <= dim) {
    v8f acc = v8f{};
    add_rows(acc, dy, ld, c, kWindow, idx + s);
    store8(dst + c, acc);
  } else {
    for (int64_t e = c; e < dim; ++e) {
      float acc = 0.0f;
      add_rows(acc, dy, ld, e, kWindow, idx + s);
      dst[e] = acc;
    }
  }
}

// First sorted position whose key is not below `key`, within [lo, lo + len]:
// the wave probes 64 places at a time.
__device__ __forceinline__ int64_t lower_bound(const uint32_t* __restrict__ keys, int64_t lo,
                                               int64_t len, uint32_t key) {
  const int lane = threadIdx.x & 63;
  while (len > 0) {
    const int64_t step = (len + 63) / 64;
    const int64_t off = lane * step;
    const bool below = off < len && keys[lo + off] < key;
    const int cnt = __popcll(__ballot(below));
    if (cnt == 0) return lo;
    const int64_t next = lo + (cnt - 1) * step + 1;
    const int64_t end = lo + len;
    lo = next;
    len = step - 1 < end - next ? step - 1 : end - next;
  }
  return lo;
}

struct RowArgs {
  const uint32_t* keys;
  const uint32_t* idx;
  int64_t n, vocab, dim, ld_dy, ld_dw;
  const float* partial;
  float scale;
  int rows_per;       // vocabulary rows per wave
  int64_t cols_per;   // columns per wave (a multiple of kWaveCols)
  bool accumulate;
};

__device__ __forceinline__ void add_partial(v8f& acc, const float* p) { acc += load8(p); }
__device__ __forceinline__ void add_partial(float& acc, const float* p) { acc += *p; }

// The whole sum of run [s, e) at columns c .. c + 7 (v8f) or column c (float).
template <class A, class Y>
__device__ __forceinline__ A run_sum(const RowArgs& r, const Y* __restrict__ dy, int64_t s,
                                     int64_t e, int64_t c) {
  A acc = A{};
  const int64_t w0 = (s + kWindow - 1) / kWindow, w1 = e / kWindow;   // whole windows
  if (w0 >= w1) {
    add_rows(acc, dy, r.ld_dy, c, e - s, r.idx + s);
    return acc;
  }
  add_rows(acc, dy, r.ld_dy, c, w0 * kWindow - s, r.idx + s);
  for (int64_t w = w0; w < w1; ++w) add_partial(acc, r.partial + w * r.dim + c);
  add_rows(acc, dy, r.ld_dy, c, e - w1 * kWindow, r.idx + w1 * kWindow);
  return acc;
}

// dW rows: a wave owns rows_per consecutive vocabulary rows (and a column
// range when the vocabulary alone does not fill the chip).  It finds its
// first sorted position by probing, then walks the runs with a 64-key window
// held one key per lane.  Rows of absent words are zeros (or stay as they
// are when accumulating).
template <class Y, class G>
__global__ __launch_bounds__(64) void k_embed_rows(RowArgs r, const Y* __restrict__ dy,
                                                   G* __restrict__ dw) {
  const int lane = threadIdx.x;
  const int64_t v0 = (int64_t)blockIdx.x * r.rows_per;
  const int64_t v1 = v0 + r.rows_per < r.vocab ? v0 + r.rows_per : r.vocab;
  const int64_t c0 = blockIdx.y * r.cols_per;
  const int64_t c1 = c0 + r.cols_per < r.dim ? c0 + r.cols_per : r.dim;
  int64_t s = uniform64(lower_bound(r.keys, 0, r.n, (uint32_t)v0));
  int64_t wb = s;
  uint32_t key = wb + lane < r.n ? r.keys[wb + lane] : kNoKey;
  for (int64_t v = v0; v < v1; ++v) {
    int64_t e;
    if ((uint32_t)__builtin_amdgcn_readlane((int)key, 63) <= (uint32_t)v) {
      // the run may go past the window
      e = uniform64(lower_bound(r.keys, s, r.n - s, (uint32_t)v + 1u));
      wb = e;
      key = wb + lane < r.n ? r.keys[wb + lane] : kNoKey;
    } else {
      e = s + __popcll(__ballot(key == (uint32_t)v));
    }
    if (e > s || !r.accumulate) {
      G* dst = dw + v * r.ld_dw;
      for (int64_t c = c0 + lane * kVec; c < c1; c += kWaveCols) {
        if (c + kVec <= c1) {
          v8f sum = v8f{};
          if (e > s) sum = run_sum<v8f>(r, dy, s, e, c) * r.scale;
          if (r.accumulate) sum += load8(dst + c);
          store8(dst + c, sum);
        } else {
          for (int64_t k = c; k < c1; ++k) {
            float sum = e > s ? run_sum<float>(r, dy, s, e, k) * r.scale : 0.0f;
            if (r.accumulate) sum += load1(dst + k);
            store1(dst + k, sum);
          }
        }
      }
    }
    s = e;
  }
}

struct SortPlan { int bits, passes; };

SortPlan sort_plan(int64_t vocab) {   // keys 0 .. vocab
  int total = 1;
  while ((vocab >> total) != 0) ++total;
  const int passes = (total + kDigitMax - 1) / kDigitMax;
  return {(total + passes - 1) / passes, passes};
}

int64_t pad256(int64_t b) { return (b + 255) / 256 * 256; }

// Workspace: sorted keys and tokens, the second pair of buffers and the
// counters of the multi-workgroup sort, the window partials.
struct EmbedWs {
  int64_t keys, idx, keys2, idx2, hist, partial, total, tiles;
};

EmbedWs embed_ws(int64_t n, int64_t vocab, int64_t dim) {
  EmbedWs w{};
  const SortPlan p = sort_plan(vocab);
  const int64_t list = pad256(n * 4);
  w.tiles = (n + kTileKeys - 1) / kTileKeys;
  w.keys = 0;
  w.idx = list;
  int64_t at = 2 * list;
  if (n > kSmallSort) {
    w.keys2 = at;
    w.idx2 = at + list;
    w.hist = at + 2 * list;
    at = w.hist + pad256(((int64_t)1 << p.bits) * w.tiles * 4);
  }
  w.partial = at;
  w.total = at + pad256(n / kWindow * dim * 4);
  return w;
}

template <int STEPS>
hipError_t sort_small(const EmbedArgs& a, const SortPlan& p, uint32_t* keys, uint32_t* idx,
                      hipStream_t s) {
  const size_t lds = (kSortWaves * kBinsMax + kBinsMax + kSortWaves) * 4 + STEPS * kSortThreads * 6;
  // above the 64 KiB default of dynamic LDS
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_sort_small<STEPS>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_sort_small<STEPS>, dim3(1), dim3(kSortThreads), lds, s, a, p.bits, p.passes,
                     keys, idx);
  return hipGetLastError();
}

hipError_t sort_tokens(const EmbedArgs& a, const EmbedWs& w, uint8_t* ws, hipStream_t s) {
  const SortPlan p = sort_plan(a.vocab);
  uint32_t* keys = reinterpret_cast<uint32_t*>(ws + w.keys);
  uint32_t* idx = reinterpret_cast<uint32_t*>(ws + w.idx);
  if (a.n <= kSmallSort) {
    if (a.n <= 1 * kSortThreads) return sort_small<1>(a, p, keys, idx, s);
    if (a.n <= 4 * kSortThreads) return sort_small<4>(a, p, keys, idx, s);
    if (a.n <= 8 * kSortThreads) return sort_small<8>(a, p, keys, idx, s);
    return sort_small<16>(a, p, keys, idx, s);
  }
  uint32_t* keys2 = reinterpret_cast<uint32_t*>(ws + w.keys2);
  uint32_t* idx2 = reinterpret_cast<uint32_t*>(ws + w.idx2);
  uint32_t* hist = reinterpret_cast<uint32_t*>(ws + w.hist);
  const uint32_t *kin = nullptr, *iin = nullptr;
  for (int q = 0; q < p.passes; ++q) {
    const bool to_first = (p.passes - 1 - q) % 2 == 0;   // the last pass ends in keys / idx
    SortPass sp{a, kin, iin, to_first ? keys : keys2, to_first ? idx : idx2, hist, w.tiles,
                q * p.bits, p.bits};
    hipLaunchKernelGGL(k_sort_count, dim3((uint32_t)w.tiles), dim3(kSortThreads), 0, s, sp);
    hipLaunchKernelGGL(k_sort_scan, dim3(1), dim3(kSortThreads), 0, s, hist,
                       ((int64_t)1 << p.bits) * w.tiles);
    hipLaunchKernelGGL(k_sort_move, dim3((uint32_t)w.tiles), dim3(kSortThreads), 0, s, sp);
    kin = sp.keys_out;
    iin = sp.idx_out;
  }
  return hipGetLastError();
}

constexpr int64_t kFillWaves = 16384;   // two rounds of 32 waves on each of 256 CUs

template <class Y, class G>
hipError_t embed_grad(const EmbedArgs& a, const Y* dy, int64_t ld_dy, G* dw, int64_t ld_dw,
                      bool accumulate, uint8_t* ws, hipStream_t s) {
  const EmbedWs w = embed_ws(a.n, a.vocab, a.dim);
  const uint32_t* keys = reinterpret_cast<const uint32_t*>(ws + w.keys);
  const uint32_t* idx = reinterpret_cast<const uint32_t*>(ws + w.idx);
  float* partial = reinterpret_cast<float*>(ws + w.partial);
  const int64_t col_chunks = (a.dim + kWaveCols - 1) / kWaveCols;
  if (a.n > 0) {
    hipError_t e = sort_tokens(a, w, ws, s);
    if (e != hipSuccess) return e;
    if (a.n >= kWindow)
      hipLaunchKernelGGL(k_embed_window<Y>, dim3((uint32_t)(a.n / kWindow), (uint32_t)col_chunks),
                         dim3(64), 0, s, keys, idx, a.vocab, a.dim, dy, ld_dy, partial);
  }
  RowArgs r{keys, idx, a.n, a.vocab, a.dim, ld_dy, ld_dw, partial, a.scale, 1, 0, accumulate};
  int64_t per = a.vocab / kFillWaves;
  r.rows_per = (int)(per < 1 ? 1 : per > 16 ? 16 : per);
  const int64_t waves = (a.vocab + r.rows_per - 1) / r.rows_per;
  int64_t cut = (kFillWaves + waves - 1) / waves;
  if (cut > col_chunks) cut = col_chunks;
  r.cols_per = (col_chunks + cut - 1) / cut * kWaveCols;
  cut = (a.dim + r.cols_per - 1) / r.cols_per;
  hipLaunchKernelGGL((k_embed_rows<Y, G>), dim3((uint32_t)waves, (uint32_t)cut), dim3(64), 0, s, r,
                     dy, dw);
  return hipGetLastError();
}

template <class W, class O>
hipError_t embed(const EmbedArgs& a, const W* w, int64_t ldw, O* out, int64_t ldo, hipStream_t s) {
  // whole rows per wave once the tokens alone give every CU 8 waves
  const bool many = a.n >= 2048;
  const int64_t chunks = (a.dim + kWaveCols - 1) / kWaveCols;
  const int64_t cols_per = many ? chunks * kWaveCols : kWaveCols;
  hipLaunchKernelGGL((k_embed<W, O>),
                     dim3((uint32_t)((a.n + kEmbedWaves - 1) / kEmbedWaves),
                          (uint32_t)(many ? 1 : chunks)),
                     dim3(64 * kEmbedWaves), 0, s, a, w, ldw, out, ldo, cols_per);
  return hipGetLastError();
}

}  // namespace

int64_t embed_grad_workspace_bytes(int64_t n, int64_t vocab, int64_t dim) {
  return embed_ws(n, vocab, dim).total;
}

hipError_t launch_embed(const EmbedArgs& a, const void* w, int w_type, int64_t ldw, void* out,
                        int out_type, int64_t ldo, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  const auto* wb = reinterpret_cast<const bf16_t*>(w);
  const auto* wf = reinterpret_cast<const float*>(w);
  auto* ob = reinterpret_cast<bf16_t*>(out);
  auto* of = reinterpret_cast<float*>(out);
  if (w_type == NVFP4_TYPE_BF16)
    return out_type == NVFP4_TYPE_BF16 ? embed(a, wb, ldw, ob, ldo, s) : embed(a, wb, ldw, of, ldo, s);
  return out_type == NVFP4_TYPE_BF16 ? embed(a, wf, ldw, ob, ldo, s) : embed(a, wf, ldw, of, ldo, s);
}

hipError_t launch_embed_grad(const EmbedArgs& a, const void* dy, int dy_type, int64_t ld_dy,
                             void* dw, int dw_type, int64_t ld_dw, bool accumulate, void* ws,
                             hipStream_t s) {
  auto* p = reinterpret_cast<uint8_t*>(ws);
  const auto* yb = reinterpret_cast<const bf16_t*>(dy);
  const auto* yf = reinterpret_cast<const float*>(dy);
  auto* gb = reinterpret_cast<bf16_t*>(dw);
  auto* gf = reinterpret_cast<float*>(dw);
  if (dy_type == NVFP4_TYPE_BF16)
    return dw_type == NVFP4_TYPE_BF16 ? embed_grad(a, yb, ld_dy, gb, ld_dw, accumulate, p, s)
                                      : embed_grad(a, yb, ld_dy, gf, ld_dw, accumulate, p, s);
  return dw_type == NVFP4_TYPE_BF16 ? embed_grad(a, yf, ld_dy, gb, ld_dw, accumulate, p, s)
                                    : embed_grad(a, yf, ld_dy, gf, ld_dw, accumulate, p, s);
}

}  // namespace nvfp4
