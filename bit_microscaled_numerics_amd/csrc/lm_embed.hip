// lm_embed.hip -- token embedding with scaling, and its gradient.
//
//   forward   y[t] = scale * W[id_t]                       (a row of zeros where
//                                                           id_t is outside [0, V))
//   gradient  dW[v] = scale * sum over {t : id_t = v} dY[t]
//
// Both are bound by HBM: the forward moves T * D elements in and out, the
// gradient reads T * D and writes all V * D.  The gradient is deterministic:
// a stable sort of the tokens by id puts the rows of one word side by side in
// ascending t, and every dW row is the FP32 sum, in that order, of pieces of up to
// 16 rows, each summed in that order (no atomics).
// The sort needs one or a few workgroups and the zeros of dW need no sort, so
// the sort's first launch writes them with all its other workgroups; the rows
// of the words that occur are then written over them, at most T rows.
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
// columns when there are too few tokens to fill the chip.  Bound by HBM: 8192 x 5120
// BF16 in 24 us (7 TB/s with the words that the cache holds), one token in 3 us.
constexpr int kEmbedWaves = 4, kVec = 8, kWaveCols = 64 * kVec;

template <class W, class O>
__global__ __launch_bounds__(64 * kEmbedWaves) void k_embed(EmbedArgs a, const W* __restrict__ w,
                                                            int64_t ldw, O* __restrict__ out,
                                                            int64_t ldo, int64_t cols_per) {
  const int lane = threadIdx.x & 63;
  const int64_t t = block_xz() * kEmbedWaves + uniform(threadIdx.x >> 6);
  if (t >= a.n) return;
  const int64_t id = uniform64(load_id(a.ids, a.ids_type == NVFP4_TYPE_I64, t));
  const bool live = id >= 0 && id < a.vocab;
  const W* src = w + (live ? id : 0) * ldw;
  O* dst = out + t * ldo;
  const int64_t c0 = blockIdx.y * cols_per;
  const int64_t c1 = c0 + cols_per < a.dim ? c0 + cols_per : a.dim;
  if (a.dim < kVec) {
    if (lane < a.dim && c0 == 0) store1(dst + lane, live ? load1(src + lane) * a.scale : 0.0f);
    return;
  }
  for (int64_t c = c0 + lane * kVec; c < c1; c += 4 * kWaveCols) {
    v8f v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t cu = c + u * kWaveCols;
      v[u] = v8f{};
      if (live && cu < c1) v[u] = load8(src + Cols(cu, a.dim).at) * a.scale;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t cu = c + u * kWaveCols;
      if (cu < c1) store8_from(dst, Cols(cu, a.dim), v[u]);
    }
  }
}

// --------------------------------------------------------------- token sort
// Stable least-significant-digit radix sort of (id, t) by id; ids outside
// [0, V) get the key V and end up last.  Digits have at most 9 bits, so a
// vocabulary below 2^18 takes two passes.  A wave ranks 64 keys at a time:
// one ballot per digit bit gives every lane the mask of the lanes that share
// its digit; the lowest of them adds the count to the wave's LDS counter.  What
// bounds it is the ballots, five instructions per bit and 64 keys, in few workgroups.
constexpr int kDigitMax = 9, kBinsMax = 1 << kDigitMax;
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kTileSteps = 4, kTileKeys = kTileSteps * kSortThreads;

__device__ __forceinline__ uint32_t key_of(const void* ids, bool wide, int64_t t, int64_t n,
                                           int64_t vocab) {
  if (t >= n) return kNoKey;
  const int64_t id = load_id(ids, wide, t);
  return id >= 0 && id < vocab ? (uint32_t)id : (uint32_t)vocab;
}

// rank[s]: how many of the wave's keys before this lane's s-th have its digit (bits
// shift ..).  `counts` are this wave's own.  The steps' ballots side by side: one
// after the other they are a chain of latencies.
template <int STEPS>
__device__ __forceinline__ void wave_ranks(const uint32_t (&key)[STEPS], uint32_t (&rank)[STEPS],
                                           int shift, int bits, uint32_t* counts) {
  uint32_t lo[STEPS], hi[STEPS];   // the lanes with the same digit
#pragma unroll
  for (int s = 0; s < STEPS; ++s) lo[s] = hi[s] = ~0u;
  for (int b = shift; b < shift + bits; ++b) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int mine = __builtin_amdgcn_sbfe((int)key[s], b, 1);   // the bit in every place
      const uint64_t m = __ballot(mine);
      lo[s] &= ~((uint32_t)m ^ (uint32_t)mine);
      hi[s] &= ~((uint32_t)(m >> 32) ^ (uint32_t)mine);
    }
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    uint32_t* count = &counts[(key[s] >> shift) & ((1u << bits) - 1)];
    const uint32_t before = __builtin_amdgcn_mbcnt_hi(hi[s], __builtin_amdgcn_mbcnt_lo(lo[s], 0));
    const uint32_t base = *count;
    rank[s] = base + before;
    // the lowest lane of a digit adds all of them, in the wave's order: no atomic
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (before == 0) *count = base + (uint32_t)(__popc(lo[s]) + __popc(hi[s]));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
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
  if ((int)threadIdx.x < bins) {
    uint32_t c[kSortWaves];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) c[w] = counts[w * kBinsMax + threadIdx.x];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      counts[w * kBinsMax + threadIdx.x] = run;
      run += c[w];
    }
  }
  return run;
}

// Zeros of dW, written by the workgroups of a sort launch that do not sort:
// `rows` rows of `cols` elements (a contiguous dW as one row).
struct Fill {
  uint8_t* p;
  int64_t rows, row_bytes, pitch;   // bytes; rows 0: nothing
};

// 4 KiB pieces (whole rows where dW has gaps) dealt in turn to kFillBlocks workgroups,
// 256 threads of each: what is in flight is one narrow window of dW.  1.3 GB take 204 us (6.6 TB/s) so; 1024
// threads 230 us, 255 workgroups 235 .. 280 us, 64 KiB pieces 218 us and more.
constexpr int kFillBlocks = 128, kFillThreads = 256;

__device__ __forceinline__ void fill_zero(const Fill& f, int64_t block) {
  constexpr int64_t kPiece = 16 * kFillThreads;
  if (threadIdx.x >= kFillThreads) return;
  if (f.rows == 1) {
    const int64_t whole = f.row_bytes / 16 * 16;
#pragma unroll 4
    for (int64_t o = block * kPiece + 16 * threadIdx.x; o < whole; o += kFillBlocks * kPiece)
      *reinterpret_cast<v4u_any2*>(f.p + o) = v4u_any2{};
    if (block == 0)
      for (int64_t e = whole + 2 * threadIdx.x; e < f.row_bytes; e += 2 * kFillThreads)
        *reinterpret_cast<uint16_t*>(f.p + e) = 0;
    return;
  }
  for (int64_t r = block; r < f.rows; r += kFillBlocks) {
    uint8_t* p = f.p + r * f.pitch;
    for (int64_t o = 16 * threadIdx.x; o < f.row_bytes; o += kPiece) {
      if (o + 16 <= f.row_bytes) {
        *reinterpret_cast<v4u_any2*>(p + o) = v4u_any2{};
      } else {
        for (int64_t e = o; e < f.row_bytes; e += 2) *reinterpret_cast<uint16_t*>(p + e) = 0;
      }
    }
  }
}

__global__ __launch_bounds__(kFillThreads) void k_fill(Fill fill) {
  fill_zero(fill, blockIdx.x);
}

// All passes over a tile of tokens in one workgroup, keys and token numbers in LDS
// between passes.  Up to 4096 tokens (8192 beside a long fill) are one tile and sorted by
// this launch alone.
template <int STEPS>
__global__ __launch_bounds__(kSortThreads) void k_sort_tile(EmbedArgs a, int bits, int passes,
                                                            int tiles,
                                                            uint32_t* __restrict__ keys_out,
                                                            uint32_t* __restrict__ idx_out,
                                                            Fill fill) {
  if ((int)blockIdx.x >= tiles) {
    fill_zero(fill, blockIdx.x - tiles);
    return;
  }
  const int64_t base = (int64_t)blockIdx.x * STEPS * kSortThreads;
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
    key[s] = key_of(a.ids, wide, base + at[s], a.n, a.vocab);
  }
  const int bins = 1 << bits;
  for (int p = 0; p < passes; ++p) {
    for (int i = threadIdx.x; i < kSortWaves * kBinsMax; i += kSortThreads) counts[i] = 0;
    __syncthreads();
    wave_ranks(key, rank, p * bits, bits, counts + wave * kBinsMax);
    __syncthreads();
    uint32_t total;
    const uint32_t mine = scan_waves(counts, bins);
    const uint32_t start = block_exclusive(mine, scratch, &total);
    if ((int)threadIdx.x < bins) bin_base[threadIdx.x] = start;
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
    if (base + first + 64 * s < a.n) {
      keys_out[base + first + 64 * s] = key[s];
      idx_out[base + first + 64 * s] = (uint32_t)base + at[s];
    }
}

// Up to 16 sorted tiles merged: a key's place is its place in its tile, the keys not
// above it in the tiles before, and the keys below it in the tiles after.  Every
// workgroup holds all keys in LDS (up to 128 KiB) and counts by halving for 128 of
// them, 8 lanes a key: with one lane a key the random reads of LDS take twice as long
// as all else.  30001 tokens: 16 us with the tiles' sort (2 more with tiles of 4096); the six
// launches of the pass-by-pass sort below, 31 us.
constexpr int kMergeTiles = 16, kMergeMax = 32768, kMergeLanes = 8;
constexpr int kMergeKeys = kSortThreads / kMergeLanes;   // of a workgroup

__global__ __launch_bounds__(kSortThreads) void k_sort_merge(const uint32_t* __restrict__ keys_in,
                                                             const uint32_t* __restrict__ idx_in,
                                                             int n, int tile_keys,
                                                             uint32_t* __restrict__ keys_out,
                                                             uint32_t* __restrict__ idx_out) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem);
  // 16 bytes at a time, all loads out at once (the list is padded to 256 bytes)
  constexpr int kLoads = kMergeMax / 4 / kSortThreads;
  v4u v[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u)
    if (4 * (u * kSortThreads + (int)threadIdx.x) < n)
      v[u] = reinterpret_cast<const v4u*>(keys_in)[u * kSortThreads + threadIdx.x];
#pragma unroll
  for (int u = 0; u < kLoads; ++u)
    if (4 * (u * kSortThreads + (int)threadIdx.x) < n)
      reinterpret_cast<v4u*>(keys)[u * kSortThreads + threadIdx.x] = v[u];
  // neighbouring lanes share a key, each counts in two of the tiles
  constexpr int kEach = kMergeTiles / kMergeLanes;
  const int i = blockIdx.x * kMergeKeys + threadIdx.x / kMergeLanes;
  const int t0 = threadIdx.x % kMergeLanes * kEach;
  const uint32_t at = i < n ? idx_in[i] : 0;
  __syncthreads();
  if (i >= n) return;
  const uint32_t key = keys[i];
  const int tile = i / tile_keys;
  int below[kEach], len[kEach];
  uint32_t limit[kEach];
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int t = t0 + u;
    below[u] = 0;
    len[u] = t == tile ? 0 : min(max(n - t * tile_keys, 0), tile_keys);
    limit[u] = key + (t < tile ? 1u : 0u);
  }
  for (int step = tile_keys; step > 0; step >>= 1)
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int to = below[u] + step;
      if (to <= len[u] && keys[(t0 + u) * tile_keys + to - 1] < limit[u]) below[u] = to;
    }
  int pos = below[0] + below[1];
#pragma unroll
  for (int off = 1; off < kMergeLanes; off <<= 1) pos += __shfl_xor(pos, off, 64);
  pos += i - tile * tile_keys;
  if (threadIdx.x % kMergeLanes == 0) {
    keys_out[pos] = key;
    idx_out[pos] = at;
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
  Fill fill;        // count kernel: workgroups past the tiles
};

__device__ __forceinline__ uint32_t tile_key(const SortPass& p, int64_t i) {
  if (p.keys_in == nullptr)
    return key_of(p.a.ids, p.a.ids_type == NVFP4_TYPE_I64, i, p.a.n, p.a.vocab);
  return i < p.a.n ? p.keys_in[i] : kNoKey;
}

__global__ __launch_bounds__(kSortThreads) void k_sort_count(SortPass p) {
  __shared__ uint32_t bin[kBinsMax];
  if (blockIdx.x >= p.tiles) {
    fill_zero(p.fill, blockIdx.x - p.tiles);
    return;
  }
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
  for (int s = 0; s < kTileSteps; ++s) key[s] = tile_key(p, first + 64 * s);
  wave_ranks(key, rank, p.shift, p.bits, counts + wave * kBinsMax);
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
// The sorted tokens are cut into windows of 64, a workgroup each and 16 rows a wave,
// which has all its rows on the way at once (a chain of single rows is bound by
// their latency); every row of dY is read once.  A run of one word inside the rows
// of a wave goes straight to dW; the piece of a run that came in (`head`) or goes on
// (`tail`) goes to LDS, and the wave where the run starts joins the pieces in order.
// A run that crosses windows leaves one FP32 partial row per window, joined in order
// by a second kernel.  Windows of 128 are as fast with many tokens and 1 us slower
// with few.  8192 x 5120 BF16 with words as in text: 43 + 5 us, much of it while the
// zeros drain; 30001 x 771, few words: 15 + 6 us.
constexpr int kWaveRows = 16, kSumWaves = 4, kWindow = kWaveRows * kSumWaves;

// Eight values (for v8f) or one (float) as they lie in memory, and their value.
__device__ __forceinline__ v4u load_as(const v8f&, const bf16_t* p) {
  return *reinterpret_cast<const v4u_any2*>(p);
}
__device__ __forceinline__ v8f load_as(const v8f&, const float* p) { return load8(p); }
__device__ __forceinline__ float load_as(const float&, const bf16_t* p) { return load1(p); }
__device__ __forceinline__ float load_as(const float&, const float* p) { return load1(p); }
__device__ __forceinline__ v8f value(v4u v) { return unpack8(v); }
__device__ __forceinline__ v8f value(v8f v) { return v; }
__device__ __forceinline__ float value(float v) { return v; }

struct RowArgs {
  const uint32_t* keys;
  const uint32_t* idx;
  int64_t n, vocab, dim, ld_dy, ld_dw;
  float* partial;
  float scale;
};

// Columns c .. c + 7 of a row (v8f), or column c.  At the end of a row a thread's
// eight overlap those of the thread before, and both hold the same bits there; only
// a sum that is added to what the row holds has to be written once.
template <bool ONCE, class G>
__device__ __forceinline__ void write_row(G* row, const Cols& k, v8f v) {
  if (ONCE) store8_from(row, k, v);
  else store8(row + k.at, v);
}
template <bool ONCE, class G>
__device__ __forceinline__ void write_row(G* row, int c, float v) { store1(row + c, v); }
__device__ __forceinline__ int64_t col(const Cols& k) { return k.at; }
__device__ __forceinline__ int64_t col(int c) { return c; }

template <bool ADD, class A, class G, class K>
__device__ __forceinline__ void finish_row(const RowArgs& r, G* __restrict__ dw, uint32_t word, K k,
                                           A sum) {
  G* row = dw + (int64_t)word * r.ld_dw;
  sum *= r.scale;
  if (ADD) sum += value(load_as(A{}, row + col(k)));
  write_row<ADD>(row, k, sum);
}

// What a wave leaves in LDS for the run that came in or goes on: values by lane.
template <class A>
struct Pieces {
  A head[kSumWaves][64], tail[kSumWaves][64];
  bool through[kSumWaves];   // head holds all rows of the wave and its run goes on
};

// The rows of a window at this lane's columns; `on`: the lane has columns.  ADD: the
// sums are added to dW, whose rows are then on the way with dY's.
template <bool ADD, class A, class Y, class G, class K>
__device__ __forceinline__ void sum_window(const RowArgs& r, const Y* __restrict__ dy,
                                           G* __restrict__ dw, Pieces<A>& lds, K k, bool on) {
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int64_t win = block_xz(), p0 = win * kWindow + wave * kWaveRows;
  const int count = uniform((int)(r.n - p0 < 0 ? 0 : r.n - p0 < kWaveRows ? r.n - p0 : kWaveRows));
  // lane l: the key of position p0 + l - 1 (no key outside the list), and its row
  const int64_t at = p0 + lane - 1;
  const bool real = lane <= kWaveRows + 1 && at >= 0 && at < r.n;
  const uint32_t key = real ? r.keys[at] : kNoKey;
  const uint32_t row = real ? r.idx[at] : 0;
  // bit j: the words of rows j - 1 and j differ, so a run starts at row j
  const uint64_t starts = __ballot(key != (uint32_t)__shfl_down((int)key, 1, 64));
  const auto word = [&](int j) {
    return (uint32_t)__builtin_amdgcn_readlane((int)key, j + 1);
  };
  // row j ends a run that starts in these rows, of a word of the vocabulary
  const auto whole = [&](int j) {
    return j < count && (starts >> (j + 1) & 1) && (starts & ((2ull << j) - 1)) != 0 &&
           word(j) < (uint32_t)r.vocab;
  };
  constexpr int kBatch = ADD ? kWaveRows / 2 : kWaveRows;   // rows in registers at once
  A acc = A{};
#pragma unroll 1
  for (int j0 = 0; j0 < count; j0 += kBatch) {
    if (!on) break;
    decltype(load_as(A{}, dy)) v[kBatch];
    decltype(load_as(A{}, dw)) old[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {   // past the end the last row again, not used
      const int j = j0 + u < count ? j0 + u : count - 1;
      const uint32_t from = (uint32_t)__builtin_amdgcn_readlane((int)row, j + 1);
      v[u] = load_as(A{}, dy + (int64_t)from * r.ld_dy + col(k));
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (ADD && whole(j0 + u))
        old[u] = load_as(A{}, dw + (int64_t)word(j0 + u) * r.ld_dw + col(k));
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int j = j0 + u;
      if (j < count) {
        acc += value(v[u]);
        if (starts >> (j + 1) & 1) {
          if ((starts & ((2ull << j) - 1)) == 0) {
            lds.head[wave][lane] = acc;
          } else if (whole(j)) {
            acc *= r.scale;
            if (ADD) acc += value(old[u]);
            write_row<ADD>(dw + (int64_t)word(j) * r.ld_dw, k, acc);
          }
          acc = A{};
        }
      }
    }
  }
  // the last run goes on past these rows
  const bool onward = count > 0 && !(starts >> count & 1);
  const bool fresh = (starts & ((1ull << count) - 1)) != 0;   // and starts in them
  if (onward) (fresh ? lds.tail : lds.head)[wave][lane] = acc;
  if (lane == 0) lds.through[wave] = onward && !fresh;
  __syncthreads();
  if (!on || count == 0) return;
  // the pieces of the run that waves w .. go on with, until it ends
  const auto join = [&](A& sum, int w, bool going) {
    for (; going && w < kSumWaves; ++w) {
      sum += lds.head[w][lane];
      going = uniform((int)lds.through[w]) != 0;
    }
    return going;
  };
  if (wave == 0 && !(starts & 1) && word(0) < (uint32_t)r.vocab) {
    A sum = A{};
    join(sum, 0, true);
    write_row<false>(r.partial + 2 * win * r.dim, k, sum);
  }
  if (onward && fresh && word(count - 1) < (uint32_t)r.vocab) {
    A sum = lds.tail[wave][lane];
    if (join(sum, wave + 1, true)) write_row<false>(r.partial + (2 * win + 1) * r.dim, k, sum);
    else finish_row<ADD>(r, dw, word(count - 1), k, sum);
  }
}

template <bool ADD, class Y, class G>
__global__ __launch_bounds__(64 * kSumWaves) void k_embed_sum(RowArgs r, const Y* __restrict__ dy,
                                                              G* __restrict__ dw) {
  const int lane = threadIdx.x & 63;
  if (r.dim < kVec) {
    __shared__ Pieces<float> lds;
    sum_window<ADD>(r, dy, dw, lds, lane, lane < r.dim);
  } else {
    __shared__ Pieces<v8f> lds;
    const int64_t c = (int64_t)blockIdx.y * kWaveCols + lane * kVec;
    sum_window<ADD>(r, dy, dw, lds, Cols(c < r.dim ? c : 0, r.dim), c < r.dim);
  }
}

// acc += at(j) + .. + at(j + N - 1), in this order, with all N loads out first.
template <int N, class A, class At>
__device__ __forceinline__ void add_batch(A& acc, int64_t j, At at) {
  decltype(at(j)) v[N];   // as loaded: eight BF16 values wait in four registers
#pragma unroll
  for (int u = 0; u < N; ++u) v[u] = at(j + u);
#pragma unroll
  for (int u = 0; u < N; ++u) acc += value(v[u]);
}

// acc += at(0) + .. + at(count - 1), in this order; count is the same for the
// whole wave.
template <class A, class At>
__device__ __forceinline__ void add_all(A& acc, int64_t count, At at) {
  int64_t j = 0;
  for (; j + 16 <= count; j += 16) add_batch<16>(acc, j, at);
  if (count & 8) { add_batch<8>(acc, j, at); j += 8; }
  if (count & 4) { add_batch<4>(acc, j, at); j += 4; }
  if (count & 2) { add_batch<2>(acc, j, at); j += 2; }
  if (count & 1) add_batch<1>(acc, j, at);
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

// The dW rows of the runs that cross windows, by the window each starts in: piece 1
// of that window, then piece 0 of those after it.
template <bool ADD, class G>
__global__ __launch_bounds__(64) void k_embed_join(RowArgs r, G* __restrict__ dw) {
  const int64_t win = block_xz(), s = win * kWindow, e = s + kWindow;
  if (e >= r.n) return;
  const uint32_t word = r.keys[e];
  if (word >= (uint32_t)r.vocab || r.keys[e - 1] != word) return;
  if (s > 0 && r.keys[s - 1] == word) return;   // it starts in a window before
  const int64_t end = uniform64(lower_bound(r.keys, e, r.n - e, word + 1u));
  const int64_t after = (end - 1) / kWindow - win;
  const float* first = r.partial + (2 * win + 1) * r.dim;
  const float* next = r.partial + 2 * (win + 1) * r.dim;
  if (r.dim < kVec) {
    const int c = threadIdx.x;
    if (c >= r.dim) return;
    float sum = first[c];
    add_all(sum, after, [&](int64_t w) { return next[2 * w * r.dim + c]; });
    finish_row<ADD>(r, dw, word, c, sum);
    return;
  }
  const int64_t c = (int64_t)blockIdx.y * kWaveCols + threadIdx.x * kVec;
  if (c >= r.dim) return;
  const Cols k(c, r.dim);
  v8f sum = load8(first + k.at);
  add_all(sum, after, [&](int64_t w) { return load8(next + 2 * w * r.dim + k.at); });
  finish_row<ADD>(r, dw, word, k, sum);
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
  if (n > kTileKeys) {
    w.keys2 = at;
    w.idx2 = at + list;
    w.hist = at + 2 * list;
    at = w.hist + (n > kMergeMax ? pad256(((int64_t)1 << p.bits) * w.tiles * 4) : 0);
  }
  w.partial = at;
  w.total = at + (n > kWindow ? pad256((n + kWindow - 1) / kWindow * 2 * dim * 4) : 0);
  return w;
}

template <int STEPS>
hipError_t sort_tile(const EmbedArgs& a, const SortPlan& p, uint32_t* keys, uint32_t* idx,
                     const Fill& fill, hipStream_t s) {
  const size_t lds = (kSortWaves * kBinsMax + kBinsMax + kSortWaves) * 4 + STEPS * kSortThreads * 6;
  if (lds > 64 * 1024) {   // above the default of dynamic LDS
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_sort_tile<STEPS>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  const int tiles = (int)((a.n + STEPS * kSortThreads - 1) / (STEPS * kSortThreads));
  const int blocks = tiles + (fill.rows > 0 ? kFillBlocks : 0);
  hipLaunchKernelGGL(k_sort_tile<STEPS>, dim3(blocks), dim3(kSortThreads), lds, s, a, p.bits,
                     p.passes, tiles, keys, idx, fill);
  return hipGetLastError();
}

template <int STEPS>
hipError_t sort_merge(const EmbedArgs& a, const SortPlan& p, uint32_t* keys, uint32_t* idx,
                      uint32_t* keys2, uint32_t* idx2, const Fill& fill, hipStream_t s) {
  hipError_t e = sort_tile<STEPS>(a, p, keys2, idx2, fill, s);
  if (e != hipSuccess) return e;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_sort_merge),
                          hipFuncAttributeMaxDynamicSharedMemorySize, kMergeMax * 4);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_sort_merge, dim3((uint32_t)((a.n + kMergeKeys - 1) / kMergeKeys)),
                     dim3(kSortThreads), (size_t)pad256(a.n * 4), s, keys2, idx2, (int)a.n,
                     STEPS * kSortThreads, keys, idx);
  return hipGetLastError();
}

// The fewer keys a workgroup sorts the sooner it is done (5, 9 and 16 .. 19 us for
// 1024, 4096 and 8192), and a merge takes 4 us more; a sort that is done before the
// zeros are written needs no second launch.
constexpr int64_t kLongFill = int64_t(96) << 20;   // bytes, 15 us

hipError_t sort_tokens(const EmbedArgs& a, const EmbedWs& w, uint8_t* ws, const Fill& fill,
                       hipStream_t s) {
  const SortPlan p = sort_plan(a.vocab);
  uint32_t* keys = reinterpret_cast<uint32_t*>(ws + w.keys);
  uint32_t* idx = reinterpret_cast<uint32_t*>(ws + w.idx);
  if (a.n <= 1 * kSortThreads) return sort_tile<1>(a, p, keys, idx, fill, s);
  if (a.n <= 2 * kSortThreads) return sort_tile<2>(a, p, keys, idx, fill, s);
  if (a.n <= kTileKeys) return sort_tile<kTileSteps>(a, p, keys, idx, fill, s);
  if (a.n <= 8 * kSortThreads && fill.rows * fill.row_bytes >= kLongFill)
    return sort_tile<8>(a, p, keys, idx, fill, s);
  uint32_t* keys2 = reinterpret_cast<uint32_t*>(ws + w.keys2);
  uint32_t* idx2 = reinterpret_cast<uint32_t*>(ws + w.idx2);
  if (a.n <= kMergeTiles * 1 * kSortThreads)
    return sort_merge<1>(a, p, keys, idx, keys2, idx2, fill, s);
  if (a.n <= kMergeMax)
    return sort_merge<2>(a, p, keys, idx, keys2, idx2, fill, s);
  uint32_t* hist = reinterpret_cast<uint32_t*>(ws + w.hist);
  const uint32_t *kin = nullptr, *iin = nullptr;
  for (int q = 0; q < p.passes; ++q) {
    const bool to_first = (p.passes - 1 - q) % 2 == 0;   // the last pass ends in keys / idx
    SortPass sp{a, kin, iin, to_first ? keys : keys2, to_first ? idx : idx2, hist, w.tiles,
                q * p.bits, p.bits, fill};
    const int64_t blocks = w.tiles + (q == 0 && fill.rows > 0 ? kFillBlocks : 0);
    hipLaunchKernelGGL(k_sort_count, dim3((uint32_t)blocks), dim3(kSortThreads), 0, s, sp);
    hipLaunchKernelGGL(k_sort_scan, dim3(1), dim3(kSortThreads), 0, s, hist,
                       ((int64_t)1 << p.bits) * w.tiles);
    hipLaunchKernelGGL(k_sort_move, dim3((uint32_t)w.tiles), dim3(kSortThreads), 0, s, sp);
    kin = sp.keys_out;
    iin = sp.idx_out;
  }
  return hipGetLastError();
}

template <bool ADD, class Y, class G>
void sum_rows(const RowArgs& r, const Y* dy, G* dw, hipStream_t s) {
  const dim3 grid = grid_xz((r.n + kWindow - 1) / kWindow, (r.dim + kWaveCols - 1) / kWaveCols);
  hipLaunchKernelGGL((k_embed_sum<ADD, Y, G>), grid, dim3(64 * kSumWaves), 0, s, r, dy, dw);
  if (r.n > kWindow) hipLaunchKernelGGL((k_embed_join<ADD, G>), grid, dim3(64), 0, s, r, dw);
}

template <class Y, class G>
hipError_t embed_grad(const EmbedArgs& a, const Y* dy, int64_t ld_dy, G* dw, int64_t ld_dw,
                      bool accumulate, uint8_t* ws, hipStream_t s) {
  const EmbedWs w = embed_ws(a.n, a.vocab, a.dim);
  const uint32_t* keys = reinterpret_cast<const uint32_t*>(ws + w.keys);
  const uint32_t* idx = reinterpret_cast<const uint32_t*>(ws + w.idx);
  float* partial = reinterpret_cast<float*>(ws + w.partial);
  Fill fill{};
  if (!accumulate) {
    const bool flat = ld_dw == a.dim;
    fill = Fill{reinterpret_cast<uint8_t*>(dw), flat ? 1 : a.vocab,
                (flat ? a.vocab * a.dim : a.dim) * (int64_t)sizeof(G), ld_dw * (int64_t)sizeof(G)};
  }
  if (a.n == 0) {
    if (!accumulate)
      hipLaunchKernelGGL(k_fill, dim3(kFillBlocks), dim3(kFillThreads), 0, s, fill);
    return hipGetLastError();
  }
  const hipError_t e = sort_tokens(a, w, ws, fill, s);
  if (e != hipSuccess) return e;
  const RowArgs r{keys, idx, a.n, a.vocab, a.dim, ld_dy, ld_dw, partial, a.scale};
  if (accumulate) sum_rows<true>(r, dy, dw, s);
  else sum_rows<false>(r, dy, dw, s);
  return hipGetLastError();
}

template <class W, class O>
hipError_t embed(const EmbedArgs& a, const W* w, int64_t ldw, O* out, int64_t ldo, hipStream_t s) {
  // whole rows per wave once the tokens alone give every CU 8 waves
  const bool many = a.n >= 2048;
  const int64_t chunks = (a.dim + kWaveCols - 1) / kWaveCols;
  const int64_t cols_per = many ? chunks * kWaveCols : kWaveCols;
  hipLaunchKernelGGL((k_embed<W, O>),
                     grid_xz((a.n + kEmbedWaves - 1) / kEmbedWaves, many ? 1 : chunks),
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
