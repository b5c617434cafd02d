// lm_ce.hip -- softmax cross entropy of an output head z = h w^T over a large
// vocabulary, with its gradient, without logits in FP32:
//
//   lse_t  = log sum_v exp(z_tv),   loss_t = lse_t - z_t,target
//   d_tv   = g_t (exp(z_tv - lse_t) - [v = target_t])
//   dH     = d W,   dW = d^T H
//
// Three matrix products of 2 T V D operations each (one for the loss alone);
// everything else is fused around them.
//
//  k_ce_logits   z tile by tile on the matrix cores (lm_gemm.h).  Per token and
//                span of 128 words the epilogue leaves the maximum and the sum
//                of exponentials, and for the gradient a 16-bit code per entry:
//                how far log2 of its exponential lies below the span's maximum,
//                in steps of 64/65535 (an absolute step in the logarithm, so a
//                relative error of at most 3.4e-4 in the exponential, a twelfth
//                of the BF16 rounding d gets anyway; entries more than 2^-64
//                below their span's maximum become 0).  FP32 logits would be
//                twice the bytes, BF16 ones off by 2% at a logit of 10; a
//                second product to recompute them is a fourth product.
//  k_ce_rows     the spans' statistics joined into lse_t and loss_t.
//  k_ce_dlogits  codes -> d in BF16, in place.
//  k_ce_dh       dH = d W: few tiles, a long sum over the vocabulary, cut in
//                equal parts when the tiles do not fill the compute units.
//  k_ce_dw       dW = d^T H.
//
// 8192 tokens x 131072 words x 5120: logits 8.6 .. 9.2 ms, dH 8.3 .. 8.6, dW 7.9 .. 8.2
// (1.2 .. 1.39 PFLOP/s), codes to d 0.8, the rest 0.2.  The products are bound by
// power there: 71 .. 78% of the matrix cores' cycles at a clock of 1.7 GHz.  With few
// tokens or a short K it is the epilogues: 1003 x 32003 x 512 takes 52 us for the
// logits, half of it their epilogue.
//
// Tokens without a target are taken out first (k_ce_prep, k_ce_gather): they
// cost nothing in any product, and nothing they hold can reach a gradient.  The
// number of remaining tokens stays on the device; the products run a fixed grid
// of one workgroup per compute unit that walks as many tiles as there are.
// Tokens may be taken in pieces to bound the code buffer; dW is then held in
// FP32 between pieces.
#include "gemm_tiles.h"
#include "lm_gemm.h"
#include "lm_kernels.h"

namespace nvfp4 {

namespace {

using namespace lm;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kSpan = 128;                 // words per softmax partial (a wave's m range)
constexpr float kCodeSpan = 64.0f;         // log2 range of a code
constexpr float kCodeStep = kCodeSpan / 65535.0f;
constexpr int kMaxItems = 2048;            // parts x tiles of a cut dH product

struct Meta {
  uint32_t pace[2][kXcds][32];   // arrivals in dH and dW by XCD, a line of memory each
  int n;        // tokens with a target
  int split;    // parts of the dH product's sum
  float scale;  // of the row weights: the results are multiplied by it
};

struct CeArgs {
  const uint16_t* h;       // [.][ldh]: the tokens themselves, or the gathered ones
  const uint16_t* w;
  uint16_t* hc;            // h where it is the gathered ones, else null
  int64_t ldh, ldw, T, V, D;
  Meta* meta;              // null: all T tokens
  int64_t first, piece;    // this piece's first row and most rows
  const int32_t* idx;      // row -> token (null: the same)
  const void* targets;
  int targets_type;
  const int32_t* tgt;      // gathered targets
  const float* weight;     // gathered row weights g, divided by the scale
  float* tlogit;           // [rows] the target's logit
  float2* stats;           // [piece][spans] (log2 maximum, sum)
  float* lse2;             // [rows] lse / ln 2
  float* rloss;            // [rows]
  uint16_t* codes;         // [piece][ldc] codes, then d
  int64_t ldc, spans, wide;   // pitch of codes, spans, words with their padding (spans * 128)
  float* loss;             // by token
  float* lse;              // by token (nullable)
  uint16_t* dh;
  int64_t ld_dh;
  uint16_t* dw;
  int64_t ld_dw;
  float* part;             // FP32 parts of dH, in accumulator order
  float* dw_acc;           // FP32 dW between pieces, in accumulator order
  int tiles_dh_m;          // ceil(D / 256)
  bool keep, add, finish;  // codes wanted; dW adds to dw_acc; dW is written out
};

__device__ __forceinline__ int64_t piece_rows(const CeArgs& g) {
  const int64_t n = g.meta == nullptr ? g.T : (int64_t)g.meta->n;
  const int64_t r = n - g.first;
  return r < 0 ? 0 : r < g.piece ? r : g.piece;
}

__device__ __forceinline__ int64_t target_of(const void* t, int type, int64_t i) {
  return type == NVFP4_TYPE_I64 ? reinterpret_cast<const int64_t*>(t)[i]
                                : (int64_t) reinterpret_cast<const int32_t*>(t)[i];
}

// A row's target, loaded without waiting for it.
struct Target {
  uint32_t lo, hi;
  __device__ __forceinline__ void load(const CeArgs& g, int64_t row) {
    hi = 0;
    if (g.tgt != nullptr) {
      lo = (uint32_t)g.tgt[row];
    } else if (g.targets_type == NVFP4_TYPE_I64) {
      const v2u w = reinterpret_cast<const v2u*>(g.targets)[row];
      lo = w.x;
      hi = w.y;
    } else {
      lo = reinterpret_cast<const uint32_t*>(g.targets)[row];
    }
  }
  __device__ __forceinline__ bool exists(const CeArgs& g) const {
    return hi == 0 && lo < (uint32_t)g.V;
  }
  // Its place in the span of words from m0 on; outside 0 .. 127 where it has none there.
  __device__ __forceinline__ int in_span(const CeArgs& g, int64_t m0) const {
    return exists(g) ? (int)lo - (int)m0 : -1;
  }
};

// Of a product's four quarters of loads: those due before block j of N.
template <int N, class F>
__device__ __forceinline__ void for_parts(int j, F f) {
#pragma unroll
  for (int p = 0; p < 4; ++p)
    if (p * N / 4 == j) f(p);
}

// The tiles of a product, walked by a fixed grid.  Each XCD (workgroups are
// dealt to the 8 in turn) owns a contiguous range of items; inside it tiles run
// in groups of 8 tile columns m, m fastest, so that the 32 workgroups of an XCD
// share 8 stretches of A and 4 of B in its L2 (81% of its reads hit).  `parts`
// repeats all tiles, part by part.  Counts fit 32 bits: T * V and T * D are at
// most 2^40, tiles 256 x 64 or larger.
struct Walk {
  uint32_t tm_all, tn_all, total, at, end, stride;
  uint32_t tm, tn, part, item;

  __device__ __forceinline__ Walk(int64_t tiles_m, int64_t tiles_n, int64_t parts) {
    tm_all = uniform((int)tiles_m);
    tn_all = uniform((int)tiles_n);
    total = uniform((int)(tiles_m * tiles_n * parts));
    const uint32_t per = (total + kXcds - 1) / kXcds, xcd = blockIdx.x % kXcds;
    at = xcd * per + blockIdx.x / kXcds;
    end = (xcd + 1) * per < total ? (xcd + 1) * per : total;
    stride = gridDim.x / kXcds;
  }
  // The next tile; false: no more.
  __device__ __forceinline__ bool next() {
    if (at >= end) return false;
    item = at;
    at += stride;
    locate(item);
    return true;
  }
  __device__ __forceinline__ void locate(uint32_t i) {
    const uint32_t tiles = tm_all * tn_all;
    part = i / tiles;
    i -= part * tiles;
    const uint32_t group = i / (kGroupM * tn_all), first = group * kGroupM;
    const uint32_t gm = min(tm_all - first, (uint32_t)kGroupM), in = i - first * tn_all;
    tn = in / gm;
    tm = first + in % gm;
  }
};

// Keeps the workgroups of an XCD near each other in k.  They read the same
// stretches of A and B, which the L2 holds for about ten steps; nothing else ties them
// together, and over thousands of steps they drift apart: of 8192 x 131072 x 5120,
// 53% (dH) and 40% (dW) of the reads missed the L2, and the traffic takes power that
// the matrix cores need (their clock is bound by it).  Every 32 steps each of them
// counts up and, four steps later, waits for the others: 19% misses, the least the
// shapes allow, and 1 to 3% less time for the loss with its gradient (26.5 -> 25.8,
// 27.1 -> 26.7 ms on two cards).  At 1300 steps a workgroup it gains nothing.  The
// wait is a hint only: it is bounded, and a workgroup that waits in vain (mates not
// running yet) stops taking part.
// Kernels for shorter products are built without it (ON false): the test in the loop
// alone costs dW 5% where it has 16 steps a tile.
constexpr int64_t kPaceSteps = 2048;   // from so many steps a workgroup on

template <bool ON>
struct Pace {
  uint32_t* count;
  uint32_t due, mates;   // count when all have arrived; workgroups of the XCD
  uint32_t short_by;     // arrivals that this item's mates make and it does not
  bool on;

  __device__ __forceinline__ Pace(Meta* meta, int which, int64_t steps)
      : count(meta->pace[which][blockIdx.x % kXcds]), due(0), mates(gridDim.x / kXcds),
        short_by(0), on(ON && steps >= kPaceSteps) {}
  __device__ __forceinline__ void arrive(uint32_t n) {
    if ((threadIdx.x & 63) == 0)
      __hip_atomic_fetch_add(count, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  // Before an item of `steps` steps; the longest of its round has `most`.  The last
  // round of the XCD may be short of some mates.
  __device__ __forceinline__ void item(const Walk& t, int wave, int64_t steps, int64_t most) {
    if (!ON) return;
    if (t.item - blockIdx.x / kXcds + mates > t.end) on = false;
    if (!on || wave != 0) return;
    due += short_by * mates;
    short_by = (uint32_t)((most + 31) / 32 - (steps + 31) / 32);
    if (short_by != 0) arrive(short_by);
  }
  __device__ __forceinline__ void operator()(int step, int wave) {
    if (!ON || !on || wave != 0) return;
    if (step % 32 == 0) {
      due += mates;
      arrive(1);
    } else if (step % 32 == 4) {
      for (int tries = 64; on; --tries) {
        const uint32_t seen =
            __hip_atomic_load(count, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if ((int)((uint32_t)uniform((int)seen) - due) >= 0) break;
        on = tries > 0;
        __builtin_amdgcn_s_sleep(1);
      }
    }
  }
};

// A wave's 32 n x 128 m half-words staged in its own 8 KiB of LDS, row n in 256
// bytes, chunk c at c ^ (n & 15): 8-byte writes of 4 consecutive m, 16-byte
// reads of whole rows.
__device__ __forceinline__ uint32_t stage_base(int lane) {
  const int n = lane & 31;
  return (uint32_t)(n * 256 + ((n & 15) << 4) + (lane >> 5) * 8);
}
__device__ __forceinline__ void stage_put(uint8_t* region, uint32_t base, int i, int q, v2u v) {
  *reinterpret_cast<v2u*>(region + (base ^ (uint32_t)((4 * i + q) << 4))) = v;
}
// Piece p of the readback: rows 4 p + lane / 16, chunk lane % 16.
__device__ __forceinline__ v4u stage_get(const uint8_t* region, int lane, int p) {
  const int r = 4 * p + (lane >> 4);
  return *reinterpret_cast<const v4u*>(region + r * 256 + (((lane & 15) ^ (r & 15)) << 4));
}
__device__ __forceinline__ void wave_lds_done() {
  __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
  __builtin_amdgcn_wave_barrier();
}

// ------------------------------------------------------------------- logits
// What the epilogue does with block column j of a wave (32 rows, the 128 words
// from m0 on); `left` words of the span exist (128 or more: WHOLE).
template <int WN, bool KEEP, bool WHOLE>
__device__ __forceinline__ void logits_block(const CeArgs& g, const v16f (&acc)[kWM][WN], int j,
                                             int left, int at, int64_t m0, int64_t row0,
                                             int64_t rows, uint8_t* region) {
  const int lane = fresh_lane(), half = lane >> 5;
  const int64_t row = row0 + (lane & 31);
  // words past the vocabulary take no part
  const auto z = [&](int i, int v) {
    return WHOLE || acc_m(i, v, half) < left ? acc[i][j][v] : -__builtin_inff();
  };
  float mx = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < kWM; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) mx = fmaxf(mx, z(i, v));
  mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
  // the reference of the span: this binary32 value itself, so its rounding
  // costs nothing; 0 where every logit is -inf (all exponentials are 0)
  const float m2 = mx == -__builtin_inff() ? 0.0f : mx * kLog2e;
  // Eight at a time and four chains of sums: a single wave per SIMD hides no latency,
  // and left alone the compiler takes them one by one.
  float part[4] = {};
#pragma unroll
  for (int i = 0; i < kWM; ++i)
#pragma unroll
    for (int v0 = 0; v0 < 16; v0 += 8) {
      float e[8];
#pragma unroll
      for (int v = 0; v < 8; ++v) e[v] = __builtin_fmaf(z(i, v0 + v), kLog2e, -m2);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int v = 0; v < 8; ++v) e[v] = __builtin_amdgcn_exp2f(e[v]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int v = 0; v < 8; ++v) part[v & 3] += e[v];
    }
  float sum = (part[0] + part[1]) + (part[2] + part[3]);
  sum += __shfl_xor(sum, 32, 64);
  if (row < rows && half == 0) g.stats[row * g.spans + m0 / kSpan] = float2{m2, sum};
  if (__ballot(at >= 0 && at < kSpan)) {
    float own = 0.0f;
#pragma unroll
    for (int i = 0; i < kWM; ++i)
#pragma unroll
      for (int v = 0; v < 16; ++v) own = at == acc_m(i, v, half) ? acc[i][j][v] : own;
    if (row < rows && at >= 0 && at < kSpan && ((at >> 2) & 1) == half)
      g.tlogit[g.first + row] = own;
  }
  if (KEEP) {
    const float c0 = m2 / kCodeSpan;
    const uint32_t base = stage_base(lane);
#pragma unroll
    for (int i = 0; i < kWM; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = __builtin_fmaf(z(i, 4 * q + e), -kLog2e / kCodeSpan, c0);
        stage_put(region, base, i, q,
                  v2u{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pknorm_u16(x[0], x[1])),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pknorm_u16(x[2], x[3]))});
      }
    wave_lds_done();
    // rows past the end lie past num_records and are dropped
    const int left_rows = (int)(rows - row0 < 32 ? rows - row0 : 32);
    const __amdgpu_buffer_rsrc_t out =
        rsrc(g.codes + row0 * g.ldc + m0, left_rows > 0 ? ((left_rows - 1) * (int)g.ldc + kSpan) * 2 : 0);
    uint32_t off = (uint32_t)((lane >> 4) * (int)g.ldc * 2 + (lane & 15) * 16);
#pragma unroll
    for (int p = 0; p < 8; ++p, off += 4 * (uint32_t)g.ldc * 2)
      __builtin_amdgcn_raw_buffer_store_b128(stage_get(region, lane, p), out, off, 0, 0);
    wave_lds_done();
  }
}

// Every product kernel loads the next tile's first two stages under the epilogue
// of this one, which has LDS of its own (all 160 KiB are in use): a quarter of the
// loads before each block of rows, since issued together they stall the waves.
template <int WN, bool KEEP>
__global__ __launch_bounds__(kThreads, 1) void k_ce_logits(CeArgs g) {
  __shared__ __attribute__((aligned(1024))) uint8_t a0[32768], a1[32768], b0[8192 * WN], b1[8192 * WN];
  __shared__ __attribute__((aligned(1024))) uint8_t epi[32768];
  const int wave = uniform(threadIdx.x >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  uint8_t* region = epi + wave * 8192;
  const int64_t rows = piece_rows(g);
  Walk t((g.V + kTM - 1) / kTM, (rows + 64 * WN - 1) / (64 * WN), 1);
  Core<false, false, WN> core;
  const auto begin = [&]() {
    core.a.init(Operand{g.w, g.ldw, g.V}, (int64_t)t.tm * kTM, g.D, wave, wm * 128);
    core.b.init(Operand{g.h + g.first * g.ldh, g.ldh, rows}, (int64_t)t.tn * 64 * WN, g.D, wave,
                wn * 32 * WN);
  };
  const auto start = [&](int part) { core.start(a0, b0, a1, b1, wave, 0, part); };
  bool more = t.next();
  if (more) {
    begin();
    for_parts<1>(0, start);
  }
  while (more) {
    const int64_t m0 = (int64_t)t.tm * kTM + wm * 128;   // the wave's span of words
    const int64_t row0 = (int64_t)t.tn * 64 * WN + wn * 32 * WN;
    core.run(a0, b0, a1, b1, wave, 0, g.D);
    // the rows' targets, on their way during the set-up of the next tile
    Target target[WN];
#pragma unroll
    for (int j = 0; j < WN; ++j) {
      const int64_t row = row0 + 32 * j + (fresh_lane() & 31);
      target[j].load(g, g.first + (row < rows ? row : rows - 1));
    }
    more = t.next();
    if (more) begin();
#pragma unroll
    for (int j = 0; j < WN; ++j) {
      __builtin_amdgcn_sched_barrier(0);   // one block of rows at a time: registers
      if (more) for_parts<WN>(j, start);
      const int at = target[j].in_span(g, m0);
      if (m0 + kSpan <= g.V)
        logits_block<WN, KEEP, true>(g, core.acc, j, kSpan, at, m0, row0 + 32 * j, rows, region);
      else if (m0 < g.V)
        logits_block<WN, KEEP, false>(g, core.acc, j, (int)(g.V - m0), at, m0, row0 + 32 * j, rows,
                                      region);
    }
  }
}

// ----------------------------------------------------------------- row sums
// One wave per row: the spans' (maximum, sum) joined; loss in binary64 from
// there, so that lse - z loses nothing to the size of lse.  The sums are FP32: relative to
// a sum near 1 they are off by some 2^-24, and so is a small loss in absolute terms.  It is
// held at 0 or more (lse >= z; NaN stays).
__global__ __launch_bounds__(256) void k_ce_rows(CeArgs g) {
  const int lane = threadIdx.x & 63;
  const int64_t r = block_xz() * 4 + uniform(threadIdx.x >> 6);
  if (r >= piece_rows(g)) return;
  const float2* st = g.stats + r * g.spans;
  // four spans a lane on their way at once (1 x 131072: 10.3 -> 7.2 us,
  // 8192 x 131072: 36 -> 27)
  const auto four = [&](int64_t s, auto take) {
    float2 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = s + 64 * u < g.spans ? st[s + 64 * u] : float2{0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (v[u].y != 0.0f) take(v[u]);
  };
  float mx = -__builtin_inff();
  for (int64_t s = lane; s < g.spans; s += 256) four(s, [&](float2 v) { mx = fmaxf(mx, v.x); });
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off, 64));
  float sum = 0.0f;
  for (int64_t s = lane; s < g.spans; s += 256)
    four(s, [&](float2 v) { sum += v.y * __builtin_amdgcn_exp2f(v.x - mx); });
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
  if (lane != 0) return;
  const int64_t row = g.first + r;
  const double lse = (double)mx * (1.0 / (double)kLog2e) + log((double)sum);
  Target target;
  target.load(g, row);
  float loss = target.exists(g) ? (float)(lse - (double)g.tlogit[row]) : 0.0f;
  loss = loss < 0.0f ? 0.0f : loss;
  const int64_t t = g.idx == nullptr ? row : g.idx[row];
  g.loss[t] = loss;
  if (g.lse != nullptr) g.lse[t] = (float)lse;
  if (g.keep) {
    g.lse2[row] = (float)(lse * (double)kLog2e);
    g.rloss[row] = loss;
  }
}

// codes -> d = g (p - [target]), BF16, in place; bound by HBM (8192 x 131072: 0.78 ms,
// 5.5 TB/s).  Each thread four pieces of 8 entries of a row (1000 x 65536: 45 us,
// with one piece 62).  At the target p - 1 = exp(-loss) - 1, which loses nothing to a p
// close to 1 beyond the loss's own error: some 2^-24, more than the BF16 rounding of d once
// 1 - p is below about 1e-5.  A weight of 0 masks a row: zeros whatever it holds, and its
// gathered h is cleared too, since 0 times an infinity or NaN there would reach all of dW.
// Weights are relative to their largest (all 1 for a mean), which multiplies the FP32 results
// instead: a mean's 1/n, rounded to BF16 in every d alike, would be a common
// error of up to 2^-8.
constexpr int kDlogitsVecs = 1024;   // pieces of a workgroup and row

__global__ __launch_bounds__(256) void k_ce_dlogits(CeArgs g) {
  const int64_t vecs = g.wide / 8, rows = piece_rows(g);
  const int64_t v0 = (int64_t)blockIdx.x * kDlogitsVecs + threadIdx.x;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < 2 * kXcds * 32; i += 256) g.meta->pace[0][0][i] = 0;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    uint16_t* row = g.codes + r * g.ldc;
    const float weight = g.weight[g.first + r], lse2 = g.lse2[g.first + r];
    if (weight == 0.0f && blockIdx.x == 0)
      for (int64_t c = threadIdx.x * 8; c < g.D; c += 2048)
        *reinterpret_cast<v4u*>(g.hc + (g.first + r) * g.ldh + c) = v4u{};
    v4u code[kDlogitsVecs / 256];
    float top[kDlogitsVecs / 256];
#pragma unroll
    for (int u = 0; u < kDlogitsVecs / 256; ++u) {
      const int64_t v = v0 + 256 * u < vecs ? v0 + 256 * u : vecs - 1;
      code[u] = *reinterpret_cast<const v4u*>(row + v * 8);
      const int64_t span = v * 8 / kSpan;
      top[u] = span < g.spans ? g.stats[r * g.spans + span].x : 0.0f;
    }
    const int64_t target = (int64_t)g.tgt[g.first + r];
    const float own = expm1f(-g.rloss[g.first + r]) * weight;
#pragma unroll
    for (int u = 0; u < kDlogitsVecs / 256; ++u) {
      const int64_t v = v0 + 256 * u;
      if (v >= vecs) continue;
      const float base = top[u] - lse2;
      v8f d;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t c = i & 1 ? code[u][i >> 1] >> 16 : code[u][i >> 1] & 0xFFFFu;
        const float e = __builtin_amdgcn_exp2f(__builtin_fmaf((float)c, -kCodeStep, base));
        d[i] = c == 0xFFFFu && base == base ? 0.0f : e * weight;
      }
      const int64_t at = target - v * 8;
      if (at >= 0 && at < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = i == at ? own : d[i];
      }
      *reinterpret_cast<v4u*>(row + v * 8) = weight == 0.0f ? v4u{} : pack8(d);
    }
  }
}

// ---------------------------------------------------------------- gradients
// Block column j of a wave's BF16 results, rows n0 .. n0 + 31 and columns m0 ..
// m0 + 127, through the wave's LDS region: put(lane, p, value) takes 16 bytes of row
// n0 + 4 p + lane / 16 at column m0 + 8 (lane % 16).
template <int WN, class Put>
__device__ __forceinline__ void store_block(const v16f (&acc)[kWM][WN], int j, uint8_t* region,
                                            float scale, Put put) {
  typedef float f4 __attribute__((ext_vector_type(4)));
  typedef __bf16 b4 __attribute__((ext_vector_type(4)));
  const int lane = fresh_lane();
  const uint32_t base = stage_base(lane);
#pragma unroll
  for (int i = 0; i < kWM; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const f4 v = f4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                      acc[i][j][4 * q + 3]} * scale;
      stage_put(region, base, i, q, __builtin_bit_cast(v2u, __builtin_convertvector(v, b4)));
    }
  wave_lds_done();
#pragma unroll
  for (int p = 0; p < 8; ++p) put(lane, p, stage_get(region, lane, p));
  wave_lds_done();
}

// Rows one after the other in memory: rows past n_end and columns past m_end are
// dropped by the descriptor and by an offset past it.
template <int WN>
__device__ __forceinline__ void store_rows(const v16f (&acc)[kWM][WN], int j, uint8_t* region,
                                           float scale, uint16_t* out, int64_t ld, int64_t m0,
                                           int64_t m_end, int64_t n0, int64_t n_end) {
  const int rows = (int)(n_end - n0 < 32 ? n_end - n0 : 32), cols = (int)(m_end - m0);
  const __amdgpu_buffer_rsrc_t buf =
      rsrc(out + n0 * ld + m0, rows > 0 && cols > 0 ? ((rows - 1) * (int)ld + cols) * 2 : 0);
  store_block<WN>(acc, j, region, scale, [&](int lane, int p, v4u val) {
    const int c = (lane & 15) * 8;
    const uint32_t off = (uint32_t)(((lane >> 4) + 4 * p) * (int)ld * 2 + c * 2);
    __builtin_amdgcn_raw_buffer_store_b128(val, buf, off | (c < cols ? 0u : kDead), 0, 0);
  });
}

// Rows in the places idx gives.
template <int WN>
__device__ __forceinline__ void store_rows_at(const v16f (&acc)[kWM][WN], int j, uint8_t* region,
                                              float scale, uint16_t* out, int64_t ld, int64_t m0,
                                              int64_t m_end, int64_t n0, int64_t n_end,
                                              const int32_t* idx) {
  store_block<WN>(acc, j, region, scale, [&](int lane, int p, v4u val) {
    const int64_t n = n0 + 4 * p + (lane >> 4), m = m0 + 8 * (lane & 15);
    if (n < n_end && m < m_end) *reinterpret_cast<v4u*>(out + (int64_t)idx[n] * ld + m) = val;
  });
}

// A wave's accumulators in accumulator order: 16-byte pieces, 1 KiB per
// instruction.
template <int WN>
__device__ __forceinline__ void put_acc(const v16f (&acc)[kWM][WN], int j, float* p) {
  v4f* at = reinterpret_cast<v4f*>(p) + fresh_lane();
#pragma unroll
  for (int i = 0; i < kWM; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      at[((i * WN + j) * 4 + q) * 64] = v4f{acc[i][j][4 * q], acc[i][j][4 * q + 1],
                                            acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
}
template <int WN>
__device__ __forceinline__ void add_acc(v16f (&acc)[kWM][WN], int j, const float* p) {
  const v4f* at = reinterpret_cast<const v4f*>(p) + fresh_lane();
#pragma unroll
  for (int i = 0; i < kWM; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const v4f v = at[((i * WN + j) * 4 + q) * 64];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][4 * q + e] += v[e];
    }
}
constexpr int64_t wave_floats(int wn) { return (int64_t)kWM * wn * 16 * 64; }

// dH tile: m over D (W transposed), n over the piece's rows, k over the words.
template <int WN, bool PACED>
__global__ __launch_bounds__(kThreads, 1) void k_ce_dh(CeArgs g) {
  __shared__ __attribute__((aligned(1024))) uint8_t a0[32768], a1[32768], b0[8192 * WN], b1[8192 * WN];
  __shared__ __attribute__((aligned(1024))) uint8_t epi[32768];
  const int wave = uniform(threadIdx.x >> 6), wm = wave & 1, wn = wave >> 1;
  const int64_t rows = piece_rows(g);
  const int split = uniform(g.meta->split);
  const float scale = g.meta->scale;
  const int64_t steps = g.wide / kBK, per = (steps + split - 1) / split;
  Walk t(g.tiles_dh_m, (rows + 64 * WN - 1) / (64 * WN), split);
  Core<true, false, WN> core;
  Pace<PACED> pace(g.meta, 0, (int64_t)t.total * per / gridDim.x);
  int64_t s0 = 0, k_end = 0;
  const auto begin = [&]() {
    s0 = t.part * per;
    k_end = (s0 + per < steps ? s0 + per : steps) * kBK;
    // W's rows end at V: words past it are zeros in d and read zero in W
    core.a.init(Operand{g.w, g.ldw, g.D}, (int64_t)t.tm * kTM, k_end < g.V ? k_end : g.V, wave,
                wm * 128);
    core.b.init(Operand{g.codes, g.ldc, rows}, (int64_t)t.tn * 64 * WN, k_end, wave, wn * 32 * WN);
  };
  const auto start = [&](int part) { core.start(a0, b0, a1, b1, wave, s0, part); };
  bool more = t.next();
  if (more) {
    begin();
    for_parts<1>(0, start);
  }
  while (more) {
    const int64_t m0 = (int64_t)t.tm * kTM + wm * 128;
    const int64_t n0 = (int64_t)t.tn * 64 * WN + wn * 32 * WN;
    float* part = g.part + ((int64_t)t.item * 4 + wave) * wave_floats(WN);
    pace.item(t, wave, k_end / kBK - s0, per);
    core.run(a0, b0, a1, b1, wave, s0, k_end, [&](int step) { pace(step, wave); });
    more = t.next();
    if (more) begin();
#pragma unroll
    for (int j = 0; j < WN; ++j) {
      __builtin_amdgcn_sched_barrier(0);
      if (more) for_parts<WN>(j, start);
      if (split > 1)
        put_acc<WN>(core.acc, j, part);
      else
        store_rows_at<WN>(core.acc, j, epi + wave * 8192, scale, g.dh, g.ld_dh, m0, g.D,
                          n0 + 32 * j, rows, g.idx + g.first);
    }
  }
}

// The parts of a cut dH product added in order and written out: one wave per
// 32 x 32 block, so that few tiles in many parts still fill the chip.
template <int WN>
__global__ __launch_bounds__(256) void k_ce_dh_join(CeArgs g) {
  const int wave = uniform(threadIdx.x >> 6), wm = wave & 1, wn = wave >> 1;
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int64_t rows = piece_rows(g);
  const int64_t split = g.meta->split;
  if (split == 1) return;
  const float scale = g.meta->scale;
  Walk t(g.tiles_dh_m, (rows + 64 * WN - 1) / (64 * WN), 1);
  const int64_t tiles = t.total;
  for (int64_t u = blockIdx.x; u < tiles * kWM * WN; u += gridDim.x) {
    const int64_t tile = u / (kWM * WN);
    const int block = (int)(u % (kWM * WN)), i = block / WN, j = block % WN;
    const v4f* at = reinterpret_cast<const v4f*>(g.part + (tile * 4 + wave) * wave_floats(WN)) +
                    block * 4 * 64 + lane;
    const int64_t pitch = tiles * wave_floats(WN);   // in v4f: 4 waves of wave_floats / 4
    // eight parts on their way at once: with few tiles the chain of parts is what
    // takes the time (1 x 131072 x 1024: 21 -> 16 us)
    v4f sum[4] = {};
    int64_t s = 0;
    for (; s + 8 <= split; s += 8) {
      v4f v[8][4];
#pragma unroll
      for (int p = 0; p < 8; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) v[p][q] = at[(s + p) * pitch + q * 64];
#pragma unroll
      for (int p = 0; p < 8; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) sum[q] += v[p][q];
    }
#pragma unroll 4
    for (; s < split; ++s)
#pragma unroll
      for (int q = 0; q < 4; ++q) sum[q] += at[s * pitch + q * 64];
    t.locate((uint32_t)tile);
    const int64_t n = (int64_t)t.tn * 64 * WN + wn * 32 * WN + 32 * j + (lane & 31);
    if (n >= rows) continue;
    uint16_t* out = g.dh + (int64_t)g.idx[g.first + n] * g.ld_dh;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      typedef __bf16 b4 __attribute__((ext_vector_type(4)));
      const int64_t m = (int64_t)t.tm * kTM + wm * 128 + 32 * i + 8 * q + 4 * half;
      if (m < g.D)
        *reinterpret_cast<v2u*>(out + m) =
            __builtin_bit_cast(v2u, __builtin_convertvector(sum[q] * scale, b4));
    }
  }
}

// dW tile: m over D (H transposed), n over the words (d transposed), k over the
// piece's rows.  PIECES: the sum goes on over several pieces, held in FP32.
template <bool PIECES, bool PACED>
__global__ __launch_bounds__(kThreads, 1) void k_ce_dw(CeArgs g) {
  constexpr int WN = 4;
  __shared__ __attribute__((aligned(1024))) uint8_t a0[32768], a1[32768], b0[32768], b1[32768];
  __shared__ __attribute__((aligned(1024))) uint8_t epi[32768];
  const int wave = uniform(threadIdx.x >> 6), wm = wave & 1, wn = wave >> 1;
  const int64_t rows = piece_rows(g);
  if (PIECES && rows == 0 && g.add && !g.finish) return;   // an empty piece in the middle
  const float scale = g.meta->scale;
  Walk t((g.D + kTM - 1) / kTM, (g.V + 255) / 256, 1);
  Core<true, true, WN> core;
  Pace<PACED> pace(g.meta, 1, (int64_t)t.total * (rows / kBK) / gridDim.x);
  const auto begin = [&]() {
    core.a.init(Operand{g.h + g.first * g.ldh, g.ldh, g.D}, (int64_t)t.tm * kTM, rows, wave,
                wm * 128);
    core.b.init(Operand{g.codes, g.ldc, g.wide}, (int64_t)t.tn * 256, rows, wave, wn * 128);
  };
  const auto start = [&](int part) { core.start(a0, b0, a1, b1, wave, 0, part); };
  bool more = t.next();
  if (more) {
    begin();
    for_parts<1>(0, start);
  }
  while (more) {
    const int64_t m0 = (int64_t)t.tm * kTM + wm * 128, n0 = (int64_t)t.tn * 256 + wn * 128;
    float* acc_at = g.dw_acc + (((int64_t)t.tn * t.tm_all + t.tm) * 4 + wave) * wave_floats(WN);
    pace.item(t, wave, 0, 0);
    core.run(a0, b0, a1, b1, wave, 0, rows, [&](int step) { pace(step, wave); });
    more = t.next();
    if (more) begin();
#pragma unroll
    for (int j = 0; j < WN; ++j) {
      __builtin_amdgcn_sched_barrier(0);
      if (more) for_parts<WN>(j, start);
      if (PIECES && g.add) add_acc<WN>(core.acc, j, acc_at);
      if (!PIECES || g.finish)
        store_rows<WN>(core.acc, j, epi + wave * 8192, scale, g.dw, g.ld_dw, m0, g.D, n0 + 32 * j,
                       g.V);
      else
        put_acc<WN>(core.acc, j, acc_at);
    }
  }
}

// -------------------------------------------------------------- preparation
// dW of at most 32 tokens: K is at most one pair of MFMA steps, so nothing is staged
// and the kernel is bound by writing dW.  A wave keeps its 128 columns of h in
// registers and goes over the words 64 at a time: a lane reads two neighbouring
// words of d at once, and the even and the odd ones are a block of rows each.  1 x 65536
// x 5120: 110 us (6.1 TB/s), 32 tokens 139 (4.8).  In tiles of 256 x 256, where most of
// the time is their epilogue, all compute units in step, 33 tokens take 205.
constexpr int kFewTokens = 32;

__global__ __launch_bounds__(256) void k_ce_dw_few(CeArgs g) {
  __shared__ __attribute__((aligned(1024))) uint8_t epi[32768];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), half = lane >> 5;
  const int n = uniform((int)piece_rows(g));
  const float scale = g.meta->scale;
  const int64_t m0 = (int64_t)blockIdx.x * 128;
  v8u16 a[2][kWM];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks)
#pragma unroll
    for (int i = 0; i < kWM; ++i) {
      const int64_t m = m0 + 32 * i + (lane & 31);
      const int t = 16 * ks + 8 * half;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        a[ks][i][e] = m < g.D && t + e < n ? g.h[(t + e) * g.ldh + m] : (uint16_t)0;
    }
  for (int64_t v0 = ((int64_t)blockIdx.y * 4 + wave) * 64; v0 < g.V; v0 += (int64_t)gridDim.y * 256) {
    const int64_t v = v0 + 2 * (lane & 31);   // the row of codes goes on past an odd V
    v8u16 d[2][2];   // [even, odd words][step]
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int t = 16 * ks + 8 * half + e;
        const uint32_t two =
            v < g.V && t < n ? *reinterpret_cast<const uint32_t*>(g.codes + t * g.ldc + v) : 0u;
        d[0][ks][e] = (uint16_t)two;
        d[1][ks][e] = (uint16_t)(two >> 16);
      }
#pragma unroll
    for (int odd = 0; odd < 2; ++odd) {
      v16f acc[kWM][1];
#pragma unroll
      for (int i = 0; i < kWM; ++i)
        acc[i][0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a[0][i]),
                                                            __builtin_bit_cast(v8bf, d[odd][0]),
                                                            v16f{}, 0, 0, 0);
      if (n > 16) {
#pragma unroll
        for (int i = 0; i < kWM; ++i)
          acc[i][0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a[1][i]),
                                                              __builtin_bit_cast(v8bf, d[odd][1]),
                                                              acc[i][0], 0, 0, 0);
      }
      store_rows<1>(acc, 0, epi + wave * 8192, scale, g.dw + (v0 + odd) * g.ld_dw, 2 * g.ld_dw, m0,
                    g.D, 0, (g.V - v0 - odd + 1) / 2);
    }
  }
}

struct PrepArgs {
  const void* targets;
  int targets_type;
  int64_t T, V, D, piece;
  const float* row_weight;   // by token, null: 1 / number of targets
  Meta* meta;
  int32_t* idx;
  int32_t* tgt;
  float* loss;
  float* lse;
  int cus, rows_per_tile;    // of the dH product
  int64_t tiles_m, steps, max_items;
};

constexpr int kPrepThreads = 1024;

// One workgroup: number the tokens that have a target, in order; the others'
// loss is 0.  Then the dH product's cut: the number of equal parts that lets
// the compute units finish earliest, counting a fixed cost per part.
__global__ __launch_bounds__(kPrepThreads) void k_ce_prep(PrepArgs p) {
  __shared__ uint32_t wave_count[kPrepThreads / 64];
  __shared__ uint64_t wave_least[kPrepThreads / 64];
  __shared__ uint32_t wave_most[kPrepThreads / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t n = 0;
  uint32_t most = 0;   // bits of the largest |weight|
  for (int64_t t0 = 0; t0 < p.T; t0 += 8 * kPrepThreads) {
    // this thread's 8 consecutive tokens
    const int64_t t = t0 + 8 * threadIdx.x;
    int64_t target[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      target[i] = t + i < p.T ? target_of(p.targets, p.targets_type, t + i) : -1;
    uint32_t weight[8];   // bits of |weight|, on their way with the targets
#pragma unroll
    for (int i = 0; i < 8; ++i)
      weight[i] = p.row_weight != nullptr && t + i < p.T
                      ? __float_as_uint(p.row_weight[t + i]) & 0x7FFFFFFFu : 0u;
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) mine += target[i] >= 0 && target[i] < p.V;
    uint32_t upto = mine;   // with the wave's lanes before
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const uint32_t o = (uint32_t)__shfl_up((int)upto, off, 64);
      if (lane >= off) upto += o;
    }
    if (lane == 63) wave_count[wave] = upto;
    __syncthreads();
    int64_t at = n + upto - mine;
#pragma unroll
    for (int w = 0; w < kPrepThreads / 64; ++w) {
      at += w < wave ? wave_count[w] : 0u;
      n += wave_count[w];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (target[i] >= 0 && target[i] < p.V) {
        p.idx[at] = (int32_t)(t + i);
        p.tgt[at] = (int32_t)target[i];
        most = max(most, weight[i]);
        ++at;
      } else if (t + i < p.T) {
        p.loss[t + i] = 0.0f;
        if (p.lse != nullptr) p.lse[t + i] = 0.0f;
      }
    }
  }
  const int64_t rows = n < p.piece ? n : p.piece;
  const uint32_t tiles = (uint32_t)p.tiles_m * (uint32_t)((rows + p.rows_per_tile - 1) / p.rows_per_tile);
  const uint32_t s = threadIdx.x + 1, steps = (uint32_t)p.steps, cus = (uint32_t)p.cus;
  uint64_t least = ~0ull;   // (cost, parts)
  if (s == 1 || ((uint64_t)s * tiles <= (uint64_t)p.max_items && s * 8 <= steps)) {
    const uint32_t rounds = (s * tiles + cus - 1) / cus;
    least = ((uint64_t)rounds * ((steps + s - 1) / s + 8)) << 16 | s;
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    least = min(least, (uint64_t)__shfl_xor((unsigned long long)least, off, 64));
    most = max(most, (uint32_t)__shfl_xor((int)most, off, 64));
  }
  if (lane == 0) {
    wave_least[wave] = least;
    wave_most[wave] = most;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kPrepThreads / 64; ++w) {
    least = min(least, wave_least[w]);
    most = max(most, wave_most[w]);
  }
  // weights that are all 0, or not all finite, stay as they are
  float scale = __uint_as_float(most);
  if (p.row_weight == nullptr) scale = 1.0f / (float)(n > 0 ? n : 1);
  else if (most == 0 || most >= 0x7F800000u) scale = 1.0f;
  if (threadIdx.x == 0) {
    p.meta->n = (int)n;
    p.meta->split = (int)(least & 0xFFFFu);
    p.meta->scale = scale;
  }
}

// hc[r] = h[idx[r]] and the row's weight; the gradient of a token without a target
// is zero.
__global__ __launch_bounds__(256) void k_ce_gather(const uint16_t* __restrict__ h, int64_t ldh,
                                                   uint16_t* __restrict__ hc, int64_t ldhc,
                                                   int64_t T, int64_t V, int64_t D, const Meta* meta,
                                                   const int32_t* __restrict__ idx,
                                                   const float* __restrict__ row_weight,
                                                   float* __restrict__ weight,
                                                   const void* targets, int targets_type,
                                                   uint16_t* __restrict__ dh, int64_t ld_dh) {
  const int lane = threadIdx.x & 63;
  const int64_t r = block_xz() * 4 + uniform(threadIdx.x >> 6);
  if (r >= T) return;
  if (r < meta->n) {
    const int32_t t = idx[r];
    const uint16_t* src = h + (int64_t)t * ldh;
    if (lane == 0) weight[r] = row_weight == nullptr ? 1.0f : row_weight[t] / meta->scale;
    for (int64_t c = lane * 8; c < D; c += 512)
      *reinterpret_cast<v4u*>(hc + r * ldhc + c) = *reinterpret_cast<const v4u*>(src + c);
  }
  const int64_t target = target_of(targets, targets_type, r);
  if (target < 0 || target >= V)
    for (int64_t c = lane * 8; c < D; c += 512) *reinterpret_cast<v4u*>(dh + r * ld_dh + c) = v4u{};
}

// ---------------------------------------------------------------- the plan
int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Row pitch of an operand laid out here: an odd number of 256-byte pieces, so that
// a column of 128-byte lines (what a K-contiguous stage reads of 256 rows) spreads
// over all channels of an L2, and rows start on a piece (what the transposed
// stages read is two whole pieces of each row).  At most 2^22 elements: 256 rows then
// span less than 2^31 bytes, what a descriptor and its offsets past the end hold.
int64_t odd_pitch(int64_t cols) {
  const int64_t pieces = (cols + 127) / 128;
  return (pieces + (pieces % 2 == 0 && pieces < (1 << 22) / 128)) * 128;
}

// Width of the tiles of tokens, 64, 128 or 256 (WN 1, 2, 4): a narrower tile wastes
// less of a last one and of a last round of workgroups, but reads the words' side
// as often.  A round of the logits kernel takes 0.39 : 0.57 : 1 of the wide tile's
// (D = 2048; 0.36 : 0.58 : 1 at 512, 0.41 : 0.58 : 1 at 5120); the fewest rounds so
// weighed win.  333 tokens x 50257 words x 2048: 121, 99 and 108 us
// (narrow tiles are bound by their L2 reads, 12 .. 13 TB/s).
int tokens_wn(int64_t rows, int64_t tiles_m, int cus) {
  int best = 4;
  int64_t least = INT64_MAX;
  for (const int wn : {4, 2, 1}) {
    const int64_t tiles = tiles_m * ((rows + 64 * wn - 1) / (64 * wn));
    const int64_t cost = (tiles + cus - 1) / cus * (wn == 4 ? 100 : wn == 2 ? 57 : 39);
    if (cost < least) {
      least = cost;
      best = wn;
    }
  }
  return best;
}

struct CePlan {
  int64_t piece, pieces, spans, ldc, ldhc, max_items;
  int wn;
  // workspace offsets
  int64_t meta, idx, tgt, weight, tlogit, lse2, rloss, hc, stats, codes, part, dw_acc, total;
};

constexpr int64_t kCodeBytes = int64_t(4) << 30;   // default bound of the code buffer

CePlan ce_plan(int64_t T, int64_t V, int64_t D, bool grad, int64_t piece) {
  CePlan p{};
  p.spans = (V + kSpan - 1) / kSpan;
  p.ldc = odd_pitch(V);
  p.ldhc = odd_pitch(D);
  p.piece = T;
  if (grad) {
    if (piece <= 0) {
      const int64_t fit = kCodeBytes / (2 * p.ldc) / 256 * 256;
      piece = fit < 256 ? 256 : fit;
    }
    if (piece < T) p.piece = piece;
  }
  p.pieces = p.piece > 0 ? (T + p.piece - 1) / p.piece : 1;
  p.wn = tokens_wn(p.piece, (V + kTM - 1) / kTM, num_cus());
  int64_t at = 0;
  const auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += up(bytes, 256);
    return o;
  };
  p.meta = take(sizeof(Meta));
  p.tlogit = take(T * 4);
  p.stats = take(p.piece * p.spans * 8);
  if (grad) {
    p.idx = take(T * 4);
    p.tgt = take(T * 4);
    p.weight = take(T * 4);
    p.lse2 = take(T * 4);
    p.rloss = take(T * 4);
    p.hc = take(T * p.ldhc * 2);
    p.codes = take(p.piece * p.ldc * 2);
    const int64_t tiles = (D + kTM - 1) / kTM * ((p.piece + 64 * p.wn - 1) / (64 * p.wn));
    // 0: no token, or more tiles than that: never cut
    p.max_items = tiles == 0 ? 0 : kMaxItems / tiles * tiles;
    const int64_t most = p.spans * kSpan / kBK / 8 * tiles;
    if (p.max_items > most) p.max_items = most;
    p.part = take(p.max_items * 4 * wave_floats(p.wn) * 4);
    if (p.pieces > 1)
      p.dw_acc = take((D + kTM - 1) / kTM * ((V + 255) / 256) * 4 * wave_floats(4) * 4);
  }
  p.total = at;
  return p;
}

template <int WN>
void products(const CeArgs& a, int cus, hipStream_t s) {
  const dim3 grid(cus), block(kThreads);
  if (a.keep)
    hipLaunchKernelGGL((k_ce_logits<WN, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((k_ce_logits<WN, false>), grid, block, 0, s, a);
  hipLaunchKernelGGL(k_ce_rows, grid_xz((a.piece + 3) / 4), dim3(256), 0, s, a);
  if (!a.keep) return;
  const int64_t vecs = a.wide / 8;
  hipLaunchKernelGGL(k_ce_dlogits,
                     dim3((uint32_t)((vecs + kDlogitsVecs - 1) / kDlogitsVecs),
                          (uint32_t)(a.piece < 16384 ? a.piece : 16384)),
                     dim3(256), 0, s, a);
  // wide tiles are what long products have
  const int64_t steps = a.tiles_dh_m * ((a.piece + 255) / 256) * (a.wide / kBK);
  if (WN == 4 && steps / cus >= kPaceSteps)
    hipLaunchKernelGGL((k_ce_dh<WN, WN == 4>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((k_ce_dh<WN, false>), grid, block, 0, s, a);
  hipLaunchKernelGGL(k_ce_dh_join<WN>, dim3(8 * cus), dim3(256), 0, s, a);
}

void products(const CeArgs& a, int wn, int cus, hipStream_t s) {
  if (wn == 1) products<1>(a, cus, s);
  else if (wn == 2) products<2>(a, cus, s);
  else products<4>(a, cus, s);
}

void word_grad_few(const CeArgs& a, int cus, hipStream_t s) {
  const int64_t x = (a.D + 127) / 128, most = (a.V + 255) / 256, fill = (8 * cus + x - 1) / x;
  hipLaunchKernelGGL(k_ce_dw_few, dim3((uint32_t)x, (uint32_t)(most < fill ? most : fill)),
                     dim3(256), 0, s, a);
}

template <bool PIECES>
void word_grad(const CeArgs& a, int cus, hipStream_t s) {
  const int64_t steps = a.tiles_dh_m * ((a.V + 255) / 256) * ((a.piece + kBK - 1) / kBK);
  if (steps / cus >= kPaceSteps)
    hipLaunchKernelGGL((k_ce_dw<PIECES, true>), dim3(cus), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((k_ce_dw<PIECES, false>), dim3(cus), dim3(kThreads), 0, s, a);
}

void word_grad(const CeArgs& a, bool pieces, int cus, hipStream_t s) {
  if (pieces) word_grad<true>(a, cus, s);
  else if (a.T <= kFewTokens) word_grad_few(a, cus, s);
  else word_grad<false>(a, cus, s);
}

}  // namespace

int64_t ce_workspace_bytes(int64_t T, int64_t V, int64_t D, bool grad, int64_t piece) {
  return ce_plan(T, V, D, grad, piece).total;
}

hipError_t launch_ce(const CeCall& c, hipStream_t s) {
  const CePlan p = ce_plan(c.T, c.V, c.D, c.grad, c.piece);
  uint8_t* ws = reinterpret_cast<uint8_t*>(c.ws);
  const int cus = num_cus() / kXcds * kXcds;
  CeArgs a{};
  a.h = reinterpret_cast<const uint16_t*>(c.h);
  a.w = reinterpret_cast<const uint16_t*>(c.w);
  a.ldh = c.ldh;
  a.ldw = c.ldw;
  a.T = c.T;
  a.V = c.V;
  a.D = c.D;
  a.piece = p.piece;
  a.targets = c.targets;
  a.targets_type = c.targets_type;
  a.tlogit = reinterpret_cast<float*>(ws + p.tlogit);
  a.stats = reinterpret_cast<float2*>(ws + p.stats);
  a.ldc = p.ldc;
  a.wide = p.spans * kSpan;
  a.spans = p.spans;
  a.loss = c.loss;
  a.lse = c.lse;
  if (!c.grad) {
    if (c.T > 0) products(a, p.wn, cus, s);
    return hipGetLastError();
  }
  Meta* meta = reinterpret_cast<Meta*>(ws + p.meta);
  a.meta = meta;
  a.idx = reinterpret_cast<int32_t*>(ws + p.idx);
  a.tgt = reinterpret_cast<int32_t*>(ws + p.tgt);
  a.weight = reinterpret_cast<float*>(ws + p.weight);
  a.lse2 = reinterpret_cast<float*>(ws + p.lse2);
  a.rloss = reinterpret_cast<float*>(ws + p.rloss);
  a.codes = reinterpret_cast<uint16_t*>(ws + p.codes);
  a.dh = reinterpret_cast<uint16_t*>(c.dh);
  a.ld_dh = c.ld_dh;
  a.dw = reinterpret_cast<uint16_t*>(c.dw);
  a.ld_dw = c.ld_dw;
  a.part = reinterpret_cast<float*>(ws + p.part);
  a.dw_acc = reinterpret_cast<float*>(ws + p.dw_acc);
  a.tiles_dh_m = (int)((c.D + kTM - 1) / kTM);
  a.keep = true;
  uint16_t* hc = reinterpret_cast<uint16_t*>(ws + p.hc);
  PrepArgs pa{c.targets, c.targets_type, c.T, c.V, c.D, p.piece, c.row_weight, meta,
              reinterpret_cast<int32_t*>(ws + p.idx), reinterpret_cast<int32_t*>(ws + p.tgt),
              c.loss, c.lse, cus, 64 * p.wn,
              a.tiles_dh_m, a.wide / kBK, p.max_items};
  hipLaunchKernelGGL(k_ce_prep, dim3(1), dim3(kPrepThreads), 0, s, pa);
  if (c.T > 0)
    hipLaunchKernelGGL(k_ce_gather, grid_xz((c.T + 3) / 4), dim3(256), 0, s, a.h, c.ldh, hc,
                       p.ldhc, c.T, c.V, c.D, meta, a.idx, c.row_weight,
                       reinterpret_cast<float*>(ws + p.weight), c.targets, c.targets_type, a.dh, c.ld_dh);
  a.h = a.hc = hc;
  a.ldh = p.ldhc;
  for (int64_t q = 0; q < p.pieces; ++q) {
    a.first = q * p.piece;
    a.add = q > 0;
    a.finish = q + 1 == p.pieces;
    if (c.T > 0) products(a, p.wn, cus, s);
    word_grad(a, p.pieces > 1, cus, s);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
