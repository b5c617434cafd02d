// lm_attn.hip -- softmax attention and its gradient (internal to libnvfp4.so): which
// workgroup takes what, and the kernels.  lm_attn.h has the tiles and the arithmetic of rows.
//
// The forward pass is one pass over the keys with a running maximum and sum.  The gradient
// forms the probabilities again from lse, twice: once with the sums of dk and dv in registers, once with
// those of dq (7 products where 5 would do with dq added up by atomics in memory: those
// would change their order from run to run, and 64 key tiles adding to 21 MB of dq for each
// key head pass the L2).  In long products a wave's exponentials run with no product of its own beside
// them: at 8192 tokens, 40 heads of 128 over 8 key heads, causal, the matrix cores are busy for 53% of the forward
// kernel and 59% of the gradient, the vector units for 47% and 35%, and waves wait to issue for 40% of
// their time.  Power costs about a quarter besides: the clock is at 1.7 - 1.9 GHz, with zeros as data at 2.2.
// 640 - 730 us forward (0.94 - 1.07 PFLOP/s), 2050 - 2350 the gradient (1.0 - 1.2 PFLOP/s with what is
// formed again).  Heads of 64 have half the products to an exponential (36% and 58% busy forward, 43% and 40% in
// the gradient); small calls are bound by launches and the chain of a tile's steps.
#include <hip/hip_runtime.h>

#include "lm_attn.h"
#include "lm_kernels.h"

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
  a.neg_lse = static_cast<float*>(c.ws);   // the gradient's; launch_attn_grad places the other
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
  a.pairs = (int)((n.cu_q == nullptr ? n.batch : 1) * n.Hkv);
  a.D = (int)n.D;
  a.window = n.window < kWindowMost ? n.window : kWindowMost;   // its sums stay in int64
  a.scale = n.scale;
  a.scale2 = n.scale * 1.4426950408889634f;
  return a;
}

namespace {
constexpr int kAhead = 4;   // reads of LDS ahead of the products (2 and 6 measured the same, 0 a quarter slower)
constexpr int kRowsWG = 128, kKeys = 64;   // query rows of a workgroup, keys of a tile
constexpr int kGradRows = 256;   // query rows of a workgroup of the gradient
constexpr int kPartTiles = 512, kPartKeys = 128;   // see parts_of

struct Part {   // of a row's softmax, where several workgroups share its keys
  float* o;     // [part][row][D], not normalized
  float* ml;    // [part][row][2]: maximum (log2), sum
  int n;
};

// Forward.  4 waves of 32 query rows each (KH = 2: twice 4, which take every other tile of
// keys and are added up in LDS at the end); the keys pass in tiles of 64 through two LDS
// stages filled by loads that write LDS directly.  Scores are formed transposed (S^T = K
// Q^T): a lane then holds one query's scores of 32 keys, so the softmax needs one
// exchange (with the lane 32 away), and the probabilities are, as they stand, the second operand of
// O^T = V^T P^T; V is read transposed from LDS.  The sums are rescaled only when
// a maximum grows by more than 2^8: until then the probabilities are at most 2^8 and lose nothing.
template <int DP, int KH, bool SPLIT>
__global__ __launch_bounds__(256 * KH, 2) void k_attn(Args a, int pairs, int tiles, Part part) {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass drops the stubs of kernels with these builtins
  using T = Tile<DP, kKeys>;
  constexpr int kStage = 2 * T::kBytes;
  // one array per stage: loads into the next one are not waited for by reads of this one
  __shared__ __attribute__((aligned(1024))) uint8_t lds[KH * kStage], lds1[KH * kStage];
  const int wave = uniform(threadIdx.x >> 6) & 3, kh = KH > 1 ? uniform(threadIdx.x >> 8) : 0;
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const uint32_t block = (uint32_t)block_xz(), id = SPLIT ? block / (uint32_t)part.n : block;
  const int sp = SPLIT ? (int)(block - id * (uint32_t)part.n) : 0;
  if (id >= (uint32_t)pairs * (uint32_t)tiles) return;
  const Job job = job_of(id, pairs, tiles);
  const int b = job.pair / a.Hkv, hk = job.pair - b * a.Hkv;
  const int64_t rows = (int64_t)a.Tq * a.G;
  // long rows of a causal sequence first
  const int64_t r = (int64_t)(tiles - 1 - job.tile) * kRowsWG + wave * 32 + (lane & 31);
  const bool live = r < rows;
  const int t = live ? (int)((uint32_t)r / (uint32_t)a.G) : a.Tq, h = hk * a.G + (live ? (int)r - t * a.G : 0);
  const Range mine = keys_of<true>(a, t);

  const bool some = mine.lo < mine.hi;
  const Reach reach = reach_of(live, mine.lo, mine.lo, mine.hi);
  const int lo = reach.lo, hi = reach.hi, all_lo = reach.all_lo, all_hi = reach.all_hi;
  const Range all = reach_of_all<4>(lds, reach, wave);   // both halves write the same
  int j0 = all.lo, j1 = all.hi;
  if (SPLIT && j0 < j1) {
    const int per = ((j1 - j0 + kKeys - 1) / kKeys + part.n - 1) / part.n;
    const int64_t from = j0 + (int64_t)sp * per * kKeys, to = from + per * kKeys;
    j0 = (int)min(from, (int64_t)j1);
    j1 = (int)min(to, (int64_t)j1);
  }

  v8bf q[T::kSteps];
  row_frags<DP>(q, row_of(a.q, b, live ? t : 0, h), live, a.D, half);
  KeyLoader<DP, kKeys, 4> lk, lv;
  lk.init(a.k, b, hk, a.Tk, a.D, wave);
  lv.init(a.v, b, hk, a.Tk, a.D, wave);
  T frag;
  frag.init(0);

  v16f o[T::kBlocks] = {};
  float m = -INFINITY, l = 0.0f;   // m: of the products, before scale
  constexpr int kStep = KH * kKeys;   // the halves take every other tile
  uint8_t* const own[2] = {lds + kh * kStage, lds1 + kh * kStage};
  if (j0 + kh * kKeys < j1) {
    lk.load(own[0], wave, j0 + kh * kKeys);
    lv.load(own[0] + kStage / 2, wave, j0 + kh * kKeys);
  }
  auto tile = [&](int j, const uint8_t* at, uint8_t* next) __attribute__((always_inline)) {
    tile_landed();
    if (j + kStep < j1) {
      lk.load(next, wave, j + kStep);
      lv.load(next + kStage / 2, wave, j + kStep);
    }
    const int last = SPLIT ? min(hi, j1) : hi;
    if (j >= last || j + kKeys <= lo) return;
    v16f s[2] = {};
    pipeline<2 * T::kSteps, kAhead>([&](int i) { return frag.read(at, i >> 1, (i & 1) * 32); },
                               [&](int i, const v8bf& f) { s[i & 1] = mfma(f, q[i >> 1], s[i & 1]); });
    if (j < all_lo || j + kKeys > (SPLIT ? min(all_hi, j1) : all_hi)) {
      const uint32_t n = (uint32_t)max((SPLIT ? min(mine.hi, j1) : mine.hi) - mine.lo, 0);
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int v = 0; v < 16; ++v)
          if ((uint32_t)(j + kb * 32 + 4 * half - mine.lo + acc_row(v)) >= n) s[kb][v] = -INFINITY;
    }
    float top = s[0][0];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int v = 0; v < 16; ++v) top = fmaxf(top, s[kb][v]);
    top = fmaxf(m, pair_max(top));
    if (__any((top - m) * a.scale2 > 8.0f)) {
      const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - top) * a.scale2);
      l *= f;
#pragma unroll
      for (int db = 0; db < T::kBlocks; ++db) o[db] *= f;
      m = top;
    }
    const float shift = m == -INFINITY ? 0.0f : m * a.scale2;
    // the tile's sum by itself: added one by one, equal terms of 10^5 and more keys are all rounded to the
    // same side (lse of 262144 equal scores up to 1.2e-3 off; so 5e-5)
    float sum = 0.0f;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        s[kb][v] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][v], a.scale2, -shift));
        sum += s[kb][v];
      }
    l += sum;
    const uint8_t* vt = at + kStage / 2;
    v8bf p;
    pipeline<4 * T::kBlocks, kAhead>([&](int i) { return frag.read_t(vt, i % T::kBlocks, i / T::kBlocks); },
                                [&](int i, const v8bf& f) {
                                  const int db = i % T::kBlocks, ks = i / T::kBlocks;
                                  if (db == 0) p = pack_half(s[ks >> 1], ks & 1);
                                  o[db] = mfma(f, p, o[db]);
                                });
  };
  for (int j = j0; j < j1; j += 2 * kStep) {
    tile(j + kh * kKeys, own[0], own[1]);
    if (j + kStep < j1) tile(j + kStep + kh * kKeys, own[1], own[0]);
  }
  l = pair_sum(l);
  if constexpr (KH > 1) {   // the second half's sums to the first
    float* to = reinterpret_cast<float*>(lds + wave * (kStage / 2)) + lane * 4;
    float2* stat = reinterpret_cast<float2*>(lds1) + wave * 64 + lane;
    __syncthreads();
    if (kh == 1) {
#pragma unroll
      for (int db = 0; db < T::kBlocks; ++db)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<v4f*>(to + (db * 4 + i) * 256) =
              v4f{o[db][4 * i], o[db][4 * i + 1], o[db][4 * i + 2], o[db][4 * i + 3]};
      *stat = float2{m, l};
    }
    __syncthreads();
    if (kh == 1) return;
    const float2 other = *stat;
    const float top = fmaxf(m, other.x);
    const float f0 = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((m - top) * a.scale2);
    const float f1 = other.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((other.x - top) * a.scale2);
    m = top;
    l = l * f0 + other.y * f1;
#pragma unroll
    for (int db = 0; db < T::kBlocks; ++db)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const v4f y = *reinterpret_cast<const v4f*>(to + (db * 4 + i) * 256);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[db][4 * i + e] = o[db][4 * i + e] * f0 + y[e] * f1;
      }
  }

  // A value that is not finite may come from a key that a row does not see, multiplied by 0:
  // such rows are formed again, one by one, unless they are NaN throughout anyway: where l is, which
  // only keys that the row sees are part of, or the first of their values is.
  const float odd = odd_of(o);
  uint64_t again = __ballot(live && odd != 0.0f && l == l);
  const int64_t at = SPLIT ? (int64_t)sp * pairs * rows + job.pair * rows + r : 0;
  if (live) {
    if (SPLIT) {
      store_sums(part.o + at * a.D, o, a.D, half);
    } else {
      store_columns(row_of_out(a.out, b, t, h), o, some ? 1.0f / l : 0.0f, a.D, half);
    }
    if (half == 0) {
      if (SPLIT) {
        part.ml[2 * at] = m * a.scale2;
        part.ml[2 * at + 1] = l;
      } else {
        a.lse[stat_at(a, b, t, h)] = some ? (m * a.scale2 + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
      }
    }
  }
  for (again |= again >> 32, again &= 0xffffffffu; again != 0; again &= again - 1) {
    const int from = __builtin_ctzll(again);
    const int tt = __shfl(t, from), hh = __shfl(h, from);
    const int lo1 = SPLIT ? max(__shfl(mine.lo, from), j0) : __shfl(mine.lo, from);
    const int hi1 = SPLIT ? min(__shfl(mine.hi, from), j1) : __shfl(mine.hi, from);
    const int64_t at1 = at - (lane & 31) + from;
    if (lo1 < hi1 && nan_throughout(row_of(a.v, b, lo1, hk), a.D)) continue;
    const Soft x = row_forward(a, b, tt, hh, lo1, hi1);
    if (SPLIT) {
      x.o.store(part.o + at1 * a.D, a.D);
      if (lane == 0) part.ml[2 * at1] = x.m, part.ml[2 * at1 + 1] = x.l;
    } else {
      x.o.store(row_of_out(a.out, b, tt, hh), a.D, lo1 < hi1 ? 1.0f / x.l : 0.0f);
      if (lane == 0)
        a.lse[stat_at(a, b, tt, hh)] = lo1 < hi1 ? (x.m + __builtin_amdgcn_logf(x.l)) * kLn2 : -INFINITY;
    }
  }
#endif
}

// The parts of each row joined, in order.  Few parts: 32 lanes a row, four columns a lane
// (16 lanes up to 64 columns).
template <int LANES>
__global__ __launch_bounds__(256) void k_attn_join_few(Args a, uint32_t rows, Part part) {
  const int in_row = threadIdx.x & (LANES - 1);
  const uint32_t r = (uint32_t)block_xz() * (256 / LANES) + threadIdx.x / LANES;
  if (r >= rows) return;
  const uint32_t in_pair = (uint32_t)a.Tq * a.G, pair = r / in_pair, rr = r - pair * in_pair;
  const int b = pair / a.Hkv, t = rr / a.G, h = (pair - b * a.Hkv) * a.G + (rr - t * a.G);
  float m = -INFINITY;
  for (int i = 0; i < part.n; ++i) m = fmaxf(m, part.ml[2 * ((int64_t)i * rows + r)]);
  const bool live = 4 * in_row < a.D;
  float l = 0.0f;
  v4f x{};
#pragma unroll 4
  for (int i = 0; i < part.n; ++i) {
    const int64_t at = (int64_t)i * rows + r;
    const float2 ml = *reinterpret_cast<const float2*>(part.ml + 2 * at);
    const float f = ml.x == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml.x - m);
    l += ml.y * f;
    if (live) x += *reinterpret_cast<const v4f*>(part.o + at * a.D + 4 * in_row) * f;
  }
  const Range k = keys_of<false>(a, t);
  const bool some = k.lo < k.hi;
  const float f = some ? 1.0f / l : 0.0f;
  typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
  if (live)
    *reinterpret_cast<v4bf*>(row_of_out(a.out, b, t, h) + 4 * in_row) = __builtin_convertvector(x * f, v4bf);
  if (in_row == 0) a.lse[stat_at(a, b, t, h)] = some ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
}

// Many parts, a workgroup a row: each of the 4 waves takes every fourth part, two columns a
// lane; the waves' sums are added in LDS.
__global__ __launch_bounds__(256) void k_attn_join(Args a, uint32_t rows, Part part) {
  __shared__ float2 sums[4][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint32_t r = (uint32_t)block_xz();
  if (r >= rows) return;
  const uint32_t in_pair = (uint32_t)a.Tq * a.G, pair = r / in_pair, rr = r - pair * in_pair;
  const int b = pair / a.Hkv, t = rr / a.G, h = (pair - b * a.Hkv) * a.G + (rr - t * a.G);
  // the parts' maxima and sums, 64 at a time
  float m = -INFINITY;
  for (int i = lane; i < part.n; i += 64) m = fmaxf(m, part.ml[2 * ((int64_t)i * rows + r)]);
  m = wave_max(m);
  float l = 0.0f;
  for (int i = lane; i < part.n; i += 64) {
    const float* ml = part.ml + 2 * ((int64_t)i * rows + r);
    // a part whose scores are all NaN has no maximum, and a sum of NaN that counts
    l += ml[1] * (ml[0] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ml[0] - m));
  }
  l = wave_sum(l);
  float2 sum{0.0f, 0.0f};
  const bool live = 2 * lane < a.D;
#pragma unroll 8
  for (int i = wave; i < part.n; i += 4) {
    const int64_t at = (int64_t)i * rows + r;
    const float mi = part.ml[2 * at];
    const float f = mi == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mi - m);
    const float2 x = live ? *reinterpret_cast<const float2*>(part.o + at * a.D + 2 * lane) : float2{0.0f, 0.0f};
    sum.x += x.x * f;
    sum.y += x.y * f;
  }
  sums[wave][lane] = sum;
  __syncthreads();
  if (wave > 0) return;
  for (int w = 1; w < 4; ++w) sum.x += sums[w][lane].x, sum.y += sums[w][lane].y;
  const Range k = keys_of<false>(a, t);
  const bool some = k.lo < k.hi;
  const float f = some ? 1.0f / l : 0.0f;
  if (live) {
    bf16_t* o = row_of_out(a.out, b, t, h) + 2 * lane;
    store1(o, sum.x * f);
    store1(o + 1, sum.y * f);
  }
  if (lane == 0) a.lse[stat_at(a, b, t, h)] = some ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
}

// -lse / scale and -delta of every row, in the order of the rows of a key head: a wave 32 rows.
// delta = dout . out takes over out's rounding to BF16, which is small beside the rounding of
// ds where many keys share a row, and as large where few do.  Rows of at most 64 keys that
// fit a window of 64 therefore take delta = sum p dp, formed from the scores again: the error of
// dq and dk of 37 documents of 1 .. 663 tokens falls from 0.0027 to 0.0024 (their rounding alone:
// 0.0017 for ds, 0.0017 for the result).
template <int DP>
__global__ __launch_bounds__(256) void k_attn_stats(Args a, int tiles) {
#ifdef __HIP_DEVICE_COMPILE__
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, half = lane >> 5;
  // the first rows of all key heads first: those of a causal sequence see few keys
  const uint32_t id = (uint32_t)block_xz(), tile = id / (uint32_t)a.pairs, pair = id - tile * (uint32_t)a.pairs;
  const int b = pair / a.Hkv, hk = pair - b * a.Hkv;
  if (tile >= (uint32_t)tiles) return;
  const int64_t rows = (int64_t)a.Tq * a.G, r = (int64_t)tile * 128 + wave * 32 + (lane & 31);
  const bool live = r < rows;
  const int t = live ? (int)((uint32_t)r / (uint32_t)a.G) : a.Tq, h = hk * a.G + (live ? (int)r - t * a.G : 0);
  // dout . out: 8 lanes a row, 8 rows at a time, then to the lanes of the row
  const float lse = live ? a.lse[stat_at(a, b, t, h)] * kLog2e : 0.0f;
  const Range mine = keys_of<true>(a, t);
  constexpr int kParts = (DP + 63) / 64;
  v4u x[4][kParts], y[4][kParts];
#pragma unroll
  for (int i = 0; i < 4; ++i) {   // all loads first, those past the end from the last row
    const int64_t r8 = min((int64_t)tile * 128 + wave * 32 + i * 8 + (lane >> 3), rows - 1);
    const int t8 = (int)((uint32_t)r8 / (uint32_t)a.G), h8 = hk * a.G + (int)r8 - t8 * a.G;
    const bf16_t *o = row_of(a.out, b, t8, h8), *g = row_of(a.dout, b, t8, h8);
#pragma unroll
    for (int c = 0; c < kParts; ++c) {
      const int d = min(c * 64 + (lane & 7) * 8, a.D - 8);
      x[i][c] = *reinterpret_cast<const v4u*>(o + d);
      y[i][c] = *reinterpret_cast<const v4u*>(g + d);
    }
  }
  float delta = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < kParts; ++c) {
      const v8f u = unpack8(x[i][c]), w = unpack8(y[i][c]);
      float part = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) part = __builtin_fmaf(u[e], w[e], part);
      sum += c * 64 + (lane & 7) * 8 < a.D ? part : 0.0f;
    }
    sum = sum_of_8(sum);
    const float of_row = __shfl(sum, (lane & 7) * 8);
    if (((lane & 31) >> 3) == i) delta = of_row;
  }
  const int n = mine.hi - mine.lo;
  const bool few = live && n > 0 && n <= 64;
  if (__any(few)) {
    int from = few ? mine.lo : 0x7fffffff;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) from = min(from, __shfl_xor(from, m));
    // operands a few steps at a time: whole rows in registers would halve the occupancy of the rest
    constexpr int kBatch = DP == 96 ? 3 : 4;
    const bf16_t *q = row_of(a.q, b, live ? t : 0, h), *g = row_of(a.dout, b, live ? t : 0, h);
    float sum = 0.0f;
#pragma unroll 1
    for (int kb = 0; kb < 2; ++kb) {
      const int key = from + kb * 32 + (lane & 31);
      const bool there = key < a.Tk;
      const bf16_t *k = row_of(a.k, b, there ? key : 0, hk), *v = row_of(a.v, b, there ? key : 0, hk);
      v16f s{}, dp{};
#pragma unroll 1
      for (int d0 = 8 * half; d0 < DP; d0 += 16 * kBatch) {
        v8bf f[kBatch][4];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int d = d0 + 16 * i;
          f[i][0] = piece(k + d, there && d < a.D);
          f[i][1] = piece(q + d, live && d < a.D);
          f[i][2] = piece(v + d, there && d < a.D);
          f[i][3] = piece(g + d, live && d < a.D);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          s = mfma(f[i][0], f[i][1], s);
          dp = mfma(f[i][2], f[i][3], dp);
        }
      }
      const uint32_t first = (uint32_t)(from + kb * 32 + 4 * half - mine.lo);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (first + acc_row(i) < (uint32_t)n)
          sum = __builtin_fmaf(__builtin_amdgcn_exp2f(__builtin_fmaf(s[i], a.scale2, -lse)), dp[i], sum);
    }
    sum = pair_sum(sum);
    if (few && mine.hi - from <= 64 && __builtin_isfinite(sum)) delta = sum;
  }
  if (live && half == 0) {
    a.neg_lse[pair * rows + r] = -lse / a.scale2;
    a.neg_delta[pair * rows + r] = -delta;
  }
#endif
}

#ifdef __HIP_DEVICE_COMPILE__
template <int DP>
struct GradLds {   // one array per stage: loads into the next are not waited for by reads of this
  uint8_t *s0, *s1, *v, *stats;
};

// dk and dv of 128 keys: 8 waves, as 4 groups of 32 keys by 2 halves of the query rows.  A
// wave holds K and its sums of both results in registers (V in LDS), while the rows that see
// the keys pass in tiles of 64 through two LDS stages.  S = Q K^T and dP = dO V^T
// leave a lane one key and 16 rows; p and ds are, as they stand, the second operands of
// dV^T = dO^T P and dK^T = Q^T dS.  The rows pass from the last one down: the last
// rows of a causal sequence see all keys, so the workgroups of a key head start on the same
// rows and find them in their XCD's L2.
// parts > 1: each takes a piece of the rows and leaves FP32 sums, which k_attn_join_keys adds up.
template <int DP, bool PARTS>
__device__ __forceinline__ void grad_keys(const Args& a, const GradLds<DP>& lds, Job job, int part, int parts,
                                          float* sums, int64_t all_keys) {
  using T = Tile<DP, 64>;
  constexpr int kHalf = T::kBytes;   // of a stage: q, then dout
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, half = lane >> 5;
  const int kg = wave & 3, rg = wave >> 2;
  const int b = job.pair / a.Hkv, hk = job.pair - b * a.Hkv;
  const int64_t key = (int64_t)job.tile * 128 + kg * 32 + (lane & 31);
  const bool live = key < a.Tk;
  const int j = live ? (int)key : a.Tk;
  const Seers seen = queries_of(a, j);
  const int rlo = seen.lo * a.G, rmore = seen.more * a.G, rhi = seen.hi * a.G;
  const Reach reach = reach_of(live, rlo, rmore, rhi);
  Range all = reach_of_all<8>(lds.s0, reach, wave);
  if (PARTS) {
    const int per = ((all.hi - all.lo + 63) / 64 + parts - 1) / parts * 64;
    const int64_t from = all.lo + (int64_t)part * per;
    all = Range{(int)min(from, (int64_t)all.hi), (int)min(from + per, (int64_t)all.hi)};
  }

  v8bf k[T::kSteps];
  row_frags<DP>(k, row_of(a.k, b, live ? j : 0, hk), live, a.D, half);
  if (rg == 0) {
    v8bf v[T::kSteps];
    row_frags<DP>(v, row_of(a.v, b, live ? j : 0, hk), live, a.D, half);
#pragma unroll
    for (int ks = 0; ks < T::kSteps; ++ks)
      *reinterpret_cast<v8bf*>(lds.v + ((kg * T::kSteps + ks) * 64 + lane) * 16) = v[ks];
  }
  const uint8_t* mine_v = lds.v + (kg * T::kSteps * 64 + lane) * 16;
  T frag;
  frag.init(rg * 32);

  v16f dk[T::kBlocks] = {}, dv[T::kBlocks] = {};
  const int64_t all_rows = (int64_t)a.Tq * a.G;
  const float* stats = (wave == 0 ? a.neg_lse : a.neg_delta) + job.pair * all_rows;
  RowLoader<DP, 64, 4> rows;   // waves 0 .. 3 load q, the others dout
  auto load = [&](uint8_t* stage, int st, int r) __attribute__((always_inline)) {
    rows.load(stage + rg * kHalf, kg);
    if (wave < 2)   // -lse / scale, -delta of the rows
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          descriptor(reinterpret_cast<const uint16_t*>(stats + r)), (lds_void)(lds.stats + st * 512 + wave * 256), 4,
          r + lane < all_rows ? (uint32_t)lane * 4 : kDead, 0, 0, 0);
  };
  auto tile = [&](int r, uint8_t* now, uint8_t* next, int st) __attribute__((always_inline)) {
    tile_landed();
    if (r > all.lo) load(next, st ^ 1, r - 64);
    const int r0 = r + rg * 32;
    if (r0 >= min(reach.hi, all.hi) || r0 + 32 <= reach.lo) return;
    const uint8_t* td = now + kHalf;
    v16f s, dp;   // from -lse / scale and -delta on
    const uint8_t* st_at = lds.stats + st * 512 + rg * 128 + half * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const v4f x = *reinterpret_cast<const v4f*>(st_at + i * 32), y = *reinterpret_cast<const v4f*>(st_at + 256 + i * 32);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[4 * i + e] = x[e], dp[4 * i + e] = y[e];
    }
    struct Two {
      v8bf a, b;
    };
    pipeline<2 * T::kSteps, kAhead>(
        [&](int i) {
          if (i & 1) return Two{frag.read(td, i >> 1), *reinterpret_cast<const v8bf*>(mine_v + (i >> 1) * 1024)};
          return Two{frag.read(now, i >> 1), k[i >> 1]};
        },
        [&](int i, const Two& f) {
          v16f& sum = i & 1 ? dp : s;
          sum = mfma(f.a, f.b, sum);
        });
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      s[v] = __builtin_amdgcn_exp2f(s[v] * a.scale2);
      dp[v] *= s[v];
    }
    if (r0 < reach.all_lo || r0 + 32 > min(reach.all_hi, all.hi)) {
      const uint32_t first = (uint32_t)(r0 + 4 * half - rlo), n = (uint32_t)max(min(rhi, all.hi) - rlo, 0);
      if (r0 < reach.apart) {   // of a row that sees one key, dp - delta is 0, where their sums leave a rounding
        const uint32_t alone = (uint32_t)(rmore - rlo);
#pragma unroll
        for (int v = 0; v < 16; ++v)
          if (first + acc_row(v) < alone) dp[v] *= 0.0f;
      }
#pragma unroll
      for (int v = 0; v < 16; ++v)
        if (first + acc_row(v) >= n) s[v] = dp[v] = 0.0f;
    }
    v8bf p, ds;
    pipeline<4 * T::kBlocks, kAhead>(
        [&](int i) { return frag.read_t(i & 1 ? now : td, (i >> 1) % T::kBlocks, (i >> 1) / T::kBlocks); },
        [&](int i, const v8bf& f) {
          const int db = (i >> 1) % T::kBlocks, ks = (i >> 1) / T::kBlocks;
          if (db == 0 && i % 2 == 0) p = pack_half(s, ks), ds = pack_half(dp, ks);
          if (i & 1)
            dk[db] = mfma(f, ds, dk[db]);
          else
            dv[db] = mfma(f, p, dv[db]);
        });
  };
  if (all.lo < all.hi) {
    const int last = all.lo + (all.hi - 1 - all.lo) / 64 * 64;
    rows.init(rg ? a.dout : a.q, a, b, hk, last, kg);
    load(lds.s0, 0, last);
    for (int r = last; r >= all.lo; r -= 128) {
      tile(r, lds.s0, lds.s1, 0);
      if (r - 64 >= all.lo) tile(r - 64, lds.s1, lds.s0, 1);
    }
  }
  // the halves' sums
  uint8_t* other = (kg < 2 ? lds.s0 : lds.s1) + (kg & 1) * 64 * DP * 2 + lane * 16;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    v16f(&sum)[T::kBlocks] = x ? dv : dk;
    __syncthreads();
#pragma unroll
    for (int db = 0; db < T::kBlocks; ++db)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (rg == 1)
          *reinterpret_cast<v4f*>(other + (db * 4 + i) * 1024) =
              v4f{sum[db][4 * i], sum[db][4 * i + 1], sum[db][4 * i + 2], sum[db][4 * i + 3]};
    __syncthreads();
    if (rg == 1) continue;
#pragma unroll
    for (int db = 0; db < T::kBlocks; ++db)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const v4f y = *reinterpret_cast<const v4f*>(other + (db * 4 + i) * 1024);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[db][4 * i + e] += y[e];
      }
  }
  if (rg == 1) return;
  uint64_t odd_k = __ballot(live && odd_of(dk) != 0.0f), odd_v = __ballot(live && odd_of(dv) != 0.0f);
  odd_k |= odd_k >> 32, odd_v |= odd_v >> 32;
  float* to = PARTS ? sums + (((int64_t)part * all_keys + (int64_t)job.pair * a.Tk + key) * 2) * a.D : nullptr;
  if (live && !PARTS) {
    store_columns(row_of_out(a.dk, b, j, hk), dk, a.scale, a.D, half);
    store_columns(row_of_out(a.dv, b, j, hk), dv, 1.0f, a.D, half);
  } else if (live) {
    store_sums(to, dk, a.D, half);
    store_sums(to + a.D, dv, a.D, half);
  }
  for (uint64_t again = (odd_k | odd_v) & 0xffffffffu; again != 0; again &= again - 1) {
    const int from = __builtin_ctzll(again), jj = __shfl(j, from);
    const int lo = PARTS ? max(__shfl(rlo, from), all.lo) : __shfl(rlo, from);
    const int hi = PARTS ? min(__shfl(rhi, from), all.hi) : __shfl(rhi, from), more = __shfl(rmore, from);
    const bool k_odd = odd_k >> from & 1, v_odd = odd_v >> from & 1;
    const NanRows nan = nan_rows(a, b, hk, lo, hi, v_odd);
    if ((nan.dk || !k_odd) && (nan.dv || !v_odd)) continue;
    RowSum xk, xv;
    row_dkv(a, b, jj, hk, lo, more, hi, xk, xv);
    if (PARTS) {
      float* row = to + 2 * (int64_t)(from - (lane & 31)) * a.D;
      xk.store(row, a.D);
      xv.store(row + a.D, a.D);
      continue;
    }
    xk.store(row_of_out(a.dk, b, jj, hk), a.D, a.scale);
    xv.store(row_of_out(a.dv, b, jj, hk), a.D, 1.0f);
  }
}

// dq of 256 query rows, laid out as the forward kernel: S^T = K Q^T, dP^T = V dO^T, and
// dS^T as it stands is the second operand of dQ^T = K^T dS^T.  parts > 1: each takes a piece of
// the keys and leaves FP32 sums, which k_attn_join_rows adds up.
template <int DP, bool PARTS>
__device__ __forceinline__ void grad_queries(const Args& a, const GradLds<DP>& lds, Job job, int tiles, int part,
                                             int parts, float* sums) {
  using T = Tile<DP, kKeys>;
  constexpr int kHalf = T::kBytes;   // of a stage: K, then V
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, half = lane >> 5;
  const int b = job.pair / a.Hkv, hk = job.pair - b * a.Hkv;
  const int64_t rows = (int64_t)a.Tq * a.G;
  const int64_t r = (int64_t)(tiles - 1 - job.tile) * kGradRows + wave * 32 + (lane & 31);
  const bool live = r < rows;
  const int t = live ? (int)((uint32_t)r / (uint32_t)a.G) : a.Tq, h = hk * a.G + (live ? (int)r - t * a.G : 0);
  const Range mine = keys_of<true>(a, t);
  const Reach reach = reach_of(live, mine.lo, mine.lo, mine.hi);
  Range all = reach_of_all<8>(lds.s0, reach, wave);
  if (PARTS) {
    const int per = ((all.hi - all.lo + kKeys - 1) / kKeys + parts - 1) / parts * kKeys;
    const int64_t from = all.lo + (int64_t)part * per;
    all = Range{(int)min(from, (int64_t)all.hi), (int)min(from + per, (int64_t)all.hi)};
  }
  // The products begin from -lse / scale and -delta (heads of 64: gradient 521 -> 496 us at 8192 x
  // 16/8 heads); with 128 columns, where 32 registers for two values would spill, they are added.
  constexpr bool kFrom = DP < 128;
  const float nl = live ? a.neg_lse[job.pair * rows + r] : 0.0f, nd = live ? a.neg_delta[job.pair * rows + r] : 0.0f;
  v16f first_s{}, first_dp{};
  if (kFrom) first_s = nl, first_dp = nd;
  const float shift = kFrom ? 0.0f : nl * a.scale2, more = kFrom ? 0.0f : nd;

  v8bf q[T::kSteps], g[T::kSteps];
  row_frags<DP>(q, row_of(a.q, b, live ? t : 0, h), live, a.D, half);
  row_frags<DP>(g, row_of(a.dout, b, live ? t : 0, h), live, a.D, half);
  KeyLoader<DP, kKeys, 4> keys;   // waves 0 .. 3 load K, the others V
  const int lw = wave & 3, second = wave >> 2;
  keys.init(second ? a.v : a.k, b, hk, a.Tk, a.D, lw);
  T frag;
  frag.init(0);

  v16f dq[T::kBlocks] = {};
  auto tile = [&](int j, uint8_t* now, uint8_t* next) __attribute__((always_inline)) {
    tile_landed();
    if (j + kKeys < all.hi) keys.load(next + second * kHalf, lw, j + kKeys);
    if (j >= min(reach.hi, all.hi) || j + kKeys <= reach.lo) return;
    const uint8_t* tv = now + kHalf;
    v16f s[2], dp[2];
    pipeline<4 * T::kSteps, kAhead>(
        [&](int i) { return frag.read(i & 1 ? tv : now, i >> 2, (i & 2) * 16); },
        [&](int i, const v8bf& f) {
          const int kb = (i >> 1) & 1;
          if (i & 1)
            dp[kb] = mfma(f, g[i >> 2], i < 4 ? first_dp : dp[kb]);
          else
            s[kb] = mfma(f, q[i >> 2], i < 4 ? first_s : s[kb]);
        });
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int v = 0; v < 16; ++v)
        dp[kb][v] = __builtin_amdgcn_exp2f(kFrom ? s[kb][v] * a.scale2 : __builtin_fmaf(s[kb][v], a.scale2, shift)) *
                    (kFrom ? dp[kb][v] : dp[kb][v] + more);
    if (j < reach.all_lo || j + kKeys > min(reach.all_hi, all.hi)) {
      const uint32_t first = (uint32_t)(j + 4 * half - mine.lo), n = (uint32_t)max(min(mine.hi, all.hi) - mine.lo, 0);
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int v = 0; v < 16; ++v)
          if (first + kb * 32 + acc_row(v) >= n) dp[kb][v] = 0.0f;
    }
    v8bf ds;
    pipeline<4 * T::kBlocks, kAhead>([&](int i) { return frag.read_t(now, i % T::kBlocks, i / T::kBlocks); },
                                [&](int i, const v8bf& f) {
                                  const int db = i % T::kBlocks, ks = i / T::kBlocks;
                                  if (db == 0) ds = pack_half(dp[ks >> 1], ks & 1);
                                  dq[db] = mfma(f, ds, dq[db]);
                                });
  };
  if (all.lo < all.hi) keys.load(lds.s0 + second * kHalf, lw, all.lo);
  for (int j = all.lo; j < all.hi; j += 2 * kKeys) {
    tile(j, lds.s0, lds.s1);
    if (j + kKeys < all.hi) tile(j + kKeys, lds.s1, lds.s0);
  }
  // the dq of a row that sees one key is 0 (as in grad_keys), or NaN
  const float f = mine.hi - mine.lo == 1 ? 0.0f : 1.0f;
  if (__any(f == 0.0f)) {
#pragma unroll
    for (int db = 0; db < T::kBlocks; ++db) dq[db] *= f;
  }
  // NaN throughout anyway: where a row's lse or delta is, and it sees a key
  const bool lost = mine.lo < mine.hi && (nl != nl || nd != nd);
  uint64_t again = __ballot(live && odd_of(dq) != 0.0f && !lost);
  float* to = PARTS ? sums + (((int64_t)part * a.pairs + job.pair) * rows + r) * a.D : nullptr;
  if (live && !PARTS) store_columns(row_of_out(a.dq, b, t, h), dq, a.scale, a.D, half);
  if (live && PARTS) store_sums(to, dq, a.D, half);
  for (again |= again >> 32, again &= 0xffffffffu; again != 0; again &= again - 1) {
    const int from = __builtin_ctzll(again), tt = __shfl(t, from), hh = __shfl(h, from);
    const int lo = __shfl(mine.lo, from), hi = __shfl(mine.hi, from);
    RowSum x = row_dq(a, b, tt, hh, PARTS ? max(lo, all.lo) : lo, PARTS ? min(hi, all.hi) : hi);
    if (hi - lo == 1) x.x0 *= 0.0f, x.x1 *= 0.0f;
    if (PARTS)
      x.store(to + (int64_t)(from - (lane & 31)) * a.D, a.D);
    else
      x.store(row_of_out(a.dq, b, tt, hh), a.D, a.scale);
  }
}
#endif

// How the gradient's workgroups are shared out; sums of parts in the workspace.
struct Shares {
  int key_tiles, key_parts, row_tiles, row_parts;
  float *key_sums, *row_sums;
};

// One launch for both halves of the gradient: the keys' workgroups, which are few and
// long, come first, the queries' fill what they leave.
template <int DP, bool KP, bool RP>
__global__ __launch_bounds__(512, 2) void k_attn_grad(Args a, Shares sh) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int kRow = DP * 2;
  __shared__ __attribute__((aligned(1024))) uint8_t s0[128 * kRow], s1[128 * kRow], v[128 * kRow], stats[1024];
  const GradLds<DP> lds{s0, s1, v, stats};
  const uint32_t id = (uint32_t)block_xz(), kt = (uint32_t)a.pairs * (uint32_t)sh.key_tiles;
  const uint32_t keys = KP ? kt * (uint32_t)sh.key_parts : kt;
  if (id < keys) {
    const uint32_t part = KP ? id / kt : 0;
    grad_keys<DP, KP>(a, lds, job_of(id - part * kt, a.pairs, sh.key_tiles), (int)part, sh.key_parts, sh.key_sums,
                      (int64_t)a.pairs * a.Tk);
    return;
  }
  const uint32_t rt = (uint32_t)a.pairs * (uint32_t)sh.row_tiles, part = RP ? (id - keys) / rt : 0;
  if (id - keys < (RP ? rt * (uint32_t)sh.row_parts : rt))
    grad_queries<DP, RP>(a, lds, job_of(id - keys - part * rt, a.pairs, sh.row_tiles), sh.row_tiles, (int)part,
                         sh.row_parts, sh.row_sums);
#endif
}

// dq of each row from the parts' sums, in order, laid out as k_attn_join_keys.
template <int LANES>
__global__ __launch_bounds__(256) void k_attn_join_rows(Args a, uint32_t rows, int parts, const float* sums) {
  const uint32_t r = (uint32_t)block_xz() * (256 / LANES) + threadIdx.x / LANES;
  const int d = 4 * (threadIdx.x & (LANES - 1));
  if (r >= rows || d >= a.D) return;
  v4f dq{};
#pragma unroll 4
  for (int i = 0; i < parts; ++i) dq += *reinterpret_cast<const v4f*>(sums + ((int64_t)i * rows + r) * a.D + d);
  const uint32_t in_pair = (uint32_t)a.Tq * a.G, pair = r / in_pair, rr = r - pair * in_pair;
  const int b = pair / a.Hkv, t = rr / a.G, h = (pair - b * a.Hkv) * a.G + (rr - t * a.G);
  typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
  *reinterpret_cast<v4bf*>(row_of_out(a.dq, b, t, h) + d) = __builtin_convertvector(dq * a.scale, v4bf);
}

// dk and dv of each key from the parts' sums, in order: 32 lanes a key (16 up to 64 columns), four
// columns a lane.
template <int LANES>
__global__ __launch_bounds__(256) void k_attn_join_keys(Args a, uint32_t keys, int parts, const float* sums) {
  const uint32_t r = (uint32_t)block_xz() * (256 / LANES) + threadIdx.x / LANES;
  const int d = 4 * (threadIdx.x & (LANES - 1));
  if (r >= keys || d >= a.D) return;
  v4f dk{}, dv{};
#pragma unroll 4
  for (int i = 0; i < parts; ++i) {
    const float* at = sums + ((int64_t)i * keys + r) * 2 * a.D + d;
    dk += *reinterpret_cast<const v4f*>(at);
    dv += *reinterpret_cast<const v4f*>(at + a.D);
  }
  const uint32_t pair = r / a.Tk;
  const int j = (int)(r - pair * a.Tk), b = pair / a.Hkv, hk = pair - b * a.Hkv;
  typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
  *reinterpret_cast<v4bf*>(row_of_out(a.dk, b, j, hk) + d) = __builtin_convertvector(dk * a.scale, v4bf);
  *reinterpret_cast<v4bf*>(row_of_out(a.dv, b, j, hk) + d) = __builtin_convertvector(dv, v4bf);
}

int64_t sequences(const nvfp4_attn& a) { return a.cu_q == nullptr ? a.batch : 1; }

}  // namespace
}  // namespace attn

using namespace attn;

namespace {

// Keys of a sequence, on average.  A tile of packed rows walks the keys of all sequences in it: about as many as it
// has queries, or one sequence's, where queries and keys are the same tokens.  Few queries over long keys of
// their own are taken for less work than they are: 32 sequences of one query over 512 keys each (32/8 heads of 128) are 8
// workgroups of 256 tiles, 256 us; the same as a batch of sequences of one length takes 17.
int64_t keys_in(const nvfp4_attn& a) { return a.cu_q == nullptr || a.batch < 2 ? a.Tk : a.Tk / a.batch; }

// The n of at most `most` with the least chain / n + 8 + 1.3 n part (us).  Parts are whole tiles: of 65 tiles in 32
// parts, 22 have three and the others none.
int least_parts(double chain, double part, int64_t most) {
  int best = 1;
  double least = chain;
  for (int64_t n = 2; n <= most; ++n) {
    const double t = chain / n + 8.0 + 1.3 * n * part;
    if (t < least) least = t, best = (int)n;
  }
  return best;
}

// Workgroups that share a row's keys, at most 512 in all and parts of at least 128 keys.  A part
// costs its sums' way through memory (4.5 TB/s there and back) and the join a launch; the key
// tiles one after the other take 0.8 us each.  The n with the least sum of both.
int parts_of(const nvfp4_attn& a) {
  const int64_t G = a.Hq / a.Hkv, tiles = (a.Tq * G + kRowsWG - 1) / kRowsWG * sequences(a) * a.Hkv;
  if (tiles == 0 || tiles >= kPartTiles) return 1;
  const int64_t keys = keys_in(a);
  const int64_t most = keys / kPartKeys < kPartTiles / tiles ? keys / kPartKeys : kPartTiles / tiles;
  const double chain = (double)keys / kKeys * 0.8, part = (double)sequences(a) * a.Tq * a.Hq * a.D * 8 / 4.5e6;
  return least_parts(chain, part, most);
}

// Workgroups that share a key tile's query rows in the gradient, by the same rule: 1.1 us a step
// of 64 rows, and at most 256 in all, one for each compute unit (2048 queries of 40 heads over 8
// key heads, 128 tiles: 275 us whole, 215 in two parts, 238 in four; 4096: 628 and 682).  The
// longest chain counts, which the host does not know of packed sequences: it is taken as twice the
// average (gradient, by the average, twice and four times it: 12 documents of 1 .. 1371 in 4096, 8/2
// heads of 128: 154, 120, 130 us; 9 in 2048, 16/4 heads of 64: 79, 69, 68; of equal ones 8 in 2048: 44,
// 52, 51; 32 in 4096: 49, 49, 64).
int key_parts_of(const nvfp4_attn& a) {
  const int64_t tiles = (a.Tk + 127) / 128 * sequences(a) * a.Hkv;
  if (tiles == 0) return 1;
  const int64_t queries = a.cu_q == nullptr || a.batch < 2 ? a.Tq : a.Tq / a.batch * 2, steps = queries * (a.Hq / a.Hkv) / 64;
  return least_parts(steps * 1.1, (double)sequences(a) * a.Tk * a.Hkv * a.D * 16 / 4.5e6,
                     steps / 4 < 256 / tiles ? steps / 4 : 256 / tiles);
}

// Those that share a tile of query rows: 1.3 us a tile of keys.
int row_parts_of(const nvfp4_attn& a) {
  const int64_t tiles = (a.Tq * (a.Hq / a.Hkv) + kGradRows - 1) / kGradRows * sequences(a) * a.Hkv;
  if (tiles == 0) return 1;
  const int64_t steps = keys_in(a) / kKeys;
  return least_parts(steps * 1.3, (double)sequences(a) * a.Tq * a.Hq * a.D * 8 / 4.5e6,
                     steps / 4 < 256 / tiles ? steps / 4 : 256 / tiles);
}

// Bytes of the gradient's workspace, in this order: statistics, the keys' parts, the rows' parts.
struct GradSpace {
  int64_t stats, key_sums, row_sums;
};

// f(columns of the tiles): 64, 96 or 128.
template <class F>
void by_width(int D, F f) {
  if (D <= 64)
    f(std::integral_constant<int, 64>{});
  else if (D <= 96)
    f(std::integral_constant<int, 96>{});
  else
    f(std::integral_constant<int, 128>{});
}

int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }

GradSpace grad_space(const nvfp4_attn& a) {
  const int64_t rows = sequences(a) * a.Tq * a.Hq, keys = sequences(a) * a.Tk * a.Hkv;
  const int kp = key_parts_of(a), rp = row_parts_of(a);
  return GradSpace{up256(rows * 8), kp > 1 ? up256(keys * a.D * 8 * kp) : 0, rp > 1 ? rows * a.D * 4 * rp : 0};
}

}  // namespace

int64_t attn_workspace_bytes(const nvfp4_attn& a, bool grad) {
  const int64_t rows = sequences(a) * a.Tq * a.Hq;
  if (grad) {
    const GradSpace g = grad_space(a);
    return g.stats + g.key_sums + g.row_sums;
  }
  const int n = parts_of(a);
  return n > 1 ? up256(rows * n * a.D * 4) + rows * n * 8 : 0;
}

hipError_t launch_attn(const AttnCall& c, hipStream_t s) {
  const int64_t rows = sequences(c.a) * c.a.Tq * c.a.Hq;
  if (rows == 0) return hipSuccess;
  const Args a = make_args(c);
  const int pairs = (int)(sequences(c.a) * a.Hkv);
  const int tiles = (int)(((int64_t)a.Tq * a.G + kRowsWG - 1) / kRowsWG);
  Part part{nullptr, nullptr, parts_of(c.a)};
  const int64_t n = (int64_t)pairs * tiles;
  // Eight waves a workgroup where there is at most one for each compute unit and its keys are many
  // tiles (calls, one set of four waves and two: 188 workgroups of 24 tiles of width 64, 23.5 and 19.8 us; 128 of 32
  // of width 128, 38.5 and 34.0; 96 of 5, 11.6 and 11.5).  Up to two for each compute unit would gain as well (512
  // of 64 tiles of width 64: 16/16 heads 80 and 54, 16/4 80 and 70; of width 128 111 and 84); at four it makes no difference.
  const bool halves = part.n == 1 && n <= num_cus() && keys_in(c.a) >= 8 * kKeys;
  if (part.n > 1) {
    part.o = static_cast<float*>(c.ws);
    part.ml = reinterpret_cast<float*>(static_cast<uint8_t*>(c.ws) + up256(rows * part.n * a.D * 4));
  }
  const dim3 grid = grid_xz(n * part.n), block(halves ? 512 : 256);
  auto launch = [&](auto one, auto two) { (halves ? two : one)<<<grid, block, 0, s>>>(a, pairs, tiles, part); };
  auto width = [&](auto dp) {
    constexpr int DP = decltype(dp)::value;
    part.n == 1 ? launch(k_attn<DP, 1, false>, k_attn<DP, 2, false>) : launch(k_attn<DP, 1, true>, k_attn<DP, 1, true>);
  };
  by_width(a.D, width);
  if (part.n == 1) return hipGetLastError();
  if (part.n > 8)
    k_attn_join<<<grid_xz(rows), 256, 0, s>>>(a, (uint32_t)rows, part);
  else if (a.D <= 64)
    k_attn_join_few<16><<<grid_xz((rows + 15) / 16), 256, 0, s>>>(a, (uint32_t)rows, part);
  else
    k_attn_join_few<32><<<grid_xz((rows + 7) / 8), 256, 0, s>>>(a, (uint32_t)rows, part);
  return hipGetLastError();
}

hipError_t launch_attn_grad(const AttnCall& c, hipStream_t s) {
  const int64_t rows = sequences(c.a) * c.a.Tq * c.a.Hq;
  Args a = make_args(c);
  const GradSpace g = grad_space(c.a);
  a.neg_delta = a.neg_lse + g.stats / 8;
  Shares sh{(int)(((int64_t)a.Tk + 127) / 128),
            key_parts_of(c.a),
            (int)(((int64_t)a.Tq * a.G + kGradRows - 1) / kGradRows),
            row_parts_of(c.a),
            reinterpret_cast<float*>(static_cast<uint8_t*>(c.ws) + g.stats),
            reinterpret_cast<float*>(static_cast<uint8_t*>(c.ws) + g.stats + g.key_sums)};
  const int64_t n = (int64_t)a.pairs * sh.row_tiles * sh.row_parts + (int64_t)a.pairs * sh.key_tiles * sh.key_parts;
  if (n == 0) return hipSuccess;
  const dim3 grid = grid_xz(n);
  auto launch = [&](auto k) { k<<<grid, 512, 0, s>>>(a, sh); };
  const int stat_tiles = (int)(((int64_t)a.Tq * a.G + 127) / 128);
  const bool kp = sh.key_parts > 1, rp = sh.row_parts > 1;
  by_width(a.D, [&](auto dp) {
    constexpr int DP = decltype(dp)::value, kLanes = DP == 64 ? 16 : 32;
    if (rows > 0) k_attn_stats<DP><<<grid_xz((int64_t)a.pairs * stat_tiles), 256, 0, s>>>(a, stat_tiles);
    if (kp)
      rp ? launch(k_attn_grad<DP, true, true>) : launch(k_attn_grad<DP, true, false>);
    else
      rp ? launch(k_attn_grad<DP, false, true>) : launch(k_attn_grad<DP, false, false>);
    const int64_t keys = (int64_t)a.pairs * a.Tk;
    if (kp)
      k_attn_join_keys<kLanes><<<grid_xz((keys * kLanes + 255) / 256), 256, 0, s>>>(a, (uint32_t)keys, sh.key_parts,
                                                                                 sh.key_sums);
    if (rp)
      k_attn_join_rows<kLanes><<<grid_xz((rows * kLanes + 255) / 256), 256, 0, s>>>(a, (uint32_t)rows, sh.row_parts,
                                                                                 sh.row_sums);
  });
  return hipGetLastError();
}

}  // namespace nvfp4
