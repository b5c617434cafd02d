// lm_attn.h -- what the attention kernels share: operands, which keys a query sees, and
// the arithmetic of single rows (internal to libnvfp4.so).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>

#include "lm_attn_kernels.h"
#include "lm_device.h"

namespace nvfp4 {
namespace attn {

struct Rows {   // strides in elements
  const uint16_t* p;
  int64_t batch, token, head;
};

struct Args {
  Rows q, k, v, out, dout, dq, dk, dv;
  float* lse;      // [sequence][Tq][Hq], or [Tq][Hq]
  // gradient, of [sequence * key head][row]: -lse / scale and -delta, where the sums of the
  // scores and of dout . v begin: both come out of their products shifted
  float* neg_lse;
  float* neg_delta;
  const void* cu_q;
  const void* cu_k;
  int wide_cu, causal;
  int batch;       // sequences behind one another (cu), or the operands' first dimension
  int Tq, Tk, Hq, Hkv, G, D;
  int pairs;       // sequences (of one length; else 1) times key heads
  int64_t window;
  float scale, scale2;   // scale2 = scale * log2(e)
};

struct Range {   // of keys, or of query tokens
  int lo, hi;
};

__device__ __forceinline__ int cu_at(const void* cu, int wide, int i, int most) {
  const int64_t x = wide ? static_cast<const int64_t*>(cu)[i] : (int64_t) static_cast<const int32_t*>(cu)[i];
  return (int)(x < 0 ? 0 : x > most ? most : x);
}

// The sequence of row t: the last one that begins at or before t (empty ones before it
// begin there too); -1 if none does.
__device__ __forceinline__ int sequence_of(const void* cu, int wide, int n, int t, int most) {
  int lo = 0, hi = n + 1;   // cu[lo - 1] <= t < cu[hi], as far as looked
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu_at(cu, wide, mid, most) <= t)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo - 1;
}

// The same, formed by a whole wave, all lanes present: 64 entries are loaded at once and looked
// through by shuffles, and only what lies between two of them is searched in memory.  Up to 63
// sequences that is one load instead of six, each waiting for the last.
__device__ __forceinline__ int sequence_by_wave(const void* cu, int wide, int n, int t, int most) {
  const int lane = threadIdx.x & 63, step = n / 64 + 1;
  const int mine = cu_at(cu, wide, min(lane * step, n), most);
  int below = 0;   // of the 64, those at or before t
#pragma unroll
  for (int m = 32; m > 0; m >>= 1)
    if (__shfl(mine, below + m - 1) <= t) below += m;
  if (__shfl(mine, below) <= t) ++below;
  if (below == 0) return -1;
  int lo = min((below - 1) * step + 1, n + 1), hi = min(below * step, n + 1);
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu_at(cu, wide, mid, most) <= t)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo - 1;
}

__device__ __forceinline__ int clamp64(int64_t x, int lo, int hi) {
  return (int)(x < lo ? lo : x > hi ? hi : x);
}

struct Span {   // a sequence's queries and keys
  int q0, q1, k0, k1;
};
__device__ __forceinline__ Span span_of(const Args& a, int s) {
  if (s < 0 || s >= a.batch) return Span{0, 0, 0, 0};
  return Span{cu_at(a.cu_q, a.wide_cu, s, a.Tq), cu_at(a.cu_q, a.wide_cu, s + 1, a.Tq),
              cu_at(a.cu_k, a.wide_cu, s, a.Tk), cu_at(a.cu_k, a.wide_cu, s + 1, a.Tk)};
}

// The keys that query token t sees; empty for a t past the end.  WAVE: all lanes call.
template <bool WAVE>
__device__ __forceinline__ Range keys_of(const Args& a, int t) {
  Span s{0, a.Tq, 0, a.Tk};
  if (a.cu_q != nullptr)
    s = span_of(a, WAVE ? sequence_by_wave(a.cu_q, a.wide_cu, a.batch, t, a.Tq)
                        : sequence_of(a.cu_q, a.wide_cu, a.batch, t, a.Tq));
  if (t >= a.Tq || t < s.q0 || t >= s.q1 || s.k1 <= s.k0) return Range{0, 0};
  if (!a.causal) return Range{s.k0, s.k1};
  const int64_t end = (int64_t)(t - s.q0) + 1 + (s.k1 - s.k0) - (s.q1 - s.q0);
  const int hi = s.k0 + clamp64(end, 0, s.k1 - s.k0);
  const int lo = a.window > 0 ? s.k0 + clamp64(end - a.window, 0, s.k1 - s.k0) : s.k0;
  return Range{lo, hi};
}

// The query tokens that see key j; those before `more` see no other key.  All lanes call.
struct Seers {
  int lo, more, hi;
};
__device__ __forceinline__ Seers queries_of(const Args& a, int j) {
  Span s{0, a.Tq, 0, a.Tk};
  if (a.cu_q != nullptr) s = span_of(a, sequence_by_wave(a.cu_k, a.wide_cu, a.batch, j, a.Tk));
  if (j >= a.Tk || j < s.k0 || j >= s.k1 || s.q1 <= s.q0) return Seers{0, 0, 0};
  const bool one = s.k1 - s.k0 == 1;
  if (!a.causal) return Seers{s.q0, one ? s.q1 : s.q0, s.q1};
  const int64_t first = (int64_t)(j - s.k0) - ((s.k1 - s.k0) - (s.q1 - s.q0));
  const int lo = s.q0 + clamp64(first, 0, s.q1 - s.q0);
  const int hi = a.window > 0 ? s.q0 + clamp64(first + a.window, 0, s.q1 - s.q0) : s.q1;
  // the query whose last key is the sequence's first sees it alone
  const int more = one || a.window == 1 ? hi : j == s.k0 && first >= 0 ? min(lo + 1, hi) : lo;
  return Seers{lo, more, hi};
}

__device__ __forceinline__ int64_t stat_at(const Args& a, int b, int t, int h) {
  return ((int64_t)b * a.Tq + t) * a.Hq + h;
}
__device__ __forceinline__ const bf16_t* row_of(const Rows& r, int b, int t, int h) {
  return reinterpret_cast<const bf16_t*>(r.p) + b * r.batch + t * r.token + h * r.head;
}
__device__ __forceinline__ bf16_t* row_of_out(const Rows& r, int b, int t, int h) {
  return const_cast<bf16_t*>(row_of(r, b, t, h));
}

// The sum over aligned groups of 8 lanes, in each of them.
__device__ __forceinline__ float sum_of_8(float x) {
#define MOVED(how) __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), how, 15, 15, true))
  x += MOVED(0xB1);    // the other one of two
  x += MOVED(0x4E);    // the other two of four
  x += MOVED(0x141);   // mirrored within 8
#undef MOVED
  return x;
}
__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) x += __shfl_xor(x, m);
  return x;
}
__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) x = fmaxf(x, __shfl_xor(x, m));
  return x;
}

__device__ __forceinline__ float dot(const bf16_t* x, const bf16_t* y, int D) {
  float s = 0.0f;
  for (int d = 0; d < D; d += 8) {
    const v8f a = load8(x + d), b = load8(y + d);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(a[i], b[i], s);
  }
  return s;
}

// --------------------------------------------------------------- single rows
// One wave, one row at a time; only keys (or queries) that count are looked at, so
// nothing that a mask hides can reach a result.  A lane forms the score of one key of
// 64, then owns two columns.

struct RowSum {   // columns lane and lane + 64
  float x0 = 0.0f, x1 = 0.0f;
  // += w * row
  __device__ __forceinline__ void add(const bf16_t* row, int D, float w) {
    const int lane = threadIdx.x & 63;
    if (lane < D) x0 = fmaf(w, load1(row + lane), x0);
    if (lane + 64 < D) x1 = fmaf(w, load1(row + lane + 64), x1);
  }
  __device__ __forceinline__ void store(bf16_t* row, int D, float f) const {
    const int lane = threadIdx.x & 63;
    if (lane < D) store1(row + lane, x0 * f);
    if (lane + 64 < D) store1(row + lane + 64, x1 * f);
  }
  __device__ __forceinline__ void store(float* row, int D) const {
    const int lane = threadIdx.x & 63;
    if (lane < D) row[lane] = x0;
    if (lane + 64 < D) row[lane + 64] = x1;
  }
};

struct Soft {   // scores in log2: the running maximum, the sum relative to it
  float m, l;
  RowSum o;
};

// The query's softmax over keys lo .. hi - 1.
__device__ inline Soft row_forward(const Args& a, int b, int t, int h, int lo, int hi) {
  const int lane = threadIdx.x & 63, hk = h / a.G;
  const bf16_t* q = row_of(a.q, b, t, h);
  Soft r{-INFINITY, 0.0f, {}};
  for (int j0 = lo; j0 < hi; j0 += 64) {
    const int j = j0 + lane, n = min(64, hi - j0);
    const float s = j < hi ? dot(q, row_of(a.k, b, j, hk), a.D) * a.scale2 : -INFINITY;
    // a NaN score must not be dropped by the maximum
    const float m = fmaxf(r.m, wave_max(s)), at = m == -INFINITY ? 0.0f : m;
    const float p = j < hi ? exp2f(s - at) : 0.0f, f = r.m == -INFINITY ? 0.0f : exp2f(r.m - at);
    r.l = r.l * f + wave_sum(p);
    r.o.x0 *= f;
    r.o.x1 *= f;
    r.m = m;
    for (int i = 0; i < n; ++i) r.o.add(row_of(a.v, b, j0 + i, hk), a.D, __shfl(p, i));
  }
  return r;
}

// p and ds of one query and key.
__device__ __forceinline__ void pair_grad(const Args& a, int b, int t, int h, int j, float& p, float& ds) {
  const int hk = h / a.G;
  const int64_t r = ((int64_t)b * a.Hkv + hk) * a.Tq * a.G + (int64_t)t * a.G + (h - hk * a.G);
  p = exp2f((dot(row_of(a.q, b, t, h), row_of(a.k, b, j, hk), a.D) + a.neg_lse[r]) * a.scale2);
  ds = p * (dot(row_of(a.dout, b, t, h), row_of(a.v, b, j, hk), a.D) + a.neg_delta[r]);
}

// Keys lo .. hi - 1's part of a query's dq, before the scale.
__device__ inline RowSum row_dq(const Args& a, int b, int t, int h, int lo, int hi) {
  const int lane = threadIdx.x & 63, hk = h / a.G;
  RowSum dq;
  for (int j0 = lo; j0 < hi; j0 += 64) {
    const int j = j0 + lane, n = min(64, hi - j0);
    float p = 0.0f, ds = 0.0f;
    if (j < hi) pair_grad(a, b, t, h, j, p, ds);
    for (int i = 0; i < n; ++i) dq.add(row_of(a.k, b, j0 + i, hk), a.D, __shfl(ds, i));
  }
  return dq;
}

__device__ __forceinline__ bool nan_throughout(const bf16_t* row, int D) {
  const int lane = threadIdx.x & 63;
  const float x = lane < D ? load1(row + lane) : NAN, y = lane + 64 < D ? load1(row + lane + 64) : NAN;
  return __all(x != x && y != y);
}

// Whether query rows lo .. hi - 1 make a key that they see NaN throughout: dk and dv by an lse, dk by a
// delta, dv by a row of dout (of 64 in a row with such deltas one is looked at).  By the statistics, 64
// rows at a time: a step that has diverged is told by its first rows, where forming its keys again would
// take hundreds of times an ordinary gradient.
struct NanRows {
  bool dk, dv;
};
__device__ inline NanRows nan_rows(const Args& a, int b, int hk, int64_t lo, int64_t hi, bool dv_too) {
  const int lane = threadIdx.x & 63;
  const int64_t first = ((int64_t)b * a.Hkv + hk) * a.Tq * a.G;
  NanRows is{false, false};
  for (int64_t r0 = lo; r0 < hi && !(is.dk && (is.dv || !dv_too)); r0 += 64) {
    const bool there = r0 + lane < hi;
    const float l = there ? a.neg_lse[first + r0 + lane] : 0.0f, d = there ? a.neg_delta[first + r0 + lane] : 0.0f;
    if (__any(l != l)) return NanRows{true, true};
    const uint64_t lost = __ballot(d != d);
    if (lost == 0) continue;
    const int64_t r = r0 + __builtin_ctzll(lost);
    is.dk = true;
    is.dv = nan_throughout(row_of(a.dout, b, (int)(r / a.G), hk * a.G + (int)(r % a.G)), a.D);
  }
  return is;
}

// Query rows lo .. hi - 1 (token * G + head of the group), added to dk and dv; those before `more` see
// no other key.
__device__ inline void row_dkv(const Args& a, int b, int j, int hk, int64_t lo, int64_t more, int64_t hi,
                               RowSum& dk, RowSum& dv) {
  const int lane = threadIdx.x & 63;
  for (int64_t r0 = lo; r0 < hi; r0 += 64) {
    const int64_t r = r0 + lane;
    const int n = (int)min((int64_t)64, hi - r0);
    float p = 0.0f, ds = 0.0f;
    if (r < hi) pair_grad(a, b, (int)(r / a.G), hk * a.G + (int)(r % a.G), j, p, ds);
    if (r < more) ds *= 0.0f;
    for (int i = 0; i < n; ++i) {
      const int t = (int)((r0 + i) / a.G), h = hk * a.G + (int)((r0 + i) % a.G);
      dv.add(row_of(a.dout, b, t, h), a.D, __shfl(p, i));
      dk.add(row_of(a.q, b, t, h), a.D, __shfl(ds, i));
    }
  }
}

// ------------------------------------------------------------------- tiles
// Products run on v_mfma_f32_32x32x16_bf16.  Rows of q (and dout) are counted over the
// heads of a group: row r is token r / G of head r % G, so that all heads of a group share the
// tiles of their keys.

typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_void;
typedef __attribute__((address_space(3))) v4s* lds_v4s;

constexpr uint32_t kDead = 0x80000000u;   // a byte offset past every descriptor: reads zero
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t descriptor(const uint16_t* p) {
  return __builtin_amdgcn_make_buffer_rsrc(
      reinterpret_cast<void*>(uniform64((int64_t)(uintptr_t)p)), (short)0, 0x7fffffff, 0x00020000);
}

// N products whose operands come from LDS: each is read AHEAD products before its own.
// (Left alone, the compiler reads a product's operands right before it, to spare
// registers, and waits out the LDS each time.)  Arithmetic may move across.
template <int N, int AHEAD, class Read, class Use>
__device__ __forceinline__ void pipeline(Read read, Use use) {
  constexpr int kArithmetic = 0x2 | 0x4 | 0x400;
  decltype(read(0)) f[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) f[i] = read(i);
  __builtin_amdgcn_sched_barrier(kArithmetic);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    use(i, f[i % AHEAD]);
    if (i + AHEAD < N) f[i % AHEAD] = read(i + AHEAD);
    __builtin_amdgcn_sched_barrier(kArithmetic);
  }
}

__device__ __forceinline__ v16f mfma(v8bf a, v8bf b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// A tile of ROWS rows of DP values (64, 96 or 128) in LDS: blocks of 32 columns, in each 64
// bytes a row, whose 16-byte chunk c lies at c ^ ((row >> 2) & 3).  Both reads are free of bank
// conflicts: the same chunk of 16 rows (fragments along d) and the transposing read, where 32
// lanes take 64 bytes of 4 rows, cover 256 bytes each.  Two lane addresses serve all reads of a kind;
// blocks and steps are immediate offsets.
template <int DP, int ROWS>
struct Tile {
  static constexpr int kSteps = DP / 16, kBlocks = DP / 32;   // of 16 and of 32 columns
  static constexpr int kBlock = ROWS * 64, kBytes = kBlocks * kBlock;
  int along[2], across[2];   // by parity of the step; lower and upper rows of a step of 16

  __device__ __forceinline__ void init(int row0) {
    const int lane = threadIdx.x & 63, half = lane >> 5, r = lane & 31;
    const int g = lane >> 4, j = lane & 15;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      along[x] = (row0 + r) * 64 + (((2 * x + half) ^ ((r >> 2) & 3)) << 4);
      const int row = 4 * (g >> 1) + (j >> 2) + 8 * x;
      across[x] = (row0 + row) * 64 + (((2 * (g & 1) + ((j & 3) >> 1)) ^ ((row >> 2) & 3)) << 4) + (j & 1) * 8;
    }
  }
  // Row lane & 31 of 32, columns 16 ks + 8 half + (0 .. 7).
  __device__ __forceinline__ v8bf read(const uint8_t* tile, int ks, int row0 = 0) const {
    return *reinterpret_cast<const v8bf*>(tile + along[ks & 1] + (ks >> 1) * kBlock + row0 * 64);
  }
  // Column 32 db + (lane & 31) of rows 4 half + (0 .. 3) and those 8 on, of step t of 16 rows.
  __device__ __forceinline__ v8bf read_t(const uint8_t* tile, int db, int t) const {
    const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(tile + across[0] + db * kBlock + t * 1024));
    const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(tile + across[1] + db * kBlock + t * 1024));
    return __builtin_bit_cast(v8bf, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

// All loads to LDS have landed, in every wave; what a wave read is free.  The wait is a
// builtin: the compiler then knows that reads need no wait of their own.
__device__ __forceinline__ void tile_landed() {
  __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0), and lgkmcnt(0): its reads have ended
  asm volatile("s_barrier" ::: "memory");
}

// How WAVES waves share the loads of a tile: each takes one 1 KiB piece of 16 rows in some
// of the blocks, so that a lane has one row.
template <int DP, int ROWS, int WAVES>
struct Share {
  static constexpr int kBlocks = DP / 32;
  static constexpr int kLoads = ROWS / 16 * kBlocks / WAVES;
  static_assert(kLoads >= 1 && kBlocks % kLoads == 0, "");
  static __device__ __forceinline__ int block(int wave) { return wave * kLoads % kBlocks; }
  static __device__ __forceinline__ int group(int wave) { return wave * kLoads / kBlocks; }
  static __device__ __forceinline__ int row(int wave) { return group(wave) * 16 + ((threadIdx.x & 63) >> 2); }
  // The lane's source column in its first block; that of load q is 32 q on.
  static __device__ __forceinline__ int column(int wave) {
    const int lane = threadIdx.x & 63;
    return block(wave) * 32 + (((lane & 3) ^ ((lane >> 4) & 3)) << 3);
  }
  // off: the lane's bytes from buf, or kDead; columns from D on read zero.
  static __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t buf, uint8_t* tile, int wave, uint32_t off,
                                              int left) {
    uint8_t* to = tile + block(wave) * ROWS * 64 + group(wave) * 1024;
    load_blocks(buf, to, off, left, std::make_integer_sequence<int, kLoads>{});
  }

 private:
  template <int... Q>
  static __device__ __forceinline__ void load_blocks(__amdgpu_buffer_rsrc_t buf, uint8_t* to, uint32_t off, int left,
                                                     std::integer_sequence<int, Q...>) {
    (__builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_void)(to + Q * ROWS * 64), 16, left > Q * 32 ? off : kDead,
                                              Q * 64, 0, 0),
     ...);
  }
};

// Loads ROWS consecutive key rows into LDS, WAVES waves together; rows past the end and
// columns past D read zero.
template <int DP, int ROWS, int WAVES>
struct KeyLoader {
  using S = Share<DP, ROWS, WAVES>;
  const uint16_t* base;
  int64_t ld;
  uint32_t off;
  int end, row, left;   // left: columns from the lane's first on

  __device__ __forceinline__ void init(const Rows& x, int b, int hk, int rows, int D, int wave) {
    base = x.p + b * x.batch + hk * x.head;
    ld = x.token;
    end = rows;
    row = S::row(wave);
    off = (uint32_t)row * (uint32_t)ld * 2 + S::column(wave) * 2;
    left = D - S::column(wave);
  }
  __device__ __forceinline__ void load(uint8_t* tile, int wave, int j0) const {
    S::load(descriptor(base + (int64_t)j0 * ld), tile, wave, row < end - j0 ? off : kDead, left);
  }
};

// Loads ROWS consecutive rows of q or of dout into a tile, WAVES waves together: the rows
// of a group of heads are tokens and heads in turn.  Each call takes the rows before the last
// call's.
template <int DP, int ROWS, int WAVES>
struct RowLoader {
  using S = Share<DP, ROWS, WAVES>;
  const uint16_t* base;
  int64_t ld;
  uint32_t head;
  int step_t, step_g, G, end, t0, g0;   // t0, g0: token and head of the tile's first row
  int t, g, row, left;                  // the lane's

  __device__ __forceinline__ void init(const Rows& x, const Args& a, int b, int hk, int r0, int wave) {
    G = a.G;
    base = x.p + b * x.batch + (int64_t)hk * G * x.head;
    ld = x.token;
    head = (uint32_t)x.head * 2;
    step_t = ROWS / G, step_g = ROWS - step_t * G;
    end = a.Tq * G;
    t0 = r0 / G, g0 = r0 - t0 * G;
    row = r0 + S::row(wave);
    t = row / G;
    g = row - t * G;
    left = a.D - S::column(wave);
  }
  // The rows at hand to LDS; then back by ROWS.
  __device__ __forceinline__ void load(uint8_t* tile, int wave) {
    const uint32_t off = (uint32_t)(t - t0) * (uint32_t)ld * 2 + (uint32_t)g * head + (uint32_t)S::column(wave) * 2;
    S::load(descriptor(base + (int64_t)t0 * ld), tile, wave, row < end ? off : kDead, left);
    row -= ROWS;
    t -= step_t;
    g -= step_g;
    if (g < 0) g += G, --t;
    t0 -= step_t;
    g0 -= step_g;
    if (g0 < 0) g0 += G, --t0;
  }
};

// The range that any of the rows (or keys) of a wave reaches, and the one that all
// reach; rows that do not exist reach all.  What a row reaches before `plain` is a case of its own: the
// range of all begins behind it, and it ends at `apart` in the wave (0: none has any).
struct Reach {
  int lo, hi, all_lo, all_hi, apart;
};
__device__ __forceinline__ Reach reach_of(bool live, int lo, int plain, int hi) {
  Reach r{lo < hi ? lo : 0x7fffffff, lo < hi ? hi : 0, live ? plain : 0, live ? hi : 0x7fffffff,
          lo < plain ? plain : 0};
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    r.lo = min(r.lo, __shfl_xor(r.lo, m));
    r.hi = max(r.hi, __shfl_xor(r.hi, m));
    r.all_lo = max(r.all_lo, __shfl_xor(r.all_lo, m));
    r.all_hi = min(r.all_hi, __shfl_xor(r.all_hi, m));
    r.apart = max(r.apart, __shfl_xor(r.apart, m));
  }
  return Reach{uniform(r.lo), uniform(r.hi), uniform(r.all_lo), uniform(r.all_hi), uniform(r.apart)};
}
// The reach of WAVES waves, {0, 0} if none reaches anything; lds is free before and after.
template <int WAVES>
__device__ __forceinline__ Range reach_of_all(uint8_t* lds, const Reach& r, int wave) {
  int* ends = reinterpret_cast<int*>(lds);
  if ((threadIdx.x & 63) == 0) ends[2 * wave] = r.lo, ends[2 * wave + 1] = r.hi;
  __syncthreads();
  int lo = ends[0], hi = ends[1];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) lo = min(lo, ends[2 * w]), hi = max(hi, ends[2 * w + 1]);
  __syncthreads();
  return lo < hi ? Range{uniform(lo), uniform(hi)} : Range{0, 0};
}

// Eight values of global memory, or zeros.
__device__ __forceinline__ v8bf piece(const bf16_t* at, bool there) {
  v4u x{};
  if (there) x = *reinterpret_cast<const v4u*>(at);
  return __builtin_bit_cast(v8bf, x);
}

// Lane's fragments along d of one row of global memory.
template <int DP>
__device__ __forceinline__ void row_frags(v8bf (&f)[DP / 16], const bf16_t* row, bool live, int D, int half) {
#pragma unroll
  for (int ks = 0; ks < DP / 16; ++ks) f[ks] = piece(row + 16 * ks + 8 * half, live && 16 * ks + 8 * half < D);
}

// An accumulator of columns lane & 31 as rows of global memory, times f.
template <int BLOCKS>
__device__ __forceinline__ void store_columns(bf16_t* row, const v16f (&o)[BLOCKS], float f, int D, int half) {
  typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int db = 0; db < BLOCKS; ++db)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = db * 32 + 8 * i + 4 * half;
      if (d >= D) continue;
      v4f x;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = o[db][4 * i + e] * f;
      *reinterpret_cast<v4bf*>(row + d) = __builtin_convertvector(x, v4bf);
    }
}

// The same as FP32.
template <int BLOCKS>
__device__ __forceinline__ void store_sums(float* row, const v16f (&o)[BLOCKS], int D, int half) {
#pragma unroll
  for (int db = 0; db < BLOCKS; ++db)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = db * 32 + 8 * i + 4 * half;
      if (d < D)
        *reinterpret_cast<v4f*>(row + d) = v4f{o[db][4 * i], o[db][4 * i + 1], o[db][4 * i + 2], o[db][4 * i + 3]};
    }
}

// 0, or NaN if a sum is not finite.
template <int BLOCKS>
__device__ __forceinline__ float odd_of(const v16f (&o)[BLOCKS]) {
  float odd = 0.0f;
#pragma unroll
  for (int db = 0; db < BLOCKS; ++db)
#pragma unroll
    for (int v = 0; v < 16; ++v) odd = __builtin_fmaf(o[db][v], 0.0f, odd);
  return odd;
}

// max and sum over a lane and the one 32 away
__device__ __forceinline__ float pair_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float pair_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Eight scores or probabilities as the second operand of a product.
__device__ __forceinline__ v8bf pack_half(const v16f& x, int half) {
  v8f y;
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = x[8 * half + i];
  return __builtin_convertvector(y, v8bf);
}

// Word v of an accumulator: row (v & 3) + 8 (v >> 2) + 4 half, column lane & 31.
__device__ __forceinline__ constexpr int acc_row(int v) { return (v & 3) + 8 * (v >> 2); }

// Eight workgroups in a row run on the eight XCDs.  Sequences and key heads go round
// the XCDs, so that an XCD's L2 holds the keys of its own; what 8 does not divide comes last.
struct Job {
  int pair, tile;
};
__device__ __forceinline__ Job job_of(uint32_t id, int pairs, int tiles) {
  const uint32_t even = (uint32_t)pairs & ~7u, n = (uint32_t)tiles;
  if (id < even * n) {
    const uint32_t i = id >> 3, p = i / n;
    return Job{(int)((id & 7) + 8 * p), (int)(i - p * n)};
  }
  const uint32_t i = id - even * n, p = i / n;
  return Job{(int)(even + p), (int)(i - p * n)};
}

Args make_args(const AttnCall& c);

}  // namespace attn
}  // namespace nvfp4
