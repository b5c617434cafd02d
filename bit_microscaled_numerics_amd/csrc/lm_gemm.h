// lm_gemm.h -- the BF16 matrix-product core of the cross-entropy kernels
// (internal to libnvfp4.so).
//
// One workgroup computes a 256 x (64 WN) tile of C[n][m] = sum_k A[m][k] B[n][k]
// (m is the contiguous index of the result).  4 waves, one per SIMD, as 2 x 2:
// a wave owns 128 values of m and 32 WN of n, 4 x WN blocks of
// v_mfma_f32_32x32x16_bf16 with FP32 accumulators (256 registers at WN = 4, so
// that every operand byte read from LDS feeds four MFMAs).  The accumulator
// layout gives a lane one n and runs of 4 consecutive m, so sums over m (the
// softmax statistics over the vocabulary) stay in registers.
//
// K advances 64 at a time through two LDS stages filled by buffer loads that
// write LDS directly.  Each operand lies in memory either K-contiguous ([row][k],
// a stage row is 128 B) or transposed ([k][row], a stage row is 512 B of 256
// rows' values, read back with ds_read_b64_tr_b16, which hands each lane 4
// consecutive k of its row).  Neither product of the backward pass therefore
// needs a transposed copy of an operand.
//
// Pipeline: a step is four phases of 16 k.  In the first every wave reads the
// fragments of the other three, 96 registers; a barrier later the stage is free
// and its refill with the step after next is issued between the second and third
// phases' MFMAs, spread out: issued together, the loads stall the waves at issue
// (all four leave the barrier at once).  Before the fourth phase the next stage must
// have landed: its loads were issued a step and a half (96 MFMAs, 3072 cycles)
// earlier, with the refill just issued still in flight.  A third stage, which narrow
// tiles have room for, gained nothing (13.6 -> 14.5 us a round of 1024 x 65536 x 512).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lm_device.h"

namespace nvfp4 {
namespace lm {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef uint16_t v8u16 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_void;
typedef __attribute__((address_space(3))) v4s* lds_v4s;

constexpr int kThreads = 256;      // 4 waves
constexpr int kTM = 256;           // m per workgroup
constexpr int kBK = 64;            // k per stage
constexpr int kWM = 4;             // 32-wide m blocks per wave
constexpr uint32_t kDead = 0x80000000u;       // a byte offset past any num_records used here
constexpr uint32_t kBufFlags = 0x00020000u;   // raw buffer, 32-bit data format

// A matrix operand: rows x k values, K-contiguous (p[row * ld + k]) or
// transposed (p[k * ld + row]).
struct Operand {
  const uint16_t* p;
  int64_t ld;
  int64_t rows;   // rows that exist; others read as zero, or only reach results that are not stored
};

// A descriptor from values that are the same in every lane.  They are moved to
// scalar registers explicitly: sizes that were loaded from memory are not known
// to be uniform, and a descriptor in vector registers puts a loop around every
// load.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const uint16_t* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(
      reinterpret_cast<void*>(uniform64((int64_t)(uintptr_t)p)), (short)0, uniform(bytes),
      (int)kBufFlags);
}

// Stage position of 16-byte chunk j of row r in the K-contiguous layout:
// j ^ swz(r).  A 16-byte LDS read serves 16 lanes (16 consecutive rows, one
// chunk) per cycle over 256 B; swz is a bijection on the even and on the odd
// rows of any 16, so they touch distinct bank groups.
__device__ __forceinline__ int swz(int r) { return ((r >> 1) ^ ((r & 1) << 1)) & 7; }

// s_waitcnt immediate: vmcnt <= n, nothing else waited on
constexpr int vmcnt_imm(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }

// ROWS rows of an operand, one stage at a time.
template <bool TR, int ROWS>
struct Loader;

template <int ROWS>
struct Loader<false, ROWS> {
  static constexpr int kLoads = ROWS / 32;      // per wave and stage: 8 rows of 128 B each
  static constexpr int kReads = 1;              // LDS instructions per fragment
  __amdgpu_buffer_rsrc_t buf;
  uint32_t voff[kLoads];
  int chunk[2];       // source chunk of this lane, in even and odd loads
  uint32_t frag[4];   // LDS offset of this lane's fragment of block 0, by sub-step
  int K;

  __device__ __forceinline__ void init(const Operand& o, int64_t row0, int64_t k_total, int wave,
                                       int frag_row0) {
    const int lane = fresh_lane();
    const int64_t rem = o.rows - row0;
    const int64_t last = rem < ROWS ? rem - 1 : ROWS - 1;   // below 2^31 bytes (pitch <= 2^22)
    buf = rsrc(o.p + row0 * o.ld, rem > 0 ? (int)((last * o.ld + k_total) * 2) : 0);
    K = uniform((int)k_total);
#pragma unroll
    for (int par = 0; par < 2; ++par) chunk[par] = (lane & 7) ^ swz(par * 8 + (lane >> 3));
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int r = wave * (ROWS / 4) + q * 8 + (lane >> 3);
      voff[q] = (uint32_t)(r * o.ld * 2 + chunk[q & 1] * 16) | (r < rem ? 0u : kDead);
    }
    const int row = frag_row0 + (lane & 31);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
      frag[ks] = (uint32_t)(row * 128 + (((2 * ks + (lane >> 5)) ^ swz(row)) << 4));
  }

  // Load q of the stage that starts at k0.  Chunks at or past K read zero.
  __device__ __forceinline__ void load(uint8_t* stage, int wave, int q, int64_t k0) const {
    const uint32_t dead = (int)k0 + chunk[q & 1] * 8 >= K ? kDead : 0u;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_void)(stage + (wave * (ROWS / 4) + q * 8) * 128),
                                             16, voff[q] | dead, (uint32_t)k0 * 2, 0, 0);
  }
  __device__ __forceinline__ void step(int64_t) {}

  __device__ __forceinline__ v8bf read(const uint8_t* stage, int ks, int i) const {
    return *reinterpret_cast<const v8bf*>(stage + frag[ks] + i * 32 * 128);
  }
};

// Transposed: stage row = one k, ROWS = 256 values of it (32 chunks of 16 B);
// chunk j of row k sits at j ^ (4 (k & 3)).  A transposing read takes, per 16
// lanes, 4 rows x 32 B; the exchange spreads the 4 rows over the banks.
template <int ROWS>
struct Loader<true, ROWS> {
  static_assert(ROWS == 256, "");
  static constexpr int kLoads = 8;              // per wave and stage: 2 k rows of 512 B each
  static constexpr int kReads = 2;
  const uint16_t* base;
  int64_t ld;
  int pitch, tail, K;   // bytes per k row; bytes of the last row past the operand's end
  __amdgpu_buffer_rsrc_t buf;
  uint32_t voff[kLoads];
  uint32_t frag[4];   // by block

  __device__ __forceinline__ void init(const Operand& o, int64_t row0, int64_t k_total, int wave,
                                       int frag_row0) {
    const int lane = fresh_lane();
    base = o.p + row0;
    ld = o.ld;
    pitch = (int)(o.ld * 2);
    tail = (int)((o.ld - (o.rows - row0)) * 2);
    K = uniform((int)k_total);
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int k = wave * 16 + q * 2 + (lane >> 5);
      voff[q] = (uint32_t)(k * ld * 2 + (((lane & 31) ^ (4 * (k & 3))) << 4));
    }
    // group g of 16 lanes reads rows k = 8 (g >> 1) + .. and columns 16 (g & 1) + ..
    const int g = lane >> 4, j = lane & 15, k = 8 * (g >> 1) + (j >> 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int chunk = (frag_row0 + i * 32 + (g & 1) * 16) / 8 + ((j & 3) >> 1);
      frag[i] = (uint32_t)(k * 512 + ((chunk ^ (4 * (j >> 2))) << 4) + (j & 1) * 8);
    }
  }

  // Base the descriptor at the stage's first k, so offsets stay in 32 bits
  // however long K is; rows at or past K lie past num_records.
  __device__ __forceinline__ void step(int64_t k0) {
    const int left = min(max(K - (int)k0, 0), kBK);
    buf = rsrc(base + k0 * ld, max(left * pitch - tail, 0));
  }
  __device__ __forceinline__ void load(uint8_t* stage, int wave, int q, int64_t) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_void)(stage + (wave * 16 + q * 2) * 512), 16,
                                             voff[q], 0, 0, 0);
  }
  __device__ __forceinline__ v8bf read(const uint8_t* stage, int ks, int i) const {
    const uint8_t* at = stage + frag[i] + ks * 16 * 512;
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(at));
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(at + 4 * 512));
    return __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

template <int WN>
struct Frags {
  v8bf a[kWM], b[WN];
};

template <bool ATR, bool BTR, int WN>
struct Core {
  using LA = Loader<ATR, kTM>;
  using LB = Loader<BTR, 64 * WN>;
  LA a;
  LB b;
  v16f acc[kWM][WN];

  __device__ __forceinline__ void read(Frags<WN>& f, const uint8_t* sa, const uint8_t* sb, int ks) {
#pragma unroll
    for (int i = 0; i < kWM; ++i) f.a[i] = a.read(sa, ks, i);
#pragma unroll
    for (int j = 0; j < WN; ++j) f.b[j] = b.read(sb, ks, j);
  }

  // FIRST: the sums begin here, from the constant zero.
  template <bool FIRST = false>
  __device__ __forceinline__ void mfma(const Frags<WN>& f) {
#pragma unroll
    for (int i = 0; i < kWM; ++i)
#pragma unroll
      for (int j = 0; j < WN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[i], f.b[j],
                                                            FIRST ? v16f{} : acc[i][j], 0, 0, 0);
  }

  __device__ __forceinline__ void load_a(uint8_t* sa, int wave, int64_t k0) {
#pragma unroll
    for (int q = 0; q < LA::kLoads; ++q) a.load(sa, wave, q, k0);
  }
  __device__ __forceinline__ void load_b(uint8_t* sb, int wave, int64_t k0) {
#pragma unroll
    for (int q = 0; q < LB::kLoads; ++q) b.load(sb, wave, q, k0);
  }

  // The order of a phase: after each MFMA its share of LDS reads (0x100) and of
  // loads to LDS (0x010).
  template <int READS, int LOADS>
  __device__ __forceinline__ void interleave() {
    constexpr int kMfma = kWM * WN;
    constexpr int kPerR = (READS + kMfma - 1) / kMfma, kPerL = (LOADS + kMfma - 1) / kMfma;
    constexpr int kGap = LOADS > 0 && LOADS < kMfma ? kMfma / LOADS : 1;
#pragma unroll
    for (int m = 0; m < kMfma; ++m) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (m * kPerR < READS) __builtin_amdgcn_sched_group_barrier(0x100, kPerR, 0);
      if (m % kGap == 0 && m / kGap * kPerL < LOADS)
        __builtin_amdgcn_sched_group_barrier(0x010, kPerL, 0);
    }
  }

  // One stage: (ca, cb) holds step s, (na, nb) step s + 1; f[0] is read already.
  template <bool FIRST = false>
  __device__ __forceinline__ void stage(Frags<WN> (&f)[4], uint8_t* ca, uint8_t* cb, uint8_t* na,
                                        uint8_t* nb, int wave, int64_t s) {
    constexpr int kRead = kWM * LA::kReads + WN * LB::kReads;
    constexpr int kLoad = LA::kLoads + LB::kLoads;
#pragma unroll
    for (int ks = 1; ks < 4; ++ks) read(f[ks], ca, cb, ks);
    mfma<FIRST>(f[0]);
    interleave<3 * kRead, 0>();
    __builtin_amdgcn_sched_barrier(0);
    // this wave holds the whole stage in registers; when all do, it is free
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    a.step((s + 2) * kBK);
    b.step((s + 2) * kBK);
    load_a(ca, wave, (s + 2) * kBK);
    mfma(f[1]);
    interleave<0, LA::kLoads>();
    __builtin_amdgcn_sched_barrier(0);
    load_b(cb, wave, (s + 2) * kBK);
    mfma(f[2]);
    interleave<0, LB::kLoads>();
    __builtin_amdgcn_sched_barrier(0);
    // the next stage has landed: all but the loads just issued
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(kLoad));
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    read(f[0], na, nb, 0);
    mfma(f[3]);
    interleave<kRead, 0>();
    __builtin_amdgcn_sched_barrier(0);
  }

  // Quarter `part` of the loads of steps s0 and s0 + 1 (all four before run()).
  // The stages must be free.
  __device__ __forceinline__ void start(uint8_t* a0, uint8_t* b0, uint8_t* a1, uint8_t* b1, int wave,
                                        int64_t s0, int part) {
    const int64_t k0 = s0 * kBK, k1 = k0 + kBK;
    if (part == 0) a.step(k0), load_a(a0, wave, k0);
    if (part == 1) b.step(k0), load_b(b0, wave, k0);
    if (part == 2) a.step(k1), load_a(a1, wave, k1);
    if (part == 3) b.step(k1), load_b(b1, wave, k1);
  }

  // acc = the products of k in [64 s0, k_end), k_end the end that both
  // operands were set up with, after start(s0, 0 .. 3).  Steps past it load nothing and
  // read as zero, so the loop runs whole pairs without a branch.  Ends with the
  // stages free.
  template <class Pace>
  __device__ __forceinline__ void run(uint8_t* a0, uint8_t* b0, uint8_t* a1, uint8_t* b1, int wave,
                                      int64_t s0, int64_t k_end, Pace pace) {
#ifdef __HIP_DEVICE_COMPILE__   // the host pass rejects a second use of what this instantiates
    // Narrow tiles start their sums from the constant zero in a first pair of its own
    // (1 to 2% of 333 x 50257 x 2048); with wide ones that costs spills.
    constexpr bool kPeel = WN < 4;
    if (!kPeel) {
#pragma unroll
      for (int i = 0; i < kWM; ++i)
#pragma unroll
        for (int j = 0; j < WN; ++j) acc[i][j] = v16f{};
    }
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
    Frags<WN> f[4];
    read(f[0], a0, b0, 0);
    int64_t s = s0;
    if (kPeel) {
      stage<true>(f, a0, b0, a1, b1, wave, s);
      stage(f, a1, b1, a0, b0, wave, s + 1);
      pace(0);
      s += 2;
    }
    for (; s * kBK < k_end; s += 2) {
      stage(f, a0, b0, a1, b1, wave, s);
      stage(f, a1, b1, a0, b0, wave, s + 1);
      pace((int)(s - s0));
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
#endif
  }
  __device__ __forceinline__ void run(uint8_t* a0, uint8_t* b0, uint8_t* a1, uint8_t* b1, int wave,
                                      int64_t s0, int64_t k_end) {
    run(a0, b0, a1, b1, wave, s0, k_end, [](int) {});
  }
};

// The accumulators' places: lane l of the wave at (wm, wn) holds, in word v of
// block (i, j), m = 128 wm + 32 i + (v & 3) + 8 (v >> 2) + 4 (l >> 5) and
// n = 32 WN wn + 32 j + (l & 31) of the tile.
__device__ __forceinline__ int acc_m(int i, int v, int half) {
  return 32 * i + (v & 3) + 8 * (v >> 2) + 4 * half;
}

}  // namespace lm
}  // namespace nvfp4
