// Tile engine of the large microscaled products: a BN x BM tile of Y^T (BN
// rows of the 4-bit W, BM rows of X) per workgroup on
// v_mfma_scale_f32_32x32x64_f8f6f4, fp32 accumulators in registers.
//
// W is the instruction's first operand, so a lane ends with four consecutive
// columns of one row of Y (8-byte stores). Lane l (g = l / 32, l % 32 the row)
// supplies, of the instruction's two blocks of 32, for a 4-bit operand the 16
// bytes of block g, for an 8-bit one 16 bytes of each block (the half g), and
// the scale byte of block g.
//
// The reduction runs in steps of 128 elements, two instructions deep. Codes
// come by global_load_lds_dwordx4 into a ring of LDS stages, two or three steps
// ahead, one barrier a step; nothing is decoded. With a 4-bit X the larger tiles
// copy two steps together and have one barrier for them: 64 bytes of a row are
// half a cache line, and both halves cross to the compute unit for each (2048 x
// 22016 x 8192 210 us without it, 201 with; 301 x 4096 x 11008, where few
// workgroups wait for each other's copies, 25 without, 31 with). Scales come
// the same way into two buffers, SP pieces of 16 bytes of a row (512 elements
// each) every 4 SP steps: a piece alone costs a whole cache line on its way, so
// SP is 2 or 4 where the LDS is there (301 x 4096 x 11008 27.3 -> 26.0 us, with
// a 4-bit X 25.5 -> 23.6). The matrix instructions of a step's second half run
// after the next step's barrier: they cover its first LDS reads.
//
// Bound by the copies and the matrix cores together: 4096^3 with an 8-bit X 52
// to 55 us (2.5 PFLOP/s, the cores 69 % busy), 2048 x 22016 x 8192 with a 4-bit
// one 183 to 193 (3.8 to 4.0 PFLOP/s, 56 %). The copies alone, with the matrix
// instructions left out of builds that took 57 and 204 us: 34 and 162.
//
// LDS rows are 128 bytes (8-bit codes) or 64 (4-bit), unpadded. Sixteen lanes
// of a 16-byte read go through the 64 banks at a time, so a row's chunks are
// swapped by an exclusive or with row / 2 (128 bytes) or row / 4 (64 bytes):
// sixteen consecutive rows read at one chunk then lie on all banks. (With the
// row itself in the exclusive or, half of the LDS's cycles were conflicts. The
// counters still call 31 to 39 % of them that, about 42 cycles of a wave's step
// with either type of X; which reads they belong to is not known.) A copy
// fetches the chunk that belongs at its lane's place.
//
// Behind the end of K the last step re-reads chunks of the same rows; their
// scale bytes are the pad bytes 0 of both operands, 2^-254 together, which
// vanishes in fp32 for every finite code. Rows past M or N are read from the
// last row and not stored.
#pragma once

#include "gemm_core.h"
#include "mx_device.h"

namespace qnf4 {

typedef int mx_v4i __attribute__((ext_vector_type(4)));
typedef int mx_v8i __attribute__((ext_vector_type(8)));

// The registers of one operand: 16 bytes (4-bit codes) or two times 16.
__device__ __forceinline__ mx_v8i mx_operand(mx_v4i a) { return __builtin_shufflevector(a, mx_v4i{0, 0, 0, 0}, 0, 1, 2, 3, 4, 5, 6, 7); }
__device__ __forceinline__ mx_v8i mx_operand(mx_v4i a, mx_v4i b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

template <int XT_, int NF_, int MF_, int WN_, int WM_, int STAGES_, int SP_ = 1, int KG_ = 1, bool PAIR_ = false>
struct MxTile {
  static constexpr int XT = XT_, NF = NF_, MF = MF_, WN = WN_, WM = WM_, STAGES = STAGES_, SP = SP_, KG = KG_;
  static constexpr int kWaves = WN * WM, kThreads = 64 * kWaves * KG;   // waves of one group
  static constexpr int BN = 32 * NF * WN, BM = 32 * MF * WM;
  static constexpr int kXRow = XT == QLORA_MX_FP4 ? 64 : 128;   // bytes of a row and step
  static constexpr int kW = BN * 64, kX = BM * kXRow, kStage = kW + kX;
  static constexpr int kScale = (BN + BM) * 16 * SP;             // SP pieces of 16 scales of a row, 4 SP steps
  static constexpr int kRing = STAGES * kStage + 2 * kScale;   // of one group
  static constexpr int kLds = KG * kRing;
  static constexpr int kWCopies = kW / 1024 / kWaves, kXCopies = kX / 1024 / kWaves;
  static constexpr int kCopies = kWCopies + kXCopies;
  static_assert(kW % (1024 * kWaves) == 0 && kX % (1024 * kWaves) == 0, "whole copies per wave");
  static constexpr int kScaleRows = 64 / SP;   // rows of a scale copy
  static constexpr int kScaleBlocks = kScale / 1024, kScaleCopies = (kScaleBlocks + kWaves - 1) / kWaves;
  static_assert(BN % 64 == 0 && BM % 64 == 0 && (SP == 1 || SP == 2 || SP == 4), "whole scale copies");
  static_assert(kLds <= 160 * 1024, "LDS");
  // the steps go in pairs, copied together, two steps ahead
  static constexpr bool kPair = PAIR_;
  static constexpr int kAhead = kPair ? 2 : STAGES - 1;
  static constexpr int kNewer = kPair ? 0 : kCopies * (STAGES - 2);   // copies in flight behind a step's own
  // a buffer of scales (4 SP steps) is filled kAhead steps ahead: not before its readers are done
  static_assert(kPair ? STAGES == 4 && XT == QLORA_MX_FP4 : STAGES == 3 || STAGES == 4, "ring");
  static_assert(kNewer < 64, "vmcnt range");
  // after the main loop: the groups' sums, then 32 rows of bf16 for each wave of the first group
  static constexpr int kSums = (KG - 1) * BN * BM * 4, kStoreRow = 64 * NF + 16, kStore = 32 * kStoreRow;
  static_assert(kSums + kWaves * kStore <= kLds, "sums and rows fit the rings");
};

// Byte offset of chunk c of row r in a tile of 64-byte rows / 128-byte rows.
__device__ __forceinline__ uint32_t mx_off64(int r, int c) {
  return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 2) & 3)) << 4));
}
__device__ __forceinline__ uint32_t mx_off128(int r, int c) {
  return static_cast<uint32_t>(r * 128 + ((c ^ ((r >> 1) & 7)) << 4));
}

// A value that is the same in all lanes, in scalar registers.
__device__ __forceinline__ int64_t mx_uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(static_cast<uint64_t>(v) >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ const uint8_t *mx_uniform(const uint8_t *p) {
  return reinterpret_cast<const uint8_t *>(mx_uniform(static_cast<int64_t>(reinterpret_cast<uintptr_t>(p))));
}

// 16 bytes per lane from base + off into LDS at dst + 16 lane. Returns nothing
// into registers; waits are explicit (mx_wait).
__device__ __forceinline__ void mx_copy(uint32_t dst, uint32_t off, const uint8_t *base) {
  lds_copy16(__builtin_amdgcn_readfirstlane(dst), off, base);
}

// Until at most N vector-memory operations of the wave are in flight.
template <int N>
__device__ __forceinline__ void mx_wait() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
  asm volatile("" ::: "memory");
}

// Every LDS read of this wave is in registers, then the workgroup's barrier.
__device__ __forceinline__ void mx_barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The copies of one operand: rows of ROWB bytes a step, lane's chunk and rows.
template <int ROWB, int COPIES, int WAVES>
struct MxCopies {
  const uint8_t *base;
  uint32_t row[COPIES];   // byte offset of the lane's row per copy
  uint32_t chunk, last;   // byte of the lane's chunk in the step; the row's last chunk
  __device__ MxCopies(const uint8_t *codes, int64_t row0, int64_t rows, int64_t ld, int w) {
    base = mx_uniform(codes + row0 * ld);
    const int lane = threadIdx.x & 63;
    int r, c;   // row of the wave's first block that the lane copies, chunk that belongs at its place
    if constexpr (ROWB == 64) {
      r = lane >> 2;
      c = (lane & 3) ^ ((r >> 2) & 3);
    } else {
      static_assert(WAVES % 2 == 0, "a wave's blocks of eight rows are all even or all odd");
      r = lane >> 3;
      c = (lane & 7) ^ (4 * (w & 1) + (r >> 1));
    }
    const int64_t end = rows - 1 - row0;
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
      const int64_t at = (w + WAVES * i) * (1024 / ROWB) + r;
      row[i] = static_cast<uint32_t>((at < end ? at : end) * ld);
    }
    chunk = static_cast<uint32_t>(16 * c);
    last = static_cast<uint32_t>(ld - 16);
  }
  // Copy i of a step; dst: LDS address of the wave's first block of the tile.
  __device__ __forceinline__ void issue(int i, int step, uint32_t dst) const {
    mx_copy(dst + 1024u * WAVES * i, row[i] + min(static_cast<uint32_t>(step) * ROWB + chunk, last), base);
  }
};

template <class T>
struct MxFrags {
  mx_v8i w[T::NF], x[T::MF];
};

template <class T>
struct MxAcc {
  f32x16 v[T::NF][T::MF];
};

// One slice's matrix instructions, with the scale bytes 2 SLICE of the words;
// after(i) is called behind those of W fragment i.
template <class T, int SLICE, class F>
__device__ __forceinline__ void mx_mma(MxAcc<T> &acc, const MxFrags<T> &f, const int (&sw)[T::NF], const int (&sx)[T::MF],
                                       F after) {
#pragma unroll
  for (int i = 0; i < T::NF; ++i) {
#pragma unroll
    for (int j = 0; j < T::MF; ++j)
      acc.v[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          f.w[i], f.x[j], acc.v[i][j], 4, T::XT == QLORA_MX_FP4 ? 4 : 0, 2 * SLICE, sw[i], 2 * SLICE, sx[j]);
    after(i);
  }
}

struct MxOperands {
  const uint8_t *x, *xs, *w, *ws;
  int64_t x_rows, w_rows;      // rows that may be read
  int64_t x_ld, w_ld;          // bytes of a row of codes
  uint32_t pitch;
};

// acc += the tile at (n0, m0) over steps [s0, s1) of the wave's group; s0 a
// multiple of four, `most` the longest group's number of steps (every wave
// passes that many barriers).
template <class T>
__device__ __forceinline__ void mx_mainloop(MxAcc<T> &acc, const MxOperands &p, int64_t n0, int64_t m0, int s0, int s1,
                                            int most, char *smem, int wave) {
  const int lane = threadIdx.x & 63;
  const int r = lane & 31, g = lane >> 5;
  const int wn = wave / T::WM, wm = wave % T::WM;
  const uint32_t lds = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char *)smem));
  const MxCopies<64, T::kWCopies, T::kWaves> cw(p.w, n0, p.w_rows, p.w_ld, wave);
  const MxCopies<T::kXRow, T::kXCopies, T::kWaves> cx(p.x, m0, p.x_rows, p.x_ld, wave);
  // scales: block b of kScaleRows rows (W's rows, then X's) by wave b % kWaves,
  // a row's SP pieces swapped so that 32 rows' reads of one lie on 16 banks
  const uint8_t *sbase[T::kScaleCopies];
  uint32_t srow[T::kScaleCopies];
  const uint32_t spiece = 16u * ((lane ^ (lane >> 4)) & (T::SP - 1)), slast = p.pitch - 16;
#pragma unroll
  for (int c = 0; c < T::kScaleCopies; ++c) {
    const int first = T::kScaleRows * (wave + T::kWaves * c);
    const bool of_w = first < T::BN;
    sbase[c] = mx_uniform(of_w ? p.ws + n0 * p.pitch : p.xs + m0 * p.pitch);
    const int64_t end = of_w ? p.w_rows - 1 - n0 : p.x_rows - 1 - m0;
    const int64_t at = first - (of_w ? 0 : T::BN) + lane / T::SP;
    srow[c] = static_cast<uint32_t>((at < end ? at : end) * p.pitch);
  }
  const uint32_t sdst = lds + T::STAGES * T::kStage + 1024u * wave;

  // Copies of step `step` (and the next one, where they go in pairs), part
  // `part` of `parts`. Steps past the end copy the last one again, into a stage
  // that is not read any more: every step has the same copies, and one wait
  // count serves them all.
  auto issue = [&](int step, int part, int parts) {
    const uint32_t rel = static_cast<uint32_t>(step - s0);
    if (rel % (4 * T::SP) == 0 && part == 0) {
      // pieces behind a row's last one are not read: the last stands in for them
      const uint32_t at = min(4u * static_cast<uint32_t>(step) + spiece, slast);
#pragma unroll
      for (int c = 0; c < T::kScaleCopies; ++c)
        if (wave + T::kWaves * c < T::kScaleBlocks)
          mx_copy(sdst + (rel / (4 * T::SP) & 1) * T::kScale + 1024u * T::kWaves * c, srow[c] + at, sbase[c]);
    }
#pragma unroll
    for (int c = 0; c < T::kCopies; ++c)
      if (c * parts / T::kCopies == part) {
#pragma unroll
        for (int k = 0; k < (T::kPair ? 2 : 1); ++k) {
          const uint32_t stage = lds + static_cast<uint32_t>((step + k - s0) % T::STAGES) * T::kStage + 1024u * wave;
          const int from = min(step + k, s1 - 1);
          if (c < T::kWCopies) cw.issue(c, from, stage);
          else cx.issue(c - T::kWCopies, from, stage + T::kW);
        }
      }
  };

  // the lane's LDS offsets within a stage, slices 0 and 1
  uint32_t ow[2], oxa[2], oxb[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    ow[s] = mx_off64(32 * T::NF * wn + r, 2 * s + g);
    if constexpr (T::XT == QLORA_MX_FP4) {
      oxa[s] = T::kW + mx_off64(32 * T::MF * wm + r, 2 * s + g);
    } else {
      oxa[s] = T::kW + mx_off128(32 * T::MF * wm + r, 4 * s + g);
      oxb[s] = T::kW + mx_off128(32 * T::MF * wm + r, 4 * s + 2 + g);
    }
  }
  // part `part` of NF of a slice's fragments
  auto read = [&](MxFrags<T> &f, const char *stage, int s, int part) {
#pragma unroll
    for (int j = 0; j < T::MF; ++j) {
      if (j * T::NF / T::MF != part) continue;
      const mx_v4i xa = *reinterpret_cast<const mx_v4i *>(stage + oxa[s] + 32 * T::kXRow * j);
      if constexpr (T::XT == QLORA_MX_FP4) f.x[j] = mx_operand(xa);
      else f.x[j] = mx_operand(xa, *reinterpret_cast<const mx_v4i *>(stage + oxb[s] + 32 * T::kXRow * j));
    }
    f.w[part] = mx_operand(*reinterpret_cast<const mx_v4i *>(stage + ow[s] + 2048 * part));
  };

  const uint32_t sswap = static_cast<uint32_t>(r) >> (T::SP == 4 ? 2 : 3);   // as the copies swap a row's pieces
  int sw[T::NF], sx[T::MF];       // scale words of this step, the lane's blocks in bytes 0 and 2
  MxFrags<T> f0, f1;
  if (s1 > s0) {
#pragma unroll
    for (int i = 0; i < T::kAhead; i += T::kPair ? 2 : 1) issue(s0 + i, 0, 1);
  }

  auto step = [&](auto jc, int i) {
    constexpr int j = decltype(jc)::value;
    constexpr bool kCopying = !T::kPair || j % 2 == 0;
    if (kCopying) {
      mx_wait<T::kNewer>();
      mx_barrier();
    }
    if (T::KG > 1 && i >= s1) return;
    const char *stage = smem + static_cast<uint32_t>((i - s0) % T::STAGES) * T::kStage;
    const uint32_t rel = static_cast<uint32_t>(i - s0);
    const char *sc = smem + T::STAGES * T::kStage + (rel / (4 * T::SP) & 1) * T::kScale + 16 * T::SP * r +
                     16 * ((rel / 4 ^ sswap) & (T::SP - 1)) + 4 * j;
    uint32_t pw[T::NF], px[T::MF];
    // The LDS reads of the next half and the copies of a later step go out
    // between the matrix instructions. With the copies in front of them every
    // wave waited for the others' (the compute unit takes 16 cycles for 1 KB),
    // and the matrix cores stood still for a third of the step.
    const auto first = [&](int n) {
      read(f0, stage, 0, n);
      if (n == T::NF - 1) {
#pragma unroll
        for (int k = 0; k < T::NF; ++k) pw[k] = *reinterpret_cast<const uint32_t *>(sc + 512 * T::SP * (T::NF * wn + k));
#pragma unroll
        for (int m = 0; m < T::MF; ++m) px[m] = *reinterpret_cast<const uint32_t *>(sc + T::SP * (16 * T::BN + 512 * (T::MF * wm + m)));
      }
      if (kCopying) issue(i + T::kAhead, n, 2 * T::NF);
      __builtin_amdgcn_sched_barrier(0);
    };
    if (j > 0 || i > s0) {   // the previous step's second half
      mx_mma<T, 1>(acc, f1, sw, sx, first);
    } else {
#pragma unroll
      for (int n = 0; n < T::NF; ++n) first(n);
    }
#pragma unroll
    for (int n = 0; n < T::NF; ++n) sw[n] = static_cast<int>(pw[n] >> (8 * g));
#pragma unroll
    for (int m = 0; m < T::MF; ++m) sx[m] = static_cast<int>(px[m] >> (8 * g));
    mx_mma<T, 0>(acc, f0, sw, sx, [&](int n) {
      read(f1, stage, 1, n);
      if (kCopying) issue(i + T::kAhead, T::NF + n, 2 * T::NF);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  const int end = T::KG > 1 ? s0 + most : s1;
  for (int i = s0; i < end; i += 4) {
    step(std::integral_constant<int, 0>{}, i);
    if (i + 1 < end) step(std::integral_constant<int, 1>{}, i + 1);
    if (i + 2 < end) step(std::integral_constant<int, 2>{}, i + 2);
    if (i + 3 < end) step(std::integral_constant<int, 3>{}, i + 3);
  }
  if (s1 > s0) mx_mma<T, 1>(acc, f1, sw, sx, [](int) {});
  mx_wait<0>();   // no copy may land in LDS that somebody else has by then
}

// The whole product of a tile: the workgroup's KG groups of waves take a
// contiguous part of the steps each, with a ring of their own, and the first
// group gets the sums, added in group order. Returns whether the wave is of
// that group; `wave` is its number in the group.
template <class T>
__device__ __forceinline__ bool mx_tile_product(MxAcc<T> &acc, const MxOperands &p, int64_t n0, int64_t m0, int steps,
                                                char *smem, int &wave) {
#pragma unroll
  for (int i = 0; i < T::NF; ++i)
#pragma unroll
    for (int j = 0; j < T::MF; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc.v[i][j][e] = 0.0f;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), group = w / T::kWaves;
  wave = w % T::kWaves;
  const int per = T::KG > 1 ? (steps + 4 * T::KG - 1) / (4 * T::KG) * 4 : steps;
  const int s0 = min(steps, group * per);
  mx_mainloop<T>(acc, p, n0, m0, s0, min(steps, s0 + per), min(steps, per), smem + group * T::kRing, wave);
  __syncthreads();   // the rings are free
  if constexpr (T::KG > 1) {
    float4 *sums = reinterpret_cast<float4 *>(smem);
    constexpr int kRegs = T::NF * T::MF * 4;   // float4 a lane
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < kRegs; ++i) {
        const f32x16 &v = acc.v[i / 4 / T::MF][i / 4 % T::MF];
        const int q = 4 * (i % 4);
        sums[((group - 1) * kRegs + i) * (64 * T::kWaves) + 64 * wave + (threadIdx.x & 63)] = make_float4(v[q], v[q + 1], v[q + 2], v[q + 3]);
      }
    }
    __syncthreads();
    if (group > 0) return false;
#pragma unroll
    for (int k = 0; k < T::KG - 1; ++k)
#pragma unroll
      for (int i = 0; i < kRegs; ++i) {
        f32x16 &v = acc.v[i / 4 / T::MF][i / 4 % T::MF];
        const int q = 4 * (i % 4);
        const float4 a = sums[(k * kRegs + i) * (64 * T::kWaves) + 64 * wave + (threadIdx.x & 63)];
        v[q] += a.x, v[q + 1] += a.y, v[q + 2] += a.z, v[q + 3] += a.w;
      }
  }
  return true;
}

// Orders the wave's LDS accesses in front of it before those behind it, for
// data that passes between lanes. The LDS takes a wave's accesses in order, so
// this holds for the compiler only and costs no instruction.
__device__ __forceinline__ void mx_wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// Y[m][n] = bf16(acc), m < m_end, n < N. Lane l holds row m = l % 32 of a
// fragment, columns 8 q + 4 (l / 32) + 0 .. 3. Rows whose length is a multiple
// of eight go through LDS, 32 at a time in a place of the wave's own, and out
// as whole runs of a row, 16 bytes a lane: stored from the registers, 8 bytes
// of each of 32 rows at a time, the end of a 4096^3 product took 15 us. `smem`
// is free from kSums on.
template <class T>
__device__ __forceinline__ void mx_store(const MxAcc<T> &acc, __bf16 *y, int64_t N, int64_t n0, int64_t m0,
                                         int64_t m_end, int wave, char *smem) {
  const int lane = threadIdx.x & 63;
  const int wn = wave / T::WM, wm = wave % T::WM;
  n0 += 32 * T::NF * wn;
  m0 += 32 * T::MF * wm;
  if ((N & 7) == 0) {
    char *place = smem + T::kSums + wave * T::kStore;
    constexpr int kChunks = 4 * T::NF, kRows = 64 / kChunks;   // 16-byte runs of a row, rows a store covers
#pragma unroll
    for (int j = 0; j < T::MF; ++j) {
#pragma unroll
      for (int i = 0; i < T::NF; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16 &v = acc.v[i][j];
          *reinterpret_cast<uint2 *>(place + (lane & 31) * T::kStoreRow + 64 * i + 16 * q + 8 * (lane >> 5)) =
              make_uint2(pack_bf16x2(v[4 * q], v[4 * q + 1]), pack_bf16x2(v[4 * q + 2], v[4 * q + 3]));
        }
      mx_wave_order();
      const int c = lane % kChunks;
      const int64_t n = n0 + 8 * c;
#pragma unroll
      for (int k = 0; k < 32 / kRows; ++k) {
        const int r = kRows * k + lane / kChunks;
        const int64_t m = m0 + 32 * j + r;
        const uint4 v = *reinterpret_cast<const uint4 *>(place + r * T::kStoreRow + 16 * c);
        if (m < m_end && n < N) *reinterpret_cast<uint4 *>(y + m * N + n) = v;
      }
      mx_wave_order();   // the next rows take the place
    }
  } else {
#pragma unroll
    for (int j = 0; j < T::MF; ++j) {
      const int64_t m = m0 + 32 * j + (lane & 31);
      if (m >= m_end) continue;
#pragma unroll
      for (int i = 0; i < T::NF; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int64_t n = n0 + 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
          if (n < N) y[m * N + n] = static_cast<__bf16>(acc.v[i][j][e]);
        }
    }
  }
}

}  // namespace qnf4
