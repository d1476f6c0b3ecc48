// The gated block's forward for a few rows (M <= 32): both weights stream past
// registers once.
//
//   k_gated_low     Hs = bf16(s X [Ag; Au]^T), a workgroup for each adapter row
//   k_gated_row     one row of X: sums of both weights and the adapters' terms, the gate
//   k_gated_few     up to four rows, and longer or unaligned single ones
//   k_gated_stream  more rows
//
// k_gated_few and k_gated_stream. A unit is 16 rows, eight of the gate and the
// same eight of the other weight: the rows of one v_mfma_f32_16x16x32_bf16 whose
// columns are rows of X. The eight waves of a workgroup share a unit's reduction. Lane
// l (r = l % 16 the row, g = l / 16) loads 16 bytes, the 32 codes of a half
// block; a transposition over the four lanes of a row (permlane swaps) gives lane
// g the g-th eight codes of each of the four half blocks, so that an
// instruction's reduction lies in one block of 64 and its sums can take the
// block's constant afterwards, once for 64 products: acc += c (instruction's
// sums). A byte of codes is two bf16 levels (times level_factor) out of a table
// in LDS, in sixteen copies (entry e of copy l % 16), and goes into the
// instruction as it comes.
// Constants of a unit's rows are formed together and pass through LDS, where a
// lane reads those of its four rows of the sums at once. Codes and raw constants
// of the next turn are requested before this one's are used.
//
// Two weights of 11008 x 4096 (46 MB), double quantization, r = 64: 1 row 18.1 us
// (13.3, 3.5 TB/s, without adapters: k_gated_low, its launch and the wait for it
// are 4 of these), 4 rows 27.1, 16 rows 39.1, 32 rows 51.6. k_gated_few took 23.6
// and 17.9 us for one row, 14.5 with the table's reads left out: a product per
// instruction has 15 columns to spare there, and each turn's barrier waits for
// loads that the next turn's do not hide whole. 32 copies of its table measured
// the same, 64 leave one workgroup on a compute unit (29 us); waves that go
// through a reduction alone, without barriers, 20 to 23 us for one row.
#include <algorithm>

#include "block.h"
#include "gate.h"
#include "nf4_linear.h"

namespace qnf4 {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kCopies = 16;

constexpr int kLowWaves = 8;   // for one row (1 x 4096 x 11008 in all: 22.8 us with 4, 21.3 with 8, 20.8 with 16)

struct LowParams {
  const __bf16 *X;
  const void *A[2];
  bool bf16;
  int64_t K;
  int M, r, rp;
  float scale;
  __bf16 *Hs;   // [M][2 rp]
};

// Eight values of an adapter row as fp32 pairs' worth of bf16.
__device__ __forceinline__ bf16x8 adapter8(const void *p, bool bf16, int64_t i) {
  if (bf16) return *reinterpret_cast<const bf16x8 *>(static_cast<const __bf16 *>(p) + i);
  const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
  const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i + 4);
  return bf16x8{static_cast<__bf16>(a.x), static_cast<__bf16>(a.y), static_cast<__bf16>(a.z), static_cast<__bf16>(a.w),
                static_cast<__bf16>(b.x), static_cast<__bf16>(b.y), static_cast<__bf16>(b.z), static_cast<__bf16>(b.w)};
}

// A workgroup has one adapter row and one row or up to eight of X; its waves
// share the reduction. Sums in a fixed order.
template <int ROWS, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_gated_low(const LowParams p) {
  __shared__ float part[WAVES][ROWS];
  const int row = blockIdx.x, w = row >= p.rp, j = row - w * p.rp;
  const int m0 = ROWS * static_cast<int>(blockIdx.y), lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float acc[ROWS];
#pragma unroll
  for (int m = 0; m < ROWS; ++m) acc[m] = 0.0f;
  if (j < p.r) {
    for (int64_t k = 8 * threadIdx.x; k < p.K; k += 512 * WAVES) {
      const bf16x8 a = adapter8(w ? p.A[1] : p.A[0], p.bf16, j * p.K + k);
#pragma unroll
      for (int m = 0; m < ROWS; ++m) {
        if (ROWS > 1 && m0 + m >= p.M) break;   // uniform
        const bf16x8 x = *reinterpret_cast<const bf16x8 *>(p.X + (m0 + m) * p.K + k);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[m] = fmaf(static_cast<float>(a[e]), static_cast<float>(x[e]), acc[m]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < ROWS; ++m) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) acc[m] += __shfl_xor(acc[m], o);
    if (lane == 0) part[wave][m] = acc[m];
  }
  __syncthreads();
  if (threadIdx.x < ROWS && m0 + static_cast<int>(threadIdx.x) < p.M) {
    const int m = threadIdx.x;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += part[w][m];
    p.Hs[static_cast<int64_t>(m0 + m) * 2 * p.rp + row] = static_cast<__bf16>(p.scale * v);
  }
}

struct StreamParams {
  const __bf16 *X;
  const uint8_t *codes[2];
  const int8_t *absmax_q[2];
  const float *dq_scale[2], *dq_mean[2], *absmax[2];
  const __bf16 *Hs;
  const void *B[2];
  bool bf16;
  int r, rp;
  __bf16 *H, *G, *U;
  int64_t N, K;
  float inverse;   // of level_factor
  int M, units, chunks;
};

// What the levels are multiplied by before they are rounded to bf16, the
// operand type, and the constants divided by. All weights with one code share
// its level's rounding, and the levels' own do not cancel: the mean error of an
// NF4 weight is 4.6e-4 of the weights' standard deviation, which a sum over K
// elements of X adds up K times where X has a mean (4096 elements, mean 1:
// G off by 2.1e-2). Times 1.287 the mean error is below 6e-6 for normal,
// uniform, Laplace and t distributed weights, the root of the mean square
// 1.44e-3 (1.38e-3 without; 1.6e-3 is what rounding each weight by itself
// makes). FP4 levels are twelfths: times 1.5 they need no rounding.
inline float level_factor(int format) { return (format & kFmtFp4) ? 1.5f : 1.287f; }

// Dword g of each of the four registers of the lanes of a row: register p of
// lane g becomes dword g of lane p's.
__device__ __forceinline__ void transpose4(u32x4 &v) {
  // lanes g, g ^ 2: the upper half of a register against the lower of another
  auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  // lanes g, g ^ 1
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  v = u32x4{c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ void fill_table(uint32_t (&lut)[256 * kCopies], const Nf4Tables &tab) {
  for (int i = threadIdx.x; i < 256 * kCopies; i += kThreads) lut[i] = pack_bf16x2(tab.lv[(i / kCopies) >> 4], tab.lv[(i / kCopies) & 15]);
}

// The sums of 128 elements of the reduction of a unit's 16 rows: codes v (as
// loaded), x the operands of the four half blocks, c0 and c1 the constants of
// the lane's four rows in the two blocks.
template <int MT>
__device__ __forceinline__ void decode_step(f32x4 (&acc)[MT], u32x4 v, const u32x4 (&x)[MT][4], const float *c0, const float *c1,
                                            const char *table, uint32_t copy) {
  transpose4(v);
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    f32x4 sum[MT];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w = v[2 * b + h];
      u32x4 levels;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        levels[e] = *reinterpret_cast<const uint32_t *>(table + ((((w >> (8 * e)) & 0xffu) << 6) | copy));
#pragma unroll
      for (int t = 0; t < MT; ++t)
        sum[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, levels), __builtin_bit_cast(bf16x8, x[t][2 * b + h]),
                                                         h ? sum[t] : f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
    }
    const f32x4 k = *reinterpret_cast<const f32x4 *>(b ? c1 : c0);
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][e] = fmaf(k[e], sum[t][e], acc[t][e]);
  }
}

// A block's constant from what is stored: the bits as loaded, and converted
// where they are used. A conversion beside the load would wait for it, and for
// every load in front of it (1 x 11008 x 4096 19.6 us so, without adapters).
template <bool DQ>
__device__ __forceinline__ void request_constant(const StreamParams &p, int w, int64_t e, uint32_t &raw, float &factor) {
  if constexpr (DQ) {
    raw = static_cast<uint32_t>(static_cast<int32_t>((w ? p.absmax_q[1] : p.absmax_q[0])[e]));
    factor = (w ? p.dq_scale[1] : p.dq_scale[0])[e / kDqBlock];
  } else {
    raw = __builtin_bit_cast(uint32_t, (w ? p.absmax[1] : p.absmax[0])[e]);
  }
}
template <bool DQ>
__device__ __forceinline__ float constant_of(uint32_t raw, float factor, float mean, float inverse) {
  if constexpr (DQ) return inverse * __fadd_rn(__fmul_rn(static_cast<float>(static_cast<int32_t>(raw)), __fdiv_rn(factor, 127.0f)), mean);
  return inverse * __builtin_bit_cast(float, raw);
}

// Eight values of B's row n, adapter columns j0 .. j0 + 7: bits too.
__device__ __forceinline__ void request_b(const StreamParams &p, int up, int64_t n, int j0, uint32_t (&b)[8]) {
  const void *from = up ? p.B[1] : p.B[0];
  const int64_t at = n * p.r;
  // a column that is not there reads the last one, and its bits are dropped
  if (p.bf16) {
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = static_cast<const uint16_t *>(from)[at + min(j0 + e, p.r - 1)];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = static_cast<const uint32_t *>(from)[at + min(j0 + e, p.r - 1)];
  }
}

// acc += the adapters' terms of 32 of their columns: each weight's rows with its own half of Hs. Both halves meet all
// rows, and a lane keeps the sums of its own: rows 4 g + 0 .. 3 of the tile are the gate's for g < 2. (Rows of zeros
// in place of the other weight's would be enough but for an infinity in its half, which zeros make NaN.)
template <int MT>
__device__ __forceinline__ void adapt(f32x4 (&acc)[MT], const uint32_t (&b)[8], const u32x4 (&hs)[MT][2], const StreamParams &p, int j0, int g) {
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = j0 + e < p.r ? __builtin_bit_cast(float, p.bf16 ? b[e] << 16 : b[e]) : 0.0f;
  const bf16x8 v = __builtin_bit_cast(bf16x8, u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])});
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const f32x4 gate = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, __builtin_bit_cast(bf16x8, hs[t][0]), acc[t], 0, 0, 0);
    const f32x4 up = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, __builtin_bit_cast(bf16x8, hs[t][1]), acc[t], 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[t][e] = g < 2 ? gate[e] : up[e];
  }
}

template <int MT>
__device__ __forceinline__ void load_hs(const StreamParams &p, int row, int col, u32x4 (&hs)[MT][2]) {
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      hs[t][w] = u32x4{0, 0, 0, 0};
      if (16 * t + row < p.M) hs[t][w] = *reinterpret_cast<const u32x4 *>(p.Hs + static_cast<int64_t>(16 * t + row) * 2 * p.rp + w * p.rp + col);
    }
}

// Column n of row m of H from the waves' sums.
__device__ __forceinline__ void put_gated(const StreamParams &p, float g, float u, int m, int64_t n) {
  const int64_t at = m * p.N + n;
  p.H[at] = static_cast<__bf16>(gate_value(g, u));
  if (p.G) {
    p.G[at] = static_cast<__bf16>(g);
    p.U[at] = static_cast<__bf16>(u);
  }
}

// A load at or behind kNowhere lies past the end of every buffer here (X of at
// most 2^29 bytes, offsets within a row below 2^24) and returns zeros. Offsets
// go into the register that the bounds check looks at, none into the scalar
// one.
constexpr uint32_t kNowhere = 0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), static_cast<short>(0), static_cast<int>(bytes), 0x00020000);
}

// One row of X. A workgroup has N / 256 columns of H, one workgroup to a
// compute unit. Lane l of wave q of the W = ceil(K / 2048) that share a row of a
// weight holds X's elements 32 (64 q + l) .. + 31 in registers for the whole
// call; the 16 code bytes that meet them are one load, and a pass of the
// workgroup covers C = 8 / W columns, the gate's rows in the first C W waves and the
// other weight's in the next. A byte's two levels (bf16, out of LDS) and two
// elements of X are one v_dot2_f32_bf16, and a half block's sum takes the block's
// constant. Lanes add up sixteen passes' sums at once, halving what each holds
// by every exchange.
//
// The table has a copy for each lane, 256 bytes to an entry: an address is one
// byte permutation (code and lane), no two lanes meet in a bank, and as it lies
// at address 0 nothing is added. Constants of sixteen passes lie in memory in
// the order in which the passes use them, four to a lane and load. All loads
// are buffer loads that return zeros for what is not there, so that none is
// under a branch and waits are for no more than what is used; three passes are
// under way. 1 x 11008 x 4096: 13.3 us without adapters (k_gated_few 17.9), r =
// 64: 18.1 (23.6); 1 x 22016 x 8192 47 (60). B's rows in bf16 are requested with
// the first codes; in fp32 they are not, as the registers for them spilled others
// (19.1 us so in both).
constexpr int kRowThreads = 1024, kRowWaves = 16, kRowPasses = 16, kRowRing = 4, kRowMaxK = 16384;
struct RowLds {
  uint32_t table[256 * 64];
  float constants[2][4096];                 // [weight][column of sixteen passes][K / 64]
  uint32_t x[kRowMaxK / 2];
  float part[kRowWaves][kRowPasses + 1];
  float sums[2][kRowPasses * 8];
  uint32_t hs[2 * 256 / 2];
};

template <bool DQ>
__global__ __launch_bounds__(kRowThreads, 4) void k_gated_row(const StreamParams p, const Nf4Tables tab, int cols) {
  __shared__ __attribute__((aligned(16))) RowLds lds;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int W = static_cast<int>((p.K + 2047) / 2048), C = 8 / W;
  const int slot = wave / W, up = slot >= C, column = slot - up * C, chunk = 64 * (wave - slot * W) + lane;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * cols;
  const int count = static_cast<int>(min(p.N - c0, static_cast<int64_t>(cols)));
  const int nb = static_cast<int>(p.K / kBlock), passes = (count + C - 1) / C;
  const uint32_t row_bytes = static_cast<uint32_t>(p.K / 2);

  const auto xb = buffer_of(p.X, p.K * 2);
  const auto hb = buffer_of(p.Hs, p.r ? 4 * p.rp : 0);
  const auto cb = buffer_of((up ? p.codes[1] : p.codes[0]) + c0 * row_bytes, static_cast<int64_t>(count) * row_bytes);
  // codes of the lane's chunk, from the first pass on; past the columns nothing is there
  const bool mine = slot < 2 * C && chunk < p.K / 32;
  const uint32_t at = mine ? static_cast<uint32_t>(column) * row_bytes + 16u * static_cast<uint32_t>(chunk) : kNowhere;
  const uint32_t step = mine ? static_cast<uint32_t>(C) * row_bytes : 0;
  auto codes_of = [&](int pass) { return __builtin_amdgcn_raw_buffer_load_b128(cb, pass < passes ? at + static_cast<uint32_t>(pass) * step : kNowhere, 0, 0); };
  // four constants of each weight, of sixteen passes from column `from` on
  u32x4 raw[2];
  float factor[2] = {0.0f, 0.0f};
  auto request_constants = [&](int from) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint32_t e = static_cast<uint32_t>(from * nb + 4 * tid);
      const bool there = 4 * tid < kRowPasses * C * nb;
      if constexpr (DQ) {
        const auto b = buffer_of(p.absmax_q[w] + c0 * nb, static_cast<int64_t>(count) * nb);
        raw[w][0] = __builtin_amdgcn_raw_buffer_load_b32(b, there ? e : kNowhere, 0, 0);
        const int64_t groups = (p.N * nb + kDqBlock - 1) / kDqBlock, g = (c0 * nb + e) / kDqBlock;
        factor[w] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(buffer_of(p.dq_scale[w], 4 * groups),
                                                                                  there && e < static_cast<uint32_t>(count * nb) ? static_cast<uint32_t>(4 * g) : kNowhere, 0, 0));
      } else {
        raw[w] = __builtin_amdgcn_raw_buffer_load_b128(buffer_of(p.absmax[w] + c0 * nb, 4 * static_cast<int64_t>(count) * nb), there ? 4 * e : kNowhere, 0, 0);
      }
    }
  };
  float mean[2] = {0.0f, 0.0f};
  if constexpr (DQ) mean[0] = p.dq_mean[0][0], mean[1] = p.dq_mean[1][0];
  auto put_constants = [&]() {
    if (4 * tid >= kRowPasses * C * nb) return;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      f32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t bits = raw[w][DQ ? 0 : i];
        v[i] = constant_of<DQ>(DQ ? static_cast<uint32_t>(static_cast<int32_t>(static_cast<int8_t>(bits >> (8 * i)))) : bits, factor[w], mean[w], p.inverse);
      }
      *reinterpret_cast<f32x4 *>(&lds.constants[w][4 * tid]) = v;
    }
  };
  // the adapters' terms: four lanes share a row, of each 64 columns of B sixteen a lane
  const int side = wave >= C, in = 16 * wave + (lane >> 2) - side * kRowPasses * C, j0 = 16 * (tid & 3);
  const bool adds = wave < 2 * C;   // a row of this weight
  const bool wide = p.r % (p.bf16 ? 8 : 4) == 0;   // rows of B begin 16-byte aligned
  const auto bb = buffer_of(static_cast<const char *>(side ? p.B[1] : p.B[0]) + c0 * p.r * (p.bf16 ? 2 : 4),
                            p.r ? static_cast<int64_t>(count) * p.r * (p.bf16 ? 2 : 4) : 0);
  auto load_b = [&](int n, int j, int i) {   // 16 bytes of row n from column j on, the i-th of the lane's
    const int k = j + (p.bf16 ? 8 : 4) * i;
    return __builtin_amdgcn_raw_buffer_load_b128(bb, adds && n < count && k < p.r ? static_cast<uint32_t>((n * p.r + k) * (p.bf16 ? 2 : 4)) : kNowhere, 0, 0);
  };
  u32x4 b0[2];   // of bf16, the first 64 columns, ahead of the passes
  auto request_b = [&](int from) {
    if (wide && p.bf16 && p.r > 0) b0[0] = load_b(from + in, j0, 0), b0[1] = load_b(from + in, j0, 1);
  };

  const u32x4 x0 = __builtin_amdgcn_raw_buffer_load_b128(xb, 16 * tid, 0, 0);
  const u32x4 x1 = __builtin_amdgcn_raw_buffer_load_b128(xb, 16 * (tid + kRowThreads), 0, 0);
  request_constants(0);
  u32x4 v[kRowRing];
#pragma unroll
  for (int i = 0; i < kRowRing - 1; ++i) v[i] = codes_of(i);
  const u32x4 h0 = __builtin_amdgcn_raw_buffer_load_b128(hb, tid < 64 ? 16 * tid : kNowhere, 0, 0);
  request_b(0);
#pragma unroll
  for (int i = 0; i < 256 / kRowWaves; ++i) {
    const int e = wave + kRowWaves * i;
    lds.table[64 * e + lane] = pack_bf16x2(tab.lv[e >> 4], tab.lv[e & 15]);
  }
  *reinterpret_cast<u32x4 *>(&lds.x[4 * tid]) = x0;
  *reinterpret_cast<u32x4 *>(&lds.x[4 * (tid + kRowThreads)]) = x1;
  put_constants();
  if (tid < 64) *reinterpret_cast<u32x4 *>(&lds.hs[4 * tid]) = h0;
  __syncthreads();
  u32x4 x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const u32x4 *>(&lds.x[(16 * chunk + 4 * i) & (kRowMaxK / 2 - 1)]);
  const uint32_t copy = 4u * lane;
  const char *const table = reinterpret_cast<const char *>(lds.table);

  for (int first = 0; first < passes; first += kRowPasses) {
    float sum[kRowPasses];
    const float *c = &lds.constants[up][column * nb + (chunk >> 1)];
#pragma unroll
    for (int t = 0; t < kRowPasses; ++t) {
      sum[t] = 0.0f;
      if (first + t >= passes) continue;   // uniform
      v[(t + kRowRing - 1) % kRowRing] = codes_of(first + t + kRowRing - 1);
      const u32x4 &code = v[t % kRowRing];
      float s = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = code[q], xx = x[q][e];
          const uint32_t pair = *reinterpret_cast<const uint32_t *>(table + __builtin_amdgcn_perm(w, copy, 0x0c0c0400u + 0x100u * e));
          s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, pair), __builtin_bit_cast(bf16x2_t, xx), s, false);
        }
      sum[t] = mine ? s * c[t * C * nb] : 0.0f;
    }
    const bool more = first + kRowPasses < passes;
    if (more) request_constants((first + kRowPasses) * C);
    // lane l: pass l / 4
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const auto s = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, sum[i]), __builtin_bit_cast(uint32_t, sum[i + 8]), false, false);
      const uint32_t lo = s[0], hi = s[1];
      sum[i] = __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const auto s = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, sum[i]), __builtin_bit_cast(uint32_t, sum[i + 4]), false, false);
      const uint32_t lo = s[0], hi = s[1];
      sum[i] = __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float keep = lane & 8 ? sum[i + 2] : sum[i], send = lane & 8 ? sum[i] : sum[i + 2];
      sum[i] = keep + __shfl_xor(send, 8);
    }
    const float keep = lane & 4 ? sum[1] : sum[0], send = lane & 4 ? sum[0] : sum[1];
    float all = keep + __shfl_xor(send, 4);
    all += __shfl_xor(all, 2);
    all += __shfl_xor(all, 1);
    if ((lane & 3) == 0) lds.part[wave][lane >> 2] = all;
    __syncthreads();   // the sums; and nobody reads these constants any more
    if (more) put_constants();
    // a row's waves in order, then its adapter's terms
    const int from = first * C, n = from + in;
    if (adds) {
      float a = 0.0f;
      for (int j = j0; j < p.r; j += 64) {
        float f[16];
        if (wide && p.bf16) {
          if (j > j0) b0[0] = load_b(n, j, 0), b0[1] = load_b(n, j, 1);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const uint32_t w = b0[e >> 3][(e >> 1) & 3];
            f[e] = __builtin_bit_cast(float, e & 1 ? w & 0xffff0000u : w << 16);
          }
        } else if (wide) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const u32x4 w = load_b(n, j, i);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t bits = w[e];
              f[4 * i + e] = __builtin_bit_cast(float, bits);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            f[e] = 0.0f;
            if (n < count && j + e < p.r) {
              const int64_t i = (c0 + n) * p.r + j + e;
              const void *from_b = side ? p.B[1] : p.B[0];
              f[e] = p.bf16 ? static_cast<float>(static_cast<const __bf16 *>(from_b)[i]) : static_cast<const float *>(from_b)[i];
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const uint32_t h = lds.hs[(side * p.rp + j + e) >> 1], w = pack_bf16x2(f[e], f[e + 1]);
          a = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, w), __builtin_bit_cast(bf16x2_t, h), a, false);
        }
      }
      a += __shfl_xor(a, 1);
      a += __shfl_xor(a, 2);
      if ((tid & 3) == 0) {
        const int t = in / C, s = (side ? C : 0) + in - t * C;
        float base = 0.0f;
        for (int q = 0; q < W; ++q) base += lds.part[s * W + q][t];
        lds.sums[side][in] = base + a;
      }
    }
    if (more) request_b((first + kRowPasses) * C);
    __syncthreads();
    if (tid < kRowPasses * C && from + tid < count) put_gated(p, lds.sums[0][tid], lds.sums[1][tid], 0, c0 + from + tid);
  }
}

// Up to four rows whose X fits in LDS beside the rest. A unit is one tile of
// 16 weight rows, eight columns of H; 4096 elements of the reduction at a time,
// a wave every eighth 128 of them. X comes from LDS and not by loads of its
// own: loads return in order, and those behind the next codes' would wait for
// them (1 x 11008 x 4096 27 us so).
constexpr int kChunk = 4096, kChunkBlocks = kChunk / kBlock, kSteps = kChunk / 128 / kWaves;
constexpr int kConstantRow = 20;   // a block's constants of 16 rows: 64 lanes that write one row's lie on 16 banks
constexpr int kFewRows = 4, kFewBytes = 40 * 1024;
// Bytes between two rows of X in LDS: a step may read 64 elements behind a row, which are zero there.
inline __host__ __device__ int64_t few_row_bytes(int64_t K) { return 2 * K + 128 + 32; }

template <bool DQ>
__global__ __launch_bounds__(kThreads, 4) void k_gated_few(const StreamParams p, const Nf4Tables tab) {
  __shared__ uint32_t lut[256 * kCopies];
  __shared__ __attribute__((aligned(16))) float cs[2][kChunkBlocks][kConstantRow];
  __shared__ float part[kWaves][kFewRows][17];
  __shared__ __attribute__((aligned(16))) char xs[kFewBytes];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int r = lane & 15, g = lane >> 4;
  const int up = r >> 3;   // the lane's row is the gate's or the other weight's
  const char *const table = reinterpret_cast<const char *>(lut);
  const uint32_t copy = 4u * r;
  const int64_t row_bytes = p.K / 2, blocks = p.K / kBlock;

  // codes and raw constants of a unit's chunk; a wave has constants of one row of each weight
  u32x4 cur[kSteps], nxt[kSteps];
  uint32_t raw[2];
  float factor[2] = {0.0f, 0.0f}, mean[2] = {0.0f, 0.0f};
  const uint8_t *const codes = (up ? p.codes[1] : p.codes[0]) + (r & 7) * row_bytes + 64 * wave + 16 * g;
  auto request = [&](int unit, int chunk, u32x4 (&v)[kSteps]) {
    const int64_t first = static_cast<int64_t>(chunk) * (kChunk / 2);
    const uint8_t *at = codes + 8 * static_cast<int64_t>(unit) * row_bytes + first;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      v[i] = u32x4{0, 0, 0, 0};
      if (first + kChunk / 2 <= row_bytes || first + 64 * (kWaves * i + wave) + 16 * g < row_bytes)
        v[i] = *reinterpret_cast<const u32x4 *>(at + 64 * kWaves * i);
    }
    const int64_t b = static_cast<int64_t>(chunk) * kChunkBlocks + lane, e = (8 * static_cast<int64_t>(unit) + wave) * blocks + b;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      raw[i] = 0;
      if (b < blocks) request_constant<DQ>(p, i, e, raw[i], factor[i]);
    }
  };
  int unit = blockIdx.x, chunk = 0, turn = 0;
  request(unit, 0, cur);
  if constexpr (DQ) mean[0] = p.dq_mean[0][0], mean[1] = p.dq_mean[1][0];
  // the adapters: a wave has 32 of their columns
  const bool adapts = 32 * wave < p.r;
  uint32_t bc[8], bn[8];
  u32x4 hs[1][2];
  if (adapts) {
    request_b(p, up, 8 * static_cast<int64_t>(unit) + (r & 7), 32 * wave + 8 * g, bc);
    load_hs<1>(p, r, 32 * wave + 8 * g, hs);
  }
  const int64_t xrow = few_row_bytes(p.K);
  for (int m = 0; m < p.M; ++m)
    for (int64_t k = 8 * threadIdx.x; k < p.K + kBlock; k += 8 * kThreads)
      *reinterpret_cast<uint4 *>(xs + m * xrow + 2 * k) = k < p.K ? *reinterpret_cast<const uint4 *>(p.X + m * p.K + k) : make_uint4(0, 0, 0, 0);
  fill_table(lut, tab);
  // columns of rows that are not there are not looked at: any of X serves
  const char *const xl = xs + (r < p.M ? r : 0) * xrow + 16 * g + 256 * wave;

  f32x4 acc[1] = {f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
  while (unit < p.units) {
    float(&c)[kChunkBlocks][kConstantRow] = cs[turn & 1];
    // behind the row's end: the product with zeros, so any finite value serves
#pragma unroll
    for (int i = 0; i < 2; ++i) c[lane][8 * i + wave] = constant_of<DQ>(raw[i], factor[i], mean[i], p.inverse);
    __syncthreads();   // the constants, and in the first turn the table and X
    const bool last = chunk + 1 == p.chunks;
    const int next_unit = last ? unit + static_cast<int>(gridDim.x) : unit, next_chunk = last ? 0 : chunk + 1;
    if (next_unit < p.units) {
      request(next_unit, next_chunk, nxt);
      if (last && adapts) request_b(p, up, 8 * static_cast<int64_t>(next_unit) + (r & 7), 32 * wave + 8 * g, bn);
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int step = kWaves * i + wave;
      if (static_cast<int64_t>(chunk) * kChunk + 128 * step < p.K) {
        const char *at = xl + static_cast<int64_t>(chunk) * (2 * kChunk) + 256 * kWaves * i;
        u32x4 x[1][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) x[0][q] = *reinterpret_cast<const u32x4 *>(at + 64 * q);
        decode_step<1>(acc, cur[i], x, c[2 * step] + 4 * g, c[2 * step + 1] + 4 * g, table, copy);
      }
    }
    if (last) {
      if (adapts) {
        adapt<1>(acc, bc, hs, p, 32 * wave + 8 * g, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) bc[e] = bn[e];
      }
      // lane l holds row l % 16 of X, rows 4 g + 0 .. 3 of the unit
      if (r < kFewRows) {
#pragma unroll
        for (int e = 0; e < 4; ++e) part[wave][r][4 * g + e] = acc[0][e];
      }
      acc[0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      __syncthreads();
      if (static_cast<int>(threadIdx.x) < 8 * p.M) {
        const int m = threadIdx.x >> 3, i = threadIdx.x & 7;
        float gs = 0.0f, us = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          gs += part[w][m][i];
          us += part[w][m][8 + i];
        }
        put_gated(p, gs, us, m, 8 * static_cast<int64_t>(unit) + i);
      }
    }
    unit = next_unit;
    chunk = next_chunk;
    ++turn;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) cur[i] = nxt[i];
  }
}

// More rows, or longer ones. A unit is four tiles, 32 columns of H, which share
// the operands of X; 1024 elements of the reduction at a time, a wave 128 of
// them. Everything of the next 1024, X too, is requested before this one's are
// used, so that no wait is for part of it.
constexpr int kTiles = 4, kTurn = 128 * kWaves, kTurnBlocks = kTurn / kBlock;
constexpr int kTurnRow = 16 * kTiles + 4;

template <int MT, bool DQ>
__global__ __launch_bounds__(kThreads, MT == 1 ? 4 : 2) void k_gated_stream(const StreamParams p, const Nf4Tables tab) {
  __shared__ uint32_t lut[256 * kCopies];
  __shared__ __attribute__((aligned(16))) float cs[2][kTurnBlocks][kTurnRow];
  __shared__ float part[kWaves][MT][16][17];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int r = lane & 15, g = lane >> 4;
  const int up = r >> 3;
  const char *const table = reinterpret_cast<const char *>(lut);
  const uint32_t copy = 4u * r;
  const int64_t row_bytes = p.K / 2, blocks = p.K / kBlock;
  const int64_t unit_row = 8 * kTiles * static_cast<int64_t>(blockIdx.x);

  const __amdgpu_buffer_rsrc_t xb = buffer_of(p.X, p.M * p.K * 2);
  uint32_t xo[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) xo[t] = 16 * t + r < p.M ? static_cast<uint32_t>((16 * t + r) * p.K * 2 + 16 * g) : kNowhere;
  u32x4 cur[kTiles], nxt[kTiles], x[MT][4], xn[MT][4];
  constexpr int kRaw = 16 * kTiles * kTurnBlocks / kThreads;   // constants a thread forms
  uint32_t raw[kRaw];
  float factor[kRaw], mean[2] = {0.0f, 0.0f};
  const uint8_t *const codes = (up ? p.codes[1] : p.codes[0]) + (unit_row + (r & 7)) * row_bytes + 64 * wave + 16 * g;
  auto request = [&](int turn, u32x4 (&v)[kTiles], u32x4 (&xv)[MT][4]) {
    const int64_t first = static_cast<int64_t>(turn) * (kTurn / 2), k0 = 2 * first + 128 * wave;
    const bool there = first + 64 * wave + 16 * g < row_bytes;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      v[t] = u32x4{0, 0, 0, 0};
      if (there) v[t] = *reinterpret_cast<const u32x4 *>(codes + 8 * t * row_bytes + first);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int b = 0; b < 2; ++b) {   // a row of X ends with a block, behind it the next row begins
        const uint32_t off = k0 + 64 * b < p.K ? xo[t] + static_cast<uint32_t>(2 * k0) + 128 * b : kNowhere;
        xv[t][2 * b] = __builtin_amdgcn_raw_buffer_load_b128(xb, off, 0, 0);
        xv[t][2 * b + 1] = __builtin_amdgcn_raw_buffer_load_b128(xb, off + 64, 0, 0);
      }
#pragma unroll
    for (int i = 0; i < kRaw; ++i) {
      const int e = threadIdx.x + kThreads * i, row = e / kTurnBlocks;
      const int64_t b = static_cast<int64_t>(turn) * kTurnBlocks + e % kTurnBlocks;
      raw[i] = 0, factor[i] = 0.0f;
      if (b < blocks) request_constant<DQ>(p, (row >> 3) & 1, (unit_row + 8 * (row >> 4) + (row & 7)) * blocks + b, raw[i], factor[i]);
    }
  };
  request(0, cur, x);
  if constexpr (DQ) mean[0] = p.dq_mean[0][0], mean[1] = p.dq_mean[1][0];
  fill_table(lut, tab);
  f32x4 acc[kTiles][MT];
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int turn = 0; turn < p.chunks; ++turn) {
    float(&c)[kTurnBlocks][kTurnRow] = cs[turn & 1];
#pragma unroll
    for (int i = 0; i < kRaw; ++i) {
      const int e = threadIdx.x + kThreads * i, row = e / kTurnBlocks;
      c[e % kTurnBlocks][row] = constant_of<DQ>(raw[i], factor[i], mean[(row >> 3) & 1], p.inverse);
    }
    __syncthreads();
    if (turn + 1 < p.chunks) request(turn + 1, nxt, xn);
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
      decode_step<MT>(acc[i], cur[i], x, c[2 * wave] + 16 * i + 4 * g, c[2 * wave + 1] + 16 * i + 4 * g, table, copy);
#pragma unroll
    for (int i = 0; i < kTiles; ++i) cur[i] = nxt[i];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) x[t][q] = xn[t][q];
  }
  if (32 * wave < p.r) {
    u32x4 hs[MT][2];
    uint32_t b[kTiles][8];
    load_hs<MT>(p, r, 32 * wave + 8 * g, hs);
#pragma unroll
    for (int i = 0; i < kTiles; ++i) request_b(p, up, unit_row + 8 * i + (r & 7), 32 * wave + 8 * g, b[i]);
#pragma unroll
    for (int i = 0; i < kTiles; ++i) adapt<MT>(acc[i], b[i], hs, p, 32 * wave + 8 * g, g);
  }
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    // lane l holds row l % 16 of X, rows 4 g + 0 .. 3 of the tile
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[wave][t][r][4 * g + e] = acc[i][t][e];
    __syncthreads();
    if (threadIdx.x < 128 * MT) {
      const int t = threadIdx.x >> 7, m = (threadIdx.x >> 3) & 15, n = threadIdx.x & 7;
      if (16 * t + m < p.M) {
        float gs = 0.0f, us = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          gs += part[w][t][m][n];
          us += part[w][t][m][8 + n];
        }
        put_gated(p, gs, us, 16 * t + m, unit_row + 8 * i + n);
      }
    }
    __syncthreads();
  }
}

template <int MT, bool DQ>
void run_stream(StreamParams p, const Nf4Tables &tab, hipStream_t s) {
  p.units = static_cast<int>(p.N / (8 * kTiles));
  p.chunks = static_cast<int>(ceil_div(p.K, kTurn));
  k_gated_stream<MT, DQ><<<static_cast<unsigned>(p.units), kThreads, 0, s>>>(p, tab);
}

template <bool DQ>
void run_rows(StreamParams p, const Nf4Tables &tab, hipStream_t s) {
  if (p.M == 1 && p.K <= kRowMaxK && p.K % (4 * kBlock) == 0) {
    const int cols = static_cast<int>(ceil_div(p.N, kCus));
    k_gated_row<DQ><<<static_cast<unsigned>(ceil_div(p.N, cols)), kRowThreads, 0, s>>>(p, tab, cols);
  } else if (p.M <= kFewRows && p.M * few_row_bytes(p.K) <= kFewBytes) {
    p.units = static_cast<int>(p.N / 8);
    p.chunks = static_cast<int>(ceil_div(p.K, kChunk));
    k_gated_few<DQ><<<static_cast<unsigned>(std::min(p.units, kGatedFewGroups)), kThreads, 0, s>>>(p, tab);
  } else if (p.M <= 16) {
    run_stream<1, DQ>(p, tab, s);
  } else {
    run_stream<2, DQ>(p, tab, s);
  }
}

}  // namespace

hipError_t launch_gated_stream(const GatedArgs &a, const void *X, void *H, void *G, void *U, void *Hs, hipStream_t s) {
  const int rp = gated_padded_rank(a.r);
  if (a.r) {
    const LowParams p{static_cast<const __bf16 *>(X), {a.A[0], a.A[1]}, a.adapter_bf16, a.K, static_cast<int>(a.M), a.r, rp, a.scale, static_cast<__bf16 *>(Hs)};
    if (a.M == 1) k_gated_low<1, kLowWaves><<<2 * rp, 64 * kLowWaves, 0, s>>>(p);
    else k_gated_low<8, 4><<<dim3(2 * rp, static_cast<unsigned>(ceil_div(a.M, 8))), 256, 0, s>>>(p);
  }
  StreamParams p{};
  p.X = static_cast<const __bf16 *>(X);
  for (int w = 0; w < 2; ++w) {
    p.codes[w] = a.w[w].codes;
    p.absmax_q[w] = a.w[w].absmax_q;
    p.dq_scale[w] = a.w[w].dq_scale;
    p.dq_mean[w] = a.w[w].dq_mean;
    p.absmax[w] = a.w[w].absmax;
    p.B[w] = a.B[w];
  }
  p.Hs = static_cast<const __bf16 *>(Hs);
  p.bf16 = a.adapter_bf16;
  p.r = a.r;
  p.rp = rp;
  p.H = static_cast<__bf16 *>(H);
  p.G = static_cast<__bf16 *>(G);
  p.U = static_cast<__bf16 *>(U);
  p.N = a.N;
  p.K = a.K;
  p.M = static_cast<int>(a.M);
  const float by = level_factor(a.format);
  p.inverse = 1.0f / by;
  Nf4Tables tab = format_tables(a.format);
  for (float &level : tab.lv) level *= by;
  if (fmt_dq(a.format)) run_rows<true>(p, tab, s);
  else run_rows<false>(p, tab, s);
  return hipGetLastError();
}

}  // namespace qnf4
