// What the kernels of the gated product write, and the pair of weights that
// they read.
//
// H = silu(X Wg^T) * (X Wu^T), silu(g) = g / (1 + e^-g). The two weights [N, K]
// lie in one matrix of 2 N rows, eight rows of the gate and eight of the other
// one in turn: row 16 j + t is gate row 8 j + t, row 16 j + 8 + t the other
// one's. A tile of any height that is a multiple of 16 then holds both
// products of its columns of H, and in the layout in which the matrix
// instructions leave them (a lane has four consecutive rows of W of every
// eight) both of a column are in one lane: the product needs no exchange and
// the kernels of mx_gemm.h and mx_product.h run unchanged on a matrix of 2 N
// rows.
#pragma once

#include "gate.h"
#include "mx_product.h"

namespace qnf4 {

struct MxGatedOut {
  __bf16 *h;               // type < 0
  uint8_t *codes, *scales; // else: of that qlora_mx_type
  int64_t N;               // columns of H, a multiple of 32
  uint32_t pitch;
  int type;
  bool clear;              // by expert: zeros in the rows that no expert has
};

// Columns n .. n + 7 of row m. Microscaled: the four lanes of a quad hold one
// block of 32 and all of them are here; `on` says whether to store.
template <int TYPE>
__device__ __forceinline__ void mx_gated_block(const MxGatedOut &o, const float (&v)[8], int64_t m, int64_t n, bool on) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu);
  const uint32_t scale = mx_scale_byte<TYPE>(quad_max(amax));
  const uint2 codes = mx_encode8<TYPE>(v, mx_scale_value(scale));
  if (!on) return;
  if constexpr (TYPE == QLORA_MX_FP4) *reinterpret_cast<uint32_t *>(o.codes + m * (o.N >> 1) + (n >> 1)) = codes.x;
  else *reinterpret_cast<uint2 *>(o.codes + m * o.N + n) = codes;
  if ((threadIdx.x & 3) == 0) {
    uint8_t *s = o.scales + m * o.pitch;
    const uint32_t b = static_cast<uint32_t>(n >> 5), blocks = static_cast<uint32_t>(o.N >> 5);
    s[b] = static_cast<uint8_t>(scale);
    if (b == blocks - 1)
      for (uint32_t i = blocks; i < o.pitch; ++i) s[i] = 0;
  }
}

__device__ __forceinline__ void mx_gated_put(const MxGatedOut &o, const float (&v)[8], int64_t m, int64_t n, bool on) {
  if (o.type < 0) {
    if (on)
      *reinterpret_cast<uint4 *>(o.h + m * o.N + n) =
          make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else if (o.type == QLORA_MX_FP4) {
    mx_gated_block<QLORA_MX_FP4>(o, v, m, n, on);
  } else {
    mx_gated_block<QLORA_MX_FP8>(o, v, m, n, on);
  }
}

// The tile's part of H from the accumulators of its 2 N rows: values of 32 rows
// of X at a time through LDS, in fp32 (a block's scale needs all of its 32
// columns before any is rounded), and out as whole runs of a row. A wave has
// 16 NF columns; with NF = 1 the two waves of the same rows of X share a place
// and half of its rows each, which is why every wave of the workgroup comes here
// (`mine`: this one has sums). `smem` is free from kSums on.
template <class T>
__device__ __forceinline__ void mx_gated_store(const MxAcc<T> &acc, const MxGatedOut &o, int64_t n0, int64_t m0,
                                               int64_t m_end, int wave, bool mine, char *smem) {
  constexpr bool kShared = T::NF == 1;
  constexpr int kCols = kShared ? 32 : 16 * T::NF, kRow = 4 * kCols + 16, kLanes = kCols / 8, kRows = 64 / kLanes;
  static_assert(!kShared || (T::WN == 2 && T::MF == 1), "two waves to a block of 32 columns");
  static_assert(T::kSums + (kShared ? T::WM : T::kWaves) * 32 * kRow <= T::kLds, "places fit the rings");
  const int lane = threadIdx.x & 63;
  const int wn = wave / T::WM, wm = wave % T::WM;
  const int64_t c0 = (n0 >> 1) + (kShared ? 0 : kCols * wn);
  m0 += 32 * T::MF * wm;
  char *place = smem + T::kSums + (kShared ? wm : wave) * 32 * kRow;
#pragma unroll
  for (int j = 0; j < T::MF; ++j) {
    if (mine) {
#pragma unroll
      for (int i = 0; i < T::NF; ++i)
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          const f32x16 &v = acc.v[i][j];
          float h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = gate_value(v[4 * q + e], v[4 * q + 4 + e]);
          *reinterpret_cast<float4 *>(place + (lane & 31) * kRow + 64 * i + (kShared ? 64 * wn : 0) + 16 * q + 16 * (lane >> 5)) =
              make_float4(h[0], h[1], h[2], h[3]);
        }
    }
    if constexpr (kShared) __syncthreads();
    else mx_wave_order();
    if (mine) {
#pragma unroll
      for (int k = 0; k < (kShared ? 16 : 32) / kRows; ++k) {
        const int r = (kShared ? 16 * wn : 0) + kRows * k + lane / kLanes;
        const char *at = place + r * kRow + 32 * (lane % kLanes);
        const float4 a = *reinterpret_cast<const float4 *>(at), b = *reinterpret_cast<const float4 *>(at + 16);
        const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        const int64_t m = m0 + 32 * j + r, n = c0 + 8 * (lane % kLanes);
        mx_gated_put(o, v, m, n, m < m_end && n < o.N);
      }
    }
    if constexpr (!kShared) mx_wave_order();   // the next rows take the place
  }
}

}  // namespace qnf4
