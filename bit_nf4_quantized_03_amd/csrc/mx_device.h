// Device helpers of the microscaled formats.
#pragma once

#include "mx.h"

namespace qnf4 {

typedef short mx_short2 __attribute__((ext_vector_type(2)));
typedef __bf16 mx_bf16x2 __attribute__((ext_vector_type(2)));
typedef float mx_float2 __attribute__((ext_vector_type(2)));
typedef uint32_t mx_u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t mx_u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xffff0000u); }

// The larger of v over the four lanes of a quad (a block of 32 elements lies
// in one quad, eight elements to a lane).
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 0xF, 0xF, false)));
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x4E, 0xF, 0xF, false)));
}

// Scale byte of a block from the fp32 bits of its largest magnitude: the
// biased exponent less that of the element type's largest power of two, 255
// where the block holds a NaN or an Inf. (A subnormal magnitude has biased
// exponent 0 and its byte is 0 as the definition's clamp makes it.)
template <int TYPE>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  constexpr uint32_t top = TYPE == QLORA_MX_FP4 ? 2 : 8;
  const uint32_t e = amax_bits >> 23;
  return e >= 255u ? 255u : (e > top ? e - top : 0u);
}

// 2^(s - 127) as fp32 (s = 0 is the subnormal 2^-127, s = 255 NaN).
__device__ __forceinline__ float mx_scale_value(uint32_t s) {
  return __builtin_bit_cast(float, s == 0 ? 0x00400000u : s == 255 ? 0x7fc00000u : s << 23);
}

// Eight fp32 values over 2^(s - 127) as codes: 4 bytes (4 bits, in .x) or 8.
// The conversions divide by the scale and round to nearest even; the 4-bit one
// saturates, the 8-bit one turns what rounds past 448 into NaN, so its input
// is clamped first (448 * 2^(s - 127) is exact and finite for every s that a
// finite block has).
template <int TYPE>
__device__ __forceinline__ uint2 mx_encode8(const float (&v)[8], float scale) {
  uint2 r = make_uint2(0, 0);
  if constexpr (TYPE == QLORA_MX_FP4) {
    r.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r.x, v[0], v[1], scale, 0);
    r.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r.x, v[2], v[3], scale, 1);
    r.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r.x, v[4], v[5], scale, 2);
    r.x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r.x, v[6], v[7], scale, 3);
  } else {
    const float lim = 448.0f * scale;
    float c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = __builtin_amdgcn_fmed3f(v[i], -lim, lim);
    mx_short2 a = {0, 0}, b = {0, 0};
    a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, c[0], c[1], scale, 0);
    a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, c[2], c[3], scale, 1);
    b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, c[4], c[5], scale, 0);
    b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, c[6], c[7], scale, 1);
    r.x = __builtin_bit_cast(uint32_t, a);
    r.y = __builtin_bit_cast(uint32_t, b);
  }
  return r;
}

// Row and place in the row of the blocks b0 + j (j < span) of a matrix with
// nblk blocks a row; b0 is the same in the whole wave, so that the one 64-bit
// division is too.
struct MxRows {
  int64_t row0;
  uint32_t c0, nblk;
  bool wide;   // at most one row end among the span's blocks
  __device__ MxRows(int64_t b0, uint32_t nblk_, uint32_t span) : nblk(nblk_) {
    if ((b0 >> 32) == 0) row0 = static_cast<uint32_t>(b0) / nblk;
    else row0 = b0 / nblk;
    c0 = static_cast<uint32_t>(b0 - row0 * nblk);
    wide = nblk >= span;
  }
  __device__ __forceinline__ void at(uint32_t j, int64_t &row, uint32_t &c) const {
    c = c0 + j;
    uint32_t d;
    if (wide) d = c >= nblk ? 1u : 0u;
    else d = c / nblk;
    c -= d * nblk;
    row = row0 + d;
  }
};

}  // namespace qnf4
