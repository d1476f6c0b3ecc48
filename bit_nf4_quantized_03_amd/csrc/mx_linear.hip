// Products of microscaled operands: Y = X W^T, W in 4-bit and X in 8- or 4-bit
// floats, dense or one W per expert.
//
// The scaled matrix instruction v_mfma_scale_f32_16x16x128_f8f6f4 takes the
// codes as they are stored. Its reduction of 128 is four blocks of 32; lane l
// (g = l / 16, l % 16 the row) supplies for a 4-bit operand the 16 bytes of
// block g, for an 8-bit one 16 bytes each of blocks g / 2 and 2 + g / 2 (the
// half g % 2), and the scale byte of block g, picked from a register by a
// selector that is the same for all lanes. The sum does not care which blocks
// of the row an instruction takes, so 512 elements of a row (one 16-byte piece
// of its scales) are taken in four steps, step i using blocks 4 b + i: a lane
// then needs one 4-byte word of scales (blocks 4 g .. 4 g + 3, the selector
// counting the steps) and 64 contiguous bytes of 4-bit codes.
#include "mx_device.h"

namespace qnf4 {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

struct GemvParams {
  const uint8_t *x, *xs, *w, *ws;
  const int32_t *offsets;
  __bf16 *y;
  int64_t M, N;       // N: rows of one weight
  int64_t xrow, wrow; // bytes of a row of codes
  uint32_t nblk, pitch;
  int experts;        // 0: one weight, all rows
};

__device__ __forceinline__ uint4 load16(const uint8_t *p, bool ok) {
  return ok ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0, 0, 0, 0);
}

template <int XT, int STEP>
__device__ __forceinline__ v4f mma(const uint4 &w, const uint4 &xa, const uint4 &xb, v4f acc, int sw, int sx) {
  v8i a = {static_cast<int>(w.x), static_cast<int>(w.y), static_cast<int>(w.z), static_cast<int>(w.w), 0, 0, 0, 0};
  v8i b = {static_cast<int>(xa.x), static_cast<int>(xa.y), static_cast<int>(xa.z), static_cast<int>(xa.w),
           static_cast<int>(xb.x), static_cast<int>(xb.y), static_cast<int>(xb.z), static_cast<int>(xb.w)};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, XT == QLORA_MX_FP4 ? 4 : 0, STEP, sw, STEP, sx);
}

// A workgroup takes 16 rows of W (of one expert) and all of the expert's rows
// of X, 16 MT at a time; its WAVES waves take the 512-element pieces of the
// reduction in turn and add their sums through LDS in wave order.
template <int XT, int MT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_mx_gemv(const GemvParams p) {
  __shared__ float part[WAVES][MT][16][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  int64_t m_begin = 0, m_end = p.M;
  int64_t wbase = 0;
  if (p.experts) {
    const int e = blockIdx.y;
    m_begin = min(max(static_cast<int64_t>(p.offsets[e]), int64_t(0)), p.M);
    m_end = min(max(static_cast<int64_t>(p.offsets[e + 1]), int64_t(0)), p.M);
    wbase = static_cast<int64_t>(e) * p.N;
  }
  const int64_t n = wbase + min(n0 + r, p.N - 1);
  const uint8_t *wr = p.w + n * p.wrow;
  const uint8_t *wsr = p.ws + n * p.pitch;
  const uint32_t pieces = (p.nblk + 15) / 16;
  for (int64_t m0 = m_begin; m0 < m_end; m0 += 16 * MT) {
    v4f acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    for (uint32_t q = wave; q < pieces; q += WAVES) {
      uint4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t b = 16 * q + 4 * g + i;
        w[i] = load16(wr + static_cast<int64_t>(b) * 16, b < p.nblk);
      }
      const int sw = *reinterpret_cast<const int *>(wsr + 16 * q + 4 * g);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int64_t m = min(m0 + 16 * t + r, m_end - 1);
        const uint8_t *xr = p.x + m * p.xrow;
        uint4 xa[4], xb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (XT == QLORA_MX_FP4) {
            const uint32_t b = 16 * q + 4 * g + i;
            xa[i] = load16(xr + static_cast<int64_t>(b) * 16, b < p.nblk);
            xb[i] = make_uint4(0, 0, 0, 0);
          } else {
            const uint32_t b = 16 * q + 4 * (g >> 1) + i;
            xa[i] = load16(xr + static_cast<int64_t>(b) * 32 + 16 * (g & 1), b < p.nblk);
            xb[i] = load16(xr + static_cast<int64_t>(b + 8) * 32 + 16 * (g & 1), b + 8 < p.nblk);
          }
        }
        const int sx = *reinterpret_cast<const int *>(p.xs + m * p.pitch + 16 * q + 4 * g);
        acc[t] = mma<XT, 0>(w[0], xa[0], xb[0], acc[t], sw, sx);
        acc[t] = mma<XT, 1>(w[1], xa[1], xb[1], acc[t], sw, sx);
        acc[t] = mma<XT, 2>(w[2], xa[2], xb[2], acc[t], sw, sx);
        acc[t] = mma<XT, 3>(w[3], xa[3], xb[3], acc[t], sw, sx);
      }
    }
    // lane l holds X row l % 16 of a tile, W rows 4 (l / 16) + 0 .. 3
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) part[wave][t][r][4 * g + v] = acc[t][v];
    __syncthreads();
    for (int i = threadIdx.x; i < 256 * MT; i += 64 * WAVES) {
      const int t = i >> 8, m = (i >> 4) & 15, c = i & 15;
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < WAVES; ++k) sum += part[k][t][m][c];
      const int64_t row = m0 + 16 * t + m;
      if (row < m_end && n0 + c < p.N) p.y[row * p.N + n0 + c] = static_cast<__bf16>(sum);
    }
    __syncthreads();
  }
}

template <int XT>
hipError_t run_gemv(const GemvParams &p, hipStream_t s) {
  const dim3 g(static_cast<unsigned>(ceil_div(p.N, 16)), p.experts ? p.experts : 1);
  k_mx_gemv<XT, 2, 4><<<g, 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

size_t mx_linear_ws_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_mx_linear(const MxLinear &a, void *, hipStream_t s) {
  GemvParams p;
  p.x = a.x;
  p.xs = a.xs;
  p.w = a.w;
  p.ws = a.ws;
  p.offsets = a.offsets;
  p.y = static_cast<__bf16 *>(a.Y);
  p.M = a.M;
  p.N = a.N;
  p.xrow = mx_row_bytes(a.K, a.x_type);
  p.wrow = mx_row_bytes(a.K, QLORA_MX_FP4);
  p.nblk = static_cast<uint32_t>(a.K / kMxBlock);
  p.pitch = static_cast<uint32_t>(mx_pitch(a.K));
  p.experts = a.experts;
  return a.x_type == QLORA_MX_FP4 ? run_gemv<QLORA_MX_FP4>(p, s) : run_gemv<QLORA_MX_FP8>(p, s);
}

}  // namespace qnf4
