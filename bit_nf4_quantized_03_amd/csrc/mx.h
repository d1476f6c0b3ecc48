// Private declarations of the microscaled kernels and of RMSNorm, shared by
// their C-ABI layer (api_mx.cpp) and their translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <cstddef>
#include <cstdint>

#include "../../include/qlora_mx.h"
#include "internal.h"

namespace qnf4 {

constexpr int kMxBlock = QLORA_MX_BLOCK;

// A launch holds fewer than 2^32 threads: longer runs go out in pieces of this
// many workgroups (of at most 1024 threads).
constexpr int64_t kMaxGroups = int64_t(1) << 21;

inline int64_t mx_pitch(int64_t cols) { return 16 * ceil_div(cols, 512); }
inline int64_t mx_row_bytes(int64_t cols, int type) { return type == QLORA_MX_FP4 ? cols / 2 : cols; }

hipError_t launch_mx_quantize(const void *X, bool x_bf16, int64_t rows, int64_t cols, int type, uint8_t *codes,
                              uint8_t *scales, hipStream_t s);
hipError_t launch_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols, int type,
                                void *out, bool out_bf16, hipStream_t s);

// Y: bf16 [rows, cols] where `codes` is null, else codes and scales of `type`.
struct RmsFwd {
  const void *X, *residual, *weight;
  bool w_bf16;
  int64_t rows, cols;
  double eps;
  void *Y;
  uint8_t *codes, *scales;
  int type;
  void *H;
  float *rstd;
};
constexpr int64_t kRmsMaxCols = 32768;
hipError_t launch_rms_fwd(const RmsFwd &a, hipStream_t s);
size_t rms_bwd_ws_bytes(int64_t rows, int64_t cols);
hipError_t launch_rms_bwd(const void *dY, const void *H, const void *weight, bool w_bf16, const float *rstd,
                          const void *dH, int64_t rows, int64_t cols, void *dX, float *dW, void *ws, hipStream_t s);

// experts = 0: one product for all M rows, offsets unused.
struct MxLinear {
  int64_t M, N, K;
  int x_type;
  const uint8_t *x, *xs;   // codes and scales
  const uint8_t *w, *ws;
  const int32_t *offsets;
  int experts;
  void *Y;
};
constexpr int64_t kMxMaxK = int64_t(1) << 22;
// What keeps a product's launch below 2^32 threads, with the weight stream and
// with the tile that the rule of mx_tiles.h chooses.
constexpr int64_t kMxMaxRows = int64_t(1) << 24, kMxMaxExpertRows = int64_t(1) << 28, kMxMaxOut = int64_t(1) << 37;
hipError_t launch_mx_linear(const MxLinear &a, hipStream_t s);

}  // namespace qnf4
