// Private declarations of what stands between a decoder layer's projections,
// shared by their C-ABI layer (api_block.cpp) and their translation units.
#pragma once

#include "mx.h"

namespace qnf4 {

// rows: those of the pair
struct MxPair {
  const uint8_t *gate, *gate_scales, *up, *up_scales;
  uint8_t *out, *out_scales;
  int64_t rows, K;
};
hipError_t launch_mx_pair(const MxPair &a, hipStream_t s);

// a.N: rows of one pair. H is a.Y in bf16, or codes and scales of `type` where
// that is null. clear: by expert, rows that no expert has become zeros.
hipError_t launch_mx_gated(const MxLinear &a, uint8_t *codes, uint8_t *scales, int type, bool clear, hipStream_t s);

// Heads [rows][heads][dim], the elements of a head next to each other; strides
// in elements. No heads: not there.
struct RopeHeads {
  const void *in;
  void *out;
  int64_t heads, in_row, in_head, out_row, out_head;
};
struct Rope {
  RopeHeads q, k;
  bool bf16;
  int64_t rows;
  int dim, rot;
  const void *positions;
  bool wide_positions;   // int64, else int32
  const double *freqs;   // [rot / 2]
  double amplitude;
  bool interleaved, backward;
};
constexpr int kRopeMaxDim = 1024;
constexpr int64_t kRopeMaxHeads = 1 << 15;   // of q and k together
hipError_t launch_rope(const Rope &a, hipStream_t s);

// The gated block around two 4-bit weights [N, K] of one format, gate first;
// adapters A [r, K], B [N, r] of each, or r = 0.
struct GatedWeight {
  const uint8_t *codes;
  const int8_t *absmax_q;   // with DQ
  const float *dq_scale, *dq_mean;
  const float *absmax;      // without
};
struct GatedArgs {
  int64_t M, N, K;
  int format, r;
  float scale;
  bool adapter_bf16;
  GatedWeight w[2];
  const void *A[2], *B[2];
};
// Adapter columns in Hs and in the kernels' operands.
inline int gated_padded_rank(int r) { return static_cast<int>(ceil_div(r, 64) * 64); }
constexpr int64_t kGatedMaxRows = int64_t(1) << 24, kGatedMaxDim = int64_t(1) << 23, kGatedMaxOut = int64_t(1) << 36;
size_t gated_ws_bytes(int64_t M, int64_t N, int64_t K, int r, bool backward);
// The forward of at most kGatedStreamRows rows; Hs [M][2 padded rank] as above (r > 0).
constexpr int64_t kGatedStreamRows = 32;
constexpr int kGatedFewGroups = 512;
hipError_t launch_gated_stream(const GatedArgs &a, const void *X, void *H, void *G, void *U, void *Hs, hipStream_t s);
// G, U, Hs: kept for the backward, or null.
hipError_t launch_gated_fwd(const GatedArgs &a, const void *X, void *H, void *G, void *U, void *Hs, void *ws, hipStream_t s);
hipError_t launch_gated_bwd(const GatedArgs &a, const void *dH, const void *X, const void *G, const void *U, const void *Hs,
                            void *dX, void *const (&dA)[2], void *const (&dB)[2], void *ws, hipStream_t s);

}  // namespace qnf4
