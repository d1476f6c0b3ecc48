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
// that is null.
hipError_t launch_mx_gated(const MxLinear &a, uint8_t *codes, uint8_t *scales, int type, hipStream_t s);

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

}  // namespace qnf4
