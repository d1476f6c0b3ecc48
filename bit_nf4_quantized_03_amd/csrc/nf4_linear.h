// What the QLoRA linear layer (linear.hip) and the gated feed-forward block
// around two of them (gated.hip) share: the level table in LDS, sums of split
// partials, how a reduction is split, and workspace regions.
#pragma once

#include <algorithm>

#include "gemm_big.h"

namespace qnf4 {

// LDS table of level pairs for every code byte: (level[b >> 4], level[b & 15]),
// kLvCopies interleaved copies; returns this lane's copy.
__device__ __forceinline__ const float2 *load_level_pairs(float2 *lv2, const Nf4Tables &tab) {
  for (int i = threadIdx.x; i < 256 * kLvCopies; i += blockDim.x) {
    const int b = i / kLvCopies;
    lv2[i] = make_float2(tab.lv[b >> 4], tab.lv[b & 15]);
  }
  return lv2 + (threadIdx.x & (kLvCopies - 1));
}

// sum_z part[z * plane + e] for z = 0 .. splits - 1, added in that order; the
// loads go out eight at a time (clamped indices, the extra terms dropped), so
// the sum costs a few memory round trips instead of one per split.
__device__ __forceinline__ float split_sum(const float *part, int64_t plane, int64_t e, int splits) {
  float v = 0.0f;
  for (int z0 = 0; z0 < splits; z0 += 8) {
    float t[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) t[u] = part[static_cast<int64_t>(min(z0 + u, splits - 1)) * plane + e];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (z0 + u < splits) v += t[u];
  }
  return v;
}

// The same sum for four consecutive elements (16-byte loads).
__device__ __forceinline__ float4 split_sum4(const float *part, int64_t plane, int64_t e, int splits) {
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int z0 = 0; z0 < splits; z0 += 8) {
    float4 t[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      t[u] = *reinterpret_cast<const float4 *>(part + static_cast<int64_t>(min(z0 + u, splits - 1)) * plane + e);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (z0 + u < splits) {
        v.x += t[u].x;
        v.y += t[u].y;
        v.z += t[u].z;
        v.w += t[u].w;
      }
  }
  return v;
}

constexpr int kTargetGroups = 512;

inline int64_t grid_blocks(int64_t n, int64_t b) { return ceil_div(n, b); }

struct Split {
  int splits;
  int steps_per_split;
};

// Split `steps` reduction steps so that tiles * splits reaches the target.
inline Split choose_split(int64_t tiles, int steps, int max_splits, int target = kTargetGroups) {
  int want = static_cast<int>(ceil_div(target, tiles > 0 ? tiles : 1));
  want = std::max(1, std::min({want, steps, max_splits}));
  const int per = static_cast<int>(ceil_div(steps, want));
  return {static_cast<int>(ceil_div(steps, per)), per};
}

// Workspace carve-out: sequential 256-byte-aligned regions.
struct Carve {
  char *base;
  size_t off = 0;
  template <class T>
  T *take(size_t count) {
    T *p = reinterpret_cast<T *>(base ? base + off : nullptr);
    off = align_up(off + count * sizeof(T), 256);
    return p;
  }
};

constexpr int kCus = 256;                             // compute units of the GPU
constexpr int kMinSplitSteps = 4;                     // 64-deep steps per split at least
constexpr size_t kSplitPartMax = size_t(128) << 20;   // bytes of fp32 partials at most

// Reduction splits of a large-tile GEMM with `tiles` 256 x 256 output tiles
// of an M x cols output over `steps` 64-deep steps: none while the tiles fill
// half the GPU or more; otherwise as many as keep every workgroup in one
// round on the compute units, each split at least kMinSplitSteps long.
inline Split gemm_split(int64_t tiles, int steps, int64_t M, int64_t cols, bool allow) {
  int S = 1;
  if (allow && tiles * 2 <= kCus) {
    S = static_cast<int>(std::min<int64_t>(kCus / tiles, steps / kMinSplitSteps));
    while (S > 1 && static_cast<size_t>(S) * M * cols * sizeof(float) > kSplitPartMax) --S;
    S = std::max(S, 1);
  }
  const int per = static_cast<int>(ceil_div(steps, S));
  return {static_cast<int>(ceil_div(steps, per)), per};
}

}  // namespace qnf4
