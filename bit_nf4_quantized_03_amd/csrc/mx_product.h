// What the kernels of microscaled products share, the plain ones (mx_linear.hip)
// and those with a gated epilogue (mx_gated.hip): the weight stream for few
// rows, and the tiles' places in the product by expert.
//
// The scaled matrix instructions take the codes as they are stored.
// v_mfma_scale_f32_16x16x128_f8f6f4 (few rows; mx_gemm.h has the larger one)
// reduces over four blocks of 32; lane l (g = l / 16, l % 16 the row) supplies
// for a 4-bit operand the 16 bytes of block g, for an 8-bit one 16 bytes each
// of blocks g / 2 and 2 + g / 2 (the half g % 2), and the scale byte of block
// g. The four lanes of a row so read 64 contiguous bytes. A row's 16-byte piece
// of scales serves four instructions, 512 elements.
#pragma once

#include "mx_gemm.h"
#include "mx_tiles.h"

namespace qnf4 {

typedef float mx_v4f __attribute__((ext_vector_type(4)));

struct MxGemvParams {
  const uint8_t *x, *xs, *w, *ws;
  const int32_t *offsets;
  int64_t M, N;       // N: rows of one weight
  int64_t xrow, wrow; // bytes of a row of codes
  uint32_t nblk, pitch;
  int experts;        // 0: one weight, all rows
};

// 16 bytes at p, zeros where the block lies behind the row's end.
__device__ __forceinline__ mx_v4i mx_load16(const uint8_t *p, bool ok) {
  return ok ? *reinterpret_cast<const mx_v4i *>(p) : mx_v4i{0, 0, 0, 0};
}

// Rows of X of expert e, clamped to X; none where its end lies before its start.
__device__ __forceinline__ void mx_expert_rows(const int32_t *offsets, int experts, int64_t M, int e, int64_t &b, int64_t &end) {
  b = end = 0;
  if (e >= experts) return;
  b = min(max(static_cast<int64_t>(offsets[e]), int64_t(0)), M);
  end = max(min(max(static_cast<int64_t>(offsets[e + 1]), int64_t(0)), M), b);
}

// Finds number `t` among the pieces that `count(b, end)` gives each expert's
// rows, expert after expert: the expert, its rows and the number within it.
// False where there are fewer. The lanes count 64 experts at a time.
template <class F>
__device__ __forceinline__ bool mx_find_piece(const int32_t *offsets, int experts, int64_t M, int &t, int &expert, int64_t &b,
                                           int64_t &end, F count) {
  const int lane = threadIdx.x & 63;
  for (int e0 = 0; e0 < experts; e0 += 64) {
    int64_t lb, lend;
    mx_expert_rows(offsets, experts, M, e0 + lane, lb, lend);
    const int n = count(lb, lend);
    int upto = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(upto, o);
      if (lane >= o) upto += v;
    }
    const uint64_t here = __ballot(t < upto);
    if (here == 0) {
      t = __builtin_amdgcn_readfirstlane(t - __shfl(upto, 63));
      continue;
    }
    const int l = __ffsll(static_cast<unsigned long long>(here)) - 1;
    t = __builtin_amdgcn_readfirstlane(t - __shfl(upto - n, l));
    expert = __builtin_amdgcn_readfirstlane(e0 + l);
    b = mx_uniform(__shfl(lb, l));
    end = mx_uniform(__shfl(lend, l));
    return true;
  }
  return false;
}

// A workgroup takes 16 RT rows of W and up to 16 MT rows of X: all of them,
// or by expert 16 of the expert's. Its WAVES waves take the 512-element pieces
// of the reduction in turn; their sums are in `part` once the workgroup has
// passed a barrier, to be added in wave order. Rows [m0, m_end) of X are the
// workgroup's; false where it has none.
//
// By expert blockIdx.y < experts is an expert and its first 16 rows; the
// numbers behind them are the further runs of 16 of the experts that have
// them, found from the offsets: an expert with many rows has as many
// workgroups (512 rows of one expert among 64: 57 us; by the workgroups of its
// first 16 rows in turn 160).
template <int XT, int MT, int RT, int WAVES>
__device__ __forceinline__ bool mx_stream(const MxGemvParams &p, float (&part)[WAVES][MT][RT][16][17], int64_t &m0,
                                          int64_t &m_end) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * RT);
  m0 = 0, m_end = p.M;
  int64_t wbase = 0;
  if (p.experts) {
    int e = blockIdx.y;
    if (e < p.experts) {
      mx_expert_rows(p.offsets, p.experts, p.M, e, m0, m_end);
    } else {
      int piece = e - p.experts;
      const auto further = [](int64_t b, int64_t end) { return end > b ? static_cast<int>((end - b - 1) >> 4) : 0; };
      if (!mx_find_piece(p.offsets, p.experts, p.M, piece, e, m0, m_end, further)) return false;
      m0 += 16 * (piece + 1);
    }
    if (m0 >= m_end) return false;
    m_end = min(m_end, m0 + 16);
    wbase = static_cast<int64_t>(e) * p.N;
  }
  const uint8_t *wr[RT], *wsr[RT];
#pragma unroll
  for (int k = 0; k < RT; ++k) {
    const int64_t n = wbase + min(n0 + 16 * k + r, p.N - 1);
    wr[k] = p.w + n * p.wrow + 16 * g;
    wsr[k] = p.ws + n * p.pitch;
  }
  const uint32_t pieces = (p.nblk + 15) / 16;
  mx_v4f acc[MT][RT];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int k = 0; k < RT; ++k) acc[t][k] = mx_v4f{0.0f, 0.0f, 0.0f, 0.0f};
  for (uint32_t q = wave; q < pieces; q += WAVES) {
    mx_v4i w[RT][4], sw[RT];
#pragma unroll
    for (int k = 0; k < RT; ++k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[k][i] = mx_load16(wr[k] + 256 * q + 64 * i, 16 * q + 4 * i + g < p.nblk);
      sw[k] = *reinterpret_cast<const mx_v4i *>(wsr[k] + 16 * q);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      // lanes of rows that are not there load nothing: with one row a
      // sixteenth of a load's addresses (1 x 4096 x 11008 7.7 -> 7.0 us)
      const bool on = m0 + 16 * t + r < m_end;
      const int64_t m = min(m0 + 16 * t + r, m_end - 1);
      const uint8_t *xr = p.x + m * p.xrow + 16 * g;
      mx_v8i x[4];
      const mx_v4i sx = *reinterpret_cast<const mx_v4i *>(p.xs + m * p.pitch + 16 * q);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (XT == QLORA_MX_FP4) {
          x[i] = mx_operand(mx_load16(xr + 256 * q + 64 * i, on && 16 * q + 4 * i + g < p.nblk));
        } else {
          const uint32_t b = 16 * q + 4 * i + (g >> 1);
          x[i] = mx_operand(mx_load16(xr + 512 * q + 128 * i, on && b < p.nblk),
                            mx_load16(xr + 512 * q + 128 * i + 64, on && b + 2 < p.nblk));
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int si = static_cast<int>(static_cast<uint32_t>(sx[i]) >> (8 * g));
#pragma unroll
        for (int k = 0; k < RT; ++k)
          acc[t][k] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              mx_operand(w[k][i]), x[i], acc[t][k], 4, XT == QLORA_MX_FP4 ? 4 : 0, 0,
              static_cast<int>(static_cast<uint32_t>(sw[k][i]) >> (8 * g)), 0, si);
      }
    }
  }
  // lane l holds X row l % 16 of a tile, W rows 4 (l / 16) + 0 .. 3
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int k = 0; k < RT; ++k)
#pragma unroll
      for (int v = 0; v < 4; ++v) part[wave][t][k][r][4 * g + v] = acc[t][k][v];
  return true;
}

struct MxGemmParams {
  MxOperands op;
  const int32_t *offsets;
  int64_t M, N;
  int steps;      // of 128 elements
  int experts;
};

// Tile of a workgroup in the product by expert. Tiles are counted expert after
// expert; each XCD takes a contiguous range of them (consecutive workgroups go
// to the XCDs in turn). Every wave finds its tile by itself.
struct MxGroupTile {
  int expert, tm, tn;
  int64_t m_begin, m_end;
};

template <class T>
__device__ __forceinline__ bool mx_group_tile(const MxGemmParams &p, int bid, MxGroupTile &out) {
  const int lane = threadIdx.x & 63;
  const int tiles_n = static_cast<int>((p.N + T::BN - 1) / T::BN);
  const auto tiles = [=](int64_t b, int64_t end) { return static_cast<int>((end - b + T::BM - 1) / T::BM) * tiles_n; };
  int total = 0;
  for (int e0 = 0; e0 < p.experts; e0 += 64) {
    int64_t b, end;
    mx_expert_rows(p.offsets, p.experts, p.M, e0 + lane, b, end);
    total += tiles(b, end);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o);
  if (bid >= total) return false;
  const int base = total / 8, extra = total % 8, x = bid % 8;
  int t = x * base + min(x, extra) + bid / 8;
  if (!mx_find_piece(p.offsets, p.experts, p.M, t, out.expert, out.m_begin, out.m_end, tiles)) return false;
  // within the expert: groups of four tile rows, as tile_of
  const int tiles_m = static_cast<int>((out.m_end - out.m_begin + T::BM - 1) / T::BM);
  const int group = t / (4 * tiles_n), first = 4 * group, gm = min(tiles_m - first, 4), in = t - group * 4 * tiles_n;
  out.tm = first + in % gm;
  out.tn = in / gm;
  return true;
}

// The kernels' arguments from the call's (its Y apart).
inline void mx_product_params(const MxLinear &a, MxGemvParams &p, MxGemmParams &q) {
  p.x = a.x;
  p.xs = a.xs;
  p.w = a.w;
  p.ws = a.ws;
  p.offsets = a.offsets;
  p.M = a.M;
  p.N = a.N;
  p.xrow = mx_row_bytes(a.K, a.x_type);
  p.wrow = mx_row_bytes(a.K, QLORA_MX_FP4);
  p.nblk = static_cast<uint32_t>(a.K / kMxBlock);
  p.pitch = static_cast<uint32_t>(mx_pitch(a.K));
  p.experts = a.experts;
  q.op = {a.x, a.xs, a.w, a.ws, a.M, a.N, p.xrow, p.wrow, p.pitch};
  q.offsets = a.offsets;
  q.M = a.M;
  q.N = a.N;
  q.steps = static_cast<int>(ceil_div(a.K, 128));
  q.experts = a.experts;
}

}  // namespace qnf4
