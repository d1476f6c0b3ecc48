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
#include <type_traits>

#include "mx_gemm.h"

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

// ---------------------------------------------------------------- large tiles

struct GemmParams {
  MxOperands op;
  const int32_t *offsets;
  __bf16 *y;
  int64_t M, N;
  int steps, experts;
};

template <class T>
__global__ __launch_bounds__(T::kThreads, 1) void k_mx_gemm(const GemmParams p) {
  __shared__ __attribute__((aligned(16))) char smem[T::kLds];
  const int tiles_m = static_cast<int>((p.M + T::BM - 1) / T::BM), tiles_n = static_cast<int>((p.N + T::BN - 1) / T::BN);
  int tm, tn;
  tile_of(static_cast<int>(blockIdx.x), tiles_m, tiles_n, tm, tn);
  const int64_t n0 = static_cast<int64_t>(tn) * T::BN, m0 = static_cast<int64_t>(tm) * T::BM;
  MxAcc<T> acc;
#pragma unroll
  for (int i = 0; i < T::NF; ++i)
#pragma unroll
    for (int j = 0; j < T::MF; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc.v[i][j][e] = 0.0f;
  mx_mainloop<T>(acc, p.op, n0, m0, 0, p.steps, smem);
  mx_store<T>(acc, p.y, p.N, n0, m0, p.M);
}

// Tile of a workgroup in the product by expert. Tiles are counted expert after
// expert; each XCD takes a contiguous range of them (consecutive workgroups go
// to the XCDs in turn). Every wave finds its tile by itself: the lanes count
// the tiles of 64 experts at a time.
struct GroupTile {
  int expert, tm, tn;
  int64_t m_begin, m_end;
};

__device__ __forceinline__ int expert_tiles(const GemmParams &p, int e, int bm, int tiles_n, int64_t &b, int64_t &end) {
  b = end = 0;
  if (e >= p.experts) return 0;
  b = min(max(static_cast<int64_t>(p.offsets[e]), int64_t(0)), p.M);
  end = min(max(static_cast<int64_t>(p.offsets[e + 1]), int64_t(0)), p.M);
  return end > b ? static_cast<int>((end - b + bm - 1) / bm) * tiles_n : 0;
}

template <class T>
__device__ __forceinline__ bool group_tile(const GemmParams &p, int bid, GroupTile &out) {
  const int lane = threadIdx.x & 63;
  const int tiles_n = static_cast<int>((p.N + T::BN - 1) / T::BN);
  int64_t b, end;
  int total = 0;
  for (int e0 = 0; e0 < p.experts; e0 += 64) total += expert_tiles(p, e0 + lane, T::BM, tiles_n, b, end);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o);
  if (bid >= total) return false;
  const int base = total / 8, extra = total % 8, x = bid % 8;
  int t = x * base + min(x, extra) + bid / 8;
  for (int e0 = 0;; e0 += 64) {
    const int n = expert_tiles(p, e0 + lane, T::BM, tiles_n, b, end);
    int upto = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(upto, o);
      if (lane >= o) upto += v;
    }
    const uint64_t here = __ballot(t < upto);
    if (here == 0) {
      t -= __shfl(upto, 63);
      continue;   // ends: t is below the sum over all experts
    }
    const int l = __ffsll(static_cast<unsigned long long>(here)) - 1;
    t -= __shfl(upto - n, l);
    out.expert = __builtin_amdgcn_readfirstlane(e0 + l);
    out.m_begin = mx_uniform(__shfl(b, l));
    out.m_end = mx_uniform(__shfl(end, l));
    break;
  }
  t = __builtin_amdgcn_readfirstlane(t);
  // within the expert: groups of four tile rows, as tile_of
  const int tiles_m = static_cast<int>((out.m_end - out.m_begin + T::BM - 1) / T::BM);
  const int group = t / (4 * tiles_n), first = 4 * group, gm = min(tiles_m - first, 4), in = t - group * 4 * tiles_n;
  out.tm = first + in % gm;
  out.tn = in / gm;
  return true;
}

template <class T>
__global__ __launch_bounds__(T::kThreads, 1) void k_mx_gemm_grouped(const GemmParams p) {
  __shared__ __attribute__((aligned(16))) char smem[T::kLds];
  GroupTile t;
  if (!group_tile<T>(p, static_cast<int>(blockIdx.x), t)) return;
  const int64_t n0 = static_cast<int64_t>(t.tn) * T::BN;
  const int64_t m0 = t.m_begin + static_cast<int64_t>(t.tm) * T::BM;
  MxOperands op = p.op;
  op.w += static_cast<int64_t>(t.expert) * p.N * op.w_ld;
  op.ws += static_cast<int64_t>(t.expert) * p.N * op.pitch;
  op.x_rows = t.m_end;
  MxAcc<T> acc;
#pragma unroll
  for (int i = 0; i < T::NF; ++i)
#pragma unroll
    for (int j = 0; j < T::MF; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc.v[i][j][e] = 0.0f;
  mx_mainloop<T>(acc, op, n0, m0, 0, p.steps, smem);
  mx_store<T>(acc, p.y, p.N, n0, m0, t.m_end);
}

template <int XT>
hipError_t run_gemv(const GemvParams &p, hipStream_t s) {
  const dim3 g(static_cast<unsigned>(ceil_div(p.N, 16)), p.experts ? p.experts : 1);
  k_mx_gemv<XT, 2, 4><<<g, 256, 0, s>>>(p);
  return hipGetLastError();
}

template <class T>
hipError_t run_gemm(const GemmParams &p, hipStream_t s) {
  const int64_t tiles_n = ceil_div(p.N, T::BN);
  if (p.experts) {
    // an expert's rows end in at most one partial tile
    const int64_t most = (p.M / T::BM + p.experts) * tiles_n;
    k_mx_gemm_grouped<T><<<static_cast<unsigned>(most), T::kThreads, 0, s>>>(p);
  } else {
    k_mx_gemm<T><<<static_cast<unsigned>(ceil_div(p.M, T::BM) * tiles_n), T::kThreads, 0, s>>>(p);
  }
  return hipGetLastError();
}

template <int XT>
hipError_t run_gemm_any(const GemmParams &p, hipStream_t s) {
  using Big = MxTile<XT, 4, 2, 2, 4, 3>;
  using Mid = MxTile<XT, 2, 2, 2, 2, 3>;
  const int64_t rows = p.experts ? p.M / p.experts : p.M;
  if (rows >= 256) return run_gemm<Big>(p, s);
  return run_gemm<Mid>(p, s);
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
  const int64_t rows = a.experts ? a.M / a.experts : a.M;   // of one weight, on average
  if (rows <= 32) return a.x_type == QLORA_MX_FP4 ? run_gemv<QLORA_MX_FP4>(p, s) : run_gemv<QLORA_MX_FP8>(p, s);
  GemmParams q;
  q.op = {a.x, a.xs, a.w, a.ws, a.M, a.N, p.xrow, p.wrow, p.pitch};
  q.offsets = a.offsets;
  q.y = p.y;
  q.M = a.M;
  q.N = a.N;
  q.steps = static_cast<int>(ceil_div(a.K, 128));
  q.experts = a.experts;
  return a.x_type == QLORA_MX_FP4 ? run_gemm_any<QLORA_MX_FP4>(q, s) : run_gemm_any<QLORA_MX_FP8>(q, s);
}

}  // namespace qnf4
