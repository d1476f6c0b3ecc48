// Products of microscaled operands: Y = X W^T, W in 4-bit and X in 8- or 4-bit
// floats, dense or one W per expert.
//
// The scaled matrix instructions take the codes as they are stored.
// v_mfma_scale_f32_16x16x128_f8f6f4 (few rows; mx_gemm.h has the larger one)
// reduces over four blocks of 32; lane l (g = l / 16, l % 16 the row) supplies
// for a 4-bit operand the 16 bytes of block g, for an 8-bit one 16 bytes each
// of blocks g / 2 and 2 + g / 2 (the half g % 2), and the scale byte of block
// g. The four lanes of a row so read 64 contiguous bytes. A row's 16-byte piece
// of scales serves four instructions, 512 elements.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "mx_gemm.h"
#include "mx_tiles.h"

namespace qnf4 {
namespace {

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

// 16 bytes at p, zeros where the block lies behind the row's end.
__device__ __forceinline__ mx_v4i load16(const uint8_t *p, bool ok) {
  return ok ? *reinterpret_cast<const mx_v4i *>(p) : mx_v4i{0, 0, 0, 0};
}

// Rows of X of expert e, clamped to X; none where its end lies before its start.
__device__ __forceinline__ void expert_rows(const int32_t *offsets, int experts, int64_t M, int e, int64_t &b, int64_t &end) {
  b = end = 0;
  if (e >= experts) return;
  b = min(max(static_cast<int64_t>(offsets[e]), int64_t(0)), M);
  end = max(min(max(static_cast<int64_t>(offsets[e + 1]), int64_t(0)), M), b);
}

// Finds number `t` among the pieces that `count(b, end)` gives each expert's
// rows, expert after expert: the expert, its rows and the number within it.
// False where there are fewer. The lanes count 64 experts at a time.
template <class F>
__device__ __forceinline__ bool find_piece(const int32_t *offsets, int experts, int64_t M, int &t, int &expert, int64_t &b,
                                           int64_t &end, F count) {
  const int lane = threadIdx.x & 63;
  for (int e0 = 0; e0 < experts; e0 += 64) {
    int64_t lb, lend;
    expert_rows(offsets, experts, M, e0 + lane, lb, lend);
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
// of the reduction in turn and add their sums through LDS in wave order.
//
// By expert blockIdx.y < experts is an expert and its first 16 rows; the
// numbers behind them are the further runs of 16 of the experts that have
// them, found from the offsets: an expert with many rows has as many
// workgroups (512 rows of one expert among 64: 57 us; by the workgroups of its
// first 16 rows in turn 160).
//
// Bound by the weight's bytes: 1 x 11008 x 4096 8.2 us (2.9 TB/s: one load's
// round trip for each wave, then the sums), 33 rows over eight 11008 x 4096
// 32 us (5.5 TB/s of the weights that have a row), 64 over 64 4096 x 4096 98 us
// (5.8 TB/s).
template <int XT, int MT, int RT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_mx_gemv(const GemvParams p) {
  __shared__ float part[WAVES][MT][RT][16][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * RT);
  int64_t m0 = 0, m_end = p.M;
  int64_t wbase = 0;
  if (p.experts) {
    int e = blockIdx.y;
    if (e < p.experts) {
      expert_rows(p.offsets, p.experts, p.M, e, m0, m_end);
    } else {
      int piece = e - p.experts;
      const auto further = [](int64_t b, int64_t end) { return end > b ? static_cast<int>((end - b - 1) >> 4) : 0; };
      if (!find_piece(p.offsets, p.experts, p.M, piece, e, m0, m_end, further)) return;
      m0 += 16 * (piece + 1);
    }
    if (m0 >= m_end) return;
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
  v4f acc[MT][RT];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int k = 0; k < RT; ++k) acc[t][k] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  for (uint32_t q = wave; q < pieces; q += WAVES) {
    mx_v4i w[RT][4], sw[RT];
#pragma unroll
    for (int k = 0; k < RT; ++k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[k][i] = load16(wr[k] + 256 * q + 64 * i, 16 * q + 4 * i + g < p.nblk);
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
          x[i] = mx_operand(load16(xr + 256 * q + 64 * i, on && 16 * q + 4 * i + g < p.nblk));
        } else {
          const uint32_t b = 16 * q + 4 * i + (g >> 1);
          x[i] = mx_operand(load16(xr + 512 * q + 128 * i, on && b < p.nblk),
                            load16(xr + 512 * q + 128 * i + 64, on && b + 2 < p.nblk));
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
  __syncthreads();
  for (int i = threadIdx.x; i < 256 * MT * RT; i += 64 * WAVES) {
    const int c = i & 15, k = (i >> 4) % RT, m = (i >> 4) / RT & 15, t = (i >> 8) / RT;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += part[w][t][k][m][c];
    const int64_t row = m0 + 16 * t + m, n = n0 + 16 * k + c;
    if (row < m_end && n < p.N) p.y[row * p.N + n] = static_cast<__bf16>(sum);
  }
}

// ---------------------------------------------------------------- large tiles

struct GemmParams {
  MxOperands op;
  const int32_t *offsets;
  __bf16 *y;
  int64_t M, N;
  int steps;      // of 128 elements
  int experts;
};

template <class T>
__global__ __launch_bounds__(T::kThreads, 1) void k_mx_gemm(const GemmParams p) {
  __shared__ __attribute__((aligned(16))) char smem[T::kLds];
  const int tiles_m = static_cast<int>((p.M + T::BM - 1) / T::BM), tiles_n = static_cast<int>((p.N + T::BN - 1) / T::BN);
  int tm, tn, wave;
  tile_of(static_cast<int>(blockIdx.x), tiles_m, tiles_n, tm, tn);
  const int64_t n0 = static_cast<int64_t>(tn) * T::BN, m0 = static_cast<int64_t>(tm) * T::BM;
  MxAcc<T> acc;
  if (mx_tile_product<T>(acc, p.op, n0, m0, p.steps, smem, wave)) mx_store<T>(acc, p.y, p.N, n0, m0, p.M, wave, smem);
}

// Tile of a workgroup in the product by expert. Tiles are counted expert after
// expert; each XCD takes a contiguous range of them (consecutive workgroups go
// to the XCDs in turn). Every wave finds its tile by itself.
struct GroupTile {
  int expert, tm, tn;
  int64_t m_begin, m_end;
};

template <class T>
__device__ __forceinline__ bool group_tile(const GemmParams &p, int bid, GroupTile &out) {
  const int lane = threadIdx.x & 63;
  const int tiles_n = static_cast<int>((p.N + T::BN - 1) / T::BN);
  const auto tiles = [=](int64_t b, int64_t end) { return static_cast<int>((end - b + T::BM - 1) / T::BM) * tiles_n; };
  int total = 0;
  for (int e0 = 0; e0 < p.experts; e0 += 64) {
    int64_t b, end;
    expert_rows(p.offsets, p.experts, p.M, e0 + lane, b, end);
    total += tiles(b, end);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o);
  if (bid >= total) return false;
  const int base = total / 8, extra = total % 8, x = bid % 8;
  int t = x * base + min(x, extra) + bid / 8;
  if (!find_piece(p.offsets, p.experts, p.M, t, out.expert, out.m_begin, out.m_end, tiles)) return false;
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
  int wave;
  if (mx_tile_product<T>(acc, op, n0, m0, p.steps, smem, wave)) mx_store<T>(acc, p.y, p.N, n0, m0, t.m_end, wave, smem);
}

template <int XT, int MT, int RT, int WAVES>
hipError_t run_gemv(const GemvParams &p, hipStream_t s) {
  // by expert: every run of 16 rows but an expert's first is a whole one or follows one
  const dim3 g(static_cast<unsigned>(ceil_div(p.N, 16 * RT)), p.experts ? p.experts + static_cast<unsigned>(p.M / 16) : 1);
  k_mx_gemv<XT, MT, RT, WAVES><<<g, 64 * WAVES, 0, s>>>(p);
  return hipGetLastError();
}

template <int TILE, class T>
hipError_t run_gemm(const GemmParams &p, hipStream_t s) {
  static_assert(T::BN == kMxTile[TILE].bn && T::BM == kMxTile[TILE].bm && T::kThreads == kMxTile[TILE].threads, "the rule's tile");
  const unsigned groups = static_cast<unsigned>(mx_tile_groups(T::BM, T::BN, p.M, p.N, p.experts));
  if (p.experts) k_mx_gemm_grouped<T><<<groups, T::kThreads, 0, s>>>(p);
  else k_mx_gemm<T><<<groups, T::kThreads, 0, s>>>(p);
  return hipGetLastError();
}

template <int XT>
hipError_t run_tiles(const GemmParams &p, hipStream_t s) {
  constexpr bool kPair = XT == QLORA_MX_FP4;
  constexpr int kDeep = kPair ? 4 : 3;   // stages
  switch (mx_choose_tile(p.M, p.N, p.experts, XT == QLORA_MX_FP4)) {
    case 0: return run_gemm<0, MxTile<XT, 4, 2, 2, 4, kDeep, kPair ? 2 : 1, 1, kPair>>(p, s);
    case 1: return run_gemm<1, MxTile<XT, 2, 2, 4, 2, kDeep, kPair ? 2 : 4, 1, kPair>>(p, s);
    case 2: return run_gemm<2, MxTile<XT, 2, 2, 2, 2, kDeep, kPair ? 2 : 1, 1, kPair>>(p, s);
    case 3: return run_gemm<3, MxTile<XT, 2, 1, 2, 2, 4, 2>>(p, s);
    default: return run_gemm<4, MxTile<XT, 1, 1, 2, 2, 4, 4, 2>>(p, s);
  }
}

// Few rows: the matrix core's work does not matter, the weight's stream does.
// X is read by every workgroup, so a workgroup takes as many rows of W, 64, 32
// or 16, as leave the compute units about as evenly loaded as the next fewer
// would (the factors are between what 40000 and 28672, 4096 and 18432 rows of W
// ask for): `uneven` is the time of the fullest unit over the average (8 rows of X,
// K = 4096, 64 / 32 / 16 rows of W: N = 4096 8.4, 6.2, 5.7 us; 6144 8.6, 6.5,
// 7.6; 11008 8.8, 10.2, 10.5; 22016 16.5, 13.9, 17.9). Eight waves share the
// reduction, four where units have two workgroups or more (32000 17.6 us
// against 18.9).
//
// By expert 64 rows and four waves (one row for each of 64 4096 x 4096: 98 us,
// 5.8 TB/s, against 104 with 32 rows of W and 107 with 128; four for each of
// eight 11008 x 4096: 39.5, 40.4 and 48), two where the reduction has no more
// than two pieces (4096 x 1024, 16 experts of 4 rows: 9.9 against 11.2).
//
// Returns false where the tiles are faster (K = 4096, stream against tiles): N
// = 4096 from 25 rows on (24: 7.4 against 8.2 us, 32: 8.2 each), N = 8192 from
// 17 (16: 7.5 against 8.4, 24: 9.1 against 8.5), more from 9 (8 x 22016 13.8
// each, 16 x 22016 16.3 against 14.1), by expert from 9 on average on (64 4096 x
// 4096: 8 rows 108 to 113 us against 118 with 128 x 64 tiles, 16 rows 126 to
// 162 against 120 to 124).
template <int XT>
bool run_few_rows(const GemvParams &p, hipStream_t s, hipError_t *e) {
  if (p.experts) {
    if (p.M > 8 * static_cast<int64_t>(p.experts)) return false;
    *e = p.nblk <= 32 ? run_gemv<XT, 1, 4, 2>(p, s) : run_gemv<XT, 1, 4, 4>(p, s);
    return true;
  }
  const auto uneven = [&](int rows) {
    const double load = static_cast<double>(ceil_div(p.N, rows)) / kMxCus;
    return std::ceil(load) / load;
  };
  if (p.M > (p.N <= 16 * kMxCus ? 24 : p.N <= 32 * kMxCus ? 16 : 8)) return false;
  const int rows = p.M > 16 ? 16 : uneven(64) <= 1.15 * uneven(32) ? 64 : uneven(32) <= 1.25 * uneven(16) ? 32 : 16;
  if (rows == 64) *e = p.N <= 64 * kMxCus ? run_gemv<XT, 1, 4, 8>(p, s) : run_gemv<XT, 1, 4, 4>(p, s);
  else if (rows == 32) *e = run_gemv<XT, 1, 2, 8>(p, s);
  else *e = p.M > 16 ? run_gemv<XT, 2, 1, 8>(p, s) : run_gemv<XT, 1, 1, 8>(p, s);
  return true;
}

template <int XT>
hipError_t run_product(const GemvParams &p, const GemmParams &q, hipStream_t s) {
  hipError_t e;
  return run_few_rows<XT>(p, s, &e) ? e : run_tiles<XT>(q, s);
}

}  // namespace

hipError_t launch_mx_linear(const MxLinear &a, hipStream_t s) {
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
  GemmParams q;
  q.op = {a.x, a.xs, a.w, a.ws, a.M, a.N, p.xrow, p.wrow, p.pitch};
  q.offsets = a.offsets;
  q.y = p.y;
  q.M = a.M;
  q.N = a.N;
  q.steps = static_cast<int>(ceil_div(a.K, 128));
  q.experts = a.experts;
  return a.x_type == QLORA_MX_FP4 ? run_product<QLORA_MX_FP4>(p, q, s) : run_product<QLORA_MX_FP8>(p, q, s);
}

}  // namespace qnf4
