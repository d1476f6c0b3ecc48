// The gated feed-forward product on microscaled operands, dense or by expert,
// and the pair of weights that it reads.
#include <algorithm>
#include <cmath>

#include "block.h"
#include "mx_gated.h"

namespace qnf4 {
namespace {

// Rows of a pair: 16-byte pieces of a row's codes and scales, one wave a row.
struct PairParams {
  const uint8_t *codes[2], *scales[2];   // gate, up
  uint8_t *to_codes, *to_scales;
  int64_t first, rows;                   // rows of the pair that the launch begins with / that there are
  int64_t ld, pitch;
};

__global__ __launch_bounds__(256) void k_mx_pair(const PairParams p) {
  const int64_t row = p.first + 4 * static_cast<int64_t>(blockIdx.x) + (threadIdx.x >> 6);
  if (row >= p.rows) return;
  const int up = static_cast<int>(row >> 3) & 1;
  const int64_t from = (row >> 4) * 8 + (row & 7);
  const uint8_t *c = p.codes[up] + from * p.ld, *s = p.scales[up] + from * p.pitch;
  uint8_t *to = p.to_codes + row * p.ld, *ts = p.to_scales + row * p.pitch;
  for (int64_t i = 16 * (threadIdx.x & 63); i < p.ld; i += 1024) *reinterpret_cast<uint4 *>(to + i) = *reinterpret_cast<const uint4 *>(c + i);
  for (int64_t i = 16 * (threadIdx.x & 63); i < p.pitch; i += 1024) *reinterpret_cast<uint4 *>(ts + i) = *reinterpret_cast<const uint4 *>(s + i);
}

// Zeros in the rows of H in front of the first expert's and behind the last
// one's, by workgroup `part` of `parts`. These are workgroups of the product's own
// launch behind its others (a fill in front of 4096 rows over 8 experts 4096 x
// 4096 took 8 us).
__device__ __forceinline__ void clear_rest(const MxGatedOut &o, const int32_t *offsets, int experts, int64_t M, int part, int parts) {
  const int64_t first = min(max(static_cast<int64_t>(offsets[0]), int64_t(0)), M);
  const int64_t last = max(min(max(static_cast<int64_t>(offsets[experts]), int64_t(0)), M), first);
  const int64_t rows = M - (last - first);
  const auto clear = [&](void *to, int64_t bytes) {   // of a row, a multiple of 16
    const int64_t runs = bytes / 16;
    for (int64_t i = static_cast<int64_t>(part) * blockDim.x + threadIdx.x; i < rows * runs; i += static_cast<int64_t>(parts) * blockDim.x) {
      const int64_t k = i / runs, row = k < first ? k : k + (last - first);
      *reinterpret_cast<uint4 *>(static_cast<char *>(to) + row * bytes + 16 * (i - k * runs)) = make_uint4(0, 0, 0, 0);
    }
  };
  if (o.type < 0) return clear(o.h, 2 * o.N);
  clear(o.codes, o.type == QLORA_MX_FP4 ? o.N / 2 : o.N);
  clear(o.scales, o.pitch);
}
constexpr int kClearGroups = 64;

// Few rows: 16 RT rows of the pair, 8 RT columns of H a workgroup. The waves'
// sums are added in wave order, then a lane takes eight columns of a row.
template <int XT, int MT, int RT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_mx_gated_gemv(const MxGemvParams p, const MxGatedOut o) {
  __shared__ float part[WAVES][MT][RT][16][17];
  int64_t m0, m_end;
  if (!mx_stream<XT, MT, RT, WAVES>(p, part, m0, m_end)) {
    // the last row of workgroups has no piece
    if (o.clear && blockIdx.y + 1 == gridDim.y) clear_rest(o, p.offsets, p.experts, p.M, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
    return;
  }
  const int rows = static_cast<int>(min(m_end - m0, int64_t(16 * MT)));
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * RT * rows; i += 64 * WAVES) {
    const int c = i & 15, k = (i >> 4) % RT, m = (i >> 4) / RT;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += part[w][m >> 4][k][m & 15][c];
    part[0][m >> 4][k][m & 15][c] = sum;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < RT * rows; i += 64 * WAVES) {
    const int k = i % RT, m = i / RT;
    const float *both = part[0][m >> 4][k][m & 15];
    float v[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = gate_value(both[c], both[8 + c]);
    const int64_t n = static_cast<int64_t>(blockIdx.x) * (8 * RT) + 8 * k;
    mx_gated_put(o, v, m0 + m, n, n < o.N);
  }
}

// Tile number b of those of rows n_first on of the pair, tiles_n of them beside each other.
template <class T>
__device__ __forceinline__ void gated_tile(const MxGemmParams &p, const MxGatedOut &o, int b, int64_t n_first, int tiles_n, char *smem) {
  int tm, tn, wave;
  tile_of(b, static_cast<int>((p.M + T::BM - 1) / T::BM), tiles_n, tm, tn);
  const int64_t n0 = n_first + static_cast<int64_t>(tn) * T::BN, m0 = static_cast<int64_t>(tm) * T::BM;
  MxAcc<T> acc;
  const bool mine = mx_tile_product<T>(acc, p.op, n0, m0, p.steps, smem, wave);
  mx_gated_store<T>(acc, o, n0, m0, p.M, wave, mine, smem);
}

template <class T>
__global__ __launch_bounds__(T::kThreads, 1) void k_mx_gated(const MxGemmParams p, const MxGatedOut o) {
  __shared__ __attribute__((aligned(16))) char smem[T::kLds];
  gated_tile<T>(p, o, static_cast<int>(blockIdx.x), 0, static_cast<int>((p.N + T::BN - 1) / T::BN), smem);
}

// Large tiles, n_tiles beside each other, and smaller ones for the rows of the
// pair behind them.
template <class T, class S>
__global__ __launch_bounds__(T::kThreads, 1) void k_mx_gated_two(const MxGemmParams p, const MxGatedOut o, int n_tiles) {
  static_assert(T::kThreads == S::kThreads, "one launch");
  __shared__ __attribute__((aligned(16))) char smem[T::kLds > S::kLds ? T::kLds : S::kLds];
  const int large = n_tiles * static_cast<int>((p.M + T::BM - 1) / T::BM), b = static_cast<int>(blockIdx.x);
  const int64_t first = static_cast<int64_t>(n_tiles) * T::BN;
  if (b < large) gated_tile<T>(p, o, b, 0, n_tiles, smem);
  else gated_tile<S>(p, o, b - large, first, static_cast<int>((p.N - first + S::BN - 1) / S::BN), smem);
}

template <class T>
__global__ __launch_bounds__(T::kThreads, 1) void k_mx_gated_grouped(const MxGemmParams p, const MxGatedOut o) {
  __shared__ __attribute__((aligned(16))) char smem[T::kLds];
  MxGroupTile t;
  if (!mx_group_tile<T>(p, static_cast<int>(blockIdx.x), t)) {
    const int part = static_cast<int>(blockIdx.x + kClearGroups) - static_cast<int>(gridDim.x);
    if (o.clear && part >= 0) clear_rest(o, p.offsets, p.experts, p.M, part, kClearGroups);
    return;
  }
  const int64_t n0 = static_cast<int64_t>(t.tn) * T::BN;
  const int64_t m0 = t.m_begin + static_cast<int64_t>(t.tm) * T::BM;
  MxOperands op = p.op;
  op.w += static_cast<int64_t>(t.expert) * p.N * op.w_ld;
  op.ws += static_cast<int64_t>(t.expert) * p.N * op.pitch;
  op.x_rows = t.m_end;
  MxAcc<T> acc;
  int wave;
  const bool mine = mx_tile_product<T>(acc, op, n0, m0, p.steps, smem, wave);
  mx_gated_store<T>(acc, o, n0, m0, t.m_end, wave, mine, smem);
}

template <int XT, int MT, int RT, int WAVES>
hipError_t run_gemv(const MxGemvParams &p, const MxGatedOut &o, hipStream_t s) {
  // by expert: every run of 16 rows but an expert's first is a whole one or follows one
  const dim3 g(static_cast<unsigned>(ceil_div(p.N, 16 * RT)), p.experts ? p.experts + static_cast<unsigned>(p.M / 16) + o.clear : 1);
  k_mx_gated_gemv<XT, MT, RT, WAVES><<<g, 64 * WAVES, 0, s>>>(p, o);
  return hipGetLastError();
}

template <int TILE, class T>
hipError_t run_tile(const MxGemmParams &p, const MxGatedOut &o, hipStream_t s) {
  static_assert(T::BN == kMxTile[TILE].bn && T::BM == kMxTile[TILE].bm && T::kThreads == kMxTile[TILE].threads, "the rule's tile");
  const unsigned groups = static_cast<unsigned>(mx_tile_groups(T::BM, T::BN, p.M, p.N, p.experts));
  if (p.experts) k_mx_gated_grouped<T><<<groups + (o.clear ? kClearGroups : 0), T::kThreads, 0, s>>>(p, o);
  else k_mx_gated<T><<<groups, T::kThreads, 0, s>>>(p, o);
  return hipGetLastError();
}

// The N tiles of kMxTile[0] in front of smaller ones, kMxTile[1], or 0: all are
// of one kind. Large tiles come in rounds of one for each compute unit, and a
// last round that is not full costs as much as any; the smaller tiles halve it
// where that is less by the figures that choose the tile (4096 x 11008 x 4096,
// 1376 large tiles in six rounds: 293 us, 279 with 96 of them as 192 smaller
// ones; 2500 rows 188 and 180; 2048 x 22016 x 8192, 4 bits, 375 and 368).
int large_tiles(int64_t M, int64_t N, bool fp4) {
  const double tiles_m = static_cast<double>(mx_ceil(M, kMxTile[0].bm)), tiles_n = static_cast<double>(mx_ceil(N, kMxTile[0].bn));
  const double rounds = std::floor(tiles_m * tiles_n / kMxCus), n = std::floor(rounds * kMxCus / tiles_m);
  if (n < 1 || n >= tiles_n) return 0;
  const auto &c = kMxTile[1].cost[fp4];
  const double load = static_cast<double>(mx_ceil(M, kMxTile[1].bm)) * (tiles_n - n) * kMxTile[0].bn / kMxTile[1].bn / kMxCus;
  const double rest = load <= 1 ? c.light + (c.full - c.light) * load : c.full * std::ceil(load);
  return rest < kMxTile[0].cost[fp4].full ? static_cast<int>(n) : 0;
}

template <class T, class S>
hipError_t run_two(const MxGemmParams &p, const MxGatedOut &o, int n_tiles, hipStream_t s) {
  const int64_t rest = mx_tile_groups(S::BM, S::BN, p.M, p.N - static_cast<int64_t>(n_tiles) * T::BN, 0);
  k_mx_gated_two<T, S><<<static_cast<unsigned>(n_tiles * mx_ceil(p.M, T::BM) + rest), T::kThreads, 0, s>>>(p, o, n_tiles);
  return hipGetLastError();
}

template <int XT>
hipError_t run_tiles(const MxGemmParams &p, const MxGatedOut &o, hipStream_t s) {
  constexpr bool kPair = XT == QLORA_MX_FP4;
  constexpr int kDeep = kPair ? 4 : 3;   // stages
  using Large = MxTile<XT, 4, 2, 2, 4, kDeep, kPair ? 2 : 1, 1, kPair>;
  using Half = MxTile<XT, 2, 2, 4, 2, kDeep, kPair ? 2 : 4, 1, kPair>;
  switch (mx_choose_tile(p.M, p.N, p.experts, kPair)) {
    case 0: {
      const int n = p.experts ? 0 : large_tiles(p.M, p.N, kPair);
      return n ? run_two<Large, Half>(p, o, n, s) : run_tile<0, Large>(p, o, s);
    }
    case 1: return run_tile<1, Half>(p, o, s);
    case 2: return run_tile<2, MxTile<XT, 2, 2, 2, 2, kDeep, kPair ? 2 : 1, 1, kPair>>(p, o, s);
    case 3: return run_tile<3, MxTile<XT, 2, 1, 2, 2, 4, 2>>(p, o, s);
    default: return run_tile<4, MxTile<XT, 1, 1, 2, 2, 4, 4, 2>>(p, o, s);
  }
}

// Few rows, the weight's stream: false where the tiles are faster. A workgroup
// has 64 rows of the pair, the 32 columns of one block of a microscaled H. A
// bf16 H has no such blocks: half as many rows, eight waves, where that loads
// the compute units more evenly (1 row, 4096 elements: 4096 columns 8.2 us with
// 64 rows, 6.3 with 32, 6.6 with 16; 11008 15.7, 13.1, 15.4; 8 rows of 11008
// 17.2, 14.8, 19.1; but 5504 8.3, 9.0, 8.9 and 8192 columns of 8192 elements
// 19.0, 19.5, 18.9). Sixteen waves are slower with 32 rows (11008 16.6 us).
template <int XT>
bool run_few_rows(const MxGemvParams &p, const MxGatedOut &o, hipStream_t s, hipError_t *e) {
  if (p.experts) {
    if (p.M > 8 * static_cast<int64_t>(p.experts)) return false;
    *e = p.nblk <= 32 ? run_gemv<XT, 1, 4, 2>(p, o, s) : run_gemv<XT, 1, 4, 4>(p, o, s);
    return true;
  }
  if (p.M > (p.N <= 32 * kMxCus ? 16 : 8)) return false;
  const auto uneven = [&](int rows) {
    const double load = static_cast<double>(ceil_div(p.N, rows)) / kMxCus;
    return std::ceil(load) / load;
  };
  if (o.type < 0 && uneven(64) > 1.15 * uneven(32)) *e = run_gemv<XT, 1, 2, 8>(p, o, s);
  else *e = p.N <= 64 * kMxCus ? run_gemv<XT, 1, 4, 8>(p, o, s) : run_gemv<XT, 1, 4, 4>(p, o, s);
  return true;
}

template <int XT>
hipError_t run_gated(const MxLinear &a, const MxGatedOut &o, hipStream_t s) {
  MxGemvParams p;
  MxGemmParams q;
  mx_product_params(a, p, q);
  hipError_t e;
  return run_few_rows<XT>(p, o, s, &e) ? e : run_tiles<XT>(q, o, s);
}

}  // namespace

hipError_t launch_mx_pair(const MxPair &a, hipStream_t s) {
  PairParams p{{a.gate, a.up}, {a.gate_scales, a.up_scales}, a.out, a.out_scales, 0, a.rows, a.K / 2, mx_pitch(a.K)};
  for (; p.first < a.rows; p.first += 4 * kMaxGroups) {
    const int64_t groups = std::min(ceil_div(a.rows - p.first, 4), kMaxGroups);
    k_mx_pair<<<static_cast<unsigned>(groups), 256, 0, s>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_mx_gated(const MxLinear &a, uint8_t *codes, uint8_t *scales, int type, bool clear, hipStream_t s) {
  MxGatedOut o;
  o.h = static_cast<__bf16 *>(a.Y);
  o.codes = codes;
  o.scales = scales;
  o.N = a.N / 2;
  o.pitch = static_cast<uint32_t>(mx_pitch(o.N));
  o.type = a.Y ? -1 : type;
  o.clear = clear;
  return a.x_type == QLORA_MX_FP4 ? run_gated<QLORA_MX_FP4>(a, o, s) : run_gated<QLORA_MX_FP8>(a, o, s);
}

}  // namespace qnf4
