// Products of microscaled operands: Y = X W^T, W in 4-bit and X in 8- or 4-bit
// floats, dense or one W per expert.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "mx_product.h"

namespace qnf4 {
namespace {

// Few rows: the sums of mx_stream, added in wave order.
//
// Bound by the weight's bytes: 1 x 11008 x 4096 8.2 us (2.9 TB/s: one load's
// round trip for each wave, then the sums), 33 rows over eight 11008 x 4096
// 32 us (5.5 TB/s of the weights that have a row), 64 over 64 4096 x 4096 98 us
// (5.8 TB/s).
template <int XT, int MT, int RT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_mx_gemv(const MxGemvParams p, __bf16 *y) {
  __shared__ float part[WAVES][MT][RT][16][17];
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * RT);
  int64_t m0, m_end;
  if (!mx_stream<XT, MT, RT, WAVES>(p, part, m0, m_end)) return;
  __syncthreads();
  for (int i = threadIdx.x; i < 256 * MT * RT; i += 64 * WAVES) {
    const int c = i & 15, k = (i >> 4) % RT, m = (i >> 4) / RT & 15, t = (i >> 8) / RT;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += part[w][t][k][m][c];
    const int64_t row = m0 + 16 * t + m, n = n0 + 16 * k + c;
    if (row < m_end && n < p.N) y[row * p.N + n] = static_cast<__bf16>(sum);
  }
}

// ---------------------------------------------------------------- large tiles

template <class T>
__global__ __launch_bounds__(T::kThreads, 1) void k_mx_gemm(const MxGemmParams p, __bf16 *y) {
  __shared__ __attribute__((aligned(16))) char smem[T::kLds];
  const int tiles_m = static_cast<int>((p.M + T::BM - 1) / T::BM), tiles_n = static_cast<int>((p.N + T::BN - 1) / T::BN);
  int tm, tn, wave;
  tile_of(static_cast<int>(blockIdx.x), tiles_m, tiles_n, tm, tn);
  const int64_t n0 = static_cast<int64_t>(tn) * T::BN, m0 = static_cast<int64_t>(tm) * T::BM;
  MxAcc<T> acc;
  if (mx_tile_product<T>(acc, p.op, n0, m0, p.steps, smem, wave)) mx_store<T>(acc, y, p.N, n0, m0, p.M, wave, smem);
}

template <class T>
__global__ __launch_bounds__(T::kThreads, 1) void k_mx_gemm_grouped(const MxGemmParams p, __bf16 *y) {
  __shared__ __attribute__((aligned(16))) char smem[T::kLds];
  MxGroupTile t;
  if (!mx_group_tile<T>(p, static_cast<int>(blockIdx.x), t)) return;
  const int64_t n0 = static_cast<int64_t>(t.tn) * T::BN;
  const int64_t m0 = t.m_begin + static_cast<int64_t>(t.tm) * T::BM;
  MxOperands op = p.op;
  op.w += static_cast<int64_t>(t.expert) * p.N * op.w_ld;
  op.ws += static_cast<int64_t>(t.expert) * p.N * op.pitch;
  op.x_rows = t.m_end;
  MxAcc<T> acc;
  int wave;
  if (mx_tile_product<T>(acc, op, n0, m0, p.steps, smem, wave)) mx_store<T>(acc, y, p.N, n0, m0, t.m_end, wave, smem);
}

template <int XT, int MT, int RT, int WAVES>
hipError_t run_gemv(const MxGemvParams &p, __bf16 *y, hipStream_t s) {
  // by expert: every run of 16 rows but an expert's first is a whole one or follows one
  const dim3 g(static_cast<unsigned>(ceil_div(p.N, 16 * RT)), p.experts ? p.experts + static_cast<unsigned>(p.M / 16) : 1);
  k_mx_gemv<XT, MT, RT, WAVES><<<g, 64 * WAVES, 0, s>>>(p, y);
  return hipGetLastError();
}

template <int TILE, class T>
hipError_t run_gemm(const MxGemmParams &p, __bf16 *y, hipStream_t s) {
  static_assert(T::BN == kMxTile[TILE].bn && T::BM == kMxTile[TILE].bm && T::kThreads == kMxTile[TILE].threads, "the rule's tile");
  const unsigned groups = static_cast<unsigned>(mx_tile_groups(T::BM, T::BN, p.M, p.N, p.experts));
  if (p.experts) k_mx_gemm_grouped<T><<<groups, T::kThreads, 0, s>>>(p, y);
  else k_mx_gemm<T><<<groups, T::kThreads, 0, s>>>(p, y);
  return hipGetLastError();
}

template <int XT>
hipError_t run_tiles(const MxGemmParams &p, __bf16 *y, hipStream_t s) {
  constexpr bool kPair = XT == QLORA_MX_FP4;
  constexpr int kDeep = kPair ? 4 : 3;   // stages
  switch (mx_choose_tile(p.M, p.N, p.experts, XT == QLORA_MX_FP4)) {
    case 0: return run_gemm<0, MxTile<XT, 4, 2, 2, 4, kDeep, kPair ? 2 : 1, 1, kPair>>(p, y, s);
    case 1: return run_gemm<1, MxTile<XT, 2, 2, 4, 2, kDeep, kPair ? 2 : 4, 1, kPair>>(p, y, s);
    case 2: return run_gemm<2, MxTile<XT, 2, 2, 2, 2, kDeep, kPair ? 2 : 1, 1, kPair>>(p, y, s);
    case 3: return run_gemm<3, MxTile<XT, 2, 1, 2, 2, 4, 2>>(p, y, s);
    default: return run_gemm<4, MxTile<XT, 1, 1, 2, 2, 4, 4, 2>>(p, y, s);
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
bool run_few_rows(const MxGemvParams &p, __bf16 *y, hipStream_t s, hipError_t *e) {
  if (p.experts) {
    if (p.M > 8 * static_cast<int64_t>(p.experts)) return false;
    *e = p.nblk <= 32 ? run_gemv<XT, 1, 4, 2>(p, y, s) : run_gemv<XT, 1, 4, 4>(p, y, s);
    return true;
  }
  const auto uneven = [&](int rows) {
    const double load = static_cast<double>(ceil_div(p.N, rows)) / kMxCus;
    return std::ceil(load) / load;
  };
  if (p.M > (p.N <= 16 * kMxCus ? 24 : p.N <= 32 * kMxCus ? 16 : 8)) return false;
  const int rows = p.M > 16 ? 16 : uneven(64) <= 1.15 * uneven(32) ? 64 : uneven(32) <= 1.25 * uneven(16) ? 32 : 16;
  if (rows == 64) *e = p.N <= 64 * kMxCus ? run_gemv<XT, 1, 4, 8>(p, y, s) : run_gemv<XT, 1, 4, 4>(p, y, s);
  else if (rows == 32) *e = run_gemv<XT, 1, 2, 8>(p, y, s);
  else *e = p.M > 16 ? run_gemv<XT, 2, 1, 8>(p, y, s) : run_gemv<XT, 1, 1, 8>(p, y, s);
  return true;
}

template <int XT>
hipError_t run_product(const MxLinear &a, hipStream_t s) {
  MxGemvParams p;
  MxGemmParams q;
  mx_product_params(a, p, q);
  __bf16 *y = static_cast<__bf16 *>(a.Y);
  hipError_t e;
  return run_few_rows<XT>(p, y, s, &e) ? e : run_tiles<XT>(q, y, s);
}

}  // namespace

hipError_t launch_mx_linear(const MxLinear &a, hipStream_t s) {
  return a.x_type == QLORA_MX_FP4 ? run_product<QLORA_MX_FP4>(a, s) : run_product<QLORA_MX_FP8>(a, s);
}

}  // namespace qnf4
