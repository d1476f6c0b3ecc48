// The gated feed-forward block around two frozen 4-bit weights with adapters,
// forward and backward:
//
//   G = X Wg^T + s (X Ag^T) Bg^T,  U = X Wu^T + s (X Au^T) Bu^T,  H = silu(G) U
//   dG = dH U sigma (1 + G (1 - sigma)),  dU = dH G sigma,  sigma = 1 / (1 + e^-G)
//   dX = dG Wg + dU Wu + lg Ag + lu Au,  lg = s dG Bg,  lu = s dU Bu
//   dAg = lg^T X,  dBg = dG^T (s X Ag^T),  and likewise of the other weight
//
// Forward, on the caller's stream:
//   k_gated_prep   block scales of both weights, and the adapters as bf16
//                  operands: [Ag; Au] as 2 rp rows of K, Bg and Bu as rows of the
//                  interleaved tiles below (rp: r rounded up to 64, zero padded)
//   k_gated_down   split partials of X [Ag; Au]^T: X is read once for both
//   k_gated_sum    Hs = bf16(s sums) [M][2 rp]
//   k_gated_fwd    up to 256 rows by 128 columns of H a workgroup: the large-tile loop of
//                  gemm_big.h on 128 rows of each weight, 32 of one and 32 of
//                  the other in turn, so that both products of an element of H
//                  end in one lane and the gate needs no exchange
//   k_gated_out    sums and gates the tiles whose reduction was split (below)
// Backward:
//   k_gated_prep   dG, dU from dH, G, U; block scales, [Ag; Au]^T [K][2 rp] and
//                  Bg^T, Bu^T [2][rp][N]
//   k_gated_down, k_gated_sum   l = bf16(s [dG Bg, dU Bu]) [M][2 rp]
//   k_gated_dx     dX = [dG, dU, l] [Wg; Wu; [Ag; Au]]: one reduction over both
//                  weights, so dX is rounded and written once
//   k_gated_dx_sum sums the tiles whose reduction was split
//   k_gated_few_low, k_gated_few_grad   instead of k_gated_down and the next two, for few sums
//   k_gated_grad, k_gated_grad_sum   split-M partials of the adapters' gradients and their sums
//
// Roundings to bf16, the operand type of the matrix instructions: the decoded
// weights, A and B, Hs and l (as in linear.hip), and the kept G and U, dG and
// dU. H comes from the unrounded G and U.
#include "block.h"
#include "gate.h"
#include "nf4_linear.h"

namespace qnf4 {
namespace {

// Tiles of BM rows: eight waves of BM / 2 rows by 64.
template <int BM>
using TileOf = TileCfg<BM, 256, 2, 4>;
constexpr int kT = TileOf<256>::kThreads;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// --------------------------------------------------------- operands and scales

__device__ __forceinline__ float adapter_at(const void *p, bool bf16, int64_t i) {
  return bf16 ? static_cast<float>(static_cast<const __bf16 *>(p)[i]) : static_cast<const float *>(p)[i];
}

constexpr int64_t kActGroups = 8192;

struct ActParams {
  const void *dH, *G, *U;
  __bf16 *dG, *dU;
  int64_t n, groups;
};
struct PrepParams {
  ActParams act;      // backward: its workgroups in front, the longest work
  const void *A[2], *B[2];
  bool bf16;
  int64_t N, K, nb;
  int r, rp;
  const int8_t *absmax_q[2];
  const float *dq_scale[2], *dq_mean[2];
  float *cs[2];
  // forward: Acat [2 rp][K], Bi [2 N][rp]; backward: At [K][2 rp], Bt [2][rp][N]
  __bf16 *Acat, *Bi, *At, *Bt;
  int64_t g_cs, g_a, g_b;   // workgroups of a segment
};

__device__ __forceinline__ void put8(__bf16 *dst, const float (&v)[8]) {
  *reinterpret_cast<uint4 *>(dst) =
      make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// dG, dU, eight elements a lane and turn, by workgroup g of the `groups`.
__device__ __forceinline__ void gated_act(const ActParams &p, int64_t g) {
  for (int64_t e = (g * 256 + threadIdx.x) * 8; e < p.n; e += p.groups * 2048) {
    const auto in = [e](const void *p) { return *reinterpret_cast<const uint4 *>(static_cast<const __bf16 *>(p) + e); };
    const uint4 a = in(p.dH), b = in(p.G), c = in(p.U);
    const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w}, wc[4] = {c.x, c.y, c.z, c.w};
    float dg[8], du[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const auto part = [i](const uint32_t (&w)[4]) {
        return __builtin_bit_cast(float, (i & 1) ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
      };
      gate_backward(part(wa), part(wb), part(wc), dg[i], du[i]);
    }
    put8(p.dG + e, dg);
    put8(p.dU + e, du);
  }
}

__global__ __launch_bounds__(256) void k_gated_prep(const PrepParams p) {
  int64_t g = blockIdx.x;
  if (g < p.act.groups) return gated_act(p.act, g);
  g -= p.act.groups;
  if (g < p.g_cs) {   // block scales, as k_adapter_finish forms them
    const int64_t b0 = (g * 256 + threadIdx.x) * 4;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t e = b0 + u;
      const int w = e >= p.nb;
      const int64_t b = e - (w ? p.nb : 0);
      if (e < 2 * p.nb) {
        const float kd = __fdiv_rn(p.dq_scale[w][b / kDqBlock], 127.0f);
        p.cs[w][b] = __fadd_rn(__fmul_rn(static_cast<float>(p.absmax_q[w][b]), kd), p.dq_mean[w][0]);
      }
    }
    return;
  }
  g -= p.g_cs;
  float v[8];
  if (g < p.g_a) {
    const int64_t i = g * 256 + threadIdx.x;
    if (p.Acat) {   // row j of both, eight columns
      const int64_t k8 = p.K / 8;
      if (i >= 2 * p.rp * k8) return;
      const int row = static_cast<int>(i / k8), w = row >= p.rp, j = row - w * p.rp;
      const int64_t k = (i - row * k8) * 8;
#pragma unroll
      for (int t = 0; t < 8; ++t) v[t] = j < p.r ? adapter_at(p.A[w], p.bf16, j * p.K + k + t) : 0.0f;
      put8(p.Acat + row * p.K + k, v);
    } else {        // column k, eight rows; consecutive lanes take consecutive k
      const int q8 = 2 * p.rp / 8;
      if (i >= p.K * q8) return;
      const int q = static_cast<int>(i / p.K), w = 8 * q >= p.rp, j = 8 * q - w * p.rp;
      const int64_t k = i - q * p.K;
#pragma unroll
      for (int t = 0; t < 8; ++t) v[t] = j + t < p.r ? adapter_at(p.A[w], p.bf16, (j + t) * p.K + k) : 0.0f;
      put8(p.At + k * 2 * p.rp + 8 * q, v);
    }
    return;
  }
  g -= p.g_a;
  const int64_t i = g * 256 + threadIdx.x;
  if (p.Bi) {       // eight columns of row n, in the tiles' order of rows
    const int q8 = p.rp / 8;
    if (i >= 2 * p.N * q8) return;
    const int64_t row = i / q8, n = 32 * (row >> 6) + (row & 31);
    const int w = static_cast<int>(row >> 5) & 1, j = static_cast<int>(i - row * q8) * 8;
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] = j + t < p.r ? adapter_at(p.B[w], p.bf16, n * p.r + j + t) : 0.0f;
    put8(p.Bi + row * p.rp + j, v);
  } else {          // eight rows n of column j; consecutive lanes take consecutive j
    if (i >= 2 * p.rp * (p.N / 8)) return;
    const int64_t part = i / p.rp;
    const int j = static_cast<int>(i - part * p.rp), w = part >= p.N / 8;
    const int64_t n = (part - (w ? p.N / 8 : 0)) * 8;
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] = j < p.r ? adapter_at(p.B[w], p.bf16, (n + t) * p.r + j) : 0.0f;
    put8(p.Bt + (static_cast<int64_t>(w) * p.rp + j) * p.N + n, v);
  }
}

// ------------------------------------------------------- adapter down products

// Split partials of P Q^T, both bf16, for one or two such products beside each
// other: a workgroup has 128 rows of P by BN rows of Q over some 64-deep steps,
// copied into a ring of four stages three steps ahead. Behind the last step it
// is copied again, into a stage that nobody reads any more, so that every wait
// is for the same number of copies.
struct DownParams {
  const void *P[2], *Q[2];
  float *part;        // [splits][M][ld]; null: one split, out
  __bf16 *out;        // [M][ld], scale times the sums
  float scale;
  int64_t M, L;       // L: the reduction, row length of P and Q
  int rows;           // rows of each Q
  int ld;
  int r, rp;          // the columns of a weight that there are, and with those behind them, which become zeros
  int tiles_n, tiles_m, tiles;   // of one product; of all
  int steps, per;     // 64-deep steps, and those of a split
};

template <int BN>
__global__ __launch_bounds__(256, 1) void k_gated_down(const DownParams p) {
  using C = TileCfg<128, BN, 2, 2>;
  using RowsP = DirectRowsT<256, 128>;
  using RowsQ = DirectRowsT<256, BN>;
  constexpr int kCopies = RowsP::kPerWave + RowsQ::kPerWave;
  __shared__ __attribute__((aligned(16))) __bf16 ring[4][C::kLdsA + C::kLdsB];
  const int z = static_cast<int>(blockIdx.x) / p.tiles, t = static_cast<int>(blockIdx.x) - z * p.tiles;
  const int one = p.tiles_m * p.tiles_n, w = t >= one, in = t - w * one;
  const int64_t m0 = static_cast<int64_t>(in / p.tiles_n) * 128;
  const int j0 = in % p.tiles_n * BN;
  const int s0 = z * p.per, n = min(p.per, p.steps - s0);
  const int64_t k0 = static_cast<int64_t>(s0) * kBK;
  const RowsP rp(static_cast<const __bf16 *>(w ? p.P[1] : p.P[0]) + k0, p.L, p.M, m0);
  const RowsQ rq(static_cast<const __bf16 *>(w ? p.Q[1] : p.Q[0]) + k0, p.L, p.rows, j0);
  auto issue = [&](int s, int stage) {
    const int64_t red = static_cast<int64_t>(min(s, n - 1)) * kBK;
    rp.issue(red, ring[stage]);
    rq.issue(red, ring[stage] + C::kLdsA);
  };
#pragma unroll
  for (int s = 0; s < 3; ++s) issue(s, s);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const FragAddr<C::WTM> fa(wave / C::WAVES_N * C::WTM, lane);
  const FragAddr<C::WTN> fb(wave % C::WAVES_N * C::WTN, lane);
  Acc<C> acc;
  acc.zero();
  for (int s = 0; s < n; ++s) {
    RowsP::template wait_copies<2 * kCopies>();
    __syncthreads();   // the step has landed, and everybody is done with the one before
    issue(s + 3, (s + 3) & 3);
    const __bf16 *stage = ring[s & 3];
    mma_step<C>(acc, stage, stage + C::kLdsA, fa, fb);
  }
  RowsP::template wait_copies<0>();
  // Q's rows of zeros made NaN of an infinity in P
#pragma unroll
  for (int j = 0; j < C::TN; ++j) {
    const int col = j0 + wave % C::WAVES_N * C::WTN + 32 * j + (lane & 31);
    if ((col < p.rp ? col : col - p.rp) < p.r) continue;
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc.v[i][j][e] = 0.0f;
  }
  if (p.part) store_f32<C>(acc, p.part + static_cast<int64_t>(z) * p.M * p.ld + w * p.rows, p.ld, p.M, p.rows, m0, j0);
  else store_bf16<C, true>(acc, p.out + w * p.rows, p.ld, p.M, p.rows, m0, j0, p.scale);
}

// out = bf16(scale * the sum of the partials), and `wide` the unrounded ones where it is not null, four elements a lane: each of the
// four waves adds a quarter of the splits in order, then the quarters are added
// (64 rows of 11008 x 4096 with r = 64: the forward takes 72 us with one wave
// for all splits, 68 so).
constexpr int64_t kSumGroups = int64_t(1) << 20;
__global__ __launch_bounds__(256) void k_gated_sum(const float *part, int splits, int64_t n, float scale, __bf16 *out, float *wide) {
  __shared__ float4 sums[3][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, per = (splits + 3) / 4, z0 = wave * per;
  for (int64_t e0 = static_cast<int64_t>(blockIdx.x) * 256; e0 < n; e0 += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t e = e0 + 4 * lane;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (e < n && z0 < splits) v = split_sum4(part + z0 * n, n, e, min(per, splits - z0));
    __syncthreads();   // the first wave is done with the turn before
    if (wave > 0) sums[wave - 1][lane] = v;
    __syncthreads();
    if (wave > 0 || e >= n) continue;
#pragma unroll
    for (int w = 0; w < 3; ++w) {
      const float4 s = sums[w][lane];
      v.x += s.x, v.y += s.y, v.z += s.z, v.w += s.w;
    }
    v = make_float4(scale * v.x, scale * v.y, scale * v.z, scale * v.w);
    *reinterpret_cast<uint2 *>(out + e) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    if (wide) *reinterpret_cast<float4 *>(wide + e) = v;
  }
}

// -------------------------------------------------------------- split tiles

// A tile occupies a compute unit, so tiles run in rounds of one for each, and
// the last `rest` tiles, where they would fill no more than half of a round,
// are split along the reduction into S parts, fp32 sums [S][rest][BM][256]
// that a kernel behind adds in order (4096 x 11008 x 4096, 96 tiles behind five
// rounds: 738 -> 721 us; 1536 rows, both directions: 757 -> 707). Fewer tiles
// than that in all are all split.
struct Tail {
  int bm;                // rows of a tile
  int64_t whole, rest;   // tiles
  int S, per;            // steps of a part
  float *part;
};
struct Piece {
  int tile, s0, s1;
  float *part;   // null: the whole reduction
  int z;
};
__device__ __forceinline__ Piece piece_of(const Tail &t, int b, int steps) {
  if (b < t.whole) return {b, 0, steps, nullptr, 0};
  const int q = b - static_cast<int>(t.whole), rest = static_cast<int>(t.rest), z = q / rest;
  return {static_cast<int>(t.whole) + q - z * rest, z * t.per, min(steps, (z + 1) * t.per), t.part + static_cast<int64_t>(q) * 256 * t.bm, z};
}
// The sums of four columns from `col` on of row `row` of split tile `i`.
__device__ __forceinline__ float4 sums_of(const Tail &t, int i, int row, int col) {
  const int64_t size = 256 * t.bm;
  return split_sum4(t.part, t.rest * size, i * size + row * 256 + col, t.S);
}

// ------------------------------------------------------------------ forward

struct FwdParams {
  const void *X;            // bf16 [M, K]
  const uint8_t *codes[2];  // [N, K] each
  const float *cs[2];
  const void *Hs;           // bf16 [M, 2 rp]
  const void *Bi;           // bf16 [2 N, rp], rows as the tiles'
  __bf16 *H, *G, *U;        // bf16 [M, N]; G and U or null
  int64_t M, N, K;
  int rp;
  Tail tail;                // a part's columns as the tiles' rows
};

// The rows of a tile: row R of the interleaved weight is row 32 (R / 64) + R %
// 32 of the gate (R / 32 even) or of the other one. A wave decodes 32 rows, all
// of one weight.
struct PairRows {
  using One = Nf4RowBigT<kT>;
  static_assert(One::CH == 1, "a row half a thread");
  static constexpr int kLoads = One::kLoads, kWrites = One::kWrites;
  using Pairs = One::Pairs;
  One one;
  __device__ PairRows(const FwdParams &p, int64_t n0) : one(p.codes[0], p.cs[0], p.N, p.K, 0) {
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int up = wave & 1;
    const int64_t first = n0 + 32 * (wave >> 1);
    one.cbase = (up ? p.codes[1] : p.codes[0]) + min(first, p.N - 1) * p.K / 2;
    one.sbase = (up ? p.cs[1] : p.cs[0]) + min(first, p.N - 1) * p.K / kBlock;
    // N is a multiple of 64: a wave's rows are all there or none of them
    const int64_t row = first < p.N ? (threadIdx.x >> 1) & 31 : 0;
    one.coff[0] = static_cast<uint32_t>(row * p.K / 2 + (threadIdx.x & 1) * 16);
    one.soff[0] = static_cast<uint32_t>(row * p.K / kBlock);
  }
  __device__ __forceinline__ void load(int64_t red0) { one.load(red0); }
  __device__ __forceinline__ void lookup(Pairs &q, const float2 *lv2, int i) const { one.lookup(q, lv2, i); }
  __device__ __forceinline__ void finish(__bf16 *lds, const Pairs &q, int i) const { one.finish(lds, q, i); }
  __device__ __forceinline__ void store_part(__bf16 *lds, const float2 *lv2, int i) const { one.store_part(lds, lv2, i); }
};

// A wave's BM / 2 rows of 32 columns to its rows of 128 columns in LDS, as bf16.
// Neighbouring lanes have neighbouring columns: of two rows, the even one takes
// the first and the odd one the second, so that a store is of two columns. The
// four rows that one store reaches lie on different banks. (Without the detour,
// from lanes with one column each, the forward took 735 us instead of 718.)
template <class Cfg, class F>
__device__ __forceinline__ void stage_rows(__bf16 *place, F value) {
  static_assert(Cfg::WAVES_N == 4 && Cfg::kLdsA >= Cfg::WTM * 128 && Cfg::kLdsB >= Cfg::WTM * 128, "the places");
  const int lane = threadIdx.x & 63, wn = (threadIdx.x >> 6) % Cfg::WAVES_N, odd = lane & 1, upper = lane >> 5;
  uint32_t *const to = reinterpret_cast<uint32_t *>(place) + (4 * upper + odd) * 64 + ((16 * wn + ((lane & 31) >> 1)) ^ (16 * (odd + 2 * upper)));
#pragma unroll
  for (int i = 0; i < Cfg::TM; ++i)
#pragma unroll
    for (int v = 0; v < 16; v += 2) {
      const float a = value(i, v), b = value(i, v + 1);
      const int other = __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, odd ? a : b), 0xb1, 0xf, 0xf, true);   // the neighbour's
      const float o = __builtin_bit_cast(float, other);
      to[(32 * i + 8 * (v >> 2) + (v & 3)) * 64] = odd ? pack_bf16x2(o, b) : pack_bf16x2(a, o);
    }
}

// The tile's BM rows of 128 columns to C [M, N], 256 bytes of a row by 16
// lanes. KEPT: nobody reads it soon, so it does not displace what the tiles read
// from the caches (4096 x 11008 x 4096, both directions: 4 to 18 us of 1570 less;
// with H written so too the forward alone takes 726 us instead of 718).
template <class Cfg, bool KEPT>
__device__ __forceinline__ void store_rows(const __bf16 *lo, const __bf16 *hi, __bf16 *C, int64_t M, int64_t N, int64_t m0, int64_t n0) {
  const int q = threadIdx.x & 15;
  const bool there = n0 + 8 * q < N;
#pragma unroll
  for (int k = 0; k < Cfg::BM * 16 / kT; ++k) {
    const int row = static_cast<int>(threadIdx.x >> 4) + kT / 16 * k, in = row < Cfg::WTM ? row : row - Cfg::WTM, bank = (in & 1) + (in >> 1 & 2);
    const u32x4 v = *reinterpret_cast<const u32x4 *>((row < Cfg::WTM ? lo : hi) + in * 128 + 8 * (q ^ (4 * bank)));
    if (!there || m0 + row >= M) continue;
    u32x4 *const to = reinterpret_cast<u32x4 *>(C + (m0 + row) * N + n0 + 8 * q);
    if (KEPT) __builtin_nontemporal_store(v, to);
    else *to = v;
  }
}

// BM rows by 128 columns of H: a wave ends with BM / 2 rows of 32 columns, the
// gate's sums in its first fragment column and the other weight's in its second.
template <int BM>
__global__ __launch_bounds__(kT, 1) void k_gated_fwd(const FwdParams p, const Nf4Tables tab) {
  using Cfg = TileOf<BM>;
  using Rows = DirectRowsT<kT, BM>;
  static_assert(Cfg::TN == 2, "a fragment column of each weight");
  __shared__ __attribute__((aligned(16))) __bf16 sa0[Cfg::kLdsA], sa1[Cfg::kLdsA];
  __shared__ __attribute__((aligned(16))) __bf16 sb0[Cfg::kLdsB], sb1[Cfg::kLdsB];
  const BigSmem smem{sa0, sa1, sb0, sb1};
  __shared__ float2 lv_tab[256 * kLvCopies];
  const float2 *lv = load_level_pairs(lv_tab, tab);
  const int tiles_m = static_cast<int>((p.M + BM - 1) / BM), tiles_n = static_cast<int>((p.N + 127) / 128);
  const Piece piece = piece_of(p.tail, static_cast<int>(blockIdx.x), static_cast<int>(p.K / kBK));
  int tm, tn;
  tile_of(piece.tile, tiles_m, tiles_n, tm, tn);
  const int64_t n0 = static_cast<int64_t>(tn) * 128, m0 = static_cast<int64_t>(tm) * BM;
  const int s0 = piece.s0, s1 = piece.s1;
  __syncthreads();
  Acc<Cfg> acc;
  acc.zero();
  {
    Rows da(static_cast<const __bf16 *>(p.X) + static_cast<int64_t>(s0) * kBK, p.K, p.M, m0);
    PairRows l0(p, n0), l1 = l0;
    auto load = [s0](PairRows &l, int s) { l.load(static_cast<int64_t>(s0 + s) * kBK); };
    big_mainloop_nf4<Cfg>(acc, da, l0, l1, load, s1 - s0, smem, lv);
  }
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int wm = w / Cfg::WAVES_N, wn = w % Cfg::WAVES_N;
  if (p.rp > 0 && piece.z == 0) {
    // each weight's columns take its own half of Hs
    const Rows ag(p.Hs, 2 * p.rp, p.M, m0), au(static_cast<const __bf16 *>(p.Hs) + p.rp, 2 * p.rp, p.M, m0);
    const DirectRowsT<kT> db(p.Bi, p.rp, 2 * p.N, 2 * n0);
    const FragAddr<Cfg::WTM> fa(wm * Cfg::WTM, lane);
    const FragAddr<Cfg::WTN> fb(wn * Cfg::WTN, lane);
    for (int s = 0; s < p.rp / kBK; ++s) {
      const int64_t red = static_cast<int64_t>(s) * kBK;
      ag.issue(red, sa0);
      au.issue(red, sa1);
      db.issue(red, sb0);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const __bf16 *sa = j ? sa1 : sa0;
          const bf16x8 b = *reinterpret_cast<const bf16x8 *>(sb0 + fb.off[kk] + j * 32 * kLDK);
#pragma unroll
          for (int i = 0; i < Cfg::TM; ++i) {
            const bf16x8 a = *reinterpret_cast<const bf16x8 *>(sa + fa.off[kk] + i * 32 * kLDK);
            acc.v[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc.v[i][j], 0, 0, 0);
          }
        }
      __syncthreads();
    }
  }
  if (piece.part) {
    store_f32<Cfg>(acc, piece.part, 256, min(p.M - m0, int64_t(BM)), 256, 0, 0);
    return;
  }
  // through LDS, where each array is half of the tile's rows
  const auto put = [&](__bf16 *lo, __bf16 *hi, auto value) { stage_rows<Cfg>(wm ? hi : lo, value); };
  if (p.G) {
    put(sa0, sa1, [&](int i, int v) { return acc.v[i][0][v]; });
    put(sb0, sb1, [&](int i, int v) { return acc.v[i][1][v]; });
    __syncthreads();
    store_rows<Cfg, true>(sa0, sa1, p.G, p.M, p.N, m0, n0);
    store_rows<Cfg, true>(sb0, sb1, p.U, p.M, p.N, m0, n0);
    __syncthreads();
  }
  put(sa0, sa1, [&](int i, int v) { return gate_value(acc.v[i][0][v], acc.v[i][1][v]); });
  __syncthreads();
  store_rows<Cfg, false>(sa0, sa1, p.H, p.M, p.N, m0, n0);
}

// H (and G, U) of the split tiles, four columns a lane, BM / 8 workgroups a tile.
__global__ __launch_bounds__(256) void k_gated_out(const FwdParams p) {
  const int bm = p.tail.bm, i = static_cast<int>(blockIdx.x) / (bm / 8), at = (static_cast<int>(blockIdx.x) - i * (bm / 8)) * 256 + static_cast<int>(threadIdx.x);
  const int row = at >> 5, c = 4 * (at & 31);
  int tm, tn;
  tile_of(static_cast<int>(p.tail.whole) + i, static_cast<int>((p.M + bm - 1) / bm), static_cast<int>((p.N + 127) / 128), tm, tn);
  const int64_t m = static_cast<int64_t>(tm) * bm + row, n = static_cast<int64_t>(tn) * 128 + c, e = m * p.N + n;
  if (m >= p.M || n >= p.N) return;
  const int col = 64 * (c >> 5) + (c & 31);
  const float4 g = sums_of(p.tail, i, row, col), u = sums_of(p.tail, i, row, col + 32);
  *reinterpret_cast<uint2 *>(p.H + e) = make_uint2(pack_bf16x2(gate_value(g.x, u.x), gate_value(g.y, u.y)),
                                                   pack_bf16x2(gate_value(g.z, u.z), gate_value(g.w, u.w)));
  if (p.G) {
    *reinterpret_cast<uint2 *>(p.G + e) = make_uint2(pack_bf16x2(g.x, g.y), pack_bf16x2(g.z, g.w));
    *reinterpret_cast<uint2 *>(p.U + e) = make_uint2(pack_bf16x2(u.x, u.y), pack_bf16x2(u.z, u.w));
  }
}

// ----------------------------------------------------------------- backward

struct DxParams {
  const void *dG, *dU;      // bf16 [M, N]
  const uint8_t *codes[2];
  const float *cs[2];
  const void *low;          // bf16 [M, 2 rp]
  const void *At;           // bf16 [K, 2 rp]
  void *dX;                 // bf16 [M, K]
  int64_t M, N, K;
  int rp;
  Tail tail;                // of the 2 N / 64 steps, the gate's in front
};

// Rows of dG for steps below N, of dU behind them.
template <int BM>
struct DualRows {
  using Rows = DirectRowsT<kT, BM>;
  static constexpr int kPerWave = Rows::kPerWave;
  Rows rows;
  const char *base[2];
  int64_t red0, N;
  __device__ DualRows(const DxParams &p, int64_t m0, int64_t red0_)
      : rows(p.dG, p.N, p.M, m0), base{rows.base, static_cast<const char *>(p.dU) + m0 * p.N * 2}, red0(red0_), N(p.N) {}
  __device__ __forceinline__ void issue(int64_t red, __bf16 *lds) const { issue_range(red, lds, 0, kPerWave); }
  __device__ __forceinline__ void issue_range(int64_t red, __bf16 *lds, int i0, int n) const {
    red += red0;
    const bool up = red >= N;
    Rows r = rows;
    r.base = up ? base[1] : base[0];
    r.issue_range(up ? red - N : red, lds, i0, n);
  }
  template <int L>
  __device__ __forceinline__ static void wait_copies() { Rows::template wait_copies<L>(); }
};

template <int BM>
__global__ __launch_bounds__(kT, 1) void k_gated_dx(const DxParams p, const Nf4Tables tab) {
  using Cfg = TileOf<BM>;
  __shared__ __attribute__((aligned(16))) __bf16 sa0[Cfg::kLdsA], sa1[Cfg::kLdsA];
  __shared__ __attribute__((aligned(16))) __bf16 sb0[Cfg::kLdsB], sb1[Cfg::kLdsB];
  const BigSmem smem{sa0, sa1, sb0, sb1};
  __shared__ float2 lv_tab[256 * kLvCopies];
  const float2 *lv = load_level_pairs(lv_tab, tab);
  const int tiles_m = static_cast<int>((p.M + BM - 1) / BM), tiles_k = static_cast<int>((p.K + 255) / 256);
  const Piece piece = piece_of(p.tail, static_cast<int>(blockIdx.x), static_cast<int>(2 * p.N / kBK));
  int tm, tn;
  tile_of(piece.tile, tiles_m, tiles_k, tm, tn);
  const int64_t k0 = static_cast<int64_t>(tn) * 256, m0 = static_cast<int64_t>(tm) * BM;
  const int s0 = piece.s0, s1 = piece.s1;
  __syncthreads();
  Acc<Cfg> acc;
  acc.zero();
  {
    const DualRows<BM> da(p, m0, static_cast<int64_t>(s0) * kBK);
    Nf4TransBigT<kT> l0(p.codes[0], p.cs[0], p.K, k0), l1 = l0;
    const uint8_t *const codes[2] = {p.codes[0] + k0 / 2, p.codes[1] + k0 / 2};
    const float *const cs[2] = {p.cs[0] + k0 / kBlock, p.cs[1] + k0 / kBlock};
    const int64_t K = p.K, N = p.N;
    auto load = [&](Nf4TransBigT<kT> &l, int s) {
      const int64_t red = static_cast<int64_t>(s0 + s) * kBK;
      const bool up = red >= N;
      l.cbase = up ? codes[1] : codes[0];
      l.sbase = up ? cs[1] : cs[0];
      l.load(up ? red - N : red, K);
    };
    big_mainloop_nf4<Cfg>(acc, da, l0, l1, load, s1 - s0, smem, lv);
  }
  if (p.rp > 0 && piece.z == 0) {
    const DirectRowsT<kT, BM> da(p.low, 2 * p.rp, p.M, m0);
    const DirectRowsT<kT> db(p.At, 2 * p.rp, p.K, k0);
    big_mainloop_dense<Cfg>(acc, da, db, 2 * p.rp / kBK, smem);
  }
  if (piece.part)
    store_f32<Cfg>(acc, piece.part, 256, min(p.M - m0, int64_t(BM)), 256, 0, 0);
  else if (m0 + BM <= p.M && k0 + 256 <= p.K)
    store_bf16<Cfg, false>(acc, static_cast<__bf16 *>(p.dX), p.K, p.M, p.K, m0, k0, 1.0f);
  else
    store_bf16<Cfg, true>(acc, static_cast<__bf16 *>(p.dX), p.K, p.M, p.K, m0, k0, 1.0f);
}

// Split-M partials of the adapters' gradients: 64 x 256 tiles of [lg, lu]^T X
// first, then 256 x 64 tiles of dG^T Hs_g and dU^T Hs_u.
struct GradParams {
  const void *X, *d[2], *Hs, *low;
  float *a_part, *b_part;   // [splits][2 rp][K], [splits][2][N][rp]; null: one split, the gradients
  void *dA[2], *dB[2];
  bool bf16;
  int64_t M, N, K;
  int r, rp;
  int a_tiles_c, a_tiles, a_splits, a_steps;
  int b_tiles_c, b_tiles, b_splits, b_steps;   // tiles: of one weight
};

using CfgGradA = TileCfg<64, 256, 1, 4>;
using CfgGradB = TileCfg<256, 64, 4, 1>;

template <class C>
__device__ __forceinline__ void store_grad(const Acc<C> &acc, void *to, bool bf16, int64_t ld, int64_t rows, int64_t cols, int64_t m0, int64_t n0) {
  if (bf16) store_bf16<C, true>(acc, static_cast<__bf16 *>(to), ld, rows, cols, m0, n0, 1.0f);
  else store_f32<C>(acc, static_cast<float *>(to), ld, rows, cols, m0, n0);
}

__global__ __launch_bounds__(256) void k_gated_grad(const GradParams p) {
  __shared__ __attribute__((aligned(16))) __bf16 smem[2 * (CfgGradA::kLdsA + CfgGradA::kLdsB)];
  int g = blockIdx.x;
  const bool is_a = g < p.a_tiles * p.a_splits;
  if (!is_a) g -= p.a_tiles * p.a_splits;
  const int tiles = is_a ? p.a_tiles : 2 * p.b_tiles;
  const int per = is_a ? p.a_steps : p.b_steps;
  const int z = g / tiles;
  int t = g % tiles;
  const int total = static_cast<int>((p.M + kBK - 1) / kBK);
  const int s0 = z * per, steps = min(per, total - s0);
  // rows of this split's range only: the two-stage loop reads past its end
  const int64_t red_end = min(p.M, static_cast<int64_t>(s0 + steps) * kBK);
  if (is_a) {
    const int64_t c0 = static_cast<int64_t>(t % p.a_tiles_c) * 256, r0 = static_cast<int64_t>(t / p.a_tiles_c) * 64;
    Acc<CfgGradA> acc;
    acc.zero();
    TransBf16Narrow<64, 256> la(p.low, 2 * p.rp, red_end, r0), la1 = la;
    TransBf16<256, 256> lb(p.X, p.K, red_end, p.K, c0), lb1 = lb;
    mainloop2<CfgGradA>(acc, la, la1, lb, lb1, static_cast<int64_t>(s0) * kBK, steps, smem);
    if (p.a_part) {
      store_f32<CfgGradA>(acc, p.a_part + static_cast<int64_t>(z) * 2 * p.rp * p.K, p.K, 2 * p.rp, p.K, r0, c0);
    } else {
      const int up = r0 >= p.rp;
      store_grad<CfgGradA>(acc, up ? p.dA[1] : p.dA[0], p.bf16, p.K, p.r, p.K, r0 - up * p.rp, c0);
    }
  } else {
    const int w = t >= p.b_tiles;
    t -= w * p.b_tiles;
    const int64_t c0 = static_cast<int64_t>(t % p.b_tiles_c) * 64, r0 = static_cast<int64_t>(t / p.b_tiles_c) * 256;
    Acc<CfgGradB> acc;
    acc.zero();
    TransBf16<256, 256> la(w ? p.d[1] : p.d[0], p.N, red_end, p.N, r0), la1 = la;
    TransBf16Narrow<64, 256> lb(p.Hs, 2 * p.rp, red_end, w * p.rp + c0), lb1 = lb;
    mainloop2<CfgGradB>(acc, la, la1, lb, lb1, static_cast<int64_t>(s0) * kBK, steps, smem);
    if (p.b_part) store_f32<CfgGradB>(acc, p.b_part + (2 * static_cast<int64_t>(z) + w) * p.N * p.rp, p.rp, p.N, p.rp, r0, c0);
    else store_grad<CfgGradB>(acc, w ? p.dB[1] : p.dB[0], p.bf16, p.r, p.N, p.r, r0, c0);
  }
}

struct GradSumParams {
  const float *a_part, *b_part;   // null: nothing to add
  void *dA[2], *dB[2];
  bool bf16;
  int64_t N, K;
  int r, rp, a_splits, b_splits;
};

__global__ __launch_bounds__(256) void k_gated_grad_sum(const GradSumParams p) {
  const int64_t na = p.a_part ? p.r * p.K : 0, nb = p.b_part ? p.N * p.r : 0, n = 2 * (na + nb);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
    float v;
    void *to;
    int64_t e;
    if (i < 2 * na) {
      const int w = i >= na;
      e = i - w * na;
      v = split_sum(p.a_part, 2 * p.rp * p.K, w * p.rp * p.K + e, p.a_splits);
      to = p.dA[w];
    } else {
      const int64_t b = i - 2 * na;
      const int w = b >= nb;
      e = b - w * nb;
      const int64_t row = e / p.r;
      v = split_sum(p.b_part, 2 * p.N * p.rp, (w * p.N + row) * p.rp + (e - row * p.r), p.b_splits);
      to = p.dB[w];
    }
    if (p.bf16) static_cast<__bf16 *>(to)[e] = static_cast<__bf16>(v);
    else static_cast<float *>(to)[e] = v;
  }
}

// A's gradient passes through the M r sums l. Where these are few their roundings
// do not even out (1 row, r = 8: dA off by up to 6e-3 with dG and l rounded to
// bf16 on their way, 4e-3 so), and dG, dU and l stay fp32 in products without
// matrix instructions. Both directions, so and with matrix instructions: 4 rows of
// 1024 x 1024, r = 8, 33 and 38 us; 8 rows of 4096 x 4096, r = 8, 64 and 66; 1 row of
// 11008 x 4096, r = 64, 78 and 78; 16 rows, r = 4, 98 and 95; but 32 rows, r = 64,
// 233 and 115.
struct FewParams {
  const __bf16 *dH, *G, *U, *X, *Hs;
  const void *B[2];
  void *dA[2], *dB[2];
  bool bf16;
  int64_t N, K, per;   // columns of a split
  int M, r, rp;
  float *part;         // [splits][M][2 rp]
  const float *low;    // [M][2 rp]
};
__device__ __forceinline__ void few_gate(const FewParams &p, int64_t at, float &dg, float &du) {
  gate_backward(static_cast<float>(p.dH[at]), static_cast<float>(p.G[at]), static_cast<float>(p.U[at]), dg, du);
}

// Split sums of dG Bg and dU Bu: a row of one of them and `per` columns n a
// workgroup, 256 at a time; a thread has column j of B and every (256 / J)-th n.
__global__ __launch_bounds__(256) void k_gated_few_low(const FewParams p) {
  __shared__ float d[256], sums[256];
  const int m = static_cast<int>(blockIdx.x) >> 1, w = static_cast<int>(blockIdx.x) & 1, tid = threadIdx.x;
  int J = 4;
  while (J < p.r) J *= 2;
  const int j = tid & (J - 1), slice = tid / J, slices = 256 / J;
  const int64_t n0 = blockIdx.y * p.per, n1 = min(p.N, n0 + p.per);
  const void *const B = w ? p.B[1] : p.B[0];
  float acc = 0.0f;
  for (int64_t base = n0; base < n1; base += 256) {
    float dg = 0.0f, du = 0.0f;
    if (base + tid < n1) few_gate(p, m * p.N + base + tid, dg, du);
    __syncthreads();   // the turn before is done
    d[tid] = w ? du : dg;
    __syncthreads();
    const int count = static_cast<int>(min(n1 - base, int64_t(256)));
    if (j < p.r)
#pragma unroll 8
      for (int i = slice; i < count; i += slices) acc = fmaf(d[i], adapter_at(B, p.bf16, (base + i) * p.r + j), acc);
  }
  sums[tid] = acc;
  __syncthreads();
  if (tid >= p.rp) return;
  float v = 0.0f;
  if (tid < p.r)
    for (int s = 0; s < slices; ++s) v += sums[s * J + tid];
  p.part[(static_cast<int64_t>(blockIdx.y) * p.M + m) * 2 * p.rp + w * p.rp + tid] = v;
}

// dA = l^T X, eight columns a thread, then dB = dG^T Hs, eight columns of both a thread.
__global__ __launch_bounds__(256) void k_gated_few_grad(const FewParams p) {
  const int64_t k8 = p.K / 8, na = 2 * p.r * k8;
  const int octets = (p.r + 7) / 8;
  int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i < na) {
    const int w = i >= na / 2;
    i -= w ? na / 2 : 0;
    const int j = static_cast<int>(i / k8);
    const int64_t k = 8 * (i - j * k8);
    float v[8] = {};
    for (int m = 0; m < p.M; ++m) {
      const float l = p.low[static_cast<int64_t>(m) * 2 * p.rp + w * p.rp + j];
      const bf16x8 x = *reinterpret_cast<const bf16x8 *>(p.X + m * p.K + k);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = fmaf(l, static_cast<float>(x[e]), v[e]);
    }
    if (p.bf16) {
      put8(static_cast<__bf16 *>(w ? p.dA[1] : p.dA[0]) + j * p.K + k, v);
    } else {
      float *const to = static_cast<float *>(w ? p.dA[1] : p.dA[0]) + j * p.K + k;
      *reinterpret_cast<float4 *>(to) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4 *>(to + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
    return;
  }
  i -= na;
  if (i >= p.N * octets) return;
  const int64_t n = i / octets;
  const int j0 = 8 * static_cast<int>(i - n * octets);
  float v[2][8] = {};
  for (int m = 0; m < p.M; ++m) {
    float d[2];
    few_gate(p, m * p.N + n, d[0], d[1]);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const bf16x8 h = *reinterpret_cast<const bf16x8 *>(p.Hs + static_cast<int64_t>(m) * 2 * p.rp + w * p.rp + j0);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[w][e] = fmaf(d[w], static_cast<float>(h[e]), v[w][e]);
    }
  }
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (j0 + e >= p.r) continue;
      void *const to = w ? p.dB[1] : p.dB[0];
      if (p.bf16) static_cast<__bf16 *>(to)[n * p.r + j0 + e] = static_cast<__bf16>(v[w][e]);
      else static_cast<float *>(to)[n * p.r + j0 + e] = v[w][e];
    }
}

// dX of the split tiles, four columns a lane, BM / 4 workgroups a tile.
__global__ __launch_bounds__(256) void k_gated_dx_sum(const DxParams p) {
  const int bm = p.tail.bm, i = static_cast<int>(blockIdx.x) / (bm / 4), at = (static_cast<int>(blockIdx.x) - i * (bm / 4)) * 256 + static_cast<int>(threadIdx.x);
  const int row = at >> 6, c = 4 * (at & 63);
  int tm, tn;
  tile_of(static_cast<int>(p.tail.whole) + i, static_cast<int>((p.M + bm - 1) / bm), static_cast<int>((p.K + 255) / 256), tm, tn);
  const int64_t m = static_cast<int64_t>(tm) * bm + row, k = static_cast<int64_t>(tn) * 256 + c;
  if (m >= p.M || k >= p.K) return;
  const float4 v = sums_of(p.tail, i, row, c);
  *reinterpret_cast<uint2 *>(static_cast<__bf16 *>(p.dX) + m * p.K + k) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// -------------------------------------------------------------------- plan

// Splits of the adapters' down products at most (11008 x 4096, both directions,
// 333 and 64 rows: 253 and 142 us with 64, 249 and 141 with 32, 247 and 143 with 16).
// Up to kDownSteps steps are one split, which needs no sum behind (200 rows of 1024 x 1024, both directions: 69.4 us
// split, 74.2 so).
constexpr int kDownSplits = 32, kDownSteps = 4;
Split down_split(int64_t tiles, int steps) { return choose_split(tiles, steps, steps <= kDownSteps ? 1 : kDownSplits, kCus); }
// The same of the adapters' gradients (11008 x 4096, both directions: 64 rows 141 us split, 131 so; 333 rows 239 and
// 234; but 800 rows of 2048 x 2048 127 and 134).
constexpr int kGradSteps = 8;

struct Plan {
  int rp;
  Tail tail;
  Split down, ga, gb;
};

// The tiles with BM = bm. Parts of sixteen steps at least where there are whole
// rounds in front.
Tail tail_of(int bm, int64_t tiles, int steps) {
  Tail t{bm, tiles, 0, 1, steps, nullptr};
  const int64_t rest = tiles % kCus;
  if (rest == 0 || 2 * rest > kCus) return t;
  const int S = static_cast<int>(std::min<int64_t>(kCus / rest, steps / (tiles > rest ? 16 : kMinSplitSteps)));
  if (S < 2) return t;
  t.per = static_cast<int>(ceil_div(steps, S));
  t.S = static_cast<int>(ceil_div(steps, t.per));
  t.whole = tiles - rest;
  t.rest = rest;
  return t;
}

// Fewer rows to a tile decode the weights more often for the same product but
// leave fewer rows empty and fewer compute units without a tile. A round of
// 256, 192, 128 and 64 rows costs as 1, 0.82, 0.635 and 0.485 (4096 x 11008 x
// 4096: 128, 105, 81 and 62 us), the kernel that adds split tiles about 0.1. Of
// these the least (11008 x 4096, forward, us with 256, 192, 128 and 64 rows: 64
// rows 97, 86, 78, 72; 128 rows 98, 86, 79, 93; 192 rows 97, 88, 101, 113; 333
// rows 130, 114, 132, 171; 512 rows 134, 158, 156, 213; both directions of 333
// rows 289, 260, 284, 396).
Tail make_tail(int64_t M, int64_t tiles_n, int steps) {
  constexpr struct {
    int bm;
    double cost;
  } kTiles[] = {{256, 1.0}, {192, 0.82}, {128, 0.635}, {64, 0.485}};
  Tail best{};
  double least = 0;
  for (const auto &k : kTiles) {
    const Tail t = tail_of(k.bm, grid_blocks(M, k.bm) * tiles_n, steps);
    const double rounds = static_cast<double>(ceil_div(t.whole, kCus)) + (t.rest ? 1.0 / t.S : 0.0);
    const double cost = k.cost * rounds + (t.rest ? 0.1 : 0.0);
    if (best.bm == 0 || cost < least) best = t, least = cost;
  }
  return best;
}

// Whether the adapters' gradients take the kernels for few sums.
constexpr int64_t kFewRows = 16, kFewSums = 64;
bool few_sums(int64_t M, int r) { return r > 0 && M <= kFewRows && M * r <= kFewSums; }

Plan make_plan(int64_t M, int64_t N, int64_t K, int r, bool backward) {
  Plan pl{};
  pl.rp = gated_padded_rank(r);
  if (!backward) {
    pl.tail = make_tail(M, grid_blocks(N, 128), static_cast<int>(K / kBK));
    if (r) pl.down = down_split(grid_blocks(M, 128) * (2 * pl.rp / 128), static_cast<int>(K / kBK));
    return pl;
  }
  pl.tail = make_tail(M, grid_blocks(K, 256), static_cast<int>(2 * N / kBK));
  if (few_sums(M, r)) {   // splits and columns of k_gated_few_low
    const int64_t turns = ceil_div(N, 64), splits = std::min(turns, kCus / M);
    pl.down.steps_per_split = static_cast<int>(64 * ceil_div(turns, splits));
    pl.down.splits = static_cast<int>(ceil_div(N, pl.down.steps_per_split));
  } else if (r) {
    pl.down = down_split(grid_blocks(M, 128) * 2 * (pl.rp / 64), static_cast<int>(N / kBK));
    const int msteps = static_cast<int>(ceil_div(M, kBK));
    // more splits cost more to write and add than they spread (11008 x 4096, both directions of 333, 1024 and 4096
    // rows: 247, 494 and 1540 us with at most eight, 239, 484 and 1524 with four, 238, 482 and 1527 with two)
    pl.ga = choose_split(grid_blocks(K, 256) * (2 * pl.rp / 64), msteps, msteps <= kGradSteps ? 1 : 4);
    pl.gb = choose_split(2 * grid_blocks(N, 256) * (pl.rp / 64), msteps, msteps <= kGradSteps ? 1 : 4);
  }
  return pl;
}

struct Buffers {
  float *cs[2], *down, *wide, *ga, *gb;
  __bf16 *Acat, *Bi, *At, *Bt, *low, *dG, *dU, *Hs;
};

size_t carve(void *ws, Plan &pl, int64_t M, int64_t N, int64_t K, int r, bool backward, Buffers *b) {
  Carve c{static_cast<char *>(ws)};
  if (!backward && M <= kGatedStreamRows) {
    if (pl.rp) b->Hs = c.take<__bf16>(2 * static_cast<size_t>(pl.rp) * M);
    return c.off;
  }
  const int64_t nb = N * K / kBlock;
  b->cs[0] = c.take<float>(nb);
  b->cs[1] = c.take<float>(nb);
  if (pl.tail.rest) pl.tail.part = c.take<float>(static_cast<size_t>(pl.tail.S) * pl.tail.rest * 256 * pl.tail.bm);
  const size_t cols = 2 * static_cast<size_t>(pl.rp);
  const bool few = backward && few_sums(M, r);
  if (pl.rp && (few || pl.down.splits > 1)) b->down = c.take<float>(pl.down.splits * M * cols);
  if (!backward) {
    if (pl.rp) {
      b->Acat = c.take<__bf16>(cols * K);
      b->Bi = c.take<__bf16>(cols * N);
      b->Hs = c.take<__bf16>(cols * M);
    }
    return c.off;
  }
  b->dG = c.take<__bf16>(static_cast<size_t>(M) * N);
  b->dU = c.take<__bf16>(static_cast<size_t>(M) * N);
  if (pl.rp) {
    b->At = c.take<__bf16>(cols * K);
    b->low = c.take<__bf16>(cols * M);
    if (few) {
      b->wide = c.take<float>(cols * M);
      return c.off;
    }
    b->Bt = c.take<__bf16>(cols * N);
    if (pl.ga.splits > 1) b->ga = c.take<float>(pl.ga.splits * cols * K);
    if (pl.gb.splits > 1) b->gb = c.take<float>(pl.gb.splits * cols * N);
  }
  return c.off;
}

// Block scales and bf16 operands.
void run_prep(const GatedArgs &a, const Plan &pl, const Buffers &b, bool backward, const ActParams &act, hipStream_t s) {
  PrepParams p{};
  p.act = act;
  for (int w = 0; w < 2; ++w) {
    p.A[w] = a.A[w];
    p.B[w] = a.B[w];
    p.absmax_q[w] = a.w[w].absmax_q;
    p.dq_scale[w] = a.w[w].dq_scale;
    p.dq_mean[w] = a.w[w].dq_mean;
    p.cs[w] = b.cs[w];
  }
  p.bf16 = a.adapter_bf16;
  p.N = a.N;
  p.K = a.K;
  p.nb = a.N * a.K / kBlock;
  p.r = a.r;
  p.rp = pl.rp;
  if (backward) p.At = b.At, p.Bt = b.Bt;
  else p.Acat = b.Acat, p.Bi = b.Bi;
  p.g_cs = fmt_dq(a.format) ? ceil_div(2 * p.nb, 1024) : 0;
  if (pl.rp) {
    p.g_a = ceil_div(2 * pl.rp * a.K / 8, 256);
    if (!backward || b.Bt) p.g_b = ceil_div(2 * pl.rp * a.N / 8, 256);
  }
  const int64_t groups = act.groups + p.g_cs + p.g_a + p.g_b;
  if (groups > 0) k_gated_prep<<<static_cast<unsigned>(groups), 256, 0, s>>>(p);
}

const float *scales(const GatedArgs &a, const Buffers &b, int w) { return fmt_dq(a.format) ? b.cs[w] : a.w[w].absmax; }

}  // namespace

size_t gated_ws_bytes(int64_t M, int64_t N, int64_t K, int r, bool backward) {
  Plan pl = make_plan(M, N, K, r, backward);
  Buffers b{};
  return carve(nullptr, pl, M, N, K, r, backward, &b);
}

hipError_t launch_gated_fwd(const GatedArgs &a, const void *X, void *H, void *G, void *U, void *Hs, void *ws, hipStream_t s) {
  Plan pl = make_plan(a.M, a.N, a.K, a.r, false);
  Buffers b{};
  carve(ws, pl, a.M, a.N, a.K, a.r, false, &b);
  if (Hs) b.Hs = static_cast<__bf16 *>(Hs);
  if (a.M <= kGatedStreamRows) return launch_gated_stream(a, X, H, G, U, b.Hs, s);
  run_prep(a, pl, b, false, ActParams{}, s);
  if (pl.rp) {
    DownParams d{};
    d.P[0] = X;
    d.Q[0] = b.Acat;
    d.part = b.down;
    d.out = b.Hs;
    d.scale = a.scale;
    d.M = a.M;
    d.L = a.K;
    d.rows = d.ld = 2 * pl.rp;
    d.r = a.r;
    d.rp = pl.rp;
    d.tiles_n = 2 * pl.rp / 128;
    d.tiles_m = static_cast<int>(ceil_div(a.M, 128));
    d.tiles = d.tiles_m * d.tiles_n;
    d.steps = static_cast<int>(a.K / kBK);
    d.per = pl.down.steps_per_split;
    k_gated_down<128><<<static_cast<unsigned>(d.tiles * pl.down.splits), 256, 0, s>>>(d);
    const int64_t n = a.M * 2 * pl.rp;
    if (b.down) k_gated_sum<<<static_cast<unsigned>(std::min(ceil_div(n, 256), kSumGroups)), 256, 0, s>>>(b.down, pl.down.splits, n, a.scale, b.Hs, nullptr);
  }
  FwdParams p{X, {a.w[0].codes, a.w[1].codes}, {scales(a, b, 0), scales(a, b, 1)}, b.Hs, b.Bi, static_cast<__bf16 *>(H),
              static_cast<__bf16 *>(G), static_cast<__bf16 *>(U), a.M, a.N, a.K, pl.rp, pl.tail};
  const auto run = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(pl.tail.whole + pl.tail.rest * pl.tail.S), kT, 0, s>>>(p, format_tables(a.format));
  };
  switch (pl.tail.bm) {
    case 64: run(k_gated_fwd<64>); break;
    case 128: run(k_gated_fwd<128>); break;
    case 192: run(k_gated_fwd<192>); break;
    default: run(k_gated_fwd<256>); break;
  }
  if (pl.tail.rest) k_gated_out<<<static_cast<unsigned>(pl.tail.bm / 8 * pl.tail.rest), 256, 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_gated_bwd(const GatedArgs &a, const void *dH, const void *X, const void *G, const void *U, const void *Hs,
                            void *dX, void *const (&dA)[2], void *const (&dB)[2], void *ws, hipStream_t s) {
  Plan pl = make_plan(a.M, a.N, a.K, a.r, true);
  Buffers b{};
  carve(ws, pl, a.M, a.N, a.K, a.r, true, &b);
  const int64_t n = a.M * a.N;
  run_prep(a, pl, b, true, ActParams{dH, G, U, b.dG, b.dU, n, std::min(ceil_div(n, 2048), kActGroups)}, s);
  const bool few = few_sums(a.M, a.r);
  FewParams fp{};
  if (few) {
    const auto in = [](const void *p) { return static_cast<const __bf16 *>(p); };
    fp = {in(dH), in(G), in(U), in(X), in(Hs), {a.B[0], a.B[1]}, {dA[0], dA[1]}, {dB[0], dB[1]}, a.adapter_bf16, a.N, a.K,
          pl.down.steps_per_split, static_cast<int>(a.M), a.r, pl.rp, b.down, b.wide};
    k_gated_few_low<<<dim3(static_cast<unsigned>(2 * a.M), static_cast<unsigned>(pl.down.splits)), 256, 0, s>>>(fp);
    const int64_t count = a.M * 2 * pl.rp;
    k_gated_sum<<<static_cast<unsigned>(ceil_div(count, 256)), 256, 0, s>>>(b.down, pl.down.splits, count, a.scale, b.low, b.wide);
  } else if (pl.rp) {
    DownParams d{};
    d.P[0] = b.dG;
    d.P[1] = b.dU;
    d.Q[0] = b.Bt;
    d.Q[1] = b.Bt + pl.rp * a.N;
    d.part = b.down;
    d.out = b.low;
    d.scale = a.scale;
    d.M = a.M;
    d.L = a.N;
    d.rows = d.rp = pl.rp;
    d.ld = 2 * pl.rp;
    d.r = a.r;
    d.tiles_n = pl.rp / 64;
    d.tiles_m = static_cast<int>(ceil_div(a.M, 128));
    d.tiles = 2 * d.tiles_m * d.tiles_n;
    d.steps = static_cast<int>(a.N / kBK);
    d.per = pl.down.steps_per_split;
    k_gated_down<64><<<static_cast<unsigned>(d.tiles * pl.down.splits), 256, 0, s>>>(d);
    const int64_t count = a.M * 2 * pl.rp;
    if (b.down) k_gated_sum<<<static_cast<unsigned>(std::min(ceil_div(count, 256), kSumGroups)), 256, 0, s>>>(b.down, pl.down.splits, count, a.scale, b.low, nullptr);
  }
  DxParams p{b.dG, b.dU, {a.w[0].codes, a.w[1].codes}, {scales(a, b, 0), scales(a, b, 1)}, b.low, b.At, dX, a.M, a.N, a.K,
             pl.rp, pl.tail};
  const auto run = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(pl.tail.whole + pl.tail.rest * pl.tail.S), kT, 0, s>>>(p, format_tables(a.format));
  };
  switch (pl.tail.bm) {
    case 64: run(k_gated_dx<64>); break;
    case 128: run(k_gated_dx<128>); break;
    case 192: run(k_gated_dx<192>); break;
    default: run(k_gated_dx<256>); break;
  }
  if (pl.tail.rest) k_gated_dx_sum<<<static_cast<unsigned>(pl.tail.bm / 4 * pl.tail.rest), 256, 0, s>>>(p);
  if (few) {
    const int64_t threads = 2 * a.r * (a.K / 8) + a.N * ((a.r + 7) / 8);
    k_gated_few_grad<<<static_cast<unsigned>(ceil_div(threads, 256)), 256, 0, s>>>(fp);
  } else if (pl.rp) {
    GradParams g{};
    g.X = X;
    g.d[0] = b.dG;
    g.d[1] = b.dU;
    g.Hs = Hs;
    g.low = b.low;
    g.a_part = b.ga;
    g.b_part = b.gb;
    for (int w = 0; w < 2; ++w) g.dA[w] = dA[w], g.dB[w] = dB[w];
    g.bf16 = a.adapter_bf16;
    g.r = a.r;
    g.M = a.M;
    g.N = a.N;
    g.K = a.K;
    g.rp = pl.rp;
    g.a_tiles_c = static_cast<int>(grid_blocks(a.K, 256));
    g.a_tiles = g.a_tiles_c * (2 * pl.rp / 64);
    g.a_splits = pl.ga.splits;
    g.a_steps = pl.ga.steps_per_split;
    g.b_tiles_c = pl.rp / 64;
    g.b_tiles = g.b_tiles_c * static_cast<int>(grid_blocks(a.N, 256));
    g.b_splits = pl.gb.splits;
    g.b_steps = pl.gb.steps_per_split;
    k_gated_grad<<<static_cast<unsigned>(g.a_tiles * g.a_splits + 2 * g.b_tiles * g.b_splits), 256, 0, s>>>(g);
    if (!b.ga && !b.gb) return hipGetLastError();
    const GradSumParams q{b.ga, b.gb, {dA[0], dA[1]}, {dB[0], dB[1]}, a.adapter_bf16, a.N, a.K, a.r, pl.rp, pl.ga.splits, pl.gb.splits};
    const int64_t count = 2 * a.r * ((b.gb ? a.N : 0) + (b.ga ? a.K : 0));
    k_gated_grad_sum<<<static_cast<unsigned>(std::min<int64_t>(ceil_div(count, 256), 4096)), 256, 0, s>>>(q);
  }
  return hipGetLastError();
}

}  // namespace qnf4
