// Rotary positions of queries and keys, and their gradient.
//
// Pair i of a head, (a, b), of the token at position t becomes
//     (a cos w - b sin w, b cos w + a sin w) * amplitude,   w = t f_i,
// the gradient the same with -w. A pair is elements i and i + rot / 2 of the
// head, or its neighbours 2 i and 2 i + 1; elements from rot on pass through.
//
// The angle: t f_i / (2 pi) in fp64, less the nearest whole number, is a turn
// in [-1/2, 1/2]. Three roundings of 2^-53 (of 1 / (2 pi), of f_i times that and
// of t times that) leave it off by 3 * 2^-53 of its turns, 2^-23 turns at t =
// 2^31 and f = 1; in fp32 the product alone would be off by 2^-24 of t f_i, a
// tenth of a radian at a million positions. The sine and cosine of that turn
// and the rotation are fp32, the result is rounded once.
//
// Bound by HBM: each element is read and written once. A workgroup has a few
// tokens, forms their sines and cosines once for all heads in LDS (a head's
// worth of them per token, which is little beside 40 heads) and then moves 16
// bytes of each half of a pair run per step and lane.
#include <algorithm>

#include "block.h"
#include "mx_device.h"

namespace qnf4 {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTable = 2048;   // pairs of a workgroup's tokens, 16 KB of LDS

struct RopeParams {
  RopeHeads q, k;
  const void *positions;
  const double *freqs;
  int64_t first, rows;         // token that the launch begins with
  int heads, dim, half;        // of q and k together; rot / 2
  int tokens, chunk;           // of a workgroup; heads of one
  int units, rot_units;        // of a head: P pairs or 2 P elements that pass through
  uint32_t by_units, by_chunk; // reciprocals: x / d = hi32(x r) for x d < 2^32
  float amplitude;             // negative angle: sine < 0
  bool wide, neighbours, back;
};

// Sixteen bytes at a time or one element.
template <class E, int P>
struct RopeIo;
template <>
struct RopeIo<float, 4> {
  static __device__ __forceinline__ void load(const float *p, float (&v)[4]) {
    const float4 a = *reinterpret_cast<const float4 *>(p);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  }
  static __device__ __forceinline__ void store(float *p, const float (&v)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct RopeIo<__bf16, 8> {
  static __device__ __forceinline__ void load(const __bf16 *p, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(w[i]), v[2 * i + 1] = bf16_hi(w[i]);
  }
  static __device__ __forceinline__ void store(__bf16 *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const mx_bf16x2 b = {static_cast<__bf16>(v[2 * i]), static_cast<__bf16>(v[2 * i + 1])};
      w[i] = __builtin_bit_cast(uint32_t, b);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <class E>
struct RopeIo<E, 1> {
  static __device__ __forceinline__ void load(const E *p, float (&v)[1]) { v[0] = static_cast<float>(*p); }
  static __device__ __forceinline__ void store(E *p, const float (&v)[1]) { *p = static_cast<E>(v[0]); }
};

template <class E, int P>
__global__ __launch_bounds__(kRopeThreads) void k_rope(const RopeParams p) {
  __shared__ float2 table[kRopeTable];   // cosine and sine, times the amplitude
  const int64_t t0 = p.first + static_cast<int64_t>(blockIdx.x) * p.tokens;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(p.tokens), p.rows - t0));
  const int h0 = static_cast<int>(blockIdx.y) * p.chunk;
  for (int t = 0; t < tokens; ++t) {
    const double at = p.wide ? static_cast<double>(static_cast<const int64_t *>(p.positions)[t0 + t])
                             : static_cast<double>(static_cast<const int32_t *>(p.positions)[t0 + t]);
    for (int i = threadIdx.x; i < p.half; i += kRopeThreads) {
      const double turns = at * (p.freqs[i] * 0.15915494309189533577);
      float s, c;
      sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &s, &c);
      table[t * p.half + i] = make_float2(c * p.amplitude, (p.back ? -s : s) * p.amplitude);
    }
  }
  __syncthreads();
  const int heads = min(p.chunk, p.heads - h0);
  // head fastest behind the units, all of a token's heads before the next one's
  const uint32_t items = static_cast<uint32_t>(tokens) * p.chunk * p.units;
  for (uint32_t i = threadIdx.x; i < items; i += kRopeThreads) {
    const uint32_t unit_row = p.units == 1 ? i : __umulhi(i, p.by_units);
    const int u = static_cast<int>(i - unit_row * p.units);
    const uint32_t t = p.chunk == 1 ? unit_row : __umulhi(unit_row, p.by_chunk);
    const int in = static_cast<int>(unit_row - t * p.chunk);
    if (in >= heads) continue;
    const int h = h0 + in;
    const bool is_q = h < p.q.heads;
    const RopeHeads &x = is_q ? p.q : p.k;
    const int64_t head = is_q ? h : h - p.q.heads, row = t0 + t;
    const E *src = static_cast<const E *>(x.in) + row * x.in_row + head * x.in_head;
    E *dst = static_cast<E *>(x.out) + row * x.out_row + head * x.out_head;
    float a[P], b[P];
    int ia, ib;
    if (u >= p.rot_units) {
      ia = 2 * p.half + 2 * P * (u - p.rot_units);
      ib = ia + P;
    } else if (p.neighbours) {
      ia = 2 * P * u;
      ib = ia + P;
    } else {
      ia = P * u;
      ib = ia + p.half;
    }
    RopeIo<E, P>::load(src + ia, a);
    RopeIo<E, P>::load(src + ib, b);
    if (u < p.rot_units) {
      const float2 *cs = table + t * p.half + P * u;
      if (p.neighbours && P > 1) {
        // pairs lie in order: P / 2 in the first run, P / 2 in the second
#pragma unroll
        for (int e = 0; e < P; e += 2) {
          const float2 w = cs[e / 2], z = cs[P / 2 + e / 2];
          const float x0 = a[e], y0 = a[e + 1 < P ? e + 1 : e], x1 = b[e], y1 = b[e + 1 < P ? e + 1 : e];
          a[e] = fmaf(x0, w.x, -(y0 * w.y));
          a[e + 1 < P ? e + 1 : e] = fmaf(y0, w.x, x0 * w.y);
          b[e] = fmaf(x1, z.x, -(y1 * z.y));
          b[e + 1 < P ? e + 1 : e] = fmaf(y1, z.x, x1 * z.y);
        }
      } else {
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float2 w = cs[e];
          const float x0 = a[e], y0 = b[e];
          a[e] = fmaf(x0, w.x, -(y0 * w.y));
          b[e] = fmaf(y0, w.x, x0 * w.y);
        }
      }
    }
    RopeIo<E, P>::store(dst + ia, a);
    RopeIo<E, P>::store(dst + ib, b);
  }
}

// ceil(2^32 / d): hi32(x r) = x / d for 0 <= x < 2^16 and 2 <= d <= 2^16, since
// x (r d - 2^32) < x d <= 2^32.
uint32_t reciprocal(uint32_t d) { return static_cast<uint32_t>(((uint64_t(1) << 32) + d - 1) / d); }

template <class E, int P>
hipError_t run_rope(RopeParams p, bool copies, hipStream_t s) {
  p.rot_units = p.half / P;
  p.units = p.rot_units + (copies ? (p.dim - 2 * p.half) / (2 * P) : 0);
  // about two steps a lane where there is work for it, one in a small call (4096
  // tokens of 40 heads, bf16: 20.8, 18.8, 18.8 and 21.8 us with one, two, four
  // and eight; fp32 both directions 47.1, 49.5, 52.7, 54.2). Two steps' loads
  // ahead of their use were slower: 25.8 us, fewer waves have room.
  const int64_t all = p.rows * p.heads * p.units;
  const int target = all >= int64_t(1) << 19 ? 2 * kRopeThreads : kRopeThreads;
  p.chunk = std::max(1, std::min(p.heads, target / p.units));
  p.tokens = static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>({target / (p.chunk * p.units), kRopeTable / std::max(p.half, 1), p.rows})));
  p.by_units = reciprocal(p.units);
  p.by_chunk = reciprocal(p.chunk);
  const unsigned by_head = static_cast<unsigned>(ceil_div(p.heads, p.chunk));
  const int64_t most = std::max<int64_t>(1, kMaxGroups / by_head);
  for (; p.first < p.rows; p.first += most * p.tokens) {
    const int64_t groups = std::min(ceil_div(p.rows - p.first, p.tokens), most);
    k_rope<E, P><<<dim3(static_cast<unsigned>(groups), by_head), kRopeThreads, 0, s>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_rope(const Rope &a, hipStream_t s) {
  RopeParams p{};
  p.q = a.q;
  p.k = a.k;
  p.positions = a.positions;
  p.freqs = a.freqs;
  p.rows = a.rows;
  p.heads = static_cast<int>(a.q.heads + a.k.heads);
  p.dim = a.dim;
  p.half = a.rot / 2;
  p.amplitude = static_cast<float>(a.amplitude);
  p.wide = a.wide_positions;
  p.neighbours = a.interleaved;
  p.back = a.backward;
  const int size = a.bf16 ? 2 : 4, run = 16 / size;
  // where nothing moves, what passes through is in its place already
  const auto same = [](const RopeHeads &x) { return x.heads == 0 || (x.in == x.out && x.in_row == x.out_row && x.in_head == x.out_head); };
  const bool copies = p.dim > 2 * p.half && !(same(a.q) && same(a.k));
  // 16 bytes at a time: every run of a head starts aligned
  const auto aligned = [&](const RopeHeads &x) {
    if (x.heads == 0) return true;
    const uintptr_t at = reinterpret_cast<uintptr_t>(x.in) | reinterpret_cast<uintptr_t>(x.out);
    return at % 16 == 0 && (x.in_row | x.in_head | x.out_row | x.out_head) % run == 0;
  };
  const bool whole = p.half % run == 0 && (!copies || (p.dim - 2 * p.half) % (2 * run) == 0) && aligned(a.q) && aligned(a.k);
  if (a.bf16) return whole ? run_rope<__bf16, 8>(p, copies, s) : run_rope<__bf16, 1>(p, copies, s);
  return whole ? run_rope<float, 4>(p, copies, s) : run_rope<float, 1>(p, copies, s);
}

}  // namespace qnf4
