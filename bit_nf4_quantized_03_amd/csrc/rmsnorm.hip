// RMSNorm with the residual's addition, forward (bf16 or microscaled output)
// and backward.
//
//   h = bf16(x + residual), rstd = 1 / sqrt(mean(h^2) + eps), y = h rstd w
//   u = h rstd, g = dy w:  dx = rstd (g - u mean(g u)) + dh,  dw = sum dy u
//
// A row is read once: a lane keeps its elements in registers between the sum
// and the scaling. It holds runs of eight elements, so a block of 32 of the
// microscaled output lies in a quad of lanes.
//
// The forward computes in fp64. That costs two fp64 operations an element for
// the sum and two for the scaling, at the fp32 rate of this card's vector
// units, under a memory-bound kernel, and it decides every rounding to 8 or 4
// bits as the definition does: with an fp32 sum, values within an ulp of a
// rounding border land on either side.
#include <algorithm>

#include "mx_device.h"

namespace qnf4 {
namespace {

constexpr int kOutBf16 = 2;   // besides the qlora_mx_type outputs

struct FwdParams {
  const __bf16 *x, *res;
  const void *w;
  __bf16 *y, *h;
  uint8_t *codes, *scales;
  float *rstd;
  int64_t rows, group0;   // group0: the launch's first workgroup
  double eps, inv_cols;
  uint32_t cols, pitch;
  bool w_bf16;
};

// fp64 -> fp32 keeping 20 bits of mantissa, the last one set when anything
// below it was: rounding the result to 8 or fewer bits of mantissa gives what
// rounding the fp64 value gives.
__device__ __forceinline__ float sticky_f32(double d) {
  const uint64_t b = __builtin_bit_cast(uint64_t, d);
  const uint64_t hi = (b & 0xffffffff00000000ull) | (static_cast<uint32_t>(b) != 0 ? 0x100000000ull : 0ull);
  return static_cast<float>(__builtin_bit_cast(double, hi));
}

__device__ __forceinline__ void unpack8(const mx_u32x4 &r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(r[i]);
    v[2 * i + 1] = bf16_hi(r[i]);
  }
}

__device__ __forceinline__ mx_u32x4 pack8(const float (&v)[8]) {
  mx_u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    mx_bf16x2 p;
    p[0] = static_cast<__bf16>(v[2 * i]);
    p[1] = static_cast<__bf16>(v[2 * i + 1]);
    r[i] = __builtin_bit_cast(uint32_t, p);
  }
  return r;
}

__device__ __forceinline__ mx_u32x4 load_row8(const __bf16 *p, int64_t at) {
  return __builtin_nontemporal_load(reinterpret_cast<const mx_u32x4 *>(p + at));
}

// Eight weights from col on (a clamped, valid place where col is behind the
// row's end: those lanes store nothing).
__device__ __forceinline__ void load_weight8(const void *w, bool bf16, uint32_t col, uint32_t cols, float (&v)[8]) {
  col = min(col, cols - 8);
  if (bf16) {
    const mx_u32x4 r = *reinterpret_cast<const mx_u32x4 *>(static_cast<const __bf16 *>(w) + col);
    unpack8(r, v);
  } else {
    const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(w) + col);
    const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(w) + col + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

// A thread's runs of a row; lanes behind the row's end hold zeros.
template <int T, int NV>
__device__ __forceinline__ void load_runs(mx_u32x4 (&v)[NV], const __bf16 *p, int64_t base, uint32_t cols, int t) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t col = 8u * (i * T + t);
    v[i] = col < cols ? load_row8(p, base + col) : mx_u32x4{0, 0, 0, 0};
  }
}

// Sum over the T threads of a row, in every one of them. part: the row's
// T / 64 slots of shared memory (T > 64), free again when the next call but
// one begins.
template <int T, class F>
__device__ __forceinline__ F row_sum(F v, F *part) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x % T >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int i = 1; i < T / 64; ++i) v += part[i];
  }
  return v;
}

// A workgroup of THREADS takes R = THREADS / T rows, T threads to a row with up
// to NV runs of eight elements each. Bound by memory for many rows (4096 x 4096
// with residual 25.3 us into bf16, 5.3 TB/s, 26.7 into 8 bits, 4.4), by the
// round trip of its loads and the sum for a few (1 x 4096 2.8 us). These are
// times of the kernel alone; those of two forms below are of calls in a row.
template <int T, int THREADS, int NV, int OUT>
__global__ __launch_bounds__(THREADS) void k_rms_fwd(const FwdParams p) {
  __shared__ double part[THREADS / 64];
  const int t = threadIdx.x % T, sub = threadIdx.x / T;
  const int64_t row = (p.group0 + blockIdx.x) * (THREADS / T) + sub;
  const bool live = row < p.rows;
  // rows past the end are read from the last one and stored nowhere
  const int64_t base = min(row, p.rows - 1) * p.cols;
  mx_u32x4 x[NV], res[NV];
  load_runs<T>(x, p.x, base, p.cols, t);
  if (p.res) load_runs<T>(res, p.res, base, p.cols, t);
  // With two runs a thread the weights are loaded before the sum (4096 x 4096
  // into 8 bits 24.7 -> 24.1 us, without a residual into bf16 16.5 -> 15.8); with
  // more that costs the registers of other rows (777 x 8192 14.3 -> 14.7).
  constexpr bool kEarly = NV == 2;
  float w[NV][8];
  const auto weights = [&](int i) { load_weight8(p.w, p.w_bf16, 8u * (i * T + t), p.cols, w[i]); };
  if (kEarly) {
#pragma unroll
    for (int i = 0; i < NV; ++i) weights(i);
  }
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float a[8];
    unpack8(x[i], a);
    if (p.res) {
      // fp32 holds enough of the sum of two bf16 that rounding it again is
      // rounding the exact sum
      float b[8];
      unpack8(res[i], b);
#pragma unroll
      for (int k = 0; k < 8; ++k) a[k] += b[k];
      x[i] = pack8(a);
      const uint32_t col = 8u * (i * T + t);
      if (live && col < p.cols) __builtin_nontemporal_store(x[i], reinterpret_cast<mx_u32x4 *>(p.h + base + col));
      unpack8(x[i], a);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = __builtin_fma(static_cast<double>(a[k]), static_cast<double>(a[k]), ss);
  }
  ss = row_sum<T>(ss, part + sub * (T / 64));
  const double rstd = 1.0 / sqrt(ss * p.inv_cols + p.eps);
  if (!live) return;
  if (p.rstd && t == 0) p.rstd[row] = static_cast<float>(rstd);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t col = 8u * (i * T + t);
    if (col >= p.cols) continue;   // whole quads
    float a[8], y[8];
    unpack8(x[i], a);
    if (!kEarly) weights(i);
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = sticky_f32(static_cast<double>(a[k]) * rstd * static_cast<double>(w[i][k]));
    if constexpr (OUT == kOutBf16) {
      __builtin_nontemporal_store(pack8(y), reinterpret_cast<mx_u32x4 *>(p.y + base + col));
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = max(m, __builtin_bit_cast(uint32_t, y[k]) & 0x7fffffffu);
      const uint32_t s = mx_scale_byte<OUT>(quad_max(m));
      const uint2 c = mx_encode8<OUT>(y, mx_scale_value(s));
      if constexpr (OUT == QLORA_MX_FP4) {
        *reinterpret_cast<uint32_t *>(p.codes + ((base + col) >> 1)) = c.x;
      } else {
        *reinterpret_cast<uint2 *>(p.codes + base + col) = c;
      }
      if ((t & 3) == 0) p.scales[row * p.pitch + (col >> 5)] = static_cast<uint8_t>(s);
    }
  }
  if constexpr (OUT != kOutBf16) {
    // the pad bytes behind the row's scales (at most 15)
    const uint32_t at = (p.cols >> 5) + t;
    if (at < p.pitch) p.scales[row * p.pitch + at] = 0;
  }
}

struct BwdParams {
  const __bf16 *dy, *h, *dh;
  const void *w;
  const float *rstd;
  __bf16 *dx;
  float *part;   // [workgroups][cols]
  int64_t rows;
  float inv_cols;
  uint32_t cols;
  bool w_bf16;
};

// R rows at a time as in the forward, rows b R .. for workgroup b, then G R
// further on for a grid of G. A thread keeps the sums of dy u of its columns
// over its rows; the R sums of a column are added in order through LDS, so that
// a workgroup writes one row of partial sums. Bound by memory: 4096 x 4096 with
// dh 25.0 us, 5.4 TB/s of the 134 MB that the rows are, and 4.5 for k_rms_dw.
// Where the registers are there, the next rows' loads are under way while the
// current ones are worked on, and the weights stay in registers (loaded again
// twice a row they were more bytes than the row; calls in a row, both kernels:
// 4096 x 4096 32 us against 28, 4096 x 8192 58 against 49). 300 x 24576: 29.0 us.
template <int T, int THREADS, int NV>
__global__ __launch_bounds__(THREADS) void k_rms_bwd(const BwdParams p) {
  constexpr int R = THREADS / T;
  constexpr bool kAhead = NV == 1;
  constexpr bool kKeep = NV <= 2;   // weights in registers
  __shared__ float part[2][THREADS / 64];
  __shared__ float4 sums[R > 1 ? NV * T * 2 : 1];
  int t = threadIdx.x % T;
  const int sub = threadIdx.x / T;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * R;
  int64_t first = static_cast<int64_t>(blockIdx.x) * R;
  const auto row_of = [&](int64_t f) { return min(f + sub, p.rows - 1); };
  float dw[NV][8] = {};
  mx_u32x4 dy[NV], h[NV], dh[NV], next_dy[NV], next_h[NV], next_dh[NV];
  float rstd, next_rstd = 0.0f;
  const auto load = [&](int64_t f) {
    const int64_t row = row_of(f);
    next_rstd = p.rstd[row];
    load_runs<T>(next_dy, p.dy, row * p.cols, p.cols, t);
    load_runs<T>(next_h, p.h, row * p.cols, p.cols, t);
    if (p.dh && kKeep) load_runs<T>(next_dh, p.dh, row * p.cols, p.cols, t);
  };
  if (kAhead) load(first);
  float w[NV][8];
  const auto weights = [&](int i) { load_weight8(p.w, p.w_bf16, 8u * (i * T + t), p.cols, w[i]); };
  if (kKeep) {
#pragma unroll
    for (int i = 0; i < NV; ++i) weights(i);
  }
  for (int flip = 0; first < p.rows; first += stride, flip ^= 1) {
    const bool live = R == 1 || first + sub < p.rows;   // the same in a row's threads
    const int64_t base = row_of(first) * p.cols;
    if (!kKeep) asm volatile("" : "+v"(t));   // the columns' addresses are formed again in each turn, not kept
    if (!kAhead) load(first);
    rstd = next_rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      dy[i] = next_dy[i], h[i] = next_h[i];
      if (kKeep) dh[i] = next_dh[i];
    }
    if (kAhead && first + stride < p.rows) load(first + stride);
    float c = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float a[8], b[8];
      unpack8(dy[i], a);
      unpack8(h[i], b);
      if (!kKeep) __builtin_amdgcn_sched_barrier(0), weights(i);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float du = a[k] * (b[k] * rstd);
        if (live) dw[i][k] += du;
        c = __builtin_fmaf(du, w[i][k], c);
      }
    }
    c = row_sum<T>(c, part[flip] + sub * (T / 64)) * p.inv_cols;
    if (!live) continue;
    if (!kKeep) {
      // the row stays packed: without this the compiler keeps it as fp32 for
      // the second use and spills most of it (300 x 24576, both kernels, 65 us
      // against 35; six registers of 1024 threads' 128 are still spilled)
#pragma unroll
      for (int i = 0; i < NV; ++i) asm volatile("" : "+v"(dy[i]), "+v"(h[i]));
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t col = 8u * (i * T + t);
      if (col < p.cols) {
        float a[8], b[8], d[8];
        unpack8(dy[i], a);
        unpack8(h[i], b);
        if (!kKeep) {
          __builtin_amdgcn_sched_barrier(0);
          weights(i);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] = rstd * (a[k] * w[i][k] - b[k] * rstd * c);
        if (p.dh) {
          unpack8(kKeep ? dh[i] : load_row8(p.dh, base + col), d);
#pragma unroll
          for (int k = 0; k < 8; ++k) a[k] += d[k];
        }
        __builtin_nontemporal_store(pack8(a), reinterpret_cast<mx_u32x4 *>(p.dx + base + col));
      }
    }
  }
  if constexpr (R > 1) {
    for (int s = 1; s < R; ++s) {
      if (sub == s) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          sums[(2 * i) * T + t] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
          sums[(2 * i + 1) * T + t] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        }
      }
      __syncthreads();
      if (sub == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const float4 u = sums[(2 * i) * T + t], v = sums[(2 * i + 1) * T + t];
          dw[i][0] += u.x, dw[i][1] += u.y, dw[i][2] += u.z, dw[i][3] += u.w;
          dw[i][4] += v.x, dw[i][5] += v.y, dw[i][6] += v.z, dw[i][7] += v.w;
        }
      }
      __syncthreads();
    }
    if (sub != 0) return;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t col = 8u * (i * T + t);
    if (col < p.cols) {
      float4 *o = reinterpret_cast<float4 *>(p.part + static_cast<int64_t>(blockIdx.x) * p.cols + col);
      o[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
      o[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
    }
  }
}

// dw[c] = sum over the groups of part[g][c]: a workgroup takes 32 columns,
// thread (column c, slice s of 32) the groups s, s + 32, ...; slices are added
// in order. fp64, so that the order over many groups costs no accuracy.
__global__ __launch_bounds__(1024) void k_rms_dw(const float *part, float *dw, int groups, uint32_t cols) {
  __shared__ double sum[32][32];
  const int c = threadIdx.x & 31, s = threadIdx.x >> 5;
  const uint32_t col = blockIdx.x * 32 + c;   // cols is a multiple of 32
  double v = 0.0;
#pragma unroll 8
  for (int g = s; g < groups; g += 32) v += part[static_cast<int64_t>(g) * cols + col];
  sum[s][c] = v;
  __syncthreads();
  if (s == 0) {
#pragma unroll
    for (int i = 1; i < 32; ++i) v += sum[i][c];
    dw[col] = static_cast<float>(v);
  }
}

template <int T, int THREADS, int NV>
hipError_t fwd_run(FwdParams p, int out, hipStream_t s) {
  const int64_t groups = ceil_div(p.rows, THREADS / T);
  for (p.group0 = 0; p.group0 < groups; p.group0 += kMaxGroups) {
    const unsigned g = static_cast<unsigned>(std::min(groups - p.group0, kMaxGroups));
    if (out == QLORA_MX_FP4) k_rms_fwd<T, THREADS, NV, QLORA_MX_FP4><<<g, THREADS, 0, s>>>(p);
    else if (out == QLORA_MX_FP8) k_rms_fwd<T, THREADS, NV, QLORA_MX_FP8><<<g, THREADS, 0, s>>>(p);
    else k_rms_fwd<T, THREADS, NV, kOutBf16><<<g, THREADS, 0, s>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Rows of a backward workgroup at a time (1024 threads).
int bwd_rows(int64_t cols) { return cols <= 512 ? 16 : cols <= 1024 ? 8 : cols <= 2048 ? 4 : cols <= 4096 ? 2 : 1; }

// Workgroups of the backward, and rows of partial dw sums: at most one per
// compute unit, so that the sums stay small beside the rows (two a unit cost
// 4096 x 4096 three and 4096 x 8192 five us more), and no more than are needed
// to have the rows done in as many turns. Up to 8192 columns a thread has one
// run of a row (two, with two rows at a time: 4096 x 8192 52 us against 49).
unsigned bwd_groups(int64_t rows, int64_t cols) {
  const int64_t turns = ceil_div(rows, bwd_rows(cols));
  return static_cast<unsigned>(ceil_div(turns, ceil_div(turns, 256)));
}

template <int T, int NV>
void bwd_run(const BwdParams &p, unsigned groups, hipStream_t s) {
  k_rms_bwd<T, 1024, NV><<<groups, 1024, 0, s>>>(p);
}

}  // namespace

hipError_t launch_rms_fwd(const RmsFwd &a, hipStream_t s) {
  FwdParams p;
  p.x = static_cast<const __bf16 *>(a.X);
  p.res = static_cast<const __bf16 *>(a.residual);
  p.w = a.weight;
  p.w_bf16 = a.w_bf16;
  p.y = static_cast<__bf16 *>(a.Y);
  p.h = static_cast<__bf16 *>(a.H);
  p.codes = a.codes;
  p.scales = a.scales;
  p.rstd = a.rstd;
  p.rows = a.rows;
  p.cols = static_cast<uint32_t>(a.cols);
  p.pitch = static_cast<uint32_t>(mx_pitch(a.cols));
  p.eps = a.eps;
  p.inv_cols = 1.0 / static_cast<double>(a.cols);
  const int out = a.codes ? a.type : kOutBf16;
  // Few rows: the most threads to a row (1 x 4096, calls in a row, 3.3 us
  // against 3.8 with 256). Many: 256 threads of two or four runs keep more loads in flight (777 x 8192
  // into 8 bits without a residual 10.1 us against 10.8).
  const bool few = a.rows < 512;
  if (a.cols <= 512) return fwd_run<64, 256, 1>(p, out, s);
  if (a.cols <= 1024) return fwd_run<128, 256, 1>(p, out, s);
  if (a.cols <= 2048) return fwd_run<256, 256, 1>(p, out, s);
  if (a.cols <= 4096) return few ? fwd_run<512, 512, 1>(p, out, s) : fwd_run<256, 256, 2>(p, out, s);
  if (a.cols <= 8192) return few ? fwd_run<1024, 1024, 1>(p, out, s) : fwd_run<256, 256, 4>(p, out, s);
  if (a.cols <= 16384) return fwd_run<1024, 1024, 2>(p, out, s);
  return fwd_run<1024, 1024, 4>(p, out, s);
}

size_t rms_bwd_ws_bytes(int64_t rows, int64_t cols) {
  const unsigned groups = bwd_groups(rows, cols);
  return groups > 1 ? static_cast<size_t>(groups) * static_cast<size_t>(cols) * sizeof(float) : 0;
}

hipError_t launch_rms_bwd(const void *dY, const void *H, const void *weight, bool w_bf16, const float *rstd,
                          const void *dH, int64_t rows, int64_t cols, void *dX, float *dW, void *ws, hipStream_t s) {
  BwdParams p;
  p.dy = static_cast<const __bf16 *>(dY);
  p.h = static_cast<const __bf16 *>(H);
  p.dh = static_cast<const __bf16 *>(dH);
  p.w = weight;
  p.w_bf16 = w_bf16;
  p.rstd = rstd;
  p.dx = static_cast<__bf16 *>(dX);
  p.rows = rows;
  p.cols = static_cast<uint32_t>(cols);
  p.inv_cols = 1.0f / static_cast<float>(cols);
  const unsigned groups = bwd_groups(rows, cols);
  p.part = groups > 1 ? static_cast<float *>(ws) : dW;   // one workgroup: its sums are dW
  if (cols <= 512) bwd_run<64, 1>(p, groups, s);
  else if (cols <= 1024) bwd_run<128, 1>(p, groups, s);
  else if (cols <= 2048) bwd_run<256, 1>(p, groups, s);
  else if (cols <= 4096) bwd_run<512, 1>(p, groups, s);
  else if (cols <= 8192) bwd_run<1024, 1>(p, groups, s);
  else if (cols <= 16384) bwd_run<1024, 2>(p, groups, s);
  else bwd_run<1024, 4>(p, groups, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || groups == 1) return e;
  k_rms_dw<<<static_cast<unsigned>(cols / 32), 1024, 0, s>>>(p.part, dW, static_cast<int>(groups), p.cols);
  return hipGetLastError();
}

}  // namespace qnf4
