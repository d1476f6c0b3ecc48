// C ABI of what stands between a decoder layer's projections: argument checks
// and dispatch. Every check runs on the host before anything is launched; a
// failed check launches nothing.
#include <cmath>
#include <cstdint>
#include <limits>

#include "../../include/qlora_block.h"
#include "block.h"
#include "error.h"

namespace {

using qnf4::api_fail;

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

long long ll(int64_t v) { return static_cast<long long>(v); }

// The checks that both gated products share and their arguments; n: rows of
// one pair.
int gated_args(const char *fn, const qlora_mx_matrix *X, const qlora_mx_matrix *W, int64_t n, void *H,
               const qlora_mx_matrix *Hq, qnf4::MxLinear *a) {
  if ((H == nullptr) == (Hq == nullptr)) return api_fail(QLORA_ERR_NULL, "%s: exactly one of H and Hq is given", fn);
  if (!aligned(H, 16)) return api_fail(QLORA_ERR_ALIGN, "%s: H must be 16-byte aligned", fn);
  if (W->type != QLORA_MX_FP4) return api_fail(QLORA_ERR_FORMAT, "%s: W must hold 4-bit elements", fn);
  if (X->cols != W->cols)
    return api_fail(QLORA_ERR_SHAPE, "%s: X has %lld columns but W has %lld", fn, ll(X->cols), ll(W->cols));
  if (n % (2 * QLORA_MX_BLOCK) != 0)
    return api_fail(QLORA_ERR_SHAPE, "%s: a pair of %lld rows: needs a multiple of %d", fn, ll(n), 2 * QLORA_MX_BLOCK);
  if (X->rows > qnf4::kMxMaxRows || n > qnf4::kMxMaxRows || X->rows > qnf4::kMxMaxOut / n || n / 2 > qnf4::kMxMaxK)
    return api_fail(QLORA_ERR_SHAPE, "%s: %lld rows by a pair of %lld are too large", fn, ll(X->rows), ll(n));
  if (Hq) {
    const int st = qnf4::api_check_matrix(fn, "Hq", Hq);
    if (st != QLORA_OK) return st;
    if (Hq->rows != X->rows || Hq->cols != n / 2)
      return api_fail(QLORA_ERR_SHAPE, "%s: Hq is %lld x %lld, not %lld x %lld", fn, ll(Hq->rows), ll(Hq->cols),
                      ll(X->rows), ll(n / 2));
  }
  *a = qnf4::MxLinear{};
  a->M = X->rows;
  a->N = n;
  a->K = X->cols;
  a->x_type = X->type;
  a->x = X->codes;
  a->xs = X->scales;
  a->w = W->codes;
  a->ws = W->scales;
  a->Y = H;
  return QLORA_OK;
}

int gated(const char *fn, const qnf4::MxLinear &a, const qlora_mx_matrix *Hq, bool clear, void *stream) {
  return qnf4::api_hip_status(qnf4::launch_mx_gated(a, Hq ? Hq->codes : nullptr, Hq ? Hq->scales : nullptr,
                                                    Hq ? Hq->type : 0, clear, static_cast<hipStream_t>(stream)), fn);
}

bool valid_gated(int64_t M, int64_t N, int64_t K, int32_t r) {
  return M >= 1 && M <= qnf4::kGatedMaxRows && N >= 1 && K >= 1 && N <= qnf4::kGatedMaxDim && K <= qnf4::kGatedMaxDim &&
         N % QLORA_NF4_BLOCK == 0 && K % QLORA_NF4_BLOCK == 0 && M <= qnf4::kGatedMaxOut / N && M <= qnf4::kGatedMaxOut / K &&
         N <= qnf4::kGatedMaxOut / K && r >= 0 && r <= 256;
}

// The checks that both passes of the block with adapters share, and their arguments.
int block_args(const char *fn, int64_t M, const qlora_nf4_weight *gate, const qlora_nf4_weight *up,
               const qlora_gated_adapters *ad, bool backward, const void *ws, size_t ws_bytes, qnf4::GatedArgs *a) {
  int st = qnf4::api_check_weight(gate, fn);
  if (st == QLORA_OK) st = qnf4::api_check_weight(up, fn);
  if (st != QLORA_OK) return st;
  if (gate->rows != up->rows || gate->cols != up->cols)
    return api_fail(QLORA_ERR_SHAPE, "%s: the weights are %lld x %lld and %lld x %lld", fn, ll(gate->rows), ll(gate->cols),
                    ll(up->rows), ll(up->cols));
  if (gate->format != up->format)
    return api_fail(QLORA_ERR_FORMAT, "%s: the weights' formats %d and %d differ", fn, gate->format, up->format);
  const int32_t r = ad ? ad->r : 0;
  if (ad && (r < 1 || r > 256)) return api_fail(QLORA_ERR_SHAPE, "%s: r = %d out of [1, 256]", fn, r);
  if (!valid_gated(M, gate->rows, gate->cols, r))
    return api_fail(QLORA_ERR_SHAPE, "%s: M = %lld, N = %lld, K = %lld: needs M >= 1, N and K multiples of %d, and sizes within the limits",
                    fn, ll(M), ll(gate->rows), ll(gate->cols), QLORA_NF4_BLOCK);
  *a = qnf4::GatedArgs{};
  if (ad) {
    if (ad->dtype != QLORA_F32 && ad->dtype != QLORA_BF16)
      return api_fail(QLORA_ERR_DTYPE, "%s: the adapters' dtype %d is not QLORA_F32 or QLORA_BF16", fn, ad->dtype);
    const void *const all[4] = {ad->gate_A, ad->gate_B, ad->up_A, ad->up_B};
    for (const void *p : all) {
      if (!p) return api_fail(QLORA_ERR_NULL, "%s: a factor of the adapters is NULL", fn);
      if (!aligned(p, 16)) return api_fail(QLORA_ERR_ALIGN, "%s: the adapters' factors must be 16-byte aligned", fn);
    }
    if (!std::isfinite(ad->scale)) return api_fail(QLORA_ERR_SHAPE, "%s: scale must be finite", fn);
    a->A[0] = ad->gate_A, a->B[0] = ad->gate_B, a->A[1] = ad->up_A, a->B[1] = ad->up_B;
    a->adapter_bf16 = ad->dtype == QLORA_BF16;
    a->scale = ad->scale;
  }
  a->M = M;
  a->N = gate->rows;
  a->K = gate->cols;
  a->format = gate->format;
  a->r = r;
  const qlora_nf4_weight *const both[2] = {gate, up};
  for (int i = 0; i < 2; ++i)
    a->w[i] = {both[i]->codes, both[i]->absmax_q, both[i]->dq_scale, both[i]->dq_mean, both[i]->absmax};
  const size_t need = qnf4::gated_ws_bytes(M, a->N, a->K, r, backward);
  if (need > 0 && (!ws || ws_bytes < need))
    return api_fail(QLORA_ERR_WORKSPACE, "%s: workspace needs %zu bytes, got %zu", fn, need, ws ? ws_bytes : size_t(0));
  if (!aligned(ws, 16)) return api_fail(QLORA_ERR_ALIGN, "%s: workspace must be 16-byte aligned", fn);
  return QLORA_OK;
}

int check_heads(const char *fn, const char *name, const qlora_rope_heads *x, int64_t rows, int32_t dim, int size) {
  if (!x->in || !x->out) return api_fail(QLORA_ERR_NULL, "%s: a buffer of %s is NULL", fn, name);
  if (!aligned(x->in, size) || !aligned(x->out, size))
    return api_fail(QLORA_ERR_ALIGN, "%s: the buffers of %s must be aligned to their elements", fn, name);
  if (x->heads < 1 || x->heads > qnf4::kRopeMaxHeads)
    return api_fail(QLORA_ERR_SHAPE, "%s: %s has %lld heads, not 1 to %lld", fn, name, ll(x->heads), ll(qnf4::kRopeMaxHeads));
  constexpr int64_t kMost = int64_t(1) << 46;   // elements between the first and the last
  for (int64_t stride : {x->in_row, x->in_head, x->out_row, x->out_head})
    if (stride < 0 || stride > kMost) return api_fail(QLORA_ERR_SHAPE, "%s: a stride of %s is %lld", fn, name, ll(stride));
  if ((rows > 1 && (x->in_row > kMost / rows || x->out_row > kMost / rows)) ||
      x->in_head > kMost / x->heads || x->out_head > kMost / x->heads)
    return api_fail(QLORA_ERR_SHAPE, "%s: %s spans too many elements", fn, name);
  // of the output no element may belong to two heads
  const bool row_inner = x->out_row < x->out_head;
  const int64_t near = row_inner ? x->out_row : x->out_head, far = row_inner ? x->out_head : x->out_row;
  const int64_t nears = row_inner ? rows : x->heads, fars = row_inner ? x->heads : rows;
  int64_t end = dim;
  if (nears > 1) {
    if (near < end) return api_fail(QLORA_ERR_SHAPE, "%s: the output heads of %s overlap", fn, name);
    end += near * (nears - 1);
  }
  if (fars > 1 && far < end) return api_fail(QLORA_ERR_SHAPE, "%s: the output heads of %s overlap", fn, name);
  return QLORA_OK;
}

qnf4::RopeHeads heads(const qlora_rope_heads *x) {
  return {x->in, x->out, x->heads, x->in_row, x->in_head, x->out_row, x->out_head};
}

int rope(const char *fn, const qlora_rope_heads *Q, const qlora_rope_heads *K, int dtype, int64_t rows, int32_t dim,
         int32_t rot, const void *positions, int32_t wide, const double *freqs, double amplitude, int32_t interleaved,
         bool backward, void *stream) {
  if (!Q || !positions || !freqs) return api_fail(QLORA_ERR_NULL, "%s: the first heads, positions and freqs must not be NULL", fn);
  if (dtype != QLORA_F32 && dtype != QLORA_BF16)
    return api_fail(QLORA_ERR_DTYPE, "%s: dtype %d is not QLORA_F32 or QLORA_BF16", fn, dtype);
  if (rows < 1 || rows > (int64_t(1) << 40)) return api_fail(QLORA_ERR_SHAPE, "%s: rows = %lld", fn, ll(rows));
  if (dim < 2 || dim > qnf4::kRopeMaxDim || dim % 2 != 0 || rot < 2 || rot > dim || rot % 2 != 0)
    return api_fail(QLORA_ERR_SHAPE, "%s: dim = %d, rot = %d: needs even 2 <= rot <= dim <= %d", fn, dim, rot, qnf4::kRopeMaxDim);
  if (!aligned(positions, wide ? 8 : 4) || !aligned(freqs, 8))
    return api_fail(QLORA_ERR_ALIGN, "%s: positions and freqs must be aligned to their elements", fn);
  if (!(std::fabs(amplitude) <= std::numeric_limits<float>::max())) return api_fail(QLORA_ERR_SHAPE, "%s: amplitude must be finite in fp32", fn);
  const int size = dtype == QLORA_BF16 ? 2 : 4;
  int st = check_heads(fn, "the first heads", Q, rows, dim, size);
  if (st == QLORA_OK && K) st = check_heads(fn, "the second heads", K, rows, dim, size);
  if (st != QLORA_OK) return st;
  qnf4::Rope a{};
  a.q = heads(Q);
  if (K) a.k = heads(K);
  if (a.q.heads + a.k.heads > qnf4::kRopeMaxHeads)
    return api_fail(QLORA_ERR_SHAPE, "%s: %lld heads together, more than %lld", fn, ll(a.q.heads + a.k.heads), ll(qnf4::kRopeMaxHeads));
  a.bf16 = dtype == QLORA_BF16;
  a.rows = rows;
  a.dim = dim;
  a.rot = rot;
  a.positions = positions;
  a.wide_positions = wide != 0;
  a.freqs = freqs;
  a.amplitude = amplitude;
  a.interleaved = interleaved != 0;
  a.backward = backward;
  return qnf4::api_hip_status(qnf4::launch_rope(a, static_cast<hipStream_t>(stream)), fn);
}

}  // namespace

extern "C" {

int qlora_mx_pair(const qlora_mx_matrix *gate, const qlora_mx_matrix *up, const qlora_mx_matrix *out, void *stream) {
  const char *fn = "qlora_mx_pair";
  int st = qnf4::api_check_matrix(fn, "gate", gate);
  if (st == QLORA_OK) st = qnf4::api_check_matrix(fn, "up", up);
  if (st == QLORA_OK) st = qnf4::api_check_matrix(fn, "out", out);
  if (st != QLORA_OK) return st;
  if (up->rows != gate->rows || up->cols != gate->cols || out->rows / 2 != gate->rows || out->rows % 2 != 0 || out->cols != gate->cols)
    return api_fail(QLORA_ERR_SHAPE, "%s: gate is %lld x %lld, up %lld x %lld, out %lld x %lld", fn, ll(gate->rows),
                    ll(gate->cols), ll(up->rows), ll(up->cols), ll(out->rows), ll(out->cols));
  if (gate->rows % 8 != 0) return api_fail(QLORA_ERR_SHAPE, "%s: %lld rows are not a multiple of 8", fn, ll(gate->rows));
  if (gate->type != QLORA_MX_FP4 || up->type != QLORA_MX_FP4 || out->type != QLORA_MX_FP4)
    return api_fail(QLORA_ERR_FORMAT, "%s: weights hold 4-bit elements", fn);
  const qnf4::MxPair a{gate->codes, gate->scales, up->codes, up->scales, out->codes, out->scales, out->rows, out->cols};
  return qnf4::api_hip_status(qnf4::launch_mx_pair(a, static_cast<hipStream_t>(stream)), fn);
}

int qlora_mx_gated(const qlora_mx_matrix *X, const qlora_mx_matrix *W, void *H, const qlora_mx_matrix *Hq, void *stream) {
  const char *fn = "qlora_mx_gated";
  int st = qnf4::api_check_matrix(fn, "X", X);
  if (st == QLORA_OK) st = qnf4::api_check_matrix(fn, "W", W);
  if (st != QLORA_OK) return st;
  qnf4::MxLinear a;
  st = gated_args(fn, X, W, W->rows, H, Hq, &a);
  return st != QLORA_OK ? st : gated(fn, a, Hq, false, stream);
}

int qlora_mx_gated_grouped(const qlora_mx_matrix *X, const qlora_mx_matrix *W, const int32_t *offsets, int32_t experts,
                           void *H, const qlora_mx_matrix *Hq, int32_t clear, void *stream) {
  const char *fn = "qlora_mx_gated_grouped";
  int st = qnf4::api_check_matrix(fn, "X", X);
  if (st == QLORA_OK) st = qnf4::api_check_matrix(fn, "W", W);
  if (st != QLORA_OK) return st;
  if (experts < 1 || experts > QLORA_MX_EXPERTS || W->rows % experts != 0)
    return api_fail(QLORA_ERR_SHAPE, "%s: experts = %d must be in [1, %d] and divide W's %lld rows", fn,
                    static_cast<int>(experts), QLORA_MX_EXPERTS, ll(W->rows));
  if (!offsets) return api_fail(QLORA_ERR_NULL, "%s: offsets must not be NULL", fn);
  if (!aligned(offsets, 4)) return api_fail(QLORA_ERR_ALIGN, "%s: offsets must be 4-byte aligned", fn);
  if (W->rows > qnf4::kMxMaxExpertRows)
    return api_fail(QLORA_ERR_SHAPE, "%s: W has %lld rows, more than %lld", fn, ll(W->rows), ll(qnf4::kMxMaxExpertRows));
  qnf4::MxLinear a;
  st = gated_args(fn, X, W, W->rows / experts, H, Hq, &a);
  if (st != QLORA_OK) return st;
  a.offsets = offsets;
  a.experts = experts;
  return gated(fn, a, Hq, clear != 0, stream);
}

int64_t qlora_gated_saved_cols(int32_t r) { return r < 0 || r > 256 ? 0 : 2 * qnf4::gated_padded_rank(r); }

size_t qlora_gated_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t r, int32_t backward) {
  return valid_gated(M, N, K, r) ? qnf4::gated_ws_bytes(M, N, K, r, backward != 0) : 0;
}

int qlora_gated_fwd(const void *X, int64_t M, const qlora_nf4_weight *gate, const qlora_nf4_weight *up,
                    const qlora_gated_adapters *adapters, void *H, void *G, void *U, void *Hs, void *ws, size_t ws_bytes,
                    void *stream) {
  const char *fn = "qlora_gated_fwd";
  if (!X || !H) return api_fail(QLORA_ERR_NULL, "%s: X and H must not be NULL", fn);
  qnf4::GatedArgs a;
  const int st = block_args(fn, M, gate, up, adapters, false, ws, ws_bytes, &a);
  if (st != QLORA_OK) return st;
  if (!G != !U) return api_fail(QLORA_ERR_NULL, "%s: G and U are given together", fn);
  if (!Hs != !(G && adapters)) return api_fail(QLORA_ERR_NULL, "%s: Hs is given with G, U and adapters, and only then", fn);
  if (!aligned(X, 16) || !aligned(H, 16) || !aligned(G, 16) || !aligned(U, 16) || !aligned(Hs, 16))
    return api_fail(QLORA_ERR_ALIGN, "%s: tensors must be 16-byte aligned", fn);
  return qnf4::api_hip_status(qnf4::launch_gated_fwd(a, X, H, G, U, Hs, ws, static_cast<hipStream_t>(stream)), fn);
}

int qlora_gated_bwd(const void *dH, const void *X, const void *G, const void *U, const void *Hs, int64_t M,
                    const qlora_nf4_weight *gate, const qlora_nf4_weight *up, const qlora_gated_adapters *adapters, void *dX,
                    const qlora_gated_grads *grads, void *ws, size_t ws_bytes, void *stream) {
  const char *fn = "qlora_gated_bwd";
  if (!dH || !X || !G || !U || !dX) return api_fail(QLORA_ERR_NULL, "%s: dH, X, G, U and dX must not be NULL", fn);
  qnf4::GatedArgs a;
  const int st = block_args(fn, M, gate, up, adapters, true, ws, ws_bytes, &a);
  if (st != QLORA_OK) return st;
  if (!Hs != !adapters || !grads != !adapters)
    return api_fail(QLORA_ERR_NULL, "%s: Hs and grads are given with adapters, and only then", fn);
  void *dA[2] = {}, *dB[2] = {};
  if (grads) {
    dA[0] = grads->gate_A, dB[0] = grads->gate_B, dA[1] = grads->up_A, dB[1] = grads->up_B;
    if (!dA[0] || !dB[0] || !dA[1] || !dB[1]) return api_fail(QLORA_ERR_NULL, "%s: a gradient is NULL", fn);
  }
  for (const void *p : {dH, X, G, U, Hs, static_cast<const void *>(dX), static_cast<const void *>(dA[0]), static_cast<const void *>(dB[0]),
                        static_cast<const void *>(dA[1]), static_cast<const void *>(dB[1])})
    if (!aligned(p, 16)) return api_fail(QLORA_ERR_ALIGN, "%s: tensors must be 16-byte aligned", fn);
  return qnf4::api_hip_status(qnf4::launch_gated_bwd(a, dH, X, G, U, Hs, dX, dA, dB, ws, static_cast<hipStream_t>(stream)), fn);
}

int qlora_rope_freqs(int32_t rot, double base, int32_t scaling, double factor, int64_t trained, double low,
                     double high, double *freqs, double *amplitude) {
  const char *fn = "qlora_rope_freqs";
  if (!freqs || !amplitude) return api_fail(QLORA_ERR_NULL, "%s: freqs and amplitude must not be NULL", fn);
  if (rot < 2 || rot > qnf4::kRopeMaxDim || rot % 2 != 0)
    return api_fail(QLORA_ERR_SHAPE, "%s: rot = %d: needs an even 2 <= rot <= %d", fn, rot, qnf4::kRopeMaxDim);
  if (scaling < QLORA_ROPE_PLAIN || scaling > QLORA_ROPE_PARTS)
    return api_fail(QLORA_ERR_FORMAT, "%s: scaling %d is not a qlora_rope_scaling", fn, scaling);
  if (!(base > 0.0) || !std::isfinite(base)) return api_fail(QLORA_ERR_SHAPE, "%s: base must be finite and > 0", fn);
  if (scaling != QLORA_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return api_fail(QLORA_ERR_SHAPE, "%s: factor must be finite and >= 1", fn);
  if (scaling == QLORA_ROPE_NTK && rot < 4) return api_fail(QLORA_ERR_SHAPE, "%s: this scaling needs rot > 2", fn);
  if (scaling == QLORA_ROPE_PARTS && (trained < 1 || !(low < high) || !std::isfinite(low) || !std::isfinite(high)))
    return api_fail(QLORA_ERR_SHAPE, "%s: trained must be >= 1 and low < high, both finite", fn);
  *amplitude = scaling == QLORA_ROPE_PARTS ? 0.1 * std::log(factor) + 1.0 : 1.0;
  if (scaling == QLORA_ROPE_NTK) base *= std::pow(factor, static_cast<double>(rot) / (rot - 2));
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (scaling == QLORA_ROPE_LINEAR) f /= factor;
    if (scaling == QLORA_ROPE_PARTS) {
      const double turns = static_cast<double>(trained) * f / 6.283185307179586477;
      const double keep = std::fmin(1.0, std::fmax(0.0, (turns - low) / (high - low)));
      f *= keep + (1.0 - keep) / factor;
    }
    freqs[i] = f;
  }
  return qnf4::api_hip_status(hipSuccess, fn);
}

int qlora_rope_fwd(const qlora_rope_heads *Q, const qlora_rope_heads *K, int dtype, int64_t rows, int32_t dim,
                   int32_t rot, const void *positions, int32_t wide, const double *freqs, double amplitude,
                   int32_t interleaved, void *stream) {
  return rope("qlora_rope_fwd", Q, K, dtype, rows, dim, rot, positions, wide, freqs, amplitude, interleaved, false, stream);
}

int qlora_rope_bwd(const qlora_rope_heads *dQ, const qlora_rope_heads *dK, int dtype, int64_t rows, int32_t dim,
                   int32_t rot, const void *positions, int32_t wide, const double *freqs, double amplitude,
                   int32_t interleaved, void *stream) {
  return rope("qlora_rope_bwd", dQ, dK, dtype, rows, dim, rot, positions, wide, freqs, amplitude, interleaved, true, stream);
}

}  // extern "C"
