/*
 * qlora_block.h - what stands between the projections of a decoder layer, of
 * the QLoRA library on AMD Instinct MI355X (gfx950): the gated feed-forward
 * product, served from a merged model and trained around frozen 4-bit weights
 * and their adapters, and rotary positions.
 *
 * The conventions of qlora_nf4.h and qlora_mx.h hold (row-major contiguous
 * device tensors unless strides are named, 16-byte aligned pointers,
 * caller-owned memory, work enqueued on `stream`, status codes,
 * qlora_last_error). A failed check launches nothing. Every call may be
 * captured into a graph; calls that run at the same time need workspaces of
 * their own.
 */
#ifndef QLORA_BLOCK_H
#define QLORA_BLOCK_H

#include <stddef.h>
#include <stdint.h>

#include "qlora_mx.h"
#include "qlora_nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------- the gated product, served
 *
 *     H = silu(X Wg^T) * (X Wu^T),   silu(g) = g / (1 + e^-g)
 *
 * Wg and Wu [N, K] are held as one matrix, a pair, of 2 N rows: eight rows of
 * the gate and eight of the other one in turn, so that row 16 j + t is row
 * 8 j + t of Wg and row 16 j + 8 + t that of Wu (0 <= t < 8).
 */

/* Lay two weights of the same shape and type out as a pair: out has twice
 * their rows, whose number is a multiple of 8. Done once, when a model is
 * loaded. out overlaps neither. */
int qlora_mx_pair(const qlora_mx_matrix *gate, const qlora_mx_matrix *up, const qlora_mx_matrix *out, void *stream);

/*
 * X [M, K] in microscaled 8- or 4-bit floats, W a pair [2 N, K] in microscaled
 * 4-bit floats, N a multiple of 32. H [M, N] goes to exactly one of
 *   H    bf16, rounded once
 *   Hq   microscaled (8 or 4 bits), exactly what qlora_mx_quantize would make
 *        of the unrounded H: the input of the down projection
 * Sums, sizes and NaN blocks as in qlora_mx_linear with the 2 N rows of W (a
 * NaN block of either weight makes H's column NaN, and with Hq the block of 32
 * that the column is in). The sums and silu are fp32. H overlaps no input.
 */
int qlora_mx_gated(const qlora_mx_matrix *X, const qlora_mx_matrix *W, void *H, const qlora_mx_matrix *Hq, void *stream);

/* The same by expert: rows of X sorted by expert, W [experts * 2 N, K] the
 * experts' pairs one below the other; offsets and experts as in
 * qlora_mx_linear_grouped. Rows of H (codes and scales) in front of offsets[0]
 * and from offsets[experts] on are left as they were, or with `clear` (not 0)
 * become zeros, as a new H wants them. */
int qlora_mx_gated_grouped(const qlora_mx_matrix *X, const qlora_mx_matrix *W, const int32_t *offsets,
                           int32_t experts, void *H, const qlora_mx_matrix *Hq, int32_t clear, void *stream);

/* ------------------------------------------------ the gated block, with adapters
 *
 *     G = X Wg^T + s (X Ag^T) Bg^T,  U = X Wu^T + s (X Au^T) Bu^T,  H = silu(G) * U
 *
 * around two frozen 4-bit weights [N, K] of the same shape and format (N and K
 * multiples of 64), each with an adapter of the same rank or both without. An
 * adapter on one of them only has factors of zeros for the other, one of lower
 * rank rows of A and columns of B that are zero.
 */

/* A [r, K] and B [N, r] of each weight, fp32 or bf16 (dtype), 1 <= r <= 256. */
typedef struct {
  const void *gate_A, *gate_B, *up_A, *up_B;
  int32_t r;
  int32_t dtype;
  float scale;
} qlora_gated_adapters;

/* Columns of the kept adapter activations, 2 * 64 ceil(r / 64) (0 for an invalid r and for 0). Host-only. */
int64_t qlora_gated_saved_cols(int32_t r);

/* Workspace bytes of qlora_gated_fwd (backward = 0) and qlora_gated_bwd (1): 0
 * for a few rows without adapters (ws may then be NULL) and for invalid sizes.
 * No contents are expected or kept. Host-only. */
size_t qlora_gated_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t r, int32_t backward);

/*
 * Forward. X bf16 [M, K]; adapters NULL: none. H bf16 [M, N], rounded once.
 * What the backward takes is written where it is asked for:
 *   G, U  bf16 [M, N], both or neither (NULL)
 *   Hs    bf16 [M, qlora_gated_saved_cols(r)], s X Ag^T and s X Au^T, each padded
 *         to a multiple of 64 columns with zeros; with G and U and adapters,
 *         NULL otherwise
 * M up to 2^24, N and K up to 2^23, M N, M K and N K up to 2^36. A, B and Hs
 * enter the sums as bf16, and so do the weights: above 32 rows, and in the
 * backward, decoded and rounded one by one; up to 32 rows as their levels, times
 * one factor for all, rounded, whose sums over a block take its constant in
 * fp32. Both are off by 1.4e-3 to 1.6e-3 of the weights in the root mean square and
 * by less than 1e-5 in the mean. Sums and silu are fp32, in a fixed order
 * (deterministic). No output overlaps an input, another output or the workspace.
 */
int qlora_gated_fwd(const void *X, int64_t M, const qlora_nf4_weight *gate, const qlora_nf4_weight *up,
                    const qlora_gated_adapters *adapters, void *H, void *G, void *U, void *Hs, void *ws,
                    size_t ws_bytes, void *stream);

/* Gradients of the adapters, in their type. */
typedef struct {
  void *gate_A, *gate_B, *up_A, *up_B;
} qlora_gated_grads;

/*
 * Backward, from the forward's X, G, U and Hs (of the same adapters):
 *     dG = dH U t (1 + G (1 - t)),  dU = dH G t,  t = 1 / (1 + e^-G)
 *     lg = s dG Bg,  lu = s dU Bu
 *     dX = dG Wg + dU Wu + lg Ag + lu Au
 *     dAg = lg^T X,  dBg = dG^T Hs_g,  dAu = lu^T X,  dBu = dU^T Hs_u
 * dH, dX bf16. No output overlaps an input, another output or the workspace.
 * grads NULL without adapters.
 * dG, dU, lg and lu are rounded to bf16 (for the adapters' gradients not where
 * there are few of lg and lu, M <= 16 and M r <= 64), each sum is fp32 in a fixed
 * order and rounded once.
 */
int qlora_gated_bwd(const void *dH, const void *X, const void *G, const void *U, const void *Hs, int64_t M,
                    const qlora_nf4_weight *gate, const qlora_nf4_weight *up, const qlora_gated_adapters *adapters,
                    void *dX, const qlora_gated_grads *grads, void *ws, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------ rotary positions
 *
 * Pair i of a head, (a, b), of the token at position t becomes
 *     (a cos w - b sin w, b cos w + a sin w) * amplitude,   w = t freqs[i].
 * The pairs are elements i and i + rot / 2 of the head, or with `interleaved`
 * the neighbours 2 i and 2 i + 1; elements from rot on pass through.
 */

typedef enum { QLORA_ROPE_PLAIN = 0, QLORA_ROPE_LINEAR = 1, QLORA_ROPE_NTK = 2, QLORA_ROPE_PARTS = 3 } qlora_rope_scaling;

/*
 * Frequencies of the rot / 2 pairs in radians a position (host memory), and
 * the amplitude that goes with them: f_i = base^(-2 i / rot), for contexts
 * `factor` times as long as trained
 *   PLAIN   as they are (factor and the rest unused)
 *   LINEAR  f_i / factor: positions pressed together
 *   NTK     of base factor^(rot / (rot - 2)) times as large (rot > 2): the
 *           fastest pair as it is, the slowest as LINEAR
 *   PARTS   by parts, with n_i = trained f_i / (2 pi) the turns that pair i
 *           makes in the `trained` positions: f_i (k + (1 - k) / factor), k =
 *           (n_i - low) / (high - low) within [0, 1]; amplitude
 *           0.1 ln(factor) + 1 (a model that was trained without it takes 1)
 *           The ramp goes by the turns. A model whose frequencies ramp over the
 *           pair's index between two bounds has others, which the rotation takes
 *           as they are
 * base > 0, factor >= 1, trained >= 1, low < high; finite. Host-only.
 */
int qlora_rope_freqs(int32_t rot, double base, int32_t scaling, double factor, int64_t trained, double low,
                     double high, double *freqs, double *amplitude);

/*
 * Heads [rows][heads][dim] in device memory, the dim elements of a head next
 * to each other; strides in elements, >= 0. The output heads overlap neither
 * each other nor any input, except that out may be in with its strides (in
 * place). Pointers and strides need the element's alignment only.
 */
typedef struct {
  const void *in;
  void *out;
  int64_t heads;
  int64_t in_row, in_head, out_row, out_head;
} qlora_rope_heads;

/*
 * Rotate Q and K (K may be NULL) in one launch.
 *   dtype       QLORA_F32 or QLORA_BF16, in and out
 *   dim, rot    even, 2 <= rot <= dim <= 1024; at most 32768 heads together
 *   positions   int32 (wide = 0) or int64 (wide = 1, rounded to fp64) [rows] on the device
 *   freqs       fp64 [rot / 2] on the device
 *   amplitude   finite, in fp32 too
 * The angle is formed in turns, in fp64, with three roundings, and reduced there:
 * good to 3 * 2^-53 of its turns, 2^-23 turns at |t| < 2^31 and f <= 1. Sine,
 * cosine and rotation are fp32, rounded once.
 */
int qlora_rope_fwd(const qlora_rope_heads *Q, const qlora_rope_heads *K, int dtype, int64_t rows, int32_t dim,
                   int32_t rot, const void *positions, int32_t wide, const double *freqs, double amplitude,
                   int32_t interleaved, void *stream);

/* The gradient: from that of the rotated heads to that of the heads, the same
 * rotation with -w (elements from rot on pass through here too). */
int qlora_rope_bwd(const qlora_rope_heads *dQ, const qlora_rope_heads *dK, int dtype, int64_t rows, int32_t dim,
                   int32_t rot, const void *positions, int32_t wide, const double *freqs, double amplitude,
                   int32_t interleaved, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_BLOCK_H */
