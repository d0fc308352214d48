/*
 * tq_moe.h -- the layer around a mixture of ternary experts: the step into the
 * layer (residual addition, RMS norm, rotation, int8 quantisation), the router
 * and its sort, the products grouped by expert, and the sum over a token's
 * experts.  tq.h's conventions hold for every entry point: device pointers owned by
 * the caller, work enqueued on `stream`, arguments checked before anything is
 * launched, no allocation, no synchronisation, contiguous row-major arrays,
 * outputs that overlap no input (where an entry point says otherwise, they may
 * be the same array).  (The source pages describe dense FFNs only: they have no
 * counterpart to this header; the weights' layout, the rotation, the
 * quantisation and SiLU are tq.h's.)
 *
 * One layer, for m tokens of width `hidden` (nothing here waits for the host,
 * so a captured graph replays it with other routings):
 *
 *   tq_add_rmsnorm_rotq   residual += delta; q, s = quantised norm
 *   tq_moe_route          logits -> topk experts and weights of each token
 *   tq_moe_ffn            plan, gate/up, SiLU * up, down, weighted sum
 *
 * tq_moe_ffn is tq_moe_plan, tq_moe_gateup, tq_rotate_quant, tq_moe_gemv and
 * tq_moe_combine on one workspace; each is an entry point of its own.
 *
 * Slots: the pair (token t, choice j) is slot t * topk + j.  A plan sorts the
 * slots by expert, keeping their order within an expert; the arrays between
 * the two products (h, its codes, y) have one row per sorted slot, so the
 * rows of expert e are offsets[e] .. offsets[e+1]-1, any number of them,
 * none included.
 */
#ifndef TQ_MOE_H
#define TQ_MOE_H

#include "tq.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { TQ_F32 = 0, TQ_BF16 = 1 } tq_dtype;

/* The packed weights of all experts: `experts` matrices [n][k] one behind the
 * other, each in the layout of tq.h (tq_pack_weights with n = experts * n
 * packs them).  codes: 32-byte aligned; scales: 2-byte aligned. */
typedef struct {
    const uint8_t *codes;
    const uint16_t *scales;
    int32_t experts;
    int32_t n;
    int32_t k;
    int32_t fmt; /* tq_format */
} tq_experts;

#define TQ_MOE_MAX_EXPERTS 1024
#define TQ_MOE_MAX_TOPK 32
#define TQ_MOE_MAX_SLOTS (1 << 26) /* m * topk */
#define TQ_MOE_MAX_WIDTH 32768     /* hidden, inter: n and k of an expert */

/* Residual addition, RMS norm, rotation and quantisation.  For each row r:
 *   t[i]   = residual[r][i] + delta[r][i], one fp32 addition, rounded to the
 *            residual's type (delta NULL: t = residual)
 *   inv    = fp32(1 / sqrt((sum_i t[i]^2) / n + eps))
 *   x[i]   = bf16_rn(t[i] * inv), or bf16_rn((t[i] * inv) * gamma[i])
 *   q, s   = tq_rotate_quant(x)
 * and residual_out = t, x_out = x.  The sum of squares is held as an unevaluated
 * pair of fp32 numbers and so is the mean, so inv is the correctly rounded
 * value but for about one row in 10^5 (then its neighbour), whatever the
 * order of the sum: a code that an ulp of inv would move across a rounding
 * border does not depend on how rows are split over threads.  A row's results do
 * not depend on m.  A NaN in x gives its block a NaN scale and zero codes.
 * residual_type, delta_type: tq_dtype.  gamma: bf16 bits [n], or NULL.
 * residual_out may be NULL, or `residual` itself (updated in place).  x_out
 * (bf16 bits [m][n]) may be NULL; q and s may be NULL together.
 * n: a multiple of 128 up to TQ_MOE_MAX_WIDTH; any m >= 1.  All pointers
 * 16-byte aligned (s: 4). */
tq_status tq_add_rmsnorm_rotq(const void *residual, int32_t residual_type, const void *delta,
                              int32_t delta_type, const uint16_t *gamma, int32_t m, int32_t n,
                              float eps, void *residual_out, uint16_t *x_out, int8_t *q, float *s,
                              tq_stream_t stream);

/* The router: for each token the topk experts of the largest logits, in
 * descending order, ties to the lowest index.  An expert whose logit is
 * -infinity or NaN is never chosen; choices that are left over get
 * ids = -1 and weight 0.  Weights: with l_0 the largest logit (+infinity counts
 * as the largest finite number) and e_j = exp(l_j - l_0),
 *   renormalize != 0: e_j / (sum of e over the token's choices)
 *   renormalize == 0: e_j / (sum of e over all experts that are not excluded)
 * logits: [m][experts] of logits_type; ids: int32 [m][topk]; weights: fp32
 * [m][topk].  topk <= experts <= TQ_MOE_MAX_EXPERTS, topk <= TQ_MOE_MAX_TOPK. */
tq_status tq_moe_route(const void *logits, int32_t logits_type, int32_t m, int32_t experts,
                       int32_t topk, int32_t renormalize, int32_t *ids, float *weights,
                       tq_stream_t stream);

/* Bytes of the workspace that the tq_moe_* calls take, for up to m tokens:
 * zero-filled once by tq_workspace_init, reusable after every call, 256-byte
 * aligned, not shared by calls that may overlap.  hidden and inter may both be
 * 0 for a workspace that only serves tq_moe_plan.  0 for sizes out of range.
 * Its first 4 bytes are the error word of the bounded waits (tq_read_error_word); only
 * they have to be zero.  Each wait takes about half a second before it sets its bit;
 * the call's outputs are then not valid.
 *   bit 0  (tile kernel) the decoders waited for a free buffer of weights
 *   bit 1  the matrix instructions waited for a free accumulator
 *   bit 2  for decoded weights        bit 3  for activation rows
 *   bit 4  (tile kernel) its last matrix instructions, at exit
 *   bit 5  the activation copies waited for a free stage
 *   bit 6  the scales' writers or readers waited for each other
 *   bit 7  the fold waited for an accumulator
 *   bit 8  the activation copies, bit 11 the weight copies in flight at exit
 *   bit 9  the decoders waited for packed weights
 *   bit 10 the weight copies waited for a free stage
 *   bit 12 (stream kernel) a warp waited for packed weights */
size_t tq_moe_workspace_bytes(int32_t m, int32_t topk, int32_t experts, int32_t hidden,
                              int32_t inter);

/* The same bits of every tq_moe_* call of this process on the current device since the library
 * was loaded, whatever workspace it had: for callers that keep none.  (The one thing that the
 * library itself keeps between calls.)  Synchronises the stream.  TQ_OK, or TQ_ERR_TIMEOUT if
 * a bit is set. */
tq_status tq_moe_read_error_word(uint32_t *value, tq_stream_t stream);

/* Sort the m * topk slots by expert (stable).  ids: int32 [m][topk]; an id
 * outside 0 .. experts-1 leaves its slot out.  Outputs:
 *   offsets int32 [experts + 1]: first sorted slot of each expert; the last
 *           entry is the number of slots that have an expert;
 *   rows    int32 [m * topk]: token of each sorted slot, -1 behind the last;
 *   pos     int32 [m * topk]: place of slot (t, j) in the order, -1 if left out.
 * A token may name an expert twice. */
tq_status tq_moe_plan(const int32_t *ids, int32_t m, int32_t topk, int32_t experts,
                      int32_t *offsets, int32_t *rows, int32_t *pos, void *workspace,
                      size_t workspace_bytes, tq_stream_t stream);

/* Products grouped by expert.  For sorted slot r of expert e, with a the
 * activation row of r (q[rows[r]], s[rows[r]], or q[r], s[r] where rows is
 * NULL), and output i:
 *   d_b = sum over block b of W_e[i][j] * a.q[j]                   (exact integer)
 *   y[r][i] = fold over b = 0, 1, .. of  acc = fma(d_b, scale_e[i][b] * a.s[b], acc)
 * in fp32 from +0.0, the product of the two scales rounded first.  The order
 * does not depend on m, on the other rows or on which kernel runs: a token's
 * rows have the bits that they have alone.
 * q: int8 [m][k], 16-byte aligned; s: fp32 [m][k/128]; offsets, rows: a plan
 * over `slots` slots (offsets[experts] <= slots; offsets ascending from 0; rows in
 * 0 .. m-1).  Entries of a bad plan are clamped to these ranges, not followed, and
 * offsets that do not ascend have no rows at all.
 * y: fp32 [slots][n]; rows from offsets[experts] on are left as they are.
 * n: 1 .. TQ_MOE_MAX_WIDTH, k: a multiple of 128 up to TQ_MOE_MAX_WIDTH.
 * workspace: a tq_moe_* workspace of the layer that the product belongs to, or
 * any of at least 256 + slots * (2 * k + 16 * ceil(k / 512)) bytes that
 * follows its conventions. */
tq_status tq_moe_gemv(const tq_experts *w, const int8_t *q, const float *s, int32_t m,
                      const int32_t *rows, const int32_t *offsets, int32_t slots, float *y,
                      void *workspace, size_t workspace_bytes, tq_stream_t stream);

/* Gate and up of every sorted slot in one pass, each as tq_moe_gemv (g and u):
 *   h[r][i] = bf16_rn(g / (1 + exp(-g)) * u)                       (as tq_ffn_step)
 * gate, up: same experts, n, k and format.  h: bf16 bits [slots][n]. */
tq_status tq_moe_gateup(const tq_experts *gate, const tq_experts *up, const int8_t *q,
                        const float *s, int32_t m, const int32_t *rows, const int32_t *offsets,
                        int32_t slots, uint16_t *h, void *workspace, size_t workspace_bytes,
                        tq_stream_t stream);

/* Sum over a token's experts: out[t][i] = fold over j = 0 .. topk-1 of
 * acc = fma(weights[t][j], y[pos[t][j]][i], acc) in fp32 from +0.0, slots with
 * pos outside 0 .. slots-1 left out; rounded to out_type (tq_dtype).
 * y: fp32 [slots][n]; out: [m][n].  y, out: 16-byte aligned; n a multiple of 4. */
tq_status tq_moe_combine(const float *y, const int32_t *pos, const float *weights, int32_t m,
                         int32_t topk, int32_t slots, int32_t n, void *out, int32_t out_type,
                         tq_stream_t stream);

/* The FFN of a layer for m tokens, from the codes of tq_add_rmsnorm_rotq and
 * the router's ids and weights: plan, gate/up, h rotated and quantised
 * (tq_rotate_quant), down, weighted sum.
 * gate, up: [experts][inter][hidden]; down: [experts][hidden][inter]; inter and
 * hidden multiples of 128; one format.  q: int8 [m][hidden]; s: fp32
 * [m][hidden/128]; ids, weights: [m][topk]; out: [m][hidden] of out_type.
 * workspace: >= tq_moe_workspace_bytes(m, topk, experts, hidden, inter). */
tq_status tq_moe_ffn(const tq_experts *gate, const tq_experts *up, const tq_experts *down,
                     const int8_t *q, const float *s, const int32_t *ids, const float *weights,
                     int32_t m, int32_t topk, void *out, int32_t out_type, void *workspace,
                     size_t workspace_bytes, tq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TQ_MOE_H */
