/*
 * tq_q4.h -- products with 4-bit weights: what a decode step runs next to its
 * ternary FFN.  The attention projections and the head of a model whose FFN is
 * ternary keep 4-bit weights ("rest of the model", sparkinfer PR #1154,
 * Summary), and the FFN itself runs on its 4-bit weights while the ternary
 * copy is not resident (tq_lifecycle.h: callers take the ternary path only when
 * tq_lifecycle_copy is non-NULL).  tq.h's conventions hold for every entry
 * point: device pointers owned by the caller, work enqueued on `stream`,
 * arguments checked before anything is launched, no allocation, no
 * synchronisation, contiguous row-major arrays, outputs that overlap no input.
 *
 * A matrix W [n][k] has 4-bit codes c and, for each row and each group of
 * `group` values along k, an fp16 scale s and (where mins is not NULL) an fp16
 * minimum b:
 *   W[i][j] = s * (c - 8)      without minima
 *   W[i][j] = s * c - b        with minima
 * group is 32, 64 or 128; k is a multiple of 128.  Activations are bf16 and are
 * not rotated or quantised.
 * (Q4_K is the form with minima in groups of 32, but its scales and minima are an
 * fp16 number of eight groups times a 6-bit one of the group, up to 17 bits.  Here each
 * is one fp16 number: the caller rounds that product, by up to 2^-11 of it, or half a
 * unit of fp16's smallest exponent, 2^-25.)
 *
 * Packed layout (tq_q4_pack writes it; rows are padded to a multiple of 16 with
 * zero weights).  Row i is row r = i % 16 of strip t = i / 16, value j is in
 * chunk e = j / 128; a strip's chunks follow one another, 1024 bytes each:
 *   code (r, j) is in the 32-bit word at byte
 *     (t * (k/128) + e) * 1024 + (r / 8) * 512 + (r % 8) * 64
 *       + ((j % 32) / 8) * 16 + ((j % 128) / 32) * 4
 *   at nibble (j % 8) / 2 + 4 * (j % 2), least significant first;
 *   scale (and minimum) of (r, group p of the chunk), with P = 128 / group, is
 *   entry  (t * (k/128) + e) * 16 * P + ((r % 8) * 2 + r / 8) * P + p.
 * (A lane's words are then the operands of the matrix instructions, 16 bytes of
 * one load hold a row's codes of all groups, and one load both rows' scales.)
 */
#ifndef TQ_Q4_H
#define TQ_Q4_H

#include "tq.h"
#include "tq_moe.h" /* tq_dtype */

#ifdef __cplusplus
extern "C" {
#endif

/* One packed matrix.  codes, scales, mins: 16-byte aligned; mins NULL: none. */
typedef struct {
    const uint8_t *codes;
    const uint16_t *scales;
    const uint16_t *mins;
    int32_t n;
    int32_t k;
    int32_t group;
} tq_q4_weight;

#define TQ_Q4_MAX_N (1 << 22)
#define TQ_Q4_MAX_K 32768
#define TQ_Q4_MAX_ROWS (1 << 20)

/* Bytes of the packed codes, and of the packed scales (or minima), of an n x k
 * matrix; 0 for sizes out of range. */
size_t tq_q4_codes_bytes(int32_t n, int32_t k);
size_t tq_q4_scales_bytes(int32_t n, int32_t k, int32_t group);

/* Lay a matrix out (a load-time step).  codes: uint8 [n][k], entries 0 .. 15
 * (only the low 4 bits are read), 8-byte aligned; scales, mins: fp16 bits
 * [n][k/group], mins NULL together with packed_mins.  packed_codes,
 * packed_scales, packed_mins: 16-byte aligned, of the sizes above. */
tq_status tq_q4_pack(const uint8_t *codes, const uint16_t *scales, const uint16_t *mins, int32_t n,
                     int32_t k, int32_t group, uint8_t *packed_codes, uint16_t *packed_scales,
                     uint16_t *packed_mins, tq_stream_t stream);

/* Bytes of the workspace that a product of m rows with a matrix that has minima
 * takes (the sums of x over the groups, or their parts); 0 where none is needed, up to 16 rows,
 * and for sizes out of range.  256-byte aligned, any contents, reusable after every
 * call, not shared by calls that may overlap.  Matrices without minima need none. */
size_t tq_q4_workspace_bytes(int32_t m, int32_t k, int32_t group);

/* y[r][i] = sum over j of W[i][j] * x[r][j], for m rows x (bf16 bits [m][k],
 * 16-byte aligned), rounded to y_type (tq_dtype) once.  Per group, the sum of
 * (c - 8) * x over exact products is taken in fp32 by matrix instructions, and
 * folded in fp32 as s * sum, plus (8 s - b) * (sum of x) where there are minima;
 * calls of many rows with groups of 32 or 64 have s in the matrix instructions too,
 * exactly, as the sum of two bf16, and (8 s - b) * (sum of x) as products of bf16
 * parts, to 2^-24.  An infinity or NaN in a row of x, or in a scale
 * or minimum, makes results that depend on it infinite or NaN, and no others
 * do.  So may sums that leave fp32's range on the way: a group's sums of (c - 8) * x
 * and of x stay in it for |x| up to 2^117; what is added up of them is
 * s * (c - 8) * x, and (8 s - b) * x where there are minima.
 * In calls of up to 8 rows (a packed decode step) each row has the bits that it
 * has alone; with more rows the order of the sums may differ.
 * y: [m][n], aligned to its type; n 1 .. TQ_Q4_MAX_N, k up to TQ_Q4_MAX_K, m 1 ..
 * TQ_Q4_MAX_ROWS.  workspace: as above, may be NULL where none is needed. */
tq_status tq_q4_gemv(const tq_q4_weight *w, const uint16_t *x, int32_t m, void *y, int32_t y_type,
                     void *workspace, size_t workspace_bytes, tq_stream_t stream);

/* Gate and up of a gated FFN in one pass, each as tq_q4_gemv (g and u in fp32):
 *   h[r][i] = bf16_rn(g / (1 + exp(-g)) * u)                 (as tq_ffn_step)
 * gate, up: same n, k, group, and minima in both or in neither.  h: bf16 bits
 * [m][n].  workspace: as above. */
tq_status tq_q4_gateup(const tq_q4_weight *gate, const tq_q4_weight *up, const uint16_t *x,
                       int32_t m, uint16_t *h, void *workspace, size_t workspace_bytes,
                       tq_stream_t stream);

/* The bits of the bounded waits that have run out in any tq_q4_* call of this
 * process on the current device since the library was loaded (calls of more than
 * 16 rows have such waits; one runs out after about half a second.  The call then
 * ends, whatever its size, within a second or two more, and its outputs are not
 * valid; later calls are not concerned).  Synchronises the stream.  TQ_OK, or
 * TQ_ERR_TIMEOUT if a bit is set:
 *   bit 0  the decoders waited for a free stage    bit 5  the copies of x
 *   bit 1  the matrix instructions waited for x    bit 2  for decoded weights
 *   bit 3  for a free accumulator                  bit 4  at exit
 *   bit 6  the copies of x in flight at exit
 *   bit 7  the fold, or the matrix instructions, waited for the sums of x
 *   bit 8  the fold waited for an accumulator
 *   bit 9  the copies of the sums waited for a free place */
tq_status tq_q4_read_error_word(uint32_t *value, tq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TQ_Q4_H */
