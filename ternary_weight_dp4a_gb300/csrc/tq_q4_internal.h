// tq_q4_internal.h -- what the translation units of the 4-bit products share.
#pragma once

#include <cuda_runtime.h>

#include "tq.h"
#include "tq_limits.h"
#include "tq_q4.h"

namespace tq {

constexpr int kQ4Strip = 16;            // weight rows per strip
constexpr int kQ4ChunkBytes = 1024;     // a strip's codes of 128 values of k

constexpr int64_t q4_strips(int64_t n) { return (n + kQ4Strip - 1) / kQ4Strip; }

// One product (mats == 1: y), or gate and up into h (mats == 2).
struct Q4Product {
    const uint8_t *codes[2];
    const uint16_t *scales[2];
    const uint16_t *mins[2];
    int mats, n, k, group;
    const uint16_t *x;
    int m;
    void *y;                // [m][n]: fp32, or bf16 where y_bf16 (h: bf16)
    bool y_bf16;
};

cudaError_t q4_pack_launch(const uint8_t *codes, const uint16_t *scales, const uint16_t *mins, int n, int k, int group,
                           uint8_t *out_codes, uint16_t *out_scales, uint16_t *out_mins, cudaStream_t stream);
// Calls of more rows than this run on the tile kernel.  (us, tile and two passes of the stream kernel at 20 or
// 32 rows: 5120 x 5120 group 128 12 25, 6145 x 2048 group 64 with minima 13 15, 5120 x 17408 group 32 with
// minima 47 54; gate/up 2 x 17408 x 5120 group 128 46 59, group 32 with minima 83 72; 131072 x 5120 group 64
// 185 179, group 32 with minima 297 262: large ones of small groups with minima lose 13%.)
constexpr int kQ4StreamRows = 16;

// Rows of x of a tile, a multiple of 16: even shares of `most` at most.
constexpr int kQ4TileCols = 192, kQ4ScaledCols = 176;       // (with scaled weights and minima)
constexpr int q4_tile_rows(int m, int most) {
    const int tiles = (m + most - 1) / most;
    return ((m + tiles - 1) / tiles + 15) / 16 * 16;
}

// Whether the tile kernel has the scales in the weights.  That costs twice the MMAs, whatever the rows; folds of small
// groups cost by the column, and with minima more.  (us, folded and scaled.  131072 x 5120: group 32 64 rows 259 296, 80
// rows 415 274, 192 rows 644 326; with minima 32 rows 297 294, 48 rows 401 308, 160 rows 888 331; group 64 96 rows 255
// 273, 112 rows 320 275; with minima 64 rows 284 306, 80 rows 385 289, 160 rows 478 321, 176 rows 491 335.  Gate/up 2 x
// 17408 x 5120, 512 rows: group 32 559 257, with minima 693 283; group 64 326 254, with minima 414 284.)
constexpr bool q4_scaled(int m, int group, bool mins) {
    const int rows = q4_tile_rows(m, kQ4TileCols);
    return group == 32 ? rows > (mins ? 32 : 64) : group == 64 && rows > (mins ? 64 : 96);
}

// The same for a call whose weights make `tiles` tiles.  With minima 177 to 192 rows are one folded tile and two scaled ones:
// groups of 64 are folded there, unless all scaled tiles run at once anyhow.  (us, folded and scaled, 177 rows and
// 192: 131072 x 5120 504 564, 505 565; gate/up 2 x 17408 x 5120 156 182, 157 183; 2 x 4096 x 2048, 64 tiles, 35 31, 36 33.
// Groups of 32, 131072 x 5120: 952 565, 954 565.  353 to 384 rows are two and three: 961 841, 294 262.)
constexpr bool q4_scaled_call(int m, int group, bool mins, int64_t tiles, int sms) {
    const bool two = mins && m > kQ4ScaledCols && m <= kQ4TileCols;
    return q4_scaled(m, group, mins) && !(two && group == 64 && 2 * tiles > sms);
}

// Workspace of the tile kernel, where there are minima: sums of x over the groups, [k / group][q4_sums_ld(m)], or
// with scaled weights their parts, 32 bf16 for every row and 128 values.  (The parts are the larger, and it is their size
// where a call may take either.)
constexpr int64_t q4_sums_ld(int64_t m) { return (m + 15) / 16 * 16; }
constexpr size_t q4_sums_bytes(int64_t m, int64_t k, int64_t group) {
    return static_cast<size_t>(q4_scaled(static_cast<int>(m), static_cast<int>(group), true) ? m * (k / 128) * 64
                                                                                            : q4_sums_ld(m) * (k / group) * 4);
}

// Up to kQ4StreamRows rows, and any number.
cudaError_t q4_stream_launch(const Q4Product &p, cudaStream_t stream);
cudaError_t q4_tile_launch(const Q4Product &p, float *sums, cudaStream_t stream);
// The bits of the bounded waits that have run out on the current device (copied in `stream`).
cudaError_t q4_tile_waits(unsigned *bits, cudaStream_t stream);

}  // namespace tq
