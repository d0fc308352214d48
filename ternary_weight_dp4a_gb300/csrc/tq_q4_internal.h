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
// minima 43 54; gate/up 2 x 17408 x 5120 group 128 47 59, group 32 with minima 74 72; 131072 x 5120 group 64
// 188 179, group 32 with minima 271 262: the large ones of small groups lose 5%.)
constexpr int kQ4StreamRows = 16;

// Workspace of the tile kernel, where there are minima: sums of x over the groups, [k / group][q4_sums_ld(m)].
constexpr int64_t q4_sums_ld(int64_t m) { return (m + 15) / 16 * 16; }
constexpr size_t q4_sums_bytes(int64_t m, int64_t k, int64_t group) { return static_cast<size_t>(q4_sums_ld(m) * (k / group) * 4); }

// Up to kQ4StreamRows rows, and any number.
cudaError_t q4_stream_launch(const Q4Product &p, cudaStream_t stream);
cudaError_t q4_tile_launch(const Q4Product &p, float *sums, cudaStream_t stream);
// The bits of the bounded waits that have run out on the current device (copied in `stream`).
cudaError_t q4_tile_waits(unsigned *bits, cudaStream_t stream);

}  // namespace tq
