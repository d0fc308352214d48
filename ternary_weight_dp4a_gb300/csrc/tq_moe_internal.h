// tq_moe_internal.h -- what the translation units of the mixture-of-experts layer share:
// workspace layout and the launch functions behind the C ABI (include/tq_moe.h).
#pragma once

#include <cuda_runtime.h>

#include "tq.h"
#include "tq_limits.h"
#include "tq_moe.h"
#include "tq_workspace.h"

namespace tq {

// Reading what earlier work of the stream has written.  These kernels start while it may still
// run, so it is not read-only for as long as they do: its pointers are not const __restrict__
// and its loads not __ldg, either of which would let a load stand before pdl_wait() or be
// served from a line that was cached before.  (Weights, and what a kernel only writes, may be.)

// Workspace: err u32 | operand (the tile kernel's copy of a product's input:
// 2 bytes per value and slot, and the scales) | hist (the sort's
// counts per chunk of slots, and their sums) | offsets | rows | pos | h | hq | hs | y.
struct MoeWorkspace {
    size_t err, operand, hist, offsets, rows, pos, h, hq, hs, y, total;
};

// A product's input as the tile kernel reads it: two bytes per value, and the
// scales with their rows filled up to 16 bytes.
constexpr int64_t moe_operand_bytes(int64_t slots, int64_t k) { return slots * (2 * k + ws_cdiv(k / 128, 4) * 16); }

// slots sorted by one CTA of the plan kernels
constexpr int kPlanChunk = 1024;

constexpr MoeWorkspace moe_layout(int64_t m, int64_t topk, int64_t experts, int64_t hidden, int64_t inter) {
    MoeWorkspace w{};
    const int64_t slots = m * topk;
    size_t off = 0;
    w.err = off; off = ws_round(off + 4);
    w.operand = off; off = ws_round(off + static_cast<size_t>(moe_operand_bytes(slots, hidden > inter ? hidden : inter)));
    w.hist = off; off = ws_round(off + static_cast<size_t>((ws_cdiv(slots, kPlanChunk) + 1) * experts * 4));
    w.offsets = off; off = ws_round(off + static_cast<size_t>((experts + 1) * 4));
    w.rows = off; off = ws_round(off + static_cast<size_t>(slots * 4));
    w.pos = off; off = ws_round(off + static_cast<size_t>(slots * 4));
    w.h = off; off = ws_round(off + static_cast<size_t>(slots * inter * 2));
    w.hq = off; off = ws_round(off + static_cast<size_t>(slots * inter));
    w.hs = off; off = ws_round(off + static_cast<size_t>(slots * (inter / 128) * 4));
    w.y = off; off = ws_round(off + static_cast<size_t>(slots * hidden * 4));
    w.total = off;
    return w;
}

// What a product alone needs: the error word and its input's operand copy.
constexpr size_t moe_product_bytes(int64_t slots, int64_t k) { return ws_round(4) + static_cast<size_t>(moe_operand_bytes(slots, k)); }

// One grouped product (up == nullptr: y; else gate and up into h).
struct MoeProduct {
    const uint8_t *codes[2];
    const uint16_t *scales[2];
    int experts, n, k, fmt;
    const int8_t *q;
    const float *s;
    int m;                  // rows of q
    const int *rows;        // activation row of each sorted slot, or nullptr
    const int *offsets;     // [experts + 1]
    int slots;
    float *y;
    uint16_t *h;
    int max_rows;           // most rows that an expert can be expected to have
};

// Put the clamped offsets into shared memory (all threads; synchronises).  False if they do
// not ascend: the experts' rows could then add up to more than `slots`, and counts of tiles
// to more than 32 bits, so nothing is computed.
__device__ __forceinline__ bool load_offsets(const MoeProduct &p, int *offsets) {
    bool bad = false;
    for (int e = threadIdx.x; e <= p.experts; e += blockDim.x) {
        const int at = min(max(p.offsets[e], 0), p.slots);
        const int before = e > 0 ? min(max(p.offsets[e - 1], 0), p.slots) : 0;
        bad |= at < before;
        offsets[e] = at;
    }
    return __syncthreads_or(bad) == 0;
}

// A bounded wait ran out: its bit goes into the error word of the call's workspace, and into the
// library's own, which outlives a workspace that the caller has not kept.
__device__ __forceinline__ void record_wait(unsigned *err, unsigned *own, unsigned bit) {
    atomicOr(err, bit);
    atomicOr(own, bit);
}

// The bits in the library's own words, one for each kernel's file,  of the current device (copied in `stream`).
cudaError_t moe_stream_waits(unsigned *bits, cudaStream_t stream);
cudaError_t moe_tile_waits(unsigned *bits, cudaStream_t stream);

// The experts with at most `limit` rows, and those with more than `above`
// (operand: moe_operand_bytes of workspace for the laid-out input).
cudaError_t moe_stream_launch(const MoeProduct &p, int limit, unsigned *err, cudaStream_t stream);
cudaError_t moe_tile_launch(const MoeProduct &p, int above, uint8_t *operand, unsigned *err, cudaStream_t stream);

cudaError_t moe_norm_launch(const void *res, bool res_bf16, const void *delta, bool delta_bf16, const uint16_t *gamma,
                            int m, int n, float eps, void *res_out, uint16_t *x_out, int8_t *q, float *s,
                            cudaStream_t stream);
// tq_rotate_quant of `blocks` 128-blocks behind one another (16-byte aligned).
cudaError_t moe_rotq_launch(const uint16_t *x, int64_t blocks, int8_t *q, float *s, cudaStream_t stream);
cudaError_t moe_combine_launch(const float *y, const int *pos, const float *weights, int m, int topk, int slots, int n,
                               void *out, bool out_bf16, cudaStream_t stream);
cudaError_t moe_route_launch(const void *logits, bool bf16, int m, int experts, int topk, bool renorm, int *ids,
                             float *weights, cudaStream_t stream);
cudaError_t moe_plan_launch(const int *ids, int m, int topk, int experts, int *offsets, int *rows, int *pos, int *hist,
                            cudaStream_t stream);

}  // namespace tq
