// tq_moe_api.cu -- the C ABI of the mixture-of-experts layer (declared in
// include/tq_moe.h): argument checks, workspace layout and dispatch.
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "tq_moe_internal.h"

namespace tq {
void record_cuda_error(int e);
}

namespace {

tq_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return TQ_OK;
    tq::record_cuda_error(static_cast<int>(e));
    return TQ_ERR_CUDA;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool dtype_ok(int32_t t) { return t == TQ_F32 || t == TQ_BF16; }
bool width_ok(int32_t n) { return n >= 128 && n <= TQ_MOE_MAX_WIDTH && n % 128 == 0; }

bool route_sizes_ok(int32_t m, int32_t topk, int32_t experts) {
    return m >= 1 && experts >= 1 && experts <= TQ_MOE_MAX_EXPERTS && topk >= 1 && topk <= TQ_MOE_MAX_TOPK &&
           topk <= experts && static_cast<int64_t>(m) * topk <= TQ_MOE_MAX_SLOTS;
}

tq_status check_ws(const void *ws, size_t bytes, size_t need) {
    if (ws == nullptr) return TQ_ERR_INVALID_ARG;
    if (!aligned(ws, tq::kWsAlign)) return TQ_ERR_ALIGNMENT;
    return bytes < need ? TQ_ERR_WORKSPACE : TQ_OK;
}

tq_status check_experts(const tq_experts *w) {
    if (w == nullptr || w->codes == nullptr || w->scales == nullptr) return TQ_ERR_INVALID_ARG;
    if (w->experts < 1 || w->experts > TQ_MOE_MAX_EXPERTS || w->n < 1 || w->n > TQ_MOE_MAX_WIDTH || !width_ok(w->k))
        return TQ_ERR_INVALID_ARG;
    if (w->fmt != TQ_FMT_TERNARY2 && w->fmt != TQ_FMT_BINARY1) return TQ_ERR_INVALID_ARG;
    if (!aligned(w->codes, 32) || !aligned(w->scales, 2)) return TQ_ERR_ALIGNMENT;
    return TQ_OK;
}

bool same_shape(const tq_experts *a, const tq_experts *b) {
    return a->experts == b->experts && a->n == b->n && a->k == b->k && a->fmt == b->fmt;
}

tq_status check_rows(const int8_t *q, const float *s, int32_t m, const int32_t *rows, const int32_t *offsets,
                     int32_t slots) {
    if (q == nullptr || s == nullptr || offsets == nullptr) return TQ_ERR_INVALID_ARG;
    if (m < 1 || slots < 1 || slots > TQ_MOE_MAX_SLOTS || m > TQ_MOE_MAX_SLOTS) return TQ_ERR_INVALID_ARG;
    if (rows == nullptr && slots > m) return TQ_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(s, 4) || !aligned(rows, 4) || !aligned(offsets, 4)) return TQ_ERR_ALIGNMENT;
    return TQ_OK;
}

tq::MoeProduct product(const tq_experts *w, const tq_experts *up, const int8_t *q, const float *s, int32_t m,
                       const int32_t *rows, const int32_t *offsets, int32_t slots) {
    tq::MoeProduct p{};
    p.codes[0] = w->codes;
    p.scales[0] = w->scales;
    if (up != nullptr) {
        p.codes[1] = up->codes;
        p.scales[1] = up->scales;
    }
    p.experts = w->experts;
    p.n = w->n;
    p.k = w->k;
    p.fmt = w->fmt;
    p.q = q;
    p.s = s;
    p.m = m;
    p.rows = rows;
    p.offsets = offsets;
    p.slots = slots;
    return p;
}

// Experts with more rows than this run on the tile kernel, the others on the stream
// kernel; the bits are the same.  A block of 128 weight rows costs the tile kernel about 2000
// cycles for any number of activation rows, the stream kernel 300 for every eight; the
// tile kernel's launches are paid for anyway once there is one.  Both grow alike with n and k.
// With 24, 32 and 48 (us; gate/up 2048 -> 2 x 1024, 5120 -> 2 x 1536, down 1024 -> 2048,
// 1536 -> 5120; even routing): 400 tokens, top 8 of 64, 127 127 148, 396 397 435, 75 75 83, 221
// 222 236; top 8 of 128, where most experts are near the border, 194 174 160, 585 524 514, 112
// 95 88, 334 273 262; from 1000 tokens on all are alike.
constexpr int kTileAbove = 32;
// The tile kernel's launches cost 10 us and its turns are long (2000 cycles for each of k/128
// blocks), so it is left out where few experts can have that many rows.  Without and with it, in
// the same four: 96 tokens, top 8 of 128, 57 65, 178 187, 30 38, 91 99; 256 tokens, top 4 of 32,
// 56 74, 170 213, 29 44, 85 104; top 2 of 8, 46 29, 165 80, 30 20, 48 47; 1000 tokens, top 8 of
// 64, 324 138, 1111 423, 169 81, 559 232.  Slots say nothing of a strong skew: all tokens on
// one of 64 experts, 200 of them, 20 27, 45 47, 11 20, 23 23, and 1000, which are left out, too, 50
// 30, 152 49, 27 21, 77 37.  At top 8 of 128 the 400 tokens lose, 151 174, 500 524, 79 95, 253 273.
constexpr int kTileSlots = 2560;

tq_status run_product(const tq::MoeProduct &p, void *workspace, cudaStream_t stream) {
    const tq::MoeWorkspace L = tq::moe_layout(1, 1, 1, 0, 0);      // err and operand come first
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    cudaError_t e = cudaSuccess;
    const bool tiles = p.max_rows > kTileAbove && p.slots >= 8 * p.experts &&
                       (p.slots >= kTileSlots || p.slots > 48 * p.experts);
    unsigned *err = reinterpret_cast<unsigned *>(ws + L.err);
    if (tiles) e = tq::moe_tile_launch(p, kTileAbove, ws + L.operand, err, stream);
    if (e == cudaSuccess) e = tq::moe_stream_launch(p, tiles ? kTileAbove : p.slots, err, stream);
    return cuda_status(e);
}

}  // namespace

extern "C" {

tq_status tq_add_rmsnorm_rotq(const void *residual, int32_t residual_type, const void *delta,
                              int32_t delta_type, const uint16_t *gamma, int32_t m, int32_t n,
                              float eps, void *residual_out, uint16_t *x_out, int8_t *q, float *s,
                              tq_stream_t stream) {
    if (residual == nullptr || m < 1 || !width_ok(n) || !dtype_ok(residual_type)) return TQ_ERR_INVALID_ARG;
    if (delta != nullptr && !dtype_ok(delta_type)) return TQ_ERR_INVALID_ARG;
    if ((q == nullptr) != (s == nullptr)) return TQ_ERR_INVALID_ARG;
    if (q == nullptr && x_out == nullptr && residual_out == nullptr) return TQ_ERR_INVALID_ARG;
    if (!(eps >= 0.0f)) return TQ_ERR_INVALID_ARG;
    if (!aligned(residual, 16) || !aligned(delta, 16) || !aligned(gamma, 16) || !aligned(residual_out, 16) ||
        !aligned(x_out, 16) || !aligned(q, 16) || !aligned(s, 4))
        return TQ_ERR_ALIGNMENT;
    return cuda_status(tq::moe_norm_launch(residual, residual_type == TQ_BF16, delta, delta_type == TQ_BF16, gamma, m, n,
                                           eps, residual_out, x_out, q, s, reinterpret_cast<cudaStream_t>(stream)));
}

tq_status tq_moe_route(const void *logits, int32_t logits_type, int32_t m, int32_t experts,
                       int32_t topk, int32_t renormalize, int32_t *ids, float *weights,
                       tq_stream_t stream) {
    if (logits == nullptr || ids == nullptr || weights == nullptr) return TQ_ERR_INVALID_ARG;
    if (!dtype_ok(logits_type) || !route_sizes_ok(m, topk, experts)) return TQ_ERR_INVALID_ARG;
    if (!aligned(logits, logits_type == TQ_BF16 ? 2 : 4) || !aligned(ids, 4) || !aligned(weights, 4))
        return TQ_ERR_ALIGNMENT;
    return cuda_status(tq::moe_route_launch(logits, logits_type == TQ_BF16, m, experts, topk, renormalize != 0, ids,
                                            weights, reinterpret_cast<cudaStream_t>(stream)));
}

size_t tq_moe_workspace_bytes(int32_t m, int32_t topk, int32_t experts, int32_t hidden, int32_t inter) {
    if (!route_sizes_ok(m, topk, experts)) return 0;
    if (!(hidden == 0 && inter == 0) && (!width_ok(hidden) || !width_ok(inter))) return 0;
    return tq::moe_layout(m, topk, experts, hidden, inter).total;
}

tq_status tq_moe_read_error_word(uint32_t *value, tq_stream_t stream) {
    if (value == nullptr) return TQ_ERR_INVALID_ARG;
    cudaStream_t str = reinterpret_cast<cudaStream_t>(stream);
    unsigned bits[2] = {};
    cudaError_t e = tq::moe_stream_waits(&bits[0], str);
    if (e == cudaSuccess) e = tq::moe_tile_waits(&bits[1], str);
    if (e == cudaSuccess) e = cudaStreamSynchronize(str);
    if (e != cudaSuccess) return cuda_status(e);
    *value = bits[0] | bits[1];
    return tq_error_status(*value);
}

tq_status tq_moe_plan(const int32_t *ids, int32_t m, int32_t topk, int32_t experts, int32_t *offsets,
                      int32_t *rows, int32_t *pos, void *workspace, size_t workspace_bytes,
                      tq_stream_t stream) {
    if (ids == nullptr || offsets == nullptr || rows == nullptr || pos == nullptr) return TQ_ERR_INVALID_ARG;
    if (!route_sizes_ok(m, topk, experts)) return TQ_ERR_INVALID_ARG;
    if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(pos, 4)) return TQ_ERR_ALIGNMENT;
    const tq::MoeWorkspace L = tq::moe_layout(m, topk, experts, 0, 0);
    tq_status st = check_ws(workspace, workspace_bytes, L.total);
    if (st != TQ_OK) return st;
    int *hist = reinterpret_cast<int *>(static_cast<uint8_t *>(workspace) + L.hist);
    return cuda_status(tq::moe_plan_launch(ids, m, topk, experts, offsets, rows, pos, hist,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

tq_status tq_moe_gemv(const tq_experts *w, const int8_t *q, const float *s, int32_t m,
                      const int32_t *rows, const int32_t *offsets, int32_t slots, float *y,
                      void *workspace, size_t workspace_bytes, tq_stream_t stream) {
    tq_status st;
    if ((st = check_experts(w)) != TQ_OK) return st;
    if (y == nullptr) return TQ_ERR_INVALID_ARG;
    if ((st = check_rows(q, s, m, rows, offsets, slots)) != TQ_OK) return st;
    if (!aligned(y, 4)) return TQ_ERR_ALIGNMENT;
    if ((st = check_ws(workspace, workspace_bytes, tq::moe_product_bytes(slots, w->k))) != TQ_OK) return st;
    tq::MoeProduct p = product(w, nullptr, q, s, m, rows, offsets, slots);
    p.y = y;
    p.max_rows = slots;
    return run_product(p, workspace, reinterpret_cast<cudaStream_t>(stream));
}

tq_status tq_moe_gateup(const tq_experts *gate, const tq_experts *up, const int8_t *q,
                        const float *s, int32_t m, const int32_t *rows, const int32_t *offsets,
                        int32_t slots, uint16_t *h, void *workspace, size_t workspace_bytes,
                        tq_stream_t stream) {
    tq_status st;
    if ((st = check_experts(gate)) != TQ_OK) return st;
    if ((st = check_experts(up)) != TQ_OK) return st;
    if (!same_shape(gate, up) || h == nullptr) return TQ_ERR_INVALID_ARG;
    if ((st = check_rows(q, s, m, rows, offsets, slots)) != TQ_OK) return st;
    if (!aligned(h, 2)) return TQ_ERR_ALIGNMENT;
    if ((st = check_ws(workspace, workspace_bytes, tq::moe_product_bytes(slots, gate->k))) != TQ_OK) return st;
    tq::MoeProduct p = product(gate, up, q, s, m, rows, offsets, slots);
    p.h = h;
    p.max_rows = rows != nullptr && m < slots ? m : slots;
    return run_product(p, workspace, reinterpret_cast<cudaStream_t>(stream));
}

tq_status tq_moe_combine(const float *y, const int32_t *pos, const float *weights, int32_t m,
                         int32_t topk, int32_t slots, int32_t n, void *out, int32_t out_type,
                         tq_stream_t stream) {
    if (y == nullptr || pos == nullptr || weights == nullptr || out == nullptr) return TQ_ERR_INVALID_ARG;
    if (m < 1 || topk < 1 || topk > TQ_MOE_MAX_TOPK || slots < 1 || n < 4 || n % 4 != 0 || n > TQ_MOE_MAX_WIDTH ||
        !dtype_ok(out_type) || static_cast<int64_t>(m) * topk > TQ_MOE_MAX_SLOTS)
        return TQ_ERR_INVALID_ARG;
    if (!aligned(y, 16) || !aligned(out, 16) || !aligned(pos, 4) || !aligned(weights, 4)) return TQ_ERR_ALIGNMENT;
    return cuda_status(tq::moe_combine_launch(y, pos, weights, m, topk, slots, n, out, out_type == TQ_BF16,
                                              reinterpret_cast<cudaStream_t>(stream)));
}

tq_status tq_moe_ffn(const tq_experts *gate, const tq_experts *up, const tq_experts *down,
                     const int8_t *q, const float *s, const int32_t *ids, const float *weights,
                     int32_t m, int32_t topk, void *out, int32_t out_type, void *workspace,
                     size_t workspace_bytes, tq_stream_t stream) {
    tq_status st;
    if ((st = check_experts(gate)) != TQ_OK) return st;
    if ((st = check_experts(up)) != TQ_OK) return st;
    if ((st = check_experts(down)) != TQ_OK) return st;
    const int experts = gate->experts, hidden = gate->k, inter = gate->n;
    if (!same_shape(gate, up) || down->experts != experts || down->n != hidden || down->k != inter ||
        down->fmt != gate->fmt || !width_ok(inter))
        return TQ_ERR_INVALID_ARG;
    if (q == nullptr || s == nullptr || ids == nullptr || weights == nullptr || out == nullptr || !dtype_ok(out_type))
        return TQ_ERR_INVALID_ARG;
    if (!route_sizes_ok(m, topk, experts)) return TQ_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(s, 4) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(out, 16))
        return TQ_ERR_ALIGNMENT;
    const tq::MoeWorkspace L = tq::moe_layout(m, topk, experts, hidden, inter);
    if ((st = check_ws(workspace, workspace_bytes, L.total)) != TQ_OK) return st;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const auto at = [ws](size_t off) { return ws + off; };
    int *offsets = reinterpret_cast<int *>(at(L.offsets)), *rows = reinterpret_cast<int *>(at(L.rows)),
        *pos = reinterpret_cast<int *>(at(L.pos)), *hist = reinterpret_cast<int *>(at(L.hist));
    uint16_t *h = reinterpret_cast<uint16_t *>(at(L.h));
    int8_t *hq = reinterpret_cast<int8_t *>(at(L.hq));
    float *hs = reinterpret_cast<float *>(at(L.hs)), *y = reinterpret_cast<float *>(at(L.y));
    const int slots = m * topk;
    cudaStream_t str = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = tq::moe_plan_launch(ids, m, topk, experts, offsets, rows, pos, hist, str);
    if (e != cudaSuccess) return cuda_status(e);
    tq::MoeProduct a = product(gate, up, q, s, m, rows, offsets, slots);
    a.h = h;
    a.max_rows = m;
    if ((st = run_product(a, workspace, str)) != TQ_OK) return st;
    if ((e = tq::moe_rotq_launch(h, static_cast<int64_t>(slots) * (inter / 128), hq, hs, str)) != cudaSuccess)
        return cuda_status(e);
    tq::MoeProduct b = product(down, nullptr, hq, hs, slots, nullptr, offsets, slots);
    b.y = y;
    b.max_rows = m;
    if ((st = run_product(b, workspace, str)) != TQ_OK) return st;
    return cuda_status(tq::moe_combine_launch(y, pos, weights, m, topk, slots, hidden, out, out_type == TQ_BF16, str));
}

}  // extern "C"
