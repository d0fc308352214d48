// tq_q4_api.cu -- the C ABI of the 4-bit products (declared in include/tq_q4.h):
// argument checks and dispatch.
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "tq_q4_internal.h"

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
bool sizes_ok(int32_t n, int32_t k) { return n >= 1 && n <= TQ_Q4_MAX_N && k >= 128 && k <= TQ_Q4_MAX_K && k % 128 == 0; }
bool group_ok(int32_t group) { return group == 32 || group == 64 || group == 128; }

tq_status check_weight(const tq_q4_weight *w) {
    if (w == nullptr || w->codes == nullptr || w->scales == nullptr || !sizes_ok(w->n, w->k) || !group_ok(w->group))
        return TQ_ERR_INVALID_ARG;
    if (!aligned(w->codes, 16) || !aligned(w->scales, 16) || !aligned(w->mins, 16)) return TQ_ERR_ALIGNMENT;
    return TQ_OK;
}

tq_status check_rows(const uint16_t *x, int32_t m, const void *y, size_t size) {
    if (x == nullptr || y == nullptr || m < 1 || m > TQ_Q4_MAX_ROWS) return TQ_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(y, size)) return TQ_ERR_ALIGNMENT;
    return TQ_OK;
}

tq::Q4Product product(const tq_q4_weight *w, const tq_q4_weight *up, const uint16_t *x, int32_t m) {
    tq::Q4Product p{};
    p.mats = up != nullptr ? 2 : 1;
    for (int i = 0; i < p.mats; ++i) {
        const tq_q4_weight *of = i == 0 ? w : up;
        p.codes[i] = of->codes;
        p.scales[i] = of->scales;
        p.mins[i] = of->mins;
    }
    p.n = w->n;
    p.k = w->k;
    p.group = w->group;
    p.x = x;
    p.m = m;
    return p;
}

tq_status run(const tq::Q4Product &p, void *workspace, size_t workspace_bytes, tq_stream_t stream) {
    cudaStream_t str = reinterpret_cast<cudaStream_t>(stream);
    if (p.m <= tq::kQ4StreamRows) return cuda_status(tq::q4_stream_launch(p, str));
    if (p.mins[0] != nullptr) {
        if (workspace == nullptr) return TQ_ERR_INVALID_ARG;
        if (!aligned(workspace, 256)) return TQ_ERR_ALIGNMENT;
        if (workspace_bytes < tq::q4_sums_bytes(p.m, p.k, p.group)) return TQ_ERR_WORKSPACE;
    }
    return cuda_status(tq::q4_tile_launch(p, static_cast<float *>(workspace), str));
}

}  // namespace

extern "C" {

size_t tq_q4_codes_bytes(int32_t n, int32_t k) {
    return sizes_ok(n, k) ? static_cast<size_t>(tq::q4_strips(n)) * (k / 128) * tq::kQ4ChunkBytes : 0;
}

size_t tq_q4_scales_bytes(int32_t n, int32_t k, int32_t group) {
    return sizes_ok(n, k) && group_ok(group) ? static_cast<size_t>(tq::q4_strips(n)) * tq::kQ4Strip * (k / group) * 2 : 0;
}

size_t tq_q4_workspace_bytes(int32_t m, int32_t k, int32_t group) {
    if (m < 1 || m > TQ_Q4_MAX_ROWS || !sizes_ok(1, k) || !group_ok(group) || m <= tq::kQ4StreamRows) return 0;
    return tq::q4_sums_bytes(m, k, group);
}

tq_status tq_q4_pack(const uint8_t *codes, const uint16_t *scales, const uint16_t *mins, int32_t n,
                     int32_t k, int32_t group, uint8_t *packed_codes, uint16_t *packed_scales,
                     uint16_t *packed_mins, tq_stream_t stream) {
    if (codes == nullptr || scales == nullptr || packed_codes == nullptr || packed_scales == nullptr || !sizes_ok(n, k) ||
        !group_ok(group) || (mins == nullptr) != (packed_mins == nullptr))
        return TQ_ERR_INVALID_ARG;
    if (!aligned(codes, 8) || !aligned(scales, 2) || !aligned(mins, 2) || !aligned(packed_codes, 16) ||
        !aligned(packed_scales, 16) || !aligned(packed_mins, 16))
        return TQ_ERR_ALIGNMENT;
    return cuda_status(tq::q4_pack_launch(codes, scales, mins, n, k, group, packed_codes, packed_scales, packed_mins,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

tq_status tq_q4_gemv(const tq_q4_weight *w, const uint16_t *x, int32_t m, void *y, int32_t y_type,
                     void *workspace, size_t workspace_bytes, tq_stream_t stream) {
    tq_status st = check_weight(w);
    if (st != TQ_OK) return st;
    if (y_type != TQ_F32 && y_type != TQ_BF16) return TQ_ERR_INVALID_ARG;
    if ((st = check_rows(x, m, y, y_type == TQ_BF16 ? 2 : 4)) != TQ_OK) return st;
    tq::Q4Product p = product(w, nullptr, x, m);
    p.y = y;
    p.y_bf16 = y_type == TQ_BF16;
    return run(p, workspace, workspace_bytes, stream);
}

tq_status tq_q4_gateup(const tq_q4_weight *gate, const tq_q4_weight *up, const uint16_t *x,
                       int32_t m, uint16_t *h, void *workspace, size_t workspace_bytes,
                       tq_stream_t stream) {
    tq_status st = check_weight(gate);
    if (st != TQ_OK) return st;
    if ((st = check_weight(up)) != TQ_OK) return st;
    if (gate->n != up->n || gate->k != up->k || gate->group != up->group || (gate->mins == nullptr) != (up->mins == nullptr))
        return TQ_ERR_INVALID_ARG;
    if ((st = check_rows(x, m, h, 2)) != TQ_OK) return st;
    tq::Q4Product p = product(gate, up, x, m);
    p.y = h;
    p.y_bf16 = true;
    return run(p, workspace, workspace_bytes, stream);
}

tq_status tq_q4_read_error_word(uint32_t *value, tq_stream_t stream) {
    if (value == nullptr) return TQ_ERR_INVALID_ARG;
    cudaStream_t str = reinterpret_cast<cudaStream_t>(stream);
    unsigned bits = 0;
    cudaError_t e = tq::q4_tile_waits(&bits, str);
    if (e == cudaSuccess) e = cudaStreamSynchronize(str);
    if (e != cudaSuccess) return cuda_status(e);
    *value = bits;
    return tq_error_status(bits);
}

}  // extern "C"
