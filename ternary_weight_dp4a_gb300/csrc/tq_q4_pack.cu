// tq_q4_pack.cu -- 4-bit matrices into the packed layout of include/tq_q4.h: a
// load-time step, one thread per packed word and per packed scale.
#include <cuda_runtime.h>

#include <cstdint>

#include "tq_q4_internal.h"

namespace tq {
namespace {

// One thread per 32-bit word: the codes of 8 consecutive values of one row.
__global__ void __launch_bounds__(256) q4_pack_codes_kernel(const uint8_t *codes, int n, int k, int64_t words, uint32_t *out) {
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (w >= words) return;
    const int64_t block = w >> 8;                       // (strip, chunk)
    const int in = static_cast<int>(w & 255);
    const int chunks = k >> 7;
    const int64_t strip = block / chunks;
    const int chunk = static_cast<int>(block - strip * chunks);
    const int g = in & 3, q = (in >> 2) & 3, r = (in >> 4) & 7, half = in >> 7;
    const int64_t row = strip * kQ4Strip + half * 8 + r;
    uint32_t v = 0x88888888u;                           // a padded row: codes 8
    if (row < n) {
        const uint2 c = *reinterpret_cast<const uint2 *>(codes + row * k + chunk * 128 + g * 32 + q * 8);
        v = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t code = ((j < 4 ? c.x : c.y) >> (8 * (j & 3))) & 15u;
            v |= code << (4 * (j / 2 + 4 * (j & 1)));
        }
    }
    out[w] = v;
}

__global__ void __launch_bounds__(256) q4_pack_scales_kernel(const uint16_t *scales, const uint16_t *mins, int n, int groups,
                                                             int per, int64_t entries, uint16_t *out, uint16_t *out_mins) {
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (w >= entries) return;
    const int64_t block = w / (16 * per);
    const int in = static_cast<int>(w - block * (16 * per));
    const int chunks = groups / per;
    const int64_t strip = block / chunks;
    const int chunk = static_cast<int>(block - strip * chunks);
    const int p = in % per, slot = in / per;
    const int64_t row = strip * kQ4Strip + (slot & 1) * 8 + (slot >> 1);
    const int64_t from = row * groups + chunk * per + p;
    out[w] = row < n ? scales[from] : 0;
    if (mins != nullptr) out_mins[w] = row < n ? mins[from] : 0;
}

}  // namespace

cudaError_t q4_pack_launch(const uint8_t *codes, const uint16_t *scales, const uint16_t *mins, int n, int k, int group,
                           uint8_t *out_codes, uint16_t *out_scales, uint16_t *out_mins, cudaStream_t stream) {
    const int64_t blocks = q4_strips(n) * (k / 128), words = blocks * (kQ4ChunkBytes / 4);
    q4_pack_codes_kernel<<<static_cast<unsigned>((words + 255) / 256), 256, 0, stream>>>(
        codes, n, k, words, reinterpret_cast<uint32_t *>(out_codes));
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int per = 128 / group;
    const int64_t entries = blocks * 16 * per;
    q4_pack_scales_kernel<<<static_cast<unsigned>((entries + 255) / 256), 256, 0, stream>>>(
        scales, mins, n, k / group, per, entries, out_scales, out_mins);
    return cudaGetLastError();
}

}  // namespace tq
