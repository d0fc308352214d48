// Every fp32 gate through the tile kernel's SiLU (two at a time, without a branch for ordinary
// arguments) and through tq_silu: the number of gates whose bits differ, and one of them.
#include "tq_moe_codes.cuh"

namespace {

__global__ void compare(unsigned long long *differ, unsigned *example) {
    constexpr int kPer = 8;                          // the tile kernel's number of gates at a time
    const uint64_t step = static_cast<uint64_t>(gridDim.x) * blockDim.x * kPer;
    for (uint64_t at = (static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * kPer; at < 1ull << 32; at += step) {
        float g[kPer], s[kPer];
        for (int i = 0; i < kPer; ++i) g[i] = __uint_as_float(static_cast<uint32_t>(at) + i);
        tq::moe_silu(g, s);
        for (int i = 0; i < kPer; ++i) {
            const float want = tq::tq_silu(g[i]);
            const bool same = __float_as_uint(s[i]) == __float_as_uint(want) || (s[i] != s[i] && want != want);
            if (!same) {
                atomicAdd(differ, 1ull);
                *example = __float_as_uint(g[i]);
            }
        }
    }
}

}  // namespace

// differ, example: device memory, zero before the call.
extern "C" int silu_compare(unsigned long long *differ, unsigned *example) {
    compare<<<152 * 8, 256>>>(differ, example);
    return cudaGetLastError();
}
