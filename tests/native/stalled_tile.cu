// The tile kernel of the 4-bit products over copies that never complete: every stage expects `stall` bytes more than are
// copied, so that the waits for it run out.  With 0 it is the library's kernel.
#include "tq_device.cuh"
__device__ unsigned stall = 16;
#define mbar_arrive_expect_tx(bar, bytes) (mbar_arrive_expect_tx)(bar, (bytes) + stall)
#include "tq_q4_tile.cu"

extern "C" int set_stall(unsigned bytes) { return cudaMemcpyToSymbol(stall, &bytes, sizeof(bytes)); }

extern "C" int lost_waits(unsigned *bits) {
    const cudaError_t e = tq::q4_tile_waits(bits, nullptr);
    return e != cudaSuccess ? e : cudaStreamSynchronize(nullptr);
}

extern "C" int product(const uint8_t *codes, const uint16_t *scales, const uint16_t *mins, int n, int k, int group,
                       const uint16_t *x, int m, float *y, float *sums, void *stream) {
    tq::Q4Product p{};
    p.mats = 1;
    p.codes[0] = codes;
    p.scales[0] = scales;
    p.mins[0] = mins;
    p.n = n;
    p.k = k;
    p.group = group;
    p.x = x;
    p.m = m;
    p.y = y;
    return tq::q4_tile_launch(p, sums, static_cast<cudaStream_t>(stream));
}
