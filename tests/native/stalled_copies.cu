// The stream kernel over copies that never complete: every stage expects 16 bytes more than are
// copied, so each of its waits runs out.
#include "tq_device.cuh"
#define mbar_arrive_expect_tx(bar, bytes) (mbar_arrive_expect_tx)(bar, (bytes) + 16)
#include "tq_moe_stream.cu"

extern "C" int lost_waits(unsigned *bits) {
    const cudaError_t e = tq::moe_stream_waits(bits, nullptr);
    return e != cudaSuccess ? e : cudaStreamSynchronize(nullptr);
}

extern "C" int stalled_product(const uint8_t *codes, const uint16_t *scales, int experts, int n, int k, int fmt,
                               const int8_t *q, const float *s, const int *offsets, int slots, float *y, unsigned *err) {
    tq::MoeProduct p{};
    p.codes[0] = codes;
    p.scales[0] = scales;
    p.experts = experts;
    p.n = n;
    p.k = k;
    p.fmt = fmt;
    p.q = q;
    p.s = s;
    p.m = p.slots = p.max_rows = slots;
    p.offsets = offsets;
    p.y = y;
    return tq::moe_stream_launch(p, slots, err, nullptr);
}
