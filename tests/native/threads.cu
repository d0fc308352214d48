// Two host threads that call tq_moe_gemv in a loop, without an interpreter's lock between them.
#include <atomic>
#include <thread>

#include <cuda_runtime.h>

#include "tq_moe.h"

struct Product {
    const tq_experts *w;
    const int8_t *q;
    const float *s;
    const int32_t *offsets;
    int32_t slots;
    float *y;
    void *workspace;
    size_t workspace_bytes;
    cudaStream_t stream;
};

// gemv: the library's tq_moe_gemv.  Returns how many of the calls failed.
extern "C" int call_from_threads(decltype(&tq_moe_gemv) gemv, const Product *products, int count, int calls) {
    std::atomic<int> failed{0}, ready{0};
    std::thread threads[8];
    for (int t = 0; t < count; ++t)
        threads[t] = std::thread([&, t] {
            const Product &p = products[t];
            cudaStreamSynchronize(p.stream);
            ready.fetch_add(1);
            while (ready.load() < count) {}
            for (int i = 0; i < calls; ++i) {
                failed += gemv(p.w, p.q, p.s, p.slots, nullptr, p.offsets, p.slots, p.y, p.workspace, p.workspace_bytes,
                               reinterpret_cast<tq_stream_t>(p.stream)) != TQ_OK;
                if (i % 64 == 63) cudaStreamSynchronize(p.stream);
            }
            cudaStreamSynchronize(p.stream);
        });
    for (int t = 0; t < count; ++t) threads[t].join();
    return failed.load();
}
