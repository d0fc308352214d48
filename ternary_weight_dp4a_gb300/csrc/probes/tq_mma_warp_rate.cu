// tq_mma_warp_rate.cu -- throughput of tcgen05.mma by how it is issued: M = 128, f32 accumulators in tensor memory, kind::f16
// (bf16, K = 16, as the tile kernel of the 4-bit products) and kind::f8f6f4 (e4m3, K = 32, as the tensor-core kernels
// of the ternary products), A in tensor memory or in shared memory, B in shared memory, both with the 128-byte
// swizzle.  Every SM runs one CTA, whose first warp issues, either
//   together: the whole warp runs the loop, one elected thread's instructions are predicated on, or
//   in a branch that one thread takes.
// MMAs are committed and waited for in batches of 32 and of 256: the difference of the two is free of the commit and its
// wait.  Groups of four (one 128-byte row of operands) go into one accumulator or into as many as fit 256
// columns, in turn.
//
// Every tensor-memory column and every byte of shared memory that is read is written before, and every wait is bounded
// (error flags instead of a hang).  Build and run:
//   nvcc -gencode arch=compute_103a,code=sm_103a -O3 -o tq_mma_warp_rate tq_mma_warp_rate.cu
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include <cuda_runtime.h>

#define CK(x)                                                                                \
    do {                                                                                     \
        cudaError_t e_ = (x);                                                                \
        if (e_ != cudaSuccess) {                                                             \
            printf("CUDA %s at %d: %s\n", #x, __LINE__, cudaGetErrorString(e_));             \
            exit(1);                                                                         \
        }                                                                                    \
    } while (0)

constexpr uint32_t kABytes = 128 * 128, kBBytes = 256 * 128;    // rows of 64 bf16
constexpr size_t kSmem = 1024 + kABytes + kBBytes;

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
    const long long t0 = clock64();
    for (;;) {
        uint32_t ok;
        asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                     : "=r"(ok)
                     : "r"(bar), "r"(parity)
                     : "memory");
        if (ok) return true;
        if (clock64() - t0 > (1ll << 30)) return false;
    }
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// K-major, 128-byte swizzle: atoms of 8 rows x 128 bytes, 1024 bytes apart
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {
    uint64_t d = static_cast<uint64_t>((saddr & 0x3ffffu) >> 4);
    d |= 1ull << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= 1ull << 46;
    d |= 2ull << 61;
    return d;
}

#define MMA(KIND, A, AREG)                                                                     \
    asm volatile(                                                                             \
        "{ .reg .pred p, q; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0;\n"                    \
        "@q tcgen05.mma.cta_group::1.kind::" KIND " [%0], " A ", %2, %3, p; }" ::"r"(d),       \
        AREG, "l"(bd), "r"(idesc), "r"(accumulate), "r"(issue)                                \
        : "memory")

template <bool F8, bool A_SMEM>
__device__ __forceinline__ void mma(uint32_t issue, uint32_t d, uint32_t at, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t accumulate) {
    if constexpr (F8 && A_SMEM) MMA("f8f6f4", "%1", "l"(ad));
    else if constexpr (F8) MMA("f8f6f4", "[%1]", "r"(at));
    else if constexpr (A_SMEM) MMA("f16", "%1", "l"(ad));
    else MMA("f16", "[%1]", "r"(at));
}

// Tensor memory: A in the first 256 columns (four operands of 8 are used), accumulators in the others.
template <bool F8, bool A_SMEM>
__global__ void __launch_bounds__(128, 1) rate(int commits, int batch, int n, int accumulators, bool together, unsigned *err,
                                               long long *cycles) {
    extern __shared__ uint8_t raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t bar;
    __shared__ uint32_t tmem;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (threadIdx.x == 0) {
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&bar)) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (uint32_t i = threadIdx.x; i < (kABytes + kBBytes) / 4; i += 128) reinterpret_cast<uint32_t *>(sm)[i] = F8 ? 0x38383838u : 0x3f803f80u;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = tmem, lanes = static_cast<uint32_t>(warp * 32) << 16;
    for (int c0 = 0; c0 < 512; c0 += 16) {
        const uint32_t v = c0 < 256 ? (F8 ? 0x38383838u : 0x3f803f80u) : 0u;
        asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1,%1};" ::"r"(tb + lanes + c0), "r"(v)
                     : "memory");
    }
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t idesc = (1u << 4) | (F8 ? 0u : (1u << 7) | (1u << 10)) | (static_cast<uint32_t>(n >> 3) << 17) | (128u >> 4 << 24);
    const uint64_t a_desc = desc_sw128(smem_u32(sm)), b_desc = desc_sw128(smem_u32(sm + kABytes));
    const uint32_t stride = (n + 31) / 32 * 32, done = smem_u32(&bar);
    auto loop = [&](uint32_t issue) {
        const long long t0 = clock64();
        bool ok = true;
        uint32_t d = 0;
        int left = accumulators;
        for (int c = 0; c < commits && ok; ++c) {
            for (int m = 0; m < batch; m += 4) {
#pragma unroll
                for (int i = 0; i < 4; ++i) mma<F8, A_SMEM>(issue, tb + 256 + d, tb + 8 * i, a_desc + 2 * i, b_desc + 2 * i, idesc, i > 0);
                d += stride;
                if (--left == 0) {
                    left = accumulators;
                    d = 0;
                }
            }
            asm volatile(
                "{ .reg .pred q; setp.ne.b32 q, %1, 0;\n"
                "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(done),
                "r"(issue)
                : "memory");
            ok = mbar_wait(done, c & 1);
        }
        const long long t1 = clock64();
        if (!ok) atomicOr(err, 1u);
        if (issue) cycles[blockIdx.x] = t1 - t0;
    };
    if (warp == 0) {
        uint32_t one;
        asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(one));
        if (together) loop(one);
        else if (threadIdx.x == 0) loop(1);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tb) : "memory");
}

struct Card {
    int sms;
    unsigned *err;
    long long *cycles, *host;
};

// Cycles per batch, the mean over the SMs.
template <bool F8, bool A_SMEM>
double run(const Card &card, int batch, int n, int accumulators, bool together) {
    const int commits = 200;
    CK(cudaFuncSetAttribute(rate<F8, A_SMEM>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem)));
    CK(cudaMemset(card.err, 0, 4));
    rate<F8, A_SMEM><<<card.sms, 128, kSmem>>>(commits, batch, n, accumulators, together, card.err, card.cycles);
    CK(cudaGetLastError());
    CK(cudaDeviceSynchronize());
    unsigned bad = 0;
    CK(cudaMemcpy(card.host, card.cycles, sizeof(long long) * card.sms, cudaMemcpyDeviceToHost));
    CK(cudaMemcpy(&bad, card.err, 4, cudaMemcpyDeviceToHost));
    if (bad) {
        printf("a wait ran out\n");
        exit(1);
    }
    double mean = 0;
    for (int i = 0; i < card.sms; ++i) mean += static_cast<double>(card.host[i]) / card.sms;
    return mean / commits;
}

template <bool F8, bool A_SMEM>
void table(const Card &card) {
    for (int together = 1; together >= 0; --together)
        for (int n : {16, 32, 64, 96, 128, 176, 192, 224, 256}) {
            const int most = 256 / ((n + 31) / 32 * 32);
            for (int accumulators = 1; accumulators <= most; accumulators += most > 1 ? most - 1 : 1) {
                const double few = run<F8, A_SMEM>(card, 32, n, accumulators, together), many = run<F8, A_SMEM>(card, 256, n, accumulators, together);
                const double per = (many - few) / 224;
                printf("%s, A in %s memory, issued %s, N %3d, accumulators %d: %6.1f cycles in batches of 32, %6.1f of 256, difference %6.1f (%.0f MACs per cycle and SM)\n",
                       F8 ? "f8f6f4 K 32" : "f16 K 16", A_SMEM ? "shared" : "tensor", together ? "together" : "in a branch", n, accumulators, few / 32,
                       many / 256, per, 128.0 * n * (F8 ? 32 : 16) / per);
            }
        }
}

int main() {
    Card card{};
    CK(cudaDeviceGetAttribute(&card.sms, cudaDevAttrMultiProcessorCount, 0));
    CK(cudaMalloc(&card.err, 4));
    CK(cudaMalloc(&card.cycles, sizeof(long long) * card.sms));
    card.host = static_cast<long long *>(malloc(sizeof(long long) * card.sms));
    table<false, false>(card);
    table<false, true>(card);
    table<true, false>(card);
    table<true, true>(card);
    free(card.host);
    return 0;
}
