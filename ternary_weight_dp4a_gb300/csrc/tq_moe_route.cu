// tq_moe_route.cu -- the router (top-k and softmax weights) and the plan: a
// stable counting sort of the (token, choice) slots by expert.
#include <cfloat>

#include <cuda_runtime.h>

#include "tq_device.cuh"
#include "tq_launch.h"
#include "tq_moe_internal.h"

namespace tq {
namespace {

constexpr uint32_t kFull = 0xffffffffu;

// Order-preserving key of a logit: larger floats have larger keys (-0 counts
// as +0, so that equal logits tie); 0 for -infinity and NaN, which are never
// chosen.
__device__ __forceinline__ uint32_t logit_key(float l) {
    if (!(l > -INFINITY)) return 0u;
    const uint32_t u = __float_as_uint(__fadd_rn(l, 0.0f));
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_logit(uint32_t k) {
    const float l = __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
    return fminf(l, FLT_MAX);
}

// One warp per token; lane l holds experts l, l + 32, ..  Each choice is one
// warp-wide maximum over the keys and one minimum over the indices that have it, so the
// choices' chain of reductions is the bound: 16384 tokens, top 8 of 256: 16.7 us, 8 tokens 2.1.
template <bool BF16, int PER>
__global__ void __launch_bounds__(256) route_kernel(const void *logits, int m, int experts, int topk,
                                                    int renorm, int *__restrict__ ids, float *__restrict__ weights) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (t >= m) return;
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        float l = -INFINITY;
        if (e < experts)
            l = BF16 ? bf16_bits_to_f32(static_cast<const uint16_t *>(logits)[t * experts + e])
                     : static_cast<const float *>(logits)[t * experts + e];
        key[i] = logit_key(l);
    }
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) best = max(best, key[i]);
    const uint32_t first = __reduce_max_sync(kFull, best);
    const float top = first != 0 ? key_logit(first) : 0.0f;
    float total = 0.0f;
    if (!renorm) {
#pragma unroll
        for (int i = 0; i < PER; ++i) total += key[i] != 0 ? expf(__fsub_rn(key_logit(key[i]), top)) : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
    }
    // lane j keeps choice j
    int my_id = -1;
    float my_e = 0.0f;
    for (int j = 0; j < topk; ++j) {
        uint32_t b = 0;
        int at = 0x7fffffff;
#pragma unroll
        for (int i = PER - 1; i >= 0; --i)
            if (key[i] >= b) { b = key[i]; at = lane + 32 * i; }   // the lowest of this lane's indices
        const uint32_t win = __reduce_max_sync(kFull, b);
        if (win == 0) break;
        const int e = __reduce_min_sync(kFull, b == win ? at : 0x7fffffff);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 32 * i == e) key[i] = 0;
        if (lane == j) {
            my_id = e;
            my_e = expf(__fsub_rn(key_logit(win), top));
        }
    }
    if (renorm) {
        total = my_e;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
    }
    if (lane < topk) {
        ids[t * topk + lane] = my_id;
        weights[t * topk + lane] = my_id >= 0 ? __fdiv_rn(my_e, total) : 0.0f;
    }
}

// ---------------------------------------------------------------------------
// The plan.  Slots are dealt to CTAs in chunks of kPlanChunk in order, one slot
// per thread.  count_kernel writes each chunk's slots per expert; scan_kernel
// turns them into the slots of the chunks before, and the sums; place_kernel
// adds every expert before each expert and ranks its slots: within a warp by
// match, across the warps by a prefix over per-warp counts in shared memory.
// One chunk needs place_kernel alone: 2.1 us.  Every step reads the chunks once, so the
// time is that of three launches until there are thousands of them: 131072 slots of 256
// experts 10.8 us.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int slot_expert(const int *ids, int64_t slot, int64_t slots, int experts) {
    if (slot >= slots) return -1;
    const int e = ids[slot];
    return e >= 0 && e < experts ? e : -1;
}

__global__ void __launch_bounds__(kPlanChunk) count_kernel(const int *ids, int64_t slots, int experts,
                                                           int *__restrict__ hist) {
    extern __shared__ int count[];
    pdl_launch_dependents();
    pdl_wait();
    for (int e = threadIdx.x; e < experts; e += kPlanChunk) count[e] = 0;
    __syncthreads();
    const int e = slot_expert(ids, static_cast<int64_t>(blockIdx.x) * kPlanChunk + threadIdx.x, slots, experts);
    if (e >= 0) atomicAdd(&count[e], 1);
    __syncthreads();
    for (int i = threadIdx.x; i < experts; i += kPlanChunk) hist[static_cast<int64_t>(blockIdx.x) * experts + i] = count[i];
}

// hist [chunks][experts] -> exclusive sums over the chunks; the whole sums go behind them.
// A CTA takes 32 experts, its warps a run of the chunks each.
__global__ void __launch_bounds__(1024) scan_kernel(int *hist, int chunks, int experts) {
    __shared__ int sum[32][33];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e = blockIdx.x * 32 + lane;
    const int per = (chunks + 31) / 32, first = min(warp * per, chunks), last = min(first + per, chunks);
    int *column = hist + e;
    int run = 0;
    if (e < experts) {
#pragma unroll 8
        for (int c = first; c < last; ++c) run += column[static_cast<int64_t>(c) * experts];
    }
    sum[warp][lane] = run;
    __syncthreads();
    if (e >= experts) return;
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < 32; ++w) {
        if (w == warp) before = all;
        all += sum[w][lane];
    }
    if (warp == 0) column[static_cast<int64_t>(chunks) * experts] = all;
    constexpr int kAhead = 8;                                    // loads under way before the stores
    for (int c0 = first; c0 < last; c0 += kAhead) {
        int v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) v[i] = c0 + i < last ? column[static_cast<int64_t>(c0 + i) * experts] : 0;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (c0 + i < last) column[static_cast<int64_t>(c0 + i) * experts] = before;
            before += v[i];
        }
    }
}

// shared memory: warp counts [32][experts] (16 bits), base [experts + 1], scan [32]
constexpr size_t place_smem(int experts) {
    return (experts + 1 + 32) * sizeof(int) + static_cast<size_t>(32) * experts * sizeof(uint16_t);
}

__global__ void __launch_bounds__(kPlanChunk) place_kernel(const int *ids, int64_t slots, int experts,
                                                           int topk, const int *hist,
                                                           int *__restrict__ offsets, int *__restrict__ rows,
                                                           int *__restrict__ pos) {
    extern __shared__ int smem[];
    int *base = smem;
    int *scan = base + experts + 1;
    uint16_t *wcount = reinterpret_cast<uint16_t *>(scan + 32);
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t slot = static_cast<int64_t>(blockIdx.x) * kPlanChunk + tid;
    const int mine = slot_expert(ids, slot, slots, experts);
    for (int i = tid; i < 32 * experts; i += kPlanChunk) wcount[i] = 0;
    __syncthreads();
    // rank among the lanes of this warp with the same expert
    const unsigned same = __match_any_sync(kFull, mine);
    const int rank = __popc(same & ((1u << lane) - 1));
    if (mine >= 0 && rank == 0) wcount[warp * experts + mine] = static_cast<uint16_t>(__popc(same));
    __syncthreads();
    // thread e: slots of expert e in this chunk, before it, and in all
    int before = 0, all = 0;
    if (tid < experts) {
        int run = 0;
        for (int w = 0; w < kPlanChunk / 32; ++w) {
            const int c = wcount[w * experts + tid];
            wcount[w * experts + tid] = static_cast<uint16_t>(run);
            run += c;
        }
        all = run;
        if (hist != nullptr) {
            before = hist[static_cast<int64_t>(blockIdx.x) * experts + tid];
            all = hist[static_cast<int64_t>(gridDim.x) * experts + tid];
        }
    }
    // exclusive scan of `all` over the experts (one per thread; experts <= 1024)
    int incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int v = scan[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(kFull, v, o);
            if (lane >= o) v += u;
        }
        scan[lane] = v;
    }
    __syncthreads();
    const int excl = incl - all + (warp > 0 ? scan[warp - 1] : 0);
    const int total = scan[31];
    if (tid < experts) {
        base[tid] = excl + before;
        if (blockIdx.x == 0) offsets[tid] = excl;
    }
    if (blockIdx.x == 0 && tid == 0) offsets[experts] = total;
    __syncthreads();
    if (slot < slots) {
        int p = -1;
        if (mine >= 0) {
            p = base[mine] + wcount[warp * experts + mine] + rank;
            rows[p] = static_cast<int>(slot / topk);
        }
        pos[slot] = p;
        if (slot >= total) rows[slot] = -1;
    }
}

template <bool BF16>
cudaError_t route_launch(const void *logits, int m, int experts, int topk, int renorm, int *ids, float *weights,
                         cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(m) + 7) / 8)), block(256);
#define TQ_ROUTE(PER) \
    return launch_pdl(route_kernel<BF16, PER>, grid, block, 0, stream, logits, m, experts, topk, renorm, ids, weights)
    if (experts <= 32) TQ_ROUTE(1);
    if (experts <= 64) TQ_ROUTE(2);
    if (experts <= 128) TQ_ROUTE(4);
    if (experts <= 256) TQ_ROUTE(8);
    if (experts <= 512) TQ_ROUTE(16);
    TQ_ROUTE(32);
#undef TQ_ROUTE
}

}  // namespace

cudaError_t moe_route_launch(const void *logits, bool bf16, int m, int experts, int topk, bool renorm, int *ids,
                             float *weights, cudaStream_t stream) {
    return bf16 ? route_launch<true>(logits, m, experts, topk, renorm, ids, weights, stream)
                : route_launch<false>(logits, m, experts, topk, renorm, ids, weights, stream);
}

cudaError_t moe_plan_launch(const int *ids, int m, int topk, int experts, int *offsets, int *rows, int *pos, int *hist,
                            cudaStream_t stream) {
    const int64_t slots = static_cast<int64_t>(m) * topk;
    const unsigned chunks = static_cast<unsigned>(ws_cdiv(slots, kPlanChunk));
    cudaError_t e = cudaSuccess;
    if (chunks > 1) {
        e = launch_pdl(count_kernel, dim3(chunks), dim3(kPlanChunk), experts * sizeof(int), stream, ids, slots, experts,
                       hist);
        if (e != cudaSuccess) return e;
        e = launch_pdl(scan_kernel, dim3((experts + 31) / 32), dim3(1024), 0, stream, hist, static_cast<int>(chunks),
                       experts);
        if (e != cudaSuccess) return e;
    }
    static SmemLimit limit;
    if ((e = limit.raise(place_kernel, place_smem(TQ_MOE_MAX_EXPERTS))) != cudaSuccess) return e;
    return launch_pdl(place_kernel, dim3(chunks), dim3(kPlanChunk), place_smem(experts), stream, ids, slots, experts, topk,
                      chunks > 1 ? static_cast<const int *>(hist) : nullptr, offsets, rows, pos);
}

}  // namespace tq
