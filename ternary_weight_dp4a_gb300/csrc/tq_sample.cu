// tq_sample.cu -- a token for each row of logits: temperature, top-k, min-p, top-p and the draw
// (include/tq_sample.h).
//
// The kernel keeps a row's cut as a place in the order of descending logits with ties to the
// lowest index: (key, index) of the last that stays, the key being the logit's bits made ascending.  top-k
// and top-p are the same search, for the place at which a sum over the order reaches a target: of
// ones, or of weights; min-p is a threshold on the logit.  The draw is a search over the indices.
//
// Weights are whole numbers: 2^42 exp((l - l_max) / T), rounded.  Sums of them are exact, so
// no result depends on how a row is split, and a border (a sum that equals a target in real
// arithmetic, as with equal logits) is met exactly.  exp is 2^(i/32) from a table of 32 (31-bit mantissas) times 2^r,
// |r| <= 1/64, by its Taylor polynomial; the argument is held as the sum of two
// fp32 numbers (difference by Knuth's TwoSum; product by fused multiply-add), so that the error is
// 2^-30 of a weight.  fp32 alone would move one border in some thousand draws; binary64 runs at
// 1/60 of the rate here.
#include <cuda_runtime.h>

#include <cstdint>

#include "tq.h"
#include "tq_device.cuh"
#include "tq_launch.h"
#include "tq_sample.h"

namespace tq {
void record_cuda_error(int e);

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 256;
constexpr int kOneBits = 42;                    // the largest weight is 2^42: a sum of 2^20 stays below 2^63
constexpr uint32_t kKeyNone = 0x007fffffu;      // key of -infinity: no candidate
constexpr float kColdest = 1.5777218104420236e-30f;     // 2^-99: below, as 0

__constant__ uint32_t kExp2[32] = {             // 2^(31 + i/32)
    0x80000000u, 0x82cd8699u, 0x85aac368u, 0x88980e81u, 0x8b95c1e4u, 0x8ea4398bu, 0x91c3d374u, 0x94f4efa9u,
    0x9837f052u, 0x9b8d39bau, 0x9ef53261u, 0xa2704303u, 0xa5fed6aau, 0xa9a15ab5u, 0xad583eeau, 0xb123f582u,
    0xb504f334u, 0xb8fbaf47u, 0xbd08a39fu, 0xc12c4ccau, 0xc5672a11u, 0xc9b9bd86u, 0xce248c15u, 0xd2a81d92u,
    0xd744fccbu, 0xdbfbb798u, 0xe0ccdeecu, 0xe5b906e7u, 0xeac0c6e8u, 0xefe4b99cu, 0xf5257d15u, 0xfa83b2dbu};

struct SampleArgs {
    const void *logits;
    int m, vocab, cluster;
    const float *temperature;
    const int *top_k;
    const float *top_p, *min_p, *uniform;
    int *ids;
    float *probs;
};

struct Shared {
    unsigned long long hist[kBins];
    unsigned long long warp_sum[kWarps];
    unsigned long long cta_sum;
    uint32_t cta_max;
    int found;
    uint32_t exp2[32];
    uint32_t bin;
    unsigned long long above;
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void sync_all(int cluster) {
    if (cluster > 1) asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
    else __syncthreads();
}

__device__ __forceinline__ uint32_t peer(const void *p, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}

__device__ __forceinline__ unsigned long long ld_peer_u64(const unsigned long long *p, int rank, int cluster) {
    if (cluster == 1) return *p;
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(peer(p, rank)) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t ld_peer_u32(const uint32_t *p, int rank, int cluster) {
    if (cluster == 1) return *p;
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer(p, rank)) : "memory");
    return v;
}

__device__ __forceinline__ void st_peer_s32(int *p, int rank, int cluster, int v) {
    if (cluster == 1) *p = v;
    else asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(peer(p, rank)), "r"(v) : "memory");
}

// Ascending in the logit; -0 is +0, NaN is -infinity, +infinity the largest finite number of the type.
template <bool BF16>
__device__ __forceinline__ uint32_t key_of(float l) {
    if (l != l) return kKeyNone;
    l = fminf(l, BF16 ? 3.3895313892515355e38f : 3.4028234663852886e38f) + 0.0f;
    const uint32_t b = __float_as_uint(l);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float logit_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// One row's weights.  Logits are halved so that no difference overflows.
struct Weights {
    float half_max, ch, cl;
    bool equal;                                 // infinite temperature

    __device__ __forceinline__ void set(uint32_t max_key, float t) {
        half_max = 0.5f * logit_of(max_key);
        equal = t > 3.4028234663852886e38f;
        const double c = 2.0 * 1.4426950408889634074 / static_cast<double>(t);
        ch = static_cast<float>(c);
        cl = static_cast<float>(c - static_cast<double>(ch));
    }

    __device__ __forceinline__ unsigned long long of(uint32_t key, const uint32_t *exp2) const {
        if (equal) return 1ull << kOneBits;
        const float l = 0.5f * logit_of(key), b = -half_max;
        const float d = __fadd_rn(l, b);
        const float bp = __fsub_rn(d, l);
        const float dl = __fadd_rn(__fsub_rn(l, __fsub_rn(d, bp)), __fsub_rn(b, bp));
        if (__fmul_rn(d, ch) < -64.0f) return 0;
        const float t = __fmaf_rn(d, ch, 393216.0f);                       // 1.5 * 2^18: a multiple of 1/32
        const float whole = __fsub_rn(t, 393216.0f);
        float r = __fmaf_rn(d, ch, -whole);
        r = __fmaf_rn(d, cl, r);
        r = __fmaf_rn(dl, ch, r);
        float q = __fmaf_rn(r, 9.6181291e-3f, 5.5504109e-2f);              // ln(2)^j / j!
        q = __fmaf_rn(r, q, 2.4022651e-1f);
        q = __fmaf_rn(r, q, 6.9314718e-1f);
        q = __fmul_rn(r, q);
        const int at = __float_as_int(t) - __float_as_int(393216.0f);      // 32 * (exponent), <= 0
        const uint32_t m = exp2[at & 31];
        const uint32_t w = m + static_cast<uint32_t>(__mulhi(static_cast<int>(m >> 1), __float2int_rn(q * 137438953472.0f)) >> 4);
        // w * 2^(floor(at / 32) - 31), scaled by 2^42 and rounded
        const int down = -(at >> 5);
        return ((static_cast<unsigned long long>(w) << (kOneBits - 31 + 1) >> min(down, 63)) + 1) >> 1;
    }
};

// The place in the order up to which a row's entries stay.
struct Cut {
    uint32_t key;
    int index;
    __device__ __forceinline__ bool keeps(uint32_t k, int i) const { return k > key || (k == key && i <= index); }
};

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <bool BF16>
struct Row {
    const void *logits;
    int from, to;                               // this CTA's part
    int seg_from, seg_to;                       // this warp's
    int rank, cluster;
    Shared &sm;

    __device__ __forceinline__ uint32_t key(int i) const {
        if constexpr (BF16) return key_of<true>(bf16_bits_to_f32(static_cast<const uint16_t *>(logits)[i]));
        else return key_of<false>(static_cast<const float *>(logits)[i]);
    }

    // Sum over the cluster of each thread's v.  base: the sum of the CTAs before; warp sums stay in sm.warp_sum.
    __device__ unsigned long long total(unsigned long long v, unsigned long long *base) const {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        v = warp_sum(v);
        if (lane == 0) sm.warp_sum[warp] = v;
        __syncthreads();
        if (threadIdx.x == 0) {
            unsigned long long s = 0;
            for (int w = 0; w < kWarps; ++w) s += sm.warp_sum[w];
            sm.cta_sum = s;
        }
        sync_all(cluster);
        unsigned long long all = 0, before = 0;
        for (int r = 0; r < cluster; ++r) {
            if (r == rank) before = all;
            all += ld_peer_u64(&sm.cta_sum, r, cluster);
        }
        sync_all(cluster);
        *base = before;
        return all;
    }

    // The lowest index at which the sum of value(i) over the indices up to it exceeds target (below the total),
    // for the warp sums and base that total() has left.  Runs on the warp that has it; -1 on the others.
    template <typename Value>
    __device__ int ordered(unsigned long long target, unsigned long long base, Value value) const {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        for (int w = 0; w < warp; ++w) base += sm.warp_sum[w];
        if (target < base || target >= base + sm.warp_sum[warp]) return -1;
        for (int i = seg_from; i < seg_to; i += 32) {
            unsigned long long v = i + lane < seg_to ? value(i + lane) : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, base + v > target);
            if (hit) return i + __ffs(hit) - 1;
            base += __shfl_sync(0xffffffffu, v, 31);
        }
        return -1;
    }

    // Narrow the cut to the shortest run of the order whose sum of value(key) reaches target (1 .. the sum of all that stay).
    template <typename Value>
    __device__ void narrow(Cut &cut, unsigned long long target, Value value) const {
        const int tid = threadIdx.x, lane = tid & 31;
        uint32_t prefix = 0;
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int b = tid; b < kBins; b += kThreads) sm.hist[b] = 0;
            __syncthreads();
            for (int i = seg_from + lane; i < seg_to; i += 32) {
                const uint32_t k = key(i);
                if (!cut.keeps(k, i) || (shift < 24 && k >> (shift + 8) != prefix)) continue;
                atomicAdd(&sm.hist[(k >> shift) & 255], value(k));
            }
            sync_all(cluster);
            unsigned long long mine = 0;
            if (tid < kBins)
                for (int r = 0; r < cluster; ++r) mine += ld_peer_u64(&sm.hist[kBins - 1 - tid], r, cluster);
            sync_all(cluster);
            if (tid < kBins) sm.hist[tid] = mine;               // descending bins now
            __syncthreads();
            if (tid == 0) {
                unsigned long long above = 0;
                int b = 0;
                while (b < kBins - 1 && above + sm.hist[b] < target) above += sm.hist[b++];
                sm.bin = kBins - 1 - b;
                sm.above = above;
            }
            __syncthreads();
            prefix = prefix << 8 | sm.bin;
            target -= sm.above;
            __syncthreads();
        }
        // equal keys have equal values: the first `need` of them in the order of the indices
        const unsigned long long each = value(prefix);
        const unsigned long long need = (target + each - 1) / each;
        auto tie = [&](int i) -> unsigned long long {
            const uint32_t k = key(i);
            return k == prefix && cut.keeps(k, i);
        };
        unsigned long long n = 0, base;
        for (int i = seg_from + lane; i < seg_to; i += 32) n += tie(i);
        total(n, &base);
        const int at = ordered(need - 1, base, tie);
        if (at >= 0 && lane == 0)
            for (int r = 0; r < cluster; ++r) st_peer_s32(&sm.found, r, cluster, at);
        sync_all(cluster);
        cut.key = prefix;
        cut.index = sm.found;
        sync_all(cluster);
    }
};

// floor(f * s) for a finite f in 0 .. 1.
__device__ __forceinline__ unsigned long long scaled(float f, unsigned long long s, bool up) {
    const uint32_t b = __float_as_uint(f);
    const int e = b >> 23;
    const unsigned long long mant = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
    const int shift = 150 - (e ? e : 1);                                   // f = mant * 2^-shift, 23 <= shift <= 149
    const unsigned long long lo = mant * s, hi = __umul64hi(mant, s);
    unsigned long long v;
    bool rest;
    if (shift < 64) {
        v = hi << (64 - shift) | lo >> shift;
        rest = (lo & ((1ull << shift) - 1)) != 0;
    } else {
        const int more = shift - 64;
        v = more < 64 ? hi >> more : 0;
        rest = lo != 0 || (more < 64 ? (hi & ((1ull << more) - 1)) != 0 : hi != 0);
    }
    return v + (up && rest);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
    __shared__ Shared sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = a.cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int row = blockIdx.x / a.cluster;
    if (tid < 32) sm.exp2[tid] = kExp2[tid];
    pdl_launch_dependents();
    pdl_wait();

    const int part = (a.vocab + a.cluster - 1) / a.cluster;
    Row<BF16> v{static_cast<const uint8_t *>(a.logits) + static_cast<int64_t>(row) * a.vocab * (BF16 ? 2 : 4), 0, 0, 0, 0, rank, a.cluster, sm};
    v.from = min(rank * part, a.vocab);
    v.to = min(v.from + part, a.vocab);
    const int seg = ((v.to - v.from + kWarps - 1) / kWarps + 31) / 32 * 32;
    v.seg_from = min(v.from + warp * seg, v.to);
    v.seg_to = min(v.seg_from + seg, v.to);

    // the largest
    uint32_t top = kKeyNone;
    for (int i = v.seg_from + lane; i < v.seg_to; i += 32) top = max(top, v.key(i));
    top = __reduce_max_sync(0xffffffffu, top);
    if (tid == 0) sm.cta_max = kKeyNone;
    __syncthreads();
    if (lane == 0) atomicMax(&sm.cta_max, top);
    sync_all(a.cluster);
    for (int r = 0; r < a.cluster; ++r) top = max(top, ld_peer_u32(&sm.cta_max, r, a.cluster));
    sync_all(a.cluster);
    if (top == kKeyNone) {
        if (rank == 0 && tid == 0) {
            a.ids[row] = -1;
            if (a.probs != nullptr) a.probs[row] = 0.0f;
        }
        return;
    }

    const float t = a.temperature != nullptr ? a.temperature[row] : 1.0f;
    unsigned long long base;
    if (!(t >= kColdest)) {                     // the first of the order
        auto tie = [&](int i) -> unsigned long long { return v.key(i) == top; };
        unsigned long long n = 0;
        for (int i = v.seg_from + lane; i < v.seg_to; i += 32) n += tie(i);
        v.total(n, &base);
        const int at = v.ordered(0, base, tie);
        if (at >= 0 && lane == 0) {
            a.ids[row] = at;
            if (a.probs != nullptr) a.probs[row] = 1.0f;
        }
        return;
    }
    Weights w;
    w.set(top, t);
    Cut cut{kKeyNone, -1};

    const int k = a.top_k != nullptr ? a.top_k[row] : 0;
    if (k > 0 && k < a.vocab) {
        unsigned long long n = 0;
        for (int i = v.seg_from + lane; i < v.seg_to; i += 32) n += v.key(i) > kKeyNone;
        n = v.total(n, &base);
        if (static_cast<unsigned long long>(k) < n) v.narrow(cut, k, [](uint32_t) { return 1ull; });
    }
    const float floor = a.min_p != nullptr ? a.min_p[row] : 0.0f;
    if (floor > 0.0f && !w.equal) {
        // w >= min_p  <=>  l >= l_max + T ln(min_p)
        const double least = static_cast<double>(logit_of(top)) + static_cast<double>(t) * log(static_cast<double>(fminf(floor, 1.0f)));
        const uint32_t key = min(key_of<false>(__double2float_ru(least)), top) - 1;
        if (key >= cut.key) cut = Cut{key, -1};
    }
    auto weight = [&](uint32_t key) { return w.of(key, sm.exp2); };
    const float p = a.top_p != nullptr ? a.top_p[row] : 1.0f;
    if (p < 1.0f) {
        unsigned long long s = 0;
        for (int i = v.seg_from + lane; i < v.seg_to; i += 32) {
            const uint32_t key = v.key(i);
            if (cut.keeps(key, i)) s += weight(key);
        }
        s = v.total(s, &base);
        const unsigned long long target = p > 0.0f ? scaled(p, s, true) : 1;
        v.narrow(cut, target > 0 ? target : 1, weight);
    }
    auto kept = [&](int i) -> unsigned long long {
        const uint32_t key = v.key(i);
        return cut.keeps(key, i) ? weight(key) : 0;
    };
    unsigned long long s = 0;
    for (int i = v.seg_from + lane; i < v.seg_to; i += 32) s += kept(i);
    s = v.total(s, &base);
    float u = a.uniform[row];
    u = u > 0.0f ? fminf(u, 1.0f) : 0.0f;
    const unsigned long long target = min(scaled(u, s, false), s - 1);
    const int at = v.ordered(target, base, kept);
    if (at >= 0 && lane == 0) {
        a.ids[row] = at;
        if (a.probs != nullptr) a.probs[row] = static_cast<float>(static_cast<double>(kept(at)) / static_cast<double>(s));
    }
}

cudaError_t sample_launch(SampleArgs a, bool bf16, cudaStream_t stream) {
    a.cluster = 1;
    while (a.cluster < kMaxCluster && a.vocab > a.cluster * 8192) a.cluster *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.m) * a.cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster > 1 ? 2 : 1;
    return bf16 ? cudaLaunchKernelEx(&cfg, sample_kernel<true>, a) : cudaLaunchKernelEx(&cfg, sample_kernel<false>, a);
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace
}  // namespace tq

extern "C" tq_status tq_sample(const void *logits, int32_t logits_type, int32_t m, int32_t vocab,
                               const float *temperature, const int32_t *top_k, const float *top_p,
                               const float *min_p, const float *uniform, int32_t *ids, float *probs,
                               tq_stream_t stream) {
    if (logits == nullptr || uniform == nullptr || ids == nullptr) return TQ_ERR_INVALID_ARG;
    if ((logits_type != TQ_F32 && logits_type != TQ_BF16) || m < 1 || m > TQ_SAMPLE_MAX_ROWS || vocab < 1 ||
        vocab > TQ_SAMPLE_MAX_VOCAB)
        return TQ_ERR_INVALID_ARG;
    if (!tq::aligned(logits, logits_type == TQ_BF16 ? 2 : 4) || !tq::aligned(temperature, 4) || !tq::aligned(top_k, 4) ||
        !tq::aligned(top_p, 4) || !tq::aligned(min_p, 4) || !tq::aligned(uniform, 4) || !tq::aligned(ids, 4) ||
        !tq::aligned(probs, 4))
        return TQ_ERR_ALIGNMENT;
    tq::SampleArgs a{};
    a.logits = logits;
    a.m = m;
    a.vocab = vocab;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.uniform = uniform;
    a.ids = ids;
    a.probs = probs;
    const cudaError_t e = tq::sample_launch(a, logits_type == TQ_BF16, reinterpret_cast<cudaStream_t>(stream));
    if (e == cudaSuccess) return TQ_OK;
    tq::record_cuda_error(static_cast<int>(e));
    return TQ_ERR_CUDA;
}
