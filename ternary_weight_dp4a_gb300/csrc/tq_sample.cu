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
// arithmetic, as with equal logits) is met exactly.  exp is 2^(i/32) from a table of 32 (31 bits) times 2^r,
// |r| <= 1/64, by its Taylor polynomial; the argument is held as the sum of two
// fp32 numbers (difference by Knuth's TwoSum; product by fused multiply-add), so that the error is
// 2^-30 of a weight and half a unit, 2^-43 (over a flat tail of 2^20 weights of a unit or so, 2^-23 of the sum).  fp32 alone
// would move one border in some thousand draws; binary64 runs at 1/60 of the rate here.
//
// A cluster of CTAs has a row, a part of it in each CTA's shared memory; the first CTA finishes.
//   top_k <= 512: the top_k-th largest of a CTA's threads' maxima bounds the cut from below, so a few
//     times top_k entries are candidates; the first CTA sorts them and does the rest on them.  (Near 512 the bound
//     is that of almost all threads, and where one CTA has a row they are more than its list holds: see below.  256
//     rows of 131072: top_k 50 84 us, 300 93, 400 111, 512 1980, 1000 2040.)
//   top_p: a histogram of the weights over 1024 bins, even in the logit, brackets the cut to a bin and 0.02%
//     of the sum; one pass then adds up the exact weights above the bracket and lists its entries,
//     and the first CTA sorts those.  (A bin counts in whole numbers and may pass 2^32 where a CTA has more than
//     2^18 entries: the bracket is checked against the exact sums, and one that misses takes the radix search.)
//   the draw: every warp's segment has its sum, the first CTA finds the segment and reads it again.
// Where candidates do not fit their list (thousands of equal logits, or a top_k beyond), the
// cut is found by a radix search over the key's bytes, which takes any input.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <type_traits>

#include "tq.h"
#include "tq_device.cuh"
#include "tq_limits.h"
#include "tq_sample.h"

namespace tq {
void record_cuda_error(int e);

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2 * kThreads;             // of the histogram
constexpr int kRadix = 256;                     // of the radix search
constexpr int kList = 4096;                     // candidates of a row, sorted by its first CTA
constexpr int local_most(int cluster) { return cluster == 1 ? kList : 2 * kList / cluster; }    // of one CTA
constexpr int kSmallK = kThreads;               // top_k up to this: by the threads' maxima
constexpr float kNats = 24.0f;                  // the histogram's range of ln(weight)
constexpr float kSlack = 1e-4f;                 // of the estimated sums (the neglected terms are 1e-4 of each bin, and alike)
constexpr int kOneBits = 42;                    // the largest weight is 2^42: a sum of 2^20 stays below 2^63
constexpr float kColdest = 1.5777218104420236e-30f;     // 2^-99: below, as 0

typedef unsigned long long u64;

__constant__ uint32_t kExp2[32] = {             // 2^(30 + i/32)
    0x40000000u, 0x4166c34cu, 0x42d561b4u, 0x444c0740u, 0x45cae0f2u, 0x47521cc6u, 0x48e1e9bau, 0x4a7a77d4u,
    0x4c1bf829u, 0x4dc69cddu, 0x4f7a9930u, 0x51382182u, 0x52ff6b55u, 0x54d0ad5au, 0x56ac1f75u, 0x5891fac1u,
    0x5a82799au, 0x5c7dd7a4u, 0x5e8451d0u, 0x60962665u, 0x62b39509u, 0x64dcdec3u, 0x6712460bu, 0x69540ec9u,
    0x6ba27e65u, 0x6dfddbccu, 0x70666f76u, 0x72dc8374u, 0x75606374u, 0x77f25cceu, 0x7a92be8bu, 0x7d41d96eu};

struct SampleArgs {
    const void *logits;
    int m, vocab, cluster, resident;            // resident: a CTA's part is kept in shared memory
    const float *temperature;
    const int *top_k;
    const float *top_p, *min_p, *uniform;
    int *ids;
    float *probs;
};

struct Shared {
    union {
        uint32_t hist[kBins];
        u64 radix[kRadix];
    };
    u64 warp_sum[kWarps];                       // of the draw's segments
    u64 best;                                   // key << 32 | ~index of the largest
    u64 sum_all, sum_above, sum_listed;
    u64 scan[kWarps];
    u64 buckets[kMaxCluster * kWarps];
    u64 rest;
    u64 parts[3][kWarps];
    uint32_t bound[2], listed, bin, lo, hi;
    float least;
    double drop;                                // T ln(min_p)
    int found;
    uint32_t exp2[32];
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

// *p of the cluster's CTA `rank`.
__device__ __forceinline__ u64 at_peer(const u64 *p, int rank, int cluster) {
    if (cluster == 1) return *p;
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(peer(p, rank)) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t at_peer(const uint32_t *p, int rank, int cluster) {
    if (cluster == 1) return *p;
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer(p, rank)) : "memory");
    return v;
}

__device__ __forceinline__ float at_peer(const float *p, int rank, int cluster) {
    return __uint_as_float(at_peer(reinterpret_cast<const uint32_t *>(p), rank, cluster));
}

// f(r) of every CTA r of the cluster, one lane each (a warp's lanes all call); `none` on the others.
template <typename T, typename F>
__device__ __forceinline__ T by_lanes(int cluster, T none, F f) {
    const int lane = threadIdx.x & 31;
    return lane < cluster ? f(lane) : none;
}

__device__ __forceinline__ void put_peer(int *p, int rank, int cluster, int v) {
    if (cluster == 1) *p = v;
    else asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(peer(p, rank)), "r"(v) : "memory");
}

// *p += v if `on`, without a branch.
__device__ __forceinline__ void add_if(bool on, uint32_t p, uint32_t v) {
    asm volatile("{ .reg .pred q; setp.ne.u32 q, %2, 0; @q red.shared.add.u32 [%0], %1; }" ::"r"(p), "r"(v),
                 "r"(static_cast<uint32_t>(on))
                 : "memory");
}

// A logit as it counts: NaN is -infinity (the larger of it and that), +infinity the largest finite number of the type.
template <bool BF16>
__device__ __forceinline__ float clean(float l) {
    return fminf(fmaxf(l, -INFINITY), BF16 ? 3.3895313892515355e38f : 3.4028234663852886e38f);
}

// Ascending in the (clean) logit; -0 as +0.
__device__ __forceinline__ uint32_t key_of(float l) {
    const uint32_t b = __float_as_uint(l + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
constexpr uint32_t kKeyNone = 0x007fffffu;      // of -infinity: no candidate

__device__ __forceinline__ float logit_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

__device__ __forceinline__ u64 entry_of(uint32_t key, int i) { return static_cast<u64>(key) << 32 | ~static_cast<uint32_t>(i); }
__device__ __forceinline__ int index_of(u64 entry) { return static_cast<int>(~static_cast<uint32_t>(entry)); }

// w / 2^k rounded (k > 0), or w * 2^-k, for w below 2^31 and k from -12 on: shifts by amounts that are negative or above 31
// give 0 in PTX, so both forms are computed and one of them is 0 (or, at k = 0, both are w).
__device__ __forceinline__ u64 shifted(uint32_t w, int k) {
    uint32_t half, down, up, high;
    asm("shl.b32 %0, %1, %2;" : "=r"(half) : "r"(1u), "r"(k - 1));
    asm("shr.u32 %0, %1, %2;" : "=r"(down) : "r"(w + half), "r"(k));
    asm("shl.b32 %0, %1, %2;" : "=r"(up) : "r"(w), "r"(-k));
    asm("shr.u32 %0, %1, %2;" : "=r"(high) : "r"(w), "r"(32 + k));
    return static_cast<u64>(high) << 32 | (down | up);
}

// One row's weights.  Logits are halved so that no difference overflows.  An infinite temperature has factor 0.
struct Weights {
    float half_max, ch, cl, least;

    __device__ __forceinline__ void set(float largest, float t) {
        half_max = 0.5f * largest;
        // 2 log2(e) / t as a pair: the quotient of the constant's upper part, and of what that leaves
        const float c = 2.8853900432586670f, rest = 3.8519242e-8f;
        ch = __fdiv_rn(c, t);
        cl = t <= 3.4028234663852886e38f ? __fdiv_rn(__fadd_rn(__fmaf_rn(-ch, t, c), rest), t) : 0.0f;
        least = -64.0f / ch;                    // below, the weight is 0
    }

    // (-infinity: 0; its NaNs end in the conversion to a whole number, which makes them 0.)
    __device__ __forceinline__ u64 of(float logit, const uint32_t *exp2) const {
        const float l = 0.5f * logit, b = -half_max;
        const float e = __fadd_rn(l, b);
        const float bp = __fsub_rn(e, l);
        const float dl = __fadd_rn(__fsub_rn(l, __fsub_rn(e, bp)), __fsub_rn(b, bp));
        const float d = fmaxf(e, least);
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
        const uint32_t w = m + static_cast<uint32_t>(__mulhi(static_cast<int>(m), __float2int_rn(q * 137438953472.0f)) >> 5);
        // w * 2^(floor(at / 32) + 12), rounded
        return shifted(w, -(at >> 5) - (kOneBits - 30));
    }
};

// The place in the order up to which a row's entries stay.
struct Cut {
    float logit;
    int index;
    __device__ __forceinline__ bool keeps(float l, int i) const { return l > logit || (l == logit && i <= index); }
};

__device__ __forceinline__ u64 warp_total(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ u64 warp_inclusive(u64 v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Sum over the threads before this one (scratch: kWarps entries; synchronises, and again before its next use).
__device__ __forceinline__ u64 block_exclusive(u64 v, u64 *scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const u64 in = warp_inclusive(v);
    __syncthreads();
    if (lane == 31) scratch[warp] = in;
    __syncthreads();
    u64 before = in - v;
    for (int w = 0; w < warp; ++w) before += scratch[w];
    return before;
}

// A range of a row's indices.
struct Segment {
    int from, to;
};

// How a row is dealt out.  Four neighbouring entries at an address that is a multiple of their size are a
// vector; places count entries from the first vector's beginning, so index = place - lead.  A CTA has `part` places,
// a warp `len` of them, whole rounds of 32 vectors.
struct Deal {
    int vocab, lead, part, len;

    __device__ __forceinline__ Deal(const void *row, int size, int vocab_, int cluster) : vocab(vocab_) {
        lead = static_cast<int>(reinterpret_cast<uintptr_t>(row) / size % 4);
        part = ((vocab + lead + cluster - 1) / cluster + 3) / 4 * 4;
        len = ((part + kWarps - 1) / kWarps + 127) / 128 * 128;
    }
    // The indices of CTA r's warp w.
    __device__ __forceinline__ Segment segment(int r, int w) const {
        const int from = r * part + w * len, to = min(from + len, (r + 1) * part);
        return {min(max(from - lead, 0), vocab), min(max(to - lead, 0), vocab)};
    }
};
constexpr size_t kMostShared = 200 * 1024;      // dynamic

// AGAIN: one CTA has the row and reads it again in every pass.
template <bool BF16, bool AGAIN>
struct Row {
    const void *logits;
    const float *held;                          // this CTA's part in shared memory, or nullptr
    u64 *local;                                 // its candidates: key << 32 | ~index
    Deal deal;
    Segment seg;                                // this warp's
    int rank, cluster;
    Shared &sm;

    __device__ __forceinline__ float read(int i) const {
        if constexpr (BF16) return clean<true>(bf16_bits_to_f32(static_cast<const uint16_t *>(logits)[i]));
        else return clean<false>(static_cast<const float *>(logits)[i]);
    }
    __device__ __forceinline__ int index(int offset) const { return rank * deal.part + offset - deal.lead; }
    __device__ __forceinline__ float at(int i) const { return held != nullptr ? held[i + deal.lead - rank * deal.part] : read(i); }
    // A vector's bits, as loaded: where all of it is in the part and the row.
    using Bits = std::conditional_t<BF16, uint2, float4>;
    __device__ __forceinline__ bool whole(int offset) const {
        const int i = index(offset);
        return offset < deal.part && i >= 0 && i + 4 <= deal.vocab;
    }
    __device__ __forceinline__ Bits bits(int offset) const {
        if constexpr (BF16) return *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(logits) + index(offset));
        else return *reinterpret_cast<const float4 *>(static_cast<const float *>(logits) + index(offset));
    }
    static __device__ __forceinline__ float4 values(const Bits &u) {
        float4 v;
        if constexpr (BF16)
            v = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                            __uint_as_float(u.y & 0xffff0000u));
        else v = u;
        return make_float4(clean<BF16>(v.x), clean<BF16>(v.y), clean<BF16>(v.z), clean<BF16>(v.w));
    }
    // The four entries from this CTA's place `offset` on, -infinity outside of the part or the row.
    __device__ __forceinline__ float4 fetch(int offset) const {
        const int i = index(offset);
        float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (offset >= deal.part) return v;
        if (whole(offset)) {
            v = values(bits(offset));
        } else {
            if (i >= 0 && i < deal.vocab) v.x = read(i);
            if (i + 1 >= 0 && i + 1 < deal.vocab) v.y = read(i + 1);
            if (i + 2 >= 0 && i + 2 < deal.vocab) v.z = read(i + 2);
            if (i + 3 >= 0 && i + 3 < deal.vocab) v.w = read(i + 3);
        }
        return v;
    }
    // visit(the four entries, index of the first) for all of this warp's.
    template <typename Visit>
    __device__ __forceinline__ void all(Visit visit) const {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const int end = (warp + 1) * deal.len;
        int o = warp * deal.len + 4 * lane;
        // One CTA loads a vector ahead of its use (256 rows of 131072, top-p 225 us to 204).  Parts of a row that are
        // read again come from L2, and gain nothing (64 rows 67, 73).
        Bits next{};
        if (AGAIN && whole(o)) next = bits(o);
        for (; o < end; o += 128) {
            float4 v;
            if constexpr (AGAIN) {
                v = whole(o) ? values(next) : fetch(o);
                if (o + 128 < end && whole(o + 128)) next = bits(o + 128);
            } else {
                v = held != nullptr ? *reinterpret_cast<const float4 *>(held + o) : fetch(o);
            }
            const float l[4] = {v.x, v.y, v.z, v.w};
            visit(l, index(o));
        }
    }

    // Sum over the cluster of each thread's v.  base: the sum of the CTAs before; warp sums stay in sm.warp_sum.
    __device__ u64 total(u64 v, u64 *base) const {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        v = warp_total(v);
        if (lane == 0) sm.warp_sum[warp] = v;
        __syncthreads();
        if (threadIdx.x == 0) {
            u64 s = 0;
            for (int w = 0; w < kWarps; ++w) s += sm.warp_sum[w];
            sm.sum_all = s;
        }
        sync_all(cluster);
        u64 all = 0, before = 0;
        for (int r = 0; r < cluster; ++r) {
            if (r == rank) before = all;
            all += at_peer(&sm.sum_all, r, cluster);
        }
        sync_all(cluster);
        *base = before;
        return all;
    }

    // The lowest index of a segment at which base and the sum of value(i) up to it exceed target; -1 if none does.  One warp.
    template <typename Value>
    __device__ int ordered(Segment s, u64 target, u64 base, Value value) const {
        const int lane = threadIdx.x & 31;
        for (int i = s.from; i < s.to; i += 32) {
            const u64 v = warp_inclusive(i + lane < s.to ? value(i + lane) : 0);
            const unsigned hit = __ballot_sync(0xffffffffu, base + v > target);
            if (hit) return i + __ffs(hit) - 1;
            base += __shfl_sync(0xffffffffu, v, 31);
        }
        return -1;
    }

    // Narrow the cut to the shortest run of the order whose sum of value(logit) reaches target (1 .. the sum
    // of all that stay), by the bytes of the key.
    template <typename Value>
    __device__ void narrow(Cut &cut, u64 target, Value value) const {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        uint32_t prefix = 0;
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int b = tid; b < kRadix; b += kThreads) sm.radix[b] = 0;
            __syncthreads();
            for (int i = seg.from + lane; i < seg.to; i += 32) {
                const float l = at(i);
                const uint32_t k = key_of(l);
                if (cut.keeps(l, i) && (shift == 24 || k >> (shift + 8) == prefix)) atomicAdd(&sm.radix[(k >> shift) & 255], value(l));
            }
            sync_all(cluster);
            u64 mine = 0;                                           // descending bins
            if (tid < kRadix)
                for (int r = 0; r < cluster; ++r) mine += at_peer(&sm.radix[kRadix - 1 - tid], r, cluster);
            const u64 before = block_exclusive(mine, sm.scan);
            if (tid < kRadix && before < target && before + mine >= target) {
                sm.bin = kRadix - 1 - tid;
                sm.rest = target - before;
            }
            sync_all(cluster);
            prefix = prefix << 8 | sm.bin;
            target = sm.rest;
            __syncthreads();
        }
        // equal keys have equal values: the first `need` of them in the order of the indices
        const float logit = logit_of(prefix);
        const u64 each = value(logit), need = (target + each - 1) / each;
        auto tie = [&](int i) -> u64 {
            const float l = at(i);
            return l == logit && cut.keeps(l, i);
        };
        u64 n = 0, base;
        for (int i = seg.from + lane; i < seg.to; i += 32) n += tie(i);
        total(n, &base);
        for (int w = 0; w < warp; ++w) base += sm.warp_sum[w];
        if (need - 1 >= base && need - 1 < base + sm.warp_sum[warp]) {
            const int found = ordered(seg, need - 1, base, tie);
            if (lane == 0)
                for (int r = 0; r < cluster; ++r) put_peer(&sm.found, r, cluster, found);
        }
        sync_all(cluster);
        cut.logit = logit;
        cut.index = sm.found;
        sync_all(cluster);
    }

    // List those of a lane's four entries whose bit is set (all lanes call).  The count goes on past the list's end.
    __device__ __forceinline__ void list(unsigned take, const float (&l)[4], int i) const {
        if (!__any_sync(0xffffffffu, take != 0)) return;
        const int lane = threadIdx.x & 31, mine = __popc(take);
        int before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += u;
        }
        uint32_t n = 0;
        if (lane == 31) n = atomicAdd(&sm.listed, before);
        n = __shfl_sync(0xffffffffu, n, 31) + before - mine;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (take >> j & 1) {
                if (n < local_most(cluster)) local[n] = entry_of(key_of(l[j]), i + j);
                ++n;
            }
    }

    // Entries listed in all CTAs; more than kList if they do not fit (all CTAs agree).
    __device__ int listed() const {
        const uint32_t c = by_lanes(cluster, 0u, [&](int r) { return at_peer(&sm.listed, r, cluster); });
        return static_cast<int>(__reduce_add_sync(0xffffffffu, c > local_most(cluster) ? kList + 1 : c));
    }

    // First CTA: all lists one behind the other.
    __device__ void collect(u64 *list, int n) const {
        const uint32_t c = by_lanes(cluster, 0u, [&](int r) { return at_peer(&sm.listed, r, cluster); });
        for (int i = threadIdx.x; i < (n + kThreads - 1) / kThreads * kThreads; i += kThreads) {
            int at = i, rank = 0;
#pragma unroll
            for (int r = 0; r < kMaxCluster - 1; ++r) {
                const int here = static_cast<int>(__shfl_sync(0xffffffffu, c, r));
                if (rank == r && at >= here) {
                    at -= here;
                    ++rank;
                }
            }
            if (i < n) list[i] = at_peer(&local[at], rank, cluster);
        }
    }
};

// Sort n entries descending (at most E per thread; a bitonic network, thread t having entries t, t + kThreads, ..):
// exchanges within a warp by shuffles, within a thread by registers, others through the list.
template <int E>
__device__ void sort_network(u64 *list, int n) {
    const int tid = threadIdx.x;
    u64 x[E];
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = e * kThreads + tid < n ? list[e * kThreads + tid] : 0;
    for (int k = 2; k <= E * kThreads; k <<= 1) {
        for (int j = k >> 1; j > 0; j >>= 1) {
            if (j >= kThreads) {
                const int step = j / kThreads;
#pragma unroll
                for (int e = 0; e < E; ++e)
#pragma unroll
                    for (int f = e + 1; f < E; ++f)
                        if ((e ^ f) == step) {
                            const bool down = ((e * kThreads + tid) & k) == 0;
                            const u64 hi = max(x[e], x[f]), lo = min(x[e], x[f]);
                            x[e] = down ? hi : lo;
                            x[f] = down ? lo : hi;
                        }
                continue;
            }
            if (j >= 32) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < E; ++e) list[e * kThreads + tid] = x[e];
                __syncthreads();
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int i = e * kThreads + tid;
                const u64 y = j >= 32 ? list[i ^ j] : __shfl_xor_sync(0xffffffffu, x[e], j);
                const bool first = (i & j) == 0, down = (i & k) == 0;
                x[e] = first == down ? max(x[e], y) : min(x[e], y);
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) list[e * kThreads + tid] = x[e];
    __syncthreads();
}

__device__ void sort(u64 *list, int n) {
    if (n <= kThreads) sort_network<1>(list, n);
    else if (n <= 2 * kThreads) sort_network<2>(list, n);
    else if (n <= 4 * kThreads) sort_network<4>(list, n);
    else sort_network<kList / kThreads>(list, n);
}

// floor(f * s) for a finite f in 0 .. 1.
__device__ __forceinline__ u64 scaled(float f, u64 s, bool up) {
    const uint32_t b = __float_as_uint(f);
    const int e = b >> 23;
    const u64 mant = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
    const int shift = 150 - (e ? e : 1);                                   // f = mant * 2^-shift, 23 <= shift <= 149
    const u64 lo = mant * s, hi = __umul64hi(mant, s);
    u64 v;
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

// The target of the draw: the first index whose sum exceeds it is drawn.
__device__ __forceinline__ u64 draw_target(float u, u64 sum) {
    u = u > 0.0f ? fminf(u, 1.0f) : 0.0f;
    return min(scaled(u, sum, false), sum - 1);
}

template <bool BF16, bool AGAIN>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) uint8_t dynamic[];
    __shared__ Shared sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = a.cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int row = blockIdx.x / a.cluster;
    if (tid < 32) sm.exp2[tid] = kExp2[tid];
    if (tid == 0) {
        sm.best = 0;
        sm.least = INFINITY;
        sm.listed = 0;
        sm.lo = kBins;
        sm.hi = kBins;
    }
    for (int b = tid; b < kBins; b += kThreads) sm.hist[b] = 0;
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();

    // (binary64 runs at 1/60 of the rate: one thread's, while the row is on its way)
    if (tid == kThreads - 1 && a.min_p != nullptr) {
        const float f = a.min_p[row];
        if (f > 0.0f) sm.drop = static_cast<double>(a.temperature != nullptr ? a.temperature[row] : 1.0f) * log(static_cast<double>(fminf(f, 1.0f)));
    }
    const void *logits = static_cast<const uint8_t *>(a.logits) + static_cast<int64_t>(row) * a.vocab * (BF16 ? 2 : 4);
    const Deal deal(logits, BF16 ? 2 : 4, a.vocab, a.cluster);
    u64 *local = reinterpret_cast<u64 *>(dynamic);
    Row<BF16, AGAIN> v{logits, nullptr, local, deal, deal.segment(rank, warp), rank, a.cluster, sm};
    const float t = a.temperature != nullptr ? a.temperature[row] : 1.0f;
    const int k = a.top_k != nullptr ? a.top_k[row] : 0;
    const float p = a.top_p != nullptr ? a.top_p[row] : 1.0f, floor = a.min_p != nullptr ? a.min_p[row] : 0.0f;
    const float u = a.uniform[row];

    // the row's part, its largest and smallest
    // shared memory: this CTA's candidates | its part of the row, or (in the first CTA, when that is done with) all candidates
    float *held = reinterpret_cast<float *>(local + local_most(a.cluster));
    float top = -INFINITY, least = INFINITY;
    int where = 0;
#pragma unroll 4
    for (int o = warp * deal.len + 4 * lane; o < (warp + 1) * deal.len; o += 128) {
        const float4 f = v.fetch(o);
        if (a.resident) *reinterpret_cast<float4 *>(held + o) = f;
        const float most = fmaxf(fmaxf(f.x, f.y), fmaxf(f.z, f.w)), fewest = fminf(fminf(f.x, f.y), fminf(f.z, f.w));
        if (most > top) {
            top = most;
            where = v.index(o) + (f.x == most ? 0 : f.y == most ? 1 : f.z == most ? 2 : 3);
        }
        if (fewest > -INFINITY) {
            least = fminf(least, fewest);
        } else {
            const float l[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) least = l[j] > -INFINITY ? fminf(least, l[j]) : least;
        }
    }
    if (a.resident) v.held = held;
    u64 best = top > -INFINITY ? entry_of(key_of(top), where) : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
        least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
    }
    if (lane == 0) {
        atomicMax(&sm.best, best);
        sm.scan[warp] = __float_as_uint(least);
    }
    __syncthreads();
    if (tid < kWarps) {
        least = __uint_as_float(static_cast<uint32_t>(sm.scan[tid]));
        for (int o = kWarps / 2; o > 0; o >>= 1) least = fminf(least, __shfl_xor_sync(kWarps < 32 ? (1u << kWarps % 32) - 1 : 0xffffffffu, least, o));
        if (tid == 0) sm.least = least;
    }
    const bool small_k = k > 0 && k <= kSmallK;
    if (small_k) {
        // Keys that at least k entries of the row reach: of the threads' maxima, k of this CTA's (warp 0), or
        // its share of k of each CTA's (warp 1).
        uint32_t *maxima = reinterpret_cast<uint32_t *>(local);
        maxima[tid] = top > -INFINITY ? key_of(top) : 0;
        __syncthreads();
        if (warp < 2) {
            const int want = warp == 0 ? k : (k + a.cluster - 1) / a.cluster;
            uint32_t m[kWarps], lo = 0, hi = static_cast<uint32_t>(sm.best >> 32);
#pragma unroll
            for (int j = 0; j < kWarps; ++j) m[j] = maxima[32 * j + lane];
            for (int i = 0; i < 20 && lo < hi; ++i) {
                const uint32_t mid = lo + (hi - lo + 1) / 2;
                int n = 0;
#pragma unroll
                for (int j = 0; j < kWarps; ++j) n += m[j] >= mid;
                if (__reduce_add_sync(0xffffffffu, n) >= want) lo = mid;
                else hi = mid - 1;
            }
            if (lane == 0) sm.bound[warp] = lo;
        }
    }
    sync_all(a.cluster);
    best = by_lanes(a.cluster, static_cast<u64>(0), [&](int r) { return at_peer(&sm.best, r, a.cluster); });
    least = by_lanes(a.cluster, INFINITY, [&](int r) { return at_peer(&sm.least, r, a.cluster); });
    uint32_t bound = small_k ? by_lanes(a.cluster, 0u, [&](int r) { return at_peer(&sm.bound[0], r, a.cluster); }) : 0;
    uint32_t shares = small_k ? by_lanes(a.cluster, 0xffffffffu, [&](int r) { return at_peer(&sm.bound[1], r, a.cluster); }) : 0;
#pragma unroll
    for (int o = kMaxCluster / 2; o > 0; o >>= 1) {
        best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
        least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
        bound = max(bound, __shfl_xor_sync(0xffffffffu, bound, o));
        shares = min(shares, __shfl_xor_sync(0xffffffffu, shares, o));
    }
    best = __shfl_sync(0xffffffffu, best, 0);
    least = __shfl_sync(0xffffffffu, least, 0);
    bound = __shfl_sync(0xffffffffu, max(bound, shares), 0);
    if (best == 0 || !(t >= kColdest)) {        // no candidate, or the first of the order
        if (rank == 0 && tid == 0) {
            a.ids[row] = best == 0 ? -1 : index_of(best);
            if (a.probs != nullptr) a.probs[row] = best == 0 ? 0.0f : 1.0f;
        }
        sync_all(a.cluster);
        return;
    }
    const float largest = logit_of(static_cast<uint32_t>(best >> 32));
    Weights w;
    w.set(largest, t);
    auto weight = [&](float l) { return w.of(l, sm.exp2); };
    Cut cut{-INFINITY, INT_MIN};
    float lowest = -INFINITY;                   // min-p: entries below go
    if (floor > 0.0f && t <= 3.4028234663852886e38f) {
        // w >= min_p  <=>  l >= l_max + T ln(min_p)
        lowest = fminf(__double2float_ru(static_cast<double>(largest) + sm.drop), largest);
    }
    u64 *list = reinterpret_cast<u64 *>(held);

    if (small_k) {
        const float from = fmaxf(bound > kKeyNone ? logit_of(bound) : -INFINITY, lowest);
        const float low = fmaxf(from, -3.4028234663852886e38f);
        v.all([&](const float(&l)[4], int i) {
            v.list((l[0] >= low) | (l[1] >= low) << 1 | (l[2] >= low) << 2 | (l[3] >= low) << 3, l, i);
        });
        sync_all(a.cluster);
        const int n = v.listed();
        if (n <= kList) {
            if (rank == 0) v.collect(list, n);
            sync_all(a.cluster);
            if (rank != 0) return;
            sort(list, n);
            const int stay = min(k, n);
            // weights, in place of the candidates behind the first k (at most kSmallK)
            u64 *ws = list + kSmallK;
            __syncthreads();
            const u64 mine = tid < stay ? weight(logit_of(static_cast<uint32_t>(list[tid] >> 32))) : 0;
            const u64 before = block_exclusive(mine, sm.scan);
            if (tid == stay - 1) sm.sum_all = before + mine;
            __syncthreads();
            u64 target = sm.sum_all;
            if (p < 1.0f) target = p > 0.0f ? max(scaled(p, target, true), static_cast<u64>(1)) : 1;
            const bool kept = tid < stay && before < target;
            ws[tid] = kept ? mine : 0;
            const int count = __syncthreads_count(kept);
            if (tid == count - 1) sm.sum_all = before + mine;
            __syncthreads();
            const u64 sum = sm.sum_all, drawn = draw_target(u, sum);
            if (kept) {
                // the sum over the indices up to this one, and without it
                const int me = index_of(list[tid]);
                u64 upto = 0;
                for (int j = 0; j < count; ++j) upto += index_of(list[j]) <= me ? ws[j] : 0;
                if (upto > drawn && upto - mine <= drawn) {
                    a.ids[row] = me;
                    if (a.probs != nullptr) a.probs[row] = static_cast<float>(static_cast<double>(mine) / static_cast<double>(sum));
                }
            }
            return;
        }
        sync_all(a.cluster);                    // all have read the counts
        if (tid == 0) sm.listed = 0;
        __syncthreads();
    }
    if (k > 0 && k < a.vocab) {
        u64 n = 0, base;
        v.all([&](const float(&l)[4], int) {
#pragma unroll
            for (int j = 0; j < 4; ++j) n += l[j] > -INFINITY;
        });
        n = v.total(n, &base);
        if (static_cast<u64>(k) < n) v.narrow(cut, k, [](float) { return static_cast<u64>(1); });
        for (int b = tid; b < kBins; b += kThreads) sm.hist[b] = 0;
        __syncthreads();
    }
    const bool tied = cut.index != INT_MIN;     // some of the entries at the cut go: below, only the cut itself tells
    if (lowest > cut.logit) cut = Cut{lowest, INT_MAX};
    // what stays, where `plain`, is what reaches this
    const bool plain = !tied || cut.index == INT_MAX;
    const float low = fmaxf(cut.logit, -3.4028234663852886e38f);

    u64 mine = 0, above = 0;                    // weights of all that stay, of those that surely do
    bool done = false;
    if (p < 1.0f && plain) {
        const float range = fminf(kNats * t, largest - least), scale = range > 0.0f ? (kBins - 1) / range : 0.0f;
        const float step = range / t / (kBins - 1);         // of ln(weight), per bin
        const float fine = scale * 1048576.0f;
        const uint32_t slope = static_cast<uint32_t>(step * 16384.0f), hist = smem_u32(sm.hist);
        v.all([&](const float(&l)[4], int) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t x = static_cast<uint32_t>(fminf((largest - l[j]) * fine, (kBins - 1) * 1048576.0f));
                // a share of 1 - (x - bin) step of its bin's upper end is the weight, to the second order
                add_if(l[j] >= low, hist + (x >> 18 & ~3u), 16384u - ((x >> 4 & 0xffffu) * slope >> 16));
            }
        });
        sync_all(a.cluster);
        float mass[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int b = 2 * tid + e;
            uint32_t c[kMaxCluster];
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) c[r] = r < a.cluster ? at_peer(&sm.hist[b], r, a.cluster) : 0;
            float n = 0.0f;
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) n += static_cast<float>(c[r]);
            mass[e] = n * __expf(-b * step);
        }
        // sums over the bins from the largest on, in fp32: estimates
        float in = mass[0] + mass[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float other = __shfl_up_sync(0xffffffffu, in, o);
            if (lane >= o) in += other;
        }
        if (lane == 31) sm.scan[warp] = __float_as_uint(in);
        __syncthreads();
        float all = 0.0f, before = in - mass[0] - mass[1];
        for (int o = 0; o < kWarps; ++o) {
            const float s = __uint_as_float(static_cast<uint32_t>(sm.scan[o]));
            all += s;
            if (o < warp) before += s;
        }
        const float aim = fmaxf(p, 0.0f) * all, aim_low = aim - kSlack * all, aim_high = aim + kSlack * all;
        float upto[3] = {before, before + mass[0], before + mass[0] + mass[1]};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            // the first bins to reach the one and the other (sums of neighbours may differ by a rounding: the lowest such bin)
            if (upto[e + 1] >= aim_low) atomicMin(&sm.lo, 2 * tid + e);
            if (upto[e + 1] >= aim_high) atomicMin(&sm.hi, 2 * tid + e);
        }
        __syncthreads();
        // the bins as logits (whatever the rounding: what they bracket is looked at below)
        const float above_this = largest - sm.lo / scale, from_this = fmaxf(largest - (sm.hi + 1) / scale, low);
        u64 bracket = 0;
        v.all([&](const float(&l)[4], int i) {
            unsigned take = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const u64 value = weight(l[j] >= low ? l[j] : -INFINITY);
                mine += value;
                const bool sure = l[j] > above_this;
                above += sure ? value : 0;
                if (l[j] >= from_this && !sure) {
                    bracket += value;
                    take |= 1u << j;
                }
            }
            v.list(take, l, i);
        });
        const u64 sums[3] = {warp_total(mine), warp_total(above), warp_total(bracket)};
        if (lane == 0) {
            sm.warp_sum[warp] = sums[1];
#pragma unroll
            for (int i = 0; i < 3; ++i) sm.parts[i][warp] = sums[i];
        }
        __syncthreads();
        if (warp < 3) {
            const u64 sum = warp_total(lane < kWarps ? sm.parts[warp][lane] : 0);
            if (lane == 0) (warp == 0 ? sm.sum_all : warp == 1 ? sm.sum_above : sm.sum_listed) = sum;
        }
        sync_all(a.cluster);
        const u64 total = warp_total(by_lanes(a.cluster, static_cast<u64>(0), [&](int r) { return at_peer(&sm.sum_all, r, a.cluster); }));
        const u64 sure = warp_total(by_lanes(a.cluster, static_cast<u64>(0), [&](int r) { return at_peer(&sm.sum_above, r, a.cluster); }));
        const u64 listed = warp_total(by_lanes(a.cluster, static_cast<u64>(0), [&](int r) { return at_peer(&sm.sum_listed, r, a.cluster); }));
        const u64 target = p > 0.0f ? max(scaled(p, total, true), static_cast<u64>(1)) : 1;
        const int n = v.listed();
        done = n <= kList && sure < target && target <= sure + listed;
        if (done) {
            if (rank == 0) {
                v.collect(list, n);
                if (tid < a.cluster * kWarps) sm.buckets[tid] = at_peer(&sm.warp_sum[tid % kWarps], tid / kWarps, a.cluster);
            }
            sync_all(a.cluster);
            if (rank != 0) return;
            sort(list, n);
            // the cut: the entry at which the sum reaches the target
            u64 run = sure;
            for (int i0 = 0; run < target && i0 < n; i0 += kThreads) {
                const int i = i0 + tid;
                const u64 own = i < n ? weight(logit_of(static_cast<uint32_t>(list[i] >> 32))) : 0;
                const u64 before = run + block_exclusive(own, sm.scan);
                if (i < n && before < target) {
                    const int index = index_of(list[i]), place = index + deal.lead, r = place / deal.part;
                    atomicAdd(&sm.buckets[r * kWarps + (place - r * deal.part) / deal.len], own);
                    if (before + own >= target) {
                        sm.found = index;
                        sm.bound[0] = static_cast<uint32_t>(list[i] >> 32);
                    }
                }
                if (tid == kThreads - 1) sm.sum_listed = before + own;
                __syncthreads();
                run = sm.sum_listed;
            }
            __syncthreads();
            cut = Cut{logit_of(sm.bound[0]), sm.found};
        } else {
            v.narrow(cut, target, weight);
        }
    } else if (p < 1.0f) {
        u64 base;
        v.all([&](const float(&l)[4], int i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) mine += cut.keeps(l[j], i + j) ? weight(l[j]) : 0;
        });
        const u64 total = v.total(mine, &base), target = p > 0.0f ? max(scaled(p, total, true), static_cast<u64>(1)) : 1;
        v.narrow(cut, target, weight);
    }
    if (!done) {
        mine = 0;
        v.all([&](const float(&l)[4], int i) {
            if (!__any_sync(0xffffffffu, fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])) >= cut.logit)) return;
#pragma unroll
            for (int j = 0; j < 4; ++j) mine += weight(cut.keeps(l[j], i + j) ? l[j] : -INFINITY);
        });
        mine = warp_total(mine);
        if (lane == 0) sm.warp_sum[warp] = mine;
        sync_all(a.cluster);
        if (rank == 0 && tid < a.cluster * kWarps) sm.buckets[tid] = at_peer(&sm.warp_sum[tid % kWarps], tid / kWarps, a.cluster);
        sync_all(a.cluster);
        if (rank != 0) return;
    }

    // first CTA: the segment that has the draw, then the index in it
    const int buckets = a.cluster * kWarps;
    const u64 in = tid < buckets ? sm.buckets[tid] : 0;
    const u64 before = block_exclusive(in, sm.scan);
    if (tid == buckets - 1) sm.sum_above = before + in;
    __syncthreads();
    const u64 sum = sm.sum_above, target = draw_target(u, sum);
    if (target >= before && target < before + in) {
        sm.bin = tid;
        sm.rest = target - before;
    }
    __syncthreads();
    const Segment s = deal.segment(sm.bin / kWarps, sm.bin % kWarps);
    const u64 rest = sm.rest;
    auto kept = [&](int i) -> u64 {
        const float l = v.read(i);
        return cut.keeps(l, i) ? weight(l) : 0;
    };
    const int len = ((s.to - s.from + kWarps - 1) / kWarps + 31) / 32 * 32;
    const Segment sub{min(s.from + warp * len, s.to), min(s.from + (warp + 1) * len, s.to)};
    u64 own = 0;
    for (int i = sub.from + lane; i < sub.to; i += 32) own += kept(i);
    own = warp_total(own);
    __syncthreads();
    if (lane == 0) sm.scan[warp] = own;
    __syncthreads();
    u64 base = 0;
    for (int o = 0; o < warp; ++o) base += sm.scan[o];
    if (rest < base || rest >= base + own) return;
    const int at = v.ordered(sub, rest, base, kept);
    if (lane == 0) {
        a.ids[row] = at;
        if (a.probs != nullptr) a.probs[row] = static_cast<float>(static_cast<double>(kept(at)) / static_cast<double>(sum));
    }
}

template <bool BF16, bool AGAIN>
cudaError_t sample_launch(const SampleArgs &a, size_t smem, cudaStream_t stream) {
    static SmemLimit limit;
    cudaError_t e = limit.raise(sample_kernel<BF16, AGAIN>, kMostShared);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.m) * a.cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel<BF16, AGAIN>, a);
}

template <bool BF16>
cudaError_t sample_launch(SampleArgs a, int sms, cudaStream_t stream) {
    // CTAs per row: as many as run at once, two to an SM (one, where parts get below 4096 entries), and
    // up to eight.  1, 2, 4 and 8 of them, top-p (us): 131072 entries, 16 rows 137 91 56 51, 64 rows 146 113 83 91, 128 rows
    // 199 149 154 169, 256 rows 256 232 244 295; 32003 entries, 16 rows 34 26 21 23, 64 rows 35 35 28 46, 256 rows 59 70 88 153;
    // 4000 entries, 1 row 13 14 15 16, 256 rows 20 37 63 135.
    a.cluster = 1;
    while (a.cluster < kMaxCluster && a.vocab > a.cluster * 4096 &&
           static_cast<int64_t>(a.m) * 2 * a.cluster <= (a.vocab > 2 * a.cluster * 4096 ? 2 * sms : sms))
        a.cluster *= 2;
    const int part = ((a.vocab + 3 + a.cluster - 1) / a.cluster + 3) / 4 * 4;        // (at most: as Deal)
    const size_t held = static_cast<size_t>(kWarps) * (((part + kWarps - 1) / kWarps + 127) / 128 * 128) * 4;
    const size_t local = local_most(a.cluster) * sizeof(u64);
    // A part is kept in shared memory where that does not cost the SM its second CTA: else it is read again, from
    // L2 (131072 entries, top-k, four CTAs per row: 16 rows 20 kept, 24 not; 64 rows 38 kept, 29 not).
    const int per_sm = static_cast<int64_t>(a.m) * a.cluster > sms ? 2 : 1;
    a.resident = (held + local) * per_sm <= kMostShared;
    const size_t smem = local + max(a.resident ? held : 0, kList * sizeof(u64));
    return a.cluster == 1 && !a.resident ? sample_launch<BF16, true>(a, smem, stream) : sample_launch<BF16, false>(a, smem, stream);
}

cudaError_t sample_launch(const SampleArgs &a, bool bf16, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    return bf16 ? sample_launch<true>(a, sms, stream) : sample_launch<false>(a, sms, stream);
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
