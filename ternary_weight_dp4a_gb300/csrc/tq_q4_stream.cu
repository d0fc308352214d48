// tq_q4_stream.cu -- products with 4-bit weights for few rows: the weights are read once, as a
// stream, and everything else is kept off their way.
//
//   y[r][i] = sum over the groups g of  s_ig * sum_{j in g} (c_ij - 8) x_rj  [+ (8 s_ig - b_ig) * sum_{j in g} x_rj]
//
// A warp takes chunks of 16 weight rows x 128 values (1 KB of codes, two 16-byte loads per lane).
// A word's nibbles become bf16 in place: (w >> 4 i) & 0x000f000f | 0x4300'4300 is the pair 128 + c,
// and minus 136 it is c - 8, exactly.  They are the A operand (16 x 16) of
// mma.m16n8k16, up to 8 rows of x the B operand; products are exact in fp32, a group's sum is the
// accumulator, and the fold by scales is done in fp32 on the accumulators, where the lane has the same
// two weight rows.  x lies in shared memory in the order of the B operand, one 16-byte load per
// two instructions.
//
// The chunks of a CTA's strips form one contiguous run, of which each warp has an even
// share, whatever strips it begins and ends in; a warp that leaves a strip stores its sums, and
// the CTA adds the parts of a strip in ascending order of k.  Where x does not fit into one
// CTA's shared memory, a cluster's CTAs have a range of k each and the parts are read across the
// cluster.  Neither depends on the number of rows up to 8, so a row's bits do not either.
#include <cuda_runtime.h>

#include <cstdint>

#include "tq_device.cuh"
#include "tq_launch.h"
#include "tq_moe_internal.h"
#include "tq_q4_internal.h"

namespace tq {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kBatch = 32;                      // strips between two reductions
constexpr int kSlots = kBatch + kWarps;         // parts of strips in a batch: strip + warp is unique
constexpr int kDepth = 4;                       // chunks in flight per warp

// Chunks of k per CTA: what x, its group sums and the parts leave room for in 227 KB.
template <int NT>
constexpr int max_chunks() {
    return (227 * 1024 - kSlots * NT * 512) / (NT * (2048 + 128));
}

struct StreamArgs {
    Q4Product p;
    int row0;               // first row of this pass
    int rows;               // rows of this pass
    int cluster;
};

// Chunks of codes are read once and not kept in L1.
__device__ __forceinline__ uint4 load_codes(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// PER scales of row r and PER of row r + 8.
template <int PER>
struct Scales {
    uint32_t v[PER];
};

template <int PER>
__device__ __forceinline__ Scales<PER> load_scales(const uint16_t *p) {
    Scales<PER> s;
    if constexpr (PER == 1) {
        asm volatile("ld.global.u32 %0, [%1];" : "=r"(s.v[0]) : "l"(p));
    } else if constexpr (PER == 2) {
        asm volatile("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(s.v[0]), "=r"(s.v[1]) : "l"(p));
    } else {
        asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(s.v[0]), "=r"(s.v[1]), "=r"(s.v[2]), "=r"(s.v[3])
                     : "l"(p));
    }
    return s;
}

template <int PER>
__device__ __forceinline__ float scale_at(const Scales<PER> &s, int half, int p) {
    const int e = half * PER + p;
    return f16_bits_to_f32(static_cast<uint16_t>(e & 1 ? s.v[e >> 1] >> 16 : s.v[e >> 1] & 0xffffu));
}

// Pair i of a word's codes as bf16 c - 8.
__device__ __forceinline__ uint32_t decode_pair(uint32_t w, int i) {
    const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(0x43084308u));
    return d;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, uint32_t rank) {
    float v;
    asm volatile("{ .reg .u32 a; mapa.shared::cluster.u32 a, %1, %2; ld.shared::cluster.f32 %0, [a]; }"
                 : "=f"(v)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}

// The warp that has item i of `total` dealt evenly to kWarps warps.
__device__ __forceinline__ int share_begin(int w, int total) { return static_cast<int>(static_cast<int64_t>(w) * total / kWarps); }
__device__ __forceinline__ int share_of(int i, int total) { return (kWarps * (i + 1) - 1) / total; }

// NT: groups of 8 rows.  PER: scale groups per chunk.  MATS: 1, or gate and up, whose strips alternate.
template <int NT, int PER, bool MINS, int MATS>
__global__ void __launch_bounds__(kThreads, 1) q4_stream_kernel(const StreamArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    const Q4Product &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int chunks = p.k >> 7;
    const int rank = a.cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int first = rank * chunks / a.cluster, mine = (rank + 1) * chunks / a.cluster - first;
    float4 *slots = reinterpret_cast<float4 *>(smem);                       // [kSlots][NT][32]
    uint4 *xs = reinterpret_cast<uint4 *>(slots + kSlots * NT * 32);        // [chunk][4][rows][4]
    float *sums = reinterpret_cast<float *>(xs + mine * 16 * a.rows);       // [chunk][PER][rows]

    const int clusters = gridDim.x / a.cluster, me = blockIdx.x / a.cluster;
    const int64_t strips = q4_strips(p.n);
    const int64_t from = MATS * (me * strips / clusters), to = MATS * ((me + 1) * strips / clusters);

    pdl_launch_dependents();
    pdl_wait();

    // x, in the order in which lanes read it: 16 bytes are 8 values, chunk = piece / 16,
    // group of 32 = piece / 4 % 4, lane of the quad = piece % 4
    for (int i = tid; i < mine * 16 * a.rows; i += kThreads) {
        const int row = i / (mine * 16), piece = i - row * (mine * 16);
        const uint4 v = *reinterpret_cast<const uint4 *>(p.x + (static_cast<int64_t>(a.row0 + row) * p.k + (first * 16 + piece) * 8));
        xs[((piece >> 2) * a.rows + row) * 4 + (piece & 3)] = v;
    }
    if constexpr (MINS) {
        __syncthreads();
        constexpr int kPieces = 16 / PER;               // of a group
        for (int i = tid; i < mine * PER * a.rows; i += kThreads) {
            const int row = i % a.rows, g = i / a.rows;
            float s = 0.0f;
            for (int j = 0; j < kPieces; ++j) {
                const int piece = g * kPieces + j;
                const uint4 v = xs[((piece >> 2) * a.rows + row) * 4 + (piece & 3)];
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) s += __uint_as_float(u[e] << 16) + __uint_as_float(u[e] & 0xffff0000u);
            }
            sums[i] = s;
        }
    }
    __syncthreads();

    int col[NT];                                        // row of x of this lane's B operand; any one behind the last
#pragma unroll
    for (int t = 0; t < NT; ++t) col[t] = min(8 * t + (lane >> 2), a.rows - 1);

    for (int64_t batch = from; batch < to; batch += kBatch) {
        const int count = static_cast<int>(min(static_cast<int64_t>(kBatch), to - batch));
        const int total = count * mine;
        const int begin = share_begin(warp, total), end = share_begin(warp + 1, total);

        uint4 lo[kDepth], hi[kDepth];
        Scales<PER> sc[kDepth], mn[MINS ? kDepth : 1];
        int lunit = begin / mine, lchunk = begin - lunit * mine;            // what is loaded next
        auto load = [&](int j) {
            const int64_t unit = batch + lunit;
            const int mat = MATS == 2 ? static_cast<int>(unit & 1) : 0;
            const int64_t block = (MATS == 2 ? unit >> 1 : unit) * chunks + first + lchunk;
            const uint8_t *c = p.codes[mat] + block * kQ4ChunkBytes + lane * 16;
            lo[j] = load_codes(c);
            hi[j] = load_codes(c + 512);
            const int64_t at = (block * 8 + (lane >> 2)) * (2 * PER);
            sc[j] = load_scales<PER>(p.scales[mat] + at);
            if constexpr (MINS) mn[j] = load_scales<PER>(p.mins[mat] + at);
            if (++lchunk == mine) {
                lchunk = 0;
                ++lunit;
            }
        };
#pragma unroll
        for (int j = 0; j < kDepth; ++j)
            if (begin + j < end) load(j);

        float acc[NT][4] = {};
        int unit = begin / mine, chunk = begin - unit * mine;
        for (int i = begin; i < end; i += kDepth) {
#pragma unroll
            for (int j = 0; j < kDepth; ++j) {
                if (i + j >= end) break;
                const uint32_t wl[4] = {lo[j].x, lo[j].y, lo[j].z, lo[j].w}, wh[4] = {hi[j].x, hi[j].y, hi[j].z, hi[j].w};
                float c[NT][4];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (g % (4 / PER) == 0)
#pragma unroll
                        for (int t = 0; t < NT; ++t) c[t][0] = c[t][1] = c[t][2] = c[t][3] = 0.0f;
                    uint32_t al[4], ah[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        al[e] = decode_pair(wl[g], e);
                        ah[e] = decode_pair(wh[g], e);
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const uint4 b = xs[((chunk * 4 + g) * a.rows + col[t]) * 4 + (lane & 3)];
                        mma_bf16(c[t], al[0], ah[0], al[1], ah[1], b.x, b.y);
                        mma_bf16(c[t], al[2], ah[2], al[3], ah[3], b.z, b.w);
                    }
                    if (g % (4 / PER) == 4 / PER - 1) {
                        const int q = g / (4 / PER);
                        const float s0 = scale_at<PER>(sc[j], 0, q), s1 = scale_at<PER>(sc[j], 1, q);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            acc[t][0] = __fmaf_rn(s0, c[t][0], acc[t][0]);
                            acc[t][1] = __fmaf_rn(s0, c[t][1], acc[t][1]);
                            acc[t][2] = __fmaf_rn(s1, c[t][2], acc[t][2]);
                            acc[t][3] = __fmaf_rn(s1, c[t][3], acc[t][3]);
                        }
                        if constexpr (MINS) {
                            const float b0 = __fmaf_rn(8.0f, s0, -scale_at<PER>(mn[j], 0, q));
                            const float b1 = __fmaf_rn(8.0f, s1, -scale_at<PER>(mn[j], 1, q));
                            const float *row = sums + (chunk * PER + q) * a.rows;
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                const int r0 = min(8 * t + 2 * (lane & 3), a.rows - 1), r1 = min(8 * t + 2 * (lane & 3) + 1, a.rows - 1);
                                const float x0 = row[r0], x1 = row[r1];
                                acc[t][0] = __fmaf_rn(b0, x0, acc[t][0]);
                                acc[t][1] = __fmaf_rn(b0, x1, acc[t][1]);
                                acc[t][2] = __fmaf_rn(b1, x0, acc[t][2]);
                                acc[t][3] = __fmaf_rn(b1, x1, acc[t][3]);
                            }
                        }
                    }
                }
                if (i + j + kDepth < end) load(j);
                if (++chunk == mine || i + j + 1 == end) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        slots[((unit + warp) * NT + t) * 32 + lane] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
                        acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.0f;
                    }
                    if (chunk == mine) {
                        chunk = 0;
                        ++unit;
                    }
                }
            }
        }
        if (a.cluster > 1) cluster_sync();
        else __syncthreads();

        // add up the parts, k ascending; a cluster's CTAs deal the strips to one another
        const uint32_t base = smem_u32(slots);
        auto value = [&](int u, int e, int row) {       // strip u of the batch, weight row e
            const uint32_t in = ((row >> 3) * 32 + (e & 7) * 4 + ((row & 7) >> 1)) * 16 + ((e >> 3) * 2 + (row & 1)) * 4;
            float v = 0.0f;
            for (int r = 0; r < a.cluster; ++r) {
                const int its = (r + 1) * chunks / a.cluster - r * chunks / a.cluster, all = count * its;
                const int w1 = share_of(u * its + its - 1, all);
                for (int w = share_of(u * its, all); w <= w1; ++w) {
                    if (share_begin(w, all) == share_begin(w + 1, all)) continue;
                    const uint32_t at = base + (u + w) * (NT * 512) + in;
                    v += a.cluster > 1 ? ld_cluster_f32(at, r) : *reinterpret_cast<const float *>(smem + (at - base));
                }
            }
            return v;
        };
        const int groups = count / MATS;                // strips, or pairs of them
        const int own = (groups - rank + a.cluster - 1) / a.cluster;
        for (int i = tid; i < own * 16 * a.rows; i += kThreads) {
            const int e = i & 15, row = (i >> 4) % a.rows, u = ((i >> 4) / a.rows) * a.cluster + rank;
            const int64_t out = (batch / MATS + u) * kQ4Strip + e;
            if (out >= p.n) continue;
            const int64_t at = static_cast<int64_t>(a.row0 + row) * p.n + out;
            float v = value(u * MATS, e, row);
            if constexpr (MATS == 2) v = __fmul_rn(tq_silu(v), value(u * 2 + 1, e, row));
            if (MATS == 2 || p.y_bf16) static_cast<uint16_t *>(p.y)[at] = f32_to_bf16_bits(v);
            else static_cast<float *>(p.y)[at] = v;
        }
        if (a.cluster > 1) cluster_sync();
        else __syncthreads();
    }
}

template <int NT, int PER, bool MINS, int MATS>
cudaError_t launch(const StreamArgs &a, int sms, cudaStream_t stream) {
    static SmemLimit limit;
    cudaError_t e = limit.raise(q4_stream_kernel<NT, PER, MINS, MATS>, 227 * 1024);
    if (e != cudaSuccess) return e;
    const int chunks = a.p.k / 128, mine = (chunks + a.cluster - 1) / a.cluster;
    const size_t smem = kSlots * NT * 512 + static_cast<size_t>(mine) * a.rows * (256 + (MINS ? PER * 4 : 0));
    const int64_t strips = q4_strips(a.p.n);
    const int most = sms / a.cluster;
    const int clusters = static_cast<int>(strips < most ? strips : most);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(clusters * a.cluster);
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
    return cudaLaunchKernelEx(&cfg, q4_stream_kernel<NT, PER, MINS, MATS>, a);
}

template <int NT, int PER>
cudaError_t pick(const StreamArgs &a, int sms, cudaStream_t stream) {
    const bool mins = a.p.mins[0] != nullptr;
    if (a.p.mats == 1) return mins ? launch<NT, PER, true, 1>(a, sms, stream) : launch<NT, PER, false, 1>(a, sms, stream);
    return mins ? launch<NT, PER, true, 2>(a, sms, stream) : launch<NT, PER, false, 2>(a, sms, stream);
}

template <int NT>
cudaError_t pass(StreamArgs &a, int sms, cudaStream_t stream) {
    a.cluster = (a.p.k / 128 + max_chunks<NT>() - 1) / max_chunks<NT>();
    return a.p.group == 128 ? pick<NT, 1>(a, sms, stream) : a.p.group == 64 ? pick<NT, 2>(a, sms, stream) : pick<NT, 4>(a, sms, stream);
}

}  // namespace

cudaError_t q4_stream_launch(const Q4Product &p, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    StreamArgs a{};
    a.p = p;
    for (a.row0 = 0; a.row0 < p.m; a.row0 += 16) {
        a.rows = p.m - a.row0 < 16 ? p.m - a.row0 : 16;
        e = a.rows > 8 ? pass<2>(a, sms, stream) : pass<1>(a, sms, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace tq
