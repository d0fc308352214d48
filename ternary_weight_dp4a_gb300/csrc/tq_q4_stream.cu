// tq_q4_stream.cu -- products with 4-bit weights for few rows: the weights are read once, as a
// stream, and everything else is kept off their way.
//
//   y[r][i] = sum over the groups g of  s_ig * sum_{j in g} (c_ij - 8) x_rj  [+ (8 s_ig - b_ig) * sum_{j in g} x_rj]
//
// A warp takes chunks of two strips of 16 weight rows x 128 values (2 KB of codes, four 16-byte loads per lane;
// gate/up: a strip of each).  A word's nibbles become bf16 in place: (w >> 4 i) & 0x000f000f | 0x43004300 is
// the pair 128 + c, and minus 136 it is c - 8, exactly.  They are the A operand (16 x 16) of
// mma.m16n8k16, 8 rows of x the B operand; products are exact in fp32, a group's sum is the
// accumulator, and the fold by scales is done in fp32 on the accumulators, where the lane has the same
// two weight rows.  x lies in shared memory in the order of the B operand, one 16-byte load per
// four instructions.
//
// The chunks of a CTA's units (pairs of strips, or single strips where there are few) form one run, of
// which each warp has an even share, whatever units it begins and ends in.  A unit that one warp has alone it
// stores by itself; of the others (two per warp at most) it leaves its sums in shared memory, and they are added up
// in ascending order of k at the end.  Where x does not fit into one CTA's shared memory, a cluster's CTAs have a
// range of k each, and the parts are read across the cluster, a batch of units at a time.  Neither depends on
// the number of rows up to 8, so a row's bits do not either.
//
// What bounds it.  One row, large matrices, group 128: memory (131072 x 5120 64 us, 5.4 TB/s; gate and up 17408 x 5120
// 22 us, of which 4 before the first weights).  Small groups and more rows: instructions (a word is 20 for
// 8 weights, a group's fold 8 more per 8 rows of x, minima as many again; 13 rows, gate and up 17408 x 5120, group
// 32 with minima 45 us, 2.5 TB/s).  Small matrices: latency (5120 x 5120 6.3 us).  Split k: the same, and the registers
// that its indices take (20 of the 30 instances spill; 8 x 5120 x 17408, group 32 with minima, 60 bytes of stores and
// 68 of loads, 22 us; up to 504 and 292 for gate/up in groups of 64 with minima.  13 rows, gate and up 28672 x 8192: group 128
// 84 us, 2.8 TB/s, group 32 with minima 109).
#include <cuda_runtime.h>

#include <cstdint>

#include "tq_device.cuh"
#include "tq_launch.h"
#include "tq_q4_internal.h"

namespace tq {
namespace {

// NT: groups of 8 rows of x in a pass.  RS: strips of a unit.  SPLIT: k is split over a cluster.
template <int NT, int RS, bool SPLIT>
struct Shape {
    static constexpr int kWarps = NT == 1 ? 16 : 12;
    static constexpr int kThreads = 32 * kWarps;
    // Chunks in flight per warp.  (Of two strips, two of them, for 16 warps; 12 warps have registers for three.  12
    // warps for up to 8 rows, or bulk prefetches into L2 ahead of the loads, are not faster.)
    static constexpr int kDepth = (NT == 1 ? 4 : 6) / RS;
    static constexpr int kBatch = NT == 1 ? 32 : 8;             // units between two reductions over a cluster
    static constexpr int kSlots = SPLIT ? kBatch + kWarps : 2 * kWarps;     // parts of units
    static constexpr int kSlotBytes = RS * NT * 512;
    static constexpr int kChunkBytes = NT * 2048;               // of x
    // Chunks of k per CTA: what x, its group sums and the parts leave room for in 227 KB.
    static constexpr int kMaxChunks = (227 * 1024 - kSlots * kSlotBytes) / (kChunkBytes + NT * 8 * 4 * 4);
};

struct StreamArgs {
    Q4Product p;
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
__device__ __forceinline__ uint32_t decode_pair(uint32_t w, int i, uint32_t mask, uint32_t base) {
    uint32_t v, d;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(v) : "r"(w >> (4 * i)), "r"(mask), "r"(base));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(0x43084308u));
    return d;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first of a sum: from zero.
__device__ __forceinline__ void mma_bf16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ float4 ld_cluster(uint32_t addr, uint32_t rank) {
    float4 v;
    asm volatile("{ .reg .u32 a; mapa.shared::cluster.u32 a, %4, %5; ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [a]; }"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}

// Items dealt evenly to W warps: where warp w's share begins, and the warp that has item i.
template <int W>
__device__ __forceinline__ int share_begin(int w, int total) { return static_cast<int>(static_cast<int64_t>(w) * total / W); }
template <int W>
__device__ __forceinline__ int share_of(int i, int total) { return (W * (i + 1) - 1) / total; }

// PER: scale groups per chunk.
template <int NT, int RS, int PER, bool MINS, bool GATEUP, bool SPLIT>
__global__ void __launch_bounds__(Shape<NT, RS, SPLIT>::kThreads, 1) q4_stream_kernel(const StreamArgs a) {
    using S = Shape<NT, RS, SPLIT>;
    static_assert(RS == 2 || !GATEUP);
    extern __shared__ __align__(16) uint8_t smem[];
    const Q4Product &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int chunks = p.k >> 7;
    const int cluster = SPLIT ? a.cluster : 1, rank = SPLIT ? static_cast<int>(cluster_rank()) : 0;
    const int first = rank * chunks / cluster, mine = (rank + 1) * chunks / cluster - first;
    float4 *slots = reinterpret_cast<float4 *>(smem);                       // [kSlots][RS][NT][32]
    uint4 *xs = reinterpret_cast<uint4 *>(smem + S::kSlots * S::kSlotBytes);        // [chunk][4][8 NT rows][4]
    float *sums = reinterpret_cast<float *>(smem + S::kSlots * S::kSlotBytes + mine * S::kChunkBytes);  // [chunk][PER][8 NT]

    const int clusters = gridDim.x / cluster, me = blockIdx.x / cluster;
    const int64_t strips = q4_strips(p.n), units = GATEUP ? strips : (strips + RS - 1) / RS;
    const int64_t from = me * units / clusters, to = (me + 1) * units / clusters;

    pdl_launch_dependents();
    pdl_wait();

    uint4 code[S::kDepth][RS][2];                       // [strip][rows r, r + 8]
    Scales<PER> sc[S::kDepth][RS], mn[MINS ? S::kDepth : 1][RS];
    const uint8_t *cp[RS];
    const uint16_t *sp[RS], *mp[RS];
    int64_t batch = from;
    int count, begin, end, lunit, lchunk;               // units of the batch, this warp's share; what is loaded next
    auto point = [&] {
#pragma unroll
        for (int h = 0; h < RS; ++h) {
            // (an odd last strip stands in for its pair, whose results go nowhere)
            const int64_t strip = GATEUP ? batch + lunit : min(RS * (batch + lunit) + h, strips - 1);
            const int64_t block = strip * chunks + first + lchunk;
            const int mat = GATEUP ? h : 0;
            cp[h] = p.codes[mat] + block * kQ4ChunkBytes + lane * 16;
            sp[h] = p.scales[mat] + (block * 8 + (lane >> 2)) * (2 * PER);
            if constexpr (MINS) mp[h] = p.mins[mat] + (block * 8 + (lane >> 2)) * (2 * PER);
        }
    };
    auto load = [&](int j) {
#pragma unroll
        for (int h = 0; h < RS; ++h) {
            code[j][h][0] = load_codes(cp[h]);
            code[j][h][1] = load_codes(cp[h] + 512);
            sc[j][h] = load_scales<PER>(sp[h]);
            if constexpr (MINS) mn[j][h] = load_scales<PER>(mp[h]);
            cp[h] += kQ4ChunkBytes;
            sp[h] += 16 * PER;
            if constexpr (MINS) mp[h] += 16 * PER;
        }
        if (++lchunk == mine) {
            lchunk = 0;
            ++lunit;
            point();
        }
    };
    // This warp's share of the batch (without a cluster, of all units), and its first loads: they are on
    // their way while x is laid out.
    auto open = [&] {
        count = static_cast<int>(SPLIT ? min(static_cast<int64_t>(S::kBatch), to - batch) : to - batch);
        begin = share_begin<S::kWarps>(warp, count * mine);
        end = share_begin<S::kWarps>(warp + 1, count * mine);
        lunit = begin / mine;
        lchunk = begin - lunit * mine;
        point();
#pragma unroll
        for (int j = 0; j < S::kDepth; ++j)
            if (begin + j < end) load(j);
    };
    open();

    // x, in the order in which lanes read it: 16 bytes are 8 values, chunk = piece / 16,
    // group of 32 = piece / 4 % 4, lane of the quad = piece % 4
    for (int i = tid; i < mine * 16 * p.m; i += S::kThreads) {
        const int row = i / (mine * 16), piece = i - row * (mine * 16);
        const uint4 v = *reinterpret_cast<const uint4 *>(p.x + (static_cast<int64_t>(row) * p.k + (first * 16 + piece) * 8));
        xs[((piece >> 2) * (8 * NT) + row) * 4 + (piece & 3)] = v;
    }
    if constexpr (MINS) {
        __syncthreads();
        constexpr int kPieces = 16 / PER;               // of a group
        for (int i = tid; i < mine * PER * p.m; i += S::kThreads) {
            const int row = i % p.m, g = i / p.m;
            float s = 0.0f;
            for (int j = 0; j < kPieces; ++j) {
                const int piece = g * kPieces + j;
                const uint4 v = xs[((piece >> 2) * (8 * NT) + row) * 4 + (piece & 3)];
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) s += __uint_as_float(u[e] << 16) + __uint_as_float(u[e] & 0xffff0000u);
            }
            sums[g * (8 * NT) + row] = s;
        }
    }
    __syncthreads();

    // rows of x of this lane's B operand: any one behind the last
    const uint4 *xl[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) xl[t] = xs + min(8 * t + (lane >> 2), p.m - 1) * 4 + (lane & 3);
    const uint64_t *xsum = reinterpret_cast<const uint64_t *>(sums) + (lane & 3);       // of its accumulators' two
    uint32_t mask = 0x000f000fu, base = 0x43004300u;
    asm volatile("" : "+r"(mask), "+r"(base));          // in registers: two constants do not fit one instruction

    // A float4 of a unit (strip h, rows of x 8 t and on, lane) is two weight rows, r and r + 8, by two rows of x.
    auto store = [&](int64_t u, int f, float4 v, float4 up) {
        const int t = f / 32 % NT, h = f / 32 / NT, e = f % 32 >> 2, row = 8 * t + 2 * (f & 3);
        const int64_t out = (u * (GATEUP ? 1 : RS) + h) * kQ4Strip + e;
        const float g[4] = {v.x, v.y, v.z, v.w}, w[4] = {up.x, up.y, up.z, up.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (row + (i & 1) >= p.m || out + 8 * (i >> 1) >= p.n) continue;
            const int64_t at = static_cast<int64_t>(row + (i & 1)) * p.n + out + 8 * (i >> 1);
            const float y = GATEUP ? __fmul_rn(tq_silu(g[i]), w[i]) : g[i];
            if (GATEUP || p.y_bf16) static_cast<uint16_t *>(p.y)[at] = f32_to_bf16_bits(y);
            else static_cast<float *>(p.y)[at] = y;
        }
    };
    constexpr int kAll = RS * NT * 32, kEach = GATEUP ? NT * 32 : kAll;     // float4 of a unit, and with outputs
    auto plus = [](float4 v, float4 q) { return make_float4(v.x + q.x, v.y + q.y, v.z + q.z, v.w + q.w); };

    while (batch < to) {
        uint64_t acc[RS][NT][2] = {};                   // weight rows r and r + 8, two rows of x each
        int unit = begin / mine, chunk = begin - unit * mine;
        for (int i = begin; i < end; i += S::kDepth) {
#pragma unroll
            for (int j = 0; j < S::kDepth; ++j) {
                if (i + j >= end) break;
                const int xo = chunk * (S::kChunkBytes / 16);
                float c[RS][NT][4];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const bool fresh = g % (4 / PER) == 0;
                    uint4 b[NT];
#pragma unroll
                    for (int t = 0; t < NT; ++t) b[t] = xl[t][xo + g * (8 * NT * 4)];
#pragma unroll
                    for (int h = 0; h < RS; ++h) {
                        const uint4 lo = code[j][h][0], hi = code[j][h][1];
                        const uint32_t wl = g == 0 ? lo.x : g == 1 ? lo.y : g == 2 ? lo.z : lo.w;
                        const uint32_t wh = g == 0 ? hi.x : g == 1 ? hi.y : g == 2 ? hi.z : hi.w;
                        uint32_t al[4], ah[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            al[e] = decode_pair(wl, e, mask, base);
                            ah[e] = decode_pair(wh, e, mask, base);
                        }
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            if (fresh) mma_bf16_first(c[h][t], al[0], ah[0], al[1], ah[1], b[t].x, b[t].y);
                            else mma_bf16(c[h][t], al[0], ah[0], al[1], ah[1], b[t].x, b[t].y);
                        }
#pragma unroll
                        for (int t = 0; t < NT; ++t) mma_bf16(c[h][t], al[2], ah[2], al[3], ah[3], b[t].z, b[t].w);
                    }
                    if (g % (4 / PER) == 4 / PER - 1) {
                        const int q = g / (4 / PER);
                        uint64_t x2[NT];
                        if constexpr (MINS)
#pragma unroll
                            for (int t = 0; t < NT; ++t) x2[t] = xsum[(chunk * PER + q) * (4 * NT) + 4 * t];
#pragma unroll
                        for (int h = 0; h < RS; ++h) {
                            const float s0 = scale_at<PER>(sc[j][h], 0, q), s1 = scale_at<PER>(sc[j][h], 1, q);
                            const uint64_t s00 = pack2(s0, s0), s11 = pack2(s1, s1);
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                acc[h][t][0] = fma2(s00, pack2(c[h][t][0], c[h][t][1]), acc[h][t][0]);
                                acc[h][t][1] = fma2(s11, pack2(c[h][t][2], c[h][t][3]), acc[h][t][1]);
                            }
                            if constexpr (MINS) {
                                const float b0 = __fmaf_rn(8.0f, s0, -scale_at<PER>(mn[j][h], 0, q));
                                const float b1 = __fmaf_rn(8.0f, s1, -scale_at<PER>(mn[j][h], 1, q));
                                const uint64_t b00 = pack2(b0, b0), b11 = pack2(b1, b1);
#pragma unroll
                                for (int t = 0; t < NT; ++t) {
                                    acc[h][t][0] = fma2(b00, x2[t], acc[h][t][0]);
                                    acc[h][t][1] = fma2(b11, x2[t], acc[h][t][1]);
                                }
                            }
                        }
                    }
                }
                if (i + j + S::kDepth < end) load(j);
                if (++chunk == mine || i + j + 1 == end) {
                    const float4 v0 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    float4 part[RS][NT];
#pragma unroll
                    for (int h = 0; h < RS; ++h)
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const float2 lo = unpack2(acc[h][t][0]), hi = unpack2(acc[h][t][1]);
                            part[h][t] = make_float4(lo.x, lo.y, hi.x, hi.y);
                            acc[h][t][0] = acc[h][t][1] = 0;
                        }
                    if (!SPLIT && chunk == mine && unit * mine >= begin) {          // all of the unit is this warp's
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            if constexpr (GATEUP) {
                                store(batch + unit, t * 32 + lane, part[0][t], part[1][t]);
                            } else {
#pragma unroll
                                for (int h = 0; h < RS; ++h) store(batch + unit, (h * NT + t) * 32 + lane, part[h][t], v0);
                            }
                        }
                    } else {
                        const int slot = SPLIT ? unit + warp : 2 * warp + (unit * mine >= begin);
#pragma unroll
                        for (int h = 0; h < RS; ++h)
#pragma unroll
                            for (int t = 0; t < NT; ++t) slots[slot * kAll + (h * NT + t) * 32 + lane] = part[h][t];
                    }
                    if (chunk == mine) {
                        chunk = 0;
                        ++unit;
                    }
                }
            }
        }
        const int total = count * mine;
        __syncthreads();
        // a CTA's own parts of a unit, k ascending
        auto own_sum = [&](int u, int f) {
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const int w1 = share_of<S::kWarps>(u * mine + mine - 1, total);
            for (int w = share_of<S::kWarps>(u * mine, total); w <= w1; ++w) {
                const int w_begin = share_begin<S::kWarps>(w, total);
                if (w_begin == share_begin<S::kWarps>(w + 1, total)) continue;
                v = plus(v, slots[(SPLIT ? u + w : 2 * w + (u * mine >= w_begin)) * kAll + f]);
            }
            return v;
        };
        if constexpr (!SPLIT) {
            // the unit that begins before warp w's share and goes on in it, if no warp before has it, too
            for (int i = tid; i < (S::kWarps - 1) * kEach; i += S::kThreads) {
                const int w = 1 + i / kEach, f = i % kEach;
                const int at = share_begin<S::kWarps>(w, total), u = at / mine;
                if (at == total || at % mine == 0) continue;
                const int before = share_begin<S::kWarps>(w - 1, total);
                if (before % mine != 0 && before / mine == u) continue;
                const float4 v = own_sum(u, f);
                store(batch + u, f, v, GATEUP ? own_sum(u, NT * 32 + f) : v);
            }
            return;
        } else {
            // (a unit's sum goes where its first part was: only the thread that adds it up reads that)
            for (int i = tid; i < count * kAll; i += S::kThreads) {
                const int u = i / kAll, f = i % kAll;
                const float4 v = own_sum(u, f);
                slots[(u + share_of<S::kWarps>(u * mine, total)) * kAll + f] = v;
            }
            cluster_sync();
            // the units dealt to one another
            auto all_sum = [&](int u, int f) {
                float4 q[8], v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < cluster) {
                        const int its = (r + 1) * chunks / cluster - r * chunks / cluster;
                        q[r] = ld_cluster(smem_u32(slots + (u + share_of<S::kWarps>(u * its, count * its)) * kAll + f), r);
                    }
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < cluster) v = plus(v, q[r]);
                return v;
            };
            const int own = (count - rank + cluster - 1) / cluster;
            for (int i = tid; i < own * kEach; i += S::kThreads) {
                const int u = i / kEach * cluster + rank, f = i % kEach;
                const float4 v = all_sum(u, f);
                store(batch + u, f, v, GATEUP ? all_sum(u, NT * 32 + f) : v);
            }
            cluster_sync();
            batch += S::kBatch;
            if (batch < to) open();
        }
    }
}

template <int NT, int RS, int PER, bool MINS, bool GATEUP, bool SPLIT>
cudaError_t launch(StreamArgs &a, int dev, int sms, cudaStream_t stream) {
    using S = Shape<NT, RS, SPLIT>;
    const int chunks = a.p.k / 128;
    if constexpr (!SPLIT)
        if (chunks > S::kMaxChunks) return launch<NT, RS, PER, MINS, GATEUP, true>(a, dev, sms, stream);
    static SmemLimit limit;
    cudaError_t e = limit.raise(q4_stream_kernel<NT, RS, PER, MINS, GATEUP, SPLIT>, 227 * 1024);
    if (e != cudaSuccess) return e;
    const int64_t strips = q4_strips(a.p.n), units = GATEUP ? strips : (strips + RS - 1) / RS;
    a.cluster = SPLIT ? (chunks + S::kMaxChunks - 1) / S::kMaxChunks : 1;
    int most = sms;
    if constexpr (SPLIT) {
        static ClusterLimit cluster_limit;
        e = cluster_limit.most(q4_stream_kernel<NT, RS, PER, MINS, GATEUP, SPLIT>, dev, a.cluster, S::kThreads, 227 * 1024, sms, &most);
        if (e != cudaSuccess) return e;
    }
    const int clusters = static_cast<int>(units < most ? units : most);
    const int mine = (chunks + a.cluster - 1) / a.cluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(clusters * a.cluster);
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSlots * S::kSlotBytes + static_cast<size_t>(mine) * (S::kChunkBytes + (MINS ? NT * 8 * PER * 4 : 0));
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = SPLIT ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, q4_stream_kernel<NT, RS, PER, MINS, GATEUP, SPLIT>, a);
}

template <int NT, int PER>
cudaError_t pick(StreamArgs &a, int dev, int sms, cudaStream_t stream) {
    const bool mins = a.p.mins[0] != nullptr;
    if (a.p.mats == 2) return mins ? launch<NT, 2, PER, true, true, false>(a, dev, sms, stream) : launch<NT, 2, PER, false, true, false>(a, dev, sms, stream);
    // a strip per unit where pairs are too few to come out even (one row: 5120 x 5120 6.3 us, with pairs 8.1; 131072 x
    // 5120 67, with pairs 64)
    if constexpr (NT == 1)
        if (q4_strips(a.p.n) < 8 * sms)
            return mins ? launch<1, 1, PER, true, false, false>(a, dev, sms, stream) : launch<1, 1, PER, false, false, false>(a, dev, sms, stream);
    return mins ? launch<NT, 2, PER, true, false, false>(a, dev, sms, stream) : launch<NT, 2, PER, false, false, false>(a, dev, sms, stream);
}

template <int NT>
cudaError_t pick(StreamArgs &a, int dev, int sms, cudaStream_t stream) {
    return a.p.group == 128 ? pick<NT, 1>(a, dev, sms, stream) : a.p.group == 64 ? pick<NT, 2>(a, dev, sms, stream) : pick<NT, 4>(a, dev, sms, stream);
}

}  // namespace

cudaError_t q4_stream_launch(const Q4Product &p, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    StreamArgs a{};
    a.p = p;
    return p.m > 8 ? pick<2>(a, dev, sms, stream) : pick<1>(a, dev, sms, stream);
}

}  // namespace tq
