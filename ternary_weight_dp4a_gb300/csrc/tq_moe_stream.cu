// tq_moe_stream.cu -- products grouped by expert for few rows per expert: the
// weights stream from HBM through registers into warp-level matrix
// instructions, the activations of up to 8 rows wait in shared memory.
//
// Mathematics.  A block dot d = sum w*q over 128 weights in {-1, 0, +1} and int8
// q is an exact integer below 2^14; fp16 operands hold both sides exactly and
// the matrix instruction (m16n8k16, the weights as its 16 rows) adds in fp32.
//   2-bit: codes 0, 1, 2 become 0, 1, 3 (one operation for 16 codes); the two bits of
//   0, 1, 3, moved to the top of a half word, are the fp16 numbers 0, +2, -2:
//   a shift and a mask make two weights.  The activations are q / 2.
//   1-bit: the bit, moved to the sign, turns -1 into +1: a shift and a mask-and-xor.
// Per 128-block and output the kernel then adds one fma(d, scale_w * scale_a,
// acc), blocks in ascending order, the order that tq_moe.h documents.
//
// (fp8 operands would need fewer decode operations, but mma.sync on fp8 is
// emulated here: 11 instructions and 6.1 cycles per SM for m16n8k32, against
// 2.0 for a native fp16 m16n8k16.)
#include <cuda_runtime.h>

#include "tq_device.cuh"
#include "tq_launch.h"
#include "tq_moe_internal.h"

namespace tq {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kCols = 8;                     // activation rows per chunk
constexpr int kMaxWarps = 8;

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The weights of one row that a lane holds per block: 32 of them, 8 bytes (2-bit) or 4 (1-bit).
template <int FMT> struct Codes { uint32_t w[FMT == 0 ? 2 : 1]; };

template <int FMT>
__device__ __forceinline__ Codes<FMT> load_codes(const uint8_t *p) {
    Codes<FMT> c;
    if (FMT == 0)
        asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(c.w[0]), "=r"(c.w[FMT == 0 ? 1 : 0]) : "l"(p));
    else
        asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(c.w[0]) : "l"(p));
    return c;
}

// Two weights as fp16: pair i (0..15) of a lane's 32.  2-bit: weights 7 - i and 15 - i
// of the first word for i < 8, of the second for the others (each +-2 or 0, codes
// already 0, 1, 3).  1-bit: weights 15 - i and 31 - i (+-1).
template <int FMT>
__device__ __forceinline__ uint32_t weight_pair(const Codes<FMT> &c, int i) {
    if (FMT == 0) return (c.w[FMT == 0 ? i >> 3 : 0] << (2 * (i & 7))) & 0xc000c000u;
    return ((c.w[0] << i) & 0x80008000u) ^ 0xbc00bc00u;
}

// Codes 0, 1, 2 -> 0, 1, 3.
template <int FMT>
__device__ __forceinline__ void signed_codes(Codes<FMT> &c) {
    if (FMT == 0) {
        c.w[0] |= (c.w[0] >> 1) & 0x55555555u;
        c.w[FMT == 0 ? 1 : 0] |= (c.w[FMT == 0 ? 1 : 0] >> 1) & 0x55555555u;
    }
}

// Two int8 codes (bytes i and j of w ^ 0x80808080, so 0..255) as fp16: q / 2 or q.
template <int FMT>
__device__ __forceinline__ uint32_t act_pair(uint32_t a, uint32_t b, uint32_t sel) {
    // 0x64nn is 1024 + n
    const uint32_t u = prmt(prmt(a, b, sel), 0x64646464u, 0x4140u);
    __half2 h = *reinterpret_cast<const __half2 *>(&u);
    h = FMT == 0 ? __hfma2(h, __half2half2(__ushort_as_half(0x3800)), __half2half2(__ushort_as_half(0xe080)))   // * 0.5 - 576
                 : __hadd2(h, __half2half2(__ushort_as_half(0xe480)));                                          // - 1152
    return *reinterpret_cast<const uint32_t *>(&h);
}

struct StreamArgs {
    MoeProduct p;
    int chunk;      // rows of an expert that share a pass over its weights, at most kCols
    int limit;      // experts with more rows are another kernel's
};

// Shared memory of a CTA, behind one another:
//   offsets, chunks (of the experts before) int [experts + 1] each
//   activations fp16 [chunk][block][quarter][t][8]: the 32 of lane t in the order of its
//     weight pairs, 8 at a time; 64 bytes between rows
//   scales [block][8]
//   per warp the weight scales of 8 blocks, [2][32 rows][8] fp16
__host__ __device__ constexpr int list_bytes(int experts) { return (2 * (experts + 1) * 4 + 15) / 16 * 16; }
__host__ __device__ constexpr int row_pitch(int nb) { return nb * 256 + 64; }
constexpr int kScaleBytes = 2 * 32 * 8 * 2;

size_t stream_smem(int experts, int chunk, int nb, int warps) {
    return static_cast<size_t>(list_bytes(experts)) + static_cast<size_t>(chunk) * row_pitch(nb) +
           static_cast<size_t>(nb) * kCols * sizeof(float) + static_cast<size_t>(warps) * kScaleBytes;
}

// Fill offsets (clamped) and chunks (all threads); returns the number of chunks.
__device__ __forceinline__ int list_chunks(const MoeProduct &p, int chunk, int limit, int *offsets, int *chunks) {
    const int tid = threadIdx.x, lane = tid & 31;
    for (int e = tid; e <= p.experts; e += blockDim.x) offsets[e] = min(max(p.offsets[e], 0), p.slots);
    __syncthreads();
    if (tid < 32) {
        int base = 0;
        for (int e0 = 0; e0 < p.experts; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < p.experts ? max(offsets[e + 1] - offsets[e], 0) : 0;
            const int c = n <= limit ? (n + chunk - 1) / chunk : 0;
            int incl = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFull, incl, o);
                if (lane >= o) incl += v;
            }
            if (e < p.experts) chunks[e] = base + incl - c;
            base += __shfl_sync(kFull, incl, 31);
        }
        if (lane == 0) chunks[p.experts] = base;
    }
    __syncthreads();
    return chunks[p.experts];
}

// Lay the codes of `rows` activation rows out in shared memory (all threads).
template <int FMT>
__device__ __forceinline__ void stage_rows(const MoeProduct &p, int row0, int rows, uint8_t *act, float *meta) {
    const int tid = threadIdx.x, nb = p.k / kBlock, pitch = row_pitch(nb), per = nb * 4;
#pragma unroll 2
    for (int i = tid; i < rows * per; i += blockDim.x) {
        const int r = i / per, c = i - r * per;                      // c: group of 32 codes
        int a = p.rows != nullptr ? p.rows[row0 + r] : row0 + r;
        a = min(max(a, 0), p.m - 1);
        const uint4 *qp = reinterpret_cast<const uint4 *>(p.q + static_cast<int64_t>(a) * p.k + c * 32);
        const uint4 q0 = __ldg(qp), q1 = __ldg(qp + 1);
        const float sa = (c & 3) == 0 ? __ldg(p.s + static_cast<int64_t>(a) * nb + (c >> 2)) : 0.0f;
        const uint32_t flip = 0x80808080u;
        const uint32_t w[8] = {q0.x ^ flip, q0.y ^ flip, q0.z ^ flip, q0.w ^ flip,
                               q1.x ^ flip, q1.y ^ flip, q1.z ^ flip, q1.w ^ flip};
        uint8_t *dst = act + r * pitch + (c >> 2) * 256 + (c & 3) * 16;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            uint32_t o[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int i = 4 * x + y;                             // the pair
                const int e0 = FMT == 0 ? 16 * (i >> 3) + 7 - (i & 7) : 15 - i, e1 = e0 + (FMT == 0 ? 8 : 16);
                o[y] = act_pair<FMT>(w[e0 >> 2], w[e1 >> 2], (e0 & 3) | ((4 + (e1 & 3)) << 4));
            }
            *reinterpret_cast<uint4 *>(dst + 64 * x) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        if ((c & 3) == 0) meta[(c >> 2) * kCols + r] = sa;
    }
    const int none = kCols - rows;
    for (int i = tid; i < none * nb; i += blockDim.x) meta[(i / none) * kCols + rows + i % none] = 0.0f;
}

// The blocks whose codes are on their way while one is computed.
template <int FMT> constexpr int kAhead = FMT == 0 ? 4 : 8;

// A warp's unit: 32 weight rows (16 of gate and of up, or 32 of one matrix) against
// the staged activation rows, over all of k.
template <int FMT, bool GATEUP>
__device__ __forceinline__ void unit(const MoeProduct &p, int expert, int row0, int rows, int n0, bool wide,
                                     const uint8_t *act, const float *meta, uint16_t *wsc) {
    constexpr int kA = kAhead<FMT>;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int nb = p.k / kBlock;
    constexpr int kBlockBytes = FMT == 0 ? 32 : 16;
    const int64_t row_bytes = static_cast<int64_t>(nb) * kBlockBytes;

    // rows g and g + 8 of the row tiles mt = 0, 1 (gate and up, or two of one matrix)
    const uint8_t *src[2][2];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = min(n0 + (GATEUP ? 0 : 16 * mt) + g + 8 * h, p.n - 1);
            src[mt][h] = p.codes[GATEUP ? mt : 0] + (static_cast<int64_t>(expert) * p.n + r) * row_bytes + t * (kBlockBytes / 4);
        }
    Codes<FMT> ring[kA][2][2];
#pragma unroll
    for (int a = 0; a < kA; ++a)
        if (a < nb)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) ring[a][mt][h] = load_codes<FMT>(src[mt][h] + a * kBlockBytes);

    // weight scales: lane (g, t) brings row g of (mt, h) = (t / 2, t % 2), 8 blocks at a time
    const int sr = min(n0 + (GATEUP ? 0 : 16 * (t >> 1)) + g + 8 * (t & 1), p.n - 1);
    const uint16_t *ssrc = p.scales[GATEUP ? t >> 1 : 0] + (static_cast<int64_t>(expert) * p.n + sr) * nb;
    const auto load_scales = [&](int b) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (wide) {
            v = __ldg(reinterpret_cast<const uint4 *>(ssrc + b));
        } else {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = ldg_u16(ssrc + min(b + i, nb - 1));
            v = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
        }
        return v;
    };
    uint4 snext = load_scales(0);

    float acc[2][4] = {};
    const bool have = g < rows;
    const uint8_t *ap = act + (have ? g : 0) * row_pitch(nb) + t * 16;
#pragma unroll 1
    for (int b0 = 0; b0 < nb; b0 += 8) {
        uint16_t *sbuf = wsc + ((b0 >> 3) & 1) * 256;
        *reinterpret_cast<uint4 *>(sbuf + (8 * t + g) * 8) = snext;
        if (b0 + 8 < nb) snext = load_scales(b0 + 8);
        __syncwarp();
#pragma unroll
        for (int a = 0; a < 8; ++a) {
            const int b = b0 + a, x = a % kA;
            if (b >= nb) break;
            uint4 bq[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                bq[i] = have ? *reinterpret_cast<const uint4 *>(ap + b * 256 + 64 * i)
                             : make_uint4(0, 0, 0, 0);
            const float2 sa = *reinterpret_cast<const float2 *>(meta + b * kCols + 2 * t);   // of columns 2t, 2t + 1
            float c[2][4] = {};
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                signed_codes<FMT>(ring[x][mt][0]);
                signed_codes<FMT>(ring[x][mt][1]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 &v = bq[i >> 1];
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
                    mma_f16(c[mt], weight_pair<FMT>(ring[x][mt][0], 2 * i), weight_pair<FMT>(ring[x][mt][1], 2 * i),
                            weight_pair<FMT>(ring[x][mt][0], 2 * i + 1), weight_pair<FMT>(ring[x][mt][1], 2 * i + 1),
                            (i & 1) ? v.z : v.x, (i & 1) ? v.w : v.y);
            }
            if (b + kA < nb)
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        ring[x][mt][h] = load_codes<FMT>(src[mt][h] + static_cast<int64_t>(b + kA) * kBlockBytes);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float sw = f16_bits_to_f32(sbuf[(16 * mt + 8 * h + g) * 8 + a]);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[mt][2 * h + j] = __fmaf_rn(c[mt][2 * h + j], __fmul_rn(sw, j == 0 ? sa.x : sa.y), acc[mt][2 * h + j]);
                }
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int col = 2 * t + j;
        if (col >= rows) continue;
        const int64_t out = static_cast<int64_t>(row0 + col) * p.n;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (GATEUP) {
                const int r = n0 + g + 8 * h;
                if (r < p.n) p.h[out + r] = f32_to_bf16_bits(__fmul_rn(tq_silu(acc[0][2 * h + j]), acc[1][2 * h + j]));
            } else {
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    const int r = n0 + 16 * mt + g + 8 * h;
                    if (r < p.n) p.y[out + r] = acc[mt][2 * h + j];
                }
            }
        }
    }
    __syncwarp();                                                    // wsc is the next unit's
}

// A CTA takes a contiguous share of the rounds (chunk by chunk, `warps` units
// each), so that it stages a chunk's activations once for many units.
template <int FMT, bool GATEUP>
__global__ void __launch_bounds__(32 * kMaxWarps, 2) stream_kernel(const __grid_constant__ StreamArgs args) {
    extern __shared__ __align__(16) uint8_t smem[];
    const MoeProduct &p = args.p;
    pdl_launch_dependents();
    pdl_wait();
    const int nb = p.k / kBlock, warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
    int *offsets = reinterpret_cast<int *>(smem), *chunks = offsets + p.experts + 1;
    uint8_t *act = smem + list_bytes(p.experts);
    float *meta = reinterpret_cast<float *>(act + args.chunk * row_pitch(nb));
    uint16_t *wsc = reinterpret_cast<uint16_t *>(meta + nb * kCols) + warp * (kScaleBytes / 2);
    constexpr int kUnitRows = GATEUP ? 16 : 32;
    const int units = (p.n + kUnitRows - 1) / kUnitRows, per_chunk = (units + warps - 1) / warps;
    const int64_t rounds = static_cast<int64_t>(list_chunks(p, args.chunk, args.limit, offsets, chunks)) * per_chunk;
    int64_t r = rounds * blockIdx.x / gridDim.x;
    const int64_t end = rounds * (blockIdx.x + 1) / gridDim.x;
    const bool wide = nb % 8 == 0 && (reinterpret_cast<uintptr_t>(p.scales[0]) & 15) == 0 &&
                      (!GATEUP || (reinterpret_cast<uintptr_t>(p.scales[1]) & 15) == 0);
    int staged = -1, expert = 0, row0 = 0, rows = 0;
    for (; r < end; ++r) {
        const int chunk = static_cast<int>(r / per_chunk), u = static_cast<int>(r % per_chunk) * warps + warp;
        if (chunk != staged) {
            int lo = 0, hi = p.experts;                              // chunks[lo] <= chunk < chunks[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (chunks[mid] <= chunk) lo = mid;
                else hi = mid;
            }
            expert = lo;
            row0 = offsets[lo] + (chunk - chunks[lo]) * args.chunk;
            rows = min(args.chunk, offsets[lo + 1] - row0);
            if (staged >= 0) __syncthreads();                        // every warp is done with the chunk before
            stage_rows<FMT>(p, row0, rows, act, meta);
            __syncthreads();
            staged = chunk;
        }
        if (u < units) unit<FMT, GATEUP>(p, expert, row0, rows, u * kUnitRows, wide, act, meta, wsc);
    }
}

template <int FMT, bool GATEUP>
cudaError_t launch(const MoeProduct &p, int limit, cudaStream_t stream) {
    StreamArgs a{p, 0, limit};
    const int nb = p.k / kBlock;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    constexpr int64_t kUnitRows = GATEUP ? 16 : 32;
    const int64_t units = ws_cdiv(p.n, kUnitRows);
    // fewer warps to a CTA where one chunk for each expert would not give every SM two CTAs
    const int64_t active = p.experts < p.slots ? p.experts : p.slots;
    int warps = kMaxWarps;
    while (warps > 2 && active * ws_cdiv(units, warps) < 2 * sms) warps /= 2;
    // as many rows at once as fit in shared memory (two CTAs on an SM), at most 8 and no more than an expert has
    constexpr size_t kSmem = 227 * 1024;
    int chunk = p.max_rows < kCols ? p.max_rows : kCols;
    while (chunk > 1 && stream_smem(p.experts, chunk, nb, warps) > kSmem) --chunk;
    const size_t smem = stream_smem(p.experts, chunk, nb, warps);
    if (smem > kSmem) return cudaErrorInvalidValue;
    a.chunk = chunk;
    e = cudaFuncSetAttribute(stream_kernel<FMT, GATEUP>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    int per_sm = static_cast<int>((kSmem + 1024) / (smem + 1024));
    if (per_sm > 16 / warps) per_sm = 16 / warps;
    if (per_sm < 1) per_sm = 1;
    // an upper bound of the chunks: one per expert and one more for every full one
    int64_t most = static_cast<int64_t>(p.experts) + p.slots / chunk;
    if (most > p.slots) most = p.slots;
    const int64_t cap = static_cast<int64_t>(p.experts) * ws_cdiv(limit, chunk);
    if (most > cap) most = cap;
    int64_t grid = most * ws_cdiv(units, warps);
    if (grid > static_cast<int64_t>(sms) * per_sm) grid = static_cast<int64_t>(sms) * per_sm;
    return launch_pdl(stream_kernel<FMT, GATEUP>, dim3(static_cast<unsigned>(grid)), dim3(32 * warps), smem, stream, a);
}

}  // namespace

cudaError_t moe_stream_launch(const MoeProduct &p, int limit, cudaStream_t stream) {
    if (p.h != nullptr) return p.fmt == TQ_FMT_TERNARY2 ? launch<0, true>(p, limit, stream) : launch<1, true>(p, limit, stream);
    return p.fmt == TQ_FMT_TERNARY2 ? launch<0, false>(p, limit, stream) : launch<1, false>(p, limit, stream);
}

}  // namespace tq
