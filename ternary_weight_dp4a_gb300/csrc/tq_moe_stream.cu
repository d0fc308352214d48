// tq_moe_stream.cu -- products grouped by expert for few rows per expert: the
// weights stream from HBM through registers into warp-level matrix
// instructions, the activations of up to 8 rows wait in shared memory.
//
// Mathematics.  A block dot d = sum w*q over 128 weights in {-1, 0, +1} and int8
// q is an exact integer.  The matrix instruction multiplies e4m3 numbers
// exactly and adds in fp32, so q goes in as two e4m3 numbers, both exact, in
// units of 2^-9: |q| = 16 H + L, with L (0..15) the e4m3 bit pattern itself (the
// subnormals and the first binade of e4m3 are linear: pattern p is p * 2^-9)
// and 16 H * 2^-9 a power of two times 0..7; the sign is the byte's top bit.
// 2-bit codes decode to w + 1 = 1, 2, 0 (one prmt per four codes, in the order
// of tq_dp4a.cuh), and the accumulators start at -sum(q) * 2^-9 instead of 0.
// 1-bit codes decode to +-1.  Every partial sum is an integer below 2^16 in
// units of 2^-9: exact in fp32.
//
// Per 128-block and output the kernel then adds one fma(d, scale_w * scale_a,
// acc), blocks in ascending order, the order that tq_moe.h documents.
#include <cuda_runtime.h>

#include "tq_device.cuh"
#include "tq_dp4a.cuh"
#include "tq_launch.h"
#include "tq_moe_codes.cuh"
#include "tq_moe_internal.h"

namespace tq {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTileM = 32 * kWarps;          // weight rows per CTA
constexpr int kCols = 8;                     // activation rows per CTA
constexpr int kScalePitch = kTileM + 2;      // odd number of words: no bank conflicts on either side

// e4m3 numbers 1.0 (codes w + 1 = 1) and 2.0 (w + 1 = 2): pools for prmt
constexpr uint32_t kOne = 0x38383838u, kTwo = 0x40404040u;

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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

// Eight registers of four e4m3 weights each, in staged order.
template <int FMT>
__device__ __forceinline__ void decode(const Codes<FMT> &c, uint32_t (&r)[8]) {
    if (FMT == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t w = c.w[FMT == 0 ? h : 0];
            r[4 * h + 0] = prmt(kOne, kTwo, w << 2);
            r[4 * h + 1] = prmt(kOne, kTwo, w >> 14);
            r[4 * h + 2] = prmt(kOne, kTwo, w);
            r[4 * h + 3] = prmt(kOne, kTwo, w >> 16);
        }
    } else {
#pragma unroll
        for (int s = 0; s < 8; ++s) r[s] = ((c.w[0] << (7 - s)) & 0x80808080u) ^ 0xb8b8b8b8u;   // 1 -> +1, 0 -> -1
    }
}

struct StreamArgs {
    MoeProduct p;
    int chunk;      // rows of an expert per CTA, at most kCols
    int limit;      // experts with more rows are another kernel's
};

// One warp looks for the pair'th (expert, chunk of its rows); false behind the last.
__device__ __forceinline__ bool find_chunk(const int *offsets, int experts, int slots, int chunk, int limit, int pair,
                                           int &expert, int &row0, int &rows) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int e0 = 0; e0 < experts; e0 += 32) {
        const int e = e0 + lane;
        int lo = 0, n = 0;
        if (e < experts) {
            lo = min(max(offsets[e], 0), slots);
            n = max(min(max(offsets[e + 1], 0), slots) - lo, 0);
        }
        const int c = n <= limit ? (n + chunk - 1) / chunk : 0;
        int incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += v;
        }
        const unsigned hit = __ballot_sync(kFull, pair < base + incl);
        if (hit != 0) {
            const int src = __ffs(hit) - 1;
            const int first = (pair - base - __shfl_sync(kFull, incl - c, src)) * chunk;
            expert = e0 + src;
            row0 = __shfl_sync(kFull, lo, src) + first;
            rows = min(chunk, __shfl_sync(kFull, n, src) - first);
            return true;
        }
        base += __shfl_sync(kFull, incl, 31);
    }
    return false;
}

constexpr int kAhead = 4;   // blocks whose codes are on their way

template <int FMT, bool GATEUP>
__global__ void __launch_bounds__(kThreads) stream_kernel(const __grid_constant__ StreamArgs args) {
    extern __shared__ __align__(16) uint8_t smem[];
    const MoeProduct &p = args.p;
    pdl_launch_dependents();
    pdl_wait();
    int expert, row0, rows;
    if (!find_chunk(p.offsets, p.experts, p.slots, args.chunk, args.limit, blockIdx.x, expert, row0, rows)) return;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int nb = p.k / kBlock;
    const int n0 = blockIdx.y * (GATEUP ? kTileM / 2 : kTileM);
    constexpr int kBlockBytes = FMT == 0 ? 32 : 16;
    const int64_t row_bytes = static_cast<int64_t>(nb) * kBlockBytes;

    // this lane's four weight rows: row tiles mt = 0, 1 (gate and up, or two
    // tiles of one matrix), rows g and g + 8 of each
    const uint8_t *src[2][2];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int r = GATEUP ? n0 + 16 * warp + g + 8 * h : n0 + 32 * warp + 16 * mt + g + 8 * h;
            r = min(r, p.n - 1);
            src[mt][h] = p.codes[GATEUP ? mt : 0] + (static_cast<int64_t>(expert) * p.n + r) * row_bytes +
                         t * (kBlockBytes / 4);
        }
    Codes<FMT> ring[kAhead][2][2];
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
        if (a < nb)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) ring[a][mt][h] = load_codes<FMT>(src[mt][h] + a * kBlockBytes);

    // activations: [row][block][hi 128 | lo 128] with 16 bytes between rows,
    // then (scale, -sum q * 2^-9) [block][8], then the weight scales [block][tile row]
    const int pitch = nb * 256 + 16;
    float2 *meta = reinterpret_cast<float2 *>(smem + args.chunk * pitch);
    uint16_t *wsc = reinterpret_cast<uint16_t *>(meta + nb * kCols);
    for (int i = tid; i < rows * nb * 4; i += kThreads) {
        const int r = i / (nb * 4), c = i - r * (nb * 4);            // c: group of 32 codes
        int a = p.rows != nullptr ? p.rows[row0 + r] : row0 + r;
        a = min(max(a, 0), p.m - 1);
        const uint4 *qp = reinterpret_cast<const uint4 *>(p.q + static_cast<int64_t>(a) * p.k + c * 32);
        const uint4 q0 = __ldg(qp), q1 = __ldg(qp + 1);
        const uint32_t w[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
        uint32_t o[8], hi[8], lo[8];
        stage_order<FMT>(w, o);
        int sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sum = __dp4a(static_cast<int>(w[j]), 0x01010101, sum);
            split4(o[j], hi[j], lo[j]);
        }
        const unsigned quad = 0xfu << (lane & ~3);                   // a block's four lanes take this turn together
        sum += __shfl_xor_sync(quad, sum, 1);
        sum += __shfl_xor_sync(quad, sum, 2);
        uint8_t *dst = smem + r * pitch + (c >> 2) * 256 + (c & 3) * 32;
        *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(dst + 16) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
        *reinterpret_cast<uint4 *>(dst + 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<uint4 *>(dst + 144) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
        if ((c & 3) == 0)
            meta[(c >> 2) * kCols + r] =
                make_float2(__ldg(p.s + static_cast<int64_t>(a) * nb + (c >> 2)),
                            FMT == 0 ? __fmul_rn(static_cast<float>(-sum), 0.001953125f) : 0.0f);
    }
    for (int i = tid; i < (kCols - rows) * nb; i += kThreads)
        meta[(i / (kCols - rows)) * kCols + rows + i % (kCols - rows)] = make_float2(0.0f, 0.0f);
    for (int i = tid; i < kTileM * nb; i += kThreads) {
        const int lr = i / nb, b = i - lr * nb;
        const int r = GATEUP ? n0 + (lr >> 5) * 16 + (lr & 15) : n0 + lr;
        const uint16_t *sp = p.scales[GATEUP ? (lr >> 4) & 1 : 0];
        wsc[b * kScalePitch + lr] = ldg_u16(sp + (static_cast<int64_t>(expert) * p.n + min(r, p.n - 1)) * nb + b);
    }
    __syncthreads();

    float acc[2][4] = {};
    const bool have = g < rows;
    const uint8_t *act = smem + (have ? g : 0) * pitch + t * 32;
#pragma unroll 1
    for (int b0 = 0; b0 < nb; b0 += kAhead) {
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const int b = b0 + a;
            if (b >= nb) break;
            uint4 bq[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                bq[i] = have ? *reinterpret_cast<const uint4 *>(act + b * 256 + (i & 1) * 16 + (i >> 1) * 128)
                             : make_uint4(0, 0, 0, 0);
            const float4 mm = *reinterpret_cast<const float4 *>(meta + b * kCols + 2 * t);   // (s, -sum) of columns 2t, 2t+1
            float c[2][4];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                c[mt][0] = c[mt][2] = mm.y;
                c[mt][1] = c[mt][3] = mm.w;
                uint32_t w0[8], w1[8];
                decode<FMT>(ring[a][mt][0], w0);
                decode<FMT>(ring[a][mt][1], w1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 &bh = bq[i >> 1], &bl = bq[2 + (i >> 1)];
                    mma_e4m3(c[mt], w0[2 * i], w1[2 * i], w0[2 * i + 1], w1[2 * i + 1], (i & 1) ? bh.z : bh.x,
                             (i & 1) ? bh.w : bh.y);
                    mma_e4m3(c[mt], w0[2 * i], w1[2 * i], w0[2 * i + 1], w1[2 * i + 1], (i & 1) ? bl.z : bl.x,
                             (i & 1) ? bl.w : bl.y);
                }
            }
            if (b + kAhead < nb)
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        ring[a][mt][h] = load_codes<FMT>(src[mt][h] + static_cast<int64_t>(b + kAhead) * kBlockBytes);
            const uint16_t *ws = wsc + b * kScalePitch + 32 * warp + g;
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float sw = f16_bits_to_f32(ws[16 * mt + 8 * h]);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[mt][2 * h + j] = __fmaf_rn(__fmul_rn(c[mt][2 * h + j], 512.0f),
                                                       __fmul_rn(sw, j == 0 ? mm.x : mm.z), acc[mt][2 * h + j]);
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
                const int r = n0 + 16 * warp + g + 8 * h;
                if (r < p.n) p.h[out + r] = f32_to_bf16_bits(__fmul_rn(tq_silu(acc[0][2 * h + j]), acc[1][2 * h + j]));
            } else {
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    const int r = n0 + 32 * warp + 16 * mt + g + 8 * h;
                    if (r < p.n) p.y[out + r] = acc[mt][2 * h + j];
                }
            }
        }
    }
}

size_t stream_smem(int chunk, int nb) {
    return static_cast<size_t>(chunk) * (nb * 256 + 16) + static_cast<size_t>(nb) * kCols * sizeof(float2) +
           static_cast<size_t>(nb) * kScalePitch * sizeof(uint16_t);
}

template <int FMT, bool GATEUP>
cudaError_t launch(const MoeProduct &p, int limit, cudaStream_t stream) {
    StreamArgs a{p, 0, limit};
    const int nb = p.k / kBlock;
    // as many rows per CTA as fit in shared memory, at most 8 and no more than an expert has
    int chunk = p.max_rows < kCols ? p.max_rows : kCols;
    constexpr size_t kSmem = 227 * 1024;
    while (chunk > 1 && stream_smem(chunk, nb) > kSmem) --chunk;
    const size_t smem = stream_smem(chunk, nb);
    if (smem > kSmem) return cudaErrorInvalidValue;
    a.chunk = chunk;
    cudaError_t e = cudaFuncSetAttribute(stream_kernel<FMT, GATEUP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    // an upper bound of the (expert, chunk) pairs; CTAs behind the last pair leave at once
    int64_t most = static_cast<int64_t>(p.experts) + p.slots / chunk;
    if (most > p.slots) most = p.slots;
    const int64_t cap = static_cast<int64_t>(p.experts) * ws_cdiv(limit, chunk);
    if (most > cap) most = cap;
    const int tile = GATEUP ? kTileM / 2 : kTileM;
    const dim3 grid(static_cast<unsigned>(most), static_cast<unsigned>((p.n + tile - 1) / tile));
    return launch_pdl(stream_kernel<FMT, GATEUP>, grid, dim3(kThreads), smem, stream, a);
}

}  // namespace

cudaError_t moe_stream_launch(const MoeProduct &p, int limit, cudaStream_t stream) {
    if (p.h != nullptr) return p.fmt == TQ_FMT_TERNARY2 ? launch<0, true>(p, limit, stream) : launch<1, true>(p, limit, stream);
    return p.fmt == TQ_FMT_TERNARY2 ? launch<0, false>(p, limit, stream) : launch<1, false>(p, limit, stream);
}

}  // namespace tq
