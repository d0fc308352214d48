// tq_moe_norm.cu -- the ends of a mixture-of-experts layer: residual addition +
// RMS norm + rotation + int8 quantisation (tq_add_rmsnorm_rotq), and the
// weighted sum over a token's experts (tq_moe_combine).
#include <cuda_runtime.h>

#include "tq_device.cuh"
#include "tq_launch.h"
#include "tq_moe_codes.cuh"
#include "tq_moe_internal.h"

namespace tq {
namespace {

// A warp works on four 128-blocks at a time: lane l holds elements 16 (l % 8) .. + 15 of
// block l / 8, so the transform's spans 1 .. 8 stay in registers and three
// exchanges do the rest (with four elements of one block per lane it takes five, and
// the shuffles alone then bound the kernel).

constexpr uint32_t kFull = 0xffffffffu;

// (hi, lo) += v as an unevaluated sum (T. J. Dekker, D. E. Knuth: two-sum).
__device__ __forceinline__ void pair_add(float &hi, float &lo, float v, float v_lo) {
    const float t = __fadd_rn(hi, v);
    const float b = __fsub_rn(t, hi);
    const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(v, b));
    hi = t;
    lo = __fadd_rn(lo, __fadd_rn(e, v_lo));
}

// Sixteen elements from i on (plain loads: the residual may be updated in place).
template <bool BF16>
__device__ __forceinline__ void load16(const void *p, int64_t i, float (&v)[16]) {
    if (BF16) {
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint4 w = src[j];
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                v[8 * j + 2 * x] = __uint_as_float(u[x] << 16);
                v[8 * j + 2 * x + 1] = __uint_as_float(u[x] & 0xffff0000u);
            }
        }
    } else {
        const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 w = src[j];
            v[4 * j] = w.x; v[4 * j + 1] = w.y; v[4 * j + 2] = w.z; v[4 * j + 3] = w.w;
        }
    }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}

// Round to bf16, store where asked, and go on with the rounded values.
__device__ __forceinline__ void round_store_bf16(float (&v)[16], uint16_t *out) {
    uint32_t w[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
        w[x] = pack_bf16x2(v[2 * x], v[2 * x + 1]);
        v[2 * x] = __uint_as_float(w[x] << 16);
        v[2 * x + 1] = __uint_as_float(w[x] & 0xffff0000u);
    }
    if (out != nullptr) {
        reinterpret_cast<uint4 *>(out)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4 *>(out)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// Sum of the squares of a lane's 16 values as a pair, in four operations each: with
// t = fma(x, x, hi), t - hi is exact as long as hi >= x^2, and fma(x, x, -(t - hi)) is what the
// rounding of t lost (the product's own low half with it).  So the sum starts from the largest
// square, which is taken off again.
__device__ __forceinline__ void pair_squares(const float (&v)[16], float &hi, float &lo) {
    float top = fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, fabsf(v[i]));
    const float base = __fmul_rn(top, top), base_lo = __fmaf_rn(top, top, -base);
    hi = base;
    lo = base_lo;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float t = __fmaf_rn(v[i], v[i], hi);
        lo = __fadd_rn(lo, __fmaf_rn(v[i], v[i], __fsub_rn(hi, t)));
        hi = t;
    }
    pair_add(hi, lo, -base, -base_lo);
}

// tq_rotate_quant's transform of the warp's four blocks, stage by stage in its order.
// Elements i and i + 8 are the halves of one packed operation.
__device__ __forceinline__ void wht128_x16(float (&v)[16], int lane) {
    uint64_t w[8];
    const uint64_t minus = pack2(-1.0f, -1.0f);                  // a - b is fma(b, -1, a)
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack2(v[i], v[i + 8]);
#pragma unroll
    for (int h = 1; h < 8; h <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & h)) {
                const uint64_t a = w[i], b = w[i + h];
                w[i] = add2(a, b);
                w[i + h] = fma2(b, minus, a);
            }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float a, b;
        unpack2(w[i], a, b);
        v[i] = __fadd_rn(a, b);
        v[i + 8] = __fsub_rn(a, b);
    }
#pragma unroll
    for (int h = 1; h < 8; h <<= 1) {
        const float sign = (lane & h) ? -1.0f : 1.0f;            // upper: other - mine; lower: other + mine
#pragma unroll
        for (int i = 0; i < 8; ++i)
            unpack2(fma2(pack2(v[i], v[i + 8]), pack2(sign, sign),
                         pack2(__shfl_xor_sync(kFull, v[i], h), __shfl_xor_sync(kFull, v[i + 8], h))),
                    v[i], v[i + 8]);
    }
    const float c128 = __uint_as_float(0x3db504f3u);             // (float)(1/sqrt(128))
#pragma unroll
    for (int i = 0; i < 8; ++i) unpack2(mul2(pack2(v[i], v[i + 8]), pack2(c128, c128)), v[i], v[i + 8]);
}

// Quantise as tq_rotate_quant: s = max|v| / 127 and round-half-even(v / s), both IEEE
// divisions.  The quotient is first taken through a reciprocal, off by less than 4e-5; only
// where that leaves the rounding open (nearer than 4e-5 to a half) is it divided out.
__device__ __forceinline__ float quant_x16(const float (&v)[16], uint32_t (&word)[4]) {
    float top = fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, fabsf(v[i]));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    const float s = __fdiv_rn(top, 127.0f);
#pragma unroll
    for (int j = 0; j < 4; ++j) word[j] = 0;
    if (!(s > 0.0f && s < INFINITY)) return s;                   // a block of zeros, or not finite
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    float off = 0.0f;
    uint32_t z[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float y = __fmul_rn(v[i], inv);
        const float m = __fadd_rn(y, 12582912.0f);               // its low byte is the rounded y
        off = fmaxf(off, fabsf(__fsub_rn(y, __fsub_rn(m, 12582912.0f))));
        z[i] = __float_as_uint(m);
    }
    if (!(s > 1e-36f) || off > 0.49996f) {
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = static_cast<uint32_t>(__float2int_rn(__fdiv_rn(v[i], s)));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        word[j] = prmt(prmt(z[4 * j], z[4 * j + 1], 0x0040u), prmt(z[4 * j + 2], z[4 * j + 3], 0x0040u), 0x5410u);
    return s;
}

// fp32(1 / sqrt((hi + lo) / n + eps)) for a sum of ordinary size, to about 2^-44 before the
// rounding: the mean as a pair, and one Newton step from the approximate root.
__device__ __forceinline__ float inv_rms(float hi, float lo, float n, float eps) {
    const float q = __fdiv_rn(hi, n);
    const float q_lo = __fdiv_rn(__fadd_rn(__fmaf_rn(-q, n, hi), lo), n);
    float s = q, s_lo = q_lo;
    pair_add(s, s_lo, eps, 0.0f);
    const float h = __fadd_rn(s, s_lo), l = __fsub_rn(s_lo, __fsub_rn(h, s));
    const float y = rsqrtf(h);
    const float y2 = __fmul_rn(y, y), y2_lo = __fmaf_rn(y, y, -y2);
    const float p = __fmul_rn(h, y2), p_lo = __fmaf_rn(h, y2, -p);
    const float d = __fsub_rn(__fsub_rn(1.0f, p), __fadd_rn(p_lo, __fmaf_rn(h, y2_lo, __fmul_rn(l, y2))));
    return __fmaf_rn(y, __fmaf_rn(__fmul_rn(0.375f, d), d, __fmul_rn(0.5f, d)), y);
}

// ---------------------------------------------------------------------------
// Residual addition, RMS norm, rotation, quantisation: one CTA per row; a warp's
// sums t stay in registers between the two passes (sum of squares; normalise,
// rotate, quantise), so the row is read once.  Bound by latency (the barrier between
// the passes) and instructions before memory: 8192 x 5120 bf16 with gamma 71 us, 4.1 TB/s (the
// bytes alone: 43 us); one row 3.5 us, launch to launch.  48 registers let four CTAs of this width
// share an SM: 79 us with the 49 that the compiler takes by itself, 72 with 32.
// ---------------------------------------------------------------------------
template <bool RB, bool DB, int G>
__global__ void __maxnreg__(G == 1 ? 48 : 64) add_rmsnorm_rotq_kernel(const void *res, const void *delta,
                                                                const uint16_t *__restrict__ gamma, int n, float eps,
                                                                void *res_out, uint16_t *__restrict__ x_out,
                                                                int8_t *__restrict__ q, float *__restrict__ s) {
    __shared__ float2 warp_sum[32];
    __shared__ double warp_sum64[32];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * n;
    float t[G][16];
    float hi = 0.0f, lo = 0.0f;
#pragma unroll
    for (int j = 0; j < G; ++j) {
        const int col = (warp + j * warps) * 512 + 16 * lane;
#pragma unroll
        for (int i = 0; i < 16; ++i) t[j][i] = 0.0f;
        if (col < n) {                                           // whole blocks: n is a multiple of 128
            const int64_t at = row + col;
            load16<RB>(res, at, t[j]);
            if (delta != nullptr) {
                float d[16];
                load16<DB>(delta, at, d);
#pragma unroll
                for (int i = 0; i < 16; ++i) t[j][i] = __fadd_rn(t[j][i], d[i]);
            }
            if (RB) {
                round_store_bf16(t[j], res_out != nullptr ? static_cast<uint16_t *>(res_out) + at : nullptr);
            } else if (res_out != nullptr) {
                float4 *out = reinterpret_cast<float4 *>(static_cast<float *>(res_out) + at);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    out[i] = make_float4(t[j][4 * i], t[j][4 * i + 1], t[j][4 * i + 2], t[j][4 * i + 3]);
            }
            float sum, sum_lo;
            pair_squares(t[j], sum, sum_lo);
            if (j == 0) {
                hi = sum;
                lo = sum_lo;
            } else {
                pair_add(hi, lo, sum, sum_lo);
            }
        }
    }
    if (q == nullptr && x_out == nullptr) return;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        pair_add(hi, lo, __shfl_xor_sync(kFull, hi, o), __shfl_xor_sync(kFull, lo, o));
    if (lane == 0) warp_sum[warp] = make_float2(hi, lo);
    __syncthreads();
    {
        const float2 w = lane < warps ? warp_sum[lane] : make_float2(0.0f, 0.0f);
        hi = w.x;
        lo = w.y;
        for (int o = warps > 16 ? 16 : warps > 8 ? 8 : 4; o > 0; o >>= 1)
            pair_add(hi, lo, __shfl_xor_sync(kFull, hi, o), __shfl_xor_sync(kFull, lo, o));
        hi = __shfl_sync(kFull, hi, 0);                          // lanes may differ in lo's last bit
        lo = __shfl_sync(kFull, lo, 0);
    }
    float inv;
    // (with an ordinary eps small sums are fine, too: what they lose is far below eps's last bit;
    // beyond 1e33 the low half of 1 / mean is subnormal and loses bits that the root needs)
    if ((hi > 1e-25f || eps > 1e-12f) && hi < 1e33f && eps < 1e30f) {
        inv = inv_rms(hi, lo, static_cast<float>(n), eps);
    } else {                                                     // out of binary32's comfortable range: in 64 bits
        double acc = 0.0;
#pragma unroll
        for (int j = 0; j < G; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc = fma(static_cast<double>(t[j][i]), static_cast<double>(t[j][i]), acc);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(kFull, acc, o);
        if (lane == 0) warp_sum64[warp] = acc;
        __syncthreads();
        double sum = 0.0;
        for (int w = 0; w < warps; ++w) sum += warp_sum64[w];
        inv = static_cast<float>(1.0 / sqrt(sum / n + static_cast<double>(eps)));
    }
#pragma unroll
    for (int j = 0; j < G; ++j) {
        const int col = (warp + j * warps) * 512 + 16 * lane;
        if ((warp + j * warps) * 512 >= n) break;                // the same for the whole warp
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __fmul_rn(t[j][i], inv);
        if (gamma != nullptr && col < n) {
            float g[16];
            load16<true>(gamma, col, g);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __fmul_rn(v[i], g[i]);
        }
        round_store_bf16(v, x_out != nullptr && col < n ? x_out + row + col : nullptr);
        if (q == nullptr) continue;
        wht128_x16(v, lane);
        uint32_t word[4];
        const float sc = quant_x16(v, word);
        if (col < n) {
            *reinterpret_cast<uint4 *>(q + row + col) = make_uint4(word[0], word[1], word[2], word[3]);
            if ((lane & 7) == 0) s[(row + col) / kBlock] = sc;
        }
    }
}

// tq_rotate_quant of `blocks` 128-blocks that lie behind one another: four per warp.
__global__ void __launch_bounds__(256) rotq_kernel(const uint16_t *x, int64_t blocks, int8_t *__restrict__ q,
                                                   float *__restrict__ s) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5)) * 4;
    if (first >= blocks) return;
    const int64_t block = first + (lane >> 3), at = first * kBlock + 16 * lane;
    float v[16] = {};
    if (block < blocks) load16<true>(x, at, v);
    wht128_x16(v, lane);
    uint32_t word[4];
    const float sc = quant_x16(v, word);
    if (block < blocks) {
        *reinterpret_cast<uint4 *>(q + at) = make_uint4(word[0], word[1], word[2], word[3]);
        if ((lane & 7) == 0) s[block] = sc;
    }
}

template <bool RB, bool DB>
cudaError_t norm_launch(const void *res, const void *delta, const uint16_t *gamma, int m, int n, float eps,
                        void *res_out, uint16_t *x_out, int8_t *q, float *s, cudaStream_t stream) {
    // a warp for every four blocks; two turns beyond 16384
    const int groups = (n + 511) / 512;
    if (groups <= 32)
        return launch_pdl(add_rmsnorm_rotq_kernel<RB, DB, 1>, dim3(m), dim3(32 * groups), 0, stream, res, delta, gamma, n,
                          eps, res_out, x_out, q, s);
    return launch_pdl(add_rmsnorm_rotq_kernel<RB, DB, 2>, dim3(m), dim3(32 * ((groups + 1) / 2)), 0, stream, res, delta,
                      gamma, n, eps, res_out, x_out, q, s);
}

// ---------------------------------------------------------------------------
// Weighted sum over a token's experts: four columns per thread, choices in order.  Bound
// by memory: 4096 x 5120, top 8: 104 us, 6.8 TB/s.
// ---------------------------------------------------------------------------
template <bool OB>
__global__ void __launch_bounds__(256) combine_kernel(const float *y, const int *pos, const float *weights,
                                                      int64_t quads, int topk, int slots, int n,
                                                      void *__restrict__ out) {
    pdl_launch_dependents();
    pdl_wait();
    const int per_row = n / 4;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < quads;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t t = i / per_row;
        const int c = static_cast<int>(i - t * per_row) * 4;
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int j = 0; j < topk; ++j) {
            const int p = pos[t * topk + j];
            if (p < 0 || p >= slots) continue;
            const float w = weights[t * topk + j];
            const float4 v = *reinterpret_cast<const float4 *>(y + static_cast<int64_t>(p) * n + c);
            acc[0] = __fmaf_rn(w, v.x, acc[0]);
            acc[1] = __fmaf_rn(w, v.y, acc[1]);
            acc[2] = __fmaf_rn(w, v.z, acc[2]);
            acc[3] = __fmaf_rn(w, v.w, acc[3]);
        }
        if (OB)
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + t * n + c) =
                make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
        else
            *reinterpret_cast<float4 *>(static_cast<float *>(out) + t * n + c) =
                make_float4(acc[0], acc[1], acc[2], acc[3]);
    }
}

}  // namespace

cudaError_t moe_norm_launch(const void *res, bool res_bf16, const void *delta, bool delta_bf16, const uint16_t *gamma,
                            int m, int n, float eps, void *res_out, uint16_t *x_out, int8_t *q, float *s,
                            cudaStream_t stream) {
    if (res_bf16)
        return delta_bf16 ? norm_launch<true, true>(res, delta, gamma, m, n, eps, res_out, x_out, q, s, stream)
                          : norm_launch<true, false>(res, delta, gamma, m, n, eps, res_out, x_out, q, s, stream);
    return delta_bf16 ? norm_launch<false, true>(res, delta, gamma, m, n, eps, res_out, x_out, q, s, stream)
                      : norm_launch<false, false>(res, delta, gamma, m, n, eps, res_out, x_out, q, s, stream);
}

cudaError_t moe_rotq_launch(const uint16_t *x, int64_t blocks, int8_t *q, float *s, cudaStream_t stream) {
    return launch_pdl(rotq_kernel, dim3(static_cast<unsigned>((blocks + 31) / 32)), dim3(256), 0, stream, x, blocks, q, s);
}

cudaError_t moe_combine_launch(const float *y, const int *pos, const float *weights, int m, int topk, int slots, int n,
                               void *out, bool out_bf16, cudaStream_t stream) {
    const int64_t quads = static_cast<int64_t>(m) * (n / 4);
    const int64_t want = (quads + 255) / 256;
    const unsigned grid = static_cast<unsigned>(want < (1 << 20) ? want : (1 << 20));
    return out_bf16 ? launch_pdl(combine_kernel<true>, dim3(grid), dim3(256), 0, stream, y, pos, weights, quads, topk,
                                 slots, n, out)
                    : launch_pdl(combine_kernel<false>, dim3(grid), dim3(256), 0, stream, y, pos, weights, quads, topk,
                                 slots, n, out);
}

}  // namespace tq
