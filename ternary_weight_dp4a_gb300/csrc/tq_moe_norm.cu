// tq_moe_norm.cu -- the ends of a mixture-of-experts layer: residual addition +
// RMS norm + rotation + int8 quantisation (tq_add_rmsnorm_rotq), and the
// weighted sum over a token's experts (tq_moe_combine).
#include <cuda_runtime.h>

#include "tq_device.cuh"
#include "tq_launch.h"
#include "tq_moe_internal.h"

namespace tq {
namespace {

// ---------------------------------------------------------------------------
// Residual addition, RMS norm, rotation, quantisation: one CTA per row, a warp
// takes blocks w, w + warps, .. and keeps their sums t in registers between
// the two passes (sum of squares; normalise, rotate, quantise), so the row is
// read once.  Lane l holds elements 4l .. 4l+3 of a block: 16-byte (fp32) or
// 8-byte (bf16) loads, the transform's spans 1 and 2 in registers and spans
// 4 .. 64 by shuffles.
// ---------------------------------------------------------------------------

// (hi, lo) += v as an unevaluated sum (T. J. Dekker, D. E. Knuth: two-sum).
__device__ __forceinline__ void pair_add(float &hi, float &lo, float v, float v_lo) {
    const float t = __fadd_rn(hi, v);
    const float b = __fsub_rn(t, hi);
    const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(v, b));
    hi = t;
    lo = __fadd_rn(lo, __fadd_rn(e, v_lo));
}

// (plain loads: the residual may be updated in place)
template <bool BF16>
__device__ __forceinline__ void load4(const void *p, int64_t i, float (&v)[4]) {
    if (BF16) {
        const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i);
        v[0] = __uint_as_float(w.x << 16);
        v[1] = __uint_as_float(w.x & 0xffff0000u);
        v[2] = __uint_as_float(w.y << 16);
        v[3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
        const float4 w = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
    }
}

__device__ __forceinline__ uint2 pack_bf16x4(const float (&v)[4]) {
    uint2 w;
    w.x = f32_to_bf16_bits(v[0]) | (static_cast<uint32_t>(f32_to_bf16_bits(v[1])) << 16);
    w.y = f32_to_bf16_bits(v[2]) | (static_cast<uint32_t>(f32_to_bf16_bits(v[3])) << 16);
    return w;
}

// The stages of tq_rotate_quant on elements 4 * lane .. 4 * lane + 3.
__device__ __forceinline__ void wht128_quad(float (&v)[4], int lane) {
    float a = v[0], b = v[1], c = v[2], d = v[3];
    v[0] = __fadd_rn(a, b); v[1] = __fsub_rn(a, b);
    v[2] = __fadd_rn(c, d); v[3] = __fsub_rn(c, d);
    a = v[0]; b = v[1]; c = v[2]; d = v[3];
    v[0] = __fadd_rn(a, c); v[2] = __fsub_rn(a, c);
    v[1] = __fadd_rn(b, d); v[3] = __fsub_rn(b, d);
#pragma unroll
    for (int h = 1; h < 32; h <<= 1) {
        const bool upper = (lane & h) != 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float o = __shfl_xor_sync(0xffffffffu, v[i], h);
            v[i] = upper ? __fsub_rn(o, v[i]) : __fadd_rn(v[i], o);
        }
    }
    const float c128 = __uint_as_float(0x3db504f3u);   // (float)(1/sqrt(128))
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __fmul_rn(v[i], c128);
}

template <bool RB, bool DB, int NBW>
__global__ void __launch_bounds__(1024) add_rmsnorm_rotq_kernel(const void *res, const void *delta,
                                                                const uint16_t *__restrict__ gamma, int n, float eps,
                                                                void *res_out, uint16_t *__restrict__ x_out,
                                                                int8_t *__restrict__ q, float *__restrict__ s) {
    __shared__ float2 warp_sum[32];
    __shared__ double warp_sum64[32];
    __shared__ float inv_smem;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int nb = n / kBlock;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * n;
    float t[NBW][4];
    float hi = 0.0f, lo = 0.0f;
#pragma unroll
    for (int j = 0; j < NBW; ++j) {
        const int b = warp + j * warps;
#pragma unroll
        for (int i = 0; i < 4; ++i) t[j][i] = 0.0f;
        if (b >= nb) continue;
        const int64_t at = row + b * kBlock + 4 * lane;
        load4<RB>(res, at, t[j]);
        if (delta != nullptr) {
            float d[4];
            load4<DB>(delta, at, d);
#pragma unroll
            for (int i = 0; i < 4; ++i) t[j][i] = __fadd_rn(t[j][i], d[i]);
        }
        if (RB) {
            const uint2 w = pack_bf16x4(t[j]);
            if (res_out != nullptr) *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(res_out) + at) = w;
            t[j][0] = __uint_as_float(w.x << 16);
            t[j][1] = __uint_as_float(w.x & 0xffff0000u);
            t[j][2] = __uint_as_float(w.y << 16);
            t[j][3] = __uint_as_float(w.y & 0xffff0000u);
        } else if (res_out != nullptr) {
            *reinterpret_cast<float4 *>(static_cast<float *>(res_out) + at) = make_float4(t[j][0], t[j][1], t[j][2], t[j][3]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float p = __fmul_rn(t[j][i], t[j][i]);
            pair_add(hi, lo, p, __fmaf_rn(t[j][i], t[j][i], -p));
        }
    }
    if (q == nullptr && x_out == nullptr) return;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        pair_add(hi, lo, __shfl_xor_sync(0xffffffffu, hi, o), __shfl_xor_sync(0xffffffffu, lo, o));
    if (lane == 0) warp_sum[warp] = make_float2(hi, lo);
    __syncthreads();
    {
        const float2 w = lane < warps ? warp_sum[lane] : make_float2(0.0f, 0.0f);
        hi = w.x;
        lo = w.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            pair_add(hi, lo, __shfl_xor_sync(0xffffffffu, hi, o), __shfl_xor_sync(0xffffffffu, lo, o));
    }
    double sum = static_cast<double>(hi) + static_cast<double>(lo);
    // squares beyond binary32's range (or all tiny): the same sum in 64 bits
    if (!(hi > 1e-25f && hi < 1e37f)) {
        double acc = 0.0;
#pragma unroll
        for (int j = 0; j < NBW; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc = fma(static_cast<double>(t[j][i]), static_cast<double>(t[j][i]), acc);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
        if (lane == 0) warp_sum64[warp] = acc;
        __syncthreads();
        sum = 0.0;
        for (int w = 0; w < warps; ++w) sum += warp_sum64[w];
    }
    if (threadIdx.x == 0) inv_smem = static_cast<float>(1.0 / sqrt(sum / n + static_cast<double>(eps)));
    __syncthreads();
    const float inv = inv_smem;
#pragma unroll
    for (int j = 0; j < NBW; ++j) {
        const int b = warp + j * warps;
        if (b >= nb) continue;
        const int col = b * kBlock + 4 * lane;
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __fmul_rn(t[j][i], inv);
        if (gamma != nullptr) {
            float g[4];
            load4<true>(gamma, col, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __fmul_rn(v[i], g[i]);
        }
        const uint2 xb = pack_bf16x4(v);
        if (x_out != nullptr) *reinterpret_cast<uint2 *>(x_out + row + col) = xb;
        if (q == nullptr) continue;
        v[0] = __uint_as_float(xb.x << 16);
        v[1] = __uint_as_float(xb.x & 0xffff0000u);
        v[2] = __uint_as_float(xb.y << 16);
        v[3] = __uint_as_float(xb.y & 0xffff0000u);
        wht128_quad(v, lane);
        float top = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float sc = top == 0.0f ? 0.0f : __fdiv_rn(top, 127.0f);
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            int c = sc == 0.0f ? 0 : __float2int_rn(__fdiv_rn(v[i], sc));
            c = c > 127 ? 127 : (c < -127 ? -127 : c);
            word |= static_cast<uint32_t>(c & 255) << (8 * i);
        }
        *reinterpret_cast<uint32_t *>(q + row + col) = word;
        if (lane == 0) s[static_cast<int64_t>(blockIdx.x) * nb + b] = sc;
    }
}

template <bool RB, bool DB>
cudaError_t norm_launch(const void *res, const void *delta, const uint16_t *gamma, int m, int n, float eps,
                        void *res_out, uint16_t *x_out, int8_t *q, float *s, cudaStream_t stream) {
    const int nb = n / kBlock;
    // enough warps that a warp holds at most 8 blocks of the row in registers (n <= 32768)
    int warps = nb < 4 ? nb : 4;
    while (warps < 32 && warps * 8 < nb) warps *= 2;
    const int per = (nb + warps - 1) / warps;
#define TQ_NORM(NBW)                                                                                                  \
    return launch_pdl(add_rmsnorm_rotq_kernel<RB, DB, NBW>, dim3(m), dim3(32 * warps), 0, stream, res, delta, gamma, n, \
                      eps, res_out, x_out, q, s)
    if (per <= 1) TQ_NORM(1);
    if (per <= 2) TQ_NORM(2);
    if (per <= 4) TQ_NORM(4);
    TQ_NORM(8);
#undef TQ_NORM
}

// ---------------------------------------------------------------------------
// Weighted sum over a token's experts: four columns per thread, choices in order.
// ---------------------------------------------------------------------------
template <bool OB>
__global__ void __launch_bounds__(256) combine_kernel(const float *__restrict__ y, const int *__restrict__ pos,
                                                      const float *__restrict__ weights, int64_t quads, int topk,
                                                      int slots, int n, void *out) {
    pdl_launch_dependents();
    pdl_wait();
    const int per_row = n / 4;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < quads;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t t = i / per_row;
        const int c = static_cast<int>(i - t * per_row) * 4;
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int j = 0; j < topk; ++j) {
            const int p = __ldg(pos + t * topk + j);
            if (p < 0 || p >= slots) continue;
            const float w = __ldg(weights + t * topk + j);
            const float4 v = __ldg(reinterpret_cast<const float4 *>(y + static_cast<int64_t>(p) * n + c));
            acc[0] = __fmaf_rn(w, v.x, acc[0]);
            acc[1] = __fmaf_rn(w, v.y, acc[1]);
            acc[2] = __fmaf_rn(w, v.z, acc[2]);
            acc[3] = __fmaf_rn(w, v.w, acc[3]);
        }
        if (OB)
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + t * n + c) = pack_bf16x4(acc);
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
