// tq_moe_codes.cuh -- codes to e4m3, for the grouped products: int8 activations as two
// exact e4m3 numbers, and the order in which decoded weights meet them.
#pragma once

#include "tq_device.cuh"

namespace tq {

// 32 consecutive codes (8 words) in the order in which the decoded weights meet
// them (tq_dp4a.cuh, staged_pos).
template <int FMT>
__device__ __forceinline__ void stage_order(const uint32_t (&w)[8], uint32_t (&o)[8]) {
    if (FMT == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            o[4 * h + 0] = prmt(w[4 * h], w[4 * h + 1], 0x6420u);
            o[4 * h + 1] = prmt(w[4 * h + 2], w[4 * h + 3], 0x6420u);
            o[4 * h + 2] = prmt(w[4 * h], w[4 * h + 1], 0x7531u);
            o[4 * h + 3] = prmt(w[4 * h + 2], w[4 * h + 3], 0x7531u);
        }
    } else {
        // o[s] byte k = element 8k + s = byte s & 3 of word 2k + (s >> 2)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t a = prmt(w[h], w[2 + h], 0x5140u), b = prmt(w[4 + h], w[6 + h], 0x5140u);
            const uint32_t c = prmt(w[h], w[2 + h], 0x7362u), d = prmt(w[4 + h], w[6 + h], 0x7362u);
            o[4 * h + 0] = prmt(a, b, 0x5410u);
            o[4 * h + 1] = prmt(a, b, 0x7632u);
            o[4 * h + 2] = prmt(c, d, 0x5410u);
            o[4 * h + 3] = prmt(c, d, 0x7632u);
        }
    }
}

// Four int8 codes -> the e4m3 numbers 16 H and L themselves, |q| = 16 H + L, H in 0 .. 8, L in
// 0 .. 15, both with q's sign.
__device__ __forceinline__ void split4_whole(uint32_t w, uint32_t &hi, uint32_t &lo) {
    const uint32_t sign = w & 0x80808080u;
    const uint32_t mask = prmt(w, w, 0xba98u);
    const uint32_t a = (w ^ mask) + (mask & 0x01010101u);
    uint32_t sel = (a >> 4) & 0x07070707u;
    sel = (sel | (sel >> 4)) & 0x00ff00ffu;
    sel = sel | (sel >> 8);
    const uint32_t full = a & 0x80808080u;                      // -128: 0x70 is 128 (0x80 - 0x10)
    hi = prmt(0x64605800u, 0x6e6c6a68u, sel) | (full - (full >> 3)) | sign;  // 0, 16, 32, 48 | 64, 80, 96, 112
    uint32_t low = a & 0x07070707u;
    low = (low | (low >> 4)) & 0x00ff00ffu;
    low = low | (low >> 8);
    const uint32_t small = prmt(0x44403800u, 0x4e4c4a48u, low); // 0 .. 7
    const uint32_t large = (a & 0x07070707u) | 0x50505050u;     // 8 .. 15: one binade, linear
    const uint32_t pick = prmt((a & 0x08080808u) << 4, 0u, 0xba98u);
    lo = ((small & ~pick) | (large & pick)) | sign;
}

// Half (s = 0, 1) of one row's 128 weights (32 or 16 bytes of codes) -> 16 registers of
// four e4m3 numbers -1, 0, +1 each, in staged order.
template <int FMT>
__device__ __forceinline__ void decode_half(const uint4 *c, int s, uint32_t (&v)[16]) {
    if (FMT == 0) {
        constexpr uint32_t kTable = 0x00b83800u;                // codes 0, 1, 2 -> 0, +1, -1
        const uint32_t w[4] = {c[s].x, c[s].y, c[s].z, c[s].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t even = w[i] & 0x33333333u, odd = (w[i] >> 2) & 0x33333333u;
            v[4 * i + 0] = prmt(kTable, 0u, even);
            v[4 * i + 1] = prmt(kTable, 0u, even >> 16);
            v[4 * i + 2] = prmt(kTable, 0u, odd);
            v[4 * i + 3] = prmt(kTable, 0u, odd >> 16);
        }
    } else {
        const uint32_t w[2] = {s == 0 ? c[0].x : c[0].z, s == 0 ? c[0].y : c[0].w};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int b = 0; b < 8; ++b) v[8 * i + b] = ((w[i] << (7 - b)) & 0x80808080u) ^ 0xb8b8b8b8u;
    }
}

// Two fp32 lanes per instruction, each rounded to nearest.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ uint64_t pack2(uint32_t both) { return pack2(__uint_as_float(both), __uint_as_float(both)); }
__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t neg2(uint64_t a) { return a ^ 0x8000000080000000ull; }

// SiLU of N (even) gates, g / (1 + exp(-g)), the division correctly rounded.  For
// 2^-80 <= |g| < 64 without a branch and two at a time: tq_expf's polynomial
// with 2^n put in at once (2^n is a normal number there), a reciprocal refined by one
// Newton step, and the quotient corrected with its exact remainder (P. Markstein,
// "IA-64 and Elementary Functions", 2000, chapter 8).  Other arguments take tq_silu.
// The bits are tq_silu's for every g (compared over all 2^32).
template <int N>
__device__ __forceinline__ void moe_silu(const float (&g)[N], float (&s)[N]) {
    uint32_t far = 0;                               // |g|'s distance above 2^-80, as bits
#pragma unroll
    for (int i = 0; i < N; i += 2) {
#pragma unroll
        for (int j = 0; j < 2; ++j) far = max(far, (__float_as_uint(g[i + j]) & 0x7fffffffu) - 0x17800000u);
        const uint64_t gg = pack2(g[i], g[i + 1]), z = neg2(gg);
        const uint64_t magic = pack2(0x4b400000u), minus = pack2(0xcb400000u);   // +-12582912
        // (a packed product here would be fused with the addition: the product is rounded by itself)
        const float log2e = __uint_as_float(0x3fb8aa3bu);
        const uint64_t t = add2(pack2(__fmul_rn(-g[i], log2e), __fmul_rn(-g[i + 1], log2e)), magic);
        const uint64_t n = neg2(add2(t, minus));
        uint64_t r = fma2(n, pack2(0x3f317000u), z);
        r = fma2(n, pack2(0x3805fdf4u), r);
        uint64_t p = fma2(pack2(0x39500d01u), r, pack2(0x3ab60b61u));            // 1/7!, 1/6!
        p = fma2(p, r, pack2(0x3c088889u));
        p = fma2(p, r, pack2(0x3d2aaaabu));
        p = fma2(p, r, pack2(0x3e2aaaabu));
        p = fma2(p, r, pack2(0x3f000000u));
        p = fma2(p, r, pack2(0x3f800000u));
        p = fma2(p, r, pack2(0x3f800000u));
        float p0, p1, t0, t1, d0, d1, y0, y1;
        unpack2(p, p0, p1);
        unpack2(t, t0, t1);
        const uint64_t d = add2(pack2(__int_as_float(__float_as_int(p0) + ((__float_as_int(t0) - 0x4b400000) << 23)),
                                      __int_as_float(__float_as_int(p1) + ((__float_as_int(t1) - 0x4b400000) << 23))),
                                pack2(0x3f800000u));
        unpack2(d, d0, d1);
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y0) : "f"(d0));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y1) : "f"(d1));
        uint64_t y = pack2(y0, y1);
        const uint64_t nd = neg2(d);
        y = fma2(fma2(nd, y, pack2(0x3f800000u)), y, y);
        const uint64_t q = mul2(gg, y);
        unpack2(fma2(fma2(nd, q, gg), y, q), s[i], s[i + 1]);
    }
    if (far >= 0x42800000u - 0x17800000u) {         // some |g| below 2^-80 (0, too) or at least 64
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = tq_silu(g[i]);
    }
}

}  // namespace tq
