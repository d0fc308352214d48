// tq_q4_tile.cu -- products with 4-bit weights for many rows, on the 5th-generation tensor core.
//
// A tile is up to 128 rows of x (the A operand: 64 values of k per stage by TMA, 128-byte swizzle)
// by 256 weight rows (the B operand: decoded from their codes to bf16 c - 8, which is exact, into
// shared memory); gate/up: 128 rows of each.  A group's products add up in one of two accumulators in
// tensor memory; the fold reads it back and multiplies by the scales in fp32,
//   acc = fma(s, d, acc)   [acc = fma(8 s - b, sum of x, acc)],
// while the tensor core works on the next group.  With minima 16 of the 256 rows of B are ones, so the sum of x
// over the group comes out beside the products.
//
// Why the weights are B: an MMA of M = 128 costs about the same for every N (150 cycles for K = 16 here), so
// 256 weight rows per MMA are twice as many weights per cycle as 128, and that is what bounds calls
// of up to 128 rows.
//
// Rows of x are dealt to the four quarters of tensor memory alike, since a warp reads only its
// own quarter.  Few tiles are split along k over the CTAs of a cluster, which add up their parts through shared
// memory.
//
// Warps: 0-3 decode, 4 issues MMAs, 5 copies x, 8-15 fold (a quarter of the lanes and half of the columns each).
#include <cuda_runtime.h>

#include <type_traits>

#include "tq_device.cuh"
#include "tq_moe_internal.h"
#include "tq_q4_internal.h"
#include "tq_tcgen05.cuh"
#include "tq_tmap.h"

namespace tq {
namespace {

constexpr int kRows = 128;                      // of x, per tile
constexpr int kCols = 256;                      // rows of B
constexpr int kStageK = 64;
constexpr int kStages = 4;
// Groups whose scales are kept.  The decode of stage s + 4 knows that the MMAs of stage s are done, hence the
// fold of all groups but the last two of them: 4, 6 and 10 groups can be between the two.
template <int GROUP>
constexpr int scale_groups() { return GROUP == 128 ? 4 : GROUP == 64 ? 6 : 10; }
constexpr int kFoldWarps = 8;
constexpr int kThreads = 256 + 32 * kFoldWarps;
constexpr uint32_t kABytes = kRows * kStageK * 2;
// B, no swizzle: core matrices of 8 rows x 8 values (128 bytes), those of 8 further rows behind
// it, those of the next 8 values kLbo on; 32 bytes more than the rows take, so that the four lanes that decode
// a row's words of one chunk store to different banks.
constexpr uint32_t kLbo = kCols / 8 * 128 + 32;
constexpr uint32_t kBBytes = kStageK / 8 * kLbo;
constexpr int kAhead = 8;                       // chunks of codes in L2 ahead of the decode
constexpr int kPartLd = kCols + 4;              // floats per row of a part in shared memory

// register shares (launched with 128 per thread): 128 x (120 + 40 + 2 x 176) = 512 x 128
constexpr int kRegsDecode = 120, kRegsIssue = 40, kRegsFold = 176;

__device__ unsigned lost_waits;                 // bits of all waits that have run out on this device

struct __align__(1024) TileSmem {
    union {
        struct {
            uint8_t a[kStages][kABytes];
            uint8_t b[kStages][kBBytes];
        };
        float part[kRows][kPartLd];             // this CTA's sums, when a tile is split along k
    };
    // per group: the scales, each twice (the operand of a packed multiply-add), and 8 s - b; in fold
    // order, columns c, c + 4, c + 8, c + 12 of 16 side by side
    uint8_t scales[scale_groups<32>() * kCols * 12];
    uint64_t a_full[kStages], b_full[kStages], empty[kStages], s_full[scale_groups<32>()], d_full[2], d_empty[2], drain;
    uint32_t tmem;
    uint32_t dead;                              // a bounded wait ran out
};

struct TileArgs {
    Q4Product p;
    CUtensorMap x;                              // [m][k] bf16, boxes of 32 rows x 64 values
    int row_tiles, rows;                        // rows of x per tile
    int split;                                  // CTAs along k
};

constexpr uint32_t idesc_bf16(int m, int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void mma_bf16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {
    // K-major, 128-byte swizzle: atoms of 8 rows x 128 bytes, 1024 bytes apart
    uint64_t d = static_cast<uint64_t>((saddr & 0x3ffffu) >> 4);
    d |= 1ull << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= 1ull << 46;
    d |= 2ull << 61;
    return d;
}

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

template <int R>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// 16 lanes x 16 columns in the 16x128b shape: register 2 n + j is row 8 j + lane / 4, column 4 n + lane % 4.
__device__ __forceinline__ void ld_half(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x128b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

// tcgen05.wait::ld; the registers pass through it, so nothing reads them before.
__device__ __forceinline__ void wait_ld(uint32_t (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ uint64_t pack2(uint32_t a, uint32_t b) { return static_cast<uint64_t>(b) << 32 | a; }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ float half2of(uint64_t v, int j) { return __uint_as_float(static_cast<uint32_t>(j ? v >> 32 : v)); }

// A bounded wait.  One that runs out sets `dead` and the error word; every later
// wait of the CTA then gives up at once, so that all roles come to their end.
template <int SLEEP>
__device__ __forceinline__ void wait_slow(TileSmem &sm, uint32_t bar, uint32_t parity, unsigned bit) {
    const long long t0 = clock64();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i) {
            if (mbar_try_wait(bar, parity)) return;
            if (SLEEP > 0) __nanosleep(SLEEP);
        }
        if (*reinterpret_cast<volatile uint32_t *>(&sm.dead)) return;
        if (clock64() - t0 > kWaitBudgetCycles) {
            *reinterpret_cast<volatile uint32_t *>(&sm.dead) = 1;
            atomicOr(&lost_waits, bit);
            return;
        }
    }
}
// Waits, and says whether the CTA is still alive (one answer for the whole warp).
template <int SLEEP = 0>
__device__ __forceinline__ bool warp_wait(TileSmem &sm, uint32_t bar, uint32_t parity, unsigned bit) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        wait_slow<SLEEP>(sm, bar, parity, bit);
        ok = *reinterpret_cast<volatile uint32_t *>(&sm.dead) == 0;
    }
    return __all_sync(0xffffffffu, ok);
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

// Pair i of a word's codes as bf16 c - 8: (w >> 4 i) & mask | 128, minus 136.
__device__ __forceinline__ uint32_t decode_pair(uint32_t w, int i, uint32_t mask, uint32_t base) {
    uint32_t v, d;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(v) : "r"(w >> (4 * i)), "r"(mask), "r"(base));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(0x43084308u));
    return d;
}

__device__ __forceinline__ void prefetch_l2(const void *p, int bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t at, float a, float b) {
    asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(at), "f"(a), "f"(b) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t at, float a) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(a) : "memory"); }
__device__ __forceinline__ void lds128(uint32_t at, uint64_t &a, uint64_t &b) {
    asm volatile("ld.shared.v2.b64 {%0,%1}, [%2];" : "=l"(a), "=l"(b) : "r"(at) : "memory");
}

template <int GROUP, bool MINS, bool GATEUP>
__global__ void __launch_bounds__(kThreads, 1) q4_tile_kernel(const __grid_constant__ TileArgs args) {
    extern __shared__ uint8_t smem_raw[];
    TileSmem &sm = *reinterpret_cast<TileSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const Q4Product &p = args.p;
    constexpr int kPer = 128 / GROUP;                               // groups per chunk
    constexpr int kKept = scale_groups<GROUP>();
    // strips of 16 weight rows per tile and matrix; the ones behind them where there are minima
    constexpr int kStrips = GATEUP ? (MINS ? 7 : 8) : (MINS ? 15 : 16);
    constexpr int kUsed = GATEUP ? 2 * kStrips : kStrips;
    constexpr int kN = (kUsed + MINS) * 16;                         // columns of D
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (warp == 4) {
        tmem_alloc(smem_u32(&sm.tmem), 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&sm.a_full[i]), 1);
            mbar_init(smem_u32(&sm.b_full[i]), 4);
            mbar_init(smem_u32(&sm.empty[i]), 1);
        }
        for (int i = 0; i < scale_groups<32>(); ++i) mbar_init(smem_u32(&sm.s_full[i]), 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sm.d_full[i]), 1);
            mbar_init(smem_u32(&sm.d_empty[i]), kFoldWarps);
        }
        mbar_init(smem_u32(&sm.drain), 1);
        sm.dead = 0;
        mbar_init_fence();
    }
    if (MINS)
        for (int i = tid; i < kStages * (kStageK / 8) * 16; i += kThreads) {
            const int row = i & 15, oct = (i >> 4) % (kStageK / 8), st = (i >> 4) / (kStageK / 8);
            sts128(smem_u32(sm.b[st]) + oct * kLbo + (kUsed * 2 + row / 8) * 128 + row % 8 * 16, 0x3f803f80u, 0x3f803f80u,
                   0x3f803f80u, 0x3f803f80u);
        }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    const int chunks = p.k >> 7;
    const int rank = blockIdx.x % args.split, tile = blockIdx.x / args.split;
    const int row0 = tile % args.row_tiles * args.rows, ntile = tile / args.row_tiles;
    const int rows = min(args.rows, p.m - row0);
    const int quarter_rows = ((rows + 3) / 4 + 7) / 8 * 8;          // rows of x in a quarter of the lanes
    const int chunk0 = rank * chunks / args.split, chunk1 = (rank + 1) * chunks / args.split;
    const int stages = 2 * (chunk1 - chunk0), groups = (chunk1 - chunk0) * kPer;

    // Packed codes come to L2 well ahead of the decode's loads, which have one chunk in flight: lanes 0-3 of a
    // decode warp ask for its four strips'.
    const int my_slot = warp * 4 + lane, my_mat = GATEUP && my_slot >= kStrips;
    const int64_t my_strip = static_cast<int64_t>(ntile) * kStrips + my_slot - my_mat * kStrips;
    const bool asks = warp < 4 && lane < 4 && my_slot < kUsed && my_strip < q4_strips(p.n);
    auto ask = [&](int from, int to) {
        to = min(to, chunk1 - chunk0);
        if (asks && from < to)
            prefetch_l2(p.codes[my_mat] + (my_strip * chunks + chunk0 + from) * kQ4ChunkBytes, (to - from) * kQ4ChunkBytes);
    };
    ask(0, kAhead);
    pdl_launch_dependents();
    pdl_wait();

    if (warp < 4) {
        // ---- decode: a warp has four strips, a lane one row's 16 bytes of each half strip ----
        regs_down<kRegsDecode>();
        const int64_t strips = q4_strips(p.n);
        const uint8_t *src[4];
        bool have[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int slot = warp * 4 + i, mat = GATEUP ? slot / kStrips : 0;
            const int64_t strip = static_cast<int64_t>(ntile) * kStrips + (GATEUP ? slot % kStrips : slot);
            have[i] = slot < kUsed && strip < strips;
            src[i] = p.codes[have[i] ? mat : 0] + ((have[i] ? strip : 0) * chunks + chunk0) * kQ4ChunkBytes + lane * 16;
        }
        // scales: a thread has rows r and r + 8 of one strip
        const int sslot = tid >> 3, smat = GATEUP ? min(sslot / kStrips, 1) : 0;
        const int64_t sstrip = static_cast<int64_t>(ntile) * kStrips + (GATEUP ? sslot - smat * kStrips : sslot);
        const bool shave = sslot < kUsed && sstrip < strips;
        const int64_t sat = (((shave ? sstrip : 0) * chunks + chunk0) * 8 + (tid & 7)) * (2 * kPer);
        const uint16_t *ssrc = p.scales[smat] + sat, *msrc = MINS ? p.mins[smat] + sat : nullptr;
        // place of rows r and r + 8 in fold order: columns c, c + 4, c + 8, c + 12 of 16 side by side
        const int place = 16 * sslot + 4 * (tid & 3) + ((tid >> 2) & 1);    // r + 8: two places on
        uint4 code[2][8];
        uint16_t sc[2][2 * kPer], mn[2][MINS ? 2 * kPer : 1];
        auto load = [&](int buf, int c) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                code[buf][i] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
                if (have[i >> 1]) {
                    const uint8_t *at = src[i >> 1] + static_cast<int64_t>(c) * kQ4ChunkBytes + (i & 1) * 512;
                    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(code[buf][i].x), "=r"(code[buf][i].y), "=r"(code[buf][i].z), "=r"(code[buf][i].w)
                                 : "l"(at));
                }
            }
#pragma unroll
            for (int i = 0; i < 2 * kPer; ++i) {
                sc[buf][i] = 0;
                if (MINS) mn[buf][i] = 0;
                if (shave) {
                    sc[buf][i] = *reinterpret_cast<const volatile uint16_t *>(ssrc + static_cast<int64_t>(c) * (16 * kPer) + i);
                    if (MINS) mn[buf][i] = *reinterpret_cast<const volatile uint16_t *>(msrc + static_cast<int64_t>(c) * (16 * kPer) + i);
                }
            }
        };
        const int total = chunk1 - chunk0;
        const uint32_t codes_at = smem_u32(sm.b[0]) + warp * 8 * 128 + (lane >> 2) * 16 + (lane & 3) * kLbo;
        const uint32_t scales_at = smem_u32(sm.scales), bars = smem_u32(sm.b_full);
        uint32_t mask = 0x000f000fu, base = 0x43004300u;
        asm volatile("" : "+r"(mask), "+r"(base));                  // in registers: two constants do not fit one instruction
        load(0, 0);
        bool ok = true;
        for (int c0 = 0; c0 < total && ok; c0 += 2) {
#pragma unroll
            for (int buf = 0; buf < 2; ++buf) {
                const int c = c0 + buf;
                if (c >= total || !ok) break;
                if (c + 1 < total) load(buf ^ 1, c + 1);
                if (c % 4 == 0) ask(c + kAhead, c + kAhead + 4);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int st = 2 * c + half, ring = st % kStages;
                    ok = warp_wait<32>(sm, smem_u32(&sm.empty[ring]), ((st / kStages) & 1) ^ 1, 1u << 0);
                    if (!ok) break;
                    if (GROUP < 128 || half == 0) {
                        constexpr int kHere = GROUP == 32 ? 2 : 1;
#pragma unroll
                        for (int g = 0; g < kHere; ++g) {
                            const int e = GROUP == 128 ? 0 : half * kHere + g;
                            const int slot = (c * kPer + e) % kKept;
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const float s = f16_bits_to_f32(sc[buf][r * kPer + e]);
                                sts64(scales_at + (slot * kCols + place + 2 * r) * 8, s, s);
                                if (MINS)
                                    sts32(scales_at + kKept * kCols * 8 + (slot * kCols + place + 2 * r) * 4,
                                          __fmaf_rn(8.0f, s, -f16_bits_to_f32(mn[buf][r * kPer + e])));
                            }
                            __syncwarp();
                            if (lane == 0) mbar_arrive(smem_u32(&sm.s_full[slot]));
                        }
                    }
                    const uint32_t dst = codes_at + ring * kBBytes;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (kUsed < 16 && warp * 4 + (i >> 1) >= kUsed) continue;
                        const uint32_t w[2] = {half ? code[buf][i].z : code[buf][i].x, half ? code[buf][i].w : code[buf][i].y};
#pragma unroll
                        for (int g = 0; g < 2; ++g)
                            sts128(dst + i * 128 + 4 * g * kLbo, decode_pair(w[g], 0, mask, base), decode_pair(w[g], 1, mask, base),
                                   decode_pair(w[g], 2, mask, base), decode_pair(w[g], 3, mask, base));
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bars + ring * 8);
                }
            }
        }
    } else if (warp < 8) {
        regs_down<kRegsIssue>();
        if (warp == 4) {
            // ---- issue ----
            constexpr uint32_t idesc = idesc_bf16(kRows, kN);
            int group = 0;
            for (int st = 0; st < stages; ++st) {
                const int ring = st % kStages;
                bool ok = warp_wait(sm, smem_u32(&sm.a_full[ring]), (st / kStages) & 1, 1u << 1) &&
                          warp_wait(sm, smem_u32(&sm.b_full[ring]), (st / kStages) & 1, 1u << 2);
                constexpr int kSubs = GROUP == 32 ? 2 : 1;
#pragma unroll
                for (int sub = 0; sub < kSubs && ok; ++sub) {
                    const bool start = GROUP < 128 || (st & 1) == 0, end = GROUP < 128 || (st & 1) == 1;
                    if (start) ok = warp_wait(sm, smem_u32(&sm.d_empty[group & 1]), ((group >> 1) & 1) ^ 1, 1u << 3);
                    if (!ok) break;
                    if (lane == 0) {
                        tc_fence_after();
                        const uint32_t d = tmem + (group & 1) * kCols;
                        const uint64_t a = desc_sw128(smem_u32(sm.a[ring]));
                        const uint64_t b = smem_desc_kmajor(smem_u32(sm.b[ring]), kLbo, 128);
#pragma unroll
                        for (int i = sub * (4 / kSubs); i < (sub + 1) * (4 / kSubs); ++i)
                            mma_bf16_ss(d, a + 2 * i, b + i * (2 * kLbo >> 4), idesc, !(start && i == sub * (4 / kSubs)));
                        if (end) tc_commit(smem_u32(&sm.d_full[group & 1]));
                    }
                    __syncwarp();
                    if (end) ++group;
                }
                if (!ok) break;
                if (lane == 0) tc_commit(smem_u32(&sm.empty[ring]));
                __syncwarp();
            }
            if (lane == 0) {
                tc_commit(smem_u32(&sm.drain));
                if (!mbar_wait(smem_u32(&sm.drain), 0)) atomicOr(&lost_waits, 1u << 4);
            }
        } else if (warp == 5) {
            // ---- copies of x: 32 rows for each quarter, whatever it has of them ----
            int st = 0;
            for (; st < stages; ++st) {
                const int ring = st % kStages;
                if (!warp_wait<32>(sm, smem_u32(&sm.empty[ring]), ((st / kStages) & 1) ^ 1, 1u << 5)) break;
                const uint32_t bar = smem_u32(&sm.a_full[ring]);
                if (lane == 0) mbar_arrive_expect_tx(bar, kABytes);
                __syncwarp();
                if (lane < 4)
                    load_box(smem_u32(sm.a[ring]) + lane * (kABytes / 4), &args.x, chunk0 * 128 + st * kStageK,
                             row0 + lane * quarter_rows, bar);
            }
            // none of this CTA's copies may be in flight when it leaves
            for (int j = max(st - kStages, 0); j < st; ++j)
                if (!mbar_wait(smem_u32(&sm.a_full[j % kStages]), (j / kStages) & 1)) atomicOr(&lost_waits, 1u << 6);
        }
        __syncwarp();
    } else {
        // ---- fold: a lane has rows i, i + 8, i + 16, i + 24 of its quarter and every fourth column from t on ----
        regs_up<kRegsFold>();
        const int quarter = warp & 3, part = (warp - 8) >> 2, i = lane >> 2, t = lane & 3;
        // chunk e (16 columns) of this warp: 8 of 16; gate/up: four of each matrix
        auto column = [&](int e) { return GATEUP ? (e >> 2) * kStrips + 4 * part + (e & 3) : 8 * part + e; };
        auto active = [&](int e) { return GATEUP ? 4 * part + (e & 3) < kStrips : 8 * part + e < kStrips; };
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        uint64_t acc[8][4][2];                                      // [chunk][column 4 n + t][rows 16 h + i and + 8]
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int n = 0; n < 4; ++n) acc[e][n][0] = acc[e][n][1] = 0;
        const uint32_t s_at = smem_u32(sm.scales) + (column(0) * 16 + 4 * t) * 8;
        const uint32_t m_at = smem_u32(sm.scales) + kKept * kCols * 8 + (column(0) * 16 + 4 * t) * 4;
        // WIDE: a quarter has more than 16 rows
        auto fold = [&](auto wide) {
            constexpr int kHalves = decltype(wide)::value ? 2 : 1;
            int slot = 0;
            uint32_t turn = 0;
#pragma unroll 1
            for (int group = 0; group < groups; ++group) {
                if (!(warp_wait(sm, smem_u32(&sm.s_full[slot]), turn, 1u << 7) &&
                      warp_wait(sm, smem_u32(&sm.d_full[group & 1]), (group >> 1) & 1, 1u << 8)))
                    break;
                tc_fence_after();
                const uint32_t d = lane_base + (group & 1) * kCols;
                uint64_t sums[kHalves];
                if (MINS) {
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) {
                        uint32_t x[8];
                        ld_half(d + kUsed * 16 + ((16u * h) << 16), x);
                        wait_ld(x);
                        sums[h] = pack2(x[0], x[1]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (kStrips % 8 != 0 && !active(e)) continue;
                    uint32_t x[kHalves][8];
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) ld_half(d + column(e) * 16 + ((16u * h) << 16), x[h]);
                    const uint32_t off = slot * kCols + (column(e) - column(0)) * 16;
                    uint64_t s2[4];
                    lds128(s_at + off * 8, s2[0], s2[1]);
                    lds128(s_at + off * 8 + 16, s2[2], s2[3]);
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) wait_ld(x[h]);
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int h = 0; h < kHalves; ++h)
                            acc[e][n][h] = fma2(pack2(x[h][2 * n], x[h][2 * n + 1]), s2[n], acc[e][n][h]);
                    if (MINS) {
                        uint64_t m01, m23;
                        lds128(m_at + off * 4, m01, m23);
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            const float m = half2of(n < 2 ? m01 : m23, n & 1);
                            const uint64_t m2 = pack2(m, m);
#pragma unroll
                            for (int h = 0; h < kHalves; ++h) acc[e][n][h] = fma2(sums[h], m2, acc[e][n][h]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.d_empty[group & 1]));
                if (++slot == kKept) {
                    slot = 0;
                    turn ^= 1;
                }
            }
        };
        if (quarter_rows > 16) fold(std::true_type{});
        else fold(std::false_type{});
        if (args.split > 1) {
            // (every copy and MMA of this CTA has ended: its stages hold the parts now)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (active(e))
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                sm.part[32 * quarter + 16 * h + 8 * j + i][column(e) * 16 + 4 * n + t] = half2of(acc[e][n][h], j);
            cluster_sync();
            constexpr int kOut = kStrips * 16;
            const int c0 = rank * kOut / args.split, width = (rank + 1) * kOut / args.split - c0;
            const uint32_t base = smem_u32(sm.part);
            for (int o = tid - 256; o < rows * width; o += 32 * kFoldWarps) {
                const int r = o / width, c = c0 + o - r * width;
                const int64_t out = static_cast<int64_t>(ntile) * kOut + c;
                if (out >= p.n) continue;
                const int q = r / quarter_rows;
                const uint32_t at = base + static_cast<uint32_t>((32 * q + r - q * quarter_rows) * kPartLd + c) * 4;
                float v = 0.0f, u = 0.0f;
                for (int s = 0; s < args.split; ++s) {
                    v += ld_cluster_f32(at, s);
                    if (GATEUP) u += ld_cluster_f32(at + kOut * 4, s);
                }
                const int64_t to = static_cast<int64_t>(row0 + r) * p.n + out;
                if (GATEUP) v = __fmul_rn(tq_silu(v), u);
                if (GATEUP || p.y_bf16) static_cast<uint16_t *>(p.y)[to] = f32_to_bf16_bits(v);
                else static_cast<float *>(p.y)[to] = v;
            }
            cluster_sync();
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int local = 16 * h + 8 * j + i, r = quarter * quarter_rows + local;
                    if (local >= quarter_rows || r >= rows) continue;
                    const int64_t to = static_cast<int64_t>(row0 + r) * p.n;
#pragma unroll
                    for (int e = 0; e < (GATEUP ? 4 : 8); ++e) {
                        if (!active(e)) continue;
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            const int64_t out = (static_cast<int64_t>(ntile) * kStrips + column(e)) * 16 + 4 * n + t;
                            if (out >= p.n) continue;
                            float v = half2of(acc[e][n][h], j);
                            if (GATEUP) v = __fmul_rn(tq_silu(v), half2of(acc[(e + 4) % 8][n][h], j));
                            if (GATEUP || p.y_bf16) static_cast<uint16_t *>(p.y)[to + out] = f32_to_bf16_bits(v);
                            else static_cast<float *>(p.y)[to + out] = v;
                        }
                    }
                }
        }
    }
    if (warp < 8 && args.split > 1) {
        cluster_sync();
        cluster_sync();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 4) tmem_dealloc(tmem, 512);
}

template <int GROUP, bool MINS, bool GATEUP>
cudaError_t launch(TileArgs &a, int sms, cudaStream_t stream) {
    constexpr size_t smem = sizeof(TileSmem) + 1024;
    static_assert(smem <= 227 * 1024, "shared memory");
    static SmemLimit limit;
    cudaError_t e = limit.raise(q4_tile_kernel<GROUP, MINS, GATEUP>, smem);
    if (e != cudaSuccess) return e;
    constexpr int kStrips = GATEUP ? (MINS ? 7 : 8) : (MINS ? 15 : 16);
    const int64_t tiles = (q4_strips(a.p.n) + kStrips - 1) / kStrips * a.row_tiles;
    const int chunks = a.p.k / 128;
    a.split = 1;
    while (a.split < 8 && tiles * (a.split + 1) <= sms && chunks >= 2 * (a.split + 1)) ++a.split;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * a.split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, q4_tile_kernel<GROUP, MINS, GATEUP>, a);
}

template <int GROUP>
cudaError_t pick(TileArgs &a, int sms, cudaStream_t stream) {
    const bool mins = a.p.mins[0] != nullptr;
    if (a.p.mats == 1) return mins ? launch<GROUP, true, false>(a, sms, stream) : launch<GROUP, false, false>(a, sms, stream);
    return mins ? launch<GROUP, true, true>(a, sms, stream) : launch<GROUP, false, true>(a, sms, stream);
}

}  // namespace

cudaError_t q4_tile_waits(unsigned *bits, cudaStream_t stream) {
    return cudaMemcpyFromSymbolAsync(bits, lost_waits, sizeof(*bits), 0, cudaMemcpyDeviceToHost, stream);
}

cudaError_t q4_tile_launch(const Q4Product &p, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    TileArgs a{};
    a.p = p;
    a.row_tiles = (p.m + kRows - 1) / kRows;
    a.rows = (p.m + a.row_tiles - 1) / a.row_tiles;
    e = make_tmap_2d(&a.x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.x, static_cast<uint64_t>(p.k), static_cast<uint64_t>(p.m),
                     static_cast<uint64_t>(p.k) * 2, kStageK, 32, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    return p.group == 128 ? pick<128>(a, sms, stream) : p.group == 64 ? pick<64>(a, sms, stream) : pick<32>(a, sms, stream);
}

}  // namespace tq
