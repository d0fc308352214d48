// tq_moe_tile.cu -- products grouped by expert for many rows per expert, on the
// 5th-generation tensor core.
//
// A tile is 128 weight rows x up to 224 activation rows of one expert (gate/up:
// 64 rows of each, interleaved, so that a pair of lanes holds both values of an
// output).  The weights are the A operand, decoded from their codes to e4m3
// -1, 0, +1 straight into tensor memory; the activations are the B operand in
// shared memory, each int8 code as two exact e4m3 numbers q = 16 h + l (sign
// and magnitude), both multiplied with the same A.  One 128-block is 2 x 4
// tcgen05.mma of K = 32 into one accumulator: an exact integer below 2^15.
// The block's accumulator is then read back and folded,
//   acc = fma(d, scale_w * scale_a, acc),
// in registers, blocks in ascending order: the stream kernel's bits.
//
// What bounds it.  With A in tensor memory an MMA of M = 128, K = 32 takes 128
// cycles for every N <= 224 (measured; 140 at N = 256, and 173 with A in shared
// memory), so N = 224 gives 7159 MACs per cycle and SM, half of them for each part
// of the code: 3580 int8 x ternary MACs.  224 columns also leave room for
// two accumulators (448 of 512 columns) and two blocks of A (64 columns).
//
// Warps: 0-3 decode weights, 4 issues MMAs, 5 copies activation rows (TMA),
// 6-7 their scales, 8-15 fold (a quarter of the lanes and half of the columns
// each).  The fold's 112 accumulators per thread need more than an even share of
// the registers, so the roles resize theirs.
#include <cuda_runtime.h>

#include "tq_device.cuh"
#include "tq_launch.h"
#include "tq_moe_codes.cuh"
#include "tq_moe_internal.h"
#include "tq_tcgen05.cuh"
#include "tq_tmap.h"

namespace tq {
namespace {

constexpr int kCols = 224;                          // most activation rows per tile
constexpr int kStages = 3;
constexpr int kBoxRows = 32;                        // rows per TMA copy
constexpr int kDone = 6;                            // multiple of the 3 stages and the 2 buffers
constexpr int kGroup = 4;                           // blocks whose scales come together
constexpr int kGroups = 3;
constexpr int kThreads = 512;
constexpr int kScaleThreads = 64;                   // warps 6 and 7
constexpr uint32_t kHalf = kCols * 128;             // bytes of one part of a stage
constexpr uint32_t kStageBytes = 2 * kHalf;
constexpr uint32_t kTmemA = 2 * kCols;              // first column of the A buffers
constexpr int kFoldCols = kCols / 2;                // columns per fold warp

// register shares (launched with 128 per thread): 128 x (96 + 48 + 2 x 184) = 512 x 128
constexpr int kRegsDecode = 96, kRegsIssue = 48, kRegsFold = 184;

struct __align__(1024) TileSmem {
    uint8_t b[kStages][kStageBytes];
    float as[kGroups][kGroup][kCols];
    uint64_t b_full[kStages], a_full[2], d_empty[2], done[kDone], s_full[kGroups], s_empty[kGroups], drain;
    uint32_t tmem;
    uint32_t dead;                                  // a bounded wait ran out
};

struct TileArgs {
    MoeProduct p;
    CUtensorMap map;            // the operand, [slots][k/128][16 h: 128 | l: 128] bytes, boxes of kBoxRows x 128
    unsigned *err;
    int above;                  // experts with more rows than this are this kernel's
};

// The pair'th (expert, part of its rows); false behind the last.  An expert's
// rows are dealt to as few tiles as hold them, evenly.
__device__ __forceinline__ bool find_tile(const MoeProduct &p, int above, int pair, int &expert, int &row0, int &cols) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 32) {
        const int e = e0 + lane;
        int lo = 0, n = 0;
        if (e < p.experts) {
            lo = min(max(p.offsets[e], 0), p.slots);
            n = max(min(max(p.offsets[e + 1], 0), p.slots) - lo, 0);
        }
        const int c = n > above ? (n + kCols - 1) / kCols : 0;
        int incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, pair < base + incl);
        if (hit != 0) {
            const int src = __ffs(hit) - 1;
            const int part = pair - base - __shfl_sync(0xffffffffu, incl - c, src);
            const int parts = __shfl_sync(0xffffffffu, c, src), rows = __shfl_sync(0xffffffffu, n, src);
            const int each = ((rows + parts - 1) / parts + 15) / 16 * 16;    // at most kCols, a multiple of 16
            expert = e0 + src;
            row0 = __shfl_sync(0xffffffffu, lo, src) + part * each;
            cols = min(each, rows - part * each);
            return true;                             // cols may be 0 or less for the last part
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
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

// kBoxRows rows of 128 bytes at (byte x, row y) of the operand; counted on `bar`.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int R>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// tcgen05.wait::ld; the registers pass through it, so nothing reads them before.
__device__ __forceinline__ void wait_ld8(uint32_t (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
}

// A bounded wait; once one ran out every later wait of the CTA gives up at once.
template <int SLEEP = 0>
__device__ __forceinline__ bool wait_or_die(TileSmem &sm, uint64_t &bar, uint32_t parity, unsigned *err, unsigned bit) {
    const uint32_t addr = smem_u32(&bar);
    if (mbar_try_wait(addr, parity)) return true;
    const long long t0 = clock64();
    for (;;) {
        // polls take issue slots and shared memory from the fold: few, with pauses
#pragma unroll 1
        for (int i = 0; i < 32; ++i) {
            if (mbar_try_wait(addr, parity)) return true;
            if (SLEEP > 0) __nanosleep(SLEEP);
        }
        if (*reinterpret_cast<volatile uint32_t *>(&sm.dead)) return false;
        if (clock64() - t0 > kWaitBudgetCycles) {
            *reinterpret_cast<volatile uint32_t *>(&sm.dead) = 1;
            atomicOr(err, bit);
            return false;
        }
    }
}

// The same for a whole warp, with one answer for all of its lanes.
template <int SLEEP = 0>
__device__ __forceinline__ bool warp_wait(TileSmem &sm, uint64_t &bar, uint32_t parity, unsigned *err, unsigned bit) {
    return __all_sync(0xffffffffu, wait_or_die<SLEEP>(sm, bar, parity, err, bit));
}

template <int FMT, bool GATEUP>
__global__ void __launch_bounds__(kThreads, 1) tile_kernel(const __grid_constant__ TileArgs args) {
    extern __shared__ uint8_t smem_raw[];
    TileSmem &sm = *reinterpret_cast<TileSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const MoeProduct &p = args.p;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (warp == 4) {
        tmem_alloc(smem_u32(&sm.tmem), 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(&sm.b_full[i]), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sm.a_full[i]), 4);
            mbar_init(smem_u32(&sm.d_empty[i]), 8);
        }
        for (int i = 0; i < kDone; ++i) mbar_init(smem_u32(&sm.done[i]), 1);
        for (int i = 0; i < kGroups; ++i) {
            mbar_init(smem_u32(&sm.s_full[i]), kScaleThreads);
            mbar_init(smem_u32(&sm.s_empty[i]), 8);
        }
        mbar_init(smem_u32(&sm.drain), 1);
        sm.dead = 0;
        mbar_init_fence();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    pdl_launch_dependents();
    pdl_wait();

    const int nb = p.k / kBlock;
    constexpr int kRowsPerTile = GATEUP ? 64 : 128;
    const int ntiles = (p.n + kRowsPerTile - 1) / kRowsPerTile;
    constexpr int kBlockBytes = FMT == 0 ? 32 : 16;
    int it = 0;                                     // blocks since the start, over all tiles
    int expert, row0, cols;

    if (warp < 4) regs_down<kRegsDecode>();
    else if (warp < 8) regs_down<kRegsIssue>();
    else regs_up<kRegsFold>();

    if (warp < 4) {
        // ---- decode: thread = lane of tensor memory = weight row ----
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16) + kTmemA;
        for (int item = blockIdx.x; find_tile(p, args.above, item / ntiles, expert, row0, cols); item += gridDim.x) {
            const int n0 = (item % ntiles) * kRowsPerTile;
            const int r = min(GATEUP ? n0 + (tid >> 1) : n0 + tid, p.n - 1);
            const uint8_t *codes = p.codes[GATEUP ? tid & 1 : 0];
            const uint4 *src = reinterpret_cast<const uint4 *>(
                codes + (static_cast<int64_t>(expert) * p.n + r) * nb * kBlockBytes);
            constexpr int kVec = kBlockBytes / 16;
            // four blocks per fetch, one fetch ahead
            uint4 next[4 * kVec];
#pragma unroll
            for (int i = 0; i < 4 * kVec; ++i)
                if (i < nb * kVec) next[i] = __ldg(src + i);
            for (int b0 = 0; b0 < nb; b0 += 4) {
                uint4 cur[4 * kVec];
#pragma unroll
                for (int i = 0; i < 4 * kVec; ++i) {
                    cur[i] = next[i];
                    if ((b0 + 4) * kVec + i < nb * kVec) next[i] = __ldg(src + (b0 + 4) * kVec + i);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (b0 + j >= nb) break;
                    const int buf = it & 1;
                    uint32_t v[32];
                    decode_block<FMT>(&cur[j * kVec], v);
                    if (it >= 2 && !warp_wait<64>(sm, sm.done[(it - 2) % kDone], ((it - 2) / kDone) & 1, args.err, 1u << 0))
                        goto done;
                    tc_fence_after();
                    __syncwarp();
                    tmem_st_x32(lane_base + buf * 32, v);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sm.a_full[buf]));
                    ++it;
                }
            }
        }
    } else if (warp == 4) {
        // ---- issue ----
        for (int item = blockIdx.x; find_tile(p, args.above, item / ntiles, expert, row0, cols); item += gridDim.x) {
            const uint32_t n16 = static_cast<uint32_t>(max(cols + 15, 16)) / 16 * 16;
            const uint32_t idesc = idesc_e4m3(128, static_cast<int>(n16));
            bool ok = true;
            if (lane == 0) {
                for (int b = 0; b < nb && ok; ++b, ++it) {
                    const int st = it % kStages, buf = it & 1;
                    ok = wait_or_die(sm, sm.d_empty[buf], ((it >> 1) & 1) ^ 1, args.err, 1u << 1) &&
                         wait_or_die(sm, sm.a_full[buf], (it >> 1) & 1, args.err, 1u << 2) &&
                         wait_or_die(sm, sm.b_full[st], (it / kStages) & 1, args.err, 1u << 3);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + buf * kCols, a = tmem + kTmemA + buf * 32;
                    const uint64_t hi = desc_sw128(smem_u32(sm.b[st])), lo = desc_sw128(smem_u32(sm.b[st]) + kHalf);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        tc_mma_e4m3_ts(d, a + 8 * i, hi + 2 * i, idesc, i > 0);
                        tc_mma_e4m3_ts(d, a + 8 * i, lo + 2 * i, idesc, 1);
                    }
                    // one commit frees the stage and the A buffer and hands over the accumulator
                    // (each waits for the block that it needs; none is ever six blocks behind)
                    tc_commit(smem_u32(&sm.done[it % kDone]));
                }
            }
            it = __shfl_sync(0xffffffffu, it, 0);
            if (!__shfl_sync(0xffffffffu, static_cast<int>(ok), 0)) break;
        }
        if (lane == 0) {
            tc_commit(smem_u32(&sm.drain));
            if (!mbar_wait(smem_u32(&sm.drain), 0)) atomicOr(args.err, 1u << 4);
        }
        __syncwarp();
    } else if (warp < 8) {
        // ---- copy: warp 5 brings activation rows, 32 per copy, lane i rows 32 i
        // (i < 7) of one part and lane 8 + i of the other; warps 6 and 7 the scales ----
        if (warp == 5) {
            bool ok = true;
            for (int item = blockIdx.x; ok && find_tile(p, args.above, item / ntiles, expert, row0, cols); item += gridDim.x) {
                const int boxes = (cols + kBoxRows - 1) / kBoxRows;
                const int part = lane >> 3, box = lane & 7;
                for (int b = 0; b < nb; ++b, ++it) {
                    const int st = it % kStages;
                    ok = it < kStages || warp_wait<64>(sm, sm.done[(it - kStages) % kDone], ((it - kStages) / kDone) & 1,
                                                       args.err, 1u << 5);
                    if (!ok) break;
                    const uint32_t bar = smem_u32(&sm.b_full[st]);
                    if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(boxes) * 2 * kBoxRows * 128);
                    __syncwarp();
                    if (lane < 16 && box < boxes)
                        copy_box(smem_u32(sm.b[st]) + part * kHalf + box * kBoxRows * 128, &args.map, b * 256 + part * 128,
                                 row0 + box * kBoxRows, bar);
                }
            }
            // none of this CTA's copies may be in flight when it leaves
            for (int j = max(it - kStages, 0); j < it; ++j)
                if (!mbar_wait(smem_u32(&sm.b_full[j % kStages]), (j / kStages) & 1)) atomicOr(args.err, 1u << 8);
        } else {
            const int ct = tid - 192;
            bool ok = true;
            for (int item = blockIdx.x; ok && find_tile(p, args.above, item / ntiles, expert, row0, cols); item += gridDim.x) {
                const float *src[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = row0 + min(ct + kScaleThreads * i, cols - 1);
                    src[i] = p.s + static_cast<int64_t>(min(max(p.rows != nullptr ? p.rows[r] : r, 0), p.m - 1)) * nb;
                }
                for (int b = 0; b < nb; b += kGroup, ++it) {
                    const int slot = it % kGroups;
                    ok = warp_wait<64>(sm, sm.s_empty[slot], ((it / kGroups) & 1) ^ 1, args.err, 1u << 6);
                    if (!ok) break;
#pragma unroll
                    for (int j = 0; j < kGroup; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (b + j < nb && ct + kScaleThreads * i < cols)
                                cp_async4(smem_u32(&sm.as[slot][j][ct + kScaleThreads * i]), src[i] + b + j);
                    cp_async_commit();
                    if (it >= 1) {
                        cp_async_wait<1>();         // the group before has landed
                        mbar_arrive(smem_u32(&sm.s_full[(it - 1) % kGroups]));
                    }
                }
            }
            cp_async_wait<0>();
            if (it >= 1) mbar_arrive(smem_u32(&sm.s_full[(it - 1) % kGroups]));
        }
    } else {
        // ---- fold ----
        const int quarter = warp & 3, half = (warp - 8) >> 2;
        const int r_tile = 32 * quarter + lane;
        int group = 0;                              // groups of scales since the start
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * kFoldCols;
        for (int item = blockIdx.x; find_tile(p, args.above, item / ntiles, expert, row0, cols); item += gridDim.x) {
            const int n0 = (item % ntiles) * kRowsPerTile;
            const int out_r = GATEUP ? n0 + (r_tile >> 1) : n0 + r_tile;
            const uint16_t *wsp = p.scales[GATEUP ? r_tile & 1 : 0] +
                                  (static_cast<int64_t>(expert) * p.n + min(out_r, p.n - 1)) * nb;
            const int mine = min(max(cols - half * kFoldCols, 0), kFoldCols);   // columns of this warp
            uint64_t acc[kFoldCols / 2];
#pragma unroll
            for (int i = 0; i < kFoldCols / 2; ++i) acc[i] = 0;
            uint16_t ws_next[2] = {ldg_u16(wsp), ldg_u16(wsp + min(1, nb - 1))};   // two blocks ahead
            for (int b = 0; b < nb; ++b, ++it) {
                const int buf = it & 1, slot = group % kGroups, in_group = b % kGroup;
                const float ws = f16_bits_to_f32(ws_next[0]);
                ws_next[0] = ws_next[1];
                if (b + 2 < nb) ws_next[1] = ldg_u16(wsp + b + 2);
                const uint64_t ws2 = pack2(ws, ws);
                if (in_group == 0 && !warp_wait(sm, sm.s_full[slot], (group / kGroups) & 1, args.err, 1u << 6)) goto done;
                if (!warp_wait(sm, sm.done[it % kDone], (it / kDone) & 1, args.err, 1u << 7)) goto done;
                tc_fence_after();
                const float *as = &sm.as[slot][in_group][half * kFoldCols];
                const uint32_t dcol = lane_base + buf * kCols;
                // all columns, whether the tile has them or not (what the others hold goes
                // nowhere), eight at a time: while they are folded the next are on their way
                uint32_t v[2][8];
                ulonglong2 s4[2][2];
                tmem_ld<8>(dcol, v[0]);
                s4[0][0] = *reinterpret_cast<const ulonglong2 *>(as);
                s4[0][1] = *reinterpret_cast<const ulonglong2 *>(as + 4);
#pragma unroll
                for (int c = 0; c < kFoldCols / 8; ++c) {
                    const int x = c & 1;
                    wait_ld8(v[x]);
                    if (c + 1 < kFoldCols / 8) {
                        tmem_ld<8>(dcol + 8 * c + 8, v[x ^ 1]);
                        s4[x ^ 1][0] = *reinterpret_cast<const ulonglong2 *>(as + 8 * c + 8);
                        s4[x ^ 1][1] = *reinterpret_cast<const ulonglong2 *>(as + 8 * c + 12);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[4 * c + i] = fma2(pack2(__uint_as_float(v[x][2 * i]), __uint_as_float(v[x][2 * i + 1])),
                                              mul2(ws2, i & 1 ? s4[x][i >> 1].y : s4[x][i >> 1].x), acc[4 * c + i]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&sm.d_empty[buf]));
                    if (in_group == kGroup - 1 || b + 1 == nb) mbar_arrive(smem_u32(&sm.s_empty[slot]));
                }
                if (in_group == kGroup - 1 || b + 1 == nb) ++group;
            }
            const int64_t first = row0 + half * kFoldCols;
            if (GATEUP) {
                // even lanes hold gate and take column 2i, odd lanes hold up and take 2i + 1
                const bool odd = (lane & 1) != 0;
                uint16_t *out = p.h + (first + (odd ? 1 : 0)) * p.n + out_r;
                const int have = out_r < p.n ? mine - (odd ? 1 : 0) : 0;
#pragma unroll
                for (int i0 = 0; i0 < kFoldCols / 2; i0 += 8) {
                    if (2 * i0 >= mine) break;
                    float g[8], u[8], s[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float x, y;
                        unpack2(acc[i0 + i], x, y);
                        const float other = __shfl_xor_sync(0xffffffffu, odd ? x : y, 1);
                        g[i] = odd ? other : x;
                        u[i] = odd ? y : other;
                    }
                    moe_silu(g, s);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (2 * (i0 + i) < have) out[static_cast<int64_t>(2 * (i0 + i)) * p.n] = f32_to_bf16_bits(__fmul_rn(s[i], u[i]));
                }
            } else if (out_r < p.n) {
                float *out = p.y + first * p.n + out_r;
#pragma unroll
                for (int i = 0; i < kFoldCols / 2; ++i) {
                    if (2 * i >= mine) break;
                    float x, y;
                    unpack2(acc[i], x, y);
                    out[static_cast<int64_t>(2 * i) * p.n] = x;
                    if (2 * i + 1 < mine) out[static_cast<int64_t>(2 * i + 1) * p.n] = y;
                }
            }
        }
    }
done:
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 4) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// The operand: the codes of each sorted slot in the order in which the decoded
// weights meet them, as two e4m3 numbers each, [block][16 h: 128 bytes | l: 128].
// One thread per 32 codes.  Rows are gathered here and not by the tile kernel's
// copies: a TMA gather of four rows runs at 13 cycles per 128-byte row
// (measured), four times slower than the MMAs use them up.
// ---------------------------------------------------------------------------
template <int FMT>
__global__ void __launch_bounds__(256) operand_kernel(const int8_t *__restrict__ q, const int *__restrict__ rows,
                                                      const int *__restrict__ offsets, int experts, int m, int slots,
                                                      int k, uint8_t *__restrict__ out) {
    pdl_launch_dependents();
    pdl_wait();
    const int per_row = k / 32;
    const int64_t groups = static_cast<int64_t>(min(max(offsets[experts], 0), slots)) * per_row;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < groups;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int r = static_cast<int>(i / per_row), c = static_cast<int>(i - static_cast<int64_t>(r) * per_row);
        const int a = min(max(rows != nullptr ? rows[r] : r, 0), m - 1);
        const uint4 *src = reinterpret_cast<const uint4 *>(q + static_cast<int64_t>(a) * k + c * 32);
        const uint4 q0 = __ldg(src), q1 = __ldg(src + 1);
        const uint32_t w[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
        uint32_t o[8], hi[8], lo[8];
        stage_order<FMT>(w, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) split4_whole(o[j], hi[j], lo[j]);
        uint8_t *dst = out + (i >> 2) * 256 + (i & 3) * 32;
        *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(dst + 16) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
        *reinterpret_cast<uint4 *>(dst + 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<uint4 *>(dst + 144) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
    }
}

template <int FMT, bool GATEUP>
cudaError_t launch(const MoeProduct &p, int above, uint8_t *operand, unsigned *err, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int64_t groups = static_cast<int64_t>(p.slots) * p.k / 32;
    const int64_t want = (groups + 255) / 256;
    e = launch_pdl(operand_kernel<FMT>, dim3(static_cast<unsigned>(want < (1 << 20) ? want : (1 << 20))), dim3(256), 0,
                   stream, p.q, p.rows, p.offsets, p.experts, p.m, p.slots, p.k, operand);
    if (e != cudaSuccess) return e;
    constexpr size_t smem = sizeof(TileSmem) + 1024;
    e = cudaFuncSetAttribute(tile_kernel<FMT, GATEUP>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    TileArgs a{};
    a.p = p;
    a.err = err;
    a.above = above;
    e = make_tmap_2d(&a.map, CU_TENSOR_MAP_DATA_TYPE_UINT8, operand, static_cast<uint64_t>(2) * p.k,
                     static_cast<uint64_t>(p.slots), static_cast<uint64_t>(2) * p.k, 128, kBoxRows, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    return launch_pdl(tile_kernel<FMT, GATEUP>, dim3(sms), dim3(kThreads), smem, stream, a);
}

}  // namespace

cudaError_t moe_tile_launch(const MoeProduct &p, int above, uint8_t *operand, unsigned *err, cudaStream_t stream) {
    if (p.h != nullptr)
        return p.fmt == TQ_FMT_TERNARY2 ? launch<0, true>(p, above, operand, err, stream)
                                        : launch<1, true>(p, above, operand, err, stream);
    return p.fmt == TQ_FMT_TERNARY2 ? launch<0, false>(p, above, operand, err, stream)
                                    : launch<1, false>(p, above, operand, err, stream);
}

}  // namespace tq
