// tq_moe_tile.cu -- products grouped by expert for many rows per expert, on the
// 5th-generation tensor core.
//
// A tile is 128 weight rows x up to 192 activation rows of one expert (gate/up:
// 64 rows of each, eight by eight, so that one lane folds both values of an
// output).  The weights are the A operand, decoded from their codes to e4m3
// -1, 0, +1 straight into tensor memory; the activations are the B operand in
// shared memory, each int8 code as two exact e4m3 numbers q = 16 h + l (sign
// and magnitude), both multiplied with the same A.  One 128-block is 2 x 4
// tcgen05.mma of K = 32 into one accumulator: an exact integer below 2^15.
// The block's accumulator is then read back and folded,
//   acc = fma(d, scale_w * scale_a, acc),
// in registers, blocks in ascending order: the stream kernel's bits.
//
// What bounds it.  With A in tensor memory an MMA of M = 128, K = 32 takes N / 2 cycles (measured; and 51
// at least, issued by one thread in a branch, as here): 768 cycles for a block of 192 columns.  Every
// block's accumulator has to leave tensor memory and be folded meanwhile, and the hand-over (commit,
// wait, read, release) has its latency on each side:
// a block takes about 2000 cycles, and that is the bound, not the tensor core, nor memory.
// Two accumulators of 192 columns leave room for four blocks of A, and a third of them for
// each of three warps to a quarter of the lanes (two of 224: two blocks of A, two warps;
// with the shorter waits that came with it 465 us, 408 then, for the gate/up below).
// 4096 tokens, top 8 of 64 experts, 2 x 1024 x 2048: 417 us, 330 T code products/s (twice
// as many e4m3 ones); 2 x 1536 x 5120 with its down product: 1252 + 734 us, 389 T/s.  The fold
// keeps 32 pairs of sums in 112 registers: a 64-byte stack, 108 to 116 bytes of spill stores and 200 to
// 216 of loads.  Activation rows come to every CTA by its own copies; shared by the two CTAs of
// a cluster, which halved what L2 delivers, they took 1% less time.
//
// Warps: 0-3 decode weights, 4 issues MMAs, 5 copies activation rows (TMA), 6 packed
// weights (TMA), 7 activation scales, 8-19 fold (a quarter of the lanes and a third of the
// columns each).  The fold needs more than an even share of the registers, so the roles
// resize theirs.
#include <cuda_runtime.h>

#include "tq_device.cuh"
#include "tq_launch.h"
#include "tq_moe_codes.cuh"
#include "tq_moe_internal.h"
#include "tq_tcgen05.cuh"
#include "tq_tmap.h"

namespace tq {
namespace {

constexpr int kCols = 192;                          // most activation rows per tile
constexpr int kStages = 3;                          // blocks of activations in shared memory
constexpr int kBoxRows = 32;                        // rows per TMA copy
constexpr int kDone = 4;                            // blocks between a barrier's uses
constexpr int kGroup = 4;                           // blocks whose scales come together
constexpr int kGroups = 4;                          // groups of scales in shared memory
constexpr int kCodeGroups = 2;                      // groups of packed codes in shared memory
constexpr int kFoldWarps = 12;
constexpr int kThreads = 256 + 32 * kFoldWarps;
constexpr uint32_t kHalf = kCols * 128;             // bytes of one part of a stage
constexpr uint32_t kStageBytes = 2 * kHalf;
constexpr uint32_t kTmemA = 2 * kCols;              // first column of the A buffers
constexpr int kFoldCols = kCols / (kFoldWarps / 4); // columns per fold warp

// register shares (launched with 96 per thread): 128 x (96 + 48 + 3 x 112) = 640 x 96
constexpr int kRegsIssue = 48, kRegsFold = 112;
constexpr int kABufs = kDone;                           // blocks of decoded weights: 32 columns each

__device__ unsigned lost_waits;                     // bits of all waits that have run out on this device

struct __align__(1024) TileSmem {
    uint8_t b[kStages][kStageBytes];
    uint8_t codes[kCodeGroups][128 * 128];          // 128 rows x 4 blocks (1-bit: 64 bytes a row), swizzled
    float2 as[kGroups][kGroup][kCols];              // activation scales, each twice, in fold order
    float ws[kGroups][kGroup][128];                 // weight scales, in fold order
    int offsets[TQ_MOE_MAX_EXPERTS + 1];            // clamped to 0 .. slots
    int tiles[TQ_MOE_MAX_EXPERTS + 1];              // column tiles of the experts before
    int warp_sum[kThreads / 32];
    uint64_t b_full[kStages], b_empty[kStages], a_full[kABufs], d_empty[2], done[kDone];
    uint64_t c_full[kCodeGroups], c_empty[kCodeGroups], s_full[kGroups], s_empty[kGroups], drain;
    uint32_t tmem;
    uint32_t dead;                                  // a bounded wait ran out
};

struct TileArgs {
    MoeProduct p;
    CUtensorMap codes[2];       // packed weights, [experts * n][row bytes], boxes of 64 rows x 4 blocks
    const float *scales;        // [slots][k/128 rounded up to 4]: the operand's scales
    CUtensorMap map;            // the operand, [slots][k/128][16 h: 128 | l: 128] bytes, boxes of kBoxRows x 128
    unsigned *err;
    int above;                  // experts with more rows than this are this kernel's
};

// An expert's rows are dealt to as few tiles as hold them, evenly, in multiples of 16.
__device__ __forceinline__ int expert_tiles(int rows, int above) { return rows > above ? (rows + kCols - 1) / kCols : 0; }

// Fill sm.offsets and sm.tiles (all threads).
__device__ __forceinline__ void list_tiles(TileSmem &sm, const MoeProduct &p, int above) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool ok = load_offsets(p, sm.offsets);
    int base = 0;
    for (int e0 = 0; e0 < p.experts; e0 += kThreads) {
        const int e = e0 + tid;
        const int c = ok && e < p.experts ? expert_tiles(sm.offsets[e + 1] - sm.offsets[e], above) : 0;
        int incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) sm.warp_sum[warp] = incl;
        __syncthreads();
        int all = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            const int s = sm.warp_sum[w];
            if (w < warp) incl += s;
            all += s;
        }
        if (e < p.experts) sm.tiles[e] = base + incl - c;
        base += all;
        __syncthreads();
    }
    if (tid == 0) sm.tiles[p.experts] = base;
    __syncthreads();
}

// The expert and rows of column tile `pair`; false behind the last.
__device__ __forceinline__ bool find_tile(const TileSmem &sm, int experts, int pair, int &expert, int &row0, int &cols) {
    if (pair >= sm.tiles[experts]) return false;
    int lo = 0, hi = experts;                       // tiles[lo] <= pair < tiles[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sm.tiles[mid] <= pair) lo = mid;
        else hi = mid;
    }
    const int parts = sm.tiles[lo + 1] - sm.tiles[lo], part = pair - sm.tiles[lo];
    const int rows = sm.offsets[lo + 1] - sm.offsets[lo];
    const int each = ((rows + parts - 1) / parts + 15) / 16 * 16;            // at most kCols
    expert = lo;
    row0 = sm.offsets[lo] + part * each;
    cols = min(each, rows - part * each);           // at least 1: (parts - 1) * kCols < rows
    return true;
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

// The box of `map` at (byte x, row y); counted on `bar`.
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

// tcgen05.wait::ld; the registers pass through it, so nothing reads them before.
__device__ __forceinline__ void wait_ld16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// 32 lanes x 16 columns in the 16x128b shape, lanes 0-15 and 16-31: register
// 8 h + 2 n + j is row 16 h + 8 j + lane / 4, column 4 n + lane % 4.
__device__ __forceinline__ void ld_chunk(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.16x128b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
    asm volatile("tcgen05.ld.sync.aligned.16x128b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr + (16u << 16))
                 : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}

// A bounded wait.  One that runs out sets `dead` and the error word; every later
// wait of the CTA then gives up at once, so that all roles come to their end.
template <int SLEEP>
__device__ __forceinline__ void wait_slow(TileSmem &sm, uint32_t bar, uint32_t parity, unsigned *err, unsigned bit) {
    const long long t0 = clock64();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i) {
            if (mbar_try_wait(bar, parity)) return;
            if (SLEEP > 0) __nanosleep(SLEEP);      // polls take issue slots from the fold
        }
        if (*reinterpret_cast<volatile uint32_t *>(&sm.dead)) return;
        if (clock64() - t0 > kWaitBudgetCycles) {
            *reinterpret_cast<volatile uint32_t *>(&sm.dead) = 1;
            record_wait(err, &lost_waits, bit);
            return;
        }
    }
}
template <int SLEEP = 0>
__device__ __forceinline__ void warp_wait(TileSmem &sm, uint32_t bar, uint32_t parity, unsigned *err, unsigned bit) {
    if (!mbar_try_wait(bar, parity)) wait_slow<SLEEP>(sm, bar, parity, err, bit);
    __syncwarp();
}
// The same, and whether the CTA is still alive (one answer for the whole warp).  Lanes may wait for different barriers:
// __syncwarp orders memory between them, which a vote does not.
template <int SLEEP = 0>
__device__ __forceinline__ bool warp_wait_alive(TileSmem &sm, uint32_t bar, uint32_t parity, unsigned *err, unsigned bit) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        wait_slow<SLEEP>(sm, bar, parity, err, bit);
        ok = *reinterpret_cast<volatile uint32_t *>(&sm.dead) == 0;
    }
    ok = __all_sync(0xffffffffu, ok);
    __syncwarp();
    return ok;
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
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&sm.b_full[i]), 1);
            mbar_init(smem_u32(&sm.b_empty[i]), 1);
        }
        for (int i = 0; i < kABufs; ++i) mbar_init(smem_u32(&sm.a_full[i]), 4);
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&sm.d_empty[i]), kFoldWarps);
        for (int i = 0; i < kCodeGroups; ++i) {
            mbar_init(smem_u32(&sm.c_full[i]), 1);
            mbar_init(smem_u32(&sm.c_empty[i]), 4);
        }
        for (int i = 0; i < kDone; ++i) mbar_init(smem_u32(&sm.done[i]), 1);
        for (int i = 0; i < kGroups; ++i) {
            mbar_init(smem_u32(&sm.s_full[i]), 1 + 4);
            mbar_init(smem_u32(&sm.s_empty[i]), kFoldWarps);
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
    list_tiles(sm, p, args.above);

    const int nb = p.k / kBlock;
    constexpr int kRowsPerTile = GATEUP ? 64 : 128;
    // neighbouring CTAs take neighbouring row tiles of one column tile: its activation rows meet in L2
    const int nparts = (p.n + kRowsPerTile - 1) / kRowsPerTile;
    const int first_item = blockIdx.x, item_step = gridDim.x;
    constexpr int kBlockBytes = FMT == 0 ? 32 : 16;
    int it = 0;                                     // blocks since the start, over all tiles
    int expert, row0, cols;

    // (the decode warps keep what they have)
    if (warp >= 8) regs_up<kRegsFold>();
    else if (warp >= 4) regs_down<kRegsIssue>();

    if (warp < 4) {
        // ---- decode: thread = lane of tensor memory = weight row ----
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16) + kTmemA;
        int group = 0;
        // this lane's row in shared memory: gate/up hold 64 rows each
        const int tile_row = GATEUP ? 16 * warp + 8 * (lane >> 4) + (lane & 7) : tid;
        const int smem_row = GATEUP ? 64 * ((lane >> 3) & 1) + tile_row : tid;
        const bool wide = nb % 4 == 0 && (reinterpret_cast<uintptr_t>(p.scales[0]) & 7) == 0 &&
                          (!GATEUP || (reinterpret_cast<uintptr_t>(p.scales[1]) & 7) == 0);
        for (int item = first_item; find_tile(sm, p.experts, item / nparts, expert, row0, cols); item += item_step) {
            const int n0 = item % nparts * kRowsPerTile;
            const int r = min(n0 + tile_row, p.n - 1);
            const uint16_t *wsp = p.scales[GATEUP ? (lane >> 3) & 1 : 0] + (static_cast<int64_t>(expert) * p.n + r) * nb;
            for (int b0 = 0; b0 < nb; b0 += kGroup, ++group) {
                // the group's weight scales, to the fold's place
                float w[kGroup];
                if (wide) {
                    const uint2 h = __ldg(reinterpret_cast<const uint2 *>(wsp + b0));
                    w[0] = f16_bits_to_f32(h.x & 0xffffu); w[1] = f16_bits_to_f32(h.x >> 16);
                    w[2] = f16_bits_to_f32(h.y & 0xffffu); w[3] = f16_bits_to_f32(h.y >> 16);
                } else {
#pragma unroll
                    for (int j = 0; j < kGroup; ++j) w[j] = f16_bits_to_f32(ldg_u16(wsp + min(b0 + j, nb - 1)));
                }
                const int slot = group % kGroups, cslot = group % kCodeGroups;
                warp_wait<64>(sm, smem_u32(&sm.s_empty[slot]), ((group / kGroups) & 1) ^ 1, args.err, 1u << 6);
#pragma unroll
                for (int j = 0; j < kGroup; ++j) sm.ws[slot][j][32 * warp + 4 * (lane & 7) + (lane >> 3)] = w[j];
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.s_full[slot]));
                warp_wait<64>(sm, smem_u32(&sm.c_full[cslot]), (group / kCodeGroups) & 1, args.err, 1u << 9);
                const uint8_t *row = sm.codes[cslot] + smem_row * (kGroup * kBlockBytes);
#pragma unroll
                for (int j = 0; j < kGroup; ++j) {
                    if (b0 + j >= nb) break;
                    const int abuf = it % kABufs;
                    uint4 c[kBlockBytes / 16];
#pragma unroll
                    for (int i = 0; i < kBlockBytes / 16; ++i) {
                        const int chunk = j * (kBlockBytes / 16) + i;
                        c[i] = *reinterpret_cast<const uint4 *>(
                            row + ((FMT == 0 ? chunk ^ (smem_row & 7) : chunk ^ ((smem_row >> 1) & 3)) << 4));
                    }
                    if (j == kGroup - 1 || b0 + j + 1 == nb) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&sm.c_empty[cslot]));
                    }
                    // the buffer's last reader is done (kABufs == kDone: the phase before this block's)
                    warp_wait<64>(sm, smem_u32(&sm.done[abuf]), ((it / kDone) & 1) ^ 1, args.err, 1u << 0);
                    tc_fence_after();
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        uint32_t v[16];
                        decode_half<FMT>(c, s, v);
                        tmem_st_x16(lane_base + abuf * 32 + 16 * s, v);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sm.a_full[abuf]));
                    ++it;
                }
            }
        }
    } else if (warp == 4) {
        // ---- issue ----
        for (int item = first_item; find_tile(sm, p.experts, item / nparts, expert, row0, cols); item += item_step) {
            const uint32_t n16 = static_cast<uint32_t>(max(cols + 15, 16)) / 16 * 16;
            const uint32_t idesc = idesc_e4m3(128, static_cast<int>(n16));
            bool ok = true;
            for (int b = 0; b < nb; ++b, ++it) {
                const int st = it % kStages, buf = it & 1, abuf = it % kABufs;
                // three waits at once, one lane each
                const uint32_t bar = smem_u32(lane == 0 ? &sm.a_full[abuf] : lane == 1 ? &sm.b_full[st] : &sm.d_empty[buf]);
                const uint32_t parity = lane == 1 ? (it / kStages) & 1 : lane == 0 ? (it / kABufs) & 1 : ((it >> 1) & 1) ^ 1;
                ok = warp_wait_alive(sm, bar, parity, args.err, 1u << (lane < 2 ? lane + 2 : 1));
                if (!ok) break;
                if (lane == 0) {
                    tc_fence_after();
                    const uint32_t d = tmem + buf * kCols, a = tmem + kTmemA + abuf * 32;
                    const uint64_t hi = desc_sw128(smem_u32(sm.b[st])), lo = desc_sw128(smem_u32(sm.b[st]) + kHalf);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        tc_mma_e4m3_ts(d, a + 8 * i, hi + 2 * i, idesc, i > 0);
                        tc_mma_e4m3_ts(d, a + 8 * i, lo + 2 * i, idesc, 1);
                    }
                    // frees the stage; frees the A buffer and hands over the accumulator (who waits,
                    // waits for the block that it needs: the fold for one of the last two, the decode
                    // for the one before kDone more, so a barrier is never a whole turn ahead of a waiter)
                    tc_commit(smem_u32(&sm.b_empty[st]));
                    tc_commit(smem_u32(&sm.done[it % kDone]));
                }
                __syncwarp();
            }
            if (!ok) break;
        }
        if (lane == 0) {
            tc_commit(smem_u32(&sm.drain));
            if (!mbar_wait(smem_u32(&sm.drain), 0)) record_wait(args.err, &lost_waits, 1u << 4);
        }
        __syncwarp();
    } else if (warp < 8) {
        // ---- copy: warp 5 brings both parts of the activation rows' codes, 32 rows per copy;
        // warp 6 the packed weights, warp 7 the activation scales ----
        if (warp == 5) {
            bool ok = true;
            for (int item = first_item; ok && find_tile(sm, p.experts, item / nparts, expert, row0, cols); item += item_step) {
                const int boxes = (cols + kBoxRows - 1) / kBoxRows;
                for (int b = 0; b < nb; ++b, ++it) {
                    const int st = it % kStages;
                    ok = warp_wait_alive<64>(sm, smem_u32(&sm.b_empty[st]), ((it / kStages) & 1) ^ 1, args.err, 1u << 5);
                    if (!ok) break;
                    const uint32_t bar = smem_u32(&sm.b_full[st]);
                    if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(boxes) * 2 * kBoxRows * 128);
                    __syncwarp();
                    if (lane < 2 * boxes) {
                        const int part = lane & 1, box = lane >> 1;
                        load_box(smem_u32(sm.b[st]) + part * kHalf + box * kBoxRows * 128, &args.map, b * 256 + part * 128,
                                 row0 + box * kBoxRows, bar);
                    }
                }
            }
            // none of this CTA's copies may be in flight when it leaves
            for (int j = max(it - kStages, 0); j < it; ++j)
                if (!mbar_wait(smem_u32(&sm.b_full[j % kStages]), (j / kStages) & 1)) record_wait(args.err, &lost_waits, 1u << 8);
        } else if (warp == 6) {
            // packed weights: two boxes of 64 rows, gate and up or one matrix's 128
            bool ok = true;
            for (int item = first_item; ok && find_tile(sm, p.experts, item / nparts, expert, row0, cols); item += item_step) {
                const int y = expert * p.n + item % nparts * kRowsPerTile;
                for (int b = 0; b < nb; b += kGroup, ++it) {
                    const int slot = it % kCodeGroups;
                    ok = warp_wait_alive<64>(sm, smem_u32(&sm.c_empty[slot]), ((it / kCodeGroups) & 1) ^ 1, args.err, 1u << 10);
                    if (!ok) break;
                    if (lane == 0) {
                        const uint32_t bar = smem_u32(&sm.c_full[slot]), dst = smem_u32(sm.codes[slot]);
                        constexpr uint32_t kBox = 64 * kGroup * kBlockBytes;
                        mbar_arrive_expect_tx(bar, 2 * kBox);
                        load_box(dst, &args.codes[0], b * kBlockBytes, y, bar);
                        load_box(dst + kBox, &args.codes[1], b * kBlockBytes, GATEUP ? y : y + 64, bar);
                    }
                    __syncwarp();
                }
            }
            for (int j = max(it - kCodeGroups, 0); j < it; ++j)
                if (!mbar_wait(smem_u32(&sm.c_full[j % kCodeGroups]), (j / kCodeGroups) & 1)) record_wait(args.err, &lost_waits, 1u << 11);
        } else {
            // activation scales of four blocks at a time, each lane six rows
            constexpr int kRows = kCols / 32;
            const int ld = (nb + 3) / 4 * 4;
            for (int item = first_item; find_tile(sm, p.experts, item / nparts, expert, row0, cols); item += item_step) {
                const float *src = args.scales + static_cast<int64_t>(row0) * ld;
                for (int b = 0; b < nb; b += kGroup, ++it) {
                    const int slot = it % kGroups;
                    float4 v[kRows];
#pragma unroll
                    for (int i = 0; i < kRows; ++i)
                        v[i] = *reinterpret_cast<const float4 *>(src + min(lane + 32 * i, cols - 1) * ld + b);
                    warp_wait<64>(sm, smem_u32(&sm.s_empty[slot]), ((it / kGroups) & 1) ^ 1, args.err, 1u << 6);
#pragma unroll
                    for (int i = 0; i < kRows; ++i) {
                        const int c = lane + 32 * i;
                        // columns c, c + 4, c + 8, c + 12 of 16 are one fold lane's: side by side
                        float2 *dst = &sm.as[slot][0][(c & ~15) + 4 * (c & 3) + ((c >> 2) & 3)];
                        dst[0] = make_float2(v[i].x, v[i].x);
                        dst[kCols] = make_float2(v[i].y, v[i].y);
                        dst[2 * kCols] = make_float2(v[i].z, v[i].z);
                        dst[3 * kCols] = make_float2(v[i].w, v[i].w);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sm.s_full[slot]));
                }
            }
        }
    } else {
        // ---- fold ----
        // A lane (i = lane / 4, t = lane % 4) holds rows i, i + 8, i + 16, i + 24 of its
        // quarter and every fourth column from t on (shape 16x128b, register pairs are
        // rows i and i + 8), so a column's scale serves eight lanes and four rows.  With
        // a row and all columns per lane (32x32b) every scale is read in all 32 lanes, 530 of
        // the 768 cycles that a block's MMAs take, from the shared memory that also feeds
        // the MMAs (896): the fold of a block then took 1200 cycles.
        const int quarter = warp & 3, part = (warp - 8) >> 2, i = lane >> 2, t = lane & 3;
        int group = 0;                              // groups of scales since the start
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + part * kFoldCols;
        for (int item = first_item; find_tile(sm, p.experts, item / nparts, expert, row0, cols); item += item_step) {
            const int n0 = item % nparts * kRowsPerTile;
            const int mine = min(max(cols - part * kFoldCols, 0), kFoldCols);   // columns of this warp
            uint64_t acc[kFoldCols / 4][2];         // [column t + 4 n][h]
#pragma unroll
            for (int n = 0; n < kFoldCols / 4; ++n) acc[n][0] = acc[n][1] = 0;
            for (int b0 = 0; b0 < nb; b0 += kGroup, ++group) {
                const int slot = group % kGroups;
                const float2 *as = &sm.as[slot][0][part * kFoldCols + 4 * t];
                const float *ws = &sm.ws[slot][0][32 * quarter + 4 * i];
                warp_wait(sm, smem_u32(&sm.s_full[slot]), (group / kGroups) & 1, args.err, 1u << 6);
                const int end = it + min(nb - b0, kGroup);
#pragma unroll 1
                for (; it < end; ++it, as += kCols, ws += 128) {
                    const ulonglong2 ws2 = *reinterpret_cast<const ulonglong2 *>(ws);  // lane rows 16 h + i, 16 h + 8 + i
                    const uint32_t dcol = lane_base + (it & 1) * kCols;
                    warp_wait(sm, smem_u32(&sm.done[it % kDone]), (it / kDone) & 1, args.err, 1u << 7);
                    tc_fence_after();
                    // all columns, whether the tile has them or not (what the others hold goes nowhere)
#pragma unroll
                    for (int c = 0; c < kFoldCols / 16; ++c) {
                        uint32_t x[16];
                        ld_chunk(dcol + 16 * c, x);
                        const ulonglong2 s01 = *reinterpret_cast<const ulonglong2 *>(as + 16 * c),
                                         s23 = *reinterpret_cast<const ulonglong2 *>(as + 16 * c + 2);
                        wait_ld16(x);
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            const uint64_t s = n == 0 ? s01.x : n == 1 ? s01.y : n == 2 ? s23.x : s23.y;
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                acc[4 * c + n][h] =
                                    fma2(pack2(__uint_as_float(x[8 * h + 2 * n]), __uint_as_float(x[8 * h + 2 * n + 1])),
                                         mul2(h == 0 ? ws2.x : ws2.y, s), acc[4 * c + n][h]);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sm.d_empty[it & 1]));
                }
                if (lane == 0) mbar_arrive(smem_u32(&sm.s_empty[slot]));
            }
            // outputs of lane rows 16 h + i, 16 h + 8 + i: gate and up of one, or two
            int out_r[2][2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    out_r[h][j] = GATEUP ? n0 + 16 * quarter + 8 * h + i : n0 + 32 * quarter + 16 * h + 8 * j + i;
            const int64_t first = static_cast<int64_t>(row0 + part * kFoldCols + t) * p.n;
            const int have = mine - t;              // columns 4 n below this are the lane's own
#pragma unroll
            for (int c = 0; c < kFoldCols / 4; c += 4) {
                if (4 * c >= mine) break;
                if (GATEUP) {
                    float gate[8], up[8], s[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) unpack2(acc[c + (x >> 1)][x & 1], gate[x], up[x]);
                    moe_silu(gate, s);
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const int n = c + (x >> 1), h = x & 1;
                        if (4 * n < have && out_r[h][0] < p.n)
                            p.h[first + static_cast<int64_t>(4 * n) * p.n + out_r[h][0]] = f32_to_bf16_bits(__fmul_rn(s[x], up[x]));
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const int n = c + (x >> 1), h = x & 1;
                        float y[2];
                        unpack2(acc[n][h], y[0], y[1]);
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (4 * n < have && out_r[h][j] < p.n)
                                p.y[first + static_cast<int64_t>(4 * n) * p.n + out_r[h][j]] = y[j];
                    }
                }
            }
        }
    }
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
__global__ void __launch_bounds__(256) operand_kernel(const int8_t *q, const int *rows, const int *offsets,
                                                      int experts, int m, int slots, int k,
                                                      uint8_t *__restrict__ out, const float *s,
                                                      float *__restrict__ s_out) {
    pdl_launch_dependents();
    pdl_wait();
    const int per_row = k / 32;
    const int64_t groups = static_cast<int64_t>(min(max(offsets[experts], 0), slots)) * per_row;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < groups;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int r = static_cast<int>(i / per_row), c = static_cast<int>(i - static_cast<int64_t>(r) * per_row);
        const int a = min(max(rows != nullptr ? rows[r] : r, 0), m - 1);
        const uint4 *src = reinterpret_cast<const uint4 *>(q + static_cast<int64_t>(a) * k + c * 32);
        const uint4 q0 = src[0], q1 = src[1];
        const uint32_t w[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
        uint32_t o[8], hi[8], lo[8];
        stage_order<FMT>(w, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) split4_whole(o[j], hi[j], lo[j]);
        if ((c & 3) == 0)
            s_out[static_cast<int64_t>(r) * ((k / kBlock + 3) / 4 * 4) + (c >> 2)] = s[static_cast<int64_t>(a) * (k / kBlock) + (c >> 2)];
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
    float *scales = reinterpret_cast<float *>(operand + static_cast<int64_t>(2) * p.slots * p.k);
    const int64_t groups = static_cast<int64_t>(p.slots) * p.k / 32;
    const int64_t want = (groups + 255) / 256;
    e = launch_pdl(operand_kernel<FMT>, dim3(static_cast<unsigned>(want < (1 << 20) ? want : (1 << 20))), dim3(256), 0,
                   stream, p.q, p.rows, p.offsets, p.experts, p.m, p.slots, p.k, operand, p.s, scales);
    if (e != cudaSuccess) return e;
    constexpr size_t smem = sizeof(TileSmem) + 1024;
    static SmemLimit limit;
    e = limit.raise(tile_kernel<FMT, GATEUP>, smem);
    if (e != cudaSuccess) return e;
    TileArgs a{};
    a.p = p;
    a.err = err;
    a.above = above;
    e = make_tmap_2d(&a.map, CU_TENSOR_MAP_DATA_TYPE_UINT8, operand, static_cast<uint64_t>(2) * p.k,
                     static_cast<uint64_t>(p.slots), static_cast<uint64_t>(2) * p.k, 128, kBoxRows, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    a.scales = scales;
    constexpr int kBlockBytes = FMT == 0 ? 32 : 16;
    for (int i = 0; i < 2; ++i) {
        const uint64_t row_bytes = static_cast<uint64_t>(p.k / kBlock) * kBlockBytes;
        e = make_tmap_2d(&a.codes[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, p.codes[GATEUP ? i : 0], row_bytes,
                         static_cast<uint64_t>(p.experts) * p.n, row_bytes, kGroup * kBlockBytes, 64,
                         FMT == 0 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(tile_kernel<FMT, GATEUP>, dim3(static_cast<unsigned>(sms)), dim3(kThreads), smem, stream, a);
}

}  // namespace

cudaError_t moe_tile_waits(unsigned *bits, cudaStream_t stream) {
    return cudaMemcpyFromSymbolAsync(bits, lost_waits, sizeof(*bits), 0, cudaMemcpyDeviceToHost, stream);
}

cudaError_t moe_tile_launch(const MoeProduct &p, int above, uint8_t *operand, unsigned *err, cudaStream_t stream) {
    if (p.h != nullptr)
        return p.fmt == TQ_FMT_TERNARY2 ? launch<0, true>(p, above, operand, err, stream)
                                        : launch<1, true>(p, above, operand, err, stream);
    return p.fmt == TQ_FMT_TERNARY2 ? launch<0, false>(p, above, operand, err, stream)
                                    : launch<1, false>(p, above, operand, err, stream);
}

}  // namespace tq
