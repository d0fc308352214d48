// tq_q4_tile.cu -- products with 4-bit weights for many rows, on the 5th-generation tensor core.
//
// A tile is 128 weight rows (the A operand, decoded from their codes to bf16 c - 8, which is exact, straight
// into tensor memory) by up to 192 rows of x (the B operand, by TMA); gate/up: 64 rows of each, 16 and 16 in each
// quarter of the lanes.  A group's products add up in one of two accumulators in tensor memory;
// the fold reads it back and multiplies by the scales in fp32,
//   acc = fma(s, d, acc)   [acc = fma(8 s - b, sum of x over the group, acc)],
// while the tensor core works on the next group.  A lane is a weight row, so its scales are the thread's own
// and never leave its registers.  The sums of x come from a kernel of their own, through a workspace.
//
// Why the weights are A: with A in tensor memory an MMA takes N / 2 cycles for K = 16 from N = 32 on, and shared
// memory carries x alone.  With the weights as B, in shared memory, the decoded weights' stores (512 cycles per
// 128 values of k), the MMAs' reads (768) and
// the copies of x (256) share one 128-byte port: 3000 cycles per 256 rows and 128 values were measured, 1500 for
// 128 rows; here it is 1170, 704 of them MMAs (176 columns).
//
// Groups of 32 or 64 and many rows: a fold per group would take longer than the MMAs (an accumulator's hand-over
// and 192 columns: 990 cycles per group of 32, whose MMAs take 192).  There the scale goes into the weights, exactly:
// an fp16 scale is the sum of two bf16 of five bits, and five bits times c - 8 is exact in bf16, so two MMAs
// instead of one bring s (c - 8) x, and the fold adds up one accumulator per 128 values of k.  Minima are then a product
// of their own in the tensor core: (8 s - b) (sum of x) of the chunk's groups, both factors in three bf16 and six
// of the nine products, 6 values of k per group in one or two MMAs more.
//
// What bounds it (gate and up 17408 x 5120, 512 rows; cycles per 128 values of k by clocks around the waits).  Group
// 128 175 us, 1040 TFLOP/s: 1170 cycles of the issuing warp, 704 of them the MMAs' (176 columns: 512 rows are three
// tiles of 171), the others the latencies of its waits and commits one behind the other.  Groups of 32 256 us: the MMAs
// twice, 1408 of 1800; with minima 288, two more of 18.  Group 128 with minima 235: the fold reads every group's sums
// of x from shared memory, 64 of them in every lane, at 128 bytes per cycle.  Up to 64 rows: the issuing warp's
// latencies alone, 1020 to 1330 cycles with 128 to 256 of MMAs, while decode and fold wait (131072 x 5120
// by 32 rows 164 us at group 128, 212 at 32).
//
// Few tiles are split along k over the CTAs of a cluster, which add up their parts through shared memory.
//
// Warps: 0-7 decode (four for every other chunk of 128 values), 8 issues MMAs, 9 copies x, 10 its sums,
// 12-23 fold (a quarter of the lanes and a third of the columns each).
#include <cuda_runtime.h>

#include "tq_device.cuh"
#include "tq_launch.h"
#include "tq_q4_internal.h"
#include "tq_tcgen05.cuh"
#include "tq_tmap.h"

namespace tq {
namespace {

constexpr int kCols = kQ4TileCols;              // most rows of x per tile
constexpr int kABufs = 4;                       // of decoded weights: 64 values of k, 32 columns of tensor memory each
constexpr int kStages = 4;                      // of x in shared memory: 128 values each, in two halves
constexpr int kMaxSets = 3;                     // of accumulators
constexpr int kFoldWarps = 12;
constexpr int kFoldCols = kCols / (kFoldWarps / 4);
constexpr int kDecodeWarps = 8;
constexpr int kFirstFold = kDecodeWarps + 4;
constexpr int kThreads = 32 * (kFirstFold + kFoldWarps);
constexpr uint32_t kHalfBytes = kCols * 128;     // of a stage: 64 values
constexpr uint32_t kTmemA = 2 * kCols;
constexpr uint32_t kTmemMins = kQ4ScaledCols;   // 16 columns behind either accumulator's, where scaled weights have minima
constexpr int kAhead = 16;                      // chunks of codes in L2 ahead of the decode
constexpr int kPartLd = 128 + 4;                // floats per row of x of a part

// Register shares (launched with 80 per thread): 128 x (2 x 64 + 32 + 3 x 104) and 128 x (2 x 72 + 32 + 3 x 96) are less
// than 768 x 80.  `light`: the fold has one scale per chunk or none.  (us, 56 and 112, 64 and 104, 72 and 96: gate/up of
// 512 rows, scaled 292 - 254; group 128 186 177 176, with minima 252 234 272; 32 x 131072 x 5120 group 128 164 170 164,
// group 32 216 212 227; 64 rows, group 64 with minima 285 268 283.)
constexpr int kRegsIssue = 32;
constexpr int regs_decode(bool light) { return light ? 72 : 64; }
constexpr int regs_fold(bool light) { return light ? 96 : 104; }

__device__ unsigned lost_waits;                 // bits of all waits that have run out on this device
// The launch that the last of them was in.  CTAs of it that start later copy nothing and give up at their first
// wait, so that the launch ends whatever its size.  (A graph's replays are one launch by this number: the first CTA
// clears it, and only CTAs that cannot run beside the first look.)
__device__ unsigned long long lost_grid = ~0ull;

struct __align__(1024) TileSmem {
    union {
        uint8_t x[kStages][2][kHalfBytes];
        float part[kCols][kPartLd];             // this CTA's sums, when a tile is split along k
    };
    union {
        float sums[kMaxSets][4][kCols];         // of x over a set's groups
        uint8_t parts[2][kCols * 64];           // or, with scaled weights, their parts: a chunk's 32 per row
    };
    uint64_t x_full[kStages], x_empty[kStages], a_full[kABufs], a_empty[kABufs], d_full[kMaxSets], d_empty[kMaxSets];
    uint64_t s_full[kMaxSets], s_empty[kMaxSets], p_full[2], p_empty[2], m_full[2], drain;
    uint32_t tmem;
    uint32_t dead;                              // a bounded wait ran out
};

struct TileArgs {
    Q4Product p;
    CUtensorMap x;                              // [m][k] bf16, boxes of a tile's rows x 64 values
    CUtensorMap parts;                          // [m][k / 128 * 32] bf16, boxes of a tile's rows x 32
    const float *sums;                          // [k / group][sums_ld]: sums of x over the groups, where there are minima
    int64_t sums_ld;
    int tiles;                                  // of the weights
    int row_tiles, rows;                        // rows of x per tile
    bool scaled;
    int split;                                  // CTAs along k
    int first;                                  // tile of this launch
    int at_once;                                // CTAs that can run at the same time
};

constexpr uint32_t idesc_bf16(int m, int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// The whole warp runs this, one thread issues: a branch around it would take the operands out of the uniform registers.
__device__ __forceinline__ void mma_bf16_ts(uint32_t issue, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{ .reg .pred p, q; setp.ne.b32 p, %4, 0; setp.ne.b32 q, %5, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(issue)
        : "memory");
}

__device__ __forceinline__ void commit_if(uint32_t issue, uint32_t bar) {
    asm volatile(
        "{ .reg .pred q; setp.ne.b32 q, %1, 0;\n"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(bar),
        "r"(issue)
        : "memory");
}

__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(e));
    return e;
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

__device__ __forceinline__ uint64_t desc_sw64(uint32_t saddr) {
    // the same with rows of 64 bytes: atoms of 512
    uint64_t d = static_cast<uint64_t>((saddr & 0x3ffffu) >> 4);
    d |= 1ull << 16;
    d |= static_cast<uint64_t>(512 >> 4) << 32;
    d |= 1ull << 46;
    d |= 4ull << 61;
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

// 32 lanes x 16 columns, as pairs of neighbouring columns.  The wait is part of it: nothing reads the registers before.
__device__ __forceinline__ void ld_16(uint32_t taddr, uint64_t (&x)[8]) {
    asm volatile(
        "{ .reg .b32 t<16>;\n"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {t0,t1,t2,t3,t4,t5,t6,t7,t8,t9,t10,t11,t12,t13,t14,t15}, [%8];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        "mov.b64 %0, {t0,t1}; mov.b64 %1, {t2,t3}; mov.b64 %2, {t4,t5}; mov.b64 %3, {t6,t7};\n"
        "mov.b64 %4, {t8,t9}; mov.b64 %5, {t10,t11}; mov.b64 %6, {t12,t13}; mov.b64 %7, {t14,t15}; }"
        : "=l"(x[0]), "=l"(x[1]), "=l"(x[2]), "=l"(x[3]), "=l"(x[4]), "=l"(x[5]), "=l"(x[6]), "=l"(x[7])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void st_16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ float half2of(uint64_t v, int j) { return __uint_as_float(static_cast<uint32_t>(j ? v >> 32 : v)); }

__device__ __forceinline__ unsigned long long grid_id() {
    unsigned long long g;
    asm volatile("mov.u64 %0, %%gridid;" : "=l"(g));
    return g;
}

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
// Waits, and says whether the CTA is still alive.
template <int SLEEP = 0>
__device__ __forceinline__ bool wait_alive(TileSmem &sm, uint32_t bar, uint32_t parity, unsigned bit) {
    if (mbar_try_wait(bar, parity)) return true;
    wait_slow<SLEEP>(sm, bar, parity, bit);
    return *reinterpret_cast<volatile uint32_t *>(&sm.dead) == 0;
}
// The same for a whole warp: one answer.  Lanes may wait for different barriers; what any of them announces is there for
// all lanes behind __syncwarp, which orders memory between them (a vote does not).
template <int SLEEP = 0>
__device__ __forceinline__ bool warp_wait(TileSmem &sm, uint32_t bar, uint32_t parity, unsigned bit) {
    const bool ok = __all_sync(0xffffffffu, wait_alive<SLEEP>(sm, bar, parity, bit));
    __syncwarp();
    return ok;
}

// A wait for a copy in flight at the CTA's end, bounded from t0 on: all of its copies together have the time of one.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, long long t0) {
    while (!mbar_try_wait(bar, parity))
        if (clock64() - t0 > kWaitBudgetCycles) {
            atomicOr(&lost_waits, 1u << 6);
            return;
        }
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

// A float of CTA `rank`'s shared memory.
__device__ __forceinline__ float ld_part(uint32_t addr, uint32_t rank, int cluster) {
    float v;
    if (cluster == 1) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    else
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

__device__ __forceinline__ void lds128(uint32_t at, uint64_t &a, uint64_t &b) {
    asm volatile("ld.shared.v2.b64 {%0,%1}, [%2];" : "=l"(a), "=l"(b) : "r"(at) : "memory");
}

// PER scales (or minima) of one row.
template <int PER>
__device__ __forceinline__ void load_scales(uint32_t (&v)[(PER + 1) / 2], const uint16_t *p) {
    if constexpr (PER == 1) {
        uint16_t h;
        asm volatile("ld.global.u16 %0, [%1];" : "=h"(h) : "l"(p));
        v[0] = h;
    } else if constexpr (PER == 2) {
        asm volatile("ld.global.u32 %0, [%1];" : "=r"(v[0]) : "l"(p));
    } else {
        asm volatile("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "l"(p));
    }
}
template <int N>
__device__ __forceinline__ float scale_at(const uint32_t (&v)[N], int e) {
    const uint32_t w = N == 2 && e >= 2 ? v[N - 1] : v[0];
    return f16_bits_to_f32(static_cast<uint16_t>(e & 1 ? w >> 16 : w & 0xffffu));
}

// A scale as the sum of two bf16 of five bits each, twice each: times c - 8 either is exact in bf16.  (fp16 has 11
// bits; what rounding to five leaves is at most half of the fifth's unit, so five bits and a sign.)
__device__ __forceinline__ void split_scale(float s, uint32_t &hi, uint32_t &lo) {
    const uint32_t u = __float_as_uint(s);
    const bool finite = (u & 0x7f800000u) != 0x7f800000u;
    const uint32_t h = finite ? (u + 0x40000u) & 0xfff80000u : u;
    const uint32_t l = finite ? __float_as_uint(s - __uint_as_float(h)) : 0u;
    hi = __byte_perm(h, h, 0x3232);
    lo = __byte_perm(l, l, 0x3232);
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The sum of x over a group and 8 s - b, each as three bf16 (24 bits), and six of their products: all but 2^-24 of
// the whole one (the second part is up to 2^-8 of the first's unit, the third 2^-17: 2 * 2^-8 * 2^-17).
__device__ __forceinline__ void split_parts(float v, uint32_t (&p)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        p[i] = f32_to_bf16_bits(v);
        v -= __uint_as_float(p[i] << 16);
    }
}
// Of the weights: 1 1, 2 1, 2 3.
__device__ __forceinline__ void weight_parts(float v, uint32_t (&w)[3]) {
    uint32_t p[3];
    split_parts(v, p);
    w[0] = p[0] | p[0] << 16;
    w[1] = p[1] | p[0] << 16;
    w[2] = p[1] | p[2] << 16;
}
// Of x: 1 2, 1 3, 2 1.
__device__ __forceinline__ void sum_parts(float v, uint32_t (&w)[3]) {
    uint32_t p[3];
    split_parts(v, p);
    w[0] = p[0] | p[1] << 16;
    w[1] = p[0] | p[2] << 16;
    w[2] = p[1] | p[0] << 16;
}

template <int GROUP, bool MINS, bool GATEUP, bool SCALED>
__global__ void __launch_bounds__(kThreads, 1) q4_tile_kernel(const __grid_constant__ TileArgs args) {
    extern __shared__ uint8_t smem_raw[];
    TileSmem &sm = *reinterpret_cast<TileSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const Q4Product &p = args.p;
    constexpr int kPer = 128 / GROUP;                               // groups per chunk
    constexpr int kOut = GATEUP ? 64 : 128;                         // outputs per tile
    constexpr bool kLight = SCALED || (GROUP == 128 && !MINS);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int chunks = p.k >> 7;
    const int rank = blockIdx.x % args.split, tile = args.first + blockIdx.x / args.split;
    const int row0 = tile % args.row_tiles * args.rows, ntile = tile / args.row_tiles;
    const int rows = min(args.rows, p.m - row0), cols = (rows + 15) / 16 * 16;      // (args.rows: a multiple of 16)
    const int chunk0 = rank * chunks / args.split, chunk1 = (rank + 1) * chunks / args.split;
    const int total = chunk1 - chunk0;                              // chunks of this CTA
    // Accumulators change hands as sets of some of a chunk's groups, one set being added to while the fold has others; a
    // hand-over costs some 300 cycles on either side.  Up to 64 rows of x there are three sets of 128
    // columns, each folded by a third of the warps; else two of 192, all warps having a third of the columns.
    const int dcols = (cols + 31) / 32 * 32, teams = cols <= kFoldCols ? 3 : 1;
    const int sets = teams == 3 ? 3 : 2, set_cols = SCALED && MINS && teams == 3 ? 96 : 2 * kCols / sets;
    const int per_set = SCALED || kPer * dcols <= set_cols ? kPer : kPer == 4 && 2 * dcols <= set_cols ? 2 : 1;

    // (asked for here, so that the answer is there when the copies begin)
    unsigned long long lost = ~0ull;
    if (static_cast<int>(blockIdx.x) >= args.at_once && (warp == kDecodeWarps + 1 || warp == kDecodeWarps + 2))
        lost = *const_cast<volatile unsigned long long *>(&lost_grid);
    if (warp == kDecodeWarps) {
        tmem_alloc(smem_u32(&sm.tmem), 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&sm.x_full[i]), 1);
            mbar_init(smem_u32(&sm.x_empty[i]), 1);
        }
        for (int i = 0; i < kABufs; ++i) {
            mbar_init(smem_u32(&sm.a_full[i]), 4);
            mbar_init(smem_u32(&sm.a_empty[i]), 1);
        }
        for (int i = 0; i < kMaxSets; ++i) {
            mbar_init(smem_u32(&sm.d_full[i]), 1);
            mbar_init(smem_u32(&sm.d_empty[i]), kFoldWarps / teams);
            mbar_init(smem_u32(&sm.s_full[i]), 1);
            mbar_init(smem_u32(&sm.s_empty[i]), kFoldWarps / teams);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sm.p_full[i]), 1);
            mbar_init(smem_u32(&sm.p_empty[i]), 1);
            mbar_init(smem_u32(&sm.m_full[i]), 4);
        }
        mbar_init(smem_u32(&sm.drain), 1);
        sm.dead = 0;
        mbar_init_fence();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    // The weight row of this thread's lane of tensor memory (decode and fold): a quarter of the lanes is two
    // strips, gate and up of one or two neighbours.  Behind the last strip: the last one, whose results go nowhere.
    const int quarter = warp & 3, mat = GATEUP ? lane >> 4 : 0;
    const int64_t strips = q4_strips(p.n), first_strip = static_cast<int64_t>(ntile) * (GATEUP ? 4 : 8);
    const int64_t strip = min(first_strip + (GATEUP ? quarter : 2 * quarter + (lane >> 4)), strips - 1);
    const int64_t block0 = strip * chunks + chunk0;
    // Packed codes come to L2 well ahead of the decode's loads, which have a chunk or two in flight.
    auto ask = [&](int from, int to) {
        to = min(to, total);
        if (warp < kDecodeWarps && (lane & 15) == 0 && from < to)
            prefetch_l2(p.codes[mat] + (block0 + from) * kQ4ChunkBytes, (to - from) * kQ4ChunkBytes);
    };
    if (warp < 4) ask(0, kAhead);
    pdl_launch_dependents();
    pdl_wait();

    if (SCALED && warp < kDecodeWarps) {
        // ---- decode with scales: 32 values' two parts a buffer, two buffers of every chunk for either four warps ----
        regs_down<regs_decode(kLight)>();
        const int second = warp >> 2;                               // half of the chunk
        const uint8_t *src = p.codes[mat] + block0 * kQ4ChunkBytes + ((lane >> 3) & 1) * 512 + (lane & 7) * 64 + second * 8;
        const uint16_t *ssrc = p.scales[mat] + (block0 * 8 + (lane & 7)) * (2 * kPer) + ((lane >> 3) & 1) * kPer;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16), a_at = lanes + kTmemA + second * 64;
        const uint32_t empty = smem_u32(sm.a_empty) + second * 16, a_full = smem_u32(sm.a_full) + second * 16;
        uint32_t mask = 0x000f000fu, base = 0x43004300u;
        asm volatile("" : "+r"(mask), "+r"(base));
        const uint16_t *msrc = MINS ? p.mins[mat] + (ssrc - p.scales[mat]) : nullptr;
        constexpr int kWords = (kPer + 1) / 2;
        uint2 code[4];
        uint32_t sc[kWords], mn[kWords], sc_next[kWords], mn_next[kWords];
        auto load = [&](int c) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                asm volatile("ld.global.v2.u32 {%0,%1}, [%2];"
                             : "=r"(code[q].x), "=r"(code[q].y)
                             : "l"(src + static_cast<int64_t>(c) * kQ4ChunkBytes + q * 16));
        };
        auto load_row = [&](int c) {
            load_scales<kPer>(sc_next, ssrc + static_cast<int64_t>(c) * (16 * kPer));
            if (MINS) load_scales<kPer>(mn_next, msrc + static_cast<int64_t>(c) * (16 * kPer));
        };
        load(0);
        load_row(0);
        bool ok = true;
        uint32_t turn = 1;
        for (int c = 0; c < total && ok; ++c, turn ^= 1) {
            if (second == 0 && c % 4 == 0) ask(c + kAhead, c + kAhead + 4);
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                sc[i] = sc_next[i];
                if (MINS) mn[i] = mn_next[i];
            }
            if (c + 1 < total) load_row(c + 1);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                ok = warp_wait<32>(sm, empty + 8 * g, turn, 1u << 0);
                if (!ok) break;
                tc_fence_after();
                // (group 64: one scale of the pair for each half of the chunk; 32: one of its half's pair for each buffer)
                const uint32_t two = kPer == 4 && second ? sc[kWords - 1] : sc[0];
                uint32_t hi, lo;
                split_scale(f16_bits_to_f32(static_cast<uint16_t>((kPer == 4 ? g : second) ? two >> 16 : two & 0xffffu)), hi, lo);
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    uint32_t v[16];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[4 * q + i] = mul_bf16x2(decode_pair(g ? code[q].y : code[q].x, i, mask, base), part ? lo : hi);
                    st_16(a_at + 32 * g + 16 * part, v);
                }
                if (g == 1 && c + 1 < total) load(c + 1);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(a_full + 8 * g);
            }
            if constexpr (MINS) {
                // the minima: every other chunk's for either four warps
                if (!ok) break;
                if (second == (c & 1)) {
                    ok = warp_wait<32>(sm, smem_u32(&sm.p_empty[second]), (c >> 1 & 1) ^ 1, 1u << 0);
                    if (!ok) break;
                    uint32_t extra[16];
#pragma unroll
                    for (int e = 0; e < kPer; ++e) {
                        uint32_t w[3];
                        weight_parts(__fmaf_rn(8.0f, scale_at(sc, e), -scale_at(mn, e)), w);
                        extra[3 * e] = w[0];
                        extra[3 * e + 1] = w[1];
                        extra[3 * e + 2] = w[2];
                    }
#pragma unroll
                    for (int i = 3 * kPer; i < 16; ++i) extra[i] = 0;
                    tc_fence_after();
                    st_16(lanes + kTmemMins + second * kCols, extra);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sm.m_full[second]));
                }
            }
        }
    } else if (warp < kDecodeWarps) {
        // ---- decode: a lane's 128 codes of a chunk are 64 bytes, two halves of them one buffer each ----
        regs_down<regs_decode(kLight)>();
        const int odd = warp >> 2;                                  // which chunks
        const uint8_t *src = p.codes[mat] + block0 * kQ4ChunkBytes + ((lane >> 3) & 1) * 512 + (lane & 7) * 64;
        const uint32_t a_at = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + kTmemA + odd * 64;
        const uint32_t empty = smem_u32(sm.a_empty) + odd * 16, a_full = smem_u32(sm.a_full) + odd * 16;
        uint32_t mask = 0x000f000fu, base = 0x43004300u;
        asm volatile("" : "+r"(mask), "+r"(base));                  // in registers: two constants do not fit one instruction
        uint4 code[4];
        auto load = [&](int c) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(code[q].x), "=r"(code[q].y), "=r"(code[q].z), "=r"(code[q].w)
                             : "l"(src + static_cast<int64_t>(c) * kQ4ChunkBytes + q * 16));
        };
        if (odd < total) load(odd);
        bool ok = true;
        uint32_t turn = 1;
        for (int c = odd; c < total && ok; c += 2, turn ^= 1) {
            if (c % 4 == 0) ask(c + kAhead, c + kAhead + 4);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                ok = warp_wait<32>(sm, empty + 8 * half, turn, 1u << 0);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    // 32 values: word g of each quarter of them
                    uint32_t v[16];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t w = half ? (g ? code[q].w : code[q].z) : (g ? code[q].y : code[q].x);
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[4 * q + i] = decode_pair(w, i, mask, base);
                    }
                    st_16(a_at + half * 32 + 16 * g, v);
                }
                if (half == 1 && c + 2 < total) load(c + 2);        // the other four warps decode meanwhile
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(a_full + 8 * half);
            }
        }
    } else if (warp < kFirstFold) {
        regs_down<kRegsIssue>();
        const bool give_up = lost != ~0ull && lost == grid_id();
        if (give_up) *reinterpret_cast<volatile uint32_t *>(&sm.dead) = 1;
        const int copied = give_up ? 0 : total;                     // chunks
        if (warp == kDecodeWarps) {
            // ---- issue: one thread issues, the warp stays together ----
            const uint32_t issue = elect_one();
            const uint32_t idesc = idesc_bf16(128, cols);
            const uint32_t x_full = smem_u32(sm.x_full), x_empty = smem_u32(sm.x_empty);
            const uint32_t a_full = smem_u32(sm.a_full), a_empty = smem_u32(sm.a_empty);
            const uint32_t d_full = smem_u32(sm.d_full), d_empty = smem_u32(sm.d_empty);
            const uint64_t x_desc = desc_sw128(smem_u32(sm.x));
            // (tensor memory is this CTA's as a whole, so its columns count from 0)
            uint32_t turn = 0, set = 0, d_turn = 1, d_set = 0, x_at = 0, x_turn = 0;
            uint64_t x_set = x_desc;
            bool ok = true;
            if constexpr (SCALED) {
                const uint32_t p_full = smem_u32(sm.p_full), p_empty = smem_u32(sm.p_empty), m_full = smem_u32(sm.m_full);
                const uint64_t p_desc = desc_sw64(smem_u32(sm.parts));
                for (int c = 0; c < total && ok; ++c, turn ^= 1) {
                    ok = wait_alive(sm, x_full + 8 * x_at, x_turn, 1u << 1) && wait_alive(sm, d_empty + 8 * set, d_turn, 1u << 3);
#pragma unroll
                    for (int ring = 0; ring < kABufs; ++ring) {
                        ok = ok && wait_alive(sm, a_full + 8 * ring, turn, 1u << 2);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int i = 0; i < 4; ++i)                 // (both parts: the same values of x)
                            mma_bf16_ts(issue, d_set, kTmemA + 32 * ring + 8 * i,
                                        x_set + (ring / 2 * (kHalfBytes >> 4) + 4 * (ring % 2) + 2 * (i % 2)), idesc, ring + i > 0);
                        commit_if(issue, a_empty + 8 * ring);
                    }
                    if (!ok) break;
                    if constexpr (MINS) {
                        // the minima: 6 values per group, 24 or 12 of 32
                        const uint32_t at = c & 1, phase = c >> 1 & 1;
                        ok = wait_alive(sm, p_full + 8 * at, phase, 1u << 7) && wait_alive(sm, m_full + 8 * at, phase, 1u << 2);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int i = 0; i < kPer / 2; ++i)
                            mma_bf16_ts(issue, d_set, kTmemMins + at * kCols + 8 * i, p_desc + (at * (kCols * 64 >> 4) + 2 * i), idesc, 1);
                        commit_if(issue, p_empty + 8 * at);
                    }
                    commit_if(issue, d_full + 8 * set);
                    d_set += set_cols;
                    if (++set == sets) {
                        set = d_set = 0;
                        d_turn ^= 1;
                    }
                    commit_if(issue, x_empty + 8 * x_at);
                    x_set += 2 * kHalfBytes >> 4;
                    if (++x_at == kStages) {
                        x_at = 0;
                        x_set = x_desc;
                        x_turn ^= 1;
                    }
                }
            }
            for (int c0 = 0; !SCALED && c0 < total && ok; c0 += 2, turn ^= 1) {
#pragma unroll
                for (int ring = 0; ring < kABufs; ++ring) {
                    if (c0 + ring / 2 >= total || !ok) break;
                    constexpr int kSubs = GROUP == 32 ? 2 : 1, kEach = 4 / kSubs;
                    const bool start = GROUP < 128 || ring % 2 == 0, end = GROUP < 128 || ring % 2 == 1;
                    if (ring % 2 == 0) ok = wait_alive(sm, x_full + 8 * x_at, x_turn, 1u << 1);
                    ok = ok && wait_alive(sm, a_full + 8 * ring, turn, 1u << 2);
#pragma unroll
                    for (int sub = 0; sub < kSubs; ++sub) {
                        // group e of the chunk, place `in` of its set
                        const int e = GROUP == 128 ? 0 : ring % 2 * kSubs + sub, in = e & (per_set - 1);
                        if (start && in == 0) ok = ok && wait_alive(sm, d_empty + 8 * set, d_turn, 1u << 3);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t d = d_set + in * dcols;
#pragma unroll
                        for (int i = sub * kEach; i < (sub + 1) * kEach; ++i)
                            mma_bf16_ts(issue, d, kTmemA + 32 * ring + 8 * i, x_set + (ring % 2 * (kHalfBytes >> 4) + 2 * i), idesc,
                                        !(start && i == sub * kEach));
                        if (end && in == per_set - 1) {
                            commit_if(issue, d_full + 8 * set);
                            d_set += set_cols;
                            if (++set == sets) {
                                set = d_set = 0;
                                d_turn ^= 1;
                            }
                        }
                    }
                    if (!ok) break;
                    commit_if(issue, a_empty + 8 * ring);
                    if (ring % 2 == 1) {
                        commit_if(issue, x_empty + 8 * x_at);
                        x_set += 2 * kHalfBytes >> 4;
                        if (++x_at == kStages) {
                            x_at = 0;
                            x_set = x_desc;
                            x_turn ^= 1;
                        }
                    }
                }
            }
            __syncwarp();
            commit_if(issue, smem_u32(&sm.drain));
            if (!mbar_wait(smem_u32(&sm.drain), 0) && issue) atomicOr(&lost_waits, 1u << 4);
            __syncwarp();
        } else if (warp == kDecodeWarps + 1) {
            // ---- copies of x: one thread ----
            if (lane == 0) {
                int c = 0;
                for (; c < copied; ++c) {
                    const int ring = c % kStages;
                    if (!wait_alive<32>(sm, smem_u32(&sm.x_empty[ring]), ((c / kStages) & 1) ^ 1, 1u << 5)) break;
                    const uint32_t bar = smem_u32(&sm.x_full[ring]);
                    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(args.rows) * 256);
                    load_box(smem_u32(sm.x[ring][0]), &args.x, (chunk0 + c) * 128, row0, bar);
                    load_box(smem_u32(sm.x[ring][1]), &args.x, (chunk0 + c) * 128 + 64, row0, bar);
                }
                // none of this CTA's copies may be in flight when it leaves
                const long long t0 = clock64();
                for (int j = max(c - kStages, 0); j < c; ++j) drain_wait(smem_u32(&sm.x_full[j % kStages]), (j / kStages) & 1, t0);
            }
            __syncwarp();
        } else if (warp == kDecodeWarps + 2 && MINS) {
            // ---- copies of the sums, or of their parts ----
            if (SCALED && lane == 0) {
                int c = 0;
                for (; c < copied; ++c) {
                    if (!wait_alive<64>(sm, smem_u32(&sm.p_empty[c & 1]), (c >> 1 & 1) ^ 1, 1u << 9)) break;
                    const uint32_t bar = smem_u32(&sm.p_full[c & 1]);
                    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(args.rows) * 64);
                    load_box(smem_u32(sm.parts[c & 1]), &args.parts, (chunk0 + c) * 32, row0, bar);
                }
                const long long t0 = clock64();
                for (int j = max(c - 2, 0); j < c; ++j) drain_wait(smem_u32(&sm.p_full[j & 1]), j >> 1 & 1, t0);
            } else if (lane == 0) {
                const float *src = args.sums + static_cast<int64_t>(chunk0) * kPer * args.sums_ld + row0;
                int set = 0, turn = 1, g = 0;
                for (; g < copied * kPer; g += per_set) {
                    if (!wait_alive<64>(sm, smem_u32(&sm.s_empty[set]), turn, 1u << 9)) break;
                    const uint32_t bar = smem_u32(&sm.s_full[set]);
                    mbar_arrive_expect_tx(bar, per_set * cols * 4);
                    for (int e = 0; e < per_set; ++e)
                        bulk_copy_g2s(smem_u32(sm.sums[set][e]), src + static_cast<int64_t>(g + e) * args.sums_ld, cols * 4, bar);
                    if (++set == sets) {
                        set = 0;
                        turn ^= 1;
                    }
                }
                const long long t0 = clock64();
                for (int j = max(g / per_set - sets, 0); j < g / per_set; ++j) drain_wait(smem_u32(&sm.s_full[j % sets]), (j / sets) & 1, t0);
            }
            __syncwarp();
        } else if (warp == kFirstFold - 1) {
            if (blockIdx.x == 0 && lane == 0) atomicCAS(&lost_grid, grid_id(), ~0ull);
            __syncwarp();
        }
        __syncwarp();
    } else {
        // ---- fold: a lane is a weight row, a warp has a third of the rows of x ----
        regs_up<regs_fold(kLight)>();
        const int third = (warp - kFirstFold) / 4, team = teams > 1 ? third : 0;
        const int col0 = teams > 1 ? 0 : third * kFoldCols, mine = min(max(cols - col0, 0), kFoldCols);
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + col0;
        const int64_t sat = (block0 * 8 + (lane & 7)) * (2 * kPer) + ((lane >> 3) & 1) * kPer;
        const uint16_t *ssrc = p.scales[mat] + sat, *msrc = MINS ? p.mins[mat] + sat : nullptr;
        uint64_t acc[kFoldCols / 2];
#pragma unroll
        for (int i = 0; i < kFoldCols / 2; ++i) acc[i] = 0;
        constexpr int kWords = (kPer + 1) / 2;
        uint32_t sc[kWords], next[kWords], mn[kWords], mnext[kWords];
        const int shift = kPer / per_set >> 1, all = total << shift;           // sets (1, 2 or 4 of a chunk)
        const uint32_t d_full = smem_u32(sm.d_full), d_empty = smem_u32(sm.d_empty);
        const uint32_t s_full = smem_u32(sm.s_full), s_empty = smem_u32(sm.s_empty);
        auto ahead = [&](int i) {                                   // the scales of set i's chunk
            if (SCALED || i >= all) return;
            const int64_t at = static_cast<int64_t>(i >> shift) * (16 * kPer);
            load_scales<kPer>(next, ssrc + at);
            if (MINS) load_scales<kPer>(mnext, msrc + at);
        };
        ahead(team);
        uint32_t set = team, turn = 0;
#pragma unroll 1
        for (int i = team; i < all; i += teams) {
#pragma unroll
            for (int j = 0; j < kWords; ++j) {
                sc[j] = next[j];
                if (MINS) mn[j] = mnext[j];
            }
            ahead(i + teams);
            const bool sums_lane = MINS && !SCALED && (lane & 1);              // both waits at once
            if (!warp_wait<20>(sm, (sums_lane ? s_full : d_full) + 8 * set, turn, sums_lane ? 1u << 7 : 1u << 8)) break;
            tc_fence_after();
            if (SCALED) {
                const uint32_t d = lane_base + set * set_cols;
                const uint64_t one = pack2(1.0f, 1.0f);
#pragma unroll
                for (int q = 0; q < kFoldCols / 16; ++q) {
                    if (16 * q >= mine) break;
                    uint64_t x[8];
                    ld_16(d + 16 * q, x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[8 * q + j] = fma2(x[j], one, acc[8 * q + j]);
                }
            }
#pragma unroll 1
            for (int in = 0; in < (SCALED ? 0 : per_set); ++in) {
                const int e = (i & ((1 << shift) - 1)) * per_set + in;
                const float s = scale_at(sc, e);
                const uint64_t s2 = pack2(s, s);
                float m = 0.0f;
                if (MINS) m = __fmaf_rn(8.0f, s, -scale_at(mn, e));
                const uint64_t m2 = pack2(m, m);
                const uint32_t d = lane_base + set * set_cols + in * dcols;
                const uint32_t sums = smem_u32(sm.sums[set][in]) + col0 * 4;
#pragma unroll
                for (int q = 0; q < kFoldCols / 16; ++q) {
                    if (16 * q >= mine) break;
                    uint64_t x[8];
                    ld_16(d + 16 * q, x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[8 * q + j] = fma2(x[j], s2, acc[8 * q + j]);
                    if (MINS) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint64_t x0, x1;
                            lds128(sums + 64 * q + 16 * j, x0, x1);
                            acc[8 * q + 2 * j] = fma2(x0, m2, acc[8 * q + 2 * j]);
                            acc[8 * q + 2 * j + 1] = fma2(x1, m2, acc[8 * q + 2 * j + 1]);
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(d_empty + 8 * set);
                if (MINS && !SCALED) mbar_arrive(s_empty + 8 * set);
            }
            if (teams == 3) {                                       // (set i % 3 is the team's own)
                turn ^= 1;
            } else if (++set == sets) {
                set = 0;
                turn ^= 1;
            }
        }
        const int local = 32 * quarter + lane;                      // row of the tile
        if (args.split > 1 || teams > 1) {
            // the stages hold this CTA's parts now: no copy or MMA uses them once all teams are here
            named_barrier(1, 32 * kFoldWarps);
#pragma unroll
            for (int i = 0; i < kFoldCols; ++i)
                if (i < mine) sm.part[(teams > 1 ? team * kFoldCols : col0) + i][local] = half2of(acc[i >> 1], i & 1);
            if (teams > 1) {
                named_barrier(1, 32 * kFoldWarps);
                for (int o = tid - 32 * kFirstFold; o < rows * 128; o += 32 * kFoldWarps) {
                    float *at = &sm.part[o >> 7][o & 127];
                    *at = *at + at[kFoldCols * kPartLd] + at[2 * kFoldCols * kPartLd];
                }
            }
            if (args.split > 1) cluster_sync();
            else named_barrier(1, 32 * kFoldWarps);
            const int o0 = rank * kOut / args.split, width = (rank + 1) * kOut / args.split - o0;
            const uint32_t base = smem_u32(sm.part);
            for (int o = tid - 32 * kFirstFold; o < rows * width; o += 32 * kFoldWarps) {
                const int r = o / width, e = o0 + o - r * width;
                const int64_t out = static_cast<int64_t>(ntile) * kOut + e;
                if (out >= p.n) continue;
                // gate/up: output e of the tile is lane 32 (e / 16) + e % 16, its up 16 lanes on
                const uint32_t at = base + static_cast<uint32_t>(r * kPartLd + (GATEUP ? (e >> 4) * 32 + (e & 15) : e)) * 4;
                float vs[8], us[8], v = 0.0f, u = 0.0f;
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    if (s < args.split) {
                        vs[s] = ld_part(at, s, args.split);
                        if (GATEUP) us[s] = ld_part(at + 64, s, args.split);
                    }
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    if (s < args.split) {
                        v += vs[s];
                        if (GATEUP) u += us[s];
                    }
                const int64_t to = static_cast<int64_t>(row0 + r) * p.n + out;
                if (GATEUP) v = __fmul_rn(tq_silu(v), u);
                if (GATEUP || p.y_bf16) static_cast<uint16_t *>(p.y)[to] = f32_to_bf16_bits(v);
                else static_cast<float *>(p.y)[to] = v;
            }
            if (args.split > 1) cluster_sync();
        } else {
            const int64_t out = static_cast<int64_t>(ntile) * kOut + (GATEUP ? 16 * quarter + (lane & 15) : local);
#pragma unroll
            for (int i = 0; i < kFoldCols / 2; ++i) {
                if (2 * i >= mine) break;
                float v[2] = {half2of(acc[i], 0), half2of(acc[i], 1)};
                if (GATEUP) {
                    // gate lanes take the first row of the pair, up lanes the second
                    const bool up = lane >= 16;
                    const float other = __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 16);
                    const float g = up ? other : v[0], u = up ? v[1] : other;
                    const int r = col0 + 2 * i + up;
                    if (r < rows && out < p.n)
                        static_cast<uint16_t *>(p.y)[static_cast<int64_t>(row0 + r) * p.n + out] = f32_to_bf16_bits(__fmul_rn(tq_silu(g), u));
                } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int r = col0 + 2 * i + j;
                        if (r >= rows || out >= p.n) continue;
                        const int64_t to = static_cast<int64_t>(row0 + r) * p.n + out;
                        if (p.y_bf16) static_cast<uint16_t *>(p.y)[to] = f32_to_bf16_bits(v[j]);
                        else static_cast<float *>(p.y)[to] = v[j];
                    }
                }
            }
        }
    }
    if (warp < kFirstFold && args.split > 1) {
        cluster_sync();
        cluster_sync();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kDecodeWarps) tmem_dealloc(tmem, 512);
    // (here, before a later CTA has its place: in the waits it took the fold of small groups 4% more time)
    if (tid == 0 && sm.dead) atomicExch(&lost_grid, grid_id());
}

// Sums of x over the groups, a thread each: [k / group][ld] (rows from m on: zero), or with `parts` their six parts,
// [m][k / 128][32] (behind the last: zero).
__global__ void __launch_bounds__(256) q4_sums_kernel(const uint16_t *x, int m, int k, int group, int64_t ld, float *sums, uint32_t *parts) {
    pdl_launch_dependents();
    pdl_wait();
    const int per_row = k / group;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= ld * per_row) return;
    const int64_t row = i / per_row;
    const int g = static_cast<int>(i - row * per_row);
    float s = 0.0f;
    if (row < m)
        for (int j = 0; j < group / 8; ++j) {
            const uint4 v = *reinterpret_cast<const uint4 *>(x + row * k + g * group + j * 8);
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) s += __uint_as_float(u[e] << 16) + __uint_as_float(u[e] & 0xffff0000u);
        }
    if (parts == nullptr) {
        sums[g * ld + row] = s;
    } else if (row < m) {
        const int per = 128 / group, e = g % per;
        uint32_t w[3];
        sum_parts(s, w);
        uint32_t *out = parts + (row * (k / 128) + g / per) * 16;
#pragma unroll
        for (int i = 0; i < 3; ++i) out[3 * e + i] = w[i];
        for (int i = 3 * per + e; i < 16; i += per) out[i] = 0;
    }
}

template <int GROUP, bool MINS, bool GATEUP, bool SCALED>
cudaError_t launch(TileArgs &a, int dev, int sms, cudaStream_t stream) {
    constexpr size_t smem = sizeof(TileSmem) + 1024;
    static_assert(smem <= 227 * 1024, "shared memory");
    static SmemLimit limit;
    cudaError_t e = limit.raise(q4_tile_kernel<GROUP, MINS, GATEUP, SCALED>, smem);
    if (e != cudaSuccess) return e;
    const int tiles = a.tiles * a.row_tiles;
    const int chunks = a.p.k / 128;
    a.at_once = sms;
    // `count` tiles from a.first on, each split along k over as many CTAs as run at once with at least two chunks each.
    static ClusterLimit cluster_limit;
    auto some = [&](int count) {
        a.split = 1;
        for (int more = 2; more <= 8 && count * more <= sms && chunks >= 2 * more; ++more) {
            int most = 0;
            const cudaError_t e = cluster_limit.most(q4_tile_kernel<GROUP, MINS, GATEUP, SCALED>, dev, more, kThreads, smem, sms, &most);
            if (e != cudaSuccess) return e;
            if (count <= most) a.split = more;
        }
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(count) * a.split);
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
        return cudaLaunchKernelEx(&cfg, q4_tile_kernel<GROUP, MINS, GATEUP, SCALED>, a);
    };
    // A last round of up to half the SMs' tiles is a launch of its own, split along k; it waits for the rounds before.
    // (us, one launch and two: gate/up of 64 rows, 160 tiles, 5120 51 37, 2048 32 26, 1024 25 21; 32 x 20480 x 1024
    // group 128 with minima 25 22; 64 x 28672 x 4096, 224 tiles 46 40; gate/up of 512 rows, 816 tiles, 5120 190 187.)
    const int rest = tiles % sms;
    if (tiles > sms && rest > 0 && 2 * rest <= sms && chunks >= 8) {
        e = some(tiles - rest);
        if (e != cudaSuccess) return e;
        a.first = tiles - rest;
        return some(rest);
    }
    return some(tiles);
}

template <int GROUP, bool MINS, bool GATEUP>
cudaError_t pick(TileArgs &a, int dev, int sms, cudaStream_t stream) {
    if constexpr (GROUP < 128)
        if (a.scaled) return launch<GROUP, MINS, GATEUP, true>(a, dev, sms, stream);
    return launch<GROUP, MINS, GATEUP, false>(a, dev, sms, stream);
}

template <int GROUP>
cudaError_t pick(TileArgs &a, int dev, int sms, cudaStream_t stream) {
    const bool mins = a.p.mins[0] != nullptr;
    if (a.p.mats == 1) return mins ? pick<GROUP, true, false>(a, dev, sms, stream) : pick<GROUP, false, false>(a, dev, sms, stream);
    return mins ? pick<GROUP, true, true>(a, dev, sms, stream) : pick<GROUP, false, true>(a, dev, sms, stream);
}

}  // namespace

cudaError_t q4_tile_waits(unsigned *bits, cudaStream_t stream) {
    return cudaMemcpyFromSymbolAsync(bits, lost_waits, sizeof(*bits), 0, cudaMemcpyDeviceToHost, stream);
}

cudaError_t q4_tile_launch(const Q4Product &p, float *sums, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    TileArgs a{};
    a.p = p;
    const int per = p.mats == 2 ? 4 : 8;        // strips of each matrix in a tile
    a.tiles = static_cast<int>((q4_strips(p.n) + per - 1) / per);
    a.scaled = q4_scaled_call(p.m, p.group, p.mins[0] != nullptr, a.tiles, sms);
    a.rows = q4_tile_rows(p.m, a.scaled && p.mins[0] != nullptr ? kQ4ScaledCols : kCols);
    a.row_tiles = (p.m + a.rows - 1) / a.rows;
    if (p.mins[0] != nullptr) {
        uint32_t *parts = a.scaled ? reinterpret_cast<uint32_t *>(sums) : nullptr;
        a.sums = sums;
        a.sums_ld = q4_sums_ld(p.m);
        const int64_t entries = a.sums_ld * (p.k / p.group);
        e = launch_pdl(q4_sums_kernel, dim3(static_cast<unsigned>((entries + 255) / 256)), dim3(256), 0, stream, p.x, p.m, p.k,
                       p.group, a.sums_ld, sums, parts);
        if (e == cudaSuccess && parts != nullptr)
            e = make_tmap_2d(&a.parts, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, parts, static_cast<uint64_t>(p.k) / 4, static_cast<uint64_t>(p.m),
                             static_cast<uint64_t>(p.k) / 2, 32, static_cast<uint32_t>(a.rows), CU_TENSOR_MAP_SWIZZLE_64B);
        if (e != cudaSuccess) return e;
    }
    e = make_tmap_2d(&a.x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.x, static_cast<uint64_t>(p.k), static_cast<uint64_t>(p.m),
                     static_cast<uint64_t>(p.k) * 2, 64, static_cast<uint32_t>(a.rows), CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
    return p.group == 128 ? pick<128>(a, dev, sms, stream) : p.group == 64 ? pick<64>(a, dev, sms, stream) : pick<32>(a, dev, sms, stream);
}

}  // namespace tq
