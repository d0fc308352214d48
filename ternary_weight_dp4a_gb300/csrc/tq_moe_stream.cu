// tq_moe_stream.cu -- products grouped by expert for few rows per expert: the
// weights stream from HBM through registers into warp-level matrix
// instructions, the activations of up to 8 rows wait in shared memory.
//
// Mathematics.  A block dot d = sum w*q over 128 weights in {-1, 0, +1} and int8
// q is an exact integer below 2^14; fp16 operands hold both sides exactly and
// the matrix instruction (m16n8k16, the weights as its 16 rows) adds in fp32.
//   A weight's bits stay where they are in the word: masked out and joined with
//   the exponent of 1.0 they are the mantissa of 1 + v * 2^(p - 10), p the lowest
//   bit's place in its half word, one operation for two weights.  p is kept in
//   2 .. 9, where q * 2^(10 - p) is still an fp16 number (2-bit: the word itself, and
//   with its bytes changed in pairs; 1-bit: 4 .. 9, the word itself, and it shifted by
//   6 right and by 4 left).  The activation there is q * s, s = 2^(10 - p) (1-bit:
//   2^(11 - p)), so the product is q * s + q * v (1-bit: + 2 q v), and the sums over
//   q * s and over v's offset are known when the activations are laid out: with a
//   minus they are what the sum starts from.
//   2-bit: codes 0, 1, 2 become 0, 1, 3 (two operations for 16 codes); with their
//   upper bit inverted, in the masking operation, v = w + 2.   1-bit: w = 2 v - 1.
//   Everything is a whole number below 2^23.
// Per 128-block and output the kernel then adds one fma(d, scale_w * scale_a,
// acc), blocks in ascending order, the order that tq_moe.h documents.
//
// What bounds it.  With some rows for every expert the weights are read once and turned
// into fp16 once for eight rows; four masking operations and one matrix instruction per
// 512 weights share a scheduler at 10.5 cycles (8.0 for the matrix instruction by
// itself), what prepares and folds them comes on top: 267 (1-bit) and 313 (2-bit)
// cycles per warp for 32 weight rows and a block of 128.  Memory would take a quarter to
// a half of that: 8 tokens, top 4 of 32 experts, 5120 x 1536 take 22.8 us, two less with
// all weights in L2, 6.4 for the bytes.  16 rows at a time (two matrix instructions for a
// masked pair) gain 5% where experts have many rows and lose 22% where they have few.
//
// (fp8 operands would need fewer decode operations, but mma.sync on fp8 is
// emulated here: 11 instructions and 6.1 cycles per SM for m16n8k32, against
// 2.0 for a native fp16 m16n8k16.)
#include <cuda_runtime.h>

#include "tq_device.cuh"
#include "tq_launch.h"
#include "tq_moe_codes.cuh"
#include "tq_moe_internal.h"
#include "tq_tmap.h"

namespace tq {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kCols = 8;                     // activation rows per chunk
constexpr int kMaxWarps = 16;
constexpr int kSplitWarps = 8;

__device__ unsigned lost_waits;              // bits of all waits that have run out on this device

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

// Where pair i (0..15) of a lane's 32 weights sits: the weight of its lower half
// (the other is 8 or 16 further), and the place p of its lowest bit in the word that is masked.
template <int FMT>
__host__ __device__ constexpr int pair_weight(int i) {
    return FMT == 0 ? 16 * (i >> 3) + ((i & 7) + 1) % 8 : (i < 12 ? i + 4 : i - 12);
}
template <int FMT>
__host__ __device__ constexpr int pair_place(int i) {
    return FMT == 0 ? 2 + 2 * (i & 3) : 4 + i % 6;
}

// A lane's weights of one row and block, ready for masking: each word as it is, and
// (2-bit) with bytes 0, 1 and 2, 3 changed, (1-bit) shifted right by 6 and left by 4.
template <int FMT> struct Fields { uint32_t w[FMT == 0 ? 2 : 1][FMT == 0 ? 2 : 3]; };

template <int FMT>
__device__ __forceinline__ Fields<FMT> fields(const Codes<FMT> &c) {
    Fields<FMT> f;
#pragma unroll
    for (int i = 0; i < (FMT == 0 ? 2 : 1); ++i) {
        const uint32_t w = FMT == 0 ? c.w[i] | ((c.w[i] >> 1) & 0x55555555u) : c.w[i];       // codes 0, 1, 2 -> 0, 1, 3
        f.w[i][0] = w;
        if (FMT == 0) {
            f.w[i][1] = prmt(w, w, 0x2301u);
        } else {
            f.w[i][1] = w >> 6;
            f.w[i][FMT == 0 ? 1 : 2] = w << 4;
        }
    }
    return f;
}

// What joins the masked bits: the exponent of 1.0, and for 2-bit codes the inversion of
// the upper bit (one word for each place).  Kept in registers: lop3 takes one
// immediate, and as two immediates the compiler makes two instructions of it.
template <int FMT> struct Joins { uint32_t w[FMT == 0 ? 4 : 1]; };

template <int FMT>
__device__ __forceinline__ Joins<FMT> joins() {
    Joins<FMT> j;
#pragma unroll
    for (int i = 0; i < (FMT == 0 ? 4 : 1); ++i)
        asm volatile("mov.b32 %0, %1;" : "=r"(j.w[i]) : "r"(0x3c003c00u | (FMT == 0 ? 0x00020002u << (2 + 2 * i) : 0u)));
    return j;
}

// Pair i as two fp16 numbers.
template <int FMT>
__device__ __forceinline__ uint32_t weight_pair(const Fields<FMT> &f, const Joins<FMT> &join, int i) {
    const int p = pair_place<FMT>(i);
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;"                         // (field & mask) ^ join
        : "=r"(r)
        : "r"(FMT == 0 ? f.w[FMT == 0 ? i >> 3 : 0][(i & 7) / 4] : f.w[0][FMT == 0 ? 0 : i / 6]),
          "r"((FMT == 0 ? 0x00030003u : 0x00010001u) << p), "r"(join.w[FMT == 0 ? i & 3 : 0]));
    return r;
}

// What the activation of pair i is multiplied with.
template <int FMT>
__host__ __device__ constexpr int pair_scale(int i) { return 1 << ((FMT == 0 ? 10 : 11) - pair_place<FMT>(i)); }

// The same / 4 for four consecutive weights e .. e + 3, as bytes for dp4a.
template <int FMT>
__host__ __device__ constexpr uint32_t scale_bytes(int e) {
    uint32_t r = 0;
    for (int j = 0; j < 4; ++j)
        for (int i = 0; i < 16; ++i) {
            const int w = pair_weight<FMT>(i);
            if (w == e + j || w + (FMT == 0 ? 8 : 16) == e + j)
                r |= static_cast<uint32_t>(pair_scale<FMT>(i) / 4) << (8 * j);
        }
    return r;
}

// The first of a block's matrix instructions: it starts from the columns' start values.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1, float2 start) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(start.x), "f"(start.y));
}

// Two int8 codes (plus 128, picked from the bytes of a and b) as fp16, times s.
__device__ __forceinline__ uint32_t act_pair(uint32_t a, uint32_t b, uint32_t sel, int s) {
    const uint32_t u = prmt(prmt(a, b, sel), 0x64646464u, 0x4140u);                          // 0x64nn is 1024 + n
    __half2 h = *reinterpret_cast<const __half2 *>(&u);
    h = __hmul2(__hadd2(h, __half2half2(__ushort_as_half(0xe480))), __half2half2(__int2half_rn(s)));   // - 1152
    return *reinterpret_cast<const uint32_t *>(&h);
}

struct StreamArgs {
    MoeProduct p;
    int chunk;      // rows of an expert that share a pass over its weights, at most kCols
    int limit;      // experts with more rows are another kernel's
    unsigned *err;
    CUtensorMap codes[2];   // packed weights, [experts * n][row bytes], boxes of 16 rows x 4 blocks
};

// Shared memory of a CTA, behind one another (the rings only in the stream kernel):
//   per warp a ring of stages of four blocks: packed weights [32 rows][4 blocks], swizzled, and
//     behind all rings the stages' weight scales [32 rows][4] fp16 and barriers
//   offsets, chunks (of the experts before) int [experts + 1] each
//   activations fp16 [chunk][block][quarter][t][8]: the 32 of lane t in the order of its
//     weight pairs, 8 at a time; 64 bytes between rows
//   per two columns their scales and the values that their sums start from [block][4][4]
__host__ __device__ constexpr int list_bytes(int experts) { return (2 * (experts + 1) * 4 + 15) / 16 * 16; }
__host__ __device__ constexpr int row_pitch(int nb) { return nb * 256 + 64; }
constexpr int kStageBlocks = 4;
// stages per warp: 16 warps have 128 KB (1-bit: 96 KB) on their way on an SM
template <int FMT> constexpr int kDepth = FMT == 0 ? 2 : 3;
template <int FMT> constexpr int kStageBytes = 32 * kStageBlocks * (FMT == 0 ? 32 : 16);
template <int FMT> constexpr int kSideBytes = 32 * 8 + 16;           // a stage's scales, and its barrier

template <int FMT>
size_t stream_smem(int experts, int chunk, int nb, int warps) {
    return 1024 + static_cast<size_t>(warps) * kDepth<FMT> * (kStageBytes<FMT> + kSideBytes<FMT>) +
           static_cast<size_t>(list_bytes(experts)) + static_cast<size_t>(chunk) * row_pitch(nb) +
           static_cast<size_t>(nb) * kCols * 8;
}

// Fill offsets (clamped) and chunks (all threads); returns the number of chunks.
__device__ __forceinline__ int list_chunks(const MoeProduct &p, int chunk, int limit, int *offsets, int *chunks) {
    const int tid = threadIdx.x, lane = tid & 31;
    if (!load_offsets(p, offsets)) return 0;
    if (tid < 32) {
        int base = 0;
        for (int e0 = 0; e0 < p.experts; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < p.experts ? offsets[e + 1] - offsets[e] : 0;
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

// a / b for 0 <= a; in 32 bits where they hold it (64 take some 400 cycles).
__device__ __forceinline__ int64_t quotient(int64_t a, unsigned b) {
    return a <= 0xffffffffll ? static_cast<int64_t>(static_cast<uint32_t>(a) / b) : a / b;
}

// This CTA's share of `all` items: first .. end - 1.
__device__ __forceinline__ void share(int64_t all, int64_t &first, int64_t &end) {
    const int64_t each = quotient(all, gridDim.x), more = all - each * gridDim.x;
    first = each * blockIdx.x + min(static_cast<int64_t>(blockIdx.x), more);
    end = first + each + (blockIdx.x < more ? 1 : 0);
}

// The expert of a chunk: chunks[expert] <= chunk < chunks[expert + 1] (a whole warp, every
// lane with the same chunk): its 32 lanes look at every 32nd entry, then at the 32 behind it.
__device__ __forceinline__ int find_expert(const int *chunks, int experts, int chunk) {
    const int lane = threadIdx.x & 31;
    int lo = 0;
    if (experts > 32) lo = 32 * (__popc(__ballot_sync(kFull, 32 * lane < experts && chunks[min(32 * lane, experts)] <= chunk)) - 1);
    return lo + __popc(__ballot_sync(kFull, lo + lane < experts && chunks[min(lo + lane, experts)] <= chunk)) - 1;
}

// A column's scale in its block's row of `meta`; the start value is two further.
__device__ __forceinline__ int meta_column(int c) { return 4 * (c >> 1) + (c & 1); }

// 32 codes of activation row `a`, its c-th group; a block's first has its scale, too.
struct RowPart { uint4 q0, q1; float s; };

__device__ __forceinline__ int activation_row(const MoeProduct &p, int slot) {
    return min(max(p.rows != nullptr ? p.rows[slot] : slot, 0), p.m - 1);
}
__device__ __forceinline__ RowPart load_part(const MoeProduct &p, int a, int c) {
    RowPart v;
    const uint4 *qp = reinterpret_cast<const uint4 *>(p.q + static_cast<int64_t>(a) * p.k + c * 32);
    v.q0 = qp[0];
    v.q1 = qp[1];
    v.s = (c & 3) == 0 ? p.s[static_cast<int64_t>(a) * (p.k / kBlock) + (c >> 2)] : 0.0f;
    return v;
}

// Lay the codes of `rows` activation rows out in shared memory (all threads).  part: what
// thread tid < 4 rows nb loads first, group tid % (4 nb) of row tid / (4 nb).
template <int FMT>
__device__ __forceinline__ void stage_rows(const MoeProduct &p, int row0, int rows, RowPart part, uint8_t *act, float *meta) {
    const int tid = threadIdx.x, nb = p.k / kBlock, pitch = row_pitch(nb), per = nb * 4;
#pragma unroll 2
    for (int i = tid; i < rows * per; i += blockDim.x) {
        const int r = i / per, c = i - r * per;                      // c: group of 32 codes
        if (i != tid) part = load_part(p, activation_row(p, row0 + r), c);
        const uint4 q0 = part.q0, q1 = part.q1;
        const float sa = part.s;
        // minus the sums over q * s and over the offset of v
        const uint32_t raw[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
        int sum = 0, scaled = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sum = __dp4a(static_cast<int>(raw[j]), 0x01010101, sum);
            scaled = __dp4a(static_cast<int>(raw[j]), static_cast<int>(scale_bytes<FMT>(4 * j)), scaled);
        }
        int start = -(4 * scaled + (FMT == 0 ? 2 : 1) * sum);
        const unsigned quad = 0xfu << (tid & 28);                    // a block's four lanes take this turn together
        start += __shfl_xor_sync(quad, start, 1);
        start += __shfl_xor_sync(quad, start, 2);
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
                const int e0 = pair_weight<FMT>(i), e1 = e0 + (FMT == 0 ? 8 : 16);
                o[y] = act_pair(w[e0 >> 2], w[e1 >> 2], (e0 & 3) | ((4 + (e1 & 3)) << 4), pair_scale<FMT>(i));
            }
            *reinterpret_cast<uint4 *>(dst + 64 * x) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        if ((c & 3) == 0) {
            float *m = meta + (c >> 2) * 2 * kCols + meta_column(r);
            m[0] = sa;
            m[2] = static_cast<float>(start);
        }
    }
    const int none = kCols - rows;
    for (int i = tid; i < none * nb; i += blockDim.x) {
        float *m = meta + (i / none) * 2 * kCols + meta_column(rows + i % none);
        m[0] = m[2] = 0.0f;
    }
}

// The blocks whose codes are on their way while one is computed.
template <int FMT> constexpr int kAhead = FMT == 0 ? 4 : 8;

// This lane's four weight rows of the unit from output n0 on: rows g and g + 8 of the
// row tiles mt = 0, 1 (gate and up, or two of one matrix).
template <int FMT, bool GATEUP>
__device__ __forceinline__ void unit_rows(const MoeProduct &p, int expert, int n0, const uint8_t *(&src)[2][2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    constexpr int kBlockBytes = FMT == 0 ? 32 : 16;
    const int64_t row_bytes = static_cast<int64_t>(p.k / kBlock) * kBlockBytes;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = min(n0 + (GATEUP ? 0 : 16 * mt) + g + 8 * h, p.n - 1);
            src[mt][h] = p.codes[GATEUP ? mt : 0] + (static_cast<int64_t>(expert) * p.n + r) * row_bytes + t * (kBlockBytes / 4);
        }
}

template <int FMT>
__device__ __forceinline__ void load_block(const uint8_t *const (&src)[2][2], int b, Codes<FMT> (&c)[2][2]) {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) c[mt][h] = load_codes<FMT>(src[mt][h] + b * (FMT == 0 ? 32 : 16));
}

// c[mt][2 h + j]: the block's products of weight row 16 mt + 8 h + g and column 2 t + j.
// ap: this lane's column and t; start: the start values of columns 2 t, 2 t + 1.
template <int FMT>
__device__ __forceinline__ void block_products(const Codes<FMT> (&codes)[2][2], const uint8_t *ap, float2 start,
                                               const Joins<FMT> &join, float (&c)[2][4]) {
    uint4 bq[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) bq[i] = *reinterpret_cast<const uint4 *>(ap + 64 * i);
    Fields<FMT> f[2][2];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) f[mt][h] = fields<FMT>(codes[mt][h]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint4 &v = bq[i >> 1];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {                             // two sums in turn: neither waits for itself
            const Fields<FMT> &f0 = f[mt][0], &f1 = f[mt][1];
            const uint32_t a0 = weight_pair<FMT>(f0, join, 2 * i), a1 = weight_pair<FMT>(f1, join, 2 * i),
                           a2 = weight_pair<FMT>(f0, join, 2 * i + 1), a3 = weight_pair<FMT>(f1, join, 2 * i + 1);
            if (i == 0) mma_f16_first(c[mt], a0, a1, a2, a3, v.x, v.y, start);
            else mma_f16(c[mt], a0, a1, a2, a3, (i & 1) ? v.z : v.x, (i & 1) ? v.w : v.y);
        }
    }
}

__device__ __forceinline__ void cp_async8(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// A unit is 32 weight rows (16 of gate and of up, or 32 of one matrix) against one chunk
// of activation rows.  A CTA takes a contiguous share of all units, chunk by chunk, so
// that it stages a chunk's activations once for many units; its warps take them in
// turn.  Each warp brings its own units' codes through a ring in shared memory, four
// blocks at a time and across the ends of units.  (Copies by TMA: with a cp.async per
// lane every row costs the load pipe a turn of its own, which then bounds the kernel.)
template <int FMT, bool GATEUP>
__global__ void __launch_bounds__(32 * kMaxWarps, 1) stream_kernel(const __grid_constant__ StreamArgs args) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const MoeProduct &p = args.p;
    constexpr int kD = kDepth<FMT>, kBlockBytes = FMT == 0 ? 32 : 16, kUnitRows = GATEUP ? 16 : 32;
    const int nb = p.k / kBlock, warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    uint8_t *ring = smem + warp * kD * kStageBytes<FMT>;
    uint8_t *side = smem + warps * kD * kStageBytes<FMT> + warp * kD * kSideBytes<FMT>;
    const auto bar = [&](int slot) { return smem_u32(side + slot * kSideBytes<FMT> + 256); };
    int *offsets = reinterpret_cast<int *>(smem + warps * kD * (kStageBytes<FMT> + kSideBytes<FMT>));
    int *chunks = offsets + p.experts + 1;
    uint8_t *act = reinterpret_cast<uint8_t *>(offsets) + list_bytes(p.experts);
    float *meta = reinterpret_cast<float *>(act + args.chunk * row_pitch(nb));
    if (lane == 0) {
        for (int i = 0; i < kD; ++i) mbar_init(bar(i), 1);
        mbar_init_fence();
    }
    pdl_launch_dependents();
    pdl_wait();
    const int units = (p.n + kUnitRows - 1) / kUnitRows;
    const int64_t all = static_cast<int64_t>(list_chunks(p, args.chunk, args.limit, offsets, chunks)) * units;
    int64_t first, end;
    share(all, first, end);
    if (first >= end) return;
    const bool wide = nb % 4 == 0 && (reinterpret_cast<uintptr_t>(p.scales[0]) & 7) == 0 &&
                      (!GATEUP || (reinterpret_cast<uintptr_t>(p.scales[1]) & 7) == 0);
    // this warp's units: warp, warp + warps, .. of the `mine` in the CTA's share
    const int mine = static_cast<int>(end - first);
    const int first_chunk = static_cast<int>(quotient(first, units));
    const int first_u = static_cast<int>(first - static_cast<int64_t>(first_chunk) * units);
    int expert = find_expert(chunks, p.experts, first_chunk);
    int row0 = offsets[expert] + (first_chunk - chunks[expert]) * args.chunk;
    int rows = min(args.chunk, offsets[expert + 1] - row0);
    // what is staged first is on its way while the first weights are asked for
    const int part_r = threadIdx.x / (4 * nb), part_c = threadIdx.x - part_r * 4 * nb;
    const bool has_part = part_r < rows;
    const int part_a = has_part ? activation_row(p, row0 + part_r) : 0;

    // the issuing side; lane l brings the scales of row l of the unit (gate 0-15, up 16-31)
    int in_unit = warp, in_u = first_u + warp, in_chunk = first_chunk, in_block = 0, in_slot = 0, in_expert = expert, in_y = 0;
    const uint16_t *scale_src = nullptr;
    bool ok = true;                                                  // false: a wait ran out, nothing is copied or written any more
    const auto issue = [&]() {
        if (in_unit < mine) {
            if (in_block == 0) {                                     // a new unit
                while (in_u >= units) {
                    in_u -= units;
                    ++in_chunk;
                    in_expert = -1;
                }
                if (in_expert < 0) in_expert = find_expert(chunks, p.experts, in_chunk);
                in_y = in_expert * p.n + in_u * kUnitRows;
                const int n = min(in_u * kUnitRows + (GATEUP ? lane & 15 : lane), p.n - 1);
                scale_src = p.scales[GATEUP ? lane >> 4 : 0] + (static_cast<int64_t>(in_expert) * p.n + n) * nb;
            }
            if (lane == 0 && ok) {
                const uint32_t dst = smem_u32(ring + in_slot * kStageBytes<FMT>);
                mbar_arrive_expect_tx(bar(in_slot), kStageBytes<FMT>);
                load_box(dst, &args.codes[0], in_block * kBlockBytes, in_y, bar(in_slot));
                load_box(dst + kStageBytes<FMT> / 2, &args.codes[1], in_block * kBlockBytes, GATEUP ? in_y : in_y + 16, bar(in_slot));
            }
            uint16_t *sd = reinterpret_cast<uint16_t *>(side + in_slot * kSideBytes<FMT>) + lane * 4;
            if (wide) {
                cp_async8(sd, scale_src + in_block);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) sd[i] = ldg_u16(scale_src + min(in_block + i, nb - 1));
            }
            in_block += kStageBlocks;
            if (in_block >= nb) {
                in_block = 0;
                in_unit += warps;
                in_u += warps;
            }
            in_slot = in_slot == kD - 1 ? 0 : in_slot + 1;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    __syncwarp();
    issue();
    RowPart part{};
    if (has_part) part = load_part(p, part_a, part_c);
#pragma unroll 1
    for (int i = 1; i < kD; ++i) issue();

    const Joins<FMT> join = joins<FMT>();
    int slot = 0, unit = warp, u = first_u + warp;
    uint32_t phase = 0;
    for (int chunk = first_chunk, chunk_end = units - first_u;; ++chunk, u -= units, chunk_end += units) {
        if (chunk > first_chunk) {
            expert = find_expert(chunks, p.experts, chunk);
            row0 = offsets[expert] + (chunk - chunks[expert]) * args.chunk;
            rows = min(args.chunk, offsets[expert + 1] - row0);
            if (part_r < rows) part = load_part(p, activation_row(p, row0 + part_r), part_c);
            __syncthreads();                                         // every warp is done with the chunk before
        }
        stage_rows<FMT>(p, row0, rows, part, act, meta);
        __syncthreads();
        // a column without a row computes the last row's products again; they go nowhere
        const uint32_t piece = g * kStageBlocks * kBlockBytes +
                               (FMT == 0 ? (((t >> 1) ^ g) << 4) + 8 * (t & 1) : ((g >> 1) << 4) + 4 * t);
        const uint8_t *act_lane = act + min(g, rows - 1) * row_pitch(nb) + t * 16;
        for (; unit < min(mine, chunk_end); unit += warps, u += warps) {
            const uint8_t *ap = act_lane;
            const float *mp = meta + 4 * t;
            uint64_t acc[2][2] = {};                                 // [mt][h]: columns 2 t, 2 t + 1
#pragma unroll 1
            for (int b0 = 0; b0 < nb; b0 += kStageBlocks) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kD - 1) : "memory");
                if (ok && !mbar_wait(bar(slot), phase)) {
                    record_wait(args.err, &lost_waits, 1u << 12);
                    ok = false;
                    // the stages behind it are on their way, too: they land before the warp goes on, and out
                    uint32_t turn = phase;
#pragma unroll 1
                    for (int i = slot + 1; i < slot + kD; ++i) {
                        if (i == kD) turn ^= 1;
                        mbar_wait(bar(i % kD), turn);
                    }
                }
                __syncwarp();
                const uint8_t *stage = ring + slot * kStageBytes<FMT>;
                const uint16_t *ws = reinterpret_cast<const uint16_t *>(side + slot * kSideBytes<FMT>) + 4 * g;
                const int end_b = nb - b0;
#pragma unroll
                for (int b = 0; b < kStageBlocks; ++b, ap += 256, mp += 2 * kCols, ++ws) {
                    if (b >= end_b) break;
                    Codes<FMT> c[2][2];
                    // rows g + 8 x: 16-byte pieces of a row change places by the row's number
                    const uint8_t *cp = stage + (piece ^ (b * (FMT == 0 ? 32 : 16)));
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint8_t *cx = cp + x * 8 * kStageBlocks * kBlockBytes;
                        if (FMT == 0) {
                            const uint2 v = *reinterpret_cast<const uint2 *>(cx);
                            c[x >> 1][x & 1].w[0] = v.x;
                            c[x >> 1][x & 1].w[FMT == 0 ? 1 : 0] = v.y;
                        } else {
                            c[x >> 1][x & 1].w[0] = *reinterpret_cast<const uint32_t *>(cx);
                        }
                    }
                    // scales and start values of columns 2 t, 2 t + 1
                    const float4 sa = *reinterpret_cast<const float4 *>(mp);
                    float d[2][4];
                    block_products<FMT>(c, ap, make_float2(sa.z, sa.w), join, d);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float sw = f16_bits_to_f32(ws[32 * x]);
                        uint64_t &a = acc[x >> 1][x & 1];
                        a = fma2(pack2(d[x >> 1][2 * (x & 1)], d[x >> 1][2 * (x & 1) + 1]),
                                 mul2(pack2(sw, sw), pack2(sa.x, sa.y)), a);
                    }
                }
                __syncwarp();                                        // the stage is read
                issue();
                if (slot == kD - 1) {
                    slot = 0;
                    phase ^= 1;
                } else {
                    ++slot;
                }
            }
            const int n0 = u * kUnitRows;
            float y[2][4];
#pragma unroll
            for (int x = 0; x < 4; ++x) unpack2(acc[x >> 1][x & 1], y[x >> 1][2 * (x & 1)], y[x >> 1][2 * (x & 1) + 1]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = 2 * t + j;
                if (col >= rows || !ok) continue;
                const int64_t out = static_cast<int64_t>(row0 + col) * p.n;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (GATEUP) {
                        const int n = n0 + g + 8 * h;
                        if (n < p.n) p.h[out + n] = f32_to_bf16_bits(__fmul_rn(tq_silu(y[0][2 * h + j]), y[1][2 * h + j]));
                    } else {
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt) {
                            const int n = n0 + 16 * mt + g + 8 * h;
                            if (n < p.n) p.y[out + n] = y[mt][2 * h + j];
                        }
                    }
                }
            }
        }
        if (chunk_end >= mine) break;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---------------------------------------------------------------------------
// The same for few units in all (one or a few tokens): the four warps of a unit
// take a quarter of the blocks each, so that a warp's chain of loads and matrix
// instructions is a quarter as long; the exact block products meet in shared
// memory, where one thread per output folds them in order.  The codes of the
// next round are on their way while a round is folded.
// ---------------------------------------------------------------------------
// Up to this many units per SM: 3.4 (one token, top 8 of 64 experts, 2 x 1024 x 2048) take 7.6 us split and
// 12.7 whole; 27 (33 tokens, 1-bit) 44 and 29; 34 (8 tokens, 5120 x 1536) 31 and 23.
constexpr int kSplitMost = 8;
constexpr int kSplit = 4, kSplitUnits = kSplitWarps / kSplit;
constexpr int kDotPitch = 36;                       // 32 rows; columns 2t two apart fall on other banks
constexpr int kSplitScalePitch = 32 * kSplitUnits + 2;

// Behind the activations and their scales: [2] weight scales fp16 [block][row],
// [2][unit] products [block][column][row]
size_t split_smem(int experts, int chunk, int nb) {
    return static_cast<size_t>(list_bytes(experts)) + static_cast<size_t>(chunk) * row_pitch(nb) +
           static_cast<size_t>(nb) * kCols * 8 + 2 * static_cast<size_t>(nb) * kSplitScalePitch * 2 +
           2 * static_cast<size_t>(kSplitUnits) * nb * chunk * kDotPitch * 4;
}

template <int FMT, bool GATEUP>
__global__ void __launch_bounds__(32 * kSplitWarps, 2) split_kernel(const __grid_constant__ StreamArgs args) {
    extern __shared__ __align__(16) uint8_t smem[];
    const MoeProduct &p = args.p;
    constexpr int kA = kAhead<FMT>, kUnitRows = GATEUP ? 16 : 32;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int nb = p.k / kBlock, slot = warp / kSplit;
    const int per = (nb + kSplit - 1) / kSplit, lo = min((warp % kSplit) * per, nb), hi = min(lo + per, nb);
    int *offsets = reinterpret_cast<int *>(smem), *chunks = offsets + p.experts + 1;
    uint8_t *act = smem + list_bytes(p.experts);
    float *meta = reinterpret_cast<float *>(act + args.chunk * row_pitch(nb));
    float *dots = meta + nb * 2 * kCols;
    const int unit_dots = nb * args.chunk * kDotPitch;
    uint16_t *wsc = reinterpret_cast<uint16_t *>(dots + 2 * kSplitUnits * unit_dots);
    const int units = (p.n + kUnitRows - 1) / kUnitRows, per_chunk = (units + kSplitUnits - 1) / kSplitUnits;
    const int64_t rounds = static_cast<int64_t>(list_chunks(p, args.chunk, args.limit, offsets, chunks)) * per_chunk;
    int64_t first, end;
    share(rounds, first, end);
    const Joins<FMT> join = joins<FMT>();

    struct Place { int chunk, expert, row0, rows, n0; };            // n0: first output of the round
    const auto locate = [&](int64_t r) {
        Place q;
        q.chunk = static_cast<int>(quotient(r, per_chunk));
        q.n0 = static_cast<int>(r - static_cast<int64_t>(q.chunk) * per_chunk) * kSplitUnits * kUnitRows;
        q.expert = find_expert(chunks, p.experts, q.chunk);
        q.row0 = offsets[q.expert] + (q.chunk - chunks[q.expert]) * args.chunk;
        q.rows = min(args.chunk, offsets[q.expert + 1] - q.row0);
        return q;
    };
    const uint8_t *src[2][2];
    Codes<FMT> ring[kA][2][2];
    const auto fetch = [&](const Place &q) {
        unit_rows<FMT, GATEUP>(p, q.expert, q.n0 + slot * kUnitRows, src);
#pragma unroll
        for (int a = 0; a < kA; ++a)
            if (lo + a < hi) load_block<FMT>(src, lo + a, ring[a]);
    };

    if (first >= end) return;
    int staged = -1;
    Place at = locate(first);
    fetch(at);
    for (int64_t r = first; r < end; ++r) {
        const int buf = static_cast<int>(r - first) & 1;
        for (int i = tid; i < 32 * kSplitUnits * nb; i += blockDim.x) {
            const int lr = i / nb, b = i - lr * nb;
            const int n = at.n0 + (lr >> 5) * kUnitRows + (GATEUP ? lr & 15 : lr & 31);
            wsc[(buf * nb + b) * kSplitScalePitch + lr] =
                ldg_u16(p.scales[GATEUP ? (lr >> 4) & 1 : 0] + (static_cast<int64_t>(at.expert) * p.n + min(n, p.n - 1)) * nb + b);
        }
        if (at.chunk != staged) {
            if (staged >= 0) __syncthreads();                       // the fold before reads what is staged now
            const int part_r = tid / (4 * nb);
            RowPart part{};
            if (part_r < at.rows) part = load_part(p, activation_row(p, at.row0 + part_r), tid - part_r * 4 * nb);
            stage_rows<FMT>(p, at.row0, at.rows, part, act, meta);
            __syncthreads();
            staged = at.chunk;
        }
        float *mine = dots + (buf * kSplitUnits + slot) * unit_dots;
        const uint8_t *ap = act + min(g, at.rows - 1) * row_pitch(nb) + t * 16 + lo * 256;
#pragma unroll 1
        for (int b0 = lo; b0 < hi; b0 += kA, ap += kA * 256)
#pragma unroll
            for (int a = 0; a < kA; ++a) {
                const int b = b0 + a;
                if (b >= hi) break;
                float c[2][4];
                block_products<FMT>(ring[a], ap + a * 256,
                                    *reinterpret_cast<const float2 *>(meta + b * 2 * kCols + 4 * t + 2), join, c);
                if (b + kA < hi) load_block<FMT>(src, b + kA, ring[a]);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (2 * t + j < at.rows) {
                        float *d = mine + (b * at.rows + 2 * t + j) * kDotPitch + g;
#pragma unroll
                        for (int x = 0; x < 4; ++x) d[8 * x] = c[x >> 1][2 * (x & 1) + j];
                    }
            }
        const Place done = at;
        if (r + 1 < end) {
            at = locate(r + 1);
            fetch(at);
        }
        __syncthreads();
        for (int i = tid; i < kSplitUnits * kUnitRows * done.rows; i += blockDim.x) {
            const int o = i % kUnitRows, rest = i / kUnitRows, col = rest % done.rows, s = rest / done.rows;
            const int n = done.n0 + s * kUnitRows + o;
            if (n >= p.n) continue;
            const float *d = dots + (buf * kSplitUnits + s) * unit_dots + col * kDotPitch + o;
            const uint16_t *w = wsc + buf * nb * kSplitScalePitch + 32 * s + o;
            float acc[2] = {0.0f, 0.0f};
#pragma unroll 4
            for (int b = 0; b < nb; ++b) {
                const float sa = meta[b * 2 * kCols + meta_column(col)];
#pragma unroll
                for (int x = 0; x < (GATEUP ? 2 : 1); ++x)
                    acc[x] = __fmaf_rn(d[b * done.rows * kDotPitch + 16 * x],
                                       __fmul_rn(f16_bits_to_f32(w[b * kSplitScalePitch + 16 * x]), sa), acc[x]);
            }
            const int64_t out = static_cast<int64_t>(done.row0 + col) * p.n + n;
            if (GATEUP) p.h[out] = f32_to_bf16_bits(__fmul_rn(tq_silu(acc[0]), acc[1]));
            else p.y[out] = acc[0];
        }
    }
}

template <int FMT, bool GATEUP>
cudaError_t launch(const MoeProduct &p, int limit, unsigned *err, cudaStream_t stream) {
    StreamArgs a{};
    a.p = p;
    a.limit = limit;
    a.err = err;
    const int nb = p.k / kBlock;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    constexpr int64_t kUnitRows = GATEUP ? 16 : 32;
    const int64_t units = ws_cdiv(p.n, kUnitRows);
    constexpr size_t kSmem = 227 * 1024, kSplitSmem = kSmem / 2 - 1024;
    static SmemLimit limits[2];
    // the chunks that an even routing of few slots gives, and with them the units
    const int64_t active = p.experts < p.slots ? p.experts : p.slots;
    int chunk = p.max_rows < kCols ? p.max_rows : kCols;
    // an upper bound of the chunks: one per expert and one more for every full one
    const auto most_chunks = [&](int c) {
        int64_t most = static_cast<int64_t>(p.experts) + p.slots / c;
        if (most > p.slots) most = p.slots;
        const int64_t cap = static_cast<int64_t>(p.experts) * ws_cdiv(limit, c);
        return most > cap ? cap : most;
    };
    if (active * units <= kSplitMost * sms && split_smem(p.experts, chunk, nb) <= kSplitSmem) {
        const size_t smem = split_smem(p.experts, chunk, nb);
        a.chunk = chunk;
        e = limits[0].raise(split_kernel<FMT, GATEUP>, kSplitSmem);
        if (e != cudaSuccess) return e;
        int64_t grid = most_chunks(chunk) * ws_cdiv(units, kSplitUnits);
        if (grid > 2 * sms) grid = 2 * sms;
        return launch_pdl(split_kernel<FMT, GATEUP>, dim3(static_cast<unsigned>(grid)), dim3(32 * kSplitWarps), smem, stream, a);
    }
    // fewer warps to a CTA where one chunk for each expert would not give every SM a CTA
    int warps = kMaxWarps;
    while (warps > 4 && active * ws_cdiv(units, warps) < sms) warps /= 2;
    // as many rows at once as fit in shared memory, at most 8 and no more than an expert has
    while (warps > 4 && stream_smem<FMT>(p.experts, chunk, nb, warps) > kSmem) warps /= 2;
    while (chunk > 1 && stream_smem<FMT>(p.experts, chunk, nb, warps) > kSmem) --chunk;
    const size_t smem = stream_smem<FMT>(p.experts, chunk, nb, warps);
    if (smem > kSmem) return cudaErrorInvalidValue;
    a.chunk = chunk;
    constexpr int kBlockBytes = FMT == 0 ? 32 : 16;
    const uint64_t row_bytes = static_cast<uint64_t>(nb) * kBlockBytes;
    for (int i = 0; i < 2; ++i) {
        e = make_tmap_2d(&a.codes[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, p.codes[GATEUP ? i : 0], row_bytes,
                         static_cast<uint64_t>(p.experts) * p.n, row_bytes, kStageBlocks * kBlockBytes, 16,
                         FMT == 0 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
        if (e != cudaSuccess) return e;
    }
    e = limits[1].raise(stream_kernel<FMT, GATEUP>, kSmem);
    if (e != cudaSuccess) return e;
    int per_sm = static_cast<int>((kSmem + 1024) / (smem + 1024));
    if (per_sm > kMaxWarps / warps) per_sm = kMaxWarps / warps;
    if (per_sm < 1) per_sm = 1;
    int64_t grid = most_chunks(chunk) * ws_cdiv(units, warps);
    if (grid > static_cast<int64_t>(sms) * per_sm) grid = static_cast<int64_t>(sms) * per_sm;
    return launch_pdl(stream_kernel<FMT, GATEUP>, dim3(static_cast<unsigned>(grid)), dim3(32 * warps), smem, stream, a);
}

}  // namespace

cudaError_t moe_stream_waits(unsigned *bits, cudaStream_t stream) {
    return cudaMemcpyFromSymbolAsync(bits, lost_waits, sizeof(*bits), 0, cudaMemcpyDeviceToHost, stream);
}

cudaError_t moe_stream_launch(const MoeProduct &p, int limit, unsigned *err, cudaStream_t stream) {
    if (p.h != nullptr) return p.fmt == TQ_FMT_TERNARY2 ? launch<0, true>(p, limit, err, stream) : launch<1, true>(p, limit, err, stream);
    return p.fmt == TQ_FMT_TERNARY2 ? launch<0, false>(p, limit, err, stream) : launch<1, false>(p, limit, err, stream);
}

}  // namespace tq
