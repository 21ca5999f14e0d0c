// kvq_paged_chunk.cuh -- attention of many queries per sequence over the paged cache, on the
// fifth-generation tensor cores (tcgen05, accumulators in tensor memory).
//
// Mathematics: as kvq_paged_split.cuh; token i of a sequence sees positions 0 .. len - n + i.
//
// Work.  The n G query rows of a (sequence, KV head) form units of 256 rows (two tiles of 128; one
// tile for 256-wide heads, whose O fills half of tensor memory).  A unit times a block of 64 keys is
// a step; all steps of the batch are laid end to end and cut into equal spans, one per CTA (one CTA
// per SM), so ragged and causal work is even whatever the lengths.  A unit cut by a span boundary
// leaves pieces (m, l, o) in the workspace, which a second kernel merges.
//
// A step, by warps: warp 0 streams the block's f16 operands K^ (keys x D) and V^ (D x keys) into a ring;
// S = Q K^T of each tile is issued by a warp of its own (1, and 2 for the second tile), O += P V^ by one
// more; four warps per tile hold one row per thread: running maximum, weights, P into tensor memory, and
// the rescale of O when the maximum moves by more than kChunkDrift.  S of the next block is computed
// while the softmax of this one runs (S and P have their own columns).
//
// Lifted.  Converting codes costs about as many instructions as the softmax of 256 rows, once per unit; so a
// kernel before this one makes the operands of every block once, in the order the MMA reads them, and the
// chunk kernel streams them from the workspace (LIFT): 32 KB per step and head of 128 instead of 9 to 32 KB of
// codes.  Where that workspace would be too large (kLiftBytes) warp 0 streams tile records and eight converter
// warps make the operands in shared memory.
//
// Measured (4096 bf16 queries, 40 heads over 8, the end of 16384 positions, q4_0): 840 us, 1430 TFLOP/s, of it
// lift 15 and merge 22 us; a step of 256 rows takes 1710 cycles, its products 1160 (N = 64: 32 cycles with
// Q in tensor memory, 48 from shared memory; N = 128: 64), and waits for the softmax of its rows (700 cycles of
// arithmetic, 300 of tensor-memory loads and stores, the rest barriers).  256-wide, 128 rows: 1500 cycles, products
// 1024 (f16 over quantised pages, as pairs: about 2300 and 2048).  Tried and dropped: two buffers of P (256-wide the same, 128-wide 898 us, for Q then leaves tensor
// memory), a warp per tile for O, test_wait before try_wait, spinning waits (worse).
//
// Orders.  The values of K^ and Q sit in the order 0, 2, 1, 3 within each four (as the bytes of a code
// word come out), and the rows of V^ (columns of O) in the order 0, 2, .., 14, 1, 3, .., 15 within each
// sixteen, so that a warp's stores of V^ fill whole core matrices; the epilogue puts them back.
//
// Rounding.  Q is f16; a bf16 row outside f16's range is moved by a power of two.
// K^ and V^ are scale x code rounded once to f16 (2^-11), P is f16 (2^-11); with f16 activations over
// quantised pages K^ and P are pairs hi + lo (chunk_fine).  S, O, the maxima and sums are
// fp32.  The output has 16 bits (2^-11 or 2^-8).  A block with scales that would leave f16
// is stored times 2^-e, and S or P is multiplied by 2^e, both exact.
#pragma once
#include <math_constants.h>

#include "kvq_paged.cuh"

namespace kvq {
namespace {

constexpr float kChunkLn2 = 0.69314718055994530942f, kChunkLog2e = 1.44269504088896340736f;
// weights are 2^(s - m) <= 2^kChunkDrift, times 2^e <= 2^11 in f16
constexpr float kChunkDrift = 4.0f;

// ---- tcgen05 and tensor memory (inline PTX) ----
__device__ __forceinline__ void t5_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void t5_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
// One lane of a converged warp, always the same.  MMAs are issued under this predicate in code that the
// whole warp runs: issued from a branch on the thread index, whose operands the compiler cannot keep in
// uniform registers, every tcgen05.mma took 97 cycles whatever its N (measured; 32 for N = 64 this way).
// Operands that depend on values loaded from memory go through t5_uniform for the same reason.
__device__ __forceinline__ bool t5_elect() {
    uint32_t r;
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ uint32_t t5_uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ uint64_t t5_plus(uint64_t desc, uint32_t bytes) {  // a descriptor `bytes` further on
    return (desc & 0xffffffff00000000ull) | t5_uniform(static_cast<uint32_t>(desc) + (bytes >> 4));
}
// shared-memory operand without swizzle: 8-row x 16-byte core matrices, `lbo` bytes apart along K
// and `sbo` along M or N
__device__ __forceinline__ uint64_t t5_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return static_cast<uint64_t>((addr >> 4) & 0x3fffu) | (static_cast<uint64_t>((lbo >> 4) & 0x3fffu) << 16) |
           (static_cast<uint64_t>((sbo >> 4) & 0x3fffu) << 32) | (static_cast<uint64_t>(1) << 46);
}
// kind::f16, fp32 accumulator, f16 A and B, both K-major
__host__ __device__ constexpr uint32_t t5_idesc(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void t5_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void t5_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void t5_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void t5_ld32(uint32_t t, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(t));
}
__device__ __forceinline__ void t5_st32(uint32_t t, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
        "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n" ::"r"(t),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
        "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
        "r"(r[31]));
}
__device__ __forceinline__ void t5_st16(uint32_t t, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};\n" ::"r"(t),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}
__device__ __forceinline__ void t5_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void t5_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void smem_to_async() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }
__device__ __forceinline__ float chunk_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// fp32 pairs, one instruction each
__device__ __forceinline__ float2 pair_fma(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n .reg .b64 ra, rb, rc, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n mov.b64 rc, {%6, %7};\n"
        " fma.rn.f32x2 rd, ra, rb, rc;\n mov.b64 {%0, %1}, rd;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 pair_add(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n add.rn.f32x2 rd, ra, rb;\n"
        " mov.b64 {%0, %1}, rd;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 pair_mul(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n mul.rn.f32x2 rd, ra, rb;\n"
        " mov.b64 {%0, %1}, rd;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ uint32_t perm(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;\n" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}
// byte offset of (row, k) in an operand of `kext` elements per row: core matrices of 8 rows x 8 elements
__device__ __forceinline__ int core_at(int row, int k, int kext) {
    return (row >> 3) * (kext * 16) + (k >> 3) * 128 + (row & 7) * 16 + (k & 7) * 2;
}

// ---- codes to operands ----
constexpr int kChunkKeys = 64, kChunkTiles = kChunkKeys / kTileRows;

// Rows of a block's tiles in use: bit i of `got` set if tile i has a page; the sequence ends `left` rows
// after the block's first.
struct BlockRows {
    int got, left;
    __device__ __forceinline__ int of(int i) const {
        return ((got >> i) & 1) ? max(0, min(kTileRows, left - i * kTileRows)) : 0;
    }
};
// a pair of halves of rows r, r + 1, those from `use` on replaced by 0
__device__ __forceinline__ uint32_t cut_pair(uint32_t x, int r, int use) {
    return r >= use ? 0u : (r + 1 >= use ? (x & 0xffffu) : x);
}
__device__ __forceinline__ float pow2i_f(int e) { return __int_as_float((127 + e) << 23); }
__device__ __forceinline__ __half2 half_twice(uint32_t pair, int upper) {  // one half of a pair, twice
    return u32_as_h2(perm(pair, 0u, upper ? 0x3232u : 0x1010u));
}
// q8_0 codes (sign in bit 15, magnitude in the low bits: a subnormal q 2^-24) times 2^14: q 2^-10, exactly
__device__ __forceinline__ __half2 q8_small(uint32_t x) { return __hmul2(u32_as_h2(x & 0x807f807fu), __float2half2_rn(16384.0f)); }
// q4_0 codes in the low or high nibble of each half's low byte: c - 8
__device__ __forceinline__ __half2 q4_low(uint32_t x) {
    return __hsub2(u32_as_h2((x & 0x000f000fu) | 0x64006400u), __float2half2_rn(1032.0f));
}
__device__ __forceinline__ __half2 q4_high(uint32_t x) {
    return __hfma2(u32_as_h2((x & 0x00f000f0u) | 0x64006400u), __float2half2_rn(0.0625f), __float2half2_rn(-72.0f));
}

// Exponent e >= 0 with |value| 2^-e below 2^14 (q4_0) or 2^12 (q8_0, whose scale meets codes times 2^-10) over
// the block's rows in use; at most 11.  OFF: the scales in a tile record.  By a whole warp.
template <int TYPE, int OFF, int NS, class TileAt>
__device__ __forceinline__ int block_exp(TileAt tile, const BlockRows &use) {
    if constexpr (TYPE == KVQ_F16) {
        return 0;
    } else {
        const float cmax = TYPE == KVQ_Q8_0 ? 127.f : 8.f;
        constexpr int most = TYPE == KVQ_Q8_0 ? 12 : 14;
        const int lane = threadIdx.x & 31;
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < NS; ++k) {
            const int gi = k * 32 + lane, i = gi / (8 * NS), in = gi % (8 * NS);  // tile, 16-byte group of its scales
            uint4 w = *reinterpret_cast<const uint4 *>(tile(i) + OFF + in * 16);
            const int n = use.of(i), ka = 2 * ((in & 7) >> 1);
            if (n < kTileRows) {
                keep_branch();
                w = make_uint4(cut_pair(w.x, ka, n), cut_pair(w.y, ka + 8, n), cut_pair(w.z, ka, n), cut_pair(w.w, ka + 8, n));
            }
            const __half2 a = __hmax2(__habs2(u32_as_h2(w.x)), __habs2(u32_as_h2(w.y)));
            const __half2 b = __hmax2(__habs2(u32_as_h2(w.z)), __habs2(u32_as_h2(w.w)));
            m = h2_as_u32(__hmax2(u32_as_h2(m), __hmax2(a, b)));
        }
        const float2 f = __half22float2(u32_as_h2(m));
        float top = fmaxf(f.x, f.y) * cmax;
        if (!__any_sync(0xffffffffu, top > static_cast<float>(1 << most))) return 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        return min(11, max(0, ilogbf(top) - (most - 1)));
    }
}

// K^ of a block times 2^-e, by warps cw, cw + nw, ..: rows past the sequence's end may become anything (their
// scores are masked).  tile(i): record of tile i; kh: the operand, shared or global memory.
// FINE: hi = f16(scale x code) and, an operand further on, lo = scale x code - hi.
template <int KT, int VT, int NS, bool FINE, class TileAt>
__device__ __forceinline__ void convert_keys(TileAt tile, uint8_t *kh, int e, int cw, const int nw) {
    using T = PagedTile<KT, VT, NS>;
    constexpr int D = T::D;
    const int lane = threadIdx.x & 31, n = lane >> 2, jd = lane & 3;  // key n (and n + 8) of the tile, 4-value group jd
    const __half2 fk = __float2half2_rn(pow2i_f(KT == KVQ_Q8_0 ? 10 - e : -e));
    uint8_t *lane_at = kh + (jd >> 1) * 128 + n * 16 + (jd & 1) * 8;  // core_at(n, 4 jd, D)
    auto put = [&](int at, __half2 c02, __half2 c13, __half2 d2) {
        const __half2 a = __hmul2(c02, d2), b = __hmul2(c13, d2);
        *reinterpret_cast<uint2 *>(lane_at + at) = make_uint2(h2_as_u32(a), h2_as_u32(b));
        if constexpr (FINE)
            *reinterpret_cast<uint2 *>(lane_at + at + kChunkKeys * D * 2) =
                make_uint2(h2_as_u32(__hfma2(c02, d2, __hneg2(a))), h2_as_u32(__hfma2(c13, d2, __hneg2(b))));
    };
    // core_at(16 i + n + 8 s8, dim + 4 jd, D) less lane_at, for dim a multiple of 16
    auto at = [](int i, int s8, int dim) { return (2 * i + s8) * (D * 16) + dim * 16; };
    if constexpr (KT == KVQ_Q8_0) {
#pragma unroll 4
        for (int wu = cw; wu < kChunkTiles * NS * 4; wu += nw) {
            const int ts = wu >> 2, b = wu & 3, i = ts / NS, sl = ts % NS, dim = sl * kSlice + 32 * b;
            const uint8_t *t = tile(i);
            const uint4 c = *reinterpret_cast<const uint4 *>(t + sl * 2048 + (b * 32 + lane) * 16);
            const uint2 sc = *reinterpret_cast<const uint2 *>(t + T::OFF_KS + sl * kScaleTile + (n >> 1) * 32 + b * 8);
            const __half2 da = __hmul2(half_twice(sc.x, n & 1), fk), db = __hmul2(half_twice(sc.y, n & 1), fk);
            auto lo = [](uint32_t w) { return q8_small(perm(w, 0u, 0xA280u)); };
            auto hi = [](uint32_t w) { return q8_small(perm(w, 0u, 0xB391u)); };
            put(at(i, 0, dim), lo(c.x), hi(c.x), da);
            put(at(i, 0, dim + 16), lo(c.y), hi(c.y), da);
            put(at(i, 1, dim), lo(c.z), hi(c.z), db);
            put(at(i, 1, dim + 16), lo(c.w), hi(c.w), db);
        }
    } else if constexpr (KT == KVQ_Q4_0) {
#pragma unroll 2
        for (int wu = cw; wu < kChunkTiles * NS * 2; wu += nw) {
            const int ts = wu >> 1, b2 = wu & 1, i = ts / NS, sl = ts % NS;
            const uint8_t *t = tile(i);
            const uint4 c = *reinterpret_cast<const uint4 *>(t + sl * 1024 + (b2 * 32 + lane) * 16);
            const uint4 sc = *reinterpret_cast<const uint4 *>(t + T::OFF_KS + sl * kScaleTile + (n >> 1) * 32 + b2 * 16);
            const uint32_t cs[4] = {c.x, c.y, c.z, c.w}, ss[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {  // block 2 b2 + q / 2, key n + 8 (q % 2)
                const int dim = sl * kSlice + 64 * b2 + 32 * (q >> 1);
                const __half2 d2 = __hmul2(half_twice(ss[q], n & 1), fk);
                const uint32_t odd = cs[q] >> 8;
                put(at(i, q & 1, dim), q4_low(cs[q]), q4_low(odd), d2);
                put(at(i, q & 1, dim + 16), q4_high(cs[q]), q4_high(odd), d2);
            }
        }
    } else {
#pragma unroll 4
        for (int wu = cw; wu < kChunkTiles * NS * 8; wu += nw) {
            const int ts = wu >> 3, ch = wu & 7, i = ts / NS, sl = ts % NS, dim = sl * kSlice + 32 * (ch >> 1);
            const uint4 c = *reinterpret_cast<const uint4 *>(tile(i) + sl * 4096 + (ch * 32 + lane) * 16);
            *reinterpret_cast<uint2 *>(lane_at + at(i, ch & 1, dim)) = make_uint2(c.x, c.y);
            *reinterpret_cast<uint2 *>(lane_at + at(i, ch & 1, dim + 16)) = make_uint2(c.z, c.w);
        }
    }
}

// V^ of a block times 2^-e: rows past the sequence's end may hold any bits and become 0.
template <int KT, int VT, int NS, class TileAt>
__device__ __forceinline__ void convert_values(TileAt tile, uint8_t *vh, int e, const BlockRows &use, int cw, const int nw) {
    using T = PagedTile<KT, VT, NS>;
    const int lane = threadIdx.x & 31, np = lane >> 2, j = lane & 3;
    const __half2 fv = __float2half2_rn(pow2i_f(VT == KVQ_Q8_0 ? 10 - e : -e));
    uint8_t *lane_at = vh + np * 16 + j * 4;  // row np of a core matrix, keys 2j, 2j + 1
    // value dim + 2 np + odd of keys 16 i + 2j, + 1 (and + 8, + 9): row (dim / 8 + odd) * 8 + np
    auto at = [](int i, int dim, int odd) { return ((dim >> 3) + odd) * (kChunkKeys * 16) + 2 * i * 128; };
    auto put = [&](int a, __half2 ca, __half2 cb, __half2 da, __half2 db) {
        *reinterpret_cast<uint32_t *>(lane_at + a) = h2_as_u32(__hmul2(ca, da));
        *reinterpret_cast<uint32_t *>(lane_at + a + 128) = h2_as_u32(__hmul2(cb, db));
    };
    if constexpr (VT == KVQ_Q8_0) {
#pragma unroll 4
        for (int wu = cw; wu < kChunkTiles * NS * 4; wu += nw) {
            const int ts = wu >> 2, b = wu & 3, i = ts / NS, sl = ts % NS, n = use.of(i);
            const uint8_t *t = tile(i);
            const uint4 c = *reinterpret_cast<const uint4 *>(t + T::OFF_V + sl * 2048 + (b * 32 + lane) * 16);
            const uint2 sc = *reinterpret_cast<const uint2 *>(t + T::OFF_VS + sl * kScaleTile + j * 32 + b * 8);
            const __half2 da = __hmul2(u32_as_h2(cut_pair(sc.x, 2 * j, n)), fv), db = __hmul2(u32_as_h2(cut_pair(sc.y, 2 * j + 8, n)), fv);
            const uint32_t cs[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int q = 0; q < 4; ++q)
                put(at(i, sl * kSlice + 32 * b + 16 * (q >> 1), q & 1), q8_small(perm(cs[q], 0u, 0xA280u)), q8_small(perm(cs[q], 0u, 0xB391u)), da, db);
        }
    } else if constexpr (VT == KVQ_Q4_0) {
#pragma unroll 2
        for (int wu = cw; wu < kChunkTiles * NS * 2; wu += nw) {
            const int ts = wu >> 1, b2 = wu & 1, i = ts / NS, sl = ts % NS, n = use.of(i);
            const uint8_t *t = tile(i);
            const uint4 c = *reinterpret_cast<const uint4 *>(t + T::OFF_V + sl * 1024 + (b2 * 32 + lane) * 16);
            const uint4 sc = *reinterpret_cast<const uint4 *>(t + T::OFF_VS + sl * kScaleTile + j * 32 + b2 * 16);
            const __half2 d[4] = {__hmul2(u32_as_h2(cut_pair(sc.x, 2 * j, n)), fv), __hmul2(u32_as_h2(cut_pair(sc.y, 2 * j + 8, n)), fv),
                                  __hmul2(u32_as_h2(cut_pair(sc.z, 2 * j, n)), fv), __hmul2(u32_as_h2(cut_pair(sc.w, 2 * j + 8, n)), fv)};
            const uint32_t cs[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {  // block 2 b2 + q / 2, value 2 np + q % 2 (and + 16)
                const int dim = sl * kSlice + 64 * b2 + 32 * (q >> 1);
                const uint32_t odd = cs[q] >> 8;
                put(at(i, dim, q & 1), q4_low(cs[q]), q4_low(odd), d[2 * (q >> 1)], d[2 * (q >> 1) + 1]);
                put(at(i, dim + 16, q & 1), q4_high(cs[q]), q4_high(odd), d[2 * (q >> 1)], d[2 * (q >> 1) + 1]);
            }
        }
    } else {
#pragma unroll 4
        for (int wu = cw; wu < kChunkTiles * NS * 8; wu += nw) {
            const int ts = wu >> 3, ch = wu & 7, i = ts / NS, sl = ts % NS, n = use.of(i);
            const uint4 c = *reinterpret_cast<const uint4 *>(tile(i) + T::OFF_V + sl * 4096 + (ch * 32 + lane) * 16);
            const int dim = sl * kSlice + 32 * (ch >> 1) + 16 * (ch & 1);
#pragma unroll
            for (int odd = 0; odd < 2; ++odd) {
                uint8_t *to = lane_at + at(i, dim, odd);
                *reinterpret_cast<uint32_t *>(to) = cut_pair(odd ? c.z : c.x, 2 * j, n);
                *reinterpret_cast<uint32_t *>(to + 128) = cut_pair(odd ? c.w : c.y, 2 * j + 8, n);
            }
        }
    }
}

// FINE (f16 activations over quantised pages): K^ is a pair hi + lo and so are the weights, twice the products.
// One f16 rounding each of K^, V^ and P adds 3.6e-4 to 8.4e-4 of the outputs' norm (the more the wider the scores) to
// the 2.1e-4 of an f16 output's own rounding (bf16: 1.7e-3); with the pairs V^'s alone is left, 2.1e-4.
template <int KT, int DT>
constexpr bool chunk_fine() { return KT != KVQ_F16 && DT == KVQ_DT_F16; }

template <int KT, int VT, int NS, bool LIFT, bool FINE>
struct ChunkCfg {
    using T = PagedTile<KT, VT, NS>;
    static constexpr int D = T::D, M = 128, NK = kChunkKeys, TILES = kChunkTiles;
    static constexpr int NT = NS == 1 ? 2 : 1;  // tiles of 128 rows per unit
    static constexpr int ROWS = NT * M;
    static constexpr int PARTS = FINE ? 2 : 1;  // of K^ and of P
    static constexpr int KHAT = PARTS * NK * D * 2, VHAT = NK * D * 2, IMAGE = KHAT + VHAT;
    // Q of tile 0 is in tensor memory where there is room, of the others in shared memory
    static constexpr bool Q0_TMEM = !(FINE && NT == 2);
    static constexpr int QSM = (NT - (Q0_TMEM ? 1 : 0)) * M * D * 2;
    static constexpr int LIMIT = 224 * 1024;             // of the CTA's 227 KB, the rest for barriers and statics
    // operand buffers: all that fit when lifted, else two of each, or one where two raw stages would not fit
    static constexpr int STAGE = LIFT ? 1 : TILES * T::BYTES;
    static constexpr int KB = LIFT ? (LIMIT - QSM) / IMAGE : (FINE && NS == 2 ? 1 : 2);
    static constexpr int VB = LIFT ? KB : ((LIMIT - QSM - KB * KHAT - 2 * VHAT) / STAGE >= 2 ? 2 : 1);
    static constexpr int OPS = QSM + KB * KHAT + VB * VHAT;
    static constexpr int STAGES_RAW = (LIMIT - OPS) / STAGE;
    static constexpr int STAGES = LIFT ? 0 : (STAGES_RAW > 4 ? 4 : STAGES_RAW);  // of raw tiles
    static constexpr int OFF_Q = STAGES * STAGE, OFF_K = OFF_Q + QSM, OFF_V = OFF_K + KB * KHAT;
    static constexpr int SMEM = OFF_V + VB * VHAT;
    // tensor memory columns: O of each tile, S of each, P of each, Q of tile 0
    static constexpr int PCOLS = PARTS * NK / 2;
    static constexpr int T_O = 0, T_S = NT * D, T_P = T_S + NT * NK, T_Q = T_P + NT * PCOLS;
    static_assert(T_Q + (Q0_TMEM ? D / 2 : 0) <= 512, "tensor memory");
    static_assert((LIFT || STAGES >= 2) && KB >= 1 && (!LIFT || KB >= 2) && VB >= 1 && KB <= 6 && SMEM <= LIMIT, "shared memory");
    static constexpr int SOFT0 = 4, CONV0 = SOFT0 + 4 * NT, CONV_WARPS = LIFT ? 0 : 8;  // first softmax / converter warp
    static constexpr int HALF = CONV_WARPS / 2;                                         // converters of K^, and of V^
    static constexpr int WARPS = CONV0 + CONV_WARPS;
    static constexpr int q_at(int tile) { return OFF_Q + (Q0_TMEM && tile > 0 ? tile - 1 : tile) * M * D * 2; }  // if not in tensor memory
    static constexpr int THREADS = WARPS * 32;
};

// ---- workspace: [per CTA: the unit it starts in][pieces: m, l][pieces: o][lifted: info][lifted: operands] ----
struct ChunkWork {
    int32_t *first;  // [CTAs][8]: sequence, head, unit, the unit's first step, its steps, span
    float *ml;       // [2 CTAs][ROWS][2]
    float *o;        // [2 CTAs][ROWS][D]
    int4 *info;      // [lift_cap]: copied tiles, exponents of K^ and V^
    uint8_t *image;  // [lift_cap][K^, V^]
    int lift_cap;    // blocks that fit; 0: not lifted
};
constexpr size_t kLiftBytes = size_t(2) << 30;  // most that lifted operands may take

// Most steps that one sequence of the call can have.
inline long long chunk_seq_steps(const PagedAttnParams &p, int rows) {
    return paged_steps((static_cast<long long>(p.v.max_len) + kChunkKeys) / kChunkKeys, static_cast<long long>(p.v.max_q) * p.G, rows, p.v.Hkv);
}

// Blocks (of one KV head) that the chunk class of a call can have, all heads together; 0 if their operands
// would pass kLiftBytes.
inline size_t image_bytes(int D, bool fine) { return static_cast<size_t>(kChunkKeys) * D * (fine ? 6 : 4); }
inline long long lift_blocks(const PagedAttnParams &p, int D, bool fine) {
    const long long seqs = p.v.n_tokens / p.from_q < p.v.n_seqs ? p.v.n_tokens / p.from_q : p.v.n_seqs;
    const long long per = p.v.max_len > 0 ? (static_cast<long long>(p.v.max_len) + kChunkKeys - 1) / kChunkKeys : 1;
    const long long most = static_cast<long long>(kLiftBytes / image_bytes(D, fine)), one = per * p.v.Hkv;
    return one <= most && seqs * one <= most ? seqs * one : 0;
}
inline ChunkWork chunk_work(const PagedAttnParams &p, int ctas, int rows, int D, bool fine, size_t *bytes) {
    uint8_t *w = static_cast<uint8_t *>(p.workspace);
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t ml = up(static_cast<size_t>(ctas) * 32), o = ml + up(static_cast<size_t>(2) * ctas * rows * 8);
    const size_t info = o + up(static_cast<size_t>(2) * ctas * rows * D * 4);
    const long long cap = lift_blocks(p, D, fine);
    const size_t image = info + up(static_cast<size_t>(cap) * 16);
    if (bytes) *bytes = image + static_cast<size_t>(cap) * image_bytes(D, fine);
    return ChunkWork{reinterpret_cast<int32_t *>(w), reinterpret_cast<float *>(w + ml), reinterpret_cast<float *>(w + o),
                     reinterpret_cast<int4 *>(w + info), w + image, static_cast<int>(cap)};
}

constexpr int kChunkMaxSeqs = 256;  // sequences of one launch (their prefix sums sit in shared memory)

// Units of a sequence and their steps.  A unit has at least one step, so that rows which attend to
// nothing are written too.
struct ChunkSeq {
    int first, n, len, units;  // units per KV head
};
template <int ROWS>
__device__ __forceinline__ ChunkSeq chunk_seq(const PagedView &v, int G, int from_q, int b) {
    const PagedSeq s = paged_seq(v, b);
    ChunkSeq c;
    c.first = s.first;
    c.n = s.n >= from_q ? s.n : 0;  // shorter ones belong to the split kernel
    c.len = s.len;
    c.units = static_cast<int>((static_cast<long long>(c.n) * G + ROWS - 1) / ROWS);
    return c;
}
template <int ROWS, int NK>
__device__ __forceinline__ int chunk_steps(const ChunkSeq &s, int G, int u) {
    const long long last_row = min(static_cast<long long>(s.n) * G, (static_cast<long long>(u) + 1) * ROWS) - 1;
    const int last = s.len - s.n + static_cast<int>(last_row / G);  // last position any row sees
    return max(1, (last + NK) / NK);
}

// blocks of 64 positions of a sequence (at least one, as its units have)
__device__ __forceinline__ int lift_blocks_of(const ChunkSeq &s) { return s.units > 0 ? max(1, (s.len + kChunkKeys - 1) / kChunkKeys) : 0; }

// In place: a[0 .. n) (counts) to a[0 .. n] (sums of those before), by one warp.
__device__ __forceinline__ void warp_prefix(int *a, int n) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int b0 = 0; b0 < n; b0 += 32) {
        const int own = b0 + lane < n ? a[b0 + lane] : 0;
        int x = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (b0 + lane < n) a[b0 + lane] = base + x - own;
        base += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) a[n] = base;
}

// The operands of every block of the sequences of the chunk class: one warp per (block, K^ or V^).
constexpr int kLiftWarps = 8;
template <int KT, int VT, int NS, bool FINE>
__global__ void __launch_bounds__(32 * kLiftWarps) paged_lift_kernel(const PagedAttnParams p, const ChunkWork work) {
    using C = ChunkCfg<KT, VT, NS, true, FINE>;
    using T = typename C::T;
    __shared__ int s_blocks[kChunkMaxSeqs + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PagedView &v = p.v;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    for (int b = threadIdx.x; b < v.n_seqs; b += 32 * kLiftWarps)
        s_blocks[b] = lift_blocks_of(chunk_seq<C::ROWS>(v, p.G, p.from_q, b)) * v.Hkv;
    __syncthreads();
    if (warp == 0) warp_prefix(s_blocks, v.n_seqs);
    __syncthreads();
    const int total = s_blocks[v.n_seqs];
    for (int item = blockIdx.x * kLiftWarps + warp; item < 2 * total; item += gridDim.x * kLiftWarps) {
        const int blk = item >> 1;
        const bool keys = (item & 1) == 0;
        int lo = 0, hi = v.n_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_blocks[mid] <= blk)
                lo = mid;
            else
                hi = mid;
        }
        if (s_blocks[lo + 1] > work.lift_cap) continue;  // left out of the chunk kernel, too
        const ChunkSeq s = chunk_seq<C::ROWS>(v, p.G, p.from_q, lo);
        const int per = lift_blocks_of(s), h = (blk - s_blocks[lo]) / per, kb = blk - s_blocks[lo] - h * per;
        // lane i has the page of tile i
        const int t = kb * C::TILES + (lane & (C::TILES - 1)), entry = t / v.page_tiles;
        const int page = t * kTileRows < s.len ? __ldg(v.table + static_cast<size_t>(lo) * v.stride + entry) : -1;
        const bool in = page >= 0 && page < v.n_pages;
        if (keys && !in && t * kTileRows < s.len && lane < C::TILES) paged_error(v);
        const BlockRows use{static_cast<int>(__ballot_sync(0xffffffffu, in) & ((1u << C::TILES) - 1u)), s.len - kb * C::NK};
        // a tile without a page reads the pool's first record; its rows are not in use
        const long long record = in ? (static_cast<long long>(page) * v.Hkv + h) * v.page_tiles + (t - entry * v.page_tiles) : 0;
        auto tile = [&](int i) -> const uint8_t * {  // by the whole warp; i may differ between lanes
            return v.pool + __shfl_sync(0xffffffffu, record, i) * T::BYTES;
        };
        uint8_t *image = work.image + static_cast<size_t>(blk) * C::IMAGE;
        int32_t *info = reinterpret_cast<int32_t *>(work.info + blk);
        if (keys) {
            const int e = block_exp<KT, T::OFF_KS, NS>(tile, use);
            if (lane == 0) info[0] = use.got, info[1] = e;
            convert_keys<KT, VT, NS, FINE>(tile, image, e, 0, 1);
        } else {
            const int e = block_exp<VT, T::OFF_VS, NS>(tile, use);
            if (lane == 0) info[2] = e;
            convert_values<KT, VT, NS>(tile, image + C::KHAT, e, use, 0, 1);
        }
    }
}

// A walk over the units of a span: unit u of head h of sequence b, its steps, and the range of them
// that belongs to this CTA.
struct ChunkWalk {
    ChunkSeq s;
    int b, h, u, steps;
};

template <int KT, int VT, int NS, int DT, bool LIFT>
__global__ void __launch_bounds__(ChunkCfg<KT, VT, NS, LIFT, chunk_fine<KT, DT>()>::THREADS, 1)
    paged_chunk_kernel(const PagedAttnParams p, const ChunkWork work) {
    constexpr bool FINE = chunk_fine<KT, DT>();
    using C = ChunkCfg<KT, VT, NS, LIFT, FINE>;
    using T = typename C::T;
    using X = typename Act<DT>::type;
    constexpr int D = C::D, NK = C::NK, NT = C::NT, ROWS = C::ROWS;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t raw_full[4], raw_empty[4], k_ready[6], k_free[6], v_ready[6], v_free[6];
    __shared__ __align__(8) uint64_t s_ready[2], s_free[2], p_ready[2], pv_done[2], q_ready[2], drain[3];
    __shared__ int s_pre[kChunkMaxSeqs + 1], s_blocks[LIFT ? kChunkMaxSeqs + 1 : 1];
    __shared__ int s_start[4];                       // sequence, head, unit, step of this CTA's first step
    __shared__ int s_ok[8], s_exp[8][2];             // per block: copied tiles; exponents of K^ and V^
    __shared__ uint32_t s_tmem;
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const PagedView &v = p.v;
    const int G = p.G;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(raw_full + i, 1);
            mbar_init(raw_empty + i, C::CONV_WARPS);
        }
        for (int i = 0; i < C::KB; ++i) {
            mbar_init(k_ready + i, LIFT ? 1 : C::HALF);
            mbar_init(k_free + i, NT);
        }
        for (int i = 0; i < C::VB; ++i) {
            mbar_init(v_ready + i, LIFT ? 1 : C::HALF);
            mbar_init(v_free + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_ready + i, 1);
            mbar_init(s_free + i, 4);
            mbar_init(p_ready + i, 4);
            mbar_init(pv_done + i, 1);
            mbar_init(q_ready + i, 4);
        }
        for (int i = 0; i < 3; ++i) mbar_init(drain + i, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&s_tmem)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    }
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

    // ---- steps before each sequence, and where this CTA starts ----
    if constexpr (LIFT) {
        for (int b = threadIdx.x; b < v.n_seqs; b += C::THREADS)
            s_blocks[b] = lift_blocks_of(chunk_seq<ROWS>(v, G, p.from_q, b)) * v.Hkv;
        __syncthreads();
        if (warp == 0) warp_prefix(s_blocks, v.n_seqs);
        __syncthreads();
    }
    for (int b = warp; b < v.n_seqs; b += C::WARPS) {
        const ChunkSeq s = chunk_seq<ROWS>(v, G, p.from_q, b);
        int sum = 0;
        for (int u = lane; u < s.units; u += 32) sum += chunk_steps<ROWS, NK>(s, G, u);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        bool ok = paged_seq(v, b).ok;
        if (LIFT && s_blocks[b + 1] > work.lift_cap) {  // more tokens than the call has: offsets that overlap
            ok = false;
            sum = 0;
        }
        if (lane == 0) s_pre[b] = sum * v.Hkv;
        if (blockIdx.x == 0 && lane == 0 && !ok) paged_error(v);
    }
    t5_fence_before();
    __syncthreads();
    t5_fence_after();
    if (warp == 0) warp_prefix(s_pre, v.n_seqs);
    __syncthreads();
    const int total = s_pre[v.n_seqs];
    // at least kMinSpan steps per CTA: shorter spans cost more in pieces than they gain
    constexpr int kMinSpan = 4;
    const int span = max(kMinSpan, (total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x));
    const long long x0l = static_cast<long long>(blockIdx.x) * span;
    const int x0 = x0l < total ? static_cast<int>(x0l) : total, x1 = min(total, x0 + span);
    const int NX = x1 - x0;  // steps of this CTA
    if (NX > 0 && warp == 0) {
        int lo = 0, hi = v.n_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_pre[mid] <= x0)
                lo = mid;
            else
                hi = mid;
        }
        const ChunkSeq s = chunk_seq<ROWS>(v, G, p.from_q, lo);
        const int per_head = (s_pre[lo + 1] - s_pre[lo]) / v.Hkv;
        int r = x0 - s_pre[lo];
        const int h = r / per_head;
        r -= h * per_head;
        // the unit: 32 at a time
        for (int u0 = 0; u0 < s.units; u0 += 32) {
            const int own = u0 + lane < s.units ? chunk_steps<ROWS, NK>(s, G, u0 + lane) : 0;
            int inc = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, r < inc);
            if (hit) {
                const int w = __ffs(hit) - 1;
                const int before = __shfl_sync(0xffffffffu, inc - own, w);
                if (lane == 0) {
                    s_start[0] = lo;
                    s_start[1] = h;
                    s_start[2] = u0 + w;
                    s_start[3] = r - before;
                }
                break;
            }
            r -= __shfl_sync(0xffffffffu, inc, 31);
        }
    }
    __syncthreads();
    const uint32_t tm = __shfl_sync(0xffffffffu, s_tmem, 0);

    // every role walks the same segments: [c0, c1) are the steps of unit (b, h, u) in this CTA
    auto begin = [&]() {
        ChunkWalk w;
        w.b = s_start[0];
        w.h = s_start[1];
        w.u = s_start[2];
        w.s = chunk_seq<ROWS>(v, G, p.from_q, w.b);
        w.steps = chunk_steps<ROWS, NK>(w.s, G, w.u);
        return w;
    };
    auto advance = [&](ChunkWalk &w) {
        if (++w.u == w.s.units) {
            w.u = 0;
            if (++w.h == v.Hkv) {
                w.h = 0;
                ++w.b;
                while (s_pre[w.b + 1] == s_pre[w.b]) ++w.b;
                w.s = chunk_seq<ROWS>(v, G, p.from_q, w.b);
            }
        }
        w.steps = chunk_steps<ROWS, NK>(w.s, G, w.u);
    };
    // rows of tile t in a unit
    auto tile_rows = [&](const ChunkWalk &w, int t) {
        const long long left = static_cast<long long>(w.s.n) * G - static_cast<long long>(w.u) * ROWS - t * C::M;
        return static_cast<int>(left < 0 ? 0 : (left > C::M ? C::M : left));
    };

    if (NX > 0) {
        if (LIFT && warp == 0) {
            // ---------------- copies of lifted operands ----------------
            ChunkWalk w = begin();
            int t = s_start[3], issued = 0;
            bool ok = true;
            int4 info = make_int4(0, 0, 0, 0);
            size_t blk = 0;
            auto look_up = [&]() {  // a step ahead
                blk = static_cast<size_t>(s_blocks[w.b] + w.h * lift_blocks_of(w.s) + t);
                info = __ldcg(work.info + blk);
            };
            look_up();
            for (int x = 0; x < NX; ++x) {
                const int buf = x % C::KB, use = x / C::KB;
                if (use > 0) ok = __all_sync(0xffffffffu, paged_wait(k_free + buf, (use - 1) & 1));
                if (!ok) break;
                const uint8_t *src = work.image + blk * C::IMAGE;
                if (lane == 0) {
                    s_ok[x & 7] = info.x;
                    s_exp[x & 7][0] = info.y;
                    s_exp[x & 7][1] = info.z;
                }
                __syncwarp();
                if (t5_elect()) {
                    mbar_arrive_expect_tx(k_ready + buf, C::KHAT);
                    bulk_g2s(smem + C::OFF_K + buf * C::KHAT, src, C::KHAT, k_ready + buf);
                }
                __syncwarp();
                if (use > 0) ok = __all_sync(0xffffffffu, paged_wait(v_free + buf, (use - 1) & 1));
                if (ok && t5_elect()) {
                    mbar_arrive_expect_tx(v_ready + buf, C::VHAT);
                    bulk_g2s(smem + C::OFF_V + buf * C::VHAT, src + C::KHAT, C::VHAT, v_ready + buf);
                }
                __syncwarp();
                issued = x + 1;
                if (!ok) break;
                if (x + 1 < NX) {
                    if (++t == w.steps) {
                        advance(w);
                        t = 0;
                    }
                    look_up();
                }
            }
            if (!ok && lane == 0) atomicOr(v.err, KVQ_DEVERR_TIMEOUT);
            for (int i = 0; i < C::KB; ++i)  // every copy lands before the memory is freed
                if (i < issued) {
                    (void)paged_wait(k_ready + i, ((issued - 1 - i) / C::KB) & 1);
                    (void)paged_wait(v_ready + i, ((issued - 1 - i) / C::KB) & 1);
                }
            __syncwarp();
        } else if (!LIFT && warp == 0) {
            // ---------------- copies of raw tiles ----------------
            // lane i < 4 has tile i of the block; its page number is looked up one step ahead
            ChunkWalk w = begin();
            int t = s_start[3], issued = 0, page = -1, tile = 0, tiles = 0;
            const size_t page_bytes = static_cast<size_t>(v.page_tiles) * T::BYTES;
            const bool one_page = v.page_tiles % C::TILES == 0;  // a block never crosses a page: one copy
            auto look_up = [&]() {
                tiles = (w.s.len + kTileRows - 1) / kTileRows;
                tile = t * C::TILES + (lane & (C::TILES - 1));
                page = tile < tiles ? __ldg(v.table + static_cast<size_t>(w.b) * v.stride + tile / v.page_tiles) : -1;
            };
            look_up();
            bool ok = true;
            for (int x = 0; x < NX; ++x) {
                constexpr int STAGES = LIFT ? 1 : C::STAGES;
                const int st = x % STAGES, use = x / STAGES;
                if (use > 0) ok = __all_sync(0xffffffffu, paged_wait(raw_empty + st, (use - 1) & 1));
                if (!ok) break;
                const bool in = page >= 0 && page < v.n_pages;
                if (!in && tile < tiles && lane < C::TILES) paged_error(v);
                const int got = __ballot_sync(0xffffffffu, in) & ((1 << C::TILES) - 1);
                if (lane == 0) {
                    s_ok[x & 7] = got;
                    mbar_arrive_expect_tx(raw_full + st, static_cast<uint32_t>(__popc(got) * T::BYTES));
                }
                __syncwarp();
                const uint8_t *src = v.pool + (static_cast<size_t>(page) * v.Hkv + w.h) * page_bytes +
                                     static_cast<size_t>(tile % v.page_tiles) * T::BYTES;
                if (one_page) {
                    if (lane == 0 && got) bulk_g2s(smem + st * C::STAGE, src, __popc(got) * T::BYTES, raw_full + st);
                } else if (in && lane < C::TILES) {
                    bulk_g2s(smem + st * C::STAGE + lane * T::BYTES, src, T::BYTES, raw_full + st);
                }
                issued = x + 1;
                if (x + 1 < NX) {
                    if (++t == w.steps) {
                        advance(w);
                        t = 0;
                    }
                    look_up();
                }
            }
            if (!ok && lane == 0) atomicOr(v.err, KVQ_DEVERR_TIMEOUT);
            for (int i = 0; i < C::STAGES; ++i)  // every copy lands before the memory is freed
                if (i < issued) (void)paged_wait(raw_full + i, ((issued - 1 - i) / (LIFT ? 1 : C::STAGES)) & 1);
            __syncwarp();
        } else if (warp < C::SOFT0) {
            // ---------------- MMA issue: warp 1 S = Q K^T of every tile, warps 2 and 3 O += P V^ of one ----------------
            // A step costs each of these warps about 100 cycles per wait besides the MMAs, so the products that
            // wait for the softmax have their own streams.
            if (warp == 3 && lane == 0) {  // for the merge: the unit that this CTA starts in
                const ChunkWalk w = begin();
                int32_t *e = work.first + 8 * blockIdx.x;
                e[0] = w.b;
                e[1] = w.h;
                e[2] = w.u;
                e[3] = x0 - s_start[3];  // its first step
                e[4] = w.steps;
                e[5] = span;
            }
            __syncwarp();
            constexpr uint32_t ID_S = t5_idesc(C::M, NK), ID_O = t5_idesc(C::M, D);
            auto wait = [&](uint64_t *bar, int phase) {
                const bool got = __all_sync(0xffffffffu, paged_wait(bar, phase)) != 0;
                t5_fence_after();
                return got;
            };
            ChunkWalk w = begin();
            int c0 = s_start[3], x = 0;
            bool ok = true;
            if (warp == 1 || (NT == 2 && warp == 2)) {
                const int tile = warp - 1;
                const uint64_t qd = t5_desc(smem_u32(smem + C::q_at(tile)), 128, D * 16), kd = t5_desc(smem_u32(smem + C::OFF_K), 128, D * 16);
                int buf = 0, kphase = 0, sphase = 0, qphase = 0;  // the next phase of each barrier
                while (x < NX && ok) {
                    const int n = min(w.steps - c0, NX - x);  // steps of this segment
                    const bool live = tile_rows(w, tile) > 0;
                    for (int c = 0; c < n && ok; ++c, ++x) {
                        const uint64_t b = t5_plus(kd, buf * C::KHAT);
                        ok = wait(k_ready + buf, kphase);
                        if (!live) {
                            if (lane == 0) mbar_arrive(k_free + buf);
                        } else {
                            if (c == 0) {
                                ok = ok && wait(q_ready + tile, qphase);
                                qphase ^= 1;
                            } else {
                                ok = ok && wait(s_free + tile, sphase ^ 1);
                            }
                            sphase ^= 1;
                            if (ok && t5_elect()) {
                                // lo follows hi by NK D 2 bytes
                                constexpr int QK = D / 16, LO = NK * D * 2 / 16 - 16 * QK;
                                if (C::Q0_TMEM && tile == 0) {
#pragma unroll
                                    for (int k = 0; k < C::PARTS * QK; ++k) t5_mma_ts(tm + C::T_S, tm + C::T_Q + 8 * (k % QK), b + 16 * k + k / QK * LO, ID_S, k > 0);
                                } else {
#pragma unroll
                                    for (int k = 0; k < C::PARTS * QK; ++k) t5_mma_ss(tm + C::T_S + tile * NK, qd + 16 * (k % QK), b + 16 * k + k / QK * LO, ID_S, k > 0);
                                }
                                t5_commit(s_ready + tile);
                                t5_commit(k_free + buf);
                            }
                            __syncwarp();
                        }
                        if (++buf == C::KB) buf = 0, kphase ^= 1;
                    }
                    if (x < NX && ok) advance(w);
                    c0 = 0;
                }
            } else if (NT == 2 || warp == 2) {
                const uint64_t vd = t5_desc(smem_u32(smem + C::OFF_V), 128, NK * 16);
                int buf = 0, vphase = 0, pphase[2] = {0, 0};
                while (x < NX && ok) {
                    const int n = min(w.steps - c0, NX - x);
                    const int nt = NT == 2 && tile_rows(w, NT - 1) > 0 ? 2 : 1;
                    for (int c = 0; c < n && ok; ++c, ++x) {
                        const uint64_t b = t5_plus(vd, buf * C::VHAT);
                        const uint32_t add = t5_uniform(c == 0 ? 0u : 1u);
                        ok = wait(v_ready + buf, vphase);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            if (t >= nt || !ok) break;
                            ok = wait(p_ready + t, pphase[t]);
                            pphase[t] ^= 1;
                            if (ok && t5_elect()) {
#pragma unroll
                                for (int k = 0; k < C::PARTS * NK / 16; ++k) t5_mma_ts(tm + C::T_O + t * D, tm + C::T_P + t * C::PCOLS + 8 * k, b + 16 * (k % (NK / 16)), ID_O, k > 0 ? 1u : add);
                                t5_commit(pv_done + t);
                            }
                            __syncwarp();
                        }
                        if (ok && t5_elect()) t5_commit(v_free + buf);
                        __syncwarp();
                        if (++buf == C::VB) buf = 0, vphase ^= 1;
                    }
                    if (x < NX && ok) advance(w);
                    c0 = 0;
                }
            }
            if (!ok && lane == 0) atomicOr(v.err, KVQ_DEVERR_TIMEOUT);
            // every MMA has completed before tensor memory is freed
            if (t5_elect()) t5_commit(drain + warp - 1);
            __syncwarp();
            (void)paged_wait(drain + warp - 1, 0);
        } else if (!LIFT && warp >= C::CONV0) {
            // ---------------- converters: codes -> K^ (first half of the warps), V^ (second half) ----------------
            const bool keys = warp < C::CONV0 + C::HALF;
            const int cw = warp - C::CONV0 - (keys ? 0 : C::HALF);
            ChunkWalk w = begin();
            int t = s_start[3];
            bool ok = true;
            for (int x = 0; x < NX && ok; ++x) {
                constexpr int STAGES = LIFT ? 1 : C::STAGES, HALF = LIFT ? 1 : C::HALF;
                const int sg = x % STAGES;
                const uint8_t *st = smem + sg * C::STAGE;
                ok = paged_wait(raw_full + sg, (x / STAGES) & 1);
                const int buf = keys ? x % C::KB : x % C::VB, use_no = keys ? x / C::KB : x / C::VB;
                if (use_no > 0) ok = paged_wait((keys ? k_free : v_free) + buf, (use_no - 1) & 1) && ok;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const BlockRows use{s_ok[x & 7], w.s.len - t * NK};
                auto tile = [&](int i) { return st + i * T::BYTES; };
                if (keys) {
                    const int e = block_exp<KT, T::OFF_KS, NS>(tile, use);
                    if (cw == 0 && lane == 0) s_exp[x & 7][0] = e;
                    if (cw == 1) {  // the softmax warps need V^'s exponent with S, perhaps before V^ is made
                        const int ev = block_exp<VT, T::OFF_VS, NS>(tile, use);
                        if (lane == 0) s_exp[x & 7][1] = ev;
                    }
                    convert_keys<KT, VT, NS, FINE>(tile, smem + C::OFF_K + buf * C::KHAT, e, cw, HALF);
                } else {
                    const int e = block_exp<VT, T::OFF_VS, NS>(tile, use);
                    convert_values<KT, VT, NS>(tile, smem + C::OFF_V + buf * C::VHAT, e, use, cw, HALF);
                }
                smem_to_async();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive((keys ? k_ready : v_ready) + buf);
                    mbar_arrive(raw_empty + sg);  // this warp's part of the stage has been read
                }
                if (++t == w.steps && x + 1 < NX) {
                    advance(w);
                    t = 0;
                }
            }
            if (!ok && lane == 0) atomicOr(v.err, KVQ_DEVERR_TIMEOUT);
        } else if (warp >= C::SOFT0 && warp < C::CONV0) {
            // ---------------- one query row per thread ----------------
            const int tile = (warp - C::SOFT0) >> 2, quarter = warp & 3;
            const int r = 32 * quarter + lane;  // row of the tile = lane of tensor memory
            const uint32_t trow = tm + (static_cast<uint32_t>(32 * quarter) << 16);
            const uint32_t tS = trow + C::T_S + tile * NK, tP = trow + C::T_P + tile * C::PCOLS, tO = trow + C::T_O + tile * D;
            const bool q_tmem = C::Q0_TMEM && tile == 0;
            ChunkWalk w = begin();
            int c0 = s_start[3], x = 0, done = 0;
            bool ok = true;
            while (x < NX && ok) {
                const int n = min(w.steps - c0, NX - x);
                const int rows = tile_rows(w, tile);
                const bool live = rows > 0;
                const long long rr = static_cast<long long>(w.u) * ROWS + tile * C::M + r;  // row of the (sequence, head)
                const bool rv = r < rows;
                const int i = rv ? static_cast<int>(rr / G) : 0;
                const size_t orow = (static_cast<size_t>(w.s.first) + i) * p.Hq + static_cast<size_t>(w.h) * G + (rv ? rr % G : 0);
                const int lim = w.s.len - w.s.n + i;  // last position of the row
                // ---- the row's query as f16 ----
                const X *src = static_cast<const X *>(p.q) + (static_cast<size_t>(w.s.first) + i) * p.q_stride +
                               (static_cast<size_t>(w.h) * G + (rv ? rr % G : 0)) * D;
                float rs = 0.f;
                if (live) {
                    // a part of the row is loaded at once: a load at a time would wait for memory each time
                    constexpr int PART = LIFT ? 128 : 64;
                    auto stage = [&](float up) {  // the row times `up` (a power of two); its largest |value|
                        float top = 0.f;
#pragma unroll 1
                        for (int p0 = 0; p0 < D; p0 += PART) {
                            uint4 raw[PART / 8];
#pragma unroll
                            for (int e = 0; e < PART / 8; ++e)
                                raw[e] = rv ? *reinterpret_cast<const uint4 *>(src + p0 + 8 * e) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                            for (int d0 = 0; d0 < PART; d0 += 32) {
                                uint32_t h[16];
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const uint4 r4 = raw[d0 / 8 + e / 2];
                                    const float4 q4 = Act<DT>::widen((e & 1) ? make_uint2(r4.z, r4.w) : make_uint2(r4.x, r4.y));
                                    top = max3(top, fabsf(q4.x), fabsf(q4.y));
                                    top = max3(top, fabsf(q4.z), fabsf(q4.w));
                                    h[2 * e] = h2_as_u32(__floats2half2_rn(q4.x * up, q4.z * up));
                                    h[2 * e + 1] = h2_as_u32(__floats2half2_rn(q4.y * up, q4.w * up));
                                }
                                if (q_tmem) {
                                    t5_st16(trow + C::T_Q + (p0 + d0) / 2, h);
                                } else {
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        *reinterpret_cast<uint4 *>(smem + C::q_at(tile) + core_at(r, p0 + d0 + 8 * e, D)) =
                                            make_uint4(h[4 * e], h[4 * e + 1], h[4 * e + 2], h[4 * e + 3]);
                                }
                            }
                        }
                        return top;
                    };
                    // a negative scale goes to the query: rs >= 0, so the largest score is the largest product
                    const float sign = p.scale < 0.f ? -1.f : 1.f;
                    rs = fabsf(p.scale) * kChunkLog2e;
                    const float top = stage(sign);
                    if constexpr (DT == KVQ_DT_BF16) {
                        // rows whose largest value is outside 2^-6 .. 2^15 once more, moved to 2^10 .. 2^11: f16 then
                        // holds values down to 2^-27 of it exactly, smaller ones to 2^-35 of it (inside, the least
                        // case is a largest value of 2^-6: to 2^-19 of it)
                        const int ex = static_cast<int>(__float_as_uint(top) >> 23);
                        const bool off = top != 0.f && ex != 255 && (ex < 127 - 6 || ex > 127 + 14);
                        if (__any_sync(0xffffffffu, off)) {
                            keep_branch();
                            const int k = off ? max(-120, min(120, 10 - (ex - 127))) : 0;
                            if (q_tmem) t5_wait_st();
                            (void)stage(sign * __int_as_float((127 + k) << 23));
                            rs *= __int_as_float((127 - k) << 23);
                        }
                    }
                    if (q_tmem)
                        t5_wait_st();
                    else
                        smem_to_async();
                }
                t5_fence_before();
                __syncwarp();
                if (live && lane == 0) mbar_arrive(q_ready + tile);
                float m_run = -CUDART_INF_F, l = 0.f;
                if (!live) {
                    x += n;
                } else {
                    for (int c = 0; c < n && ok; ++c, ++x, ++done) {
                        ok = __all_sync(0xffffffffu, paged_wait(s_ready + tile, done & 1));
                        if (!ok) break;
                        t5_fence_after();
                        uint32_t su[NK];
                        t5_ld32(tS, su);
                        t5_ld32(tS + 32, su + 32);
                        const int got = s_ok[x & 7], ek = s_exp[x & 7][0], ev = s_exp[x & 7][1];
                        t5_wait_ld();
                        t5_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(s_free + tile);
                        float s[NK];
#pragma unroll
                        for (int k = 0; k < NK; ++k) s[k] = __uint_as_float(su[k]);
                        // never 0, so that a masked score stays -inf
                        const float f = fmaxf(rs * __int_as_float((127 + ek) << 23), 1e-36f);
                        // keys behind the row's position (and so past the end) and those in no page
                        const int key0 = (c0 + c) * NK;
                        if (__any_sync(0xffffffffu, rv && key0 + NK - 1 > lim) || got != (1 << C::TILES) - 1) {
                            keep_branch();
#pragma unroll
                            for (int k = 0; k < NK; ++k)
                                if (key0 + k > lim || !((got >> (k / kTileRows)) & 1)) s[k] = -CUDART_INF_F;
                        }
                        float mq[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                        for (int k = 4; k + 8 <= NK; k += 8)
#pragma unroll
                            for (int e = 0; e < 4; ++e) mq[e] = max3(mq[e], s[k + 2 * e], s[k + 2 * e + 1]);
                        mq[0] = max3(mq[0], s[NK - 4], s[NK - 3]);
                        mq[1] = max3(mq[1], s[NK - 2], s[NK - 1]);
                        const float mx = fmaxf(max3(mq[0], mq[1], mq[2]), mq[3]) * f;
                        const bool need = mx > m_run + kChunkDrift;
                        float alpha = 1.f;
                        if (need) {
                            alpha = m_run == -CUDART_INF_F ? 0.f : chunk_ex2(m_run - mx);
                            m_run = mx;
                            l *= alpha;
                        }
                        // weights times 2^ev (the values were stored times 2^-ev)
                        const float base = (m_run == -CUDART_INF_F ? 0.f : m_run) - static_cast<float>(ev);
                        const float2 f2 = make_float2(f, f), nb2 = make_float2(-base, -base);
                        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                        uint32_t pw[NK / 2], pl[FINE ? NK / 2 : 1];  // weights, and what their rounding left
#pragma unroll
                        for (int k = 0; k < NK / 2; ++k) {
                            float2 a = pair_fma(make_float2(s[2 * k], s[2 * k + 1]), f2, nb2);
                            a.x = chunk_ex2(a.x);
                            a.y = chunk_ex2(a.y);
                            sum[k & 1] = pair_add(sum[k & 1], a);
                            const __half2 hi = __floats2half2_rn(a.x, a.y);
                            pw[k] = h2_as_u32(hi);
                            if constexpr (FINE) {
                                const float2 f = __half22float2(hi);
                                pl[k] = h2_as_u32(__floats2half2_rn(a.x - f.x, a.y - f.y));
                            }
                        }
                        sum[0] = pair_add(sum[0], sum[1]);
                        l += (sum[0].x + sum[0].y) * __int_as_float((127 - ev) << 23);
                        // P and O are free once the previous block's P V^ is done
                        if (c > 0) ok = __all_sync(0xffffffffu, paged_wait(pv_done + tile, (done - 1) & 1));
                        if (!ok) break;
                        t5_fence_after();
                        if (c > 0 && __any_sync(0xffffffffu, need)) {
#pragma unroll 1
                            for (int d0 = 0; d0 < D; d0 += 32) {
                                uint32_t o[32];
                                t5_ld32(tO + d0, o);
                                t5_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const float2 y = pair_mul(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), make_float2(alpha, alpha));
                                    o[e] = __float_as_uint(y.x);
                                    o[e + 1] = __float_as_uint(y.y);
                                }
                                t5_st32(tO + d0, o);
                            }
                        }
                        t5_st32(tP, pw);
                        if constexpr (FINE) t5_st32(tP + NK / 2, pl);
                        t5_wait_st();
                        t5_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(p_ready + tile);
                    }
                    if (!ok) break;
                    ok = __all_sync(0xffffffffu, paged_wait(pv_done + tile, (done - 1) & 1));
                    if (!ok) break;
                    t5_fence_after();
                    const bool whole = c0 == 0 && n == w.steps;
                    if (whole) {
                        const float inv = l > 0.f ? 1.f / l : 0.f;
                        X *dst = static_cast<X *>(p.out) + orow * D;
#pragma unroll 1
                        for (int d0 = 0; d0 < D; d0 += 32) {
                            uint32_t o[32];
                            t5_ld32(tO + d0, o);
                            t5_wait_ld();
                            if (rv)
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const int i0 = 16 * (e >> 2) + 2 * (e & 3);
                                    Act<DT>::store4(dst + d0 + 4 * e, make_float4(__uint_as_float(o[i0]) * inv, __uint_as_float(o[i0 + 8]) * inv,
                                                                                  __uint_as_float(o[i0 + 1]) * inv, __uint_as_float(o[i0 + 9]) * inv));
                                }
                        }
                        if (rv && p.lse) p.lse[orow] = l > 0.f ? (m_run + __log2f(l)) * kChunkLn2 : -CUDART_INF_F;
                    } else {
                        // the first segment of the CTA, or its last
                        const size_t piece = (static_cast<size_t>(2) * blockIdx.x + (x - n > 0 ? 1 : 0)) * ROWS + tile * C::M + r;
                        float *dst = work.o + piece * D;
#pragma unroll 1
                        for (int d0 = 0; d0 < D; d0 += 32) {
                            uint32_t o[32];
                            t5_ld32(tO + d0, o);
                            t5_wait_ld();
                            if (rv)
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const int i0 = 16 * (e >> 2) + 2 * (e & 3);
                                    *reinterpret_cast<uint4 *>(dst + d0 + 4 * e) = make_uint4(o[i0], o[i0 + 8], o[i0 + 1], o[i0 + 9]);
                                }
                        }
                        work.ml[2 * piece] = m_run;
                        work.ml[2 * piece + 1] = l;
                    }
                }
                if (x < NX) advance(w);
                c0 = 0;
            }
            if (!ok && lane == 0) atomicOr(v.err, KVQ_DEVERR_TIMEOUT);
        }
    } else if (threadIdx.x == 0) {
        work.first[8 * blockIdx.x + 4] = 0;  // nothing starts here
    }
    t5_fence_before();
    __syncthreads();
    t5_fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tm), "r"(512));
}

// Merge of the pieces.  Block (c, group of 8 rows): the unit that CTA c starts in, if CTA c - 1 began it.
template <int NS, int DT>
__global__ void __launch_bounds__(256)
    paged_chunk_merge(const PagedAttnParams p, const ChunkWork work, const int rows_per_unit) {
    using X = typename Act<DT>::type;
    constexpr int D = NS * kSlice, DQ = D / 4;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int c = blockIdx.x + 1;
    const int32_t *e = work.first + 8 * c;
    const int steps = e[4];
    if (steps == 0) return;
    const int b = e[0], h = e[1], u = e[2], u0 = e[3], span = e[5];
    const long long here = static_cast<long long>(c) * span;
    if (u0 == here || u0 < here - span) return;  // the unit starts with CTA c, or before CTA c - 1
    const PagedSeq s = paged_seq(p.v, b);
    const int cl = (u0 + steps - 1) / span;  // last CTA with a piece
    const int pieces = cl - (c - 1) + 1;
    const int first_slot = 2 * (c - 1) + (u0 == here - span ? 0 : 1);
    for (int item = threadIdx.x; item < 8 * DQ; item += blockDim.x) {
        const int row = blockIdx.y * 8 + item / DQ, col = item % DQ;
        const long long rr = static_cast<long long>(u) * rows_per_unit + row;
        if (rr >= static_cast<long long>(s.n) * p.G) continue;
        float M = -CUDART_INF_F, L = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kAt = 4;
        for (int i0 = 0; i0 < pieces; i0 += kAt) {
            float pm[kAt], pl[kAt];
            float4 po[kAt];
#pragma unroll
            for (int k = 0; k < kAt; ++k) {
                pm[k] = -CUDART_INF_F;
                pl[k] = 0.f;
                po[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i0 + k < pieces) {
                    const int slot = i0 + k == 0 ? first_slot : 2 * (c - 1 + i0 + k);
                    const size_t at = static_cast<size_t>(slot) * rows_per_unit + row;
                    pm[k] = __ldcg(work.ml + 2 * at);
                    pl[k] = __ldcg(work.ml + 2 * at + 1);
                    po[k] = __ldcg(reinterpret_cast<const float4 *>(work.o + at * D) + col);
                }
            }
            float mn = M;
#pragma unroll
            for (int k = 0; k < kAt; ++k) mn = fmaxf(mn, pm[k]);
            if (mn == -CUDART_INF_F) continue;
            const float k0 = M == -CUDART_INF_F ? 0.f : chunk_ex2(M - mn);
            a = make_float4(a.x * k0, a.y * k0, a.z * k0, a.w * k0);
            L *= k0;
#pragma unroll
            for (int k = 0; k < kAt; ++k) {
                const float q = pm[k] == -CUDART_INF_F ? 0.f : chunk_ex2(pm[k] - mn);
                a = make_float4(fmaf(q, po[k].x, a.x), fmaf(q, po[k].y, a.y), fmaf(q, po[k].z, a.z), fmaf(q, po[k].w, a.w));
                L = fmaf(q, pl[k], L);
            }
            M = mn;
        }
        const size_t orow = (static_cast<size_t>(s.first) + rr / p.G) * p.Hq + static_cast<size_t>(h) * p.G + rr % p.G;
        const float inv = L > 0.f ? 1.f / L : 0.f;
        Act<DT>::store4(static_cast<X *>(p.out) + orow * D + 4 * col, make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv));
        if (col == 0 && p.lse) p.lse[orow] = L > 0.f ? (M + __log2f(L)) * kChunkLn2 : -CUDART_INF_F;
    }
}

template <int KT, int VT, int NS, int DT, bool LIFT>
cudaError_t launch_chunk_t(const PagedAttnParams &p, cudaStream_t stream) {
    constexpr bool FINE = chunk_fine<KT, DT>();
    using C = ChunkCfg<KT, VT, NS, LIFT, FINE>;
    static bool configured[kPagedMaxDevices] = {};
    int dev = 0, sms = 0;
    cudaError_t e = paged_device(&dev, &sms);
    if (e != cudaSuccess) return e;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(paged_chunk_kernel<KT, VT, NS, DT, LIFT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    const ChunkWork work = chunk_work(p, sms, C::ROWS, C::D, FINE, nullptr);
    // sequences of one launch: their prefix sums fit shared memory, their steps 2^30
    const long long fit = kPagedMaxSteps / chunk_seq_steps(p, C::ROWS);
    const int most = static_cast<int>(fit < kChunkMaxSeqs ? fit : kChunkMaxSeqs);
    if (most < 1) return cudaErrorNotSupported;
    for (int b = 0; b < p.v.n_seqs; b += most) {
        const PagedAttnParams q = paged_some(p, b, most);
        if (LIFT) {
            e = launch_dependent(paged_lift_kernel<KT, VT, NS, FINE>, dim3(sms * 4), 32 * kLiftWarps, 0, stream, q, work);
            if (e != cudaSuccess) return e;
        }
        e = launch_dependent(paged_chunk_kernel<KT, VT, NS, DT, LIFT>, dim3(sms), C::THREADS, C::SMEM, stream, q, work);
        if (e != cudaSuccess) return e;
        if (sms == 1) continue;
        e = launch_dependent(paged_chunk_merge<NS, DT>, dim3(sms - 1, C::ROWS / 8), 256, 0, stream, q, work, static_cast<int>(C::ROWS));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <int DT>
cudaError_t launch_chunk_dt(int type_k, int type_v, int D, const PagedAttnParams &p, cudaStream_t s) {
    const bool lift = lift_blocks(p, D, type_k != KVQ_F16 && DT == KVQ_DT_F16) > 0;
#define KVQ_CHUNK_CASE(KT_, VT_)                                                  \
    if (type_k == KT_ && type_v == VT_) {                                                            \
        if (D == kSlice) return lift ? launch_chunk_t<KT_, VT_, 1, DT, true>(p, s) : launch_chunk_t<KT_, VT_, 1, DT, false>(p, s);     \
        if (D == 2 * kSlice) return lift ? launch_chunk_t<KT_, VT_, 2, DT, true>(p, s) : launch_chunk_t<KT_, VT_, 2, DT, false>(p, s); \
    }
    KVQ_CHUNK_CASE(KVQ_F16, KVQ_F16)
    KVQ_CHUNK_CASE(KVQ_Q8_0, KVQ_Q8_0)
    KVQ_CHUNK_CASE(KVQ_Q8_0, KVQ_Q4_0)
    KVQ_CHUNK_CASE(KVQ_Q4_0, KVQ_Q4_0)
#undef KVQ_CHUNK_CASE
    return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace kvq
