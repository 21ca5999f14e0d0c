// kvq_paged_split.cuh -- attention of few queries per sequence over the paged cache: a split-K
// kernel whose warps share all live keys evenly, and the merge of its pieces.
//
// Mathematics.  For up to eight query rows r of one (sequence, KV head), s = scale q_r.k_t,
// out = sum_t 2^(s'_t - m) v_t / sum_t 2^(s'_t - m) with s' = s log2(e) and m a running
// maximum; any cut of the keys into ranges merges exactly from (sum p v, sum p, m).
//
// Split.  The keys of all (sequence, KV head, row group) units are laid end to end, in steps of
// one or two 16-key tiles, and cut into equal spans, one per warp of a grid with one CTA per SM:
// whatever the lengths, every warp reads the same number of bytes.  A warp keeps its own ring of
// shared-memory slots, filled by one bulk copy per tile record (or per pair in one page), so no
// warp waits for another until the end, where the warps that worked on one unit merge in shared
// memory.  What is not the whole of its unit goes to the workspace as a piece (m, l, o), and a
// second kernel merges the pieces; a unit that lay in one CTA is written at once.  Short contexts in few
// units take one CTA per unit instead (UNITS): no sums over the batch, no pieces and no second kernel.
//
// Products.  Keys and values are the A operands of mma.sync m16n8k16 (16 keys, or 16 values, by
// 16) and the query rows its eight columns, so one instruction serves 16 keys x 8 rows without
// waste, and the accumulators of O^T need four registers per 16 values.  Codes enter as f16
// subnormals (a permute or a mask and no arithmetic; for fp32 activations as normal numbers); scales multiply S in fp32 and P in f16.
// tcgen05 would need M = 128 query rows and the codes converted to f16 in shared memory, more
// instructions per byte than this kernel issues in all.
//
// Measured (bf16 or as said, 8 KV heads of 128, 40 query heads): 16 sequences of 8192 to 65536 positions, q8_0 / q4_0,
// f16 queries, 133 us (5.6 TB/s, 83 % of measured copy bandwidth, bound by memory and the instructions of its 12
// warps alike); one of 131072, q4_0, 44 us (3.4 TB/s: 10 us of launches, sums and merge, then 4 instructions per
// byte at 46 % issue); one of 513 positions 8.7 us; 4 of 4095 to 65535, 2 KV heads of 256, q8_0, fp32, 36 us.
//
// Rounding.  A query row is scaled by a power of two to a largest value of 2^10 .. 2^11, so that
// f16 holds every 16-bit input; fp32 queries keep a second f16 part (hi + lo).  Weights are f16
// for bf16 outputs (2^-11 beside the output's 2^-8) and hi + lo pairs for f16 and fp32 outputs.
// Sums, maxima and S are fp32.
#pragma once
#include <math_constants.h>

#include "kvq_paged.cuh"

namespace kvq {
namespace {

constexpr int kSplitMaxSeqs = 512;  // sequences of one launch (their prefix sums and shapes sit in shared memory)
constexpr int kRows = 8;             // query rows of a unit: the columns of the MMA
constexpr float kDrift = 4.0f;       // the running maximum is moved when a score passes it by this (log2)
// Weights are 2^(s - m + bias).  bias 10 puts the largest weight at 2^10 .. 2^14, so that weights of
// 2^-24 of the largest are still normal f16 numbers and weight x scale < 2^16 for scales below 2;
// a unit that meets a larger scale continues with bias -4 (weight x scale <= 65504 for any scale).
constexpr float kBias = 10.0f, kBiasBig = -4.0f;
constexpr float kSplitLn2 = 0.69314718055994530942f, kSplitLog2e = 1.44269504088896340736f;

template <int KT, int VT, int NS, int DT>
struct SplitCfg {
    using T = PagedTile<KT, VT, NS>;
    static constexpr bool QLO = DT == KVQ_DT_F32;   // queries as hi + lo
    static constexpr bool PLO = DT != KVQ_DT_BF16;  // weights as hi + lo
    // tiles per step (32 keys share one softmax step where the ring allows), warps, ring slots
    static constexpr int TPS = NS == 1 && KT != KVQ_F16 && !QLO ? 2 : 1;
    static constexpr int WARPS = NS == 1 ? (KT == KVQ_F16 ? 8 : (QLO ? 16 : 12)) : (KT == KVQ_F16 ? 4 : (QLO ? 8 : 12));
    static constexpr int STEP = TPS * T::BYTES;
    static constexpr int RING_MAX = 223000;
    static constexpr int SLOTS_RAW = RING_MAX / (WARPS * STEP);
    static constexpr int SLOTS = SLOTS_RAW > 6 ? 6 : SLOTS_RAW;
    static constexpr int RING = WARPS * SLOTS * STEP;
    static constexpr int THREADS = WARPS * 32;
    static constexpr int OFF_PRE = RING;                                    // int [kSplitMaxSeqs + 1]
    static constexpr int OFF_SHAPE = OFF_PRE + (kSplitMaxSeqs + 2) * 4;     // int2 [kSplitMaxSeqs]: tiles, row groups
    static constexpr int OFF_BAR = OFF_SHAPE + kSplitMaxSeqs * 8;           // full barriers [WARPS][SLOTS]
    static constexpr int SMEM = OFF_BAR + WARPS * SLOTS * 8;
    static constexpr int D = T::D;
    static_assert(SLOTS >= 2, "a step in flight while one is read");
    static_assert(SMEM + 2560 <= 232448, "shared memory of one CTA");
    static_assert(WARPS * (kRows * D + 2 * kRows) * 4 <= RING, "merge buffer in the ring");
};

// ---- workspace: [steps before each sequence][span][pieces: m, l, o] ----
struct SplitWork {
    int32_t *pre;  // [n_seqs + 1]; pre[n_seqs + 1] = steps per warp
    float *m, *l;  // [pieces][kRows]
    float *o;      // [pieces][kRows][D]
};
constexpr size_t kSplitHead = (kSplitMaxSeqs + 2 + 62) / 64 * 64 * 4;
__host__ __device__ inline SplitWork split_work(void *ws, int pieces) {
    uint8_t *w = static_cast<uint8_t *>(ws);
    SplitWork r;
    r.pre = reinterpret_cast<int32_t *>(w);
    r.m = reinterpret_cast<float *>(w + kSplitHead);
    r.l = r.m + static_cast<size_t>(pieces) * kRows;
    r.o = r.l + static_cast<size_t>(pieces) * kRows;
    return r;
}
inline size_t split_work_bytes(int pieces, int D) { return kSplitHead + static_cast<size_t>(pieces) * kRows * (D + 2) * 4; }

__device__ __forceinline__ float fast_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {  // an 8x8 matrix of 16-bit values
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}
template <uint32_t SEL>
__device__ __forceinline__ uint32_t byte_perm0(uint32_t a) {
    uint32_t d;
    asm("prmt.b32 %0, %1, 0, %2;\n" : "=r"(d) : "r"(a), "n"(SEL));
    return d;
}
// Codes as f16 operands.  Plain: subnormals, by a permute or a mask alone.  EXACT (fp32 activations): one operation
// more makes normal numbers, and 4-bit codes lose their offset, because sums of products of subnormals keep fewer
// bits: 3e-6 to 1e-5 of the outputs' norm for 4-bit values (2e-7 to 9e-7 this way), nothing beside the rounding of a
// 16-bit output but 4 to 18 times the error of plain fp32.
//
// bytes 0, 2 / 1, 3 of a word of q8_0 codes (sign and magnitude): q 2^-24, or EXACT q 2^-10
template <bool EXACT>
__device__ __forceinline__ uint32_t code8(uint32_t x) {
    if constexpr (EXACT) return h2_as_u32(__hmul2(u32_as_h2(x & 0x807f807fu), __float2half2_rn(16384.0f)));
    return x & 0x807f807fu;
}
template <bool EXACT>
__device__ __forceinline__ uint32_t code8_02(uint32_t w) { return code8<EXACT>(byte_perm0<0xA280u>(w)); }
template <bool EXACT>
__device__ __forceinline__ uint32_t code8_13(uint32_t w) { return code8<EXACT>(byte_perm0<0xB391u>(w)); }
constexpr uint32_t kLowNib = 0x000f000fu, kHighNib = 0x00f000f0u;
// nibbles of q4_0 codes: c 2^-24 and 16 c 2^-24, or EXACT the integers c - 8
template <bool EXACT>
__device__ __forceinline__ uint32_t code4_low(uint32_t x) {
    if constexpr (EXACT) return h2_as_u32(__hsub2(u32_as_h2((x & kLowNib) | 0x64006400u), __float2half2_rn(1032.0f)));
    return x & kLowNib;
}
template <bool EXACT>
__device__ __forceinline__ uint32_t code4_high(uint32_t x) {
    if constexpr (EXACT)
        return h2_as_u32(__hfma2(u32_as_h2((x & kHighNib) | 0x64006400u), __float2half2_rn(0.0625f), __float2half2_rn(-72.0f)));
    return x & kHighNib;
}
constexpr float kUnit24 = 16777216.0f, kUnit20 = 1048576.0f, kUnit10 = 1024.0f;

// d = A B + C with C = (c0, c1) in every row
__device__ __forceinline__ void mma_16816_c(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0, float c1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) { return h2_as_u32(__floats2half2_rn(a, b)); }

// The query rows of a unit as B operands, and what belongs to the rows this lane's accumulator
// columns stand for (rows 2j and 2j + 1, j = lane % 4).
template <int KT, int NS, bool QLO>
struct QueryFrags {
    uint32_t hi[NS * 8][2], lo[QLO ? NS * 8 : 1][2];
    float corr[KT == KVQ_Q4_0 && !QLO ? NS * 4 : 1][2];  // -8 times the sum of q over each block, in accumulator units
    float scale[2];                              // raw scores (accumulator units) to log2 units, >= 0
};

template <int KT, int NS, bool QLO, int DT>
__device__ __forceinline__ void load_queries(QueryFrags<KT, NS, QLO> &f, const typename Act<DT>::type *row, float scale) {
    const int lane = threadIdx.x & 31, j = lane & 3;
    float4 x[NS * 8];
    float top = 0.f;
#pragma unroll
    for (int c = 0; c < NS * 8; ++c) {
        x[c] = row ? Act<DT>::load4(row + 16 * c + 4 * j) : make_float4(0.f, 0.f, 0.f, 0.f);
        top = fmaxf(top, fmaxf(fmaxf(fabsf(x[c].x), fabsf(x[c].y)), fmaxf(fabsf(x[c].z), fabsf(x[c].w))));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // 2^k with the largest value of the row at 2^10 .. 2^11 (k = 0 for rows of zeros, inf or NaN)
    const int ex = static_cast<int>(__float_as_uint(top) >> 23);
    int k = (ex == 0 && top == 0.f) || ex == 255 ? 0 : 10 - (ex - 127);
    k = max(-120, min(120, k));
    // a negative scale goes to the query, so that the largest raw score of a row is its largest score
    const float up = __int_as_float(((127 + k) << 23) | (scale < 0.f ? 0x80000000 : 0)), down = __int_as_float((127 - k) << 23);
    constexpr float unit = KT == KVQ_F16 ? 1.f : KT == KVQ_Q4_0 ? (QLO ? 1.f : kUnit20) : (QLO ? kUnit10 : kUnit24);
    const float rs = fabsf(scale) * kSplitLog2e * down * unit;
#pragma unroll
    for (int c = 0; c < NS * 8; ++c) {
        // low nibbles count 1 and high nibbles 16 of the accumulator's unit
        const float u = (KT == KVQ_Q4_0 && !QLO && (c & 1) == 0) ? up * 16.f : up;
        const float a = x[c].x * u, b = x[c].y * u, e = x[c].z * u, d = x[c].w * u;
        // k = 2j, 2j + 1 of the MMA are values 0, 2 of the four and 2j + 8, 2j + 9 values 1, 3 (the
        // order in which the key codes' bytes come out of a word)
        f.hi[c][0] = pack_half2(a, e);
        f.hi[c][1] = pack_half2(b, d);
        if constexpr (QLO) {
            const float2 h0 = __half22float2(u32_as_h2(f.hi[c][0])), h1 = __half22float2(u32_as_h2(f.hi[c][1]));
            f.lo[c][0] = pack_half2(a - h0.x, e - h0.y);
            f.lo[c][1] = pack_half2(b - h1.x, d - h1.y);
        }
    }
    if constexpr (KT == KVQ_Q4_0 && !QLO) {
        // the score of a key whose codes are all 8, block by block: what the offset adds
        const uint32_t lo8[4] = {0x00080008u, 0x00080008u, 0x00080008u, 0x00080008u};
        const uint32_t hi8[4] = {0x00800080u, 0x00800080u, 0x00800080u, 0x00800080u};
#pragma unroll
        for (int b = 0; b < NS * 4; ++b) {
            float acc[4];
            mma_16816_z(acc, lo8, f.hi[2 * b][0], f.hi[2 * b][1]);
            mma_16816(acc, hi8, f.hi[2 * b + 1][0], f.hi[2 * b + 1][1]);
            f.corr[b][0] = -acc[0];
            f.corr[b][1] = -acc[1];
        }
    }
    // rows 2j, 2j + 1 sit in lanes 8j .. 8j + 7; never 0, so that a masked score stays -inf
    f.scale[0] = fmaxf(__shfl_sync(0xffffffffu, rs, 8 * j), 1e-36f);
    f.scale[1] = fmaxf(__shfl_sync(0xffffffffu, rs, 8 * j + 4), 1e-36f);
}

// Raw scores of one tile: s[0], s[1] = key g with rows 2j, 2j + 1; s[2], s[3] = key g + 8 (g = lane / 4).
template <int KT, int NS, bool QLO>
__device__ __forceinline__ void tile_s(const uint8_t *kc, const uint8_t *ks, const QueryFrags<KT, NS, QLO> &f, float (&s)[4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2;
    if constexpr (KT == KVQ_F16) {
        float acc[2][4];
#pragma unroll
        for (int b = 0; b < NS * 4; ++b) {
            const uint4 w0 = lds128(kc + (2 * b) * 512 + lane * 16), w1 = lds128(kc + (2 * b + 1) * 512 + lane * 16);
            const uint32_t a0[4] = {w0.x, w1.x, w0.y, w1.y}, a1[4] = {w0.z, w1.z, w0.w, w1.w};
            if (b == 0 || QLO) {  // QLO: short chains of products, summed in fp32
                mma_16816_z(acc[0], a0, f.hi[2 * b][0], f.hi[2 * b][1]);
                mma_16816_z(acc[1], a1, f.hi[2 * b + 1][0], f.hi[2 * b + 1][1]);
            } else {
                mma_16816(acc[0], a0, f.hi[2 * b][0], f.hi[2 * b][1]);
                mma_16816(acc[1], a1, f.hi[2 * b + 1][0], f.hi[2 * b + 1][1]);
            }
            if constexpr (QLO) {
                mma_16816(acc[0], a0, f.lo[2 * b][0], f.lo[2 * b][1]);
                mma_16816(acc[1], a1, f.lo[2 * b + 1][0], f.lo[2 * b + 1][1]);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i] = (b == 0 ? 0.f : s[i]) + (acc[0][i] + acc[1][i]);
            }
        }
        if constexpr (!QLO)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] = acc[0][i] + acc[1][i];
    } else {
        s[0] = s[1] = s[2] = s[3] = 0.f;
        // key g is member g % 2 of the pairs of lane group g / 2, key g + 8 member 2 + g % 2
        const uint32_t pick = (g & 1) ? 0x4432u : 0x4410u;
#pragma unroll
        for (int sl = 0; sl < NS; ++sl) {
            const uint8_t *kcs = kc + sl * code_tile_bytes(KT);
            const uint4 s0 = lds128(ks + sl * kScaleTile + (g >> 1) * 32), s1 = lds128(ks + sl * kScaleTile + (g >> 1) * 32 + 16);
            const uint32_t sw[4][2] = {{s0.x, s0.y}, {s0.z, s0.w}, {s1.x, s1.y}, {s1.z, s1.w}};
            uint4 w4 = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int c = sl * 8 + 2 * b;
                uint32_t a0[4], a1[4];
                float acc[4];
                if constexpr (KT == KVQ_Q8_0) {
                    const uint4 w = lds128(kcs + b * 512 + lane * 16);
                    a0[0] = code8_02<QLO>(w.x), a0[1] = code8_02<QLO>(w.z), a0[2] = code8_13<QLO>(w.x), a0[3] = code8_13<QLO>(w.z);
                    a1[0] = code8_02<QLO>(w.y), a1[1] = code8_02<QLO>(w.w), a1[2] = code8_13<QLO>(w.y), a1[3] = code8_13<QLO>(w.w);
                    mma_16816_z(acc, a0, f.hi[c][0], f.hi[c][1]);
                } else {
                    if ((b & 1) == 0) w4 = lds128(kcs + (b >> 1) * 512 + lane * 16);
                    const uint32_t u = (b & 1) ? w4.z : w4.x, w = (b & 1) ? w4.w : w4.y, u8 = u >> 8, w8 = w >> 8;
                    a0[0] = code4_low<QLO>(u), a0[1] = code4_low<QLO>(w), a0[2] = code4_low<QLO>(u8), a0[3] = code4_low<QLO>(w8);
                    a1[0] = code4_high<QLO>(u), a1[1] = code4_high<QLO>(w), a1[2] = code4_high<QLO>(u8), a1[3] = code4_high<QLO>(w8);
                    if constexpr (QLO)
                        mma_16816_z(acc, a0, f.hi[c][0], f.hi[c][1]);
                    else
                        mma_16816_c(acc, a0, f.hi[c][0], f.hi[c][1], f.corr[sl * 4 + b][0], f.corr[sl * 4 + b][1]);
                }
                mma_16816(acc, a1, f.hi[c + 1][0], f.hi[c + 1][1]);
                if constexpr (QLO) {
                    mma_16816(acc, a0, f.lo[c][0], f.lo[c][1]);
                    mma_16816(acc, a1, f.lo[c + 1][0], f.lo[c + 1][1]);
                }
                uint32_t h0, h1;
                asm("prmt.b32 %0, %1, 0, %2;\n" : "=r"(h0) : "r"(sw[b][0]), "r"(pick));
                asm("prmt.b32 %0, %1, 0, %2;\n" : "=r"(h1) : "r"(sw[b][1]), "r"(pick));
                const float d0 = __low2float(u32_as_h2(h0)), d1 = __low2float(u32_as_h2(h1));
                s[0] = fmaf(d0, acc[0], s[0]);
                s[1] = fmaf(d0, acc[1], s[1]);
                s[2] = fmaf(d1, acc[2], s[2]);
                s[3] = fmaf(d1, acc[3], s[3]);
            }
        }
    }
}

// Whether rows [0, valid) of a tile have a value scale of 2 or more (bit 14 of a half; inf and NaN included):
// each lane looks at one word, keys 2j, 2j + 1 (+ 8 in odd words) of lane group j = lane / 8.
template <int NS>
__device__ __forceinline__ bool big_scales(const uint8_t *vs, int valid) {
    const int lane = threadIdx.x & 31;
    uint32_t e = 0;
#pragma unroll
    for (int sl = 0; sl < NS; ++sl) e |= *reinterpret_cast<const uint32_t *>(vs + sl * kScaleTile + lane * 4);
    e &= 0x40004000u;
    if (valid < kTileRows) {
        keep_branch();
        const int k = 2 * (lane >> 3) + 8 * (lane & 1);
        e &= k >= valid ? 0u : (k + 1 >= valid ? 0x0000ffffu : 0xffffffffu);
    }
    return e != 0;
}

// O^T += V^T P^T for one tile.  ph / pl: weights of keys (2j, 2j + 1) and (2j + 8, 2j + 9) of row g;
// mab / mcd: masks of those keys (rows past the sequence's end may hold any bits).  o[2b], o[2b + 1]:
// values 32b + 2g, + 1 and 32b + 16 + 2g, + 1 of rows 2j, 2j + 1.  For q4_0 without EXACT, corr row b
// collects the sum of weight x scale of block b, by which 8 has been added to every code.
template <int VT, int NS, bool PLO, bool EXACT, bool MASK>
__device__ __forceinline__ void tile_o(const uint8_t *vc, const uint8_t *vs, const uint32_t (&ph)[2], const uint32_t (&pl)[2],
                                       uint32_t mab, uint32_t mcd, float (&o)[NS * 8][4], float (&corr)[4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
    if constexpr (VT == KVQ_F16) {
#pragma unroll
        for (int b = 0; b < NS * 4; ++b) {
            uint4 w0 = lds128(vc + (2 * b) * 512 + lane * 16), w1 = lds128(vc + (2 * b + 1) * 512 + lane * 16);
            if constexpr (MASK) {
                w0.x &= mab, w0.z &= mab, w0.y &= mcd, w0.w &= mcd;
                w1.x &= mab, w1.z &= mab, w1.y &= mcd, w1.w &= mcd;
            }
            const uint32_t a0[4] = {w0.x, w0.z, w0.y, w0.w}, a1[4] = {w1.x, w1.z, w1.y, w1.w};
            mma_16816(o[2 * b], a0, ph[0], ph[1]);
            mma_16816(o[2 * b + 1], a1, ph[0], ph[1]);
            if constexpr (PLO) {
                mma_16816(o[2 * b], a0, pl[0], pl[1]);
                mma_16816(o[2 * b + 1], a1, pl[0], pl[1]);
            }
        }
    } else {
#pragma unroll
        for (int sl = 0; sl < NS; ++sl) {
            const uint8_t *vcs = vc + sl * code_tile_bytes(VT);
            const uint4 s0 = lds128(vs + sl * kScaleTile + j * 32), s1 = lds128(vs + sl * kScaleTile + j * 32 + 16);
            const uint32_t sw[4][2] = {{s0.x, s0.y}, {s0.z, s0.w}, {s1.x, s1.y}, {s1.z, s1.w}};
            uint4 w4 = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int t = sl * 8 + 2 * b;
                uint32_t dab = sw[b][0], dcd = sw[b][1];
                if constexpr (MASK) dab &= mab, dcd &= mcd;
                // weight x scale, rounded once to f16; with PLO also the rest: the product's error
                // (exact by fma) plus lo x scale
                const __half2 xab = __hmul2(u32_as_h2(ph[0]), u32_as_h2(dab)), xcd = __hmul2(u32_as_h2(ph[1]), u32_as_h2(dcd));
                const uint32_t b0 = h2_as_u32(xab), b1 = h2_as_u32(xcd);
                uint32_t l0 = 0, l1 = 0;
                if constexpr (PLO) {
                    l0 = h2_as_u32(__hfma2(u32_as_h2(pl[0]), u32_as_h2(dab), __hfma2(u32_as_h2(ph[0]), u32_as_h2(dab), __hneg2(xab))));
                    l1 = h2_as_u32(__hfma2(u32_as_h2(pl[1]), u32_as_h2(dcd), __hfma2(u32_as_h2(ph[1]), u32_as_h2(dcd), __hneg2(xcd))));
                }
                uint32_t a0[4], a1[4];
                if constexpr (VT == KVQ_Q8_0) {
                    const uint4 w = lds128(vcs + b * 512 + lane * 16);
                    a0[0] = code8_02<EXACT>(w.x), a0[1] = code8_02<EXACT>(w.y), a0[2] = code8_13<EXACT>(w.x), a0[3] = code8_13<EXACT>(w.y);
                    a1[0] = code8_02<EXACT>(w.z), a1[1] = code8_02<EXACT>(w.w), a1[2] = code8_13<EXACT>(w.z), a1[3] = code8_13<EXACT>(w.w);
                } else {
                    if ((b & 1) == 0) w4 = lds128(vcs + (b >> 1) * 512 + lane * 16);
                    const uint32_t u = (b & 1) ? w4.z : w4.x, w = (b & 1) ? w4.w : w4.y, u8 = u >> 8, w8 = w >> 8;
                    a0[0] = code4_low<EXACT>(u), a0[1] = code4_low<EXACT>(w), a0[2] = code4_low<EXACT>(u8), a0[3] = code4_low<EXACT>(w8);
                    a1[0] = code4_high<EXACT>(u), a1[1] = code4_high<EXACT>(w), a1[2] = code4_high<EXACT>(u8), a1[3] = code4_high<EXACT>(w8);
                    if constexpr (!EXACT) {
                        const uint32_t one = g == sl * 4 + b ? 0x3c003c00u : 0u;  // row b of the collecting operand
                        const uint32_t ac[4] = {one, 0u, one, 0u};
                        mma_16816(corr, ac, b0, b1);
                        if constexpr (PLO) mma_16816(corr, ac, l0, l1);
                    }
                }
                mma_16816(o[t], a0, b0, b1);
                mma_16816(o[t + 1], a1, b0, b1);
                if constexpr (PLO) {
                    mma_16816(o[t], a0, l0, l1);
                    mma_16816(o[t + 1], a1, l0, l1);
                }
            }
        }
    }
}

// ---- the walk over steps ----
struct Walk {
    int b, h, qg;  // sequence, KV head, row group: the unit
    int t;         // step of the unit
    int tiles, steps, groups;  // of the sequence
};

// sequence b, without tokens if it belongs to the chunk kernel
__device__ __forceinline__ PagedSeq split_seq(const PagedAttnParams &p, int b) {
    PagedSeq s = paged_seq(p.v, b);
    if (s.n >= p.from_q) s.n = 0;
    return s;
}
template <int TPS>
__device__ __forceinline__ void walk_seq(Walk &w, const int2 *shape, int b) {
    const int2 s = shape[b];
    w.b = b;
    w.h = w.qg = w.t = 0;
    w.tiles = s.x;
    w.steps = (s.x + TPS - 1) / TPS;
    w.groups = s.y;
}
// position at step x of all steps; pre[b] <= x < pre[n_seqs]
template <int TPS>
__device__ __forceinline__ Walk walk_to(const int *pre, const int2 *shape, int n_seqs, int x) {
    int lo = 0, hi = n_seqs;  // last b with pre[b] <= x (it has steps, for pre[b + 1] > x)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    Walk w;
    walk_seq<TPS>(w, shape, lo);
    const unsigned r = x - pre[lo], unit = r / static_cast<unsigned>(w.steps);
    w.t = r - unit * w.steps;
    w.h = unit / static_cast<unsigned>(w.groups);
    w.qg = unit - w.h * w.groups;
    return w;
}
// the first step of the next unit (a step follows: the caller counts)
template <int TPS>
__device__ __forceinline__ void walk_next_unit(Walk &w, const int *pre, const int2 *shape, int Hkv) {
    w.t = 0;
    if (++w.qg < w.groups) return;
    w.qg = 0;
    if (++w.h < Hkv) return;
    int b = w.b + 1;
    while (pre[b + 1] == pre[b]) ++b;
    walk_seq<TPS>(w, shape, b);
}

// Row r of a unit (row group qg of KV head h of sequence b): token i of the sequence, query head h G + g.
// The quotient by G is exact in fp32: rr < 2^20 and the half keeps it off whole numbers.
struct UnitRows {
    int first, Hq, h0, G, r0, rows;
    float inv_g;
    __device__ __forceinline__ int token(int r) const { return static_cast<int>((r0 + r + 0.5f) * inv_g); }
    __device__ __forceinline__ int head(int r, int i) const { return h0 + r0 + r - i * G; }
    __device__ __forceinline__ long long out_row(int r) const {
        if (r >= rows) return -1;
        const int i = token(r);
        return static_cast<long long>(first + i) * Hq + head(r, i);
    }
};
__device__ __forceinline__ UnitRows unit_rows(const PagedAttnParams &p, const PagedSeq &s, int h, int qg) {
    return UnitRows{s.first, p.Hq, h * p.G, p.G, qg * kRows, min(kRows, s.n * p.G - qg * kRows), 1.0f / p.G};
}

template <int KT, int VT, int NS, int DT>
__global__ void __launch_bounds__(SplitCfg<KT, VT, NS, DT>::THREADS, 1)
    paged_split_kernel(const PagedAttnParams p, const SplitWork work, const int unit_groups) {
    using C = SplitCfg<KT, VT, NS, DT>;
    using T = typename C::T;
    using X = typename Act<DT>::type;
    constexpr int TPS = C::TPS, D = C::D;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_scan[32];
    __shared__ int s_unit[C::WARPS], s_b[C::WARPS];  // the unit a warp's accumulators hold at the end (-1: none)
    __shared__ float s_ml[C::WARPS][2 * kRows];
    // where a warp's issuing and reading sides stand: kept out of the registers of the loop, which needs them
    // once per page and once per unit
    __shared__ Walk s_walk[C::WARPS][2];
    int *pre = reinterpret_cast<int *>(smem + C::OFF_PRE);
    int2 *shape = reinterpret_cast<int2 *>(smem + C::OFF_SHAPE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR) + warp * C::SLOTS;
    if (lane < C::SLOTS) mbar_init(full + lane, 1);
    fence_mbar_init();
    // everything below reads what earlier kernels of the stream wrote
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

    const PagedView &v = p.v;
    int x0, x1, span = 0, total = 0;  // this warp's steps
    Walk w0;                          // where they start
    if (unit_groups > 0) {
        // ---- one unit per CTA, its steps shared by the warps ----
        const int r = blockIdx.x / unit_groups;
        w0.qg = blockIdx.x - r * unit_groups;
        w0.b = r / v.Hkv;
        w0.h = r - w0.b * v.Hkv;
        const PagedSeq q = split_seq(p, w0.b);
        if (threadIdx.x == 0 && w0.h == 0 && w0.qg == 0 && !paged_seq(v, w0.b).ok) paged_error(v);
        w0.tiles = (q.len + kTileRows - 1) / kTileRows;
        w0.steps = (w0.tiles + TPS - 1) / TPS;
        w0.groups = (q.n * p.G + kRows - 1) / kRows;
        if (w0.qg >= w0.groups) return;
        if (w0.steps == 0) {  // nothing to attend to
            const UnitRows rows = unit_rows(p, q, w0.h, w0.qg);
            for (int i = threadIdx.x; i < rows.rows * (D / 4); i += C::THREADS) {
                const long long row = rows.out_row(i / (D / 4));
                Act<DT>::store4(static_cast<X *>(p.out) + row * D + i % (D / 4) * 4, make_float4(0.f, 0.f, 0.f, 0.f));
                if (i % (D / 4) == 0 && p.lse) p.lse[row] = -CUDART_INF_F;
            }
            return;
        }
        const int share = (w0.steps + C::WARPS - 1) / C::WARPS;
        x0 = min(w0.steps, warp * share);
        x1 = min(w0.steps, x0 + share);
        w0.t = x0;
    } else {
        // ---- steps before each sequence: every CTA adds them up for itself ----
        {
            const int per = (v.n_seqs + C::THREADS - 1) / C::THREADS;
            const int b0 = min(v.n_seqs, static_cast<int>(threadIdx.x) * per), b1 = min(v.n_seqs, b0 + per);
            int sum = 0;
            for (int b = b0; b < b1; ++b) {
                PagedSeq q = paged_seq(v, b);
                if (blockIdx.x == 0 && !q.ok) paged_error(v);
                if (q.n >= p.from_q) q.n = 0;
                const int tiles = (q.len + kTileRows - 1) / kTileRows, groups = (q.n * p.G + kRows - 1) / kRows;
                shape[b] = make_int2(tiles, groups);
                pre[b] = sum;
                sum += (tiles + TPS - 1) / TPS * groups * v.Hkv;
            }
            int inc = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            if (lane == 31) s_scan[warp] = inc;
            __syncthreads();
            int before = inc - sum;
            for (int w = 0; w < warp; ++w) before += s_scan[w];
            for (int b = b0; b < b1; ++b) pre[b] += before;
            if (threadIdx.x == C::THREADS - 1) pre[v.n_seqs] = before + sum;
            __syncthreads();
        }
        total = pre[v.n_seqs];
        span = (total + static_cast<int>(gridDim.x) * C::WARPS - 1) / (static_cast<int>(gridDim.x) * C::WARPS);
        if (blockIdx.x == 0) {  // for the merge
            for (int b = threadIdx.x; b <= v.n_seqs; b += C::THREADS) work.pre[b] = pre[b];
            if (threadIdx.x == 0) work.pre[v.n_seqs + 1] = span;
        }
        const long long x0l = static_cast<long long>(blockIdx.x * C::WARPS + warp) * span;
        x0 = x0l < total ? static_cast<int>(x0l) : total;
        x1 = min(total, x0 + span);
        if (x0 < x1) w0 = walk_to<TPS>(pre, shape, v.n_seqs, x0);
    }
    float o[NS * 8][4], corr[4], m_run[2], l[2], bias = kBias;
    if (lane == 0) s_unit[warp] = -1;
    // output rows of a unit
    auto rows_of = [&](const Walk &w) { return unit_rows(p, split_seq(p, w.b), w.h, w.qg); };

    // a finished segment in its registers: l summed over the keys' lanes, o in real units
    auto finish = [&]() {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 4);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 8);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 16);
        }
        if constexpr (VT == KVQ_Q8_0 || (VT == KVQ_Q4_0 && !C::QLO)) {
#pragma unroll
            for (int t = 0; t < NS * 8; ++t) {
                const float unit = (VT == KVQ_Q4_0 && (t & 1)) ? kUnit20 : (C::QLO ? kUnit10 : kUnit24);
                float c0 = 0.f, c1 = 0.f;
                if constexpr (VT == KVQ_Q4_0) {  // row t / 2 of corr: lanes 4 (t / 2) + j
                    c0 = 8.f * __shfl_sync(0xffffffffu, corr[0], (t >> 1) * 4 + j);
                    c1 = 8.f * __shfl_sync(0xffffffffu, corr[1], (t >> 1) * 4 + j);
                }
                o[t][0] = o[t][0] * unit - c0;
                o[t][2] = o[t][2] * unit - c0;
                o[t][1] = o[t][1] * unit - c1;
                o[t][3] = o[t][3] * unit - c1;
            }
        }
    };
    // the unit's output rows, from a segment that is all of it
    auto write_out = [&](const UnitRows &rows) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const long long row = rows.out_row(2 * j + i);
            if (row < 0) continue;
            const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
            X *dst = static_cast<X *>(p.out) + row * D + 2 * g;
#pragma unroll
            for (int t = 0; t < NS * 8; ++t) Act<DT>::store2(dst + 16 * t, o[t][i] * inv, o[t][2 + i] * inv);
            if (g == 0 && p.lse)
                p.lse[row] = l[i] > 0.f ? (m_run[i] - bias + __log2f(l[i])) * kSplitLn2 : -CUDART_INF_F;
        }
    };
    auto write_piece = [&](int piece) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const size_t r = static_cast<size_t>(piece) * kRows + 2 * j + i;
            float *dst = work.o + r * D + 2 * g;
#pragma unroll
            for (int t = 0; t < NS * 8; ++t) *reinterpret_cast<float2 *>(dst + 16 * t) = make_float2(o[t][i], o[t][2 + i]);
            if (g == 0) {
                work.m[r] = m_run[i] == -CUDART_INF_F ? -CUDART_INF_F : m_run[i] - bias;
                work.l[r] = l[i];
            }
        }
    };

    Walk *const w_iss = &s_walk[warp][0], *const w_cur = &s_walk[warp][1];
    if (x0 < x1) {
        uint8_t *const ring = smem + warp * (C::SLOTS * C::STEP);
        constexpr unsigned kAll = (1u << TPS) - 1u;
        if (lane == 0) *w_iss = *w_cur = w0;
        __syncwarp();
        // ---- the issuing side runs SLOTS steps ahead.  Steps whose tiles follow one another in a page form a
        // run, found once: within it a step is one copy from `src`.  A lane holds one entry of the unit's
        // block table (entries tab0 .. tab0 + 31), the next 32 are on their way. ----
        int to_issue = x1 - x0, run = 0;
        const uint8_t *src = nullptr;
        unsigned held = 0;  // bit slot * TPS + i: tile i of the slot's step was copied
        int tab = -1, tab_next = -1, tab0 = 0;
        auto load_tab = [&](const Walk &w, int e0) {
            return (e0 + lane) * v.page_tiles < w.tiles ? __ldg(v.table + static_cast<size_t>(w.b) * v.stride + e0 + lane) : -1;
        };
        auto enter_unit = [&](const Walk &w) {
            tab0 = static_cast<unsigned>(w.t * TPS) / static_cast<unsigned>(v.page_tiles);
            tab = load_tab(w, tab0);
            tab_next = load_tab(w, tab0 + 32);
        };
        enter_unit(*w_iss);
        auto copy = [&](uint8_t *dst, const uint8_t *from, int bytes, uint64_t *bar) {
            if (lane == 0) bulk_g2s(dst, from, bytes, bar);
        };
        auto issue = [&](int slot) {  // the next step into a slot
            uint8_t *dst = ring + slot * C::STEP;
            if (run == 0) {
                Walk w = *w_iss;
                if (w.t == w.steps) {
                    walk_next_unit<TPS>(w, pre, shape, v.Hkv);
                    enter_unit(w);
                }
                const int t0 = w.t * TPS;
                auto entry = [&](int e) {  // e grows by at most one per call
                    if (e - tab0 >= 32) {
                        tab = tab_next;
                        tab0 += 32;
                        tab_next = load_tab(w, tab0 + 32);
                    }
                    return __shfl_sync(0xffffffffu, tab, e - tab0);
                };
                auto record = [&](int page, int q) {
                    return v.pool + ((static_cast<size_t>(page) * v.Hkv + w.h) * v.page_tiles + q) * T::BYTES;
                };
                const int e = static_cast<unsigned>(t0) / static_cast<unsigned>(v.page_tiles), q = t0 - e * v.page_tiles;
                const int page = entry(e);
                const bool in = page >= 0 && page < v.n_pages;
                const int whole = min(v.page_tiles - q, w.tiles - t0) / TPS;  // steps of this page from here
                int done = 1;
                if (in && whole > 0) {
                    src = record(page, q);
                    run = done = min(whole, to_issue);
                } else {
                    // a step that crosses a page, ends the sequence or has no page: tile by tile
                    bool ok[TPS];
                    const uint8_t *from[TPS];
                    int n = 0;
#pragma unroll
                    for (int i = 0; i < TPS; ++i) {
                        int ei = e, qi = q + i;
                        if (qi >= v.page_tiles) qi -= v.page_tiles, ++ei;
                        const bool live = t0 + i < w.tiles;
                        const int pi = i == 0 ? page : (live ? entry(ei) : -1);
                        ok[i] = live && pi >= 0 && pi < v.n_pages;
                        from[i] = ok[i] ? record(pi, qi) : nullptr;
                        if (live && !ok[i] && lane == 0) paged_error(v);
                        n += ok[i] ? 1 : 0;
                        const unsigned bit = 1u << (slot * TPS + i);
                        held = ok[i] ? held | bit : held & ~bit;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(full + slot, static_cast<uint32_t>(n * T::BYTES));
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < TPS; ++i)
                        if (ok[i]) copy(dst + i * T::BYTES, from[i], T::BYTES, full + slot);
                }
                __syncwarp();
                if (lane == 0) {
                    w.t += done;
                    *w_iss = w;
                }
                __syncwarp();
            }
            if (run > 0) {
                if (lane == 0) mbar_arrive_expect_tx(full + slot, C::STEP);
                copy(dst, src, C::STEP, full + slot);
                src += C::STEP;
                --run;
                held |= kAll << (slot * TPS);
            }
            --to_issue;
        };
#pragma unroll 1
        for (int i = 0; i < C::SLOTS; ++i)
            if (to_issue > 0) issue(i);

        // ---- the reading side ----
        QueryFrags<KT, NS, C::QLO> f;
        int lim[2] = {0, 0}, lim_min = 0, len = 0, key0 = 0, unit_left = 0, left = x1 - x0;
        bool first = true;  // the segment in hand is the span's first
        int slot = 0;
        unsigned phase = 0;
        while (true) {
            if (unit_left == 0) {  // a unit: its queries, empty accumulators
                const Walk w = *w_cur;
                const PagedSeq s = split_seq(p, w.b);
                const UnitRows rows = unit_rows(p, s, w.h, w.qg);
                const int i0 = rows.token(g);
                const X *qr = nullptr;
                if (g < rows.rows)
                    qr = static_cast<const X *>(p.q) + (s.first + i0) * p.q_stride + static_cast<size_t>(rows.head(g, i0)) * D;
                len = s.len;
                lim_min = s.len - s.n;  // the first token's position
                lim[0] = lim_min + rows.token(2 * j);
                lim[1] = lim_min + rows.token(2 * j + 1);
                key0 = w.t * TPS * kTileRows;
                unit_left = w.steps - w.t;
                load_queries<KT, NS, C::QLO, DT>(f, qr, p.scale);
#pragma unroll
                for (int t = 0; t < NS * 8; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
                corr[0] = corr[1] = corr[2] = corr[3] = 0.f;
                m_run[0] = m_run[1] = -CUDART_INF_F;
                l[0] = l[1] = 0.f;
                bias = kBias;
            }
            const uint8_t *st = ring + slot * C::STEP;
            if (__any_sync(0xffffffffu, !paged_wait(full + slot, phase))) {
                // gave up: the outputs of the call are undefined and the error word says so.  Copies in
                // flight land before the memory is used again.
                if (lane == 0) atomicOr(v.err, KVQ_DEVERR_TIMEOUT);
                for (int i = left - to_issue; i > 0; --i) {
                    (void)paged_wait(full + slot, phase);
                    if (++slot == C::SLOTS) slot = 0, phase ^= 1u;
                }
                break;
            }
            const unsigned got = (held >> (slot * TPS)) & kAll;
            float s[TPS][4];
#pragma unroll
            for (int i = 0; i < TPS; ++i)
                tile_s<KT, NS, C::QLO>(st + i * T::BYTES, st + i * T::BYTES + T::OFF_KS, f, s[i]);
            // keys behind a row's own position, past the end or in no page
            const bool cut = key0 + TPS * kTileRows - 1 > lim_min || got != kAll;
            int valid[TPS];  // rows of each tile in use
#pragma unroll
            for (int i = 0; i < TPS; ++i) valid[i] = kTileRows;
            if (cut) {
                keep_branch();
#pragma unroll
                for (int i = 0; i < TPS; ++i) {
                    valid[i] = ((got >> i) & 1u) ? len - key0 - i * kTileRows : 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = i * kTileRows + g + (e >> 1) * 8;
                        if (key0 + key > lim[e & 1] || key - i * kTileRows >= valid[i]) s[i][e] = -CUDART_INF_F;
                    }
                }
            }
            // ---- running maximum: moved only when a score passes it by kDrift ----
            float mx[2] = {s[0][0], s[0][1]};
#pragma unroll
            for (int i = 0; i < TPS; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) mx[e] = fmaxf(mx[e], fmaxf(s[i][e], s[i][2 + e]));
            mx[0] *= f.scale[0];
            mx[1] *= f.scale[1];
            bool big = false;
            if constexpr (VT != KVQ_F16) {
#pragma unroll
                for (int i = 0; i < TPS; ++i) big = big_scales<NS>(st + i * T::BYTES + T::OFF_VS, valid[i]) || big;
                big = big && bias == kBias;
            }
            if (__any_sync(0xffffffffu, mx[0] > m_run[0] + kDrift || mx[1] > m_run[1] + kDrift || big)) {
                float shift = 0.f;
                if (VT != KVQ_F16 && __any_sync(0xffffffffu, big)) {
                    shift = kBiasBig - kBias;
                    bias = kBiasBig;
                }
                float a[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 4));
                    mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 8));
                    mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 16));
                    const float mn = fmaxf(m_run[e], mx[e]);
                    a[e] = m_run[e] == -CUDART_INF_F ? 0.f : fast_ex2(m_run[e] - mn + shift);
                    m_run[e] = mn;
                    l[e] *= a[e];
                }
#pragma unroll
                for (int t = 0; t < NS * 8; ++t) {
                    o[t][0] *= a[0];
                    o[t][2] *= a[0];
                    o[t][1] *= a[1];
                    o[t][3] *= a[1];
                }
                if constexpr (VT == KVQ_Q4_0) {
                    corr[0] *= a[0];
                    corr[1] *= a[1];
                }
            }
            const float ms[2] = {m_run[0] == -CUDART_INF_F ? 0.f : bias - m_run[0], m_run[1] == -CUDART_INF_F ? 0.f : bias - m_run[1]};
#pragma unroll
            for (int i = 0; i < TPS; ++i) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = fast_ex2(fmaf(s[i][e], f.scale[e & 1], ms[e & 1]));
                l[0] += w[0] + w[2];
                l[1] += w[1] + w[3];
                uint32_t ph[2] = {pack_half2(w[0], w[1]), pack_half2(w[2], w[3])}, pl[2] = {0u, 0u};
                if constexpr (C::PLO) {
                    const float2 h0 = __half22float2(u32_as_h2(ph[0])), h1 = __half22float2(u32_as_h2(ph[1]));
                    pl[0] = transpose8x8(pack_half2(w[0] - h0.x, w[1] - h0.y));
                    pl[1] = transpose8x8(pack_half2(w[2] - h1.x, w[3] - h1.y));
                }
                ph[0] = transpose8x8(ph[0]);
                ph[1] = transpose8x8(ph[1]);
                const uint8_t *tv = st + i * T::BYTES + T::OFF_V, *tvs = st + i * T::BYTES + T::OFF_VS;
                if (cut) {
                    keep_branch();
                    auto mask = [&](int k) { return k + 1 < valid[i] ? 0xffffffffu : (k < valid[i] ? 0x0000ffffu : 0u); };
                    tile_o<VT, NS, C::PLO, C::QLO, true>(tv, tvs, ph, pl, mask(2 * j), mask(2 * j + 8), o, corr);
                } else {
                    tile_o<VT, NS, C::PLO, C::QLO, false>(tv, tvs, ph, pl, 0u, 0u, o, corr);
                }
            }
            __syncwarp();  // the slot has been read
            if (to_issue > 0) issue(slot);
            if (++slot == C::SLOTS) {
                slot = 0;
                phase ^= 1u;
            }
            key0 += TPS * kTileRows;
            --unit_left;
            if (--left == 0) break;
            if (unit_left == 0) {  // the unit ends inside this warp's span
                Walk w = *w_cur;
                finish();
                if (!first || w.t == 0)
                    write_out(rows_of(w));
                else
                    write_piece((blockIdx.x * C::WARPS + warp) * 2 + 1);
                walk_next_unit<TPS>(w, pre, shape, v.Hkv);
                __syncwarp();
                if (lane == 0) *w_cur = w;
                __syncwarp();
                first = false;
            }
        }
        finish();
        if (lane == 0) {
            s_unit[warp] = w_cur->h * w_cur->groups + w_cur->qg;
            s_b[warp] = w_cur->b;
        }
    }
    // ---- the warps of this CTA whose last segments are of one unit merge ----
    __syncthreads();
    const int unit = s_unit[warp], ub = unit >= 0 ? s_b[warp] : -1;
    int first = warp, last = warp;
    if (unit >= 0) {  // the run of warps around this one with the same unit
        const bool eq = lane < C::WARPS && s_unit[lane] == unit && s_b[lane] == ub;
        const unsigned other = ~__ballot_sync(0xffffffffu, eq);
        first = 32 - __clz(other & ((1u << warp) - 1u));
        last = __ffs(other & ~((2u << warp) - 1u)) - 2;
    }
    // the group holds steps [its first warp's segment start, the end of the unit or of its spans)
    const int steps = unit >= 0 ? w_cur->steps : 0, u0 = unit >= 0 && unit_groups == 0 ? pre[ub] + unit * steps : 0;
    UnitRows rows{};
    if (unit >= 0) rows = rows_of(*w_cur);
    const int g0 = max(u0, (blockIdx.x * C::WARPS + first) * span), g1 = min(total, (static_cast<int>(blockIdx.x) * C::WARPS + last + 1) * span);
    const bool whole = unit >= 0 && (unit_groups > 0 || (g0 == u0 && g1 >= u0 + steps));
    if (unit >= 0 && first == last) {
        if (whole)
            write_out(rows);
        else
            write_piece((blockIdx.x * C::WARPS + warp) * 2);
    }
    float *buf = reinterpret_cast<float *>(smem);  // [WARPS][kRows][D]
    if (unit >= 0 && first != last) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float *dst = buf + (warp * kRows + 2 * j + i) * D + 2 * g;
#pragma unroll
            for (int t = 0; t < NS * 8; ++t) *reinterpret_cast<float2 *>(dst + 16 * t) = make_float2(o[t][i], o[t][2 + i]);
            if (g == 0) {
                s_ml[warp][2 * j + i] = m_run[i] == -CUDART_INF_F ? -CUDART_INF_F : m_run[i] - bias;
                s_ml[warp][kRows + 2 * j + i] = l[i];
            }
        }
    }
    __syncthreads();
    if (unit < 0 || first == last) return;
    // the group's warps share its rows and columns
    const int gt = (warp - first) * 32 + lane, gn = (last - first + 1) * 32;
    for (int item = gt; item < rows.rows * (D / 4); item += gn) {
        const int r = item / (D / 4), c = item % (D / 4);
        float M = -CUDART_INF_F;
#pragma unroll 4
        for (int w = first; w <= last; ++w) M = fmaxf(M, s_ml[w][r]);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        float L = 0.f;
        if (M != -CUDART_INF_F) {
#pragma unroll 4
            for (int w = first; w <= last; ++w) {
                const float k = fast_ex2(s_ml[w][r] - M);
                const float4 y = *reinterpret_cast<const float4 *>(buf + (w * kRows + r) * D + 4 * c);
                a = make_float4(fmaf(k, y.x, a.x), fmaf(k, y.y, a.y), fmaf(k, y.z, a.z), fmaf(k, y.w, a.w));
                L = fmaf(k, s_ml[w][kRows + r], L);
            }
        }
        if (whole) {
            const long long row = rows.out_row(r);
            if (row < 0) continue;
            const float inv = L > 0.f ? 1.f / L : 0.f;
            Act<DT>::store4(static_cast<X *>(p.out) + row * D + 4 * c, make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv));
            if (c == 0 && p.lse) p.lse[row] = L > 0.f ? (M + __log2f(L)) * kSplitLn2 : -CUDART_INF_F;
        } else {
            const size_t pr = static_cast<size_t>((blockIdx.x * C::WARPS + first) * 2) * kRows + r;
            *reinterpret_cast<float4 *>(work.o + pr * D + 4 * c) = a;
            if (c == 0) {
                work.m[pr] = M;
                work.l[pr] = L;
            }
        }
    }
}

// Merge of the pieces, one CTA per (unit, row): column threads x kMergeWays shares of the pieces.
// The pieces of a unit follow from its steps and the span: one per CTA that ends with it, and one
// from the warp that finished it and went on.  Units that nothing attends to get zeros here.
constexpr int kMergeWays = 4;
template <int NS, int DT>
__global__ void __launch_bounds__(NS * 32 * kMergeWays)
    paged_merge_kernel(const PagedAttnParams p, const SplitWork work, const int warps, const int tps, const int max_groups) {
    using X = typename Act<DT>::type;
    constexpr int D = NS * kSlice, DQ = D / 4;
    __shared__ float4 s_a[kMergeWays][DQ];
    __shared__ float s_m[kMergeWays], s_l[kMergeWays];
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int row = blockIdx.x % kRows, rest = blockIdx.x / kRows;
    const int qg = rest % max_groups, h = (rest / max_groups) % p.v.Hkv, b = rest / max_groups / p.v.Hkv;
    const PagedSeq s = split_seq(p, b);
    const int groups = (s.n * p.G + kRows - 1) / kRows;
    if (qg >= groups) return;
    const UnitRows rows = unit_rows(p, s, h, qg);
    const long long orow = rows.out_row(row);
    if (orow < 0) return;
    const int c = threadIdx.x % DQ, way = threadIdx.x / DQ;
    const int tiles = (s.len + kTileRows - 1) / kTileRows, steps = (tiles + tps - 1) / tps;
    const int span = work.pre[p.v.n_seqs + 1], total = work.pre[p.v.n_seqs];
    const int u0 = work.pre[b] + (h * groups + qg) * steps, u1 = u0 + steps;
    X *dst = static_cast<X *>(p.out) + orow * D + 4 * c;
    if (steps == 0) {
        if (way == 0) Act<DT>::store4(dst, make_float4(0.f, 0.f, 0.f, 0.f));
        if (threadIdx.x == 0 && p.lse) p.lse[orow] = -CUDART_INF_F;
        return;
    }
    const int wf = u0 / span, wl = (u1 - 1) / span;
    if (wf == wl) return;  // one warp had all of it
    const bool tail = u1 < min(static_cast<long long>(total), (static_cast<long long>(wl) + 1) * span);  // warp wl went on
    const int lastg = tail ? wl - 1 : wl;
    const int c0 = wf / warps, n_cta = lastg / warps - c0 + 1;
    const int n = n_cta + (tail ? 1 : 0);
    if (n == 1) return;  // one CTA had all of it
    float M = -CUDART_INF_F, L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kChunk = 8;  // pieces in flight per thread
    for (int i0 = way; i0 < n; i0 += kChunk * kMergeWays) {
        float pm[kChunk], pl[kChunk];
        float4 po[kChunk];
#pragma unroll
        for (int u = 0; u < kChunk; ++u) {
            const int i = i0 + u * kMergeWays;
            pm[u] = -CUDART_INF_F;
            pl[u] = 0.f;
            po[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < n) {
                const int slot = i < n_cta ? 2 * max(wf, (c0 + i) * warps) : 2 * wl + 1;
                const size_t r = static_cast<size_t>(slot) * kRows + row;
                pm[u] = __ldcg(work.m + r);
                pl[u] = __ldcg(work.l + r);
                po[u] = __ldcg(reinterpret_cast<const float4 *>(work.o + r * D + 4 * c));
            }
        }
        float mn = M;
#pragma unroll
        for (int u = 0; u < kChunk; ++u) mn = fmaxf(mn, pm[u]);
        if (mn == -CUDART_INF_F) continue;
        const float k0 = M == -CUDART_INF_F ? 0.f : fast_ex2(M - mn);
        a = make_float4(a.x * k0, a.y * k0, a.z * k0, a.w * k0);
        L *= k0;
#pragma unroll
        for (int u = 0; u < kChunk; ++u) {
            const float k = pm[u] == -CUDART_INF_F ? 0.f : fast_ex2(pm[u] - mn);
            a = make_float4(fmaf(k, po[u].x, a.x), fmaf(k, po[u].y, a.y), fmaf(k, po[u].z, a.z), fmaf(k, po[u].w, a.w));
            L = fmaf(k, pl[u], L);
        }
        M = mn;
    }
    s_a[way][c] = a;
    if (c == 0) {
        s_m[way] = M;
        s_l[way] = L;
    }
    __syncthreads();
    if (way != 0) return;
    M = s_m[0];
#pragma unroll
    for (int w = 1; w < kMergeWays; ++w) M = fmaxf(M, s_m[w]);
    a = make_float4(0.f, 0.f, 0.f, 0.f);
    L = 0.f;
#pragma unroll
    for (int w = 0; w < kMergeWays; ++w) {
        const float k = s_m[w] == -CUDART_INF_F ? 0.f : fast_ex2(s_m[w] - M);
        const float4 y = s_a[w][c];
        a = make_float4(fmaf(k, y.x, a.x), fmaf(k, y.y, a.y), fmaf(k, y.z, a.z), fmaf(k, y.w, a.w));
        L = fmaf(k, s_l[w], L);
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    Act<DT>::store4(dst, make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv));
    if (c == 0 && p.lse) p.lse[orow] = L > 0.f ? (M + __log2f(L)) * kSplitLn2 : -CUDART_INF_F;
}

constexpr int kSplitMaxWarps = 16;
// Most query rows per KV head, and most steps, of a sequence of this kernel's class.
inline long long split_max_rows(const PagedAttnParams &p) {
    return static_cast<long long>(p.v.max_q < p.from_q ? p.v.max_q : p.from_q - 1) * p.G;
}
inline long long split_seq_steps(const PagedAttnParams &p) {
    return paged_steps((static_cast<long long>(p.v.max_len) + kTileRows - 1) / kTileRows, split_max_rows(p), kRows, p.v.Hkv);
}
// One CTA per unit, or equal spans?  A unit costs its CTA about 4.5 us + 4.9 us per 1024 keys; equal spans
// cost 9.5 us (sums over the batch, the merge) and then 2 us + 4.7 us per 1024 keys for each unit per SM
// (q4_0, 128-wide; measured over 1 to 128 sequences of 8 KV heads, 128 to 4096 positions: 8 units of 128 /
// 512 / 1024 keys 5.5 / 7.4 / 10.3 against 9.9 / 10.7 / 11.0 us, 128 units of 2048 keys 15.9 against 20.0,
// 304 units of 1024 keys 20.8 against 23.7, 512 units of 512 keys 28.4 against 25.0).  Lengths are known
// here by their bound alone, and a CTA per unit waits for the longest, so the bound stays near the point
// where the two are equal for even lengths in one wave, and below it in two.
inline bool unit_per_cta(long long units, int max_len, int sms) {
    if (units <= sms) return max_len <= 1024 + 1024 * units / sms;
    return units <= 2ll * sms && 2 * units >= 3ll * sms && max_len <= 1024;
}

template <int KT, int VT, int NS, int DT>
cudaError_t launch_split_t(const PagedAttnParams &p, cudaStream_t stream) {
    using C = SplitCfg<KT, VT, NS, DT>;
    static_assert(C::WARPS <= kSplitMaxWarps, "workspace");
    static bool configured[kPagedMaxDevices] = {};
    int dev = 0, sms = 0;
    cudaError_t e = paged_device(&dev, &sms);
    if (e != cudaSuccess) return e;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(paged_split_kernel<KT, VT, NS, DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        // the merge runs right after the split kernel: with the same division of the SM's memory, no SM has
        // to be drained and set up anew between the two
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(paged_merge_kernel<NS, DT>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    const SplitWork work = split_work(p.workspace, 2 * kSplitMaxWarps * sms);
    const int max_groups = static_cast<int>((split_max_rows(p) + kRows - 1) / kRows);
    // sequences of one launch: their prefix sums fit shared memory, their steps 2^30
    const long long fit = kPagedMaxSteps / split_seq_steps(p);
    const int most = static_cast<int>(fit < kSplitMaxSeqs ? fit : kSplitMaxSeqs);
    if (most < 1) return cudaErrorNotSupported;
    for (int b = 0; b < p.v.n_seqs; b += most) {
        const PagedAttnParams q = paged_some(p, b, most);
        const long long units = static_cast<long long>(q.v.n_seqs) * p.v.Hkv * max_groups;
        if (unit_per_cta(units, p.v.max_len, sms)) {
            e = launch_dependent(paged_split_kernel<KT, VT, NS, DT>, dim3(static_cast<unsigned>(units)), C::THREADS, C::SMEM, stream,
                                 q, work, max_groups);
            if (e != cudaSuccess) return e;
            continue;
        }
        e = launch_dependent(paged_split_kernel<KT, VT, NS, DT>, dim3(sms), C::THREADS, C::SMEM, stream, q, work, 0);
        if (e != cudaSuccess) return e;
        e = launch_dependent(paged_merge_kernel<NS, DT>, dim3(static_cast<unsigned>(units * kRows)), NS * 32 * kMergeWays, 0, stream,
                             q, work, static_cast<int>(C::WARPS), static_cast<int>(C::TPS), max_groups);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <int DT>
cudaError_t launch_split_dt(int type_k, int type_v, int D, const PagedAttnParams &p, cudaStream_t s) {
#define KVQ_SPLIT_CASE(KT_, VT_)                                                  \
    if (type_k == KT_ && type_v == VT_) {                                         \
        if (D == kSlice) return launch_split_t<KT_, VT_, 1, DT>(p, s);            \
        if (D == 2 * kSlice) return launch_split_t<KT_, VT_, 2, DT>(p, s);        \
    }
    KVQ_SPLIT_CASE(KVQ_F16, KVQ_F16)
    KVQ_SPLIT_CASE(KVQ_Q8_0, KVQ_Q8_0)
    KVQ_SPLIT_CASE(KVQ_Q8_0, KVQ_Q4_0)
    KVQ_SPLIT_CASE(KVQ_Q4_0, KVQ_Q4_0)
#undef KVQ_SPLIT_CASE
    return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace kvq
