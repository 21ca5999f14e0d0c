// kvq_paged_append.cu -- rows of the paged cache: append (rotary position embedding and
// quantisation on the way in) and gather (values out).
#include "kvq_paged.cuh"

// Bound by memory for chunks and by latency for single tokens (us on a GB300, of measured copy bandwidth):
// append of 10017 tokens in 3 chunks, 8 KV and 40 query heads of 128 rotated, bf16 to q4_0, 69 us (3.9 TB/s, 57 %:
// half the grid quantises, bound by its instructions, half rotates queries, bound by memory); 4096 tokens, 2 and 16
// heads of 256, fp32 to q8_0, 39 us (4.0 TB/s); one token 7.1 us, 64 tokens 8.2 us.  Gather of 65536 positions,
// q8_0 / q4_0 to bf16: 67 us (5.7 TB/s, 83 %); five short sequences 4.4 us.
namespace kvq {
namespace {

// Four consecutive values at `dim` of a row, rotated: y = x cos -/+ partner sin, one fp32
// rounding per operation.  `row` is the head's row, `ang` the token's angles (cosines, then
// sines).  rot_dim is a multiple of 8, so the four values are on one side of a pair.
template <int DT>
__device__ __forceinline__ float4 rotated4(const typename Act<DT>::type *row, int dim, const float *ang, int rot_dim,
                                           int interleaved) {
    const float4 x = Act<DT>::load4(row + dim);
    if (ang == nullptr || dim >= rot_dim) return x;
    const int half = rot_dim >> 1;
    float4 y;
    if (interleaved) {  // pairs (x, y) and (z, w), angles dim / 2 and dim / 2 + 1
        const float2 c = __ldg(reinterpret_cast<const float2 *>(ang + (dim >> 1)));
        const float2 s = __ldg(reinterpret_cast<const float2 *>(ang + half + (dim >> 1)));
        y.x = __fsub_rn(__fmul_rn(x.x, c.x), __fmul_rn(x.y, s.x));
        y.y = __fadd_rn(__fmul_rn(x.y, c.x), __fmul_rn(x.x, s.x));
        y.z = __fsub_rn(__fmul_rn(x.z, c.y), __fmul_rn(x.w, s.y));
        y.w = __fadd_rn(__fmul_rn(x.w, c.y), __fmul_rn(x.z, s.y));
        return y;
    }
    const bool low = dim < half;
    const int j = low ? dim : dim - half;
    const float4 o = Act<DT>::load4(row + (low ? dim + half : dim - half));
    const float4 c = __ldg(reinterpret_cast<const float4 *>(ang + j));
    const float4 s = __ldg(reinterpret_cast<const float4 *>(ang + half + j));
    auto turn = [&](float a, float b, float cc, float ss) {
        const float p = __fmul_rn(a, cc), q = __fmul_rn(b, ss);
        return low ? __fsub_rn(p, q) : __fadd_rn(p, q);
    };
    return make_float4(turn(x.x, o.x, c.x, s.x), turn(x.y, o.y, c.y, s.y), turn(x.z, o.z, c.z, s.z),
                       turn(x.w, o.w, c.w, s.w));
}

// every sequence's entries, by one block of the launch
__device__ __forceinline__ void check_batch(const PagedView &v) {
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int b = threadIdx.x; b < v.n_seqs; b += blockDim.x)
            if (!paged_seq(v, b).ok) paged_error(v);
}

// A lane's share of a rotated head: two groups of four values that rotate together, [a, a + 4) and
// [b, b + 4).  D / 8 lanes hold a head, so that no value is loaded twice.
struct TurnPair {
    int a, b;
    bool turn;  // false: values behind rot_dim, passed through
};
__device__ __forceinline__ TurnPair turn_pair(int u, int rot_dim, int interleaved) {
    const bool turn = 8 * u < rot_dim;
    if (interleaved || !turn) return TurnPair{8 * u, 8 * u + 4, turn};
    return TurnPair{4 * u, 4 * u + (rot_dim >> 1), true};
}
// in place; c, s: the four angles from 4 u on
__device__ __forceinline__ void turn4(float4 &x, float4 &y, float4 c, float4 s, int interleaved) {
    auto turn = [](float &a, float &b, float cc, float ss) {
        const float p = __fsub_rn(__fmul_rn(a, cc), __fmul_rn(b, ss));
        b = __fadd_rn(__fmul_rn(b, cc), __fmul_rn(a, ss));
        a = p;
    };
    if (interleaved) {
        turn(x.x, x.y, c.x, s.x);
        turn(x.z, x.w, c.y, s.y);
        turn(y.x, y.y, c.z, s.z);
        turn(y.z, y.w, c.w, s.w);
    } else {
        turn(x.x, y.x, c.x, s.x);
        turn(x.y, y.y, c.y, s.y);
        turn(x.z, y.z, c.z, s.z);
        turn(x.w, y.w, c.w, s.w);
    }
}

// Append, one warp per (token, KV head or query head): the rows of a KV head are rotated,
// quantised and stored at their places of the tile; those of a query head are rotated.
template <int KT, int VT, int NS, int DT>
__global__ void __launch_bounds__(256) paged_append_rows(const PagedAppendParams p) {
    using T = PagedTile<KT, VT, NS>;
    using X = typename Act<DT>::type;
    check_batch(p.v);
    const int lane = threadIdx.x & 31;
    const int slots = p.v.Hkv + p.Hq;
    const long long items = static_cast<long long>(p.v.n_tokens) * slots;
    const long long n_warps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
    for (long long it = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); it < items; it += n_warps) {
        const int token = static_cast<int>(it / slots), slot = static_cast<int>(it % slots);
        const int b = paged_find(p.v, token);
        if (b < 0) continue;
        const PagedSeq s = paged_seq(p.v, b);
        if (!s.ok || token < s.first || token >= s.first + s.n) {
            if (lane == 0) paged_error(p.v);
            continue;
        }
        const int pos = s.len - s.n + (token - s.first);
        if (pos < 0) continue;
        const float *ang = nullptr;
        if (p.cos_sin) {
            const int r = p.positions ? __ldg(p.positions + token) : pos;
            if (r < 0 || r >= p.n_positions) {
                if (lane == 0) paged_error(p.v);
                continue;
            }
            ang = p.cos_sin + static_cast<size_t>(r) * p.rot_dim;
        }
        if (slot >= p.v.Hkv) {  // a query head; every value is read before any is written
            const X *src = static_cast<const X *>(p.q) + token * p.q_stride + static_cast<size_t>(slot - p.v.Hkv) * T::D;
            X *dst = static_cast<X *>(p.q_out) + token * p.q_out_stride + static_cast<size_t>(slot - p.v.Hkv) * T::D;
            float4 y[NS];
#pragma unroll
            for (int sl = 0; sl < NS; ++sl) y[sl] = rotated4<DT>(src, sl * kSlice + 4 * lane, ang, p.rot_dim, p.interleaved);
            __syncwarp();
#pragma unroll
            for (int sl = 0; sl < NS; ++sl) Act<DT>::store4(dst + sl * kSlice + 4 * lane, y[sl]);
            continue;
        }
        uint8_t *rec = paged_tile<T>(p.v, b, slot, pos >> 4);
        if (!rec) {
            if (lane == 0) paged_error(p.v);
            continue;
        }
        const X *kr = static_cast<const X *>(p.k) + token * p.k_stride + static_cast<size_t>(slot) * T::D;
        const X *vr = static_cast<const X *>(p.v_in) + token * p.v_stride + static_cast<size_t>(slot) * T::D;
#pragma unroll
        for (int sl = 0; sl < NS; ++sl) {
            const float4 xk = rotated4<DT>(kr, sl * kSlice + 4 * lane, ang, p.rot_dim, p.interleaved);
            const float4 xv = Act<DT>::load4(vr + sl * kSlice + 4 * lane);
            quantize_store_vals<KT, false>(xk, rec + sl * code_tile_bytes(KT),
                                           rec + T::OFF_KS + sl * scale_tile_bytes(KT), pos & 15, lane);
            quantize_store_vals<VT, true>(xv, rec + T::OFF_V + sl * code_tile_bytes(VT),
                                          rec + T::OFF_VS + sl * scale_tile_bytes(VT), pos & 15, lane);
        }
    }
}

// Gather, one warp per (token, KV head).
template <int KT, int VT, int NS, int DT>
__global__ void __launch_bounds__(256) paged_gather_rows(const PagedGatherParams p) {
    using T = PagedTile<KT, VT, NS>;
    using X = typename Act<DT>::type;
    check_batch(p.v);
    const int lane = threadIdx.x & 31;
    const long long items = static_cast<long long>(p.v.n_tokens) * p.v.Hkv;
    const long long n_warps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
    for (long long it = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); it < items; it += n_warps) {
        const int token = static_cast<int>(it / p.v.Hkv), h = static_cast<int>(it % p.v.Hkv);
        const int b = paged_find(p.v, token);
        if (b < 0) continue;
        const PagedSeq s = paged_seq(p.v, b);
        if (!s.ok || token < s.first || token >= s.first + s.n) {
            if (lane == 0) paged_error(p.v);
            continue;
        }
        const int pos = s.len - s.n + (token - s.first);
        const uint8_t *rec = pos >= 0 ? paged_tile<T>(p.v, b, h, pos >> 4) : nullptr;
        if (!rec && pos >= 0 && lane == 0) paged_error(p.v);
        const size_t row = static_cast<size_t>(it) * T::D;
#pragma unroll
        for (int sl = 0; sl < NS; ++sl) {
            float4 xk = make_float4(0.f, 0.f, 0.f, 0.f), xv = xk;
            if (rec) {
                xk = dequantize4<KT, false>(rec + sl * code_tile_bytes(KT), rec + T::OFF_KS + sl * scale_tile_bytes(KT), pos & 15, lane);
                xv = dequantize4<VT, true>(rec + T::OFF_V + sl * code_tile_bytes(VT), rec + T::OFF_VS + sl * scale_tile_bytes(VT), pos & 15, lane);
            }
            Act<DT>::store4(static_cast<X *>(p.k_out) + row + sl * kSlice + 4 * lane, xk);
            Act<DT>::store4(static_cast<X *>(p.v_out) + row + sl * kSlice + 4 * lane, xv);
        }
    }
}

// ---- whole tiles ----
// Chunks: one CTA takes one 16-row tile of a sequence and one KV head.  In the tile layout the codes of
// a row lie between those of other rows, so rows written one by one are byte stores over the whole
// record; a tile that the call fills is assembled in shared memory instead and leaves as 16-byte
// stores (a tile that it fills in part is written row by row, other rows' bytes untouched).

// The tile piece of a block: sequence, tile, first and last row of it that belong to the call.  Sequence b
// owns the pieces from cu_q[b] / 16 + 2 b on: n tokens touch at most n / 16 + 2 tiles.
struct Piece {
    PagedSeq s;
    int b, tile, r0, r1;  // rows [r0, r1) of the tile; r0 >= r1: nothing
};
__device__ __forceinline__ Piece find_piece(const PagedView &v, int p) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = v.n_seqs;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5;
        const int i = lo + lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, i < hi && (i == 0 || (__ldg(v.cu_q + i) >> 4) + 2 * i <= p));
        lo += (__popc(below) - 1) * step;
        hi = min(hi, lo + step);
    }
    Piece c;
    c.b = lo;
    c.s = paged_seq(v, lo);
    const int k = p - ((c.s.first >> 4) + 2 * lo), pos0 = c.s.len - c.s.n;  // pos0 < 0: tokens before position 0
    const int tile0 = max(pos0, 0) >> 4, tiles = (c.s.len + (kTileRows - 1)) / kTileRows;
    const bool any = k >= 0 && k < tiles - tile0 && c.s.n > 0;  // else no tile of the sequence
    c.tile = any ? tile0 + k : tile0;
    c.r0 = max(0, max(pos0, 0) - c.tile * kTileRows);
    c.r1 = any ? min(kTileRows, c.s.len - c.tile * kTileRows) : 0;
    return c;
}
__host__ __device__ inline long long piece_bound(const PagedView &v) { return v.n_tokens / kTileRows + 2ll * v.n_seqs; }

// One thread quantises one 32-value block of one row, of K or of V (quantize_block_store): one search and
// two divisions per block and no shuffles, a third of the instructions of a warp per row.
template <int NS>
struct TileThreads {
    static constexpr int HALF = kTileRows * NS * 4, ALL = 2 * HALF;  // blocks of K; of K and V
};

constexpr int kQueryHeads = 4;  // query heads that one block rotates

template <int KT, int VT, int NS, int DT>
__global__ void __launch_bounds__(TileThreads<NS>::ALL, 8 / NS) paged_append_tiles(const PagedAppendParams p) {
    using T = PagedTile<KT, VT, NS>;
    using X = typename Act<DT>::type;
    constexpr int THREADS = TileThreads<NS>::ALL, HALF = TileThreads<NS>::HALF;
    __shared__ __align__(16) uint8_t image[T::BYTES];
    check_batch(p.v);
    // a piece's blocks: one per KV head to quantise, then those that rotate kQueryHeads query heads each; the
    // former are bound by their instructions, the latter by memory, so they are neighbours in the grid
    const int parts = p.v.Hkv + (p.Hq + kQueryHeads - 1) / kQueryHeads;
    const int h = static_cast<int>(blockIdx.x % parts);
    const bool queries = h >= p.v.Hkv;
    const Piece c = find_piece(p.v, blockIdx.x / parts);
    if (c.r0 >= c.r1) return;
    const int token0 = c.s.first + c.tile * kTileRows - (c.s.len - c.s.n);  // token of row 0
    auto angle_row = [&](int r) -> const float * {  // nullptr: outside the table
        const int a = p.positions ? __ldg(p.positions + token0 + r) : c.tile * kTileRows + r;
        return a < 0 || a >= p.n_positions ? nullptr : p.cos_sin + static_cast<size_t>(a) * p.rot_dim;
    };
    if (!queries) {
        // ---- keys and values ----
        uint8_t *rec = paged_tile<T>(p.v, c.b, h, c.tile);
        if (!rec && threadIdx.x == 0) paged_error(p.v);
        const bool is_v = threadIdx.x >= HALF;
        const int idx = threadIdx.x % HALF, r = idx / (NS * 4), blk = idx % (NS * 4), sl = blk >> 2, b = blk & 3;
        bool in = rec && r >= c.r0 && r < c.r1;
        const float *ang = nullptr;
        if (in && p.cos_sin) {  // a row without angles is left out, its values too
            ang = angle_row(r);
            if (!ang) {
                paged_error(p.v);
                in = false;
            }
        }
        // a tile that the call fills leaves through the image; else its rows are written in place
        const bool full = __syncthreads_and(in);
        if (in) {
            float x[kBlock];
            if (is_v) {
                const X *row = static_cast<const X *>(p.v_in) + (token0 + r) * p.v_stride + static_cast<size_t>(h) * T::D + kBlock * blk;
    #pragma unroll
                for (int i = 0; i < kBlock; i += 4) {
                    const float4 y = Act<DT>::load4(row + i);
                    x[i] = y.x, x[i + 1] = y.y, x[i + 2] = y.z, x[i + 3] = y.w;
                }
            } else {
                const X *row = static_cast<const X *>(p.k) + (token0 + r) * p.k_stride + static_cast<size_t>(h) * T::D;
    #pragma unroll
                for (int i = 0; i < kBlock; i += 4) {
                    const float4 y = rotated4<DT>(row, kBlock * blk + i, ang, p.rot_dim, p.interleaved);
                    x[i] = y.x, x[i + 1] = y.y, x[i + 2] = y.z, x[i + 3] = y.w;
                }
            }
            uint8_t *to = full ? image : rec;
            if (is_v)
                quantize_block_store<VT, true>(x, to + T::OFF_V + sl * code_tile_bytes(VT), to + T::OFF_VS + sl * scale_tile_bytes(VT), r, b);
            else
                quantize_block_store<KT, false>(x, to + sl * code_tile_bytes(KT), to + T::OFF_KS + sl * scale_tile_bytes(KT), r, b);
        }
        if (full) {
            __syncthreads();
            for (int o = threadIdx.x * 16; o < T::BYTES; o += THREADS * 16)
                *reinterpret_cast<uint4 *>(rec + o) = *reinterpret_cast<const uint4 *>(image + o);
        }
    } else {
        // ---- query heads [q0, q0 + n): UNIT lanes per row, a row's angles read once ----
        const int q0 = (h - p.v.Hkv) * kQueryHeads, n = min(kQueryHeads, p.Hq - q0);
        constexpr int UNIT = T::D / 8, ROWS = THREADS / UNIT, kAhead = 4;
        const int u = threadIdx.x % UNIT;
        const TurnPair tp = turn_pair(u, p.rot_dim, p.interleaved);
        for (int qr = c.r0 + threadIdx.x / UNIT; qr < c.r1; qr += ROWS) {
            const float *qa = angle_row(qr);
            if (!qa) {
                paged_error(p.v);
                continue;
            }
            float4 cs = make_float4(0.f, 0.f, 0.f, 0.f), sn = cs;
            if (tp.turn) {
                cs = __ldg(reinterpret_cast<const float4 *>(qa + 4 * u));
                sn = __ldg(reinterpret_cast<const float4 *>(qa + (p.rot_dim >> 1) + 4 * u));
            }
            const X *src = static_cast<const X *>(p.q) + (token0 + qr) * p.q_stride + static_cast<size_t>(q0) * T::D;
            X *dst = static_cast<X *>(p.q_out) + (token0 + qr) * p.q_out_stride + static_cast<size_t>(q0) * T::D;
            for (int g0 = 0; g0 < n; g0 += kAhead) {  // q_out may be q: a lane reads what it writes first
                float4 x[kAhead], y[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (g0 + k < n) {
                        x[k] = Act<DT>::load4(src + (g0 + k) * T::D + tp.a);
                        y[k] = Act<DT>::load4(src + (g0 + k) * T::D + tp.b);
                    }
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (g0 + k < n) {
                        if (tp.turn) turn4(x[k], y[k], cs, sn, p.interleaved);
                        Act<DT>::store4(dst + (g0 + k) * T::D + tp.a, x[k]);
                        Act<DT>::store4(dst + (g0 + k) * T::D + tp.b, y[k]);
                    }
            }
        }
    }
}

// Gather of tiles, one warp per (piece, KV head).  A lane loads the 16-byte groups that belong to it (a warp's
// loads are contiguous), turns codes into values two at a time, and lays them in a row-major stage in
// shared memory, from which the rows leave as 16-byte stores.
constexpr int kGatherWarps = 4;

// A pair of exact code values (f16 integers) times a scale, rounded once to the output type.
template <int DT>
__device__ __forceinline__ void emit2(typename Act<DT>::type *p, __half2 c, __half2 d2) {
    if constexpr (DT == KVQ_DT_F16) {
        *reinterpret_cast<__half2 *>(p) = __hmul2(c, d2);
    } else {
        const float2 f = __half22float2(c);
        const float d = __low2float(d2);
        Act<DT>::store2(p, f.x * d, f.y * d);
    }
}
__device__ __forceinline__ uint32_t byte_perm(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;\n" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}
// q8_0 codes: sign in bit 15, magnitude in the low bits (a subnormal q 2^-24) to the f16 integer q, exactly
__device__ __forceinline__ __half2 code8(uint32_t x) {
    return __hmul2(__hmul2(u32_as_h2(x & 0x807f807fu), __float2half2_rn(16384.0f)), __float2half2_rn(1024.0f));
}
// q4_0 codes in the low or high nibble of each half's low byte: c - 8, exactly
__device__ __forceinline__ __half2 code4_low(uint32_t x) {
    return __hsub2(u32_as_h2((x & 0x000f000fu) | 0x64006400u), __float2half2_rn(1032.0f));
}
__device__ __forceinline__ __half2 code4_high(uint32_t x) {
    return __hfma2(u32_as_h2((x & 0x00f000f0u) | 0x64006400u), __float2half2_rn(0.0625f), __float2half2_rn(-72.0f));
}
__device__ __forceinline__ __half2 twice(uint32_t pair, int upper) {  // one half of a pair, twice
    return u32_as_h2(byte_perm(pair, 0u, upper ? 0x3232u : 0x1010u));
}

// The values of one 128-value slice of a tile into the stage: [16][128 + padding] of the output type.
template <int KT, int DT, int RS>
__device__ __forceinline__ void stage_keys(const uint8_t *codes, const uint8_t *scales, typename Act<DT>::type *stage) {
    using X = typename Act<DT>::type;
    const int lane = threadIdx.x & 31, n = lane >> 2, jd = lane & 3;  // keys n, n + 8; values 4 jd .. of each sixteen
    auto put = [&](int key, int dim, __half2 c02, __half2 c13, __half2 d2) {
        // codes of values (0, 2) and (1, 3) of the four
        const __half2 c01 = u32_as_h2(byte_perm(h2_as_u32(c02), h2_as_u32(c13), 0x5410u));
        const __half2 c23 = u32_as_h2(byte_perm(h2_as_u32(c02), h2_as_u32(c13), 0x7632u));
        X *to = stage + key * RS + dim + 4 * jd;
        emit2<DT>(to, c01, d2);
        emit2<DT>(to + 2, c23, d2);
    };
    if constexpr (KT == KVQ_F16) {
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
            const uint4 c = __ldg(reinterpret_cast<const uint4 *>(codes + (ch * 32 + lane) * 16));
            const __half2 one = __float2half2_rn(1.0f);
            put(n + 8 * (ch & 1), 32 * (ch >> 1), u32_as_h2(c.x), u32_as_h2(c.y), one);
            put(n + 8 * (ch & 1), 32 * (ch >> 1) + 16, u32_as_h2(c.z), u32_as_h2(c.w), one);
        }
    } else if constexpr (KT == KVQ_Q8_0) {
        uint4 c[4];
        uint2 sc[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            c[b] = __ldg(reinterpret_cast<const uint4 *>(codes + (b * 32 + lane) * 16));
            sc[b] = __ldg(reinterpret_cast<const uint2 *>(scales + (n >> 1) * 32 + b * 8));
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const __half2 da = twice(sc[b].x, n & 1), db = twice(sc[b].y, n & 1);
            auto lo = [](uint32_t w) { return code8(byte_perm(w, 0u, 0xA280u)); };
            auto hi = [](uint32_t w) { return code8(byte_perm(w, 0u, 0xB391u)); };
            put(n, 32 * b, lo(c[b].x), hi(c[b].x), da);
            put(n, 32 * b + 16, lo(c[b].y), hi(c[b].y), da);
            put(n + 8, 32 * b, lo(c[b].z), hi(c[b].z), db);
            put(n + 8, 32 * b + 16, lo(c[b].w), hi(c[b].w), db);
        }
    } else {
        uint4 c[2], sc[2];
#pragma unroll
        for (int b2 = 0; b2 < 2; ++b2) {
            c[b2] = __ldg(reinterpret_cast<const uint4 *>(codes + (b2 * 32 + lane) * 16));
            sc[b2] = __ldg(reinterpret_cast<const uint4 *>(scales + (n >> 1) * 32 + b2 * 16));
        }
#pragma unroll
        for (int b2 = 0; b2 < 2; ++b2) {
            const uint32_t cs[4] = {c[b2].x, c[b2].y, c[b2].z, c[b2].w}, ss[4] = {sc[b2].x, sc[b2].y, sc[b2].z, sc[b2].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {  // block 2 b2 + q / 2, key n + 8 (q % 2)
                const __half2 d2 = twice(ss[q], n & 1);
                const uint32_t odd = cs[q] >> 8;
                put(n + 8 * (q & 1), 64 * b2 + 32 * (q >> 1), code4_low(cs[q]), code4_low(odd), d2);
                put(n + 8 * (q & 1), 64 * b2 + 32 * (q >> 1) + 16, code4_high(cs[q]), code4_high(odd), d2);
            }
        }
    }
}
template <int VT, int DT, int RS>
__device__ __forceinline__ void stage_values(const uint8_t *codes, const uint8_t *scales, typename Act<DT>::type *stage) {
    using X = typename Act<DT>::type;
    const int lane = threadIdx.x & 31, np = lane >> 2, j = lane & 3;  // values 2 np, 2 np + 1 of each sixteen; keys 2j, 2j + 1, + 8
    auto put = [&](int key, int dim, __half2 c, __half2 d2) { emit2<DT>(stage + key * RS + dim + 2 * np, c, d2); };
    // byte i of a code word belongs to key kk(i)
    auto kk = [&](int i) { return 2 * j + (i >> 1) + 8 * (i & 1); };
    if constexpr (VT == KVQ_F16) {
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
            const uint4 c = __ldg(reinterpret_cast<const uint4 *>(codes + (ch * 32 + lane) * 16));
            const __half2 one = __float2half2_rn(1.0f);
            const int dim = 32 * (ch >> 1) + 16 * (ch & 1);
            put(2 * j, dim, u32_as_h2(byte_perm(c.x, c.z, 0x5410u)), one);
            put(2 * j + 1, dim, u32_as_h2(byte_perm(c.x, c.z, 0x7632u)), one);
            put(2 * j + 8, dim, u32_as_h2(byte_perm(c.y, c.w, 0x5410u)), one);
            put(2 * j + 9, dim, u32_as_h2(byte_perm(c.y, c.w, 0x7632u)), one);
        }
    } else {
        constexpr int NG = VT == KVQ_Q8_0 ? 4 : 2;
        uint4 c[NG];
        uint2 sc[4];
#pragma unroll
        for (int i = 0; i < NG; ++i) c[i] = __ldg(reinterpret_cast<const uint4 *>(codes + (i * 32 + lane) * 16));
#pragma unroll
        for (int b = 0; b < 4; ++b) sc[b] = __ldg(reinterpret_cast<const uint2 *>(scales + j * 32 + b * 8));
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const __half2 d[4] = {twice(sc[b].x, 0), twice(sc[b].y, 0), twice(sc[b].x, 1), twice(sc[b].y, 1)};  // of kk(0) .. kk(3)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (VT == KVQ_Q8_0) {  // sign and magnitude of byte i of both words
                    put(kk(i), 32 * b, code8(byte_perm(c[b].x, c[b].y, 0xC480u + 0x1111u * i)), d[i]);
                    put(kk(i), 32 * b + 16, code8(byte_perm(c[b].z, c[b].w, 0xC480u + 0x1111u * i)), d[i]);
                } else {
                    const uint32_t x = (b & 1) ? c[b >> 1].z : c[b >> 1].x, y = (b & 1) ? c[b >> 1].w : c[b >> 1].y;
                    const uint32_t two = byte_perm(x, y, 0x4400u + 0x1111u * i);
                    put(kk(i), 32 * b, code4_low(two), d[i]);
                    put(kk(i), 32 * b + 16, code4_high(two), d[i]);
                }
            }
        }
    }
}

template <int KT, int VT, int NS, int DT>
__global__ void __launch_bounds__(32 * kGatherWarps) paged_gather_tiles(const PagedGatherParams p) {
    using T = PagedTile<KT, VT, NS>;
    using X = typename Act<DT>::type;
    constexpr int RS = kSlice + 16 / static_cast<int>(sizeof(X));  // 16 bytes of padding: stage stores without conflicts
    constexpr int PER = 16 / static_cast<int>(sizeof(X));          // values of a 16-byte store
    __shared__ __align__(16) X stage_all[kGatherWarps][kTileRows * RS];
    check_batch(p.v);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * kGatherWarps + warp;
    if (item >= piece_bound(p.v) * p.v.Hkv) return;
    X *stage = stage_all[warp];
    const int h = static_cast<int>(item % p.v.Hkv), pi = static_cast<int>(item / p.v.Hkv);
    const Piece c = find_piece(p.v, pi);
    const int pos0 = c.s.len - c.s.n;
    if (pos0 < 0 && c.s.n > 0 && pi == (c.s.first >> 4) + 2 * c.b) {  // tokens of no position: zeros
        const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < min(c.s.n, -pos0); ++i) {
            const size_t row = (static_cast<size_t>(c.s.first + i) * p.v.Hkv + h) * T::D;
#pragma unroll
            for (int sl = 0; sl < NS; ++sl) {
                Act<DT>::store4(static_cast<X *>(p.k_out) + row + sl * kSlice + 4 * lane, z);
                Act<DT>::store4(static_cast<X *>(p.v_out) + row + sl * kSlice + 4 * lane, z);
            }
        }
    }
    if (c.r0 >= c.r1) return;
    const uint8_t *rec = paged_tile<T>(p.v, c.b, h, c.tile);
    if (!rec && lane == 0) paged_error(p.v);
    const int token0 = c.s.first + c.tile * kTileRows - pos0;  // token of row 0
#pragma unroll
    for (int part = 0; part < 2 * NS; ++part) {
        const int sl = part >> 1;
        if (rec) {
            if (part & 1)
                stage_values<VT, DT, RS>(rec + T::OFF_V + sl * code_tile_bytes(VT), rec + T::OFF_VS + sl * scale_tile_bytes(VT), stage);
            else
                stage_keys<KT, DT, RS>(rec + sl * code_tile_bytes(KT), rec + T::OFF_KS + sl * scale_tile_bytes(KT), stage);
        }
        __syncwarp();
        X *out = static_cast<X *>((part & 1) ? p.v_out : p.k_out);
#pragma unroll
        for (int i = 0; i < kTileRows * kSlice / PER / 32; ++i) {
            const int e = i * 32 + lane, r = e / (kSlice / PER), at = (e % (kSlice / PER)) * PER;
            const uint4 w = rec ? *reinterpret_cast<const uint4 *>(stage + r * RS + at) : make_uint4(0u, 0u, 0u, 0u);
            if (r >= c.r0 && r < c.r1)
                *reinterpret_cast<uint4 *>(out + (static_cast<size_t>(token0 + r) * p.v.Hkv + h) * T::D + sl * kSlice + at) = w;
        }
        __syncwarp();
    }
}

// Chunks of a tile or more go tile by tile, single tokens and drafts row by row (a tile's CTA would have
// one or a few of its 16 rows to do).
bool by_tiles(const PagedView &v) { return v.max_q >= kTileRows; }

int grid_for(long long warps) {
    const long long blocks = (warps + 7) / 8;
    return static_cast<int>(blocks < 8 * 152 ? (blocks > 0 ? blocks : 1) : 8 * 152);
}

template <int KT, int VT, int NS, int DT>
cudaError_t append_t(const PagedAppendParams &p, cudaStream_t s) {
    const long long tiles = by_tiles(p.v) ? piece_bound(p.v) * (p.v.Hkv + (p.Hq + kQueryHeads - 1) / kQueryHeads) : 0;
    if (tiles > 0 && tiles < (1ll << 31)) {
        paged_append_tiles<KT, VT, NS, DT><<<static_cast<unsigned>(tiles), TileThreads<NS>::ALL, 0, s>>>(p);
        return cudaGetLastError();
    }
    const long long warps = static_cast<long long>(p.v.n_tokens) * (p.v.Hkv + p.Hq);
    paged_append_rows<KT, VT, NS, DT><<<grid_for(warps), 256, 0, s>>>(p);
    return cudaGetLastError();
}
template <int KT, int VT, int NS, int DT>
cudaError_t gather_t(const PagedGatherParams &p, cudaStream_t s) {
    const long long tiles = by_tiles(p.v) ? (piece_bound(p.v) * p.v.Hkv + kGatherWarps - 1) / kGatherWarps : 0;
    if (tiles > 0 && tiles < (1ll << 31)) {
        paged_gather_tiles<KT, VT, NS, DT><<<static_cast<unsigned>(tiles), 32 * kGatherWarps, 0, s>>>(p);
        return cudaGetLastError();
    }
    const long long warps = static_cast<long long>(p.v.n_tokens) * p.v.Hkv;
    paged_gather_rows<KT, VT, NS, DT><<<grid_for(warps), 256, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(int type_k, int type_v, int D, int dtype, const PagedAppendParams &p, cudaStream_t s) {
    KVQ_PAGED_DISPATCH(append_t, (p, s))
}
cudaError_t launch_paged_gather(int type_k, int type_v, int D, int dtype, const PagedGatherParams &p, cudaStream_t s) {
    KVQ_PAGED_DISPATCH(gather_t, (p, s))
}

}  // namespace kvq
