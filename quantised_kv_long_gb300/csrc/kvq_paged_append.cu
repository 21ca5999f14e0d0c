// kvq_paged_append.cu -- rows of the paged cache: append (rotary position embedding and
// quantisation on the way in) and gather (values out).
#include "kvq_paged.cuh"

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

// Append, one warp per (token, KV head or query head): the rows of a KV head are rotated,
// quantised and stored at their places of the tile; those of a query head are rotated.
template <int KT, int VT, int NS, int DT>
__global__ void __launch_bounds__(256) paged_append_rows(const PagedAppendParams p) {
    using T = PagedTile<KT, VT, NS>;
    using X = typename Act<DT>::type;
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

int grid_for(long long warps) {
    const long long blocks = (warps + 7) / 8;
    return static_cast<int>(blocks < 8 * 152 ? (blocks > 0 ? blocks : 1) : 8 * 152);
}

template <int KT, int VT, int NS, int DT>
cudaError_t append_t(const PagedAppendParams &p, cudaStream_t s) {
    const long long warps = static_cast<long long>(p.v.n_tokens) * (p.v.Hkv + p.Hq);
    paged_append_rows<KT, VT, NS, DT><<<grid_for(warps), 256, 0, s>>>(p);
    return cudaGetLastError();
}
template <int KT, int VT, int NS, int DT>
cudaError_t gather_t(const PagedGatherParams &p, cudaStream_t s) {
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
