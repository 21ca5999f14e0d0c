// kvq_paged_attn.cu -- attention over the paged cache.
#include <math_constants.h>

#include "kvq_paged.cuh"

namespace kvq {
namespace {

// One CTA per (token, query head); its warps take keys in turn with a running maximum each.
template <int KT, int VT, int NS, int DT>
__global__ void __launch_bounds__(128) paged_attn_rows(const PagedAttnParams p) {
    using T = PagedTile<KT, VT, NS>;
    using X = typename Act<DT>::type;
    __shared__ float s_o[4][T::D], s_m[4], s_l[4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int token = blockIdx.x, hq = blockIdx.y, h = hq / p.G;
    const int b = paged_find(p.v, token);
    if (b < 0) return;
    const PagedSeq s = paged_seq(p.v, b);
    if (!s.ok || token < s.first || token >= s.first + s.n) {
        if (threadIdx.x == 0) paged_error(p.v);
        return;
    }
    const int keys = s.len - s.n + (token - s.first) + 1;
    float4 q[NS], o[NS];
    const X *src = static_cast<const X *>(p.q) + token * p.q_stride + static_cast<size_t>(hq) * T::D;
#pragma unroll
    for (int sl = 0; sl < NS; ++sl) {
        q[sl] = Act<DT>::load4(src + sl * kSlice + 4 * lane);
        o[sl] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float m = -CUDART_INF_F, l = 0.f;
    for (int key = warp; key < keys; key += 4) {
        const uint8_t *rec = paged_tile<T>(p.v, b, h, key >> 4);
        if (!rec) {
            if (lane == 0) paged_error(p.v);
            continue;
        }
        float dot = 0.f;
#pragma unroll
        for (int sl = 0; sl < NS; ++sl) {
            const float4 k = dequantize4<KT, false>(rec + sl * code_tile_bytes(KT), rec + T::OFF_KS + sl * scale_tile_bytes(KT), key & 15, lane);
            dot += q[sl].x * k.x + q[sl].y * k.y + q[sl].z * k.z + q[sl].w * k.w;
        }
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, i);
        dot *= p.scale;
        const float mn = fmaxf(m, dot);
        const float a = m == -CUDART_INF_F ? 0.f : expf(m - mn);
        const float w = mn == -CUDART_INF_F ? 0.f : expf(dot - mn);
        l = l * a + w;
        m = mn;
#pragma unroll
        for (int sl = 0; sl < NS; ++sl) {
            const float4 v = dequantize4<VT, true>(rec + T::OFF_V + sl * code_tile_bytes(VT), rec + T::OFF_VS + sl * scale_tile_bytes(VT), key & 15, lane);
            o[sl] = make_float4(o[sl].x * a + w * v.x, o[sl].y * a + w * v.y, o[sl].z * a + w * v.z, o[sl].w * a + w * v.w);
        }
    }
#pragma unroll
    for (int sl = 0; sl < NS; ++sl) *reinterpret_cast<float4 *>(&s_o[warp][sl * kSlice + 4 * lane]) = o[sl];
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
    __syncthreads();
    const float M = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
    float w[4], L = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = s_m[i] == -CUDART_INF_F ? 0.f : expf(s_m[i] - M);
        L += w[i] * s_l[i];
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    const size_t row = (static_cast<size_t>(token) * p.Hq + hq) * T::D;
    if (threadIdx.x < T::D / 4) {
        float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 x = *reinterpret_cast<const float4 *>(&s_o[i][4 * threadIdx.x]);
            r = make_float4(r.x + w[i] * x.x, r.y + w[i] * x.y, r.z + w[i] * x.z, r.w + w[i] * x.w);
        }
        Act<DT>::store4(static_cast<X *>(p.out) + row + 4 * threadIdx.x, make_float4(r.x * inv, r.y * inv, r.z * inv, r.w * inv));
    }
    if (threadIdx.x == 0 && p.lse) p.lse[static_cast<size_t>(token) * p.Hq + hq] = L > 0.f ? M + logf(L) : -CUDART_INF_F;
}

template <int KT, int VT, int NS, int DT>
cudaError_t attn_t(const PagedAttnParams &p, cudaStream_t s) {
    paged_attn_rows<KT, VT, NS, DT><<<dim3(p.v.n_tokens, p.Hq), 128, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_attention(int type_k, int type_v, int D, int dtype, const PagedAttnParams &p, cudaStream_t s) {
    if (p.v.max_q <= KVQ_MAX_VERIFY_QUERIES) {
        if (dtype == KVQ_DT_F32) return launch_paged_split_f32(type_k, type_v, D, p, s);
        if (dtype == KVQ_DT_F16) return launch_paged_split_f16(type_k, type_v, D, p, s);
        return launch_paged_split_bf16(type_k, type_v, D, p, s);
    }
    KVQ_PAGED_DISPATCH(attn_t, (p, s))
}
cudaError_t paged_attention_workspace(int, int, int D, int, const PagedAttnParams &p, size_t *bytes) {
    if (p.v.max_q <= KVQ_MAX_VERIFY_QUERIES) return paged_split_workspace(D, bytes);
    *bytes = 16;
    return cudaSuccess;
}

}  // namespace kvq
