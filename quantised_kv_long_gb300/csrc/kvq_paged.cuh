// kvq_paged.cuh -- what the kernels of the paged cache share: tile records, the batch
// description on the device, activation types, and the launch entry points.
#pragma once

#include <cuda_bf16.h>

#include "kvq_internal.cuh"

namespace kvq {

// The pool, and the sequences of one call (include/kvq.h, kvq_paged_batch).
struct PagedView {
    uint8_t *pool;
    int32_t *err;
    const int32_t *cu_q, *lens, *table;
    int n_seqs, n_tokens, max_q, max_len, width, stride;
    int n_pages, page_tiles, Hkv;
    int token0;  // without cu_q: the token of sequence 0
};

// One tile record: 16 rows of one KV head.  A record holds K and V together so that one bulk
// copy (or one run of 16-byte loads) fetches all of it, whatever page it lies in; the
// contiguous cache's four separate planes would make four copies of it, two of them of 128
// bytes.  Every size is a multiple of 128 bytes.
template <int KT, int VT, int NS>
struct PagedTile {
    static constexpr int KC = code_tile_bytes(KT) * NS, VC = code_tile_bytes(VT) * NS;
    static constexpr int KS = scale_tile_bytes(KT) * NS, VS = scale_tile_bytes(VT) * NS;
    static constexpr int OFF_V = KC, OFF_KS = KC + VC, OFF_VS = KC + VC + KS;
    static constexpr int BYTES = KC + VC + KS + VS;
    static constexpr int D = NS * kSlice;
};

__device__ __forceinline__ void paged_error(const PagedView &v) { atomicOr(v.err, KVQ_DEVERR_BATCH); }

// Sequence b of the batch: its tokens [first, first + n) are positions [len - n, len).
struct PagedSeq {
    int first, n, len;
    bool ok;
};
__device__ __forceinline__ PagedSeq paged_seq(const PagedView &v, int b) {
    PagedSeq s;
    s.first = v.cu_q ? __ldg(v.cu_q + b) : v.token0 + b;
    // the difference in 64 bits: entries may be any integers
    const long long n = v.cu_q ? static_cast<long long>(__ldg(v.cu_q + b + 1)) - s.first : 1;
    s.len = __ldg(v.lens + b);
    s.ok = n >= 0 && n <= v.max_q && s.first >= 0 && s.first + n <= v.n_tokens && s.len >= 0 && s.len <= v.max_len;
    s.n = s.ok ? static_cast<int>(n) : 0;
    if (!s.ok) s.len = 0;
    return s;
}

// The sequence that holds a packed token, or -1 (padding); called by a whole warp.  Each round
// narrows the range 32 times, so up to 1024 sequences take two dependent loads.
__device__ __forceinline__ int paged_find(const PagedView &v, int token) {
    if (!v.cu_q) return token < v.n_seqs ? token : -1;
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = v.n_seqs + 1;  // the last entry is the end of the last sequence
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5;
        const int i = lo + lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, i < hi && __ldg(v.cu_q + i) <= token);
        const int k = __popc(below);
        if (k == 0) return -1;
        lo += (k - 1) * step;
        hi = min(hi, lo + step);
    }
    return lo < v.n_seqs && __ldg(v.cu_q + lo) <= token ? lo : -1;
}

// The record of tile t (positions 16 t ..) of sequence b's KV head h; nullptr when its page
// number is outside the pool.  t * 16 < max_len <= width * page_size.
template <class T>
__device__ __forceinline__ uint8_t *paged_tile(const PagedView &v, int b, int h, int t) {
    const int page = __ldg(v.table + static_cast<size_t>(b) * v.stride + t / v.page_tiles);
    if (page < 0 || page >= v.n_pages) return nullptr;
    return v.pool + ((static_cast<size_t>(page) * v.Hkv + h) * v.page_tiles + t % v.page_tiles) * T::BYTES;
}

// Bounded wait for a barrier phase: false after about two seconds.  The hardware holds the warp for up
// to 20 us per try, so that a waiting warp takes few issue slots from the working ones.
__device__ __forceinline__ bool paged_try(uint32_t addr, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok)
                 : "r"(addr), "r"(parity)
                 : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool paged_wait(uint64_t *bar, uint32_t parity) {
    const uint32_t addr = smem_u32(bar);
    if (paged_try(addr, parity)) return true;
    const long long t0 = clock64();
    while (!paged_try(addr, parity))
        if (clock64() - t0 > kWaitCycles) return false;
    return true;
}

// At the head of a rarely taken branch: keeps the compiler from turning the branch into selects that every
// pass would execute.
__device__ __forceinline__ void keep_branch() { asm volatile("" ::: "memory"); }

// ---- activations: fp32, f16, bf16 ----
template <int DT>
struct Act;
template <>
struct Act<KVQ_DT_F32> {
    using type = float;
    static __device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
    static __device__ __forceinline__ void store4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }
    static __device__ __forceinline__ void store2(float *p, float a, float b) { *reinterpret_cast<float2 *>(p) = make_float2(a, b); }
};
template <>
struct Act<KVQ_DT_F16> {
    using type = __half;
    static __device__ __forceinline__ float4 load4(const __half *p) { return widen(*reinterpret_cast<const uint2 *>(p)); }
    static __device__ __forceinline__ float4 widen(uint2 w) {  // four values, as loaded
        const float2 a = __half22float2(u32_as_h2(w.x)), b = __half22float2(u32_as_h2(w.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
    static __device__ __forceinline__ void store4(__half *p, float4 x) {
        *reinterpret_cast<uint2 *>(p) =
            make_uint2(h2_as_u32(__floats2half2_rn(x.x, x.y)), h2_as_u32(__floats2half2_rn(x.z, x.w)));
    }
    static __device__ __forceinline__ void store2(__half *p, float a, float b) {
        *reinterpret_cast<uint32_t *>(p) = h2_as_u32(__floats2half2_rn(a, b));
    }
};
template <>
struct Act<KVQ_DT_BF16> {
    using type = __nv_bfloat16;
    static __device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) { return widen(*reinterpret_cast<const uint2 *>(p)); }
    static __device__ __forceinline__ float4 widen(uint2 w) {  // a bf16 is the upper half of an fp32
        return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                           __uint_as_float(w.y & 0xffff0000u));
    }
    static __device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 x) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
        *reinterpret_cast<uint2 *>(p) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
    static __device__ __forceinline__ void store2(__nv_bfloat16 *p, float a, float b) {
        *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(a, b);
    }
};

// Values 4l .. 4l + 3 of row kt of a tile slice (the inverse of quantize_store_vals).
template <int T, bool IS_V>
__device__ __forceinline__ float4 dequantize4(const uint8_t *codes, const uint8_t *scales, int kt, int lane) {
    if constexpr (T == KVQ_F16) {
        return load_f16_row<IS_V>(codes, kt, lane);
    } else {
        const int b = lane >> 3, i0 = (4 * lane) & 31, n = kt & 7, st = kt >> 3;
        int j, pos;
        pair_slot(kt, j, pos);
        const float d = __half2float(*reinterpret_cast<const __half *>(scales + j * 32 + b * 8 + pos * 2));
        uint32_t byte[4];
        if constexpr (T == KVQ_Q8_0) {
            if constexpr (!IS_V) {
                const int jd = (i0 & 15) >> 2, hd = i0 >> 4;
                const uint32_t w = *reinterpret_cast<const uint32_t *>(codes + b * 512 + (4 * n + jd) * 16 + (2 * st + hd) * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) byte[e] = (w >> (8 * e)) & 0xffu;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = i0 + e, r = i & 15, hv = i >> 4, n2 = r >> 1;
                    byte[e] = codes[b * 512 + (4 * n2 + j) * 16 + ((r & 1) + 2 * hv) * 4 + vword_byte(pos)];
                }
            }
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // sign and magnitude
                const float m = static_cast<float>(byte[e] & 0x7fu);
                x[e] = d * ((byte[e] & 0x80u) ? -m : m);
            }
            return make_float4(x[0], x[1], x[2], x[3]);
        } else {
            const int shift = i0 >= 16 ? 4 : 0;
            if constexpr (!IS_V) {
                const int jb = (i0 & 15) >> 2;
                const uint32_t w =
                    *reinterpret_cast<const uint32_t *>(codes + (b >> 1) * 512 + (4 * n + jb) * 16 + (2 * (b & 1) + st) * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) byte[e] = (w >> (8 * e)) & 0xffu;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = (i0 & 15) + e, n2 = r >> 1;
                    byte[e] = codes[(b >> 1) * 512 + (4 * n2 + j) * 16 + (2 * (b & 1) + (r & 1)) * 4 + vword_byte(pos)];
                }
            }
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = d * (static_cast<float>((byte[e] >> shift) & 15u) - 8.0f);
            return make_float4(x[0], x[1], x[2], x[3]);
        }
    }
}

// ---- launch parameters ----
struct PagedAppendParams {
    PagedView v;
    const void *k, *v_in, *q;
    void *q_out;
    long long k_stride, v_stride, q_stride, q_out_stride;
    const float *cos_sin;      // nullptr: no rotation
    const int32_t *positions;  // nullptr: the position in the sequence
    int n_positions, rot_dim, interleaved, Hq;
};
struct PagedGatherParams {
    PagedView v;
    void *k_out, *v_out;
};
struct PagedAttnParams {
    PagedView v;
    const void *q;
    void *out;
    float *lse;  // or nullptr
    long long q_stride;
    int Hq, G;
    float scale;
    void *workspace;
    // sequences with fewer tokens than this belong to the split kernel, the others to the chunk kernel
    int from_q;
};

cudaError_t launch_paged_append(int type_k, int type_v, int D, int dtype, const PagedAppendParams &p, cudaStream_t s);
cudaError_t launch_paged_gather(int type_k, int type_v, int D, int dtype, const PagedGatherParams &p, cudaStream_t s);
cudaError_t launch_paged_attention(int type_k, int type_v, int D, int dtype, const PagedAttnParams &p, cudaStream_t s);
// workspace bytes of a call, from sizes known on the host; cudaErrorNotSupported past kPagedMaxSteps
cudaError_t paged_attention_workspace(int type_k, int type_v, int D, int dtype, const PagedAttnParams &p, size_t *bytes);
// few queries per sequence (kvq_paged_split.cuh), one translation unit per activation type
cudaError_t launch_paged_split_f32(int type_k, int type_v, int D, const PagedAttnParams &p, cudaStream_t s);
cudaError_t launch_paged_split_f16(int type_k, int type_v, int D, const PagedAttnParams &p, cudaStream_t s);
cudaError_t launch_paged_split_bf16(int type_k, int type_v, int D, const PagedAttnParams &p, cudaStream_t s);
cudaError_t paged_split_workspace(int D, const PagedAttnParams &p, size_t *bytes);
// many queries per sequence (kvq_paged_chunk.cuh)
cudaError_t launch_paged_chunk_f16(int type_k, int type_v, int D, const PagedAttnParams &p, cudaStream_t s);
cudaError_t launch_paged_chunk_bf16(int type_k, int type_v, int D, const PagedAttnParams &p, cudaStream_t s);
cudaError_t paged_chunk_workspace(int type_k, int D, int dtype, const PagedAttnParams &p, size_t *bytes);

// ---- what the attention launches share ----
constexpr int kPagedMaxDevices = 64;
// the current device and its SMs (looked up once per device)
inline cudaError_t paged_device(int *dev, int *sms) {
    static int cached[kPagedMaxDevices] = {};
    cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess) return e;
    if (*dev < 0 || *dev >= kPagedMaxDevices) return cudaErrorInvalidDevice;
    if (cached[*dev] == 0) {
        int n = 0;
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, *dev);
        if (e != cudaSuccess) return e;
        cached[*dev] = n > 0 ? n : 1;
    }
    *sms = cached[*dev];
    return cudaSuccess;
}
// Steps of one sequence, over all KV heads, that the attention kernels can count: their sums over a launch are
// 32-bit.  A call whose sizes allow more is refused.
constexpr long long kPagedMaxSteps = 1ll << 30;
// most steps of a sequence: `blocks` of keys times units of `unit` rows; at least 1, at most kPagedMaxSteps + 1
inline long long paged_steps(long long blocks, long long rows, int unit, int Hkv) {
    const __int128 n = static_cast<__int128>(blocks) * ((rows + unit - 1) / unit) * Hkv;
    return n > kPagedMaxSteps ? kPagedMaxSteps + 1 : (n > 1 ? static_cast<long long>(n) : 1);
}
// sequences b .. b + most - 1 of a call
inline PagedAttnParams paged_some(const PagedAttnParams &p, int b, int most) {
    PagedAttnParams q = p;
    q.v.n_seqs = p.v.n_seqs - b < most ? p.v.n_seqs - b : most;
    q.v.lens += b;
    q.v.table += static_cast<size_t>(b) * p.v.stride;
    if (p.v.cu_q)
        q.v.cu_q += b;
    else
        q.v.token0 += b;
    return q;
}
// a launch that may start while the previous kernel of its stream finishes (every kernel launched so
// waits for it before it reads or writes anything)
template <class... A, class... B>
cudaError_t launch_dependent(void (*kernel)(A...), dim3 grid, int threads, int smem, cudaStream_t s, B... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// (K, V) type pairs of the paged cache
constexpr bool is_paged_pair(int tk, int tv) {
    return (tk == KVQ_F16 && tv == KVQ_F16) || (tk == KVQ_Q8_0 && tv == KVQ_Q8_0) ||
           (tk == KVQ_Q8_0 && tv == KVQ_Q4_0) || (tk == KVQ_Q4_0 && tv == KVQ_Q4_0);
}

}  // namespace kvq

// CALL<KT, VT, NS, DT>(args) for the instance of (type_k, type_v, D, dtype)
#define KVQ_PAGED_DT(KT_, VT_, NS_, CALL, ARGS)                                         \
    if (type_k == KT_ && type_v == VT_ && D == NS_ * kSlice) {                          \
        if (dtype == KVQ_DT_F32) return CALL<KT_, VT_, NS_, KVQ_DT_F32> ARGS;           \
        if (dtype == KVQ_DT_F16) return CALL<KT_, VT_, NS_, KVQ_DT_F16> ARGS;           \
        if (dtype == KVQ_DT_BF16) return CALL<KT_, VT_, NS_, KVQ_DT_BF16> ARGS;         \
    }
#define KVQ_PAGED_DISPATCH(CALL, ARGS)                 \
    KVQ_PAGED_DT(KVQ_F16, KVQ_F16, 1, CALL, ARGS)      \
    KVQ_PAGED_DT(KVQ_F16, KVQ_F16, 2, CALL, ARGS)      \
    KVQ_PAGED_DT(KVQ_Q8_0, KVQ_Q8_0, 1, CALL, ARGS)    \
    KVQ_PAGED_DT(KVQ_Q8_0, KVQ_Q8_0, 2, CALL, ARGS)    \
    KVQ_PAGED_DT(KVQ_Q8_0, KVQ_Q4_0, 1, CALL, ARGS)    \
    KVQ_PAGED_DT(KVQ_Q8_0, KVQ_Q4_0, 2, CALL, ARGS)    \
    KVQ_PAGED_DT(KVQ_Q4_0, KVQ_Q4_0, 1, CALL, ARGS)    \
    KVQ_PAGED_DT(KVQ_Q4_0, KVQ_Q4_0, 2, CALL, ARGS)    \
    return cudaErrorInvalidValue;
