// kvq_paged_attn.cu -- attention over the paged cache: which kernel takes which sequences.
#include "kvq_paged.cuh"

namespace kvq {
namespace {

// Query rows (tokens x query heads per KV head) from which a sequence goes to the chunk kernel.
constexpr int kChunkMinRows = 33;

// Tokens from which a sequence goes to the chunk kernel.  fp32 queries stay with the split kernel, whose
// products keep their precision; a single sequence goes to one of the two by its bound alone.
int split_below(int dtype, const PagedAttnParams &p) {
    if (dtype == KVQ_DT_F32) return KVQ_MAX_VERIFY_QUERIES + 1;
    const int from = (kChunkMinRows + p.G - 1) / p.G > 2 ? (kChunkMinRows + p.G - 1) / p.G : 2;
    return p.v.n_seqs == 1 && p.v.max_q >= from ? 1 : from;
}

}  // namespace

cudaError_t launch_paged_attention(int type_k, int type_v, int D, int dtype, const PagedAttnParams &params, cudaStream_t s) {
    PagedAttnParams p = params;
    p.from_q = split_below(dtype, p);
    if (p.from_q > 1) {
        const cudaError_t e = dtype == KVQ_DT_F32   ? launch_paged_split_f32(type_k, type_v, D, p, s)
                              : dtype == KVQ_DT_F16 ? launch_paged_split_f16(type_k, type_v, D, p, s)
                                                    : launch_paged_split_bf16(type_k, type_v, D, p, s);
        if (e != cudaSuccess || p.v.max_q < p.from_q) return e;
    }
    return dtype == KVQ_DT_F16 ? launch_paged_chunk_f16(type_k, type_v, D, p, s) : launch_paged_chunk_bf16(type_k, type_v, D, p, s);
}

cudaError_t paged_attention_workspace(int, int, int D, int dtype, const PagedAttnParams &params, size_t *bytes) {
    PagedAttnParams p = params;
    p.from_q = split_below(dtype, p);
    // the two kernels of a mixed call run one after the other and share it
    size_t split = 0, chunk = 0;
    cudaError_t e = p.from_q > 1 ? paged_split_workspace(D, &split) : cudaSuccess;
    if (e == cudaSuccess && p.v.max_q >= p.from_q) e = paged_chunk_workspace(D, p, &chunk);
    *bytes = split > chunk ? split : chunk;
    return e;
}

}  // namespace kvq
