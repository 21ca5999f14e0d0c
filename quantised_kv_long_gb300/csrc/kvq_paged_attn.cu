// kvq_paged_attn.cu -- attention over the paged cache: which kernel takes which sequences.
#include "kvq_paged.cuh"

namespace kvq {
namespace {

// Query rows (tokens x query heads per KV head) from which a sequence goes to the chunk kernel.
constexpr int kChunkMinRows = 33;

// Tokens from which a sequence goes to the chunk kernel.  fp32 queries stay with the split kernel,
// whose products keep their precision.
int split_below(int dtype, const PagedAttnParams &p) {
    if (dtype == KVQ_DT_F32) return KVQ_MAX_VERIFY_QUERIES + 1;
    return (kChunkMinRows + p.G - 1) / p.G > 2 ? (kChunkMinRows + p.G - 1) / p.G : 2;
}

}  // namespace

cudaError_t launch_paged_attention(int type_k, int type_v, int D, int dtype, const PagedAttnParams &params, cudaStream_t s) {
    PagedAttnParams p = params;
    p.split_below = split_below(dtype, p);
    const bool chunks = p.v.max_q >= p.split_below;
    if (chunks && p.v.n_seqs == 1) p.split_below = 1;  // one launch pair takes the sequence, however few its tokens
    if (p.split_below > 1) {
        const cudaError_t e = dtype == KVQ_DT_F32   ? launch_paged_split_f32(type_k, type_v, D, p, s)
                              : dtype == KVQ_DT_F16 ? launch_paged_split_f16(type_k, type_v, D, p, s)
                                                    : launch_paged_split_bf16(type_k, type_v, D, p, s);
        if (e != cudaSuccess || !chunks) return e;
    }
    return dtype == KVQ_DT_F16 ? launch_paged_chunk_f16(type_k, type_v, D, p, s) : launch_paged_chunk_bf16(type_k, type_v, D, p, s);
}

cudaError_t paged_attention_workspace(int, int, int D, int dtype, const PagedAttnParams &p, size_t *bytes) {
    // the two kernels of a mixed call run one after the other and share it
    size_t split = 0, chunk = 0;
    cudaError_t e = paged_split_workspace(D, &split);
    if (e == cudaSuccess && p.v.max_q >= split_below(dtype, p)) e = paged_chunk_workspace(D, &chunk);
    *bytes = split > chunk ? split : chunk;
    return e;
}

}  // namespace kvq
