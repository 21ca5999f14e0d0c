// kvq_paged_attn.cu -- attention over the paged cache: which kernel takes which sequences.
#include "kvq_paged.cuh"

namespace kvq {
namespace {

// Query rows (tokens x query heads per KV head) from which a sequence goes to the chunk kernel.  The split kernel
// reads a sequence once per eight rows, the chunk kernel costs the same up to 128 rows; per call, us, split / chunk,
// over 16 sequences of 8192 positions: q4_0 128-wide 139 / 239 at 32 rows, 202 / 241 at 48, 264 / 241 at 64;
// q8_0/q4_0 256-wide 137 / 257, 199 / 260, 272 / 262; f16 128-wide, whose reads are the bound, 237 / 315 at 24 rows,
// 311 / 315 at 32, 461 / 318 at 48.
int chunk_min_rows(int type_k) { return type_k == KVQ_F16 ? 33 : 57; }

// Tokens from which a sequence goes to the chunk kernel.  fp32 queries stay with the split kernel, whose
// products keep their precision; a single sequence goes to one of the two by its bound alone.
int split_below(int type_k, int dtype, const PagedAttnParams &p) {
    if (dtype == KVQ_DT_F32) return KVQ_MAX_VERIFY_QUERIES + 1;
    const int from = (chunk_min_rows(type_k) + p.G - 1) / p.G > 2 ? (chunk_min_rows(type_k) + p.G - 1) / p.G : 2;
    return p.v.n_seqs == 1 && p.v.max_q >= from ? 1 : from;
}

}  // namespace

cudaError_t launch_paged_attention(int type_k, int type_v, int D, int dtype, const PagedAttnParams &params, cudaStream_t s) {
    PagedAttnParams p = params;
    p.from_q = split_below(type_k, dtype, p);
    if (p.from_q > 1) {
        const cudaError_t e = dtype == KVQ_DT_F32   ? launch_paged_split_f32(type_k, type_v, D, p, s)
                              : dtype == KVQ_DT_F16 ? launch_paged_split_f16(type_k, type_v, D, p, s)
                                                    : launch_paged_split_bf16(type_k, type_v, D, p, s);
        if (e != cudaSuccess || p.v.max_q < p.from_q) return e;
    }
    return dtype == KVQ_DT_F16 ? launch_paged_chunk_f16(type_k, type_v, D, p, s) : launch_paged_chunk_bf16(type_k, type_v, D, p, s);
}

cudaError_t paged_attention_workspace(int type_k, int, int D, int dtype, const PagedAttnParams &params, size_t *bytes) {
    PagedAttnParams p = params;
    p.from_q = split_below(type_k, dtype, p);
    // the two kernels of a mixed call run one after the other and share it
    size_t split = 0, chunk = 0;
    cudaError_t e = p.from_q > 1 ? paged_split_workspace(D, p, &split) : cudaSuccess;
    if (e == cudaSuccess && p.v.max_q >= p.from_q) e = paged_chunk_workspace(type_k, D, dtype, p, &chunk);
    *bytes = split > chunk ? split : chunk;
    return e;
}

}  // namespace kvq
