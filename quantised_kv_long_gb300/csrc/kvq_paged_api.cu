// kvq_paged_api.cu -- the paged cache's part of the C ABI (include/kvq.h): argument checks, the
// host handle and the launches.  No device memory is allocated here.
#include <new>

#include "kvq_paged.cuh"

struct kvq_paged {
    kvq_paged_desc desc;
    uint8_t *pool;
    int32_t *state;  // [error word][pad]
    int device;
};

namespace {

constexpr size_t kPagedStateBytes = 16;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

kvq_status check_desc(const kvq_paged_desc *d, size_t *pool_bytes) {
    if (!d) return KVQ_ERR_INVALID_ARG;
    if (d->n_pages < 1 || d->n_kv_heads < 1 || d->page_size < 1 || d->page_size % kvq::kTileRows != 0)
        return KVQ_ERR_INVALID_ARG;
    if (!kvq::is_paged_pair(d->type_k, d->type_v)) return KVQ_ERR_UNSUPPORTED;
    if (d->head_dim != 128 && d->head_dim != 256) return KVQ_ERR_UNSUPPORTED;
    const unsigned long long record =
        static_cast<unsigned long long>(d->head_dim / kvq::kSlice) *
        (kvq::code_tile_bytes(d->type_k) + kvq::code_tile_bytes(d->type_v) + kvq::scale_tile_bytes(d->type_k) +
         kvq::scale_tile_bytes(d->type_v));
    // n_kv_heads * tiles of a page fit 63 bits, times the pages and the record in 128
    const unsigned __int128 bytes = static_cast<unsigned __int128>(static_cast<unsigned long long>(d->n_kv_heads) *
                                                                   static_cast<unsigned long long>(d->page_size / kvq::kTileRows)) *
                                    static_cast<unsigned long long>(d->n_pages) * record;
    if (bytes > static_cast<unsigned __int128>(~0ull >> 1)) return KVQ_ERR_INVALID_ARG;
    *pool_bytes = static_cast<size_t>(bytes);
    return KVQ_OK;
}

// The host's part of a batch; KVQ_OK with n_seqs or n_tokens 0 is a call that does nothing.
kvq_status check_batch(const kvq_paged *c, const kvq_paged_batch *b, kvq::PagedView *v) {
    if (!c || !b) return KVQ_ERR_INVALID_ARG;
    if (b->n_seqs < 0 || b->n_tokens < 0) return KVQ_ERR_INVALID_ARG;
    if (b->n_seqs == 0 || b->n_tokens == 0) return KVQ_OK;
    if (b->max_q < 1 || b->max_len < 0 || b->table_width < 1 || b->table_stride < b->table_width) return KVQ_ERR_INVALID_ARG;
    if (b->max_len > static_cast<long long>(b->table_width) * c->desc.page_size) return KVQ_ERR_INVALID_ARG;
    if (b->max_len > INT32_MAX - 1024) return KVQ_ERR_UNSUPPORTED;  // the kernels round lengths up to blocks in 32 bits
    if (!b->lens || !b->block_table) return KVQ_ERR_INVALID_ARG;
    if (!b->cu_q && b->n_tokens < b->n_seqs) return KVQ_ERR_INVALID_ARG;
    if (!aligned4(b->lens) || !aligned4(b->block_table) || !aligned4(b->cu_q)) return KVQ_ERR_ALIGNMENT;
    v->pool = c->pool;
    v->err = c->state;
    v->cu_q = b->cu_q;
    v->lens = b->lens;
    v->table = b->block_table;
    v->n_seqs = b->n_seqs;
    v->n_tokens = b->n_tokens;
    v->max_q = b->cu_q ? (b->max_q < b->n_tokens ? b->max_q : b->n_tokens) : 1;
    v->max_len = b->max_len;
    v->width = b->table_width;
    v->stride = b->table_stride;
    v->n_pages = c->desc.n_pages;
    v->page_tiles = c->desc.page_size / kvq::kTileRows;
    v->Hkv = c->desc.n_kv_heads;
    return KVQ_OK;
}

bool valid_dtype(int dt) { return dt == KVQ_DT_F32 || dt == KVQ_DT_F16 || dt == KVQ_DT_BF16; }
kvq_status check_rows(const void *p, int64_t stride, int64_t heads, int64_t dim) {
    if (!p || stride < heads * dim) return KVQ_ERR_INVALID_ARG;
    if (!aligned16(p) || stride % 8 != 0) return KVQ_ERR_ALIGNMENT;
    return KVQ_OK;
}

// The handle's memory belongs to one device, which has to be current.
kvq_status check_device(const kvq_paged *c) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return KVQ_ERR_CUDA;
    return dev == c->device ? KVQ_OK : KVQ_ERR_INVALID_ARG;
}

#define KVQ_TRY(x)                          \
    do {                                    \
        const kvq_status st_ = (x);         \
        if (st_ != KVQ_OK) return st_;      \
    } while (0)

kvq_status attention_params(const kvq_paged *c, const kvq_paged_batch *b, int32_t n_q_heads, kvq_dtype dtype,
                            kvq::PagedAttnParams *p) {
    KVQ_TRY(check_batch(c, b, &p->v));
    if (!valid_dtype(dtype)) return KVQ_ERR_UNSUPPORTED;
    if (n_q_heads < 1 || n_q_heads % c->desc.n_kv_heads != 0) return KVQ_ERR_INVALID_ARG;
    if (n_q_heads > 65535) return KVQ_ERR_UNSUPPORTED;
    if (dtype == KVQ_DT_F32 && p->v.max_q > KVQ_MAX_VERIFY_QUERIES) return KVQ_ERR_UNSUPPORTED;
    p->Hq = n_q_heads;
    p->G = n_q_heads / c->desc.n_kv_heads;
    return KVQ_OK;
}

kvq_status workspace_of(const kvq_paged *c, kvq_dtype dtype, const kvq::PagedAttnParams &p, size_t *bytes) {
    const cudaError_t e = kvq::paged_attention_workspace(c->desc.type_k, c->desc.type_v, c->desc.head_dim, dtype, p, bytes);
    return e == cudaSuccess ? KVQ_OK : e == cudaErrorNotSupported ? KVQ_ERR_UNSUPPORTED : KVQ_ERR_CUDA;
}

}  // namespace

extern "C" {

kvq_status kvq_paged_size(const kvq_paged_desc *desc, size_t *pool_bytes, size_t *state_bytes) {
    size_t bytes = 0;
    KVQ_TRY(check_desc(desc, &bytes));
    if (!pool_bytes || !state_bytes) return KVQ_ERR_INVALID_ARG;
    *pool_bytes = bytes;
    *state_bytes = kPagedStateBytes;
    return KVQ_OK;
}

kvq_status kvq_paged_create(const kvq_paged_desc *desc, void *pool, void *state, kvq_paged **out) {
    size_t bytes = 0;
    KVQ_TRY(check_desc(desc, &bytes));
    if (!pool || !state || !out) return KVQ_ERR_INVALID_ARG;
    if (!aligned16(pool) || !aligned16(state)) return KVQ_ERR_ALIGNMENT;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return KVQ_ERR_CUDA;
    kvq_paged *c = new (std::nothrow) kvq_paged;
    if (!c) return KVQ_ERR_INVALID_ARG;
    c->desc = *desc;
    c->pool = static_cast<uint8_t *>(pool);
    c->state = static_cast<int32_t *>(state);
    c->device = dev;
    *out = c;
    return KVQ_OK;
}

kvq_status kvq_paged_destroy(kvq_paged *cache) {
    if (!cache) return KVQ_ERR_INVALID_ARG;
    delete cache;
    return KVQ_OK;
}

kvq_status kvq_paged_read_error(kvq_paged *cache, void *stream, int32_t *h_err) {
    if (!cache || !h_err) return KVQ_ERR_INVALID_ARG;
    KVQ_TRY(check_device(cache));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemcpyAsync(h_err, cache->state, sizeof(int32_t), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(cache->state, 0, sizeof(int32_t), s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_paged_append(kvq_paged *cache, const kvq_paged_batch *batch, const void *k, const void *v, kvq_dtype dtype,
                            int64_t k_stride, int64_t v_stride, const kvq_rope *rope, const void *q, int32_t n_q_heads,
                            int64_t q_stride, void *q_out, int64_t q_out_stride, void *stream) {
    kvq::PagedAppendParams p{};
    KVQ_TRY(check_batch(cache, batch, &p.v));
    if (!valid_dtype(dtype)) return KVQ_ERR_UNSUPPORTED;
    const int64_t D = cache->desc.head_dim;
    if (rope) {
        if (!rope->cos_sin || rope->n_positions < 1) return KVQ_ERR_INVALID_ARG;
        if (rope->rot_dim < 8 || rope->rot_dim % 8 != 0 || rope->rot_dim > D) return KVQ_ERR_INVALID_ARG;
        if (!aligned16(rope->cos_sin) || !aligned4(rope->positions)) return KVQ_ERR_ALIGNMENT;
        p.cos_sin = rope->cos_sin;
        p.positions = rope->positions;
        p.n_positions = rope->n_positions;
        p.rot_dim = rope->rot_dim;
        p.interleaved = rope->interleaved != 0;
    }
    if (q) {
        if (!rope || n_q_heads < 1 || n_q_heads % cache->desc.n_kv_heads != 0) return KVQ_ERR_INVALID_ARG;
        if (q_out == q && q_out_stride != q_stride) return KVQ_ERR_INVALID_ARG;
    }
    if (batch->n_seqs == 0 || batch->n_tokens == 0) return KVQ_OK;
    KVQ_TRY(check_rows(k, k_stride, cache->desc.n_kv_heads, D));
    KVQ_TRY(check_rows(v, v_stride, cache->desc.n_kv_heads, D));
    if (q) {
        KVQ_TRY(check_rows(q, q_stride, n_q_heads, D));
        KVQ_TRY(check_rows(q_out, q_out_stride, n_q_heads, D));
        p.q = q;
        p.q_out = q_out;
        p.q_stride = q_stride;
        p.q_out_stride = q_out_stride;
        p.Hq = n_q_heads;
    }
    KVQ_TRY(check_device(cache));
    p.k = k;
    p.v_in = v;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    return kvq::launch_paged_append(cache->desc.type_k, cache->desc.type_v, cache->desc.head_dim, dtype, p,
                                    static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KVQ_OK
               : KVQ_ERR_CUDA;
}

kvq_status kvq_paged_gather(const kvq_paged *cache, const kvq_paged_batch *batch, void *k_out, void *v_out, kvq_dtype dtype,
                            void *stream) {
    kvq::PagedGatherParams p{};
    KVQ_TRY(check_batch(cache, batch, &p.v));
    if (!valid_dtype(dtype)) return KVQ_ERR_UNSUPPORTED;
    if (batch->n_seqs == 0 || batch->n_tokens == 0) return KVQ_OK;
    if (!k_out || !v_out) return KVQ_ERR_INVALID_ARG;
    if (!aligned16(k_out) || !aligned16(v_out)) return KVQ_ERR_ALIGNMENT;
    KVQ_TRY(check_device(cache));
    p.k_out = k_out;
    p.v_out = v_out;
    return kvq::launch_paged_gather(cache->desc.type_k, cache->desc.type_v, cache->desc.head_dim, dtype, p,
                                    static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KVQ_OK
               : KVQ_ERR_CUDA;
}

kvq_status kvq_paged_attention_workspace_size(const kvq_paged *cache, const kvq_paged_batch *batch, int32_t n_q_heads,
                                              kvq_dtype dtype, size_t *bytes) {
    kvq::PagedAttnParams p{};
    KVQ_TRY(attention_params(cache, batch, n_q_heads, dtype, &p));
    if (!bytes) return KVQ_ERR_INVALID_ARG;
    *bytes = 16;
    if (batch->n_seqs == 0 || batch->n_tokens == 0) return KVQ_OK;
    KVQ_TRY(check_device(cache));
    return workspace_of(cache, dtype, p, bytes);
}

kvq_status kvq_paged_attention(const kvq_paged *cache, const kvq_paged_batch *batch, const void *q, kvq_dtype dtype,
                               int32_t n_q_heads, int64_t q_stride, float scale, void *workspace, size_t workspace_bytes,
                               void *out, float *lse, void *stream) {
    kvq::PagedAttnParams p{};
    KVQ_TRY(attention_params(cache, batch, n_q_heads, dtype, &p));
    if (batch->n_seqs == 0 || batch->n_tokens == 0) return KVQ_OK;
    KVQ_TRY(check_rows(q, q_stride, n_q_heads, cache->desc.head_dim));
    if (!out || !workspace) return KVQ_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(workspace) || !aligned4(lse)) return KVQ_ERR_ALIGNMENT;
    KVQ_TRY(check_device(cache));
    const int tk = cache->desc.type_k, tv = cache->desc.type_v, D = cache->desc.head_dim;
    size_t need = 0;
    KVQ_TRY(workspace_of(cache, dtype, p, &need));
    if (workspace_bytes < need) return KVQ_ERR_SCRATCH;
    p.q = q;
    p.out = out;
    p.lse = lse;
    p.q_stride = q_stride;
    p.scale = scale;
    p.workspace = workspace;
    return kvq::launch_paged_attention(tk, tv, D, dtype, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK
                                                                                                             : KVQ_ERR_CUDA;
}

}  // extern "C"
