// kvq_paged_chunk_f16.cu -- paged attention of many queries per sequence, f16 activations.
#include "kvq_paged_chunk.cuh"

namespace kvq {

cudaError_t launch_paged_chunk_f16(int type_k, int type_v, int D, const PagedAttnParams &p, cudaStream_t s) {
    return launch_chunk_dt<KVQ_DT_F16>(type_k, type_v, D, p, s);
}

cudaError_t paged_chunk_workspace(int type_k, int D, int dtype, const PagedAttnParams &p, size_t *bytes) {
    int dev = 0, sms = 0;
    const cudaError_t e = paged_device(&dev, &sms);
    if (e != cudaSuccess) return e;
    const int rows = D == kSlice ? ChunkCfg<KVQ_F16, KVQ_F16, 1, true, false>::ROWS : ChunkCfg<KVQ_F16, KVQ_F16, 2, true, false>::ROWS;
    if (chunk_seq_steps(p, rows) > kPagedMaxSteps) return cudaErrorNotSupported;
    (void)chunk_work(p, sms, rows, D, type_k != KVQ_F16 && dtype == KVQ_DT_F16, bytes);
    return cudaSuccess;
}

}  // namespace kvq
