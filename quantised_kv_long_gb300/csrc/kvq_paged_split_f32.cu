// kvq_paged_split_f32.cu -- paged attention of few queries per sequence, f32 activations.
#include "kvq_paged_split.cuh"

namespace kvq {

cudaError_t launch_paged_split_f32(int type_k, int type_v, int D, const PagedAttnParams &p, cudaStream_t s) {
    return launch_split_dt<KVQ_DT_F32>(type_k, type_v, D, p, s);
}

cudaError_t paged_split_workspace(int D, const PagedAttnParams &p, size_t *bytes) {
    if (split_seq_steps(p) > kPagedMaxSteps) return cudaErrorNotSupported;
    int dev = 0, sms = 0;
    const cudaError_t e = paged_device(&dev, &sms);
    if (e != cudaSuccess) return e;
    *bytes = split_work_bytes(2 * kSplitMaxWarps * sms, D);
    return cudaSuccess;
}

}  // namespace kvq
