// kvq_paged_split_bf16.cu -- paged attention of few queries per sequence, bf16 activations.
#include "kvq_paged_split.cuh"

namespace kvq {

cudaError_t launch_paged_split_bf16(int type_k, int type_v, int D, const PagedAttnParams &p, cudaStream_t s) {
    return launch_split_dt<KVQ_DT_BF16>(type_k, type_v, D, p, s);
}

}  // namespace kvq
