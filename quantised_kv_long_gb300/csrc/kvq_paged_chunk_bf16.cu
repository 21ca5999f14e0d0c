// kvq_paged_chunk_bf16.cu -- paged attention of many queries per sequence, bf16 activations.
#include "kvq_paged_chunk.cuh"

namespace kvq {

cudaError_t launch_paged_chunk_bf16(int type_k, int type_v, int D, const PagedAttnParams &p, cudaStream_t s) {
    return launch_chunk_dt<KVQ_DT_BF16>(type_k, type_v, D, p, s);
}

}  // namespace kvq
