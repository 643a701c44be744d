// kvq_paged_chunk_q8.cu -- the chunk attention kernel for q8_0 V.
#include "kvq_paged_chunk.cuh"

namespace kvq {

cudaError_t prepare_chunk_q8() { return prepare_chunk_t<KVQ_V_Q8_0>(); }
cudaError_t launch_chunk_q8(const PagedAttnParams &p, int out_type, int n_ctas, cudaStream_t s, bool pdl)
{
    return launch_chunk_t<KVQ_V_Q8_0>(p, out_type, n_ctas, s, pdl);
}

}  // namespace kvq
