// kvq_paged_chunk_q4.cu -- the chunk attention kernel for q4_0 V.
#include "kvq_paged_chunk.cuh"

namespace kvq {

cudaError_t prepare_chunk_q4() { return prepare_chunk_t<KVQ_V_Q4_0>(); }
cudaError_t launch_chunk_q4(const PagedAttnParams &p, int out_type, int n_ctas, cudaStream_t s, bool pdl)
{
    return launch_chunk_t<KVQ_V_Q4_0>(p, out_type, n_ctas, s, pdl);
}
cudaError_t launch_chunk_lose(const PagedAttnParams &p, int n_ctas, cudaStream_t s, bool pdl)
{
    const cudaError_t e = cudaFuncSetAttribute(paged_chunk_kernel<KVQ_V_Q4_0, false, true>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkCfg<KVQ_V_Q4_0>::SMEM);
    return e != cudaSuccess ? e : launch_chunk_t<KVQ_V_Q4_0, true>(p, KVQ_OUT_F32, n_ctas, s, pdl);
}

}  // namespace kvq
