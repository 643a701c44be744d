// kvq_paged_attn_q4.cu -- the paged attention kernels for q4_0 V.
#include "kvq_paged_attn.cuh"

namespace kvq {

KVQ_DEFINE_PAGED_ENTRY(q4, KVQ_V_Q4_0)

cudaError_t launch_paged_lose(const PagedAttnParams &p, int n_ctas, cudaStream_t s, bool pdl)
{
    using C = PagedCfg<1, KVQ_V_Q4_0, KVQ_K_I8>;
    const cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<1, KVQ_V_Q4_0, KVQ_K_I8, false, true>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    return e != cudaSuccess ? e : launch_paged_t<1, KVQ_V_Q4_0, KVQ_K_I8, false, true>(p, n_ctas, s, pdl);
}

}  // namespace kvq
