// kvq_paged_attn_q4.cu -- the paged attention kernels for q4_0 V.
#include "kvq_paged_attn.cuh"

namespace kvq {

KVQ_DEFINE_PAGED_ENTRY(q4, KVQ_V_Q4_0)

}  // namespace kvq
