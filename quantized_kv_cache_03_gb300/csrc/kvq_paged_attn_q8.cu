// kvq_paged_attn_q8.cu -- the paged attention kernels for q8_0 V.
#include "kvq_paged_attn.cuh"

namespace kvq {

KVQ_DEFINE_PAGED_ENTRY(q8, KVQ_V_Q8_0)

}  // namespace kvq
