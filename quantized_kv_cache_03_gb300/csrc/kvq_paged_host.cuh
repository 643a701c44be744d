// kvq_paged_host.cuh -- argument checks that the paged cache's calls share
// (kvq_paged_api.cu, kvq_tokens_api.cu).
#pragma once

#include <climits>
#include <cstdlib>

#include "kvq_paged.cuh"

namespace kvq {

constexpr int kMaxDevices = 64;

inline bool pdl_on()
{
    const char *e = std::getenv("KVQ_PDL");
    return !(e && e[0] == '0');
}

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool int_ptr(const void *p) { return p && aligned(p, 4); }

inline kvq_status done(cudaError_t e)
{
    if (e == cudaSuccess) return KVQ_OK;
    cudaGetLastError();
    return KVQ_ERR_CUDA;
}

inline int page_shift(int tokens)
{
    for (int s = 4; s <= 8; ++s)
        if (tokens == 1 << s) return s;
    return -1;
}

// Shape of a pool (data aside).
inline kvq_status check_shape(const kvq_pages *p)
{
    if (!p || p->n_pages < 0 || page_shift(p->page_tokens) < 0) return KVQ_ERR_INVALID_ARG;
    if (p->n_kv_heads < 1 || p->n_kv_heads > KVQ_MAX_HEADS) return KVQ_ERR_INVALID_ARG;
    if ((p->v_type != KVQ_V_Q4_0 && p->v_type != KVQ_V_Q8_0) || (p->k_type != KVQ_K_I8 && p->k_type != KVQ_K_F16))
        return KVQ_ERR_INVALID_ARG;
    if (p->head_dim != KVQ_HEAD_DIM) return p->head_dim % KVQ_QBLOCK ? KVQ_ERR_INVALID_ARG : KVQ_ERR_UNSUPPORTED;
    if ((long long)p->n_pages * p->page_tokens > INT_MAX) return KVQ_ERR_INVALID_ARG;
    return KVQ_OK;
}

inline kvq_status check_pool(const kvq_pages *p)
{
    const kvq_status st = check_shape(p);
    if (st != KVQ_OK) return st;
    return p->n_pages > 0 && (!p->data || !aligned(p->data, 128)) ? KVQ_ERR_INVALID_ARG : KVQ_OK;
}

inline PoolDesc pool_of(const kvq_pages *p)
{
    return PoolDesc{static_cast<uint8_t *>(p->data), p->n_pages, p->n_pages * p->page_tokens, page_shift(p->page_tokens),
                    p->n_kv_heads};
}

// A table row of max_blocks pages holds fewer than 2^30 positions.
inline bool table_ok(int stride, int max_blocks, int page_tokens)
{
    return max_blocks >= 0 && stride >= max_blocks && (long long)max_blocks * page_tokens <= 1 << 30;
}

}  // namespace kvq
