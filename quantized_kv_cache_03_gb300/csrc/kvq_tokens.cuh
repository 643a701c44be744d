// kvq_tokens.cuh -- launch parameters and device helpers of the calls around the
// paged cache's append and attention (include/kvq_tokens.h).
#pragma once

#include "kvq_paged.cuh"
#include "kvq_tokens.h"

namespace kvq {

struct RopeDesc {
    const unsigned long long *turns;   // [n_rot / 2]
    int n_rot;                         // 0: no rotation
    int pairs;                         // KVQ_ROPE_PAIRS
    float amplitude;
};

// cos and sin of position * rate, both times amplitude.  The product of the
// position and the rate (parts of a turn, 2^-64) wraps at full turns; its top
// 32 bits as a signed number are the angle in (-1, 1) half turns, exact to
// 2^-32 of a turn for the rate as it is kept and rounded to 24 bits: 1.9e-7 rad at
// most.
__device__ __forceinline__ float2 angle_of(unsigned long long rate, int pos, float amplitude)
{
    const unsigned long long t = rate * (unsigned long long)(long long)pos;
    float s, c;
    sincospif((float)(int)(t >> 32) * 0x1p-31f, &s, &c);
    return make_float2(c * amplitude, s * amplitude);
}

struct PositionsParams {
    const int *q_start, *lens;
    int *positions;
    int n_seqs, n_tokens;
};

struct QkvParams {
    PoolDesc pool;              // keys and values into pages, if `paged`
    RopeDesc rope;
    const uint16_t *q, *k, *v;
    long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
    uint16_t *q_out, *k_out;
    const float *q_norm, *k_norm;   // may be null
    const int *positions, *slots;   // slots may be null
    float eps;
    int n_tokens, n_q_heads, n_kv_heads;
    int paged;
    int full;                        // blocks that take all heads of their tokens; the others
    int chunks, q_heads, kv_heads;   // a share of so many, of so many heads
};

struct ForkParams {
    const int *lens, *parent, *keep, *table, *n_free;
    int *table_out, *lens_out, *free_pages, *n_free_out, *copy_from, *copy_to, *copy_held, *status;
    uint8_t *old_mark, *full_mark, *tail_mark;   // [n_pages]: listed by an old row, by a new one as a whole page, as its last one in part
    int *owner;                 // [n_pages], of pages with a tail mark: the first place that ends in it
    int *seqs;                  // [8][n_seqs]
    int *counts, *totals;       // [blocks]: pages given back by each block's share of the pool; the old stack's size, copies needed
    int blocks;                 // of the launches that count and push
    int n_seqs, pshift, n_pages, stride, out_stride, max_blocks;
};

// Two sizes: a launch carries its parameters along, and 1.5 KB of them take 0.2 us longer than 200 bytes.
constexpr int kFewPools = 8;
template <int POOLS>
struct CopyParams {
    uint8_t *data[POOLS];
    uint16_t heads[POOLS], tile_bytes[POOLS];
    const int *from, *to, *held;
    int n_pools, n_copies, n_pages, most_heads, tiles;
    int pieces, blocks;   // of a head's run of bytes; of a page in one pool
};

struct GatherParams {
    PoolDesc pool;
    const int *slots;
    int n_tokens;
    void *k_out, *v_out;
    int heads, chunks;             // kv heads of a warp, and such pieces of a token's
};

struct MoveParams {
    PoolDesc pool;
    RopeDesc rope;
    const int *from, *to, *turn;   // turn: null without a rotation
    int n_tokens;
    int heads, chunks;             // kv heads of a warp, and such pieces of a token's
    uint8_t *rows;                 // staged: [n_tokens][kv heads] rows of staged_row_bytes()
};

// With programmatic dependent launch the next launch is prepared while one runs, but its blocks are placed only as this
// one's end: these kernels do not call pdl_trigger.  Blocks that are placed early wait on the few SMs with room for them
// and crowd there (kvq_qkv of 777 tokens and their gather, in a stream: 16.8 us, 13.4 so; 8192 tokens 45.2, 42.7; a page
// copied 1.76, 1.53).  The fork's one cluster, which leaves most SMs free, does call it (7.1 us, 7.2 without).
cudaError_t launch_positions(const PositionsParams &p, cudaStream_t s, bool pdl);
cudaError_t prepare_qkv();
cudaError_t launch_qkv(const QkvParams &p, int v_type, int k_type, int n_sms, cudaStream_t s, bool pdl);
cudaError_t prepare_page_fork();
cudaError_t launch_page_fork(const ForkParams &p, int n_sms, cudaStream_t s, bool pdl);
template <int POOLS>
cudaError_t launch_page_copy(const CopyParams<POOLS> &p, cudaStream_t s, bool pdl);
// rows null: from slots to slots; else through them.
int staged_row_bytes(int v_type, int k_type);
cudaError_t launch_paged_move(const MoveParams &p, int v_type, int k_type, int n_sms, cudaStream_t s, bool pdl);

}  // namespace kvq
