// kvq_paged.cuh -- launch parameters and device helpers of the paged cache's
// kernels (include/kvq_paged.h): the tile record, slots, and the deterministic
// split of a ragged batch over persistent CTAs.
#pragma once

#include "kvq_internal.cuh"
#include "kvq_paged.h"

namespace kvq {

// ------------------------------------------------------------ tile record --
// 16 positions of one kv head in one run of bytes: K codes, K scales (int8 K),
// V codes, V scales.  Code bytes in the fragment order of kvq_internal.cuh,
// int8 codes biased by 128 (the form the byte-permute conversion wants, which
// saves it an xor per word).  The scales of positions (2i, 2i + 1) sit side by
// side, block after block, so lane c of an 8-position group gets the scale
// pairs of its two positions for all four blocks in one 16-byte load.
template <int VT, int KT>
struct PageTile {
    static constexpr int K = kWTile * kD * (KT == KVQ_K_F16 ? 2 : 1);
    static constexpr int S = kWTile * kNB * 2;
    static constexpr int V = kWTile * (VT == KVQ_V_Q4_0 ? kD / 2 : kD);
    static constexpr int KS_OFF = K;
    static constexpr int V_OFF = K + (KT == KVQ_K_F16 ? 0 : S);
    static constexpr int VS_OFF = V_OFF + V;
    static constexpr int BYTES = VS_OFF + S;
};
__host__ __device__ constexpr int page_tile_bytes(int v_type, int k_type)
{
    return kWTile * (kD * (k_type == KVQ_K_F16 ? 2 : 1) + (v_type == KVQ_V_Q4_0 ? kD / 2 : kD)) +
           kWTile * kNB * 2 * (k_type == KVQ_K_F16 ? 1 : 2);
}
// Byte offset of block b's scale of position u in a scale area.
__host__ __device__ constexpr int scale_off(int u, int b) { return 2 * (((u / 8) * 4 + (u % 8) / 2) * 8 + 2 * b + u % 2); }

// Codes of four fp16 values x01, x23 for the block scale s (fp32 copy of an fp16
// number): x / s to the nearest integer, halves away from zero, held to lo..hi;
// NaN gives lo.  As bytes of (code + bias).  Without a division: x and s have 11
// bits, so x / s below 191 that is not a half is 2.4e-4 or more away from the
// next one (1.3e-6 of itself), and x times 1/s, off by 2e-7 of itself, gives the
// same integer once it is nudged by 8e-7 of itself, which takes the halves
// outward.  The addition of 1.5 * 2^23 rounds the exact product.
__device__ __forceinline__ uint32_t codes4(uint32_t x01, uint32_t x23, float s, float lo, float hi, int bias)
{
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    inv = s == 0.f ? 0.f : inv * 1.0000008f;   // s = inf: 0, and inf * 0 is NaN
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&x01)), b = __half22float2(*reinterpret_cast<const __half2 *>(&x23));
    const float x[4] = {a.x, a.y, b.x, b.y}, zero = 12582912.f + (float)bias;
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = __float_as_uint(fminf(fmaxf(fmaf(x[k], inv, zero), zero + lo), zero + hi));
    return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
}

// quant_token for the paged cache: the same codes and scales; kw is biased by
// 128, and so is vw for q8_0.  (a / 127, a of 11 bits, stays 1.9e-6 of itself
// away from the middle of two fp16 numbers, so the product's rounding, 1e-7,
// cannot change the scale.)
template <int VT, int KT>
__device__ __forceinline__ TokenRow paged_token(const uint16_t *k_row, const uint16_t *v_row, int lane)
{
    TokenRow t;
    const uint2 k = *reinterpret_cast<const uint2 *>(k_row + 4 * lane), v = *reinterpret_cast<const uint2 *>(v_row + 4 * lane);
    // the blocks' largest magnitudes, K's in the low half, V's in the high one
    auto h2 = [](uint32_t w) { return *reinterpret_cast<const __half2 *>(&w); };
    auto bits = [](const __half2 &h) { return *reinterpret_cast<const uint32_t *>(&h); };
    const uint32_t mk = bits(__hmax2(h2(k.x & 0x7fff7fffu), h2(k.y & 0x7fff7fffu))), mv = bits(__hmax2(h2(v.x & 0x7fff7fffu), h2(v.y & 0x7fff7fffu)));
    __half2 m = __hmax2(h2(__byte_perm(mk, mv, 0x5410)), h2(__byte_perm(mk, mv, 0x7632)));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = __hmax2(m, h2(__shfl_xor_sync(0xffffffffu, bits(m), o)));
    const float2 a = __half22float2(m);
    if (KT == KVQ_K_F16) {
        t.kw = k.x;
        t.kw2 = k.y;
        t.ks = 0;
    } else {
        const __half s = __float2half_rn(a.x * (1.f / 127.f));
        t.ks = __half_as_ushort(s);
        t.kw = codes4(k.x, k.y, __half2float(s), -127.f, 127.f, 128);
        t.kw2 = 0;
    }
    if (VT == KVQ_V_Q8_0) {
        const __half s = __float2half_rn(a.y * (1.f / 127.f));
        t.vs = __half_as_ushort(s);
        t.vw = codes4(v.x, v.y, __half2float(s), -127.f, 127.f, 128);
    } else {
        const __half s = __float2half_rn(a.y * 0.125f);   // exact before rounding
        t.vs = __half_as_ushort(s);
        const uint32_t q = codes4(v.x, v.y, __half2float(s), -8.f, 7.f, 8);
        t.vw = q | __shfl_down_sync(0xffffffffu, q, 4) << 4;   // elements 16.. of the block
    }
    return t;
}

// V codes of positions u, u + 1 (u even) sit in the same words: byte offset of
// lane's word pair (q8_0: 8 bytes, both positions' codes of its four dims) or
// word (q4_0: 4 bytes, code bytes 2g, 2g + 1 of block b for lane 8b + g).
__device__ __forceinline__ int v8_pair_off(int u, int lane)
{
    return ((2 * (u / 8) + (lane >> 4)) * 32 + 4 * (lane & 7) + (u % 8) / 2) * 16 + 8 * ((lane >> 3) & 1);
}
__device__ __forceinline__ int v4_pair_off(int u, int b, int g) { return ((u / 8) * 32 + 4 * g + (u % 8) / 2) * 16 + 4 * b; }

// K codes (and, int8, nothing else) of a quantized row into place u.
template <int VT, int KT>
__device__ __forceinline__ void store_k_paged(const TokenRow &t, int u, int lane, uint8_t *tile)
{
    if (KT == KVQ_K_F16) {
        *reinterpret_cast<uint32_t *>(tile + k16_tile_off(u, 4 * lane)) = t.kw;
        *reinterpret_cast<uint32_t *>(tile + k16_tile_off(u, 4 * lane + 2)) = t.kw2;
    } else {
        *reinterpret_cast<uint32_t *>(tile + k_tile_off(u, 4 * lane)) = t.kw;
    }
}

// A quantized row (paged_token) into place u of a tile.
template <int VT, int KT>
__device__ __forceinline__ void store_token_paged(const TokenRow &t, int u, int lane, uint8_t *tile)
{
    using T = PageTile<VT, KT>;
    store_k_paged<VT, KT>(t, u, lane, tile);
    if (KT != KVQ_K_F16 && (lane & 7) == 0) *reinterpret_cast<uint16_t *>(tile + T::KS_OFF + scale_off(u, lane >> 3)) = t.ks;
    uint8_t *vt = tile + T::V_OFF;
    if (VT == KVQ_V_Q8_0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) vt[v8_tile_off(u, 4 * lane + k)] = (uint8_t)(t.vw >> (8 * k));
    } else if ((lane & 7) < 4) {
        const int j = 16 * (lane >> 3) + 4 * (lane & 3);
        *reinterpret_cast<uint16_t *>(vt + v4_tile_off(u, j)) = (uint16_t)t.vw;
        *reinterpret_cast<uint16_t *>(vt + v4_tile_off(u, j + 2)) = (uint16_t)(t.vw >> 16);
    }
    if ((lane & 7) == 0) *reinterpret_cast<uint16_t *>(tile + T::VS_OFF + scale_off(u, lane >> 3)) = t.vs;
}

// Two rows into places u, u + 1 (u even): whole words of V codes and scales.
template <int VT, int KT>
__device__ __forceinline__ void store_pair_paged(const TokenRow &a, const TokenRow &b, int u, int lane, uint8_t *tile)
{
    using T = PageTile<VT, KT>;
    store_k_paged<VT, KT>(a, u, lane, tile);
    store_k_paged<VT, KT>(b, u + 1, lane, tile);
    uint8_t *vt = tile + T::V_OFF;
    if (VT == KVQ_V_Q8_0) {
        *reinterpret_cast<uint2 *>(vt + v8_pair_off(u, lane)) = make_uint2(__byte_perm(a.vw, b.vw, 0x5140), __byte_perm(a.vw, b.vw, 0x7362));
    } else {   // lanes 8b .. 8b + 3 hold the block's 16 bytes
        const int src = (lane & 24) + ((lane & 7) >> 1);
        const uint32_t x = __shfl_sync(0xffffffffu, a.vw, src), y = __shfl_sync(0xffffffffu, b.vw, src);
        *reinterpret_cast<uint32_t *>(vt + v4_pair_off(u, lane >> 3, lane & 7)) = __byte_perm(x, y, lane & 1 ? 0x7632 : 0x5410);
    }
    if ((lane & 7) == 0) {
        const int o = scale_off(u, lane >> 3);
        if (KT != KVQ_K_F16) *reinterpret_cast<uint32_t *>(tile + T::KS_OFF + o) = a.ks | (uint32_t)b.ks << 16;
        *reinterpret_cast<uint32_t *>(tile + T::VS_OFF + o) = a.vs | (uint32_t)b.vs << 16;
    }
}

struct PoolDesc {
    uint8_t *data;
    int n_pages;
    int n_slots;        // n_pages * page_tokens
    int pshift;         // log2(page_tokens)
    int n_kv_heads;
};

// Tile of (slot, head): its first byte.  Offsets in 64 bits.
__device__ __forceinline__ uint8_t *tile_of(const PoolDesc &p, int page, int h, int tile, int tile_bytes)
{
    return p.data + ((((size_t)page * p.n_kv_heads + h) << (p.pshift - 4)) + tile) * tile_bytes;
}

struct TableParams {
    const int *lens, *n_new, *n_free;
    int *free_pages, *block_table, *lens_out, *n_free_out, *q_start, *slots, *status;
    int n_seqs, pshift, n_pages, stride, max_blocks, n_tokens;
    bool slots_here;   // the table kernel fills the slots too
};

struct PagedRowsParams {      // append and gather
    PoolDesc pool;
    const uint16_t *k16, *v16;
    long long stride;         // elements between tokens
    const int *slots;
    int n_tokens;
    void *k_out, *v_out;
};

// ------------------------------------------------------- paged attention --
constexpr int kStagePos = 32;           // positions per work unit ("stage")
constexpr int kChunkRows = 128;         // the chunk kernel: query rows per tile,
constexpr int kChunkPositions = 128;    // positions per tile,
constexpr int kChunkMinTiles = 3;       // and the least piece in tiles
constexpr int kChunkSums = kChunkRows * kD;   // fp32: a row tile's sums
constexpr int kPagedMinStages = 4;      // a CTA's least piece of the line: one stage per warp

// A query-row tile of one kv head that several CTAs attend: what the combine
// needs to merge its pieces (np = 0: none).
struct PagedCut {
    int b;        // sequence
    int h_rt;     // kv head | row tile << 8
    int c0, np;   // pieces: slot 1 of CTA c0, slot 0 of CTAs c0 + 1 .. c0 + np - 1
};

// The cut tiles and pieces of one attention launch, for the combine.
struct PagedPieces {
    const PagedCut *cuts;
    const float *lse, *o;
    int rows;     // rows of a tile
    int ctas;     // of the launch; 0: it cut nothing
    int spread;   // combine blocks per CTA
};
constexpr int kAttnParts = 3;   // launches of a call: row tiles of 8 rows, of 16, the chunk kernel
struct PagedCuts {
    PagedPieces part[kAttnParts];
};

struct PagedAttnParams {
    PoolDesc pool;
    const uint16_t *q;
    long long q_stride;
    const int *q_start, *seq_lens, *block_table;
    void *out;
    float *lse;                         // may be null
    PagedCut *cuts;                     // [CTAs][2]
    float *ws_lse;                      // [CTAs][2][row tile]
    float *ws_o;                        // [CTAs][2][row tile][kD]
    float *sums;                        // chunk kernel: [CTAs][kChunkSums]
    unsigned int *timeouts;
    int n_seqs, n_tokens, max_q, n_q_heads, table_stride, max_blocks, causal;
    int gmax;                           // query heads of the busiest kv head
    int uniform;                        // every kv head has gmax query heads
    int min_rows, max_rows;             // sequences with min_rows <= rows <= max_rows per kv head are this launch's
    float qk_scale_log2;
    int lose;                           // test flavours: which copy CTA 0 leaves out
    uint16_t grp_begin[KVQ_MAX_HEADS + 1];   // kv head h owns grp_q[grp_begin[h] .. grp_begin[h + 1])
    uint8_t grp_q[KVQ_MAX_HEADS];
};

// New rows and visible length of sequence b, held to the arrays' bounds, and
// the last position its first row sees under the causal mask, row i being the
// sequence's i-th also where rows past max_q are left out.
__device__ __forceinline__ void seq_shape(const PagedAttnParams &p, int b, int &t0, int &n, int &len, int &lim0)
{
    t0 = min(max(p.q_start[b], 0), p.n_tokens);
    const int rows = min(max(p.q_start[b + 1], 0), p.n_tokens) - t0;
    n = min(rows, p.max_q);
    len = max(0, (int)min((long long)p.seq_lens[b], (long long)p.max_blocks << p.pool.pshift));
    lim0 = len - rows;
}

// Work of a sequence, in stages of kStagePos positions for every row tile of
// every kv head (at least one each: rows that see nothing are still written);
// 0 when its rows belong to another launch.
__device__ __forceinline__ bool seq_mine(const PagedAttnParams &p, int n)
{
    const long long rows = (long long)n * p.gmax;
    return n > 0 && rows >= p.min_rows && rows <= p.max_rows;
}

cudaError_t prepare_page_tables();
cudaError_t launch_page_tables(TableParams p, cudaStream_t s, bool pdl);
cudaError_t launch_paged_append(const PagedRowsParams &p, int v_type, int k_type, cudaStream_t s, bool pdl);
cudaError_t launch_paged_gather(const PagedRowsParams &p, int v_type, int k_type, int out_type, int n_sms, cudaStream_t s,
                                bool pdl);
// The same for many rows (kvq_held.cu).
cudaError_t launch_gather_many(const PagedRowsParams &p, int v_type, int k_type, int out_type, int n_sms, cudaStream_t s, bool pdl);
cudaError_t launch_paged_combine(const PagedAttnParams &p, const PagedCuts &cuts, int out_type, cudaStream_t s, bool pdl);
// Row-tile attention (kvq_paged_attn_q4.cu / _q8.cu): nt = 8-row tiles per CTA (1 or 2).
cudaError_t prepare_paged_q4(int nt, int k_type, int out_type, int *ctas_per_sm);
cudaError_t prepare_paged_q8(int nt, int k_type, int out_type, int *ctas_per_sm);
cudaError_t launch_paged_q4(const PagedAttnParams &p, int nt, int k_type, int out_type, int n_ctas, cudaStream_t s,
                            bool pdl);
cudaError_t launch_paged_q8(const PagedAttnParams &p, int nt, int k_type, int out_type, int n_ctas, cudaStream_t s,
                            bool pdl);

// Chunk attention on tcgen05 (kvq_paged_chunk_q4.cu / _q8.cu), int8 K.
cudaError_t prepare_chunk_q4();
cudaError_t prepare_chunk_q8();
cudaError_t launch_chunk_q4(const PagedAttnParams &p, int out_type, int n_ctas, cudaStream_t s, bool pdl);
cudaError_t launch_chunk_q8(const PagedAttnParams &p, int out_type, int n_ctas, cudaStream_t s, bool pdl);

// Test flavours (int8 K, q4_0 V, fp32 output; row tiles of 8 rows, chunks) in
// which CTA 0 arms one copy's barrier and leaves the copy out, so that the wait
// for it, given a short limit, runs out: kvq_debug_paged_lose_copy.
constexpr uint32_t kLostCopySpins = 1 << 15;   // of the lost stage's wait; in the chunk kernel of every wait but those for copies and MMAs in flight
cudaError_t launch_paged_lose(const PagedAttnParams &p, int n_ctas, cudaStream_t s, bool pdl);
cudaError_t launch_chunk_lose(const PagedAttnParams &p, int n_ctas, cudaStream_t s, bool pdl);

// The current device's SM count and the address of the bounded waits' counter
// (kvq_api.cu).
kvq_status device_common(int *dev, int *n_sms, unsigned int **timeouts);

template <typename P>
static inline cudaError_t launch_pdl(void (*fn)(P), const P &p, int grid, int block, int smem, cudaStream_t s, bool pdl)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, p);
}

}  // namespace kvq
