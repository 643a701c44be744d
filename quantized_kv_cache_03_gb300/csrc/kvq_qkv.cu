// kvq_qkv.cu -- new tokens on their way into the paged cache: heads normalized
// and rotated, queries (and keys, without pages) written as fp16, keys and values
// quantized into their slots.
#include "kvq_tokens.cuh"

namespace kvq {

constexpr int kQkvWarps = 8;

// A half-warp holds a row (token, head), eight values a lane, as two groups of
// four dims.  The groups are chosen so that both values of a pair are the same
// lane's: with pairs side by side (and without a rotation) the lane's groups are,
// with pairs half of n_rot apart the groups are too, and what is not rotated is
// shared out over the lanes behind.  Either way lanes below n_rot / 8 rotate, by
// rates 4 * lane and on.
template <int PAIRS>
struct Lane {
    int a, b;        // first dims of the groups
    bool rotates;
    __device__ __forceinline__ Lane(const RopeDesc &r, int l)
    {
        const int h4 = r.n_rot >> 3;
        rotates = l < h4;
        a = PAIRS ? 8 * l : rotates ? 4 * l : r.n_rot + 8 * (l - h4);
        b = PAIRS ? a + 4 : rotates ? a + 4 * h4 : a + 4;
    }
};

struct Raw {
    uint2 a, b;
};
template <int PAIRS>
__device__ __forceinline__ Raw load_row(const uint16_t *row, const Lane<PAIRS> &ln)
{
    Raw r;
    if (PAIRS) {
        const uint4 w = *reinterpret_cast<const uint4 *>(row + ln.a);
        r.a = make_uint2(w.x, w.y);
        r.b = make_uint2(w.z, w.w);
    } else {
        r.a = *reinterpret_cast<const uint2 *>(row + ln.a);
        r.b = *reinterpret_cast<const uint2 *>(row + ln.b);
    }
    return r;
}
template <int PAIRS>
__device__ __forceinline__ void store_row(uint16_t *row, const Lane<PAIRS> &ln, const Raw &r)
{
    if (PAIRS) {
        *reinterpret_cast<uint4 *>(row + ln.a) = make_uint4(r.a.x, r.a.y, r.b.x, r.b.y);
    } else {
        *reinterpret_cast<uint2 *>(row + ln.a) = r.a;
        *reinterpret_cast<uint2 *>(row + ln.b) = r.b;
    }
}

struct Weights {
    float4 a, b;
    template <int PAIRS>
    __device__ __forceinline__ Weights(const float *norm, const Lane<PAIRS> &ln)
    {
        a = b = make_float4(1.f, 1.f, 1.f, 1.f);
        if (norm) {
            a = *reinterpret_cast<const float4 *>(norm + ln.a);
            b = *reinterpret_cast<const float4 *>(norm + ln.b);
        }
    }
};

// The half-warp's row, normalized and rotated.  cs: the lane's four angles.
template <int PAIRS>
__device__ __forceinline__ Raw turn_row(const Raw &r, const Lane<PAIRS> &ln, const Weights &w, bool norm, float eps, const float2 (&cs)[4])
{
    float x[8];
    {
        auto two = [](uint32_t v, float &lo, float &hi) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v));
            lo = f.x;
            hi = f.y;
        };
        two(r.a.x, x[0], x[1]);
        two(r.a.y, x[2], x[3]);
        two(r.b.x, x[4], x[5]);
        two(r.b.y, x[6], x[7]);
    }
    if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fmaf(x[k], x[k], ss);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float f = rsqrtf(fmaf(ss, 1.f / kD, eps));
        const float wv[8] = {w.a.x, w.a.y, w.a.z, w.a.w, w.b.x, w.b.y, w.b.z, w.b.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = x[k] * f * wv[k];
    }
    if (ln.rotates) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float &p = x[PAIRS ? 2 * i : i], &q = x[PAIRS ? 2 * i + 1 : i + 4];
            const float u = p * cs[i].x - q * cs[i].y, v = p * cs[i].y + q * cs[i].x;
            p = u;
            q = v;
        }
    }
    Raw o;
    o.a = make_uint2(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]));
    o.b = make_uint2(pack_half2(x[4], x[5]), pack_half2(x[6], x[7]));
    return o;
}

__device__ __forceinline__ void angles(const QkvParams &p, int pos, int l, bool rotates, float2 (&cs)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) cs[i] = make_float2(1.f, 0.f);
    if (rotates)
#pragma unroll
        for (int i = 0; i < 4; ++i) cs[i] = angle_of(p.rope.turns[4 * l + i], pos, p.rope.amplitude);
}

// Heads [h0, h1) of a token that stay fp16: src to dst.
template <int PAIRS>
__device__ __forceinline__ void rows(const uint16_t *src, uint16_t *dst, const float *norm, float eps, const Lane<PAIRS> &ln,
                                     const float2 (&cs)[4], int h0, int h1, bool mine)
{
    constexpr int kDepth = 4;
    const Weights w(norm, ln);
    for (int h = h0; h < h1; h += kDepth) {
        Raw r[kDepth];
#pragma unroll
        for (int k = 0; k < kDepth; ++k) {
            r[k].a = r[k].b = make_uint2(0, 0);
            if (mine && h + k < h1) r[k] = load_row<PAIRS>(src + (size_t)(h + k) * kD, ln);
        }
        __syncwarp();   // in place: the row is read before it is written
#pragma unroll
        for (int k = 0; k < kDepth; ++k) {
            if (h + k >= h1) break;
            const Raw o = turn_row<PAIRS>(r[k], ln, w, norm != nullptr, eps, cs);
            if (mine) store_row<PAIRS>(dst + (size_t)(h + k) * kD, ln, o);
        }
    }
}

template <int VT, int KT, int PAIRS>
__global__ void __launch_bounds__(kQkvWarps * 32) qkv_kernel(const __grid_constant__ QkvParams p)
{
    __shared__ __align__(16) uint16_t key[kQkvWarps][2][kD];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 15, half = lane >> 4;
    const Lane<PAIRS> ln(p.rope, l);
    float2 cs[4];
    if ((int)blockIdx.x >= p.kv_blocks) {
        // rows that stay fp16: a warp takes tokens 2i, 2i + 1, a half-warp each
        const long long job = (long long)(blockIdx.x - p.kv_blocks) * kQkvWarps + warp;
        const long long pair = job / p.row_chunks;
        const int c = (int)(job - pair * p.row_chunks);
        if (2 * pair >= p.n_tokens) return;
        const int tok = (int)(2 * pair) + half;
        const bool mine = tok < p.n_tokens && (!p.slots || p.slots[tok] >= 0);
        if (!__any_sync(0xffffffffu, mine)) return;
        angles(p, mine && p.rope.n_rot ? p.positions[tok] : 0, l, ln.rotates, cs);
        const int heads = p.n_q_heads + (p.paged ? 0 : p.n_kv_heads), h0 = c * p.row_heads, h1 = min(heads, h0 + p.row_heads);
        if (h0 < p.n_q_heads)
            rows<PAIRS>(p.q + tok * p.q_stride, p.q_out + tok * p.q_out_stride, p.q_norm, p.eps, ln, cs, h0, min(h1, p.n_q_heads), mine);
        if (h1 > p.n_q_heads)
            rows<PAIRS>(p.k + tok * p.k_stride, p.k_out + tok * p.k_out_stride, p.k_norm, p.eps, ln, cs, max(h0, p.n_q_heads) - p.n_q_heads, h1 - p.n_q_heads, mine);
        return;
    }
    // pages: a warp takes a token, or two whose slots are an even place and the next
    const long long job = (long long)blockIdx.x * kQkvWarps + warp;
    const int c = (int)(job / ((p.n_tokens + kQkvWarps - 1) / kQkvWarps * kQkvWarps)), tok = (int)(job % ((p.n_tokens + kQkvWarps - 1) / kQkvWarps * kQkvWarps));
    if (tok >= p.n_tokens) return;
    const int slot = p.slots[tok], before = tok > 0 ? p.slots[tok - 1] : -1, after = tok + 1 < p.n_tokens ? p.slots[tok + 1] : -1;
    if (slot < 0 || slot >= p.pool.n_slots || ((slot & 1) && before == slot - 1)) return;
    const bool pair = !(slot & 1) && after == slot + 1;
    const int my = tok + (pair ? half : 0);   // alone: both half-warps work on the one row
    angles(p, p.rope.n_rot ? p.positions[my] : 0, l, ln.rotates, cs);
    const Weights w(p.k_norm, ln);
    const int place = slot & ((1 << p.pool.pshift) - 1), h1 = min(p.n_kv_heads, (c + 1) * p.kv_heads);
    for (int h = c * p.kv_heads; h < h1; ++h) {
        const uint16_t *vrow = p.v + tok * p.v_stride + (size_t)h * kD;
        const Raw o = turn_row<PAIRS>(load_row<PAIRS>(p.k + my * p.k_stride + (size_t)h * kD, ln), ln, w, p.k_norm != nullptr, p.eps, cs);
        __syncwarp();
        store_row<PAIRS>(key[warp][half], ln, o);
        __syncwarp();
        uint8_t *tile = tile_of(p.pool, slot >> p.pool.pshift, h, place >> 4, PageTile<VT, KT>::BYTES);
        const TokenRow t = paged_token<VT, KT>(key[warp][0], vrow, lane);
        if (pair) {
            const TokenRow t1 = paged_token<VT, KT>(key[warp][1], vrow + p.v_stride, lane);
            store_pair_paged<VT, KT>(t, t1, place & 15, lane, tile);
        } else {
            store_token_paged<VT, KT>(t, place & 15, lane, tile);
        }
    }
}

template <int VT, int KT>
static cudaError_t qkv_t(const QkvParams &p, int blocks, cudaStream_t s, bool pdl)
{
    return p.rope.pairs || p.rope.n_rot == 0 ? launch_pdl(qkv_kernel<VT, KT, 1>, p, blocks, kQkvWarps * 32, 0, s, pdl)
                                             : launch_pdl(qkv_kernel<VT, KT, 0>, p, blocks, kQkvWarps * 32, 0, s, pdl);
}

cudaError_t launch_qkv(const QkvParams &in, int v_type, int k_type, int n_sms, cudaStream_t s, bool pdl)
{
    QkvParams p = in;
    const long long warps = (long long)n_sms * 48;
    // as many heads to a warp as leaves each SM its warps
    auto pieces = [&](int heads, long long tokens, int least, int &each, int &n) {
        const long long want = heads * tokens / warps;
        each = want < least ? least : want > 16 ? 16 : (int)want;
        each = each > heads ? (heads > 0 ? heads : 1) : each;
        n = (heads + each - 1) / each;
    };
    const int row_heads = p.n_q_heads + (p.paged ? 0 : p.n_kv_heads);
    const long long pairs = ((long long)p.n_tokens + 1) / 2;
    pieces(row_heads, pairs, 4, p.row_heads, p.row_chunks);
    pieces(p.paged ? p.n_kv_heads : 0, pairs, 1, p.kv_heads, p.kv_chunks);
    const long long token_blocks = ((long long)p.n_tokens + kQkvWarps - 1) / kQkvWarps;
    p.kv_blocks = (int)(token_blocks * p.kv_chunks);
    const long long blocks = p.kv_blocks + (pairs * p.row_chunks + kQkvWarps - 1) / kQkvWarps;
    if (v_type == KVQ_V_Q4_0)
        return k_type == KVQ_K_F16 ? qkv_t<KVQ_V_Q4_0, KVQ_K_F16>(p, (int)blocks, s, pdl) : qkv_t<KVQ_V_Q4_0, KVQ_K_I8>(p, (int)blocks, s, pdl);
    return k_type == KVQ_K_F16 ? qkv_t<KVQ_V_Q8_0, KVQ_K_F16>(p, (int)blocks, s, pdl) : qkv_t<KVQ_V_Q8_0, KVQ_K_I8>(p, (int)blocks, s, pdl);
}

}  // namespace kvq
