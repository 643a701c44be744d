// kvq_quad.cuh -- a held cache row (one token of one head) in four lanes, a quad, so
// that a warp works on eight rows: taken out of a page's tile, its key turned and
// quantized anew, put into a tile (kvq_paged_move, the gather of many rows).  What
// rotation and quantization need of eight neighbouring values also serves kvq_qkv,
// which has eight lanes to a row.
//
// Lane c of a quad holds values 32 b + 8 c + i of the row (b < 4, i < 8): eight
// neighbours of every 32-block.  The two values of a pair are then one lane's, side
// by side and for halves of 128 values too (b and b + 2), a block's largest value
// takes two shuffles, and a tile's 16-byte words of K codes are a lane's own: words
// b = 0, 1 and b = 2, 3 of its token.  The words of V codes hold two tokens;
// quads of neighbours (lane ^ 4) exchange halves and write one word each.
// Codes and scales are those of paged_token (kvq_paged.cuh), bit for bit.
//
// Where pairs lie half of fewer than 128 values apart, a lane holds both values of
// its pairs in another order while it rotates: group pairs m = c + 4 b, four values
// each, group m and m + n_rot / 8 below that bound, and neighbouring groups of what
// does not rotate behind it.
#pragma once

#include "kvq_paged_line.cuh"
#include "kvq_tokens.cuh"

namespace kvq {

__device__ __forceinline__ __half2 h2_of(uint32_t w) { return *reinterpret_cast<const __half2 *>(&w); }
__device__ __forceinline__ uint32_t bits_of(const __half2 &h) { return *reinterpret_cast<const uint32_t *>(&h); }

// 16 bytes from global to shared memory; the copies of a thread form groups, of
// which all but the newest N have arrived.
__device__ __forceinline__ void copy16(uint32_t to, const void *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// What rotates, and so how a lane's values are paired.
constexpr int kRotNone = 0, kRotPairs = 1, kRotHalf = 2, kRotPart = 3;   // half: n_rot = 128; part: halves of less

// A lane's fp16 values: eight neighbours of each 32-block.
struct Quad16 {
    uint4 b[4];
};
// Group pair m of a row (part).
struct PartGroups {
    int a, b;        // first dims of the groups
    bool rotates;
    __device__ __forceinline__ PartGroups(int m, int n_rot)
    {
        const int h4 = n_rot >> 3;
        rotates = m < h4;
        a = rotates ? 4 * m : n_rot + 8 * (m - h4);
        b = rotates ? a + 4 * h4 : a + 4;
    }
};

// The same values in fp32, as pairs for packed arithmetic: of neighbours
// (x0 x1), (x2 x3), ..., or, where pairs side by side rotate, of their first
// values and of their second ones: (x0 x2), (x4 x6), (x1 x3), (x5 x7).
template <int ROT>
__device__ __forceinline__ void quad_floats(const uint4 &w, float2 (&x)[4])
{
    const float2 a = half2_of(w.x), b = half2_of(w.y), c = half2_of(w.z), d = half2_of(w.w);
    if (ROT == kRotPairs) {
        x[0] = make_float2(a.x, b.x);
        x[1] = make_float2(c.x, d.x);
        x[2] = make_float2(a.y, b.y);
        x[3] = make_float2(c.y, d.y);
    } else {
        x[0] = a;
        x[1] = b;
        x[2] = c;
        x[3] = d;
    }
}
template <int ROT>
__device__ __forceinline__ uint4 quad_halves(const float2 (&x)[4])
{
    if (ROT == kRotPairs)
        return make_uint4(pack_half2(x[0].x, x[2].x), pack_half2(x[0].y, x[2].y), pack_half2(x[1].x, x[3].x), pack_half2(x[1].y, x[3].y));
    return make_uint4(pack_half2(x[0].x, x[0].y), pack_half2(x[1].x, x[1].y), pack_half2(x[2].x, x[2].y), pack_half2(x[3].x, x[3].y));
}

// Cosines and sines of a token, pair after pair; rows of a table are kAngleRow
// floats apart, which keeps the quads of a warp in different banks.
constexpr int kAngleRow = kD / 2 + 4;
__device__ __forceinline__ void quad_turn2(float2 &a, float2 &b, float2 c, float2 s)
{
    const float2 u = sub2(mul2(a, c), mul2(b, s)), v = fma2(a, s, mul2(b, c));
    a = u;
    b = v;
}
// Four pairs at `at` of a token's table: x[0], x[1] their first values, x[2], x[3] the second.
__device__ __forceinline__ void quad_turn4(float2 (&x)[4], const float *cosines, const float *sines, int at)
{
    const float4 cs = *reinterpret_cast<const float4 *>(cosines + at), sn = *reinterpret_cast<const float4 *>(sines + at);
    quad_turn2(x[0], x[2], make_float2(cs.x, cs.y), make_float2(sn.x, sn.y));
    quad_turn2(x[1], x[3], make_float2(cs.z, cs.w), make_float2(sn.z, sn.w));
}
// Eight pairs: x the first values, y the second.
__device__ __forceinline__ void quad_turn8(float2 (&x)[4], float2 (&y)[4], const float *cosines, const float *sines, int at)
{
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
        const float4 cs = *reinterpret_cast<const float4 *>(cosines + at + 2 * k), sn = *reinterpret_cast<const float4 *>(sines + at + 2 * k);
        quad_turn2(x[k], y[k], make_float2(cs.x, cs.y), make_float2(sn.x, sn.y));
        quad_turn2(x[k + 1], y[k + 1], make_float2(cs.z, cs.w), make_float2(sn.z, sn.w));
    }
}

// Codes of eight fp16 values for scale s, as bytes of code + bias: those of
// codes4.  The sums' low 16 bits are code + (bias - lo), so a packed minimum that
// also cuts off at 0 holds two of them to lo..hi in one instruction (NaN: all
// bits, which as a negative number gives lo).
template <bool Q4>
__device__ __forceinline__ uint2 codes8(const uint4 &x, float s)
{
    constexpr int lo = Q4 ? -8 : -127, hi = Q4 ? 7 : 127, back = Q4 ? 0 : 0x01010101;   // int8 codes: lo + 128 = 1
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    inv = s == 0.f ? 0.f : inv * 1.0000008f;
    const float2 f2 = make_float2(inv, inv), z2 = make_float2(12582912.f - (float)lo, 12582912.f - (float)lo);
    auto two = [&](uint32_t w) {
        const float2 v = fma2(half2_of(w), f2, z2);
        const uint32_t p = __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x5410);
        return __vimin_s16x2_relu(p, (uint32_t)(hi - lo) * 0x10001u);
    };
    return make_uint2(__byte_perm(two(x.x), two(x.y), 0x6420) + back, __byte_perm(two(x.z), two(x.w), 0x6420) + back);
}

// Largest magnitudes of eight fp16 values: of the low halves, of the high ones.
__device__ __forceinline__ uint32_t top8(const uint4 &w)
{
    return bits_of(__hmax2(__hmax2(__habs2(h2_of(w.x)), __habs2(h2_of(w.y))), __hmax2(__habs2(h2_of(w.z)), __habs2(h2_of(w.w)))));
}
// The scales of two blocks from their largest magnitudes.
template <bool Q4>
__device__ __forceinline__ __half2 scales_of(uint32_t top)
{
    const float2 a = half2_of(top);
    return __floats2half2_rn(a.x * (Q4 ? 0.125f : 1.f / 127.f), a.y * (Q4 ? 0.125f : 1.f / 127.f));
}

// The row's int8 codes and scales: word 2 b + g of a block's lane holds codes 8 c + 4 g
// and on.
struct QuadCodes {
    uint32_t w[8];
    uint32_t s[2];   // scales of blocks 0, 1 and 2, 3 (fp16 bits)
};
__device__ __forceinline__ QuadCodes quad_quantize(const Quad16 &x)
{
    uint32_t top[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t m[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) m[k] = top8(x.b[2 * h + k]);
        top[h] = bits_of(__hmax2(h2_of(__byte_perm(m[0], m[1], 0x5410)), h2_of(__byte_perm(m[0], m[1], 0x7632))));   // a block to a half
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) top[h] = bits_of(__hmax2(h2_of(top[h]), h2_of(__shfl_xor_sync(0xffffffffu, top[h], o))));
    }
    QuadCodes r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const __half2 s = scales_of<false>(top[h]);
        r.s[h] = bits_of(s);
        const float2 f = __half22float2(s);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint2 w = codes8<false>(x.b[2 * h + k], k ? f.y : f.x);
            r.w[4 * h + 2 * k] = w.x;
            r.w[4 * h + 2 * k + 1] = w.y;
        }
    }
    return r;
}
// The scale of block c, for its lane.
__device__ __forceinline__ uint32_t own_scale(const uint32_t (&s)[2], int c) { return (c & 2 ? s[1] : s[0]) >> (c & 1 ? 16 : 0) & 0xffff; }

// Of a block's q4_0 code bytes lane c has 4 quart .. + 3, quart = 0, 2, 1, 3.
__device__ __forceinline__ int quart_of(int c) { return (c & 1) << 1 | c >> 1; }

// ---- in and out of tiles ----
// A lane's part of K: eight words of codes, or sixteen of fp16 values, and the
// row's scales.  Of V: eight words of q8_0 codes (as QuadCodes) or four of q4_0
// code bytes, and the scale of block c.
template <int VT, int KT>
struct QuadRow {
    static constexpr int KW = KT == KVQ_K_F16 ? 16 : 8, VW = VT == KVQ_V_Q8_0 ? 8 : 4;
    uint32_t k[KW], ks[2], v[VW], vs;
};

__device__ __forceinline__ int quad_k_off(int u, int c, int jh) { return ((2 * (u / 8) + jh) * 32 + 4 * (u % 8) + c) * 16; }
__device__ __forceinline__ int quad_v8_off(int u, int c, int gi, int jh) { return ((2 * (u / 8) + jh) * 32 + 4 * (2 * c + gi) + (u % 8) / 2) * 16; }
__device__ __forceinline__ int quad_v4_off(int u, int quart, int i) { return ((u / 8) * 32 + 4 * (2 * quart + i) + (u % 8) / 2) * 16; }

template <int VT, int KT>
__device__ __forceinline__ void quad_get_key(QuadRow<VT, KT> &r, const uint8_t *tile, int u, int c)
{
    if (KT == KVQ_K_F16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) r.k[i] = *reinterpret_cast<const uint32_t *>(tile + k16_tile_off(u, 32 * (i / 4) + 8 * c + 2 * (i % 4)));
        r.ks[0] = r.ks[1] = 0;
    } else {
#pragma unroll
        for (int jh = 0; jh < 2; ++jh) {
            const uint4 w = *reinterpret_cast<const uint4 *>(tile + quad_k_off(u, c, jh));
            r.k[4 * jh] = w.x;
            r.k[4 * jh + 1] = w.y;
            r.k[4 * jh + 2] = w.z;
            r.k[4 * jh + 3] = w.w;
        }
        const uint4 s = *reinterpret_cast<const uint4 *>(tile + PageTile<VT, KT>::KS_OFF + 16 * (u / 2));   // both places' scales, block after block
        const uint32_t sel = u & 1 ? 0x7632 : 0x5410;
        r.ks[0] = __byte_perm(s.x, s.y, sel);
        r.ks[1] = __byte_perm(s.z, s.w, sel);
    }
}
template <int VT, int KT>
__device__ __forceinline__ void quad_put_key(const QuadRow<VT, KT> &r, uint8_t *tile, int u, int c)
{
    if (KT == KVQ_K_F16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) *reinterpret_cast<uint32_t *>(tile + k16_tile_off(u, 32 * (i / 4) + 8 * c + 2 * (i % 4))) = r.k[i];
    } else {
#pragma unroll
        for (int jh = 0; jh < 2; ++jh)
            *reinterpret_cast<uint4 *>(tile + quad_k_off(u, c, jh)) = make_uint4(r.k[4 * jh], r.k[4 * jh + 1], r.k[4 * jh + 2], r.k[4 * jh + 3]);
        *reinterpret_cast<uint16_t *>(tile + PageTile<VT, KT>::KS_OFF + scale_off(u, c)) = (uint16_t)own_scale(r.ks, c);
    }
}

template <int VT, int KT>
__device__ __forceinline__ void quad_get_value(QuadRow<VT, KT> &r, const uint8_t *tile, int u, int c)
{
    const uint8_t *vt = tile + PageTile<VT, KT>::V_OFF;
    if (VT == KVQ_V_Q8_0) {
        const uint32_t sel = u & 1 ? 0x7531 : 0x6420;
#pragma unroll
        for (int gi = 0; gi < 2; ++gi)
#pragma unroll
            for (int jh = 0; jh < 2; ++jh) {
                const uint4 w = *reinterpret_cast<const uint4 *>(vt + quad_v8_off(u, c, gi, jh));
                r.v[4 * jh + gi] = __byte_perm(w.x, w.y, sel);
                r.v[4 * jh + 2 + gi] = __byte_perm(w.z, w.w, sel);
            }
    } else {
        const uint32_t sel = u & 1 ? 0x7632 : 0x5410;
        const uint4 x = *reinterpret_cast<const uint4 *>(vt + quad_v4_off(u, quart_of(c), 0)), y = *reinterpret_cast<const uint4 *>(vt + quad_v4_off(u, quart_of(c), 1));
        r.v[0] = __byte_perm(x.x, y.x, sel);
        r.v[1] = __byte_perm(x.y, y.y, sel);
        r.v[2] = __byte_perm(x.z, y.z, sel);
        r.v[3] = __byte_perm(x.w, y.w, sel);
    }
    r.vs = *reinterpret_cast<const uint16_t *>(tile + PageTile<VT, KT>::VS_OFF + scale_off(u, c));
}

// V of the quad's row to place u.  Called by the whole warp.  paired: the quads of
// lanes and lanes ^ 4 hold places u (even) and u + 1 of one tile, and share the
// words; write: the row is to be written at all.
template <int VT, int KT>
__device__ __forceinline__ void quad_put_value(const QuadRow<VT, KT> &r, uint8_t *tile, int u, int c, bool paired, bool write)
{
    uint8_t *vt = tile + PageTile<VT, KT>::V_OFF;
    const bool odd = u & 1;
    if (__any_sync(0xffffffffu, paired && write)) {
        if (VT == KVQ_V_Q8_0) {   // the even place's lane writes words of codes 8 c .. + 3, the other's those of the next four
            const uint32_t s0 = odd ? 0x1504 : 0x5140, s1 = odd ? 0x3726 : 0x7362;
#pragma unroll
            for (int jh = 0; jh < 2; ++jh) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t even_word = r.v[4 * jh + 2 * k], odd_word = r.v[4 * jh + 2 * k + 1];
                    const uint32_t keep = odd ? odd_word : even_word, got = __shfl_xor_sync(0xffffffffu, odd ? even_word : odd_word, 4);
                    w[2 * k] = __byte_perm(keep, got, s0);
                    w[2 * k + 1] = __byte_perm(keep, got, s1);
                }
                if (paired && write) *reinterpret_cast<uint4 *>(vt + quad_v8_off(u, c, odd, jh)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {
            const uint32_t sel = odd ? 0x3276 : 0x5410;
            uint32_t w[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) w[b] = __byte_perm(r.v[b], __shfl_xor_sync(0xffffffffu, r.v[b], 4), sel);
            if (paired && write) *reinterpret_cast<uint4 *>(vt + quad_v4_off(u, quart_of(c), odd)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    if (write && !paired) {   // the bytes of its own place
        if (VT == KVQ_V_Q8_0) {
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int k = 0; k < 8; ++k) vt[v8_tile_off(u, 32 * b + 8 * c + k)] = (uint8_t)(r.v[2 * b + (k >> 2)] >> (8 * (k & 3)));
        } else {
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<uint16_t *>(vt + quad_v4_off(u, quart_of(c), i) + 4 * b + 2 * (u % 2)) = (uint16_t)(r.v[b] >> (16 * i));
        }
    }
    if (write) *reinterpret_cast<uint16_t *>(tile + PageTile<VT, KT>::VS_OFF + scale_off(u, c)) = (uint16_t)r.vs;
}

// What a warp does with a list of slots: places that begin a pair of neighbours
// (an even slot, the next token's one further), or stand alone.
struct SlotPairs {
    unsigned lead, pair;   // bits 1 .. n of the window's tokens
    int leads;
};
// slot: lane i holds the slot of token first - 1 + i of the list (i < n + 2; -1
// where there is none); inside: it may be written.
__device__ __forceinline__ SlotPairs slot_pairs(int slot, bool inside, int n)
{
    const int lane = threadIdx.x & 31;
    const unsigned in = __ballot_sync(0xffffffffu, inside);
    const int before = __shfl_up_sync(0xffffffffu, slot, 1), after = __shfl_down_sync(0xffffffffu, slot, 1);
    const bool second = (slot & 1) && before == slot - 1 && lane > 0 && (in >> (lane - 1) & 1);
    const bool first = !(slot & 1) && after == slot + 1 && lane < 31 && (in >> (lane + 1) & 1);
    SlotPairs q;
    q.lead = __ballot_sync(0xffffffffu, inside && lane >= 1 && lane <= n && !second);
    q.pair = __ballot_sync(0xffffffffu, inside && first);
    q.leads = __popc(q.lead);
    return q;
}
// list: [n] bytes of the warp's in shared memory: the lanes of the leads, in order.
__device__ __forceinline__ void slot_list(const SlotPairs &q, uint8_t *list)
{
    const int lane = threadIdx.x & 31;
    if (q.lead >> lane & 1) list[__popc(q.lead & ((1u << lane) - 1))] = (uint8_t)lane;
    __syncwarp();
}

}  // namespace kvq
