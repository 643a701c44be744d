// kvq_qkv.cu -- new tokens on their way into the paged cache: heads normalized
// and rotated, queries (and keys, without pages) written as fp16, keys and values
// quantized into their slots.
#include <cfloat>
#include <cstddef>

#include "kvq_quad.cuh"

namespace kvq {

constexpr int kQkvWarps = 8;
constexpr int kQkvTokens = 8;   // tokens of a block
constexpr int kQkvBlocks = 3;   // on an SM

constexpr int kBatch = 4;       // rows that an octet takes at a time
static_assert(kQkvWarps * 32 == 2 * kD, "a thread to each weight of the two norms");
static_assert(kQkvTokens == 8 && kQkvWarps % 4 == 0, "four tokens to a warp, and four groups of them in a block at most");

constexpr int kSharedAlign = 1024;
struct alignas(16) QkvShared {
    uint16_t ring[kQkvWarps][kBatch][4][2][kD];   // the places of a row in the two batches side by side: kRowBytes apart in any aligned memory
    float cosines[kQkvTokens + 1][kAngleRow], sines[kQkvTokens + 1][kAngleRow];
    float norm[2][kD];          // of queries, of keys
    uint8_t list[kQkvWarps][kQkvTokens];
};
constexpr uint32_t kRowBytes = kD * 2;
static_assert((kRowBytes & (kRowBytes - 1)) == 0 && kSharedAlign % (2 * kRowBytes) == 0 && offsetof(QkvShared, ring) % (2 * kRowBytes) == 0,
              "one bit of an address tells the two places of a row apart");

// ---- eight lanes (an octet) to a row ----
// A row's 256 bytes are read and written as whole lines, and what multiplies a
// token's rows fits into a lane's registers.  Lane c holds values 8 c + i and
// 64 + 8 c + i, or, where pairs lie half of fewer than 128 apart, the group pairs
// m = c and c + 8 (PartGroups), so that both values of a pair are always its own.
struct Oct16 {
    uint4 b[2];
};
template <int ROT>
__device__ __forceinline__ Oct16 oct_load(const uint16_t *row, int c, int n_rot)
{
    Oct16 r;
#pragma unroll
    for (int b = 0; b < 2; ++b)
        if (ROT == kRotPart) {
            const PartGroups g(c + 8 * b, n_rot);
            const uint2 x = *reinterpret_cast<const uint2 *>(row + g.a), y = *reinterpret_cast<const uint2 *>(row + g.b);
            r.b[b] = make_uint4(x.x, x.y, y.x, y.y);
        } else {
            r.b[b] = *reinterpret_cast<const uint4 *>(row + 64 * b + 8 * c);
        }
    return r;
}
template <int ROT>
__device__ __forceinline__ void oct_store(uint16_t *row, int c, int n_rot, const Oct16 &r)
{
#pragma unroll
    for (int b = 0; b < 2; ++b)
        if (ROT == kRotPart) {
            const PartGroups g(c + 8 * b, n_rot);
            *reinterpret_cast<uint2 *>(row + g.a) = make_uint2(r.b[b].x, r.b[b].y);
            *reinterpret_cast<uint2 *>(row + g.b) = make_uint2(r.b[b].z, r.b[b].w);
        } else {
            *reinterpret_cast<uint4 *>(row + 64 * b + 8 * c) = r.b[b];
        }
}

// 1 / sqrt(x), 2^-22 off at most.  No argument but 0 is below 2^-55 (a square of an fp16 value over 128; eps is held to
// the normal numbers), so nothing is flushed.
__device__ __forceinline__ float inv_sqrt(float x)
{
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (a, b) -> (a A + b B, a C + b D) for the lane's eight pairs of values, two side by
// side; the weights of the norm are in it, its factor of the row comes last.  Which
// values are a pair's: those of x.b[0] and x.b[1] (half), or of one x.b's first and
// second two float2 (quad_floats).
struct OctCoef {
    float2 A[4], B[4], C[4], D[4];
    bool rotates[2];   // of x.b[0], x.b[1]
};
template <int ROT>
__device__ __forceinline__ OctCoef oct_coef(const float *norm, const float *cosines, const float *sines, int c, int n_rot)
{
    OctCoef k;
    float2 w[2][4];   // weights in the order of quad_floats
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        float4 u = make_float4(1.f, 1.f, 1.f, 1.f), v = u;
        if (norm) {
            const PartGroups g(c + 8 * b, n_rot);
            u = *reinterpret_cast<const float4 *>(norm + (ROT == kRotPart ? g.a : 64 * b + 8 * c));
            v = *reinterpret_cast<const float4 *>(norm + (ROT == kRotPart ? g.b : 64 * b + 8 * c + 4));
        }
        const bool first = ROT == kRotPairs;
        w[b][0] = first ? make_float2(u.x, u.z) : make_float2(u.x, u.y);
        w[b][1] = first ? make_float2(v.x, v.z) : make_float2(u.z, u.w);
        w[b][2] = first ? make_float2(u.y, u.w) : make_float2(v.x, v.y);
        w[b][3] = first ? make_float2(v.y, v.w) : make_float2(v.z, v.w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int b = i >> 1, at = ROT == kRotHalf ? 8 * c + 2 * i : ROT == kRotPairs ? 32 * b + 4 * c + 2 * (i & 1) : 4 * (c + 8 * b) + 2 * (i & 1);
        const bool rot = ROT != kRotNone && 2 * (at & ~3) < n_rot;
        if (i % 2 == 0) k.rotates[b] = rot;
        float2 cs = make_float2(1.f, 1.f), sn = make_float2(0.f, 0.f);
        if (rot) {
            cs = *reinterpret_cast<const float2 *>(cosines + at);
            sn = *reinterpret_cast<const float2 *>(sines + at);
        }
        const float2 wa = ROT == kRotHalf ? w[0][i] : w[b][i & 1], wb = ROT == kRotHalf ? w[1][i] : w[b][2 + (i & 1)];
        k.A[i] = mul2(wa, cs);
        k.B[i] = mul2(make_float2(-wb.x, -wb.y), sn);
        k.C[i] = mul2(wa, sn);
        k.D[i] = mul2(wb, cs);
    }
    return k;
}
template <int ROT>
__device__ __forceinline__ Oct16 oct_turn(const Oct16 &raw, const OctCoef &k, bool norm, float eps)
{
    float2 x[2][4];
#pragma unroll
    for (int b = 0; b < 2; ++b) quad_floats<ROT>(raw.b[b], x[b]);
    float f = 1.f;
    if (norm) {
        float2 s2 = mul2(x[0][0], x[0][0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) s2 = fma2(x[i >> 2][i & 3], x[i >> 2][i & 3], s2);
        float ss = s2.x + s2.y;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        f = inv_sqrt(fmaf(ss, 1.f / kD, eps));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 &a = ROT == kRotHalf ? x[0][i] : x[i >> 1][i & 1], &b = ROT == kRotHalf ? x[1][i] : x[i >> 1][2 + (i & 1)];
        float2 u = mul2(a, k.A[i]), v = mul2(b, k.D[i]);
        if (ROT == kRotHalf || (ROT != kRotNone && k.rotates[i >> 1])) {   // (elsewhere B and C are 0, and an infinity times 0 is no value of the row)
            u = fma2(b, k.B[i], u);
            v = fma2(a, k.C[i], v);
        }
        if (norm) {
            u = mul2(u, make_float2(f, f));
            v = mul2(v, make_float2(f, f));
        }
        a = u;
        b = v;
    }
    Oct16 o;
#pragma unroll
    for (int b = 0; b < 2; ++b) o.b[b] = quad_halves<ROT>(x[b]);
    return o;
}

// A token's V codes and K codes as the lanes hold them: codes 8 c .. 8 c + 7 and
// those 64 further, the scales of their two blocks.
struct OctCodes {
    uint2 w[2];
    uint32_t s;      // of block c / 4, of block 2 + c / 4
};
template <bool Q4>
__device__ __forceinline__ OctCodes oct_quantize(const Oct16 &x)
{
    uint32_t m[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) m[b] = top8(x.b[b]);
    uint32_t top = bits_of(__hmax2(h2_of(__byte_perm(m[0], m[1], 0x5410)), h2_of(__byte_perm(m[0], m[1], 0x7632))));
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) top = bits_of(__hmax2(h2_of(top), h2_of(__shfl_xor_sync(0xffffffffu, top, o))));
    const __half2 s = scales_of<Q4>(top);
    const float2 f = __half22float2(s);
    OctCodes r;
    r.s = bits_of(s);
    r.w[0] = codes8<Q4>(x.b[0], f.x);
    r.w[1] = codes8<Q4>(x.b[1], f.y);
    return r;
}
// Where a lane's parts of place u lie in a tile: its K codes (the others 64 dims
// on), V codes, and scales of its first block (of the second 8 bytes on).
struct OctPlace {
    int k, v, s;
    bool odd, paired;
};
template <int VT, int KT>
__device__ __forceinline__ OctPlace oct_place(int u, int c, bool paired)
{
    OctPlace o;
    o.odd = u & 1;
    o.paired = paired;
    o.k = KT == KVQ_K_F16 ? k16_tile_off(u, 8 * c) : k_tile_off(u, 8 * c);
    if (VT == KVQ_V_Q8_0) o.v = quad_v8_off(u, c & 3, paired && o.odd, 0) + 8 * (c >> 2) + (paired ? 0 : o.odd);
    else o.v = quad_v4_off(u, quart_of(c & 3), paired && o.odd) + 4 * (c >> 2) + (paired ? 0 : 2 * o.odd);
    o.v += PageTile<VT, KT>::V_OFF;
    o.s = scale_off(u, c >> 2);
    return o;
}
__device__ __forceinline__ void oct_put_scales(uint8_t *at, int c, uint32_t s)
{
    if ((c & 3) == 0) {
        *reinterpret_cast<uint16_t *>(at) = (uint16_t)s;
        *reinterpret_cast<uint16_t *>(at + 8) = (uint16_t)(s >> 16);
    }
}
template <int VT, int KT>
__device__ __forceinline__ void oct_put_key(const Oct16 &x, uint8_t *tile, const OctPlace &at, int c, bool write)
{
    if (KT == KVQ_K_F16) {
        if (!write) return;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const uint32_t w[4] = {x.b[b].x, x.b[b].y, x.b[b].z, x.b[b].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t *>(tile + at.k + 2048 * b + 16 * i) = w[i];
        }
    } else {
        const OctCodes q = oct_quantize<false>(x);
        if (!write) return;
#pragma unroll
        for (int b = 0; b < 2; ++b) *reinterpret_cast<uint2 *>(tile + at.k + 512 * b) = q.w[b];
        oct_put_scales(tile + PageTile<VT, KT>::KS_OFF + at.s, c, q.s);
    }
}
// paired: octets of lanes and lanes ^ 8 hold places u (even) and u + 1 of one tile,
// whose words of V codes they share: each writes half of them.
template <int VT, int KT>
__device__ __forceinline__ void oct_put_value(const Oct16 &x, uint8_t *tile, const OctPlace &at, int c, bool write)
{
    const OctCodes q = oct_quantize<VT == KVQ_V_Q4_0>(x);
    uint8_t *to = tile + at.v;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        if (VT == KVQ_V_Q8_0) {
            const uint32_t keep = at.odd ? q.w[b].y : q.w[b].x, got = __shfl_xor_sync(0xffffffffu, at.odd ? q.w[b].x : q.w[b].y, 8);
            if (write && at.paired) {
                *reinterpret_cast<uint2 *>(to + 512 * b) = make_uint2(__byte_perm(keep, got, at.odd ? 0x1504 : 0x5140), __byte_perm(keep, got, at.odd ? 0x3726 : 0x7362));
            } else if (write) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    to[512 * b + 64 * (k >> 2) + 4 * ((k & 3) >> 1) + 2 * (k & 1)] = (uint8_t)((k < 4 ? q.w[b].x : q.w[b].y) >> (8 * (k & 3)));
            }
        } else {   // code bytes 4 quart .. + 3 of the block; high nibbles are lane c ^ 2's, or low ones
            const uint32_t keep = c & 2 ? q.w[b].y : q.w[b].x, nib = __shfl_xor_sync(0xffffffffu, c & 2 ? q.w[b].x : q.w[b].y, 2);
            const uint32_t w = c & 2 ? nib | keep << 4 : keep | nib << 4, got = __shfl_xor_sync(0xffffffffu, w, 8);
            if (write && at.paired) {
                *reinterpret_cast<uint32_t *>(to + 8 * b) = __byte_perm(w, got, at.odd ? 0x3276 : 0x5410);
            } else if (write) {
#pragma unroll
                for (int i = 0; i < 2; ++i) *reinterpret_cast<uint16_t *>(to + 8 * b + 64 * i) = (uint16_t)(w >> (16 * i));
            }
        }
    }
    if (write) oct_put_scales(tile + PageTile<VT, KT>::VS_OFF + at.s, c, q.s);
}

// The rows a warp works on, one of each octet's token at a time: some neighbouring
// heads of its queries, then of its keys, on their way into pages with its values.
// They come through a ring of two batches in shared memory, the first of them
// while the block still works out its angles.
struct Stream {
    const uint16_t *q, *k, *v;     // the lane's part of the next rows of its octet's tokens
    int nq, nk;                    // rows of each still to come
    uint32_t to;                   // the lane's part of the next batch's first row, in shared memory
    bool q_there, k_mine;          // q rows are read before their slots are known
};
constexpr uint32_t kStep = 4 * 2 * kRowBytes;   // from row to row of an octet's batch
__device__ __forceinline__ void stream_row(uint32_t to, const uint16_t *from, bool there)
{
    if (there) {
        copy16(to, from);
        copy16(to + kD, from + kD / 2);
    }
}
template <bool PAGED>
__device__ __forceinline__ void stream_get(Stream &w)
{
    if (w.nq > 0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) stream_row(w.to + i * kStep, w.q + i * kD, w.q_there && i < w.nq);
        w.q += kBatch * kD;
        w.nq -= kBatch;
    } else if (w.nk > 0) {
        if (PAGED) {
#pragma unroll
            for (int i = 0; i < kBatch / 2; ++i) {
                stream_row(w.to + 2 * i * kStep, w.k + i * kD, w.k_mine && i < w.nk);
                stream_row(w.to + (2 * i + 1) * kStep, w.v + i * kD, w.k_mine && i < w.nk);
            }
            w.k += kBatch / 2 * kD;
            w.v += kBatch / 2 * kD;
            w.nk -= kBatch / 2;
        } else {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) stream_row(w.to + i * kStep, w.k + i * kD, w.k_mine && i < w.nk);
            w.k += kBatch * kD;
            w.nk -= kBatch;
        }
    }
    w.to ^= kRowBytes;
    copy_commit();
}

// y = x * rsqrt(mean(x^2) + eps) * w for a head's row, then its pairs (a, b) turned:
// (a cos - b sin, a sin + b cos), then, for keys and values in pages, a scale of
// fp16 for every 32 values and codes.  Sums, norms and rotations are fp32; a row
// that stays fp16 is rounded once, and so is a key before it is quantized, so that
// its codes are those of an append of the fp16 row.
//
// Bound by memory, with the arithmetic close behind: 8192 tokens of 40 + 2 * 8 heads
// (q4_0 V, norms, halves) 34.7 us for 215 MB, 6.2 TB/s, 0.91 of a copy's rate, at half
// of the issue slots and 20 warps on an SM.  What a row costs in instructions decides
// how much of a copy's rate is left, so
//  - a block takes eight tokens and a share of the heads: angles are worked out once
//    for all heads (by 64-bit turns and one sincospif each), and so are norms;
//  - an octet takes rows of one token, its cosines, sines and weights in registers
//    (a warp to a pair of rows 62.7 us; half-warps, angles from shared memory 46;
//    quads, eight rows to a warp, 44);
//  - rows come in through a ring in shared memory, two batches of four rows to an
//    octet, because loads into registers leave too few registers for the warps (a row
//    ahead in registers 52; a ring of eight rows with a wait for each 41.4; this 38.6,
//    38.0 with the rates and positions asked for before the slots are looked at, 36.0
//    with the last wave cut up, 34.7 with the first queries asked for then too);
//  - queries and then keys and values go through one stream of batches (a loop for
//    keys and one for values 46; two blocks on an SM with no spill 40.8, three 38.0).
// 777 tokens (64 + 2 * 8 heads, F16 K) take 8 us, 64 tokens 3.5: a launch, slots, rows
// and angles each waiting for memory once.
// Pairs side by side take 42.6 us for the 8192 tokens (q8_0 V 36.9), halves of part of
// a head, whose keys pass through shared memory and back to neighbours, 47.5 (rows that
// stay fp16 40.7).
template <int VT, int KT, int ROT, bool PAGED>
__global__ void __launch_bounds__(kQkvWarps * 32, kQkvBlocks) qkv_kernel(const __grid_constant__ QkvParams p)
{
    extern __shared__ __align__(kSharedAlign) uint8_t qkv_smem[];
    QkvShared &sh = *reinterpret_cast<QkvShared *>(qkv_smem);
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & 7, oct = lane >> 3, n_rot = p.rope.n_rot;
    // blocks of all heads, then those that take a share
    const int part = (int)blockIdx.x - p.full, cut = part < 0 ? 0 : part / p.chunks, share = part < 0 ? 0 : part - cut * p.chunks;
    const int t0 = (part < 0 ? (int)blockIdx.x : p.full + cut) * kQkvTokens, q_heads = part < 0 ? p.n_q_heads : p.q_heads, kv_heads = part < 0 ? p.n_kv_heads : p.kv_heads;
    // slots of the token before the block's, of its own, and of the one behind
    const int at = t0 - 1 + lane;
    const int slot = lane < kQkvTokens + 2 && at >= 0 && at < p.n_tokens ? (p.slots ? p.slots[at] : 0) : -1;
    // what the thread's angles and weights are made of: asked for before anything waits for the slots
    const int aj = threadIdx.x % (kD / 2), at0 = threadIdx.x / (kD / 2);
    const bool turns = ROT != kRotNone && aj < n_rot / 2;
    constexpr int kAngles = kQkvTokens * (kD / 2) / (kQkvWarps * 32);   // of a thread, and one more in some blocks
    unsigned long long rate = 0;
    int pos[kAngles];
    if (turns) rate = p.rope.turns[aj];
#pragma unroll
    for (int i = 0; i < kAngles; ++i) {
        const int t = t0 + at0 + i * (kQkvTokens / kAngles);
        pos[i] = turns && t < p.n_tokens ? p.positions[t] : 0;
    }
    const float *norm = threadIdx.x < kD ? p.q_norm : p.k_norm;
    const float weight = norm ? norm[threadIdx.x % kD] : 0.f;
    const int q1 = min(p.n_q_heads, (share + 1) * q_heads), k1 = min(p.n_kv_heads, (share + 1) * kv_heads);
    auto piece = [](int h0, int h1, int parts, int part, int &first) {   // heads of one of the warps that share tokens
        const int each = (max(0, h1 - h0) + parts - 1) / parts;
        first = h0 + part * each;
        return max(0, min(each, h1 - first));
    };
    Stream w;
    const int qi = 4 * (warp & 1) + oct;
    int q_first, k_first, ki = qi, sl = 0;
    const int nq = piece(share * q_heads, q1, kQkvWarps / 2, warp >> 1, q_first);
    w.q_there = t0 + qi < p.n_tokens;
    w.q = p.q + (t0 + qi) * p.q_stride + q_first * kD + 8 * c;
    w.nq = nq;
    w.nk = 0;
    w.to = smem_u32(sh.ring[warp][0][oct][0]) + 16 * c;
    stream_get<PAGED>(w);
    const bool q_mine = __shfl_sync(0xffffffffu, slot, 1 + qi) >= 0;
    int nk;
    bool pair = false, beyond = false;
    if (!PAGED) {
        nk = piece(share * kv_heads, k1, kQkvWarps / 2, warp >> 1, k_first);
        w.k_mine = q_mine;
    } else {
        // pages: two octets to a token that begins a pair and its partner; without pairs an octet to each token
        const SlotPairs q = slot_pairs(slot, slot >= 0 && slot < p.pool.n_slots, kQkvTokens);
        slot_list(q, sh.list[warp]);
        const bool pairs = (q.pair & q.lead) != 0;
        beyond = q.pair & q.lead & 1u << kQkvTokens;   // with the first token of the block behind
        const int per = pairs ? 2 : 4, groups = max(1, (q.leads + per - 1) / per), parts = kQkvWarps / groups, which = warp / groups;   // (at most four groups)
        const int n = (warp - which * groups) * per + (pairs ? oct >> 1 : oct), e = pairs ? oct & 1 : 0;
        const int lead = n < q.leads ? sh.list[warp][n] : 1;
        pair = n < q.leads && (q.pair >> lead & 1);
        w.k_mine = n < q.leads && (e == 0 || pair);
        ki = lead - 1 + (pair ? e : 0);
        sl = __shfl_sync(0xffffffffu, slot, 1 + ki);
        nk = q.leads > 0 ? piece(share * kv_heads, k1, parts, which, k_first) : 0;
    }
    w.k = p.k + (t0 + ki) * p.k_stride + k_first * kD + 8 * c;
    w.v = p.v + (t0 + ki) * p.v_stride + k_first * kD + 8 * c;
    w.nk = nk;
    if (nq == 0) {   // (the first batch was empty: the next is the first)
        w.to ^= kRowBytes;
        stream_get<PAGED>(w);
    }
    stream_get<PAGED>(w);
    if (turns) {
        auto put = [&](int t, int position) {
            const float2 a = angle_of(rate, position, p.rope.amplitude);
            sh.cosines[t][aj] = a.x;
            sh.sines[t][aj] = a.y;
        };
#pragma unroll
        for (int i = 0; i < kAngles; ++i) put(at0 + i * (kQkvTokens / kAngles), pos[i]);
        if (beyond && at0 == 0) put(kQkvTokens, p.positions[t0 + kQkvTokens]);
    }
    sh.norm[threadIdx.x / kD][threadIdx.x % kD] = weight;
    __syncthreads();
    const float *q_norm = p.q_norm ? sh.norm[0] : nullptr, *k_norm = p.k_norm ? sh.norm[1] : nullptr;
    OctCoef k;
    int at_batch = 0;
    // rows that stay fp16: queries, and keys without pages
    auto rows = [&](int n, uint16_t *dst, bool mine, bool norm) {
        for (; n > 0; n -= kBatch) {
            copy_wait<1>();
            if (ROT == kRotPart) __syncwarp();   // (elsewhere a lane reads what it copied itself)
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (i >= n) break;
                const Oct16 o = oct_turn<ROT>(oct_load<ROT>(sh.ring[warp][i][oct][at_batch], c, n_rot), k, norm, p.eps);
                if (mine) oct_store<ROT>(dst + i * kD, c, n_rot, o);
            }
            dst += kBatch * kD;
            at_batch ^= 1;
            __syncwarp();   // the batch has been read: its place may be filled again
            stream_get<PAGED>(w);
        }
    };
    if (nq > 0) {
        k = oct_coef<ROT>(q_norm, sh.cosines[qi], sh.sines[qi], c, n_rot);
        rows(nq, p.q_out + (t0 + qi) * p.q_out_stride + q_first * kD, q_mine, q_norm != nullptr);
    }
    if (nk == 0) return;
    k = oct_coef<ROT>(k_norm, sh.cosines[ki], sh.sines[ki], c, n_rot);
    if (!PAGED) {
        rows(nk, p.k_out + (t0 + ki) * p.k_out_stride + k_first * kD, w.k_mine, k_norm != nullptr);
        return;
    }
    const OctPlace place = oct_place<VT, KT>(sl & 15, c, pair);
    uint8_t *tile16 = tile_of(p.pool, sl >> p.pool.pshift, k_first, (sl & ((1 << p.pool.pshift) - 1)) >> 4, PageTile<VT, KT>::BYTES);
    const uint32_t head_bytes = (uint32_t)PageTile<VT, KT>::BYTES << (p.pool.pshift - 4);
    for (int n = nk; n > 0; n -= kBatch / 2) {
        copy_wait<1>();
        if (ROT == kRotPart) __syncwarp();
#pragma unroll
        for (int i = 0; i < kBatch / 2; ++i) {
            if (i >= n) break;
            uint16_t *krow = sh.ring[warp][2 * i][oct][at_batch];
            Oct16 o = oct_turn<ROT>(oct_load<ROT>(krow, c, n_rot), k, k_norm != nullptr, p.eps);
            if (ROT == kRotPart) {   // back to neighbours
                __syncwarp();
                oct_store<ROT>(krow, c, n_rot, o);
                __syncwarp();
                o = oct_load<kRotNone>(krow, c, 0);
            }
            oct_put_key<VT, KT>(o, tile16, place, c, w.k_mine);
            oct_put_value<VT, KT>(oct_load<kRotNone>(sh.ring[warp][2 * i + 1][oct][at_batch], c, 0), tile16, place, c, w.k_mine);
            tile16 += head_bytes;
        }
        at_batch ^= 1;
        __syncwarp();
        stream_get<PAGED>(w);
    }
}

// Rows that stay fp16 know no formats.
template <int VT, int KT, bool PAGED>
static void (*qkv_fn(const RopeDesc &r))(QkvParams)
{
    return r.n_rot == 0 ? qkv_kernel<VT, KT, kRotNone, PAGED> : r.pairs ? qkv_kernel<VT, KT, kRotPairs, PAGED>
           : r.n_rot == kD ? qkv_kernel<VT, KT, kRotHalf, PAGED> : qkv_kernel<VT, KT, kRotPart, PAGED>;
}
static void (*qkv_fn(const QkvParams &p, int v_type, int k_type))(QkvParams)
{
    if (!p.paged) return qkv_fn<KVQ_V_Q4_0, KVQ_K_I8, false>(p.rope);
    if (v_type == KVQ_V_Q4_0) return k_type == KVQ_K_F16 ? qkv_fn<KVQ_V_Q4_0, KVQ_K_F16, true>(p.rope) : qkv_fn<KVQ_V_Q4_0, KVQ_K_I8, true>(p.rope);
    return k_type == KVQ_K_F16 ? qkv_fn<KVQ_V_Q8_0, KVQ_K_F16, true>(p.rope) : qkv_fn<KVQ_V_Q8_0, KVQ_K_I8, true>(p.rope);
}

cudaError_t prepare_qkv()
{
    const int rots[4][2] = {{0, 0}, {kD, 1}, {kD, 0}, {64, 0}};
    for (auto &r : rots)
        for (int form = 0; form < 5; ++form) {
            QkvParams p = {};
            p.rope.n_rot = r[0];
            p.rope.pairs = r[1];
            p.paged = form < 4;
            const cudaError_t e = cudaFuncSetAttribute(qkv_fn(p, form & 1, form >> 1 & 1), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(QkvShared));
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}

cudaError_t launch_qkv(const QkvParams &in, int v_type, int k_type, int n_sms, cudaStream_t s, bool pdl)
{
    QkvParams p = in;
    const int tiles = (int)(((long long)p.n_tokens + kQkvTokens - 1) / kQkvTokens);
    const int most = (p.n_q_heads > p.n_kv_heads ? p.n_q_heads : p.n_kv_heads) / 2;
    // Few tokens: shares of the heads, as many as leave so many blocks to each SM.  Another block to an SM costs what
    // about 17 rows of a query head do (what it works out before its first row; a kv head counts as five), so one block
    // until shares get large (32 + 8 heads, single tokens, one / two / three: 256 tokens 4.8 / 5.1 / 6.1 us, 500 tokens
    // 6.9 / 6.8 / 8.5, 700 tokens 10.8 / 8.5 / 9.0; prompts of 1100 tokens 8.3 / 6.5 / 7.1).
    // Many tokens: whole ones in full waves, and the last wave's shared by all SMs (40 + 8 heads, 8192 tokens, two and a
    // quarter waves: 34.7 us, 36.1 uncut, 35.4 at two blocks for every SM; 4096 tokens: 20.1, 21.4, 20.3; 16384: 65, all
    // alike).
    const int room = kQkvBlocks * n_sms, rest = tiles % room, rows = p.n_q_heads + 5 * p.n_kv_heads;
    int chunks = rest ? (n_sms + rest - 1) / rest : 1;
    if (tiles < room) {
        float least = FLT_MAX;
        for (int blocks = 1; blocks <= kQkvBlocks; ++blocks) {
            const int shares = blocks * n_sms / rest;
            const float cost = shares ? (float)rows / shares + 17.f * (blocks - 1) : FLT_MAX;
            if (cost < least) {
                least = cost;
                chunks = shares;
            }
        }
    }
    chunks = chunks > most ? most : chunks;
    p.chunks = chunks < 1 ? 1 : chunks;
    p.full = tiles - rest;
    p.q_heads = (p.n_q_heads + p.chunks - 1) / p.chunks;
    p.kv_heads = (p.n_kv_heads + p.chunks - 1) / p.chunks;
    return launch_pdl(qkv_fn(p, v_type, k_type), p, p.full + rest * p.chunks, kQkvWarps * 32, (int)sizeof(QkvShared), s, pdl);
}

}  // namespace kvq
