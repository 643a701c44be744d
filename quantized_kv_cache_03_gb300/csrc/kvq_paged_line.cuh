// kvq_paged_line.cuh -- what both paged attention kernels share: the V code
// conversion and the split of a batch's line of work over the CTAs.
#pragma once

#include "kvq_paged.cuh"

namespace kvq {

// Two signed int8 codes (bytes k0, k0 + 1 of w) as an exact fp16 pair.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int k0)
{
    const __half2 h = __halves2half2(__int2half_rn((int)(int8_t)(w >> (8 * k0))), __int2half_rn((int)(int8_t)(w >> (8 * k0 + 8))));
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 half2_of(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }

// (a & mask) | bits in one instruction (left to itself the compiler uses two,
// each with a constant of its own).
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t bits)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(mask), "r"(bits));
    return r;
}

// V A-fragment registers of one 32-block for the position pair (t, t + 1):
// reg[h2][half] = the exact codes of head dim g + 8 half of m-tile 2 bb + h2
// (dims as pv_dim: q4_0 32bb + 16h2 + 2g + half, q8_0 32bb + 4g + 2h2 + half).
template <int VT>
__device__ __forceinline__ void v_codes(uint32_t w0, uint32_t w1, uint32_t (&reg)[2][2])
{
    auto h2 = [](uint32_t x) { return *reinterpret_cast<__half2 *>(&x); };
    auto put = [](uint32_t &r, __half2 v) { r = *reinterpret_cast<uint32_t *>(&v); };
    if (VT == KVQ_V_Q4_0) {   // nibbles under the exponent of 1024, minus 1032; high ones weigh 16
        const __half2 k1032 = __half2half2(__ushort_as_half(0x6408)), k16th = __half2half2(__ushort_as_half(0x2c00)),
                      km72 = __half2half2(__ushort_as_half(0xd480));
        const uint32_t w8 = w0 >> 8;
        put(reg[0][0], __hsub2(h2(and_or(w0, 0x000F000Fu, 0x64006400u)), k1032));
        put(reg[0][1], __hsub2(h2(and_or(w8, 0x000F000Fu, 0x64006400u)), k1032));
        put(reg[1][0], __hfma2(h2(and_or(w0, 0x00F000F0u, 0x64006400u)), k16th, km72));
        put(reg[1][1], __hfma2(h2(and_or(w8, 0x00F000F0u, 0x64006400u)), k16th, km72));
    } else {                  // code + 128 under the exponent of 1024, minus 1152
        const __half2 k1152 = __half2half2(__ushort_as_half(0x6480));
        put(reg[0][0], __hsub2(h2(__byte_perm(w0, 0x64646464u, 0x4140)), k1152));
        put(reg[0][1], __hsub2(h2(__byte_perm(w0, 0x64646464u, 0x4342)), k1152));
        put(reg[1][0], __hsub2(h2(__byte_perm(w1, 0x64646464u, 0x4140)), k1152));
        put(reg[1][1], __hsub2(h2(__byte_perm(w1, 0x64646464u, 0x4342)), k1152));
    }
}
template <int VT>
__device__ __forceinline__ int v_dim(int mt, int g)   // the pair's first dim: half 0 of m-tile mt
{
    return VT == KVQ_V_Q4_0 ? 32 * (mt >> 1) + 16 * (mt & 1) + 2 * g : 32 * (mt >> 1) + 4 * g + 2 * (mt & 1);
}

// Where a CTA's piece of the line of stages begins: scanned by the whole block.
struct LineStart {
    int b;               // first sequence with work at or after the start
    long long off;       // stages into it
    long long total;     // stages of the line
};

// stages(n, len, lim0): the sequence's stages over all kv heads and row tiles.
template <int THREADS, typename F>
__device__ __forceinline__ void line_find(const PagedAttnParams &p, long long gmin, F stages, LineStart *res,
                                          long long *tmp, long long &begin, long long &per)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int each = (p.n_seqs + THREADS - 1) / THREADS, i0 = min(p.n_seqs, tid * each), i1 = min(p.n_seqs, i0 + each);
    long long sum = 0;
    for (int i = i0; i < i1; ++i) {
        int t0, n, len, lim0;
        seq_shape(p, i, t0, n, len, lim0);
        if (seq_mine(p, n)) sum += stages(n, len, lim0);
    }
    long long x = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) tmp[warp] = x;
    __syncthreads();
    long long base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) base += tmp[w];
        total += tmp[w];
    }
    per = max(gmin, (total + gridDim.x - 1) / gridDim.x);
    begin = per * blockIdx.x;
    long long at = base + x - sum;
    if (begin >= at && begin < at + sum)
        for (int i = i0; i < i1; ++i) {
            int t0, n, len, lim0;
            seq_shape(p, i, t0, n, len, lim0);
            const long long s = seq_mine(p, n) ? stages(n, len, lim0) : 0;
            if (begin < at + s) {
                res->b = i;
                res->off = begin - at;
                break;
            }
            at += s;
        }
    if (tid == 0) res->total = total;
    __syncthreads();
}

}  // namespace kvq
