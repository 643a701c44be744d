// kvq_paged_small.cu -- page tables, append, gather and the piece combine of
// the paged cache.
#include "kvq_paged.cuh"
#include "kvq_paged_line.cuh"

namespace kvq {

// ---------------------------------------------------------------------------
// Page tables.  Three prefix sums over the sequences (rows, pages given back,
// pages needed) say everything: row t of the batch belongs to the sequence
// whose row range holds it, new page f to the sequence whose range of needed
// pages holds it, and entry v of the stack past the free pages to the released
// sequence whose range holds it.  Every CTA of one cluster computes the sums
// for itself (n_seqs loads, two block scans: cheaper than passing them
// around), the cluster synchronizes once, so that lens and n_free may be
// updated in place, and the outputs are dealt out flat over its threads with
// a binary search each; a warp copies a released sequence's pages.  Latency-bound
// (256 sequences, a row each: 6.2 us; its bytes take 0.1 us): the launch, one
// round of loads, two scans, the cluster's barrier.  One CTA alone instead of
// eight is no faster.  The rows' slots are filled here up to one pass of
// the cluster's threads (16384 rows), beyond that by a second, wide launch:
// 17942 rows 7.15 us here, 6.6 there; 272442 rows 36.8 and 10.5; 7726 rows 5.6
// and 6.6.
// ---------------------------------------------------------------------------
constexpr int kTabThreads = 512;

// Exclusive sums of N values over the block's threads, and the totals.
template <int N>
__device__ __forceinline__ void block_scan(long long (&v)[N], long long (&total)[N], long long (*tmp)[kTabThreads / 32])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x[N];
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = v[k];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const long long y = __shfl_up_sync(0xffffffffu, x[k], d);
            if (lane >= d) x[k] += y;
        }
    __syncthreads();   // tmp may still be read by the previous scan
    if (lane == 31)
#pragma unroll
        for (int k = 0; k < N; ++k) tmp[k][warp] = x[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        long long base = 0;
        total[k] = 0;
#pragma unroll
        for (int w = 0; w < kTabThreads / 32; ++w) {
            if (w < warp) base += tmp[k][w];
            total[k] += tmp[k][w];
        }
        v[k] = base + x[k] - v[k];
    }
}

// Last i in [0, n) with a[i] <= x (a non-decreasing, a[0] <= x).
__device__ __forceinline__ int last_at_most(const int *a, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kTabThreads) page_tables_kernel(const TableParams p)
{
    extern __shared__ int tab[];
    __shared__ long long tmp[2][kTabThreads / 32];
    __shared__ int popped_s;
    const int n = p.n_seqs, tid = threadIdx.x, P = 1 << p.pshift;
    int *qs = tab, *need0 = qs + n + 1, *back0 = need0 + n + 1, *len_s = back0 + n + 1, *add_s = len_s + n;
    uint32_t rank, ranks;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
    const long long lmax = (long long)p.max_blocks << p.pshift;
    pdl_wait();
    pdl_trigger();
    const int n_free = min(max(*p.n_free, 0), p.n_pages);
    if (tid == 0) popped_s = 0x7fffffff;
    // rows and pages given back
    const int per = (n + kTabThreads - 1) / kTabThreads, i0 = min(n, tid * per), i1 = min(n, i0 + per);
    long long rows = 0, back = 0;
    for (int i = i0; i < i1; ++i) {
        const int len = (int)min(max((long long)p.lens[i], 0ll), lmax), add = p.n_new[i];
        len_s[i] = len;
        add_s[i] = add;
        rows += max(add, 0);
        if (add < 0) back += (len + P - 1) >> p.pshift;
    }
    long long first[2] = {rows, back}, all2[2];
    block_scan(first, all2, tmp);
    const long long rows0 = first[0], backs0 = first[1], rows_all = all2[0], back_all = all2[1];
    // pages needed by the sequences that fit their row of the table and the batch
    auto fits = [&](int len, int add, long long end) { return (long long)len + add <= lmax && end <= p.n_tokens; };
    auto pages = [&](int len, int add) { return (int)((((long long)len + add + P - 1) >> p.pshift) - ((len + P - 1) >> p.pshift)); };
    long long need = 0, r = rows0, bk = backs0;
    for (int i = i0; i < i1; ++i) {
        const int len = len_s[i], add = add_s[i];
        qs[i] = (int)min(r, 0x7fffffffll);
        back0[i] = (int)min(bk, 0x7fffffffll);
        r += max(add, 0);
        if (add < 0) bk += (len + P - 1) >> p.pshift;
        if (add > 0 && fits(len, add, r)) need += pages(len, add);
    }
    long long needs[1] = {need}, all1[1];
    block_scan(needs, all1, tmp);
    const long long needs0 = needs[0], need_all = all1[0];
    const int avail = (int)min((long long)n_free + back_all, (long long)p.n_pages);
    // the grant: pages in order, and nothing after the first that does not fit
    long long nd = needs0;
    r = rows0;
    for (int i = i0; i < i1; ++i) {
        const int len = len_s[i], add = add_s[i];
        r += max(add, 0);
        need0[i] = (int)min(nd, 0x7fffffffll);
        if (add > 0 && fits(len, add, r)) {
            const int k = pages(len, add);
            if (k > 0 && nd + k > avail) atomicMin(&popped_s, (int)min(nd, 0x7fffffffll));
            nd += k;
        }
    }
    if (tid == 0) {
        qs[n] = (int)min(rows_all, 0x7fffffffll);
        need0[n] = (int)min(need_all, 0x7fffffffll);
        back0[n] = (int)min(back_all, 0x7fffffffll);
    }
    // every CTA has read lens and n_free; the sums are in place
    asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
    const int popped = min(popped_s, need0[n]), n_free_out = avail - popped;
    // entry v < avail of the stack with the returned pages on top
    auto stack = [&](int v) {
        if (v < n_free) return p.free_pages[v];
        const int x = v - n_free, b = last_at_most(back0, n, x);
        return p.block_table[(size_t)b * p.stride + (x - back0[b])];
    };
    auto granted = [&](int b, int add) {   // of a sequence with add > 0
        const int len = len_s[b];
        if (!fits(len, add, qs[b + 1])) return 2;
        const int k = pages(len, add);
        return k > 0 && (long long)need0[b] + k > popped ? 1 : 0;
    };
    const int at = rank * kTabThreads + tid, all = ranks * kTabThreads;
    for (int b = at; b < n; b += all) {
        const int add = add_s[b], st = add > 0 ? granted(b, add) : 0;
        p.status[b] = st;
        p.lens_out[b] = add < 0 ? 0 : st == 0 ? len_s[b] + add : len_s[b];
    }
    for (int b = at; b <= n; b += all) p.q_start[b] = qs[b];
    if (at == 0) *p.n_free_out = n_free_out;
    for (int f = at; f < popped; f += all) {   // new pages, in order
        const int b = last_at_most(need0, n, f);
        const int j = ((len_s[b] + P - 1) >> p.pshift) + f - need0[b];
        p.block_table[(size_t)b * p.stride + j] = stack(avail - 1 - f);
    }
    // what stays of the returned pages: a warp per released sequence, the warp's sequences asked 32 at a time
    const int warp = at >> 5, warps = all >> 5, lane = tid & 31;
    for (int b0 = warp; b0 < n; b0 += 32 * warps) {
        const int mine = b0 + lane * warps;
        for (unsigned set = __ballot_sync(0xffffffffu, mine < n && add_s[mine] < 0); set; set &= set - 1) {
            const int b = b0 + (__ffs(set) - 1) * warps;
            const long long v0 = (long long)n_free + back0[b];   // past 2^31 if lens claims more pages than there are
            const int m = (int)max(0ll, min((long long)(back0[b + 1] - back0[b]), n_free_out - v0));
            const int *from = p.block_table + (size_t)b * p.stride;
            for (int k0 = lane; k0 < m; k0 += 256) {   // eight loads in flight
                int v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = k0 + 32 * k < m ? from[k0 + 32 * k] : 0;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k0 + 32 * k < m) p.free_pages[v0 + k0 + 32 * k] = v[k];
            }
        }
    }
    if (!p.slots_here) return;
    // slots, four rows a thread: one search, then forward
    const int owned = min(qs[n], p.n_tokens);
    for (int t = 4 * at; t < p.n_tokens; t += 4 * all) {
        int s4[4] = {-1, -1, -1, -1};
        if (t < owned) {
            int b = last_at_most(qs, n, t), st = granted(b, add_s[b]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (t + k >= owned) break;
                if (t + k >= qs[b + 1]) {
                    do ++b;
                    while (t + k >= qs[b + 1]);
                    st = granted(b, add_s[b]);
                }
                if (st) continue;
                const int len = len_s[b], pos = len + (t + k - qs[b]), j = pos >> p.pshift, have = (len + P - 1) >> p.pshift;
                const int page = j < have ? p.block_table[(size_t)b * p.stride + j] : stack(avail - 1 - (need0[b] + j - have));
                if (page >= 0 && page < p.n_pages) s4[k] = (page << p.pshift) + (pos & (P - 1));
            }
        }
        if (t + 4 <= p.n_tokens && (reinterpret_cast<uintptr_t>(p.slots) & 15) == 0)
            *reinterpret_cast<int4 *>(p.slots + t) = make_int4(s4[0], s4[1], s4[2], s4[3]);
        else
            for (int k = 0; k < 4 && t + k < p.n_tokens; ++k) p.slots[t + k] = s4[k];
    }
}

// The slots of many rows, from the tables as page_tables_kernel left them: a
// row's sequence by a search over q_start, four rows a thread.
constexpr int kSlotThreads = 256;

__global__ void __launch_bounds__(kSlotThreads) page_slots_kernel(const TableParams p)
{
    extern __shared__ int qs[];
    const int n = p.n_seqs;
    const long long t0 = 4 * ((long long)blockIdx.x * kSlotThreads + threadIdx.x);
    pdl_wait();
    pdl_trigger();
    for (int i = threadIdx.x; i <= n; i += kSlotThreads) qs[i] = p.q_start[i];
    __syncthreads();
    if (t0 >= p.n_tokens) return;
    const int t = (int)t0, owned = min(qs[n], p.n_tokens), left = p.n_tokens - t;
    int s4[4] = {-1, -1, -1, -1};
    if (t < owned) {
        int b = last_at_most(qs, n, t), at = 0;
        const int *row = nullptr;   // the sequence's table, if its rows were granted
        auto enter = [&]() {
            row = p.status[b] == 0 ? p.block_table + (size_t)b * p.stride : nullptr;
            at = p.lens_out[b] - qs[b + 1];   // position of row t: at + t
        };
        enter();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k >= owned - t) break;
            if (t + k >= qs[b + 1]) {
                do ++b;
                while (t + k >= qs[b + 1]);
                enter();
            }
            if (!row) continue;
            const int pos = at + t + k, page = row[pos >> p.pshift];
            if (page >= 0 && page < p.n_pages) s4[k] = (page << p.pshift) + (pos & ((1 << p.pshift) - 1));
        }
    }
    if (left >= 4 && (reinterpret_cast<uintptr_t>(p.slots) & 15) == 0)
        *reinterpret_cast<int4 *>(p.slots + t) = make_int4(s4[0], s4[1], s4[2], s4[3]);
    else
        for (int k = 0; k < 4 && k < left; ++k) p.slots[t + k] = s4[k];
}

cudaError_t prepare_page_tables()
{
    constexpr int most = (5 * KVQ_MAX_PAGED_SEQS + 3) * (int)sizeof(int);
    static_assert(most <= 100 * 1024, "the sums of every sequence fit in shared memory");
    return cudaFuncSetAttribute(page_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

cudaError_t launch_page_tables(TableParams p, cudaStream_t s, bool pdl)
{
    cudaLaunchConfig_t cfg = {};
    const int ctas = 8;   // the portable cluster size
    p.slots_here = p.n_tokens <= 4 * ctas * kTabThreads;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kTabThreads);
    cfg.dynamicSmemBytes = (5 * (size_t)p.n_seqs + 3) * sizeof(int);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = ctas;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, page_tables_kernel, p);
    if (e != cudaSuccess || p.slots_here) return e;
    return launch_pdl(page_slots_kernel, p, (int)(((long long)p.n_tokens + 4 * kSlotThreads - 1) / (4 * kSlotThreads)), kSlotThreads,
                      (p.n_seqs + 1) * sizeof(int), s, pdl);
}

// ---------------------------------------------------------------------------
// Append and gather work on rows (token, kv head), a warp each, a block eight
// tokens of one head.  Two tokens of the batch side by side whose slots are an
// even place and the next one share their tile's V words and scale words: the
// warp of the first takes both, that of the second leaves.
// ---------------------------------------------------------------------------
constexpr int kRowWarps = 8;

struct RowJob {
    int tok, h, slot;   // slot < 0: nothing to do
    bool pair;          // and token tok + 1, slot + 1
};
__device__ __forceinline__ RowJob row_job(const PagedRowsParams &p)
{
    RowJob r;
    const unsigned group = blockIdx.x / (unsigned)p.pool.n_kv_heads;
    r.h = (int)(blockIdx.x - group * p.pool.n_kv_heads);
    r.tok = (int)(group * kRowWarps + (threadIdx.x >> 5));
    r.pair = false;
    r.slot = -1;
    if (r.tok >= p.n_tokens) return r;
    const int slot = p.slots[r.tok];
    const int before = r.tok > 0 ? p.slots[r.tok - 1] : -1, after = r.tok + 1 < p.n_tokens ? p.slots[r.tok + 1] : -1;
    if (slot < 0 || slot >= p.pool.n_slots) return r;
    if ((slot & 1) && before == slot - 1) return r;
    r.slot = slot;
    r.pair = !(slot & 1) && after == slot + 1;   // pages hold a multiple of 16: the same tile
    return r;
}
static int row_blocks(const PagedRowsParams &p)   // at most 2^28: the callers hold tokens * heads below 2^30
{
    return (p.n_tokens + kRowWarps - 1) / kRowWarps * p.pool.n_kv_heads;
}

// ---------------------------------------------------------------------------
// Append: paged_token's codes into the slot's tile.  It moves 512 bytes in and
// 208 to 400 out per row; at thousands of rows bound by instructions (340 per
// pair) and the latency of two loads in a row, at a decode step's by the
// latency alone.  8192 tokens, 8 heads, q8_0 V: 16.4 us in a chain of calls, 3.1
// TB/s (F16 K 16.7); a row alone with byte stores and a division per value 37.6.
// ---------------------------------------------------------------------------
template <int VT, int KT>
__global__ void __launch_bounds__(kRowWarps * 32) paged_append_kernel(const PagedRowsParams p)
{
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const RowJob r = row_job(p);
    if (r.slot < 0) return;
    const size_t src = (size_t)r.tok * p.stride + (size_t)r.h * kD;
    const int place = r.slot & ((1 << p.pool.pshift) - 1);
    uint8_t *tile = tile_of(p.pool, r.slot >> p.pool.pshift, r.h, place >> 4, PageTile<VT, KT>::BYTES);
    const TokenRow t = paged_token<VT, KT>(p.k16 + src, p.v16 + src, lane);
    if (r.pair) {
        const TokenRow t1 = paged_token<VT, KT>(p.k16 + src + p.stride, p.v16 + src + p.stride, lane);
        store_pair_paged<VT, KT>(t, t1, place & 15, lane, tile);
    } else {
        store_token_paged<VT, KT>(t, place & 15, lane, tile);
    }
}

cudaError_t launch_paged_append(const PagedRowsParams &p, int v_type, int k_type, cudaStream_t s, bool pdl)
{
    void (*fn)(PagedRowsParams) =
        k_type == KVQ_K_F16 ? (v_type == KVQ_V_Q4_0 ? paged_append_kernel<KVQ_V_Q4_0, KVQ_K_F16> : paged_append_kernel<KVQ_V_Q8_0, KVQ_K_F16>)
                            : (v_type == KVQ_V_Q4_0 ? paged_append_kernel<KVQ_V_Q4_0, KVQ_K_I8> : paged_append_kernel<KVQ_V_Q8_0, KVQ_K_I8>);
    return launch_pdl(fn, p, row_blocks(p), kRowWarps * 32, 0, s, pdl);
}

// ---------------------------------------------------------------------------
// Gather, some rows: four values a lane of a row's K and V, for a pair of both
// rows.  64 tokens, 8 heads: 1.6 us, launch latency.  (Many rows are bound by
// instructions here, 140 a row, and go to gather_kernel of kvq_held.cu.)
// ---------------------------------------------------------------------------
template <bool O16>
__device__ __forceinline__ void put4(void *base, size_t elem, const float (&x)[4])
{
    if (O16)
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(base) + elem) = make_uint2(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]));
    else
        *reinterpret_cast<float4 *>(static_cast<float *>(base) + elem) = make_float4(x[0], x[1], x[2], x[3]);
}

// The lane's four values of code bytes w (biased by bias) times s.
__device__ __forceinline__ void scaled4(uint32_t w, int bias, float s, float (&x)[4])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = (float)((int)(w >> (8 * k) & 0xff) - bias) * s;
}

template <int VT, int KT, bool O16>
__global__ void __launch_bounds__(kRowWarps * 32) paged_gather_kernel(const PagedRowsParams p)
{
    using T = PageTile<VT, KT>;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, b = lane >> 3;
    const RowJob r = row_job(p);
    if (r.slot < 0) return;
    const int place = r.slot & ((1 << p.pool.pshift) - 1), u = place & 15, ue = u & ~1;
    const uint8_t *tile = tile_of(p.pool, r.slot >> p.pool.pshift, r.h, place >> 4, T::BYTES);
    // V words and scales of places ue, ue + 1; K of the rows asked for
    const uint8_t *vt = tile + T::V_OFF;
    uint32_t va, vb;
    if (VT == KVQ_V_Q8_0) {
        const uint2 w = *reinterpret_cast<const uint2 *>(vt + v8_pair_off(ue, lane));
        va = __byte_perm(w.x, w.y, 0x6420);
        vb = __byte_perm(w.x, w.y, 0x7531);
    } else {   // bytes 4 (lane % 4) .. + 3 of the block, the low nibbles first
        const uint32_t x = *reinterpret_cast<const uint32_t *>(vt + v4_pair_off(ue, b, 2 * (lane & 3)));
        const uint32_t y = *reinterpret_cast<const uint32_t *>(vt + v4_pair_off(ue, b, 2 * (lane & 3) + 1));
        const int sh = lane & 4;
        va = __byte_perm(x, y, 0x5410) >> sh & 0x0f0f0f0fu;
        vb = __byte_perm(x, y, 0x7632) >> sh & 0x0f0f0f0fu;
    }
    const float2 d = half2_of(*reinterpret_cast<const uint32_t *>(tile + T::VS_OFF + scale_off(ue, b)));
    float2 ks = make_float2(0.f, 0.f);
    if (KT != KVQ_K_F16) ks = half2_of(*reinterpret_cast<const uint32_t *>(tile + T::KS_OFF + scale_off(ue, b)));
    uint32_t k0[2], k1[2];   // row u; row u + 1 of a pair
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (e == 1 && !r.pair) break;
        if (KT == KVQ_K_F16) {
            k0[e] = *reinterpret_cast<const uint32_t *>(tile + k16_tile_off(u + e, 4 * lane));
            k1[e] = *reinterpret_cast<const uint32_t *>(tile + k16_tile_off(u + e, 4 * lane + 2));
        } else {
            k0[e] = *reinterpret_cast<const uint32_t *>(tile + k_tile_off(u + e, 4 * lane));
        }
    }
    size_t dst = ((size_t)r.tok * p.pool.n_kv_heads + r.h) * kD + 4 * lane;
#pragma unroll
    for (int e = 0; e < 2; ++e, dst += (size_t)p.pool.n_kv_heads * kD) {
        if (e == 1 && !r.pair) break;
        const bool odd = (u + e) & 1;
        float x[4];
        if (KT == KVQ_K_F16) {
            const float2 lo = half2_of(k0[e]), hi = half2_of(k1[e]);
            x[0] = lo.x; x[1] = lo.y; x[2] = hi.x; x[3] = hi.y;
        } else {
            scaled4(k0[e], 128, odd ? ks.y : ks.x, x);
        }
        put4<O16>(p.k_out, dst, x);
        scaled4(odd ? vb : va, VT == KVQ_V_Q8_0 ? 128 : 8, odd ? d.y : d.x, x);
        put4<O16>(p.v_out, dst, x);
    }
}

template <bool O16>
static cudaError_t gather_t(const PagedRowsParams &p, int v_type, int k_type, cudaStream_t s, bool pdl)
{
    void (*fn)(PagedRowsParams) =
        k_type == KVQ_K_F16 ? (v_type == KVQ_V_Q4_0 ? paged_gather_kernel<KVQ_V_Q4_0, KVQ_K_F16, O16> : paged_gather_kernel<KVQ_V_Q8_0, KVQ_K_F16, O16>)
                            : (v_type == KVQ_V_Q4_0 ? paged_gather_kernel<KVQ_V_Q4_0, KVQ_K_I8, O16> : paged_gather_kernel<KVQ_V_Q8_0, KVQ_K_I8, O16>);
    return launch_pdl(fn, p, row_blocks(p), kRowWarps * 32, 0, s, pdl);
}

cudaError_t launch_paged_gather(const PagedRowsParams &p, int v_type, int k_type, int out_type, int n_sms, cudaStream_t s, bool pdl)
{
    // Eight rows to a warp from 4096 rows on (8 heads, q8_0 V, fp16 / fp32 output: 512 tokens 2.2 / 2.4 us here and 1.7 /
    // 2.0 there, 256 tokens 1.5 / 1.7 and 1.7 / 2.0).
    if ((long long)p.n_tokens * p.pool.n_kv_heads >= 4096) return launch_gather_many(p, v_type, k_type, out_type, n_sms, s, pdl);
    return out_type == KVQ_OUT_F16 ? gather_t<true>(p, v_type, k_type, s, pdl) : gather_t<false>(p, v_type, k_type, s, pdl);
}

// ---------------------------------------------------------------------------
// Combine: the pieces of the row tiles that several CTAs of an attention launch
// attended, for all launches of a call at once.  The pieces of a tile are
// weighted by exp(lse_i - max lse) / sum; what bounds it is the latency of its
// rounds of loads.  The blocks of CTA i share the merge of the tile its slot 1
// began and of the one its slot 0 went on with, so a tile cut into np pieces is
// merged by np * spread blocks; the chunk launch's tiles of 128 rows have a
// spread that leaves each warp about one row.  Few pieces: a warp per row, the
// pieces one after another.  Many: a block per row, 16 dims to a warp, eight
// pieces side by side in its lanes, joined by shuffles.  Both orders are fixed
// by the lengths alone.  Four loads in flight at 64 registers measured better
// than eight at 80: more blocks fit beside the attention's last CTAs (512-token
// chunk over 32768 positions: 463 against 466 us for the whole call).
// ---------------------------------------------------------------------------
constexpr int kPcWarps = 8;
constexpr int kPcFew = 8;    // pieces up to which a warp takes a row alone
constexpr int kPcLoads = 4;  // pieces in flight per lane

struct Merged {
    float m, w;
    float4 o;
    bool poisoned;

    __device__ __forceinline__ Merged() : m(-INFINITY), w(0.f), o(make_float4(0.f, 0.f, 0.f, 0.f)), poisoned(false) {}
    // joins weight w2 at maximum m2, with its sums
    __device__ __forceinline__ void join(float m2, float w2, const float4 &v)
    {
        if (!(m2 > -INFINITY)) return;
        const float mx = fmaxf(m, m2);
        const float f = m == -INFINITY ? 0.f : expf(m - mx), e = expf(m2 - mx);
        w = fmaf(w, f, w2 * e);
        o.x = fmaf(e, v.x, o.x * f);
        o.y = fmaf(e, v.y, o.y * f);
        o.z = fmaf(e, v.z, o.z * f);
        o.w = fmaf(e, v.w, o.w * f);
        m = mx;
    }
};

// Pieces first, first + step, ... of a row, four dims from d on.
__device__ __forceinline__ Merged merge_pieces(const PagedPieces &g, const PagedCut &c, int r, int first, int step, int d)
{
    Merged a;
    for (int k0 = first; k0 < c.np; k0 += kPcLoads * step) {
        float lv[kPcLoads];
        float4 v[kPcLoads];
#pragma unroll
        for (int k = 0; k < kPcLoads; ++k) {
            const int j = k0 + k * step;
            lv[k] = -INFINITY;
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j < c.np) {
                const size_t at = ((size_t)(c.c0 + j) * 2 + (j == 0 ? 1 : 0)) * g.rows + r;
                lv[k] = g.lse[at];
                v[k] = *reinterpret_cast<const float4 *>(g.o + at * kD + d);
            }
        }
#pragma unroll
        for (int k = 0; k < kPcLoads; ++k) {
            a.poisoned |= lv[k] != lv[k];   // a piece whose CTA lost a copy: the row is NaN
            a.join(lv[k], 1.f, v[k]);
        }
    }
    return a;
}

template <bool O16>
__device__ __forceinline__ void put_merged(const PagedAttnParams &p, size_t row, const Merged &a, int d)
{
    const float nan = __int_as_float(0x7fc00000);
    const bool any = a.w > 0.f;
    const float inv = a.poisoned ? nan : any ? 1.f / a.w : 0.f;
    const float x[4] = {a.o.x * inv, a.o.y * inv, a.o.z * inv, a.o.w * inv};
    put4<O16>(p.out, row * kD + d, x);
    if (d == 0 && p.lse) p.lse[row] = a.poisoned ? nan : any ? a.m + logf(a.w) : -INFINITY;
}

template <bool O16>
__global__ void __launch_bounds__(kPcWarps * 32, 4) paged_combine_kernel(const __grid_constant__ PagedAttnParams p,
                                                                      const __grid_constant__ PagedCuts cuts)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int block = blockIdx.x, k = 0;
    while (k < kAttnParts - 1 && block >= cuts.part[k].ctas * cuts.part[k].spread) block -= cuts.part[k].ctas * cuts.part[k].spread, ++k;
    const PagedPieces &g = cuts.part[k];
    const int cta = block / g.spread;
    pdl_wait();
    pdl_trigger();
    for (int slot = 0; slot < 2; ++slot) {
        const PagedCut c = g.cuts[(size_t)cta * 2 + slot];
        if (c.np < 2) continue;   // block-uniform
        const int h = c.h_rt & 255, rt = c.h_rt >> 8;
        const int share = (cta - c.c0) * g.spread + block % g.spread, shares = c.np * g.spread;
        int t0, n, len, lim0;
        seq_shape(p, c.b, t0, n, len, lim0);
        const int gb = p.grp_begin[h], gsz = p.grp_begin[h + 1] - gb;
        const int row0 = rt * g.rows, R = min(g.rows, n * gsz - row0);
        auto out_row = [&](int r) {
            return (size_t)(t0 + (row0 + r) / gsz) * p.n_q_heads + p.grp_q[gb + (row0 + r) % gsz];
        };
        if (c.np <= kPcFew) {
            for (int r = share * kPcWarps + warp; r < R; r += shares * kPcWarps)
                put_merged<O16>(p, out_row(r), merge_pieces(g, c, r, 0, 1, 4 * lane), 4 * lane);
        } else {
            const int d = kD / kPcWarps * warp + 4 * (lane & 3);
            for (int r = share; r < R; r += shares) {
                Merged a = merge_pieces(g, c, r, lane >> 2, 8, d);
                a.poisoned = __any_sync(0xffffffffu, a.poisoned);
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) {
                    float4 v;
                    v.x = __shfl_xor_sync(0xffffffffu, a.o.x, k);
                    v.y = __shfl_xor_sync(0xffffffffu, a.o.y, k);
                    v.z = __shfl_xor_sync(0xffffffffu, a.o.z, k);
                    v.w = __shfl_xor_sync(0xffffffffu, a.o.w, k);
                    const float m2 = __shfl_xor_sync(0xffffffffu, a.m, k), w2 = __shfl_xor_sync(0xffffffffu, a.w, k);
                    a.join(m2, w2, v);
                }
                if (lane < 4) put_merged<O16>(p, out_row(r), a, d);
            }
        }
    }
}

cudaError_t launch_paged_combine(const PagedAttnParams &p, const PagedCuts &cuts, int out_type, cudaStream_t s, bool pdl)
{
    int blocks = 0;
    for (const PagedPieces &g : cuts.part) blocks += g.ctas * g.spread;
    if (blocks == 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kPcWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (out_type == KVQ_OUT_F16) return cudaLaunchKernelEx(&cfg, paged_combine_kernel<true>, p, cuts);
    return cudaLaunchKernelEx(&cfg, paged_combine_kernel<false>, p, cuts);
}

}  // namespace kvq
