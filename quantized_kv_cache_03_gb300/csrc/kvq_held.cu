// kvq_held.cu -- what the paged cache holds: positions of a step's rows, tables
// forked, pages copied, tokens moved and their keys turned.
#include "kvq_paged_line.cuh"
#include "kvq_tokens.cuh"

namespace kvq {

// ---------------------------------------------------------------------------
// Positions: a row's sequence by a search over q_start in shared memory, four
// rows a thread.
// ---------------------------------------------------------------------------
constexpr int kPosThreads = 256;

__global__ void __launch_bounds__(kPosThreads) positions_kernel(const PositionsParams p)
{
    extern __shared__ int qs[];
    const int n = p.n_seqs;
    pdl_wait();
    pdl_trigger();
    for (int i = threadIdx.x; i <= n; i += kPosThreads) qs[i] = min(max(p.q_start[i], 0), p.n_tokens);
    __syncthreads();
    const long long t0 = 4 * ((long long)blockIdx.x * kPosThreads + threadIdx.x);
    int lo = 0, end = 0, base = 0;   // the sequence of the row before, its end and the position of row 0 in it
    bool known = false;
    for (int k = 0; k < 4 && t0 + k < p.n_tokens; ++k) {
        const int t = (int)t0 + k;
        int pos = -1;
        if (t >= qs[0] && t < qs[n]) {
            if (!known || t >= end) {
                int a = known ? lo : 0, b = n;   // last sequence that begins at t or before
                while (b - a > 1) {
                    const int mid = (a + b) >> 1;
                    if (qs[mid] <= t) a = mid;
                    else b = mid;
                }
                lo = a;
                end = qs[a + 1];
                base = (int)((unsigned)p.lens[a] - (unsigned)end);
                known = true;
            }
            pos = (int)((unsigned)base + (unsigned)t);
        }
        p.positions[t] = pos;
    }
}

cudaError_t launch_positions(const PositionsParams &p, cudaStream_t s, bool pdl)
{
    const int per = 4 * kPosThreads;
    return launch_pdl(positions_kernel, p, (int)(((long long)p.n_tokens + per - 1) / per), kPosThreads, (p.n_seqs + 1) * (int)sizeof(int), s, pdl);
}

// ---------------------------------------------------------------------------
// Fork.  Whether a page is given back, and whether a row may go on writing into
// its last page, depends on every row's list, so the work is three launches: the
// marks are cleared, the lists are marked and the rows copied, and one cluster
// counts what is marked old and not new, pushes it in order and deals out pages
// for copies.  Marks are bytes, stored without reading (any number of rows may
// mark a page); the first place that ends inside a page is a minimum: nothing
// depends on an order.
// ---------------------------------------------------------------------------
struct ForkRow {
    int from, keep;   // old row (-1: none), positions kept
};
__device__ __forceinline__ int old_len(const ForkParams &p, int b)
{
    return (int)min(max((long long)p.lens[b], 0ll), (long long)p.max_blocks << p.pshift);
}
__device__ __forceinline__ ForkRow fork_row(const ForkParams &p, int b)
{
    ForkRow r;
    r.from = p.parent ? p.parent[b] : b;
    if (r.from < 0 || r.from >= p.n_seqs) r.from = -1;
    r.keep = r.from < 0 ? 0 : old_len(p, r.from);
    if (p.keep) r.keep = max(0, min(r.keep, p.keep[b]));
    return r;
}
__device__ __forceinline__ bool is_page(const ForkParams &p, int page) { return page >= 0 && page < p.n_pages; }

__global__ void __launch_bounds__(256) fork_clear_kernel(const ForkParams p)
{
    pdl_wait();
    pdl_trigger();
    const long long at = (long long)blockIdx.x * 256 + threadIdx.x, all = (long long)gridDim.x * 256;
    const long long words = ((long long)(p.full_mark - p.old_mark)) * 3 / 16;   // the three marks lie side by side
    for (long long i = at; i < words; i += all) reinterpret_cast<uint4 *>(p.old_mark)[i] = make_uint4(0, 0, 0, 0);
    for (long long b = at; b < p.n_seqs; b += all) {
        const ForkRow r = fork_row(p, (int)b);
        p.kept[b] = r.keep;
        if ((r.keep & ((1 << p.pshift) - 1)) == 0) continue;
        const int tail = p.table[(size_t)r.from * p.stride + (r.keep >> p.pshift)];
        p.tail[b] = tail;
        if (is_page(p, tail)) p.owner[tail] = p.n_seqs;
    }
}

constexpr int kForkRun = 1024;   // entries of a row that a block takes

__global__ void __launch_bounds__(256) fork_mark_kernel(const ForkParams p)
{
    pdl_wait();
    pdl_trigger();
    const int runs = (p.max_blocks + kForkRun - 1) / kForkRun;
    const int b = blockIdx.x / runs, e0 = (blockIdx.x - b * runs) * kForkRun, P = 1 << p.pshift;
    const ForkRow r = fork_row(p, b);
    const int olds = (old_len(p, b) + P - 1) >> p.pshift, whole = r.keep >> p.pshift, used = (r.keep + P - 1) >> p.pshift;
    const int *old_row = p.table + (size_t)b * p.stride, *row = p.table + (size_t)max(r.from, 0) * p.stride;
    int *out = p.table_out + (size_t)b * p.out_stride;
    const bool same = out == row;   // in place: the entries are there
#pragma unroll
    for (int k = 0; k < kForkRun / 256; ++k) {
        const int e = e0 + k * 256 + (int)threadIdx.x;
        if (e < olds) {
            const int page = old_row[e];
            if (is_page(p, page)) p.old_mark[page] = 1;
        }
        if (e < used) {
            const int page = row[e];
            if (e < whole) {
                if (!same) out[e] = page;
                if (is_page(p, page)) p.full_mark[page] = 1;
            } else if (is_page(p, page)) {   // (its entry is written once it is known which page the row ends in)
                p.tail_mark[page] = 1;
                atomicMin(p.owner + page, b);
            }
        }
    }
}

// Exclusive sum over the block's threads, and the total.
__device__ __forceinline__ int fork_scan(int x, int &total, int *tmp)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int y = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, d);
        if (lane >= d) y += z;
    }
    __syncthreads();   // tmp may still be read by the scan before
    if (lane == 31) tmp[warp] = y;
    __syncthreads();
    int base = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kForkThreads / 32; ++w) {
        if (w < warp) base += tmp[w];
        total += tmp[w];
    }
    return base + y - x;
}

__device__ __forceinline__ void cluster_sync() { asm volatile("barrier.cluster.arrive;\n barrier.cluster.wait;" ::: "memory"); }

__global__ void __cluster_dims__(kForkCtas, 1, 1) __launch_bounds__(kForkThreads) fork_deal_kernel(const ForkParams p)
{
    __shared__ int tmp[kForkThreads / 32];
    const int tid = threadIdx.x, rank = blockIdx.x, P = 1 << p.pshift;
    pdl_wait();
    pdl_trigger();
    const int n_free = min(max(*p.n_free, 0), p.n_pages);
    // a thread's pages: a run of 16-byte words of marks
    const int words = (p.n_pages + 15) / 16, per = (words + kForkCtas * kForkThreads - 1) / (kForkCtas * kForkThreads);
    const int w0 = (int)min((long long)words, (long long)(rank * kForkThreads + tid) * per), w1 = min(words, w0 + per);
    auto gone = [&](int w) {   // a bit per byte: listed before and not now (marks past the last page are clear)
        const uint4 o = reinterpret_cast<const uint4 *>(p.old_mark)[w], f = reinterpret_cast<const uint4 *>(p.full_mark)[w],
                    t = reinterpret_cast<const uint4 *>(p.tail_mark)[w];
        return make_uint4(o.x & ~(f.x | t.x), o.y & ~(f.y | t.y), o.z & ~(f.z | t.z), o.w & ~(f.w | t.w));
    };
    int n = 0;
    for (int w = w0; w < w1; ++w) {
        const uint4 g = gone(w);
        n += __popc(g.x) + __popc(g.y) + __popc(g.z) + __popc(g.w);
    }
    int mine;
    const int first = fork_scan(n, mine, tmp);
    if (tid == 0) p.counts[rank] = mine;
    cluster_sync();
    int before = 0, back = 0;
#pragma unroll
    for (int k = 0; k < kForkCtas; ++k) {
        const int c = __ldcg(p.counts + k);
        before += k < rank ? c : 0;
        back += c;
    }
    const int avail = (int)min((long long)n_free + back, (long long)p.n_pages);
    long long at = (long long)n_free + before + first;
    if (n > 0)
        for (int w = w0; w < w1; ++w) {
            const uint4 g = gone(w);
            const uint32_t v[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                for (uint32_t bits = v[k]; bits; bits &= bits - 1) {
                    if (at < p.n_pages) p.free_pages[at] = 16 * w + 4 * k + (__ffs(bits) >> 3);
                    ++at;
                }
        }
    cluster_sync();   // the stack is whole
    if (rank != 0) return;
    // pages for copies, in order of place
    const int each = (p.n_seqs + kForkThreads - 1) / kForkThreads, b0 = min(p.n_seqs, tid * each), b1 = min(p.n_seqs, b0 + each);
    auto shared_tail = [&](int b, int kept) {   // the row ends inside a page that it may not write to
        if ((kept & (P - 1)) == 0) return false;
        const int page = p.tail[b];
        return is_page(p, page) && (p.full_mark[page] || p.owner[page] != b);
    };
    int need = 0;
    for (int b = b0; b < b1; ++b) need += shared_tail(b, p.kept[b]);
    int needs;
    int rank_of = fork_scan(need, needs, tmp);
    for (int b = b0; b < b1; ++b) {
        int kept = p.kept[b], from = -1, to = -1, held = 0, st = 0;
        const bool in_part = (kept & (P - 1)) != 0, shared = shared_tail(b, kept);
        int *entry = p.table_out + (size_t)b * p.out_stride + (kept >> p.pshift);
        if (shared && rank_of < avail) {
            from = p.tail[b];
            to = __ldcg(p.free_pages + (avail - 1 - rank_of));
            held = kept & (P - 1);
            *entry = to;
        } else if (shared) {
            kept &= ~(P - 1);
            st = 1;
        } else if (in_part) {
            *entry = p.tail[b];
        }
        rank_of += shared;
        p.copy_from[b] = from;
        p.copy_to[b] = to;
        p.copy_held[b] = held;
        p.status[b] = st;
        p.lens_out[b] = kept;
    }
    if (tid == 0) *p.n_free_out = avail - min(needs, avail);
}

cudaError_t launch_page_fork(const ForkParams &p, cudaStream_t s, bool pdl)
{
    const long long words = ((long long)(p.full_mark - p.old_mark)) * 3 / 16;
    const long long items = words > p.n_seqs ? words : p.n_seqs;
    const int clear = (int)(items / 256 + 1 < 608 ? items / 256 + 1 : 608);
    cudaError_t e = launch_pdl(fork_clear_kernel, p, clear, 256, 0, s, pdl);
    const long long runs = (p.max_blocks + kForkRun - 1) / kForkRun;
    if (e == cudaSuccess && p.n_seqs * runs > 0) e = launch_pdl(fork_mark_kernel, p, (int)(p.n_seqs * runs), 256, 0, s, pdl);
    if (e == cudaSuccess) e = launch_pdl(fork_deal_kernel, p, kForkCtas, kForkThreads, 0, s, pdl);
    return e;
}

// ---------------------------------------------------------------------------
// Copy: a block takes one head of one page in one pool, whose tiles are one run
// of bytes.
// ---------------------------------------------------------------------------
constexpr int kCopyThreads = 128;
constexpr int kCopyLoads = 8;

__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const __grid_constant__ CopyParams p)
{
    pdl_wait();
    pdl_trigger();
    const unsigned pool = blockIdx.y, i = blockIdx.x / (unsigned)p.most_heads, h = blockIdx.x - i * p.most_heads, heads = p.heads[pool];
    if (h >= heads) return;
    const int from = p.from[i], to = p.to[i];
    if (from < 0 || to < 0 || from >= p.n_pages || to >= p.n_pages || from == to) return;
    int tiles = p.tiles;
    if (p.held) tiles = min(tiles, (int)(((long long)max(p.held[i], 0) + 15) >> 4));
    const int n = tiles * (p.tile_bytes[pool] / 16);
    const size_t run = (size_t)p.tiles * p.tile_bytes[pool];
    const uint4 *src = reinterpret_cast<const uint4 *>(p.data[pool] + ((size_t)from * heads + h) * run);
    uint4 *dst = reinterpret_cast<uint4 *>(p.data[pool] + ((size_t)to * heads + h) * run);
    for (int k0 = threadIdx.x; k0 < n; k0 += kCopyThreads * kCopyLoads) {
        uint4 v[kCopyLoads];
#pragma unroll
        for (int k = 0; k < kCopyLoads; ++k)
            if (k0 + k * kCopyThreads < n) v[k] = src[k0 + k * kCopyThreads];
#pragma unroll
        for (int k = 0; k < kCopyLoads; ++k)
            if (k0 + k * kCopyThreads < n) dst[k0 + k * kCopyThreads] = v[k];
    }
}

cudaError_t launch_page_copy(const CopyParams &p, cudaStream_t s, bool pdl)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.n_copies * p.most_heads, p.n_pools);
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, page_copy_kernel, p);
}

// ---------------------------------------------------------------------------
// Move: a warp takes a token (four values a lane), or two whose new slots are an
// even place and the next, which share words of V codes and scales.
// ---------------------------------------------------------------------------
constexpr int kMoveWarps = 8;

// The row at place u of a tile, as paged_token would give it.
template <int VT, int KT>
__device__ __forceinline__ TokenRow load_token_paged(const uint8_t *tile, int u, int lane, bool want_v)
{
    using T = PageTile<VT, KT>;
    TokenRow t;
    const int b = lane >> 3, ue = u & ~1;
    t.kw = *reinterpret_cast<const uint32_t *>(tile + (KT == KVQ_K_F16 ? k16_tile_off(u, 4 * lane) : k_tile_off(u, 4 * lane)));
    t.kw2 = KT == KVQ_K_F16 ? *reinterpret_cast<const uint32_t *>(tile + k16_tile_off(u, 4 * lane + 2)) : 0;
    t.ks = KT == KVQ_K_F16 ? 0 : *reinterpret_cast<const uint16_t *>(tile + T::KS_OFF + scale_off(u, b));
    t.vw = 0;
    t.vs = 0;
    if (!want_v) return t;
    const uint8_t *vt = tile + T::V_OFF;
    if (VT == KVQ_V_Q8_0) {
        const uint2 w = *reinterpret_cast<const uint2 *>(vt + v8_pair_off(ue, lane));
        t.vw = __byte_perm(w.x, w.y, u & 1 ? 0x7531 : 0x6420);
    } else {
        const uint32_t x = *reinterpret_cast<const uint32_t *>(vt + v4_pair_off(ue, b, 2 * (lane & 3)));
        const uint32_t y = *reinterpret_cast<const uint32_t *>(vt + v4_pair_off(ue, b, 2 * (lane & 3) + 1));
        t.vw = __byte_perm(x, y, u & 1 ? 0x7632 : 0x5410);
    }
    t.vs = *reinterpret_cast<const uint16_t *>(tile + T::VS_OFF + scale_off(u, b));
    return t;
}

// A lane's part in a rotation: four values of which the other half of each pair is
// its own (pairs side by side) or those of lane `other`.
struct MoveTurn {
    float2 cs[4];
    int other;
    bool rotates, second;
    template <int PAIRS>
    __device__ __forceinline__ void set(const RopeDesc &r, int pos, int lane)
    {
        const int h4 = r.n_rot >> 3;   // lanes of first values
        rotates = lane < 2 * h4;
        second = !PAIRS && lane >= h4;
        other = PAIRS || !rotates ? lane : second ? lane - h4 : lane + h4;
#pragma unroll
        for (int i = 0; i < (PAIRS ? 2 : 4); ++i)
            cs[i] = rotates ? angle_of(r.turns[PAIRS ? 2 * lane + i : 4 * (second ? other : lane) + i], pos, 1.f) : make_float2(1.f, 0.f);
    }
};

template <int KT, int PAIRS>
__device__ __forceinline__ void turn_key(TokenRow &t, const MoveTurn &m, const RopeDesc &r, int lane)
{
    auto values = [&](uint32_t w, uint32_t w2, float s, float (&x)[4]) {
        if (KT == KVQ_K_F16) {
            const float2 a = half2_of(w), b = half2_of(w2);
            x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = (float)((int)(w >> (8 * k) & 0xff) - 128) * s;
        }
    };
    const float s = __half2float(__ushort_as_half(t.ks));
    float x[4], y[4];
    values(t.kw, t.kw2, s, x);
    if (PAIRS) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            y[2 * i] = x[2 * i] * m.cs[i].x - x[2 * i + 1] * m.cs[i].y;
            y[2 * i + 1] = x[2 * i] * m.cs[i].y + x[2 * i + 1] * m.cs[i].x;
        }
    } else {
        float o[4];
        const uint32_t w = __shfl_sync(0xffffffffu, t.kw, m.other), w2 = KT == KVQ_K_F16 ? __shfl_sync(0xffffffffu, t.kw2, m.other) : 0;
        values(w, w2, KT == KVQ_K_F16 ? 0.f : __shfl_sync(0xffffffffu, s, m.other), o);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = m.second ? o[i] * m.cs[i].y + x[i] * m.cs[i].x : x[i] * m.cs[i].x - o[i] * m.cs[i].y;
    }
    const uint32_t a = pack_half2(y[0], y[1]), b = pack_half2(y[2], y[3]);
    if (KT == KVQ_K_F16) {
        if (m.rotates) t.kw = a, t.kw2 = b;
        return;
    }
    // values of the block that do not rotate are code * scale, rounded like the others
    auto h2 = [](uint32_t w) { return *reinterpret_cast<const __half2 *>(&w); };
    const uint32_t a1 = m.rotates ? a : pack_half2(x[0], x[1]), b1 = m.rotates ? b : pack_half2(x[2], x[3]);
    __half2 top = __hmax2(h2(a1 & 0x7fff7fffu), h2(b1 & 0x7fff7fffu));
    top = __hmax2(top, __lowhigh2highlow(top));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        const uint32_t z = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<const uint32_t *>(&top), o);
        top = __hmax2(top, h2(z));
    }
    const __half sn = __float2half_rn(__low2float(top) * (1.f / 127.f));
    const uint32_t codes = codes4(a1, b1, __half2float(sn), -127.f, 127.f, 128);
    if ((lane & ~7) * 4 < r.n_rot) {   // the block holds a value that rotates
        t.kw = codes;
        t.ks = __half_as_ushort(sn);
    }
}

// Which half of the way: from slots to slots, from slots to the staged rows, from those to slots.
constexpr int kMoveDirect = 0, kMoveOut = 1, kMoveIn = 2;

template <int VT, int KT>
__device__ __forceinline__ void stage_row(uint8_t *row, const TokenRow &t, int lane)
{
    if (KT == KVQ_K_F16) reinterpret_cast<uint2 *>(row)[lane] = make_uint2(t.kw, t.kw2);
    else reinterpret_cast<uint32_t *>(row)[lane] = t.kw;
    row += KT == KVQ_K_F16 ? 256 : 128;
    if (VT == KVQ_V_Q8_0) reinterpret_cast<uint32_t *>(row)[lane] = t.vw;
    else if ((lane & 7) < 4) reinterpret_cast<uint32_t *>(row)[(lane >> 3) * 4 + (lane & 3)] = t.vw;
    row += VT == KVQ_V_Q8_0 ? 128 : 64;
    if ((lane & 7) == 0) {
        if (KT != KVQ_K_F16) reinterpret_cast<uint16_t *>(row)[4 + (lane >> 3)] = t.ks;
        reinterpret_cast<uint16_t *>(row)[lane >> 3] = t.vs;
    }
}
template <int VT, int KT>
__device__ __forceinline__ TokenRow unstage_row(const uint8_t *row, int lane)
{
    TokenRow t;
    if (KT == KVQ_K_F16) {
        const uint2 w = reinterpret_cast<const uint2 *>(row)[lane];
        t.kw = w.x;
        t.kw2 = w.y;
    } else {
        t.kw = reinterpret_cast<const uint32_t *>(row)[lane];
        t.kw2 = 0;
    }
    row += KT == KVQ_K_F16 ? 256 : 128;
    t.vw = reinterpret_cast<const uint32_t *>(row)[VT == KVQ_V_Q8_0 ? lane : (lane >> 3) * 4 + (lane & 3)];
    row += VT == KVQ_V_Q8_0 ? 128 : 64;
    t.ks = KT == KVQ_K_F16 ? 0 : reinterpret_cast<const uint16_t *>(row)[4 + (lane >> 3)];
    t.vs = reinterpret_cast<const uint16_t *>(row)[lane >> 3];
    return t;
}

template <int VT, int KT, int PAIRS, int WAY>
__global__ void __launch_bounds__(kMoveWarps * 32) move_kernel(const MoveParams p)
{
    using T = PageTile<VT, KT>;
    constexpr int kRow = T::BYTES / kWTile;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned token_blocks = (unsigned)(p.n_tokens + kMoveWarps - 1) / kMoveWarps;
    const int c = blockIdx.x / token_blocks, tok = (int)(blockIdx.x - c * token_blocks) * kMoveWarps + warp;
    if (tok >= p.n_tokens) return;
    auto inside = [&](int slot) { return slot >= 0 && slot < p.pool.n_slots; };
    auto moves = [&](int i) { return i >= 0 && i < p.n_tokens && inside(p.from[i]) && inside(p.to[i]); };
    if (!moves(tok)) return;
    const int to = p.to[tok];
    if ((to & 1) && tok > 0 && p.to[tok - 1] == to - 1 && moves(tok - 1)) return;   // the warp before takes it
    const bool pair = !(to & 1) && tok + 1 < p.n_tokens && p.to[tok + 1] == to + 1 && moves(tok + 1);
    int from[2] = {p.from[tok], pair ? p.from[tok + 1] : -1}, turn[2] = {0, 0};
    MoveTurn m[2];
    if (WAY != kMoveIn && p.turn) {
        turn[0] = p.turn[tok];
        if (pair) turn[1] = p.turn[tok + 1];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            if (turn[e] != 0) m[e].template set<PAIRS>(p.rope, turn[e], lane);
    }
    const int P1 = (1 << p.pool.pshift) - 1;
    const bool still = WAY == kMoveDirect && from[0] == to && (!pair || from[1] == to + 1);   // only keys change
    if (still && turn[0] == 0 && turn[1] == 0) return;
    const int h1 = min(p.pool.n_kv_heads, (c + 1) * p.heads);
    for (int h = c * p.heads; h < h1; ++h) {
        TokenRow t[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (e == 1 && !pair) break;
            if (WAY == kMoveIn) {
                t[e] = unstage_row<VT, KT>(p.rows + ((size_t)(tok + e) * p.pool.n_kv_heads + h) * kRow, lane);
                continue;
            }
            const int place = from[e] & P1;
            t[e] = load_token_paged<VT, KT>(tile_of(p.pool, from[e] >> p.pool.pshift, h, place >> 4, T::BYTES), place & 15, lane, !still);
            if (turn[e] != 0) turn_key<KT, PAIRS>(t[e], m[e], p.rope, lane);
            if (WAY == kMoveOut) stage_row<VT, KT>(p.rows + ((size_t)(tok + e) * p.pool.n_kv_heads + h) * kRow, t[e], lane);
        }
        if (WAY == kMoveOut) continue;
        const int place = to & P1;
        uint8_t *tile = tile_of(p.pool, to >> p.pool.pshift, h, place >> 4, T::BYTES);
        if (still) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (e == 1 && !pair) break;
                store_k_paged<VT, KT>(t[e], (place & 15) + e, lane, tile);
                if (KT != KVQ_K_F16 && (lane & 7) == 0) *reinterpret_cast<uint16_t *>(tile + T::KS_OFF + scale_off((place & 15) + e, lane >> 3)) = t[e].ks;
            }
        } else if (pair) {
            store_pair_paged<VT, KT>(t[0], t[1], place & 15, lane, tile);
        } else {
            store_token_paged<VT, KT>(t[0], place & 15, lane, tile);
        }
    }
}

template <int VT, int KT, int PAIRS>
static cudaError_t move_t(const MoveParams &p, int blocks, cudaStream_t s, bool pdl)
{
    if (!p.rows) return launch_pdl(move_kernel<VT, KT, PAIRS, kMoveDirect>, p, blocks, kMoveWarps * 32, 0, s, pdl);
    const cudaError_t e = launch_pdl(move_kernel<VT, KT, PAIRS, kMoveOut>, p, blocks, kMoveWarps * 32, 0, s, pdl);
    return e != cudaSuccess ? e : launch_pdl(move_kernel<VT, KT, PAIRS, kMoveIn>, p, blocks, kMoveWarps * 32, 0, s, pdl);
}

cudaError_t launch_paged_move(const MoveParams &in, int v_type, int k_type, int n_sms, cudaStream_t s, bool pdl)
{
    MoveParams p = in;
    const long long want = (long long)p.pool.n_kv_heads * p.n_tokens / 2 / ((long long)n_sms * 48);
    p.heads = want < 1 ? 1 : want > p.pool.n_kv_heads ? p.pool.n_kv_heads : (int)want;
    p.chunks = (p.pool.n_kv_heads + p.heads - 1) / p.heads;
    const int blocks = (int)(((long long)p.n_tokens + kMoveWarps - 1) / kMoveWarps * p.chunks);
    const bool pairs = p.rope.pairs, f16 = k_type == KVQ_K_F16;
    if (v_type == KVQ_V_Q4_0) {
        if (f16) return pairs ? move_t<KVQ_V_Q4_0, KVQ_K_F16, 1>(p, blocks, s, pdl) : move_t<KVQ_V_Q4_0, KVQ_K_F16, 0>(p, blocks, s, pdl);
        return pairs ? move_t<KVQ_V_Q4_0, KVQ_K_I8, 1>(p, blocks, s, pdl) : move_t<KVQ_V_Q4_0, KVQ_K_I8, 0>(p, blocks, s, pdl);
    }
    if (f16) return pairs ? move_t<KVQ_V_Q8_0, KVQ_K_F16, 1>(p, blocks, s, pdl) : move_t<KVQ_V_Q8_0, KVQ_K_F16, 0>(p, blocks, s, pdl);
    return pairs ? move_t<KVQ_V_Q8_0, KVQ_K_I8, 1>(p, blocks, s, pdl) : move_t<KVQ_V_Q8_0, KVQ_K_I8, 0>(p, blocks, s, pdl);
}

}  // namespace kvq
