// kvq_held.cu -- what the paged cache holds: positions of a step's rows, tables
// forked, pages copied, tokens moved and their keys turned.
#include "kvq_quad.cuh"

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
// Copy: a warp takes up to 4 KB of one head of one page in one pool, whose tiles are
// one run of bytes; all of it is on its way before the first is written.
// ---------------------------------------------------------------------------
constexpr int kCopyWarps = 8;
constexpr int kCopyLoads = 8;                 // of 16 bytes a lane
constexpr int kCopyPiece = 32 * kCopyLoads;   // words of 16 bytes

__global__ void __launch_bounds__(kCopyWarps * 32) page_copy_kernel(const __grid_constant__ CopyParams p)
{
    pdl_wait();
    pdl_trigger();
    const unsigned pool = blockIdx.y, i = blockIdx.x / (unsigned)p.blocks, unit = (blockIdx.x - i * p.blocks) * kCopyWarps + (threadIdx.x >> 5);
    const int from = p.from[i], to = p.to[i], lane = threadIdx.x & 31;
    if (from < 0 || to < 0 || from >= p.n_pages || to >= p.n_pages || from == to) return;
    const unsigned heads = p.heads[pool], h = unit / (unsigned)p.pieces, piece = unit - h * p.pieces;
    if (h >= heads) return;
    int tiles = p.tiles;
    if (p.held) tiles = min(tiles, (int)(((long long)max(p.held[i], 0) + 15) >> 4));
    const int n = tiles * (p.tile_bytes[pool] / 16);
    const size_t run = (size_t)p.tiles * p.tile_bytes[pool];
    const uint4 *src = reinterpret_cast<const uint4 *>(p.data[pool] + ((size_t)from * heads + h) * run);
    uint4 *dst = reinterpret_cast<uint4 *>(p.data[pool] + ((size_t)to * heads + h) * run);
    const int at = (int)piece * kCopyPiece + lane;
    uint4 v[kCopyLoads];
#pragma unroll
    for (int k = 0; k < kCopyLoads; ++k)
        if (at + 32 * k < n) v[k] = __ldcs(src + at + 32 * k);
#pragma unroll
    for (int k = 0; k < kCopyLoads; ++k)
        if (at + 32 * k < n) __stcs(dst + at + 32 * k, v[k]);
}

cudaError_t launch_page_copy(const CopyParams &in, cudaStream_t s, bool pdl)
{
    CopyParams p = in;
    int words = 0;
    for (int i = 0; i < p.n_pools; ++i) words = p.tiles * (p.tile_bytes[i] / 16) > words ? p.tiles * (p.tile_bytes[i] / 16) : words;
    p.pieces = (words + kCopyPiece - 1) / kCopyPiece;
    p.blocks = (p.most_heads * p.pieces + kCopyWarps - 1) / kCopyWarps;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.n_copies * p.blocks, p.n_pools);
    cfg.blockDim = dim3(kCopyWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, page_copy_kernel, p);
}

// ---------------------------------------------------------------------------
// Move: a quad of lanes takes a token of a head (kvq_quad.cuh), a warp eight at a
// time: four pairs of tokens whose new slots are an even place and the next, which
// share words of V codes, or, where the list has no pairs, eight tokens.  A warp
// looks at eight tokens of the list and goes over some of the heads.
// ---------------------------------------------------------------------------
constexpr int kMoveWarps = 4;
constexpr int kMoveTokens = 8;   // of a warp

// Which half of the way: from slots to slots, from slots to the staged rows, from those to slots.
constexpr int kMoveDirect = 0, kMoveOut = 1, kMoveIn = 2;

struct alignas(16) MoveShared {   // (read in words of 16 bytes, warp after warp)
    float cosines[kMoveTokens][kAngleRow], sines[kMoveTokens][kAngleRow];   // of the quads' turns; of row 0 alone where they are the same
    uint8_t list[kMoveTokens];
};

// The lane's values of a held key in fp32, a block at a time as quad_floats has them.
template <int KT, int ROT>
__device__ __forceinline__ void key_floats(const uint32_t *w, float scale, float2 (&x)[4])
{
    if (KT == KVQ_K_F16) {
        quad_floats<ROT>(make_uint4(w[0], w[1], w[2], w[3]), x);
    } else {   // code + 128 under the exponent of 2^23
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(__byte_perm(w[k >> 2], 0x4b000000u, 0x7440 | (k & 3)));
        const float2 less = make_float2(-8388736.f, -8388736.f), s2 = make_float2(scale, scale);
        if (ROT == kRotPairs) {
            x[0] = make_float2(v[0], v[2]);
            x[1] = make_float2(v[4], v[6]);
            x[2] = make_float2(v[1], v[3]);
            x[3] = make_float2(v[5], v[7]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = make_float2(v[2 * k], v[2 * k + 1]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = mul2(add2(x[k], less), s2);
    }
}

// The quad's key turned; SOME: only where `turns`, the others' stay as they are.
// scratch: the quad's 128 floats in shared memory (part).
template <bool SOME, int VT, int KT, int ROT>
__device__ __forceinline__ void turn_key(QuadRow<VT, KT> &r, bool turns, const float *cosines, const float *sines, int c, int n_rot, float *scratch)
{
    constexpr int kWords = KT == KVQ_K_F16 ? 4 : 2;   // of a block
    const float2 s01 = half2_of(r.ks[0]), s23 = half2_of(r.ks[1]);
    const float scale[4] = {s01.x, s01.y, s23.x, s23.y};
    QuadF x;
#pragma unroll
    for (int b = 0; b < 4; ++b) key_floats<KT, ROT>(r.k + kWords * b, scale[b], x.b[b]);
    if (ROT == kRotPart) {   // neighbours to group pairs, and back
        __syncwarp();
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                *reinterpret_cast<float4 *>(scratch + 32 * b + 8 * c + 4 * k) = make_float4(x.b[b][2 * k].x, x.b[b][2 * k].y, x.b[b][2 * k + 1].x, x.b[b][2 * k + 1].y);
        __syncwarp();
        QuadF y;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const PartGroups g(c + 4 * b, n_rot);
            const float4 u = *reinterpret_cast<const float4 *>(scratch + g.a), v = *reinterpret_cast<const float4 *>(scratch + g.b);
            y.b[b][0] = make_float2(u.x, u.y);
            y.b[b][1] = make_float2(u.z, u.w);
            y.b[b][2] = make_float2(v.x, v.y);
            y.b[b][3] = make_float2(v.z, v.w);
        }
        quad_turn<ROT>(y, cosines, sines, c, n_rot);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const PartGroups g(c + 4 * b, n_rot);
            *reinterpret_cast<float4 *>(scratch + g.a) = make_float4(y.b[b][0].x, y.b[b][0].y, y.b[b][1].x, y.b[b][1].y);
            *reinterpret_cast<float4 *>(scratch + g.b) = make_float4(y.b[b][2].x, y.b[b][2].y, y.b[b][3].x, y.b[b][3].y);
        }
        __syncwarp();
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float4 u = *reinterpret_cast<const float4 *>(scratch + 32 * b + 8 * c + 4 * k);
                x.b[b][2 * k] = make_float2(u.x, u.y);
                x.b[b][2 * k + 1] = make_float2(u.z, u.w);
            }
    } else {
        quad_turn<ROT>(x, cosines, sines, c, n_rot);
    }
    Quad16 h;
#pragma unroll
    for (int b = 0; b < 4; ++b) h.b[b] = quad_halves<ROT>(x.b[b]);
    if (KT == KVQ_K_F16) {
        if (!SOME || turns)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                r.k[kWords * b] = h.b[b].x;
                r.k[kWords * b + 1] = h.b[b].y;
                r.k[kWords * b + kWords - 2] = h.b[b].z;
                r.k[kWords * b + kWords - 1] = h.b[b].w;
            }
        return;
    }
    const QuadCodes q = quad_quantize<false>(h);
#pragma unroll
    for (int b = 0; b < 4; ++b)
        if ((!SOME || turns) && (ROT == kRotHalf || 32 * b < n_rot)) {   // the block holds a value that rotates
            r.k[kWords * b] = q.w[2 * b];
            r.k[kWords * b + 1] = q.w[2 * b + 1];
            r.ks[b >> 1] = __byte_perm(r.ks[b >> 1], q.s[b >> 1], b & 1 ? 0x7610 : 0x3254);
        }
}

// A staged row: the lanes' parts one after another, then the scales.
template <int VT, int KT>
struct Staged {
    static constexpr int K = 4 * QuadRow<VT, KT>::KW, V = 4 * QuadRow<VT, KT>::VW;   // bytes of a lane
    static constexpr int BYTES = (4 * (K + V) + (KT == KVQ_K_F16 ? 8 : 16) + 15) / 16 * 16;
};
template <int N>
__device__ __forceinline__ void put_words(uint8_t *to, const uint32_t (&w)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<uint4 *>(to + 4 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
}
template <int N>
__device__ __forceinline__ void get_words(const uint8_t *from, uint32_t (&w)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(from + 4 * i);
        w[i] = v.x;
        w[i + 1] = v.y;
        w[i + 2] = v.z;
        w[i + 3] = v.w;
    }
}
template <int VT, int KT>
__device__ __forceinline__ void stage_put(uint8_t *row, const QuadRow<VT, KT> &r, int c)
{
    using S = Staged<VT, KT>;
    put_words(row + S::K * c, r.k);
    put_words(row + 4 * S::K + S::V * c, r.v);
    uint8_t *scales = row + 4 * (S::K + S::V);
    reinterpret_cast<uint16_t *>(scales)[c] = (uint16_t)r.vs;
    if (KT != KVQ_K_F16 && c == 0) *reinterpret_cast<uint2 *>(scales + 8) = make_uint2(r.ks[0], r.ks[1]);
}
template <int VT, int KT>
__device__ __forceinline__ void stage_get(const uint8_t *row, QuadRow<VT, KT> &r, int c)
{
    using S = Staged<VT, KT>;
    get_words(row + S::K * c, r.k);
    get_words(row + 4 * S::K + S::V * c, r.v);
    const uint8_t *scales = row + 4 * (S::K + S::V);
    r.vs = reinterpret_cast<const uint16_t *>(scales)[c];
    r.ks[0] = r.ks[1] = 0;
    if (KT != KVQ_K_F16) {
        const uint2 s = *reinterpret_cast<const uint2 *>(scales + 8);
        r.ks[0] = s.x;
        r.ks[1] = s.y;
    }
}

template <int VT, int KT, int ROT, int WAY>
__global__ void __launch_bounds__(kMoveWarps * 32, 7) move_kernel(const MoveParams p)
{
    constexpr int kTile = PageTile<VT, KT>::BYTES, kRow = Staged<VT, KT>::BYTES;
    __shared__ __align__(16) MoveShared shared[kMoveWarps];
    __shared__ __align__(16) float scratch[ROT == kRotPart ? kMoveWarps : 1][8][ROT == kRotPart ? kD + 4 : 1];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & 3, quad = lane >> 2;
    MoveShared &sh = shared[warp];
    const long long job = (long long)blockIdx.x * kMoveWarps + warp;
    const int window = (int)(job / p.chunks), share = (int)(job - (long long)window * p.chunks);
    const long long t0 = (long long)window * kMoveTokens;
    if (t0 >= p.n_tokens) return;
    // the list's tokens: the one before the window, its own, the one behind
    const long long at = t0 - 1 + lane;
    const bool there = lane < kMoveTokens + 2 && at >= 0 && at < p.n_tokens;
    const int from_all = there ? p.from[at] : -1, to_all = there ? p.to[at] : -1;
    const int turn_all = ROT != kRotNone && there ? p.turn[at] : 0;
    auto inside = [&](int slot) { return slot >= 0 && slot < p.pool.n_slots; };
    const SlotPairs q = slot_pairs(to_all, inside(from_all) && inside(to_all), kMoveTokens);
    if (q.leads == 0) return;
    slot_list(q, sh.list);
    const bool pairs = (q.pair & q.lead) != 0;
    const int per = pairs ? 4 : 8, e = pairs ? quad & 1 : 0, P1 = (1 << p.pool.pshift) - 1;
    const int h0 = share * p.heads, h1 = min(p.pool.n_kv_heads, h0 + p.heads);
    const size_t head_bytes = (size_t)kTile << (p.pool.pshift - 4);
    for (int g = 0; g < q.leads; g += per) {
        const int n = g + (pairs ? quad >> 1 : quad), lead = sh.list[min(n, q.leads - 1)];
        const bool pair = q.pair >> lead & 1, mine = n < q.leads && (e == 0 || pair);
        const int i = lead + (pair ? e : 0);
        const int from = __shfl_sync(0xffffffffu, from_all, i), to = __shfl_sync(0xffffffffu, to_all, i), turn = __shfl_sync(0xffffffffu, turn_all, i);
        const bool turns = mine && turn != 0;
        // a token that stays keeps its V, unless the other of its pair comes from elsewhere and they share words
        const bool stays = WAY == kMoveDirect && from == to, other_stays = __shfl_xor_sync(0xffffffffu, stays, 4);
        const bool still = stays && (!pair || other_stays);
        const bool values = __any_sync(0xffffffffu, mine && !still), any = ROT != kRotNone && __any_sync(0xffffffffu, turns);
        if (!values && !any) continue;   // nothing changes
        const int fu = from & 15, tu = to & 15;
        const uint8_t *src = tile_of(p.pool, from >> p.pool.pshift, h0, (from & P1) >> 4, kTile);
        uint8_t *dst = tile_of(p.pool, to >> p.pool.pshift, h0, (to & P1) >> 4, kTile);
        uint8_t *staged = WAY == kMoveDirect ? nullptr : p.rows + ((size_t)(t0 + i - 1) * p.pool.n_kv_heads + h0) * kRow;
        QuadRow<VT, KT> r;
#pragma unroll
        for (int k = 0; k < QuadRow<VT, KT>::KW; ++k) r.k[k] = 0;
#pragma unroll
        for (int k = 0; k < QuadRow<VT, KT>::VW; ++k) r.v[k] = 0;
        r.ks[0] = r.ks[1] = r.vs = 0;
        auto get = [&]() {
            if (!mine) return;
            if (WAY == kMoveIn) {
                stage_get<VT, KT>(staged, r, c);
            } else {
                quad_get_key<VT, KT>(r, src, fu, c);
                if (values) quad_get_value<VT, KT>(r, src, fu, c);
            }
        };
        get();   // the first head's row, on its way while the angles are worked out
        int row = 0;
        if (ROT != kRotNone && any) {   // angles of the quads' turns, one row for all where they are the same
            const int one = __shfl_sync(0xffffffffu, turn, __ffs(__ballot_sync(0xffffffffu, turns)) - 1);
            const bool same = __all_sync(0xffffffffu, !turns || turn == one);
            __syncwarp();   // the rows before may still be read
            for (int k = 0; k < (same ? 1 : kMoveTokens); ++k) {
                const int t = same ? one : __shfl_sync(0xffffffffu, turn, 4 * k);
                for (int j = lane; j < p.rope.n_rot / 2; j += 32) {
                    const float2 a = angle_of(p.rope.turns[j], t, 1.f);
                    sh.cosines[k][j] = a.x;
                    sh.sines[k][j] = a.y;
                }
            }
            __syncwarp();
            row = same ? 0 : quad;
        }
        const float *cosines = sh.cosines[row], *sines = sh.sines[row];
        float *const mem = scratch[ROT == kRotPart ? warp : 0][ROT == kRotPart ? quad : 0];
        if (WAY == kMoveDirect && !values) {   // keys turn where they lie: only those that do are written
            for (int h = h0;;) {
                turn_key<false, VT, KT, ROT>(r, true, cosines, sines, c, p.rope.n_rot, mem);
                if (turns) quad_put_key<VT, KT>(r, dst, tu, c);
                if (++h >= h1) break;
                src += head_bytes;
                dst += head_bytes;
                if (mine) quad_get_key<VT, KT>(r, src, fu, c);
            }
            continue;
        }
        for (int h = h0;;) {
            if (ROT != kRotNone && any) turn_key<true, VT, KT, ROT>(r, turns, cosines, sines, c, p.rope.n_rot, mem);
            if (WAY == kMoveOut) {
                if (mine) stage_put<VT, KT>(staged, r, c);
            } else {
                if (mine) quad_put_key<VT, KT>(r, dst, tu, c);
                quad_put_value<VT, KT>(r, dst, tu, c, pair, mine);
            }
            if (++h >= h1) break;
            src += head_bytes;
            dst += head_bytes;
            staged += kRow;
            get();
        }
    }
}

template <int VT, int KT, int ROT>
static cudaError_t move_t(const MoveParams &p, int blocks, cudaStream_t s, bool pdl)
{
    if (!p.rows) return launch_pdl(move_kernel<VT, KT, ROT, kMoveDirect>, p, blocks, kMoveWarps * 32, 0, s, pdl);
    const cudaError_t e = launch_pdl(move_kernel<VT, KT, ROT, kMoveOut>, p, blocks, kMoveWarps * 32, 0, s, pdl);
    return e != cudaSuccess ? e : launch_pdl(move_kernel<VT, KT, kRotNone, kMoveIn>, p, blocks, kMoveWarps * 32, 0, s, pdl);
}

template <int VT, int KT>
static cudaError_t move_rot(const MoveParams &p, int blocks, cudaStream_t s, bool pdl)
{
    if (!p.turn) return move_t<VT, KT, kRotNone>(p, blocks, s, pdl);
    if (p.rope.pairs) return move_t<VT, KT, kRotPairs>(p, blocks, s, pdl);
    return p.rope.n_rot == kD ? move_t<VT, KT, kRotHalf>(p, blocks, s, pdl) : move_t<VT, KT, kRotPart>(p, blocks, s, pdl);
}

int staged_row_bytes(int v_type, int k_type)
{
    if (v_type == KVQ_V_Q4_0) return k_type == KVQ_K_F16 ? Staged<KVQ_V_Q4_0, KVQ_K_F16>::BYTES : Staged<KVQ_V_Q4_0, KVQ_K_I8>::BYTES;
    return k_type == KVQ_K_F16 ? Staged<KVQ_V_Q8_0, KVQ_K_F16>::BYTES : Staged<KVQ_V_Q8_0, KVQ_K_I8>::BYTES;
}

cudaError_t launch_paged_move(const MoveParams &in, int v_type, int k_type, int n_sms, cudaStream_t s, bool pdl)
{
    MoveParams p = in;
    const long long windows = ((long long)p.n_tokens + kMoveTokens - 1) / kMoveTokens;
    const long long want = windows * p.pool.n_kv_heads / ((long long)n_sms * 24);
    p.heads = want < 1 ? 1 : want > p.pool.n_kv_heads ? p.pool.n_kv_heads : (int)want;
    p.chunks = (p.pool.n_kv_heads + p.heads - 1) / p.heads;
    const int blocks = (int)((windows * p.chunks + kMoveWarps - 1) / kMoveWarps);
    if (v_type == KVQ_V_Q4_0) return k_type == KVQ_K_F16 ? move_rot<KVQ_V_Q4_0, KVQ_K_F16>(p, blocks, s, pdl) : move_rot<KVQ_V_Q4_0, KVQ_K_I8>(p, blocks, s, pdl);
    return k_type == KVQ_K_F16 ? move_rot<KVQ_V_Q8_0, KVQ_K_F16>(p, blocks, s, pdl) : move_rot<KVQ_V_Q8_0, KVQ_K_I8>(p, blocks, s, pdl);
}

}  // namespace kvq
