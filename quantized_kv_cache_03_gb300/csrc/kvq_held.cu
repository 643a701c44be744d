// kvq_held.cu -- what the paged cache holds: positions of a step's rows, tables
// forked, pages copied, tokens moved and their keys turned.
#include "kvq_quad.cuh"

namespace kvq {

// ---------------------------------------------------------------------------
// Positions: a row's sequence by a search over q_start in shared memory; it stands
// at the sequence's length less the rows from it to the sequence's end.  Latency
// alone: one round of loads and a search, a row to each thread: 64 rows of 64
// sequences 1.0 us, 8192 of 20 1.4 us, 40000 of 1024 1.8 us (four rows to a thread,
// which share a search where they can: 2.4, 1.7, 3.2; lengths from global memory after
// it 0.1 us more).
// ---------------------------------------------------------------------------
constexpr int kPosThreads = 256;

__global__ void __launch_bounds__(kPosThreads) positions_kernel(const PositionsParams p)
{
    extern __shared__ int qs[];
    const int n = p.n_seqs;
    int *const lens = qs + n + 1;
    pdl_wait();
#pragma unroll 4
    for (int i = threadIdx.x; i <= n; i += kPosThreads) {
        const int q = p.q_start[i];
        if (i < n) lens[i] = p.lens[i];
        qs[i] = min(max(q, 0), p.n_tokens);
    }
    __syncthreads();
    const long long t = (long long)blockIdx.x * kPosThreads + threadIdx.x;
    if (t >= p.n_tokens) return;
    int pos = -1;
    if (t >= qs[0] && t < qs[n]) {
        int a = 0, b = n;   // last sequence that begins at t or before
        while (b - a > 1) {
            const int mid = (a + b) >> 1;
            if (qs[mid] <= t) a = mid;
            else b = mid;
        }
        pos = (int)((unsigned)lens[a] - (unsigned)qs[a + 1] + (unsigned)t);
    }
    p.positions[t] = pos;
}

cudaError_t launch_positions(const PositionsParams &p, cudaStream_t s, bool pdl)
{
    return launch_pdl(positions_kernel, p, (int)(((long long)p.n_tokens + kPosThreads - 1) / kPosThreads), kPosThreads, (2 * p.n_seqs + 1) * (int)sizeof(int), s, pdl);
}

// ---------------------------------------------------------------------------
// Fork.  Whether a page is given back, and whether a row may go on writing into
// its last page, depends on every row's list.  Pages are marked in bytes, stored
// without reading: those that a new row lists whole (an old row's entries up to the
// longest that a place keeps of it: once, however many keep them), those that one
// ends in, and those past all that is kept of an old row, which are given back
// unless they are also one of the others.  The first place that ends in a page is
// a minimum.  Nothing depends on an order.
//
// In phases: lengths, and marks cleared; rows marked and copied; pages to give back
// counted and last pages that are shared listed; pages pushed, in order of
// their numbers, and dealt out.  Small batches go through them in one cluster, with
// marks as bits in shared memory, each CTA's own until they are joined: a scattered
// store to global memory costs an SM a cycle a byte (256 places of 129 entries: 13 us
// so, 7.1 with the bits).  What is left is latency: the lengths, the rows and the
// cluster's two barriers each wait for memory once.  Large batches take a launch for
// each phase over the whole GPU, with bytes in global memory.
// ---------------------------------------------------------------------------
constexpr int kForkCtas = 8, kForkThreads = 1024;   // of the one cluster
constexpr int kForkWide = 1024, kForkMark = 256;    // threads of a block otherwise

// What the phases know about each place, in shared memory (one cluster) or in the workspace.
struct ForkSeqs {
    int *from, *kept;     // old row (-1: none), positions kept
    int *tail;            // the entry of the page the place ends inside; -1: it ends with a page
    int *olds;            // pages of the old row of that number,
    int *whole, *used;    // and most that a place keeps of it, whole ones and all
    int *rank;            // among the places that need a copy, in order; -1: it needs none
    int *list;            // those places
    static constexpr int kArrays = 8;
    __device__ __forceinline__ ForkSeqs(int *at, int n)
        : from(at), kept(at + n), tail(at + 2 * n), olds(at + 3 * n), whole(at + 4 * n), used(at + 5 * n), rank(at + 6 * n), list(at + 7 * n) {}
};
__device__ __forceinline__ bool is_page(const ForkParams &p, int page) { return page >= 0 && page < p.n_pages; }

// Lengths, by one block (in a cluster by every one).
template <int THREADS>
__device__ __forceinline__ void fork_lengths(const ForkParams &p, const ForkSeqs &q)
{
    const int P = 1 << p.pshift;
    for (int b = threadIdx.x; b < p.n_seqs; b += THREADS) {
        const int len = (int)min(max((long long)p.lens[b], 0ll), (long long)p.max_blocks << p.pshift);
        int from = p.parent ? p.parent[b] : b;
        if (from < 0 || from >= p.n_seqs) from = -1;
        q.from[b] = from;
        q.kept[b] = p.keep ? p.keep[b] : len;
        q.olds[b] = (len + P - 1) >> p.pshift;
        q.whole[b] = q.used[b] = 0;
        q.rank[b] = len;   // (for the moment)
    }
    __syncthreads();
    for (int b = threadIdx.x; b < p.n_seqs; b += THREADS) {
        const int from = q.from[b], len = from < 0 ? 0 : q.rank[from], keep = p.keep ? max(0, min(len, q.kept[b])) : len;
        if (keep > 0) {
            atomicMax(q.whole + from, keep >> p.pshift);
            atomicMax(q.used + from, (keep + P - 1) >> p.pshift);
        }
        q.kept[b] = keep;
    }
    __syncthreads();
}
// The entry of the page that place b ends inside, -1 if it ends with one.
__device__ __forceinline__ int fork_tail(const ForkParams &p, const ForkSeqs &q, int b)
{
    const int kept = q.kept[b];
    return kept & ((1 << p.pshift) - 1) ? p.table[(size_t)q.from[b] * p.stride + (kept >> p.pshift)] : -1;
}

// 128 entries of a row, marked and copied by a warp: read, then written.
struct ForkRun {
    int b, e0, whole, mine;
    bool copies;
    int old_page[4], page[4];

    __device__ __forceinline__ ForkRun(const ForkParams &p, const ForkSeqs &q, int row_of, int run) : b(row_of), e0(run * 128 + (int)(threadIdx.x & 31))
    {
        const int used = q.used[b], olds = q.olds[b], from = q.from[b];
        whole = q.whole[b];
        mine = q.kept[b] >> p.pshift;
        const int *old_row = p.table + (size_t)b * p.stride, *row = p.table + (size_t)max(from, 0) * p.stride;
        copies = p.table_out + (size_t)b * p.out_stride != row;   // (in place the entries are there)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int e = e0 + 32 * k;
            old_page[k] = e < olds && (e < whole || e >= used) ? old_row[e] : -1;
            page[k] = copies && e < mine ? row[e] : -1;
        }
    }
    // mark(page, whole): it is one that a new row lists whole, or one that no place keeps of this row
    template <typename F>
    __device__ __forceinline__ void write(const ForkParams &p, F mark) const
    {
        int *out = p.table_out + (size_t)b * p.out_stride;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int e = e0 + 32 * k;
            if (is_page(p, old_page[k])) mark(old_page[k], e < whole);
            if (copies && e < mine) out[e] = page[k];
        }
    }
};
__device__ __forceinline__ int fork_runs(const ForkParams &p) { return (p.max_blocks + 127) / 128; }

// Exclusive sums of two values over the block's threads, and the totals.
template <int THREADS>
__device__ __forceinline__ int2 fork_scan(int2 x, int2 &total, int2 *tmp)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int2 y = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, y.x, d), v = __shfl_up_sync(0xffffffffu, y.y, d);
        if (lane >= d) y.x += u, y.y += v;
    }
    __syncthreads();   // tmp may still be read by the scan before
    if (lane == 31) tmp[warp] = y;
    __syncthreads();
    int2 z = lane < THREADS / 32 ? tmp[lane] : make_int2(0, 0), sum = z;   // every warp adds the warps up
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, sum.x, d), v = __shfl_up_sync(0xffffffffu, sum.y, d);
        if (lane >= d) sum.x += u, sum.y += v;
    }
    total = make_int2(__shfl_sync(0xffffffffu, sum.x, 31), __shfl_sync(0xffffffffu, sum.y, 31));
    return make_int2(__shfl_sync(0xffffffffu, sum.x - z.x, warp) + y.x - x.x, __shfl_sync(0xffffffffu, sum.y - z.y, warp) + y.y - x.y);
}

// The stack between the pushes and the pops: entries below n_free are the old
// ones, `back` new ones follow; `needs` are taken off its top, the first place's first.
struct ForkStack {
    int n_free, avail, needs;
    __device__ __forceinline__ ForkStack(const ForkParams &p, int n, int back, int want) : n_free(n), needs(want)
    {
        avail = (int)min((long long)n + back, (long long)p.n_pages);
    }
};
__device__ __forceinline__ void fork_give(const ForkParams &p, const ForkSeqs &q, int b, int page)
{
    p.copy_to[b] = page;
    p.table_out[(size_t)b * p.out_stride + (q.kept[b] >> p.pshift)] = page;
}
// A page that is given back, entry `at` of the stack.
__device__ __forceinline__ void fork_push(const ForkParams &p, const ForkSeqs &q, const ForkStack &st, long long at, int page)
{
    if (at >= p.n_pages) return;
    p.free_pages[at] = page;
    const int r = st.avail - 1 - (int)at;
    if (r < st.needs) fork_give(p, q, q.list[r], page);
}
// Every place's results but a copy's page where it was pushed just now.
__device__ __forceinline__ void fork_results(const ForkParams &p, const ForkSeqs &q, const ForkStack &st, int at, int all)
{
    const int P = 1 << p.pshift;
    for (int b = at; b < p.n_seqs; b += all) {
        int kept = q.kept[b], from = -1, held = 0, status = 0;
        const int rank = q.rank[b], entry = st.avail - 1 - rank;
        const bool in_part = (kept & (P - 1)) != 0;
        if (rank >= 0 && entry >= 0) {
            from = q.tail[b];
            held = kept & (P - 1);
            if (entry < st.n_free) fork_give(p, q, b, p.free_pages[entry]);
        } else {
            p.copy_to[b] = -1;
            if (rank >= 0) {
                kept &= ~(P - 1);
                status = 1;
            } else if (in_part) {
                p.table_out[(size_t)b * p.out_stride + (kept >> p.pshift)] = q.tail[b];
            }
        }
        p.copy_from[b] = from;
        p.copy_held[b] = held;
        p.status[b] = status;
        p.lens_out[b] = kept;
    }
    if (at == 0) *p.n_free_out = st.avail - min(st.needs, st.avail);
}

__device__ __forceinline__ void cluster_sync() { asm volatile("barrier.cluster.arrive;\n barrier.cluster.wait;" ::: "memory"); }
// A word of another CTA's shared memory.
__device__ __forceinline__ uint32_t of_cta(const uint32_t *mine, int rank)
{
    uint32_t at, v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(mine)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ void to_cta(uint32_t *mine, int rank, uint32_t v)
{
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(mine)), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// The least place that ends in a page, by page: a table in shared memory, probed
// in a row, at most half full.
struct PageTable {
    static constexpr int kSlots = 2048;
    int *page, *place;
    __device__ __forceinline__ explicit PageTable(int *at) : page(at), place(at + kSlots) {}
    __device__ __forceinline__ void clear() const
    {
        for (int i = threadIdx.x; i < kSlots; i += kForkThreads) {
            page[i] = -1;
            place[i] = 0x7fffffff;
        }
    }
    static __device__ __forceinline__ unsigned slot(int p) { return (unsigned)p * 2654435769u >> 21; }
    __device__ __forceinline__ void least(int p, int b) const
    {
        unsigned h = slot(p);
        for (int k = 0; k < kSlots; ++k, h = (h + 1) % kSlots) {
            const int had = atomicCAS(page + h, -1, p);
            if (had == -1 || had == p) {
                atomicMin(place + h, b);
                return;
            }
        }
    }
    __device__ __forceinline__ int of(int p) const   // p is in it
    {
        unsigned h = slot(p);
        for (int k = 0; k < kSlots && page[h] != p; ++k) h = (h + 1) % kSlots;
        return place[h];
    }
};

constexpr int kForkMaxSeqs = 1024, kForkMaxPages = 64 * 1024;   // of the cluster
static_assert(2 * kForkMaxSeqs <= PageTable::kSlots && kForkMaxSeqs <= kForkThreads && kForkMaxPages / 32 / kForkCtas <= kForkThreads, "a place and a word of marks to a thread");

__global__ void __cluster_dims__(kForkCtas, 1, 1) __launch_bounds__(kForkThreads) fork_cluster_kernel(const ForkParams p)
{
    extern __shared__ int seqs[];
    __shared__ int2 tmp[kForkThreads / 32];
    __shared__ uint32_t counts[kForkCtas], needs[kForkMaxSeqs / 32];
    const int tid = threadIdx.x, rank = blockIdx.x, at = rank * kForkThreads + tid, all = kForkCtas * kForkThreads, n = p.n_seqs, words = (p.n_pages + 31) / 32;
    const ForkSeqs q(seqs, n);
    uint32_t *const old = reinterpret_cast<uint32_t *>(seqs) + ForkSeqs::kArrays * n, *const full = old + words, *const tails = full + words;
    for (int i = tid; i < 3 * words; i += kForkThreads) old[i] = 0;
    const PageTable ends(reinterpret_cast<int *>(tails + words));
    ends.clear();
    pdl_wait();
    pdl_trigger();
    const int n_free = min(max(*p.n_free, 0), p.n_pages);
    fork_lengths<kForkThreads>(p, q);   // (its barriers also order the marks' clearing)
    // rows marked and copied, the first two of a warp read before the ends of the places are
    auto mark = [&](int page, bool whole) { atomicOr((whole ? full : old) + (page >> 5), 1u << (page & 31)); };
    const int runs = fork_runs(p), warps = all >> 5, items = n * runs;   // (few: the launch sees to it)
    auto run = [&](int item) { return ForkRun(p, q, item / runs, item % runs); };
    if (items > 0) {
        const ForkRun one = run(min(at >> 5, items - 1)), two = run(min((at >> 5) + warps, items - 1));   // (the last one again does no harm)
        if (tid < n) {
            const int tail = fork_tail(p, q, tid);
            q.tail[tid] = tail;
            if (is_page(p, tail)) {
                atomicOr(tails + (tail >> 5), 1u << (tail & 31));
                ends.least(tail, tid);
            }
        }
        one.write(p, mark);
        two.write(p, mark);
        for (int item = (at >> 5) + 2 * warps; item < items; item += warps) run(item).write(p, mark);
    } else if (tid < n) {   // rows without entries
        q.tail[tid] = -1;
    }
    cluster_sync();   // marks are set; and every CTA has read lens and n_free, which results may replace
    // the CTA's share of the pool, a word of 32 pages a thread
    const int share = (words + kForkCtas - 1) / kForkCtas, w = rank * share + tid;
    uint32_t gone = 0;
    if (tid < share && w < words) {
        uint32_t o = 0, f = tails[w];
#pragma unroll
        for (int k = 0; k < kForkCtas; ++k) {
            o |= of_cta(old + w, k);
            f |= of_cta(full + w, k);
        }
        gone = o & ~f;
    }
    // the CTA's places that end inside a page they may not write to: one that a row lists whole, or that an earlier
    // place ends in too; a bit each, to every CTA
    const int places = (n + 32 * kForkCtas - 1) / (32 * kForkCtas) * 32, b = rank * places + tid;
    if (tid < places) {
        bool need = false;
        const int tail = b < n ? q.tail[b] : -1;
        if (is_page(p, tail)) {
            uint32_t f = 0;
#pragma unroll
            for (int k = 0; k < kForkCtas; ++k) f |= of_cta(full + (tail >> 5), k);
            need = (f >> (tail & 31) & 1) || ends.of(tail) != b;
        }
        const unsigned bits = __ballot_sync(0xffffffffu, need);
        if ((tid & 31) < kForkCtas && b - (tid & 31) < kForkMaxSeqs) to_cta(needs + (b >> 5), tid & 31, bits);
    }
    int2 total;
    const int first = fork_scan<kForkThreads>(make_int2(__popc(gone), 0), total, tmp).x;
    if (tid < kForkCtas) to_cta(counts + rank, tid, (uint32_t)total.x);   // this CTA's count, to every other
    cluster_sync();
    int before = 0, back = 0;
#pragma unroll
    for (int k = 0; k < kForkCtas; ++k) {
        before += k < rank ? (int)counts[k] : 0;
        back += (int)counts[k];
    }
    const bool need = tid < n && (needs[tid >> 5] >> (tid & 31) & 1);
    const int mine = fork_scan<kForkThreads>(make_int2(need, 0), total, tmp).x;
    if (tid < n) q.rank[tid] = need ? mine : -1;
    if (need) q.list[mine] = tid;
    __syncthreads();
    const ForkStack st(p, n_free, back, total.x);
    long long to = (long long)n_free + before + first;
    for (; gone; gone &= gone - 1) fork_push(p, q, st, to++, 32 * w + __ffs(gone) - 1);
    fork_results(p, q, st, at, all);
}

__global__ void __launch_bounds__(kForkWide) fork_clear_kernel(const ForkParams p)
{
    pdl_wait();
    if (blockIdx.x == 0) {   // lengths in shared memory, where their maxima cost no trips, then to the workspace
        extern __shared__ int seqs[];
        const ForkSeqs q(seqs, p.n_seqs), out(p.seqs, p.n_seqs);
        fork_lengths<kForkWide>(p, q);
        for (int b = threadIdx.x; b < p.n_seqs; b += kForkWide) {
            const int tail = fork_tail(p, q, b);
            out.from[b] = q.from[b];
            out.kept[b] = q.kept[b];
            out.olds[b] = q.olds[b];
            out.whole[b] = q.whole[b];
            out.used[b] = q.used[b];
            out.tail[b] = tail;
            if (is_page(p, tail)) p.owner[tail] = p.n_seqs;
        }
        if (threadIdx.x == 0) p.totals[0] = min(max(*p.n_free, 0), p.n_pages);
    } else {   // the marks, three kinds side by side
        const long long words = (long long)(p.full_mark - p.old_mark) * 3 / 16, at = (long long)(blockIdx.x - 1) * kForkWide + threadIdx.x;
        for (long long i = at; i < words; i += (long long)(gridDim.x - 1) * kForkWide) reinterpret_cast<uint4 *>(p.old_mark)[i] = make_uint4(0, 0, 0, 0);
    }
}
__global__ void __launch_bounds__(kForkMark) fork_mark_kernel(const ForkParams p)
{
    pdl_wait();
    const int at = blockIdx.x * kForkMark + threadIdx.x, all = gridDim.x * kForkMark, runs = fork_runs(p);
    const ForkSeqs q(p.seqs, p.n_seqs);
    for (long long item = at >> 5; item < (long long)p.n_seqs * runs; item += all >> 5) {
        const int b = (int)(item / runs);
        ForkRun(p, q, b, (int)(item - (long long)b * runs)).write(p, [&](int page, bool whole) { (whole ? p.full_mark : p.old_mark)[page] = 1; });
    }
    for (int b = at; b < p.n_seqs; b += all) {
        const int tail = q.tail[b];
        if (is_page(p, tail)) {
            p.tail_mark[tail] = 1;
            atomicMin(p.owner + tail, b);
        }
    }
}
// Four pages' marks: a bit per byte, listed before and not now (marks past the last page are clear).
__device__ __forceinline__ uint32_t fork_gone(const ForkParams &p, long long w)
{
    auto of = [&](const uint8_t *marks) { return reinterpret_cast<const uint32_t *>(marks)[w]; };
    return of(p.old_mark) & ~(of(p.full_mark) | of(p.tail_mark));
}
// A thread's share of the pool: words w0 .. w1 - 1 of a block's, the first of them kept in hand.
struct ForkShare {
    long long w0, w1;
    uint32_t g;
    int n;
    __device__ __forceinline__ ForkShare(const ForkParams &p) : g(0)
    {
        const long long words = ((long long)p.n_pages + 3) / 4, of_block = (words + p.blocks - 1) / p.blocks, per = (of_block + kForkWide - 1) / kForkWide;
        const long long b0 = min(words, blockIdx.x * of_block), b1 = min(words, b0 + of_block);
        w0 = min(b1, b0 + threadIdx.x * per);
        w1 = min(b1, w0 + per);
        if (w0 < w1) g = fork_gone(p, w0);
        n = __popc(g);
        for (long long w = w0 + 1; w < w1; ++w) n += __popc(fork_gone(p, w));
    }
};
__global__ void __launch_bounds__(kForkWide) fork_count_kernel(const ForkParams p)
{
    __shared__ int2 tmp[kForkWide / 32];
    pdl_wait();
    int2 total;
    if ((int)blockIdx.x < p.blocks) {
        fork_scan<kForkWide>(make_int2(ForkShare(p).n, 0), total, tmp);
        if (threadIdx.x == 0) p.counts[blockIdx.x] = total.x;
        return;
    }
    // one block more: places that end inside a page they may not write to
    const ForkSeqs q(p.seqs, p.n_seqs);
    const int each = (p.n_seqs + kForkWide - 1) / kForkWide, b0 = min(p.n_seqs, (int)threadIdx.x * each), b1 = min(p.n_seqs, b0 + each);
    int n = 0;
    for (int b = b0; b < b1; ++b) {
        const int tail = q.tail[b];
        int needs = 0;
        if (is_page(p, tail)) {
            const int full = p.full_mark[tail], owner = p.owner[tail];
            needs = full != 0 || owner != b;
        }
        q.rank[b] = needs - 1;   // -1 or 0
        n += needs;
    }
    int at = fork_scan<kForkWide>(make_int2(0, n), total, tmp).y;
    for (int b = b0; b < b1; ++b)
        if (q.rank[b] >= 0) {
            q.list[at] = b;
            q.rank[b] = at++;
        }
    if (threadIdx.x == 0) p.totals[1] = total.y;
}
__global__ void __launch_bounds__(kForkWide) fork_deal_kernel(const ForkParams p)
{
    __shared__ int2 tmp[kForkWide / 32];
    pdl_wait();
    const ForkSeqs q(p.seqs, p.n_seqs);
    const ForkShare share(p);
    int2 blocks = make_int2(0, 0), total;   // pages of the blocks before this one, of all
    for (int k = threadIdx.x; k < p.blocks; k += kForkWide) {
        const int c = p.counts[k];
        blocks.x += k < (int)blockIdx.x ? c : 0;
        blocks.y += c;
    }
    fork_scan<kForkWide>(blocks, total, tmp);
    const ForkStack st(p, p.totals[0], total.y, p.totals[1]);
    int2 mine;
    long long at = (long long)st.n_free + total.x + fork_scan<kForkWide>(make_int2(share.n, 0), mine, tmp).x;
    if (share.n > 0)
        for (long long w = share.w0; w < share.w1; ++w) {
            for (uint32_t bits = w == share.w0 ? share.g : fork_gone(p, w); bits; bits &= bits - 1) fork_push(p, q, st, at++, (int)(4 * w) + (__ffs(bits) >> 3));
        }
    fork_results(p, q, st, blockIdx.x * kForkWide + threadIdx.x, p.blocks * kForkWide);
}

constexpr int fork_cluster_smem(int n_seqs, int n_pages) { return (ForkSeqs::kArrays * n_seqs + 3 * ((n_pages + 31) / 32) + 2 * PageTable::kSlots) * (int)sizeof(int); }
constexpr int fork_clear_smem(int n_seqs) { return ForkSeqs::kArrays * n_seqs * (int)sizeof(int); }
cudaError_t prepare_page_fork()
{
    const cudaError_t e = cudaFuncSetAttribute(fork_clear_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, fork_clear_smem(KVQ_MAX_PAGED_SEQS));
    return e != cudaSuccess ? e : cudaFuncSetAttribute(fork_cluster_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, fork_cluster_smem(kForkMaxSeqs, kForkMaxPages));
}

cudaError_t launch_page_fork(const ForkParams &in, int n_sms, cudaStream_t s, bool pdl)
{
    ForkParams p = in;
    const long long entries = (long long)p.n_seqs * p.max_blocks;
    // Eight SMs against all of them and four launches: 256 places of 129 entries 7.1 us against 9.8, 1024 of 126 10.8
    // against 12.7, 256 of 501 9.4 against 10.7; beyond, 256 of 1001 (75000 pages) 12.5 against 11.9, 512 of 501 (77000)
    // 13.2 against 12.3, 1024 of 501 21.6 against 15.7.
    if (p.n_seqs <= kForkMaxSeqs && p.n_pages <= kForkMaxPages && entries <= 128 * 1024)
        return launch_pdl(fork_cluster_kernel, p, kForkCtas, kForkThreads, fork_cluster_smem(p.n_seqs, p.n_pages), s, pdl);
    auto grid = [&](long long items, int most) { return (int)(items < 1 ? 1 : items > most ? most : items); };
    cudaError_t e = launch_pdl(fork_clear_kernel, p, 1 + grid(((long long)p.n_pages * 3 / 16 + kForkWide - 1) / kForkWide, 2 * n_sms), kForkWide, fork_clear_smem(p.n_seqs), s, pdl);
    if (e == cudaSuccess) e = launch_pdl(fork_mark_kernel, p, grid((long long)p.n_seqs * ((p.max_blocks + 127) / 128) / (kForkMark / 32) + 1, 8 * n_sms), kForkMark, 0, s, pdl);
    if (e == cudaSuccess) e = launch_pdl(fork_count_kernel, p, p.blocks + 1, kForkWide, 0, s, pdl);
    if (e == cudaSuccess) e = launch_pdl(fork_deal_kernel, p, p.blocks, kForkWide, 0, s, pdl);
    return e;
}

// ---------------------------------------------------------------------------
// Copy: a warp takes up to 4 KB of one head of one page in one pool, whose tiles are
// one run of bytes; all of it is on its way before the first is written.  Bound by
// memory: 2048 pages of 64 tokens, 8 heads, 570 MB both ways in 84.2 us, a plain
// copy's rate (1.00); 256 pages of 16 tokens, two in five of them copied, in each
// of 32 pools 182 MB in 29.4 us (0.91: a short launch's ramps; blocks with nothing to do
// cost nothing: two pools to a block 29.8, four 30.3).
// Streaming loads and stores, since neither side is read again soon.  A page of one
// head 1.6 us.
// ---------------------------------------------------------------------------
constexpr int kCopyWarps = 8;
constexpr int kCopyLoads = 8;                 // of 16 bytes a lane
constexpr int kCopyPiece = 32 * kCopyLoads;   // words of 16 bytes

template <int POOLS>
__global__ void __launch_bounds__(kCopyWarps * 32) page_copy_kernel(const __grid_constant__ CopyParams<POOLS> p)
{
    pdl_wait();
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

template <int POOLS>
cudaError_t launch_page_copy(const CopyParams<POOLS> &in, cudaStream_t s, bool pdl)
{
    CopyParams<POOLS> p = in;
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
    return cudaLaunchKernelEx(&cfg, page_copy_kernel<POOLS>, p);
}
template cudaError_t launch_page_copy(const CopyParams<kFewPools> &, cudaStream_t, bool);
template cudaError_t launch_page_copy(const CopyParams<KVQ_MAX_COPY_POOLS> &, cudaStream_t, bool);

// ---------------------------------------------------------------------------
// Gather, many rows: a quad of lanes takes a token of a head (kvq_quad.cuh), a warp
// eight tokens.  Bound by memory: 131072 tokens, 8 heads, q8_0 V: 218 us in fp32, 0.92
// of a copy's rate (a lane's 32 bytes stored as they lie, half a sector at a time:
// 351), 131 us in fp16, 0.92 (a warp to a pair of rows: 179); q4_0 V in fp16 121 us,
// 0.92.
// ---------------------------------------------------------------------------
constexpr int kGatherWarps = 4;

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

// A block's words of a quad, w[0] and w[1] (N of them each) of lane c being dims 8 c and on and 8 c + 4 and on, dealt out
// so that those of its four lanes are neighbours: dims 4 c and on, and 16 + 4 c and on.  Stores of 16 bytes a lane then
// fill whole sectors.
template <int N>
__device__ __forceinline__ void spread(const uint32_t *w, int c, uint32_t (&x)[2][N])
{
    const int lane = (threadIdx.x & 28) + (c >> 1);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t a = __shfl_sync(0xffffffffu, w[i], lane + 2 * j), b = __shfl_sync(0xffffffffu, w[N + i], lane + 2 * j);
            x[j][i] = c & 1 ? b : a;
        }
}
// Four values, as fp16 or fp32.
template <bool O16>
__device__ __forceinline__ void put4(void *base, size_t elem, float2 x, float2 y)
{
    if (O16) *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(base) + elem) = make_uint2(pack_half2(x.x, x.y), pack_half2(y.x, y.y));
    else *reinterpret_cast<float4 *>(static_cast<float *>(base) + elem) = make_float4(x.x, x.y, y.x, y.y);
}
// The four values of code bytes w (code + bias) times s.
template <int BIAS>
__device__ __forceinline__ void scaled4(uint32_t w, float s, float2 &x, float2 &y)
{
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 | k));
    const float2 less = make_float2(-8388608.f - BIAS, -8388608.f - BIAS), s2 = make_float2(s, s);
    x = mul2(add2(make_float2(v[0], v[1]), less), s2);
    y = mul2(add2(make_float2(v[2], v[3]), less), s2);
}

template <int VT, int KT, bool O16>
__global__ void __launch_bounds__(kGatherWarps * 32) gather_kernel(const GatherParams p)
{
    using T = PageTile<VT, KT>;
    pdl_wait();
    const int lane = threadIdx.x & 31, c = lane & 3, quad = lane >> 2;
    const long long job = (long long)blockIdx.x * kGatherWarps + (threadIdx.x >> 5);
    const int window = (int)(job / p.chunks), h0 = (int)(job - (long long)window * p.chunks) * p.heads, h1 = min(p.pool.n_kv_heads, h0 + p.heads);
    const long long tok = (long long)window * 8 + quad;
    const int slot = tok < p.n_tokens ? p.slots[tok] : -1;
    const bool mine = slot >= 0 && slot < p.pool.n_slots;
    if (!__any_sync(0xffffffffu, mine)) return;
    const int place = slot & ((1 << p.pool.pshift) - 1), u = place & 15;
    const uint8_t *tile = tile_of(p.pool, mine ? slot >> p.pool.pshift : 0, h0, place >> 4, T::BYTES);
    size_t at = ((size_t)tok * p.pool.n_kv_heads + h0) * kD;
    QuadRow<VT, KT> r;
#pragma unroll
    for (int k = 0; k < QuadRow<VT, KT>::KW; ++k) r.k[k] = 0;
#pragma unroll
    for (int k = 0; k < QuadRow<VT, KT>::VW; ++k) r.v[k] = 0;
    r.ks[0] = r.ks[1] = 0;
    uint4 vs = make_uint4(0, 0, 0, 0);
    for (int h = h0; h < h1; ++h, tile += (size_t)T::BYTES << (p.pool.pshift - 4), at += kD) {
        if (mine) {
            quad_get_key<VT, KT>(r, tile, u, c);
            quad_get_value<VT, KT>(r, tile, u, c);
            vs = *reinterpret_cast<const uint4 *>(tile + T::VS_OFF + 16 * (u / 2));
        }
        const uint32_t sel = u & 1 ? 0x7632 : 0x5410;
        const float2 k01 = half2_of(r.ks[0]), k23 = half2_of(r.ks[1]), v01 = half2_of(__byte_perm(vs.x, vs.y, sel)), v23 = half2_of(__byte_perm(vs.z, vs.w, sel));
        const float ks[4] = {k01.x, k01.y, k23.x, k23.y}, ds[4] = {v01.x, v01.y, v23.x, v23.y};
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            float2 x[4];
            constexpr int N = KT == KVQ_K_F16 ? 2 : 1;
            if (O16) {
                key_floats<KT, kRotNone>(r.k + 2 * N * b, ks[b], x);
                if (mine) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.k_out) + at + 32 * b + 8 * c) = quad_halves<kRotNone>(x);
            } else {
                uint32_t w[2][N];
                spread<N>(r.k + 2 * N * b, c, w);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (KT == KVQ_K_F16) x[0] = half2_of(w[j][0]), x[1] = half2_of(w[j][N - 1]);
                    else scaled4<128>(w[j][0], ks[b], x[0], x[1]);
                    if (mine) put4<O16>(p.k_out, at + 32 * b + 16 * j + 4 * c, x[0], x[1]);
                }
            }
            if (VT == KVQ_V_Q8_0 && O16) {
                scaled4<128>(r.v[2 * b], ds[b], x[0], x[1]);
                scaled4<128>(r.v[2 * b + 1], ds[b], x[2], x[3]);
                if (mine) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.v_out) + at + 32 * b + 8 * c) = quad_halves<kRotNone>(x);
            } else if (VT == KVQ_V_Q8_0) {
                uint32_t w[2][1];
                spread<1>(r.v + 2 * b, c, w);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    scaled4<128>(w[j][0], ds[b], x[0], x[1]);
                    if (mine) put4<O16>(p.v_out, at + 32 * b + 16 * j + 4 * c, x[0], x[1]);
                }
            } else {   // code bytes 4 quart .. + 3: their low nibbles, their high ones 16 values on
                scaled4<8>(r.v[b] & 0x0f0f0f0fu, ds[b], x[0], x[1]);
                scaled4<8>(r.v[b] >> 4 & 0x0f0f0f0fu, ds[b], x[2], x[3]);
                if (mine) {
                    put4<O16>(p.v_out, at + 32 * b + 4 * quart_of(c), x[0], x[1]);
                    put4<O16>(p.v_out, at + 32 * b + 16 + 4 * quart_of(c), x[2], x[3]);
                }
            }
        }
    }
}

template <bool O16>
static cudaError_t gather_t(const GatherParams &p, int v_type, int k_type, int blocks, cudaStream_t s, bool pdl)
{
    void (*fn)(GatherParams) =
        k_type == KVQ_K_F16 ? (v_type == KVQ_V_Q4_0 ? gather_kernel<KVQ_V_Q4_0, KVQ_K_F16, O16> : gather_kernel<KVQ_V_Q8_0, KVQ_K_F16, O16>)
                            : (v_type == KVQ_V_Q4_0 ? gather_kernel<KVQ_V_Q4_0, KVQ_K_I8, O16> : gather_kernel<KVQ_V_Q8_0, KVQ_K_I8, O16>);
    return launch_pdl(fn, p, blocks, kGatherWarps * 32, 0, s, pdl);
}

cudaError_t launch_gather_many(const PagedRowsParams &rows, int v_type, int k_type, int out_type, int n_sms, cudaStream_t s, bool pdl)
{
    GatherParams p = {rows.pool, rows.slots, rows.n_tokens, rows.k_out, rows.v_out, 1, 1};
    const long long windows = ((long long)p.n_tokens + 7) / 8;
    // Heads to a warp while 48 warps are left for every SM (8192 tokens: 15.5 us at 24, 14.7 at 48, 14.6 at 96).
    const long long want = windows * p.pool.n_kv_heads / ((long long)n_sms * 48);
    p.heads = want < 1 ? 1 : want > p.pool.n_kv_heads ? p.pool.n_kv_heads : (int)want;
    p.chunks = (p.pool.n_kv_heads + p.heads - 1) / p.heads;
    const int blocks = (int)((windows * p.chunks + kGatherWarps - 1) / kGatherWarps);
    return out_type == KVQ_OUT_F16 ? gather_t<true>(p, v_type, k_type, blocks, s, pdl) : gather_t<false>(p, v_type, k_type, blocks, s, pdl);
}

// ---------------------------------------------------------------------------
// Move: a quad of lanes takes a token of a head (kvq_quad.cuh), a warp eight at a
// time: four pairs of tokens whose new slots are an even place and the next, which
// share words of V codes, or, where the list has no pairs, eight tokens.  A warp
// looks at eight tokens of the list and goes over some of the heads; angles are worked
// out once for those.  A key's codes are turned as code * scale in fp32, rounded to
// fp16 and quantized anew, as an append would; a key that does not turn keeps its bits.
//
// Where tokens move, each slot may be another's source, so more than a few rows go
// through the workspace (one launch out, one in) unless the caller says that none is.  8092 tokens
// of 8 heads (q8_0 V, keys turned): 35 MB in and out, 5.2 us at a copy's rate; directly
// 11.7 us, through the workspace, which doubles the bytes, 15.7.  Both wait for rows: a
// quad whose keys turn has one in flight at a time.  Pairs half of part of a head apart
// pass through shared memory and back (16.4 and 22.8 us).  F16 K goes word by word, 18.0
// and 31.4 us for 7.5.  131072 keys turned where they lie 61 us, 4.7 TB/s, 0.69 of a
// copy's rate: instructions, some 400 for eight rows (codes to numbers, the turn,
// largest values, new codes), three quarters of what the SMs can issue.  There the next
// two heads' int8 keys are on their way in shared memory: loaded into registers when
// they are needed 71 us, a head ahead 77-99, since that costs more warps than the wait
// does; three heads ahead 62.  72 registers (seven blocks on an SM) 61, six blocks the
// same, five 63, eight 68; through the workspace six take 18.6.
// ---------------------------------------------------------------------------
constexpr int kMoveWarps = 4;
constexpr int kMoveTokens = 8;   // of a warp

// Which half of the way: from slots to slots, from slots to the staged rows, from those to slots.
constexpr int kMoveDirect = 0, kMoveOut = 1, kMoveIn = 2;

struct alignas(16) MoveShared {   // (read in words of 16 bytes, warp after warp)
    float cosines[kMoveTokens][kAngleRow], sines[kMoveTokens][kAngleRow];   // of the quads' turns; of row 0 alone where they are the same
    uint8_t list[kMoveTokens];
};

// The quad's key turned; SOME: only where `turns`, the others' stay as they are.
// scratch: the quad's 128 floats in shared memory (part).
template <bool SOME, int VT, int KT, int ROT>
__device__ __forceinline__ void turn_key(QuadRow<VT, KT> &r, bool turns, const float *cosines, const float *sines, int c, int n_rot, float *scratch)
{
    constexpr int kWords = KT == KVQ_K_F16 ? 4 : 2;   // of a block
    const float2 s01 = half2_of(r.ks[0]), s23 = half2_of(r.ks[1]);
    const float scale[4] = {s01.x, s01.y, s23.x, s23.y};
    Quad16 h;
    if (ROT == kRotHalf) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            float2 x[4], y[4];
            key_floats<KT, ROT>(r.k + kWords * b, scale[b], x);
            key_floats<KT, ROT>(r.k + kWords * (b + 2), scale[b + 2], y);
            quad_turn8(x, y, cosines, sines, 32 * b + 8 * c);
            h.b[b] = quad_halves<ROT>(x);
            h.b[b + 2] = quad_halves<ROT>(y);
        }
    } else if (ROT == kRotPairs) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            float2 x[4];
            key_floats<KT, ROT>(r.k + kWords * b, scale[b], x);
            if (32 * b + 8 * c < n_rot) quad_turn4(x, cosines, sines, 16 * b + 4 * c);   // all of the lane's four pairs or none
            h.b[b] = quad_halves<ROT>(x);
        }
    } else {   // neighbours to group pairs, and back
        float2 x[4];
        __syncwarp();
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            key_floats<KT, ROT>(r.k + kWords * b, scale[b], x);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                *reinterpret_cast<float4 *>(scratch + 32 * b + 8 * c + 4 * k) = make_float4(x[2 * k].x, x[2 * k].y, x[2 * k + 1].x, x[2 * k + 1].y);
        }
        __syncwarp();
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const PartGroups g(c + 4 * b, n_rot);
            float4 *const first = reinterpret_cast<float4 *>(scratch + g.a), *const second = reinterpret_cast<float4 *>(scratch + g.b);
            const float4 u = *first, v = *second;
            x[0] = make_float2(u.x, u.y);
            x[1] = make_float2(u.z, u.w);
            x[2] = make_float2(v.x, v.y);
            x[3] = make_float2(v.z, v.w);
            if (g.rotates) quad_turn4(x, cosines, sines, 4 * (c + 4 * b));
            *first = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
            *second = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
        }
        __syncwarp();
#pragma unroll
        for (int b = 0; b < 4; ++b) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float4 u = *reinterpret_cast<const float4 *>(scratch + 32 * b + 8 * c + 4 * k);
                x[2 * k] = make_float2(u.x, u.y);
                x[2 * k + 1] = make_float2(u.z, u.w);
            }
            h.b[b] = quad_halves<kRotNone>(x);
        }
    }
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
    const QuadCodes q = quad_quantize(h);
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

// A lane's rates: of pairs lane and lane + 32; loaded once for all tokens (64 tokens of
// move_once_kernel 3.5 us, 4.9 with a load for each token's angles).
struct MoveRates {
    unsigned long long r[2];
    __device__ __forceinline__ explicit MoveRates(const RopeDesc &rope)
    {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = (int)(threadIdx.x & 31) + 32 * i;
            r[i] = j < rope.n_rot / 2 ? rope.turns[j] : 0;
        }
    }
};
// Angles of the quads' turns, one row for all where they are the same; the lane's
// row.  Called by the whole warp, some of whose quads turn.
__device__ __forceinline__ int move_angles(MoveShared &sh, const MoveRates &rates, int turn, bool turns)
{
    const int lane = threadIdx.x & 31;
    const int one = __shfl_sync(0xffffffffu, turn, __ffs(__ballot_sync(0xffffffffu, turns)) - 1);
    const bool same = __all_sync(0xffffffffu, !turns || turn == one);
    __syncwarp();   // the rows before may still be read
    for (int k = 0; k < (same ? 1 : kMoveTokens); ++k) {
        const int t = same ? one : __shfl_sync(0xffffffffu, turn, 4 * k);
#pragma unroll
        for (int i = 0; i < 2; ++i) {   // (behind n_rot / 2 nobody reads)
            const float2 a = angle_of(rates.r[i], t, 1.f);
            sh.cosines[k][lane + 32 * i] = a.x;
            sh.sines[k][lane + 32 * i] = a.y;
        }
    }
    __syncwarp();
    return same ? 0 : lane >> 2;
}

template <int VT, int KT, int ROT, int WAY>
__global__ void __launch_bounds__(kMoveWarps * 32, 7) move_kernel(const MoveParams p)
{
    constexpr int kTile = PageTile<VT, KT>::BYTES, kRow = Staged<VT, KT>::BYTES;
    __shared__ __align__(16) MoveShared shared[kMoveWarps];
    __shared__ __align__(16) float scratch[ROT == kRotPart ? kMoveWarps : 1][8][ROT == kRotPart ? kD + 4 : 1];
    constexpr bool kRinged = WAY == kMoveDirect && KT == KVQ_K_I8 && ROT != kRotNone;
    __shared__ uint4 ring[kRinged ? kMoveWarps : 1][2][3][kRinged ? 32 : 1];   // K codes and scales of two heads, for keys that turn where they lie
    pdl_wait();
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
        auto clear = [](QuadRow<VT, KT> &r) {
#pragma unroll
            for (int k = 0; k < QuadRow<VT, KT>::KW; ++k) r.k[k] = 0;
#pragma unroll
            for (int k = 0; k < QuadRow<VT, KT>::VW; ++k) r.v[k] = 0;
            r.ks[0] = r.ks[1] = r.vs = 0;
        };
        clear(r);
        auto get = [&](QuadRow<VT, KT> &r) {
            if (!mine) return;
            if (WAY == kMoveIn) {
                stage_get<VT, KT>(staged, r, c);
            } else {
                quad_get_key<VT, KT>(r, src, fu, c);
                if (values) quad_get_value<VT, KT>(r, src, fu, c);
            }
        };
        const bool ringed = kRinged && !values;
        auto fetch = [&](int h, int at) {
            if (mine && h < h1) {
                const uint8_t *tile = src + (size_t)(h - h0) * head_bytes;
                const uint32_t to = smem_u32(&ring[warp][at][0][lane]);
                copy16(to, tile + quad_k_off(fu, c, 0));
                copy16(to + 512, tile + quad_k_off(fu, c, 1));
                copy16(to + 1024, tile + PageTile<VT, KT>::KS_OFF + 16 * (fu / 2));
            }
            copy_commit();
        };
        if (ringed) {   // the first heads' rows, on their way while the angles are worked out
            fetch(h0, 0);
            fetch(h0 + 1, 1);
        } else {
            get(r);
        }
        const int row = ROT != kRotNone && any ? move_angles(sh, MoveRates(p.rope), turn, turns) : 0;
        const float *cosines = sh.cosines[row], *sines = sh.sines[row];
        float *const mem = scratch[ROT == kRotPart ? warp : 0][ROT == kRotPart ? quad : 0];
        if (ringed) {
            for (int h = h0, at = 0; h < h1; ++h, at ^= 1) {
                copy_wait<1>();
                if (mine) {
                    const uint4 a = ring[warp][at][0][lane], b = ring[warp][at][1][lane], s = ring[warp][at][2][lane];
                    const uint32_t sel = fu & 1 ? 0x7632 : 0x5410;
                    r.k[0] = a.x, r.k[1] = a.y, r.k[2] = a.z, r.k[3] = a.w;
                    r.k[4] = b.x, r.k[5] = b.y, r.k[6] = b.z, r.k[7] = b.w;
                    r.ks[0] = __byte_perm(s.x, s.y, sel);
                    r.ks[1] = __byte_perm(s.z, s.w, sel);
                }
                turn_key<false, VT, KT, ROT>(r, true, cosines, sines, c, p.rope.n_rot, mem);
                if (turns) quad_put_key<VT, KT>(r, dst, tu, c);
                dst += head_bytes;
                __syncwarp();   // the row has been read: its place may be filled again
                fetch(h + 2, at);
            }
            copy_wait<0>();
            continue;
        }
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
            src += head_bytes;
            QuadRow<VT, KT> next;   // (without a turn there are registers for it: 16.3 us through the workspace without)
            clear(next);
            uint8_t *const to_staged = staged;
            staged += kRow;
            if (ROT == kRotNone && h + 1 < h1) get(next);
            if (WAY == kMoveOut) {
                if (mine) stage_put<VT, KT>(to_staged, r, c);
            } else {
                if (mine) quad_put_key<VT, KT>(r, dst, tu, c);
                quad_put_value<VT, KT>(r, dst, tu, c, pair, mine);
            }
            if (++h >= h1) break;
            dst += head_bytes;
            if (ROT == kRotNone) r = next;
            else get(r);
        }
    }
}

// Few tokens that may be one another's source: a cluster takes all of them, of one
// head, in registers, and writes none before every one has been read.  A launch less
// than by way of the workspace: 64 tokens of 8 heads (q4_0 V) 2.4 us against 5.0, with
// keys turned, each otherwise, 3.5 against 5.6; F16 K and q8_0 V, no two slots neighbours, 3.6 against
// 9.6, 256 tokens 9.1 against 10.2 (bytes stored one by one: an SM's store unit; so the
// tokens go to as many CTAs as there are: 64 in two 7.2).  Clusters of more than eight
// CTAs are not portable, and with 512 tokens the way through the workspace is as fast.
template <int VT, int KT, int ROT>
__global__ void __launch_bounds__(kMoveWarps * 32) move_once_kernel(const MoveParams p)
{
    constexpr int kTile = PageTile<VT, KT>::BYTES;
    __shared__ __align__(16) MoveShared shared[kMoveWarps];
    __shared__ __align__(16) float scratch[ROT == kRotPart ? kMoveWarps : 1][8][ROT == kRotPart ? kD + 4 : 1];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & 3, quad = lane >> 2;
    MoveShared &sh = shared[warp];
    const int h = (int)blockIdx.x / p.chunks, t0 = (((int)blockIdx.x - h * p.chunks) * (int)(blockDim.x / 32) + warp) * kMoveTokens;
    const int at = t0 - 1 + lane;
    const bool there = lane < kMoveTokens + 2 && at >= 0 && at < p.n_tokens;
    const int from_all = there ? p.from[at] : -1, to_all = there ? p.to[at] : -1;
    const int turn_all = ROT != kRotNone && there ? p.turn[at] : 0;
    const MoveRates rates(p.rope);   // (n_rot is 0 without a turn)
    auto inside = [&](int slot) { return slot >= 0 && slot < p.pool.n_slots; };
    const SlotPairs q = slot_pairs(to_all, t0 < p.n_tokens && inside(from_all) && inside(to_all), kMoveTokens);
    slot_list(q, sh.list);
    const bool pairs = (q.pair & q.lead) != 0;
    const int e = pairs ? quad & 1 : 0, P1 = (1 << p.pool.pshift) - 1;
    constexpr int kGroups = 2;   // four pairs each, or all eight tokens in the first
    QuadRow<VT, KT> r[kGroups];
    int to[kGroups];
    bool pair[kGroups], mine[kGroups], turns[kGroups];
    int turn[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        const int n = pairs ? 4 * g + (quad >> 1) : 8 * g + quad;
        const int lead = n < q.leads ? sh.list[n] : 1;
        pair[g] = n < q.leads && (q.pair >> lead & 1);
        mine[g] = n < q.leads && (e == 0 || pair[g]);
        const int i = lead + (pair[g] ? e : 0), from = __shfl_sync(0xffffffffu, from_all, i);
        to[g] = __shfl_sync(0xffffffffu, to_all, i);
        turn[g] = __shfl_sync(0xffffffffu, turn_all, i);
        turns[g] = mine[g] && turn[g] != 0;
#pragma unroll
        for (int k = 0; k < QuadRow<VT, KT>::KW; ++k) r[g].k[k] = 0;
#pragma unroll
        for (int k = 0; k < QuadRow<VT, KT>::VW; ++k) r[g].v[k] = 0;
        r[g].ks[0] = r[g].ks[1] = r[g].vs = 0;
        if (mine[g]) {
            const uint8_t *src = tile_of(p.pool, from >> p.pool.pshift, h, (from & P1) >> 4, kTile);
            quad_get_key<VT, KT>(r[g], src, from & 15, c);
            quad_get_value<VT, KT>(r[g], src, from & 15, c);
        }
    }
    if (ROT != kRotNone) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
            if (__any_sync(0xffffffffu, turns[g])) {
                const int row = move_angles(sh, rates, turn[g], turns[g]);
                turn_key<true, VT, KT, ROT>(r[g], turns[g], sh.cosines[row], sh.sines[row], c, p.rope.n_rot, scratch[ROT == kRotPart ? warp : 0][ROT == kRotPart ? quad : 0]);
            }
    }
    cluster_sync();
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        if (!__any_sync(0xffffffffu, mine[g])) continue;
        uint8_t *dst = tile_of(p.pool, to[g] >> p.pool.pshift, h, (to[g] & P1) >> 4, kTile);
        if (mine[g]) quad_put_key<VT, KT>(r[g], dst, to[g] & 15, c);
        quad_put_value<VT, KT>(r[g], dst, to[g] & 15, c, pair[g], mine[g]);
    }
}
constexpr int kOnceCtas = 8;   // of a cluster

template <int VT, int KT, int ROT>
static cudaError_t move_once(const MoveParams &in, cudaStream_t s, bool pdl)
{
    MoveParams p = in;
    p.heads = 1;
    const int windows = (p.n_tokens + kMoveTokens - 1) / kMoveTokens;
    p.chunks = 1;   // CTAs of a cluster
    while (p.chunks < kOnceCtas && p.chunks < windows) p.chunks *= 2;
    const int warps = (windows + p.chunks - 1) / p.chunks;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.chunks * p.pool.n_kv_heads);
    cfg.blockDim = dim3(warps * 32);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = p.chunks;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, move_once_kernel<VT, KT, ROT>, p);
}

template <int VT, int KT, int ROT>
static cudaError_t move_t(const MoveParams &p, int blocks, cudaStream_t s, bool pdl)
{
    if (p.rows && p.n_tokens <= kOnceCtas * kMoveWarps * kMoveTokens) return move_once<VT, KT, ROT>(p, s, pdl);
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
    // All heads to a warp, which works its angles out once, as long as that leaves 24 warps for every SM (8092 tokens
    // through the workspace: 18.7 us at 12, 16.4 at 24, 18.3 at 48; 131072 alike).
    const long long want = windows * p.pool.n_kv_heads / ((long long)n_sms * 24);
    p.heads = want < 1 ? 1 : want > p.pool.n_kv_heads ? p.pool.n_kv_heads : (int)want;
    p.chunks = (p.pool.n_kv_heads + p.heads - 1) / p.heads;
    const int blocks = (int)((windows * p.chunks + kMoveWarps - 1) / kMoveWarps);
    if (v_type == KVQ_V_Q4_0) return k_type == KVQ_K_F16 ? move_rot<KVQ_V_Q4_0, KVQ_K_F16>(p, blocks, s, pdl) : move_rot<KVQ_V_Q4_0, KVQ_K_I8>(p, blocks, s, pdl);
    return k_type == KVQ_K_F16 ? move_rot<KVQ_V_Q8_0, KVQ_K_F16>(p, blocks, s, pdl) : move_rot<KVQ_V_Q8_0, KVQ_K_I8>(p, blocks, s, pdl);
}

}  // namespace kvq
