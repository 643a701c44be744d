// kvq_tokens_api.cu -- the C ABI of include/kvq_tokens.h: argument checks and
// launches.  Nothing here allocates, throws or synchronizes.
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>

#include "kvq_paged_host.cuh"
#include "kvq_tokens.cuh"

using namespace kvq;

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

std::mutex g_mu;
bool g_ready[kMaxDevices];

// The current device's SM count; its kernels' attributes are set by the first call.
kvq_status tokens_setup(int *n_sms)
{
    int dev = 0;
    unsigned int *timeouts = nullptr;
    const kvq_status st = device_common(&dev, n_sms, &timeouts);
    if (st != KVQ_OK) return st;
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_ready[dev]) {
        cudaError_t e = prepare_qkv();
        if (e == cudaSuccess) e = prepare_page_fork();
        if (e != cudaSuccess) return done(e);
        g_ready[dev] = true;
    }
    return KVQ_OK;
}

kvq_status check_rope(const kvq_rope *r)
{
    if (!r) return KVQ_OK;
    if (r->n_rot < 0 || r->n_rot > KVQ_HEAD_DIM || r->n_rot % 8) return KVQ_ERR_INVALID_ARG;
    if ((r->layout != KVQ_ROPE_HALF && r->layout != KVQ_ROPE_PAIRS) || !std::isfinite(r->amplitude)) return KVQ_ERR_INVALID_ARG;
    return r->n_rot > 0 && (!r->turns || !aligned(r->turns, 8)) ? KVQ_ERR_INVALID_ARG : KVQ_OK;
}

RopeDesc rope_of(const kvq_rope *r)
{
    if (!r || r->n_rot == 0) return RopeDesc{nullptr, 0, 1, 1.f};
    return RopeDesc{reinterpret_cast<const unsigned long long *>(r->turns), r->n_rot, r->layout == KVQ_ROPE_PAIRS, r->amplitude};
}

// fp16 rows [tokens][heads][head_dim] with a token stride.
bool rows_ok(const void *p, int64_t stride, int heads)
{
    return p && aligned(p, 16) && stride % 8 == 0 && stride >= (int64_t)heads * kD;
}
bool norm_ok(const float *p) { return aligned(p, 16); }

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

struct ForkPlan {
    size_t marks, owner, seqs, counts, totals, bytes;   // bytes of one kind of marks, offsets, and all
    int blocks;
};
ForkPlan plan_fork(int n_seqs, int n_pages)
{
    ForkPlan f;
    f.blocks = n_pages / 4096 + 1 < 1024 ? n_pages / 4096 + 1 : 1024;   // 4 pages a thread, more in very large pools
    f.marks = up256((size_t)n_pages);
    f.owner = 3 * f.marks;
    f.seqs = f.owner + up256((size_t)n_pages * sizeof(int));
    f.counts = f.seqs + up256(8 * (size_t)n_seqs * sizeof(int));
    f.totals = f.counts + up256((size_t)f.blocks * sizeof(int));
    f.bytes = f.totals + up256(2 * sizeof(int));
    return f;
}

bool move_size_ok(const kvq_pages *p, int n_tokens) { return n_tokens >= 0 && (long long)n_tokens * p->n_kv_heads <= INT_MAX / 2; }

}  // namespace

extern "C" {

kvq_status kvq_rope_turns(int32_t n_rot, double base, int32_t scaling, double factor, double original, double fast, double slow,
                          uint64_t *turns, float *amplitude)
{
    if (n_rot < 0 || n_rot > KVQ_HEAD_DIM || n_rot % 8 || !amplitude || (n_rot > 0 && !turns)) return KVQ_ERR_INVALID_ARG;
    if (scaling < KVQ_ROPE_PLAIN || scaling > KVQ_ROPE_BY_TURNS || !std::isfinite(base) || !(base > 1)) return KVQ_ERR_INVALID_ARG;
    if (scaling != KVQ_ROPE_PLAIN && !(std::isfinite(factor) && factor > 0)) return KVQ_ERR_INVALID_ARG;
    const bool blend = scaling == KVQ_ROPE_BY_INDEX || scaling == KVQ_ROPE_BY_TURNS;
    if (blend && !(std::isfinite(original) && original > 0 && std::isfinite(fast) && slow > 0 && fast > slow)) return KVQ_ERR_INVALID_ARG;
    if (scaling == KVQ_ROPE_BASE && n_rot > 0) base *= std::pow(factor, n_rot / (n_rot - 2.0));
    if (!std::isfinite(base) || !(base > 0)) return KVQ_ERR_INVALID_ARG;
    const float amp = scaling == KVQ_ROPE_BY_INDEX ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
    // the index of the pair that makes so many turns within `original`
    auto index_at = [&](double n) { return n_rot * std::log(original / (kTwoPi * n)) / (2 * std::log(base)); };
    double lo = 0, hi = 0;
    if (scaling == KVQ_ROPE_BY_INDEX) {
        lo = std::fmax(std::floor(index_at(fast)), 0.0);
        hi = std::fmin(std::ceil(index_at(slow)), n_rot - 1.0);
    }
    for (int i = 0; i < n_rot / 2; ++i) {
        double rate = std::pow(base, -2.0 * i / n_rot);
        double slowed = scaling == KVQ_ROPE_LINEAR ? 1 : 0;   // share of the slowed rate
        if (scaling == KVQ_ROPE_BY_INDEX) slowed = (i - lo) / std::fmax(hi - lo, 1e-3);
        if (scaling == KVQ_ROPE_BY_TURNS) slowed = (fast - original * rate / kTwoPi) / (fast - slow);
        slowed = std::fmin(std::fmax(slowed, 0.0), 1.0);
        if (slowed > 0) rate = rate / factor * slowed + rate * (1 - slowed);
        double part = rate / kTwoPi;
        part = std::floor(std::ldexp(part - std::floor(part), 64) + 0.5);
        turns[i] = part < 18446744073709551616.0 ? (uint64_t)part : 0;
    }
    *amplitude = amp;
    return KVQ_OK;
}

kvq_status kvq_page_positions(int32_t n_seqs, const int32_t *q_start, const int32_t *seq_lens, int32_t n_tokens, int32_t *positions,
                              void *stream)
{
    if (n_seqs < 0 || n_seqs > KVQ_MAX_PAGED_SEQS || n_tokens < 0 || n_tokens == INT_MAX) return KVQ_ERR_INVALID_ARG;
    if (n_tokens == 0) return KVQ_OK;
    if (!int_ptr(q_start) || (n_seqs > 0 && !int_ptr(seq_lens)) || !int_ptr(positions)) return KVQ_ERR_INVALID_ARG;
    int n_sms = 0;
    const kvq_status st = tokens_setup(&n_sms);
    if (st != KVQ_OK) return st;
    return done(launch_positions(PositionsParams{q_start, seq_lens, positions, n_seqs, n_tokens}, static_cast<cudaStream_t>(stream), pdl_on()));
}

kvq_status kvq_qkv(const kvq_qkv_desc *a, void *stream)
{
    if (!a || a->n_tokens < 0 || a->n_q_heads < 0 || a->n_q_heads > KVQ_MAX_HEADS || a->n_kv_heads < 0 || a->n_kv_heads > KVQ_MAX_HEADS)
        return KVQ_ERR_INVALID_ARG;
    if (!std::isfinite(a->eps) || a->eps < 0) return KVQ_ERR_INVALID_ARG;
    kvq_status st = check_rope(a->rope);
    if (st != KVQ_OK) return st;
    const bool keys = a->n_kv_heads > 0;
    if ((a->pages && a->k_out) || keys != (a->pages || a->k_out)) return KVQ_ERR_INVALID_ARG;
    if (a->pages) {
        st = check_pool(a->pages);
        if (st != KVQ_OK) return st;
        if (a->pages->n_kv_heads != a->n_kv_heads) return KVQ_ERR_INVALID_ARG;
    }
    if ((long long)a->n_tokens * (a->n_q_heads + a->n_kv_heads) > INT_MAX / 2) return KVQ_ERR_INVALID_ARG;
    if (a->n_tokens == 0 || a->n_q_heads + a->n_kv_heads == 0) return KVQ_OK;
    if (a->n_q_heads > 0 && (!rows_ok(a->q16, a->q_stride, a->n_q_heads) || !rows_ok(a->q_out, a->q_out_stride, a->n_q_heads)))
        return KVQ_ERR_INVALID_ARG;
    if (keys && !rows_ok(a->k16, a->k_stride, a->n_kv_heads)) return KVQ_ERR_INVALID_ARG;
    if (a->pages && !rows_ok(a->v16, a->v_stride, a->n_kv_heads)) return KVQ_ERR_INVALID_ARG;
    if (a->k_out && !rows_ok(a->k_out, a->k_out_stride, a->n_kv_heads)) return KVQ_ERR_INVALID_ARG;
    // in place a row is read and written by the same lanes, so the rows have to be the same ones
    if ((a->n_q_heads > 0 && a->q_out == a->q16 && a->q_out_stride != a->q_stride) || (a->k_out && a->k_out == a->k16 && a->k_out_stride != a->k_stride))
        return KVQ_ERR_INVALID_ARG;
    if (!norm_ok(a->q_norm) || !norm_ok(a->k_norm)) return KVQ_ERR_INVALID_ARG;
    if ((a->pages && !int_ptr(a->slots)) || !aligned(a->slots, 4)) return KVQ_ERR_INVALID_ARG;
    const RopeDesc rope = rope_of(a->rope);
    if (rope.n_rot > 0 && !int_ptr(a->positions)) return KVQ_ERR_INVALID_ARG;
    int n_sms = 0;
    st = tokens_setup(&n_sms);
    if (st != KVQ_OK) return st;
    QkvParams p = {};
    if (a->pages) p.pool = pool_of(a->pages);
    p.rope = rope;
    p.q = static_cast<const uint16_t *>(a->q16);
    p.k = static_cast<const uint16_t *>(a->k16);
    p.v = static_cast<const uint16_t *>(a->v16);
    p.q_stride = a->q_stride;
    p.k_stride = a->k_stride;
    p.v_stride = a->v_stride;
    p.q_out = static_cast<uint16_t *>(a->q_out);
    p.q_out_stride = a->q_out_stride;
    p.k_out = static_cast<uint16_t *>(a->k_out);
    p.k_out_stride = a->k_out_stride;
    p.q_norm = a->q_norm;
    p.k_norm = a->k_norm;
    p.positions = a->positions;
    p.slots = a->slots;
    p.eps = a->eps > 0 && a->eps < FLT_MIN ? FLT_MIN : a->eps;   // (below every mean of squares that is not 0)
    p.n_tokens = a->n_tokens;
    p.n_q_heads = a->n_q_heads;
    p.n_kv_heads = a->n_kv_heads;
    p.paged = a->pages != nullptr;
    return done(launch_qkv(p, a->pages ? a->pages->v_type : KVQ_V_Q4_0, a->pages ? a->pages->k_type : KVQ_K_I8, n_sms,
                           static_cast<cudaStream_t>(stream), pdl_on()));
}

kvq_status kvq_page_fork_workspace_size(int32_t n_seqs, int32_t n_pages, size_t *bytes)
{
    if (!bytes || n_seqs < 0 || n_seqs > KVQ_MAX_PAGED_SEQS || n_pages < 0) return KVQ_ERR_INVALID_ARG;
    *bytes = plan_fork(n_seqs, n_pages).bytes;
    return KVQ_OK;
}

kvq_status kvq_page_fork(int32_t n_seqs, int32_t page_tokens, int32_t n_pages, const int32_t *lens, const int32_t *parent,
                         const int32_t *keep, const int32_t *block_table, int32_t table_stride, int32_t max_blocks, int32_t *table_out,
                         int32_t out_stride, int32_t *lens_out, int32_t *free_pages, const int32_t *n_free, int32_t *n_free_out,
                         int32_t *copy_from, int32_t *copy_to, int32_t *copy_held, int32_t *status, void *workspace,
                         size_t workspace_bytes, void *stream)
{
    if (n_seqs < 0 || n_seqs > KVQ_MAX_PAGED_SEQS || page_shift(page_tokens) < 0 || n_pages < 0) return KVQ_ERR_INVALID_ARG;
    if ((long long)n_pages * page_tokens > INT_MAX || !table_ok(table_stride, max_blocks, page_tokens) || out_stride < max_blocks)
        return KVQ_ERR_INVALID_ARG;
    if (!int_ptr(n_free) || !int_ptr(n_free_out) || (n_pages > 0 && !int_ptr(free_pages))) return KVQ_ERR_INVALID_ARG;
    if (n_seqs > 0) {
        if (!int_ptr(lens) || !aligned(parent, 4) || !aligned(keep, 4) || !int_ptr(lens_out) || !int_ptr(status)) return KVQ_ERR_INVALID_ARG;
        if (!int_ptr(copy_from) || !int_ptr(copy_to) || !int_ptr(copy_held)) return KVQ_ERR_INVALID_ARG;
        if (max_blocks > 0 && (!int_ptr(block_table) || !int_ptr(table_out))) return KVQ_ERR_INVALID_ARG;
        if (max_blocks > 0 && table_out == block_table && (parent || out_stride != table_stride)) return KVQ_ERR_INVALID_ARG;
    }
    int n_sms = 0;
    const kvq_status st = tokens_setup(&n_sms);
    if (st != KVQ_OK) return st;
    const ForkPlan f = plan_fork(n_seqs, n_pages);
    if (!workspace || workspace_bytes < f.bytes || !aligned(workspace, 256)) return KVQ_ERR_WORKSPACE;
    ForkParams p = {};
    uint8_t *w = static_cast<uint8_t *>(workspace);
    p.lens = lens;
    p.parent = parent;
    p.keep = keep;
    p.table = block_table;
    p.n_free = n_free;
    p.table_out = table_out;
    p.lens_out = lens_out;
    p.free_pages = free_pages;
    p.n_free_out = n_free_out;
    p.copy_from = copy_from;
    p.copy_to = copy_to;
    p.copy_held = copy_held;
    p.status = status;
    p.old_mark = w;
    p.full_mark = w + f.marks;
    p.tail_mark = w + 2 * f.marks;
    p.owner = reinterpret_cast<int *>(w + f.owner);
    p.seqs = reinterpret_cast<int *>(w + f.seqs);
    p.counts = reinterpret_cast<int *>(w + f.counts);
    p.totals = reinterpret_cast<int *>(w + f.totals);
    p.blocks = f.blocks;
    p.n_seqs = n_seqs;
    p.pshift = page_shift(page_tokens);
    p.n_pages = n_pages;
    p.stride = table_stride;
    p.out_stride = out_stride;
    p.max_blocks = max_blocks;
    return done(launch_page_fork(p, n_sms, static_cast<cudaStream_t>(stream), pdl_on()));
}

kvq_status kvq_page_copy(const kvq_pages *pools, int32_t n_pools, const int32_t *from, const int32_t *to, const int32_t *held,
                         int32_t n_copies, void *stream)
{
    if (n_pools < 0 || n_pools > KVQ_MAX_COPY_POOLS || n_copies < 0 || (n_pools > 0 && !pools)) return KVQ_ERR_INVALID_ARG;
    int most = 0;
    for (int i = 0; i < n_pools; ++i) {
        const kvq_status st = check_pool(pools + i);
        if (st != KVQ_OK) return st;
        if (pools[i].n_pages != pools->n_pages || pools[i].page_tokens != pools->page_tokens) return KVQ_ERR_INVALID_ARG;
        most = pools[i].n_kv_heads > most ? pools[i].n_kv_heads : most;
    }
    if ((long long)n_pools * most * n_copies > 1 << 28) return KVQ_ERR_INVALID_ARG;
    if (n_copies == 0 || n_pools == 0 || pools->n_pages == 0) return KVQ_OK;
    if (!int_ptr(from) || !int_ptr(to) || !aligned(held, 4)) return KVQ_ERR_INVALID_ARG;
    int n_sms = 0;
    const kvq_status st = tokens_setup(&n_sms);
    if (st != KVQ_OK) return st;
    auto run = [&](auto &p) {
        for (int i = 0; i < n_pools; ++i) {
            p.data[i] = static_cast<uint8_t *>(pools[i].data);
            p.heads[i] = (uint16_t)pools[i].n_kv_heads;
            p.tile_bytes[i] = (uint16_t)page_tile_bytes(pools[i].v_type, pools[i].k_type);
        }
        p.from = from;
        p.to = to;
        p.held = held;
        p.n_pools = n_pools;
        p.n_copies = n_copies;
        p.n_pages = pools->n_pages;
        p.most_heads = most;
        p.tiles = pools->page_tokens / kWTile;
        return done(launch_page_copy(p, static_cast<cudaStream_t>(stream), pdl_on()));
    };
    if (n_pools <= kFewPools) {
        CopyParams<kFewPools> p;
        return run(p);
    }
    CopyParams<KVQ_MAX_COPY_POOLS> p;
    return run(p);
}

kvq_status kvq_paged_move_workspace_size(const kvq_pages *p, int32_t n_tokens, size_t *bytes)
{
    if (!bytes) return KVQ_ERR_INVALID_ARG;
    const kvq_status st = check_shape(p);
    if (st != KVQ_OK) return st;
    if (!move_size_ok(p, n_tokens)) return KVQ_ERR_INVALID_ARG;
    *bytes = (size_t)n_tokens * p->n_kv_heads * staged_row_bytes(p->v_type, p->k_type);
    return KVQ_OK;
}

kvq_status kvq_paged_move(const kvq_pages *p, const int32_t *from, const int32_t *to, int32_t n_tokens, const kvq_rope *rope,
                          const int32_t *turn, int32_t staged, void *workspace, size_t workspace_bytes, void *stream)
{
    kvq_status st = check_pool(p);
    if (st != KVQ_OK) return st;
    if (!move_size_ok(p, n_tokens) || (rope != nullptr) != (turn != nullptr) || !aligned(turn, 4)) return KVQ_ERR_INVALID_ARG;
    st = check_rope(rope);
    if (st != KVQ_OK) return st;
    if (n_tokens == 0 || p->n_pages == 0) return KVQ_OK;
    if (!int_ptr(from) || !int_ptr(to)) return KVQ_ERR_INVALID_ARG;
    int n_sms = 0;
    st = tokens_setup(&n_sms);
    if (st != KVQ_OK) return st;
    size_t need = 0;
    if (staged) kvq_paged_move_workspace_size(p, n_tokens, &need);
    if (staged && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return KVQ_ERR_WORKSPACE;
    MoveParams m = {};
    m.pool = pool_of(p);
    m.rope = rope_of(rope);
    m.from = from;
    m.to = to;
    m.turn = m.rope.n_rot > 0 ? turn : nullptr;
    m.n_tokens = n_tokens;
    m.rows = staged ? static_cast<uint8_t *>(workspace) : nullptr;
    return done(launch_paged_move(m, p->v_type, p->k_type, n_sms, static_cast<cudaStream_t>(stream), pdl_on()));
}

}  // extern "C"
