// kvq_paged_api.cu -- the C ABI of the paged cache (include/kvq_paged.h):
// argument checks, workspace layout and launches.  Nothing here allocates,
// throws or synchronizes.
#include <climits>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "kvq_paged.cuh"

using namespace kvq;

namespace {

constexpr int kMaxDevices = 64;

bool pdl_on()
{
    const char *e = std::getenv("KVQ_PDL");
    return !(e && e[0] == '0');
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool int_ptr(const void *p) { return p && aligned(p, 4); }

struct PagedDevice {
    bool ready = false;
    int ctas[2][2][3][2] = {};   // [k_type][v_type][nt][out_type] resident CTAs per SM
};
std::mutex g_mu;
PagedDevice g_dev[kMaxDevices];

kvq_status paged_setup(PagedDevice **out, int *n_sms, unsigned int **timeouts)
{
    int dev = 0;
    const kvq_status st = device_common(&dev, n_sms, timeouts);
    if (st != KVQ_OK) return st;
    std::lock_guard<std::mutex> lk(g_mu);
    PagedDevice &d = g_dev[dev];
    if (!d.ready) {
        cudaError_t e = prepare_page_tables();
        for (int kt = 0; kt < 2; ++kt)
            for (int nt = 1; nt <= 2; ++nt)
                for (int ot = 0; ot < 2; ++ot) {
                    if (e == cudaSuccess) e = prepare_paged_q4(nt, kt, ot, &d.ctas[kt][KVQ_V_Q4_0][nt][ot]);
                    if (e == cudaSuccess) e = prepare_paged_q8(nt, kt, ot, &d.ctas[kt][KVQ_V_Q8_0][nt][ot]);
                }
        if (e == cudaSuccess) e = prepare_chunk_q4();
        if (e == cudaSuccess) e = prepare_chunk_q8();
        if (e != cudaSuccess) {
            cudaGetLastError();
            return KVQ_ERR_CUDA;
        }
        d.ready = true;
    }
    *out = &d;
    return KVQ_OK;
}

kvq_status done(cudaError_t e)
{
    if (e == cudaSuccess) return KVQ_OK;
    cudaGetLastError();
    return KVQ_ERR_CUDA;
}

int page_shift(int tokens)
{
    for (int s = 4; s <= 8; ++s)
        if (tokens == 1 << s) return s;
    return -1;
}

// Shape of a pool (data aside).
kvq_status check_shape(const kvq_pages *p)
{
    if (!p || p->n_pages < 0 || page_shift(p->page_tokens) < 0) return KVQ_ERR_INVALID_ARG;
    if (p->n_kv_heads < 1 || p->n_kv_heads > KVQ_MAX_HEADS) return KVQ_ERR_INVALID_ARG;
    if ((p->v_type != KVQ_V_Q4_0 && p->v_type != KVQ_V_Q8_0) || (p->k_type != KVQ_K_I8 && p->k_type != KVQ_K_F16))
        return KVQ_ERR_INVALID_ARG;
    if (p->head_dim != KVQ_HEAD_DIM) return p->head_dim % KVQ_QBLOCK ? KVQ_ERR_INVALID_ARG : KVQ_ERR_UNSUPPORTED;
    if ((long long)p->n_pages * p->page_tokens > INT_MAX) return KVQ_ERR_INVALID_ARG;
    return KVQ_OK;
}

kvq_status check_pool(const kvq_pages *p)
{
    const kvq_status st = check_shape(p);
    if (st != KVQ_OK) return st;
    return p->n_pages > 0 && (!p->data || !aligned(p->data, 128)) ? KVQ_ERR_INVALID_ARG : KVQ_OK;
}

PoolDesc pool_of(const kvq_pages *p)
{
    return PoolDesc{static_cast<uint8_t *>(p->data), p->n_pages, p->n_pages * p->page_tokens, page_shift(p->page_tokens),
                    p->n_kv_heads};
}

// A table row of max_blocks pages holds fewer than 2^30 positions.
bool table_ok(int stride, int max_blocks, int page_tokens)
{
    return max_blocks >= 0 && stride >= max_blocks && (long long)max_blocks * page_tokens <= 1 << 30;
}

// ---- attention ----
// One launch: its CTAs (0: not made), its row tile, the rows per kv head of the
// sequences it takes, and where its pieces lie in the workspace.
struct Part {
    int n_ctas = 0, rows = 0, least = 0, most = 0;
    size_t cut_off = 0, lse_off = 0, o_off = 0, sum_off = 0;
};

struct AttnPlan {
    int gmax;            // query heads of the busiest kv head
    int uniform;
    Part part[kAttnParts];   // row tiles of 8 rows, of 16 rows, the chunk kernel
    size_t bytes;
    uint16_t grp_begin[KVQ_MAX_HEADS + 1];
    uint8_t grp_q[KVQ_MAX_HEADS];
};

// Rows per kv head from which a sequence goes to the chunk kernel (int8 K);
// KVQ_TC_ROWS and KVQ_PREFILL steer it as they steer kvq_decode_attn's.
constexpr int kChunkMinRows = KVQ_MAX_ROWS + 1;
int chunk_min_rows(const kvq_pages *g)
{
    const char *off = std::getenv("KVQ_PREFILL"), *e = std::getenv("KVQ_TC_ROWS");
    if (g->k_type != KVQ_K_I8 || (off && off[0] == '0')) return INT_MAX;
    return e && std::atoi(e) > 0 ? std::atoi(e) : kChunkMinRows;
}

kvq_status check_attn(const kvq_paged_desc *a, AttnPlan &pl)
{
    if (!a) return KVQ_ERR_INVALID_ARG;
    const kvq_status st = check_shape(a->pages);
    if (st != KVQ_OK) return st;
    const int H = a->pages->n_kv_heads, Hq = a->n_q_heads;
    if (Hq < 1 || Hq > KVQ_MAX_HEADS || a->n_tokens < 0 || a->n_seqs < 0 || a->n_seqs > KVQ_MAX_PAGED_SEQS)
        return KVQ_ERR_INVALID_ARG;
    if ((long long)a->n_tokens * Hq > INT_MAX / 2) return KVQ_ERR_INVALID_ARG;
    if (!table_ok(a->table_stride, a->max_blocks, a->pages->page_tokens)) return KVQ_ERR_INVALID_ARG;
    if (!std::isfinite(a->sm_scale) || (a->out_type != KVQ_OUT_F32 && a->out_type != KVQ_OUT_F16)) return KVQ_ERR_INVALID_ARG;
    int cnt[KVQ_MAX_HEADS] = {}, kv[KVQ_MAX_HEADS];
    if (!a->head_map && Hq % H) return KVQ_ERR_INVALID_ARG;
    for (int h = 0; h < Hq; ++h) {
        kv[h] = a->head_map ? a->head_map[h] : h / (Hq / H);
        if (kv[h] < 0 || kv[h] >= H) return KVQ_ERR_INVALID_ARG;
        ++cnt[kv[h]];
    }
    int n = 0;
    pl.gmax = 0;
    for (int k = 0; k < H; ++k) {
        pl.grp_begin[k] = (uint16_t)n;
        pl.gmax = cnt[k] > pl.gmax ? cnt[k] : pl.gmax;
        for (int h = 0; h < Hq; ++h)
            if (kv[h] == k) pl.grp_q[n++] = (uint8_t)h;
    }
    pl.grp_begin[H] = (uint16_t)n;
    pl.uniform = 1;
    for (int k = 0; k < H; ++k) pl.uniform = pl.uniform && cnt[k] == pl.gmax;
    if (a->n_tokens > 0 && a->n_seqs > 0 && (a->max_q < 1 || a->max_q > a->n_tokens)) return KVQ_ERR_INVALID_ARG;
    if ((long long)a->max_q * pl.gmax > 1 << 26) return KVQ_ERR_INVALID_ARG;   // PagedCut: a row tile's number has 23 bits
    return KVQ_OK;
}

bool idle(const kvq_paged_desc *a) { return a->n_tokens == 0 || a->n_seqs == 0; }

// No more CTAs than the longest possible batch has pieces of `least` units of
// `unit` positions.
void size_part(const kvq_paged_desc *a, const AttnPlan &pl, Part &pt, int ctas, int rows, int unit, int least, size_t &at)
{
    const long long tiles = ((long long)a->max_q * pl.gmax + rows - 1) / rows;
    const long long len = ((long long)a->max_blocks * a->pages->page_tokens + unit - 1) / unit;
    const double most = (double)a->n_seqs * a->pages->n_kv_heads * tiles * (len > 1 ? len : 1) / least + 1.0;
    pt.n_ctas = most < ctas ? (int)most : ctas;
    pt.rows = rows;
    const size_t slots = (size_t)pt.n_ctas * 2;
    auto take = [&](size_t n) {
        const size_t off = at;
        at += (n + 255) / 256 * 256;
        return off;
    };
    pt.cut_off = take(slots * sizeof(PagedCut));
    pt.lse_off = take(slots * rows * sizeof(float));
    pt.o_off = take(slots * rows * kD * sizeof(float));
}

void plan_attn(const kvq_paged_desc *a, const PagedDevice *dev, int n_sms, AttnPlan &pl)
{
    const kvq_pages *g = a->pages;
    const long long rows = (long long)a->max_q * pl.gmax;   // most rows of a sequence per kv head
    const int chunk = chunk_min_rows(g), bound[kAttnParts + 1] = {1, chunk < 9 ? chunk : 9, chunk, INT_MAX};
    int top = 0;   // the kind that the longest sequence goes to
    while (top < kAttnParts - 1 && rows >= bound[top + 1]) ++top;
    // Sequences that all have max_q rows, as n_tokens then says, are one launch
    // (an idle one costs 3 to 5 us).  What q_start holds is known on the device
    // alone, so that launch takes fewer rows too: row tiles of 16 at up to 1.4
    // times the cost of row tiles of 8, the chunk kernel at several times, which
    // is why it stands for others only where there is a single sequence.
    // Otherwise each sequence goes to its kind (40 single tokens beside four
    // chunks: 315 us, with row tiles of 16 for all the short ones 351).
    const bool alike = (long long)a->n_seqs * a->max_q == a->n_tokens && (top < 2 || a->n_seqs == 1);
    pl.bytes = 0;
    for (int k = 0; k < kAttnParts; ++k) {
        Part &pt = pl.part[k];
        pt = Part();
        if (k > top || (alike && k != top) || bound[k] >= bound[k + 1]) continue;
        pt.least = alike ? 1 : bound[k];
        pt.most = k == top ? INT_MAX : bound[k + 1] - 1;
        if (k < 2) {
            const int per_sm = dev->ctas[g->k_type][g->v_type][k + 1][a->out_type];
            size_part(a, pl, pt, n_sms * (per_sm > 0 ? per_sm : 1), 8 * (k + 1), kStagePos, kPagedMinStages, pl.bytes);
        } else {
            size_part(a, pl, pt, n_sms, kChunkRows, kChunkPositions, kChunkMinTiles, pl.bytes);
            pt.sum_off = pl.bytes;
            pl.bytes += ((size_t)pt.n_ctas * kChunkSums * sizeof(float) + 255) / 256 * 256;
        }
    }
}

// kvq_paged_attn; lose >= 0: with the test flavours, which leave out that copy.
kvq_status run_attn(const kvq_paged_desc *a, void *workspace, size_t workspace_bytes, void *stream, int lose)
{
    AttnPlan pl;
    kvq_status st = check_attn(a, pl);
    if (st != KVQ_OK) return st;
    st = check_pool(a->pages);
    if (st != KVQ_OK) return st;
    if (lose >= 0 && (a->pages->k_type != KVQ_K_I8 || a->pages->v_type != KVQ_V_Q4_0 || a->out_type != KVQ_OUT_F32)) return KVQ_ERR_UNSUPPORTED;
    if (idle(a)) return KVQ_OK;
    const int Hq = a->n_q_heads;
    if (!a->q16 || !aligned(a->q16, 16) || a->q_stride % 8 || a->q_stride < (int64_t)Hq * kD) return KVQ_ERR_INVALID_ARG;
    if (!int_ptr(a->q_start) || !int_ptr(a->seq_lens) || (a->max_blocks > 0 && !int_ptr(a->block_table))) return KVQ_ERR_INVALID_ARG;
    if (!a->out || !aligned(a->out, 16) || !aligned(a->lse, 4)) return KVQ_ERR_INVALID_ARG;
    PagedDevice *dev = nullptr;
    int n_sms = 0;
    unsigned int *timeouts = nullptr;
    st = paged_setup(&dev, &n_sms, &timeouts);
    if (st != KVQ_OK) return st;
    plan_attn(a, dev, n_sms, pl);
    if (!workspace || workspace_bytes < pl.bytes || !aligned(workspace, 256)) return KVQ_ERR_WORKSPACE;
    static thread_local PagedAttnParams p;
    std::memset(&p, 0, sizeof(p));
    p.pool = pool_of(a->pages);
    p.q = static_cast<const uint16_t *>(a->q16);
    p.q_stride = a->q_stride;
    p.q_start = a->q_start;
    p.seq_lens = a->seq_lens;
    p.block_table = a->block_table;
    p.out = a->out;
    p.lse = a->lse;
    p.timeouts = timeouts;
    p.n_seqs = a->n_seqs;
    p.n_tokens = a->n_tokens;
    p.max_q = a->max_q;
    p.n_q_heads = Hq;
    p.table_stride = a->table_stride;
    p.max_blocks = a->max_blocks;
    p.causal = a->causal ? 1 : 0;
    p.gmax = pl.gmax;
    p.uniform = pl.uniform;
    p.qk_scale_log2 = a->sm_scale * 1.4426950408889634f;
    p.lose = lose;
    std::memcpy(p.grp_begin, pl.grp_begin, sizeof(p.grp_begin));
    std::memcpy(p.grp_q, pl.grp_q, sizeof(p.grp_q));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool pdl = pdl_on();
    const kvq_pages *g = a->pages;
    const bool q4 = g->v_type == KVQ_V_Q4_0;
    PagedCuts cuts = {};
    cudaError_t e = cudaSuccess;
    for (int k = 0; k < kAttnParts && e == cudaSuccess; ++k) {
        const Part &pt = pl.part[k];
        if (pt.n_ctas == 0) continue;
        char *w = static_cast<char *>(workspace);
        p.cuts = reinterpret_cast<PagedCut *>(w + pt.cut_off);
        p.ws_lse = reinterpret_cast<float *>(w + pt.lse_off);
        p.ws_o = reinterpret_cast<float *>(w + pt.o_off);
        p.sums = reinterpret_cast<float *>(w + pt.sum_off);
        p.min_rows = pt.least;
        p.max_rows = pt.most;
        // a cut tile is merged by at least two CTAs' blocks of eight warps
        cuts.part[k] = PagedPieces{p.cuts, p.ws_lse, p.ws_o, pt.rows, pt.n_ctas > 1 ? pt.n_ctas : 0, (pt.rows + 15) / 16};
        if (lose >= 0 && k != 1)
            e = k == 0 ? launch_paged_lose(p, pt.n_ctas, s, pdl && pt.n_ctas <= n_sms) : launch_chunk_lose(p, pt.n_ctas, s, pdl);
        else if (k < 2)
            e = q4 ? launch_paged_q4(p, k + 1, g->k_type, a->out_type, pt.n_ctas, s, pdl && pt.n_ctas <= n_sms)
                   : launch_paged_q8(p, k + 1, g->k_type, a->out_type, pt.n_ctas, s, pdl && pt.n_ctas <= n_sms);
        else
            e = q4 ? launch_chunk_q4(p, a->out_type, pt.n_ctas, s, pdl) : launch_chunk_q8(p, a->out_type, pt.n_ctas, s, pdl);
    }
    if (e == cudaSuccess) e = launch_paged_combine(p, cuts, a->out_type, s, pdl);
    return done(e);
}

}  // namespace

extern "C" {

kvq_status kvq_page_bytes(const kvq_pages *p, size_t *bytes)
{
    if (!bytes) return KVQ_ERR_INVALID_ARG;
    const kvq_status st = check_shape(p);
    if (st != KVQ_OK) return st;
    *bytes = (size_t)p->n_kv_heads * (p->page_tokens / kWTile) * page_tile_bytes(p->v_type, p->k_type);
    return KVQ_OK;
}

kvq_status kvq_page_tables(int32_t n_seqs, int32_t page_tokens, int32_t n_pages, const int32_t *lens,
                           const int32_t *n_new, int32_t *free_pages, const int32_t *n_free, int32_t *block_table,
                           int32_t table_stride, int32_t max_blocks, int32_t *lens_out, int32_t *n_free_out,
                           int32_t *q_start, int32_t *slots, int32_t n_tokens, int32_t *status, void *stream)
{
    // (row sums are held to INT_MAX, so that has to stay past n_tokens)
    if (n_seqs < 0 || n_seqs > KVQ_MAX_PAGED_SEQS || page_shift(page_tokens) < 0 || n_pages < 0 || n_tokens < 0 || n_tokens == INT_MAX)
        return KVQ_ERR_INVALID_ARG;
    if ((long long)n_pages * page_tokens > INT_MAX || !table_ok(table_stride, max_blocks, page_tokens)) return KVQ_ERR_INVALID_ARG;
    if (!int_ptr(n_free) || !int_ptr(n_free_out) || !int_ptr(q_start)) return KVQ_ERR_INVALID_ARG;
    if (n_pages > 0 && !int_ptr(free_pages)) return KVQ_ERR_INVALID_ARG;
    if (n_tokens > 0 && !int_ptr(slots)) return KVQ_ERR_INVALID_ARG;
    if (n_seqs > 0 && (!int_ptr(lens) || !int_ptr(n_new) || !int_ptr(lens_out) || !int_ptr(status) ||
                       (max_blocks > 0 && !int_ptr(block_table))))
        return KVQ_ERR_INVALID_ARG;
    PagedDevice *dev = nullptr;
    int n_sms = 0;
    unsigned int *timeouts = nullptr;
    const kvq_status st = paged_setup(&dev, &n_sms, &timeouts);
    if (st != KVQ_OK) return st;
    const TableParams p{lens, n_new, n_free, free_pages, block_table, lens_out, n_free_out, q_start, slots, status,
                        n_seqs, page_shift(page_tokens), n_pages, table_stride, max_blocks, n_tokens, true};
    return done(launch_page_tables(p, static_cast<cudaStream_t>(stream), pdl_on()));
}

kvq_status kvq_paged_append(const kvq_pages *p, const void *k16, const void *v16, int64_t kv_stride, const int32_t *slots,
                            int32_t n_tokens, void *stream)
{
    kvq_status st = check_pool(p);
    if (st != KVQ_OK) return st;
    if (n_tokens < 0 || (long long)n_tokens * p->n_kv_heads > INT_MAX / 2) return KVQ_ERR_INVALID_ARG;
    if (n_tokens == 0 || p->n_pages == 0) return KVQ_OK;
    if (!k16 || !v16 || !aligned(k16, 16) || !aligned(v16, 16) || !int_ptr(slots)) return KVQ_ERR_INVALID_ARG;
    if (kv_stride < (int64_t)p->n_kv_heads * kD || kv_stride % 8) return KVQ_ERR_INVALID_ARG;
    PagedDevice *dev = nullptr;
    int n_sms = 0;
    unsigned int *timeouts = nullptr;
    st = paged_setup(&dev, &n_sms, &timeouts);
    if (st != KVQ_OK) return st;
    PagedRowsParams r = {};
    r.pool = pool_of(p);
    r.k16 = static_cast<const uint16_t *>(k16);
    r.v16 = static_cast<const uint16_t *>(v16);
    r.stride = kv_stride;
    r.slots = slots;
    r.n_tokens = n_tokens;
    return done(launch_paged_append(r, p->v_type, p->k_type, static_cast<cudaStream_t>(stream), pdl_on()));
}

kvq_status kvq_paged_gather(const kvq_pages *p, const int32_t *slots, int32_t n_tokens, int32_t out_type, void *k_out,
                            void *v_out, void *stream)
{
    kvq_status st = check_pool(p);
    if (st != KVQ_OK) return st;
    if (n_tokens < 0 || (long long)n_tokens * p->n_kv_heads > INT_MAX / 2) return KVQ_ERR_INVALID_ARG;
    if (out_type != KVQ_OUT_F32 && out_type != KVQ_OUT_F16) return KVQ_ERR_INVALID_ARG;
    if (n_tokens == 0 || p->n_pages == 0) return KVQ_OK;
    if (!k_out || !v_out || !aligned(k_out, 16) || !aligned(v_out, 16) || !int_ptr(slots)) return KVQ_ERR_INVALID_ARG;
    PagedDevice *dev = nullptr;
    int n_sms = 0;
    unsigned int *timeouts = nullptr;
    st = paged_setup(&dev, &n_sms, &timeouts);
    if (st != KVQ_OK) return st;
    PagedRowsParams r = {};
    r.pool = pool_of(p);
    r.slots = slots;
    r.n_tokens = n_tokens;
    r.k_out = k_out;
    r.v_out = v_out;
    return done(launch_paged_gather(r, p->v_type, p->k_type, out_type, static_cast<cudaStream_t>(stream), pdl_on()));
}

kvq_status kvq_paged_attn_workspace_size(const kvq_paged_desc *a, size_t *bytes)
{
    AttnPlan pl;
    if (!bytes) return KVQ_ERR_INVALID_ARG;
    kvq_status st = check_attn(a, pl);
    if (st != KVQ_OK) return st;
    *bytes = 0;
    if (idle(a)) return KVQ_OK;
    PagedDevice *dev = nullptr;
    int n_sms = 0;
    unsigned int *timeouts = nullptr;
    st = paged_setup(&dev, &n_sms, &timeouts);
    if (st != KVQ_OK) return st;
    plan_attn(a, dev, n_sms, pl);
    *bytes = pl.bytes;
    return KVQ_OK;
}

kvq_status kvq_paged_attn(const kvq_paged_desc *a, void *workspace, size_t workspace_bytes, void *stream)
{
    return run_attn(a, workspace, workspace_bytes, stream, -1);
}

kvq_status kvq_debug_paged_lose_copy(const kvq_paged_desc *a, int32_t copy, void *workspace, size_t workspace_bytes, void *stream)
{
    if (copy < 0) return KVQ_ERR_INVALID_ARG;
    return run_attn(a, workspace, workspace_bytes, stream, copy);
}

}  // extern "C"
