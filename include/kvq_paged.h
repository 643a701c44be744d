/*
 * kvq_paged.h -- C ABI of libkvq.so, second part: the quantized KV cache kept
 * in pages, for servers whose sequences grow, finish and share one pool.
 *
 * The formats and the arithmetic are those of kvq.h (int8 K with fp16 scales
 * per 32 values or fp16 K; q4_0 or q8_0 V; the query quantized like an int8
 * K), so attention over a paged cache is attention over the same tokens held
 * in segments.  What differs is where lengths live: a segment's length is host
 * bookkeeping, everything here is device memory that kernels read when they
 * run.  A step (tables -> append -> attention, layer by layer) needs no host
 * synchronization and can be captured into a CUDA graph and replayed while the
 * sequences grow, start and finish.
 *
 * The pool.  One device array of n_pages pages.  A page holds page_tokens
 * positions of one sequence for every kv head:
 *     [n_pages][n_kv_heads][page_tokens / 16][tile]
 * A tile is 16 positions of one head in one run of bytes:
 *     K codes | K scales (int8 K only) | V codes | V scales
 *     int8 K  2048 + 128    F16 K  4096    q4_0 V  1024 + 128    q8_0 V  2048 + 128
 * so one bulk copy moves a tile (or a page's neighbouring tiles).  With u the
 * position in the tile and j the byte (F16 K: element) of the logical row, the
 * code bytes sit at the tile offsets that kvq.h gives under "Tiles"; int8 K
 * and q8_0 V codes are stored as code + 128; the fp16 scale of block b of
 * position u sits at byte 2 * (((u/8)*4 + (u%8)/2) * 8 + 2*b + u%2) of its
 * scale area.  kvq_page_bytes() gives the size of a page.
 *
 * Slots.  slot = page * page_tokens + place names one position of the pool
 * (int32: n_pages * page_tokens stays below 2^31).  Negative slots name none.
 *
 * Block tables.  Device int32 [n_seqs][table_stride]: entry i of a sequence is
 * the page of its positions i*page_tokens and on.  An entry outside
 * [0, n_pages) hides the positions it would hold: attention treats them as
 * masked.  Two sequences may list the same page (a shared prefix).
 *
 * Memory, streams, errors and programmatic dependent launch are as kvq.h says:
 * the library allocates nothing, every call only enqueues work on `stream`,
 * arguments are checked before anything is enqueued, and KVQ_PDL=0 launches
 * plainly.  Values in device memory cannot be checked on the host; where they
 * are out of range the kernels clamp or skip them as each call states, and
 * touch nothing outside the arrays.
 */
#ifndef KVQ_PAGED_H
#define KVQ_PAGED_H

#include "kvq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KVQ_MAX_PAGED_SEQS 4096    /* sequences of one call                        */
#define KVQ_PAGE_RELEASE (-1)      /* n_new of a finished sequence (any value < 0) */

/* Type of computed values: out of kvq_paged_attn, K and V of kvq_paged_gather. */
typedef enum kvq_out_type {
    KVQ_OUT_F32 = 0,
    KVQ_OUT_F16 = 1
} kvq_out_type;

/* Host descriptor of a page pool.  data: device, 128-byte aligned, n_pages *
 * kvq_page_bytes() bytes.  page_tokens: 16, 32, 64, 128 or 256. */
typedef struct kvq_pages {
    int32_t n_pages;
    int32_t page_tokens;
    int32_t n_kv_heads;
    int32_t head_dim;          /* must be KVQ_HEAD_DIM */
    int32_t k_type;            /* kvq_ktype */
    int32_t v_type;            /* kvq_vtype */
    void *data;
} kvq_pages;

/* kvq_page_bytes -- bytes of one page (data of p is not read).  bytes: host out. */
kvq_status kvq_page_bytes(const kvq_pages *p, size_t *bytes);

/*
 * kvq_page_tables -- the tables of one step, built on the GPU from the lengths.
 *
 *  n_seqs       places of the batch, 0..KVQ_MAX_PAGED_SEQS.
 *  page_tokens, n_pages  as the pool the tables are for.
 *  lens         device int32 [n_seqs]: positions each sequence holds.
 *  n_new        device int32 [n_seqs]: tokens the step adds; 0 leaves the
 *               sequence alone; negative (KVQ_PAGE_RELEASE) ends it and gives
 *               its pages back.
 *  free_pages   device int32 [n_pages]: a stack of unused pages, its first
 *               *n_free entries valid.  Pages given back are pushed in order of
 *               sequence and place, then the step's new pages are popped, in
 *               the same order.  Only entries at and past *n_free are written.
 *  n_free       device int32 [1].
 *  block_table  device int32 [n_seqs][table_stride], updated in place: the new
 *               pages of a sequence follow the ceil(len / page_tokens) it has;
 *               other entries stay.  max_blocks <= table_stride entries of a
 *               row may be used.
 *  lens_out     device int32 [n_seqs]: lengths after the step (0 for an ended
 *               sequence).  May be lens itself.
 *  n_free_out   device int32 [1]: the stack's size after the step.  May be n_free.
 *  q_start      device int32 [n_seqs + 1]: first row of each sequence's new
 *               tokens in the step's packed batch (rows of sequence 0 first;
 *               sums past 2^31 - 1 stay there).
 *  slots        device int32 [n_tokens]: the slot of every row; rows no
 *               sequence owns get -1.
 *  n_tokens     host: rows of the packed batch, at least the sum of the
 *               positive n_new for every sequence to be served; below 2^31 - 1.
 *  status       device int32 [n_seqs]: 0, or why nothing was added: 1 the pool
 *               has too few free pages, 2 the length would pass max_blocks pages or
 *               the rows would pass n_tokens.  Pages are granted in order of
 *               sequence: after the first that does not fit (1), only
 *               sequences that need no new page are served.  A sequence that
 *               is not served keeps its length, and its rows get slot -1.
 * Lengths below 0 count as 0 and above max_blocks * page_tokens as that;
 * *n_free is held to [0, n_pages].  A new token whose page entry lies outside
 * [0, n_pages) gets slot -1.  Pushes past n_pages entries are dropped.
 * Entries are given back as they stand in the table and handed out again: a
 * sequence to be ended must list only pages that are its own to give, none that
 * another sequence still lists (a shared prefix), none twice, and no entry
 * outside [0, n_pages) (a hidden page).
 * One launch, two for more than 16384 rows.
 */
kvq_status kvq_page_tables(int32_t n_seqs, int32_t page_tokens, int32_t n_pages, const int32_t *lens,
                           const int32_t *n_new, int32_t *free_pages, const int32_t *n_free,
                           int32_t *block_table, int32_t table_stride, int32_t max_blocks, int32_t *lens_out,
                           int32_t *n_free_out, int32_t *q_start, int32_t *slots, int32_t n_tokens,
                           int32_t *status, void *stream);

/*
 * kvq_paged_append -- quantize fp16 K/V tokens into their slots (the rules of
 * kvq_append, bit for bit).
 *
 *  k16, v16   device fp16, token i at k16 + i * kv_stride, [n_kv_heads][head_dim]
 *             each; 16-byte aligned.  kv_stride: elements between tokens, a
 *             multiple of 8, at least n_kv_heads * head_dim (columns of a fused
 *             projection's output are read where they are).
 *  slots      device int32 [n_tokens]; tokens whose slot is negative or past the
 *             pool are skipped.  Two tokens of a call must not share a slot
 *             (the slot's bytes would then be a mix of both).
 */
kvq_status kvq_paged_append(const kvq_pages *p, const void *k16, const void *v16, int64_t kv_stride,
                            const int32_t *slots, int32_t n_tokens, void *stream);

/*
 * kvq_paged_gather -- the values of listed slots, dequantized: k = code * scale
 * (F16 K: the stored value), v = code * scale, each computed in fp32 and, for
 * KVQ_OUT_F16, rounded once.  The counterpart of kvq_paged_append: a prefix
 * handed to a kernel that takes plain K and V, or requantized elsewhere.
 *
 *  k_out, v_out  device [n_tokens][n_kv_heads][head_dim] of out_type, 16-byte
 *             aligned.  Rows whose slot is negative or past the pool are left
 *             as they were.  A slot may be listed more than once.
 */
kvq_status kvq_paged_gather(const kvq_pages *p, const int32_t *slots, int32_t n_tokens, int32_t out_type,
                            void *k_out, void *v_out, void *stream);

/*
 * One kvq_paged_attn call.
 *  pages       the pool.
 *  q16         device fp16, token row t at q16 + t * q_stride,
 *              [n_q_heads][head_dim], 16-byte aligned; q_stride in elements, a
 *              multiple of 8, at least n_q_heads * head_dim.
 *  n_tokens    rows of q16, out and lse.
 *  n_seqs      0..KVQ_MAX_PAGED_SEQS.
 *  q_start     device int32 [n_seqs + 1]: sequence b owns rows q_start[b] ..
 *              q_start[b+1] - 1: its newest positions, in order.  Non-decreasing;
 *              values are held to [0, n_tokens].  Rows no sequence owns (behind
 *              q_start[n_seqs]) are not touched.
 *  max_q       host: upper bound of the rows of one sequence, 1..n_tokens.  Rows of a
 *              sequence past max_q are not computed (left as they were).  At most
 *              2^26 rows per kv head (max_q times its query heads).
 *  seq_lens    device int32 [n_seqs]: positions of each sequence, the new ones
 *              included (held to [0, max_blocks * page_tokens]).
 *  block_table, table_stride, max_blocks  as kvq_page_tables.
 *  causal      nonzero: row i of the n that q_start gives the sequence (rows
 *              past max_q counted) sees positions 0 .. len - n + i; zero: all
 *              len positions.
 *  head_map    host int32 [n_q_heads] or NULL, as kvq_decode_attn.
 *  sm_scale    softmax scale.
 *  out_type    kvq_out_type of out.
 *  out         device [n_tokens][n_q_heads][head_dim], 16-byte aligned.
 *  lse         device fp32 [n_tokens][n_q_heads], natural log, or NULL.
 * A row that sees no position gets out = 0 and lse = -inf.  One that sees some
 * and whose query holds an infinity or NaN, or a score of which is NaN or
 * +inf, gets NaN in both.  Whatever positions
 * that no row of the sequence sees hold (behind len, in hidden pages, never
 * written) has no effect.  A position that some rows see and others do not
 * enters the latter with weight 0, so a V that is not finite there makes their
 * out NaN too, as it does in a product of matrices; a K that is not finite has
 * no effect on rows that do not see it.
 */
typedef struct kvq_paged_desc {
    const kvq_pages *pages;
    const void *q16;
    int64_t q_stride;
    int32_t n_q_heads;
    int32_t n_tokens;
    int32_t n_seqs;
    int32_t max_q;
    const int32_t *q_start;
    const int32_t *seq_lens;
    const int32_t *block_table;
    int32_t table_stride;
    int32_t max_blocks;
    int32_t causal;
    const int32_t *head_map;
    float sm_scale;
    int32_t out_type;
    void *out;
    float *lse;
} kvq_paged_desc;

/*
 * kvq_paged_attn -- attention of every sequence's new tokens (one of a decode
 * step, a few to verify, a chunk of a prompt, none) over its pages, for a
 * ragged batch in one call.  The split of the work over the GPU is derived
 * from the device lengths by the kernels themselves, in a fixed way: the same
 * inputs give the same bits.  Sequences go to a kernel by their rows per kv
 * head (up to 8, up to 32, more), each kind in a launch of its own; where n_seqs *
 * max_q == n_tokens says that all have max_q rows (at most 32 per kv head, or a
 * single sequence), one launch takes them all, whatever q_start holds.  A decode
 * step in buffers for more (64 single tokens, n_tokens 4096, max_q 512) takes 5 to
 * 6 us longer than with max_q 1, for the launches that find nothing to do.
 *  workspace   device, 256-byte aligned, kvq_paged_attn_workspace_size() bytes.
 *              Its contents need no preparation and mean nothing after the
 *              call; calls that may overlap on the GPU need one each.
 * KVQ_OUT_F32 keeps p * d at about 22 bits in P.V (as kvq_decode_attn);
 * KVQ_OUT_F16 rounds it to fp16 once.
 */
kvq_status kvq_paged_attn(const kvq_paged_desc *a, void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace kvq_paged_attn needs for a.  Device pointers are not read:
 * it depends on the device and on the numbers in a (n_tokens among them), not on
 * what device memory holds.  bytes: host out. */
kvq_status kvq_paged_attn_workspace_size(const kvq_paged_desc *a, size_t *bytes);

/*
 * kvq_debug_paged_lose_copy -- TEST HOOK, the counterpart of
 * kvq_debug_lose_stage: kvq_paged_attn (same arguments and rules) on test
 * flavours of its kernels in which the first CTA arms the barrier of one copy
 * without issuing the copy.  The bounded wait for it (a short limit here) runs
 * out; the CTA waits for the copies it did issue, the wait counter of
 * kvq_wait_timeouts grows by one, and the rows of the CTA's pieces come out as
 * NaN: in row tiles those of the piece that lost the copy and of the later ones,
 * in the chunk kernel all of them.  Nothing faults and nothing waits without a
 * limit.  Of the launches of a call those for up to 8 rows per kv head (copy:
 * which stage of 32 positions of the first warp) and for more than 32 (copy / 2:
 * which half tile of 64 positions; even: its K part, odd: its V part) lose one.
 * int8 K, q4_0 V and KVQ_OUT_F32; others return KVQ_ERR_UNSUPPORTED.
 */
kvq_status kvq_debug_paged_lose_copy(const kvq_paged_desc *a, int32_t copy, void *workspace, size_t workspace_bytes,
                                     void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_PAGED_H */
