/*
 * kvq_tokens.h -- C ABI of libkvq.so, third part: what surrounds append and
 * attention of the paged cache (kvq_paged.h).  New tokens on their way in: heads
 * normalized, positions rotated, keys and values quantized into pages, in one
 * pass over a projection's output.  Sequences forked, cut back and ended by their
 * tables alone, pages copied in the pools of all layers, and held tokens moved
 * and turned to other positions without their fp16 originals.
 *
 * A step of beam search or of a server that shares prefixes is
 *     kvq_page_fork -> kvq_page_copy -> kvq_page_tables -> kvq_page_positions
 * once, and kvq_qkv -> kvq_paged_attn layer by layer.  A context that lets go of
 * its middle is kvq_paged_move in every layer, then kvq_page_fork with the
 * shorter lengths.
 *
 * Memory, streams, errors, programmatic dependent launch and values in device
 * memory that are out of range are as kvq_paged.h says: the library allocates
 * nothing, calls only enqueue work on `stream`, and each can be captured into a
 * CUDA graph once the first call on the device has run outside capture.  No
 * kernel waits for another, and none adds floating-point numbers in an order that
 * changes: the same inputs give the same bits.  Outputs must not overlap inputs or
 * each other except where a call allows it.
 */
#ifndef KVQ_TOKENS_H
#define KVQ_TOKENS_H

#include "kvq_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KVQ_MAX_COPY_POOLS 128     /* pools of one kvq_page_copy */

/* ------------------------------------------------------------- positions --
 * Rotary positions: pair i of the first n_rot values of a head, (a, b), becomes
 * (a cos x - b sin x, a sin x + b cos x), both times `amplitude`, where x is
 * position times the pair's rate; the values behind n_rot stay.  Two layouts:
 *   KVQ_ROPE_HALF   pair i is values i and i + n_rot/2
 *   KVQ_ROPE_PAIRS  pair i is values 2i and 2i + 1
 * The angle of a far position does not survive in 32 bits (131071 * 0.9 rad is
 * known to 0.004 there).  A rate is therefore kept as the part of a full turn
 * that one position makes, in units of 2^-64: position times rate in 64-bit
 * integers drops the full turns and nothing else, and its top 32 bits give the
 * angle to 2^-32 of a turn for every int32 position, also a negative one: the
 * angle of the rate as it is kept.  A rate of kvq_rope_turns comes from arithmetic
 * in double and is off by up to 2^-54 of a turn per position (scaled ones 2^-52, and
 * 1/factor times that where factor is below 1), which is 2^-32 of a turn at
 * position 2^22 and 2^-23 at the ends of int32.
 */
typedef enum kvq_rope_layout {
    KVQ_ROPE_HALF = 0,
    KVQ_ROPE_PAIRS = 1
} kvq_rope_layout;

/* Host descriptor.  turns: device uint64 [n_rot/2], 8-byte aligned (not read
 * where n_rot is 0).  n_rot: 0..KVQ_HEAD_DIM, a multiple of 8.  amplitude: finite. */
typedef struct kvq_rope {
    const uint64_t *turns;
    int32_t n_rot;
    int32_t layout;            /* kvq_rope_layout */
    float amplitude;
} kvq_rope;

/*
 * kvq_rope_turns -- the rates of a rotation, on the host: r_i = base^(-2i/n_rot)
 * radians per position, or, for contexts `factor` times as long as the
 * `original` one that a model was trained on,
 *   KVQ_ROPE_PLAIN     as they are (factor, original, fast, slow are not read)
 *   KVQ_ROPE_LINEAR    r_i / factor
 *   KVQ_ROPE_BASE      with base * factor^(n_rot / (n_rot - 2)) for base: the
 *                      first pair keeps its rate, the last is slowed by factor
 *   KVQ_ROPE_BY_INDEX  pairs that make `fast` turns or more within `original`
 *                      keep their rate, those that make `slow` or fewer are
 *                      slowed by factor, and between them the share of the slowed
 *                      rate grows linearly with i (from the largest i below the
 *                      first bound to the smallest above the second, held to
 *                      0..n_rot - 1); amplitude 0.1 ln(factor) + 1
 *   KVQ_ROPE_BY_TURNS  the same with the share linear in the turns that a pair
 *                      makes within `original`; amplitude 1
 * n_rot: 0..KVQ_HEAD_DIM, a multiple of 8.  base above 1; factor above 0; original
 * above 0 and fast > slow > 0 (BY_INDEX, BY_TURNS); all finite.  turns: host out
 * [n_rot/2].  amplitude: host out.
 */
typedef enum kvq_rope_scaling {
    KVQ_ROPE_PLAIN = 0,
    KVQ_ROPE_LINEAR = 1,
    KVQ_ROPE_BASE = 2,
    KVQ_ROPE_BY_INDEX = 3,
    KVQ_ROPE_BY_TURNS = 4
} kvq_rope_scaling;

kvq_status kvq_rope_turns(int32_t n_rot, double base, int32_t scaling, double factor, double original, double fast,
                          double slow, uint64_t *turns, float *amplitude);

/*
 * kvq_page_positions -- the position of every row of a step's packed batch, from
 * the tables of kvq_page_tables (its lens_out and q_start): row t of sequence b
 * is at seq_lens[b] - q_start[b+1] + t, the place that kvq_paged_attn gives it.
 * Once per step; every layer's kvq_qkv reads it.
 *  n_seqs     0..KVQ_MAX_PAGED_SEQS.
 *  q_start    device int32 [n_seqs + 1], non-decreasing; values are held to
 *             [0, n_tokens].
 *  seq_lens   device int32 [n_seqs], the new tokens counted.
 *  n_tokens   rows of the batch, below 2^31 - 1.
 *  positions  device int32 [n_tokens]; rows no sequence owns get -1.
 */
kvq_status kvq_page_positions(int32_t n_seqs, const int32_t *q_start, const int32_t *seq_lens, int32_t n_tokens,
                              int32_t *positions, void *stream);

/*
 * One kvq_qkv call: every head of q16 and k16 (a row x of 128 values) becomes
 *   n = x / sqrt(mean(x^2) + eps) * norm    (norm NULL: n = x)
 *   y = n rotated to the token's position   (rope NULL: y = n)
 * in fp32 and is rounded to fp16 once.  Queries go to q_out; keys either go to
 * k_out, or are quantized with v16 into the tokens' slots as kvq_paged_append
 * would: the same bytes as k_out handed to kvq_paged_append.
 *  q16, k16, v16  device fp16, token i at + i * stride, [heads][head_dim] each;
 *                 16-byte aligned.  q_stride, k_stride, v_stride: elements between
 *                 tokens, multiples of 8, at least heads * head_dim (columns of a
 *                 fused projection's output are read where they are).
 *  n_q_heads, n_kv_heads  0..KVQ_MAX_HEADS; 0: no queries, or no keys and values
 *                 (their pointers are not read, pages and k_out are NULL).
 *  q_norm, k_norm device fp32 [head_dim], 16-byte aligned, or NULL.
 *  eps            finite, not negative.
 *  rope           host, or NULL.
 *  positions      device int32 [n_tokens] (any int32); not read without a rotation.
 *  q_out          device fp16, [n_q_heads][head_dim] per token, 16-byte aligned;
 *                 q_out_stride as q_stride.  May be q16 itself, with its stride.
 *  pages, slots   the pool (n_kv_heads heads) and device int32 [n_tokens], or
 *                 pages NULL.  slots may be given without pages too.
 *  k_out          device fp16 like q_out, or NULL: exactly one of pages and k_out is
 *                 given where n_kv_heads > 0.  May be k16 itself, with its stride.
 *                 v16 is read only with pages.
 * A token whose slot is negative is left out altogether (its rows of q_out and
 * k_out stay as they were): the padding of a batch, sequences that were not
 * served.  One whose slot lies past the pool gets its query, and its key and value
 * go nowhere (a token whose page already holds them).  Two tokens of a call must
 * not share a slot.
 */
typedef struct kvq_qkv_desc {
    const void *q16, *k16, *v16;
    int64_t q_stride, k_stride, v_stride;
    int32_t n_tokens, n_q_heads, n_kv_heads;
    float eps;
    const float *q_norm, *k_norm;
    const kvq_rope *rope;
    const int32_t *positions;
    void *q_out;
    int64_t q_out_stride;
    const kvq_pages *pages;
    const int32_t *slots;
    void *k_out;
    int64_t k_out_stride;
} kvq_qkv_desc;

kvq_status kvq_qkv(const kvq_qkv_desc *a, void *stream);

/* ------------------------------------------------------------ held pages --
 * kvq_page_fork -- new tables from old ones: place b of the batch goes on with the
 * first keep[b] positions of what place parent[b] held.  One call reorders beams,
 * starts requests on the prefixes of others, takes rejected tokens back, ends
 * sequences, and gives back the pages that nothing lists any more; pages listed
 * more than once are shared.  (kvq_page_tables can end sequences too, but must not
 * where a page of theirs is shared.)  A cached prefix is a place like any other.
 *
 *  n_seqs       places, 0..KVQ_MAX_PAGED_SEQS.
 *  page_tokens, n_pages  as the pool the tables are for; n_pages * page_tokens
 *               below 2^31.
 *  lens         device int32 [n_seqs], held to [0, max_blocks * page_tokens].
 *  parent       device int32 [n_seqs]; a value outside [0, n_seqs) empties the
 *               place.  NULL: every place is its own parent.
 *  keep         device int32 [n_seqs], held to [0, lens[parent]].  NULL: all.
 *  block_table  device int32 [n_seqs][table_stride], max_blocks <= table_stride
 *               entries of a row used.
 *  table_out    device int32 [n_seqs][out_stride], out_stride >= max_blocks: the
 *               first ceil(lens_out / page_tokens) entries of each row are written.
 *               May be block_table (with its stride) where parent is NULL.
 *  lens_out     device int32 [n_seqs].  May be lens.
 *  free_pages   device int32 [n_pages], n_free device int32 [1]: the stack of
 *               kvq_page_tables.  Pages that an old row lists (within its length)
 *               and no new one does are pushed, in order of their numbers, each
 *               once; pages for copies are then popped.  Entries at and past *n_free
 *               are written, up to the most that the stack held meanwhile.
 *  n_free_out   device int32 [1].  May be n_free.
 *  copy_from, copy_to, copy_held  device int32 [n_seqs]: where a new row ends
 *               inside a page that it would share, it gets a page of its own
 *               instead, since its next token goes there.  copy_from[b] is the page
 *               to copy, copy_to[b] the new page (in table_out already), copy_held[b]
 *               the positions that matter; -1, -1, 0: nothing to copy.  Hand
 *               them to kvq_page_copy as they are, before anything else writes to
 *               the pools.  Where no new row lists the page otherwise, the first
 *               of those that end in it keeps it.
 *  status       device int32 [n_seqs]: 0, or 1 where the pool had no page left for
 *               the copy (pages are given in order of place): the place then holds
 *               only its whole pages, lens_out says how many positions that is.
 *  workspace    device, 256-byte aligned, kvq_page_fork_workspace_size() bytes; as
 *               kvq_paged_attn's.
 * Entries outside [0, n_pages) are handed on as they are, and are never given back
 * or copied.  Pushes past n_pages entries are dropped.
 */
kvq_status kvq_page_fork(int32_t n_seqs, int32_t page_tokens, int32_t n_pages, const int32_t *lens,
                         const int32_t *parent, const int32_t *keep, const int32_t *block_table,
                         int32_t table_stride, int32_t max_blocks, int32_t *table_out, int32_t out_stride,
                         int32_t *lens_out, int32_t *free_pages, const int32_t *n_free, int32_t *n_free_out,
                         int32_t *copy_from, int32_t *copy_to, int32_t *copy_held, int32_t *status, void *workspace,
                         size_t workspace_bytes, void *stream);

/* Bytes of workspace kvq_page_fork needs.  bytes: host out. */
kvq_status kvq_page_fork_workspace_size(int32_t n_seqs, int32_t n_pages, size_t *bytes);

/*
 * kvq_page_copy -- page from[i] to page to[i], byte for byte, in each of n_pools
 * pools (the layers of a model) in one launch.
 *  pools      host array [n_pools], 0..KVQ_MAX_COPY_POOLS, with the same n_pages and
 *             page_tokens; heads and formats may differ.
 *  from, to   device int32 [n_copies]; pairs with a number outside [0, n_pages), or
 *             the same twice, are skipped.  A page may be copied to several; no
 *             page is written that another pair reads or writes.
 *  held       device int32 [n_copies]: only the tiles of the first held[i] positions
 *             are copied (whole tiles of 16).  NULL: whole pages.
 *  n_copies   0 or more; n_copies * n_pools * the most n_kv_heads at most 2^28.
 */
kvq_status kvq_page_copy(const kvq_pages *pools, int32_t n_pools, const int32_t *from, const int32_t *to,
                         const int32_t *held, int32_t n_copies, void *stream);

/*
 * kvq_paged_move -- held tokens to other slots, their keys turned by so many
 * positions: token i of slot from[i] goes to slot to[i], for every head.  Accepted
 * tokens of a verified tree close ranks, a context drops a stretch and the rest
 * moves up, or (from = to) keys turn where they lie when whole pages were dropped.
 *  from, to   device int32 [n_tokens]; tokens with a slot that is negative or past
 *             the pool are skipped.  Two tokens must not share a `to`.  A page that
 *             several places list changes for all of them.
 *  rope, turn the rotation the keys were written with (host; its amplitude is not
 *             applied: the held keys carry it) and device int32 [n_tokens], the positions
 *             to turn each token by (negative: back); both or neither NULL.
 *  staged     nonzero: every slot is read before any is written, so a slot may be one
 *             token's `to` and another's `from`; the tokens pass through the
 *             workspace.  Zero: no slot is both, except a token's own (from = to).
 *  workspace  device, 256-byte aligned, kvq_paged_move_workspace_size() bytes; as
 *             kvq_paged_attn's.  Not read where staged is 0.  (Up to 256 tokens stay
 *             on the chip; it is asked for all the same.)
 * Without a turn (turn NULL or 0) a token's bytes go over as they are, and V's always
 * do.  A turned int8 key is dequantized (code * scale), turned in fp32, rounded to
 * fp16 and quantized again by kvq_append's rule, 32-blocks past n_rot excepted; a turned
 * F16 key is rounded to fp16.  Each turn thus costs a key one more quantization.
 */
kvq_status kvq_paged_move(const kvq_pages *p, const int32_t *from, const int32_t *to, int32_t n_tokens,
                          const kvq_rope *rope, const int32_t *turn, int32_t staged, void *workspace,
                          size_t workspace_bytes, void *stream);

/* Bytes of workspace a staged kvq_paged_move of n_tokens needs (data of p is not
 * read).  bytes: host out. */
kvq_status kvq_paged_move_workspace_size(const kvq_pages *p, int32_t n_tokens, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* KVQ_TOKENS_H */
