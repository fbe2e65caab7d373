/*
 * moe_drafted.h -- C ABI of the operators of a drafted (speculative) decode step on MI355X
 * (gfx950), beside the expert layer and the lm_head of moe_latent.h, in the same library.
 *
 * A step passes, for every sequence, its last token and the tokens drafted after it through
 * the model at once. The rows of a step lie one sequence after another: sequence b has the rows
 * row_start[b] .. row_start[b + 1] - 1, its row 0 being the last token that is certain and the
 * others drafts, each after its parent (a chain, or a tree). Over one paged key/value cache:
 *
 *   moe_rope_append   rotary positions of the new queries and keys; keys and values into the cache
 *   moe_tree_attend   attention of the rows over the cached tokens and their own ancestors
 *   moe_draft_verify  which drafts the target's probabilities accept, and the token after them
 *   moe_path_keep     the accepted path's keys and values moved behind the cached tokens
 *
 * Every pointer is a device pointer on the current GPU unless stated otherwise. Every call checks
 * its arguments on the host, enqueues its launches on hip_stream (NULL: the null stream) and
 * returns; no call allocates, synchronises or sets memory, so each can be captured in a HIP
 * graph. Status codes and moe_latent_last_error() as in moe_latent.h. What only the device
 * knows (row_start, len, page numbers, paths, tokens) is checked there: a bad value sets a bit of
 * the caller's flags word and is never read through or written through.
 */
#ifndef MOE_DRAFTED_H
#define MOE_DRAFTED_H

#include "moe_latent.h"

#ifdef __cplusplus
extern "C" {
#endif

/* bits of the device flags word, set when a kernel meets */
enum moe_drafted_flag {
    MOE_FLAG_PAGE = 1,      /* a page number outside the cache, or a token past the page table */
    MOE_FLAG_LEN = 2,       /* a negative length, or one past the page table */
    MOE_FLAG_ROWS = 4,      /* row_start not ascending from 0 to the number of rows */
    MOE_FLAG_PATH = 8,      /* a kept path that is not ascending rows of its sequence */
    MOE_FLAG_TOKEN = 16,    /* a drafted token outside the vocabulary */
    MOE_FLAG_LOGITS = 32    /* a row of logits on the walk without a value above -infinity */
};

/* A paged key/value cache (borrowed). Token t of sequence b lies in slot t % page of page
 * table[b][t / page].
 *   k, v   [pages][page][kv_heads][dim]  bf16 or f16 (both the same). Any strides with the last
 *                     dim contiguous and the others multiples of 8 elements (so [pages][kv_heads]
 *                     [page][dim] storage can be described too); 16-byte aligned. page a
 *                     multiple of 16; dim 32, 64, 80, 96, 112, 128, 192 or 256; at most
 *                     2^31 - 1 pages; a page spans less than 2^30 elements.
 *   table  [seqs][width]  i32, rows any stride, columns contiguous
 *   len    [seqs]         i32: tokens cached so far, without those of this step
 *   flags  one u32 (zeroed by the caller at first) that collects moe_drafted_flag bits */
typedef struct {
    moe_tensor k, v, table, len;
    uint32_t *flags;
} moe_paged_cache;

/* Check a cache's descriptors (no device access): MOE_OK or the refusal of the calls below. */
int moe_paged_cache_check(const moe_paged_cache *c);

/* pairs of a rotated head */
enum moe_rope_layout {
    MOE_ROPE_HALF = 1,          /* dims (j, j + rotary / 2) */
    MOE_ROPE_INTERLEAVED = 2    /* dims (2 j, 2 j + 1) */
};

/* Rotary positions: the pair j of a head at position t turns by the angle t * freqs[j]; cosine
 * and sine are then multiplied by magnitude. The first 2 * pairs dims turn, the others stay.
 *   freqs  [pairs] f64 radians per position (device)  */
typedef struct {
    const double *freqs;
    int32_t pairs;       /* 1 .. dim / 2 */
    int32_t layout;      /* moe_rope_layout */
    float magnitude;     /* 1, or the scaling method's factor on cosine and sine */
} moe_rope;

/* Rotate the step's queries into q_out and its keys into the cache, and copy its values there:
 * row i of sequence b becomes cached token len[b] + i (len itself does not change).
 *   q [rows][q_heads * dim], k and v [rows][kv_heads * dim] in the cache's type, rows at the
 *     given strides (elements); heads side by side. Any alignment of 2 bytes (16 is fastest);
 *     interleaved pairs need 4.
 *   positions  [rows] i32, or NULL: row i of sequence b is at len[b] + i
 *   q_out      [rows][q_heads * dim]; may be q itself (same pointer and stride), no other overlap
 * The angle is formed in 64 bits, so far positions lose nothing. Rows that row_start gives to no
 * sequence are not touched. */
int moe_rope_append(const moe_paged_cache *c, const moe_rope *r, int32_t rows, const void *q, int64_t q_stride,
                    int32_t q_heads, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                    const int32_t *row_start, const int32_t *positions, void *q_out, int64_t q_out_stride,
                    void *hip_stream);

/* Attention of the step's rows, whose keys and values are in the cache already: row i of
 * sequence b sees the len[b] cached tokens, and of the step's tokens len[b] + j those with bit j of
 * its mask (j < 64; with mask NULL: j <= i). out = softmax(scale * q k) v over what it sees;
 * a row that sees nothing gives zeros, and what is not seen is not used, whatever it holds.
 * Scores, statistics and sums in fp32; probabilities are rounded to the cache's type for the
 * product with v, the result once.
 *   q, out  [rows][q_heads * dim], q_heads a multiple of kv_heads (head h reads key head h /
 *           (q_heads / kv_heads)); 16-byte aligned, strides multiples of 8; out overlaps nothing
 *   mask    [rows] u64, or NULL
 *   workspace  moe_tree_attend_workspace bytes, 16-byte aligned, used by this call alone until
 *           its launches are done
 * The same inputs give the same bits on every run. */
int moe_tree_attend(const moe_paged_cache *c, int32_t rows, const void *q, int64_t q_stride, int32_t q_heads,
                    const int32_t *row_start, const uint64_t *mask, float scale, void *out, int64_t out_stride,
                    void *workspace, size_t workspace_bytes, void *hip_stream);

/* Bytes of workspace moe_tree_attend needs for so many rows (0 bytes is possible); negative: the
 * status code of a refusal, negated. */
int64_t moe_tree_attend_workspace(const moe_paged_cache *c, int32_t rows, int32_t q_heads);

/* Test the drafted tokens. For each sequence the walk starts at row 0; at row `cur`, with p the
 * target's probabilities softmax(logits[cur] / T) (T <= 0: all on the largest logit, the
 * lowest index among equals) and q = draft_probs[cur]:
 *   with draft_probs: S = 0, rest = 1; every later row c with parent[c] == cur, in order, with x =
 *     tokens[c]: accepted if u_test[c] * q[x] * rest < max(p[x] - S q[x], 0), and the walk goes on
 *     at c; else S += rest and rest = sum max(p - S q, 0). When no child is left, the next token
 *     is drawn from max(p - S q, 0) (from p if that is all zero).
 *   without: the next token is drawn from p, and the walk goes to the first child that holds it.
 * A draw with u = u_pick[cur] takes the first index whose running sum passes u times the whole sum.
 * Without draft_probs tokens follow the target's distribution whatever the drafts; with them, where the drafts
 * after a row were drawn from its q independently of each other (a token may then come twice). Drafts chosen otherwise
 * (the most likely ones, or drawn without replacement) are for the form without. Probabilities and sums are held in
 * 64 bits. NaN logits count as -infinity.
 *   logits       [rows][vocab] f32, bf16 or f16, rows at any stride >= vocab
 *   tokens       [rows] i32: the token each row holds (that of row 0 is not read); one outside
 *                the vocabulary is never accepted and changes nothing else
 *   parent       [rows] i32: a row's parent as its number within the sequence, less than its own;
 *                NULL: a chain
 *   u_test, u_pick  [rows] f32 in [0, 1) (u_test may be NULL without draft_probs)
 *   draft_probs  [rows][vocab] f32, or NULL: what the drafts after each row were drawn from, each for itself
 *   temperature  [seqs] f32, or NULL: 1
 *   n_keep       [seqs] i32: rows of the path, row 0 included
 *   path         [rows] i32: from row_start[b] on its rows, then -1
 *   out_tokens   [rows] i32: from row_start[b] on the n_keep[b] tokens that follow, then -1
 *   logprobs     [rows] f32: log p of each of them, then 0
 *   flags        as in moe_paged_cache
 * vocab 1 .. 2^20. workspace as in moe_tree_attend. */
int moe_draft_verify(const moe_tensor *logits, const int32_t *tokens, const int32_t *row_start, int32_t seqs,
                     const int32_t *parent, const float *u_test, const float *u_pick, const float *draft_probs,
                     int64_t draft_stride, const float *temperature, int32_t *n_keep, int32_t *path,
                     int32_t *out_tokens, float *logprobs, uint32_t *flags, void *workspace, size_t workspace_bytes,
                     void *hip_stream);

/* Bytes of workspace moe_draft_verify needs; negative: a status code, negated. */
int64_t moe_draft_verify_workspace(int32_t rows, int32_t seqs, int32_t vocab);

/* Move the kept rows' keys and values together: cached token len[b] + i becomes what token
 * len[b] + path[row_start[b] + i] was, for i < n_keep[b]; new_len[b] = len[b] + n_keep[b] (new_len
 * may be the cache's len; of layers whose caches share one, that of the last call alone). A path ascends
 * strictly; one that does not, or leaves its sequence's rows, moves nothing, sets MOE_FLAG_PATH and leaves
 * the length as it was; so does, with MOE_FLAG_PAGE, one of whose moved rows comes from or goes to a page
 * outside the cache or past the table. */
int moe_path_keep(const moe_paged_cache *c, const int32_t *row_start, int32_t rows, const int32_t *n_keep,
                  const int32_t *path, int32_t *new_len, void *hip_stream);

/* Synchronise hip_stream, read and clear a flags word: MOE_OK, or MOE_ERR_DEVICE_CHECK with a
 * message that names what was met. */
int moe_drafted_status(uint32_t *flags, void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_DRAFTED_H */
