/*
 * moe_serving.h -- C ABI of the operators of a served batch's decode step on MI355X (gfx950), beside the expert
 * layer and the lm_head of moe_latent.h and the drafted step of moe_drafted.h, in the same library:
 *
 *   moe_norm_rope_append   moe_rope_append with queries and keys normed for each head before they turn
 *   moe_mx_append          the same into a cache held in 8 or 4 bits, norms or not
 *   moe_mx_read            what such a cache holds for the step's rows, in 16 bits
 *   moe_mx_attend          moe_tree_attend over such a cache
 *   moe_mx_keep            moe_path_keep of such a cache
 *   moe_shared_attend      moe_tree_attend of a batch whose sequences begin with the same tokens, in groups
 *   moe_sample             a token for each row of logits, with temperature, top-k, top-p and min-p
 *
 * Conventions (pointers, streams, status codes, what is checked on the device) as in moe_drafted.h.
 */
#ifndef MOE_SERVING_H
#define MOE_SERVING_H

#include "moe_drafted.h"

#ifdef __cplusplus
extern "C" {
#endif

/* a further bit of the device flags word (moe_drafted_status names it too) */
enum moe_serving_flag {
    MOE_FLAG_GROUPS = 64    /* group_start not ascending from 0 to the number of sequences */
};

/* RMS norms of the heads before they turn: x <- x / sqrt(mean(x^2) + eps) * (offset + w), in fp32.
 *   q_weight, k_weight  [heads][dim] at a row stride (elements), or [dim] for all heads (stride 0); dtype bf16, f16 or
 *                       f32 (both the same), any alignment of the type
 *   eps                 0 or more, finite; a head that is all zero stays zero
 *   offset              0, or 1 where the weights are stored as differences from 1 */
typedef struct {
    const void *q_weight, *k_weight;
    int64_t q_stride, k_stride;
    int32_t dtype;
    float eps, offset;
} moe_head_norm;

/* moe_rope_append with the norm applied to every head of q and k first (norm NULL: none). Norm and rotation are in fp32,
 * rounded once to the cache's type. Arguments and refusals as there. */
int moe_norm_rope_append(const moe_paged_cache *c, const moe_head_norm *norm, const moe_rope *r, int32_t rows, const void *q,
                         int64_t q_stride, int32_t q_heads, const void *k, int64_t k_stride, const void *v,
                         int64_t v_stride, const int32_t *row_start, const int32_t *positions, void *q_out,
                         int64_t q_out_stride, void *hip_stream);

/* formats of a cache of codes */
enum moe_mx_format {
    MOE_MX8 = 1,    /* e4m3, largest 448: 8.25 bits a value */
    MOE_MX4 = 2     /* e2m1, largest 6: 4.25 bits a value; the even dim in the low four bits */
};

/* A paged key/value cache in blocks of 32 values along a head: codes, and a byte e for each block, whose values are code *
 * 2^(e - 127) (e = 255: the block is NaN). Written with the smallest power of two, 2^-126 at least, under which the block's
 * largest magnitude does not pass the largest code, each value rounded once from fp32, to nearest even; a block that holds
 * an infinity or a NaN becomes NaN. The powers stop where the largest code is finite in the rows' type (2^119 and 2^125 in
 * bf16, 2^7 and 2^13 in f16), and larger values take the largest code, so that what is read back is finite.
 *   k, v              [pages][page][kv_heads][bytes of a head: dim, or dim / 2] bytes (dtype U8), last dim contiguous, other strides
 *                     multiples of 16, 16-byte aligned; page as in moe_paged_cache; dim 32, 64, 96, 128, 192 or 256
 *   k_scale, v_scale  [pages][page][kv_heads][dim / 32] bytes, last dim contiguous
 *   table, len, flags as in moe_paged_cache
 *   format            moe_mx_format
 *   dtype             bf16 or f16: of the rows given to it, of queries and results, and what codes are read as
 * Heads that lie apart ([pages][kv_heads][page][bytes] storage) are read fastest. */
typedef struct {
    moe_tensor k, v, k_scale, v_scale, table, len;
    uint32_t *flags;
    int32_t format, dtype;
} moe_mx_cache;

int moe_mx_cache_check(const moe_mx_cache *c);

/* As moe_norm_rope_append, into a cache of codes (norm NULL: none). */
int moe_mx_append(const moe_mx_cache *c, const moe_head_norm *norm, const moe_rope *r, int32_t rows, const void *q,
                  int64_t q_stride, int32_t q_heads, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                  const int32_t *row_start, const int32_t *positions, void *q_out, int64_t q_out_stride, void *hip_stream);

/* Keys and values that the cache holds: row i of sequence b is token start[b] + i (start NULL: len[b] + i, where
 * moe_mx_append put the step's rows). Rows of a token without a page, or past the table, are not written, and reported.
 *   k_out, v_out  [rows][kv_heads * dim] in the cache's dtype, 16-byte aligned, strides multiples of 8 */
int moe_mx_read(const moe_mx_cache *c, int32_t rows, const int32_t *row_start, const int32_t *start, void *k_out,
                int64_t k_stride, void *v_out, int64_t v_stride, void *hip_stream);

/* Sequences that begin with the same tokens: group g has the sequences group_start[g] .. group_start[g + 1] - 1, whose first
 * len[g] tokens are the same. They are read from the pages of the group's first sequence (the other tables usually name
 * the same pages). len[g] may be anything from 0 up to the shortest cached length of the group's sequences. */
typedef struct {
    const int32_t *group_start;    /* [groups + 1], ascending from 0 to the number of sequences (device) */
    const int32_t *len;            /* [groups] (device) */
    int32_t groups;                /* 1 .. the number of sequences */
} moe_shared_prefix;

/* moe_tree_attend, with the groups' common tokens read once for all rows of a group. Same results, but for the order of
 * sums. It needs its own workspace size. */
int moe_shared_attend(const moe_paged_cache *c, const moe_shared_prefix *shared, int32_t rows, const void *q,
                      int64_t q_stride, int32_t q_heads, const int32_t *row_start, const uint64_t *mask, float scale,
                      void *out, int64_t out_stride, void *workspace, size_t workspace_bytes, void *hip_stream);
int64_t moe_shared_attend_workspace(const moe_paged_cache *c, int32_t groups, int32_t rows, int32_t q_heads);

/* moe_tree_attend over a cache of codes; shared NULL: none. Codes are read as the cache's dtype before the products. */
int moe_mx_attend(const moe_mx_cache *c, const moe_shared_prefix *shared, int32_t rows, const void *q, int64_t q_stride,
                  int32_t q_heads, const int32_t *row_start, const uint64_t *mask, float scale, void *out,
                  int64_t out_stride, void *workspace, size_t workspace_bytes, void *hip_stream);
int64_t moe_mx_attend_workspace(const moe_mx_cache *c, int32_t groups, int32_t rows, int32_t q_heads);

/* moe_path_keep of a cache of codes. */
int moe_mx_keep(const moe_mx_cache *c, const int32_t *row_start, int32_t rows, const int32_t *n_keep, const int32_t *path,
                int32_t *new_len, void *hip_stream);

/* A token for each row. With w_i = exp((z_i - max z) / T), the tokens in order of falling logits (equal ones: the lower index
 * first) are cut to
 *   top-k: the first top_k (0 or less: no cut);
 *   top-p: the shortest beginning whose weight reaches top_p times that of the first top_k (1 or more: no cut; one token is left always);
 *   min-p: those with w_i >= min_p (0 or less: no cut; above 1 it counts as 1),
 * whichever leaves the fewest. The token is the first in that order whose running weight passes u times that of all that are left.
 * T <= 0: the largest logit's lowest index, and logprob 0. Weights are held in 64 bits, the largest
 * logit's as exactly 1, so that a border exactly between logits equal to it lies there. Where weights are added in an order that
 * varies, they are whole numbers of a unit, and the same inputs always give the same token: the unit is 2^-50 of the largest weight of
 * 4096 neighbouring logits; where a border is looked for among n logits within a quarter octave of weight, 2^-39 of theirs
 * or less (n up to 2^20; 2^-49 for 2000). NaN logits count as -infinity, which is never drawn; a row without a value above that
 * gives token 0 and sets MOE_FLAG_LOGITS. NaN in top_p, min_p: no cut; in T: as 0; u is taken into [0, 1).
 *   logits       [rows][vocab] f32, bf16 or f16, rows at any stride >= vocab; vocab 1 .. 2^20
 *   u            [rows] f32
 *   temperature, top_p, min_p  [rows] f32, top_k [rows] i32; each may be NULL: 1, and no cut
 *   tokens       [rows] i32
 *   logprobs     [rows] f32: log of the token's share of all w_i, before the cuts
 * workspace as in moe_tree_attend. */
int moe_sample(const moe_tensor *logits, const float *u, const float *temperature, const int32_t *top_k, const float *top_p,
               const float *min_p, int32_t *tokens, float *logprobs, uint32_t *flags, void *workspace,
               size_t workspace_bytes, void *hip_stream);
int64_t moe_sample_workspace(int32_t rows, int32_t vocab);

#ifdef __cplusplus
}
#endif

#endif /* MOE_SERVING_H */
