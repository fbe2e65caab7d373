// attend_launch.hip -- host side of the attention kernels: their choice by type, head width, tile and format, their workspace
// and their launches.
#include "api_checks.h"

namespace moe {
template <bool F16, int D, int NQ, int QW, int FMT, bool SHARED> __global__ void moe_attend_kernel(AttendParams p);
template <bool F16, int D> __global__ void moe_attend_join_kernel(AttendParams p);

typedef void (*AttendKernel)(AttendParams);

template <bool F16, int D, int FMT, bool SHARED> static AttendKernel of_tile(int queries) {
    return queries == 16   ? moe_attend_kernel<F16, D, 1, 1, FMT, SHARED>
           : queries == 32 ? moe_attend_kernel<F16, D, 2, 1, FMT, SHARED>
           : queries == 64 ? moe_attend_kernel<F16, D, 2, 2, FMT, SHARED>
                           : moe_attend_kernel<F16, D, 2, 4, FMT, SHARED>;
}
template <bool F16, int D> static AttendKernel of_format(int format, bool groups, int queries) {
    if constexpr (D % 32 == 0) {
        if (format == MX_E4M3) return of_tile<F16, D, MX_E4M3, true>(queries);
        if (format == MX_E2M1) return of_tile<F16, D, MX_E2M1, true>(queries);
    }
    return groups ? of_tile<F16, D, MX_NONE, true>(queries) : of_tile<F16, D, MX_NONE, false>(queries);
}
template <bool F16> static void of_dim(int dim, int format, bool groups, int queries, AttendKernel *main, AttendKernel *join) {
    switch (dim) {
#define ATTEND_DIM(D)                                      \
    case D:                                                \
        *main = of_format<F16, D>(format, groups, queries); \
        *join = moe_attend_join_kernel<F16, D>;            \
        break
        ATTEND_DIM(32);
        ATTEND_DIM(64);
        ATTEND_DIM(80);
        ATTEND_DIM(96);
        ATTEND_DIM(112);
        ATTEND_DIM(128);
        ATTEND_DIM(192);
        default: ATTEND_DIM(256);
#undef ATTEND_DIM
    }
}

// How the work is cut (the lengths are known on the device only): queries of a tile, ranges of
// work; and the workspace's layout.
struct AttendShape {
    int queries, ranges;
    int64_t stat, sum, bytes;
};
// entries: the sequences, or the groups of them that a shared prompt's tokens are computed for together.
static AttendShape attend_shape(const CacheParams &c, int32_t rows, int32_t q_heads, int32_t entries) {
    AttendShape s;
    // The least tile that holds the queries that share a key head, on average over the entries (their
    // own numbers are on the device): a sequence with more of them reads its cache again. (8 trees of 8 to 16 rows, 4
    // heads a key head, mean 56: the main launch 87 us with 64, 109 with 128, before items' starts counted as work.)
    const int64_t mean = ((int64_t)rows * (q_heads / c.heads) + entries - 1) / entries;
    s.queries = mean <= 16 ? 16 : mean <= 32 ? 32 : mean <= 64 ? 64 : 128;
    s.ranges = COMPUTE_UNITS * attend_blocks(c.dim, s.queries);     // as many workgroups as the card holds at once
    s.stat = (int64_t)s.ranges * sizeof(AttendPart);
    s.sum = s.stat + (int64_t)s.ranges * 2 * 2 * s.queries * 4;
    s.bytes = s.sum + (int64_t)s.ranges * 2 * s.queries * c.dim * 4;
    return s;
}

// What a shared prompt's pass leaves for the second one, behind the parts: tokens taken of each sequence, statistics, sums.
struct PriorShape {
    int64_t skip, stat, sum, bytes;
};
static PriorShape prior_shape(const CacheParams &c, int32_t rows, int32_t q_heads, int64_t parts) {
    PriorShape s;
    s.skip = (parts + 15) & ~15ll;
    s.stat = (s.skip + (int64_t)c.seqs * 4 + 15) & ~15ll;
    s.sum = (s.stat + (int64_t)rows * q_heads * 8 + 15) & ~15ll;
    s.bytes = s.sum + (int64_t)rows * q_heads * c.dim * 4;
    return s;
}

int64_t attend_workspace(const CacheParams &c, int32_t rows, int32_t q_heads, int32_t groups) {
    const int64_t own = attend_shape(c, rows, q_heads, c.seqs).bytes;
    if (!groups) return own;
    const int64_t common = attend_shape(c, rows, q_heads, groups).bytes;
    return prior_shape(c, rows, q_heads, own > common ? own : common).bytes;
}

static int launch_pass(const AttendCall &a, AttendParams &p, const AttendShape &shape) {
    p.tile_queries = shape.queries;
    p.ranges = shape.ranges;
    p.parts = (AttendPart *)a.workspace;
    p.part_stat = (float *)((char *)a.workspace + shape.stat);
    p.part_sum = (float *)((char *)a.workspace + shape.sum);
    AttendKernel main, join;
    if (a.f16)
        of_dim<true>(p.c.dim, a.format, a.shared != nullptr, shape.queries, &main, &join);
    else
        of_dim<false>(p.c.dim, a.format, a.shared != nullptr, shape.queries, &main, &join);
    int rc;
    if ((rc = launch("attend", main, dim3((unsigned)shape.ranges), dim3(256), p, a.stream))) return rc;
    // More workgroups join more queries at once, but each lists the work first: few queries a key head make few
    // (item, query) pairs (one row over 777 tokens: 5.9 us with 512, 6.4 with 1024), many make thousands (64-row trees
    // over 4100: 14.7 and 10.3).
    return launch("attend join", join, dim3(shape.queries == 16 ? 512 : 1024), dim3(256), p, a.stream);
}

int check_shared(const moe_shared_prefix *s, const CacheParams &c) {
    int rc;
    if ((rc = check_words("shared group_start", s->group_start)) || (rc = check_words("shared len", s->len))) return rc;
    if (s->groups < 1 || s->groups > c.seqs)
        return api_fail(MOE_ERR_SHAPE, "shared: %d groups, %d sequences", s->groups, c.seqs);
    return MOE_OK;
}

int attend_run(const AttendCall &a, AttendParams &p) {
    int rc;
    if ((rc = check_rows(a.rows, a.q_heads, p.c))) return rc;
    const int64_t w = (int64_t)a.q_heads * p.c.dim;
    if ((rc = check_matrix("q", a.q, a.q_stride, w, 16)) || (rc = check_matrix("out", a.out, a.out_stride, w, 16)) ||
        (rc = check_words("row_start", a.row_start)))
        return rc;
    if (a.mask && (rc = check_words("mask", a.mask, 8))) return rc;
    if (!std::isfinite(a.scale)) return api_fail(MOE_ERR_INVALID_ARG, "scale is not finite");
    if (rows_overlap(a.out, a.out_stride, w, a.q, a.q_stride, w, a.rows))
        return api_fail(MOE_ERR_ALIAS, "out overlaps q");
    if (a.shared && (rc = check_shared(a.shared, p.c))) return rc;
    const AttendShape own = attend_shape(p.c, a.rows, a.q_heads, p.c.seqs);
    const int32_t groups = a.shared ? a.shared->groups : 0;
    if ((rc = check_workspace(a.workspace, a.workspace_bytes, attend_workspace(p.c, a.rows, a.q_heads, groups))) ||
        (rc = check_device()))
        return rc;
    p.q = (const uint16_t *)a.q;
    p.out = (uint16_t *)a.out;
    p.q_stride = a.q_stride;
    p.out_stride = a.out_stride;
    p.row_start = a.row_start;
    // The kernel takes maxima of unscaled scores, so its factor is positive: a negative scale turns the queries'
    // signs instead, and one of 0 (or nearly) becomes so small that all weights are 1.
    p.scale_log2 = std::fmin(std::fmax(std::fabs(a.scale) * 1.44269504088896340736f, 1e-30f), 3.4e38f);
    p.q_sign = a.scale < 0 ? (int16_t)0x8000 : 0;
    p.rows = a.rows;
    p.q_heads = a.q_heads;
    p.group = a.q_heads / p.c.heads;
    if (a.shared) {
        const AttendShape common = attend_shape(p.c, a.rows, a.q_heads, groups);
        const PriorShape prior = prior_shape(p.c, a.rows, a.q_heads, own.bytes > common.bytes ? own.bytes : common.bytes);
        int32_t *skip = (int32_t *)((char *)a.workspace + prior.skip);
        p.prior_stat = (float *)((char *)a.workspace + prior.stat);
        p.prior_sum = (float *)((char *)a.workspace + prior.sum);
        p.entries = p.groups = groups;
        p.group_start = a.shared->group_start;
        p.shared_len = a.shared->len;
        p.skip_out = skip;
        if ((rc = launch_pass(a, p, common))) return rc;
        p.group_start = p.shared_len = nullptr;
        p.skip_out = nullptr;
        p.skip = skip;
    }
    p.entries = p.c.seqs;
    p.mask = a.mask;
    return launch_pass(a, p, own);
}

}  // namespace moe
