// attend_launch.hip -- host side of the attention kernels: their choice by type, head width, tile and format, their workspace
// and their launches.
#include "api_checks.h"

namespace moe {
template <bool F16, int D, int NQ, int QW, int FMT, bool SHARED> __global__ void moe_attend_kernel(AttendParams p);
template <bool F16, int D> __global__ void moe_attend_join_kernel(AttendParams p);
template <bool F16, int D> __global__ void moe_shared_join_kernel(SharedJoinParams p);

typedef void (*AttendKernel)(AttendParams);
typedef void (*SharedJoin)(SharedJoinParams);

struct Kernels {
    AttendKernel main, join;
    SharedJoin shared_join;
};

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
template <bool F16> static void of_dim(int dim, int format, bool groups, int queries, Kernels *k) {
    switch (dim) {
#define ATTEND_DIM(D)                                      \
    case D:                                                \
        k->main = of_format<F16, D>(format, groups, queries); \
        k->join = moe_attend_join_kernel<F16, D>;          \
        k->shared_join = moe_shared_join_kernel<F16, D>;   \
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
    int64_t items, stat, sum, bytes;
};
// entries: the sequences, or the groups of them that a shared prompt's tokens are computed for together. shares: of a batch that
// shares prompts, whose items are all parts.
static AttendShape attend_shape(const CacheParams &c, int32_t rows, int32_t q_heads, int32_t entries, bool shares) {
    AttendShape s;
    // The least tile that holds the queries that share a key head, on average over the entries (their
    // own numbers are on the device): a sequence with more of them reads its cache again. (8 trees of 8 to 16 rows, 4
    // heads a key head, mean 56: the main launch 87 us with 64, 109 with 128, before items' starts counted as work.)
    const int64_t mean = ((int64_t)rows * (q_heads / c.heads) + entries - 1) / entries;
    s.queries = mean <= 16 ? 16 : mean <= 32 ? 32 : mean <= 64 ? 64 : 128;
    s.ranges = COMPUTE_UNITS * attend_blocks(c.dim, s.queries);     // as many workgroups as the card holds at once
    // at most two parts a range; and where all are, a number for each item and a range's number more
    s.items = shares ? ((int64_t)rows * (q_heads / c.heads) / s.queries + entries) * c.heads : 0;
    const int64_t parts = shares ? s.items + s.ranges : 2 * s.ranges;
    s.stat = (int64_t)s.ranges * sizeof(AttendPart);
    s.sum = s.stat + parts * 2 * s.queries * 4;
    s.bytes = s.sum + parts * s.queries * c.dim * 4;
    return s;
}

static int64_t aligned(int64_t n) { return (n + 15) & ~15ll; }

// The workspace of a batch that shares prompts: the parts and items of both launches, and of each sequence its group and the tokens
// that are taken for it.
struct SharedShape {
    AttendShape common, own;
    int64_t own_at, common_items, own_items, shares, bytes;
};
static SharedShape shared_shape(const CacheParams &c, int32_t rows, int32_t q_heads, int32_t groups) {
    SharedShape s;
    s.common = attend_shape(c, rows, q_heads, groups, true);
    s.own = attend_shape(c, rows, q_heads, c.seqs, true);
    s.own_at = aligned(s.common.bytes);
    s.common_items = s.own_at + aligned(s.own.bytes);
    s.own_items = s.common_items + aligned(s.common.items * sizeof(AttendItem));
    s.shares = s.own_items + aligned(s.own.items * sizeof(AttendItem));
    s.bytes = s.shares + (int64_t)c.seqs * sizeof(SequenceShare);
    return s;
}

int64_t attend_workspace(const CacheParams &c, int32_t rows, int32_t q_heads, int32_t groups) {
    return groups ? shared_shape(c, rows, q_heads, groups).bytes : attend_shape(c, rows, q_heads, c.seqs, false).bytes;
}

// The launch of a pass whose parts lie at `base`.
static int launch_pass(const AttendCall &a, AttendParams &p, const AttendShape &shape, char *base, Kernels *k) {
    p.tile_queries = shape.queries;
    p.ranges = shape.ranges;
    p.parts = (AttendPart *)base;
    p.part_stat = (float *)(base + shape.stat);
    p.part_sum = (float *)(base + shape.sum);
    if (a.f16)
        of_dim<true>(p.c.dim, a.format, a.shared != nullptr, shape.queries, k);
    else
        of_dim<false>(p.c.dim, a.format, a.shared != nullptr, shape.queries, k);
    return launch("attend", k->main, dim3((unsigned)shape.ranges), dim3(256), p, a.stream);
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
    char *const base = (char *)a.workspace;
    Kernels k;
    if (!a.shared) {
        const AttendShape own = attend_shape(p.c, a.rows, a.q_heads, p.c.seqs, false);
        p.entries = p.c.seqs;
        p.mask = a.mask;
        if ((rc = launch_pass(a, p, own, base, &k))) return rc;
        // More workgroups join more queries at once, but each lists the work first: few queries a key head make few
        // (item, query) pairs (one row over 777 tokens: 5.9 us with 512, 6.4 with 1024), many make thousands (64-row trees
        // over 4100: 14.7 and 10.3).
        return launch("attend join", k.join, dim3(own.queries == 16 ? 512 : 1024), dim3(256), p, a.stream);
    }
    const SharedShape s = shared_shape(p.c, a.rows, a.q_heads, groups);
    SharedJoinParams j;
    memset(&j, 0, sizeof j);
    p.entries = p.groups = groups;
    p.group_start = a.shared->group_start;
    p.shared_len = a.shared->len;
    p.tell = (SequenceShare *)(base + s.shares);
    p.items = (AttendItem *)(base + s.common_items);
    if ((rc = launch_pass(a, p, s.common, base, &k))) return rc;
    j.common = {p.items, p.part_stat, p.part_sum, p.tile_queries, p.ranges};
    p.entries = p.c.seqs;
    p.group_start = p.shared_len = nullptr;
    p.shares = p.tell;
    p.tell = nullptr;
    p.mask = a.mask;
    p.items = (AttendItem *)(base + s.own_items);
    if ((rc = launch_pass(a, p, s.own, base + s.own_at, &k))) return rc;
    j.own = {p.items, p.part_stat, p.part_sum, p.tile_queries, p.ranges};
    j.row_start = a.row_start;
    j.shares = p.shares;
    j.out = p.out;
    j.out_stride = p.out_stride;
    j.rows = p.rows;
    j.q_heads = p.q_heads;
    j.kv_heads = p.c.heads;
    j.group = p.group;
    j.seqs = p.c.seqs;
    // A workgroup for each query while all run at once (512 queries of 16 rows after 16000 tokens: the call 44.7 us, 47.8 with a
    // wave for each; 128 queries: 20.7 and 22.4; 2048: the same); past that its other waves and its barrier cost more than
    // they save (4096: 109 and 106 us; 8192 of 256 short sequences: 67 and 57).
    const int64_t queries = (int64_t)p.rows * p.q_heads;
    j.apart = queries < 8 * COMPUTE_UNITS;
    // a grid's x holds less than 2^32 threads (past that a launch wrapped, without an error): more workgroups go on along y
    const int64_t blocks = j.apart ? queries : (queries + 3) / 4, x = blocks < 1 << 20 ? blocks : 1 << 20;
    return launch("shared join", k.shared_join, dim3((unsigned)x, (unsigned)((blocks + x - 1) / x)), dim3(256), j, a.stream);
}

}  // namespace moe
