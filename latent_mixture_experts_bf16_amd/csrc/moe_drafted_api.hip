// moe_drafted_api.hip -- host side of the C ABI declared in include/moe_drafted.h: argument
// checks, launch shapes, launches. Refusals name the argument; nothing is enqueued after one.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstring>

#include "drafted_plan.h"

namespace moe {
template <bool F16, bool HALF, int W> __global__ void moe_rope_kernel(RopeParams p);
template <bool F16, int D, int NQ, int QW> __global__ void moe_attend_kernel(AttendParams p);
template <bool F16, int D> __global__ void moe_attend_join_kernel(AttendParams p);
template <typename L> __global__ void moe_verify_stats_kernel(VerifyParams p);
template <typename L> __global__ void moe_verify_walk_kernel(VerifyParams p);
template <typename L> __global__ void moe_verify_left_kernel(VerifyParams p);
struct LogitF32;
struct LogitBf16;
struct LogitF16;
__global__ void moe_keep_kernel(KeepParams p);
}  // namespace moe

using namespace moe;

static const char *type_name(int dt) {
    switch (dt) {
    case MOE_DT_BF16: return "bf16";
    case MOE_DT_F16: return "f16";
    case MOE_DT_F32: return "f32";
    case MOE_DT_U32: return "u32";
    case MOE_DT_I32: return "i32";
    default: return "unknown";
    }
}

// MOE_OK where the current device is a gfx950. Asked of the runtime once per device.
static int check_device() {
    constexpr int MOST = 64;
    static std::atomic<bool> known[MOST];
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess || dev < 0) return api_fail(MOE_ERR_DEVICE, "no HIP device (%s)", hipGetErrorString(e));
    if (dev < MOST && known[dev].load(std::memory_order_relaxed)) return MOE_OK;
    hipDeviceProp_t prop;
    if ((e = hipGetDeviceProperties(&prop, dev)) != hipSuccess)
        return api_fail(MOE_ERR_DEVICE, "hipGetDeviceProperties: %s", hipGetErrorString(e));
    if (strncmp(prop.gcnArchName, "gfx950", 6) != 0)
        return api_fail(MOE_ERR_DEVICE, "device %d is %s; this library is built for gfx950 (MI355X)", dev,
                        prop.gcnArchName);
    if (dev < MOST) known[dev].store(true, std::memory_order_relaxed);
    return MOE_OK;
}

template <typename P>
static int launch(const char *what, void (*kernel)(P), dim3 grid, dim3 block, P p, void *stream) {
    void *args[] = {&p};
    const hipError_t e = hipLaunchKernel((const void *)kernel, grid, block, args, 0, (hipStream_t)stream);
    if (e != hipSuccess) return api_fail(MOE_ERR_HIP, "%s launch: %s", what, hipGetErrorString(e));
    return MOE_OK;
}

// ------------------------------------------------------------------ the cache

static bool dim_ok(int64_t d) {
    return d == 32 || d == 64 || d == 80 || d == 96 || d == 112 || d == 128 || d == 192 || d == 256;
}

static int check_kv(const char *name, const moe_tensor &t) {
    if (!t.data) return api_fail(MOE_ERR_MISSING_TENSOR, "%s: missing (data == NULL)", name);
    if (t.dtype != MOE_DT_BF16 && t.dtype != MOE_DT_F16)
        return api_fail(MOE_ERR_DTYPE, "%s: dtype %s (bf16 or f16)", name, type_name(t.dtype));
    if (t.ndim != 4)
        return api_fail(MOE_ERR_LAYOUT, "%s: rank %d, expected 4 ([pages][page][kv_heads][dim])", name, t.ndim);
    for (int i = 0; i < 4; ++i)
        if (t.shape[i] < 1) return api_fail(MOE_ERR_SHAPE, "%s: dim %d is %lld", name, i, (long long)t.shape[i]);
    if (t.shape[0] > 0x7FFFFFFF) return api_fail(MOE_ERR_SHAPE, "%s: %lld pages", name, (long long)t.shape[0]);
    if (t.shape[1] % 16 || t.shape[1] > 1 << 20)
        return api_fail(MOE_ERR_SHAPE, "%s: page of %lld tokens (a multiple of 16, at most 2^20)", name,
                        (long long)t.shape[1]);
    if (t.shape[2] > 1 << 16) return api_fail(MOE_ERR_SHAPE, "%s: %lld heads", name, (long long)t.shape[2]);
    if (!dim_ok(t.shape[3]))
        return api_fail(MOE_ERR_SHAPE, "%s: head width %lld (32, 64, 80, 96, 112, 128, 192 or 256)", name,
                        (long long)t.shape[3]);
    if (t.stride[3] != 1) return api_fail(MOE_ERR_LAYOUT, "%s: last dim not contiguous", name);
    int64_t span = t.shape[3];
    for (int i = 0; i < 3; ++i) {
        if (t.stride[i] < 0 || t.stride[i] % 8)
            return api_fail(MOE_ERR_LAYOUT, "%s: stride[%d] = %lld (a multiple of 8, not negative)", name, i,
                            (long long)t.stride[i]);
        if (t.shape[i] > 1 && t.stride[i] < t.shape[3])
            return api_fail(MOE_ERR_LAYOUT, "%s: stride[%d] = %lld: elements overlap", name, i, (long long)t.stride[i]);
        if (i) {
            if (t.stride[i] >= (int64_t)1 << 30)
                return api_fail(MOE_ERR_SHAPE, "%s: stride[%d] = %lld (below 2^30)", name, i, (long long)t.stride[i]);
            span += (t.shape[i] - 1) * t.stride[i];
        }
    }
    if (span >= (int64_t)1 << 30) return api_fail(MOE_ERR_SHAPE, "%s: a page spans %lld elements (below 2^30)", name,
                                                  (long long)span);
    if ((uintptr_t)t.data & 15) return api_fail(MOE_ERR_LAYOUT, "%s: data pointer not 16-byte aligned", name);
    return MOE_OK;
}

static int check_i32(const char *name, const moe_tensor &t, int ndim) {
    if (!t.data) return api_fail(MOE_ERR_MISSING_TENSOR, "%s: missing (data == NULL)", name);
    if (t.dtype != MOE_DT_I32) return api_fail(MOE_ERR_DTYPE, "%s: dtype %s, expected i32", name, type_name(t.dtype));
    if (t.ndim != ndim) return api_fail(MOE_ERR_LAYOUT, "%s: rank %d, expected %d", name, t.ndim, ndim);
    for (int i = 0; i < ndim; ++i)
        if (t.shape[i] < 1) return api_fail(MOE_ERR_SHAPE, "%s: dim %d is %lld", name, i, (long long)t.shape[i]);
    if (t.shape[ndim - 1] > 1 && t.stride[ndim - 1] != 1)
        return api_fail(MOE_ERR_LAYOUT, "%s: last dim not contiguous", name);
    if ((uintptr_t)t.data & 3) return api_fail(MOE_ERR_LAYOUT, "%s: data pointer not 4-byte aligned", name);
    return MOE_OK;
}

static int check_cache(const moe_paged_cache *c, CacheParams &p) {
    int rc;
    if (!c) return api_fail(MOE_ERR_INVALID_ARG, "cache: descriptor is NULL");
    if ((rc = check_kv("cache k", c->k)) || (rc = check_kv("cache v", c->v))) return rc;
    if (c->k.dtype != c->v.dtype)
        return api_fail(MOE_ERR_DTYPE, "cache v: dtype %s, k is %s", type_name(c->v.dtype), type_name(c->k.dtype));
    for (int i = 0; i < 4; ++i)
        if (c->k.shape[i] != c->v.shape[i])
            return api_fail(MOE_ERR_SHAPE, "cache v: dim %d is %lld, k's is %lld", i, (long long)c->v.shape[i],
                            (long long)c->k.shape[i]);
    if ((rc = check_i32("cache table", c->table, 2)) || (rc = check_i32("cache len", c->len, 1))) return rc;
    const int64_t seqs = c->table.shape[0];
    if (seqs > 1 << 16) return api_fail(MOE_ERR_SHAPE, "cache table: %lld sequences (at most 2^16)", (long long)seqs);
    if (c->table.shape[1] > 0x7FFFFFFF)
        return api_fail(MOE_ERR_SHAPE, "cache table: %lld pages a sequence", (long long)c->table.shape[1]);
    if (c->len.shape[0] != seqs)
        return api_fail(MOE_ERR_SHAPE, "cache len: %lld sequences, the table has %lld", (long long)c->len.shape[0],
                        (long long)seqs);
    if (seqs > 1 && c->table.stride[0] < 0)
        return api_fail(MOE_ERR_LAYOUT, "cache table: stride[0] = %lld", (long long)c->table.stride[0]);
    if (!c->flags) return api_fail(MOE_ERR_INVALID_ARG, "cache flags: NULL");
    if ((uintptr_t)c->flags & 3) return api_fail(MOE_ERR_LAYOUT, "cache flags: not 4-byte aligned");
    p.k = {(const uint16_t *)c->k.data, c->k.stride[0], c->k.stride[1], c->k.stride[2]};
    p.v = {(const uint16_t *)c->v.data, c->v.stride[0], c->v.stride[1], c->v.stride[2]};
    p.table = (const int32_t *)c->table.data;
    p.len = (const int32_t *)c->len.data;
    p.flags = c->flags;
    p.table_stride = c->table.stride[0];
    p.pages = (int32_t)c->k.shape[0];
    p.page = (int32_t)c->k.shape[1];
    p.heads = (int32_t)c->k.shape[2];
    p.dim = (int32_t)c->k.shape[3];
    p.seqs = (int32_t)seqs;
    const int64_t cap = c->table.shape[1] * c->k.shape[1], most = ((int64_t)1 << 31) - 64;
    p.cap = (int32_t)(cap < most ? cap : most);
    return MOE_OK;
}

static int check_rows(int32_t rows, int32_t q_heads, const CacheParams &c) {
    if (rows < 1 || rows > 1 << 20) return api_fail(MOE_ERR_ROWS, "rows %d outside 1..2^20", rows);
    if (q_heads < 1 || q_heads > 1 << 16 || q_heads % c.heads)
        return api_fail(MOE_ERR_SHAPE, "q: %d heads (a multiple of the cache's %d)", q_heads, c.heads);
    return MOE_OK;
}

// A row matrix of 16-bit elements: `width` used of each `stride`.
static int check_matrix(const char *name, const void *p, int64_t stride, int64_t width, int align) {
    if (!p) return api_fail(MOE_ERR_INVALID_ARG, "%s: NULL", name);
    if (stride < width || stride >= (int64_t)1 << 40)
        return api_fail(MOE_ERR_LAYOUT, "%s: row stride %lld, %lld wide", name, (long long)stride, (long long)width);
    if ((uintptr_t)p % align || stride * 2 % align)
        return api_fail(MOE_ERR_LAYOUT, "%s: pointer and row stride must be %d-byte aligned", name, align);
    return MOE_OK;
}

static int check_words(const char *name, const void *p, int align = 4) {
    if (!p) return api_fail(MOE_ERR_INVALID_ARG, "%s: NULL", name);
    if ((uintptr_t)p % align) return api_fail(MOE_ERR_LAYOUT, "%s: not %d-byte aligned", name, align);
    return MOE_OK;
}

static int check_workspace(const void *p, size_t bytes, int64_t need) {
    if (need && !p) return api_fail(MOE_ERR_INVALID_ARG, "workspace: NULL");
    if ((uintptr_t)p & 15) return api_fail(MOE_ERR_LAYOUT, "workspace: not 16-byte aligned");
    if (bytes < (size_t)need)
        return api_fail(MOE_ERR_SHAPE, "workspace: %zu bytes, %lld needed", bytes, (long long)need);
    return MOE_OK;
}

static bool overlap(const void *a, int64_t abytes, const void *b, int64_t bbytes) {
    const char *x = (const char *)a, *y = (const char *)b;
    return x < y + bbytes && y < x + abytes;
}

// Whether two row matrices share an element: their ranges meet, and they are not different columns
// of the same rows (the parts of one projection's output).
static bool rows_overlap(const void *a, int64_t as, int64_t aw, const void *b, int64_t bs, int64_t bw, int64_t rows) {
    if (!overlap(a, ((rows - 1) * as + aw) * 2, b, ((rows - 1) * bs + bw) * 2)) return false;
    if (as != bs) return true;
    const int64_t d = ((const char *)b - (const char *)a) % (as * 2), at = d < 0 ? d + as * 2 : d;   // of b in a's rows
    return !(at >= aw * 2 && at + bw * 2 <= as * 2);
}

extern "C" int moe_paged_cache_check(const moe_paged_cache *c) {
    api_clear();
    CacheParams p;
    return check_cache(c, p);
}

// ------------------------------------------------------------------ rotary append

template <bool F16, bool HALF> static void (*rope_kernel(int w))(RopeParams) {
    if (w == 8) return moe_rope_kernel<F16, HALF, 8>;
    if (w == 4) return moe_rope_kernel<F16, HALF, 4>;
    if constexpr (HALF) {
        if (w == 1) return moe_rope_kernel<F16, HALF, 1>;
    }
    return moe_rope_kernel<F16, HALF, 2>;
}

extern "C" int moe_rope_append(const moe_paged_cache *c, const moe_rope *r, int32_t rows, const void *q,
                               int64_t q_stride, int32_t q_heads, const void *k, int64_t k_stride, const void *v,
                               int64_t v_stride, const int32_t *row_start, const int32_t *positions, void *q_out,
                               int64_t q_out_stride, void *hip_stream) {
    api_clear();
    RopeParams p;
    memset(&p, 0, sizeof p);
    int rc;
    if ((rc = check_cache(c, p.c)) || (rc = check_rows(rows, q_heads, p.c))) return rc;
    if (!r) return api_fail(MOE_ERR_INVALID_ARG, "rope: NULL");
    if ((rc = check_words("rope freqs", r->freqs, 8))) return rc;
    if (r->pairs < 1 || r->pairs > p.c.dim / 2)
        return api_fail(MOE_ERR_SHAPE, "rope: %d pairs, heads of %d", r->pairs, p.c.dim);
    if (r->layout != MOE_ROPE_HALF && r->layout != MOE_ROPE_INTERLEAVED)
        return api_fail(MOE_ERR_INVALID_ARG, "rope: layout %d", r->layout);
    if (!std::isfinite(r->magnitude)) return api_fail(MOE_ERR_INVALID_ARG, "rope: magnitude is not finite");
    const int64_t qw = (int64_t)q_heads * p.c.dim, kw = (int64_t)p.c.heads * p.c.dim;
    if ((rc = check_matrix("q", q, q_stride, qw, 2)) || (rc = check_matrix("k", k, k_stride, kw, 2)) ||
        (rc = check_matrix("v", v, v_stride, kw, 2)) || (rc = check_matrix("q_out", q_out, q_out_stride, qw, 2)) ||
        (rc = check_words("row_start", row_start)))
        return rc;
    if (positions && (rc = check_words("positions", positions))) return rc;
    if (rows_overlap(q_out, q_out_stride, qw, q, q_stride, qw, rows) && !(q_out == q && q_out_stride == q_stride))
        return api_fail(MOE_ERR_ALIAS, "q_out partially overlaps q");
    if (rows_overlap(q_out, q_out_stride, qw, k, k_stride, kw, rows) ||
        rows_overlap(q_out, q_out_stride, qw, v, v_stride, kw, rows))
        return api_fail(MOE_ERR_ALIAS, "q_out overlaps k or v");
    // the widest piece that divides the rotated part and that every row is aligned for
    const bool half = r->layout == MOE_ROPE_HALF, f16 = c->k.dtype == MOE_DT_F16;
    const uint64_t odd = (uint64_t)(half ? r->pairs : 2 * r->pairs) | (uint64_t)q_stride | (uint64_t)k_stride |
                         (uint64_t)v_stride | (uint64_t)q_out_stride |
                         (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q_out) >> 1);
    const int w = odd % 8 == 0 ? 8 : odd % 4 == 0 ? 4 : odd % 2 == 0 ? 2 : 1;
    if (w == 1 && !half)
        return api_fail(MOE_ERR_LAYOUT, "interleaved pairs need rows aligned to 4 bytes");
    if ((rc = check_device())) return rc;
    p.freqs = r->freqs;
    p.pairs = r->pairs;
    p.magnitude = r->magnitude;
    p.q = (const uint16_t *)q;
    p.kn = (const uint16_t *)k;
    p.vn = (const uint16_t *)v;
    p.qo = (uint16_t *)q_out;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.qo_stride = q_out_stride;
    p.row_start = row_start;
    p.positions = positions;
    p.rows = rows;
    p.q_heads = q_heads;
    void (*kern)(RopeParams) = f16 ? (half ? rope_kernel<true, true>(w) : rope_kernel<true, false>(w))
                                   : (half ? rope_kernel<false, true>(w) : rope_kernel<false, false>(w));
    return launch("rope_append", kern, dim3((unsigned)rows), dim3(256), p, hip_stream);
}

// ------------------------------------------------------------------ tree attention

typedef void (*AttendKernel)(AttendParams);

template <bool F16, int D> static AttendKernel attend_kernel(int queries) {
    return queries == 16   ? moe_attend_kernel<F16, D, 1, 1>
           : queries == 32 ? moe_attend_kernel<F16, D, 2, 1>
           : queries == 64 ? moe_attend_kernel<F16, D, 2, 2>
                           : moe_attend_kernel<F16, D, 2, 4>;
}
template <bool F16> static void attend_kernels(int dim, int queries, AttendKernel *main, AttendKernel *join) {
    switch (dim) {
#define ATTEND_DIM(D)                            \
    case D:                                      \
        *main = attend_kernel<F16, D>(queries);  \
        *join = moe_attend_join_kernel<F16, D>;  \
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
static AttendShape attend_shape(const CacheParams &c, int32_t rows, int32_t q_heads) {
    AttendShape s;
    // The least tile that holds the queries that share a key head, on average over the sequences (their
    // own numbers are on the device): a sequence with more of them reads its cache again. (8 trees of 8 to 16 rows, 4
    // heads a key head, mean 56: the main launch 87 us with 64, 109 with 128, before items' starts counted as work.)
    const int64_t mean = ((int64_t)rows * (q_heads / c.heads) + c.seqs - 1) / c.seqs;
    s.queries = mean <= 16 ? 16 : mean <= 32 ? 32 : mean <= 64 ? 64 : 128;
    s.ranges = COMPUTE_UNITS * attend_blocks(c.dim, s.queries);     // as many workgroups as the card holds at once
    s.stat = (int64_t)s.ranges * sizeof(AttendPart);
    s.sum = s.stat + (int64_t)s.ranges * 2 * 2 * s.queries * 4;
    s.bytes = s.sum + (int64_t)s.ranges * 2 * s.queries * c.dim * 4;
    return s;
}

extern "C" int64_t moe_tree_attend_workspace(const moe_paged_cache *c, int32_t rows, int32_t q_heads) {
    api_clear();
    CacheParams p;
    int rc;
    if ((rc = check_cache(c, p)) || (rc = check_rows(rows, q_heads, p))) return -rc;
    return attend_shape(p, rows, q_heads).bytes;
}

extern "C" int moe_tree_attend(const moe_paged_cache *c, int32_t rows, const void *q, int64_t q_stride,
                               int32_t q_heads, const int32_t *row_start, const uint64_t *mask, float scale,
                               void *out, int64_t out_stride, void *workspace, size_t workspace_bytes,
                               void *hip_stream) {
    api_clear();
    AttendParams p;
    memset(&p, 0, sizeof p);
    int rc;
    if ((rc = check_cache(c, p.c)) || (rc = check_rows(rows, q_heads, p.c))) return rc;
    const int64_t w = (int64_t)q_heads * p.c.dim;
    if ((rc = check_matrix("q", q, q_stride, w, 16)) || (rc = check_matrix("out", out, out_stride, w, 16)) ||
        (rc = check_words("row_start", row_start)))
        return rc;
    if (mask && (rc = check_words("mask", mask, 8))) return rc;
    if (!std::isfinite(scale)) return api_fail(MOE_ERR_INVALID_ARG, "scale is not finite");
    if (rows_overlap(out, out_stride, w, q, q_stride, w, rows))
        return api_fail(MOE_ERR_ALIAS, "out overlaps q");
    const AttendShape shape = attend_shape(p.c, rows, q_heads);
    if ((rc = check_workspace(workspace, workspace_bytes, shape.bytes)) || (rc = check_device())) return rc;
    p.q = (const uint16_t *)q;
    p.out = (uint16_t *)out;
    p.q_stride = q_stride;
    p.out_stride = out_stride;
    p.row_start = row_start;
    p.mask = mask;
    // The kernel takes maxima of unscaled scores, so its factor is positive: a negative scale turns the queries'
    // signs instead, and one of 0 (or nearly) becomes so small that all weights are 1.
    p.scale_log2 = std::fmin(std::fmax(std::fabs(scale) * 1.44269504088896340736f, 1e-30f), 3.4e38f);
    p.q_sign = scale < 0 ? (int16_t)0x8000 : 0;
    p.rows = rows;
    p.q_heads = q_heads;
    p.group = q_heads / p.c.heads;
    p.tile_queries = shape.queries;
    p.ranges = shape.ranges;
    p.parts = (AttendPart *)workspace;
    p.part_stat = (float *)((char *)workspace + shape.stat);
    p.part_sum = (float *)((char *)workspace + shape.sum);
    AttendKernel main, join;
    if (c->k.dtype == MOE_DT_F16)
        attend_kernels<true>(p.c.dim, shape.queries, &main, &join);
    else
        attend_kernels<false>(p.c.dim, shape.queries, &main, &join);
    if ((rc = launch("tree_attend", main, dim3((unsigned)shape.ranges), dim3(256), p, hip_stream))) return rc;
    // More workgroups join more queries at once, but each lists the work first: few queries a key head make few
    // (item, query) pairs (one row over 777 tokens: 5.9 us with 512, 6.4 with 1024), many make thousands (64-row trees
    // over 4100: 14.7 and 10.3).
    return launch("tree_attend join", join, dim3(shape.queries == 16 ? 512 : 1024), dim3(256), p, hip_stream);
}

// ------------------------------------------------------------------ draft verification

static int check_verify_sizes(int64_t rows, int32_t seqs, int64_t vocab) {
    if (rows < 1 || rows > 1 << 20) return api_fail(MOE_ERR_ROWS, "rows %lld outside 1..2^20", (long long)rows);
    if (seqs < 1 || seqs > 1 << 16) return api_fail(MOE_ERR_SHAPE, "%d sequences outside 1..2^16", seqs);
    if (vocab < 1 || vocab > MAX_VOCAB)
        return api_fail(MOE_ERR_SHAPE, "vocabulary %lld outside 1..2^20", (long long)vocab);
    return MOE_OK;
}

// Bytes of workspace; with a base and p, also its parts.
static int64_t verify_layout(int64_t rows, int64_t seqs, int64_t vocab, char *base, VerifyParams *p) {
    const int64_t chunks = (vocab + VOCAB_CHUNK - 1) / VOCAB_CHUNK;
    const int64_t row_stat = rows * chunks * (int64_t)sizeof(LogitStat);
    const int64_t state = row_stat + rows * (int64_t)sizeof(LogitStat);
    const int64_t left = state + seqs * (int64_t)sizeof(WalkState);
    const int64_t token_p = left + seqs * chunks * 8;
    const int64_t pick = token_p + rows * 8;
    const int64_t arrived = pick + rows * 4;
    if (p) {
        p->chunks = (int32_t)chunks;
        p->chunk_stat = (LogitStat *)base;
        p->row_stat = (LogitStat *)(base + row_stat);
        p->state = (WalkState *)(base + state);
        p->left = (double *)(base + left);
        p->token_p = (double *)(base + token_p);
        p->pick = (int32_t *)(base + pick);
        p->arrived = (uint32_t *)(base + arrived);
    }
    return arrived + seqs * 4;
}

extern "C" int64_t moe_draft_verify_workspace(int32_t rows, int32_t seqs, int32_t vocab) {
    api_clear();
    const int rc = check_verify_sizes(rows, seqs, vocab);
    return rc ? -rc : verify_layout(rows, seqs, vocab, nullptr, nullptr);
}

// Tests of whole rows that are launched before the last one, whose own workgroups take what is left: a chain
// never needs a second one. An empty one costs 2 to 5 us (also with fewer workgroups), one too few a row
// summed by a single workgroup (128 chunks, four at a time).
constexpr int TREE_ROUNDS = 3;

template <typename L> static int verify_launches(VerifyParams &p, void *stream) {
    int rc;
    const unsigned y = (unsigned)(p.rows < 32768 ? p.rows : 32768);
    if ((rc = launch("draft_verify", moe_verify_stats_kernel<L>,
                     dim3((unsigned)(p.chunks + 3) / 4, y, ((unsigned)p.rows + y - 1) / y), dim3(256), p, stream)) ||
        (rc = launch("draft_verify walk", moe_verify_walk_kernel<L>, dim3((unsigned)p.seqs), dim3(1024), p, stream)))
        return rc;
    const int rounds = !p.draft ? 0 : p.parent ? TREE_ROUNDS : 1;
    for (int i = 0; i < rounds; ++i) {
        p.last_round = i == rounds - 1;
        if ((rc = launch("draft_verify left", moe_verify_left_kernel<L>,
                         dim3((unsigned)p.seqs, (unsigned)(p.chunks + 3) / 4), dim3(256), p, stream)))
            return rc;
    }
    return MOE_OK;
}

extern "C" int moe_draft_verify(const moe_tensor *logits, const int32_t *tokens, const int32_t *row_start,
                                int32_t seqs, const int32_t *parent, const float *u_test, const float *u_pick,
                                const float *draft_probs, int64_t draft_stride, const float *temperature,
                                int32_t *n_keep, int32_t *path, int32_t *out_tokens, float *logprobs, uint32_t *flags,
                                void *workspace, size_t workspace_bytes, void *hip_stream) {
    api_clear();
    int rc;
    if (!logits) return api_fail(MOE_ERR_INVALID_ARG, "logits: descriptor is NULL");
    if (!logits->data) return api_fail(MOE_ERR_MISSING_TENSOR, "logits: missing (data == NULL)");
    if (logits->dtype != MOE_DT_F32 && logits->dtype != MOE_DT_BF16 && logits->dtype != MOE_DT_F16)
        return api_fail(MOE_ERR_DTYPE, "logits: dtype %s (f32, bf16 or f16)", type_name(logits->dtype));
    if (logits->ndim != 2) return api_fail(MOE_ERR_LAYOUT, "logits: rank %d, expected 2", logits->ndim);
    const int64_t rows = logits->shape[0], vocab = logits->shape[1];
    if ((rc = check_verify_sizes(rows, seqs, vocab))) return rc;
    if ((vocab > 1 && logits->stride[1] != 1) || (rows > 1 && logits->stride[0] < vocab))
        return api_fail(MOE_ERR_LAYOUT, "logits: strides %lld, %lld (rows of contiguous logits)",
                        (long long)logits->stride[0], (long long)logits->stride[1]);
    if ((rc = check_words("logits", logits->data, logits->dtype == MOE_DT_F32 ? 4 : 2)) ||
        (rc = check_words("tokens", tokens)) || (rc = check_words("row_start", row_start)) ||
        (rc = check_words("u_pick", u_pick)) || (rc = check_words("n_keep", n_keep)) ||
        (rc = check_words("path", path)) || (rc = check_words("out_tokens", out_tokens)) ||
        (rc = check_words("logprobs", logprobs)) || (rc = check_words("flags", flags)))
        return rc;
    if ((parent && (rc = check_words("parent", parent))) ||
        (temperature && (rc = check_words("temperature", temperature))))
        return rc;
    if (draft_probs) {
        if ((rc = check_words("draft_probs", draft_probs)) || (rc = check_words("u_test", u_test))) return rc;
        if (rows > 1 && draft_stride < vocab)
            return api_fail(MOE_ERR_LAYOUT, "draft_probs: row stride %lld, %lld wide", (long long)draft_stride,
                            (long long)vocab);
    }
    if ((rc = check_workspace(workspace, workspace_bytes, verify_layout(rows, seqs, vocab, nullptr, nullptr))) ||
        (rc = check_device()))
        return rc;
    VerifyParams p;
    memset(&p, 0, sizeof p);
    p.logits = logits->data;
    p.logit_stride = logits->stride[0];
    p.draft_stride = draft_stride;
    p.tokens = tokens;
    p.row_start = row_start;
    p.parent = parent;
    p.u_test = u_test;
    p.u_pick = u_pick;
    p.draft = draft_probs;
    p.temperature = temperature;
    p.n_keep = n_keep;
    p.path = path;
    p.out_tokens = out_tokens;
    p.logprobs = logprobs;
    p.flags = flags;
    p.rows = (int32_t)rows;
    p.seqs = seqs;
    p.vocab = (int32_t)vocab;
    verify_layout(rows, seqs, vocab, (char *)workspace, &p);
    return logits->dtype == MOE_DT_F32    ? verify_launches<LogitF32>(p, hip_stream)
           : logits->dtype == MOE_DT_BF16 ? verify_launches<LogitBf16>(p, hip_stream)
                                          : verify_launches<LogitF16>(p, hip_stream);
}

// ------------------------------------------------------------------ path keeping

extern "C" int moe_path_keep(const moe_paged_cache *c, const int32_t *row_start, int32_t rows, const int32_t *n_keep,
                             const int32_t *path, int32_t *new_len, void *hip_stream) {
    api_clear();
    KeepParams p;
    memset(&p, 0, sizeof p);
    int rc;
    if ((rc = check_cache(c, p.c)) || (rc = check_rows(rows, p.c.heads, p.c))) return rc;
    if ((rc = check_words("row_start", row_start)) || (rc = check_words("n_keep", n_keep)) ||
        (rc = check_words("path", path)) || (rc = check_words("new_len", new_len)))
        return rc;
    if ((rc = check_device())) return rc;
    p.row_start = row_start;
    p.n_keep = n_keep;
    p.path = path;
    p.new_len = new_len;
    p.rows = rows;
    return launch("path_keep", moe_keep_kernel, dim3((unsigned)p.c.seqs), dim3(256), p, hip_stream);
}

// ------------------------------------------------------------------ status

extern "C" int moe_drafted_status(uint32_t *flags, void *hip_stream) {
    api_clear();
    int rc;
    if ((rc = check_words("flags", flags))) return rc;
    uint32_t v = 0;
    const uint32_t zero = 0;
    hipError_t e = hipMemcpyAsync(&v, flags, 4, hipMemcpyDeviceToHost, (hipStream_t)hip_stream);
    if (e == hipSuccess) e = hipStreamSynchronize((hipStream_t)hip_stream);
    if (e == hipSuccess && v) e = hipMemcpyAsync(flags, &zero, 4, hipMemcpyHostToDevice, (hipStream_t)hip_stream);
    if (e == hipSuccess && v) e = hipStreamSynchronize((hipStream_t)hip_stream);
    if (e != hipSuccess) return api_fail(MOE_ERR_HIP, "status: %s", hipGetErrorString(e));
    if (!v) return MOE_OK;
    return api_fail(MOE_ERR_DEVICE_CHECK, "met on the device:%s%s%s%s%s%s",
                    v & MOE_FLAG_PAGE ? " a page outside the cache or past the table;" : "",
                    v & MOE_FLAG_LEN ? " a length outside the table;" : "",
                    v & MOE_FLAG_ROWS ? " row_start not ascending over the rows;" : "",
                    v & MOE_FLAG_PATH ? " a path that is not ascending rows of its sequence;" : "",
                    v & MOE_FLAG_TOKEN ? " a drafted token outside the vocabulary;" : "",
                    v & MOE_FLAG_LOGITS ? " logits without a value above -infinity;" : "");
}
