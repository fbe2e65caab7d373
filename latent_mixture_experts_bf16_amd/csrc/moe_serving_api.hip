// moe_serving_api.hip -- host side of the C ABI declared in include/moe_serving.h: argument checks, launches.
#include <utility>

#include "api_checks.h"

namespace moe {
template <bool F16, int FMT, int MOST> __global__ void moe_append_kernel(AppendParams a);
template <bool F16, int FMT> __global__ void moe_read_kernel(ReadParams p);
template <int FMT> __global__ void moe_keep_kernel(KeepParams p);
template <typename L> __global__ void moe_sample_cells_kernel(SampleParams p);
template <typename L> __global__ void moe_sample_row_kernel(SampleParams p);
struct LogitF32;
struct LogitBf16;
struct LogitF16;
}  // namespace moe

using namespace moe;

// ------------------------------------------------------------------ a cache of codes

static int check_bytes(const char *name, const moe_tensor &t, int unit, int align) {
    if (!t.data) return api_fail(MOE_ERR_MISSING_TENSOR, "%s: missing (data == NULL)", name);
    if (t.dtype != MOE_DT_U8) return api_fail(MOE_ERR_DTYPE, "%s: dtype %s, expected u8", name, type_name(t.dtype));
    const int rc = check_paged(name, t, unit, align);
    if (rc) return rc;
    // no two elements in one place: each dim's stride past all that the dims of lesser strides reach
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (t.stride[order[j]] < t.stride[order[i]]) std::swap(order[i], order[j]);
    int64_t reach = t.shape[3];
    for (const int i : order) {
        if (t.shape[i] == 1) continue;
        if (t.stride[i] < reach)
            return api_fail(MOE_ERR_LAYOUT, "%s: stride[%d] = %lld: elements overlap", name, i, (long long)t.stride[i]);
        reach += (t.shape[i] - 1) * t.stride[i];
    }
    return MOE_OK;
}

static int check_mx(const moe_mx_cache *c, CacheParams &p) {
    int rc;
    if (!c) return api_fail(MOE_ERR_INVALID_ARG, "cache: descriptor is NULL");
    if (c->format != MOE_MX8 && c->format != MOE_MX4)
        return api_fail(MOE_ERR_INVALID_ARG, "cache: format %d (MX8 or MX4)", c->format);
    if (c->dtype != MOE_DT_BF16 && c->dtype != MOE_DT_F16)
        return api_fail(MOE_ERR_DTYPE, "cache: dtype %s (bf16 or f16)", type_name(c->dtype));
    if ((rc = check_bytes("cache k", c->k, 16, 16)) || (rc = check_bytes("cache v", c->v, 16, 16)) ||
        (rc = check_bytes("cache k_scale", c->k_scale, 1, 1)) || (rc = check_bytes("cache v_scale", c->v_scale, 1, 1)))
        return rc;
    const int64_t dim = c->format == MOE_MX8 ? c->k.shape[3] : 2 * c->k.shape[3];
    if (!dim_ok(dim) || dim % 32)
        return api_fail(MOE_ERR_SHAPE, "cache k: head width %lld (32, 64, 96, 128, 192 or 256)", (long long)dim);
    for (int i = 0; i < 4; ++i) {
        if (c->v.shape[i] != c->k.shape[i])
            return api_fail(MOE_ERR_SHAPE, "cache v: dim %d is %lld, k's is %lld", i, (long long)c->v.shape[i],
                            (long long)c->k.shape[i]);
        const long long want = i < 3 ? c->k.shape[i] : dim / 32;
        if (c->k_scale.shape[i] != want || c->v_scale.shape[i] != want)
            return api_fail(MOE_ERR_SHAPE, "cache %s: dim %d is %lld, expected %lld",
                            c->k_scale.shape[i] != want ? "k_scale" : "v_scale", i,
                            (long long)(c->k_scale.shape[i] != want ? c->k_scale.shape[i] : c->v_scale.shape[i]), want);
    }
    if ((rc = check_table(c->table, c->len, c->flags, c->k.shape[1], p))) return rc;
    p.k = {(const uint16_t *)c->k.data, c->k.stride[0], c->k.stride[1], c->k.stride[2]};
    p.v = {(const uint16_t *)c->v.data, c->v.stride[0], c->v.stride[1], c->v.stride[2]};
    p.ks = {(const uint8_t *)c->k_scale.data, c->k_scale.stride[0], c->k_scale.stride[1], c->k_scale.stride[2]};
    p.vs = {(const uint8_t *)c->v_scale.data, c->v_scale.stride[0], c->v_scale.stride[1], c->v_scale.stride[2]};
    p.pages = (int32_t)c->k.shape[0];
    p.page = (int32_t)c->k.shape[1];
    p.heads = (int32_t)c->k.shape[2];
    p.dim = (int32_t)dim;
    return MOE_OK;
}

extern "C" int moe_mx_cache_check(const moe_mx_cache *c) {
    api_clear();
    CacheParams p;
    memset(&p, 0, sizeof p);
    return check_mx(c, p);
}

// ------------------------------------------------------------------ norm, rotation, append

static int check_norm(const moe_head_norm *n, int32_t dim, AppendParams &a) {
    if (!n) return MOE_OK;
    const int size = n->dtype == MOE_DT_F32 ? 4 : 2;
    if (n->dtype != MOE_DT_F32 && n->dtype != MOE_DT_BF16 && n->dtype != MOE_DT_F16)
        return api_fail(MOE_ERR_DTYPE, "norm: dtype %s (f32, bf16 or f16)", type_name(n->dtype));
    int rc;
    if ((rc = check_words("norm q_weight", n->q_weight, size)) || (rc = check_words("norm k_weight", n->k_weight, size)))
        return rc;
    for (const int64_t s : {n->q_stride, n->k_stride})
        if (s && (s < dim || s >= (int64_t)1 << 40))
            return api_fail(MOE_ERR_LAYOUT, "norm: row stride %lld, heads of %d (0: one row for all)", (long long)s, dim);
    if (!(n->eps >= 0.0f) || !std::isfinite(n->eps))
        return api_fail(MOE_ERR_INVALID_ARG, "norm: eps %g (0 or more)", (double)n->eps);
    if (!std::isfinite(n->offset)) return api_fail(MOE_ERR_INVALID_ARG, "norm: offset is not finite");
    a.q_weight = n->q_weight;
    a.k_weight = n->k_weight;
    a.qw_stride = n->q_stride;
    a.kw_stride = n->k_stride;
    a.norm = n->dtype;
    a.eps = n->eps;
    a.offset = n->offset;
    return MOE_OK;
}

template <int MOST> static void (*append_kernel(bool f16, int format))(AppendParams) {
    return format == MX_NONE   ? (f16 ? moe_append_kernel<true, MX_NONE, MOST> : moe_append_kernel<false, MX_NONE, MOST>)
           : format == MX_E4M3 ? (f16 ? moe_append_kernel<true, MX_E4M3, MOST> : moe_append_kernel<false, MX_E4M3, MOST>)
                               : (f16 ? moe_append_kernel<true, MX_E2M1, MOST> : moe_append_kernel<false, MX_E2M1, MOST>);
}

static int run_append(bool f16, int format, const moe_head_norm *norm, const AppendCall &call, AppendParams &a, void *stream) {
    int rc, piece;
    if ((rc = check_norm(norm, a.r.c.dim, a)) || (rc = check_append(call, a.r, &piece))) return rc;
    a.half = call.rope->layout == MOE_ROPE_HALF;
    a.inv_dim = 1.0f / (float)a.r.c.dim;
    a.wide = ((((uintptr_t)call.q | (uintptr_t)call.k | (uintptr_t)call.v | (uintptr_t)call.q_out) & 15) |
              ((call.q_stride | call.k_stride | call.v_stride | call.q_out_stride) & 7)) == 0;
    const int64_t unit = a.norm == MOE_DT_F32 ? 3 : 7;      // elements in 16 bytes, but one
    a.wide_weights = ((((uintptr_t)a.q_weight | (uintptr_t)a.k_weight) & 15) | ((a.qw_stride | a.kw_stride) & unit)) == 0;
    for (a.lanes = 4; a.lanes * 8 < a.r.c.dim; a.lanes *= 2) {}
    // Few rows (one to a compute unit): as many threads as their heads take, whole waves, at least as many as pairs; more rows: 256
    // (the kernel of one row of 48 heads of 128: 4.2 us, 5.8 with 256 threads; the call of 2001 rows: 33.2 us with
    // 768, 17.6 with 256, when both were measured; 18.1 since).
    const int threads = ((call.q_heads + 2 * a.r.c.heads) * a.lanes + 63) & ~63;
    const bool few = call.rows <= COMPUTE_UNITS && threads > 256;
    const int block = !few ? 256 : threads < 1024 ? threads : 1024;
    void (*kern)(AppendParams) = few ? append_kernel<1024>(f16, format) : append_kernel<256>(f16, format);
    return launch("append", kern, dim3((unsigned)call.rows), dim3((unsigned)block), a, stream);
}

extern "C" int moe_norm_rope_append(const moe_paged_cache *c, const moe_head_norm *norm, const moe_rope *r, int32_t rows,
                                    const void *q, int64_t q_stride, int32_t q_heads, const void *k, int64_t k_stride,
                                    const void *v, int64_t v_stride, const int32_t *row_start, const int32_t *positions,
                                    void *q_out, int64_t q_out_stride, void *hip_stream) {
    api_clear();
    AppendParams a;
    memset(&a, 0, sizeof a);
    int rc;
    if ((rc = check_cache(c, a.r.c))) return rc;
    return run_append(c->k.dtype == MOE_DT_F16, MX_NONE, norm,
                      {r, rows, q, q_stride, q_heads, k, k_stride, v, v_stride, row_start, positions, q_out, q_out_stride}, a,
                      hip_stream);
}

extern "C" int moe_mx_append(const moe_mx_cache *c, const moe_head_norm *norm, const moe_rope *r, int32_t rows,
                             const void *q, int64_t q_stride, int32_t q_heads, const void *k, int64_t k_stride, const void *v,
                             int64_t v_stride, const int32_t *row_start, const int32_t *positions, void *q_out,
                             int64_t q_out_stride, void *hip_stream) {
    api_clear();
    AppendParams a;
    memset(&a, 0, sizeof a);
    int rc;
    if ((rc = check_mx(c, a.r.c))) return rc;
    return run_append(c->dtype == MOE_DT_F16, c->format, norm,
                      {r, rows, q, q_stride, q_heads, k, k_stride, v, v_stride, row_start, positions, q_out, q_out_stride}, a,
                      hip_stream);
}

// ------------------------------------------------------------------ reading back

extern "C" int moe_mx_read(const moe_mx_cache *c, int32_t rows, const int32_t *row_start, const int32_t *start, void *k_out,
                           int64_t k_stride, void *v_out, int64_t v_stride, void *hip_stream) {
    api_clear();
    ReadParams p;
    memset(&p, 0, sizeof p);
    int rc;
    if ((rc = check_mx(c, p.c)) || (rc = check_rows(rows, p.c.heads, p.c))) return rc;
    const int64_t w = (int64_t)p.c.heads * p.c.dim;
    if ((rc = check_matrix("k_out", k_out, k_stride, w, 16)) || (rc = check_matrix("v_out", v_out, v_stride, w, 16)) ||
        (rc = check_words("row_start", row_start)))
        return rc;
    if (start && (rc = check_words("start", start))) return rc;
    if (rows_overlap(k_out, k_stride, w, v_out, v_stride, w, rows))
        return api_fail(MOE_ERR_ALIAS, "k_out overlaps v_out");
    if ((rc = check_device())) return rc;
    p.row_start = row_start;
    p.start = start;
    p.k = (uint16_t *)k_out;
    p.v = (uint16_t *)v_out;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.rows = rows;
    const bool f16 = c->dtype == MOE_DT_F16;
    void (*kern)(ReadParams) = c->format == MX_E4M3 ? (f16 ? moe_read_kernel<true, MX_E4M3> : moe_read_kernel<false, MX_E4M3>)
                                                    : (f16 ? moe_read_kernel<true, MX_E2M1> : moe_read_kernel<false, MX_E2M1>);
    return launch("mx_read", kern, dim3((unsigned)rows), dim3(256), p, hip_stream);
}

extern "C" int moe_mx_keep(const moe_mx_cache *c, const int32_t *row_start, int32_t rows, const int32_t *n_keep,
                           const int32_t *path, int32_t *new_len, void *hip_stream) {
    api_clear();
    KeepParams p;
    memset(&p, 0, sizeof p);
    int rc;
    if ((rc = check_mx(c, p.c)) || (rc = check_keep(row_start, rows, n_keep, path, new_len, p))) return rc;
    void (*kern)(KeepParams) = c->format == MX_E4M3 ? moe_keep_kernel<MX_E4M3> : moe_keep_kernel<MX_E2M1>;
    return launch("mx_keep", kern, dim3((unsigned)p.c.seqs), dim3(256), p, hip_stream);
}

// ------------------------------------------------------------------ attention

static int64_t workspace_of(CacheParams &p, int32_t groups, int32_t rows, int32_t q_heads) {
    int rc;
    if ((rc = check_rows(rows, q_heads, p))) return -rc;
    if (groups < 0 || groups > p.seqs)
        return -api_fail(MOE_ERR_SHAPE, "shared: %d groups, %d sequences", groups, p.seqs);
    return attend_workspace(p, rows, q_heads, groups);
}

extern "C" int64_t moe_shared_attend_workspace(const moe_paged_cache *c, int32_t groups, int32_t rows, int32_t q_heads) {
    api_clear();
    CacheParams p;
    memset(&p, 0, sizeof p);
    const int rc = check_cache(c, p);
    return rc ? -rc : workspace_of(p, groups, rows, q_heads);
}

extern "C" int64_t moe_mx_attend_workspace(const moe_mx_cache *c, int32_t groups, int32_t rows, int32_t q_heads) {
    api_clear();
    CacheParams p;
    memset(&p, 0, sizeof p);
    const int rc = check_mx(c, p);
    return rc ? -rc : workspace_of(p, groups, rows, q_heads);
}

extern "C" int moe_shared_attend(const moe_paged_cache *c, const moe_shared_prefix *shared, int32_t rows, const void *q,
                                 int64_t q_stride, int32_t q_heads, const int32_t *row_start, const uint64_t *mask, float scale,
                                 void *out, int64_t out_stride, void *workspace, size_t workspace_bytes, void *hip_stream) {
    api_clear();
    AttendParams p;
    memset(&p, 0, sizeof p);
    int rc;
    if ((rc = check_cache(c, p.c))) return rc;
    if (!shared) return api_fail(MOE_ERR_INVALID_ARG, "shared: NULL");
    return attend_run({c->k.dtype == MOE_DT_F16, MX_NONE, shared, rows, q, q_stride, q_heads, row_start, mask, scale, out,
                       out_stride, workspace, workspace_bytes, hip_stream}, p);
}

extern "C" int moe_mx_attend(const moe_mx_cache *c, const moe_shared_prefix *shared, int32_t rows, const void *q,
                             int64_t q_stride, int32_t q_heads, const int32_t *row_start, const uint64_t *mask, float scale,
                             void *out, int64_t out_stride, void *workspace, size_t workspace_bytes, void *hip_stream) {
    api_clear();
    AttendParams p;
    memset(&p, 0, sizeof p);
    int rc;
    if ((rc = check_mx(c, p.c))) return rc;
    return attend_run({c->dtype == MOE_DT_F16, c->format, shared, rows, q, q_stride, q_heads, row_start, mask, scale, out,
                       out_stride, workspace, workspace_bytes, hip_stream}, p);
}

// ------------------------------------------------------------------ sampling

static int check_sample_sizes(int64_t rows, int64_t vocab) {
    if (rows < 1 || rows > 1 << 20) return api_fail(MOE_ERR_ROWS, "rows %lld outside 1..2^20", (long long)rows);
    if (vocab < 1 || vocab > MAX_VOCAB)
        return api_fail(MOE_ERR_SHAPE, "vocabulary %lld outside 1..2^20", (long long)vocab);
    return MOE_OK;
}

// Bytes of workspace; with a base and p, also its parts.
static int64_t sample_layout(int64_t rows, int64_t vocab, char *base, SampleParams *p) {
    const int64_t chunks = (vocab + SAMPLE_CHUNK - 1) / SAMPLE_CHUNK;
    const int64_t mass = rows * chunks * (int64_t)sizeof(SampleHead);
    const int64_t count = mass + rows * chunks * SAMPLE_CELLS * 8;
    const int64_t start = count + rows * chunks * SAMPLE_CELLS * 2;
    const int64_t list = start + rows * chunks * SAMPLE_CELLS * 2;
    if (p) {
        p->chunks = (int32_t)chunks;
        p->head = (SampleHead *)base;
        p->mass = (uint64_t *)(base + mass);
        p->count = (uint16_t *)(base + count);
        p->start = (uint16_t *)(base + start);
        p->list = (uint16_t *)(base + list);
    }
    return list + rows * chunks * SAMPLE_CHUNK * 2;
}

extern "C" int64_t moe_sample_workspace(int32_t rows, int32_t vocab) {
    api_clear();
    const int rc = check_sample_sizes(rows, vocab);
    return rc ? -rc : sample_layout(rows, vocab, nullptr, nullptr);
}

template <typename L> static int sample_launches(SampleParams &p, void *stream) {
    int rc;
    const unsigned y = (unsigned)(p.rows < 32768 ? p.rows : 32768);
    if ((rc = launch("sample", moe_sample_cells_kernel<L>, dim3((unsigned)p.chunks, y, ((unsigned)p.rows + y - 1) / y),
                     dim3(256), p, stream)))
        return rc;
    return launch("sample row", moe_sample_row_kernel<L>, dim3((unsigned)p.rows), dim3(1024), p, stream);
}

extern "C" int moe_sample(const moe_tensor *logits, const float *u, const float *temperature, const int32_t *top_k,
                          const float *top_p, const float *min_p, int32_t *tokens, float *logprobs, uint32_t *flags,
                          void *workspace, size_t workspace_bytes, void *hip_stream) {
    api_clear();
    int rc;
    if (!logits) return api_fail(MOE_ERR_INVALID_ARG, "logits: descriptor is NULL");
    if (!logits->data) return api_fail(MOE_ERR_MISSING_TENSOR, "logits: missing (data == NULL)");
    if (logits->dtype != MOE_DT_F32 && logits->dtype != MOE_DT_BF16 && logits->dtype != MOE_DT_F16)
        return api_fail(MOE_ERR_DTYPE, "logits: dtype %s (f32, bf16 or f16)", type_name(logits->dtype));
    if (logits->ndim != 2) return api_fail(MOE_ERR_LAYOUT, "logits: rank %d, expected 2", logits->ndim);
    const int64_t rows = logits->shape[0], vocab = logits->shape[1];
    if ((rc = check_sample_sizes(rows, vocab))) return rc;
    if ((vocab > 1 && logits->stride[1] != 1) || (rows > 1 && logits->stride[0] < vocab))
        return api_fail(MOE_ERR_LAYOUT, "logits: strides %lld, %lld (rows of contiguous logits)",
                        (long long)logits->stride[0], (long long)logits->stride[1]);
    if ((rc = check_words("logits", logits->data, logits->dtype == MOE_DT_F32 ? 4 : 2)) || (rc = check_words("u", u)) ||
        (rc = check_words("tokens", tokens)) || (rc = check_words("logprobs", logprobs)) || (rc = check_words("flags", flags)))
        return rc;
    if ((temperature && (rc = check_words("temperature", temperature))) || (top_k && (rc = check_words("top_k", top_k))) ||
        (top_p && (rc = check_words("top_p", top_p))) || (min_p && (rc = check_words("min_p", min_p))))
        return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, sample_layout(rows, vocab, nullptr, nullptr))) ||
        (rc = check_device()))
        return rc;
    SampleParams p;
    memset(&p, 0, sizeof p);
    p.logits = logits->data;
    p.stride = logits->stride[0];
    p.u = u;
    p.temperature = temperature;
    p.top_k = top_k;
    p.top_p = top_p;
    p.min_p = min_p;
    p.tokens = tokens;
    p.logprobs = logprobs;
    p.flags = flags;
    p.rows = (int32_t)rows;
    p.vocab = (int32_t)vocab;
    sample_layout(rows, vocab, (char *)workspace, &p);
    return logits->dtype == MOE_DT_F32    ? sample_launches<LogitF32>(p, hip_stream)
           : logits->dtype == MOE_DT_BF16 ? sample_launches<LogitBf16>(p, hip_stream)
                                          : sample_launches<LogitF16>(p, hip_stream);
}
