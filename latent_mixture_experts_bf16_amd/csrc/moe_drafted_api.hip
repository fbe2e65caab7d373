// moe_drafted_api.hip -- host side of the C ABI declared in include/moe_drafted.h: argument
// checks, launch shapes, launches. Refusals name the argument; nothing is enqueued after one.
#include <hip/hip_runtime.h>

#include <atomic>

#include "api_checks.h"

namespace moe {
template <bool F16, bool HALF, int W> __global__ void moe_rope_kernel(RopeParams p);
template <typename L> __global__ void moe_verify_stats_kernel(VerifyParams p);
template <typename L> __global__ void moe_verify_walk_kernel(VerifyParams p);
template <typename L> __global__ void moe_verify_left_kernel(VerifyParams p);
struct LogitF32;
struct LogitBf16;
struct LogitF16;
template <int FMT> __global__ void moe_keep_kernel(KeepParams p);
}  // namespace moe

using namespace moe;

const char *moe::type_name(int dt) {
    switch (dt) {
    case MOE_DT_BF16: return "bf16";
    case MOE_DT_F16: return "f16";
    case MOE_DT_F32: return "f32";
    case MOE_DT_U32: return "u32";
    case MOE_DT_I32: return "i32";
    case MOE_DT_U8: return "u8";
    default: return "unknown";
    }
}

int moe::check_device() {
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

// ------------------------------------------------------------------ the cache

bool moe::dim_ok(int64_t d) {
    return d == 32 || d == 64 || d == 80 || d == 96 || d == 112 || d == 128 || d == 192 || d == 256;
}

int moe::check_paged(const char *name, const moe_tensor &t, int unit, int align) {
    if (t.ndim != 4)
        return api_fail(MOE_ERR_LAYOUT, "%s: rank %d, expected 4 ([pages][page][kv_heads][dim])", name, t.ndim);
    for (int i = 0; i < 4; ++i)
        if (t.shape[i] < 1) return api_fail(MOE_ERR_SHAPE, "%s: dim %d is %lld", name, i, (long long)t.shape[i]);
    if (t.shape[0] > 0x7FFFFFFF) return api_fail(MOE_ERR_SHAPE, "%s: %lld pages", name, (long long)t.shape[0]);
    if (t.shape[1] % 16 || t.shape[1] > 1 << 20)
        return api_fail(MOE_ERR_SHAPE, "%s: page of %lld tokens (a multiple of 16, at most 2^20)", name,
                        (long long)t.shape[1]);
    if (t.shape[2] > 1 << 16) return api_fail(MOE_ERR_SHAPE, "%s: %lld heads", name, (long long)t.shape[2]);
    if (t.stride[3] != 1 && t.shape[3] > 1) return api_fail(MOE_ERR_LAYOUT, "%s: last dim not contiguous", name);
    int64_t span = t.shape[3];
    for (int i = 0; i < 3; ++i) {
        if (t.stride[i] < 0 || t.stride[i] % unit)
            return api_fail(MOE_ERR_LAYOUT, "%s: stride[%d] = %lld (a multiple of %d, not negative)", name, i,
                            (long long)t.stride[i], unit);
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
    if ((uintptr_t)t.data % align) return api_fail(MOE_ERR_LAYOUT, "%s: data pointer not %d-byte aligned", name, align);
    return MOE_OK;
}

static int check_kv(const char *name, const moe_tensor &t) {
    if (!t.data) return api_fail(MOE_ERR_MISSING_TENSOR, "%s: missing (data == NULL)", name);
    if (t.dtype != MOE_DT_BF16 && t.dtype != MOE_DT_F16)
        return api_fail(MOE_ERR_DTYPE, "%s: dtype %s (bf16 or f16)", name, type_name(t.dtype));
    const int rc = check_paged(name, t, 8, 16);
    if (rc) return rc;
    if (!dim_ok(t.shape[3]))
        return api_fail(MOE_ERR_SHAPE, "%s: head width %lld (32, 64, 80, 96, 112, 128, 192 or 256)", name,
                        (long long)t.shape[3]);
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

int moe::check_table(const moe_tensor &table, const moe_tensor &len, uint32_t *flags, int64_t page, CacheParams &p) {
    int rc;
    if ((rc = check_i32("cache table", table, 2)) || (rc = check_i32("cache len", len, 1))) return rc;
    const int64_t seqs = table.shape[0];
    if (seqs > 1 << 16) return api_fail(MOE_ERR_SHAPE, "cache table: %lld sequences (at most 2^16)", (long long)seqs);
    if (table.shape[1] > 0x7FFFFFFF)
        return api_fail(MOE_ERR_SHAPE, "cache table: %lld pages a sequence", (long long)table.shape[1]);
    if (len.shape[0] != seqs)
        return api_fail(MOE_ERR_SHAPE, "cache len: %lld sequences, the table has %lld", (long long)len.shape[0],
                        (long long)seqs);
    if (seqs > 1 && table.stride[0] < 0)
        return api_fail(MOE_ERR_LAYOUT, "cache table: stride[0] = %lld", (long long)table.stride[0]);
    if (!flags) return api_fail(MOE_ERR_INVALID_ARG, "cache flags: NULL");
    if ((uintptr_t)flags & 3) return api_fail(MOE_ERR_LAYOUT, "cache flags: not 4-byte aligned");
    p.table = (const int32_t *)table.data;
    p.len = (const int32_t *)len.data;
    p.flags = flags;
    p.table_stride = table.stride[0];
    p.seqs = (int32_t)seqs;
    const int64_t cap = table.shape[1] * page, most = ((int64_t)1 << 31) - 64;
    p.cap = (int32_t)(cap < most ? cap : most);
    return MOE_OK;
}

int moe::check_cache(const moe_paged_cache *c, CacheParams &p) {
    int rc;
    if (!c) return api_fail(MOE_ERR_INVALID_ARG, "cache: descriptor is NULL");
    if ((rc = check_kv("cache k", c->k)) || (rc = check_kv("cache v", c->v))) return rc;
    if (c->k.dtype != c->v.dtype)
        return api_fail(MOE_ERR_DTYPE, "cache v: dtype %s, k is %s", type_name(c->v.dtype), type_name(c->k.dtype));
    for (int i = 0; i < 4; ++i)
        if (c->k.shape[i] != c->v.shape[i])
            return api_fail(MOE_ERR_SHAPE, "cache v: dim %d is %lld, k's is %lld", i, (long long)c->v.shape[i],
                            (long long)c->k.shape[i]);
    if ((rc = check_table(c->table, c->len, c->flags, c->k.shape[1], p))) return rc;
    p.k = {(const uint16_t *)c->k.data, c->k.stride[0], c->k.stride[1], c->k.stride[2]};
    p.v = {(const uint16_t *)c->v.data, c->v.stride[0], c->v.stride[1], c->v.stride[2]};
    p.pages = (int32_t)c->k.shape[0];
    p.page = (int32_t)c->k.shape[1];
    p.heads = (int32_t)c->k.shape[2];
    p.dim = (int32_t)c->k.shape[3];
    return MOE_OK;
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

int moe::check_append(const AppendCall &a, RopeParams &p, int *piece) {
    int rc;
    if ((rc = check_rows(a.rows, a.q_heads, p.c))) return rc;
    if (!a.rope) return api_fail(MOE_ERR_INVALID_ARG, "rope: NULL");
    if ((rc = check_words("rope freqs", a.rope->freqs, 8))) return rc;
    if (a.rope->pairs < 1 || a.rope->pairs > p.c.dim / 2)
        return api_fail(MOE_ERR_SHAPE, "rope: %d pairs, heads of %d", a.rope->pairs, p.c.dim);
    if (a.rope->layout != MOE_ROPE_HALF && a.rope->layout != MOE_ROPE_INTERLEAVED)
        return api_fail(MOE_ERR_INVALID_ARG, "rope: layout %d", a.rope->layout);
    if (!std::isfinite(a.rope->magnitude)) return api_fail(MOE_ERR_INVALID_ARG, "rope: magnitude is not finite");
    const int64_t qw = (int64_t)a.q_heads * p.c.dim, kw = (int64_t)p.c.heads * p.c.dim;
    if ((rc = check_matrix("q", a.q, a.q_stride, qw, 2)) || (rc = check_matrix("k", a.k, a.k_stride, kw, 2)) ||
        (rc = check_matrix("v", a.v, a.v_stride, kw, 2)) || (rc = check_matrix("q_out", a.q_out, a.q_out_stride, qw, 2)) ||
        (rc = check_words("row_start", a.row_start)))
        return rc;
    if (a.positions && (rc = check_words("positions", a.positions))) return rc;
    if (rows_overlap(a.q_out, a.q_out_stride, qw, a.q, a.q_stride, qw, a.rows) &&
        !(a.q_out == a.q && a.q_out_stride == a.q_stride))
        return api_fail(MOE_ERR_ALIAS, "q_out partially overlaps q");
    if (rows_overlap(a.q_out, a.q_out_stride, qw, a.k, a.k_stride, kw, a.rows) ||
        rows_overlap(a.q_out, a.q_out_stride, qw, a.v, a.v_stride, kw, a.rows))
        return api_fail(MOE_ERR_ALIAS, "q_out overlaps k or v");
    // the widest piece that divides the rotated part and that every row is aligned for
    const bool half = a.rope->layout == MOE_ROPE_HALF;
    const uint64_t odd = (uint64_t)(half ? a.rope->pairs : 2 * a.rope->pairs) | (uint64_t)a.q_stride |
                         (uint64_t)a.k_stride | (uint64_t)a.v_stride | (uint64_t)a.q_out_stride |
                         (((uintptr_t)a.q | (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)a.q_out) >> 1);
    const int w = odd % 8 == 0 ? 8 : odd % 4 == 0 ? 4 : odd % 2 == 0 ? 2 : 1;
    if (w == 1 && !half)
        return api_fail(MOE_ERR_LAYOUT, "interleaved pairs need rows aligned to 4 bytes");
    *piece = w;
    if ((rc = check_device())) return rc;
    p.freqs = a.rope->freqs;
    p.pairs = a.rope->pairs;
    p.magnitude = a.rope->magnitude;
    p.q = (const uint16_t *)a.q;
    p.kn = (const uint16_t *)a.k;
    p.vn = (const uint16_t *)a.v;
    p.qo = (uint16_t *)a.q_out;
    p.q_stride = a.q_stride;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.qo_stride = a.q_out_stride;
    p.row_start = a.row_start;
    p.positions = a.positions;
    p.rows = a.rows;
    p.q_heads = a.q_heads;
    return MOE_OK;
}

extern "C" int moe_rope_append(const moe_paged_cache *c, const moe_rope *r, int32_t rows, const void *q,
                               int64_t q_stride, int32_t q_heads, const void *k, int64_t k_stride, const void *v,
                               int64_t v_stride, const int32_t *row_start, const int32_t *positions, void *q_out,
                               int64_t q_out_stride, void *hip_stream) {
    api_clear();
    RopeParams p;
    memset(&p, 0, sizeof p);
    int rc, w;
    if ((rc = check_cache(c, p.c)) ||
        (rc = check_append({r, rows, q, q_stride, q_heads, k, k_stride, v, v_stride, row_start, positions, q_out,
                            q_out_stride}, p, &w)))
        return rc;
    const bool half = r->layout == MOE_ROPE_HALF, f16 = c->k.dtype == MOE_DT_F16;
    void (*kern)(RopeParams) = f16 ? (half ? rope_kernel<true, true>(w) : rope_kernel<true, false>(w))
                                   : (half ? rope_kernel<false, true>(w) : rope_kernel<false, false>(w));
    return launch("rope_append", kern, dim3((unsigned)rows), dim3(256), p, hip_stream);
}

// ------------------------------------------------------------------ tree attention

extern "C" int64_t moe_tree_attend_workspace(const moe_paged_cache *c, int32_t rows, int32_t q_heads) {
    api_clear();
    CacheParams p;
    int rc;
    if ((rc = check_cache(c, p)) || (rc = check_rows(rows, q_heads, p))) return -rc;
    return attend_workspace(p, rows, q_heads, 0);
}

extern "C" int moe_tree_attend(const moe_paged_cache *c, int32_t rows, const void *q, int64_t q_stride,
                               int32_t q_heads, const int32_t *row_start, const uint64_t *mask, float scale,
                               void *out, int64_t out_stride, void *workspace, size_t workspace_bytes,
                               void *hip_stream) {
    api_clear();
    AttendParams p;
    memset(&p, 0, sizeof p);
    int rc;
    if ((rc = check_cache(c, p.c))) return rc;
    return attend_run({c->k.dtype == MOE_DT_F16, MX_NONE, nullptr, rows, q, q_stride, q_heads, row_start, mask, scale, out,
                       out_stride, workspace, workspace_bytes, hip_stream}, p);
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

int moe::check_keep(const int32_t *row_start, int32_t rows, const int32_t *n_keep, const int32_t *path, int32_t *new_len,
                    KeepParams &p) {
    int rc;
    if ((rc = check_rows(rows, p.c.heads, p.c))) return rc;
    if ((rc = check_words("row_start", row_start)) || (rc = check_words("n_keep", n_keep)) ||
        (rc = check_words("path", path)) || (rc = check_words("new_len", new_len)))
        return rc;
    if ((rc = check_device())) return rc;
    p.row_start = row_start;
    p.n_keep = n_keep;
    p.path = path;
    p.new_len = new_len;
    p.rows = rows;
    return MOE_OK;
}

extern "C" int moe_path_keep(const moe_paged_cache *c, const int32_t *row_start, int32_t rows, const int32_t *n_keep,
                             const int32_t *path, int32_t *new_len, void *hip_stream) {
    api_clear();
    KeepParams p;
    memset(&p, 0, sizeof p);
    int rc;
    if ((rc = check_cache(c, p.c)) || (rc = check_keep(row_start, rows, n_keep, path, new_len, p))) return rc;
    return launch("path_keep", moe_keep_kernel<MX_NONE>, dim3((unsigned)p.c.seqs), dim3(256), p, hip_stream);
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
    return api_fail(MOE_ERR_DEVICE_CHECK, "met on the device:%s%s%s%s%s%s%s",
                    v & MOE_FLAG_PAGE ? " a page outside the cache or past the table;" : "",
                    v & MOE_FLAG_LEN ? " a length outside the table;" : "",
                    v & MOE_FLAG_ROWS ? " row_start not ascending over the rows;" : "",
                    v & MOE_FLAG_PATH ? " a path that is not ascending rows of its sequence;" : "",
                    v & MOE_FLAG_TOKEN ? " a drafted token outside the vocabulary;" : "",
                    v & MOE_FLAG_LOGITS ? " logits without a value above -infinity;" : "",
                    v & MOE_FLAG_GROUPS ? " group_start not ascending over the sequences;" : "");
}
