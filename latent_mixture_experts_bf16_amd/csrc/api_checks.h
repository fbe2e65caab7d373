// api_checks.h -- argument checks and launches that the host files of the C ABI share (drafted and serving operators).
// Refusals name the argument; nothing is enqueued after one.
#pragma once
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>

#include "drafted_plan.h"

namespace moe {

const char *type_name(int dt);

// MOE_OK where the current device is a gfx950. Asked of the runtime once per device.
int check_device();

// The cache's arguments; what the kernels take of them in p.
int check_cache(const moe_paged_cache *c, CacheParams &p);

// A tensor of keys, values, codes or scales: [pages][page][kv_heads][width], shapes positive, last dim contiguous, other
// strides multiples of `unit` elements without overlap, a page spanning less than 2^30 elements, the data aligned to `align`
// bytes.
int check_paged(const char *name, const moe_tensor &t, int unit, int align);

// The table and lengths of a cache whose k and page are checked, and its flags.
int check_table(const moe_tensor &table, const moe_tensor &len, uint32_t *flags, int64_t page, CacheParams &p);

bool dim_ok(int64_t d);

// Rows that are rotated and appended: their arguments, checked; what the kernels take of them in p, whose cache is there. *piece: elements
// that every row is aligned for and that divide the rotated part.
struct AppendCall {
    const moe_rope *rope;
    int32_t rows;
    const void *q;
    int64_t q_stride;
    int32_t q_heads;
    const void *k;
    int64_t k_stride;
    const void *v;
    int64_t v_stride;
    const int32_t *row_start, *positions;
    void *q_out;
    int64_t q_out_stride;
};
int check_append(const AppendCall &a, RopeParams &p, int *piece);

// The arguments of path keeping, whose cache is in p.
int check_keep(const int32_t *row_start, int32_t rows, const int32_t *n_keep, const int32_t *path, int32_t *new_len, KeepParams &p);

template <typename P>
static inline int launch(const char *what, void (*kernel)(P), dim3 grid, dim3 block, P p, void *stream) {
    void *args[] = {&p};
    const hipError_t e = hipLaunchKernel((const void *)kernel, grid, block, args, 0, (hipStream_t)stream);
    if (e != hipSuccess) return api_fail(MOE_ERR_HIP, "%s launch: %s", what, hipGetErrorString(e));
    return MOE_OK;
}

static inline int check_rows(int32_t rows, int32_t q_heads, const CacheParams &c) {
    if (rows < 1 || rows > 1 << 20) return api_fail(MOE_ERR_ROWS, "rows %d outside 1..2^20", rows);
    if (q_heads < 1 || q_heads > 1 << 16 || q_heads % c.heads)
        return api_fail(MOE_ERR_SHAPE, "q: %d heads (a multiple of the cache's %d)", q_heads, c.heads);
    return MOE_OK;
}

// A row matrix of 16-bit elements: `width` used of each `stride`.
static inline int check_matrix(const char *name, const void *p, int64_t stride, int64_t width, int align) {
    if (!p) return api_fail(MOE_ERR_INVALID_ARG, "%s: NULL", name);
    if (stride < width || stride >= (int64_t)1 << 40)
        return api_fail(MOE_ERR_LAYOUT, "%s: row stride %lld, %lld wide", name, (long long)stride, (long long)width);
    if ((uintptr_t)p % align || stride * 2 % align)
        return api_fail(MOE_ERR_LAYOUT, "%s: pointer and row stride must be %d-byte aligned", name, align);
    return MOE_OK;
}

static inline int check_words(const char *name, const void *p, int align = 4) {
    if (!p) return api_fail(MOE_ERR_INVALID_ARG, "%s: NULL", name);
    if ((uintptr_t)p % align) return api_fail(MOE_ERR_LAYOUT, "%s: not %d-byte aligned", name, align);
    return MOE_OK;
}

static inline int check_workspace(const void *p, size_t bytes, int64_t need) {
    if (need && !p) return api_fail(MOE_ERR_INVALID_ARG, "workspace: NULL");
    if ((uintptr_t)p & 15) return api_fail(MOE_ERR_LAYOUT, "workspace: not 16-byte aligned");
    if (bytes < (size_t)need)
        return api_fail(MOE_ERR_SHAPE, "workspace: %zu bytes, %lld needed", bytes, (long long)need);
    return MOE_OK;
}

static inline bool overlap(const void *a, int64_t abytes, const void *b, int64_t bbytes) {
    const char *x = (const char *)a, *y = (const char *)b;
    return x < y + bbytes && y < x + abytes;
}

// Whether two row matrices share an element: their ranges meet, and they are not different columns
// of the same rows (the parts of one projection's output).
static inline bool rows_overlap(const void *a, int64_t as, int64_t aw, const void *b, int64_t bs, int64_t bw, int64_t rows) {
    if (!overlap(a, ((rows - 1) * as + aw) * 2, b, ((rows - 1) * bs + bw) * 2)) return false;
    if (as != bs) return true;
    const int64_t d = ((const char *)b - (const char *)a) % (as * 2), at = d < 0 ? d + as * 2 : d;   // of b in a's rows
    return !(at >= aw * 2 && at + bw * 2 <= as * 2);
}

}  // namespace moe
