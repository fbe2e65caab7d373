// drafted_items.h -- device helpers of the drafted step's kernels (gfx950).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "drafted_plan.h"
#include "layer_items.h"   // number formats, vector types

namespace moe {

__device__ __forceinline__ void raise_flag(uint32_t *flags, uint32_t bit) {
    atomicOr(flags, bit);
}

__device__ __forceinline__ int lane_id() { return (int)(threadIdx.x & 63); }

// A value that is the same in every lane of the wave, moved to a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <bool F16> __device__ __forceinline__ float to_f32(uint32_t h) { return F16 ? h2f(h) : bf2f(h); }
template <bool F16> __device__ __forceinline__ uint16_t from_f32(float v) { return F16 ? f2h(v) : f2bf(v); }

// The sequence whose rows hold `row`, or -1: the last one that starts at or before it, if it also
// ends after it. Every lane of the wave calls it with the same row; the 64 lanes read starts that cut
// what is left into 64, so 64 sequences take one step and 2^16 take three.
__device__ __forceinline__ int seq_of_row(const int32_t *row_start, int seqs, int row, int *first) {
    int lo = 0, n = seqs + 1;          // the starts lo .. lo + n - 1 are left
    for (;;) {
        const int step = (n + 63) >> 6, at = lane_id() * step;
        const int s = at < n ? row_start[lo + at] : 0x7FFFFFFF;
        const int before = __popcll(__ballot(s <= row));      // ascending: these are the first lanes
        if (before == 0) return -1;
        const int skip = (before - 1) * step;
        lo += skip;
        n = min(step, n - skip);
        if (step == 1) break;
    }
    const int b = uniform(lo);
    if (b >= seqs) return -1;
    *first = uniform(row_start[b]);
    return *first >= 0 && row >= *first && row < row_start[b + 1] ? b : -1;
}

// Whether the starts cover the pass: from row 0 to its last. One thread of a launch calls it.
__device__ __forceinline__ void check_ends(const int32_t *row_start, int seqs, int rows, uint32_t *flags) {
    if (row_start[0] != 0 || row_start[seqs] != rows) raise_flag(flags, MOE_FLAG_ROWS);
}

// Rows of sequence b, bounded to the pass: [first, first + returned count).
__device__ __forceinline__ int seq_rows(const int32_t *row_start, int b, int rows, int *first, uint32_t *flags) {
    const int s = uniform(row_start[b]), e = uniform(row_start[b + 1]);
    if (s < 0 || e < s || e > rows) {
        if (lane_id() == 0) raise_flag(flags, MOE_FLAG_ROWS);
        *first = 0;
        return 0;
    }
    *first = s;
    return e - s;
}

// Page and slot of token t of sequence b: false (and a flag) where the cache has no such token.
__device__ __forceinline__ bool find_slot(const CacheParams &c, int b, int64_t t, int *page, int *slot) {
    bool ok = t >= 0 && t < c.cap;
    if (ok) {
        const int at = (int)t / c.page;
        *page = c.table[b * c.table_stride + at];
        *slot = (int)t - at * c.page;
        ok = *page >= 0 && *page < c.pages;
    }
    if (!ok) raise_flag(c.flags, MOE_FLAG_PAGE);
    return ok;
}

}  // namespace moe
