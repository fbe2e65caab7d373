// drafted_kernels.hip -- rotary append and path keeping (gfx950).
#include <type_traits>

#include "drafted_items.h"

namespace moe {

// ------------------------------------------------------------------ rotary append

// Elements of a row that one thread moves at a time, as one load.
template <int W> struct Vec;
template <> struct Vec<8> { typedef uint4 T; };
template <> struct Vec<4> { typedef uint2 T; };
template <> struct Vec<2> { typedef uint32_t T; };
template <> struct Vec<1> { typedef uint16_t T; };

template <int W> union Piece {
    typename Vec<W>::T v;
    uint16_t e[W];
};

template <int W> __device__ __forceinline__ Piece<W> load_piece(const uint16_t *p) {
    Piece<W> r;
    r.v = *(const typename Vec<W>::T *)p;
    return r;
}
template <int W> __device__ __forceinline__ void store_piece(uint16_t *p, const Piece<W> &r) {
    *(typename Vec<W>::T *)p = r.v;
}

// One workgroup per row. Cosine and sine of the row's angles, one pair a thread, go through LDS:
// the angle in turns is formed in 64 bits and its fraction alone rounded to 32, which leaves
// 2 pi 2^-25 of error in the angle at any position. Then each thread takes pieces of W elements of
// the heads (queries, keys, values in turn): half layout, a piece and its partner rotary / 2 on;
// interleaved, W / 2 whole pairs; the dims after the rotated ones and the values are copied.
// Products and their sum in fp32 without fusing, rounded once to the type. Bound by bandwidth: 4096 rows of 32 + 16
// heads of 128 (101 MB) take 19 us, 5.3 TB/s; one row takes 5 us, a launch and a chain of loads.
template <bool F16, bool HALF, int W>
__global__ void __launch_bounds__(256) moe_rope_kernel(RopeParams p) {
    __shared__ float2 cs[128];
    const int row = (int)blockIdx.x, tid = (int)threadIdx.x;
    const int end = p.row_start[p.c.seqs];
    int first = 0;
    const int b = seq_of_row(p.row_start, p.c.seqs, row, &first);
    if (b < 0) {
        if (tid == 0) raise_flag(p.c.flags, MOE_FLAG_ROWS);
        return;
    }
    const int len = p.c.len[b];
    const bool len_ok = len >= 0 && len <= p.c.cap;
    const int64_t token = (int64_t)len + (row - first);
    if (tid < p.pairs) {
        const int64_t pos = p.positions ? (int64_t)p.positions[row] : token;
        const double turns = (double)pos * p.freqs[tid] * 0.15915494309189533577;   // 1 / (2 pi)
        const float t = (float)(2.0 * (turns - rint(turns)));
        cs[tid] = make_float2(cospif(t) * p.magnitude, sinpif(t) * p.magnitude);
    }
    int page = 0, slot = 0;
    bool ok = len_ok && token < p.c.cap;     // a row after a negative length would fall on a cached token
    if (ok) {
        const int at = (int)token / p.c.page;
        page = p.c.table[b * p.c.table_stride + at];
        slot = (int)token - at * p.c.page;
        ok = page >= 0 && page < p.c.pages;
    }
    if (!ok && tid == 0) raise_flag(p.c.flags, len_ok ? MOE_FLAG_PAGE : MOE_FLAG_LEN);
    // rows before the first start or past the last are met above; here a sequence that goes on past the pass
    if (row == 0 && tid == 0 && end != p.rows) raise_flag(p.c.flags, MOE_FLAG_ROWS);
    __syncthreads();

    const int D = p.c.dim, rd = 2 * p.pairs;
    const int turned = HALF ? p.pairs / W : rd / W;   // pieces of a head that turn
    const int pieces = turned + (D - rd) / W;
    const int all = (p.q_heads + 2 * p.c.heads) * pieces;
    for (int i = tid; i < all; i += 256) {
        int h = i / pieces;
        const int u = i - h * pieces;
        const uint16_t *src;
        uint16_t *dst;
        bool value = false;
        if (h < p.q_heads) {
            src = p.q + row * p.q_stride + (int64_t)h * D;
            dst = p.qo + row * p.qo_stride + (int64_t)h * D;
        } else {
            if (!ok) break;
            h -= p.q_heads;
            value = h >= p.c.heads;
            if (value) h -= p.c.heads;
            const KvView &kv = value ? p.c.v : p.c.k;
            src = (value ? p.vn + row * p.v_stride : p.kn + row * p.k_stride) + (int64_t)h * D;
            dst = (uint16_t *)kv.p + page * kv.page + slot * kv.slot + h * kv.head;
        }
        if (u >= turned) {
            const int d = rd + (u - turned) * W;
            store_piece<W>(dst + d, load_piece<W>(src + d));
            continue;
        }
        if (HALF) {
            const int j = u * W;
            Piece<W> a = load_piece<W>(src + j), c = load_piece<W>(src + j + p.pairs);
            if (!value) {
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    const float x = to_f32<F16>(a.e[e]), y = to_f32<F16>(c.e[e]);
                    const float2 t = cs[j + e];
                    a.e[e] = from_f32<F16>(x * t.x - y * t.y);
                    c.e[e] = from_f32<F16>(x * t.y + y * t.x);
                }
            }
            store_piece<W>(dst + j, a);
            store_piece<W>(dst + j + p.pairs, c);
        } else {
            Piece<W> a = load_piece<W>(src + u * W);
            if (!value) {
#pragma unroll
                for (int e = 0; e + 1 < W; e += 2) {
                    const float x = to_f32<F16>(a.e[e]), y = to_f32<F16>(a.e[e + 1]);
                    const float2 t = cs[(u * W + e) / 2];
                    a.e[e] = from_f32<F16>(x * t.x - y * t.y);
                    a.e[e + 1] = from_f32<F16>(x * t.y + y * t.x);
                }
            }
            store_piece<W>(dst + u * W, a);
        }
    }
}

#define ROPE_KERNELS(F16)                                              \
    template __global__ void moe_rope_kernel<F16, true, 8>(RopeParams);  \
    template __global__ void moe_rope_kernel<F16, true, 4>(RopeParams);  \
    template __global__ void moe_rope_kernel<F16, true, 2>(RopeParams);  \
    template __global__ void moe_rope_kernel<F16, true, 1>(RopeParams);  \
    template __global__ void moe_rope_kernel<F16, false, 8>(RopeParams); \
    template __global__ void moe_rope_kernel<F16, false, 4>(RopeParams); \
    template __global__ void moe_rope_kernel<F16, false, 2>(RopeParams)
ROPE_KERNELS(false);
ROPE_KERNELS(true);
// (interleaved pairs need two elements at least: 2-byte alignment is refused on the host)

// ------------------------------------------------------------------ path keeping

// One workgroup per sequence. The path is checked, and the slots that its rows come from and go to are looked up, before
// the first one moves: a path out of order, or a page that the cache does not have, moves nothing. Row i of the path comes
// from a row at or after i (paths ascend), so with each thread owning the same 16 bytes of every row, and loading KEEP_STEP
// rows before it stores them, nothing is overwritten before it is read: every source of a later step lies after the
// places of the earlier ones. Bound by a launch and three loads one after another (path, page, rows): 64 paths of up to
// 24 rows take 5.5 us as a pass among others (7.2 where every thread looks the slots up for itself at each step), one 5.3.
constexpr int KEEP_STEP = 8, KEEP_CHUNK = 256;

// A cache of codes (FMT) has strides in bytes, and its blocks' scales move with them.
template <int FMT> __global__ void __launch_bounds__(KEEP_CHUNK) moe_keep_kernel(KeepParams p) {
    typedef typename std::conditional<FMT == MX_NONE, uint16_t, uint8_t>::type T;
    constexpr int PIECE = 16 / (int)sizeof(T);
    __shared__ int4 moves[KEEP_CHUNK];    // of a chunk of the path: page and slot from, page and slot to; page -1: it stays
    const int b = (int)blockIdx.x, tid = (int)threadIdx.x;
    if (b == 0 && tid == 64) check_ends(p.row_start, p.c.seqs, p.rows, p.c.flags);
    int first = 0;
    const int n = seq_rows(p.row_start, b, p.rows, &first, p.c.flags);
    const int len = p.c.len[b], keep = p.n_keep[b];
    const int32_t *path = p.path + first;
    auto look_up = [&](int i) {
        int4 m = make_int4(-1, 0, 0, 0);
        const int s = path[i];
        const bool ok = s == i || (find_slot(p.c, b, (int64_t)len + s, &m.x, &m.y) &&
                                   find_slot(p.c, b, (int64_t)len + i, &m.z, &m.w));
        moves[tid] = m;
        return ok;
    };
    const bool bad_len = len < 0 || (int64_t)len + keep > p.c.cap;
    bool bad_path = keep < 0 || keep > n, bad_page = false;
    // the first chunk last, whose slots are then in LDS
    for (int i = bad_path ? -1 : ((keep - 1) & ~(KEEP_CHUNK - 1)) + tid; i >= 0; i -= KEEP_CHUNK) {
        if (i >= keep) continue;
        const int s = path[i], prev = i ? path[i - 1] : -1;
        if (s <= prev || s >= n) bad_path = true;
        else if (!bad_len && !look_up(i)) bad_page = true;
    }
    if (bad_path) raise_flag(p.c.flags, MOE_FLAG_PATH);
    const bool bad = __syncthreads_or(bad_path || bad_page) != 0;
    if (bad || bad_len) {
        if (tid == 0) {
            if (!bad) raise_flag(p.c.flags, MOE_FLAG_LEN);
            p.new_len[b] = len;
        }
        return;
    }
    const int per = mx_row_bytes(FMT, p.c.dim) / 16, heads = p.c.heads;
    for (int c0 = 0; c0 < keep; c0 += KEEP_CHUNK) {
        const int here = min(KEEP_CHUNK, keep - c0);
        if (c0) {
            __syncthreads();
            if (tid < here) look_up(c0 + tid);
            __syncthreads();
        }
        for (int u = tid; u < 2 * heads * per; u += KEEP_CHUNK) {
            const bool value = u >= heads * per;
            const int w = value ? u - heads * per : u;
            const int h = w / per, d = (w - h * per) * PIECE;
            const KvView &kv = value ? p.c.v : p.c.k;
            T *base = (T *)kv.p + h * kv.head + d;
            for (int i0 = 0; i0 < here; i0 += KEEP_STEP) {
                uint4 x[KEEP_STEP];
                int64_t to[KEEP_STEP];
#pragma unroll
                for (int k = 0; k < KEEP_STEP; ++k) {
                    const int4 m = moves[min(i0 + k, here - 1)];
                    to[k] = -1;
                    if (i0 + k >= here || m.x < 0) continue;
                    x[k] = *(const uint4 *)(base + m.x * kv.page + m.y * kv.slot);
                    to[k] = m.z * kv.page + m.w * kv.slot;
                }
#pragma unroll
                for (int k = 0; k < KEEP_STEP; ++k)
                    if (to[k] >= 0) *(uint4 *)(base + to[k]) = x[k];
            }
        }
        if (FMT != MX_NONE) {
            const int blocks = p.c.dim / 32;
            for (int u = tid; u < 2 * heads * blocks; u += KEEP_CHUNK) {
                const bool value = u >= heads * blocks;
                const int w = value ? u - heads * blocks : u, h = w / blocks;
                const ScaleView &sv = value ? p.c.vs : p.c.ks;
                uint8_t *base = (uint8_t *)sv.p + h * sv.head + (w - h * blocks);
                for (int i = 0; i < here; ++i) {
                    const int4 m = moves[i];
                    if (m.x >= 0) base[m.z * sv.page + m.w * sv.slot] = base[m.x * sv.page + m.y * sv.slot];
                }
            }
        }
    }
    // every thread read the length before the barrier above, so the cache's own may be written
    if (tid == 0) p.new_len[b] = len + keep;
}
template __global__ void moe_keep_kernel<MX_NONE>(KeepParams);
template __global__ void moe_keep_kernel<MX_E4M3>(KeepParams);
template __global__ void moe_keep_kernel<MX_E2M1>(KeepParams);

}  // namespace moe
