// attend_kernels.hip -- attention of a drafted step's rows over the paged cache (gfx950).
#include "drafted_items.h"

namespace moe {

constexpr int ATTEND_WAVES = 4;

// One workgroup per row and query head: each wave takes every fourth token, its lanes the dims (up
// to four each); scores, the running maximum and sum of the softmax and the weighted values in fp32,
// the four waves joined through LDS.
template <bool F16>
__global__ void __launch_bounds__(256) moe_attend_kernel(AttendParams p) {
    __shared__ float so[ATTEND_WAVES][256], sm[ATTEND_WAVES], sl[ATTEND_WAVES];
    const int row = (int)blockIdx.x, head = (int)blockIdx.y, lane = lane_id(), wave = uniform((int)threadIdx.x >> 6);
    int first = 0;
    const int b = seq_of_row(p.row_start, p.c.seqs, row, &first);
    if (b < 0) {
        if (threadIdx.x == 0) raise_flag(p.c.flags, MOE_FLAG_ROWS);
        return;
    }
    int f2 = 0;
    const int n = seq_rows(p.row_start, b, p.rows, &f2, p.c.flags);
    const int len = seq_len(p.c, b), i = row - first, D = p.c.dim, kvh = head / p.group;
    int64_t end = (int64_t)len + n;
    if (end > p.c.cap) {
        if (threadIdx.x == 0) raise_flag(p.c.flags, MOE_FLAG_PAGE);
        end = p.c.cap;
    }
    const uint64_t mask = p.mask ? p.mask[row] : 0;
    float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -__builtin_inff(), l = 0.0f;
    for (int e = 0; e < 4; ++e) {
        const int d = lane + 64 * e;
        q[e] = d < D ? to_f32<F16>(p.q[row * p.q_stride + (int64_t)head * D + d]) : 0.0f;
    }
    for (int t = wave; t < end; t += ATTEND_WAVES) {
        const int j = t - len;
        if (j >= 0 && !(p.mask ? j < 64 && (mask >> j & 1) : j <= i)) continue;
        const int at = t / p.c.page, page = p.c.table[b * p.c.table_stride + at], slot = t - at * p.c.page;
        if (page < 0 || page >= p.c.pages) {
            if (lane == 0) raise_flag(p.c.flags, MOE_FLAG_PAGE);
            continue;
        }
        const uint16_t *k = p.c.k.p + page * p.c.k.page + slot * p.c.k.slot + kvh * p.c.k.head;
        const uint16_t *v = p.c.v.p + page * p.c.v.page + slot * p.c.v.slot + kvh * p.c.v.head;
        float s = 0.0f;
        for (int e = 0; e < 4; ++e)
            if (lane + 64 * e < D) s = fmaf(q[e], to_f32<F16>(k[lane + 64 * e]), s);
        for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
        s *= p.scale_log2;
        const float m2 = fmaxf(m, s), base = m2 == -__builtin_inff() ? 0.0f : m2;
        const float old = exp2f(m - base), w = exp2f(s - base);
        l = l * old + w;
        for (int e = 0; e < 4; ++e)
            if (lane + 64 * e < D) o[e] = fmaf(w, to_f32<F16>(v[lane + 64 * e]), o[e] * old);
        m = m2;
    }
    for (int e = 0; e < 4; ++e) so[wave][lane + 64 * e] = o[e];
    if (lane == 0) { sm[wave] = m; sl[wave] = l; }
    __syncthreads();
    const int d = (int)threadIdx.x;
    if (d >= D) return;
    float M = sm[0];
    for (int w = 1; w < ATTEND_WAVES; ++w) M = fmaxf(M, sm[w]);
    if (M == -__builtin_inff()) M = 0.0f;
    float O = 0.0f, S = 0.0f;
    for (int w = 0; w < ATTEND_WAVES; ++w) {
        const float f = exp2f(sm[w] - M);
        O += so[w][d] * f;
        S += sl[w] * f;
    }
    p.out[row * p.out_stride + (int64_t)head * D + d] = from_f32<F16>(S == 0.0f ? 0.0f : O / S);
}
template __global__ void moe_attend_kernel<false>(AttendParams);
template __global__ void moe_attend_kernel<true>(AttendParams);

}  // namespace moe
