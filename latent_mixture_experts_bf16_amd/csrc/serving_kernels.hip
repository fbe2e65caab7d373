// serving_kernels.hip -- rows normed for each head, rotated and appended to a cache in 16 bits or in codes; codes read back
// (gfx950).
#include "drafted_items.h"
#include "mx_items.h"

namespace moe {

typedef float round_f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 round_bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 round_f16x2 __attribute__((ext_vector_type(2)));
// Two values rounded to the 16-bit type, to nearest even.
template <bool F16> __device__ __forceinline__ uint32_t round2(float a, float b) {
    const round_f32x2 v = {a, b};
    if constexpr (F16)
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, round_f16x2));
    else
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, round_bf16x2));
}

// A lane's value from a neighbour of its row of 16: by a data-parallel move.
template <int CTRL> __device__ __forceinline__ uint32_t from_lane(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
// The sum over `lanes` neighbours (4, 8, 16 or 32) in each of them: within a quad by exchanges, then mirrored halves of 8 and 16
// lanes, all lanes of a smaller group having the same by then.
__device__ __forceinline__ float sum_lanes(float v, int lanes) {
    v += __uint_as_float(from_lane<0xB1>(__float_as_uint(v)));
    v += __uint_as_float(from_lane<0x4E>(__float_as_uint(v)));
    if (lanes >= 8) v += __uint_as_float(from_lane<0x141>(__float_as_uint(v)));
    if (lanes >= 16) v += __uint_as_float(from_lane<0x140>(__float_as_uint(v)));
    if (lanes >= 32) v += __shfl_xor(v, 16);
    return v;
}

// Eight weights of a head's norm from element e on, of the type `dtype`; wide: 16-byte aligned.
__device__ __forceinline__ void norm_weights(const void *p, int dtype, bool wide, int64_t e, float *w) {
    if (dtype == MOE_DT_F32) {
        const float *f = (const float *)p + e;
        if (wide) {
            *(float4 *)w = *(const float4 *)f;
            *(float4 *)(w + 4) = *(const float4 *)(f + 4);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = f[i];
        }
        return;
    }
    uint16_t raw[8];
    const uint16_t *h = (const uint16_t *)p + e;
    if (wide) {
        *(uint4 *)raw = *(const uint4 *)h;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) raw[i] = h[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = dtype == MOE_DT_BF16 ? bf2f(raw[i]) : h2f(raw[i]);
}

// Eight dims of head `at` of a row, queries, keys and values in turn; zeros past the last one.
__device__ __forceinline__ uint4 load_head(const uint16_t *q, int64_t q_row, int q_heads, const uint16_t *k, int64_t k_row,
                                           const uint16_t *v, int64_t v_row, int kv_heads, int at, int dim, bool live, bool wide) {
    if (at >= q_heads + 2 * kv_heads || !live) return make_uint4(0, 0, 0, 0);
    const uint16_t *src = q + q_row + at * dim;
    if (at >= q_heads) src = k + k_row + (at - q_heads) * dim;
    if (at >= q_heads + kv_heads) src = v + v_row + (at - q_heads - kv_heads) * dim;
    if (wide) return *(const uint4 *)src;
    return make_uint4(src[0] | (uint32_t)src[1] << 16, src[2] | (uint32_t)src[3] << 16, src[4] | (uint32_t)src[5] << 16,
                      src[6] | (uint32_t)src[7] << 16);
}

// One workgroup per row. A head's eight dims lie in one lane, the head in `lanes` neighbours of a wave (a power of two, the last
// ones idle where the head is no power of two wide), so a head's mean square is a few cross-lane sums, a block of 32 codes
// four lanes, and a rotated pair one lane (interleaved) or two of the same head (half), which meet through LDS. The angle is
// formed in 64 bits; the part of its half turns that fp32 does not hold turns cosine and sine once more (first order, the rest is below
// 2^-50), so that what is left is their own rounding. One rounding at the end: to 16 bits, or to the codes.
//
// A pass's loads are on the way before the pass before it is computed, the first ones before the row's sequence, page and angles are
// found: what bounds a call of few rows is that chain of loads (the kernel of one row: 4.4 us). MOST threads: of few rows all heads at
// once (1024), of many 256, six of whose workgroups a compute unit holds (80 registers, and 24 bytes of scratch a lane in 16 bits,
// 40 and 48 to codes): vector instructions take 62 % of those' time (2001 rows of 56 heads of 128, 57 MB: 18 us, of which the floor
// of bytes is 12) and 57 % (2808 rows to 4-bit codes: 19 us), and the rows past the first 1536 wait for a place. Before sums went by
// data-parallel moves, roundings by pairs and the loads ahead, the former took 28.
template <bool F16, int FMT, int MOST> __global__ void __launch_bounds__(MOST, MOST > 256 ? 1 : 6) moe_append_kernel(AppendParams a) {
    __shared__ __align__(16) float2 cs[128];
    __shared__ __align__(16) float xs[MOST * 8];
    const RopeParams &p = a.r;
    const int row = (int)blockIdx.x, tid = (int)threadIdx.x;
    const int D = p.c.dim, lanes = a.lanes, pairs = p.pairs, rd = 2 * pairs;
    const int sub = tid & (lanes - 1), d0 = sub * 8;
    const bool live = d0 < D;
    float *const head_x = xs + (tid - sub) * 8;
    const int heads = p.q_heads + 2 * p.c.heads, step = (int)blockDim.x / lanes;

    const int64_t q_row = row * p.q_stride + d0, k_row = row * p.k_stride + d0, v_row = row * p.v_stride + d0;
    const int q_heads = p.q_heads, kv_heads = p.c.heads, wide = a.wide;
    const uint16_t *const qp = p.q, *const kp = p.kn, *const vp = p.vn;
    uint4 ahead = load_head(qp, q_row, q_heads, kp, k_row, vp, v_row, kv_heads, tid / lanes, D, live, wide);

    const int end = p.row_start[p.c.seqs];
    int first = 0;
    const int b = seq_of_row(p.row_start, p.c.seqs, row, &first);
    if (b < 0) {
        if (tid == 0) raise_flag(p.c.flags, MOE_FLAG_ROWS);
        return;
    }
    const int len = uniform(p.c.len[b]);
    const bool len_ok = len >= 0 && len <= p.c.cap;
    const int64_t token = (int64_t)len + (row - first);
    int page = 0, slot = 0;
    bool ok = len_ok && token < p.c.cap;     // a row after a negative length would fall on a cached token
    if (ok) {
        const int at = (int)token / p.c.page;
        page = uniform(p.c.table[b * p.c.table_stride + at]);
        slot = uniform((int)token - at * p.c.page);
        ok = page >= 0 && page < p.c.pages;
    }
    if (tid < pairs) {
        const int64_t pos = p.positions ? (int64_t)p.positions[row] : token;
        const double turns = (double)pos * p.freqs[tid] * 0.15915494309189533577;   // 1 / (2 pi)
        const double half_turns = 2.0 * (turns - rint(turns));
        const float t = (float)half_turns, rest = (float)(half_turns - (double)t) * 3.14159274f;
        const float c = cospif(t), s = sinpif(t);
        cs[tid] = make_float2(fmaf(-rest, s, c) * p.magnitude, fmaf(rest, c, s) * p.magnitude);
    }
    if (!ok && tid == 0) raise_flag(p.c.flags, len_ok ? MOE_FLAG_PAGE : MOE_FLAG_LEN);
    if (row == 0 && tid == 0 && end != p.rows) raise_flag(p.c.flags, MOE_FLAG_ROWS);
    __syncthreads();

    const int64_t k_at = page * p.c.k.page + slot * p.c.k.slot, v_at = page * p.c.v.page + slot * p.c.v.slot;
#pragma unroll 1
    for (int at = tid / lanes; at - tid / lanes < heads; at += step) {
        const bool any = at < heads && live, query = at < p.q_heads, value = at >= p.q_heads + p.c.heads;
        const int h = query ? at : value ? at - p.q_heads - p.c.heads : at - p.q_heads;
        float x[8];
        const uint32_t raw[4] = {ahead.x, ahead.y, ahead.z, ahead.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = to_f32<F16>(raw[e / 2] >> (e & 1) * 16 & 0xFFFFu);
        ahead = load_head(qp, q_row, q_heads, kp, k_row, vp, v_row, kv_heads, at + step, D, live, wide);
        if (a.norm) {
            float sum = 0.0f, w[8];
            if (any && !value)
                norm_weights(query ? a.q_weight : a.k_weight, a.norm, a.wide_weights, h * (query ? a.qw_stride : a.kw_stride) + d0, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
            sum = sum_lanes(sum, lanes);
            float mean = fmaf(sum, a.inv_dim, a.eps);
            if (!(mean > 0x1p-100f && mean < __builtin_inff())) {
                // squares that leave fp32 (of bf16 values past 2^60 or all below 2^-50): the head and the root of eps times a power of
                // two that brings them back, which the quotient does not see; the head's lanes all come here
                const float k = mean > 1.0f ? 0x1p-70f : 0x1p70f;
                sum = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] *= value ? 1.0f : k;
                    sum = fmaf(x[e], x[e], sum);
                }
                mean = fmaf(sum_lanes(sum, lanes), a.inv_dim, a.eps * k * k);
            }
            if (any && !value) {
                const float inv = mean == 0.0f ? 0.0f : rsqrtf(mean);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * (a.offset + w[e]);
            }
        }
        if (a.half) {
            // the other of each pair, through LDS; the lanes of a head are in one wave, whose LDS accesses keep their order
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            *(float4 *)(head_x + d0) = make_float4(x[0], x[1], x[2], x[3]);
            *(float4 *)(head_x + d0 + 4) = make_float4(x[4], x[5], x[6], x[7]);
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            if (!value && d0 < rd && (pairs & 3) == 0) {
                // four at a time: single ones would meet on an eighth of the banks
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const int d = d0 + e;
                    if (d >= rd) continue;
                    const bool second = d >= pairs;
                    const int j = second ? d - pairs : d;
                    const float4 t0 = *(const float4 *)(cs + j), t1 = *(const float4 *)(cs + j + 2);
                    const float4 y = *(const float4 *)(head_x + (second ? j : d + pairs));
                    const float s = second ? 1.0f : -1.0f;
                    x[e] = fmaf(x[e], t0.x, s * (y.x * t0.y));
                    x[e + 1] = fmaf(x[e + 1], t0.z, s * (y.y * t0.w));
                    x[e + 2] = fmaf(x[e + 2], t1.x, s * (y.z * t1.y));
                    x[e + 3] = fmaf(x[e + 3], t1.z, s * (y.w * t1.w));
                }
            } else if (!value && d0 < rd) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int d = d0 + e;
                    if (d >= rd) continue;
                    const bool second = d >= pairs;
                    const float2 t = cs[second ? d - pairs : d];
                    const float y = head_x[second ? d - pairs : d + pairs];
                    x[e] = fmaf(x[e], t.x, second ? y * t.y : -(y * t.y));
                }
            }
        } else if (!value && d0 < rd) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                if (d0 + e >= rd) continue;
                const float2 t = cs[(d0 + e) / 2];
                const float u = x[e], w = x[e + 1];
                x[e] = fmaf(u, t.x, -(w * t.y));
                x[e + 1] = fmaf(w, t.x, u * t.y);
            }
        }
        uint32_t scale = 0;
        if constexpr (FMT != MX_NONE) {
            // the largest magnitude of a block, as an integer: the order of numbers without a sign, NaN above infinity
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
            top = max(top, from_lane<0xB1>(top));
            top = max(top, from_lane<0x4E>(top));
            scale = mx_scale<F16, FMT>(__uint_as_float(top));
        }
        if (!any || (!query && !ok)) continue;
        if (FMT == MX_NONE || query) {
            const uint4 out = make_uint4(round2<F16>(x[0], x[1]), round2<F16>(x[2], x[3]), round2<F16>(x[4], x[5]), round2<F16>(x[6], x[7]));
            uint16_t *dst = p.qo + row * p.qo_stride + d0;
            int64_t head = D;
            if (!query) {
                dst = (uint16_t *)p.c.k.p + k_at + d0;
                head = p.c.k.head;
            }
            if (value) {
                dst = (uint16_t *)p.c.v.p + v_at + d0;
                head = p.c.v.head;
            }
            dst += h * head;
            if (!query || a.wide) {
                *(uint4 *)dst = out;
            } else {
                const uint32_t w[4] = {out.x, out.y, out.z, out.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) dst[e] = (uint16_t)(w[e / 2] >> (e & 1) * 16);
            }
        } else {
            uint8_t *dst = (uint8_t *)p.c.k.p + k_at + h * p.c.k.head;
            uint8_t *scales = (uint8_t *)p.c.ks.p + page * p.c.ks.page + slot * p.c.ks.slot + h * p.c.ks.head;
            if (value) {
                dst = (uint8_t *)p.c.v.p + v_at + h * p.c.v.head;
                scales = (uint8_t *)p.c.vs.p + page * p.c.vs.page + slot * p.c.vs.slot + h * p.c.vs.head;
            }
            if (scale == mx_last_scale<F16, FMT>()) {
                const float most = __uint_as_float(scale << 23) * (FMT == MX_E4M3 ? 448.0f : 6.0f);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = fminf(fmaxf(x[e], -most), most);
            }
            const uint2 codes = mx_codes<FMT>(x, scale);
            if (FMT == MX_E4M3)
                *(uint2 *)(dst + d0) = codes;
            else
                *(uint32_t *)(dst + d0 / 2) = codes.x;
            if ((sub & 3) == 0) scales[sub / 4] = (uint8_t)scale;
        }
    }
}

// One workgroup per row: 16 bytes of codes a thread and step. Bound by the workgroups' starts and their chain of loads (the row's
// sequence, its page, the codes): 2808 rows of 4-bit codes 8.4 us.
template <bool F16, int FMT> __global__ void __launch_bounds__(256) moe_read_kernel(ReadParams p) {
    constexpr int SPREAD = FMT == MX_E4M3 ? 2 : 4;
    const int row = (int)blockIdx.x, tid = (int)threadIdx.x;
    const int end = p.row_start[p.c.seqs];
    int first = 0;
    const int b = seq_of_row(p.row_start, p.c.seqs, row, &first);
    if (row == 0 && tid == 0 && end != p.rows) raise_flag(p.c.flags, MOE_FLAG_ROWS);
    if (b < 0) {
        if (tid == 0) raise_flag(p.c.flags, MOE_FLAG_ROWS);
        return;
    }
    const int from = p.start ? p.start[b] : p.c.len[b];
    const int64_t token = (int64_t)from + (row - first);
    int page = 0, slot = 0;
    bool ok = from >= 0 && token < p.c.cap;
    if (ok) {
        const int at = (int)token / p.c.page;
        page = p.c.table[b * p.c.table_stride + at];
        slot = (int)token - at * p.c.page;
        ok = page >= 0 && page < p.c.pages;
    }
    if (!ok) {
        if (tid == 0) raise_flag(p.c.flags, from < 0 || from > p.c.cap ? MOE_FLAG_LEN : MOE_FLAG_PAGE);
        return;
    }
    const int pieces = mx_row_bytes(FMT, p.c.dim) / 16, each = p.c.heads * pieces;
    for (int i = tid; i < 2 * each; i += 256) {
        const bool value = i >= each;
        const int j = value ? i - each : i, h = j / pieces, c = j - h * pieces;
        const KvView &kv = value ? p.c.v : p.c.k;
        const ScaleView &sv = value ? p.c.vs : p.c.ks;
        const u32x4 r = *(const u32x4 *)((const uint8_t *)kv.p + page * kv.page + slot * kv.slot + h * kv.head + c * 16);
        const uint32_t e = sv.p[page * sv.page + slot * sv.slot + h * sv.head + c * SPREAD / 4];
        u32x4 x[SPREAD];
        mx_expand<F16, FMT>(r, e, x);
        uint16_t *dst = (value ? p.v + row * p.v_stride : p.k + row * p.k_stride) + (int64_t)h * p.c.dim + c * SPREAD * 8;
#pragma unroll
        for (int s = 0; s < SPREAD; ++s) *(u32x4 *)(dst + s * 8) = x[s];
    }
}

template __global__ void moe_append_kernel<false, MX_NONE, 256>(AppendParams);
template __global__ void moe_append_kernel<false, MX_NONE, 1024>(AppendParams);
template __global__ void moe_append_kernel<true, MX_NONE, 256>(AppendParams);
template __global__ void moe_append_kernel<true, MX_NONE, 1024>(AppendParams);
template __global__ void moe_append_kernel<false, MX_E4M3, 256>(AppendParams);
template __global__ void moe_append_kernel<false, MX_E4M3, 1024>(AppendParams);
template __global__ void moe_append_kernel<true, MX_E4M3, 256>(AppendParams);
template __global__ void moe_append_kernel<true, MX_E4M3, 1024>(AppendParams);
template __global__ void moe_append_kernel<false, MX_E2M1, 256>(AppendParams);
template __global__ void moe_append_kernel<false, MX_E2M1, 1024>(AppendParams);
template __global__ void moe_append_kernel<true, MX_E2M1, 256>(AppendParams);
template __global__ void moe_append_kernel<true, MX_E2M1, 1024>(AppendParams);
template __global__ void moe_read_kernel<false, MX_E4M3>(ReadParams);
template __global__ void moe_read_kernel<true, MX_E4M3>(ReadParams);
template __global__ void moe_read_kernel<false, MX_E2M1>(ReadParams);
template __global__ void moe_read_kernel<true, MX_E2M1>(ReadParams);

}  // namespace moe
