// serving_kernels.hip -- rows normed for each head, rotated and appended to a cache in 16 bits or in codes; codes read back
// (gfx950).
#include "drafted_items.h"
#include "mx_items.h"

namespace moe {

// Weight e of a head's norm, of the type `dtype`.
__device__ __forceinline__ float norm_weight(const void *p, int dtype, int64_t e) {
    return dtype == MOE_DT_F32    ? ((const float *)p)[e]
           : dtype == MOE_DT_BF16 ? bf2f(((const uint16_t *)p)[e])
                                  : h2f(((const uint16_t *)p)[e]);
}

// One workgroup per row. A head's eight dims lie in one lane, the head in `lanes` neighbours of a wave (a power of two, the last
// ones idle where the head is no power of two wide), so a head's mean square is a few cross-lane sums, a block of 32 codes
// four lanes, and a rotated pair one lane (interleaved) or two of the same head (half), which meet through LDS. The angle is
// formed in 64 bits; the part of its half turns that fp32 does not hold turns cosine and sine once more (first order, the rest is below
// 2^-50), so that what is left is their own rounding. One rounding at the end: to 16 bits, or to the codes.
template <bool F16, int FMT> __global__ void __launch_bounds__(256) moe_append_kernel(AppendParams a) {
    __shared__ float2 cs[128];
    __shared__ __align__(16) float xs[256 * 8];
    const RopeParams &p = a.r;
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
        const double half_turns = 2.0 * (turns - rint(turns));
        const float t = (float)half_turns, rest = (float)(half_turns - (double)t) * 3.14159274f;
        const float c = cospif(t), s = sinpif(t);
        cs[tid] = make_float2(fmaf(-rest, s, c) * p.magnitude, fmaf(rest, c, s) * p.magnitude);
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
    if (row == 0 && tid == 0 && end != p.rows) raise_flag(p.c.flags, MOE_FLAG_ROWS);
    __syncthreads();

    const int D = p.c.dim, lanes = a.lanes, pairs = p.pairs, rd = 2 * pairs;
    const int sub = tid & (lanes - 1), d0 = sub * 8;
    const bool live = d0 < D;
    float *const head_x = xs + (tid - sub) * 8;
    const int heads = p.q_heads + 2 * p.c.heads, step = 256 / lanes;
    for (int at = tid / lanes; at - tid / lanes < heads; at += step) {
        // queries, keys, values in turn
        const bool any = at < heads && live, query = at < p.q_heads, value = at >= p.q_heads + p.c.heads;
        const int h = query ? at : value ? at - p.q_heads - p.c.heads : at - p.q_heads;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.0f;
        if (any) {
            const uint16_t *src = (query ? p.q + row * p.q_stride : value ? p.vn + row * p.v_stride : p.kn + row * p.k_stride) +
                                  (int64_t)h * D + d0;
            uint16_t raw[8];
            if (a.wide) {
                *(uint4 *)raw = *(const uint4 *)src;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) raw[e] = src[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = to_f32<F16>(raw[e]);
        }
        if (a.norm) {
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
            for (int d = 1; d < lanes; d <<= 1) sum += __shfl_xor(sum, d);
            if (any && !value) {
                const float mean = sum / (float)D + a.eps, inv = mean == 0.0f ? 0.0f : 1.0f / sqrtf(mean);
                const void *w = query ? a.q_weight : a.k_weight;
                const int64_t from = h * (query ? a.qw_stride : a.kw_stride) + d0;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * (a.offset + norm_weight(w, a.norm, from + e));
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
            if (!value && d0 < rd) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int d = d0 + e;
                    if (d >= rd) continue;
                    const bool second = d >= pairs;
                    const float2 t = cs[second ? d - pairs : d];
                    const float y = head_x[second ? d - pairs : d + pairs];
                    x[e] = second ? fmaf(x[e], t.x, y * t.y) : fmaf(x[e], t.x, -(y * t.y));
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
            top = max(top, (uint32_t)__shfl_xor((int)top, 1));
            top = max(top, (uint32_t)__shfl_xor((int)top, 2));
            scale = mx_scale<F16, FMT>(__uint_as_float(top));
        }
        if (!any || (!query && !ok)) continue;
        if (FMT == MX_NONE || query) {
            uint16_t out[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) out[e] = from_f32<F16>(x[e]);
            const KvView &kv = value ? p.c.v : p.c.k;
            uint16_t *dst = query ? p.qo + row * p.qo_stride + (int64_t)h * D + d0
                                  : (uint16_t *)kv.p + page * kv.page + slot * kv.slot + h * kv.head + d0;
            if (!query || a.wide) {
                *(uint4 *)dst = *(const uint4 *)out;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) dst[e] = out[e];
            }
        } else {
            const KvView &kv = value ? p.c.v : p.c.k;
            const ScaleView &sv = value ? p.c.vs : p.c.ks;
            uint8_t *dst = (uint8_t *)kv.p + page * kv.page + slot * kv.slot + h * kv.head;
            if (F16 && scale != 255) {
                const float most = __uint_as_float(scale << 23) * (FMT == MX_E4M3 ? 448.0f : 6.0f);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = fminf(fmaxf(x[e], -most), most);
            }
            const uint2 codes = mx_codes<FMT>(x, scale);
            if (FMT == MX_E4M3)
                *(uint2 *)(dst + d0) = codes;
            else
                *(uint32_t *)(dst + d0 / 2) = codes.x;
            if ((sub & 3) == 0)
                ((uint8_t *)sv.p)[page * sv.page + slot * sv.slot + h * sv.head + sub / 4] = (uint8_t)scale;
        }
    }
}

// One workgroup per row: 16 bytes of codes a thread and step.
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

template __global__ void moe_append_kernel<false, MX_NONE>(AppendParams);
template __global__ void moe_append_kernel<true, MX_NONE>(AppendParams);
template __global__ void moe_append_kernel<false, MX_E4M3>(AppendParams);
template __global__ void moe_append_kernel<true, MX_E4M3>(AppendParams);
template __global__ void moe_append_kernel<false, MX_E2M1>(AppendParams);
template __global__ void moe_append_kernel<true, MX_E2M1>(AppendParams);
template __global__ void moe_read_kernel<false, MX_E4M3>(ReadParams);
template __global__ void moe_read_kernel<true, MX_E4M3>(ReadParams);
template __global__ void moe_read_kernel<false, MX_E2M1>(ReadParams);
template __global__ void moe_read_kernel<true, MX_E2M1>(ReadParams);

}  // namespace moe
