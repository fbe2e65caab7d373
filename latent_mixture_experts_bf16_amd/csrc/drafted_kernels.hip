// drafted_kernels.hip -- rotary append, draft verification and path keeping (gfx950).
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
// Products and their sum in fp32 without fusing, rounded once to the type.
template <bool F16, bool HALF, int W>
__global__ void __launch_bounds__(256) moe_rope_kernel(RopeParams p) {
    __shared__ float2 cs[128];
    const int row = (int)blockIdx.x, tid = (int)threadIdx.x;
    int first = 0;
    const int b = seq_of_row(p.row_start, p.c.seqs, row, &first);
    if (b < 0) {
        if (tid == 0) raise_flag(p.c.flags, MOE_FLAG_ROWS);
        return;
    }
    const int64_t token = (int64_t)p.c.len[b] + (row - first);
    if (tid < p.pairs) {
        const int64_t pos = p.positions ? (int64_t)p.positions[row] : token;
        const double turns = (double)pos * p.freqs[tid] * 0.15915494309189533577;   // 1 / (2 pi)
        const float t = (float)(2.0 * (turns - rint(turns)));
        cs[tid] = make_float2(cospif(t) * p.magnitude, sinpif(t) * p.magnitude);
    }
    int page = 0, slot = 0;
    bool ok = token >= 0 && token < p.c.cap;
    if (ok) {
        const int at = (int)token / p.c.page;
        page = p.c.table[b * p.c.table_stride + at];
        slot = (int)token - at * p.c.page;
        ok = page >= 0 && page < p.c.pages;
    }
    if (!ok && tid == 0) raise_flag(p.c.flags, MOE_FLAG_PAGE);
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

// One workgroup per sequence. Row i of the path comes from a row at or after i (paths ascend), so
// with each thread owning the same 16 bytes of every row, and loading KEEP_STEP rows before it
// stores them, nothing is overwritten before it is read: every source of a later step lies
// after the places of the earlier ones.
constexpr int KEEP_STEP = 8;

__global__ void __launch_bounds__(256) moe_keep_kernel(KeepParams p) {
    const int b = (int)blockIdx.x, tid = (int)threadIdx.x;
    int first = 0;
    const int n = seq_rows(p.row_start, b, p.rows, &first, p.c.flags);
    const int len = p.c.len[b], keep = p.n_keep[b];
    const int32_t *path = p.path + first;
    bool bad = keep < 0 || keep > n;
    for (int i = tid; !bad && i < keep; i += 256) {
        const int s = path[i], prev = i ? path[i - 1] : -1;
        bad = s <= prev || s >= n;
    }
    bad = __syncthreads_or(bad) != 0;
    if (bad || len < 0 || (int64_t)len + keep > p.c.cap) {
        if (tid == 0) {
            raise_flag(p.c.flags, bad ? MOE_FLAG_PATH : MOE_FLAG_LEN);
            p.new_len[b] = len;
        }
        return;
    }
    const int per = p.c.dim / 8, heads = p.c.heads;
    for (int u = tid; u < 2 * heads * per; u += 256) {
        const bool value = u >= heads * per;
        const int w = value ? u - heads * per : u;
        const int h = w / per, d = (w - h * per) * 8;
        const KvView &kv = value ? p.c.v : p.c.k;
        uint16_t *base = (uint16_t *)kv.p + h * kv.head + d;
        for (int i0 = 0; i0 < keep; i0 += KEEP_STEP) {
            uint4 x[KEEP_STEP];
            int64_t to[KEEP_STEP];
#pragma unroll
            for (int k = 0; k < KEEP_STEP; ++k) {
                to[k] = -1;
                const int i = i0 + k;
                if (i >= keep || path[i] == i) continue;
                int ps, ss, pd, sd;
                if (!find_slot(p.c, b, (int64_t)len + path[i], &ps, &ss) ||
                    !find_slot(p.c, b, (int64_t)len + i, &pd, &sd))
                    continue;
                x[k] = *(const uint4 *)(base + ps * kv.page + ss * kv.slot);
                to[k] = pd * kv.page + sd * kv.slot;
            }
#pragma unroll
            for (int k = 0; k < KEEP_STEP; ++k)
                if (to[k] >= 0) *(uint4 *)(base + to[k]) = x[k];
        }
    }
    // every thread read the length before the barrier above, so the cache's own may be written
    if (tid == 0) p.new_len[b] = len + keep;
}

// ------------------------------------------------------------------ draft verification

// Probabilities and their running sums decide which whole token comes out, so they are
// held in 64 bits throughout: a running sum over 10^5 terms in 32 bits is off by more than the
// probability of most tokens.
struct LogitF32 {
    static __device__ __forceinline__ float at(const void *z, int64_t i) { return ((const float *)z)[i]; }
};
struct LogitBf16 {
    static __device__ __forceinline__ float at(const void *z, int64_t i) { return bf2f(((const uint16_t *)z)[i]); }
};
struct LogitF16 {
    static __device__ __forceinline__ float at(const void *z, int64_t i) { return h2f(((const uint16_t *)z)[i]); }
};

// The weight of one token in a row: exp((z - top) / T) / Z - S q, not below 0; T <= 0: all on `best`.
struct RowState {
    float top;
    int best;
    double inv_t, inv_z, S;     // inv_t 0: greedy
};

template <typename L>
__device__ __forceinline__ double target_weight(const RowState &r, const void *z, int64_t base, int i) {
    if (r.inv_t == 0.0) return i == r.best ? 1.0 : 0.0;
    const float x = L::at(z, base + i);
    // equal first: the largest may be +infinity; NaN compares false and weighs nothing
    return x == r.top ? r.inv_z : x < r.top ? exp(((double)x - (double)r.top) * r.inv_t) * r.inv_z : 0.0;
}

template <typename L>
__device__ __forceinline__ double weight(const RowState &r, const void *z, int64_t base, const float *q, int64_t qbase,
                                         int i) {
    double w = target_weight<L>(r, z, base, i);
    if (r.S > 0.0) {
        w -= r.S * (double)q[qbase + i];
        w = w > 0.0 ? w : 0.0;
    }
    return w;
}

__device__ __forceinline__ double wave_sum(double v) {
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}
__device__ __forceinline__ double wave_scan(double v) {     // inclusive
    for (int d = 1; d < 64; d <<= 1) {
        const double u = __shfl_up(v, d);
        if (lane_id() >= d) v += u;
    }
    return v;
}

constexpr int VERIFY_THREADS = 1024, VERIFY_WAVES = VERIFY_THREADS / 64;

struct VerifyLds {
    double part[MAX_CHUNKS];
    float wave_top[VERIFY_WAVES];
    int wave_best[VERIFY_WAVES];
    int pick;
};

// Sums of the row's weights by chunk into s.part; returns the whole sum, the same in every thread
// (each wave adds the chunks in the same order).
template <typename L>
__device__ double sum_row(const RowState &r, const VerifyParams &p, int64_t base, int64_t qbase, VerifyLds &s) {
    const int chunks = (p.vocab + VOCAB_CHUNK - 1) / VOCAB_CHUNK, wave = (int)threadIdx.x >> 6, lane = lane_id();
    __syncthreads();
    for (int c = wave; c < chunks; c += VERIFY_WAVES) {
        double a = 0.0;
        for (int i = c * VOCAB_CHUNK + lane; i < min(p.vocab, (c + 1) * VOCAB_CHUNK); i += 64)
            a += weight<L>(r, p.logits, base, p.draft, qbase, i);
        a = wave_sum(a);
        if (lane == 0) s.part[c] = a;
    }
    __syncthreads();
    double a = 0.0;
    for (int c = lane; c < chunks; c += 64) a += s.part[c];
    __syncthreads();
    return wave_sum(a);
}

// The first index whose running sum passes u * (the whole sum), from the chunk sums in s.part.
template <typename L>
__device__ int pick_row(const RowState &r, const VerifyParams &p, int64_t base, int64_t qbase, double total, float u,
                        VerifyLds &s) {
    if (threadIdx.x < 64) {
        const int chunks = (p.vocab + VOCAB_CHUNK - 1) / VOCAB_CHUNK, lane = lane_id();
        const double target = (double)u * total;
        // the chunk: the first whose running sum passes, or (a last rounding) the last with weight
        double before = 0.0, at = 0.0;
        int chunk = -1;
        for (int c = 0; c < chunks; ++c) {
            const double w = s.part[c];
            if (w > 0.0) { chunk = c; at = before; }
            before += w;
            if (before > target) break;
        }
        int found = -1;
        if (chunk >= 0) {
            double run = at;
            for (int i0 = chunk * VOCAB_CHUNK; i0 < min(p.vocab, (chunk + 1) * VOCAB_CHUNK); i0 += 64) {
                const int i = i0 + lane;
                const double w = i < p.vocab ? weight<L>(r, p.logits, base, p.draft, qbase, i) : 0.0;
                const double cum = run + wave_scan(w);
                const uint64_t some = __ballot(w > 0.0), past = __ballot(w > 0.0 && cum > target);
                if (past) { found = i0 + __builtin_ctzll(past); break; }
                if (some) found = i0 + 63 - __builtin_clzll(some);
                run = __shfl(cum, 63);
            }
        }
        if (lane == 0) s.pick = found < 0 ? 0 : found;
    }
    __syncthreads();
    const int t = s.pick;
    __syncthreads();
    return t;
}

// One workgroup per sequence walks it.
template <typename L>
__global__ void __launch_bounds__(VERIFY_THREADS) moe_verify_kernel(VerifyParams p) {
    __shared__ VerifyLds s;
    const int b = (int)blockIdx.x, tid = (int)threadIdx.x, lane = lane_id(), wave = tid >> 6;
    int first = 0;
    const int n = seq_rows(p.row_start, b, p.rows, &first, p.flags);
    if (n == 0) {
        if (tid == 0) p.n_keep[b] = 0;
        return;
    }
    const float T = p.temperature ? p.temperature[b] : 1.0f;
    int cur = 0, kept = 1;
    for (;;) {
        const int row = first + cur;
        const int64_t base = row * p.logit_stride, qbase = row * p.draft_stride;
        // the largest logit, the lowest index among equals
        float top = -__builtin_inff();
        int best = p.vocab;
        for (int i = tid; i < p.vocab; i += VERIFY_THREADS) {
            const float x = L::at(p.logits, base + i);
            if (x > top) { top = x; best = i; }
        }
        for (int d = 32; d; d >>= 1) {
            const float t2 = __shfl_xor(top, d);
            const int b2 = __shfl_xor(best, d);
            if (t2 > top || (t2 == top && b2 < best)) { top = t2; best = b2; }
        }
        __syncthreads();
        if (lane == 0) { s.wave_top[wave] = top; s.wave_best[wave] = best; }
        __syncthreads();
        for (int w = 0; w < VERIFY_WAVES; ++w) {
            const float t2 = s.wave_top[w];
            const int b2 = s.wave_best[w];
            if (t2 > top || (t2 == top && b2 < best)) { top = t2; best = b2; }
        }
        RowState r;
        r.top = top;
        r.best = best;
        r.S = 0.0;
        r.inv_z = 1.0;
        r.inv_t = T > 0.0f ? 1.0 / (double)T : 0.0;
        if (best >= p.vocab) {       // nothing above -infinity: token 0, for want of a distribution
            if (tid == 0) raise_flag(p.flags, MOE_FLAG_LOGITS);
            r.best = 0;
            r.inv_t = 0.0;
        }
        const double z = sum_row<L>(r, p, base, qbase, s);
        r.inv_z = 1.0 / z;
        double total = z * r.inv_z;
        int token = -1, next = -1;
        if (!p.draft) {
            for (int c = tid; c < (p.vocab + VOCAB_CHUNK - 1) / VOCAB_CHUNK; c += VERIFY_THREADS) s.part[c] *= r.inv_z;
            __syncthreads();
            token = pick_row<L>(r, p, base, qbase, total, p.u_pick[row], s);
            for (int c = cur + 1; c < n; ++c) {
                if ((p.parent ? p.parent[first + c] : c - 1) != cur) continue;
                const int x = p.tokens[first + c];
                if (x < 0 || x >= p.vocab) {
                    if (tid == 0) raise_flag(p.flags, MOE_FLAG_TOKEN);
                } else if (x == token) {
                    next = c;
                    break;
                }
            }
        } else {
            double rest = 1.0;
            bool fresh = false;      // s.part holds the weights at this S
            for (int c = cur + 1; c < n; ++c) {
                if ((p.parent ? p.parent[first + c] : c - 1) != cur) continue;
                const int x = p.tokens[first + c];
                if (x < 0 || x >= p.vocab) {
                    if (tid == 0) raise_flag(p.flags, MOE_FLAG_TOKEN);
                    continue;
                }
                if ((double)p.u_test[first + c] * (double)p.draft[qbase + x] * rest <
                    weight<L>(r, p.logits, base, p.draft, qbase, x)) {
                    next = c;
                    token = x;
                    break;
                }
                r.S += rest;
                rest = sum_row<L>(r, p, base, qbase, s);
                fresh = true;
            }
            if (next < 0) {
                if (!(rest > 0.0)) { r.S = 0.0; fresh = false; }
                if (!fresh) rest = sum_row<L>(r, p, base, qbase, s);
                token = pick_row<L>(r, p, base, qbase, rest, p.u_pick[row], s);
            }
        }
        if (tid == 0) {
            r.S = 0.0;
            p.path[first + kept - 1] = cur;
            p.out_tokens[first + kept - 1] = token;
            p.logprobs[first + kept - 1] = (float)log(target_weight<L>(r, p.logits, base, token));
        }
        if (next < 0) break;
        cur = next;
        ++kept;
    }
    if (tid == 0) p.n_keep[b] = kept;
    for (int i = kept + tid; i < n; i += VERIFY_THREADS) {
        p.path[first + i] = -1;
        p.out_tokens[first + i] = -1;
        p.logprobs[first + i] = 0.0f;
    }
}
template __global__ void moe_verify_kernel<LogitF32>(VerifyParams);
template __global__ void moe_verify_kernel<LogitBf16>(VerifyParams);
template __global__ void moe_verify_kernel<LogitF16>(VerifyParams);

}  // namespace moe
