// logit_items.h -- what the operators over rows of logits share (gfx950): logits' types, sums along the lanes, chunks of a row,
// exponentials in 64 bits.
#pragma once
#include "drafted_items.h"

namespace moe {

struct LogitF32 {
    typedef float T;
    static __device__ __forceinline__ float value(float v) { return v; }
};
struct LogitBf16 {
    typedef uint16_t T;
    static __device__ __forceinline__ float value(uint16_t v) { return bf2f(v); }
};
struct LogitF16 {
    typedef uint16_t T;
    static __device__ __forceinline__ float value(uint16_t v) { return h2f(v); }
};

// The value that a lane gets from another by a data-parallel move, 0 where the move gives none.
template <int CTRL, int ROWS> __device__ __forceinline__ double moved(double v) {
    const uint64_t x = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)x, CTRL, ROWS, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(x >> 32), CTRL, ROWS, 0xF, false);
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
// Inclusive sums along the lanes: within rows of 16 (shifts by 1, 2, 4, 8), then the ends of rows 0 and 2 into rows 1 and
// 3, then the end of row 1 into rows 2 and 3.
__device__ __forceinline__ double wave_scan(double v) {
    v += moved<0x111, 0xF>(v);
    v += moved<0x112, 0xF>(v);
    v += moved<0x114, 0xF>(v);
    v += moved<0x118, 0xF>(v);
    v += moved<0x142, 0xA>(v);
    v += moved<0x143, 0xC>(v);
    return v;
}
__device__ __forceinline__ double lane_value(double v, int lane) {      // lane: the same in all
    const uint64_t x = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)x, lane), hi = __builtin_amdgcn_readlane((int)(x >> 32), lane);
    return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ float wave_max(float v) {
    const int low = __float_as_int(-__builtin_inff());
#define MOE_MAX_STEP(CTRL, ROWS) \
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(low, __float_as_int(v), CTRL, ROWS, 0xF, false)))
    MOE_MAX_STEP(0x111, 0xF);
    MOE_MAX_STEP(0x112, 0xF);
    MOE_MAX_STEP(0x114, 0xF);
    MOE_MAX_STEP(0x118, 0xF);
    MOE_MAX_STEP(0x142, 0xA);
    MOE_MAX_STEP(0x143, 0xC);
#undef MOE_MAX_STEP
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ double wave_sum(double v) { return lane_value(wave_scan(v), 63); }

// A lane's share of a chunk: four times four neighbours, 256 apart; rows start anywhere, so the
// loads are of the element's alignment.
constexpr int SHARE = VOCAB_CHUNK / 64;
__device__ __forceinline__ int share_index(int k) { return (k >> 2) * 256 + lane_id() * 4 + (k & 3); }

template <typename T> struct __attribute__((packed)) Four {
    T v[4];
};

// The share of chunk c of a row; past the vocabulary `fill`.
template <typename L, typename F>
__device__ __forceinline__ void load_share(const typename L::T *row, int c, int vocab, float fill, F *x) {
    const int base = c * VOCAB_CHUNK;
    if (base + VOCAB_CHUNK <= vocab) {
#pragma unroll
        for (int k = 0; k < SHARE; k += 4) {
            const Four<typename L::T> f = *(const Four<typename L::T> *)(row + base + share_index(k));
#pragma unroll
            for (int e = 0; e < 4; ++e) x[k + e] = L::value(f.v[e]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < SHARE; ++k) {
            const int i = base + share_index(k);
            x[k] = i < vocab ? L::value(row[i]) : fill;
        }
    }
}

// e^y for y <= 0, to about one unit in the last place: y = n log(2) / 32 + r with |r| <= log(2) / 64 (Cody and Waite's
// reduction: the constant in two parts, the first short enough that n times it is exact), then 2^(n / 32) from a table of
// 32 (they lie on different banks of LDS) and the exponent, times the Taylor polynomial of degree 6 at r (its remainder
// is below 4e-18). n is rounded by adding 1.5 2^52, which leaves it in the low bits. Below e^-708, and for a NaN, 0.
//
// Without the table, at degree 12, the statistics of 64 x 5 rows of 100003 took 37 us, with it 36; the library's
// function 41.
__device__ const double EXP2_TABLE[32] = {
    1.0, 1.0218971486541166, 1.0442737824274138, 1.0671404006768237,
    1.0905077326652577, 1.1143867425958924, 1.1387886347566916, 1.1637248587775775,
    1.189207115002721, 1.215247359980469, 1.241857812073484, 1.2690509571917332,
    1.2968395546510096, 1.3252366431597413, 1.3542555469368927, 1.383909881963832,
    1.4142135623730951, 1.4451808069770467, 1.4768261459394993, 1.5091644275934228,
    1.5422108254079407, 1.5759808451078865, 1.6104903319492543, 1.645755478153965,
    1.681792830507429, 1.718619298122478, 1.7562521603732995, 1.7947090750031072,
    1.8340080864093424, 1.8741676341103, 1.9152065613971474, 1.9571441241754002,
};
__device__ __forceinline__ double *exp_table() {
    __shared__ double t[32];
    return t;
}
// A kernel that takes exponentials calls this before the first of them, with all its threads.
__device__ __forceinline__ void fill_exp_table() {
    if (threadIdx.x < 32) exp_table()[threadIdx.x] = EXP2_TABLE[threadIdx.x];
    __syncthreads();
}
__device__ __forceinline__ double exp_down(double y) {
    constexpr double ROUND = 6755399441055744.0;
    const double t = fma(y, 46.16624130844683, ROUND), n = t - ROUND;
    double r = fma(n, -0.02166084938653512, y);
    r = fma(n, -5.9631716539705866e-12, r);
    const int k = (int)(uint32_t)(uint64_t)__double_as_longlong(t);
    const double m = exp_table()[k & 31];
    double e = fma(r, 1.0 / 720.0, 1.0 / 120.0);
    e = fma(e, r, 1.0 / 24.0);
    e = fma(e, r, 1.0 / 6.0);
    e = fma(e, r, 0.5);
    e = fma(e, r, 1.0);
    e = fma(m, e * r, m);
    const uint64_t bits = (uint64_t)__double_as_longlong(e) + ((uint64_t)(uint32_t)((k >> 5) * (1 << 20)) << 32);
    return y >= -708.0 ? __longlong_as_double((long long)bits) : 0.0;
}

// exp((x - top) / T), x at most top. Where the largest is infinite (INF), all weight is on it. NaN weighs nothing.
template <bool INF> __device__ __forceinline__ double relative(float x, float top, double inv_t) {
    return INF ? (x == top ? 1.0 : 0.0) : exp_down(((double)x - (double)top) * inv_t);
}
__device__ __forceinline__ double relative(float x, float top, double inv_t) {
    return top == __builtin_inff() ? relative<true>(x, top, inv_t) : relative<false>(x, top, inv_t);
}

}  // namespace moe
