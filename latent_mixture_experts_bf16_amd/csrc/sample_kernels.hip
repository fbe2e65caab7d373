// sample_kernels.hip -- a token for each row of logits, with temperature, top-k, top-p and min-p (gfx950).
//
// All three cuts, and the draw, are places in one order: falling logits, equal ones by index. None of them needs the row
// sorted, only the running count or weight at a few places. So the logits of a row are counted, and their weights summed, over
// the cells of a grid of an eighth of an octave of weight (a workgroup per chunk, whole card), and one workgroup per
// row finds the cells that matter and looks at their logits alone, narrowing to one value in steps of 10 bits of its
// ordered bits. Whole tokens come out, so weights and sums are in 64 bits. Where atomics add in an order that varies, they add
// whole numbers (the weight in 2^-50 of the largest one), so that the same inputs always give the same token.
#include <type_traits>

#include "logit_items.h"

namespace moe {

// Logits as whole numbers in their order; infinities and both zeros too. A NaN counts as -infinity: key() 0 to below().
template <typename L> struct Ordered;
template <> struct Ordered<LogitF32> {
    static constexpr uint32_t SIGN = 0x80000000u, LOW = 0x007FFFFFu;     // LOW: of -infinity
    static __device__ __forceinline__ uint32_t bits(float v) { return __float_as_uint(v); }
    static __device__ __forceinline__ float value(uint32_t b) { return __uint_as_float(b); }
};
template <> struct Ordered<LogitBf16> {
    static constexpr uint32_t SIGN = 0x8000u, LOW = 0x007Fu;
    static __device__ __forceinline__ uint32_t bits(uint16_t v) { return v; }
    static __device__ __forceinline__ float value(uint32_t b) { return bf2f((uint16_t)b); }
};
template <> struct Ordered<LogitF16> {
    static constexpr uint32_t SIGN = 0x8000u, LOW = 0x03FFu;
    static __device__ __forceinline__ uint32_t bits(uint16_t v) { return v; }
    static __device__ __forceinline__ float value(uint32_t b) { return h2f((uint16_t)b); }
};
template <typename L> __device__ __forceinline__ uint32_t key_of(typename L::T v) {
    typedef Ordered<L> O;
    constexpr uint32_t MASK = O::SIGN | (O::SIGN - 1);
    uint32_t b = O::bits(v);
    const float x = L::value(v);
    if (x == 0.0f) b = 0;                                                 // -0 is 0
    if (!(x == x)) return O::LOW;
    return b & O::SIGN ? ~b & MASK : b | O::SIGN;
}
template <typename L> __device__ __forceinline__ float value_of(uint32_t key) {
    typedef Ordered<L> O;
    constexpr uint32_t MASK = O::SIGN | (O::SIGN - 1);
    return O::value(key & O::SIGN ? key & ~O::SIGN : ~key & MASK);
}

// Temperature of a row as cells (eighths of an octave of weight) of a logit, and whether only the largest logit counts. A greedy
// row is one that keeps the first token of the order; its weights are then of no matter. (An infinite T counts as the
// largest finite one, so that a logit of -infinity still weighs nothing.)
struct RowHeat {
    double cells;
    bool greedy;
};
__device__ __forceinline__ RowHeat row_heat(const SampleParams &p, int row) {
    const float T = p.temperature ? p.temperature[row] : 1.0f;
    const bool greedy = !(T > 0.0f);
    return {(greedy ? 1.0 : 1.0 / (double)fminf(T, 3.4028234e38f)) * (8.0 * 1.4426950408889634), greedy};
}
// How many cells below the one of the largest a cell is, 0 .. SAMPLE_CELLS - 1 (the last one holds all that lie further down).
__device__ __forceinline__ int cells_below(double top, double cell) {
    const double d = top == cell ? 0.0 : top - cell;
    return d < (double)(SAMPLE_CELLS - 1) ? (int)d : SAMPLE_CELLS - 1;
}

// 2^(y / 8) for y <= 0, to about 2^-48: y = n / 4 + r with |r| <= 1/8, 2^(n / 32) from a table (its entries lie on different
// banks of LDS) and the exponent, times the Taylor polynomial of degree 5 of e^(r log(2) / 8) (its remainder is below
// 3e-15 of the value where r is largest). n is rounded by adding 1.5 2^52, which leaves it in the low bits. Below 2^-64, where
// nothing is left of it in what follows, 2^-64.
__device__ __forceinline__ double weight_of(double y) {
    constexpr double ROUND = 6755399441055744.0, C = 0.08664339756999316;     // log(2) / 8
    y = fmax(y, -512.0);
    const double t = fma(y, 4.0, ROUND);
    const double r = fma(t - ROUND, -0.25, y);
    const int k = (int)(uint32_t)(uint64_t)__double_as_longlong(t);
    const double m = exp_table()[k & 31];
    double e = fma(r, C * C * C * C * C / 120.0, C * C * C * C / 24.0);
    e = fma(e, r, C * C * C / 6.0);
    e = fma(e, r, C * C / 2.0);
    e = fma(e, r, C);
    e = fma(m, e * r, m);
    const uint64_t bits = (uint64_t)__double_as_longlong(e) + ((uint64_t)(uint32_t)((k >> 5) * (1 << 20)) << 32);
    return __longlong_as_double((long long)bits);
}
// The weight of a logit beside the largest, y and top_y in cells. Where the largest is infinite, all weight is on it.
__device__ __forceinline__ double beside(double y, double top_y) {
    return y == top_y ? 1.0 : top_y == __builtin_inf() ? 0.0 : weight_of(y - top_y);
}
// A weight of at most 1 as a whole number of 2^-50, to nearest: the low bits of its sum with 4.
__device__ __forceinline__ uint64_t whole50(double w) {
    return (uint64_t)__double_as_longlong(fma(w, 0x1p50, 0x1p52)) & 0xFFFFFFFFFFFFFull;
}
// A weight as a whole number of 2^-shift.
__device__ __forceinline__ double power2(int e) { return __longlong_as_double((long long)(1023 + e) << 52); }
__device__ __forceinline__ uint64_t whole(double w, int shift) { return (uint64_t)fma(w, power2(shift), 0.5); }

template <typename L> __device__ __forceinline__ const typename L::T *row_of(const SampleParams &p, int row) {
    return (const typename L::T *)p.logits + (int64_t)row * p.stride;
}

// Add to a cell of a histogram in LDS. Where the lanes that do all have the same one (rows of equal logits), once for all.
__device__ __forceinline__ void add_to(uint64_t *mass, uint32_t *count, int at, uint64_t w, bool on) {
    if (!on) return;
    if (__all(at == uniform(at))) {
        const uint64_t who = __ballot(true);
        if (__popcll(who) == 64) {
            for (int d = 32; d; d >>= 1) w += (uint64_t)__shfl_xor((long long)w, d);
            if (lane_id() == 0) {
                atomicAdd((unsigned long long *)mass + at, (unsigned long long)w);
                atomicAdd(count + at, 64u);
            }
            return;
        }
    }
    atomicAdd((unsigned long long *)mass + at, (unsigned long long)w);
    atomicAdd(count + at, 1u);
}

// ------------------------------------------------------------------ the histogram of a chunk

template <typename L> __global__ void __launch_bounds__(256) moe_sample_cells_kernel(SampleParams p) {
    __shared__ uint64_t mass[SAMPLE_CELLS];
    __shared__ uint32_t count[SAMPLE_CELLS];
    __shared__ float tops[4];
    const int row = (int)(blockIdx.z * gridDim.y + blockIdx.y), tid = (int)threadIdx.x, wave = tid >> 6;
    if (row >= p.rows) return;
    const int c = (int)blockIdx.x;
    float x[SHARE];
    const int part = c * (SAMPLE_CHUNK / VOCAB_CHUNK) + wave;
    load_share<L>(row_of<L>(p, row), part, p.vocab, -__builtin_inff(), x);
    mass[tid] = 0;
    count[tid] = 0;
    fill_exp_table();
    const RowHeat h = row_heat(p, row);
    float top = -__builtin_inff();
#pragma unroll
    for (int k = 0; k < SHARE; ++k) top = fmaxf(top, x[k]);      // not a NaN: the other operand
    top = wave_max(top);
    if (lane_id() == 0) tops[wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    const int64_t at = (int64_t)row * p.chunks + c;
    const double top_y = (double)top * h.cells, cell = floor(top_y);
    if (tid == 0) p.head[at] = {top_y, top, 0};
    if (!(top > -__builtin_inff())) return;
    if (top < __builtin_inff()) {
#pragma unroll
        for (int k = 0; k < SHARE; ++k) {
            const double y = (double)x[k] * h.cells;
            const double d = fmin(cell - floor(y), (double)(SAMPLE_CELLS - 1));
            add_to(mass, count, (int)d, whole50(weight_of(y - top_y)), x[k] > -__builtin_inff());     // a NaN is not
        }
    } else {
#pragma unroll
        for (int k = 0; k < SHARE; ++k) {
            const bool on = x[k] > -__builtin_inff(), is = x[k] == top;
            add_to(mass, count, is ? 0 : SAMPLE_CELLS - 1, is ? 1ull << 50 : 0, on);
        }
    }
    __syncthreads();
    p.mass[at * SAMPLE_CELLS + tid] = mass[tid];
    p.count[at * SAMPLE_CELLS + tid] = (uint16_t)count[tid];
}

// ------------------------------------------------------------------ the row

// LIST: logits of the cells that matter that are kept in LDS; more are read from the row each time.
constexpr int ROW_THREADS = 1024, LIST = 8192, STEP_BITS = 10, MOST_CHUNKS = MAX_VOCAB / SAMPLE_CHUNK;

struct RowLds {
    double upto_mass[SAMPLE_CELLS + 1];                           // of all cells above
    uint32_t upto_count[SAMPLE_CELLS + 1];
    uint32_t low[SAMPLE_CELLS], high[SAMPLE_CELLS];               // least and largest key of a cell that is looked at
    uint8_t want[SAMPLE_CELLS];
    double factor[MOST_CHUNKS];                                   // of a chunk's weights
    int below[MOST_CHUNKS];                                       // its first cell
    uint64_t mass[ROW_THREADS];
    uint32_t count[ROW_THREADS];
    uint32_t key[LIST], index[LIST];
    double wave_mass[16];
    uint32_t wave_count[16], wave_first[16], wave_last[16];
    float wave_top[16];
    double found_mass;
    uint32_t found_count, found_ties, n, token;
};

// A place in the order: a value, how many logits have it, the weight of one, and the weight and number of those above.
struct Place {
    uint32_t key, ties, above_count;
    double above, weight;
};

template <typename L> struct Row {
    const SampleParams &p;
    RowLds &s;
    const typename L::T *logits;
    RowHeat h;
    double top_y;
    bool in_list;

    __device__ __forceinline__ double y_of(float x) const { return (double)x * h.cells; }
    __device__ __forceinline__ double weight(uint32_t key) const { return beside(y_of(value_of<L>(key)), top_y); }
    __device__ __forceinline__ int cell(float x) const { return cells_below(floor(top_y), floor(y_of(x))); }

    // The first cell whose weight with all above it reaches x (or passes it), else the last with logits. In every lane.
    template <bool PAST> __device__ __forceinline__ int cell_by(double x) const {
        return first_cell([&](int c) { return PAST ? s.upto_mass[c + 1] > x : s.upto_mass[c + 1] >= x; });
    }
    template <typename F> __device__ __forceinline__ int first_cell(F yes) const {
        int first = SAMPLE_CELLS, last = -1;
#pragma unroll
        for (int k = 3; k >= 0; --k) {
            const int c = lane_id() * 4 + k;
            const bool some = s.upto_count[c + 1] > s.upto_count[c];
            if (some && last < 0) last = c;
            if (some && yes(c)) first = c;
        }
        const uint64_t a = __ballot(first < SAMPLE_CELLS), b = __ballot(last >= 0);
        return a ? __builtin_amdgcn_readlane(first, (int)__builtin_ctzll(a))
                 : __builtin_amdgcn_readlane(last, 63 - (int)__builtin_clzll(b));
    }

    // Lists the logits of the cells from `from` to `to` that s.want names, and finds the bounds of each cell's keys.
    __device__ void gather(int from, int to) {
        // no logit of these cells lies outside: y's rounding is below the half cell that is added
        const double most = (floor(top_y) - from + 1.5) / h.cells, least = (floor(top_y) - to - 0.5) / h.cells;
        const float hi = top_y == __builtin_inf() || from == 0 ? __builtin_inff() : __double2float_ru(most);
        // (the lowest number, since -infinity is in no cell)
        const float lo = top_y == __builtin_inf() ? (to ? -3.4028234e38f : __builtin_inff())
                         : to == SAMPLE_CELLS - 1 ? -3.4028234e38f : fmaxf(__double2float_rd(least), -3.4028234e38f);
        const int tid = (int)threadIdx.x;
        constexpr int DEEP = 8;
        auto test = [&](typename L::T v, int i, bool on) {
            const float x = L::value(v);
            on = on && x >= lo && x <= hi;
            int c = 0;
            if (on) {
                c = cell(x);
                on = s.want[c];
            }
            const uint64_t who = __ballot(on);
            if (!who) return;
            uint32_t base = 0;
            const int leader = (int)__builtin_ctzll(who);
            if (lane_id() == leader) base = atomicAdd(&s.n, (uint32_t)__popcll(who));
            base = (uint32_t)__builtin_amdgcn_readlane((int)base, leader);
            if (on) {
                const uint32_t key = key_of<L>(v), at = base + (uint32_t)__popcll(who & ((1ull << lane_id()) - 1));
                if (at < LIST) {
                    s.key[at] = key;
                    s.index[at] = (uint32_t)i;
                }
                if (key < *(volatile uint32_t *)&s.low[c]) atomicMin(&s.low[c], key);
                if (key > *(volatile uint32_t *)&s.high[c]) atomicMax(&s.high[c], key);
            }
        };
        const int whole_steps = p.vocab / (ROW_THREADS * 4);
        int b = 0;
        for (; b + DEEP <= whole_steps; b += DEEP) {
            Four<typename L::T> v[DEEP];
#pragma unroll
            for (int k = 0; k < DEEP; ++k) v[k] = *(const Four<typename L::T> *)(logits + ((b + k) * ROW_THREADS + tid) * 4);
#pragma unroll
            for (int k = 0; k < DEEP; ++k) {
                float t = L::value(v[k].v[0]);
                bool near = t >= lo && t <= hi;
#pragma unroll
                for (int e = 1; e < 4; ++e) {
                    t = L::value(v[k].v[e]);
                    near |= t >= lo && t <= hi;
                }
                if (__any(near))
#pragma unroll
                    for (int e = 0; e < 4; ++e) test(v[k].v[e], ((b + k) * ROW_THREADS + tid) * 4 + e, true);
            }
        }
        for (int i0 = b * ROW_THREADS * 4; i0 < p.vocab; i0 += ROW_THREADS) {
            const int i = i0 + tid;
            const bool on = i < p.vocab;
            test(on ? logits[i] : typename L::T(0), i, on);
        }
    }

    // f(key, index) of every logit whose key is from lo to hi, in cells that were gathered.
    template <typename F> __device__ __forceinline__ void each(uint32_t lo, uint32_t hi, F f) const {
        const int tid = (int)threadIdx.x, n = in_list ? (int)s.n : p.vocab;
        for (int i = tid; i < n; i += ROW_THREADS) {
            const uint32_t key = in_list ? s.key[i] : key_of<L>(logits[i]);
            if (key >= lo && key <= hi) f(key, in_list ? s.index[i] : (uint32_t)i);
        }
    }

    // Sums over the threads before each one, the first thread for which `yes` holds of the sums up to it (else the last with a
    // count), and what lies before that one.
    template <typename F> __device__ __forceinline__ int first_step(uint32_t n, double m, F yes) {
        const int tid = (int)threadIdx.x, lane = lane_id(), wave = uniform(tid >> 6);
        uint32_t upto_n = n;
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t u = (uint32_t)__shfl_up((int)upto_n, d);
            if (lane >= d) upto_n += u;
        }
        double upto_m = wave_scan(m);
        if (lane == 63) {
            s.wave_count[wave] = upto_n;
            s.wave_mass[wave] = upto_m;
        }
        __syncthreads();
        uint32_t before_n = 0;
        double before_m = 0.0;
        for (int k = 0; k < wave; ++k) {
            before_n += s.wave_count[k];
            before_m += s.wave_mass[k];
        }
        upto_n += before_n;
        upto_m += before_m;
        const uint64_t a = __ballot(n && yes(upto_n, upto_m)), b = __ballot(n > 0);
        if (lane == 0) {
            s.wave_first[wave] = a ? (uint32_t)(wave * 64 + (int)__builtin_ctzll(a)) : ROW_THREADS;
            s.wave_last[wave] = b ? (uint32_t)(wave * 64 + 64 - (int)__builtin_clzll(b)) : 0;
        }
        __syncthreads();
        const uint32_t f = s.wave_first[lane & 15], l = s.wave_last[lane & 15];
        const uint64_t c = __ballot(f < ROW_THREADS) & 0xFFFF, d = __ballot(l > 0) & 0xFFFF;
        int t = 0;
        if (c) t = __builtin_amdgcn_readlane((int)f, (int)__builtin_ctzll(c));
        else if (d) t = __builtin_amdgcn_readlane((int)l, 63 - (int)__builtin_clzll(d)) - 1;
        if (tid == t) {
            s.found_count = upto_n - n;
            s.found_mass = upto_m - m;
            s.found_ties = n;
        }
        __syncthreads();
        return t;
    }

    // The value of cell c at which the running count (BY_COUNT) or weight reaches `goal` (or passes it: PAST).
    template <bool BY_COUNT, bool PAST> __device__ Place find(int c, double goal) {
        const int tid = (int)threadIdx.x;
        uint32_t lo = s.low[c], hi = s.high[c];
        Place r;
        r.above = s.upto_mass[c];
        r.above_count = s.upto_count[c];
        r.ties = s.upto_count[c + 1] - r.above_count;
        // weights of this cell are below 2^(1/8 - c/8) of the largest
        const int n_bits = 32 - __builtin_clz(max(r.ties, 1u)), shift = c / 8 + 61 - n_bits;
        const double unit = power2(-shift);
        while (hi > lo) {
            const int cut = max(0, 32 - __builtin_clz(hi - lo) - STEP_BITS);
            s.mass[tid] = 0;
            s.count[tid] = 0;
            __syncthreads();
            each(lo, hi, [&](uint32_t key, uint32_t) {
                add_to(s.mass, s.count, (int)((hi - key) >> cut), whole(weight(key), shift), true);
            });
            __syncthreads();
            const int t = first_step(s.count[tid], (double)s.mass[tid] * unit, [&](uint32_t n, double m) {
                return BY_COUNT ? (double)(r.above_count + n) >= goal : PAST ? r.above + m > goal : r.above + m >= goal;
            });
            r.above += s.found_mass;
            r.above_count += s.found_count;
            r.ties = s.found_ties;
            hi -= (uint32_t)t << cut;
            lo = max(lo, hi - ((1u << cut) - 1u));
        }
        r.key = hi;
        r.weight = weight(hi);
        return r;
    }

    // The index of the t-th (from 0) of the logits whose key is `key`, of which there are `ties`.
    __device__ uint32_t nth_index(uint32_t key, uint32_t t, uint32_t ties) {
        const int tid = (int)threadIdx.x;
        if (ties == 1) {
            each(key, key, [&](uint32_t, uint32_t at) { s.token = at; });
            __syncthreads();
            return s.token;
        }
        uint32_t lo = 0, hi = (uint32_t)p.vocab - 1;
        while (hi > lo) {
            const int cut = max(0, 32 - __builtin_clz(hi - lo) - STEP_BITS);
            s.count[tid] = 0;
            __syncthreads();
            each(key, key, [&](uint32_t, uint32_t at) {
                if (at >= lo && at <= hi) atomicAdd(&s.count[(at - lo) >> cut], 1u);
            });
            __syncthreads();
            const int f = first_step(s.count[tid], 0.0, [&](uint32_t n, double) { return n > t; });
            t -= min(t, s.found_count);
            lo += (uint32_t)f << cut;
            hi = min(hi, lo + ((1u << cut) - 1u));
        }
        return lo;
    }
};

template <typename L> __global__ void __launch_bounds__(ROW_THREADS) moe_sample_row_kernel(SampleParams p) {
    __shared__ RowLds s;
    const int row = (int)blockIdx.x, tid = (int)threadIdx.x, lane = lane_id(), group = tid >> 8, cell = tid & 255;
    const RowHeat h = row_heat(p, row);
    SampleHead head = {0.0, -__builtin_inff(), 0};
    if (tid < p.chunks) head = p.head[(int64_t)row * p.chunks + tid];
    if (tid < SAMPLE_CELLS) {
        s.want[tid] = 0;
        s.low[tid] = 0xFFFFFFFFu;
        s.high[tid] = 0;
    }
    if (tid == 0) s.n = 0;
    float top = wave_max(head.top);
    if (lane == 0) s.wave_top[tid >> 6] = top;
    fill_exp_table();
    top = wave_max(s.wave_top[lane & 15]);
    if (!(top > -__builtin_inff())) {
        if (tid == 0) {
            raise_flag(p.flags, MOE_FLAG_LOGITS);
            p.tokens[row] = 0;
            p.logprobs[row] = 0.0f;
        }
        return;
    }
    const double top_y = (double)top * h.cells;
    if (tid < p.chunks) {
        const bool some = head.top > -__builtin_inff();
        s.below[tid] = some ? cells_below(floor(top_y), floor(head.top_y)) : -1;
        s.factor[tid] = some ? beside(head.top_y, top_y) * power2(-50) : 0.0;
    }
    __syncthreads();
    // the chunks' cells on the row's: thread (group, cell) takes every fourth chunk; what goes into the last cell from
    // elsewhere is added by all threads
    double m = 0.0, tail = 0.0;
    uint32_t n = 0, tail_n = 0;
    const int64_t base = (int64_t)row * p.chunks * SAMPLE_CELLS;
#pragma unroll 8
    for (int c = group; c < p.chunks; c += 4) {
        const int off = s.below[c], from = cell - off;
        const bool here = off >= 0 && from >= 0;
        const int64_t at = base + (int64_t)c * SAMPLE_CELLS + (here ? from : 0);
        const uint64_t w = p.mass[at];
        const uint32_t k = p.count[at];
        if (here && cell < SAMPLE_CELLS - 1) {
            m += (double)w * s.factor[c];
            n += k;
        }
        if (off >= 0 && cell + off >= SAMPLE_CELLS - 1) {
            tail += (double)p.mass[base + (int64_t)c * SAMPLE_CELLS + cell] * s.factor[c];
            tail_n += p.count[base + (int64_t)c * SAMPLE_CELLS + cell];
        }
    }
    s.count[tid] = n;
    ((double *)s.mass)[tid] = m;
    tail = wave_sum(tail);
    for (int d = 32; d; d >>= 1) tail_n += (uint32_t)__shfl_xor((int)tail_n, d);
    if (lane == 0) {
        s.wave_mass[tid >> 6] = tail;
        s.wave_count[tid >> 6] = tail_n;
    }
    __syncthreads();
    if (tid < 64) {
        double w[4], sum = 0.0;
        uint32_t k[4], sum_n = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = tid * 4 + e;
            w[e] = 0.0;
            k[e] = 0;
            for (int g = 0; g < 4; ++g) {
                w[e] += ((double *)s.mass)[g * 256 + c];
                k[e] += s.count[g * 256 + c];
            }
            if (c == SAMPLE_CELLS - 1)
                for (int g = 0; g < 16; ++g) {
                    w[e] += s.wave_mass[g];
                    k[e] += s.wave_count[g];
                }
            sum += w[e];
            sum_n += k[e];
        }
        double before = wave_scan(sum) - sum;
        uint32_t upto = sum_n;
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t u = (uint32_t)__shfl_up((int)upto, d);
            if (tid >= d) upto += u;
        }
        uint32_t before_n = upto - sum_n;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s.upto_mass[tid * 4 + e] = before;
            s.upto_count[tid * 4 + e] = before_n;
            before += w[e];
            before_n += k[e];
        }
        if (tid == 63) {
            s.upto_mass[SAMPLE_CELLS] = before;
            s.upto_count[SAMPLE_CELLS] = before_n;
        }
    }
    __syncthreads();
    const double all = s.upto_mass[SAMPLE_CELLS];
    Row<L> r = {p, s, row_of<L>(p, row), h, top_y, true};

    // the cells that the cuts and the draw fall into: of top-p and the draw a first and a last one, since what the cuts before
    // them leave is known to a cell only
    const uint32_t k = h.greedy ? 1u : p.top_k && p.top_k[row] > 0 ? (uint32_t)p.top_k[row] : 0xFFFFFFFFu;
    const float top_p = p.top_p ? p.top_p[row] : 1.0f, asked = p.min_p ? p.min_p[row] : 0.0f;
    const float min_p = asked > 1.0f ? 1.0f : asked, given = p.u[row];
    const double u = (double)(given > 0.0f ? fminf(given, 0.99999994f) : 0.0f);
    const bool by_k = k < s.upto_count[SAMPLE_CELLS], by_p = !h.greedy && top_p < 1.0f, by_m = !h.greedy && min_p > 0.0f;
    const int k_cell = by_k ? r.first_cell([&](int c) { return s.upto_count[c + 1] >= k; }) : 0;
    double least = all, most = all;
    if (by_k) least = s.upto_mass[k_cell], most = s.upto_mass[k_cell + 1];
    int p_from = 0, p_to = -1, m_cell = 0;
    if (by_p) {
        p_from = r.template cell_by<false>((double)top_p * least);
        p_to = r.template cell_by<false>((double)top_p * most);
        least = fmin(least, s.upto_mass[p_from]);
        most = fmin(most, s.upto_mass[p_to + 1]);
    }
    double floor_y = 0.0;
    if (by_m) {
        // the cell that the least weight lies in
        floor_y = top_y == __builtin_inf() ? top_y : top_y + 8.0 * log2((double)min_p);
        m_cell = cells_below(floor(top_y), floor(floor_y));
        least = fmin(least, s.upto_mass[m_cell]);
        most = fmin(most, s.upto_mass[m_cell + 1]);
    }
    const int d_from = r.template cell_by<true>(u * least), d_to = r.template cell_by<true>(u * most);
    int from = d_from, to = d_to;
    if (by_k) from = min(from, k_cell), to = max(to, k_cell);
    if (by_p) from = min(from, p_from), to = max(to, p_to);
    if (by_m) from = min(from, m_cell), to = max(to, m_cell);
    if (tid < SAMPLE_CELLS)
        s.want[tid] = (tid >= d_from && tid <= d_to) || (by_k && tid == k_cell) || (by_p && tid >= p_from && tid <= p_to) ||
                      (by_m && tid == m_cell);
    __syncthreads();
    r.gather(from, to);
    __syncthreads();
    r.in_list = s.n <= LIST;

    double kept = all;
    if (by_k) {
        const Place at = r.template find<true, false>(k_cell, (double)k);
        kept = at.above + (double)(k - at.above_count) * at.weight;
    }
    if (by_p) {
        const double goal = (double)top_p * kept;
        const Place at = r.template find<false, false>(min(max(r.template cell_by<false>(goal), p_from), p_to), goal);
        const double ties = at.weight > 0.0 ? ceil((goal - at.above) / at.weight) : 1.0;
        kept = fmin(kept, at.above + fmin(fmax(ties, 1.0), (double)at.ties) * at.weight);
    }
    if (by_m) {
        // the part of its cell that is not below the least weight
        const uint32_t count = s.upto_count[m_cell + 1] - s.upto_count[m_cell];
        const int n_bits = 32 - __builtin_clz(max(count, 1u)), shift = m_cell / 8 + 61 - n_bits;
        if (tid == 0) s.mass[0] = 0;
        __syncthreads();
        uint64_t sum = 0;
        if (count)
            r.each(s.low[m_cell], s.high[m_cell], [&](uint32_t key, uint32_t) {
                const double w = r.weight(key);
                if (w >= (double)min_p) sum += whole(w, shift);
            });
        for (int d = 32; d; d >>= 1) sum += (uint64_t)__shfl_xor((long long)sum, d);
        if (lane == 0 && sum) atomicAdd((unsigned long long *)s.mass, (unsigned long long)sum);
        __syncthreads();
        kept = fmin(kept, s.upto_mass[m_cell] + (double)s.mass[0] * power2(-shift));
        __syncthreads();
    }
    const double goal = u * kept;
    const Place at = r.template find<false, true>(min(max(r.template cell_by<true>(goal), d_from), d_to), goal);
    const double t = at.weight > 0.0 ? floor((goal - at.above) / at.weight) : 0.0;
    const uint32_t token = r.nth_index(at.key, (uint32_t)fmin(fmax(t, 0.0), (double)(at.ties - 1)), at.ties);
    if (tid == 0) {
        const double y = r.y_of(value_of<L>(at.key));
        p.tokens[row] = (int32_t)token;
        p.logprobs[row] = h.greedy ? 0.0f : (float)((y == top_y ? 0.0 : (y - top_y) * 0.08664339756999316) - log(all));
    }
}

template __global__ void moe_sample_cells_kernel<LogitF32>(SampleParams);
template __global__ void moe_sample_cells_kernel<LogitBf16>(SampleParams);
template __global__ void moe_sample_cells_kernel<LogitF16>(SampleParams);
template __global__ void moe_sample_row_kernel<LogitF32>(SampleParams);
template __global__ void moe_sample_row_kernel<LogitBf16>(SampleParams);
template __global__ void moe_sample_row_kernel<LogitF16>(SampleParams);

}  // namespace moe
