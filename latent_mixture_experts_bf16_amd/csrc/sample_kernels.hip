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

// Temperature of a row: 1 / T, the cells of a logit, and whether only the largest logit counts. A greedy row is one that keeps
// the first token of the order; its weights are then of no matter.
struct RowHeat {
    double inv, cells;
    bool greedy;
};
__device__ __forceinline__ RowHeat row_heat(const SampleParams &p, int row) {
    const float T = p.temperature ? p.temperature[row] : 1.0f;
    const bool greedy = !(T > 0.0f);
    const double inv = greedy ? 1.0 : 1.0 / (double)fminf(T, 3.4028234e38f);
    return {inv, inv * (8.0 * 1.4426950408889634), greedy};
}
// The cell of the grid that a logit lies in: rising with it.
__device__ __forceinline__ double cell_of(float x, const RowHeat &h) { return floor((double)x * h.cells); }
// How many cells below, 0 .. SAMPLE_CELLS - 1 (the last one holds all that lie further down).
__device__ __forceinline__ int cells_below(double top, double cell) {
    const double d = top == cell ? 0.0 : top - cell;
    return d < (double)(SAMPLE_CELLS - 1) ? (int)d : SAMPLE_CELLS - 1;
}
// A weight as a whole number of 2^-shift.
__device__ __forceinline__ uint64_t whole(double w, int shift) {
    return (uint64_t)fma(w, __longlong_as_double((long long)(1023 + shift) << 52), 0.5);
}
__device__ __forceinline__ double power2(int e) { return __longlong_as_double((long long)(1023 + e) << 52); }

template <typename L> __device__ __forceinline__ const typename L::T *row_of(const SampleParams &p, int row) {
    return (const typename L::T *)p.logits + (int64_t)row * p.stride;
}

// Add to a cell of a histogram in LDS. Where a wave's lanes all have the same one (rows of equal logits), once for all.
__device__ __forceinline__ void add_to(uint64_t *mass, uint32_t *count, int at, uint64_t w, bool on) {
    const uint64_t who = __ballot(on);
    if (!who) return;
    const int one = __builtin_amdgcn_readlane(at, (int)__builtin_ctzll(who));
    if (__ballot(on && at == one) == who && __popcll(who) > 8) {
        uint64_t sum = on ? w : 0;
        for (int d = 32; d; d >>= 1) sum += (uint64_t)__shfl_xor((long long)sum, d);
        if (lane_id() == 0) {
            atomicAdd((unsigned long long *)mass + one, (unsigned long long)sum);
            atomicAdd(count + one, (uint32_t)__popcll(who));
        }
    } else if (on) {
        atomicAdd((unsigned long long *)mass + at, (unsigned long long)w);
        atomicAdd(count + at, 1u);
    }
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
    const double cell = cell_of(top, h);
    if (tid == 0) p.head[at] = {cell, top, 0};
    if (!(top > -__builtin_inff())) return;
#pragma unroll
    for (int k = 0; k < SHARE; ++k) {
        const bool on = x[k] > -__builtin_inff();                // a NaN is not
        const double w = on ? relative(x[k], top, h.inv) : 0.0;
        add_to(mass, count, on ? cells_below(cell, cell_of(x[k], h)) : 0, whole(w, 50), on);
    }
    __syncthreads();
    p.mass[at * SAMPLE_CELLS + tid] = mass[tid];
    p.count[at * SAMPLE_CELLS + tid] = (uint16_t)count[tid];
}

// ------------------------------------------------------------------ the row

constexpr int ROW_THREADS = 1024, ROW_LIST = 8192, STEP_BITS = 10;

struct RowLds {
    double cell_mass[SAMPLE_CELLS], upto_mass[SAMPLE_CELLS];      // by cell, and with all cells above it
    uint32_t cell_count[SAMPLE_CELLS], upto_count[SAMPLE_CELLS];
    uint64_t mass[ROW_THREADS];
    uint32_t count[ROW_THREADS];
    uint32_t key[ROW_LIST], index[ROW_LIST];                      // of the cell that was looked at last
    double wave_mass[16];
    uint32_t wave_count[16];
    double found_mass;
    uint32_t found_count, found_some, n_found, n, lo, hi;
    int found;
};

// Inclusive sums over the workgroup's threads, in their order.
__device__ __forceinline__ uint32_t scan_counts(RowLds &s, uint32_t v) {
    const int lane = lane_id(), wave = (int)threadIdx.x >> 6;
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t u = (uint32_t)__shfl_up((int)v, d);
        if (lane >= d) v += u;
    }
    if (lane == 63) s.wave_count[wave] = v;
    __syncthreads();
    for (int k = 0; k < wave; ++k) v += s.wave_count[k];
    __syncthreads();
    return v;
}
__device__ __forceinline__ double scan_masses(RowLds &s, double v) {
    const int lane = lane_id(), wave = (int)threadIdx.x >> 6;
    v = wave_scan(v);
    if (lane == 63) s.wave_mass[wave] = v;
    __syncthreads();
    double before = 0.0;
    for (int k = 0; k < wave; ++k) before += s.wave_mass[k];
    __syncthreads();
    return before + v;
}
// The first thread for which `yes` holds, else the last of those with `some`; -1: none of either.
__device__ __forceinline__ int first_thread(RowLds &s, bool yes, bool some) {
    const int tid = (int)threadIdx.x;
    if (tid == 0) s.found = 0x7FFFFFFF, s.found_some = 0;
    __syncthreads();
    const uint64_t a = __ballot(yes), b = __ballot(some);
    if (lane_id() == 0) {
        if (a) atomicMin(&s.found, tid + (int)__builtin_ctzll(a));
        if (b) atomicMax(&s.found_some, (uint32_t)(tid + 64 - __builtin_clzll(b)));
    }
    __syncthreads();
    const int r = s.found != 0x7FFFFFFF ? s.found : (int)s.found_some - 1;
    __syncthreads();
    return r;
}

// A place in the order: a value, what lies above it, how many logits have it, and the weight of one.
struct Place {
    uint32_t key, ties;
    double above, weight;
    uint32_t above_count;
};

template <typename L> struct Row {
    const SampleParams &p;
    RowLds &s;
    const typename L::T *logits;
    RowHeat h;
    float top;
    double top_cell;
    int listed;          // the cell in s.key and s.index, -1: none; its bounds are in s.lo and s.hi
    bool in_list;

    __device__ __forceinline__ double weight(uint32_t key) const { return relative(value_of<L>(key), top, h.inv); }

    // The keys of cell c, from the last one below the cell above it down to its own lowest: both found by halving.
    __device__ void bounds(int c) {
        const int tid = (int)threadIdx.x;
        if (tid < 2) {
            // the least key whose logit lies less than c + 1 cells (thread 0) or c cells (thread 1) below the top
            const int cells = c + 1 - tid;
            uint32_t lo = Ordered<L>::LOW + 1, hi = key_of_top() + 1;
            if (cells == SAMPLE_CELLS) hi = lo;
            while (lo < hi) {
                const uint32_t mid = lo + (hi - lo) / 2;
                if (cells_below(top_cell, cell_of(value_of<L>(mid), h)) < cells) hi = mid; else lo = mid + 1;
            }
            if (tid == 0) s.lo = lo; else s.hi = lo - 1;
        }
    }
    __device__ __forceinline__ uint32_t key_of_top() const { return key_from(top); }
    static __device__ __forceinline__ uint32_t key_from(float v) {
        if constexpr (sizeof(typename L::T) == 4)
            return key_of<L>(v);
        else
            return key_of<L>(std::is_same<L, LogitF16>::value ? f2h(v) : f2bf(v));
    }

    // Makes cell c the one that is looked at: its bounds, and its logits where they fit.
    __device__ void look_at(int c) {
        if (listed == c) return;
        __syncthreads();
        bounds(c);
        if (threadIdx.x == 0) s.n = 0;
        __syncthreads();
        listed = c;
        in_list = s.cell_count[c] <= ROW_LIST;
        if (!in_list) return;
        const uint32_t lo = s.lo, hi = s.hi;
        each_logit([&](uint32_t key, int i) {
            if (key >= lo && key <= hi) {
                const uint32_t at = atomicAdd(&s.n, 1u);
                if (at < ROW_LIST) {
                    s.key[at] = key;
                    s.index[at] = (uint32_t)i;
                }
            }
        });
        __syncthreads();
    }

    // f(key, index) of every logit of the row.
    template <typename F> __device__ __forceinline__ void each_logit(F f) const {
        for (int i = (int)threadIdx.x; i < p.vocab; i += ROW_THREADS) f(key_of<L>(logits[i]), i);
    }
    // f(on, key, index) of every logit in the cell that is looked at, whole waves at a time.
    template <typename F> __device__ __forceinline__ void each(F f) const {
        const int tid = (int)threadIdx.x, n = in_list ? min((int)s.n, ROW_LIST) : p.vocab;
        const uint32_t lo = s.lo, hi = s.hi;
        for (int i0 = 0; i0 < n; i0 += ROW_THREADS) {
            const int i = i0 + tid;
            const bool some = i < n;
            uint32_t key = 0, at = (uint32_t)i;
            if (some) {
                key = in_list ? s.key[i] : key_of<L>(logits[i]);
                if (in_list) at = s.index[i];
            }
            f(some && key >= lo && key <= hi, key, at);
        }
    }

    // The value of cell c at which the running count (BY_COUNT) or weight reaches `goal` (or passes it: PAST).
    template <bool BY_COUNT, bool PAST> __device__ Place find(int c, double goal) {
        look_at(c);
        const int tid = (int)threadIdx.x;
        Place r;
        r.above = c ? s.upto_mass[c - 1] : 0.0;
        r.above_count = c ? s.upto_count[c - 1] : 0;
        uint32_t lo = s.lo, hi = s.hi;
        // weights of this cell are below 2^(1/8 - c/8) of the largest
        const int n_bits = 32 - __builtin_clz(max(s.cell_count[c], 1u)), shift = c / 8 + 61 - n_bits;
        const double unit = power2(-shift);
        for (;;) {
            const int cut = max(0, 32 - (hi == lo ? 32 : __builtin_clz(hi - lo)) - STEP_BITS);
            s.mass[tid] = 0;
            s.count[tid] = 0;
            __syncthreads();
            each([&](bool on, uint32_t key, uint32_t) {
                on = on && key >= lo && key <= hi;
                const uint64_t w = on ? whole(weight(key), shift) : 0;
                add_to(s.mass, s.count, on ? (int)((hi - key) >> cut) : 0, w, on);
            });
            __syncthreads();
            const uint32_t n = s.count[tid];
            const double m = (double)s.mass[tid] * unit;
            const uint32_t upto_n = scan_counts(s, n);
            const double upto_m = scan_masses(s, m);
            const bool yes = n && (BY_COUNT ? (double)(r.above_count + upto_n) >= goal
                                            : PAST ? r.above + upto_m > goal : r.above + upto_m >= goal);
            const int t = max(first_thread(s, yes, n > 0), 0);
            if (tid == t) {
                s.found_count = upto_n - n;
                s.found_mass = upto_m - m;
                s.n_found = n;
            }
            __syncthreads();
            r.above += s.found_mass;
            r.above_count += s.found_count;
            r.ties = s.n_found;
            hi -= (uint32_t)t << cut;
            lo = max(lo, hi - ((1u << cut) - 1u));
            __syncthreads();
            if (cut == 0) break;
        }
        r.key = hi;
        r.weight = weight(hi);
        return r;
    }

    // The index of the t-th (from 0) of the logits whose key is `key`, in the cell that is looked at.
    __device__ int nth_index(uint32_t key, uint32_t t) {
        const int tid = (int)threadIdx.x;
        uint32_t lo = 0, hi = (uint32_t)p.vocab - 1;
        for (;;) {
            const int cut = max(0, 32 - (hi == lo ? 32 : __builtin_clz(hi - lo)) - STEP_BITS);
            s.mass[tid] = 0;
            s.count[tid] = 0;
            __syncthreads();
            each([&](bool on, uint32_t k, uint32_t at) {
                on = on && k == key && at >= lo && at <= hi;
                add_to(s.mass, s.count, on ? (int)((at - lo) >> cut) : 0, 0, on);
            });
            __syncthreads();
            const uint32_t n = s.count[tid], upto = scan_counts(s, n);
            const int f = max(first_thread(s, upto > t, n > 0), 0);
            if (tid == f) s.found_count = upto - n;
            __syncthreads();
            t -= min(t, s.found_count);
            lo += (uint32_t)f << cut;
            hi = min(hi, lo + ((1u << cut) - 1u));
            __syncthreads();
            if (cut == 0) break;
        }
        return (int)lo;
    }
};

template <typename L> __global__ void __launch_bounds__(ROW_THREADS) moe_sample_row_kernel(SampleParams p) {
    __shared__ RowLds s;
    const int row = (int)blockIdx.x, tid = (int)threadIdx.x, group = tid >> 8, cell = tid & 255;
    fill_exp_table();
    const RowHeat h = row_heat(p, row);
    const SampleHead *head = p.head + (int64_t)row * p.chunks;
    // the largest logit (at most 256 chunks: a lane has up to 4 of them), the same in every wave
    float top = -__builtin_inff();
    for (int c = lane_id(); c < p.chunks; c += 64) top = fmaxf(top, head[c].top);
    top = wave_max(top);
    if (!(top > -__builtin_inff())) {
        if (tid == 0) {
            raise_flag(p.flags, MOE_FLAG_LOGITS);
            p.tokens[row] = 0;
            p.logprobs[row] = 0.0f;
        }
        return;
    }
    const double top_cell = cell_of(top, h);
    // the chunks' cells on the row's: thread (group, cell) takes every fourth chunk
    double m = 0.0, tail = 0.0;
    uint32_t n = 0, tail_n = 0;
    for (int c = group; c < p.chunks; c += 4) {
        const SampleHead hd = head[c];
        if (!(hd.top > -__builtin_inff())) continue;
        const int off = cells_below(top_cell, hd.cell);
        const double f = relative(hd.top, top, h.inv) * power2(-50);
        const int64_t at = ((int64_t)row * p.chunks + c) * SAMPLE_CELLS;
        if (cell < SAMPLE_CELLS - 1 && cell >= off) {
            m += (double)p.mass[at + cell - off] * f;
            n += p.count[at + cell - off];
        }
        if (cell + off >= SAMPLE_CELLS - 1) {
            tail += (double)p.mass[at + cell] * f;
            tail_n += p.count[at + cell];
        }
    }
    // what goes into the last cell, from all threads
    tail = scan_masses(s, tail);
    tail_n = scan_counts(s, tail_n);
    if (tid == ROW_THREADS - 1) { s.found_mass = tail; s.found_count = tail_n; }
    s.count[tid] = n;
    ((double *)s.mass)[tid] = m;
    __syncthreads();
    if (group == 0) {
        for (int k = 1; k < 4; ++k) {
            n += s.count[tid + 256 * k];
            m += ((double *)s.mass)[tid + 256 * k];
        }
        if (cell == SAMPLE_CELLS - 1) { n = s.found_count; m = s.found_mass; }
    } else {
        n = 0;
        m = 0.0;
    }
    const uint32_t upto_n = scan_counts(s, n);
    const double upto_m = scan_masses(s, m);
    if (group == 0) {
        s.cell_mass[cell] = m;
        s.cell_count[cell] = n;
        s.upto_mass[cell] = upto_m;
        s.upto_count[cell] = upto_n;
    }
    __syncthreads();
    const uint32_t all_n = s.upto_count[SAMPLE_CELLS - 1];
    const double all = s.upto_mass[SAMPLE_CELLS - 1];

    Row<L> r = {p, s, row_of<L>(p, row), h, top, top_cell, -1, false};
    // the first cell that reaches a count or a weight
    auto cell_by = [&](bool yes) { return max(first_thread(s, group == 0 && n && yes, group == 0 && n), 0); };
    double kept = all;
    const uint32_t k = h.greedy ? 1u : p.top_k && p.top_k[row] > 0 ? (uint32_t)p.top_k[row] : 0xFFFFFFFFu;
    if (k < all_n) {
        const Place at = r.template find<true, false>(cell_by(upto_n >= k), (double)k);
        kept = at.above + (double)(k - at.above_count) * at.weight;
    }
    const double first_k = kept;
    const float top_p = p.top_p ? p.top_p[row] : 1.0f, asked = p.min_p ? p.min_p[row] : 0.0f;
    const float min_p = asked > 1.0f ? 1.0f : asked;
    if (!h.greedy && top_p < 1.0f) {
        const double goal = (double)top_p * first_k;
        const Place at = r.template find<false, false>(cell_by(upto_m >= goal), goal);
        const double ties = at.weight > 0.0 ? ceil((goal - at.above) / at.weight) : 1.0;
        kept = fmin(kept, at.above + fmin(fmax(ties, 1.0), (double)at.ties) * at.weight);
    }
    if (!h.greedy && min_p > 0.0f) {
        // the cell that the least weight lies in, and the part of it that is not below that
        const double least = top == __builtin_inff() ? (double)top : (double)top + log((double)min_p) / h.inv;
        const int c = cells_below(top_cell, floor(least * h.cells));
        r.look_at(c);
        const int n_bits = 32 - __builtin_clz(max(s.cell_count[c], 1u)), shift = c / 8 + 61 - n_bits;
        if (tid == 0) s.mass[0] = 0;
        __syncthreads();
        uint64_t sum = 0;
        r.each([&](bool on, uint32_t key, uint32_t) {
            const double w = on ? r.weight(key) : 0.0;
            if (on && w >= (double)min_p) sum += whole(w, shift);
        });
        for (int d = 32; d; d >>= 1) sum += (uint64_t)__shfl_xor((long long)sum, d);
        if (lane_id() == 0) atomicAdd((unsigned long long *)s.mass, (unsigned long long)sum);
        __syncthreads();
        kept = fmin(kept, (c ? s.upto_mass[c - 1] : 0.0) + (double)s.mass[0] * power2(-shift));
        __syncthreads();
    }
    const float u = p.u[row];
    const double goal = (double)(u > 0.0f ? fminf(u, 0.99999994f) : 0.0f) * kept;
    const Place at = r.template find<false, true>(cell_by(upto_m > goal), goal);
    const double t = at.weight > 0.0 ? floor((goal - at.above) / at.weight) : 0.0;
    const int token = r.nth_index(at.key, (uint32_t)fmin(fmax(t, 0.0), (double)(at.ties - 1)));
    if (tid == 0) {
        const float x = value_of<L>(at.key);
        p.tokens[row] = token;
        p.logprobs[row] = h.greedy ? 0.0f : (float)((x == top ? 0.0 : ((double)x - (double)top) * h.inv) - log(all));
    }
}

template __global__ void moe_sample_cells_kernel<LogitF32>(SampleParams);
template __global__ void moe_sample_cells_kernel<LogitBf16>(SampleParams);
template __global__ void moe_sample_cells_kernel<LogitF16>(SampleParams);
template __global__ void moe_sample_row_kernel<LogitF32>(SampleParams);
template __global__ void moe_sample_row_kernel<LogitBf16>(SampleParams);
template __global__ void moe_sample_row_kernel<LogitF16>(SampleParams);

}  // namespace moe
