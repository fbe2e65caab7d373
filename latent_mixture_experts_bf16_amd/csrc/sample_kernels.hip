// sample_kernels.hip -- a token for each row of logits, with temperature, top-k, top-p and min-p (gfx950).
//
// All three cuts, and the draw, are places in one order: falling logits, equal ones by index. None of them needs the row
// sorted, only the running count or weight at a few places. So the logits of a row are counted, and their weights summed, over
// the cells of a grid of a quarter of an octave of weight (a workgroup per chunk, whole card), and one workgroup per
// row finds the cells that matter and looks at their logits alone, narrowing to one value in steps of 10 bits of its
// ordered bits. Whole tokens come out, so weights and sums are in 64 bits. Where atomics add in an order that varies, they add
// whole numbers, so that the same inputs always give the same token: weights in 2^-50 of their chunk's largest one, and within a
// cell in the least unit that its number of logits leaves room for in 64 bits (Row::shift_of).
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

// Temperature of a row, as 32nds of an octave of weight for each unit of a logit, and whether only the largest logit counts. A
// greedy row is one that keeps the first token of the order; its weights are then of no matter. (An infinite T counts as the
// largest finite one, so that a logit of -infinity still weighs nothing.)
struct RowHeat {
    double steps;
    bool greedy;
};
__device__ __forceinline__ RowHeat row_heat(const SampleParams &p, int row) {
    const float T = p.temperature ? p.temperature[row] : 1.0f;
    const bool greedy = !(T > 0.0f);
    return {(greedy ? 1.0 : 1.0 / (double)fminf(T, 3.4028234e38f)) * (32.0 * 1.4426950408889634), greedy};
}

// The grid that all logits of a row are placed on: the nearest whole number of steps, rising with the logit, the same wherever
// it is computed. Eight steps make a cell. (1.5 2^52 added leaves the number in the low bits. From 2^50 on, where that does not
// hold, the product is taken as it is: two different logits are then millions of steps apart.)
constexpr double ROUND = 6755399441055744.0;
__device__ __forceinline__ double grid(float x, double steps) {
    const double near = fma((double)x, steps, ROUND) - ROUND, far = (double)x * steps;
    return fabs(far) < 0x1p50 ? near : far;
}
// How many cells below the one of the largest, 0 .. SAMPLE_CELLS - 1 (the last one holds all that lie further down: nearly 64
// octaves, where weights are nothing in 2^-50).
__device__ __forceinline__ int cells_below(double top, double g) {
    const double d = top == g ? 0.0 : floor(top * 0.125) - floor(g * 0.125);
    return d < (double)(SAMPLE_CELLS - 1) ? (int)d : SAMPLE_CELLS - 1;
}

// 2^((k + r) / 32) for a whole k <= 0 and |r| <= 1/2, to about 2^-48: 2^(k / 32) from a table (its entries lie on different
// banks of LDS) and the exponent, times the Taylor polynomial of degree 5 of e^(r log(2) / 32), whose remainder is below
// 3e-15 of the value where r is largest.
struct Power32 {
    // the coefficients, kept in scalar registers
    double c1 = 0.02166084939249829, c2 = c1 * c1 / 2.0, c3 = c1 * c1 * c1 / 6.0, c4 = c1 * c1 * c1 * c1 / 24.0,
           c5 = c1 * c1 * c1 * c1 * c1 / 120.0;     // c1: log(2) / 32
    __device__ __forceinline__ Power32() { asm("" : "+s"(c1), "+s"(c2), "+s"(c3), "+s"(c4), "+s"(c5)); }
    // 2^(r / 32) - 1
    __device__ __forceinline__ double rest(double r) const {
        double e = fma(r, c5, c4);
        e = fma(e, r, c3);
        e = fma(e, r, c2);
        e = fma(e, r, c1);
        return e * r;
    }
    __device__ __forceinline__ double operator()(int k, double r) const {
        const double m = exp_table()[k & 31], e = fma(m, rest(r), m);
        return __hiloint2double(__double2hiint(e) + ((k >> 5) * (1 << 20)), __double2loint(e));
    }
};
__device__ __forceinline__ double power32(int k, double r) { return Power32()(k, r); }
// The weight of a logit x beside the largest one of its chunk or row, `top`: that one weighs exactly 1, and so does every
// other that is equal to it, so that a border that falls exactly between two of them (top-p of one half over two equal logits)
// falls there in these sums and quotients too. (Borders of different weights are never exact: exponentials of different
// rational numbers have no such sums.) Where the largest is infinite, all weight is on it. What lies 64 octaves below weighs
// nothing.
__device__ __forceinline__ double weight_of(float x, float top, double steps) {
    if (top == __builtin_inff()) return x == top ? 1.0 : 0.0;
    const double t = (double)x - (double)top, d = t * steps, k = rint(d);
    return d > -2048.0 ? power32((int)k, fma(t, steps, -k)) : 0.0;
}
// A weight of at most 2 as a whole number of 2^-50, to nearest: the low bits of its sum with 4.
__device__ __forceinline__ uint64_t whole50(double w) {
    return (uint64_t)__double_as_longlong(fma(w, 0x1p50, 0x1p52)) & 0xFFFFFFFFFFFFFull;
}
// A weight as a whole number of 2^-shift.
__device__ __forceinline__ double power2(int e) { return __longlong_as_double((long long)(1023 + e) << 52); }
__device__ __forceinline__ uint64_t whole(double w, int shift) { return (uint64_t)fma(w, power2(shift), 0.5); }

template <typename L> __device__ __forceinline__ const typename L::T *row_of(const SampleParams &p, int row) {
    return (const typename L::T *)p.logits + (int64_t)row * p.stride;
}

// Inclusive sums of counts along the lanes.
__device__ __forceinline__ uint32_t wave_count_scan(uint32_t v) {
#define MOE_ADD_STEP(CTRL, ROWS) v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false)
    MOE_ADD_STEP(0x111, 0xF);
    MOE_ADD_STEP(0x112, 0xF);
    MOE_ADD_STEP(0x114, 0xF);
    MOE_ADD_STEP(0x118, 0xF);
    MOE_ADD_STEP(0x142, 0xA);
    MOE_ADD_STEP(0x143, 0xC);
#undef MOE_ADD_STEP
    return v;
}

// Add a logit's weight to a cell of a histogram in LDS: where all lanes have the same logit, once for all.
__device__ __forceinline__ void add_to(uint64_t *mass, uint32_t *count, int at, uint64_t w, float x) {
    const uint64_t on = __ballot(true);
    const bool same = __ballot(__float_as_int(x) == uniform(__float_as_int(x))) == on;
    const uint32_t n = same ? (uint32_t)__popcll(on) : 1u;
    if (!same || lane_id() == (int)__builtin_ctzll(on)) {
        atomicAdd((unsigned long long *)mass + at, (unsigned long long)(w * n));
        atomicAdd(count + at, n);
    }
}

// ------------------------------------------------------------------ the cells of a chunk

// Besides counts and weights, the chunk's logits but those of its last cell are listed by cell (their numbers within the chunk), so that
// the row's workgroup reads only those of the cells that matter: a pass over the row by one workgroup takes 11 us and more.
//
// Bound by LDS atomics (one of 64 bits and one of 32 a logit; the former some 20 us of the 47) and the vector instructions of the
// weight (three quarters of the time): 256 rows of 100003 fp32 logits, 102 MB, 47 us; 64 rows of 131072 bf16 logits 21 us; one
// row, whose 32 workgroups leave most of the card idle, 7.4 us. Three atomics of 32 bits in place of the one of 64 took 55 us, a
// form without branches, which holds 107 registers, 50 (this one 47 then).
template <typename L> __global__ void __launch_bounds__(256) moe_sample_cells_kernel(SampleParams p) {
    __shared__ uint64_t mass[SAMPLE_CELLS];
    __shared__ uint32_t count[SAMPLE_CELLS];
    __shared__ __align__(16) uint16_t list[SAMPLE_CHUNK];
    __shared__ uint16_t start[SAMPLE_CELLS];
    __shared__ float tops[4];
    const int row = (int)(blockIdx.z * gridDim.y + blockIdx.y), tid = (int)threadIdx.x, wave = tid >> 6, lane = lane_id();
    if (row >= p.rows) return;
    const int c = (int)blockIdx.x;
    float x[SHARE];
    load_share<L>(row_of<L>(p, row), c * (SAMPLE_CHUNK / VOCAB_CHUNK) + wave, p.vocab, -__builtin_inff(), x);
    mass[tid] = 0;
    count[tid] = 0;
    fill_exp_table();
    const RowHeat h = row_heat(p, row);
    float top = -__builtin_inff();
#pragma unroll
    for (int k = 0; k < SHARE; ++k) top = fmaxf(top, x[k]);      // not a NaN: the other operand
    top = wave_max(top);
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    const int64_t at = (int64_t)row * p.chunks + c;
    const double top_g = grid(top, h.steps);
    // Two kinds of chunks are taken slowly, and not listed: with an infinite logit, or a temperature next to 0 (places that 32 bits
    // do not hold) or so large that no number is low enough to weigh nothing; with many equal logits (a wave's first ones), whose
    // additions at one place would take one after another
    const float lowest = (float)((top_g - 2304.0) / h.steps);      // what lies below weighs nothing
    const bool equal = x[0] > lowest && __ballot(x[0] == __int_as_float(uniform(__float_as_int(x[0])))) == ~0ull;
    const Power32 power;
    // The table of powers over the power of the largest logit's own rest on the grid: the weights below are places' on the grid, and
    // are so beside the largest logit. Its own is then 1 to within three roundings, which is 2^50 whole numbers of 2^-50.
    if (tid < 32) exp_table()[tid] /= 1.0 + power.rest(fma((double)top, h.steps, -top_g));
    const bool slow = __syncthreads_or(equal || !(fabs(top_g) < 0x1p29 && lowest > -__builtin_inff())) != 0;
    if (tid == 0) p.head[at] = {top_g, top, !slow};
    if (!(top > -__builtin_inff())) return;
    if (slow) {
        fill_exp_table();
#pragma unroll 1
        for (int i = c * SAMPLE_CHUNK + tid; i < min(p.vocab, (c + 1) * SAMPLE_CHUNK); i += 256) {
            const float v = L::value(row_of<L>(p, row)[i]);
            if (v > -__builtin_inff())
                add_to(mass, count, cells_below(top_g, grid(v, h.steps)), whole50(weight_of(v, top, h.steps)), v);
        }
        __syncthreads();
        p.mass[at * SAMPLE_CELLS + tid] = mass[tid];
        p.count[at * SAMPLE_CELLS + tid] = (uint16_t)count[tid];
        return;
    }
    // Cell and number within it; a logit in the last cell has none. Places on the grid are 32-bit whole numbers. What lies far
    // below, or is a NaN, is taken to the last cell, where a weight is nothing in 2^-50.
    uint32_t place[SHARE], last_n = 0;
    const int top_n = (int)top_g, top_d = top_n >> 3;
#pragma unroll
    for (int k = 0; k < SHARE; ++k) {
        const double v = (double)fmaxf(x[k], lowest), t = fma(v, h.steps, ROUND);
        const int n = max((int)(uint32_t)(uint64_t)__double_as_longlong(t), top_n - 2048);
        const uint64_t w = whole50(power(n - top_n, fma(v, h.steps, ROUND - t)));
        place[k] = (uint32_t)(top_d - (n >> 3));
        if (place[k] < SAMPLE_CELLS - 1) {
            atomicAdd((unsigned long long *)mass + place[k], (unsigned long long)w);
            place[k] = place[k] << 16 | atomicAdd(count + place[k], 1u);
        } else {       // the last cell, where masked tokens often are: added once at the end
            place[k] = 0xFFFFFFFFu;
            last_n += x[k] > -__builtin_inff();
        }
    }
    if (last_n) atomicAdd(count + SAMPLE_CELLS - 1, last_n);
    __syncthreads();
    if (tid < 64) {
        constexpr int EACH = SAMPLE_CELLS / 64;
        uint32_t n[EACH], sum = 0;
#pragma unroll
        for (int e = 0; e < EACH; ++e) sum += n[e] = count[tid * EACH + e];
        uint32_t upto = wave_count_scan(sum) - sum;
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            start[tid * EACH + e] = (uint16_t)upto;
            upto += n[e];
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < SHARE; ++k)
        if (place[k] != 0xFFFFFFFFu)
            list[start[place[k] >> 16] + (place[k] & 0xFFFFu)] = (uint16_t)(wave * VOCAB_CHUNK + share_index(k));
    p.mass[at * SAMPLE_CELLS + tid] = mass[tid];
    p.count[at * SAMPLE_CELLS + tid] = (uint16_t)count[tid];
    p.start[at * SAMPLE_CELLS + tid] = start[tid];
    __syncthreads();
    for (int i = tid * 8; i < start[SAMPLE_CELLS - 1]; i += 256 * 8)
        *(uint4 *)(p.list + at * SAMPLE_CHUNK + i) = *(const uint4 *)(list + i);
}

// ------------------------------------------------------------------ the row

// LIST: logits of the cells that matter that are kept in LDS; more are read from the row each time. RUNS: of neighbouring cells that
// matter (those of the three cuts and of the draw). FEW: so many equal or nearly equal logits are compared in a wave's lanes.
// Sixteen waves, which hide the latency of a list's entries (a cell of some thousand logits takes 40 us with four). What is a chain of
// a few scalars is left to the first of them. The code runs once through, from memory where other kernels ran in
// between, so what is not hot is kept short rather than unrolled (53 KB of it took twice the time).
constexpr int ROW_THREADS = 1024, ROW_WAVES = ROW_THREADS / 64, LIST = 12288, RUNS = 4, FEW = 64;
constexpr int MOST_CHUNKS = MAX_VOCAB / SAMPLE_CHUNK;
constexpr int STEP_BITS = 10, STEPS = 1 << STEP_BITS, CELLS_EACH = SAMPLE_CELLS / 64;
static_assert(STEPS == ROW_THREADS, "a thread has a step, and a pair of chunk and run");
static_assert(MOST_CHUNKS * RUNS <= ROW_THREADS, "a thread has a step, and a pair of chunk and run");

// A place in the order: a value, how many logits have it, the weight of one, and the weight and number of those above.
struct Place {
    uint32_t key, ties, above_count;
    double above, weight;
};

// Cells from .. to, none where to is less.
struct Span {
    int from, to;
    __device__ __forceinline__ bool has(int c) const { return c >= from && c <= to; }
};

struct RowLds {
    double upto_mass[SAMPLE_CELLS + 1];                           // of all cells above
    uint32_t upto_count[SAMPLE_CELLS + 1];
    uint32_t low[SAMPLE_CELLS], high[SAMPLE_CELLS];               // least and largest key of a cell that is listed
    double factor[MOST_CHUNKS];                                   // of a chunk's weights
    int below[MOST_CHUNKS];                                       // its first cell
    uint64_t mass[STEPS];
    uint32_t count[STEPS];
    uint32_t key[LIST], index[LIST];
    uint32_t run_end[MOST_CHUNKS * RUNS];                         // of a chunk's part of a run in the list
    uint16_t run_from[MOST_CHUNKS * RUNS];                        // and where the chunk's own list has it
    uint32_t few_key[FEW];
    double wave_mass[ROW_WAVES];
    uint32_t wave_count[ROW_WAVES];
    int wave_first[ROW_WAVES], wave_last[ROW_WAVES];
    float wave_top[ROW_WAVES];
    // what the first wave tells the others
    Span at[4], runs[RUNS], look;
    int n_runs, at_once, listed;
    double goal, found_mass;
    uint32_t found_count, found_ties, found_key, n, n_few, token;
};

template <typename L> struct Row {
    const SampleParams &p;
    RowLds &s;
    const typename L::T *logits;
    double steps, top_g;
    float top;
    bool in_list;

    __device__ __forceinline__ double weight(uint32_t key) const { return weight_of(value_of<L>(key), top, steps); }
    __device__ __forceinline__ int cell(float x) const { return cells_below(top_g, grid(x, steps)); }
    // Weights of cell c are below 2^((1 - c) / 4 + 1 / 32), so that whole numbers of 2^-shift, the weight of at most 2^(32 - clz)
    // logits, add up in 64 bits (below 2^61.3).
    __device__ __forceinline__ int shift_of(int c) const {
        return c / 4 + 29 + __builtin_clz(max(s.upto_count[c + 1] - s.upto_count[c], 1u));
    }

    // The first cell up to which the count, or the weight, reaches a goal, else the last with logits. In every lane of a wave.
    __device__ __forceinline__ int first_cell(bool by_count, double goal) const {
        int first = SAMPLE_CELLS, last = -1;
        const int c0 = lane_id() * CELLS_EACH;
        uint32_t n[CELLS_EACH + 1];
        double m[CELLS_EACH];
#pragma unroll
        for (int e = 0; e <= CELLS_EACH; ++e) n[e] = s.upto_count[c0 + e];
#pragma unroll
        for (int e = 0; e < CELLS_EACH; ++e) m[e] = s.upto_mass[c0 + e + 1];
#pragma unroll
        for (int e = CELLS_EACH - 1; e >= 0; --e)
            if (n[e + 1] > n[e]) {
                last = max(last, c0 + e);
                if ((by_count ? (double)n[e + 1] : m[e]) >= goal) first = c0 + e;
            }
        const uint64_t a = __ballot(first < SAMPLE_CELLS), b = __ballot(last >= 0);
        return a ? __builtin_amdgcn_readlane(first, (int)__builtin_ctzll(a))
                 : __builtin_amdgcn_readlane(last, 63 - (int)__builtin_clzll(b));
    }

    // The least and largest key of a cell that is listed.
    __device__ __forceinline__ void bound(int c, uint32_t key) {
        if (key < *(volatile uint32_t *)&s.low[c]) atomicMin(&s.low[c], key);
        if (key > *(volatile uint32_t *)&s.high[c]) atomicMax(&s.high[c], key);
    }

    // Lists the logits of the cells in s.runs (all of them listed by the chunks).
    __device__ __forceinline__ void collect() {
        const int tid = (int)threadIdx.x, wave = uniform(tid >> 6), n_runs = uniform(s.n_runs), pairs = p.chunks * n_runs;
        uint32_t n = 0;
        if (tid < pairs) {
            const int c = tid / n_runs, off = s.below[c];
            const Span run = s.runs[tid - c * n_runs];
            const int from = max(run.from - off, 0), to = run.to - off;      // of the chunk's cells
            const int64_t at = (int64_t)blockIdx.x * p.chunks + c;
            if (off >= 0 && to >= 0) {
                const uint32_t first = p.start[at * SAMPLE_CELLS + from];
                n = p.start[at * SAMPLE_CELLS + to] + (uint32_t)p.count[at * SAMPLE_CELLS + to] - first;
                s.run_from[tid] = (uint16_t)first;
            }
        }
        uint32_t upto = wave_count_scan(n);
        if (lane_id() == 63) s.wave_count[wave] = upto;
        __syncthreads();
        for (int k = 0; k < wave; ++k) upto += s.wave_count[k];
        if (tid < pairs) s.run_end[tid] = upto;
        if (tid == pairs - 1) s.n = upto;
        __syncthreads();
        const int all = (int)s.n;
        constexpr int DEEP = 4;                // entries on their way at once
#pragma unroll 1
        for (int i0 = tid; i0 < all; i0 += ROW_THREADS * DEEP) {
            int part[DEEP], at[DEEP];
            typename L::T v[DEEP];
#pragma unroll
            for (int e = 0; e < DEEP; ++e) part[e] = 0;
#pragma unroll 1
            for (int step = 512; step; step >>= 1)               // the parts that end at or before the entry
#pragma unroll
                for (int e = 0; e < DEEP; ++e)
                    if (part[e] + step <= pairs - 1 && s.run_end[part[e] + step - 1] <= (uint32_t)(i0 + e * ROW_THREADS))
                        part[e] += step;
#pragma unroll
            for (int e = 0; e < DEEP; ++e) {
                const int i = min(i0 + e * ROW_THREADS, all - 1), c = part[e] / n_runs;
                const int from = min(s.run_from[part[e]] + i - (part[e] ? (int)s.run_end[part[e] - 1] : 0), SAMPLE_CHUNK - 1);
                at[e] = c * SAMPLE_CHUNK + p.list[((int64_t)blockIdx.x * p.chunks + c) * SAMPLE_CHUNK + max(from, 0)];
            }
#pragma unroll
            for (int e = 0; e < DEEP; ++e) v[e] = logits[i0 + e * ROW_THREADS < all ? at[e] : 0];
#pragma unroll
            for (int e = 0; e < DEEP; ++e)
                if (i0 + e * ROW_THREADS < all) {
                    const uint32_t key = key_of<L>(v[e]);
                    s.key[i0 + e * ROW_THREADS] = key;
                    s.index[i0 + e * ROW_THREADS] = (uint32_t)at[e];
                    bound(cell(L::value(v[e])), key);
                }
        }
    }

    // The same for any cells by a pass over the row; where they are more than LIST, the bounds of their keys alone.
    __device__ __forceinline__ void gather() {
        const int tid = (int)threadIdx.x;
        const Span want[RUNS] = {s.runs[0], s.runs[1], s.runs[2], s.runs[3]};
        float *const stage = (float *)s.mass;
        constexpr int DEEP = STEPS * 2 / ROW_THREADS;
#pragma unroll 1
        for (int i0 = 0; i0 < p.vocab; i0 += ROW_THREADS * DEEP) {
            typename L::T v[DEEP];
#pragma unroll
            for (int e = 0; e < DEEP; ++e) v[e] = logits[min(i0 + e * ROW_THREADS + tid, p.vocab - 1)];
            // each thread reads back what it wrote
#pragma unroll
            for (int e = 0; e < DEEP; ++e) stage[e * ROW_THREADS + tid] = L::value(v[e]);
#pragma unroll 1
            for (int e = 0; e < DEEP; ++e) {
                const int i = i0 + e * ROW_THREADS + tid;
                const float x = stage[e * ROW_THREADS + tid];
                int c = 0;
                bool on = i < p.vocab && x > -__builtin_inff();
                if (on) {
                    c = cell(x);
                    on = want[0].has(c) || want[1].has(c) || want[2].has(c) || want[3].has(c);
                }
                const uint64_t who = __ballot(on);
                if (!who) continue;
                uint32_t base = 0;
                const int leader = (int)__builtin_ctzll(who);
                if (lane_id() == leader) base = atomicAdd(&s.n, (uint32_t)__popcll(who));
                base = (uint32_t)__builtin_amdgcn_readlane((int)base, leader);
                if (on) {
                    const uint32_t key = key_of<L>(logits[i]), at = base + (uint32_t)__popcll(who & ((1ull << lane_id()) - 1));
                    if (at < LIST) {
                        s.key[at] = key;
                        s.index[at] = (uint32_t)i;
                    }
                    bound(c, key);
                }
            }
        }
    }

    // Lists the logits of the cells in s.runs, and finds the bounds of each cell's keys.
    __device__ __forceinline__ void list() {
        const int tid = (int)threadIdx.x;
        if (tid < SAMPLE_CELLS) {
            s.low[tid] = 0xFFFFFFFFu;
            s.high[tid] = 0;
        }
        if (tid == 0) s.n = 0;
        __syncthreads();
        if (s.listed) collect(); else gather();
        __syncthreads();
        in_list = s.n <= LIST;
    }

    // f(key, index) of every logit whose key is from lo to hi, in cells that were listed.
    template <typename F> __device__ __forceinline__ void each(uint32_t lo, uint32_t hi, F f) const {
        const int n = in_list ? (int)s.n : p.vocab;
#pragma unroll 1
        for (int i = (int)threadIdx.x; i < n; i += ROW_THREADS) {
            const uint32_t key = in_list ? s.key[i] : key_of<L>(logits[i]);
            if (key >= lo && key <= hi) f(key, in_list ? s.index[i] : (uint32_t)i);
        }
    }

    // The first step of s.count and s.mass (in units) for which `yes` holds of the sums up to it, else the last with a count;
    // in s.found_* what lies before it and its count.
    template <typename F> __device__ __forceinline__ int first_step(double unit, F yes) {
        const int tid = (int)threadIdx.x, lane = lane_id(), wave = uniform(tid >> 6);
        const uint32_t n = s.count[tid];
        const double m = (double)s.mass[tid] * unit;
        uint32_t upto_n = wave_count_scan(n);
        double upto_m = wave_scan(m);
        if (lane == 63) {
            s.wave_count[wave] = upto_n;
            s.wave_mass[wave] = upto_m;
        }
        __syncthreads();
#pragma unroll 1
        for (int k = 0; k < wave; ++k) {
            upto_n += s.wave_count[k];
            upto_m += s.wave_mass[k];
        }
        const uint64_t a = __ballot(n && yes(upto_n, upto_m)), b = __ballot(n > 0);
        if (lane == 0) {
            s.wave_first[wave] = a ? tid + (int)__builtin_ctzll(a) : STEPS;
            s.wave_last[wave] = b ? tid + 63 - (int)__builtin_clzll(b) : -1;
        }
        __syncthreads();
        const int f = s.wave_first[lane & (ROW_WAVES - 1)], l = s.wave_last[lane & (ROW_WAVES - 1)];
        const uint64_t c = __ballot(f < STEPS) & ((1u << ROW_WAVES) - 1), d = __ballot(l >= 0) & ((1u << ROW_WAVES) - 1);
        const int t = c ? __builtin_amdgcn_readlane(f, (int)__builtin_ctzll(c))
                        : d ? __builtin_amdgcn_readlane(l, 63 - (int)__builtin_clzll(d)) : 0;
        if (tid == t) {
            s.found_count = upto_n - n;
            s.found_mass = upto_m - m;
            s.found_ties = n;
        }
        __syncthreads();
        return t;
    }
    __device__ __forceinline__ void clear_steps() {
        s.mass[threadIdx.x] = 0;
        s.count[threadIdx.x] = 0;
        __syncthreads();
    }

    // The value of cell c at which the goal is fulfilled.
    __device__ __forceinline__ Place find(int c, bool by_count, double goal) {
        uint32_t lo = s.low[c], hi = s.high[c];
        Place r;
        r.above = s.upto_mass[c];
        r.above_count = s.upto_count[c];
        r.ties = s.upto_count[c + 1] - r.above_count;
        const int shift = shift_of(c);
        const double unit = power2(-shift);
        auto yes = [&](uint32_t n, double m) {
            return (by_count ? (double)(r.above_count + n) : r.above + m) >= goal;
        };
#pragma unroll 1
        while (hi > lo && r.ties > FEW) {
            const int cut = max(0, 32 - __builtin_clz(hi - lo) - STEP_BITS);
            clear_steps();
            each(lo, hi, [&](uint32_t key, uint32_t) {
                add_to(s.mass, s.count, (int)((hi - key) >> cut), whole(weight(key), shift), value_of<L>(key));
            });
            __syncthreads();
            const int t = first_step(unit, yes);
            r.above += s.found_mass;
            r.above_count += s.found_count;
            r.ties = s.found_ties;
            hi -= (uint32_t)t << cut;
            lo = max(lo, hi - ((1u << cut) - 1u));
        }
        if (hi > lo) {
            // few are left: a lane each of the first wave, which adds those above it and those of its own value
            if (threadIdx.x == 0) s.n_few = 0;
            __syncthreads();
            each(lo, hi, [&](uint32_t key, uint32_t) {
                const uint32_t at = atomicAdd(&s.n_few, 1u);
                if (at < FEW) s.few_key[at] = key;
            });
            __syncthreads();
            if (threadIdx.x < 64) {
                const int n = min((int)s.n_few, FEW), lane = lane_id();
                const uint32_t key = lane < n ? s.few_key[lane] : 0;
                const uint64_t own = lane < n ? whole(weight(key), shift) : 0;
                const uint32_t own_lo = (uint32_t)own, own_hi = (uint32_t)(own >> 32);
                uint32_t above = 0, ties = 0;
                uint64_t above_w = 0, ties_w = 0;
#pragma unroll 1
                for (int j = 0; j < n; ++j) {
                    const uint32_t k = (uint32_t)__builtin_amdgcn_readlane((int)key, j);
                    const uint64_t w = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)own_hi, j) << 32 |
                                       (uint32_t)__builtin_amdgcn_readlane((int)own_lo, j);
                    above += k > key;
                    above_w += k > key ? w : 0;
                    ties += k == key;
                    ties_w += k == key ? w : 0;
                }
                // the largest that fulfils the goal with all of its value, else the least
                const bool on = lane < n, enough = on && yes(above + ties, (double)(above_w + ties_w) * unit);
                const uint64_t any = __ballot(enough);
                uint32_t best = any ? (enough ? key : 0) : (on ? ~key : 0);
                for (int d = 32; d; d >>= 1) best = max(best, (uint32_t)__shfl_xor((int)best, d));
                if (!any) best = ~best;
                if (lane == (int)__builtin_ctzll(__ballot(on && key == best))) {
                    s.found_key = best;
                    s.found_mass = (double)above_w * unit;
                    s.found_count = above;
                    s.found_ties = ties;
                }
            }
            __syncthreads();
            hi = s.found_key;
            r.above += s.found_mass;
            r.above_count += s.found_count;
            r.ties = s.found_ties;
            __syncthreads();
        }
        r.key = hi;
        r.weight = weight(hi);
        return r;
    }

    // The index of the t-th (from 0) of the logits whose key is `key`, of which there are `ties`.
    __device__ __forceinline__ uint32_t nth_index(uint32_t key, uint32_t t, uint32_t ties) {
        if (ties == 1) {
            each(key, key, [&](uint32_t, uint32_t at) { s.token = at; });
            __syncthreads();
            return s.token;
        }
        uint32_t lo = 0, hi = (uint32_t)p.vocab - 1;
#pragma unroll 1
        while (hi > lo) {
            const int cut = max(0, 32 - __builtin_clz(hi - lo) - STEP_BITS);
            clear_steps();
            each(key, key, [&](uint32_t, uint32_t at) {
                if (at >= lo && at <= hi) atomicAdd(&s.count[(at - lo) >> cut], 1u);
            });
            __syncthreads();
            const int f = first_step(0.0, [&](uint32_t n, double) { return n > t; });
            t -= min(t, s.found_count);
            lo += (uint32_t)f << cut;
            hi = min(hi, lo + ((1u << cut) - 1u));
        }
        return lo;
    }
};

// Bound by its chains: loads of the chunks' heads and cells (5 us), the cells' decisions by one wave (4 us), lists and then values of
// the cells that matter and the steps through their bits (4 to 20 us), and the fetch of its instructions: one row 20 us, 64
// rows of bf16 logits with all cuts 34, 256 rows 38. With 256 threads the last took 65 us.
template <typename L> __global__ void __launch_bounds__(ROW_THREADS) moe_sample_row_kernel(SampleParams p) {
    __shared__ RowLds s;
    const int row = (int)blockIdx.x, tid = (int)threadIdx.x, lane = lane_id(), wave = uniform(tid >> 6);
    SampleHead head = {0.0, -__builtin_inff(), 1};
    if (tid < p.chunks) head = p.head[(int64_t)row * p.chunks + tid];
    const RowHeat h = row_heat(p, row);
    // what is asked for, in scalar registers
    const int asked_k = p.top_k ? uniform(p.top_k[row]) : 0;
    auto scalar = [](float v) { return __int_as_float(uniform(__float_as_int(v))); };
    const float top_p = p.top_p ? scalar(p.top_p[row]) : 1.0f, asked_m = p.min_p ? scalar(p.min_p[row]) : 0.0f;
    const float min_p = asked_m > 1.0f ? 1.0f : asked_m, given = scalar(p.u[row]);
    const double u = (double)(given > 0.0f ? fminf(given, 0.99999994f) : 0.0f);
    float top = wave_max(head.top);      // (only the first waves have chunks)
    if (lane == 0) s.wave_top[wave] = top;
    fill_exp_table();
    top = wave_max(s.wave_top[lane & (ROW_WAVES - 1)]);
    if (!(top > -__builtin_inff())) {
        if (tid == 0) {
            raise_flag(p.flags, MOE_FLAG_LOGITS);
            p.tokens[row] = 0;
            p.logprobs[row] = 0.0f;
        }
        return;
    }
    const double top_g = grid(top, h.steps);
    if (tid < p.chunks) {
        const bool some = head.top > -__builtin_inff();
        s.below[tid] = some ? cells_below(top_g, head.top_g) : -1;
        s.factor[tid] = some ? weight_of(head.top, top, h.steps) * power2(-50) : 0.0;
    }
    // whether the chunks of the row listed their logits
    const bool listed = !__syncthreads_or(!head.listed && head.top > -__builtin_inff());
    // The chunks' cells on the row's, a thread each for every fourth chunk. A chunk whose largest logit is `off` cells down has
    // its cells that much later; the threads before that take those that would lie past the last cell, which are added to it.
    double m = 0.0, tail = 0.0;
    uint32_t n = 0, tail_n = 0;
    const int64_t base = (int64_t)row * p.chunks * SAMPLE_CELLS;
    constexpr int DEEP = 8, GROUPS = ROW_THREADS / SAMPLE_CELLS;
    const int group = tid / SAMPLE_CELLS, cell = tid & (SAMPLE_CELLS - 1);
#pragma unroll 1
    for (int c0 = group; c0 < p.chunks; c0 += DEEP * GROUPS) {
        uint64_t w[DEEP];
        uint32_t q[DEEP];
        int off[DEEP];
#pragma unroll
        for (int e = 0; e < DEEP; ++e) off[e] = c0 + e * GROUPS < p.chunks ? s.below[c0 + e * GROUPS] : -1;
#pragma unroll
        for (int e = 0; e < DEEP; ++e) {      // all on their way before the first is used
            const int at = min(c0 + e * GROUPS, p.chunks - 1) * SAMPLE_CELLS + ((cell - off[e]) & (SAMPLE_CELLS - 1));
            w[e] = p.mass[base + at];
            q[e] = p.count[base + at];
        }
#pragma unroll
        for (int e = 0; e < DEEP; ++e) {
            if (off[e] < 0) continue;         // a chunk without logits: its cells were not written
            const double v = (double)w[e] * s.factor[c0 + e * GROUPS];
            const bool own = cell >= off[e];
            m += own ? v : 0.0;
            n += own ? q[e] : 0;
            tail += own ? 0.0 : v;
            tail_n += own ? 0 : q[e];
        }
    }
    tail = wave_sum(tail);
    tail_n = (uint32_t)__builtin_amdgcn_readlane((int)wave_count_scan(tail_n), 63);
    if (lane == 0) {
        s.wave_mass[wave] = tail;
        s.wave_count[wave] = tail_n;
    }
    ((double *)s.mass)[tid] = m;
    s.count[tid] = n;
    __syncthreads();
    enum { K, P, M, D };
    const uint32_t k = h.greedy ? 1u : asked_k > 0 ? (uint32_t)asked_k : 0xFFFFFFFFu;
    const double least_weight = (double)min_p;
    Row<L> r = {p, s, row_of<L>(p, row), h.steps, top_g, top, true};
    // what has to be reached, where `left` is left by the cuts before: the draw passes its part of that, and so reaches the next number
    auto goal_of = [&](int i, double left) {
        return i == K ? (double)k : i == P ? (double)top_p * left
                                           : __longlong_as_double(__double_as_longlong(u * left) + 1);
    };
    // which of them there are, a bit each
    int by = (!h.greedy && top_p < 1.0f) << P | (!h.greedy && min_p > 0.0f) << M | 1 << D;
    if (wave == 0) {
        double w[CELLS_EACH], sum = 0.0;
        uint32_t q[CELLS_EACH], sum_n = 0;
#pragma unroll
        for (int e = 0; e < CELLS_EACH; ++e) {
            const int c = lane * CELLS_EACH + e;
            w[e] = 0.0;
            q[e] = 0;
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                w[e] += ((double *)s.mass)[g * SAMPLE_CELLS + c];
                q[e] += s.count[g * SAMPLE_CELLS + c];
            }
        }
        const double tails = wave_sum(lane < ROW_WAVES ? s.wave_mass[lane & (ROW_WAVES - 1)] : 0.0);
        const uint32_t tails_n = (uint32_t)__builtin_amdgcn_readlane(
            (int)wave_count_scan(lane < ROW_WAVES ? s.wave_count[lane & (ROW_WAVES - 1)] : 0), 63);
        if (lane == 63) {
            w[CELLS_EACH - 1] += tails;
            q[CELLS_EACH - 1] += tails_n;
        }
#pragma unroll
        for (int e = 0; e < CELLS_EACH; ++e) {
            sum += w[e];
            sum_n += q[e];
        }
        double before = wave_scan(sum) - sum;
        uint32_t before_n = wave_count_scan(sum_n) - sum_n;
#pragma unroll
        for (int e = 0; e < CELLS_EACH; ++e) {
            s.upto_mass[lane * CELLS_EACH + e] = before;
            s.upto_count[lane * CELLS_EACH + e] = before_n;
            before += w[e];
            before_n += q[e];
        }
        if (lane == 63) {
            s.upto_mass[SAMPLE_CELLS] = before;
            s.upto_count[SAMPLE_CELLS] = before_n;
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");

        // The cells that the cuts and the draw fall into: but for top-k a first and a last one, since what the cuts before them
        // leave (and for min-p its place) is not known to more than a cell yet.
        by |= k < s.upto_count[SAMPLE_CELLS] ? 1 << K : 0;
        if (lane < 4) s.at[lane] = {1, 0};
        double least = s.upto_mass[SAMPLE_CELLS], most = least;
#pragma unroll 1
        for (int i = K; i <= D; ++i) {
            if (!(by >> i & 1)) continue;
            Span c;
            if (i == M) {
                // the logarithm in 32 bits is within 1/100 of a step
                const double g = (double)top * h.steps + (double)(32.0f * __log2f((float)least_weight));
                c = {max(cells_below(top_g, g + 0.75), 0), cells_below(top_g, g - 0.75)};
                if (top_g == __builtin_inf()) c = {0, 0};
            } else {
#pragma unroll 1
                for (int end = 0; end < 2; ++end) {
                    const int f = r.first_cell(i == K, goal_of(i, end ? most : least));
                    if (!end) c.from = f;
                    c.to = f;
                }
            }
            s.at[i] = c;
            least = fmin(least, s.upto_mass[c.from]);
            most = fmin(most, s.upto_mass[c.to + 1]);
        }
        // as runs of neighbouring cells, in their order: the next one begins at the least cell that is left
        int n_runs = 0, last = 0;
        uint32_t in_runs = 0;
        const Span at[4] = {s.at[K], s.at[P], s.at[M], s.at[D]};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            last = max(last, at[i].to);
            s.runs[i] = {1, 0};
        }
#pragma unroll 1
        for (int c = 0; n_runs < RUNS;) {
            int from = SAMPLE_CELLS;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (at[i].to >= c && at[i].from <= at[i].to) from = min(from, max(at[i].from, c));
            if (from == SAMPLE_CELLS) break;
            int to = from;
#pragma unroll 1
            for (int again = 0; again < RUNS; ++again)         // as often as there are parts that may go on where another ends
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (at[i].from <= to + 1 && at[i].to > to) to = at[i].to;
            s.runs[n_runs++] = {from, to};
            in_runs += s.upto_count[to + 1] - s.upto_count[from];
            c = to + 1;
        }
        // all of them listed at once where they fit, else those of one cut after the other
        s.n_runs = n_runs;
        s.at_once = in_runs <= LIST;
        s.listed = listed && last < SAMPLE_CELLS - 1;
    }
    __syncthreads();
    by |= k < s.upto_count[SAMPLE_CELLS] ? 1 << K : 0;
    const double all = s.upto_mass[SAMPLE_CELLS];
    const bool at_once = s.at_once;
    bool have = false;

    double kept = all;
    Place found = {};
    double goal = 0.0;
#pragma unroll 1
    for (int i = K; i <= D; ++i) {
        if (!(by >> i & 1)) continue;
        if (wave == 0) {
            s.goal = goal_of(i, kept);
            Span c = s.at[i];
            if (i != M) c.from = c.to = min(max(r.first_cell(i == K, goal_of(i, kept)), c.from), c.to);
            s.look = c;
            if (!at_once) {
                s.runs[0] = c;
                s.runs[1] = s.runs[2] = s.runs[3] = {1, 0};
                s.n_runs = 1;
                s.listed = listed && c.to < SAMPLE_CELLS - 1 && s.upto_count[c.to + 1] - s.upto_count[c.from] <= LIST;
            }
        }
        __syncthreads();
        const Span c = s.look;
        goal = s.goal;
        if (i == K && s.upto_mass[c.to + 1] == s.upto_mass[c.from]) {      // a cut among weights of nothing
            kept = s.upto_mass[c.from];
            __syncthreads();
            continue;
        }
        if (!have) {
            r.list();
            have = at_once;
        }
        if (i == M) {
            // the part of its cells that is not below the least weight
            double sum = 0.0;
#pragma unroll 1
            for (int b = c.from; b <= c.to; ++b) {
                if (s.upto_count[b + 1] == s.upto_count[b]) continue;
                const int shift = r.shift_of(b);
                if (tid == 0) s.mass[0] = 0;
                __syncthreads();
                uint64_t w = 0;
                r.each(s.low[b], s.high[b], [&](uint32_t key, uint32_t) {
                    const double v = r.weight(key);
                    w += v >= least_weight ? whole(v, shift) : 0;
                });
                if (w) atomicAdd((unsigned long long *)s.mass, (unsigned long long)w);
                __syncthreads();
                sum += (double)s.mass[0] * power2(-shift);
                __syncthreads();
            }
            kept = fmin(kept, s.upto_mass[c.from] + sum);
            __syncthreads();
            continue;
        }
        found = r.find(c.from, i == K, goal);
        // how many of that value are left
        const double need = i == K ? (double)(k - found.above_count) : ((i == D ? u * kept : goal) - found.above) / found.weight;
        if (i == D) {
            goal = need;
            break;
        }
        kept = fmin(kept, found.above + fmin(fmax(ceil(need), 1.0), (double)found.ties) * found.weight);
        __syncthreads();
    }
    const uint32_t token = r.nth_index(found.key, (uint32_t)fmin(fmax(floor(goal), 0.0), (double)(found.ties - 1)), found.ties);
    if (tid == 0) {
        p.tokens[row] = (int32_t)token;
        // the logarithm of the rounded share, and of what the rounding left
        const double share = found.weight / all;
        const float near = (float)share;
        p.logprobs[row] = h.greedy ? 0.0f : logf(near) + (float)(share - (double)near) / near;
    }
}

template __global__ void moe_sample_cells_kernel<LogitF32>(SampleParams);
template __global__ void moe_sample_cells_kernel<LogitBf16>(SampleParams);
template __global__ void moe_sample_cells_kernel<LogitF16>(SampleParams);
template __global__ void moe_sample_row_kernel<LogitF32>(SampleParams);
template __global__ void moe_sample_row_kernel<LogitBf16>(SampleParams);
template __global__ void moe_sample_row_kernel<LogitF16>(SampleParams);

}  // namespace moe
