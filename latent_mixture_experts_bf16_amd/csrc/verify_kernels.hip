// verify_kernels.hip -- verification of drafted tokens against the target's probabilities (gfx950).
//
// Probabilities and their running sums decide which whole token comes out, so they are held in
// 64 bits throughout: a running sum over 10^5 terms in 32 bits is off by more than the probability
// of most tokens.
//
//   stats  every row's logits once, a wave per chunk of 1024: largest, its index, sum of exponentials.
//          The walk needs the path's rows only, but does not know them before it has their sums, and one
//          row after another would leave most of the card idle.
//   walk   a workgroup per sequence: its rows' chunks joined, a wave a row; without draft
//          probabilities also each row's pick, after which the walk itself only compares tokens; with
//          them the drafted tokens' probabilities, after which it needs a whole row again only where a
//          draft is refused (the sum of max(p - S q, 0)) -- there it stops and leaves its state.
//   left   that sum, for all sequences that stopped, a wave per chunk; the last workgroup of a
//          sequence to finish goes on with its walk. A chain needs it once. Trees, whose later
//          siblings may be refused too, get it a few times; what then still waits is summed by the
//          last launch's own workgroup.
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

// The sums of max(p - S q, 0) are read by another workgroup of the same launch: written through to memory and read
// around the caches, as layer_items.h does for smaller types.
__device__ __forceinline__ void st_shared64(double *p, double v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ double ld_shared64(const double *p) {
    return __hip_atomic_load(const_cast<double *>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

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

// Temperature of a sequence: 1 / T, and whether all weight is on the largest logit. (An infinite T
// counts as the largest finite one, so that a logit of -infinity still weighs nothing.)
struct Heat {
    double inv;
    bool greedy;
};
__device__ __forceinline__ Heat heat(const VerifyParams &p, int b) {
    const float T = p.temperature ? p.temperature[b] : 1.0f;
    return {1.0 / (double)fminf(T, 3.4028234e38f), !(T > 0.0f)};
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
// Every kernel below calls this first, with all its threads.
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

// p of index i with logit x in a row whose statistics are r.
__device__ __forceinline__ double target(const LogitStat &r, const Heat &h, int i, float x) {
    if (h.greedy || r.best < 0) return i == max(r.best, 0) ? 1.0 : 0.0;
    return relative(x, r.top, h.inv) * r.sum;
}

template <typename L> __device__ __forceinline__ const typename L::T *logits_of(const VerifyParams &p, int row) {
    return (const typename L::T *)p.logits + (int64_t)row * p.logit_stride;
}

// ------------------------------------------------------------------ stats

// Largest logit of chunk c, in registers, and what the temperature asks for: its lowest index, or the sum.
__device__ __forceinline__ LogitStat chunk_stat(const Heat &h, int c, const float *x) {
    float top = -__builtin_inff();
#pragma unroll
    for (int k = 0; k < SHARE; ++k) top = fmaxf(top, x[k]);      // not a NaN: the other operand
    top = wave_max(top);
    LogitStat r = {0.0, top, -1};
    if (!(top > -__builtin_inff())) return r;
    r.best = c * VOCAB_CHUNK;
    if (h.greedy) {
        // the first quarter of the chunk that has the value, its first lane, that lane's first
#pragma unroll
        for (int k = SHARE - 4; k >= 0; k -= 4) {
            int at = 4;
#pragma unroll
            for (int e = 3; e >= 0; --e) at = x[k + e] == top ? e : at;
            const uint64_t some = __ballot(at < 4);
            if (some) {
                const int l = __builtin_ctzll(some);
                r.best = c * VOCAB_CHUNK + (k >> 2) * 256 + l * 4 + __builtin_amdgcn_readlane(at, l);
            }
        }
        return r;
    }
    double sum = 0.0;
    if (top == __builtin_inff())
#pragma unroll
        for (int k = 0; k < SHARE; ++k) sum += relative<true>(x[k], top, h.inv);
    else
#pragma unroll
        for (int k = 0; k < SHARE; ++k) sum += relative<false>(x[k], top, h.inv);
    r.sum = wave_sum(sum);
    return r;
}

// One chunk a wave: two, with the row's sequence looked up once, took 40 us instead of 37 over 64 x 5 rows of 100003.
// What bounds it is the vector instructions, some 20 of 64 bits an element (117 MB in 36 us, 3.3 TB/s; a copy moves
// 4.8): leaving out the search for the largest logit's index where T > 0 changed nothing that could be measured.
template <typename L> __global__ void __launch_bounds__(256) moe_verify_stats_kernel(VerifyParams p) {
    const int row = (int)(blockIdx.z * gridDim.y + blockIdx.y), lane = lane_id();
    const int c = (int)blockIdx.x * 4 + uniform((int)threadIdx.x >> 6);
    const bool some = row < p.rows && c < p.chunks;
    float x[SHARE];      // on its way before the table is filled and the row's sequence looked up
    if (some) load_share<L>(logits_of<L>(p, row), c, p.vocab, -__builtin_inff(), x);
    fill_exp_table();
    if (!some) return;
    int first = 0;
    // a row of no sequence is not walked; but where row_start is not ascending the walk may read it all the same
    const int b = seq_of_row(p.row_start, p.seqs, row, &first);
    const Heat h = b < 0 ? Heat{1.0, false} : heat(p, b);
    const LogitStat r = chunk_stat(h, c, x);
    if (lane == 0) p.chunk_stat[(int64_t)row * p.chunks + c] = r;
}

// ------------------------------------------------------------------ picking

// Statistics of a whole row from its chunks, the same in every lane. Each lane has a run of neighbouring chunks (at most
// 16), so that the lowest index is that of the first lane with the largest logit.
__device__ __forceinline__ LogitStat join_chunks(const VerifyParams &p, const Heat &h, int row) {
    const LogitStat *s = p.chunk_stat + (int64_t)row * p.chunks;
    const int per = (p.chunks + 63) >> 6, from = lane_id() * per, to = min(p.chunks, from + per);
    LogitStat r = {0.0, -__builtin_inff(), -1};
    for (int c = from; c < to; ++c)
        if (s[c].top > r.top) { r.top = s[c].top; r.best = s[c].best; }
    const float top = wave_max(r.top);
    const uint64_t have = __ballot(r.top == top && r.best >= 0);
    r.top = top;
    r.best = have ? __builtin_amdgcn_readlane(r.best, (int)__builtin_ctzll(have)) : -1;
    if (r.best < 0 || h.greedy) return r;
    for (int c = from; c < to; ++c) r.sum += s[c].sum * relative(s[c].top, r.top, h.inv);
    r.sum = 1.0 / wave_sum(r.sum);
    return r;
}

// The first index of row `row` whose running sum of weights passes u times the whole sum: of p where S is 0, else of
// max(p - S q, 0), whose sums by chunk are in p.left. By one wave.
template <typename L>
__device__ int pick_token(const VerifyParams &p, const LogitStat &r, const Heat &h, int b, int row, double S, float u) {
    if (S == 0.0 && (h.greedy || r.best < 0)) return max(r.best, 0);
    const LogitStat *s = p.chunk_stat + (int64_t)row * p.chunks;
    const double *left = p.left + (int64_t)b * p.chunks;
    const int lane = lane_id();
    auto chunk_weight = [&](int c) {
        if (c >= p.chunks) return 0.0;
        return S > 0.0 ? ld_shared64(left + c) : s[c].best < 0 ? 0.0 : s[c].sum * relative(s[c].top, r.top, h.inv) * r.sum;
    };
    // Each lane sums a run of neighbouring chunks (at most 16); then the lane, and the chunk of its run, whose running sum
    // is the first past the goal, or (a last rounding) the last with weight.
    const int per = (p.chunks + 63) >> 6;
    double mine = 0.0;
    for (int k = 0; k < per; ++k) mine += chunk_weight(lane * per + k);
    const double lanes = wave_scan(mine), goal = (double)u * lane_value(lanes, 63);
    // the first lane of those with weight whose sum passes; its place and the sum before it
    auto place = [&](double w, double upto, double *before) {
        const uint64_t some = __ballot(w > 0.0), over = __ballot(upto > goal) & some;
        if (!some) return -1;
        const int l = uniform(over ? __builtin_ctzll(over) : 63 - __builtin_clzll(some));
        if (l) *before = lane_value(upto, l - 1);
        return l;
    };
    double before = 0.0;
    int chunk = place(mine, lanes, &before);
    if (chunk < 0) return 0;
    chunk *= per;
    if (per > 1) {
        const double w = lane < per ? chunk_weight(chunk + lane) : 0.0;
        const int l = place(w, before + wave_scan(w), &before);
        chunk += max(l, 0);
    }
    // the same within it
    float x[SHARE], q[SHARE];
    load_share<L>(logits_of<L>(p, row), chunk, p.vocab, -__builtin_inff(), x);
    if (S > 0.0) load_share<LogitF32>(p.draft + (int64_t)row * p.draft_stride, chunk, p.vocab, 0.0f, q);
    double w[SHARE], upto[SHARE / 4];
#pragma unroll
    for (int k = 0; k < SHARE; ++k) {
        const int i = chunk * VOCAB_CHUNK + share_index(k);
        w[k] = i < p.vocab ? target(r, h, i, x[k]) : 0.0;
        if (S > 0.0) w[k] = fmax(w[k] - S * (double)q[k], 0.0);
    }
#pragma unroll
    for (int k = 0; k < SHARE; k += 4) upto[k / 4] = wave_scan((w[k] + w[k + 1]) + (w[k + 2] + w[k + 3]));
    int found = 0;
    bool past = false;
#pragma unroll
    for (int k = 0; k < SHARE; k += 4)
        if (!past) {
            const double own = (w[k] + w[k + 1]) + (w[k + 2] + w[k + 3]);
            double run = before + (upto[k / 4] - own);
            int first = -1, last = -1;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                run += w[k + e];
                if (w[k + e] > 0.0) last = e;
                if (w[k + e] > 0.0 && run > goal && first < 0) first = e;
            }
            const uint64_t over = __ballot(first >= 0), any = __ballot(last >= 0);
            past = over != 0;
            if (any) {
                const int l = past ? __builtin_ctzll(over) : 63 - __builtin_clzll(any);
                found = chunk * VOCAB_CHUNK + (k >> 2) * 256 + l * 4 + __shfl(past ? first : last, l);
            }
            before += lane_value(upto[k / 4], 63);
        }
    return found;
}

// ------------------------------------------------------------------ the walk

// Chunk c of max(p - S q, 0) over a row, summed by one wave.
template <typename L>
__device__ __forceinline__ double left_of_chunk(const VerifyParams &p, const LogitStat &r, const Heat &h, int row, int c,
                                                double S) {
    float x[SHARE], q[SHARE];
    load_share<L>(logits_of<L>(p, row), c, p.vocab, -__builtin_inff(), x);
    load_share<LogitF32>(p.draft + (int64_t)row * p.draft_stride, c, p.vocab, 0.0f, q);
    double sum = 0.0;
    if (h.greedy || r.best < 0 || r.top == __builtin_inff())
#pragma unroll
        for (int k = 0; k < SHARE; ++k)
            sum += fmax(target(r, h, c * VOCAB_CHUNK + share_index(k), x[k]) - S * (double)q[k], 0.0);
    else
#pragma unroll
        for (int k = 0; k < SHARE; ++k)
            sum += fmax(relative<false>(x[k], r.top, h.inv) * r.sum - S * (double)q[k], 0.0);
    return wave_sum(sum);
}

// 64 rows of a sequence, one a lane: as children, and (without draft probabilities) their own picks.
struct Kids {
    int parent, token, drawn;   // token -1: outside the vocabulary
    double p, lp;               // p of the token at its parent; its log, or that of the row's own pick
    float q, u;
    bool empty;                 // the parent's row (or the row itself, without draft probabilities) holds no logit
};
template <typename L>
__device__ __forceinline__ Kids load_kids(const VerifyParams &p, const Heat &h, int first, int n, int c) {
    Kids k = {-1, -1, -1, 0.0, 0.0, 0.0f, 0.0f, false};
    if (c >= n) return k;
    k.parent = c == 0 ? -1 : p.parent ? p.parent[first + c] : c - 1;
    const int x = p.tokens[first + c];
    if (c && x >= 0 && x < p.vocab) k.token = x;
    if (!p.draft) {
        k.drawn = p.pick[first + c];
        k.lp = p.token_p[first + c];
        k.empty = p.row_stat[first + c].best < 0;
    } else if (k.parent >= 0 && k.parent < c && k.token >= 0) {
        const int row = first + k.parent;
        const LogitStat r = p.row_stat[row];
        k.p = target(r, h, x, L::value(logits_of<L>(p, row)[x]));
        k.lp = log(k.p);
        k.q = p.draft[(int64_t)row * p.draft_stride + x];
        k.u = p.u_test[first + c];
        k.empty = r.best < 0;
    }
    return k;
}

// One wave walks on from st. true: the sequence is done; false: st waits for the sum of max(p - S q, 0).
template <typename L>
__device__ bool walk(const VerifyParams &p, const Heat &h, int b, int first, int n, WalkState &st) {
    const int lane = lane_id();
    int have = (st.after + 1) & ~63;
    if (have >= n) have = (n - 1) & ~63;
    Kids k = load_kids<L>(p, h, first, n, have + lane);
    // without draft probabilities the walk is not interrupted: it starts at row 0, in lane 0
    int drawn = __shfl(k.drawn, 0);
    double drawn_lp = __shfl(k.lp, 0);
    bool drawn_empty = __shfl((int)k.empty, 0);
    for (;;) {
        const int row = first + st.cur;
        int kid = -1;
        for (int c0 = (st.after + 1) & ~63; c0 < n; c0 += 64) {
            if (c0 != have) k = load_kids<L>(p, h, first, n, c0 + lane);
            have = c0;
            const bool is = c0 + lane > st.after && k.parent == st.cur;
            const uint64_t fits = __ballot(is && k.token >= 0 && (p.draft || k.token == drawn));
            const uint64_t wrong = __ballot(is && k.token < 0);
            if (wrong && (!fits || __builtin_ctzll(wrong) < __builtin_ctzll(fits)) && lane == 0)
                raise_flag(p.flags, MOE_FLAG_TOKEN);
            if (fits) {
                kid = c0 + __builtin_ctzll(fits);
                break;
            }
        }
        const int l = kid & 63;
        int token;
        double lp;
        bool empty;
        if (!p.draft) {
            token = drawn;
            lp = drawn_lp;
            empty = drawn_empty;
        } else if (kid >= 0) {
            const double px = __shfl(k.p, l), qx = (double)__shfl(k.q, l);
            if (!((double)__shfl(k.u, l) * qx * st.rest < fmax(px - st.S * qx, 0.0))) {
                st.S += st.rest;
                st.after = kid;
                return false;
            }
            token = __shfl(k.token, l);
            lp = __shfl(k.lp, l);
            empty = __shfl((int)k.empty, l);
        } else {
            const LogitStat r = p.row_stat[row];
            token = pick_token<L>(p, r, h, b, row, st.rest > 0.0 ? st.S : 0.0, p.u_pick[row]);
            lp = log(target(r, h, token, L::value(logits_of<L>(p, row)[token])));
            empty = r.best < 0;
        }
        if (lane == 0) {
            p.path[first + st.kept - 1] = st.cur;
            p.out_tokens[first + st.kept - 1] = token;
            p.logprobs[first + st.kept - 1] = (float)lp;
            if (empty) raise_flag(p.flags, MOE_FLAG_LOGITS);
        }
        if (kid < 0) break;
        drawn = __shfl(k.drawn, l);
        drawn_lp = __shfl(k.lp, l);
        drawn_empty = __shfl((int)k.empty, l);
        st.cur = st.after = kid;
        st.S = 0.0;
        st.rest = 1.0;
        ++st.kept;
    }
    if (lane == 0) p.n_keep[b] = st.kept;
    for (int i = st.kept + lane; i < n; i += 64) {
        p.path[first + i] = -1;
        p.out_tokens[first + i] = -1;
        p.logprobs[first + i] = 0.0f;
    }
    return true;
}

// A workgroup per sequence, a wave per row at a time. Bound by its chain of loads: 6 us for a chain of 5 over 131072
// logits, 16 us for 8 trees of up to 16 rows (each row's pick, 16 at once), 15 us for 64 chains of 6.
template <typename L> __global__ void __launch_bounds__(1024) moe_verify_walk_kernel(VerifyParams p) {
    const int b = (int)blockIdx.x, tid = (int)threadIdx.x, lane = lane_id(), wave = uniform(tid >> 6);
    fill_exp_table();
    int first = 0;
    const int n = seq_rows(p.row_start, b, p.rows, &first, p.flags);
    WalkState &out = p.state[b];
    if (tid == 0) p.arrived[b] = 0;
    if (b == 0 && tid == 1023) check_ends(p.row_start, p.seqs, p.rows, p.flags);
    if (n == 0) {
        if (tid == 0) {
            p.n_keep[b] = 0;
            out.pending = 0;
        }
        return;
    }
    const Heat h = heat(p, b);
    for (int i = wave; i < n; i += 16) {
        const int row = first + i;
        const LogitStat r = join_chunks(p, h, row);
        if (lane == 0) p.row_stat[row] = r;
        if (!p.draft) {
            const int t = pick_token<L>(p, r, h, b, row, 0.0, p.u_pick[row]);
            if (lane == 0) {
                p.pick[row] = t;
                p.token_p[row] = log(target(r, h, t, L::value(logits_of<L>(p, row)[t])));
            }
        }
    }
    __syncthreads();
    if (wave == 0) {
        WalkState st = {0.0, 1.0, 0, 1, 0, 0};
        st.pending = !walk<L>(p, h, b, first, n, st);
        if (lane == 0) out = st;
    }
}

// Workgroup (b, y): sums of 4 chunks of sequence b's row, if it waits for them. 64 rows of 100003 logits and draft
// probabilities (51 MB): 22 us, of which the last workgroups' walks and picks are about 10; one row of 131072: 13 us.
// Four waves at 128 registers leave four workgroups a compute unit (the walk spills some; eight waves at 151
// registers took 28 us), and the sums go round the caches (device fences in every wave: 128 us).
template <typename L> __global__ void __launch_bounds__(256, 4) moe_verify_left_kernel(VerifyParams p) {
    __shared__ int ours;
    const int b = (int)blockIdx.x, part = (int)blockIdx.y, lane = lane_id();
    const int wave = uniform((int)threadIdx.x >> 6);
    WalkState st = p.state[b];
    if (!st.pending) return;       // all threads of the workgroup, or none
    fill_exp_table();
    const int first = uniform(p.row_start[b]), n = uniform(p.row_start[b + 1]) - first;     // checked by the walk
    const Heat h = heat(p, b);
    double *left = p.left + (int64_t)b * p.chunks;
    const int c = part * 4 + wave;
    if (c < p.chunks) {
        const double v = left_of_chunk<L>(p, p.row_stat[first + st.cur], h, first + st.cur, c, st.S);
        if (lane == 0) st_shared64(left + c, v);
    }
    if (!last_arriver(p.arrived + b, gridDim.y, &ours)) return;
    for (;;) {
        if (wave == 0) {
            double sum = 0.0;
            for (int k = lane; k < p.chunks; k += 64) sum += ld_shared64(left + k);
            st.rest = wave_sum(sum);
            st.pending = !walk<L>(p, h, b, first, n, st);
            if (lane == 0) p.state[b] = st;
        }
        if (!p.last_round) return;
        __syncthreads();
        st = p.state[b];
        __syncthreads();
        if (!st.pending) return;
        for (int k = wave; k < p.chunks; k += 4) {
            const double s = left_of_chunk<L>(p, p.row_stat[first + st.cur], h, first + st.cur, k, st.S);
            if (lane == 0) st_shared64(left + k, s);
        }
        wait_vmem();
        __syncthreads();
    }
}

#define VERIFY_KERNELS(L)                                            \
    template __global__ void moe_verify_stats_kernel<L>(VerifyParams); \
    template __global__ void moe_verify_walk_kernel<L>(VerifyParams);  \
    template __global__ void moe_verify_left_kernel<L>(VerifyParams)
VERIFY_KERNELS(LogitF32);
VERIFY_KERNELS(LogitBf16);
VERIFY_KERNELS(LogitF16);

}  // namespace moe
