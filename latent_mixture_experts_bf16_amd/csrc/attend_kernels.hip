// attend_kernels.hip -- attention of a drafted step's rows over the paged cache (gfx950).
//
// One pass over the cached keys and values with a running maximum and sum of the softmax. The
// queries of a sequence that read one key head (rows x group of them) are cut into query tiles of MQ,
// the tokens into tiles of 64; the tiles of all (sequence, key head, query tile), in this order, make
// one long row of work that is cut into equal ranges, one per workgroup, whatever the lengths are: a
// range may end inside an item (one sequence, head and query tile), whose parts are then joined by
// a second, small launch. Lengths are known on the device only, so each workgroup finds its range
// itself, from row_start and len.
//
// A workgroup has four waves. Each loads 16 tokens' keys and values of a tile into registers while
// the tile before it is computed from LDS (two buffers, one barrier a tile). Scores are the
// MFMA product K Q^T, so that a query is a column: the four lanes that share a column hold its
// scores and its sums, and the scores lie in the registers as the product V^T P^T takes them. V is
// transposed on its way out of LDS. The waves lie side by side along the queries (QW of them, each with
// 16 NQ queries) and along the tokens (4 / QW); the latter are joined through LDS at an item's end.
//
// Long caches are bound by reading them once: 16 chains of up to 5 rows over up to 32700 tokens (40 heads on 8
// of 128, 1.56 GB) take 295 us, 5.3 TB/s, and fetch 1.002 of their bytes. 8 trees over up to 8200 (162 MB): 39 us,
// 4.1 TB/s, and 8 us for the join. 64-row trees over 4100 (32 heads on 4 of 64): 26 us, in which the vector units
// are busy for 8; the rest is the start and end of two items a workgroup. One row over 777: 8 us, a chain of loads
// (starts and lengths, page, keys), and 6 us for the join. LDS reads and writes meet no bank conflicts.
#include "drafted_items.h"

namespace moe {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

template <bool F16> __device__ __forceinline__ f32x4 mfma32(s16x8 a, s16x8 b, f32x4 c) {
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                      0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
}
template <bool F16> __device__ __forceinline__ f32x4 mfma16(s16x4 a, s16x4 b, f32x4 c) {
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(f16x4, a), __builtin_bit_cast(f16x4, b), c, 0, 0,
                                                     0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(a, b, c, 0, 0, 0);
}

// Two elements rounded to the cache's type (to nearest even), the first in the low half: results, and the probabilities for
// the product with V, since the matrix instructions take both operands in one type (fp32 ones do a sixteenth of the
// work a cycle). Their sum is of the unrounded ones, in fp32. Against 64 bits the rms error of one row's result over 777
// tokens is then 0.0020 of its size in bf16, where products of fp32 probabilities, rounded once, leave 0.0017.
template <bool F16> __device__ __forceinline__ uint32_t pack2(float a, float b) {
    const f32x2 v = {a, b};
    if constexpr (F16)
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
    else
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// Whether one of two packed elements is infinite or NaN.
template <bool F16> __device__ __forceinline__ int odd2(uint32_t v) {
    constexpr uint32_t E = F16 ? 0x7C00u : 0x7F80u;
    return (int)((v & E) == E) | (int)((v >> 16 & E) == E);
}

// The 4 x 16 elements that 16 lanes' addresses name (four lanes a row of 16), transposed: lane i
// gets column i, one element of each row.
__device__ __forceinline__ s16x4 read_columns(const uint16_t *lds) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)lds);
}

// The largest value of the four lanes that share a column.
__device__ __forceinline__ float across_quads_max(float v) {
    const uint32_t x = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    const uint32_t y = __float_as_uint(v);
    const auto q = __builtin_amdgcn_permlane16_swap(y, y, false, false);
    return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

constexpr int low_bit(int v) { return v & -v; }
constexpr int least(int a, int b) { return a < b ? a : b; }
constexpr int log2_of(int v) { return v <= 1 ? 0 : 1 + log2_of(v / 2); }

// Where piece c (16 bytes) of token t lies in a group of 16 tokens in LDS, in elements. Rows of D
// elements start on few different banks where D is a multiple of 16 banks' worth; the pieces are
// exchanged within a row by the token's number, so that the 16 rows that a K read takes at one piece,
// and the 8 that a V read takes at one 32-byte unit, lie on different banks.
template <int D> __device__ __forceinline__ int k_place(int t, int c) {
    constexpr int P = least(16, low_bit(D / 8)), SH = log2_of(16 / P);
    return t * D + (c ^ ((t >> SH) & (P - 1))) * 8;
}
template <int D> __device__ __forceinline__ int v_unit(int t, int u) {
    constexpr int P = least(8, low_bit(D / 16)), SH = log2_of(8 / P);
    return t * D + (u ^ ((t >> SH) & (P - 1))) * 16;
}

// Work of sequence b: rows, tokens, and how they are cut. An item counts as its tiles and ITEM_COST more,
// for its start and end, in which no tile is in flight: so a range of many short items takes no longer
// than one of a long one (an empty sequence beside seven of 8200 tokens: 108 -> 58 us
// at 16 rows).
constexpr int ITEM_COST = 3;
struct SeqWork {
    int first, n, len, end, mts, tts;
    int64_t units;
};
template <int MQ> __device__ __forceinline__ SeqWork seq_work(const AttendParams &p, int b, bool tell) {
    SeqWork w;
    const int s = p.row_start[b], e = p.row_start[b + 1], t = p.c.len[b];
    const bool rows_bad = s < 0 || e < s || e > p.rows, len_bad = t < 0 || t > p.c.cap;
    w.first = rows_bad ? 0 : s;
    w.n = rows_bad ? 0 : e - s;
    w.len = t < 0 ? 0 : min(t, p.c.cap);
    const bool past = w.len + (int64_t)w.n > p.c.cap;
    w.end = past ? p.c.cap : w.len + w.n;
    w.mts = (int)(((int64_t)w.n * p.group + MQ - 1) / MQ);
    w.tts = (int)(((int64_t)w.end + 63) >> 6);
    w.units = (int64_t)w.mts * (w.tts + ITEM_COST) * p.c.heads;
    if (tell) {
        const uint32_t f = (rows_bad ? MOE_FLAG_ROWS : 0) | (len_bad ? MOE_FLAG_LEN : 0) | (past ? MOE_FLAG_PAGE : 0);
        if (f) raise_flag(p.c.flags, f);
    }
    return w;
}

// a / b, neither negative: in 32 bits where both fit (a 64-bit division takes some 150 instructions, and a short
// call has five of them in a row before its first load).
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

struct PlanLds {
    int64_t wave[4];
    int64_t base;
    int b;
};

// All units of work, and the range of them that this workgroup has: [x, xe), starting in sequence b
// whose units start at base. false: none. Each thread sums a run of sequences.
template <int MQ>
__device__ __forceinline__ bool find_range(const AttendParams &p, PlanLds &s, int *w, int64_t *total, int64_t *groups,
                                           int64_t *x, int64_t *xe, int *b, int64_t *base) {
    const int tid = (int)threadIdx.x, lane = lane_id(), wave = tid >> 6, per = (p.c.seqs + 255) >> 8;
    const bool tell = blockIdx.x == 0;
    int64_t sum = 0;
    for (int k = 0; k < per; ++k) {
        const int q = tid * per + k;
        if (q < p.c.seqs) sum += seq_work<MQ>(p, q, tell).units;
    }
    if (tell && tid == 0 && (p.row_start[0] != 0 || p.row_start[p.c.seqs] != p.rows))
        raise_flag(p.c.flags, MOE_FLAG_ROWS);
    int64_t run = sum;
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t u = __shfl_up(run, d);
        if (lane >= d) run += u;
    }
    if (lane == 63) s.wave[wave] = run;
    __syncthreads();
    int64_t before = run - sum, N = 0;
    for (int k = 0; k < 4; ++k) {
        if (k < wave) before += s.wave[k];
        N += s.wave[k];
    }
    const int64_t G = N < (int64_t)gridDim.x ? N : (int64_t)gridDim.x;
    // a full grid: neighbours in the order of work, who share queries' keys, on one XCD (workgroups go
    // round the eight of them)
    const int id = (int)blockIdx.x, at = G == (int64_t)gridDim.x ? (id & 7) * (int)(gridDim.x >> 3) + (id >> 3) : id;
    *w = at;
    *total = N;
    *groups = G;
    if (at >= G) return false;
    *x = divide(at * N, G);
    *xe = divide((at + 1) * N, G);
    if (sum && before <= *x && *x < before + sum) {
        int q = tid * per;
        for (int64_t t; q + 1 < p.c.seqs && *x >= before + (t = seq_work<MQ>(p, q, false).units); ++q) before += t;
        s.b = q;
        s.base = before;
    }
    __syncthreads();
    *b = uniform(s.b);
    *base = s.base;
    return true;
}

template <bool F16, int D, int NQ, int QW>
__global__ void __launch_bounds__(256, attend_blocks(D, 16 * NQ * QW)) moe_attend_kernel(AttendParams p) {
    constexpr int MQ = 16 * NQ * QW, TG = 4 / QW, NS = QW;     // a wave's 16-token groups in a tile: 4 / TG
    constexpr int KS = (D + 31) / 32, DB = D / 16, PIECES = 2 * D, LOADS = (PIECES + 63) / 64;
    constexpr bool RAGGED = PIECES % 64 != 0;
    constexpr int GE = 16 * D;                                 // elements of a group of 16 tokens
    __shared__ __align__(16) uint16_t lds[2][2][4 * GE];
    __shared__ float sm[4][16 * NQ], sl[4][16 * NQ];
    __shared__ __align__(16) int note[2][4];                   // per buffer and group: 1 page bad, 2 V not finite
    __shared__ PlanLds plan;
    const int tid = (int)threadIdx.x, lane = lane_id(), wave = uniform(tid >> 6), wq = wave % QW, wt = wave / QW;
    const int col = lane & 15, quad = lane >> 4;

    int w, b;
    int64_t total, groups, x, xe, base;
    const bool any = find_range<MQ>(p, plan, &w, &total, &groups, &x, &xe, &b, &base);
    AttendPart &part = p.parts[w];
    if (tid == 0) part.count = 0;
    if (!any) return;

    // this lane's pieces of a group of 16 tokens: where they come from and where they go
    uint32_t ko[LOADS], vo[LOADS];
    int kp[LOADS], vp[LOADS], pt[LOADS];
#pragma unroll
    for (int k = 0; k < LOADS; ++k) {
        const int at = min(k * 64 + lane, PIECES - 1), t = at / (D / 8), c = at % (D / 8);
        pt[k] = t;
        ko[k] = (uint32_t)(t * p.c.k.slot + c * 8) * 2;
        vo[k] = (uint32_t)(t * p.c.v.slot + c * 8) * 2;
        kp[k] = wave * GE + k_place<D>(t, c);
        vp[k] = wave * GE + v_unit<D>(t, c >> 1) + (c & 1) * 8;
    }

    while (x < xe) {
        SeqWork sq = seq_work<MQ>(p, b, false);
        if (x >= base + sq.units) {
            base += sq.units;
            if (++b >= p.c.seqs) break;     // cannot be, unless lengths change while this runs
            continue;
        }
        const int first = uniform(sq.first), n = uniform(sq.n), len = uniform(sq.len), end = uniform(sq.end);
        const int tts = uniform(sq.tts), mts = uniform(sq.mts), all_units = tts + ITEM_COST;
        const int64_t rel = x - base, item = divide(rel, all_units);
        const int u_from = uniform((int)(rel - item * all_units));
        const int u_to = uniform((int)min((int64_t)all_units, u_from + (xe - x)));
        const int t_from = max(0, u_from - ITEM_COST), t_to = u_to - ITEM_COST;
        const int h = uniform((int)divide(item, mts)), mt = uniform((int)(item - (int64_t)h * mts));
        x += u_to - u_from;
        if (t_to <= t_from) continue;
        const int queries = min((int64_t)MQ, (int64_t)n * p.group - (int64_t)mt * MQ);
        // rows without a mask see no token after their own: tiles past the last row's are not read
        int t_last = t_to;
        if (!p.mask) {
            const int i_last = (mt * MQ + queries - 1) / p.group;
            t_last = min(t_to, (int)(((int64_t)len + i_last + 64) >> 6));
        }

        s16x8 qf[NQ][KS];
        uint64_t mask[NQ];
        int late[NQ];                     // the last row past the 64th that is seen
        f32x4 o[NQ][DB];
        float m[NQ], l[NQ];
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
            const int q = (wq * NQ + u) * 16 + col, z = mt * MQ + q;
            const bool ok = q < queries;
            const int i = ok ? z / p.group : 0, g = ok ? z - i * p.group : 0;
            const uint16_t *src = p.q + (int64_t)(first + i) * p.q_stride + (int64_t)(h * p.group + g) * D;
            // without masks: the rows up to its own
            mask[u] = p.mask ? p.mask[first + i] : i < 63 ? (2ull << i) - 1 : ~0ull;
            late[u] = p.mask ? -1 : i;
#pragma unroll
            for (int k = 0; k < KS; ++k)
                qf[u][k] = ok && k * 32 + quad * 8 < D ? *(const s16x8 *)(src + k * 32 + quad * 8) ^ p.q_sign
                                                       : s16x8{0, 0, 0, 0, 0, 0, 0, 0};
            m[u] = -__builtin_inff();
            l[u] = 0.0f;
#pragma unroll
            for (int d = 0; d < DB; ++d) o[u][d] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        // whether the query of this lane's column sees token t (without branches)
        auto sees = [&](int u, int t) {
            const int j = t - len;
            return (int)(j < 0) | ((int)(j < 64) & (int)(mask[u] >> (j & 63)) & 1) | ((int)(j >= 64) & (int)(j <= late[u]));
        };

        const int32_t *table = p.c.table + b * p.c.table_stride;
        u32x4 kr[LOADS], vr[LOADS];
        // the page of this wave's group of a tile; looked up a tile before it is needed
        auto page_of = [&](int tile) {
            const int64_t t = (int64_t)tile * 64 + wave * 16;      // a tile past the last may lie past 2^31
            return t < end ? table[(int)t / p.c.page] : -1;
        };
        // A group without a page reads the first one's slots instead: its scores are masked and its values zeroed.
        auto load = [&](int tile, int page) {
            const int t = tile * 64 + wave * 16;
            const bool ok = t < end && page >= 0 && page < p.c.pages;
            if (!ok && t < end && lane == 0) raise_flag(p.c.flags, MOE_FLAG_PAGE);
            const int slot = t % p.c.page;
            const int64_t pg = ok ? page : 0;
            const char *kb = (const char *)(p.c.k.p + pg * p.c.k.page + slot * p.c.k.slot + h * p.c.k.head);
            const char *vb = (const char *)(p.c.v.p + pg * p.c.v.page + slot * p.c.v.slot + h * p.c.v.head);
#pragma unroll
            for (int k = 0; k < LOADS; ++k) kr[k] = *(const u32x4 *)(kb + ko[k]);
#pragma unroll
            for (int k = 0; k < LOADS; ++k) vr[k] = *(const u32x4 *)(vb + vo[k]);
            return ok || t >= end;
        };

        int page = t_from < t_last ? uniform(page_of(t_from)) : 0;
        bool good = true;
        if (t_from < t_last) {
            good = load(t_from, page);
            page = page_of(t_from + 1);
        }
        for (int tile = t_from; tile < t_last; ++tile) {
            const int buf = tile & 1, t0 = tile * 64;
            uint16_t *const kl = lds[buf][0], *const vl = lds[buf][1];
            int told = good ? 0 : 1;
            if (t0 + wave * 16 + 16 > len || !good) {
                // the step's own tokens: slots behind the last hold anything, and are zeroed; a value that is not finite
                // must not reach the rows that do not see it
                int odd = 0;
#pragma unroll
                for (int k = 0; k < LOADS; ++k) {
                    const int t = t0 + wave * 16 + pt[k];
                    if (t >= end || !good) vr[k] = u32x4{0, 0, 0, 0};
                    odd |= (int)(t >= len) & (odd2<F16>(vr[k].x) | odd2<F16>(vr[k].y) | odd2<F16>(vr[k].z) | odd2<F16>(vr[k].w));
                }
                if (__any(odd)) told |= 2;
            }
#pragma unroll
            for (int k = 0; k < LOADS; ++k)
                if (!RAGGED || k * 64 + lane < PIECES) {
                    *(u32x4 *)(kl + kp[k]) = kr[k];
                    *(u32x4 *)(vl + vp[k]) = vr[k];
                }
            if (lane == 0) note[buf][wave] = told;
            if (tile + 1 < t_last) {
                good = load(tile + 1, uniform(page));
                page = page_of(tile + 2);
            }
            __syncthreads();
            const int4 notes = *(const int4 *)note[buf];
            const int all = uniform(notes.x | notes.y << 4 | notes.z << 8 | notes.w << 12);   // four bits a group
            const bool special = t0 + 64 > len || all;

            f32x4 s[NS][NQ];
#pragma unroll
            for (int a = 0; a < NS; ++a) {
                const uint16_t *kg = kl + (wt * NS + a) * GE;
#pragma unroll
                for (int u = 0; u < NQ; ++u) s[a][u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    // The last 32 dims may be 16: the other half's pieces are zero on both sides. (A shorter MFMA for
                    // them at the end of a chain of longer ones, into the same sums, gave wrong ones.)
                    s16x8 f = {0, 0, 0, 0, 0, 0, 0, 0};
                    if (k * 32 + 32 <= D || quad < 2) f = *(const s16x8 *)(kg + k_place<D>(col, k * 4 + quad));
#pragma unroll
                    for (int u = 0; u < NQ; ++u) s[a][u] = mfma32<F16>(f, qf[u][k], s[a][u]);
                }
            }
            if (special) {
#pragma unroll
                for (int a = 0; a < NS; ++a) {
                    const int g = wt * NS + a, good_page = ~(all >> 4 * g);
#pragma unroll
                    for (int u = 0; u < NQ; ++u)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int t = t0 + g * 16 + quad * 4 + r;
                            s[a][u][r] = sees(u, t) & (int)(t < end) & good_page & 1 ? s[a][u][r] : -__builtin_inff();
                        }
                }
            }
            uint32_t pr[NS][NQ][2];
#pragma unroll
            for (int u = 0; u < NQ; ++u) {
                float top = -__builtin_inff();
#pragma unroll
                for (int a = 0; a < NS; ++a)
#pragma unroll
                    for (int r = 0; r < 4; ++r) top = fmaxf(top, s[a][u][r]);
                top = fmaxf(m[u], across_quads_max(top) * p.scale_log2);
                const float from = top == -__builtin_inff() ? 0.0f : top;
                if (__any(top > m[u])) {
                    const float keep = __builtin_amdgcn_exp2f(m[u] - from);
                    l[u] *= keep;
#pragma unroll
                    for (int d = 0; d < DB; ++d) o[u][d] *= keep;
                }
                m[u] = top;
#pragma unroll
                for (int a = 0; a < NS; ++a) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        s[a][u][r] = __builtin_amdgcn_exp2f(fmaf(s[a][u][r], p.scale_log2, -from));
                        l[u] += s[a][u][r];
                    }
                    pr[a][u][0] = pack2<F16>(s[a][u][0], s[a][u][1]);
                    pr[a][u][1] = pack2<F16>(s[a][u][2], s[a][u][3]);
                }
            }
            if (all & 0x2222) {
                // values that are not finite: added for the rows that see them, then taken out of the tile, so that
                // no probability of 0 meets them
                for (int t = 0; t < NS * 16; ++t) {
                    const int tt = wt * NS * 16 + t;
                    const uint16_t *row = vl + (tt >> 4) * GE;
                    if (t0 + tt < len) continue;
                    int see[NQ];
#pragma unroll
                    for (int u = 0; u < NQ; ++u) see[u] = sees(u, t0 + tt);
#pragma unroll
                    for (int d = 0; d < DB; ++d) {
                        const uint2 e = *(const uint2 *)(row + v_unit<D>(tt & 15, d) + quad * 4);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const uint32_t v = (r < 2 ? e.x : e.y) >> (r & 1) * 16 & 0xFFFFu;
                            const float add = odd2<F16>(v) ? to_f32<F16>(v) : 0.0f;
#pragma unroll
                            for (int u = 0; u < NQ; ++u) o[u][d][r] += see[u] ? add : 0.0f;
                        }
                    }
                }
                __syncthreads();
                for (int e = tid; e < 4 * GE; e += 256)
                    if (t0 + e / D >= len && odd2<F16>(vl[e])) vl[e] = 0;
                __syncthreads();
            }
            const int vt = quad * 4 + (col >> 2);
#pragma unroll
            for (int d = 0; d < DB; ++d) {
                const uint16_t *at = vl + wt * NS * GE + v_unit<D>(vt, d) + (col & 3) * 4;
                if constexpr (NS == 1) {
                    const s16x4 f = read_columns(at);
#pragma unroll
                    for (int u = 0; u < NQ; ++u) {
                        const uint2 q2 = make_uint2(pr[0][u][0], pr[0][u][1]);
                        o[u][d] = mfma16<F16>(f, __builtin_bit_cast(s16x4, q2), o[u][d]);
                    }
                } else {
#pragma unroll
                    for (int a = 0; a < NS; a += 2) {
                        const s16x4 f0 = read_columns(at + a * GE), f1 = read_columns(at + (a + 1) * GE);
                        const s16x8 f = __builtin_shufflevector(f0, f1, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
                        for (int u = 0; u < NQ; ++u) {
                            const uint4 q4 = make_uint4(pr[a][u][0], pr[a][u][1], pr[a + 1][u][0], pr[a + 1][u][1]);
                            o[u][d] = mfma32<F16>(f, __builtin_bit_cast(s16x8, q4), o[u][d]);
                        }
                    }
                }
            }
        }

        // join the waves along the tokens, and write the item, or this range's part of it
        __syncthreads();
        constexpr int PU = least(16, low_bit(D / 4));
        float *const stage = (float *)lds;
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
            l[u] += __shfl_xor(l[u], 16);
            l[u] += __shfl_xor(l[u], 32);
            const int q = u * 16 + col;
            if (quad == 0) { sm[wave][q] = m[u]; sl[wave][q] = l[u]; }
#pragma unroll
            for (int d = 0; d < DB; ++d)
                *(f32x4 *)(stage + (wave * 16 * NQ + q) * D + ((d * 4 + quad) ^ (q & (PU - 1))) * 4) = o[u][d];
        }
        __syncthreads();
        const bool whole = t_from == 0 && t_to == tts;
        const int slot = 2 * w + (t_from == 0 ? 1 : 0);
        float *const pm = p.part_stat + (int64_t)slot * 2 * MQ, *const po = p.part_sum + (int64_t)slot * MQ * D;
        for (int at = tid; at < queries * (D / 8); at += 256) {
            const int q = at / (D / 8), d8 = at % (D / 8), ql = q % (16 * NQ), wv = q / (16 * NQ);
            float top = sm[wv][ql];
#pragma unroll
            for (int a = 1; a < TG; ++a) top = fmaxf(top, sm[a * QW + wv][ql]);
            const float from = top == -__builtin_inff() ? 0.0f : top;
            float sum = 0.0f;
            f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
#pragma unroll
            for (int a = 0; a < TG; ++a) {
                const int v = a * QW + wv;
                const float f = __builtin_amdgcn_exp2f(sm[v][ql] - from);
                const float *src = stage + (v * 16 * NQ + ql) * D;
                sum += f * sl[v][ql];
                lo += f * *(const f32x4 *)(src + ((2 * d8) ^ (ql & (PU - 1))) * 4);
                hi += f * *(const f32x4 *)(src + ((2 * d8 + 1) ^ (ql & (PU - 1))) * 4);
            }
            if (whole) {
                const int z = mt * MQ + q, i = z / p.group, g = z - i * p.group;
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                const f32x4 a = sum == 0.0f ? f32x4{0.f, 0.f, 0.f, 0.f} : lo * inv;
                const f32x4 c = sum == 0.0f ? f32x4{0.f, 0.f, 0.f, 0.f} : hi * inv;
                *(uint4 *)(p.out + (int64_t)(first + i) * p.out_stride + (int64_t)(h * p.group + g) * D + d8 * 8) =
                    make_uint4(pack2<F16>(a[0], a[1]), pack2<F16>(a[2], a[3]), pack2<F16>(c[0], c[1]), pack2<F16>(c[2], c[3]));
            } else {
                if (d8 == 0) { pm[q] = top; pm[MQ + q] = sum; }
                *(f32x4 *)(po + q * D + d8 * 8) = lo;
                *(f32x4 *)(po + q * D + d8 * 8 + 4) = hi;
            }
        }
        if (!whole && t_from == 0 && tid == 0) {
            // the first part of a cut item: the ranges that hold it are this one and the next ones
            const int64_t last = x - u_to + all_units;
            part.first = first;
            part.mt = mt;
            part.head = h;
            part.queries = queries;
            part.count = (int)min(divide(last * groups - 1, total), groups - 1) - w + 1;
        }
        __syncthreads();
    }
}

// What some parts of one query sum to.
struct JoinSum {
    float top, sum;   // sum: this lane's share
    f32x4 o;
};

// One wave adds parts [lo, hi) of query q of the item that begins in range w (part a lies in slot 1 of
// range w, then in slot 0 of the ranges after it). Maxima and sums lie along the lanes, 64 parts a
// step; then the lanes lie along the head (D / 4 of them) and along the parts.
template <int D> __device__ __forceinline__ JoinSum join_parts(const AttendParams &p, int w, int q, int lo, int hi) {
    constexpr int U = D / 4, PL = 64 / U;
    const int lane = lane_id(), k = lane / U, u = lane % U, MQ = p.tile_queries;
    JoinSum j = {-__builtin_inff(), 0.0f, {0.f, 0.f, 0.f, 0.f}};
    for (int a0 = lo; a0 < hi; a0 += 64) {
        const int a = a0 + lane, here = min(64, hi - a0);
        float m = -__builtin_inff(), s = 0.0f;
        if (a < hi) {
            const int64_t slot = 2 * (int64_t)(w + a) + (a == 0);
            m = p.part_stat[slot * 2 * MQ + q];
            s = p.part_stat[slot * 2 * MQ + MQ + q];
        }
        float best = fmaxf(j.top, m);
        for (int d = 32; d; d >>= 1) best = fmaxf(best, __shfl_xor(best, d));
        const float from = best == -__builtin_inff() ? 0.0f : best;
        const float old = __builtin_amdgcn_exp2f(j.top - from), f = __builtin_amdgcn_exp2f(m - from);
        j.sum = j.sum * old + f * s;
        j.o *= old;
        j.top = best;
        for (int i0 = 0; i0 < here; i0 += 8 * PL) {
            f32x4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {       // all on their way before the first is used
                const int at = i0 + i * PL + k;
                const int64_t slot = 2 * (int64_t)(w + a0 + at) + (a0 + at == 0);
                v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (k < PL && at < here) v[i] = *(const f32x4 *)(p.part_sum + (slot * MQ + q) * D + u * 4);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int at = i0 + i * PL + k;
                const float g = __shfl(f, at & 63);
                j.o += (k < PL && at < here ? g : 0.0f) * v[i];
            }
        }
    }
    const f32x4 own = j.o;
    for (int i = 1; i < PL; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) j.o[e] += __shfl(own[e], (lane + i * U) & 63);
    for (int d = 32; d; d >>= 1) j.sum += __shfl_xor(j.sum, d);
    return j;     // o in the lanes below U
}

// Joins the parts of cut items. Every workgroup lists the (item, query) pairs that the ranges' records
// name; a pair is one wave's work, or, where there are no more of them than workgroups (few queries
// over a long cache: many parts each), one workgroup's, its waves taking a quarter of the parts each.
template <bool F16, int D>
__global__ void __launch_bounds__(256) moe_attend_join_kernel(AttendParams p) {
    constexpr int U = D / 4;
    __shared__ int start[ATTEND_MOST_RANGES + 1], wave_sum[4];
    __shared__ float sm[4], ss[4];
    __shared__ f32x4 so[4][U];
    const int tid = (int)threadIdx.x, lane = lane_id(), wave = uniform(tid >> 6), per = p.ranges >> 8;
    int mine = 0, n[ATTEND_MOST_RANGES / 256];
#pragma unroll
    for (int k = 0; k < ATTEND_MOST_RANGES / 256; ++k) {
        n[k] = 0;
        if (k < per) {
            const AttendPart &part = p.parts[tid * per + k];
            n[k] = part.count > 0 ? part.queries : 0;
        }
        mine += n[k];
    }
    int run = mine;
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(run, d);
        if (lane >= d) run += v;
    }
    if (lane == 63) wave_sum[wave] = run;
    __syncthreads();
    int at = run - mine, total = 0;
    for (int k = 0; k < 4; ++k) {
        if (k < wave) at += wave_sum[k];
        total += wave_sum[k];
    }
#pragma unroll
    for (int k = 0; k < ATTEND_MOST_RANGES / 256; ++k)
        if (k < per) {
            start[tid * per + k] = at;
            at += n[k];
        }
    if (tid == 0) start[p.ranges] = total;
    __syncthreads();
    const bool shared = total <= (int)gridDim.x;
    const int step = shared ? (int)gridDim.x : (int)gridDim.x * 4;
    for (int i = shared ? (int)blockIdx.x : (int)blockIdx.x * 4 + wave; i < total; i += step) {
        int lo = 0, hi = p.ranges;       // the last range that starts at or before pair i: the one that holds it
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start[mid] <= i) lo = mid; else hi = mid;
        }
        const int w = uniform(lo), q = uniform(i - start[lo]);
        const AttendPart part = p.parts[w];
        JoinSum j;
        if (shared) {
            const int each = (part.count + 3) >> 2;
            j = join_parts<D>(p, w, q, min(part.count, wave * each), min(part.count, (wave + 1) * each));
            if (lane < U) so[wave][lane] = j.o;
            if (lane == 0) { sm[wave] = j.top; ss[wave] = j.sum; }
            __syncthreads();
            const float best = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3])), from = best == -__builtin_inff() ? 0.0f : best;
            j.o = f32x4{0.f, 0.f, 0.f, 0.f};
            j.sum = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float f = __builtin_amdgcn_exp2f(sm[k] - from);
                j.sum += f * ss[k];
                if (lane < U) j.o += f * so[k][lane];
            }
        } else {
            j = join_parts<D>(p, w, q, 0, part.count);
        }
        if (lane < U && (!shared || wave == 0)) {
            const int z = part.mt * p.tile_queries + q, row = z / p.group, g = z - row * p.group;
            const float inv = 1.0f / j.sum;
            const f32x4 r = j.sum == 0.0f ? f32x4{0.f, 0.f, 0.f, 0.f} : j.o * inv;
            *(uint2 *)(p.out + (int64_t)(part.first + row) * p.out_stride + (int64_t)(part.head * p.group + g) * D + lane * 4) =
                make_uint2(pack2<F16>(r[0], r[1]), pack2<F16>(r[2], r[3]));
        }
        if (shared) __syncthreads();
    }
}

#define ATTEND_KERNELS(D)                                              \
    template __global__ void moe_attend_kernel<false, D, 1, 1>(AttendParams); \
    template __global__ void moe_attend_kernel<false, D, 2, 1>(AttendParams); \
    template __global__ void moe_attend_kernel<false, D, 2, 2>(AttendParams); \
    template __global__ void moe_attend_kernel<false, D, 2, 4>(AttendParams); \
    template __global__ void moe_attend_kernel<true, D, 1, 1>(AttendParams);  \
    template __global__ void moe_attend_kernel<true, D, 2, 1>(AttendParams);  \
    template __global__ void moe_attend_kernel<true, D, 2, 2>(AttendParams);  \
    template __global__ void moe_attend_kernel<true, D, 2, 4>(AttendParams);  \
    template __global__ void moe_attend_join_kernel<false, D>(AttendParams);  \
    template __global__ void moe_attend_join_kernel<true, D>(AttendParams)
ATTEND_KERNELS(32);
ATTEND_KERNELS(64);
ATTEND_KERNELS(80);
ATTEND_KERNELS(96);
ATTEND_KERNELS(112);
ATTEND_KERNELS(128);
ATTEND_KERNELS(192);
ATTEND_KERNELS(256);

}  // namespace moe
