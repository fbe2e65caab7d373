// drafted_plan.h -- launch parameters of the drafted decode step's operators, shared by host
// and device, and the error helper the two host files share.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_drafted.h"

namespace moe {

// Sets this thread's message (moe_latent_last_error) and returns code.
int api_fail(int code, const char *fmt, ...);
void api_clear();

struct KvView {
    const uint16_t *p;
    int64_t page, slot, head;   // strides in elements
};

struct CacheParams {
    KvView k, v;
    const int32_t *table, *len;
    uint32_t *flags;
    int64_t table_stride;
    int32_t pages, page, heads, dim, seqs;
    int32_t cap;                // tokens the table has room for (at most 2^31 - 64)
};

struct RopeParams {
    CacheParams c;
    const double *freqs;
    int32_t pairs;
    float magnitude;
    const uint16_t *q, *kn, *vn;
    uint16_t *qo;
    int64_t q_stride, k_stride, v_stride, qo_stride;
    const int32_t *row_start, *positions;
    int32_t rows, q_heads;
};

// Workgroups of the attention kernel that a compute unit holds at once: by LDS (two buffers of 64
// tokens take 512 dim bytes of 160 KB) and by the registers of a wave's queries and sums.
constexpr int attend_blocks(int dim, int queries) {
    return dim <= 64 ? (queries == 16 ? 4 : queries == 128 ? 2 : 3) : dim <= 96 ? 3 : dim <= 128 ? 2 : 1;
}

constexpr int COMPUTE_UNITS = 256;      // of an MI355X: workspaces are sized without asking a device
constexpr int ATTEND_MOST_RANGES = COMPUTE_UNITS * attend_blocks(32, 16);

// The first part of an item of attention work that was cut between workgroups: written by the range
// that holds it, read by the launch that joins the parts.
struct AttendPart {
    int32_t count, first, mt, head, queries, pad[3];   // count 0: this range starts no cut item
};

struct AttendParams {
    CacheParams c;
    const uint16_t *q;
    uint16_t *out;
    int64_t q_stride, out_stride;
    const int32_t *row_start;
    const uint64_t *mask;
    float scale_log2;           // |scale| * log2(e), above 0: scores are exponents of 2
    int16_t q_sign;             // xor on the queries: the sign bit where the scale is negative
    int32_t rows, q_heads, group;
    int32_t tile_queries, ranges;
    AttendPart *parts;          // [ranges]
    float *part_stat;           // [2 ranges][2][tile_queries]: maximum, sum
    float *part_sum;            // [2 ranges][tile_queries][dim]
};

constexpr int MAX_VOCAB = 1 << 20;
constexpr int VOCAB_CHUNK = 1024;   // logits of a row that one wave takes at a time

// Of one chunk of a row, and of a whole row: the largest logit; where T <= 0 its lowest index, else
// the sum of exp((z - top) / T) (chunk) or 1 / that sum (row).
struct LogitStat {
    double sum;
    float top;
    int32_t best;               // -1: nothing above -infinity; where T > 0 no more than that there is something
};

// Where the walk of one sequence stands between launches.
struct WalkState {
    double S, rest;             // as moe_drafted.h names them
    int32_t cur, kept, after;   // the row, the rows of the path so far, the last child that was tested
    int32_t pending;            // 1: waits for the sum of max(p - S q, 0) over row cur
};

struct VerifyParams {
    const void *logits;
    int64_t logit_stride, draft_stride;
    const int32_t *tokens, *row_start, *parent;
    const float *u_test, *u_pick, *draft, *temperature;
    int32_t *n_keep, *path, *out_tokens;
    float *logprobs;
    uint32_t *flags;
    int32_t rows, seqs, vocab, chunks;
    int32_t last_round;
    LogitStat *chunk_stat;      // [rows][chunks]
    LogitStat *row_stat;        // [rows]
    double *token_p;            // [rows]: without draft_probs, log p of the pick
    int32_t *pick;              // [rows]: without draft_probs, the token drawn after the row
    double *left;               // [seqs][chunks]: sums of max(p - S q, 0)
    WalkState *state;           // [seqs]
    uint32_t *arrived;          // [seqs]: workgroups that have added their part of a sum; apart from the state, which is
                                // copied and stored whole
};

struct KeepParams {
    CacheParams c;
    const int32_t *row_start, *n_keep, *path;
    int32_t *new_len;
    int32_t rows;
};

}  // namespace moe
