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
    int32_t pages, page, heads, dim, seqs, width;
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
    return dim <= 64 ? (queries == 16 ? 4 : 3) : dim <= 96 ? 3 : dim <= 128 ? 2 : 1;
}

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
    int32_t tile_queries;
    AttendPart *parts;          // [ranges]
    float *part_stat;           // [2 ranges][2][tile_queries]: maximum, sum
    float *part_sum;            // [2 ranges][tile_queries][dim]
};

constexpr int MAX_VOCAB = 1 << 20;
constexpr int VOCAB_CHUNK = 2048;   // logits per partial sum
constexpr int MAX_CHUNKS = MAX_VOCAB / VOCAB_CHUNK;

struct VerifyParams {
    const void *logits;
    int64_t logit_stride, draft_stride;
    const int32_t *tokens, *row_start, *parent;
    const float *u_test, *u_pick, *draft, *temperature;
    int32_t *n_keep, *path, *out_tokens;
    float *logprobs;
    uint32_t *flags;
    int32_t rows, seqs, vocab;
};

struct KeepParams {
    CacheParams c;
    const int32_t *row_start, *n_keep, *path;
    int32_t *new_len;
    int32_t rows;
};

}  // namespace moe
