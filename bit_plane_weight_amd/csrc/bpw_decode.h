// bpw_decode.h - records and launchers shared by the host checks (bpw_decode_host.cpp) and the kernels
// of the decode-step operators (bpw_heads.hip, bpw_attention*.hip, bpw_verify.hip). Not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace bpw {

// Most workgroups of a launch: a grid of 2^32 threads or more is not run as asked, and no error says so. What needs more
// workgroups (of 256 threads) goes in several launches.
constexpr int32_t kMaxWgs = 1 << 22;

// ---------------------------------------------------------------- heads (norm, rotation, append)

// One set of heads: inputs and outputs by element strides. With slots, out_ts is the stride of a cache
// row and out_ps of a page.
struct HeadSet {
    const void *in;
    void *out;
    int64_t in_ts, in_hs;
    int64_t out_ts, out_hs, out_ps;
    const float *gain;  // null: no norm
    int32_t heads;
    int32_t to_cache;   // 1: the output row is slots[t]
};

struct HeadsArgs {
    HeadSet q, k, v;    // v: copied only (append)
    const int32_t *positions;
    const double *inv_freq;
    const int64_t *slots;
    int64_t n_slots;
    int32_t n_tokens, head_dim, rot_dim, interleaved;
    int32_t page_log2;
    int32_t lanes_log2;      // lanes of one head
    int32_t tokens_per_wg;
    int32_t first_wg;        // of this launch
    float eps;
};

constexpr int kHeadThreads = 256;
// Paths: rows of any alignment; rows read and written 16 bytes at a time (alignment and divisibility checked by the
// host), with pairs anywhere in them, or with pairs of whole chunks.
constexpr int32_t kHeadsAny = 0, kHeadsMixed = 1, kHeadsVec = 2;
int launch_heads(const HeadsArgs &a, int32_t dt_in, int32_t dt_out, int32_t path, void *stream);

// ---------------------------------------------------------------- attention

constexpr int kAttnWaves = 4;
constexpr int kAttnThreads = 64 * kAttnWaves;
constexpr int kAttnStep = 32;                      // positions a wave takes at a time: its unit of work
constexpr int kWideTile = 64;                      // positions a workgroup takes at a time of a prefix that many rows share
constexpr int kAttnMaxSeqs = 1024;
constexpr int kAttnWgs = 512;                      // most workgroups of a launch: two to each of 256 CUs
constexpr int kAttnPieces = 64;                    // most pieces that the host cuts an item of a wide prefix into
// Most parts of a query row: one from each wave's run, and beside those a wide prefix's pieces.
constexpr int kAttnParts = kAttnWaves * kAttnWgs + kAttnPieces;

struct AttnArgs {
    const void *q;
    void *out;
    float *lse;
    int64_t q_ts, q_hs, o_ts, o_hs;
    const void *k, *v;
    int64_t k_ps, k_hs, v_ps, v_hs;
    int32_t k_rs, v_rs;      // row strides (elements)
    const int32_t *prefix_pages;
    const int32_t *table;
    int64_t table_stride;
    const int32_t *lens, *q_starts;
    int32_t n_tokens, n_seqs, max_q, q_heads, kv_heads, group, head_dim;
    int32_t page_log2, n_pages, prefix_len, cap;  // cap: positions a table row can hold
    float scale_log2;
    int32_t n_wgs;
    int32_t tiles_p;         // query tiles of the prefix per kv head
    int32_t splits, split_units;  // of a wide prefix: equal pieces of an item, units of one
    // workspace
    int32_t *sched;          // kSchedHead words, then units before each sequence, then items before each
    float *part_o;           // [parts][rows of a tile][padded dim]
    float4 *part_ml;         // [parts][rows of a tile]: shift (log2 units), sum of the weights, sum of the rounded ones
    int64_t part_s;          // offset (floats) of the suffixes' parts in part_o
    int64_t ml_s;            // and in part_ml
};
constexpr int kSchedHead = 8;  // units of a prefix item, units of the two lengths of runs, runs of the first

// Costs for the dealing, in steps of one suffix wave: a tile of a wide prefix, and what an item costs beyond its steps.
constexpr float kWideCost64 = 0.5f, kWideCost128 = 0.6f, kItemCost = 4.0f;

// The dealing of units (kAttnStep positions of an item) to the runs of the 4 n_wgs waves. The first runs_f runs hold qf
// units, the others qb. Narrow prefix: its units and the suffixes' in equal runs, wp of them the prefix's. Wide prefix:
// the waves of the `idle` workgroups, which had one piece less, take more of the suffixes and come first.
struct AttnDeal {
    int32_t qf, qb, wp, runs_f;
    // run of unit u of the suffixes
    __host__ __device__ int32_t run_of(int32_t u) const { return u < runs_f * qf ? u / qf : runs_f + (u - runs_f * qf) / qb; }
};

inline __host__ __device__ AttnDeal deal_narrow(int32_t total_p, int32_t total_s, int32_t n_wgs) {
    AttnDeal d{0, 1, 0, 0};
    const int32_t even = (total_p + total_s + kAttnWaves * n_wgs - 1) / (kAttnWaves * n_wgs);
    for (d.qb = even > 1 ? even : 1;; ++d.qb) {
        d.wp = (total_p + d.qb - 1) / d.qb;
        if (d.wp + (total_s + d.qb - 1) / d.qb <= kAttnWaves * n_wgs) break;
    }
    d.qf = d.qb;
    return d;
}

inline __host__ __device__ AttnDeal deal_wide(int32_t total_s, int32_t items_s, int32_t idle, int32_t split_units, bool tile64,
                                              int32_t n_wgs) {
    AttnDeal d{0, 1, 0, kAttnWaves * idle};
    const float cost_s = total_s > 0 ? 1.0f + kItemCost * (float)items_s / (float)total_s : 1.0f;
    const int32_t more = (int32_t)((float)split_units * (tile64 ? kWideCost64 : kWideCost128) / cost_s);
    const int64_t first = (int64_t)d.runs_f * more;  // units that the idle ones take meanwhile
    if (idle > 0 && total_s <= first) {
        const int32_t even = (total_s + d.runs_f - 1) / d.runs_f;
        d.qf = even > 1 ? even : 1;
    } else {
        d.qb = (total_s - (int32_t)first + kAttnWaves * n_wgs - 1) / (kAttnWaves * n_wgs);
        d.qf = d.qb + more;
    }
    return d;
}

// Wide prefix: the run of a wave. `busy` workgroups of each XCD had all the pieces of a turn; workgroup b runs on XCD b % 8.
inline __host__ __device__ int32_t wide_run(int32_t block, int32_t wave, int32_t busy, int32_t idle) {
    const int32_t xcd = block & 7, at = block >> 3;
    return at < busy ? kAttnWaves * idle + wave * 8 * busy + xcd + 8 * at : wave * idle + xcd + 8 * (at - busy);
}

int launch_attn_d64(const AttnArgs &a, int32_t dtype, int32_t mp, int32_t ms, void *stream);
int launch_attn_d128(const AttnArgs &a, int32_t dtype, int32_t mp, int32_t ms, void *stream);
int launch_attn_d256(const AttnArgs &a, int32_t dtype, int32_t mp, int32_t ms, void *stream);

// ---------------------------------------------------------------- draft verification

constexpr int kVerifyThreads = 256;
constexpr int kVerifyChunk = 4096;  // vocabulary entries summed by one workgroup

struct VerifyArgs {
    const void *target, *draft;
    int64_t t_seq, t_step, d_seq, d_step;
    const int32_t *tokens, *n_draft;
    const float *accept_u, *sample_u;
    int32_t *out_tokens, *accepted;
    double *sums;           // [n_seqs][chunks]
    int32_t *found;         // [n_seqs][2]: drafts accepted, whether one was refused
    int32_t n_seqs, max_drafts, vocab, chunks;
};
int launch_verify(const VerifyArgs &a, int32_t dtype, void *stream);

}  // namespace bpw
