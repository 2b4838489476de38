// bpw_decode_host.cpp - host side of the decode-step operators (head norms with rotation, paged append,
// shared-prefix attention, draft verification): argument checks, choice of kernel, launch. See include/bpw.h
// for the contract.
#include <cmath>

#include "bpw_checks.h"

namespace {

// Path, lanes of a head, tokens of a workgroup.
bpw_status run_heads(bpw::HeadsArgs &a, int32_t dt_in, int32_t dt_out, bool vec, const char *who, void *stream) {
    const int D = a.head_dim, R = a.rot_dim;
    const int heads = a.q.heads + a.k.heads + a.v.heads;
    vec = vec && aligned(a.q.gain, 16) && aligned(a.k.gain, 16);
    // 8192 tokens of 32 + 8 heads of 128 in bf16, us: 34 with 128 or 80 elements turned (vec); with 66, 47-48 (mixed) or
    // 136-142 (any). The mixed path holds a head in one wave, 8 elements to a lane, hence the 512.
    const int32_t path = vec && D % 16 == 0 && R % 16 == 0 ? bpw::kHeadsVec : vec && D % 8 == 0 && D <= 512 ? bpw::kHeadsMixed : bpw::kHeadsAny;
    a.lanes_log2 = log2_of(path == bpw::kHeadsVec ? D / 16 : path == bpw::kHeadsMixed ? D / 8 : D / 2);
    if (a.lanes_log2 > 6) a.lanes_log2 = 6;
    const int at_once = bpw::kHeadThreads >> a.lanes_log2;
    // Many tokens with few heads: as many to a workgroup as one sweep over its lanes holds. (More, so that a last sweep
    // over 40 heads is fuller, measured no faster: 69.5-72 us against 69.9 for 16384 tokens of 32 + 8 heads of 128.)
    a.tokens_per_wg = a.n_tokens >= 2048 && heads < at_once ? at_once / heads : 1;
    bpw_status st = (bpw_status)bpw::host_check_device();
    if (st) return st;
    return hip_status(bpw::launch_heads(a, dt_in, dt_out, path, stream), who);
}

}  // namespace

extern "C" {

bpw_status bpw_qk_norm_rope(const bpw_qk_norm_rope_args *a, void *stream) {
    const char *who = "qk norm rope";
    if (!a) return fail(BPW_E_INVAL, "%s: NULL arguments", who);
    if (a->n_tokens < 0) return fail(BPW_E_INVAL, "%s: n_tokens %d is negative", who, (int)a->n_tokens);
    if (a->head_dim < 2 || a->head_dim > 1024 || a->head_dim % 2)
        return fail(BPW_E_UNSUPPORTED, "%s: head_dim %d is not even in [2, 1024]", who, (int)a->head_dim);
    if (a->n_tokens == 0) return (bpw_status)bpw::host_check_device();  // (an empty buffer's address may be NULL)
    bpw_status st;
    if ((st = check_eps(a->eps, who)) || (st = check_heads(a->q, who, "q")) || (st = check_heads(a->k, who, "k")) ||
        (st = check_heads(a->q_out, who, "q_out")) || (st = check_heads(a->k_out, who, "k_out")) ||
        (st = check_rotation(a->rot, a->head_dim, who)))
        return st;
    if (a->q.heads != a->q_out.heads || a->k.heads != a->k_out.heads)
        return fail(BPW_E_INVAL, "%s: outputs have other head counts than inputs", who);
    if (a->q.heads && a->k.heads && (a->q.dtype != a->k.dtype || a->q_out.dtype != a->k_out.dtype))
        return fail(BPW_E_UNSUPPORTED, "%s: q and k have different types", who);
    if (!aligned(a->d_q_gain, 4) || !aligned(a->d_k_gain, 4)) return fail(BPW_E_INVAL, "%s: a gain is misaligned", who);
    if (a->q.heads + a->k.heads == 0) return (bpw_status)bpw::host_check_device();
    bpw::HeadsArgs h{};
    h.q = head_set(a->q, a->q_out, a->d_q_gain);
    h.k = head_set(a->k, a->k_out, a->d_k_gain);
    h.positions = a->rot.d_positions;
    h.inv_freq = a->rot.d_inv_freq;
    h.n_tokens = a->n_tokens;
    h.head_dim = a->head_dim;
    h.rot_dim = a->rot.rot_dim;
    h.interleaved = a->rot.interleaved;
    h.eps = a->eps;
    bool vec = true;
    const bpw_heads *all[] = {&a->q, &a->k, &a->q_out, &a->k_out};
    for (const bpw_heads *x : all)
        if (x->heads) vec = vec && wide(x->d, x->dtype, x->token_stride, x->head_stride, 0);
    const bpw_heads &in = a->q.heads ? a->q : a->k, &out = a->q.heads ? a->q_out : a->k_out;
    return run_heads(h, in.dtype, out.dtype, vec, who, stream);
}

bpw_status bpw_kv_append(const bpw_kv_append_args *a, void *stream) {
    const char *who = "kv append";
    if (!a) return fail(BPW_E_INVAL, "%s: NULL arguments", who);
    if (a->n_tokens < 0) return fail(BPW_E_INVAL, "%s: n_tokens %d is negative", who, (int)a->n_tokens);
    const bpw_paged_kv &c = a->kv;
    if (c.head_dim < 2 || c.head_dim > 1024 || c.head_dim % 2)
        return fail(BPW_E_UNSUPPORTED, "%s: head_dim %d is not even in [2, 1024]", who, (int)c.head_dim);
    bpw_status st;
    if ((st = check_kv(c, who))) return st;
    if (a->n_tokens == 0) return (bpw_status)bpw::host_check_device();
    if ((st = check_eps(a->eps, who)) || (st = check_heads(a->k, who, "k")) ||
        (st = check_heads(a->v, who, "v")) || (st = check_heads(a->q, who, "q")) ||
        (st = check_heads(a->q_out, who, "q_out")) || (st = check_rotation(a->rot, c.head_dim, who)))
        return st;
    if (a->k.heads != c.kv_heads || a->v.heads != c.kv_heads)
        return fail(BPW_E_INVAL, "%s: k and v need the cache's %d heads", who, (int)c.kv_heads);
    if (a->q.heads != a->q_out.heads) return fail(BPW_E_INVAL, "%s: q_out has another head count than q", who);
    if (a->v.dtype != a->k.dtype || (a->q.heads && a->q.dtype != a->k.dtype))
        return fail(BPW_E_UNSUPPORTED, "%s: q, k and v have different types", who);
    if (a->q.heads && a->q_out.dtype != c.dtype) return fail(BPW_E_UNSUPPORTED, "%s: q_out is not of the cache's type", who);
    if (!aligned(a->d_q_gain, 4) || !aligned(a->d_k_gain, 4)) return fail(BPW_E_INVAL, "%s: a gain is misaligned", who);
    if (!a->d_slots || !aligned(a->d_slots, 8)) return fail(BPW_E_INVAL, "%s: slots are NULL or misaligned", who);
    bpw::HeadsArgs h{};
    h.q = head_set(a->q, a->q_out, a->d_q_gain);
    const bpw_heads kc{c.d_k, c.kv_heads, c.dtype, c.k_row_stride, c.k_head_stride};
    const bpw_heads vc{c.d_v, c.kv_heads, c.dtype, c.v_row_stride, c.v_head_stride};
    h.k = head_set(a->k, kc, a->d_k_gain);
    h.v = head_set(a->v, vc, nullptr);
    h.k.out_ps = c.k_page_stride;
    h.v.out_ps = c.v_page_stride;
    h.k.to_cache = h.v.to_cache = 1;
    h.positions = a->rot.d_positions;
    h.inv_freq = a->rot.d_inv_freq;
    h.slots = a->d_slots;
    h.page_log2 = log2_of(c.page_size);
    h.n_slots = (int64_t)c.n_pages * c.page_size;
    h.n_tokens = a->n_tokens;
    h.head_dim = c.head_dim;
    h.rot_dim = a->rot.rot_dim;
    h.interleaved = a->rot.interleaved;
    h.eps = a->eps;
    bool vec = wide(c.d_k, c.dtype, c.k_page_stride, c.k_head_stride, c.k_row_stride) &&
               wide(c.d_v, c.dtype, c.v_page_stride, c.v_head_stride, c.v_row_stride);
    const bpw_heads *all[] = {&a->k, &a->v, &a->q, &a->q_out};
    for (const bpw_heads *x : all)
        if (x->heads) vec = vec && wide(x->d, x->dtype, x->token_stride, x->head_stride, 0);
    return run_heads(h, a->k.dtype, c.dtype, vec, who, stream);
}

}  // extern "C"

// ------------------------------------------------------------------------------ attention

namespace {

struct AttnShape {
    int32_t dp, mp, ms;
    int32_t group, tiles_p, splits, split_units;
    bool one_launch;
    int64_t cap, pieces_p, pieces_s;
    int32_t n_wgs;
    size_t sched, po, pml, total;  // workspace: bytes of the schedule, offsets of the parts, all
};

// Most work (steps of single waves x padded head size) that a prefix of more than 16 rows is given to single waves,
// whose first results come sooner; beyond it workgroups share the keys through LDS. Measured, us a call (waves, workgroups):
// 8 x 96 rows of 64 over 1000 positions, 49 k: 16.6, 19.5; 8 x 32 rows of 128 over 2000, 129 k: 18.1, 15.7; 5 x 64 rows of
// 128 over 1024, 82 k: 16.8, 15.1; 8 x 32 rows of 64 over 8000, 128 k: 17.9, 16.1.
constexpr int64_t kNarrowWork = 65536;
// Most positions (x padded head size) of a row of the page table for the one-launch kernel, those of a prefix twice, as every
// sequence reads them. Measured, us a call (one launch, two): one sequence of 20 / 5 heads of 128, 128 positions 5.3, 9.3;
// 256: 7.2, 9.1; 512: 9.0, 9.4; 704: 10.8, 9.6. 64 sequences of 256: 15.2, 17.0; with 256 of a prefix before them 23.6, 18.9.
constexpr int64_t kShortWork = 65536;
// Most of all its workgroups' steps (x padded head size), as each of them reads the sequence and the prefix for its 16 rows.
// Measured over 582 calls within the bound above (heads of 64, 128, 256; 1 to 256 sequences of 1 to 128 tokens; with and
// without a prefix): one launch takes 0.36 to 1.2 of two's time below 2^20 steps, 0.6 to 1.5 up to 2^21, 0.7 to 2.4 beyond.
// 256 sequences of 8 heads of 128 over 240 shared and 32 own positions: 50.8, two launches 21.4. With both bounds the calls
// take 1.7 % more than the better of the two on average (3.1 % without this one).
constexpr int64_t kShortSteps = 1 << 21;
constexpr int64_t kPieceCost = 3;   // tiles that a piece of a wide prefix costs beyond its own (queries in, parts out)
constexpr int64_t kBusyCost = 32;   // tiles that all workgroups being busy with pieces costs

bpw_status attn_shape(const bpw_attn_shared_prefix_args *a, AttnShape *s) {
    const char *who = "attention";
    if (!a) return fail(BPW_E_INVAL, "%s: NULL arguments", who);
    const bpw_paged_kv &c = a->kv;
    bpw_status st;
    if ((st = check_kv(c, who))) return st;
    if (c.head_dim < 8 || c.head_dim > 256 || c.head_dim % 8)
        return fail(BPW_E_UNSUPPORTED, "%s: head_dim %d is not a multiple of 8 in [8, 256]", who, (int)c.head_dim);
    if (c.k_row_stride < c.head_dim || c.v_row_stride < c.head_dim)
        return fail(BPW_E_INVAL, "%s: cache row strides below head_dim %d: rows would overlap", who, (int)c.head_dim);
    if (a->n_tokens < 0 || a->n_tokens > (1 << 24)) return fail(BPW_E_INVAL, "%s: n_tokens %d outside [0, 2^24]", who, (int)a->n_tokens);
    if (a->n_seqs < 1 || a->n_seqs > bpw::kAttnMaxSeqs)
        return fail(BPW_E_UNSUPPORTED, "%s: n_seqs %d outside [1, %d]", who, (int)a->n_seqs, (int)bpw::kAttnMaxSeqs);
    if (a->max_q < 1 || a->max_q > (1 << 24)) return fail(BPW_E_INVAL, "%s: max_q %d outside [1, 2^24]", who, (int)a->max_q);
    if (a->prefix_len < 0 || a->prefix_len > (INT64_C(1) << 30)) return fail(BPW_E_INVAL, "%s: prefix_len outside [0, 2^30]", who);
    if (a->max_pages < 0 || (int64_t)a->max_pages * c.page_size > (INT64_C(1) << 30))
        return fail(BPW_E_INVAL, "%s: max_pages %d outside what 2^30 positions hold", who, (int)a->max_pages);
    if (a->q.heads < 1 || a->q.heads % c.kv_heads || a->q.heads > kMaxHeads)
        return fail(BPW_E_INVAL, "%s: %d query heads are not a multiple of %d key/value heads (up to %d)", who,
                    (int)a->q.heads, (int)c.kv_heads, (int)kMaxHeads);
    s->group = a->q.heads / c.kv_heads;
    s->dp = c.head_dim <= 64 ? 64 : c.head_dim <= 128 ? 128 : 256;
    s->cap = (int64_t)a->max_pages * c.page_size;
    // Query rows of a tile: 16 of a suffix's (32 for heads of up to 64), or of a prefix that few rows share or that is
    // little work; else 64 or 128 rows share a prefix's keys through LDS.
    const int64_t rows_p = (int64_t)a->n_tokens * s->group;
    const int64_t max_q = a->max_q < a->n_tokens ? a->max_q : (a->n_tokens > 0 ? a->n_tokens : 1);
    const int64_t rows_s = max_q * s->group;
    s->ms = rows_s <= 16 || s->dp > 64 ? 16 : 32;
    const int64_t up = (a->prefix_len + bpw::kAttnStep - 1) / bpw::kAttnStep;
    const int narrow = s->dp > 64 ? 16 : 32;
    if (a->prefix_len == 0 || rows_p <= s->ms)
        s->mp = s->ms;
    else if (rows_p <= 16 || c.kv_heads * ((rows_p + narrow - 1) / narrow) * up * s->dp <= kNarrowWork)
        s->mp = narrow;
    else
        s->mp = rows_p <= 64 ? 64 : 128;
    const int64_t mp = s->mp, ms = s->ms;
    const int64_t tiles_p = (rows_p + mp - 1) / mp, tiles_s = (rows_s + ms - 1) / ms;
    const int64_t us = (s->cap + bpw::kAttnStep - 1) / bpw::kAttnStep;
    const int64_t items_p = c.kv_heads * tiles_p, items_s = (int64_t)a->n_seqs * c.kv_heads * tiles_s;
    const double work = (double)items_p * (double)up + (double)items_s * (double)us;
    if (work >= 2.0e9 || rows_p * c.kv_heads >= INT32_MAX || (double)a->n_seqs * (double)max_q * a->q.heads >= 2.0e9)
        return fail(BPW_E_UNSUPPORTED, "%s: more work than one launch deals out", who);
    s->tiles_p = (int32_t)tiles_p;
    const int64_t most = items_p * up + items_s * us;
    s->n_wgs = (int32_t)(most < 2 ? 2 : most < bpw::kAttnWgs ? most : bpw::kAttnWgs);
    s->splits = s->split_units = 0;
    if (mp > 32) {
        // Pieces of a wide prefix: items cut alike, in as many as end soonest: whole turns of all workgroups, each
        // piece costing some tiles beyond its own, and workgroups with a piece being lost to the suffixes (and to
        // memory traffic) meanwhile. Measured without that last term, us a call, 64 sequences of 20 + 5 heads of 128
        // over a prefix of 4096 with some 1000 positions each: 60.6 (320 pieces), with it 56.6 (110); over 16384:
        // 72.6 (430), 59.9 (200).
        s->n_wgs = (s->n_wgs + 7) / 8 * 8;
        const int64_t tiles = (a->prefix_len + bpw::kWideTile - 1) / bpw::kWideTile;
        int64_t best = INT64_MAX;
        for (int64_t n = 1; n <= tiles && n <= bpw::kAttnPieces; ++n) {
            const int64_t turns = (items_p * n + s->n_wgs - 1) / s->n_wgs, len = (tiles + n - 1) / n;
            const int64_t cost = turns * (len + kPieceCost) * s->n_wgs + kBusyCost * items_p * n;
            if (cost < best) {
                best = cost;
                s->splits = (int32_t)n;
                s->split_units = (int32_t)len;
            }
        }
        s->splits = (int32_t)((tiles + s->split_units - 1) / s->split_units);
    }
    // (nothing to see has no steps, but its items may be more than one grid takes)
    const int64_t items = (int64_t)a->n_seqs * c.kv_heads * ((rows_s + 15) / 16), steps = items * (up + us) * s->dp;
    s->one_launch = (s->cap + 2 * a->prefix_len) * s->dp <= kShortWork && steps <= kShortSteps && items <= bpw::kMaxWgs;
    // one part per item and per run, or per piece of a wide prefix
    const int64_t waves = (int64_t)bpw::kAttnWaves * s->n_wgs;
    s->pieces_p = mp > 32 ? items_p * s->splits : up > 0 ? items_p + waves : 0;
    s->pieces_s = us > 0 ? items_s + waves : 0;
    s->sched = up256((size_t)(bpw::kSchedHead + 2 * (a->n_seqs + 1)) * 4);
    s->po = s->sched;
    const size_t rows = (size_t)(s->pieces_p * mp + s->pieces_s * ms);
    s->pml = s->po + up256(rows * (size_t)s->dp * 4);
    s->total = s->pml + up256(rows * 16);
    return BPW_OK;
}

}  // namespace

extern "C" {

size_t bpw_attn_shared_prefix_workspace_bytes(const bpw_attn_shared_prefix_args *a) {
    AttnShape s{};
    return attn_shape(a, &s) == BPW_OK ? s.total : 0;
}

bpw_status bpw_attn_shared_prefix(const bpw_attn_shared_prefix_args *a, void *d_ws, size_t ws_len, void *stream) {
    const char *who = "attention";
    AttnShape s{};
    bpw_status st = attn_shape(a, &s);
    if (st) return st;
    const bpw_paged_kv &c = a->kv;
    if (a->n_tokens == 0) return (bpw_status)bpw::host_check_device();
    if ((st = check_heads(a->q, who, "q")) || (st = check_heads(a->out, who, "out"))) return st;
    if (a->q.heads != a->out.heads) return fail(BPW_E_INVAL, "%s: out has another head count than q", who);
    if (a->q.dtype != c.dtype || a->out.dtype != c.dtype)
        return fail(BPW_E_UNSUPPORTED, "%s: q and out need the cache's type", who);
    const float scale_log2 = a->scale * 1.44269504088896341f;  // scores in units of log 2: v_exp_f32 is 2^x
    if (!(std::isfinite(scale_log2) && scale_log2 > 0.0f)) return fail(BPW_E_INVAL, "%s: scale is not finite and positive", who);
    if (!wide(a->q.d, c.dtype, a->q.token_stride, a->q.head_stride, 0) ||
        !wide(a->out.d, c.dtype, a->out.token_stride, a->out.head_stride, 0) ||
        !wide(c.d_k, c.dtype, c.k_page_stride, c.k_head_stride, c.k_row_stride) ||
        !wide(c.d_v, c.dtype, c.v_page_stride, c.v_head_stride, c.v_row_stride))
        return fail(BPW_E_INVAL, "%s: q, out and the cache need 16-byte alignment and strides of multiples of 8 elements", who);
    if (!a->d_lens || !a->d_q_starts || (a->max_pages > 0 && !a->d_table) || (a->prefix_len > 0 && !a->d_prefix_pages))
        return fail(BPW_E_INVAL, "%s: NULL lengths, starts or page table", who);
    if (a->table_stride < a->max_pages || a->table_stride > kMaxStride)
        return fail(BPW_E_INVAL, "%s: table_stride %lld below max_pages %d", who, (long long)a->table_stride, (int)a->max_pages);
    if (!aligned(a->d_lens, 4) || !aligned(a->d_q_starts, 4) || !aligned(a->d_table, 4) || !aligned(a->d_prefix_pages, 4) ||
        !aligned(a->d_lse, 4))
        return fail(BPW_E_INVAL, "%s: misaligned lengths, starts, table or lse", who);
    if (!d_ws || !aligned(d_ws, 256)) return fail(BPW_E_INVAL, "%s: workspace is NULL or not 256-byte aligned", who);
    if (ws_len < s.total) return fail(BPW_E_SIZE, "%s: workspace %zu bytes, needs %zu", who, ws_len, s.total);
    if ((st = (bpw_status)bpw::host_check_device())) return st;
    bpw::AttnArgs k{};
    k.q = a->q.d;
    k.out = a->out.d;
    k.lse = a->d_lse;
    k.q_ts = a->q.token_stride;
    k.q_hs = a->q.head_stride;
    k.o_ts = a->out.token_stride;
    k.o_hs = a->out.head_stride;
    k.k = c.d_k;
    k.v = c.d_v;
    k.k_ps = c.k_page_stride;
    k.k_hs = c.k_head_stride;
    k.k_rs = (int32_t)c.k_row_stride;
    k.v_ps = c.v_page_stride;
    k.v_hs = c.v_head_stride;
    k.v_rs = (int32_t)c.v_row_stride;
    k.prefix_pages = a->d_prefix_pages;
    k.table = a->d_table;
    k.table_stride = a->table_stride;
    k.lens = a->d_lens;
    k.q_starts = a->d_q_starts;
    k.n_tokens = a->n_tokens;
    k.n_seqs = a->n_seqs;
    k.max_q = a->max_q < a->n_tokens ? a->max_q : a->n_tokens;
    k.q_heads = a->q.heads;
    k.kv_heads = c.kv_heads;
    k.group = s.group;
    k.head_dim = c.head_dim;
    k.page_log2 = log2_of(c.page_size);
    k.n_pages = c.n_pages;
    k.prefix_len = (int32_t)a->prefix_len;
    k.cap = (int32_t)s.cap;
    k.scale_log2 = scale_log2;
    k.n_wgs = s.n_wgs;
    k.tiles_p = s.tiles_p;
    k.splits = s.splits;
    k.split_units = s.split_units;
    char *ws = static_cast<char *>(d_ws);
    k.sched = reinterpret_cast<int32_t *>(ws);
    k.part_o = reinterpret_cast<float *>(ws + s.po);
    k.part_ml = reinterpret_cast<float4 *>(ws + s.pml);
    k.part_s = s.pieces_p * s.mp * s.dp;
    k.ml_s = s.pieces_p * s.mp;
    const int32_t mp = s.one_launch ? 0 : s.mp;
    const int e = s.dp == 64    ? bpw::launch_attn_d64(k, c.dtype, mp, s.ms, stream)
                  : s.dp == 128 ? bpw::launch_attn_d128(k, c.dtype, mp, s.ms, stream)
                                : bpw::launch_attn_d256(k, c.dtype, mp, s.ms, stream);
    return hip_status(e, "attention launch");
}

// ------------------------------------------------------------------------------ draft verification

size_t bpw_verify_draft_workspace_bytes(int32_t n_seqs, int32_t vocab) {
    if (n_seqs < 1 || vocab < 1 || vocab > (1 << 24)) return 0;
    const size_t chunks = ((size_t)vocab + bpw::kVerifyChunk - 1) / bpw::kVerifyChunk;
    return up256((size_t)n_seqs * (chunks * sizeof(double) + 2 * sizeof(int32_t)));
}

bpw_status bpw_verify_draft(const bpw_verify_draft_args *a, void *d_ws, size_t ws_len, void *stream) {
    const char *who = "verify draft";
    if (!a) return fail(BPW_E_INVAL, "%s: NULL arguments", who);
    if (a->n_seqs < 0 || a->n_seqs > 65535) return fail(BPW_E_INVAL, "%s: n_seqs %d outside [0, 65535]", who, (int)a->n_seqs);
    if (a->max_drafts < 1 || a->max_drafts > 64)
        return fail(BPW_E_UNSUPPORTED, "%s: max_drafts %d outside [1, 64]", who, (int)a->max_drafts);
    if (a->vocab < 1 || a->vocab > (1 << 24)) return fail(BPW_E_UNSUPPORTED, "%s: vocab %d outside [1, 2^24]", who, (int)a->vocab);
    if (!dtype_ok(a->dtype)) return fail(BPW_E_INVAL, "%s: no type %d", who, (int)a->dtype);
    const int64_t st4[] = {a->target_seq_stride, a->target_step_stride, a->d_draft ? a->draft_seq_stride : 0,
                           a->d_draft ? a->draft_step_stride : 0};
    for (int64_t x : st4)
        if (x < 0 || x > kMaxStride) return fail(BPW_E_INVAL, "%s: strides outside [0, 2^40]", who);
    if (a->n_seqs == 0) return (bpw_status)bpw::host_check_device();
    if (!a->d_target || !a->d_tokens || !a->d_accept_u || !a->d_sample_u || !a->d_out_tokens || !a->d_accepted)
        return fail(BPW_E_INVAL, "%s: NULL argument", who);
    const size_t es = dtype_size(a->dtype);
    if (!aligned(a->d_target, es) || !aligned(a->d_draft, es) || !aligned(a->d_tokens, 4) || !aligned(a->d_n_draft, 4) ||
        !aligned(a->d_accept_u, 4) || !aligned(a->d_sample_u, 4) || !aligned(a->d_out_tokens, 4) || !aligned(a->d_accepted, 4))
        return fail(BPW_E_INVAL, "%s: misaligned argument", who);
    const size_t need = bpw_verify_draft_workspace_bytes(a->n_seqs, a->vocab);
    if (!d_ws || !aligned(d_ws, 256)) return fail(BPW_E_INVAL, "%s: workspace is NULL or not 256-byte aligned", who);
    if (ws_len < need) return fail(BPW_E_SIZE, "%s: workspace %zu bytes, needs %zu", who, ws_len, need);
    bpw_status st = (bpw_status)bpw::host_check_device();
    if (st) return st;
    bpw::VerifyArgs v{};
    v.target = a->d_target;
    v.draft = a->d_draft;
    v.t_seq = a->target_seq_stride;
    v.t_step = a->target_step_stride;
    v.d_seq = a->draft_seq_stride;
    v.d_step = a->draft_step_stride;
    v.tokens = a->d_tokens;
    v.n_draft = a->d_n_draft;
    v.accept_u = a->d_accept_u;
    v.sample_u = a->d_sample_u;
    v.out_tokens = a->d_out_tokens;
    v.accepted = a->d_accepted;
    v.chunks = (a->vocab + bpw::kVerifyChunk - 1) / bpw::kVerifyChunk;
    v.sums = static_cast<double *>(d_ws);
    v.found = reinterpret_cast<int32_t *>(v.sums + (size_t)a->n_seqs * v.chunks);
    v.n_seqs = a->n_seqs;
    v.max_drafts = a->max_drafts;
    v.vocab = a->vocab;
    return hip_status(bpw::launch_verify(v, a->dtype, stream), "verify launch");
}

}  // extern "C"
