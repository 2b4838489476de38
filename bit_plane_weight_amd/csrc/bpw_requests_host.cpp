// bpw_requests_host.cpp - host side of what a request needs around the 16-bit decode step: attention over whole prompts, the
// cache held in 4 bits (append and attention), log probabilities of given tokens. Argument checks, choice of kernel, launch.
// See include/bpw.h for the contract.
#include "bpw_checks.h"

namespace {

bpw_status check_kv4(const bpw_paged_kv4 &c, const char *who) {
    if (c.kv_heads < 1 || c.kv_heads > kMaxHeads) return fail(BPW_E_INVAL, "%s: kv_heads %d outside [1, %d]", who, (int)c.kv_heads, (int)kMaxHeads);
    if (c.head_dim < 32 || c.head_dim > 256 || c.head_dim % bpw::kKv4Block)
        return fail(BPW_E_UNSUPPORTED, "%s: head_dim %d is not a multiple of 32 in [32, 256]", who, (int)c.head_dim);
    if (c.page_size < 16 || c.page_size > 1024 || (c.page_size & (c.page_size - 1)))
        return fail(BPW_E_UNSUPPORTED, "%s: page_size %d is not a power of two in [16, 1024]", who, (int)c.page_size);
    if (c.n_pages < 0) return fail(BPW_E_INVAL, "%s: n_pages %d is negative", who, (int)c.n_pages);
    if (c.n_pages > 0 && (!c.d_k || !c.d_v || !c.d_k_scale || !c.d_v_scale)) return fail(BPW_E_INVAL, "%s: cache pointer is NULL", who);
    if (!aligned(c.d_k, 16) || !aligned(c.d_v, 16)) return fail(BPW_E_INVAL, "%s: codes are not aligned to 16 bytes", who);
    const int64_t codes[] = {c.k_page_stride, c.k_head_stride, c.k_row_stride, c.v_page_stride, c.v_head_stride, c.v_row_stride};
    for (int64_t x : codes)
        if (x < 0 || x > kMaxStride || x % 16) return fail(BPW_E_INVAL, "%s: a stride of the codes is no multiple of 16 in [0, 2^40]", who);
    const int64_t scales[] = {c.ks_page_stride, c.ks_head_stride, c.vs_page_stride, c.vs_head_stride};
    for (int64_t x : scales)
        if (x < 0 || x > kMaxStride) return fail(BPW_E_INVAL, "%s: a stride of the powers is outside [0, 2^40]", who);
    const int64_t code_rows[] = {c.k_row_stride, c.v_row_stride}, scale_rows[] = {c.ks_row_stride, c.vs_row_stride};
    for (int64_t x : code_rows)
        if (x < c.head_dim / 2 || x > kMaxRowStride) return fail(BPW_E_INVAL, "%s: a row stride of the codes is outside [head_dim / 2, 2^24]", who);
    for (int64_t x : scale_rows)
        if (x < c.head_dim / bpw::kKv4Block || x > kMaxRowStride)
            return fail(BPW_E_INVAL, "%s: a row stride of the powers is outside [head_dim / 32, 2^24]", who);
    return BPW_OK;
}

bpw::Kv4Rows kv4_keys(const bpw_paged_kv4 &c) {
    return {c.d_k, c.d_k_scale, c.k_page_stride, c.k_head_stride, c.ks_page_stride, c.ks_head_stride, (int32_t)c.k_row_stride, (int32_t)c.ks_row_stride};
}
bpw::Kv4Rows kv4_values(const bpw_paged_kv4 &c) {
    return {c.d_v, c.d_v_scale, c.v_page_stride, c.v_head_stride, c.vs_page_stride, c.vs_head_stride, (int32_t)c.v_row_stride, (int32_t)c.vs_row_stride};
}

// Query rows of all heads, in tiles of 128, from which a wave of the prompt kernel takes all positions of a tile and a workgroup
// 128 rows; below it two waves share the positions of 32 rows and a workgroup takes 64, which puts more CUs to work on
// few rows. One prompt, us, two waves to a row against one: 20 heads of 128 13.1 : 14.4 at 80 tiles, 17.4 : 18.0 at 120, 23.5 : 21.7 at
// 160, 34.4 : 29.1 at 240; 32 heads 19.0 : 18.5 at 192, 33.0 : 33.9 at 384, 175 : 145 at 1024; 16 heads of 256 36.8 : 39.1 at 128, 47.8 :
// 45.6 at 160, 80.7 : 69.9 at 256; of 192 31.5 : 32.1 at 128, 38.0 : 37.8 at 160. Heads of 64, of which more workgroups fit a CU: 21.7 :
// 22.8 at 384, 30.3 : 30.5 at 512, 93.9 : 86.8 at 1024.
int64_t prompt_many_tiles(int32_t padded_dim) { return padded_dim == 64 ? 512 : 160; }

int32_t padded(int32_t head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }

}  // namespace

extern "C" {

// ------------------------------------------------------------------------------ whole prompts

bpw_status bpw_prompt_attn(const bpw_prompt_attn_args *a, void *stream) {
    const char *who = "prompt attention";
    if (!a) return fail(BPW_E_INVAL, "%s: NULL arguments", who);
    if (a->n_tokens < 0) return fail(BPW_E_INVAL, "%s: n_tokens %d is negative", who, (int)a->n_tokens);
    if (a->n_seqs < 1 || a->n_seqs > (1 << 20)) return fail(BPW_E_UNSUPPORTED, "%s: n_seqs %d outside [1, 2^20]", who, (int)a->n_seqs);
    if (a->head_dim < 8 || a->head_dim > 256 || a->head_dim % 8)
        return fail(BPW_E_UNSUPPORTED, "%s: head_dim %d is not a multiple of 8 in [8, 256]", who, (int)a->head_dim);
    if (a->n_tokens == 0) return (bpw_status)bpw::host_check_device();
    bpw_status st;
    if ((st = check_heads(a->q, who, "q")) || (st = check_heads(a->k, who, "k")) || (st = check_heads(a->v, who, "v")) ||
        (st = check_heads(a->out, who, "out")))
        return st;
    if (a->k.heads < 1 || a->v.heads != a->k.heads || a->q.heads < 1 || a->q.heads % a->k.heads)
        return fail(BPW_E_INVAL, "%s: %d query heads are not a multiple of %d key heads, or v has another count (%d)", who,
                    (int)a->q.heads, (int)a->k.heads, (int)a->v.heads);
    if (a->out.heads != a->q.heads) return fail(BPW_E_INVAL, "%s: out has another head count than q", who);
    const int32_t dt = a->q.dtype;
    if (dt == BPW_F32 || a->k.dtype != dt || a->v.dtype != dt || a->out.dtype != dt)
        return fail(BPW_E_UNSUPPORTED, "%s: q, k, v and out share a type, bfloat16 or float16", who);
    const bpw_heads *all[] = {&a->q, &a->k, &a->v, &a->out};
    for (const bpw_heads *x : all)
        if (!wide(x->d, x->dtype, x->token_stride, x->head_stride, 0))
            return fail(BPW_E_INVAL, "%s: q, k, v and out need 16-byte alignment and strides of multiples of 8 elements", who);
    if (a->n_tokens > 1 && (a->k.token_stride < a->head_dim || a->v.token_stride < a->head_dim))
        return fail(BPW_E_INVAL, "%s: a token's stride of k or v is below head_dim %d: rows would overlap", who, (int)a->head_dim);
    if (a->k.token_stride > kMaxRowStride || a->v.token_stride > kMaxRowStride)
        return fail(BPW_E_UNSUPPORTED, "%s: a token's stride of k or v is above 2^24", who);
    const float scale_log2 = a->scale * 1.44269504088896341f;
    if (!(std::isfinite(scale_log2) && scale_log2 > 0.0f)) return fail(BPW_E_INVAL, "%s: scale is not finite and positive", who);
    if (!a->d_starts || !aligned(a->d_starts, 4) || !aligned(a->d_lse, 4))
        return fail(BPW_E_INVAL, "%s: starts are NULL, or starts or lse misaligned", who);
    const int32_t group = a->q.heads / a->k.heads;
    if ((int64_t)a->n_tokens * group > (INT64_C(1) << 30))
        return fail(BPW_E_UNSUPPORTED, "%s: more than 2^30 query rows to a key/value head", who);
    if ((st = (bpw_status)bpw::host_check_device())) return st;
    bpw::PromptArgs p{};
    p.q = a->q.d, p.k = a->k.d, p.v = a->v.d, p.out = a->out.d, p.lse = a->d_lse;
    p.q_ts = a->q.token_stride, p.q_hs = a->q.head_stride;
    p.k_ts = a->n_tokens > 1 ? (int32_t)a->k.token_stride : a->head_dim, p.k_hs = a->k.head_stride;
    p.v_ts = a->n_tokens > 1 ? (int32_t)a->v.token_stride : a->head_dim, p.v_hs = a->v.head_stride;
    p.o_ts = a->out.token_stride, p.o_hs = a->out.head_stride;
    p.starts = a->d_starts;
    p.n_tokens = a->n_tokens, p.n_seqs = a->n_seqs;
    p.q_heads = a->q.heads, p.kv_heads = a->k.heads, p.group = group, p.head_dim = a->head_dim;
    p.scale_log2 = scale_log2;
    const int32_t dp = padded(a->head_dim);
    const bool many = (int64_t)a->n_tokens * a->q.heads >= 128 * prompt_many_tiles(dp);
    const int e = dp == 64    ? bpw::launch_prompt_d64(p, dt, many, stream)
                  : dp == 128 ? bpw::launch_prompt_d128(p, dt, many, stream)
                              : bpw::launch_prompt_d256(p, dt, many, stream);
    return hip_status(e, "prompt attention launch");
}

// ------------------------------------------------------------------------------ a cache held in 4 bits

bpw_status bpw_kv4_append(const bpw_kv4_append_args *a, void *stream) {
    const char *who = "kv4 append";
    if (!a) return fail(BPW_E_INVAL, "%s: NULL arguments", who);
    if (a->n_tokens < 0) return fail(BPW_E_INVAL, "%s: n_tokens %d is negative", who, (int)a->n_tokens);
    const bpw_paged_kv4 &c = a->kv;
    bpw_status st;
    if ((st = check_kv4(c, who))) return st;
    if (a->n_tokens == 0) return (bpw_status)bpw::host_check_device();
    if ((st = check_eps(a->eps, who)) || (st = check_heads(a->k, who, "k")) || (st = check_heads(a->v, who, "v")) ||
        (st = check_heads(a->q, who, "q")) || (st = check_heads(a->q_out, who, "q_out")) ||
        (st = check_heads(a->k_values, who, "k_values")) || (st = check_heads(a->v_values, who, "v_values")) ||
        (st = check_rotation(a->rot, c.head_dim, who)))
        return st;
    if (a->k.heads != c.kv_heads || a->v.heads != c.kv_heads)
        return fail(BPW_E_INVAL, "%s: k and v need the cache's %d heads", who, (int)c.kv_heads);
    if (a->q.heads != a->q_out.heads) return fail(BPW_E_INVAL, "%s: q_out has another head count than q", who);
    if ((a->k_values.heads && a->k_values.heads != c.kv_heads) || (a->v_values.heads && a->v_values.heads != c.kv_heads))
        return fail(BPW_E_INVAL, "%s: k_values and v_values need the cache's %d heads", who, (int)c.kv_heads);
    if (a->v.dtype != a->k.dtype || (a->q.heads && a->q.dtype != a->k.dtype))
        return fail(BPW_E_UNSUPPORTED, "%s: q, k and v have different types", who);
    int32_t dt_out = BPW_BF16;
    bool one = true, any = false;
    const bpw_heads *outs[] = {&a->q_out, &a->k_values, &a->v_values};
    for (const bpw_heads *x : outs) {
        if (!x->heads) continue;
        one = one && x->dtype != BPW_F32 && (!any || x->dtype == dt_out);
        dt_out = x->dtype;
        any = true;
    }
    if (!one) return fail(BPW_E_UNSUPPORTED, "%s: q_out, k_values and v_values share a type, bfloat16 or float16", who);
    if (!aligned(a->d_q_gain, 4) || !aligned(a->d_k_gain, 4)) return fail(BPW_E_INVAL, "%s: a gain is misaligned", who);
    if (!a->d_slots || !aligned(a->d_slots, 8)) return fail(BPW_E_INVAL, "%s: slots are NULL or misaligned", who);
    if ((st = (bpw_status)bpw::host_check_device())) return st;
    bpw::Kv4AppendArgs h{};
    h.q = head_set(a->q, a->q_out, a->d_q_gain);
    h.k = head_set(a->k, a->k_values, a->d_k_gain);
    h.v = head_set(a->v, a->v_values, nullptr);
    if (!a->k_values.heads) h.k.out = nullptr;
    if (!a->v_values.heads) h.v.out = nullptr;
    h.kc = kv4_keys(c);
    h.vc = kv4_values(c);
    h.positions = a->rot.d_positions;
    h.inv_freq = a->rot.d_inv_freq;
    h.slots = a->d_slots;
    h.n_slots = (int64_t)c.n_pages * c.page_size;
    h.n_tokens = a->n_tokens;
    h.head_dim = c.head_dim;
    h.rot_dim = a->rot.rot_dim;
    h.interleaved = a->rot.interleaved;
    h.page_log2 = log2_of(c.page_size);
    h.lanes_log2 = log2_of(c.head_dim / 8);
    h.vec = 1;
    const bpw_heads *all[] = {&a->k, &a->v, &a->q, &a->q_out, &a->k_values, &a->v_values};
    for (const bpw_heads *x : all)
        if (x->heads && !wide(x->d, x->dtype, x->token_stride, x->head_stride, 0)) h.vec = 0;
    h.eps = a->eps;
    h.inv_head_dim = 1.0 / c.head_dim;
    return hip_status(bpw::launch_kv4_append(h, a->k.dtype, dt_out, stream), "kv4 append launch");
}

}  // extern "C"

namespace {

struct Attn4Shape {
    int32_t dp, group, n_wgs;
    int64_t cap;
    bool one_launch;
    size_t po, pml, total;  // workspace: offsets of the parts, all
};

// One launch, a workgroup to an item (sequence, key/value head, 16 query rows), or even runs of positions over all waves and a
// join, which take 9 us at least. Measured (us, one launch against two; tables full; 32 query heads to 8 key/value heads at 64 and
// 128, 16 to 4 at 256; a token to a sequence unless said).
// Up to so many positions of a row of the page table (x padded head size): one sequence of heads of 128 9.8 : 9.7 at 1024 positions,
// 12.0 : 10.8 at 1536; of heads of 256 11.5 : 11.0 at 512, 16.7 : 11.6 at 1024.
constexpr int64_t kShort4Work = 163840;
// And from 128 items on, half of the CUs: 16 sequences of heads of 64 14.3 : 16.0 at 2560, 19.6 : 18.7 at 4096, 26.4 : 22.3 at 6144; 32 of
// them 20.1 : 25.4 at 4096; 16 of heads of 128 15.0 : 17.2 at 2048, 17.0 : 18.8 at 2560, 23.7 : 23.2 at 4096; 64 of them 33.1 : 34.9 at
// 2048, 54.4 : 56.5 at 4096, but, with lengths spread from 1 on, 59.5 : 49.4 at 6144.
constexpr int64_t kShort4WorkFull = 262144, kShort4Items = 128;
// And so many steps of a wave beside one more for every 16 items, as few items leave CUs idle for as long: one sequence of heads of
// 64 8.7 : 9.4 at 1024 positions (4 steps), 10.5 : 9.7 at 1536 (6), 14.0 : 10.9 at 2560 (10); 4 of them 10.7 : 11.4, 14.3 : 12.4 at the
// last two.
constexpr int64_t kShort4WaveSteps = 5;
// And so many items beside one for every 16 query rows, by padded head size, about two turns of all workgroups (heads of 128: one to a CU,
// of 64, whose turns are short, more): 64 sequences of 512 positions, heads of 128 14.8 : 17.5, 128 29.5 : 24.6, 512 110.6 : 72.1;
// heads of 256 128 26.3 : 35.6, 256 51.3 : 49.9, 512 99.1 : 82.2; heads of 64 512 55.2 : 53.8, 1024 113.5 : 101.4. Rows cost the join:
// 8 sequences of 64 tokens of heads of 128 33.6 : 36.4 (1024 items).
int64_t short4_items(int32_t padded_dim) { return padded_dim == 64 ? 4096 : padded_dim == 128 ? 512 : 1024; }
// And most of all items' steps (x padded head size), where the items are many by their rows: 4 sequences of 200 tokens of heads of 128
// 55.4 : 53.4 at 512 positions, 113.2 : 101.3 at 2048; 2 of 1000 185 : 160 at 1024.
constexpr int64_t kShort4Steps = 1 << 22;

bpw_status attn4_shape(const bpw_kv4_attn_args *a, Attn4Shape *s) {
    const char *who = "kv4 attention";
    if (!a) return fail(BPW_E_INVAL, "%s: NULL arguments", who);
    const bpw_paged_kv4 &c = a->kv;
    bpw_status st;
    if ((st = check_kv4(c, who))) return st;
    if (a->n_tokens < 0 || a->n_tokens > (1 << 24)) return fail(BPW_E_INVAL, "%s: n_tokens %d outside [0, 2^24]", who, (int)a->n_tokens);
    if (a->n_seqs < 1 || a->n_seqs > bpw::kAttnMaxSeqs)
        return fail(BPW_E_UNSUPPORTED, "%s: n_seqs %d outside [1, %d]", who, (int)a->n_seqs, (int)bpw::kAttnMaxSeqs);
    if (a->max_q < 1 || a->max_q > (1 << 24)) return fail(BPW_E_INVAL, "%s: max_q %d outside [1, 2^24]", who, (int)a->max_q);
    if (a->max_pages < 0 || (int64_t)a->max_pages * c.page_size > (INT64_C(1) << 30))
        return fail(BPW_E_INVAL, "%s: max_pages %d outside what 2^30 positions hold", who, (int)a->max_pages);
    if (a->q.heads < 1 || a->q.heads % c.kv_heads || a->q.heads > kMaxHeads)
        return fail(BPW_E_INVAL, "%s: %d query heads are not a multiple of %d key/value heads (up to %d)", who,
                    (int)a->q.heads, (int)c.kv_heads, (int)kMaxHeads);
    s->group = a->q.heads / c.kv_heads;
    s->dp = padded(c.head_dim);
    s->cap = (int64_t)a->max_pages * c.page_size;
    const int64_t max_q = a->max_q < a->n_tokens ? a->max_q : (a->n_tokens > 0 ? a->n_tokens : 1);
    const int64_t tiles = (max_q * s->group + 15) / 16, units = (s->cap + bpw::kAttnStep - 1) / bpw::kAttnStep;
    const int64_t items = (int64_t)a->n_seqs * c.kv_heads * tiles;
    if ((double)items * (double)units >= 2.0e9 || (double)a->n_seqs * (double)max_q * a->q.heads >= 2.0e9)
        return fail(BPW_E_UNSUPPORTED, "%s: more work than one launch deals out", who);
    const int64_t most = items * units;
    s->n_wgs = (int32_t)(most < 2 ? 2 : most < bpw::kAttnWgs ? most : bpw::kAttnWgs);
    const int64_t waves = s->dp == 256 ? 4 : 8, query_rows = a->n_seqs * max_q * a->q.heads;
    // (a table without columns has no steps, but its items may be more than one grid takes)
    s->one_launch = s->cap * s->dp <= (items >= kShort4Items ? kShort4WorkFull : kShort4Work) &&
                    (units + waves - 1) / waves <= kShort4WaveSteps + items / 16 &&
                    items <= short4_items(s->dp) + query_rows / 16 && most * s->dp <= kShort4Steps && items <= bpw::kMaxWgs;
    const size_t rows = units > 0 ? (size_t)(items + (int64_t)bpw::kAttnWaves * s->n_wgs) * 16 : 0;  // a part per item and per run
    s->po = up256((size_t)(bpw::kSchedHead + 2 * (a->n_seqs + 1)) * 4);
    s->pml = s->po + up256(rows * (size_t)s->dp * 4);
    s->total = s->pml + up256(rows * 16);
    return BPW_OK;
}

}  // namespace

extern "C" {

size_t bpw_kv4_attn_workspace_bytes(const bpw_kv4_attn_args *a) {
    Attn4Shape s{};
    return attn4_shape(a, &s) == BPW_OK ? s.total : 0;
}

bpw_status bpw_kv4_attn(const bpw_kv4_attn_args *a, void *d_ws, size_t ws_len, void *stream) {
    const char *who = "kv4 attention";
    Attn4Shape s{};
    bpw_status st = attn4_shape(a, &s);
    if (st) return st;
    const bpw_paged_kv4 &c = a->kv;
    if (a->n_tokens == 0) return (bpw_status)bpw::host_check_device();
    if ((st = check_heads(a->q, who, "q")) || (st = check_heads(a->out, who, "out"))) return st;
    if (a->q.heads != a->out.heads) return fail(BPW_E_INVAL, "%s: out has another head count than q", who);
    if (a->q.dtype == BPW_F32 || a->out.dtype != a->q.dtype)
        return fail(BPW_E_UNSUPPORTED, "%s: q and out share a type, bfloat16 or float16", who);
    const float scale_log2 = a->scale * 1.44269504088896341f;  // scores in units of log 2: v_exp_f32 is 2^x
    if (!(std::isfinite(scale_log2) && scale_log2 > 0.0f)) return fail(BPW_E_INVAL, "%s: scale is not finite and positive", who);
    if (!wide(a->q.d, a->q.dtype, a->q.token_stride, a->q.head_stride, 0) ||
        !wide(a->out.d, a->out.dtype, a->out.token_stride, a->out.head_stride, 0))
        return fail(BPW_E_INVAL, "%s: q and out need 16-byte alignment and strides of multiples of 8 elements", who);
    if (!a->d_lens || !a->d_q_starts || (a->max_pages > 0 && !a->d_table))
        return fail(BPW_E_INVAL, "%s: NULL lengths, starts or page table", who);
    if (a->table_stride < a->max_pages || a->table_stride > kMaxStride)
        return fail(BPW_E_INVAL, "%s: table_stride %lld below max_pages %d", who, (long long)a->table_stride, (int)a->max_pages);
    if (!aligned(a->d_lens, 4) || !aligned(a->d_q_starts, 4) || !aligned(a->d_table, 4) || !aligned(a->d_lse, 4))
        return fail(BPW_E_INVAL, "%s: misaligned lengths, starts, table or lse", who);
    if (!d_ws || !aligned(d_ws, 256)) return fail(BPW_E_INVAL, "%s: workspace is NULL or not 256-byte aligned", who);
    if (ws_len < s.total) return fail(BPW_E_SIZE, "%s: workspace %zu bytes, needs %zu", who, ws_len, s.total);
    if ((st = (bpw_status)bpw::host_check_device())) return st;
    bpw::Attn4Args b{};
    bpw::AttnArgs &k = b.a;
    k.q = a->q.d;
    k.out = a->out.d;
    k.lse = a->d_lse;
    k.q_ts = a->q.token_stride;
    k.q_hs = a->q.head_stride;
    k.o_ts = a->out.token_stride;
    k.o_hs = a->out.head_stride;
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
    k.cap = (int32_t)s.cap;
    k.scale_log2 = scale_log2;
    k.n_wgs = s.n_wgs;
    char *ws = static_cast<char *>(d_ws);
    k.sched = reinterpret_cast<int32_t *>(ws);
    k.part_o = reinterpret_cast<float *>(ws + s.po);
    k.part_ml = reinterpret_cast<float4 *>(ws + s.pml);
    b.kc = kv4_keys(c);
    b.vc = kv4_values(c);
    const auto dense = [&](const bpw::Kv4Rows &r) {
        return aligned(r.scales, 4) && r.s_rs == c.head_dim / bpw::kKv4Block && r.s_ps % 4 == 0 && r.s_hs % 4 == 0;
    };
    b.dense = c.head_dim == s.dp && dense(b.kc) && dense(b.vc);
    const int e = s.dp == 64    ? bpw::launch_attn4_d64(b, a->q.dtype, s.one_launch, stream)
                  : s.dp == 128 ? bpw::launch_attn4_d128(b, a->q.dtype, s.one_launch, stream)
                                : bpw::launch_attn4_d256(b, a->q.dtype, s.one_launch, stream);
    return hip_status(e, "kv4 attention launch");
}

}  // extern "C"

// ------------------------------------------------------------------------------ log probabilities

namespace {

constexpr int64_t kLogprobWgs = 1024;  // workgroups that fill the GPU: four to each of 256 CUs

// Workgroups of a row and rounds of each: rows are cut where there are too few to fill the GPU.
void logprob_parts(int32_t n_tokens, int32_t vocab, int32_t *parts, int32_t *rounds) {
    const int32_t all = (vocab + bpw::kLogprobRound - 1) / bpw::kLogprobRound;
    const int64_t want = n_tokens >= kLogprobWgs ? 1 : (kLogprobWgs + n_tokens - 1) / n_tokens;
    *rounds = (int32_t)((all + want - 1) / want);
    *parts = (all + *rounds - 1) / *rounds;
}

}  // namespace

extern "C" {

size_t bpw_token_logprobs_workspace_bytes(int32_t n_tokens, int32_t vocab, int32_t n_top) {
    if (n_tokens < 1 || vocab < 1 || vocab > (1 << 24) || n_top < 0 || n_top > bpw::kLogprobTop) return 0;
    int32_t parts, rounds;
    logprob_parts(n_tokens, vocab, &parts, &rounds);
    if (parts == 1) return 0;
    return up256((size_t)n_tokens * parts * 16) + up256((size_t)n_tokens * parts * n_top * 8);
}

bpw_status bpw_token_logprobs(const bpw_token_logprobs_args *a, void *d_ws, size_t ws_len, void *stream) {
    const char *who = "token logprobs";
    if (!a) return fail(BPW_E_INVAL, "%s: NULL arguments", who);
    if (a->n_tokens < 0) return fail(BPW_E_INVAL, "%s: n_tokens %d is negative", who, (int)a->n_tokens);
    if (a->vocab < 1 || a->vocab > (1 << 24)) return fail(BPW_E_UNSUPPORTED, "%s: vocab %d outside [1, 2^24]", who, (int)a->vocab);
    if (a->n_top < 0 || a->n_top > bpw::kLogprobTop)
        return fail(BPW_E_UNSUPPORTED, "%s: n_top %d outside [0, %d]", who, (int)a->n_top, (int)bpw::kLogprobTop);
    if (!dtype_ok(a->dtype)) return fail(BPW_E_INVAL, "%s: no type %d", who, (int)a->dtype);
    if (a->row_stride < 0 || a->row_stride > kMaxStride) return fail(BPW_E_INVAL, "%s: row_stride outside [0, 2^40]", who);
    const float scale_log2 = a->scale * 1.44269504088896341f;
    if (!(std::isfinite(scale_log2) && scale_log2 > 0.0f)) return fail(BPW_E_INVAL, "%s: scale is not finite and positive", who);
    if (a->n_tokens == 0) return (bpw_status)bpw::host_check_device();
    if (!a->d_logits) return fail(BPW_E_INVAL, "%s: logits are NULL", who);
    if (!a->d_tokens != !a->d_logprobs) return fail(BPW_E_INVAL, "%s: one of tokens and logprobs is NULL", who);
    if (a->n_top > 0 && (!a->d_top_tokens || !a->d_top_logprobs)) return fail(BPW_E_INVAL, "%s: top_tokens or top_logprobs is NULL", who);
    if (!aligned(a->d_logits, dtype_size(a->dtype)) || !aligned(a->d_tokens, 4) || !aligned(a->d_logprobs, 4) || !aligned(a->d_entropy, 4) ||
        !aligned(a->d_top_tokens, 4) || !aligned(a->d_top_logprobs, 4))
        return fail(BPW_E_INVAL, "%s: misaligned argument", who);
    bpw::LogprobArgs k{};
    logprob_parts(a->n_tokens, a->vocab, &k.parts, &k.part_rounds);
    const size_t need = bpw_token_logprobs_workspace_bytes(a->n_tokens, a->vocab, a->n_top);
    if (need && (!d_ws || !aligned(d_ws, 256))) return fail(BPW_E_INVAL, "%s: workspace is NULL or not 256-byte aligned", who);
    if (ws_len < need) return fail(BPW_E_SIZE, "%s: workspace %zu bytes, needs %zu", who, ws_len, need);
    bpw_status st = (bpw_status)bpw::host_check_device();
    if (st) return st;
    k.logits = a->d_logits;
    k.row_stride = a->row_stride;
    k.tokens = a->d_tokens;
    k.logprobs = a->d_logprobs;
    k.entropy = a->d_entropy;
    k.top_tokens = a->d_top_tokens;
    k.top_logprobs = a->d_top_logprobs;
    k.n_tokens = a->n_tokens;
    k.vocab = a->vocab;
    k.n_top = a->n_top;
    k.scale = a->scale;
    k.stats = static_cast<float4 *>(d_ws);
    k.tops = reinterpret_cast<uint64_t *>(static_cast<char *>(d_ws) + up256((size_t)a->n_tokens * k.parts * 16));
    return hip_status(bpw::launch_logprobs(k, a->dtype, stream), "token logprobs launch");
}

}  // extern "C"
