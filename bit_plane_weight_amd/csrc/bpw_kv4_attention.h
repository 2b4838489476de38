// bpw_kv4_attention.h - attention of a decode step over a paged cache held in 4 bits (gfx950, wave64), instantiated per padded
// head size by bpw_kv4_attention_d*.hip. Dealing of the work, parts and joins are those of bpw_attention.h without a
// prefix; what a wave does with its positions is here.
//
// Mathematics as there. Operands: a code times its block's power of two is exact in bfloat16, and
// v_cvt_scalef32_pk_bf16_fp4 makes two of them in one instruction, so keys and values enter the products as they are.
// Float16 queries are the sum of two bfloat16 numbers (11 bits of 8 + 8), and so are the softmax weights to 2^-17 of
// each; the second products cost little where memory is the bound.
//
// Layouts. The order in which a product adds up elements is free, so lane g = lane / 16 takes a quarter of a key's row,
// DP / 4 neighbours (one 16-byte load of 32 elements at heads of 128: one block, one power), and the query's elements
// are laid out alike. A value row is read by 16 lanes, 8 neighbours each (4 bytes), and turned by v_perm after the
// conversion.
#pragma once

#include "bpw_attention.h"

namespace bpw {

constexpr uint32_t kPlainUnit = 0x3F800000u;  // 2^0, for positions whose weight is zero

template <class T>
constexpr int kQueryPieces = __is_same(T, __bf16) ? 1 : 2;

__device__ __forceinline__ uint32_t two_of(uint32_t codes, float unit, int which) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    bf16x2 x;
    switch (which) {
        case 0: x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, 0); break;
        case 1: x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, 1); break;
        case 2: x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, 2); break;
        default: x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, unit, 3); break;
    }
    return __builtin_bit_cast(uint32_t, x);
}
__device__ __forceinline__ float unit_of_byte(uint32_t b) { return __builtin_bit_cast(float, b << 23); }

// The sum of eight numbers of bfloat16 or float16 as bfloat16 operands: x itself, or its upper and lower parts.
__device__ __forceinline__ void split8(u32v4 x, u32v4 (&p)[1], __bf16) { p[0] = x; }
__device__ __forceinline__ void split8(u32v4 x, u32v4 (&p)[2], _Float16) {
    const f32x8 f = as_f32(__builtin_bit_cast(f16x8, x));
    const bf16x8 hi = __builtin_convertvector(f, bf16x8);
    p[0] = __builtin_bit_cast(u32v4, hi);
    p[1] = __builtin_bit_cast(u32v4, __builtin_convertvector(f - __builtin_convertvector(hi, f32x8), bf16x8));
}

// One tile of 16 query rows over positions [pos0, pos1) of a page list (s), 32 positions at a time.
template <class T, int DP>
__device__ __forceinline__ void attend4(const Attn4Args &b, const AttnSpan &s) {
    constexpr int QP = kQueryPieces<T>;
    constexpr int KC = DP / 32;                        // products of a tile of keys
    constexpr int KB = DP / 8, KW = KB / 4;            // bytes and words of a lane's key elements
    constexpr int KS = DP / 128 > 0 ? DP / 128 : 1;    // powers of them
    constexpr int EL = DP < 128 ? DP / 16 : 8, NH = DP / (16 * EL), VW = EL / 2;  // as in attend()
    const AttnArgs &a = b.a;
    const int lane = threadIdx.x & 63;
    const int n = lane & 15, g = lane >> 4;
    const int D = a.head_dim, pmask = (1 << a.page_log2) - 1;

    u32v4 q[KC][QP];
    int vis;
    {
        const int row = s.row0 + n, j = row / a.group;
        const T *p = static_cast<const T *>(a.q) + (int64_t)(s.tok0 + j) * a.q_ts +
                     (int64_t)(s.head * a.group + row - j * a.group) * a.q_hs;
        vis = s.causal ? s.len - (s.n_tok - 1 - j) : s.len;
        if (row >= s.n_rows) vis = s.len;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            const int d0 = DP / 4 * g + 8 * c;
            u32v4 x = {0, 0, 0, 0};
            if (row < s.n_rows && d0 < D) x = *reinterpret_cast<const u32v4 *>(p + d0);
            split8(x, q[c], T());
        }
    }
    const int all_see = s.causal ? s.len - (s.n_tok - 1) : s.len;

    // byte offsets of this lane inside a 16-position tile of a page; what lies past head_dim is read from its start
    const bool key_in[2] = {DP / 4 * g < D, DP / 4 * g + 32 < D};  // (the second: heads of 256)
    int koff[2], ksoff[2], voff[NH], vsoff[NH];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        koff[i] = n * b.kc.rs + (key_in[i] ? KB * g + 16 * i : 0);
        ksoff[i] = n * b.kc.s_rs + (key_in[i] ? (DP / 4 * g + 32 * i) / kKv4Block : 0);
    }
#pragma unroll
    for (int h = 0; h < NH; ++h) {
        const int d0 = 16 * EL * h + EL * n < D ? 16 * EL * h + EL * n : 0;
        voff[h] = 4 * g * b.vc.rs + d0 / 2;
        vsoff[h] = 4 * g * b.vc.s_rs + d0 / kKv4Block;
    }
    const uint8_t *kbase = b.kc.codes + (int64_t)s.head * b.kc.hs, *ksbase = b.kc.scales + (int64_t)s.head * b.kc.s_hs;
    const uint8_t *vbase = b.vc.codes + (int64_t)s.head * b.vc.hs, *vsbase = b.vc.scales + (int64_t)s.head * b.vc.s_hs;

    f32x4 o[NH * EL];
    float m = kNone, l = 0.0f;
#pragma unroll
    for (int c = 0; c < NH * EL; ++c) o[c] = f32x4{0, 0, 0, 0};

    struct Keys {
        uint32_t w[KW], unit[KS];
    };
    struct Values {
        uint32_t w[4][NH], unit[4][NH];
    };
    const auto load_keys = [&](int pos, int id, Keys &k) {
#pragma unroll
        for (int i = 0; i < KW; ++i) k.w[i] = 0;
#pragma unroll
        for (int i = 0; i < KS; ++i) k.unit[i] = 127;
        if (id >= 0) {
            const uint8_t *p = kbase + (int64_t)id * b.kc.ps + (int64_t)(pos & pmask) * b.kc.rs;
            const uint8_t *ps = ksbase + (int64_t)id * b.kc.s_ps + (int64_t)(pos & pmask) * b.kc.s_rs;
            if constexpr (KW == 2) {
                const u32x2 x = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(p + koff[0]));
                k.w[0] = x.x, k.w[1] = x.y;
            } else {
#pragma unroll
                for (int i = 0; i < KW / 4; ++i) {
                    const u32v4 x = __builtin_nontemporal_load(reinterpret_cast<const u32v4 *>(p + koff[i]));
                    k.w[4 * i] = x.x, k.w[4 * i + 1] = x.y, k.w[4 * i + 2] = x.z, k.w[4 * i + 3] = x.w;
                }
            }
#pragma unroll
            for (int i = 0; i < KS; ++i) k.unit[i] = ps[ksoff[i]];
        }
    };
    const auto load_values = [&](int pos, int id, Values &v) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int h = 0; h < NH; ++h) v.w[r][h] = 0, v.unit[r][h] = 127;
        if (id >= 0) {
            const uint8_t *p = vbase + (int64_t)id * b.vc.ps + (int64_t)(pos & pmask) * b.vc.rs;
            const uint8_t *ps = vsbase + (int64_t)id * b.vc.s_ps + (int64_t)(pos & pmask) * b.vc.s_rs;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const uint8_t *e = p + r * b.vc.rs + voff[h];
                    if constexpr (EL == 8)
                        v.w[r][h] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t *>(e));
                    else
                        v.w[r][h] = __builtin_nontemporal_load(reinterpret_cast<const uint16_t *>(e));
                    v.unit[r][h] = ps[r * b.vc.s_rs + vsoff[h]];
                }
        }
    };
    // Scores of 16 positions.
    const auto scores = [&](const Keys &k) {
        f32x4 sc = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            u32v4 f;
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = two_of(k.w[c], unit_of_byte(k.unit[c / 4 < KS ? c / 4 : 0]), i);
            if (D != DP && DP / 4 * g + 8 * c >= D) f = u32v4{0, 0, 0, 0};  // (a power of 255 there must not meet the query's zeros)
#pragma unroll
            for (int x = 0; x < QP; ++x) sc = mma<__bf16>(f, q[c][x], sc);
        }
        return sc;
    };

    AttnPages pages;
    int kv0 = s.pos0;
    const int end = min(s.len, s.pos1);
    pages.start(a, s, kv0);
    int id0 = pages.of(a, s, kv0 >> 4), id1 = pages.of(a, s, (kv0 >> 4) + 1);
    Keys k0, k1;
    load_keys(kv0, id0, k0);
    load_keys(kv0 + 16, id1, k1);
    while (kv0 < end) {
        Values v0, v1;
        load_values(kv0, id0, v0);
        load_values(kv0 + 16, id1, v1);
        f32x4 sc[2] = {scores(k0), scores(k1)};
        const int here = kv0, c0 = id0, c1 = id1;
        kv0 += kAttnStep;
        if (kv0 < end) {  // the next step's keys
            id0 = pages.of(a, s, kv0 >> 4);
            id1 = pages.of(a, s, (kv0 >> 4) + 1);
            load_keys(kv0, id0, k0);
            load_keys(kv0 + 16, id1, k1);
        }
        bool odd = false;  // a value that only some rows see is NaN
        if (here + kAttnStep > all_see || (c0 | c1) < 0) {
            bool found = false;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int pos = here + 16 * t + 4 * g + r;
                    const bool page = (t ? c1 : c0) >= 0;
                    if (!page || pos >= vis) sc[t][r] = kNone;
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        uint32_t &u = t ? v1.unit[r][h] : v0.unit[r][h];
                        if (pos >= s.len)
                            u = 127;  // zero weight times whatever the page holds there is not zero
                        else if (pos >= all_see)
                            found |= u > 252;
                    }
                }
            odd = __any(found);
        }
        // weights against a shift that is raised where a lane's sum of a step passes the limit, as in attend()
        f32x8 w;
        float sum = 0.0f;
        const auto weigh = [&](float shift) {
            sum = 0.0f;
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                w[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[r >> 2][r & 3], a.scale_log2, -shift));
                sum += w[r];
            }
        };
        weigh(m);
        if (__any(!(sum < kShiftLimit<__bf16>))) {
            float top = kNone;
#pragma unroll
            for (int r = 0; r < 4; ++r) top = fmaxf(top, fmaxf(sc[0][r], sc[1][r]));
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32)) * a.scale_log2;
            const float up = fmaxf(m, top);
            const float f = up == m ? 1.0f : __builtin_amdgcn_exp2f(m - up);
            m = up;
            l *= f;
#pragma unroll
            for (int c = 0; c < NH * EL; ++c) o[c] *= f;
            weigh(up == kNone ? 0.0f : up);
        }
        l += sum;
        const bf16x8 hi = __builtin_convertvector(w, bf16x8);
        const u32v4 p0 = __builtin_bit_cast(u32v4, hi);
        const u32v4 p1 = __builtin_bit_cast(u32v4, __builtin_convertvector(w - __builtin_convertvector(hi, f32x8), bf16x8));

        uint32_t v[8][NH][VW];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int i = 0; i < VW; ++i) {
                    v[r][h][i] = two_of(v0.w[r][h], unit_of_byte(v0.unit[r][h]), i);
                    v[4 + r][h][i] = two_of(v1.w[r][h], unit_of_byte(v1.unit[r][h]), i);
                }
        const auto turned = [&](int h, int c) {
            u32v4 f;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                f[x] = __builtin_amdgcn_perm(v[2 * x + 1][h][c >> 1], v[2 * x][h][c >> 1], c & 1 ? 0x07060302u : 0x05040100u);
            return f;
        };
        if (!odd) {
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int c = 0; c < EL; ++c) {
                    const u32v4 f = turned(h, c);
                    o[h * EL + c] = mma<__bf16>(f, p1, mma<__bf16>(f, p0, o[h * EL + c]));
                }
        } else {
            // one query token at a time, the last first: the values that it does not see are set to zero, and only its
            // rows take the result
            const int last = min(s.n_tok, (s.row0 + 15) / a.group + 1);
            for (int j = last - 1; j >= s.row0 / a.group; --j) {
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    if (here + 16 * (x >> 2) + 4 * g + (x & 3) >= s.len - (s.n_tok - 1 - j)) {
#pragma unroll
                        for (int h = 0; h < NH; ++h)
#pragma unroll
                            for (int i = 0; i < VW; ++i) v[x][h][i] = 0;
                    }
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int c = 0; c < EL; ++c) {
                        const u32v4 f = turned(h, c);
                        const f32x4 x = mma<__bf16>(f, p1, mma<__bf16>(f, p0, o[h * EL + c]));
                        if ((s.row0 + n) / a.group == j) o[h * EL + c] = x;
                    }
            }
        }
    }

    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (s.row0 + n >= s.n_rows) return;
    if (g == 0) s.pml[n] = make_float4(stored_shift(m, l), l, l, 0.0f);
    float *po = s.po + n * DP;
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < EL; c += 4) {
                f32x4 x;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = o[h * EL + c + e][r];
                *reinterpret_cast<f32x4 *>(po + 16 * EL * h + EL * (4 * g + r) + c) = x;
            }
}

// Long sequences: the units (32 positions of an item: sequence x key/value head x 16 query rows) are dealt to the waves in
// equal contiguous runs, each part joined by the second launch.
template <class T, int DP>
__global__ __launch_bounds__(kAttnThreads, 2) void attn4_split_kernel(Attn4Args b) {
    const AttnArgs &a = b.a;
    extern __shared__ int32_t dynamic[];
    __shared__ int32_t wave_sum[kAttnWaves][2];
    AttnSeqs seqs(dynamic, a.n_seqs);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    // units and items before each sequence: four sequences a thread, then a scan
    int un[4], it[4], su = 0, si = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int i = 4 * tid + x;
        un[x] = it[x] = 0;
        if (i < a.n_seqs) {
            const int2 tok = seq_tokens(a, i);
            const int len = seq_len(a, i), u = (len + kAttnStep - 1) / kAttnStep;
            seqs.tok0[i] = tok.x;
            seqs.n_tok[i] = tok.y;
            seqs.len[i] = len;
            it[x] = u > 0 ? a.kv_heads * ((tok.y * a.group + 15) / 16) : 0;
            un[x] = it[x] * u;
        }
        su += un[x];
        si += it[x];
    }
    int iu = scan_add(su), ii = scan_add(si);
    if (lane == 63) wave_sum[wave][0] = iu, wave_sum[wave][1] = ii;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int x = 0; x < kAttnWaves; ++x) {
        if (x < wave) iu += wave_sum[x][0], ii += wave_sum[x][1];
        total += wave_sum[x][0];
    }
    total = __builtin_amdgcn_readfirstlane(total);
    int eu = iu - su, ei = ii - si;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int i = 4 * tid + x;
        if (i < a.n_seqs) seqs.units[i] = eu, seqs.items[i] = ei;
        eu += un[x], ei += it[x];
        if (i == a.n_seqs - 1) seqs.units[a.n_seqs] = eu, seqs.items[a.n_seqs] = ei;
    }
    const AttnDeal deal = deal_narrow(0, total, gridDim.x);
    __syncthreads();
    if (blockIdx.x == 0) {  // what the join needs
        if (tid == 0) a.sched[0] = 0, a.sched[1] = deal.qf, a.sched[2] = deal.qb, a.sched[3] = deal.runs_f;
        for (int i = tid; i <= a.n_seqs; i += kAttnThreads) {
            a.sched[kSchedHead + i] = seqs.units[i];
            a.sched[kSchedHead + a.n_seqs + 1 + i] = seqs.items[i];
        }
    }
    // this wave's run; runs are spread over the workgroups first, so that few of them use many CUs
    const int w = wave * gridDim.x + blockIdx.x;
    int u = w * deal.qb;
    const int stop = min(total, u + deal.qb);
    if (u >= stop) return;
    int i = 0;  // the sequence that holds unit u: one lane finds it
    {
        int found = -1;
        for (int x = lane; x < a.n_seqs; x += 64)
            if (seqs.units[x] <= u && u < seqs.units[x + 1]) found = x;
        i = __builtin_amdgcn_readlane(found, __builtin_ctzll(__ballot(found >= 0)));
    }
    AttnSpan s;
    while (u < stop) {
        while (seqs.units[i + 1] <= u) ++i;  // past idle sequences
        i = __builtin_amdgcn_readfirstlane(i);
        const int len = __builtin_amdgcn_readfirstlane(seqs.len[i]), ub = (len + kAttnStep - 1) / kAttnStep;
        const int n_tok = __builtin_amdgcn_readfirstlane(seqs.n_tok[i]), tiles = (n_tok * a.group + 15) / 16;
        const int rest = u - __builtin_amdgcn_readfirstlane(seqs.units[i]);
        const int item = rest / ub, at = rest - item * ub, n = min(ub - at, stop - u);
        const int64_t part = __builtin_amdgcn_readfirstlane(seqs.items[i]) + item + w;
        s.pages = a.table + (int64_t)i * a.table_stride;
        s.len = len;
        s.tok0 = __builtin_amdgcn_readfirstlane(seqs.tok0[i]);
        s.n_tok = n_tok;
        s.causal = 1;
        s.head = item / tiles;
        s.row0 = (item - s.head * tiles) * 16;
        s.n_rows = n_tok * a.group;
        s.pos0 = at * kAttnStep;
        s.pos1 = (at + n) * kAttnStep;
        s.po = a.part_o + part * (16 * DP);
        s.pml = a.part_ml + part * 16;
        attend4<T, DP>(b, s);
        u += n;
    }
}

// Few positions: a workgroup takes a (sequence, key/value head, 16 query rows), its waves equal runs of its steps, and joins
// their parts through LDS.
template <int DP>
constexpr int kShort4Waves = DP == 256 ? 4 : 8;

template <class T, int DP>
__global__ __launch_bounds__(64 * kShort4Waves<DP>) void attn4_short_kernel(Attn4Args b, int tiles) {
    constexpr int WAVES = kShort4Waves<DP>;
    const AttnArgs &a = b.a;
    __shared__ float part_o[WAVES][16][DP];
    __shared__ float4 part_ml[WAVES][16];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int bh = blockIdx.x / tiles, tile = blockIdx.x - bh * tiles, i = bh / a.kv_heads;
    const int2 tok = seq_tokens(a, i);
    AttnSpan s;
    s.head = bh - i * a.kv_heads;
    s.row0 = 16 * tile;
    s.n_rows = tok.y * a.group;
    if (s.row0 >= s.n_rows) return;
    s.tok0 = tok.x;
    s.n_tok = tok.y;
    s.len = seq_len(a, i);
    const int run = ((s.len + kAttnStep - 1) / kAttnStep + WAVES - 1) / WAVES;  // steps of a wave
    s.pages = a.table + (int64_t)i * a.table_stride;
    s.causal = 1;
    s.pos0 = wave * run * kAttnStep;
    s.pos1 = s.pos0 + run * kAttnStep;
    s.po = &part_o[wave][0][0];
    s.pml = part_ml[wave];
    if (s.pos0 < s.len)
        attend4<T, DP>(b, s);
    else if ((tid & 63) < 16)
        part_ml[wave][tid & 63] = make_float4(kNone, 0.0f, 0.0f, 0.0f);
    __syncthreads();
    for (int x = tid; x < 16 * (DP / 4); x += 64 * WAVES) {
        const int row = x / (DP / 4), d = 4 * (x - row * (DP / 4));
        if (s.row0 + row >= s.n_rows) break;
        float top = kNone;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) top = fmaxf(top, part_ml[w][row].x);
        float sum = 0.0f;
        f32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float4 y = part_ml[w][row];
            if (y.x == kNone) continue;  // (such a part's outputs may not be there)
            const float f = __builtin_amdgcn_exp2f(y.x - top);
            sum += f * y.y;
            acc += *reinterpret_cast<const f32x4 *>(&part_o[w][row][d]) * f;
        }
        const int j = (s.row0 + row) / a.group;
        write_out<T>(a, tok.x + j, s.head * a.group + s.row0 + row - j * a.group, d, acc, top, sum, sum);
    }
}

template <class T, int DP>
static int run_attn4(const Attn4Args &b, bool one_launch, hipStream_t st) {
    const AttnArgs &a = b.a;
    if (one_launch) {
        const int tiles = (a.max_q * a.group + 15) / 16;
        attn4_short_kernel<T, DP><<<(unsigned)(a.n_seqs * a.kv_heads * tiles), 64 * kShort4Waves<DP>, 0, st>>>(b, tiles);
        return (int)hipGetLastError();
    }
    attn4_split_kernel<T, DP><<<(unsigned)a.n_wgs, kAttnThreads, (size_t)(5 * (a.n_seqs + 1)) * 4, st>>>(b);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? (int)e : run_join<T, DP>(a, 16, 16, st);
}

}  // namespace bpw
