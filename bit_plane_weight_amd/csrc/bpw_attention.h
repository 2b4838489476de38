// bpw_attention.h - attention of a decode step over a shared prefix and per-sequence suffixes in a paged
// cache (gfx950, wave64): the split kernel, instantiated per padded head size by bpw_attention_d*.hip.
//
// Mathematics. For a query row q and positions i: s_i = scale <q, K_i>; with a running maximum m and sum
// l = sum exp(s_i - m), o = sum exp(s_i - m) V_i, parts over disjoint positions join exactly:
// m = max m_p, l = sum exp(m_p - m) l_p, o = sum exp(m_p - m) o_p. So the positions of one
// (segment, key/value head, tile of query rows) - an item - are cut into units, units are dealt to the waves (or
// workgroups, for prefixes that many rows share) in equal contiguous runs, and a second launch joins
// the parts in order.
//
// The rows of a tile are the queries that read the same keys: the heads of one group, times the query
// tokens of a sequence, and in the prefix times all sequences, so the prefix is read once for them.
//
// Matrix products. A wave takes kAttnStep = 32 positions at a time and forms S^T = K Q^T and O^T += V^T
// P^T with 16x16x32 products, so that
//  - keys come straight from memory as the first operand (lane: position lane % 16, 8 elements);
//  - the scores of one query lie in the four lanes n, n + 16, n + 32, n + 48, each holding 2 x 4
//    positions, which is already the second operand's layout of P^T once the positions of a step are
//    numbered (tile, lane / 16, register): the weights never leave the registers;
//  - values are read row-wise in the same numbering (lane: 8 positions x 8 elements) and turned by
//    v_perm_b32 (32 for 64 elements), tile c of V^T holding elements 8 m + c, so that a lane's results are
//    8 neighbours of the output row.
// No LDS is used and no wave waits for another; bound: memory (6.47 TB/s over 964 MB of four sequences, 90 % of a
// plain read), or the latency of a few dependent loads where there is little. Keys and values are loaded non-temporally, as they are read once:
// 964 MB over four sequences take 155 us so and 174 us without.
#pragma once

#include <type_traits>

#include "bpw_decode.h"
#include "bpw_elem.h"

namespace bpw {

template <class T>
__device__ __forceinline__ f32x4 mma(u32v4 a, u32v4 b, f32x4 c);
template <>
__device__ __forceinline__ f32x4 mma<__bf16>(u32v4 a, u32v4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x4 mma<_Float16>(u32v4 a, u32v4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// c + the sum of eight 16-bit weights, in float32.
template <class T>
__device__ __forceinline__ float sum8(u32v4 p, float c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = p[i];
        if constexpr (__is_same(T, __bf16)) {
            typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
            c = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, x), bf16x2{(__bf16)1.0f, (__bf16)1.0f}, c, false);
        } else {
            typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
            c = __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, x), f16x2{(_Float16)1.0f, (_Float16)1.0f}, c, false);
        }
    }
    return c;
}

// Not zero if a 16-bit half of x is infinite or NaN (and for some finite ones above an infinite one).
template <class T>
__device__ __forceinline__ uint32_t maybe_not_finite(uint32_t x) {
    constexpr uint32_t ones = __is_same(T, __bf16) ? 0x7F807F80u : 0x7C007C00u;
    const uint32_t y = (x & ones) ^ ones;  // a half of zero: exponent all ones
    return (y - 0x00010001u) & ~y & 0x80008000u;
}

// The work of one wave or workgroup on one item: positions [pos0, pos1) of a page list for a tile of query rows.
struct AttnSpan {
    const int32_t *pages;
    int32_t len;       // positions of the segment
    int32_t tok0;      // first token of its rows
    int32_t n_tok;     // tokens of its rows
    int32_t causal;    // row of token j sees len - (n_tok - 1 - j) positions
    int32_t head;      // key/value head
    int32_t row0;      // first row of the tile
    int32_t n_rows;    // rows of all tiles
    int32_t pos0, pos1;
    float *po;         // results of the tile: [rows][DP]
    float4 *pml;       // [rows]: shift (log2 units; -inf: nothing seen), sum of the weights, sum of the rounded weights
};

constexpr float kNone = -__builtin_inff();

// A raised shift makes the largest weight 2^kLift, and a lane's sum of a step stays below kShiftLimit: about 1000 times that.
// float16 holds weights from half of 2^-24 to 65504, so they begin at 2^6: one is lost only below 2^-31 of the largest
// (at 2^0, a thousand positions at 2^-25 were all lost); bfloat16 has the exponents of float32.
template <class T>
constexpr float kLift = __is_same(T, __bf16) ? 0.0f : 6.0f;
template <class T>
constexpr float kShiftLimit = __is_same(T, __bf16) ? 1024.0f : 61440.0f;

// The shift that a part is stored with. Maxima pass over NaN, so a row whose scores are all NaN has a sum of NaN at a shift
// that is still kNone; any finite shift tells it from a row that saw nothing.
__device__ __forceinline__ float stored_shift(float m, float l) { return m == kNone && l != 0.0f ? 0.0f : m; }

// Pages of the positions to come, one granule of 16 positions a lane (pages hold a multiple of 16, so a granule
// never straddles two): two runs of 64 granules, the second loaded while the first is in use, so that
// no load of keys waits for a page number.
struct AttnPages {
    int32_t cur, next;  // as in the list; -1 past the end
    int32_t base;       // first granule of `cur`

    __device__ __forceinline__ int32_t fetch(const AttnArgs &a, const AttnSpan &s, int granule) const {
        const int pos = 16 * (granule + (int)(threadIdx.x & 63));
        int32_t id = -1;
        if (pos < s.len) id = s.pages[pos >> a.page_log2];
        return id;
    }
    __device__ __forceinline__ void start(const AttnArgs &a, const AttnSpan &s, int pos) {
        base = pos >> 4;
        cur = fetch(a, s, base);
        next = fetch(a, s, base + 64);
    }
    // Page of granule `granule`, which is at most 64 past the last one asked for, or -1: past the end, or not a
    // page of the cache. The same in all lanes.
    __device__ __forceinline__ int32_t of(const AttnArgs &a, const AttnSpan &s, int granule) {
        if (granule >= base + 64) {
            base += 64;
            cur = next;
            next = fetch(a, s, base + 64);
        }
        const int32_t id = __builtin_amdgcn_readlane(cur, granule - base);
        return (uint32_t)id < (uint32_t)a.n_pages ? id : -1;
    }
};

template <class T, int NQ, int DP>
__device__ __forceinline__ void attend(const AttnArgs &a, const AttnSpan &s) {
    constexpr int KC = DP / 32;            // key chunks of 32 elements
    constexpr int EL = DP < 128 ? DP / 16 : 8;  // neighbouring elements of a value row in one lane
    constexpr int NH = DP / (16 * EL);     // such runs
    constexpr int VW = EL / 2;             // their words
    const int lane = threadIdx.x & 63;
    const int n = lane & 15, g = lane >> 4;
    const int D = a.head_dim, pmask = (1 << a.page_log2) - 1;

    // query rows as second operands; rows past the last and elements past head_dim are zero
    u32v4 q[NQ][KC];
    int vis[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const int row = s.row0 + 16 * i + n;
        const int j = row / a.group;
        const T *p = static_cast<const T *>(a.q) + (int64_t)(s.tok0 + j) * a.q_ts +
                     (int64_t)(s.head * a.group + row - j * a.group) * a.q_hs;
        vis[i] = s.causal ? s.len - (s.n_tok - 1 - j) : s.len;
        if (row >= s.n_rows) vis[i] = s.len;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            const int d0 = 32 * c + 8 * g;
            q[i][c] = u32v4{0, 0, 0, 0};
            if (row < s.n_rows && d0 < D) q[i][c] = *reinterpret_cast<const u32v4 *>(p + d0);
        }
    }
    // positions every row of the segment sees: steps below need no mask
    const int all_see = s.causal ? s.len - (s.n_tok - 1) : s.len;

    // element offsets of this lane inside a 16-position tile of a page
    int koff[KC], voff[NH];
#pragma unroll
    for (int c = 0; c < KC; ++c) koff[c] = n * a.k_rs + (32 * c + 8 * g < D ? 32 * c + 8 * g : 0);
#pragma unroll
    for (int h = 0; h < NH; ++h) voff[h] = 4 * g * a.v_rs + (16 * EL * h + EL * n < D ? 16 * EL * h + EL * n : 0);
    const T *kbase = static_cast<const T *>(a.k) + (int64_t)s.head * a.k_hs;
    const T *vbase = static_cast<const T *>(a.v) + (int64_t)s.head * a.v_hs;

    f32x4 o[NQ][NH * EL];
    float m[NQ], l[NQ], lr[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        m[i] = kNone;
        l[i] = lr[i] = 0.0f;
#pragma unroll
        for (int c = 0; c < NH * EL; ++c) o[i][c] = f32x4{0, 0, 0, 0};
    }

    AttnPages pages;
    auto load_keys = [&](int pos, int id, u32v4 (&k)[KC]) {
#pragma unroll
        for (int c = 0; c < KC; ++c) k[c] = u32v4{0, 0, 0, 0};
        if (id >= 0) {
            const T *p = kbase + (int64_t)id * a.k_ps + (int64_t)(pos & pmask) * a.k_rs;
#pragma unroll
            for (int c = 0; c < KC; ++c) k[c] = __builtin_nontemporal_load(reinterpret_cast<const u32v4 *>(p + koff[c]));
        }
    };
    auto load_values = [&](int pos, int id, uint32_t (&v)[4][NH][VW]) {
        if (id >= 0) {
            const T *p = vbase + (int64_t)id * a.v_ps + (int64_t)(pos & pmask) * a.v_rs;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const T *e = p + r * a.v_rs + voff[h];
                    if constexpr (VW == 4) {
                        const u32v4 w = __builtin_nontemporal_load(reinterpret_cast<const u32v4 *>(e));
                        v[r][h][0] = w.x, v[r][h][1] = w.y, v[r][h][2] = w.z, v[r][h][3] = w.w;
                    } else {
                        const u32x2 w = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(e));
                        v[r][h][0] = w.x, v[r][h][1] = w.y;
                    }
                }
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int w = 0; w < VW; ++w) v[r][h][w] = 0;
        }
    };

    int kv0 = s.pos0;
    const int end = min(s.len, s.pos1);
    u32v4 k0[KC], k1[KC];
    pages.start(a, s, kv0);
    int id0 = pages.of(a, s, kv0 >> 4), id1 = pages.of(a, s, (kv0 >> 4) + 1);
    load_keys(kv0, id0, k0);
    load_keys(kv0 + 16, id1, k1);
    while (kv0 < end) {
        uint32_t v[8][NH][VW];
        load_values(kv0, id0, *reinterpret_cast<uint32_t(*)[4][NH][VW]>(&v[0]));
        load_values(kv0 + 16, id1, *reinterpret_cast<uint32_t(*)[4][NH][VW]>(&v[4]));

        f32x4 sc[NQ][2];
#pragma unroll
        for (int i = 0; i < NQ; ++i) sc[i][0] = sc[i][1] = f32x4{0, 0, 0, 0};
        if (D != DP) {  // elements past head_dim: the query's are zero, a non-finite key's must not meet them
#pragma unroll
            for (int c = 0; c < KC; ++c)
                if (32 * c + 8 * g >= D) k0[c] = k1[c] = u32v4{0, 0, 0, 0};
        }
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                sc[i][0] = mma<T>(k0[c], q[i][c], sc[i][0]);
                sc[i][1] = mma<T>(k1[c], q[i][c], sc[i][1]);
            }
        const int here = kv0, c0 = id0, c1 = id1;
        kv0 += kAttnStep;
        if (kv0 < end) {  // the next step's keys
            id0 = pages.of(a, s, kv0 >> 4);
            id1 = pages.of(a, s, (kv0 >> 4) + 1);
            load_keys(kv0, id0, k0);
            load_keys(kv0 + 16, id1, k1);
        }
        bool odd = false;  // a value that only some rows see is not finite
        if (here + kAttnStep > all_see || (c0 | c1) < 0) {
            uint32_t found = 0;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int pos = here + 16 * t + 4 * g + r;
                    const bool page = (t ? c1 : c0) >= 0;
#pragma unroll
                    for (int i = 0; i < NQ; ++i)
                        if (!page || pos >= vis[i]) sc[i][t][r] = kNone;
                    if (pos >= s.len) {  // zero weight times whatever the page holds there is not zero
#pragma unroll
                        for (int h = 0; h < NH; ++h)
#pragma unroll
                            for (int w = 0; w < VW; ++w) v[4 * t + r][h][w] = 0;
                    } else if (pos >= all_see) {
#pragma unroll
                        for (int h = 0; h < NH; ++h)
#pragma unroll
                            for (int w = 0; w < VW; ++w) found |= maybe_not_finite<T>(v[4 * t + r][h][w]);
                    }
                }
            odd = __any(found != 0);
        }
        u32v4 p[NQ];
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            // The weights are taken against a shift, not the exact maximum: while a lane's sum of a step stays
            // below kShiftLimit no weight has lost anything, in float32 or in 16 bits, and no maximum is formed.
            // Otherwise (the first step, a score far above all before it, NaN) the shift becomes the maximum less kLift.
            f32x8 w;
            float sum = 0.0f;
            const auto weigh = [&](float shift) {
                sum = 0.0f;
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    w[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i][r >> 2][r & 3], a.scale_log2, -shift));
                    sum += w[r];
                }
            };
            weigh(m[i]);  // (a shift of minus infinity gives infinities or NaN, which take the branch)
            if (__any(!(sum < kShiftLimit<T>))) {
                float top = kNone;
#pragma unroll
                for (int r = 0; r < 4; ++r) top = fmaxf(top, fmaxf(sc[i][0][r], sc[i][1][r]));
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32)) * a.scale_log2;
                const float up = fmaxf(m[i], top - kLift<T>);
                const float f = up == m[i] ? 1.0f : __builtin_amdgcn_exp2f(m[i] - up);
                m[i] = up;
                l[i] *= f;
                lr[i] *= f;
#pragma unroll
                for (int c = 0; c < NH * EL; ++c) o[i][c] *= f;
                weigh(up == kNone ? 0.0f : up);
            }
            l[i] += sum;
            // Weights in 16 bits: the matrix cores' operand. Half a step of relative error each, averaged over the
            // positions; o is divided by the sum of the weights as rounded, so that errors that they share (weights
            // nearly alike round alike) cancel. lse takes the sum of the unrounded ones.
            p[i] = __builtin_bit_cast(u32v4, __builtin_convertvector(w, typename Vec8<T>::type));
            lr[i] = sum8<T>(p[i], lr[i]);
        }
        // Tile c of V^T (elements 8 m + c of run h): two positions of one element from two words.
        const auto turned = [&](int h, int c) {
            u32v4 f;
#pragma unroll
            for (int w = 0; w < 4; ++w)
                f[w] = __builtin_amdgcn_perm(v[2 * w + 1][h][c >> 1], v[2 * w][h][c >> 1], c & 1 ? 0x07060302u : 0x05040100u);
            return f;
        };
        if (!odd) {
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int c = 0; c < EL; ++c) {
                    const u32v4 f = turned(h, c);
#pragma unroll
                    for (int i = 0; i < NQ; ++i) o[i][h * EL + c] = mma<T>(f, p[i], o[i][h * EL + c]);
                }
        } else {
            // One query token at a time, the last first: the values that it does not see are set to zero, and only its
            // rows take the result.
            const int last = min(s.n_tok, (s.row0 + 16 * NQ - 1) / a.group + 1);
            for (int j = last - 1; j >= s.row0 / a.group; --j) {
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    if (here + 16 * (x >> 2) + 4 * g + (x & 3) >= s.len - (s.n_tok - 1 - j)) {
#pragma unroll
                        for (int h = 0; h < NH; ++h)
#pragma unroll
                            for (int w = 0; w < VW; ++w) v[x][h][w] = 0;
                    }
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int c = 0; c < EL; ++c) {
                        const u32v4 f = turned(h, c);
#pragma unroll
                        for (int i = 0; i < NQ; ++i) {
                            const f32x4 x = mma<T>(f, p[i], o[i][h * EL + c]);
                            if ((s.row0 + 16 * i + n) / a.group == j) o[i][h * EL + c] = x;
                        }
                    }
            }
        }
    }

#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        l[i] += __shfl_xor(l[i], 16);
        l[i] += __shfl_xor(l[i], 32);
        lr[i] += __shfl_xor(lr[i], 16);
        lr[i] += __shfl_xor(lr[i], 32);
        const int row = 16 * i + n;
        if (s.row0 + row >= s.n_rows) continue;
        if (g == 0) s.pml[row] = make_float4(stored_shift(m[i], l[i]), l[i], lr[i], 0.0f);
        float *po = s.po + row * DP;
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < EL; c += 4) {
                    f32x4 x;
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = o[i][h * EL + c + e][r];
                    *reinterpret_cast<f32x4 *>(po + 16 * EL * h + EL * (4 * g + r) + c) = x;
                }
    }
}

// ------------------------------------------------------------------------------------------------
// Many query rows (the prefix of a batch). Here the matrix cores and the exponentials are the bound, not
// the memory (256 query tokens of 32 heads over 32768 positions: 0.97 PFLOP/s, matrix cores 38 % busy): 64 or 128 rows share each key, so keys and values go once through LDS for the four waves,
// moved there by the loads themselves (16 bytes a lane, no registers), one tile of kWideTile positions
// ahead of its use. A wave holds 32 rows: with 32x32x16 products an operand read from LDS serves 32
// rows, and two waves share a SIMD, so one's products run under the other's exponentials.
//  - WQ = 4: a wave to each 32 of 128 rows, all positions; WQ = 2: 64 rows, two waves to each 32, half of a
//    tile's positions each, joined at the end.
//  - Weights stay in registers as above: a lane's 16 scores of 32 positions are the second operands of
//    two products once their 16 positions each are numbered (register / 4, lane / 32, register % 4).
//  - Values are read from LDS transposed (ds_read_b64_tr_b16: 16 lanes read 4 positions x 16 elements, each
//    gets 4 positions of one element).
//  - The 16-byte chunks of a row are permuted by an exclusive-or with a key of the row, chosen so that the
//    rows one instruction reads lie in different banks.

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) uint8_t lds_u8;

template <class T>
__device__ __forceinline__ f32x16 mma32(u32v4 a, u32v4 b, f32x16 c);
template <>
__device__ __forceinline__ f32x16 mma32<__bf16>(u32v4 a, u32v4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x16 mma32<_Float16>(u32v4 a, u32v4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Loads straight to LDS: N times 16 bytes a lane, the i-th from `base` (the same in all lanes) + offset[i] to LDS at
// `dst` (the same) + 1024 i + 16 * lane. Waited for by vmcnt. Written as asm (m0, which holds the LDS
// address, is put back) because the compiler makes every later LDS read wait for loads to LDS that it knows
// of, whatever part of LDS they write; the asm writes no register that a load fills. An instruction's
// offset moves both of its addresses, so the i-th lane offset is given 1024 i less.
template <int N>
__device__ __forceinline__ void load_to_lds(uint32_t dst, const void *base, const uint32_t (&offset)[N]) {
    uint32_t keep;
    if constexpr (N == 4)
        asm volatile(
            "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
            "global_load_lds_dwordx4 %2, %6\n\tglobal_load_lds_dwordx4 %3, %6 offset:0x400\n\t"
            "global_load_lds_dwordx4 %4, %6 offset:0x800\n\tglobal_load_lds_dwordx4 %5, %6 offset:0xc00\n\t"
            "s_mov_b32 m0, %0"
            : "=&s"(keep)
            : "s"(dst), "v"(offset[0]), "v"(offset[1]), "v"(offset[2]), "v"(offset[3]), "s"(base)
            : "memory");
    else if constexpr (N == 2)
        asm volatile(
            "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\t"
            "global_load_lds_dwordx4 %2, %4\n\tglobal_load_lds_dwordx4 %3, %4 offset:0x400\n\t"
            "s_mov_b32 m0, %0"
            : "=&s"(keep)
            : "s"(dst), "v"(offset[0]), "v"(offset[1]), "s"(base)
            : "memory");
    else
        asm volatile(
            "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3\n\ts_mov_b32 m0, %0"
            : "=&s"(keep)
            : "s"(dst), "v"(offset[0]), "s"(base)
            : "memory");
}
__device__ __forceinline__ void wait_loads_to_lds() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Chunk keys. Rows of 128 bytes (DP = 64) come two to the 256 bytes of all banks, longer ones one or less.
template <int DP>
__device__ __forceinline__ int key_of_k(int row) {
    return DP == 64 ? (row >> 1) & 7 : row & 15;
}
template <int DP>
__device__ __forceinline__ int key_of_v(int row) {
    return DP == 64 ? ((row >> 1) & 1) << 2 : ((row & 3) << 2) | ((row >> 2) & 3);
}

template <int DP>
struct WideLds {
    alignas(16) uint8_t k[2][kWideTile * DP * 2];
    alignas(16) uint8_t v[2][kWideTile * DP * 2];
};

template <class T, int DP, int WQ>
__device__ __forceinline__ void attend_wide(const AttnArgs &a, const AttnSpan &s, WideLds<DP> &lds) {
    constexpr int ROW = DP * 2, CPR = DP / 8, RPI = 64 / CPR;  // row bytes, chunks of a row, rows of one load
    constexpr int KC = DP / 16, DB = DP / 32;
    constexpr int PARTS = kAttnWaves / WQ, NB = kWideTile / 32 / PARTS;  // waves along a tile, blocks of 32 of each
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, g = lane >> 5, part = wave / WQ;
    const int D = a.head_dim, pmask = (1 << a.page_log2) - 1;
    const int row_first = s.row0 + 32 * (wave % WQ), row = row_first + n;

    u32v4 q[KC];
    {
        const int j = row / a.group;
        const T *p = static_cast<const T *>(a.q) + (int64_t)(s.tok0 + j) * a.q_ts +
                     (int64_t)(s.head * a.group + row - j * a.group) * a.q_hs;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            q[c] = u32v4{0, 0, 0, 0};
            if (row < s.n_rows && 16 * c + 8 * g < D) q[c] = *reinterpret_cast<const u32v4 *>(p + 16 * c + 8 * g);
        }
    }
    const T *kbase = static_cast<const T *>(a.k) + (int64_t)s.head * a.k_hs;
    const T *vbase = static_cast<const T *>(a.v) + (int64_t)s.head * a.v_hs;

    constexpr int LOADS = 16 / RPI, GROUP = LOADS < 4 ? LOADS : 4;  // loads of a wave's sixteen rows, of one asm block
    const uint32_t lds_k = (uint32_t)(size_t)(lds_u8 *)lds.k, lds_v = (uint32_t)(size_t)(lds_u8 *)lds.v;
    // byte offsets of this lane's chunks within its wave's sixteen rows (less 1024 for each place in its block)
    uint32_t ks[LOADS], vs[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int r = RPI * i + lane / CPR;
        ks[i] = 2 * (r * a.k_rs + 8 * ((lane % CPR) ^ key_of_k<DP>(r))) - 1024 * (i % GROUP);
        vs[i] = 2 * (r * a.v_rs + 8 * ((lane % CPR) ^ key_of_v<DP>(r))) - 1024 * (i % GROUP);
    }
    // Pages, a granule of 16 positions a lane: the byte addresses of the granules of 16 tiles, and which of them are
    // there; the page numbers of the 16 tiles after.
    int32_t next;
    uint64_t kat, vat, there;
    const auto fetch = [&](int pos) {
        const int at = pos + 16 * lane;
        next = -1;
        if (at < s.len) next = s.pages[at >> a.page_log2];
    };
    const auto turn_pages = [&](int pos) {
        const bool in = (uint32_t)next < (uint32_t)a.n_pages;
        const int64_t id = in ? next : 0;
        const int64_t first = (pos + 16 * lane) & pmask;
        kat = (uint64_t)(kbase + id * a.k_ps + first * a.k_rs);
        vat = (uint64_t)(vbase + id * a.v_ps + first * a.v_rs);
        there = __ballot(in);
        fetch(pos + 1024);
    };
    const auto lane_of = [](uint64_t x, int l) {
        return (const uint8_t *)(((uint64_t)(uint32_t)__builtin_amdgcn_readlane((uint32_t)(x >> 32), l) << 32) |
                                 (uint32_t)__builtin_amdgcn_readlane((uint32_t)x, l));
    };
    // Moves tile `pos` to LDS, this wave's 16 positions of it: hidden positions and elements past head_dim become
    // zeros (a zero weight times whatever memory holds there would not be one). Gives which granules are there.
    const auto issue = [&](int buf, int pos) -> uint32_t {
        if (((pos - s.pos0) & 1023) == 0) turn_pages(pos);
        const int tile = ((pos - s.pos0) >> 4) & 63, first = pos + 16 * wave;
        const uint32_t seen = (uint32_t)(there >> tile) & 15;
        const uint8_t *kp = lane_of(kat, tile + wave), *vp = lane_of(vat, tile + wave);
        const uint32_t at = buf * (kWideTile * ROW) + 16 * wave * ROW;
        if (seen == 15 && pos + kWideTile <= s.len && D == DP) {
#pragma unroll
            for (int i = 0; i < LOADS; i += GROUP) {
                load_to_lds<GROUP>(lds_k + at + 1024 * i, kp, reinterpret_cast<const uint32_t(&)[GROUP]>(ks[i]));
                load_to_lds<GROUP>(lds_v + at + 1024 * i, vp, reinterpret_cast<const uint32_t(&)[GROUP]>(vs[i]));
            }
            return seen;
        }
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int r = RPI * i + lane / CPR;  // of the wave's sixteen
            const bool in = ((seen >> wave) & 1) && first + r < s.len;
            const int ck = (lane % CPR) ^ key_of_k<DP>(r), cv = (lane % CPR) ^ key_of_v<DP>(r);
            const uint32_t ko[1] = {ks[i] + 1024 * (i % GROUP)}, vo[1] = {vs[i] + 1024 * (i % GROUP)};
            if (in && 8 * ck < D)
                load_to_lds<1>(lds_k + at + 1024 * i, kp, ko);
            else
                *reinterpret_cast<u32v4 *>(&lds.k[buf][16 * wave * ROW + 1024 * i + 16 * lane]) = u32v4{0, 0, 0, 0};
            if (in && 8 * cv < D)
                load_to_lds<1>(lds_v + at + 1024 * i, vp, vo);
            else
                *reinterpret_cast<u32v4 *>(&lds.v[buf][16 * wave * ROW + 1024 * i + 16 * lane]) = u32v4{0, 0, 0, 0};
        }
        return seen;
    };

    // LDS addresses of this lane's reads; blocks of 32 (and 16) positions are whole keys apart
    uint32_t ka[KC], va[DB][2];
#pragma unroll
    for (int c = 0; c < KC; ++c) ka[c] = n * ROW + (((2 * c + g) ^ key_of_k<DP>(n)) * 16);
#pragma unroll
    for (int c = 0; c < DB; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = lane & 15, r = 8 * h + 4 * g + (i >> 2);
            const int chunk = 4 * c + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
            va[c][h] = r * ROW + ((chunk ^ key_of_v<DP>(r)) * 16) + (i & 1) * 8;
        }

    f32x16 o[DB];
#pragma unroll
    for (int c = 0; c < DB; ++c) o[c] = f32x16{};
    float m = kNone, l = 0.0f, lr = 0.0f;

    const int end = min(s.len, s.pos1);
    int pos0 = s.pos0;
    fetch(pos0);
    uint32_t seen_next = issue(0, pos0);
    // Tile `pos0`, which lies in LDS buffer BUF.
    const auto tile = [&](auto which) {
        constexpr int buf = decltype(which)::value;
        const uint32_t seen = seen_next;
        const bool hidden = seen != 15 || pos0 + kWideTile > s.len;
        wait_loads_to_lds();
        __syncthreads();  // this tile is there, and nobody reads the one before it any more
        if (pos0 + kWideTile < end) seen_next = issue(buf ^ 1, pos0 + kWideTile);

        // The tile's blocks of 32 positions, one after another: a block's weights are formed beside the products of
        // the next block's scores and of the last block's values, which wait for nothing of them. Operands are read
        // from LDS a group of products ahead.
        constexpr int GK = 4, NGB = KC / GK, NG = NB * NGB;
        f32x16 sc[NB];
        u32v4 kf[2][GK], vf[2][DB], p[NB][2];
        const auto read_k = [&](int x) {
            const uint8_t *q0 = &lds.k[buf][(part * NB + x / NGB) * 32 * ROW];
#pragma unroll
            for (int c = 0; c < GK; ++c) kf[x & 1][c] = *reinterpret_cast<const u32v4 *>(q0 + ka[(x * GK + c) % KC]);
        };
        const auto read_v = [&](int x) {  // positions 16 x .. 16 x + 15 of this wave's blocks
            const uint8_t *v0 = &lds.v[buf][(32 * part * NB + 16 * x) * ROW];
#pragma unroll
            for (int c = 0; c < DB; ++c) {
                const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(lds_u8 *)(v0 + va[c][0])));
                const u32x2 z = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(lds_u8 *)(v0 + va[c][1])));
                vf[x & 1][c] = u32v4{y.x, y.y, z.x, z.y};
            }
        };
        const auto scores = [&](int b) {
            sc[b] = f32x16{};
#pragma unroll
            for (int x = b * NGB; x < (b + 1) * NGB; ++x) {
                if (x + 1 < NG) read_k(x + 1);
#pragma unroll
                for (int c = 0; c < GK; ++c) sc[b] = mma32<T>(kf[x & 1][c], q[(x * GK + c) % KC], sc[b]);
            }
        };
        const auto values = [&](int b) {
#pragma unroll
            for (int x = 2 * b; x < 2 * b + 2; ++x) {
                if (x + 1 < 2 * NB) read_v(x + 1);
#pragma unroll
                for (int c = 0; c < DB; ++c) o[c] = mma32<T>(vf[x & 1][c], p[b][x & 1], o[c]);
            }
        };
        f32x8 w[2];
        float sum;
        const auto hide = [&](int b) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int at = 32 * (part * NB + b) + 8 * (r >> 2) + 4 * g + (r & 3);
                if (pos0 + at >= s.len || !((seen >> (at >> 4)) & 1)) sc[b][r] = kNone;
            }
        };
        const auto weigh = [&](int b, float shift) {
            float part_sum[2] = {0.0f, 0.0f};
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[b][r], a.scale_log2, -shift));
                w[r >> 3][r & 7] = e;
                part_sum[r >> 3] += e;
            }
            sum = part_sum[0] + part_sum[1];
        };
        const auto settle = [&](int b) {  // the shift raised where it has to be, as in the narrow path; weights in 16 bits
            if (__any(!(sum < kShiftLimit<T>))) {
                float top = kNone;
#pragma unroll
                for (int r = 0; r < 16; ++r) top = fmaxf(top, sc[b][r]);
                top = fmaxf(top, __shfl_xor(top, 32)) * a.scale_log2;
                const float up = fmaxf(m, top - kLift<T>);
                const float f = up == m ? 1.0f : __builtin_amdgcn_exp2f(m - up);
                m = up;
                l *= f;
                lr *= f;
#pragma unroll
                for (int c = 0; c < DB; ++c) o[c] *= f;
                weigh(b, up == kNone ? 0.0f : up);
            }
            l += sum;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                p[b][h] = __builtin_bit_cast(u32v4, __builtin_convertvector(w[h], typename Vec8<T>::type));
                lr = sum8<T>(p[b][h], lr);
            }
        };
        // Where a SIMD holds one wave (DP = 256): one product, then VALU instructions that issue while it runs. A wave
        // issues in order, so the order in the program is what overlaps: 102 us with it, 114 without (64 tokens of
        // 32 heads over 16384 positions). With two waves a SIMD the other one fills in: 179 us without it, 185 with.
        const auto alternate = [](auto products) {
            if constexpr (DP > 128) {
#pragma unroll
                for (int i = 0; i < decltype(products)::value; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, 7, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        read_k(0);
        scores(0);
        read_v(0);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (NB == 2) {
            if (hidden) hide(0);
            weigh(0, m);
            scores(1);
            alternate(std::integral_constant<int, KC>{});
            settle(0);
            if (hidden) hide(1);
            values(0);
            weigh(1, m);
            alternate(std::integral_constant<int, 2 * DB>{});
            settle(1);
            values(1);
        } else {
            if (hidden) hide(0);
            weigh(0, m);
            settle(0);
            values(0);
        }
        pos0 += kWideTile;
    };
    while (true) {
        tile(std::integral_constant<int, 0>{});
        if (pos0 >= end) break;
        tile(std::integral_constant<int, 1>{});
        if (pos0 >= end) break;
    }

    l += __shfl_xor(l, 32);
    lr += __shfl_xor(lr, 32);
    m = stored_shift(m, l);
    if constexpr (PARTS == 2) {  // the second wave of the same rows hands over through LDS
        constexpr int PAD = DP + 4;
        float *box = reinterpret_cast<float *>(&lds) + (wave % WQ) * (32 * PAD);
        float4 *ml = reinterpret_cast<float4 *>(reinterpret_cast<float *>(&lds) + WQ * 32 * PAD) + 32 * (wave % WQ);
        static_assert((WQ * 32 * PAD + 4 * 32 * WQ) * 4 <= sizeof(WideLds<DP>), "the join fits the tiles' LDS");
        __syncthreads();
        if (part == 1) {
#pragma unroll
            for (int c = 0; c < DB; ++c)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    *reinterpret_cast<f32x4 *>(box + n * PAD + 32 * c + 8 * r + 4 * g) =
                        f32x4{o[c][4 * r], o[c][4 * r + 1], o[c][4 * r + 2], o[c][4 * r + 3]};
            if (g == 0) ml[n] = make_float4(m, l, lr, 0.0f);
        }
        __syncthreads();
        if (part == 0) {
            const float4 x = ml[n];
            const float up = fmaxf(m, x.x);
            const float f0 = m == kNone ? 0.0f : __builtin_amdgcn_exp2f(m - up), f1 = x.x == kNone ? 0.0f : __builtin_amdgcn_exp2f(x.x - up);
            m = up;
            l = l * f0 + x.y * f1;
            lr = lr * f0 + x.z * f1;
#pragma unroll
            for (int c = 0; c < DB; ++c)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const f32x4 y = *reinterpret_cast<const f32x4 *>(box + n * PAD + 32 * c + 8 * r + 4 * g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[c][4 * r + e] = o[c][4 * r + e] * f0 + y[e] * f1;
                }
        }
    }
    if (part == 0 && row < s.n_rows) {
        const int at = 32 * (wave % WQ) + n;
        if (g == 0) s.pml[at] = make_float4(m, l, lr, 0.0f);
        float *po = s.po + (int64_t)at * DP;
#pragma unroll
        for (int c = 0; c < DB; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                *reinterpret_cast<f32x4 *>(po + 32 * c + 8 * r + 4 * g) =
                    f32x4{o[c][4 * r], o[c][4 * r + 1], o[c][4 * r + 2], o[c][4 * r + 3]};
    }
    __syncthreads();  // LDS is free for the next item
}

// Query tokens of sequence b: first token and count, cut to what exists.
__device__ __forceinline__ int2 seq_tokens(const AttnArgs &a, int b) {
    const int t0 = min(max(a.q_starts[b], 0), a.n_tokens), t1 = min(max(a.q_starts[b + 1], t0), a.n_tokens);
    return make_int2(t0, min(t1 - t0, a.max_q));
}
__device__ __forceinline__ int seq_len(const AttnArgs &a, int b) { return min(max(a.lens[b], 0), a.cap); }

// What the workgroups know of the sequences, in LDS: [n_seqs + 1] units and items before each, then first token,
// tokens and length of each.
struct AttnSeqs {
    int32_t *units, *items, *tok0, *n_tok, *len;
    __device__ __forceinline__ AttnSeqs(int32_t *p, int n)
        : units(p), items(p + n + 1), tok0(p + 2 * (n + 1)), n_tok(p + 3 * (n + 1)), len(p + 4 * (n + 1)) {}
};

// MP, MS: query rows of a tile in the prefix (16, 32: a wave's, from registers; 64, 128: a workgroup's, through
// LDS) and in a suffix (16, 32: a wave's).
template <class T, int DP, int MP, int MS>
__global__ __launch_bounds__(kAttnThreads, DP <= 128 ? 2 : 1) void attn_split_kernel(AttnArgs a) {
    constexpr bool WIDE = MP > 32;
    constexpr int UNIT_P = WIDE ? kWideTile : kAttnStep;
    extern __shared__ int32_t dynamic[];
    __shared__ int32_t wave_sum[kAttnWaves][2];
    AttnSeqs seqs(dynamic, a.n_seqs);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    // The sequences' tokens and lengths, read ahead of everything else (each thread reads back its own).
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int b = 4 * tid + x;
        if (b < a.n_seqs) {
            const int2 tok = seq_tokens(a, b);
            seqs.tok0[b] = tok.x;
            seqs.n_tok[b] = tok.y;
            seqs.len[b] = seq_len(a, b);
        }
    }

    AttnSpan s;
    s.pages = a.prefix_pages;
    s.len = a.prefix_len;
    s.tok0 = 0;
    s.n_tok = a.n_tokens;
    s.causal = 0;
    s.n_rows = a.n_tokens * a.group;

    // A wide prefix comes first: the host has cut every item (head x tile) alike into pieces, so that workgroups that
    // read the same keys for other rows go through them together, and each XCD's workgroups (workgroup b runs on
    // XCD b % 8) take `per_xcd` neighbouring pieces in turns, sharing that XCD's L2. The suffixes come after it.
    // (Letting half of the workgroups take their suffixes first, to run memory-bound work beside the products,
    // measured slower: 186 us against 179 for 256 tokens over a prefix of 32768, by spilled registers.)
    const int up = (a.prefix_len + UNIT_P - 1) / UNIT_P, total_p = a.kv_heads * a.tiles_p * up;
    const int pieces = a.kv_heads * a.tiles_p * a.splits, per_xcd = (pieces + 7) / 8, wgs_xcd = gridDim.x >> 3;
    const int xcd = blockIdx.x & 7, at = blockIdx.x >> 3;
    if constexpr (WIDE) {
        __shared__ WideLds<DP> lds;
        for (int i = at; i < per_xcd; i += wgs_xcd) {
            const int piece = xcd * per_xcd + i;
            if (piece >= pieces) break;
            const int hs = piece / a.tiles_p, tile = piece - hs * a.tiles_p;
            s.head = hs / a.splits;
            s.row0 = tile * MP;
            s.pos0 = (hs - s.head * a.splits) * a.split_units * UNIT_P;
            s.pos1 = s.pos0 + a.split_units * UNIT_P;
            s.po = a.part_o + (int64_t)piece * (MP * DP);
            s.pml = a.part_ml + (int64_t)piece * MP;
            attend_wide<T, DP, MP / 32>(a, s, lds);
        }
    }

    // Units and items before each sequence: four sequences a thread, then a scan.
    int un[4], it[4], su = 0, si = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int b = 4 * tid + x;
        un[x] = it[x] = 0;
        if (b < a.n_seqs) {
            const int u = (seqs.len[b] + kAttnStep - 1) / kAttnStep;
            it[x] = u > 0 ? a.kv_heads * ((seqs.n_tok[b] * a.group + MS - 1) / MS) : 0;
            un[x] = it[x] * u;
        }
        su += un[x];
        si += it[x];
    }
    int iu = scan_add(su), ii = scan_add(si);
    if (lane == 63) wave_sum[wave][0] = iu, wave_sum[wave][1] = ii;
    __syncthreads();
    int total_s = 0, items_s = 0;
#pragma unroll
    for (int x = 0; x < kAttnWaves; ++x) {
        if (x < wave) iu += wave_sum[x][0], ii += wave_sum[x][1];
        total_s += wave_sum[x][0];
        items_s += wave_sum[x][1];
    }
    total_s = __builtin_amdgcn_readfirstlane(total_s);
    items_s = __builtin_amdgcn_readfirstlane(items_s);
    int eu = iu - su, ei = ii - si;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int b = 4 * tid + x;
        if (b < a.n_seqs) seqs.units[b] = eu, seqs.items[b] = ei;
        eu += un[x], ei += it[x];
        if (b == a.n_seqs - 1) seqs.units[a.n_seqs] = eu, seqs.items[a.n_seqs] = ei;
    }

    // The dealing (deal_narrow, deal_wide).
    const int turns = WIDE ? (per_xcd + wgs_xcd - 1) / wgs_xcd : 0, busy_xcd = per_xcd - (turns - 1) * wgs_xcd;
    const int idle = WIDE ? 8 * (wgs_xcd - busy_xcd) : 0;
    const AttnDeal deal = WIDE ? deal_wide(total_s, items_s, idle, a.split_units, MP == 64, gridDim.x)
                               : deal_narrow(total_p, total_s, gridDim.x);
    const int qf = deal.qf, qb = deal.qb, wp = deal.wp, runs_f = deal.runs_f;
    __syncthreads();
    if (blockIdx.x == 0) {  // what the join needs
        if (tid == 0) a.sched[0] = up, a.sched[1] = qf, a.sched[2] = qb, a.sched[3] = runs_f;
        for (int b = tid; b <= a.n_seqs; b += kAttnThreads) {
            a.sched[kSchedHead + b] = seqs.units[b];
            a.sched[kSchedHead + a.n_seqs + 1 + b] = seqs.items[b];
        }
    }
    // This wave's run of the suffixes, run w: units [u, stop).
    const auto suffixes = [&](int w, int u, int stop) {
        if (u >= stop) return;
        int b = 0;  // the sequence that holds unit u: one lane finds it
        {
            int found = -1;
            for (int i = lane; i < a.n_seqs; i += 64)
                if (seqs.units[i] <= u && u < seqs.units[i + 1]) found = i;
            b = __builtin_amdgcn_readlane(found, __builtin_ctzll(__ballot(found >= 0)));
        }
        AttnSpan s;
        while (u < stop) {
            while (seqs.units[b + 1] <= u) ++b;  // past idle sequences
            b = __builtin_amdgcn_readfirstlane(b);
            const int len = __builtin_amdgcn_readfirstlane(seqs.len[b]), ub = (len + kAttnStep - 1) / kAttnStep;
            const int n_tok = __builtin_amdgcn_readfirstlane(seqs.n_tok[b]), tiles = (n_tok * a.group + MS - 1) / MS;
            const int rest = u - __builtin_amdgcn_readfirstlane(seqs.units[b]);
            const int item = rest / ub, at = rest - item * ub, n = min(ub - at, stop - u);
            const int64_t part = __builtin_amdgcn_readfirstlane(seqs.items[b]) + item + w;
            s.pages = a.table + (int64_t)b * a.table_stride;
            s.len = len;
            s.tok0 = __builtin_amdgcn_readfirstlane(seqs.tok0[b]);
            s.n_tok = n_tok;
            s.causal = 1;
            s.head = item / tiles;
            s.row0 = (item - s.head * tiles) * MS;
            s.n_rows = n_tok * a.group;
            s.pos0 = at * kAttnStep;
            s.pos1 = (at + n) * kAttnStep;
            s.po = a.part_o + a.part_s + part * (MS * DP);
            s.pml = a.part_ml + a.ml_s + part * MS;
            attend<T, MS / 16, DP>(a, s);
            u += n;
        }
    };
    if constexpr (WIDE) {
        const int w = wide_run(blockIdx.x, wave, busy_xcd, idle);
        const int u = w < runs_f ? w * qf : runs_f * qf + (w - runs_f) * qb;
        suffixes(w, u, min(total_s, u + (w < runs_f ? qf : qb)));
    } else {
        // Runs are spread over the workgroups first, so that few of them use many CUs.
        const int w = wave * gridDim.x + blockIdx.x;
        if (w >= wp) {
            suffixes(w - wp, (w - wp) * qb, min(total_s, (w - wp + 1) * qb));
            return;
        }
        int v = w * qb;
        const int last = min(total_p, v + qb);
        while (v < last) {
            const int item = v / up, at = v - item * up, n = min(up - at, last - v);
            s.head = item / a.tiles_p;
            s.row0 = (item - s.head * a.tiles_p) * MP;
            s.pos0 = at * UNIT_P;
            s.pos1 = (at + n) * UNIT_P;
            s.po = a.part_o + (int64_t)(item + w) * (MP * DP);
            s.pml = a.part_ml + (int64_t)(item + w) * MP;
            attend<T, MP / 16, DP>(a, s);
            v += n;
        }
    }
}

// The parts of one query row: np of the prefix, then ns of its sequence.
struct AttnParts {
    int np, ns;
    int t;                    // token, or -1: none
    int64_t row_p, row_s;     // first part's row among all rows of parts
    int step_p, ms;           // rows from one part to the next

    __device__ __forceinline__ AttnParts(const AttnArgs &a, int mp, int ms_, int b, int j, int hq) : step_p(0), ms(ms_) {
        const int2 tok = seq_tokens(a, b);
        const int up = a.sched[0], qb = a.sched[2];
        const AttnDeal deal{a.sched[1], qb, 0, a.sched[3]};
        const int before_u = a.sched[kSchedHead + b], before_i = a.sched[kSchedHead + a.n_seqs + 1 + b];
        const int ub = (seq_len(a, b) + kAttnStep - 1) / kAttnStep;
        const int head = hq / a.group, gi = hq - head * a.group;
        np = ns = 0;
        row_p = row_s = 0;
        t = j < tok.y ? tok.x + j : -1;
        if (t < 0) return;
        if (up > 0) {
            const int row = t * a.group + gi, tile = row / mp, item = head * a.tiles_p + tile;
            if (mp > 32) {
                np = (up + a.split_units - 1) / a.split_units;
                row_p = ((int64_t)head * a.splits * a.tiles_p + tile) * mp + row - tile * mp;
                step_p = a.tiles_p * mp;
            } else {
                const int w0 = item * up / qb;
                np = (item * up + up - 1) / qb - w0 + 1;
                row_p = (int64_t)(item + w0) * mp + row - tile * mp;
                step_p = mp;
            }
        }
        if (ub > 0) {
            const int row = j * a.group + gi, tile = row / ms, item = head * ((tok.y * a.group + ms - 1) / ms) + tile;
            const int u0 = before_u + item * ub, w0 = deal.run_of(u0);
            ns = deal.run_of(u0 + ub - 1) - w0 + 1;
            row_s = (int64_t)(before_i + item + w0) * ms + row - tile * ms;
        }
    }
    __device__ __forceinline__ float4 ml(const AttnArgs &a, int k) const {
        return k < np ? a.part_ml[row_p + (int64_t)k * step_p] : a.part_ml[a.ml_s + row_s + (int64_t)(k - np) * ms];
    }
    template <int DP>
    __device__ __forceinline__ const float *o(const AttnArgs &a, int k) const {
        return k < np ? a.part_o + (row_p + (int64_t)k * step_p) * DP : a.part_o + a.part_s + (row_s + (int64_t)(k - np) * ms) * DP;
    }
};

// Four elements of a row of out, its lse. top: log2 units. A sum of zero: nothing seen. (NaN is not zero.)
template <class T>
__device__ __forceinline__ void write_out(const AttnArgs &a, int t, int hq, int d, f32x4 acc, float top, float sum, float rounded) {
    if (d < a.head_dim) {
        typedef T T4 __attribute__((ext_vector_type(4)));
        T *out = static_cast<T *>(a.out) + (int64_t)t * a.o_ts + (int64_t)hq * a.o_hs + d;
        *reinterpret_cast<T4 *>(out) = __builtin_convertvector(acc * (sum == 0.0f ? 0.0f : 1.0f / rounded), T4);
    }
    if (d == 0 && a.lse)
        a.lse[(int64_t)t * a.q_heads + hq] = sum == 0.0f ? kNone : (top + __builtin_amdgcn_logf(sum)) * 0.69314718055994531f;
}

constexpr int kJoinRows = 1024;

// Joins the parts of a query row, few rows: one workgroup to a (sequence, query token, query head). The weights
// of the parts are formed once in LDS; then DP / 4 threads hold a row, so that many parts are in flight.
template <class T, int DP>
__global__ __launch_bounds__(kAttnThreads) void attn_join_kernel(AttnArgs a, int mp, int ms) {
    constexpr int LANES = DP / 4, GROUPS = kAttnThreads / LANES;
    __shared__ float weight[kAttnParts];
    __shared__ f32x4 sums[GROUPS][LANES];
    __shared__ float red[3][kAttnWaves];
    const int tid = threadIdx.x;
    const int hq = blockIdx.x % a.q_heads, bj = blockIdx.x / a.q_heads;
    const AttnParts p(a, mp, ms, bj / a.max_q, bj % a.max_q, hq);
    if (p.t < 0) return;
    const int parts = p.np + p.ns;
    const int gr = tid / LANES, ln = tid - gr * LANES;
    f32x4 y[4];  // the first parts' outputs are on their way while the weights are formed
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[i] = f32x4{0, 0, 0, 0};
        if (gr + i * GROUPS < parts) y[i] = *reinterpret_cast<const f32x4 *>(p.template o<DP>(a, gr + i * GROUPS) + 4 * ln);
    }
    float top = kNone;
    for (int k = tid; k < parts; k += kAttnThreads) top = fmaxf(top, p.ml(a, k).x);
    top = wave_max(top);
    if ((tid & 63) == 0) red[0][tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    float sum = 0.0f, rounded = 0.0f;
    for (int k = tid; k < parts; k += kAttnThreads) {
        const float4 x = p.ml(a, k);
        const float f = x.x == kNone ? 0.0f : __builtin_amdgcn_exp2f(x.x - top);
        weight[k] = f;
        sum += x.x == kNone ? 0.0f : f * x.y;
        rounded += x.x == kNone ? 0.0f : f * x.z;
    }
    sum = wave_add(sum);
    rounded = wave_add(rounded);
    if ((tid & 63) == 0) red[1][tid >> 6] = sum, red[2][tid >> 6] = rounded;
    __syncthreads();
    sum = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
    rounded = (red[2][0] + red[2][1]) + (red[2][2] + red[2][3]);
    f32x4 acc = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (gr + i * GROUPS < parts) acc += y[i] * weight[gr + i * GROUPS];
#pragma unroll 4
    for (int k = gr + 4 * GROUPS; k < parts; k += GROUPS) acc += *reinterpret_cast<const f32x4 *>(p.template o<DP>(a, k) + 4 * ln) * weight[k];
    sums[gr][ln] = acc;
    __syncthreads();
    if (gr) return;
#pragma unroll
    for (int y = 1; y < GROUPS; ++y) acc += sums[y][ln];
    write_out<T>(a, p.t, hq, 4 * ln, acc, top, sum, rounded);
}

// Many rows, which have few parts each: one wave to a row, no barriers. Row r0 is the launch's first.
template <class T, int DP>
__global__ __launch_bounds__(kAttnThreads) void attn_join_rows_kernel(AttnArgs a, int mp, int ms, int r0, int rows) {
    constexpr int LANES = DP / 4, GROUPS = 64 / LANES;
    const int lane = threadIdx.x & 63;
    const int r = __builtin_amdgcn_readfirstlane(r0 + blockIdx.x * kAttnWaves + (threadIdx.x >> 6));
    if (r >= rows) return;
    const int hq = r % a.q_heads, bj = r / a.q_heads;
    const AttnParts p(a, mp, ms, bj / a.max_q, bj % a.max_q, hq);
    if (p.t < 0) return;
    const int parts = p.np + p.ns;
    const int gr = lane / LANES, ln = lane - gr * LANES;
    f32x4 y[4];  // four outputs of each lane in flight, the first ones while the weights are formed
    const auto load = [&](int k, int n) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            y[i] = *reinterpret_cast<const f32x4 *>(p.template o<DP>(a, min(k + i * GROUPS + gr, n - 1)) + 4 * ln);
    };
    if (parts > 0) load(0, parts);
    float top = kNone;
    for (int k = lane; k < parts; k += 64) top = fmaxf(top, p.ml(a, k).x);
    top = wave_max(top);
    f32x4 acc = {0, 0, 0, 0};
    float sum = 0.0f, rounded = 0.0f;
    for (int k0 = 0; k0 < parts; k0 += 64) {
        const float4 x = k0 + lane < parts ? p.ml(a, k0 + lane) : make_float4(kNone, 0.0f, 0.0f, 0.0f);
        const float f = x.x == kNone ? 0.0f : __builtin_amdgcn_exp2f(x.x - top);  // of part k0 + lane; 0 past the last
        sum += x.x == kNone ? 0.0f : f * x.y;
        rounded += x.x == kNone ? 0.0f : f * x.z;
        const int n = min(64, parts - k0);
        for (int k = 0; k < n; k += 4 * GROUPS) {
            f32x4 z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = y[i];
            if (k0 + k + 4 * GROUPS < parts) load(k0 + k + 4 * GROUPS, parts);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float w = __shfl(f, (k + i * GROUPS + gr) & 63);
                if (k + i * GROUPS + gr < n) acc += z[i] * w;
            }
        }
    }
    sum = wave_add(sum);
    rounded = wave_add(rounded);
#pragma unroll
    for (int d = LANES; d < 64; d <<= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] += __shfl_xor(acc[e], d);
    if (gr == 0) write_out<T>(a, p.t, hq, 4 * ln, acc, top, sum, rounded);
}

// Short contexts (prefix and page table together hold few positions, and not many rows read them): one launch. A workgroup of eight waves (four where
// one needs more than half of its SIMD's registers) takes one
// (sequence, key/value head, tile of 16 query rows), its waves equal runs of the prefix's and the sequence's steps,
// and joins their parts through LDS. The prefix is read by each sequence; at these lengths it comes from the caches.
template <int DP>
constexpr int kShortWaves = DP == 256 ? 4 : 8;

template <class T, int DP>
__global__ __launch_bounds__(64 * kShortWaves<DP>) void attn_short_kernel(AttnArgs a, int tiles) {
    constexpr int WAVES = kShortWaves<DP>;
    __shared__ float part_o[WAVES][16][DP];
    __shared__ float4 part_ml[WAVES][16];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int bh = blockIdx.x / tiles, tile = blockIdx.x - bh * tiles, b = bh / a.kv_heads;
    const int2 tok = seq_tokens(a, b);
    AttnSpan s;
    s.head = bh - b * a.kv_heads;
    s.row0 = 16 * tile;
    s.n_rows = tok.y * a.group;
    if (s.row0 >= s.n_rows) return;
    s.tok0 = tok.x;
    s.n_tok = tok.y;
    const int len = seq_len(a, b), steps_p = (a.prefix_len + kAttnStep - 1) / kAttnStep, steps_s = (len + kAttnStep - 1) / kAttnStep;
    int run = max(1, (steps_p + steps_s + WAVES - 1) / WAVES);  // steps of a wave, all of one segment
    while ((steps_p + run - 1) / run + (steps_s + run - 1) / run > WAVES) ++run;
    const int waves_p = (steps_p + run - 1) / run;
    const bool own = wave >= waves_p;
    const int first = (own ? wave - waves_p : wave) * run;
    s.pages = own ? a.table + (int64_t)b * a.table_stride : a.prefix_pages;
    s.len = own ? len : a.prefix_len;
    s.causal = own;
    s.pos0 = first * kAttnStep;
    s.pos1 = s.pos0 + run * kAttnStep;
    s.po = &part_o[wave][0][0];
    s.pml = part_ml[wave];
    if (s.pos0 < s.len)
        attend<T, 1, DP>(a, s);
    else if ((tid & 63) < 16)
        part_ml[wave][tid & 63] = make_float4(kNone, 0.0f, 0.0f, 0.0f);
    __syncthreads();
    for (int i = tid; i < 16 * (DP / 4); i += 64 * kShortWaves<DP>) {
        const int row = i / (DP / 4), d = 4 * (i - row * (DP / 4));
        if (s.row0 + row >= s.n_rows) break;
        float top = kNone;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) top = fmaxf(top, part_ml[w][row].x);
        float sum = 0.0f, rounded = 0.0f;
        f32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float4 x = part_ml[w][row];
            if (x.x == kNone) continue;  // (such a part's outputs may not be there)
            const float f = __builtin_amdgcn_exp2f(x.x - top);
            sum += f * x.y;
            rounded += f * x.z;
            acc += *reinterpret_cast<const f32x4 *>(&part_o[w][row][d]) * f;
        }
        const int j = (s.row0 + row) / a.group;
        write_out<T>(a, tok.x + j, s.head * a.group + s.row0 + row - j * a.group, d, acc, top, sum, rounded);
    }
}

template <class T, int DP, int MP, int MS>
static int run_attn(const AttnArgs &a, hipStream_t st) {
    attn_split_kernel<T, DP, MP, MS><<<(unsigned)a.n_wgs, kAttnThreads, (size_t)(5 * (a.n_seqs + 1)) * 4, st>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
    const int rows = a.n_seqs * a.max_q * a.q_heads;
    if (rows < kJoinRows) {
        attn_join_kernel<T, DP><<<(unsigned)rows, kAttnThreads, 0, st>>>(a, MP, MS);
        return (int)hipGetLastError();
    }
    const int wgs = (rows + kAttnWaves - 1) / kAttnWaves;
    for (int first = 0; first < wgs && e == hipSuccess; first += kMaxWgs) {
        attn_join_rows_kernel<T, DP><<<(unsigned)min(wgs - first, kMaxWgs), kAttnThreads, 0, st>>>(a, MP, MS, first * kAttnWaves, rows);
        e = hipGetLastError();
    }
    return (int)e;
}

// Heads beyond 64 take tiles of 16 rows only from registers: with 32 the outputs spill, and reading the keys twice costs
// less (eight sequences of some 3000 positions, 32 rows to a key/value head: 24 us against 31 with heads of 128, 43
// against 79 with 256; with heads of 64, 40 rows: 26 against 23).
template <class T, int DP>
static int run_attn_tiles(const AttnArgs &a, int32_t mp, int32_t ms, hipStream_t st) {
    if (mp == 0) {  // short contexts
        const int tiles = (a.max_q * a.group + 15) / 16;
        attn_short_kernel<T, DP><<<(unsigned)(a.n_seqs * a.kv_heads * tiles), 64 * kShortWaves<DP>, 0, st>>>(a, tiles);
        return (int)hipGetLastError();
    }
    if (ms == 16) {
        if (mp == 16) return run_attn<T, DP, 16, 16>(a, st);
        if (mp == 64) return run_attn<T, DP, 64, 16>(a, st);
        if (mp == 128) return run_attn<T, DP, 128, 16>(a, st);
        if constexpr (DP == 64) return run_attn<T, DP, 32, 16>(a, st);
    } else if constexpr (DP == 64) {
        if (mp == 32) return run_attn<T, DP, 32, 32>(a, st);
        if (mp == 64) return run_attn<T, DP, 64, 32>(a, st);
        return run_attn<T, DP, 128, 32>(a, st);
    }
    return (int)hipErrorInvalidValue;
}

}  // namespace bpw
