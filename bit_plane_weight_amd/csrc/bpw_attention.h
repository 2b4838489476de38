// bpw_attention.h - attention of a decode step over a shared prefix and per-sequence suffixes in a paged
// cache (gfx950, wave64): the split kernel, instantiated per padded head size by bpw_attention_d*.hip.
//
// Mathematics. For a query row q and positions i: s_i = scale <q, K_i>; with a running maximum m and sum
// l = sum exp(s_i - m), o = sum exp(s_i - m) V_i, parts over disjoint positions join exactly:
// m = max m_p, l = sum exp(m_p - m) l_p, o = sum exp(m_p - m) o_p. So the positions of one
// (segment, key/value head, tile of query rows) are cut into units of kAttnUnit, units are dealt to the
// workgroups in equal contiguous runs, and a second launch joins the parts in order.
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
// No LDS is used until the four waves of a workgroup join their parts.
#pragma once

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

// The work of one workgroup on one item: units [u0, u1) of a page list for a tile of query rows.
struct AttnSpan {
    const int32_t *pages;
    int32_t len;       // positions of the segment
    int32_t tok0;      // first token of its rows
    int32_t n_tok;     // tokens of its rows
    int32_t causal;    // row of token j sees len - (n_tok - 1 - j) positions
    int32_t head;      // key/value head
    int32_t row0;      // first row of the tile
    int32_t n_rows;    // rows of all tiles
    int32_t u0, u1;
    float *po;         // results of the tile: [rows][DP]
    float2 *pml;       // [rows]
};

constexpr float kNone = -__builtin_inff();

// LDS of the join of four waves: 16 rows of outputs, and the maxima and sums of all rows.
template <int DP>
struct AttnLds {
    float o[kAttnWaves][16][DP + 4];
    float2 ml[kAttnWaves][64];
};

template <class T, int NQ, int DP>
__device__ __forceinline__ void attend(const AttnArgs &a, const AttnSpan &s, AttnLds<DP> &lds) {
    constexpr int KC = DP / 32;            // key chunks of 32 elements
    constexpr int EL = DP < 128 ? DP / 16 : 8;  // neighbouring elements of a value row in one lane
    constexpr int NH = DP / (16 * EL);     // such runs
    constexpr int VW = EL / 2;             // their words
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
    float m[NQ], l[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        m[i] = kNone;
        l[i] = 0.0f;
#pragma unroll
        for (int c = 0; c < NH * EL; ++c) o[i][c] = f32x4{0, 0, 0, 0};
    }

    // page of the 16 positions from `pos` on, or -1: past the end or not a page of the cache. Pages hold
    // a multiple of 16 positions, so such a tile never straddles two.
    auto page_of = [&](int pos) -> int {
        if (pos >= s.len) return -1;
        const int id = s.pages[pos >> a.page_log2];
        return (uint32_t)id < (uint32_t)a.n_pages ? id : -1;
    };
    auto load_keys = [&](int pos, int id, u32v4 (&k)[KC]) {
#pragma unroll
        for (int c = 0; c < KC; ++c) k[c] = u32v4{0, 0, 0, 0};
        if (id >= 0) {
            const T *p = kbase + (int64_t)id * a.k_ps + (int64_t)(pos & pmask) * a.k_rs;
#pragma unroll
            for (int c = 0; c < KC; ++c) k[c] = *reinterpret_cast<const u32v4 *>(p + koff[c]);
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
                        const u32v4 w = *reinterpret_cast<const u32v4 *>(e);
                        v[r][h][0] = w.x, v[r][h][1] = w.y, v[r][h][2] = w.z, v[r][h][3] = w.w;
                    } else {
                        const u32x2 w = *reinterpret_cast<const u32x2 *>(e);
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

    int kv0 = s.u0 * kAttnUnit + wave * kAttnStep;
    const int end = min(s.len, s.u1 * kAttnUnit);
    int id0 = -1, id1 = -1;
    u32v4 k0[KC], k1[KC];
    if (kv0 < end) {
        id0 = page_of(kv0);
        id1 = page_of(kv0 + 16);
        load_keys(kv0, id0, k0);
        load_keys(kv0 + 16, id1, k1);
    }
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
        kv0 += kAttnUnit;
        if (kv0 < end) {  // the next step's keys
            id0 = page_of(kv0);
            id1 = page_of(kv0 + 16);
            load_keys(kv0, id0, k0);
            load_keys(kv0 + 16, id1, k1);
        }
        if (here + kAttnStep > all_see || (c0 | c1) < 0) {
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
                    }
                }
        }
        u32v4 p[NQ];
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            float top = kNone;
#pragma unroll
            for (int r = 0; r < 4; ++r) top = fmaxf(top, fmaxf(sc[i][0][r], sc[i][1][r]));
            top *= a.scale_log2;
            // The maximum is a common shift of a row, not its exact maximum: it is raised only when a
            // score exceeds it by 2^8 (weights up to 256 lose nothing in float32, nor in the 16-bit types),
            // so most steps skip the exchange between lanes and the rescaling of o.
            if (__any(top > m[i] + 8.0f)) {
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                const float up = fmaxf(m[i], top);
                const float f = up == m[i] ? 1.0f : __builtin_amdgcn_exp2f(m[i] - up);
                m[i] = up;
                l[i] *= f;
#pragma unroll
                for (int c = 0; c < NH * EL; ++c) o[i][c] *= f;
            }
            const float shift = m[i] == kNone ? 0.0f : m[i];
            f32x8 w;
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                w[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i][r >> 2][r & 3], a.scale_log2, -shift));
                l[i] += w[r];
            }
            // weights in 16 bits: the matrix cores' operand. Its relative error of half a step is averaged
            // over the positions; the sum l is of the unrounded weights.
            p[i] = __builtin_bit_cast(u32v4, __builtin_convertvector(w, typename Vec8<T>::type));
        }
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int c = 0; c < EL; ++c) {
                u32v4 f;
                const uint32_t sel = c & 1 ? 0x07060302u : 0x05040100u;
#pragma unroll
                for (int w = 0; w < 4; ++w) f[w] = __builtin_amdgcn_perm(v[2 * w + 1][h][c >> 1], v[2 * w][h][c >> 1], sel);
#pragma unroll
                for (int i = 0; i < NQ; ++i) o[i][h * EL + c] = mma<T>(f, p[i], o[i][h * EL + c]);
            }
    }

    // join the four waves
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        l[i] += __shfl_xor(l[i], 16);
        l[i] += __shfl_xor(l[i], 32);
        if (g == 0) lds.ml[wave][16 * i + n] = make_float2(m[i], l[i]);
    }
    __syncthreads();
    const int row = threadIdx.x >> 4, part = threadIdx.x & 15;  // 16 threads to a row
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        float top = kNone, sum = 0.0f;
        float2 w[kAttnWaves];
#pragma unroll
        for (int x = 0; x < kAttnWaves; ++x) {
            w[x] = lds.ml[x][16 * i + n];
            top = fmaxf(top, w[x].x);
        }
#pragma unroll
        for (int x = 0; x < kAttnWaves; ++x)
            if (w[x].x != kNone) sum += w[x].y * __builtin_amdgcn_exp2f(w[x].x - top);
        const float f = m[i] == kNone ? 0.0f : __builtin_amdgcn_exp2f(m[i] - top);
        if (threadIdx.x < 16 && s.row0 + 16 * i + n < s.n_rows) s.pml[16 * i + n] = make_float2(top, sum);
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < EL; c += 4) {
                    f32x4 x;
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = o[i][h * EL + c + e][r] * f;
                    *reinterpret_cast<f32x4 *>(&lds.o[wave][n][16 * EL * h + EL * (4 * g + r) + c]) = x;
                }
        __syncthreads();
        if (s.row0 + 16 * i + row < s.n_rows) {
#pragma unroll
            for (int d = 4 * part; d < DP; d += 64) {
                f32x4 x = *reinterpret_cast<const f32x4 *>(&lds.o[0][row][d]);
#pragma unroll
                for (int y = 1; y < kAttnWaves; ++y) x += *reinterpret_cast<const f32x4 *>(&lds.o[y][row][d]);
                *reinterpret_cast<f32x4 *>(s.po + (int64_t)(16 * i + row) * DP + d) = x;
            }
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------------------------------------
// Many query rows (the prefix of a batch). Here the matrix cores and the exponentials are the bound, not
// the memory: 64 or 128 rows share each key, so keys and values go once through LDS for the four waves,
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

constexpr int kWideTile = 64;

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

// 16 bytes a lane from memory to LDS at `dst` (the same in all lanes) + 16 * lane. Waited for by vmcnt.
// Written as one asm block (m0, which holds the LDS address, is put back) because the compiler makes every later
// LDS read wait for loads to LDS that it knows of, whatever part of LDS they write; the block writes no register.
__device__ __forceinline__ void load_to_lds(void *dst, const void *src) {
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(size_t)(lds_u8 *)dst);
    uint32_t keep;
    asm volatile(
        "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, off\n\ts_mov_b32 m0, %0"
        : "=&s"(keep)
        : "s"(at), "v"(src)
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

    auto page_of = [&](int pos) -> int {
        if (pos >= s.len) return -1;
        const int id = s.pages[pos >> a.page_log2];
        return (uint32_t)id < (uint32_t)a.n_pages ? id : -1;
    };
    // This wave's 16 positions of the tile at `pos0`; hidden positions and elements past head_dim are zeros
    // (a zero weight times whatever memory holds there would not be).
    auto issue = [&](int buf, int pos0, int id) {
        const int first = pos0 + 16 * wave;
        const T *kp = kbase + (int64_t)id * a.k_ps + (int64_t)(first & pmask) * a.k_rs;
        const T *vp = vbase + (int64_t)id * a.v_ps + (int64_t)(first & pmask) * a.v_rs;
        if (id >= 0 && first + 16 <= s.len && D == DP) {
#pragma unroll
            for (int i = 0; i < 16 / RPI; ++i) {
                const int r = RPI * i + lane / CPR;
                const int ck = (lane % CPR) ^ key_of_k<DP>(r), cv = (lane % CPR) ^ key_of_v<DP>(r);
                load_to_lds(&lds.k[buf][(16 * wave + RPI * i) * ROW], kp + r * a.k_rs + 8 * ck);
                load_to_lds(&lds.v[buf][(16 * wave + RPI * i) * ROW], vp + r * a.v_rs + 8 * cv);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < 16 / RPI; ++i) {
            const int r = RPI * i + lane / CPR;  // of the wave's sixteen
            const bool in = id >= 0 && first + r < s.len;
            const int ck = (lane % CPR) ^ key_of_k<DP>(r), cv = (lane % CPR) ^ key_of_v<DP>(r);
            uint8_t *dk = &lds.k[buf][(16 * wave + RPI * i) * ROW], *dv = &lds.v[buf][(16 * wave + RPI * i) * ROW];
            if (in && 8 * ck < D)
                load_to_lds(dk, kp + r * a.k_rs + 8 * ck);
            else
                *reinterpret_cast<u32v4 *>(dk + 16 * lane) = u32v4{0, 0, 0, 0};
            if (in && 8 * cv < D)
                load_to_lds(dv, vp + r * a.v_rs + 8 * cv);
            else
                *reinterpret_cast<u32v4 *>(dv + 16 * lane) = u32v4{0, 0, 0, 0};
        }
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
    float m = kNone, l = 0.0f;

    int pos0 = s.u0 * kAttnUnit, buf = 0;
    const int end = min(s.len, s.u1 * kAttnUnit);
    int id[kAttnWaves];
#pragma unroll
    for (int x = 0; x < kAttnWaves; ++x) id[x] = page_of(pos0 + 16 * x);
    issue(0, pos0, wave == 0 ? id[0] : wave == 1 ? id[1] : wave == 2 ? id[2] : id[3]);
    while (pos0 < end) {
        const bool hidden = (id[0] | id[1] | id[2] | id[3]) < 0 || pos0 + kWideTile > s.len;
        uint32_t pages = 0;  // bit x: positions 16 x .. 16 x + 15 of this tile are a page's
#pragma unroll
        for (int x = 0; x < kAttnWaves; ++x) {
            pages |= id[x] >= 0 ? 1u << x : 0u;
            id[x] = page_of(pos0 + kWideTile + 16 * x);
        }
        wait_loads_to_lds();
        __syncthreads();  // this tile is there, and nobody reads the one before it any more
        if (pos0 + kWideTile < end)
            issue(buf ^ 1, pos0 + kWideTile, wave == 0 ? id[0] : wave == 1 ? id[1] : wave == 2 ? id[2] : id[3]);

        // Operands are read from LDS a group of products ahead: the reads of group x + 1 run under the products
        // of group x (the scheduling barriers keep the compiler from sinking each read to its use).
        f32x16 sc[NB];
        {
            constexpr int GK = 4, NG = NB * KC / GK;
            u32v4 kf[2][GK];
            auto read_k = [&](int x, u32v4 (&f)[GK]) {
                const uint8_t *p = &lds.k[buf][(part * NB + x * GK / KC) * 32 * ROW];
#pragma unroll
                for (int c = 0; c < GK; ++c) f[c] = *reinterpret_cast<const u32v4 *>(p + ka[(x * GK + c) % KC]);
            };
            read_k(0, kf[0]);
#pragma unroll
            for (int x = 0; x < NG; ++x) {
                if (x + 1 < NG) read_k(x + 1, kf[(x + 1) & 1]);
                __builtin_amdgcn_sched_barrier(0);
                const int b = x * GK / KC;
                if (x * GK % KC == 0) sc[b] = f32x16{};
#pragma unroll
                for (int c = 0; c < GK; ++c) sc[b] = mma32<T>(kf[x & 1][c], q[(x * GK + c) % KC], sc[b]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        u32v4 vf[2][DB];
        auto read_v = [&](int x, u32v4 (&f)[DB]) {  // positions 16 x .. 16 x + 15 of this wave's blocks
            const uint8_t *vp = &lds.v[buf][(32 * part * NB + 16 * x) * ROW];
#pragma unroll
            for (int c = 0; c < DB; ++c) {
                const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(lds_u8 *)(vp + va[c][0])));
                const u32x2 z = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(lds_u8 *)(vp + va[c][1])));
                f[c] = u32v4{y.x, y.y, z.x, z.y};
            }
        };
        read_v(0, vf[0]);
        __builtin_amdgcn_sched_barrier(0);
        if (hidden) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int at = 32 * (part * NB + b) + 8 * (r >> 2) + 4 * g + (r & 3);
                    if (pos0 + at >= s.len || !((pages >> (at >> 4)) & 1)) sc[b][r] = kNone;
                }
        }
        float top = kNone;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int r = 0; r < 16; r += 2) top = fmaxf(top, fmaxf(sc[b][r], sc[b][r + 1]));
        top *= a.scale_log2;
        if (__any(top > m + 8.0f)) {  // as above: the shift is raised only by more than 2^8
            top = fmaxf(top, __shfl_xor(top, 32));
            const float up = fmaxf(m, top);
            const float f = up == m ? 1.0f : __builtin_amdgcn_exp2f(m - up);
            m = up;
            l *= f;
#pragma unroll
            for (int c = 0; c < DB; ++c) o[c] *= f;
        }
        const float shift = m == kNone ? 0.0f : m;
        u32v4 p[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f32x8 w;
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    w[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[b][8 * h + r], a.scale_log2, -shift));
                    l += w[r];
                }
                p[b][h] = __builtin_bit_cast(u32v4, __builtin_convertvector(w, typename Vec8<T>::type));
            }
#pragma unroll
        for (int x = 0; x < 2 * NB; ++x) {
            if (x + 1 < 2 * NB) read_v(x + 1, vf[(x + 1) & 1]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int c = 0; c < DB; ++c) o[c] = mma32<T>(vf[x & 1][c], p[x >> 1][x & 1], o[c]);
            __builtin_amdgcn_sched_barrier(0);
        }
        pos0 += kWideTile;
        buf ^= 1;
    }

    l += __shfl_xor(l, 32);
    if constexpr (PARTS == 2) {  // the second wave of the same rows hands over through LDS
        constexpr int PAD = DP + 4;
        float *box = reinterpret_cast<float *>(&lds) + (wave % WQ) * (32 * PAD);
        float2 *ml = reinterpret_cast<float2 *>(reinterpret_cast<float *>(&lds) + WQ * 32 * PAD) + 32 * (wave % WQ);
        static_assert((WQ * 32 * PAD + 2 * 32 * WQ) * 4 <= sizeof(WideLds<DP>), "the join fits the tiles' LDS");
        __syncthreads();
        if (part == 1) {
#pragma unroll
            for (int c = 0; c < DB; ++c)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    *reinterpret_cast<f32x4 *>(box + n * PAD + 32 * c + 8 * r + 4 * g) =
                        f32x4{o[c][4 * r], o[c][4 * r + 1], o[c][4 * r + 2], o[c][4 * r + 3]};
            if (g == 0) ml[n] = make_float2(m, l);
        }
        __syncthreads();
        if (part == 0) {
            const float2 x = ml[n];
            const float up = fmaxf(m, x.x);
            const float f0 = m == kNone ? 0.0f : __builtin_amdgcn_exp2f(m - up), f1 = x.x == kNone ? 0.0f : __builtin_amdgcn_exp2f(x.x - up);
            m = up;
            l = l * f0 + x.y * f1;
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
        if (g == 0) s.pml[at] = make_float2(m, l);
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

// MP, MS: query rows of a tile in the prefix (16, 32: from registers; 64, 128: through LDS) and in a
// suffix (16, 32).
template <class T, int DP, int MP, int MS>
__global__ __launch_bounds__(kAttnThreads, DP <= 128 ? 2 : 1) void attn_split_kernel(AttnArgs a) {
    constexpr bool WIDE = MP > 32;
    constexpr size_t LDS = WIDE && sizeof(WideLds<DP>) > sizeof(AttnLds<DP>) ? sizeof(WideLds<DP>) : sizeof(AttnLds<DP>);
    __shared__ alignas(16) uint8_t lds[LDS];
    __shared__ int32_t units[kAttnMaxSeqs + 1], items[kAttnMaxSeqs + 1];
    __shared__ int32_t wave_sum[kAttnWaves][2];
    __shared__ int32_t first_seq;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;

    // Units and items (head x tile) before each sequence: four sequences a thread, then a scan.
    int un[4], it[4], su = 0, si = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int b = 4 * tid + x;
        un[x] = it[x] = 0;
        if (b < a.n_seqs) {
            const int n = seq_tokens(a, b).y;
            const int u = (seq_len(a, b) + kAttnUnit - 1) / kAttnUnit;
            it[x] = u > 0 ? a.kv_heads * ((n * a.group + MS - 1) / MS) : 0;
            un[x] = it[x] * u;
        }
        su += un[x];
        si += it[x];
    }
    int iu = su, ii = si;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int x = __shfl_up(iu, d), y = __shfl_up(ii, d);
        if (lane >= d) iu += x, ii += y;
    }
    if (lane == 63) wave_sum[wave][0] = iu, wave_sum[wave][1] = ii;
    if (tid == 0) first_seq = 0;
    __syncthreads();
    int total_s = 0;
#pragma unroll
    for (int x = 0; x < kAttnWaves; ++x) {
        if (x < wave) iu += wave_sum[x][0], ii += wave_sum[x][1];
        total_s += wave_sum[x][0];
    }
    int eu = iu - su, ei = ii - si;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int b = 4 * tid + x;
        if (b < a.n_seqs) units[b] = eu, items[b] = ei;
        eu += un[x], ei += it[x];
        if (b == a.n_seqs - 1) units[a.n_seqs] = eu, items[a.n_seqs] = ei;
    }
    // Equal shares by the cost of a unit.
    constexpr int COST_P = MP <= 32 ? 2 : MP == 64 ? 3 : 4, COST_S = 2;
    const int up = (a.prefix_len + kAttnUnit - 1) / kAttnUnit, total_p = a.kv_heads * a.tiles_p * up;
    int qp = 1, qs = 1, wp = total_p, ws = total_s;
    if (wp + ws > a.n_wgs) {
        int share = (int)(((int64_t)total_p * COST_P + (int64_t)total_s * COST_S + a.n_wgs - 1) / a.n_wgs);
        do {
            qp = max(1, share / COST_P);
            qs = max(1, share / COST_S);
            wp = (total_p + qp - 1) / qp;
            ws = (total_s + qs - 1) / qs;
            share += 1 + share / 16;
        } while (wp + ws > a.n_wgs);
    }
    __syncthreads();
    if (blockIdx.x == 0) {  // what the join needs
        if (tid == 0) a.sched[0] = up, a.sched[1] = qp, a.sched[2] = qs;
        for (int b = tid; b <= a.n_seqs; b += kAttnThreads) {
            a.sched[kSchedHead + b] = units[b];
            a.sched[kSchedHead + a.n_seqs + 1 + b] = items[b];
        }
    }
    // Workgroup b runs on XCD b % 8: neighbours in the dealing, which read the same keys for other rows,
    // share one XCD's L2.
    int w = blockIdx.x;
    const int per = gridDim.x >> 3;
    if (w < 8 * per) w = (w & 7) * per + (w >> 3);
    AttnSpan s;
    if (w < wp) {
        int u = w * qp;
        const int stop = min(total_p, u + qp);
        while (u < stop) {
            const int item = u / up, at = u - item * up;
            s.pages = a.prefix_pages;
            s.len = a.prefix_len;
            s.tok0 = 0;
            s.n_tok = a.n_tokens;
            s.causal = 0;
            s.head = item / a.tiles_p;
            s.row0 = (item - s.head * a.tiles_p) * MP;
            s.n_rows = a.n_tokens * a.group;
            s.u0 = at;
            s.u1 = min(up, at + stop - u);
            s.po = a.part_o + (int64_t)(item + w) * (MP * DP);
            s.pml = a.part_ml + (int64_t)(item + w) * MP;
            if constexpr (WIDE)
                attend_wide<T, DP, MP / 32>(a, s, reinterpret_cast<WideLds<DP> &>(lds));
            else
                attend<T, MP / 16, DP>(a, s, reinterpret_cast<AttnLds<DP> &>(lds));
            u += s.u1 - s.u0;
        }
        return;
    }
    w -= wp;
    if (w >= ws) return;
    int u = w * qs;
    const int stop = min(total_s, u + qs);
#pragma unroll
    for (int x = 0; x < 4; ++x) {  // the sequence that holds unit u
        const int b = 4 * tid + x;
        if (b < a.n_seqs && units[b] <= u && u < units[b + 1]) first_seq = b;
    }
    __syncthreads();
    int b = __builtin_amdgcn_readfirstlane(first_seq);
    while (u < stop) {
        while (units[b + 1] <= u) ++b;  // past idle sequences
        b = __builtin_amdgcn_readfirstlane(b);
        const int2 tok = seq_tokens(a, b);
        const int len = seq_len(a, b), ub = (len + kAttnUnit - 1) / kAttnUnit;
        const int tiles = (tok.y * a.group + MS - 1) / MS;
        const int rest = u - __builtin_amdgcn_readfirstlane(units[b]);
        const int item = rest / ub, at = rest - item * ub;
        const int64_t piece = __builtin_amdgcn_readfirstlane(items[b]) + item + w;
        s.pages = a.table + (int64_t)b * a.table_stride;
        s.len = len;
        s.tok0 = tok.x;
        s.n_tok = tok.y;
        s.causal = 1;
        s.head = item / tiles;
        s.row0 = (item - s.head * tiles) * MS;
        s.n_rows = tok.y * a.group;
        s.u0 = at;
        s.u1 = min(ub, at + stop - u);
        s.po = a.part_o + a.part_s + piece * (MS * DP);
        s.pml = a.part_ml + a.ml_s + piece * MS;
        attend<T, MS / 16, DP>(a, s, reinterpret_cast<AttnLds<DP> &>(lds));
        u += s.u1 - s.u0;
    }
}

// Joins the parts of one query row: one workgroup to a (sequence, query token, query head). The weights of the
// parts are formed once in LDS; then DP / 4 threads hold a row, so that several parts are in flight.
template <class T, int DP>
__global__ __launch_bounds__(kAttnThreads) void attn_join_kernel(AttnArgs a, int mp, int ms) {
    constexpr int LANES = DP / 4, GROUPS = kAttnThreads / LANES;
    __shared__ float weight[2 * kAttnMaxWgs + 2];
    __shared__ f32x4 sums[GROUPS][LANES];
    __shared__ float red[kAttnWaves];
    const int tid = threadIdx.x;
    const int hq = blockIdx.x % a.q_heads, bj = blockIdx.x / a.q_heads, j = bj % a.max_q, b = bj / a.max_q;
    const int2 tok = seq_tokens(a, b);
    if (j >= tok.y) return;
    const int t = tok.x + j, head = hq / a.group, gi = hq - head * a.group;
    const int up = a.sched[0], qp = a.sched[1], qs = a.sched[2];
    int np = 0, ns = 0;
    int64_t first_p = 0, first_s = 0;  // pieces
    int row_p = 0, row_s = 0;
    if (up > 0) {
        const int row = t * a.group + gi, tile = row / mp, item = head * a.tiles_p + tile;
        const int w0 = item * up / qp, w1 = (item * up + up - 1) / qp;
        np = w1 - w0 + 1;
        first_p = item + w0;
        row_p = row - tile * mp;
    }
    const int ub = (seq_len(a, b) + kAttnUnit - 1) / kAttnUnit;
    if (ub > 0) {
        const int tiles = (tok.y * a.group + ms - 1) / ms;
        const int row = j * a.group + gi, tile = row / ms, item = head * tiles + tile;
        const int u0 = a.sched[kSchedHead + b] + item * ub;
        const int w0 = u0 / qs, w1 = (u0 + ub - 1) / qs;
        ns = w1 - w0 + 1;
        first_s = a.sched[kSchedHead + a.n_seqs + 1 + b] + item + w0;
        row_s = row - tile * ms;
    }
    auto ml_of = [&](int k) -> float2 {
        return k < np ? a.part_ml[(first_p + k) * mp + row_p] : a.part_ml[a.ml_s + (first_s + k - np) * ms + row_s];
    };
    const int parts = np + ns;
    float top = kNone;
    for (int k = tid; k < parts; k += kAttnThreads) top = fmaxf(top, ml_of(k).x);
#pragma unroll
    for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    if ((tid & 63) == 0) red[tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    __syncthreads();
    float sum = 0.0f;
    for (int k = tid; k < parts; k += kAttnThreads) {
        const float2 x = ml_of(k);
        const float f = x.x == kNone ? 0.0f : __builtin_amdgcn_exp2f(x.x - top);
        weight[k] = f;
        sum += x.x == kNone ? 0.0f : f * x.y;
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    if ((tid & 63) == 0) red[tid >> 6] = sum;
    __syncthreads();
    sum = (red[0] + red[1]) + (red[2] + red[3]);
    const int gr = tid / LANES, ln = tid - gr * LANES;
    f32x4 acc = {0, 0, 0, 0};
#pragma unroll 4
    for (int k = gr; k < parts; k += GROUPS) {
        const float *p = k < np ? a.part_o + ((first_p + k) * mp + row_p) * DP
                                : a.part_o + a.part_s + ((first_s + k - np) * ms + row_s) * DP;
        const float f = weight[k];
        const f32x4 x = *reinterpret_cast<const f32x4 *>(p + 4 * ln);
        acc += x * f;
    }
    sums[gr][ln] = acc;
    __syncthreads();
    if (gr == 0 && 4 * ln < a.head_dim) {
#pragma unroll
        for (int y = 1; y < GROUPS; ++y) acc += sums[y][ln];
        // nothing seen: zeros. (A NaN sum is not equal to zero and goes through.)
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        T *out = static_cast<T *>(a.out) + (int64_t)t * a.o_ts + (int64_t)hq * a.o_hs + 4 * ln;
        typedef T T4 __attribute__((ext_vector_type(4)));
        *reinterpret_cast<T4 *>(out) = __builtin_convertvector(acc * inv, T4);
    }
    if (tid == 0 && a.lse)
        a.lse[(int64_t)t * a.q_heads + hq] =
            sum == 0.0f ? kNone : (top + __builtin_amdgcn_logf(sum)) * 0.69314718055994531f;
}

template <class T, int DP, int MP, int MS>
static int run_attn(const AttnArgs &a, hipStream_t st) {
    attn_split_kernel<T, DP, MP, MS><<<(unsigned)a.n_wgs, kAttnThreads, 0, st>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
    attn_join_kernel<T, DP><<<(unsigned)((int64_t)a.n_seqs * a.max_q * a.q_heads), kAttnThreads, 0, st>>>(a, MP, MS);
    return (int)hipGetLastError();
}

template <class T, int DP>
static int run_attn_tiles(const AttnArgs &a, int32_t mp, int32_t ms, hipStream_t st) {
    if (ms == 16) {
        if (mp == 16) return run_attn<T, DP, 16, 16>(a, st);
        if (mp == 32) return run_attn<T, DP, 32, 16>(a, st);
        if (mp == 64) return run_attn<T, DP, 64, 16>(a, st);
        return run_attn<T, DP, 128, 16>(a, st);
    }
    if (mp == 32) return run_attn<T, DP, 32, 32>(a, st);
    if (mp == 64) return run_attn<T, DP, 64, 32>(a, st);
    return run_attn<T, DP, 128, 32>(a, st);
}

}  // namespace bpw
