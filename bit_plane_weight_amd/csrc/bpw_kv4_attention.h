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
// DP / 4 neighbours (at heads of 128 one block, one power), and the query's elements are laid out alike. A value row is
// read by 16 lanes, 8 neighbours each (4 bytes), and turned by v_perm after the conversion.
//
// Codes and powers go through LDS, moved there by the loads themselves some steps of 32 positions ahead, in an order that makes a
// lane's operands neighbours (Ring4): with loads to registers a step of heads of 128 took 20 loads of 1 to 16 bytes a lane
// and waited for all of them (8 sequences of 57000 positions, 8 heads: 125 us; this way 5 loads, 90-93 us). Bound there: the
// vector units issue half of the time (64 conversions, 32 v_perm, 24 for the weights' two parts of 215 in a step)
// beside loads that alone take 84 us.
#pragma once

#include <type_traits>

#include "bpw_attention.h"

namespace bpw {

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

// What a wave keeps on its way from the cache, in LDS: steps of 32 positions, of each the codes of keys and values and their
// powers. A load moves 64 chunks of 16 bytes (a block of 32 elements). DENSE: heads of DP elements whose rows of powers lie one
// after another, those of 16 positions whole words; otherwise a load moves 64 of them, a byte to a word (a step of heads of
// 128 takes five loads or eight).
template <int DP, bool DENSE>
struct Ring4 {
    static constexpr int BLOCKS = DP / kKv4Block;       // of a row
    static constexpr int LOADS = 32 * BLOCKS / 64;      // of a step's codes of keys (or values)
    static constexpr int VALUES = 1024 * LOADS, POWERS = 2 * VALUES;
    static constexpr int POWER_LOADS = DENSE ? (DP == 256 ? 2 : 1) : 2 * LOADS;
    static constexpr int ALL = 2 * LOADS + POWER_LOADS, STEP = POWERS + 256 * POWER_LOADS;
    // Steps: 70 to 140 KB of a CU's LDS for two workgroups of four waves.
    static constexpr int STEPS = DP == 64 ? 4 : DP == 128 ? 3 : 2;
    static constexpr int BYTES = STEPS * STEP;
};

// A load of BYTES a lane from p + AT to LDS at m0 + AT (+ 16 or 4 a lane). Waited for by vmcnt; asm for the reason given at load_to_lds(). Its
// address is in vector registers: a scalar one that a vector instruction wrote (v_readlane) needs five wait states before a
// load reads it, which the compiler does not see to for asm.
template <int AT, int BYTES>
__device__ __forceinline__ void ring_load(const uint8_t *p) {
    static_assert(AT < 4096, "an instruction's offset has 12 bits");
    if constexpr (BYTES == 16)
        asm volatile("global_load_lds_dwordx4 %0, off offset:%1 nt" ::"v"(p), "n"(AT) : "memory");
    else if constexpr (BYTES == 4)
        asm volatile("global_load_lds_dword %0, off offset:%1" ::"v"(p), "n"(AT) : "memory");
    else
        asm volatile("global_load_lds_ubyte %0, off offset:%1" ::"v"(p), "n"(AT) : "memory");
}
// m0 for the loads that follow; what was read from LDS before is there.
__device__ __forceinline__ void ring_base(uint32_t at) {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_mov_b32 m0, %0\n\ts_nop 0" ::"s"(at) : "m0", "memory");
}
template <int N>
__device__ __forceinline__ void wait_all_but() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

typedef __attribute__((address_space(3))) const u32v4 lds_u32v4;
typedef __attribute__((address_space(3))) const u32x2 lds_u32x2;
typedef __attribute__((address_space(3))) const uint32_t lds_u32;
typedef __attribute__((address_space(3))) const uint16_t lds_u16;
typedef __attribute__((address_space(3))) const uint8_t lds_cu8;

// The pages of a list, 64 at a time, one a lane. A fetch is waited for at once: waits in the loop would be for all loads to LDS.
struct Pages4 {
    int32_t ids, base;
    __device__ __forceinline__ void fetch(const AttnArgs &a, const AttnSpan &s, int page) {
        base = page;
        const int at = page + (int)(threadIdx.x & 63);
        ids = -1;
        if ((int64_t)at << a.page_log2 < s.len) ids = s.pages[at];
        asm volatile("" : "+v"(ids));
    }
    // Page `page` of the list (the last one asked for, or the next), or -1: past the end, or not a page of the cache. The same in all lanes.
    __device__ __forceinline__ int32_t of(const AttnArgs &a, const AttnSpan &s, int page) {
        if (page >= base + 64) fetch(a, s, page);
        const int32_t id = __builtin_amdgcn_readlane(ids, page - base);
        return (uint32_t)id < (uint32_t)a.n_pages ? id : -1;
    }
};

// One tile of 16 query rows over positions [pos0, pos1) of a page list (s), 32 positions at a time; ring: LDS address of this
// wave's Ring4.
template <class T, int DP, bool DENSE>
__device__ __forceinline__ void attend4(const Attn4Args &b, const AttnSpan &s, uint32_t ring) {
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

    // Loads: lane x of load j takes chunk 64 j + x of a step. Keys go to LDS by (tile of 16 positions, block, position), values by
    // (tile, position % 4, position / 4, block) and their powers by (tile, position / 4, block, position % 4), so that a
    // lane's operands are neighbours there and the banks are shared evenly. Blocks past head_dim are the first one again.
    using Ring = Ring4<DP, DENSE>;
    constexpr int BLOCKS = Ring::BLOCKS, LOADS = Ring::LOADS, STEPS = Ring::STEPS, ALL = Ring::ALL;
    // Load j of a step: where its part of the step begins in LDS, from the base that m0 has for it; its address in this lane for
    // page 0 and the page's first rows. Lanes of one load may be of two tiles, and, with DENSE, of keys and values.
    constexpr auto lds_at = [](int j) { return j < 2 * LOADS ? 1024 * (j % 4) : (Ring::POWERS > 2048 ? 0 : Ring::POWERS) + 256 * (j - 2 * LOADS); };
    constexpr auto tile_of = [](int j, int lane) {
        const int i = j < 2 * LOADS ? j : j - 2 * LOADS;
        if (DENSE && j >= 2 * LOADS) return (lane & (DP == 256 ? 32 : 16)) != 0;
        return LOADS == 1 ? lane >= 32 : LOADS == 2 ? (i & 1) != 0 : (i & 2) != 0;
    };
    constexpr auto values_of = [](int j, int lane) {
        if (DENSE && j >= 2 * LOADS) return DP == 256 ? j > 2 * LOADS : (lane & 32) != 0;
        return (j / LOADS & 1) != 0;
    };
    const bool own_pages = pmask == 15;  // tiles of 16 positions have pages of their own; otherwise a step is on one page
    const uint8_t *lane_base[ALL];
#pragma unroll
    for (int j = 0; j < ALL; ++j) {
        int32_t off;
        const bool codes = j < 2 * LOADS;
        const int i = codes ? j : j - 2 * LOADS, x = (LOADS == 4 ? 64 * (i & 1) : 0) + lane, used = D / kKv4Block;
        const bool values = values_of(j, lane);
        if (DENSE && !codes) {
            off = 4 * (lane & (DP == 256 ? 31 : 15));  // (DP 64: a tile has eight words, and the rest is not read)
            if (DP == 64) off &= 31;
        } else if (i < LOADS) {
            const int block = (x >> 4) % BLOCKS < used ? (x >> 4) % BLOCKS : 0;
            off = codes ? (x & 15) * b.kc.rs + 16 * block : (x & 15) * b.kc.s_rs + block;
        } else if (codes) {
            const int block = x % BLOCKS < used ? x % BLOCKS : 0, r = (x / BLOCKS) & 15;
            off = (4 * (r & 3) + (r >> 2)) * b.vc.rs + 16 * block;
        } else {
            const int block = (x >> 2) % BLOCKS < used ? (x >> 2) % BLOCKS : 0;
            off = (4 * (x / (4 * BLOCKS) & 3) + (x & 3)) * b.vc.s_rs + block;
        }
        const uint8_t *base = codes ? (values ? b.vc.codes : b.kc.codes) : values ? b.vc.scales : b.kc.scales;
        const int64_t hs = codes ? (values ? b.vc.hs : b.kc.hs) : values ? b.vc.s_hs : b.kc.s_hs;
        const int32_t rs = codes ? (values ? b.vc.rs : b.kc.rs) : values ? b.vc.s_rs : b.kc.s_rs;
        lane_base[j] = base + (s.head * hs + off + (tile_of(j, lane) && !own_pages ? 16 * rs : 0) - lds_at(j));
    }
    // this lane's reads
    const uint32_t kr = ring + (DP == 64 ? 256 * (g >> 1) + 16 * n + 8 * (g & 1) : (DP == 128 ? 256 : 512) * g + 16 * n);
    const uint32_t vr = ring + Ring::VALUES + DP / 2 * g + EL / 2 * n;
    const int kblock = DP == 64 ? g >> 1 : DP == 128 ? g : 2 * g, vblock = (EL * n) / kKv4Block;  // the first ones of this lane
    const uint32_t ksr = ring + Ring::POWERS + (DENSE ? n * BLOCKS + kblock : 64 * kblock + 4 * n);
    const uint32_t vsr = ring + Ring::POWERS + (DENSE ? (DP == 256 ? 256 : 128) + 4 * g * BLOCKS + vblock : 256 * LOADS + 16 * (BLOCKS * g + vblock));
    const bool key_in[2] = {DP / 4 * g < D, DP / 4 * g + 32 < D};  // (the second: heads of 256)

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
    // Loads that are issued next: addresses of this lane, the ids they come from.
    struct Issued {
        Pages4 pages;
        const uint8_t *p[ALL];
        int64_t k32, v32, ks32, vs32;  // bytes of 32 rows
        uint32_t bad, none;  // tiles that no page holds: two bits a step on its way; the last ones
    };
    const auto place = [&](Issued &x, int pos, int id0, int id1) __attribute__((always_inline)) {
        x.none = (id0 < 0 ? 1 : 0) | (id1 < 0 ? 2 : 0);
        const int64_t page = max(id0, 0), row = pos & pmask;  // (a tile without a page takes page 0's)
        const int64_t k = page * b.kc.ps + row * b.kc.rs, v = page * b.vc.ps + row * b.vc.rs;
        const int64_t ks = page * b.kc.s_ps + row * b.kc.s_rs, vs = page * b.vc.s_ps + row * b.vc.s_rs;
#pragma unroll
        for (int j = 0; j < ALL; ++j) x.p[j] = lane_base[j] + (j < 2 * LOADS ? (values_of(j, lane) ? v : k) : values_of(j, lane) ? vs : ks);
        if (own_pages) {
            const int64_t more = max(id1, 0) - page;
#pragma unroll
            for (int j = 0; j < ALL; ++j) {
                const int64_t ps = j < 2 * LOADS ? (values_of(j, lane) ? b.vc.ps : b.kc.ps) : values_of(j, lane) ? b.vc.s_ps : b.kc.s_ps;
                x.p[j] += tile_of(j, lane) ? more * ps : 0;
            }
        }
    };
    // Starts the loads of the step at `pos`; steps come in order.
    const auto issue = [&](Issued &x, int pos, uint32_t at) __attribute__((always_inline)) {
        if (own_pages) {
            const int id = x.pages.of(a, s, pos >> 4);
            place(x, pos, id, x.pages.of(a, s, (pos >> 4) + 1));
        } else if (pos == s.pos0 || (pos & pmask) == 0) {
            const int id = x.pages.of(a, s, pos >> a.page_log2);
            place(x, pos, id, id);
        } else {  // on the last step's page
#pragma unroll
            for (int j = 0; j < ALL; ++j) x.p[j] += j < LOADS ? x.k32 : j < 2 * LOADS ? x.v32 : DENSE ? 32 * BLOCKS : j < 3 * LOADS ? x.ks32 : x.vs32;
        }
        x.bad = x.bad << 2 | x.none;
#pragma unroll
        for (int j = 0; j < 2 * LOADS; j += 4) {
            ring_base(at + 1024 * j);
            ring_load<1024 * 0, 16>(x.p[j]);
            ring_load<1024 * 1, 16>(x.p[j + 1]);
            if constexpr (LOADS > 1) {
                ring_load<1024 * 2, 16>(x.p[j + 2]);
                ring_load<1024 * 3, 16>(x.p[j + 3]);
            }
        }
        if constexpr (Ring::POWERS > 2048) ring_base(at + Ring::POWERS);
        constexpr int AT = lds_at(2 * LOADS), P = 2 * LOADS, BYTES = DENSE ? 4 : 1;
        ring_load<AT, BYTES>(x.p[P]);
        if constexpr (Ring::POWER_LOADS > 1) ring_load<AT + 256, BYTES>(x.p[P + 1]);
        if constexpr (Ring::POWER_LOADS > 2) ring_load<AT + 512, BYTES>(x.p[P + 2]), ring_load<AT + 768, BYTES>(x.p[P + 3]);
        if constexpr (Ring::POWER_LOADS > 4) {
            ring_load<AT + 1024, BYTES>(x.p[P + 4]), ring_load<AT + 1280, BYTES>(x.p[P + 5]);
            ring_load<AT + 1536, BYTES>(x.p[P + 6]), ring_load<AT + 1792, BYTES>(x.p[P + 7]);
        }
    };
    // A step's reads; opaque to the compiler, so that the distances between them are the instructions' offsets.
    struct Reads {
        uint32_t kr, ksr, vr, vsr;
    };
    const auto reads_of = [&](uint32_t at) __attribute__((always_inline)) {
        Reads r = {kr + at, ksr + at, vr + at, vsr + at};
        asm volatile("" : "+v"(r.kr), "+v"(r.ksr), "+v"(r.vr), "+v"(r.vsr));
        return r;
    };
    const auto read_keys = [&](const Reads &r0, int t, Keys &k) __attribute__((always_inline)) {
        if constexpr (DP == 64) {
            const u32x2 x = *(lds_u32x2 *)(r0.kr + 512 * t);
            k.w[0] = x.x, k.w[1] = x.y;
        } else {
#pragma unroll
            for (int i = 0; i < KW / 4; ++i) {
                const u32v4 x = *(lds_u32v4 *)(r0.kr + 8 * DP * t + 256 * i);
                k.w[4 * i] = x.x, k.w[4 * i + 1] = x.y, k.w[4 * i + 2] = x.z, k.w[4 * i + 3] = x.w;
            }
        }
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            uint32_t u;
            if constexpr (DENSE)
                u = *(lds_cu8 *)(r0.ksr + (DP == 256 ? 128 : 64) * t + i);
            else
                u = *(lds_u32 *)(r0.ksr + 64 * BLOCKS * t + 64 * i);
            k.unit[i] = DENSE || key_in[i] ? u : 127;  // (a power of 255 past head_dim must not meet the query's zeros)
        }
    };
    const auto read_values = [&](const Reads &r0, int t, Values &v) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < NH; ++h) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t e = r0.vr + 8 * DP * t + 2 * DP * r + 64 * h;
                if constexpr (EL == 8)
                    v.w[r][h] = *(lds_u32 *)e;
                else
                    v.w[r][h] = *(lds_u16 *)e;
            }
            if constexpr (DENSE) {
#pragma unroll
                for (int r = 0; r < 4; ++r) v.unit[r][h] = *(lds_cu8 *)(r0.vsr + (DP == 256 ? 128 : 64) * t + r * BLOCKS + 4 * h);
            } else {
                const u32v4 u = *(lds_u32v4 *)(r0.vsr + 64 * BLOCKS * t + 64 * h);
                v.unit[0][h] = u.x, v.unit[1][h] = u.y, v.unit[2][h] = u.z, v.unit[3][h] = u.w;
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
#pragma unroll
            for (int x = 0; x < QP; ++x) sc = mma<__bf16>(f, q[c][x], sc);
        }
        return sc;
    };

    const int end = a.n_pages > 0 ? min(s.len, s.pos1) : s.pos0;
    bool found = false;  // a value that only some rows see is NaN: a weight of zero does not hide it
    const auto pass = [&](auto slow) __attribute__((always_inline)) {
        int kv0 = s.pos0, next = kv0;
        Issued x;
        x.bad = x.none = 0;
        x.k32 = 32 * b.kc.rs, x.v32 = 32 * b.vc.rs, x.ks32 = 32 * b.kc.s_rs, x.vs32 = 32 * b.vc.s_rs;
        asm volatile("" : "+s"(x.k32), "+s"(x.v32), "+s"(x.ks32), "+s"(x.vs32));
        x.pages.fetch(a, s, kv0 >> a.page_log2);
        // The queries are waited for with the pages, not in the loop, where a wait for them would be one for all loads to LDS.
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
            for (int i = 0; i < QP; ++i) asm volatile("" : "+v"(q[c][i]));
        uint32_t at = 0;
#pragma unroll 1
        for (int i = 0; i < STEPS; ++i, next += kAttnStep, at += Ring::STEP) {
            if (next < end)
                issue(x, next, ring + at);
            else
                x.bad <<= 2;
        }
        at = 0;
        for (; kv0 < end; kv0 += kAttnStep, next += kAttnStep) {
            if (next - kAttnStep < end)
                wait_all_but<Ring::ALL * (STEPS - 1)>();
            else
                wait_all_but<0>();
            Keys k0, k1;
            Values v0, v1;
            const Reads r = reads_of(at);
            read_keys(r, 0, k0);
            read_keys(r, 1, k1);
            read_values(r, 0, v0);
            read_values(r, 1, v1);
            const int here = kv0;
            const uint32_t none = x.bad >> (2 * (STEPS - 1)) & 3;
            if (next < end)
                issue(x, next, ring + at);
            else
                x.bad <<= 2;
            at = at == (STEPS - 1) * Ring::STEP ? 0 : at + Ring::STEP;
            f32x4 sc[2] = {scores(k0), scores(k1)};
            bool odd = false;
            if (here + kAttnStep > all_see || none) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int pos = here + 16 * t + 4 * g + r;
                        const bool page = !(none >> t & 1);
                        if (!page || pos >= vis) sc[t][r] = kNone;
#pragma unroll
                        for (int h = 0; h < NH; ++h) {
                            uint32_t &u = t ? v1.unit[r][h] : v0.unit[r][h];
                            if (!page || pos >= s.len)
                                u = 127;  // zero weight times whatever the page holds there is not zero
                            else if (pos >= all_see)
                                found |= u > 252;
                        }
                    }
                odd = slow;
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
            // weights as two numbers of bfloat16, the second the rest of the first (2^-17 of a weight are lost)
            u32v4 w0, w1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
                typedef float f32x2 __attribute__((ext_vector_type(2)));
                const f32x2 x = {w[2 * i], w[2 * i + 1]};
                w0[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
                const f32x2 rest = {x.x - __builtin_bit_cast(float, w0[i] << 16), x.y - __builtin_bit_cast(float, w0[i] & 0xFFFF0000u)};
                w1[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest, bf16x2));
            }

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
            if (!slow || !odd) {
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int c = 0; c < EL; ++c) {
                        const u32v4 f = turned(h, c);
                        o[h * EL + c] = mma<__bf16>(f, w1, mma<__bf16>(f, w0, o[h * EL + c]));
                    }
            } else if constexpr (slow) {
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
                            const f32x4 x = mma<__bf16>(f, w1, mma<__bf16>(f, w0, o[h * EL + c]));
                            if ((s.row0 + n) / a.group == j) o[h * EL + c] = x;
                        }
                }
            }
        }
    };
    pass(std::false_type{});
    if (__any(found)) {  // once more, with what a token does not see set to zero for it
        m = kNone;
        l = 0.0f;
#pragma unroll
        for (int c = 0; c < NH * EL; ++c) o[c] = f32x4{0, 0, 0, 0};
        pass(std::true_type{});
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
template <class T, int DP, bool DENSE>
__global__ __launch_bounds__(kAttnThreads, DP <= 128 ? 2 : 1) void attn4_split_kernel(Attn4Args b) {
    const AttnArgs &a = b.a;
    extern __shared__ int32_t dynamic[];
    __shared__ __attribute__((aligned(16))) uint8_t rings[kAttnWaves][Ring4<DP, DENSE>::BYTES];
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
    const uint32_t ring = (uint32_t)(size_t)(lds_u8 *)rings[wave];
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
        attend4<T, DP, DENSE>(b, s, ring);
        u += n;
    }
}

// Few positions: a workgroup takes a (sequence, key/value head, 16 query rows), its waves equal runs of its steps, and joins
// their parts through LDS.
template <int DP>
constexpr int kShort4Waves = DP == 256 ? 4 : 8;

template <class T, int DP, bool DENSE>
__global__ __launch_bounds__(64 * kShort4Waves<DP>) void attn4_short_kernel(Attn4Args b, int tiles) {
    constexpr int WAVES = kShort4Waves<DP>;
    const AttnArgs &a = b.a;
    // a wave's results take the place of what it read
    struct Part {
        float o[16][DP];
        float4 ml[16];
    };
    union Wave {
        Part part;
        uint8_t ring[Ring4<DP, DENSE>::BYTES];
    };
    __shared__ __attribute__((aligned(16))) Wave waves[WAVES];
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
    s.po = &waves[wave].part.o[0][0];
    s.pml = waves[wave].part.ml;
    if (s.pos0 < s.len)
        attend4<T, DP, DENSE>(b, s, (uint32_t)(size_t)(lds_u8 *)waves[wave].ring);
    else if ((tid & 63) < 16)
        waves[wave].part.ml[tid & 63] = make_float4(kNone, 0.0f, 0.0f, 0.0f);
    __syncthreads();
    for (int x = tid; x < 16 * (DP / 4); x += 64 * WAVES) {
        const int row = x / (DP / 4), d = 4 * (x - row * (DP / 4));
        if (s.row0 + row >= s.n_rows) break;
        float top = kNone;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) top = fmaxf(top, waves[w].part.ml[row].x);
        float sum = 0.0f;
        f32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float4 y = waves[w].part.ml[row];
            if (y.x == kNone) continue;  // (such a part's outputs may not be there)
            const float f = __builtin_amdgcn_exp2f(y.x - top);
            sum += f * y.y;
            acc += *reinterpret_cast<const f32x4 *>(&waves[w].part.o[row][d]) * f;
        }
        const int j = (s.row0 + row) / a.group;
        write_out<T>(a, tok.x + j, s.head * a.group + s.row0 + row - j * a.group, d, acc, top, sum, sum);
    }
}

template <class T, int DP, bool DENSE>
static int run_attn4_as(const Attn4Args &b, bool one_launch, hipStream_t st) {
    const AttnArgs &a = b.a;
    if (one_launch) {
        const int tiles = (a.max_q * a.group + 15) / 16;
        attn4_short_kernel<T, DP, DENSE><<<(unsigned)(a.n_seqs * a.kv_heads * tiles), 64 * kShort4Waves<DP>, 0, st>>>(b, tiles);
        return (int)hipGetLastError();
    }
    attn4_split_kernel<T, DP, DENSE><<<(unsigned)a.n_wgs, kAttnThreads, (size_t)(5 * (a.n_seqs + 1)) * 4, st>>>(b);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? (int)e : run_join<T, DP>(a, 16, 16, st);
}

template <class T, int DP>
static int run_attn4(const Attn4Args &b, bool one_launch, hipStream_t st) {
    return b.dense ? run_attn4_as<T, DP, true>(b, one_launch, st) : run_attn4_as<T, DP, false>(b, one_launch, st);
}

}  // namespace bpw
