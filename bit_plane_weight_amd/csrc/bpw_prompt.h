// bpw_prompt.h - causal attention over whole prompts packed one after another (gfx950, wave64), instantiated per padded head
// size by bpw_prompt_d*.hip.
//
// Mathematics. For a query row q and the positions i that it sees: s_i = scale <q, k_i>, a running shift m and sum
// l = sum exp(s_i - m), o = sum exp(s_i - m) v_i; a raised shift scales l and o by exp(m_old - m_new); out = o / l.
//
// Bound: matrix cores, 4 head_dim operations a score. The query heads that share a key/value head are rows of one tile (row
// = token * group + head), so that keys and values go once through LDS for 128 rows, moved there by the
// loads themselves one tile of 64 positions ahead of their use, and a tile of few tokens wastes little above the diagonal. A wave
// holds 32 rows and forms S^T = K Q^T and O^T += V^T P^T with 32x32x16 products as the wide path of bpw_attention.h does
// (the weights of a score tile are already the second operand of the next product; values are read transposed).
// Tiles that every row sees are a software pipeline: products of one block's values beside the next one's
// exponentials, products of scores beside the rounding of weights. Two workgroups fit a CU (one at heads of 256), whose waves
// fill each other's gaps; with 64 rows a wave and one workgroup LDS is read half as often, and long prompts ran as fast,
// all others slower. Tiles on the diagonal, whose hidden positions cost registers that the pipeline needs, come last, without it.
// Measured (causal half counted): 16384 tokens of 32 / 8 heads of 128 1.91-2.04 ms, 1.08-1.15 PFLOP/s, against 3.33 ms product by
// product; 2048 tokens of 20 / 5 heads 40-44 us; 4096 tokens of 16 / 4 heads of 256 152-183 us (0.75-0.9 PFLOP/s), where LDS and
// registers leave one wave a SIMD and nothing fills its gaps. The matrix cores are busy two
// thirds of the time at the clock that this load sustains (1.6 to 2.0 GHz), which is what bounds long prompts now.
// Within a sequence tiles with the most positions start first; sequences start in the reverse of their order. The key/value
// heads are dealt round the XCDs, so that with eight of them each XCD's L2 holds one.
#pragma once

#include <type_traits>

#include "bpw_attention.h"

namespace bpw {

#define BPW_INLINE __attribute__((always_inline))

// The sequence whose tiles of ROWS query rows hold a slot: its first token, its tokens, its first slot.
struct PromptSeq {
    int first, tokens, slot;
};

// It is the last sequence whose first slot is not beyond `slot`; no tokens if there is none. Every wave by itself, 63 probes at a
// time, the last of which have the starts of the sequence and of the next. Starts that do not rise give some sequence.
template <int ROWS>
__device__ __forceinline__ PromptSeq prompt_seq(const PromptArgs &a, int slot) {
    const int lane = threadIdx.x & 63;
    int lo = 0, hi = a.n_seqs;
    while (true) {
        const int step = (hi - lo + 62) / 63, at = min(lo + lane * step, a.n_seqs);
        const int start = min(max(a.starts[at], 0), a.n_tokens), first = prompt_slot(start * a.group, at, ROWS);
        const uint64_t below = __ballot(lane < 63 && lo + lane * step < hi && first <= slot);
        if (!below) return {0, 0, 0};
        const int l = 63 - __builtin_clzll(below);
        if (step == 1) {
            const int t0 = __builtin_amdgcn_readlane(start, l), t1 = __builtin_amdgcn_readlane(start, l + 1);
            return {t0, max(t1 - t0, 0), __builtin_amdgcn_readlane(first, l)};
        }
        lo += l * step;
        hi = min(lo + step, hi);
    }
}

// N times 16 bytes a lane from a buffer (offsets beyond its end give zeros): the i-th from offset[i] + 1024 i to LDS at `at` +
// 1024 i + 16 * lane; `at` and the buffer are the same in all lanes. Waited for by vmcnt; asm, as load_to_lds() is. m0 is set
// once, because each write of it waits for the loads to LDS before it (160 cycles a load); nothing else here uses it. A
// vector instruction's write of a scalar register (v_readlane) needs five wait states before a load reads it, which the
// compiler does not see to for asm.
template <int N>
__device__ __forceinline__ void buffer_to_lds(uint32_t at, u32v4 buffer, const uint32_t *offset) {
    static_assert(N == 2 || N == 4, "an instruction's offset has 12 bits");
    if constexpr (N == 4)
        asm volatile(
            "s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %2, %1, 0 offen lds\n\t"
            "buffer_load_dwordx4 %3, %1, 0 offen offset:0x400 lds\n\tbuffer_load_dwordx4 %4, %1, 0 offen offset:0x800 lds\n\t"
            "buffer_load_dwordx4 %5, %1, 0 offen offset:0xc00 lds"
            ::"s"(at), "s"(buffer), "v"(offset[0]), "v"(offset[1]), "v"(offset[2]), "v"(offset[3]) : "m0", "memory");
    else
        asm volatile(
            "s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %2, %1, 0 offen lds\n\t"
            "buffer_load_dwordx4 %3, %1, 0 offen offset:0x400 lds"
            ::"s"(at), "s"(buffer), "v"(offset[0]), "v"(offset[1]) : "m0", "memory");
}

// c + the two numbers of a word. (Not by a dot product: v_dot2 holds the matrix cores up, 50 cycles a product with one
// beside it, 33 without.)
template <class T>
__device__ __forceinline__ float add2(uint32_t x, float c) {
    if constexpr (__is_same(T, __bf16)) {
        return (c + __builtin_bit_cast(float, x << 16)) + __builtin_bit_cast(float, x & 0xFFFF0000u);
    } else {
        typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
        const f16x2 y = __builtin_bit_cast(f16x2, x);
        return __builtin_fmaf((float)y.y, 1.0f, __builtin_fmaf((float)y.x, 1.0f, c));
    }
}

// The halves of a word that are finite, zeros for the others; a half's number where it is not finite, zero otherwise.
template <class T>
__device__ __forceinline__ uint32_t finite_halves(uint32_t x) {
    constexpr uint32_t lo = __is_same(T, __bf16) ? 0x7F80u : 0x7C00u, hi = lo << 16;
    return ((x & lo) == lo ? 0u : x & 0xFFFFu) | ((x & hi) == hi ? 0u : x & 0xFFFF0000u);
}
template <class T>
__device__ __forceinline__ float odd_value(uint32_t half) {
    constexpr uint32_t ones = __is_same(T, __bf16) ? 0x7F80u : 0x7C00u;
    return (half & ones) == ones ? (float)__builtin_bit_cast(T, (uint16_t)half) : 0.0f;
}

typedef __attribute__((address_space(3))) const u32v4 lds_u32v4;
typedef __attribute__((address_space(3))) const u32x2 lds_u32x2;

// A workgroup of four waves takes 128 / PARTS query rows, 32 a wave, and 64 positions at a time; with two PARTS the waves of part
// p take the p-th 32 of them, and part 1's results are joined with part 0's at the end.
// Rows in LDS are of DP elements; products are formed of the first DU, a multiple of 32.
template <class T, int DP, int DU, int PARTS, bool PIPE, bool LSE>
__global__ __launch_bounds__(256, DP <= 128 ? 2 : 1) void prompt_kernel(PromptArgs a) {
    constexpr int KT = 64, M = 128 / PARTS, NB = 2 / PARTS;  // positions and rows of a tile, blocks of 32 positions of a wave
    constexpr int ROW = DP * 2, CPR = DP / 8, RPI = 64 / CPR;  // row bytes, chunks of a row, rows of one load
    constexpr int KC = DU / 16, DB = DU / 32, TILE = KT * ROW;  // bytes of a tile of keys or values
    __shared__ __attribute__((aligned(2 * TILE))) uint8_t lds[4 * TILE];  // keys twice, values twice (a buffer is chosen by an exclusive-or)
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, g = lane >> 5, part = PARTS == 2 ? wave >> 1 : 0, rows_of = PARTS == 2 ? wave & 1 : wave;
    const int D = a.head_dim;

    // A sequence's tiles of many positions first, the last sequence's before the others'; workgroup id runs on XCD id % 8, so that
    // with eight key/value heads each L2 holds one.
    const int id = a.first_wg + (int)blockIdx.x, head = id % a.kv_heads, slot = a.slots - 1 - id / a.kv_heads;
    const PromptSeq seq = prompt_seq<M>(a, slot);
    const int t0 = seq.first, len = seq.tokens, n_rows = len * a.group, row0 = (slot - seq.slot) * M;
    if (row0 >= n_rows) return;
    const int end = (min(row0 + M, n_rows) - 1) / a.group + 1;  // positions that the tile's last row sees
    const int tiles = (end + KT - 1) / KT;

    const int row_first = row0 + 32 * rows_of, row = row_first + n;
    const int token = row / a.group, hq = head * a.group + row - token * a.group;
    const int vis = row < n_rows ? token + 1 : len;
    const int all_see = __builtin_amdgcn_readfirstlane(row_first / a.group + 1);  // what every row of the wave sees
    u32v4 q[KC];
    {
        const T *p = static_cast<const T *>(a.q) + (int64_t)(t0 + token) * a.q_ts + (int64_t)hq * a.q_hs;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            q[c] = u32v4{0, 0, 0, 0};
            if (row < n_rows && 16 * c + 8 * g < D) q[c] = *reinterpret_cast<const u32v4 *>(p + 16 * c + 8 * g);
        }
    }
    const T *kbase = static_cast<const T *>(a.k) + (int64_t)t0 * a.k_ts + (int64_t)head * a.k_hs;
    const T *vbase = static_cast<const T *>(a.v) + (int64_t)t0 * a.v_ts + (int64_t)head * a.v_hs;

    // Moves of tiles to LDS, 16 bytes a lane. A wave takes sixteen positions of a tile, RPI a load, by a buffer that ends with
    // them: positions past the sequence, elements past head_dim (lanes with an offset beyond every buffer) and
    // tiles past the last become zeros (a zero weight times whatever memory holds there would not be one).
    constexpr int LOADS = 16 / RPI, GROUP = LOADS < 4 ? LOADS : 4;  // loads; after one setting of m0
    constexpr int BACK = 1024 * (GROUP - 1);  // (a load's AT moves both addresses, so that buffers begin this much earlier)
    const uint32_t lds0 = (uint32_t)(size_t)(lds_u8 *)lds;
    uint32_t ks[LOADS], vs[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int r = RPI * i + lane / CPR, ck = (lane % CPR) ^ key_of_k<DP>(r), cv = (lane % CPR) ^ key_of_v<DP>(r);
        ks[i] = 8 * ck < D ? 2 * (r * a.k_ts + 8 * ck) + BACK - 1024 * (i % GROUP) : 0x80000000u;
        vs[i] = 8 * cv < D ? 2 * (r * a.v_ts + 8 * cv) + BACK - 1024 * (i % GROUP) : 0x80000000u;
    }
    const auto move_tile = [&](bool values, int t) BPW_INLINE {
        const T *base = values ? vbase : kbase;
        const int32_t stride = values ? a.v_ts : a.k_ts;
        const int first = KT * t + 16 * wave, here = min(16, len - first);
        const uint32_t there = (uint32_t)((-here & (t - tiles)) >> 31);  // all ones, or 0: nothing (without a branch)
        const uint64_t at = (uint64_t)(base + (int64_t)first * stride) - BACK;
        const u32v4 buffer = {(uint32_t)at, (uint32_t)(at >> 32) & 0xFFFFu, (uint32_t)(2 * ((here - 1) * stride + D) + BACK) & there, 0x00020000u};
#pragma unroll
        for (int i = 0; i < LOADS; i += GROUP)
            buffer_to_lds<GROUP>(lds0 + (values ? 2 * TILE : 0) + (t & 1) * TILE + 16 * wave * ROW + 1024 * i, buffer, (values ? vs : ks) + i);
    };

    // LDS addresses of this lane's reads of the current tiles. The chunk of element group c is chosen by an exclusive-or of the
    // first one's address (blocks of 32 and 16 positions are whole keys apart), and so is the other buffer.
    uint32_t ka = lds0 + (32 * part + n) * ROW + ((g ^ key_of_k<DP>(n)) * 16), va;
    constexpr uint32_t V8 = 16 * (key_of_v<DP>(8) ^ key_of_v<DP>(0));  // of the row 8 further on
    {
        const int i = lane & 15, r = 4 * g + (i >> 2), chunk = 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
        va = lds0 + 2 * TILE + (32 * part + r) * ROW + ((chunk ^ key_of_v<DP>(r)) * 16) + (i & 1) * 8;
    }
    const auto key_frag = [&](int blk, int c) BPW_INLINE { return *(lds_u32v4 *)((ka ^ (32 * c)) + blk * 32 * ROW); };
    const auto value_frag = [&](int x, int c) BPW_INLINE {  // positions 16 x .. 16 x + 15 of this wave's
        const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)((va ^ (64 * c)) + 16 * x * ROW)));
        const u32x2 z = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)((va ^ (64 * c) ^ V8) + (16 * x + 8) * ROW)));
        return u32v4{y.x, y.y, z.x, z.y};
    };

    // sc: scores of two blocks of 32 positions; w, p: weights of the last one, in float32 and as operands; bs, bl: their sums
    // over this lane's positions, rounded and not
    f32x16 o[DB], sc[2];
    f32x8 w[2];
    u32v4 p[2];
    float m = kNone, l = 0.0f, lr = 0.0f, bs, bl;
#pragma unroll
    for (int c = 0; c < DB; ++c) o[c] = f32x16{};
    const auto weigh_one = [&](int which, int r, float shift) BPW_INLINE {
        w[r >> 3][r & 7] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[which][r], a.scale_log2, -shift));
    };
    // Weights 2 i and 2 i + 1 of operand h in 16 bits: half a step of relative error each; o is divided by the sum of the rounded
    // weights, so that errors they share cancel. lse takes the sum of the unrounded ones.
    const auto round_two = [&](int h, int i) BPW_INLINE {
        typedef T T2 __attribute__((ext_vector_type(2)));
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        const f32x2 y = {w[h][2 * i], w[h][2 * i + 1]};
        p[h][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, T2));
        bs = add2<T>(p[h][i], h + i == 0 ? 0.0f : bs);
        if constexpr (LSE) bl = (h + i == 0 ? y.x : bl + y.x) + y.y;
    };
    const auto weigh = [&](int which, float shift) BPW_INLINE {
#pragma unroll
        for (int r = 0; r < 16; ++r) weigh_one(which, r, shift);
#pragma unroll
        for (int e = 0; e < 8; ++e) round_two(e / 4, e % 4);
    };
    // The weights are taken against a shift, not the exact maximum: while a lane's sum of a block stays below kShiftLimit nothing
    // is lost, in float32 or in 16 bits, and no maximum is formed. Otherwise (the first block, a score far above all
    // before it, NaN) the shift becomes the maximum less kLift, and the block's weights are formed again.
    const auto settle = [&](int which) BPW_INLINE {
        if (__any(!(bs < kShiftLimit<T>))) {
            float top = kNone;
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, sc[which][r]);
            top = fmaxf(top, __shfl_xor(top, 32)) * a.scale_log2;
            const float up = fmaxf(m, top - kLift<T>);
            const float f = up == m ? 1.0f : __builtin_amdgcn_exp2f(m - up);
            m = up;
            l *= f;
            lr *= f;
#pragma unroll
            for (int c = 0; c < DB; ++c) o[c] *= f;
            weigh(which, up == kNone ? 0.0f : up);
        }
        lr += bs;
        if constexpr (LSE) l += bl;
    };
    // Positions that a row does not see, in the scores of block blk of tile t.
    const auto hide = [&](int which, int t, int blk) BPW_INLINE {
        const int first = KT * t + 32 * (part + blk);
#pragma unroll
        for (int r = 0; r < 16; ++r)
            if (first + 8 * (r >> 2) + 4 * g + (r & 3) >= vis) sc[which][r] = kNone;
    };
    // The main loop's two regions. A wave issues its instructions one after another, and the matrix cores take one of its products
    // (32 cycles) while the vector units take what stands behind it: so each product is followed by its share of the other
    // work and of the operand reads, two operands ahead, and kept in that order.
    constexpr int VF = 2 * DB;
    u32v4 kf[KC], vf[VF];
    const auto first_keys = [&](int blk) BPW_INLINE { kf[0] = key_frag(blk, 0), kf[1] = key_frag(blk, 1); };
    const auto first_values = [&](int blk) BPW_INLINE { vf[0] = value_frag(2 * blk, 0), vf[1] = value_frag(2 * blk + 1 / DB, 1 % DB); };
    // Products of the values of block blk; weights of sc[which], of which the first `ahead` come before the products
    // (whose operands are still on their way).
    const auto values_and_weights = [&](int blk, int which, int ahead) BPW_INLINE {
#pragma unroll
        for (int e = 0; e < ahead; ++e) weigh_one(which, e, m);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < VF; ++i) {
            if (i + 2 < VF) vf[i + 2] = value_frag(2 * blk + (i + 2) / DB, (i + 2) % DB);
            o[i % DB] = mma32<T>(vf[i], p[i / DB], o[i % DB]);
#pragma unroll
            for (int e = ahead + i * (16 - ahead) / VF; e < ahead + (i + 1) * (16 - ahead) / VF; ++e) weigh_one(which, e, m);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // Products of block blk's scores, into sc[which]; the weights in 16 bits.
    const auto scores_and_rounding = [&](int blk, int which) BPW_INLINE {
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            if (i + 2 < KC) kf[i + 2] = key_frag(blk, i + 2);
            sc[which] = mma32<T>(kf[i], q[i], i ? sc[which] : f32x16{});
#pragma unroll
            for (int e = i * 8 / KC; e < (i + 1) * 8 / KC; ++e) round_two(e / 4, e % 4);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    const auto scores = [&](int blk, int which) BPW_INLINE {
#pragma unroll
        for (int i = 0; i < KC; ++i) sc[which] = mma32<T>(key_frag(blk, i), q[i], i ? sc[which] : f32x16{});
    };

    const auto values = [&](int blk) BPW_INLINE {
#pragma unroll
        for (int i = 0; i < VF; ++i) o[i % DB] = mma32<T>(value_frag(2 * blk + i / DB, i % DB), p[i / DB], o[i % DB]);
    };

    uint32_t odd = 0;  // a value that only some rows of the wave see is not finite: a weight of zero does not hide it
    const auto look_for_odd = [&] BPW_INLINE {
#pragma unroll 4
        for (int j = 0; j < 2 * NB * DB; ++j) {
            const u32v4 f = value_frag(j / DB, j % DB);
#pragma unroll
            for (int e = 0; e < 4; ++e) odd |= maybe_not_finite<T>(f[e]);
        }
    };
    const int wave_end = row_first < n_rows ? (min(row_first + 32, n_rows) - 1) / a.group + 1 : 0;  // what some row of the wave sees
    const auto arrive = [&] BPW_INLINE {
        wait_loads_to_lds();
        __syncthreads();  // what was on its way is there, and nobody reads the tiles before any more
    };
    int t = 0;
    move_tile(false, 0);
    move_tile(true, 0);
    if constexpr (PIPE) {
        // Tiles that all rows see, a block of 32 positions after another: the products of the last block's values beside this
        // block's exponentials, those of the next block's scores beside the rounding of its weights.
        const int full = (row0 / a.group + 1) / KT;
        if (full > 0) {
            move_tile(false, 1);  // keys run a tile ahead of values
            arrive();
            scores(0, 0);
            weigh(0, m);
            settle(0);
            scores(1, 1);
            ka ^= TILE;
            for (; t + 1 < full; ++t) {
                arrive();
                first_values(0);
                first_keys(0);
                move_tile(true, t + 1);
                move_tile(false, t + 2);
                values_and_weights(0, 1, 4);
                first_values(1);
                scores_and_rounding(0, 0);
                settle(1);
                first_keys(1);
                values_and_weights(1, 0, 0);
                scores_and_rounding(1, 1);
                settle(0);
                ka ^= TILE;
                va ^= TILE;
            }
            arrive();
            move_tile(true, t + 1);
            values(0);
            weigh(1, m);
            settle(1);
            values(1);
            va ^= TILE;
            ++t;
        }
    }
    for (; t < tiles; ++t) {
        arrive();
        move_tile(false, t + 1);
        move_tile(true, t + 1);
        if (KT * t + 32 * part < wave_end) {
            const bool all = KT * t + 64 <= all_see;
            scores(0, 0);
            if constexpr (NB == 2) scores(1, 1);
            if (!all) {
                look_for_odd();
                hide(0, t, 0);
                if constexpr (NB == 2) hide(1, t, 1);
            }
            weigh(0, m);
            settle(0);
            values(0);
            if constexpr (NB == 2) {
                weigh(1, m);
                settle(1);
                values(1);
            }
        }
        ka ^= TILE;
        va ^= TILE;
    }

    // In float16 a weight below 2^-31 of the largest is zero, and zero times an infinite value is NaN, which the value's own
    // weight would not have made of it: looked for in the outputs.
    if constexpr (__is_same(T, _Float16)) {
        float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < DB; ++c)
#pragma unroll
            for (int r = 0; r < 16; ++r) z[r & 3] = __builtin_fmaf(o[c][r], 0.0f, z[r & 3]);
        const float any = (z[0] + z[1]) + (z[2] + z[3]);
        if (any != any && lr == lr) odd = 1;
    }
    wait_loads_to_lds();  // (zeros of tiles past the last: LDS is used anew)
    // Values that are not finite and not seen by all, or that met a weight of zero: the tile of rows once more, step by step, with zeros
    // in the place of such values, which are then added to the rows that see them (times any weight above zero they stay what they are).
    if (__syncthreads_or((int)odd)) {
        m = kNone;
        l = lr = 0.0f;
#pragma unroll
        for (int c = 0; c < DB; ++c) o[c] = f32x16{};
        if (tiles % 2) ka ^= TILE, va ^= TILE;
        for (int t = 0; t < tiles; ++t) {
            __syncthreads();
            move_tile(false, t);
            move_tile(true, t);
            wait_loads_to_lds();
            __syncthreads();
#pragma unroll 1
            for (int blk = 0; blk < NB; ++blk) {
                scores(blk, 0);
                hide(0, t, blk);
                weigh(0, m);
                settle(0);
                const int first = KT * t + 32 * (part + blk);
                const bool some = __is_same(T, _Float16) || first + 32 > all_see;
                uint32_t found = 0;
#pragma unroll
                for (int i = 0; i < VF; ++i) {
                    u32v4 f = value_frag(2 * blk + i / DB, i % DB);
                    if (some) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) found |= maybe_not_finite<T>(f[e]), f[e] = finite_halves<T>(f[e]);
                    }
                    o[i % DB] = mma32<T>(f, p[i / DB], o[i % DB]);
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (!__any(found != 0)) continue;  // (all of the block's values were among the wave's operands)
#pragma unroll 1
                for (int i = 0; i < 32; ++i) {
                    const int r = 32 * (part + blk) + i;  // of the tile
                    const bool sees = row < n_rows && first + i <= token;
#pragma unroll
                    for (int c = 0; c < DB; ++c) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const u32x2 v = *(lds_u32x2 *)(lds0 + 2 * TILE + (t & 1) * TILE + r * ROW + (((4 * c + j) ^ key_of_v<DP>(r)) * 16) + 8 * g);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float y = odd_value<T>((e & 2 ? v.y : v.x) >> (16 * (e & 1)));
                                o[c][4 * j + e] += sees ? y : 0.0f;
                            }
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    }
                }
            }
            ka ^= TILE;
            va ^= TILE;
        }
    }

    l += __shfl_xor(l, 32);
    lr += __shfl_xor(lr, 32);
    m = stored_shift(m, lr);
    if constexpr (PARTS == 2) {  // part 1 hands over through LDS
        constexpr int PAD = DU + 4;
        static_assert(M * (PAD + 4) * 4 <= sizeof lds, "the join fits the tiles' LDS");
        float *box = reinterpret_cast<float *>(lds) + (32 * rows_of + n) * PAD;
        float4 *ml = reinterpret_cast<float4 *>(reinterpret_cast<float *>(lds) + M * PAD) + 32 * rows_of + n;
        __syncthreads();
        if (part == 1) {
#pragma unroll
            for (int c = 0; c < DB; ++c)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    *reinterpret_cast<f32x4 *>(box + 32 * c + 8 * r + 4 * g) = f32x4{o[c][4 * r], o[c][4 * r + 1], o[c][4 * r + 2], o[c][4 * r + 3]};
            if (g == 0) *ml = make_float4(m, l, lr, 0.0f);
        }
        __syncthreads();
        if (part == 1) return;
        const float4 x = *ml;
        const float up = fmaxf(m, x.x);
        const float f0 = m == kNone ? 0.0f : __builtin_amdgcn_exp2f(m - up), f1 = x.x == kNone ? 0.0f : __builtin_amdgcn_exp2f(x.x - up);
        m = up;
        l = l * f0 + x.y * f1;
        lr = lr * f0 + x.z * f1;
#pragma unroll
        for (int c = 0; c < DB; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const f32x4 y = *reinterpret_cast<const f32x4 *>(box + 32 * c + 8 * r + 4 * g);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[c][4 * r + e] = o[c][4 * r + e] * f0 + y[e] * f1;
            }
    }
    if (row >= n_rows) return;
    const float inv = 1.0f / lr;
    typedef T T4 __attribute__((ext_vector_type(4)));
    T *out = static_cast<T *>(a.out) + (int64_t)(t0 + token) * a.o_ts + (int64_t)hq * a.o_hs;
#pragma unroll
    for (int c = 0; c < DB; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int d = 32 * c + 8 * r + 4 * g;
            if (d < D)
                *reinterpret_cast<T4 *>(out + d) =
                    __builtin_convertvector((f32x4{o[c][4 * r], o[c][4 * r + 1], o[c][4 * r + 2], o[c][4 * r + 3]}) * inv, T4);
        }
    if (LSE && g == 0) a.lse[(int64_t)(t0 + token) * a.q_heads + hq] = (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
}

template <class T, int DP, int DU, int PARTS, bool PIPE>
static int run_prompt_parts(PromptArgs a, hipStream_t s) {
    a.slots = prompt_slot(a.n_tokens * a.group, a.n_seqs, 128 / PARTS);
    const int64_t wgs = (int64_t)a.slots * a.kv_heads;
    if (wgs > INT32_MAX) return (int)hipErrorInvalidValue;
    for (;; a.first_wg += kMaxWgs) {
        const int64_t left = wgs - a.first_wg;
        const unsigned grid = (unsigned)(left < kMaxWgs ? left : kMaxWgs);
        if (a.lse)
            prompt_kernel<T, DP, DU, PARTS, PIPE, true><<<grid, 256, 0, s>>>(a);
        else
            prompt_kernel<T, DP, DU, PARTS, PIPE, false><<<grid, 256, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || left <= kMaxWgs) return (int)e;
    }
}

template <class T, int DP, int DU>
static int run_prompt_of(const PromptArgs &a, bool many, hipStream_t s) {
    return many ? run_prompt_parts<T, DP, DU, 1, true>(a, s) : run_prompt_parts<T, DP, DU, 2, false>(a, s);
}
// Heads of up to three quarters of DP leave out the last quarter of the products (4096 tokens of 32 / 8 heads of 96: 124 us, 141 with
// all of them; of 16 / 4 heads of 192 136, 160).
template <class T, int DP>
static int run_prompt(const PromptArgs &a, bool many, hipStream_t s) {
    if constexpr (DP > 64)
        if (a.head_dim <= DP * 3 / 4) return run_prompt_of<T, DP, DP * 3 / 4>(a, many, s);
    return run_prompt_of<T, DP, DP>(a, many, s);
}

#undef BPW_INLINE

}  // namespace bpw
