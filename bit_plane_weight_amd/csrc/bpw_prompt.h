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
// Tiles with the most positions start first. The key/value heads are dealt round the XCDs, so that with eight of them each
// XCD's L2 holds one.
#pragma once

#include "bpw_attention.h"

namespace bpw {

// The sequence whose tiles hold slot `slot`: the last whose first slot is not beyond it, or -1. Every wave by itself, 64
// probes at a time. Starts that do not rise give some sequence.
__device__ __forceinline__ int prompt_seq(const PromptArgs &a, int slot, int rows) {
    const auto first = [&](int b) { return prompt_slot(min(max(a.starts[b], 0), a.n_tokens) * a.group, b, rows); };
    int lo = 0, hi = a.n_seqs;
    while (true) {
        const int step = (hi - lo + 63) / 64, at = lo + (int)(threadIdx.x & 63) * step;
        const uint64_t below = __ballot(at < hi && first(at) <= slot);
        if (!below) return -1;
        lo += (63 - __builtin_clzll(below)) * step;
        if (step == 1) return __builtin_amdgcn_readfirstlane(lo);
        hi = min(lo + step, hi);
    }
}

// 16 bytes a lane from a buffer (offsets beyond its end give zeros) to LDS at `to` + 16 * lane; `to` and the buffer are the same
// in all lanes. Waited for by vmcnt; asm, as load_to_lds() is.
__device__ __forceinline__ void buffer_to_lds(uint32_t to, uint32_t offset, u32v4 buffer) {
    uint32_t keep;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds\n\ts_mov_b32 m0, %0"
                 : "=&s"(keep)
                 : "s"(to), "v"(offset), "s"(buffer)
                 : "memory");
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

// Shape of a kernel: a wave holds S sets of 32 query rows, WQ waves lie along the rows of a tile and the others along the
// positions, of which a workgroup takes KT at a time and a wave two blocks of 32.
template <int DP_, int S_, int WQ_>
struct PromptShape {
    static constexpr int DP = DP_, S = S_, WQ = WQ_;
    static constexpr int PARTS = kAttnWaves / WQ, KT = 64 * PARTS, ROWS = 32 * S * WQ;
};

template <class T, class P, bool LSE>
__global__ __launch_bounds__(kAttnThreads, 1) void prompt_kernel(PromptArgs a) {
    constexpr int DP = P::DP, S = P::S, WQ = P::WQ, PARTS = P::PARTS, KT = P::KT, M = P::ROWS;
    constexpr int ROW = DP * 2, CPR = DP / 8, RPI = 64 / CPR;  // row bytes, chunks of a row, rows of one load
    constexpr int KC = DP / 16, DB = DP / 32, TILE = KT * ROW;  // bytes of a tile of keys or values
    __shared__ __attribute__((aligned(4096))) uint8_t lds[4 * TILE];  // keys twice, values twice
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 31, g = lane >> 5, part = wave / WQ;
    const int D = a.head_dim;

    const int id = a.first_wg + (int)blockIdx.x, head = id % a.kv_heads, slot = a.slots - 1 - id / a.kv_heads;
    const int b = prompt_seq(a, slot, M);
    if (b < 0) return;
    const int t0 = min(max(a.starts[b], 0), a.n_tokens), t1 = min(max(a.starts[b + 1], t0), a.n_tokens);
    const int len = t1 - t0, n_rows = len * a.group, row0 = (slot - prompt_slot(t0 * a.group, b, M)) * M;
    if (row0 < 0 || row0 >= n_rows) return;
    const int end = (min(row0 + M, n_rows) - 1) / a.group + 1;  // positions that the tile's last row sees
    // tiles of positions, and those of them that every row sees whole
    const int tiles = (end + KT - 1) / KT, full = (row0 / a.group + 1) / KT;

    const int row_first = row0 + 32 * S * (wave % WQ);
    const int some_see = row_first < n_rows ? (min(row_first + 32 * S, n_rows) - 1) / a.group + 1 : 0;
    u32v4 q[S][KC];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int row = row_first + 32 * s + n, token = row / a.group, hq = head * a.group + row - token * a.group;
        const T *p = static_cast<const T *>(a.q) + (int64_t)(t0 + token) * a.q_ts + (int64_t)hq * a.q_hs;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            q[s][c] = u32v4{0, 0, 0, 0};
            if (row < n_rows && 16 * c + 8 * g < D) q[s][c] = *reinterpret_cast<const u32v4 *>(p + 16 * c + 8 * g);
        }
    }
    const T *kbase = static_cast<const T *>(a.k) + (int64_t)t0 * a.k_ts + (int64_t)head * a.k_hs;
    const T *vbase = static_cast<const T *>(a.v) + (int64_t)t0 * a.v_ts + (int64_t)head * a.v_hs;

    // Moves of tiles to LDS, 16 bytes a lane. A wave takes sixteen of each 64 positions, RPI a load, by a buffer that ends with
    // them: positions past the sequence, elements past head_dim (lanes with an offset beyond every buffer) and
    // tiles past the last become zeros (a zero weight times whatever memory holds there would not be one).
    constexpr int LOADS = 16 / RPI;  // of sixteen positions
    const uint32_t lds0 = (uint32_t)(size_t)(lds_u8 *)lds;
    uint32_t ks[LOADS], vs[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int r = RPI * i + lane / CPR, ck = (lane % CPR) ^ key_of_k<DP>(r), cv = (lane % CPR) ^ key_of_v<DP>(r);
        ks[i] = 8 * ck < D ? 2 * (r * a.k_ts + 8 * ck) : 0x80000000u;
        vs[i] = 8 * cv < D ? 2 * (r * a.v_ts + 8 * cv) : 0x80000000u;
    }
    constexpr int MOVES = KT / 64 * LOADS;  // loads of a wave's share of a tile
    const auto move = [&](const T *base, int32_t stride, const uint32_t (&offset)[LOADS], uint32_t to, int t, int i) {
        const int first = KT * t + 64 * (i / LOADS) + 16 * wave, here = t < tiles ? min(16, len - first) : 0;
        const uint64_t at = (uint64_t)(base + (int64_t)first * stride);
        const u32v4 buffer = {(uint32_t)at, (uint32_t)(at >> 32), (uint32_t)max(0, 2 * ((here - 1) * stride + D)), 0x00020000u};
        buffer_to_lds(lds0 + to + (t & 1) * TILE + (64 * (i / LOADS) + 16 * wave) * ROW + 1024 * (i % LOADS), offset[i % LOADS], buffer);
    };
    const auto move_key = [&](int t, int i) { move(kbase, a.k_ts, ks, 0, t, i); };
    const auto move_value = [&](int t, int i) { move(vbase, a.v_ts, vs, 2 * TILE, t, i); };
    const auto move_keys = [&](int t) {
#pragma unroll
        for (int i = 0; i < MOVES; ++i) move_key(t, i);
    };
    const auto move_values = [&](int t) {
#pragma unroll
        for (int i = 0; i < MOVES; ++i) move_value(t, i);
    };

    // LDS addresses of this lane's reads of the current tiles. The chunk of element group c is chosen by an exclusive-or of the
    // first one's address (blocks of 32 and 16 positions are whole keys apart), and so is the other buffer.
    uint32_t ka = lds0 + (64 * part + n) * ROW + ((g ^ key_of_k<DP>(n)) * 16), va;
    constexpr uint32_t V8 = 16 * (key_of_v<DP>(8) ^ key_of_v<DP>(0));  // of the row 8 further on
    {
        const int i = lane & 15, r = 4 * g + (i >> 2), chunk = 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
        va = lds0 + 2 * TILE + (64 * part + r) * ROW + ((chunk ^ key_of_v<DP>(r)) * 16) + (i & 1) * 8;
    }
    const auto key_frag = [&](int blk, int c) { return *(lds_u32v4 *)((ka ^ (32 * c)) + blk * 32 * ROW); };
    const auto value_frag = [&](int x, int c) {  // positions 16 x .. 16 x + 15 of this wave's
        const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)((va ^ (64 * c)) + 16 * x * ROW)));
        const u32x2 z = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)((va ^ (64 * c) ^ V8) + (16 * x + 8) * ROW)));
        return u32v4{y.x, y.y, z.x, z.y};
    };

    // sc: scores of two blocks of 32 positions; w, p: weights of the last one, in float32 and as operands; bs, bl: their sums
    // over this lane's positions, rounded and not
    f32x16 o[S][DB], sc[2][S];
    f32x8 w[S][2];
    u32v4 p[S][2];
    float m[S], l[S], lr[S], bs[S], bl[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        m[s] = kNone;
        l[s] = lr[s] = 0.0f;
#pragma unroll
        for (int c = 0; c < DB; ++c) o[s][c] = f32x16{};
    }
    const auto scores = [&](int which, int blk) {
#pragma unroll
        for (int s = 0; s < S; ++s) sc[which][s] = f32x16{};
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            const u32v4 f = key_frag(blk, c);
#pragma unroll
            for (int s = 0; s < S; ++s) sc[which][s] = mma32<T>(f, q[s][c], sc[which][s]);
        }
    };
    const auto values = [&](int blk) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < DB; ++c) {
                const u32v4 f = value_frag(2 * blk + h, c);
#pragma unroll
                for (int s = 0; s < S; ++s) o[s][c] = mma32<T>(f, p[s][h], o[s][c]);
            }
    };
    const auto weigh_one = [&](int which, int s, int r, float shift) {
        w[s][r >> 3][r & 7] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[which][s][r], a.scale_log2, -shift));
    };
    // Weights 2 i and 2 i + 1 of operand h in 16 bits: half a step of relative error each; o is divided by the sum of the rounded
    // weights, so that errors they share cancel. lse takes the sum of the unrounded ones.
    const auto round_two = [&](int s, int h, int i) {
        typedef T T2 __attribute__((ext_vector_type(2)));
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        const f32x2 y = {w[s][h][2 * i], w[s][h][2 * i + 1]};
        p[s][h][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, T2));
        bs[s] = add2<T>(p[s][h][i], h + i == 0 ? 0.0f : bs[s]);
        if constexpr (LSE) bl[s] = (h + i == 0 ? y.x : bl[s] + y.x) + y.y;
    };
    const auto weigh = [&](int which, int s, float shift) {
#pragma unroll
        for (int r = 0; r < 16; ++r) weigh_one(which, s, r, shift);
#pragma unroll
        for (int e = 0; e < 8; ++e) round_two(s, e / 4, e % 4);
    };
    // The weights are taken against a shift, not the exact maximum: while a lane's sum of a block stays below kShiftLimit nothing
    // is lost, in float32 or in 16 bits, and no maximum is formed. Otherwise (the first block, a score far above all
    // before it, NaN) the shift becomes the maximum less kLift, and the block's weights are formed again.
    const auto settle = [&](int which) {
        bool high = false;
#pragma unroll
        for (int s = 0; s < S; ++s) high = high || !(bs[s] < kShiftLimit<T>);
        if (__any(high)) {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float top = kNone;
#pragma unroll
                for (int r = 0; r < 16; ++r) top = fmaxf(top, sc[which][s][r]);
                top = fmaxf(top, __shfl_xor(top, 32)) * a.scale_log2;
                const float up = fmaxf(m[s], top - kLift<T>);
                const float f = up == m[s] ? 1.0f : __builtin_amdgcn_exp2f(m[s] - up);
                m[s] = up;
                l[s] *= f;
                lr[s] *= f;
#pragma unroll
                for (int c = 0; c < DB; ++c) o[s][c] *= f;
                weigh(which, s, up == kNone ? 0.0f : up);
            }
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            lr[s] += bs[s];
            if constexpr (LSE) l[s] += bl[s];
        }
    };

    // The main loop's two regions. A wave issues its instructions one after another, and the matrix cores take one of its products
    // (32 cycles) while the vector units take what stands behind it: so each product is followed by its share of the other
    // work and of the operand reads, two operands ahead, and kept in that order.
    constexpr int VF = 2 * DB, PB = S * VF, PA = S * KC;  // operands and products
    u32v4 kf[KC], vf[VF];
    const auto first_keys = [&](int blk) { kf[0] = key_frag(blk, 0), kf[1] = key_frag(blk, 1); };
    const auto first_values = [&](int blk) { vf[0] = value_frag(2 * blk, 0), vf[1] = value_frag(2 * blk + 1 / DB, 1 % DB); };
    // Products of block vblk's values; weights of sc[which], of which `early` come before the first product (above 0: the
    // operands are still on their way) or begin `-early` products later (the scores are). The loads of the tiles to come.
    const auto values_and_weights = [&](int vblk, int which, int early, int loads_of) {
        const int lead = early < 0 ? -early : 0, ahead = early > 0 ? early : 0;
        const auto weights = [&](int e0, int e1) {
#pragma unroll
            for (int e = e0; e < e1; ++e) weigh_one(which, e / 16, e % 16, m[e / 16]);
        };
        weights(0, ahead);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            const int j = i / S, s = i % S, rest = 16 * S - ahead;
            if (s == 0 && j + 2 < VF) vf[j + 2] = value_frag(2 * vblk + (j + 2) / DB, (j + 2) % DB);
            o[s][j % DB] = mma32<T>(vf[j], p[s][j / DB], o[s][j % DB]);
            weights(ahead + max(0, i - lead) * rest / (PB - lead), ahead + max(0, i + 1 - lead) * rest / (PB - lead));
            if (loads_of >= 0)
#pragma unroll
                for (int x = i * 2 * MOVES / PB; x < (i + 1) * 2 * MOVES / PB; ++x) x % 2 ? move_key(loads_of + 2, x / 2) : move_value(loads_of + 1, x / 2);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // Products of block kblk's scores, into sc[which]; the weights in 16 bits.
    const auto scores_and_rounding = [&](int kblk, int which) {
#pragma unroll
        for (int i = 0; i < PA; ++i) {
            const int x = i / KC, c = i % KC;
            if (x == 0 && c + 2 < KC) kf[c + 2] = key_frag(kblk, c + 2);
            sc[which][x] = mma32<T>(kf[c], q[x][c], c ? sc[which][x] : f32x16{});
#pragma unroll
            for (int e = i * 8 * S / PA; e < (i + 1) * 8 * S / PA; ++e) round_two(e / 8, e / 4 % 2, e % 4);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    move_keys(0);
    move_values(0);
    move_keys(1);
    int t = 0;
    // Tiles that every row sees whole, a block of 32 positions after another: the products of the last block's values beside
    // this block's exponentials, those of the next block's scores beside the rounding of its weights. Keys run a tile ahead.
    if (full > 0) {
        wait_loads_to_lds();
        __syncthreads();
        scores(0, 0);
#pragma unroll
        for (int s = 0; s < S; ++s) weigh(0, s, m[s]);
        settle(0);
        scores(1, 1);
        ka ^= TILE;
        for (; t + 1 < full; ++t) {
            wait_loads_to_lds();
            __syncthreads();  // these tiles are there, and nobody reads those before them any more
            first_values(0);
            first_keys(0);
            values_and_weights(0, 1, 8, t);
            first_values(1);
            scores_and_rounding(0, 0);
            settle(1);
            first_keys(1);
            values_and_weights(1, 0, -2, -1);
            scores_and_rounding(1, 1);
            settle(0);
            ka ^= TILE;
            va ^= TILE;
        }
        wait_loads_to_lds();
        __syncthreads();
        move_values(t + 1);
        move_keys(t + 2);
        values(0);
#pragma unroll
        for (int s = 0; s < S; ++s) weigh(1, s, m[s]);
        settle(1);
        values(1);
        va ^= TILE;
        ++t;
    }
    for (; t < tiles; ++t) {  // tiles on the diagonal, each step by itself
        wait_loads_to_lds();
        __syncthreads();
        move_values(t + 1);
#pragma unroll 1
        for (int blk = 0; blk < 2; ++blk) {
            const int here = KT * t + 64 * part + 32 * blk;
            if (here >= some_see) break;
#pragma unroll
            for (int s = 0; s < S; ++s) sc[0][s] = f32x16{};
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const u32v4 f = key_frag(blk, c);
#pragma unroll
                for (int s = 0; s < S; ++s) sc[0][s] = mma32<T>(f, q[s][c], sc[0][s]);
            }
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int row = row_first + 32 * s + n, vis = row < n_rows ? row / a.group + 1 : len;
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (here + 8 * (r >> 2) + 4 * g + (r & 3) >= vis) sc[0][s][r] = kNone;
            }
#pragma unroll
            for (int s = 0; s < S; ++s) weigh(0, s, m[s]);
            settle(0);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int x = 2 * blk + h;
                uint32_t found = 0;
#pragma unroll
                for (int c = 0; c < DB; ++c) {
                    const u32v4 f = value_frag(x, c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) found |= maybe_not_finite<T>(f[e]);
                }
                const bool odd = __any(found != 0);
#pragma unroll
                for (int c = 0; c < DB; ++c) {
                    u32v4 f = value_frag(x, c);
                    if (odd) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) f[e] = finite_halves<T>(f[e]);
                    }
#pragma unroll
                    for (int s = 0; s < S; ++s) o[s][c] = mma32<T>(f, p[s][h], o[s][c]);
                }
                if (odd) {
                    // Values that are not finite, taken out above as a weight of zero does not hide them, are added to the rows
                    // that see them (times any weight above zero they stay what they are).
#pragma unroll 1
                    for (int i = 0; i < 16; ++i) {
                        const int r = 64 * part + 16 * x + i;  // of the tile
#pragma unroll
                        for (int c = 0; c < DB; ++c)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const u32x2 v = *(lds_u32x2 *)(lds0 + 2 * TILE + (t & 1) * TILE + r * ROW + (((4 * c + j) ^ key_of_v<DP>(r)) * 16) + 8 * g);
#pragma unroll
                                for (int s = 0; s < S; ++s) {
                                    const int row = row_first + 32 * s + n;
                                    const bool sees = row < n_rows && KT * t + r <= row / a.group;
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        const float y = odd_value<T>((e & 2 ? v.y : v.x) >> (16 * (e & 1)));
                                        o[s][c][4 * j + e] += sees ? y : 0.0f;
                                    }
                                }
                            }
                    }
                }
            }
        }
        __syncthreads();  // nobody reads these keys any more
        move_keys(t + 2);
        ka ^= TILE;
        va ^= TILE;
    }

#pragma unroll
    for (int s = 0; s < S; ++s) {
        l[s] += __shfl_xor(l[s], 32);
        lr[s] += __shfl_xor(lr[s], 32);
        m[s] = stored_shift(m[s], lr[s]);
    }
    if constexpr (PARTS == 2) {  // the wave of the same rows' other positions hands over through LDS
        constexpr int PAD = DP + 4;
        static_assert(WQ * S * 32 * (PAD + 4) * 4 <= sizeof lds, "the join fits the tiles' LDS");
        float *box = reinterpret_cast<float *>(lds) + (wave % WQ) * (S * 32 * PAD);
        float4 *ml = reinterpret_cast<float4 *>(reinterpret_cast<float *>(lds) + WQ * S * 32 * PAD) + S * 32 * (wave % WQ);
        __syncthreads();
        if (part == 1) {
#pragma unroll
            for (int s = 0; s < S; ++s) {
#pragma unroll
                for (int c = 0; c < DB; ++c)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        *reinterpret_cast<f32x4 *>(box + (32 * s + n) * PAD + 32 * c + 8 * r + 4 * g) =
                            f32x4{o[s][c][4 * r], o[s][c][4 * r + 1], o[s][c][4 * r + 2], o[s][c][4 * r + 3]};
                if (g == 0) ml[32 * s + n] = make_float4(m[s], l[s], lr[s], 0.0f);
            }
        }
        __syncthreads();
        if (part == 1) return;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const float4 x = ml[32 * s + n];
            const float up = fmaxf(m[s], x.x);
            const float f0 = m[s] == kNone ? 0.0f : __builtin_amdgcn_exp2f(m[s] - up), f1 = x.x == kNone ? 0.0f : __builtin_amdgcn_exp2f(x.x - up);
            m[s] = up;
            l[s] = l[s] * f0 + x.y * f1;
            lr[s] = lr[s] * f0 + x.z * f1;
#pragma unroll
            for (int c = 0; c < DB; ++c)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const f32x4 y = *reinterpret_cast<const f32x4 *>(box + (32 * s + n) * PAD + 32 * c + 8 * r + 4 * g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[s][c][4 * r + e] = o[s][c][4 * r + e] * f0 + y[e] * f1;
                }
        }
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int row = row_first + 32 * s + n, token = row / a.group, hq = head * a.group + row - token * a.group;
        if (row >= n_rows) continue;
        const float inv = 1.0f / lr[s];
        typedef T T4 __attribute__((ext_vector_type(4)));
        T *out = static_cast<T *>(a.out) + (int64_t)(t0 + token) * a.o_ts + (int64_t)hq * a.o_hs;
#pragma unroll
        for (int c = 0; c < DB; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = 32 * c + 8 * r + 4 * g;
                if (d < D)
                    *reinterpret_cast<T4 *>(out + d) = __builtin_convertvector(
                        (f32x4{o[s][c][4 * r], o[s][c][4 * r + 1], o[s][c][4 * r + 2], o[s][c][4 * r + 3]}) * inv, T4);
            }
        if (LSE && g == 0) a.lse[(int64_t)(t0 + token) * a.q_heads + hq] = (m[s] + __builtin_amdgcn_logf(l[s])) * 0.69314718055994531f;
    }
}

template <class T, class P>
static int run_prompt_shape(PromptArgs a, hipStream_t s) {
    a.slots = prompt_slot(a.n_tokens * a.group, a.n_seqs, P::ROWS);
    const int64_t wgs = (int64_t)a.slots * a.kv_heads;
    if (wgs > INT32_MAX) return (int)hipErrorInvalidValue;
    for (;; a.first_wg += kMaxWgs) {
        const int64_t left = wgs - a.first_wg;
        const unsigned grid = (unsigned)(left < kMaxWgs ? left : kMaxWgs);
        if (a.lse)
            prompt_kernel<T, P, true><<<grid, kAttnThreads, 0, s>>>(a);
        else
            prompt_kernel<T, P, false><<<grid, kAttnThreads, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || left <= kMaxWgs) return (int)e;
    }
}

template <class T, int DP>
static int run_prompt(const PromptArgs &a, bool many, hipStream_t s) {
    if constexpr (DP == 256)  // (the outputs of 32 rows fill the registers, two tiles of 64 positions the LDS)
        return run_prompt_shape<T, PromptShape<256, 1, 4>>(a, s);
    else
        return many ? run_prompt_shape<T, PromptShape<DP, 2, 4>>(a, s) : run_prompt_shape<T, PromptShape<DP, 2, 2>>(a, s);
}

}  // namespace bpw
