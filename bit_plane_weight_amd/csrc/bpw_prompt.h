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

template <class T, int DP, int WQ>
__global__ __launch_bounds__(kAttnThreads, DP <= 128 ? 2 : 1) void prompt_kernel(PromptArgs a) {
    constexpr int ROW = DP * 2, CPR = DP / 8, RPI = 64 / CPR;  // row bytes, chunks of a row, rows of one load
    constexpr int KC = DP / 16, DB = DP / 32, M = 32 * WQ;
    constexpr int PARTS = kAttnWaves / WQ, NB = kPromptTile / 32 / PARTS;  // waves along a tile, blocks of 32 of each
    __shared__ WideLds<DP> lds;
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

    const int row_first = row0 + 32 * (wave % WQ), row = row_first + n;
    const int token = row / a.group, hq = head * a.group + row - token * a.group;
    const int vis = row < n_rows ? token + 1 : len;
    // what all and what some of the wave's rows see
    const int all_see = __builtin_amdgcn_readfirstlane(row_first / a.group + 1);
    const int some_see = row_first < n_rows ? (min(row_first + 32, n_rows) - 1) / a.group + 1 : 0;

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

    constexpr int LOADS = 16 / RPI, GROUP = LOADS < 4 ? LOADS : 4;  // loads of a wave's sixteen rows, of one asm block
    const uint32_t lds_k = (uint32_t)(size_t)(lds_u8 *)lds.k, lds_v = (uint32_t)(size_t)(lds_u8 *)lds.v;
    uint32_t ks[LOADS], vs[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int r = RPI * i + lane / CPR;
        ks[i] = 2 * (r * a.k_ts + 8 * ((lane % CPR) ^ key_of_k<DP>(r))) - 1024 * (i % GROUP);
        vs[i] = 2 * (r * a.v_ts + 8 * ((lane % CPR) ^ key_of_v<DP>(r))) - 1024 * (i % GROUP);
    }
    // Moves tile `pos` to LDS, this wave's 16 positions of it. Positions past the sequence and elements past head_dim become
    // zeros (a zero weight times whatever memory holds there would not be one).
    const auto issue = [&](int buf, int pos) {
        const int first = pos + 16 * wave;
        const T *kp = kbase + (int64_t)first * a.k_ts, *vp = vbase + (int64_t)first * a.v_ts;
        const uint32_t at = buf * (kPromptTile * ROW) + 16 * wave * ROW;
        if (pos + kPromptTile <= len && D == DP) {
#pragma unroll
            for (int i = 0; i < LOADS; i += GROUP) {
                load_to_lds<GROUP>(lds_k + at + 1024 * i, kp, reinterpret_cast<const uint32_t(&)[GROUP]>(ks[i]));
                load_to_lds<GROUP>(lds_v + at + 1024 * i, vp, reinterpret_cast<const uint32_t(&)[GROUP]>(vs[i]));
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int r = RPI * i + lane / CPR;  // of the wave's sixteen
            const bool in = first + r < len;
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

    int pos0 = 0;
    issue(0, 0);
    // Tile `pos0`, which lies in LDS buffer `buf`.
    const auto tile = [&](auto which) {
        constexpr int buf = decltype(which)::value;
        wait_loads_to_lds();
        __syncthreads();  // this tile is there, and nobody reads the one before it any more
        if (pos0 + kPromptTile < end) issue(buf ^ 1, pos0 + kPromptTile);
        const int here = pos0 + 32 * part * NB;  // this wave's first position
        pos0 += kPromptTile;
        if (here >= some_see) return;
        const bool hidden = here + 32 * NB > all_see;

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
        const auto scores = [&](int blk) {
            sc[blk] = f32x16{};
#pragma unroll
            for (int x = blk * NGB; x < (blk + 1) * NGB; ++x) {
                if (x + 1 < NG) read_k(x + 1);
#pragma unroll
                for (int c = 0; c < GK; ++c) sc[blk] = mma32<T>(kf[x & 1][c], q[(x * GK + c) % KC], sc[blk]);
            }
        };
        // Values that only some rows see and that are not finite: one token at a time, the last first, with the values
        // that it does not see set to zero; only its rows take the result.
        const auto values_by_token = [&](int x, u32v4 w) {
            for (int t = (min(row_first + 32, n_rows) - 1) / a.group; t >= row_first / a.group; --t) {
#pragma unroll
                for (int c = 0; c < DB; ++c) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int at = here + 16 * x + 8 * (e >> 1) + 4 * g + 2 * (e & 1);
                        if (at > t) vf[x & 1][c][e] &= 0xFFFF0000u;
                        if (at + 1 > t) vf[x & 1][c][e] &= 0x0000FFFFu;
                    }
                    const f32x16 y = mma32<T>(vf[x & 1][c], w, o[c]);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[c][e] = token == t ? y[e] : o[c][e];
                }
            }
        };
        const auto values = [&](int blk) {
#pragma unroll
            for (int x = 2 * blk; x < 2 * blk + 2; ++x) {
                if (x + 1 < 2 * NB) read_v(x + 1);
                if (hidden) {
                    uint32_t found = 0;
#pragma unroll
                    for (int c = 0; c < DB; ++c)
#pragma unroll
                        for (int e = 0; e < 4; ++e) found |= maybe_not_finite<T>(vf[x & 1][c][e]);
                    if (__any(found != 0)) {
                        values_by_token(x, p[blk][x & 1]);
                        continue;
                    }
                }
#pragma unroll
                for (int c = 0; c < DB; ++c) o[c] = mma32<T>(vf[x & 1][c], p[blk][x & 1], o[c]);
            }
        };
        f32x8 w[2];
        float sum;
        const auto hide = [&](int blk) {
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (here + 32 * blk + 8 * (r >> 2) + 4 * g + (r & 3) >= vis) sc[blk][r] = kNone;
        };
        const auto weigh = [&](int blk, float shift) {
            float part_sum[2] = {0.0f, 0.0f};
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[blk][r], a.scale_log2, -shift));
                w[r >> 3][r & 7] = e;
                part_sum[r >> 3] += e;
            }
            sum = part_sum[0] + part_sum[1];
        };
        // The shift raised where a lane's sum passes the limit (as in attend()), the weights in 16 bits: half a step of relative
        // error each; o is divided by the sum of the rounded weights, so that errors they share cancel.
        const auto settle = [&](int blk) {
            if (__any(!(sum < kShiftLimit<T>))) {
                float top = kNone;
#pragma unroll
                for (int r = 0; r < 16; ++r) top = fmaxf(top, sc[blk][r]);
                top = fmaxf(top, __shfl_xor(top, 32)) * a.scale_log2;
                const float up = fmaxf(m, top - kLift<T>);
                const float f = up == m ? 1.0f : __builtin_amdgcn_exp2f(m - up);
                m = up;
                l *= f;
                lr *= f;
#pragma unroll
                for (int c = 0; c < DB; ++c) o[c] *= f;
                weigh(blk, up == kNone ? 0.0f : up);
            }
            l += sum;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                p[blk][h] = __builtin_bit_cast(u32v4, __builtin_convertvector(w[h], typename Vec8<T>::type));
                lr = sum8<T>(p[blk][h], lr);
            }
        };
        read_k(0);
        scores(0);
        read_v(0);
        __builtin_amdgcn_sched_barrier(0);
        if (hidden) hide(0);
        weigh(0, m);
        if constexpr (NB == 2) scores(1);
        settle(0);
        if constexpr (NB == 2) {
            if (hidden) hide(1);
            values(0);
            weigh(1, m);
            settle(1);
        }
        values(NB - 1);
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
        if (part == 1) return;
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
    if (a.lse && g == 0) a.lse[(int64_t)(t0 + token) * a.q_heads + hq] = (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
}

template <class T, int DP>
static int run_prompt(PromptArgs a, int32_t rows, hipStream_t s) {
    const int64_t wgs = (int64_t)a.slots * a.kv_heads;
    if (wgs > INT32_MAX) return (int)hipErrorInvalidValue;
    for (;; a.first_wg += kMaxWgs) {
        const int64_t left = wgs - a.first_wg;
        const unsigned grid = (unsigned)(left < kMaxWgs ? left : kMaxWgs);
        if (rows == 64)
            prompt_kernel<T, DP, 2><<<grid, kAttnThreads, 0, s>>>(a);
        else
            prompt_kernel<T, DP, 4><<<grid, kAttnThreads, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || left <= kMaxWgs) return (int)e;
    }
}

}  // namespace bpw
