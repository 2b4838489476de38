// bpw_heads.hip - RMS norm and position rotation of query and key heads, and the append of keys and
// values to a paged cache, in one pass over the heads (gfx950, wave64). Launched only by
// bpw_decode_host.cpp after its checks.
//
// Mathematics. n = x * rsqrt(mean(x^2) + eps) * gain in float32; a pair (a, b) of frequency i becomes
// (a cos - b sin, b cos + a sin). The angle is formed as turns = position * inv_freq / 2 pi in float64
// and reduced to [-1/2, 1/2] there, because in float32 the angle of position 131072 at frequency 1
// is already wrong in its third decimal; sine and cosine of the reduced turn are float32.
//
// Bound: HBM for prompts (each element read once and written once: 16384 tokens of 40 heads of 128 in bf16, 336 MB,
// 66.3 us = 5.06 TB/s, where a copy of as many bytes with non-temporal loads and stores reaches 6.33), the launch for a
// decode step (one token 2.8 us). A
// workgroup takes whole tokens, so that the rot_dim / 2 sines and cosines are formed once per token
// (by as many threads) and shared by its heads through LDS. In the vector path 2^lanes_log2 lanes hold one
// head, each both partners of its pairs (8 elements of the first half and the 8 opposite ones, or 16
// neighbours), so the rotation needs no exchange and the norm one sum over the lanes; pairs that are not whole chunks
// exchange through LDS (mixed path).
#include "bpw_decode.h"
#include "bpw_elem.h"

namespace bpw {

// Sum over the 2^n consecutive lanes of a head: every lane gets it. Within 16 lanes by DPP (swap pairs,
// swap halves of a quad, mirror within 8, mirror within 16).
__device__ __forceinline__ float lanes_sum(float s, int n) {
#define BPW_DPP_ADD(ctrl) \
    s += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, s), ctrl, 0xF, 0xF, false))
    if (n >= 1) BPW_DPP_ADD(0xB1);
    if (n >= 2) BPW_DPP_ADD(0x4E);
    if (n >= 3) BPW_DPP_ADD(0x141);
    if (n >= 4) BPW_DPP_ADD(0x140);
#undef BPW_DPP_ADD
    if (n >= 5) s += __shfl_xor(s, 16);
    if (n >= 6) s += __shfl_xor(s, 32);
    return s;
}

// Cosine and sine of position * inv_freq.
__device__ __forceinline__ float2 turn(int32_t position, double inv_freq) {
    double t = (double)position * inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
    t -= __builtin_rint(t);
    const float x = (float)(t + t);
    return make_float2(cospif(x), sinpif(x));
}

// cs[t][i] for the workgroup's tokens.
__device__ __forceinline__ void fill_turns(const HeadsArgs &a, int t0, int nt, float2 *cs) {
    const int nf = a.rot_dim >> 1;
    for (int i = threadIdx.x; i < nt * nf; i += kHeadThreads) {
        const int t = i / nf;
        cs[i] = turn(a.positions[t0 + t], a.inv_freq[i - t * nf]);
    }
}

// One head of one token: where it is read and written. set 0: q, 1: k, 2: v.
template <class TI, class TO>
struct HeadRow {
    const TI *in;
    TO *out;
    const float *gain;
    int set;
    bool store;
};

template <class TI, class TO>
__device__ __forceinline__ HeadRow<TI, TO> head_row(const HeadsArgs &a, int64_t t, int h) {
    HeadRow<TI, TO> r;
    r.set = h < a.q.heads ? 0 : h < a.q.heads + a.k.heads ? 1 : 2;
    const HeadSet &s = r.set == 0 ? a.q : r.set == 1 ? a.k : a.v;
    h -= r.set == 0 ? 0 : r.set == 1 ? a.q.heads : a.q.heads + a.k.heads;
    r.in = static_cast<const TI *>(s.in) + t * s.in_ts + h * s.in_hs;
    r.gain = s.gain;
    r.store = true;
    int64_t off;
    if (s.to_cache) {
        const int64_t slot = a.slots[t];
        r.store = slot >= 0 && slot < a.n_slots;
        const int64_t page = slot >> a.page_log2;
        off = page * s.out_ps + (slot - (page << a.page_log2)) * s.out_ts;
    } else {
        off = t * s.out_ts;
    }
    r.out = static_cast<TO *>(s.out) + off + h * s.out_hs;
    return r;
}

// LDS of heads_mixed_kernel: the turns (an even number of them, so that rows are 16-byte aligned), then a padded row for
// each head that a workgroup holds at once.
__device__ __host__ __forceinline__ int mixed_turns(const HeadsArgs &a) { return (a.tokens_per_wg * (a.rot_dim >> 1) + 1) & ~1; }
__device__ __host__ __forceinline__ int mixed_pitch(const HeadsArgs &a) { return a.head_dim + 4; }

template <class TI, class TO>
__global__ __launch_bounds__(kHeadThreads) void heads_vec_kernel(HeadsArgs a) {
    extern __shared__ float2 cs[];
    const int heads = a.q.heads + a.k.heads + a.v.heads;
    const int t0 = (a.first_wg + (int)blockIdx.x) * a.tokens_per_wg;
    const int nt = min(a.tokens_per_wg, a.n_tokens - t0);
    const int c = threadIdx.x & ((1 << a.lanes_log2) - 1);
    const int step = kHeadThreads >> a.lanes_log2, total = nt * heads;
    const bool in = 16 * c < a.head_dim;
    const bool turned = 16 * c < a.rot_dim;
    // this lane's two chunks of eight elements
    const int half = a.rot_dim >> 1;
    const int i0 = !in ? 0 : turned && !a.interleaved ? 8 * c : 16 * c;
    const int i1 = !in ? 0 : turned && !a.interleaved ? half + 8 * c : i0 + 8;

    int u = threadIdx.x >> a.lanes_log2;
    HeadRow<TI, TO> r;
    Raw8<TI> n0, n1;
    int t = 0;
    const auto fetch = [&] {
        t = u / heads;
        r = head_row<TI, TO>(a, t0 + t, u - t * heads);
        n0 = raw8(r.in + i0);
        n1 = raw8(r.in + i1);
    };
    if (u < total) fetch();  // the first head's loads leave before the angles are formed
    fill_turns(a, t0, nt, cs);
    __syncthreads();
    while (u < total) {
        f32x8 x0 = as_f32(n0), x1 = as_f32(n1);
        if (r.gain) {
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s = __builtin_fmaf(x0[e], x0[e], __builtin_fmaf(x1[e], x1[e], s));
            s = lanes_sum(in ? s : 0.0f, a.lanes_log2);
            const float f = rsqrtf(s / (float)a.head_dim + a.eps);
            x0 = x0 * f * load8(r.gain + i0);
            x1 = x1 * f * load8(r.gain + i1);
        }
        if (turned && r.set != 2) {
            const f32x4 *w = reinterpret_cast<const f32x4 *>(cs + t * half + 8 * c);
            float co[8], si[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x4 p = w[e];
                co[2 * e] = p.x, si[2 * e] = p.y, co[2 * e + 1] = p.z, si[2 * e + 1] = p.w;
            }
            f32x8 y0, y1;
            if (!a.interleaved) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    y0[e] = x0[e] * co[e] - x1[e] * si[e];
                    y1[e] = x1[e] * co[e] + x0[e] * si[e];
                }
            } else {
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    y0[2 * p] = x0[2 * p] * co[p] - x0[2 * p + 1] * si[p];
                    y0[2 * p + 1] = x0[2 * p + 1] * co[p] + x0[2 * p] * si[p];
                    y1[2 * p] = x1[2 * p] * co[4 + p] - x1[2 * p + 1] * si[4 + p];
                    y1[2 * p + 1] = x1[2 * p + 1] * co[4 + p] + x1[2 * p] * si[4 + p];
                }
            }
            x0 = y0;
            x1 = y1;
        }
        if (in && r.store) {
            store8(r.out + i0, x0);
            store8(r.out + i1, x1);
        }
        u += step;
        if (u < total) fetch();
    }
}

// Rotations whose halves are not whole chunks (rot_dim not a multiple of 16), head_dim a multiple of 8: a lane takes eight
// neighbours of a head, and the pairs' partners are read back from the normed row in LDS, which the lanes of a head (of
// one wave, so no barrier) have just written there. 8192 tokens of 32 + 8 heads of 128 in bf16 with 66 turned: 48 us,
// 3.5 TB/s, where pairs of whole chunks take 34.
template <class TI, class TO>
__global__ __launch_bounds__(kHeadThreads) void heads_mixed_kernel(HeadsArgs a) {
    extern __shared__ float2 cs[];
    const int heads = a.q.heads + a.k.heads + a.v.heads, half = a.rot_dim >> 1;
    const int t0 = (a.first_wg + (int)blockIdx.x) * a.tokens_per_wg;
    const int nt = min(a.tokens_per_wg, a.n_tokens - t0);
    const int c = threadIdx.x & ((1 << a.lanes_log2) - 1), i0 = 8 * c;
    const int step = kHeadThreads >> a.lanes_log2, total = nt * heads;
    const bool in = i0 < a.head_dim;
    float *row = reinterpret_cast<float *>(cs + mixed_turns(a)) + (threadIdx.x >> a.lanes_log2) * mixed_pitch(a);
    fill_turns(a, t0, nt, cs);
    __syncthreads();
    for (int u = threadIdx.x >> a.lanes_log2; u < total; u += step) {
        const int t = u / heads;
        const HeadRow<TI, TO> r = head_row<TI, TO>(a, t0 + t, u - t * heads);
        f32x8 x = load8(r.in + (in ? i0 : 0));
        if (r.gain) {
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s = __builtin_fmaf(x[e], x[e], s);
            s = lanes_sum(in ? s : 0.0f, a.lanes_log2);
            x = x * rsqrtf(s / (float)a.head_dim + a.eps) * load8(r.gain + (in ? i0 : 0));
        }
        if (in && i0 < a.rot_dim && r.set != 2) {
            *reinterpret_cast<f32x4 *>(row + i0) = __builtin_shufflevector(x, x, 0, 1, 2, 3);
            *reinterpret_cast<f32x4 *>(row + i0 + 4) = __builtin_shufflevector(x, x, 4, 5, 6, 7);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = i0 + e;
                if (i >= a.rot_dim) break;
                const bool second = a.interleaved ? i & 1 : i >= half;
                const int f = a.interleaved ? i >> 1 : second ? i - half : i;
                const float y = row[a.interleaved ? i ^ 1 : second ? i - half : i + half];
                const float2 w = cs[t * half + f];
                x[e] = x[e] * w.x + (second ? y * w.y : -(y * w.y));
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
        if (in && r.store) store8(r.out + i0, x);
    }
}

// Any even head_dim, rot_dim, stride and alignment: a lane takes pairs of elements one at a time (1.2 TB/s).
template <class TI, class TO>
__global__ __launch_bounds__(kHeadThreads) void heads_any_kernel(HeadsArgs a) {
    extern __shared__ float2 cs[];
    const int heads = a.q.heads + a.k.heads + a.v.heads;
    const int t0 = (a.first_wg + (int)blockIdx.x) * a.tokens_per_wg;
    const int nt = min(a.tokens_per_wg, a.n_tokens - t0);
    const int lanes = 1 << a.lanes_log2, c = threadIdx.x & (lanes - 1);
    const int step = kHeadThreads >> a.lanes_log2, total = nt * heads, pairs = a.head_dim >> 1, half = a.rot_dim >> 1;
    fill_turns(a, t0, nt, cs);
    __syncthreads();
    for (int u = threadIdx.x >> a.lanes_log2; u < total; u += step) {
        const int t = u / heads;
        const HeadRow<TI, TO> r = head_row<TI, TO>(a, t0 + t, u - t * heads);
        float f = 1.0f;
        if (r.gain) {
            float s = 0.0f;
            for (int p = c; p < pairs; p += lanes) {
                const float x = (float)r.in[2 * p], y = (float)r.in[2 * p + 1];
                s = __builtin_fmaf(x, x, __builtin_fmaf(y, y, s));
            }
            f = rsqrtf(lanes_sum(s, a.lanes_log2) / (float)a.head_dim + a.eps);
        }
        for (int p = c; p < pairs; p += lanes) {
            const bool split = p < half && !a.interleaved;
            const int i0 = split ? p : 2 * p, i1 = split ? p + half : 2 * p + 1;
            float x = (float)r.in[i0], y = (float)r.in[i1];
            if (r.gain) {
                x = x * f * r.gain[i0];
                y = y * f * r.gain[i1];
            }
            if (p < half && r.set != 2) {
                const float2 w = cs[t * half + p];
                const float z = x * w.x - y * w.y;
                y = y * w.x + x * w.y;
                x = z;
            }
            if (r.store) {
                r.out[i0] = (TO)x;
                r.out[i1] = (TO)y;
            }
        }
    }
}

template <class TI, class TO>
static int launch_typed(HeadsArgs a, int32_t path, hipStream_t s) {
    const int32_t wgs = (a.n_tokens - 1) / a.tokens_per_wg + 1;
    const size_t turns = (size_t)a.tokens_per_wg * (size_t)(a.rot_dim / 2) * sizeof(float2);
    const size_t mixed = (size_t)mixed_turns(a) * sizeof(float2) + (size_t)(kHeadThreads >> a.lanes_log2) * mixed_pitch(a) * sizeof(float);
    for (; a.first_wg < wgs; a.first_wg += kMaxWgs) {
        const unsigned grid = (unsigned)(wgs - a.first_wg < kMaxWgs ? wgs - a.first_wg : kMaxWgs);
        if (path == kHeadsVec)
            heads_vec_kernel<TI, TO><<<grid, kHeadThreads, turns, s>>>(a);
        else if (path == kHeadsMixed)
            heads_mixed_kernel<TI, TO><<<grid, kHeadThreads, mixed, s>>>(a);
        else
            heads_any_kernel<TI, TO><<<grid, kHeadThreads, turns, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return (int)e;
        if (wgs - a.first_wg <= kMaxWgs) break;  // (before first_wg can pass 2^31)
    }
    return (int)hipSuccess;
}

template <class TI>
static int launch_from(const HeadsArgs &a, int32_t dt_out, int32_t path, hipStream_t s) {
    if (dt_out == 0) return launch_typed<TI, float>(a, path, s);
    if (dt_out == 1) return launch_typed<TI, __bf16>(a, path, s);
    return launch_typed<TI, _Float16>(a, path, s);
}

int launch_heads(const HeadsArgs &a, int32_t dt_in, int32_t dt_out, int32_t path, void *stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dt_in == 0) return launch_from<float>(a, dt_out, path, s);
    if (dt_in == 1) return launch_from<__bf16>(a, dt_out, path, s);
    return launch_from<_Float16>(a, dt_out, path, s);
}

}  // namespace bpw
