// bpw_kv4_append.hip - append of keys and values to a paged cache held in 4 bits, keys normed and rotated on the way, and the
// queries of the same tokens beside them (gfx950, wave64). Launched only by bpw_requests_host.cpp after its checks.
//
// Mathematics. A block of 32 elements shares the smallest power of two 2^e, e in [-125, 125], with max |x| <= 7 2^e. An
// element becomes the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 times 2^e (code = the number of borders 0.25, 0.75, 1.25, 1.75,
// 2.5, 3.5, 5 below |x| 2^-e, a border itself going to the even code), which is off by at most 2^e. Which side of a border a
// key lies on is decided after norm and rotation; these are held in float64, as in float32 one element in some 10^6 would
// get the neighbouring code, a whole step away.
//
// Bound: HBM for prompts, the launch for a decode step. A workgroup takes a token: sines and cosines are
// formed once for all of its heads; a lane holds eight neighbours of a head, a block is four lanes, its largest element two
// DPP steps away, and its 32 codes four words of 32 bits. Partners of a rotation are read from the normed row in LDS,
// which the lanes of a head (of one wave) have just written there.
#include "bpw_decode.h"
#include "bpw_elem.h"

namespace bpw {

constexpr int kAppendThreads = 256;

template <class R>
__device__ __forceinline__ R lanes_total(R s, int n) {  // over the 2^n consecutive lanes of a head
    if (n >= 1) s += dpp<0xB1>(s);
    if (n >= 2) s += dpp<0x4E>(s);
    if (n >= 3) s += dpp<0x141>(s);
    if (n >= 4) s += dpp<0x140>(s);
    if (n >= 5) s += __shfl_xor(s, 16);
    return s;
}

template <class T>
__device__ __forceinline__ Raw8<T> eight(const T *p, bool vec) {
    if (vec) return raw8(p);
    Raw8<T> x;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = p[e];
    return x;
}
template <class T>
__device__ __forceinline__ void put_eight(T *p, f32x8 x, bool vec) {
    if (vec) {
        store8(p, x);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = (T)x[e];
}

// The word of an element's magnitude that a block's power of two is found from: float32's bits; float64's upper half, its
// last bit set where the lower half is not zero. Larger magnitudes have no smaller words, NaN the largest.
__device__ __forceinline__ uint32_t size_word(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t size_word(double x) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    return ((uint32_t)(b >> 32) & 0x7FFFFFFFu) | ((uint32_t)b != 0 ? 1u : 0u);
}
// Power byte of a block whose largest size word is w: the exponent field's value less 2, one more above 1.75 times it.
__device__ __forceinline__ uint32_t power_byte(uint32_t w, float) {
    const int field = (int)(w >> 23), e = field - 127 - 2 + ((w & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return field == 255 ? 255u : (uint32_t)(min(max(e, -125), 125) + 127);
}
__device__ __forceinline__ uint32_t power_byte(uint32_t w, double) {
    const int field = (int)(w >> 20), e = field - 1023 - 2 + ((w & 0xFFFFFu) > 0xC0000u ? 1 : 0);
    return field == 2047 ? 255u : (uint32_t)(min(max(e, -125), 125) + 127);
}
__device__ __forceinline__ float unit_of(uint32_t byte, float) { return __builtin_bit_cast(float, (254u - byte) << 23); }
__device__ __forceinline__ double unit_of(uint32_t byte, double) {
    return __builtin_bit_cast(double, (uint64_t)(1023 + 127 - (int)byte) << 52);
}

// Eight neighbours of a row: their codes, low half byte first; `power` gets the byte of their block, which four lanes share.
template <class R>
__device__ __forceinline__ uint32_t quantise(const R (&x)[8], uint32_t &power) {
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) w = max(w, size_word(x[e]));
    w = max(w, (uint32_t)dpp<0xB1>((int)w));
    w = max(w, (uint32_t)dpp<0x4E>((int)w));
    power = power_byte(w, R());
    if (power == 255) return 0;
    const R up = unit_of(power, R());
    uint32_t codes = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const R a = (x[e] < 0 ? -x[e] : x[e]) * up;
        const uint32_t c = (a > R(0.25)) + (a >= R(0.75)) + (a > R(1.25)) + (a >= R(1.75)) + (a > R(2.5)) + (a >= R(3.5)) + (a > R(5));
        codes |= (c | (x[e] < 0 ? 8u : 0u)) << (4 * e);
    }
    return codes;
}
__device__ __forceinline__ f32x8 stands_for(uint32_t codes, uint32_t power) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const float unit = __builtin_bit_cast(float, power << 23);  // (255: the conversion gives NaN)
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, unit, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, unit, 1),
                c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, unit, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, unit, 3);
    return f32x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// LDS: the turns (cosine, sine) of a token, then a padded row for each head that a workgroup holds at once.
__device__ __host__ __forceinline__ int append_pitch(int head_dim) { return head_dim + 2; }

// Norm and rotation of the eight elements from i0 on of a head, in R.
template <class R>
__device__ __forceinline__ void norm_turn(const Kv4AppendArgs &a, R (&x)[8], int i0, bool in, const float *gain, const double2 *turns, R *row) {
    if (gain) {
        R s = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) s += x[e] * x[e];
        s = lanes_total(in ? s : R(0), a.lanes_log2);
        const R f = R(1) / sqrt(s / (R)a.head_dim + (R)a.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * f * (R)gain[(in ? i0 : 0) + e];
    }
    if (!a.rot_dim) return;
    const int half = a.rot_dim >> 1;
    if (in && i0 < a.rot_dim) {
#pragma unroll
        for (int e = 0; e < 8; ++e) row[i0 + e] = x[e];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (in && i0 < a.rot_dim) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = i0 + e;
            if (i >= a.rot_dim) break;
            const bool second = a.interleaved ? i & 1 : i >= half;
            const double2 w = turns[a.interleaved ? i >> 1 : second ? i - half : i];
            const R y = row[a.interleaved ? i ^ 1 : second ? i - half : i + half];
            x[e] = x[e] * (R)w.x + (second ? y * (R)w.y : -(y * (R)w.y));
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <class TI, class TO>
__global__ __launch_bounds__(kAppendThreads) void kv4_append_kernel(Kv4AppendArgs a) {
    extern __shared__ double2 turns[];
    const int64_t t = a.first_wg + (int64_t)blockIdx.x;
    const int half = a.rot_dim >> 1, heads = a.q.heads + a.k.heads + a.v.heads;
    for (int i = threadIdx.x; i < half; i += kAppendThreads) {
        double x = (double)a.positions[t] * a.inv_freq[i] * 0.15915494309189533577;  // turns
        x -= __builtin_rint(x);
        turns[i] = make_double2(cospi(x + x), sinpi(x + x));
    }
    __syncthreads();
    const int group = threadIdx.x >> a.lanes_log2, c = threadIdx.x & ((1 << a.lanes_log2) - 1), i0 = 8 * c;
    const bool in = i0 < a.head_dim;
    double *row = reinterpret_cast<double *>(turns + half) + group * append_pitch(a.head_dim);
    const int64_t slot = a.slots[t];
    const bool stored = slot >= 0 && slot < a.n_slots;
    const int64_t page = slot >> a.page_log2, at = slot - (page << a.page_log2);
    for (int h = group; h < heads; h += kAppendThreads >> a.lanes_log2) {
        const int set = h < a.q.heads ? 0 : h < a.q.heads + a.k.heads ? 1 : 2;
        const HeadSet &s = set == 0 ? a.q : set == 1 ? a.k : a.v;
        const int head = h - (set == 0 ? 0 : set == 1 ? a.q.heads : a.q.heads + a.k.heads);
        const TI *p = static_cast<const TI *>(s.in) + t * s.in_ts + head * s.in_hs + (in ? i0 : 0);
        const Raw8<TI> raw = eight(p, a.vec);
        TO *out = s.out ? static_cast<TO *>(s.out) + t * s.out_ts + head * s.out_hs + i0 : nullptr;
        uint32_t codes = 0, power = 0;
        if (set == 1) {
            double x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = in ? (double)(float)raw[e] : 0.0;
            norm_turn(a, x, i0, in, s.gain, turns, row);
            codes = quantise(x, power);
        } else {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = in ? (float)raw[e] : 0.0f;
            if (set == 0) {
                norm_turn(a, x, i0, in, s.gain, turns, reinterpret_cast<float *>(row));
                if (in) put_eight(out, f32x8{x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]}, a.vec);
                continue;
            }
            codes = quantise(x, power);
        }
        if (!in) continue;
        if (stored) {
            const Kv4Rows &r = set == 1 ? a.kc : a.vc;
            *reinterpret_cast<uint32_t *>(r.codes + page * r.ps + head * r.hs + at * r.rs + 4 * c) = codes;
            if ((c & 3) == 0) r.scales[page * r.s_ps + head * r.s_hs + at * r.s_rs + (c >> 2)] = (uint8_t)power;
        }
        if (out) put_eight(out, stands_for(codes, power), a.vec);
    }
}

template <class TI, class TO>
static int run_append(Kv4AppendArgs a, hipStream_t s) {
    const size_t lds = (size_t)(a.rot_dim / 2) * sizeof(double2) + (size_t)(kAppendThreads >> a.lanes_log2) * append_pitch(a.head_dim) * sizeof(double);
    const int32_t n = a.n_tokens;
    for (;; a.first_wg += kMaxWgs) {
        const int32_t left = n - a.first_wg;
        kv4_append_kernel<TI, TO><<<(unsigned)(left < kMaxWgs ? left : kMaxWgs), kAppendThreads, lds, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || left <= kMaxWgs) return (int)e;
    }
}

template <class TI>
static int run_append_from(const Kv4AppendArgs &a, int32_t dt_out, hipStream_t s) {
    return dt_out == 1 ? run_append<TI, __bf16>(a, s) : run_append<TI, _Float16>(a, s);
}

int launch_kv4_append(const Kv4AppendArgs &a, int32_t dt_in, int32_t dt_out, void *stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dt_in == 0) return run_append_from<float>(a, dt_out, s);
    if (dt_in == 1) return run_append_from<__bf16>(a, dt_out, s);
    return run_append_from<_Float16>(a, dt_out, s);
}

}  // namespace bpw
