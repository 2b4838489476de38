// bpw_kv4_append.hip - append of keys and values to a paged cache held in 4 bits, keys normed and rotated on the way, and the
// queries of the same tokens beside them (gfx950, wave64). Launched only by bpw_requests_host.cpp after its checks.
//
// Mathematics. A block of 32 elements shares the smallest power of two 2^e, e in [-125, 125], with max |x| <= 7 2^e. An
// element becomes the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 times 2^e (code = the number of borders 0.25, 0.75, 1.25, 1.75,
// 2.5, 3.5, 5 below |x| 2^-e, a border itself going to the even code), which is off by at most 2^e. Which side of a border a
// key lies on is decided after norm and rotation; these are held in float64, as in float32 one element in some 10^6 would
// get the neighbouring code, a whole step away.
//
// Bound: HBM for prompts (8192 tokens of 32 + 8 + 8 heads of 128 in bfloat16, 210 MB read and written: 56-60 us over memory that no
// cache holds, 3.5-3.7 TB/s; three items are on their way beside the one worked on, with two 63 us, with four or five
// 58-60), while the vector units issue half of the time; the launch for a decode step (64
// tokens: 6 us). The wave's work is one head set's at a time, so that what differs between them is in
// scalar registers (93 us when lanes of a wave chose); sines and cosines are formed once for all heads of a token; a lane
// holds eight neighbours of a head, a block is four lanes, its largest element two DPP steps away, and its 32 codes four
// words of 32 bits, from the conversion instruction. Partners of a rotation go through LDS, 16 bytes of each lane beside
// the next lane's (eight numbers of a lane in a row: 65 us, bank conflicts).
#include "bpw_decode.h"
#include "bpw_elem.h"

namespace bpw {

constexpr int kAppendThreads = 256;
// Tokens from which a workgroup takes two of them, not one: its waves then have more to do between loads, but fewer workgroups
// share few tokens. Over memory that no cache holds, us with one and with two: 32 + 8 + 8 heads of 128 9.7, 11.8 at 1024 tokens, 14.1,
// 13.1 at 1536, 16.3, 16.9 at 2048, 31.5, 30.9 at 4096, 56.4, 56.3 at 8192 (four 56.4); 16 + 4 + 4 of 256 9.7, 11.8 at 1024, 16.8,
// 15.5 at 2048; 8 + 2 + 2 of 64 5.1, 5.7 at 1024, 8.8, 7.1 at 2048, 49.0, 36.7 at 16384 (four 28.8).
constexpr int32_t kAppendManyTokens = 2048;

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
// The elements times 2^-e as float32 for the conversion to codes, which rounds as the codes are defined (to the nearest, ties to the
// even one). Float32: the product, exact but far below the smallest code; zeros lose their sign. Float64: the upper 20 bits of the
// fraction and whether anything follows, which decides the same way, or the smallest normal number, code 0 too.
__device__ __forceinline__ float for_code(float x, uint32_t power) { return __builtin_fmaf(x, __builtin_bit_cast(float, (254u - power) << 23), 0.0f); }
__device__ __forceinline__ float for_code(double x, uint32_t power) {
    x += 0.0;
    const int32_t w = max((int32_t)size_word(x) - (((int32_t)power - 127) << 20), 897 << 20);
    const uint32_t sign = (uint32_t)(__builtin_bit_cast(uint64_t, x) >> 32) & 0x80000000u;
    return __builtin_bit_cast(float, (((uint32_t)w << 3) + 0x40000000u) | sign);  // (exponents of 1023 become those of 127)
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
    uint32_t codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0, for_code(x[0], power), for_code(x[1], power), 1.0f, 0);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, for_code(x[2], power), for_code(x[3], power), 1.0f, 1);
    codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, for_code(x[4], power), for_code(x[5], power), 1.0f, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, for_code(x[6], power), for_code(x[7], power), 1.0f, 3);
}
__device__ __forceinline__ f32x8 stands_for(uint32_t codes, uint32_t power) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const float unit = __builtin_bit_cast(float, power << 23);  // (255: the conversion gives NaN)
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, unit, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, unit, 1),
                c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, unit, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, unit, 3);
    return f32x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// 1 / sqrt(x), x > 0, to a step or two: the instruction's estimate and Newton's steps y (3 - x y^2) / 2.
__device__ __forceinline__ float inverse_root(float x) {
    const float y = __builtin_amdgcn_rsqf(x);
    return __builtin_fmaf(0.5f * y, __builtin_fmaf(-x * y, y, 1.0f), y);
}
__device__ __forceinline__ double inverse_root(double x) {
    double y = __builtin_amdgcn_rsq(x);
    y = __builtin_fma(0.5 * y, __builtin_fma(-x * y, y, 1.0), y);
    return __builtin_fma(0.5 * y, __builtin_fma(-x * y, y, 1.0), y);
}

__device__ __forceinline__ float fma_of(float a, float b, float c) { return __builtin_fmaf(a, b, c); }
__device__ __forceinline__ double fma_of(double a, double b, double c) { return __builtin_fma(a, b, c); }

template <class R>
__device__ __forceinline__ void norm(const Kv4AppendArgs &a, R (&x)[8], const f32x8 &gain) {
    R s = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fma_of(x[e], x[e], s);
    s = lanes_total(s, a.lanes_log2);
    const R v = s * (R)a.inv_head_dim + (R)a.eps;
    const R f = v > R(1e-30) && v < R(1e30) ? inverse_root(v) : R(1) / sqrt(v);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = x[e] * f * (R)gain[e];
}

// In LDS, 16 bytes hold four or two numbers, and a lane's eight are apart so that those of neighbouring lanes are neighbours: no
// two lanes of a read are in one bank (32 or 64 bytes a lane in a row took two and four times as long).
template <class R>
constexpr int kVec = 16 / (int)sizeof(R);
template <class R>
__device__ __forceinline__ int apart(int i, int chunks) {  // place of number i of `chunks` chunks of eight
    return ((i & 7) / kVec<R> * chunks + (i >> 3)) * kVec<R> + (i & (kVec<R> - 1));
}
template <class R>
__device__ __forceinline__ void read_chunk(const R *p, int chunk, int chunks, R (&x)[8]) {
    typedef R Vec __attribute__((ext_vector_type(kVec<R>)));
#pragma unroll
    for (int v = 0; v < 8 / kVec<R>; ++v) {
        const Vec y = reinterpret_cast<const Vec *>(p)[v * chunks + chunk];
#pragma unroll
        for (int e = 0; e < kVec<R>; ++e) x[v * kVec<R> + e] = y[e];
    }
}

// Rotation of the eight elements from i0 on of a head, whose cosines and sines are c and s. CHUNKS: pairs are whole chunks of eight
// apart, and c and s by chunks, or pairs are neighbours in one. row: the wave's 64 chunks; first: the chunk where the head begins.
template <class R, bool CHUNKS>
__device__ __forceinline__ void turn(const Kv4AppendArgs &a, R (&x)[8], int i0, const R *c, const R *s, R *row, int first) {
    const int half = a.rot_dim >> 1;
    if (CHUNKS && a.interleaved) {
        if (i0 >= a.rot_dim) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const R u = x[2 * e], v = x[2 * e + 1], cos = c[(i0 >> 1) + e], sin = s[(i0 >> 1) + e];
            x[2 * e] = fma_of(-v, sin, u * cos);
            x[2 * e + 1] = fma_of(u, sin, v * cos);
        }
        return;
    }
    typedef R Vec __attribute__((ext_vector_type(kVec<R>)));
#pragma unroll
    for (int v = 0; v < 8 / kVec<R>; ++v) {
        Vec y;
#pragma unroll
        for (int e = 0; e < kVec<R>; ++e) y[e] = x[v * kVec<R> + e];
        reinterpret_cast<Vec *>(row)[v * 64 + first + (i0 >> 3)] = y;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (i0 < a.rot_dim) {
        if constexpr (CHUNKS) {
            const bool lower = i0 < half;
            const int at = (lower ? i0 : i0 - half) >> 3;
            R cos[8], sin[8], other[8];
            read_chunk(row, first + ((lower ? i0 + half : i0 - half) >> 3), 64, other);
            read_chunk(c, at, half >> 3, cos);
            read_chunk(s, at, half >> 3, sin);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const R y = sin[e] * other[e];
                x[e] = fma_of(x[e], cos[e], lower ? -y : y);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = i0 + e;
                if (i >= a.rot_dim) break;
                const bool second = a.interleaved ? i & 1 : i >= half;
                const int at = a.interleaved ? i >> 1 : second ? i - half : i;
                const R y = s[at] * row[apart<R>(8 * first + (a.interleaved ? i ^ 1 : second ? at : i + half), 64)];
                x[e] = fma_of(x[e], c[at], second ? y : -y);
            }
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// A wave takes as many heads of one kind as it has lanes for (an item); the four waves of a workgroup take the items of TOKENS tokens
// in turn, the keys' first.
template <class TI, class TO, bool CHUNKS, int TOKENS>
__global__ __launch_bounds__(kAppendThreads, 4) void kv4_append_kernel(Kv4AppendArgs a) {
    extern __shared__ __attribute__((aligned(16))) double lds[];
    const int half = a.rot_dim >> 1, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    double *kc = lds, *ks = kc + TOKENS * half;  // cosines and sines of the tokens, for the keys
    float *qc = reinterpret_cast<float *>(ks + TOKENS * half), *qs = qc + TOKENS * half;  // and for the queries
    double *rows = static_cast<double *>(__builtin_assume_aligned(lds + 3 * TOKENS * half + (3 * TOKENS * half & 1) + 512 * wave, 16));
    const int64_t t0 = (a.first_wg + (int64_t)blockIdx.x) * TOKENS;
    const int lanes = 1 << a.lanes_log2, c = lane & (lanes - 1), i0 = 8 * c, place = lane >> a.lanes_log2, per = 64 >> a.lanes_log2;
    const bool in = i0 < a.head_dim;
    const int chunk0 = lanes * place;  // of the lane's head

    const int nk = (a.k.heads + per - 1) >> (6 - a.lanes_log2), nv = (a.v.heads + per - 1) >> (6 - a.lanes_log2);
    const int items = nk + nv + ((a.q.heads + per - 1) >> (6 - a.lanes_log2));
    const int tokens = (int)min((int64_t)TOKENS, a.n_tokens - t0);
    int token = 0, item = wave;  // of the next load
    const auto settle = [&] {
        while (item >= items) item -= items, ++token;
    };
    struct Item {
        Raw8<TI> raw;
        int64_t slot;
        int set, head, token;
    };
    const auto load = [&](Item &x) {
        x.set = item < nk ? 1 : item < nk + nv ? 2 : 0;
        x.token = token;
        const int64_t t = t0 + token;
        const HeadSet &s = x.set == 0 ? a.q : x.set == 1 ? a.k : a.v;
        const void *from = s.in;
        const int64_t ts = s.in_ts, hs = s.in_hs;
        const int heads = s.heads;
        x.head = (item - (x.set == 0 ? nk + nv : x.set == 1 ? 0 : nk)) * per + place;
        x.slot = a.slots[t];
        x.raw = eight(static_cast<const TI *>(from) + t * ts + min(x.head, heads - 1) * hs + (in ? i0 : 0), a.vec);
    };
    const auto gains = [&](const float *gain) {
        f32x8 x = {1, 1, 1, 1, 1, 1, 1, 1};
        typedef float f32x8u __attribute__((ext_vector_type(8), aligned(4)));
        if (gain) x = *reinterpret_cast<const f32x8u *>(gain + (in ? i0 : 0));
        return x;
    };
    constexpr int AHEAD = 3;
    Item next[AHEAD];
    const auto advance = [&](Item &x) {
        settle();
        x.token = -1;
        if (token < tokens) load(x);
        item += kAppendThreads / 64;
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) advance(next[i]);
    const f32x8 q_gain = gains(a.q.gain);
    for (int i = threadIdx.x; i < TOKENS * half; i += kAppendThreads) {
        const int u = TOKENS == 1 ? 0 : i / half;
        double x = (double)a.positions[min(t0 + u, (int64_t)a.n_tokens - 1)] * a.inv_freq[i - u * half] * 0.15915494309189533577;  // turns
        x -= __builtin_rint(x);
        const double cos = cospi(x + x), sin = sinpi(x + x);
        const bool by_chunk = CHUNKS && !a.interleaved;
        const int j = i - u * half, d = u * half + (by_chunk ? apart<double>(j, half >> 3) : j), f = u * half + (by_chunk ? apart<float>(j, half >> 3) : j);
        kc[d] = cos, ks[d] = sin;
        qc[f] = (float)cos, qs[f] = (float)sin;
    }
    __syncthreads();
    const auto work = [&](const Item &x) __attribute__((always_inline)) {
        const HeadSet &s = x.set == 0 ? a.q : x.set == 1 ? a.k : a.v;
        TO *out = static_cast<TO *>(s.out);
        const bool has_out = out, valid = in && x.head < s.heads;
        out += (t0 + x.token) * s.out_ts + x.head * s.out_hs + i0;
        uint32_t codes = 0, power = 0;
        if (x.set == 1) {
            double y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = in ? (double)(float)x.raw[e] : 0.0;
            if (a.k.gain) norm(a, y, gains(a.k.gain));
            if (half) turn<double, CHUNKS>(a, y, i0, kc + x.token * half, ks + x.token * half, rows, chunk0);
            codes = quantise(y, power);
        } else {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = in ? (float)x.raw[e] : 0.0f;
            if (x.set == 0) {
                if (a.q.gain) norm(a, y, q_gain);
                if (half) turn<float, CHUNKS>(a, y, i0, qc + x.token * half, qs + x.token * half, reinterpret_cast<float *>(rows), chunk0);
                if (valid) put_eight(out, f32x8{y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]}, a.vec);
                return;
            }
            codes = quantise(y, power);
        }
        if (!valid) return;
        if (x.slot >= 0 && x.slot < a.n_slots) {
            const Kv4Rows &r = x.set == 1 ? a.kc : a.vc;
            const int64_t page = x.slot >> a.page_log2, at = x.slot - (page << a.page_log2);
            *reinterpret_cast<uint32_t *>(r.codes + page * r.ps + at * r.rs + x.head * r.hs + 4 * c) = codes;
            if ((c & 3) == 0) r.scales[page * r.s_ps + at * r.s_rs + x.head * r.s_hs + (c >> 2)] = (uint8_t)power;
        }
        if (has_out) put_eight(out, stands_for(codes, power), a.vec);
    };
    while (true) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (next[i].token < 0) return;
            const Item x = next[i];
            advance(next[i]);
            work(x);
        }
    }
}

template <class TI, class TO, bool CHUNKS, int TOKENS>
static int run_append_as(Kv4AppendArgs a, hipStream_t s) {
    const size_t doubles = (size_t)3 * TOKENS * (a.rot_dim / 2);
    const size_t lds = (doubles + doubles % 2 + 512 * (kAppendThreads / 64)) * sizeof(double);
    const int32_t n = (a.n_tokens - 1) / TOKENS + 1;
    for (;; a.first_wg += kMaxWgs) {
        const int32_t left = n - a.first_wg;
        kv4_append_kernel<TI, TO, CHUNKS, TOKENS><<<(unsigned)(left < kMaxWgs ? left : kMaxWgs), kAppendThreads, lds, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || left <= kMaxWgs) return (int)e;
    }
}
template <class TI, class TO>
static int run_append(const Kv4AppendArgs &a, hipStream_t s) {
    if (a.rot_dim % (a.interleaved ? 8 : 16)) return run_append_as<TI, TO, false, 1>(a, s);
    return a.n_tokens >= kAppendManyTokens ? run_append_as<TI, TO, true, 2>(a, s) : run_append_as<TI, TO, true, 1>(a, s);
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
