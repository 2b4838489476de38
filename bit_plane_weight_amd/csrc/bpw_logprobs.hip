// bpw_logprobs.hip - log probabilities of given tokens, entropy and top alternatives of rows of logits (gfx950, wave64).
// Launched only by bpw_requests_host.cpp after its checks.
//
// Mathematics. With M the largest logit of a row, d_v = scale (x_v - M), l = sum exp(d_v) and t = sum d_v exp(d_v):
//   log p_v = d_v - log l,   H = -sum p_v log p_v = log l - t / l,
// both terms of H positive, so that a nearly certain row loses nothing. Partial sums against a shift m join by
// l' = f l, t' = f (t + d l) with d = scale (m - M), f = exp(d). The shift of a lane is raised only when a logit passes it by
// 2^16 in weight, so most rounds form no maximum against the running one.
//
// Bound: HBM, each logit read once. A wave takes 512 neighbours at a time, eight a lane, one round ahead of their use. The
// best n entries are kept by each wave: a list of 64 places in LDS to which lanes add what exceeds the wave's
// n-th best; a full list is ranked (each lane counts the keys above its own) and cut to n. The first
// round's n-th largest of the 64 lanes' maxima is a first bar, so that little is added: n log(entries / n) in expectation.
// Few rows are cut into parts, one workgroup each, joined by a second launch.
#include "bpw_decode.h"
#include "bpw_elem.h"

namespace bpw {

constexpr int kWavesLp = kLogprobThreads / 64;
constexpr float kLowest = -3.4028234663852886e38f;
constexpr float kMinusInf = -__builtin_inff();
constexpr float kLazy = 16.0f;  // log2 units that a logit may lie above the shift
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;

// Larger logit first, then lower index: keys fall in that order. Zeros of both signs are one.
__device__ __forceinline__ uint64_t key_of(float x, int32_t i) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
    return ((uint64_t)(b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u)) << 32) | (0xFFFFFFFFu - (uint32_t)i);
}
__device__ __forceinline__ float logit_of(uint64_t key) {
    const uint32_t b = (uint32_t)(key >> 32);
    return __builtin_bit_cast(float, b & 0x80000000u ? b ^ 0x80000000u : ~b);
}
__device__ __forceinline__ int32_t index_of(uint64_t key) { return (int32_t)(0xFFFFFFFFu - (uint32_t)key); }
__device__ __forceinline__ uint64_t read_lane(uint64_t x, int l) {
    return ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((uint32_t)(x >> 32), l) << 32) |
           (uint32_t)__builtin_amdgcn_readlane((uint32_t)x, l);
}
__device__ __forceinline__ void lds_of_wave_settled() {  // what lanes of this wave wrote to LDS is seen by the others
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The best entries that a wave has seen, as keys.
struct WaveTop {
    uint64_t *place;  // 64 places in LDS
    int n, want;      // places used, entries wanted (the same in all lanes)
    uint64_t bar;     // only keys above it are added

    __device__ __forceinline__ WaveTop(uint64_t *p, int k) : place(p), n(0), want(k), bar(0) {}

    // Cut to the best, in order.
    __device__ __forceinline__ void rank() {
        const int lane = threadIdx.x & 63;
        lds_of_wave_settled();
        const uint64_t mine = lane < n ? place[lane] : 0;
        int above = 0;
        for (int j = 0; j < n; ++j) above += read_lane(mine, j) > mine ? 1 : 0;
        lds_of_wave_settled();
        if (lane < n && above < want) place[above] = mine;
        lds_of_wave_settled();
        n = min(n, want);
        if (n == want) bar = read_lane(lane < n ? place[lane] : 0, want - 1);
    }
    // A key of each lane, those above the bar (0: none).
    __device__ __forceinline__ void add(uint64_t key) {
        uint64_t mask = __ballot(key > bar);
        while (mask) {
            const int lane = threadIdx.x & 63, at = n + __builtin_popcountll(mask & ((1ull << lane) - 1));
            const bool mine = (mask >> lane) & 1;
            if (mine && at < 64) place[at] = key;
            n += __builtin_popcountll(mask);
            if (n <= 64) return;
            n = 64;
            rank();
            mask = __ballot(mine && at >= 64 && key > bar);
        }
    }
};

// Weights of a lane's entries against its shift m: l = sum 2^d, t = sum d 2^d, d = (x - m) c.
struct LaneSums {
    float m, l, t;
    __device__ __forceinline__ void to(float top, float c) {
        const float d = fmaxf((m - top) * c, kLowest), f = __builtin_amdgcn_exp2f(d);
        t = f == 0.0f && l == l ? 0.0f : f * (t + d * l);  // (d * l may be infinite)
        l *= f;
        m = top;
    }
};

template <class T>
__device__ __forceinline__ void load_eight(const T *row, int64_t i, int vocab, float (&x)[8]) {
    if (i >= 0 && i + 8 <= vocab) {  // 16-byte aligned
        typedef float f4 __attribute__((ext_vector_type(4)));
        if constexpr (sizeof(T) == 4) {
            const f4 a = __builtin_nontemporal_load(reinterpret_cast<const f4 *>(row + i));
            const f4 b = __builtin_nontemporal_load(reinterpret_cast<const f4 *>(row + i + 4));
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = a[e], x[4 + e] = b[e];
        } else {
            const Raw8<T> a = __builtin_nontemporal_load(reinterpret_cast<const Raw8<T> *>(row + i));
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = (float)a[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = i + e >= 0 && i + e < vocab ? (float)row[i + e] : kMinusInf;
    }
}

// What a row's sums give, by the first wave: `top` holds its best entries in order.
template <class T>
__device__ __forceinline__ void write_row(const LogprobArgs &a, int t, float m, float l, float tt, const WaveTop &top) {
    const int lane = threadIdx.x & 63;
    const float log_l = logf(l);
    const auto logp = [&](float x) {
        if (l == 0.0f) return kMinusInf;
        return (float)(((double)x - (double)m) * (double)a.scale - (double)log_l);
    };
    if (lane == 0) {
        if (a.logprobs) {
            const int32_t tok = a.tokens[t];
            const bool in = tok >= 0 && tok < a.vocab;
            a.logprobs[t] = logp(in ? (float)static_cast<const T *>(a.logits)[(int64_t)t * a.row_stride + tok] : kMinusInf);
        }
        if (a.entropy) a.entropy[t] = l == 0.0f ? 0.0f : log_l - tt / l * kLn2;
    }
    if (lane < a.n_top) {
        const bool is = lane < top.n;
        const uint64_t key = is ? top.place[lane] : 0;
        a.top_tokens[(int64_t)t * a.n_top + lane] = is ? index_of(key) : -1;
        a.top_logprobs[(int64_t)t * a.n_top + lane] = l != l ? l : is ? logp(logit_of(key)) : kMinusInf;
    }
}

template <class T, bool TOP>
__global__ __launch_bounds__(kLogprobThreads) void logprobs_kernel(LogprobArgs a) {
    __shared__ uint64_t places[kWavesLp][64];
    __shared__ float sums[kWavesLp][3];
    __shared__ int counts[kWavesLp];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t = a.first + (int)blockIdx.x / a.parts, part = (int)blockIdx.x % a.parts;
    const T *row = static_cast<const T *>(a.logits) + (int64_t)t * a.row_stride;
    const int before = (int)(((uintptr_t)row & 15) / sizeof(T));  // the row's entries count from the last 16-byte border
    const float c = a.scale * kLog2e;
    const int64_t end = min((int64_t)a.vocab, (int64_t)(part + 1) * a.part_rounds * kLogprobRound - before);
    int64_t i = (int64_t)part * a.part_rounds * kLogprobRound - before + 8 * tid;

    WaveTop top(places[wave], a.n_top);
    LaneSums s{kLowest, 0.0f, 0.0f};
    float next[8], most = kLowest;
    bool first = true;
    float top_logit = kMinusInf;
    load_eight(row, i, a.vocab, next);
    for (; i - 8 * lane < end; i += kLogprobRound) {  // (the same in all lanes of a wave)
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = next[e];
        const int64_t here = i;
        if (i + kLogprobRound - 8 * lane < end) load_eight(row, i + kLogprobRound, a.vocab, next);
        float mx = kMinusInf;
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = fmaxf(mx, x[e]);
        most = fmaxf(most, mx);
        if (__any((mx - s.m) * c > kLazy)) s.to(most, c);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = (x[e] - s.m) * c, w = __builtin_amdgcn_exp2f(d);
            s.l += w;
            s.t = __builtin_fmaf(fmaxf(d, -1024.0f), w, s.t);  // (0 for a weight of 0, whose d may be infinite)
        }
        if constexpr (TOP) {
            if (first) {  // the n-th largest of the lanes' maxima: what is below it is not among the best
                first = false;
                int above = 0;
                for (int j = 0; j < 64; ++j) {
                    const float y = read_lane(mx, j);
                    above += y > mx || (y == mx && j < lane) ? 1 : 0;
                }
                const uint64_t it = __ballot(above == a.n_top - 1);
                const float y = read_lane(mx, __builtin_ctzll(it));
                if (y > kMinusInf) top.bar = key_of(y, -1);  // (below every key of this logit)
            } else if (!__any(mx > top_logit)) {
                continue;  // (an equal logit further on is no better)
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) top.add(x[e] > kMinusInf ? key_of(x[e], (int32_t)(here + e)) : 0);
            top_logit = top.bar ? logit_of(top.bar) : kMinusInf;
        }
    }
    if constexpr (TOP) top.rank();

    // the lanes, then the waves
    const float m_wave = wave_max(most);
    s.to(m_wave, c);
    const float l_wave = wave_add(s.l), t_wave = wave_add(s.t);
    if (lane == 0) sums[wave][0] = m_wave, sums[wave][1] = l_wave, sums[wave][2] = t_wave, counts[wave] = top.n;
    __syncthreads();
    if (wave) return;
    float m = kLowest;
#pragma unroll
    for (int w = 0; w < kWavesLp; ++w) m = fmaxf(m, sums[w][0]);
    LaneSums all{m, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < kWavesLp; ++w) {
        LaneSums y{sums[w][0], sums[w][1], sums[w][2]};
        y.to(m, c);
        all.l += y.l;
        all.t += y.t;
    }
    if constexpr (TOP) {
#pragma unroll
        for (int w = 1; w < kWavesLp; ++w) top.add(lane < counts[w] ? places[w][lane] : 0);
        top.rank();
        lds_of_wave_settled();
    }
    if (a.parts == 1) {
        write_row<T>(a, t, all.m, all.l, all.t, top);
    } else {
        const int64_t at = (int64_t)t * a.parts + part;
        if (lane == 0) a.stats[at] = make_float4(all.m, all.l, all.t, 0.0f);
        if (TOP && lane < a.n_top) a.tops[at * a.n_top + lane] = lane < top.n ? top.place[lane] : 0;
    }
}

// Joins the parts of a row: one wave.
template <class T, bool TOP>
__global__ __launch_bounds__(64) void logprobs_join_kernel(LogprobArgs a) {
    __shared__ uint64_t places[64];
    const int lane = threadIdx.x, t = a.first + (int)blockIdx.x;
    const float c = a.scale * kLog2e;
    float m = kLowest;
    for (int p = lane; p < a.parts; p += 64) m = fmaxf(m, a.stats[(int64_t)t * a.parts + p].x);
    m = wave_max(m);
    float l = 0.0f, tt = 0.0f;
    for (int p = lane; p < a.parts; p += 64) {
        const float4 x = a.stats[(int64_t)t * a.parts + p];
        LaneSums y{x.x, x.y, x.z};
        y.to(m, c);
        l += y.l;
        tt += y.t;
    }
    l = wave_add(l);
    tt = wave_add(tt);
    WaveTop top(places, a.n_top);
    if constexpr (TOP) {
        const int total = a.parts * a.n_top;
        for (int i = lane; i - lane < total; i += 64) {
            top.add(i < total ? a.tops[(int64_t)t * total + i] : 0);
        }
        top.rank();
        lds_of_wave_settled();
    }
    write_row<T>(a, t, m, l, tt, top);
}

template <class T, bool TOP>
static int run_logprobs(LogprobArgs a, hipStream_t s) {
    const int32_t most = kMaxWgs / a.parts;  // rows of a launch
    for (const int32_t n = a.n_tokens; a.first < n; a.first += most) {
        const int32_t rows = n - a.first < most ? n - a.first : most;
        logprobs_kernel<T, TOP><<<(unsigned)(rows * a.parts), kLogprobThreads, 0, s>>>(a);
        hipError_t e = hipGetLastError();
        if (e == hipSuccess && a.parts > 1) {
            logprobs_join_kernel<T, TOP><<<(unsigned)rows, 64, 0, s>>>(a);
            e = hipGetLastError();
        }
        if (e != hipSuccess) return (int)e;
        if (n - a.first <= most) break;  // (before `first` can pass 2^31)
    }
    return (int)hipSuccess;
}

int launch_logprobs(const LogprobArgs &a, int32_t dtype, void *stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == 0) return a.n_top ? run_logprobs<float, true>(a, s) : run_logprobs<float, false>(a, s);
    if (dtype == 1) return a.n_top ? run_logprobs<__bf16, true>(a, s) : run_logprobs<__bf16, false>(a, s);
    return a.n_top ? run_logprobs<_Float16, true>(a, s) : run_logprobs<_Float16, false>(a, s);
}

}  // namespace bpw
