// bpw_logprobs.hip - log probabilities of given tokens, entropy and top alternatives of rows of logits (gfx950, wave64).
// Launched only by bpw_requests_host.cpp after its checks.
//
// Mathematics. With M the largest logit of a row, d_v = scale (x_v - M), l = sum exp(d_v) and t = sum d_v exp(d_v):
//   log p_v = d_v - log l,   H = -sum p_v log p_v = log l - t / l,
// both terms of H positive, so that a nearly certain row loses nothing. Partial sums against a shift m join by
// l' = f l, t' = f (t + d l) with d = scale (m - M), f = exp(d). The shift of a wave is its largest logit so far, so that no d is
// above zero by more than the shift's rounding and these sums' terms are of one sign, too. (A shift that a logit may pass by 2^16 in
// weight is raised less often, but t + d l then loses 5e-7 of the entropy where the largest follows one 8 to 11 below it.)
//
// Bound: HBM, each logit read once. A workgroup takes four rounds of 2048 entries (eight a lane) while the next four are on their
// way. 2048 rows of 128256 in bfloat16, the best one: 84-110 us by the box and the values (4.8-6.2 TB/s; 84-90 without best
// entries), 168 a round at a time; 64 rows in float32, the best twenty: 22 us, 35 before. The vector units bound it then: 59
// instructions for eight entries.
// The best n entries are kept by each wave: a list of 64 places in LDS to which lanes add what exceeds a bar. The first is
// the n-th largest of the 64 lanes' maxima over the first four rounds; a list of 2 n or a full one is ranked (each lane
// counts the keys above its own) and cut to n, whose last is the next bar: n log(entries / n) are added in expectation.
// Few rows are cut into parts, one workgroup each, joined by a second launch.
#include "bpw_decode.h"
#include "bpw_elem.h"

namespace bpw {

constexpr int kWavesLp = kLogprobThreads / 64;
constexpr int kGroup = 4;  // rounds that a workgroup works on while as many are on their way
constexpr float kLowest = -3.4028234663852886e38f;
constexpr float kMinusInf = -__builtin_inff();
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

// The float after x towards larger ones.
__device__ __forceinline__ float above(float x) {
    const int32_t b = __builtin_bit_cast(int32_t, x + 0.0f);
    return __builtin_bit_cast(float, b < 0 ? b - 1 : b + 1);
}

// The best entries that a wave has seen, as keys.
struct WaveTop {
    uint64_t *place;  // 64 places in LDS
    int n, want;      // places used, entries wanted (the same in all lanes)
    uint64_t bar;     // only keys above it are added
    float logit;      // of the bar

    __device__ __forceinline__ WaveTop(uint64_t *p, int k) : place(p), n(0), want(k), bar(0), logit(kMinusInf) {}

    // A first bar: the n-th largest of the lanes' values, to its upper 20 bits (2^-11 of it), which are found one by one.
    __device__ __forceinline__ void bar_of_maxima(float x) {
        const uint32_t mine = (uint32_t)(key_of(x, 0) >> 32);
        uint32_t it = 0;
        for (uint32_t bit = 1u << 31; bit >= 1u << 12; bit >>= 1)
            if (__builtin_popcountll(__ballot(mine >= (it | bit))) >= want) it |= bit;
        const float y = logit_of((uint64_t)it << 32);
        if (y > kMinusInf) logit = y, bar = key_of(y, -1);  // (below every key of this logit)
    }
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
        if (n == want) {
            bar = read_lane(lane < n ? place[lane] : 0, want - 1);
            logit = logit_of(bar);
        }
    }
    // The keys of these lanes, for which there is room.
    __device__ __forceinline__ void append(uint64_t mask, uint64_t key) {
        const int at = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
        if (mask >> (threadIdx.x & 63) & 1) place[at] = key;
        n += __builtin_popcountll(mask);
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
    __device__ __forceinline__ void to(float top, float c) { move(top, (m - top) * c); }
    __device__ __forceinline__ void move(float top, float by) {  // to the shift of `top`; by: the old one less the new one, in units of log 2
        const float d = fmaxf(by, kLowest), f = __builtin_amdgcn_exp2f(d);
        t = f == 0.0f && l == l ? 0.0f : f * (t + d * l);  // (d * l may be infinite)
        l *= f;
        m = top;
    }
};

// A round of a row: 2048 entries, eight a lane, loaded 16 bytes at a time (rows of any alignment).
template <class T>
struct Round {
    static constexpr int LOADS = sizeof(T) == 4 ? 2 : 1, EACH = 8 / LOADS;
    typedef T Vec __attribute__((ext_vector_type(EACH), aligned(sizeof(T))));
    Vec v[LOADS];
    // the first entry of a lane's load j, from the round's; entry e is (at(e / EACH) + e % EACH)
    static __device__ __forceinline__ int at(int j) { return j * EACH * kLogprobThreads + EACH * (int)threadIdx.x; }
    static constexpr __device__ __forceinline__ int from_first(int e) { return e / EACH * EACH * kLogprobThreads + e % EACH; }
    static __device__ __forceinline__ int index(int e) { return at(0) + from_first(e); }
    __device__ __forceinline__ void load(const T *first) {
#pragma unroll
        for (int j = 0; j < LOADS; ++j) v[j] = __builtin_nontemporal_load(reinterpret_cast<const Vec *>(first + at(j)));
    }
    __device__ __forceinline__ void values(float *x) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (float)v[e / EACH][e % EACH];
    }
};

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
__global__ __launch_bounds__(kLogprobThreads, sizeof(T) == 2 ? 5 : 4) void logprobs_kernel(LogprobArgs a) {
    __shared__ uint64_t places[kWavesLp][64];
    __shared__ float sums[kWavesLp][3];
    __shared__ int counts[kWavesLp];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t = a.first + (int)blockIdx.x / a.parts, part = (int)blockIdx.x % a.parts;
    const T *row = static_cast<const T *>(a.logits) + (int64_t)t * a.row_stride;
    const float c = a.scale * kLog2e;

    WaveTop top(places[wave], a.n_top);
    // The shift of a wave's lanes is one, `level` in units of log 2: the product m c rounded, so that an exponent is one fma, or,
    // from 2^20 on, where the rounding is no longer small beside 1, the product itself (far).
    LaneSums s{kLowest, 0.0f, 0.0f};
    float most = kLowest, level = 0.0f;  // the lane's largest logit
    bool far = true;
    const auto level_of = [&] { return far ? (double)s.m * (double)c : (double)level; };
    const int32_t begin = part * a.part_rounds, end = min(begin + a.part_rounds, (a.vocab + kLogprobRound - 1) / kLogprobRound);
    const int32_t full = min(end, a.vocab / kLogprobRound);  // (the round that follows it may have some entries)
    Round<T> next[kGroup];
    if (begin < full) {
#pragma unroll
        for (int u = 0; u < kGroup; ++u) next[u].load(row + (int64_t)min(begin + u, full - 1) * kLogprobRound);
    }
    for (int32_t r = begin; r < end; r += kGroup) {
        float x[8 * kGroup];
        if (r < full) {
#pragma unroll
            for (int u = 0; u < kGroup; ++u) next[u].values(x + 8 * u);
#pragma unroll
            for (int u = 0; u < kGroup; ++u) next[u].load(row + (int64_t)min(r + kGroup + u, full - 1) * kLogprobRound);
        }
        if (r + kGroup > full) {  // the row's last entries, and what is none
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = kMinusInf;
            if (full < end) {
                int32_t i = full * kLogprobRound + Round<T>::at(0);
                asm volatile("" : "+v"(i));  // (nor are these addresses)
                T z[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] = row[min(i + Round<T>::from_first(e), a.vocab - 1)];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = i + Round<T>::from_first(e) < a.vocab ? (float)z[e] : kMinusInf;
            }
#pragma unroll
            for (int u = 0; u < kGroup; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[8 * u + e] = r + u > full ? kMinusInf : r + u == full ? y[e] : x[8 * u + e];
        }
        float mu[kGroup], mx = kMinusInf;
#pragma unroll
        for (int u = 0; u < kGroup; ++u) {
            mu[u] = x[8 * u];
#pragma unroll
            for (int e = 1; e < 7; e += 2) mu[u] = fmaxf(fmaxf(mu[u], x[8 * u + e]), x[8 * u + e + 1]);
            mu[u] = fmaxf(mu[u], x[8 * u + 7]);
            mx = fmaxf(mx, mu[u]);
        }
        most = fmaxf(most, mx);
        if (__ballot(mx > s.m)) {
            const float up = wave_max(most);
            const double old = level_of();
            level = up * c;
            far = !(fabsf(level) < 0x1p20f);
            s.m = up;
            s.move(up, (float)(old - level_of()));
        }
        // A group's sums by themselves first: in one chain of hundreds the roundings of entries that are nearly alike add up (a row of
        // 262144 was off by 1e-5).
        const auto weigh = [&](auto exponent) __attribute__((always_inline)) {
            float l = 0.0f, t = 0.0f;
#pragma unroll
            for (int e = 0; e < 8 * kGroup; ++e) {
                const float d = exponent(x[e]), w = __builtin_amdgcn_exp2f(d);
                l += w;
                t = __builtin_fmaf(fmaxf(d, -1024.0f), w, t);  // (0 for a weight of 0, whose d may be infinite)
            }
            s.l += l;
            s.t += t;
        };
        if (far)
            weigh([&](float y) { return (y - s.m) * c; });
        else
            weigh([&](float y) { return __builtin_fmaf(y, c, -level); });
        if constexpr (TOP) {
            // Entries that may be among the best: in the first group those that reach the n-th largest of the lanes' maxima, later
            // those above the n-th best so far (an equal logit further on is no better).
            const bool first = r == begin;
            if (first)
                top.bar_of_maxima(mx);
            else if (!__ballot(mx > top.logit))
                continue;
            float least = first ? fmaxf(top.logit, kLowest) : above(top.logit);
            bool fits = true;
#pragma unroll 1
            for (int again = 0;; ++again) {
                const int before = top.n;
                fits = true;
#pragma unroll
                for (int u = 0; u < kGroup; ++u) {
                    if (!__ballot(mu[u] >= least)) continue;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint64_t mask = __ballot(x[8 * u + e] >= least);
                        if (!mask) continue;
                        fits = fits && top.n + __builtin_popcountll(mask) <= 64;
                        if (fits) {
                            float y = x[8 * u + e];
                            int32_t i = Round<T>::at(0);
                            asm volatile("" : "+v"(y), "+v"(i));  // (keys are not worth registers of their own before they are needed)
                            top.append(mask, key_of(y, i + (r + u) * kLogprobRound + Round<T>::from_first(e)));
                        }
                    }
                }
                if (fits) break;
                top.n = before;
                if (again) break;
                top.rank();
                if (!first) least = above(top.logit);
            }
            if (!fits) {  // many at once (logits that rise, or are alike): one by one
#pragma unroll 1
                for (int e = 0; e < 8 * kGroup; ++e) {
                    const int32_t i = (r + e / 8) * kLogprobRound + Round<T>::index(e % 8);
                    const float y = r + e / 8 < end && i < a.vocab ? (float)row[i] : kMinusInf;
                    top.add(y > kMinusInf ? key_of(y, i) : 0);
                }
            }
            if (top.n >= 2 * top.want) top.rank();  // (a higher bar spares more groups than it costs)
        }
    }

    // the lanes, then the waves
    const float m_wave = wave_max(most);
    s.move(m_wave, (float)(level_of() - (double)m_wave * (double)c));
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
#pragma unroll 1
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
        // the best of every part first, so that the bar is soon high
        for (int i = lane; i - lane < total; i += 64) {
            const int place = i / a.parts, part = i - place * a.parts;
            top.add(i < total ? a.tops[((int64_t)t * a.parts + part) * a.n_top + place] : 0);
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
