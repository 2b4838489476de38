// bpw_verify.hip - verification of drafted tokens against the target's probabilities from given random
// numbers (gfx950, wave64). Launched only by bpw_decode_host.cpp after its checks.
//
// Mathematics. Draft i is accepted while u_i q_i(x_i) < p_i(x_i); both sides are exact in float64, so the
// decision has no rounding. After n accepted drafts the last token is the first whose running sum of
// masses exceeds r times their total, masses max(p_n - q_n, 0) after a refusal and p_n otherwise.
// Differences of float32 are formed and summed in float64: a running sum of 128256 float32 in float32
// would move the border by thousands of steps.
//
// Bound: HBM, one row of p and one of q per sequence (64 sequences of 128256 entries: 65.7 MB in 13 us, after two
// dependent gathers), then the draw's latency (7.6 us; 4.4 for one sequence). A row is cut into
// chunks of kVerifyChunk entries, one workgroup each, so that one sequence's rows are read by many CUs;
// the second launch (one workgroup per sequence) finds the chunk that holds the border from the chunks' sums
// and walks that chunk alone. Sums have a fixed order whatever the launch: a lane's four neighbours, the lanes of
// a wave, the sixteen wave rounds of a chunk, the chunks.
#include "bpw_decode.h"
#include "bpw_elem.h"

namespace bpw {

constexpr int kRounds = kVerifyChunk / (4 * kVerifyThreads);  // a wave takes 256 neighbours at a time, four a lane
constexpr int kSubs = 4 * kRounds;                            // wave rounds of a chunk
constexpr int kSub = 256;                                     // entries of one

// What sequence b draws from: drafts accepted, whether one was refused, the rows.
template <class T>
struct Drawn {
    int n;
    bool refused;
    int x;        // the refused token (draft given as certain tokens)
    const T *p, *q;
};

// Every wave finds it by itself: lane i holds draft i.
template <class T>
__device__ __forceinline__ Drawn<T> accept(const VerifyArgs &a, int b) {
    const int lane = threadIdx.x & 63;
    const int given = a.n_draft ? a.n_draft[b] : a.max_drafts;  // (loaded beside the tokens)
    const T *t = static_cast<const T *>(a.target) + (int64_t)b * a.t_seq;
    const T *d = static_cast<const T *>(a.draft) + (int64_t)b * a.d_seq;
    bool ok = false;
    int x = -1;
    if (lane < a.max_drafts) {
        x = a.tokens[(int64_t)b * a.max_drafts + lane];
        const float u = a.accept_u[(int64_t)b * a.max_drafts + lane];
        if (x >= 0 && x < a.vocab) {
            const double p = (double)(float)t[lane * a.t_step + x];
            const double q = a.draft ? (double)(float)d[lane * a.d_step + x] : 1.0;
            ok = (double)u * q < p;
        }
    }
    const int most = min(max(given, 0), a.max_drafts);
    ok = ok && lane < most;
    const uint64_t no = ~__ballot(ok);
    Drawn<T> r;
    r.n = no ? min((int)__builtin_ctzll(no), most) : most;
    r.refused = r.n < most;
    r.x = __builtin_amdgcn_readlane(x, r.n & 63);
    r.p = t + r.n * a.t_step;
    r.q = r.refused && a.draft ? d + r.n * a.d_step : nullptr;
    return r;
}

template <class T>
__device__ __forceinline__ Drawn<T> drawn_from(const VerifyArgs &a, int b, int n, bool refused) {
    Drawn<T> r;
    r.n = n;
    r.refused = refused;
    r.x = refused ? a.tokens[(int64_t)b * a.max_drafts + n] : -1;
    r.p = static_cast<const T *>(a.target) + (int64_t)b * a.t_seq + n * a.t_step;
    r.q = refused && a.draft ? static_cast<const T *>(a.draft) + (int64_t)b * a.d_seq + n * a.d_step : nullptr;
    return r;
}

// Four neighbours of a row from entry i on; zeros past the vocabulary.
template <class T>
__device__ __forceinline__ void four(const T *row, int i, int vocab, float (&x)[4]) {
    typedef T T4 __attribute__((ext_vector_type(4)));
    if (((uintptr_t)row & (sizeof(T4) - 1)) == 0 && i + 4 <= vocab) {
        const T4 v = *reinterpret_cast<const T4 *>(row + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = (float)v[e];
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = i + e < vocab ? (float)row[i + e] : 0.0f;
    }
}

// The masses of this lane's entries of round j of a chunk; rest: the draft's are taken away.
template <class T>
__device__ __forceinline__ void masses(const VerifyArgs &a, const Drawn<T> &r, bool rest, int i, double (&m)[4]) {
    float p[4], q[4] = {0, 0, 0, 0};
    four(r.p, i, a.vocab, p);
    if (rest && r.q) four(r.q, i, a.vocab, q);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        double x = (double)p[e] - (double)q[e];
        if (rest && !r.q && i + e == r.x) x = 0.0;  // p - 1 is never positive
        m[e] = x > 0.0 && x < __builtin_inf() ? x : 0.0;
    }
}

// First entry of this lane in wave round `sub` (0 .. kSubs - 1, in the order of entries) of chunk c.
__device__ __forceinline__ int entry_of(int c, int sub) { return c * kVerifyChunk + sub * kSub + 4 * (threadIdx.x & 63); }

// The sums of the chunk's wave rounds, in LDS (a wave makes kRounds of them); a barrier makes them seen.
template <class T>
__device__ __forceinline__ void sub_sums(const VerifyArgs &a, const Drawn<T> &r, bool rest, int c, double *subs) {
    const int wave = threadIdx.x >> 6;
    double m[kRounds][4];
#pragma unroll
    for (int j = 0; j < kRounds; ++j) masses(a, r, rest, entry_of(c, wave * kRounds + j), m[j]);
#pragma unroll
    for (int j = 0; j < kRounds; ++j) {
        const double s = wave_add((m[j][0] + m[j][1]) + (m[j][2] + m[j][3]));
        if ((threadIdx.x & 63) == 0) subs[wave * kRounds + j] = s;
    }
}

__device__ __forceinline__ double sum_of(const double *subs) {
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < kSubs; ++j) s += subs[j];
    return s;
}

template <class T>
__global__ __launch_bounds__(kVerifyThreads) void verify_sums_kernel(VerifyArgs a) {
    __shared__ double subs[kSubs];
    const int b = blockIdx.y, c = blockIdx.x;
    const Drawn<T> r = accept<T>(a, b);
    sub_sums(a, r, r.refused, c, subs);
    __syncthreads();
    if (threadIdx.x == 0) {
        a.sums[(int64_t)b * a.chunks + c] = sum_of(subs);
        if (c == 0) a.found[2 * b] = r.n, a.found[2 * b + 1] = r.refused;
    }
}

// Running sums over up to 64 lanes, and the first lane whose running sum exceeds the border (or, if none does, the last
// with a positive value): that lane, or -1 if none is positive, the sum before it and whether it exceeds. (before + its v may
// not, as floating point sums.)
__device__ __forceinline__ int border_lane(double v, double run, double border, double &before, double &after, bool &exceeds) {
    const double inc = scan_add(v);
    after = run + read_lane(inc, 63);
    const uint64_t some = __ballot(v > 0.0), over = __ballot(v > 0.0 && run + inc > border);
    exceeds = over != 0;
    const int lane = over ? __builtin_ctzll(over) : some ? 63 - __builtin_clzll(some) : -1;
    before = lane < 0 ? run : run + read_lane(inc - v, lane < 0 ? 0 : lane);
    return lane;
}

// The last token of a sequence: the first entry whose running sum exceeds the border, from the wave round that holds it
// and the sum before that round. Every wave by itself, the same.
template <class T>
__device__ __forceinline__ int entry_in(const VerifyArgs &a, const Drawn<T> &r, bool rest, int c, int sub, double before,
                                        double border) {
    double m[4], after;
    bool exceeds;
    const int i = entry_of(c, sub);
    masses(a, r, rest, i, m);
    const int l = border_lane((m[0] + m[1]) + (m[2] + m[3]), before, border, before, after, exceeds);
    // the lane's own entry: the first over the border, else its last with mass (the sums' order can put the border past the
    // last)
    double cum = before;
    int hit = -1, last = -1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        cum += m[e];
        if (m[e] > 0.0) {
            if (hit < 0 && cum > border) hit = e;
            last = e;
        }
    }
    return __builtin_amdgcn_readlane(i + (hit >= 0 ? hit : last), l);
}

template <class T>
__device__ __forceinline__ void write_tokens(const VerifyArgs &a, int b, int n, int token) {
    for (int i = threadIdx.x; i <= a.max_drafts; i += kVerifyThreads)
        a.out_tokens[(int64_t)b * (a.max_drafts + 1) + i] = i < n ? a.tokens[(int64_t)b * a.max_drafts + i] : i == n ? token : -1;
    if (threadIdx.x == 0) a.accepted[b] = n;
}

template <class T>
__global__ __launch_bounds__(kVerifyThreads) void verify_draw_kernel(VerifyArgs a) {
    __shared__ double subs[kSubs];
    extern __shared__ double sums[];  // [chunks]
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
    const int n = a.found[2 * b];
    const Drawn<T> r = drawn_from<T>(a, b, n, a.found[2 * b + 1] != 0);
    for (int c = tid; c < a.chunks; c += kVerifyThreads) sums[c] = a.sums[(int64_t)b * a.chunks + c];
    __syncthreads();
    bool rest = r.refused;
    double total = 0.0;  // every wave by itself, the same
    for (int c0 = 0; c0 < a.chunks; c0 += 64) total += wave_add(c0 + lane < a.chunks ? sums[c0 + lane] : 0.0);
    if (rest && total == 0.0) {  // nothing left after the draft's mass: the target's row itself
        rest = false;
        for (int c = 0; c < a.chunks; ++c) {
            sub_sums(a, r, rest, c, subs);
            __syncthreads();
            if (tid == 0) sums[c] = sum_of(subs);
            __syncthreads();
        }
        for (int c0 = 0; c0 < a.chunks; c0 += 64) total += wave_add(c0 + lane < a.chunks ? sums[c0 + lane] : 0.0);
    }
    int token = -1;
    if (total > 0.0) {
        const double border = (double)a.sample_u[b] * total;
        // the first chunk whose running sum exceeds the border, else the last with mass
        double run = 0.0, base = 0.0, before, after;
        bool exceeds;
        int chunk = -1;
        for (int c0 = 0; c0 < a.chunks; c0 += 64) {
            const int l = border_lane(c0 + lane < a.chunks ? sums[c0 + lane] : 0.0, run, border, before, after, exceeds);
            if (l >= 0) {
                chunk = c0 + l;
                base = before;
                if (exceeds) break;
            }
            run = after;
        }
        // in it the wave round, and in that the entry
        sub_sums(a, r, rest, chunk, subs);
        __syncthreads();
        const int sub = border_lane(lane < kSubs ? subs[lane] : 0.0, base, border, before, after, exceeds);
        token = entry_in(a, r, rest, chunk, sub, before, border);
    }
    write_tokens<T>(a, b, n, token);
}

// A small vocabulary: one workgroup to a sequence does it all in one launch.
constexpr int kSmallChunks = 2;
static_assert(kSmallChunks * kSubs <= 64, "a lane holds a wave round's sum");
template <class T>
__global__ __launch_bounds__(kVerifyThreads) void verify_small_kernel(VerifyArgs a) {
    __shared__ double subs[kSmallChunks * kSubs];
    const int b = blockIdx.x, lane = threadIdx.x & 63;
    const Drawn<T> r = accept<T>(a, b);
    bool rest = r.refused;
    double total = 0.0;
    while (true) {
        for (int c = 0; c < a.chunks; ++c) sub_sums(a, r, rest, c, subs + c * kSubs);
        __syncthreads();
        total = wave_add(lane < a.chunks * kSubs ? subs[lane] : 0.0);
        if (!rest || total > 0.0) break;
        rest = false;  // nothing left after the draft's mass: the target's row itself
        __syncthreads();
    }
    int token = -1;
    if (total > 0.0) {
        const double border = (double)a.sample_u[b] * total;
        double before, after;
        bool exceeds;
        const int sub = border_lane(lane < a.chunks * kSubs ? subs[lane] : 0.0, 0.0, border, before, after, exceeds);
        token = entry_in(a, r, rest, sub / kSubs, sub % kSubs, before, border);
    }
    write_tokens<T>(a, b, r.n, token);
}

template <class T>
static int run_verify(const VerifyArgs &a, hipStream_t s) {
    // One launch or two, us a call: 1000 entries 4.6 and 8.4 (one sequence), 5.5 and 10.4 (64); 8000 entries 6.6 and 9.0,
    // 7.4 and 10.1; 16384 entries 9.2 and 8.2, 14.7 and 12.9.
    if (a.chunks <= kSmallChunks) {
        verify_small_kernel<T><<<(unsigned)a.n_seqs, kVerifyThreads, 0, s>>>(a);
        return (int)hipGetLastError();
    }
    verify_sums_kernel<T><<<dim3((unsigned)a.chunks, (unsigned)a.n_seqs), kVerifyThreads, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return (int)e;
    verify_draw_kernel<T><<<(unsigned)a.n_seqs, kVerifyThreads, (size_t)a.chunks * sizeof(double), s>>>(a);
    return (int)hipGetLastError();
}

int launch_verify(const VerifyArgs &a, int32_t dtype, void *stream) {
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == 0) return run_verify<float>(a, s);
    if (dtype == 1) return run_verify<__bf16>(a, s);
    return run_verify<_Float16>(a, s);
}

}  // namespace bpw
