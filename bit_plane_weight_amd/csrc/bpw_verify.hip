// bpw_verify.hip - verification of drafted tokens against the target's probabilities from given random
// numbers (gfx950, wave64). Launched only by bpw_decode_host.cpp after its checks.
//
// Mathematics. Draft i is accepted while u_i q_i(x_i) < p_i(x_i); both sides are exact in float64, so the
// decision has no rounding. After n accepted drafts the last token is the first whose running sum of
// masses exceeds r times their total, masses max(p_n - q_n, 0) after a refusal and p_n otherwise.
// Differences of float32 are formed and summed in float64: a running sum of 128256 float32 in float32
// would move the border by thousands of steps.
//
// Bound: HBM, one row of p and one of q per sequence; for one sequence the two launches. A row is cut into
// chunks of kVerifyChunk entries, one workgroup each, so that one sequence's rows are read by many CUs;
// the second launch (one workgroup per sequence) finds the chunk that holds the border from the chunks' sums
// and walks that chunk alone. Sums have a fixed order whatever the launch.
#include "bpw_decode.h"
#include "bpw_elem.h"

namespace bpw {

constexpr int kPer = kVerifyChunk / kVerifyThreads;  // entries of one thread

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
    const int most = a.n_draft ? min(max(a.n_draft[b], 0), a.max_drafts) : a.max_drafts;
    const T *t = static_cast<const T *>(a.target) + (int64_t)b * a.t_seq;
    const T *d = static_cast<const T *>(a.draft) + (int64_t)b * a.d_seq;
    bool ok = false;
    int x = -1;
    if (lane < most) {
        x = a.tokens[(int64_t)b * a.max_drafts + lane];
        if (x >= 0 && x < a.vocab) {
            const double p = (double)(float)t[lane * a.t_step + x];
            const double q = a.draft ? (double)(float)d[lane * a.d_step + x] : 1.0;
            ok = (double)a.accept_u[(int64_t)b * a.max_drafts + lane] * q < p;
        }
    }
    const uint64_t no = ~__ballot(ok);
    Drawn<T> r;
    r.n = no ? min((int)__builtin_ctzll(no), most) : most;
    r.refused = r.n < most;
    r.x = __shfl(x, r.n & 63);
    r.p = t + r.n * a.t_step;
    r.q = r.refused && a.draft ? d + r.n * a.d_step : nullptr;
    return r;
}

// The mass of an entry: rest == true takes the draft's away.
template <class T>
__device__ __forceinline__ double mass(const Drawn<T> &r, bool rest, int i) {
    double m = (double)(float)r.p[i];
    if (rest) {
        if (r.q) m -= (double)(float)r.q[i];
        else if (i == r.x) m = 0.0;  // p - 1 is never positive
    }
    return m > 0.0 && m < __builtin_inf() ? m : 0.0;
}

__device__ __forceinline__ double wave_sum(double s) {
#pragma unroll
    for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
    return s;
}

// Sum of the chunk's masses, the same in every thread: thread sums in entry order, then a tree. Entry
// c * kVerifyChunk + e * kVerifyThreads + tid for e = 0 .. kPer - 1.
template <class T>
__device__ __forceinline__ double chunk_sum(const VerifyArgs &a, const Drawn<T> &r, bool rest, int c, double *red) {
    double s = 0.0;
    const int i0 = c * kVerifyChunk + threadIdx.x;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int i = i0 + e * kVerifyThreads;
        if (i < a.vocab) s += mass(r, rest, i);
    }
    s = wave_sum(s);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

template <class T>
__global__ __launch_bounds__(kVerifyThreads) void verify_sums_kernel(VerifyArgs a) {
    __shared__ double red[4];
    const int b = blockIdx.y, c = blockIdx.x;
    const Drawn<T> r = accept<T>(a, b);
    const double s = chunk_sum(a, r, r.refused, c, red);
    if (threadIdx.x == 0) a.sums[(int64_t)b * a.chunks + c] = s;
}

// First index of the workgroup's threads for which `hit` holds, or -1.
__device__ __forceinline__ int first_hit(bool hit, int *red) {
    const uint64_t w = __ballot(hit);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = w ? (int)threadIdx.x + __builtin_ctzll(w) : -1;
    __syncthreads();
    return red[0] >= 0 ? red[0] : red[1] >= 0 ? red[1] : red[2] >= 0 ? red[2] : red[3];
}
__device__ __forceinline__ int last_hit(bool hit, int *red) {
    const uint64_t w = __ballot(hit);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = w ? (int)threadIdx.x + 63 - __builtin_clzll(w) : -1;
    __syncthreads();
    return red[3] >= 0 ? red[3] : red[2] >= 0 ? red[2] : red[1] >= 0 ? red[1] : red[0];
}

// Sum before this thread's value over the workgroup.
__device__ __forceinline__ double before(double v, double *red) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double inc = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double x = __shfl_up(inc, d);
        if (lane >= d) inc += x;
    }
    __syncthreads();
    if (lane == 63) red[wave] = inc;
    __syncthreads();
    double base = 0.0;
    for (int w = 0; w < wave; ++w) base += red[w];
    return base + (inc - v);
}

template <class T>
__global__ __launch_bounds__(kVerifyThreads) void verify_draw_kernel(VerifyArgs a) {
    __shared__ double red[4];
    __shared__ int ired[4], found;
    extern __shared__ double sums[];  // [chunks], then running sums
    const int b = blockIdx.x, tid = threadIdx.x;
    const Drawn<T> r = accept<T>(a, b);
    bool rest = r.refused;
    for (int c = tid; c < a.chunks; c += kVerifyThreads) sums[c] = a.sums[(int64_t)b * a.chunks + c];
    __syncthreads();
    double total = 0.0;
    for (int c = 0; c < a.chunks; ++c) total += sums[c];
    if (rest && total == 0.0) {  // nothing left after the draft's mass: the target's row itself
        rest = false;
        for (int c = 0; c < a.chunks; ++c) {
            const double s = chunk_sum(a, r, rest, c, red);
            if (tid == 0) sums[c] = s;
            total += s;
        }
        __syncthreads();
    }
    int token = -1;
    if (total > 0.0) {
        const double border = (double)a.sample_u[b] * total;
        // the first chunk whose running sum exceeds the border, else the last with mass
        double run = 0.0, base = 0.0;
        int at = -1;
        for (int c = 0; c < a.chunks; ++c) {
            if (sums[c] > 0.0) {
                at = c;
                base = run;
            }
            run += sums[c];
            if (run > border) break;
        }
        // inside it: kPer neighbours a thread
        double m[kPer], mine = 0.0;
        const int i0 = at * kVerifyChunk + tid * kPer;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            m[e] = i0 + e < a.vocab ? mass(r, rest, i0 + e) : 0.0;
            mine += m[e];
        }
        double cum = base + before(mine, red);
        int hit = -1, last = -1;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            cum += m[e];
            if (m[e] > 0.0) {
                if (hit < 0 && cum > border) hit = e;
                last = e;
            }
        }
        int who = first_hit(hit >= 0, ired);
        if (who < 0) {  // the sums' order put the border past the chunk's last entry
            who = last_hit(last >= 0, ired);
            hit = last;
        }
        if (tid == who) found = i0 + hit;
        __syncthreads();
        token = found;
    }
    for (int i = tid; i <= a.max_drafts; i += kVerifyThreads)
        a.out_tokens[(int64_t)b * (a.max_drafts + 1) + i] =
            i < r.n ? a.tokens[(int64_t)b * a.max_drafts + i] : i == r.n ? token : -1;
    if (tid == 0) a.accepted[b] = r.n;
}

template <class T>
static int run_verify(const VerifyArgs &a, hipStream_t s) {
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
