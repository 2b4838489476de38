// bpw_checks.h - argument checks that the host sides of the decode-step operators share (bpw_decode_host.cpp,
// bpw_requests_host.cpp).
#pragma once

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include <hip/hip_runtime.h>

#include "../../include/bpw.h"
#include "bpw_decode.h"
#include "bpw_internal.h"

namespace {

bpw_status fail(bpw_status code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
bpw_status fail(bpw_status code, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    bpw::record_error(buf);
    return code;
}

bpw_status hip_status(int e, const char *what) {
    if (e == (int)hipSuccess) return BPW_OK;
    return fail(BPW_E_HIP, "%s failed: %s", what, hipGetErrorString((hipError_t)e));
}

constexpr int64_t kMaxStride = INT64_C(1) << 40;   // elements: offsets stay below 2^63 bytes
constexpr int64_t kMaxRowStride = INT64_C(1) << 24;  // of a cache row: sixteen of them fit 32 bits
constexpr int32_t kMaxHeads = 1024;

size_t dtype_size(int32_t dt) { return dt == BPW_F32 ? 4 : 2; }
bool dtype_ok(int32_t dt) { return dt == BPW_F32 || dt == BPW_BF16 || dt == BPW_F16; }
bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// A set of heads: present (heads > 0) ones need a pointer, aligned to an element, and sane strides.
bpw_status check_heads(const bpw_heads &h, const char *who, const char *what) {
    if (h.heads < 0 || h.heads > kMaxHeads) return fail(BPW_E_INVAL, "%s: %s.heads %d outside [0, %d]", who, what, (int)h.heads, (int)kMaxHeads);
    if (h.heads == 0) return BPW_OK;
    if (!dtype_ok(h.dtype)) return fail(BPW_E_INVAL, "%s: %s has no type %d", who, what, (int)h.dtype);
    if (!h.d) return fail(BPW_E_INVAL, "%s: %s is NULL", who, what);
    if (!aligned(h.d, dtype_size(h.dtype))) return fail(BPW_E_INVAL, "%s: %s is not aligned to its elements", who, what);
    if (h.token_stride < 0 || h.head_stride < 0 || h.token_stride > kMaxStride || h.head_stride > kMaxStride)
        return fail(BPW_E_INVAL, "%s: strides of %s outside [0, 2^40]", who, what);
    return BPW_OK;
}

bpw_status check_rotation(const bpw_rotation &r, int32_t head_dim, const char *who) {
    if (r.rot_dim < 0 || r.rot_dim > head_dim || r.rot_dim % 2)
        return fail(BPW_E_INVAL, "%s: rot_dim %d is not even in [0, %d]", who, (int)r.rot_dim, (int)head_dim);
    if (r.interleaved != 0 && r.interleaved != 1) return fail(BPW_E_INVAL, "%s: interleaved is neither 0 nor 1", who);
    if (r.rot_dim > 0 && (!r.d_positions || !r.d_inv_freq))
        return fail(BPW_E_INVAL, "%s: positions or frequencies are NULL", who);
    if (!aligned(r.d_positions, 4) || !aligned(r.d_inv_freq, 8))
        return fail(BPW_E_INVAL, "%s: positions or frequencies are misaligned", who);
    return BPW_OK;
}

bpw_status check_kv(const bpw_paged_kv &c, const char *who) {
    if (c.dtype != BPW_BF16 && c.dtype != BPW_F16) return fail(BPW_E_INVAL, "%s: a cache is bfloat16 or float16", who);
    if (c.kv_heads < 1 || c.kv_heads > kMaxHeads) return fail(BPW_E_INVAL, "%s: kv_heads %d outside [1, %d]", who, (int)c.kv_heads, (int)kMaxHeads);
    if (c.page_size < 16 || c.page_size > 1024 || (c.page_size & (c.page_size - 1)))
        return fail(BPW_E_UNSUPPORTED, "%s: page_size %d is not a power of two in [16, 1024]", who, (int)c.page_size);
    if (c.n_pages < 0) return fail(BPW_E_INVAL, "%s: n_pages %d is negative", who, (int)c.n_pages);
    if (c.n_pages > 0 && (!c.d_k || !c.d_v)) return fail(BPW_E_INVAL, "%s: cache pointer is NULL", who);
    if (!aligned(c.d_k, 2) || !aligned(c.d_v, 2)) return fail(BPW_E_INVAL, "%s: cache is not aligned to its elements", who);
    const int64_t st[] = {c.k_page_stride, c.k_head_stride, c.v_page_stride, c.v_head_stride};
    for (int64_t x : st)
        if (x < 0 || x > kMaxStride) return fail(BPW_E_INVAL, "%s: cache strides outside [0, 2^40]", who);
    if (c.k_row_stride < 0 || c.v_row_stride < 0 || c.k_row_stride > kMaxRowStride || c.v_row_stride > kMaxRowStride)
        return fail(BPW_E_INVAL, "%s: cache row strides outside [0, 2^24]", who);
    return BPW_OK;
}

int log2_of(int32_t x) {
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

// Whether a set of heads can be moved 16 bytes at a time (8 elements of 16 bits).
bool wide(const void *p, int32_t dt, int64_t a, int64_t b, int64_t c) {
    const int64_t n = dt == BPW_F32 ? 4 : 8;
    return aligned(p, 16) && a % n == 0 && b % n == 0 && c % n == 0;
}

bpw::HeadSet head_set(const bpw_heads &in, const bpw_heads &out, const float *gain) {
    bpw::HeadSet s{};
    s.in = in.d;
    s.in_ts = in.token_stride;
    s.in_hs = in.head_stride;
    s.out = out.d;
    s.out_ts = out.token_stride;
    s.out_hs = out.head_stride;
    s.gain = gain;
    s.heads = in.heads;
    return s;
}

bpw_status check_eps(float eps, const char *who) {
    if (!(std::isfinite(eps) && eps >= 0.0f)) return fail(BPW_E_INVAL, "%s: eps is negative or not finite", who);
    return BPW_OK;
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace
