// bpw_elem.h - element types of the decode-step operators on the device: loads, stores and the one
// rounding to 16 bits (to nearest, ties to even).
#pragma once

#include <hip/hip_runtime.h>

namespace bpw {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32v4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

template <class T>
struct Vec8;
template <>
struct Vec8<float> { typedef f32x8 type; };
template <>
struct Vec8<__bf16> { typedef bf16x8 type; };
template <>
struct Vec8<_Float16> { typedef f16x8 type; };

// Eight consecutive elements, 16-byte aligned, as they are in memory and as float32.
template <class T>
using Raw8 = typename Vec8<T>::type;

template <class T>
__device__ __forceinline__ Raw8<T> raw8(const T *p) {
    if constexpr (sizeof(T) == 4) {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
        return *reinterpret_cast<const Raw8<T> *>(p);
    }
}

template <class V>
__device__ __forceinline__ f32x8 as_f32(V x) {
    return __builtin_convertvector(x, f32x8);
}

template <class T>
__device__ __forceinline__ f32x8 load8(const T *p) {
    return as_f32(raw8(p));
}

// Stored non-temporally: what a prompt's heads write is not read again by this launch (16384 tokens of 40 heads of
// 128 in bf16: 69.5 us, 73.1 with ordinary stores).
template <class T>
__device__ __forceinline__ void store8(T *p, f32x8 x) {
    if constexpr (sizeof(T) == 4) {
        __builtin_nontemporal_store(__builtin_shufflevector(x, x, 0, 1, 2, 3), reinterpret_cast<f32x4 *>(p));
        __builtin_nontemporal_store(__builtin_shufflevector(x, x, 4, 5, 6, 7), reinterpret_cast<f32x4 *>(p + 4));
    } else {
        __builtin_nontemporal_store(__builtin_convertvector(x, typename Vec8<T>::type), reinterpret_cast<typename Vec8<T>::type *>(p));
    }
}

// Cross-lane steps by DPP: a few cycles each, where a shuffle through LDS costs a round trip.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ int dpp(int x) {  // 0 where a lane has no source
    return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float dpp(float x) {
    return __builtin_bit_cast(float, dpp<CTRL, ROWS>(__builtin_bit_cast(int, x)));
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double dpp(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = dpp<CTRL, ROWS>((int)(uint32_t)u), hi = dpp<CTRL, ROWS>((int)(uint32_t)(u >> 32));
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ float read_lane(float x, int l) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), l));
}
__device__ __forceinline__ double read_lane(double x, int l) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, l), hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), l);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Sums over lanes 0 .. l in lane l: shifts by 1, 2, 4, 8 within rows of 16, then the last lane of a row to the next one,
// and lane 31 to the upper half.
template <class V>
__device__ __forceinline__ V scan_add(V x) {
    x += dpp<0x111>(x);
    x += dpp<0x112>(x);
    x += dpp<0x114>(x);
    x += dpp<0x118>(x);
    x += dpp<0x142, 0xA>(x);
    x += dpp<0x143, 0xC>(x);
    return x;
}

// Maximum and sum over the wave, in every lane: pairs, quads, mirrored eights and sixteens, then the four rows.
__device__ __forceinline__ float wave_max(float x) {
    x = fmaxf(x, dpp<0xB1>(x));
    x = fmaxf(x, dpp<0x4E>(x));
    x = fmaxf(x, dpp<0x141>(x));
    x = fmaxf(x, dpp<0x140>(x));
    return fmaxf(fmaxf(read_lane(x, 0), read_lane(x, 16)), fmaxf(read_lane(x, 32), read_lane(x, 48)));
}
template <class V>
__device__ __forceinline__ V wave_add(V x) {
    x += dpp<0xB1>(x);
    x += dpp<0x4E>(x);
    x += dpp<0x141>(x);
    x += dpp<0x140>(x);
    return (read_lane(x, 0) + read_lane(x, 16)) + (read_lane(x, 32) + read_lane(x, 48));
}

}  // namespace bpw
