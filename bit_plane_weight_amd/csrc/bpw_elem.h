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

// Eight consecutive elements, 16-byte aligned, as float32.
template <class T>
__device__ __forceinline__ f32x8 load8(const T *p) {
    if constexpr (sizeof(T) == 4) {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
        return __builtin_convertvector(*reinterpret_cast<const typename Vec8<T>::type *>(p), f32x8);
    }
}

template <class T>
__device__ __forceinline__ void store8(T *p, f32x8 x) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<f32x4 *>(p) = __builtin_shufflevector(x, x, 0, 1, 2, 3);
        *reinterpret_cast<f32x4 *>(p + 4) = __builtin_shufflevector(x, x, 4, 5, 6, 7);
    } else {
        *reinterpret_cast<typename Vec8<T>::type *>(p) = __builtin_convertvector(x, typename Vec8<T>::type);
    }
}

}  // namespace bpw
