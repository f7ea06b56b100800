// Element types of the operators on queries, keys and values: eight elements
// at a time to and from float.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bbpe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <typename T> struct Vec8;
template <> struct Vec8<__bf16> { typedef bf16x8 type; };
template <> struct Vec8<_Float16> { typedef f16x8 type; };
template <> struct Vec8<float> { typedef f32x8 type; };
// The same in memory, where 16 bytes are all that is asked for (a vector of
// eight floats would have its accesses taken for 32-byte aligned ones).
template <typename T> struct Mem8 { typedef typename Vec8<T>::type type __attribute__((aligned(16))); };
static_assert(alignof(Mem8<float>::type) == 16 && alignof(Mem8<__bf16>::type) == 16, "");

// Eight consecutive elements as they lie in memory.  VEC: p is 16-byte aligned.
template <typename T>
__device__ __forceinline__ typename Vec8<T>::type load8_raw(const T *p, bool vec) {
  typename Vec8<T>::type v;
  if (vec) {
    v = *reinterpret_cast<const typename Mem8<T>::type *>(p);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[i];
  }
  return v;
}
template <typename T>
__device__ __forceinline__ void store8_raw(T *p, typename Vec8<T>::type v, bool vec) {
  if (vec) {
    *reinterpret_cast<typename Mem8<T>::type *>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = v[i];
  }
}
template <typename T>
__device__ __forceinline__ f32x8 to_float(typename Vec8<T>::type v) {
  return __builtin_convertvector(v, f32x8);
}
// round to nearest even
template <typename T>
__device__ __forceinline__ typename Vec8<T>::type from_float(f32x8 v) {
  return __builtin_convertvector(v, typename Vec8<T>::type);
}

}  // namespace bbpe
