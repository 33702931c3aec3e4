// Sixteen-byte vectors of a row's elements and their fp32 values.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssc {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

template <typename T>
struct Vec {
  static constexpr int N = 8;
  __device__ static __forceinline__ void unpack(const u32x4& v, float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (__is_same(T, __bf16)) {
        f[2 * e] = __uint_as_float(v[e] << 16);
        f[2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
      } else {
        f[2 * e] = float(__builtin_bit_cast(_Float16, uint16_t(v[e] & 0xffffu)));
        f[2 * e + 1] = float(__builtin_bit_cast(_Float16, uint16_t(v[e] >> 16)));
      }
    }
  }
  __device__ static __forceinline__ u32x4 pack(const float (&f)[8]) {
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const f32x2 p{f[2 * e], f[2 * e + 1]};
      if constexpr (__is_same(T, __bf16))
        v[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
      else
        v[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, f16x2));
    }
    return v;
  }
};

template <>
struct Vec<float> {
  static constexpr int N = 4;
  __device__ static __forceinline__ void unpack(const u32x4& v, float (&f)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(v[e]);
  }
  __device__ static __forceinline__ u32x4 pack(const float (&f)[4]) {
    u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __float_as_uint(f[e]);
    return v;
  }
};

}  // namespace
}  // namespace ssc
