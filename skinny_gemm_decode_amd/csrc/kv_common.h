// Shared by the cache, rotation and attention kernels.
#pragma once

#include "common.h"
#include "kv_layout.h"

namespace skg {

typedef float f32x2 __attribute__((ext_vector_type(2)));

// A value of a row in memory, as binary32 and back (nearest even).
template <class T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kVec = 4;  // elements of a 16-byte unit
  __device__ static void unpack(u32x4 u, float (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = u[i];  // a bit_cast of a vector element's lvalue reads element 0
      x[i] = __builtin_bit_cast(float, w);
    }
  }
  __device__ static u32x4 pack(const float (&x)[4]) {
    u32x4 u;
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __builtin_bit_cast(uint32_t, x[i]);
    return u;
  }
  __device__ static void put_pair(void* p, float a, float b) { *static_cast<f32x2*>(p) = f32x2{a, b}; }
};
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ inline uint32_t bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(a), static_cast<__bf16>(b)});
}
__device__ inline float bf16_lo(uint32_t u) { return __builtin_bit_cast(float, u << 16); }
__device__ inline float bf16_hi(uint32_t u) { return __builtin_bit_cast(float, u & 0xFFFF0000u); }
template <>
struct Elem<__bf16> {
  static constexpr int kVec = 8;
  __device__ static void unpack(u32x4 u, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(u[i]);
      x[2 * i + 1] = bf16_hi(u[i]);
    }
  }
  __device__ static u32x4 pack(const float (&x)[8]) {
    u32x4 u;
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = bf16_pair(x[2 * i], x[2 * i + 1]);
    return u;
  }
  __device__ static void put_pair(void* p, float a, float b) { *static_cast<uint32_t*>(p) = bf16_pair(a, b); }
};

}  // namespace skg
