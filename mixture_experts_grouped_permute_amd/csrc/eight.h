// 8 consecutive bf16 or fp32 values as loaded, for kernels that read tensors from any address on.
#pragma once
#include "common.h"

namespace moe {

// 8 consecutive values.  kAligned: at 16 bytes; else at the type's alignment, which global memory's wide
// accesses take as well.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));

// (global memory said outright: addresses out of a table would be generic ones)
template <class T>
__device__ __forceinline__ const __attribute__((address_space(1))) T* global(const void* p) {
  return (const __attribute__((address_space(1))) T*)p;
}
template <class T>
__device__ __forceinline__ __attribute__((address_space(1))) T* global(void* p) {
  return (__attribute__((address_space(1))) T*)p;
}

template <bool kF32, bool kAligned>
struct Eight {
  u32x4 w[kF32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    const char* b = reinterpret_cast<const char*>(p) + at * (kF32 ? 4 : 2);
    if constexpr (kAligned) {
      w[0] = global<u32x4>(b)[0];
      if constexpr (kF32) w[1] = global<u32x4>(b)[1];
    } else {
      w[0] = global<u32x4_any>(b)[0];
      if constexpr (kF32) w[1] = global<u32x4_any>(b)[1];
    }
  }
  // the same past the caches, for values that are read once
  __device__ __forceinline__ void load_once(const void* p, int64_t at) {
    const char* b = reinterpret_cast<const char*>(p) + at * (kF32 ? 4 : 2);
    if constexpr (kAligned) {
      w[0] = __builtin_nontemporal_load(global<u32x4>(b));
      if constexpr (kF32) w[1] = __builtin_nontemporal_load(global<u32x4>(b) + 1);
    } else {
      w[0] = __builtin_nontemporal_load(global<u32x4_any>(b));
      if constexpr (kF32) w[1] = __builtin_nontemporal_load(global<u32x4_any>(b) + 1);
    }
  }
  // the first n of them, the others left as they are; the address is the type's
  __device__ __forceinline__ void load_some(const void* p, int64_t at, int n) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if constexpr (kF32) {
          w[i >> 2][i & 3] = global<uint32_t>(p)[at + i];
        } else {
          const uint32_t u = global<uint16_t>(p)[at + i];
          w[0][i >> 1] = (i & 1) ? (w[0][i >> 1] & 0xFFFFu) | u << 16 : (w[0][i >> 1] & 0xFFFF0000u) | u;
        }
      }
  }
  __device__ __forceinline__ void store_some(void* p, int64_t at, int n) const {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if constexpr (kF32) global<uint32_t>(p)[at + i] = w[i >> 2][i & 3];
        else global<uint16_t>(p)[at + i] = (uint16_t)(w[0][i >> 1] >> (i & 1) * 16);
      }
  }
  // without the first `skip` of them
  __device__ __forceinline__ void store_from(void* p, int64_t at, int skip) const {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i >= skip) {
        if constexpr (kF32) global<uint32_t>(p)[at + i] = w[i >> 2][i & 3];
        else global<uint16_t>(p)[at + i] = (uint16_t)(w[0][i >> 1] >> (i & 1) * 16);
      }
  }
  __device__ __forceinline__ void zero() {
    w[0] = u32x4{0u, 0u, 0u, 0u};
    if constexpr (kF32) w[1] = u32x4{0u, 0u, 0u, 0u};
  }
  __device__ __forceinline__ float at(int i) const {
    // (the word is copied first: a bit cast of the vector's element itself reads element 0)
    const uint32_t u = kF32 ? w[kF32 ? i >> 2 : 0][i & 3] : (i & 1) ? w[0][i >> 1] & 0xFFFF0000u : w[0][i >> 1] << 16;
    return __builtin_bit_cast(float, u);
  }
  __device__ __forceinline__ void set(const float* v) {
    if constexpr (kF32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i >> 2][i & 3] = __builtin_bit_cast(uint32_t, v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[0][i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    }
  }
  // kOnce: past the caches
  template <bool kOnce = false>
  __device__ __forceinline__ void store(void* p, int64_t at) const {
    char* b = reinterpret_cast<char*>(p) + at * (kF32 ? 4 : 2);
    if constexpr (kAligned) {
      if constexpr (kOnce) {
        __builtin_nontemporal_store(w[0], global<u32x4>(b));
        if constexpr (kF32) __builtin_nontemporal_store(w[1], global<u32x4>(b) + 1);
      } else {
        global<u32x4>(b)[0] = w[0];
        if constexpr (kF32) global<u32x4>(b)[1] = w[1];
      }
    } else if constexpr (kOnce) {
      __builtin_nontemporal_store(w[0], global<u32x4_any>(b));
      if constexpr (kF32) __builtin_nontemporal_store(w[1], global<u32x4_any>(b) + 1);
    } else {
      global<u32x4_any>(b)[0] = w[0];
      if constexpr (kF32) global<u32x4_any>(b)[1] = w[1];
    }
  }
};

}  // namespace moe
