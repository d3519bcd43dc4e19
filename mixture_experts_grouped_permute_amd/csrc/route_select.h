// Selection of a token's largest numbers by the lanes that share it: exchanges between lanes, keys that order a value
// and its expert as one number, and merge networks on them.
#pragma once
#include "common.h"

namespace moe {

// ---- exchange between the L lanes of a token: DPP moves, which the VALU does without LDS.  Step st
// pairs each lane with one of the other half of its group of 2^(st+1): xor 1, xor 2, then mirrors of
// 8 and 16 lanes, which pair the halves as well once the lanes within a half agree.
template <int st>
__device__ __forceinline__ int dpp_pair(int v) {
  if constexpr (st == 0) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);
  else if constexpr (st == 1) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);
  else if constexpr (st == 2) return __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true);
  else return __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true);
}
template <int st>
__device__ __forceinline__ float pair(float v) {
  return __builtin_bit_cast(float, dpp_pair<st>(__builtin_bit_cast(int, v)));
}
template <int st>
__device__ __forceinline__ uint32_t pair(uint32_t v) { return (uint32_t)dpp_pair<st>((int)v); }
template <int st>
__device__ __forceinline__ double pair(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)dpp_pair<st>((int)(uint32_t)u), hi = (uint32_t)dpp_pair<st>((int)(uint32_t)(u >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
  v += pair<0>(v);
  v += pair<1>(v);
  v += pair<2>(v);
  if constexpr (L == 16) v += pair<3>(v);
  return v;
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
  v = fmaxf(v, pair<0>(v));
  v = fmaxf(v, pair<1>(v));
  v = fmaxf(v, pair<2>(v));
  if constexpr (L == 16) v = fmaxf(v, pair<3>(v));
  return v;
}

// ---- keys that order (logit descending, expert ascending) as one number, so that a compare-exchange
// is a max and a min.  fp32 logits: the double of the same value, whose 29 free mantissa bits take the
// expert (its complement where a larger mantissa means a larger number).  An fp32 number's exponent field is 0 or
// within 0x369 .. 0x47E there, 0x7FF for infinities and NaN: without its bit 0x100 it is 0, 0x269 .. 0x2FF,
// 0x400 .. 0x47E, 0x6FF, in the same order, so that infinities and NaN become numbers as well, a NaN
// (one pattern for all, its sign clear) the largest.  bf16 logits: their rank above the expert, in 32 bits.
template <bool kF32>
struct Key;

// The magnitude's bits on either side of 0x7F800000: an unsigned number in the order of the logits, with -inf
// at 0, both zeros in the middle and +inf at 0xFF000000.  What lies beyond, above (a NaN) or wrapped around
// from below (one with its sign set, what a host's conversion to bf16 writes), becomes the one NaN on top.
template <uint32_t kStep>   // the lowest bit that a logit uses
__device__ __forceinline__ uint32_t rank_of(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v), s = (uint32_t)((int32_t)u >> 31);
  const uint32_t x = ((u & 0x7FFFFFFFu) ^ s) - s + 0x7F800000u;
  return x < 0xFF000000u + kStep ? x : 0xFF000000u + kStep;
}
__device__ __forceinline__ float value_of(uint32_t rank) {
  const uint32_t x = rank - 0x7F800000u, s = (uint32_t)((int32_t)x >> 31);
  return __builtin_bit_cast(float, ((x ^ s) - s) | (s & 0x80000000u));
}
template <>
struct Key<true> {
  using type = double;
  static __device__ __forceinline__ double none() { return -__builtin_huge_val(); }
  static __device__ __forceinline__ double make(float v, int e) {
    const uint32_t w = v != v ? 0x7FC00000u : __builtin_bit_cast(uint32_t, v);
    const double d = (double)(__builtin_bit_cast(float, w) + 0.0f);   // -0 -> +0: equal logits tie
    const uint64_t u = __builtin_bit_cast(uint64_t, d) & ~(1ull << 60);
    return __builtin_bit_cast(double, u | (uint64_t)((u >> 63) ? e : 255 - e));
  }
  static __device__ __forceinline__ int expert(double k) {
    const uint64_t u = __builtin_bit_cast(uint64_t, k);
    const int low = (int)(u & 255u);
    return (u >> 63) ? low : 255 - low;
  }
  static __device__ __forceinline__ float value(double k) {
    const uint64_t u = __builtin_bit_cast(uint64_t, k) & ~(uint64_t)255;
    return (float)__builtin_bit_cast(double, u | (u >> 1 & 1ull << 60));   // (fields with 0x200 had 0x100 as well)
  }
  // (keys are never NaN: the instruction itself, without the quieting that fmax puts before it)
  static __device__ __forceinline__ double hi(double a, double b) {
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
  }
  static __device__ __forceinline__ double lo(double a, double b) {
    double r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
  }
};
template <>
struct Key<false> {
  using type = uint32_t;
  // (no expert: also the key of -inf at expert 255, but of 256 experts none is missing)
  static __device__ __forceinline__ uint32_t none() { return 0u; }
  static __device__ __forceinline__ uint32_t make(float v, int e) { return rank_of<0x10000u>(v) | (uint32_t)(255 - e); }
  static __device__ __forceinline__ int expert(uint32_t k) { return 255 - (int)(k & 255u); }
  static __device__ __forceinline__ float value(uint32_t k) { return value_of(k & 0xFFFF0000u); }
  static __device__ __forceinline__ uint32_t hi(uint32_t a, uint32_t b) { return a > b ? a : b; }
  static __device__ __forceinline__ uint32_t lo(uint32_t a, uint32_t b) { return a < b ? a : b; }
};

// Sorts the bitonic a[0 .. n) descending.
template <class K, int n>
__device__ __forceinline__ void bitonic(typename K::type* a) {
#pragma unroll
  for (int d = n / 2; d >= 1; d /= 2)
#pragma unroll
    for (int i = 0; i < n; ++i)
      if ((i & d) == 0) {
        const typename K::type x = a[i], y = a[i + d];
        a[i] = K::hi(x, y);
        a[i + d] = K::lo(x, y);
      }
}

// a[0 .. n) -> its min(n, kK) largest, descending, in a[0 ..): merge sort whose lists are cut at kK.
template <class K, int n, int kK>
__device__ __forceinline__ void sort_top(typename K::type* a) {
  if constexpr (n > 1) {
    constexpr int h = n / 2, m = h < kK ? h : kK;      // length of each half's list
    sort_top<K, h, kK>(a);
    sort_top<K, h, kK>(a + h);
    if constexpr (2 * m <= kK) {
      // h <= kK / 2: the lists are whole and adjacent
#pragma unroll
      for (int i = 0; i < m; ++i) {
        const typename K::type x = a[i], y = a[2 * m - 1 - i];
        a[i] = K::hi(x, y);
        a[2 * m - 1 - i] = K::lo(x, y);
      }
      bitonic<K, m>(a);
      bitonic<K, m>(a + m);
    } else {
#pragma unroll
      for (int i = 0; i < m; ++i) a[i] = K::hi(a[i], a[h + m - 1 - i]);
      bitonic<K, m>(a);
    }
  }
}

// Merges every lane's descending list a[0 .. M) with its partners', from step st up to the L lanes of
// the token: all of them end with the token's kK largest, descending.
template <class K, int L, int M, int kK, int st>
__device__ __forceinline__ void merge_lanes(typename K::type* a) {
  if constexpr ((1 << st) < L) {
    typename K::type p[M];
#pragma unroll
    for (int i = 0; i < M; ++i) p[i] = pair<st>(a[i]);
    if constexpr (2 * M <= kK) {
#pragma unroll
      for (int i = 0; i < M; ++i) {
        const typename K::type x = a[i], y = p[M - 1 - i];
        a[i] = K::hi(x, y);
        p[M - 1 - i] = K::lo(x, y);
      }
#pragma unroll
      for (int i = 0; i < M; ++i) a[M + i] = p[i];
      bitonic<K, M>(a);
      bitonic<K, M>(a + M);
      merge_lanes<K, L, 2 * M, kK, st + 1>(a);
    } else {
#pragma unroll
      for (int i = 0; i < M; ++i) a[i] = K::hi(a[i], p[M - 1 - i]);
      bitonic<K, M>(a);
      merge_lanes<K, L, M, kK, st + 1>(a);
    }
  }
}

}  // namespace moe
