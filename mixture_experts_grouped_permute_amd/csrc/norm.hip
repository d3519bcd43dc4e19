// Residual addition and root-mean-square norm for gfx950, forward and backward.
//
//   s = x + r, rounded to the type of x: the sum as the residual stream carries it, and what is normalized
//   y[t, h] = s[t, h] rstd[t] w[h],   rstd[t] = 1 / sqrt(mean_h s[t, h]^2 + eps)
//   codes and scales: E4M3 with one fp32 scale per 128 columns (block_scale.h) of the fp32 y, not of the rounded one
// Gradient, xh = s rstd and g = dy w:
//   dx = rstd (g - xh mean_h(g xh)) + ds,    dw[h] = sum_t dy xh
// rstd is formed again from s, which the backward reads anyway.
#include "common.h"
#include "kernels.h"
#include "block_scale.h"

namespace moe {
namespace {

template <bool kF32>
__device__ __forceinline__ float get(const void* p, int64_t i) {
  if constexpr (kF32) return reinterpret_cast<const float*>(p)[i];
  else return bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
}
template <bool kF32>
__device__ __forceinline__ void put(void* p, int64_t i, float v) {
  if constexpr (kF32) reinterpret_cast<float*>(p)[i] = v;
  else reinterpret_cast<uint16_t*>(p)[i] = f32_to_bf16(v);
}
template <bool kF32>
__device__ __forceinline__ float sum_at(const NormFwd& p, int64_t i) {
  const float v = get<kF32>(p.x, i);
  if (!p.residual) return v;
  const float a = v + get<kF32>(p.residual, i);
  if constexpr (kF32) return a;
  else return bf16_to_f32(f32_to_bf16(a));
}

// The sum over a workgroup of 256, in every thread.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return red[0] + red[1] + red[2] + red[3];
}

// A workgroup takes a row.
template <bool kF32, bool kW32>
__global__ __launch_bounds__(256) void add_rmsnorm_kernel(const NormFwd p) {
  __shared__ float red[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    const int64_t at = t * p.H;
    float sq = 0.f;
    for (int64_t h = tid; h < p.H; h += 256) {
      const float v = sum_at<kF32>(p, at + h);
      sq += v * v;
    }
    const float rstd = 1.0f / sqrtf(block_sum(sq, red) / (float)p.H + p.eps);
    // a wave takes 128 columns at a time: what one scale covers (all reads of x and r ahead of the sum's writes)
    for (int64_t b = wave; b * 128 < p.H; b += 4) {
      float v[2];
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t h = b * 128 + 2 * lane + i;
        v[i] = 0.f;
        if (h < p.H) {
          const float s = sum_at<kF32>(p, at + h);
          if (p.sum) put<kF32>(p.sum, at + h, s);
          v[i] = s * rstd * get<kW32>(p.weight, h);
          if (p.y) put<kF32>(p.y, at + h, v[i]);
        }
        m = umax(m, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
      }
      if (p.q) {
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) m = umax(m, (uint32_t)__shfl_xor((int)m, d, 64));
        const BlockScale s = block_scale(m);
        const uint32_t c = codes2<false>(v[0], v[1], s.factor, 0u);
        reinterpret_cast<uint16_t*>(p.q)[(at + b * 128) / 2 + lane] = (uint16_t)c;
        if (lane == 0) p.scales[b * p.T + t] = s.d;
      }
    }
  }
}

// dx, and rstd for the weight's gradient.
template <bool kF32, bool kW32>
__global__ __launch_bounds__(256) void rmsnorm_dx_kernel(const NormBwd p) {
  __shared__ float red[4];
  const int tid = threadIdx.x;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
    const int64_t at = t * p.H;
    float sq = 0.f, dot = 0.f;
    for (int64_t h = tid; h < p.H; h += 256) {
      const float s = get<kF32>(p.s, at + h);
      sq += s * s;
      dot += s * get<kF32>(p.dy, at + h) * get<kW32>(p.weight, h);
    }
    const float rstd = 1.0f / sqrtf(block_sum(sq, red) / (float)p.H + p.eps);
    const float mean = block_sum(dot, red) * rstd / (float)p.H;         // of g xh
    for (int64_t h = tid; h < p.H; h += 256) {
      const float xh = get<kF32>(p.s, at + h) * rstd, g = get<kF32>(p.dy, at + h) * get<kW32>(p.weight, h);
      float d = rstd * (g - xh * mean);
      if (p.dsum) d += get<kF32>(p.dsum, at + h);
      put<kF32>(p.dx, at + h, d);
    }
    if (tid == 0) p.part[t] = rstd;
  }
}

// dw of 64 columns by a workgroup: 4 waves take every fourth row.
template <bool kF32>
__global__ __launch_bounds__(256) void rmsnorm_dw_kernel(const NormBwd p) {
  __shared__ float red[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t h = (int64_t)blockIdx.x * 64 + lane;
  double sum = 0.0;
  if (h < p.H)
    for (int64_t t = wave; t < p.T; t += 4)
      sum += get<kF32>(p.dy, t * p.H + h) * (get<kF32>(p.s, t * p.H + h) * p.part[t]);
  red[wave][lane] = (float)sum;
  __syncthreads();
  if (wave == 0 && h < p.H) p.dw[h] = red[0][lane] + red[1][lane] + red[2][lane] + red[3][lane];
}

}  // namespace

size_t norm_bwd_part_bytes(int64_t T, int64_t H) { return (size_t)T * sizeof(float); }

hipError_t launch_add_rmsnorm(const NormFwd& p, bool f32, bool w32, hipStream_t st) {
  const int nb = (int)(p.T < 4096 ? p.T : 4096);
  if (f32 && w32) add_rmsnorm_kernel<true, true><<<nb, 256, 0, st>>>(p);
  else if (f32) add_rmsnorm_kernel<true, false><<<nb, 256, 0, st>>>(p);
  else if (w32) add_rmsnorm_kernel<false, true><<<nb, 256, 0, st>>>(p);
  else add_rmsnorm_kernel<false, false><<<nb, 256, 0, st>>>(p);
  return hipGetLastError();
}

hipError_t launch_rmsnorm_bwd(const NormBwd& p, bool f32, bool w32, hipStream_t st) {
  const int nb = (int)(p.T < 4096 ? p.T : 4096);
  if (f32 && w32) rmsnorm_dx_kernel<true, true><<<nb, 256, 0, st>>>(p);
  else if (f32) rmsnorm_dx_kernel<true, false><<<nb, 256, 0, st>>>(p);
  else if (w32) rmsnorm_dx_kernel<false, true><<<nb, 256, 0, st>>>(p);
  else rmsnorm_dx_kernel<false, false><<<nb, 256, 0, st>>>(p);
  const unsigned cols = (unsigned)((p.H + 63) / 64);
  if (f32) rmsnorm_dw_kernel<true><<<cols, 256, 0, st>>>(p);
  else rmsnorm_dw_kernel<false><<<cols, 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace moe
