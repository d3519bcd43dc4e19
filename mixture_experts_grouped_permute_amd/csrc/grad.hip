// The global norm of many gradients and their clipped copies for gfx950.
//
//   sumsq = sum over all tensors and values of g^2;   c = min(1, max_norm / (sqrt(sumsq) + 1e-6));   out = g c
// Tensors come as a table in the kernel arguments, kGradTable at a launch, each cut into chunks of kChunk values
// that workgroups take in a fixed order.  Squares are summed in 64 bits: one of an fp32 value beyond 2^64 passes
// fp32, and the sum of 10^9 of them would lose its last ones.  Memory bounds both; the 64-bit products fit
// beside the loads several times over.
#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kChunk = 32768;

struct Table {
  const void* g[kGradTable];
  void* out[kGradTable];
  int64_t n[kGradTable];
  int32_t first[kGradTable + 1];       // chunk of the launch that the tensor begins with
  uint8_t kind[kGradTable];            // bit 0: g is fp32, bit 1: out is
  int tensors;
};

__device__ __forceinline__ float value(const void* p, int64_t i, bool f32) {
  return f32 ? reinterpret_cast<const float*>(p)[i] : bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
}

// The tensor that holds chunk c.
__device__ __forceinline__ int tensor_of(const Table& tab, int c) {
  int lo = 0, hi = tab.tensors - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[kThreads / 64];
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
  for (int i = 0; i < kThreads / 64; ++i) v += red[i];
  return v;
}

__global__ __launch_bounds__(kThreads) void grad_sumsq_kernel(const Table tab, double* __restrict__ part) {
  double acc = 0.0;
  const int chunks = tab.first[tab.tensors];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int e = tensor_of(tab, c);
    const int64_t lo = (int64_t)(c - tab.first[e]) * kChunk, n = tab.n[e], hi = lo + kChunk < n ? lo + kChunk : n;
    const bool f32 = tab.kind[e] & 1;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
      const double v = value(tab.g[e], i, f32);
      acc += v * v;
    }
  }
  acc = block_sum(acc);
  if (threadIdx.x == 0) part[blockIdx.x] = acc;
}

__global__ __launch_bounds__(kThreads) void grad_sumsq_finish_kernel(const double* __restrict__ part, int64_t n,
                                                                     double* __restrict__ sumsq) {
  double acc = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) acc += part[i];
  acc = block_sum(acc);
  if (threadIdx.x == 0) *sumsq = acc;
}

__global__ __launch_bounds__(kThreads) void grad_clip_kernel(const Table tab, const double* __restrict__ sumsq, float max_norm,
                                                             float* __restrict__ norm) {
  const double total = sqrt(*sumsq);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)total;
  const double ratio = (double)max_norm / (total + 1e-6);
  const float k = ratio >= 1.0 || max_norm == __builtin_huge_valf() ? 1.0f : (float)ratio;   // (a NaN stays)
  const int chunks = tab.first[tab.tensors];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int e = tensor_of(tab, c);
    if (k == 1.0f && tab.g[e] == tab.out[e]) continue;                 // in place, and nothing to change
    const int64_t lo = (int64_t)(c - tab.first[e]) * kChunk, n = tab.n[e], hi = lo + kChunk < n ? lo + kChunk : n;
    const bool f32 = tab.kind[e] & 1, o32 = tab.kind[e] & 2;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
      const float v = value(tab.g[e], i, f32) * k;
      if (o32) reinterpret_cast<float*>(tab.out[e])[i] = v;
      else reinterpret_cast<uint16_t*>(tab.out[e])[i] = f32_to_bf16(v);
    }
  }
}

// The next table of tensors from *at on, empty ones left out; returns its chunks (0: nothing is left).
int64_t next_table(const GradList& l, int* at, Table* tab) {
  int64_t chunks = 0;
  tab->tensors = 0;
  while (*at < l.n && tab->tensors < kGradTable) {
    const int64_t n = l.numel[*at], add = (n + kChunk - 1) / kChunk;
    if (n > 0) {
      const int e = tab->tensors++;
      tab->g[e] = l.g[*at];
      tab->out[e] = l.out ? l.out[*at] : nullptr;
      tab->n[e] = n;
      tab->kind[e] = (uint8_t)((l.dtype[*at] == 0 ? 1 : 0) | (l.out && l.out_dtype[*at] == 0 ? 2 : 0));
      tab->first[e] = (int32_t)chunks;
      chunks += add;
    }
    ++*at;
  }
  tab->first[tab->tensors] = (int32_t)chunks;
  return chunks;
}

constexpr int kMostBlocks = 2048;
int blocks_of(int64_t chunks) { return (int)(chunks < kMostBlocks ? chunks : kMostBlocks); }

}  // namespace

int64_t grad_parts(const int64_t* numel, int n) {
  int64_t launches = 1, in = 0;
  for (int i = 0; i < n; ++i)
    if (numel[i] > 0 && ++in > kGradTable) {
      ++launches;
      in = 1;
    }
  return launches * kMostBlocks;
}

hipError_t launch_grad_sumsq(const GradList& l, double* part, double* sumsq, hipStream_t st) {
  Table tab;
  int at = 0;
  int64_t parts = 0;
  while (const int64_t chunks = next_table(l, &at, &tab)) {
    const int nb = blocks_of(chunks);
    grad_sumsq_kernel<<<nb, kThreads, 0, st>>>(tab, part + parts);
    parts += nb;
  }
  grad_sumsq_finish_kernel<<<1, kThreads, 0, st>>>(part, parts, sumsq);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const GradList& l, const double* sumsq, float max_norm, float* norm, hipStream_t st) {
  Table tab;
  int at = 0;
  bool first = true;
  while (true) {
    const int64_t chunks = next_table(l, &at, &tab);
    if (!chunks && !first) break;
    const int nb = blocks_of(chunks);
    grad_clip_kernel<<<nb > 0 ? nb : 1, kThreads, 0, st>>>(tab, sumsq, max_norm, first ? norm : nullptr);
    first = false;
  }
  return hipGetLastError();
}

}  // namespace moe
