// The global norm of many gradients and their clipped copies for gfx950.
//
//   sumsq = sum over all tensors and values of g^2;   c = min(1, max_norm / (sqrt(sumsq) + 1e-6));   out = g c
// Squares are summed in 64 bits: one of an fp32 value beyond 2^64 passes fp32, and the sum of 10^9 of them would lose
// its last ones.  Memory bounds both passes; the 64-bit products fit beside the loads several times over.
//
// Tensors come as a table in the kernel arguments (which end at 4 KB), each cut into chunks of 8192 values: what a
// workgroup's 256 threads have in flight at once.  Workgroups take the chunks in a fixed order, so that the sum does
// not change from call to call.  A thread keeps the tensors' first chunks in registers, so that finding a chunk's
// tensor is a vote of the wave and not a search through memory.
//
// Measured: 554M fp32 values into bf16 947 us -- 355 for the sum, 6.2 TB/s, and 590 for the scaling, 5.6 TB/s; 200
// tensors with 32M values of both types into fp32 64 us, 27 and 38 (71 with 64-bit addresses, of which a table with
// outputs holds 176: 27 and 33 + 12 in two launches); 300 of up to 5000 values 22 (25).
#include "common.h"
#include "kernels.h"
#include "eight.h"

#include <type_traits>

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192, kPieces = kChunk / (8 * kThreads);
constexpr int kSumTable = 312, kClipTable = 216;
constexpr uint64_t kF32Bit = 1ull << 47;                // in a table's address: fp32 values (else bf16)

// Addresses in 48 bits (a process has 47), so that a launch takes a quarter more tensors; all in whole words, which are
// read as scalars.
template <int kTensors, bool kOut>
struct Table {
  uint32_t g[kTensors], g_last[kTensors];                // lower word; upper 16 bits, and << 16 the values of the last chunk
  uint32_t out[kOut ? kTensors : 1], out_up[kOut ? kTensors / 2 : 1];   // lower word; upper 16 bits, two in a word
  int32_t first[kTensors + 1];         // chunk of the launch that the tensor begins with
  int tensors;
  __device__ __forceinline__ uint64_t grad(int e) const { return g[e] | (uint64_t)(g_last[e] & 0xFFFFu) << 32; }
  __device__ __forceinline__ uint64_t to(int e) const {
    return out[e] | (uint64_t)(out_up[e / 2] >> 16 * (e & 1) & 0xFFFFu) << 32;
  }
  __device__ __forceinline__ int last(int e) const { return (int)(g_last[e] >> 16); }
  void set(int e, uint64_t a, int values) {
    g[e] = (uint32_t)a;
    g_last[e] = (uint32_t)(a >> 32) | (uint32_t)values << 16;
  }
  void set_out(int e, uint64_t a) {
    const uint32_t up = (uint32_t)(a >> 32);
    out[e] = (uint32_t)a;
    out_up[e / 2] = e & 1 ? out_up[e / 2] | up << 16 : up;
  }
};
static_assert(sizeof(Table<kSumTable, false>) <= 4000 && sizeof(Table<kClipTable, true>) <= 4000, "kernel arguments");

// A chunk: its tensor, its first value and how many it has.
struct Chunk {
  int e;
  int64_t at;
  int n;
};
template <int kTensors, bool kOut>
struct Finder {
  static constexpr int kR = (kTensors + 63) / 64;
  int first[kR];
  __device__ __forceinline__ explicit Finder(const Table<kTensors, kOut>& t) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const int e = lane + 64 * i;
      first[i] = e < t.tensors ? t.first[e] : INT32_MAX;
    }
  }
  __device__ __forceinline__ Chunk find(const Table<kTensors, kOut>& t, int c) const {
    int e = -1;
#pragma unroll
    for (int i = 0; i < kR; ++i) e += __popcll(__ballot(first[i] <= c));
    const int k = c - t.first[e];
    return {e, (int64_t)k * kChunk, c + 1 == t.first[e + 1] ? t.last(e) : kChunk};
  }
};

// Piece u of a thread's chunk: values (u kThreads + tid) 8 .. + 8, `n` of the chunk.
template <bool kF32, bool kOnce, class F>
__device__ __forceinline__ void for_pieces(const void* base, int64_t at, int n, F&& f) {
  Eight<kF32, false> v[kPieces];
  if (n == kChunk) {
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int64_t i = at + (u * kThreads + threadIdx.x) * 8;
      if constexpr (kOnce) v[u].load_once(base, i);
      else v[u].load(base, i);
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) f(v[u], (u * kThreads + (int)threadIdx.x) * 8, 8);
  } else {
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int i = (u * kThreads + (int)threadIdx.x) * 8, left = n - i;
      v[u].zero();
      if (left >= 8) v[u].load(base, at + i);
      else if (left > 0) v[u].load_some(base, at + i, left);
      if (left > 0) f(v[u], i, left < 8 ? left : 8);
    }
  }
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

template <bool kOnce>
__global__ __launch_bounds__(kThreads) void grad_sumsq_kernel(const Table<kSumTable, false> tab, double* __restrict__ part) {
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  const auto add = [&](const auto& v, int, int) {       // (what is past the end is zero)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double d = v.at(j);
      acc[j & 3] = __builtin_fma(d, d, acc[j & 3]);
    }
  };
  const Finder<kSumTable, false> finder(tab);
  const int chunks = tab.first[tab.tensors];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const Chunk k = finder.find(tab, c);
    const uint64_t g = tab.grad(k.e);
    const void* base = reinterpret_cast<const void*>(g & ~kF32Bit);
    if (g & kF32Bit) for_pieces<true, kOnce>(base, k.at, k.n, add);
    else for_pieces<false, kOnce>(base, k.at, k.n, add);
  }
  const double sum = block_sum((acc[0] + acc[1]) + (acc[2] + acc[3]));
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__device__ __forceinline__ double sum_parts(const double* __restrict__ part, int64_t n) {
  double acc = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) acc += part[i];
  return block_sum(acc);
}
__global__ __launch_bounds__(kThreads) void grad_sumsq_finish_kernel(const double* __restrict__ part, int64_t n,
                                                                     double* __restrict__ sumsq) {
  const double acc = sum_parts(part, n);
  if (threadIdx.x == 0) *sumsq = acc;
}

// kTensors, kOut: the table's; without outputs of their own the gradients are scaled in place.
template <bool kOnce, int kTensors, bool kOut>
__global__ __launch_bounds__(kThreads) void grad_clip_kernel(const Table<kTensors, kOut> tab, const double* __restrict__ sumsq,
                                                             int parts, float max_norm, float* __restrict__ norm) {
  const double total = sqrt(parts == 1 ? *sumsq : sum_parts(sumsq, parts));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)total;
  const double ratio = (double)max_norm / (total + 1e-6);
  // (a NaN total stays one, also without a limit)
  const float by = ratio >= 1.0 || (max_norm == __builtin_huge_valf() && total == total) ? 1.0f : (float)ratio;
  const Finder<kTensors, kOut> finder(tab);
  const int chunks = tab.first[tab.tensors];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const Chunk k = finder.find(tab, c);
    const uint64_t g = tab.grad(k.e), o = kOut ? tab.to(kOut ? k.e : 0) : g;
    if (by == 1.0f && g == o) continue;                 // in place, and nothing to change
    const void* base = reinterpret_cast<const void*>(g & ~kF32Bit);
    void* to = reinterpret_cast<void*>(o & ~kF32Bit);
    const auto scale = [&](auto f32, auto o32) {
      for_pieces<decltype(f32)::value, kOnce>(base, k.at, k.n, [&](const auto& v, int i, int n) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = v.at(j) * by;
        Eight<decltype(o32)::value, false> e;
        e.set(x);
        if (n == 8) e.template store<kOnce>(to, k.at + i);
        else e.store_some(to, k.at + i, n);
      });
    };
    const std::true_type yes;
    const std::false_type no;
    if (g & kF32Bit) {
      if (o & kF32Bit) scale(yes, yes);
      else scale(yes, no);
    } else {
      if (o & kF32Bit) scale(no, yes);
      else scale(no, no);
    }
  }
}

uint64_t entry(const void* p, int dtype) { return reinterpret_cast<uint64_t>(p) | (dtype == 0 ? kF32Bit : 0); }

// The next table of tensors from *at on, empty ones left out; returns its chunks (0: nothing is left).
template <int kTensors, bool kOut>
int next_table(const GradList& l, int* at, Table<kTensors, kOut>* tab) {
  int64_t chunks = 0;
  int e = 0;
  for (; *at < l.n && e < kTensors; ++*at) {
    const int i = *at;
    const int64_t n = l.numel[i];
    if (n == 0) continue;
    tab->set(e, entry(l.g[i], l.dtype[i]), (int)((n - 1) % kChunk) + 1);
    if constexpr (kOut) tab->set_out(e, entry(l.out[i], l.out_dtype[i]));
    tab->first[e] = (int32_t)chunks;
    chunks += (n - 1) / kChunk + 1;
    ++e;
  }
  tab->first[e] = (int32_t)chunks;
  tab->tensors = e;
  return (int)chunks;
}

constexpr int kSumBlocks = 1024, kClipBlocks = 2048;

// Whether the gradients are more than the last cache (256 MB) holds, so that none is left in it for the clipping: both
// passes then go past the caches (1.4 GB + 0.7 GB in fp32 into bf16: 948 us instead of 1000; 96 MB of 200 tensors 3 us
// less through the caches).
bool past_caches(const GradList& l) {
  double bytes = 0.0;
  for (int i = 0; i < l.n; ++i) bytes += (double)l.numel[i] * (l.dtype[i] == 0 ? 4 : 2);
  return bytes > 256e6;
}

}  // namespace

int64_t grad_parts(const int64_t* numel, int n) {
  int64_t launches = 1, in = 0;
  for (int i = 0; i < n; ++i)
    if (numel[i] > 0 && ++in > kSumTable) {
      ++launches;
      in = 1;
    }
  return launches * kSumBlocks + 1;
}

namespace {
// Sums of squares of the workgroups; how many of them.
int64_t launch_parts(const GradList& l, double* part, hipStream_t st) {
  Table<kSumTable, false> tab;
  const bool once = past_caches(l);
  int at = 0;
  int64_t parts = 0;
  while (const int chunks = next_table(l, &at, &tab)) {
    const int nb = chunks < kSumBlocks ? chunks : kSumBlocks;
    if (once) grad_sumsq_kernel<true><<<nb, kThreads, 0, st>>>(tab, part + parts);
    else grad_sumsq_kernel<false><<<nb, kThreads, 0, st>>>(tab, part + parts);
    parts += nb;
  }
  return parts;
}

template <int kTensors, bool kOut>
void launch_scaled(const GradList& l, const double* sumsq, int parts, float max_norm, float* norm, hipStream_t st) {
  Table<kTensors, kOut> tab;
  const bool once = past_caches(l);
  int at = 0;
  bool first = true;
  while (true) {
    const int chunks = next_table(l, &at, &tab);
    if (!chunks && !first) break;                       // (with nothing but empty tensors: the norm alone)
    const int nb = chunks < kClipBlocks ? chunks : kClipBlocks, grid = nb > 0 ? nb : 1;
    float* to = first ? norm : nullptr;
    if (once) grad_clip_kernel<true, kTensors, kOut><<<grid, kThreads, 0, st>>>(tab, sumsq, parts, max_norm, to);
    else grad_clip_kernel<false, kTensors, kOut><<<grid, kThreads, 0, st>>>(tab, sumsq, parts, max_norm, to);
    first = false;
  }
}
}  // namespace

hipError_t launch_grad_sumsq(const GradList& l, double* part, double* sumsq, hipStream_t st) {
  const int64_t parts = launch_parts(l, part, st);
  grad_sumsq_finish_kernel<<<1, kThreads, 0, st>>>(part, parts, sumsq);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const GradList& l, const double* sumsq, double* part, float max_norm, float* norm, hipStream_t st) {
  int64_t parts = 1;
  if (!sumsq) {
    // each workgroup adds the parts of one launch up by itself, 8 KB of them, in place of a launch that does it (4.7 us
    // for 200 tensors); more are added up once
    parts = launch_parts(l, part, st);
    sumsq = part;
    if (parts > kSumBlocks || parts == 0) {
      double* total = part + grad_parts(l.numel, l.n) - 1;
      grad_sumsq_finish_kernel<<<1, kThreads, 0, st>>>(part, parts, total);
      sumsq = total;
      parts = 1;
    }
  }
  bool in_place = true;
  for (int i = 0; i < l.n; ++i) in_place &= l.numel[i] == 0 || (l.g[i] == l.out[i] && l.dtype[i] == l.out_dtype[i]);
  // (312 tensors a launch in place, 216 with outputs of their own)
  if (in_place) launch_scaled<kSumTable, false>(l, sumsq, (int)parts, max_norm, norm, st);
  else launch_scaled<kClipTable, true>(l, sumsq, (int)parts, max_norm, norm, st);
  return hipGetLastError();
}

}  // namespace moe
