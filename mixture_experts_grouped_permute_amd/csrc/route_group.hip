// Routing by sigmoid or softmax scores with a selection bias and expert groups for gfx950, and its gradient.
//
// With l [T, E] the logits, s = sigmoid(l) or softmax(l) over all experts, c = s + b (-inf where l is):
//   the G groups of n = E / G consecutive experts are ordered by the sum of their `best` (1 or 2) largest c, the
//   kg best stay (equal sums: lower group), experts of the others have c = -inf;
//   idx = the k largest c (equal: lower id);  w_j = s[idx_j], 0 where c is -inf, divided by their sum if
//   renormalised (0 if that is 0), times scale.
// The order is that of 64-bit values, so that it does not hang on how an exponential rounds.
//
// Gradient, g = dprob and w = prob: with S_j = (1 - s_j) for sigmoid and 1 for softmax scores,
//   renormalised:  dl[idx_j] = S_j w_j (g_j - sum_m w_m g_m / scale), else 0
//   not:           dl[idx_j] = S_j w_j g_j, and for softmax scores also -p_e sum_m w_m g_m at every expert.
#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kWaves = 4;

// A number in the order of the doubles: -inf lowest, both zeros equal, every NaN on top.
__device__ __forceinline__ uint64_t order_of(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
  if (v != v) return ~0ull;
  return (u >> 63) ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double shfl_f64(double v, int src) { return __shfl(v, src, 64); }
__device__ __forceinline__ uint64_t shfl_u64(uint64_t v, int src) {
  return (uint64_t)__shfl((unsigned long long)v, src, 64);
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

template <bool kF32>
__device__ __forceinline__ float logit(const void* lg, int64_t at) {
  if constexpr (kF32) return reinterpret_cast<const float*>(lg)[at];
  else return bf16_to_f32(reinterpret_cast<const uint16_t*>(lg)[at]);
}

// One token by one wave, in 64 bits throughout: lane i holds experts i, i + 64, ..; cs: E doubles of the wave's.
// Returns the lane's slot (lane < k).
struct Slot {
  int e;
  float w;
};
template <bool kF32>
__device__ __noinline__ Slot route_token(const GroupRoute& p, int64_t t, int lane, double* cs) {
  constexpr int kC = kMaxExperts / 64;
  const double none = -__builtin_huge_val();
  double s[kC];
  uint64_t key[kC];
  bool out[kC];                                         // -inf: no weight
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const int e = lane + 64 * c;
    s[c] = e < p.E ? (double)logit<kF32>(p.logits, t * p.E + e) : none;
    out[c] = s[c] == none;
  }
  if (p.sigmoid) {
#pragma unroll
    for (int c = 0; c < kC; ++c) s[c] = 1.0 / (1.0 + exp(-s[c]));
  } else {
    double m = none;
#pragma unroll
    for (int c = 0; c < kC; ++c) m = fmax(m, s[c]);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) m = fmax(m, __shfl_xor(m, d, 64));
    if (m == none) m = 0.0;
    double total = 0.0;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      s[c] = exp(s[c] - m);
      total += s[c];
    }
    total = wave_sum(total);
#pragma unroll
    for (int c = 0; c < kC; ++c) s[c] = total == 0.0 ? 0.0 : s[c] / total;
  }
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const int e = lane + 64 * c;
    double v = s[c] + (p.bias && e < p.E ? (double)p.bias[e] : 0.0);
    if (out[c]) v = none;
    out[c] = v == none;
    key[c] = order_of(v);
    if (p.G > 1 && e < p.E) cs[e] = v;
  }
  if (p.G > 1) {
    const int n = p.E / p.G;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    uint64_t mine = 0;
    if (lane < p.G) {
      double a = none, b = none;                        // the two largest
      uint64_t ka = 0, kb = 0;
      for (int i = 0; i < n; ++i) {
        const double v = cs[lane * n + i];
        const uint64_t kv = order_of(v);
        if (i == 0 || kv > ka) {
          b = a; kb = ka;
          a = v; ka = kv;
        } else if (kv > kb) {
          b = v; kb = kv;
        }
      }
      mine = order_of(p.best == 2 ? a + b : a);
    }
    int rank = 0;
    for (int h = 0; h < p.G; ++h) {
      const uint64_t o = shfl_u64(mine, h);
      rank += o > mine || (o == mine && h < lane);
    }
    const uint64_t kept = __ballot(lane < p.G && rank < p.kg);
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int e = lane + 64 * c;
      if (e < p.E && !(kept >> (e / n) & 1)) {
        key[c] = order_of(none);
        out[c] = true;
      }
    }
  }
  // k times the largest; a lane's own experts rise with c
  unsigned gone = 0;
#pragma unroll
  for (int c = 0; c < kC; ++c)
    if (lane + 64 * c >= p.E) gone |= 1u << c;
  Slot r{0, 0.f};
  double w = 0.0;
  for (int j = 0; j < p.k; ++j) {
    uint64_t bk = 0;
    int be = kMaxExperts;
    double bs = 0.0;
#pragma unroll
    for (int c = 0; c < kC; ++c)
      if (!(gone >> c & 1) && (be == kMaxExperts || key[c] > bk)) {
        bk = key[c];
        be = lane + 64 * c;
        bs = out[c] ? 0.0 : s[c];
      }
    uint64_t tk = bk;
    int te = be;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
      const uint64_t ok = (uint64_t)__shfl_xor((unsigned long long)tk, d, 64);
      const int oe = __shfl_xor(te, d, 64);
      if (oe < kMaxExperts && (te == kMaxExperts || ok > tk || (ok == tk && oe < te))) {
        tk = ok;
        te = oe;
      }
    }
    const double sel = shfl_f64(bs, te & 63);           // (the owner's best is the wave's)
    if ((te & 63) == lane) gone |= 1u << (te >> 6);
    if (lane == j) {
      r.e = te;
      w = sel;
    }
  }
  if (p.renorm) {
    const double total = wave_sum(w);
    w = total == 0.0 ? 0.0 : w / total;
  }
  r.w = (float)(w * (double)p.scale);
  return r;
}

template <bool kF32>
__global__ __launch_bounds__(64 * kWaves) void route_group_kernel(const GroupRoute p) {
  __shared__ double cs[kWaves][kMaxExperts];
  __shared__ int cnt[kMaxExperts];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid < kMaxExperts) cnt[tid] = 0;
  __syncthreads();
  for (int64_t t = (int64_t)blockIdx.x * kWaves + wave; t < p.T; t += (int64_t)gridDim.x * kWaves) {
    const Slot s = route_token<kF32>(p, t, lane, cs[wave]);
    if (lane < p.k) {
      p.idx[t * p.k + lane] = s.e;
      p.prob[t * p.k + lane] = s.w;
      if (p.counts && (!p.mask || p.mask[t] != 0)) atomicAdd(&cnt[s.e], 1);
    }
  }
  if (p.counts) {
    __syncthreads();
    int32_t* to = gridDim.x == 1 ? p.counts : p.part + (int64_t)blockIdx.x * p.E;
    if (tid < p.E) to[tid] = cnt[tid];
  }
}

// counts[e] = sum over the nb blocks; a workgroup takes 16 experts.
__global__ __launch_bounds__(256) void route_counts_kernel(const int32_t* __restrict__ part, int nb, int E,
                                                           int32_t* __restrict__ counts) {
  __shared__ int red[16][16];
  const int le = threadIdx.x & 15, s = threadIdx.x >> 4, e = blockIdx.x * 16 + le;
  int c = 0;
  if (e < E)
    for (int b = s; b < nb; b += 16) c += part[(int64_t)b * E + e];
  red[s][le] = c;
  __syncthreads();
  if (s == 0 && e < E) {
    for (int i = 1; i < 16; ++i) c += red[i][le];
    counts[e] = c;
  }
}

// ---- backward: a wave takes a token.
template <bool kF32>
__global__ __launch_bounds__(64 * kWaves) void route_group_bwd_kernel(const GroupRouteBwd p) {
  __shared__ float row[kWaves][kMaxExperts];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int64_t t = (int64_t)blockIdx.x * kWaves + wave; t < p.T; t += (int64_t)gridDim.x * kWaves) {
    int e = -1;
    float w = 0.f, g = 0.f;
    if (lane < p.k) {
      e = p.idx[t * p.k + lane];
      w = p.prob[t * p.k + lane];
      g = p.dprob[t * p.k + lane];
    }
    float sum = w * g;
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, 64);   // (k <= 16; in the first 16 lanes)
    sum = __shfl(sum, 0, 64);
    float d = w * (p.renorm ? g - sum / p.scale : g);
    const bool has = e >= 0 && e < p.E;
    if (p.sigmoid && has) d *= 1.0f / (1.0f + expf(logit<kF32>(p.logits, t * p.E + e)));
    float p_scale = 0.f, m = 0.f;
    if (!p.sigmoid && !p.renorm) {
      m = -__builtin_huge_valf();
      for (int i = lane; i < p.E; i += 64) m = fmaxf(m, logit<kF32>(p.logits, t * p.E + i));
#pragma unroll
      for (int x = 32; x >= 1; x >>= 1) m = fmaxf(m, __shfl_xor(m, x, 64));
      if (m == -__builtin_huge_valf()) m = 0.f;
      float s = 0.f;
      for (int i = lane; i < p.E; i += 64) s += expf(logit<kF32>(p.logits, t * p.E + i) - m);
#pragma unroll
      for (int x = 32; x >= 1; x >>= 1) s += __shfl_xor(s, x, 64);
      p_scale = s == 0.f ? 0.f : -sum / s;
    }
    for (int i = lane; i < p.E; i += 64) {
      float v = 0.f;
      if (!p.sigmoid && !p.renorm) v = p_scale * expf(logit<kF32>(p.logits, t * p.E + i) - m);
      row[wave][i] = v;
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    for (int j = 0; j < p.k; ++j) {                     // in the slots' order, also where an id repeats
      if (lane == j && has) row[wave][e] += d;
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    for (int i = lane; i < p.E; i += 64) {
      const float v = row[wave][i];
      if constexpr (kF32) reinterpret_cast<float*>(p.dlogits)[t * p.E + i] = v;
      else reinterpret_cast<uint16_t*>(p.dlogits)[t * p.E + i] = f32_to_bf16(v);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

}  // namespace

int route_group_blocks(int64_t T) {
  const int64_t nb = (T + kWaves - 1) / kWaves;
  return (int)(nb < kGroupMaxBlocks ? nb : kGroupMaxBlocks);
}

hipError_t launch_route_group(const GroupRoute& p, bool f32, hipStream_t st) {
  const int nb = route_group_blocks(p.T);
  if (f32) route_group_kernel<true><<<nb, 64 * kWaves, 0, st>>>(p);
  else route_group_kernel<false><<<nb, 64 * kWaves, 0, st>>>(p);
  if (p.counts && nb > 1) route_counts_kernel<<<(p.E + 15) / 16, 256, 0, st>>>(p.part, nb, p.E, p.counts);
  return hipGetLastError();
}

hipError_t launch_route_group_bwd(const GroupRouteBwd& p, bool f32, hipStream_t st) {
  const int64_t nb = (p.T + kWaves - 1) / kWaves;
  const int grid = (int)(nb < 2048 ? nb : 2048);
  if (f32) route_group_bwd_kernel<true><<<grid, 64 * kWaves, 0, st>>>(p);
  else route_group_bwd_kernel<false><<<grid, 64 * kWaves, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace moe
