// The router of a training step for gfx950: top-k routing with per-expert counts, the load-balance
// loss and the router z-loss, and the gradient of all of them with respect to the logits.
//
// With l [T, E] the logits, p = softmax(l) over all E experts, lse = log sum exp l, n the number of
// tokens that count, C_e how many of their k slots went to expert e:
//   topk_prob[t, j] = softmax of the k selected logits
//   L_b = E / (k n^2) sum_e C_e sum_t p[t, e],      L_z = 1/n sum_t lse_t^2       (t that count)
//   d/dl[t, e] = g_b p (f_e - sum_i p_i f_i) + g_z (2/n) lse p,    f_e = E C_e / (k n^2)
//              + sum over j with idx[t, j] = e of w_j (dprob_j - sum_m w_m dprob_m)
// (C_e is a count, so L_b reaches the logits through p alone.)
//
// Both kernels read the logits once.  L lanes (16, or 8 where E <= 8) share a token, lane s holding
// experts s, s + L, ... in registers: the row's statistics, its top-k and its gradient need no second
// read and no LDS, and the lanes of a load cover whole 64-byte pieces of a row for any E.
//
// Measured: forward 131072 x 256 f32, k = 8: 46 us and 4 for the totals, of 28 that its bytes take; the VALU
// issues 76 % of the time, most of it the selection (sorting networks, 16 of a lane's 16 logits into
// lists of 8, four merges); bf16 44 us with the totals, of 15.  256 x 4: 6.4 us, a launch.  Backward
// 131072 x 256 f32: 49 us, 5.6 TB/s; bf16 36.
#include "common.h"
#include "kernels.h"
#include "route_select.h"

namespace moe {
namespace {

// The lane's logits of its token, one of the kG that start at t0, -inf past the last expert.  A buffer
// descriptor over those tokens: the lane's offset is the same for all of them, the experts' 16-lane
// strides are immediate offsets, and a token past the last reads zeros.  (64-bit addresses per load
// were 50 of the forward's 950 instructions a token, which bound it.)
template <bool kF32, int L, int kN, int kG>
__device__ __forceinline__ void load_row(const void* lg, int64_t t0, int64_t T, int E, int grp, int sub,
                                         float (&v)[kN]) {
  constexpr int kB = kF32 ? 4 : 2;
  const int64_t left = T - t0;
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<char*>(reinterpret_cast<const char*>(lg)) + t0 * E * kB, (short)0,
      (int)(left < kG ? left : kG) * E * kB, 0x00020000);
  const uint32_t at = (uint32_t)(grp * E + sub) * kB;
#pragma unroll
  for (int c = 0; c < kN; ++c) {
    if constexpr (kF32) {
      const uint32_t u = __builtin_amdgcn_raw_buffer_load_b32(r, at + c * L * kB, 0, 0);
      v[c] = __builtin_bit_cast(float, u);
    } else {
      v[c] = bf16_to_f32(__builtin_amdgcn_raw_buffer_load_b16(r, at + c * L * kB, 0, 0));
    }
  }
  // E > L kN / 2 (kN > 1): the first half of the chunks is whole
#pragma unroll
  for (int c = kN / 2; c < kN; ++c) v[c] = sub + L * c < E ? v[c] : -__builtin_huge_valf();
}

constexpr int kThreads = kBalanceThreads;

struct FwdP {
  const void* logits;
  const uint8_t* mask;
  int64_t T;
  int E, k;
  int32_t* idx;
  float* prob;
  int32_t* counts;
  float* losses;
  float* psum;       // [nb][E] sums of p, then [nb] sums of lse^2
  int32_t* cnt;      // [nb][E] counts, then [nb] tokens that count
  double* prod;      // [kBalanceFinish] partial sums of C_e P_e
  int* arrived;      // workgroups of the finish that are done; the first kernel clears it
};

// Totals of nb blocks' sums -> counts and both losses, 64-bit from here on.  Workgroup f of nf takes
// experts 16 f + [0, 16) (one workgroup reads 64 bytes a cycle: 512 KB for 256 blocks of 256 experts would
// take 9 us), leaves sum_e C_e P_e of them in `prod`, and the one that arrives last adds those in order.
constexpr int kFinExperts = 16, kFinThreads = 256;
template <int kT>
__device__ __forceinline__ void finish(const FwdP& p, int nb, int nf) {
  constexpr int kS = kT / kFinExperts;                  // slices of the nb rows
  __shared__ double es[kS][kFinExperts];
  __shared__ int ec[kS][kFinExperts];
  __shared__ double wz[kT / 64];
  __shared__ int64_t wn[kT / 64];
  __shared__ int s_last;
  const int tid = threadIdx.x, le = tid % kFinExperts, s = tid / kFinExperts;
  double total = 0.0;
  for (int f = blockIdx.x; f * kFinExperts < p.E; f += nf) {
    const int e = f * kFinExperts + le;
    double ps = 0.0;
    int c = 0;
    if (e < p.E) {
      constexpr int kU = 16;                            // rows in flight
      int b = s;
      for (; b + (kU - 1) * kS < nb; b += kU * kS) {
        float v[kU];
        int w[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          v[u] = p.psum[(int64_t)(b + u * kS) * p.E + e];
          w[u] = p.cnt[(int64_t)(b + u * kS) * p.E + e];
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) { ps += v[u]; c += w[u]; }
      }
      for (; b < nb; b += kS) {
        ps += p.psum[(int64_t)b * p.E + e];
        c += p.cnt[(int64_t)b * p.E + e];
      }
    }
    es[s][le] = ps;
    ec[s][le] = c;
    __syncthreads();
    for (int h = kS / 2; h >= 1; h /= 2) {
      if (s < h) {
        es[s][le] += es[s + h][le];
        ec[s][le] += ec[s + h][le];
      }
      __syncthreads();
    }
    if (tid < kFinExperts) {
      if (e < p.E) p.counts[e] = ec[0][le];
      double q = e < p.E ? es[0][le] * (double)ec[0][le] : 0.0;
#pragma unroll
      for (int d = kFinExperts / 2; d >= 1; d >>= 1) q += __shfl_xor(q, d, 64);
      total += q;
    }
    __syncthreads();
  }
  if (nf > 1) {
    if (tid == 0) {
      // device-wide atomics, each complete before the next: no other write has to be seen
      __hip_atomic_store(p.prod + blockIdx.x, total, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __builtin_amdgcn_s_waitcnt(0);
      s_last = __hip_atomic_fetch_add(p.arrived, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == nf - 1;
    }
    __syncthreads();
    if (!s_last) return;
  }
  double z = 0.0;
  int64_t n = 0;
  for (int b = tid; b < nb; b += kT) {
    z += p.psum[(int64_t)nb * p.E + b];
    n += p.cnt[(int64_t)nb * p.E + b];
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    z += __shfl_xor(z, d, 64);
    n += __shfl_xor(n, d, 64);
  }
  if ((tid & 63) == 0) { wz[tid >> 6] = z; wn[tid >> 6] = n; }
  __syncthreads();
  if (tid == 0) {
    double zz = 0.0;
    int64_t nn = 0;
    for (int w = 0; w < kT / 64; ++w) { zz += wz[w]; nn += wn[w]; }
    if (nf > 1) {
      total = 0.0;
      for (int f = 0; f < nf; ++f) total += __hip_atomic_load(p.prod + f, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    const double dn = nn > 0 ? (double)nn : 1.0;        // nothing counts: both losses are 0
    p.losses[0] = (float)(total * (double)p.E / ((double)p.k * dn * dn));
    p.losses[1] = (float)(zz / dn);
  }
}

// kN experts per lane, lists of kK >= k.  Block b's groups of L lanes take tokens b, b + nb, ... of
// the blocks' stripes; sums over the tokens stay in registers until the block's end.
template <bool kF32, int L, int kN, int kK>
__global__ __launch_bounds__(kThreads) void route_balance_kernel(const FwdP p) {
  using K = Key<kF32>;
  constexpr int kG = kThreads / L;                      // tokens per block at a time
  __shared__ int cnt[kMaxExperts];
  __shared__ float red[kThreads / 64][L * kN];
  __shared__ float zred[kThreads / 64];
  __shared__ int nred[kThreads / 64];
  const int tid = threadIdx.x, sub = tid & (L - 1), grp = tid / L;
  const int E = p.E, k = p.k, nb = gridDim.x;
  if (tid < kMaxExperts) cnt[tid] = 0;
  __syncthreads();
  float acc[kN];
#pragma unroll
  for (int c = 0; c < kN; ++c) acc[c] = 0.f;
  float z = 0.f;
  int nv = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * kG; t0 < p.T; t0 += (int64_t)nb * kG) {
    const int64_t t = t0 + grp;
    const bool in = t < p.T;
    float v[kN];
    load_row<kF32, L, kN, kG>(p.logits, t0, p.T, E, grp, sub, v);
    const bool counts = in && (!p.mask || p.mask[in ? t : p.T - 1] != 0);
    constexpr int kA = kN > kK ? kN : kK;
    typename K::type a[kA];
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      const typename K::type key = K::make(v[c], sub + L * c);
      a[c] = c < kN / 2 || sub + L * c < E ? key : K::none();
    }
    sort_top<K, kN, kK>(a);
    constexpr int kM = kN < kK ? kN : kK;
    merge_lanes<K, L, kM, kK, 0>(a);
    // statistics of the row; its largest logit heads the list
    float m = K::value(a[0]);
    m = m == -__builtin_huge_valf() ? 0.f : m;          // nothing above -inf: every term below is 0
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      v[c] = __expf(v[c] - m);
      s += v[c];
    }
    s = group_sum<L>(s);
    const bool live = s != 0.f;
    // the lane's slot of the list
    typename K::type mine = a[0];
#pragma unroll
    for (int j = 1; j < (kK < L ? kK : L); ++j) mine = sub == j ? a[j] : mine;
    float w = sub < k ? __expf(K::value(mine) - m) : 0.f;
    const float ws = group_sum<L>(w);
    w = live ? w / ws : 0.f;
    if (in && sub < k) {
      const int e = K::expert(mine);
      p.idx[t * k + sub] = e;
      p.prob[t * k + sub] = w;
      if (counts && live) atomicAdd(&cnt[e], 1);
    }
    if (counts && live) {
      const float inv = 1.0f / s;
#pragma unroll
      for (int c = 0; c < kN; ++c) acc[c] += v[c] * inv;
      const float lse = m + __logf(s);
      if (sub == 0) { z += lse * lse; ++nv; }
    }
  }
  // the block's sums: lanes of one wave that hold the same experts, then the waves in order
#pragma unroll
  for (int c = 0; c < kN; ++c) {
#pragma unroll
    for (int d = L; d < 64; d <<= 1) acc[c] += __shfl_xor(acc[c], d, 64);
    if ((tid & 63) < L) red[tid >> 6][sub + L * c] = acc[c];
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    z += __shfl_xor(z, d, 64);
    nv += __shfl_xor(nv, d, 64);
  }
  if ((tid & 63) == 0) { zred[tid >> 6] = z; nred[tid >> 6] = nv; }
  __syncthreads();
  if (tid < E) {
    float q = 0.f;
    for (int w = 0; w < kThreads / 64; ++w) q += red[w][tid];
    p.psum[(int64_t)blockIdx.x * E + tid] = q;
    p.cnt[(int64_t)blockIdx.x * E + tid] = cnt[tid];
  }
  if (tid == 0) {
    float zz = 0.f;
    int n = 0;
    for (int w = 0; w < kThreads / 64; ++w) { zz += zred[w]; n += nred[w]; }
    p.psum[(int64_t)nb * E + blockIdx.x] = zz;
    p.cnt[(int64_t)nb * E + blockIdx.x] = n;
  }
  if (nb == 1) {
    __syncthreads();                                    // (a block sees its own global writes)
    finish<kThreads>(p, 1, 1);
  } else if (blockIdx.x == 0 && tid == 0) {
    *p.arrived = 0;
  }
}

__global__ __launch_bounds__(kFinThreads) void route_balance_finish_kernel(const FwdP p, int nb) {
  finish<kFinThreads>(p, nb, (int)gridDim.x);
}

template <bool kF32, int L, int kN>
void launch_fwd_k(const FwdP& p, int nb, hipStream_t st) {
  if (p.k <= 2) route_balance_kernel<kF32, L, kN, 2><<<nb, kThreads, 0, st>>>(p);
  else if (p.k <= 4) route_balance_kernel<kF32, L, kN, 4><<<nb, kThreads, 0, st>>>(p);
  else if (p.k <= 8) route_balance_kernel<kF32, L, kN, 8><<<nb, kThreads, 0, st>>>(p);
  else if constexpr (L == 16) route_balance_kernel<kF32, L, kN, 16><<<nb, kThreads, 0, st>>>(p);
}

template <bool kF32>
void launch_fwd(const FwdP& p, int nb, hipStream_t st) {
  if (p.E <= 8) launch_fwd_k<kF32, 8, 1>(p, nb, st);
  else if (p.E <= 16) launch_fwd_k<kF32, 16, 1>(p, nb, st);
  else if (p.E <= 32) launch_fwd_k<kF32, 16, 2>(p, nb, st);
  else if (p.E <= 64) launch_fwd_k<kF32, 16, 4>(p, nb, st);
  else if (p.E <= 128) launch_fwd_k<kF32, 16, 8>(p, nb, st);
  else launch_fwd_k<kF32, 16, 16>(p, nb, st);
}

// ---- backward
struct BwdP {
  const void* logits;
  const uint8_t* mask;
  const int32_t* idx;
  const float* prob;
  const int32_t* counts;
  const float* dprob;
  const float* dlosses;
  int64_t T;
  int E, k;
  void* dlogits;
};

constexpr int kBwdThreads = 256;

template <bool kF32, int L, int kN>
__global__ __launch_bounds__(kBwdThreads) void route_balance_bwd_kernel(const BwdP p) {
  constexpr int kG = kBwdThreads / L;
  // the gradients of the k selected weights, at their experts: each group's row is all zeros but for
  // the k entries of its token, which it clears again
  __shared__ float sel[kG][L * kN];
  __shared__ int wsum[kBwdThreads / 64];
  const int tid = threadIdx.x, sub = tid & (L - 1), grp = tid / L;
  const int E = p.E, k = p.k;
  // tokens that count: each put k slots into the counts
  int c0 = tid < E ? p.counts[tid] : 0;
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) c0 += __shfl_xor(c0, d, 64);
  if ((tid & 63) == 0) wsum[tid >> 6] = c0;
#pragma unroll
  for (int c = 0; c < kN; ++c) sel[grp][sub + L * c] = 0.f;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kBwdThreads / 64; ++w) total += wsum[w];
  const double n = total > 0 ? (double)(total / k) : 1.0;
  const float gb = p.dlosses ? p.dlosses[0] : 0.f, gz = p.dlosses ? p.dlosses[1] : 0.f;
  const float cz = (float)(2.0 / n) * gz;
  const double cf = (double)E / ((double)k * n * n);
  float f[kN];                                          // g_b f_e of the lane's experts
#pragma unroll
  for (int c = 0; c < kN; ++c) f[c] = sub + L * c < E ? gb * (float)(cf * (double)p.counts[sub + L * c]) : 0.f;
  for (int64_t t0 = (int64_t)blockIdx.x * kG; t0 < p.T; t0 += (int64_t)gridDim.x * kG) {
    const int64_t t = t0 + grp;
    const bool in = t < p.T;
    const int64_t tr = in ? t : p.T - 1;
    float v[kN], m = -__builtin_huge_valf();
    load_row<kF32, L, kN, kG>(p.logits, t0, p.T, E, grp, sub, v);
    int e_sel = -1;
    float w = 0.f, g = 0.f;
    if (p.dprob && in && sub < k) {
      e_sel = p.idx[tr * k + sub];
      w = p.prob[tr * k + sub];
      g = p.dprob[tr * k + sub];
    }
    const bool counts = !p.mask || p.mask[tr] != 0;
#pragma unroll
    for (int c = 0; c < kN; ++c) m = fmaxf(m, v[c]);
    m = group_max<L>(m);
    m = m == -__builtin_huge_valf() ? 0.f : m;
    float s = 0.f, dot = 0.f;
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      v[c] = __expf(v[c] - m);
      s += v[c];
      dot += v[c] * f[c];
    }
    s = group_sum<L>(s);
    dot = group_sum<L>(dot);
    const bool live = s != 0.f && counts;               // a row without a logit above -inf has no gradient
    const float inv = 1.0f / s;
    dot *= inv;
    const float zl = cz != 0.f ? cz * (m + __logf(s)) : 0.f;
    // w (dprob - sum w dprob) to the selected experts (ids outside [0, E) have none)
    const float wg = group_sum<L>(w * g);
    const bool has = e_sel >= 0 && e_sel < E;
    if (has) atomicAdd(&sel[grp][e_sel], w * (g - wg));
    asm volatile("" ::: "memory");                      // one wave's LDS operations run in order
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      const int e = sub + L * c;
      const float a = live ? v[c] * inv * (f[c] - dot + zl) : 0.f;
      const float d = a + sel[grp][e];
      if (in && e < E) {
        if constexpr (kF32) reinterpret_cast<float*>(p.dlogits)[t * E + e] = d;
        else reinterpret_cast<uint16_t*>(p.dlogits)[t * E + e] = f32_to_bf16(d);
      }
    }
    asm volatile("" ::: "memory");
    if (has) sel[grp][e_sel] = 0.f;
    asm volatile("" ::: "memory");
  }
}

template <bool kF32>
void launch_bwd(const BwdP& p, hipStream_t st) {
  const int L = p.E <= 8 ? 8 : 16;
  const int64_t need = (p.T * L + kBwdThreads - 1) / kBwdThreads;
  // 8 workgroups of 4 waves per CU; of the widest rows' kernel, whose 73 registers leave room for 6, 5: with 8 some
  // would wait for a second turn (131072 x 256 f32: 53.5 us, 49.9 with 5; 5 and 6 are alike: f32 48.9 and 48.5, bf16
  // 35.8 and 36.1; 131072 x 64 bf16: 14.2 us with 8, 14.7 with 5)
  const int64_t most = p.E > 128 ? 1280 : 2048;
  const int nb = (int)(need < most ? need : most);
  if (p.E <= 8) route_balance_bwd_kernel<kF32, 8, 1><<<nb, kBwdThreads, 0, st>>>(p);
  else if (p.E <= 16) route_balance_bwd_kernel<kF32, 16, 1><<<nb, kBwdThreads, 0, st>>>(p);
  else if (p.E <= 32) route_balance_bwd_kernel<kF32, 16, 2><<<nb, kBwdThreads, 0, st>>>(p);
  else if (p.E <= 64) route_balance_bwd_kernel<kF32, 16, 4><<<nb, kBwdThreads, 0, st>>>(p);
  else if (p.E <= 128) route_balance_bwd_kernel<kF32, 16, 8><<<nb, kBwdThreads, 0, st>>>(p);
  else route_balance_bwd_kernel<kF32, 16, 16><<<nb, kBwdThreads, 0, st>>>(p);
}

}  // namespace

int balance_blocks(int64_t T, int E) {
  const int64_t per = kThreads / (E <= 8 ? 8 : 16);
  if (T <= 2 * per) return 1;
  const int64_t nb = (T + per - 1) / per;
  return (int)(nb < kBalanceMaxBlocks ? nb : kBalanceMaxBlocks);
}

hipError_t launch_route_balance(const void* logits, bool f32, const uint8_t* mask, int64_t T, int E, int k,
                                int32_t* idx, float* prob, int32_t* counts, float* losses, float* psum, int32_t* cnt,
                                double* prod, int* arrived, hipStream_t st) {
  const FwdP p{logits, mask, T, E, k, idx, prob, counts, losses, psum, cnt, prod, arrived};
  const int nb = balance_blocks(T, E);
  if (f32) launch_fwd<true>(p, nb, st);
  else launch_fwd<false>(p, nb, st);
  if (nb > 1) route_balance_finish_kernel<<<(E + kFinExperts - 1) / kFinExperts, kFinThreads, 0, st>>>(p, nb);
  return hipGetLastError();
}

hipError_t launch_route_balance_bwd(const void* logits, bool f32, const uint8_t* mask, int64_t T, int E, int k,
                                    const int32_t* idx, const float* prob, const int32_t* counts, const float* dprob,
                                    const float* dlosses, void* dlogits, hipStream_t st) {
  const BwdP p{logits, mask, idx, prob, counts, dprob, dlosses, T, E, k, dlogits};
  if (f32) launch_bwd<true>(p, st);
  else launch_bwd<false>(p, st);
  return hipGetLastError();
}

}  // namespace moe
