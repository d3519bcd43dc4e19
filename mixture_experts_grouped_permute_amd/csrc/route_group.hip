// Routing by sigmoid or softmax scores with a selection bias and expert groups for gfx950, and its gradient.
//
// With l [T, E] the logits, s = sigmoid(l) or softmax(l) over all experts, c = s + b (-inf where l is):
//   the G groups of n = E / G consecutive experts are ordered by the sum of their `best` (1 or 2) largest c, the
//   kg best stay (equal sums: lower group), experts of the others have c = -inf;
//   idx = the k largest c (equal: lower id);  w_j = s[idx_j], 0 where c is -inf, divided by their sum if
//   renormalised (0 if that is 0), times scale.  (0 as 64-bit numbers are: a sigmoid below l = -709.78.)
// Without a bias experts are ordered by their logits, as their scores are, and groups of one best by their best's; else
// c and the sums are compared as 64-bit values, so that the order does not hang on how an exponential rounds.
//
// Gradient, g = dprob and w = prob: with S_j = (1 - s_j) for sigmoid and 1 for softmax scores,
//   renormalised:  dl[idx_j] = S_j w_j (g_j - sum_m w_m g_m / scale), else 0
//   not:           dl[idx_j] = S_j w_j g_j, and for softmax scores also -p_e sum_m w_m g_m at every expert.
//
// Forward: 16 lanes share a token; a group's experts lie with 16 / (power of two >= G) of them.  Scores are fp32
// first: their error is known, and where two numbers whose order counts are nearer than that -- neighbours in the list,
// the last one in and the first one out, the last group in and the first one out -- the token is done again in 64 bits
// (one of 460 with sigmoids of fp32 logits, a bias and 8 groups of 256 experts; of softmax scores with a bias far more).
#include "common.h"
#include "kernels.h"
#include "eight.h"
#include "route_select.h"

namespace moe {
namespace {

constexpr int kWaves = 4, kTokens = 4 * kWaves;         // tokens of a workgroup at a time
constexpr float kNone = -__builtin_huge_valf();
// The least logit whose sigmoid 1 / (1 + exp(-l)) is not 0 in 64 bits: -709.7827, the largest double's logarithm, cut to fp32.
constexpr float kLeast = -0x1.62e42ep9f;

// A number in the order of the doubles: -inf lowest, both zeros equal, every NaN on top.
__device__ __forceinline__ uint64_t order_of(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
  if (v != v) return ~0ull;
  return (u >> 63) ? ~u : u | 1ull << 63;
}
// A lane's value, in all of them (the lane is the same for all).
__device__ __forceinline__ int from_lane(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ uint64_t from_lane(uint64_t v, int lane) {
  return (uint64_t)(uint32_t)from_lane((int)(uint32_t)(v >> 32), lane) << 32 | (uint32_t)from_lane((int)(uint32_t)v, lane);
}
__device__ __forceinline__ double from_lane(double v, int lane) {
  return __builtin_bit_cast(double, from_lane(__builtin_bit_cast(uint64_t, v), lane));
}
template <int st>
__device__ __forceinline__ uint64_t pair64(uint64_t v) {
  return (uint64_t)(uint32_t)dpp_pair<st>((int)(uint32_t)(v >> 32)) << 32 | (uint32_t)dpp_pair<st>((int)(uint32_t)v);
}
__device__ __forceinline__ double sum16(double v) {      // over each 16 lanes
  v += pair<0>(v);
  v += pair<1>(v);
  v += pair<2>(v);
  return v + pair<3>(v);
}
__device__ __forceinline__ double wave_sum(double v) {
  v = sum16(v);
  return (from_lane(v, 0) + from_lane(v, 16)) + (from_lane(v, 32) + from_lane(v, 48));
}
__device__ __forceinline__ double wave_max(double v) {
  v = fmax(v, pair<0>(v));
  v = fmax(v, pair<1>(v));
  v = fmax(v, pair<2>(v));
  v = fmax(v, pair<3>(v));
  return fmax(fmax(from_lane(v, 0), from_lane(v, 16)), fmax(from_lane(v, 32), from_lane(v, 48)));
}
// The larger key, of equal ones the lower id.
__device__ __forceinline__ void take_larger(uint64_t& k, int& e, uint64_t ok, int oe) {
  const bool other = ok > k || (ok == k && oe < e);
  k = other ? ok : k;
  e = other ? oe : e;
}
template <int st>
__device__ __forceinline__ void larger_pair(uint64_t& k, int& e) { take_larger(k, e, pair64<st>(k), dpp_pair<st>(e)); }
__device__ __forceinline__ void wave_lds() {            // LDS writes of the wave's lanes ahead of its later reads
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <bool kF32>
__device__ __forceinline__ float logit(const void* lg, int64_t at) {
  if constexpr (kF32) return reinterpret_cast<const float*>(lg)[at];
  else return bf16_to_f32(reinterpret_cast<const uint16_t*>(lg)[at]);
}

// One token by one wave, in 64 bits throughout: lane i holds experts i, i + 64, ..; cs: E doubles of the wave's.
// Returns the lane's slot (lane < k).  Few tokens come here and each is waited for, so what counts is the time of one: lanes
// exchange by moves in the VALU and whole waves by reading a lane, not through LDS (13 us a launch for 131072 tokens,
// 15 through LDS).
struct Slot {
  int e;
  float w;
};
template <bool kF32>
__device__ __forceinline__ Slot route_token(const GroupRoute& p, int64_t t, int lane, double* cs) {
  constexpr int kC = kMaxExperts / 64;
  const double none = -__builtin_huge_val();
  double s[kC];
  float bias[kC];
  uint64_t key[kC];
  bool out[kC];                                         // -inf: no weight
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const int e = lane + 64 * c;
    s[c] = e < p.E ? (double)logit<kF32>(p.logits, t * p.E + e) : none;
    bias[c] = p.bias && e < p.E ? p.bias[e] : 0.f;
  }
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const int e = lane + 64 * c;
    out[c] = s[c] == none;
    key[c] = order_of(s[c]);
    if (p.G > 1 && p.best == 1 && !p.bias && e < p.E) cs[e] = s[c];
  }
  if (p.sigmoid) {
#pragma unroll
    for (int c = 0; c < kC; ++c) s[c] = 1.0 / (1.0 + exp(-s[c]));
  } else {
    double m = none;
#pragma unroll
    for (int c = 0; c < kC; ++c) m = fmax(m, s[c]);
    m = wave_max(m);
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
  if (p.bias || (p.G > 1 && p.best == 2)) {
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int e = lane + 64 * c;
      double v = s[c] + (double)bias[c];
      if (out[c]) v = none;
      if (p.bias) {
        key[c] = order_of(v);
        out[c] = v == none;
      }
      if (p.G > 1 && e < p.E) cs[e] = v;
    }
  }
  if (p.G > 1) {
    const int n = p.E / p.G;
    wave_lds();
    // 4 p.lanes lanes to a group, which then compare what they have found
    const int per = 4 * p.lanes, gi = lane / per;
    double a = none, b = none;                          // the two largest
    uint64_t ka = 0, kb = 0;                            // (0: none yet)
    if (gi < p.G)
      for (int i = lane % per; i < n; i += per) {
        const double v = cs[gi * n + i];
        const uint64_t kv = order_of(v);
        if (kv > ka) {
          b = a; kb = ka;
          a = v; ka = kv;
        } else if (kv > kb) {
          b = v; kb = kv;
        }
      }
    for (int d = 1; d < per; d *= 2) {
      const double oa = __shfl_xor(a, d, 64), ob = __shfl_xor(b, d, 64);
      const uint64_t ka2 = order_of(oa) & (uint64_t)-(int64_t)(__shfl_xor((int)(ka != 0), d, 64)),
                     kb2 = order_of(ob) & (uint64_t)-(int64_t)(__shfl_xor((int)(kb != 0), d, 64));
      if (ka2 > ka) {
        if (ka >= kb2) { b = a; kb = ka; } else { b = ob; kb = kb2; }
        a = oa; ka = ka2;
      } else if (ka2 > kb) {
        b = oa; kb = ka2;
      }
    }
    const uint64_t sum = order_of(p.best == 2 ? a + b : a);   // of group gi
    wave_lds();
    int rank = 0;
    for (int h = 0; h < p.G; ++h) {
      const uint64_t o = from_lane(sum, h * per);
      rank += o > sum || (o == sum && h < gi);
    }
    const uint64_t kept = __ballot(gi < p.G && rank < p.kg);   // bit e / n per: whether expert e's group is
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int e = lane + 64 * c;
      if (e < p.E && !(kept >> (e / n * per) & 1)) {
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
    larger_pair<0>(bk, be);
    larger_pair<1>(bk, be);
    larger_pair<2>(bk, be);
    larger_pair<3>(bk, be);
    uint64_t tk = from_lane(bk, 0);
    int te = from_lane(be, 0);
#pragma unroll
    for (int r = 16; r < 64; r += 16) take_larger(tk, te, from_lane(bk, r), from_lane(be, r));
    te = __builtin_amdgcn_readfirstlane(te);
    const double sel = from_lane(bs, te & 63);          // (the owner's best is the wave's)
    if ((te & 63) == lane) gone |= 1u << (te >> 6);
    if (lane == j) {
      r.e = te;
      w = sel;
    }
  }
  if (p.renorm) {
    const double total = sum16(w);                      // (k <= 16)
    w = total == 0.0 ? 0.0 : w / total;
  }
  r.w = (float)(w * (double)p.scale);
  return r;
}

__device__ __forceinline__ void token_again(const GroupRoute& p, int64_t t, int lane, double* cs, int* cnt) {
  const Slot s = p.f32 ? route_token<true>(p, t, lane, cs) : route_token<false>(p, t, lane, cs);
  if (lane < p.k) {
    p.idx[t * p.k + lane] = s.e;
    p.prob[t * p.k + lane] = s.w;
    if (p.counts && (!p.mask || p.mask[t] != 0)) atomicAdd(&cnt[s.e], 1);
  }
}

// ---- the logits of a wave's 4 tokens, which lie one after the other, in LDS: loads of 16 bytes a lane whatever E is,
// and the lanes take their experts from there.  2 words of room after each 32 keep the lanes of groups of 16 or 32
// experts on banks of their own.  Places are counted through the workgroup's stage, kSpan for each wave (4 x 256 values,
// and what a group's last lanes read past them), in bytes: a place is then two instructions.
constexpr uint32_t kSpan = 1088;
__device__ __forceinline__ constexpr uint32_t room(uint32_t i) { return i * 4 + (i * 4 >> 7) * 8; }
template <class T = float>
__device__ __forceinline__ T& at_room(char* stage, uint32_t i) { return *reinterpret_cast<T*>(stage + room(i)); }

// n values of lg from `at` on to places `to` .. (kRoom) or words `to` .. of `stage`.  kU: 256-value pieces that n has at
// most.  Lanes past the end repeat the last piece, so that no branch parts the loads.
template <bool kF32, int kU, bool kRoom = true>
__device__ __forceinline__ void stage_logits(const void* lg, int64_t at, int n, int lane, char* stage, uint32_t to) {
  const auto put = [&](uint32_t i, f32x2_t v) {
    *reinterpret_cast<f32x2_t*>(stage + (kRoom ? room(to + i) : (to + i) * 4)) = v;
  };
  if (n & 3) {                                          // the last tokens
    for (int i = lane; i < n; i += 64)
      *reinterpret_cast<float*>(stage + (kRoom ? room(to + i) : (to + i) * 4)) = logit<kF32>(lg, at + i);
  } else if (n) {
    f32x2_t v[kU][2];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int i = min((u * 64 + lane) * 4, n - 4);
      const char* b = reinterpret_cast<const char*>(lg) + (at + i) * (kF32 ? 4 : 2);
      if constexpr (kF32) {
        const u32x4_any w = *global<u32x4_any>(b);
        const uint32_t x[4] = {w[0], w[1], w[2], w[3]};
        v[u][0] = f32x2_t{__builtin_bit_cast(float, x[0]), __builtin_bit_cast(float, x[1])};
        v[u][1] = f32x2_t{__builtin_bit_cast(float, x[2]), __builtin_bit_cast(float, x[3])};
      } else {
        const u32x2_any w = *global<u32x2_any>(b);
        const uint32_t x = w[0], y = w[1];
        v[u][0] = f32x2_t{__builtin_bit_cast(float, x << 16), __builtin_bit_cast(float, x & 0xFFFF0000u)};
        v[u][1] = f32x2_t{__builtin_bit_cast(float, y << 16), __builtin_bit_cast(float, y & 0xFFFF0000u)};
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const uint32_t i = (uint32_t)min((u * 64 + lane) * 4, n - 4);
      put(i, v[u][0]);                                  // (4 values of a multiple of 4 lie between two rooms)
      put(i + 2, v[u][1]);
    }
  }
}

// Exchange among 16 lanes: rotation by r, and lane j - 1's value for lane j.  (All lanes take part: one that is switched
// off by a condition gives zeros.)
template <int r>
__device__ __forceinline__ int ror16(int v) { return __builtin_amdgcn_mov_dpp(v, 0x120 + r, 0xF, 0xF, true); }
template <int r>
__device__ __forceinline__ float ror16(float v) { return __builtin_bit_cast(float, ror16<r>(__builtin_bit_cast(int, v))); }
__device__ __forceinline__ float before(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x111, 0xF, 0xF, true));
}
// How many groups are ahead of the lane's own, kL lanes to a group: those kL, 2 kL, .. lanes away.
template <int kL, int r = kL>
__device__ __forceinline__ int rank_groups(float score, int g) {
  if constexpr (r < 16) {
    const float o = ror16<r>(score);
    const int og = ror16<r>(g);
    return (int)(o > score || (o == score && og < g)) + rank_groups<kL, r + kL>(score, g);
  } else {
    return 0;
  }
}
// The two largest of two lanes' two.
template <int st>
__device__ __forceinline__ void merge_best(float& a, float& b) {
  const float oa = pair<st>(a), ob = pair<st>(b);
  b = fmaxf(fminf(a, oa), fmaxf(b, ob));
  a = fmaxf(a, oa);
}

// key = the upper 24 bits of x, the lower 8 of id.
__device__ __forceinline__ uint32_t with_id(uint32_t x, int id) { return (x & ~255u) | ((uint32_t)id & 255u); }

// x as an unsigned number, cut off: 0 for what is below it and for a NaN, the largest for what is above (the instruction's
// way; the language leaves these open).
__device__ __forceinline__ uint32_t whole(float x) {
  uint32_t r;
  asm("v_cvt_u32_f32 %0, %1" : "=v"(r) : "v"(x));
  return r;
}

// kN experts a lane, lists of kK >= k.  Keys are 24 bits of a number in the order of what counts, above 255 - id (so that
// of equal ones the lower id is the larger key), and a selection is max and min of 32-bit numbers, of which those between
// lanes read their neighbour as they go:
//   bf16 logits, no bias   the logit itself
//   fp32 logits, no bias   the logit's distance from the row's largest in steps of 2^-19, 32 of it
//   bias                   the score with its bias over the lowest bias, from 0 to the largest it can be
// The first is exact.  The others' roundings keep the order, so that one step apart is right without a bias, and as far
// apart as twice the scores' errors with one; what is nearer and not of equal logits and biases is done again.
// (Keys of the fp32 number in a double's mantissa, the id below it, need no second look at logits but 64-bit max and min
// and moves of 2 words between lanes: 98 us at 131072 x 256 with a bias and 8 groups, where these took 75.)
// kInline: the wave does such tokens itself; else it marks them with id -1 for route_again_kernel, whose 64-bit code would
// take half of this one's waves for its registers (140 us in one kernel, 98 and 19 in two).
// kHalf: half of the groups stay at most.  Those next in rank give their lanes to them: each takes over half the experts of
// the one kg ahead, and the selection has half as many a lane.  131072 x 256 of 8 groups 83 us with it, 88 without (bf16 74
// and 84), 50021 x 160 26 and 29, 131072 x 64 of 4 groups 43 and 45.
// Measured: 131072 x 256 f32, bias, 4 of 8 groups, k = 8, with counts: 82 us of 28 that its bytes take; VALU issue is 68 %
// busy with 870 instructions for 4 tokens, 180 of them the scores.  Profiled, where the three kernels overlap less, 69
// here, 12.8 for the 285 tokens done again, 4.9 for the counts' total.  Without groups, bias and counts 52.
template <int kN, int kK, bool kInline, bool kHalf>
__global__ __launch_bounds__(64 * kWaves, kInline ? 1 : kN <= 16 ? 4 : 2) void route_group_kernel(const GroupRoute p) {
  using K = Key<false>;
  constexpr int kS = kHalf ? kN / 2 : kN;                // experts a lane in the selection
  __shared__ uint8_t holder[kHalf ? kWaves * 64 : 1];    // the lane that holds the experts of the group of a rank
  __shared__ __attribute__((aligned(16))) char stage[room(kWaves * kSpan)];
  __shared__ int cnt[kMaxExperts];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, sub = lane & 15, grp = lane >> 4;
  const int E = p.E, k = p.k, n = E / p.G, lanes = p.lanes, g = sub / lanes, q = sub % lanes;
  const uint32_t place = wave * kSpan + grp * E;        // of the token's first logit
  if (tid < kMaxExperts) cnt[tid] = 0;
  __syncthreads();
  // what the order goes by: scores where a bias or sums of two count, else the logits themselves
  const bool sums = p.G > 1 && p.best == 2, scored = p.bias || sums, exact = !p.bias && !p.f32;
  const bool stats = !p.sigmoid && (scored || !p.renorm);
  const int own = g < p.G ? n : 0;                      // experts of the lane's group
  const bool full = lanes * kN == n && lanes * p.G == 16;
  const bool steps = n <= 32 && 32 % n == 0 && E % 32 == 0;   // a group lies between two rooms
  const int mine_n = (own - q + lanes - 1) / lanes;     // experts of the lane
  // biases over the lowest one (-inf aside), and how far the largest sum is from 0
  float lo = 0.f, range = 0.f;
  if (p.bias) {
    lo = -kNone;
    float hi = kNone;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < kMaxExperts / 64; ++i) {
      const float x = lane + 64 * i < E ? p.bias[lane + 64 * i] : kNone;
      lo = x > kNone ? fminf(lo, x) : lo;
      hi = fmaxf(hi, x);
      odd |= x != x;
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
      lo = fminf(lo, __shfl_xor(lo, d, 64));
      hi = fmaxf(hi, __shfl_xor(hi, d, 64));
    }
    // (infinite, NaN or so large that 64 bits round the scores away: every token is done in 64 bits)
    range = __any(odd) || fmaxf(fabsf(lo), fabsf(hi)) > 0x1p20f ? -kNone : hi - lo + 1.f;
  }
  // Errors, u = 2^-24: of a sigmoid 4 u (exponential and reciprocal an ulp each, its argument's rounding), of a softmax 24 u;
  // with the bias over the lowest, two roundings of up to `range` more.  So two scores differ by what they seem to within
  // 2 (4 + 1 + 2 range) u, two sums of two within 2 (10 + 6 range) u: at least as much is allowed for.
  // (For softmax scores that is the error of one near 1, and 256 experts whose logits are close have scores of 1 / 256 that
  // differ by less: 131072 x 256 with a bias takes 104 us at logits of deviation 1.5, 359 at 0.1.)
  const float t0_err = p.sigmoid ? 0x1p-20f : 0x1p-17f;
  const float near = t0_err + 0x1p-21f * range;
  const bool hopeless = p.bias && !(range < 0x1p60f);    // (64-bit roundings of what is below: 2^-33 at most, within the errors)
  float b[kN];
#pragma unroll
  for (int c = 0; c < kN; ++c) b[c] = p.bias && q + lanes * c < own ? p.bias[g * n + q + lanes * c] - lo : 0.f;
  constexpr float kTop = 0x1p32f - 0x1p16f;
  float by = 0x1p27f, plus = 0.f;                        // key = by x + plus
  uint32_t apart = 0;
  if (p.bias) {
    by = kTop / range;
    plus = 4096.f;
    apart = whole(near * by * 0x1p-8f) + 2u;
  }
  for (int64_t t0 = (int64_t)blockIdx.x * kTokens; t0 < p.T; t0 += (int64_t)gridDim.x * kTokens) {
    const int64_t tw = t0 + 4 * wave, t = tw + grp;
    const int64_t left = p.T - tw;
    const bool in = t < p.T;
    const int have = left >= 4 ? 4 * E : left > 0 ? (int)left * E : 0;
    wave_lds();
    // (E <= 16 kN and 256)
    constexpr int kU = kN < 4 ? 1 : kN < 16 ? kN / 4 : 4;
    if (p.f32) stage_logits<true, kU>(p.logits, tw * E, have, lane, stage, wave * kSpan);
    else stage_logits<false, kU>(p.logits, tw * E, have, lane, stage, wave * kSpan);
    wave_lds();
    // (not known to be the same in every turn: places and ids would all be kept in registers)
    int e0 = (own ? g * n : 0) + q;
    asm volatile("" : "+v"(e0));
    float v[kN];                                         // (-inf: no expert, which like one of -inf is never selected here)
    const uint32_t from = place + e0;
    if (lanes == 16 && E % 32 == 0) {                    // (places without arithmetic where no group crosses a room)
#pragma unroll
      for (int c = 0; c < kN; ++c) v[c] = *reinterpret_cast<const float*>(stage + room(from) + c * 64 + c / 2 * 8);
    } else if (steps) {
      uint32_t at = room(from);
#pragma unroll
      for (int c = 0; c < kN; ++c, at += 4 * lanes) v[c] = *reinterpret_cast<const float*>(stage + at);
    } else {
#pragma unroll
      for (int c = 0; c < kN; ++c) v[c] = at_room(stage, from + lanes * c);
    }
    if (!full) {
      int end = mine_n;
      asm volatile("" : "+v"(end));                      // (a branch, and 16 comparisons in it, not their results kept)
#pragma unroll
      for (int c = 0; c < kN; ++c) v[c] = c < end ? v[c] : kNone;
    }
    float m = 0.f, total = 0.f;                          // largest logit, and of the row's exponentials
    if (stats || !(exact || p.bias)) {
      m = v[0];
#pragma unroll
      for (int c = 1; c < kN; ++c) m = fmaxf(m, v[c]);
      m = group_max<16>(m);
      if (!p.bias) plus = kTop - m * 0x1p27f;
      m = m == kNone ? 0.f : m;
    }
    bool bad = hopeless;
    if (!p.bias && !exact) bad |= !(fabsf(m) < 4096.f);  // (plus would round by more than its room)
    if (!exact || p.G > 1) {
      bool nan = false;
#pragma unroll
      for (int c = 0; c < kN; ++c) nan |= v[c] != v[c];
      bad |= nan;
    }
    if (stats) {
#pragma unroll
      for (int c = 0; c < kN; ++c) total += __expf(v[c] - m);
      total = group_sum<16>(total);
    }
    // scores with their biases (0 without), -inf where the logit is
    const auto score_all = [&]() {
      if (p.sigmoid) {
#pragma unroll
        for (int c = 0; c < kN; ++c) {
          const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-v[c])) + b[c];
          v[c] = v[c] == kNone ? kNone : s;
        }
      } else {
        const float inv = 1.0f / total;
#pragma unroll
        for (int c = 0; c < kN; ++c) {
          const float s = __builtin_fmaf(__expf(v[c] - m), inv, b[c]);
          v[c] = v[c] == kNone ? kNone : s;
        }
      }
    };
    // what becomes the keys' upper bits; with a bias the scores do
    uint32_t x[kN];
    int id = 255 - e0;                                   // of the lane's first expert, counted down
    if (p.bias) {
      score_all();
    } else if (exact) {
#pragma unroll
      for (int c = 0; c < kN; ++c) x[c] = rank_of<0x10000u>(v[c]);
    } else {
#pragma unroll
      for (int c = 0; c < kN; ++c) x[c] = whole(__builtin_fmaf(v[c], by, plus));
    }
    if (p.G > 1) {
      if (sums && !p.bias) score_all();
      float first = kNone, second = kNone;               // the two largest
#pragma unroll
      for (int c = 0; c < kN; ++c) {
        second = __builtin_amdgcn_fmed3f(first, second, v[c]);
        first = fmaxf(first, v[c]);
      }
      if (lanes > 1) merge_best<0>(first, second);
      if (lanes > 2) merge_best<1>(first, second);
      if (lanes > 4) merge_best<2>(first, second);
      const float score = sums ? first + second : first;
      int rank;
      if (lanes == 8) rank = rank_groups<8>(score, g);
      else if (lanes == 4) rank = rank_groups<4>(score, g);
      else if (lanes == 2) rank = rank_groups<2>(score, g);
      else rank = rank_groups<1>(score, g);
      const bool kept = own && rank < p.kg;
      if (scored) {
        const float least = -group_max<16>(kept ? -score : kNone), most = group_max<16>(kept ? kNone : score);
        bad |= !(least - most > 2.f * t0_err + 0x1p-20f * (range + 2.f));
      }
      if constexpr (kHalf) {
        uint8_t* const at = holder + (tid & ~15) + q;
        if (kept) at[rank * lanes] = (uint8_t)lane;
        wave_lds();
        const bool helps = own && !kept && rank < 2 * p.kg;
        const int from_it = helps ? at[(rank - p.kg) * lanes] & 63 : lane;
        wave_lds();
        if (p.bias) {
#pragma unroll
          for (int c = 0; c < kN; ++c) x[c] = __builtin_bit_cast(uint32_t, v[c]);
        }
        const uint32_t none = p.bias ? 0xFF800000u : 0u;   // -inf, or the lowest number
#pragma unroll
        for (int c = 0; c < kS; ++c) {
          const uint32_t other = (uint32_t)__shfl((int)x[kS + c], from_it, 64);
          x[c] = kept ? x[c] : helps ? other : none;
        }
        const int half = __shfl(id, from_it, 64) - lanes * kS;
        id = kept ? id : half;
        if (p.bias) {
#pragma unroll
          for (int c = 0; c < kS; ++c) v[c] = __builtin_bit_cast(float, x[c]);
        }
      } else if (p.bias) {
#pragma unroll
        for (int c = 0; c < kN; ++c) v[c] = kept ? v[c] : kNone;
      } else {
#pragma unroll
        for (int c = 0; c < kN; ++c) x[c] = kept ? x[c] : 0u;
      }
    }
    if (p.bias) {
#pragma unroll
      for (int c = 0; c < kS; ++c) x[c] = whole(__builtin_fmaf(v[c], by, plus));
    }
    uint32_t key[kS];
#pragma unroll
    for (int c = 0; c < kS; ++c, id -= lanes) key[c] = with_id(x[c], id);
    constexpr int kA = kS > kK ? kS : kK;
    uint32_t a[kA];
#pragma unroll
    for (int c = 0; c < kS; ++c) a[c] = key[c];
    sort_top<K, kS, kK>(a);
    constexpr int kM = kS < kK ? kS : kK;
    merge_lanes<K, 16, kM, kK, 0>(a);
    // the lane's slot, and the last one
#pragma unroll
    for (int h = 1; h < kK; h *= 2) {
      const uint32_t upper = sub & h ? ~0u : 0u;         // (masks: a choice of an array's elements becomes a search in it)
#pragma unroll
      for (int j = 0; j < kK; j += 2 * h) a[j] = (a[j] & ~upper) | (a[j + h] & upper);
    }
    const uint32_t mine = a[0], end = (uint32_t)__shfl((int)mine, (lane & 48) + k - 1, 64);
    bad |= end < 256u;                                   // fewer experts than k, or below the keys' range: by their ids
    const bool slot = sub < k;
    const int e = slot ? 255 - (int)(mine & 255u) : 0;
    const float le = slot ? at_room(stage, place + (e < E ? e : 0)) : kNone;
    if (!exact) {
      const uint32_t above = (uint32_t)__builtin_amdgcn_mov_dpp((int)mine, 0x111, 0xF, 0xF, true) >> 8;
      const uint32_t at = mine >> 8, last = end >> 8;
      const bool close = slot && sub > 0 && !(above - at > apart);
      // every expert that reaches the last one's neighbourhood is in the list
      const uint32_t floor = (last > apart ? last - apart : 0u) << 8;
      int reach = 0;
#pragma unroll
      for (int c = 0; c < kS; ++c) reach += key[c] >= floor;
      reach += dpp_pair<0>(reach);
      reach += dpp_pair<1>(reach);
      reach += dpp_pair<2>(reach);
      reach += dpp_pair<3>(reach);
      if (__any(close || reach != k)) {
        // equal logits with equal biases are equal in any arithmetic, and in the right order already: they pass
        // (the biases themselves: over the lowest one two may round to the same)
        const float be = slot && p.bias ? p.bias[e < E ? e : 0] : 0.f;
        const float lp = before(le), bp = before(be);
        bool odd = close && !(le == lp && be == bp);
        const int end_lane = (lane & 48) + k - 1;
        const float ll = __shfl(le, end_lane, 64), bl = __shfl(be, end_lane, 64);
        int others = slot && !(le == ll && be == bl) ? -1 : 0;
#pragma unroll
        for (int c = 0; c < kS; ++c) {
          const int ec = kHalf ? 255 - (int)(key[c] & 255u) : e0 + lanes * c;
          if (key[c] >= floor) others += !(at_room(stage, place + ec) == ll && (!p.bias || p.bias[ec < E ? ec : 0] == bl));
        }
        others += dpp_pair<0>(others);
        others += dpp_pair<1>(others);
        others += dpp_pair<2>(others);
        others += dpp_pair<3>(others);
        bad |= odd || others != 0;
      }
    }
    // weights: of sigmoids as multiples of e^top, which the quotient drops, so that tiny ones keep their ratios, down to
    // those that are 0 in 64 bits; softmax scores among which a bias has selected none that is near the row's largest
    // may be 0 as well, and are left to 64 bits
    float w = 0.f;
    if (p.sigmoid) {
      const float top = p.renorm ? fminf(group_max<16>(le), 0.f) : 0.f;
      w = le >= 0.f ? 1.0f / (1.0f + expf(-le)) : le < kLeast ? 0.f : expf(le - top) / (1.0f + expf(le));
    } else if (p.renorm) {
      const float top = group_max<16>(le);
      if (p.bias) bad |= !(top - m > -700.f);
      w = expf(le - top);
    } else {
      w = expf(le - m) / total;
    }
    w = slot ? w : 0.f;
    if (p.renorm) {
      const float sum = group_sum<16>(w);
      w = sum == 0.f ? 0.f : w / sum;
    }
    const uint64_t again = __ballot(bad && in);
    const bool done = (again >> (lane & 48) & 0xFFFFu) == 0;
    if (in && done && slot) {
      p.idx[t * k + sub] = e;
      p.prob[t * k + sub] = w * p.scale;
      if (p.counts && (!p.mask || p.mask[t] != 0)) atomicAdd(&cnt[e], 1);
    }
    if constexpr (!kInline) {
      if (in && !done && sub == 0) p.idx[t * k] = -1;
    } else if (again) {
      wave_lds();                                        // the stage is free: it holds the 64-bit scores now
#pragma unroll 1
      for (int i = 0; i < 4; ++i)
        if (again >> (16 * i) & 0xFFFFu) token_again(p, tw + i, lane, reinterpret_cast<double*>(stage + room(wave * kSpan)), cnt);
    }
  }
  if (p.counts) {
    __syncthreads();
    int32_t* to = kInline && gridDim.x == 1 ? p.counts : p.part + (int64_t)blockIdx.x * E;
    if (tid < E) to[tid] = cnt[tid];
  }
}

// The tokens that route_group_kernel has marked, in 64 bits: a workgroup looks through 256 and deals the marked ones to
// its waves.  Its counts follow the first kernel's.
__global__ __launch_bounds__(64 * kWaves) void route_again_kernel(const GroupRoute p, int32_t* part) {
  __shared__ double cs[kWaves][kMaxExperts];
  __shared__ int cnt[kMaxExperts], list[64 * kWaves], marked;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid < kMaxExperts) cnt[tid] = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * 64 * kWaves; t0 < p.T; t0 += (int64_t)gridDim.x * 64 * kWaves) {
    if (tid == 0) marked = 0;
    __syncthreads();
    const int64_t t = t0 + tid;
    if (t < p.T && p.idx[t * p.k] < 0) list[atomicAdd(&marked, 1)] = tid;
    __syncthreads();
    for (int i = wave; i < marked; i += kWaves) token_again(p, t0 + list[i], lane, cs[wave], cnt);
    __syncthreads();
  }
  if (p.counts && tid < p.E) part[(int64_t)blockIdx.x * p.E + tid] = cnt[tid];
}

template <int kN, bool kInline, bool kHalf>
void launch_k(const GroupRoute& p, int nb, hipStream_t st) {
  if (p.k <= 2) route_group_kernel<kN, 2, kInline, kHalf><<<nb, 64 * kWaves, 0, st>>>(p);
  else if (p.k <= 4) route_group_kernel<kN, 4, kInline, kHalf><<<nb, 64 * kWaves, 0, st>>>(p);
  else if (p.k <= 8) route_group_kernel<kN, 8, kInline, kHalf><<<nb, 64 * kWaves, 0, st>>>(p);
  else route_group_kernel<kN, 16, kInline, kHalf><<<nb, 64 * kWaves, 0, st>>>(p);
}
template <bool kInline>
void launch_n(const GroupRoute& p, int nb, hipStream_t st) {
  const int per = (p.E / p.G + p.lanes - 1) / p.lanes;   // experts a lane
  const bool half = !kInline && p.G > 1 && 2 * p.kg <= p.G;
  constexpr bool kHalf = !kInline;
  if (per <= 1) launch_k<1, kInline, false>(p, nb, st);
  else if (per <= 2) launch_k<2, kInline, false>(p, nb, st);
  else if (per <= 4 && half) launch_k<4, kInline, kHalf>(p, nb, st);
  else if (per <= 4) launch_k<4, kInline, false>(p, nb, st);
  else if (per <= 8 && half) launch_k<8, kInline, kHalf>(p, nb, st);
  else if (per <= 8) launch_k<8, kInline, false>(p, nb, st);
  else if (per <= 16 && half) launch_k<16, kInline, kHalf>(p, nb, st);
  else if (per <= 16) launch_k<16, kInline, false>(p, nb, st);
  else if (half) launch_k<32, kInline, kHalf>(p, nb, st);
  else launch_k<32, kInline, false>(p, nb, st);
}

// counts[e] = sum over the nb blocks; a workgroup takes 16 experts, 64 slices of the blocks.
constexpr int kCountThreads = 1024;
__global__ __launch_bounds__(kCountThreads) void route_counts_kernel(const int32_t* __restrict__ part, int nb, int E,
                                                                     int32_t* __restrict__ counts) {
  constexpr int kS = kCountThreads / 16;
  __shared__ int red[kS][16];
  const int le = threadIdx.x & 15, s = threadIdx.x >> 4, e = blockIdx.x * 16 + le;
  int c = 0;
  if (e < E) {
    int i = s;
    for (; i + 7 * kS < nb; i += 8 * kS) {
      int v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = part[(int64_t)(i + u * kS) * E + e];
#pragma unroll
      for (int u = 0; u < 8; ++u) c += v[u];
    }
    for (; i < nb; i += kS) c += part[(int64_t)i * E + e];
  }
  red[s][le] = c;
  __syncthreads();
  for (int h = kS / 2; h >= 1; h /= 2) {
    if (s < h) red[s][le] += red[s + h][le];
    __syncthreads();
  }
  if (s == 0 && e < E) counts[e] = red[0][le];
}

// ---- backward.  A wave takes 4 tokens, whose rows of dlogits lie one after the other: they are put together in LDS and
// leave as 16 bytes a lane, whatever E is.  kN: experts a lane where every logit has a gradient (softmax weights as they
// are), 0 where only the selected ones have.  Measured: 131072 x 256 f32, k = 8, sigmoid weights 39 us: it writes 134 MB
// and reads 101, nearly all lines of the logits for 8 of each row; 30011 x 157 bf16 softmax weights as they are 9 us.
template <bool kF32>
__device__ __forceinline__ void store_rows(void* to, int64_t at, int n, int lane, const float* from) {
  constexpr int kV = kF32 ? 4 : 8;
  for (int i = lane * kV; i < n; i += 64 * kV) {
    float v[8];
    *reinterpret_cast<f32x4*>(v) = *reinterpret_cast<const f32x4*>(from + i);
    if constexpr (!kF32) *reinterpret_cast<f32x4*>(v + 4) = *reinterpret_cast<const f32x4*>(from + i + 4);
    char* b = reinterpret_cast<char*>(to) + (at + i) * (kF32 ? 4 : 2);
    if (i + kV <= n) {
      u32x4 w;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = kF32 ? __builtin_bit_cast(uint32_t, v[j]) : pack_bf16x2(v[2 * j], v[2 * j + 1]);
      // (past the caches: 131072 x 256 f32 39 us, 46 through them, bf16 of softmax weights as they are 27, 42; alike below 30 MB)
      __builtin_nontemporal_store(w, global<u32x4_any>(b));
    } else {
#pragma unroll
      for (int j = 0; j < kV; ++j)
        if (i + j < n) {
          if constexpr (kF32) reinterpret_cast<float*>(b)[j] = v[j];
          else reinterpret_cast<uint16_t*>(b)[j] = f32_to_bf16(v[j]);
        }
    }
  }
}

// d summed over the slots of the same expert, in a fixed order; whether the lane's is the first of them.
template <int r>
__device__ __forceinline__ void add_same(int e, float d, int sub, float& sum, bool& first) {
  if constexpr (r < 16) {
    const int oe = ror16<r>(e), os = ror16<r>(sub);
    const float od = ror16<r>(d);
    sum += oe == e ? od : 0.f;
    first = first && !(oe == e && os < sub);
    add_same<r + 1>(e, d, sub, sum, first);
  }
}

template <bool kF32, int kN>
__global__ __launch_bounds__(64 * kWaves) void route_group_bwd_kernel(const GroupRouteBwd p) {
  __shared__ __attribute__((aligned(16))) float rows[kWaves][4 * kMaxExperts + 8];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, sub = lane & 15, grp = lane >> 4, E = p.E, k = p.k;
  float* const row = rows[wave];
  for (int i = lane; i < 4 * kMaxExperts + 8; i += 64) row[i] = 0.f;
  for (int64_t t0 = (int64_t)blockIdx.x * kTokens; t0 < p.T; t0 += (int64_t)gridDim.x * kTokens) {
    const int64_t tw = t0 + 4 * wave, t = tw + grp, left = p.T - tw;
    if (left <= 0) break;                               // (the wave's last turn: nothing below waits for the others)
    const int have = left >= 4 ? 4 * E : (int)left * E;
    int e = -1 - sub;                                   // (no slot: an id of its own)
    float w = 0.f, g = 0.f;
    if (t < p.T && sub < k) {
      const int64_t at = t * k + sub;
      e = p.idx[at];
      w = p.prob[at];
      g = p.dprob[at];
    }
    const bool has = e >= 0 && e < E;
    // in 64 bits: g and the mean of all cancel, with one slot to nothing at all
    double dot = (double)w * (double)g;
    dot += pair<0>(dot);
    dot += pair<1>(dot);
    dot += pair<2>(dot);
    dot += pair<3>(dot);
    float d = (float)((double)w * (p.renorm ? (double)g - dot / (double)p.scale : (double)g));
    const float sum = (float)dot;
    if (p.sigmoid && has) d *= 1.0f / (1.0f + expf(logit<kF32>(p.logits, t * E + e)));
    float* const mine = row + grp * E;
    if constexpr (kN > 0) {
      float v[kN > 0 ? kN : 1], m = kNone, s = 0.f;
      // (bf16 through LDS: 131072 x 256 71 us with 2-byte loads of 16 lanes, 42 so, both stored through the caches; fp32 46, 52)
      if constexpr (kF32) {
#pragma unroll
        for (int c = 0; c < kN; ++c) {
          v[c] = kNone;
          if (t < p.T && sub + 16 * c < E) v[c] = logit<kF32>(p.logits, t * E + sub + 16 * c);
        }
      } else {
        stage_logits<kF32, kN / 4 < 1 ? 1 : kN / 4, false>(p.logits, tw * E, have, lane, reinterpret_cast<char*>(row), 0u);
        wave_lds();
#pragma unroll
        for (int c = 0; c < kN; ++c) v[c] = mine[sub + 16 * c < E ? sub + 16 * c : 0];
      }
#pragma unroll
      for (int c = 0; c < kN; ++c) {
        v[c] = sub + 16 * c < E ? v[c] : kNone;
        m = fmaxf(m, v[c]);
      }
      m = group_max<16>(m);
      m = m == kNone ? 0.f : m;
#pragma unroll
      for (int c = 0; c < kN; ++c) {
        v[c] = __expf(v[c] - m);
        s += v[c];
      }
      s = group_sum<16>(s);
      const float by = s == 0.f ? 0.f : -sum / s;
      wave_lds();
#pragma unroll
      for (int c = 0; c < kN; ++c)
        if (sub + 16 * c < E) mine[sub + 16 * c] = v[c] * by;
    }
    wave_lds();
    // the selected ones' own part; a slot that finds another's number at its expert shares it
    const float before_it = has ? mine[e] : 0.f;
    wave_lds();
    if (has) mine[e] = __builtin_bit_cast(float, sub);
    wave_lds();
    const bool shared = has && __builtin_bit_cast(int, mine[e]) != sub;
    bool first = has;
    if (__any(shared)) {
      float all = d;
      add_same<1>(e, d, sub, all, first);
      d = all;
    }
    wave_lds();
    if (first) mine[e] = before_it + d;
    wave_lds();
    store_rows<kF32>(p.dlogits, tw * E, have, lane, row);
    wave_lds();
    if (kN == 0 && has) mine[e] = 0.f;
    wave_lds();
  }
}

template <bool kF32>
void launch_bwd(const GroupRouteBwd& p, hipStream_t st) {
  const int64_t nb = (p.T + kTokens - 1) / kTokens;
  const int grid = (int)(nb < 2048 ? nb : 2048);
  if (p.sigmoid || p.renorm) route_group_bwd_kernel<kF32, 0><<<grid, 64 * kWaves, 0, st>>>(p);
  else if (p.E <= 32) route_group_bwd_kernel<kF32, 2><<<grid, 64 * kWaves, 0, st>>>(p);
  else if (p.E <= 64) route_group_bwd_kernel<kF32, 4><<<grid, 64 * kWaves, 0, st>>>(p);
  else if (p.E <= 128) route_group_bwd_kernel<kF32, 8><<<grid, 64 * kWaves, 0, st>>>(p);
  else route_group_bwd_kernel<kF32, 16><<<grid, 64 * kWaves, 0, st>>>(p);
}

}  // namespace

namespace {
// Tokens up to which a workgroup a CU takes them, marked ones and all, in one launch.
constexpr int64_t kInlineTokens = 256 * kTokens;
int most(int64_t n, int m) { return (int)(n < m ? n : m); }
int group_blocks(int64_t T) { return most((T + kTokens - 1) / kTokens, kGroupMaxBlocks); }
int again_blocks(int64_t T) { return T <= kInlineTokens ? 0 : most((T + 64 * kWaves - 1) / (64 * kWaves), kGroupMaxBlocks); }
}  // namespace

int route_group_parts(int64_t T) { return group_blocks(T) + again_blocks(T); }

hipError_t launch_route_group(GroupRoute p, bool f32, hipStream_t st) {
  const int nb = group_blocks(p.T), more = again_blocks(p.T);
  int wide = 1;
  while (wide < p.G) wide *= 2;
  p.f32 = f32;
  p.lanes = 16 / wide;
  if (more) {
    launch_n<false>(p, nb, st);
    route_again_kernel<<<more, 64 * kWaves, 0, st>>>(p, p.part + (int64_t)nb * p.E);
  } else {
    launch_n<true>(p, nb, st);
  }
  if (p.counts && nb + more > 1)
    route_counts_kernel<<<(p.E + 15) / 16, kCountThreads, 0, st>>>(p.part, nb + more, p.E, p.counts);
  return hipGetLastError();
}

hipError_t launch_route_group_bwd(const GroupRouteBwd& p, bool f32, hipStream_t st) {
  if (f32) launch_bwd<true>(p, st);
  else launch_bwd<false>(p, st);
  return hipGetLastError();
}

}  // namespace moe
