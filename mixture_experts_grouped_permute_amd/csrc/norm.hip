// Residual addition and root-mean-square norm for gfx950, forward and backward.
//
//   s = x + r, rounded to the type of x: the sum as the residual stream carries it, and what is normalized
//   y[t, h] = s[t, h] rstd[t] w[h],   rstd[t] = 1 / sqrt(mean_h s[t, h]^2 + eps)
//   codes and scales: E4M3 with one fp32 scale per 128 columns (block_scale.h) of the fp32 y, not of the rounded one
// Gradient, xh = s rstd and g = dy w:
//   dx = rstd (g - xh mean_h(g xh)) + ds,    dw[h] = sum_t dy xh
// rstd is formed again from s, which the backward reads anyway: both of its sums come from the same read.
//
// Memory bounds both.  A row stays in the registers of kL lanes between the sums and the results, kN pieces of 8
// columns each, so that everything is read and written once; the next row's loads are in flight behind the sums.
#include "common.h"
#include "kernels.h"
#include "block_scale.h"

#include <type_traits>

namespace moe {
namespace {

// 8 consecutive values.  kAligned: at 16 bytes; else at the type's alignment, which global memory's wide
// accesses take as well.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));

template <bool kF32, bool kAligned>
struct Eight {
  u32x4 w[kF32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    const char* b = reinterpret_cast<const char*>(p) + at * (kF32 ? 4 : 2);
    if constexpr (kAligned) {
      w[0] = reinterpret_cast<const u32x4*>(b)[0];
      if constexpr (kF32) w[1] = reinterpret_cast<const u32x4*>(b)[1];
    } else {
      w[0] = reinterpret_cast<const u32x4_any*>(b)[0];
      if constexpr (kF32) w[1] = reinterpret_cast<const u32x4_any*>(b)[1];
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
  __device__ __forceinline__ void store(void* p, int64_t at) const {
    char* b = reinterpret_cast<char*>(p) + at * (kF32 ? 4 : 2);
    if constexpr (kAligned) {
      reinterpret_cast<u32x4*>(b)[0] = w[0];
      if constexpr (kF32) reinterpret_cast<u32x4*>(b)[1] = w[1];
    } else {
      reinterpret_cast<u32x4_any*>(b)[0] = w[0];
      if constexpr (kF32) reinterpret_cast<u32x4_any*>(b)[1] = w[1];
    }
  }
};

template <int ctrl, int rows>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), ctrl, rows, 0xF, false));
}
// Sums over each 16 lanes (in all of them), and over the wave (uniform).
__device__ __forceinline__ float sum16(float v) {
  v = dpp_add<0xB1, 0xF>(v);       // lanes ^ 1, ^ 2, mirrors of 8 and 16
  v = dpp_add<0x4E, 0xF>(v);
  v = dpp_add<0x141, 0xF>(v);
  return dpp_add<0x140, 0xF>(v);
}
__device__ __forceinline__ float sum64(float v) {
  v = sum16(v);
  v = dpp_add<0x142, 0xA>(v);      // a row's last lane to the next row, then row 1's to the upper half
  v = dpp_add<0x143, 0xC>(v);
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

constexpr int threads_of(int kL) { return kL > 256 ? kL : 256; }

// Sums of kS numbers over the kL lanes of a row.  red: two sets, used in turn, so that one barrier a turn is enough.
template <int kL, int kS>
struct RowSum {
  static constexpr int kW = kL / 64 > 1 ? kL / 64 : 1, kRows = threads_of(kL) / kL;
  static constexpr int kWords = kL > 64 ? 2 * kRows * kW * kS : 1;
  static __device__ __forceinline__ void sum(float (&v)[kS], float* red, int turn) {
#pragma unroll
    for (int i = 0; i < kS; ++i) v[i] = kL == 16 ? sum16(v[i]) : sum64(v[i]);
    if constexpr (kL > 64) {
      const int wave = threadIdx.x >> 6;
      float* to = red + (turn & 1) * kRows * kW * kS;
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < kS; ++i) to[wave * kS + i] = v[i];
      __syncthreads();
      const float* row = to + wave / kW * kW * kS;
#pragma unroll
      for (int i = 0; i < kS; ++i) {
        v[i] = row[i];
#pragma unroll
        for (int w = 1; w < kW; ++w) v[i] += row[w * kS + i];
      }
    }
  }
};

// The columns of a lane's piece c: 8 from `col` on.  Where a row ends inside the piece it is moved back to end with
// the row: its first `skip` columns are another lane's, whose results it repeats and whose sums it leaves out.
// Rows of fewer than 8 columns never get here unaligned (the launcher pads nothing: they take kernel `narrow`).
struct Piece {
  int col, skip;
  bool in;
};
template <int kL, bool kAligned>
__device__ __forceinline__ Piece piece(int c, int sub, int H) {
  Piece q{(c * kL + sub) * 8, 0, true};
  q.in = q.col < H;
  if constexpr (!kAligned) {
    if (q.in && q.col + 8 > H) {
      q.skip = q.col + 8 - H;
      q.col -= q.skip;
    }
  }
  return q;
}

// ---- forward.  A workgroup takes `unit` consecutive rows, kRows at a time.
template <bool kF32, bool kW32, int kL, int kN, bool kAligned>
__global__ __launch_bounds__(threads_of(kL)) void add_rmsnorm_kernel(const NormFwd p, int unit) {
  using Sum = RowSum<kL, 1>;
  constexpr int kRows = Sum::kRows;
  __shared__ float red[Sum::kWords];
  extern __shared__ float sc[];                         // [H / 128][unit] scales, which leave as runs of rows
  const int tid = threadIdx.x, sub = tid % kL, slot = tid / kL, H = (int)p.H;
  const int64_t r0 = (int64_t)blockIdx.x * unit;
  Piece q[kN];
  Eight<kW32, kAligned> w[kN];
#pragma unroll
  for (int c = 0; c < kN; ++c) {
    q[c] = piece<kL, kAligned>(c, sub, H);
    if (q[c].in) w[c].load(p.weight, q[c].col);
    else w[c].zero();
  }
  Eight<kF32, kAligned> x[kN], r[kN];
  const auto fetch = [&](int64_t t) {
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      if (q[c].in && t < p.T) x[c].load(p.x, t * H + q[c].col);
      else x[c].zero();
    }
    if (p.residual) {
#pragma unroll
      for (int c = 0; c < kN; ++c) {
        if (q[c].in && t < p.T) r[c].load(p.residual, t * H + q[c].col);
        else r[c].zero();
      }
    }
  };
  fetch(r0 + slot);
  for (int i = 0; i < unit && r0 + i < p.T; i += kRows) {
    const int64_t t = r0 + i + slot;
    const bool live = t < p.T;
    float s[kN][8], sq[1] = {0.f};
#pragma unroll
    for (int c = 0; c < kN; ++c) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[c][j] = x[c].at(j);
      if (p.residual) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s[c][j] += r[c].at(j);
        Eight<kF32, kAligned> o;
        o.set(s[c]);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[c][j] = o.at(j);   // as it is stored
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sq[0] += kAligned || j >= q[c].skip ? s[c][j] * s[c][j] : 0.f;
    }
    if (i + kRows < unit) fetch(t + kRows);
    Sum::sum(sq, red, i / kRows);
    // (the sums are stored behind the row's last read, which may be of the same memory)
    const float rstd = 1.0f / sqrtf(sq[0] / (float)H + p.eps);
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      const bool out = q[c].in && live;
      const int64_t at = t * H + q[c].col;
      Eight<kF32, kAligned> o;
      if (p.sum && out) {
        o.set(s[c]);
        o.store(p.sum, at);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s[c][j] = s[c][j] * rstd * w[c].at(j);
      if (p.y && out) {
        o.set(s[c]);
        o.store(p.y, at);
      }
      if constexpr (kAligned) {
        if (p.q) {
          uint32_t m = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) m = umax(m, __builtin_bit_cast(uint32_t, s[c][j]) & 0x7FFFFFFFu);
          const BlockScale b = block_scale(max16(m));
          if (out) {
            u32x2 o8;
            o8[0] = codes4(s[c][0], s[c][1], s[c][2], s[c][3], b.factor);
            o8[1] = codes4(s[c][4], s[c][5], s[c][6], s[c][7], b.factor);
            *reinterpret_cast<u32x2*>(p.q + at) = o8;
            if ((tid & 15) == 0) {
              const int blk = q[c].col >> 7;
              if (unit == 1) p.scales[(int64_t)blk * p.T + t] = b.d;
              else sc[blk * unit + i + slot] = b.d;
            }
          }
        }
      }
    }
  }
  if constexpr (kAligned) {
    if (p.q && unit > 1) {
      __syncthreads();
      for (int i = tid; i < H / 128 * unit; i += threads_of(kL)) {
        const int blk = i / unit, u = i % unit;
        if (r0 + u < p.T) p.scales[(int64_t)blk * p.T + r0 + u] = sc[i];
      }
    }
  }
}

// ---- backward.  Workgroup b takes rows b kRows, (b + grid) kRows, ..: dx, and sums of dy xh over them for each
// of its slots, in registers till its end.
template <bool kF32, bool kW32, int kL, int kN, bool kAligned>
__global__ __launch_bounds__(threads_of(kL)) void rmsnorm_bwd_kernel(const NormBwd p) {
  using Sum = RowSum<kL, 2>;
  constexpr int kRows = Sum::kRows;
  __shared__ float red[Sum::kWords];
  const int tid = threadIdx.x, sub = tid % kL, slot = tid / kL, H = (int)p.H;
  Piece q[kN];
  Eight<kW32, kAligned> w[kN];
  float acc[kN][8];
#pragma unroll
  for (int c = 0; c < kN; ++c) {
    q[c] = piece<kL, kAligned>(c, sub, H);
    if (q[c].in) w[c].load(p.weight, q[c].col);
    else w[c].zero();
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[c][j] = 0.f;
  }
  Eight<kF32, kAligned> rs[kN], rd[kN], ra[kN];
  const auto fetch = [&](int64_t t) {
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      const bool in = q[c].in && t < p.T;
      if (in) {
        rs[c].load(p.s, t * H + q[c].col);
        rd[c].load(p.dy, t * H + q[c].col);
      } else {
        rs[c].zero();
        rd[c].zero();
      }
    }
    if (p.dsum) {
#pragma unroll
      for (int c = 0; c < kN; ++c)
        if (q[c].in && t < p.T) ra[c].load(p.dsum, t * H + q[c].col);
    }
  };
  const int64_t step = (int64_t)gridDim.x * kRows;
  fetch((int64_t)blockIdx.x * kRows + slot);
  int turn = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < p.T; t0 += step, ++turn) {
    const int64_t t = t0 + slot;
    float s[kN][8], d[kN][8], a[kN][8], v[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < kN; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[c][j] = rs[c].at(j);
        d[c][j] = rd[c].at(j);
        a[c][j] = p.dsum ? ra[c].at(j) : 0.f;
        const bool mine = kAligned || j >= q[c].skip;
        v[0] += mine ? s[c][j] * s[c][j] : 0.f;
        v[1] += mine ? s[c][j] * d[c][j] * w[c].at(j) : 0.f;
      }
    fetch(t + step);
    Sum::sum(v, red, turn);
    const float rstd = 1.0f / sqrtf(v[0] / (float)H + p.eps);
    const float mean = v[1] * rstd / (float)H;          // of g xh
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = s[c][j] * rstd;
        o[j] = rstd * (d[c][j] * w[c].at(j) - xh * mean) + a[c][j];
        acc[c][j] += d[c][j] * xh;
      }
      if (q[c].in && t < p.T) {
        Eight<kF32, kAligned> e;
        e.set(o);
        e.store(p.dx, t * H + q[c].col);
      }
    }
  }
  float* to = p.part + ((int64_t)blockIdx.x * kRows + slot) * H;
#pragma unroll
  for (int c = 0; c < kN; ++c)
    if (q[c].in)
#pragma unroll
      for (int j = 0; j < 8; ++j) to[q[c].col + j] = acc[c][j];
}

// dw[h] = sum of the parts, in 64 bits: 16 columns by a workgroup, 64 slices of the parts.
constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void rmsnorm_dw_kernel(const float* __restrict__ part, int parts, int H,
                                                                 float* __restrict__ dw) {
  constexpr int kS = kSumThreads / 16;
  __shared__ double red[kS][16];
  const int le = threadIdx.x & 15, s = threadIdx.x >> 4, h = blockIdx.x * 16 + le;
  double sum = 0.0;
  if (h < H) {
    int i = s;
    for (; i + 7 * kS < parts; i += 8 * kS) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = part[(int64_t)(i + u * kS) * H + h];
#pragma unroll
      for (int u = 0; u < 8; ++u) sum += v[u];
    }
    for (; i < parts; i += kS) sum += part[(int64_t)i * H + h];
  }
  red[s][le] = sum;
  __syncthreads();
  for (int n = kS / 2; n >= 1; n /= 2) {
    if (s < n) red[s][le] += red[s + n][le];
    __syncthreads();
  }
  if (s == 0 && h < H) dw[h] = (float)red[0][le];
}

// ---- rows of fewer than 8 columns: a thread takes a row.
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

template <bool kF32, bool kW32>
__global__ __launch_bounds__(256) void narrow_rmsnorm_kernel(const NormFwd p) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= p.T) return;
  float s[8], sq = 0.f;
#pragma unroll
  for (int h = 0; h < 8; ++h) {
    s[h] = 0.f;
    if (h < p.H) {
      s[h] = get<kF32>(p.x, t * p.H + h);
      if (p.residual) {
        s[h] += get<kF32>(p.residual, t * p.H + h);
        if constexpr (!kF32) s[h] = bf16_to_f32(f32_to_bf16(s[h]));
      }
      sq += s[h] * s[h];
    }
  }
  const float rstd = 1.0f / sqrtf(sq / (float)p.H + p.eps);
#pragma unroll
  for (int h = 0; h < 8; ++h)
    if (h < p.H) {
      if (p.sum) put<kF32>(p.sum, t * p.H + h, s[h]);
      if (p.y) put<kF32>(p.y, t * p.H + h, s[h] * rstd * get<kW32>(p.weight, h));
    }
}

template <bool kF32, bool kW32>
__global__ __launch_bounds__(256) void narrow_rmsnorm_bwd_kernel(const NormBwd p) {
  __shared__ float red[4][8];
  float acc[8];
#pragma unroll
  for (int h = 0; h < 8; ++h) acc[h] = 0.f;
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < p.T; t += (int64_t)gridDim.x * 256) {
    float s[8], d[8], sq = 0.f, dot = 0.f;
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      s[h] = d[h] = 0.f;
      if (h < p.H) {
        s[h] = get<kF32>(p.s, t * p.H + h);
        d[h] = get<kF32>(p.dy, t * p.H + h);
        sq += s[h] * s[h];
        dot += s[h] * d[h] * get<kW32>(p.weight, h);
      }
    }
    const float rstd = 1.0f / sqrtf(sq / (float)p.H + p.eps), mean = dot * rstd / (float)p.H;
#pragma unroll
    for (int h = 0; h < 8; ++h)
      if (h < p.H) {
        const float xh = s[h] * rstd;
        float o = rstd * (d[h] * get<kW32>(p.weight, h) - xh * mean);
        if (p.dsum) o += get<kF32>(p.dsum, t * p.H + h);
        put<kF32>(p.dx, t * p.H + h, o);
        acc[h] += d[h] * xh;
      }
  }
#pragma unroll
  for (int h = 0; h < 8; ++h) {
    const float v = sum64(acc[h]);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6][h] = v;
  }
  __syncthreads();
  if (threadIdx.x < p.H) {
    float v = 0.f;
    for (int i = 0; i < 4; ++i) v += red[i][threadIdx.x];
    p.part[(int64_t)blockIdx.x * p.H + threadIdx.x] = v;
  }
}

// Lanes a row and pieces a lane.
struct Shape {
  int L, N;
};
Shape shape_of(int64_t H) {
  if (H <= 128) return {16, 1};
  if (H <= 256) return {16, 2};
  if (H <= 512) return {64, 1};
  if (H <= 1024) return {64, 2};
  if (H <= 2048) return {128, 2};
  if (H <= 4096) return {256, 2};
  if (H <= 8192) return {256, 4};
  if (H <= 16384) return {512, 4};
  return {1024, 4};
}
// Few rows: one piece a lane, for the time of one row.
Shape shape_few(int64_t H) {
  if (H <= 512) return {64, 1};
  if (H <= 2048) return {256, 1};
  if (H <= 4096) return {512, 1};
  if (H <= 8192) return {1024, 1};
  if (H <= 16384) return {1024, 2};
  return {1024, 4};
}
constexpr int64_t kFewRows = 512;

template <class F>
hipError_t with_shape(Shape s, F&& f) {
#define MOE_NORM_SHAPE(l, n) \
  if (s.L == l && s.N == n) return f(std::integral_constant<int, l>{}, std::integral_constant<int, n>{});
  MOE_NORM_SHAPE(16, 1) MOE_NORM_SHAPE(16, 2) MOE_NORM_SHAPE(64, 1) MOE_NORM_SHAPE(64, 2) MOE_NORM_SHAPE(128, 2)
  MOE_NORM_SHAPE(256, 1) MOE_NORM_SHAPE(256, 2) MOE_NORM_SHAPE(256, 4) MOE_NORM_SHAPE(512, 1) MOE_NORM_SHAPE(512, 4)
  MOE_NORM_SHAPE(1024, 1) MOE_NORM_SHAPE(1024, 2) MOE_NORM_SHAPE(1024, 4)
#undef MOE_NORM_SHAPE
  return hipErrorInvalidValue;
}

bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <bool kF32, bool kW32>
hipError_t launch_fwd(const NormFwd& p, hipStream_t st) {
  if (p.H < 8) {
    narrow_rmsnorm_kernel<kF32, kW32><<<(unsigned)((p.T + 255) / 256), 256, 0, st>>>(p);
    return hipGetLastError();
  }
  const bool few = p.T <= kFewRows;
  const Shape s = few ? shape_few(p.H) : shape_of(p.H);
  const bool aligned = p.H % 8 == 0 && at16(p.x) && at16(p.residual) && at16(p.weight) && at16(p.sum) && at16(p.y);
  const int rows = threads_of(s.L) / s.L;
  const int unit = few ? rows : rows > 16 ? rows : 16;
  const unsigned grid = (unsigned)((p.T + unit - 1) / unit);
  const size_t lds = p.q && unit > 1 ? (size_t)(p.H / 128) * unit * sizeof(float) : 0;
  return with_shape(s, [&](auto l, auto n) {
    constexpr int kL = decltype(l)::value, kN = decltype(n)::value;
    if (aligned) add_rmsnorm_kernel<kF32, kW32, kL, kN, true><<<grid, threads_of(kL), lds, st>>>(p, unit);
    else add_rmsnorm_kernel<kF32, kW32, kL, kN, false><<<grid, threads_of(kL), 0, st>>>(p, unit);
    return hipGetLastError();
  });
}

// Workgroups of the backward: kBwdBlocks at most, so that the sums' parts stay few.
constexpr int kBwdBlocks = 1024;
int bwd_blocks(int64_t T, int rows) {
  const int64_t need = (T + rows - 1) / rows;
  return (int)(need < kBwdBlocks ? need : kBwdBlocks);
}
struct BwdPlan {
  Shape s;
  int rows, blocks;       // rows: slots a workgroup, and so parts
};
BwdPlan plan_bwd(int64_t T, int64_t H) {
  if (H < 8) return {{0, 0}, 1, bwd_blocks(T, 256)};
  const Shape s = T <= kFewRows ? shape_few(H) : shape_of(H);
  const int rows = threads_of(s.L) / s.L;
  return {s, rows, bwd_blocks(T, rows)};
}

template <bool kF32, bool kW32>
hipError_t launch_bwd(const NormBwd& p, hipStream_t st) {
  const BwdPlan b = plan_bwd(p.T, p.H);
  hipError_t e;
  if (p.H < 8) {
    narrow_rmsnorm_bwd_kernel<kF32, kW32><<<b.blocks, 256, 0, st>>>(p);
    e = hipGetLastError();
  } else {
    const bool aligned = p.H % 8 == 0 && at16(p.dy) && at16(p.s) && at16(p.dsum) && at16(p.weight) && at16(p.dx);
    e = with_shape(b.s, [&](auto l, auto n) {
      constexpr int kL = decltype(l)::value, kN = decltype(n)::value;
      if (aligned) rmsnorm_bwd_kernel<kF32, kW32, kL, kN, true><<<b.blocks, threads_of(kL), 0, st>>>(p);
      else rmsnorm_bwd_kernel<kF32, kW32, kL, kN, false><<<b.blocks, threads_of(kL), 0, st>>>(p);
      return hipGetLastError();
    });
  }
  if (e != hipSuccess) return e;
  rmsnorm_dw_kernel<<<(unsigned)((p.H + 15) / 16), kSumThreads, 0, st>>>(p.part, b.blocks * b.rows, (int)p.H, p.dw);
  return hipGetLastError();
}

}  // namespace

size_t norm_bwd_part_bytes(int64_t T, int64_t H) {
  const BwdPlan b = plan_bwd(T, H);
  return (size_t)b.blocks * (size_t)b.rows * (size_t)H * sizeof(float);
}

hipError_t launch_add_rmsnorm(const NormFwd& p, bool f32, bool w32, hipStream_t st) {
  if (f32) return launch_fwd<true, true>(p, st);
  return w32 ? launch_fwd<false, true>(p, st) : launch_fwd<false, false>(p, st);
}

hipError_t launch_rmsnorm_bwd(const NormBwd& p, bool f32, bool w32, hipStream_t st) {
  if (f32) return launch_bwd<true, true>(p, st);
  return w32 ? launch_bwd<false, true>(p, st) : launch_bwd<false, false>(p, st);
}

}  // namespace moe
