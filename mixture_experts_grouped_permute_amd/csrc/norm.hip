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
// columns each, so that everything is read and written once.  Measured: 16384 x 4096 bf16 with residual, y and codes
// 98 us, 6.2 TB/s; 100003 x 1003 f32 169 us, 4.7 TB/s (rows at odd places: 14 % more is written, in partly filled lines);
// one row of 4096 2.4 us.  Backward 16384 x 4096 bf16 90 us, 6.0 TB/s, of which 5 are the weight's sum; 20011 x 1407
// f32 75 us, 4.5 TB/s.
#include "common.h"
#include "kernels.h"
#include "block_scale.h"
#include "eight.h"

#include <type_traits>

namespace moe {
namespace {

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
// (Rows of fewer than 8 columns have kernels of their own.)
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

// ---- forward.  A workgroup takes the kRows rows that its lanes hold and ends: others begin in its place, and their
// loads overlap (several rows one after the other, with the next one's loads behind the sums and the scales gathered
// in LDS into runs: 126 us at 16384 x 4096 bf16 with 16 rows, 117 with 4, 109 so).
// kOnce: the sum and y are stored past the caches.
template <bool kF32, bool kW32, int kL, int kN, bool kAligned, bool kOnce>
__global__ __launch_bounds__(threads_of(kL)) void add_rmsnorm_kernel(const NormFwd p, int64_t t0) {
  using Sum = RowSum<kL, 1>;
  __shared__ float red[Sum::kWords];
  const int tid = threadIdx.x, sub = tid % kL, H = (int)p.H;
  const int64_t t = t0 + (int64_t)blockIdx.x * Sum::kRows + tid / kL;
  Piece q[kN];
  bool in[kN];
  Eight<kF32, kAligned> x[kN], r[kN];
  Eight<kW32, kAligned> w[kN];
#pragma unroll
  for (int c = 0; c < kN; ++c) {
    q[c] = piece<kL, kAligned>(c, sub, H);
    in[c] = q[c].in && t < p.T;
    x[c].zero();
    r[c].zero();
    w[c].zero();
    if (in[c]) x[c].load_once(p.x, t * H + q[c].col);
  }
  if (p.residual) {
#pragma unroll
    for (int c = 0; c < kN; ++c)
      if (in[c]) r[c].load_once(p.residual, t * H + q[c].col);
  }
#pragma unroll
  for (int c = 0; c < kN; ++c)
    if (in[c]) w[c].load(p.weight, q[c].col);
  float s[kN][8], sq[1] = {0.f};
#pragma unroll
  for (int c = 0; c < kN; ++c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s[c][j] = x[c].at(j);
    if (p.residual) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[c][j] += r[c].at(j);
      x[c].set(s[c]);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[c][j] = x[c].at(j);   // as it is stored
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sq[0] += kAligned || j >= q[c].skip ? s[c][j] * s[c][j] : 0.f;
  }
  Sum::sum(sq, red, 0);
  const float rstd = 1.0f / sqrtf(sq[0] / (float)H + p.eps);
#pragma unroll
  for (int c = 0; c < kN; ++c) {
    const int64_t at = t * H + q[c].col;
    // (stored behind the row's last read, which may be of the same memory)
    if (p.sum && in[c]) x[c].template store<kOnce>(p.sum, at);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[c][j] = s[c][j] * rstd * w[c].at(j);
    if (p.y && in[c]) {
      x[c].set(s[c]);
      x[c].template store<kOnce>(p.y, at);
    }
    if constexpr (kAligned) {
      if (p.q) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = umax(m, __builtin_bit_cast(uint32_t, s[c][j]) & 0x7FFFFFFFu);
        const BlockScale b = block_scale(max16(m));      // 16 lanes hold 128 columns
        if (in[c]) {
          u32x2 o;
          o[0] = codes4(s[c][0], s[c][1], s[c][2], s[c][3], b.factor);
          o[1] = codes4(s[c][4], s[c][5], s[c][6], s[c][7], b.factor);
          *reinterpret_cast<u32x2*>(p.q + at) = o;
          if ((tid & 15) == 0) p.scales[(int64_t)(q[c].col >> 7) * p.T + t] = b.d;
        }
      }
    }
  }
}

// ---- backward.  Workgroup b takes rows b kRows, (b + grid) kRows, ..: dx, and sums of dy xh over them in registers
// till its end; the next rows' loads are in flight behind the sums of a row.  (kLate: where 1024 lanes hold 16 columns
// each or more, or 512 hold 32 in fp32, that would take more registers than there are -- 460 us at 2000 x 32768 bf16 --
// so the weight and ds are read when they are needed, and the next row when this one is done: 179 us, 2.9 TB/s.  1024
// lanes of 32 columns have too few even so, and keep 29 registers of each in scratch memory in bf16, 63 in fp32 -- 427 us
// at 2000 x 32768 -- and 55 and 89 at odd widths.)  The sums are fp32, T / (512 kRows) terms in turn; the parts are added
// in 64 bits.
// kOnce: dx is stored past the caches.
template <bool kF32, bool kW32, int kL, int kN, bool kAligned, bool kOnce>
__global__ __launch_bounds__(threads_of(kL)) void rmsnorm_bwd_kernel(const NormBwd p) {
  using Sum = RowSum<kL, 2>;
  constexpr int kRows = Sum::kRows;
  constexpr bool kLate = (kL == 1024 && kN >= 2) || (kF32 && kL == 512 && kN == 4);
  constexpr int kK = kLate ? 1 : kN;                    // pieces of the weight and ds in registers
  __shared__ float red[Sum::kWords];
  const int tid = threadIdx.x, sub = tid % kL, slot = tid / kL, H = (int)p.H;
  Piece q[kN];
  Eight<kW32, kAligned> w[kK];
  float acc[kN][8];
#pragma unroll
  for (int c = 0; c < kN; ++c) {
    q[c] = piece<kL, kAligned>(c, sub, H);
    if constexpr (!kLate) {
      w[c].zero();
      if (q[c].in) w[c].load(p.weight, q[c].col);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[c][j] = 0.f;
  }
  Eight<kF32, kAligned> rs[kN], rd[kN], ra[kK];
  const auto fetch = [&](int64_t t) {
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      rs[c].zero();
      rd[c].zero();
      if (q[c].in && t < p.T) {
        rs[c].load_once(p.s, t * H + q[c].col);
        rd[c].load_once(p.dy, t * H + q[c].col);
      }
    }
    if constexpr (!kLate)
      if (p.dsum) {
#pragma unroll
        for (int c = 0; c < kN; ++c)
          if (q[c].in && t < p.T) ra[c].load_once(p.dsum, t * H + q[c].col);
      }
  };
  const auto weight = [&](int c) -> const Eight<kW32, kAligned>& {
    if constexpr (kLate) {
      w[0].zero();
      if (q[c].in) w[0].load(p.weight, q[c].col);
      return w[0];
    } else {
      return w[c];
    }
  };
  const int64_t step = (int64_t)gridDim.x * kRows;
  fetch((int64_t)blockIdx.x * kRows + slot);
  int turn = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * kRows; t0 < p.T; t0 += step, ++turn) {
    const int64_t t = t0 + slot;
    float s[kN][8], d[kN][8], a[kK][8], v[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      const Eight<kW32, kAligned>& wc = weight(c);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[c][j] = rs[c].at(j);
        d[c][j] = rd[c].at(j);
        if constexpr (!kLate) a[c][j] = p.dsum ? ra[c].at(j) : 0.f;
        const bool mine = kAligned || j >= q[c].skip;
        v[0] += mine ? s[c][j] * s[c][j] : 0.f;
        v[1] += mine ? s[c][j] * d[c][j] * wc.at(j) : 0.f;
      }
    }
    if constexpr (!kLate) {
      fetch(t + step);
    } else {
      // (the values are unpacked again from the words: unpacked ones across the sums would not fit)
#pragma unroll
      for (int c = 0; c < kN; ++c)
#pragma unroll
        for (int i = 0; i < (kF32 ? 2 : 1); ++i) asm volatile("" : "+v"(rs[c].w[i]), "+v"(rd[c].w[i]));
    }
    Sum::sum(v, red, turn);
    // (a place without a row adds nothing to dw, also where eps is 0: its zeros times infinity would)
    const float rstd = t < p.T ? 1.0f / sqrtf(v[0] / (float)H + p.eps) : 0.f;
    const float mean = v[1] * rstd / (float)H;          // of g xh
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      const bool in = q[c].in && t < p.T;
      const Eight<kW32, kAligned>& wc = weight(c);
      if constexpr (kLate) {
        ra[0].zero();
        if (p.dsum && in) ra[0].load_once(p.dsum, t * H + q[c].col);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[0][j] = ra[0].at(j);
      }
      if constexpr (kLate) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s[c][j] = rs[c].at(j);
          d[c][j] = rd[c].at(j);
        }
      }
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = s[c][j] * rstd;
        o[j] = rstd * (d[c][j] * wc.at(j) - xh * mean) + a[kLate ? 0 : c][j];
        acc[c][j] += d[c][j] * xh;
      }
      if (in) {
        Eight<kF32, kAligned> e;
        e.set(o);
        // (late, and dx over ds: another wave may not have read its ds yet where a piece that was moved back repeats it)
        if (kLate && !kAligned && q[c].skip) e.store_from(p.dx, t * H + q[c].col, q[c].skip);
        else e.template store<kOnce>(p.dx, t * H + q[c].col);
      }
    }
    if constexpr (kLate) fetch(t + step);
  }
  // the slots' sums in turn, so that a workgroup leaves one part
  __shared__ float all[kRows > 1 ? kRows * kL * kN * 8 : 1];
  float* part = p.part + (int64_t)blockIdx.x * H;
  float* to = kRows > 1 ? all + slot * H : part;
#pragma unroll
  for (int c = 0; c < kN; ++c)
    if (q[c].in)
#pragma unroll
      for (int j = 0; j < 8; ++j) to[q[c].col + j] = acc[c][j];
  if constexpr (kRows > 1) {
    __syncthreads();
    for (int h = tid; h < H; h += threads_of(kL)) {
      float v = all[h];
#pragma unroll
      for (int i = 1; i < kRows; ++i) v += all[i * H + h];
      part[h] = v;
    }
  }
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
// Whether shape_of gives it as well: 512 rows of the others (of up to 16384 columns, 134 MB) stay in the caches.
constexpr bool for_many(int L, int N) { return !(N == 1 && L >= 256) && !(N == 2 && L == 1024); }
constexpr int64_t kOnceBytes = (int64_t)384 << 20, kOnceBytesBwd = (int64_t)576 << 20;

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
  // Past the caches where the call moves more than the last of them (256 MB) holds: 16384 x 4096 bf16 with residual,
  // y and codes 96 us instead of 109, and with two products that read y and the codes behind it 186 instead of 199;
  // 8192 x 4096, which the cache still holds, 112 with them against 115; 16384 x 4095 107 instead of 117, 8192 x 4095 55
  // against 51.
  const int64_t moved = p.T * p.H * (kF32 ? 4 : 2) * (1 + (p.y != nullptr) + 2 * (p.residual != nullptr));
  const bool once = moved > kOnceBytes;
  return with_shape(s, [&](auto l, auto n) {
    constexpr int kL = decltype(l)::value, kN = decltype(n)::value, kT = threads_of(kL);
    constexpr int64_t kMost = ((int64_t)1 << 31) / kT;   // workgroups of a launch (which takes fewer than 2^32 threads)
    for (int64_t t0 = 0; t0 < p.T; t0 += kMost * rows) {
      const int64_t need = (p.T - t0 + rows - 1) / rows;
      const unsigned grid = (unsigned)(need < kMost ? need : kMost);
      const auto go = [&](auto past) {
        constexpr bool kOnce = decltype(past)::value;
        if (aligned) add_rmsnorm_kernel<kF32, kW32, kL, kN, true, kOnce><<<grid, kT, 0, st>>>(p, t0);
        else add_rmsnorm_kernel<kF32, kW32, kL, kN, false, kOnce><<<grid, kT, 0, st>>>(p, t0);
      };
      if (once) go(std::bool_constant<for_many(kL, kN)>{});
      else go(std::false_type{});
    }
    return hipGetLastError();
  });
}

// Workgroups of the backward: few, since each leaves a part of dw (16384 x 4096 bf16: 88 us with 512, 96 with 1024;
// 65536 x 512: 47 with 512, 60 with 256), and one a CU where a row takes most of its registers (8192 x 8192 bf16: 94 us
// with 512, 89 with 256; 4096 x 16384: 109 and 98).
int bwd_blocks(int64_t T, int rows, int most) {
  const int64_t need = (T + rows - 1) / rows;
  return (int)(need < most ? need : most);
}
struct BwdPlan {
  Shape s;
  int blocks;
};
BwdPlan plan_bwd(int64_t T, int64_t H) {
  if (H < 8) return {{0, 0}, bwd_blocks(T, 256, 512)};
  const Shape s = T <= kFewRows ? shape_few(H) : shape_of(H);
  return {s, bwd_blocks(T, threads_of(s.L) / s.L, s.N >= 4 ? 256 : 512)};
}

template <bool kF32, bool kW32>
hipError_t launch_bwd(NormBwd p, hipStream_t st) {
  const BwdPlan b = plan_bwd(p.T, p.H);
  if (b.blocks == 1) p.part = p.dw;                     // the only part
  hipError_t e;
  if (p.H < 8) {
    narrow_rmsnorm_bwd_kernel<kF32, kW32><<<b.blocks, 256, 0, st>>>(p);
    e = hipGetLastError();
  } else {
    // past the caches from more on than forward, whose outputs are most of what it moves: 32768 x 4096 bf16 173 us instead
    // of 185, 100000 x 1003 149 instead of 163, 16384 x 4096 alike, 20011 x 1407 f32 (338 MB) 77 instead of 75
    const bool once = p.T * p.H * (kF32 ? 4 : 2) * (p.dsum ? 4 : 3) > kOnceBytesBwd;
    const bool aligned = p.H % 8 == 0 && at16(p.dy) && at16(p.s) && at16(p.dsum) && at16(p.weight) && at16(p.dx);
    e = with_shape(b.s, [&](auto l, auto n) {
      constexpr int kL = decltype(l)::value, kN = decltype(n)::value;
      const auto go = [&](auto past) {
        constexpr bool kOnce = decltype(past)::value;
        if (aligned) rmsnorm_bwd_kernel<kF32, kW32, kL, kN, true, kOnce><<<b.blocks, threads_of(kL), 0, st>>>(p);
        else rmsnorm_bwd_kernel<kF32, kW32, kL, kN, false, kOnce><<<b.blocks, threads_of(kL), 0, st>>>(p);
      };
      if (once) go(std::bool_constant<for_many(kL, kN)>{});
      else go(std::false_type{});
      return hipGetLastError();
    });
  }
  if (e != hipSuccess || b.blocks == 1) return e;
  rmsnorm_dw_kernel<<<(unsigned)((p.H + 15) / 16), kSumThreads, 0, st>>>(p.part, b.blocks, (int)p.H, p.dw);
  return hipGetLastError();
}

}  // namespace

size_t norm_bwd_part_bytes(int64_t T, int64_t H) {
  const BwdPlan b = plan_bwd(T, H);
  return (size_t)b.blocks * (size_t)H * sizeof(float);
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
