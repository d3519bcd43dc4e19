// FP8 quantization with one fp32 scale per block of 128 for gfx950: rows (1 x 128), tokens (128 x 1,
// transposed) and weights (128 x 128).
//
// The rule of a block's scale and codes is block_scale.h's.  One read of x and one write of the codes bound all three.
#include "common.h"
#include "kernels.h"
#include "block_scale.h"

namespace moe {
namespace {

// 8 values of a row as loaded: bf16 in 4 words, fp32 in 8.
template <bool kF32>
struct Raw8 {
  u32x4 w[kF32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* x, int64_t off) {
    const u32x4* s = reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(x) + off * (kF32 ? 4 : 2));
    w[0] = s[0];
    if constexpr (kF32) w[1] = s[1];
  }
  // the same past the caches, for values that are read once
  __device__ __forceinline__ void load_once(const void* x, int64_t off) {
    const u32x4* s = reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(x) + off * (kF32 ? 4 : 2));
    w[0] = __builtin_nontemporal_load(s);
    if constexpr (kF32) w[1] = __builtin_nontemporal_load(s + 1);
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
  __device__ __forceinline__ uint32_t mag(int i) const { return __builtin_bit_cast(uint32_t, at(i)) & 0x7FFFFFFFu; }
};

// ---- rows.  A wave takes 4 blocks (512 columns) of kRowsPerWave rows, 16 lanes per block: all its
// loads are in flight at once, and a load covers 1 KB (bf16) of one row.  The scales leave block-major
// ([cols / 128, rows], the layout a product's stages read), so the workgroup gathers those of its
// rows in LDS and writes them as runs of consecutive rows.  Workgroups run along a row's columns first, so
// that those in flight together cover whole rows: 51 us at 16384 x 4096 bf16 with the rows first, 34 so, 33
// with 4 rows a wave instead of 8.
constexpr int kRowsPerWave = 4;
constexpr int kRowTile = 4 * kRowsPerWave;

template <bool kF32>
__global__ __launch_bounds__(256) void block_rows_kernel(const void* __restrict__ x, int64_t rows, int64_t cols,
                                                           const int32_t* __restrict__ src_index, int src_k,
                                                           const int32_t* live, uint8_t* __restrict__ q,
                                                           float* __restrict__ scales) {
  __shared__ float sc[4][kRowTile];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int nc = (int)((cols + 511) / 512);
  const int64_t bx = blockIdx.x / nc, by = blockIdx.x % nc;
  const int64_t r0 = bx * kRowTile, n = live ? min((int64_t)*live, rows) : rows;
  if (r0 >= n) return;
  const int64_t col = by * 512 + lane * 8;
  const bool in_c = col < cols;                          // uniform over the 16 lanes of a block
  Raw8<kF32> v[kRowsPerWave];
#pragma unroll
  for (int i = 0; i < kRowsPerWave; ++i) {
    const int64_t r = r0 + wave * kRowsPerWave + i;
    int64_t src = r < n ? r : 0;
    if (src_index) src = src_index[src] / src_k;
    v[i].load(x, src * cols + (in_c ? col : 0));
  }
#pragma unroll
  for (int i = 0; i < kRowsPerWave; ++i) {
    const int64_t r = r0 + wave * kRowsPerWave + i;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = umax(m, v[i].mag(j));
    const BlockScale s = block_scale(max16(m));
    if ((lane & 15) == 0) sc[lane >> 4][wave * kRowsPerWave + i] = s.d;
    if (in_c && r < n) {
      u32x2 o;
      o[0] = codes4(v[i].at(0), v[i].at(1), v[i].at(2), v[i].at(3), s.factor);
      o[1] = codes4(v[i].at(4), v[i].at(5), v[i].at(6), v[i].at(7), s.factor);
      *reinterpret_cast<u32x2*>(q + r * cols + col) = o;
    }
  }
  __syncthreads();
  if (tid < 4 * kRowTile) {
    const int b = tid / kRowTile, rr = tid % kRowTile;
    const int64_t kb = by * 4 + b;
    if (kb < cols / 128 && r0 + rr < n) scales[kb * rows + r0 + rr] = sc[b][rr];
  }
}

// ---- tiles of 128 rows x 128 columns: a thread holds 8 rows x 8 columns, so that a column's 8 codes
// are packed straight from its registers -- the transpose costs no data movement there -- and each
// thread's 8 bytes of a column meet those of the 15 other row groups in LDS, to leave as whole
// 128-byte lines.  Loads and stores pass the caches by: 131072 x 1408 tokens 120 -> 105 us, 8 matrices of
// 4096 x 14336 transposed 275 -> 245 (the rows' kernel, whose codes a product reads next, gains nothing by it).
//   kTokens  blocks of 128 rows x 1 column; the rows are the padded rows of expert segments
//   kPlain   one 128 x 128 block of a weight matrix, codes in its own layout
//   kTrans   the same, codes transposed
enum { kTokens, kPlain, kTrans };

struct WTab {
  const uint16_t* w[kMaxExperts];
};
struct TileP {
  const void* x;
  int64_t rows, cols;
  const int32_t* goff;       // kTokens: [groups + 1], or null: one group of all rows
  int groups;
  int64_t rows_pad;
  const int32_t* src_index;  // kTokens: segmented row r is row src_index[r] / src_k of x, or null
  int src_k;
  const int32_t* skip;       // weights: matrices with skip[e] == 0 are left alone
  uint8_t* q;
  float* scales;
};

// The order of a weight matrix's tiles.  kPlain: along the rows, which it reads and writes (28672 x 4096, 8
// matrices: 485 us; down the columns, 256 bytes of every 8 KB at a time, 669).  kTrans reads along the rows and
// writes along the columns: 8 tiles of a row, then the next row's (28672 x 4096: 526 us, 587 down
// the columns, 535 along the rows; 4096 x 14336: 245, 251, 281; 64 of 2816 x 2048: 201, 193, 208).
__host__ __device__ constexpr int64_t walk_cols(int64_t tiles) { return tiles < 8 ? tiles : 8; }

constexpr int kPitch = 128 + 8;   // LDS bytes per output row

template <bool kF32, int kMode>
__global__ __launch_bounds__(256) void block_tile_kernel(const TileP p, const WTab tab) {
  __shared__ int s_src[128];
  __shared__ int s_pad[kMaxExperts + 1], s_off[kMaxExperts + 1];
  __shared__ uint32_t s_max[16][kMode == kTokens ? 128 : 1];
  __shared__ __attribute__((aligned(16))) float s_f[128];
  __shared__ __attribute__((aligned(16))) uint8_t stage[kMode == kPlain ? 16 : 128 * kPitch];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int ck = tid & 15, g = tid >> 4;                  // columns 8 ck .., rows 8 g ..
  const void* x = p.x;
  int64_t e = 0;
  if constexpr (kMode != kTokens) {
    e = blockIdx.z;
    if (p.skip && p.skip[e] == 0) return;
#if defined(__HIP_DEVICE_COMPILE__)
    // the table stays in the kernel-argument segment (a uniform load, no private copy)
    x = *reinterpret_cast<const uint16_t* const*>(reinterpret_cast<const char*>(__builtin_amdgcn_kernarg_segment_ptr()) +
                                                  sizeof(TileP) + sizeof(const uint16_t*) * (size_t)e);
#else
    x = tab.w[e];
#endif
  }
  const int64_t nct = (p.cols + 127) / 128;
  int64_t rb = blockIdx.x, ct0 = blockIdx.y;
  if constexpr (kMode == kPlain) {
    rb = blockIdx.x / nct;
    ct0 = blockIdx.x % nct;
  } else if constexpr (kMode == kTrans) {
    const int64_t n = walk_cols(nct), per = (p.rows + 127) / 128 * n, in = blockIdx.x % per;
    rb = in / n;
    ct0 = blockIdx.x / per * n + in % n;
  }
  const int64_t p0 = rb * 128;
  bool dead = false;                                      // kTokens: no row of this tile has a token
  if constexpr (kMode == kTokens) {
    // padded segment starts, one wave scanning 64 groups at a time.  The offsets are device data:
    // clamped into [0, rows] and made non-decreasing, so no access leaves x.
    int groups = p.groups;
    if (wave == 0) {
      int carry = 0, top = p.goff ? min(max(p.goff[0], 0), (int)p.rows) : 0;
      for (int g0 = 0; g0 < groups; g0 += 64) {
        const int gi = g0 + lane;
        int hi = gi < groups ? (p.goff ? min(max(p.goff[gi + 1], 0), (int)p.rows) : (int)p.rows) : 0;
        hi = max(hi, top);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
          const int o = __shfl_up(hi, d, 64);
          if (lane >= d) hi = max(hi, o);
        }
        int lo = __shfl_up(hi, 1, 64);
        if (lane == 0) lo = top;
        const int pad = gi < groups ? (hi - lo + 127) / 128 * 128 : 0;
        int inc = pad;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
          const int o = __shfl_up(inc, d, 64);
          if (lane >= d) inc += o;
        }
        if (gi < groups) {
          s_off[gi] = lo;
          s_pad[gi] = carry + inc - pad;
        }
        const int last = min(63, groups - g0 - 1);
        top = __shfl(hi, last, 64);
        carry += __shfl(inc, 63, 64);
      }
      if (lane == 0) {
        s_off[groups] = top;
        s_pad[groups] = carry;
      }
    }
    __syncthreads();
    dead = p0 >= s_pad[groups];
    if (tid < 128) {
      int src = -1;
      if (!dead) {
        int lo = 0, hi = groups - 1;                      // largest group with s_pad <= p0
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (s_pad[mid] <= p0) lo = mid; else hi = mid - 1;
        }
        const int64_t sr = s_off[lo] + (p0 + tid - s_pad[lo]);
        if (sr < s_off[lo + 1]) {
          src = (int)sr;
          if (p.src_index) {
            src = p.src_index[src];
            src = src < 0 ? -1 : src / p.src_k;
          }
        }
      }
      s_src[tid] = src;
    }
    __syncthreads();
  }
  for (int64_t ct = ct0; ct < nct; ct += kMode == kTokens ? gridDim.y : nct) {
    const int64_t c0 = ct * 128, col = c0 + 8 * ck;
    const bool in_c = col < p.cols;
    Raw8<kF32> v[8];
    if (!dead) {
      // a piece without a source reads the start of x and is replaced by zeros, so that no branch
      // separates the loads
      bool ok[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        int64_t src;
        if constexpr (kMode == kTokens) {
          src = s_src[8 * g + i];
          ok[i] = in_c && src >= 0;
        } else {
          src = p0 + 8 * g + i;
          ok[i] = in_c && src < p.rows;
        }
        v[i].load_once(x, ok[i] ? src * p.cols + col : 0);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!ok[i]) v[i].zero();
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i].zero();
    }
    float f[8];
    if constexpr (kMode == kTokens) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = umax(m, v[i].mag(j));
        s_max[g][8 * ck + j] = m;
      }
      __syncthreads();
      if (tid < 128) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = umax(m, s_max[i][tid]);
        const BlockScale s = block_scale(m);
        s_f[tid] = s.factor;
        if (c0 + tid < p.cols) p.scales[rb * p.cols + c0 + tid] = s.d;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = s_f[8 * ck + j];
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) m = umax(m, v[i].mag(j));
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) m = umax(m, (uint32_t)__shfl_xor((int)m, d, 64));
      if (lane == 0) s_max[wave][0] = m;
      __syncthreads();
      m = umax(umax(s_max[0][0], s_max[1][0]), umax(s_max[2][0], s_max[3][0]));
      const BlockScale s = block_scale(m);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = s.factor;
      const int64_t nb = (p.rows + 127) / 128, kb = (p.cols + 127) / 128;
      if (tid == 0)
        p.scales[e * nb * kb + (kMode == kPlain ? rb * kb + ct : ct * nb + rb)] = s.d;
      if constexpr (kMode == kPlain) {
        uint8_t* qe = p.q + e * p.rows * p.cols;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t r = p0 + 8 * g + i;
          if (in_c && r < p.rows) {
            u32x2 o;
            o[0] = codes4(v[i].at(0), v[i].at(1), v[i].at(2), v[i].at(3), s.factor);
            o[1] = codes4(v[i].at(4), v[i].at(5), v[i].at(6), v[i].at(7), s.factor);
            __builtin_nontemporal_store(o, reinterpret_cast<u32x2*>(qe + r * p.cols + col));
          }
        }
        __syncthreads();                                  // s_max is used again by the next tile
      }
    }
    if constexpr (kMode != kPlain) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u32x2 o;
        o[0] = codes4(v[0].at(j), v[1].at(j), v[2].at(j), v[3].at(j), f[j]);
        o[1] = codes4(v[4].at(j), v[5].at(j), v[6].at(j), v[7].at(j), f[j]);
        *reinterpret_cast<u32x2*>(stage + (8 * ck + j) * kPitch + 8 * g) = o;
      }
      __syncthreads();
      const int64_t ld = kMode == kTokens ? p.rows_pad : p.rows;
      uint8_t* qe = p.q + (kMode == kTokens ? 0 : e * p.rows * p.cols);
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int id = tid + 256 * it, lc = id >> 3, pc = id & 7;
        const u32x2* s2 = reinterpret_cast<const u32x2*>(stage + lc * kPitch + 16 * pc);
        const u32x2 a = s2[0], b = s2[1];
        if (c0 + lc < p.cols)
          __builtin_nontemporal_store(u32x4{a[0], a[1], b[0], b[1]}, reinterpret_cast<u32x4*>(qe + (c0 + lc) * ld + p0 + 16 * pc));
      }
      __syncthreads();                                    // the stage and s_max are used again
    }
  }
}

}  // namespace

namespace {
int64_t block_rows_groups(int64_t rows, int64_t cols) { return (rows + kRowTile - 1) / kRowTile * ((cols + 511) / 512); }
}  // namespace

bool block_rows_fits(int64_t rows, int64_t cols) { return block_rows_groups(rows, cols) < ((int64_t)1 << 32) / 256; }

hipError_t launch_block_rows(const void* x, bool x_f32, int64_t rows, int64_t cols, const int32_t* src_index, int src_k,
                             const int32_t* live, uint8_t* q, float* scales, hipStream_t st) {
  const dim3 grid((unsigned)block_rows_groups(rows, cols));
  if (x_f32) block_rows_kernel<true><<<grid, 256, 0, st>>>(x, rows, cols, src_index, src_k, live, q, scales);
  else block_rows_kernel<false><<<grid, 256, 0, st>>>(x, rows, cols, src_index, src_k, live, q, scales);
  return hipGetLastError();
}

hipError_t launch_block_tokens(const void* x, bool x_f32, int64_t rows, int64_t cols, const int32_t* offsets, int groups,
                               int64_t rows_pad, const int32_t* src_index, int src_k, uint8_t* q, float* scales,
                               hipStream_t st) {
  TileP p{};
  p.x = x;
  p.rows = rows;
  p.cols = cols;
  p.goff = offsets;
  p.groups = groups;
  p.rows_pad = rows_pad;
  p.src_index = src_index;
  p.src_k = src_k;
  p.q = q;
  p.scales = scales;
  const int64_t bx = rows_pad / 128, ct = (cols + 127) / 128;
  const dim3 grid((unsigned)bx, (unsigned)(ct < 65535 ? ct : 65535));
  const WTab none{};
  if (x_f32) block_tile_kernel<true, kTokens><<<grid, 256, 0, st>>>(p, none);
  else block_tile_kernel<false, kTokens><<<grid, 256, 0, st>>>(p, none);
  return hipGetLastError();
}

hipError_t launch_block_weights(const void* const* w, int E, int64_t rows, int64_t cols, bool transposed,
                                const int32_t* skip, uint8_t* q, float* scales, hipStream_t st) {
  TileP p{};
  p.rows = rows;
  p.cols = cols;
  p.skip = skip;
  p.q = q;
  p.scales = scales;
  WTab tab{};
  for (int e = 0; e < E; ++e) tab.w[e] = reinterpret_cast<const uint16_t*>(w[e]);
  const int64_t ct = (cols + 127) / 128;
  const int64_t n = walk_cols(ct), walk = transposed ? (ct + n - 1) / n * n : ct;
  const dim3 grid((unsigned)((rows + 127) / 128 * walk), 1, (unsigned)E);
  if (transposed) block_tile_kernel<false, kTrans><<<grid, 256, 0, st>>>(p, tab);
  else block_tile_kernel<false, kPlain><<<grid, 256, 0, st>>>(p, tab);
  return hipGetLastError();
}

}  // namespace moe
