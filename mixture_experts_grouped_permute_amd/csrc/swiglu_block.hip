// ScaledSwiGLU between the block-scaled products of the expert MLP, forward and backward (gfx950).
//
//   forward   h = silu(g) u p, quantized in blocks of 128 columns (the down product's operand)
//   backward  a = silu(g) u;  dprob = sum_i dh_i a_i;  du = dh p silu(g);
//             dg = dh p u s (1 + g (1 - s)), s = sigmoid(g); [dg | du] rounded to bf16 and quantized in blocks
//             of 128 columns (the gate-up dgrad's operand)
//
// One read of the gate-up output (and dh), one write each of the codes and of the bf16 copies that a
// later product needs: memory bounds both (16384 rows, I = 14336: 242 us forward, 570 backward, 4.9 and 5.0
// TB/s, of a copy's 5.2).  16 lanes hold a block of 128 columns, 8 each, as in the
// row quantizer, and share its amax by DPP.
#include "common.h"
#include "kernels.h"
#include "block_scale.h"

namespace moe {
namespace {

__device__ __forceinline__ void load8_bf16(const uint16_t* x, float (&v)[8]) {
  const u32x4 w = *reinterpret_cast<const u32x4*>(x);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = w[i];
    v[2 * i] = __builtin_bit_cast(float, u << 16);
    v[2 * i + 1] = __builtin_bit_cast(float, u & 0xFFFF0000u);
  }
}
__device__ __forceinline__ u32x4 pack8_bf16(const float (&v)[8]) {
  return u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}
// codes of the lane's 8 values of a block shared by 16 lanes; d: the block's scale
__device__ __forceinline__ u32x2 quant8(const float (&v)[8], float& d) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = umax(m, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
  const BlockScale s = block_scale(max16(m));
  d = s.d;
  return u32x2{codes4(v[0], v[1], v[2], v[3], s.factor), codes4(v[4], v[5], v[6], v[7], s.factor)};
}
__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

// Workgroup (x, y): rows 32 x + [0, 32), a wave 8 of them, columns 512 y + [0, 512).
constexpr int kRows = 8;

__global__ __launch_bounds__(256) void swiglu_block_kernel(const uint16_t* __restrict__ gu, const float* __restrict__ prob,
                                                             const int32_t* live, int64_t R, int64_t I,
                                                             uint8_t* __restrict__ q, float* __restrict__ scales,
                                                             uint16_t* __restrict__ save_h, float* __restrict__ h_f32) {
  __shared__ float sc[4][4 * kRows];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t n = min((int64_t)*live, R), r0 = (int64_t)blockIdx.x * 4 * kRows;
  if (r0 >= n) return;
  const int64_t col = (int64_t)blockIdx.y * 512 + lane * 8;
  const bool in_c = col < I;                              // uniform over the 16 lanes of a block
#pragma unroll 2
  for (int i = 0; i < kRows; ++i) {
    const int64_t r = r0 + wave * kRows + i, rr = r < n ? r : n - 1;
    float g[8], u[8], v[8], d;
    load8_bf16(gu + rr * 2 * I + (in_c ? col : 0), g);
    load8_bf16(gu + rr * 2 * I + I + (in_c ? col : 0), u);
    const float p = prob[rr];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = g[j] * sigmoid(g[j]) * u[j] * p;
    const u32x2 o = quant8(v, d);
    if ((lane & 15) == 0) sc[lane >> 4][wave * kRows + i] = d;
    if (in_c && r < n) {
      *reinterpret_cast<u32x2*>(q + r * I + col) = o;
      if (save_h) *reinterpret_cast<u32x4*>(save_h + r * I + col) = pack8_bf16(v);
      if (h_f32) {
        f32x4* h = reinterpret_cast<f32x4*>(h_f32 + r * I + col);
        h[0] = f32x4{v[0], v[1], v[2], v[3]};
        h[1] = f32x4{v[4], v[5], v[6], v[7]};
      }
    }
  }
  __syncthreads();
  if (tid < 16 * kRows) {
    const int b = tid / (4 * kRows), rr = tid % (4 * kRows);
    const int64_t kb = (int64_t)blockIdx.y * 4 + b;
    if (kb < I / 128 && r0 + rr < n) scales[kb * R + r0 + rr] = sc[b][rr];
  }
}

// A wave takes a whole row (its dprob is a sum over the row), 512 columns of each half at a time.
__global__ __launch_bounds__(256) void swiglu_block_bwd_kernel(const uint16_t* __restrict__ dh, const uint16_t* __restrict__ gu,
                                                                 const float* __restrict__ prob, const int32_t* live,
                                                                 int64_t R, int64_t I, uint16_t* __restrict__ dgu,
                                                                 uint8_t* __restrict__ q, float* __restrict__ scales,
                                                                 float* __restrict__ dprob) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t n = min((int64_t)*live, R), r = (int64_t)blockIdx.x * 4 + wave;
  if (r >= n) return;                                     // uniform over the wave
  const float p = prob[r];
  float dot = 0.f;
  for (int64_t c0 = 0; c0 < I; c0 += 512) {
    const int64_t col = c0 + lane * 8;
    const bool in_c = col < I;                            // uniform over the 16 lanes of a block
    const int64_t at = in_c ? col : 0;
    float g[8], u[8], e[8];
    load8_bf16(gu + r * 2 * I + at, g);
    load8_bf16(gu + r * 2 * I + I + at, u);
    load8_bf16(dh + r * I + at, e);
    float dg[8], du[8], sg, su;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = sigmoid(g[j]), sl = g[j] * s, x = in_c ? e[j] : 0.f;
      dot += x * (sl * u[j]);
      const float da = x * p;
      // the operand of both of FC1's gradients is the bf16 value
      du[j] = bf16_to_f32(f32_to_bf16(da * sl));
      dg[j] = bf16_to_f32(f32_to_bf16(da * u[j] * (s * (1.0f + g[j] * (1.0f - s)))));
    }
    const u32x2 og = quant8(dg, sg), ou = quant8(du, su);
    if (in_c) {
      *reinterpret_cast<u32x4*>(dgu + r * 2 * I + col) = pack8_bf16(dg);
      *reinterpret_cast<u32x4*>(dgu + r * 2 * I + I + col) = pack8_bf16(du);
      *reinterpret_cast<u32x2*>(q + r * 2 * I + col) = og;
      *reinterpret_cast<u32x2*>(q + r * 2 * I + I + col) = ou;
      if ((lane & 15) == 0) {
        scales[(col / 128) * R + r] = sg;
        scales[((I + col) / 128) * R + r] = su;
      }
    }
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) dot += __shfl_xor(dot, d, 64);
  if (lane == 0) dprob[r] = dot;
}

// The E pointers of a host table, in device memory (a kernel that reads one per tile takes them there).
struct PtrTab {
  void* p[kMaxExperts];
};
__global__ __launch_bounds__(256) void pointer_table_kernel(const PtrTab tab, int E, void** out) {
  if ((int)threadIdx.x >= E) return;
#if defined(__HIP_DEVICE_COMPILE__)
  out[threadIdx.x] = reinterpret_cast<void* const*>(
      reinterpret_cast<const char*>(__builtin_amdgcn_kernarg_segment_ptr()))[threadIdx.x];
#else
  out[threadIdx.x] = tab.p[threadIdx.x];
#endif
}

}  // namespace

hipError_t launch_swiglu_block(const void* gu, const float* prob, const int32_t* live, int64_t R, int64_t I, uint8_t* q,
                               float* scales, void* save_h, float* h_f32, hipStream_t st) {
  const dim3 grid((unsigned)((R + 4 * kRows - 1) / (4 * kRows)), (unsigned)((I + 511) / 512));
  swiglu_block_kernel<<<grid, 256, 0, st>>>(reinterpret_cast<const uint16_t*>(gu), prob, live, R, I, q, scales,
                                           reinterpret_cast<uint16_t*>(save_h), h_f32);
  return hipGetLastError();
}

hipError_t launch_swiglu_block_bwd(const void* dh, const void* gu, const float* prob, const int32_t* live, int64_t R,
                                   int64_t I, void* dgu, uint8_t* q, float* scales, float* dprob, hipStream_t st) {
  swiglu_block_bwd_kernel<<<(unsigned)((R + 3) / 4), 256, 0, st>>>(
      reinterpret_cast<const uint16_t*>(dh), reinterpret_cast<const uint16_t*>(gu), prob, live, R, I,
      reinterpret_cast<uint16_t*>(dgu), q, scales, dprob);
  return hipGetLastError();
}

hipError_t launch_pointer_table(void* const* ptrs, int E, void** out, hipStream_t st) {
  PtrTab t{};
  for (int e = 0; e < E; ++e) t.p[e] = ptrs[e];
  pointer_table_kernel<<<1, 256, 0, st>>>(t, E, out);
  return hipGetLastError();
}

}  // namespace moe
