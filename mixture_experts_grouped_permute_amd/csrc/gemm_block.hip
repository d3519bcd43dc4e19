// Grouped products of E4M3 operands that carry one fp32 scale per block of 128 along K (gfx950).
//
//   product          out[r, n]  = sum_b a_s[b, r] w_s[e, n / 128, b] sum_{k in b} a[r, k] w[e, n, k]
//                    for the rows r of expert e (forward: N outputs; dgrad: the transposed weights)
//   weight gradient  dw[e, n, k] = sum_b dy_s[b, n] x_s[b, k] sum_{t in b} dy[n, t] x[k, t]
//                    over the blocks b of 128 tokens of expert e (token-axis operands)
//
// The matrix cores have no fp32 block scale (their scaled form takes powers of two per 32 values), so
// a block's 128 products are summed by one v_mfma_f32_16x16x128_f8f6f4 from a zero accumulator and the
// four results a lane holds are added, scaled, to the running sum by four VALU fused multiply-adds.
// 16 x 16 x 128 is the shape whose K is exactly one block: a 32 x 32 x 64 pair would need 16 temporary
// registers per tile instead of 4.  The running sums have to be in registers the VALU reads, so a wave
// owns 128 x 64 outputs (128 registers) and 8 waves, two per SIMD, share a 256 x 256 tile: while one
// wave's VALU adds a block, the other's MFMAs run.  An MFMA takes 32 cycles and 16 of the VALU's issue: four
// adds fit beside it (measured 33 cycles), the weight gradient's eight instructions, whose scale differs
// in every column as well, make it 48.
//
// fp32 outputs take another path (kWide).  The E4M3 matrix instructions align the products of a group to
// its largest one and drop what falls below about 2^-16 of it: 1.3e-5 (normwise) off on Gaussian
// codes, under a bf16 output's own 1.7e-3, but not what an fp32 output promises.  The same codes,
// converted to bf16 (exact) and multiplied by v_mfma_f32_16x16x32_bf16, gave 1e-8.  That costs twice the
// matrix cycles and 16 registers per converted fragment, so its waves own 64 x 64 of a 256 x 128 tile.
// (16384 x 4096 x 14336: 1627 us, of 1607 at a large bf16 library product's rate, where bf16 outputs take 810-840.)
//
// A stage is one block of K: 128 bytes of 256 A rows and 256 B rows, loaded straight to LDS into one
// of two buffers while the other is multiplied, with the stage's 512 scales beside them.  Tiles are
// dealt to a persistent grid of one workgroup per CU from the expert offsets on the device.  Products of
// few rows an expert (blk_few_kernel) only read the weights, with 16-row tiles and no LDS stages.
#include "gemm_core.h"

namespace moe {
namespace {
using namespace gemm;

typedef float f32x4v __attribute__((ext_vector_type(4)));

constexpr int kPartRounds = 2;   // rounds of parts of the split tiles, at most

struct BlkKArgs {
  const uint8_t* a;
  const float* a_s;
  const uint8_t* b;
  const float* b_s;
  const int32_t* offsets;
  uint8_t* out;
  void* const* tab;  // weight gradient: the experts' outputs, in place of out, or null
  int64_t rows;      // product: R; weight gradient: rows_pad (the token axis' length)
  int64_t N, K;      // outputs per row, and product: the contracted length / weight gradient: columns
  int E, nN;
  float* part;       // fp32 sums of the split tiles' parts, or null: no tile is split
  int part_rows;     // rows of a part's slot
  int part_cost;     // of a part, in blocks' products
};

// Row offsets, K units (weight gradient) and tile prefix of the experts.
struct BlkSched {
  int off[kMaxExperts + 1];    // first row of the expert; weight gradient: its first block of 128 tokens
  int units[kMaxExperts];      // product: rows of the expert; weight gradient: its blocks
  int tile[kMaxExperts + 1];   // product: first tile of the expert
  int order[kMaxExperts];      // weight gradient: the experts by falling number of blocks
  int total;                   // tiles
};

// One wave scans the offsets, 64 experts at a time.  They are device data: clamped into [0, rows] and
// made non-decreasing, so that no access leaves the buffers whatever they hold.  kRows: of a tile.
// Every expert has the same number of weight-gradient tiles, but tiles of its own length; in falling order
// of length, and dealt to the workgroups in alternating directions, their sums come out even (64 experts of
// Zipf popularity, 176 tiles each: the longest workgroup has 1.08 times the mean, 1.22 in the experts' own
// order; 1769 -> 1682 us).
template <bool kWgrad, int kRows = kBM>
__device__ __forceinline__ void build_blk_sched(BlkSched& s, const BlkKArgs& p, int nM) {
  const int lane = threadIdx.x & 63;
  if (threadIdx.x < 64) {
    const int R = (int)p.rows;
    int carry = 0, tcarry = 0, top = min(max(p.offsets[0], 0), R);
    for (int e0 = 0; e0 < p.E; e0 += 64) {
      const int e = e0 + lane;
      int hi = e < p.E ? min(max(p.offsets[e + 1], 0), R) : 0;
      hi = max(hi, top);
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(hi, d, 64);
        if (lane >= d) hi = max(hi, o);
      }
      int lo = __shfl_up(hi, 1, 64);
      if (lane == 0) lo = top;
      const int cnt = e < p.E ? hi - lo : 0;
      const int nblk = (cnt + 127) / 128;
      int t = (cnt + kRows - 1) / kRows * p.nN;
      int inc = kWgrad ? nblk : 0;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(inc, d, 64), ot = __shfl_up(t, d, 64);
        if (lane >= d) { inc += o; t += ot; }
      }
      int before = __shfl_up(t, 1, 64);
      if (lane == 0) before = 0;
      if (e < p.E) {
        if (kWgrad) {
          // the padded segments fit the token axis unless the offsets lie: cut there
          const int all = R / 128, first = min(carry + inc - nblk, all);
          s.off[e] = first;
          s.units[e] = min(nblk, all - first);
        } else {
          s.off[e] = lo;
          s.units[e] = cnt;
          s.tile[e] = tcarry + before;
        }
      }
      const int last = min(63, p.E - e0 - 1);
      top = __shfl(hi, last, 64);
      carry += __shfl(inc, 63, 64);
      tcarry += __shfl(t, 63, 64);
    }
    if (lane == 0) {
      if (!kWgrad) s.tile[p.E] = tcarry;
      s.total = kWgrad ? p.E * nM * p.nN : tcarry;
    }
  }
  __syncthreads();
  if (kWgrad) {
    const int e = threadIdx.x;
    if (e < p.E) {
      const int u = s.units[e];
      int rank = 0;
      for (int i = 0; i < p.E; ++i) rank += s.units[i] > u || (s.units[i] == u && i < e);
      s.order[rank] = e;
    }
    __syncthreads();
  }
}

// Largest e with tile[e] <= t, for the whole wave: the prefix does not fall, and of experts without
// tiles, which share a value, that is the last, which has the tiles.  (One LDS read in place of log2 E
// dependent ones.)
__device__ __forceinline__ int blk_find(const BlkSched& s, int E, int t) {
  const int lane = threadIdx.x & 63;
  int n = -1;
  for (int e0 = 0; e0 < E; e0 += 64) n += __popcll(__ballot(e0 + lane < E && s.tile[e0 + lane] <= t));
  return n;
}

// Expert of a tile, and the tile's index among the expert's.
template <bool kWgrad>
__device__ __forceinline__ int blk_expert(const BlkSched& s, const BlkKArgs& p, int nM, int tile, int& local) {
  if (kWgrad) {
    const int per = nM * p.nN, r = tile / per;
    local = tile - r * per;
    return s.order[r];
  }
  const int e = blk_find(s, p.E, tile);
  local = tile - s.tile[e];
  return e;
}

// The tiles of the last, partly filled round -- of all of them, where there are fewer than workgroups --
// are split along the contracted axis into S parts each: tiles [full, total) as (total - full) S items, which
// the workgroups take in one round, or in two where that is shorter (more than half of the workgroups had a
// tile).  A part has more blocks than part_cost, which is what writing and reading it takes, in blocks'
// products.  S = 1: none are split.
struct BlkSplit {
  int full, S;
};
template <bool kWgrad>
__device__ __forceinline__ BlkSplit blk_split(const BlkSched& s, const BlkKArgs& p, int nM, int G) {
  const int total = s.total, rem = total % G;
  if (!p.part || rem == 0) return {total, 1};
  int local, units = (int)(p.K / 128);
  if (kWgrad) units = s.units[blk_expert<true>(s, p, nM, total - rem, local)];   // (the longest of them)
  int best = units, S = 1;
  for (int k = 1; k <= kPartRounds; ++k) {
    const int n = min(k * G / rem, units / (1 + p.part_cost));
    if (n < 2) continue;
    const int cost = k * ((units + n - 1) / n + p.part_cost);
    if (cost < best) { best = cost; S = n; }
  }
  return S < 2 ? BlkSplit{total, 1} : BlkSplit{total - rem, S};
}

// Row 0 of what tiles of expert e write: the product's one output, or the expert's weight gradient.
template <bool kWgrad>
__device__ __forceinline__ uint8_t* blk_out(const BlkKArgs& p, int e, int esz) {
  if (!kWgrad) return p.out;
  return p.tab ? reinterpret_cast<uint8_t*>(p.tab[e]) : p.out + (int64_t)e * p.N * p.K * esz;
}

struct BlkItem {
  int t, e, mt, nt;
  int part, u0, n;           // part of a split tile (-1: whole), first block of the contracted axis, blocks
  int row0, mrows;           // A rows: first (product: of all rows; weight gradient: of dw's N) and valid
};

constexpr int kBlkThreads = 512;
constexpr int kScaleBytes = 2048;                       // A scales of a stage, then B scales
constexpr int kBlkScOff = 2 * kStageBytes;
constexpr int kBlkEpOff = kBlkScOff + 2 * kScaleBytes;  // 2 KB per wave for the epilogue's full-line stores
constexpr int kBlkLds = kBlkEpOff + 8 * 2048;

typedef __bf16 bf16x2w __attribute__((ext_vector_type(2)));

// A fragment's 32 codes as the matrix instructions take them: as they are, or as bf16.  Group c of 8
// codes (c < 4) is the lane's share of one 16 x 16 x 32 product.
template <bool kWide>
struct Frag;
template <>
struct Frag<false> {
  i32x8 v;
  __device__ __forceinline__ void set(const i32x8& r) { v = r; }
  __device__ __forceinline__ void half(const i32x8&, int, int) {}
};
template <>
struct Frag<true> {
  bf16x8 v[4];
  __device__ __forceinline__ void set(const i32x8&) {}
  __device__ __forceinline__ void half(const i32x8& r, int c, int w) {   // 4 codes of group c
    {
      const bf16x2w lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r[2 * c + w], 1.0f, false);
      const bf16x2w hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r[2 * c + w], 1.0f, true);
      v[c][4 * w] = lo[0];
      v[c][4 * w + 1] = lo[1];
      v[c][4 * w + 2] = hi[0];
      v[c][4 * w + 3] = hi[1];
    }
  }
};
// One matrix instruction of the block's products of B fragment j and an A fragment: all of them, or
// (bf16) those of group c of the codes, c = 0 first.
__device__ __forceinline__ void blk_mma(const Frag<false>& b, const Frag<false>& a, f32x4v& t, int) {
  t = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.v, a.v, f32x4v{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ void blk_mma(const Frag<true>& b, const Frag<true>& a, f32x4v& t, int c) {
  t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.v[c], a.v[c], c == 0 ? f32x4v{0.f, 0.f, 0.f, 0.f} : t, 0, 0, 0);
}

// kWide (fp32 output): bf16 products.  kPartial: waves past a tile's last row or column skip its products.
template <bool kWgrad, bool kWide, bool kPartial>
__global__ __launch_bounds__(kBlkThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
void blk_gemm_kernel(const BlkKArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[kBlkLds];
  __shared__ BlkSched sched;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  constexpr int kTN = kWide ? 128 : 256;                // tile columns
  constexpr int kI = kWide ? 4 : 8;                     // 16-row fragments of a wave; its columns are 64
  constexpr int kAt = kWide ? 1 : 2;                    // the fragment whose products free the B rows' buffer
  constexpr int kQB = kTN / 64;                         // B loads per wave and stage
  const int wm = wave / (kTN / 64), wn = wave % (kTN / 64);
  const int64_t N = p.N, K = p.K;
  const int nM_w = (int)((N + kBM - 1) / kBM);          // weight gradient: tiles along dw's rows
  build_blk_sched<kWgrad>(sched, p, nM_w);
  const int tiles = __builtin_amdgcn_readfirstlane(sched.total);
  const int G = gridDim.x, per = G >> 3, xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
  BlkSplit sp = blk_split<kWgrad>(sched, p, nM_w, G);
  sp.full = __builtin_amdgcn_readfirstlane(sp.full);
  sp.S = __builtin_amdgcn_readfirstlane(sp.S);
  const int total = sp.full + (tiles - sp.full) * sp.S;   // items
  const uint32_t lda = kWgrad ? (uint32_t)p.rows : (uint32_t)K;   // bytes per operand row
  const int kU = (int)(K / 128);                        // product: blocks of K

  auto decode = [&](int round, BlkItem& it) {
    const int at = xcd * per + slot;
    it.t = round * G + (kWgrad && (round & 1) ? G - 1 - at : at);
    it.n = it.u0 = 0;
    if (it.t >= total) return;
    int tile = it.t;
    it.part = -1;
    if (it.t >= sp.full) {
      tile = sp.full + (it.t - sp.full) / sp.S;
      if (sp.S > 1) it.part = (it.t - sp.full) % sp.S;
    }
    int local;
    it.e = __builtin_amdgcn_readfirstlane(blk_expert<kWgrad>(sched, p, nM_w, tile, local));
    local = __builtin_amdgcn_readfirstlane(local);
    const int units = __builtin_amdgcn_readfirstlane(sched.units[it.e]);
    const int nM = kWgrad ? nM_w : (units + kBM - 1) / kBM;
    tile_coords(local, nM, p.nN, it.mt, it.nt);
    if (kWgrad) {
      it.row0 = it.mt * kBM;
      it.mrows = min(kBM, (int)N - it.row0);
      it.n = units;
    } else {
      it.row0 = __builtin_amdgcn_readfirstlane(sched.off[it.e]) + it.mt * kBM;
      it.mrows = min(kBM, units - it.mt * kBM);
      it.n = kU;
    }
    it.u0 = 0;
    if (it.part >= 0) {
      it.u0 = it.part * it.n / sp.S;
      it.n = (it.part + 1) * it.n / sp.S - it.u0;
    }
  };
  // Descriptors: the valid rows of the tile, so that everything past them reads zeros.  Scale rows are
  // block-major; a stage's are 256 consecutive words, of which those past the valid rows belong to
  // other rows and only ever multiply zeros.
  struct Desc { i32x4 va, vb, vs; int u0, s0; };  // vs: the scales this wave loads; u0, s0: first block within the rows, the scales
  auto descs = [&](const BlkItem& it, Desc& d) {
    d.u0 = d.s0 = it.u0;
    if (it.t >= total) {
      d.va = make_vsharp(p.a, 0); d.vb = d.va; d.vs = d.va;
      return;
    }
    const int n0 = it.nt * kTN;
    if (kWgrad) {
      const int first = __builtin_amdgcn_readfirstlane(sched.off[it.e]);
      const int nrows = min(kTN, (int)K - n0);
      const int64_t blocks = p.rows / 128;
      d.va = make_vsharp(p.a + (int64_t)it.row0 * lda, (uint32_t)it.mrows * lda);
      d.vb = make_vsharp(p.b + (int64_t)n0 * lda, (uint32_t)nrows * lda);
      const float* base = wave < 4 ? p.a_s : p.b_s;
      const int64_t ldsc = wave < 4 ? N : K, r0 = wave < 4 ? it.row0 : n0;
      d.vs = make_vsharp(base + (int64_t)first * ldsc + r0, (uint32_t)(((blocks - first) * ldsc - r0) * 4));
      d.u0 += first;
    } else {
      const int nrows = min(kTN, (int)N - n0);
      const int64_t nb = (N + 127) / 128;
      d.va = make_vsharp(p.a + (int64_t)it.row0 * K, (uint32_t)it.mrows * lda);
      d.vb = make_vsharp(p.b + ((int64_t)it.e * N + n0) * K, (uint32_t)nrows * lda);
      const int b0 = n0 / 128;
      const float* base = wave < 4 ? p.a_s + it.row0 : p.b_s + ((int64_t)it.e * nb + b0) * kU;
      d.vs = make_vsharp(base, (uint32_t)((wave < 4 ? (int64_t)kU * p.rows - it.row0 : (nb - b0) * kU) * 4));
    }
  };

  // Loads straight to LDS: 1 KB per load, the swz layout; load q of wave w fills row pairs
  // 4 (n w + q) + lane / 16 of an operand of which a wave loads n KB.  One 4-byte load per stage brings
  // the scales of A row 64 w + lane (waves 0-3) or B row 64 (w - 4) + lane (waves 4-7).
  auto row_off = [&](int j) {
    const uint32_t hs = (uint32_t)((j & 7) | ((j & 4) << 1));
    const uint32_t sl = (uint32_t)(lane & 15) ^ hs;
    return (2u * (uint32_t)j + (sl >> 3)) * lda + (sl & 7u) * 16u;
  };
  uint32_t vo[4], vob[kQB];
#pragma unroll
  for (int q = 0; q < 4; ++q) vo[q] = row_off((wave * 4 + q) * 4 + (lane >> 4));
#pragma unroll
  for (int q = 0; q < kQB; ++q) vob[q] = kQB == 4 ? vo[q] : row_off((wave * kQB + q) * 4 + (lane >> 4));
  const uint32_t sr = (uint32_t)((wave & 3) * 64 + lane);
  const uint32_t svo = (wave < 4 || kWgrad) ? sr * 4u : (sr >> 7) * (uint32_t)kU * 4u;
  const uint32_t lds0 = lds_addr(smem) + (uint32_t)wave * 4096u;
  const uint32_t ldsb = lds_addr(smem) + (uint32_t)kTileBytes + (uint32_t)(wave * kQB) * 1024u;
  const uint32_t lds_sc = lds_addr(smem + kBlkScOff) + (uint32_t)wave * 256u;
  // bytes from one stage's scales to the next
  const uint32_t s_step = (uint32_t)(wave < 4 ? (kWgrad ? N : p.rows) : (kWgrad ? K : 1)) * 4u;
  auto dma_a = [&](const Desc& d, int b, int kt, int q) {
    dma16(d.va, lds0 + (uint32_t)b * (uint32_t)kStageBytes + q * 1024u, vo[q], (uint32_t)(d.u0 + kt) * 128u);
  };
  auto dma_b = [&](const Desc& d, int b, int kt, int q) {
    dma16(d.vb, ldsb + (uint32_t)b * (uint32_t)kStageBytes + q * 1024u, vob[q], (uint32_t)(d.u0 + kt) * 128u);
  };
  auto dma_s = [&](const Desc& d, int b, int kt) {
    dma4(d.vs, lds_sc + (uint32_t)b * (uint32_t)kScaleBytes, svo, (uint32_t)(d.s0 + kt) * s_step);
  };

  // The lane's place in the fragments: row lane % 16 of a 16-row block, 16-byte chunks g and g + 4 of
  // its 128 bytes (g = lane / 16).  Which of a block's 128 values a lane holds does not matter as long
  // as A and B agree.  Rows of block i sit 2048 i bytes on, the second chunk at the address ^ 64.
  const int r16 = lane & 15, g = lane >> 4;
  const uint32_t fa = swz((uint32_t)(wm * 16 * kI + r16), (uint32_t)g);
  const uint32_t fb = (uint32_t)kTileBytes + swz((uint32_t)(wn * 64 + r16), (uint32_t)g);
  auto frag = [&](const uint8_t* st, uint32_t at, int i) {
    const u32x4 lo = *reinterpret_cast<const u32x4*>(st + at + i * 2048);
    const u32x4 hi = *reinterpret_cast<const u32x4*>(st + (at ^ 64u) + i * 2048);
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  };

  // Loads run two stages ahead of the products, so every item has at least two: those past its blocks
  // (an expert without tokens, a single block) load zeros.
  const i32x4 none = make_vsharp(p.a, 0);
  // part 0: the A rows and the scales; 1: the B rows.
  auto issue = [&](const Desc& d, int n, int kt, int b, int part) {
    const bool live = kt < n;
    Desc l;
    l.va = live ? d.va : none;
    l.vb = live ? d.vb : none;
    l.vs = live ? d.vs : none;
    l.u0 = d.u0;
    l.s0 = d.s0;
    if (part == 0) {
#pragma unroll
      for (int q = 0; q < 4; ++q) dma_a(l, b, kt, q);
      dma_s(l, b, kt);
    } else {
#pragma unroll
      for (int q = 0; q < kQB; ++q) dma_b(l, b, kt, q);
    }
  };
  // this wave's LDS reads returned, then every wave's
  auto barrier = [&]() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  BlkItem cur, nxt;
  Desc dc, dn;
  decode(0, cur);
  if (cur.t >= total) return;
  descs(cur, dc);
  issue(dc, cur.n, 0, 0, 0);
  issue(dc, cur.n, 0, 0, 1);
  wait_vmcnt<0>();
  barrier();
  issue(dc, cur.n, 1, 1, 1);
  issue(dc, cur.n, 1, 1, 0);

  // The stage being multiplied is in buffer `b`, its B fragments and first A fragment in registers.
  // Stage schedule: the products of A fragment i run in four quarters, behind each of which a quarter of
  // the sums of fragment i - 1 is added (and of the conversions to bf16 done): a wave's VALU work hides
  // behind its own matrix instructions only if it comes between them (8 instructions of 32 cycles with
  // 32 fused multiply-adds took 292 cycles so, 384 in groups of 4 and 16).  The B rows' buffer is free
  // once every wave holds its B fragments (the first barrier, after which the B rows of the stage after
  // next are loaded), the A rows' once the last two A fragments are in registers (the second, ahead of
  // the products of the last but one, after which the next stage has landed).  The next stage's B fragments
  // and first A fragment are read behind the last products, into the registers that these free: read
  // after them, with the second barrier a fragment later, the matrix cores waited some 600 cycles a stage
  // for LDS (16384 x 4096 x 14336: 871 -> 849 us, the earlier barrier 847 -> 826).
  int b = 0;
  i32x8 rb[4], ra;
  auto first_frags = [&](int buf) {
    const uint8_t* st = smem + buf * kStageBytes;
#pragma unroll
    for (int j = 0; j < 4; ++j) rb[j] = frag(st, fb, j);
    ra = frag(st, fa, 0);
  };
  first_frags(0);
  for (int round = 0; cur.t < total; ++round) {
    decode(round + 1, nxt);
    descs(nxt, dn);
    const int ns = max(cur.n, 2);
    // kPartial: a wave whose rows or columns are all past the tile's last only loads and keeps the barriers: its
    // SIMD's other wave, which holds rows of the tile's other half, has the matrix core to itself.
    const bool active =
        !kPartial || (wm * 16 * kI < cur.mrows && (int64_t)cur.nt * kTN + wn * 64 < (kWgrad ? K : N));
    f32x4v acc[kI][4];
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int s = 0; s < ns; ++s) {
      const uint8_t* st = smem + b * kStageBytes;
      const float* sc = reinterpret_cast<const float*>(smem + kBlkScOff + b * kScaleBytes);
      // the stage after next, of this item or the next one, into this stage's buffer
      auto issue_ahead = [&](int part) {
        const bool in = s + 2 < ns;
        Desc l;
        l.va = in ? dc.va : dn.va;
        l.vb = in ? dc.vb : dn.vb;
        l.vs = in ? dc.vs : dn.vs;
        l.u0 = in ? dc.u0 : dn.u0;
        l.s0 = in ? dc.s0 : dn.s0;
        issue(l, in ? cur.n : nxt.n, in ? s + 2 : s + 2 - ns, b, part);
      };
      if (!active) {
        barrier();
        issue_ahead(1);
        wait_vmcnt<kQB>();
        barrier();
        issue_ahead(0);
        first_frags(b ^ 1);
        b ^= 1;
        continue;
      }
      f32x4v t[2][4];
      float sa[2], sal[2] = {0.f, 0.f};
      i32x8 rl;
      f32x4v sbv[kWgrad ? 4 : 1];
      // sums of A fragment u: element r of its products with B fragment j
      auto add = [&](int u, int j, int r) {
        const float sv = u >= kI - 2 ? sal[u - kI + 2] : sa[u & 1];
        if constexpr (kWgrad) acc[u][j][r] += (sv * sbv[j][r]) * t[u & 1][j][r];
        else acc[u][j][r] += (sv * sbv[0][0]) * t[u & 1][j][r];
      };
      Frag<kWide> bf[4], af[2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bf[j].set(rb[j]);
        bf[j].half(rb[j], 0, 0);
        bf[j].half(rb[j], 0, 1);
      }
      af[0].set(ra);
#pragma unroll
      for (int c = 0; c < 8; ++c) af[0].half(ra, c / 2, c & 1);
#pragma unroll
      for (int i = 0; i < kI; ++i) {
        if (i == kAt) {                                 // every wave holds the stage's B fragments
          barrier();
          issue_ahead(1);
        }
        if (i == kI - 2) {
          wait_vmcnt<kQB>();                            // the next stage landed: all but the kQB loads above
          barrier();
        }
        constexpr int kM = kWide ? 16 : 4;              // matrix instructions of a fragment
#pragma unroll
        for (int n = 0; n < kM; ++n) {
          blk_mma(bf[n & 3], af[i & 1], t[i & 1][n & 3], n >> 2);
          __builtin_amdgcn_sched_barrier(0);
          if (n == 0) {
            // scales: all of the stage's are read ahead of the second barrier
            if (i + 2 < kI) {
              ra = frag(st, fa, i + 1);
              sa[i & 1] = sc[wm * 16 * kI + i * 16 + r16];
            }
            if (i + 3 == kI) {
              rl = frag(st, fa, kI - 1);
              sal[0] = sc[wm * 16 * kI + (kI - 2) * 16 + r16];
              sal[1] = sc[wm * 16 * kI + (kI - 1) * 16 + r16];
            }
            if (i == 0) {
              if constexpr (kWgrad) {
#pragma unroll
                for (int j = 0; j < 4; ++j) sbv[j] = *reinterpret_cast<const f32x4v*>(sc + 256 + wn * 64 + j * 16 + g * 4);
              } else {
                sbv[0][0] = sc[256 + wn * 64];
              }
            }
            if (i == kI - 2) issue_ahead(0);
          }
          if (i == kI - 1) {                            // the next stage's first fragments, where these were
            const uint8_t* const nst = smem + (b ^ 1) * kStageBytes;
            if (kWide ? (n & 3) == 0 : true) rb[kWide ? n >> 2 : n] = frag(nst, fb, kWide ? n >> 2 : n);
            if (n == (kWide ? 1 : 3)) ra = frag(nst, fa, 0);
          }
          if constexpr (kWide) {
            if (i > 0) add(i - 1, n >> 2, n & 3);
            if (i == 0 && n < 12) {                     // the B fragments' next group, one fragment at a time
              bf[n & 3].half(rb[n & 3], (n >> 2) + 1, 0);
              bf[n & 3].half(rb[n & 3], (n >> 2) + 1, 1);
            }
            if (i + 1 < kI && n >= 8) af[(i + 1) & 1].half(i + 2 == kI ? rl : ra, (n - 8) / 2, n & 1);   // (ra has arrived)
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (i > 0) add(i - 1, n, r);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        if (i + 1 < kI) af[(i + 1) & 1].set(i + 2 == kI ? rl : ra);
      }
#pragma unroll
      for (int n = 0; n < 16; ++n) add(kI - 1, n >> 2, n & 3);
      b ^= 1;
    }

    // ---- epilogue: lane l holds row 16 i + l % 16 of the wave's block at columns 16 j + 4 (l / 16) + r.
    // Through the wave's LDS slot 16 rows x 128 bytes at a time, so that stores move whole lines;
    // the slot's 16-byte chunks are placed at chunk ^ (row & 7).
    const int64_t ncols = kWgrad ? K : N;
    uint8_t* const out = blk_out<kWgrad>(p, cur.e, kWide ? 4 : 2);
    uint8_t* sl = smem + kBlkEpOff + wave * 2048;
    // (the lane is laundered, so that its addresses are not worked out ahead of the stages and kept)
    int el = lane;
    asm volatile("" : "+v"(el));
    const uint32_t row_r = (uint32_t)el >> 3, ch_r = (uint32_t)el & 7u;
    const uint32_t er = (uint32_t)el & 15u, eg = (uint32_t)el >> 4;
    // rows of `ld` bytes from the tile's first one, its columns from byte c0; chunks past the last
    // column and rows past the tile's last are outside the descriptor
    auto store = [&](const rsrc_t& ro, uint32_t ld, uint32_t c0, uint32_t i, uint32_t c) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t row = 8u * q + row_r;
        const u32x4 v = *reinterpret_cast<const u32x4*>(sl + row * 128u + ((ch_r ^ (row & 7u)) << 4));
        const uint32_t col = c0 + c + ch_r * 16u;
        const uint32_t at = col < ld ? ((uint32_t)(wm * 16 * kI) + i * 16u + row) * ld + col : 0xFFFFFFF0u;
        __builtin_amdgcn_raw_buffer_store_b128(v, ro, at, 0, 0);
      }
    };
    if (kWide || cur.part >= 0) {
      const bool whole = cur.part < 0;
      const uint32_t ld = whole ? (uint32_t)ncols * 4u : kTN * 4u;
      const int64_t o0 = (int64_t)cur.row0 * ncols;
      const rsrc_t ro = make_rsrc(whole ? reinterpret_cast<float*>(out) + o0
                                        : p.part + (int64_t)(cur.t - sp.full) * p.part_rows * kTN,
                                  (uint32_t)cur.mrows * ld);
      const uint32_t c0 = ((whole ? (uint32_t)cur.nt * kTN : 0u) + (uint32_t)wn * 64u) * 4u;
#pragma unroll
      for (int i = 0; i < kI; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int jj = 0; jj < 2; ++jj)
            *reinterpret_cast<f32x4v*>(sl + er * 128u + (((uint32_t)jj * 4u + eg) ^ (er & 7u)) * 16u) = acc[i][2 * h + jj];
          asm volatile("" ::: "memory");   // the LDS unit runs one wave's operations in order
          store(ro, ld, c0, (uint32_t)i, (uint32_t)h * 128u);
          asm volatile("" ::: "memory");
        }
      }
    } else {
      const uint32_t ld = (uint32_t)ncols * 2u;
      const int64_t o0 = (int64_t)cur.row0 * ncols;
      const rsrc_t ro = make_rsrc(reinterpret_cast<uint16_t*>(out) + o0, (uint32_t)cur.mrows * ld);
      const uint32_t c0 = (uint32_t)(cur.nt * kTN + wn * 64) * 2u;
#pragma unroll
      for (int i = 0; i < kI; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<u32x2*>(sl + er * 128u + (((uint32_t)j * 2u + (eg >> 1)) ^ (er & 7u)) * 16u + (eg & 1u) * 8u) =
              u32x2{pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3])};
        asm volatile("" ::: "memory");
        store(ro, ld, c0, (uint32_t)i, 0u);
        asm volatile("" ::: "memory");
      }
    }
    cur = nxt;
    dc = dn;
  }
  wait_vmcnt<0>();
}

// The split tiles' parts, added in their order: kJoinRows rows of a tile at a time, at most kJoinGrid
// workgroups going over them.  (2000 rows x 1024 x 8192: 44 us with 2048 workgroups, 46 with 1024, 50 with
// 512; with one for each 8 rows of every tile that could be split, 8160, building their schedules took 8 us.)
// Eight parts' loads are in flight at once.
constexpr int kJoinRows = 8, kJoinGrid = 2048;
template <bool kWgrad, bool kWide>
__global__ __launch_bounds__(256) void blk_join_kernel(const BlkKArgs p, int G) {
  __shared__ BlkSched sched;
  constexpr int kTN = kWide ? 128 : 256;
  const int nM_w = (int)((p.N + kBM - 1) / kBM);
  build_blk_sched<kWgrad>(sched, p, nM_w);
  const BlkSplit sp = blk_split<kWgrad>(sched, p, nM_w, G);
  if (sp.S < 2) return;
  const int64_t ncols = kWgrad ? p.K : p.N;
  constexpr int kT = kTN / 4;                           // threads of a row, 4 columns each
  const int c = (int)(threadIdx.x % kT) * 4, mr = (int)threadIdx.x / kT;
  const int64_t slot = (int64_t)p.part_rows * kTN;
  const int tiles = sched.total - sp.full;
  for (int item = blockIdx.x;; item += gridDim.x) {
    // rows 0..7 of all tiles first: a tile of few rows ends early
    const int m0 = item / tiles * kJoinRows, at = item - m0 / kJoinRows * tiles;
    if (m0 >= p.part_rows) return;
    int local, mt, nt;
    const int e = blk_expert<kWgrad>(sched, p, nM_w, sp.full + at, local), units = sched.units[e];
    tile_coords(local, kWgrad ? nM_w : (units + kBM - 1) / kBM, p.nN, mt, nt);
    const int row0 = kWgrad ? mt * kBM : sched.off[e] + mt * kBM;
    const int end = min(min(kBM, kWgrad ? (int)p.N - row0 : units - mt * kBM), m0 + kJoinRows);
    const int64_t col = (int64_t)nt * kTN + c;
    if (col >= ncols) continue;
    uint8_t* const out = blk_out<kWgrad>(p, e, kWide ? 4 : 2);
    const float* src = p.part + (int64_t)at * sp.S * slot + c;
    for (int m = m0 + mr; m < end; m += 256 / kT) {
      f32x4v a = {0.f, 0.f, 0.f, 0.f};
      const float* q = src + (int64_t)m * kTN;
      int i = 0;
      for (; i + 8 <= sp.S; i += 8, q += 8 * slot) {
        f32x4v v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = *reinterpret_cast<const f32x4v*>(q + u * slot);
#pragma unroll
        for (int u = 0; u < 8; ++u) a += v[u];
      }
      for (; i < sp.S; ++i, q += slot) a += *reinterpret_cast<const f32x4v*>(q);
      const int64_t o = (int64_t)(row0 + m) * ncols + col;
      if constexpr (kWide) *reinterpret_cast<f32x4v*>(reinterpret_cast<float*>(out) + o) = a;
      else *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(out) + o) = u32x2{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3])};
    }
  }
}

// 32 codes of a lane: 16 bytes, and 16 that lie 64 bytes further, half a block of 128.
__device__ __forceinline__ i32x8 load256(const rsrc_t& r, uint32_t off) {
  const i32x4 a = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
  const i32x4 b = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off + 64, 0, 0));
  return i32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// Products of few rows an expert, decoding's: their time is that of reading the weights, once each, so
// nothing is shared through LDS.  A tile is 16 rows of a by 16 kCols of w; the four waves of a workgroup
// take a quarter of K each and their sums meet in LDS, in the waves' order.  A lane loads its 32 codes of
// a fragment as the matrix instructions take them, 64 consecutive bytes of 16 rows at a time, kUnroll
// blocks ahead of their products.  The persistent workgroups (six of four waves fit a CU) take
// consecutive tiles at the same time, so the weights are read as they lie; with each XCD in a stretch of
// its own, and with a workgroup for each of min(R, E) N / (16 kCols) possible tiles, 8 rows of 8 experts
// (28672 x 4096) took 99 and 90 us, against 91; rows that crowd on one expert, 38 and 128.
// Measured: 8 rows, 28672 x 4096, 4.3 experts chosen: 91 us (5.6 TB/s of weights), 117 in the kernel above;
// one row, 4096 x 14336: 16, was 22.  fp32 outputs 83 us where bf16 took 82 (4 experts), and 17 (15).
constexpr int kFewRows = 16, kFewWaves = 4, kFewGrid = 6 * kGemmGrid;
template <bool kWide, int kCols, int kUnroll>
__global__ __launch_bounds__(64 * kFewWaves) void blk_few_kernel(const BlkKArgs p) {
  __shared__ BlkSched sched;
  __shared__ f32x4v sums[2][kCols][kFewWaves][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  build_blk_sched<false, kFewRows>(sched, p, 0);
  const int total = __builtin_amdgcn_readfirstlane(sched.total);
  const int R = (int)p.rows, N = (int)p.N, nb = (int)(p.K / 128), r = lane & 15;
  const int b0 = wave * nb / kFewWaves, b1 = (wave + 1) * nb / kFewWaves;
  const uint32_t K = (uint32_t)p.K, off0 = (uint32_t)r * K + (uint32_t)(lane >> 4) * 16;
  constexpr uint32_t kOut = 0xffffff00u;                // past every range: reads zeros
  const rsrc_t rs = make_rsrc(p.a_s, (uint32_t)((int64_t)nb * R * 4));
  int buf = 0;
  for (int t = blockIdx.x; t < total; t += gridDim.x, buf ^= 1) {
    const int e = __builtin_amdgcn_readfirstlane(blk_find(sched, p.E, t));
    const int units = __builtin_amdgcn_readfirstlane(sched.units[e]), groups = (units + kFewRows - 1) / kFewRows;
    const int local = t - __builtin_amdgcn_readfirstlane(sched.tile[e]), g = local % groups;
    const int n0 = local / groups * 16 * kCols, m0 = __builtin_amdgcn_readfirstlane(sched.off[e]) + g * kFewRows;
    const int rows = min(kFewRows, units - g * kFewRows);
    const rsrc_t ra = make_rsrc(p.a + (int64_t)m0 * K, (uint32_t)rows * K);
    const rsrc_t rw = make_rsrc(p.b + ((int64_t)e * N + n0) * K, (uint32_t)min(16 * kCols, N - n0) * K);
    const float* ws = p.b_s + ((int64_t)e * ((N + 127) / 128) + n0 / 128) * nb;
    f32x4v acc[kCols];
#pragma unroll
    for (int j = 0; j < kCols; ++j) acc[j] = f32x4v{0.f, 0.f, 0.f, 0.f};
    for (int b = b0; b < b1; b += kUnroll) {
      i32x8 x[kUnroll], w[kUnroll][kCols];
      float sc[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const bool in = b + u < b1;
        const uint32_t o = off0 + (uint32_t)(b + u) * 128;
        x[u] = load256(ra, in ? o : kOut);
#pragma unroll
        for (int j = 0; j < kCols; ++j) w[u][j] = load256(rw, in ? o + 16 * j * K : kOut);
        const uint32_t so = in ? (uint32_t)((b + u) * R + m0 + r) * 4 : kOut;
        sc[u] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, so, 0, 0)) * (in ? ws[b + u] : 0.f);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
          Frag<kWide> fx, fw;
          fx.set(x[u]);
          fw.set(w[u][j]);
          f32x4v v;
#pragma unroll
          for (int c = 0; c < (kWide ? 4 : 1); ++c) {
#pragma unroll
            for (int h = 0; h < 2; ++h) { fx.half(x[u], c, h); fw.half(w[u][j], c, h); }
            blk_mma(fw, fx, v, c);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[j][i] = fmaf(sc[u], v[i], acc[j][i]);
        }
      }
    }
    // one barrier a tile: a wave is past the reads of one tile's sums before it meets the next one's barrier
#pragma unroll
    for (int j = 0; j < kCols; ++j) sums[buf][j][wave][lane] = acc[j];
    __syncthreads();
    if (wave < kCols && r < rows && n0 + 16 * wave < N) {
      f32x4v a = sums[buf][wave][0][lane];
#pragma unroll
      for (int i = 1; i < kFewWaves; ++i) a += sums[buf][wave][i][lane];
      const int64_t o = (int64_t)(m0 + r) * N + n0 + 16 * wave + 4 * (lane >> 4);
      if constexpr (kWide) *reinterpret_cast<f32x4v*>(reinterpret_cast<float*>(p.out) + o) = a;
      else *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(p.out) + o) = u32x2{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3])};
    }
  }
}

// Whether a product of so many rows is one of few: 8 an expert on average (64 rows of 8 experts, 4096 x 14336:
// 91 us here, 94 in the kernel of 256-row tiles; 100 rows: 111 and 97), or 16 in all (one expert's 16
// rows, 4096 x 14336: 20 and 24), but 512 at most.  The host does not know how the rows spread, and each 16 of an
// expert's read its weights again.  Measured here and there, in us, with 2816 x 2048 weights of 256 experts, rows
// spread evenly, by Zipf's law (exponent 1.2), over 8 experts, on one:
//    512 rows  222 246 | 124 140 |  43 34 |  38 39
//   1024 rows  254 282 | 180 174 |  73 40 |  68 41
//   2048 rows  287 284 | 279 234 | 133 47 | 129 48
// (64 rows all on one of 8 experts, 28672 x 4096, which nothing here rules out: 80 and 36; evenly 169 and 218.)
constexpr int64_t kFewMost = 512;
bool few_rows(int64_t R, int E) { return R <= kFewRows || R <= std::min(8 * (int64_t)E, kFewMost); }

// A part writes its rows' fp32 sums and reads them back once: a full tile's 256 rows take about as long as
// 9 blocks' products, a few rows next to nothing.  rows: of a tile, on average.  (At 2000 rows x 1024 x 8192
// and for the gradients of 20000 tokens, 512 x 1024, parts of 18 blocks or more took 64 and 62 us, of 10
// 54 and 45; unsplit 105 and 89.)
int part_cost(int64_t rows) { return 1 + (int)(rows < kBM ? rows : kBM) / 32; }
// Whether tiles of `most` blocks are ever split.
bool may_split(int64_t most, int cost) { return most >= 2 * (1 + cost); }

}  // namespace

size_t block_gemm_part_bytes(bool wgrad, bool out_f32, int64_t rows, int64_t N, int64_t K, int E) {
  const int64_t prow = wgrad ? N : rows, most = (wgrad ? rows : K) / 128;
  if (!wgrad && few_rows(rows, E)) return 0;
  if (!may_split(most, part_cost(wgrad ? N : rows / E))) return 0;
  return (size_t)(kPartRounds * kGemmGrid) * (size_t)(prow < kBM ? prow : kBM) * (out_f32 ? 128 : 256) * sizeof(float);
}

hipError_t launch_block_gemm(const BlockGemm& g, hipStream_t st) {
  BlkKArgs k{};
  k.a = g.a;
  k.a_s = g.a_scales;
  k.b = g.b;
  k.b_s = g.b_scales;
  k.offsets = g.offsets;
  k.out = reinterpret_cast<uint8_t*>(g.out);
  k.tab = g.tab;
  k.rows = g.rows;
  k.N = g.N;
  k.K = g.K;
  k.E = g.E;
  if (!g.wgrad && few_rows(g.rows, g.E)) {
    // Two fragments of columns share one of a's, unless the tiles are then fewer than two a CU: with one, twice
    // as many tiles, and as many loads in flight (one row, 4096 x 14336: 16 and 25 us; 8 rows, 28672 x 4096: 97 and 91).
    const bool two = std::min<int64_t>(g.rows, g.E) * (g.N / 32) >= 2 * kGemmGrid;
    k.nN = (int)(two ? (g.N + 31) / 32 : g.N / 16);
    auto few = [&](auto wide) {
      constexpr bool kWd = decltype(wide)::value;
      if (two) blk_few_kernel<kWd, 2, 2><<<kFewGrid, 64 * kFewWaves, 0, st>>>(k);
      else blk_few_kernel<kWd, 1, 4><<<kFewGrid, 64 * kFewWaves, 0, st>>>(k);
    };
    if (g.out_f32) few(std::true_type{});
    else few(std::false_type{});
    return hipGetLastError();
  }
  const int tn = g.out_f32 ? 128 : 256;
  k.nN = (int)(((g.wgrad ? g.K : g.N) + tn - 1) / tn);
  const int64_t prow = g.wgrad ? g.N : g.rows, most = (g.wgrad ? g.rows : g.K) / 128;
  k.part_rows = (int)(prow < kBM ? prow : kBM);
  k.part_cost = part_cost(g.wgrad ? g.N : g.rows / g.E);
  const bool split = g.part && may_split(most, k.part_cost);
  const int join_grid = std::min(kJoinGrid, (kGemmGrid - 1) * ((k.part_rows + kJoinRows - 1) / kJoinRows));
  k.part = split ? g.part : nullptr;
  // Products whose experts have two tiles of rows or fewer, on average, are mostly edges: skipping the
  // empty halves takes 100 rows x 4096 x 14336 (8 experts) from 100 to 94 us, 500 x 2048 x 4096 (8) from 31 to
  // 28, and 500 rows of one or two experts nowhere (34-36); the branch costs the full tiles 1 % (16384 x 4096 x
  // 14336: 843 and 852 us).  The join runs wherever these sizes could be split: 4-5 us where nothing was.
  const bool partial = !g.wgrad && g.rows < 2 * kBM * (int64_t)g.E;
  auto launch = [&](auto wg, auto wide) {
    constexpr bool kWg = decltype(wg)::value, kWd = decltype(wide)::value;
    if (partial) blk_gemm_kernel<kWg, kWd, !kWg><<<kGemmGrid, kBlkThreads, 0, st>>>(k);
    else blk_gemm_kernel<kWg, kWd, false><<<kGemmGrid, kBlkThreads, 0, st>>>(k);
    if (split) blk_join_kernel<kWg, kWd><<<join_grid, 256, 0, st>>>(k, kGemmGrid);
  };
  if (g.wgrad && g.out_f32) launch(std::true_type{}, std::true_type{});
  else if (g.wgrad) launch(std::true_type{}, std::false_type{});
  else if (g.out_f32) launch(std::false_type{}, std::true_type{});
  else launch(std::false_type{}, std::false_type{});
  return hipGetLastError();
}

}  // namespace moe
