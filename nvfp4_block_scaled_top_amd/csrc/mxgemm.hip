// MXFP4 x MXFP4 products: dense, and grouped over experts (gate+up with SiLU(gate)*up, and down).
//
//   out[m, n] = sum over 32-element blocks b of 2^(ea[m,b] + ew[n,b]) * sum_{k in b} e2m1(a) * e2m1(w)
//
// gfx950 multiplies both operands' codes and scales in the matrix core: lane l of
// v_mfma_scale_f32_16x16x128_f8f6f4 holds the 32 codes (16 bytes) of block l / 16 of row l % 16 and
// that block's scale byte, so an MXFP4 block is one lane's operand and nothing is decoded.
// Products and sums are exact up to the fp32 accumulation.
//
// The weights are the MFMA's A operand and the token rows its B operand, so a lane ends with four
// consecutive output columns of one token.  Gate and up rows of an expert are interleaved two by two
// within a 16-row block: a lane then holds gate and up of the same two h columns.
#include <atomic>

#include "device_common.h"
#include "internal.h"
#include "lds_dma.h"

namespace megamoe {

constexpr int kMxDevices = 64;

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kMxGemmThreads = 256;

__device__ __forceinline__ f32x4 mx_mfma16(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
  const i32x8 av{(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv{(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

__device__ __forceinline__ f32x16 mx_mfma32_lo(u32x4 a, u32x4 b, f32x16 c, uint32_t sa, uint32_t sb) {
  const i32x8 av{(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv{(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0, (int)sb);
}
__device__ __forceinline__ f32x16 mx_mfma32_hi(u32x4 a, u32x4 b, f32x16 c, uint32_t sa, uint32_t sb) {
  const i32x8 av{(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv{(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, 1, (int)sa, 1, (int)sb);
}

__device__ __forceinline__ float mx_silu(float g) {
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-g * 1.4426950408889634f));
}

// Rows of expert e and their first row; without tables there is one group of all p.M rows.
__device__ __forceinline__ int mx_count(const MxGemmArgs& p, int e) { return p.counts ? p.counts[e] : (int)p.M; }

// ============================================================================================
// Experts (or a dense call) of at most kMxSmallRows rows.
// ============================================================================================
constexpr int kMxSmallRows = 16;

template <bool kL1>
__global__ __launch_bounds__(kMxGemmThreads) void mx_small_kernel(MxGemmArgs p) {
  const int lane = lane_id(), r = lane & 15, g = lane >> 4;
  const int K = p.K, Kh = K / 2, Ks = K / 32;
  const int unit = kL1 ? 8 : 16;  // output columns of a 16-row weight block
  const int nt = (p.N + unit - 1) / unit;
  const int wave = (int)(blockIdx.x * (kMxGemmThreads / kWave)) + (int)(threadIdx.x / kWave);
  const int nwaves = (int)gridDim.x * (kMxGemmThreads / kWave);
  const int64_t Nw = kL1 ? 2 * (int64_t)p.N : p.N;
  int64_t t0 = 0;  // tiles of the experts before e
  for (int e = 0; e < p.E; ++e) {
    const int cnt = mx_count(p, e);
    if (cnt > kMxSmallRows && !p.cover_large) continue;  // the tile kernel's
    const int64_t tiles = (int64_t)((cnt + 15) / 16) * nt;
    int64_t t = (wave - t0 % nwaves + nwaves) % nwaves;  // first tile of e that this wave takes
    for (; t < tiles; t += nwaves) {
      const int mt = (int)(t / nt), j = (int)(t % nt);
      const int left = cnt - 16 * mt;
      const int64_t row0 = (p.padded_offsets ? p.padded_offsets[e] : 0) + 16 * (int64_t)mt;
      // A lane outside the tile reads a valid row of it instead; what it feeds is not stored.
      const int64_t tr = row0 + (r < left ? r : 0);
      const int64_t ar = p.row_token ? p.row_token[tr] : tr;
      int col = j * unit + (kL1 ? (r >> 2) * 2 + (r & 1) : r);  // weight row of lane row r
      if (col >= p.N) col = p.N - 1;
      const int64_t wr = e * Nw + (kL1 && (r & 2) ? p.N + col : col);
      const uint8_t* a = p.a_codes + ar * Kh + 16 * g;
      const uint8_t* as = p.a_scales + ar * Ks + g;
      const uint8_t* w = p.w_codes + wr * Kh + 16 * g;
      const uint8_t* ws = p.w_scales + wr * Ks + g;
      f32x4 c{0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < K / 128; ++k)
        c = mx_mfma16(*reinterpret_cast<const u32x4*>(w + 64 * k), *reinterpret_cast<const u32x4*>(a + 64 * k), c,
                      ws[4 * k], as[4 * k]);
      // lane: token row r of the tile, weight rows 4g .. 4g+3
      if (r < left) {
        uint16_t* out = static_cast<uint16_t*>(p.out) + (row0 + r) * (int64_t)p.N;
        if constexpr (kL1) {
          for (int i = 0; i < 2; ++i)
            if (j * 8 + 2 * g + i < p.N) out[j * 8 + 2 * g + i] = (uint16_t)f32_to_bf16_any(mx_silu(c[i]) * c[i + 2]);
        } else {
          for (int i = 0; i < 4; ++i)
            if (j * 16 + 4 * g + i < p.N) out[j * 16 + 4 * g + i] = (uint16_t)f32_to_bf16_any(c[i]);
        }
      }
    }
    t0 += tiles;
  }
}

// ============================================================================================
// Experts of more rows: 256 weight rows x BM token rows a tile, BM = 256, or 128 or 64 for an
// expert's last rows when they fit; one persistent workgroup of 8 waves a CU.
//
// Stages of 128 K elements go from global memory straight into an LDS ring (no registers); a wave
// waits for its own loads (vmcnt), one barrier makes everyone's visible, and the stage three ahead
// is requested right after it, into the slot that the barrier has just freed.  A stage holds, per
// operand, 64 code bytes a row (16-byte chunk c of row R in slot c ^ mx_swz(R), so that the 16-byte
// reads of consecutive rows hit distinct banks) and 4 scale bytes a row.
//
// The 32x32x64 form is used: it sustains 9.2 PFLOP/s from registers (6.6 on random data, where the
// chip lowers its clock), the 16x16x128 form 6.9 (5.5).  Lane (r, h) of a 32-row fragment takes blocks
// 2h and 2h + 1 of its row, one a step, so its two scale bytes are neighbours: one 2-byte read, and
// the instruction picks the byte.  Both operands use the same order, so every block is met once.
//
// A wave computes 64 token rows x 32 * WB weight rows (WB = 4, 2, 1 for BM = 256, 128, 64).  Gate+up:
// the first half of a wave's weight rows are gate rows, the second half the up rows of the same h
// columns, so both meet in one lane.
// ============================================================================================
constexpr int kMxWaves = 8, kMxThreads = kMxWaves * kWave;
constexpr int kMxGrid = 256;   // one workgroup a CU
constexpr int kMxBn = 256;     // weight rows of a tile
constexpr int kMxBm = 256;     // token rows of a full tile
constexpr int kMxSlots = 4, kMxAhead = kMxSlots - 1;
constexpr int kMxBand = 8;     // m-tiles walked together, for L2 reuse of the weights

__device__ __forceinline__ constexpr int mx_swz(int R) { return ((R >> 1) ^ (R >> 3)) & 3; }

template <int BM>
struct MxShape {
  static constexpr int kWM = BM / 64, kWN = kMxWaves / kWM;
  static constexpr int kWB = kMxBn / kWN / 32;                     // 32-row weight blocks a wave
  static constexpr int kACodeDma = BM >= 128 ? BM / 128 : 1;       // 16-row loads a wave (BM = 64: two waves load the same)
  static constexpr int kDma = kACodeDma + 2 + 1;                   // loads a wave and stage
  static constexpr int kACodes = kMxBn * 64, kWScales = kACodes + BM * 64;
  static constexpr int kAScales = kWScales + kMxBn * 4;
  static constexpr int kStage = kAScales + BM * 4;
};
constexpr int kMxRing = kMxSlots * MxShape<kMxBm>::kStage;
static_assert(kMxRing + 4 * (MEGAMOE_MAX_EXPERTS + 1) <= 160 * 1024, "the ring and the tables fit");

// Waits for this wave's loads but those of the last `after` stages, and for its LDS reads.
template <class S, int K>
__device__ __forceinline__ void mx_wait_stages(int after) {
  constexpr int n = K * S::kDma;
  static_assert(n < 64, "vmcnt range");
  if constexpr (K > 0) {
    if (after < K) {
      mx_wait_stages<S, K - 1>(after);
      return;
    }
  }
  __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (0x7 << 4));  // vmcnt(n) lgkmcnt(0)
}

// Workgroup barrier that no LDS access is moved across.  Vector memory loads stay in flight.
__device__ __forceinline__ void mx_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <bool kL1, int BM>
__device__ __forceinline__ void mx_tile(const MxGemmArgs& p, uint8_t* smem, int e, int64_t row0, int left, int nt) {
  using S = MxShape<BM>;
  constexpr int WB = S::kWB;
  const int K = p.K, nks = K / 128;
  const int64_t Kh = K / 2, Ks = K / 32;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
  const int wm = wave / S::kWN, wn = wave % S::kWN;
  const int r = lane & 31, h = lane >> 5;

  // Rows past the tile's end read its first row, columns past the last one the last column's weights:
  // what they feed is not stored.
  auto a_row = [&](int R) -> int64_t {
    const int64_t t = row0 + (R < left ? R : 0);
    return p.row_token ? p.row_token[t] : t;
  };
  auto w_row = [&](int R) -> int64_t {
    if constexpr (kL1) {
      const int w = R / (32 * WB), x = R % (32 * WB);
      int c = nt * (kMxBn / 2) + w * 16 * WB + x % (16 * WB);
      c = c < p.N ? c : p.N - 1;
      return (int64_t)e * 2 * p.N + (x < 16 * WB ? c : p.N + c);
    } else {
      const int c = nt * kMxBn + R;
      return (int64_t)e * p.N + (c < p.N ? c : p.N - 1);
    }
  };
  // Code loads cover 16 rows: lane l brings chunk (l % 4) ^ mx_swz(row) of row l / 4.
  const uint8_t* a_src[S::kACodeDma];
  int a_lds[S::kACodeDma];
#pragma unroll
  for (int j = 0; j < S::kACodeDma; ++j) {
    const int R0 = (16 * S::kACodeDma * wave + 16 * j) % BM, R = R0 + lane / 4;
    a_src[j] = p.a_codes + a_row(R) * Kh + 16 * ((lane & 3) ^ mx_swz(R));
    a_lds[j] = S::kACodes + R0 * 64;
  }
  const uint8_t* w_src[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int R = 32 * wave + 16 * j + lane / 4;
    w_src[j] = p.w_codes + w_row(R) * Kh + 16 * ((lane & 3) ^ mx_swz(R));
  }
  // Scale loads cover 64 rows: waves 0-3 the weights', waves 4-7 the tokens' (repeated when BM < 256).
  const int s_row0 = wave < 4 ? 64 * wave : 64 * ((wave - 4) % (BM / 64));
  const uint8_t* s_src = wave < 4 ? p.w_scales + w_row(s_row0 + lane) * Ks : p.a_scales + a_row(s_row0 + lane) * Ks;
  const int s_lds = (wave < 4 ? S::kWScales : S::kAScales) + 4 * s_row0;

  auto issue = [&](int ks) {
    const uint32_t base = lds_addr(smem + (ks % kMxSlots) * S::kStage);
    const int off = ks * 64;
#pragma unroll
    for (int j = 0; j < 2; ++j) dma16(w_src[j] + off, base + (32 * wave + 16 * j) * 64);
#pragma unroll
    for (int j = 0; j < S::kACodeDma; ++j) dma16(a_src[j] + off, base + a_lds[j]);
    dma4(s_src + 4 * ks, base + s_lds);
  };

  f32x16 acc[2][WB];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int f = 0; f < WB; ++f)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][f][q] = 0.f;

  const int swz = mx_swz(r);  // of rows 32 i + r too
  for (int ks = 0; ks < kMxAhead && ks < nks; ++ks) issue(ks);
  for (int ks = 0; ks < nks; ++ks) {
    const int after = nks - 1 - ks;
    mx_wait_stages<S, kMxAhead - 1>(after < kMxAhead - 1 ? after : kMxAhead - 1);
    mx_barrier();
    if (ks + kMxAhead < nks) issue(ks + kMxAhead);
    const uint8_t* st = smem + (ks % kMxSlots) * S::kStage;
    u32x4 w[WB][2], a[2][2];
    uint32_t wsc[WB], asc[2];
#pragma unroll
    for (int f = 0; f < WB; ++f) {
      const int R = (wn * WB + f) * 32 + r;
#pragma unroll
      for (int s = 0; s < 2; ++s) w[f][s] = *reinterpret_cast<const u32x4*>(st + R * 64 + 16 * ((2 * h + s) ^ swz));
      wsc[f] = *reinterpret_cast<const uint16_t*>(st + S::kWScales + R * 4 + 2 * h);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int R = wm * 64 + 32 * i + r;
#pragma unroll
      for (int s = 0; s < 2; ++s)
        a[i][s] = *reinterpret_cast<const u32x4*>(st + S::kACodes + R * 64 + 16 * ((2 * h + s) ^ swz));
      asc[i] = *reinterpret_cast<const uint16_t*>(st + S::kAScales + R * 4 + 2 * h);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int f = 0; f < WB; ++f) acc[i][f] = mx_mfma32_lo(w[f][0], a[i][0], acc[i][f], wsc[f], asc[i]);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int f = 0; f < WB; ++f) acc[i][f] = mx_mfma32_hi(w[f][1], a[i][1], acc[i][f], wsc[f], asc[i]);
  }

  // Accumulator q of block (i, f): weight row 32 f + 8 (q / 4) + 4 h + q % 4 of the wave, token row 32 i + r.
  uint16_t* out = static_cast<uint16_t*>(p.out);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int R = wm * 64 + 32 * i + r;
    if (R >= left) continue;
    uint16_t* o = out + (row0 + R) * (int64_t)p.N;
    if constexpr (kL1) {
      const int c0 = nt * (kMxBn / 2) + wn * 16 * WB;
#pragma unroll
      for (int f = 0; f < (WB + 1) / 2; ++f)
#pragma unroll
        for (int q4 = 0; q4 < (WB == 1 ? 2 : 4); ++q4) {
          const int c = c0 + 32 * f + 8 * q4 + 4 * h;
          if (c >= p.N) continue;
          uint32_t b[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float gt = acc[i][f][4 * q4 + j];
            const float up = WB == 1 ? acc[i][0][(4 * q4 + j + 8) & 15] : acc[i][(f + WB / 2) % WB][4 * q4 + j];
            b[j] = f32_to_bf16_any(mx_silu(gt) * up);
          }
          *reinterpret_cast<u32x2*>(o + c) = u32x2{b[0] | b[1] << 16, b[2] | b[3] << 16};
        }
    } else {
#pragma unroll
      for (int f = 0; f < WB; ++f)
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          const int c = nt * kMxBn + (wn * WB + f) * 32 + 8 * q4 + 4 * h;
          if (c >= p.N) continue;
          uint32_t b[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) b[j] = f32_to_bf16_any(acc[i][f][4 * q4 + j]);
          *reinterpret_cast<u32x2*>(o + c) = u32x2{b[0] | b[1] << 16, b[2] | b[3] << 16};
        }
    }
  }
  __syncthreads();  // every wave is done with the ring before the next tile's loads refill it
}

template <bool kL1>
__global__ __launch_bounds__(kMxThreads, 1) void mx_tile_kernel(MxGemmArgs p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t s_mx[];  // ring, then the m-tile prefix [E + 1]
  int* const pref = reinterpret_cast<int*>(s_mx + kMxRing);
  const int E = p.E;
  if (threadIdx.x < kWave) {  // exclusive prefix of the experts' m-tiles
    const int lane = lane_id();
    int carry = 0;
    for (int c = 0; c < E; c += kWave) {
      const int cnt = c + lane < E ? mx_count(p, c + lane) : 0;
      int incl = cnt > kMxSmallRows ? (cnt + kMxBm - 1) / kMxBm : 0;
      const int own = incl;
#pragma unroll
      for (int o = 1; o < kWave; o <<= 1) {
        const int t = __shfl_up(incl, o, kWave);
        if (lane >= o) incl += t;
      }
      if (c + lane < E) pref[c + lane] = carry + incl - own;
      carry += __shfl(incl, kWave - 1, kWave);
    }
    if (lane == 0) pref[E] = carry;
  }
  __syncthreads();
  const int ntn = (p.N + (kL1 ? kMxBn / 2 : kMxBn) - 1) / (kL1 ? kMxBn / 2 : kMxBn);
  const int64_t total = (int64_t)pref[E] * ntn;
  // Workgroup b runs on XCD b % 8: the 32 workgroups of an XCD take 32 tiles in a row, which share
  // rows and weights in its L2.
  for (int64_t t = (blockIdx.x % 8) * (kMxGrid / 8) + blockIdx.x / 8; t < total; t += kMxGrid) {
    int lo = 0, hi = E;  // pref[lo] * ntn <= t < pref[hi] * ntn
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((int64_t)pref[mid] * ntn <= t) lo = mid; else hi = mid;
    }
    const int e = lo, mts = pref[e + 1] - pref[e];
    const int64_t local = t - (int64_t)pref[e] * ntn;
    const int band = (int)(local / ((int64_t)kMxBand * ntn)), in = (int)(local % ((int64_t)kMxBand * ntn));
    const int width = min(kMxBand, mts - band * kMxBand);
    const int nt = in / width, mt = band * kMxBand + in % width;
    const int left = mx_count(p, e) - mt * kMxBm;
    const int64_t row0 = (p.padded_offsets ? p.padded_offsets[e] : 0) + (int64_t)mt * kMxBm;
    if (left > 128) mx_tile<kL1, 256>(p, s_mx, e, row0, left, nt);
    else if (left > 64) mx_tile<kL1, 128>(p, s_mx, e, row0, left, nt);
    else mx_tile<kL1, 64>(p, s_mx, e, row0, left, nt);
  }
}

template <bool kL1>
static hipError_t launch_mx(const MxGemmArgs& a, bool small, bool large, hipStream_t stream) {
  if (small) {
    hipLaunchKernelGGL(mx_small_kernel<kL1>, dim3(2048), dim3(kMxGemmThreads), 0, stream, a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  if (large) {
    const size_t lds = kMxRing + sizeof(int) * ((size_t)a.E + 1);
    static std::atomic<bool> set[2][kMxDevices];  // the kernel's dynamic LDS limit, raised once a device
    int dev = 0;
    hipError_t err = hipGetDevice(&dev);
    if (err != hipSuccess) return err;
    if (dev >= kMxDevices || !set[kL1][dev].load(std::memory_order_acquire)) {
      err = hipFuncSetAttribute(reinterpret_cast<const void*>(mx_tile_kernel<kL1>),
                                hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
      if (err != hipSuccess) return err;
      if (dev < kMxDevices) set[kL1][dev].store(true, std::memory_order_release);
    }
    hipLaunchKernelGGL(mx_tile_kernel<kL1>, dim3(kMxGrid), dim3(kMxThreads), lds, stream, a);
    return hipGetLastError();
  }
  return hipSuccess;
}

hipError_t launch_mx_gemm(const MxGemmArgs& a0, bool l1, int64_t max_rows, hipStream_t stream) {
  MxGemmArgs a = a0;
  // A dense call knows its rows.  A grouped one launches both kernels unless the caller's bound says
  // that no expert has more than the small kernel's rows; it then covers every expert, should the
  // bound be wrong.
  const bool small = a.counts != nullptr || a.M <= kMxSmallRows;
  const bool large = a.counts != nullptr ? !(max_rows > 0 && max_rows <= kMxSmallRows) : a.M > kMxSmallRows;
  a.cover_large = !large;
  return l1 ? launch_mx<true>(a, small, large, stream) : launch_mx<false>(a, small, large, stream);
}

}  // namespace megamoe
