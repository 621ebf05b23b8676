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
#include "device_common.h"
#include "internal.h"

namespace megamoe {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kMxGemmThreads = 256;

__device__ __forceinline__ f32x4 mx_mfma16(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
  const i32x8 av{(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv{(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

__device__ __forceinline__ float mx_silu(float g) {
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-g * 1.4426950408889634f));
}

// Rows of expert e and their first row; without tables there is one group of all p.M rows.
__device__ __forceinline__ int mx_count(const MxGemmArgs& p, int e) { return p.counts ? p.counts[e] : (int)p.M; }

template <bool kL1>
__global__ __launch_bounds__(kMxGemmThreads) void mx_gemm_kernel(MxGemmArgs p) {
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

hipError_t launch_mx_gemm(const MxGemmArgs& a, bool l1, hipStream_t stream) {
  const dim3 grid(2048), block(kMxGemmThreads);
  if (l1) hipLaunchKernelGGL(mx_gemm_kernel<true>, grid, block, 0, stream, a);
  else hipLaunchKernelGGL(mx_gemm_kernel<false>, grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace megamoe
