// Products of 16-bit and 8-bit integer operands, dense and grouped over experts of ragged sizes, and the
// 16-bit product's gradients.
#include "device_common.h"
#include "internal.h"

namespace megamoe {

typedef __bf16 bf16s;

__device__ __forceinline__ float g_silu(float g) {
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-g * 1.4426950408889634f));
}

template <int kDtype>
__device__ __forceinline__ float g_load(const void* p, int64_t i) {
  if constexpr (kDtype == kOperandI8) return (float)static_cast<const int8_t*>(p)[i];
  else if constexpr (kDtype == MEGAMOE_DTYPE_BF16) return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return (float)static_cast<const _Float16*>(p)[i];
}

__device__ __forceinline__ void g_store(void* p, int64_t i, int dtype, float v) {
  if (dtype == MEGAMOE_DTYPE_F32) static_cast<float*>(p)[i] = v;
  else if (dtype == MEGAMOE_DTYPE_BF16) static_cast<uint16_t*>(p)[i] = (uint16_t)f32_to_bf16_any(v);
  else static_cast<_Float16*>(p)[i] = (_Float16)v;
}
__device__ __forceinline__ float g_old(const void* p, int64_t i, int dtype) {
  return dtype == MEGAMOE_DTYPE_F32 ? static_cast<const float*>(p)[i]
         : dtype == MEGAMOE_DTYPE_BF16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i])
                                       : (float)static_cast<const _Float16*>(p)[i];
}

// One output element a thread; the reduced dimension from memory.
template <int kDtype, bool kL1>
__global__ __launch_bounds__(256) void g_rows_kernel(GroupedArgs p) {
  const int e = blockIdx.y;
  const int64_t cnt = p.counts ? p.counts[e] : p.M, first = p.padded_offsets ? p.padded_offsets[e] : 0;
  const int col = blockIdx.x * 16 + threadIdx.x % 16;
  if (col >= p.N) return;
  for (int64_t r = blockIdx.z * 16 + threadIdx.x / 16; r < cnt; r += 16 * gridDim.z) {
    const int64_t row = first + r, src = p.row_token ? p.row_token[row] : row;
    float z[2];
    for (int up = 0; up < (kL1 ? 2 : 1); ++up) {
      // weights [E, N or 2N, K], or [E, K, N] where they are read across
      const int64_t wrow = ((int64_t)e * (kL1 ? 2 : 1) + up) * p.N + col;
      float acc = 0.0f;
      int iacc = 0;
      for (int k = 0; k < p.K; ++k) {
        const float x = g_load<kDtype>(p.a, src * p.K + k);
        const float w = p.across ? g_load<kDtype>(p.w, ((int64_t)e * p.K + k) * p.N + col) : g_load<kDtype>(p.w, wrow * p.K + k);
        if constexpr (kDtype == kOperandI8) iacc += (int)x * (int)w;
        else acc += x * w;
      }
      if constexpr (kDtype == kOperandI8) acc = (float)iacc * p.w_scales[wrow] * p.a_scales[src];
      z[up] = acc;
    }
    g_store(p.out, row * p.N + col, p.out_dtype, kL1 ? g_silu(z[0]) * z[1] : z[0]);
  }
}

template <int kDtype>
__global__ __launch_bounds__(256) void g_weights_kernel(GroupedWgradArgs p) {
  const int e = blockIdx.z;
  const int64_t first = p.padded_offsets[e];
  const int k = blockIdx.x * 16 + threadIdx.x % 16, n = blockIdx.y * 16 + threadIdx.x / 16;
  if (k >= p.K || n >= p.N) return;
  float acc = 0.0f;
  for (int r = 0; r < p.counts[e]; ++r) {
    const int64_t row = first + r, src = p.row_token ? p.row_token[row] : row;
    acc += g_load<kDtype>(p.dy, row * p.N + n) * g_load<kDtype>(p.x, src * p.K + k);
  }
  const int64_t at = ((int64_t)e * p.N + n) * p.K + k;
  g_store(p.dw, at, p.dw_dtype, p.accumulate ? g_old(p.dw, at, p.dw_dtype) + acc : acc);
}

template <bool kL1>
static void launch_rows(const GroupedArgs& a, dim3 grid, hipStream_t s) {
  if (a.dtype == kOperandI8) hipLaunchKernelGGL((g_rows_kernel<kOperandI8, kL1>), grid, dim3(256), 0, s, a);
  else if (a.dtype == MEGAMOE_DTYPE_BF16) hipLaunchKernelGGL((g_rows_kernel<MEGAMOE_DTYPE_BF16, kL1>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((g_rows_kernel<MEGAMOE_DTYPE_F16, kL1>), grid, dim3(256), 0, s, a);
}

hipError_t launch_grouped(const GroupedArgs& a, bool l1, int64_t max_rows, hipStream_t stream) {
  (void)max_rows;
  const dim3 grid((a.N + 15) / 16, a.E, 64);
  if (l1) launch_rows<true>(a, grid, stream);
  else launch_rows<false>(a, grid, stream);
  return hipGetLastError();
}

hipError_t launch_grouped_wgrad(const GroupedWgradArgs& a, hipStream_t stream) {
  const dim3 grid((a.K + 15) / 16, (a.N + 15) / 16, a.E);
  if (a.dtype == MEGAMOE_DTYPE_BF16) hipLaunchKernelGGL((g_weights_kernel<MEGAMOE_DTYPE_BF16>), grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((g_weights_kernel<MEGAMOE_DTYPE_F16>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace megamoe
