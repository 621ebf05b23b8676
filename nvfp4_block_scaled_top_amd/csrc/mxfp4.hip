// MXFP4 quantizer and decoder (OCP microscaling: E2M1 elements, one E8M0 scale per 32).
//
// The scale of a block is 2^e with e = floor(log2(amax)) - 2 (2 = the exponent of E2M1's largest
// power of two, 4), at least -127; an element's code is the E2M1 point nearest to x / 2^e, ties to
// the even code, saturating at +-6, with x's sign.  floor(log2(amax)) is the exponent field of amax
// and v_cvt_scalef32_pk_fp4_* divides by the power of two and rounds exactly so (every bf16 input
// and scales at both ends of the range compared equal), so results are bit-exact with that
// definition.  A block that holds an infinity or a NaN gets the NaN scale 0xFF and zero codes: every
// product that reads it is NaN.
//
// Memory-bound: four lanes a block, 16 bytes of bf16 a lane, the block's amax over the quad.
#include "device_common.h"
#include "internal.h"

namespace megamoe {

typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));

constexpr int kMxThreads = 256;

__device__ __forceinline__ uint32_t quad_max_u32(uint32_t v) {
  uint32_t o = __shfl_xor(v, 1, kWave);
  v = v > o ? v : o;
  o = __shfl_xor(v, 2, kWave);
  return v > o ? v : o;
}

__device__ __forceinline__ bf16x2v as_bf16x2(uint32_t w) {
  bf16x2v v;
  __builtin_memcpy(&v, &w, 4);
  return v;
}

// Eight elements of a lane: their code word and the block's scale byte.
struct Mx8 {
  uint32_t codes, scale;
};

__device__ __forceinline__ Mx8 mx_quant8(u32x4 v) {  // bf16, the lower element in the low half
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = v[j] & 0x7FFFu, hi = (v[j] >> 16) & 0x7FFFu;
    m = m > lo ? m : lo;
    m = m > hi ? m : hi;
  }
  m = quad_max_u32(m);
  const uint32_t ex = m >> 7;
  if (ex == 0xFFu) return {0u, 0xFFu};
  const uint32_t sc = ex > 2u ? ex - 2u : 0u;
  const float s = __uint_as_float(sc << 23);
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(0u, as_bf16x2(v[0]), s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(v[1]), s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(v[2]), s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(v[3]), s, 3);
  return {w, sc};
}

__device__ __forceinline__ Mx8 mx_quant8(u32x4 a, u32x4 b) {  // float32
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = a[j] & 0x7FFFFFFFu, hi = b[j] & 0x7FFFFFFFu;
    m = m > lo ? m : lo;
    m = m > hi ? m : hi;
  }
  m = quad_max_u32(m);
  const uint32_t ex = m >> 23;
  if (ex == 0xFFu) return {0u, 0xFFu};
  const uint32_t sc = ex > 2u ? ex - 2u : 0u;
  const float s = __uint_as_float(sc << 23);
  const auto f = [](uint32_t x) { return __uint_as_float(x); };
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, f(a[0]), f(a[1]), s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(a[2]), f(a[3]), s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(b[0]), f(b[1]), s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f(b[2]), f(b[3]), s, 3);
  return {w, sc};
}

// n8 = elements / 8; rows with row_valid[r] < 0 get zero codes and scales and are not read.
template <bool kF32>
__global__ __launch_bounds__(kMxThreads) void mx_quant_kernel(const void* __restrict__ x, int64_t n8, int64_t cols8,
                                                              const int32_t* __restrict__ row_valid,
                                                              uint32_t* __restrict__ codes,
                                                              uint8_t* __restrict__ scales) {
  const int64_t step = (int64_t)gridDim.x * kMxThreads;
  // the four lanes of a block hold the same block in every iteration (n8 and step are multiples of 4)
  for (int64_t i = (int64_t)blockIdx.x * kMxThreads + threadIdx.x; i < n8; i += step) {
    Mx8 q{0u, 0u};
    if (row_valid == nullptr || row_valid[i / cols8] >= 0) {
      const u32x4* src = static_cast<const u32x4*>(x) + (kF32 ? 2 * i : i);
      if constexpr (kF32) q = mx_quant8(src[0], src[1]);
      else q = mx_quant8(src[0]);
    }
    codes[i] = q.codes;
    if ((i & 3) == 0) scales[i >> 2] = (uint8_t)q.scale;
  }
}

static unsigned mx_grid(int64_t n8) {
  const int64_t g = (n8 + kMxThreads - 1) / kMxThreads;
  return (unsigned)(g > 8192 ? 8192 : g);
}

hipError_t launch_mx_quant(const void* x, int dtype, int64_t rows, int64_t cols, const int32_t* row_valid,
                           uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  const int64_t n8 = rows * (cols / 8);
  if (n8 == 0) return hipSuccess;
  uint32_t* c = reinterpret_cast<uint32_t*>(codes);
  if (dtype == MEGAMOE_DTYPE_F32)
    hipLaunchKernelGGL(mx_quant_kernel<true>, dim3(mx_grid(n8)), dim3(kMxThreads), 0, stream, x, n8, cols / 8,
                       row_valid, c, scales);
  else
    hipLaunchKernelGGL(mx_quant_kernel<false>, dim3(mx_grid(n8)), dim3(kMxThreads), 0, stream, x, n8, cols / 8,
                       row_valid, c, scales);
  return hipGetLastError();
}

// Decoder: one lane per code word (eight elements, 16 bytes of bf16).  e2m1 * 2^(scale - 127) has two
// significant bits and is exact in bf16, the subnormal products of scale 0 included; above the range
// (6 * 2^126 and up) it is the infinity of bf16.
__device__ __forceinline__ uint32_t mx_value_bits(uint32_t code, uint32_t scale) {
  if (scale == 0xFFu) return 0x7FC0u;
  const uint32_t mag = code & 7u, sign = (code & 8u) << 12;
  if (mag == 0) return sign;
  // value = (1 + man / 2) * 2^(ex): magnitude 1 is 2^-1, magnitude m >= 2 has ex = m / 2 - 1
  int ex = mag == 1 ? -1 : (int)(mag >> 1) - 1;
  const uint32_t man = mag == 1 ? 0u : mag & 1u;
  ex += (int)scale;  // biased exponent
  if (ex >= 255) return sign | 0x7F80u;
  if (ex >= 1) return sign | ((uint32_t)ex << 7) | (man << 6);
  return sign | ((0x80u | man << 6) >> (1 - ex));  // subnormal: ex = 0 or -1, the shifted-out bits are zero
}

__global__ __launch_bounds__(kMxThreads) void mx_dequant_kernel(const uint32_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, int64_t n8,
                                                                u32x4* __restrict__ out) {
  const int64_t step = (int64_t)gridDim.x * kMxThreads;
  for (int64_t i = (int64_t)blockIdx.x * kMxThreads + threadIdx.x; i < n8; i += step) {
    const uint32_t w = codes[i], sc = scales[i >> 2];
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = mx_value_bits((w >> (8 * j)) & 15u, sc) | (mx_value_bits((w >> (8 * j + 4)) & 15u, sc) << 16);
    out[i] = o;
  }
}

hipError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out,
                             hipStream_t stream) {
  const int64_t n8 = rows * (cols / 8);
  if (n8 == 0) return hipSuccess;
  hipLaunchKernelGGL(mx_dequant_kernel, dim3(mx_grid(n8)), dim3(kMxThreads), 0, stream,
                     reinterpret_cast<const uint32_t*>(codes), scales, n8, static_cast<u32x4*>(out));
  return hipGetLastError();
}

}  // namespace megamoe
