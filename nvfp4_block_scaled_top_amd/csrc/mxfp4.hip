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

// n8 = elements / 8; rows with row_valid[r] < 0 get zero codes and scales and are not read.  kItems strided
// items a thread, all loaded before the first is used.
template <bool kF32, int kItems>
__global__ __launch_bounds__(kMxThreads) void mx_quant_kernel(const void* __restrict__ x, int64_t n8, int64_t cols8,
                                                              const int32_t* __restrict__ row_valid,
                                                              uint32_t* __restrict__ codes,
                                                              uint8_t* __restrict__ scales) {
  constexpr int kV = kF32 ? 2 : 1;
  const int64_t step = (int64_t)gridDim.x * kMxThreads, i0 = (int64_t)blockIdx.x * kMxThreads + threadIdx.x;
  u32x4 v[kItems][kV];
  bool ok[kItems];
  // the four lanes of a block hold the same block (n8 and step are multiples of 4)
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int64_t i = i0 + k * step;
    ok[k] = i < n8 && (row_valid == nullptr || row_valid[i / cols8] >= 0);
    const u32x4* src = static_cast<const u32x4*>(x) + kV * i;
#pragma unroll
    for (int j = 0; j < kV; ++j) v[k][j] = ok[k] ? __builtin_nontemporal_load(src + j) : u32x4{0u, 0u, 0u, 0u};
  }
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int64_t i = i0 + k * step;
    Mx8 q;
    if constexpr (kF32) q = mx_quant8(v[k][0], v[k][1]);
    else q = mx_quant8(v[k][0]);
    if (i < n8) {
      codes[i] = q.codes;
      if ((i & 3) == 0) scales[i >> 2] = (uint8_t)q.scale;
    }
  }
}

// Items a thread: 4 once that still fills the chip with threads, else 1.  (49152 x 2048 bf16: 51 us with
// one and a loop, 43.5 with four; 8 x 7168: 2.2 us with one.)
constexpr int64_t kMxManyItems = (int64_t)4 * kMxThreads * 2048;
static unsigned mx_grid(int64_t n8, int items) {
  return (unsigned)((n8 + (int64_t)kMxThreads * items - 1) / ((int64_t)kMxThreads * items));
}

hipError_t launch_mx_quant(const void* x, int dtype, int64_t rows, int64_t cols, const int32_t* row_valid,
                           uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  const int64_t n8 = rows * (cols / 8);
  if (n8 == 0) return hipSuccess;
  uint32_t* c = reinterpret_cast<uint32_t*>(codes);
  const bool f32 = dtype == MEGAMOE_DTYPE_F32, many = n8 >= kMxManyItems;
  const auto kernel = f32 ? (many ? mx_quant_kernel<true, 4> : mx_quant_kernel<true, 1>)
                          : (many ? mx_quant_kernel<false, 4> : mx_quant_kernel<false, 1>);
  hipLaunchKernelGGL(kernel, dim3(mx_grid(n8, many ? 4 : 1)), dim3(kMxThreads), 0, stream, x, n8, cols / 8, row_valid,
                     c, scales);
  return hipGetLastError();
}

// Decoder: one lane per code word (eight elements, 16 bytes of bf16).  e2m1 * 2^(scale - 127) has two
// significant bits and is exact in bf16, the subnormal products of scale 0 included; above the range
// (2^128 and up) it is the infinity of bf16.
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

// Inside the normal range the conversion instruction gives the same values four times as fast.
__device__ __forceinline__ u32x4 mx_values8(uint32_t w, uint32_t sc) {
  u32x4 o;
  if (sc >= 2u && sc <= 251u) {
    const float s = __uint_as_float(sc << 23);
    const auto bits = [](bf16x2v v) {
      uint32_t u;
      __builtin_memcpy(&u, &v, 4);
      return u;
    };
    o[0] = bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
    o[1] = bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
    o[2] = bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
    o[3] = bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = mx_value_bits((w >> (8 * j)) & 15u, sc) | (mx_value_bits((w >> (8 * j + 4)) & 15u, sc) << 16);
  }
  return o;
}

template <int kItems>
__global__ __launch_bounds__(kMxThreads) void mx_dequant_kernel(const uint32_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, int64_t n8,
                                                                u32x4* __restrict__ out) {
  const int64_t step = (int64_t)gridDim.x * kMxThreads, i0 = (int64_t)blockIdx.x * kMxThreads + threadIdx.x;
  uint32_t w[kItems], sc[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int64_t i = i0 + k * step;
    w[k] = i < n8 ? codes[i] : 0u;
    sc[k] = i < n8 ? scales[i >> 2] : 127u;
  }
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int64_t i = i0 + k * step;
    const u32x4 o = mx_values8(w[k], sc[k]);
    if (i < n8) __builtin_nontemporal_store(o, out + i);
  }
}

hipError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out,
                             hipStream_t stream) {
  const int64_t n8 = rows * (cols / 8);
  if (n8 == 0) return hipSuccess;
  const bool many = n8 >= kMxManyItems;
  hipLaunchKernelGGL(many ? mx_dequant_kernel<4> : mx_dequant_kernel<1>, dim3(mx_grid(n8, many ? 4 : 1)),
                     dim3(kMxThreads), 0, stream, reinterpret_cast<const uint32_t*>(codes), scales, n8,
                     static_cast<u32x4*>(out));
  return hipGetLastError();
}

}  // namespace megamoe
