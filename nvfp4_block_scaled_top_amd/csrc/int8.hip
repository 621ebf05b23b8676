// 8-bit integers with a scale a row: quantizer and decoder.
//
//   scale = fl32(amax / 127),  code = the whole number nearest to 127 x / amax, ties to even,
// of the exact quotient: the fp32 product x * fl32(127 / amax) is within 127 * 2^-23 < 2^-16 of it, so
// only pieces with an element whose product lies within 2^-15 of a border are taken again, by the sign of
// 254 |x| - (2k + 1) amax, without a rounding.  (16-bit rows meet borders often: amax / 2 is one, 63.5.)  A row with
// an infinity or a NaN gets a NaN scale and zero codes: every product that reads it is NaN.
//
// Memory-bound.  A row stays in registers between its maximum and its codes, so it is read once: 49152 x 2048 in bf16
// takes 49 us (6.2 TB/s read and written), in float32 79 (6.4); decoded 48 and 92 (6.3 and 5.5).
#include "device_common.h"
#include "internal.h"

namespace megamoe {

typedef __bf16 bf16x2n __attribute__((ext_vector_type(2)));
typedef float f32x2n __attribute__((ext_vector_type(2)));

constexpr float kI8Border = 0.5f - 1.0f / 32768.0f;
constexpr float kI8Tiny = 7.8886090522101181e-31f;  // 2^-100: below it 127 / amax may overflow

// Elements of a 16-byte piece as floats.
template <int kDtype>
struct I8In {
  static constexpr int kElems = kDtype == MEGAMOE_DTYPE_F32 ? 4 : 8;
  static __device__ __forceinline__ float get(const u32x4& v, int j) {
    if constexpr (kDtype == MEGAMOE_DTYPE_F32) return __uint_as_float(v[j]);
    else if constexpr (kDtype == MEGAMOE_DTYPE_BF16)
      return __uint_as_float(j & 1 ? v[j / 2] & 0xFFFF0000u : v[j / 2] << 16);
    else {
      const uint32_t pair = v[j / 2];
      return (float)__builtin_bit_cast(f16x2, pair)[j & 1];
    }
  }
};

template <int kDtype>
__device__ __forceinline__ uint32_t i8_amax(const u32x4& v, uint32_t m) {  // bits of |x|: a NaN's are above infinity's
#pragma unroll
  for (int j = 0; j < I8In<kDtype>::kElems; ++j) {
    const uint32_t b = __float_as_uint(I8In<kDtype>::get(v, j)) & 0x7FFFFFFFu;
    m = m > b ? m : b;
  }
  return m;
}

template <int kDtype>
__device__ __forceinline__ void i8_encode(const u32x4& v, float amax, float inv, uint32_t (&w)[2]) {
  constexpr int n = I8In<kDtype>::kElems;
  float q[n], off = 0.0f;
#pragma unroll
  for (int j = 0; j < n; ++j) {
    const float x = I8In<kDtype>::get(v, j) * inv;
    q[j] = rintf(x);
    off = fmaxf(off, fabsf(x - q[j]));
  }
  if (!(off <= kI8Border) || !(amax >= kI8Tiny)) {
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const float x = I8In<kDtype>::get(v, j), ax = fabsf(x);
      if (amax >= kI8Tiny) {  // k or k + 1: whether x is above the border between them, or on it and k is odd
        const float k = floorf(ax * inv);
        bool above, on;
        if constexpr (kDtype == MEGAMOE_DTYPE_F32) {  // 32 and 32 bits
          const double d = fma(-(double)(2.0f * k + 1.0f), (double)amax, 254.0 * (double)ax);
          above = d > 0.0, on = d == 0.0;
        } else {  // (over 256, as 254 |x| may overflow) 18 and 19 bits
          const float d = fmaf(-(2.0f * k + 1.0f) / 256.0f, amax, ax * (254.0f / 256.0f));
          above = d > 0.0f, on = d == 0.0f;
        }
        q[j] = copysignf(k + (above || (on && ((int)k & 1)) ? 1.0f : 0.0f), x);
      } else {  // a quotient that is no border is 2^-33 and more away from one, and a border is met exactly
        q[j] = (float)rint((double)x * 127.0 / (double)amax);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < n / 4; ++j)
    w[j] = ((uint32_t)(int)q[4 * j] & 255u) | ((uint32_t)(int)q[4 * j + 1] & 255u) << 8 |
           ((uint32_t)(int)q[4 * j + 2] & 255u) << 16 | (uint32_t)(int)q[4 * j + 3] << 24;
}

struct I8QuantArgs {
  const u32x4* x;
  const int32_t* row_valid;
  uint8_t* codes;
  float* scales;
  int64_t rows;
  int32_t pieces;  // of 16 bytes a row
};

// kLanes threads a row (a wave, or a workgroup), NP pieces a thread in registers; NP = 0: any number, the row
// is read a second time for its codes.
template <int kDtype, int kLanes, int NP>
__global__ __launch_bounds__(256) void i8_quant_kernel(I8QuantArgs p) {
  constexpr int kRows = 256 / kLanes, n = I8In<kDtype>::kElems;
  __shared__ uint32_t s_max[4];
  const int t = threadIdx.x % kLanes;
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kLanes; row < p.rows;
       row += (int64_t)gridDim.x * kRows) {
    const u32x4* x = p.x + row * p.pieces;
    uint8_t* codes = p.codes + row * (int64_t)p.pieces * n;
    const bool valid = p.row_valid == nullptr || p.row_valid[row] >= 0;
    u32x4 v[NP > 0 ? NP : 1];
    uint32_t m = 0;
    if constexpr (NP > 0) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        v[i] = u32x4{0u, 0u, 0u, 0u};
        if (valid && t + i * kLanes < p.pieces) v[i] = __builtin_nontemporal_load(x + t + i * kLanes);
      }
#pragma unroll
      for (int i = 0; i < NP; ++i) m = i8_amax<kDtype>(v[i], m);
    } else {
      for (int i = t; valid && i < p.pieces; i += kLanes) m = i8_amax<kDtype>(x[i], m);
    }
    m = wave_max_u32(m);
    if constexpr (kLanes > kWave) {
      __syncthreads();  // the row before has been read from s_max
      if (lane_id() == 0) s_max[threadIdx.x / kWave] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) m = m > s_max[i] ? m : s_max[i];
    }
    const bool number = m < 0x7F800000u;
    const float amax = __uint_as_float(m);
    if (t == 0) p.scales[row] = number ? amax / 127.0f : __uint_as_float(0x7FC00000u);
    const bool zero = !number || m == 0;
    const float inv = zero ? 0.0f : 127.0f / amax;
    const auto put = [&](int i, const u32x4& piece) {
      uint32_t w[2] = {0u, 0u};
      if (!zero) i8_encode<kDtype>(piece, amax, inv, w);
      if constexpr (n == 8) reinterpret_cast<u32x2*>(codes)[i] = u32x2{w[0], w[1]};
      else reinterpret_cast<uint32_t*>(codes)[i] = w[0];
    };
    if constexpr (NP > 0) {
#pragma unroll
      for (int i = 0; i < NP; ++i)
        if (t + i * kLanes < p.pieces) put(t + i * kLanes, v[i]);
    } else {
      for (int i = t; i < p.pieces; i += kLanes) put(i, valid ? x[i] : u32x4{0u, 0u, 0u, 0u});
    }
  }
}

// 16 bytes of output a lane and store, so that a wave's stores cover whole lines (16 codes a lane, stored by quarters of a
// line, took 307 us for 49152 x 2048 in float32); kI8Ahead of them a thread, their codes requested first.
constexpr int kI8Ahead = 4, kI8Block = 256 * kI8Ahead;

template <int kDtype>
__global__ __launch_bounds__(256) void i8_dequant_kernel(const uint8_t* codes, const float* scales, int64_t total,
                                                         uint32_t pieces, u32x4* out) {
  constexpr int n = I8In<kDtype>::kElems;  // codes of a piece
  for (int64_t at = (int64_t)blockIdx.x * kI8Block; at < total; at += (int64_t)gridDim.x * kI8Block) {
    const int64_t row0 = at / pieces;
    const uint32_t in0 = (uint32_t)(at - row0 * pieces) + threadIdx.x;
    u32x2 c[kI8Ahead];
    float s[kI8Ahead];
#pragma unroll
    for (int u = 0; u < kI8Ahead; ++u) {
      const int64_t i = at + 256 * u + threadIdx.x;
      if (i >= total) break;
      if constexpr (n == 8) c[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(codes) + i);
      else c[u][0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(codes) + i);
      s[u] = scales[row0 + (in0 + 256 * u) / pieces];
    }
#pragma unroll
    for (int u = 0; u < kI8Ahead; ++u) {
      const int64_t i = at + 256 * u + threadIdx.x;
      if (i >= total) break;
      float f[n];
#pragma unroll
      for (int j = 0; j < n; ++j) f[j] = (float)(int)(int8_t)(c[u][j / 4] >> (8 * (j % 4))) * s[u];
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (kDtype == MEGAMOE_DTYPE_F32) o[j] = __float_as_uint(f[j]);
        else if constexpr (kDtype == MEGAMOE_DTYPE_BF16)
          o[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2n{f[2 * j], f[2 * j + 1]}, bf16x2n));
        else o[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2n{f[2 * j], f[2 * j + 1]}, f16x2));
      }
      __builtin_nontemporal_store(o, out + i);
    }
  }
}

template <int kDtype, int kLanes, int NP>
static void i8_quant_as(const I8QuantArgs& a, hipStream_t stream) {
  constexpr int kRows = 256 / kLanes;
  const int64_t blocks = (a.rows + kRows - 1) / kRows;
  hipLaunchKernelGGL((i8_quant_kernel<kDtype, kLanes, NP>), dim3((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20)), dim3(256),
                     0, stream, a);
}

// Many short rows: a wave a row, else a workgroup (4096 x 2048: 7.5 us and 11.2 in bf16, 6.9 and 7.4 in float32; 16384 x
// 4096: 38.5 and 36.5, 56 and 53; 512 x 2048: 5.4 and 5.3).  Rows of more than 16 pieces a thread are read twice.
template <int kDtype>
static void i8_quant(const I8QuantArgs& a, hipStream_t stream) {
  constexpr int kMost = 2048 / (kWave * I8In<kDtype>::kElems);
  if (a.rows >= 2048 && a.pieces <= kMost * kWave) {
    if (a.pieces <= kWave) i8_quant_as<kDtype, kWave, 1>(a, stream);
    else if (a.pieces <= kMost / 2 * kWave) i8_quant_as<kDtype, kWave, kMost / 2>(a, stream);
    else i8_quant_as<kDtype, kWave, kMost>(a, stream);
    return;
  }
  const int np = (a.pieces + 255) / 256;
  if (np <= 1) i8_quant_as<kDtype, 256, 1>(a, stream);
  else if (np <= 2) i8_quant_as<kDtype, 256, 2>(a, stream);
  else if (np <= 4) i8_quant_as<kDtype, 256, 4>(a, stream);
  else if (np <= 8) i8_quant_as<kDtype, 256, 8>(a, stream);
  else if (np <= 16) i8_quant_as<kDtype, 256, 16>(a, stream);
  else i8_quant_as<kDtype, 256, 0>(a, stream);
}

hipError_t launch_int8_quant(const void* x, int dtype, int64_t rows, int64_t cols, const int32_t* row_valid,
                             int8_t* codes, float* scales, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const I8QuantArgs a{static_cast<const u32x4*>(x), row_valid, reinterpret_cast<uint8_t*>(codes), scales, rows,
                      (int32_t)(cols / (dtype == MEGAMOE_DTYPE_F32 ? 4 : 8))};
  if (dtype == MEGAMOE_DTYPE_F32) i8_quant<MEGAMOE_DTYPE_F32>(a, stream);
  else if (dtype == MEGAMOE_DTYPE_BF16) i8_quant<MEGAMOE_DTYPE_BF16>(a, stream);
  else i8_quant<MEGAMOE_DTYPE_F16>(a, stream);
  return hipGetLastError();
}

hipError_t launch_int8_dequant(const int8_t* codes, const float* scales, int64_t rows, int64_t cols, int dtype,
                               void* out, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  const int64_t pieces = cols / (dtype == MEGAMOE_DTYPE_F32 ? 4 : 8), total = rows * pieces;
  const int64_t blocks = (total + kI8Block - 1) / kI8Block;
  const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20)), block(256);
  const uint8_t* c = reinterpret_cast<const uint8_t*>(codes);
  u32x4* o = static_cast<u32x4*>(out);
  const uint32_t per = (uint32_t)pieces;
  const auto kernel = dtype == MEGAMOE_DTYPE_F32    ? i8_dequant_kernel<MEGAMOE_DTYPE_F32>
                      : dtype == MEGAMOE_DTYPE_BF16 ? i8_dequant_kernel<MEGAMOE_DTYPE_BF16>
                                                    : i8_dequant_kernel<MEGAMOE_DTYPE_F16>;
  hipLaunchKernelGGL(kernel, grid, block, 0, stream, c, scales, total, per, o);
  return hipGetLastError();
}

}  // namespace megamoe
