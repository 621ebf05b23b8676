// Scored router: logits -> top-k expert ids and weights with sigmoid or softmax scores, a balance
// bias, expert groups and renormalised weights, and the gradient of those weights.
//
// With z the logits of a token, s_e = sigmoid(z_e) or softmax(z)_e in float64 and the choice
// c_e = fl32(s_e) + b_e in float32.  An expert is available unless its logit or choice is NaN or
// -inf.  Experts lie in n_group groups of consecutive ids; a group's score is the sum of its
// group_top largest choices, the topk_group best groups stay, and the k largest choices among
// their experts win (ties, of groups and of experts, go to the lower index).  The weights come
// from the scores, without the bias: w_j = scale * s_j / S, S the sum over the winners
// (renormalised) or 1.
//
// The choice is float32 so that it is the same number in any implementation: float64 scores that
// differ in their last bits round to the same float32 but for one pair in 2^29.
#include "device_common.h"
#include "internal.h"

namespace megamoe {

constexpr int kScoreWaves = 4;  // tokens per workgroup, one wave each

// A logit as float64; NaN is taken as -inf (not available), +inf as the largest float.
template <typename T>
__device__ __forceinline__ float load_logit(const T* p);
template <>
__device__ __forceinline__ float load_logit<float>(const float* p) {
  const float v = *p;
  return v != v ? -__builtin_huge_valf() : fminf(v, 3.402823466e38f);
}
template <>
__device__ __forceinline__ float load_logit<uint16_t>(const uint16_t* p) {
  const float v = bf16_bits_to_f32(*p);
  return v != v ? -__builtin_huge_valf() : fminf(v, 3.402823466e38f);
}

__device__ __forceinline__ float score_wave_max(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, kWave));
  return v;
}

__device__ __forceinline__ double score_wave_sum(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

// Unsigned key whose order is the order of the floats (-0 below +0 is not wanted: both map to +0).
__device__ __forceinline__ uint32_t sort_key(float c) {
  const uint32_t b = __float_as_uint(c + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unsort_key(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}

// One wave per token.  The wave's lanes are split into equal power-of-two runs of `span` lanes, one
// run a group (span = 64 without groups), so a group's best choices are a butterfly over its own
// lanes; lane (q, u) of group q holds its experts q * size + u + span * i.
template <typename T, int PL>
__global__ __launch_bounds__(kScoreWaves* kWave) void router_scores_kernel(RouterScoreArgs p) {
  const int lane = lane_id();
  const int t = blockIdx.x * kScoreWaves + threadIdx.x / kWave;
  if (t >= p.T) return;  // whole waves only
  const int size = p.E / p.n_group, q = lane / p.span, u = lane & (p.span - 1);
  const T* __restrict__ row = static_cast<const T*>(p.logits) + (int64_t)t * p.E;
  const bool sigmoid = p.score == MEGAMOE_SCORE_SIGMOID;

  float z[PL];
  float m = -__builtin_huge_valf();
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int x = u + p.span * i;
    const bool in = q < p.n_group && x < size;
    z[i] = in ? load_logit<T>(row + q * size + x) : -__builtin_huge_valf();
    m = fmaxf(m, z[i]);
  }
  double s[PL];
  double sum = 1.0;
  if (sigmoid) {
#pragma unroll
    for (int i = 0; i < PL; ++i) s[i] = 1.0 / (1.0 + exp(-(double)z[i]));
  } else {
    m = score_wave_max(m);
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      s[i] = z[i] > -__builtin_huge_valf() ? exp((double)z[i] - (double)m) : 0.0;
      sum += s[i];
    }
    sum = score_wave_sum(sum);
#pragma unroll
    for (int i = 0; i < PL; ++i) s[i] = sum > 0.0 ? s[i] / sum : 0.0;
  }
  // Keys of the choices: 0 for an expert that is not available.
  uint32_t key[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int x = u + p.span * i;
    float c = (float)s[i];
    if (p.bias != nullptr && q < p.n_group && x < size) c += p.bias[q * size + x];
    const bool ok = z[i] > -__builtin_huge_valf() && c > -__builtin_huge_valf();
    key[i] = ok ? sort_key(c) : 0u;
  }
  if (p.topk_group < p.n_group) {
    uint32_t k1 = 0, k2 = 0;  // the two largest keys of the group
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const uint32_t lo = key[i] < k1 ? key[i] : k1;
      k1 = key[i] > k1 ? key[i] : k1;
      k2 = lo > k2 ? lo : k2;
    }
    for (int o = 1; o < p.span; o <<= 1) {
      const uint32_t o1 = __shfl_xor(k1, o, kWave), o2 = __shfl_xor(k2, o, kWave);
      const uint32_t lo = o1 < k1 ? o1 : k1;
      const uint32_t hi2 = o2 > k2 ? o2 : k2;
      k1 = o1 > k1 ? o1 : k1;
      k2 = lo > hi2 ? lo : hi2;
    }
    // A group without an available expert comes after every other one.
    float gs = k1 ? unsort_key(k1) : -__builtin_huge_valf();
    if (p.group_top > 1 && k2) gs += unsort_key(k2);
    int rank = 0;
    for (int g = 0; g < p.n_group; ++g) {
      const float og = __shfl(gs, g * p.span, kWave);
      rank += (og > gs || (og == gs && g < q)) ? 1 : 0;
    }
    if (rank >= p.topk_group) {
#pragma unroll
      for (int i = 0; i < PL; ++i) key[i] = 0u;
    }
  }
  // k rounds: the largest key, the lowest expert among equal ones; the winner's key is then cleared.
  int my_id = -1;
  double my_s = 0.0, total = 0.0;
  for (int r = 0; r < p.k; ++r) {
    uint32_t bk = 0;
    int bi = 0x7FFFFFFF;
    double bs = 0.0;
#pragma unroll
    for (int i = 0; i < PL; ++i) {  // ascending expert ids within the lane
      if (key[i] > bk) {
        bk = key[i];
        bi = q * size + u + p.span * i;
        bs = s[i];
      }
    }
    uint32_t wk = bk;
    int wi = bi;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
      const uint32_t ok = __shfl_xor(wk, o, kWave);
      const int oi = __shfl_xor(wi, o, kWave);
      if (ok > wk || (ok == wk && oi < wi)) {
        wk = ok;
        wi = oi;
      }
    }
    if (wk == 0) break;  // nothing available is left: the remaining slots stay empty
    const uint64_t owner = __ballot(bk == wk && bi == wi);
    const double ws = __shfl(bs, __ffsll((unsigned long long)owner) - 1, kWave);
    total += ws;
    if (lane == r) {
      my_id = wi;
      my_s = ws;
    }
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (q * size + u + p.span * i == wi) key[i] = 0u;
  }
  if (lane < p.k) {
    const double d = p.renormalize ? total : 1.0;
    p.ids[(int64_t)t * p.k + lane] = my_id;
    p.weights[(int64_t)t * p.k + lane] = my_id >= 0 && d > 0.0 ? (float)(my_s * (double)p.scale / d) : 0.0f;
  }
}

template <typename T>
static hipError_t launch_scores_t(const RouterScoreArgs& a, hipStream_t stream) {
  const int per = (a.E / a.n_group + a.span - 1) / a.span;
  const dim3 grid((a.T + kScoreWaves - 1) / kScoreWaves), block(kScoreWaves * kWave);
#define MEGAMOE_SCORES(PL)                                                                  \
  if (per <= PL) {                                                                          \
    hipLaunchKernelGGL((router_scores_kernel<T, PL>), grid, block, 0, stream, a);           \
    return hipGetLastError();                                                               \
  }
  MEGAMOE_SCORES(2)
  MEGAMOE_SCORES(4)
  MEGAMOE_SCORES(6)
  MEGAMOE_SCORES(8)
  MEGAMOE_SCORES(16)
  MEGAMOE_SCORES(32)
#undef MEGAMOE_SCORES
  return hipErrorInvalidValue;  // not reached: at most 1024 experts, a span of at least 64 / (2 * n_group)
}

hipError_t launch_router_scores(const RouterScoreArgs& a0, int dtype, hipStream_t stream) {
  if (a0.T == 0) return hipSuccess;
  RouterScoreArgs a = a0;
  a.span = kWave;
  while (a.span * a.n_group > kWave) a.span >>= 1;
  return dtype == MEGAMOE_DTYPE_F32 ? launch_scores_t<float>(a, stream) : launch_scores_t<uint16_t>(a, stream);
}

// ---- gradient ------------------------------------------------------------------------------------
// With g the gradient of the weights and n_j = s_j / S: the gradient of the chosen scores is
// g'_j = scale * g_j (weights kept) or scale / S * (g_j - sum_i g_i n_i) (renormalised), and
//   sigmoid: dz_e = g'_e s_e (1 - s_e);    softmax: dz_e = s_e (g'_e - sum_j g'_j s_j),
// with g'_e = 0 for experts that were not chosen (an expert listed twice takes both slots' share).
// float64 up to the one rounding of dz.  One wave per token, lane l holding experts l + 64 i; the
// chosen experts' scores are computed one per lane.
template <typename T>
__device__ __forceinline__ void store_logit(T* p, double v);
template <>
__device__ __forceinline__ void store_logit<float>(float* p, double v) { *p = (float)v; }
template <>
__device__ __forceinline__ void store_logit<uint16_t>(uint16_t* p, double v) {
  *p = (uint16_t)f64_to_bf16_bits(v);
}

template <typename T, int PL>
__global__ __launch_bounds__(kScoreWaves* kWave) void router_scores_bwd_kernel(RouterScoreBwdArgs p) {
  const int lane = lane_id();
  const int t = blockIdx.x * kScoreWaves + threadIdx.x / kWave;
  if (t >= p.T) return;  // whole waves only
  // may be the same memory: a wave reads its whole row before it writes it
  const T* row = static_cast<const T*>(p.logits) + (int64_t)t * p.E;
  T* out = static_cast<T*>(p.grad_logits) + (int64_t)t * p.E;
  const bool sigmoid = p.score == MEGAMOE_SCORE_SIGMOID;

  int id = -1;
  double g = 0.0;
  if (lane < p.k) {
    id = p.ids[(int64_t)t * p.k + lane];
    if (id < 0 || id >= p.E) id = -1;
    g = id >= 0 ? (double)p.grad_weights[(int64_t)t * p.k + lane] * (double)p.scale : 0.0;
  }
  double s[PL];
  double m = 0.0, sum = 1.0;
  if (!sigmoid) {
    float z[PL], mf = -__builtin_huge_valf();
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + kWave * i;
      z[i] = e < p.E ? load_logit<T>(row + e) : -__builtin_huge_valf();
      mf = fmaxf(mf, z[i]);
    }
    m = (double)score_wave_max(mf);
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      s[i] = z[i] > -__builtin_huge_valf() ? exp((double)z[i] - m) : 0.0;
      sum += s[i];
    }
    sum = score_wave_sum(sum);
#pragma unroll
    for (int i = 0; i < PL; ++i) s[i] = sum > 0.0 ? s[i] / sum : 0.0;
  }
  double sj = 0.0;  // score of this lane's chosen expert
  if (id >= 0) {
    const float zj = load_logit<T>(row + id);
    if (sigmoid) sj = 1.0 / (1.0 + exp(-(double)zj));
    else sj = zj > -__builtin_huge_valf() && sum > 0.0 ? exp((double)zj - m) / sum : 0.0;
  }
  if (p.renormalize) {
    const double S = score_wave_sum(sj), gs = score_wave_sum(g * sj);
    g = S > 0.0 && id >= 0 ? (g - gs / S) / S : 0.0;
  }
  const double dot = sigmoid ? 0.0 : score_wave_sum(g * sj);
  const double d1 = sigmoid ? g * sj * (1.0 - sj) : g;  // what slot `lane` adds to its expert
  double acc[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) acc[i] = 0.0;
  for (int j = 0; j < p.k; ++j) {
    const int ej = __shfl(id, j, kWave);
    const double dj = __shfl(d1, j, kWave);
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (lane + kWave * i == ej) acc[i] += dj;
  }
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + kWave * i;
    if (e < p.E) store_logit<T>(out + e, sigmoid ? acc[i] : s[i] * (acc[i] - dot));
  }
}

template <typename T>
static hipError_t launch_scores_bwd_t(const RouterScoreBwdArgs& a, hipStream_t stream) {
  const int per = (a.E + kWave - 1) / kWave;
  const dim3 grid((a.T + kScoreWaves - 1) / kScoreWaves), block(kScoreWaves * kWave);
#define MEGAMOE_SCORES(PL)                                                                  \
  if (per <= PL) {                                                                          \
    hipLaunchKernelGGL((router_scores_bwd_kernel<T, PL>), grid, block, 0, stream, a);       \
    return hipGetLastError();                                                               \
  }
  MEGAMOE_SCORES(2)
  MEGAMOE_SCORES(6)
  MEGAMOE_SCORES(16)
#undef MEGAMOE_SCORES
  return hipErrorInvalidValue;  // not reached: at most 1024 experts
}

hipError_t launch_router_scores_bwd(const RouterScoreBwdArgs& a, int dtype, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  return dtype == MEGAMOE_DTYPE_F32 ? launch_scores_bwd_t<float>(a, stream) : launch_scores_bwd_t<uint16_t>(a, stream);
}

}  // namespace megamoe
