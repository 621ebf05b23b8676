// Scored router: logits -> top-k expert ids and weights with sigmoid or softmax scores, a balance
// bias, expert groups and renormalised weights, and the gradient of those weights.
//
// With z the logits of a token, s_e = sigmoid(z_e) or softmax(z)_e in float64 and the choice
// c_e = fl32(s_e) + b_e in float32.  An expert is available unless its logit or choice is NaN or
// -inf.  Experts lie in n_group groups of consecutive ids; a group's score is the sum of its
// group_top largest choices, the topk_group best groups stay, and the k largest choices among
// their experts win (ties, of groups and of experts, go to the lower index).  The weights come
// from the scores, without the bias: w_j = scale * s_j / S, S the sum over the winners
// (renormalised) or 1; s_j / S keeps its value where the scores underflow.
//
// The choice is float32 so that it is the same number in any implementation: float64 scores that
// differ in their last bits round to the same float32 but for one pair in 2^29.
#include "device_common.h"
#include "internal.h"

namespace megamoe {

constexpr int kScoreWaves = 4;  // tokens per workgroup, one wave each

// A logit as float32; NaN is taken as -inf (not available), +inf as the largest float.
__device__ __forceinline__ float logit_of(float v) { return v != v ? -__builtin_huge_valf() : fminf(v, 3.402823466e38f); }
__device__ __forceinline__ float logit_of(uint16_t v) { return logit_of(bf16_bits_to_f32(v)); }

// Reductions over a wave with data-parallel-primitive moves (a few cycles a step; a shuffle through LDS
// takes some 100): rows of 16 lanes by shifts, then lane 15 of a row to the next one and lane 31 to the upper
// half.  Lane 63 holds the result; a lane that receives nothing receives 0, so 0 must not change it.
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_move(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, true);
}
template <typename F>
__device__ __forceinline__ uint32_t dpp_reduce(uint32_t v, F f) {
  v = f(v, dpp_move<0x111>(v));
  v = f(v, dpp_move<0x112>(v));
  v = f(v, dpp_move<0x114>(v));
  v = f(v, dpp_move<0x118>(v));
  v = f(v, dpp_move<0x142>(v));
  v = f(v, dpp_move<0x143>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, kWave - 1);
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <int kCtrl>
__device__ __forceinline__ double dpp_move(double v) {
  const uint64_t b = __double_as_longlong(v);
  return __longlong_as_double((long long)((uint64_t)dpp_move<kCtrl>((uint32_t)(b >> 32)) << 32 |
                                          dpp_move<kCtrl>((uint32_t)b)));
}
__device__ __forceinline__ double read_lane(double v, int lane) {
  const uint64_t b = __double_as_longlong(v);
  return __longlong_as_double((long long)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), lane) << 32 |
                                          (uint32_t)__builtin_amdgcn_readlane((int)b, lane)));
}
__device__ __forceinline__ double score_wave_sum(double v) {
  v += dpp_move<0x111>(v);
  v += dpp_move<0x112>(v);
  v += dpp_move<0x114>(v);
  v += dpp_move<0x118>(v);
  v += dpp_move<0x142>(v);
  v += dpp_move<0x143>(v);
  return read_lane(v, kWave - 1);
}

// e^t: t = n ln 2 + r with |r| <= ln 2 / 2, the Taylor polynomial of e^r up to r^12 / 12! (its
// remainder is at most 1.04 * 2^-52 of e^r) and a scaling by 2^n: 18 instructions, where exp() takes some 40.  The
// constants are held in scalar registers: left to itself the compiler moves each into vector registers before
// every use, two moves a multiplication.
struct ExpConstants {
  double c[13], log2e, ln2_hi, ln2_lo;
};
__device__ __forceinline__ ExpConstants exp_constants() {
  ExpConstants k{{1.0, 1.0, 0.5, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040, 1.0 / 40320, 1.0 / 362880,
                  1.0 / 3628800, 1.0 / 39916800, 1.0 / 479001600},
                 1.4426950408889634,
                 0x1.62e42fefa39efp-1,  // ln 2 to 53 bits, and what is left of it
                 0x1.abc9e3b39803fp-56};
#pragma unroll
  for (int i = 3; i < 12; ++i) asm volatile("" : "+s"(k.c[i]));  // 0.5 and 1 are operands of an instruction
  asm volatile("" : "+s"(k.log2e));
  asm volatile("" : "+s"(k.ln2_hi));
  asm volatile("" : "+s"(k.ln2_lo));
  return k;
}
__device__ __forceinline__ double exp_f64(const ExpConstants& k, double t) {
  t = fmin(fmax(t, -800.0), 800.0);  // beyond: 0 and infinity by the scaling
  const double n = rint(t * k.log2e);
  double r = fma(-n, k.ln2_hi, t);
  r = fma(-n, k.ln2_lo, r);
  double p = k.c[12];
#pragma unroll
  for (int i = 11; i >= 0; --i) p = fma(p, r, k.c[i]);
  return ldexp(p, (int)n);
}

// 1 / d by Newton's steps from the hardware's estimate (d normal).
__device__ __forceinline__ double reciprocal_f64(double d) {
  double y = __builtin_amdgcn_rcp(d);
  y = fma(y, fma(-d, y, 1.0), y);
  return fma(y, fma(-d, y, 1.0), y);
}
// 1 / (1 + e^-z)
__device__ __forceinline__ double sigmoid_f64(const ExpConstants& k, float z) {
  const double y = reciprocal_f64(1.0 + exp_f64(k, -(double)z));
  return z < -709.0f ? 0.0 : y;  // there d is infinite, or 1 / d below every float
}

// Unsigned key whose order is the order of the floats (-0 below +0 is not wanted: both map to +0).
__device__ __forceinline__ uint32_t sort_key(float c) {
  const uint32_t b = __float_as_uint(c + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unsort_key(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}

// A sum of chosen scores below this is taken of relative_score instead.
constexpr double kFarScores = 0x1p-60;

// Key of a chosen lane's logit, 0 for the others; the wave's largest is relative_score's `top`.
__device__ __forceinline__ uint32_t chosen_key(float z, bool chosen) { return chosen ? sort_key(z) : 0u; }
// e^(z - the largest chosen logit), 0 for the other lanes: chosen scores up to a common factor, where the scores
// themselves lose bits or underflow.  Softmax scores are that, and so are sigmoids below 2^-60, which are e^z to
// float64's last bit.
__device__ __forceinline__ double relative_score(const ExpConstants& ec, float z, bool chosen, uint32_t top) {
  return chosen && z > -__builtin_huge_valf() ? exp_f64(ec, (double)z - (double)unsort_key(top)) : 0.0;
}

// One wave per token.  The wave's lanes are split into equal power-of-two runs of `span` lanes, one
// run a group (span = 64 without groups), so a group's best choices are a butterfly over its own
// lanes; lane (q, u) of group q holds its experts q * size + u + span * i.
template <typename T, int PL>
__global__ __launch_bounds__(kScoreWaves* kWave) void router_scores_kernel(RouterScoreArgs p) {
  const int lane = lane_id();
  const int t = blockIdx.x * kScoreWaves + threadIdx.x / kWave;
  if (t >= p.T) return;  // whole waves only
  const int span = 1 << p.span_log2, size = p.E / p.n_group, q = lane >> p.span_log2, u = lane & (span - 1);
  const T* __restrict__ row = static_cast<const T*>(p.logits) + (int64_t)t * p.E;
  const bool sigmoid = p.score == MEGAMOE_SCORE_SIGMOID;

  const ExpConstants ec = exp_constants();
  const float kNone = -__builtin_huge_valf();
  // All loads before their first use, at valid addresses also where a lane has no expert: a guarded load each
  // would wait for the one before.
  float z[PL], bias[PL];
  {
    T raw[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int x = u + span * i, e = q < p.n_group && x < size ? q * size + x : 0;
      raw[i] = row[e];
      bias[i] = p.bias != nullptr ? p.bias[e] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < PL; ++i) z[i] = q < p.n_group && u + span * i < size ? logit_of(raw[i]) : kNone;
  }
  double m = 0.0, inv = 1.0;  // softmax: largest logit, one over the sum
  // Keys of the choices: 0 for an expert that is not available.
  uint32_t key[PL];
  const auto set_key = [&](int i, float s) {
    const float c = s + bias[i];  // (s is not -0)
    key[i] = z[i] > kNone && c > kNone ? sort_key(c) : 0u;
  };
  if (sigmoid) {
#pragma unroll
    for (int i = 0; i < PL; ++i) set_key(i, (float)sigmoid_f64(ec, z[i]));
  } else {
    uint32_t mk = 0;
#pragma unroll
    for (int i = 0; i < PL; ++i) mk = umax(mk, sort_key(z[i]));
    m = (double)unsort_key(dpp_reduce(mk, umax));
    double e[PL], sum = 0.0;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      e[i] = z[i] > kNone ? exp_f64(ec, (double)z[i] - m) : 0.0;
      sum += e[i];
    }
    sum = score_wave_sum(sum);
    inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
    for (int i = 0; i < PL; ++i) set_key(i, (float)(e[i] * inv));
  }
  if (p.topk_group < p.n_group) {
    uint32_t k1 = 0, k2 = 0;  // the two largest keys of the group
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const uint32_t lo = key[i] < k1 ? key[i] : k1;
      k1 = umax(key[i], k1);
      k2 = umax(lo, k2);
    }
    for (int o = 1; o < span; o <<= 1) {
      const uint32_t o1 = __shfl_xor(k1, o, kWave), o2 = __shfl_xor(k2, o, kWave);
      const uint32_t lo = o1 < k1 ? o1 : k1;
      k1 = umax(o1, k1);
      k2 = umax(lo, umax(o2, k2));
    }
    // A group without an available expert has key 0 and comes after every other one, also after a sum that
    // overflows to -inf.
    const uint32_t gk = p.group_top > 1 && k2 ? sort_key(unsort_key(k1) + unsort_key(k2)) : k1;
    int rank = 0;
    for (int g = 0; g < p.n_group; ++g) {
      const uint32_t og = (uint32_t)__builtin_amdgcn_readlane((int)gk, g << p.span_log2);
      rank += (og > gk || (og == gk && g < q)) ? 1 : 0;
    }
    if (rank >= p.topk_group) {
#pragma unroll
      for (int i = 0; i < PL; ++i) key[i] = 0u;
    }
  }
  // k rounds: the largest key of the wave, the lowest expert that has it; its key is then cleared.  Which
  // lanes hold the key is a lane mask for each i, so the search for the expert is scalar work.
  int my_id = -1;
  for (int r = 0; r < p.k; ++r) {
    uint32_t wk = key[0];
#pragma unroll
    for (int i = 1; i < PL; ++i) wk = umax(wk, key[i]);
    wk = dpp_reduce(wk, umax);
    if (wk == 0) break;  // nothing available is left: the remaining slots stay empty
    int win = 0x7FFFFFFF, wi = 0, wl = 0;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const uint64_t mask = __ballot(key[i] == wk);
      if (mask) {  // expert ids ascend with the lane
        const int l = __builtin_ctzll(mask), e = (l >> p.span_log2) * size + (l & (span - 1)) + span * i;
        if (e < win) {
          win = e;
          wi = i;
          wl = l;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (i == wi && lane == wl) key[i] = 0u;
    if (lane == r) my_id = win;
  }
  // The winners' weights, one lane each.
  double ws = 0.0;
  float wz = kNone;
  if (my_id >= 0) {
    wz = logit_of(row[my_id]);
    ws = sigmoid ? sigmoid_f64(ec, wz) : exp_f64(ec, (double)wz - m) * inv;
  }
  double d = 1.0;
  if (p.renormalize) {
    d = score_wave_sum(ws);
    if (d < kFarScores) {  // the bias or the groups left only experts far below the others
      ws = relative_score(ec, wz, my_id >= 0, dpp_reduce(chosen_key(wz, my_id >= 0), umax));
      d = score_wave_sum(ws);
    }
  }
  if (lane < p.k) {
    p.ids[(int64_t)t * p.k + lane] = my_id;
    p.weights[(int64_t)t * p.k + lane] = d > 0.0 ? (float)(ws * (double)p.scale / d) : 0.0f;
  }
}

// Tokens of a launch: a grid holds fewer than 2^32 threads, 2^26 tokens.
constexpr int64_t kScoreTokens = (int64_t)1 << 24;
static int64_t logit_bytes(int dtype) { return dtype == MEGAMOE_DTYPE_F32 ? 4 : 2; }

template <typename T>
static hipError_t launch_scores_t(const RouterScoreArgs& a, hipStream_t stream) {
  const int span = 1 << a.span_log2, per = (a.E / a.n_group + span - 1) / span;
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
  RouterScoreArgs a = a0;
  a.span_log2 = 6;
  while ((a.n_group << a.span_log2) > kWave) --a.span_log2;
  hipError_t err = hipSuccess;
  for (int64_t t = 0; t < a0.T && err == hipSuccess; t += kScoreTokens) {
    a.T = (int32_t)(a0.T - t < kScoreTokens ? a0.T - t : kScoreTokens);
    a.logits = static_cast<const char*>(a0.logits) + t * a.E * logit_bytes(dtype);
    a.ids = a0.ids + t * a.k;
    a.weights = a0.weights + t * a.k;
    err = dtype == MEGAMOE_DTYPE_F32 ? launch_scores_t<float>(a, stream) : launch_scores_t<uint16_t>(a, stream);
  }
  return err;
}

// ---- gradient ------------------------------------------------------------------------------------
// With g the gradient of the weights and n_j = s_j / S: the gradient of the chosen scores is
// g'_j = scale * g_j (weights kept) or scale / S * (g_j - sum_i g_i n_i) (renormalised), and
//   sigmoid: dz_e = g'_e s_e (1 - s_e);    softmax: dz_e = s_e (g'_e - sum_j g'_j s_j),
// with g'_e = 0 for experts that were not chosen (an expert listed twice takes both slots' share).
// Renormalised, sum_j g'_j s_j = 0: a softmax's gradient is then that of a softmax over the chosen experts
// alone and 0 elsewhere, the other logits are not read, and only ratios of chosen scores remain, which
// relative_score gives at any distance from the row's largest logit.
// float64 up to the one rounding of dz, and 1 - s_e never by a subtraction, which would leave no correct bit from
// z = 37 on (or such a distance to a softmax's other logits): for a sigmoid it is sigmoid(-z_e), and a
// softmax's g'_e - sum_j g'_j s_j is taken relative to the expert x of the largest logit, the only one whose score
// may be near 1, as (g'_e - g'_x) - sum_{i != x} (g'_i - g'_x) s_i, and g_j - sum_i g_i n_i relative to the slot of
// the largest chosen logit (one renormalised weight alone: 0 exactly).  8192 tokens x 384 experts, k = 6, float32:
// 8.5 us with sigmoid scores, 8.4 with a renormalised softmax, 12.5 with softmax weights kept as they are (a launch
// takes 2.2, the bytes 2.7 to 4).  One wave per token, lane l holding experts l + 64 i; the
// chosen experts' scores are computed one per lane.
template <typename T>
__device__ __forceinline__ T round_logit(double v);
template <>
__device__ __forceinline__ float round_logit<float>(double v) { return (float)v; }
template <>
__device__ __forceinline__ uint16_t round_logit<uint16_t>(double v) { return (uint16_t)f64_to_bf16_bits(v); }

__device__ __forceinline__ float read_lane(float v, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
__device__ __forceinline__ uint16_t read_lane(uint16_t v, int lane) {
  return (uint16_t)__builtin_amdgcn_readlane((int)v, lane);
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
  const bool every = !sigmoid && !p.renormalize;  // every logit has a gradient

  int id = -1;
  double g = 0.0;
  if (lane < p.k) {
    id = p.ids[(int64_t)t * p.k + lane];
    if (id < 0 || id >= p.E) id = -1;
    g = id >= 0 ? (double)p.grad_weights[(int64_t)t * p.k + lane] * (double)p.scale : 0.0;
  }
  const ExpConstants ec = exp_constants();
  double s[PL];
  double m = 0.0, inv = 1.0, rest = 0.0;  // softmax: largest logit, one over the sum, the sum but for the largest
  int x = 0;                              // the expert of the largest logit
  if (every) {
    const float kNone = -__builtin_huge_valf();
    float z[PL];
    T raw[PL];
    uint32_t mk = 0;
#pragma unroll
    for (int i = 0; i < PL; ++i) raw[i] = row[lane + kWave * i < p.E ? lane + kWave * i : 0];  // all in flight
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      z[i] = lane + kWave * i < p.E ? logit_of(raw[i]) : kNone;
      mk = umax(mk, sort_key(z[i]));
    }
    const uint32_t top = dpp_reduce(mk, umax);
    const float mz = unsort_key(top);
    m = (double)mz;
#pragma unroll
    for (int i = PL - 1; i >= 0; --i) x = z[i] == mz ? lane + kWave * i : x;
    x = __builtin_amdgcn_readlane(x, __builtin_ctzll(__ballot(mk == top)));
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      s[i] = z[i] > kNone ? exp_f64(ec, (double)z[i] - m) : 0.0;
      rest += lane + kWave * i == x ? 0.0 : s[i];
    }
    rest = score_wave_sum(rest);
    inv = mz > kNone ? reciprocal_f64(1.0 + rest) : 0.0;
  }
  // This lane's chosen expert: its score, up to a common factor where it is divided by the sum, and what its g'
  // is multiplied with, s or for a sigmoid s (1 - s).
  double sj = 0.0, fj = 0.0;
  const float zj = id >= 0 ? logit_of(row[id]) : -__builtin_huge_valf();
  if (sigmoid) {
    const double e = exp_f64(ec, -fabs((double)zj)), y = reciprocal_f64(1.0 + e);
    sj = zj < 0.0f ? e * y : y;
    fj = e * y * y;
  } else if (every) {
    fj = sj = zj > -__builtin_huge_valf() ? exp_f64(ec, (double)zj - m) * inv : 0.0;
  }
  if (p.renormalize) {
    const uint32_t key = chosen_key(zj, id >= 0), top = dpp_reduce(key, umax);
    g -= read_lane(g, __builtin_ctzll(__ballot(key == top)));
    if (!sigmoid) fj = sj = relative_score(ec, zj, id >= 0, top);
    double S = score_wave_sum(sj), gs = score_wave_sum(g * sj);
    if (sigmoid && S < kFarScores) {
      fj = sj = relative_score(ec, zj, id >= 0, top);
      S = score_wave_sum(sj);
      gs = score_wave_sum(g * sj);
    }
    const double rS = S > 0.0 ? reciprocal_f64(S) : 0.0;
    g = id >= 0 ? (g - gs * rS) * rS : 0.0;
  }
  // g'_e of this lane's expert: the slots that name it, in slot order; then its gradient.
  double ge = 0.0;
  for (int j = 0; j < p.k; ++j) {
    const double gj = read_lane(g, j);
    ge += __builtin_amdgcn_readlane(id, j) == id ? gj : 0.0;
  }
  T v[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) v[i] = round_logit<T>(0.0);
  if (every) {
    const uint64_t named = __ballot(id == x);
    const double gx = named ? read_lane(ge, __builtin_ctzll(named)) : 0.0;
    const double dot = score_wave_sum(id == x ? 0.0 : g * sj) - gx * (rest * inv);  // sum_{i != x} (g'_i - g'_x) s_i
#pragma unroll
    for (int i = 0; i < PL; ++i) v[i] = round_logit<T>(-(s[i] * inv * (gx + dot)));
    ge = ge - gx - dot;
  }
  const T mine = round_logit<T>(fj * ge);
  for (int j = 0; j < p.k; ++j) {
    const int ej = __builtin_amdgcn_readlane(id, j);  // -1 is no expert: -1 / 64 is no i
    const T vj = read_lane(mine, j);
    const bool here = lane == (ej & (kWave - 1));
#pragma unroll
    for (int i = 0; i < PL; ++i) v[i] = here && (ej >> 6) == i ? vj : v[i];
  }
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + kWave * i;
    if (e < p.E) out[e] = v[i];
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

hipError_t launch_router_scores_bwd(const RouterScoreBwdArgs& a0, int dtype, hipStream_t stream) {
  RouterScoreBwdArgs a = a0;
  hipError_t err = hipSuccess;
  for (int64_t t = 0; t < a0.T && err == hipSuccess; t += kScoreTokens) {
    a.T = (int32_t)(a0.T - t < kScoreTokens ? a0.T - t : kScoreTokens);
    a.logits = static_cast<const char*>(a0.logits) + t * a.E * logit_bytes(dtype);
    a.grad_logits = static_cast<char*>(a0.grad_logits) + t * a.E * logit_bytes(dtype);
    a.ids = a0.ids + t * a.k;
    a.grad_weights = a0.grad_weights + t * a.k;
    err = dtype == MEGAMOE_DTYPE_F32 ? launch_scores_bwd_t<float>(a, stream) : launch_scores_bwd_t<uint16_t>(a, stream);
  }
  return err;
}

}  // namespace megamoe
