// Routing of tokens to experts: scores, groups, the top-k and its weights.
//
//   s_e = softmax(x)_e or 1 / (1 + exp(-x_e)),  order by s_e + bias_e
//   (without a bias by x_e, which orders alike), of the topk_groups best
//   groups only; w = s of the chosen, renormalised, times the scale.
//
// The choice is that of f64 scores: f32 makes near ones equal.  Nearly all of
// the work is done in f32 all the same, with bounds on what it may be off by;
// the few candidates that are left are ordered by f64 scores, and a token that
// the bounds do not decide is done again in f64 throughout: 0.005 % of them with
// 8 of 256 experts in groups and f32 logits of any values, 0.1 to 1 % where f32
// logits hold bf16 values, half and more of them where the logits are so coarse
// that most rows tie at the last choice.
//
// Bound by instructions and latency (980 vector instructions for the four
// tokens of a wave with 256 experts in groups, 450 with 128 bf16 ones).
// Measured on MI355X, in a captured graph: 16384 tokens of 128 bf16 experts 5.0
// us and 16381 of 256 f32 experts in groups, with a bias, 11.5 us, 14.5 where a
// token is done again; in f64 throughout they took 54 and 80.  Memory alone
// would take 0.9 and 3.0 us, an empty launch 1.9.  16384 of 128 f32 experts: 5.9
// us, with bf16 values 9.4, with multiples of a half 28.  16384 of 72 experts in
// groups of 9: 6.8 us, in f64 34.
#include <cmath>

#include "dev_common.h"
#include "hum_internal.h"
#include "rows.h"

namespace hum {

constexpr int kRouteMaxExperts = 512;
constexpr int kRouteMaxTopk = 64;

struct RouteParams {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  int64_t tokens, ld;
  int32_t experts, topk, groups, topk_groups, per_group;
  int32_t sigmoid, bf16, top2, renormalize;
  int32_t vec;         // four logits at once
  int32_t candidates;  // topk, and two more where a cut key is not exact
  int32_t exact_cut;   // a cut key holds the whole of its key
  uint32_t low_mask;   // of a cut key: the expert's number
  float inv_group, scale;  // 1 / (per_group, or per_group / 4 where groups are of whole quads)
};

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)dpp<CTRL>((uint32_t)b) | ((uint64_t)dpp<CTRL>((uint32_t)(b >> 32)) << 32));
}
// Over the 16 lanes of a token.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  auto up = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  v = up(v, dpp<0x128>(v));
  v = up(v, dpp<0x124>(v));
  v = up(v, dpp<0x122>(v));
  return up(v, dpp<0x121>(v));
}
__device__ __forceinline__ double row16_sum(double v) {
  v += dpp<0x128>(v);
  v += dpp<0x124>(v);
  v += dpp<0x122>(v);
  return v + dpp<0x121>(v);
}
__device__ __forceinline__ double row16_max(double v) {
  v = fmax(v, dpp<0x128>(v));
  v = fmax(v, dpp<0x124>(v));
  v = fmax(v, dpp<0x122>(v));
  return fmax(v, dpp<0x121>(v));
}
__device__ __forceinline__ double lane_of(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, lane), hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)lo | (uint64_t)hi << 32);
}
// Over the 64 lanes of a wave, the same in all of them.
__device__ __forceinline__ double wave_max(double v) {
  v = row16_max(v);
  return fmax(fmax(lane_of(v, 0), lane_of(v, 16)), fmax(lane_of(v, 32), lane_of(v, 48)));
}
__device__ __forceinline__ double wave_sum(double v) {
  v = row16_sum(v);
  return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}

// 2^1023 for infinity; smaller numbers as they are.
__device__ __forceinline__ double below_nan(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const int32_t hi = (int32_t)(b >> 32);
  return __builtin_bit_cast(double, (uint64_t)(uint32_t)(hi < 0x7FE00000 ? hi : 0x7FE00000) << 32 | (uint32_t)b);
}

// One token by one wave, all in f64; lane l has the experts l, l + 64, ... (N of them)
// keys: LDS of this wave alone.  What calls exp stays rolled: it runs seldom,
// and what it holds in registers the kernel around it does not have.
template <int N>
__device__ __forceinline__ void route_exactly(const RouteParams& p, int64_t t, double* keys) {
  const int lane = threadIdx.x & 63;
  const double none = -__builtin_inf();
  auto logit = [&](int e) {
    return p.bf16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(p.logits)[t * p.ld + e]) : static_cast<const float*>(p.logits)[t * p.ld + e];
  };
  auto fence = [] {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
  double top = none, sum = 0.0;
  // (the rolled loops read the logits from LDS: one latency for four loads)
#pragma unroll 4
  for (int j = 0; j < N; ++j) {
    const int e = j * 64 + lane;
    const float x = logit(e < p.experts ? e : 0);
    keys[e] = x;
    if (e < p.experts) top = fmax(top, (double)x);
  }
  fence();
  if (!p.sigmoid) {
    top = wave_max(top);
#pragma unroll 1
    for (int e = lane; e < p.experts; e += 64) {
      const double x = keys[e];
      if (x != none) sum += exp(x - top);
    }
    sum = wave_sum(sum);
  }
  auto score = [&](double x) {
    const double v = exp(p.sigmoid ? -x : x - top);
    return p.sigmoid ? 1.0 / (1.0 + v) : v / sum;
  };
  // (where a NaN leaves no softmax, the logits order)
  const bool by_bias = p.bias && sum == sum, by_score = p.groups > 1 && p.top2 && !p.bias && sum == sum;
  // What an expert is ordered by, and its group (by its score then).  NaNs come
  // first: infinity is theirs, what is infinite of itself becomes 2^1023.
#pragma unroll 2
  for (int e = lane; e < p.experts; e += 64) {
    const double by = p.bias ? (double)p.bias[e] : 0.0;
    double k = by == none ? none : keys[e];
    if (k != none && (by_bias || by_score)) k = score(k) + by;
    keys[e] = k == k ? below_nan(k) : -none;
  }
  fence();
  double key[N];
#pragma unroll
  for (int j = 0; j < N; ++j) key[j] = j * 64 + lane < p.experts ? keys[j * 64 + lane] : none;
  if (p.groups > 1) {
    // lane g looks at group g (at most 64 of them)
    double a = none, b = none;
    const int from = lane < p.groups ? lane * p.per_group : 0;
#pragma unroll 8
    for (int i = 0; i < p.per_group; ++i) {
      const double v = keys[from + i];
      b = fmax(b, fmin(a, v));
      a = fmax(a, v);
    }
    if (p.top2 && b != none && a != -none) a = below_nan(a + b);
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const double o = lane_of(a, g);
      rank += (int)(o > a) | ((int)(o == a) & (int)(g < lane));
    }
    const uint64_t kept = __ballot(lane < p.groups && rank < p.topk_groups);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = j * 64 + lane;
      if (e >= p.experts) continue;
      if (by_score && key[j] != none) {  // (their own order is that of the logits)
        const double x = logit(e);
        key[j] = x == x ? below_nan(x) : -none;
      }
      if (!((kept >> (e / p.per_group)) & 1)) key[j] = none;
    }
  }
  int id = -1;  // lane n: the n-th choice
  for (int n = 0; n < p.topk; ++n) {
    double best = none;
#pragma unroll
    for (int j = 0; j < N; ++j) best = fmax(best, key[j]);
    best = wave_max(best);
    if (best == none) break;  // nothing is left (the same in every lane)
    int at = -1;              // the lowest of those that have it
#pragma unroll
    for (int j = N - 1; j >= 0; --j) {
      const uint64_t have = __ballot(key[j] == best);
      if (have) at = j * 64 + __builtin_ctzll(have);
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (at == j * 64 + lane) key[j] = none;
    if (lane == n) id = at;
  }
  double w = id < 0 ? 0.0 : score(logit(id));
  if (p.renormalize) {
    const double all = wave_sum(w);
    if (all != 0.0 && id >= 0) w /= all;  // (ids of -1 keep 0 where the others' sum is a NaN)
  }
  if (lane < p.topk) {
    p.ids[t * p.topk + lane] = id;
    p.weights[t * p.topk + lane] = (float)(w * p.scale);
  }
  fence();
}

// Calls fn with lane I of the token's lanes broadcast by `DPP row_newbcast`,
// I = 0 .. n - 1 (n the same in the whole wave).
template <int I, typename F>
__device__ __forceinline__ void each_lane(int n, F&& fn) {
  if constexpr (I < 16) {
    if (I < n) {
      fn(std::integral_constant<int, 0x150 + I>{});
      each_lane<I + 1>(n, fn);
    }
  }
}

// f32 bits that compare as unsigned numbers as the values do, and back.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// The cut key of -inf is below this, that of any number above.
constexpr uint32_t kNoKey = 0x00800000u;
constexpr int kRowShl1 = 0x101;  // DPP row_shl:1, a lane gets the next one's

// 1 / d to f64's last bit or two, d in [2^-1000, 2^1000]: the instruction's
// estimate and two Newton steps.
__device__ __forceinline__ double reciprocal(double d) {
  double y = __builtin_amdgcn_rcp(d);
  y = __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
  return __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
}

// exp(d), d <= 0, to 2^-33 of itself (0 from -690 down, to 2^-995): d log2(e)
// is a whole number n, which the sum with 1.5 * 2^52 holds in its low bits, and
// a rest f in [-1/2, 1/2]; 2^f by the polynomial through its values at the
// eight Chebyshev points (2^-34 off at most); n goes to the exponent's bits.
__device__ __forceinline__ double exp_of(double d) {
  constexpr double kLog2e = 1.4426950408889634, kWhole = 0x1.8p52;
  d = fmax(d, -690.0);
  const double m = __builtin_fma(d, kLog2e, kWhole);
  const double f = __builtin_fma(d, kLog2e, kWhole - m);
  double y = 1.5303700711365693e-05;
  y = __builtin_fma(y, f, 0.00015469729214118296);
  y = __builtin_fma(y, f, 0.0013333478473685416);
  y = __builtin_fma(y, f, 0.009618025613318034);
  y = __builtin_fma(y, f, 0.055504109063258665);
  y = __builtin_fma(y, f, 0.24022651213498092);
  y = __builtin_fma(y, f, 0.6931471805568324);
  y = __builtin_fma(y, f, 0.9999999999595618);
  return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, y) + (__builtin_bit_cast(uint64_t, m) << 52));
}

// What the experts are ordered by: their logits, or scores with a bias.
enum { kByLogit = 0, kBySigmoid = 1, kBySoftmax = 2 };
// Groups: none, of a multiple of 4 experts, of any number of them.
enum { kNoGroups = 0, kQuadGroups = 1, kAnyGroups = 2 };

// 16 lanes per token, four tokens per wave.  Lane l has the experts 64 b + 4 l
// .. + 3 of NB blocks.  Keys are formed in f32 and cut to what leaves room for
// the expert's number below them, so that one maximum finds both; topk + 2 of
// them are taken.  Those candidates then get f64 keys, a lane each, and their
// exact order; the first topk stand if the last of them is above whatever was
// not taken can be, and a token for which that (or the choice of groups) is
// too near to tell is done again by route_exactly.
template <typename T, int NB, int ORDER, int GROUPS>
__global__ __launch_bounds__(256, 4) void route_kernel(const RouteParams p) {
  constexpr int kOfGroups = GROUPS == kAnyGroups ? NB * 64 * 2 : 0;  // four tokens' f32 keys
  __shared__ double keys[4][kOfGroups > kRouteMaxExperts ? kOfGroups : kRouteMaxExperts];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane & 15;
  constexpr bool BIAS = ORDER != kByLogit;
  const bool sigmoid = ORDER == kBySigmoid || (ORDER == kByLogit && p.sigmoid);
  const float none = -__builtin_inff();
  const uint32_t low = p.low_mask;
  const int64_t tw = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 4;
  const bool have = tw < p.tokens;
  const int64_t t = have ? tw : p.tokens - 1;
  const T* row = static_cast<const T*>(p.logits) + t * p.ld;
  float x[NB][4], bias[NB][4];
  if (p.vec) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int e = b * 64 + l * 4;
      const bool in = e < p.experts;
      const int at = in ? e : 0;  // (no branch between the loads)
      if constexpr (sizeof(T) == 2) {
        const u32x2_t v = *reinterpret_cast<const u32x2_t*>(row + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[b][i] = in ? __uint_as_float(i & 1 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16) : none;
      } else {
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(row + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[b][i] = in ? v[i] : none;
      }
      if constexpr (BIAS) {
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(p.bias + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) bias[b][i] = v[i];
      }
    }
  } else {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = b * 64 + l * 4 + i;
        const bool in = e < p.experts;
        x[b][i] = none;
        bias[b][i] = 0.0f;
        if (in) {
          if constexpr (sizeof(T) == 2) x[b][i] = bf16_bits_to_f32(row[e]);
          else x[b][i] = row[e];
          if constexpr (BIAS) bias[b][i] = p.bias[e];
        }
      }
  }
  bool ok = true;
  // The largest logit, and the sum of exp(x - top): in f32, which the margins
  // below and renormalised weights (they do not depend on it) allow.  Other
  // weights are quotients by it, and an f32 one would move them by up to 7 times
  // what their rounding does: they have the sum of f64 terms, here or, where the
  // biases leave too few registers here, behind the choice (16384 tokens, 8 of
  // 256 experts: 9.6 us, renormalised 8.1; with a bias 11.7 and 9.2).
  constexpr bool kSumLater = ORDER == kBySoftmax;
  float top = none, sum = 0.0f;
  double total = 0.0;
  if (!sigmoid) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = __builtin_fmaxf(top, x[b][i]);
    top = row16_max(top);
    if (kSumLater || p.renormalize) {
      const float shift = top > none ? top : 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = __builtin_amdgcn_exp2f((x[b][i] - shift) * 1.44269504f);
        sum += (e[0] + e[1]) + (e[2] + e[3]);
      }
      sum = row16_sum(sum);
      total = sum;
    } else {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) total += exp_of((double)x[b][i] - (double)top);
      total = row16_sum(total);
      sum = (float)total;
    }
  }
  // scores of logits (of -inf: 0)
  auto scores = [&](float (&v)[NB][4]) {
    if (sigmoid) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[b][i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v[b][i] * -1.44269504f));
    } else {
      const float r = __builtin_amdgcn_rcpf(sum);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[b][i] = __builtin_amdgcn_exp2f((v[b][i] - top) * 1.44269504f) * r;
    }
  };
  // what the experts are ordered by: -inf for those that take no part; whether
  // a NaN or +inf is among them
  float key[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) key[b][i] = x[b][i] + (BIAS ? -0.0f : 0.0f);  // (a zero's sign orders nothing)
  if constexpr (BIAS) {
    scores(key);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) key[b][i] = x[b][i] == none ? none : key[b][i] + bias[b][i];
  }
  bool odd = false;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) odd = odd || !(key[b][i] < __builtin_inff());
  if constexpr (GROUPS != kNoGroups) {
    float v[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[b][i] = key[b][i];
    if (!BIAS && p.top2) {
      scores(v);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[b][i] = key[b][i] > none ? v[b][i] : none;
    }
    float a = none, c = none;  // lane g: group g's best two
    if constexpr (GROUPS == kQuadGroups) {
      // each lane's four experts to LDS: their best two
      typedef float f32x2_t __attribute__((ext_vector_type(2)));
      f32x2_t* mine = reinterpret_cast<f32x2_t*>(keys[wave]) + (lane >> 4) * (kRouteMaxExperts / 4);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float a0 = __builtin_fmaxf(v[b][0], v[b][1]), c0 = __builtin_fminf(v[b][0], v[b][1]);
        const float a1 = __builtin_fmaxf(v[b][2], v[b][3]), c1 = __builtin_fminf(v[b][2], v[b][3]);
        mine[b * 16 + l] = f32x2_t{__builtin_fmaxf(a0, a1), __builtin_fmaxf(__builtin_fminf(a0, a1), __builtin_fmaxf(c0, c1))};
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const int quads = p.per_group / 4, mine0 = l < p.groups ? l * quads : 0;
#pragma unroll 4
      for (int i = 0; i < quads; ++i) {
        const f32x2_t v = mine[mine0 + i];
        c = __builtin_fmaxf(__builtin_fmaxf(c, v[1]), __builtin_fminf(a, v[0]));
        a = __builtin_fmaxf(a, v[0]);
      }
    } else {
      float* mine = reinterpret_cast<float*>(keys[wave]) + (lane >> 4) * (NB * 64);
#pragma unroll
      for (int b = 0; b < NB; ++b) *reinterpret_cast<f32x4_t*>(mine + b * 64 + l * 4) = f32x4_t{v[b][0], v[b][1], v[b][2], v[b][3]};
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const int mine0 = l < p.groups ? l * p.per_group : 0;
#pragma unroll 4
      for (int i = 0; i < p.per_group; ++i) {
        const float v = mine[mine0 + i];
        c = __builtin_fmaxf(c, __builtin_fminf(a, v));
        a = __builtin_fmaxf(a, v);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    // How far a group's f32 score may be off.  A sigmoid by 2^-22 (the
    // exponential, its argument's rounding, the sum and the reciprocal); a
    // softmax, d below the top one, by (2.25 d + 3) 2^-24 of itself, which is
    // below 2^-22 of the largest, 1 / sum, and by the sum's 2^-19 and the
    // reciprocal's 2^-23, one factor for all scores, which orders nothing where
    // there is no bias; the sum with the bias by half an ulp, and so the sum of
    // two and the bounds.
    float err = sigmoid ? 0x1p-21f : __builtin_amdgcn_rcpf(sum) * (BIAS ? 0x1p-21f + 0x1.2p-18f : 0x1p-21f);
    err = __builtin_fmaf(__builtin_fabsf(a), 0x1.9p-23f, err);
    float down = a;
    if (p.top2 && c > none) {
      err = __builtin_fmaf(__builtin_fabsf(c), 0x1.9p-23f, err);
      down = a + c;
      a = __builtin_fmaxf(down, -0x1.fffffep127f);  // (two lowest values: not an empty group yet)
    }
    if (l >= p.groups) a = none;
    const float lowest = a > none ? down - err : __builtin_inff(), highest = a > none ? a + err : none;
    int rank = 0;
    each_lane<0>(p.groups, [&](auto ctrl) {
      constexpr int C = decltype(ctrl)::value;
      const float o = __uint_as_float(dpp<C>(__float_as_uint(a)));
      rank += (int)(o > a) | ((int)(o == a) & (int)(C - 0x150 < l));
    });
    const bool keep = l < p.groups && rank < p.topk_groups;
    // the least of those that stay and the most of the others (by logits the
    // comparison is exact; where an empty group stays, the others are empty)
    const float least = -row16_max(keep ? -lowest : none), most = row16_max(keep ? none : highest);
    if (BIAS || p.top2) ok = least > most;
    const uint32_t kept = (uint32_t)(__ballot(keep) >> (lane & 48)) & 0xFFFFu;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      int g = (int)(((float)(b * 16 + l) + 0.5f) * p.inv_group);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (GROUPS == kAnyGroups) g = (int)(((float)(b * 64 + l * 4 + i) + 0.5f) * p.inv_group);
        key[b][i] = (kept >> (g & 31)) & 1 ? key[b][i] : none;
      }
    }
  }
  // Cut keys: what takes no part lies below kNoKey.
  uint32_t cut[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) cut[b][i] = (ordered(key[b][i]) & ~low) | ((low - (uint32_t)(l * 4) - (uint32_t)(b * 64 + i)) & low);
  // the candidates, lane n the n-th
  const int n_cand = p.candidates;
  uint32_t best = 0, mine = 0;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) best = cut[b][i] > best ? cut[b][i] : best;
  best = row16_max(best);
  for (int n = 0;; ++n) {
    mine = l == n ? best : mine;
    if (n + 1 == n_cand) break;
    // The largest below `best`: keys minus it wrap to the top of the range,
    // those already taken to its bottom.
    uint32_t next = 0;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t d = cut[b][i] - best;
        next = d > next ? d : next;
      }
    next = row16_max(next);
    best = best < kNoKey ? best : best + next;
  }
  if (kSumLater && !p.renormalize) {
    total = 0.0;
#pragma unroll 2
    for (int e = l; e < p.experts; e += 16) {
      float v;
      if constexpr (sizeof(T) == 2) v = bf16_bits_to_f32(row[e]);
      else v = row[e];
      total += exp_of((double)v - (double)top);
    }
    total = row16_sum(total);
  }
  // their exact keys
  const int id = mine >= kNoKey ? (int)(low - (mine & low)) : -1;
  double s = 0.0, k = -__builtin_inf();
  if (id >= 0) {
    float v;
    if constexpr (sizeof(T) == 2) v = bf16_bits_to_f32(row[id]);
    else v = row[id];
    const double by = BIAS ? (double)p.bias[id] : 0.0;
    const double e = exp(sigmoid ? -(double)v : (double)v - (double)top);
    if (!sigmoid) s = e * reciprocal(total);
    else s = e < 0x1p1000 ? reciprocal(1.0 + e) : 1.0 / e;
    k = BIAS ? s + by : (double)v;
  }
  // Their exact order: mostly that of the cut keys.
  const int place = id >= 0 ? id : kRouteMaxExperts + l;  // (what is no candidate comes last, in order)
  int rank = l;
  const bool inside = l + 1 < n_cand;
  const double after = dpp<kRowShl1>(k);
  const int place_after = (int)dpp<kRowShl1>((uint32_t)place);
  const bool sorted = !inside || k > after || (k == after && place < place_after);
  // The softmax's sum is an f32 one (a term is off by 2^-23 and 2.6 |x - top|
  // 2^-24 of itself, |x - top| is at most ln 512 on average, the additions give
  // 13 times 2^-24: below 2^-19), and with it all scores by one factor: keys
  // that differ by more of their scores' difference than that stand as they
  // are.  In a sorted row it is enough to look at neighbours.
  constexpr bool soft = ORDER == kBySoftmax;
  auto apart = [](double ka, double sa, double kb, double sb) {
    return (ka == kb && sa == sb) || __builtin_fabs(ka - kb) > __builtin_fabs(sa - sb) * 0x1.1p-19;
  };
  if (__ballot(!sorted)) {
    rank = 0;
    each_lane<0>(n_cand, [&](auto ctrl) {
      constexpr int C = decltype(ctrl)::value;
      const double o = dpp<C>(k);
      const int other = (int)dpp<C>((uint32_t)place);
      rank += (int)(o > k) | ((int)(o == k) & (int)(other < place));
      if (soft) {
        const double so = dpp<C>(s);
        if (id >= 0 && other < kRouteMaxExperts && !apart(k, s, o, so)) ok = false;
      }
    });
  } else if (soft) {
    const double s_after = dpp<kRowShl1>(s);
    if (inside && place_after < kRouteMaxExperts && !apart(k, s, after, s_after)) ok = false;
  }
  // What was not taken is below the last candidate's cut key and a step of it.
  // With a bias its f32 key may be off by 2^-21 (twice a score's 2^-22; of a
  // softmax's largest score, 1 / sum) and a rounding of it, and the softmax's
  // factor moves scores, none above 1 / sum, against one another.
  if (!p.exact_cut) {
    const float hi = from_ordered(mine | low);
    const double err = !BIAS ? 0.0 : (double)__builtin_fabsf(hi) * 0x1p-22 + (soft ? (double)((0x1p-21f + 0x1.2p-19f) * __builtin_amdgcn_rcpf(sum)) : 0x1p-21);
    // (the last candidate's lane asks for the worst of the chosen)
    const double worst = -row16_max(rank < p.topk && id >= 0 ? -k : -__builtin_inf());
    if (l == n_cand - 1 && id >= 0 && !(worst > (double)hi + err)) ok = false;
  }
  if (odd) ok = false;
  const bool chosen = rank < p.topk && id >= 0;
  if (p.renormalize) {
    const double all = row16_sum(chosen ? s : 0.0);
    if (all > 0x1p-1000) s *= reciprocal(all);
    else if (all != 0.0) s /= all;
  }
  const uint64_t bad = __ballot(have && !ok);
  if (have && !((bad >> (lane & 48)) & 0xFFFF)) {
    if (rank < p.topk && l < n_cand) {
      p.ids[t * p.topk + rank] = id;
      p.weights[t * p.topk + rank] = chosen ? (float)(s * p.scale) : 0.0f;
    }
  }
  if (__builtin_expect(bad != 0, 0)) {  // (so that the loop's invariants are formed in here)
#pragma unroll 1
    for (int n = 0; n < 4; ++n)
      if ((bad >> (16 * n)) & 0xFFFF) route_exactly<NB>(p, tw - (lane >> 4) + n, keys[wave]);
  }
}

// Whatever the kernel above does not take: one wave per token.
template <int N>
__global__ __launch_bounds__(256) void route_exact_kernel(const RouteParams p) {
  __shared__ double keys[4][N * 64];
  const int wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t < p.tokens) route_exactly<N>(p, t, keys[wave]);
}

template <typename T, int ORDER, int GROUPS>
static void launch_route(const RouteParams& p, hipStream_t s) {
  // Four waves to a workgroup where the chip is full (16384 tokens, 8 of 128 bf16
  // experts: 4.8 us, with one wave 6.6), one where it is not (1024 tokens: 3.0,
  // with four 3.3); at 4096 tokens they are even (3.4 and 3.2; in groups of 256
  // experts 7.8 and 7.7).
  const int block = p.tokens >= 4096 ? 256 : 64;
  const unsigned grid = (unsigned)((p.tokens * 16 + block - 1) / block);
  switch ((p.experts + 63) / 64) {
    case 1: route_kernel<T, 1, ORDER, GROUPS><<<grid, block, 0, s>>>(p); break;
    case 2: route_kernel<T, 2, ORDER, GROUPS><<<grid, block, 0, s>>>(p); break;
    case 3: route_kernel<T, 3, ORDER, GROUPS><<<grid, block, 0, s>>>(p); break;
    case 4: route_kernel<T, 4, ORDER, GROUPS><<<grid, block, 0, s>>>(p); break;
    case 5:
    case 6: route_kernel<T, 6, ORDER, GROUPS><<<grid, block, 0, s>>>(p); break;
    default: route_kernel<T, 8, ORDER, GROUPS><<<grid, block, 0, s>>>(p); break;
  }
}
template <typename T, int ORDER>
static void launch_route(const RouteParams& p, hipStream_t s) {
  if (p.groups == 1) launch_route<T, ORDER, kNoGroups>(p, s);
  else if (p.per_group % 4 == 0) launch_route<T, ORDER, kQuadGroups>(p, s);
  else launch_route<T, ORDER, kAnyGroups>(p, s);
}
template <typename T>
static void launch_route(const RouteParams& p, hipStream_t s) {
  if (!p.bias) launch_route<T, kByLogit>(p, s);
  else if (p.sigmoid) launch_route<T, kBySigmoid>(p, s);
  else launch_route<T, kBySoftmax>(p, s);
}

}  // namespace hum

using namespace hum;

extern "C" hum_status hum_moe_route(const hum_route_desc* d, int64_t num_tokens, const void* logits, int64_t ld_logits,
                                    const float* bias, int32_t* topk_ids, float* topk_weights, void* stream) {
  clear_error();
  if (!d) return set_error(HUM_ERR_INVALID_ARG, "desc is NULL");
  if (d->logits_dtype != HUM_BF16 && d->logits_dtype != HUM_F32) return set_error(HUM_ERR_UNSUPPORTED, "logits must be bf16 or f32");
  if (d->score != HUM_SCORE_SOFTMAX && d->score != HUM_SCORE_SIGMOID) return set_error(HUM_ERR_INVALID_ARG, "bad score");
  if (d->group_score != HUM_GROUP_MAX && d->group_score != HUM_GROUP_TOP2) return set_error(HUM_ERR_INVALID_ARG, "bad group_score");
  if (d->num_experts < 1 || d->num_experts > kRouteMaxExperts)
    return set_error(HUM_ERR_UNSUPPORTED, "num_experts must be 1 .. %d", kRouteMaxExperts);
  if (d->topk < 1 || d->topk > d->num_experts || d->topk > kRouteMaxTopk)
    return set_error(HUM_ERR_INVALID_ARG, "topk must be 1 .. num_experts, at most %d", kRouteMaxTopk);
  if (d->num_groups < 1 || d->num_groups > 64 || d->num_experts % d->num_groups)
    return set_error(HUM_ERR_INVALID_ARG, "num_groups must divide num_experts, 1 .. 64");
  if (d->topk_groups < 1 || d->topk_groups > d->num_groups) return set_error(HUM_ERR_INVALID_ARG, "topk_groups must be 1 .. num_groups");
  if (d->renormalize != 0 && d->renormalize != 1) return set_error(HUM_ERR_INVALID_ARG, "renormalize must be 0/1");
  if (!std::isfinite(d->scale)) return set_error(HUM_ERR_INVALID_ARG, "scale must be finite");
  if (num_tokens < 0) return set_error(HUM_ERR_INVALID_ARG, "num_tokens must be >= 0");
  // (a grid holds at most 2^32 - 1 threads)
  if (num_tokens >= (int64_t)1 << 24) return set_error(HUM_ERR_UNSUPPORTED, "at most 2^24 - 1 tokens in a call");
  if (num_tokens == 0) return HUM_OK;
  if (!logits || !topk_ids || !topk_weights) return set_error(HUM_ERR_INVALID_ARG, "NULL pointer");
  const int size = d->logits_dtype == HUM_BF16 ? 2 : 4;
  auto addr = [](const void* x) { return reinterpret_cast<uintptr_t>(x); };
  if (addr(logits) % size || (addr(bias) | addr(topk_ids) | addr(topk_weights)) % 4)
    return set_error(HUM_ERR_INVALID_ARG, "tensors must be aligned to their elements");
  const Rows in[2] = {Rows{(int64_t)addr(logits), num_tokens, 1, (wide_t)ld_logits * size, 0, (int64_t)d->num_experts * size},
                      bytes_at(bias, bias ? d->num_experts * 4 : 0)};
  const Rows out[2] = {bytes_at(topk_ids, num_tokens * d->topk * 4), bytes_at(topk_weights, num_tokens * d->topk * 4)};
  if (overlap(out[0], out[1]) != Overlap::kNo) return set_error(HUM_ERR_INVALID_ARG, "topk_ids and topk_weights must not overlap");
  for (const Rows& i : in)
    for (const Rows& o : out)
      if (overlap(o, i) != Overlap::kNo) return set_error(HUM_ERR_INVALID_ARG, "outputs must not overlap the logits or the bias");
  RouteParams p{};
  p.logits = logits;
  p.bias = bias;
  p.ids = topk_ids;
  p.weights = topk_weights;
  p.tokens = num_tokens;
  p.ld = ld_logits;
  p.experts = d->num_experts;
  p.topk = d->topk;
  p.groups = d->topk_groups == d->num_groups ? 1 : d->num_groups;  // (all of them stay: no groups)
  p.topk_groups = d->topk_groups;
  p.per_group = d->num_experts / d->num_groups;
  p.sigmoid = d->score == HUM_SCORE_SIGMOID;
  p.bf16 = size == 2;
  p.top2 = d->group_score == HUM_GROUP_TOP2;
  p.renormalize = d->renormalize;
  p.scale = d->scale;
  const int quad = 4 * size;
  p.vec = addr(logits) % quad == 0 && addr(bias) % 16 == 0 && (num_tokens == 1 || ld_logits % 4 == 0) && d->num_experts % 4 == 0;
  p.exact_cut = size == 2 && !bias;
  p.candidates = d->topk + (p.exact_cut ? 0 : 2);
  int bits = 0;
  while (1 << bits < d->num_experts) ++bits;
  p.low_mask = (1u << bits) - 1u;
  p.inv_group = (p.per_group % 4 == 0 ? 4.0f : 1.0f) / (float)p.per_group;
  hipStream_t s = static_cast<hipStream_t>(stream);
  // The fast kernel holds topk + 2 candidates in 16 lanes, and the groups too.
  if (d->topk <= 14 && p.groups <= 16) {
    if (p.bf16) launch_route<uint16_t>(p, s);
    else launch_route<float>(p, s);
  } else {
    const unsigned grid = (unsigned)((num_tokens + 3) / 4);
    const int blocks = (d->num_experts + 63) / 64;
    if (blocks <= 1) route_exact_kernel<1><<<grid, 256, 0, s>>>(p);
    else if (blocks <= 2) route_exact_kernel<2><<<grid, 256, 0, s>>>(p);
    else if (blocks <= 4) route_exact_kernel<4><<<grid, 256, 0, s>>>(p);
    else route_exact_kernel<8><<<grid, 256, 0, s>>>(p);
  }
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return set_error(HUM_ERR_HIP, "moe_route launch: %s", hipGetErrorString(err));
  return HUM_OK;
}
