// Routing of tokens to experts: scores, groups, the top-k and its weights.
//
//   s_e = softmax(x)_e or 1 / (1 + exp(-x_e)),  order by s_e + bias_e
//   (without a bias by x_e, which orders alike), of the topk_groups best
//   groups only; w = s of the chosen, renormalised, times the scale.
//
// Scores are formed in f64: an expert is chosen by the comparison of two
// scores, and f32 makes near ones equal.
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
  float scale;
};

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) v = fmax(v, __shfl_xor(v, o));
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) v += __shfl_xor(v, o);
  return v;
}

// The largest key of the wave, of equal ones that of the lowest index: every
// lane gets both.
__device__ __forceinline__ void wave_best(double& key, int& idx) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const double k = __shfl_xor(key, o);
    const int i = __shfl_xor(idx, o);
    if (k > key || (k == key && i < idx)) {
      key = k;
      idx = i;
    }
  }
}

// One wave per token; lane l has the experts l, l + 64, ...
__global__ __launch_bounds__(256) void route_kernel(const RouteParams p) {
  constexpr int N = kRouteMaxExperts / 64;
  __shared__ double keys[4][kRouteMaxExperts];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const double none = -__builtin_inf();
  for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < p.tokens; t += (int64_t)gridDim.x * 4) {
    double s[N], key[N];
    double top = none;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = j * 64 + lane;
      key[j] = none;
      if (e < p.experts)
        key[j] = p.bf16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(p.logits)[t * p.ld + e]) : static_cast<const float*>(p.logits)[t * p.ld + e];
      top = fmax(top, key[j]);
    }
    bool by_score = p.bias || (p.groups > 1 && p.top2);
    if (!p.sigmoid) {
      top = wave_max(top);
      double sum = 0.0;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        s[j] = key[j] == none ? 0.0 : exp(key[j] - top);
        sum += s[j];
      }
      sum = wave_sum(sum);
#pragma unroll
      for (int j = 0; j < N; ++j) s[j] = sum == 0.0 ? 0.0 : s[j] / sum;
      by_score = by_score && sum == sum;  // (where a NaN leaves no score, the logits order)
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) s[j] = 1.0 / (1.0 + exp(-key[j]));
    }
    // what the experts are ordered by; a NaN comes first
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = j * 64 + lane;
      if (p.bias && by_score && e < p.experts && key[j] != none) key[j] = s[j] + (double)p.bias[e];
      if (key[j] != key[j]) key[j] = -none;
    }
    if (p.groups > 1) {
      // (one wave's own part of LDS: no other wave reads it)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int e = j * 64 + lane;
        if (e < p.experts) keys[wave][e] = key[j] == none || !by_score || p.bias ? key[j] : s[j] == s[j] ? s[j] : -none;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      // lane g looks at group g (at most 64 of them)
      double a = none, b = none;
      if (lane < p.groups) {
        for (int i = 0; i < p.per_group; ++i) {
          const double v = keys[wave][lane * p.per_group + i];
          if (v > a) {
            b = a;
            a = v;
          } else if (v > b) {
            b = v;
          }
        }
        if (p.top2 && b != none) a += b;
      }
      uint64_t kept = 0;
      for (int n = 0; n < p.topk_groups; ++n) {
        double best = lane < p.groups && !((kept >> lane) & 1) ? a : none;
        int at = lane < p.groups && !((kept >> lane) & 1) ? lane : 64 + lane;
        wave_best(best, at);
        if (at < 64) kept |= 1ull << at;
      }
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int e = j * 64 + lane;
        if (e < p.experts && !((kept >> (e / p.per_group)) & 1)) key[j] = none;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    int id = -1;       // lane n: the n-th choice
    double w = 0.0;
    for (int n = 0; n < p.topk; ++n) {
      double best = none;
      int at = 1 << 20;
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (key[j] > best) {
          best = key[j];
          at = j * 64 + lane;
        }
      wave_best(best, at);
      if (best == none) break;  // nothing is left (the same in every lane)
      double sc = 0.0;
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (j * 64 + lane == at) {
          key[j] = none;
          sc = s[j];
        }
      sc = __shfl(sc, at & 63);
      if (lane == n) {
        id = at;
        w = sc;
      }
    }
    if (p.renormalize) {
      const double sum = wave_sum(w);
      if (sum != 0.0) w /= sum;
    }
    if (lane < p.topk) {
      p.ids[t * p.topk + lane] = id;
      p.weights[t * p.topk + lane] = (float)(w * p.scale);
    }
  }
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
  if (num_tokens >= (int64_t)1 << 31) return set_error(HUM_ERR_UNSUPPORTED, "at most 2^31 - 1 tokens in a call");
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
  const int64_t wgs = (num_tokens + 3) / 4;
  route_kernel<<<(unsigned)(wgs < 1 << 20 ? wgs : 1 << 20), 256, 0, static_cast<hipStream_t>(stream)>>>(p);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return set_error(HUM_ERR_HIP, "moe_route launch: %s", hipGetErrorString(err));
  return HUM_OK;
}
