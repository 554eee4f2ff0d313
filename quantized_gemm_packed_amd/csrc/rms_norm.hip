// Root-mean-square norm of rows, with the residual's addition before it and
// the activation quantizer behind it, in one pass:
//   h = x + residual, residual' = round(h),
//   y = h * r * (w + offset),  r = 1 / sqrt(mean(h^2) + eps),
// y in f32, rounded once: to bf16, or to the codes of hum_quant_act's rules.
//
// Memory bound: x and the residual are read once, everything that is written
// is written once.  A row stays in the registers of its waves between the two
// passes over it (the sum of squares, then y), 8 elements of a thread side by
// side; all loads of a row are on their way before the first is used.  Which
// elements a thread has, and so the order of the sums, goes by k alone: a
// row's bits are the same in every batch and at every alignment.
//
// Measured on MI355X, in a captured graph, inputs that change from call to call:
// 16384 rows of 8192 with a bf16 residual to FP8 codes 161 us, 5.8 TB/s read +
// written (a large copy reaches 5.1), to MXFP4 151, to FP8 codes and bf16 with
// f32 weights 212; 3001 rows of 4100 with an f32 residual 29 us, 5.1 TB/s; 256
// rows of 7168 to FP8 codes in groups 5.0 us and one row of 4096 3.3 us, of
// which an empty launch is 1.9.  Rows past 16384 elements: 3.9 to 4.3 TB/s.
#include <cmath>

#include "dev_common.h"
#include "hum_internal.h"
#include "rows.h"

namespace hum {

struct NormParams {
  const uint16_t* x;
  const void* res;
  void* res_out;
  const void* w;
  uint16_t* out;
  uint8_t* q;
  void* scales;
  int64_t m, ld_x, ld_res, ld_res_out, ld_out;
  int32_t k;
  int32_t w_f32;
  float inv_k, eps, offset;
};

// What a row's residual is.
enum { kNoRes = 0, kResBf16 = 1, kResF32 = 2 };

__device__ __forceinline__ float norm_ld(uint16_t v) { return bf16_bits_to_f32(v); }
__device__ __forceinline__ float norm_ld(float v) { return v; }

// Eight elements of a row as they lie in memory: 16 bytes of bf16, 32 of f32.
template <typename T>
struct Raw {
  static constexpr int kWords = sizeof(T) * 2;
  uint32_t w[kWords];
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 2) f[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
      else f[i] = __uint_as_float(w[i]);
    }
  }
  __device__ __forceinline__ void pack(const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 2) w[i] = f32x2_to_bf16x2_bits(f[2 * i], f[2 * i + 1]);
      else w[i] = __float_as_uint(f[i]);
    }
  }
};

// Its loads and stores at `at`, where all eight lie within k (else zeros): 16
// bytes each, which FAST says are aligned.  Otherwise they are aligned to
// their elements, which the vector memory takes at any width.
template <typename T, bool FAST>
__device__ __forceinline__ Raw<T> load8(const T* row, int at, int k) {
  using V = std::conditional_t<FAST, u32x4_t, std::conditional_t<sizeof(T) == 2, u32x4_at2_t, u32x4_at4_t>>;
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < Raw<T>::kWords; ++i) r.w[i] = 0;
  if (at + 8 <= k) {
#pragma unroll
    for (int i = 0; i < Raw<T>::kWords; i += 4) {
      const u32x4_t v = *reinterpret_cast<const V*>(row + at + i * 4 / (int)sizeof(T));
#pragma unroll
      for (int e = 0; e < 4; ++e) r.w[i + e] = v[e];
    }
  }
  return r;
}
template <typename T, bool FAST>
__device__ __forceinline__ void store8(T* row, int at, int k, const float (&f)[8]) {
  using V = std::conditional_t<FAST, u32x4_t, std::conditional_t<sizeof(T) == 2, u32x4_at2_t, u32x4_at4_t>>;
  Raw<T> r;
  r.pack(f);
  if (at + 8 <= k) {
#pragma unroll
    for (int i = 0; i < Raw<T>::kWords; i += 4)
      *reinterpret_cast<V*>(row + at + i * 4 / (int)sizeof(T)) = u32x4_t{r.w[i], r.w[i + 1], r.w[i + 2], r.w[i + 3]};
  }
}

// Sum / max over the row: the wave's lanes, then the WAVES waves in order.
template <int WAVES, bool MAX>
__device__ __forceinline__ float over_row(float v, float* red) {
  auto join = [](float a, float b) { return MAX ? __builtin_fmaxf(a, b) : a + b; };
  v = MAX ? row16_max(v) : row16_sum(v);
  v = join(v, __shfl_xor(v, 16));
  v = join(v, __shfl_xor(v, 32));
  if constexpr (WAVES > 1) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) v = join(v, red[i]);
  }
  return v;
}

__device__ __forceinline__ u32x2_t e4m3x8(const float (&f)[8]) {
  return u32x2_t{f32x2_to_e4m3x2(f[0], f[1]) | (f32x2_to_e4m3x2(f[2], f[3]) << 16),
                 f32x2_to_e4m3x2(f[4], f[5]) | (f32x2_to_e4m3x2(f[6], f[7]) << 16)};
}
// The largest magnitude of eight; infinity where one is a NaN (the maximum
// that keeps NaNs takes as many instructions as the one that drops them).
__device__ __forceinline__ float max8(const float (&f)[8]) {
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = __builtin_elementwise_maximum(a, __builtin_fabsf(f[i]));
  return a == a ? a : __builtin_inff();
}

// WAVES waves have a row (one: a workgroup has four rows), NV pieces of 8
// elements each thread.
template <int FMT, int RES, bool FAST, int WAVES, int NV>
__global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) void norm_kernel(const NormParams p) {
  constexpr int kLanes = WAVES * 64;
  __shared__ float red[2][2][WAVES];
  const int lane = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int rows = WAVES == 1 ? 4 : 1;
  const int k = p.k;
  constexpr bool kLast = FMT == HUM_ACT_BF16 && !FAST;  // (codes have whole pieces only)
  int turn = 0;  // (the rows' exchanges alternate between two places: one barrier each)
  for (int64_t row = (int64_t)blockIdx.x * rows + (WAVES == 1 ? threadIdx.x >> 6 : 0); row < p.m;
       row += (int64_t)gridDim.x * rows, turn ^= 1) {
    using ResT = std::conditional_t<RES == kResF32, float, uint16_t>;
    // (long rows in parts: all of their loads at once would not fit the registers)
    constexpr int kPart = NV > 4 ? 2 : NV;
    float h[NV][8];
    float sum = 0.0f;
    // the last k % 8 elements: one each of the first threads
    const int last = (k & ~7) + lane;
    const bool has_last = kLast && last < k;
    float h_last = 0.0f;
    if (has_last) {
      h_last = norm_ld(p.x[row * p.ld_x + last]);
      if constexpr (RES != kNoRes) {
        h_last += norm_ld(static_cast<const ResT*>(p.res)[row * p.ld_res + last]);
        if constexpr (RES == kResF32) static_cast<float*>(p.res_out)[row * p.ld_res_out + last] = h_last;
        else static_cast<uint16_t*>(p.res_out)[row * p.ld_res_out + last] = (uint16_t)f32_to_bf16_bits(h_last);
      }
      sum = h_last * h_last;
    }
#pragma unroll
    for (int part = 0; part < NV; part += kPart) {
      Raw<uint16_t> xr[NV];
      Raw<ResT> rr[NV];
#pragma unroll
      for (int j = part; j < part + kPart; ++j) {
        xr[j] = load8<uint16_t, FAST>(p.x + row * p.ld_x, (j * kLanes + lane) * 8, k);
        if constexpr (RES != kNoRes) rr[j] = load8<ResT, FAST>(static_cast<const ResT*>(p.res) + row * p.ld_res, (j * kLanes + lane) * 8, k);
      }
#pragma unroll
      for (int j = part; j < part + kPart; ++j) {
        xr[j].unpack(h[j]);
        if constexpr (RES != kNoRes) {
          float b[8];
          rr[j].unpack(b);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[j][i] += b[i];
          store8<ResT, FAST>(static_cast<ResT*>(p.res_out) + row * p.ld_res_out, (j * kLanes + lane) * 8, k, h[j]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(h[j][i], h[j][i], sum);
      }
      if constexpr (kPart < NV) __builtin_amdgcn_sched_barrier(0);
    }
    sum = over_row<WAVES, false>(sum, red[0][turn]);
    const float r = 1.0f / __builtin_sqrtf(sum * p.inv_k + p.eps);
    // Codes hold no infinity and no NaN, so a scale of NaN shows them: in all of
    // a row whose squares have no finite sum, and where y alone is not finite
    // (by its weight), `amax` infinite then.
    auto fine = [&](float amax) { return sum < __builtin_inff() && amax < __builtin_inff(); };
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int at = (j * kLanes + lane) * 8;
      if constexpr (kPart < NV) __builtin_amdgcn_sched_barrier(0);
      float w[8];
      if (p.w_f32) load8<float, FAST>(static_cast<const float*>(p.w), at, k).unpack(w);
      else load8<uint16_t, FAST>(static_cast<const uint16_t*>(p.w), at, k).unpack(w);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] = h[j][i] * r * (w[i] + p.offset);
      if (p.out) store8<uint16_t, FAST>(p.out + row * p.ld_out, at, k, h[j]);
      if constexpr (FMT == HUM_ACT_FP8_TOKEN) amax = __builtin_fmaxf(amax, max8(h[j]));
    }
    if (has_last) {
      const float w = p.w_f32 ? static_cast<const float*>(p.w)[last] : norm_ld(static_cast<const uint16_t*>(p.w)[last]);
      p.out[row * p.ld_out + last] = (uint16_t)f32_to_bf16_bits(h_last * r * (w + p.offset));
    }
    if constexpr (FMT == HUM_ACT_FP8_TOKEN) {
      amax = over_row<WAVES, true>(amax, red[1][turn]);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int at = (j * kLanes + lane) * 8;
        const float s = fp8_row<true>(h[j], amax);
        if (j == 0 && lane == 0) static_cast<float*>(p.scales)[row] = fine(amax) ? s : __builtin_nanf("");
        if (at < k) *reinterpret_cast<u32x2_t*>(p.q + row * k + at) = e4m3x8(h[j]);
      }
    }
    if constexpr (FMT == HUM_ACT_FP8_GROUP) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int at = (j * kLanes + lane) * 8;
        amax = row16_max(max8(h[j]));  // 16 lanes have a group of 128
        const float s = fp8_row<true>(h[j], amax);
        if (at < k) {
          *reinterpret_cast<u32x2_t*>(p.q + row * k + at) = e4m3x8(h[j]);
          if ((lane & 15) == 0) static_cast<float*>(p.scales)[row * (k / 128) + at / 128] = fine(amax) ? s : __builtin_nanf("");
        }
      }
    }
    if constexpr (FMT == HUM_ACT_MXFP8 || FMT == HUM_ACT_MXFP4) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int at = (j * kLanes + lane) * 8;
        amax = quad_max(max8(h[j]));  // 4 lanes have a block of 32
        const int e = mx_scale_code_emax(amax, FMT == HUM_ACT_MXFP8 ? 8 : 2);
        if (at >= k) continue;
        const float sc = e8m0_to_f32((uint32_t)e);
        if constexpr (FMT == HUM_ACT_MXFP8) *reinterpret_cast<u32x2_t*>(p.q + row * k + at) = mx_e4m3x8(h[j], sc);
        else *reinterpret_cast<uint32_t*>(p.q + (row * k + at) / 2) = mx_e2m1x8(h[j], sc);
        if ((lane & 3) == 0) static_cast<uint8_t*>(p.scales)[row * (k / 32) + at / 32] = fine(amax) ? (uint8_t)e : 255;
      }
    }
  }
}

// Waves per row and pieces per thread, by the row's length alone.  Measured
// (waves x pieces; bf16 residual, FP8 codes, 2^26 elements, and one row):
//   512   1x1 97 us, 3.6     2x1 124, 3.2
//   1024  2x1 87, 3.3        1x2 87, 3.4      4x1 122, 3.3
//   2048  2x2 86, 3.8        4x1 89, 3.4      1x4 95, 4.5
//   4096  4x2 86, 3.9        8x1 89, 3.9      2x4 95, 4.9
//   5120  4x3 91, 4.4        8x2 94, 4.2
//   8192  8x2 87, 4.5        4x4 96, 5.1      16x1 95, 4.7
//   12288 8x3 91, 5.3        16x2 94, 5.4
//   16384 16x2 96, 6.1       8x4 101, 6.4
// (and in a captured graph:)
//   20480 16x4 115, 7.0      8x8 132, 8.0
//   32768 16x4 110, 7.5      8x8 118, 8.9
//   65536 16x8 121, 12.4     (the only one that holds it; 4 to 26 registers spill)
template <int FMT, int RES, bool FAST>
static void launch_norm(const NormParams& p, hipStream_t s) {
  auto go = [&](auto waves, auto nv) {
    constexpr int W = decltype(waves)::value;
    const int64_t wgs = W == 1 ? (p.m + 3) / 4 : p.m;
    const int64_t most = (int64_t)1 << 20;
    norm_kernel<FMT, RES, FAST, W, decltype(nv)::value><<<(unsigned)(wgs < most ? wgs : most), W == 1 ? 256 : W * 64, 0, s>>>(p);
  };
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I3 = std::integral_constant<int, 3>;
  using I4 = std::integral_constant<int, 4>;
  using I8 = std::integral_constant<int, 8>;
  using I16 = std::integral_constant<int, 16>;
  if (p.k <= 512) go(I1{}, I1{});
  else if (p.k <= 1024) go(I2{}, I1{});
  else if (p.k <= 2048) go(I2{}, I2{});
  else if (p.k <= 4096) go(I4{}, I2{});
  else if (p.k <= 6144) go(I4{}, I3{});
  else if (p.k <= 8192) go(I8{}, I2{});
  else if (p.k <= 12288) go(I8{}, I3{});
  else if (p.k <= 16384) go(I16{}, I2{});
  else if (p.k <= 32768) go(I16{}, I4{});
  else go(I16{}, I8{});
}

constexpr int64_t kNormMaxK = 65536;

}  // namespace hum

using namespace hum;

extern "C" hum_status hum_rms_norm(const hum_norm_desc* d, int64_t m, int64_t k, const void* x, int64_t ld_x,
                                   const void* residual, int64_t ld_res, void* residual_out, int64_t ld_res_out,
                                   const void* weight, void* out, int64_t ld_out, void* q, void* scales, void* stream) {
  clear_error();
  if (!d) return set_error(HUM_ERR_INVALID_ARG, "desc is NULL");
  const int32_t fmt = d->act_fmt;
  if (fmt < HUM_ACT_BF16 || fmt > HUM_ACT_FP8_GROUP) return set_error(HUM_ERR_INVALID_ARG, "bad act_fmt");
  if (d->residual_dtype != HUM_BF16 && d->residual_dtype != HUM_F32)
    return set_error(HUM_ERR_UNSUPPORTED, "residual_dtype must be bf16 or f32");
  if (d->weight_dtype != HUM_BF16 && d->weight_dtype != HUM_F32)
    return set_error(HUM_ERR_UNSUPPORTED, "weight_dtype must be bf16 or f32");
  if (!(d->eps > 0.0f) || !std::isfinite(d->eps)) return set_error(HUM_ERR_INVALID_ARG, "eps must be a number above 0");
  if (!std::isfinite(d->weight_offset)) return set_error(HUM_ERR_INVALID_ARG, "weight_offset must be finite");
  if (m < 0 || k < 1) return set_error(HUM_ERR_INVALID_ARG, "m must be >= 0 and k >= 1");
  if (k > kNormMaxK) return set_error(HUM_ERR_UNSUPPORTED, "k must be at most %lld", (long long)kNormMaxK);
  const int unit = fmt == HUM_ACT_FP8_TOKEN ? 8 : fmt == HUM_ACT_FP8_GROUP ? 128 : fmt == HUM_ACT_BF16 ? 1 : 32;
  if (k % unit) return set_error(HUM_ERR_UNSUPPORTED, "k must be a multiple of %d for this format", unit);
  if (m >= (int64_t)1 << 40) return set_error(HUM_ERR_UNSUPPORTED, "at most 2^40 - 1 rows in a call");
  if (m == 0) return HUM_OK;
  const bool quant = fmt != HUM_ACT_BF16;
  if (quant != (q != nullptr) || quant != (scales != nullptr))
    return set_error(HUM_ERR_INVALID_ARG, quant ? "q and scales must be given for this format" : "q and scales must be NULL for bf16");
  if (!quant && !out) return set_error(HUM_ERR_INVALID_ARG, "out must be given for bf16");
  if ((residual != nullptr) != (residual_out != nullptr))
    return set_error(HUM_ERR_INVALID_ARG, "residual and residual_out go together");
  if (!x || !weight) return set_error(HUM_ERR_INVALID_ARG, "NULL pointer");
  const int rsize = d->residual_dtype == HUM_BF16 ? 2 : 4, wsize = d->weight_dtype == HUM_BF16 ? 2 : 4;
  auto addr = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  const int ssize = fmt == HUM_ACT_MXFP8 || fmt == HUM_ACT_MXFP4 ? 1 : 4;
  if (addr(x) % 2 || addr(out) % 2 || addr(weight) % wsize || (addr(residual) | addr(residual_out)) % rsize || addr(scales) % ssize)
    return set_error(HUM_ERR_INVALID_ARG, "tensors must be aligned to their elements");
  if (addr(q) % 8) return set_error(HUM_ERR_INVALID_ARG, "q must be 8-byte aligned");
  // What workgroups store while others read: no output may lie in an input or
  // another output, but for whole rows in place (a thread stores what it has
  // read itself).
  auto extent = [&](const void* at, int64_t ld, int64_t row_bytes, int size) {
    return Rows{(int64_t)(intptr_t)at, m, 1, (wide_t)ld * size, 0, row_bytes};
  };
  struct Part {
    const char* name;
    Rows at;
    bool output;
    int64_t ld;
    int size;
  };
  Part parts[7];
  int n = 0;
  auto add = [&](const char* name, const void* p, int64_t ld, int size, bool output) {
    if (p) parts[n++] = Part{name, extent(p, ld, k * size, size), output, ld, size};
  };
  add("x", x, ld_x, 2, false);
  add("residual", residual, ld_res, rsize, false);
  add("residual_out", residual_out, ld_res_out, rsize, true);
  add("out", out, ld_out, 2, true);
  parts[n++] = Part{"weight", bytes_at(weight, k * wsize), false, 0, 0};
  if (quant) {
    const int64_t qrow = fmt == HUM_ACT_MXFP4 ? k / 2 : k;
    const int64_t srow = fmt == HUM_ACT_FP8_TOKEN ? 4 : fmt == HUM_ACT_FP8_GROUP ? k / 128 * 4 : k / 32;
    parts[n++] = Part{"q", bytes_at(q, m * qrow), true, 0, 0};
    parts[n++] = Part{"scales", bytes_at(scales, m * srow), true, 0, 0};
  }
  for (int i = 0; i < n; ++i) {
    if (!parts[i].output) continue;
    if (overlaps_itself(parts[i].at)) return set_error(HUM_ERR_INVALID_ARG, "the rows of %s must not overlap", parts[i].name);
    for (int j = 0; j < n; ++j) {
      if (j == i || (parts[j].output && j > i)) continue;
      const bool in_place = !parts[j].output && parts[i].size && parts[i].size == parts[j].size && parts[i].at.at == parts[j].at.at &&
                            (parts[i].ld == parts[j].ld || m == 1);
      if (!in_place && overlap(parts[i].at, parts[j].at) != Overlap::kNo)
        return set_error(HUM_ERR_INVALID_ARG, "%s and %s must not overlap", parts[i].name, parts[j].name);
    }
  }
  NormParams p{};
  p.x = static_cast<const uint16_t*>(x);
  p.res = residual;
  p.res_out = residual_out;
  p.w = weight;
  p.out = static_cast<uint16_t*>(out);
  p.q = static_cast<uint8_t*>(q);
  p.scales = scales;
  p.m = m;
  p.k = (int32_t)k;
  p.ld_x = ld_x;
  p.ld_res = ld_res;
  p.ld_res_out = ld_res_out;
  p.ld_out = ld_out;
  p.w_f32 = wsize == 4;
  p.inv_k = (float)(1.0 / (double)k);
  p.eps = d->eps;
  p.offset = d->weight_offset;
  // Whether every piece of 8 elements is whole and 16-byte aligned.
  uintptr_t all = addr(x) | addr(out) | addr(weight) | addr(residual) | addr(residual_out);
  if (m > 1) {
    all |= (uintptr_t)(ld_x * 2) | (out ? (uintptr_t)(ld_out * 2) : 0);
    if (residual) all |= (uintptr_t)(ld_res * rsize) | (uintptr_t)(ld_res_out * rsize);
  }
  const bool fast = k % 8 == 0 && all % 16 == 0;
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto by_res = [&](auto f) {
    constexpr int F = decltype(f)::value;
    auto by_fast = [&](auto res) {
      constexpr int R = decltype(res)::value;
      if (fast) launch_norm<F, R, true>(p, s);
      else launch_norm<F, R, false>(p, s);
    };
    if (!residual) by_fast(std::integral_constant<int, kNoRes>{});
    else if (rsize == 2) by_fast(std::integral_constant<int, kResBf16>{});
    else by_fast(std::integral_constant<int, kResF32>{});
  };
  switch (fmt) {
    case HUM_ACT_BF16: by_res(std::integral_constant<int, HUM_ACT_BF16>{}); break;
    case HUM_ACT_FP8_TOKEN: by_res(std::integral_constant<int, HUM_ACT_FP8_TOKEN>{}); break;
    case HUM_ACT_MXFP8: by_res(std::integral_constant<int, HUM_ACT_MXFP8>{}); break;
    case HUM_ACT_MXFP4: by_res(std::integral_constant<int, HUM_ACT_MXFP4>{}); break;
    default: by_res(std::integral_constant<int, HUM_ACT_FP8_GROUP>{}); break;
  }
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return set_error(HUM_ERR_HIP, "rms_norm launch: %s", hipGetErrorString(err));
  return HUM_OK;
}
