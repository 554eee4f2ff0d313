// Device helpers shared by the gfx950 kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <cstdint>

namespace hum {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
// (16 bytes at an address that is aligned to elements of 2 or 4 only)
typedef u32x4_t u32x4_at2_t __attribute__((aligned(2)));
typedef u32x4_t u32x4_at4_t __attribute__((aligned(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x3_t __attribute__((ext_vector_type(3)));
typedef uint32_t u32x1_t __attribute__((ext_vector_type(1)));
typedef uint32_t u32x6_t __attribute__((ext_vector_type(6)));

__device__ __forceinline__ float bf16_bits_to_f32(uint32_t b16) {
  return __uint_as_float(b16 << 16);
}

// float -> bf16 bits, round to nearest even (NaN kept quiet).
__device__ __forceinline__ uint32_t f32_to_bf16_bits(float f) {
  // the gfx950 conversion instruction (v_cvt_pk_bf16_f32): round to nearest
  // even, a NaN stays a (quiet) NaN
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}

// Two floats -> a packed bf16 pair (a in the low half), one instruction.
__device__ __forceinline__ uint32_t f32x2_to_bf16x2_bits(float a, float b) {
  typedef float f32x2_v __attribute__((ext_vector_type(2)));
  const f32x2_v v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

// E8M0 code -> float 2^(c-127); 255 -> NaN.  Branch free: code 0 is the
// subnormal 2^-127 (mantissa bit 22 alone), code 255 the quiet NaN
// (all-ones exponent and mantissa bit 22).
__device__ __forceinline__ float e8m0_to_f32(uint32_t c) {
  const uint32_t edge = (((c + 1u) & 0xFFu) <= 1u) ? 0x00400000u : 0u;
  return __uint_as_float((c << 23) | edge);
}

// Two floats -> two E4M3 codes (RNE, saturated to +-448, signed zero kept).
// The hardware conversion rounds to nearest even; the clamp makes it
// saturate instead of producing NaN above 448.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float a, float b) {
  a = __builtin_fminf(__builtin_fmaxf(a, -448.0f), 448.0f);
  b = __builtin_fminf(__builtin_fmaxf(b, -448.0f), 448.0f);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false) & 0xFFFFu;
}

// One float -> E2M1 code (nearest, ties to the even code, saturated to +-6,
// sign bit kept for values that round to zero): a comparison against the
// midpoints of the E2M1 grid {0, .5, 1, 1.5, 2, 3, 4, 6}.
__device__ __forceinline__ uint32_t f32_to_e2m1(float v) {
  const float a = __builtin_fabsf(v);
  const uint32_t c = a <= 0.25f ? 0u
                     : a < 0.75f ? 1u
                     : a <= 1.25f ? 2u
                     : a < 1.75f ? 3u
                     : a <= 2.5f ? 4u
                     : a < 3.5f ? 5u
                     : a <= 5.0f ? 6u
                     : 7u;
  return c | ((__float_as_uint(v) >> 28) & 8u);
}

// Sum / max over the 16 lanes of a DPP row (lanes 16r .. 16r+15); every lane
// of the row receives the result.
__device__ __forceinline__ float row16_sum(float v) {
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xF, 0xF, false));  // row_ror:8
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x124, 0xF, 0xF, false));  // row_ror:4
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x122, 0xF, 0xF, false));  // row_ror:2
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x121, 0xF, 0xF, false));  // row_ror:1
  return v;
}

__device__ __forceinline__ float row16_max(float v) {
  v = __builtin_fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xF, 0xF, false)));
  v = __builtin_fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x124, 0xF, 0xF, false)));
  v = __builtin_fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x122, 0xF, 0xF, false)));
  v = __builtin_fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x121, 0xF, 0xF, false)));
  return v;
}

// Max over the 4 lanes of a DPP quad.
__device__ __forceinline__ float quad_max(float v) {
  v = __builtin_fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false)));  // quad_perm 1,0,3,2
  v = __builtin_fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false)));  // quad_perm 2,3,0,1
  return v;
}

// floor(log2(a)) for a finite float a > 0, from the exponent field.
__device__ __forceinline__ int floor_log2_f32(float a) {
  uint32_t u = __float_as_uint(a);
  int e = (int)((u >> 23) & 0xFF);
  if (e == 0) return 31 - __builtin_clz(u & 0x007FFFFFu) - 149;  // subnormal
  return e - 127;
}

// MX scale exponent code for a block whose absolute maximum is `amax`, for
// elements whose largest power of two is 2^emax (E4M3: 8, E2M1: 2).
__device__ __forceinline__ int mx_scale_code_emax(float amax, int emax) {
  if (!(amax > 0.0f)) return 127;
  int e = floor_log2_f32(amax) - emax + 127;
  return e < 0 ? 0 : (e > 254 ? 254 : e);
}
__device__ __forceinline__ int mx_scale_code(float amax) { return mx_scale_code_emax(amax, 8); }

// 2^(127 - e) as an exact float for e in [0, 254] (the reciprocal of the
// MX block scale 2^(e-127)).
__device__ __forceinline__ float mx_inv_scale(int e) {
  int p = 127 - e;  // -127 .. 127
  if (p >= -126) return __uint_as_float((uint32_t)(p + 127) << 23);
  return __uint_as_float(0x00400000u);  // 2^-127
}

// One step towards x / d as an IEEE f32 division rounds it, from an estimate q
// of it and y = RN(1 / d): with the exact remainder r = q d - x, RN(q - r y)
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990).  It is the division's own result where q is within one
// ulp of x / d and nothing over- or underflows.  A zero keeps its sign: r is
// then +0, and q - 0 is q.
__device__ __forceinline__ float divide_step(float q, float x, float d, float y) {
  return __builtin_fmaf(-__builtin_fmaf(q, d, -x), y, q);
}

// A scale by the FP8 rule, amax / 448 (1 for zeros), and values over it, as
// IEEE f32 divisions give them (a code can hang on the quotient's last bit) in
// three or five instructions a value instead of eleven.  Maxima outside
// [2^-70, 2^120] divide; inside, values below 2^-10 of the scale, whose
// remainder may underflow, become zero codes either way.  The reciprocal is
// correctly rounded for every mantissa of a scale, as was the scale itself
// (all 2^23 of each compared).  x y is within 1.5 ulps of x / s, so that after
// one step it is within one and after the second right.  Values and a maximum
// of bf16 need one step: the quotients of all of their mantissas and scales
// were compared with the division's.  ANY: they may be any f32.
__device__ __forceinline__ bool fp8_in_range(float amax) { return amax >= 0x1p-70f && amax <= 0x1p120f; }
template <bool ANY>
__device__ __forceinline__ float fp8_scale_in_range(float amax) {
  const float q = divide_step(amax * (1.0f / 448.0f), amax, 448.0f, 1.0f / 448.0f);
  return ANY ? divide_step(q, amax, 448.0f, 1.0f / 448.0f) : q;
}
template <bool ANY>
__device__ __forceinline__ void fp8_divide_in_range(float (&f)[8], float s) {
  const float y0 = __builtin_amdgcn_rcpf(s);
  const float y = __builtin_fmaf(__builtin_fmaf(-s, y0, 1.0f), y0, y0);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = divide_step(f[i] * y, f[i], s, y);
    f[i] = ANY ? divide_step(q, f[i], s, y) : q;
  }
}
// The scale of a maximum, and the values over it.
template <bool ANY>
__device__ __forceinline__ float fp8_row(float (&f)[8], float amax) {
  float s = 1.0f;
  if (fp8_in_range(amax)) {
    s = fp8_scale_in_range<ANY>(amax);
    fp8_divide_in_range<ANY>(f, s);
  } else if (amax > 0.0f) {  // (lanes without a row hold zeros)
    s = amax / 448.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f[i] / s;
  }
  return s;
}

// Eight floats over a power of two -> eight codes, nearest even, saturated
// (the hardware conversions; E2M1 saturates by itself, E4M3 becomes NaN past
// 448, so what the rule saturates is clamped first).
__device__ __forceinline__ u32x2_t mx_e4m3x8(const float (&f)[8], float scale) {
  typedef short s16x2_v __attribute__((ext_vector_type(2)));
  const float top = 448.0f * scale;
  float c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = __builtin_fminf(__builtin_fmaxf(f[i], -top), top);
  s16x2_v o[2] = {{0, 0}, {0, 0}};
  o[0] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o[0], c[0], c[1], scale, false);
  o[0] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o[0], c[2], c[3], scale, true);
  o[1] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o[1], c[4], c[5], scale, false);
  o[1] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o[1], c[6], c[7], scale, true);
  return u32x2_t{__builtin_bit_cast(uint32_t, o[0]), __builtin_bit_cast(uint32_t, o[1])};
}
__device__ __forceinline__ uint32_t mx_e2m1x8(const float (&f)[8], float scale) {
  uint32_t o = 0;
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, f[0], f[1], scale, 0);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, f[2], f[3], scale, 1);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, f[4], f[5], scale, 2);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, f[6], f[7], scale, 3);
  return o;
}

}  // namespace hum
