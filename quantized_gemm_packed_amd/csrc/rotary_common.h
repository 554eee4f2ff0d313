// The coefficients of a rotary pair, shared by the kernels that turn.
#pragma once

#include "dev_common.h"

namespace hum {

// cos and sin of position * inv_freq times the factor (and sin's sign), each
// rounded once.  The turn count position * inv_freq / 2 pi is formed and
// reduced to [-1/2, 1/2] in f64; the remainder goes to the f32 functions as an
// f32 and the rest of it, to first order.
__device__ __forceinline__ void rotary_coefficients(int64_t position, double inv_freq, float factor, float sign, float* c_out, float* s_out) {
  const double turns = (double)position * (inv_freq * 0.15915494309189535);
  const double rem = turns - __builtin_rint(turns);
  const float r = (float)rem, lo = (float)(rem - r) * 6.28318531f;
  float s, c;
  sincospif(2.0f * r, &s, &c);
  // (each rounded once, the factor included)
  const float fs = factor * sign;
  *c_out = __builtin_fmaf(c, factor, -s * lo * factor);
  *s_out = __builtin_fmaf(s, fs, c * lo * fs);
}

// (the fused product named: every kernel and instance gives the same bits)
__device__ __forceinline__ float rotary_first(float x0, float x1, float c, float s) { return __builtin_fmaf(x0, c, -(x1 * s)); }
__device__ __forceinline__ float rotary_second(float x0, float x1, float c, float s) { return __builtin_fmaf(x0, s, x1 * c); }

}  // namespace hum
