// The paged key-value cache's layout (the one hum.h documents), shared by
// the kernels that write, read and attend over it.
#pragma once

#include <type_traits>

#include "dev_common.h"
#include "hum_internal.h"

namespace hum {

// Bytes and offsets inside one (page, head) unit.
template <int FMT, int D>
struct KvUnit {
  static constexpr bool kMx = FMT == HUM_ACT_MXFP8 || FMT == HUM_ACT_MXFP4;
  static constexpr int kRow = FMT == HUM_ACT_BF16 ? 2 * D : FMT == HUM_ACT_MXFP4 ? D / 2 : D;  // code bytes of a row
  static constexpr int kScale = FMT == HUM_ACT_FP8_TOKEN ? 4 : kMx ? D / 32 : 0;               // scale bytes of a row
};

// Host side of the same, in bytes.
struct KvLayout {
  int64_t row = 0, scale = 0, unit = 0, bytes = 0;
};

// Checks the description and fills the layout.
hum_status kv_layout(const hum_kv_desc* d, KvLayout* l);

// Calls fn(format, head size), both as integral constants, for a checked
// description.
template <typename F>
void kv_dispatch(const hum_kv_desc* d, F&& fn) {
  auto by_dim = [&](auto fmt) {
    if (d->head_dim == 64) fn(fmt, std::integral_constant<int, 64>{});
    else if (d->head_dim == 128) fn(fmt, std::integral_constant<int, 128>{});
    else fn(fmt, std::integral_constant<int, 256>{});
  };
  switch (d->fmt) {
    case HUM_ACT_BF16: by_dim(std::integral_constant<int, HUM_ACT_BF16>{}); break;
    case HUM_ACT_FP8_TOKEN: by_dim(std::integral_constant<int, HUM_ACT_FP8_TOKEN>{}); break;
    case HUM_ACT_MXFP8: by_dim(std::integral_constant<int, HUM_ACT_MXFP8>{}); break;
    default: by_dim(std::integral_constant<int, HUM_ACT_MXFP4>{}); break;
  }
}

// Eight codes of a row -> eight bf16 (packed pairs), times a power-of-two
// scale: at most four significant bits, so exact where the product lies in
// bf16's range.  What kv_write stores does (its inputs are bf16, multiples of
// 2^-133, and their codes times their scales are so too); other bytes may hold
// products below 2^-133, which are rounded or lost, and past 2^128, which
// become infinite.  w: the codes' 8 (E4M3) or 4 (E2M1) bytes.
__device__ __forceinline__ u32x4_t e4m3x8_to_bf16(u32x2_t w, float scale) {
  u32x4_t o;
  o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], scale, false));
  o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], scale, true));
  o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], scale, false));
  o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], scale, true));
  return o;
}
__device__ __forceinline__ u32x4_t e2m1x8_to_bf16(uint32_t w, float scale) {
  u32x4_t o;
  o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
  o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
  o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
  o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  return o;
}

// Max over the N lanes (8, 16 or 32) that hold one row.
template <int N>
__device__ __forceinline__ float row_max(float v) {
  v = quad_max(v);
  auto with = [&](auto ctrl) {
    v = __builtin_fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, false)));
  };
  with(std::integral_constant<int, 0x141>{});                         // row_half_mirror: the other quad of eight
  if constexpr (N >= 16) with(std::integral_constant<int, 0x140>{});  // row_mirror: the other eight of sixteen
  if constexpr (N >= 32) v = __builtin_fmaxf(v, __shfl_xor(v, 16));
  return v;
}

// Byte offsets of token `at` of a page inside its (page, head) unit: its code
// row, and its scale (or the first of them) with the step to the next.
template <int FMT, int D>
struct KvOffsets {
  int64_t code, scale;
  int32_t scale_step;
  __device__ __forceinline__ KvOffsets(int which, int at, int page_size) {
    using U = KvUnit<FMT, D>;
    code = (int64_t)(which * page_size + at) * U::kRow;
    const int64_t scales = (int64_t)2 * page_size * U::kRow + which * page_size * U::kScale;
    if (U::kMx && which) {
      scale = scales + at;
      scale_step = page_size;
    } else {
      scale = scales + at * U::kScale;
      scale_step = 1;
    }
  }
};

// Quantizes one row, of which the lane has the eight values f, and stores the
// lane's codes at `code` and the row's scale (of the lane's block of 32:
// block b's at b * scale_step) at `scale`, where `live`.  Every lane of the
// row calls it together.  ANY: the values are any f32 (fp8_row says what
// that changes), not bf16.
template <int FMT, int D, bool ANY>
__device__ __forceinline__ void kv_store_row(float (&f)[8], int lane, uint8_t* code, uint8_t* scale, int32_t scale_step, bool live) {
  if constexpr (FMT == HUM_ACT_BF16) {
    u32x4_t o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = f32x2_to_bf16x2_bits(f[2 * i], f[2 * i + 1]);
    if (live) *reinterpret_cast<u32x4_t*>(code) = o;
  } else {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = __builtin_fmaxf(amax, __builtin_fabsf(f[i]));
    if constexpr (FMT == HUM_ACT_FP8_TOKEN) {
      amax = row_max<D / 8>(amax);
      const float sc = fp8_row<ANY>(f, amax);
      u32x2_t o;
      o[0] = f32x2_to_e4m3x2(f[0], f[1]) | (f32x2_to_e4m3x2(f[2], f[3]) << 16);
      o[1] = f32x2_to_e4m3x2(f[4], f[5]) | (f32x2_to_e4m3x2(f[6], f[7]) << 16);
      if (live) {
        *reinterpret_cast<u32x2_t*>(code) = o;
        if (lane == 0) *reinterpret_cast<float*>(scale) = sc;
      }
    } else {
      amax = quad_max(amax);  // four lanes hold one block of 32
      const int e = mx_scale_code_emax(amax, FMT == HUM_ACT_MXFP8 ? 8 : 2);
      const float sc = e8m0_to_f32((uint32_t)e);
      if (live) {
        if constexpr (FMT == HUM_ACT_MXFP8) *reinterpret_cast<u32x2_t*>(code) = mx_e4m3x8(f, sc);
        else *reinterpret_cast<uint32_t*>(code) = mx_e2m1x8(f, sc);
        if ((lane & 3) == 0) scale[(lane >> 2) * scale_step] = (uint8_t)e;
      }
    }
  }
}

}  // namespace hum
