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

}  // namespace hum
