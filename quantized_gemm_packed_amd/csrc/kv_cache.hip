// Paged key-value cache: quantising rows as they are written, reading them
// back.
//
// A row (one token's K or V of one head) is quantized by the rules of
// hum_quant_act: FP8 with one f32 scale per row (amax / 448), or MXFP8 /
// MXFP4 with one E8M0 scale per 32.  D / 8 neighbouring lanes hold one row,
// 16 bytes of bf16 each; the maximum is a shuffle inside them (a DPP quad
// for an MX block), so nothing goes through LDS.  Memory bound: each row is
// read once and its codes written once.
#include "kv_common.h"

namespace hum {

struct KvMoveParams {
  uint8_t* cache;
  int64_t unit;       // bytes of a (page, head) unit
  int64_t slots_all;  // num_pages * page_size
  int32_t heads, page_shift;
  int64_t tokens;
  const int64_t* slots;
  const uint16_t* x[2];  // write: k, v
  int64_t ts[2], hs[2];
  uint16_t* out[2];  // read: k, v, contiguous
};

// A lane's place: which row (token, K or V, head) and which 8 of its values.
template <int D>
struct KvPlace {
  int64_t token;
  int32_t which, head, lane;
  bool valid;
  __device__ __forceinline__ KvPlace(const KvMoveParams& p) {
    constexpr int kLanes = D / 8;
    const int64_t rows = p.tokens * 2 * p.heads;
    const int64_t row = (int64_t)blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
    lane = threadIdx.x % kLanes;
    valid = row < rows;
    const int64_t r = valid ? row : 0;
    token = r / (2 * p.heads);
    const int32_t rest = (int32_t)(r - token * 2 * p.heads);
    which = rest >= p.heads;
    head = rest - which * p.heads;
  }
};

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

template <int FMT, int D, bool VEC>
__global__ __launch_bounds__(256) void kv_write_kernel(const KvMoveParams p) {
  using U = KvUnit<FMT, D>;
  constexpr int kLanes = D / 8;
  const KvPlace<D> me(p);
  const int64_t slot = me.valid ? p.slots[me.token] : -1;
  // (unsigned: negative slots are past the end too; a row's lanes agree)
  const bool live = (uint64_t)slot < (uint64_t)p.slots_all;
  u32x4_t v = {0, 0, 0, 0};
  if (live) {
    const uint16_t* x = p.x[me.which] + me.token * p.ts[me.which] + me.head * p.hs[me.which] + me.lane * 8;
    if constexpr (VEC) {
      v = *reinterpret_cast<const u32x4_t*>(x);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = (uint32_t)x[2 * i] | ((uint32_t)x[2 * i + 1] << 16);
    }
  }
  const int64_t page = slot >> p.page_shift;
  const int page_size = 1 << p.page_shift;
  const KvOffsets<FMT, D> off(me.which, (int)(slot & (page_size - 1)), page_size);
  uint8_t* unit = p.cache + (live ? page * p.heads + me.head : 0) * p.unit;
  if constexpr (FMT == HUM_ACT_BF16) {
    if (live) *reinterpret_cast<u32x4_t*>(unit + off.code + me.lane * 16) = v;
  } else {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_bits_to_f32(v[i] & 0xFFFF);
      f[2 * i + 1] = bf16_bits_to_f32(v[i] >> 16);
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = __builtin_fmaxf(amax, __builtin_fabsf(f[i]));
    if constexpr (FMT == HUM_ACT_FP8_TOKEN) {
#pragma unroll
      for (int m = 1; m < kLanes; m *= 2) amax = __builtin_fmaxf(amax, __shfl_xor(amax, m));
      const float sc = amax > 0.0f ? amax / 448.0f : 1.0f;  // IEEE f32 division
      if (!live) return;
      u32x2_t o;
      o[0] = f32x2_to_e4m3x2(f[0] / sc, f[1] / sc) | (f32x2_to_e4m3x2(f[2] / sc, f[3] / sc) << 16);
      o[1] = f32x2_to_e4m3x2(f[4] / sc, f[5] / sc) | (f32x2_to_e4m3x2(f[6] / sc, f[7] / sc) << 16);
      *reinterpret_cast<u32x2_t*>(unit + off.code + me.lane * 8) = o;
      if (me.lane == 0) *reinterpret_cast<float*>(unit + off.scale) = sc;
    } else {
      amax = quad_max(amax);  // four lanes hold one block of 32
      const int e = mx_scale_code_emax(amax, FMT == HUM_ACT_MXFP8 ? 8 : 2);
      const float inv = mx_inv_scale(e);
      if (!live) return;
      if constexpr (FMT == HUM_ACT_MXFP8) {
        u32x2_t o;
        o[0] = f32x2_to_e4m3x2(f[0] * inv, f[1] * inv) | (f32x2_to_e4m3x2(f[2] * inv, f[3] * inv) << 16);
        o[1] = f32x2_to_e4m3x2(f[4] * inv, f[5] * inv) | (f32x2_to_e4m3x2(f[6] * inv, f[7] * inv) << 16);
        *reinterpret_cast<u32x2_t*>(unit + off.code + me.lane * 8) = o;
      } else {
        uint32_t o = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) o |= f32_to_e2m1(f[i] * inv) << (4 * i);
        *reinterpret_cast<uint32_t*>(unit + off.code + me.lane * 4) = o;
      }
      if ((me.lane & 3) == 0) unit[off.scale + (me.lane >> 2) * off.scale_step] = (uint8_t)e;
    }
  }
}

template <int FMT, int D>
__global__ __launch_bounds__(256) void kv_read_kernel(const KvMoveParams p) {
  const KvPlace<D> me(p);
  if (!me.valid) return;
  const int64_t slot = p.slots[me.token];
  u32x4_t o = {0, 0, 0, 0};
  if ((uint64_t)slot < (uint64_t)p.slots_all) {
    const int64_t page = slot >> p.page_shift;
    const int page_size = 1 << p.page_shift;
    const KvOffsets<FMT, D> off(me.which, (int)(slot & (page_size - 1)), page_size);
    const uint8_t* unit = p.cache + (page * p.heads + me.head) * p.unit;
    if constexpr (FMT == HUM_ACT_BF16) {
      o = *reinterpret_cast<const u32x4_t*>(unit + off.code + me.lane * 16);
    } else {
      // codes as exact bf16, then one f32 product with the scale, rounded once
      float sc;
      if constexpr (FMT == HUM_ACT_FP8_TOKEN) sc = *reinterpret_cast<const float*>(unit + off.scale);
      else sc = e8m0_to_f32(unit[off.scale + (me.lane >> 2) * off.scale_step]);
      if constexpr (FMT == HUM_ACT_MXFP4)
        o = e2m1x8_to_bf16(*reinterpret_cast<const uint32_t*>(unit + off.code + me.lane * 4), 1.0f);
      else
        o = e4m3x8_to_bf16(*reinterpret_cast<const u32x2_t*>(unit + off.code + me.lane * 8), 1.0f);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = f32x2_to_bf16x2_bits(bf16_bits_to_f32(o[i] & 0xFFFF) * sc, bf16_bits_to_f32(o[i] >> 16) * sc);
    }
  }
  *reinterpret_cast<u32x4_t*>(p.out[me.which] + (me.token * p.heads + me.head) * D + me.lane * 8) = o;
}

hum_status kv_layout(const hum_kv_desc* d, KvLayout* l) {
  if (!d) return set_error(HUM_ERR_INVALID_ARG, "desc is NULL");
  if (d->fmt != HUM_ACT_BF16 && d->fmt != HUM_ACT_FP8_TOKEN && d->fmt != HUM_ACT_MXFP8 && d->fmt != HUM_ACT_MXFP4)
    return set_error(HUM_ERR_UNSUPPORTED, "the cache holds bf16, FP8_TOKEN, MXFP8 or MXFP4 rows");
  if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256)
    return set_error(HUM_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256 (got %d)", d->head_dim);
  if (d->page_size < 16 || d->page_size > 256 || (d->page_size & (d->page_size - 1)))
    return set_error(HUM_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256 (got %d)", d->page_size);
  if (d->num_kv_heads < 1 || d->num_kv_heads > 1024)
    return set_error(HUM_ERR_INVALID_ARG, "num_kv_heads must be 1 .. 1024");
  if (d->num_pages < 1 || d->num_pages > (int64_t)0x7FFFFFFF)
    return set_error(HUM_ERR_INVALID_ARG, "num_pages must be 1 .. 2^31 - 1");
  const bool mx = d->fmt == HUM_ACT_MXFP8 || d->fmt == HUM_ACT_MXFP4;
  l->row = d->fmt == HUM_ACT_BF16 ? 2 * d->head_dim : d->fmt == HUM_ACT_MXFP4 ? d->head_dim / 2 : d->head_dim;
  l->scale = d->fmt == HUM_ACT_FP8_TOKEN ? 4 : mx ? d->head_dim / 32 : 0;
  l->unit = 2 * d->page_size * (l->row + l->scale);
  l->bytes = d->num_pages * d->num_kv_heads * l->unit;
  return HUM_OK;
}

static hum_status kv_move_params(const hum_kv_desc* d, const void* cache, size_t cache_bytes, int64_t num_tokens,
                                 const int64_t* slots, KvMoveParams* p) {
  KvLayout l;
  hum_status st = kv_layout(d, &l);
  if (st != HUM_OK) return st;
  if (num_tokens < 0) return set_error(HUM_ERR_INVALID_ARG, "num_tokens must be >= 0");
  if (num_tokens == 0) return HUM_OK;
  if (!cache || !slots) return set_error(HUM_ERR_INVALID_ARG, "NULL pointer");
  if (reinterpret_cast<uintptr_t>(cache) % 16) return set_error(HUM_ERR_INVALID_ARG, "the cache must be 16-byte aligned");
  if (cache_bytes < (size_t)l.bytes)
    return set_error(HUM_ERR_WORKSPACE, "cache of %zu bytes, the description takes %lld", cache_bytes, (long long)l.bytes);
  // (a grid holds at most 2^32 - 1 threads, D / 8 of them a row)
  if (num_tokens > ((int64_t)1 << 32) / (2 * d->num_kv_heads * (d->head_dim / 8)) - 256)
    return set_error(HUM_ERR_UNSUPPORTED, "too many tokens for one call");
  p->cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  p->unit = l.unit;
  p->slots_all = d->num_pages * d->page_size;
  p->heads = d->num_kv_heads;
  p->page_shift = __builtin_ctz((unsigned)d->page_size);
  p->tokens = num_tokens;
  p->slots = slots;
  return HUM_OK;
}

static unsigned kv_move_grid(const hum_kv_desc* d, int64_t num_tokens) {
  const int64_t rows = num_tokens * 2 * d->num_kv_heads, per = 256 / (d->head_dim / 8);
  return (unsigned)((rows + per - 1) / per);
}

}  // namespace hum

using namespace hum;

extern "C" {

size_t hum_kv_cache_bytes(const hum_kv_desc* desc) {
  clear_error();
  KvLayout l;
  return kv_layout(desc, &l) == HUM_OK ? (size_t)l.bytes : 0;
}

hum_status hum_kv_write(const hum_kv_desc* desc, void* cache, size_t cache_bytes, int64_t num_tokens,
                        const int64_t* slots, const void* k_bf16, int64_t k_ts, int64_t k_hs, const void* v_bf16,
                        int64_t v_ts, int64_t v_hs, void* stream) {
  clear_error();
  KvMoveParams p{};
  hum_status st = kv_move_params(desc, cache, cache_bytes, num_tokens, slots, &p);
  if (st != HUM_OK || num_tokens == 0) return st;
  if (!k_bf16 || !v_bf16) return set_error(HUM_ERR_INVALID_ARG, "NULL pointer");
  const uintptr_t at = reinterpret_cast<uintptr_t>(k_bf16) | reinterpret_cast<uintptr_t>(v_bf16);
  if (at % 2) return set_error(HUM_ERR_INVALID_ARG, "k and v must be aligned to their elements");
  p.x[0] = static_cast<const uint16_t*>(k_bf16);
  p.x[1] = static_cast<const uint16_t*>(v_bf16);
  p.ts[0] = k_ts;
  p.ts[1] = v_ts;
  p.hs[0] = k_hs;
  p.hs[1] = v_hs;
  const bool vec = at % 16 == 0 && (k_ts | k_hs | v_ts | v_hs) % 8 == 0;
  const unsigned grid = kv_move_grid(desc, num_tokens);
  hipStream_t s = static_cast<hipStream_t>(stream);
  kv_dispatch(desc, [&](auto fmt, auto dim) {
    constexpr int F = decltype(fmt)::value, D = decltype(dim)::value;
    if (vec) kv_write_kernel<F, D, true><<<grid, 256, 0, s>>>(p);
    else kv_write_kernel<F, D, false><<<grid, 256, 0, s>>>(p);
  });
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return set_error(HUM_ERR_HIP, "kv_write launch: %s", hipGetErrorString(err));
  return HUM_OK;
}

hum_status hum_kv_read(const hum_kv_desc* desc, const void* cache, size_t cache_bytes, int64_t num_tokens,
                       const int64_t* slots, void* k_out, void* v_out, void* stream) {
  clear_error();
  KvMoveParams p{};
  hum_status st = kv_move_params(desc, cache, cache_bytes, num_tokens, slots, &p);
  if (st != HUM_OK || num_tokens == 0) return st;
  if (!k_out || !v_out) return set_error(HUM_ERR_INVALID_ARG, "NULL pointer");
  if ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) % 16)
    return set_error(HUM_ERR_INVALID_ARG, "k_out and v_out must be 16-byte aligned");
  p.out[0] = static_cast<uint16_t*>(k_out);
  p.out[1] = static_cast<uint16_t*>(v_out);
  const unsigned grid = kv_move_grid(desc, num_tokens);
  hipStream_t s = static_cast<hipStream_t>(stream);
  kv_dispatch(desc, [&](auto fmt, auto dim) {
    kv_read_kernel<decltype(fmt)::value, decltype(dim)::value><<<grid, 256, 0, s>>>(p);
  });
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return set_error(HUM_ERR_HIP, "kv_read launch: %s", hipGetErrorString(err));
  return HUM_OK;
}

}  // extern "C"
