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
  int32_t tok_per_wg;  // tokens of a workgroup
  int32_t head_step;   // rows (K's heads, then V's) of a token that a workgroup takes (grid.y slices them)
  const int64_t* slots;
  const uint16_t* x[2];  // write: k, v
  int64_t ts[2], hs[2];
  uint16_t* out[2];  // read: k, v, contiguous
};

constexpr int kMoveRows = 4;  // rows whose loads a thread has in flight at once

// A workgroup's rows, and a lane's place in one: which token, K or V, head.
template <int D>
struct KvRows {
  static constexpr int kLanes = D / 8;
  static constexpr int kStep = 256 / kLanes;  // rows at once
  int64_t t0;
  int32_t r0, nr, rows, lane;
  float inv_nr;
  __device__ __forceinline__ KvRows(const KvMoveParams& p) {
    t0 = (int64_t)blockIdx.x * p.tok_per_wg;
    const int nt = (int)(p.tokens - t0 < p.tok_per_wg ? p.tokens - t0 : p.tok_per_wg);
    r0 = (int)blockIdx.y * p.head_step;
    nr = 2 * p.heads - r0 < p.head_step ? 2 * p.heads - r0 : p.head_step;
    rows = nt * nr;
    inv_nr = 1.0f / (float)nr;  // rows below 2^17: (row + 1/2) inv_nr is never a whole step off
    lane = threadIdx.x % kLanes;
  }
  __device__ __forceinline__ void place(const KvMoveParams& p, int row, int64_t* token, int* which, int* head) const {
    const int t = (int)(((float)row + 0.5f) * inv_nr);
    const int r = r0 + row - t * nr;
    *token = t0 + t;
    *which = r >= p.heads;
    *head = r - *which * p.heads;
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
  const KvRows<D> me(p);
  const int page_size = 1 << p.page_shift;
  // (the same number of passes for every thread: a row's lanes agree)
  for (int row0 = threadIdx.x / me.kLanes; row0 < me.rows; row0 += me.kStep * kMoveRows) {
    u32x4_t v[kMoveRows];
    int64_t slot[kMoveRows];
    int which[kMoveRows], head[kMoveRows];
#pragma unroll
    for (int k = 0; k < kMoveRows; ++k) {
      const int row = row0 + k * me.kStep;
      v[k] = u32x4_t{0, 0, 0, 0};
      slot[k] = -1;
      which[k] = head[k] = 0;
      if (row >= me.rows) continue;
      int64_t token;
      me.place(p, row, &token, &which[k], &head[k]);
      slot[k] = p.slots[token];
      const uint16_t* x = which[k] ? p.x[1] + token * p.ts[1] + head[k] * p.hs[1] : p.x[0] + token * p.ts[0] + head[k] * p.hs[0];
      x += me.lane * 8;
      if constexpr (VEC) {
        v[k] = *reinterpret_cast<const u32x4_t*>(x);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[k][i] = (uint32_t)x[2 * i] | ((uint32_t)x[2 * i + 1] << 16);
      }
    }
#pragma unroll
    for (int k = 0; k < kMoveRows; ++k) {
      // (unsigned: negative slots are past the end too)
      const bool live = (uint64_t)slot[k] < (uint64_t)p.slots_all;
      const int64_t page = live ? slot[k] >> p.page_shift : 0;
      const KvOffsets<FMT, D> off(which[k], (int)slot[k] & (page_size - 1), page_size);
      uint8_t* unit = p.cache + (page * p.heads + head[k]) * p.unit;
      if constexpr (FMT == HUM_ACT_BF16) {
        if (live) *reinterpret_cast<u32x4_t*>(unit + off.code + me.lane * 16) = v[k];
      } else {
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = bf16_bits_to_f32(v[k][i] & 0xFFFF);
          f[2 * i + 1] = bf16_bits_to_f32(v[k][i] >> 16);
        }
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = __builtin_fmaxf(amax, __builtin_fabsf(f[i]));
        if constexpr (FMT == HUM_ACT_FP8_TOKEN) {
#pragma unroll
          for (int m = 1; m < me.kLanes; m *= 2) amax = __builtin_fmaxf(amax, __shfl_xor(amax, m));
          const float sc = amax > 0.0f ? amax / 448.0f : 1.0f;  // IEEE f32 division
          u32x2_t o;
          o[0] = f32x2_to_e4m3x2(f[0] / sc, f[1] / sc) | (f32x2_to_e4m3x2(f[2] / sc, f[3] / sc) << 16);
          o[1] = f32x2_to_e4m3x2(f[4] / sc, f[5] / sc) | (f32x2_to_e4m3x2(f[6] / sc, f[7] / sc) << 16);
          if (live) {
            *reinterpret_cast<u32x2_t*>(unit + off.code + me.lane * 8) = o;
            if (me.lane == 0) *reinterpret_cast<float*>(unit + off.scale) = sc;
          }
        } else {
          amax = quad_max(amax);  // four lanes hold one block of 32
          const int e = mx_scale_code_emax(amax, FMT == HUM_ACT_MXFP8 ? 8 : 2);
          const float inv = mx_inv_scale(e);
          if (live) {
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
    }
  }
}

template <int FMT, int D>
__global__ __launch_bounds__(256) void kv_read_kernel(const KvMoveParams p) {
  using U = KvUnit<FMT, D>;
  const KvRows<D> me(p);
  const int page_size = 1 << p.page_shift;
  for (int row0 = threadIdx.x / me.kLanes; row0 < me.rows; row0 += me.kStep * kMoveRows) {
    constexpr int kB = 8 * U::kRow / D;  // code bytes of a lane
    uint32_t w[kMoveRows][kB / 4];
    float sc[kMoveRows];
    int64_t slot[kMoveRows], token[kMoveRows];
    int which[kMoveRows], head[kMoveRows];
#pragma unroll
    for (int k = 0; k < kMoveRows; ++k) {
      const int row = row0 + k * me.kStep < me.rows ? row0 + k * me.kStep : row0;
      me.place(p, row, &token[k], &which[k], &head[k]);
      slot[k] = p.slots[token[k]];
    }
#pragma unroll
    for (int k = 0; k < kMoveRows; ++k) {
      // (a slot outside the cache: read slot 0, write zeros)
      const int64_t s = (uint64_t)slot[k] < (uint64_t)p.slots_all ? slot[k] : 0;
      const KvOffsets<FMT, D> off(which[k], (int)s & (page_size - 1), page_size);
      const uint8_t* unit = p.cache + ((s >> p.page_shift) * p.heads + head[k]) * p.unit;
      const uint8_t* code = unit + off.code + me.lane * kB;
      if constexpr (kB == 16) {
        const u32x4_t c = *reinterpret_cast<const u32x4_t*>(code);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[k][i] = c[i];
      } else if constexpr (kB == 8) {
        const u32x2_t c = *reinterpret_cast<const u32x2_t*>(code);
        w[k][0] = c[0];
        w[k][1] = c[1];
      } else {
        w[k][0] = *reinterpret_cast<const uint32_t*>(code);
      }
      if constexpr (FMT == HUM_ACT_FP8_TOKEN) sc[k] = *reinterpret_cast<const float*>(unit + off.scale);
      if constexpr (U::kMx) sc[k] = __uint_as_float(unit[off.scale + (me.lane >> 2) * off.scale_step]);
    }
#pragma unroll
    for (int k = 0; k < kMoveRows; ++k) {
      if (row0 + k * me.kStep >= me.rows) continue;
      u32x4_t o;
      if constexpr (FMT == HUM_ACT_BF16) {
        o = u32x4_t{w[k][0], w[k][1], w[k][2], w[k][3]};
      } else {
        // codes as exact bf16, then one f32 product with the scale, rounded once
        if constexpr (FMT == HUM_ACT_MXFP4) o = e2m1x8_to_bf16(w[k][0], 1.0f);
        else o = e4m3x8_to_bf16(u32x2_t{w[k][0], w[k][1]}, 1.0f);
        const float s = U::kMx ? e8m0_to_f32(__float_as_uint(sc[k])) : sc[k];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = f32x2_to_bf16x2_bits(bf16_bits_to_f32(o[i] & 0xFFFF) * s, bf16_bits_to_f32(o[i] >> 16) * s);
      }
      if ((uint64_t)slot[k] >= (uint64_t)p.slots_all) o = u32x4_t{0, 0, 0, 0};
      *reinterpret_cast<u32x4_t*>((which[k] ? p.out[1] : p.out[0]) + (token[k] * p.heads + head[k]) * D + me.lane * 8) = o;
    }
  }
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
  // (a grid holds at most 2^32 - 1 threads)
  if (num_tokens >= (int64_t)1 << 24) return set_error(HUM_ERR_UNSUPPORTED, "at most 2^24 - 1 tokens in a call");
  p->cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  p->unit = l.unit;
  p->slots_all = d->num_pages * d->page_size;
  p->heads = d->num_kv_heads;
  p->page_shift = __builtin_ctz((unsigned)d->page_size);
  p->tokens = num_tokens;
  p->slots = slots;
  return HUM_OK;
}

// Workgroups: kMoveRows passes of rows each, fewer where the rows would
// otherwise leave compute units without one (a token's rows are cut over
// grid.y if need be).
static dim3 kv_move_grid(const hum_kv_desc* d, KvMoveParams* p) {
  const int64_t per_tok = 2 * d->num_kv_heads, step = 256 / (d->head_dim / 8);
  int64_t rows = step * kMoveRows;
  while (rows > step && p->tokens * per_tok / rows < 1024) rows /= 2;
  p->tok_per_wg = (int32_t)(rows >= per_tok ? rows / per_tok : 1);
  p->head_step = (int32_t)(rows >= per_tok ? per_tok : rows);
  return dim3((unsigned)((p->tokens + p->tok_per_wg - 1) / p->tok_per_wg),
              (unsigned)((per_tok + p->head_step - 1) / p->head_step));
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
  const dim3 grid = kv_move_grid(desc, &p);
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
  const dim3 grid = kv_move_grid(desc, &p);
  hipStream_t s = static_cast<hipStream_t>(stream);
  kv_dispatch(desc, [&](auto fmt, auto dim) {
    kv_read_kernel<decltype(fmt)::value, decltype(dim)::value><<<grid, 256, 0, s>>>(p);
  });
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return set_error(HUM_ERR_HIP, "kv_read launch: %s", hipGetErrorString(err));
  return HUM_OK;
}

}  // extern "C"
