// Paged key-value cache: quantising rows as they are written, reading them
// back.
//
// A row (one token's K or V of one head) is quantized by the rules of
// hum_quant_act: FP8 with one f32 scale per row (amax / 448), or MXFP8 /
// MXFP4 with one E8M0 scale per 32.  D / 8 neighbouring lanes hold one row,
// 16 bytes of bf16 each; the maximum moves between them (by DPP; the two
// halves of an FP8 row of 256 by one permute), so nothing is stored in LDS.
// Memory bound: each row is read once and its codes written once.
//
// Measured on MI355X, 16384 tokens of 8 heads of 128 in MXFP8, inputs that
// change from call to call: written in 21.6 us (4.7 TB/s read + written; a
// large copy reaches 4.85), read back in 19.9 us (5.1 TB/s).  The same inputs
// again, partly from the last-level cache: 17.8 and 17.6 us; in FP8, which
// has the most arithmetic, 18.8 and 17.6.  256 tokens in FP8: 3.3 and 3.1 us,
// a launch's own time.
#include "kv_common.h"
#include "rows.h"

namespace hum {

struct KvMoveParams {
  uint8_t* cache;
  uint32_t unit;         // bytes of a (page, head) unit
  uint32_t page_stride;  // bytes of a page
  int64_t slots_all;     // num_pages * page_size
  int32_t heads, page_shift;
  int64_t tokens;
  int32_t rows_wg;   // rows (K's heads, then V's) of a token that a workgroup takes; grid.y slices them
  int32_t tok_pass;  // tokens whose rows a workgroup moves at once
  int32_t passes;    // and how often it does
  const int64_t* slots;
  const uint16_t* x[2];  // write: k, v
  int64_t ts[2], hs[2];
  uint16_t* out[2];  // read: k, v, contiguous
};

constexpr int kMoveRows = 4;  // tokens whose rows a thread has in flight at once

// A thread's place: the same head of K or V, and the same 8 of its values,
// for every token it moves (what would otherwise be an index calculation per
// row bounds these kernels: they have one to four bytes to move per
// instruction).
template <int D>
struct KvPlace {
  static constexpr int kLanes = D / 8;
  int64_t t0;      // its first token
  int32_t tokens;  // how many, tok_pass apart (none for a thread without a row)
  int32_t which, head, lane;
  __device__ __forceinline__ KvPlace(const KvMoveParams& p) {
    const int row = threadIdx.x / kLanes;
    lane = threadIdx.x % kLanes;
    const int tt = (int)((uint32_t)row / (uint32_t)p.rows_wg);
    const int r = (int)blockIdx.y * p.rows_wg + row - tt * p.rows_wg;
    which = r >= p.heads;
    head = r - which * p.heads;
    t0 = (int64_t)blockIdx.x * (p.tok_pass * p.passes) + tt;
    const int64_t left = p.tokens - t0;  // of them, every tok_pass-th
    const int mine = left <= 0 ? 0 : left >= (int64_t)p.tok_pass * p.passes ? p.passes : (int)((uint32_t)(left + p.tok_pass - 1) / (uint32_t)p.tok_pass);
    tokens = tt < p.tok_pass && r < 2 * p.heads ? mine : 0;
  }
};

template <int FMT, int D, bool VEC>
__global__ __launch_bounds__(256) void kv_write_kernel(const KvMoveParams p) {
  using U = KvUnit<FMT, D>;
  constexpr int kB = 8 * U::kRow / D;  // code bytes of a lane
  const KvPlace<D> me(p);
  const int page_size = 1 << p.page_shift;
  const KvOffsets<FMT, D> off0(me.which, 0, page_size);
  uint8_t* const base = p.cache + (uint64_t)me.head * p.unit;
  const int64_t* slots = p.slots + me.t0;
  const int64_t ts = (me.which ? p.ts[1] : p.ts[0]) * p.tok_pass;
  const uint16_t* x = (me.which ? p.x[1] + me.t0 * p.ts[1] + me.head * p.hs[1] : p.x[0] + me.t0 * p.ts[0] + me.head * p.hs[0]) + me.lane * 8;
  // (every thread makes every pass: the lanes of a row exchange their maxima)
  for (int n = 0; n < p.passes; n += kMoveRows) {
    u32x4_t v[kMoveRows];
    int64_t slot[kMoveRows];
#pragma unroll
    for (int k = 0; k < kMoveRows; ++k) {
      v[k] = u32x4_t{0, 0, 0, 0};
      slot[k] = -1;
      if (n + k < me.tokens) {
        slot[k] = slots[k * p.tok_pass];
        const uint16_t* xr = x + k * ts;
        if constexpr (VEC) {
          v[k] = *reinterpret_cast<const u32x4_t*>(xr);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[k][i] = (uint32_t)xr[2 * i] | ((uint32_t)xr[2 * i + 1] << 16);
        }
      }
    }
    slots += kMoveRows * p.tok_pass;
    x += kMoveRows * ts;
#pragma unroll
    for (int k = 0; k < kMoveRows; ++k) {
      // (unsigned: negative slots are past the end too)
      const bool live = (uint64_t)slot[k] < (uint64_t)p.slots_all;
      const uint32_t page = (uint32_t)(slot[k] >> p.page_shift);
      const uint32_t at = (uint32_t)slot[k] & (uint32_t)(page_size - 1);
      uint8_t* unit = base + (uint64_t)page * p.page_stride;
      uint8_t* code = unit + (uint32_t)(off0.code + at * U::kRow + me.lane * kB);
      uint8_t* scale = unit + (uint32_t)(off0.scale + at * (U::kMx && me.which ? 1 : U::kScale));
      if constexpr (FMT == HUM_ACT_BF16) {
        if (live) *reinterpret_cast<u32x4_t*>(code) = v[k];
      } else {
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = bf16_bits_to_f32(v[k][i] & 0xFFFF);
          f[2 * i + 1] = bf16_bits_to_f32(v[k][i] >> 16);
        }
        kv_store_row<FMT, D, false>(f, me.lane, code, scale, off0.scale_step, live);
      }
    }
  }
}

template <int FMT, int D>
__global__ __launch_bounds__(256) void kv_read_kernel(const KvMoveParams p) {
  using U = KvUnit<FMT, D>;
  constexpr int kB = 8 * U::kRow / D;  // code bytes of a lane
  const KvPlace<D> me(p);
  const int page_size = 1 << p.page_shift;
  const KvOffsets<FMT, D> off0(me.which, 0, page_size);
  const uint8_t* const base = p.cache + (uint64_t)me.head * p.unit;
  const int64_t* slots = p.slots + me.t0;
  const int64_t os = (int64_t)p.tok_pass * p.heads * D;
  uint16_t* out = (me.which ? p.out[1] : p.out[0]) + (me.t0 * p.heads + me.head) * D + me.lane * 8;
  for (int n = 0; n < me.tokens; n += kMoveRows) {
    uint32_t w[kMoveRows][kB / 4];
    uint32_t sc[kMoveRows];
    bool live[kMoveRows];
#pragma unroll
    for (int k = 0; k < kMoveRows; ++k) {
      const int64_t slot = slots[n + k < me.tokens ? k * p.tok_pass : 0];
      live[k] = (uint64_t)slot < (uint64_t)p.slots_all;
      // (a slot outside the cache: read slot 0, write zeros)
      const uint32_t page = live[k] ? (uint32_t)(slot >> p.page_shift) : 0u;
      const uint32_t at = live[k] ? (uint32_t)slot & (uint32_t)(page_size - 1) : 0u;
      const uint8_t* unit = base + (uint64_t)page * p.page_stride;
      const uint8_t* code = unit + (uint32_t)(off0.code + at * U::kRow + me.lane * kB);
      const uint8_t* scale = unit + (uint32_t)(off0.scale + at * (U::kMx && me.which ? 1 : U::kScale));
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
      if constexpr (FMT == HUM_ACT_FP8_TOKEN) sc[k] = *reinterpret_cast<const uint32_t*>(scale);
      if constexpr (U::kMx) sc[k] = scale[(me.lane >> 2) * off0.scale_step];
    }
#pragma unroll
    for (int k = 0; k < kMoveRows; ++k) {
      if (n + k >= me.tokens) break;
      u32x4_t o;
      if constexpr (FMT == HUM_ACT_BF16) {
        o = u32x4_t{w[k][0], w[k][1], w[k][2], w[k][3]};
      } else {
        // codes as exact bf16, then one f32 product with the scale, rounded once
        if constexpr (FMT == HUM_ACT_MXFP4) o = e2m1x8_to_bf16(w[k][0], 1.0f);
        else o = e4m3x8_to_bf16(u32x2_t{w[k][0], w[k][1]}, 1.0f);
        const float s = U::kMx ? e8m0_to_f32(sc[k]) : __uint_as_float(sc[k]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = f32x2_to_bf16x2_bits(bf16_bits_to_f32(o[i] & 0xFFFF) * s, bf16_bits_to_f32(o[i] >> 16) * s);
      }
      if (!live[k]) o = u32x4_t{0, 0, 0, 0};
      *reinterpret_cast<u32x4_t*>(out + k * os) = o;
    }
    slots += kMoveRows * p.tok_pass;
    out += kMoveRows * os;
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
  if (reinterpret_cast<uintptr_t>(slots) % 8) return set_error(HUM_ERR_INVALID_ARG, "slots must be aligned to its elements");
  if (cache_bytes < (size_t)l.bytes)
    return set_error(HUM_ERR_WORKSPACE, "cache of %zu bytes, the description takes %lld", cache_bytes, (long long)l.bytes);
  // (a grid holds at most 2^32 - 1 threads)
  if (num_tokens >= (int64_t)1 << 24) return set_error(HUM_ERR_UNSUPPORTED, "at most 2^24 - 1 tokens in a call");
  p->cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  p->unit = (uint32_t)l.unit;
  p->page_stride = (uint32_t)(l.unit * d->num_kv_heads);
  p->slots_all = d->num_pages * d->page_size;
  p->heads = d->num_kv_heads;
  p->page_shift = __builtin_ctz((unsigned)d->page_size);
  p->tokens = num_tokens;
  p->slots = slots;
  return HUM_OK;
}

// Workgroups: the rows of a token are sliced so that as few threads as
// possible are left without one; kMoveRows passes each, fewer where the
// tokens would otherwise leave compute units without a workgroup.
static dim3 kv_move_grid(const hum_kv_desc* d, KvMoveParams* p) {
  const int all = 2 * d->num_kv_heads, step = 256 / (d->head_dim / 8);
  int best = 0;
  double best_use = 0.0;
  for (int y = (all + step - 1) / step; y <= all; ++y) {
    const int rows = (all + y - 1) / y, slices = (all + rows - 1) / rows;
    const double use = (double)(step / rows) * all / ((double)step * slices);
    if (use > best_use + 1e-9) {
      best_use = use;
      best = rows;
    }
    if (use > 0.9) break;
  }
  p->rows_wg = best;
  p->tok_pass = step / best;
  const int64_t slices = (all + best - 1) / best;
  p->passes = kMoveRows;
  while (p->passes > 1 && p->tokens * slices / (p->tok_pass * p->passes) < 1024) p->passes /= 2;
  const int64_t tok = (int64_t)p->tok_pass * p->passes;
  return dim3((unsigned)((p->tokens + tok - 1) / tok), (unsigned)slices);
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
  const uintptr_t ka = reinterpret_cast<uintptr_t>(k_out), va = reinterpret_cast<uintptr_t>(v_out);
  if ((ka < va ? va - ka : ka - va) < (uintptr_t)num_tokens * desc->num_kv_heads * desc->head_dim * 2)
    return set_error(HUM_ERR_INVALID_ARG, "k_out and v_out must not overlap");
  if ((ka | va) % 16)
    return set_error(HUM_ERR_INVALID_ARG, "k_out and v_out must be 16-byte aligned");
  const int64_t bytes = num_tokens * desc->num_kv_heads * desc->head_dim * 2;
  for (void* o : {k_out, v_out})
    if (overlap(bytes_at(o, bytes), bytes_at(cache, hum_kv_cache_bytes(desc))) != Overlap::kNo ||
        overlap(bytes_at(o, bytes), bytes_at(slots, num_tokens * 8)) != Overlap::kNo)
      return set_error(HUM_ERR_INVALID_ARG, "k_out and v_out must not overlap the cache or the slots");
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
