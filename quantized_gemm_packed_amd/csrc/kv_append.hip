// Rotary positions and the paged cache in one launch: q is turned, k is
// turned, quantized and written to its slots beside v.
//
// Per row (one head of one token): the head's norm, where there is one,
//   x' = x * (1 / sqrt(mean(x^2) + eps)) * (w + offset),
// the turn of its first rotary_dim elements (hum_rotary's coefficients and
// products: the same bits), and for k and v the cache's quantizer; f32 between
// them, rounded once at the end.  D / 8 neighbouring lanes have one row, 8
// elements each.  Memory bound: q is read and written once, k and v are read
// once and their codes written once; apart, the turned k would be written and
// read once more, and a launch paid twice.
//
// Measured on MI355X, in a captured graph, inputs that change from call to call:
// 16384 tokens of 32 + 8 heads of 128 into MXFP8 78 us, 4.7 TB/s read + written
// (a large copy reaches 5.1, the norm 5.8; hum_rotary and hum_kv_write together
// take 89), into MXFP4 74; 5003 tokens of 16 + 4 normed heads of 256, bf16, 25
// to 28 us; a decode step of 64 tokens 3.2 us, of which an empty launch is 1.9.
#include <cmath>

#include "kv_common.h"
#include "rotary_common.h"
#include "rows.h"

namespace hum {

struct AppendParams {
  uint8_t* cache;
  uint32_t unit, page_stride;
  int64_t slots_all;
  int32_t page_shift;
  int32_t heads[2];  // of q, of k and v
  const int64_t *slots, *positions;
  const double* inv_freq;
  const uint16_t* x[3];  // q, k, v
  int64_t ts[3], hs[3];
  uint16_t* q_out;
  int64_t qo_ts, qo_hs;
  const void* w[2];  // head norms of q, of k
  int64_t tokens;
  int32_t half;        // rotary_dim / 2
  int32_t row_step;    // rows (q's heads, k's, v's) per wave (grid.y slices them)
  int32_t w_f32;
  float factor, eps, offset;
};

// Sum over the N lanes (8, 16 or 32) that hold one row.
template <int N>
__device__ __forceinline__ float row_sum(float v) {
  auto with = [&](auto ctrl) {
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, false));
  };
  with(std::integral_constant<int, 0xB1>{});   // quad_perm 1,0,3,2
  with(std::integral_constant<int, 0x4E>{});   // quad_perm 2,3,0,1
  with(std::integral_constant<int, 0x141>{});  // row_half_mirror
  if constexpr (N >= 16) with(std::integral_constant<int, 0x140>{});
  if constexpr (N >= 32) v += __shfl_xor(v, 16);
  return v;
}

__device__ __forceinline__ void unpack8(const u32x4_t v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
  }
}
// Eight floats of LDS (16-byte aligned).
__device__ __forceinline__ void lds8(const float* at, float (&f)[8]) {
  const f32x4_t a = *reinterpret_cast<const f32x4_t*>(at), b = *reinterpret_cast<const f32x4_t*>(at + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = a[i];
    f[4 + i] = b[i];
  }
}

// FAST: every piece of 8 elements lies at 16 bytes and turns as a whole, with
// another whole piece (half layout: the half a multiple of 8 elements) or
// within itself (interleaved: rotary_dim a multiple of 8), and the offsets in
// a token fit 32 bits.  In the half layout the two lanes of a pair of pieces
// exchange them and form one result each:
//   y0 = x0 c + (-x1) s,   y1 = x0 s + x1 c,
// the same products with the coefficients exchanged.  (Loading both pieces in
// both lanes instead stalls the vector cache on the line that is on its way:
// 16384 tokens of 32 + 8 heads of 128 in MXFP8 117 us, with the exchange 107.)
// Otherwise accesses are aligned to their elements, which the vector memory
// takes at any width, and the other element of each pair comes from the row's
// copy in LDS (16384 tokens as above in FP8, 24 of 128 elements turned: 121 us
// with loads of single elements, 84 so).
//
// A wave has one token (its slot and addresses are scalars) or a slice of its
// rows, 64 / (D / 8) of them at once; the coefficients lie in its own part of
// LDS, so the waves of a workgroup do not wait for one another.
template <int FMT, int D, bool HALF, bool FAST, bool NORM>
__global__ __launch_bounds__(256) void append_kernel(const AppendParams p) {
  using U = KvUnit<FMT, D>;
  using off_t = std::conditional_t<FAST, int32_t, int64_t>;
  using V = std::conditional_t<FAST, u32x4_t, u32x4_at2_t>;
  constexpr int kLanes = D / 8;
  constexpr int kStep = 64 / kLanes;  // rows a wave moves at once
  constexpr int kB = 8 * U::kRow / D;
  extern __shared__ __attribute__((aligned(16))) float lds[];
  __shared__ __attribute__((aligned(16))) uint16_t copies[HALF && !FAST ? 4 : 1][512];  // of the rows a wave works on
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), sub = threadIdx.x & 63, lane = sub % kLanes;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  const bool have = t < p.tokens;
  float* cs = lds + wave * 2 * p.half;
  float* sn = cs + p.half;
  float* wt = lds + 8 * p.half;  // the norms' weights, q's and k's
  const int hq = p.heads[0], hk = p.heads[1], all = hq + 2 * hk;
  const int end = ((int)blockIdx.y + 1) * p.row_step < all ? ((int)blockIdx.y + 1) * p.row_step : all;
  int row = (int)blockIdx.y * p.row_step + sub / kLanes;

  const off_t hs_q = (off_t)p.hs[0], hs_k = (off_t)p.hs[1], hs_v = (off_t)p.hs[2], qo_hs = (off_t)p.qo_hs;
  const bool norm_q = NORM && p.w[0], norm_k = NORM && p.w[1];
  const uint32_t unit_bytes = p.unit;
  const int half = p.half;
  const float eps = p.eps;

  // a lane's place among the pieces of the turned part
  const int m = p.half / 8;
  const bool first = lane < m, turn = lane < (HALF ? 2 * m : p.half / 4);
  const int at0 = HALF && turn ? (first ? lane : lane - m) * 8 : lane * 8;  // where the turn's x0 lies
  const int partner = (sub + (HALF && turn ? (first ? m : -m) : 0)) * 4;
  const uint32_t flip = first ? 0x80008000u : 0u;

  const uint16_t *const xq = p.x[0] + t * p.ts[0], *const xk = p.x[1] + t * p.ts[1], *const xv = p.x[2] + t * p.ts[2];

  if constexpr (NORM) {
    for (int i = threadIdx.x; i < 2 * D; i += 256) {
      const void* w = i < D ? p.w[0] : p.w[1];
      const int e = i < D ? i : i - D;
      if (w) wt[i] = (p.w_f32 ? static_cast<const float*>(w)[e] : bf16_bits_to_f32(static_cast<const uint16_t*>(w)[e])) + p.offset;
    }
    __syncthreads();
  }
  if (!have) return;
  const int64_t slot = p.slots[t], position = p.positions[t];
  for (int i = sub; i < half; i += 64) rotary_coefficients(position, p.inv_freq[i], p.factor, 1.0f, cs + i, sn + i);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  // (unsigned: negative slots are past the end too)
  const bool live = (uint64_t)slot < (uint64_t)p.slots_all;
  const int page_size = 1 << p.page_shift, at = (int)(slot & (page_size - 1));
  const KvOffsets<FMT, D> off_k(0, at, page_size), off_v(1, at, page_size);
  uint8_t* const page = p.cache + (uint64_t)(uint32_t)(slot >> p.page_shift) * p.page_stride;
  uint16_t* const yq = p.q_out + t * p.qo_ts + lane * 8;

  // One row is loaded while the one before it is worked on.
  u32x4_t x0_next;
  int kind_next = -1, head_next = 0;
  const int steps = (end - (int)blockIdx.y * p.row_step + kStep - 1) / kStep;
  for (int n = -1; n < steps; ++n) {
    u32x4_t x0 = x0_next;
    const int kind = kind_next, head = head_next;
    kind_next = -1;
    if (row < end) {
      kind_next = (row >= hq) + (row >= hq + hk);
      head_next = row - (kind_next ? hq : 0) - (kind_next == 2 ? hk : 0);
      const uint16_t* x = (kind_next == 0 ? xq : kind_next == 1 ? xk : xv) + head_next * (kind_next == 0 ? hs_q : kind_next == 1 ? hs_k : hs_v) + lane * 8;
      x0_next = *reinterpret_cast<const V*>(x);
    }
    row += kStep;
    if (kind >= 0) {
      float f[8];
      if (kind < 2) {
        float g[8];
        float sum = 0.0f;  // of the squares of its own elements
        if constexpr (NORM) {
          unpack8(x0, f);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(f[i], f[i], sum);
        }
        u32x4_t x1;
        if constexpr (HALF && !FAST) {
          uint16_t* mine = copies[wave] + sub / kLanes * D;
          *reinterpret_cast<u32x4_t*>(mine + lane * 8) = x0;
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          __builtin_amdgcn_wave_barrier();
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const int e = lane * 8 + i, o = e + 1;
            const uint32_t a = mine[e < half ? e + half : e < 2 * half ? e - half : e];
            const uint32_t b = mine[o < half ? o + half : o < 2 * half ? o - half : o];
            x1[i / 2] = a | b << 16;
          }
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          __builtin_amdgcn_wave_barrier();
        }
        if constexpr (HALF && FAST) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t o = (uint32_t)__builtin_amdgcn_ds_bpermute(partner, (int)x0[i]), me = x0[i];
            x0[i] = first || !turn ? me : o;
            x1[i] = (first ? o : me) ^ flip;
          }
        }
        unpack8(x0, f);
        if constexpr (HALF) unpack8(x1, g);
        if (NORM && (kind ? norm_k : norm_q)) {
          const float* w = wt + (kind ? D : 0);
          const float r = 1.0f / __builtin_sqrtf(row_sum<kLanes>(sum) * (1.0f / D) + eps);
          if constexpr (FAST) {
            float v[8];
            lds8(w + at0, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = f[i] * r * v[i];
            if (HALF && turn) {
              lds8(w + at0 + half, v);
#pragma unroll
              for (int i = 0; i < 8; ++i) g[i] = g[i] * r * v[i];
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int e = lane * 8 + i;
              f[i] = f[i] * r * w[e];
              if (HALF && e < 2 * half) g[i] = g[i] * r * w[e < half ? e + half : e - half];
            }
          }
        }
        if constexpr (FAST && HALF) {
          if (turn) {
            float ca[8], cb[8];
            lds8(cs + (at0 + (first ? 0 : half)), ca);
            lds8(cs + (at0 + (first ? half : 0)), cb);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __builtin_fmaf(f[i], ca[i], g[i] * cb[i]);
          }
        } else if constexpr (HALF) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int e = lane * 8 + i;
            if (e < half) f[i] = rotary_first(f[i], g[i], cs[e], sn[e]);
            else if (e < 2 * half) f[i] = rotary_second(g[i], f[i], cs[e - half], sn[e - half]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int pr = lane * 4 + i;
            if (FAST ? turn : pr < half) {
              const float a = f[2 * i], b = f[2 * i + 1];
              f[2 * i] = rotary_first(a, b, cs[pr], sn[pr]);
              f[2 * i + 1] = rotary_second(a, b, cs[pr], sn[pr]);
            }
          }
        }
      } else {
        unpack8(x0, f);
      }
      if (kind == 0) {
        u32x4_t o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = f32x2_to_bf16x2_bits(f[2 * i], f[2 * i + 1]);
        *reinterpret_cast<V*>(yq + head * qo_hs) = o;
      } else {
        uint8_t* unit = page + (uint32_t)head * unit_bytes;
        if (FMT == HUM_ACT_BF16 && kind == 2) {
          if (live) *reinterpret_cast<u32x4_t*>(unit + off_v.code + lane * kB) = x0;
        } else if (kind == 2) {
          kv_store_row<FMT, D, false>(f, lane, unit + off_v.code + lane * kB, unit + off_v.scale, off_v.scale_step, live);
        } else {
          kv_store_row<FMT, D, true>(f, lane, unit + off_k.code + lane * kB, unit + off_k.scale, off_k.scale_step, live);
        }
      }
    }
  }
}

}  // namespace hum

using namespace hum;

extern "C" hum_status hum_rotary_kv_write(const hum_rotary_desc* rot, const hum_kv_desc* kv, const hum_head_norm* norm,
                                          void* cache, size_t cache_bytes, int64_t num_tokens, const int64_t* positions,
                                          const double* inv_freq, const int64_t* slots, const void* q, int64_t q_ts,
                                          int64_t q_hs, void* q_out, int64_t qo_ts, int64_t qo_hs, const void* k,
                                          int64_t k_ts, int64_t k_hs, const void* v, int64_t v_ts, int64_t v_hs,
                                          void* stream) {
  clear_error();
  if (!rot) return set_error(HUM_ERR_INVALID_ARG, "the rotary description is NULL");
  KvLayout l;
  const hum_status st = kv_layout(kv, &l);
  if (st != HUM_OK) return st;
  if (rot->dtype != HUM_BF16) return set_error(HUM_ERR_UNSUPPORTED, "dtype must be bf16");
  if (rot->layout != HUM_ROPE_HALF && rot->layout != HUM_ROPE_INTERLEAVED)
    return set_error(HUM_ERR_INVALID_ARG, "bad layout");
  if (rot->head_dim != kv->head_dim || rot->num_kv_heads != kv->num_kv_heads)
    return set_error(HUM_ERR_INVALID_ARG, "head_dim and num_kv_heads must be the cache's");
  if (rot->rotary_dim < 2 || rot->rotary_dim % 2 || rot->rotary_dim > rot->head_dim)
    return set_error(HUM_ERR_INVALID_ARG, "rotary_dim must be even, 2 .. head_dim");
  if (rot->num_q_heads < 0 || rot->num_q_heads > 4096) return set_error(HUM_ERR_INVALID_ARG, "num_q_heads must be 0 .. 4096");
  if (rot->inverse != 0) return set_error(HUM_ERR_INVALID_ARG, "inverse must be 0");
  if (norm) {
    if (norm->weight_dtype != HUM_BF16 && norm->weight_dtype != HUM_F32)
      return set_error(HUM_ERR_UNSUPPORTED, "weight_dtype must be bf16 or f32");
    if (!(norm->eps > 0.0f) || !std::isfinite(norm->eps)) return set_error(HUM_ERR_INVALID_ARG, "eps must be a number above 0");
    if (!std::isfinite(norm->weight_offset)) return set_error(HUM_ERR_INVALID_ARG, "weight_offset must be finite");
  }
  if (num_tokens < 0) return set_error(HUM_ERR_INVALID_ARG, "num_tokens must be >= 0");
  // (a grid holds at most 2^32 - 1 threads)
  if (num_tokens >= (int64_t)1 << 24) return set_error(HUM_ERR_UNSUPPORTED, "at most 2^24 - 1 tokens in a call");
  if (num_tokens == 0) return HUM_OK;
  const int hq = rot->num_q_heads, hk = kv->num_kv_heads, d = kv->head_dim;
  if (!cache || !positions || !inv_freq || !slots || !k || !v || (hq && (!q || !q_out)))
    return set_error(HUM_ERR_INVALID_ARG, "NULL pointer");
  auto addr = [](const void* x) { return reinterpret_cast<uintptr_t>(x); };
  if (addr(cache) % 16) return set_error(HUM_ERR_INVALID_ARG, "the cache must be 16-byte aligned");
  if ((addr(positions) | addr(inv_freq) | addr(slots)) % 8)
    return set_error(HUM_ERR_INVALID_ARG, "positions, inv_freq and slots must be aligned to their elements");
  if (cache_bytes < (size_t)l.bytes)
    return set_error(HUM_ERR_WORKSPACE, "cache of %zu bytes, the description takes %lld", cache_bytes, (long long)l.bytes);
  if ((addr(k) | addr(v) | (hq ? addr(q) | addr(q_out) : 0)) % 2)
    return set_error(HUM_ERR_INVALID_ARG, "q, q_out, k and v must be aligned to their elements");
  const int wsize = norm && norm->weight_dtype == HUM_F32 ? 4 : 2;
  if (norm && (addr(norm->q_weight) | addr(norm->k_weight)) % wsize)
    return set_error(HUM_ERR_INVALID_ARG, "the norms' weights must be aligned to their elements");
  const bool in_place = q == q_out && ((q_ts == qo_ts) || num_tokens == 1) && (q_hs == qo_hs || hq == 1);
  // q_out and the cache are stored while other workgroups still read: neither
  // may lie in an input, but q_out in q's place, row by row.
  auto rows = [&](const void* at, int heads, int64_t ts, int64_t hs) {
    return Rows{(int64_t)(intptr_t)at, num_tokens, heads, (wide_t)ts * 2, (wide_t)hs * 2, (int64_t)d * 2};
  };
  struct In {
    const char* name;
    Rows at;
  };
  const In in[] = {{"q", rows(q, hq, q_ts, q_hs)},
                   {"k", rows(k, hk, k_ts, k_hs)},
                   {"v", rows(v, hk, v_ts, v_hs)},
                   {"positions", bytes_at(positions, num_tokens * 8)},
                   {"slots", bytes_at(slots, num_tokens * 8)},
                   {"inv_freq", bytes_at(inv_freq, rot->rotary_dim / 2 * 8)},
                   {"q_weight", bytes_at(norm ? norm->q_weight : nullptr, norm && norm->q_weight ? d * wsize : 0)},
                   {"k_weight", bytes_at(norm ? norm->k_weight : nullptr, norm && norm->k_weight ? d * wsize : 0)}};
  const Rows of_q = rows(q_out, hq, qo_ts, qo_hs), of_cache = bytes_at(cache, l.bytes);
  if (overlaps_itself(of_q)) return set_error(HUM_ERR_INVALID_ARG, "the rows of q_out must not overlap");
  if (overlap(of_q, of_cache) != Overlap::kNo) return set_error(HUM_ERR_INVALID_ARG, "q_out and the cache must not overlap");
  for (const In& i : in) {
    if (!(i.at.at == of_q.at && in_place && &i == in) && overlap(of_q, i.at) != Overlap::kNo)
      return set_error(HUM_ERR_INVALID_ARG, "q_out and %s must not overlap", i.name);
    if (overlap(of_cache, i.at) != Overlap::kNo)
      return set_error(HUM_ERR_INVALID_ARG, "the cache and %s must not overlap", i.name);
  }
  AppendParams p{};
  p.cache = static_cast<uint8_t*>(cache);
  p.unit = (uint32_t)l.unit;
  p.page_stride = (uint32_t)(l.unit * hk);
  p.slots_all = kv->num_pages * kv->page_size;
  p.page_shift = __builtin_ctz((unsigned)kv->page_size);
  p.heads[0] = hq;
  p.heads[1] = hk;
  p.slots = slots;
  p.positions = positions;
  p.inv_freq = inv_freq;
  const void* xs[3] = {q, k, v};
  const int64_t strides[3][2] = {{q_ts, q_hs}, {k_ts, k_hs}, {v_ts, v_hs}};
  int64_t any = hq ? (int64_t)(addr(q) | addr(q_out)) / 2 | q_ts | q_hs | qo_ts | qo_hs : 0;
  any |= (int64_t)(addr(k) | addr(v)) / 2 | k_ts | k_hs | v_ts | v_hs;
  for (int i = 0; i < 3; ++i) {
    p.x[i] = static_cast<const uint16_t*>(xs[i]);
    p.ts[i] = strides[i][0];
    p.hs[i] = strides[i][1];
  }
  p.q_out = static_cast<uint16_t*>(q_out);
  p.qo_ts = qo_ts;
  p.qo_hs = qo_hs;
  p.tokens = num_tokens;
  p.half = rot->rotary_dim / 2;
  p.factor = rot->factor;
  if (norm) {
    p.w[0] = norm->q_weight;
    p.w[1] = norm->k_weight;
    p.w_f32 = wsize == 4;
    p.eps = norm->eps;
    p.offset = norm->weight_offset;
  }
  const bool half = rot->layout == HUM_ROPE_HALF;
  // (heads that lie further apart than 2^18 elements leave the fast path, whose offsets are of 32 bits)
  auto near = [](int64_t hs) { return hs < 1 << 18 && hs > -(1 << 18); };
  const bool fast = any % 8 == 0 && p.half % (half ? 8 : 4) == 0 && (!hq || (near(q_hs) && near(qo_hs))) && near(k_hs) && near(v_hs);
  // A token to a wave, four to a workgroup; rows are sliced over grid.y where
  // the tokens alone would leave compute units without a workgroup (32 + 8 heads
  // of 128 into FP8: 64 tokens 3.2 us, unsliced 9.1; 512 tokens 5.8 and 10.2.
  // Slices for 2048 workgroups in place of 512 would take 5.4 there and 3.9
  // instead of 4.5 for 256 tokens; below that the two are alike).
  const int all = hq + 2 * hk, at_once = 64 / (d / 8);
  const int64_t gx = (num_tokens + 3) / 4;
  int64_t gy = 1;
  if (gx < 512) {
    gy = (512 + gx - 1) / gx;
    const int64_t most = (all + at_once - 1) / at_once;
    if (gy > most) gy = most;
  }
  p.row_step = (int)((all + gy - 1) / gy);
  p.row_step = (p.row_step + at_once - 1) / at_once * at_once;
  gy = (all + p.row_step - 1) / p.row_step;
  const bool normed = p.w[0] || p.w[1];
  const size_t lds = ((size_t)p.half * 8 + (normed ? 2 * d : 0)) * sizeof(float);
  const dim3 grid((unsigned)gx, (unsigned)gy);
  hipStream_t s = static_cast<hipStream_t>(stream);
  kv_dispatch(kv, [&](auto fmt, auto dim) {
    constexpr int F = decltype(fmt)::value, D = decltype(dim)::value;
    auto by = [&](auto h, auto f) {
      constexpr bool H = decltype(h)::value, FA = decltype(f)::value;
      if (normed) append_kernel<F, D, H, FA, true><<<grid, 256, lds, s>>>(p);
      else append_kernel<F, D, H, FA, false><<<grid, 256, lds, s>>>(p);
    };
    if (half && fast) by(std::true_type{}, std::true_type{});
    else if (half) by(std::true_type{}, std::false_type{});
    else if (fast) by(std::false_type{}, std::true_type{});
    else by(std::false_type{}, std::false_type{});
  });
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return set_error(HUM_ERR_HIP, "rotary_kv_write launch: %s", hipGetErrorString(err));
  return HUM_OK;
}
