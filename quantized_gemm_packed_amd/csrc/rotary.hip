// Rotary positions: q and k of a decode step or a prompt in one launch.
//
// Pair i of a head turns by the angle positions[t] * inv_freq[i]:
//   y0 = x0 c - x1 s, y1 = x0 s + x1 c,  c = a cos, s = a sin.
// Memory bound (q and k are read and written once).  An angle in radians at
// position 10^6 has lost 16 of f32's 24 bits, so the turn count
// positions * inv_freq / 2 pi is formed and reduced to [-1/2, 1/2] in f64
// (two multiplies, a round and a subtract).  The remainder goes to the f32
// sine and cosine as an f32 and the rest of it, to first order: without the
// rest the angle is off by up to 2 pi 2^-26, more than the functions' own
// error, and sines next to half a turn by thousands of their ulps.  They are
// the same for every head of a token: a workgroup computes them once, into
// LDS.
//
// Measured on MI355X: 16384 tokens of 32 + 8 bf16 heads of 128, 64 elements
// turned in adjacent pairs, inputs that change from call to call: 73 us,
// 4.6 TB/s read + written (a large copy reaches 4.85); a decode step of 64 tokens: 3.3 us, a launch's own time.
#include <cmath>

#include "dev_common.h"
#include "hum_internal.h"
#include "rows.h"

namespace hum {

struct RotaryParams {
  const int64_t* positions;
  const double* inv_freq;
  const void* x[2];  // q, k
  void* y[2];
  int64_t x_ts[2], x_hs[2], y_ts[2], y_hs[2];
  int64_t tokens;
  int32_t heads[2];
  int32_t half;        // rotary_dim / 2
  int32_t rest;        // head_dim - rotary_dim elements to copy (0 when in place)
  int32_t units;       // rotating units (VEC pairs) and copied ones (2 VEC elements) of a head
  int32_t lanes;       // that share a head (all its units at once, at most 256)
  int32_t tok_per_wg;
  int32_t head_step;   // heads per workgroup (grid.y slices the heads)
  float factor;
  float sign;          // -1: inverse
};

template <typename T>
__device__ __forceinline__ float ld1(T v) {
  if constexpr (sizeof(T) == 2) return bf16_bits_to_f32(v);
  else return v;
}
template <typename T>
__device__ __forceinline__ T st1(float v) {
  if constexpr (sizeof(T) == 2) return (T)f32_to_bf16_bits(v);
  else return v;
}

template <typename T, int VEC>
struct Pack {
  T v[VEC];
};

// VEC: elements per access, as many as every address and the sizes allow (16
// bytes, then halves of it down to one element).
// A lane's unit is two pieces of VEC elements of one head: the two halves of
// VEC pairs, VEC / 2 adjacent pairs of either half of the turned part (one
// pair, VEC = 1), or two pieces to copy, of 16 bytes from either half of what
// is copied (neighbouring lanes access neighbouring pieces: 16384 tokens, 40
// bf16 heads of 128 turned in adjacent pairs, 72.7 us with 2 VEC of them side
// by side, 64.8), smaller ones side by side (72 f32 heads of 80 with 20
// turned, 11886 tokens: 124 us, 130 apart).  Each thread has
// the loads of kRows heads in flight at once (with one the loop waits for
// memory at every head), the first of them while the angles are computed.
template <typename T, bool HALF, int VEC>
__global__ __launch_bounds__(256) void rotary_kernel(const RotaryParams p) {
  typedef Pack<T, VEC> __attribute__((aligned(sizeof(T) * VEC))) P;
  constexpr int kRows = 4;
  constexpr bool kPair = !HALF && VEC == 1;
  constexpr bool kApart = VEC * sizeof(T) == 16;
  extern __shared__ float lds[];
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * p.tok_per_wg;
  const int nt = (int)(p.tokens - t0 < p.tok_per_wg ? p.tokens - t0 : p.tok_per_wg);
  float* cs = lds;
  float* sn = lds + p.tok_per_wg * p.half;

  const int lanes = p.lanes;
  const int rot = p.half / VEC;
  const int hall = p.heads[0] + p.heads[1];
  const int h0 = (int)blockIdx.y * p.head_step;
  const int nh = hall - h0 < p.head_step ? hall - h0 : p.head_step;
  const float inv_nh = 1.0f / (float)nh;  // rows below 2^17: (row + 1/2) inv_nh is never a whole step off
  const int step = (int)(256u / (uint32_t)lanes);
  const int rows = nt * nh;

  // the rows row0, row0 + step, ... and the unit u of each
  const int first_row = (int)(((float)tid + 0.5f) / (float)lanes), first_u = tid - first_row * lanes;
  int row0 = first_row, u = first_u;
  bool live = row0 < step && row0 < rows;
  T* y[kRows];
  int tok[kRows];
  int at0 = 0, at1 = 0;
  bool turn = false, two = false;
  P a[kRows], b[kRows];
  auto load = [&]() {
    turn = u < rot;
    at0 = turn ? (kPair ? 2 * u : u * VEC) : 2 * p.half + (u - rot) * VEC * (kApart ? 1 : 2);
    at1 = at0 + (turn ? (kPair ? 1 : p.half) : (kApart ? p.units - rot : 1) * VEC);
    two = turn || at1 + VEC <= 2 * p.half + p.rest;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int row = row0 + k * step < rows ? row0 + k * step : row0;
      tok[k] = (int)(((float)row + 0.5f) * inv_nh);
      const int hh = h0 + row - tok[k] * nh;
      const int which = hh >= p.heads[0];
      const int h = hh - (which ? p.heads[0] : 0);
      const T* x = static_cast<const T*>(which ? p.x[1] : p.x[0]) + (t0 + tok[k]) * (which ? p.x_ts[1] : p.x_ts[0]) +
                   h * (which ? p.x_hs[1] : p.x_hs[0]);
      y[k] = static_cast<T*>(which ? p.y[1] : p.y[0]) + (t0 + tok[k]) * (which ? p.y_ts[1] : p.y_ts[0]) +
             h * (which ? p.y_hs[1] : p.y_hs[0]);
      // (of a row past the last nothing is read or stored)
      if (row0 + k * step < rows) {
        a[k] = *reinterpret_cast<const P*>(x + at0);
        if (two) b[k] = *reinterpret_cast<const P*>(x + at1);
      }
    }
  };
  if (live) load();

  for (int i = tid; i < nt * p.half; i += 256) {
    const int t = i / p.half;
    const double turns = (double)p.positions[t0 + t] * (p.inv_freq[i - t * p.half] * 0.15915494309189535);
    const double rem = turns - __builtin_rint(turns);
    const float r = (float)rem, lo = (float)(rem - r) * 6.28318531f;
    float s, c;
    sincospif(2.0f * r, &s, &c);
    // (each rounded once, the factor included)
    const float fs = p.factor * p.sign;
    cs[i] = __builtin_fmaf(c, p.factor, -s * lo * p.factor);
    sn[i] = __builtin_fmaf(s, fs, c * lo * fs);
  }
  __syncthreads();

  while (live) {
    if (turn) {
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        // coefficients of the unit's first pair, and of the second piece's first
        const int c0 = tok[k] * p.half + (HALF || kPair ? u * VEC : u * VEC / 2), c1 = c0 + p.half / 2;
        T e[2 * VEC];  // the unit's elements, pairs at (i, i + VEC) or (2 i, 2 i + 1)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          e[i] = a[k].v[i];
          e[VEC + i] = b[k].v[i];
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const int i0 = HALF ? i : 2 * i, i1 = HALF ? VEC + i : 2 * i + 1;
          const float x0 = ld1<T>(e[i0]), x1 = ld1<T>(e[i1]);
          const int at = HALF || kPair || i < VEC / 2 ? c0 + i : c1 + i - VEC / 2;
          // (the fused product named: every instance gives the same bits)
          e[i0] = st1<T>(__builtin_fmaf(x0, cs[at], -(x1 * sn[at])));
          e[i1] = st1<T>(__builtin_fmaf(x0, sn[at], x1 * cs[at]));
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          a[k].v[i] = e[i];
          b[k].v[i] = e[VEC + i];
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (row0 + k * step >= rows) continue;
      *reinterpret_cast<P*>(y[k] + at0) = a[k];
      if (two) *reinterpret_cast<P*>(y[k] + at1) = b[k];
    }
    u += lanes;
    if (u >= p.units) {
      u = first_u;
      row0 += step * kRows;
    }
    live = row0 < rows;
    if (live) load();
  }
}

template <typename T, int VEC>
static void launch_rotary(const RotaryParams& p, bool half, dim3 grid, size_t lds, hipStream_t s) {
  if (half) rotary_kernel<T, true, VEC><<<grid, 256, lds, s>>>(p);
  else rotary_kernel<T, false, VEC><<<grid, 256, lds, s>>>(p);
}

}  // namespace hum

using namespace hum;

extern "C" {

hum_status hum_rotary_inv_freq(int32_t rotary_dim, double base, int32_t scaling, double factor, double original_len,
                               double fast_turns, double slow_turns, double* inv_freq_host, float* factor_out) {
  clear_error();
  if (!inv_freq_host || !factor_out) return set_error(HUM_ERR_INVALID_ARG, "NULL pointer");
  if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > 1024)
    return set_error(HUM_ERR_INVALID_ARG, "rotary_dim must be even, 2 .. 1024");
  if (!(base > 1.0) || !std::isfinite(base)) return set_error(HUM_ERR_INVALID_ARG, "base must be a number above 1");
  if (scaling < HUM_ROPE_NONE || scaling > HUM_ROPE_YARN) return set_error(HUM_ERR_INVALID_ARG, "bad scaling");
  if (scaling != HUM_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
    return set_error(HUM_ERR_INVALID_ARG, "factor must be a number of at least 1");
  const double r = rotary_dim;
  if (scaling == HUM_ROPE_NTK) {
    if (rotary_dim == 2) return set_error(HUM_ERR_UNSUPPORTED, "NTK scaling needs more than one pair");
    base *= std::pow(factor, r / (r - 2.0));
  }
  double lo = 0, hi = 0;
  if (scaling == HUM_ROPE_YARN) {
    if (!(original_len >= 1.0) || !std::isfinite(original_len) || !(fast_turns > slow_turns) || !(slow_turns > 0.0) ||
        !std::isfinite(fast_turns))
      return set_error(HUM_ERR_INVALID_ARG, "YaRN needs original_len >= 1 and fast_turns > slow_turns > 0");
    // the (real) pair index that turns n times over original_len positions:
    // original_len * base^(-2i/R) = 2 pi n
    auto pair_of = [&](double n) { return r * std::log(original_len / (n * 2.0 * M_PI)) / (2.0 * std::log(base)); };
    lo = std::fmax(std::floor(pair_of(fast_turns)), 0.0);
    hi = std::fmin(std::ceil(pair_of(slow_turns)), r - 1.0);
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / r);
    if (scaling == HUM_ROPE_LINEAR) f /= factor;
    if (scaling == HUM_ROPE_YARN) {
      const double slow = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 1e-3), 0.0), 1.0);
      f = f * (1.0 - slow) + f / factor * slow;
    }
    inv_freq_host[i] = f;
  }
  *factor_out = scaling == HUM_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return HUM_OK;
}

hum_status hum_rotary(const hum_rotary_desc* d, int64_t num_tokens, const int64_t* positions, const double* inv_freq,
                      const void* q, int64_t q_ts, int64_t q_hs, void* q_out, int64_t qo_ts, int64_t qo_hs,
                      const void* k, int64_t k_ts, int64_t k_hs, void* k_out, int64_t ko_ts, int64_t ko_hs,
                      void* stream) {
  clear_error();
  if (!d) return set_error(HUM_ERR_INVALID_ARG, "desc is NULL");
  if (d->dtype != HUM_BF16 && d->dtype != HUM_F32) return set_error(HUM_ERR_UNSUPPORTED, "dtype must be bf16 or f32");
  if (d->layout != HUM_ROPE_HALF && d->layout != HUM_ROPE_INTERLEAVED)
    return set_error(HUM_ERR_INVALID_ARG, "bad layout");
  if (d->head_dim < 1 || d->head_dim > 1024) return set_error(HUM_ERR_UNSUPPORTED, "head_dim must be 1 .. 1024");
  if (d->rotary_dim < 2 || d->rotary_dim % 2 || d->rotary_dim > d->head_dim)
    return set_error(HUM_ERR_INVALID_ARG, "rotary_dim must be even, 2 .. head_dim");
  if (d->num_q_heads < 0 || d->num_kv_heads < 0 || d->num_q_heads > 4096 || d->num_kv_heads > 4096)
    return set_error(HUM_ERR_INVALID_ARG, "head counts must be 0 .. 4096");
  if (d->inverse != 0 && d->inverse != 1) return set_error(HUM_ERR_INVALID_ARG, "inverse must be 0/1");
  if (num_tokens < 0) return set_error(HUM_ERR_INVALID_ARG, "num_tokens must be >= 0");
  // (a grid holds at most 2^32 - 1 threads)
  if (num_tokens >= (int64_t)1 << 24) return set_error(HUM_ERR_UNSUPPORTED, "at most 2^24 - 1 tokens in a call");
  const int hall = d->num_q_heads + d->num_kv_heads;
  if (num_tokens == 0 || hall == 0) return HUM_OK;
  if (!positions || !inv_freq || (d->num_q_heads && (!q || !q_out)) || (d->num_kv_heads && (!k || !k_out)))
    return set_error(HUM_ERR_INVALID_ARG, "NULL pointer");
  if ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(inv_freq)) % 8)
    return set_error(HUM_ERR_INVALID_ARG, "positions and inv_freq must be aligned to their elements");
  if (d->num_q_heads && d->num_kv_heads && (q_out == k_out || q_out == k || k_out == q))
    return set_error(HUM_ERR_INVALID_ARG, "q's output must be another buffer than k and its output, k's another than q");
  const int size = d->dtype == HUM_BF16 ? 2 : 4;
  RotaryParams p{};
  p.positions = positions;
  p.inv_freq = inv_freq;
  const void* xs[2] = {q, k};
  void* ys[2] = {q_out, k_out};
  const int64_t st[2][4] = {{q_ts, q_hs, qo_ts, qo_hs}, {k_ts, k_hs, ko_ts, ko_hs}};
  const int heads[2] = {d->num_q_heads, d->num_kv_heads};
  // whatever an access has to divide, in elements: the two halves, the rest of
  // a head, the strides and the addresses
  int64_t all = (d->rotary_dim / 2) | (d->head_dim - d->rotary_dim);
  bool in_place = true;
  for (int i = 0; i < 2; ++i) {
    p.x[i] = xs[i];
    p.y[i] = ys[i];
    p.x_ts[i] = st[i][0];
    p.x_hs[i] = st[i][1];
    p.y_ts[i] = st[i][2];
    p.y_hs[i] = st[i][3];
    p.heads[i] = heads[i];
    if (!heads[i]) continue;
    if (reinterpret_cast<uintptr_t>(xs[i]) % size || reinterpret_cast<uintptr_t>(ys[i]) % size)
      return set_error(HUM_ERR_INVALID_ARG, "q, k and their outputs must be aligned to their elements");
    if (xs[i] == ys[i] && (st[i][0] != st[i][2] || st[i][1] != st[i][3]))
      return set_error(HUM_ERR_INVALID_ARG, "in place, input and output strides must be the same");
    if (xs[i] != ys[i]) in_place = false;
    all |= (int64_t)(reinterpret_cast<uintptr_t>(xs[i]) | reinterpret_cast<uintptr_t>(ys[i])) / size;
    for (int j = 0; j < 4; ++j) all |= st[i][j];
  }
  // A workgroup's rows are read while others are stored: no output may lie in
  // what is not its own input.
  auto extent = [&](const void* at, int i, int out) {
    return Rows{(int64_t)(intptr_t)at, num_tokens, heads[i], (wide_t)st[i][out] * size, (wide_t)st[i][out + 1] * size,
                (int64_t)d->head_dim * size};
  };
  for (int i = 0; i < 2; ++i) {
    if (!heads[i]) continue;
    const Rows y = extent(ys[i], i, 2);
    if (overlaps_itself(y)) return set_error(HUM_ERR_INVALID_ARG, "the rows of an output must not overlap");
    for (int j = 0; j < 2; ++j) {
      if (!heads[j] || (i == j && xs[i] == ys[i])) continue;
      if (overlap(y, extent(xs[j], j, 0)) != Overlap::kNo)
        return set_error(HUM_ERR_INVALID_ARG, "an output must not overlap q or k, unless it is the same tensor as its input");
    }
  }
  if (heads[0] && heads[1] && overlap(extent(ys[0], 0, 2), extent(ys[1], 1, 2)) != Overlap::kNo)
    return set_error(HUM_ERR_INVALID_ARG, "q's output and k's must not overlap");
  int v = 16 / size;
  while (all % v) v /= 2;
  p.tokens = num_tokens;
  p.half = d->rotary_dim / 2;
  p.rest = in_place ? 0 : d->head_dim - d->rotary_dim;
  p.units = p.half / v + (p.rest / v + 1) / 2;
  p.lanes = p.units < 256 ? p.units : 256;
  p.factor = d->factor;
  p.sign = d->inverse ? -1.0f : 1.0f;
  // Tokens per workgroup: as many as fill 256 threads with one sine and
  // cosine each; heads are sliced over grid.y where the tokens alone would
  // leave compute units without a workgroup.
  int64_t tok = 256 / p.half;
  tok = tok < 1 ? 1 : tok > 8 ? 8 : tok;
  while (tok > 1 && (num_tokens + tok - 1) / tok < 1024) tok /= 2;
  p.tok_per_wg = (int)tok;
  const int64_t gx = (num_tokens + tok - 1) / tok;
  const int rows = 256 / p.lanes;  // heads a workgroup turns at once
  int64_t gy = 1;
  if (gx < 512) {
    gy = (512 + gx - 1) / gx;
    const int64_t most = (hall + rows - 1) / rows;
    if (gy > most) gy = most;
  }
  p.head_step = (int)((hall + gy - 1) / gy);
  gy = (hall + p.head_step - 1) / p.head_step;
  const size_t lds = (size_t)tok * p.half * 2 * sizeof(float);
  const dim3 grid((unsigned)gx, (unsigned)gy);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool hf = d->layout == HUM_ROPE_HALF;
  if (size == 2) {
    if (v == 8) launch_rotary<uint16_t, 8>(p, hf, grid, lds, s);
    else if (v == 4) launch_rotary<uint16_t, 4>(p, hf, grid, lds, s);
    else if (v == 2) launch_rotary<uint16_t, 2>(p, hf, grid, lds, s);
    else launch_rotary<uint16_t, 1>(p, hf, grid, lds, s);
  } else {
    if (v == 4) launch_rotary<float, 4>(p, hf, grid, lds, s);
    else if (v == 2) launch_rotary<float, 2>(p, hf, grid, lds, s);
    else launch_rotary<float, 1>(p, hf, grid, lds, s);
  }
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return set_error(HUM_ERR_HIP, "rotary launch: %s", hipGetErrorString(err));
  return HUM_OK;
}

}  // extern "C"
