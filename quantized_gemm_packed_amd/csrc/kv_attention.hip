// Attention of one query row per sequence and head over the paged cache.
//
//   out = sum_t softmax_t(scale q . K_t) V_t over the sequence's tokens.
//
// One workgroup per (sequence, query head); its waves take every fourth
// token, a lane D / 64 elements of the row, with the softmax's running
// maximum and sum per wave in f32; the waves join through LDS.
#include "kv_common.h"

namespace hum {

struct KvAttnParams {
  const uint8_t* cache;
  int64_t unit, num_pages;
  int32_t kv_heads, q_heads, page_shift;
  const uint16_t* q;
  int64_t q_ts, q_hs;
  const int32_t* table;
  int64_t table_stride, max_pages;
  const int32_t* seq_lens;
  int64_t window;
  float scale;
  uint16_t* out;
  float* lse;
};

// Elements at .. at + N - 1 of a row as f32.
template <int FMT, int D, int N>
__device__ __forceinline__ void kv_row(const uint8_t* unit, int which, int at_token, int page_size, int at,
                                       float (&x)[N]) {
  using U = KvUnit<FMT, D>;
  const uint8_t* row = unit + (int64_t)(which * page_size + at_token) * U::kRow;
  const uint8_t* scales = unit + (int64_t)2 * page_size * U::kRow + which * page_size * U::kScale;
  float sc = 1.0f;
  if constexpr (FMT == HUM_ACT_FP8_TOKEN) sc = reinterpret_cast<const float*>(scales)[at_token];
  if constexpr (U::kMx)
    sc = e8m0_to_f32(which ? scales[(at / 32) * page_size + at_token] : scales[at_token * U::kScale + at / 32]);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (FMT == HUM_ACT_BF16) {
      x[i] = bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(row)[at + i]);
    } else if constexpr (FMT == HUM_ACT_MXFP4) {
      const uint32_t c = (row[(at + i) / 2] >> (4 * ((at + i) & 1))) & 15u;
      x[i] = bf16_bits_to_f32(e2m1x8_to_bf16(c, 1.0f)[0] & 0xFFFF) * sc;
    } else {
      const u32x2_t w = {row[at + i], 0};
      x[i] = bf16_bits_to_f32(e4m3x8_to_bf16(w, 1.0f)[0] & 0xFFFF) * sc;
    }
  }
}

template <int FMT, int D>
__global__ __launch_bounds__(256) void kv_attention_kernel(const KvAttnParams p) {
  constexpr int N = D / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t b = blockIdx.x;
  const int h = blockIdx.y, hk = h / (p.q_heads / p.kv_heads);
  const int page_size = 1 << p.page_shift;
  int64_t n = p.seq_lens[b];
  n = n < 0 ? 0 : n > (p.max_pages << p.page_shift) ? (p.max_pages << p.page_shift) : n;
  const int64_t lo = p.window > 0 && n > p.window ? n - p.window : 0;
  const uint16_t* qr = p.q + b * p.q_ts + h * p.q_hs + lane * N;
  float q[N], acc[N] = {};
#pragma unroll
  for (int i = 0; i < N; ++i) q[i] = bf16_bits_to_f32(qr[i]) * p.scale;
  float m = -__builtin_inff(), l = 0.0f;
  for (int64_t t = lo + wave; t < n; t += 4) {
    const int64_t page = p.table[b * p.table_stride + (t >> p.page_shift)];
    if ((uint64_t)page >= (uint64_t)p.num_pages) continue;
    const uint8_t* unit = p.cache + (page * p.kv_heads + hk) * p.unit;
    float x[N];
    kv_row<FMT, D, N>(unit, 0, (int)(t & (page_size - 1)), page_size, lane * N, x);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) s += q[i] * x[i];
#pragma unroll
    for (int w = 1; w < 64; w *= 2) s += __shfl_xor(s, w);
    const float mn = __builtin_fmaxf(m, s);
    const float a = m == mn ? 1.0f : __expf(m - mn), e = __expf(s - mn);
    kv_row<FMT, D, N>(unit, 1, (int)(t & (page_size - 1)), page_size, lane * N, x);
    l = l * a + e;
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = acc[i] * a + e * x[i];
    m = mn;
  }
  __shared__ float sm[4], sl[4], so[4][D];
  if (lane == 0) {
    sm[wave] = m;
    sl[wave] = l;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) so[wave][lane * N + i] = acc[i];
  __syncthreads();
  const float top = __builtin_fmaxf(__builtin_fmaxf(sm[0], sm[1]), __builtin_fmaxf(sm[2], sm[3]));
  float total = 0.0f, w[4];
  for (int i = 0; i < 4; ++i) {
    w[i] = sm[i] == -__builtin_inff() ? 0.0f : __expf(sm[i] - top);
    total += sl[i] * w[i];
  }
  for (int d = threadIdx.x; d < D; d += 256) {
    float o = 0.0f;
    for (int i = 0; i < 4; ++i) o += so[i][d] * w[i];
    p.out[(b * p.q_heads + h) * D + d] = (uint16_t)f32_to_bf16_bits(total == 0.0f ? 0.0f : o / total);
  }
  if (p.lse && threadIdx.x == 0) p.lse[b * p.q_heads + h] = total == 0.0f ? -__builtin_inff() : top + __logf(total);
}

}  // namespace hum

using namespace hum;

extern "C" {

size_t hum_kv_attention_workspace_bytes(const hum_kv_desc* desc, int32_t num_q_heads, int64_t batch,
                                        int64_t max_pages) {
  clear_error();
  KvLayout l;
  if (kv_layout(desc, &l) != HUM_OK) return 0;
  if (num_q_heads < 1 || num_q_heads % desc->num_kv_heads || batch < 0 || max_pages < 0) {
    set_error(HUM_ERR_INVALID_ARG, "num_q_heads must be a multiple of num_kv_heads, batch and max_pages >= 0");
    return 0;
  }
  return HUM_WS_HEADER_BYTES;
}

hum_status hum_kv_attention(const hum_kv_desc* desc, const void* cache, size_t cache_bytes, int32_t num_q_heads,
                            int64_t batch, const void* q_bf16, int64_t q_ts, int64_t q_hs, const int32_t* block_table,
                            int64_t table_stride, int64_t max_pages, const int32_t* seq_lens, int64_t window,
                            float scale, void* out_bf16, float* lse, void* workspace, size_t ws_bytes, void* stream) {
  clear_error();
  KvLayout l;
  hum_status st = kv_layout(desc, &l);
  if (st != HUM_OK) return st;
  if (num_q_heads < 1 || num_q_heads % desc->num_kv_heads || num_q_heads / desc->num_kv_heads > 1024)
    return set_error(HUM_ERR_INVALID_ARG, "num_q_heads must be a multiple of num_kv_heads (at most 1024 times)");
  if (batch < 0 || batch > 0xFFFF) return set_error(HUM_ERR_INVALID_ARG, "batch must be 0 .. 65535");
  if (max_pages < 0 || max_pages > (int64_t)0x7FFFFFFF / desc->page_size)
    return set_error(HUM_ERR_INVALID_ARG, "max_pages must be >= 0, sequences below 2^31 tokens");
  if (window < 0) return set_error(HUM_ERR_INVALID_ARG, "window must be >= 0");
  if (!(scale - scale == 0.0f)) return set_error(HUM_ERR_INVALID_ARG, "scale must be finite");
  if (batch == 0) return HUM_OK;
  if (!cache || !q_bf16 || (max_pages && !block_table) || !seq_lens || !out_bf16 || !workspace)
    return set_error(HUM_ERR_INVALID_ARG, "NULL pointer");
  if (reinterpret_cast<uintptr_t>(cache) % 16) return set_error(HUM_ERR_INVALID_ARG, "the cache must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(q_bf16) % 2 || reinterpret_cast<uintptr_t>(out_bf16) % 16)
    return set_error(HUM_ERR_INVALID_ARG, "q must be aligned to its elements, out to 16 bytes");
  if (cache_bytes < (size_t)l.bytes)
    return set_error(HUM_ERR_WORKSPACE, "cache of %zu bytes, the description takes %lld", cache_bytes, (long long)l.bytes);
  const size_t need = hum_kv_attention_workspace_bytes(desc, num_q_heads, batch, max_pages);
  if (ws_bytes < need) return set_error(HUM_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws_bytes, need);
  KvAttnParams p{};
  p.cache = static_cast<const uint8_t*>(cache);
  p.unit = l.unit;
  p.num_pages = desc->num_pages;
  p.kv_heads = desc->num_kv_heads;
  p.q_heads = num_q_heads;
  p.page_shift = __builtin_ctz((unsigned)desc->page_size);
  p.q = static_cast<const uint16_t*>(q_bf16);
  p.q_ts = q_ts;
  p.q_hs = q_hs;
  p.table = block_table;
  p.table_stride = table_stride;
  p.max_pages = max_pages;
  p.seq_lens = seq_lens;
  p.window = window;
  p.scale = scale;
  p.out = static_cast<uint16_t*>(out_bf16);
  p.lse = lse;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)batch, (unsigned)num_q_heads);
  kv_dispatch(desc, [&](auto fmt, auto dim) {
    kv_attention_kernel<decltype(fmt)::value, decltype(dim)::value><<<grid, 256, 0, s>>>(p);
  });
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return set_error(HUM_ERR_HIP, "kv_attention launch: %s", hipGetErrorString(err));
  return HUM_OK;
}

}  // extern "C"
