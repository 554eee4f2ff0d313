// Attention of one query row per sequence and head over the paged cache.
//
//   out = sum_t softmax_t(scale q . K_t) V_t over the sequence's tokens.
//
// Two thin matrix products per sequence and key-value head, with the up to 16
// query heads that share it as columns: S^T = K Q^T (rows = tokens) and
// O^T = V^T P^T (rows = head elements).  What bounds them is the cache's
// bytes; the kernel is built around one pass over those.
//
// * A wave works alone on 32 tokens at a time (no barrier in the loop): K and
//   V go from memory to registers, never through LDS.  The 16x16x32 MFMA
//   wants 8 consecutive k per lane, and which token or element is "row i" or
//   "step k" is free as long as both operands agree, so K's rows are assigned
//   so that the scores a lane receives are those of the 8 tokens whose
//   probabilities it has to supply to the second product: the softmax'd
//   scores are packed to bf16 in place, with no exchange between lanes.
// * V arrives with a token's head elements side by side in a lane, and a lane
//   holds 8 tokens: pairs of tokens are interleaved with one byte permute per
//   two values to form V^T's rows.
// * Codes become bf16 on the way (hardware conversions; MX scales go into
//   them), exactly for every row that kv_write stores.  An FP8 row's f32 scale multiplies its score (K) or its
//   probability (V) in f32.
// * Scores stay in the exponent's base 2.  The reference maximum m of a head
//   is only raised when a score exceeds it by more than 8: the probabilities
//   stay below 2^8 times the wave's first, their f32 sums and bf16 roundings
//   do not care, and most tiles need no exchange for a maximum and no pass
//   over the accumulators.  Sums, maxima and accumulators are f32.
// * What multiplies V is the probability times a power of two, 2^-8 over the
//   tokens that may take part (known on the host), which the result's
//   division takes out again: no weight then passes 1 over their number, and
//   no sum of finite V passes the largest of them.  (Exact, where the same
//   shift of m, which costs no product, rounds score - m in larger steps:
//   log-sum-exps were up to ten times further off.)
// * A probability goes into the second product as the sum of two bf16, its
//   rounding and what that left (2^-16 of it in all): with one alone the
//   result's error against float64 is 1.4 times that of its own rounding to
//   bf16.  The matrix units are idle most of the time (the twice as many
//   products cost 0 to 3 %).
// * Work: the tiles of 128 tokens of all (sequence, key-value head) pairs laid
//   end to end are cut into equal shares, one per workgroup, whatever the
//   lengths are; every workgroup finds its share from seq_lens itself, so
//   nothing is planned on the host.  A pair cut between workgroups is joined
//   by whichever of them finishes last, from f32 parts, in the order of the
//   parts (the same bits whatever finishes last).
//
// Measured on MI355X: 48 sequences of 8192 to 16384 bf16 tokens (8 heads of
// 128, 32 query heads, 2.4 GB) 400 us, 6.0 TB/s; 64 sequences of 1 to 8191 in
// MXFP8 110 us (5.2 TB/s); one of 131072 in FP8 53 us (5.2 TB/s); 256 of 0 to
// 515 in bf16 with 16 heads of 64 60 us (4.5 TB/s); one of 333 tokens 8.2 us.
#include <cmath>

#include "kv_common.h"
#include "rows.h"

namespace hum {

struct KvAttnParams {
  const uint8_t* cache;
  int64_t unit;
  int32_t num_pages, kv_heads, group, head_tiles, page_shift;  // group: query heads per key-value head
  const uint16_t* q;
  int64_t q_ts, q_hs;
  const int32_t* table;
  int64_t table_stride;
  int32_t max_pages, batch, window;
  const int32_t* seq_lens;
  float scale_log2;  // scale * log2(e)
  float down, up;    // the power of two on V's weights, and its reciprocal
  uint16_t* out;
  float* lse;
  uint32_t* count;  // arrival counters (3 kAttnWgs, in the workspace's header), zero between calls
  float* part;      // kSlots slots per workgroup
  uint32_t part_bytes;
  int32_t part_heads;  // heads of a slot: m, l and O rows
  int32_t wgs;         // workgroups of one head tile
};

constexpr int kWaves = 4;                  // of a workgroup
constexpr int kThreads = 64 * kWaves;
constexpr int kTile = 32 * kWaves;         // tokens of a workgroup tile
constexpr int kAttnWgs = 512;   // most workgroups: two on every CU
constexpr int kSlots = 4;       // of a workgroup: its two parts, and the joins of a group of parts that it leads
constexpr int kJoin = 8;        // parts read at once when a cut pair is joined
constexpr int kDevScope = 16;   // sc1: through to memory, around the XCD's L2 (parts cross XCDs)

// Where a lane's pieces of a row lie.
template <int FMT, int D>
struct AttnTile {
  using U = KvUnit<FMT, D>;
  static constexpr int kRow = U::kRow;
  static constexpr int kKB = kRow / 4 < 16 ? kRow / 4 : 16;  // bytes of one K load
  static constexpr int kKL = kRow / 4 / kKB;                 // K loads per row and lane
  static constexpr int kKE = kKB * D / kRow;                 // elements of one K load
  static constexpr int kChunks = D / 32;                     // MFMA steps of a score
  static constexpr int kVN = D >= 128 ? D / 128 : 1;         // V loads per row and lane
  static constexpr int kVE = D >= 128 ? 8 : 4;               // elements of one V load
  static constexpr int kVB = kVE * kRow / D;                 // its bytes
  static constexpr int kVW = kVB < 4 ? 1 : kVB / 4;          // words of a V load
};

template <int B>
__device__ __forceinline__ void load_bytes(const uint8_t* p, uint32_t* o) {
  if constexpr (B == 16) {
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = v[i];
  } else if constexpr (B == 8) {
    const u32x2_t v = *reinterpret_cast<const u32x2_t*>(p);
    o[0] = v[0];
    o[1] = v[1];
  } else if constexpr (B == 4) {
    o[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (B == 2) {
    o[0] = *reinterpret_cast<const uint16_t*>(p);
  }
}

// N / 2 words of bf16 pairs from N codes.
template <int FMT, int N>
__device__ __forceinline__ void to_bf16(const uint32_t* w, float scale, uint32_t* o) {
  if constexpr (FMT == HUM_ACT_BF16) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) o[i] = w[i];
  } else if constexpr (FMT == HUM_ACT_MXFP4) {
    const u32x4_t v = e2m1x8_to_bf16(w[0], scale);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) o[i] = v[i];
  } else {
    const u32x2_t c = {w[0], N > 4 ? w[N > 4] : 0u};
    const u32x4_t v = e4m3x8_to_bf16(c, scale);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) o[i] = v[i];
  }
}

// Byte i of w, an E8M0 code, as the scale operand of the conversions.  They
// read its exponent field only, so that code 0 (2^-127, an f32 zero) is right
// too: checked for every code of E4M3 and E2M1 and every scale whose product
// bf16 holds.
__device__ __forceinline__ float mx_scale_bits(uint32_t w, int i) {
  return __uint_as_float((i < 3 ? w << (23 - 8 * i) : w >> 1) & 0x7F800000u);
}

__device__ __forceinline__ f32x4_t mfma_bf16(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0,
                                                 0, 0);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// What turns sums with reference maximum m into sums with the larger one.
// Where m is -inf nothing has been added (the sums are zero), or only NaN,
// which has to stay.
__device__ __forceinline__ float rescale(float m, float larger) {
  return m == larger || m == -__builtin_inff() ? 1.0f : exp2_fast(m - larger);
}

// A sequence's tokens [lo, n) and its tiles.
struct SeqSpan {
  int32_t lo, n, first;  // first: token of the first tile
  int32_t tiles;         // at least one (an empty row is written too)
  __device__ __forceinline__ SeqSpan(const KvAttnParams& p, int32_t len) {
    const int32_t most = p.max_pages << p.page_shift;
    n = len < 0 ? 0 : len > most ? most : len;
    lo = p.window > 0 && n > p.window ? n - p.window : 0;
    first = lo & ~(kTile - 1);
    tiles = (n - first + kTile - 1) / kTile;
    tiles = tiles < 1 ? 1 : tiles;
  }
};

// One (sequence, key-value head), for a workgroup's 16 query heads of it.
struct AttnItem {
  int32_t b, hk;
  SeqSpan seq;
};

// Scalar loads: the lengths and the block table do not change under the call.
typedef const __attribute__((address_space(4))) int32_t* scalar_i32_t;
__device__ __forceinline__ scalar_i32_t scalar_ptr(const int32_t* p) { return (scalar_i32_t)(uintptr_t)p; }

// 16 bytes at any 2-byte boundary.
struct __attribute__((packed, aligned(2))) Bytes16 {
  uint32_t w[4];
};

// Inclusive sum over the wave's lanes: inside each row of 16, then row 0's
// and row 2's totals into the next row, then the lower half's into the upper.
__device__ __forceinline__ uint32_t wave_scan_add(uint32_t v) {
  auto add = [&](auto ctrl, auto rows) {
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, decltype(rows)::value, 0xF, false);
  };
  using std::integral_constant;
  add(integral_constant<int, 0x111>{}, integral_constant<int, 0xF>{});  // row_shr:1
  add(integral_constant<int, 0x112>{}, integral_constant<int, 0xF>{});
  add(integral_constant<int, 0x114>{}, integral_constant<int, 0xF>{});
  add(integral_constant<int, 0x118>{}, integral_constant<int, 0xF>{});
  add(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});  // row_bcast:15
  add(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});  // row_bcast:31
  return v;
}

template <int FMT, int D>
__global__ __launch_bounds__(kThreads, FMT == HUM_ACT_BF16 && D == 256 ? 1 : 2) void kv_attention_kernel(
    const KvAttnParams p) {
  using T = AttnTile<FMT, D>;
  using U = KvUnit<FMT, D>;
  constexpr bool kFp8 = FMT == HUM_ACT_FP8_TOKEN;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, kq = lane >> 4;  // MFMA row / column, and which 8 of 32 steps
  const int page_size = 1 << p.page_shift;
  const float kNegInf = -__builtin_inff();

  // ---- this workgroup's share ------------------------------------------------
  // Lane i sums the tiles of a run of sequences; a scan over the lanes places
  // the share's first tile in one run, which is then walked.  (What this
  // costs is latency before the first load: the lengths are read once, the
  // scan stays in registers, and tiles are counted in 32 bits, which the host
  // checks.)
  // Where more than 16 query heads share a key-value head, as many
  // workgroups as that takes have the same share of the cache, on one XCD
  // (workgroups go to the eight in turn): they read it at about the same
  // time, so that all but one find it in the XCD's L2 (32 sequences of 8192
  // bf16 tokens, 2 heads of 128 with 32 query heads each: 48.8 us; one
  // workgroup after another in a share of its own, which reads the cache
  // from memory twice: 79.8).
  const int turn = (int)blockIdx.x >> 3;
  const int wg8 = p.head_tiles == 1 ? turn : (int)((uint32_t)turn / (uint32_t)p.head_tiles);
  const int wg = wg8 * 8 + ((int)blockIdx.x & 7);   // among those of its 16 query heads
  const int ht = turn - wg8 * p.head_tiles;         // which 16
  const int wg_base = ht * p.wgs;                   // of its slots and counters
  const int heads = p.group - ht * 16 < 16 ? p.group - ht * 16 : 16;  // live columns
  const int items_per_seq = p.kv_heads;
  const int run = (p.batch + 63) / 64;
  int32_t len = 0;  // of the lane's last sequence: the only one in batches of up to 64
  int32_t mine = 0;
  for (int i = 0; i < run; ++i) {
    const int b = lane * run + i;
    if (b < p.batch) {
      len = p.seq_lens[b];
      mine += SeqSpan(p, len).tiles;
    }
  }
  const int32_t upto = (int32_t)wave_scan_add((uint32_t)mine);
  const int32_t total = __builtin_amdgcn_readlane(upto, 63) * items_per_seq;
  // No more workgroups than tiles (every share that counts is non-empty), and
  // where a head has up to three tiles on average, none than heads: two more
  // tiles in a row cost about as much as joining parts (16 sequences of 333
  // FP8 tokens: 9.8 us cut, 8.2 whole; one of 200: 8.3 and 6.9).  The shares
  // are equal all the same: heads are whole where their lengths are, and
  // ragged ones are cut where a border falls.
  const int32_t items = p.batch * items_per_seq, most = total <= 3 * (int64_t)items ? items : total;
  const int32_t nwg = most < p.wgs ? most : p.wgs;
  if (wg >= nwg) return;
  // shares of `each` tiles, the first `longer` of them one more
  const int32_t each = nwg == total ? 1 : (int32_t)((uint32_t)total / (uint32_t)nwg), longer = total - each * nwg;
  int32_t pos = wg * each + (wg < longer ? wg : longer);
  const int32_t end = pos + each + (wg < longer ? 1 : 0);
  // the workgroup whose share holds tile t
  auto owner = [&](int32_t t) -> int32_t {
    const int32_t border = longer * (each + 1);
    return t < border ? (int32_t)((uint32_t)t / (uint32_t)(each + 1))
                      : longer + (int32_t)((uint32_t)(t - border) / (uint32_t)each);
  };
  auto length_of = [&](int b) -> int32_t {
    return run == 1 ? __builtin_amdgcn_readlane(len, b & 63) : scalar_ptr(p.seq_lens)[b];
  };
  int tile;  // of the first item
  auto first_item = [&]() {
    const int run_lane = __builtin_ctzll(__ballot(upto * items_per_seq > pos));
    int32_t begin = __builtin_amdgcn_readlane(upto - mine, run_lane) * items_per_seq;  // first tile of sequence b
    int b = run_lane * run;
    SeqSpan seq(p, length_of(b));
    while (begin + seq.tiles * items_per_seq <= pos) {
      begin += seq.tiles * items_per_seq;
      seq = SeqSpan(p, length_of(++b));
    }
    tile = pos - begin;
    int item = 0;
    if (tile >= seq.tiles) {
      item = (int)((uint32_t)tile / (uint32_t)seq.tiles);
      tile -= item * seq.tiles;
    }
    return AttnItem{b, item, seq};
  };
  auto next_item = [&](AttnItem& i) {
    if (++i.hk == p.kv_heads) {
      i.hk = 0;
      ++i.b;
      i.seq = SeqSpan(p, length_of(i.b));
    }
  };
  AttnItem cur = first_item();

  __shared__ float s_m[2][kWaves][16], s_l[2][kWaves][16];
  __shared__ float s_o[kWaves][16][D + 4];
  __shared__ __attribute__((aligned(16))) uint16_t s_q[16][D + 8];
  __shared__ int s_last;

  // ---- loads ---------------------------------------------------------------
  // Every wave has one tile in registers and the next in flight.  The number
  // of loads between two points of the loop is fixed (a tile with nothing in
  // it reads page 0, which stays in the L2; page numbers are scalar), so that
  // the wait for K leaves V in flight, and the wait for V the next K.
  const uint32_t page_stride = (uint32_t)p.kv_heads * (uint32_t)p.unit;
  const int kg = (lane >> 2) & 3;  // the granule of 8 tokens this lane's K rows lie in
  const uint32_t in_k = (uint32_t)(kg * 8 + (lane & 3)) & (uint32_t)(page_size - 1);
  const uint32_t in_v = (uint32_t)(kq * 8) & (uint32_t)(page_size - 1);
  const uint32_t off_k = in_k * T::kRow + kq * T::kKB;
  const uint32_t off_v = ((uint32_t)page_size + in_v) * T::kRow + r * T::kVB;
  const uint32_t scales = 2u * (uint32_t)page_size * T::kRow;

  uint32_t kw[2][T::kKL][T::kKB / 4];
  uint32_t ks[2][2];  // MX: scale bytes of the two K rows
  uint32_t vw[8][T::kVN][T::kVW];
  uint32_t vs[T::kVN][2];  // MX: scale bytes of the 8 tokens
  float kf[8], vf[8];      // FP8: row scales of the 8 tokens

  // A tile on its way: the units its two halves of 16 tokens lie in.
  struct Fetch {
    int32_t t0;
    const uint8_t *u0, *u1;
    bool ok0, ok1;
  };
  auto load_k = [&](const Fetch& f) {
    const uint8_t* u = kg >= 2 ? f.u1 : f.u0;
    const uint32_t in = (uint32_t)f.t0 & (uint32_t)(page_size - 1);
    const uint8_t* row = u + (in * T::kRow + off_k);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int j = 0; j < T::kKL; ++j) load_bytes<T::kKB>(row + s * 4 * T::kRow + j * 4 * T::kKB, kw[s][j]);
      if constexpr (U::kMx) load_bytes<U::kScale>(u + (scales + (in + in_k + s * 4) * U::kScale), ks[s]);
    }
    if constexpr (kFp8) {  // (of the tokens whose scores the lane receives)
      const uint8_t* sc = (kq >= 2 ? f.u1 : f.u0) + (scales + (in + in_v) * 4);
      load_bytes<16>(sc, reinterpret_cast<uint32_t*>(kf));
      load_bytes<16>(sc + 16, reinterpret_cast<uint32_t*>(kf + 4));
    }
  };
  auto load_v = [&](const Fetch& f) {
    const uint8_t* u = kq >= 2 ? f.u1 : f.u0;
    const uint32_t in = (uint32_t)f.t0 & (uint32_t)(page_size - 1);
    const uint8_t* row = u + (in * T::kRow + off_v);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < T::kVN; ++j) load_bytes<T::kVB>(row + i * T::kRow + j * 16 * T::kVB, vw[i][j]);
    if constexpr (kFp8) {
      const uint8_t* sc = u + (scales + (page_size + in + in_v) * 4);
      load_bytes<16>(sc, reinterpret_cast<uint32_t*>(vf));
      load_bytes<16>(sc + 16, reinterpret_cast<uint32_t*>(vf + 4));
    }
    if constexpr (U::kMx) {
      const uint8_t* sc = u + (scales + (U::kScale + (r * T::kVE) / 32) * page_size + in + in_v);
#pragma unroll
      for (int j = 0; j < T::kVN; ++j) load_bytes<8>(sc + j * 4 * page_size, vs[j]);
    }
  };

  // The fetch runs two tiles ahead of the arithmetic, through the items:
  // page numbers of one tile, then its K and V.
  AttnItem ft = cur;
  int ft_tile = tile;
  int32_t ft_left = end - pos;
  struct Pages {
    int32_t t0, lo, p0, p1;
    const uint8_t* base;
  };
  auto fetch_pages = [&]() -> Pages {
    Pages g;
    g.t0 = ft.seq.first + wave * 32 + ft_tile * kTile;
    g.lo = ft.seq.lo;
    g.base = p.cache + (int64_t)ft.hk * p.unit;
    g.p0 = g.p1 = -1;
    if (ft_left > 0) {
      const scalar_i32_t table = scalar_ptr(p.table + ft.b * p.table_stride);
      if (g.t0 < ft.seq.n) g.p0 = table[g.t0 >> p.page_shift];
      if (g.t0 + 16 < ft.seq.n) g.p1 = table[(g.t0 + 16) >> p.page_shift];
      --ft_left;
      if (++ft_tile == ft.seq.tiles && ft_left > 0) {
        ft_tile = 0;
        next_item(ft);
      }
    }
    return g;
  };
  // a page outside the cache, or none: read page 0 instead, masked
  auto resolve = [&](const Pages& g) -> Fetch {
    Fetch f;
    f.t0 = g.t0;
    f.ok0 = (uint32_t)g.p0 < (uint32_t)p.num_pages && g.t0 + 16 > g.lo;
    f.ok1 = (uint32_t)g.p1 < (uint32_t)p.num_pages && g.t0 + 32 > g.lo;
    f.u0 = g.base + (uint64_t)(f.ok0 ? (uint32_t)g.p0 : 0u) * page_stride;
    f.u1 = g.base + (uint64_t)(f.ok1 ? (uint32_t)g.p1 : 0u) * page_stride;
    return f;
  };

  // The query rows go through LDS: the next item's are loaded while this one
  // runs and stored when it ends.
  constexpr int kQN = 16 * (D / 8) > kThreads ? 16 * (D / 8) / kThreads : 1;  // 16-byte pieces of a thread
  u32x4_t qn[kQN];
  auto load_q = [&](const AttnItem& w) {
    const uint16_t* q = p.q + w.b * p.q_ts + (int64_t)(w.hk * p.group + ht * 16) * p.q_hs;
#pragma unroll
    for (int i = 0; i < kQN; ++i) {
      int h = (threadIdx.x + i * kThreads) / (D / 8);
      h = h < heads ? h : heads - 1;  // (dead columns repeat a live row and are never stored)
      const Bytes16 v = *reinterpret_cast<const Bytes16*>(q + h * p.q_hs + (threadIdx.x % (D / 8)) * 8);
      qn[i] = u32x4_t{v.w[0], v.w[1], v.w[2], v.w[3]};
    }
  };
  auto stage_q = [&]() {
#pragma unroll
    for (int i = 0; i < kQN; ++i) {
      const int h = (threadIdx.x + i * kThreads) / (D / 8);
      if (h < 16) *reinterpret_cast<u32x4_t*>(&s_q[h][(threadIdx.x % (D / 8)) * 8]) = qn[i];
    }
  };
  // MFMA B operand of step c: column = head r, steps = the elements that a
  // lane's K loads bring
  auto q_frag = [&](int c) -> u32x4_t {
    constexpr int kPer = T::kKE / 8;
    const int d0 = (c / kPer) * 4 * T::kKE + kq * T::kKE + (c % kPer) * 8;
    return *reinterpret_cast<const u32x4_t*>(&s_q[r][d0]);
  };

  load_q(cur);
  Pages pages = fetch_pages();
  Fetch ahead = resolve(pages);
  load_k(ahead);
  load_v(ahead);
  pages = fetch_pages();
  stage_q();
  int buf = 0;
  __syncthreads();

  while (true) {
    const int q_head = cur.hk * p.group + ht * 16;
    const int32_t share = end - pos;
    const int tile_end = cur.seq.tiles - tile < share ? cur.seq.tiles : tile + share;
    const int32_t left = share - (tile_end - tile);
    AttnItem nxt = cur;
    if (left > 0) next_item(nxt);

    u32x4_t qf[D == 256 ? 1 : T::kChunks];
    if constexpr (D < 256) {
#pragma unroll
      for (int c = 0; c < T::kChunks; ++c) qf[c] = q_frag(c);
    }
    load_q(nxt);

    f32x4_t acc[T::kVN * T::kVE];
#pragma unroll
    for (int i = 0; i < T::kVN * T::kVE; ++i) acc[i] = f32x4_t{0, 0, 0, 0};
    float m = kNegInf, m_safe = 0.0f, l = 0.0f;

    int t = tile;
    do {
      const int32_t t0 = ahead.t0;
      const bool ok0 = ahead.ok0, ok1 = ahead.ok1;
      ahead = resolve(pages);
      pages = fetch_pages();
      // scores: rows 4 kq + j of sub-tile s are tokens 8 kq + 4 s + j
      float x[8];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        f32x4_t c4 = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < T::kChunks; ++c) {
          constexpr int kPer = T::kKE / 8;
          constexpr int kW = T::kKB / 4 / kPer;  // code words of a chunk
          float sc = 1.0f;
          if constexpr (U::kMx) {
            // (the word is known at compile time, the byte goes by the lane)
            const int g0 = (c / kPer) * 4 * T::kKE / 32;
            sc = __uint_as_float(((ks[s][g0 / 4] >> (8 * ((g0 & 3) + kq * T::kKE / 32))) & 0xFFu) << 23);
          }
          uint32_t o[4];
          to_bf16<FMT, 8>(&kw[s][c / kPer][(c % kPer) * kW], sc, o);
          u32x4_t q;
          if constexpr (D == 256) q = q_frag(c);
          else q = qf[c];
          c4 = mfma_bf16(u32x4_t{o[0], o[1], o[2], o[3]}, q, c4);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[s * 4 + j] = c4[j] * p.scale_log2;
          if constexpr (kFp8) x[s * 4 + j] *= kf[s * 4 + j];
        }
      }
      // tokens outside the span or on a page outside the cache
      if (__builtin_expect(!(ok0 && ok1 && t0 >= cur.seq.lo && t0 + 32 <= cur.seq.n), 0)) {
        const bool page_ok = kq >= 2 ? ok1 : ok0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int32_t tok = t0 + kq * 8 + i;
          if (!(page_ok && tok >= cur.seq.lo && tok < cur.seq.n)) {
            x[i] = kNegInf;
            // whatever the cache holds there: 0 * NaN is NaN
            vf[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < T::kVN; ++j) {
#pragma unroll
              for (int w = 0; w < T::kVW; ++w) vw[i][j][w] = 0;
              if constexpr (U::kMx) vs[j][i >> 2] &= ~(0xFFu << (8 * (i & 3)));
            }
          }
        }
      }
      load_k(ahead);
      __builtin_amdgcn_sched_barrier(0);
      float top = x[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) top = __builtin_fmaxf(top, x[i]);
      if (__ballot(top > m + 8.0f)) {
        top = __builtin_fmaxf(top, __shfl_xor(top, 16));
        top = __builtin_fmaxf(top, __shfl_xor(top, 32));
        const float mn = __builtin_fmaxf(m, top);
        const float a = rescale(m, mn);
        m = mn;
        m_safe = mn == kNegInf ? 0.0f : mn;
        l *= a;
#pragma unroll
        for (int i = 0; i < T::kVN * T::kVE; ++i) acc[i] *= a;
      }
      float pr[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        pr[i] = exp2_fast(x[i] - m_safe);
        l += pr[i];
        pr[i] *= p.down;
        if constexpr (kFp8) pr[i] *= vf[i];
      }
      // probabilities as the sum of two bf16 (16 significant bits)
      u32x4_t pb, pl;
#pragma unroll
      for (int i = 0; i < 4; ++i) pb[i] = f32x2_to_bf16x2_bits(pr[2 * i], pr[2 * i + 1]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        pl[i] = f32x2_to_bf16x2_bits(pr[2 * i] - bf16_bits_to_f32(pb[i] & 0xFFFF),
                                     pr[2 * i + 1] - __uint_as_float(pb[i] & 0xFFFF0000u));
#pragma unroll
      for (int j = 0; j < T::kVN; ++j) {
        uint32_t w[8][T::kVE / 2];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float sc = 1.0f;
          if constexpr (U::kMx) sc = mx_scale_bits(vs[j][i >> 2], i & 3);
          to_bf16<FMT, T::kVE>(vw[i][j], sc, w[i]);
        }
#pragma unroll
        for (int e = 0; e < T::kVE; ++e) {
          // element e of tokens 2 i, 2 i + 1: their low or high halves
          const uint32_t sel = e & 1 ? 0x07060302u : 0x05040100u;
          u32x4_t a;
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = __builtin_amdgcn_perm(w[2 * i + 1][e / 2], w[2 * i][e / 2], sel);
          acc[j * T::kVE + e] = mfma_bf16(a, pb, acc[j * T::kVE + e]);
          acc[j * T::kVE + e] = mfma_bf16(a, pl, acc[j * T::kVE + e]);
        }
      }
      load_v(ahead);
      __builtin_amdgcn_sched_barrier(0);
    } while (++t < tile_end);

    // ---- join the waves ----------------------------------------------------
    // (s_m and s_l alternate between two buffers, s_o is written only after
    // every wave has read it: no barrier is needed after the rows are out)
    auto waves_m = [&](int h) {
      float top = s_m[buf][0][h];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) top = __builtin_fmaxf(top, s_m[buf][w][h]);
      return top;
    };
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (kq == 0) {
      s_m[buf][wave][r] = m;
      s_l[buf][wave][r] = l;
    }
    __syncthreads();
    {
      const float top = waves_m(r);
      const float a = rescale(m, top);
      if (r < heads) {
        // accumulator (j, e), register i: element j * 128 + (4 kq + i) * kVE + e
#pragma unroll
        for (int j = 0; j < T::kVN; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < T::kVE; e += 4) {
              float4 v;
              v.x = acc[j * T::kVE + e][i] * a;
              v.y = acc[j * T::kVE + e + 1][i] * a;
              v.z = acc[j * T::kVE + e + 2][i] * a;
              v.w = acc[j * T::kVE + e + 3][i] * a;
              *reinterpret_cast<float4*>(&s_o[wave][r][j * 128 + (4 * kq + i) * T::kVE + e]) = v;
            }
      }
    }
    stage_q();  // (every wave is past its last read of the rows)
    __syncthreads();
    auto waves_l = [&](int h, float top) {
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
        sum += s_l[buf][w][h] * rescale(s_m[buf][w][h], top);
      return sum;
    };
    auto waves_o = [&](int h, int d) {
      f32x4_t o = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(&s_o[w][h][d]);
        o += f32x4_t{v.x, v.y, v.z, v.w};
      }
      return o;
    };
    // the finished row of head h, elements d .. d + 3
    auto store_out = [&](int h, int d, f32x4_t o, float top, float sum) {
      const int64_t row = (int64_t)cur.b * p.kv_heads * p.group + q_head + h;
      const float inv = p.up / sum;
      u32x2_t w = {f32x2_to_bf16x2_bits(o[0] * inv, o[1] * inv), f32x2_to_bf16x2_bits(o[2] * inv, o[3] * inv)};
      if (sum == 0.0f) w = u32x2_t{0, 0};
      *reinterpret_cast<u32x2_t*>(p.out + row * D + d) = w;
      if (d == 0 && p.lse) p.lse[row] = sum == 0.0f ? kNegInf : (top + __log2f(sum)) * 0.6931471805599453f;
    };
    if (tile == 0 && tile_end == cur.seq.tiles) {
      for (int i = threadIdx.x * 4; i < heads * D; i += 4 * kThreads) {
        const int h = i / D, d = i - h * D;
        const float top = waves_m(h), sum = waves_l(h, top);
        store_out(h, d, waves_o(h, d), top, sum);
      }
    } else {
      // The workgroups first .. last hold a part of this item each, joined by
      // whichever arrives last.  It reads kJoin parts per thread at once, and
      // has threads for `lanes` parts of every element; more than two such
      // rounds of parts are joined in groups first, whose joins are then
      // joined (a round of reads costs about half of a level: storing, the
      // arrival and reading again).
      const int32_t begin = pos - tile;
      const int w0 = __builtin_amdgcn_readfirstlane(owner(begin));
      const int nseg = __builtin_amdgcn_readfirstlane(owner(begin + cur.seq.tiles - 1)) - w0 + 1, seg = wg - w0;
      const __amdgpu_buffer_rsrc_t rp =
          __builtin_amdgcn_make_buffer_rsrc(p.part, (short)0, (int)p.part_bytes, 0x00020000);
      const uint32_t part_floats = (uint32_t)p.part_heads * (D + 2);
      // Of a workgroup's slots, 0 is the part of an item that its share begins
      // inside, 1 of one that it begins; 2 and 3 the joins of the groups of
      // parts that those lead.
      auto slot = [&](int sg, bool joined) {
        return (uint32_t)((wg_base + w0 + sg) * kSlots + (sg == 0 ? 1 : 0) + (joined ? 2 : 0)) * part_floats * 4;
      };
      auto put = [&](uint32_t at, int h, int d, f32x4_t o, float top, float sum) {
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, o), rp, at + (h * D + d) * 4, 0, kDevScope);
        if (d == 0) {
          const u32x2_t ml = {__float_as_uint(top), __float_as_uint(sum)};
          __builtin_amdgcn_raw_buffer_store_b64(ml, rp, at + (p.part_heads * D + 2 * h) * 4, 0, kDevScope);
        }
      };
      // whether this workgroup is the last of n to arrive at a counter, which
      // is left at zero; what each stored before is in memory by then
      auto arrive = [&](int counter, int n) -> bool {
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (threadIdx.x == 0) {
          const uint32_t old = __hip_atomic_fetch_add(p.count + counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          const int is_last = old + 1 == (uint32_t)n;
          if (is_last) __hip_atomic_store(p.count + counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          s_last = is_last;
        }
        __syncthreads();
        return s_last != 0;
      };
      // joins the slots of segments sg, sg + step, ... (n of them), four
      // elements per thread; threads to spare take every groups-th of them
      auto join = [&](int sg, int step, int n, bool joined, auto&& sink) {
        const int units = heads * (D / 4);
        const int groups = units >= kThreads ? 1 : kThreads / units;
        float* s_j = &s_o[0][0][0];  // [kThreads][6]: the groups' top, sum, o
        for (int i0 = 0; i0 < units; i0 += kThreads) {
          const int grp = groups == 1 ? 0 : (int)threadIdx.x / units;
          const int i = i0 + (int)threadIdx.x - grp * units;
          const bool live = grp < groups && i < units;
          const int h = i / (D / 4), d = (i - h * (D / 4)) * 4;
          float top = kNegInf, sum = 0.0f;
          f32x4_t o = {0, 0, 0, 0};
          if (live) {
            for (int g = grp; g < n; g += groups * kJoin) {
              u32x2_t ml[kJoin];
              f32x4_t go[kJoin];
#pragma unroll
              for (int k = 0; k < kJoin; ++k) {
                const int gk = g + k * groups;
                if (gk < n) {
                  const uint32_t at = slot(sg + gk * step, joined);
                  ml[k] = __builtin_amdgcn_raw_buffer_load_b64(rp, at + (p.part_heads * D + 2 * h) * 4, 0, kDevScope);
                  go[k] = __builtin_bit_cast(
                      f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rp, at + (h * D + d) * 4, 0, kDevScope));
                } else {
                  ml[k] = u32x2_t{__float_as_uint(kNegInf), 0u};
                  go[k] = f32x4_t{0, 0, 0, 0};
                }
              }
              float mn = top;
#pragma unroll
              for (int k = 0; k < kJoin; ++k) mn = __builtin_fmaxf(mn, __uint_as_float(ml[k][0]));
              const float ao = rescale(top, mn);
              sum *= ao;
              o *= ao;
#pragma unroll
              for (int k = 0; k < kJoin; ++k) {
                const float ag = rescale(__uint_as_float(ml[k][0]), mn);
                sum += __uint_as_float(ml[k][1]) * ag;
                o += go[k] * ag;
              }
              top = mn;
            }
          }
          if (groups > 1) {
            float* j = s_j + threadIdx.x * 6;
            j[0] = top;
            j[1] = sum;
#pragma unroll
            for (int k = 0; k < 4; ++k) j[2 + k] = o[k];
            __syncthreads();
            if (grp == 0) {
              for (int k = 1; k < groups; ++k) {
                const float* v = s_j + (threadIdx.x + k * units) * 6;
                const float mn = __builtin_fmaxf(top, v[0]);
                const float ao = rescale(top, mn), ag = rescale(v[0], mn);
                sum = sum * ao + v[1] * ag;
                o = o * ao + f32x4_t{v[2], v[3], v[4], v[5]} * ag;
                top = mn;
              }
            }
          }
          if (live && grp == 0) sink(h, d, o, top, sum);
        }
      };
      for (int i = threadIdx.x * 4; i < heads * D; i += 4 * kThreads) {
        const int h = i / D, d = i - h * D;
        const float top = waves_m(h), sum = waves_l(h, top);
        put(slot(seg, false), h, d, waves_o(h, d), top, sum);
      }
      // counters: of an item at its first workgroup; of a group at the slot
      // of the part that leads it, after those
      const int lanes = heads * (D / 4) >= kThreads ? 1 : kThreads / (heads * (D / 4));
      const int round = kJoin * lanes;
      int counter = wg_base + w0, sg = 0, step = 1, n = nseg, size = 0;
      bool joined = false;  // whether the parts are joins of groups
      if (nseg > 2 * round) {
        size = 8;
        while (size < round || size * 2 * round < nseg) size *= 2;
        sg = seg & ~(size - 1);
        n = nseg - sg < size ? nseg - sg : size;
        counter = kAttnWgs + 2 * (wg_base + w0 + sg) + (sg == 0 ? 1 : 0);
      }
      while (arrive(counter, n)) {
        const bool final = size == 0 || joined;
        const uint32_t to = slot(sg, true);
        join(sg, step, n, joined, [&](int h, int d, f32x4_t o, float top, float sum) {
          if (final) store_out(h, d, o, top, sum);
          else put(to, h, d, o, top, sum);
        });
        if (final) break;
        joined = true;
        counter = wg_base + w0;
        sg = 0;
        step = size;
        n = (nseg + size - 1) / size;
      }
    }
    // ---- next item -------------------------------------------------------------
    if (left <= 0) return;
    pos = end - left;
    tile = 0;
    cur = nxt;
    buf ^= 1;
  }
}

// Blocks of 16 query heads that share a key-value head.
static int attn_head_tiles(const hum_kv_desc* d, int32_t num_q_heads) {
  return (num_q_heads / d->num_kv_heads + 15) / 16;
}

// Workgroups of a call, per block of 16 query heads: never more than there can be tiles.  One on every CU
// where there are fewer heads (of all sequences) than kAttnWgs and a wave's
// tile is large enough to keep the memory busy (rows of 128 bytes and more;
// E2M1 codes take too many instructions a byte for one wave per SIMD): fewer
// parts to join (one sequence of 131072 FP8 tokens, 8 heads of 128: 57.3 us
// with 512, 54.1 with 256; 48 bf16 sequences, 384 heads: 405 and 401), and
// the bf16 kernel of 256-wide heads fits a CU once.  Two with more heads,
// where a second workgroup works while the first ends one head and begins
// the next (64 ragged sequences, 512 heads: 110 us with 512, 118 with 256;
// 256 short ones, 4096 heads: 59 and 82), and with small rows (32 sequences
// in MXFP4 of 128-wide heads, 512 MiB: 5.3 TB/s with 512, 4.0 with 256).
static int attn_wgs(const hum_kv_desc* d, int32_t num_q_heads, int64_t batch, int64_t max_pages) {
  const int64_t tiles = max_pages * d->page_size / kTile + 1, items = batch * d->num_kv_heads;
  const int head_tiles = attn_head_tiles(d, num_q_heads);
  const bool once = d->fmt == HUM_ACT_BF16 && d->head_dim == 256;
  const bool wide = d->fmt != HUM_ACT_MXFP4 && d->head_dim * (d->fmt == HUM_ACT_BF16 ? 2 : 1) >= 128;
  int64_t most = (once || (wide && items * head_tiles < kAttnWgs) ? kAttnWgs / 2 : kAttnWgs) / head_tiles;
  if (most > 8) most &= ~7;  // the grid is made of eights
  return (int)(items * tiles >= most ? most : items * tiles < 1 ? 1 : items * tiles);
}

// Heads of a slot (even: slots stay 16-byte aligned), and the slots' bytes.
static int attn_part_heads(const hum_kv_desc* d, int32_t num_q_heads) {
  const int group = num_q_heads / d->num_kv_heads;
  return group >= 16 ? 16 : (group + 1) & ~1;
}
static size_t attn_part_bytes(const hum_kv_desc* d, int32_t num_q_heads, int64_t batch, int64_t max_pages) {
  return (size_t)attn_wgs(d, num_q_heads, batch, max_pages) * attn_head_tiles(d, num_q_heads) * kSlots * attn_part_heads(d, num_q_heads) *
         (d->head_dim + 2) * 4;
}

static hum_status check_attn(const hum_kv_desc* d, int32_t num_q_heads, int64_t batch, int64_t max_pages, KvLayout* l) {
  hum_status st = kv_layout(d, l);
  if (st != HUM_OK) return st;
  if (num_q_heads < 1 || num_q_heads % d->num_kv_heads || num_q_heads / d->num_kv_heads > 1024)
    return set_error(HUM_ERR_INVALID_ARG, "num_q_heads must be 1 .. 1024 times num_kv_heads");
  if (batch < 0 || batch > 0xFFFF) return set_error(HUM_ERR_INVALID_ARG, "batch must be 0 .. 65535");
  if (max_pages < 0 || max_pages > ((int64_t)1 << 30) / d->page_size)
    return set_error(HUM_ERR_INVALID_ARG, "max_pages must be >= 0, sequences at most 2^30 tokens");
  if (batch * d->num_kv_heads * (max_pages * d->page_size / kTile + 1) >= (int64_t)1 << 31)
    return set_error(HUM_ERR_UNSUPPORTED, "batch x num_kv_heads x max_pages x page_size must stay below 2^38");
  return HUM_OK;
}

}  // namespace hum

using namespace hum;

extern "C" {

size_t hum_kv_attention_workspace_bytes(const hum_kv_desc* desc, int32_t num_q_heads, int64_t batch,
                                        int64_t max_pages) {
  clear_error();
  KvLayout l;
  if (check_attn(desc, num_q_heads, batch, max_pages, &l) != HUM_OK) return 0;
  return HUM_WS_HEADER_BYTES + attn_part_bytes(desc, num_q_heads, batch, max_pages);
}

hum_status hum_kv_attention(const hum_kv_desc* desc, const void* cache, size_t cache_bytes, int32_t num_q_heads,
                            int64_t batch, const void* q_bf16, int64_t q_ts, int64_t q_hs, const int32_t* block_table,
                            int64_t table_stride, int64_t max_pages, const int32_t* seq_lens, int64_t window,
                            float scale, void* out_bf16, float* lse, void* workspace, size_t ws_bytes, void* stream) {
  clear_error();
  KvLayout l;
  hum_status st = check_attn(desc, num_q_heads, batch, max_pages, &l);
  if (st != HUM_OK) return st;
  if (window < 0) return set_error(HUM_ERR_INVALID_ARG, "window must be >= 0");
  const float scale_log2 = (float)((double)scale * 1.4426950408889634);
  if (!(scale_log2 - scale_log2 == 0.0f)) return set_error(HUM_ERR_INVALID_ARG, "scale must be finite (times log2 e too)");
  if (batch == 0) return HUM_OK;
  if (!cache || !q_bf16 || (max_pages && !block_table) || !seq_lens || !out_bf16 || !workspace)
    return set_error(HUM_ERR_INVALID_ARG, "NULL pointer");
  if (reinterpret_cast<uintptr_t>(cache) % 16) return set_error(HUM_ERR_INVALID_ARG, "the cache must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(workspace) % 16)
    return set_error(HUM_ERR_INVALID_ARG, "the workspace must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(q_bf16) % 2 || reinterpret_cast<uintptr_t>(out_bf16) % 16)
    return set_error(HUM_ERR_INVALID_ARG, "q must be aligned to its elements, out to 16 bytes");
  // (scalar loads drop an address's low bits)
  if ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(seq_lens) | reinterpret_cast<uintptr_t>(lse)) % 4)
    return set_error(HUM_ERR_INVALID_ARG, "block_table, seq_lens and lse must be aligned to their elements");
  if (cache_bytes < (size_t)l.bytes)
    return set_error(HUM_ERR_WORKSPACE, "cache of %zu bytes, the description takes %lld", cache_bytes, (long long)l.bytes);
  const size_t need = hum_kv_attention_workspace_bytes(desc, num_q_heads, batch, max_pages);
  if (ws_bytes < need) return set_error(HUM_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws_bytes, need);
  // What is written may not lie in what other workgroups read; a row of out
  // may be its own query (it is stored when the last reader has passed it).
  const int64_t row = (int64_t)desc->head_dim * 2, rows = batch * num_q_heads;
  const Rows q_rows{(int64_t)(intptr_t)q_bf16, batch, num_q_heads, (wide_t)q_ts * 2, (wide_t)q_hs * 2, row};
  const bool same = q_bf16 == out_bf16 && (batch == 1 || q_ts == (int64_t)num_q_heads * desc->head_dim) &&
                    (num_q_heads == 1 || q_hs == desc->head_dim);
  const Rows in[4] = {bytes_at(cache, l.bytes), bytes_at(seq_lens, batch * 4),
                      Rows{(int64_t)(intptr_t)block_table, batch, 1, (wide_t)table_stride * 4, 0, max_pages * 4}, q_rows};
  const Rows out[3] = {bytes_at(workspace, (int64_t)need), bytes_at(lse, lse ? rows * 4 : 0), bytes_at(out_bf16, rows * row)};
  for (int i = 0; i < 3; ++i) {
    bool bad = false;
    for (int j = 0; j < 4; ++j) bad |= !(same && i == 2 && j == 3) && overlap(out[i], in[j]) != Overlap::kNo;
    for (int j = 0; j < i; ++j) bad |= overlap(out[i], out[j]) != Overlap::kNo;
    if (bad) return set_error(HUM_ERR_INVALID_ARG, "out, lse and the workspace must not overlap the inputs or one another");
  }
  KvAttnParams p{};
  p.cache = static_cast<const uint8_t*>(cache);
  p.unit = l.unit;
  p.num_pages = (int32_t)desc->num_pages;
  p.kv_heads = desc->num_kv_heads;
  p.group = num_q_heads / desc->num_kv_heads;
  p.head_tiles = attn_head_tiles(desc, num_q_heads);
  p.wgs = attn_wgs(desc, num_q_heads, batch, max_pages);
  p.page_shift = __builtin_ctz((unsigned)desc->page_size);
  p.q = static_cast<const uint16_t*>(q_bf16);
  p.q_ts = q_ts;
  p.q_hs = q_hs;
  p.table = block_table;
  p.table_stride = table_stride;
  p.max_pages = (int32_t)max_pages;
  p.batch = (int32_t)batch;
  p.window = (int32_t)(window < ((int64_t)1 << 30) ? window : (int64_t)1 << 30);
  p.seq_lens = seq_lens;
  p.scale_log2 = scale_log2;
  const int64_t all = max_pages * desc->page_size, most = window > 0 && window < all ? window : all;
  const int shift = 8 + (most > 1 ? 64 - __builtin_clzll((uint64_t)most - 1) : 0);
  p.down = std::ldexp(1.0f, -shift);
  p.up = std::ldexp(1.0f, shift);
  p.out = static_cast<uint16_t*>(out_bf16);
  p.lse = lse;
  p.count = static_cast<uint32_t*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + HUM_WS_HEADER_BYTES);
  p.part_bytes = (uint32_t)attn_part_bytes(desc, num_q_heads, batch, max_pages);
  p.part_heads = attn_part_heads(desc, num_q_heads);
  hipStream_t s = static_cast<hipStream_t>(stream);
  kv_dispatch(desc, [&](auto fmt, auto dim) {
    kv_attention_kernel<decltype(fmt)::value, decltype(dim)::value><<<(p.wgs + 7) / 8 * 8 * p.head_tiles, kThreads, 0, s>>>(p);
  });
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return set_error(HUM_ERR_HIP, "kv_attention launch: %s", hipGetErrorString(err));
  return HUM_OK;
}

}  // extern "C"
