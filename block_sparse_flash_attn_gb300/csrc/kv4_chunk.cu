// Attention of a chunk of new tokens over the 4-bit cache, one token to whole
// prompts, with scores that may be capped, biased by distance and opened to a
// prefix.
//
// Query t of the count c new tokens of a sequence of length n sits at i = n - c + t
// and sees the cached tokens j <= i, and those of the prefix, j < f.  With keys and
// values decoded as step * code + least (kv4.cu):
//   x_j = scale q . k_j;  x_j = cap tanh(x_j / cap);  x_j -= slope |i - j|
//   p = softmax(x),  o = sum_j p_j v_j,  lse = ln sum_j exp(x_j)
//   a query that sees nothing, or lies behind the count: o = 0, lse = -inf.
//
// Bound: the tensor cores where there are many rows (4 D multiply-adds a query and
// key), the codes' expansion where there are few.  So a CTA takes 256 query rows of
// one key/value head, its G query heads' tokens interleaved (row = token G + head:
// a tile ends where its last token does), and expands each tile of 128 tokens
// once for all of them, to operands of tcgen05 in shared memory:
//
// - A code in bits 0-3 or 4-7 of an fp16 is a subnormal number; so a mask and one fused
//   multiply-add with a power of two more take two codes to two operands.
// - K without a rounding that counts.  An fp16 holds step (code - 8) exactly (8 bits
//   times 3), and the rest of a key is one number a group, c = least + 8 step:
//     q . k = sum_d q_d step (code_d - 8) + sum_groups c sum_d q_d.
//   The second sum is one more 16-channel step of the same product: c and the sums
//   of q are split into two fp16 each, (q hi, q lo, q hi) beside (c hi, c hi, c lo),
//   off by 2^-22 of a product.  Queries are bf16, exact in fp16 beside their
//   row's largest; keys are taken beside the largest of 32 tokens (held to 2^-17 of it,
//   exactly where a group's step is 2^-10 of it or more); both are powers of two that
//   the softmax puts back.  So scores and lse are those of 32-bit products, at the cost of
//   a ninth step for 8.
// - V in fp16, rounded once (2^-11), beside a power of two that the CTA takes from its
//   first step (1 to 2^-20): the mean exponent of its groups of channels goes to 2^-10.
//   Where a group of 32 tokens passes 2^-6 there, or 2^-14 the other way, those tokens are
//   taken in bf16 (2^-8), their weights too.  Weights are off by that rounding, or by 2^-25
//   beside a row's largest weight of one or more.
//
// Work of a CTA (896 threads, one CTA an SM, 218 KB of shared memory for heads of 128):
//   warps 0-7, 8-15   softmax of the first and the second 128 rows: 16 rows a warp, two
//                     threads a row, a half of the tokens and of the channels each
//   warps 16-19       the keys' expansion, 32 tokens a warp
//   warps 20-23       the values'
//   warps 24, 25      issue S = Q K^T of a row tile each; 24 owns the tensor memory
//   warps 26, 27      issue O += P V
// Tensor memory: S of both row tiles (128 columns each; the weights replace the
// scores they come from) and O of both.  While one tile's softmax runs, the tensor
// core works for the other.
//
// Up to 128 rows a key/value head both row tiles hold the same rows and take every other
// step, so that one's chain of products and softmax runs beside the other's.
// Few rows and long contexts: the tokens are cut into `splits` ranges, a CTA each.
// Partial results (maximum, sum, O) of ranges and tiles are joined, in order, by a second
// launch.
// Every wait is bounded; a wait that runs out is reported by bsattn_kv4_status.
#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda_fp16.h>

#include "kv4.cuh"
#include "ptx.cuh"

namespace bsattn {
namespace {

constexpr int kChunkThreads = 896;
constexpr int kSoftmaxWarps = 8;            // a row tile
constexpr int kTileRows = 128;              // rows of a softmax tile: lanes of tensor memory
constexpr int kCtaRows = 2 * kTileRows;
constexpr int kKeys = 128;                  // tokens that are expanded at once: a step
// Tokens of a score product: a step, or a half of it (SCORED).  With whole steps a row tile's
// chain of products and softmax is hidden by the other tile's, which takes turns with it;
// with halves by its own other half too, and scores stay in registers while they are
// capped and biased, at a third more shared-memory reads (Q is read for 64 tokens).  4096
// tokens behind 61440: 3.5 ms as steps, 4.0 as halves; capped scores, 1024 behind 15360:
// 541 and 432 us (390 since).
template <bool SCORED>
constexpr int kPiece = SCORED ? 64 : 128;
template <bool SCORED>
constexpr int kPieces = kKeys / kPiece<SCORED>;
constexpr int kStages = 2;                  // of the expanded K and V
constexpr int kInfos = 4;                   // steps whose ChunkInfo is kept
constexpr int kWarpK = 16, kWarpV = 20, kWarpScores = 24, kWarpValues = 26;
// 512 x 96 + 256 x 48 + 128 x 24 = 896 x 72 registers; the expansion of four groups a row
// wants more: 512 x 88 + 256 x 64 + 128 x 24.  4096 tokens behind 61440 in groups of 32:
// 3.6 ms, with the former 4.0; 1024 behind 15360 in groups of 128: 275 us, with the latter 309.
template <int NG, bool SCORED>
constexpr int kSoftmaxRegs = SCORED && NG < 4 ? 96 : 88;
template <int NG, bool SCORED>
constexpr int kExpandRegs = SCORED && NG < 4 ? 48 : 64;
constexpr int kIssueRegs = 24;
constexpr uint32_t kTmemColumns = 512;
constexpr float kLagBits = 8.0f;            // a row's reference may lie 2^8 below its maximum
constexpr float kMostSum = 32768.0f;        // of a step's weights: each then fits fp16
constexpr int kJoinWarps = 4;
constexpr int kMostSplits = 64;             // ranges of the tokens
constexpr int kMostParts = 2 * kMostSplits;  // of a row: both row tiles may hold it
constexpr unsigned long long kDrainLimitNs = 200ull * 1000 * 1000;

struct ChunkParams {
  Kv4View c;
  const uint16_t* q;  // [B][H][T][D]
  const int* table;
  int64_t table_stride;
  int columns;
  const int* lengths;
  const int* counts;   // null: T each
  const int* prefix;   // null: none
  const float* slopes; // null: none
  int B, H, T, G;
  int items;           // row tiles (of kCtaRows) a key/value head
  int splits;
  int twin;            // both row tiles hold the same rows (up to kTileRows)
  float scale_log2;    // |scale| log2 e, above 0
  float sign;          // of the scale
  float cap_log2;      // cap log2 e; 0: no cap
  void* out;
  float* lse;
  int out_f32;
  float* partial;      // [B * Hkv * items * splits][2 tiles][kTileRows * (D + 2)]; null: none
  unsigned long long timeout_ns;
};

// What the softmax needs of 32 tokens of a step.
struct TokenInfo {
  float factor;     // the keys' power of two
  uint32_t there;   // bits 0, 1: the first, the second 16 tokens are there
  uint32_t v_bf16;  // the values' type
  uint32_t unused;
};

struct __align__(16) ChunkBars {
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t q_full[2];
  uint64_t turn[2];  // the other row tile's softmax of a step is about over
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // by row tile and piece of a step
  // (a step's slot is taken again four steps on: two steps after its scores were read)
  uint64_t info_full[kInfos];
  uint64_t drain[4];
  TokenInfo info[kInfos][4];
  int nan_from[4];  // by group of channels: the first token whose values are not numbers
  uint32_t tmem_base;
  int abort_flag;
  float v_scale;      // what O is multiplied by
  int v_exponents[4][2];  // of each V warp's first step: sum, number
  uint2 factors[8][4 * 32];  // by warp, group and token: what codes are multiplied by, and a summand
};

template <int D>
struct ChunkCfg {
  static constexpr int kBoxes = D / 64;  // of 64 channels, 128 bytes a row, swizzled
  static constexpr int kBoxBytes = 128 * 128;
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  static constexpr int kSumBytes = 128 * 32;  // the 16 channels of the group sums
  static constexpr int kQ = 0;
  static constexpr int kQSums = kQ + 2 * kTileBytes;
  static constexpr int kKSums = kQSums + 2 * kSumBytes;
  static constexpr int kK = kKSums + kStages * kSumBytes;
  static constexpr int kV = kK + kStages * kTileBytes;
  static constexpr int kBars = kV + kStages * kTileBytes;
  static constexpr int kSmem = kBars + (int)sizeof(ChunkBars) + 1024;
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(kKSums % 1024 == 0 && kK % 1024 == 0, "swizzled tiles begin at multiples of 1024");
  static constexpr uint32_t kTmemS = 0, kTmemO = 256;
  static constexpr uint32_t kIdescO16 = idesc_f16kind_f32(128, D, true, false, true);
  static constexpr uint32_t kIdescOBf = idesc_f16kind_f32(128, D, true, false, false);
};

// K-major operand of 16 channels without a swizzle: 8 rows of 16 bytes are a core
// matrix; the next 8 rows follow 128 bytes on, the next 8 channels 2048.
__device__ __forceinline__ uint64_t sums_desc(uint32_t at) {
  uint64_t d = 0;
  d |= (uint64_t)((at >> 4) & 0x3FFFu);
  d |= (uint64_t)(2048 >> 4) << 16;
  d |= (uint64_t)(128 >> 4) << 32;
  d |= 1ull << 46;
  return d;
}

// What a CTA works on.
struct ChunkWork {
  int b, h, split;
  int len, count, first_pos;  // tokens, new ones, position of the first new one
  int open;                   // positions below it are seen by all
  int keys;                   // tokens that the table has room for
  int rows;                   // G * count: rows that have a query
  int row0;                   // the CTA's first
  int64_t slot;               // partial result
  int j0;                     // the range's first 128 tokens: step s has j0 + total - 1 - s
  int steps[2];               // of each row tile: the last ones, or every other one
  int total;
  bool twin;

  __device__ __forceinline__ int first_row(int tile) const { return row0 + (twin ? 0 : tile * kTileRows); }
  // the tile's n-th step
  __device__ __forceinline__ int step_of(int tile, int n) const {
    return twin ? 2 * n + tile : total - steps[tile] + n;
  }

  __device__ __forceinline__ int first_key(int s) const { return (j0 + total - 1 - s) * kKeys; }
  __device__ __forceinline__ int limit(int t) const {  // last position that token t sees
    return min(max(first_pos + t, open - 1), keys - 1);
  }
};

__device__ __forceinline__ ChunkWork chunk_work(const ChunkParams& p) {
  ChunkWork w;
  // row tiles with the longest contexts first
  const int item = p.items - 1 - (int)blockIdx.z;
  const unsigned bh = blockIdx.y, splits = p.splits;
  w.split = blockIdx.x;
  w.b = bh / (unsigned)p.c.Hkv;
  w.h = bh - w.b * p.c.Hkv;
  // (all loads at once, whatever there is)
  const int len = load(p.lengths + w.b), count = load((p.counts ? p.counts : p.lengths) + w.b),
            open = load((p.prefix ? p.prefix : p.lengths) + w.b);
  w.slot = ((int64_t)bh * p.items + item) * p.splits + w.split;
  w.len = max(len, 0);
  w.count = p.counts ? min(max(count, 0), p.T) : p.T;
  w.first_pos = w.len - w.count;
  w.open = p.prefix ? max(open, 0) : 0;
  const int64_t room = (int64_t)p.columns * p.c.page;
  w.keys = (int)min((int64_t)w.len, room);
  if (w.len > room && threadIdx.x == 0) p.c.report();
  w.rows = p.G * w.count;
  w.row0 = item * kCtaRows;
  w.twin = p.twin != 0;
  int most[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int first = w.first_row(i);
    const int last = min(first + kTileRows, w.rows) - 1;
    const int lim = first < w.rows ? w.limit(last / p.G) : -1;
    most[i] = lim >= 0 ? lim / kKeys + 1 : 0;
  }
  const int all = max(most[0], most[1]);
  w.j0 = 0;
  int j1 = all;
  if (splits > 1) {  // (all: at most 2^24, splits: 2^6)
    w.j0 = (unsigned)all * w.split / splits;
    j1 = (unsigned)all * (w.split + 1) / splits;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) w.steps[i] = max(min(j1, most[i]) - w.j0, 0);
  w.total = max(w.steps[0], w.steps[1]);
  if (w.twin) w.steps[0] = (w.total + 1) / 2, w.steps[1] = w.total / 2;
  return w;
}

__device__ __forceinline__ bool wait_all(const uint64_t* bar, uint32_t parity,
                                         volatile int* abort_flag, const ChunkParams& p) {
  const bool ok = wait_bounded(smem_u32(bar), parity, abort_flag, p.c.status, p.timeout_ns);
  return __all_sync(0xffffffffu, ok);
}

// Waits, with a limit of its own, for all products that this warp issued.
__device__ __forceinline__ void drain(uint64_t* bar) {
  if (elect_one()) mma_commit(smem_u32(bar));
  __syncwarp();
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(smem_u32(bar), 0)) {
    if (globaltimer_ns() - t0 > kDrainLimitNs) return;
  }
}

// ---------------------------------------------------------------------------
// warps 16-23: codes to operands
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t half_bits(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }
__device__ __forceinline__ __half2 half2_of(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
// The eight codes of a word times a step and plus a number, as four pairs of fp16 (codes
// 0 and 4, 1 and 5, ...): low = 2^24 step, high = 2^20 step.
__device__ __forceinline__ void expand_codes(uint32_t w, __half2 low, __half2 high, __half2 plus,
                                             uint32_t (&x)[4]) {
  const uint32_t y = w >> 8;
  x[0] = half_bits(__hfma2(half2_of(w & 0x000F000Fu), low, plus));
  x[1] = half_bits(__hfma2(half2_of(w & 0x00F000F0u), high, plus));
  x[2] = half_bits(__hfma2(half2_of(y & 0x000F000Fu), low, plus));
  x[3] = half_bits(__hfma2(half2_of(y & 0x00F000F0u), high, plus));
}
__device__ __forceinline__ uint32_t half_pair(__half lo, __half hi) {
  return half_bits(__halves2half2(lo, hi));
}

// A group's scales; a group with one that is not finite stands for NaN.
struct Scales {
  float step, least;
  bool finite;
  __device__ __forceinline__ explicit Scales(uint32_t word)
      : step(bf16_lo(word)), least(bf16_hi(word)),
        finite((word & 0x7F80u) != 0x7F80u && (word & 0x7F800000u) != 0x7F800000u) {
    if (!finite) step = least = 0.0f;
  }
  // the largest magnitude that the group stands for
  __device__ __forceinline__ float most() const {
    return fmaxf(fabsf(least), fabsf(fmaf(15.0f, step, least)));
  }
};

// What a warp of either kind needs to expand its 32 tokens of a step.  A lane is a token
// where steps and minima are concerned, and a 16-byte piece (32 codes) of a row where
// codes are; what it works out of the former passes through shared memory.
template <int D, int NG>
struct Expander {
  using C = ChunkCfg<D>;
  static constexpr int LR = D / 32;       // lanes a row
  static constexpr int RL = 32 / LR;      // rows a load
  static constexpr int NL = 32 / RL;      // loads a warp and step
  static constexpr int GL = D / NG / 32;  // lanes a group
  const ChunkParams& p;
  const ChunkWork& w;
  const uint4* codes;
  const uint32_t* scales;
  uint2* factors;
  int lane, warp, row, log16;
  uint32_t at;         // where its first 16 bytes go
  uint4 word[NL];
  uint32_t scale[NG];  // of token `lane`

  __device__ __forceinline__ Expander(const ChunkParams& pp, const ChunkWork& ww, ChunkBars* bars,
                                      bool keys)
      : p(pp), w(ww), lane(threadIdx.x & 31), warp((threadIdx.x >> 5) & 3) {
    // eight lanes in a row hold eight rows' same piece: their stores meet 32 banks
    row = lane % RL;
    const int piece = lane / RL;
    codes = reinterpret_cast<const uint4*>(keys ? p.c.k_codes : p.c.v_codes) + row * LR + piece;
    scales = reinterpret_cast<const uint32_t*>(keys ? p.c.k_scales : p.c.v_scales);
    factors = bars->factors[(keys ? 0 : 4) + warp];
    log16 = p.c.log_page - 4;
    const int r = warp * 32 + row;
    at = (D == 128 ? (uint32_t)(piece >> 1) * C::kBoxBytes : 0u) + r * 128 +
         ((4 * (piece & 1) ^ (r & 7)) << 4);
  }
  // Lanes 0 to 15: where the first 16 of the warp's tokens of step s are, in units of 16
  // rows; the others: the second 16; -1: nowhere.
  __device__ __forceinline__ int look_up(int s) const {
    if (s >= w.total) return -1;
    const int pos = w.first_key(s) + warp * 32 + (lane & 16);
    if (pos >= w.keys) return -1;
    const int pg = load(p.table + w.b * p.table_stride + (pos >> p.c.log_page));  // (keys end with it)
    if (pg < 0 || pg >= p.c.pages) {
      p.c.report();
      return -1;
    }
    return ((pg * p.c.Hkv + w.h) << log16) + ((pos & (p.c.page - 1)) >> 4);
  }
  // Where a step's codes are (look_up's answer, for the warp).
  struct Place {
    int r16[2], there;  // 16 rows each; tokens that there are, or more
    bool all;
  };
  __device__ __forceinline__ Place place_of(int where, int s) const {
    Place x;
    x.there = s < w.total ? w.keys - (w.first_key(s) + warp * 32) : 0;
    x.r16[0] = __shfl_sync(0xffffffffu, where, 0);
    x.r16[1] = __shfl_sync(0xffffffffu, where, 16);
    x.all = x.there >= 32 && (x.r16[0] | x.r16[1]) >= 0;
    return x;
  }
  __device__ __forceinline__ void load_word(const Place& x, int i) {
    const int h = i * RL / 16;  // (RL divides 16)
    word[i] = make_uint4(0, 0, 0, 0);
    if (x.all || (x.r16[h] >= 0 && i * RL + row < x.there))
      word[i] = load(codes + (int64_t)x.r16[h] * (16 * LR) + (i * RL & 15) * LR);
  }
  __device__ __forceinline__ void load_scales(int where, int s) {
    const int there = s < w.total ? w.keys - (w.first_key(s) + warp * 32) : 0;
    const uint32_t* mine = scales + ((int64_t)where * 16 + (lane & 15)) * NG;
    const bool seen = where >= 0 && lane < there;
    if constexpr (NG == 4) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (seen) v = load(reinterpret_cast<const uint4*>(mine));
      scale[0] = v.x, scale[1] = v.y, scale[2] = v.z, scale[3] = v.w;
    } else if constexpr (NG == 2) {
      uint2 v = make_uint2(0, 0);
      if (seen) v = load(reinterpret_cast<const uint2*>(mine));
      scale[0] = v.x, scale[1] = v.y;
    } else {
      scale[0] = seen ? load(mine) : 0u;
    }
  }
  __device__ __forceinline__ void load_step(int where, int s) {
    const Place x = place_of(where, s);
#pragma unroll
    for (int i = 0; i < NL; ++i) load_word(x, i);
    load_scales(where, s);
  }
  // of this lane's codes of load i
  __device__ __forceinline__ uint2 factors_of(int i) const {
    return factors[(NG > 1 ? lane / RL / GL * 32 : 0) + i * RL + row];
  }
  // f(word, place) for the four words of load i
  template <typename F>
  __device__ __forceinline__ void each(int i, uint32_t tile, F f) const {
    const uint32_t n[4] = {word[i].x, word[i].y, word[i].z, word[i].w};
#pragma unroll
    for (int c = 0; c < 4; ++c) f(n[c], tile + ((at ^ (c << 4)) + i * (RL * 128)));
  }
  // all codes, in fp16: token `lane` has factors (2^24 step, 2^20 step), summand
  __device__ __forceinline__ void put(int g, float step, float plus) {
    const uint32_t both = pack_f16x2(step * 16777216.0f, step * 1048576.0f);
    factors[g * 32 + lane] = make_uint2(both, pack_f16x2(plus, plus));
  }
  // (each word's place is taken at once by the next step's)
  __device__ __forceinline__ void expand(uint32_t tile, const Place& next) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const uint2 v = factors_of(i);
      const __half2 low = half2_of(__byte_perm(v.x, v.x, 0x1010)),
                    high = half2_of(__byte_perm(v.x, v.x, 0x3232)), plus = half2_of(v.y);
      each(i, tile, [&](uint32_t n, uint32_t to) {
        uint32_t y[4];
        expand_codes(n, low, high, plus, y);
        st_shared_v4(to, y[0], y[1], y[2], y[3]);
      });
      load_word(next, i);
    }
  }
};

template <int D, int NG>
__device__ void run_expand_keys(const ChunkParams& p, const ChunkWork& w, ChunkBars* bars,
                                uint32_t base, volatile int* abort_flag) {
  using C = ChunkCfg<D>;
  Expander<D, NG> e(p, w, bars, true);
  const int lane = e.lane, warp = e.warp;
  int where = e.look_up(0), next = e.look_up(1);
  e.load_step(where, 0);
#pragma unroll 1
  for (int s = 0; s < w.total; ++s) {
    const int st = s % kStages;
    // ---- the keys' power of two
    float most = 0.0f;
#pragma unroll
    for (int g = 0; g < NG; ++g) most = fmaxf(most, Scales(e.scale[g]).most());
    const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
    // the largest goes to [2^-7, 2^-6): 2^24 of a step to 2^15.1 at most (below 2^-112:
    // times 2^105)
    const int x = min(max((int)(top >> 23), 15), 246);
    const float scale = __uint_as_float((uint32_t)(254 - 7 - x) << 23);
    const uint32_t there = __ballot_sync(0xffffffffu, where >= 0);
    if (!wait_all(&bars->k_empty[st], ((uint32_t)(s / kStages) & 1u) ^ 1u, abort_flag, p)) return;
    if (lane == 0) {
      TokenInfo* info = &bars->info[s % kInfos][warp];
      info->factor = 1.0f / scale;
      info->there = (there & 1u) | (there >> 15 & 2u);
      mbar_arrive(smem_u32(&bars->info_full[s % kInfos]));
    }
    {  // c of each group, twice its high half and once its low one
      __half hi[4] = {}, lo[4] = {};
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const Scales k(e.scale[g]);
        const float step = k.step * scale;
        e.put(g, step, step * -8.0f);
        float c = fmaf(8.0f, step, k.least * scale) * 16384.0f;
        if (!k.finite) c = __int_as_float(0x7FC00000);
        hi[g] = __float2half_rn(c);
        lo[g] = __float2half_rn(c - __half2float(hi[g]));
      }
      const uint32_t to = base + C::kKSums + st * C::kSumBytes + (warp * 32 + lane) * 16;
      if constexpr (NG == 4) {
        const uint32_t h01 = half_pair(hi[0], hi[1]), h23 = half_pair(hi[2], hi[3]);
        st_shared_v4(to, h01, h23, h01, h23);
        st_shared_v4(to + 2048, half_pair(lo[0], lo[1]), half_pair(lo[2], lo[3]), 0, 0);
      } else if constexpr (NG == 2) {
        const uint32_t h01 = half_pair(hi[0], hi[1]);
        st_shared_v4(to, h01, h01, half_pair(lo[0], lo[1]), 0);
        st_shared_v4(to + 2048, 0, 0, 0, 0);
      } else {
        st_shared_v4(to, half_pair(hi[0], hi[0]), half_pair(lo[0], lo[1]), 0, 0);
        st_shared_v4(to + 2048, 0, 0, 0, 0);
      }
    }
    e.load_scales(next, s + 1);
    __syncwarp();
    e.expand(base + C::kK + st * C::kTileBytes, e.place_of(next, s + 1));
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->k_full[st]));
    where = next;
    next = e.look_up(s + 2);
  }
}

template <int D, int NG>
__device__ void run_expand_values(const ChunkParams& p, const ChunkWork& w, ChunkBars* bars,
                                  uint32_t base, volatile int* abort_flag) {
  using C = ChunkCfg<D>;
  using E = Expander<D, NG>;
  E e(p, w, bars, false);
  const int lane = e.lane, warp = e.warp;
  int next = e.look_up(1);
  e.load_step(e.look_up(0), 0);
  float v_scale;
  // ---- the CTA's power of two
  {
    int sum = 0, n = 0;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const float most = Scales(e.scale[g]).most();
      if (most > 0.0f) sum += (int)(__float_as_uint(most) >> 23), ++n;
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) bars->v_exponents[warp][0] = sum, bars->v_exponents[warp][1] = n;
    named_bar_sync(1, 128);
    sum = n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += bars->v_exponents[i][0], n += bars->v_exponents[i][1];
    // Powers of 1 to 2^-20 only, for means of 2^-10 to 2^10: beside others the sums of large values
    // (below 2^104, 2^13 tokens, weights of 2^10) would pass 2^127, and small ones (2^-100) 2^-126.
    const int mean = n > 0 ? min(max(sum / n, 127 - 10), 127 + 10) : 127;
    v_scale = __uint_as_float((uint32_t)(254 - 10 - mean) << 23);
    if (lane == 0 && warp == 0) bars->v_scale = 1.0f / v_scale;
  }
#pragma unroll 1
  for (int s = 0; s < w.total; ++s) {
    const int st = s % kStages;
    bool fits = true;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const Scales v(e.scale[g]);
      const float most = v.most() * v_scale;
      fits = fits && most <= 0.015625f && (most >= 6.103515625e-5f || most == 0.0f);
      if (!v.finite) atomicMin(&bars->nan_from[g], w.first_key(s) + warp * 32 + lane);
    }
    const bool bf16 = !__all_sync(0xffffffffu, fits);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const Scales v(e.scale[g]);
      if (bf16)
        e.factors[g * 32 + lane] =
            make_uint2(__float_as_uint(v.step * v_scale), __float_as_uint(v.least * v_scale));
      else
        e.put(g, v.step * v_scale, v.least * v_scale);
    }
    // (the step four before this one is read: its values' stage was free a step ago)
    if (lane == 0) {
      bars->info[s % kInfos][warp].v_bf16 = bf16 ? 1u : 0u;
      mbar_arrive(smem_u32(&bars->info_full[s % kInfos]));
    }
    if (!wait_all(&bars->v_empty[st], ((uint32_t)(s / kStages) & 1u) ^ 1u, abort_flag, p)) return;
    const uint32_t tile = base + C::kV + st * C::kTileBytes;
    e.load_scales(next, s + 1);
    const auto place = e.place_of(next, s + 1);
    __syncwarp();
    if (!bf16) {
      e.expand(tile, place);
    } else {
#pragma unroll
      for (int i = 0; i < E::NL; ++i) {
        const uint2 v = e.factors_of(i);
        const float step = __uint_as_float(v.x), least = __uint_as_float(v.y);
        e.each(i, tile, [&](uint32_t n, uint32_t to) {
          uint32_t y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            y[k] = pack_bf16x2(fmaf((float)(n >> (4 * k) & 15u), step, least),
                               fmaf((float)(n >> (4 * k + 16) & 15u), step, least));
          st_shared_v4(to, y[0], y[1], y[2], y[3]);
        });
        e.load_word(place, i);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->v_full[st]));
    next = e.look_up(s + 2);
  }
}

// ---------------------------------------------------------------------------
// warps 24 and 25: the two products
// ---------------------------------------------------------------------------
// A warp a product and row tile, so that none waits behind another tile's issue.  (What the
// loops turn on is broadcast: the instruction's operands are uniform registers.)
//
// The scores of a piece replace what the product with V of the same piece read a step
// before, so they wait for that; another's softmax runs meanwhile.
template <int D, bool SCORED>
__device__ void run_scores(const ChunkParams& p, const ChunkWork& w, ChunkBars* bars,
                           uint32_t tmem, uint32_t base, volatile int* abort_flag, int tile) {
  using C = ChunkCfg<D>;
  constexpr int N = kPiece<SCORED>;
  const int total = __shfl_sync(0xffffffffu, w.total, 0);
  const int steps = __shfl_sync(0xffffffffu, w.steps[tile], 0), twin = p.twin;
  const int skip = total - steps;
  int n = 0;  // the tile's steps so far
  const uint32_t to = __shfl_sync(0xffffffffu, tmem, 0) + C::kTmemS + tile * kKeys;
  constexpr uint32_t kIdesc = idesc_f16kind_f32(128, N, false, false, true);
  const uint64_t qd = smem_desc_sw128(base + C::kQ + tile * C::kTileBytes, 16, 1024);
  const uint64_t qs = sums_desc(base + C::kQSums + tile * C::kSumBytes);
  bool ok = steps == 0 || wait_all(&bars->q_full[tile], 0, abort_flag, p);
  for (int s = 0; s < total && ok; ++s) {
    const int st = s % kStages;
    ok = wait_all(&bars->k_full[st], (uint32_t)(s / kStages) & 1u, abort_flag, p);
    const uint64_t kd = smem_desc_sw128(base + C::kK + st * C::kTileBytes, 16, 1024);
    const uint64_t ks = sums_desc(base + C::kKSums + st * C::kSumBytes);
    const bool mine = twin ? (s & 1) == tile : s >= skip;
#pragma unroll
    for (int h = 0; h < kPieces<SCORED>; ++h) {
      if (!ok || !mine) break;
      if (n > 0) ok = wait_all(&bars->pv_done[tile][h], (uint32_t)(n - 1) & 1u, abort_flag, p);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * C::kBoxBytes + (k & 3) * 32) >> 4;
          mma_ss(to + h * N, qd + off, kd + off + (h * N * 128 >> 4), kIdesc, k > 0 ? 1u : 0u);
        }
        mma_ss(to + h * N, qs, ks + (h * N * 16 >> 4), kIdesc, 1u);
        mma_commit(smem_u32(&bars->s_full[tile][h]));
      }
      __syncwarp();
    }
    n += mine ? 1 : 0;
    if (ok && elect_one()) mma_commit(smem_u32(&bars->k_empty[st]));
    __syncwarp();
  }
  drain(&bars->drain[tile]);
}

template <int D, bool SCORED>
__device__ void run_values(const ChunkParams& p, const ChunkWork& w, ChunkBars* bars,
                           uint32_t tmem, uint32_t base, volatile int* abort_flag, int tile) {
  using C = ChunkCfg<D>;
  constexpr int N = kPiece<SCORED>;
  const int total = __shfl_sync(0xffffffffu, w.total, 0);
  const int steps = __shfl_sync(0xffffffffu, w.steps[tile], 0), twin = p.twin;
  const int skip = total - steps;
  int n = 0;  // the tile's steps so far
  tmem = __shfl_sync(0xffffffffu, tmem, 0);
  const uint32_t from = tmem + C::kTmemS + tile * kKeys, to = tmem + C::kTmemO + tile * D;
  bool ok = true;
  for (int s = 0; s < total && ok; ++s) {
    const int st = s % kStages;
    ok = wait_all(&bars->v_full[st], (uint32_t)(s / kStages) & 1u, abort_flag, p);
    uint32_t bf16 = 0;  // by 32 tokens
#pragma unroll
    for (int c = 0; c < 4; ++c) bf16 |= bars->info[s % kInfos][c].v_bf16 << c;
    bf16 = __shfl_sync(0xffffffffu, bf16, 0);
    const uint64_t vd = smem_desc_sw128(base + C::kV + st * C::kTileBytes, C::kBoxBytes, 1024);
    const bool mine = twin ? (s & 1) == tile : s >= skip;
#pragma unroll
    for (int h = 0; h < kPieces<SCORED>; ++h) {
      if (!ok || !mine) break;
      ok = wait_all(&bars->p_full[tile][h], (uint32_t)n & 1u, abort_flag, p);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        // 16 tokens each; whole steps have tokens 64 on 64 columns on
        auto product = [&](int k, uint32_t idesc) {
          const int at = N == 64 ? h * N + k * 8 : (k & 3) * 8 + (k >> 2) * 64;
          mma_ts(to, from + at, vd + (uint32_t)((h * N / 16 + k) * 2048 >> 4), idesc,
                 n > 0 || h > 0 || k > 0 ? 1u : 0u);
        };
        if (bf16 == 0u) {
#pragma unroll
          for (int k = 0; k < N / 16; ++k) product(k, C::kIdescO16);
        } else {
          for (int k = 0; k < N / 16; ++k)
            product(k, bf16 >> (h * N / 32 + (k >> 1)) & 1u ? C::kIdescOBf : C::kIdescO16);
        }
        mma_commit(smem_u32(&bars->pv_done[tile][h]));
      }
      __syncwarp();
    }
    n += mine ? 1 : 0;
    if (ok && elect_one()) mma_commit(smem_u32(&bars->v_empty[st]));
    __syncwarp();
  }
  drain(&bars->drain[2 + tile]);
}

// ---------------------------------------------------------------------------
// warps 0-15: queries, softmax, results
// ---------------------------------------------------------------------------
// A softmax thread's query: a half of the channels, lanes 16 on the second.  (A thread pair a
// row, as the softmax has it.  With 16 lanes a row and maxima and sums by shuffles the first
// product waited for the queries, 13000 clocks of a CTA; 10000 now.  8 prompts of up to 2048
// tokens: 358 us, now 334.)
template <int D>
struct Query {
  static constexpr int N = D / 16;
  uint4 raw[N];
  int row, t, g;  // row of the key/value head, token, head of the group
  __device__ __forceinline__ void fetch(const ChunkParams& p, const ChunkWork& w, int first) {
    const int lane = threadIdx.x & 31;
    row = first + (lane & 15);
    t = (unsigned)row / (unsigned)p.G;
    g = row - t * p.G;
    const uint4* from =
        reinterpret_cast<const uint4*>(p.q + (((int64_t)w.b * p.H + w.h * p.G + g) * p.T + t) * D) +
        (lane >> 4) * N;
#pragma unroll
    for (int i = 0; i < N; ++i)
      raw[i] = row < w.rows ? load(from + i) : make_uint4(0, 0, 0, 0);
  }
};

// The queries as fp16 beside each row's largest (which goes to [2^14, 2^15)), channels in the
// codes' order, and the sums of their groups.  Returns the row's power of two.
template <int D, int NG>
__device__ __forceinline__ int load_queries(const ChunkParams& p, ChunkBars* bars, uint32_t base,
                                            int tile, int row_in, const Query<D>& q) {
  using C = ChunkCfg<D>;
  constexpr int N = Query<D>::N;
  constexpr int SG = NG == 4 ? 2 : 1;  // sums of a half: of two groups, one, or half a group
  const int lane = threadIdx.x & 31, half = lane >> 4, r = row_in + (lane & 15);
  uint32_t top = 0;  // (magnitudes of bf16 compare as whole numbers)
#pragma unroll
  for (int i = 0; i < N; ++i) {
    top = __vmaxu2(top, __vmaxu2(q.raw[i].x & 0x7FFF7FFFu, q.raw[i].y & 0x7FFF7FFFu));
    top = __vmaxu2(top, __vmaxu2(q.raw[i].z & 0x7FFF7FFFu, q.raw[i].w & 0x7FFF7FFFu));
  }
  top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 16));
  const float most = __uint_as_float(max(top & 0xFFFFu, top >> 16) << 16);
  // (a row with an infinity or NaN is spoiled whatever its power; one that is below 2^-112
  // stays below 2^14)
  const int sh = most > 0.0f ? min(14 + 127 - (int)(__float_as_uint(most) >> 23), 126) : 0;
  const float f = p.sign * __uint_as_float((uint32_t)(127 + sh) << 23);
  const uint64_t f2 = f2_pack(f, f);
  uint64_t sums[SG] = {};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t u[4] = {q.raw[i].x, q.raw[i].y, q.raw[i].z, q.raw[i].w};
    float x[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint64_t v = f2_mul(f2_pack(bf16_lo(u[k]), bf16_hi(u[k])), f2);
      sums[i * SG / N] = f2_add(sums[i * SG / N], v);
      f2_unpack(v, x[2 * k], x[2 * k + 1]);
    }
    const int piece = half * N + i;
    st_shared_v4(base + C::kQ + tile * C::kTileBytes + piece / 8 * C::kBoxBytes + r * 128 +
                     ((piece % 8 ^ (r & 7)) << 4),
                 pack_f16x2(x[0], x[4]), pack_f16x2(x[1], x[5]), pack_f16x2(x[2], x[6]),
                 pack_f16x2(x[3], x[7]));
  }
  float all[4] = {};  // of each group
#pragma unroll
  for (int i = 0; i < SG; ++i) {
    float a, b;
    f2_unpack(sums[i], a, b);
    const float mine = (a + b) * 6.103515625e-5f;  // (2^-14: c has 2^14)
    const float other = __shfl_xor_sync(0xffffffffu, mine, 16);
    if constexpr (NG == 1) {
      all[0] = mine + other;
    } else {
      all[i] = half ? other : mine;
      all[SG + i] = half ? mine : other;
    }
  }
  // (q hi, q lo, q hi) of NG groups each, then zeros: the lanes' halves 8 of the 16 each
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half h = __float2half_rn(all[i]);
    hi[i] = __half_as_ushort(h);
    lo[i] = __half_as_ushort(__float2half_rn(all[i] - __half2float(h)));
  }
  uint32_t y[8] = {};
#pragma unroll
  for (int k = 0; k < 3 * NG; ++k) {
    const uint32_t v = k < NG || k >= 2 * NG ? hi[k % NG] : lo[k % NG];
    y[k / 2] |= k & 1 ? v << 16 : v;
  }
  const uint32_t to = base + C::kQSums + tile * C::kSumBytes + r * 16 + half * 2048;
  if (half)
    st_shared_v4(to, y[4], y[5], y[6], y[7]);
  else
    st_shared_v4(to, y[0], y[1], y[2], y[3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(&bars->q_full[tile]));
  return sh;
}

__device__ __forceinline__ float largest32(const uint32_t (&x)[32]) {
  float a[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = fmaxf(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
#pragma unroll
  for (int c = 8; c < 32; c += 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a[i] = max3(a[i], __uint_as_float(x[c + 2 * i]), __uint_as_float(x[c + 2 * i + 1]));
  }
  return fmaxf(max3(a[0], a[1], a[2]), a[3]);
}

// The row's results to `out` and `lse`, or to the partial result.
template <int D>
__device__ __forceinline__ void write_row(const ChunkParams& p, int64_t at, const float (&x)[16],
                                          int c0) {
  const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
  if (p.out_f32) {
    uint32_t y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(x[i]);
    float* dst = static_cast<float*>(p.out) + at * D + c0;
    store32(dst, *reinterpret_cast<const uint32_t(*)[8]>(y), wide);
    store32(dst + 8, *reinterpret_cast<const uint32_t(*)[8]>(y + 8), wide);
  } else {
    uint32_t y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    store32(static_cast<uint16_t*>(p.out) + at * D + c0, y, wide);
  }
}

// What there is to write where a row tile has nothing to see.
template <int D>
__device__ __forceinline__ void write_nothing(const ChunkParams& p, const ChunkWork& w, int tile,
                                              int r) {
  const int row = w.first_row(tile) + r;
  if (row >= p.G * p.T) return;
  if (p.partial && row < w.rows) {
    float* slot = p.partial + (w.slot * 2 + tile) * (kTileRows * (D + 2)) + r;
    slot[0] = -INFINITY;
    slot[kTileRows] = 0.0f;
    return;
  }
  if (w.split != 0 || (w.twin && tile != 0)) return;
  const int t = row / p.G, g = row - t * p.G;
  const int64_t at = ((int64_t)w.b * p.H + w.h * p.G + g) * p.T + t;
  const float zero[16] = {};
#pragma unroll 1
  for (int c = 0; c < D; c += 16) write_row<D>(p, at, zero, c);
  p.lse[at] = -INFINITY;
}

// A softmax thread's row.
struct ChunkRow {
  int tile, half, row_in, row, t, g;  // row_in: the warp's first row of the tile
  bool there;                         // there is a query
  int lim, pos;                       // last position that it sees, its own
  float factor;                       // of the products, but for the keys' power of two
  float slope, inv_cap;
  uint32_t s, o;                      // its warp's part of tensor memory
  float m;       // reference: a maximum of scores (base 2) so far, or up to kLagBits below
  uint64_t sum;  // of the weights of this half, two partial sums

  // the row's new maximum: what was weighed before is to be multiplied by this
  __device__ __forceinline__ float move_to(float top, bool moves) {
    if (!moves) return 1.0f;
    const float f = ex2_approx(m - top);  // (0 from no reference)
    m = top;
    sum = f2_mul(sum, f2_pack(f, f));
    return f;
  }
  __device__ __forceinline__ float reference() const { return m == -INFINITY ? 0.0f : m; }
  // of tokens first .. first + 31 those that the row sees (pieces: bits 0, 1: 16 tokens are there)
  __device__ __forceinline__ uint32_t seen(int first, uint32_t pieces) const {
    const int last = lim - first;
    uint32_t m32 = last >= 31 ? 0xFFFFFFFFu : last < 0 ? 0u : (2u << last) - 1u;
    if (!(pieces & 1u)) m32 &= 0xFFFF0000u;
    if (!(pieces & 2u)) m32 &= 0x0000FFFFu;
    return m32;
  }
  template <int DH>
  __device__ __forceinline__ void rescale(float f) const {
#pragma unroll 1
    for (int k = 0; k < DH; k += 16) {
      uint32_t x[16];
      tmem_ld16x2_16<DH>(o + k, x);
      tmem_wait_ld();
      reg_fence(x, 16);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
      tmem_st16x2_16<DH>(o + k, x);
    }
  }
};
__device__ __forceinline__ void hide(uint32_t (&x)[32], uint32_t seen) {
#pragma unroll
  for (int i = 0; i < 32; ++i) x[i] = seen >> i & 1u ? x[i] : 0xff800000u;  // -inf
}
// (not zero: what is hidden is -inf times it)
__device__ __forceinline__ float at_least_normal(float x) { return fmaxf(x, 1.17549435e-38f); }

// 32 products to scores in base 2: `f` is their factor, d0 the distance of the first key
// from the query, `past` whether keys behind the query are seen.
__device__ __forceinline__ void score(const ChunkParams& p, const ChunkRow& r, uint32_t (&x)[32],
                                      float f, int d0, bool past) {
      if (p.cap_log2 > 0.0f) {
        const float k = f * r.inv_cap;
        float big = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; i += 2)
          big = max3(big, fabsf(__uint_as_float(x[i])), fabsf(__uint_as_float(x[i + 1])));
        // By the row's own scores: no vote, another row's leave its bits alone.  Most rows of
        // most models are near zero; 1024 tokens behind 15360, capped: 437 us without a shorter
        // polynomial for them, 390 with it (441 if it is not the first that is asked for).
        // (Not where 1 / cap leaves the factor few bits.)
        if (big * k <= kNearRange && k > 1e-30f) {
          const uint64_t k2 = f2_pack(k, k);
          const float n0 = kNear0 * p.cap_log2, n1 = kNear1 * p.cap_log2, n2 = kNear2 * p.cap_log2,
                      n3 = kNear3 * p.cap_log2;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const uint64_t y = f2_mul(f2_pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), k2),
                           u = f2_mul(y, y);
            uint64_t a = f2_fma(f2_pack(n3, n3), u, f2_pack(n2, n2));
            a = f2_fma(a, u, f2_pack(n1, n1));
            a = f2_fma(a, u, f2_pack(n0, n0));
            a = f2_mul(a, y);
            float lo, hi;
            f2_unpack(a, lo, hi);
            x[i] = __float_as_uint(lo), x[i + 1] = __float_as_uint(hi);
          }
        } else if (big * k <= kTanhRange) {
          const uint64_t k2 = f2_pack(k, k), f2 = f2_pack(f, f);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const uint64_t raw = f2_pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1]));
            const uint64_t y = f2_mul(raw, k2), u = f2_mul(y, y);
            uint64_t a = f2_fma(f2_pack(kTanh5, kTanh5), u, f2_pack(kTanh4, kTanh4));
            a = f2_fma(a, u, f2_pack(kTanh3, kTanh3));
            a = f2_fma(a, u, f2_pack(kTanh2, kTanh2));
            a = f2_fma(a, u, f2_pack(kTanh1, kTanh1));
            a = f2_fma(a, u, f2_pack(kTanh0, kTanh0));
            a = f2_mul(a, f2_mul(raw, f2));
            float lo, hi;
            f2_unpack(a, lo, hi);
            x[i] = __float_as_uint(lo), x[i + 1] = __float_as_uint(hi);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            x[i] = __float_as_uint(p.cap_log2 * tanh_any(__uint_as_float(x[i]) * k));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
      }
      if (p.slopes) {
        if (past) {  // (by the row's own place, no vote: the two forms round otherwise)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            x[i] = __float_as_uint(fmaf(-r.slope, fabsf((float)(d0 + i)), __uint_as_float(x[i])));
        } else {
          const float b0 = r.slope * (float)d0;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            x[i] = __float_as_uint(__uint_as_float(x[i]) + fmaf(r.slope, (float)i, b0));
        }
      }
}

constexpr unsigned kAll = 0xffffffffu;

// The softmax by whole steps: 64 of a row's 128 scores a thread (tokens 64 half on).
template <int D>
__device__ bool softmax_steps(const ChunkParams& p, const ChunkWork& w, ChunkBars* bars, ChunkRow& r,
                              volatile int* abort_flag) {
  const int lane = threadIdx.x & 31, tile = r.tile;
  const int steps = w.steps[tile], both = min(w.steps[0], w.steps[1]);
  // What a step needs besides its scores: read while the tensor core works on them.
  TokenInfo info[2];
  float factor[2];
  bool whole = false, any_bf16 = false, find = true;
  auto prepare = [&](int s) -> bool {
    if (!wait_all(&bars->info_full[s % kInfos], (uint32_t)(s / kInfos) & 1u, abort_flag, p))
      return false;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      info[c] = bars->info[s % kInfos][2 * r.half + c];
      factor[c] = at_least_normal(r.factor * info[c].factor);
    }
    const int rel = r.lim - (w.first_key(s) + 64 * r.half);
    whole = __all_sync(kAll, rel >= 63 && (info[0].there & info[1].there) == 3u);
    any_bf16 = __any_sync(kAll, (info[0].v_bf16 | info[1].v_bf16) != 0u);
    // Weights are formed beside the reference of the steps before, without a look for
    // the maximum; with one where their sum shows that scores rose far above it, where
    // there is no reference yet, and where scores are to be masked first (they go back to
    // tensor memory for that).  A row that has no reason of its own (`find`) keeps its
    // reference, and with it its bits, whatever the other rows of the warp have.
    find = !whole || r.m == -INFINITY;
    return true;
  };
  if (!prepare(w.step_of(tile, 0))) return false;
#pragma unroll 1
  for (int n = 0; n < steps; ++n) {
    // The row tiles' softmaxes take turns: while one has the issue slots, the tensor core
    // works for the other.  (Odd lanes wait for the turn.)
    // (Not where both hold the same few rows: 64 rows, 8 sequences of 49152 tokens, 323 us
    // with turns, 288 without.)
    const int k = n - (steps - both);  // of the steps that both have
    const bool paired = k >= 0 && !w.twin;
    const bool turns = paired && (tile == 1 || k > 0) && (threadIdx.x & 1);
    if (!wait_all(turns ? &bars->turn[tile] : &bars->s_full[tile][0],
                  (uint32_t)(turns ? (tile ? k : k - 1) : n) & 1u, abort_flag, p))
      return false;
    tc_fence_after();
    const int key0 = w.first_key(w.step_of(tile, n)) + 64 * r.half;
    uint32_t weights[32];
    bool hand = paired;  // the other tile's turn is to come
    uint64_t part;
    for (;;) {
      if (__any_sync(kAll, find)) {
        float top = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          uint32_t x[32];
          tmem_ld16x2_32<64>(r.s + 32 * c, x);
          tmem_wait_ld();
          reg_fence(x, 32);
          if (!whole) {
            hide(x, r.seen(key0 + 32 * c, c ? info[1].there : info[0].there));
            tmem_st16x2_32<64>(r.s + 32 * c, x);
          }
          top = fmaxf(top, largest32(x) * (c ? factor[1] : factor[0]));
        }
        if (!whole) tmem_wait_st();
        top = fmaxf(top, __shfl_xor_sync(kAll, top, 16));
        const bool moves = find && top > r.m + kLagBits;
        const bool any = __any_sync(kAll, moves);
        const float f = r.move_to(top, moves);
        // (O is complete: the step's scores waited for the last step's product)
        if (any && n > 0) r.template rescale<D / 2>(f);
      }
      const uint64_t nm2 = f2_pack(-r.reference(), -r.reference());
      auto weigh = [&](auto type) {
        uint64_t parts[2] = {0, 0};
        uint32_t x[2][16];
        tmem_ld16x2_16<64>(r.s, x[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // 16 at once, the next 16 on their way
          uint32_t(&now)[16] = x[c & 1];
          if (c == 3) {  // (the others hear of it about when this is done)
            if (lane == 0 && hand) mbar_arrive(smem_u32(&bars->turn[1 - tile]));
            hand = false;
          }
          tmem_wait_ld();
          reg_fence(now, 16);
          if (c < 3) tmem_ld16x2_16<64>(r.s + 16 * (c + 1), x[(c + 1) & 1]);
          const uint64_t f2 = f2_pack(factor[c / 2], factor[c / 2]);
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            float a, b;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(now[i]), __uint_as_float(now[i + 1])), f2, nm2),
                      a, b);
            a = ex2_approx(a), b = ex2_approx(b);
            parts[i / 2 & 1] = f2_add(parts[i / 2 & 1], f2_pack(a, b));
            weights[8 * c + i / 2] = pack_f16x2(a, b);
            if (decltype(type)::value && info[c / 2].v_bf16)
              weights[8 * c + i / 2] = pack_bf16x2(a, b);
          }
        }
        part = f2_add(parts[0], parts[1]);
      };
      if (any_bf16)
        weigh(std::true_type{});
      else
        weigh(std::false_type{});
      float a, b;
      f2_unpack(part, a, b);
      const bool over = !(a + b <= kMostSum);  // (NaN, too)
      if (!__any_sync(kAll, over && !find)) break;
      // (by all lanes: no short circuit around the exchange)
      const int others = __shfl_xor_sync(kAll, over ? 1 : 0, 16);
      find = find || over || others != 0;
    }
    r.sum = f2_add(r.sum, part);
    tmem_st16x2_32<64>(r.s, weights);
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[tile][0]));
    if (n + 1 < steps && !prepare(w.step_of(tile, n + 1))) return false;
  }
  return wait_all(&bars->pv_done[tile][0], (uint32_t)(steps - 1) & 1u, abort_flag, p);
}

// The softmax by half steps, scores capped and biased: 32 of a row's 64 a thread (tokens 32
// half on).
template <int D>
__device__ bool softmax_halves(const ChunkParams& p, const ChunkWork& w, ChunkBars* bars,
                               ChunkRow& r, volatile int* abort_flag) {
  constexpr int N = kPiece<true>;
  const int lane = threadIdx.x & 31, tile = r.tile;
  const int steps = w.steps[tile];
  // What a step needs besides its scores, of this thread's 32 tokens of each half: read
  // while the tensor core works on them.
  float factor[2];
  uint32_t bits = 0;  // by half: 0, 1: 16 tokens are there; 2: V is bf16
  bool plain[2], bf16[2];  // all rows see all tokens; V is bf16 for some
  auto prepare = [&](int s) -> bool {
    if (!wait_all(&bars->info_full[s % kInfos], (uint32_t)(s / kInfos) & 1u, abort_flag, p))
      return false;
    const int rel = r.lim - (w.first_key(s) + 32 * r.half);
    bits = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const TokenInfo info = bars->info[s % kInfos][2 * h + r.half];
      factor[h] = at_least_normal(r.factor * info.factor);
      bits |= (info.there | info.v_bf16 << 2) << (4 * h);
      plain[h] = __all_sync(kAll, rel - N * h >= 31 && info.there == 3u);
      bf16[h] = __any_sync(kAll, info.v_bf16 != 0u);
    }
    return true;
  };
  if (!prepare(w.step_of(tile, 0))) return false;
#pragma unroll 1
  for (int u = 0; u < 2 * steps; ++u) {
    const int n = u >> 1, h = u & 1;  // the tile's n-th step, its half
    if (!wait_all(&bars->s_full[tile][h], (uint32_t)n & 1u, abort_flag, p)) return false;
    tc_fence_after();
    uint32_t x[32];
    tmem_ld16x2_32<32>(r.s + h * N, x);
    const int key0 = w.first_key(w.step_of(tile, n)) + h * N + 32 * r.half;
    const float f = h ? factor[1] : factor[0];
    const uint32_t my_bits = bits >> (4 * h);
    tmem_wait_ld();
    reg_fence(x, 32);
    score(p, r, x, f, key0 - r.pos, min(r.lim, key0 + 31) > r.pos);
    if (!(h ? plain[1] : plain[0])) hide(x, r.seen(key0, my_bits));
    // Weights are formed beside the reference of the tokens before, without a look for
    // the maximum; with one where their sum shows that scores rose far above it, or where
    // there is no reference yet.
    uint32_t weights[16];
    uint64_t part;
    auto weigh = [&](auto type) {
      const uint64_t nm2 = f2_pack(-r.reference(), -r.reference());
      uint64_t parts[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const uint64_t v = f2_pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1]));
        float a, b;
        f2_unpack(f2_add(v, nm2), a, b);
        a = ex2_approx(a), b = ex2_approx(b);
        parts[i / 2 & 1] = f2_add(parts[i / 2 & 1], f2_pack(a, b));
        weights[i / 2] = pack_f16x2(a, b);
        if (decltype(type)::value && my_bits & 4u) weights[i / 2] = pack_bf16x2(a, b);
      }
      part = f2_add(parts[0], parts[1]);
    };
    for (;;) {
      if (h ? bf16[1] : bf16[0])
        weigh(std::true_type{});
      else
        weigh(std::false_type{});
      float a, b;
      f2_unpack(part, a, b);
      // (a sum that is not a number too)
      const bool find = r.m == -INFINITY || !(a + b <= kMostSum);
      if (!__any_sync(kAll, find)) break;
      float top = largest32(x);
      top = fmaxf(top, __shfl_xor_sync(kAll, top, 16));
      // (a row without a reason of its own keeps its reference, and its bits)
      const int others = __shfl_xor_sync(kAll, find ? 1 : 0, 16);
      const bool moves = (find || others != 0) && top > r.m + kLagBits;
      if (!__any_sync(kAll, moves)) break;
      const float g = r.move_to(top, moves);
      if (u > 0) {  // O, once the product before is complete
        if (!wait_all(&bars->pv_done[tile][1 - h], (uint32_t)(u - 1 >> 1) & 1u, abort_flag, p))
          return false;
        tc_fence_after();
        r.template rescale<D / 2>(g);
      }
    }
    r.sum = f2_add(r.sum, part);
    tmem_st16x2_16<16>(r.s + h * N, weights);
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[tile][h]));
    if (h == 1 && n + 1 < steps && !prepare(w.step_of(tile, n + 1))) return false;
  }
  return wait_all(&bars->pv_done[tile][1], (uint32_t)(steps - 1) & 1u, abort_flag, p);
}

template <int D, int NG, bool SCORED>
__device__ void run_softmax(const ChunkParams& p, const ChunkWork& w, ChunkBars* bars,
                            uint32_t tmem, uint32_t base, volatile int* abort_flag) {
  using C = ChunkCfg<D>;
  constexpr int DH = D / 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  ChunkRow r;
  r.tile = warp / kSoftmaxWarps;
  // 16 of the 32 rows of this warp's part of tensor memory; lanes 16 on take the same
  // rows' second half of a piece's tokens and of the channels
  r.row_in = (warp & 3) * 32 + (warp >> 2 & 1) * 16;
  r.half = lane >> 4;
  const int in = r.row_in + (lane & 15);
  if (w.steps[r.tile] == 0) {
    if (r.half == 0) write_nothing<D>(p, w, r.tile, in);
    return;
  }
  Query<D> query;
  query.fetch(p, w, w.first_row(r.tile) + r.row_in);
  const int shift = load_queries<D, NG>(p, bars, base, r.tile, r.row_in, query);
  r.row = query.row;
  r.t = query.t;
  r.g = query.g;
  r.there = r.row < w.rows;
  // (rows without a query: all keys, with scores of zero)
  r.lim = r.there ? w.limit(r.t) : 0x7FFFFFFF;
  r.pos = w.first_pos + r.t;
  r.factor = ldexpf(p.scale_log2, -shift);
  r.slope = r.inv_cap = 0.0f;
  if constexpr (SCORED) {
    if (p.slopes && r.there) r.slope = load(p.slopes + w.h * p.G + r.g) * 1.4426950408889634f;
    if (p.cap_log2 > 0.0f) r.inv_cap = 1.0f / p.cap_log2;
  }
  const uint32_t lanes = (uint32_t)r.row_in << 16;
  r.s = tmem + C::kTmemS + r.tile * kKeys + lanes;
  r.o = tmem + C::kTmemO + r.tile * D + lanes;
  r.m = -INFINITY;
  r.sum = 0;
  if constexpr (SCORED) {
    if (!softmax_halves<D>(p, w, bars, r, abort_flag)) return;
  } else {
    if (!softmax_steps<D>(p, w, bars, r, abort_flag)) return;
  }
  // ---- the results
  tc_fence_after();
  float s0, s1;
  f2_unpack(r.sum, s0, s1);
  float sum = s0 + s1;
  sum += __shfl_xor_sync(kAll, sum, 16);
  const float v_scale = bars->v_scale;
  const float inv = sum == 0.0f ? 0.0f : v_scale / sum;
  const bool partial = p.partial != nullptr;
  float* slot = p.partial + (w.slot * 2 + r.tile) * (kTileRows * (D + 2));
  const int64_t at = ((int64_t)w.b * p.H + w.h * p.G + r.g) * p.T + r.t;
  if (r.there && r.half == 0) {
    if (partial) {
      slot[in] = r.m;
      slot[kTileRows + in] = sum;
    } else {
      p.lse[at] = (r.m + __log2f(sum)) * kLn2;
    }
  }
#pragma unroll 1
  for (int k = 0; k < DH; k += 16) {
    uint32_t o[16];
    tmem_ld16x2_16<DH>(r.o + k, o);
    tmem_wait_ld();
    reg_fence(o, 16);
    const int c = r.half * DH + k;
    // channels from the codes' order
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int k8 = i & 7;
      x[i] = __uint_as_float(o[(i & 8) + (k8 < 4 ? 2 * k8 : 2 * k8 - 7)]) * (partial ? v_scale : inv);
    }
    const int nan_from = bars->nan_from[c / (D / NG)];
    if (r.lim >= nan_from) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __int_as_float(0x7FC00000);
    }
    if (r.there && partial) {
      float4* dst = reinterpret_cast<float4*>(slot + 2 * kTileRows + in * D + c);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else if (r.there) {
      write_row<D>(p, at, x, c);
    }
  }
  if (!r.there && r.half == 0) write_nothing<D>(p, w, r.tile, in);  // behind the count
}

template <int D, int NG, bool SCORED>
__global__ void __launch_bounds__(kChunkThreads, 1) kv4_chunk_kernel(const ChunkParams p) {
  using C = ChunkCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // swizzled tiles begin at multiples of 1024
  ChunkBars* bars = reinterpret_cast<ChunkBars*>(smem_raw + (base - raw) + C::kBars);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // (the same for the warp)

  wait_for_previous_launch();
  const ChunkWork w = chunk_work(p);
  if (w.total == 0) {  // (the whole CTA)
    allow_next_launch();
    if (threadIdx.x < kCtaRows)
      write_nothing<D>(p, w, threadIdx.x / kTileRows, threadIdx.x % kTileRows);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&bars->k_full[i]), 4);
      mbar_init(smem_u32(&bars->k_empty[i]), 2);
      mbar_init(smem_u32(&bars->v_full[i]), 4);
      mbar_init(smem_u32(&bars->v_empty[i]), 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->q_full[i]), kSoftmaxWarps);
      mbar_init(smem_u32(&bars->turn[i]), kSoftmaxWarps);
      for (int h = 0; h < 2; ++h) {
        mbar_init(smem_u32(&bars->s_full[i][h]), 1);
        mbar_init(smem_u32(&bars->p_full[i][h]), kSoftmaxWarps);
        mbar_init(smem_u32(&bars->pv_done[i][h]), 1);
      }
    }
    for (int i = 0; i < kInfos; ++i) mbar_init(smem_u32(&bars->info_full[i]), 8);
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&bars->drain[i]), 1);
    for (int i = 0; i < 4; ++i) bars->nan_from[i] = 0x7FFFFFFF;
    bars->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpScores) {
    tmem_alloc(smem_u32(&bars->tmem_base), kTmemColumns);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  allow_next_launch();
  const uint32_t tmem = bars->tmem_base;
  volatile int* abort_flag = &bars->abort_flag;

  if (warp < kWarpK) {
    regs_inc<kSoftmaxRegs<NG, SCORED>>();
    run_softmax<D, NG, SCORED>(p, w, bars, tmem, base, abort_flag);
  } else if (warp < kWarpScores) {
    regs_dec<kExpandRegs<NG, SCORED>>();
    if (warp < kWarpV)
      run_expand_keys<D, NG>(p, w, bars, base, abort_flag);
    else
      run_expand_values<D, NG>(p, w, bars, base, abort_flag);
  } else {
    regs_dec<kIssueRegs>();
    if (warp < kWarpValues)
      run_scores<D, SCORED>(p, w, bars, tmem, base, abort_flag, warp - kWarpScores);
    else
      run_values<D, SCORED>(p, w, bars, tmem, base, abort_flag, warp - kWarpValues);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpScores) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemColumns);
  }
}

// A warp a row: joins the splits' results in their order.
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) kv4_chunk_join_kernel(const ChunkParams p) {
  constexpr int V = D / 32;  // channels a lane
  wait_for_previous_launch();
  allow_next_launch();
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  const int bh = blockIdx.y, b = bh / p.c.Hkv, h = bh - b * p.c.Hkv;
  int count = p.T;
  if (p.counts) count = min(max(load(p.counts + b), 0), p.T);
  if (row >= p.G * count) return;  // (written by the first split)
  // the ranges' results of the row's tile; of both, if they hold the same rows
  constexpr int64_t kSlot = kTileRows * (D + 2);
  const int r = row % kTileRows, parts = p.twin ? 2 * p.splits : p.splits;
  const int64_t next = p.twin ? kSlot : 2 * kSlot;
  const float* slot = p.partial + ((int64_t)bh * p.items + row / kCtaRows) * p.splits * 2 * kSlot +
                      row / kTileRows % 2 * kSlot;
  // Maxima and sums a lane a part, then the parts' O in their order, with all loads known
  // beforehand: part by part, each behind the last one's maximum, 30 of them took 20 us.
  float factor[kMostParts / 32], top = -INFINITY, sum = 0.0f;
  uint32_t written[kMostParts / 32], seen = 0;  // parts that have an O
#pragma unroll
  for (int k = 0; k < kMostParts / 32; ++k) {
    const int s = k * 32 + lane;
    factor[k] = s < parts ? __ldcg(slot + s * next + r) : -INFINITY;
    top = fmaxf(top, factor[k]);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
  for (int k = 0; k < kMostParts / 32; ++k) {
    const int s = k * 32 + lane;
    const float l = s < parts ? __ldcg(slot + s * next + kTileRows + r) : 0.0f;
    const bool there = !(factor[k] == -INFINITY && l == 0.0f);
    written[k] = __ballot_sync(0xffffffffu, there);
    seen |= written[k];
    factor[k] = there ? ex2_approx(factor[k] - top) : 0.0f;
    if (there) sum = fmaf(l, factor[k], sum);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  float x[V];
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = 0.0f;
  const float* from = slot + 2 * kTileRows + r * D + lane * V;
#pragma unroll
  for (int k = 0; k < kMostParts / 32; ++k) {
#pragma unroll 16
    for (int s = k * 32; s < min(parts, k * 32 + 32); ++s) {
      const float f = __shfl_sync(0xffffffffu, factor[k], s & 31);
      using Piece = std::conditional_t<V == 4, float4, float2>;
      Piece v{};
      // (whatever its factor: a value that is not a number is not one times zero)
      if (written[k] >> (s & 31) & 1u) v = __ldcg(reinterpret_cast<const Piece*>(from + s * next));
      const float* vs = reinterpret_cast<const float*>(&v);
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = fmaf(vs[i], f, x[i]);
    }
  }
  const float inv = seen != 0u ? 1.0f / sum : 0.0f;
  const int t = row / p.G, g = row - t * p.G;
  const int64_t at = ((int64_t)b * p.H + h * p.G + g) * p.T + t;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t to = at * D + lane * V + i;
    if (p.out_f32)
      static_cast<float*>(p.out)[to] = x[i] * inv;
    else
      static_cast<__nv_bfloat16*>(p.out)[to] = __float2bfloat16_rn(x[i] * inv);
  }
  if (lane == 0) p.lse[at] = seen != 0u ? (top + __log2f(sum)) * kLn2 : -INFINITY;
}

// How many ranges the tokens of a row tile are cut into, by sizes that the host
// knows: waves of CTAs times the steps of each, a CTA's start counted as kStart
// steps and the join as kJoin.
constexpr double kStart = 3.0, kJoin = 4.0;
int chunk_splits(int64_t ctas, int64_t steps, int sms) {
  int best = 1;
  double least = 0.0;
  for (int n = 1; n <= kMostSplits && n <= steps; ++n) {
    const double waves = (double)((ctas * n + sms - 1) / sms);
    const double cost = waves * ((double)((steps + n - 1) / n) + kStart) + (n > 1 ? kJoin : 0.0);
    if (n == 1 || cost < least) best = n, least = cost;
    if (ctas * n > 8 * (int64_t)sms) break;
  }
  return best;
}

// Up to so many rows a key/value head the kernels of kv4_attn.cuh take the call: they read
// the cache once for 16 rows, with less to set up.  8 sequences of 49152 tokens, 8 heads of
// 128: 16 rows 161 us, 32 rows 276, 48 rows 430; here 215 to 245 us for 17 to 128.  Where there
// is little to read in all (16 rows' tiles times tokens) they take more: 6 heads of 1000
// tokens, 17 to 96 rows: 12 us, here 19; 128 rows 14 and 22; 128 heads of 1000 tokens, 40
// rows: 40 and 27.  (The border lies below where the two meet: the last ones' 32 rows, 256000
// tiles times tokens, take 27 here, 24 there.)  Tokens are those that the table has room for.
constexpr int64_t kFewRows = 16, kMostFewRows = 128, kLittle = 3 << 16;
constexpr int kMostFewRowsBatch = 4096;
bool few_rows(int B, int kv_heads, int64_t rows, int64_t tokens) {
  if (B > kMostFewRowsBatch || rows > kMostFewRows) return false;
  return rows <= kFewRows || (rows + 15) / 16 * B * kv_heads * tokens <= kLittle;
}

constexpr int64_t kMostRows = 65535 * kCtaRows;  // a grid's third size
constexpr int64_t kLeastTwin = 512;  // tokens from which the join is worth it

struct ChunkSplit {
  int64_t items, ctas;
  int splits;
  bool twin;
  size_t workspace;
};
ChunkSplit chunk_split(int B, int kv_heads, int64_t rows, int64_t tokens, int D, int sms) {
  ChunkSplit s{};
  s.items = (rows + kCtaRows - 1) / kCtaRows;
  const int64_t tiles = s.items * B * kv_heads;
  s.splits = chunk_splits(tiles, (tokens + kKeys - 1) / kKeys, sms);
  s.ctas = tiles * s.splits;
  s.twin = rows <= kTileRows && tokens > kLeastTwin;
  if (s.splits > 1 || s.twin) s.workspace = (size_t)s.ctas * kCtaRows * (D + 2) * sizeof(float);
  return s;
}

template <int D, int NG>
cudaError_t launch_chunk(const ChunkParams& p, bool scored, cudaStream_t st) {
  using C = ChunkCfg<D>;
  const dim3 grid(p.splits, p.B * p.c.Hkv, p.items);
  cudaError_t e;
  if (scored) {
    constexpr auto kernel = kv4_chunk_kernel<D, NG, true>;
    e = allow_shared_memory<kernel>(C::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kernel, grid, dim3(kChunkThreads), C::kSmem, st, p);
  } else {
    constexpr auto kernel = kv4_chunk_kernel<D, NG, false>;
    e = allow_shared_memory<kernel>(C::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kernel, grid, dim3(kChunkThreads), C::kSmem, st, p);
  }
  if (e != cudaSuccess || !p.partial) return e;
  const int64_t rows = (int64_t)p.G * p.T;
  return launch_dependent(kv4_chunk_join_kernel<D>,
                          dim3((unsigned)((rows + kJoinWarps - 1) / kJoinWarps), p.B * p.c.Hkv),
                          dim3(kJoinWarps * 32), 0, st, p);
}

}  // namespace
}  // namespace bsattn

using namespace bsattn;

extern "C" {

size_t bsattn_kv4_attn_chunk_workspace(int B, int H, int kv_heads, int T, int D, int page_size,
                                       int columns) {
  if (B <= 0 || H <= 0 || kv_heads <= 0 || T <= 0 || H % kv_heads != 0 || page_size <= 0 ||
      columns <= 0)
    return 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const int64_t rows = (int64_t)(H / kv_heads) * T, tokens = (int64_t)columns * page_size;
  if (few_rows(B, kv_heads, rows, tokens)) return kv4_few_rows_workspace(B, kv_heads, (int)rows, D, tokens);
  return chunk_split(B, kv_heads, rows, tokens, D, device_sm_count(dev)).workspace;
}

bsattn_status bsattn_kv4_attn_chunk(const bsattn_kv4_cache* cache, const void* q, int B, int H,
                                    int T, const int32_t* block_table, int64_t table_stride,
                                    int columns, const int32_t* lengths, const int32_t* counts,
                                    const int32_t* prefix, float scale, float cap,
                                    const float* slopes, unsigned flags, void* out, float* lse,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  ChunkParams p{};
  const bsattn_status rc = check_cache(cache, &p.c);
  if (rc != BSATTN_OK) return rc;
  if (!q || !out || !lse || !aligned16(q) || !aligned16(out) || !aligned16(lse) ||
      !aligned16(workspace))
    return BSATTN_ERR_INVALID_ARG;
  if (!block_table || !lengths ||
      ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(lengths) |
        reinterpret_cast<uintptr_t>(counts) | reinterpret_cast<uintptr_t>(prefix) |
        reinterpret_cast<uintptr_t>(slopes)) & 3u))
    return BSATTN_ERR_INVALID_ARG;
  if (B <= 0 || H <= 0 || T <= 0 || columns <= 0 || table_stride < 0 || H % cache->kv_heads != 0)
    return BSATTN_ERR_INVALID_ARG;
  if (flags & ~(unsigned)BSATTN_OUT_F32) return BSATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !std::isfinite(cap) || cap < 0.0f) return BSATTN_ERR_INVALID_ARG;
  // (a cap that underflows in the kernel's units would cap nothing)
  if (cap > 0.0f && (cap < 1e-30f || cap > 1e30f)) return BSATTN_ERR_UNSUPPORTED;
  const int64_t rows = (int64_t)(H / cache->kv_heads) * T;
  if (B > 65535 || rows > kMostRows || (int64_t)B * cache->kv_heads > 65535 ||
      (int64_t)columns * cache->page_size > (1ll << 31) - 2 * kKeys ||  // positions are 32-bit
      (int64_t)cache->pages * cache->kv_heads * cache->page_size / 16 >= (1ll << 31))
    return BSATTN_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (few_rows(B, cache->kv_heads, rows, (int64_t)columns * cache->page_size))
    return kv4_few_rows({cache, q, B, H, T, block_table, table_stride, columns, lengths, counts,
                         prefix, scale, cap, slopes, (flags & BSATTN_OUT_F32) ? 1 : 0, out, lse},
                        workspace, workspace_bytes, st);
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSATTN_ERR_CUDA;
  const ChunkSplit split =
      chunk_split(B, cache->kv_heads, rows, (int64_t)columns * cache->page_size, cache->head_dim,
                  device_sm_count(dev));
  if (split.workspace > 0 && (!workspace || workspace_bytes < split.workspace))
    return BSATTN_ERR_INVALID_ARG;
  p.q = static_cast<const uint16_t*>(q);
  p.table = block_table;
  p.table_stride = table_stride;
  p.columns = columns;
  p.lengths = lengths;
  p.counts = counts;
  p.prefix = prefix;
  p.slopes = slopes;
  p.B = B;
  p.H = H;
  p.T = T;
  p.G = H / cache->kv_heads;
  p.items = (int)split.items;
  p.splits = split.splits;
  p.scale_log2 = (float)(std::fabs((double)scale) * 1.4426950408889634074);
  p.sign = scale < 0.0f ? -1.0f : 1.0f;
  p.cap_log2 = (float)((double)cap * 1.4426950408889634074);
  p.out = out;
  p.lse = lse;
  p.out_f32 = (flags & BSATTN_OUT_F32) ? 1 : 0;
  p.twin = split.twin ? 1 : 0;
  p.partial = split.workspace > 0 ? static_cast<float*>(workspace) : nullptr;
  p.timeout_ns = kDefaultWaitTimeoutNs;
  const bool scored = cap > 0.0f || slopes;
  const int groups = cache->head_dim / cache->group;
  cudaError_t e;
  if (cache->head_dim == 64)
    e = groups == 1 ? launch_chunk<64, 1>(p, scored, st)
                    : launch_chunk<64, 2>(p, scored, st);
  else
    e = groups == 1   ? launch_chunk<128, 1>(p, scored, st)
        : groups == 2 ? launch_chunk<128, 2>(p, scored, st)
                      : launch_chunk<128, 4>(p, scored, st);
  return from_cuda(e);
}

}  // extern "C"
