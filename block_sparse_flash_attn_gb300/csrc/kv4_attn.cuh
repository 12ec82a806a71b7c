// Attention of new tokens over the 4-bit cache: the kernels of kv4_attn.cu and, with
// scores that are capped, biased or opened to a prefix, of kv4_attn_scored.cu (SCORED).
//
// Query t of T of a sequence of length n sits at position n - T + t and sees
// the cached tokens up to its own position (all of them, or those of a list of
// pages).  With K and V rows decoded as step * code + least (kv4.cu):
//   s_i = scale q . k_i,  p = softmax(s),  o = sum_i p_i v_i,
//   lse = ln sum_i exp(s_i);  a query that sees nothing: o = 0, lse = -inf.
//
// The codes are never expanded to values.  With n_i the codes of a token,
//   q . k_i = step_i (q . n_i) + least_i sum(q)           (per group of channels)
//   sum_i p_i v_i = sum_i (p_i step_i) n_i + sum_i p_i least_i
// so both products run on the codes themselves, and steps and minima touch
// one number a (token, query, group).  A code masked out of a 32-bit word IS a
// 16-bit float: the low bits of one hold n as a subnormal, an exact operand.  One
// AND makes two operands; powers of two go into the queries and a final factor.
// But the tensor instruction lines products up by their operands' exponents and
// cuts them 25 bits below the largest, and a subnormal has the exponent of 1
// times its type's least normal number, however small it is (seen with single
// products): a code in the low bits of an fp16 loses up to 10 of those bits.  So
// - K's codes are bf16 operands, in its bits 0-3 and 4-7 (the latter reach the
//   exponent's last bit, where bf16 is linear still): 2^-18 and 2^-22 of a code
//   beside a row's largest query; queries are bf16 themselves;
// - V's are fp16 operands, for the weights' sake, moved to the mantissa's top, bits
//   6-9: 2^-21 of a code beside a row's largest weight.
// Every other token's codes are taken as complements: p step n + p least =
// -p step (15 - n) + p (15 step + least).  Codes are positive and least mostly not,
// so sums of either alone grow with the context while the output shrinks, and what
// is cut off adds up; in turn the sums stay near zero and the cuts cancel.
// Off the 64-bit result, of the output's norm (norm of the difference): 777 tokens
// 4e-7, 32768 to 65536 tokens 1.9e-6; with all codes as fp16 subnormals in place
// and complements by tiles 4.5e-5 and 3.7e-5.
//
// Tokens are the MMA's M (16 a tile), queries its N (8 a tile): S^T = K Q^T and
// O^T = V^T P^T, since a key/value head has few query rows (G T <= 16 a tile).
// P step goes from S^T's accumulator layout to O^T's operand layout with
// movmatrix, as an fp16 pair hi + lo.  Each query row and group of channels has
// its own power of two beside the largest p step that it has met: that one lies
// between 2^6 and 2^15, and the pair ends at fp16's 2^-24, so a weight is off by
// 2^-23 of itself or by 2^-31 of the largest, whatever is larger.  A token of a
// wide step and no weight takes no bits from the others.
//
// Bound: memory.  D + 8 bytes (groups of D) a token and head for 4 D G T
// operations: at G T = 8 some 30 operations a byte, a tenth of the card's
// tensor-to-memory ratio; mma.sync (no TMEM round trip, operands straight from
// registers) is ample.  Each warp streams 16-token tiles through its own ring
// of cp.async stages, with no CTA barrier in the loop.
//
// Work, split from the device's lengths (so a captured graph follows them):
// - Long or ragged contexts: the (sequence, head, 128-token step) units in order
//   are cut into equal ranges, one a CTA.  A range that ends inside a sequence's
//   head leaves a partial result (maximum, sum, O) in the workspace, and a second
//   launch joins those: ragged batches and single long sequences fill the
//   machine alike.
// - Short contexts and lists: a head is a cluster of up to 8 CTAs, which share
//   its steps and join their results through each other's shared memory; where
//   there are more heads than CTAs, 8, 4, 2 or 1 warps of a CTA.  One launch
//   without a workspace.
// All join in a fixed order: results repeat bit for bit.
//
// Measured: 32 sequences of 32768 to 65536 tokens, 8 heads of 128, 4 query heads
// each: 310 us, 5.5 TB/s, 83% of a plain copy's rate, and 303 of 306 us when all pages
// lie in L2: what is left is instructions (59% of issue slots, the integer pipe,
// masks and shifts of codes, 57%), not bandwidth.  CUDA-core products on decoded
// values: 10 ms.  One sequence of 777 tokens: 8 us, launch and five loads in a
// row.
#pragma once

#include <cmath>
#include <cstdint>
#include <mutex>

#include <cuda_fp16.h>

#include "kv4.cuh"

#ifndef BSATTN_SCORED  // which of the two a translation unit builds
#error "define BSATTN_SCORED"
#endif

namespace bsattn {
namespace {

constexpr bool kScored = BSATTN_SCORED;
constexpr int kAttnThreads = 256;
constexpr int kAttnWarps = kAttnThreads / 32;
constexpr int kTile = 16;                      // tokens a warp takes at once
constexpr int kStep = kTile * kAttnWarps;      // tokens a CTA takes at once
constexpr int kStages = 4;                     // tiles in a warp's ring
constexpr int kPerSm = 2;                      // CTAs an SM with up to 8 query rows
constexpr int kMostSequences = 4096;
constexpr int kJoinThreads = 128;
// At most so many CTAs share a head: more start sooner than their results are
// joined.  One head of 131072 tokens: 27 us with 64, 46 us with 304; two of
// 65536: 23 and 32 us.
constexpr int kMostParts = 64;
// Steps that ranges cost beside a cluster (see attn_split).  8 heads of 8192
// tokens: 13 us as clusters of 8, 18 us as ranges; 128 heads: 40 and 45 us;
// 16 heads of 16384 tokens: 23 and 21 us.
constexpr int kSegmentSteps = 8;
// What a head costs a group of warps beside its steps, and a segment a CTA of
// ranges (which is a chain of loads, barriers and stores too, with less beside it
// to run meanwhile; once more for the second launch).
constexpr int kGroupStart = 4;
constexpr int kSegmentStart = 6;
// The most steps that a group of warps or a CTA of a cluster is given: a sequence
// much longer than the others holds the call up by no more.
constexpr int kMostGroupSteps = 64;
constexpr int kMostCluster = 8;  // CTAs, the portable most
// Running maximum before any score: no finite score lies below it, and differences
// of it are 0 or infinite, never NaN.
constexpr float kNoMax = -3.402823466e38f;
// Weights are taken beside 2^8 times the largest one so far: later scores may pass
// the running maximum by that, and no weight is above 1.
constexpr float kLag = 8.0f;
// p step is brought to [2^6, 2^7) and may grow to 2^15 (as fp16 bits)
constexpr uint32_t kMostWeight = 0x7800u;

struct AttnParams {
  Kv4View c;
  const uint16_t* q;  // [B][H][T][D]
  const int* table;
  int64_t table_stride;
  int columns;
  const int* lengths;
  const int* selected;  // [B][Hkv][n_selected] ascending pages, or null
  int n_selected;
  int B, T, rows;  // rows = G * T
  int mt;          // row tiles a head
  float scale_log2;
  void* out;
  float* lse;
  int out_f32;
  int* prefix;     // [B + 1] steps before each sequence (written by CTA 0 for the join)
  float* partial;  // [2 * CTAs][RP * (D + 2)]
  int ctas;
  int cluster;  // CTAs a head
  int group;    // or warps a head; both 0: ranges
  int tiles;    // row tiles of all heads and sequences
  // SCORED: null or 0: none
  const int* counts;    // new tokens of each sequence
  const int* open;      // positions below it are seen by all
  const float* slopes;  // [H]
  float cap_log2;       // cap log2 e
};

// The tokens of a sequence, none where none is new.
template <bool SCORED>
__device__ __forceinline__ int length_of(const AttnParams& p, int b) {
  if (SCORED && p.counts && load(p.counts + b) <= 0) return 0;
  return max(load(p.lengths + b), 0);
}

__device__ __forceinline__ uint32_t word(const uint8_t* shared) {
  return *reinterpret_cast<const uint32_t*>(shared);
}
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* shared, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(shared);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(shared);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = word(shared);
  }
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Four 8 x 8 matrices of 16-bit words, transposed: of each pair of pieces (16
// bytes) this lane's word of rows 2j and 2j + 1, and of those 8 on.
__device__ __forceinline__ void load_transposed(uint32_t at, uint32_t (&a)[2], uint32_t (&b)[2]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a[0]), "=r"(a[1]), "=r"(b[0]), "=r"(b[1])
               : "r"(at));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half(uint32_t x) {
  return __half22float2(*reinterpret_cast<__half2*>(&x));
}

// Of a pair of tokens' codes in bits 6-9 and 22-25 the even token's code and the
// odd one's complement.  One instruction, if one of its two constants comes from a
// register: the long contexts below 332 us (by twos), with two instructions 372,
// with the loaded words turned over first 338.
__device__ __forceinline__ uint32_t complements(uint32_t x, uint32_t flip) {
  uint32_t y;  // (x ^ flip) & mask
  asm("lop3.b32 %0, %1, %2, %3, 0x48;" : "=r"(y) : "r"(x), "n"(0x03C003C0u), "r"(flip));
  return y;
}

// The larger magnitudes of two fp16 pairs; a NaN gives way to a number.
__device__ __forceinline__ uint32_t larger_halves(uint32_t a, uint32_t b) {
  const __half2 m = __hmax2(*reinterpret_cast<__half2*>(&a), __habs2(*reinterpret_cast<__half2*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// The power of two that brings x > 0 to [2^6, 2^7), 2^106 for x below 2^-100; and
// the lower end of what such a scale brings there, 2^6 / |scale|.
__device__ __forceinline__ float scale_beside(float x) {
  const int e = max((int)(__float_as_uint(x) >> 23), 27);
  return __uint_as_float((uint32_t)(254 + 6 - e) << 23);
}
__device__ __forceinline__ float largest_beside(float scale) {
  return __uint_as_float((254u + 6u << 23) - (__float_as_uint(scale) & 0x7FFFFFFFu));
}

// This CTA's shared-memory word in another CTA of the cluster.
__device__ __forceinline__ float peer_word(const float* shared, int rank) {
  uint32_t at;
  float v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(shared_address(shared)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

// Where each CTA's range of units begins.
__device__ __forceinline__ int64_t range_begin(int64_t units, int ctas, int c) {
  // (32-bit division where it does: a 64-bit one is some hundred instructions)
  if (units < (1 << 20)) return (unsigned)units * (unsigned)c / (unsigned)ctas;
  return units * c / ctas;
}
// The CTA whose range holds unit u.
__device__ __forceinline__ int range_of(int64_t units, int ctas, int64_t u) {
  int c = units < (1 << 20) ? (int)((unsigned)u * (unsigned)ctas / (unsigned)units)
                            : (int)((u * ctas) / units);
  while (c + 1 < ctas && range_begin(units, ctas, c + 1) <= u) ++c;
  while (c > 0 && range_begin(units, ctas, c) > u) --c;
  return c;
}

// The page of the tile that starts at token v0 of a (sequence, head)'s list,
// and that tile's first position; -1 when it holds nothing to see.
__device__ __forceinline__ int tile_page(const AttnParams& p, int b, int h, int64_t v0, int len,
                                         int& pos) {
  int64_t logical = v0 >> p.c.log_page;
  const int place = (int)(v0 & (p.c.page - 1));
  if (p.selected) {
    if (logical >= p.n_selected) return -1;
    const int* sel = p.selected + ((int64_t)b * p.c.Hkv + h) * p.n_selected;
    const int64_t e = logical;
    logical = load(sel + e);
    if (logical < 0) return -1;
    if (e > 0) {  // a page named twice, out of order or behind a negative entry
      const int64_t before = load(sel + e - 1);
      if (before < 0 || logical <= before) {
        p.c.report();
        return -1;
      }
    }
  }
  const int64_t first = (logical << p.c.log_page) + place;
  if (first >= len) return -1;
  pos = (int)first;
  return page_at(p.c, p.table + b * p.table_stride, p.columns, logical);
}

// What a CTA takes: a range of units, a share of one head (the CTAs of a cluster
// share it), or a head for each group of p.group warps.
enum : int { kRanges, kClusters, kGroups };

// NG groups of channels share a step each, NT
// tiles of 8 query rows.  TWICE: up to 4 rows, each in two columns of the one
// tile, of which the second carries the low halves of the weights: one product
// for hi + lo instead of two.
template <int D, int NG, int NT, bool TWICE>
struct Attn {
  static constexpr int C = D / 32;        // 16-byte pieces (32 channels) of a row of codes
  static constexpr int CG = C / NG;       // pieces a group
  static constexpr int RB = D / 2;        // bytes of a row of codes
  static constexpr int RP = TWICE ? 4 : 8 * NT;  // query rows a tile
  static constexpr int kCodes = kTile * RB;
  static constexpr int kScales = kTile * NG * 4;
  static constexpr int kStage = 2 * kCodes + 2 * kScales;  // K, V codes, K, V scales
  static constexpr int kWarpRing = kStages * kStage;
  static constexpr int kSmem = kAttnWarps * kWarpRing;
  // (the join of a warp's results takes the place of its ring)
  static_assert(RP * (D + 3) * 4 <= kWarpRing, "shared memory");
  static constexpr int kSlot = RP * (D + 2);  // floats of a partial result
  // Tiles a pass of the loop: a turn of the ring, whose places are constants then;
  // fewer in four groups, where registers run out and code is long.  32 sequences of
  // 32768 to 65536 tokens, groups of 128: 310 us, by twos 332, one by one 355; 256
  // heads of 32768 tokens, groups of 32: 342 us, by twos 334; 64 heads of 16 rows and
  // 49152 tokens: 241 and 232; 12 heads of 16 rows over 24 pages of 32 tokens, page
  // choice included: by twos 21, one by one 19.
  template <int MODE>
  static constexpr int kUnroll = NG < 4 ? kStages : MODE == kRanges ? 2 : 1;

  // pieces of a row are stored permuted by its token, so that the 32-bit reads
  // of both products meet 32 banks
  static __device__ __forceinline__ int swizzle(int token) {
    return D == 128 ? (token >> 1) & 3 : (token >> 2) & 1;
  }
};

// A group's step and least; SCORED: NaN both where one is not finite (an infinity times the
// sum of a query's channels would have a sign that the channels' own products have not).
template <bool SCORED>
__device__ __forceinline__ uint32_t scales_of(const uint8_t* shared) {
  const uint32_t x = word(shared);
  if (SCORED && ((x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u)) return 0x7FC07FC0u;
  return x;
}

// A pair of scores (base 2) capped.  32 sequences of up to 65536 tokens: see launch_attn.
__device__ __forceinline__ F2 capped(F2 s, float cap, float inv_cap) {
  const F2 y = s * f2(inv_cap), u = y * y;
  F2 a = fma2(f2(kTanh5), u, f2(kTanh4));
  a = fma2(a, u, f2(kTanh3));
  a = fma2(a, u, f2(kTanh2));
  a = fma2(a, u, f2(kTanh1));
  a = fma2(a, u, f2(kTanh0));
  a = a * s;
  const float2 v = split(y), w = split(a);
  float x0 = w.x, x1 = w.y;
  if (!(fabsf(v.x) <= kTanhRange)) x0 = cap * tanh_any(v.x);
  if (!(fabsf(v.y) <= kTanhRange)) x1 = cap * tanh_any(v.y);
  return f2(x0, x1);
}

template <int D, int NG, int NT, bool TWICE, int MODE, bool SCORED>
__global__ void __launch_bounds__(kAttnThreads, NT == 1 ? kPerSm : 1)
    kv4_attn_kernel(const AttnParams p) {
  using A = Attn<D, NG, NT, TWICE>;
  constexpr int C = A::C, RB = A::RB, RP = A::RP, KW = A::CG;
  constexpr int kUnroll = A::template kUnroll<MODE>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int warp_sums[kAttnWarps];
  constexpr int kMostGroups = MODE == kGroups ? kAttnWarps : 1;
  __shared__ uint4 queries_of[kMostGroups][NT][C][32];  // operands of S^T = K Q^T, a lane's four words
  __shared__ int2 tiles[kAttnWarps][128];  // (row / 16, position) of four batches of tiles
  int* prefix = reinterpret_cast<int*>(smem + A::kSmem);  // [B + 1]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, j = lane & 3;
  // this warp's group, its place there, and this thread's
  const int warps = MODE == kGroups ? p.group : kAttnWarps;
  const int group = MODE == kGroups ? warp / warps : 0;
  const int gwarp = warp - group * warps, gtid = tid - group * warps * 32, threads = warps * 32;
  auto group_barrier = [&] {
    if (MODE == kGroups)
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
    else
      __syncthreads();
  };
  auto& queries = queries_of[group];

  wait_for_previous_launch();
  const int heads = p.c.Hkv * p.mt;
  const int64_t most = (int64_t)p.columns * p.c.page;  // tokens that the table has room for
  auto steps_of = [&](int b) -> int {
    const int step = kTile * warps;
    if (p.selected) return (int)(((int64_t)p.n_selected * p.c.page + step - 1) / step);
    int64_t n = length_of<SCORED>(p, b);
    if (n > most) {
      p.c.report();
      n = most;
    }
    return (int)((n + step - 1) / step);
  };
  int64_t units = 0, u = 0, u_end = 1;
  bool first_segment = true;
  if (MODE != kRanges) {
    allow_next_launch();
  } else {
    // steps before each sequence
    const int per = (p.B + kAttnThreads - 1) / kAttnThreads;
    const int b0 = tid * per;
    int sum = 0;
    for (int i = 0; i < per; ++i)
      if (b0 + i < p.B) sum += steps_of(b0 + i);
    int s = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += t;
    }
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    int at = s - sum;
    for (int w = 0; w < warp; ++w) at += warp_sums[w];
    for (int i = 0; i < per; ++i)
      if (b0 + i < p.B) {
        prefix[b0 + i] = at;
        at += steps_of(b0 + i);
        if (b0 + i == p.B - 1) prefix[p.B] = at;
      }
    __syncthreads();
    if (blockIdx.x == 0)
      for (int i = tid; i <= p.B; i += kAttnThreads) p.prefix[i] = prefix[i];
    allow_next_launch();
    units = (int64_t)prefix[p.B] * heads;
    if (units == 0) return;
    const int ctas = (int)min((int64_t)p.ctas, units);
    if ((int)blockIdx.x >= ctas) return;
    u = range_begin(units, ctas, blockIdx.x);
    u_end = range_begin(units, ctas, blockIdx.x + 1);
  }

  const uint32_t ring = shared_address(smem) + warp * A::kWarpRing;
  const uint8_t* my_ring = smem + warp * A::kWarpRing;
  // Where this lane's words begin.  K: tokens g and g + 8, words j KW .. j KW +
  // KW - 1 of each group.  V: the row that it points out to the transposing load,
  // piece lane / 16 of token lane mod 16.  A row's 16-byte piece c is at the offset
  // with 16 c in its swizzled bits.
  const uint32_t k_at = g * RB + (4 * KW * j & 15) + 16 * (A::swizzle(g) ^ (KW * j / 4));
  const uint32_t v_at =
      ring + A::kCodes + lane % 16 * RB + 16 * (A::swizzle(lane % 16) ^ (lane / 16));
  int2* my_tiles = tiles[warp];
  // this lane's pieces of a tile: codes (token, piece) = lane / C, lane % C, and
  // for D = 128 eight tokens on; one piece of the scales
  const uint32_t code_at = ring + lane / C * RB + 16 * ((lane % C) ^ A::swizzle(lane / C));
  const uint8_t* k_src = p.c.k_codes + lane * 16;
  const uint8_t* v_src = p.c.v_codes + lane * 16;
  const int scale_kv = lane / (4 * NG), scale_piece = lane % (4 * NG);
  const uint32_t scale_at =
      ring + 2 * A::kCodes + scale_kv * A::kScales + scale_piece * 16;
  const uint8_t* scale_src =
      reinterpret_cast<const uint8_t*>(scale_kv ? p.c.v_scales : p.c.k_scales) + scale_piece * 16;

  while (u < u_end) {
    // the segment: steps [s0, s1) of row tile m of head h of sequence b
    int b, hm, steps, s0, s1;
    if (MODE == kGroups) {
      const int hh = blockIdx.x * (kAttnWarps / warps) + group;
      if (hh >= p.tiles) return;  // (the whole group)
      b = hh / heads;
      hm = hh - b * heads;
      steps = s1 = steps_of(b);
      s0 = 0;
    } else if (MODE == kClusters) {
      const int hh = blockIdx.x / p.cluster, rank = blockIdx.x - hh * p.cluster;
      b = hh / heads;
      hm = hh - b * heads;
      steps = steps_of(b);
      s0 = (int)((int64_t)steps * rank / p.cluster);
      s1 = (int)((int64_t)steps * (rank + 1) / p.cluster);
    } else {
      int lo = 0, hi = p.B;  // last b with prefix[b] * heads <= u
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)prefix[mid] * heads <= u) lo = mid; else hi = mid;
      }
      b = lo;
      steps = prefix[b + 1] - prefix[b];
      const int64_t off = u - (int64_t)prefix[b] * heads;
      hm = (int)(off / steps);
      s0 = (int)(off - (int64_t)hm * steps);
      s1 = (int)min((int64_t)steps, s0 + (u_end - u));
    }
    const int h = hm / p.mt, row0 = (hm - h * p.mt) * RP;
    const int len = length_of<SCORED>(p, b);
    const int64_t bh = (int64_t)b * p.c.Hkv + h;
    const int n_tiles = s1 - s0;  // this warp's, one a step
    const int count = SCORED && p.counts ? min(max(load(p.counts + b), 0), p.T) : p.T;
    const int open = SCORED && p.open ? min(max(load(p.open + b), 0), len) : 0;
    // tiles that begin later need the mask (all, where rows are behind the count)
    const int seen_by_all = count < p.T ? -1 : max(len - p.T, open - 1) - (kTile - 1);

    // ---- tiles: pages are looked up 32 steps at a time, one batch ahead (the
    // next batch's loads are in flight while this one's tiles run)
    int2 next_tile;
    auto look_up = [&](int batch) {
      next_tile = make_int2(-1, -1);
      const int i = batch * 32 + lane;
      if (i < n_tiles) {
        int pos = 0;
        const int pg =
            tile_page(p, b, h, ((int64_t)(s0 + i) * warps + gwarp) * kTile, len, pos);
        if (pg >= 0)
          next_tile = make_int2((int)(p.c.row(pg, h, pos & (p.c.page - 1)) / kTile), pos);
      }
    };
    look_up(0);
    uint32_t to = 0;  // the ring's place for the next copy
    auto issue = [&](int i) {
      if ((i & 31) == 0) {
        my_tiles[(i & 127) + lane] = next_tile;
        __syncwarp();
        look_up((i >> 5) + 1);
      }
      const int row16 = my_tiles[i & 127].x;
      if (row16 >= 0) {
        const uint8_t* kc = k_src + (int64_t)row16 * A::kCodes;
        const uint8_t* vc = v_src + (int64_t)row16 * A::kCodes;
        copy16(code_at + to, kc);
        copy16(code_at + to + A::kCodes, vc);
        if (D == 128) {
          copy16(code_at + to + 8 * RB, kc + 512);
          copy16(code_at + to + A::kCodes + 8 * RB, vc + 512);
        }
        if (lane < 8 * NG) copy16(scale_at + to, scale_src + (int64_t)row16 * A::kScales);
      }
      copy_commit();
      to = to == (kStages - 1) * A::kStage ? 0 : to + A::kStage;
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) issue(i);

    // ---- queries: operands, the factor of the code product, the group sums
    F2 mul[NT], qs[NT][NG];  // of rows 2j, 2j + 1 of the accumulators
    int lim[NT][2];          // last position that the row sees
    F2 slope[SCORED ? NT : 1];        // SCORED: of rows 2j, 2j + 1 (base 2)
    int place[SCORED ? NT : 1][2];    // their positions
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row0 + nt * 8 + (TWICE ? g & 3 : g);
      float x[C][8], top = 0.0f, sum[NG];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (r < p.rows)
          raw = load(reinterpret_cast<const uint4*>(p.q + (bh * p.rows + r) * D) +
                      (c / KW * 4 + j) * KW + c % KW);
        unpack8(raw, x[c]);
        if (c % A::CG == 0) sum[c / A::CG] = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          top = fmaxf(top, fabsf(x[c][i]));
          sum[c / A::CG] += x[c][i];
        }
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
#pragma unroll
        for (int n = 0; n < NG; ++n) sum[n] += __shfl_xor_sync(0xFFFFFFFFu, sum[n], o);
      }
      // the row's largest query goes to [2^120, 2^121), so that products with codes
      // (n 2^-133) are normal numbers and the factor below is small; in two factors,
      // for 2^sh may pass fp32's range
      int sh = 120;
      if (top > 0.0f && top <= 3.4e38f) sh = 120 - ilogbf(top);
      const float fa = ldexpf(1.0f, sh / 2), fb = ldexpf(1.0f, sh - sh / 2);
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[c][i] = x[c][i] * fa * fb;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (gwarp == 0)  // (the same for all warps)
          queries[nt][c][lane] = make_uint4(
              pack_bf16(x[c][0], x[c][4]), pack_bf16(x[c][2], x[c][6]),
              pack_bf16(x[c][1] * 0.0625f, x[c][5] * 0.0625f),
              pack_bf16(x[c][3] * 0.0625f, x[c][7] * 0.0625f));
      }
      const float m = p.scale_log2 * ldexpf(1.0f, 133 - sh);
      auto rows2 = [&](float v) {  // of rows 2j and 2j + 1, from the lanes that loaded them
        return f2(__shfl_sync(0xFFFFFFFFu, v, 8 * j), __shfl_sync(0xFFFFFFFFu, v, 8 * j + 4));
      };
      mul[nt] = rows2(m);
#pragma unroll
      for (int n = 0; n < NG; ++n) qs[nt][n] = rows2(sum[n] * p.scale_log2);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = row0 + nt * 8 + (TWICE ? (2 * j + e) & 3 : 2 * j + e);
        if constexpr (SCORED) {
          const int t = rr % p.T;
          place[nt][e] = len - count + t;
          lim[nt][e] = rr < p.rows && t < count ? max(place[nt][e], open - 1) : -1;
        } else {
          lim[nt][e] = rr < p.rows ? len - p.T + rr % p.T : -1;
        }
      }
    }

    if constexpr (SCORED) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[2] = {0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rr = row0 + nt * 8 + (TWICE ? (2 * j + e) & 3 : 2 * j + e);
          if (p.slopes && rr < p.rows)
            x[e] = -1.4426950408889634f * load(p.slopes + h * (p.rows / p.T) + rr / p.T);
        }
        slope[nt] = f2(x[0], x[1]);
      }
    }
    const float inv_cap = SCORED && p.cap_log2 > 0.0f ? 1.0f / p.cap_log2 : 0.0f;
    group_barrier();
    F2 mx[NT], l[NT], vm[NT][NG];  // -(maximum + kLag), sum of weights, of weights * least
    F2 inv[NT][NG];  // what p step is multiplied by: a power of two, below 0 for complements
    const float sign = g & 1 ? -1.0f : 1.0f, fifteen = g & 1 ? 15.0f : 0.0f;
    float o[C][2][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      mx[nt] = f2(-kNoMax);
      l[nt] = f2(0.0f);
#pragma unroll
      for (int n = 0; n < NG; ++n) vm[nt][n] = f2(0.0f), inv[nt][n] = f2(sign * scale_beside(0.0f));
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[c][t][nt][e] = 0.0f;
    }

    uint32_t from = 0;  // the ring's place of the tile
    uint32_t flip;      // the odd tokens' halves (kept in a register: see complements)
    asm volatile("mov.b32 %0, 0xFFFF0000;" : "=r"(flip));
#pragma unroll kUnroll
    for (int i = 0; i < n_tiles; ++i) {
      copy_wait<kStages - 2>();
      __syncwarp();
      issue(i + kStages - 1);
      const uint32_t at_stage = from;
      const uint8_t* stage = my_ring + at_stage;
      from = from == (kStages - 1) * A::kStage ? 0 : from + A::kStage;
      const int pos = my_tiles[i & 127].y;
      if (pos < 0) continue;

      // ---- scores (base 2): token g (t = 0) and g + 8, rows 2j and 2j + 1 as a pair
      F2 s[NT][2];
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        float acc[NT][4], acc16[NT][4];  // (two chains of products, half as long)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nt][e] = acc16[nt][e] = 0.0f;
        const uint8_t* at = stage + (k_at ^ (16 * KW * n));
        uint32_t w0[KW], w1[KW];
        load_words<KW>(at, w0);
        load_words<KW>(at + 8 * RB, w1);
#pragma unroll
        for (int k = 0; k < KW; ++k) {
          const uint32_t y0 = w0[k] >> 8, y1 = w1[k] >> 8;
          const uint32_t a[4] = {w0[k] & 0x000F000Fu, w1[k] & 0x000F000Fu, y0 & 0x000F000Fu,
                                 y1 & 0x000F000Fu};
          const uint32_t a16[4] = {w0[k] & 0x00F000F0u, w1[k] & 0x00F000F0u, y0 & 0x00F000F0u,
                                   y1 & 0x00F000F0u};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint4 qf = queries[nt][n * KW + k][lane];
            mma_bf16(acc[nt], a, qf.x, qf.y);
            mma_bf16(acc16[nt], a16, qf.z, qf.w);
          }
        }
        const uint8_t* ks = stage + 2 * A::kCodes + (g * NG + n) * 4;
        const uint32_t k[2] = {scales_of<SCORED>(ks), scales_of<SCORED>(ks + 8 * NG * 4)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const F2 dot = f2(acc[nt][2 * t], acc[nt][2 * t + 1]) +
                           f2(acc16[nt][2 * t], acc16[nt][2 * t + 1]);
            const F2 by_least = f2(bf16_hi(k[t])) * qs[nt][n];
            s[nt][t] = fma2(dot, mul[nt] * f2(bf16_lo(k[t])),
                            n == 0 ? by_least : by_least + s[nt][t]);
          }
      }
      if constexpr (SCORED) {
        if (p.cap_log2 > 0.0f) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int t = 0; t < 2; ++t) s[nt][t] = capped(s[nt][t], p.cap_log2, inv_cap);
        }
        if (p.slopes) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int at = pos + g;
            const float d0 = (float)(place[nt][0] - at), d1 = (float)(place[nt][1] - at);
#pragma unroll
            for (int t = 0; t < 2; ++t)
              s[nt][t] = fma2(slope[nt], f2(fabsf(d0 - 8.0f * t), fabsf(d1 - 8.0f * t)), s[nt][t]);
          }
        }
      }
      // ---- V's steps and minima; what a row does not see weighs nothing
      uint32_t v[NG][2];
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const uint8_t* sc = stage + 2 * A::kCodes + A::kScales + (g * NG + n) * 4;
        v[n][0] = scales_of<SCORED>(sc);
        v[n][1] = scales_of<SCORED>(sc + 8 * NG * 4);
      }
      uint32_t hidden = 0;  // bits 4 nt + 2 t + e
      if (pos > seen_by_all) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          bool any = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float2 x = split(s[nt][t]);
            const bool h0 = pos + g + 8 * t > lim[nt][0], h1 = pos + g + 8 * t > lim[nt][1];
            if (h0) x.x = -INFINITY;
            if (h1) x.y = -INFINITY;
            s[nt][t] = f2(x.x, x.y);
            hidden |= (h0 ? 1u : 0u) << (4 * nt + 2 * t) | (h1 ? 2u : 0u) << (4 * nt + 2 * t);
            any = any || !h0 || !h1;
          }
#pragma unroll
          for (int n = 0; n < NG; ++n)
            if (!any) v[n][t] = 0u;
        }
      }
      // ---- weights p and p step
      F2 pr[NT][2], w[NG][NT][2];
      auto step_of = [&](int nt, int t, int n) {  // 0 * NaN must stay 0
        const float step = bf16_lo(v[n][t]);
        if (!hidden) return f2(step);
        return f2(hidden >> (4 * nt + 2 * t) & 1 ? 0.0f : step,
                  hidden >> (4 * nt + 2 * t) & 2 ? 0.0f : step);
      };
      uint32_t wh[NG][NT][2];
      auto weigh = [&] {  // whether a weight passes its bound
        float most = 0.0f;
        uint32_t most16 = 0u;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const float2 x = split(s[nt][t] + mx[nt]);
            const float p0 = exp2_fast(x.x), p1 = exp2_fast(x.y);
            most = fmaxf(most, fmaxf(p0, p1));
            pr[nt][t] = f2(p0, p1);
#pragma unroll
            for (int n = 0; n < NG; ++n) {
              w[n][nt][t] = pr[nt][t] * step_of(nt, t, n) * inv[nt][n];
              const float2 ws = split(w[n][nt][t]);
              wh[n][nt][t] = pack_half(ws.x, ws.y);
              most16 = larger_halves(most16, wh[n][nt][t]);
            }
          }
        return most > 1.0f || (most16 & 0xFFFFu) > kMostWeight || (most16 >> 16) > kMostWeight;
      };
      // ---- rare: a score far above the running maximum, or p step of another scale;
      // then once more with the scales that hold them (one copy of the code).  A row
      // that has neither stays as it is, whatever the others have.
#pragma unroll 1
      for (bool again = false; __any_sync(0xFFFFFFFFu, weigh()) && !again; again = true) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float2 a = split(s[nt][0]), c = split(s[nt][1]), old = split(mx[nt]);
          float top[2] = {fmaxf(a.x, c.x), fmaxf(a.y, c.y)};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int sft = 4; sft < 32; sft <<= 1)
              top[e] = fmaxf(top[e], __shfl_xor_sync(0xFFFFFFFFu, top[e], sft));
            const float reference = e ? -old.y : -old.x;
            top[e] = top[e] > reference ? top[e] + kLag : reference;
          }
          const F2 f = f2(exp2_fast(-old.x - top[0]), exp2_fast(-old.y - top[1]));
          mx[nt] = f2(-top[0], -top[1]);
          l[nt] = l[nt] * f;
          const float2 p0 = split(s[nt][0] + mx[nt]), p1 = split(s[nt][1] + mx[nt]);
          const F2 q0 = f2(exp2_fast(p0.x), exp2_fast(p0.y)), q1 = f2(exp2_fast(p1.x), exp2_fast(p1.y));
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            vm[nt][n] = vm[nt][n] * f;
            // beside the largest of this tile, or of the ones before it
            const float2 b0 = split(q0 * step_of(nt, 0, n)), b1 = split(q1 * step_of(nt, 1, n));
            const float2 was = split(inv[nt][n]), fs = split(f);
            float large[2] = {fmaxf(fabsf(b0.x), fabsf(b1.x)), fmaxf(fabsf(b0.y), fabsf(b1.y))};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
              for (int sft = 4; sft < 32; sft <<= 1)
                large[e] = fmaxf(large[e], __shfl_xor_sync(0xFFFFFFFFu, large[e], sft));
              const float before = largest_beside(e ? was.y : was.x), fe = e ? fs.y : fs.x;
              // (512 = 2^15 / 2^6: what the scale leaves room for)
              if (fe == 1.0f && large[e] <= 512.0f * before) large[e] = 0.0f;
              large[e] = scale_beside(fmaxf(large[e], fe * before));
            }
            inv[nt][n] = f2(sign * large[0], sign * large[1]);
            // f new / old, at most 2 (f new first: new / old alone may overflow)
            const float2 of = split(f * f2(large[0], large[1]) *
                                    f2(largest_beside(was.x), largest_beside(was.y)) * f2(0.015625f));
#pragma unroll
            for (int c = n * A::CG; c < (n + 1) * A::CG; ++c)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                o[c][k][nt][0] *= of.x, o[c][k][nt][1] *= of.y;
                o[c][k][nt][2] *= of.x, o[c][k][nt][3] *= of.y;
              }
          }
        }
      }
      // ---- hi + lo, turned to the operand layout
      uint32_t wl[NG][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          l[nt] = l[nt] + pr[nt][t];
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            F2 least = f2(fmaf(bf16_lo(v[n][t]), fifteen, bf16_hi(v[n][t])));
            if (hidden) {
              const float2 a = split(least);
              least = f2(hidden >> (4 * nt + 2 * t) & 1 ? 0.0f : a.x,
                         hidden >> (4 * nt + 2 * t) & 2 ? 0.0f : a.y);
            }
            vm[nt][n] = fma2(pr[nt][t], least, vm[nt][n]);
            const uint32_t hi16 = wh[n][nt][t];
            const float2 back = unpack_half(hi16);
            const float2 rest = split(fma2(f2(back.x, back.y), f2(-1.0f), w[n][nt][t]));
            const uint32_t lo16 = pack_half(rest.x, rest.y);
            if (TWICE) {
              wh[n][nt][t] = transpose8x8(j < 2 ? hi16 : lo16);
            } else {
              wh[n][nt][t] = transpose8x8(hi16);
              wl[n][nt][t] = transpose8x8(lo16);
            }
          }
        }
      }
      // ---- O^T += V^T P^T: of each half word (channels 32 c + 4 g on, tokens 2j
      // and 2j + 1, and 8 on), M tile 0 is made of codes 0 (rows g) and 2 (rows
      // g + 8), M tile 1 of codes 1 and 3
      uint32_t x[C][2];
#pragma unroll
      for (int c = 0; c < C; c += 2) load_transposed((v_at + at_stage) ^ (16 * c), x[c], x[c + 1]);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t x0 = x[c][0], x1 = x[c][1];
        const uint32_t a[2][4] = {
            {complements(x0 << 6, flip), complements(x0 >> 2, flip), complements(x1 << 6, flip),
             complements(x1 >> 2, flip)},
            {complements(x0 << 2, flip), complements(x0 >> 6, flip), complements(x1 << 2, flip),
             complements(x1 >> 6, flip)}};
        const int n = c / A::CG;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            mma_f16(o[c][k][nt], a[k], wh[n][nt][0], wh[n][nt][1]);
            if (!TWICE) mma_f16(o[c][k][nt], a[k], wl[n][nt][0], wl[n][nt][1]);
          }
        }
      }
    }
    copy_wait<0>();

    // ---- join the group's warps (their rings are free): maxima, sums, O in 32 bits
    group_barrier();
    float* sm = reinterpret_cast<float*>(smem + group * warps * A::kWarpRing);  // [warp][RP] maxima
    float* sl = sm + warps * RP;      // [warp][RP] sums
    float* so = sl + warps * RP;      // [warp][RP][D]
    float* sf = so + warps * RP * D;  // [warp][RP] factors
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (TWICE) {  // the columns of the low halves onto those of the high ones
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[c][k][nt][e] += __shfl_xor_sync(0xFFFFFFFFu, o[c][k][nt][e], 2);
      }
      const float2 m2 = split(mx[nt]);
      float2 l2 = split(l[nt]), vm2[NG];
#pragma unroll
      for (int n = 0; n < NG; ++n) vm2[n] = split(vm[nt][n]);
#pragma unroll
      for (int sft = 4; sft < 32; sft <<= 1) {
        l2.x += __shfl_xor_sync(0xFFFFFFFFu, l2.x, sft);
        l2.y += __shfl_xor_sync(0xFFFFFFFFu, l2.y, sft);
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          vm2[n].x += __shfl_xor_sync(0xFFFFFFFFu, vm2[n].x, sft);
          vm2[n].y += __shfl_xor_sync(0xFFFFFFFFu, vm2[n].y, sft);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = nt * 8 + 2 * j + e;
        if (r >= RP) continue;
        if (g == 0) {
          sm[gwarp * RP + r] = -(e ? m2.y : m2.x);
          sl[gwarp * RP + r] = e ? l2.y : l2.x;
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
          // 2^18 / |inv| in two factors, 2^12 and 2^6 / |inv|: it may pass fp32's range
          // where the value does not
          const float2 iv = split(inv[nt][c / A::CG]);
          const float base = e ? vm2[c / A::CG].y : vm2[c / A::CG].x;
          const float top = largest_beside(e ? iv.y : iv.x);
          auto value = [&](float sum) { return fmaf(sum * 4096.0f, top, base); };
          *reinterpret_cast<float4*>(so + (gwarp * RP + r) * D + 32 * c + 4 * g) =
              make_float4(value(o[c][0][nt][e]), value(o[c][1][nt][e]), value(o[c][0][nt][e + 2]),
                          value(o[c][1][nt][e + 2]));
        }
      }
    }
    group_barrier();
    if (gtid < RP) {
      float top = kNoMax, sum = 0.0f;
      for (int w = 0; w < warps; ++w) top = fmaxf(top, sm[w * RP + gtid]);
      for (int w = 0; w < warps; ++w) {
        const float f = exp2_fast(sm[w * RP + gtid] - top);
        sf[w * RP + gtid] = f;
        sum += sl[w * RP + gtid] * f;
      }
      sm[gtid] = top;  // (this thread's column only)
      sl[gtid] = sum;
    }
    group_barrier();
    auto write = [&](int r, int ch, float v) {
      const int64_t at = (bh * p.rows + row0 + r) * D + ch;
      if (p.out_f32)
        static_cast<float*>(p.out)[at] = v;
      else
        static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
    };
    auto sum_of_warps = [&](int x) {
      const int r = x / D;
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < kAttnWarps; ++w) {
        if (w < warps) t = fmaf(so[w * RP * D + x], sf[w * RP + r], t);
      }
      return t;
    };
    auto write_whole = [&] {
      for (int x = gtid; x < min(RP, p.rows - row0) * D; x += threads) {
        const int r = x / D;
        write(r, x % D, sum_of_warps(x) * (sl[r] == 0.0f ? 0.0f : 1.0f / sl[r]));
      }
      if (gtid < min(RP, p.rows - row0))
        p.lse[bh * p.rows + row0 + gtid] = (sm[gtid] + log2f(sl[gtid])) * kLn2;
    };
    if (MODE == kGroups) return write_whole();
    if (MODE == kClusters) {
      // the CTA's O in place of its first warp's; then each CTA joins a share of it
      for (int x = tid; x < RP * D; x += kAttnThreads) so[x] = sum_of_warps(x);
      cluster_barrier();
      const int rank = blockIdx.x % p.cluster;
      const int n = min(RP, p.rows - row0) * D;
      for (int x = rank * kAttnThreads + tid; x < n; x += p.cluster * kAttnThreads) {
        const int r = x / D, ch = x % D;
        float m[kMostCluster], l8[kMostCluster], v[kMostCluster];
#pragma unroll
        for (int k = 0; k < kMostCluster; ++k) {  // (all loads at once)
          const bool there = k < p.cluster;
          m[k] = there ? peer_word(sm + r, k) : kNoMax;
          l8[k] = there ? peer_word(sl + r, k) : 0.0f;
          v[k] = there ? peer_word(so + x, k) : 0.0f;
        }
        float top = kNoMax, sum = 0.0f, t = 0.0f;
#pragma unroll
        for (int k = 0; k < kMostCluster; ++k) top = fmaxf(top, m[k]);
#pragma unroll
        for (int k = 0; k < kMostCluster; ++k) {
          const float f = exp2_fast(m[k] - top);
          sum = fmaf(l8[k], f, sum);
          t = fmaf(v[k], f, t);
        }
        write(r, ch, t * (sum == 0.0f ? 0.0f : 1.0f / sum));
        if (ch == 0) p.lse[bh * p.rows + row0 + r] = (top + log2f(sum)) * kLn2;
      }
      cluster_barrier();  // no CTA leaves while another reads its memory
      return;
    }
    if (s0 == 0 && s1 == steps) {
      write_whole();
    } else {
      float* slot = p.partial + (int64_t)(2 * blockIdx.x + (first_segment ? 0 : 1)) * A::kSlot;
      for (int x = tid; x < RP * D; x += kAttnThreads) slot[2 * RP + x] = sum_of_warps(x);
      if (tid < RP) {
        slot[tid] = sm[tid];
        slot[RP + tid] = sl[tid];
      }
    }
    __syncthreads();
    u += n_tiles;
    first_segment = false;
  }
}

// One CTA per (row of a tile, row tile, head, sequence): joins the partial
// results of a head that several CTAs shared, in their order (a lane group
// reads a slot's row, 16 bytes a lane; the groups' sums are added in a fixed
// order); writes the empty result where there is nothing to see.
template <int D, int RP>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(const AttnParams p) {
  constexpr int kSlot = RP * (D + 2);
  constexpr int L = D / 4, kParts = kJoinThreads / L;  // slots read at once
  __shared__ float4 red[kParts][L];
  __shared__ float sums[kParts];
  __shared__ float tops[kJoinThreads / 32];
  wait_for_previous_launch();
  allow_next_launch();
  const int heads = p.c.Hkv * p.mt;
  const int b = blockIdx.x / heads, hm = blockIdx.x - b * heads;
  const int h = hm / p.mt, r = blockIdx.y;
  const int row = (hm - h * p.mt) * RP + r;
  if (row >= p.rows) return;
  const int64_t before = __ldcg(p.prefix + b), steps = __ldcg(p.prefix + b + 1) - before;
  const int64_t units = (int64_t)__ldcg(p.prefix + p.B) * heads;
  const int64_t out_row = ((int64_t)b * p.c.Hkv + h) * p.rows + row;
  const int cl = threadIdx.x % L, part = threadIdx.x / L;
  auto write = [&](float4 v, float lse) {
    if (part != 0) return;
    const int64_t at = out_row * D + cl * 4;
    if (p.out_f32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = v;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
          make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
    if (cl == 0) p.lse[out_row] = lse;
  };
  if (steps == 0) return write(make_float4(0, 0, 0, 0), -INFINITY);
  const int ctas = (int)min((int64_t)p.ctas, units);
  const int64_t u0 = before * heads + hm * steps;
  const int c0 = range_of(units, ctas, u0), c1 = range_of(units, ctas, u0 + steps - 1);
  if (c0 == c1) return;  // one CTA had it all and wrote the result
  // the head is CTA c's first segment unless c's range began before it
  auto slot_of = [&](int c) -> const float* {
    const bool first = range_begin(units, ctas, c) >= u0;
    return p.partial + (int64_t)(2 * c + (first ? 0 : 1)) * kSlot;
  };
  float top = kNoMax;
  for (int c = c0 + threadIdx.x; c <= c1; c += kJoinThreads)
    top = fmaxf(top, __ldcg(slot_of(c) + r));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if ((threadIdx.x & 31) == 0) tops[threadIdx.x / 32] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) top = fmaxf(top, tops[w]);
  float4 t = make_float4(0, 0, 0, 0);
  float sum = 0.0f;
#pragma unroll 4
  for (int c = c0 + part; c <= c1; c += kParts) {
    const float* s = slot_of(c);
    const float f = exp2_fast(__ldcg(s + r) - top);
    const float4 v = __ldcg(reinterpret_cast<const float4*>(s + 2 * RP + r * D) + cl);
    sum = fmaf(__ldcg(s + RP + r), f, sum);
    t.x = fmaf(v.x, f, t.x), t.y = fmaf(v.y, f, t.y);
    t.z = fmaf(v.z, f, t.z), t.w = fmaf(v.w, f, t.w);
  }
  red[part][cl] = t;
  if (cl == 0) sums[part] = sum;
  __syncthreads();
  if (part != 0) return;
  t = make_float4(0, 0, 0, 0);
  sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kParts; ++w) {
    const float4 v = red[w][cl];
    t.x += v.x, t.y += v.y, t.z += v.z, t.w += v.w;
    sum += sums[w];
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  write(make_float4(t.x * inv, t.y * inv, t.z * inv, t.w * inv), (top + log2f(sum)) * kLn2);
}

template <int D, int NG, int NT, bool TWICE, bool SCORED>
cudaError_t launch_attn(const AttnParams& p, int grid, cudaStream_t st) {
  using A = Attn<D, NG, NT, TWICE>;
  constexpr size_t most = A::kSmem + (size_t)(kMostSequences + 1) * sizeof(int);
  static_assert(most <= 210 * 1024, "shared memory");
  if (p.group) {
    constexpr auto kernel = kv4_attn_kernel<D, NG, NT, TWICE, kGroups, SCORED>;
    cudaError_t e = allow_shared_memory<kernel>(A::kSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(grid), dim3(kAttnThreads), A::kSmem, st, p);
  }
  if (p.cluster) {
    constexpr auto kernel = kv4_attn_kernel<D, NG, NT, TWICE, kClusters, SCORED>;
    cudaError_t e = allow_shared_memory<kernel>(A::kSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent_clusters(kernel, dim3(grid), dim3(kAttnThreads), p.cluster, A::kSmem,
                                     st, p);
  }
  const size_t smem = A::kSmem + (size_t)(p.B + 1) * sizeof(int);
  cudaError_t e = allow_shared_memory<kv4_attn_kernel<D, NG, NT, TWICE, kRanges, SCORED>>((int)most);
  if (e != cudaSuccess) return e;
  e = launch_dependent(kv4_attn_kernel<D, NG, NT, TWICE, kRanges, SCORED>, dim3(grid), dim3(kAttnThreads),
                       smem, st, p);
  if (e != cudaSuccess) return e;
  return launch_dependent(kv4_join_kernel<D, A::RP>,
                          dim3(p.B * p.c.Hkv * p.mt, p.rows < A::RP ? p.rows : A::RP),
                          dim3(kJoinThreads), 0, st, p);
}

// Up to 4 rows a head: each row twice (32 x 8 heads of 32768 tokens: 211 us, one
// tile of 8 230 us); up to 8: one tile; more: tiles of 16 rows, which decode the
// codes once for both halves (16 rows, 8 x 8 heads of 49152 tokens: 163 us when two
// tiles of 8 took 183 us, 157 us now; one sequence: 33 and 37 us).
template <int D, int NG, bool SCORED>
cudaError_t launch_attn(const AttnParams& p, int grid, cudaStream_t st) {
  if (p.rows <= 4) return launch_attn<D, NG, 1, true, SCORED>(p, grid, st);
  if (p.rows <= 8) return launch_attn<D, NG, 1, false, SCORED>(p, grid, st);
  return launch_attn<D, NG, 2, false, SCORED>(p, grid, st);
}

// How many clusters of 1 to kMostCluster CTAs run at once, by tiles of 8 rows a
// CTA.  A cluster stays inside one of the chip's groups of SMs, so these are
// fewer than the CTAs that the SMs hold: with 16 rows 15 clusters of 8 on 152
// SMs, not 19.  One too many costs a second wave (16 heads of 16 rows, 8192
// tokens: 33 us as clusters of 8, 21 us of 6).  Asked once a device, of the
// kernels with the most shared memory.
struct ActiveClusters {
  int n[2][kMostCluster + 1];
};
template <int NT>
void ask_active_clusters(int sms, int (&n)[kMostCluster + 1]) {
  using A = Attn<128, 4, NT, false>;
  constexpr auto kernel = kv4_attn_kernel<128, 4, NT, false, kClusters, kScored>;
  n[0] = 0;
  for (int c = 1; c <= kMostCluster; ++c) {
    n[c] = (NT == 1 ? kPerSm : 1) * sms / (2 * c);  // where the question fails
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(c);
    cfg.blockDim = dim3(kAttnThreads);
    cfg.dynamicSmemBytes = A::kSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = c;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int most = 0;
    if (allow_shared_memory<kernel>(A::kSmem) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&most, kernel, &cfg) == cudaSuccess)
      n[c] = most;
    else
      cudaGetLastError();
  }
}
const int (&active_clusters(int nt, int sms))[kMostCluster + 1] {
  constexpr int kDevices = 64;
  static ActiveClusters known[kDevices];
  static std::once_flag asked[kDevices];
  int dev = 0;
  cudaGetDevice(&dev);
  dev = dev < kDevices ? dev : kDevices - 1;
  std::call_once(asked[dev], [&] {
    ask_active_clusters<1>(sms, known[dev].n[0]);
    ask_active_clusters<2>(sms, known[dev].n[1]);
  });
  return known[dev].n[nt - 1];
}

// How a call is split: by its sizes and the device only, so that the workspace's
// size is known beforehand.
struct AttnSplit {
  int nt, mt;      // tiles of 8 rows a CTA, row tiles a head
  int64_t steps;   // of a sequence, by the room of its table or list
  int ctas, grid, cluster, group;
  size_t prefix_bytes, workspace;
};
AttnSplit attn_split(int B, int kv_heads, int64_t rows, int64_t tokens, int D, int sms) {
  AttnSplit s{};
  s.nt = rows <= 8 ? 1 : 2;
  s.mt = (int)((rows + 8 * s.nt - 1) / (8 * s.nt));
  s.steps = (tokens + kStep - 1) / kStep;
  s.ctas = s.nt == 1 ? kPerSm * sms : sms;  // as many as run at once
  const int64_t heads = (int64_t)B * kv_heads * s.mt;
  // Up to as many heads as CTAs: a cluster a head, the largest of which all run at
  // once, where that leaves no CTA with more to do than ranges over all CTAs would:
  // those cost most CTAs a second start and everyone the second launch, about
  // kSegmentSteps steps.
  const auto& active = active_clusters(s.nt, sms);
  int64_t share = kMostCluster;
  while (share > 0 && heads > active[share]) --share;
  if (share > s.steps) share = s.steps;
  if (share >= 1) {
    const int64_t most = (s.steps + share - 1) / share;
    if (most <= kMostGroupSteps && most <= s.steps * heads / s.ctas + kSegmentSteps) {
      if (share == 1)
        s.group = kAttnWarps;
      else
        s.cluster = (int)share;
      s.grid = (int)(heads * share);
      return s;
    }
  } else {
    // More heads than CTAs: a group of 8, 4, 2 or 1 warps a head.  Fewer warps a
    // head take fewer waves of CTAs, each with a start of its own, of more steps.
    // 2048 heads of 128 tokens, 4 rows each: 45, 30, 23, 19 us, as ranges 54;
    // of 512 tokens 68, 52, 47, 41 (83); of 2048 140, 123, 129, 127 (158); 384
    // heads of 4096 tokens 60, 68, 84, 160 (68).
    double best = (double)s.steps * heads / s.ctas +
                  kSegmentStart * ((double)heads / s.ctas + 2);
    for (int warps = kAttnWarps; warps >= 1; warps /= 2) {
      const int64_t a_cta = kAttnWarps / warps, steps = (tokens + kTile * warps - 1) / (kTile * warps);
      const int64_t grid = (heads + a_cta - 1) / a_cta, waves = (grid + s.ctas - 1) / s.ctas;
      const double cost = (double)waves * (steps + kGroupStart);
      if (steps <= kMostGroupSteps && cost < best) {
        best = cost;
        s.group = warps;
        s.grid = (int)grid;
      }
    }
    if (s.group) return s;
  }
  if (heads * kMostParts < s.ctas) s.ctas = (int)(heads * kMostParts);
  if (s.steps * heads < s.ctas) s.ctas = (int)(s.steps * heads);  // no more than units
  s.grid = s.ctas;
  s.prefix_bytes = ((size_t)(B + 1) * sizeof(int) + 15) / 16 * 16;
  s.workspace = s.prefix_bytes + (size_t)2 * s.ctas * 8 * s.nt * (D + 2) * sizeof(float);
  return s;
}

// Tokens that a call may see of a sequence; 0 for sizes that no call takes.
int64_t attn_tokens(int page_size, int columns, int n_selected) {
  if (page_size <= 0 || columns <= 0 || n_selected < 0) return 0;
  return (int64_t)page_size * (n_selected > 0 ? n_selected : columns);
}

// One launch with everything checked: p without what the split says.
template <bool SCORED>
cudaError_t launch_split(AttnParams& p, const AttnSplit& split, const bsattn_kv4_cache* cache,
                         void* workspace, cudaStream_t st) {
  p.mt = split.mt;
  p.prefix = static_cast<int*>(workspace);
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + split.prefix_bytes);
  p.ctas = split.ctas;
  p.cluster = split.cluster;
  p.group = split.group;
  p.tiles = (int)(p.B * cache->kv_heads * split.mt);
  const int groups = cache->head_dim / cache->group;
  if (cache->head_dim == 64)
    return groups == 1 ? launch_attn<64, 1, SCORED>(p, split.grid, st)
                       : launch_attn<64, 2, SCORED>(p, split.grid, st);
  return groups == 1   ? launch_attn<128, 1, SCORED>(p, split.grid, st)
         : groups == 2 ? launch_attn<128, 2, SCORED>(p, split.grid, st)
                       : launch_attn<128, 4, SCORED>(p, split.grid, st);
}

}  // namespace
}  // namespace bsattn
