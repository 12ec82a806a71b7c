// The paged key/value cache in 4 bits: writing new tokens into it, reading
// tokens back, and choosing pages for a query.  (Attention over it:
// kv4_attn.cu.)
//
// Per (token, head) row and group of g channels (g = 32, 64 or 128):
//   minimum = min x,  step = bf16((max x - min x) / 15),
//   code = (x - minimum) / step rounded to the nearest whole number, half to even,
//   value = step * code + minimum.
// The minimum is one of the inputs, so bf16 holds it exactly; the step's
// rounding is part of the format (codes are taken with the rounded step).  A
// group whose step is below 2^-100 counts as constant (codes 0); a group with
// a NaN or an infinity, or whose range overflows, decodes to NaN.
#include <cmath>
#include <cstdint>

#include "kv4.cuh"

namespace bsattn {
namespace {

constexpr int kRowThreads = 128;  // write_rounded_mean takes a CTA of 128
constexpr int kFewTokens = 8;
constexpr int kReadRows = 4;      // rows a lane group reads back at once
constexpr float kLeastStep = 7.888609e-31f;  // 2^-100

struct AppendParams {
  Kv4View c;
  const uint16_t* k;  // [B][Hkv][T][D], strides in elements
  const uint16_t* v;
  int64_t kb, kh, kt, vb, vh, vt;
  const int* table;
  int64_t table_stride;
  int columns;
  const int* lengths;
  const int* counts;  // null: T each
  int T;
};

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {  // of bf16 pairs; NaN stays
  __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<__nv_bfloat162*>(&a),
                                 *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&a),
                                 *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}

// A pair with its magnitudes brought up to `least`; zeros stay.
__device__ __forceinline__ uint32_t at_least(uint32_t a, __nv_bfloat162 least) {
  const __nv_bfloat162 v = *reinterpret_cast<__nv_bfloat162*>(&a);
  const __nv_bfloat162 m = __hmax2(__habs2(v), least);
  const uint32_t up = *reinterpret_cast<const uint32_t*>(&m) | (a & 0x80008000u);
  const unsigned there = __hne2_mask(v, __float2bfloat162_rn(0.0f));
  return (a & ~there) | (up & there);
}

// Sixteen channels of one group's row -> codes (a nibble each, the first
// lowest; n[i]: channels 2i, 2i + 1 as floats), and the group's step and least.
// GL lanes hold a group.
//
// d / step, d = x - least, is estimated with the reciprocal and corrected by its
// exact remainder: q = q0 + (d - q0 step) / step, good to 2^-46 before its one
// rounding; adding 1.5 2^23 then rounds it half to even with no conversion
// instruction.  The codes are those of the real quotient of d: at a border it is
// k + 1/2 exactly, which 32 bits hold, and next to one d differs from
// (k + 1/2) step, a number of 13 bits, by a step of d at least, so the quotient
// by more than its own rounding.  d itself would be rounded where x and least are
// more than 2^16 apart, which matters at a border: d = (k + 1/2) step would stand
// for numbers on both sides of it.  Either least is the small one, or x is and
// -least lies on the border; the small one then counts as 2^-15 of the other, of
// its own sign: d is exact, on its side of the border, and as far from others
// (2^-12 of the range at least) as before.  The step's (most - least) / 15 is
// taken the same way, and is the 32-bit quotient: no a / 15 comes closer to the
// middle between two floats than 2^-29 of itself.
template <int GL>
__device__ __forceinline__ uint2 quantise(uint32_t (&w)[8], F2 (&n)[8], float& step,
                                          float& least) {
  uint32_t lo = w[0], hi = w[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) lo = min2(lo, w[i]), hi = max2(hi, w[i]);
  lo = min2(lo, __byte_perm(lo, lo, 0x1032));
  hi = max2(hi, __byte_perm(hi, hi, 0x1032));
  // (least, -most) in one word: one shuffle a level
  uint32_t both = (lo & 0x0000FFFFu) | ((hi ^ 0x80000000u) & 0xFFFF0000u);
#pragma unroll
  for (int o = 1; o < GL; o <<= 1) both = min2(both, __shfl_xor_sync(0xFFFFFFFFu, both, o));
  least = bf16_lo(both);
  const float range = -bf16_hi(both) - least;  // NaN or infinite for a group that is not finite
  constexpr float kFifteenth = 1.0f / 15.0f;
  const float r0 = range * kFifteenth;
  step = __bfloat162float(__float2bfloat16_rn(fmaf(fmaf(-15.0f, r0, range), kFifteenth, r0)));
  const bool finite = range <= 3.4028234e38f, flat = step < kLeastStep;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(step));
  constexpr float kFar = 3.0517578125e-5f;  // 2^-15
  float from = least;
  if (least != 0.0f && fabsf(least) < kFar * range)
    from = copysignf(kFar * __uint_as_float(__float_as_uint(range) & 0x7F800000u), least);
  if (least != 0.0f && fmaf(rintf(-2.0f * least * inv), step, 2.0f * least) == 0.0f) {
    const __nv_bfloat162 far = __float2bfloat162_rn(kFar * fabsf(least));
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = at_least(w[i], far);
  }
  const F2 vinv = f2(inv), vstep = f2(-step), vleast = f2(-from);
  const F2 magic = f2(12582912.0f), unmagic = f2(-12582912.0f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const F2 d = bf16_pair(w[i]) + vleast;
    const F2 q0 = d * vinv;
    n[i] = fma2(fma2(q0, vstep, d), vinv, q0) + magic + unmagic;
  }
  if (!finite || flat) {
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] = f2(0.0f);
    step = finite ? 0.0f : __int_as_float(0x7FC00000);
    least = finite ? least : step;
  }
  // four codes a sum, exactly: (n0, n1) + 256 (n2, n3), then n0 + 16 n1
  uint32_t half[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 s = split(fma2(n[2 * i + 1], f2(256.0f), n[2 * i]));
    half[i] = __float_as_uint(fmaf(s.y, 16.0f, s.x) + 8388608.0f);
  }
  return make_uint2(__byte_perm(half[0], half[1], 0x5410), __byte_perm(half[2], half[3], 0x5410));
}

// The values of eight codes.  Code i is read as (2^23 + code 16^i) - 2^23 in
// place (codes 5 to 7 after one shift) and multiplied by step 16^-i: the same
// product, exactly, as step * code.
struct Decoder {
  F2 s01, s23, s4, s12, least;

  __device__ __forceinline__ Decoder(float step, float l) {
    const float s1 = step * 0.0625f, s2 = step * 0.00390625f;
    s01 = f2(step, s1);
    s23 = f2(s2, step * 2.44140625e-4f);
    s4 = f2(step * 1.52587890625e-5f, step);
    s12 = f2(s1, s2);
    least = f2(l);
  }
  __device__ __forceinline__ void decode8(uint32_t codes, F2* x) const {
    const uint32_t up = codes >> 20;
    const F2 off = f2(-8388608.0f);
    auto field = [](uint32_t v, int bit) {
      return __uint_as_float((v & (15u << bit)) | 0x4B000000u);
    };
    x[0] = fma2(f2(field(codes, 0), field(codes, 4)) + off, s01, least);
    x[1] = fma2(f2(field(codes, 8), field(codes, 12)) + off, s23, least);
    x[2] = fma2(f2(field(codes, 16), field(up, 0)) + off, s4, least);
    x[3] = fma2(f2(field(up, 4), field(up, 8)) + off, s12, least);
  }
};

// Rows first .. of the cnt new tokens of sequence b, token by token, the heads of
// K and then of V: a lane group a row.
template <int D, int GL>
__device__ __forceinline__ void append_rows(const AppendParams& p, int b, int len, int cnt,
                                            int first, int sub, int cl) {
  constexpr int L = D / 16, NG = L / GL;
  const int heads = 2 * p.c.Hkv, r = first + sub, t = r / heads, place = r - t * heads;
  const bool is_k = place < p.c.Hkv;
  const int h = is_k ? place : place - p.c.Hkv;
  uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
  int pg = -1;
  if (t < cnt) {
    const uint16_t* src = is_k ? p.k + b * p.kb + h * p.kh + t * p.kt
                               : p.v + b * p.vb + h * p.vh + t * p.vt;
    lo = load(reinterpret_cast<const uint4*>(src) + 2 * cl);
    hi = load(reinterpret_cast<const uint4*>(src) + 2 * cl + 1);
    pg = page_at(p.c, p.table + b * p.table_stride, p.columns, ((int64_t)len + t) >> p.c.log_page);
  }
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  F2 x[8];
  float step, least;
  const uint2 packed = quantise<GL>(w, x, step, least);  // (every lane: shuffles)
  if (pg < 0) return;
  const int64_t row = p.c.row(pg, h, (int)(((int64_t)len + t) & (p.c.page - 1)));
  reinterpret_cast<uint2*>(is_k ? p.c.k_codes : p.c.v_codes)[row * L + cl] = packed;
  if (cl % GL == 0)
    reinterpret_cast<uint32_t*>(is_k ? p.c.k_scales : p.c.v_scales)[row * NG + cl / GL] =
        pack_bf16(step, least);
}

// One CTA: K or V of one page of one sequence and head, the tokens of this call
// that fall into it.  A row is held by D / 16 lanes, and the next row's load is
// in flight while one is quantised.  When the call fills the page the CTA of K
// adds up the page's decoded keys (those of earlier calls are read back) and
// writes their rounded mean.
//
// 512 bytes read and 160 written a token and head (groups of 32): the bound is
// memory on paper, instructions in fact, some 20 a channel's lane.  8 x 4096
// tokens (three quarters of them there), 8 heads of 128: 43 us, 70% of issue
// slots, 3.4 TB/s (42 us without the care for far values); with conversions and comparisons a code 104 us, with a lane
// for 8 channels instead of 16 59 us, with the next two rows in flight no less,
// with 8 CTAs an SM (64 registers, spilling) 47 us.
//
// FEW tokens (up to kFewTokens, decoding steps): CTAs behind those of the heads of
// K write all rows, as many a CTA as it holds, and those of the heads only see to
// the means of pages that fill, which one token in a page's does.
// 512 sequences, 8 heads of 128, of one token: 9 us (a CTA for each head's K and
// V: 17 us), of 8 tokens: 13 us (21 us).
template <int D, int GL, bool FEW>
__global__ void __launch_bounds__(kRowThreads, 6) kv4_append_kernel(const AppendParams p) {
  constexpr int L = D / 16, NG = L / GL, kRows = kRowThreads / L;  // rows the CTA holds at once
  const bool is_k = blockIdx.y < p.c.Hkv;
  const int h = is_k ? blockIdx.y : blockIdx.y - p.c.Hkv, b = blockIdx.z;
  wait_for_previous_launch();
  allow_next_launch();
  const int len = load(p.lengths + b);
  int cnt = p.T;
  if (p.counts) cnt = min(max(load(p.counts + b), 0), p.T);
  if (cnt == 0) return;
  if (len < 0) {
    if (threadIdx.x == 0) p.c.report();
    return;
  }
  const int sub = threadIdx.x / L, cl = threadIdx.x % L;
  if (FEW) {
    if (!is_k) return append_rows<D, GL>(p, b, len, cnt, h * kRows, sub, cl);
    if ((((int64_t)len + cnt) >> p.c.log_page) == (len >> p.c.log_page)) return;
  }
  const int64_t logical = (len >> p.c.log_page) + (int64_t)blockIdx.x;
  const int64_t end = min((int64_t)len + cnt, (logical + 1) << p.c.log_page);
  const int64_t begin = max((int64_t)len, logical << p.c.log_page);
  if (begin >= end) return;
  const int n = (int)(end - begin), place0 = (int)(begin & (p.c.page - 1));
  // the first row is on its way while the table is asked
  const int64_t token = is_k ? p.kt : p.vt;
  const uint16_t* src = (is_k ? p.k + b * p.kb + h * p.kh : p.v + b * p.vb + h * p.vh) +
                        (begin - len + sub) * token + cl * 16;
  uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
  if (sub < n) {
    lo = load(reinterpret_cast<const uint4*>(src));
    hi = load(reinterpret_cast<const uint4*>(src) + 1);
  }
  const int pg = page_at(p.c, p.table + b * p.table_stride, p.columns, logical);
  if (pg < 0) return;
  const bool sums = is_k && end == (logical + 1) << p.c.log_page;
  const int64_t row0 = p.c.row(pg, h, 0);

  Sum2x2 s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i].hi = s[i].lo = f2(0.0f);
  const int rounds = (n + kRows - 1) / kRows;
  const int64_t row = row0 + place0 + sub;
  uint2* codes = reinterpret_cast<uint2*>(is_k ? p.c.k_codes : p.c.v_codes) + row * L + cl;
  uint32_t* scales =
      reinterpret_cast<uint32_t*>(is_k ? p.c.k_scales : p.c.v_scales) + row * NG + cl / GL;
  for (int i = 0; i < rounds; ++i) {  // (as many for every lane: shuffles)
    const bool there = i * kRows + sub < n;
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    src += kRows * token;
    if ((i + 1) * kRows + sub < n) {
      lo = load(reinterpret_cast<const uint4*>(src));
      hi = load(reinterpret_cast<const uint4*>(src) + 1);
    }
    F2 x[8];
    float step, least;
    const uint2 packed = quantise<GL>(w, x, step, least);
    if (there) {
      if (!FEW) {
        *codes = packed;
        if (cl % GL == 0) *scales = pack_bf16(step, least);
      }
      if (sums) {
#pragma unroll
        for (int k = 0; k < 8; ++k) add_exact(s[k], fma2(x[k], f2(step), f2(least)));
      }
    }
    codes += kRows * L;
    scales += kRows * NG;
  }
  if (!sums) return;
  for (int r = sub; r < place0; r += kRows) {
    const int64_t at = row0 + r;
    const uint2 packed = reinterpret_cast<const uint2*>(p.c.k_codes)[at * L + cl];
    const uint32_t sc = reinterpret_cast<const uint32_t*>(p.c.k_scales)[at * NG + cl / GL];
    const Decoder dec(bf16_lo(sc), bf16_hi(sc));
    F2 x[8];
    dec.decode8(packed.x, x);
    dec.decode8(packed.y, x + 4);
#pragma unroll
    for (int k = 0; k < 8; ++k) add_exact(s[k], x[k]);
  }
  write_rounded_mean<D>(s, p.c.page, false, p.c.k_means + ((int64_t)pg * p.c.Hkv + h) * D);
}

struct ReadParams {
  Kv4View c;
  const int* table;
  int64_t table_stride;
  int columns;
  const int* start;
  const int* counts;
  int T;
  uint16_t* k;
  uint16_t* v;
  int wide;  // k and v are aligned to 32 bytes
};

// One CTA: consecutive rows of one sequence and head; a lane group (D / 16
// lanes) decodes kReadRows of them, K and V.  Rows behind the count are zero.
// Bound by its stores: the tokens above in 26 us, 5.1 TB/s.
template <int D, int GL>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(const ReadParams p) {
  constexpr int L = D / 16, NG = L / GL;
  constexpr int kGroups = kRowThreads / L;
  const int cl = threadIdx.x % L, group = threadIdx.x / L;
  const int h = blockIdx.y, b = blockIdx.z;
  const int t0 = blockIdx.x * (kGroups * kReadRows) + group;
  wait_for_previous_launch();
  allow_next_launch();
  const int count = p.counts ? min(load(p.counts + b), p.T) : p.T;
  const int64_t start = load(p.start + b);
  const int* table = p.table + b * p.table_stride;
  // the table's answers for all rows, then all rows' loads
  int pg[kReadRows];
#pragma unroll
  for (int u = 0; u < kReadRows; ++u) {
    const int t = t0 + u * kGroups;
    const int64_t logical = (start + t) >> p.c.log_page;
    pg[u] = -2;  // nothing to read
    if (t < count) pg[u] = logical >= 0 && logical < p.columns ? load(table + logical) : -1;
  }
  uint2 code[kReadRows][2];
  uint32_t sc[kReadRows][2];
#pragma unroll
  for (int u = 0; u < kReadRows; ++u) {
    const bool there = pg[u] >= 0 && pg[u] < p.c.pages;
    if (!there && pg[u] != -2) p.c.report();
    const int64_t row =
        p.c.row(there ? pg[u] : 0, h, (int)((start + t0 + u * kGroups) & (p.c.page - 1)));
    code[u][0] = code[u][1] = make_uint2(0, 0);
    sc[u][0] = sc[u][1] = 0u;
    if (there) {
      code[u][0] = reinterpret_cast<const uint2*>(p.c.k_codes)[row * L + cl];
      code[u][1] = reinterpret_cast<const uint2*>(p.c.v_codes)[row * L + cl];
      sc[u][0] = reinterpret_cast<const uint32_t*>(p.c.k_scales)[row * NG + cl / GL];
      sc[u][1] = reinterpret_cast<const uint32_t*>(p.c.v_scales)[row * NG + cl / GL];
    }
  }
  const int64_t out = (((int64_t)b * p.c.Hkv + h) * p.T + t0) * D + cl * 16;
#pragma unroll
  for (int u = 0; u < kReadRows; ++u) {
    if (t0 + u * kGroups >= p.T) continue;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const Decoder dec(bf16_lo(sc[u][kv]), bf16_hi(sc[u][kv]));
      F2 x[8];
      dec.decode8(code[u][kv].x, x);
      dec.decode8(code[u][kv].y, x + 4);
      uint32_t y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = pack_bf16(x[i]);
      store32((kv ? p.v : p.k) + out + u * kGroups * D, y, p.wide != 0);
    }
  }
}

// ---------------------------------------------------------------------------
// Choosing pages: the single-token form of the block choice in select.cu.
// The queries of one key/value head (G heads, T tokens) are rounded to 7 bits
// beside their largest entry (whole numbers t); a page's score is the largest
// of t . mean over those queries: a whole number times the page's power of
// two, exact in 32 bits.  The last `recent` pages and the first `sink` are
// always taken; of the others the best, the lowest index first among equals.
//
// Bound: memory, one row of D bf16 a page, or latency where there are few.  One
// CTA scores a head's pages and chooses among them while that keeps the
// machine busy or the list is short; else scores and choice are two launches.
// ---------------------------------------------------------------------------
constexpr int kPageThreads = 512;
// More heads than SMs: CTAs of 128 threads, four of which an SM holds, so that the
// starts, barriers and searches of one pass beside the others.  2048 heads of 64
// pages: 21 us, with 512 threads 64 us; of 1024 pages 88 and 131 us; 256 heads of
// 16 pages 7 and 11 us.
constexpr int kFewPageThreads = 128;
constexpr int kTiles = 2;        // tiles of 16 pages that a warp has in flight
constexpr int kMostRows = 128;   // G * T
constexpr int kVec = 4;          // 16-byte pieces of the queries a thread
template <int THREADS>
constexpr int kRound = THREADS / 32 * kTiles * 16;  // pages that a CTA scores at once
constexpr int kRoundPages = kRound<kPageThreads>;  // all of a CTA's in the split form
// One launch for lists up to this room: 8 heads of 500 pages 8 us (two launches 10),
// of 2000 pages 15 us (12, but another launch for the host); 128 heads of 1000
// pages 13 us (19).
constexpr int kOneCtaPages = 2048;
constexpr int kMostShared = 16 * kPageThreads;  // keys in shared memory
constexpr uint32_t kForcedPage = 0xFFFFFFFFu;
static_assert(kMostRows * 128 <= kPageThreads * kVec * 8, "queries");
// (a call with kFewPageThreads asks for no more than the usual shared memory: rows to a
// multiple of 8)
static_assert(kFewPageThreads * kVec * 16 + 7 * 256 + kOneCtaPages * 4 <= 48 << 10, "shared memory");
constexpr uint32_t kNoPage = 0u;

struct PagesParams {
  Kv4View c;
  const uint16_t* q;  // [B][H][T][D]
  const int* table;
  int64_t table_stride;
  int columns;
  const int* lengths;
  int rows;  // G * T
  int keep, sink, recent;
  uint32_t* keys;  // [B * Hkv][columns] (the split form)
  int* out;        // [B * Hkv][keep]
};

__device__ __forceinline__ int pages_of(const PagesParams& p, int b) {
  const int64_t n = ((int64_t)max(load(p.lengths + b), 0) + p.c.page - 1) >> p.c.log_page;
  if (n > p.columns && threadIdx.x == 0) p.c.report();
  return (int)min(n, (int64_t)p.columns);
}

// Rounds the queries of (sequence, head) bh into `whole` ([rows, to a multiple
// of 8][D] bf16, zero rows at the end).  All threads of the CTA.
template <int D, int THREADS>
__device__ __forceinline__ void round_queries(const PagesParams& p, int64_t bh, uint16_t* whole) {
  constexpr int kWarps = THREADS / 32;
  __shared__ uint32_t top[kWarps];
  const uint4* q = reinterpret_cast<const uint4*>(p.q + bh * p.rows * D);
  const int pieces = p.rows * D / 8, room = (p.rows + 7) / 8 * 8 * D / 8;
  uint4 v[kVec];
  uint32_t most = 0;  // bits of the largest finite |q|
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int at = threadIdx.x + i * THREADS;
    v[i] = make_uint4(0, 0, 0, 0);
    if (at >= pieces) continue;
    v[i] = load(q + at);
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t lo = w[k] & 0x7FFFu, hi = (w[k] >> 16) & 0x7FFFu;
      most = max(most, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
    }
  }
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = most;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) most = max(most, top[w]);
  // t = rint(q 2^(6 - e)), in two factors, for 2^(6 - e) may pass fp32's range
  const int shift = most ? 6 - ilogbf(__uint_as_float(most << 16)) : 0;
  const float f1 = ldexpf(1.0f, shift / 2), f2 = ldexpf(1.0f, shift - shift / 2);
  auto round1 = [&](float x) { return fabsf(x) <= 3.4e38f ? rintf(x * f1 * f2) : 0.0f; };
  auto round2 = [&](uint32_t w) { return pack_bf16(round1(bf16_lo(w)), round1(bf16_hi(w))); };
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int at = threadIdx.x + i * THREADS;
    if (at < room)
      reinterpret_cast<uint4*>(whole)[at] =
          make_uint4(round2(v[i].x), round2(v[i].y), round2(v[i].z), round2(v[i].w));
  }
  __syncthreads();
}

// Scores pages first .. end - 1 of a sequence with n pages into keys[page]: each
// warp kTiles tiles of 16 pages at once, pages as the product's rows and
// queries as its columns, so that a page's best query is two shuffles away.
// The loads of a round are issued before `whole` is needed (ready() fills it).
template <int D, int THREADS, typename Ready>
__device__ __forceinline__ void score_pages(const PagesParams& p, int b, int h, int n, int first,
                                            int end, const uint16_t* whole, uint32_t* keys,
                                            Ready ready) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, j = lane & 3;
  const int* table = p.table + b * p.table_stride;
  bool waiting = true;
  int next[2 * kTiles];  // the table's answers for the next round
  auto look_up = [&](int at) {
#pragma unroll
    for (int k = 0; k < 2 * kTiles; ++k)
      next[k] = at + 8 * k < end ? load(table + at + 8 * k) : -1;
  };
  look_up(first + warp * (kTiles * 16) + g);
  for (int base = first; base < end; base += kRound<THREADS>) {
    const int at = base + warp * (kTiles * 16) + g;  // this lane's pages: at + 8 k
    bool there[2 * kTiles];
    uint4 w[2 * kTiles][C];
#pragma unroll
    for (int k = 0; k < 2 * kTiles; ++k) {
      there[k] = next[k] >= 0 && next[k] < p.c.pages;
      if (!there[k] && at + 8 * k < end) p.c.report();
      // (a page that is not there: the first one's mean, and no key below)
      const uint4* mean = reinterpret_cast<const uint4*>(
          p.c.k_means + ((int64_t)(there[k] ? next[k] : 0) * p.c.Hkv + h) * D);
#pragma unroll
      for (int c = 0; c < C; ++c) w[k][c] = mean[4 * c + j];
    }
    look_up(at + kRound<THREADS>);
    if (waiting) ready();
    waiting = false;
    float best[2 * kTiles];
#pragma unroll
    for (int k = 0; k < 2 * kTiles; ++k) best[k] = -INFINITY;
    for (int row0 = 0; row0 < p.rows; row0 += 8) {
      const uint4* row = reinterpret_cast<const uint4*>(whole + (row0 + g) * D);
      float acc[kTiles][4];
#pragma unroll
      for (int k = 0; k < kTiles; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[k][i] = 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint4 q = row[4 * c + j];
#pragma unroll
        for (int k = 0; k < kTiles; ++k) {
          const uint4 lo = w[2 * k][c], hi = w[2 * k + 1][c];
          const uint32_t a0[4] = {lo.x, hi.x, lo.y, hi.y};
          const uint32_t a1[4] = {lo.z, hi.z, lo.w, hi.w};
          mma_bf16(acc[k], a0, q.x, q.y);
          mma_bf16(acc[k], a1, q.z, q.w);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (row0 + 2 * j + e < p.rows) {
#pragma unroll
          for (int k = 0; k < kTiles; ++k) {
            best[2 * k] = fmaxf(best[2 * k], acc[k][e]);
            best[2 * k + 1] = fmaxf(best[2 * k + 1], acc[k][2 + e]);
          }
        }
    }
#pragma unroll
    for (int k = 0; k < 2 * kTiles; ++k) {
      best[k] = fmaxf(best[k], __shfl_xor_sync(0xFFFFFFFFu, best[k], 1));
      best[k] = fmaxf(best[k], __shfl_xor_sync(0xFFFFFFFFu, best[k], 2));
      const int page = at + 8 * k;
      if (j == (k & 3) && page < end) {
        const bool forced = page < p.sink || page >= n - p.recent;
        keys[page] = !there[k] ? kNoPage : forced ? kForcedPage : ordered_bits(best[k]);
      }
    }
  }
  if (waiting) ready();
}

// Barrier of the CTA's first CT threads.
template <int CT>
__device__ __forceinline__ void choose_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(CT) : "memory");
}

// Sum over those threads of one number each (two uses in a row need other slots).
template <int CT>
__device__ __forceinline__ int block_sum(int v, int* slots) {
  v = __reduce_add_sync(0xFFFFFFFFu, v);
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
  choose_barrier<CT>();
  int s = 0;
#pragma unroll
  for (int w = 0; w < CT / 32; ++w) s += slots[w];
  return s;
}

// Exclusive prefix over them.
template <int CT>
__device__ __forceinline__ int block_prefix(int v, int* slots) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xFFFFFFFFu, s, o);
    if (lane >= o) s += t;
  }
  if (lane == 31) slots[warp] = s;
  choose_barrier<CT>();
  int before = 0;
#pragma unroll
  for (int w = 0; w < CT / 32; ++w) before += w < warp ? slots[w] : 0;
  return before + s - v;
}

// The best of n keys, by the first CT threads of the CTA of one
// (sequence, head): thread i holds KP consecutive keys (KP = 0: reads them again
// each time, for more pages than registers hold).  `keys` may be shared or global
// memory.  Each step of the search is a barrier of those threads.
template <int KP, int CT>
__device__ __forceinline__ void choose_pages(const PagesParams& p, const uint32_t* keys, int n,
                                             int* out) {
  __shared__ int slots[4][CT / 32];
  __shared__ uint32_t ends[2][CT / 32];
  const int per = KP > 0 ? KP : (n + CT - 1) / CT;
  const int64_t base = (int64_t)threadIdx.x * per;
  auto read = [&](int i) -> uint32_t { return base + i < n ? keys[base + i] : kNoPage; };
  uint32_t k[KP > 0 ? KP : 1];
  if (KP > 0) {
#pragma unroll
    for (int i = 0; i < KP; ++i) k[i] = read(i);
  }
  auto key = [&](int i) -> uint32_t { return KP > 0 ? k[i] : read(i); };
  auto each = [&](auto f) {
    if (KP > 0) {
#pragma unroll
      for (int i = 0; i < KP; ++i) f(k[i]);
    } else {
#pragma unroll 8
      for (int i = 0; i < per; ++i) f(read(i));
    }
  };
  int turn = 0;
  auto total = [&](int c) {
    turn ^= 1;
    return block_sum<CT>(c, slots[turn]);
  };
  // largest and least of the keys that are neither forced nor ruled out
  uint32_t top = 0, least = kForcedPage;
  int c = 0, f = 0;
  each([&](uint32_t x) {
    c += x != kNoPage ? 1 : 0;
    f += x == kForcedPage ? 1 : 0;
    top = max(top, x == kForcedPage ? 0u : x);
    least = min(least, x - 1u);  // 0 wraps: never the least
  });
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  least = __reduce_min_sync(0xFFFFFFFFu, least);
  if ((threadIdx.x & 31) == 0) {
    ends[0][threadIdx.x >> 5] = top;
    ends[1][threadIdx.x >> 5] = least;
  }
  const int there = total(c), forced = total(f);
#pragma unroll
  for (int w = 0; w < CT / 32; ++w) {
    top = max(top, ends[0][w]);
    least = min(least, ends[1][w]);
  }
  const int want = min(p.keep, there);
  uint32_t t = 1u;
  int have = there;
  if (want == forced) {
    t = kForcedPage;
    have = forced;
  } else if (want < there) {
    KeySearch search(least + 1u, top, there, forced, want);
    while (search.open()) {
      const uint32_t c = search.probe();
      int cnt = 0;
      each([&](uint32_t x) { cnt += x >= c ? 1 : 0; });
      search.count(c, total(cnt));
    }
    t = search.t;
    have = search.have;
  }
  // all of those above t, and the first of those equal to it
  const bool all = have == want;
  int above = 0, equal = 0;
  each([&](uint32_t x) {
    above += (all ? x >= t : x > t) ? 1 : 0;
    equal += (!all && x == t) ? 1 : 0;
  });
  const int before = block_prefix<CT>(above, slots[2]);
  int taken = 0, ties = 0;
  if (!all) {
    const int equal_before = block_prefix<CT>(equal, slots[3]);
    ties = want - total(above);
    taken = min(equal_before, ties);
  }
  int pos = before + taken;
#pragma unroll
  for (int i = 0; i < (KP > 0 ? KP : per); ++i) {
    const uint32_t x = key(i);
    bool take = all ? x >= t : x > t;
    if (!all && x == t && taken < ties) {
      take = true;
      ++taken;
    }
    if (take) out[pos++] = (int)(base + i);
  }
  for (int i = want + threadIdx.x; i < p.keep; i += CT) out[i] = -1;
}

// As many of the CTA's threads as the list needs, 4 warps for up to 2048 pages.
template <int THREADS>
__device__ __forceinline__ void choose_pages(const PagesParams& p, const uint32_t* keys, int n,
                                             int* out) {
  if (n <= 16 * 128) {
    if (threadIdx.x >= 128) return;
    if (n <= 4 * 128)
      choose_pages<4, 128>(p, keys, n, out);
    else
      choose_pages<16, 128>(p, keys, n, out);
  } else if constexpr (THREADS == kPageThreads) {  // (kFewPageThreads: no longer lists)
    if (n <= 16 * kPageThreads)
      choose_pages<16, kPageThreads>(p, keys, n, out);
    else
      choose_pages<0, kPageThreads>(p, keys, n, out);
  }
}

// The split form: scores of kRoundPages pages a CTA, then one CTA a head.
template <int D>
__global__ void __launch_bounds__(kPageThreads) page_scores_kernel(const PagesParams p) {
  extern __shared__ __align__(16) uint16_t whole[];
  wait_for_previous_launch();
  allow_next_launch();
  const int h = blockIdx.y, b = blockIdx.z;
  const int n = pages_of(p, b), first = blockIdx.x * kRoundPages;
  if (first >= n) return;
  const int64_t bh = (int64_t)b * p.c.Hkv + h;
  score_pages<D, kPageThreads>(p, b, h, n, first, min(n, first + kRoundPages), whole,
                               p.keys + bh * p.columns,
                               [&] { round_queries<D, kPageThreads>(p, bh, whole); });
}

__global__ void __launch_bounds__(kPageThreads) choose_pages_kernel(const PagesParams p) {
  wait_for_previous_launch();
  allow_next_launch();
  const int64_t bh = blockIdx.x;
  choose_pages<kPageThreads>(p, p.keys + bh * p.columns, pages_of(p, (int)(bh / p.c.Hkv)),
                             p.out + bh * p.keep);
}

// Both in one: a head a CTA, the keys in shared memory.
template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS) select_pages_kernel(const PagesParams p) {
  extern __shared__ __align__(16) uint16_t whole[];
  wait_for_previous_launch();
  allow_next_launch();
  const int64_t bh = blockIdx.x;
  const int b = (int)(bh / p.c.Hkv), h = (int)(bh - (int64_t)b * p.c.Hkv);
  const int n = pages_of(p, b);
  uint32_t* keys = reinterpret_cast<uint32_t*>(whole + (p.rows + 7) / 8 * 8 * D);
  score_pages<D, THREADS>(p, b, h, n, 0, n, whole, keys,
                          [&] { round_queries<D, THREADS>(p, bh, whole); });
  __syncthreads();
  choose_pages<THREADS>(p, keys, n, p.out + bh * p.keep);
}

bool one_cta_a_head(int heads, int columns, int sms) {
  return columns <= kOneCtaPages || (heads >= sms && columns <= kMostShared);
}

template <int D>
cudaError_t launch_pages(const PagesParams& p, int B, int sms, cudaStream_t st) {
  const size_t queries = (size_t)(p.rows + 7) / 8 * 8 * D * 2;
  const int heads = B * p.c.Hkv;
  if (one_cta_a_head(heads, p.columns, sms)) {
    const size_t smem = queries + (size_t)p.columns * sizeof(uint32_t);
    if (heads > sms && p.columns <= kOneCtaPages && p.rows * D <= kFewPageThreads * kVec * 8)
      return launch_dependent(select_pages_kernel<D, kFewPageThreads>, dim3(heads),
                              dim3(kFewPageThreads), smem, st, p);
    constexpr auto kernel = select_pages_kernel<D, kPageThreads>;
    cudaError_t e = allow_shared_memory<kernel>(64 << 10);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(heads), dim3(kPageThreads), smem, st, p);
  }
  cudaError_t e = launch_dependent(
      page_scores_kernel<D>, dim3((p.columns + kRoundPages - 1) / kRoundPages, p.c.Hkv, B),
      dim3(kPageThreads), queries, st, p);
  if (e != cudaSuccess) return e;
  return launch_dependent(choose_pages_kernel, dim3(heads), dim3(kPageThreads), 0, st, p);
}

bool strides_ok(const int64_t (&s)[6]) {
  for (int64_t x : s)
    if (x < 0 || x % 8 != 0) return false;
  return true;
}

bool ints_ok(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Dispatch over head_dim and group: f<D, lanes a group>.
#define BSATTN_KV4_DISPATCH(c, CALL)                                \
  do {                                                              \
    if ((c)->head_dim == 64) {                                      \
      if ((c)->group == 32) { CALL(64, 2); } else { CALL(64, 4); }  \
    } else {                                                        \
      if ((c)->group == 32) { CALL(128, 2); }                       \
      else if ((c)->group == 64) { CALL(128, 4); }                  \
      else { CALL(128, 8); }                                        \
    }                                                               \
  } while (0)

}  // namespace

bsattn_status check_cache(const bsattn_kv4_cache* c, Kv4View* view) {
  if (!c || !c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales || !c->k_means || !c->status)
    return BSATTN_ERR_INVALID_ARG;
  if (!aligned16(c->k_codes) || !aligned16(c->v_codes) || !aligned16(c->k_scales) ||
      !aligned16(c->v_scales) || !aligned16(c->k_means) || !ints_ok(c->status))
    return BSATTN_ERR_INVALID_ARG;
  if (c->pages <= 0 || c->kv_heads <= 0) return BSATTN_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return BSATTN_ERR_UNSUPPORTED;
  if (c->group != 32 && c->group != 64 && c->group != 128) return BSATTN_ERR_UNSUPPORTED;
  if (c->group > c->head_dim) return BSATTN_ERR_INVALID_ARG;
  const int ps = c->page_size;
  if (ps < 16 || ps > 256 || (ps & (ps - 1)) != 0) return BSATTN_ERR_UNSUPPORTED;
  if (c->kv_heads > 32767) return BSATTN_ERR_UNSUPPORTED;
  view->k_codes = static_cast<uint8_t*>(c->k_codes);
  view->v_codes = static_cast<uint8_t*>(c->v_codes);
  view->k_scales = static_cast<uint16_t*>(c->k_scales);
  view->v_scales = static_cast<uint16_t*>(c->v_scales);
  view->k_means = static_cast<uint16_t*>(c->k_means);
  view->status = c->status;
  view->pages = c->pages;
  view->Hkv = c->kv_heads;
  view->page = ps;
  view->log_page = __builtin_ctz((unsigned)ps);
  return BSATTN_OK;
}

}  // namespace bsattn

using namespace bsattn;

extern "C" {

bsattn_status bsattn_kv4_append(const bsattn_kv4_cache* cache, const void* k, int64_t k_batch,
                                int64_t k_head, int64_t k_token, const void* v, int64_t v_batch,
                                int64_t v_head, int64_t v_token, int B, int T,
                                const int32_t* block_table, int64_t table_stride, int columns,
                                const int32_t* lengths, const int32_t* counts, void* stream) {
  AppendParams p{};
  const bsattn_status rc = check_cache(cache, &p.c);
  if (rc != BSATTN_OK) return rc;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return BSATTN_ERR_INVALID_ARG;
  if (!ints_ok(block_table) || !ints_ok(lengths) || (counts && !ints_ok(counts)))
    return BSATTN_ERR_INVALID_ARG;
  if (B <= 0 || T <= 0 || columns <= 0 || table_stride < 0) return BSATTN_ERR_INVALID_ARG;
  if (B > 65535 || T > (1 << 30)) return BSATTN_ERR_UNSUPPORTED;
  if (!strides_ok({k_batch, k_head, k_token, v_batch, v_head, v_token}))
    return BSATTN_ERR_INVALID_ARG;
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.kb = k_batch;
  p.kh = k_head;
  p.kt = k_token;
  p.vb = v_batch;
  p.vh = v_head;
  p.vt = v_token;
  p.table = block_table;
  p.table_stride = table_stride;
  p.columns = columns;
  p.lengths = lengths;
  p.counts = counts;
  p.T = T;
  // T tokens touch at most this many pages
  const int touched = (T + cache->page_size - 2) / cache->page_size + 1;
  const bool few = T <= kFewTokens && cache->kv_heads <= 2048;  // (one page fills at most)
  const int rows = kRowThreads / (cache->head_dim / 16), all = few ? 2 * T * cache->kv_heads : 0;
  const dim3 grid(few ? 1 : touched,
                  cache->kv_heads + (few ? (all + rows - 1) / rows : cache->kv_heads), B);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
#define BSATTN_CALL(D, GL)                                                                  \
  e = few ? launch_dependent(kv4_append_kernel<D, GL, true>, grid, dim3(kRowThreads), 0, st, p) \
          : launch_dependent(kv4_append_kernel<D, GL, false>, grid, dim3(kRowThreads), 0, st, p)
  cudaError_t e;
  BSATTN_KV4_DISPATCH(cache, BSATTN_CALL);
#undef BSATTN_CALL
  return from_cuda(e);
}

bsattn_status bsattn_kv4_read(const bsattn_kv4_cache* cache, int B, int T,
                              const int32_t* block_table, int64_t table_stride, int columns,
                              const int32_t* start, const int32_t* counts, void* k, void* v,
                              void* stream) {
  ReadParams p{};
  const bsattn_status rc = check_cache(cache, &p.c);
  if (rc != BSATTN_OK) return rc;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return BSATTN_ERR_INVALID_ARG;
  if (!ints_ok(block_table) || !ints_ok(start) || (counts && !ints_ok(counts)))
    return BSATTN_ERR_INVALID_ARG;
  if (B <= 0 || T <= 0 || columns <= 0 || table_stride < 0) return BSATTN_ERR_INVALID_ARG;
  if (B > 65535 || T > (1 << 30)) return BSATTN_ERR_UNSUPPORTED;
  p.table = block_table;
  p.table_stride = table_stride;
  p.columns = columns;
  p.start = start;
  p.counts = counts;
  p.T = T;
  p.k = static_cast<uint16_t*>(k);
  p.v = static_cast<uint16_t*>(v);
  p.wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31u) == 0;
  const int per_cta = kRowThreads / (cache->head_dim / 16) * kReadRows;
  const dim3 grid((T + per_cta - 1) / per_cta, cache->kv_heads, B);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
#define BSATTN_CALL(D, GL) \
  e = launch_dependent(kv4_read_kernel<D, GL>, grid, dim3(kRowThreads), 0, st, p)
  cudaError_t e;
  BSATTN_KV4_DISPATCH(cache, BSATTN_CALL);
#undef BSATTN_CALL
  return from_cuda(e);
}

size_t bsattn_kv4_select_workspace(int B, int kv_heads, int columns) {
  if (B <= 0 || kv_heads <= 0 || columns <= 0) return 0;
  const int64_t heads = (int64_t)B * kv_heads;
  int dev = -1, sms = 1 << 30;
  if (columns <= kMostShared && cudaGetDevice(&dev) == cudaSuccess) sms = device_sm_count(dev);
  if (heads < (1ll << 31) && one_cta_a_head((int)heads, columns, sms)) return 0;
  return (size_t)heads * columns * sizeof(uint32_t);
}

bsattn_status bsattn_kv4_select(const bsattn_kv4_cache* cache, const void* q, int B, int H, int T,
                                const int32_t* block_table, int64_t table_stride, int columns,
                                const int32_t* lengths, int keep, int sink, int recent,
                                int32_t* selected, void* workspace, size_t workspace_bytes,
                                void* stream) {
  PagesParams p{};
  const bsattn_status rc = check_cache(cache, &p.c);
  if (rc != BSATTN_OK) return rc;
  if (!q || !aligned16(q) || !ints_ok(block_table) || !ints_ok(lengths) || !ints_ok(selected))
    return BSATTN_ERR_INVALID_ARG;
  if (B <= 0 || H <= 0 || T <= 0 || columns <= 0 || table_stride < 0 || H % cache->kv_heads != 0)
    return BSATTN_ERR_INVALID_ARG;
  if (sink < 0 || recent < 1 || (int64_t)sink + recent > keep) return BSATTN_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)(H / cache->kv_heads) * T;
  if (rows > kMostRows || B > 65535 || (int64_t)B * cache->kv_heads >= (1ll << 31))
    return BSATTN_ERR_UNSUPPORTED;
  const size_t need = bsattn_kv4_select_workspace(B, cache->kv_heads, columns);
  if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need))
    return BSATTN_ERR_INVALID_ARG;
  p.q = static_cast<const uint16_t*>(q);
  p.table = block_table;
  p.table_stride = table_stride;
  p.columns = columns;
  p.lengths = lengths;
  p.rows = (int)rows;
  p.keep = keep;
  p.sink = sink;
  p.recent = recent;
  p.keys = static_cast<uint32_t*>(workspace);
  p.out = selected;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSATTN_ERR_CUDA;
  const int sms = device_sm_count(dev);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return from_cuda(cache->head_dim == 64 ? launch_pages<64>(p, B, sms, st)
                                         : launch_pages<128>(p, B, sms, st));
}

bsattn_status bsattn_kv4_status(const bsattn_kv4_cache* cache, void* stream) {
  Kv4View view{};
  const bsattn_status rc = check_cache(cache, &view);
  if (rc != BSATTN_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int word = 0;
  if (cudaMemcpyAsync(&word, view.status, sizeof(word), cudaMemcpyDeviceToHost, st) !=
          cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return BSATTN_ERR_CUDA;
  if (!(word & kStatusPage)) return BSATTN_OK;
  // (cleared only after a report was seen: one that another stream makes in between is
  // in this answer, and none is lost)
  if (cudaMemsetAsync(view.status, 0, sizeof(word), st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return BSATTN_ERR_CUDA;
  return BSATTN_ERR_PAGE;
}

}  // extern "C"
