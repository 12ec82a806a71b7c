// From a model's projection to the attention's inputs, and back: RMS norm of
// every query and key head, rotation by position, and the head-major layout
// that the forward pass takes, in one pass over the data.
//
// Forward, per (token, head) row x of D channels, channel pairs (i, j):
//   n = x / sqrt(mean(x^2) + eps) * w
//   y_i = n_i cos - n_j sin,  y_j = n_j cos + n_i sin   (angles of the token's position)
// Backward, from g = (rotation transposed) dy:
//   dw = sum over rows of g x r,  r = 1 / sqrt(mean(x^2) + eps)
//   u = g w,  dx = r (u - x r^2 mean(u x))
// V rows are copied.
//
// Both read each input once and write each output once and do some 10 (25)
// operations an element: memory bound, if few enough instructions go into an
// element.  A row is held by D / 8 lanes, 16 bytes each, so the norm's sum and
// the exchange between the two halves of a rotated row are shuffles inside the
// lane group.  A warp takes rows of one token and one kind (Q, K or V): weights
// and angles are multiplied once for all its rows,
//   y = r (x (w cos) + x_partner (w_partner sin)),
// and all its rows' loads are in flight at once.  A CTA's eight warps take
// eight consecutive tokens of the same heads, 2 KB and more of every head-major
// row run.  The arithmetic is on register pairs (two floats an instruction).
//
// Measured, of a plain copy's rate: forward, 2 x 16384 tokens, 32 + 2 x 8 heads of
// 128: 138 us, 5.9 TB/s, 88%; backward, 4 x 4096 tokens, 16 + 2 x 16 heads of 128:
// 127 us, 6.3 TB/s, 95%.  64 tokens of a decoding step: 6 us, the launch and
// three loads in a row (position, angles, x beside them).
#include <cmath>
#include <cstdint>

#include "internal.h"
#include "ops.cuh"

namespace bsattn {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
// The backward kernel: warps a CTA, CTAs an SM and rows a lane.  Many rows a
// warp share one token's angles and read long runs of x, and four CTAs keep
// enough in flight.  At 4 x 4096 tokens, 16 + 2 x 16 heads of 128: 4, 4, 4 take
// 131 us; 2 rows a lane in 5 CTAs 151, in 6 (spilling) 188; 4 rows in 3 CTAs 147.
constexpr int kBwdWarps = 4;
constexpr int kBwdPerSm = 4;
constexpr int kBwdRows = 4;
// The forward kernel's rows a lane: 8 take 138 us at 2 x 16384 tokens, 32 + 2 x 8
// heads of 128, 4 take 140, the first kernel (all kinds of heads a warp) 197.
constexpr int kFwdRows = 8;

struct RopeParams {
  const uint16_t* x;  // [B][S][heads][D], strides xb and xs (elements)
  int64_t xb, xs;
  int tokens, S, H, Hkv;
  int q_chunks, k_chunks;  // warps' worth of heads of Q, and of K (and of V)
  const void* wq;          // [D] bf16 or fp32, null: no norm
  const void* wk;
  int w_f32;
  const float2* table;  // [n_pos][half] (cos, sin), null: no rotation
  int n_pos, half;
  const int* pos;  // [tokens], null: position s
  float eps;
  // forward: outputs; backward: upstream gradients (fp32) and dx
  void* q;
  void* k;
  void* v;
  uint16_t* dx;
  int64_t dxb, dxs;
  float* partial;  // backward: [(q_chunks + k_chunks) * groups][D] weight gradients
  int groups;      // backward: CTAs a chunk
};

// The heads of one chunk: kind 0, 1, 2 = Q, K, V; heads [first, end) of the
// kind; `row` is the first one's place in a token of x.
struct Chunk {
  int kind, first, end, row;
};
__device__ __forceinline__ Chunk chunk_of(const RopeParams& p, int chunk, int rows) {
  Chunk c;
  c.kind = chunk < p.q_chunks ? 0 : chunk < p.q_chunks + p.k_chunks ? 1 : 2;
  const int at = chunk - (c.kind == 0 ? 0 : c.kind == 1 ? p.q_chunks : p.q_chunks + p.k_chunks);
  const int heads = c.kind == 0 ? p.H : p.Hkv;
  c.first = at * rows;
  c.end = min(heads, c.first + rows);
  c.row = c.first + (c.kind == 0 ? 0 : c.kind == 1 ? p.H : p.H + p.Hkv);
  return c;
}

__device__ __forceinline__ void load_weights(const void* w, int f32, int c0, float (&out)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = 1.0f;
  } else if (f32) {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c0);
    const float4 a = load(f), b = load(f + 1);
    out[0] = a.x, out[1] = a.y, out[2] = a.z, out[3] = a.w;
    out[4] = b.x, out[5] = b.y, out[6] = b.z, out[7] = b.w;
  } else {
    unpack8(load(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + c0)), out);
  }
}

// cos and sin of this lane's 8 channels, the sine with the sign it has in
// y = n cos + n_partner sin.  Channels behind the rotated ones: cos 1, sin 0.
// A position outside the table: NaN.
template <bool INTER>
__device__ __forceinline__ void load_angles(const RopeParams& p, int token, int s, int c0,
                                            float (&cs)[8], float (&sn)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = 1.0f, sn[i] = 0.0f;
  if (c0 >= 2 * p.half) return;
  const int pos = p.pos ? load(p.pos + token) : s;
  if (pos < 0 || pos >= p.n_pos) {
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = sn[i] = __int_as_float(0x7FC00000);
    return;
  }
  const int first = INTER ? c0 / 2 : (c0 < p.half ? c0 : c0 - p.half);
  const float4* t = reinterpret_cast<const float4*>(p.table + (size_t)pos * p.half + first);
  const float sign = c0 < p.half ? -1.0f : 1.0f;
#pragma unroll
  for (int i = 0; i < (INTER ? 2 : 4); ++i) {
    const float4 f = load(t + i);
    if (INTER) {  // two pairs of channels
      cs[4 * i] = cs[4 * i + 1] = f.x;
      cs[4 * i + 2] = cs[4 * i + 3] = f.z;
      sn[4 * i] = -f.y, sn[4 * i + 1] = f.y;
      sn[4 * i + 2] = -f.w, sn[4 * i + 3] = f.w;
    } else {
      cs[2 * i] = f.x, sn[2 * i] = sign * f.y;
      cs[2 * i + 1] = f.z, sn[2 * i + 1] = sign * f.w;
    }
  }
}

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// The channel offset (0, or +-half a rotated row) of the partner's channels
// when pairs lie half a row apart; the partner lane is that / 8 away.
__device__ __forceinline__ int partner_offset(const RopeParams& p, int c0) {
  if (c0 >= 2 * p.half) return 0;
  return c0 < p.half ? p.half : -p.half;
}

// One warp: up to U * (32 / L) heads of one kind of one token.
template <int D, bool INTER, int U>
__global__ void __launch_bounds__(kRopeThreads) rope_fwd_kernel(const RopeParams p) {
  constexpr int L = D / 8;   // lanes a row
  constexpr int R = 32 / L;  // rows a warp holds at once
  wait_for_previous_launch();
  allow_next_launch();
  const int lane = threadIdx.x & 31;
  const unsigned chunks = p.q_chunks + 2 * p.k_chunks;
  const unsigned block = blockIdx.x / chunks;
  const Chunk c = chunk_of(p, blockIdx.x - block * chunks, U * R);
  const unsigned token = block * kRopeWarps + (threadIdx.x >> 5);
  if (token >= (unsigned)p.tokens) return;
  const int b = token / (unsigned)p.S, s = token - b * p.S;
  const int c0 = (lane % L) * 8, h0 = c.first + lane / L;

  const uint16_t* xr = p.x + b * p.xb + s * p.xs + (c.row + lane / L) * D + c0;
  uint4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    raw[u] = make_uint4(0, 0, 0, 0);
    if (h0 + u * R < c.end) raw[u] = load(reinterpret_cast<const uint4*>(xr + u * R * D));
  }
  const int heads = c.kind == 0 ? p.H : p.Hkv;
  uint16_t* out = static_cast<uint16_t*>(c.kind == 0 ? p.q : c.kind == 1 ? p.k : p.v) +
                  (((int64_t)b * heads + h0) * p.S + s) * D + c0;
  const int64_t next = (int64_t)R * p.S * D;
  const bool norm = p.wq != nullptr;
  if (c.kind == 2 || (!norm && p.half == 0)) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h0 + u * R < c.end) *reinterpret_cast<uint4*>(out + u * next) = raw[u];
    return;
  }
  F2 wc[4], ws[4];  // w cos, w_partner sin
  const int off = INTER ? 0 : partner_offset(p, c0);
  {
    float cs[8], sn[8], w[8];
    load_angles<INTER>(p, token, s, c0, cs, sn);
    const void* weight = c.kind == 0 ? p.wq : p.wk;
    load_weights(weight, p.w_f32, c0, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) wc[i] = f2(w[2 * i] * cs[2 * i], w[2 * i + 1] * cs[2 * i + 1]);
    if (!INTER) load_weights(weight, p.w_f32, c0 + off, w);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      ws[i] = INTER ? f2(w[2 * i + 1] * sn[2 * i], w[2 * i] * sn[2 * i + 1])
                    : f2(w[2 * i] * sn[2 * i], w[2 * i + 1] * sn[2 * i + 1]);
  }
  const int partner = lane + off / 8;
  const uint32_t turns = c0 < 2 * p.half ? 0xFFFFFFFFu : 0u;  // an infinity stays one elsewhere
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
    F2 x[4], ss = f2(0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = bf16_pair(w[i]);
      ss = fma2(x[i], x[i], ss);
    }
    F2 r = f2(1.0f);
    if (norm) {
      const float2 t = split(ss);
      r = f2(rsqrtf(group_sum<L>(t.x + t.y) * (1.0f / D) + p.eps));
    }
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t o = INTER ? __byte_perm(w[i], w[i], 0x1032)
                               : __shfl_sync(0xFFFFFFFFu, w[i], partner);
      y[i] = pack_bf16(fma2(bf16_pair(o & turns), ws[i], x[i] * wc[i]) * r);
    }
    if (h0 + u * R < c.end)
      *reinterpret_cast<uint4*>(out + u * next) = make_uint4(y[0], y[1], y[2], y[3]);
  }
}

// The gradient.  A CTA keeps to one chunk of heads and walks over tokens, so
// the weights and one weight gradient stay in registers: 32-bit sums of the
// rows a lane sees, added up over the CTA in a fixed order and written as one
// partial row a CTA, which rope_weight_kernel adds up.  No atomics: results
// repeat bit for bit.
template <int D, bool INTER, int U>
__global__ void __launch_bounds__(32 * kBwdWarps, kBwdPerSm) rope_bwd_kernel(const RopeParams p) {
  constexpr int L = D / 8;
  constexpr int R = 32 / L;
  __shared__ float red[kBwdWarps][D];
  wait_for_previous_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk = blockIdx.x / p.groups, group = blockIdx.x - chunk * p.groups;
  const Chunk c = chunk_of(p, chunk, U * R);
  const int c0 = (lane % L) * 8, h0 = c.first + lane / L;
  const int heads = c.kind == 0 ? p.H : p.Hkv;
  const float* up = static_cast<const float*>(c.kind == 0 ? p.q : c.kind == 1 ? p.k : p.v);
  const int64_t next = (int64_t)R * p.S * D;
  const int off = INTER ? 0 : partner_offset(p, c0);
  const int partner = lane + off / 8;
  const bool norm = p.wq != nullptr && c.kind != 2, turned = p.half != 0 && c.kind != 2;
  const bool turns = c0 < 2 * p.half;
  F2 w[4], acc[4];
  {
    float f[8];
    load_weights(c.kind == 0 ? p.wq : c.kind == 1 ? p.wk : nullptr, p.w_f32, c0, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f2(f[2 * i], f[2 * i + 1]), acc[i] = f2(0.0f);
  }
  for (unsigned token = group * kBwdWarps + warp; token < (unsigned)p.tokens;
       token += p.groups * kBwdWarps) {
    const int b = token / (unsigned)p.S, s = token - b * p.S;
    const int64_t row = (c.row + lane / L) * D + c0;
    const uint16_t* xr = p.x + b * p.xb + s * p.xs + row;
    const float* d = up + (((int64_t)b * heads + h0) * p.S + s) * D + c0;
    uint4 raw[U];
    float4 dy[U][2];
    constexpr uint32_t kOnes = 0x3F803F80u;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // behind the last head: dy = 0 and x = 1, so that r is finite with eps = 0 too and
      // the row adds 0 to the weights' gradient
      raw[u] = make_uint4(kOnes, kOnes, kOnes, kOnes);
      dy[u][0] = dy[u][1] = make_float4(0, 0, 0, 0);
      if (h0 + u * R < c.end) {
        dy[u][0] = load(reinterpret_cast<const float4*>(d + u * next));
        dy[u][1] = load(reinterpret_cast<const float4*>(d + u * next) + 1);
        if (norm) raw[u] = load(reinterpret_cast<const uint4*>(xr + u * R * D));
      }
    }
    float cs[8], sn[8];
    if (turned) load_angles<INTER>(p, token, s, c0, cs, sn);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float4 d0 = dy[u][0], d1 = dy[u][1];
      F2 g[4] = {f2(d0.x, d0.y), f2(d0.z, d0.w), f2(d1.x, d1.y), f2(d1.z, d1.w)};
      if (turned) {
        // turned back: the sine changes its sign
        const float e[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o[i] = INTER ? e[i ^ 1] : __shfl_sync(0xFFFFFFFFu, e[i], partner);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 t = f2(o[2 * i] * -sn[2 * i], o[2 * i + 1] * -sn[2 * i + 1]);
          if (turns) g[i] = fma2(g[i], f2(cs[2 * i], cs[2 * i + 1]), t);
        }
      }
      if (norm) {
        const uint32_t v[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
        F2 x[4], t[4], ss = f2(0.0f), dot = f2(0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = bf16_pair(v[i]);
          ss = fma2(x[i], x[i], ss);
          t[i] = g[i] * x[i];
          dot = fma2(t[i], w[i], dot);
        }
        const float2 a = split(ss), m = split(dot);
        F2 sums = f2(a.x + a.y, m.x + m.y);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) {
          const float2 t2 = split(sums);
          sums = sums + f2(__shfl_xor_sync(0xFFFFFFFFu, t2.x, o),
                           __shfl_xor_sync(0xFFFFFFFFu, t2.y, o));
        }
        const float2 total = split(sums);
        const float r = rsqrtf(total.x * (1.0f / D) + p.eps);
        const F2 r2 = f2(r), m2 = f2(-total.y * (1.0f / D) * r * r * r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[i] = fma2(t[i], r2, acc[i]);
          g[i] = fma2(x[i], m2, g[i] * w[i] * r2);
        }
      }
      if (h0 + u * R < c.end)
        *reinterpret_cast<uint4*>(p.dx + b * p.dxb + s * p.dxs + row + u * R * D) =
            make_uint4(pack_bf16(g[0]), pack_bf16(g[1]), pack_bf16(g[2]), pack_bf16(g[3]));
    }
  }
  allow_next_launch();
  if (!norm) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = split(acc[i]);
    float t[2] = {a.x, a.y};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int o = L; o < 32; o <<= 1) t[e] += __shfl_xor_sync(0xFFFFFFFFu, t[e], o);
      if (lane < L) red[warp][c0 + 2 * i + e] = t[e];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += 32 * kBwdWarps) {
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < kBwdWarps; ++k) t += red[k][i];
    p.partial[(size_t)blockIdx.x * D + i] = t;
  }
}

// Adds up the CTAs' partial weight gradients in a fixed order: 32 channels of
// one weight a CTA, 32 rows at a time, a few hundred rows.  The sums carry their
// errors along (hi + lo): as good as 64 bits, which this machine adds at 1/64 of
// the rate.
__global__ void __launch_bounds__(1024)
    rope_weight_kernel(const float* __restrict__ partial, int q_rows, int k_rows, int D,
                       float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ Sum2 sh[32][33];
  wait_for_previous_launch();
  const int col = blockIdx.x * 32 + threadIdx.x;
  const bool is_q = blockIdx.y == 0;
  const float* from = partial + (is_q ? 0 : (size_t)q_rows * D) + col;
  const int rows = is_q ? q_rows : k_rows;
  Sum2 t{0.0f, 0.0f};
  int r = threadIdx.y;
  for (; r + 7 * 32 < rows; r += 8 * 32) {  // (eight loads at once)
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __ldcg(from + (size_t)(r + i * 32) * D);
#pragma unroll
    for (int i = 0; i < 8; ++i) add_exact(t, v[i]);
  }
  for (; r < rows; r += 32) add_exact(t, __ldcg(from + (size_t)r * D));
  sh[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  t = sh[threadIdx.x][threadIdx.y];  // warp y: channel y's 32 sums
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sum2 other;
    other.hi = __shfl_xor_sync(0xFFFFFFFFu, t.hi, o);
    other.lo = __shfl_xor_sync(0xFFFFFFFFu, t.lo, o);
    add_exact(t, other);
  }
  // (an infinite sum has no rest)
  if (threadIdx.x == 0)
    (is_q ? dwq : dwk)[blockIdx.x * 32 + threadIdx.y] = isfinite(t.lo) ? t.hi + t.lo : t.hi;
}

__global__ void rope_table_kernel(const double* __restrict__ inv_freq, int n_pos, int half,
                                  float2* __restrict__ table) {
  const int64_t n = (int64_t)n_pos * half;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int pos = (int)(i / half), f = (int)(i - (int64_t)pos * half);
    double s, c;
    sincos((double)pos * inv_freq[f], &s, &c);  // 64 bits: far positions lose the angle in 32
    table[i] = make_float2((float)c, (float)s);
  }
}

bool multiple8(int64_t v) { return v % 8 == 0; }

// Rows a lane holds at once: as many as the larger kind of heads fills, at most `most`.
int rows_per_lane(int H, int D, int most) {
  const int at_once = 256 / D;
  int u = 1;
  while (u < most && u * at_once < H) u *= 2;
  return u;
}

// The backward pass's split: CTAs a chunk, so that kBwdPerSm CTAs run on each SM
// and none is without tokens.  (As many for a chunk of few heads as for a full one:
// a token costs a warp its latency.  3 x 1021 tokens, 16 + 2 x 4 heads of 64: 15 us,
// with CTAs by the number of heads 19.)
struct BwdSplit {
  int u, q_chunks, k_chunks, groups;
};
BwdSplit bwd_split(int tokens, int H, int Hkv, int D, int sms) {
  BwdSplit s;
  s.u = rows_per_lane(H, D, kBwdRows);
  const int rows = s.u * 256 / D;
  s.q_chunks = (H + rows - 1) / rows;
  s.k_chunks = (Hkv + rows - 1) / rows;
  const int chunks = s.q_chunks + 2 * s.k_chunks;
  const int most = tokens / kBwdWarps + (tokens % kBwdWarps != 0);
  s.groups = kBwdPerSm * sms / chunks;  // one wave: a CTA more would run alone at the end
  if (s.groups > most) s.groups = most;
  if (s.groups < 1) s.groups = 1;
  return s;
}

// The argument checks that both directions share.
bsattn_status check_rope(const void* x, int64_t xb, int64_t xs, int B, int S, int H, int Hkv, int D,
                         const void* wq, const void* wk, unsigned flags, const float* table,
                         int n_pos, int rotary_dim, const int32_t* pos, float eps) {
  if (!x || !aligned16(x)) return BSATTN_ERR_INVALID_ARG;
  if (B <= 0 || S <= 0 || H <= 0 || Hkv <= 0 || H % Hkv != 0) return BSATTN_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return BSATTN_ERR_UNSUPPORTED;
  const int64_t heads = (int64_t)H + 2 * (int64_t)Hkv;
  if (heads > (1 << 20) || (int64_t)B * S >= (1ll << 31) || (int64_t)B * S * heads >= (1ll << 31))
    return BSATTN_ERR_UNSUPPORTED;
  if (xb < 0 || xs < 0 || !multiple8(xb) || !multiple8(xs)) return BSATTN_ERR_INVALID_ARG;
  if ((wq == nullptr) != (wk == nullptr)) return BSATTN_ERR_INVALID_ARG;
  if (wq && (!aligned16(wq) || !aligned16(wk))) return BSATTN_ERR_INVALID_ARG;
  if (flags & ~(unsigned)(BSATTN_ROPE_INTERLEAVED | BSATTN_WEIGHT_F32)) return BSATTN_ERR_INVALID_ARG;
  if (table) {
    if (!aligned16(table) || n_pos <= 0 || rotary_dim <= 0 || rotary_dim > D)
      return BSATTN_ERR_INVALID_ARG;
    if (rotary_dim % 16 != 0) return BSATTN_ERR_UNSUPPORTED;
    if (!pos && S > n_pos) return BSATTN_ERR_INVALID_ARG;
  }
  if (pos && (reinterpret_cast<uintptr_t>(pos) & 3u)) return BSATTN_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return BSATTN_ERR_INVALID_ARG;
  return BSATTN_OK;
}

// Whether B x S rows of `row` elements at x and at dx share memory, other than each
// row with its own: dx may be x itself.
bool rows_overlap(const void* x, int64_t xb, int64_t xs, const void* dx, int64_t dxb, int64_t dxs,
                  int B, int S, int64_t row) {
  if (B == 1) xb = dxb = 0;
  if (S == 1) xs = dxs = 0;
  const int64_t apart =
      static_cast<int64_t>(reinterpret_cast<intptr_t>(dx) - reinterpret_cast<intptr_t>(x)) / 2;
  const bool same = xb == dxb && xs == dxs;
  if (apart == 0 && same) return false;
  const int64_t x_end = (B - 1) * xb + (S - 1) * xs + row;
  const int64_t dx_end = apart + (B - 1) * dxb + (S - 1) * dxs + row;
  if (apart >= x_end || dx_end <= 0) return false;
  if (!same) return true;
  // the same strides, one between the other's rows: the distance of a row of dx to the
  // nearest row of x in each other batch entry
  for (int64_t b = 1 - B; b < B; ++b) {
    const int64_t from = apart + b * xb;
    const int64_t near = xs ? -from / xs : 0;
    for (int64_t t = near - 1; t <= near + 1; ++t) {
      const int64_t off = from + t * xs;
      if (t > -S && t < S && off > -row && off < row) return true;
    }
  }
  return false;
}

RopeParams rope_params(const void* x, int64_t xb, int64_t xs, int B, int S, int H, int Hkv,
                       const void* wq, const void* wk, unsigned flags, const float* table,
                       int n_pos, int rotary_dim, const int32_t* pos, float eps) {
  RopeParams p{};
  p.x = static_cast<const uint16_t*>(x);
  p.xb = xb;
  p.xs = xs;
  p.tokens = B * S;
  p.S = S;
  p.H = H;
  p.Hkv = Hkv;
  p.wq = wq;
  p.wk = wk;
  p.w_f32 = (flags & BSATTN_WEIGHT_F32) ? 1 : 0;
  p.table = reinterpret_cast<const float2*>(table);
  p.n_pos = n_pos;
  p.half = table ? rotary_dim / 2 : 0;
  p.pos = pos;
  p.eps = eps;
  return p;
}

template <int D, bool INTER>
cudaError_t launch_rope_fwd(RopeParams& p, cudaStream_t st) {
  const int u = rows_per_lane(p.H, D, kFwdRows), rows = u * 256 / D;
  p.q_chunks = (p.H + rows - 1) / rows;
  p.k_chunks = (p.Hkv + rows - 1) / rows;
  // at most B * S * heads CTAs: below 2^31
  const int blocks = p.tokens / kRopeWarps + (p.tokens % kRopeWarps != 0);
  const int grid = blocks * (p.q_chunks + 2 * p.k_chunks);
  return launch_dependent(u == 1   ? rope_fwd_kernel<D, INTER, 1>
                          : u == 2 ? rope_fwd_kernel<D, INTER, 2>
                          : u == 4 ? rope_fwd_kernel<D, INTER, 4>
                                   : rope_fwd_kernel<D, INTER, 8>,
                          dim3(grid), dim3(kRopeThreads), 0, st, (const RopeParams&)p);
}

template <int D, bool INTER>
cudaError_t launch_rope_bwd(const RopeParams& p, int u, cudaStream_t st) {
  const int grid = (p.q_chunks + 2 * p.k_chunks) * p.groups;
  return launch_dependent(u == 1   ? rope_bwd_kernel<D, INTER, 1>
                          : u == 2 ? rope_bwd_kernel<D, INTER, 2>
                                   : rope_bwd_kernel<D, INTER, 4>,
                          dim3(grid), dim3(32 * kBwdWarps), 0, st, p);
}

}  // namespace
}  // namespace bsattn

using namespace bsattn;

extern "C" {

bsattn_status bsattn_rope_table(const double* inv_freq, int n_pos, int rotary_dim, float* table,
                                void* stream) {
  if (!inv_freq || !table || !aligned16(inv_freq) || !aligned16(table)) return BSATTN_ERR_INVALID_ARG;
  if (n_pos <= 0 || rotary_dim <= 0) return BSATTN_ERR_INVALID_ARG;
  if (rotary_dim % 16 != 0 || rotary_dim > 128) return BSATTN_ERR_UNSUPPORTED;
  const int64_t n = (int64_t)n_pos * (rotary_dim / 2);
  const int64_t blocks = (n + 255) / 256;
  rope_table_kernel<<<(int)(blocks < 65536 ? blocks : 65536), 256, 0,
                      static_cast<cudaStream_t>(stream)>>>(inv_freq, n_pos, rotary_dim / 2,
                                                           reinterpret_cast<float2*>(table));
  return from_cuda(cudaGetLastError());
}

bsattn_status bsattn_qk_norm_rope(const void* x, int64_t x_batch_stride, int64_t x_token_stride,
                                  int B, int S, int H, int Hkv, int D, const void* q_weight,
                                  const void* k_weight, const float* table, int n_pos,
                                  int rotary_dim, const int32_t* positions, float eps,
                                  unsigned flags, void* q, void* k, void* v, void* stream) {
  const bsattn_status rc = check_rope(x, x_batch_stride, x_token_stride, B, S, H, Hkv, D, q_weight,
                                      k_weight, flags, table, n_pos, rotary_dim, positions, eps);
  if (rc != BSATTN_OK) return rc;
  if (!q || !k || !v || !aligned16(q) || !aligned16(k) || !aligned16(v))
    return BSATTN_ERR_INVALID_ARG;
  RopeParams p = rope_params(x, x_batch_stride, x_token_stride, B, S, H, Hkv, q_weight, k_weight,
                             flags, table, n_pos, rotary_dim, positions, eps);
  p.q = q;
  p.k = k;
  p.v = v;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool inter = (flags & BSATTN_ROPE_INTERLEAVED) != 0;
  if (D == 64)
    return from_cuda(inter ? launch_rope_fwd<64, true>(p, st) : launch_rope_fwd<64, false>(p, st));
  return from_cuda(inter ? launch_rope_fwd<128, true>(p, st) : launch_rope_fwd<128, false>(p, st));
}

size_t bsattn_qk_norm_rope_bwd_workspace(int B, int S, int H, int Hkv, int D) {
  if (B <= 0 || S <= 0 || H <= 0 || Hkv <= 0 || (D != 64 && D != 128)) return 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if ((int64_t)B * S >= (1ll << 31)) return 0;
  const BwdSplit s = bwd_split(B * S, H, Hkv, D, device_sm_count(dev));
  return (size_t)(s.q_chunks + s.k_chunks) * s.groups * D * sizeof(float);
}

bsattn_status bsattn_qk_norm_rope_bwd(const void* x, int64_t x_batch_stride, int64_t x_token_stride,
                                      const float* dq, const float* dk, const float* dv, int B,
                                      int S, int H, int Hkv, int D, const void* q_weight,
                                      const void* k_weight, const float* table, int n_pos,
                                      int rotary_dim, const int32_t* positions, float eps,
                                      unsigned flags, void* dx, int64_t dx_batch_stride,
                                      int64_t dx_token_stride, float* dq_weight, float* dk_weight,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  const bsattn_status rc = check_rope(x, x_batch_stride, x_token_stride, B, S, H, Hkv, D, q_weight,
                                      k_weight, flags, table, n_pos, rotary_dim, positions, eps);
  if (rc != BSATTN_OK) return rc;
  if (!dq || !dk || !dv || !dx || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) ||
      !aligned16(dx))
    return BSATTN_ERR_INVALID_ARG;
  const int64_t row = (int64_t)(H + 2 * Hkv) * D;  // rows of dx must not overlap
  if (!multiple8(dx_batch_stride) || !multiple8(dx_token_stride) || dx_token_stride < row ||
      dx_batch_stride < 0 || (B > 1 && dx_batch_stride < (S - 1) * dx_token_stride + row))
    return BSATTN_ERR_INVALID_ARG;
  // (x is read with weights only)
  if (q_weight && rows_overlap(x, x_batch_stride, x_token_stride, dx, dx_batch_stride,
                               dx_token_stride, B, S, row))
    return BSATTN_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSATTN_ERR_CUDA;
  const BwdSplit split = bwd_split(B * S, H, Hkv, D, device_sm_count(dev));
  RopeParams p = rope_params(x, x_batch_stride, x_token_stride, B, S, H, Hkv, q_weight, k_weight,
                             flags, table, n_pos, rotary_dim, positions, eps);
  p.q_chunks = split.q_chunks;
  p.k_chunks = split.k_chunks;
  p.groups = split.groups;
  if (q_weight) {
    if (!dq_weight || !dk_weight || !workspace || !aligned16(workspace) ||
        workspace_bytes < bsattn_qk_norm_rope_bwd_workspace(B, S, H, Hkv, D))
      return BSATTN_ERR_INVALID_ARG;
    p.partial = static_cast<float*>(workspace);
  }
  // the forward's output slots hold the upstream gradients here (read only)
  p.q = const_cast<float*>(dq);
  p.k = const_cast<float*>(dk);
  p.v = const_cast<float*>(dv);
  p.dx = static_cast<uint16_t*>(dx);
  p.dxb = dx_batch_stride;
  p.dxs = dx_token_stride;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool inter = (flags & BSATTN_ROPE_INTERLEAVED) != 0;
  cudaError_t e =
      D == 64 ? (inter ? launch_rope_bwd<64, true>(p, split.u, st)
                       : launch_rope_bwd<64, false>(p, split.u, st))
              : (inter ? launch_rope_bwd<128, true>(p, split.u, st)
                       : launch_rope_bwd<128, false>(p, split.u, st));
  if (e != cudaSuccess || !q_weight) return from_cuda(e);
  e = launch_dependent(rope_weight_kernel, dim3(D / 32, 2), dim3(32, 32), 0, st,
                       (const float*)p.partial, split.q_chunks * split.groups,
                       split.k_chunks * split.groups, D, dq_weight, dk_weight);
  return from_cuda(e);
}

}  // extern "C"
