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
// operations an element: memory bound.  A row is held by D / 8 lanes, 16
// bytes each, so the norm's sum and the exchange between the two halves of a
// rotated row are shuffles inside the lane group; a warp takes rows of one
// token, so the token's angles are loaded once for all its rows, and has all
// its rows' loads in flight at once.
#include <cmath>
#include <cstdint>

#include "internal.h"
#include "ops.cuh"

namespace bsattn {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;

struct RopeParams {
  const uint16_t* x;  // [B][S][heads][D], strides xb and xs (elements)
  int64_t xb, xs;
  int S, H, Hkv, heads;  // heads = H + 2 Hkv
  int chunks;            // tasks a token: chunks of heads
  int tasks;             // tokens * chunks
  const void* wq;        // [D] bf16 or fp32, null: no norm
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
  float* partial;  // backward: [CTAs][2][D] weight gradients
};

template <int D>
__device__ __forceinline__ void load_weights(const void* w, int f32, int c0, float (&out)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = 1.0f;
  } else if (f32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = __ldg(static_cast<const float*>(w) + c0 + i);
  } else {
    unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + c0)), out);
  }
}

// cos and sin of this lane's 8 channels.  Pairs side by side: 4 pairs, the
// first four entries.  Pairs half a row apart: one entry a channel, the sine
// negative in the first half, so that y = n cos + n_partner sin in both.
// Channels behind the rotated ones: cos 1, sin 0.  A position outside the
// table: NaN.
template <bool INTER>
__device__ __forceinline__ void load_angles(const RopeParams& p, int token, int s, int c0,
                                            float (&cs)[8], float (&sn)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = 1.0f, sn[i] = 0.0f;
  if (p.table == nullptr || c0 >= 2 * p.half) return;
  const int pos = p.pos ? __ldg(p.pos + token) : s;
  if (pos < 0 || pos >= p.n_pos) {
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = sn[i] = __int_as_float(0x7FC00000);
    return;
  }
  const int first = INTER ? c0 / 2 : (c0 < p.half ? c0 : c0 - p.half);
  const float4* t =
      reinterpret_cast<const float4*>(p.table + (size_t)pos * p.half + first);
  const float sign = (!INTER && c0 < p.half) ? -1.0f : 1.0f;
#pragma unroll
  for (int i = 0; i < (INTER ? 2 : 4); ++i) {
    const float4 f = __ldg(t + i);
    cs[2 * i] = f.x, sn[2 * i] = sign * f.y;
    cs[2 * i + 1] = f.z, sn[2 * i + 1] = sign * f.w;
  }
}

// Rotate this lane's 8 values (dir = 1), or turn them back (dir = -1).
// `partner`: the lane that holds the other half (this lane: nothing to swap).
template <bool INTER>
__device__ __forceinline__ void rotate(float (&y)[8], const float (&cs)[8], const float (&sn)[8],
                                       float dir, int partner) {
  if (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = y[2 * i], b = y[2 * i + 1], s = dir * sn[i];
      y[2 * i] = a * cs[i] - b * s;
      y[2 * i + 1] = b * cs[i] + a * s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_sync(0xFFFFFFFFu, y[i], partner);
      y[i] = y[i] * cs[i] + o * (dir * sn[i]);
    }
  }
}

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

__device__ __forceinline__ int rotation_partner(const RopeParams& p, int lane, int c0, bool inter) {
  if (inter || p.table == nullptr || c0 >= 2 * p.half) return lane;
  return c0 < p.half ? lane + p.half / 8 : lane - p.half / 8;
}

// One warp: U * (32 / L) consecutive heads of one token.
template <int D, bool INTER, int U>
__global__ void __launch_bounds__(kRopeThreads) rope_fwd_kernel(const RopeParams p) {
  constexpr int L = D / 8;    // lanes a row
  constexpr int R = 32 / L;   // rows a warp holds at once
  const int lane = threadIdx.x & 31;
  const unsigned task = blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
  if (task >= (unsigned)p.tasks) return;
  const int token = task / (unsigned)p.chunks;
  const int h0 = (int)(task - (unsigned)token * p.chunks) * (U * R) + lane / L;
  const int b = token / p.S, s = token - b * p.S;
  const int c0 = (lane % L) * 8;

  const uint16_t* xr = p.x + b * p.xb + s * p.xs + c0;
  uint4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * R;
    raw[u] = make_uint4(0, 0, 0, 0);
    if (h < p.heads) raw[u] = __ldg(reinterpret_cast<const uint4*>(xr + h * D));
  }
  float cs[8], sn[8], wq[8], wk[8];
  load_angles<INTER>(p, token, s, c0, cs, sn);
  load_weights<D>(p.wq, p.w_f32, c0, wq);
  load_weights<D>(p.wk, p.w_f32, c0, wk);
  const int partner = rotation_partner(p, lane, c0, INTER);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * R;
    float y[8];
    unpack8(raw[u], y);
    if (p.wq != nullptr) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += y[i] * y[i];
      const float r = rsqrtf(group_sum<L>(ss) * (1.0f / D) + p.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= r * (h < p.H ? wq[i] : wk[i]);
    }
    rotate<INTER>(y, cs, sn, 1.0f, partner);
    if (h < p.H) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.q) +
                                (((int64_t)b * p.H + h) * p.S + s) * D + c0) = pack8(y);
    } else if (h < p.H + p.Hkv) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.k) +
                                (((int64_t)b * p.Hkv + h - p.H) * p.S + s) * D + c0) = pack8(y);
    } else if (h < p.heads) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.v) +
                                (((int64_t)b * p.Hkv + h - p.H - p.Hkv) * p.S + s) * D + c0) =
          raw[u];
    }
  }
}

// The gradient: the same split, each warp walking over tasks; the two weight
// gradients stay in registers (32-bit sums of the rows a lane sees), are
// added up over the CTA in a fixed order and written as one partial row a
// CTA, which rope_weight_kernel adds up: no atomics, so results repeat.
template <int D, bool INTER, int U>
__global__ void __launch_bounds__(kRopeThreads) rope_bwd_kernel(const RopeParams p) {
  constexpr int L = D / 8;
  constexpr int R = 32 / L;
  __shared__ float red[kRopeWarps][2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = (lane % L) * 8;
  const int partner = rotation_partner(p, lane, c0, INTER);
  float wq[8], wk[8], aq[8], ak[8];
  load_weights<D>(p.wq, p.w_f32, c0, wq);
  load_weights<D>(p.wk, p.w_f32, c0, wk);
#pragma unroll
  for (int i = 0; i < 8; ++i) aq[i] = ak[i] = 0.0f;

  for (unsigned task = blockIdx.x * kRopeWarps + warp; task < (unsigned)p.tasks;
       task += gridDim.x * kRopeWarps) {
    const int token = task / (unsigned)p.chunks;
    const int h0 = (int)(task - (unsigned)token * p.chunks) * (U * R) + lane / L;
    const int b = token / p.S, s = token - b * p.S;
    const uint16_t* xr = p.x + b * p.xb + s * p.xs + c0;
    uint4 raw[U];
    float4 dy[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * R;
      raw[u] = make_uint4(0, 0, 0, 0);
      dy[u][0] = dy[u][1] = make_float4(0, 0, 0, 0);
      const float* d = nullptr;
      if (h < p.H)
        d = static_cast<const float*>(p.q) + (((int64_t)b * p.H + h) * p.S + s) * D;
      else if (h < p.H + p.Hkv)
        d = static_cast<const float*>(p.k) + (((int64_t)b * p.Hkv + h - p.H) * p.S + s) * D;
      else if (h < p.heads)
        d = static_cast<const float*>(p.v) +
            (((int64_t)b * p.Hkv + h - p.H - p.Hkv) * p.S + s) * D;
      if (d != nullptr) {
        dy[u][0] = __ldg(reinterpret_cast<const float4*>(d + c0));
        dy[u][1] = __ldg(reinterpret_cast<const float4*>(d + c0) + 1);
      }
      if (h < p.H + p.Hkv && p.wq != nullptr)  // without a norm x is not needed
        raw[u] = __ldg(reinterpret_cast<const uint4*>(xr + h * D));
    }
    float cs[8], sn[8];
    load_angles<INTER>(p, token, s, c0, cs, sn);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * R;
      const float4 d0 = dy[u][0], d1 = dy[u][1];
      const float up[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
      float g[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = up[i];
      rotate<INTER>(g, cs, sn, -1.0f, partner);
      if (p.wq != nullptr) {
        float x[8], ss = 0.0f, dot = 0.0f;
        unpack8(raw[u], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss += x[i] * x[i];
          dot += g[i] * (h < p.H ? wq[i] : wk[i]) * x[i];
        }
        const float r = rsqrtf(group_sum<L>(ss) * (1.0f / D) + p.eps);
        const float m = group_sum<L>(dot) * (1.0f / D) * r * r;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float t = g[i] * x[i] * r;
          if (h < p.H)
            aq[i] += t;
          else if (h < p.H + p.Hkv)
            ak[i] += t;
          g[i] = r * (g[i] * (h < p.H ? wq[i] : wk[i]) - x[i] * m);
        }
      }
      if (h < p.heads) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = h < p.H + p.Hkv ? g[i] : up[i];
        *reinterpret_cast<uint4*>(p.dx + b * p.dxb + s * p.dxs + h * D + c0) = pack8(g);
      }
    }
  }
  if (p.partial == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int o = L; o < 32; o <<= 1) {
      aq[i] += __shfl_xor_sync(0xFFFFFFFFu, aq[i], o);
      ak[i] += __shfl_xor_sync(0xFFFFFFFFu, ak[i], o);
    }
    if (lane < L) {
      red[warp][0][c0 + i] = aq[i];
      red[warp][1][c0 + i] = ak[i];
    }
  }
  __syncthreads();
  allow_next_launch();
  for (int c = threadIdx.x; c < 2 * D; c += kRopeThreads) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kRopeWarps; ++w) t += red[w][c / D][c % D];
    p.partial[(size_t)blockIdx.x * 2 * D + c] = t;
  }
}

// Adds up the CTAs' partial weight gradients in a fixed order: 32 columns a
// CTA, 32 rows at a time.  (The sums of a few hundred rows, in 64 bits.)
__global__ void __launch_bounds__(1024)
    rope_weight_kernel(const float* __restrict__ partial, int rows, int D, float* __restrict__ dwq,
                       float* __restrict__ dwk) {
  __shared__ double sh[32][33];
  wait_for_previous_launch();
  const int col = blockIdx.x * 32 + threadIdx.x;
  double t = 0.0;
  for (int r = threadIdx.y; r < rows; r += 32) t += partial[(size_t)r * 2 * D + col];
  sh[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y == 0) {
    double s = 0.0;
    for (int r = 0; r < 32; ++r) s += sh[r][threadIdx.x];
    if (col < D)
      dwq[col] = (float)s;
    else
      dwk[col - D] = (float)s;
  }
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

// CTAs of the backward kernel, and rows of its workspace
int bwd_ctas(int tasks, int sms) {
  const int all = tasks / kRopeWarps + (tasks % kRopeWarps != 0);
  return all < 4 * sms ? all : 4 * sms;
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

RopeParams rope_params(const void* x, int64_t xb, int64_t xs, int B, int S, int H, int Hkv, int D,
                       const void* wq, const void* wk, unsigned flags, const float* table,
                       int n_pos, int rotary_dim, const int32_t* pos, float eps, int rows) {
  RopeParams p{};
  p.x = static_cast<const uint16_t*>(x);
  p.xb = xb;
  p.xs = xs;
  p.S = S;
  p.H = H;
  p.Hkv = Hkv;
  p.heads = H + 2 * Hkv;
  p.chunks = (p.heads + rows - 1) / rows;
  p.tasks = B * S * p.chunks;  // at most B * S * heads
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

// Rows a lane holds at once: as many as the heads fill, at most 4 (2 in the
// backward pass, whose rows take three times the registers).
int rows_per_lane(int heads, int D, int most) {
  const int at_once = 256 / D;
  int u = 1;
  while (u < most && u * at_once < heads) u *= 2;
  return u;
}

template <int D, bool INTER>
void launch_rope_fwd(const RopeParams& p, int u, cudaStream_t st) {
  const int grid = p.tasks / kRopeWarps + (p.tasks % kRopeWarps != 0);
  if (u == 1)
    rope_fwd_kernel<D, INTER, 1><<<grid, kRopeThreads, 0, st>>>(p);
  else if (u == 2)
    rope_fwd_kernel<D, INTER, 2><<<grid, kRopeThreads, 0, st>>>(p);
  else
    rope_fwd_kernel<D, INTER, 4><<<grid, kRopeThreads, 0, st>>>(p);
}

template <int D, bool INTER>
void launch_rope_bwd(const RopeParams& p, int u, int grid, cudaStream_t st) {
  if (u == 1)
    rope_bwd_kernel<D, INTER, 1><<<grid, kRopeThreads, 0, st>>>(p);
  else
    rope_bwd_kernel<D, INTER, 2><<<grid, kRopeThreads, 0, st>>>(p);
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
  const int u = rows_per_lane(H + 2 * Hkv, D, 4);
  RopeParams p = rope_params(x, x_batch_stride, x_token_stride, B, S, H, Hkv, D, q_weight, k_weight,
                             flags, table, n_pos, rotary_dim, positions, eps, u * 256 / D);
  p.q = q;
  p.k = k;
  p.v = v;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool inter = (flags & BSATTN_ROPE_INTERLEAVED) != 0;
  if (D == 64)
    inter ? launch_rope_fwd<64, true>(p, u, st) : launch_rope_fwd<64, false>(p, u, st);
  else
    inter ? launch_rope_fwd<128, true>(p, u, st) : launch_rope_fwd<128, false>(p, u, st);
  return from_cuda(cudaGetLastError());
}

size_t bsattn_qk_norm_rope_bwd_workspace(int B, int S, int H, int Hkv, int D) {
  if (B <= 0 || S <= 0 || H <= 0 || Hkv <= 0 || (D != 64 && D != 128)) return 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  return (size_t)4 * device_sm_count(dev) * 2 * D * sizeof(float);
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
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSATTN_ERR_CUDA;
  const int u = rows_per_lane(H + 2 * Hkv, D, 2);
  RopeParams p = rope_params(x, x_batch_stride, x_token_stride, B, S, H, Hkv, D, q_weight, k_weight,
                             flags, table, n_pos, rotary_dim, positions, eps, u * 256 / D);
  const int grid = bwd_ctas(p.tasks, device_sm_count(dev));
  if (q_weight) {
    if (!dq_weight || !dk_weight || !workspace || !aligned16(workspace) ||
        workspace_bytes < (size_t)grid * 2 * D * sizeof(float))
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
  if (D == 64)
    inter ? launch_rope_bwd<64, true>(p, u, grid, st) : launch_rope_bwd<64, false>(p, u, grid, st);
  else
    inter ? launch_rope_bwd<128, true>(p, u, grid, st) : launch_rope_bwd<128, false>(p, u, grid, st);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !q_weight) return from_cuda(e);
  e = launch_dependent(rope_weight_kernel, dim3(2 * D / 32), dim3(32, 32), 0, st,
                       (const float*)p.partial, grid, D, dq_weight, dk_weight);
  return from_cuda(e);
}

}  // extern "C"
