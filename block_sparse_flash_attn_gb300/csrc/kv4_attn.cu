// Attention of new tokens over the 4-bit cache.
//
// Query t of T of a sequence of length n sits at position n - T + t and sees
// the cached tokens up to its own position (all of them, or those of a list of
// pages).  With K and V rows decoded as step * code + minimum (kv4.cu):
//   s_i = scale q . k_i,  p = softmax(s),  o = sum_i p_i v_i,
//   lse = ln sum_i exp(s_i);  a query that sees nothing: o = 0, lse = -inf.
#include <cmath>
#include <cstdint>

#include "kv4.cuh"

namespace bsattn {
namespace {

constexpr int kAttnThreads = 256;
constexpr int kAttnWarps = kAttnThreads / 32;

struct AttnParams {
  Kv4View c;
  const uint16_t* q;  // [B][H][T][D]
  const int* table;
  int64_t table_stride;
  int columns;
  const int* lengths;
  const int* selected;  // [B][Hkv][n_selected] ascending pages, or null
  int n_selected;
  int T, rows;  // rows = G * T
  float scale_log2;
  void* out;
  float* lse;
  int out_f32;
};

// The page of list entry e of a (sequence, head), and the position of its
// first token; -1 for nothing.  Without a list entry e is page e.
__device__ __forceinline__ int listed_page(const AttnParams& p, int b, int h, int64_t e, int len,
                                           int64_t& first) {
  int64_t logical = e;
  if (p.selected) {
    const int* sel = p.selected + ((int64_t)b * p.c.Hkv + h) * p.n_selected;
    logical = __ldg(sel + e);
    if (logical < 0) return -1;
    if (e > 0 && logical <= __ldg(sel + e - 1)) {  // a page named twice, or out of order
      p.c.report();
      return -1;
    }
  }
  first = logical << p.c.log_page;
  if (first >= len) return -1;
  return page_at(p.c, p.table + b * p.table_stride, p.columns, logical);
}

// One CTA per (query row, head, sequence); each warp takes every eighth token
// of the list and keeps its own running maximum and sums, which are joined
// at the end.
template <int D, int GL>
__global__ void __launch_bounds__(kAttnThreads) kv4_attn_kernel(const AttnParams p) {
  constexpr int V = D / 32, NG = D / 8 / GL;  // channels a lane
  __shared__ float sm[kAttnWarps], sl[kAttnWarps], so[kAttnWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int len = max(p.lengths[b], 0);
  const int64_t last = (int64_t)len - p.T + r % p.T;
  const int64_t row = ((int64_t)b * p.c.Hkv + h) * p.rows + r;
  float q[V], o[V], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    q[i] = __uint_as_float((uint32_t)p.q[row * D + lane * V + i] << 16);
    o[i] = 0.0f;
  }
  const int64_t entries = p.selected ? p.n_selected : ((int64_t)len + p.c.page - 1) >> p.c.log_page;
  for (int64_t e = 0; e < entries; ++e) {
    int64_t first = 0;
    const int pg = listed_page(p, b, h, e, len, first);
    if (pg < 0) continue;
    for (int t = warp; t < p.c.page && first + t <= last; t += kAttnWarps) {
      const int64_t cr = p.c.row(pg, h, t);
      float dot = 0.0f, v[V];
      const int ch = lane * V;
      const uint32_t ks = reinterpret_cast<const uint32_t*>(p.c.k_scales)[cr * NG + ch / (8 * GL)];
      const uint32_t vs = reinterpret_cast<const uint32_t*>(p.c.v_scales)[cr * NG + ch / (8 * GL)];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int sh = 4 * (i & 1);
        const int kc = (p.c.k_codes[cr * (D / 2) + (ch + i) / 2] >> sh) & 15;
        const int vc = (p.c.v_codes[cr * (D / 2) + (ch + i) / 2] >> sh) & 15;
        dot += q[i] * fmaf(bf16_lo(ks), (float)kc, bf16_hi(ks));
        v[i] = fmaf(bf16_lo(vs), (float)vc, bf16_hi(vs));
      }
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, s);
      const float x = dot * p.scale_log2;
      const float nm = fmaxf(m, x);
      const float a = exp2f(m - nm), w = exp2f(x - nm);
      m = nm;
      l = l * a + w;
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = o[i] * a + w * v[i];
    }
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int i = 0; i < V; ++i) so[warp][lane * V + i] = o[i];
  __syncthreads();
  float top = -INFINITY, sum = 0.0f;
  for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, sm[w]);
  const float ref = top == -INFINITY ? 0.0f : top;
  for (int w = 0; w < kAttnWarps; ++w) sum += sl[w] * exp2f(sm[w] - ref);
  if (threadIdx.x == 0) p.lse[row] = (ref + log2f(sum)) * kLn2;
  for (int c = threadIdx.x; c < D; c += kAttnThreads) {
    float t = 0.0f;
    for (int w = 0; w < kAttnWarps; ++w) t += so[w][c] * exp2f(sm[w] - ref);
    t = sum > 0.0f ? t / sum : (sum == 0.0f ? 0.0f : sum);
    if (p.out_f32)
      static_cast<float*>(p.out)[row * D + c] = t;
    else
      static_cast<__nv_bfloat16*>(p.out)[row * D + c] = __float2bfloat16_rn(t);
  }
}

}  // namespace
}  // namespace bsattn

using namespace bsattn;

extern "C" {

size_t bsattn_kv4_attn_workspace(int B, int H, int kv_heads, int T, int D) {
  if (B <= 0 || H <= 0 || kv_heads <= 0 || T <= 0 || H % kv_heads != 0 || (D != 64 && D != 128))
    return 0;
  return 16;
}

bsattn_status bsattn_kv4_attn(const bsattn_kv4_cache* cache, const void* q, int B, int H, int T,
                              const int32_t* block_table, int64_t table_stride, int columns,
                              const int32_t* lengths, const int32_t* selected, int n_selected,
                              float scale, unsigned flags, void* out, float* lse, void* workspace,
                              size_t workspace_bytes, void* stream) {
  AttnParams p{};
  const bsattn_status rc = check_cache(cache, &p.c);
  if (rc != BSATTN_OK) return rc;
  if (!q || !out || !lse || !workspace || !aligned16(q) || !aligned16(out) || !aligned16(lse) ||
      !aligned16(workspace))
    return BSATTN_ERR_INVALID_ARG;
  if (!block_table || !lengths || ((reinterpret_cast<uintptr_t>(block_table) |
                                    reinterpret_cast<uintptr_t>(lengths) |
                                    reinterpret_cast<uintptr_t>(selected)) & 3u))
    return BSATTN_ERR_INVALID_ARG;
  if (B <= 0 || H <= 0 || T <= 0 || columns <= 0 || table_stride < 0 || H % cache->kv_heads != 0)
    return BSATTN_ERR_INVALID_ARG;
  if ((selected != nullptr) != (n_selected > 0) || n_selected < 0) return BSATTN_ERR_INVALID_ARG;
  if (flags & ~(unsigned)BSATTN_OUT_F32) return BSATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return BSATTN_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)(H / cache->kv_heads) * T;
  if (rows > 128 || B > 65535) return BSATTN_ERR_UNSUPPORTED;
  if (workspace_bytes < bsattn_kv4_attn_workspace(B, H, cache->kv_heads, T, cache->head_dim))
    return BSATTN_ERR_INVALID_ARG;
  p.q = static_cast<const uint16_t*>(q);
  p.table = block_table;
  p.table_stride = table_stride;
  p.columns = columns;
  p.lengths = lengths;
  p.selected = selected;
  p.n_selected = n_selected;
  p.T = T;
  p.rows = (int)rows;
  p.scale_log2 = (float)((double)scale * 1.4426950408889634074);
  p.out = out;
  p.lse = lse;
  p.out_f32 = (flags & BSATTN_OUT_F32) ? 1 : 0;
  const dim3 grid((int)rows, cache->kv_heads, B);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cache->head_dim == 64) {
    if (cache->group == 32)
      kv4_attn_kernel<64, 4><<<grid, kAttnThreads, 0, st>>>(p);
    else
      kv4_attn_kernel<64, 8><<<grid, kAttnThreads, 0, st>>>(p);
  } else {
    if (cache->group == 32)
      kv4_attn_kernel<128, 4><<<grid, kAttnThreads, 0, st>>>(p);
    else if (cache->group == 64)
      kv4_attn_kernel<128, 8><<<grid, kAttnThreads, 0, st>>>(p);
    else
      kv4_attn_kernel<128, 16><<<grid, kAttnThreads, 0, st>>>(p);
  }
  return from_cuda(cudaGetLastError());
}

}  // extern "C"
