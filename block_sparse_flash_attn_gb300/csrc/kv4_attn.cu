// Attention of new tokens over the 4-bit cache: the entry point (kernels: kv4_attn.cuh).
#define BSATTN_SCORED false
#include "kv4_attn.cuh"

using namespace bsattn;

extern "C" {

size_t bsattn_kv4_attn_workspace(int B, int H, int kv_heads, int T, int D, int page_size,
                                 int columns, int n_selected) {
  const int64_t tokens = attn_tokens(page_size, columns, n_selected);
  if (B <= 0 || H <= 0 || kv_heads <= 0 || T <= 0 || H % kv_heads != 0 || tokens == 0) return 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  return attn_split(B, kv_heads, (int64_t)(H / kv_heads) * T, tokens, D, device_sm_count(dev))
      .workspace;
}

bsattn_status bsattn_kv4_attn(const bsattn_kv4_cache* cache, const void* q, int B, int H, int T,
                              const int32_t* block_table, int64_t table_stride, int columns,
                              const int32_t* lengths, const int32_t* selected, int n_selected,
                              float scale, unsigned flags, void* out, float* lse, void* workspace,
                              size_t workspace_bytes, void* stream) {
  AttnParams p{};
  const bsattn_status rc = check_cache(cache, &p.c);
  if (rc != BSATTN_OK) return rc;
  if (!q || !out || !lse || !aligned16(q) || !aligned16(out) || !aligned16(lse) ||
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
  if (rows > 128 || B > kMostSequences ||
      (int64_t)columns * cache->page_size > (1ll << 31) - kStep ||  // positions are 32-bit
      (int64_t)cache->pages * cache->kv_heads * cache->page_size / kTile >= (1ll << 31))
    return BSATTN_ERR_UNSUPPORTED;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSATTN_ERR_CUDA;
  const AttnSplit split =
      attn_split(B, cache->kv_heads, rows, attn_tokens(cache->page_size, columns, n_selected),
                 cache->head_dim, device_sm_count(dev));
  if (split.steps * B >= (1ll << 31) || (int64_t)B * cache->kv_heads * split.mt >= (1ll << 31))
    return BSATTN_ERR_UNSUPPORTED;
  if (split.workspace > 0 && (!workspace || workspace_bytes < split.workspace))
    return BSATTN_ERR_INVALID_ARG;
  p.q = static_cast<const uint16_t*>(q);
  p.table = block_table;
  p.table_stride = table_stride;
  p.columns = columns;
  p.lengths = lengths;
  p.selected = selected;
  p.n_selected = n_selected;
  p.B = B;
  p.T = T;
  p.rows = (int)rows;
  p.scale_log2 = (float)((double)scale * 1.4426950408889634074);
  p.out = out;
  p.lse = lse;
  p.out_f32 = (flags & BSATTN_OUT_F32) ? 1 : 0;
  return from_cuda(launch_split<false>(p, split, cache, workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
