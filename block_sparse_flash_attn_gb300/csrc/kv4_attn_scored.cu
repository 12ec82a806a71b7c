// Attention of a few new tokens over the 4-bit cache with counts, a prefix, capped and
// biased scores: the few-row form of kv4_chunk.cu, by the kernels of kv4_attn.cuh.
#define BSATTN_SCORED true
#include "kv4_attn.cuh"

namespace bsattn {

size_t kv4_few_rows_workspace(int B, int kv_heads, int rows, int D, int64_t tokens) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  return attn_split(B, kv_heads, rows, tokens, D, device_sm_count(dev)).workspace;
}

bsattn_status kv4_few_rows(const FewRows& f, void* workspace, size_t workspace_bytes,
                           cudaStream_t stream) {
  const bsattn_kv4_cache* cache = f.cache;
  AttnParams p{};
  const bsattn_status rc = check_cache(cache, &p.c);
  if (rc != BSATTN_OK) return rc;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSATTN_ERR_CUDA;
  const int rows = f.H / cache->kv_heads * f.T;
  const AttnSplit split =
      attn_split(f.B, cache->kv_heads, rows, attn_tokens(cache->page_size, f.columns, 0),
                 cache->head_dim, device_sm_count(dev));
  if (split.steps * f.B >= (1ll << 31) || (int64_t)f.B * cache->kv_heads * split.mt >= (1ll << 31))
    return BSATTN_ERR_UNSUPPORTED;
  if (split.workspace > 0 && (!workspace || workspace_bytes < split.workspace))
    return BSATTN_ERR_INVALID_ARG;
  p.q = static_cast<const uint16_t*>(f.q);
  p.table = f.block_table;
  p.table_stride = f.table_stride;
  p.columns = f.columns;
  p.lengths = f.lengths;
  p.B = f.B;
  p.T = f.T;
  p.rows = rows;
  p.scale_log2 = (float)((double)f.scale * 1.4426950408889634074);
  p.out = f.out;
  p.lse = f.lse;
  p.out_f32 = f.out_f32;
  p.counts = f.counts;
  p.open = f.prefix;
  p.slopes = f.slopes;
  p.cap_log2 = (float)((double)f.cap * 1.4426950408889634074);
  return from_cuda(launch_split<true>(p, split, cache, workspace, stream));
}

}  // namespace bsattn
