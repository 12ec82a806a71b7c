// What the kernels of the 4-bit cache share (kv4.cu, kv4_attn.cu).
#pragma once

#include <cstdint>

#include "internal.h"
#include "ops.cuh"

namespace bsattn {

// Bit of a cache's status word (BSATTN_ERR_PAGE)
enum : int { kStatusPage = 8 };

// The cache in device memory, D / group = groups scale pairs a row:
//   codes   [pages][Hkv][page][D / 2]       two codes a byte, the even channel low
//   scales  [pages][Hkv][page][groups][2]   bf16 (step, minimum): value = step * code + minimum
//   k_means [pages][Hkv][D]                 bf16, the rounded mean key of a full page
struct Kv4View {
  uint8_t* k_codes;
  uint8_t* v_codes;
  uint16_t* k_scales;
  uint16_t* v_scales;
  uint16_t* k_means;
  int* status;
  int pages, Hkv, page, log_page;

  // index of the row of (page, head, place in the page)
  __device__ __forceinline__ int64_t row(int pg, int h, int place) const {
    return ((int64_t)pg * Hkv + h) * page + place;
  }
  __device__ __forceinline__ void report() const { atomicOr(status, kStatusPage); }
};

// The table's entry for one of a sequence's pages; -1, and the status word
// set, where the table has no such column or names a page that is not there.
__device__ __forceinline__ int page_at(const Kv4View& c, const int* table, int columns,
                                       int64_t logical) {
  int pg = -1;
  if (logical >= 0 && logical < columns) pg = load(table + logical);
  if (pg < 0 || pg >= c.pages) {
    c.report();
    pg = -1;
  }
  return pg;
}

// Host side: the checks of a cache that every call makes.
bsattn_status check_cache(const bsattn_kv4_cache* c, Kv4View* view);

// kv4_attn_scored.cu: bsattn_kv4_attn_chunk's arguments, checked, for few rows.
struct FewRows {
  const bsattn_kv4_cache* cache;
  const void* q;
  int B, H, T;
  const int32_t* block_table;
  int64_t table_stride;
  int columns;
  const int32_t* lengths;
  const int32_t* counts;
  const int32_t* prefix;
  float scale, cap;
  const float* slopes;
  int out_f32;
  void* out;
  float* lse;
};
size_t kv4_few_rows_workspace(int B, int kv_heads, int rows, int D, int64_t tokens);
bsattn_status kv4_few_rows(const FewRows& f, void* workspace, size_t workspace_bytes,
                           cudaStream_t stream);

// tanh(y) / y by y^2 for |y| <= 0.8, off by 6.7e-8 relative: least maximal relative
// error, by Lawson's iteration.
constexpr float kTanh0 = 0.99999994f, kTanh1 = -0.333326757f, kTanh2 = 0.13321048f,
                kTanh3 = -0.0531143136f, kTanh4 = 0.0190932993f, kTanh5 = -0.00435529929f;
constexpr float kTanhRange = 0.8f;
// The same for |y| <= 0.3, off by 2.2e-8.
constexpr float kNear0 = 1.0f, kNear1 = -0.333329618f, kNear2 = 0.133125976f, kNear3 = -0.0502224378f;
constexpr float kNearRange = 0.3f;

// tanh(y): (1 - e) / (1 + e), e = exp(-2 |y|); off by 2^-22 of one or less.
__device__ __forceinline__ float tanh_any(float y) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-2.8853900817779268f * fabsf(y)));
  return copysignf(__fdividef(1.0f - e, 1.0f + e), y);
}

}  // namespace bsattn
