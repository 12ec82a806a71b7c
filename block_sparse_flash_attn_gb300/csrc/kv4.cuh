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

}  // namespace bsattn
