// paged.cuh -- the layout of paged caches: a page's rows of one head, and 4-bit rows.
#pragma once

#include "rows.cuh"

namespace la {

constexpr int kGroup = 64;  // elements that share a scale and an offset

// Bytes of a page's tokens of one head.
__host__ __device__ __forceinline__ int page_bytes(const PagedCache& c) {
  return c.page * (c.four ? c.d * 9 / 16 : c.d * (c.bf16 ? 2 : 4));
}

// Page of column `at` of a sequence's table, or -1 where it is none of the pool's.
__device__ __forceinline__ int table_page(const PagedCache& c, int64_t b, int64_t at) {
  const int p = c.table[b * c.width + at];
  return p >= 0 && p < (int)c.pages ? p : -1;
}

// A row's word (eight codes) of group g, e = 0..7 of its 64 elements: neighbouring words belong to different groups, so
// that a lane's 8 or 16 bytes hold words of every group.
__device__ __forceinline__ int code_word(int g, int e, int groups) { return e * groups + g; }

}  // namespace la
