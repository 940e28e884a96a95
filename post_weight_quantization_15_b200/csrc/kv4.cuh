// The cache of keys and values held in 4 bits, shared by the kernels that write it, read
// it back and attend over it.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace gptq {

// Page p, head h, row r (token r of the page), feature f:
//   code    codes[((p . heads + h) . page_size + r) . d / 8 + f / 8] >> 4 (f mod 8) & 15
//   scale   params[(((p . heads + h) . page_size + r) . d / group + f / group) . 2]
//   zero    the next one.
__device__ __forceinline__ int64_t kv4_row(const KV4Cache& C, int page, int head, int r) {
  return ((int64_t)page * C.heads + head) * C.page_size + r;
}

// The page of position pos of sequence b, or -1 (a position outside the table's row, or
// an entry that names no page).
__device__ __forceinline__ int kv4_page(const KV4Cache& C, const int32_t* table, int width, int b, int64_t pos) {
  if (pos < 0 || pos >= (int64_t)width * C.page_size) return -1;
  const int p = table[(int64_t)b * width + (int)(pos / C.page_size)];
  return p >= 0 && p < C.pages ? p : -1;
}

// The sequence b with cu[b] <= t < cu[b + 1], or -1.
__device__ __forceinline__ int packed_sequence(const int32_t* cu, int count, int t) {
  int lo = 0, hi = count;                 // the largest b in [0, count] with cu[b] <= t
  if (cu[0] > t) return -1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo < count ? lo : -1;
}

}  // namespace gptq
