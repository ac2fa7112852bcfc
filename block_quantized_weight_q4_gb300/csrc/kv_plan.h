// kv_plan.h -- the integer arithmetic of calls over the paged cache that the host and the kernels share.  Plain C++,
// so that it is tested where there is no GPU: every bound that the host accepts has to stay inside its type here.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define QMV_HD __host__ __device__ __forceinline__
#else
#define QMV_HD inline
#endif

namespace qmv {

constexpr int kKvMaxLen = INT32_MAX - 1024;  // the largest max_len: lengths rounded up to a tile of keys stay positive

// The stated bound of a sequence's rows, brought down to what the call's other numbers leave (the rows in all, a
// sequence's tokens), so that a loose bound costs no CTAs.  A bound above 0 stays above 0: a call whose
// numbers contradict each other is still looked at, and recorded, on the device.
QMV_HD int kv_rows_bound(int64_t rows, int max_rows, int max_len) {
  int64_t n = max_rows;
  if (n > rows) n = rows;
  if (n > max_len) n = max_len;
  return max_rows > 0 && n < 1 ? 1 : (int)n;
}

// Pages that n rows of a sequence can fall into, wherever they start in the first; n at most kKvMaxLen.
QMV_HD int kv_pages_bound(int n, int page_tokens) { return (n + page_tokens - 2) / page_tokens + 1; }

// The i-th page, in the page table's row, of those that the last n of len tokens fall into; -1 past the last.
// (The page's number times its tokens is formed only for pages that there are.)
QMV_HD int kv_written_page(int len, int n, int i, int page_shift) {
  if (n <= 0) return -1;
  const int at = (len - n) >> page_shift;
  return i > ((len - 1) >> page_shift) - at ? -1 : at + i;
}

// Chunks of a sequence's segments in all: n_chunks of keys for each of n_blocks row blocks of each head (past 32 bits from
// a few hundred thousand rows over as many tokens on).
QMV_HD long long kv_segment_chunks(int n_chunks, int n_blocks, int heads) { return (long long)n_chunks * n_blocks * heads; }

}  // namespace qmv
