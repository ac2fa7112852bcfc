// kv.cuh -- what the kernels over the paged 8-bit cache share: a call's sequences and pages,
// read and checked on the device.
#pragma once

#include "qmv_common.cuh"
#include "qmv_internal.h"

namespace qmv {

// One sequence of a call: its cached tokens, its rows of the call and the first of them.
struct KvSeq {
  int len;
  int n;
  long long row0;
};

// Sequence s of the call; a sequence that contradicts the call's numbers gets no rows (n = 0, len = 0)
// and is recorded.
__device__ __forceinline__ KvSeq kv_seq(const KvRef& c, int s) {
  KvSeq q;
  q.len = __ldg(c.kv_len + s);
  if (c.starts != nullptr) {
    const int a = __ldg(c.starts + s), b = __ldg(c.starts + s + 1);
    q.row0 = a;
    q.n = b - a;
    if (a < 0 || b < a || b > c.rows) q.n = -1;
  } else {
    q.row0 = s;
    q.n = 1;
  }
  if (q.len < 0 || q.len > c.max_len || q.len > (long long)c.table_pages * c.page_tokens || q.n < 0 || q.n > c.max_rows ||
      q.n > q.len) {
    record_status(c.status, QMV_E_ARG);
    q.n = 0;
    q.len = 0;
    q.row0 = 0;
  }
  return q;
}

// The page that holds token i * page_tokens .. of sequence s, or -1 (recorded) where the table names
// none of the cache's.
__device__ __forceinline__ int kv_page(const KvRef& c, int s, int i) {
  const int id = __ldg(c.page_table + (long long)s * c.table_stride + i);
  if (id < 0 || id >= c.n_pages) {
    record_status(c.status, QMV_E_ARG);
    return -1;
  }
  return id;
}

// Eight consecutive values of a row.
template <bool XB>
__device__ __forceinline__ void load8(const void* x, long long at, float (&v)[8]) {
  if (XB) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  } else {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    const float4 a = __ldg(f), b = __ldg(f + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

}  // namespace qmv
