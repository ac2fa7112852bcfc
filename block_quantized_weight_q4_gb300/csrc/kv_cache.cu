// kv_cache.cu -- the paged cache of keys and values in 8 bits: rows written with one scale for each
// page and head, and read back.
#include "kv.cuh"

namespace qmv {

namespace {

constexpr int kWriteThreads = 128;

// One CTA per (page that receives rows, head, K or V).  The page's scale is the largest its tokens
// have needed: raised by the new rows, the earlier tokens' levels move to it.
template <bool XB>
__global__ void __launch_bounds__(kWriteThreads) kv_write_kernel(const __grid_constant__ KvRef c,
                                                                 const void* __restrict__ kx, long long k_stride,
                                                                 const void* __restrict__ vx, long long v_stride) {
  __shared__ float part[kWriteThreads / 32];
  const int s = blockIdx.y;
  const int head = blockIdx.z >> 1;
  const bool is_v = blockIdx.z & 1;
  const KvSeq q = kv_seq(c, s);
  const int first = q.len - q.n;
  const int pi = (first >> c.page_shift) + blockIdx.x;
  if (pi * c.page_tokens >= q.len || q.n == 0) return;
  const int id = kv_page(c, s, pi);
  if (id < 0) return;
  const int begin = pi * c.page_tokens;
  const int lo = first > begin ? first - begin : 0;
  const int hi = q.len - begin < c.page_tokens ? q.len - begin : c.page_tokens;
  const long long at = (long long)id * c.kv_heads + head;
  int8_t* lev = (is_v ? c.v : c.k) + at * c.page_tokens * c.head_dim;
  float* scale = (is_v ? c.v_scale : c.k_scale) + at;
  const void* x = is_v ? vx : kx;
  const long long stride = is_v ? v_stride : k_stride;
  const int ppr = c.head_dim / 8;  // pieces of a row
  const int pieces = (hi - lo) * ppr;
  const long long x0 = (q.row0 + (begin + lo - first)) * stride + (long long)head * c.head_dim;

  float amax = 0.f;
  for (int p = threadIdx.x; p < pieces; p += kWriteThreads) {
    float v[8];
    load8<XB>(x, x0 + (p / ppr) * stride + (p % ppr) * 8, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
  const float had = lo > 0 ? *scale : 0.f;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWriteThreads / 32; ++w) amax = fmaxf(amax, part[w]);
  const float want = amax < 1e-30f ? 0.f : __fmul_rn(amax, 1.0f / 127.0f);
  const float d = fmaxf(want, had);
  const float inv = d > 0.f ? __fdiv_rn(1.0f, d) : 0.f;

  for (int p = threadIdx.x; p < pieces; p += kWriteThreads) {
    float v[8];
    load8<XB>(x, x0 + (p / ppr) * stride + (p % ppr) * 8, v);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      int l = (int)__fadd_rn(__fmul_rn(v[e], inv), copysignf(0.5f, v[e]));
      l = l > 127 ? 127 : (l < -127 ? -127 : l);
      w[e >> 2] |= (uint32_t)(l & 0xFF) << (8 * (e & 3));
    }
    *reinterpret_cast<uint2*>(lev + (long long)lo * c.head_dim + 8 * p) = make_uint2(w[0], w[1]);
  }
  if (d > had && lo > 0) {
    const float ratio = __fdiv_rn(had, d);
    for (int p = threadIdx.x; p < lo * ppr; p += kWriteThreads) {
      uint2* g = reinterpret_cast<uint2*>(lev + 8 * p);
      const uint2 u = *g;
      const uint32_t in[2] = {u.x, u.y};
      uint32_t w[2] = {0u, 0u};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float f = (float)(int8_t)(in[e >> 2] >> (8 * (e & 3)));
        const int l = (int)__fadd_rn(__fmul_rn(f, ratio), copysignf(0.5f, f));
        w[e >> 2] |= (uint32_t)(l & 0xFF) << (8 * (e & 3));
      }
      *g = make_uint2(w[0], w[1]);
    }
  }
  if (threadIdx.x == 0) *scale = d;
}

constexpr int kReadRows = 32;  // rows of a sequence that one CTA reads back

// 16 levels a thread at a time.
template <bool XB>
__global__ void __launch_bounds__(256) kv_read_kernel(const __grid_constant__ KvRef c, void* __restrict__ ko,
                                                      void* __restrict__ vo) {
  const int s = blockIdx.y;
  const bool is_v = blockIdx.z;
  const KvSeq q = kv_seq(c, s);
  const int r0 = blockIdx.x * kReadRows;
  if (r0 >= q.n) return;
  const int nr = q.n - r0 < kReadRows ? q.n - r0 : kReadRows;
  const int8_t* lev = is_v ? c.v : c.k;
  const float* scale = is_v ? c.v_scale : c.k_scale;
  const int ppr = c.head_dim / 16;
  const int row_pieces = c.kv_heads * ppr;
  for (int p = threadIdx.x; p < nr * row_pieces; p += 256) {
    const int r = p / row_pieces, in_row = p % row_pieces;
    const int head = in_row / ppr, piece = in_row % ppr;
    const int pos = q.len - q.n + r0 + r;
    const int id = kv_page(c, s, (pos >> c.page_shift));
    if (id < 0) continue;
    const long long at = (long long)id * c.kv_heads + head;
    const float d = __ldg(scale + at);
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(
        lev + (at * c.page_tokens + (pos & (c.page_tokens - 1))) * c.head_dim + 16 * piece));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float f[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) f[e] = __fmul_rn((float)(int8_t)(w[e >> 2] >> (8 * (e & 3))), d);
    const long long o = (q.row0 + r0 + r) * c.kv_heads * c.head_dim + head * c.head_dim + 16 * piece;
    if (XB) {
      uint4* g = reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? vo : ko) + o);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        g[h] = make_uint4(pack_bf16x2(f[8 * h], f[8 * h + 1]), pack_bf16x2(f[8 * h + 2], f[8 * h + 3]),
                          pack_bf16x2(f[8 * h + 4], f[8 * h + 5]), pack_bf16x2(f[8 * h + 6], f[8 * h + 7]));
    } else {
      float4* g = reinterpret_cast<float4*>(static_cast<float*>(is_v ? vo : ko) + o);
#pragma unroll
      for (int h = 0; h < 4; ++h) g[h] = make_float4(f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]);
    }
  }
}

}  // namespace

cudaError_t launch_kv_write(const KvRef& c, bool x_bf16, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, cudaStream_t stream) {
  // pages that n rows can fall into, wherever they start in the first
  const int pages = (c.max_rows + c.page_tokens - 2) / c.page_tokens + 1;
  const dim3 grid((unsigned)pages, (unsigned)c.n_seq, (unsigned)(2 * c.kv_heads));
  auto kern = x_bf16 ? kv_write_kernel<true> : kv_write_kernel<false>;
  kern<<<grid, kWriteThreads, 0, stream>>>(c, k, k_stride, v, v_stride);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const KvRef& c, bool out_bf16, void* k, void* v, cudaStream_t stream) {
  const dim3 grid((unsigned)((c.max_rows + kReadRows - 1) / kReadRows), (unsigned)c.n_seq, 2u);
  auto kern = out_bf16 ? kv_read_kernel<true> : kv_read_kernel<false>;
  kern<<<grid, 256, 0, stream>>>(c, k, v);
  return cudaGetLastError();
}

}  // namespace qmv
