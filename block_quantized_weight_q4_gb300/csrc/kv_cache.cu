// kv_cache.cu -- the paged cache of keys and values in 8 bits: rows written with one scale for each
// page and head, and read back.
//
// Writing is bound by the rows' bytes, and below that by the instructions that a value's level takes (about 7; a third
// fewer than with conversions, clamps and packs one by one, which took 23.2 us where these took 18.7) and a chain of
// dependent loads a page (lengths, page id and rows, the old scale) around one reduction: 16384 bfloat16 rows of 8 heads
// of 128 in 19.2 us (5.2 TB/s, 77% of the measured copy rate; issue 74% busy, ALU 61%; float32 28.2 us, 5.9 TB/s), one row
// of each of 64 sequences in 2.3 us, 6.5 us where every other one raises a page of 40 earlier tokens, whose levels are then
// read, moved and written.  A page, head and side (K or V) is a CTA because its scale is what its rows share.  Reading is a
// copy that widens: 16 sequences of up to 16384 tokens as bfloat16 in 191 us (6.57 TB/s, 97%), 16 of 8000 as float32 in
// 196 us (6.69 TB/s; 273 us while a thread stored 64 bytes in a row, so that a warp's store touched 32 lines).
#include <type_traits>

#include "kv.cuh"

namespace qmv {

namespace {

// One CTA per (page that receives rows, head, K or V).  The page's scale is the largest its tokens
// have needed: raised by the new rows, the earlier tokens' levels move to it.  The new rows stay in
// registers between the maximum and their levels (P pieces of 8 values a thread), so each is read once.
template <int D, bool XB, int P>
__global__ void __launch_bounds__(512) kv_write_kernel(const __grid_constant__ KvRef c, const void* __restrict__ kx,
                                                       long long k_stride, const void* __restrict__ vx,
                                                       long long v_stride) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int kRow = D / 8;  // pieces of a row
  __shared__ float part[16];
  const int s = blockIdx.y;
  const int head = blockIdx.z >> 1;
  const bool is_v = blockIdx.z & 1;
  const int T = blockDim.x;
  const KvSeq q = kv_seq(c, s);
  const int first = q.len - q.n;
  const int pi = kv_written_page(q.len, q.n, (int)blockIdx.x, c.page_shift);
  if (pi < 0) return;
  const int begin = pi << c.page_shift;
  // the rows are asked for before the page's id is looked at
  const int id = __ldg(c.page_table + (long long)s * c.table_stride + pi);
  const int lo = first > begin ? first - begin : 0;
  const int hi = q.len - begin < c.page_tokens ? q.len - begin : c.page_tokens;
  const long long stride = is_v ? v_stride : k_stride;
  const int pieces = (hi - lo) * kRow;
  const long long x0 = (q.row0 + (begin + lo - first)) * stride + (long long)head * D;
  using Raw = typename std::conditional<XB, uint4, float4>::type;
  Raw x[P][XB ? 1 : 2];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = threadIdx.x + i * T;
    if (p < pieces) {
      const long long e = x0 + (p / kRow) * stride + (p % kRow) * 8;
      const Raw* g = XB ? reinterpret_cast<const Raw*>(static_cast<const uint16_t*>(is_v ? vx : kx) + e)
                        : reinterpret_cast<const Raw*>(static_cast<const float*>(is_v ? vx : kx) + e);
#pragma unroll
      for (int k = 0; k < (XB ? 1 : 2); ++k) x[i][k] = __ldg(g + k);
    }
  }
  if (id < 0 || id >= c.n_pages) {
    record_status(c.status, QMV_E_ARG);
    return;
  }
  const long long at = (long long)id * c.kv_heads + head;
  int8_t* lev = (is_v ? c.v : c.k) + at * c.page_tokens * D;
  float* scale = (is_v ? c.v_scale : c.k_scale) + at;
  const float had = lo > 0 ? *scale : 0.f;
  // value e of piece i
  auto value = [&](int i, int e) -> float {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&x[i][0]);
    return XB ? __uint_as_float((e & 1) ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16) : __uint_as_float(w[e]);
  };
  float amax = 0.f;
  uint32_t most = 0u;  // of a thread's bfloat16 values, in pairs
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (threadIdx.x + i * T < pieces) {
      if (XB) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&x[i][0]);
#pragma unroll
        for (int e = 0; e < 4; ++e) asm("max.bf16x2 %0, %0, %1;" : "+r"(most) : "r"(w[e] & 0x7fff7fffu));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(value(i, e)));
      }
    }
  if (XB) amax = fmaxf(__uint_as_float(most << 16), __uint_as_float(most & 0xffff0000u));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
  __syncthreads();
  for (int w = 0; w < (T >> 5); ++w) amax = fmaxf(amax, part[w]);
  const float want = amax < 1e-30f ? 0.f : __fmul_rn(amax, 1.0f / 127.0f);
  const float d = fmaxf(want, had);
  // a scale the cache never gets from its rows (below 1e-30 / 127) leaves no levels
  const float inv = d > 0x1p-110f ? __fdiv_rn(1.0f, d) : 0.f;
  uint64_t inv2;
  asm("mov.b64 %0, {%1, %1};" : "=l"(inv2) : "f"(inv));
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = threadIdx.x + i * T;
    if (p < pieces) {
      float t[8];  // (no level passes 127: d is at least the rows' amax * RN(1/127))
#pragma unroll
      for (int e = 0; e < 8; e += 2) step2(value(i, e), value(i, e + 1), inv2, t[e], t[e + 1]);
      const uint32_t w[2] = {pack_levels(t[0], t[1], t[2], t[3]), pack_levels(t[4], t[5], t[6], t[7])};
      *reinterpret_cast<uint2*>(lev + (long long)lo * D + 8 * p) = make_uint2(w[0], w[1]);
    }
  }
  if (d > had && lo > 0) {
    const float ratio = __fdiv_rn(had, d);
    for (int p = threadIdx.x; p < lo * kRow; p += T) {
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
  // (the barrier above came after every thread's read of the old scale)
  if (threadIdx.x == 0) *scale = d;
}

// Rows read back: a CTA takes U * 256 pieces of one (sequence, head, K or V), each thread U of them, whose page
// ids, then levels and scales, are all asked for before the first is used.  A piece is 16 levels for bfloat16
// and 4 for float32, so that a warp's stores leave whole lines.
template <int D, bool XB, int U>
__global__ void __launch_bounds__(256) kv_read_kernel(const __grid_constant__ KvRef c, void* __restrict__ ko,
                                                      void* __restrict__ vo) {
  griddep_wait();
  griddep_launch_dependents();
  using Piece = typename std::conditional<XB, uint4, uint32_t>::type;
  constexpr int kLevels = (int)sizeof(Piece);
  constexpr int kRow = D / kLevels;  // pieces of a row
  constexpr int kRows = 256 / kRow;
  const int s = blockIdx.y;
  // the heads of the same rows lie side by side in the output, so their CTAs follow each other
  const int head = blockIdx.x % (2 * c.kv_heads) >> 1;
  const bool is_v = blockIdx.x & 1;
  const KvSeq q = kv_seq(c, s);
  const int r0 = blockIdx.x / (2 * c.kv_heads) * (U * kRows) + threadIdx.x / kRow;
  const int piece = threadIdx.x % kRow;
  const int8_t* lev = is_v ? c.v : c.k;
  const float* scale = is_v ? c.v_scale : c.k_scale;
  const int32_t* pages = c.page_table + (long long)s * c.table_stride;
  const int first = q.len - q.n;
  int id[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = r0 + u * kRows;
    id[u] = r < q.n ? __ldg(pages + ((first + r) >> c.page_shift)) : -1;
  }
  Piece x[U];
  float d[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = r0 + u * kRows;
    if ((unsigned)id[u] >= (unsigned)c.n_pages) {
      if (r < q.n) record_status(c.status, QMV_E_ARG);
      id[u] = -1;
      continue;
    }
    const long long at = (long long)id[u] * c.kv_heads + head;
    d[u] = __ldg(scale + at);
    x[u] = __ldg(reinterpret_cast<const Piece*>(lev + (at * c.page_tokens + ((first + r) & (c.page_tokens - 1))) * D +
                                                kLevels * piece));
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (id[u] < 0) continue;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&x[u]);
    float f[kLevels];
#pragma unroll
    for (int e = 0; e < kLevels; ++e) f[e] = __fmul_rn((float)(int8_t)(w[e >> 2] >> (8 * (e & 3))), d[u]);
    const long long o = ((q.row0 + r0 + u * kRows) * c.kv_heads + head) * D + kLevels * piece;
    if constexpr (XB) {
      uint4* g = reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? vo : ko) + o);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        g[h] = make_uint4(pack_bf16x2(f[8 * h], f[8 * h + 1]), pack_bf16x2(f[8 * h + 2], f[8 * h + 3]),
                          pack_bf16x2(f[8 * h + 4], f[8 * h + 5]), pack_bf16x2(f[8 * h + 6], f[8 * h + 7]));
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(is_v ? vo : ko) + o) = make_float4(f[0], f[1], f[2], f[3]);
    }
  }
}

template <int D, bool XB>
cudaError_t launch_write(const KvRef& c, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                         cudaStream_t stream) {
  const int pages = kv_pages_bound(c.max_rows, c.page_tokens);
  const dim3 grid((unsigned)pages, (unsigned)c.n_seq, (unsigned)(2 * c.kv_heads));
  // pieces of the most rows that a page may receive, over at most 256 threads of 1 or 4, else of 8: 16384 rows of
  // 8 heads of 128, pages of 16 tokens, 18.7 us with 4 pieces a thread, 23.6 with 8; 256 single rows 5.1 with 1, 6.8
  // with 8; heads of 256 and pages of 64 (512 threads of 4) 37.0 with 4, 35.4 with 8
  const int pieces = (c.max_rows < c.page_tokens ? c.max_rows : c.page_tokens) * (D / 8);
  const int per = pieces <= 64 ? 1 : pieces <= 4 * 256 ? 4 : 8;
  auto kern = per == 1 ? kv_write_kernel<D, XB, 1> : per == 4 ? kv_write_kernel<D, XB, 4> : kv_write_kernel<D, XB, 8>;
  // 64 threads at least: they also move a raised page's levels
  const int threads = pieces <= 64 * per ? 64 : (pieces + 32 * per - 1) / (32 * per) * 32;
  return launch_dependent(kern, grid, threads, 0, stream, c, k, (long long)k_stride, v, (long long)v_stride);
}

template <int D, bool XB>
cudaError_t launch_read(const KvRef& c, void* k, void* v, const DeviceInfo& dev, cudaStream_t stream) {
  constexpr int kRows = 256 / (D / (XB ? 16 : 4)), kFew = XB ? 1 : 2, kMany = XB ? 4 : 8;
  // more pieces a thread where that still leaves every SM several CTAs (float32, 8 heads of 128, with 2 against 4 and
  // 16: 64 sequences of 33 rows 6.2, 6.5 and 7.6 us; 16 of 8000, with 2 -> 8 and 16 196 and 198 us)
  const long long one = (long long)((c.max_rows + kFew * kRows - 1) / (kFew * kRows)) * c.n_seq * 2 * c.kv_heads;
  const int u = one >= (XB ? 64LL : 32LL) * dev.sm_count ? kMany : kFew;
  const long long x = (long long)((c.max_rows + u * kRows - 1) / (u * kRows)) * (2 * c.kv_heads);
  if (x > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)x, (unsigned)c.n_seq);
  return u == kMany ? launch_dependent(kv_read_kernel<D, XB, kMany>, grid, 256, 0, stream, c, k, v)
                    : launch_dependent(kv_read_kernel<D, XB, kFew>, grid, 256, 0, stream, c, k, v);
}

}  // namespace

cudaError_t launch_kv_write(const KvRef& c, bool x_bf16, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, cudaStream_t stream) {
  switch (c.head_dim) {
    case 64:
      return x_bf16 ? launch_write<64, true>(c, k, k_stride, v, v_stride, stream)
                    : launch_write<64, false>(c, k, k_stride, v, v_stride, stream);
    case 128:
      return x_bf16 ? launch_write<128, true>(c, k, k_stride, v, v_stride, stream)
                    : launch_write<128, false>(c, k, k_stride, v, v_stride, stream);
    default:
      return x_bf16 ? launch_write<256, true>(c, k, k_stride, v, v_stride, stream)
                    : launch_write<256, false>(c, k, k_stride, v, v_stride, stream);
  }
}

cudaError_t launch_kv_read(const KvRef& c, bool out_bf16, void* k, void* v, const DeviceInfo& dev,
                           cudaStream_t stream) {
  switch (c.head_dim) {
    case 64: return out_bf16 ? launch_read<64, true>(c, k, v, dev, stream) : launch_read<64, false>(c, k, v, dev, stream);
    case 128:
      return out_bf16 ? launch_read<128, true>(c, k, v, dev, stream) : launch_read<128, false>(c, k, v, dev, stream);
    default:
      return out_bf16 ? launch_read<256, true>(c, k, v, dev, stream) : launch_read<256, false>(c, k, v, dev, stream);
  }
}

}  // namespace qmv
