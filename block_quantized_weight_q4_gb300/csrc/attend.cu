// attend.cu -- softmax attention of a call's rows over the paged 8-bit cache.
#include "kv.cuh"

namespace qmv {

namespace {

// One warp per (row, head): a lane holds head_dim / 32 values of q and of the sum; the running
// maximum and sum of the softmax go over the keys one by one.
template <int D, bool XB>
__global__ void __launch_bounds__(128) attend_plain_kernel(const __grid_constant__ KvRef c,
                                                           const __grid_constant__ AttendArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (w >= c.rows * a.heads) return;
  const long long row = w / a.heads;
  const int head = (int)(w % a.heads);
  const int kvh = head / (a.heads / c.kv_heads);
  const int s = kv_seq_of_row(c, row);
  const KvSeq sq = kv_seq(c, s);
  if (row < sq.row0 || row >= sq.row0 + sq.n) return;
  const int pos = sq.len - sq.n + (int)(row - sq.row0);
  const int end = a.causal ? pos + 1 : sq.len;
  const int begin = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;

  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const long long at = row * a.q_stride + (long long)head * D + lane * E + e;
    q[e] = XB ? bf16_bits_to_f32(static_cast<const uint16_t*>(a.q)[at]) : static_cast<const float*>(a.q)[at];
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  int id = -1;
  float dk = 0.f, dv = 0.f;
  for (int j = begin; j < end; ++j) {
    if (j == begin || j % c.page_tokens == 0) {
      id = kv_page(c, s, j / c.page_tokens);
      if (id >= 0) {
        dk = __ldg(c.k_scale + (long long)id * c.kv_heads + kvh) * a.scale;
        dv = __ldg(c.v_scale + (long long)id * c.kv_heads + kvh);
      }
    }
    if (id < 0) continue;
    const long long at = (((long long)id * c.kv_heads + kvh) * c.page_tokens + j % c.page_tokens) * D + lane * E;
    float z = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) z = fmaf(q[e], (float)c.k[at + e], z);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
    z *= dk;
    const float mn = fmaxf(m, z);
    const float keep = m == -INFINITY ? 0.f : expf(m - mn);
    const float p = expf(z - mn);
    l = l * keep + p;
    const float pv = p * dv;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(pv, (float)c.v[at + e], o[e] * keep);
    m = mn;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float y = l > 0.f ? o[e] / l : o[e];
    const long long at = row * a.out_stride + (long long)head * D + lane * E + e;
    if (XB) {
      static_cast<uint16_t*>(a.out)[at] = (uint16_t)(pack_bf16x2(y, y) & 0xFFFFu);
    } else {
      static_cast<float*>(a.out)[at] = y;
    }
  }
}

}  // namespace

cudaError_t launch_attend(const KvRef& c, const AttendArgs& a, bool x_bf16, const DeviceInfo&, cudaStream_t stream) {
  const long long warps = c.rows * a.heads;
  const unsigned grid = (unsigned)((warps + 3) / 4);
  auto kern = c.head_dim == 64    ? (x_bf16 ? attend_plain_kernel<64, true> : attend_plain_kernel<64, false>)
              : c.head_dim == 128 ? (x_bf16 ? attend_plain_kernel<128, true> : attend_plain_kernel<128, false>)
                                  : (x_bf16 ? attend_plain_kernel<256, true> : attend_plain_kernel<256, false>);
  kern<<<grid, 128, 0, stream>>>(c, a);
  return cudaGetLastError();
}

}  // namespace qmv
