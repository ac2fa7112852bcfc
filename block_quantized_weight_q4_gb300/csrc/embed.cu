// embed.cu -- rows of a block-quantized token table (Krafla page, "Body": tok_emb), scaled.
//
//   out[r][c] = fl(fl(level d) scale) of row ids[r], rounded once more to bfloat16.
//
// A gather: bound by the rows' bytes in and out, and for a few rows by three dependent loads (id, quants and
// scales together, then the store).  A thread takes 8 bytes of Q4_0 quants (half a block) or 16 of Q8_0 quants: 16 values.
#include "qmv_common.cuh"
#include "qmv_internal.h"

namespace qmv {

namespace {

constexpr int kThreads = 256;

template <bool OB>
__device__ __forceinline__ void store8(void* out, long long at, const float (&v)[8]) {
  if (OB) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
    float4* f = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
    f[0] = make_float4(v[0], v[1], v[2], v[3]);
    f[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

template <int WT, bool F16, bool OB>
__global__ void __launch_bounds__(kThreads) embed_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ d,
                                                         const int64_t* __restrict__ ids, long long rows, long long vocab,
                                                         int cols, float scale, void* __restrict__ out) {
  griddep_wait();
  griddep_launch_dependents();
  const int pieces = cols >> 4;  // of a row
  const long long at = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long row = at / pieces;
  if (row >= rows) return;
  const int piece = (int)(at - row * pieces);
  const long long id = __ldg(ids + row);
  float v[2][8];
  if (id < 0 || id >= vocab) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[0][e] = v[1][e] = 0.f;
  } else {
    const long long block = id * (cols >> 5) + (piece >> 1);
    const float s = F16 ? f16_bits_to_f32(__ldg(reinterpret_cast<const uint16_t*>(d) + block))
                        : __ldg(reinterpret_cast<const float*>(d) + block);
    auto value = [&](int level) { return __fmul_rn(__fmul_rn((float)level, s), scale); };
    if (WT == QMV_Q4_0) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(q + block * 16 + (piece & 1) * 8));
      const uint32_t w[2] = {u.x, u.y};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t b = w[e >> 2] >> (8 * (e & 3));
        v[0][e] = value((int)(b & 15u) - 8);
        v[1][e] = value((int)((b >> 4) & 15u) - 8);
      }
    } else {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(q + block * 32 + (piece & 1) * 16));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e >> 3][e & 7] = value((int)(int8_t)(w[e >> 2] >> (8 * (e & 3))));
    }
  }
  const long long base = row * cols + (piece >> 1) * 32;
  // Q4_0: elements 8h .. 8h + 7 and 16 + 8h ..; Q8_0: 16h .. 16h + 15
  const int h = piece & 1;
  store8<OB>(out, base + (WT == QMV_Q4_0 ? 8 * h : 16 * h), v[0]);
  store8<OB>(out, base + (WT == QMV_Q4_0 ? 16 + 8 * h : 16 * h + 8), v[1]);
}

}  // namespace

cudaError_t launch_embed(const MatrixRef& m, const int64_t* ids, int64_t rows, float scale, bool out_bf16, void* out,
                         cudaStream_t stream) {
  const long long total = rows * (m.cols / 16);
  const long long ctas = (total + kThreads - 1) / kThreads;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  auto go = [&](auto kern) {
    return launch_dependent(kern, dim3((unsigned)ctas), kThreads, 0, stream, m.q, m.d, ids, rows, m.rows, m.cols, scale, out);
  };
  if (m.wtype == QMV_Q4_0) {
    if (m.scale_f16) return out_bf16 ? go(embed_kernel<QMV_Q4_0, true, true>) : go(embed_kernel<QMV_Q4_0, true, false>);
    return out_bf16 ? go(embed_kernel<QMV_Q4_0, false, true>) : go(embed_kernel<QMV_Q4_0, false, false>);
  }
  if (m.scale_f16) return out_bf16 ? go(embed_kernel<QMV_Q8_0, true, true>) : go(embed_kernel<QMV_Q8_0, true, false>);
  return out_bf16 ? go(embed_kernel<QMV_Q8_0, false, true>) : go(embed_kernel<QMV_Q8_0, false, false>);
}

}  // namespace qmv
