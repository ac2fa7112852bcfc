// embed.cu -- rows of a block-quantized token table (Krafla page, "Body": tok_emb), scaled.
//
//   out[r][c] = fl(fl(level d) scale) of row ids[r], rounded once more to bfloat16.
//
// A gather: bound by the rows' bytes in and out, and for a few rows by three dependent steps (the id, quants and scale together, the
// store).  A piece is 16 bytes of the output, 8 bfloat16 or 4 float32 values, so that a warp's store is whole lines; a thread has kEach
// pieces' loads on their way at once (2, 3, 4, 6 of them: 10.6, 9.9, 10.0, 14.6 us for 4096 rows of 4096 bfloat16 values, 15.8, 14.6, 14.3,
// 16.3 us for float32 ones).  Pieces of 32 bytes a thread, half of each line at a time: 10.0 and 19.9 us.
// GB300: 4096 rows of 4096 from Q4_0, bfloat16 10.0 us (4.2 TB/s of 42 MB; 14.6 instructions a value, 77% of the issue slots, as the code
// is: each byte is loaded and masked by two threads, one for each nibble), float32 14.3 us (5.3 TB/s of 76 MB); 1 row of 1024 1.5 us.
#include "qmv_common.cuh"
#include "qmv_internal.h"

namespace qmv {

namespace {

constexpr int kThreads = 256;
constexpr int kEach = 4;

// n / d for n below 2^31 by a product (Granlund and Montgomery): shift >= log2 d, magic = floor(2^32 (2^shift - d) / d) + 1.
struct Divisor {
  uint32_t d, magic, shift;
  explicit Divisor(uint32_t by) : d(by), shift(0) {
    while ((1ull << shift) < by) ++shift;
    magic = (uint32_t)(((1ull << 32) * ((1ull << shift) - by)) / by + 1);
  }
  __device__ __forceinline__ uint32_t of(uint32_t n) const { return (__umulhi(magic, n) + n) >> shift; }
};

template <int WT, bool F16, bool OB>
__global__ void __launch_bounds__(kThreads) embed_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ d,
                                                         const int64_t* __restrict__ ids, uint32_t total, const Divisor pieces,
                                                         long long vocab, int cols, float scale, uint4* __restrict__ out) {
  constexpr int kValues = OB ? 8 : 4, kPieces = 32 / kValues;  // of a piece; pieces of a block
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t at0 = blockIdx.x * (kThreads * kEach) + threadIdx.x;
  uint32_t piece[kEach];
  long long id[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint32_t at = at0 + i * kThreads, row = pieces.of(at);
    piece[i] = at - row * pieces.d;
    id[i] = at < total ? __ldg(ids + row) : -1;
  }
  uint32_t w[kEach][kValues / 4];
  float s[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    s[i] = 0.f;
#pragma unroll
    for (int k = 0; k < kValues / 4; ++k) w[i][k] = 0u;
    if (id[i] < 0 || id[i] >= vocab) continue;
    const long long block = id[i] * (cols >> 5) + piece[i] / kPieces;
    s[i] = F16 ? f16_bits_to_f32(__ldg(reinterpret_cast<const uint16_t*>(d) + block)) : __ldg(reinterpret_cast<const float*>(d) + block);
    // Q4_0: byte j holds elements j and j + 16
    const uint8_t* from = q + (WT == QMV_Q4_0 ? block * 16 + piece[i] % (kPieces / 2) * kValues : block * 32 + piece[i] % kPieces * kValues);
    if (OB) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(from));
      w[i][0] = u.x, w[i][kValues / 4 - 1] = u.y;
    } else {
      w[i][0] = __ldg(reinterpret_cast<const uint32_t*>(from));
    }
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const uint32_t at = at0 + i * kThreads;
    if (at >= total) break;
    const bool there = id[i] >= 0 && id[i] < vocab;
    const int nibble = piece[i] % kPieces >= kPieces / 2 ? 4 : 0;
    float v[kValues];
#pragma unroll
    for (int e = 0; e < kValues; ++e) {
      // the level as a float, by bits: 2^23 + n, and what is too much taken off (conversions have a quarter of the rate)
      const uint32_t n = WT == QMV_Q4_0 ? (w[i][e >> 2] >> (8 * (e & 3) + nibble) & 15u) | 0x4B000000u
                                        : prmt(w[i][e >> 2] ^ 0x80808080u, 0x4B000000u, 0x7650 + (e & 3));
      const float level = __uint_as_float(n) - (WT == QMV_Q4_0 ? 8388616.f : 8388736.f);
      v[e] = there ? __fmul_rn(__fmul_rn(level, s[i]), scale) : 0.f;
    }
    if (OB)
      out[at] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[kValues - 4], v[kValues - 3]),
                           pack_bf16x2(v[kValues - 2], v[kValues - 1]));
    else
      out[at] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
}

}  // namespace

cudaError_t launch_embed(const MatrixRef& m, const int64_t* ids, int64_t rows, float scale, bool out_bf16, void* out,
                         cudaStream_t stream) {
  const Divisor pieces((uint32_t)(m.cols / (out_bf16 ? 8 : 4)));
  auto go = [&](auto kern) {
    // rows of fewer than 2^31 pieces (with those behind the last CTA's end) at a time
    const int64_t most = ((1ll << 31) - kThreads * kEach) / pieces.d;
    for (int64_t r = 0; r < rows; r += most) {
      const uint32_t total = (uint32_t)((rows - r < most ? rows - r : most) * pieces.d);
      const cudaError_t err = launch_dependent(kern, dim3((total + kThreads * kEach - 1) / (kThreads * kEach)), kThreads, 0, stream, m.q, m.d,
                                               ids + r, total, pieces, (long long)m.rows, m.cols, scale,
                                               static_cast<uint4*>(out) + r * pieces.d);
      if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
  };
  if (m.wtype == QMV_Q4_0) {
    if (m.scale_f16) return out_bf16 ? go(embed_kernel<QMV_Q4_0, true, true>) : go(embed_kernel<QMV_Q4_0, true, false>);
    return out_bf16 ? go(embed_kernel<QMV_Q4_0, false, true>) : go(embed_kernel<QMV_Q4_0, false, false>);
  }
  if (m.scale_f16) return out_bf16 ? go(embed_kernel<QMV_Q8_0, true, true>) : go(embed_kernel<QMV_Q8_0, true, false>);
  return out_bf16 ? go(embed_kernel<QMV_Q8_0, false, true>) : go(embed_kernel<QMV_Q8_0, false, false>);
}

}  // namespace qmv
