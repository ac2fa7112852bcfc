// norm.cu -- root-mean-square norm with the residual's addition, into the activations that the
// products read: float32, bfloat16, or the Q8_0 / f32-scale image (the layout of the runtime's
// quantized activations, Krafla page, "Quantization rule").
//
//   s = x + residual,  r = 1 / sqrt(mean s^2 + eps),  y = s w r.
//
// 8-bit output in one pass: a block's quants depend on t = s w only through t / amax(t), and r
// is common to the row, so the levels are those of t, and r only multiplies the block's scale.
// Nothing is kept but the row itself, in registers, until r is known.
//
// Bound by the bytes of the residual stream (read, written) and x: 2048 x 4096 bfloat16 rows into the image
// 15.6 us, 5.98 TB/s (88% of the measured copy rate; 16.2 us with a level's conversion, clamp and pack one by one), into
// bfloat16 6.2 TB/s; 700 x 11008 float32 into bfloat16 5.2 TB/s; one row of 4096 2.3 us, which is the launch and one
// chain of loads, the reduction and the stores.
#include "qmv_common.cuh"
#include "qmv_internal.h"

namespace qmv {

namespace {

constexpr int kNormMaxThreads = 1024;

// One CTA per row; thread t holds pieces t, t + T, ... of 8 values (NI of them at most), so that four
// neighbouring lanes hold a block of 32.
template <bool XB, int OUT, int NI>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_kernel(const void* __restrict__ x,
                                                                  const float* residual, float* residual_out,
                                                                  const float* __restrict__ weight, float eps,
                                                                  void* __restrict__ out, long long out_d_off,
                                                                  long long rows, int cols) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float part[32];
  const long long row = blockIdx.x;
  const int T = blockDim.x;
  const int pieces = cols >> 3;
  float v[NI][8];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int p = threadIdx.x + i * T;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
    if (p >= pieces) continue;
    const long long at = row * cols + 8LL * p;
    if (XB) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[i][2 * k] = __uint_as_float(w[k] << 16);
        v[i][2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    } else {
      const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
      const float4 a = __ldg(f), b = __ldg(f + 1);
      v[i][0] = a.x, v[i][1] = a.y, v[i][2] = a.z, v[i][3] = a.w;
      v[i][4] = b.x, v[i][5] = b.y, v[i][6] = b.z, v[i][7] = b.w;
    }
    if (residual != nullptr) {
      const float4* f = reinterpret_cast<const float4*>(residual + at);
      const float4 a = f[0], b = f[1];
      const float q[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = __fadd_rn(v[i][e], q[e]);
    }
    if (residual_out != nullptr) {
      float4* f = reinterpret_cast<float4*>(residual_out + at);
      f[0] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
      f[1] = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
    }
    const float4* wf = reinterpret_cast<const float4*>(weight + 8 * p);
    const float4 a = __ldg(wf), b = __ldg(wf + 1);
    const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sum = fmaf(v[i][e], v[i][e], sum);
      v[i][e] = __fmul_rn(v[i][e], w[e]);
    }
  }
  // the row's sum of squares: lanes, then warps, in a fixed order
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = 0.f;
  for (int w = 0; w < (T >> 5); ++w) sum += part[w];
  const float r = __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, (float)cols), eps));

#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int p = threadIdx.x + i * T;
    const bool live = p < pieces;
    const long long at = row * cols + 8LL * p;
    if (OUT == QMV_OUT_Q8) {
      float amax = 0.f;  // fmaxf skips a NaN operand
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[i][e]));
#pragma unroll
      for (int o = 1; o <= 2; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const bool zero = amax < 1e-30f;
      const float inv = zero ? 0.f : __fmul_rn(__frcp_rn(amax), 127.0f);
      uint64_t inv2;
      asm("mov.b64 %0, {%1, %1};" : "=l"(inv2) : "f"(inv));
      float t[8];  // within 127.5: inv is 127 / amax but for two roundings
#pragma unroll
      for (int e = 0; e < 8; e += 2) step2(v[i][e], v[i][e + 1], inv2, t[e], t[e + 1]);
      const uint32_t w[2] = {pack_levels(t[0], t[1], t[2], t[3]), pack_levels(t[4], t[5], t[6], t[7])};
      if (live) {
        uint8_t* o8 = static_cast<uint8_t*>(out);
        *reinterpret_cast<uint2*>(o8 + at) = make_uint2(w[0], w[1]);
        if ((p & 3) == 0)
          reinterpret_cast<float*>(o8 + out_d_off)[at >> 5] = zero ? 0.f : __fmul_rn(__fmul_rn(amax, 1.0f / 127.0f), r);
      }
    } else if (live) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = __fmul_rn(v[i][e], r);
      if (OUT == QMV_X_BF16) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) =
            make_uint4(pack_bf16x2(v[i][0], v[i][1]), pack_bf16x2(v[i][2], v[i][3]), pack_bf16x2(v[i][4], v[i][5]),
                       pack_bf16x2(v[i][6], v[i][7]));
      } else {
        float4* f = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
        f[0] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
        f[1] = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
      }
    }
  }
  // the image's padding between the quants and the scales (0 or 32 bytes)
  if (OUT == QMV_OUT_Q8 && row == 0 && threadIdx.x < 8) {
    const long long q_bytes = rows * cols;
    if (q_bytes + 4 * threadIdx.x < out_d_off)
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(out) + q_bytes + 4 * threadIdx.x) = 0u;
  }
}

template <bool XB, int OUT>
cudaError_t launch_typed(int64_t rows, int cols, const void* x, const float* residual, float* residual_out,
                         const float* weight, float eps, void* out, int64_t out_d_off, cudaStream_t stream) {
  const int pieces = cols / 8;
  // up to 512 threads, with up to 4 pieces each before they are more: 512 rows of 16384 float32 columns took 21.0 us
  // with 512 threads x 4 against 25.1 with 1024 x 2 (two CTAs a SM overlap their ends), 256 of 32768 took 22.3 with
  // 1024 x 4 against 26.6 with 512 x 8 (19.6 and 20.9 us since levels are packed in steps of two)
  const int ni = pieces <= 512 ? 1 : pieces <= 1024 ? 2 : 4;
  const int threads = ((pieces + ni - 1) / ni + 31) / 32 * 32;
  auto kern = ni == 1 ? rmsnorm_kernel<XB, OUT, 1> : ni == 2 ? rmsnorm_kernel<XB, OUT, 2> : rmsnorm_kernel<XB, OUT, 4>;
  return launch_dependent(kern, dim3((unsigned)rows), threads, 0, stream, x, residual, residual_out, weight, eps, out,
                          out_d_off, rows, cols);
}

}  // namespace

cudaError_t launch_rmsnorm(bool x_bf16, int64_t rows, int64_t cols, const void* x, const float* residual,
                           float* residual_out, const float* weight, float eps, int out_dtype, void* out,
                           int64_t out_d_off, cudaStream_t stream) {
  const int c = (int)cols;
  switch (out_dtype) {
    case QMV_OUT_Q8:
      return x_bf16 ? launch_typed<true, QMV_OUT_Q8>(rows, c, x, residual, residual_out, weight, eps, out, out_d_off, stream)
                    : launch_typed<false, QMV_OUT_Q8>(rows, c, x, residual, residual_out, weight, eps, out, out_d_off, stream);
    case QMV_X_BF16:
      return x_bf16 ? launch_typed<true, QMV_X_BF16>(rows, c, x, residual, residual_out, weight, eps, out, 0, stream)
                    : launch_typed<false, QMV_X_BF16>(rows, c, x, residual, residual_out, weight, eps, out, 0, stream);
    default:
      return x_bf16 ? launch_typed<true, QMV_X_F32>(rows, c, x, residual, residual_out, weight, eps, out, 0, stream)
                    : launch_typed<false, QMV_X_F32>(rows, c, x, residual, residual_out, weight, eps, out, 0, stream);
  }
}

}  // namespace qmv
