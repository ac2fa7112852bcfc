// rope.cu -- norms of queries and keys for each head, and the position rotation, in one pass.
//
//   s = x w / sqrt(mean x^2 + eps)   over a head (where a norm is asked for; else s = x)
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t) factor,   t = pos freq_i,
// for the pairs (s_2i, s_2i+1) or (s_i, s_i+rot/2) of a head's first `rot` values; the others pass.
//
// Angles: t is formed in 64 bits in turns, and what is left of whole turns goes to cospi / sinpi in float32, so a far
// position costs no accuracy.  That is rot / 2 angles a row, once for all its heads, in shared memory: the 64-bit work is
// 10 operations an angle, shared by all heads.
#include "qmv_common.cuh"
#include "qmv_internal.h"

namespace qmv {

namespace {

constexpr int kMaxThreads = 1024;

// pos * freq radians, less its whole turns, in units of pi: the product (31 + 24 bits) and its product with 1 / 2 pi (106 bits,
// in two parts) keep what 64 bits round away, so the error is the float32 rounding of the result alone.
__device__ __forceinline__ float angle(double pos, double freq) {
  const double kTurn = 0.15915494309189535, kTurnLow = -9.8393383375912e-18;  // 1 / 2 pi
  const double a = pos * freq, a_low = fma(pos, freq, -a);
  const double t = a * kTurn;
  const double low = fma(a, kTurn, -t) + fma(a, kTurnLow, a_low * kTurn);
  return (float)(2.0 * ((t - rint(t)) + low));
}

// A CTA takes one row: a group of D / 8 lanes holds a head, 8 values a lane.
template <int D, bool XB, bool OB, bool HALVES>
__global__ void __launch_bounds__(kMaxThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int L = D / 8;
  __shared__ float2 turn[D / 2];
  const long long row = blockIdx.x;
  const int heads = a.heads + a.kv_heads;
  const int gl = threadIdx.x % L;
  const int slots = blockDim.x / L;
  float v[8];
  auto load = [&](int head) {
    const bool is_k = head >= a.heads;
    const void* x = is_k ? a.k : a.q;
    const long long at = is_k ? row * a.k_stride + (long long)(head - a.heads) * D : row * a.q_stride + (long long)head * D;
    // (plain loads: the outputs may be the inputs' own places)
    if (XB) {
      const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at + 8 * gl);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at + 8 * gl);
      const float4 f0 = f[0], f1 = f[1];
      v[0] = f0.x, v[1] = f0.y, v[2] = f0.z, v[3] = f0.w;
      v[4] = f1.x, v[5] = f1.y, v[6] = f1.z, v[7] = f1.w;
    }
  };
  int head = threadIdx.x / L;
  if (head < heads) load(head);  // on its way while the angles are formed
  const int half = a.rot / 2;
  for (int i = threadIdx.x; i < half; i += blockDim.x) {
    const float half_turns = angle((double)__ldg(a.pos + row), (double)__ldg(a.freq + i));
    float c, s;
    sincospif(half_turns, &s, &c);
    turn[i] = make_float2(c * a.factor, s * a.factor);
  }
  __syncthreads();
  // every lane of a warp goes round as often: the shuffles need them all
  for (int first = 0; first < heads; first += slots, head += slots) {
    const bool live = head < heads;
    if (!live) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
    } else if (first > 0) {
      load(head);
    }
    const bool is_k = head >= a.heads;
    const float* w = is_k ? a.k_weight : a.q_weight;
    if (a.q_weight != nullptr || a.k_weight != nullptr) {
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(v[e], v[e], sum);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (w != nullptr && live) {
        const float r = __frsqrt_rn(__fadd_rn(__fmul_rn(sum, 1.0f / D), a.eps));
        const float4* wf = reinterpret_cast<const float4*>(w + 8 * gl);
        const float4 w0 = __ldg(wf), w1 = __ldg(wf + 1);
        const float ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(__fmul_rn(v[e], r), ww[e]);
      }
    }
    if (HALVES) {
      const int hl = a.rot / 16;  // lanes of a half
      const bool lower = gl < hl, in = gl < 2 * hl;
      const int lane = threadIdx.x & 31;
      const int from = !in ? lane : lower ? lane + hl : lane - hl;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float u = __shfl_sync(0xffffffffu, v[e], from);
        if (in) {
          const float2 t = turn[8 * (lower ? gl : gl - hl) + e];
          v[e] = lower ? fmaf(v[e], t.x, -__fmul_rn(u, t.y)) : fmaf(u, t.y, __fmul_rn(v[e], t.x));
        }
      }
    } else if (8 * gl < a.rot) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 t = turn[4 * gl + e / 2];
        const float x0 = v[e], x1 = v[e + 1];
        v[e] = fmaf(x0, t.x, -__fmul_rn(x1, t.y));
        v[e + 1] = fmaf(x0, t.y, __fmul_rn(x1, t.x));
      }
    }
    if (live) {
      void* out = is_k ? a.k_out : a.q_out;
      const long long at = (is_k ? row * a.k_out_stride + (long long)(head - a.heads) * D : row * a.q_out_stride + (long long)head * D) + 8 * gl;
      if (OB) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
      } else {
        float4* f = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
        f[0] = make_float4(v[0], v[1], v[2], v[3]);
        f[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
  }
}

template <int D>
cudaError_t launch_dim(const RopeArgs& a, bool x_bf16, bool out_bf16, bool halves, int64_t rows, cudaStream_t stream) {
  const int lanes = (a.heads + a.kv_heads) * (D / 8);
  const int threads = lanes >= kMaxThreads ? kMaxThreads : (lanes + 31) / 32 * 32;
  auto go = [&](auto kern) { return launch_dependent(kern, dim3((unsigned)rows), threads, 0, stream, a); };
  if (x_bf16) {
    if (out_bf16) return halves ? go(rope_kernel<D, true, true, true>) : go(rope_kernel<D, true, true, false>);
    return halves ? go(rope_kernel<D, true, false, true>) : go(rope_kernel<D, true, false, false>);
  }
  if (out_bf16) return halves ? go(rope_kernel<D, false, true, true>) : go(rope_kernel<D, false, true, false>);
  return halves ? go(rope_kernel<D, false, false, true>) : go(rope_kernel<D, false, false, false>);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int head_dim, bool x_bf16, bool out_bf16, bool halves, int64_t rows, cudaStream_t stream) {
  if (head_dim == 64) return launch_dim<64>(a, x_bf16, out_bf16, halves, rows, stream);
  if (head_dim == 128) return launch_dim<128>(a, x_bf16, out_bf16, halves, rows, stream);
  return launch_dim<256>(a, x_bf16, out_bf16, halves, rows, stream);
}

}  // namespace qmv
