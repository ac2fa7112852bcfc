// rope.cu -- norms of queries and keys for each head, and the position rotation, in one pass.
//
//   s = x w / sqrt(mean x^2 + eps)   over a head (where a norm is asked for; else s = x)
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t) factor,   t = pos freq_i,
// for the pairs (s_2i, s_2i+1) or (s_i, s_i+rot/2) of a head's first `rot` values; the others pass.
//
// Angles: a frequency in turns as an integer of 64 bits, off by 2 units at most, once a CTA; times the position, whose whole turns fall off
// the integer's top, it is the angle to 2^-32 turns at the farthest position (64 x 32-bit integer products in place of the 64-bit floating
// point that a GB300 has little of).  sinpi / cospi of its first 24 bits in float32, turned by what those leave, once for all heads of a
// row, in shared memory.
//
// Bound by the rows' bytes in and out; below that by a chain of loads, angles, one barrier and stores, so a CTA takes several rows where
// there are many: their angles together, their values two rows ahead.  The rows are cut so that the CTAs fill whole rounds of what the SMs
// hold at once, up to 8 each (powers of two of them: 8192 rows 37.6, 3000 rows 24.6, 1024 rows 9.6 us; as it is 35.0, 15.1, 7.1 us; up
// to 4: 37.6, 17.0, 7.1; up to 16: 34.2, 15.1, 7.1 and float32 rows 56.5 against 54.7 us).
// GB300, 32 + 8 heads of 128: 8192 bfloat16 rows with norms, half of each head turned, 35.4 us (4.7 TB/s; all of it 35.8, without norms 32.3),
// float32 ones 55.9 us (6.0 TB/s); 256 float32 rows 4.8, one bfloat16 row 2.8 us.  The bfloat16 rows take 17 instructions a value and 60% of
// the issue slots, as the code is: a float at a time, with selects and shuffles where a call has no norm, too.
#include <type_traits>

#include "qmv_common.cuh"
#include "qmv_internal.h"

namespace qmv {

namespace {

constexpr int kMaxThreads = 512;

// freq radians in turns, the fraction of one in units of 2^-64: |freq| / 2 pi in two parts of 53 bits, so that what is rounded is
// below two units.
__device__ __forceinline__ unsigned long long turns_of(double freq) {
  const double kTurn = 0.15915494309189535, kTurnLow = -9.839338337591243e-18;  // 1 / 2 pi
  const double f = fabs(freq), t = f * kTurn, low = fma(f, kTurn, -t) + f * kTurnLow;
  const double part = t - floor(t);  // (exact, as t is not negative)
  const unsigned long long turns = (unsigned long long)(part * 0x1p64) + (unsigned long long)(long long)(low * 0x1p64);
  return freq < 0.0 ? 0ull - turns : turns;
}

// sin and cos of t units of 2^-64 turns: of its first 24 bits, as a signed number of half turns, then turned by the rest, whose square is
// below 2^-42.
__device__ __forceinline__ void sincos_of(unsigned long long t, float& s, float& c) {
  const int first = (int)(uint32_t)(t >> 32) & ~0xff;
  const float rest = (float)(uint32_t)(t >> 16 & 0xffffffu) * (3.14159265f * 0x1p-47f);
  float s0, c0;
  sincospif((float)first * 0x1p-31f, &s0, &c0);
  s = fmaf(c0, rest, s0);
  c = fmaf(-s0, rest, c0);
}

// A CTA takes `block` rows: a group of D / 8 lanes holds a head of a row, 8 values a lane: eight in a row, or (HALVES) four of the lower half
// and the four that turn with them, so that no value changes lanes.
template <int D, bool XB, bool OB, bool HALVES>
__global__ void __launch_bounds__(kMaxThreads, 2) rope_kernel(const __grid_constant__ RopeArgs a, long long rows, int block) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int L = D / 8;
  extern __shared__ float2 turn[];  // block x rot / 2
  const long long row0 = (long long)blockIdx.x * block;
  const int n = (int)min((long long)block, rows - row0);
  const int heads = a.heads + a.kv_heads;
  const int gl = threadIdx.x % L;
  const int slots = blockDim.x / L;
  // the lane's two fours: values lo .. lo + 3 and hi .. hi + 3 of the head; four angles where it turns
  const bool turns_here = 8 * gl < a.rot;
  const int lo = HALVES && turns_here ? 4 * gl : 8 * gl, hi = HALVES && turns_here ? a.rot / 2 + 4 * gl : 8 * gl + 4;
  using Raw = typename std::conditional<XB, uint2, float4>::type;
  alignas(16) Raw raw[2][2] = {};  // two rows' values are on their way
  const int mine = threadIdx.x / L;
  // where the lane reads and writes, a row further each time
  constexpr int kIn = XB ? 2 : 4, kOut = OB ? 2 : 4;
  const uint8_t* in = nullptr;
  uint8_t* out = nullptr;
  long long in_step = 0, out_step = 0;
  bool live = false;
  const float* w = nullptr;
  auto place = [&](int head) {
    live = head < heads;
    const bool is_k = head >= a.heads;
    const int of = is_k ? head - a.heads : head;
    in_step = (is_k ? a.k_stride : a.q_stride) * kIn;
    out_step = (is_k ? a.k_out_stride : a.q_out_stride) * kOut;
    in = static_cast<const uint8_t*>(is_k ? a.k : a.q) + row0 * in_step + (of * D + lo) * kIn;
    out = static_cast<uint8_t*>(is_k ? a.k_out : a.q_out) + row0 * out_step + (of * D + lo) * kOut;
    w = is_k ? a.k_weight : a.q_weight;
  };
  const int in_far = (hi - lo) * kIn, out_far = (hi - lo) * kOut;
  auto load = [&](Raw (&to)[2], int r) {
    if (live && r < n) {
      // (plain loads: the outputs may be the inputs' own places)
      if (XB && !HALVES) {
        const uint4 u = *reinterpret_cast<const uint4*>(in);
        reinterpret_cast<uint4&>(to) = u;
      } else {
        to[0] = *reinterpret_cast<const Raw*>(in);
        to[1] = *reinterpret_cast<const Raw*>(in + in_far);
      }
    }
    in += in_step;
  };
  place(mine);
  load(raw[0], 0);  // while the angles are formed
  load(raw[1], 1);
  const int half = a.rot / 2;
  unsigned long long turns = 0;
  float none = 0.f;  // NaN where the frequency is past what two parts of 1 / 2 pi reduce, or not finite
  for (int i = threadIdx.x, held = -1; i < half * n; i += blockDim.x) {
    const int r = i / half, f = i - r * half;
    if (f != held) {
      const float freq = __ldg(a.freq + f);
      none = fabsf(freq) < 0x1p40f ? 0.f : NAN;
      turns = turns_of((double)freq), held = f;
    }
    const unsigned long long t = turns * (unsigned long long)(long long)__ldg(a.pos + row0 + r);
    float c, s;
    sincos_of(t, s, c);
    // the first pairs of the lanes' four angles, then the second: 16-byte loads of neighbours lie in different banks
    turn[r * half + ((f & 2) / 2 * (half / 4) + f / 4) * 2 + (f & 1)] = make_float2(fmaf(c, a.factor, none), fmaf(s, a.factor, none));
  }
  __syncthreads();
  // every lane of a warp goes round as often: the shuffles need them all
  for (int first = 0; first < heads; first += slots) {
    if (first > 0) {
      place(first + mine);
      load(raw[0], 0);
      load(raw[1], 1);
    }
    float ww[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) ww[e] = w != nullptr ? __ldg(w + (e < 4 ? lo + e : hi + e - 4)) : 0.f;
    auto one = [&](Raw (&from)[2], int r) {
      float v[8];
      const uint32_t* u = reinterpret_cast<const uint32_t*>(from);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = XB ? __uint_as_float((e & 1) ? u[e >> 1] & 0xffff0000u : u[e >> 1] << 16) : __uint_as_float(u[e]);
      load(from, r + 2);
      if (a.q_weight != nullptr || a.k_weight != nullptr) {
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(v[e], v[e], sum);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (w != nullptr) {
          const float s = rsqrtf(fmaf(sum, 1.0f / D, a.eps));
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(__fmul_rn(v[e], s), ww[e]);
        }
      }
      if (turns_here) {
        const float4* table = reinterpret_cast<const float4*>(turn + r * half);
        const float4 t0 = table[gl], t1 = table[half / 4 + gl];
        const float c[4] = {t0.x, t0.z, t1.x, t1.z}, s[4] = {t0.y, t0.w, t1.y, t1.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float &x = v[HALVES ? i : 2 * i], &y = v[HALVES ? i + 4 : 2 * i + 1];
          const float u = x;
          x = fmaf(u, c[i], -__fmul_rn(y, s[i]));
          y = fmaf(u, s[i], __fmul_rn(y, c[i]));
        }
      }
      if (live) {
        if (OB) {
          const uint4 u = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
          if (HALVES) {
            *reinterpret_cast<uint2*>(out) = make_uint2(u.x, u.y);
            *reinterpret_cast<uint2*>(out + out_far) = make_uint2(u.z, u.w);
          } else {
            *reinterpret_cast<uint4*>(out) = u;
          }
        } else {
          *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
          *reinterpret_cast<float4*>(out + out_far) = make_float4(v[4], v[5], v[6], v[7]);
        }
      }
      out += out_step;
    };
    for (int r = 0; r < n; r += 2) {
      one(raw[0], r);
      if (r + 1 < n) one(raw[1], r + 1);
    }
  }
}

template <int D>
cudaError_t launch_dim(const RopeArgs& a, bool x_bf16, bool out_bf16, bool halves, int64_t rows, const DeviceInfo& dev, cudaStream_t stream) {
  // the heads in as few even shares as the threads take
  const int heads = a.heads + a.kv_heads, most = kMaxThreads / (D / 8), shares = (heads + most - 1) / most;
  const int threads = ((heads + shares - 1) / shares * (D / 8) + 31) / 32 * 32;
  // rows of a CTA: up to kMaxBlock, such that the CTAs fill whole rounds of what the SMs hold (64 registers a thread)
  constexpr int kMaxBlock = 8;
  const int64_t held = (int64_t)dev.sm_count * (1024 / threads), rounds = (rows + held * kMaxBlock - 1) / (held * kMaxBlock);
  const int block = (int)((rows + held * rounds - 1) / (held * rounds));
  auto go = [&](auto kern) {
    return launch_dependent(kern, dim3((unsigned)((rows + block - 1) / block)), threads, (size_t)block * a.rot / 2 * sizeof(float2), stream, a, rows, block);
  };
  if (x_bf16) {
    if (out_bf16) return halves ? go(rope_kernel<D, true, true, true>) : go(rope_kernel<D, true, true, false>);
    return halves ? go(rope_kernel<D, true, false, true>) : go(rope_kernel<D, true, false, false>);
  }
  if (out_bf16) return halves ? go(rope_kernel<D, false, true, true>) : go(rope_kernel<D, false, true, false>);
  return halves ? go(rope_kernel<D, false, false, true>) : go(rope_kernel<D, false, false, false>);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int head_dim, bool x_bf16, bool out_bf16, bool halves, int64_t rows, const DeviceInfo& dev,
                        cudaStream_t stream) {
  if (head_dim == 64) return launch_dim<64>(a, x_bf16, out_bf16, halves, rows, dev, stream);
  if (head_dim == 128) return launch_dim<128>(a, x_bf16, out_bf16, halves, rows, dev, stream);
  return launch_dim<256>(a, x_bf16, out_bf16, halves, rows, dev, stream);
}

}  // namespace qmv
