// logprobs.cu -- log probabilities of given tokens, entropy and the top alternatives of rows of logits.
#include "qmv_common.cuh"
#include "qmv_internal.h"

namespace qmv {

namespace {

constexpr int kLpThreads = 512;

// A logit and its id as one key that orders as the result does: larger logits first, equal ones
// by the lower id.  The float's bits are mapped to an unsigned order; -0 counts as +0, NaN as the largest.
__device__ __forceinline__ unsigned long long lp_key(float x, unsigned id) {
  uint32_t b = __float_as_uint(x + 0.0f);
  if ((b & 0x7fffffffu) > 0x7f800000u) b = 0x7fffffffu;
  b = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((unsigned long long)b << 32) | (0xffffffffu - id);
}

__device__ __forceinline__ float lp_block_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < kLpThreads / 32; ++w) v += part[w];
  return v;
}

// One CTA per row: the maximum, then the sums, then one pass over the row for each alternative.
__global__ void __launch_bounds__(kLpThreads) logprobs_plain_kernel(const __grid_constant__ LogprobArgs a) {
  __shared__ float part[kLpThreads / 32];
  __shared__ unsigned long long keys[kLpThreads / 32];
  const long long row = blockIdx.x;
  const float* x = a.logits + row * a.stride;
  const int n = (int)a.vocab;
  float m = -INFINITY;
  bool bad = false;
  for (int j = threadIdx.x; j < n; j += kLpThreads) {
    const float v = x[j];
    bad |= isnan(v) || v == INFINITY;
    m = fmaxf(m, v);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  bad = __syncthreads_or(bad);
  for (int w = 0; w < kLpThreads / 32; ++w) m = fmaxf(m, part[w]);
  const bool none = m == -INFINITY && !bad;
  float z = 0.f, zx = 0.f;
  if (!none)
    for (int j = threadIdx.x; j < n; j += kLpThreads) {
      const float d = x[j] - m;
      const float e = expf(d);
      z += e;
      if (e > 0.f) zx = fmaf(e, d, zx);
    }
  z = lp_block_sum(z, part);
  zx = lp_block_sum(zx, part);
  const float lz = bad ? NAN : none ? INFINITY : logf(z);
  const float lse = none ? INFINITY : m + lz;
  if (threadIdx.x == 0 && a.entropy != nullptr) a.entropy[row] = bad ? NAN : none ? 0.f : lz - zx / z;
  for (int g = threadIdx.x; g < a.n_given; g += kLpThreads) {
    const long long id = a.given[row * a.n_given + g];
    a.given_logprob[row * a.n_given + g] = id >= 0 && id < a.vocab ? x[id] - lse : NAN;
  }
  unsigned long long last = ~0ull;
  for (int t = 0; t < a.n_top; ++t) {
    unsigned long long best = 0;
    for (int j = threadIdx.x; j < n; j += kLpThreads) {
      const unsigned long long k = lp_key(x[j], (unsigned)j);
      if (k < last && k > best) best = k;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long k = __shfl_xor_sync(0xffffffffu, best, o);
      best = k > best ? k : best;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) keys[threadIdx.x >> 5] = best;
    __syncthreads();
    for (int w = 0; w < kLpThreads / 32; ++w) best = keys[w] > best ? keys[w] : best;
    last = best;
    if (threadIdx.x == 0) {
      const unsigned id = 0xffffffffu - (unsigned)best;
      a.top_ids[row * a.n_top + t] = (int)id;
      a.top_logprob[row * a.n_top + t] = x[id] - lse;
    }
  }
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, int64_t rows, const DeviceInfo&, cudaStream_t stream) {
  logprobs_plain_kernel<<<(unsigned)rows, kLpThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace qmv
