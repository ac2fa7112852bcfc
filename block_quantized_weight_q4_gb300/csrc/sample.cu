// sample.cu -- the next ids from rows of logits: temperature, top-k, top-p and min-p, with given random numbers.
//
//   w_j = e^((x_j - max) / T),  id = the kept j with the largest (x_j - max) / T - ln e_j.
//
// With e_j exponential random numbers that is a draw from the kept w (of independent exponential clocks of rates w_j
// the first to ring is j with probability w_j over their sum), so no sum over the kept ids in an order of theirs is
// needed: the parts of a row join by a maximum, whose result does not depend on how the row is cut.
//
// The cuts are prefixes of the descending order (larger logits first, equal ones by the lower id), so each is one
// border.  Keys: a logit mapped to an unsigned order, then the id's complement: 64 bits, no two equal.  A pass over
// the row adds count and weight of 1024 buckets of (max - x) / T in shared memory (integers, so the order of the atomics
// does not matter); the bucket that holds the border, with all above it where that is few enough, is collected, sorted
// and walked.  A bucket that holds more than the list (equal or nearly equal logits) is cut again by its keys' bits.
//
// A row is one cluster's: 1, 2, 4 or 8 CTAs, which join in distributed shared memory; no workspace.
#include <cooperative_groups.h>

#include <mutex>

#include "qmv_common.cuh"
#include "qmv_internal.h"

namespace qmv {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBuckets = 1024;  // two a thread
constexpr int kList = 2048;     // keys that are collected and sorted
constexpr int kMaxRanks = 8;
using Key = unsigned long long;

// (as in logprobs.cu) larger logits first, equal ones by the lower id; -0 counts as +0
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ Key key_of(float x, uint32_t id) { return ((Key)ordered(x) << 32) | (0xffffffffu - id); }
__device__ __forceinline__ uint32_t id_of(Key k) { return 0xffffffffu - (uint32_t)k; }

// One row as its CTA sees it.
struct Row {
  const float* x;
  const float* e;
  int n;
  int head, quads, q0, q1;  // quads of 16 bytes from the row's first 16-byte boundary; the CTA's are q0 .. q1 - 1
  bool ends;                // this CTA also has the values before the first and after the last whole four
  float max, scale;         // scale: log2 e / T
};

// A logit's distance below the maximum in powers of two, its bucket and its weight.
__device__ __forceinline__ float below(const Row& r, float x) { return (r.max - x) * r.scale; }
__device__ __forceinline__ int bucket_of(float t) {  // (NaN, of 0 * inf, gives 0)
  return min((int)(t * 32.f), kBuckets - 1);
}
__device__ __forceinline__ float weight_of(float t) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(-t));
  return t == 0.f ? 1.f : y;
}
// The weight as an integer in units of 2^-31: sums of them are exact, so no order of adding matters.  An id counts
// to 2^-32 of the largest.
__device__ __forceinline__ uint32_t mass_of(float t) { return t > 0.f ? __float2uint_rn(weight_of(t) * 0x1p31f) : 0x80000000u; }

// f(x, id) for each of the CTA's logits, a thread's ids in rising order; four loads of 16 bytes are on their way at a time.
template <typename F>
__device__ __forceinline__ void for_each(const Row& r, F f) {
  if (r.ends && (int)threadIdx.x < r.head) f(__ldg(r.x + threadIdx.x), (int)threadIdx.x);
  const float4* xv = reinterpret_cast<const float4*>(r.x + r.head);
  for (int q = r.q0 + threadIdx.x; q < r.q1; q += 4 * kThreads) {
    float4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (q + i * kThreads < r.q1) v[i] = __ldg(xv + q + i * kThreads);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (q + i * kThreads < r.q1) {
        const int id = r.head + 4 * (q + i * kThreads);
        f(v[i].x, id);
        f(v[i].y, id + 1);
        f(v[i].z, id + 2);
        f(v[i].w, id + 3);
      }
  }
  const int id = r.head + 4 * r.quads + (int)threadIdx.x;
  if (r.ends && id < r.n) f(__ldg(r.x + id), id);
}

// The two best scores that a thread has seen: float32, so a draw that is close is decided again in 64 bits.
struct Best {
  float s0 = -INFINITY, s1 = -INFINITY;
  int i0 = -1, i1 = -1;
  __device__ __forceinline__ void take(float s, int id) {
    if (s > s0) {
      s1 = s0, i1 = i0;
      s0 = s, i0 = id;
    } else if (s > s1) {
      s1 = s, i1 = id;
    }
  }
};
struct Draw {  // a candidate's score in 64 bits; the larger wins, then the lower id
  double s;
  int id;
};
__device__ __forceinline__ Draw better(Draw a, Draw b) {
  if (b.id < 0) return a;
  if (a.id < 0 || b.s > a.s || (b.s == a.s && b.id < a.id)) return b;
  return a;
}

__device__ __forceinline__ float ln_of(float e) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(e));
  return y * 0.6931471805599453f;
}

struct Shared {
  uint32_t count[kBuckets], low[kBuckets], high[kBuckets];
  Key list[kList];
  uint32_t listed;
  // each rank's part of what is joined
  float rank_max;
  Key rank_key;
  int rank_bad;
  float rank_best;
  Draw rank_draw;
  // what rank 0 or every rank found
  int bucket;
  uint32_t above_count, in_count;
  Key above_mass, total_mass;
  Key border;
  Key border_mass;
  Key part_key[kWarps];
  Key scan_mass[kWarps];
  uint32_t scan_count[kWarps];
  float part[kWarps];
  Draw part_draw[kWarps];
};

__device__ __forceinline__ float block_max(Shared& sh, float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sh.part[0];
  for (int w = 1; w < kWarps; ++w) v = fmaxf(v, sh.part[w]);
  return v;
}

// Prefix sums over the threads (exclusive), and the totals.
__device__ __forceinline__ void block_scan(Shared& sh, uint32_t& c, Key& m, uint32_t& all_c, Key& all_m) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const uint32_t c0 = c;
  const Key m0 = m;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t uc = __shfl_up_sync(0xffffffffu, c, o);
    const Key um = __shfl_up_sync(0xffffffffu, m, o);
    if (lane >= o) c += uc, m += um;
  }
  __syncthreads();
  if (lane == 31) sh.scan_count[wid] = c, sh.scan_mass[wid] = m;
  __syncthreads();
  uint32_t bc = 0;
  Key bm = 0;
  all_c = 0, all_m = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w == wid) bc = all_c, bm = all_m;
    all_c += sh.scan_count[w];
    all_m += sh.scan_mass[w];
  }
  c += bc - c0;
  m += bm - m0;
}

__device__ __forceinline__ void add(Shared& sh, int b, uint32_t mass) {
  atomicAdd(&sh.count[b], 1u);
  const uint32_t old = atomicAdd(&sh.low[b], mass);
  if (old + mass < old) atomicAdd(&sh.high[b], 1u);
}

__device__ __forceinline__ void clear(Shared& sh) {
  for (int i = threadIdx.x; i < kBuckets; i += kThreads) sh.count[i] = sh.low[i] = sh.high[i] = 0u;
  if (threadIdx.x == 0) sh.listed = 0u;
}

// A thread's two buckets over all ranks.
__device__ __forceinline__ void gather(cg::cluster_group& cl, Shared& sh, int ranks, uint32_t (&c)[2], Key (&m)[2]) {
  c[0] = c[1] = 0;
  m[0] = m[1] = 0;
  for (int r = 0; r < ranks; ++r) {
    const Shared* o = ranks == 1 ? &sh : cl.map_shared_rank(&sh, r);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int b = 2 * threadIdx.x + k;
      c[k] += o->count[b];
      m[k] += ((Key)o->high[b] << 32) + o->low[b];
    }
  }
}

// Which bucket (or bin) holds the border: the first at which the count reaches `want_count`, or (want_count 0) the last whose
// exclusive mass is below `want_mass`.  Leaves it, what lies above it and what it holds in sh; every rank finds the same.
__device__ void find_border(cg::cluster_group& cl, Shared& sh, int ranks, uint32_t base_count, Key base_mass, uint32_t want_count,
                            double want_mass) {
  uint32_t c[2], all_c;
  Key m[2], all_m;
  gather(cl, sh, ranks, c, m);
  uint32_t pc = c[0] + c[1];
  Key pm = m[0] + m[1];
  block_scan(sh, pc, pm, all_c, all_m);
  pc += base_count;
  pm += base_mass;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const bool here = want_count != 0 ? pc < want_count && pc + c[k] >= want_count
                                      : c[k] != 0 && (double)pm < want_mass && (double)(pm + m[k]) >= want_mass;
    if (here) {
      sh.bucket = 2 * threadIdx.x + k;
      sh.above_count = pc;
      sh.above_mass = pm;
      sh.in_count = c[k];
    }
    pc += c[k];
    pm += m[k];
  }
  if (threadIdx.x == 0) sh.total_mass = all_m;
  __syncthreads();
}

// The smallest mapped logit whose bucket is at most b (buckets fall as logits rise).
__device__ __forceinline__ uint32_t edge_of(const Row& r, int b) {
  uint32_t lo = ordered(-INFINITY) + 1, hi = ordered(r.max);  // the maximum is in bucket 0
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (bucket_of(below(r, unordered(mid))) <= b)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// The collected keys in descending order.
__device__ void sort_list(Shared& sh, int n) {
  int size = 32;
  while (size < n) size <<= 1;
  for (int i = n + threadIdx.x; i < size; i += kThreads) sh.list[i] = 0;
  __syncthreads();
  for (int k = 2; k <= size; k <<= 1)
    for (int d = k >> 1; d > 0; d >>= 1) {
      for (int i = threadIdx.x; i < size / 2; i += kThreads) {
        const int a = 2 * i - (i & (d - 1)), b = a + d;
        const Key u = sh.list[a], v = sh.list[b];
        if ((u < v) == ((a & k) == 0)) sh.list[a] = v, sh.list[b] = u;
      }
      __syncthreads();
    }
}

// How many of the sorted list's first keys stay: those whose exclusive mass (over above_mass) is below `want`, among the
// first `n`; mass: what those weigh with above_mass.  Every thread gets the result.
__device__ int prefix_by_mass(const Row& r, Shared& sh, int n, Key above_mass, double want, Key& mass) {
  constexpr int kEach = kList / kThreads;
  uint32_t m[kEach];
  Key sum = 0;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = kEach * threadIdx.x + k;
    m[k] = i < n ? mass_of(below(r, unordered((uint32_t)(sh.list[i] >> 32)))) : 0u;
    sum += m[k];
  }
  uint32_t none = 0, all_c;
  Key all_m;
  block_scan(sh, none, sum, all_c, all_m);
  sum += above_mass;
  uint32_t stay = 0;
  Key got = 0;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    if (kEach * (int)threadIdx.x + k < n && (double)sum < want) stay += 1, got += m[k];
    sum += m[k];
  }
  uint32_t all = 0;
  block_scan(sh, stay, got, all, mass);
  mass += above_mass;
  return (int)all;
}

struct Border {
  Key key;        // kept: keys of at least this
  Key mass;       // the kept keys' weight
  int listed;     // > 0: the first `listed` of rank 0's sorted list are all that is kept
};

// The border in the bucket that find_border left in sh, among keys of at least `floor`.  want_count: that many stay; else those of exclusive mass below
// want_mass.  more_p > 0, where the list holds everything kept: the top-p cut is made in it, too.
__device__ Border resolve(cg::cluster_group& cl, const Row& r, Shared& sh, int rank, int ranks, Key floor, uint32_t want_count, double want_mass, float more_p) {
  uint32_t above = sh.above_count, inside = sh.in_count;
  Key above_mass = sh.above_mass;
  Key lo, hi;
  const bool whole = above + inside <= kList;
  lo = (Key)edge_of(r, sh.bucket) << 32;
  if (lo < floor) lo = floor;  // (the histograms count none below it)
  if (whole) {
    hi = ~(Key)0;
    above = 0;
    above_mass = 0;
  } else {
    hi = sh.bucket == 0 ? ~(Key)0 : ((Key)edge_of(r, sh.bucket - 1) << 32) - 1;
  }
  // cut again by the keys' bits: no two keys are equal, so at most 6 rounds of 10 bits leave fewer than the list holds
  for (int round = 0; !whole && inside > kList && round < 8; ++round) {
    const int bits = 64 - __clzll((long long)(hi - lo));
    const int shift = bits > 10 ? bits - 10 : 0;
    cl.sync();  // every rank has read the histograms
    clear(sh);
    __syncthreads();
    for_each(r, [&](float x, int id) {
      const Key k = key_of(x, (uint32_t)id);
      if (k >= lo && k <= hi) add(sh, (int)((hi - k) >> shift), mass_of(below(r, x)));
    });
    cl.sync();
    find_border(cl, sh, ranks, above, above_mass, want_count, want_mass);
    above = sh.above_count;
    above_mass = sh.above_mass;
    inside = sh.in_count;
    hi -= (Key)sh.bucket << shift;
    const Key low = hi - (((Key)1 << shift) - 1);
    lo = low > lo && low <= hi ? low : lo;
  }
  // collected at rank 0, in no order
  cl.sync();
  if (threadIdx.x == 0) sh.listed = 0u;
  cl.sync();
  Shared* home = ranks == 1 ? &sh : cl.map_shared_rank(&sh, 0);
  for_each(r, [&](float x, int id) {
    if (ordered(x) < (uint32_t)(lo >> 32)) return;
    const Key k = key_of(x, (uint32_t)id);
    if (k >= lo && k <= hi) {
      const uint32_t at = atomicAdd(&home->listed, 1u);
      if (at < (uint32_t)kList) home->list[at] = k;
    }
  });
  cl.sync();
  if (rank == 0) {
    const int n = min((int)sh.listed, kList);
    sort_list(sh, n);
    Key mass;
    int stay = want_count != 0 ? min(n, (int)(want_count - above)) : n;
    stay = prefix_by_mass(r, sh, stay, above_mass, want_count != 0 ? INFINITY : want_mass, mass);
    if (whole && more_p < 1.f) stay = prefix_by_mass(r, sh, stay, 0, (double)more_p * (double)mass, mass);
    if (threadIdx.x == 0) {
      sh.border = sh.list[max(stay, 1) - 1];
      sh.border_mass = mass;
      sh.bucket = max(stay, 1);
    }
  }
  cl.sync();
  Border b;
  b.key = home->border;
  b.mass = home->border_mass;
  b.listed = whole ? home->bucket : 0;
  return b;
}

struct SampleParams {
  const float* logits;
  const float* noise;
  long long stride, noise_stride;
  int vocab;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int64_t* ids;
};

__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ SampleParams p, int ranks) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ Shared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = ranks == 1 ? 0 : (int)cl.block_rank();
  const long long row = blockIdx.x / ranks;
  Row r;
  r.x = p.logits + row * p.stride;
  r.e = p.noise + row * p.noise_stride;
  r.n = p.vocab;
  r.head = min((int)((4 - ((reinterpret_cast<uintptr_t>(r.x) >> 2) & 3)) & 3), r.n);
  r.quads = (r.n - r.head) / 4;
  r.q0 = (int)((long long)r.quads * rank / ranks);
  r.q1 = (int)((long long)r.quads * (rank + 1) / ranks);
  r.ends = rank == 0;

  const float T = p.temperature != nullptr ? __ldg(p.temperature + row) : 1.f;
  const int k = p.top_k != nullptr ? __ldg(p.top_k + row) : 0;
  const float top_p = p.top_p != nullptr ? __ldg(p.top_p + row) : 1.f;
  const float min_p = p.min_p != nullptr ? __ldg(p.min_p + row) : 0.f;
  const bool by_k = k > 0 && k < r.n, by_p = top_p < 1.f, by_m = min_p > 0.f;
  const bool greedy = !(T > 0x1p-100f) || k == 1 || top_p <= 0.f;
  const bool free_draw = !greedy && !by_k && !by_p && !by_m;

  // ---- the row's maximum and its id, and whether it holds NaN
  Key top = 0;
  bool bad = false;
  Best best;
  const float inv_t = __fdiv_rn(1.f, T);
  if (free_draw) {
    // nothing is cut off: the draw needs no maximum (scores are compared, whatever is subtracted from all)
    const float* e = r.e;
    const bool wide = ((reinterpret_cast<uintptr_t>(e + r.head)) & 15) == 0;
    auto take = [&](float x, float ex, int id) {
      const Key kx = key_of(x, (uint32_t)id);
      top = kx > top ? kx : top;
      bad |= x != x;
      if (ex > 0.f && x > -INFINITY) best.take(x * inv_t - ln_of(ex), id);
    };
    if (wide) {
      if (r.ends && (int)threadIdx.x < r.head) take(__ldg(r.x + threadIdx.x), __ldg(e + threadIdx.x), (int)threadIdx.x);
      const float4* xv = reinterpret_cast<const float4*>(r.x + r.head);
      const float4* ev = reinterpret_cast<const float4*>(e + r.head);
      for (int q = r.q0 + threadIdx.x; q < r.q1; q += 4 * kThreads) {
        float4 v[4], u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (q + i * kThreads < r.q1) v[i] = __ldg(xv + q + i * kThreads), u[i] = __ldg(ev + q + i * kThreads);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (q + i * kThreads < r.q1) {
            const int id = r.head + 4 * (q + i * kThreads);
            take(v[i].x, u[i].x, id);
            take(v[i].y, u[i].y, id + 1);
            take(v[i].z, u[i].z, id + 2);
            take(v[i].w, u[i].w, id + 3);
          }
      }
      const int id = r.head + 4 * r.quads + (int)threadIdx.x;
      if (r.ends && id < r.n) take(__ldg(r.x + id), __ldg(e + id), id);
    } else {
      for_each(r, [&](float x, int id) { take(x, __ldg(e + id), id); });
    }
  } else {
    for_each(r, [&](float x, int id) {
      const Key kx = key_of(x, (uint32_t)id);
      top = kx > top ? kx : top;
      bad |= x != x;
    });
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Key u = __shfl_xor_sync(0xffffffffu, top, o);
    top = u > top ? u : top;
  }
  if ((threadIdx.x & 31) == 0) sh.part_key[threadIdx.x >> 5] = top;
  bad = __syncthreads_or(bad);
  for (int w = 0; w < kWarps; ++w) top = sh.part_key[w] > top ? sh.part_key[w] : top;
  if (ranks > 1) {
    if (threadIdx.x == 0) sh.rank_key = top, sh.rank_bad = bad;
    cl.sync();
    for (int i = 0; i < ranks; ++i) {
      const Shared* o = cl.map_shared_rank(&sh, i);
      top = o->rank_key > top ? o->rank_key : top;
      bad |= o->rank_bad != 0;
    }
  }
  r.max = unordered((uint32_t)(top >> 32));
  if (bad || r.max == -INFINITY || greedy || r.max == INFINITY) {
    if (rank == 0 && threadIdx.x == 0) p.ids[row] = bad || r.max == -INFINITY ? -1 : (int64_t)id_of(top);
    if (ranks > 1) cl.sync();  // no rank leaves while another reads its shared memory
    return;
  }
  r.scale = __fmul_rn(1.4426950408889634f, inv_t);

  // ---- the borders of top-k and top-p
  Border border{0, 0, 0};
  if (by_k || by_p) {
    clear(sh);
    __syncthreads();
    uint32_t far_count = 0, far_mass = 0;  // the last bucket takes most of a sharp row: in registers
    for_each(r, [&](float x, int id) {
      if (!(x > -INFINITY)) return;
      const float t = below(r, x);
      const int b = bucket_of(t);
      if (b == kBuckets - 1) {
        far_count += 1;
        far_mass += mass_of(t);  // at most 1 each
      } else {
        add(sh, b, mass_of(t));
      }
    });
    far_count = __reduce_add_sync(0xffffffffu, far_count);
    far_mass = __reduce_add_sync(0xffffffffu, far_mass);
    if ((threadIdx.x & 31) == 0 && far_count != 0) {
      atomicAdd(&sh.count[kBuckets - 1], far_count);
      const uint32_t old = atomicAdd(&sh.low[kBuckets - 1], far_mass);
      if (old + far_mass < old) atomicAdd(&sh.high[kBuckets - 1], 1u);
    }
    cl.sync();
    // the total first: a row may hold fewer finite logits than k
    uint32_t c[2], all_c;
    Key m[2], all_m;
    gather(cl, sh, ranks, c, m);
    uint32_t pc = c[0] + c[1];
    Key pm = m[0] + m[1];
    block_scan(sh, pc, pm, all_c, all_m);
    __syncthreads();
    const bool cut_k = by_k && (uint32_t)k < all_c;
    if (cut_k) {
      find_border(cl, sh, ranks, 0, 0, (uint32_t)k, 0.0);
      border = resolve(cl, r, sh, rank, ranks, 0, (uint32_t)k, 0.0, by_p ? top_p : 1.f);
    }
    if (by_p && border.listed == 0) {
      if (cut_k) {
        // the buckets again (the list and finer bins took their place)
        cl.sync();
        clear(sh);
        __syncthreads();
        for_each(r, [&](float x, int id) {
          if (key_of(x, (uint32_t)id) >= border.key) add(sh, bucket_of(below(r, x)), mass_of(below(r, x)));
        });
        cl.sync();
      }
      const double want = (double)top_p * (double)(cut_k ? border.mass : all_m);
      find_border(cl, sh, ranks, 0, 0, 0, want);
      const Border bp = resolve(cl, r, sh, rank, ranks, border.key, 0, want, 1.f);
      border.key = bp.key > border.key ? bp.key : border.key;
      border.listed = bp.listed;
    }
  }

  // ---- the draw among what is kept
  // (a maximum that is large beside T: scores without it would be coarse, or overflow)
  const bool far = free_draw && !(fabsf(r.max * inv_t) < 1024.f);
  if (far) best = Best{};
  auto score = [&](float x, float ex) { return (x - r.max) * inv_t - ln_of(ex); };
  auto kept_by_m = [&](float x) { return !by_m || weight_of(below(r, x)) >= min_p || x == r.max; };
  if (border.listed > 0) {
    if (rank == 0) {
      for (int i = threadIdx.x; i < border.listed; i += kThreads) {
        const float x = unordered((uint32_t)(sh.list[i] >> 32));
        const int id = (int)id_of(sh.list[i]);
        if (kept_by_m(x)) {
          const float ex = __ldg(r.e + id);
          if (ex > 0.f) best.take(score(x, ex), id);
        }
      }
    }
  } else if (!free_draw || far) {
    for_each(r, [&](float x, int id) {
      if (x > -INFINITY && key_of(x, (uint32_t)id) >= border.key && kept_by_m(x)) {
        const float ex = __ldg(r.e + id);
        if (ex > 0.f) best.take(score(x, ex), id);
      }
    });
  }
  const bool join = ranks > 1 && border.listed == 0;
  float most = block_max(sh, best.s0);
  if (join) {
    if (threadIdx.x == 0) sh.rank_best = most;
    cl.sync();
    for (int i = 0; i < ranks; ++i) most = fmaxf(most, cl.map_shared_rank(&sh, i)->rank_best);
  }
  // candidates near the best, again in 64 bits.  A float32 score is off by its logarithm's 2^-21 or so of |ln e| (< 100) at the
  // worst, the difference's and the product's roundings: a few 2^-24 of |x / T|.
  const float margin = 2e-4f + 0x1p-21f * fabsf(most) + (free_draw && !far ? 0x1p-21f * fabsf(r.max * inv_t) : 0.f);
  Draw d{0.0, -1};
  auto again = [&](float s, int id) {
    if (id >= 0 && s >= most - margin)
      d = better(d, Draw{((double)__ldg(r.x + id) - (double)r.max) / (double)T - log((double)__ldg(r.e + id)), id});
  };
  again(best.s0, best.i0);
  again(best.s1, best.i1);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Draw u;
    u.s = __shfl_xor_sync(0xffffffffu, d.s, o);
    u.id = __shfl_xor_sync(0xffffffffu, d.id, o);
    d = better(d, u);
  }
  if ((threadIdx.x & 31) == 0) sh.part_draw[threadIdx.x >> 5] = d;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWarps; ++w) d = better(d, sh.part_draw[w]);
    sh.rank_draw = d;
  }
  if (ranks > 1) cl.sync();
  if (rank == 0 && threadIdx.x == 0) {
    if (join)
      for (int i = 1; i < ranks; ++i) d = better(d, cl.map_shared_rank(&sh, i)->rank_draw);
    p.ids[row] = d.id >= 0 ? (int64_t)d.id : (int64_t)id_of(top);
  }
  if (ranks > 1) cl.sync();
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, int64_t rows, const DeviceInfo& dev, cudaStream_t stream) {
  SampleParams p;
  p.logits = a.logits;
  p.noise = a.noise;
  p.stride = a.stride;
  p.noise_stride = a.noise_stride;
  p.vocab = (int)a.vocab;
  p.temperature = a.temperature;
  p.top_k = a.top_k;
  p.top_p = a.top_p;
  p.min_p = a.min_p;
  p.ids = a.ids;
  // as many CTAs a row as keep the SMs at work, with 4096 logits each at least
  int ranks = 1;
  while (ranks < kMaxRanks && rows * ranks * 2 <= 2 * (int64_t)dev.sm_count && a.vocab / (2 * ranks) >= 4096) ranks *= 2;
  if (rows * ranks > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(rows * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel, p, ranks);
}

}  // namespace qmv
