// sample.cu -- the next ids from rows of logits: temperature, top-k, top-p and min-p, with given random numbers.
//
//   w_j = e^((x_j - max) / T),  id = the kept j with the largest (x_j - max) / T - ln e_j.
//
// With e_j exponential random numbers that is a draw from the kept w (of independent exponential clocks of rates w_j
// the first to ring is j with probability w_j over their sum), so no sum over the kept ids in an order of theirs is
// needed: the parts of a row join by a maximum, whose result does not depend on how the row is cut.
//
// The cuts are prefixes of the descending order (larger logits first, equal ones by the lower id), so each is one
// border.  One pass over the row leaves the maxima of its chunks of 128 logits (and the sum of the w, where top-p stands alone).
// k chunks whose maxima reach a value hold k logits that do, and the w of chunk maxima sum to no more than those of all logits: so
// the maxima alone give a value that the kept logits reach.  The few chunks that hold such logits are read again (from L2) and
// those logits collected, sorted by keys (value, id; no two equal) and walked.  Where they are too many (flat rows), a second pass adds
// count and weight of 1024 buckets of (max - x) / T in shared memory (integers, so the order of the atomics does not matter),
// and only the bucket that holds the border is collected, after cutting it again by its keys' bits where it holds too many.
//
// Scores are float32; those close to the best are formed again in 64 bits, so equal draws are told apart as the definition does.
// A row is one cluster's: 1, 2, 4 or 8 CTAs, which join in distributed shared memory; no workspace.
//
// Bound by the logits' bytes for many unfiltered rows (and the noise's, which only they read whole); else by a chain of passes, joins and a
// sort for few rows, and by instructions and shared-memory atomics for flat rows under top-p.  GB300, rows of 151936: one row with all cuts
// 18.0 us (17.1 without min-p's logarithm in 64 bits); 64 rows greedy 13, unfiltered 18, min-p 36, top-k 51, top-p 84, mixed 71 us; 512
// rows unfiltered 105 us (5.9 TB/s), greedy 59, all cuts 139, top-p 353 us.  (With conversions for the buckets, branches for what a draw takes and a binary search of borders: one
// row 18, 64 mixed rows 81 us.)
#include <cooperative_groups.h>

#include <cfloat>

#include "qmv_common.cuh"
#include "qmv_internal.h"

namespace qmv {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBuckets = 1024;  // two a thread
constexpr int kList = 2048;     // keys that are collected and sorted
constexpr int kChunks = 2048;   // of a row at most
constexpr int kClose = 64;      // candidates of the last comparison that are listed
constexpr int kMaxRanks = 8;
constexpr int kBatch = 8;       // loads of 16 bytes that a thread has on their way
using Key = unsigned long long;

// (as in logprobs.cu) larger logits first, equal ones by the lower id; -0 counts as +0, NaN as the largest
__device__ __forceinline__ uint32_t ordered(float x) {
  uint32_t b = __float_as_uint(x + 0.0f);
  if ((b & 0x7fffffffu) > 0x7f800000u) b = 0x7fffffffu;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ Key key_of(float x, uint32_t id) { return ((Key)ordered(x) << 32) | (0xffffffffu - id); }
__device__ __forceinline__ uint32_t id_of(Key k) { return 0xffffffffu - (uint32_t)k; }
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

constexpr uint32_t kMasked = 0x007fffffu;   // ordered(-infinity)
constexpr uint32_t kInfinite = 0xff800000u; // ordered(+infinity); NaN is above

// One row as its CTA sees it: quads of 16 bytes from the row's first 16-byte boundary, q0 .. q1 - 1 the CTA's; 32 << shift
// quads are a chunk.  `ends`: this CTA also has the up to 6 values before the first and after the last whole quad, as its last chunk.
struct Row {
  const float* x;
  const float* e;
  int n;
  int head, quads, q0, q1;
  int shift, chunks;  // the CTA's chunks, without the ends
  bool ends;
  float max, scale, floor;  // scale: log2 e / T; floor: the distance from the maximum at which a score is -1e38, or the type's lowest
};

// The id of a quad's first logit.  (Unsigned: lanes past a row's end form them, too, and in rows of nearly 2^31 ids those wrap.)
__device__ __forceinline__ int id_at(const Row& r, int q) { return (int)((uint32_t)r.head + 4u * (uint32_t)q); }

// A logit's distance below the maximum in powers of two, its bucket and its weight.
__device__ __forceinline__ float below(const Row& r, float x) { return (r.max - x) * r.scale; }
// (The nearest 32nd, by an addition that leaves it in the lowest bits: conversions have a quarter of the rate.)
__device__ __forceinline__ int bucket_of(float t) { return __float_as_int(fminf(t * 32.f, (float)(kBuckets - 1)) + 8388608.f) & (kBuckets - 1); }
static_assert((kBuckets & (kBuckets - 1)) == 0, "a mask");
__device__ __forceinline__ float exp2_of(float t) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(t));
  return y;
}
// The weight as an integer in units of 2^-31: sums of them are exact, so no order of adding matters.  An id counts
// to 2^-32 of the largest.
__device__ __forceinline__ uint32_t mass_of(float t) { return t > 0.f ? __float2uint_rn(exp2_of(-t) * 0x1p31f) : 0x80000000u; }

// f(x, id, local chunk) for the logits of the CTA's chunks whose maximum reaches `least` (mapped; 0: of all).  Whole warps
// take part: f may use neither shuffles nor barriers.
template <typename F>
__device__ __forceinline__ void for_each(const Row& r, const uint32_t* chunk_max, uint32_t least, F f) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const float4* xv = reinterpret_cast<const float4*>(r.x + r.head);
  const int subs = (r.q1 - r.q0 + 31) / 32;
  for (int s = wid; s < subs; s += 4 * kWarps) {
    float4 v[4];
    bool in[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int sub = s + i * kWarps, q = r.q0 + 32 * sub + lane;
      in[i] = q < r.q1 && (least == 0 || chunk_max[sub >> r.shift] >= least);
      if (in[i]) v[i] = __ldg(xv + q);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (in[i]) {
        const int sub = s + i * kWarps, id = r.head + 4 * (r.q0 + 32 * sub + lane);
        f(v[i].x, id, sub >> r.shift);
        f(v[i].y, id + 1, sub >> r.shift);
        f(v[i].z, id + 2, sub >> r.shift);
        f(v[i].w, id + 3, sub >> r.shift);
      }
  }
  const int tail = r.n - r.head - 4 * r.quads;
  if (r.ends && (int)threadIdx.x < r.head + tail) {
    const int id = (int)threadIdx.x < r.head ? (int)threadIdx.x : (int)threadIdx.x - r.head + r.n - tail;
    f(__ldg(r.x + id), id, r.chunks);
  }
}

struct Draw {  // a candidate's score in 64 bits; the larger wins, then the lower id
  double s;
  int id;
};
__device__ __forceinline__ Draw better(Draw a, Draw b) {
  if (b.id < 0) return a;
  if (a.id < 0 || b.s > a.s || (b.s == a.s && b.id < a.id)) return b;
  return a;
}
__device__ __forceinline__ float log2_of(float e) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(e));
  return y;
}
__device__ __forceinline__ float log2_of_normal(float e) {  // (-infinity for subnormal numbers)
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(e));
  return y;
}
// x's score in powers of two below the maximum's, with the random number e; -infinity where e is not one (not above 0, infinite, NaN).
// Any other score stays finite, however far x lies below at a low temperature: those at the floor (-1e38) are told apart in 64 bits.
__device__ __forceinline__ float score_of(const Row& r, float x, float e) {
  const float t = e >= 0x1p-126f ? log2_of_normal(e) : e > 0.f ? log2_of(e) : INFINITY;
  return fmaf(fmaxf(x - r.max, r.floor), r.scale, -t);
}

struct Shared {
  uint32_t count[kBuckets], low[kBuckets], high[kBuckets];
  Key list[kList];
  uint32_t chunk[kChunks + 1];  // the maxima of the CTA's chunks, mapped
  uint32_t listed, close;
  int close_id[kClose];
  // each rank's part of what is joined
  uint32_t rank_max;
  Key rank_sum;
  float rank_best;
  Draw rank_draw;
  int rank_id;
  // what rank 0 or every rank found
  uint32_t reaching;  // rank 0's: chunks whose maxima reach min-p's value
  uint32_t edge_m;    // the least mapped logit that min-p keeps
  float reach;  // what the chunks' maxima tell: every kept logit reaches it (NaN: they do not tell)
  int bucket;
  uint32_t above_count, in_count;
  Key above_mass;
  Key border;
  Key border_mass;
  int kept;
  Key scan_mass[kWarps];
  uint32_t scan_count[kWarps];
  float part[kWarps];
  Draw part_draw[kWarps];
  __device__ __forceinline__ float* best() { return reinterpret_cast<float*>(count); }  // a chunk's best score, once the buckets have done
};
static_assert(sizeof(float) * (kChunks + 1) <= 3 * sizeof(uint32_t) * kBuckets, "the buckets' room holds the chunks' best scores");

__device__ __forceinline__ float block_max(Shared& sh, float v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if (lane == 0) sh.part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sh.part[lane % kWarps];
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
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
  // the warps' totals, scanned by every warp for itself
  uint32_t wc = sh.scan_count[lane % kWarps];
  Key wm = sh.scan_mass[lane % kWarps];
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const uint32_t uc = __shfl_up_sync(0xffffffffu, wc, o, kWarps);
    const Key um = __shfl_up_sync(0xffffffffu, wm, o, kWarps);
    if (lane % kWarps >= o) wc += uc, wm += um;
  }
  all_c = __shfl_sync(0xffffffffu, wc, kWarps - 1);
  all_m = __shfl_sync(0xffffffffu, wm, kWarps - 1);
  const uint32_t bc = __shfl_sync(0xffffffffu, wc, (wid + 31) & 31);
  const Key bm = __shfl_sync(0xffffffffu, wm, (wid + 31) & 31);
  c += (wid > 0 ? bc : 0u) - c0;
  m += (wid > 0 ? bm : 0ull) - m0;
}

__device__ __forceinline__ void add(Shared& sh, int b, uint32_t mass) {
  atomicAdd(&sh.count[b], 1u);
  const uint32_t old = atomicAdd(&sh.low[b], mass);
  if (old + mass < old) atomicAdd(&sh.high[b], 1u);
}

__device__ __forceinline__ void clear(Shared& sh) {
  for (int i = threadIdx.x; i < kBuckets; i += kThreads) sh.count[i] = sh.low[i] = sh.high[i] = 0u;
}

// A thread's two buckets over all ranks.
__device__ void gather(cg::cluster_group& cl, Shared& sh, int ranks, uint32_t (&c)[2], Key (&m)[2]) {
  c[0] = c[1] = 0;
  m[0] = m[1] = 0;
#pragma unroll 4
  for (int r = 0; r < ranks; ++r) {
    const Shared* o = ranks == 1 ? &sh : cl.map_shared_rank(&sh, r);
    const uint2 n = reinterpret_cast<const uint2*>(o->count)[threadIdx.x], l = reinterpret_cast<const uint2*>(o->low)[threadIdx.x],
                h = reinterpret_cast<const uint2*>(o->high)[threadIdx.x];
    c[0] += n.x, c[1] += n.y;
    m[0] += ((Key)h.x << 32) + l.x, m[1] += ((Key)h.y << 32) + l.y;
  }
}

// Which bucket (or bin) holds the border: the first at which the count reaches `want_count`, or (want_count 0) the last whose
// exclusive mass is below `want_mass`.  c, m: a thread's two buckets.  Leaves it, what lies above it and what it holds in sh.  False
// where all buckets together do not reach the border.
__device__ bool find_border(Shared& sh, const uint32_t (&c)[2], const Key (&m)[2], uint32_t base_count, Key base_mass, uint32_t want_count,
                            double want_mass) {
  uint32_t all_c, pc = c[0] + c[1];
  Key all_m, pm = m[0] + m[1];
  block_scan(sh, pc, pm, all_c, all_m);
  pc += base_count;
  pm += base_mass;
  const bool found = want_count != 0 ? base_count + all_c >= want_count : (double)(base_mass + all_m) >= want_mass;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const bool here = want_count != 0 ? pc < want_count && pc + c[k] >= want_count
                                      : m[k] != 0 && (double)pm < want_mass && (double)(pm + m[k]) >= want_mass;
    if (here) {
      sh.bucket = 2 * threadIdx.x + k;
      sh.above_count = pc;
      sh.above_mass = pm;
      sh.in_count = c[k];
    }
    pc += c[k];
    pm += m[k];
  }
  __syncthreads();
  return found;
}

// The smallest mapped logit of lo .. hi that `holds`, which hi does and every logit above one that does.  (32 values at a time, one a
// lane; whole warps.)
template <typename F>
__device__ __forceinline__ uint32_t least_of(uint32_t lo, uint32_t hi, F holds) {
  const uint32_t lane = threadIdx.x & 31;
#pragma unroll 1
  while (lo < hi) {
    const uint32_t step = max((hi - lo) / 32, 1u), far = min(lane * step, hi - lo);
    const uint32_t which = __ballot_sync(0xffffffffu, holds(unordered(lo + far)));
    const uint32_t first = which != 0 ? __ffs(which) - 1 : 32;  // the first lane whose value holds
    if (first == 0) return lo;
    const uint32_t from = lo;
    lo = from + min((first - 1) * step, hi - from) + 1;
    if (first < 32) hi = from + min(first * step, hi - from);
  }
  return lo;
}
// ... whose bucket is at most b.
__device__ __forceinline__ uint32_t edge_of(const Row& r, int b) {
  return least_of(kMasked + 1, ordered(r.max), [&](float x) { return bucket_of(below(r, x)) <= b; });
}

// ... whose weight is min_p at least: x - max >= T ln min_p in 64 bits, so that how small min_p is costs no accuracy; looked for as far around
// float32's answer as that may be off.
__device__ __forceinline__ uint32_t edge_of_weight(const Row& r, float T, float min_p) {
  const double least = (double)T * log((double)min_p);
  const float z = T * logf(min_p), about = r.max + z, off = 0x1p-20f * fabsf(z) + 0x1p-21f * fabsf(r.max) + 0x1p-149f;
  const uint32_t top = ordered(r.max);
  return least_of(max(ordered(about - off), kMasked + 1), min(ordered(about + off), top),
                  [&](float x) { return (double)x - (double)r.max >= least; });
}

// The collected keys in descending order.
__device__ void sort_list(Shared& sh, int n) {
  if (n <= kThreads) {
    // a key's place is how many are larger (no two are equal): a few hundred comparisons, and two barriers
    const bool in = (int)threadIdx.x < n;
    const Key mine = in ? sh.list[threadIdx.x] : 0;
    int place = 0;
    if ((int)(threadIdx.x & ~31u) < n) {
#pragma unroll 8
      for (int i = 0; i < n; ++i) place += sh.list[i] > mine;
    }
    __syncthreads();
    if (in) sh.list[place] = mine;
    __syncthreads();
    return;
  }
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
  Key key;     // kept: keys of at least this
  Key mass;    // the kept keys' weight
  int listed;  // > 0: the first `listed` of rank 0's sorted list are all that is kept
};

// A warp's logits x[0 .. N - 1] of ids id, id + 1 .. a lane that `takes` go to rank 0's list: one addition to its length for all.
template <int N, typename F>
__device__ __forceinline__ void list_keys(Shared* home, const float (&x)[N], int id, F takes) {
  const int lane = threadIdx.x & 31;
  uint32_t in[N], total = 0;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    in[k] = __ballot_sync(0xffffffffu, takes(x[k], id + k));
    total += __popc(in[k]);
  }
  if (total == 0) return;
  uint32_t at = 0;
  if (lane == 0) at = atomicAdd(&home->listed, total);
  at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const uint32_t mine = at + __popc(in[k] & ((1u << lane) - 1u));
    if ((in[k] >> lane & 1u) && mine < (uint32_t)kList) home->list[mine] = key_of(x[k], (uint32_t)(id + k));
    at += __popc(in[k]);
  }
}

// Keys of lo .. hi go to rank 0's list, in no order.  Returns how many there are (the list holds the first kList).
__device__ uint32_t collect(cg::cluster_group& cl, const Row& r, Shared& sh, Shared* home, Key lo, Key hi) {
  const uint32_t least = (uint32_t)(lo >> 32);
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const float4* xv = reinterpret_cast<const float4*>(r.x + r.head);
  const int subs = (r.q1 - r.q0 + 31) / 32;
#pragma unroll 1
  for (int sub = wid; sub < subs; sub += kWarps) {
    if (sh.chunk[sub >> r.shift] < least) continue;  // (most of them)
    const int q = r.q0 + 32 * sub + lane, id = r.head + 4 * q;
    float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (q < r.q1) v = __ldg(xv + q);
    const float x[4] = {v.x, v.y, v.z, v.w};
    list_keys<4>(home, x, id, [&](float y, int j) {
      const Key k = key_of(y, (uint32_t)j);
      return y > -INFINITY && k >= lo && k <= hi;
    });
  }
  if (r.ends && wid == 0) {
    const int tail = r.n - r.head - 4 * r.quads;
    const int id = lane < r.head ? lane : lane - r.head + r.n - tail;
    const float x[1] = {lane < r.head + tail ? __ldg(r.x + id) : -INFINITY};
    list_keys<1>(home, x, id, [&](float y, int j) {
      const Key k = key_of(y, (uint32_t)j);
      return y > -INFINITY && k >= lo && k <= hi;
    });
  }
  cl.sync();
  return home->listed;
}

// Rank 0's list, sorted and cut: the first `count` of it (all of it for 0), of those the part whose exclusive mass, over
// above_mass, is below want_mass, of those the part whose exclusive mass is below top_p of what is left.  weigh: the kept keys'
// mass is wanted.
__device__ void cut_list(const Row& r, Shared& sh, uint32_t listed, uint32_t count, Key above_mass, double want_mass, float top_p, bool weigh) {
  const int n = (int)listed;
  sort_list(sh, n);
  Key mass = 0;
  int stay = count != 0 ? min(n, (int)count) : n;
  if (weigh || top_p < 1.f || want_mass < INFINITY) stay = prefix_by_mass(r, sh, stay, above_mass, want_mass, mass);
  if (top_p < 1.f) stay = prefix_by_mass(r, sh, stay, 0, (double)top_p * (double)mass, mass);
  if (threadIdx.x == 0) {
    sh.kept = stay;
    sh.border = stay > 0 ? sh.list[stay - 1] : ~(Key)0;
    sh.border_mass = mass;
  }
}

// The border in the bucket that find_border left in sh, among keys of at least `floor`.  want_count: that many stay; else those of exclusive
// mass below want_mass.  more_p < 1, where the list holds everything kept: the top-p cut is made in it, too.
__device__ Border resolve(cg::cluster_group& cl, const Row& r, Shared& sh, Shared* home, int rank, int ranks, Key floor, uint32_t want_count,
                          double want_mass, float more_p) {
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
    for_each(r, sh.chunk, (uint32_t)(lo >> 32), [&](float x, int id, int) {
      const Key k = key_of(x, (uint32_t)id);
      if (k >= lo && k <= hi) add(sh, (int)((hi - k) >> shift), mass_of(below(r, x)));
    });
    cl.sync();
    uint32_t c[2];
    Key m[2];
    gather(cl, sh, ranks, c, m);
    find_border(sh, c, m, above, above_mass, want_count, want_mass);
    above = sh.above_count;
    above_mass = sh.above_mass;
    inside = sh.in_count;
    hi -= (Key)sh.bucket << shift;
    const Key low = hi - (((Key)1 << shift) - 1);
    lo = low > lo && low <= hi ? low : lo;
  }
  cl.sync();
  if (threadIdx.x == 0) sh.listed = 0u;
  cl.sync();
  const uint32_t listed = collect(cl, r, sh, home, lo, hi);
  if (rank == 0)
    cut_list(r, sh, min(listed, (uint32_t)kList), want_count != 0 ? want_count - above : 0, above_mass, want_count != 0 ? INFINITY : want_mass,
             whole ? more_p : 1.f, true);
  cl.sync();
  Border b;
  b.key = home->border;
  b.mass = home->border_mass;
  b.listed = whole ? home->kept : 0;
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

// The pass over the row: the maxima of its chunks, and with SUM each thread's largest logit and sum of 2^((x - it) scale).
template <bool SUM>
__device__ __forceinline__ uint32_t first_pass(const Row& r, Shared& sh, float& own_max, float& own_sum) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const float4* xv = reinterpret_cast<const float4*>(r.x + r.head);
  const int subs = (r.q1 - r.q0 + 31) / 32;
  uint32_t most = 0;
  float m = -INFINITY, sum[kBatch] = {};
  auto take = [&](const float (&v)[4 * kBatch], float top) {
    if (!(top > -INFINITY)) return;  // (NaN: the row is refused)
    if (top > m) {
      const float f = m > -INFINITY ? exp2_of((m - top) * r.scale) : 0.f;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) sum[i] *= f;
      m = top;
    }
#pragma unroll
    for (int i = 0; i < 4 * kBatch; ++i) sum[i % kBatch] += v[i] < m ? exp2_of((v[i] - m) * r.scale) : 1.f;
  };
  for (int s = wid; s < subs; s += kBatch * kWarps) {
    float v[4 * kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int q = r.q0 + 32 * (s + i * kWarps) + lane;
      float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (q < r.q1) f = __ldg(xv + q);
      v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
    }
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float t = max_nan(max_nan(v[4 * i], v[4 * i + 1]), max_nan(v[4 * i + 2], v[4 * i + 3]));
      if (SUM) top = fmaxf(top, t);
      const uint32_t o = __reduce_max_sync(0xffffffffu, ordered(t));
      most = max(most, o);
      if (lane == 0 && s + i * kWarps < subs) {
        uint32_t* at = &sh.chunk[(s + i * kWarps) >> r.shift];
        if (r.shift == 0)
          *at = o;
        else
          atomicMax(at, o);
      }
    }
    if (SUM) take(v, top);
  }
  if (r.ends) {
    const int tail = r.n - r.head - 4 * r.quads;
    float v[4 * kBatch];
#pragma unroll
    for (int i = 0; i < 4 * kBatch; ++i) v[i] = -INFINITY;
    if (wid == 0) {
      if (lane < r.head + tail) v[0] = __ldg(r.x + (lane < r.head ? lane : lane - r.head + r.n - tail));
      const uint32_t o = __reduce_max_sync(0xffffffffu, ordered(v[0]));
      most = max(most, o);
      if (lane == 0) sh.chunk[r.chunks] = o;
      if (SUM) take(v, v[0]);
    }
  }
  if (SUM) {
    own_max = m;
    own_sum = ((sum[0] + sum[1]) + (sum[2] + sum[3])) + ((sum[4] + sum[5]) + (sum[6] + sum[7]));
    static_assert(kBatch == 8, "eight chains");
  }
  return most;
}

// Count or weight of the row's logits in the buckets.
template <bool MASS>
__device__ __forceinline__ void bucket_pass(const Row& r, Shared& sh) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const float4* xv = reinterpret_cast<const float4*>(r.x + r.head);
  const int subs = (r.q1 - r.q0 + 31) / 32;
  uint32_t far = 0;  // the last bucket takes most of a sharp row: in a register (a weight of at most 1 each)
  auto put = [&](const float (&v)[8]) {
    int b[8];
    uint32_t m[8], old[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = below(r, v[i]);
      b[i] = v[i] > -INFINITY ? bucket_of(t) : kBuckets;
      m[i] = MASS ? mass_of(t) : 1u;
      if (b[i] == kBuckets - 1) far += m[i];
    }
    // the additions first, what they carry after: none waits for another
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      old[i] = 0;
      if (b[i] < kBuckets - 1) old[i] = atomicAdd(MASS ? &sh.low[b[i]] : &sh.count[b[i]], m[i]);
    }
    if (MASS) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (b[i] < kBuckets - 1 && old[i] + m[i] < old[i]) atomicAdd(&sh.high[b[i]], 1u);
    }
  };
  for (int s = wid; s < subs; s += 4 * kWarps) {
    float v[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = r.q0 + 32 * (s + i * kWarps) + lane;
      float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (q < r.q1) f = __ldg(xv + q);
      v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float(&half)[8] = *reinterpret_cast<const float(*)[8]>(v + 8 * h);
      put(half);
    }
  }
  if (r.ends && wid == 0) {
    const int tail = r.n - r.head - 4 * r.quads;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = -INFINITY;
    if (lane < r.head + tail) v[0] = __ldg(r.x + (lane < r.head ? lane : lane - r.head + r.n - tail));
    put(v);
  }
  far = __reduce_add_sync(0xffffffffu, far);
  if (lane == 0 && far != 0) {
    const uint32_t old = atomicAdd(MASS ? &sh.low[kBuckets - 1] : &sh.count[kBuckets - 1], far);
    if (MASS && old + far < old) atomicAdd(&sh.high[kBuckets - 1], 1u);
  }
}

__device__ __forceinline__ int mapped(float v) {  // an integer that orders as the float does
  return v >= 0.f ? __float_as_int(v) : __float_as_int(v) ^ 0x7fffffff;
}

// The draw over the chunks whose maximum reaches `least`: kind(x, id) is 1 for a logit that takes part, 2 for one that goes to rank 0's
// list (where the pass `collects`), else 0.  Leaves each chunk's best score; returns the thread's.
template <typename K, typename S>
__device__ __forceinline__ float draw_pass(const Row& r, Shared& sh, Shared* home, uint32_t least, bool collects, K kind, S score) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const float4* xv = reinterpret_cast<const float4*>(r.x + r.head);
  const bool wide = ((reinterpret_cast<uintptr_t>(r.e + r.head)) & 15) == 0;
  const int subs = (r.q1 - r.q0 + 31) / 32;
  int* best = reinterpret_cast<int*>(sh.best());
  float most = -INFINITY;
  constexpr int B = 3;
  for (int s = wid; s < subs; s += B * kWarps) {
    float v[4 * B], e[4 * B];
    int part[B];  // two bits a logit
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int sub = s + i * kWarps, q = r.q0 + 32 * sub + lane;
      float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY), u = make_float4(0.f, 0.f, 0.f, 0.f);
      if (q < r.q1 && sh.chunk[sub >> r.shift] >= least) {
        // the random numbers at once: they come from memory, and chunks that get here hold kept logits
        const int id = r.head + 4 * q;
        f = __ldg(xv + q);
        if (wide)
          u = __ldg(reinterpret_cast<const float4*>(r.e + id));
        else
          u = make_float4(__ldg(r.e + id), __ldg(r.e + id + 1), __ldg(r.e + id + 2), __ldg(r.e + id + 3));
      }
      v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
      e[4 * i] = u.x, e[4 * i + 1] = u.y, e[4 * i + 2] = u.z, e[4 * i + 3] = u.w;
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int id = id_at(r, r.q0 + 32 * (s + i * kWarps) + lane);
      part[i] = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (v[4 * i + k] > -INFINITY) part[i] |= kind(v[4 * i + k], id + k) << (2 * k);
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int sub = s + i * kWarps, id = id_at(r, r.q0 + 32 * sub + lane);
      float t = -INFINITY;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int what = part[i] >> (2 * k) & 3;
        if (what == 1) t = fmaxf(t, score(v[4 * i + k], e[4 * i + k]));
      }
      if (collects) {
        const float x[4] = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
        list_keys<4>(home, x, id, [&](float, int j) { return (part[i] >> (2 * (j - id)) & 3) == 2; });
      }
      t = unordered(__reduce_max_sync(0xffffffffu, ordered(t)));
      most = fmaxf(most, t);
      if (lane == 0 && sub < subs) {
        if (r.shift == 0)
          best[sub] = mapped(t);
        else
          atomicMax(best + (sub >> r.shift), mapped(t));
      }
    }
  }
  if (r.ends && wid == 0) {
    const int tail = r.n - r.head - 4 * r.quads;
    float t = -INFINITY;
    if (lane < r.head + tail) {
      const int id = lane < r.head ? lane : lane - r.head + r.n - tail;
      const float x = __ldg(r.x + id);
      const int what = x > -INFINITY ? kind(x, id) : 0;
      if (what == 1) t = score(x, __ldg(r.e + id));
      if (what == 2) {
        const uint32_t at = atomicAdd(&home->listed, 1u);
        if (at < (uint32_t)kList) home->list[at] = key_of(x, (uint32_t)id);
      }
    }
    t = unordered(__reduce_max_sync(0xffffffffu, ordered(t)));
    most = fmaxf(most, t);
    if (lane == 0) best[r.chunks] = mapped(t);
  }
  return most;
}

// The pass of a draw from the whole row: each chunk's best score (in powers of two, nothing subtracted), and whether the row holds NaN or
// +infinity (whose score is NaN, and lost, where the random number is infinite, negative or NaN).
// A random number that is not above 0, subnormal ones among them, makes a score that is infinite or NaN: the caller looks again.
__device__ __forceinline__ bool free_pass(const Row& r, Shared& sh, float& most) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const float4* xv = reinterpret_cast<const float4*>(r.x + r.head);
  const float4* ev = reinterpret_cast<const float4*>(r.e + r.head);
  const int subs = (r.q1 - r.q0 + 31) / 32;
  int* best = reinterpret_cast<int*>(sh.best());
  float high = 0.f;
  most = -INFINITY;
  auto score = [&](float x, float e) {
    high = max_nan(high, x);
    return fmaf(x, r.scale, -log2_of_normal(e));
  };
  for (int s = wid; s < subs; s += 4 * kWarps) {
    float4 v[4], u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = r.q0 + 32 * (s + i * kWarps) + lane;
      v[i] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      u[i] = make_float4(1.f, 1.f, 1.f, 1.f);
      if (q < r.q1) v[i] = __ldg(xv + q), u[i] = __ldg(ev + q);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float t = fmaxf(fmaxf(score(v[i].x, u[i].x), score(v[i].y, u[i].y)), fmaxf(score(v[i].z, u[i].z), score(v[i].w, u[i].w)));
      const float o = unordered(__reduce_max_sync(0xffffffffu, ordered(t)));
      most = max_nan(most, o);
      if (lane == 0 && s + i * kWarps < subs) {
        if (r.shift == 0)
          best[s + i * kWarps] = mapped(o);
        else
          atomicMax(best + ((s + i * kWarps) >> r.shift), mapped(o));
      }
    }
  }
  if (r.ends && wid == 0) {
    const int tail = r.n - r.head - 4 * r.quads;
    float t = -INFINITY;
    if (lane < r.head + tail) {
      const int id = lane < r.head ? lane : lane - r.head + r.n - tail;
      t = score(__ldg(r.x + id), __ldg(r.e + id));
    }
    const float o = unordered(__reduce_max_sync(0xffffffffu, ordered(t)));
    most = max_nan(most, o);
    if (lane == 0) best[r.chunks] = mapped(o);
  }
  return !(high < INFINITY);
}

__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleParams p, int ranks) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ Shared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int rank = ranks == 1 ? 0 : (int)cl.block_rank();
  Shared* home = ranks == 1 ? &sh : cl.map_shared_rank(&sh, 0);
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
  r.shift = 0;
  while (((long long)r.quads >> (5 + r.shift)) + kMaxRanks > kChunks) ++r.shift;
  r.chunks = (((r.q1 - r.q0 + 31) / 32) + (1 << r.shift) - 1) >> r.shift;

  const float asked = p.temperature != nullptr ? __ldg(p.temperature + row) : 1.f;
  const float T = asked > 0x1p100f ? 0x1p100f : asked;
  const int k = p.top_k != nullptr ? __ldg(p.top_k + row) : 0;
  const float top_p = p.top_p != nullptr ? __ldg(p.top_p + row) : 1.f;
  const float min_p = p.min_p != nullptr ? __ldg(p.min_p + row) : 0.f;
  const bool by_k = k > 0 && k < r.n, by_p = top_p < 1.f, by_m = min_p > 0.f;
  const bool greedy = !(T > 0x1p-100f) || k == 1 || top_p <= 0.f;
  const bool whole_row = !greedy && !by_k && !by_p && !by_m;
  const float inv_t = __fdiv_rn(1.f, T);
  r.scale = __fmul_rn(1.4426950408889634f, inv_t);
  r.floor = fmaxf(__fdiv_rn(-1e38f, r.scale), -FLT_MAX);
  r.max = 0.f;
  // a score is float32: its logarithm is off by 2^-21 of |log2 e| (< 150) at most, the difference, product and sum by a few 2^-24
  // of their own size; candidates as close to the best as that are looked at again
  auto margin_of = [&](float most, float size) { return 4e-4f + 0x1p-20f * (fabsf(most) + size); };

  // each CTA's part of the row is joined by what: a maximum of mapped values
  auto over_ranks = [&](uint32_t v) {
    v = __reduce_max_sync(0xffffffffu, v);
    __syncthreads();
    if (lane == 0) sh.scan_count[wid] = v;
    __syncthreads();
    v = __reduce_max_sync(0xffffffffu, sh.scan_count[lane % kWarps]);
    if (ranks > 1) {
      if (threadIdx.x == 0) sh.rank_max = v;
      cl.sync();
      v = __reduce_max_sync(0xffffffffu, cl.map_shared_rank(&sh, lane % ranks)->rank_max);  // (a lane a rank)
    }
    return v;
  };
  // the comparison in 64 bits of the logits that visit(least, f) hands to f: those whose score reaches most - margin; writes the
  // row's id.  all_ranks: every rank calls it (else rank 0 alone)
  auto decide = [&](float most, float margin, auto visit, auto score, bool all_ranks) {
    auto meet = [&]() {
      if (all_ranks)
        cl.sync();
      else
        __syncthreads();
    };
    if (rank == 0 && threadIdx.x == 0) sh.close = 0u;
    meet();
    const float least = most - margin;
    visit(least, [&](float x, float e, int id) {
      if (score(x, e) >= least) {
        const uint32_t at = atomicAdd(&home->close, 1u);
        if (at < (uint32_t)kClose) home->close_id[at] = id;
      }
    });
    meet();
    const uint32_t n = home->close;
    if (n == 1) {
      if (rank == 0 && threadIdx.x == 0) p.ids[row] = sh.close_id[0];
      return;
    }
    auto exact = [&](float x, float e, int id) { return Draw{((double)x - (double)r.max) / (double)T - log((double)e), id}; };
    Draw d{0.0, -1};
    if (n > (uint32_t)kClose) {
      visit(least, [&](float x, float e, int id) {
        if (score(x, e) >= least) d = better(d, exact(x, e, id));
      });
    } else if (rank == 0 && threadIdx.x < n) {
      const int id = sh.close_id[threadIdx.x];
      d = exact(__ldg(r.x + id), __ldg(r.e + id), id);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      Draw u;
      u.s = __shfl_xor_sync(0xffffffffu, d.s, o);
      u.id = __shfl_xor_sync(0xffffffffu, d.id, o);
      d = better(d, u);
    }
    if (lane == 0) sh.part_draw[wid] = d;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kWarps; ++w) d = better(d, sh.part_draw[w]);
      sh.rank_draw = d;
    }
    meet();
    if (rank == 0 && threadIdx.x == 0) {
      if (all_ranks)
        for (int i = 1; i < ranks; ++i) d = better(d, cl.map_shared_rank(&sh, i)->rank_draw);
      p.ids[row] = d.id;
    }
  };
  // f(x, e, id) for the logits of chunks whose best score reaches `least`
  auto chunks_reaching = [&](float least, auto f) {
    const int* best = reinterpret_cast<const int*>(sh.best());
    const int reach = mapped(least);
    for (int c = wid; c < r.chunks + r.ends; c += kWarps) {
      if (best[c] < reach) continue;
      if (c == r.chunks) {
        const int tail = r.n - r.head - 4 * r.quads;
        if (lane < r.head + tail) {
          const int id = lane < r.head ? lane : lane - r.head + r.n - tail;
          f(__ldg(r.x + id), __ldg(r.e + id), id);
        }
        continue;
      }
      for (int j = 0; j < 1 << r.shift; ++j) {
        const int q = r.q0 + 32 * ((c << r.shift) + j) + lane;
        if (q >= r.q1) break;
        const int id = r.head + 4 * q;
        for (int i = 0; i < 4; ++i) f(__ldg(r.x + id + i), __ldg(r.e + id + i), id + i);
      }
    }
  };
  // the lowest id of the largest logit, `top` mapped; every rank calls it
  auto largest = [&](uint32_t top) {
    int id = INT32_MAX;
    __syncthreads();
    if (top <= kInfinite && top > kMasked)
      for_each(r, sh.chunk, top, [&](float x, int i, int) {
        if (ordered(x) == top) id = min(id, i);
      });
    id = __reduce_min_sync(0xffffffffu, id);
    if (lane == 0) sh.scan_count[wid] = (uint32_t)id;
    __syncthreads();
    id = __reduce_min_sync(0xffffffffu, (int)sh.scan_count[lane % kWarps]);
    if (ranks > 1) {
      if (threadIdx.x == 0) sh.rank_id = id;
      cl.sync();
      id = __reduce_min_sync(0xffffffffu, cl.map_shared_rank(&sh, lane % ranks)->rank_id);
    }
    if (rank == 0 && threadIdx.x == 0) p.ids[row] = id == INT32_MAX ? -1 : id;
  };

  if (r.shift > 0) {
    for (int i = threadIdx.x; i <= r.chunks; i += kThreads) sh.chunk[i] = 0u, reinterpret_cast<int*>(sh.best())[i] = INT32_MIN;
    __syncthreads();
  }
  // ---- a draw from the whole row: one pass over logits and random numbers, then the chunks with the best scores
  if (whole_row) {
    const bool wide = ((reinterpret_cast<uintptr_t>(r.e + r.head)) & 15) == 0;
    if (wide) {
      float most;
      const bool special = free_pass(r, sh, most);
      // NaN, infinities, infinite scores and those so large that float32 leaves them coarse are left to the passes by the maximum
      const float m = unordered(over_ranks(special || !(most < INFINITY) ? 0xffffffffu : ordered(most)));
      if (fabsf(m) < 2048.f) {
        auto score = [&](float x, float e) { return fmaf(x, r.scale, -log2_of_normal(e)); };
        // |x scale| is at most that of the score and |log2 e| together
        decide(m, margin_of(m, 150.f), chunks_reaching, score, true);
        if (ranks > 1) cl.sync();
        return;
      }
      if (ranks > 1) cl.sync();  // rank_max is written again
      if (r.shift > 0) {
        for (int i = threadIdx.x; i <= r.chunks; i += kThreads) reinterpret_cast<int*>(sh.best())[i] = INT32_MIN;
        __syncthreads();
      }
    }
  }

  // (rank 0's, for the chunks' maxima: cleared before the ranks meet over the row's maximum)
  clear(sh);
  if (threadIdx.x == 0) sh.listed = sh.reaching = 0u;
  // ---- the row's maximum, its chunks' maxima, and the sum of the weights where top-p stands alone
  const bool sum_first = !greedy && by_p && !by_k;
  float own_max = -INFINITY, own_sum = 0.f;
  const uint32_t own_top = sum_first ? first_pass<true>(r, sh, own_max, own_sum) : first_pass<false>(r, sh, own_max, own_sum);
  const uint32_t top = over_ranks(own_top);
  r.max = unordered(top);
  if (top >= kInfinite || top <= kMasked || greedy) {
    largest(top);
    if (ranks > 1) cl.sync();  // no rank leaves while another reads its shared memory
    return;
  }

  // scores in powers of two below the maximum's
  float least_m = -INFINITY;  // the least logit of min-p's weight
  if (by_m) {
    if (wid == 0) {  // (64-bit units are few)
      const uint32_t edge = edge_of_weight(r, T, fminf(min_p, 1.f));
      if (lane == 0) sh.edge_m = edge;
    }
    __syncthreads();
    least_m = unordered(sh.edge_m);
  }
  auto kept_by_m = [&](float x) { return x >= least_m; };
  auto score = [&](float x, float e) { return score_of(r, x, e); };

  const float reach_m = least_m;
  const uint32_t least = by_m ? ordered(least_m) : kMasked + 1;

  // ---- the borders of top-k and top-p
  Border border{0, 0, 0};
  int bucket = -1;  // the draw's pass takes the logits above this bucket and collects it
  double want = 0.0;
  uint32_t first = 0;
  if (by_k || by_p || reach_m > -INFINITY) {
    // what the chunks' maxima tell: a value that k logits, or logits of top_p of the weight, reach.  Rank 0's buckets take
    // all ranks' maxima.
    if (sum_first) {
      Key sum = own_max > -INFINITY ? __double2ull_rn((double)(own_sum * (own_max < r.max ? exp2_of((own_max - r.max) * r.scale) : 1.f)) * 0x1p31) : 0;
      uint32_t none = 0, all_c;
      Key all;
      block_scan(sh, none, sum, all_c, all);
      if (threadIdx.x == 0) sh.rank_sum = all;
    }
    uint32_t reaching = 0;
    for (int c = threadIdx.x; c < r.chunks + r.ends; c += kThreads) {
      const uint32_t o = sh.chunk[c];
      if (o > kMasked) {
        const float t = below(r, unordered(o));
        if (by_k || by_p) add(*home, bucket_of(t), mass_of(t));
        reaching += o >= least;
      }
    }
    if (by_m) {
      reaching = __reduce_add_sync(0xffffffffu, reaching);
      if (lane == 0) atomicAdd(&home->reaching, reaching);
    }
    cl.sync();
    if (rank == 0 && (by_k || by_p)) {
      uint32_t c[2];
      Key m[2], sum = 0;
      gather(cl, sh, 1, c, m);
      if (sum_first) {
        for (int i = 0; i < ranks; ++i) sum += (ranks == 1 ? &sh : cl.map_shared_rank(&sh, i))->rank_sum;
        want = (double)top_p * (double)sum;
      }
      uint32_t need = 0;
      if (by_k) {
        // k chunks hold k logits that reach their maxima; in a flat row fewer chunks do: where a share f of N chunks reaches a value, about
        // -ln(1 - f) N logits do.  (Too few of them collected: the passes below.)
        const float chunks = (float)((r.quads >> (5 + r.shift)) + 1);
        const float few = chunks * (1.f - expf(-(1.25f * (float)k + 32.f) / chunks));
        need = (uint32_t)max(1, min(k, (int)few));
      }
      const bool found = find_border(sh, c, m, 0, 0, need, want);
      // the bucket's lower end, and a little below: a logit more in the list does no harm
      const float edge = (float)(sh.bucket + 1) / (32.f * r.scale);
      if (threadIdx.x == 0)
        sh.reach = found && sh.bucket < kBuckets - 1 ? r.max - edge * (1.f + 0x1p-18f) - 0x1p-20f * fabsf(r.max) : NAN;
    }
    if (by_k || by_p) cl.sync();
    // the list from the higher of both values: top-p's sums are over what lies above, so what min-p cuts off below does not matter
    // (with top-k they need all of the k: its own value)
    const float reach_kp = by_k || by_p ? home->reach : -INFINITY;
    const float reach = by_k && (reach_kp > -INFINITY || by_p) ? reach_kp : fmaxf(reach_kp, reach_m);  // (fmaxf passes over NaN)
    const float share = (float)home->reaching / ((float)(r.quads >> (5 + r.shift)) + 1.f);
    // (where most chunks reach min-p's value the list would not hold the logits that do)
    bool fast = reach > -INFINITY && !(reach == reach_m && !by_k && share > 0.6f);
    if (fast) {
      const uint32_t listed = collect(cl, r, sh, home, (Key)ordered(reach) << 32, ~(Key)0);
      fast = listed <= (uint32_t)kList && (!by_k || listed >= (uint32_t)k || (!by_p && reach == reach_m));
    }
    if (fast) {
      if (rank != 0) {  // the rest is rank 0's list
        cl.sync();
        return;
      }
      cut_list(r, sh, home->listed, by_k ? (uint32_t)k : 0u, 0, by_k || !by_p ? INFINITY : want, by_k ? top_p : 1.f, false);
      __syncthreads();
      const int kept = max(sh.kept, 1);
      auto listed = [&](float, auto f) {
        for (int i = threadIdx.x; i < kept; i += kThreads) {
          const float x = unordered((uint32_t)(sh.list[i] >> 32));
          const int id = (int)id_of(sh.list[i]);
          if (kept_by_m(x)) f(x, __ldg(r.e + id), id);
        }
      };
      float most = -INFINITY;
      listed(0.f, [&](float x, float e, int) { most = fmaxf(most, score(x, e)); });
      most = block_max(sh, most);
      if (most > -INFINITY)
        decide(most, margin_of(most, 150.f), listed, score, false);
      else if (threadIdx.x == 0)  // no random number to choose by: the largest logit
        p.ids[row] = (int64_t)id_of(sh.list[0]);
      if (ranks > 1) cl.sync();  // (the others have read this CTA's shared memory by now)
      return;
    }
    // the buckets of all logits (min-p alone: the pass below)
    if (by_k || by_p) {
      const bool both = by_k && by_p;
      cl.sync();
      clear(sh);
      __syncthreads();
      if (by_k) bucket_pass<false>(r, sh);
      if (by_p) bucket_pass<true>(r, sh);
      cl.sync();
      uint32_t c[2], all_c;
      Key m[2], all_m;
      gather(cl, sh, ranks, c, m);
      uint32_t pc = c[0] + c[1];
      Key pm = m[0] + m[1];
      block_scan(sh, pc, pm, all_c, all_m);
      __syncthreads();
      const bool cut_k = by_k && (uint32_t)k < all_c;  // (a row may hold fewer finite logits)
      want = (double)top_p * (double)all_m;
      if (cut_k && both) {
        // the k-th logit itself, then the buckets of those above it
        find_border(sh, c, m, 0, 0, (uint32_t)k, 0.0);
        border = resolve(cl, r, sh, home, rank, ranks, 0, (uint32_t)k, 0.0, top_p);
        if (border.listed == 0) {
          cl.sync();
          clear(sh);
          __syncthreads();
          for_each(r, sh.chunk, (uint32_t)(border.key >> 32), [&](float x, int id, int) {
            if (key_of(x, (uint32_t)id) >= border.key) add(sh, bucket_of(below(r, x)), mass_of(below(r, x)));
          });
          cl.sync();
          gather(cl, sh, ranks, c, m);
          find_border(sh, c, m, 0, 0, 0, (double)top_p * (double)border.mass);
          const Border bp = resolve(cl, r, sh, home, rank, ranks, border.key, 0, (double)top_p * (double)border.mass, 1.f);
          border.key = bp.key > border.key ? bp.key : border.key;
        }
      } else if (cut_k || by_p) {
        first = cut_k ? (uint32_t)k : 0u;
        find_border(sh, c, m, 0, 0, first, want);
        bucket = sh.bucket;
      }
    }
  }

  // ---- the draw's pass
  cl.sync();  // the buckets have been read
  if (r.shift > 0)
    for (int i = threadIdx.x; i <= r.chunks; i += kThreads) reinterpret_cast<int*>(sh.best())[i] = INT32_MIN;
  if (threadIdx.x == 0) sh.listed = 0u;
  cl.sync();
  float most = -INFINITY;
  if (bucket >= 0) {
    const uint32_t above_count = sh.above_count;
    const Key above_mass = sh.above_mass;
    const float from = unordered(edge_of(r, bucket)), above = bucket > 0 ? unordered(edge_of(r, bucket - 1)) : INFINITY;
    auto kind = [&](float x, int) { return x >= above ? (int)kept_by_m(x) : x >= from ? 2 : 0; };
    most = draw_pass(r, sh, home, kMasked + 1, true, kind, score);  // (the bucket is collected whole, whatever min-p keeps)
    cl.sync();
    const uint32_t n = home->listed;
    if (n <= (uint32_t)kList) {
      // the bucket's logits that stay take part, too
      int kept = 0;
      auto listed = [&](float, auto f) {
        for (int i = threadIdx.x; i < kept; i += kThreads) {
          const float x = unordered((uint32_t)(sh.list[i] >> 32));
          const int id = (int)id_of(sh.list[i]);
          if (kept_by_m(x)) f(x, __ldg(r.e + id), id);
        }
      };
      if (rank == 0) {
        cut_list(r, sh, n, first != 0 ? first - above_count : 0u, above_mass, first != 0 ? INFINITY : want, 1.f, false);
        __syncthreads();
        kept = sh.kept;
        listed(0.f, [&](float x, float e, int) { most = fmaxf(most, score(x, e)); });
      }
      most = unordered(over_ranks(ordered(most)));
      if (most > -INFINITY) {
        auto visit = [&](float least, auto f) {
          chunks_reaching(least, [&](float x, float e, int id) {
            if (x > -INFINITY && kind(x, id) == 1) f(x, e, id);
          });
          listed(least, f);
        };
        decide(most, margin_of(most, 150.f), visit, score, true);
      } else {
        largest(top);
      }
      if (ranks > 1) cl.sync();
      return;
    }
    // more than the list holds (equal or nearly equal logits): count and weight of all, and the border by keys
    cl.sync();
    clear(sh);
    __syncthreads();
    bucket_pass<false>(r, sh);
    bucket_pass<true>(r, sh);
    cl.sync();
    uint32_t c[2];
    Key m[2];
    gather(cl, sh, ranks, c, m);
    find_border(sh, c, m, 0, 0, first, want);
    border = resolve(cl, r, sh, home, rank, ranks, 0, first, want, 1.f);
    cl.sync();
    if (r.shift > 0)
      for (int i = threadIdx.x; i <= r.chunks; i += kThreads) reinterpret_cast<int*>(sh.best())[i] = INT32_MIN;
    cl.sync();
  }
  auto kind = [&](float x, int id) { return (int)(key_of(x, (uint32_t)id) >= border.key && kept_by_m(x)); };
  most = draw_pass(r, sh, home, max(least, (uint32_t)(border.key >> 32)), false, kind, score);
  most = unordered(over_ranks(ordered(most)));
  if (most > -INFINITY) {
    auto visit = [&](float least, auto f) {
      chunks_reaching(least, [&](float x, float e, int id) {
        if (x > -INFINITY && kind(x, id) == 1) f(x, e, id);
      });
    };
    decide(most, margin_of(most, 150.f), visit, score, true);
  } else {
    largest(top);
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
