// logprobs.cu -- log probabilities of given tokens, entropy and the top alternatives of rows of logits.
//
//   lp_j = x_j - m - log Z,  Z = sum_j e^(x_j - m),  H = log Z - (1 / Z) sum_j e^(x_j - m) (x_j - m).
//
// Bound: the logits' bytes, read once.  Each thread keeps a running maximum m, Z and the second sum, moved
// when a batch of 16 values raises m, and has the next batch on its way; each warp keeps the largest keys
// (value, id) of what it has seen, sorted over its lanes, and a batch touches the list only if its maximum
// reaches the smallest kept value of any warp of the CTA.  A few rows are cut into parts over many CTAs; the
// last part of a row to finish joins them in their order.
//
// Measured: 512 rows of 151936 with 5 alternatives 55.7 us (5.59 TB/s, 82% of the measured copy rate; 50 us with none, 60
// with 8, 80 with 20, 99 with 32: a candidate enters a warp's list by itself, and the floor is a warp's own k-th value), one
// row with 8 alternatives 10.5 us (7.4 with none): launch, one pass, the join.
#include <mutex>

#include "qmv_common.cuh"
#include "qmv_internal.h"

namespace qmv {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// What a CTA's part of a row costs besides its values (start, lists, the join), in values: with 4096 the rows of
// 512 x 151936 are cut and take 84.9 us (5 alternatives; 61 us with none, 153 with 20), with 32768 they are whole and
// take 55.7 (50, 80); 1, 8 and 64 rows of 151936 and 200 of 32000 do not change.
constexpr long long kPartCost = 32768;
constexpr int kBatch = 16;  // values a thread takes at a time, as four 16-byte loads
using Key = unsigned long long;

// A logit and its id as one key that orders as the result does: larger logits first, equal ones
// by the lower id.  The float's bits are mapped to an unsigned order; -0 counts as +0, NaN as the largest.
__device__ __forceinline__ uint32_t ordered(float x) {
  uint32_t b = __float_as_uint(x + 0.0f);
  if ((b & 0x7fffffffu) > 0x7f800000u) b = 0x7fffffffu;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ Key key_of(float x, uint32_t id) { return ((Key)ordered(x) << 32) | (0xffffffffu - id); }

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float exp_of(float d) {  // e^d for d <= 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d * 1.4426950408889634f));
  return y;
}

// Running statistics of a row's values: the maximum, sum e^(x - m), sum e^(x - m) (x - m).
struct Stats {
  float m, z, zx;
  __device__ __forceinline__ void move_to(float to) {  // to >= m
    const float d = m == -INFINITY ? -200.f : fmaxf(m - to, -200.f);
    const float f = exp_of(d);
    zx = (zx + z * d) * f;
    z *= f;
    m = to;
  }
  __device__ __forceinline__ void join(Stats o) {
    const float to = fmaxf(m, o.m);
    if (to == -INFINITY) return;
    move_to(to);
    o.move_to(to);
    z += o.z;
    zx += o.zx;
  }
};

// The warp's list: lane i holds the i-th largest key (n_top <= 32 of them count).
__device__ __forceinline__ void insert(Key& mine, Key k, int lane) {
  const int at = __popc(__ballot_sync(0xffffffffu, mine > k));
  const Key up = __shfl_up_sync(0xffffffffu, mine, 1);
  if (lane == at) {
    mine = k;
  } else if (lane > at) {
    mine = up;
  }
}

// The warp's 32 keys in descending order over its lanes (bitonic), and the 32 largest of two such lists.
__device__ __forceinline__ void sort_keys(Key& v, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int d = size >> 1; d > 0; d >>= 1) {
      const Key u = __shfl_xor_sync(0xffffffffu, v, d);
      v = (((lane & d) == 0) == ((lane & size) == 0)) == (u > v) ? u : v;
    }
}
__device__ __forceinline__ void merge_keys(Key& mine, Key other, int lane) {
  const Key r = __shfl_sync(0xffffffffu, other, 31 - lane);
  mine = r > mine ? r : mine;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const Key u = __shfl_xor_sync(0xffffffffu, mine, d);
    mine = ((lane & d) == 0) == (u > mine) ? u : mine;
  }
}

struct Part {  // of one row, in the workspace
  Stats s;
  int bad;
  Key keys[QMV_MAX_TOP];
};

struct PartArea {
  unsigned* counters;  // one per row, zero between launches
  Part* parts;
};

__global__ void __launch_bounds__(kThreads) logprobs_kernel(const __grid_constant__ LogprobArgs a, int n_parts,
                                                            const PartArea area) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ Stats warp_stats[kWarps];
  __shared__ Key warp_keys[kWarps][QMV_MAX_TOP];
  __shared__ uint32_t floor_bits;  // no value below this can be among the largest n_top
  __shared__ int last_flag;
  __shared__ __align__(16) float stash[kWarps][32][kBatch + 4];  // a batch that may enter the lists
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const long long row = blockIdx.x / n_parts;
  const int part = blockIdx.x % n_parts;
  const float* x = a.logits + row * a.stride;
  const int n = (int)a.vocab;
  const int k = a.n_top;
  if (tid == 0) floor_bits = k > 0 ? 0u : 0xffffffffu;
  __syncthreads();

  Stats st{-INFINITY, 0.f, 0.f};
  Key mine = 0;
  bool bad = false, fresh = true;

  // 16 values a lane, absent ones -inf; id_of(lane, e): the id of a lane's value e; live: a lane's values that are there
  auto take = [&](const float (&v)[kBatch], int live, auto id_of) {
    float top = v[0];
#pragma unroll
    for (int e = 1; e < kBatch; ++e) top = max_nan(top, v[e]);
    const uint32_t fb = *reinterpret_cast<volatile uint32_t*>(&floor_bits);
    float floor = k > 0 ? (fb == 0u ? -INFINITY : unordered(fb)) : INFINITY;
    if (__any_sync(0xffffffffu, !(top < floor))) {
      bad |= !(top < INFINITY);
      if (k > 0) {
        Key least = __shfl_sync(0xffffffffu, mine, k - 1);
        int held = -1;  // this lane's value that is in the list already
        if (fresh) {
          fresh = false;
          // nothing kept yet: the lanes' largest values, sorted, are the list to begin with
#pragma unroll
          for (int e = kBatch - 1; e >= 0; --e)
            if (v[e] == top || (isnan(top) && isnan(v[e]))) held = e;
          if (held >= live) held = -1;
          mine = held >= 0 ? key_of(top, id_of(lane, held)) : 0;
          sort_keys(mine, lane);
          least = __shfl_sync(0xffffffffu, mine, k - 1);
        }
        // lanes with a value that may enter the list: not below the floor or the least kept one, nor all equal to
        // that with larger ids; the warp looks at such a lane's 16 values together
        const float lv = least == 0 ? -INFINITY : unordered((uint32_t)(least >> 32));
        floor = lv > floor ? lv : floor;
        const bool may = live > 0 && !(top < floor) && !(top == lv && id_of(lane, 0) > 0xffffffffu - (uint32_t)least);
        uint32_t who = __ballot_sync(0xffffffffu, may);
        if (may) {
#pragma unroll
          for (int e = 0; e < kBatch; e += 4)
            *reinterpret_cast<float4*>(&stash[wid][lane][e]) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
        __syncwarp();
        while (who != 0u) {
          const int src = __ffs(who) - 1;
          who &= who - 1;
          const int n_live = __shfl_sync(0xffffffffu, live, src), skip = __shfl_sync(0xffffffffu, held, src);
          const int e = lane & (kBatch - 1);
          const Key mine_key = key_of(stash[wid][src][e], id_of(src, e));
          uint32_t in = __ballot_sync(0xffffffffu, lane < n_live && lane != skip && mine_key > least);
          while (in != 0u) {
            const Key c = __shfl_sync(0xffffffffu, mine_key, __ffs(in) - 1);
            in &= in - 1;
            if (c > least) {
              insert(mine, c, lane);
              least = __shfl_sync(0xffffffffu, mine, k - 1);
            }
          }
        }
        __syncwarp();  // the stash has been read
        if (lane == 0) atomicMax(&floor_bits, (uint32_t)(least >> 32));
      }
    }
    if (top > st.m) st.move_to(top);
    const float ref = st.m == -INFINITY ? 0.f : st.m;
    // four chains of sums, joined in a fixed order
    float z[4] = {0.f, 0.f, 0.f, 0.f}, zx[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const float d = fmaxf(v[e] - ref, -200.f);  // e^-200 is 0 in float32
      const float y = exp_of(d);
      z[e & 3] += y;
      zx[e & 3] = fmaf(y, d, zx[e & 3]);
    }
    st.z += (z[0] + z[1]) + (z[2] + z[3]);
    st.zx += (zx[0] + zx[1]) + (zx[2] + zx[3]);
  };

  // the row from its first 16-byte boundary in batches of 4 x 128 values a warp, cut into n_parts; the up to
  // three values before it and after the last whole four belong to part 0
  const int head = min((int)((4 - ((reinterpret_cast<uintptr_t>(x) >> 2) & 3)) & 3), n);
  const int quads = (n - head) / 4;
  const float4* xv = reinterpret_cast<const float4*>(x + head);
  const int q0 = (int)((long long)quads * part / n_parts), q1 = (int)((long long)quads * (part + 1) / n_parts);
  float4 next[4];  // the batch after the one at hand is on its way meanwhile
  auto load = [&](int q) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int qi = q + 32 * i + lane;
      next[i] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (qi < q1) next[i] = __ldg(xv + qi);
    }
  };
  load(q0 + wid * 128);
  for (int q = q0 + wid * 128; q < q1; q += kWarps * 128) {
    float v[kBatch];
    int live = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = next[i];
      if (q + 32 * i + lane < q1) live = 4 * i + 4;
      v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
    }
    load(q + kWarps * 128);
    take(v, live, [&](int l, int e) { return (uint32_t)(head + 4 * (q + 32 * (e >> 2) + l) + (e & 3)); });
  }
  if (part == 0 && wid == 0) {
    const int tail = n - head - 4 * quads;
    if (head + tail > 0) {
      float v[kBatch];
#pragma unroll
      for (int e = 0; e < kBatch; ++e) v[e] = -INFINITY;
      auto id_of = [&](int l, int) { return (uint32_t)(l < head ? l : l - head + n - tail); };
      if (lane < head + tail) v[0] = x[id_of(lane, 0)];
      take(v, lane < head + tail ? 1 : 0, id_of);
    }
  }

  // the CTA: lanes, then warps, in a fixed order
  auto join_cta = [&]() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      Stats s;
      s.m = __shfl_xor_sync(0xffffffffu, st.m, o);
      s.z = __shfl_xor_sync(0xffffffffu, st.z, o);
      s.zx = __shfl_xor_sync(0xffffffffu, st.zx, o);
      st.join(s);
    }
    if (lane == 0) warp_stats[wid] = st;
    if (k > 0) warp_keys[wid][lane] = mine;
    bad = __syncthreads_or(bad);
#pragma unroll
    for (int half = kWarps / 2; half > 0; half >>= 1) {
      if (wid < half) {
        st.join(warp_stats[wid + half]);
        if (k > 0) merge_keys(mine, warp_keys[wid + half][lane], lane);
      }
      if (half > 1) {
        __syncthreads();
        if (wid < half) {
          if (lane == 0) warp_stats[wid] = st;
          if (k > 0) warp_keys[wid][lane] = mine;
        }
        __syncthreads();
      }
    }
  };
  join_cta();

  if (n_parts > 1) {
    Part* parts = area.parts + row * n_parts;
    if (wid == 0) {
      if (lane == 0) {
        __stcg(&parts[part].s.m, st.m);
        __stcg(&parts[part].s.z, st.z);
        __stcg(&parts[part].s.zx, st.zx);
        __stcg(&parts[part].bad, (int)bad);
      }
      if (k > 0) __stcg(&parts[part].keys[lane], mine);
      __threadfence();
      __syncwarp();
      if (lane == 0) {
        const unsigned seen = atomicAdd(area.counters + row, 1u);
        last_flag = seen == (unsigned)(n_parts - 1);
        if (last_flag) area.counters[row] = 0;
      }
    }
    __syncthreads();
    if (!last_flag) return;
    __threadfence();
    st = Stats{-INFINITY, 0.f, 0.f};
    mine = 0;
    bad = false;
#pragma unroll 2
    for (int p = wid; p < n_parts; p += kWarps) {
      // lane 0 of each warp joins the statistics, all lanes the keys
      const Key c = k > 0 ? __ldcg(&parts[p].keys[lane]) : 0;
      bad |= __ldcg(&parts[p].bad) != 0;
      if (lane == 0) st.join(Stats{__ldcg(&parts[p].s.m), __ldcg(&parts[p].s.z), __ldcg(&parts[p].s.zx)});
      if (k > 0) merge_keys(mine, c, lane);
    }
    join_cta();
  }

  if (wid == 0) {
    const bool none = st.m == -INFINITY && !bad;
    const float lz = bad ? NAN : logf(st.z);
    // the maximum goes first: beside a large one m + log Z would round log Z away
    auto logprob = [&](float v) { return none ? -INFINITY : (v - st.m) - lz; };
    if (lane == 0 && a.entropy != nullptr) a.entropy[row] = none ? 0.f : lz - st.zx / st.z;
    for (int i = lane; i < a.n_given; i += 32) {
      const long long id = a.given[row * a.n_given + i];
      a.given_logprob[row * a.n_given + i] = id >= 0 && id < a.vocab ? logprob(x[id]) : NAN;
    }
    if (lane < k) {
      const uint32_t id = 0xffffffffu - (uint32_t)mine;
      a.top_ids[row * k + lane] = (int)id;
      a.top_logprob[row * k + lane] = logprob(unordered((uint32_t)(mine >> 32)));
    }
  }
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, int64_t rows, const DeviceInfo& dev, cudaStream_t stream) {
  PartArea area{nullptr, nullptr};
  static std::mutex mu;
  static int ctas_per_sm[64] = {};
  if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidValue;
  int per_sm;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (ctas_per_sm[dev.device] == 0) {
      int k = 0;
      const cudaError_t err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&k, logprobs_kernel, kThreads, 0);
      if (err != cudaSuccess) return err;
      ctas_per_sm[dev.device] = k > 0 ? k : 1;
    }
    per_sm = ctas_per_sm[dev.device];
  }
  // parts of a row, of 4096 values at least: as many as keep the waves of CTAs times a part's length, with
  // kPartCost for what a part costs besides, shortest
  long long parts = 1;
  const long long most = (a.vocab + 4095) / 4096, slots = (long long)dev.sm_count * per_sm;
  Workspace ws;
  if (most > 1 && rows < slots && stream_serve_workspace(dev, stream, &ws) == cudaSuccess && rows <= ws.max_counters) {
    long long best = 0;
    const long long fit = (long long)(ws.max_partial_floats * sizeof(float) / sizeof(Part)) / rows;
    for (long long p = 1; p <= most && p <= fit && p <= 64; ++p) {
      const long long cost = (rows * p + slots - 1) / slots * (a.vocab / p + kPartCost);
      if (best == 0 || cost < best) {
        best = cost;
        parts = p;
      }
    }
    area.counters = ws.counters;
    area.parts = reinterpret_cast<Part*>(ws.partials);
  }
  if (rows * parts > INT32_MAX) return cudaErrorInvalidValue;
  return launch_dependent(logprobs_kernel, dim3((unsigned)(rows * parts)), kThreads, 0, stream, a, (int)parts, area);
}

}  // namespace qmv
