// attend_prompt.cu -- softmax attention of many rows a sequence (prompts, chunks of prompts) over the paged
// 8-bit cache, on the 5th-generation tensor core; bfloat16 rows, heads of 64 or 128.
//
//   S = Q K^T (levels),  x = S ks c + log2 vs,  P = 2^(x - ref),  O = P V (levels),  out = O / sum(P / vs)
//
// with a page's scales ks and vs and the row's factor c = scale log2 e.  The V scale joins the weights'
// exponent, so that the largest weight * V scale, not the largest weight, sets the range in which
// the weights are rounded to half: they are formed times 2^7 against a reference that is at most
// 2^8 behind the running maximum (the output is rescaled only when it falls further back), so they
// stay under 2^15, and those down to 2^-21 of the largest are normal halves.  A page whose V scale is 0 has no
// logarithm: its weights are 0 in P, and its keys' exponentials go to a sum with a reference of its own, on a path
// that tiles without such pages do not take.
//
// A CTA takes two tiles of 128 rows (query token, head of the group) of one key/value head and goes
// through the keys 128 at a time.  Warps 0-3 and 4-7: one row a thread of the two tiles (softmax);
// 8-11: levels to halves in shared memory, one conversion for both row tiles; 13: the pages' levels into
// shared memory by bulk copies and their scales, one tile ahead; 12: the products, P V and then the next
// Q K^T of one tile, then of the other, so that one tile's products run while the other's softmax does
// (warps 14 and 15 only make up the warpgroup whose registers the softmax warps take).  Scores lie in
// tensor memory (128 columns a tile), the weights over them as halves, the outputs beside them (head_dim
// columns a tile).
//
// Bound: 2 x 2 x 128 x 128 x head_dim operations a tile and turn on the tensor core, against one exponential for
// each score and the softmax's turn, which hides behind the other tile's products only in part.  2048 rows
// over 16384 tokens (32 heads over 8 of 128) 399 us, 1290 TFLOP/s (69% of the measured bf16 rate; tensor pipe 57%
// active on a smaller case, issue 48%); three prompts of up to 2048 tokens 87 us.  A turn of one row tile takes
// about 3500 cycles: softmax 1800, products 1300 (1024 of them at the peak rate), hand-over 400.
#include <mutex>

#include "attend.cuh"
#include "tcgen05.cuh"

namespace qmv {

namespace {

constexpr int kTileRows = 128;
constexpr int kKeys = 128;
constexpr int kThreads = 16 * 32;
constexpr int kTableStages = 4;
constexpr float kWeightBits = 7.f;
constexpr float kSlack = 8.f;
// registers: 256 threads x 192 + 128 x 88 + 128 x 40 = the 512 x 128 of the launch

constexpr uint32_t kTmemCols = 512;

// What a group of 16 keys (one page) brings to the softmax.
struct GroupScale {
  float ks;    // K scale
  float e;     // log2 of the V scale, -infinity for 0
  float back;  // 1 / V scale, 0 for 0
  uint32_t zeros;  // which of the tile's groups lie in pages of V scale 0, the same in each group
};

template <int D>
struct Smem {
  static constexpr int kPanel = kKeys * 128;         // 128 rows of 64 halves
  static constexpr int kTile = kPanel * (D / 64);
  static constexpr int kV = 0;                       // two stages
  static constexpr int kK = kV + 2 * kTile;          // two stages
  static constexpr int kQ = kK + 2 * kTile;          // two tiles
  static constexpr int kRawK = kQ + 2 * kTile;       // levels as they lie in the pages
  static constexpr int kRawV = kRawK + kKeys * D;
  static constexpr int kTable = kRawV + kKeys * D;   // kTableStages x 8 GroupScale
  static constexpr int kBars = kTable + kTableStages * 8 * 16;
  static constexpr int kMisc = kBars + 24 * 8;
  static constexpr int kBytes = kMisc + 32 + 1024;   // and room to align to 1024
  static_assert(kBytes <= 227 * 1024, "one CTA's shared memory");
};

// Barriers.
// kFree: the products up to S of keys i are done (i = 0, 1, .. in turn on the two): K(i) and V(i - 1) are free.
enum { kKFull = 0, kVFull = 2, kFree = 4, kQFull = 6, kSFull = 8, kPFull = 10, kDone = 12, kTableFull = 13, kRawKFull = 17,
       kRawVFull = 18, kRawKFree = 19, kRawVFree = 20, kBarCount = 21 };
static_assert(kBarCount <= 24, "room for the barriers");

// Wait for a phase, at most about a second: false, and every later wait gives up, when it runs out.  Kept
// short: the roles' code shares the instruction cache.
__device__ __forceinline__ bool pwait(uint64_t* bar, uint32_t parity, volatile int* failed) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = (uint32_t)clock();
  while (!mbar_try_wait(bar, parity)) {
    if (*failed != 0) return false;
    if ((uint32_t)clock() - t0 > 2000000000u) {
      *failed = 1;
      return false;
    }
  }
  return true;
}

// Global to shared memory, counted in bytes on an mbarrier; other CTAs read the same pages, so no cache hint.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(uint32_t a, uint32_t b, uint32_t c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A group's factor of a row, kept positive: a masked score of -infinity stays one (a factor this small
// makes every other score 0).
__device__ __forceinline__ float group_factor(float ks, float rowc) { return fmaxf(ks * rowc, 1.2e-38f); }

// The tensor core's instructions issued by one elected lane of a converged warp: the descriptors stay in
// uniform registers.
__device__ __forceinline__ void warp_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void warp_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void warp_commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// Blocks of 256 rows of a sequence.
__device__ __forceinline__ int blocks_of(const KvSeq& q, int group) {
  return (int)(((long long)q.n * group + 2 * kTileRows - 1) / (2 * kTileRows));
}

// Blocks from `whole` on (in the order of the grid) are cut along their keys into up to `split` parts of at
// least kMinPart tiles, whose unnormalised outputs meet in the workspace: a part's area is [dim / 4][256 rows] of
// four floats, then the rows' references and sums.
struct SplitPlan {
  int whole;
  int split;
  unsigned* counters;  // eight a cut block (one a softmax warp), zero between launches
  float* parts;
};
constexpr int kMinPart = 4;

// PG: keys that share a page's scales, 16 or 64 (pages of 64 and 128 tokens).  CUT: some blocks are cut (the code
// that joins their parts costs the launches without them 3%: prompts of 2048, 1563 and 1278 tokens 98 against 95 us).
template <int D, int PG, bool CUT>
__global__ void __launch_bounds__(kThreads, 1) attend_prompt_kernel(const __grid_constant__ KvRef c,
                                                                    const __grid_constant__ AttendArgs a,
                                                                    const SplitPlan plan) {
  using L = Smem<D>;
  constexpr int kPieces = D / 16;           // 16-byte pieces of a row of levels
  constexpr int kRowsWarp = 32 / kPieces;   // rows a converting warp takes at a time
  constexpr int kPasses = kKeys / (4 * kRowsWarp);
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  GroupScale* table = reinterpret_cast<GroupScale*>(smem + L::kTable);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* failed = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = a.heads / c.kv_heads;

  // the CTA's block: heads fastest, a sequence's last (longest) blocks first; every warp looks it up
  const int cut = CUT ? (int)blockIdx.x - plan.whole : -1;  // counted over the parts of cut blocks
  const int item = cut < 0 ? (int)blockIdx.x : plan.whole + cut / plan.split;
  const int kvh = item % c.kv_heads;
  const int want = item / c.kv_heads;
  int s = -1, rb = 0;
  for (int s0 = 0, base = 0; s0 < c.n_seq && s < 0; s0 += 32) {
    const int si = s0 + lane;
    const int nb = si < c.n_seq ? blocks_of(kv_seq(c, si), group) : 0;
    int inc = nb;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, base + inc > want);
    if (hit != 0u) {
      const int l = __ffs(hit) - 1;
      s = s0 + l;
      const int before = base + __shfl_sync(0xffffffffu, inc - nb, l);
      rb = __shfl_sync(0xffffffffu, nb, l) - 1 - (want - before);
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (s < 0) return;  // the grid is an upper bound
  const KvSeq sq = kv_seq(c, s);
  const int first = sq.len - sq.n;
  const int rho0 = rb * 2 * kTileRows;
  const int rows_all = sq.n * group - rho0 < 2 * kTileRows ? sq.n * group - rho0 : 2 * kTileRows;
  const int n_tiles = rows_all > kTileRows ? 2 : 1;
  const int i_lo = rho0 / group, i_hi = (rho0 + rows_all - 1) / group;
  const int any_end = a.causal ? first + i_hi + 1 : sq.len;
  const int any_begin = a.window > 0 && first + i_lo - a.window + 1 > 0 ? first + i_lo - a.window + 1 : 0;
  int jb = any_begin / kKeys, je = (any_end + kKeys - 1) / kKeys;
  int parts = 1, part = 0;
  if (CUT && cut >= 0) {
    const int tiles = je - jb;
    parts = tiles / kMinPart < plan.split ? (tiles / kMinPart > 1 ? tiles / kMinPart : 1) : plan.split;
    part = cut % plan.split;
    if (part >= parts) return;
    je = jb + tiles * (part + 1) / parts;
    jb += tiles * part / parts;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars + kKFull + i, 4);
      mbar_init(bars + kVFull + i, 4);
      mbar_init(bars + kFree + i, 1);
      mbar_init(bars + kQFull + i, 4);
      mbar_init(bars + kSFull + i, 1);
      mbar_init(bars + kPFull + i, 4);
    }
    mbar_init(bars + kDone, 1);
    mbar_init(bars + kRawKFull, 1);
    mbar_init(bars + kRawVFull, 1);
    mbar_init(bars + kRawKFree, 4);
    mbar_init(bars + kRawVFree, 4);
    for (int i = 0; i < kTableStages; ++i) mbar_init(bars + kTableFull + i, 1);
    *failed = 0;
    fence_mbar_init();
  }
  if (warp == 12) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
  // the first loads of the roles are under way while the CTA sets up: a softmax thread's row of q, the page of a
  // group of keys and its scales
  const int row_q = rho0 + (warp >> 2) * kTileRows + (threadIdx.x & 127);  // of warps 0-7
  const bool row_live = warp < 8 && row_q < sq.n * group;
  const int row_i = row_live ? row_q / group : 0;
  const int row_head = kvh * group + (row_live ? row_q - row_i * group : 0);
  uint4 qraw[D / 8];
  if (row_live) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (sq.row0 + row_i) * a.q_stride +
                                                      (long long)row_head * D);
#pragma unroll
    for (int k = 0; k < D / 8; ++k) qraw[k] = __ldg(src + k);
  } else {
#pragma unroll
    for (int k = 0; k < D / 8; ++k) qraw[k] = make_uint4(0u, 0u, 0u, 0u);
  }
  const int32_t* page_row = c.page_table + (long long)s * c.table_stride;
  auto page_of = [&](int id, int key) {  // a page id outside the cache is recorded and not followed; -1: none
    if ((unsigned)id < (unsigned)c.n_pages) return id;
    if (lane < 8 && key < je * kKeys && key < sq.len) record_status(c.status, QMV_E_ARG);
    return -1;
  };
  int id = -1;
  bool hidden = false;
  float gk = 0.f, gv = 0.f;
  if (warp == 13) {
    const int key = jb * kKeys + 16 * lane;
    // pages that end before any row's first key may be anything: not looked at (only the first tile can hold one)
    hidden = key < (any_begin & -c.page_tokens);
    if (lane < 8 && key < sq.len && !hidden) id = __ldg(page_row + (key >> c.page_shift));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax: thread = row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int q = warp >> 2;
    if (q < n_tiles) {
      const int r = threadIdx.x & 127;
      const bool live = row_live;
      const int i = row_i;
      const int end = !live ? 0 : a.causal ? first + i + 1 : sq.len;
      const int beg = a.window > 0 ? first + i - a.window + 1 : 0;
      // keys that every row of this tile sees
      const int t_lo = (rho0 + q * kTileRows) / group;
      const int t_last = q == 0 && n_tiles == 2 ? rho0 + kTileRows - 1 : rho0 + rows_all - 1;
      const int all_end = a.causal ? first + t_lo + 1 : sq.len;
      const int all_begin = a.window > 0 ? first + t_last / group - a.window + 1 : 0;

      // the row of q as halves, scaled by the power of two that brings its largest magnitude near 2^14
      float rowc;
      {
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          const uint4 u = qraw[k];
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u))));
        }
        float xs, xinv;
        half_stage_scale(amax, xs, xinv);
        // a negative scale goes to q, so that the largest product is the largest score
        if (a.scale < 0.f) xs = -xs;
        rowc = fabsf(a.scale) * kLog2e * xinv;
        const uint32_t dst = sbase + L::kQ + q * L::kTile + r * 128;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
          const uint4 u = qraw[k];
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            h[e] = pack_f16x2(__uint_as_float(w[e] << 16) * xs, __uint_as_float(w[e] & 0xffff0000u) * xs);
          sts_u32x4(dst + (k >> 3) * L::kPanel + (((k & 7) ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + kQFull + q);
      }

      const uint32_t quarter = (uint32_t)(32 * (warp & 3)) << 16;
      const uint32_t sp = tmem + quarter + (uint32_t)(q * kKeys);        // scores, then weights
      const uint32_t ot = tmem + quarter + (uint32_t)(256 + q * 128);    // output
      float ref = -INFINITY, l = 0.f;
      // keys of zero pages: their largest score and the sum of their exponentials against it, kept out of the registers
      volatile float zero_ref = -INFINITY, zero_sum = 0.f;
      bool ok = true;
      for (int j = jb; j < je; ++j) {
        const int n = j - jb;
        ok = pwait(bars + kTableFull + n % kTableStages, (uint32_t)((n / kTableStages) & 1), failed);
        const GroupScale* tab = table + (n % kTableStages) * 8;
        const uint32_t zeros = tab->zeros;
        ok = ok && pwait(bars + kSFull + q, (uint32_t)(n & 1), failed);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const int j0 = j * kKeys;
        if (zeros != 0u) {
#pragma unroll 1
          for (int b = 0; b < kKeys / 8; ++b) {
            if (!((zeros >> (b >> 1)) & 1u)) continue;
            uint32_t o[8];
            tmem_ld8(sp + 8 * b, o);
            tmem_ld_wait();
            const float c = group_factor(tab[b >> 1].ks, rowc);
            const float was = zero_ref;
            float m = was, x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int key = j0 + 8 * b + e;
              x[e] = key < beg || key >= end ? -INFINITY : __uint_as_float(o[e]) * c;
              m = fmaxf(m, x[e]);
            }
            if (m != -INFINITY) {
              float sum = zero_sum * (m > was ? ex2(was - m) : 1.f);
#pragma unroll
              for (int e = 0; e < 8; ++e) sum += ex2(x[e] - m);
              zero_ref = m;
              zero_sum = sum;
            }
            __syncwarp();
          }
        }
        uint32_t v[4][32];
#pragma unroll
        for (int b = 0; b < 4; ++b) tmem_ld32(sp + 32 * b, v[b]);
        tmem_ld_wait();
        if (j0 < all_begin || j0 + kKeys > all_end) {  // keys that some rows do not see
#pragma unroll
          for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int key = j0 + 32 * b + e;
              if (key < beg || key >= end) v[b][e] = 0xFF800000u;  // -inf
            }
        }
        // the tile's maximum (a group's factor is positive, so its largest product is its largest score)
        constexpr int kGroups = kKeys / PG;
        float mt = -INFINITY;
        float cg[kGroups], eg[kGroups];
#pragma unroll
        for (int x = 0; x < kGroups; ++x) {
          const GroupScale gs = tab[x * (PG / 16)];
          cg[x] = group_factor(gs.ks, rowc);
          eg[x] = gs.e;
          float m[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < PG; e += 2) {
            const int key = x * PG + e;
            m[(e >> 1) & 1] = max3(__float_as_uint(m[(e >> 1) & 1]), v[key >> 5][key & 31], v[key >> 5][(key & 31) + 1]);
          }
          mt = fmaxf(mt, fmaf(fmaxf(m[0], m[1]), cg[x], eg[x]));
        }
        // the reference follows the maximum when it has fallen 2^8 behind
        const bool move = mt > ref + kSlack;
        if (__any_sync(0xffffffffu, move)) {
          const float f = move ? ex2(ref - mt) : 1.f;
          if (move) ref = mt;
          l *= f;
          if (n > 0) {  // the scores' arrival says that the product before them is done too
#pragma unroll 1
            for (int b = 0; b < D / 16; ++b) {
              uint32_t o[16];
              tmem_ld16(ot + 16 * b, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(ot + 16 * b, o);
            }
          }
        }
        const float base = (ref == -INFINITY ? 0.f : ref) - kWeightBits;
        // the weights, over the scores
#pragma unroll
        for (int x = 0; x < kGroups; ++x) {
          const uint64_t c2 = pack2(cg[x], cg[x]), e2 = pack2(eg[x] - base, eg[x] - base);
          uint64_t sum = 0;
#pragma unroll
          for (int e = 0; e < PG; e += 2) {
            const int key = x * PG + e;
            float x0, x1;
            unpack2(fma2(pack2(__uint_as_float(v[key >> 5][key & 31]), __uint_as_float(v[key >> 5][(key & 31) + 1])), c2, e2),
                    x0, x1);
            x0 = ex2(x0);
            x1 = ex2(x1);
            sum = add2(sum, pack2(x0, x1));
            // the pair's halves in place, in the first half of its 32 scores' registers
            v[key >> 5][(key & 31) >> 1] = pack_f16x2(x0, x1);
            if ((key & 31) == 30) tmem_st16(sp + 16 * (key >> 5), *reinterpret_cast<uint32_t(*)[16]>(v[key >> 5]));
          }
          float s0, s1;
          unpack2(sum, s0, s1);
          l = fmaf(s0 + s1, tab[x * (PG / 16)].back, l);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + kPFull + q);
      }
      if (ok) ok = __all_sync(0xffffffffu, pwait(bars + kDone, 0u, failed));
      if (ok) {
        tc_fence_after();
        bool store = true;
        const float* others = nullptr;
        float* area = nullptr;
        constexpr int kPartFloats = 2 * kTileRows * (D + 2);
        const int row256 = q * kTileRows + r;
        float keep = 1.f;  // what the output is moved by when the zero pages' keys join the sum
        if (zero_sum > 0.f) {
          const float to = fmaxf(ref, zero_ref);
          keep = ref == -INFINITY ? 0.f : ex2(ref - to);
          l = l * keep + zero_sum * ex2(zero_ref - to + kWeightBits);
          ref = to;
        }
        if (CUT && parts > 1) {
          // this part's rows; the warp whose rows' last part this is puts them together
          area = plan.parts + (long long)(cut - part) * kPartFloats;  // of the block's first part
          float* mine = area + (long long)part * kPartFloats;
#pragma unroll 2
          for (int b = 0; b < D / 16; ++b) {
            uint32_t v[16];
            tmem_ld16(ot + 16 * b, v);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 4; ++e)
              __stcg(reinterpret_cast<float4*>(mine) + (4 * b + e) * (2 * kTileRows) + row256,
                     make_float4(__uint_as_float(v[4 * e]) * keep, __uint_as_float(v[4 * e + 1]) * keep,
                                 __uint_as_float(v[4 * e + 2]) * keep, __uint_as_float(v[4 * e + 3]) * keep));
          }
          __stcg(mine + 2 * kTileRows * D + row256, ref);
          __stcg(mine + 2 * kTileRows * (D + 1) + row256, l);
          __threadfence();
          __syncwarp();
          unsigned seen = 0;
          if (lane == 0) {
            unsigned* counter = plan.counters + 8 * (cut / plan.split) + warp;
            seen = atomicAdd(counter, 1u);
            if (seen == (unsigned)(parts - 1)) *counter = 0;
          }
          store = __shfl_sync(0xffffffffu, seen, 0) == (unsigned)(parts - 1);
          __threadfence();
          if (store) {
            others = area;
            keep = 1.f;  // it is in the parts
            ref = -INFINITY;
            for (int p = 0; p < parts; ++p)
              ref = fmaxf(ref, __ldcg(area + (long long)p * kPartFloats + 2 * kTileRows * D + row256));
            l = 0.f;
            for (int p = 0; p < parts; ++p) {
              const float* from = area + (long long)p * kPartFloats + 2 * kTileRows * D + row256;
              const float pr = __ldcg(from);
              if (pr != -INFINITY) l = fmaf(__ldcg(from + 2 * kTileRows), ex2(pr - ref), l);
            }
          }
        }
        if (store) {
          const float inv = keep * (l > 0.f ? __fdiv_rn(1.f, l) : l == 0.f ? 0.f : l);
          // through the rows' place in shared memory, where no product reads any more, so that whole rows leave (a
          // row a lane takes a pass of the cache's tags for each lane)
          constexpr int kLanes = D / 8, kStep = 32 / kLanes, kLoads = 32 / kStep;
          const uint32_t stage = sbase + L::kQ + q * L::kTile + 32 * (warp & 3) * (2 * D);
#pragma unroll 2
          for (int b = 0; b < D / 16; ++b) {
            uint32_t v[16], w[8];
            if (!CUT || others == nullptr) {
              tmem_ld16(ot + 16 * b, v);
              tmem_ld_wait();
            } else {
              float y[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = 0.f;
              for (int p = 0; p < parts; ++p) {
                const float* from = others + (long long)p * kPartFloats;
                const float pr = __ldcg(from + 2 * kTileRows * D + row256);
                const float f = pr == -INFINITY ? 0.f : ex2(pr - ref);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float4 x = __ldcg(reinterpret_cast<const float4*>(from) + (4 * b + e) * (2 * kTileRows) + row256);
                  y[4 * e] = fmaf(x.x, f, y[4 * e]);
                  y[4 * e + 1] = fmaf(x.y, f, y[4 * e + 1]);
                  y[4 * e + 2] = fmaf(x.z, f, y[4 * e + 2]);
                  y[4 * e + 3] = fmaf(x.w, f, y[4 * e + 3]);
                }
              }
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(y[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
              w[e] = pack_bf16x2(__uint_as_float(v[2 * e]) * inv, __uint_as_float(v[2 * e + 1]) * inv);
            sts_u32x4(stage + lane * (2 * D) + (((2 * b) ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
            sts_u32x4(stage + lane * (2 * D) + (((2 * b + 1) ^ (lane & 7)) << 4), w[4], w[5], w[6], w[7]);
          }
          __syncwarp();
          const long long row_dst = live ? (sq.row0 + i) * a.out_stride + (long long)row_head * D : -1;
#pragma unroll
          for (int x = 0; x < kLoads; ++x) {
            const int row = x * kStep + lane / kLanes;
            const long long at = __shfl_sync(0xffffffffu, row_dst, row);
            uint32_t w[4];
            lds_u32x4(stage + row * (2 * D) + (((lane % kLanes) ^ (row & 7)) << 4), w);
            if (at >= 0)
              *(reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at) + lane % kLanes) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
  } else if (warp < 12) {
    // ---------------------------------------------------------------- levels to halves
    // eight lanes of a phase: two rows, four pieces of one 64-value panel, so that their 32-byte results
    // lie in distinct banks
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    const int cw = warp - 8;
    const int piece = (lane & 3) | (kPieces == 8 ? ((lane >> 3) & 1) << 2 : 0);
    const int rw = kPieces == 8 ? ((lane >> 2) & 1) | ((lane >> 4) << 1) : lane >> 2;
    const int row = cw * kRowsWarp + rw;  // of a pass
    const uint32_t src = (uint32_t)(row * D + 16 * piece);
    // a pass is a multiple of eight rows on, so the swizzle is the same in each
    const uint32_t dst0 = (uint32_t)((piece >> 2) * L::kPanel + row * 128 + (((2 * (piece & 3)) ^ (row & 7)) << 4));
    const uint32_t dst1 = dst0 ^ 16u;
    auto convert = [&](uint32_t from, uint64_t* raw_full, uint64_t* raw_free, uint32_t to, uint64_t* full, int n,
                       int after) -> bool {
      bool ok = pwait(raw_full, (uint32_t)(n & 1), failed);
      if (!__all_sync(0xffffffffu, ok)) return false;
      uint32_t w[kPasses][4];
#pragma unroll
      for (int x = 0; x < kPasses; ++x) lds_u32x4(from + src + x * (4 * kRowsWarp * D), w[x]);
      ok = n < 2 || pwait(bars + kFree + (after & 1), (uint32_t)((after >> 1) & 1), failed);
      if (!__all_sync(0xffffffffu, ok)) return false;
#pragma unroll
      for (int x = 0; x < kPasses; ++x) {
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) q8_word_to_f16_levels(w[x][e], h[2 * e], h[2 * e + 1]);
        sts_u32x4(to + dst0 + x * (4 * kRowsWarp * 128), h[0], h[1], h[2], h[3]);
        sts_u32x4(to + dst1 + x * (4 * kRowsWarp * 128), h[4], h[5], h[6], h[7]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(full);
        // only now: the stores above have used every value read from the raw levels (an arrival right after
        // the loads can overtake them, and the next copy then lands under them)
        mbar_arrive(raw_free);
      }
      return true;
    };
    for (int n = 0; n < je - jb; ++n) {
      const int st = n & 1;
      if (!convert(sbase + L::kRawK, bars + kRawKFull, bars + kRawKFree, sbase + L::kK + st * L::kTile, bars + kKFull + st, n,
                   n - 2) ||
          !convert(sbase + L::kRawV, bars + kRawVFull, bars + kRawVFree, sbase + L::kV + st * L::kTile, bars + kVFull + st, n,
                   n - 1))
        break;
    }
  } else {
    // ---------------------------------------------------------------- products
    // One warp issues both tiles' in turn.  The tensor core takes them in order, so the scores of the next
    // keys may follow P V at once although they replace its P.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 12) {
      constexpr uint32_t id_s = idesc_f16_f32(kTileRows, kKeys, false);
      constexpr uint32_t id_o = idesc_f16_f32(kTileRows, D, true);
      // operands: the second tile, panel or stage is a fixed distance on (addresses in units of 16 bytes);
      // all of tensor memory is this CTA's, so its addresses begin at 0
      const uint32_t sb = __shfl_sync(0xffffffffu, sbase, 0);
      const uint64_t dq = smem_desc_sw128(sb + L::kQ), dk = smem_desc_sw128(sb + L::kK);
      const uint64_t dv = smem_desc_sw128_mn(sb + L::kV, L::kPanel);
      const uint32_t sbars = sb + L::kBars;
      auto scores = [&](int q, int n) {  // S of tile q and the n-th keys
        const uint64_t a0 = dq + (uint64_t)(q * (L::kTile >> 4)), b0 = dk + (uint64_t)((n & 1) * (L::kTile >> 4));
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t off = (uint64_t)(((k >> 2) * L::kPanel + (k & 3) * 32) >> 4);
          warp_mma((uint32_t)(q * kKeys), a0 + off, b0 + off, id_s, k > 0);
        }
        warp_commit(sbars + 8 * (kSFull + q));
      };
      const int keys = je - jb;
      bool ok = *tmem_slot == 0u && pwait(bars + kKFull, 0u, failed);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (q == 1 && n_tiles == 1) break;
        ok = __all_sync(0xffffffffu, ok && pwait(bars + kQFull + q, 0u, failed));
        if (!ok) break;
        tc_fence_after();
        scores(q, 0);
      }
      if (ok) warp_commit(sbars + 8 * kFree);
      // V of keys n and K of keys n + 1, which turn n needs
      auto ready = [&](int n) -> bool {
        return n >= keys || (pwait(bars + kVFull + (n & 1), (uint32_t)((n >> 1) & 1), failed) &&
                             (n + 1 >= keys || pwait(bars + kKFull + ((n + 1) & 1), (uint32_t)(((n + 1) >> 1) & 1), failed)));
      };
      ok = ok && ready(0);
#pragma unroll 1
      for (int n = 0; ok && n < keys; ++n) {
        const bool more = n + 1 < keys;
        const uint64_t v0 = dv + (uint64_t)((n & 1) * (L::kTile >> 4));
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          // between the two tiles' turns: what the next turn needs has long been under way
          if (q == 1) ok = ok && ready(n + 1);
          if (q == 1 && n_tiles == 1) break;
          ok = __all_sync(0xffffffffu, ok && pwait(bars + kPFull + q, (uint32_t)(n & 1), failed));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            warp_mma_ts((uint32_t)(256 + q * 128), (uint32_t)(q * kKeys + 8 * k), v0 + (uint64_t)(128 * k), id_o, (n | k) != 0);
          if (more) scores(q, n + 1);
        }
        if (ok && more) warp_commit(sbars + 8 * (kFree + ((n + 1) & 1)));
      }
      // every product of this warp is done when this arrives; nothing is in flight when the tensor memory goes
      warp_commit(sbars + 8 * kDone);
      if (!mbar_wait_bounded(bars + kDone, 0u) || !ok) *failed = 1;
    }
    __syncwarp();
    if (warp == 13) {
      // -------------------------------------------------------------- pages and their scales
      // lane g < 8 looks up the page of the tile's 16-key group g; the first of a page's lanes copies
      // this head's levels of it, one contiguous run
      const bool leader = lane < 8 && ((16 * lane) & (c.page_tokens - 1)) == 0;
      const uint32_t bytes = (uint32_t)(c.page_tokens * D);
      const long long page_stride = (long long)c.kv_heads * c.page_tokens * D;
      const int8_t* kbase = c.k + (long long)kvh * c.page_tokens * D;
      const int8_t* vbase = c.v + (long long)kvh * c.page_tokens * D;
      const int keys = je - jb;
      auto look = [&](int n) {  // -1 past the keys
        const int key = (jb + n) * kKeys + 16 * lane;
        return lane < 8 && n < keys && key < sq.len ? __ldg(page_row + (key >> c.page_shift)) : -1;
      };
      if (!hidden) id = page_of(id, jb * kKeys + 16 * lane);
      if (id >= 0) {
        gk = __ldg(c.k_scale + (long long)id * c.kv_heads + kvh);
        gv = __ldg(c.v_scale + (long long)id * c.kv_heads + kvh);
      }
      int copied_k = 0, copied_v = 0;
      for (int n = 0; n < keys; ++n) {
        const int next = look(n + 1);
        const bool copies = leader && id >= 0;
        const uint32_t total = bytes * (uint32_t)__popc(__ballot_sync(0xffffffffu, copies));
        bool ok = n == 0 || pwait(bars + kRawKFree, (uint32_t)((n - 1) & 1), failed);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (lane == 0) mbar_arrive_expect_tx(bars + kRawKFull, total);
        __syncwarp();
        if (copies) bulk_copy(sbase + L::kRawK + 16 * lane * D, kbase + id * page_stride, bytes, bars + kRawKFull);
        copied_k = n + 1;
        ok = n == 0 || pwait(bars + kRawVFree, (uint32_t)((n - 1) & 1), failed);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (lane == 0) mbar_arrive_expect_tx(bars + kRawVFull, total);
        __syncwarp();
        if (copies) bulk_copy(sbase + L::kRawV + 16 * lane * D, vbase + id * page_stride, bytes, bars + kRawVFull);
        copied_v = n + 1;
        // the slot's last readers were done before the levels of tile n - 1 were taken from shared memory
        const bool zero = gv < 0x1p-113f;  // (or no page)
        const uint32_t zeros = __ballot_sync(0xffffffffu, zero && id >= 0);
        if (lane < 8) {
          GroupScale gs;
          gs.ks = gk;
          gs.e = zero ? -INFINITY : log2f(gv);
          gs.back = zero ? 0.f : __frcp_rn(gv);
          gs.zeros = zeros;
          table[(n % kTableStages) * 8 + lane] = gs;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + kTableFull + n % kTableStages);
        id = page_of(next, (jb + n + 1) * kKeys + 16 * lane);
        gk = id >= 0 ? __ldg(c.k_scale + (long long)id * c.kv_heads + kvh) : 0.f;
        gv = id >= 0 ? __ldg(c.v_scale + (long long)id * c.kv_heads + kvh) : 0.f;
      }
      if (*failed) {
        // let the copies still in flight land before the shared memory is released
        if (copied_k > 0) mbar_wait_bounded(bars + kRawKFull, (uint32_t)((copied_k - 1) & 1), 400000000LL);
        if (copied_v > 0) mbar_wait_bounded(bars + kRawVFull, (uint32_t)((copied_v - 1) & 1), 400000000LL);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
    if (lane == 0 && *failed != 0) record_status(c.status, QMV_E_TIMEOUT);
  }
}

// How a call's blocks go over the SMs, by its bounds, in ns: about 1.55 us a tile of 128 keys for two row tiles, 1.35 us
// for one, 6 us more a wave of blocks, 14 us more a wave of cut ones (they write and read their parts).  Blocks that
// fill whole waves stay whole; the others, or all of a call with fewer blocks than SMs, are cut along the keys
// where that saves a tenth.  Measured, whole against cut, 32 heads over 8 of 128: 256 rows over 16384 tokens 213 against
// 73 us, 512 rows over 16384 212 against 123, 64 rows over 2048 34 against 24; 2048 rows over 16384 (256 blocks)
// 399 against 399, 640 rows over 2048 (80 blocks) 35 against 49.
struct Estimate {
  long long items;  // blocks of the grid before any cut, at most: exact for one sequence, else a block more for each
  long long whole, split, ns;
};
long long part_floats(const KvRef& c) { return 2LL * kTileRows * (c.head_dim + 2); }
Estimate estimate(const KvRef& c, const AttendArgs& a, const DeviceInfo& dev) {
  const long long group = a.heads / c.kv_heads, all = c.rows * group, block = 2 * kTileRows;
  const long long items = (c.n_seq == 1 ? (all + block - 1) / block : all / block + c.n_seq) * c.kv_heads;
  const long long span = a.window > 0 && (long long)a.window + c.max_rows < c.max_len ? a.window + c.max_rows : c.max_len;
  const long long rows = (all + c.n_seq - 1) / c.n_seq;  // of a sequence and head, on average
  const long long blocks = (long long)c.n_seq * c.kv_heads * ((rows + block - 1) / block);
  const long long tiles = (span + kKeys - 1) / kKeys, turn = rows > kTileRows ? 1550 : 1350, sms = dev.sm_count;
  Estimate best{items, items, 1, 3000 + (blocks + sms - 1) / sms * (tiles * turn + 6000)};
  // the last blocks of whole prompts are short ones: the order of the grid already evens them out
  if (blocks >= sms && 2LL * c.max_rows > span) return best;
  const long long whole = blocks / sms * sms, rest = blocks - whole, before = 3000 + whole / sms * (tiles * turn + 6000);
  const long long areas = (long long)(kPromptPartialBytes / sizeof(float)) / part_floats(c);
  const long long most = best.ns / 10 * 9;
  for (long long s = 2; s <= 16 && tiles >= s * kMinPart; ++s) {
    if (whole >= items || (items - whole) * s > areas || (items - whole) * 8 > kPromptCounters) break;
    const long long ns = before + (rest * s + sms - 1) / sms * ((tiles + s - 1) / s * turn + 14000);
    if (ns < most && ns < best.ns) best = Estimate{items, whole, s, ns};
  }
  return best;
}

template <int D, int PG, bool CUT>
cudaError_t launch_kernel(const KvRef& c, const AttendArgs& a, const DeviceInfo& dev, const SplitPlan& plan, long long grid,
                          cudaStream_t stream) {
  auto kern = attend_prompt_kernel<D, PG, CUT>;
  constexpr int kSmem = Smem<D>::kBytes;
  static std::mutex mu;
  static bool ready[64] = {};
  if (dev.device < 0 || dev.device >= 64 || grid > INT32_MAX) return cudaErrorInvalidValue;
  if ((size_t)kSmem > dev.smem_optin) return cudaErrorInvalidConfiguration;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev.device]) {
      const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (err != cudaSuccess) return err;
      ready[dev.device] = true;
    }
  }
  return launch_dependent(kern, dim3((unsigned)grid), kThreads, kSmem, stream, c, a, plan);
}

template <int D, int PG>
cudaError_t launch_dim(const KvRef& c, const AttendArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  const Estimate e = estimate(c, a, dev);
  Workspace ws;
  if (e.split == 1 || stream_prompt_workspace(dev, stream, &ws) != cudaSuccess)
    return launch_kernel<D, PG, false>(c, a, dev, SplitPlan{}, e.items, stream);
  return launch_kernel<D, PG, true>(c, a, dev, SplitPlan{(int)e.whole, (int)e.split, ws.counters, ws.partials},
                                    e.whole + (e.items - e.whole) * e.split, stream);
}

}  // namespace

// bfloat16 rows, heads of 64 or 128, where this kernel's estimated time is the shorter one; the kernel for few rows
// reads the keys once for each 16 rows (over the whole GPU about 2 ns for 32 keys of 16 rows), from about 9 us on.
// Measured, that kernel against this one, 32 heads over 8 of 128: one sequence of 2048 tokens, 64 rows 34 against
// 24 us, 1024 rows 256 against 35; 64 sequences of 4096 tokens, 4 rows each 140 against 207 us, 8 rows 258
// against 208, 16 rows 494 against 209; 4 prompts of 128 tokens 35 against 12 us.  The choice is the whole call's, by
// the average of its rows: one chunk of 256 rows among 63 single tokens of 4096 takes 205 us in one call and 33 + 95 in two.
bool attend_prompt_supported(const KvRef& c, const AttendArgs& a, bool x_bf16, const DeviceInfo& dev) {
  if (!x_bf16 || c.head_dim > 128) return false;
  const long long span = a.window > 0 && (long long)a.window + c.max_rows < c.max_len ? a.window + c.max_rows : c.max_len;
  const long long rows = (c.rows * (a.heads / c.kv_heads) + c.n_seq - 1) / c.n_seq;
  const long long there = 9000 + 2LL * c.n_seq * c.kv_heads * ((rows + 15) / 16) * ((span + 31) / 32);
  return estimate(c, a, dev).ns < there;
}

cudaError_t launch_attend_prompt(const KvRef& c, const AttendArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  if (c.page_tokens >= 64)
    return c.head_dim == 64 ? launch_dim<64, 64>(c, a, dev, stream) : launch_dim<128, 64>(c, a, dev, stream);
  return c.head_dim == 64 ? launch_dim<64, 16>(c, a, dev, stream) : launch_dim<128, 16>(c, a, dev, stream);
}

}  // namespace qmv
