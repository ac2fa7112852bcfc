// moe.cu -- a layer of experts with block-quantized weights, for a few tokens (blocks of up to 64).
//
//   E(t) = the `top` largest of token t's router logits (equal ones: the lower expert),  p = their softmax share,
//   h_e  = act(W1_e x_t) * (W3_e x_t),   out_t = scale * sum_{e in E(t)} p_e W2_e h_e.
//
// Two launches.  Every CTA of both works out the routing itself from the logits (a maximum over a warp's lanes `top` times
// a token): a launch of its own would cost more.  A unit is an expert with as many of its tokens as the 8 columns
// of an m16n8k16 MMA take: a bfloat16 activation is one column, an h of two or three parts two or four.  An expert that
// more tokens chose has more units, whose weights come from L2 after the first.
//   moe_up:   items of (unit, rows of W1 and the same rows of W3); a CTA's warps share an item's columns and meet in shared
//             memory, where gate and up become h, written as bfloat16 parts (hi, lo; three for float32 outputs).
//   moe_down: a cluster holds 32 rows of the output; its warps share the (unit, columns) stages of all units evenly, each
//             adds share * W2_e h_e into a tile of its own, and the tiles are added in a fixed order at the end.  Launched as a
//             dependent of moe_up: routing and the first weights are read while that one ends.
// Weights reach each warp through a ring of its own (cp.async, 32 rows of 128 bytes of quants a stage); levels enter the tensor core as exact
// bfloat16, a block's dot product is scaled in float32 (as in decode_mma.cu).
#include <cooperative_groups.h>

#include <mutex>

#include "qmv_common.cuh"
#include "qmv_internal.h"

namespace qmv {

namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTokens = 64;    // of a launch
constexpr int kExperts = QMV_MOE_MAX_EXPERTS;
constexpr int kTop = QMV_MOE_MAX_TOP;
constexpr int kCols = 8;       // columns of an MMA
constexpr int kUnits = kExperts + kTokens * kTop / 2;  // experts, and one more for each 2 tokens or more
constexpr int kRowsStage = 32;

// ------------------------------------------------------------------------------------------ routing
struct Routing {
  unsigned long long mask[kExperts];  // tokens of an expert
  unsigned long long bad;             // tokens whose logits hold NaN or +infinity
  float share[kTokens * kTop];
  uint16_t sel[kTokens * kTop];       // experts of a token, 0xffff: none
  uint16_t unit[kUnits];              // expert | pass << 8
  int units;
  int part[kWarps];
};

__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

// unit_cols: tokens of a unit
__device__ void route(Routing& r, const MoeParams& p, int unit_cols) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  for (int e = threadIdx.x; e < kExperts; e += kThreads) r.mask[e] = 0;
  if (threadIdx.x == 0) r.bad = 0;
  __syncthreads();
  for (int tok = wid; tok < p.tokens; tok += kWarps) {
    uint32_t key[kExperts / 32];
    float most = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kExperts / 32; ++i) {
      key[i] = 0;
      const int e = lane + 32 * i;
      if (e < p.experts) {
        const float l = __ldg(p.logits + tok * p.logits_stride + e);
        bad |= !(l < INFINITY);
        if (l > -INFINITY) key[i] = ordered(l);
        most = fmaxf(most, l);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    bad = __any_sync(0xffffffffu, bad);
    float sum = 0.f;
    if (!p.renorm) {
#pragma unroll
      for (int i = 0; i < kExperts / 32; ++i)
        if (key[i] != 0) sum += expf(unordered(key[i]) - most);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    float mine = 0.f;  // lane k: the share of the k-th
    for (int k = 0; k < p.top; ++k) {
      uint32_t best = 0;
      int at = 0;
#pragma unroll
      for (int i = 0; i < kExperts / 32; ++i)
        if (key[i] > best) best = key[i], at = lane + 32 * i;
      const uint32_t high = bad ? 0u : __reduce_max_sync(0xffffffffu, best);
      int e = 0xffff;
      if (high != 0) {
        e = (int)__reduce_min_sync(0xffffffffu, best == high ? (unsigned)at : 0xffffu);
        const float w = expf(unordered(high) - most);
        if (lane == k) mine = w;
        if (p.renorm) sum += w;
#pragma unroll
        for (int i = 0; i < kExperts / 32; ++i)
          if (e == lane + 32 * i) key[i] = 0;
        if (lane == 0) atomicOr(&r.mask[e], 1ull << tok);
      }
      if (lane == 0) r.sel[tok * p.top + k] = (uint16_t)e;
    }
    if (bad && lane == 0) atomicOr(&r.bad, 1ull << tok);
    if (lane < p.top) r.share[tok * p.top + lane] = bad ? NAN : mine == 0.f ? 0.f : __fdiv_rn(mine, sum);
  }
  __syncthreads();
  // units: experts in rising order, each with ceil(tokens / unit_cols) passes
  const int passes = (int)threadIdx.x < p.experts ? (__popcll(r.mask[threadIdx.x]) + unit_cols - 1) / unit_cols : 0;
  int upto = passes;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += u;
  }
  if (lane == 31) r.part[wid] = upto;
  __syncthreads();
  int all = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w == wid) upto += all;
    all += r.part[w];
  }
  for (int i = 0; i < passes; ++i) r.unit[upto - passes + i] = (uint16_t)(threadIdx.x | i << 8);
  if (threadIdx.x == 0) r.units = all;
  __syncthreads();
}

// A unit as a warp holds it: lane n < cols has column n's token, its row of h (token * top + place) and its share.
struct Unit {
  int expert, cols;
  int tok, slot;
  float share;
};
__device__ __forceinline__ Unit unit_of(const Routing& r, const MoeParams& p, int u, int unit_cols) {
  const int lane = threadIdx.x & 31;
  Unit c;
  c.expert = r.unit[u] & 255;
  const int pass = r.unit[u] >> 8;
  unsigned long long m = r.mask[c.expert];
  c.cols = min(__popcll(m) - unit_cols * pass, unit_cols);
  c.tok = c.slot = 0;
  c.share = 0.f;
  if (lane < c.cols) {
    for (int i = 0; i < unit_cols * pass + lane; ++i) m &= m - 1;
    c.tok = __ffsll((long long)m) - 1;
    c.slot = c.tok * p.top;
    while (r.sel[c.slot] != c.expert) ++c.slot;  // (it is there: the mask says so)
    c.share = r.share[c.slot];
  }
  return c;
}

// ------------------------------------------------------------------------------------------ stages
// 4, 8 or 16 bytes, or as many zeros.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool live) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(live ? BYTES : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Layout of a stage: q (32 rows of 128 bytes, their 16-byte pieces exchanged by row & 7), the rows' scales, then the
// activations of MMA columns (a column's values and 16 bytes, so that the 8 columns' words lie in different banks).
template <int WT, bool F16, bool XF32>
struct Stage {
  static constexpr int kChunk = WT == QMV_Q4_0 ? 256 : 128;  // weights of a row
  static constexpr int kQ = kRowsStage * 128;
  static constexpr int kScaleRow = kChunk / 32 * (F16 ? 2 : 4);
  static constexpr int kD = kRowsStage * kScaleRow;
  static constexpr int kXCol = kChunk * (XF32 ? 4 : 2) + 16;
  static __host__ __device__ int bytes(int mma_cols) { return kQ + kD + mma_cols * kXCol; }
};

// Rows row_a .. row_a + 15 of one matrix image and row_b .. row_b + 15 of another (or of the same), chunk c of `cols` columns.
template <int WT, bool F16>
__device__ __forceinline__ void load_weights(uint32_t stage, const uint8_t* qa, const uint8_t* da, const uint8_t* qb, const uint8_t* db,
                                             long long row_a, long long row_b, int c, int cols) {
  using S = Stage<WT, F16, false>;
  const int lane = threadIdx.x & 31;
  const long long row_bytes = WT == QMV_Q4_0 ? cols / 2 : cols;
  const int piece = lane & 7;
  const bool live = c * 128 + piece * 16 < row_bytes;
  const long long off = live ? (long long)c * 128 + piece * 16 : 0;
#pragma unroll
  for (int i = 0; i < kRowsStage / 4; ++i) {
    const int row = i * 4 + (lane >> 3);
    const uint8_t* src = row < 16 ? qa + (row_a + row) * row_bytes : qb + (row_b + row - 16) * row_bytes;
    copy_async<16>(stage + row * 128 + ((piece ^ (row & 7)) << 4), src + off, live);
  }
  // scales
  constexpr int kSize = F16 ? 2 : 4;
  const long long scale_bytes = cols / 32 * kSize;  // of a row
  const uint32_t sd = stage + S::kQ;
  if (cols % S::kChunk == 0) {
    const uint8_t* src = (lane < 16 ? da + (row_a + lane) * scale_bytes : db + (row_b + lane - 16) * scale_bytes) + c * S::kScaleRow;
    constexpr int kPiece = S::kScaleRow < 16 ? S::kScaleRow : 16;
#pragma unroll
    for (int i = 0; i < S::kScaleRow / kPiece; ++i)
      copy_async<kPiece>(sd + lane * S::kScaleRow + kPiece * i, src + kPiece * i, true);
  } else {  // rows on 4-byte boundaries (columns are a multiple of 64)
    constexpr int kWords = S::kScaleRow / 4;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int at = lane + 32 * i, row = at / kWords, word = at % kWords;
      const bool there = c * S::kScaleRow + 4 * word < scale_bytes;
      const uint8_t* src = (row < 16 ? da + (row_a + row) * scale_bytes : db + (row_b + row - 16) * scale_bytes) +
                           (there ? c * S::kScaleRow + 4 * word : 0);
      copy_async<4>(sd + row * S::kScaleRow + 4 * word, src, there);
    }
  }
}

// Chunk c of the activations of `n` tokens (lane k: the row of token k): token k's part p is MMA column k * SPAN + p, and lies
// p * plane elements after its first part.
template <typename S, int SPAN, int PARTS, bool XF32>
__device__ __forceinline__ void load_columns(uint32_t at, const void* x, long long plane, int row, int n, int c, int cols) {
  const int lane = threadIdx.x & 31;
  constexpr int kSize = XF32 ? 4 : 2;
  constexpr int kPieces = S::kChunk * kSize / 16;  // of a column: 16, 32 or 64
  for (int k = 0; k < n; ++k) {
    const long long base = (long long)__shfl_sync(0xffffffffu, row, k) * cols;
#pragma unroll
    for (int i = 0; i < (PARTS * kPieces + 31) / 32; ++i) {
      const int j = lane + 32 * i, part = j / kPieces, piece = j % kPieces;
      if (PARTS * kPieces % 32 != 0 && part >= PARTS) continue;
      const int v = c * S::kChunk + piece * (16 / kSize);  // the piece's first value
      const bool live = v < cols;
      copy_async<16>(at + (k * SPAN + part) * S::kXCol + piece * 16,
                     static_cast<const uint8_t*>(x) + (base + part * plane + (live ? v : 0)) * kSize, live);
    }
  }
}

// Three bfloat16 parts of two float32 values: together 24 bits.
__device__ __forceinline__ void split3(float a, float b, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = pack_bf16x2(a, b);
  const float ra = a - __uint_as_float(hi << 16), rb = b - __uint_as_float(hi & 0xffff0000u);
  mid = pack_bf16x2(ra, rb);
  lo = pack_bf16x2(ra - __uint_as_float(mid << 16), rb - __uint_as_float(mid & 0xffff0000u));
}

// One stage's products: acc[m] += the 16 x 8 products of row tile m (m = 0, 1) with the MMA columns.  live: this lane's
// column (lane / 4) is there.
template <int WT, bool F16, bool XF32>
__device__ __forceinline__ void consume(uint32_t stage, bool live, float (&acc)[2][4]) {
  using S = Stage<WT, F16, XF32>;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int lm = lane >> 3, lrow = (lane & 7) + ((lm & 1) << 3), lsub = lm >> 1, sw = lrow & 7;
  const uint32_t xs = stage + S::kQ + S::kD + (live ? g * S::kXCol : 0) + t * (XF32 ? 16 : 8);
  constexpr int kParts = XF32 ? 3 : 1;
#pragma unroll
  for (int bp = 0; bp < S::kChunk / 64; ++bp) {
    uint32_t w[2][4];
    if (WT == QMV_Q4_0) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
        ldmatrix_x4(w[m][0], w[m][1], w[m][2], w[m][3], stage + (16 * m + lrow) * 128 + (((2 * bp + lsub) ^ sw) << 4));
    }
    float d[2][2][2];  // [tile][row g, g + 8][block]
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t at = stage + S::kQ + (16 * m + 8 * h + g) * S::kScaleRow + bp * (F16 ? 4 : 8);
        if (F16) {
          const uint32_t v = lds_u32(at);
          d[m][h][0] = f16_bits_to_f32((uint16_t)(v & 0xFFFF));
          d[m][h][1] = f16_bits_to_f32((uint16_t)(v >> 16));
        } else {
          uint32_t a, b;
          lds_u32x2(at, a, b);
          d[m][h][0] = __uint_as_float(a);
          d[m][h][1] = __uint_as_float(b);
        }
      }
#pragma unroll
    for (int hb = 0; hb < 2; ++hb) {
      const int k = 2 * bp + hb;
      uint32_t b[kParts][2][2];  // [part][half block][pair]
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (XF32) {
          float v[4] = {0.f, 0.f, 0.f, 0.f};
          if (live) lds_f32x4(xs + (k * 32 + h * 16) * 4, v);
          split3(v[0], v[1], b[0][h][0], b[kParts / 3][h][0], b[kParts / 3 * 2][h][0]);
          split3(v[2], v[3], b[0][h][1], b[kParts / 3][h][1], b[kParts / 3 * 2][h][1]);
        } else {
          b[0][h][0] = b[0][h][1] = 0u;
          if (live) lds_u32x2(xs + (k * 32 + h * 16) * 2, b[0][h][0], b[0][h][1]);
        }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t a[2][4];  // [half block][fragment]
        if (WT == QMV_Q4_0) {
          q4_word_to_bf16_levels(w[m][2 * hb], a[0][0], a[0][2], a[1][0], a[1][2]);
          q4_word_to_bf16_levels(w[m][2 * hb + 1], a[0][1], a[0][3], a[1][1], a[1][3]);
        } else {
          uint32_t q[4];  // row g half 0, row g + 8 half 0, row g half 1, row g + 8 half 1
          ldmatrix_x4(q[0], q[1], q[2], q[3], stage + (16 * m + lrow) * 128 + (((2 * k + lsub) ^ sw) << 4));
          q8_word_to_bf16_levels(q[0], a[0][0], a[0][2]);
          q8_word_to_bf16_levels(q[1], a[0][1], a[0][3]);
          q8_word_to_bf16_levels(q[2], a[1][0], a[1][2]);
          q8_word_to_bf16_levels(q[3], a[1][1], a[1][3]);
        }
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int p = kParts - 1; p >= 0; --p)  // the small parts first
#pragma unroll
          for (int h = 0; h < 2; ++h)
            mma_bf16_16816(c, a[h][0], a[h][1], a[h][2], a[h][3], b[p][h][0], b[p][h][1], c);
        acc[m][0] = fmaf(d[m][0][hb], c[0], acc[m][0]);
        acc[m][1] = fmaf(d[m][0][hb], c[1], acc[m][1]);
        acc[m][2] = fmaf(d[m][1][hb], c[2], acc[m][2]);
        acc[m][3] = fmaf(d[m][1][hb], c[3], acc[m][3]);
      }
    }
  }
}

// ------------------------------------------------------------------------------------------ gate and up
constexpr int kRing = 2;

template <int WT, bool F16, bool XF32>
__global__ void __launch_bounds__(kThreads, 2) moe_up_kernel(const __grid_constant__ MoeParams p) {
  using S = Stage<WT, F16, XF32>;
  constexpr int kUnit = XF32 ? 4 : 8;  // tokens of a unit (float32 activations take twice the room)
  extern __shared__ __align__(1024) uint8_t smem[];
  Routing& r = *reinterpret_cast<Routing*>(smem);
  float* red = reinterpret_cast<float*>(smem + p.off_red);  // 32 rows x 8 columns a warp
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int stage_bytes = S::bytes(min(p.tokens, kUnit));
  const uint32_t ring = smem_u32(smem + p.off_ring) + wid * kRing * stage_bytes;
  griddep_wait();
  griddep_launch_dependents();
  route(r, p, kUnit);

  const int tiles = p.hidden / 16, chunks = (p.dim + S::kChunk - 1) / S::kChunk;
  const int tiles_item = kWarps / p.ks;
  const int items_unit = (tiles + tiles_item - 1) / tiles_item;
  const int items = r.units * items_unit;
  const int slice = wid % p.ks, tile_local = wid / p.ks;
  const int c0 = slice * chunks / p.ks, n = (slice + 1) * chunks / p.ks - c0;

  // the producer's place: stage j of the warp's columns of an item
  int pi = blockIdx.x, pj = 0, ps = 0;
  Unit pu{};
  int p_tile = 0;
  auto settle = [&]() {  // on to an item in which the warp has rows
    while (pi < items) {
      p_tile = pi % items_unit * tiles_item + tile_local;
      if (p_tile < tiles) break;
      pi += gridDim.x;
    }
    if (pi < items) pu = unit_of(r, p, pi / items_unit, kUnit);
  };
  settle();
  auto issue = [&]() {
    if (pi < items) {
      const uint32_t st = ring + ps * stage_bytes;
      const long long row = (long long)pu.expert * p.hidden + 16LL * p_tile;
      load_weights<WT, F16>(st, p.q1, p.d1, p.q3, p.d3, row, row, c0 + pj, p.dim);
      load_columns<S, 1, 1, XF32>(st + S::kQ + S::kD, p.x, 0, pu.tok, pu.cols, c0 + pj, p.dim);
      ps = ps + 1 == kRing ? 0 : ps + 1;
      if (++pj == n) {
        pj = 0;
        pi += gridDim.x;
        settle();
      }
    }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) issue();

  int cs = 0;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int tile = item % items_unit * tiles_item + tile_local;
    const Unit u = unit_of(r, p, item / items_unit, kUnit);
    float acc[2][4] = {};
    if (tile < tiles) {
      for (int j = 0; j < n; ++j) {
        __syncwarp();  // every lane is done with the slot that is filled next
        issue();
        copies_wait<kRing - 1>();
        __syncwarp();
        consume<WT, F16, XF32>(ring + cs * stage_bytes, g < u.cols, acc);
        cs = cs + 1 == kRing ? 0 : cs + 1;
      }
    }
    float* my = red + wid * (kRowsStage * kCols);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      *reinterpret_cast<float2*>(my + (16 * m + g) * kCols + 2 * t) = make_float2(acc[m][0], acc[m][1]);
      *reinterpret_cast<float2*>(my + (16 * m + g + 8) * kCols + 2 * t) = make_float2(acc[m][2], acc[m][3]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tiles_item * 16 * kCols; i += kThreads) {  // whole warps: tiles_item * 128 is a multiple of 32
      const int tl = i / (16 * kCols), col = i / 16 % kCols, row = i % 16;
      const int ht = item % items_unit * tiles_item + tl;
      const int slot = __shfl_sync(0xffffffffu, u.slot, col);
      if (col < u.cols && ht < tiles) {
        float gate = 0.f, up = 0.f;
        for (int k = 0; k < p.ks; ++k) {
          const float* part = red + (tl * p.ks + k) * (kRowsStage * kCols);
          gate += part[row * kCols + col];
          up += part[(16 + row) * kCols + col];
        }
        const float h = glu(p.act, gate, up);
        uint16_t* out = p.h + (long long)slot * p.hidden + 16 * ht + row;
        uint32_t hi, mid, lo;
        split3(h, 0.f, hi, mid, lo);
        if (!isfinite(h)) mid = lo = 0u;  // (infinity less itself)
        out[0] = (uint16_t)hi;
        out[p.h_plane] = (uint16_t)mid;
        if (p.parts > 2) out[2 * p.h_plane] = (uint16_t)lo;
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------------------------------ down
template <int WT, bool F16, int PARTS>
__global__ void __launch_bounds__(kThreads, 2) moe_down_kernel(const __grid_constant__ MoeParams p, int ranks) {
  using S = Stage<WT, F16, false>;
  constexpr int kSpan = PARTS == 2 ? 2 : 4;   // MMA columns of a token
  constexpr int kUnit = kCols / kSpan;        // tokens of a unit
  extern __shared__ __align__(1024) uint8_t smem[];
  Routing& r = *reinterpret_cast<Routing*>(smem);
  float* tiles = reinterpret_cast<float*>(smem + p.off_red);  // a warp's 32 rows x tokens
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int stage_bytes = S::bytes(min(p.tokens, kUnit) * kSpan);
  const uint32_t ring = smem_u32(smem + p.off_ring) + wid * kRing * stage_bytes;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank();
  const int row0 = (int)(blockIdx.x / ranks) * kRowsStage;
  // launched by moe_up after its own wait: what came before that, the logits and the weights among it, is complete
  route(r, p, kUnit);
  float* my = tiles + wid * kRowsStage * p.tokens;
  for (int i = lane; i < kRowsStage * p.tokens; i += 32) my[i] = 0.f;
  __syncwarp();

  const int chunks = (p.hidden + S::kChunk - 1) / S::kChunk;
  const int total = r.units * chunks, warps = ranks * kWarps, me = rank * kWarps + wid;
  const int s0 = (int)((long long)total * me / warps), s1 = (int)((long long)total * (me + 1) / warps);
  int ps = s0, slot_p = 0;
  Unit pu{};
  int p_unit = -1;
  auto weights = [&]() {
    const int u = ps / chunks, c = ps % chunks;
    if (u != p_unit) pu = unit_of(r, p, u, kUnit), p_unit = u;
    const long long row = (long long)pu.expert * p.dim + row0;
    load_weights<WT, F16>(ring + slot_p * stage_bytes, p.q2, p.d2, p.q2, p.d2, row, row + 16, c, p.hidden);
  };
  auto columns = [&]() {
    load_columns<S, kSpan, PARTS, false>(ring + slot_p * stage_bytes + S::kQ + S::kD, p.h, p.h_plane, pu.slot, pu.cols, ps % chunks, p.hidden);
    ++ps;
    slot_p = slot_p + 1 == kRing ? 0 : slot_p + 1;
  };
  static_assert(kRing == 2, "one stage's weights are asked for ahead of the wait");
  if (ps < s1) weights();
  griddep_wait();
  griddep_launch_dependents();
  if (ps < s1) columns();
  copies_commit();

  float acc[2][4] = {};
  int cs = 0, c_unit = -1;
  Unit u{};
  auto flush = [&]() {
    if (c_unit < 0) return;
    // a token's parts lie side by side: in this lane's two columns, and for three parts in its neighbour's
    const int col = 2 * t / kSpan;
    const int tok = __shfl_sync(0xffffffffu, u.tok, col);
    const float share = __shfl_sync(0xffffffffu, u.share, col);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v = acc[m][2 * h] + acc[m][2 * h + 1];
        if (PARTS == 3) v += __shfl_xor_sync(0xffffffffu, v, 1);
        if (col < u.cols && 2 * t % kSpan == 0) my[(16 * m + 8 * h + g) * p.tokens + tok] += share * v;
      }
#pragma unroll
    for (int m = 0; m < 2; ++m) acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.f;
  };
  for (int s = s0; s < s1; ++s) {
    __syncwarp();
    if (ps < s1) weights(), columns();
    copies_commit();
    const int uu = s / chunks;
    if (uu != c_unit) {
      flush();
      u = unit_of(r, p, uu, kUnit);
      c_unit = uu;
    }
    copies_wait<kRing - 1>();
    __syncwarp();
    consume<WT, F16, false>(ring + cs * stage_bytes, g / kSpan < u.cols && g % kSpan < PARTS, acc);
    cs = cs + 1 == kRing ? 0 : cs + 1;
  }
  flush();
  cl.sync();
  // the cluster's tiles: its CTAs share the sums, each in rank, then warp order
  const int values = kRowsStage * p.tokens;
  for (int i = rank * kThreads + threadIdx.x; i < values; i += ranks * kThreads) {
    const int row = i % kRowsStage, tok = i / kRowsStage;
    float sum = 0.f;
    for (int k = 0; k < ranks; ++k) {
      const float* o = cl.map_shared_rank(tiles, k);
      for (int w = 0; w < kWarps; ++w) sum += o[(w * kRowsStage + row) * p.tokens + tok];
    }
    sum *= p.scale;
    if (r.bad >> tok & 1) sum = NAN;
    const long long at = (long long)tok * p.dim + row0 + row;
    if (p.out_bf16)
      static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(sum);
    else
      static_cast<float*>(p.out)[at] = sum;
  }
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < p.tokens * p.top; i += kThreads) {
      if (p.ids != nullptr) p.ids[i] = r.sel[i] == 0xffff ? -1 : (int)r.sel[i];
      if (p.shares != nullptr) p.shares[i] = r.share[i];
    }
  }
  cl.sync();  // no CTA leaves while another reads its tiles
}

cudaError_t allow_smem(const void* kern, int device, size_t bytes) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

constexpr size_t round_up(size_t v, size_t to) { return (v + to - 1) / to * to; }

template <int WT, bool F16>
cudaError_t launch_up(MoeParams p, bool x_f32, const DeviceInfo& dev, cudaStream_t stream) {
  const int unit = x_f32 ? 4 : 8, cols = p.tokens < unit ? p.tokens : unit;
  const int stage = x_f32 ? Stage<WT, F16, true>::bytes(cols) : Stage<WT, F16, false>::bytes(cols);
  p.off_red = (int)round_up(sizeof(Routing), 128);
  p.off_ring = (int)round_up(p.off_red + kWarps * kRowsStage * kCols * 4, 1024);
  const size_t smem = p.off_ring + (size_t)kWarps * kRing * stage;
  const int chunk = Stage<WT, F16, false>::kChunk, chunks = (p.dim + chunk - 1) / chunk;
  p.ks = 1;
  while (p.ks < kWarps && 2 * p.ks <= chunks) p.ks *= 2;
  const int tiles_item = kWarps / p.ks;
  const long long units = (p.experts < p.tokens * p.top ? p.experts : p.tokens * p.top) + p.tokens * p.top / unit;
  const long long items = units * ((p.hidden / 16 + tiles_item - 1) / tiles_item);
  const long long slots = (long long)dev.sm_count * (2 * (smem + dev.smem_reserved) <= dev.smem_per_sm ? 2 : 1);
  auto kern = x_f32 ? moe_up_kernel<WT, F16, true> : moe_up_kernel<WT, F16, false>;
  cudaError_t err = allow_smem((const void*)kern, dev.device, smem);
  if (err != cudaSuccess) return err;
  return launch_dependent(kern, dim3((unsigned)(items < slots ? items : slots)), kThreads, smem, stream, p);
}

template <int WT, bool F16>
cudaError_t launch_down(MoeParams p, const DeviceInfo& dev, cudaStream_t stream) {
  const int span = p.parts == 2 ? 2 : 4, unit = kCols / span, cols = (p.tokens < unit ? p.tokens : unit) * span;
  const int stage = Stage<WT, F16, false>::bytes(cols);
  p.off_red = (int)round_up(sizeof(Routing), 128);
  p.off_ring = (int)round_up(p.off_red + (size_t)kWarps * kRowsStage * p.tokens * 4, 1024);
  const size_t smem = p.off_ring + (size_t)kWarps * kRing * stage;
  const int tiles = p.dim / kRowsStage;
  int ranks = 1;
  while (ranks < 8 && tiles * ranks * 2 <= 2 * dev.sm_count) ranks *= 2;
  auto kern = p.parts == 3 ? moe_down_kernel<WT, F16, 3> : moe_down_kernel<WT, F16, 2>;
  cudaError_t err = allow_smem((const void*)kern, dev.device, smem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
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
  return cudaLaunchKernelEx(&cfg, kern, p, ranks);
}

}  // namespace

size_t moe_scratch_bytes(int64_t tokens, int top, int hidden, bool out_bf16) {
  const size_t t = tokens < kTokens ? tokens : kTokens;
  return t * top * hidden * 2 * (out_bf16 ? 2 : 3);
}

cudaError_t launch_moe(const MoeArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  for (int64_t t0 = 0; t0 < a.tokens; t0 += kTokens) {
    MoeParams p{};
    p.tokens = (int)(a.tokens - t0 < kTokens ? a.tokens - t0 : kTokens);
    p.q1 = a.w1.q, p.d1 = a.w1.d, p.q3 = a.w3.q, p.d3 = a.w3.d, p.q2 = a.w2.q, p.d2 = a.w2.d;
    p.logits = a.logits + t0 * a.logits_stride;
    p.logits_stride = a.logits_stride;
    p.x = static_cast<const uint8_t*>(a.x) + t0 * a.dim * (a.x_bf16 ? 2 : 4);
    p.out = static_cast<uint8_t*>(a.out) + t0 * a.dim * (a.out_bf16 ? 2 : 4);
    p.out_bf16 = a.out_bf16;
    p.h = static_cast<uint16_t*>(a.scratch);
    p.h_plane = (long long)p.tokens * a.top * a.hidden;
    p.parts = a.out_bf16 ? 2 : 3;
    p.ids = a.ids == nullptr ? nullptr : a.ids + t0 * a.top;
    p.shares = a.shares == nullptr ? nullptr : a.shares + t0 * a.top;
    p.experts = a.experts;
    p.top = a.top;
    p.dim = a.dim;
    p.hidden = a.hidden;
    p.renorm = a.renorm;
    p.act = a.act;
    p.scale = a.scale;
    cudaError_t err;
    if (a.w1.wtype == QMV_Q4_0)
      err = a.w1.scale_f16 ? launch_up<QMV_Q4_0, true>(p, !a.x_bf16, dev, stream) : launch_up<QMV_Q4_0, false>(p, !a.x_bf16, dev, stream);
    else
      err = a.w1.scale_f16 ? launch_up<QMV_Q8_0, true>(p, !a.x_bf16, dev, stream) : launch_up<QMV_Q8_0, false>(p, !a.x_bf16, dev, stream);
    if (err != cudaSuccess) return err;
    if (a.w2.wtype == QMV_Q4_0)
      err = a.w2.scale_f16 ? launch_down<QMV_Q4_0, true>(p, dev, stream) : launch_down<QMV_Q4_0, false>(p, dev, stream);
    else
      err = a.w2.scale_f16 ? launch_down<QMV_Q8_0, true>(p, dev, stream) : launch_down<QMV_Q8_0, false>(p, dev, stream);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace qmv
