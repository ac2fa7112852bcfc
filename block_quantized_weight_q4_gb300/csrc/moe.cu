// moe.cu -- a layer of experts with block-quantized weights, for a few tokens (blocks of up to 64).
//
//   E(t) = the `top` largest of token t's router logits (equal ones: the lower expert),  p = their softmax share,
//   h_e  = act(W1_e x_t) * (W3_e x_t),   out_t = scale * sum_{e in E(t)} p_e W2_e h_e.
//
// Two launches.  Every CTA of the first works out the routing itself from the logits (a maximum over a warp's lanes `top` times
// a token: a launch of its own would cost more), and they leave it for the second together.  A unit is an expert with up to 4 of its tokens (2
// where they are float32: a value is two vectors then); an expert that more tokens chose has more units, whose weights come from L2 after
// the first.
//   moe_up:   items of (unit, 32 rows of W1 and of W3), each CTA a run of them; a CTA's warps share an item's columns and meet in
//             shared memory, where gate and up become h.
//   moe_down: a cluster holds 32 rows of the output; its warps share the (unit, columns) stages of all units evenly, each
//             adds share * W2_e h_e into a tile of its own, and the tiles are added in a fixed order at the end.
// Weights reach each warp through a ring of its own (cp.async, 32 rows of 128 bytes of quants a stage).
//
// Bound by the weights' bytes; below that by what comes before them: the routing, code that is fetched once, the fill of two pipelines
// (about 12 us of a call; so what runs once is small and no CTA runs code that the others do not: one CTA that alone left the routing
// cost 7 us).  TMA boxes in place of cp.async measured 53.9 against 52.7 us (1 token, two of 8 experts of 11008 x 4096) and 112 against
// 102 us (32 tokens, 8 of 128 experts of 768 x 2048).  GB300, Q4_0 with half scales, bfloat16 in and out: those two 46 us (152 MB) and 106 us
// (297 MB), in their long stretches 4.5 to 5.7 TB/s; 7 tokens over 16 Q8_0 experts of 1408 x 2048 41.5 us; 1 token, 4 of 32 of 512 x 1024
// 12.4 us.
//
// Products: m16n8k16 with IEEE halves.  Lane t of a row's four lanes takes a whole block of 32 weights (one or two 16-byte loads), so an
// MMA's k slots hold four different blocks; the columns are 2 vectors x those 4 blocks, and a lane's B values are
// zero but for its own block's column.  After the 8 MMAs of four blocks a lane holds the dot products of two blocks for two
// rows, scaled by the weights' and the activations' scales in float32: a quarter of the loads and scalings that
// one block an MMA would take, and 2 vectors fill the 8 columns.
//
// Levels, bfloat16 outputs: a Q4_0 nibble n in the lowest bits of a half is the subnormal number n 2^-24, in the next four bits n 2^-20:
// masks make MMA operands of a word of 8 nibbles, without arithmetic.  Values 16 .. 31 of a block's activations are kept as a 16th, and the
// level's -8 is taken from the block's sum: sum (n - 8) x = sum n x - 8 sum x.  The tensor core cuts a product's bits at a distance from the
// largest operands' exponents, and a subnormal operand's exponent is that of 2^-14: products lose 6 to 10 bits there, about 2^-18 of a
// result (2e-6 of the output's norm where it was left in float32, against 1.5e-7 with whole levels) and nothing beside a bfloat16's 2^-9.
// Float32 outputs and activations (WHOLE): levels as whole halves, a subtraction or an fma for two.  Those everywhere would be slower where
// the weights' bytes count: 1 token over two experts of 11008 x 4096 54.6 against 46.3 us, 32 over 128 of 768 x 2048 119 against 105 us
// (1 of 512 x 1024: no difference).  Q8_0 quants become exact halves by a magic number.
// An activation is a half after the power of two that brings its block's (32 values') largest into [2^14, 2^15): exact for bfloat16
// down to 2^-27 of the largest; float32 values and h are two halves, 22 bits.  (One half of h for bfloat16 outputs put 2e-4 of the output's
// norm beside the 1.6e-3 of the outputs' own rounding, and one output in ten on another bfloat16 than the formula's.  Its products
// were half as many: 44.4 and 95 us.)  A value's hi and lo have one factor, so their products meet in one MMA's sums; as vectors of their own
// they took 46.3 and 116 us.
#include <cooperative_groups.h>

#include <mutex>

#include "qmv_common.cuh"
#include "qmv_internal.h"

namespace qmv {

// What moe_down gets of it, in the call's scratch memory: this, the units as moe_down forms them, the shares of tokens * top places.
struct MoeTable {
  int units;
  uint32_t bad[2];
  int none;
};

namespace {

namespace cg = cooperative_groups;

constexpr int kMaxWarps = 16;
constexpr int kTokens = 64;    // of a launch
constexpr int kTokensWide = 48;  // for which moe_down's tiles leave room beside stages of units of 4
constexpr int kExperts = QMV_MOE_MAX_EXPERTS;
constexpr int kTop = QMV_MOE_MAX_TOP;
constexpr int kVectors = 4;    // of a unit: two to an MMA
constexpr int kParts = 2;      // vectors of a row of h, its halves: hi and lo
constexpr int kRowsStage = 32;

// ------------------------------------------------------------------------------------------ routing
// What moe_up's CTAs know of the routing, in shared memory; the arrays after it have the lengths that the call bounds.
struct Routing {
  uint32_t mask[2][kExperts];    // tokens of an expert, 32 a word
  uint32_t bad[2];               // tokens whose logits hold NaN or +infinity
  int units;
  int part[kMaxWarps];
  uint16_t base[kExperts];       // an expert's first unit
  uint16_t sel[kTokens * kTop];  // experts of a token, 0xffff: none
};
struct Units {
  uint2* entry;    // a unit's tokens: four of 16 bits, token << 10 | token * top + place
  uint16_t* head;  // expert | tokens << 8
  static __host__ __device__ int bytes(int n) { return n * 8 + (n * 2 + 7) / 8 * 8; }
  __device__ __forceinline__ Units(uint8_t* at, int n) : entry(reinterpret_cast<uint2*>(at)), head(reinterpret_cast<uint16_t*>(at + n * 8)) {}
};
static_assert(kTokens * kTop <= 1024 && kTokens <= 64, "a token and its place in 16 bits");
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

// The experts of the tokens that this warp routes, and their shares.  (Small rather than unrolled: code that runs once a launch costs what
// it takes to fetch.)
template <int W>
__device__ __forceinline__ void choose(Routing& r, const MoeParams& p, float* share) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  constexpr int kEach = kExperts / 32;
#pragma unroll 1
  for (int tok = wid; tok < p.tokens; tok += W) {
    uint32_t key[kEach], best = 0;
    bool bad = false;
    const float* logits = p.logits + tok * p.logits_stride + lane;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      float l = -INFINITY;
      if (lane + 32 * i < p.experts) l = __ldg(logits + 32 * i);
      bad |= !(l < INFINITY);
      key[i] = l > -INFINITY ? ordered(l) : 0u;
      best = max(best, key[i]);
    }
    bad = __any_sync(0xffffffffu, bad);
    const uint32_t high0 = __reduce_max_sync(0xffffffffu, best);
    const float most = high0 != 0 ? unordered(high0) : 0.f;
    float sum = 0.f;
    if (!p.renorm)
#pragma unroll
      for (int i = 0; i < kEach; ++i) sum += key[i] != 0 ? expf(unordered(key[i]) - most) : 0.f;
    uint32_t mine = 0u;  // lane k: the k-th's key
#pragma unroll 1
    for (int k = 0; k < p.top; ++k) {
      // the lane's best: the larger key, then the lower expert
      int at = lane;
      best = key[0];
#pragma unroll
      for (int i = 1; i < kEach; ++i) {
        at = key[i] > best ? lane + 32 * i : at;
        best = max(best, key[i]);
      }
      const uint32_t high = bad ? 0u : __reduce_max_sync(0xffffffffu, best);
      const int e = (int)__reduce_min_sync(0xffffffffu, best == high && high != 0 ? (unsigned)at : 0xffffu);
      mine = lane == k ? high : mine;
#pragma unroll
      for (int i = 0; i < kEach; ++i) key[i] = e == lane + 32 * i ? 0u : key[i];
      if (lane == 0) r.sel[tok * p.top + k] = (uint16_t)e;
    }
    if (bad && lane == 0) atomicOr(&r.bad[tok >> 5], 1u << (tok & 31));
    const float w = mine != 0 ? expf(unordered(mine) - most) : 0.f;
    float total = p.renorm ? w : sum;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane < p.top) share[tok * p.top + lane] = bad ? NAN : w == 0.f ? 0.f : __fdiv_rn(w, total);
  }
}

// The tokens' experts, and the experts' tokens.  W: the CTA's warps (8 or more: a thread for each expert).
template <int W>
__device__ __forceinline__ void route(Routing& r, const MoeParams& p, float* share) {
  for (int e = threadIdx.x; e < 2 * kExperts; e += 32 * W) r.mask[0][e] = 0u;
  if (threadIdx.x < 2) r.bad[threadIdx.x] = 0u;
  __syncthreads();
  choose<W>(r, p, share);
  __syncthreads();
  for (int i = threadIdx.x; i < p.tokens * p.top; i += 32 * W) {
    const int x = r.sel[i], tok = i / p.top;
    if (x != 0xffff) atomicOr(&r.mask[tok >> 5][x], 1u << (tok & 31));
  }
  __syncthreads();
}
// The units of up to unit_cols tokens: experts in rising order, an expert's tokens in theirs.
template <int W>
__device__ __forceinline__ void form_units(Routing& r, const Units& units, const MoeParams& p, int unit_cols) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int e = threadIdx.x;
  int tokens = e < p.experts ? __popc(r.mask[0][e]) + __popc(r.mask[1][e]) : 0;
  const int passes = (tokens + unit_cols - 1) / unit_cols;
  int upto = passes;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += u;
  }
  if (lane == 31) r.part[wid] = upto;
  __syncthreads();
  int all = 0;
#pragma unroll 1
  for (int w = 0; w < W; ++w) {
    const int n = r.part[w];
    upto += w < wid ? n : 0;
    all += n;
  }
  if (e < p.experts) r.base[e] = (uint16_t)(upto - passes);
  for (int i = upto - passes; i < upto; ++i, tokens -= unit_cols) units.head[i] = (uint16_t)(e | min(tokens, unit_cols) << 8);
  if (threadIdx.x == 0) r.units = all;
  __syncthreads();
  for (int i = threadIdx.x; i < p.tokens * p.top; i += 32 * W) {
    const int x = r.sel[i];
    if (x == 0xffff) continue;
    const int tok = i / p.top;
    const uint32_t before = (1u << (tok & 31)) - 1u;
    const int place = tok < 32 ? __popc(r.mask[0][x] & before) : __popc(r.mask[0][x]) + __popc(r.mask[1][x] & before);
    reinterpret_cast<uint16_t*>(units.entry + r.base[x] + place / unit_cols)[place % unit_cols] = (uint16_t)(tok << 10 | i);
  }
  __syncthreads();
}

// A unit as a warp holds it: lane n < cols has token n of it and that token's row of h (token * top + place).
struct Unit {
  int expert, cols;
  int tok, slot;
};
__device__ __forceinline__ Unit unit_of(const Units& units, int u) {
  const int lane = threadIdx.x & 31;
  const int head = units.head[u];
  Unit c;
  c.expert = head & 255;
  c.cols = head >> 8;
  const int entry = lane < c.cols ? reinterpret_cast<const uint16_t*>(units.entry + u)[lane] : 0;
  c.tok = entry >> 10;
  c.slot = entry & 1023;
  return c;
}
// An even share of n for each of `of`: the first of share i.
__device__ __forceinline__ int share_of(int n, int i, int of) {
  const int each = n / of, more = n - each * of;
  return i * each + min(i, more);
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

// Layout of a stage: q (32 rows of 128 bytes), then the rows' scales.  A row's 16-byte pieces are exchanged between even and
// odd rows, so that the 16-byte loads of two rows' four blocks lie in different banks.
template <int WT, bool F16>
struct Stage {
  static constexpr int kChunk = WT == QMV_Q4_0 ? 256 : 128;  // weights of a row
  static constexpr int kBlocks = kChunk / 32;
  static constexpr int kTurn = WT == QMV_Q4_0 ? 4 : 1;       // what an odd row's piece numbers are exchanged by
  static constexpr int kQ = kRowsStage * 128;
  static constexpr int kScaleRow = kBlocks * (F16 ? 2 : 4);
  static constexpr int kBytes = kQ + kRowsStage * kScaleRow;
  // a vector's chunk: its blocks' halves, 64 of 80 bytes a block, so that the lanes that read four blocks lie in different banks.
  // Then for each block what a sum of products is multiplied by at the end, and what is taken off it first.
  static constexpr int kBlock = 80;
  static constexpr int kVector = kBlocks * kBlock;
  static __host__ __device__ constexpr int columns(int vectors, int factors) { return vectors * kVector + factors * kBlocks * 8; }
};

// Where a lane reads a stage's rows: 16 rows of one matrix image and 16 of another (or of the same, at another place).  Moving to
// another chunk or 16 rows further is an offset to all of them.
template <int WT, bool F16>
struct Rows {
  using S = Stage<WT, F16>;
  const uint8_t *qa, *qb;  // this lane's first piece (lane % 4, and the fourth after it) of rows lane / 4 (and 8 further) of both
  const uint8_t *da, *db;  // the scales of the rows' first blocks: of row lane % 16 (whole chunks), else of row 0
  __device__ __forceinline__ void set(const uint8_t* q_a, const uint8_t* d_a, const uint8_t* q_b, const uint8_t* d_b, long long row_a,
                                      long long row_b, int cols) {
    const int lane = threadIdx.x & 31;
    const long long row_bytes = WT == QMV_Q4_0 ? cols / 2 : cols, scale_bytes = cols / 32 * (F16 ? 2 : 4);
    qa = q_a + (row_a + (lane >> 2)) * row_bytes + (lane & 3) * 16;
    qb = q_b + (row_b + (lane >> 2)) * row_bytes + (lane & 3) * 16;
    const int row = cols % S::kChunk == 0 ? lane & 15 : 0;
    da = d_a + (row_a + row) * scale_bytes;
    db = d_b + (row_b + row) * scale_bytes;
  }
  // Chunk c of the rows `down` rows further.
  __device__ __forceinline__ void load(uint32_t stage, int c, int down, int cols) const {
    const int lane = threadIdx.x & 31, piece = lane & 3;
    const int row_bytes = WT == QMV_Q4_0 ? cols / 2 : cols, scale_bytes = cols / 32 * (F16 ? 2 : 4);
    const long long off = (long long)down * row_bytes + c * 128;
    const uint8_t* from[4] = {qa + off, qa + off + 8 * row_bytes, qb + off, qb + off + 8 * row_bytes};
    // piece numbers are exchanged by the row's lowest bit
    const uint32_t odd = (lane >> 2 & 1) * S::kTurn;
    const uint32_t to = stage + (lane >> 2) * 128, near = (piece ^ odd) << 4, far = ((piece + 4) ^ odd) << 4;
    if ((c + 1) * 128 <= row_bytes) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        copy_async<16>(to + i * 1024 + near, from[i], true);
        copy_async<16>(to + i * 1024 + far, from[i] + 64, true);
      }
    } else {  // the row ends in this chunk: zeros after it
      const int left = row_bytes - c * 128 - piece * 16;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        copy_async<16>(to + i * 1024 + near, left > 0 ? from[i] : qa, left > 0);
        copy_async<16>(to + i * 1024 + far, left > 64 ? from[i] + 64 : qa, left > 64);
      }
    }
    const uint32_t sd = stage + S::kQ;
    const long long s_off = (long long)down * scale_bytes + c * S::kScaleRow;
    if (cols % S::kChunk == 0) {
      const uint8_t* src = (lane < 16 ? da : db) + s_off;
      constexpr int kPiece = S::kScaleRow < 16 ? S::kScaleRow : 16;
#pragma unroll
      for (int i = 0; i < S::kScaleRow / kPiece; ++i) copy_async<kPiece>(sd + lane * S::kScaleRow + kPiece * i, src + kPiece * i, true);
    } else {  // rows on 4-byte boundaries (columns are a multiple of 64)
      constexpr int kWords = S::kScaleRow / 4;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int at = lane + 32 * i, row = at / kWords, word = at % kWords;
        const bool there = c * S::kScaleRow + 4 * word < scale_bytes;
        const uint8_t* src = (row < 16 ? da : db) + (long long)(row & 15) * scale_bytes + s_off + 4 * word;
        copy_async<4>(sd + row * S::kScaleRow + 4 * word, there ? src : (row < 16 ? da : db), there);
      }
    }
  }
};

// The power of two that brings a block's largest magnitude into [2^14, 2^15), and its inverse; at most 2^126 (a block below 2^-112 stays below
// 2^14 then, its values multiples of 2^-23), so that both are normal.  1 for zeros, infinity and NaN.
__device__ __forceinline__ void block_scale(float amax, float& up, float& down) {
  const int e = (int)(__float_as_uint(amax) >> 23);
  const int scale = amax == 0.f || e == 255 ? 127 : min(268 - e, 253);
  up = __uint_as_float((uint32_t)scale << 23);
  down = __uint_as_float((uint32_t)(254 - scale) << 23);
}

// Eight values of a block of 32 (elements 8 piece ..) that four neighbouring lanes hold, as halves at the power of two that brings the block's
// largest into [2^14, 2^15): hi, and with LO what hi leaves (11 more bits).  For Q4_0 in the order in which masks take a word's nibbles (0, 2,
// 1, 3 of each four), the block's second half as a 16th (!WHOLE).  off: what is taken off the products'
// sum; mul: what it is multiplied by, after the weights' scale (before it, or with the levels' 2^24, it would pass float32's range).
template <int WT, bool LO, bool WHOLE>
__device__ __forceinline__ void to_halves(const float (&v)[8], int piece, uint32_t (&hi)[4], uint32_t (&lo)[4], float& mul, float& off) {
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  float up, down;
  block_scale(amax, up, down);
  static_assert(WHOLE || !LO, "two halves are for whole levels");
  constexpr bool kBits = WT == QMV_Q4_0 && !WHOLE;
  const float part = kBits && piece >= 2 ? 0.0625f : 1.f, back = kBits && piece >= 2 ? 16.f : 1.f;
  float sum = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int i = WT == QMV_Q4_0 ? (e & 2) * 2 + (e & 1) : 2 * e, j = WT == QMV_Q4_0 ? i + 2 : i + 1;
    const float a = v[i] * up * part, b = v[j] * up * part;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(hi[e]) : "f"(b), "f"(a));
    const float ha = __half2float(__ushort_as_half((unsigned short)(hi[e] & 0xffffu)));
    const float hb = __half2float(__ushort_as_half((unsigned short)(hi[e] >> 16)));
    sum += ha + hb;
    if (LO) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo[e]) : "f"(b - hb), "f"(a - ha));
  }
  mul = down;
  off = 0.f;
  if (kBits) {
    sum *= back;
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    off = 8.f * sum;
  }
}

// The nibbles of a word's bytes 0 and 2 as two halves: the low ones and the high ones; WHOLE: levels, else bits (see above).
template <bool WHOLE>
__device__ __forceinline__ uint32_t low_levels(uint32_t w) {
  const uint32_t n = w & 0x000F000Fu;
  return WHOLE ? f16x2_sub(n | 0x64006400u, 0x64086408u) : n;  // (1024 + n) - 1032
}
template <bool WHOLE>
__device__ __forceinline__ uint32_t high_levels(uint32_t w) {
  const uint32_t n = w & 0x00F000F0u;
  if (!WHOLE) return n;
  return f16x2_fma(n | 0x64006400u, 0x2C002C00u, 0xD480D480u);  // (1024 + 16 n) / 16 - 72
}

// Where a lane reads B from: b its column (its vector and block of the first four blocks), moving by `step` from set to set, by `group` from
// four blocks to the next and by `part` from a vector's hi to its lo (all 0 at zeros, for lanes without a column); xs the vector's factors
// of the lane's two blocks, moving by xs_step from set to set.
struct Columns {
  uint32_t b, step, group, part, xs, xs_step;
};

// One stage's products: acc[m][set] += what row tile m (rows g and g + 8 of it) gives for this lane's two blocks and vector.  PARTS 2: of a
// vector's hi and lo, which have one factor; in a sum each (each MMA cuts what it adds to: with both in one, float32 outputs were off by
// 3.4e-7 of their norm in place of 1.7e-7) but for levels as bits.
template <int WT, bool F16, bool WHOLE, int SETS, int PARTS>
__device__ __forceinline__ void consume(uint32_t stage, const Columns& at, float (&acc)[2][2][2]) {
  using S = Stage<WT, F16>;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  constexpr int kGroups = S::kBlocks / 4;
  constexpr int kPieces = WT == QMV_Q4_0 ? 1 : 2;  // of 16 bytes, of a block
  constexpr bool kBits = WT == QMV_Q4_0 && !WHOLE;
  constexpr int kSums = kBits ? 1 : PARTS;
  // this lane's piece of row g: the other four pieces (Q4_0), or the other one of two (Q8_0), lie where the exchange puts them
  const uint32_t near = ((t * kPieces) ^ ((g & 1) * S::kTurn)) << 4;
  const uint32_t q0 = stage + g * 128 + near, q1 = stage + g * 128 + (near ^ (WT == QMV_Q4_0 ? 64 : 16));
  const uint32_t d0 = stage + S::kQ + g * S::kScaleRow + 2 * (t & 1) * (F16 ? 2 : 4);
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    float c[2][SETS * kSums][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int v = 0; v < SETS * kSums; ++v) c[m][v][0] = c[m][v][1] = c[m][v][2] = c[m][v][3] = 0.f;
    uint32_t q[2][2][4 * kPieces];  // [tile][row g, g + 8][word]
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          uint32_t w[4];
          lds_u32x4(((WT == QMV_Q4_0 ? i : j) == 0 ? q0 : q1) + (16 * m + 8 * h) * 128, w);
#pragma unroll
          for (int k = 0; k < 4; ++k) q[m][h][4 * j + k] = w[k];
        }
    // eight elements of a block at a time: one load of B (two for Q4_0, whose words hold elements 16 apart)
#pragma unroll
    for (int j = 0; j < 2 * kPieces; ++j) {
      uint32_t x[SETS * PARTS][2][4];  // [set, hi and lo][first, elements 16 further][halves]
#pragma unroll
      for (int v = 0; v < SETS * PARTS; ++v) {
        const uint32_t from = at.b + v / PARTS * at.step + v % PARTS * at.part + i * at.group + j * 16;
        lds_u32x4(from, x[v][0]);
        if (WT == QMV_Q4_0) lds_u32x4(from + 32, x[v][1]);
      }
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t wg = q[m][0][2 * j + k], wh = q[m][1][2 * j + k];
          if (WT == QMV_Q4_0) {
            // nibbles of bytes 0 and 2, then of bytes 1 and 3
            const uint32_t sg = wg >> 8, sh = wh >> 8;
            const uint32_t lo[4] = {low_levels<WHOLE>(wg), low_levels<WHOLE>(wh), low_levels<WHOLE>(sg), low_levels<WHOLE>(sh)};
            const uint32_t hi[4] = {high_levels<WHOLE>(wg), high_levels<WHOLE>(wh), high_levels<WHOLE>(sg), high_levels<WHOLE>(sh)};
#pragma unroll
            for (int v = 0; v < SETS * PARTS; ++v) {
              float(&sum)[4] = c[m][v * kSums / PARTS];
              mma_f16_16816(sum, lo[0], lo[1], lo[2], lo[3], x[v][0][2 * k], x[v][0][2 * k + 1], sum);
              mma_f16_16816(sum, hi[0], hi[1], hi[2], hi[3], x[v][1][2 * k], x[v][1][2 * k + 1], sum);
            }
          } else {
            uint32_t g01, g23, h01, h23;
            q8_word_to_f16_levels(wg, g01, g23);
            q8_word_to_f16_levels(wh, h01, h23);
#pragma unroll
            for (int v = 0; v < SETS * PARTS; ++v) {
              float(&sum)[4] = c[m][v * kSums / PARTS];
              mma_f16_16816(sum, g01, h01, g23, h23, x[v][0][2 * k], x[v][0][2 * k + 1], sum);
            }
          }
        }
    }
    // columns 2 t and 2 t + 1: vector t / 2 of the set, blocks 2 (t & 1) and the next
    float f[SETS][4];  // multiplied by, taken off before; of both blocks
#pragma unroll
    for (int v = 0; v < SETS; ++v) lds_f32x4(at.xs + v * at.xs_step + i * 32, f[v]);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t from = d0 + (16 * m + 8 * h) * S::kScaleRow + 4 * i * (F16 ? 2 : 4);
        float2 d;
        if (F16) {
          const uint32_t u = lds_u32(from);
          d = __half22float2(*reinterpret_cast<const __half2*>(&u));
        } else {
          uint32_t u0, u1;
          lds_u32x2(from, u0, u1);
          d = make_float2(__uint_as_float(u0), __uint_as_float(u1));
        }
#pragma unroll
        for (int v = 0; v < SETS; ++v) {
          float s0 = c[m][v * kSums][2 * h], s1 = c[m][v * kSums][2 * h + 1];
          if (kSums == 2) s0 += c[m][v * kSums + kSums - 1][2 * h], s1 += c[m][v * kSums + kSums - 1][2 * h + 1];
          if (kBits) s0 = fmaf(s0, 0x1p24f, -f[v][1]), s1 = fmaf(s1, 0x1p24f, -f[v][3]);
          acc[m][v][h] = fmaf(s0 * d.x, f[v][0], fmaf(s1 * d.y, f[v][2], acc[m][v][h]));
        }
      }
  }
}

__device__ __forceinline__ void wait_ring(int ring) {  // all but the newest ring - 1 groups of copies have landed
  if (ring == 2)
    copies_wait<1>();
  else if (ring == 3)
    copies_wait<2>();
  else
    copies_wait<3>();
}

// A unit's columns at `columns`: PARTS halves of each of up to `most` vectors, then the vectors' factors; `zeros`: 128 bytes of zeros.
template <typename S, int PARTS>
__device__ __forceinline__ Columns columns_of(uint32_t columns, uint32_t zeros, int most) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int v = g >> 2;
  const bool mine = (g & 3) == t && v < most;
  Columns c;
  c.b = mine ? columns + v * PARTS * S::kVector + t * S::kBlock : zeros;
  c.step = mine && 2 + v < most ? 2 * PARTS * S::kVector : 0;
  c.group = mine ? 4 * S::kBlock : 0;
  c.part = mine ? S::kVector : 0;
  const int sv = t >> 1;
  c.xs = sv < most ? columns + most * PARTS * S::kVector + sv * S::kBlocks * 8 + 2 * (t & 1) * 8 : zeros;
  c.xs_step = 2 + sv < most ? 2 * S::kBlocks * 8 : 0;  // (what is read for a vector that is not there goes nowhere)
  return c;
}

// ------------------------------------------------------------------------------------------ gate and up
// A warp's columns of chunk c, converted: `vectors` halves of up to kVectors vectors, then their scales, at `to`.
template <typename S, int WT, bool XF32, bool WHOLE>
__device__ __forceinline__ void convert_columns(uint8_t* to, int max_vectors, const void* x, const Unit& u, int c, int cols) {
  const int lane = threadIdx.x & 31;
  constexpr int kPieces = S::kChunk / 8;  // of a token
  float2* factors = reinterpret_cast<float2*>(to + max_vectors * S::kVector);
#pragma unroll 1
  for (int i = 0; i < u.cols * kPieces; i += 32) {
    const int k = (i + lane) / kPieces, piece = (i + lane) % kPieces;
    const int tok = __shfl_sync(0xffffffffu, u.tok, k & 31);
    const bool in = k < u.cols;
    const int at = c * S::kChunk + 8 * piece;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
    if (in && at < cols) {
      if (XF32) {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(x) + (long long)tok * cols + at);
        const float4 a = __ldg(f), b = __ldg(f + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
      } else {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + (long long)tok * cols + at));
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[2 * e] = __uint_as_float(ww[e] << 16), v[2 * e + 1] = __uint_as_float(ww[e] & 0xffff0000u);
      }
    }
    uint32_t hi[4], lo[4];
    float mul, off;
    to_halves<WT, XF32, WHOLE>(v, piece & 3, hi, lo, mul, off);
    if (in) {
      const int vec = XF32 ? 2 * k : k;
      uint8_t* at16 = to + vec * S::kVector + (piece >> 2) * S::kBlock + (piece & 3) * 16;
      *reinterpret_cast<uint4*>(at16) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      if (XF32) *reinterpret_cast<uint4*>(at16 + S::kVector) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      if ((piece & 3) == 0) {
        factors[vec * S::kBlocks + (piece >> 2)] = make_float2(mul, off);
        if (XF32) factors[(vec + 1) * S::kBlocks + (piece >> 2)] = make_float2(mul, off);
      }
    }
  }
}

constexpr int kUpWarps = 16, kUpThreads = kUpWarps * 32;

template <int WT, bool F16, bool XF32, bool WHOLE>
__global__ void __launch_bounds__(kUpThreads, 1) moe_up_kernel(const __grid_constant__ MoeParams p) {
  using S = Stage<WT, F16>;
  constexpr int kUnit = XF32 ? kVectors / 2 : kVectors;  // tokens of a unit at most
  extern __shared__ __align__(1024) uint8_t smem[];
  Routing& r = *reinterpret_cast<Routing*>(smem);
  float* red = reinterpret_cast<float*>(smem + p.off_red);  // a warp's gate and up: [token][gate, up][32 rows]
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int max_vectors = min(p.tokens, p.unit) * (XF32 ? 2 : 1);
  const uint32_t ring = smem_u32(smem + p.off_ring) + wid * p.ring * S::kBytes;
  const int cache_bytes = S::columns(max_vectors, max_vectors);
  uint8_t* cache = smem + p.off_cols + wid * p.cached * cache_bytes;  // the warp's columns, of p.cached chunks
  griddep_wait();
  griddep_launch_dependents();
  if (threadIdx.x < 32) reinterpret_cast<uint32_t*>(smem + p.off_zero)[threadIdx.x] = 0u;
  const Units units(smem + p.off_units, p.max_units);
  // The CTAs leave the routing for moe_down, in units of its own size, and the call's ids and shares: each a part (one CTA by itself would
  // hold all others up, for code that it alone fetches).  The rings' room is free as yet.
  float* share = reinterpret_cast<float*>(smem + p.off_ring);
  route<kUpWarps>(r, p, share);
#pragma unroll 1
  for (int rounds = p.down_unit != p.unit ? 2 : 1, first = 1; rounds > 0; --rounds, first = 0) {
    form_units<kUpWarps>(r, units, p, rounds == 2 ? p.down_unit : p.unit);
    if (first != 0) {
      const int places = p.tokens * p.top, words = Units::bytes(p.max_units) / 4, step = gridDim.x * kUpThreads;
      uint32_t* to = reinterpret_cast<uint32_t*>(p.table + 1);
      for (int i = blockIdx.x * kUpThreads + threadIdx.x; i < words + places; i += step) {
        if (i < words) {
          to[i] = reinterpret_cast<const uint32_t*>(smem + p.off_units)[i];
        } else {
          const int k = i - words;
          to[i] = __float_as_uint(share[k]);
          if (p.ids != nullptr) p.ids[k] = r.sel[k] == 0xffff ? -1 : (int)r.sel[k];
          if (p.shares != nullptr) p.shares[k] = share[k];
        }
      }
      if (threadIdx.x == 0) *p.table = MoeTable{r.units, {r.bad[0], r.bad[1]}, 0};  // (the same from every CTA)
      __syncthreads();
    }
  }
  const uint32_t zeros = smem_u32(smem + p.off_zero);

  const int tiles = p.hidden / 32, chunks = (p.dim + S::kChunk - 1) / S::kChunk;
  const int items_unit = (tiles + p.tiles_item - 1) / p.tiles_item;
  const int items = r.units * items_unit;
  // a run of items: mostly one unit's, so that its columns are converted once
  const int item0 = share_of(items, blockIdx.x, gridDim.x), item1 = share_of(items, blockIdx.x + 1, gridDim.x);
  const int slice = wid & (p.ks - 1), tile_local = wid / p.ks;  // (ks is a power of two)
  const bool works = tile_local < p.tiles_item;
  const int c0 = slice * chunks / p.ks, n = (slice + 1) * chunks / p.ks - c0;

  // the producer's place: chunk j of the warp's columns of an item, rows 16 m .. of its tile
  int pi = item0, pj = 0, pm = 0, ps = 0;
  int p_unit = item0 / items_unit, p_first = item0 % items_unit * p.tiles_item;  // the item's unit and first tile
  Rows<WT, F16> rows;
  auto settle = [&]() {  // on to an item in which the warp has rows
    while (pi < item1 && !(works && p_first + tile_local < tiles)) {
      ++pi;
      if ((p_first += p.tiles_item) >= tiles) p_first = 0, ++p_unit;
    }
    if (pi < item1) {
      const long long row = (long long)(units.head[p_unit] & 255) * p.hidden + 32LL * (p_first + tile_local);
      rows.set(p.q1, p.d1, p.q3, p.d3, row, row, p.dim);
    }
  };
  settle();
  auto issue = [&]() {
    if (pi < item1) {
      rows.load(ring + ps * S::kBytes, c0 + pj, 16 * pm, p.dim);
      ps = ps + 1 == p.ring ? 0 : ps + 1;
      pm ^= 1;
      if (pm == 0 && ++pj == n) {
        pj = 0;
        ++pi;
        if ((p_first += p.tiles_item) >= tiles) p_first = 0, ++p_unit;
        settle();
      }
    }
    copies_commit();
  };
#pragma unroll 1
  for (int i = 0; i < p.ring - 1; ++i) issue();

  int cs = 0, held = -1;  // held: the unit that u is, and whose columns the cache has
  int unit = item0 / items_unit, first = item0 % items_unit * p.tiles_item;
  Unit u{};
  const Columns col0 = columns_of<S, 1>(smem_u32(cache), zeros, max_vectors);
  for (int item = item0; item < item1; ++item) {
    const int tile = first + tile_local;
    if (held != unit) {
      u = unit_of(units, unit);
      if (works && n <= p.cached) {
        __syncwarp();
        for (int j = 0; j < n; ++j) convert_columns<S, WT, XF32, WHOLE>(cache + j * cache_bytes, max_vectors, p.x, u, c0 + j, p.dim);
        __syncwarp();
      }
      held = unit;
    }
    const int sets = XF32 ? u.cols : (u.cols + 1) / 2;
    float acc[2][2][2][2] = {};  // [rows 16 m][W1, W3][set][row g, g + 8]
    if (works && tile < tiles) {
      for (int j = 0; j < n; ++j) {
        Columns c = col0;
        if (n > p.cached) {
          __syncwarp();
          convert_columns<S, WT, XF32, WHOLE>(cache, max_vectors, p.x, u, c0 + j, p.dim);
        } else {
          c.b += c.b == zeros ? 0 : j * cache_bytes;
          c.xs += c.xs == zeros ? 0 : j * cache_bytes;
        }
        // rows 0 .. 15, then 16 .. 31: the sums change places between them, so that both are one piece of code
#pragma unroll 1
        for (int m = 0; m < 2; ++m) {
          __syncwarp();  // every lane is done with the slot that is filled next
          issue();
          wait_ring(p.ring);
          __syncwarp();
          // one or two vectors, or three or four
          if (sets == 1)
            consume<WT, F16, WHOLE, 1, 1>(ring + cs * S::kBytes, c, acc[0]);
          else
            consume<WT, F16, WHOLE, 2, 1>(ring + cs * S::kBytes, c, acc[0]);
          cs = cs + 1 == p.ring ? 0 : cs + 1;
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float keep = acc[0][w][v][h];
                acc[0][w][v][h] = acc[1][w][v][h];
                acc[1][w][v][h] = keep;
              }
        }
      }
    }
    // a vector's two lanes hold two blocks each; float32 tokens: hi and lo are the set's two vectors
    float* area = red + (item & 1) * (kUpWarps * kUnit * 64);  // (two, so that one barrier an item does)
    float* my = area + wid * (kUnit * 64);
#pragma unroll
    for (int v = 0; v < 2; ++v)
      if (v < sets) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float a = acc[m][w][v][h];
              a += __shfl_xor_sync(0xffffffffu, a, 1);
              if (XF32) a += __shfl_xor_sync(0xffffffffu, a, 2);
              const int tok = XF32 ? v : 2 * v + (t >> 1);
              if (XF32 ? t == 0 : (t & 1) == 0) my[tok * 64 + w * 32 + 16 * m + 8 * h + g] = a;
            }
      }
    __syncthreads();
    // the item's tiles and tokens over the warps, another one first each time
    for (int i = (wid + item * 5) % kUpWarps; i < p.tiles_item * u.cols; i += kUpWarps) {
      const int tl = i / u.cols, col = i % u.cols, ht = first + tl;
      const int slot = __shfl_sync(0xffffffffu, u.slot, col);
      if (ht < tiles) {
        const float* part = area + tl * p.ks * (kUnit * 64) + col * 64 + lane;
        float gate = 0.f, up = 0.f;
#pragma unroll 4
        for (int k = 0; k < p.ks; ++k) {
          gate += part[k * (kUnit * 64)];
          up += part[k * (kUnit * 64) + 32];
        }
        // the tile's 32 rows are a block of W2's columns: halves at a power of two of the block's own
        const float h = glu(p.act, gate, up);
        const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(isnan(h) ? 0.f : fabsf(h))));
        float to, down;
        block_scale(amax, to, down);
        // as to_halves() leaves activations, for W2's type
        const bool bits = p.w2_q4 && p.out_bf16, split = bits && lane >= 16;
        const float v = h * to * (split ? 0.0625f : 1.f);
        const __half hi = __float2half_rn(v), lo = __float2half_rn(isfinite(v) ? v - __half2float(hi) : 0.f);
        const int place = p.w2_q4 ? (lane & ~3) | (lane & 1) << 1 | (lane >> 1 & 1) : lane;
        __half* out = reinterpret_cast<__half*>(p.h) + (long long)slot * p.hidden + 32 * ht + place;
        out[0] = hi;
        out[p.h_plane] = lo;
        float sum = 0.f;
        if (bits) {
          sum = (__half2float(hi) + __half2float(lo)) * (split ? 16.f : 1.f);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        if (lane == 0) p.h_factor[(long long)slot * (p.hidden / 32) + ht] = make_float2(down, 8.f * sum);
      }
    }
    if ((first += p.tiles_item) >= tiles) first = 0, ++unit;
  }
}

// ------------------------------------------------------------------------------------------ down
constexpr int kDownWarps = 8, kDownThreads = kDownWarps * 32;

// UNIT: tokens of a unit at most.
template <int WT, bool F16, bool WHOLE, int UNIT>
__global__ void __launch_bounds__(kDownThreads, UNIT > 2 ? 1 : 2) moe_down_kernel(const __grid_constant__ MoeParams p, int ranks) {
  using S = Stage<WT, F16>;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* tiles = reinterpret_cast<float*>(smem + p.off_red);  // a warp's tokens x 32 rows
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int most = min(p.tokens, UNIT);
  const int stage_bytes = S::kBytes + S::columns(most * kParts, most);
  const uint32_t ring = smem_u32(smem + p.off_ring) + wid * p.ring * stage_bytes;
  const uint32_t zeros = smem_u32(smem + p.off_zero);
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank();
  const int row0 = (int)(blockIdx.x / ranks) * kRowsStage;
  if (threadIdx.x < 32) reinterpret_cast<uint32_t*>(smem + p.off_zero)[threadIdx.x] = 0u;
  griddep_wait();
  griddep_launch_dependents();
  // the routing as moe_up left it
  {
    const int words = (int)(sizeof(MoeTable) + Units::bytes(p.max_units) + p.tokens * p.top * 4) / 4;
    const uint32_t* from = reinterpret_cast<const uint32_t*>(p.table);
    for (int i = threadIdx.x; i < words; i += kDownThreads) reinterpret_cast<uint32_t*>(smem)[i] = __ldcg(from + i);
  }
  const MoeTable& table = *reinterpret_cast<const MoeTable*>(smem);
  const Units units(smem + sizeof(MoeTable), p.max_units);
  const float* share = reinterpret_cast<const float*>(smem + sizeof(MoeTable) + Units::bytes(p.max_units));
  __syncthreads();
  float* my = tiles + wid * kRowsStage * p.tokens;
  for (int i = lane; i < kRowsStage * p.tokens; i += 32) my[i] = 0.f;
  __syncwarp();

  const int chunks = (p.hidden + S::kChunk - 1) / S::kChunk;
  const int total = table.units * chunks, warps = ranks * kDownWarps, me = rank * kDownWarps + wid;
  const int s0 = share_of(total, me, warps), s1 = share_of(total, me + 1, warps);
  int ps = s0, ps_c = s0 % chunks, ps_u = s0 / chunks, slot_p = 0;
  Unit pu{};
  Rows<WT, F16> rows;
  uint32_t h_at = 0;  // lane v: vector v's row of h, in 64 halves
  auto next_unit = [&]() {
    pu = unit_of(units, ps_u);
    const long long row = (long long)pu.expert * p.dim + row0;
    rows.set(p.q2, p.d2, p.q2, p.d2, row, row + 16, p.hidden);
    const int slot = __shfl_sync(0xffffffffu, pu.slot, lane / kParts);
    h_at = (uint32_t)((lane % kParts * p.h_plane + (long long)slot * p.hidden) / 64);
  };
  if (s0 < s1) next_unit();
  // the vectors' halves and scales: a piece of 16 bytes a lane and vector
  auto columns = [&](int at) {
    const uint32_t to = ring + at * stage_bytes + S::kBytes;
    constexpr int kPieces = S::kChunk / 8;       // of a vector
    constexpr int kTogether = 32 / kPieces;      // vectors of one instruction
    const int vectors = pu.cols * kParts, piece = lane % kPieces;
    const int first = ps_c * S::kChunk + piece * 8;
    const bool live = first < p.hidden;
#pragma unroll
    for (int i = 0; i < UNIT * kParts; i += kTogether) {
      if (i >= vectors) break;
      const int v = i + lane / kPieces;
      const uint32_t row = __shfl_sync(0xffffffffu, h_at, v);
      const int slot = __shfl_sync(0xffffffffu, pu.slot, v / kParts);
      if (v >= vectors) continue;
      copy_async<16>(to + v * S::kVector + (piece >> 2) * S::kBlock + (piece & 3) * 16, p.h + (long long)row * 64 + (live ? first : 0), live);
      if ((piece & 3) == 0 && v % kParts == 0)
        copy_async<8>(to + most * kParts * S::kVector + (v / kParts * S::kBlocks + (piece >> 2)) * 8,
                      p.h_factor + (long long)slot * (p.hidden / 32) + (live ? first / 32 : 0), live);
    }
  };
  auto weights = [&](int at) { rows.load(ring + at * stage_bytes, ps_c, 0, p.hidden); };
  auto advance = [&]() {
    ++ps;
    slot_p = slot_p + 1 == p.ring ? 0 : slot_p + 1;
    if (++ps_c == chunks) {
      ps_c = 0;
      ++ps_u;
      if (ps < s1) next_unit();
    }
  };
#pragma unroll 1
  for (int i = 0; i < p.ring - 1; ++i) {
    if (ps < s1) {
      weights(slot_p);
      columns(slot_p);
      advance();
    }
    copies_commit();
  }

  const Columns col0 = columns_of<S, kParts>(ring + S::kBytes, zeros, most);
  float acc[2][2][2] = {};  // [tile][set][row g, g + 8]
  int cs = 0, cc = s0 % chunks, cu = s0 / chunks;
  Unit u{};
  if (s0 < s1) u = unit_of(units, cu);
  auto flush = [&]() {
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      if (2 * v >= UNIT) break;
      const int col = 2 * v + (t >> 1);
      const int tok = __shfl_sync(0xffffffffu, u.tok, col);
      const float part = share[__shfl_sync(0xffffffffu, u.slot, col)];  // (lanes without a token: of the first, unused)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float a = acc[m][v][h];
          a += __shfl_xor_sync(0xffffffffu, a, 1);
          if (col < u.cols && (t & 1) == 0) my[tok * kRowsStage + 16 * m + 8 * h + g] += part * a;
          acc[m][v][h] = 0.f;
        }
    }
    __syncwarp();
  };
  for (int s = s0; s < s1; ++s) {
    __syncwarp();
    if (ps < s1) {
      weights(slot_p);
      columns(slot_p);
      advance();
    }
    copies_commit();
    wait_ring(p.ring);
    __syncwarp();
    Columns c = col0;
    c.b += c.b == zeros ? 0 : cs * stage_bytes;
    c.xs += c.xs == zeros ? 0 : cs * stage_bytes;
    if (UNIT <= 2 || u.cols <= 2)
      consume<WT, F16, WHOLE, 1, kParts>(ring + cs * stage_bytes, c, acc);
    else
      consume<WT, F16, WHOLE, 2, kParts>(ring + cs * stage_bytes, c, acc);
    cs = cs + 1 == p.ring ? 0 : cs + 1;
    if (++cc == chunks) {
      flush();
      cc = 0;
      if (s + 1 < s1) u = unit_of(units, ++cu);
    }
  }
  if (s0 < s1 && cc != 0) flush();
  __syncthreads();
  // this CTA's tiles in warp order, then the cluster's in rank order, its CTAs sharing the sums
  const int values = kRowsStage * p.tokens;
  for (int i = threadIdx.x; i < values; i += kDownThreads) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kDownWarps; ++w) sum += tiles[w * values + i];
    tiles[i] = sum;
  }
  if (ranks > 1)
    cl.sync();
  else
    __syncthreads();
  for (int i = rank * kDownThreads + threadIdx.x; i < values; i += ranks * kDownThreads) {
    const int row = i % kRowsStage, tok = i / kRowsStage;
    float v[8], sum = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < ranks ? cl.map_shared_rank(tiles, k)[i] : 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += v[k];
    sum *= p.scale;
    if (table.bad[tok >> 5] >> (tok & 31) & 1u) sum = NAN;
    const long long at = (long long)tok * p.dim + row0 + row;
    if (p.out_bf16)
      static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(sum);
    else
      static_cast<float*>(p.out)[at] = sum;
  }
  if (ranks > 1) cl.sync();  // no CTA leaves while another reads its tiles
}

// A kernel's dynamic shared-memory limit raised to all that a CTA may have, once for each kernel and device.
template <typename K>
cudaError_t allow_smem(K kern, const DeviceInfo& dev, bool (&done)[64]) {
  static std::mutex mu;
  if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidValue;
  std::lock_guard<std::mutex> lock(mu);
  if (done[dev.device]) return cudaSuccess;
  const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)dev.smem_optin);
  done[dev.device] = err == cudaSuccess;
  return err;
}

constexpr size_t round_up(size_t v, size_t to) { return (v + to - 1) / to * to; }

// Units of a launch at most (both kernels' arrays have this length): an expert's last one may be part full.
int max_units(int tokens, int top, int experts, int unit) {
  const int pairs = tokens * top, used = experts < pairs ? experts : pairs, n = used + pairs / unit;
  return n < pairs ? n : pairs;
}

// Shared memory of an SM's CTA, with what the system keeps, where `n` are to fit.
size_t room(const DeviceInfo& dev, int n) {
  const size_t each = dev.smem_per_sm / n;
  const size_t have = each > dev.smem_reserved ? each - dev.smem_reserved : 0;
  return have < dev.smem_optin ? have : dev.smem_optin;
}

// (sets p.max_units, for launch_down as well)
template <int WT, bool F16>
cudaError_t launch_up(MoeParams& p, bool x_f32, const DeviceInfo& dev, cudaStream_t stream) {
  using S = Stage<WT, F16>;
  const int most = x_f32 ? kVectors / 2 : kVectors;
  const int chunks = (p.dim + S::kChunk - 1) / S::kChunk;
  p.ks = 1;
  while (p.ks < kUpWarps && 2 * p.ks <= chunks) p.ks *= 2;
  const int slice = (chunks + p.ks - 1) / p.ks;
  p.off_units = (int)round_up(sizeof(Routing), 16);
  // the warps' columns are kept where they leave room for the rings; units of fewer tokens where they do not (Q4_0 with float32 scales)
  size_t smem = 0;
  bool fits = false;
  for (p.unit = p.tokens < most ? p.tokens : most; p.unit >= 1 && !fits; p.unit -= fits ? 0 : 1) {
    const int tokens = p.tokens < p.unit ? p.tokens : p.unit, vectors = x_f32 ? 2 * tokens : tokens, columns = S::columns(vectors, vectors);
    p.max_units = max_units(p.tokens, p.top, p.experts, p.unit < p.down_unit ? p.unit : p.down_unit);
    p.off_zero = (int)round_up(p.off_units + Units::bytes(p.max_units), 128);
    p.off_red = p.off_zero + 128;
    p.off_cols = p.off_red + 2 * kUpWarps * most * 64 * 4;
    for (int keep = 0; keep < 2 && !fits; ++keep) {
      p.cached = keep == 0 ? slice : 1;
      p.off_ring = (int)round_up(p.off_cols + (size_t)kUpWarps * p.cached * columns, 128);
      for (p.ring = 4; p.ring >= 2 && !fits; p.ring -= fits ? 0 : 1) {
        smem = p.off_ring + (size_t)kUpWarps * p.ring * S::kBytes;
        fits = smem <= dev.smem_optin;
      }
    }
    if (fits) break;
  }
  if (!fits) return cudaErrorInvalidValue;
  // an item: as many tiles as the warps take, or fewer where that would leave SMs without one
  const long long units = p.max_units;
  const int tiles = p.hidden / 32;
  for (p.tiles_item = kUpWarps / p.ks; p.tiles_item > 1 && units * ((tiles + p.tiles_item - 1) / p.tiles_item) < dev.sm_count;) p.tiles_item /= 2;
  const long long items = units * ((tiles + p.tiles_item - 1) / p.tiles_item);
  const int which = x_f32 ? 2 : WT == QMV_Q4_0 && !p.out_bf16;
  auto kern = which == 2   ? moe_up_kernel<WT, F16, true, true>
              : which == 1 ? moe_up_kernel<WT, F16, false, WT == QMV_Q4_0>
                           : moe_up_kernel<WT, F16, false, false>;
  static bool done[3][64] = {};
  const cudaError_t err = allow_smem(kern, dev, done[which]);
  if (err != cudaSuccess) return err;
  return launch_dependent(kern, dim3((unsigned)(items < dev.sm_count ? items : dev.sm_count)), kUpThreads, smem, stream, p);
}

template <int WT, bool F16>
cudaError_t launch_down(MoeParams p, const DeviceInfo& dev, cudaStream_t stream) {
  using S = Stage<WT, F16>;
  const int most = p.tokens < p.down_unit ? p.tokens : p.down_unit;
  const int stage = S::kBytes + S::columns(most * kParts, most);
  p.off_zero = (int)round_up(sizeof(MoeTable) + Units::bytes(p.max_units) + (size_t)p.tokens * p.top * 4, 128);
  p.off_red = p.off_zero + 128;
  p.off_ring = (int)round_up(p.off_red + (size_t)kDownWarps * kRowsStage * p.tokens * 4, 128);
  size_t smem = 0;
  int per_sm;
  for (per_sm = p.down_unit > 2 ? 1 : 2; per_sm >= 1; --per_sm) {
    for (p.ring = per_sm == 2 ? 2 : 4; p.ring >= 2; --p.ring) {
      smem = p.off_ring + (size_t)kDownWarps * p.ring * stage;
      if (smem <= room(dev, per_sm)) break;
    }
    if (p.ring >= 2) break;
  }
  if (per_sm < 1) return cudaErrorInvalidValue;
  // CTAs of a cluster: as many as the SMs take, with a stage for each of their warps
  const int tiles = p.dim / kRowsStage, chunks = (p.hidden + S::kChunk - 1) / S::kChunk;
  const long long stages = (long long)(p.experts < p.tokens * p.top ? p.experts : p.tokens * p.top) * chunks;
  int ranks = 1;
  while (ranks < 8 && tiles * ranks * 2 <= per_sm * dev.sm_count && stages >= 2 * ranks * kDownWarps) ranks *= 2;
  const bool whole = WT == QMV_Q4_0 && !p.out_bf16, wide = p.down_unit > 2;
  constexpr bool kQ4 = WT == QMV_Q4_0;
  auto kern = whole ? (wide ? moe_down_kernel<WT, F16, kQ4, 4> : moe_down_kernel<WT, F16, kQ4, 2>)
                    : (wide ? moe_down_kernel<WT, F16, false, 4> : moe_down_kernel<WT, F16, false, 2>);
  const int which = 2 * whole + wide;
  static bool done[4][64] = {};
  const cudaError_t err = allow_smem(kern, dev, done[which]);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles * ranks));
  cfg.blockDim = dim3(kDownThreads);
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

size_t moe_scratch_bytes(int64_t tokens, int top, int hidden) {
  const size_t t = tokens < kTokens ? tokens : kTokens;
  const int pairs = (int)t * top;
  return (size_t)pairs * (hidden * 2 * kParts + hidden / 32 * 8) + sizeof(MoeTable) + Units::bytes(pairs) + (size_t)pairs * 4;
}

cudaError_t launch_moe(const MoeArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  // blocks of 48 tokens, the last of up to 64 (256 over 128 experts of 768 x 2048: 717 us against 762 for blocks of 64; but 64 at once 184 against
  // 212 for 48 and 16)
  int64_t block;
  for (int64_t t0 = 0; t0 < a.tokens; t0 += block) {
    block = a.tokens - t0 <= kTokens ? a.tokens - t0 : kTokensWide;
    MoeParams p{};
    p.tokens = (int)block;
    p.q1 = a.w1.q, p.d1 = a.w1.d, p.q3 = a.w3.q, p.d3 = a.w3.d, p.q2 = a.w2.q, p.d2 = a.w2.d;
    p.logits = a.logits + t0 * a.logits_stride;
    p.logits_stride = a.logits_stride;
    p.x = static_cast<const uint8_t*>(a.x) + t0 * a.dim * (a.x_bf16 ? 2 : 4);
    p.out = static_cast<uint8_t*>(a.out) + t0 * a.dim * (a.out_bf16 ? 2 : 4);
    p.out_bf16 = a.out_bf16;
    p.hidden = a.hidden;
    p.top = a.top;
    p.experts = a.experts;
    p.h = static_cast<uint16_t*>(a.scratch);
    p.h_plane = (long long)p.tokens * a.top * a.hidden;
    p.h_factor = reinterpret_cast<float2*>(p.h + kParts * p.h_plane);
    p.table = reinterpret_cast<MoeTable*>(p.h_factor + (size_t)p.tokens * p.top * (p.hidden / 32));
    // Units of 4 tokens for moe_down from 2 tokens an expert on: one CTA of 128 to 248 registers a thread an SM, two units' weights once.  32 tokens
    // over 128 experts (2 each) 105 against 113 us, 48 (3) 128 against 148, 48 over 8 large ones (12) 591 against 670; but 1 token over two
    // large ones 49.7 against 46.5 us, 7 over 16 Q8_0 ones (1.3) 43.5 against 41.4, and none far off either way between.
    // (One or two tokens: one set of units for both kernels.)
    p.down_unit = p.tokens <= kTokensWide && p.tokens * a.top >= 2 * a.experts ? 4 : 2;
    if (p.tokens < p.down_unit) p.down_unit = p.tokens;
    p.w2_q4 = a.w2.wtype == QMV_Q4_0;
    p.ids = a.ids == nullptr ? nullptr : a.ids + t0 * a.top;
    p.shares = a.shares == nullptr ? nullptr : a.shares + t0 * a.top;
    p.dim = a.dim;
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
