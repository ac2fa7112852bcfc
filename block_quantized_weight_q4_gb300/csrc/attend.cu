// attend.cu -- softmax attention of a few rows a sequence over the paged 8-bit cache (single
// tokens, short runs of tokens, and every case that the prompt kernel does not take).
//
//   z_j = scale q . K_j,  p_j = e^(z_j - max z),  out = sum_j p_j V_j / sum_j p_j.
//
// Bound: the cache's bytes, each read once and used by the heads / kv_heads rows that share a
// key/value head.  K levels are exact halves, the A operand of mma.sync (16 keys x 16 dims a step, 8
// query rows as columns); V levels, transposed, exact bfloat16, the A operand of the second product; the
// softmax's weights times the page's V scale go from the first's sums to the second's B operand
// by an 8 x 8 transpose in registers, as two bfloat16 parts (three for float32): bfloat16
// has the whole float32 range, so that a weight counts however small it is beside the largest.
// Each warp streams chunks of 32 keys through a ring of its own (cp.async), with its own running
// maximum, sum and output; the warps of a CTA meet in shared memory, the CTAs that share a
// sequence in the stream's workspace, added in a fixed order by the last to arrive.
//
// Measured: 64 ragged sequences of up to 16384 tokens, 32 heads over 8 of 128, 197 us (6.0 TB/s, 88% of the measured
// copy rate; issue 54% busy, the ALU work is the levels' conversion, 5 operations for 4 levels of K and 7 of V); 256
// sequences of 1000 tokens 105 us (5.0 TB/s); one sequence of 1000 tokens 8.6 us, a chain of dependent latencies.
// Three CTAs of two stages a warp a SM: with three stages only two fit (224 us), with eight warps a CTA 237 us.
#include <mutex>

#include "attend.cuh"

namespace qmv {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = 32;   // keys of a stage
constexpr int kStages = 2;

template <int D>
struct Ring {
  static constexpr int kHalf = kChunk * D;                 // bytes of K (or V) of a stage
  static constexpr int kStage = 2 * kHalf + 32;            // K, V, then the scales of two tiles of 16 keys
  static constexpr int kWarp = kStages * kStage;
  static constexpr int kBytes = kWarps * kWarp;
};

// Byte offset of 16-byte piece c of row r: rows of D bytes, pieces permuted within 128 bytes so that the
// eight rows that one access touches lie in distinct banks.
template <int D>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
  if (D == 64) return (uint32_t)((r * 4 + (c ^ ((r >> 1) & 3))) * 16);
  return (uint32_t)(r * D + ((c ^ (r & 7)) * 16));
}

// The key (of a tile's first or second eight) that row i of a fragment stands for: neighbouring rows
// four keys apart where a row fills a 128-byte line, so that two rows' four pieces do not meet.
template <int D>
__device__ __forceinline__ int key_of(int i) {
  return D == 64 ? i : (i >> 1) | ((i & 1) << 2);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Bytes 0 and 2 (or, shifted, 1 and 3) of a word, signed, as a bfloat16 pair: 128 + low seven bits, less 128
// or, for a set sign, 256, all exact.
__device__ __forceinline__ uint32_t bytes_to_bf16(uint32_t w) {
  return bf16x2_sub(lop_and_or(w, 0x007F007Fu, 0x43004300u), lop_and_or(w, 0x00800080u, 0x43004300u));
}
__device__ __forceinline__ float f16_lo(uint32_t v) { return f16_bits_to_f32((uint16_t)(v & 0xFFFFu)); }
__device__ __forceinline__ float f16_hi(uint32_t v) { return f16_bits_to_f32((uint16_t)(v >> 16)); }

// Chunks and segments.  A segment is (sequence, key/value head, block of query rows); its keys are cut into
// chunks of 32.  All segments' chunks in a row are dealt to the CTAs in equal runs.
struct Shape {
  int c0;    // first chunk of the sequence's rows
  int nch;   // chunks of each of its segments
  int nrb;   // row blocks
};

template <int ROWS>
__device__ __forceinline__ Shape shape_of(const KvRef& c, const AttendArgs& a, const KvSeq& q) {
  Shape h;
  const int group = a.heads / c.kv_heads;
  h.nrb = (int)(((long long)q.n * group + ROWS - 1) / ROWS);
  const int begin = a.window > 0 && q.len - q.n - a.window + 1 > 0 ? q.len - q.n - a.window + 1 : 0;
  h.c0 = begin / kChunk;
  h.nch = q.n > 0 ? (q.len + kChunk - 1) / kChunk - h.c0 : 0;
  return h;
}

struct SplitArea {
  unsigned* counters;  // one per CTA, zero between launches
  float* parts;        // two per CTA: ROWS x (D + 2) floats
};

template <int D, bool XB, int NT>
__global__ void __launch_bounds__(kThreads) attend_rows_kernel(const __grid_constant__ KvRef c,
                                                               const __grid_constant__ AttendArgs a,
                                                               const SplitArea area) {
  constexpr int ROWS = 8 * NT;
  constexpr int KS = D / 16;       // 16-dim steps
  constexpr int QP = XB ? 1 : 2;   // parts of q (half): hi (, lo)
  constexpr int PP = XB ? 2 : 3;   // parts of the weights (bfloat16): 16 or 24 bits
  griddep_wait();
  griddep_launch_dependents();
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long scan[kWarps];
  __shared__ int found_seq;
  __shared__ long long found_base;
  __shared__ float warp_m[kWarps][ROWS], warp_l[kWarps][ROWS];
  __shared__ int last_flag;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem) + wid * Ring<D>::kWarp;
  const int group = a.heads / c.kv_heads;
  const bool split = area.counters != nullptr;

  // chunks in all, and the sequence that this CTA's run starts in
  auto weight = [&](int s) -> long long {
    const KvSeq q = kv_seq(c, s);
    const Shape h = shape_of<ROWS>(c, a, q);
    return kv_segment_chunks(h.nch, h.nrb, c.kv_heads);
  };
  auto block_scan = [&](long long v, long long& before) -> long long {  // exclusive prefix and total
    long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    __syncthreads();
    if (lane == 31) scan[wid] = inc;
    __syncthreads();
    long long total = 0;
    before = inc - v;
    for (int w = 0; w < kWarps; ++w) {
      if (w < wid) before += scan[w];
      total += scan[w];
    }
    return total;
  };
  long long total = 0, w = 0, before = 0;  // up to 128 sequences: this thread's chunks, and those before them
  for (int s0 = 0; s0 < c.n_seq; s0 += kThreads) {
    const int s = s0 + tid;
    w = s < c.n_seq ? weight(s) : 0;
    total += block_scan(w, before);
  }
  if (total == 0) return;
  // runs of at least one chunk a warp
  long long ctas = (total + kWarps - 1) / kWarps;
  if (ctas > gridDim.x) ctas = gridDim.x;
  if (blockIdx.x >= ctas) return;
  auto run_begin = [&](long long i) { return i * total / ctas; };
  const long long my0 = run_begin(blockIdx.x), my1 = run_begin(blockIdx.x + 1);
  long long pos = my0;  // next chunk, counted over all segments
  int s = 0;
  long long base = 0;   // first chunk of sequence s
  for (int s0 = 0; s0 < c.n_seq; s0 += kThreads) {
    const int si = s0 + tid;
    long long sum = total;
    if (c.n_seq > kThreads) {
      w = si < c.n_seq ? weight(si) : 0;
      sum = block_scan(w, before);
    }
    if (base + sum > pos) {
      if (base + before <= pos && pos < base + before + w) {
        found_seq = si;
        found_base = base + before;
      }
      __syncthreads();
      s = found_seq;
      base = found_base;
      break;
    }
    base += sum;
  }
  __syncthreads();

  KvSeq sq = kv_seq(c, s);
  Shape sh = shape_of<ROWS>(c, a, sq);

  while (pos < my1) {
    // the segment that chunk pos lies in
    while (pos >= base + kv_segment_chunks(sh.nch, sh.nrb, c.kv_heads) && s + 1 < c.n_seq) {
      base += kv_segment_chunks(sh.nch, sh.nrb, c.kv_heads);
      ++s;
      sq = kv_seq(c, s);
      sh = shape_of<ROWS>(c, a, sq);
    }
    if (kv_segment_chunks(sh.nch, sh.nrb, c.kv_heads) == 0) return;  // lengths that changed under the call
    const int seg = (int)((pos - base) / sh.nch);
    const long long seg0 = base + (long long)seg * sh.nch;
    const int kvh = seg / sh.nrb, rb = seg % sh.nrb;
    // without a workspace a segment belongs to the run that holds its first chunk
    if (!split && pos > seg0) {
      pos = seg0 + sh.nch;
      continue;
    }
    const long long part_end = split && my1 < seg0 + sh.nch ? my1 : seg0 + sh.nch;
    const int p0 = (int)(pos - seg0), p1 = (int)(part_end - seg0);

    // the rows of this block: row rho is query token rho / group, head kvh * group + rho % group
    const int rho0 = rb * ROWS;
    const int nrows = sq.n * group - rho0 < ROWS ? sq.n * group - rho0 : ROWS;
    const int first = sq.len - sq.n;
    const int i_lo = rho0 / group, i_hi = (rho0 + nrows - 1) / group;
    // keys that any row of the block sees, and that every row sees
    const int any_end = a.causal ? first + i_hi + 1 : sq.len;
    const int all_end = a.causal ? first + i_lo + 1 : sq.len;
    const int any_begin = a.window > 0 && first + i_lo - a.window + 1 > 0 ? first + i_lo - a.window + 1 : 0;
    const int all_begin = a.window > 0 && first + i_hi - a.window + 1 > 0 ? first + i_hi - a.window + 1 : 0;
    int ch0 = sh.c0 + p0, ch1 = sh.c0 + p1;
    if (ch0 < any_begin / kChunk) ch0 = any_begin / kChunk;
    if (ch1 > (any_end + kChunk - 1) / kChunk) ch1 = (any_end + kChunk - 1) / kChunk;

    // the ring: chunk ch into stage st
    const long long head_stride = (long long)c.page_tokens * D;
    int ids[2] = {-1, -1};  // the next chunk's pages, looked up one chunk ahead of its copies
    auto look = [&](int ch, int seen) {  // pages before key `seen` are not looked at
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int j0 = ch * kChunk + 16 * u;
        ids[u] = ch < ch1 && j0 < sq.len && j0 >= seen ? kv_page(c, s, (j0 >> c.page_shift)) : -1;
      }
    };
    auto issue = [&](int ch, int st) {
      if (ch < ch1) {
        const uint32_t sk = ring + st * Ring<D>::kStage, sv = sk + Ring<D>::kHalf, ss = sv + Ring<D>::kHalf;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int j0 = ch * kChunk + 16 * u;
          const int id = ids[u];
          if (id >= 0) {
            const long long at = (long long)id * c.kv_heads + kvh;
            const long long off = at * head_stride + (long long)((j0 & (c.page_tokens - 1))) * D;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
              const int p = i * 32 + lane;
              const int r = p / (D / 16), q = p % (D / 16);
              const uint32_t d = piece_at<D>(16 * u + r, q);
              cp16(sk + d, c.k + off + 16 * p);
              cp16(sv + d, c.v + off + 16 * p);
            }
            if (lane < 2) cp4(ss + 8 * u + 4 * lane, (lane ? c.v_scale : c.k_scale) + at);
          } else if (lane < 2) {
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(ss + 8 * u + 4 * lane), "r"(0) : "memory");
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      look(ch + kWarps, 0);
    };
    // pages that end before any row's first key may be anything; only the first chunk can hold one
    look(ch0 + wid, any_begin & -c.page_tokens);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(ch0 + wid + i * kWarps, i);

    // q of row g of each tile as B fragments: for dims 16 (t + 4 cc) + 4 w .. + 3, scaled by the power of
    // two that brings the row's largest magnitude near 2^14
    uint32_t qf[NT][QP][KS][2];
    float qc[NT][2];            // scale * log2 e / that power, of rows 2t and 2t + 1
    int end[NT][2], beg[NT][2];  // keys that these rows see
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = 8 * n + g;
      const int rho = rho0 + r;
      const bool live = r < nrows;
      const long long at = (sq.row0 + rho / group) * a.q_stride + (long long)(kvh * group + rho % group) * D;
      float v[D / 4];
      float amax = 0.f;
#pragma unroll
      for (int cc = 0; cc < D / 64; ++cc) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float w[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          if (live) load8<XB>(a.q, at + 16 * (t + 4 * cc) + 8 * h, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[16 * cc + 8 * h + e] = w[e];
            amax = fmaxf(amax, fabsf(w[e]));
          }
        }
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      float xs, xinv;
      half_stage_scale(amax, xs, xinv);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float x0 = v[4 * k + 2 * h] * xs, x1 = v[4 * k + 2 * h + 1] * xs;
          qf[n][0][k][h] = pack_f16x2(x0, x1);
          if (!XB) qf[n][QP - 1][k][h] = pack_f16x2(x0 - f16_lo(qf[n][0][k][h]), x1 - f16_hi(qf[n][0][k][h]));
        }
      }
      const float rc = a.scale * kLog2e * xinv;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        qc[n][h] = __shfl_sync(0xffffffffu, rc, 4 * (2 * t + h));
        const int rr = 8 * n + 2 * t + h;
        const int i = (rho0 + rr) / group;
        end[n][h] = rr >= nrows ? 0 : a.causal ? first + i + 1 : sq.len;
        beg[n][h] = a.window > 0 ? first + i - a.window + 1 : 0;
      }
    }

    float o[NT][KS][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][k][e] = 0.f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }

    int st = 0;
    for (int ch = ch0 + wid; ch < ch1; ch += kWarps) {
      issue(ch + (kStages - 1) * kWarps, st == 0 ? kStages - 1 : st - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();
      const uint32_t sk = ring + st * Ring<D>::kStage, sv = sk + Ring<D>::kHalf, ss = sv + Ring<D>::kHalf;
      float z[2][NT][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[u][n][e] = 0.f;
#pragma unroll
        for (int cc = 0; cc < D / 64; ++cc) {
          uint32_t w0[4], w1[4];
          lds_u32x4(sk + piece_at<D>(16 * u + key_of<D>(g), t + 4 * cc), w0);
          lds_u32x4(sk + piece_at<D>(16 * u + 8 + key_of<D>(g), t + 4 * cc), w1);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t a0, a1, a2, a3;
            q8_word_to_f16_levels(w0[w], a0, a2);
            q8_word_to_f16_levels(w1[w], a1, a3);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int p = 0; p < QP; ++p)
                mma_f16_16816(z[u][n], a0, a1, a2, a3, qf[n][p][4 * cc + w][0], qf[n][p][4 * cc + w][1], z[u][n]);
          }
        }
      }
      // scores in the log2 domain
      float ks[2], vs[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t k2, v2;
        lds_u32x2(ss + 8 * u, k2, v2);
        ks[u] = __uint_as_float(k2);
        vs[u] = __uint_as_float(v2);
      }
      const int j0 = ch * kChunk;
      const bool edge = j0 < all_begin || j0 + kChunk > all_end;
      float mx[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int h = 0; h < 2; ++h) mx[n][h] = m[n][h];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int h = e & 1;
            float x = z[u][n][e] * (ks[u] * qc[n][h]);
            if (edge) {
              const int j = j0 + 16 * u + (e >> 1) * 8 + key_of<D>(g);
              if (j >= end[n][h] || j < beg[n][h]) x = -INFINITY;
            }
            z[u][n][e] = x;
            mx[n][h] = fmaxf(mx[n][h], x);
          }
      }
      bool raise = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int x = 4; x <= 16; x <<= 1) mx[n][h] = fmaxf(mx[n][h], __shfl_xor_sync(0xffffffffu, mx[n][h], x));
          raise |= mx[n][h] > m[n][h];
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float keep[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            keep[h] = mx[n][h] > m[n][h] ? ex2(m[n][h] - mx[n][h]) : 1.f;
            m[n][h] = mx[n][h];
            l[n][h] *= keep[h];
          }
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][k][e] *= keep[e & 1];
        }
      }
      // weights: l takes them as they are, the second product times the page's V scale
      uint32_t pf[2][NT][PP][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float mm[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) mm[h] = m[n][h] == -INFINITY ? 0.f : m[n][h];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float pv[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = ex2(z[u][n][e] - mm[e & 1]);
            l[n][e & 1] += p;
            // a masked key counts for nothing whatever its page's scale
            pv[e] = edge && p == 0.f ? 0.f : p * vs[u];
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int x = 0; x < PP; ++x) {
              const uint32_t part = pack_bf16x2(pv[2 * h], pv[2 * h + 1]);
              pf[u][n][x][h] = transpose8(part);
              pv[2 * h] -= __uint_as_float(part << 16);
              pv[2 * h + 1] -= __uint_as_float(part & 0xFFFF0000u);
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int row = 16 * u + ((lane >> 3) & 1) * 8 + key_of<D>(lane & 7);
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
          uint32_t r[4];
          ldmatrix_x4_trans(r, sv + piece_at<D>(row, k + (lane >> 4)));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t a0 = bytes_to_bf16(r[2 * x]), a1 = bytes_to_bf16(r[2 * x] >> 8);
            const uint32_t a2 = bytes_to_bf16(r[2 * x + 1]), a3 = bytes_to_bf16(r[2 * x + 1] >> 8);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int p = 0; p < PP; ++p)
                mma_bf16_16816(o[n][k + x], a0, a1, a2, a3, pf[u][n][p][0], pf[u][n][p][1], o[n][k + x]);
          }
        }
      }
      __syncwarp();  // every lane is done with the stage before it is filled again
      st = st + 1 == kStages ? 0 : st + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // the warps meet: maxima first, then the outputs at the common maximum, in the ring's memory
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int x = 4; x <= 16; x <<= 1) l[n][h] += __shfl_xor_sync(0xffffffffu, l[n][h], x);
        if (g == 0) warp_m[wid][8 * n + 2 * t + h] = m[n][h];
      }
    __syncthreads();
    constexpr int kPitch = D + 4;
    float* so = reinterpret_cast<float*>(smem);  // [warp][row][pitch]
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 8 * n + 2 * t + h;
        float mm = warp_m[0][r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, warp_m[w][r]);
        f[h] = m[n][h] == -INFINITY ? 0.f : ex2(m[n][h] - mm);
        if (g == 0) warp_l[wid][r] = l[n][h] * f[h];
      }
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(so + (wid * ROWS + 8 * n + 2 * t + h) * kPitch + 16 * k + 2 * g) =
              make_float2(o[n][k][h] * f[h], o[n][k][2 + h] * f[h]);
    }
    __syncthreads();

    auto store = [&](int r, int d, float4 y) {
      const int rho = rho0 + r;
      const long long at = (sq.row0 + rho / group) * a.out_stride + (long long)(kvh * group + rho % group) * D + d;
      if (XB) {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
            make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
      } else {
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = y;
      }
    };
    const bool whole = p0 == 0 && p1 == sh.nch;
    constexpr int kPart = ROWS * (D + 2);
    // a CTA's part of a segment that began before its run, or of one that it begins
    float* mine = whole ? nullptr : area.parts + (2LL * blockIdx.x + (p0 > 0 ? 0 : 1)) * kPart;
    for (int i = tid; i < nrows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      float ll = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(so + (w * ROWS + r) * kPitch + d);
        y.x += x.x, y.y += x.y, y.z += x.z, y.w += x.w;
        ll += warp_l[w][r];
      }
      if (whole) {
        const float inv = ll > 0.f ? __fdiv_rn(1.f, ll) : ll == 0.f ? 0.f : ll;
        store(r, d, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
      } else {
        __stcg(reinterpret_cast<float4*>(mine + r * D + d), y);
        if (d == 0) {
          float mm = warp_m[0][r];
#pragma unroll
          for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, warp_m[w][r]);
          __stcg(mine + ROWS * D + r, mm);
          __stcg(mine + ROWS * D + ROWS + r, ll);
        }
      }
    }
    if (!whole) {
      // the runs that hold this segment's first and last chunk
      const long long cf = ((seg0 + 1) * ctas - 1) / total, cl = ((seg0 + sh.nch) * ctas - 1) / total;
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const unsigned seen = atomicAdd(area.counters + cf, 1u);
        last_flag = seen == (unsigned)(cl - cf);
        if (last_flag) area.counters[cf] = 0;
      }
      __syncthreads();
      if (last_flag) {
        __threadfence();
        for (int i = tid; i < nrows * (D / 4); i += kThreads) {
          const int r = i / (D / 4), d = i % (D / 4) * 4;
          float mm = -INFINITY;
#pragma unroll 8
          for (long long p = cf; p <= cl; ++p)
            mm = fmaxf(mm, __ldcg(area.parts + (2 * p + (p == cf ? 1 : 0)) * kPart + ROWS * D + r));
          float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
          float ll = 0.f;
#pragma unroll 4
          for (long long p = cf; p <= cl; ++p) {
            const float* part = area.parts + (2 * p + (p == cf ? 1 : 0)) * kPart;
            const float pm = __ldcg(part + ROWS * D + r);
            const float f = pm == -INFINITY ? 0.f : ex2(pm - mm);
            const float4 x = __ldcg(reinterpret_cast<const float4*>(part + r * D + d));
            y.x = fmaf(x.x, f, y.x), y.y = fmaf(x.y, f, y.y), y.z = fmaf(x.z, f, y.z), y.w = fmaf(x.w, f, y.w);
            ll = fmaf(__ldcg(part + ROWS * D + ROWS + r), f, ll);
          }
          const float inv = ll > 0.f ? __fdiv_rn(1.f, ll) : ll == 0.f ? 0.f : ll;
          store(r, d, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
        }
      }
    }
    __syncthreads();  // the ring and the warps' maxima are free again
    pos = part_end;
  }
}

template <int D, bool XB, int NT>
cudaError_t launch_rows(const KvRef& c, const AttendArgs& a, const DeviceInfo& dev, const Workspace* ws,
                        cudaStream_t stream) {
  auto kern = attend_rows_kernel<D, XB, NT>;
  constexpr int kMerge = kWarps * 8 * NT * (D + 4) * 4;
  constexpr int kSmem = Ring<D>::kBytes > kMerge ? Ring<D>::kBytes : kMerge;
  static std::mutex mu;
  static int ctas_per_sm[64] = {};
  if (dev.device < 0 || dev.device >= 64) return cudaErrorInvalidValue;
  if ((size_t)kSmem > dev.smem_optin) return cudaErrorInvalidConfiguration;
  int per_sm;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (ctas_per_sm[dev.device] == 0) {
      cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (err != cudaSuccess) return err;
      int k = 0;
      err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&k, kern, kThreads, kSmem);
      if (err != cudaSuccess) return err;
      ctas_per_sm[dev.device] = k > 0 ? k : 1;
    }
    per_sm = ctas_per_sm[dev.device];
  }
  long long grid = (long long)dev.sm_count * per_sm;
  SplitArea area{nullptr, nullptr};
  if (ws != nullptr) {
    const long long fit = (long long)(ws->max_partial_floats / (2 * 8 * NT * (D + 2)));
    if (grid > fit) grid = fit;
    if (grid > ws->max_counters) grid = ws->max_counters;
    area.counters = ws->counters;
    area.parts = ws->partials;
  }
  // no more CTAs than chunks that the stated bounds allow
  const int group = a.heads / c.kv_heads;
  const long long blocks = ((long long)c.max_rows * group + 8 * NT - 1) / (8 * NT);
  const long long span = a.window > 0 && (long long)a.window + c.max_rows < c.max_len ? a.window + c.max_rows : c.max_len;
  const long long most = ((span + kChunk - 1) / kChunk + 1) * blocks * c.kv_heads * c.n_seq / kWarps + 1;
  if (grid > most) grid = most;
  return launch_dependent(kern, dim3((unsigned)grid), kThreads, kSmem, stream, c, a, area);
}

template <int D, bool XB>
cudaError_t launch_dim(const KvRef& c, const AttendArgs& a, const DeviceInfo& dev, const Workspace* ws,
                       cudaStream_t stream) {
  // one tile of 8 rows, or two: a sequence with more than 8 rows a key/value head reads the cache
  // half as often (heads of 256 keep one: two tiles' sums and q leave no registers)
  if (D <= 128 && (long long)c.max_rows * (a.heads / c.kv_heads) > 8)
    return launch_rows<D, XB, D <= 128 ? 2 : 1>(c, a, dev, ws, stream);
  return launch_rows<D, XB, 1>(c, a, dev, ws, stream);
}

}  // namespace

cudaError_t launch_attend(const KvRef& c, const AttendArgs& a, bool x_bf16, const DeviceInfo& dev,
                          cudaStream_t stream) {
  if (attend_prompt_supported(c, a, x_bf16, dev)) return launch_attend_prompt(c, a, dev, stream);
  Workspace w;
  const Workspace* ws = stream_serve_workspace(dev, stream, &w) == cudaSuccess ? &w : nullptr;
  switch (c.head_dim) {
    case 64: return x_bf16 ? launch_dim<64, true>(c, a, dev, ws, stream) : launch_dim<64, false>(c, a, dev, ws, stream);
    case 128:
      return x_bf16 ? launch_dim<128, true>(c, a, dev, ws, stream) : launch_dim<128, false>(c, a, dev, ws, stream);
    default:
      return x_bf16 ? launch_dim<256, true>(c, a, dev, ws, stream) : launch_dim<256, false>(c, a, dev, ws, stream);
  }
}

}  // namespace qmv
