// Attention over 4-bit pages (pa_attention_int4).
//
// Every warp is a worker of its own: it streams pages through a private ring of
// shared memory (cp.async, no barrier with other warps), keeps the query operands, the
// softmax state and the output tile in registers, and writes its result.  A page is
// D * 17 bytes for K and V together, so at 4.25 bits a value the kernel is bound by
// instructions as much as by memory: the nibbles cost one mask per operand register
// (pa_pages.cuh), scales multiply score accumulators and softmax weights, and
// everything that only an edge page needs is behind one branch.
//
// The tiles are those of the other attention kernels: S^T[16 tokens x 8 rows] = K . Q^T and
// O^T[D x 8] += V^T . P^T, so that a page is one step.  Scores: two k steps per group of
// 32 dims, times the tokens' scales in fp32.  P.V: the weights, f16, are transposed by
// movmatrix, multiplied by the group's scales of their tokens, and meet V codes that
// ldmatrix.trans delivers as (token 2q, token 2q + 1) pairs of four dims each.  A weight is
// rounded to f16 twice, by itself (its row's sum is that of the rounded ones) and times the scale,
// 2^-11 each.  Taking the codes' offset off the output afterwards instead of off the codes is
// faster (39.2 against 40.2 us for the 64 sequences below, 107 against 109, 119 against 122), but a
// rounding then counts with a code of up to 15 instead of 7, one-sidedly where values are small;
// taken off as a sum of the rounded products it costs 40.5, 111 and 139 us.
//
// Measured (GPU time of a call, bytes of every page once, against a copy's 6780 GB/s): 64
// sequences of 512-4096 tokens, 32/8 heads of 128 dims, 40.2 us, 161 MB (0.59); 256 of 128-8192,
// 64/8 heads, 109 us, 551 MB (0.74); one of 131071 36.0 us (0.58); five drafts over 32 of
// 2048-16384 122 us, 324 MB (0.39).  What bounds it: for up to 8 rows memory and issue slots
// (DRAM 58-73 %, issue 58-62 % of the whole launch) from the first page to the last, 5 us
// before that (2 to find the work, 3 for block ids and the first page), 3 us of uneven end and
// the merge, 4 us; for 24 rows the latency of dependent tensor-core and FP32 steps with the 8 warps
// per SM that 255 registers allow (tensor pipe 48 %, issue slots 46 %).
//
// Balanced mode (kFlat): runs of pa_runs.cuh.  A job that lies in one run is written out
// directly; the others leave (m, l, O) partials, which attn4_merge_kernel joins.
// Unit mode: units of a fixed size; the split-KV merge joins the partitions.  The result of a
// sequence then does not depend on the batch it is in.
#pragma once

#include "pa_runs.cuh"

namespace pa {

// NT n-tiles of 8 query rows per warp, NTW row columns (each a worker's job of its own), STAGES
// staged pages per warp, MINB CTAs of WARPS warps per SM.
template <int NT_, int NTW_, int STAGES_, int MINB_, int WARPS_ = 4>
struct Cfg4 {
  static constexpr int NT = NT_, NTW = NTW_, STAGES = STAGES_, MINB = MINB_;
  static constexpr int kWarps = WARPS_, kThreads = 32 * kWarps, kRows = 8 * NT;
  static constexpr bool kQRegs = NT <= 2;
};

template <int D, class C>
struct Smem4 {
  using P = Page<kPageInt4, D>;
  static constexpr int kStageBytes = 2 * P::kBytes;         // a K page, then its V page
  static constexpr int kRingBytes = C::STAGES * kStageBytes;
  static constexpr int kQBytes = C::kQRegs ? 0 : C::NT * QTileSmem<kPageInt4, D>::kBytes;
  static constexpr int kWarpBytes = kRingBytes + kQBytes;
  static constexpr int kBytes = C::kWarps * kWarpBytes;
  static_assert(kStageBytes % 16 == 0 && kWarpBytes % 16 == 0, "16-byte copies");
};

__device__ __forceinline__ RunList run_list(const Attn4Params& p, int ntw) {
  return RunList{p.context_lens, p.num_seqs, p.T,         p.max_ctx, p.window,
                 p.Hkv * ntw,    p.workers,  p.min_share, p.ppb,     p.max_parts};
}

template <int D, class C, bool kFlat>
__global__ void __launch_bounds__(C::kThreads, C::MINB) paged_attn4_kernel(const Attn4Params p) {
  using P = Page<kPageInt4, D>;
  using Sm = Smem4<D, C>;
  constexpr int NT = C::NT, NTW = C::NTW, S = C::STAGES;
  constexpr int NG = P::kGroups;
  extern __shared__ __align__(128) uint8_t smem_all[];
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, q4 = lane & 3;
  uint8_t* smem = smem_all + warp * Sm::kWarpBytes;
  const int G = p.G, T = p.T, nrows = G * T;
  const RunList list = run_list(p, NTW);
  const int worker = warp * gridDim.x + blockIdx.x;

  // Per lane: its chunks within a page (chunk `lane` of K and of V, and one of the scale
  // chunks) and their place in a stage.
  const uint32_t page_stride = static_cast<uint32_t>(p.Hkv) * P::kBytes;
  constexpr int SC = P::kScales / 16;        // scale chunks of a page
  const uint32_t ring = smem_u32(smem);
  const uint32_t swz = page_swizzle<kPageInt4, D>(lane / P::kChunks, lane % P::kChunks);
  const uint32_t sdst = P::kCodes + 16 * (lane % SC) + (lane < SC ? 0 : P::kBytes);
  const uint32_t koff = ldsm_offset<kPageInt4, D>(lane);

  // One column of rows reads a page once, so V pages leave the L2 cache first: the partial sums
  // stay for the merge and the K pages for a call that sums up weights (the bounded decode step over
  // 4-bit pages 87.0 -> 84.7 us; 256 sequences of 128-8192 tokens 113.6 -> 113.2).
  const uint64_t v_policy = read_policy(NTW == 1);
  Cursor<kFlat> cur;
  Segment seg;
  bool invalid = false;
  const bool any = cur.start(list, worker, lane, invalid);
  if (kFlat && worker == 0 && invalid) atomicOr(&g_pa_err, kErrBounds);
  // With an append the launch before is the one that stores the new tokens: it started only
  // when the lengths were final, so this one may find its work alongside it.
  grid_dependency_wait();
  if (!any) return;

  while (cur.next(list, seg, invalid)) {
    const int b = seg.b, L = seg.L, n = seg.n;
    const int g = seg.job / NTW, row0 = (seg.job % NTW) * C::kRows;
    const int pg0 = seg.first + seg.page;

    // the query rows, on their way while the block ids are fetched
    QTileRaw<kPageInt4, D> raw[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
      load_q_raw(raw[j], p.q, b, g, T, G, p.Hq, row0 + 8 * j, nrows, lane);

    // -------------------------------------------------------------- page stream
    const size_t head_off = static_cast<size_t>(g) * P::kBytes;
    const uint8_t* kbase = static_cast<const uint8_t*>(p.k_pool) + head_off;
    const uint8_t* vbase = static_cast<const uint8_t*>(p.v_pool) + head_off;
    const uint8_t* ssrc = (lane < SC ? kbase : vbase) + P::kCodes + 16 * (lane % SC);
    const uint8_t* ksrc = kbase + 16 * lane;
    const uint8_t* vsrc = vbase + 16 * lane;
    const int32_t* trow = p.block_tables + static_cast<size_t>(b) * p.mbs + pg0;
    // Block ids, 32 at a time; ids outside the pool become page 0 with a bit in `bad` (bits
    // of the newest batch and of the one before it).
    int ids = 0;
    unsigned bad = 0, bad_before = 0;
    auto load_ids = [&](int i) {
      ids = i + lane < n ? __ldg(trow + i + lane) : 0;
      const bool out = static_cast<unsigned>(ids) >= static_cast<unsigned>(p.num_blocks);
      bad_before = bad;
      bad = __ballot_sync(0xffffffffu, out);
      if (out) {
        ids = 0;
        atomicOr(&g_pa_err, kErrBounds);
      }
    };
    load_ids(0);
    int it = 0;                              // next page to stage
    uint32_t st_in = ring;
    auto issue = [&]() {
      if (it < n) {
        if ((it & 31) == 0 && it > 0) load_ids(it);
        const uint32_t phys = __shfl_sync(0xffffffffu, ids, it & 31);
        const uint8_t* kp = at_page(ksrc, phys, page_stride);
        const uint8_t* vp = at_page(vsrc, phys, page_stride);
#pragma unroll
        for (int c = 0; c < P::kCodes / 512; ++c) {   // 8 (16) rows on: the same swizzle
          cp_async_16(st_in + swz + 512 * c, kp + 512 * c, 16);
          cp_async_16_hint(st_in + swz + P::kBytes + 512 * c, vp + 512 * c, v_policy);
        }
        if (lane < 2 * SC) cp_async_16(st_in + sdst, at_page(ssrc, phys, page_stride), 16);
        ++it;
        st_in = st_in + Sm::kStageBytes == ring + Sm::kRingBytes ? ring : st_in + Sm::kStageBytes;
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue();

    QOperand<kPageInt4, D, NT, C::kQRegs> qo;
    make_q_operand(qo, raw, smem + Sm::kRingBytes, p.scale_log2, p.k_scale[g], lane);

    // Softmax state of rows 2q4, 2q4 + 1 of each n-tile: minus the reference m (log2
    // domain; kUnseen until a score was seen).
    // sum: the sum of the rounded weights, in every row of a tile.
    constexpr float kUnseen = 1e30f, kTop = 3.f;
    float acc[NT][D / 16][4], sum[NT][4], nm0[NT], nm1[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      nm0[j] = nm1[j] = kUnseen;
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[j][e] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][k][e] = 0.f;
    }
    constexpr uint32_t kOnes = 0x3C003C00u;

    // Pages wholly visible to every row: first entry in [lo, hi]
    const int part_end = min(L, (pg0 + n) * kBlockSize);
    const int hi = min(L - T, part_end - 1) - (kBlockSize - 1);
    const int lo = max(0, L - p.wspan);
    int tok0 = pg0 * kBlockSize;
    uint32_t st = ring;

    for (int i = 0; i < n; ++i) {
      cp_async_wait<S - 2>();
      __syncwarp();
      issue();                               // into the stage consumed last
      float t[NT][4];
      page_scores<kPageInt4, D>(t, st, koff, qo, lane);

      const bool edge = tok0 < lo || tok0 > hi || (bad | bad_before) != 0;
      // The end of the page's entries: none of a page that was not in the pool.  The batch of ids
      // that page i came from is the newest one unless `it` has passed on.
      auto end_of_page = [&]() {
        const unsigned bits = (it - 1) >> 5 == i >> 5 ? bad : bad_before;
        return (bits >> (i & 31)) & 1u ? 0 : part_end;
      };
      if (edge) {
        const int end = end_of_page();
        const int j0 = tok0 + gid, j1 = j0 + 8;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int r = row0 + 8 * j + 2 * q4;
          const int a = r < nrows ? L - T + r / G : L - 1;
          const int c = r + 1 < nrows ? L - T + (r + 1) / G : L - 1;
          const unsigned w = p.wcap;
          if (j0 >= end || static_cast<unsigned>(a - j0) >= w) t[j][0] = -CUDART_INF_F;
          if (j0 >= end || static_cast<unsigned>(c - j0) >= w) t[j][1] = -CUDART_INF_F;
          if (j1 >= end || static_cast<unsigned>(a - j1) >= w) t[j][2] = -CUDART_INF_F;
          if (j1 >= end || static_cast<unsigned>(c - j1) >= w) t[j][3] = -CUDART_INF_F;
        }
      }

      // Online softmax: the reference m of a row moves, to kTop below the new maximum, only when a
      // score passes it by 7: a weight is at most 2^7 and, times a V scale (at most 448), an f16
      // value, and the largest weight at least 2^kTop, for f16's sake: what a weight or a product
      // loses below 2^-14 is at most 2^-25, so 2^-28 of the sum.  The reference is rounded so that
      // the maximum's own exponent is never below kTop, however large the scores.
      bool over = false;
      float e[NT][4];                        // scores less the reference
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float* y = t[j];
        fma_f32x2(e[j][0], e[j][1], y[0], y[1], qo.rs0[j], qo.rs1[j], nm0[j], nm1[j]);
        fma_f32x2(e[j][2], e[j][3], y[2], y[3], qo.rs0[j], qo.rs1[j], nm0[j], nm1[j]);
        over |= fmaxf(fmaxf(e[j][0], e[j][1]), fmaxf(e[j][2], e[j][3])) > 7.f;
      }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float x0 = fmaxf(t[j][0], t[j][2]), x1 = fmaxf(t[j][1], t[j][3]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, o));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, o));
          }
          float f0 = 1.f, f1 = 1.f;
          if (fmaf(x0, qo.rs0[j], nm0[j]) > 7.f) {
            const float nm = __fadd_ru(kTop, -__fmul_rd(x0, qo.rs0[j]));
            f0 = nm0[j] == kUnseen ? 0.f : hw_exp2(nm - nm0[j]);
            nm0[j] = nm;
          }
          if (fmaf(x1, qo.rs1[j], nm1[j]) > 7.f) {
            const float nm = __fadd_ru(kTop, -__fmul_rd(x1, qo.rs1[j]));
            f1 = nm1[j] == kUnseen ? 0.f : hw_exp2(nm - nm1[j]);
            nm1[j] = nm;
          }
          e[j][0] = fmaf(t[j][0], qo.rs0[j], nm0[j]);
          e[j][1] = fmaf(t[j][1], qo.rs1[j], nm1[j]);
          e[j][2] = fmaf(t[j][2], qo.rs0[j], nm0[j]);
          e[j][3] = fmaf(t[j][3], qo.rs1[j], nm1[j]);
          // past 2^26 the product is rounded by more than the room above kTop (NaN stays NaN)
#pragma unroll
          for (int i = 0; i < 4; ++i) e[j][i] = e[j][i] > 7.f ? 7.f : e[j][i];
          sum[j][0] *= f0;
          sum[j][1] *= f1;
          sum[j][2] *= f0;
          sum[j][3] *= f1;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            acc[j][k][0] *= f0;
            acc[j][k][1] *= f1;
            acc[j][k][2] *= f0;
            acc[j][k][3] *= f1;
          }
        }
      }
      uint32_t ph0[NT], ph1[NT];             // P^T: tokens 2q, 2q+1 and 2q+8, 2q+9 of row gid
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float p0 = hw_exp2(e[j][0]);
        const float p1 = hw_exp2(e[j][1]);
        const float p2 = hw_exp2(e[j][2]);
        const float p3 = hw_exp2(e[j][3]);
        ph0[j] = transpose_8x8(half2_bits(__floats2half2_rn(p0, p1)));
        ph1[j] = transpose_8x8(half2_bits(__floats2half2_rn(p2, p3)));
      }

      // V scales of tokens 2q, 2q+1 (w0, w1) and 2q+8, 2q+9 (w2, w3), a byte per group
      const uint32_t vp = st + P::kBytes;
      uint32_t w0, w1, w2, w3;
      {
        const uint32_t a = vp + P::kCodes + 2 * q4 * NG;
        if constexpr (NG == 4) {
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w0), "=r"(w1) : "r"(a));
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w2), "=r"(w3) : "r"(a + 32));
        } else {
          uint32_t x, y;
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(a));
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(y) : "r"(a + 16));
          w0 = x & 0xffffu;
          w1 = x >> 16;
          w2 = y & 0xffffu;
          w3 = y >> 16;
        }
      }
      if (edge) {
        // entries that no query token sees may hold any scale, even NaN
        const int nv = end_of_page() - tok0;
        const int first_seen = p.window > 0 ? max(0, L - T - p.window + 1) : 0;
        const int from = first_seen - tok0;
        w0 = 2 * q4 < nv && 2 * q4 >= from ? w0 : 0u;
        w1 = 2 * q4 + 1 < nv && 2 * q4 + 1 >= from ? w1 : 0u;
        w2 = 2 * q4 + 8 < nv && 2 * q4 + 8 >= from ? w2 : 0u;
        w3 = 2 * q4 + 9 < nv && 2 * q4 + 9 >= from ? w3 : 0u;
        // A NaN scale makes the rows that see its token NaN and no others, whose weight of zero
        // would not hold it off: it goes into the output tiles of those rows by hand.
        const uint32_t n0 = e4m3_nan_bytes(w0), n1 = e4m3_nan_bytes(w1);
        const uint32_t n2 = e4m3_nan_bytes(w2), n3 = e4m3_nan_bytes(w3);
        if (__any_sync(0xffffffffu, (n0 | n1 | n2 | n3) != 0u)) {
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) {
            auto bit = [&](uint32_t x) { return (x >> (8 * gr)) & 1u; };
            unsigned at = (bit(n0) | bit(n1) << 1 | bit(n2) << 8 | bit(n3) << 9) << (2 * q4);
            at |= __shfl_xor_sync(0xffffffffu, at, 1);
            at |= __shfl_xor_sync(0xffffffffu, at, 2);
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int r = row0 + 8 * j + 2 * q4 + h;
                const int last = r < nrows ? L - T + r / G : L - 1;
                const int first = p.window > 0 ? max(0, last - p.window + 1) : 0;
                const int lo_bit = max(0, first - tok0), hi_bit = last - tok0;
                const unsigned upto = hi_bit < 0 ? 0u : hi_bit > 15 ? 0xffffu : (2u << hi_bit) - 1u;
                if ((at & upto) >> min(lo_bit, 16) != 0u)
                  acc[j][2 * gr][h] = acc[j][2 * gr][2 + h] = acc[j][2 * gr + 1][h] =
                      acc[j][2 * gr + 1][2 + h] = CUDART_NAN_F;
              }
          }
          w0 &= ~(n0 * 0xffu);
          w1 &= ~(n1 * 0xffu);
          w2 &= ~(n2 * 0xffu);
          w3 &= ~(n3 * 0xffu);
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) mma_f16(sum[j], kOnes, kOnes, kOnes, kOnes, ph0[j], ph1[j]);
#pragma unroll
      for (int g2 = 0; g2 < NG; g2 += 2) {
        // byte pairs (token 2q, token 2q+1) of groups g2 and g2 + 1
        const uint32_t sel = g2 == 0 ? 0x5140u : 0x7362u;
        const uint32_t sa = __byte_perm(w0, w1, sel), sb = __byte_perm(w2, w3, sel);
        uint32_t fs[4];
        e4m3x4_to_f16x4(sa, fs[0], fs[1]);
        e4m3x4_to_f16x4(sb, fs[2], fs[3]);
        uint32_t w[4];
        ldsm_x4_trans(w[0], w[1], w[2], w[3], vp + (koff ^ (g2 << 4)));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int gr = g2 + h;
          const uint32_t fa = fs[h], fb = fs[2 + h];
          const uint32_t y0 = w[2 * h], y1 = w[2 * h + 1];
          const uint32_t u0 = y0 >> 8, u1 = y1 >> 8;
          // codes less 8 as f16 subnormals, exact: dims 32 gr + 4 gid + 0 and 2, then + 1 and 3
          // (times 16)
          const uint32_t x[4] = {y0, u0, y1, u1};
          uint32_t a[4], c[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[i] = f16x2_add(x[i] & kNibLo, kMinus8Lo);
            c[i] = f16x2_add(x[i] & kNibHi, kMinus8Hi);
          }
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint32_t b0 = f16x2_mul(ph0[j], fa), b1 = f16x2_mul(ph1[j], fb);
            mma_f16(acc[j][2 * gr], a[0], a[1], a[2], a[3], b0, b1);
            mma_f16(acc[j][2 * gr + 1], c[0], c[1], c[2], c[3], b0, b1);
          }
        }
      }
      tok0 += kBlockSize;
      st = st + Sm::kStageBytes == ring + Sm::kRingBytes ? ring : st + Sm::kStageBytes;
    }
    cp_async_wait<0>();
    __syncwarp();

    // -------------------------------------------------------------- result
    const float out_scale = p.v_scale[g];
    const size_t slot = kFlat ? static_cast<size_t>(worker) * 2 + seg.second : 0;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {          // rows 2q4 and 2q4 + 1
        const int r = row0 + 8 * j + 2 * q4 + h;
        if (r >= nrows) continue;
        const float l = sum[j][h];
        const bool none = (h ? nm1[j] : nm0[j]) == kUnseen;
        const float inv = l > 0.f ? out_scale / l : 0.f;
        const size_t orow = (static_cast<size_t>(b) * T + r / G) * p.Hq + g * G + r % G;
        float* po = nullptr;
        if (!seg.whole) {
          const size_t at = kFlat ? slot * C::kRows + (r - row0) : orow * p.max_parts + seg.part;
          po = p.part_o + at * D;
          if (gid == 0)
            p.part_ml[at] = make_float2(none ? -CUDART_INF_F : -(h ? nm1[j] : nm0[j]), l);
        }
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          constexpr float A = 16777216.f, B = 1048576.f;   // 2^24, 2^20
          const float* a = acc[j][2 * gr] + h;
          const float* c = acc[j][2 * gr + 1] + h;
          const float4 o =
              make_float4(a[0] * A * inv, c[0] * B * inv, a[2] * A * inv, c[2] * B * inv);
          const int d = 32 * gr + 4 * gid;
          if (seg.whole)
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + orow * D + d) =
                make_uint2(bf162_bits(__floats2bfloat162_rn(o.x, o.y)),
                           bf162_bits(__floats2bfloat162_rn(o.z, o.w)));
          else
            *reinterpret_cast<float4*>(po + d) = o;
        }
      }
    }

  }
  if (!kFlat && invalid && lane == 0) atomicOr(&g_pa_err, kErrBounds);
}

// ---------------------------------------------------------------- merge of the runs
// W warps per (job, query row), 4 / W rows per CTA of four warps (W = 1) or one row per CTA.
// Warp k of a row takes pieces k, k + W, ...
template <int D, int W>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W)
    attn4_merge_kernel(const Attn4Params p, int ntw, int tile_rows, int live) {
  constexpr int DL = D / 32;
  __shared__ float s_acc[W][D];
  __shared__ float s_ml[W][2];
  const RunList list = run_list(p, ntw);
  const int lane = threadIdx.x & 31;
  const int warp = W == 1 ? 0 : threadIdx.x >> 5;
  const int id = W == 1 ? blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
  const int r = id % live;
  const int job = id / live % list.heads;
  const int b = id / live / list.heads;
  const int row = job % ntw * tile_rows + r;
  // every CTA waits, so that this grid does not complete before the one it follows
  if (b >= p.num_seqs) {
    grid_dependency_wait();
    return;
  }
  int first;
  const int nb = visible_pages(list, p.context_lens[b], first);
  const Pieces pc = find_pieces(list, b, job, nb, lane);
  grid_dependency_wait();
  if (nb == 0 || pc.count == 1 || row >= p.G * p.T) return;
  const int parts = pc.count;
  auto slot = [&](int i) { return pc.slot(i) * tile_rows + r; };
  float M = -CUDART_INF_F, S = 0.f, acc[DL];
#pragma unroll
  for (int k = 0; k < DL; ++k) acc[k] = 0.f;
  for (int i = warp + W * lane; i < parts; i += 32 * W) M = fmaxf(M, p.part_ml[slot(i)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float u = M == -CUDART_INF_F ? 0.f : M;
#pragma unroll 8
  for (int i = warp; i < parts; i += W) {
    const size_t at = slot(i);
    const float2 ml = p.part_ml[at];
    const float w = ml.y * hw_exp2(ml.x - u);
    S += w;
    const float* src = p.part_o + at * D + lane * DL;
    if constexpr (DL == 4) {
      const float4 x = *reinterpret_cast<const float4*>(src);
      acc[0] += w * x.x;
      acc[1] += w * x.y;
      acc[2] += w * x.z;
      acc[3] += w * x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(src);
      acc[0] += w * x.x;
      acc[1] += w * x.y;
    }
  }
  if constexpr (W > 1) {
#pragma unroll
    for (int k = 0; k < DL; ++k) s_acc[warp][lane * DL + k] = acc[k];
    if (lane == 0) {
      s_ml[warp][0] = M;
      s_ml[warp][1] = S;
    }
    __syncthreads();
    if (warp != 0) return;
    M = -CUDART_INF_F;
    for (int k = 0; k < W; ++k) M = fmaxf(M, s_ml[k][0]);
    S = 0.f;
#pragma unroll
    for (int d = 0; d < DL; ++d) acc[d] = 0.f;
    for (int k = 0; k < W; ++k) {
      const float x = s_ml[k][0] == -CUDART_INF_F ? 0.f : hw_exp2(s_ml[k][0] - M);
      S += x * s_ml[k][1];
#pragma unroll
      for (int d = 0; d < DL; ++d) acc[d] += x * s_acc[k][lane * DL + d];
    }
  }
  const float inv = S > 0.f ? 1.f / S : 0.f;
  const size_t orow =
      (static_cast<size_t>(b) * p.T + row / p.G) * p.Hq + job / ntw * p.G + row % p.G;
  __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(p.out) + (orow * D + lane * DL) / 2;
#pragma unroll
  for (int k = 0; k < DL; k += 2)
    dst[k / 2] = __floats2bfloat162_rn(acc[k] * inv, acc[k + 1] * inv);
}

template <int D, class C>
cudaError_t launch_cfg4(const Attn4Params& p, cudaStream_t s) {
  constexpr int bytes = Smem4<D, C>::kBytes;
  constexpr Attn4Tile tile = attn4_tile(C::kRows * C::NTW);
  static_assert(tile.nt == C::NT && tile.ntw == C::NTW && 4 * tile.ctas == C::MINB * C::kWarps,
                "the host's tile");
  const long long jobs = static_cast<long long>(p.num_seqs) * p.Hkv * C::NTW;
  auto fn = p.flat ? paged_attn4_kernel<D, C, true> : paged_attn4_kernel<D, C, false>;
  const cudaError_t e = p.flat ? allow_smem<paged_attn4_kernel<D, C, true>>(bytes)
                               : allow_smem<paged_attn4_kernel<D, C, false>>(bytes);
  if (e != cudaSuccess) return e;
  // over the SMs first
  const unsigned grid = static_cast<unsigned>(std::max(
      std::min(p.workers, kAttn4Sms * C::MINB), (p.workers + C::kWarps - 1) / C::kWarps));
  const cudaError_t r = launch_behind(fn, dim3(grid), C::kThreads, bytes, s, p.after_store, p);
  if (r != cudaSuccess || !p.flat) return r;
  const int live = std::min(C::kRows, p.G * p.T);   // rows of a tile that are used
  const unsigned rows = static_cast<unsigned>(jobs * live);
  // More warps per row when a job has many runs.  32 warps or 8: one sequence of 16000 tokens (126
  // runs per job) 13.8 and 15.9 us, 8 of 1000-2000 (16) 15.8 and 13.7.  8 warps or 1: 8 of
  // 8000-16000 (28) 29.9 and 38.3, 16 of 1000-8000 with 32 query rows (9) 64.1 and 56.6.
  if (p.workers >= 64 * jobs)
    return launch_behind(attn4_merge_kernel<D, 32>, dim3(rows), 1024, 0, s, true, p, C::NTW,
                         C::kRows, live);
  if (p.workers >= 12 * jobs)
    return launch_behind(attn4_merge_kernel<D, 8>, dim3(rows), 256, 0, s, true, p, C::NTW, C::kRows,
                         live);
  return launch_behind(attn4_merge_kernel<D, 1>, dim3((rows + 3) / 4), 128, 0, s, true, p, C::NTW,
                       C::kRows, live);
}

template <int D>
cudaError_t launch_attn4(const Attn4Params& p, int rows, cudaStream_t s) {
  // Measured on 64 sequences of 512-4096 tokens (4 rows), 256 of 128-8192 (8 rows, with an
  // append) and one of 131071 (4 rows); other forms behind the committed one's 40.2 / 113.2 / 35.9
  // us.  One CTA of all the warps that an SM holds, so that its warps keep pace: three of four
  // warps each 40.4 / 118.1 / 37.0.  Pages in flight per warp, since with more of them the
  // queues in front of memory grow and every dependent fetch at a job's start waits longer: rings of
  // 3 pages 40.2 / 115.0 / 35.6, of 6 41.6 / 114.3 / 37.0.  16 warps (128 registers) 43.1 / 120.4 /
  // 38.8.
  if (rows <= 8) return launch_cfg4<D, Cfg4<1, 1, 4, 1, 12>>(p, s);
  // Two CTAs of four warps rather than one of eight: 16 rows (64 sequences of 512-4096 tokens) 59.4
  // and 60.3 us, 20 rows (32 of 2048-16384, with an append) 125.4 and 132.7; with 12 warps per SM
  // (168 registers: the output tile spills) 152.
  if (rows <= 16) return launch_cfg4<D, Cfg4<2, 1, 4, 2>>(p, s);
  if (rows <= 24) return launch_cfg4<D, Cfg4<3, 1, 3, 2>>(p, s);
  if (rows <= 32) return launch_cfg4<D, Cfg4<4, 1, 3, 2>>(p, s);
  return launch_cfg4<D, Cfg4<4, 2, 3, 2>>(p, s);
}

}  // namespace pa
