// Accumulated attention weights (pa_accumulate_weights).  For sequence b, kv head g
// with R = G * T query rows:
//   weights[b, g, j] = decay * weights[b, g, j] * [j < L - T] + sum_r softmax_r(j)
// A weight needs its row's final maximum and sum, so there are two launches.  The first
// reads the K pages once and writes the log2-domain scores, [pair][row][entry] in
// scratch, with a running (m, l) per row for each piece of a job; every warp is a worker
// with a page stream of its own (pa_runs.cuh).  The second joins the pieces' (m, l) and
// sums 2^(t - m) / l over the rows.  The scores are R * 4 bytes per entry against a page
// row of 2 D, D or 17 D / 32 bytes; scoring a second time instead reads the K pages twice
// and repeats the part that binds the first launch.
//
// Measured (GPU time of a call): 64 sequences of 512-4096 tokens, 32/8 heads of 128 dims, bf16
// pages, 58 us (302 MB of K; the first launch alone 53 us, 5.7 TB/s: bound by memory); five
// verified tokens over 4-bit pages, 32 sequences of 2048-16384, 113 us: 75 us of scores (160
// MB of K, 189 MB written; 69 us with the stores left out: bound by the score tiles), 37
// us of sums.  The sequences in 2, 3 or 4 parts through one smaller scratch, so that the scores
// stay in L2: 130, 146, 160 us.
#pragma once

#include "pa_runs.cuh"

namespace pa {

// NT n-tiles of 8 query rows per warp, NTW row columns, TP pages per step, STAGES staged
// steps per warp, MINB CTAs of 4 warps per SM.
template <int NT_, int NTW_, int TP_, int STAGES_, int MINB_>
struct ObserveCfg {
  static constexpr int NT = NT_, NTW = NTW_, TP = TP_, STAGES = STAGES_, MINB = MINB_;
  static constexpr int kWarps = 4, kThreads = 32 * kWarps, kRows = 8 * NT;
  static constexpr bool kQRegs = NT <= 2;
};

template <int F, int D, class C>
struct ObserveSmem {
  using P = Page<F, D>;
  static constexpr int kStageBytes = C::TP * P::kBytes;
  static constexpr int kRingBytes = C::STAGES * kStageBytes;
  static constexpr int kQBytes = C::kQRegs ? 0 : C::NT * QTileSmem<F, D>::kBytes;
  static constexpr int kWarpBytes = kRingBytes + kQBytes;
  static constexpr int kBytes = C::kWarps * kWarpBytes;
};

template <int F, int D, class C, bool kFlat>
__global__ void __launch_bounds__(C::kThreads, C::MINB)
    observe_scores_kernel(const ObserveParams p) {
  using P = Page<F, D>;
  using Sm = ObserveSmem<F, D, C>;
  constexpr int NT = C::NT, NTW = C::NTW, TP = C::TP, S = C::STAGES;
  extern __shared__ __align__(128) uint8_t smem_all[];
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, q4 = lane & 3;
  uint8_t* smem = smem_all + warp * Sm::kWarpBytes;
  const int G = p.G, T = p.T, nrows = G * T;
  const RunList list = observe_list(p, NTW);
  const int worker = blockIdx.x * C::kWarps + warp;
  const uint32_t page_stride = static_cast<uint32_t>(p.Hkv) * P::kBytes;
  const uint32_t ring = smem_u32(smem);
  const uint32_t swz = page_swizzle<F, D>(lane / P::kChunks, lane % P::kChunks);
  const uint32_t koff = ldsm_offset<F, D>(lane);

  // The scores are read again by the second launch, the pages (of a single column) not, so the
  // pages leave the L2 cache first, as the scores do once they have been summed.  64 sequences
  // of 512-4096 tokens, bf16: 61.9 -> 58.5 us; five verified tokens over 4-bit pages, whose pages
  // are fewer bytes than their scores: 111.6 -> 113.3.
  const uint64_t policy = read_policy(NTW == 1);
  Cursor<kFlat> cur;
  Segment seg;
  bool invalid = false;
  const bool any = cur.start(list, worker, lane, invalid);
  if (kFlat && worker == 0 && invalid) atomicOr(&g_pa_err, kErrBounds);
  if (!any) return;

  while (cur.next(list, seg, invalid)) {
    const int b = seg.b, L = seg.L, n = seg.n;
    const int g = seg.job / NTW, row0 = (seg.job % NTW) * C::kRows;
    QTileRaw<F, D> raw[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
      load_q_raw(raw[j], p.q, b, g, T, G, p.Hq, row0 + 8 * j, nrows, lane);

    const uint8_t* kbase =
        static_cast<const uint8_t*>(p.k_pool) + static_cast<size_t>(g) * P::kBytes;
    const uint8_t* ksrc = kbase + 16 * lane;
    const int32_t* trow = p.block_tables + static_cast<size_t>(b) * p.mbs + seg.page;
    int ids = 0;
    unsigned bad = 0, bad_before = 0;        // pages outside the pool: newest batch, the one before
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
    int it = 0;
    uint32_t st_in = ring;
    auto issue = [&]() {
      if (it < n) {
        if ((it & 31) == 0 && it > 0) load_ids(it);
#pragma unroll
        for (int k = 0; k < TP; ++k) {
          const uint32_t phys = __shfl_sync(0xffffffffu, ids, (it + k) & 31);
          const uint8_t* kp = at_page(ksrc, phys, page_stride);
          const uint32_t to = st_in + k * P::kBytes;
#pragma unroll
          for (int c = 0; c < P::kCodes / 512; ++c)
            cp_async_16_hint(to + (swz ^ swizzle_step<F, D>(c)) + 512 * c, kp + 512 * c, policy);
          if constexpr (P::kScales > 0) {
            if (lane < P::kScales / 16)
              cp_async_16_hint(to + P::kCodes + 16 * lane, kp + P::kCodes, policy);
          }
        }
        it += TP;
        st_in = st_in + Sm::kStageBytes == ring + Sm::kRingBytes ? ring : st_in + Sm::kStageBytes;
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue();

    QOperand<F, D, NT, C::kQRegs> qo;
    const float k_scale = F == kPageBf16 ? 1.f : p.k_scale[g];
    make_q_operand(qo, raw, smem + Sm::kRingBytes, p.scale_log2, k_scale, lane);

    float nm0[NT], nm1[NT], thr0[NT], thr1[NT], l0[NT], l1[NT];
    float* out[NT];                          // row 2q4 of the n-tile, entry gid
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      nm0[j] = nm1[j] = l0[j] = l1[j] = 0.f;
      thr0[j] = thr1[j] = -CUDART_INF_F;
      out[j] = p.scores +
               ((static_cast<size_t>(b) * p.Hkv + g) * nrows + row0 + 8 * j + 2 * q4) *
                   p.max_entries +
               seg.page * kBlockSize + gid;
    }
    const int part_end = min(L, (seg.page + n) * kBlockSize);
    const int hi = min(L - T, part_end - 1) - (kBlockSize - 1);   // first entry of a full page
    int tok0 = seg.page * kBlockSize;
    uint32_t st = ring;

    for (int i = 0; i * TP < n; ++i) {
      cp_async_wait<S - 2>();
      __syncwarp();
      issue();
      float t[TP][NT][4];
#pragma unroll
      for (int k = 0; k < TP; ++k) page_scores<F, D>(t[k], st + k * P::kBytes, koff, qo, lane);
      if (tok0 + (TP - 1) * kBlockSize > hi || (bad | bad_before) != 0) {
#pragma unroll
        for (int k = 0; k < TP; ++k) {
          const int i0 = i * TP + k;
          const unsigned bits = (it - 1) >> 5 == i0 >> 5 ? bad : bad_before;
          const int end = (bits >> (i0 & 31)) & 1u ? 0 : part_end;
          const int j0 = tok0 + k * kBlockSize + gid, j1 = j0 + 8;
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const int r = row0 + 8 * j + 2 * q4;
            const int a = r < nrows ? L - T + r / G : -1;
            const int c = r + 1 < nrows ? L - T + (r + 1) / G : -1;
            if (j0 >= end || j0 > a) t[k][j][0] = -CUDART_INF_F;
            if (j0 >= end || j0 > c) t[k][j][1] = -CUDART_INF_F;
            if (j1 >= end || j1 > a) t[k][j][2] = -CUDART_INF_F;
            if (j1 >= end || j1 > c) t[k][j][3] = -CUDART_INF_F;
          }
        }
      }
      bool over = false;
      float x0[NT], x1[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        x0[j] = x1[j] = -CUDART_INF_F;
#pragma unroll
        for (int k = 0; k < TP; ++k) {
          x0[j] = fmaxf(x0[j], fmaxf(t[k][j][0], t[k][j][2]));
          x1[j] = fmaxf(x1[j], fmaxf(t[k][j][1], t[k][j][3]));
        }
        over |= x0[j] > thr0[j] || x1[j] > thr1[j];
      }
      // per lane: a sum over its own entries against its own reference, joined at the end
      if (over) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if (x0[j] > thr0[j]) {
            const float nm = -x0[j] * qo.rs0[j];
            l0[j] *= thr0[j] == -CUDART_INF_F ? 0.f : hw_exp2(nm - nm0[j]);
            nm0[j] = nm;
            thr0[j] = x0[j] + 30.f / qo.rs0[j];
          }
          if (x1[j] > thr1[j]) {
            const float nm = -x1[j] * qo.rs1[j];
            l1[j] *= thr1[j] == -CUDART_INF_F ? 0.f : hw_exp2(nm - nm1[j]);
            nm1[j] = nm;
            thr1[j] = x1[j] + 30.f / qo.rs1[j];
          }
        }
      }
#pragma unroll
      for (int k = 0; k < TP; ++k) {
        // a step past the job's last page stores nothing of it
        const bool store = TP == 1 || i * TP + k < n;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const float a0 = t[k][j][0] * qo.rs0[j], a2 = t[k][j][2] * qo.rs0[j];
          const float a1 = t[k][j][1] * qo.rs1[j], a3 = t[k][j][3] * qo.rs1[j];
          l0[j] += hw_exp2(a0 + nm0[j]) + hw_exp2(a2 + nm0[j]);
          l1[j] += hw_exp2(a1 + nm1[j]) + hw_exp2(a3 + nm1[j]);
          const int r = row0 + 8 * j + 2 * q4;
          float* o = out[j] + k * kBlockSize;
          if (store && r < nrows) {
            o[0] = a0;
            o[8] = a2;
          }
          if (store && r + 1 < nrows) {
            o[p.max_entries] = a1;
            o[p.max_entries + 8] = a3;
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) out[j] += TP * kBlockSize;
      tok0 += TP * kBlockSize;
      st = st + Sm::kStageBytes == ring + Sm::kRingBytes ? ring : st + Sm::kStageBytes;
    }
    cp_async_wait<0>();
    __syncwarp();
    const size_t job_slot = static_cast<size_t>(b) * list.heads + seg.job;
    const size_t slot = !kFlat      ? job_slot * p.max_parts + seg.part
                        : seg.whole ? static_cast<size_t>(p.workers) * 2 + job_slot
                                    : static_cast<size_t>(worker) * 2 + seg.second;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float m0 = thr0[j] == -CUDART_INF_F ? -CUDART_INF_F : -nm0[j];
      float m1 = thr1[j] == -CUDART_INF_F ? -CUDART_INF_F : -nm1[j];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        const float a = __shfl_xor_sync(0xffffffffu, m0, o);
        const float x = __shfl_xor_sync(0xffffffffu, l0[j], o);
        const float c = __shfl_xor_sync(0xffffffffu, m1, o);
        const float y = __shfl_xor_sync(0xffffffffu, l1[j], o);
        const float M0 = fmaxf(m0, a), M1 = fmaxf(m1, c);
        const float u0 = M0 == -CUDART_INF_F ? 0.f : M0, u1 = M1 == -CUDART_INF_F ? 0.f : M1;
        l0[j] = l0[j] * hw_exp2(m0 - u0) + x * hw_exp2(a - u0);
        l1[j] = l1[j] * hw_exp2(m1 - u1) + y * hw_exp2(c - u1);
        m0 = M0;
        m1 = M1;
      }
      if (gid == 0) {
        float2* ml = p.ml + slot * C::kRows + 8 * j + 2 * q4;
        ml[0] = make_float2(m0, l0[j]);
        ml[1] = make_float2(m1, l1[j]);
      }
    }
  }
  if (!kFlat && invalid && lane == 0) atomicOr(&g_pa_err, kErrBounds);
}

template <int F, int D, class C>
cudaError_t launch_observe_cfg(const ObserveParams& p, cudaStream_t s) {
  constexpr int bytes = ObserveSmem<F, D, C>::kBytes;
  constexpr Attn4Tile tile = observe_tile(C::kRows * C::NTW);
  static_assert(tile.nt == C::NT && tile.ntw == C::NTW && tile.ctas == C::MINB, "the host's tile");
  auto fn = p.flat ? observe_scores_kernel<F, D, C, true> : observe_scores_kernel<F, D, C, false>;
  const cudaError_t e = p.flat ? allow_smem<observe_scores_kernel<F, D, C, true>>(bytes)
                               : allow_smem<observe_scores_kernel<F, D, C, false>>(bytes);
  if (e != cudaSuccess) return e;
  return launch_behind(fn, dim3((p.workers + C::kWarps - 1) / C::kWarps), C::kThreads, bytes, s,
                       false, p);
}

template <int F, int D>
cudaError_t launch_observe(const ObserveParams& p, int rows, cudaStream_t s) {
  // 8 to 12 KB of pages staged per warp
  constexpr int TP = F == kPageBf16 ? 1 : 2, ST = F == kPageInt4 ? 4 : 3;
  if (rows <= 8) return launch_observe_cfg<F, D, ObserveCfg<1, 1, TP, ST, 4>>(p, s);
  if (rows <= 16) return launch_observe_cfg<F, D, ObserveCfg<2, 1, 1, 3, 3>>(p, s);
  if (rows <= 24) return launch_observe_cfg<F, D, ObserveCfg<3, 1, 1, 3, 3>>(p, s);
  if (rows <= 32) return launch_observe_cfg<F, D, ObserveCfg<4, 1, 1, 3, 2>>(p, s);
  return launch_observe_cfg<F, D, ObserveCfg<4, 2, 1, 3, 2>>(p, s);
}

}  // namespace pa
