// Accumulated attention weights (pa_accumulate_weights).  For sequence b, kv head g
// with R = G * T query rows:
//   weights[b, g, j] = decay * weights[b, g, j] * [j < L - T] + sum_r softmax_r(j)
// Two launches.  The first reads the K pages once, writes the log2-domain scores
// t[j][r] to scratch with every chunk's running maximum and sum per row; the second
// joins the chunks' (m, l) and sums 2^(t - m) / l over the rows.  The scores are
// R * 4 bytes per entry against the page's 2 D, D or D/2 + D/32, and are read back
// while they are still in L2 for all but the largest batches.
#pragma once

#include "pa_pages.cuh"

namespace pa {

template <int NT_, int NTW_, int PL_, int STAGES_, int MINB_>
struct ObserveCfg {
  static constexpr int NT = NT_, NTW = NTW_, PL = PL_, STAGES = STAGES_, MINB = MINB_;
  static constexpr int kWarps = NTW * PL, kThreads = 32 * kWarps, kRows = 8 * NT * NTW;
  static constexpr bool kQRegs = NT <= 2;
};

template <int F, int D, class C>
struct ObserveSmem {
  using P = Page<F, D>;
  static constexpr int kQOff = C::kWarps * C::STAGES * P::kBytes;
  static constexpr int kMlOff = kQOff + C::kRows / 8 * QTileSmem<F, D>::kBytes;
  static constexpr int kBytes = kMlOff + C::kWarps * 8 * C::NT * 8;
};

template <int F, int D, class C>
__global__ void __launch_bounds__(C::kThreads, C::MINB) observe_scores_kernel(const ObserveParams p) {
  using P = Page<F, D>;
  using Sm = ObserveSmem<F, D, C>;
  constexpr int NT = C::NT, NTW = C::NTW, PL = C::PL, S = C::STAGES;
  extern __shared__ __align__(128) uint8_t smem[];
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, q4 = lane & 3;
  const int chunk = static_cast<int>(blockIdx.x / (p.Hkv * p.num_seqs));
  const int b = static_cast<int>((blockIdx.x / p.Hkv) % p.num_seqs);
  const int g = static_cast<int>(blockIdx.x % p.Hkv);
  const int G = p.G, T = p.T;
  const int L = p.context_lens[b];
  if (L < T || L > p.max_ctx) {
    if (threadIdx.x == 0 && chunk == 0) atomicOr(&g_pa_err, kErrBounds);
    return;
  }
  const int nblk = (L + kBlockSize - 1) / kBlockSize;
  const int pg0 = chunk * p.ppb;
  if (pg0 >= nblk) return;
  const int npages = min(pg0 + p.ppb, nblk) - pg0;
  const int nrows = G * T;
  const int col = warp % NTW, pl = warp / NTW;
  const int n = pl < npages ? (npages - pl + PL - 1) / PL : 0;
  const int32_t* trow = p.block_tables + static_cast<size_t>(b) * p.mbs + pg0 + pl;
  const uint8_t* kpool = static_cast<const uint8_t*>(p.k_pool);

  const uint32_t ring = smem_u32(smem) + warp * S * P::kBytes;
  int ids = lane < n ? __ldg(trow + lane * PL) : 0;
  unsigned okbits = 0;
  auto issue = [&](int i) {
    if (i < n) {
      if ((i & 31) == 0 && i > 0) ids = i + lane < n ? __ldg(trow + (i + lane) * PL) : 0;
      const int phys = __shfl_sync(0xffffffffu, ids, i & 31);
      const bool ok = static_cast<unsigned>(phys) < static_cast<unsigned>(p.num_blocks);
      const unsigned bit = 1u << (i % S);
      okbits = ok ? okbits | bit : okbits & ~bit;
      if (!ok && lane == 0) atomicOr(&g_pa_err, kErrBounds);
      const size_t off = (static_cast<size_t>(ok ? phys : 0) * p.Hkv + g) * P::kBytes;
      stage_page<F, D>(ring + (i % S) * P::kBytes, kpool + off, lane, ok);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(i);

  uint8_t* qt = smem + Sm::kQOff;
  for (int j = warp; j < NT * NTW; j += C::kWarps) {
    QTileRaw<F, D> raw;
    QTile<F, D> tile;
    load_q_raw(raw, p.q, b, g, T, G, p.Hq, 8 * j, nrows, lane);
    make_q_tile(tile, raw, p.scale_log2, F == kPageBf16 ? 1.f : p.k_scale[g], lane);
    put_q_tile(qt + j * QTileSmem<F, D>::kBytes, tile, lane);
  }
  __syncthreads();
  QOperand<F, D, NT, C::kQRegs> qo;
  qo.load(qt + col * NT * QTileSmem<F, D>::kBytes, lane);

  int lim0[NT], lim1[NT];
  float m0[NT], m1[NT], l0[NT], l1[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int r = 8 * (col * NT + j) + 2 * q4;
    lim0[j] = r < nrows ? L - T + r / G : -1;
    lim1[j] = r + 1 < nrows ? L - T + (r + 1) / G : -1;
    m0[j] = m1[j] = -CUDART_INF_F;
    l0[j] = l1[j] = 0.f;
  }
  const uint32_t koff = ldsm_offset<F, D>(lane);
  // scores of (b, g): [entry][row], rows padded to an even count
  float* out = p.scores + (static_cast<size_t>(b) * p.Hkv + g) * p.max_entries * p.row_stride;

  for (int i = 0; i < n; ++i) {
    cp_async_wait<S - 2>();
    __syncwarp();
    const bool ok = (okbits >> (i % S)) & 1u;
    const uint32_t st = ring + (i % S) * P::kBytes;
    issue(i + S - 1);
    const int tok0 = (pg0 + pl + i * PL) * kBlockSize;
    float t[NT][4];
    page_scores<F, D>(t, st, koff, qo, lane);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int j0 = tok0 + gid, j1 = j0 + 8;
      t[j][0] *= qo.rs0[j];
      t[j][1] *= qo.rs1[j];
      t[j][2] *= qo.rs0[j];
      t[j][3] *= qo.rs1[j];
      if (!ok || j0 > lim0[j]) t[j][0] = -CUDART_INF_F;
      if (!ok || j0 > lim1[j]) t[j][1] = -CUDART_INF_F;
      if (!ok || j1 > lim0[j]) t[j][2] = -CUDART_INF_F;
      if (!ok || j1 > lim1[j]) t[j][3] = -CUDART_INF_F;
      const int r = 8 * (col * NT + j) + 2 * q4;
      if (r < nrows) {
        if (j0 < L)
          *reinterpret_cast<float2*>(out + static_cast<size_t>(j0) * p.row_stride + r) =
              make_float2(t[j][0], t[j][1]);
        if (j1 < L)
          *reinterpret_cast<float2*>(out + static_cast<size_t>(j1) * p.row_stride + r) =
              make_float2(t[j][2], t[j][3]);
      }
      // per lane: its own entries' running maximum and sum, joined after the loop
      const float x0 = fmaxf(t[j][0], t[j][2]), x1 = fmaxf(t[j][1], t[j][3]);
      if (x0 > m0[j]) {
        l0[j] *= hw_exp2(m0[j] - x0);
        m0[j] = x0;
      }
      if (x1 > m1[j]) {
        l1[j] *= hw_exp2(m1[j] - x1);
        m1[j] = x1;
      }
      const float mu0 = m0[j] == -CUDART_INF_F ? 0.f : m0[j];
      const float mu1 = m1[j] == -CUDART_INF_F ? 0.f : m1[j];
      l0[j] += hw_exp2(t[j][0] - mu0) + hw_exp2(t[j][2] - mu0);
      l1[j] += hw_exp2(t[j][1] - mu1) + hw_exp2(t[j][3] - mu1);
    }
  }
  cp_async_wait<0>();
  float2* ml = reinterpret_cast<float2*>(smem + Sm::kMlOff);
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      const float a = __shfl_xor_sync(0xffffffffu, m0[j], o);
      const float x = __shfl_xor_sync(0xffffffffu, l0[j], o);
      const float c = __shfl_xor_sync(0xffffffffu, m1[j], o);
      const float y = __shfl_xor_sync(0xffffffffu, l1[j], o);
      const float M0 = fmaxf(m0[j], a), M1 = fmaxf(m1[j], c);
      const float u0 = M0 == -CUDART_INF_F ? 0.f : M0, u1 = M1 == -CUDART_INF_F ? 0.f : M1;
      l0[j] = l0[j] * hw_exp2(m0[j] - u0) + x * hw_exp2(a - u0);
      l1[j] = l1[j] * hw_exp2(m1[j] - u1) + y * hw_exp2(c - u1);
      m0[j] = M0;
      m1[j] = M1;
    }
    if (gid == 0) {
      ml[warp * 8 * NT + 8 * j + 2 * q4] = make_float2(m0[j], l0[j]);
      ml[warp * 8 * NT + 8 * j + 2 * q4 + 1] = make_float2(m1[j], l1[j]);
    }
  }
  __syncthreads();
  for (int r = threadIdx.x; r < nrows; r += C::kThreads) {
    const int cl = r / (8 * NT), rl = r % (8 * NT);
    float M = -CUDART_INF_F, l = 0.f;
    for (int k = 0; k < PL; ++k) M = fmaxf(M, ml[(k * NTW + cl) * 8 * NT + rl].x);
    const float u = M == -CUDART_INF_F ? 0.f : M;
    for (int k = 0; k < PL; ++k) {
      const float2 x = ml[(k * NTW + cl) * 8 * NT + rl];
      l += x.y * hw_exp2(x.x - u);
    }
    p.ml[((static_cast<size_t>(b) * p.Hkv + g) * p.max_chunks + chunk) * nrows + r] =
        make_float2(M, l);
  }
}

template <int F, int D, class C>
cudaError_t launch_observe_cfg(const ObserveParams& p, unsigned units, cudaStream_t s) {
  constexpr int bytes = ObserveSmem<F, D, C>::kBytes;
  auto fn = observe_scores_kernel<F, D, C>;
  const cudaError_t e =
      cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  fn<<<units, C::kThreads, bytes, s>>>(p);
  return cudaGetLastError();
}

template <int F, int D>
cudaError_t launch_observe(const ObserveParams& p, int rows, unsigned units, cudaStream_t s) {
  constexpr int ST = F == kPageBf16 ? 3 : (F == kPageFp8 ? 4 : 6);
  if (rows <= 8) return launch_observe_cfg<F, D, ObserveCfg<1, 1, 4, ST, 4>>(p, units, s);
  if (rows <= 16) return launch_observe_cfg<F, D, ObserveCfg<2, 1, 4, ST, 3>>(p, units, s);
  if (rows <= 32) return launch_observe_cfg<F, D, ObserveCfg<4, 1, 4, ST, 2>>(p, units, s);
  return launch_observe_cfg<F, D, ObserveCfg<4, 2, 2, ST, 2>>(p, units, s);
}

}  // namespace pa
