// Attention over 4-bit pages (pa_attention_int4): one CTA per work unit
// (partition of one sequence's pages, kv head), PL page lanes of warps that each
// stream their own pages.
#pragma once

#include "pa_pages.cuh"

namespace pa {

// NT n-tiles of 8 query rows per warp, NTW warp columns, PL page lanes, STAGES
// staged pages per warp, MINB CTAs per SM.
template <int NT_, int NTW_, int PL_, int STAGES_, int MINB_>
struct Cfg4 {
  static constexpr int NT = NT_, NTW = NTW_, PL = PL_, STAGES = STAGES_, MINB = MINB_;
  static constexpr int kWarps = NTW * PL, kThreads = 32 * kWarps, kRows = 8 * NT * NTW;
  static constexpr bool kQRegs = NT <= 2;
};

template <int D, class C>
struct Smem4 {
  using P = Page<kPageInt4, D>;
  using Q = QTile<kPageInt4, D, C::kRows>;
  static constexpr int kStageBytes = 2 * P::kBytes;         // a K page, then a V page
  static constexpr int kQOff = C::kWarps * C::STAGES * kStageBytes;
  static constexpr int kOStride = D + 4;
  // merge buffer: (m, l, O) of every warp's rows, over the drained rings
  static constexpr int kWarpFloats = 8 * C::NT * (kOStride + 2);
  static constexpr int kMergeBytes = C::kWarps * kWarpFloats * 4;
  static constexpr int kBytes = kQOff + Q::kBytes > kMergeBytes ? kQOff + Q::kBytes : kMergeBytes;
  static_assert(kStageBytes % 16 == 0 && kQOff % 16 == 0, "16-byte copies");
};

template <int D, class C>
__global__ void __launch_bounds__(C::kThreads, C::MINB) paged_attn4_kernel(const AttnParams p) {
  using P = Page<kPageInt4, D>;
  using Sm = Smem4<D, C>;
  constexpr int NT = C::NT, NTW = C::NTW, PL = C::PL, S = C::STAGES;
  constexpr int NG = P::kGroups;
  extern __shared__ __align__(128) uint8_t smem[];
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, q4 = lane & 3;

  // ---------------------------------------------------------------- unit
  const int unit_p = static_cast<int>(blockIdx.x / (p.Hkv * p.num_seqs));
  const int b = static_cast<int>((blockIdx.x / p.Hkv) % p.num_seqs);
  const int g = static_cast<int>(blockIdx.x % p.Hkv);
  const int G = p.G, T = p.T;
  const int L = p.context_lens[b];
  if (L < T || L > p.max_ctx) {
    if (threadIdx.x == 0 && unit_p == 0) atomicOr(&g_pa_err, kErrBounds);
    return;
  }
  const int nblk = (L + kBlockSize - 1) / kBlockSize;
  const int first = p.window > 0 ? max(0, L - T - p.window + 1) / kBlockSize : 0;
  const int pg0 = first + unit_p * p.ppb;
  if (pg0 >= nblk) return;
  const int pg1 = min(pg0 + p.ppb, nblk);
  const bool direct = nblk - first <= p.ppb;
  const int nrows = G * T;
  const int col = warp % NTW, pl = warp / NTW;
  const int npages = pg1 - pg0;
  const int n = pl < npages ? (npages - pl + PL - 1) / PL : 0;   // this warp's pages
  const int32_t* trow = p.block_tables + static_cast<size_t>(b) * p.mbs + pg0 + pl;
  const uint8_t* kpool = static_cast<const uint8_t*>(p.k_pool);
  const uint8_t* vpool = static_cast<const uint8_t*>(p.v_pool);

  // ---------------------------------------------------------------- page stream
  const uint32_t ring = smem_u32(smem) + warp * S * Sm::kStageBytes;
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
      const uint32_t st = ring + (i % S) * Sm::kStageBytes;
      stage_page<kPageInt4, D>(st, kpool + off, lane, ok);
      stage_page<kPageInt4, D>(st + P::kBytes, vpool + off, lane, ok);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(i);

  uint8_t* qt = smem + Sm::kQOff;
  load_q_tile<kPageInt4, D, C::kRows>(qt, p.q, b, g, T, G, p.Hq, nrows, p.scale_log2,
                                      p.k_scale[g], warp, lane, C::kWarps);
  __syncthreads();
  QOperand<kPageInt4, D, NT, C::kQRegs> qo;
  qo.template load<C::kRows>(qt, col * NT, lane);

  int lim0[NT], lim1[NT];                    // last visible position of rows 2q4, 2q4 + 1
  int minlim = 0x7fffffff;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int r = 8 * (col * NT + j) + 2 * q4;
    lim0[j] = r < nrows ? L - T + r / G : 0x7fffffff;
    lim1[j] = r + 1 < nrows ? L - T + (r + 1) / G : 0x7fffffff;
    minlim = min(minlim, min(lim0[j], lim1[j]));
  }

  float acc[NT][D / 16][4], z[NT][4], m0[NT], m1[NT], l0[NT], l1[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    m0[j] = m1[j] = -CUDART_INF_F;
    l0[j] = l1[j] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) z[j][e] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][k][e] = 0.f;
  }
  const uint32_t koff = ldsm_offset<kPageInt4, D>(lane);

  for (int i = 0; i < n; ++i) {
    cp_async_wait<S - 2>();
    __syncwarp();
    const bool ok = (okbits >> (i % S)) & 1u;
    const uint32_t st = ring + (i % S) * Sm::kStageBytes;
    issue(i + S - 1);                        // into the stage consumed last
    if (!ok) continue;
    const int tok0 = (pg0 + pl + i * PL) * kBlockSize;
    float t[NT][4];
    page_scores<kPageInt4, D>(t, st, koff, qo, lane);

    const int nvalid = L - tok0;
    const bool interior = __all_sync(0xffffffffu, tok0 + kBlockSize - 1 <= minlim &&
                                                      tok0 + p.wspan >= L && nvalid >= kBlockSize);
    if (!interior) {
      const unsigned u0 = static_cast<unsigned>(tok0 + gid), u1 = u0 + 8;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const unsigned a = static_cast<unsigned>(lim0[j]), c = static_cast<unsigned>(lim1[j]);
        t[j][0] = a - u0 < p.wcap ? t[j][0] : -CUDART_INF_F;
        t[j][1] = c - u0 < p.wcap ? t[j][1] : -CUDART_INF_F;
        t[j][2] = a - u1 < p.wcap ? t[j][2] : -CUDART_INF_F;
        t[j][3] = c - u1 < p.wcap ? t[j][3] : -CUDART_INF_F;
      }
    }

    // Online softmax: the reference m of a row moves only when a score passes it by
    // 7, so a weight is at most 2^7 and, times a V scale (at most 448), an f16 value.
    bool over = false;
#pragma unroll
    for (int j = 0; j < NT; ++j)
      over |= fmaxf(t[j][0], t[j][2]) > m0[j] + 7.f || fmaxf(t[j][1], t[j][3]) > m1[j] + 7.f;
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float x0 = fmaxf(t[j][0], t[j][2]), x1 = fmaxf(t[j][1], t[j][3]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, o));
          x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, o));
        }
        const bool up0 = x0 > m0[j] + 7.f, up1 = x1 > m1[j] + 7.f;
        const float f0 = up0 ? hw_exp2(m0[j] - x0) : 1.f, f1 = up1 ? hw_exp2(m1[j] - x1) : 1.f;
        if (up0) m0[j] = x0;
        if (up1) m1[j] = x1;
        l0[j] *= f0;
        l1[j] *= f1;
        z[j][0] *= f0;
        z[j][1] *= f1;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          acc[j][k][0] *= f0;
          acc[j][k][1] *= f1;
          acc[j][k][2] *= f0;
          acc[j][k][3] *= f1;
        }
      }
    }
    uint32_t ph0[NT], ph1[NT];               // P^T: tokens 2q, 2q+1 and 2q+8, 2q+9 of row gid
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const float mu0 = m0[j] == -CUDART_INF_F ? 0.f : m0[j];
      const float mu1 = m1[j] == -CUDART_INF_F ? 0.f : m1[j];
      const float p0 = hw_exp2(t[j][0] - mu0), p1 = hw_exp2(t[j][1] - mu1);
      const float p2 = hw_exp2(t[j][2] - mu0), p3 = hw_exp2(t[j][3] - mu1);
      l0[j] += p0 + p2;
      l1[j] += p1 + p3;
      ph0[j] = movmatrix_trans(half2_bits(__floats2half2_rn(p0, p1)));
      ph1[j] = movmatrix_trans(half2_bits(__floats2half2_rn(p2, p3)));
    }

    // V scales of tokens 2q, 2q+1 (w0, w1) and 2q+8, 2q+9 (w2, w3), a byte per group
    uint32_t w0, w1, w2, w3;
    {
      const uint32_t a = st + P::kBytes + P::kCodes + 2 * q4 * NG;
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
    if (nvalid < kBlockSize) {               // rows past the context may hold any scale, even NaN
      w0 = 2 * q4 < nvalid ? w0 : 0u;
      w1 = 2 * q4 + 1 < nvalid ? w1 : 0u;
      w2 = 2 * q4 + 8 < nvalid ? w2 : 0u;
      w3 = 2 * q4 + 9 < nvalid ? w3 : 0u;
    }
#pragma unroll
    for (int g2 = 0; g2 < NG; g2 += 2) {
      // byte pairs (token 2q, token 2q+1) of groups g2 and g2 + 1
      const uint32_t sel = g2 == 0 ? 0x5140u : 0x7362u;
      const uint32_t sa = __byte_perm(w0, w1, sel), sb = __byte_perm(w2, w3, sel);
      uint32_t w[4];
      ldsm_x4_trans(w[0], w[1], w[2], w[3], st + P::kBytes + (koff ^ (g2 << 4)));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int gr = g2 + h;
        const uint32_t fa = e4m3x2_to_f16x2(sa >> (16 * h)), fb = e4m3x2_to_f16x2(sb >> (16 * h));
        const uint32_t x0 = w[2 * h], x1 = w[2 * h + 1];
        const uint32_t y0 = x0 >> 8, y1 = x1 >> 8;
        const uint32_t one = gid == gr ? 0x3C003C00u : 0u;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint32_t b0 = half2_bits(__hmul2(*reinterpret_cast<const __half2*>(&ph0[j]),
                                                 *reinterpret_cast<const __half2*>(&fa)));
          const uint32_t b1 = half2_bits(__hmul2(*reinterpret_cast<const __half2*>(&ph1[j]),
                                                 *reinterpret_cast<const __half2*>(&fb)));
          // row gr of z: the group's sum of scaled weights (for the codes' offset 8)
          mma_f16_16816(z[j], one, 0u, one, 0u, b0, b1);
          // dims 32 gr + 4 gid + 0 and 2, then + 1 and 3 (times 16)
          mma_f16_16816(acc[j][2 * gr], x0 & kNibLo, y0 & kNibLo, x1 & kNibLo, y1 & kNibLo, b0,
                        b1);
          mma_f16_16816(acc[j][2 * gr + 1], x0 & kNibHi, y0 & kNibHi, x1 & kNibHi, y1 & kNibHi,
                        b0, b1);
        }
      }
    }
  }
  cp_async_wait<0>();

  // ---------------------------------------------------------------- merge of the page lanes
  __syncthreads();
  constexpr int OS = Sm::kOStride;
  float* mb = reinterpret_cast<float*>(smem) + warp * Sm::kWarpFloats;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l0[j] += __shfl_xor_sync(0xffffffffu, l0[j], o);
      l1[j] += __shfl_xor_sync(0xffffffffu, l1[j], o);
    }
    const int r = 8 * j + 2 * q4;
    if (gid == 0) {
      mb[r] = m0[j];
      mb[r + 1] = m1[j];
      mb[8 * NT + r] = l0[j];
      mb[8 * NT + r + 1] = l1[j];
    }
    float* o0 = mb + 16 * NT + r * OS;
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      const float z0 = 8.f * __shfl_sync(0xffffffffu, z[j][0], gr * 4 + q4);
      const float z1 = 8.f * __shfl_sync(0xffffffffu, z[j][1], gr * 4 + q4);
      const float* a = acc[j][2 * gr];
      const float* c = acc[j][2 * gr + 1];
      constexpr float A = 16777216.f, B = 1048576.f;   // 2^24, 2^20
      *reinterpret_cast<float4*>(o0 + 32 * gr + 4 * gid) =
          make_float4(fmaf(a[0], A, -z0), fmaf(c[0], B, -z0), fmaf(a[2], A, -z0),
                      fmaf(c[2], B, -z0));
      *reinterpret_cast<float4*>(o0 + OS + 32 * gr + 4 * gid) =
          make_float4(fmaf(a[1], A, -z1), fmaf(c[1], B, -z1), fmaf(a[3], A, -z1),
                      fmaf(c[3], B, -z1));
    }
  }
  __syncthreads();
  const float out_scale = p.v_scale[g];
  const float* all = reinterpret_cast<const float*>(smem);
  constexpr int CH = D / 4;                  // four dims per thread and step
  for (int idx = threadIdx.x; idx < nrows * CH; idx += C::kThreads) {
    const int r = idx / CH, ch = idx % CH;
    const int cl = r / (8 * NT), rl = r % (8 * NT);
    float M = -CUDART_INF_F;
#pragma unroll
    for (int k = 0; k < PL; ++k) M = fmaxf(M, all[(k * NTW + cl) * Sm::kWarpFloats + rl]);
    float l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < PL; ++k) {
      const float* w = all + (k * NTW + cl) * Sm::kWarpFloats;
      const float f = w[rl] == -CUDART_INF_F ? 0.f : hw_exp2(w[rl] - M);
      const float4 x = *reinterpret_cast<const float4*>(w + 16 * NT + rl * OS + 4 * ch);
      l += f * w[8 * NT + rl];
      o[0] += f * x.x;
      o[1] += f * x.y;
      o[2] += f * x.z;
      o[3] += f * x.w;
    }
    const float inv = l > 0.f ? out_scale / l : 0.f;
    const size_t orow = (static_cast<size_t>(b) * T + r / G) * p.Hq + g * G + r % G;
    if (direct) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(o[0] * inv, o[1] * inv);
      const __nv_bfloat162 c = __floats2bfloat162_rn(o[2] * inv, o[3] * inv);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + orow * D + 4 * ch) =
          make_uint2(bf162_bits(a), bf162_bits(c));
    } else {
      const size_t at = orow * p.max_parts + unit_p;
      *reinterpret_cast<float4*>(p.part_o + at * D + 4 * ch) =
          make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
      if (ch == 0) p.part_ml[at] = make_float2(M, l);
    }
  }
}

template <int D, class C>
cudaError_t launch_cfg4(const AttnParams& p, unsigned units, cudaStream_t s) {
  constexpr int bytes = Smem4<D, C>::kBytes;
  auto fn = paged_attn4_kernel<D, C>;
  const cudaError_t e =
      cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  fn<<<units, C::kThreads, bytes, s>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_attn4(const AttnParams& p, int rows, unsigned units, cudaStream_t s) {
  if (rows <= 8) return launch_cfg4<D, Cfg4<1, 1, 4, 6, 4>>(p, units, s);
  if (rows <= 16) return launch_cfg4<D, Cfg4<2, 1, 4, 6, 3>>(p, units, s);
  if (rows <= 24) return launch_cfg4<D, Cfg4<3, 1, 4, 6, 2>>(p, units, s);
  if (rows <= 32) return launch_cfg4<D, Cfg4<4, 1, 4, 6, 2>>(p, units, s);
  return launch_cfg4<D, Cfg4<4, 2, 2, 6, 2>>(p, units, s);
}

}  // namespace pa
