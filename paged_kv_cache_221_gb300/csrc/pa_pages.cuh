// K/V page formats as the warp-streaming kernels see them (attention over 4-bit
// pages, accumulated attention weights): geometry, staging of a page by one warp
// with cp.async, and the score tile S^T[16 tokens x 8 rows] of a staged K page.
//
// A page is 16 tokens of one (block, kv head).  Formats:
//   bf16   16 rows of D bf16
//   FP8    16 rows of D E4M3 codes (K; the V pages of this format are transposed)
//   INT4   16 rows of D/2 bytes, dim d in byte d/2 (even d in the low nibble), code
//          u in 1 .. 15 standing for u - 8; then 16 rows of D/32 E4M3 scales, one
//          for each group of 32 dims.  value = (u - 8) * scale * head_scale.
//
// INT4 codes become tensor-core operands with one mask each.  A nibble of an f16
// word at bits 0-3 is the f16 subnormal u * 2^-24, at bits 4-7 it is 16 u * 2^-24;
// both are exact, and mma.sync multiplies subnormal f16 operands exactly.  A 32-bit word
// of eight nibbles therefore gives its four operand registers with one shift and
// four masks; the factors 2^24 and 16 are powers of two folded elsewhere (the even
// and odd dims of Q, the output), and the offset 8 leaves the contraction as 8 * (sum
// over the group of scale * the other operand), one more small tile.  E2M1 codes would need a conversion for
// every pair of values, and have a larger error on normally distributed values.
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>

#include "pa_ptx.cuh"

namespace pa {

enum PageFormat { kPageBf16 = 0, kPageFp8 = 1, kPageInt4 = 2 };

constexpr int kGroupDims = 32;               // dims that share an INT4 scale

template <int F, int D>
struct Page {
  static constexpr int kRow = F == kPageBf16 ? 2 * D : (F == kPageFp8 ? D : D / 2);
  static constexpr int kChunks = kRow / 16;  // 16-byte chunks per token row
  static constexpr int kGroups = D / kGroupDims;
  static constexpr int kCodes = kBlockSize * kRow;
  static constexpr int kScales = F == kPageInt4 ? kBlockSize * kGroups : 0;
  static constexpr int kBytes = kCodes + kScales;
};

// Byte offset of 16-byte chunk ch of token row `row` in a staged page: chunks are
// permuted within a row so that the eight rows of an 8x8 ldmatrix tile fall in
// different banks.
template <int F, int D>
__device__ __forceinline__ uint32_t page_swizzle(int row, int ch) {
  using P = Page<F, D>;
  if constexpr (P::kChunks >= 8)
    return row * P::kRow + ((ch ^ (row & 7)) << 4);
  else if constexpr (P::kChunks == 4)
    return row * P::kRow + ((ch ^ ((row >> 1) & 3)) << 4);
  else
    return row * P::kRow + ((ch ^ ((row >> 2) & 1)) << 4);
}

__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One warp copies a page to shared memory (asynchronously); ok = false zero-fills it.
template <int F, int D>
__device__ __forceinline__ void stage_page(uint32_t dst, const uint8_t* src, int lane, bool ok) {
  using P = Page<F, D>;
  const uint32_t n = ok ? 16u : 0u;
#pragma unroll
  for (int c0 = 0; c0 < P::kCodes / 16; c0 += 32) {
    const int c = c0 + lane;
    cp_async_16(dst + page_swizzle<F, D>(c / P::kChunks, c % P::kChunks), src + 16 * c, n);
  }
  if constexpr (P::kScales > 0) {
    if (lane < P::kScales / 16)
      cp_async_16(dst + P::kCodes + 16 * lane, src + P::kCodes + 16 * lane, n);
  }
}

// This lane's ldmatrix row address within a staged page: tile i of an x4 load
// (lanes 8i .. 8i+7) covers tokens 8 (i & 1) .. + 7 and chunk c0 + (i >> 1); the
// address for the pair of chunks c0, c0 + 1 (c0 even) is `offset ^ (c0 << 4)`.
template <int F, int D>
__device__ __forceinline__ uint32_t ldsm_offset(int lane) {
  return page_swizzle<F, D>((lane & 7) + ((lane >> 3) & 1) * 8, lane >> 4);
}

// Four E4M3 codes of a word as two f16x2 (codes 0, 1 and 2, 3).
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ void f16x4_to_f32(const uint32_t (&h)[2], float (&s)[4]) {
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h[0]));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h[1]));
  s[0] = x.x;
  s[1] = x.y;
  s[2] = y.x;
  s[3] = y.y;
}

__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
  return half2_bits(__hmul2(*reinterpret_cast<const __half2*>(&a),
                            *reinterpret_cast<const __half2*>(&b)));
}

constexpr uint32_t kNibLo = 0x000f000fu, kNibHi = 0x00f000f0u;

// Query rows in shared memory, as B operands of the score tiles.
//   frag  [n-tile][16-dim k step][lane] two registers: row 8 n-tile + lane/4, the
//         dims that the K format puts into lane%4's A registers
//   off   [n-tile][lane] INT4: two registers of a k step over the groups that takes the
//         codes' offset back, with the token's scales as the A operand: row n's
//         x_g = -8 * 2^-24 * (sum of group g's operands) as f16 high part (k = g) and
//         2^11 times the f16 residual (k = g + 8; A is 2^-11 times the scale there)
//   rs    [row] positive factor from a score accumulator to the log2-domain score (the
//         sign of the softmax scale goes into the operands)
// bf16 pages take Q as it is.  FP8 and INT4 pages take it in f16: each row is
// scaled by a power of two so that its largest magnitude lies in [2^13, 2^14),
// which keeps every value within 2^-24 of the row's largest exact (the odd dims of
// INT4 pages, divided by 16, within 2^-20).
template <int F, int D, int ROWS>
struct QTile {
  static constexpr int kFragBytes = (ROWS / 8) * (D / 16) * 32 * 8;
  static constexpr int kOffOff = kFragBytes;
  static constexpr int kOffBytes = F == kPageInt4 ? ROWS / 8 * 32 * 8 : 0;
  static constexpr int kRsOff = kOffOff + kOffBytes;
  static constexpr int kBytes = kRsOff + ROWS * 4;
};

// Position, in halves, of head dim d of row n within the frag array.
template <int F, int D>
__device__ __forceinline__ int q_frag_pos(int n, int d) {
  int step, lane4, e;                        // k step, lane % 4, element 0..3 of the two registers
  if constexpr (F == kPageBf16) {
    step = d >> 4;
    const int x = d & 15;
    lane4 = (x & 7) >> 1;
    e = (x & 1) + 2 * (x >> 3);
  } else if constexpr (F == kPageFp8) {
    step = d >> 4;
    lane4 = (d & 15) >> 2;
    e = d & 3;
  } else {
    // word lane4 of the group's 16-byte chunk: nibble i; even nibbles in the first
    // of the group's two k steps, odd ones in the second; a register pairs nibbles
    // i and i + 4
    const int i = d & 7;
    step = 2 * (d >> 5) + (i & 1);
    lane4 = (d & 31) >> 3;
    e = (i & 2) + (i >> 2);
  }
  return ((((n >> 3) * (D / 16) + step) * 32) + (n & 7) * 4 + lane4) * 4 + e;
}

// Query rows row0 .. row0 + ROWS - 1 of (sequence b, kv head g) as operands; row n = t * G +
// hl, rows past nrows are zero.  Warp `part` of `parts` writes every parts-th run of RC
// rows (all its loads in flight at once); a barrier among the warps follows.
template <int F, int D, int ROWS, int RC>
__device__ __forceinline__ void load_q_tile(uint8_t* qt, const void* q, int b, int g, int T, int G,
                                            int Hq, int row0, int nrows, float scale_log2,
                                            float k_scale, int lane, int part, int parts) {
  using Q = QTile<F, D, ROWS>;
  constexpr int DL = D / 32;                 // consecutive dims per lane
  static_assert(ROWS % RC == 0, "whole runs");
  uint16_t* frag = reinterpret_cast<uint16_t*>(qt);
  uint16_t* off = reinterpret_cast<uint16_t*>(qt + Q::kOffOff);
  float* rs = reinterpret_cast<float*>(qt + Q::kRsOff);
  const float sign = scale_log2 * k_scale < 0.f ? -1.f : 1.f;
  const float size = fabsf(scale_log2 * k_scale);
  const int d0 = lane * DL;
  for (int n0 = RC * part; n0 < ROWS; n0 += RC * parts) {
    uint32_t raw[RC][DL / 2];
#pragma unroll
    for (int r = 0; r < RC; ++r) {
      const int n = row0 + n0 + r;
#pragma unroll
      for (int k = 0; k < DL / 2; ++k) raw[r][k] = 0u;
      if (n < nrows) {
        const size_t row = (static_cast<size_t>(b) * T + n / G) * Hq + g * G + n % G;
        const uint32_t* src =
            reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(q) + row * D + d0);
        if constexpr (DL == 4) {
          const uint2 v = *reinterpret_cast<const uint2*>(src);
          raw[r][0] = v.x;
          raw[r][1] = v.y;
        } else {
          raw[r][0] = *src;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < RC; ++r) {
      const int n = n0 + r;
      float x[DL];
#pragma unroll
      for (int k = 0; k < DL; ++k)
        x[k] = sign * ((k & 1) ? bf16_hi(raw[r][k / 2]) : bf16_lo(raw[r][k / 2]));
      if constexpr (F == kPageBf16) {
#pragma unroll
        for (int k = 0; k < DL; ++k)
          frag[q_frag_pos<F, D>(n, d0 + k)] = __bfloat16_as_ushort(__float2bfloat16_rn(x[k]));
        if (lane == 0) rs[n] = fmaxf(size, 1e-36f);
      } else {
        float mx = 0.f;
#pragma unroll
        for (int k = 0; k < DL; ++k) mx = fmaxf(mx, fabsf(x[k]));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        // exponent of the row's largest magnitude, kept where 2^(13 - e) and its inverse are
        // normal
        int e = static_cast<int>((__float_as_uint(mx) >> 23) & 0xffu) - 127;
        e = max(-100, min(e, 100));
        const float up = __uint_as_float(static_cast<uint32_t>(13 - e + 127) << 23);
        const float down = __uint_as_float(static_cast<uint32_t>(e - 13 + 127) << 23);
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < DL; ++k) {
          float y = x[k] * up;
          if (F == kPageInt4 && (k & 1)) y *= 0.0625f;
          const __half h = __float2half_rn(y);
          frag[q_frag_pos<F, D>(n, d0 + k)] = __half_as_ushort(h);
          sum += __half2float(h) * ((k & 1) ? 16.f : 1.f);
        }
        if constexpr (F == kPageInt4) {
          constexpr int GL = kGroupDims / DL;    // lanes of a group
#pragma unroll
          for (int o = GL / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          const float v = sum * (-8.f / 16777216.f);
          const __half vh = __float2half_rn(v);
          const __half vl = __float2half_rn((v - __half2float(vh)) * 2048.f);
          uint16_t* to = off + (n >> 3) * 128 + (n & 7) * 16;   // [lane % 4][4 halves]
          if (lane % GL == 0) {
            const int g2 = lane / GL;
            to[(g2 >> 1) * 4 + (g2 & 1)] = __half_as_ushort(vh);
            to[(g2 >> 1) * 4 + (g2 & 1) + 2] = __half_as_ushort(vl);
          } else if (lane % GL == 1 && lane / GL < 4) {
            // the k steps' other lanes: zero
            constexpr int kUsed = D / kGroupDims / 2;
            if (lane / GL >= kUsed)
              *reinterpret_cast<uint2*>(to + (lane / GL) * 4) = make_uint2(0u, 0u);
          }
          if constexpr (D / kGroupDims == 2) {
            if (lane == 2 || lane == 3) *reinterpret_cast<uint2*>(to + lane * 4) = make_uint2(0u, 0u);
          }
        }
        if (lane == 0)
          rs[n] = fmaxf(size * down * (F == kPageInt4 ? 16777216.f : 1.f), 1e-36f);
      }
    }
  }
}

// The query operands one warp needs for its n-tiles, in registers or (kRegs = false)
// read from shared memory at every page.
template <int F, int D, int NT, bool kRegs>
struct QOperand {
  uint2 f[kRegs ? NT : 1][kRegs ? D / 16 : 1];
  uint2 o[kRegs ? NT : 1];
  float rs0[NT], rs1[NT];
  const uint2* base;
  const uint2* obase;

  template <int ROWS>
  __device__ __forceinline__ void load(const uint8_t* qt, int tile0, int lane) {
    using Q = QTile<F, D, ROWS>;
    base = reinterpret_cast<const uint2*>(qt) + static_cast<size_t>(tile0) * (D / 16) * 32 + lane;
    obase = reinterpret_cast<const uint2*>(qt + Q::kOffOff) + tile0 * 32 + lane;
    const float* rs = reinterpret_cast<const float*>(qt + Q::kRsOff);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int r0 = 8 * (tile0 + j) + 2 * (lane & 3);
      rs0[j] = rs[r0];
      rs1[j] = rs[r0 + 1];
      if constexpr (kRegs && F == kPageInt4) o[j] = obase[j * 32];
      if constexpr (kRegs) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) f[j][k] = base[(j * (D / 16) + k) * 32];
      }
    }
  }
  __device__ __forceinline__ uint2 get(int j, int k) const {
    if constexpr (kRegs)
      return f[j][k];
    else
      return base[(j * (D / 16) + k) * 32];
  }
  __device__ __forceinline__ uint2 offset(int j) const {
    if constexpr (kRegs)
      return o[j];
    else
      return obase[j * 32];
  }
};

// D = A * B + C and D += A * B on f16 operands; without side effects, so that the compiler
// may move them.
__device__ __forceinline__ void mma_f16_c(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1, float c0,
                                          float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Scores of a staged K page, to be multiplied by the rows' rs: lane (gid = lane/4, q = lane%4) gets
// t[j] = S^T[gid][2q], [gid][2q+1], [gid+8][2q], [gid+8][2q+1] of n-tile j.
template <int F, int D, int NT, bool kRegs>
__device__ __forceinline__ void page_scores(float (&t)[NT][4], uint32_t page, uint32_t koff,
                                            const QOperand<F, D, NT, kRegs>& q, int lane) {
  if constexpr (F == kPageInt4) {
    using P = Page<F, D>;
    // scales of tokens gid and gid + 8, and the codes' offset taken back:
    // t = sum_g scale_g x_g
    float s0[4], s1[4];
    {
      const uint32_t a = page + P::kCodes + (lane >> 2) * P::kGroups;
      uint32_t w0, w1, h0[2], h1[2];
      if constexpr (P::kGroups == 4) {
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w0) : "r"(a));
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w1) : "r"(a + 8 * P::kGroups));
      } else {
        asm volatile("ld.shared.u16 %0, [%1];" : "=r"(w0) : "r"(a));
        asm volatile("ld.shared.u16 %0, [%1];" : "=r"(w1) : "r"(a + 8 * P::kGroups));
      }
      e4m3x4_to_f16x4(w0, h0[0], h0[1]);
      e4m3x4_to_f16x4(w1, h1[0], h1[1]);
      const bool odd = P::kGroups == 4 && (lane & 1);
      const uint32_t a0 = odd ? h0[1] : h0[0], a1 = odd ? h1[1] : h1[0];
      const uint32_t a2 = f16x2_mul(a0, 0x10001000u), a3 = f16x2_mul(a1, 0x10001000u);   // 2^-11
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const uint2 b = q.offset(j);
        mma_f16_c(t[j], a0, a1, a2, a3, b.x, b.y, 0.f, 0.f, 0.f, 0.f);
      }
      f16x4_to_f32(h0, s0);
      f16x4_to_f32(h1, s1);
    }
#pragma unroll
    for (int g2 = 0; g2 < P::kGroups; g2 += 2) {
      uint32_t w[4];
      ldsm_x4(w[0], w[1], w[2], w[3], page + (koff ^ (g2 << 4)));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int g = g2 + h;
        const uint32_t x0 = w[2 * h], x1 = w[2 * h + 1];
        const uint32_t y0 = x0 >> 8, y1 = x1 >> 8;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float d[4];
          const uint2 b0 = q.get(j, 2 * g), b1 = q.get(j, 2 * g + 1);
          mma_f16_c(d, x0 & kNibLo, x1 & kNibLo, y0 & kNibLo, y1 & kNibLo, b0.x, b0.y, 0.f, 0.f,
                    0.f, 0.f);
          mma_f16(d, x0 & kNibHi, x1 & kNibHi, y0 & kNibHi, y1 & kNibHi, b1.x, b1.y);
          t[j][0] = fmaf(d[0], s0[g], t[j][0]);
          t[j][1] = fmaf(d[1], s0[g], t[j][1]);
          t[j][2] = fmaf(d[2], s1[g], t[j][2]);
          t[j][3] = fmaf(d[3], s1[g], t[j][3]);
        }
      }
    }
  } else {
    // two accumulator chains per n-tile
    float u[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) t[j][e] = u[j][e] = 0.f;
    if constexpr (F == kPageBf16) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t a0, a1, a2, a3;
        ldsm_x4(a0, a1, a2, a3, page + (koff ^ ((2 * k) << 4)));
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint2 b = q.get(j, k);
          mma_bf16(k & 1 ? u[j] : t[j], a0, a1, a2, a3, b.x, b.y);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < D / 16; k += 2) {
        uint32_t w[4];
        ldsm_x4(w[0], w[1], w[2], w[3], page + (koff ^ (k << 4)));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a0 = e4m3x2_to_f16x2(w[2 * h]), a2 = e4m3x2_to_f16x2(w[2 * h] >> 16);
          const uint32_t a1 = e4m3x2_to_f16x2(w[2 * h + 1]);
          const uint32_t a3 = e4m3x2_to_f16x2(w[2 * h + 1] >> 16);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint2 b = q.get(j, k + h);
            mma_f16(h ? u[j] : t[j], a0, a1, a2, a3, b.x, b.y);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) t[j][e] += u[j][e];
  }
}

// ---------------------------------------------------------------- INT4 quantisation
// Four lanes hold the 32 dims of a group, eight each (bf16 pairs in w).  Returns the
// lane's eight codes (dim i in bits 4i .. 4i+3) and the group's scale byte:
//   scale = e4m3(max|x| / (7 head_scale))      (IEEE float32 division; saturates at 448)
//   code  = the integer nearest to x / (scale head_scale), ties to even, in -7 .. 7, + 8
// A zero scale gives the codes of zero; a NaN in the group gives a NaN scale.
__device__ __forceinline__ uint32_t quantize_int4_8(const uint4& v, float head_scale,
                                                    uint32_t& scale_byte) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t mb = 0;                            // largest magnitude as bf16 bits (NaN on top)
#pragma unroll
  for (int i = 0; i < 4; ++i) mb = max(mb, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
  mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
  mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
  const float amax = __uint_as_float(mb << 16);
  scale_byte = f32x2_to_e4m3x2(__fdiv_rn(amax, __fmul_rn(7.f, head_scale)), 0.f) & 0xffu;
  const uint32_t sh = e4m3x2_to_f16x2(scale_byte);
  const float step = __half2float(__ushort_as_half(static_cast<unsigned short>(sh & 0xffffu))) *
                     head_scale;
  const float inv = step > 0.f ? __fdividef(1.f, step) : 0.f;
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
    // f + 1/2 is a midpoint next to x / step (x * inv may err by a few ulp, not by half
    // a step); the sign of x - (f + 1/2) step decides, its zero is a tie
    const float y = fminf(fmaxf(x * inv, -8.f), 8.f);
    const float f = floorf(y);
    const float r = fmaf(-(f + 0.5f), step, x);
    int c = static_cast<int>(f);
    c += (r > 0.f || (r == 0.f && (c & 1))) ? 1 : 0;
    c = step > 0.f ? max(-7, min(7, c)) : 0;
    codes |= static_cast<uint32_t>(c + 8) << (4 * i);
  }
  return codes;
}

// Read and clear this translation unit's error word.
static inline cudaError_t read_error_word(unsigned* bits) {
  unsigned v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_pa_err, sizeof(v));
  if (e != cudaSuccess) return e;
  if (v) e = cudaMemcpyToSymbol(g_pa_err, &zero, sizeof(zero));
  *bits |= v;
  return e;
}

}  // namespace pa
