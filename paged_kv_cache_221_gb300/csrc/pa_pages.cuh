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
// and odd dims of Q, the output).  The offset 8: for K it leaves the contraction as 8 * (sum
// over the group of scale * the query's operand), one more small tile; the V codes take one f16
// addition more, also exact, so that a rounding of a softmax weight counts with the value
// itself.  E2M1 codes would need a conversion for every pair of values, and have a
// larger error on normally distributed values.
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>

#include <atomic>

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

// Chunk `lane + 32 c` of a page lies at (lane's offset ^ swizzle_step(c)) + 512 c.
template <int F, int D>
__device__ __forceinline__ constexpr uint32_t swizzle_step(int c) {
  constexpr int kRows = 32 / Page<F, D>::kChunks;   // rows per 32 chunks
  return Page<F, D>::kChunks >= 8 ? ((kRows * c) & 7) << 4 : 0;
}

// base + page * stride in one wide multiply-add.
__device__ __forceinline__ const uint8_t* at_page(const uint8_t* base, uint32_t page,
                                                  uint32_t stride) {
  const uint8_t* r;
  asm("mad.wide.u32 %0, %1, %2, %3;" : "=l"(r) : "r"(page), "r"(stride), "l"(base));
  return r;
}

// L2 policy of a read: the first to leave the cache, or the default.
__device__ __forceinline__ uint64_t read_policy(bool once) {
  uint64_t policy;
  if (once)
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  else
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}

__device__ __forceinline__ void cp_async_16_hint(uint32_t dst, const void* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "l"(policy)
               : "memory");
}

__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

// 1 in each byte of w that is an E4M3 NaN (0x7F, 0xFF).
__device__ __forceinline__ uint32_t e4m3_nan_bytes(uint32_t w) {
  return (((w & 0x7f7f7f7fu) + 0x01010101u) >> 7) & 0x01010101u;
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

__device__ __forceinline__ uint32_t f16x2_add(uint32_t a, uint32_t b) {
  return half2_bits(__hadd2(*reinterpret_cast<const __half2*>(&a),
                            *reinterpret_cast<const __half2*>(&b)));
}

// Nibbles 0 (and 1) of both halves of a word of codes, and -8 on the same scales.
constexpr uint32_t kNibLo = 0x000f000fu, kNibHi = 0x00f000f0u;
constexpr uint32_t kMinus8Lo = 0x80088008u, kMinus8Hi = 0x80808080u;

// Query rows as B operands of the score tiles.  Lane (gid = lane/4, q = lane%4) of a warp
// holds, for row gid of an n-tile of 8 rows, the head dims that the K format puts
// into lane q's A registers, so a warp loads a tile straight into operand order:
//   bf16  16-dim k step k: dims 16k + 2q, +1 and 16k + 2q + 8, +9
//   FP8   16-dim k step k: dims 16k + 4q .. + 3
//   INT4  group g: dims 32g + 8q .. + 7 (nibbles 0 .. 7 of the lane's word): the even
//         nibbles in k step 2g, the odd ones in 2g + 1; a register pairs nibbles i, i + 4
// bf16 pages take Q as it is.  FP8 and INT4 pages take it in f16: each row is
// scaled by a power of two so that its largest magnitude lies in [2^13, 2^14),
// which keeps every value within 2^-24 of the row's largest exact (the odd dims of
// INT4 pages, divided by 16, within 2^-20).
//   rs0, rs1  positive factors from the score accumulators of rows 2q, 2q + 1 to log2-domain
//             scores (the sign of the softmax scale goes into the operands)
//   off       INT4: operand of a k step over the groups that takes the codes' offset back,
//             with the token's scales as the A operand: x_g = -8 * 2^-24 * (sum of group g's
//             operands) as f16 high part (k = g) and 2^11 times the f16 residual (k = g +
//             8; A is 2^-11 times the scale there)
template <int F, int D>
struct QTileRaw {
  uint32_t w[D / 8];                         // the lane's D / 4 values
};

template <int F, int D>
struct QTile {
  uint2 f[D / 16];
  uint2 off;
  float rs0, rs1;
};

// Bytes of one n-tile's operands in shared memory: [k step][lane], then off.
template <int F, int D>
struct QTileSmem {
  static constexpr int kOff = (D / 16) * 32 * 8;
  static constexpr int kBytes = kOff + (F == kPageInt4 ? 32 * 8 : 0);
};

// Row n = t * G + hl of (sequence b, kv head g); rows from nrows on are zero.
template <int F, int D>
__device__ __forceinline__ void load_q_raw(QTileRaw<F, D>& raw, const void* q, int b, int g, int T,
                                           int G, int Hq, int row0, int nrows, int lane) {
  const int n = row0 + (lane >> 2), q4 = lane & 3;
  const bool live = n < nrows;
  const size_t row = (static_cast<size_t>(b) * T + (live ? n / G : 0)) * Hq + g * G +
                     (live ? n % G : 0);
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(q) + row * D;
#pragma unroll
  for (int k = 0; k < D / 8; ++k) raw.w[k] = 0u;
  if (!live) return;
  if constexpr (F == kPageBf16) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      raw.w[2 * k] = *reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * q4);
      raw.w[2 * k + 1] = *reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * q4 + 8);
    }
  } else if constexpr (F == kPageFp8) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint2 v = *reinterpret_cast<const uint2*>(src + 16 * k + 4 * q4);
      raw.w[2 * k] = v.x;
      raw.w[2 * k + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
      const uint4 v = *reinterpret_cast<const uint4*>(src + 32 * k + 8 * q4);
      raw.w[4 * k] = v.x;
      raw.w[4 * k + 1] = v.y;
      raw.w[4 * k + 2] = v.z;
      raw.w[4 * k + 3] = v.w;
    }
  }
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  return half2_bits(__floats2half2_rn(lo, hi));
}

template <int F, int D>
__device__ __forceinline__ void make_q_tile(QTile<F, D>& t, const QTileRaw<F, D>& raw,
                                            float scale_log2, float k_scale, int lane) {
  const float sign = scale_log2 * k_scale < 0.f ? -1.f : 1.f;
  float rs = fabsf(scale_log2 * k_scale);
  t.off = make_uint2(0u, 0u);
  if constexpr (F == kPageBf16) {
    const uint32_t flip = sign < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
      t.f[k] = make_uint2(raw.w[2 * k] ^ flip, raw.w[2 * k + 1] ^ flip);
  } else {
    uint32_t mb = 0;                         // largest magnitude of the row, as bf16 bits
#pragma unroll
    for (int k = 0; k < D / 8; ++k)
      mb = max(mb, max(raw.w[k] & 0x7fffu, (raw.w[k] >> 16) & 0x7fffu));
    mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
    mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
    // its exponent, kept where 2^(13 - e) and its inverse are normal
    int e = static_cast<int>(mb >> 7) - 127;
    e = max(-100, min(e, 127));
    const float up = sign * __uint_as_float(static_cast<uint32_t>(13 - e + 127) << 23);
    rs *= __uint_as_float(static_cast<uint32_t>(e - 13 + 127) << 23);
    if constexpr (F == kPageFp8) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        t.f[k] = make_uint2(pack_f16(bf16_lo(raw.w[2 * k]) * up, bf16_hi(raw.w[2 * k]) * up),
                            pack_f16(bf16_lo(raw.w[2 * k + 1]) * up, bf16_hi(raw.w[2 * k + 1]) * up));
    } else {
      constexpr int NG = D / kGroupDims;
      const float odd = up * 0.0625f;
      float sum[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t* w = raw.w + 4 * g;   // nibbles 0,1 | 2,3 | 4,5 | 6,7
        t.f[2 * g] = make_uint2(pack_f16(bf16_lo(w[0]) * up, bf16_lo(w[2]) * up),
                                pack_f16(bf16_lo(w[1]) * up, bf16_lo(w[3]) * up));
        t.f[2 * g + 1] = make_uint2(pack_f16(bf16_hi(w[0]) * odd, bf16_hi(w[2]) * odd),
                                    pack_f16(bf16_hi(w[1]) * odd, bf16_hi(w[3]) * odd));
        const uint32_t u[4] = {t.f[2 * g].x, t.f[2 * g].y, t.f[2 * g + 1].x, t.f[2 * g + 1].y};
        float part[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
          part[i] = x.x + x.y;
        }
        sum[g] = (part[0] + part[1]) + 16.f * (part[2] + part[3]);
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
        sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
      }
      const int q4 = lane & 3;
      float a = sum[0], c = sum[1];
      if constexpr (NG == 4) {
        a = q4 == 1 ? sum[2] : a;
        c = q4 == 1 ? sum[3] : c;
      }
      if (q4 < NG / 2) {
        a *= -8.f / 16777216.f;
        c *= -8.f / 16777216.f;
        const float ah = __half2float(__float2half_rn(a)), ch = __half2float(__float2half_rn(c));
        t.off = make_uint2(pack_f16(ah, ch), pack_f16((a - ah) * 2048.f, (c - ch) * 2048.f));
      }
      rs *= 16777216.f;
    }
  }
  rs = fmaxf(rs, 1e-36f);
  t.rs0 = __shfl_sync(0xffffffffu, rs, (lane & 3) * 8);        // from lanes of rows 2q, 2q + 1
  t.rs1 = __shfl_sync(0xffffffffu, rs, (lane & 3) * 8 + 4);
}

template <int F, int D>
__device__ __forceinline__ void put_q_tile(uint8_t* to, const QTile<F, D>& t, int lane) {
  using S = QTileSmem<F, D>;
#pragma unroll
  for (int k = 0; k < D / 16; ++k) reinterpret_cast<uint2*>(to)[k * 32 + lane] = t.f[k];
  if constexpr (F == kPageInt4) reinterpret_cast<uint2*>(to + S::kOff)[lane] = t.off;
}

// The query operands one warp needs for its n-tiles, in registers or (kRegs = false)
// read from shared memory (consecutive QTileSmem tiles) at every page.
template <int F, int D, int NT, bool kRegs>
struct QOperand {
  QTile<F, D> tile[kRegs ? NT : 1];
  float rs0[NT], rs1[NT];
  const uint8_t* base;

  __device__ __forceinline__ uint2 get(int j, int k) const {
    if constexpr (kRegs)
      return tile[j].f[k];
    else
      return *reinterpret_cast<const uint2*>(base + j * QTileSmem<F, D>::kBytes + k * 256);
  }
  __device__ __forceinline__ uint2 offset(int j) const {
    if constexpr (kRegs)
      return tile[j].off;
    else
      return *reinterpret_cast<const uint2*>(base + j * QTileSmem<F, D>::kBytes +
                                             QTileSmem<F, D>::kOff);
  }
};

// A warp's operands for NT n-tiles; those kept in shared memory are read back by the lane that
// wrote them.
template <int F, int D, int NT, bool kRegs>
__device__ __forceinline__ void make_q_operand(QOperand<F, D, NT, kRegs>& qo,
                                               const QTileRaw<F, D> (&raw)[NT], uint8_t* qt,
                                               float scale_log2, float k_scale, int lane) {
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    if constexpr (kRegs) {
      make_q_tile(qo.tile[j], raw[j], scale_log2, k_scale, lane);
      qo.rs0[j] = qo.tile[j].rs0;
      qo.rs1[j] = qo.tile[j].rs1;
    } else {
      QTile<F, D> tile;
      make_q_tile(tile, raw[j], scale_log2, k_scale, lane);
      put_q_tile(qt + j * QTileSmem<F, D>::kBytes, tile, lane);
      qo.rs0[j] = tile.rs0;
      qo.rs1[j] = tile.rs1;
    }
  }
  if constexpr (!kRegs) qo.base = qt + lane * 8;
}

// ---------------------------------------------------------------- pairs of fp32 values
// One instruction for two values, each rounded to nearest.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// (y0, y1) = (a0 b0 + c0, a1 b1 + c1)
__device__ __forceinline__ void fma_f32x2(float& y0, float& y1, float a0, float a1, float b0,
                                          float b1, float c0, float c1) {
  const uint64_t y = fma_f32x2(pack_f32x2(a0, a1), pack_f32x2(b0, b1), pack_f32x2(c0, c1));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(y0), "=f"(y1) : "l"(y));
}

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
      // the first k steps of both groups, then the second ones: no tile waits for its own
      float d[2][NT][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t x0 = w[2 * h], x1 = w[2 * h + 1], y0 = x0 >> 8, y1 = x1 >> 8;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint2 b0 = q.get(j, 2 * (g2 + h));
          mma_f16_c(d[h][j], x0 & kNibLo, x1 & kNibLo, y0 & kNibLo, y1 & kNibLo, b0.x, b0.y, 0.f,
                    0.f, 0.f, 0.f);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t x0 = w[2 * h], x1 = w[2 * h + 1], y0 = x0 >> 8, y1 = x1 >> 8;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint2 b1 = q.get(j, 2 * (g2 + h) + 1);
          mma_f16(d[h][j], x0 & kNibHi, x1 & kNibHi, y0 & kNibHi, y1 & kNibHi, b1.x, b1.y);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const float a = s0[g2 + h], c = s1[g2 + h];
          fma_f32x2(t[j][0], t[j][1], d[h][j][0], d[h][j][1], a, a, t[j][0], t[j][1]);
          fma_f32x2(t[j][2], t[j][3], d[h][j][2], d[h][j][3], c, c, t[j][2], t[j][3]);
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
// A thread's group of 32 dims (bf16 pairs in w): its codes (dim i in bits 4 (i % 8) of word
// i / 8) and scale byte:
//   scale = e4m3(max|x| / (7 head_scale))      (IEEE float32 division; saturates at 448)
//   code  = the integer nearest to x / (scale head_scale), ties to even, in -7 .. 7, + 8
// A zero scale gives the codes of zero; a NaN in the group gives a NaN scale.
// The quotient is x * (1 / step) with one correction by its residual, which makes
// ties come out exact; it is rounded by adding 1.5 * 2^23 + 8 (to nearest even), whose
// low bits then are the code, and the codes of a word are strung together by multiply-adds
// on the whole bit patterns, whose constant parts are taken off at the end.  Two values share
// each of these four steps.  Only a scale that saturated or is subnormal lets a quotient
// reach 7.5: rounding to nearest takes at most 1/17 off a normal one, so that it is at most
// 7 * 17 / 16 < 7.46875.
__device__ __forceinline__ void quantize_int4_32(const uint32_t (&w)[16], float head_scale,
                                                 uint32_t (&codes)[4], uint32_t& scale_byte) {
  uint32_t mb = 0;                            // largest magnitudes as bf16 bits (NaN on top)
#pragma unroll
  for (int i = 0; i < 16; ++i) mb = __vmaxu2(mb, w[i] & 0x7fff7fffu);
  mb = max(mb & 0xffffu, mb >> 16);
  const float amax = __uint_as_float(mb << 16);
  scale_byte = f32x2_to_e4m3x2(__fdiv_rn(amax, __fmul_rn(7.f, head_scale)), 0.f) & 0xffu;
  const uint32_t sh = e4m3x2_to_f16x2(scale_byte);
  const float step = __half2float(__ushort_as_half(static_cast<unsigned short>(sh & 0xffffu))) *
                     head_scale;
  const bool good = step > 0.f;               // not zero, not NaN
  const float inv = good ? __frcp_rn(step) : 0.f;
  const float lim = 7.46875f * step;          // beyond it the code is +-7
  constexpr float kMagic = 12582912.f + 8.f;
  constexpr uint32_t kBase = 0x4B400000u;     // bits of 12582912.f
  constexpr uint32_t kBases = kBase * 0x11111111u;
  const bool clamp = !(amax <= lim);
  const uint64_t inv2 = pack_f32x2(inv, inv), minus2 = pack_f32x2(-step, -step);
  const uint64_t magic2 = pack_f32x2(kMagic, kMagic);
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    uint32_t c = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      float lo = bf16_lo(w[4 * v + i]), hi = bf16_hi(w[4 * v + i]);
      if (clamp) {
        lo = fminf(fmaxf(lo, -lim), lim);
        hi = fminf(fmaxf(hi, -lim), lim);
      }
      const uint64_t x = pack_f32x2(lo, hi);
      const uint64_t y = mul_f32x2(x, inv2);
      const uint64_t q = add_f32x2(fma_f32x2(fma_f32x2(y, minus2, x), inv2, y), magic2);
      c = (c * 16u + static_cast<uint32_t>(q >> 32)) * 16u + static_cast<uint32_t>(q);
    }
    codes[v] = good ? c - kBases : 0x88888888u;
  }
}

// Launch a kernel that, with `behind`, may become resident while the one before it in the
// stream drains (programmatic stream serialisation): the later launches of a call.  It calls grid_dependency_wait() before it reads
// what earlier work wrote and before it writes; every CTA waits, so that it does not
// complete before the kernel it follows.
template <class... Params, class... Args>
cudaError_t launch_behind(void (*fn)(Params...), dim3 grid, int threads, size_t smem,
                          cudaStream_t s, bool behind, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = behind ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

// Let a kernel use `bytes` of dynamic shared memory: asked of the driver once per device.
template <auto kKernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<unsigned long long> done{0ull};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
  if (bit != 0 && (done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
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
