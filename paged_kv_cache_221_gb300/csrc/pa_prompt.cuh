// Causal attention of whole prompts over the paged cache, on the fifth-generation
// tensor cores.
//
// Query tokens of all sequences are packed; those of sequence b are the newest
// positions of its context.  With x_j = scale * q . k_j over the visible keys j,
//   out = sum_j 2^((x_j - m) log2 e) v_j / sum_j 2^((x_j - m) log2 e),
// m a running reference that follows the row's maximum.
//
// Tiles.  The query rows of one kv head are (token, query head of the group) pairs; 128
// of them (sub_tokens tokens x G heads) are the M dimension of both products:
//   S[128 rows x 128 keys] = Q . K^T        Q, K in shared memory        (tensor memory)
//   O[128 rows x D]       += P . V          P in tensor memory, over S   (tensor memory)
// A unit of work is a pair of such tiles (consecutive tokens) of one kv head, or one
// partition of its keys, so that each K/V tile that a CTA loads serves 256 rows and one
// tile's products run while the other tile's weights are computed.
//
// Roles of a CTA (one per SM, which goes on to further units):
//   warps 0-3, 4-7  softmax of the first, the second tile: thread = row.  A tile's weights are
//                   taken with the reference of the last ones at once; only where they pass
//                   2^15 and at a unit's start is the row's maximum looked for, which then
//                   becomes the reference if it is far above it.  O is then rescaled in tensor
//                   memory, which no product is using at that time: S of the next keys is
//                   issued behind P . V of the last ones.
//   warp 8          finds the units, loads Q and the K tiles by TMA, 16 keys per page box,
//                   through the block table.
//   warp 9          issues the MMAs: per K/V tile P.V (in two halves, the first while the last
//                   quarter of the weights is computed) then the next S of the first tile, the
//                   same of the second.
//   warps 10 to 15  bring the V tiles, a 16-key page at a time, as f16.
//
// Rounding.  The weights meet V as f16, times 2^7: 2^-11 of each at most, and 2^-32 of the row's
// largest (which is what f16 cannot hold then); statistics and accumulators are fp32.  As one bf16
// each they would add 1.1e-3 to 1.7e-3 of relative error to the outputs' own rounding, and both
// together pass the 2e-3 that the other attention kernels keep.
//
// V of bf16 pages.  The product takes two operands of one type, so the pages come through
// registers and become f16 there, times 2^8.  That is exact or not done: a page with an element
// that f16 does not have (2^8 and more, below 2^-25) stays bf16, and so do its weights, each in
// two parts that hold the f16, with a product for both; 16 keys are one step of the product, so
// that pages of both kinds stand in one tile.  The byte v_split tells the others which.  O carries
// 2^15 in all, weights up to 2^8 above the reference and 2^30 keys at most: values up to 2^74
// never overflow it.  Infinities and NaN stay in a page that every row sees; from others they are
// taken out, since 0 * inf would reach rows that must not see them, and added at the end to the
// rows that do.
//
// FP8 pages.  Every E4M3 value is an f16: warps 10 to 15 widen
// each tile from where TMA left it into the ring that the MMAs read (K rows as they are; V
// pages are stored by head dim, so that tile becomes a K-major operand), and the query rows in
// place, each times a power of two that puts its largest element at 2^7 .. 2^8 (a bf16 value
// may lie outside f16's range) and that the row's scores take back.  NaN are taken out of V at the
// mask's border.
//
// What bounds it.  A K/V tile of a pair is 2048 cycles of products.  A tile's weights take 1350
// alone (an exponential is 4 cycles per warp instruction and scheduler; the rest beside it), its
// P . V and next S with their hand-overs as much again, and the two tiles of a pair alternate: 2700
// at least.  The warps that bring V issue 45 instructions for 512 bytes of it from the same four
// schedulers: about 3150 in all (3500 for FP8 pages, whose K and V take two thirds of that to
// widen).  A unit's start and end are 10000 more: outputs written, 3500, and the first maximum,
// while no product runs.  32 query heads over 8 of 128 dims: 16384 tokens 1680 to 1740 us (1.31 to
// 1.26 PFLOP/s; a library matrix product in a loop 1.69), 24 prompts of 128 to 2048 tokens 367 us
// (0.81), 12 of 512 to 4096 over FP8 pages 572 us (1.13), 33 tokens behind 65519 70 us (3.8 TB/s).
//
// By values, 24 prompts: normal ones, or with half of the dims zero, 360 us; times 0.02 379, times
// 1e-3 (a third of the tiles have a page with an element below 2^-25) 520; all pages split 670.
//
// Measured on the way, 16384 tokens or as said.  The weights of bf16 pages in 8 bits, V as it is:
// 1470 us (24 prompts 305), the precision above.  In two bf16 parts for all pages: 2118 (448).  V
// made f16 where asynchronous copies left it: 1820 to 2010 (354 to 420), since shared memory is
// read and written once more.  Through registers that spill: 2180 (515).  Bits moved instead of a
// conversion, in a path for pages without zeros: 1700 (361), but 605 for 24 prompts with half of
// the dims zero.  Weights split where they are packed, ten times the code: all pages split 771.
// Without the prefetch to L2 33 tokens behind 65519 76 us against 71.  A sum of 64
// weights as their limit, where sums of eight are now: four windows of 1000 446 us against 419.
// V by TMA boxes like K, 2300 cycles of the TMA unit for a K/V tile by themselves (a box of 16 keys
// is about 70 whatever its bytes); three K and two V stages 1460 against 1417 us; two threads per
// row (16 softmax warps) 1466; the rare code between that of most tiles 1430 against 1397, since
// the roles share one instruction cache (these with V as it is); generic instead of shared-memory
// instructions in widening 653 against 590 (FP8); three pieces of a lane at a time there 766, since
// registers spill; three warps for K and three for V instead of six for each in turn 628 against
// 582.
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>
#include <stddef.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "pa_pages.cuh"
#include "pa_ptx.cuh"
#include "pa_tc.cuh"

namespace pa {

constexpr int kPromptVShift = 8;

template <int D, bool KV8>
struct PromptGeo {
  static constexpr int kSoftmaxWarps = 8;
  static constexpr int kAux = 6;                         // warps that bring V, or widen K and V
  static constexpr int kThreads = (kSoftmaxWarps + 2 + kAux) * 32;
  static constexpr int kHalves = D / 64;                 // 64-dim halves of a row (128 bytes)
  static constexpr int kHalfBytes = kPromptTile * 128;
  static constexpr int kTileBytes = kHalves * kHalfBytes;
  static constexpr int kKStages = 2;                     // K tiles ready or in flight
  static constexpr int kVStages = KV8 ? 2 : 3;
  static constexpr int kRawStages = KV8 ? 2 : 0;         // FP8 tiles in flight
  static constexpr int kRawBytes = kPromptTile * D;
  static constexpr int kShift = 7;                       // weights carry 2^kShift
  static constexpr int kVShift = KV8 ? 0 : kPromptVShift;  // and V, as f16, 2^kVShift
  static constexpr int kPages = kPromptTile / kBlockSize;
  // shared memory, from a 1024-byte aligned base
  static constexpr int kKOff = 2 * kTileBytes;           // behind the two Q tiles
  static constexpr int kVOff = kKOff + kKStages * kTileBytes;
  static constexpr int kRawOff = kVOff + kVStages * kTileBytes;
  static constexpr int kMiscOff = kRawOff + kRawStages * kRawBytes;
  static constexpr int kMiscBytes = KV8 ? 1024 : 512;
  static constexpr int kAlloc = kMiscOff + kMiscBytes + 1024;
  // tensor memory columns
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kO = 2 * kPromptTile;        // S tiles at 0 and 128, then O
  // registers per thread: launch, softmax warps, others
  static constexpr int kRegs = 128, kSoftmaxRegs = 184, kOtherRegs = 72;
  static_assert(kAlloc <= 232448, "shared memory per block");
  static_assert(kSoftmaxWarps * 32 * kSoftmaxRegs + (kThreads - kSoftmaxWarps * 32) * kOtherRegs <=
                    kThreads * kRegs, "the split takes no more than the launch has");
};

// Weights are taken with the present reference while none of them passes what f16 holds (for half
// of them by sums of eight); a reference is one of rounded products up to 2^26.
constexpr float kPromptLimit = 65504.f, kPromptExact = 67108864.f;

// What a sum of weights is multiplied by at least when a far larger one joins it: with 0 an
// infinity in it would become NaN.
constexpr float kPromptFaint = 0x1p-149f;

// A wait's limit in tries.  One that fails takes 4.0 us on GB300 (measured with 1, 32 and 512
// threads that wait, with and without a time hint, which changes nothing), so this is two seconds;
// PTX gives no bound.  The clock instead of the count costs two registers that the roles do not
// have: 24 prompts 409 us against 368.
constexpr int kPromptTries = 1 << 19;

// One unit of work.
struct alignas(16) PromptUnit {
  int b;                 // sequence, -1 behind the last unit
  int head;              // kv head
  int row0, ntok;        // packed query tokens [row0, row0 + ntok)
  int pos0;              // position of the first of them
  int L;                 // context length
  int t0, t1;            // K/V tiles [t0, t1)
  int part, parts;
  int nonfinite;         // infinities or NaN were taken out of V pages at the mask's border
};

template <int D, bool KV8>
struct PromptMisc {
  using Gm = PromptGeo<D, KV8>;
  uint64_t k_full[Gm::kKStages], k_empty[Gm::kKStages];
  uint64_t v_full[Gm::kVStages], v_empty[Gm::kVStages];
  uint64_t raw_full[Gm::kRawStages > 0 ? Gm::kRawStages : 1];
  uint64_t raw_empty[Gm::kRawStages > 0 ? Gm::kRawStages : 1];
  uint64_t q_full[2], q_empty[2];      // by tile of the pair
  uint64_t q_wide[2][2];               // by record and tile: the query rows are f16
  uint64_t s_full[2], p_half[2], p_full[2], o_full[2], o_free[2];   // by tile of the pair
  uint64_t unit_full[2], unit_empty[2], unit_checked[2]; // by record
  uint64_t fin;
  PromptUnit unit[2];
  uint32_t tmem_base;
  alignas(8) uint8_t v_split[Gm::kVStages][Gm::kPages];  // 0, kSplitPage or kOddPage
  int8_t q_exp[KV8 ? 2 : 1][2][KV8 ? kPromptTile : 1];   // by record, tile, row: of the factor
};

// The unit with index u (kv heads fastest, then pairs of tiles, then partitions), found by a
// whole warp.  Sequence b owns the pairs from query_starts[b] / pair + b on, which leaves every
// sequence enough of them without a sum over the others; those it has no use for are empty.
// Its last tokens come first, because they see the most keys.
__device__ __forceinline__ bool prompt_unit(const PromptParams& p, int u, PromptUnit& un,
                                            bool* bad) {
  const int lane = threadIdx.x & 31;
  const int pair = 2 * p.sub_tokens;
  *bad = false;
  un.head = u % p.Hkv;
  const int slot = u / p.Hkv % p.num_slots;
  un.part = u / p.Hkv / p.num_slots;
  int lo = 0, hi = p.num_seqs;
  do {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    bool below = false;
    if (at < hi) {
      const int q = min(max(__ldg(p.query_starts + at), 0), p.num_rows);
      below = q / pair + at <= slot;
    }
    const int n = __popc(__ballot_sync(0xffffffffu, below));
    if (n == 0) return false;
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
  } while (hi - lo > 1);
  const int s0 = __ldg(p.query_starts + lo), s1 = __ldg(p.query_starts + lo + 1);
  const int L = __ldg(p.context_lens + lo);
  if (s0 < 0 || s1 < s0 || s1 > p.num_rows || L < s1 - s0 || L > p.max_ctx) {
    *bad = true;
    return false;
  }
  const int nt = s1 - s0;
  const int i = slot - (s0 / pair + lo);
  const int npairs = (nt + pair - 1) / pair;
  if (i < 0 || i >= npairs) return false;
  const int at = (npairs - 1 - i) * pair;
  un.b = lo;
  un.L = L;
  un.row0 = s0 + at;
  un.ntok = min(pair, nt - at);
  un.pos0 = L - nt + at;
  const int a = p.window > 0 ? max(0, un.pos0 - p.window + 1) / kPromptTile : 0;
  const int e = (un.pos0 + un.ntok - 1) / kPromptTile + 1;
  un.parts = (e - a + p.split - 1) / p.split;
  if (un.part >= un.parts) return false;
  un.t0 = a + un.part * p.split;
  un.t1 = min(e, un.t0 + p.split);
  un.nonfinite = 0;
  return true;
}

// Tokens, first position and K/V tiles [a, e) of tile s of the pair.
struct PromptSub {
  int n, first, a, e;
};
__device__ __forceinline__ PromptSub prompt_sub(const PromptParams& p, const PromptUnit& un,
                                                int s) {
  PromptSub r;
  r.n = min(p.sub_tokens, un.ntok - s * p.sub_tokens);
  r.first = un.pos0 + s * p.sub_tokens;
  r.a = un.t0;
  if (p.window > 0) r.a = max(r.a, max(0, r.first - p.window + 1) / kPromptTile);
  r.e = r.n > 0 ? min(un.t1, (r.first + r.n - 1) / kPromptTile + 1) : r.a;
  r.e = max(r.e, r.a);
  return r;
}

// Block ids of a unit's pages for one warp: 32 (four tiles) in lane order, and the 32 behind
// them.  Pages behind the context's end, pages in front of every query token's window, whose table
// entries are not read, and ids outside the pool (an error) become num_blocks.
struct PromptPages {
  int ids, next;

  // Those from the i-th of the unit on, a multiple of 32; called for each such i in turn.
  __device__ __forceinline__ void take(const PromptParams& p, const PromptUnit& un, int i,
                                       int lane) {
    constexpr int kPages = kPromptTile / kBlockSize;
    const int first = p.window > 0 ? max(0, un.pos0 - p.window + 1) / kBlockSize : 0;
#pragma unroll 1
    for (int read = i == 0 ? 0 : 32; read <= 32; read += 32) {
      const int pg = un.t0 * kPages + i + read + lane;
      ids = next;
      next = p.num_blocks;
      if (pg >= first && pg * kBlockSize < un.L && pg < un.t1 * kPages) {
        const int id = __ldg(p.block_tables + static_cast<size_t>(un.b) * p.mbs + pg);
        if (static_cast<unsigned>(id) < static_cast<unsigned>(p.num_blocks))
          next = id;
        else
          atomicOr(&g_pa_err, kErrBounds);
      }
    }
  }
};

// Whether some query token of [first, last] does not see every key of tile t.
__device__ __forceinline__ bool prompt_masked(const PromptParams& p, int t, int first, int last) {
  return t * kPromptTile + kPromptTile - 1 > first ||
         (p.window > 0 && t * kPromptTile <= last - p.window);
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// Waits a limited number of tries, each of which sleeps a while.  There are many in the code of
// a CTA's roles, which shares one instruction cache; so a role reports the timeout at its end.
struct PromptWaits {
  int tries = kPromptTries;             // 0 behind a wait that ran out

  __device__ __forceinline__ bool ok() const { return tries != 0; }
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
    int i = 0;
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
      if (++i > tries) {
        tries = 0;
        break;
      }
    }
  }
  // All lanes of the warp go on, or none.
  __device__ __forceinline__ bool all_ok() {
    tries = __all_sync(0xffffffffu, tries != 0) ? tries : 0;
    return tries != 0;
  }
  __device__ __forceinline__ void report() const {
    if (tries == 0 && (threadIdx.x & 31) == 0) atomicOr(&g_pa_err, kErrTimeout);
  }
};

// One lane of the warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(yes));
  return yes != 0;
}

// A value that all lanes hold, in a uniform register.
__device__ __forceinline__ uint32_t uniform(uint32_t x) {
  return __reduce_max_sync(0xffffffffu, x);
}

// MMAs and commits of the lane with `leader` set, in code that the whole warp runs.
__device__ __forceinline__ void lead_mma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
// (A in tensor memory, K-major: row r in lane r, two 16-bit values per 32-bit column)
__device__ __forceinline__ void lead_mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void lead_commit(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      ::"r"(smem_u32(bar)), "r"(leader)
      : "memory");
}

// The two words of a shared-memory operand's descriptor (128-byte swizzle, 8-row groups 1024
// bytes apart): the low one takes byte offsets / 16 by addition.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo_bytes) {
  return static_cast<uint32_t>(tc::smem_desc(saddr, lbo_bytes, 1024));
}
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
  constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (tc::kSwizzle128B << 29);
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}

__device__ __forceinline__ void prefetch_l2(const uint8_t* at) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("max.u16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ uint32_t min_u16x2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("min.u16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ uint32_t add_u16x2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("add.u16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}

// 16 bytes of a page, which nothing else on this SM reads.
__device__ __forceinline__ uint4 load_once(const uint8_t* from) {
  uint4 w;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
               : "l"(from));
  return w;
}

// Bits 15 and 31: the low, the high bf16 of the word is infinite or NaN.
__device__ __forceinline__ uint32_t nonfinite_bf16x2(uint32_t w) {
  return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}
// (mask: 0xFFFF, or 0 to leave them)
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t w, uint32_t mask) {
  return w & ~((nonfinite_bf16x2(w) >> 15) * mask);
}

__device__ __forceinline__ uint32_t pack_bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// tcgen05.wait::ld, with the loaded registers tied behind it.
template <int N>
__device__ __forceinline__ void tmem_wait_regs(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

template <int kRegs>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_fewer() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Of two 16-byte pieces, a lane whose bit B is clear keeps the first and gets the first of the
// lane with that bit set in place of the second, which goes there in place of its first.
template <int B>
__device__ __forceinline__ void swap_pieces(uint4& a, uint4& b, int lane) {
  const bool up = (lane & B) != 0;
  const uint32_t* pa = reinterpret_cast<const uint32_t*>(&a);
  const uint32_t* pb = reinterpret_cast<const uint32_t*>(&b);
  uint32_t got[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    got[k] = __shfl_xor_sync(0xffffffffu, up ? pa[k] : pb[k], B);
  const uint4 x = make_uint4(got[0], got[1], got[2], got[3]);
  if (up)
    a = x;
  else
    b = x;
}

// A page of V that stays bf16, and one of them that holds infinities or NaN; a tile's as bits
// (page_bit, and the one above it).  kSplitUnknown: not looked up.
constexpr uint32_t kSplitPage = 1u, kOddPage = 3u, kSplitUnknown = 1u << 31;
__host__ __device__ constexpr uint32_t page_bit(int pg) { return 1u << (pg % 4 * 8 + pg / 4 * 4); }
__device__ __forceinline__ uint32_t split_pages(uint32_t bytes) {
  uint2 w;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "r"(bytes) : "memory");
  return w.x | w.y << 4;
}

// A row's 128 scores of a K/V tile in one thread, and the weights that take their place.
struct PromptScores {
  uint32_t x[4][32];
  uint32_t w[4][16];
  uint64_t part[4], factor, offset;

  __device__ __forceinline__ float score(int i) const { return __uint_as_float(x[i / 32][i % 32]); }
  __device__ __forceinline__ void load(uint32_t taddr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) tc::tmem_ld32(taddr + i * 32, x[i]);
    tc::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 4; ++i) tmem_wait_regs(x[i]);
  }
  __device__ __forceinline__ void multiply(float c) {
#pragma unroll
    for (int i = 0; i < 128; ++i) x[i / 32][i % 32] = __float_as_uint(score(i) * c);
  }
  // Scores outside (lo, hi] to -inf, but for quarters that lie wholly inside for the warp.
  __device__ __forceinline__ void mask(int lo, int hi) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int a = max(0, lo + 1 - 32 * i), b = hi + 1 - 32 * i;     // columns [a, b) of it
      const uint32_t in = (b <= 0 ? 0u : b >= 32 ? ~0u : (1u << b) - 1u) &
                          (a >= 32 ? 0u : ~0u << a);
      if (!__all_sync(0xffffffffu, in == ~0u)) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (!(in >> k & 1u)) x[i][k] = __float_as_uint(-CUDART_INF_F);
      }
    }
  }
  __device__ __forceinline__ float largest() const {
    float m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = fmaxf(score(2 * k), score(2 * k + 1));
#pragma unroll
    for (int k = 8; k < 128; k += 8)
#pragma unroll
      for (int a = 0; a < 4; ++a) m[a] = max3(m[a], score(k + 2 * a), score(k + 2 * a + 1));
    return fmaxf(max3(m[0], m[1], m[2]), m[3]);
  }
  __device__ __forceinline__ void begin(float c, float off) {
    factor = pack_f32x2(c, c);
    offset = pack_f32x2(off, off);
    part[0] = part[1] = part[2] = part[3] = 0ull;
  }
  // Weights 2^(factor x + offset) of the pairs of keys [FROM, TO), packed into w.  Each step
  // takes one pair through each of three stages, so that the exponentials (four cycles each)
  // run beside the rest; also(k) is an instruction or two more for step k.
  template <int FROM, int TO, typename Also>
  __device__ __forceinline__ void weights(Also also) {
    constexpr int kExp = 3, kPack = 8;                  // steps behind the argument
#pragma unroll
    for (int k = FROM; k < TO + kPack; ++k) {
      if (k < TO) {
        uint32_t* v = &x[k / 16][k % 16 * 2];
        const uint64_t y = fma_f32x2(pack_f32x2(__uint_as_float(v[0]), __uint_as_float(v[1])),
                                     factor, offset);
        v[0] = static_cast<uint32_t>(y);
        v[1] = static_cast<uint32_t>(y >> 32);
        also(k);
      }
      if (k - kExp >= FROM && k - kExp < TO) {
        const int j = k - kExp;
        uint32_t* v = &x[j / 16][j % 16 * 2];
        v[0] = __float_as_uint(hw_exp2(__uint_as_float(v[0])));
        v[1] = __float_as_uint(hw_exp2(__uint_as_float(v[1])));
      }
      if (k - kPack >= FROM) {
        const int j = k - kPack;
        const float e0 = score(2 * j), e1 = score(2 * j + 1);
        part[j & 3] = add_f32x2(part[j & 3], pack_f32x2(e0, e1));
        w[j / 16][j % 16] = half2_bits(__floats2half2_rn(e0, e1));
      }
    }
  }
  __device__ __forceinline__ float total() const {
    const uint64_t y = add_f32x2(add_f32x2(part[0], part[1]), add_f32x2(part[2], part[3]));
    return __uint_as_float(static_cast<uint32_t>(y)) + __uint_as_float(static_cast<uint32_t>(y >> 32));
  }
  // The largest sum of eight weights of the first half: no less than any of them.
  __device__ __forceinline__ float most_of_eight() const {
    float y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = __uint_as_float(static_cast<uint32_t>(part[i]));
      y[2 * i + 1] = __uint_as_float(static_cast<uint32_t>(part[i] >> 32));
    }
    return fmaxf(max3(max3(y[0], y[1], y[2]), y[3], y[4]), max3(y[5], y[6], y[7]));
  }
  // The weights over the scores, the first half of the keys announced once the third quarter is
  // computed (if that is all of them: `announce`); the second half is stored, not yet complete.
  __device__ __forceinline__ void finish(uint32_t taddr, uint64_t* half, bool announce) {
    tc::tmem_st16(taddr, w[0]);
    tc::tmem_st16(taddr + 16, w[1]);
    weights<32, 48>([](int) {});
    tc::tmem_wait_st();
    tc::fence_before_sync();
    __syncwarp();
    if (announce) mbar_arrive(half);
    tc::tmem_st16(taddr + 32, w[2]);
    weights<48, 64>([](int) {});
    tc::tmem_st16(taddr + 48, w[3]);
  }
};

// The weights of a tile, stored as f16, for the V pages of `split` that stay bf16: times
// 2^kPromptVShift and in two bf16 parts, which hold the f16 exactly; the second lies 64 columns
// behind the first.  Where they meet infinities, which every row sees, neither part is 0: weights
// are f16's smallest at least, and a second part of 2^-20 stands for none.  (A loop of little code,
// which all roles' instructions have to share a cache with.)
__device__ __forceinline__ void split_weights(uint32_t taddr, uint32_t split) {
#pragma unroll 1
  for (int pg = 0; pg < kPromptTile / kBlockSize; ++pg) {
    if (!(split & page_bit(pg))) continue;
    const bool odd = (split & page_bit(pg) << 1) != 0u;
    const float least = odd ? 0x1p-24f : 0.f, none = odd ? 0x1p-20f : 0.f;
    uint32_t x[8], rest[8];
    tc::tmem_ld8(taddr + pg * 8, x);
    tc::tmem_wait_ld();
    tmem_wait_regs(x);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float2 e = __half22float2(*reinterpret_cast<const __half2*>(&x[k]));
      e.x = fmaxf(e.x, least) * static_cast<float>(1 << kPromptVShift);
      e.y = fmaxf(e.y, least) * static_cast<float>(1 << kPromptVShift);
      x[k] = __byte_perm(__float_as_uint(e.x), __float_as_uint(e.y), 0x7632);    // towards 0
      const float r0 = e.x - bf16_lo(x[k]), r1 = e.y - bf16_hi(x[k]);
      rest[k] = pack_bf16x2_rn(r0 == 0.f ? e.x * none : r0, r1 == 0.f ? e.y * none : r1);
    }
    tc::tmem_st8(taddr + pg * 8, x);
    tc::tmem_st8(taddr + kPromptTile / 2 + pg * 8, rest);
  }
  tc::tmem_wait_st();
}

// A V element for the rows that see it, from the pool.
template <int D, bool KV8>
__device__ __forceinline__ float prompt_value(const PromptParams& p, const PromptUnit& un, int j,
                                              int d) {
  const int id = __ldg(p.block_tables + static_cast<size_t>(un.b) * p.mbs + j / kBlockSize);
  if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_blocks)) return 0.f;
  const size_t page = static_cast<size_t>(id) * p.Hkv + un.head;
  if constexpr (KV8) {
    const uint32_t c = static_cast<const uint8_t*>(p.v_pool)[(page * D + d) * kBlockSize +
                                                             j % kBlockSize];
    const uint32_t h = e4m3x2_to_f16x2(c);
    return __half2float(__low2half(*reinterpret_cast<const __half2*>(&h)));
  }
  return __bfloat162float(static_cast<const __nv_bfloat16*>(
      p.v_pool)[(page * kBlockSize + j % kBlockSize) * D + d]);
}

// 16 E4M3 codes as 16 f16.
__device__ __forceinline__ void widen16(const uint4& w, uint4& lo, uint4& hi) {
  lo = make_uint4(e4m3x2_to_f16x2(w.x), e4m3x2_to_f16x2(w.x >> 16), e4m3x2_to_f16x2(w.y),
                  e4m3x2_to_f16x2(w.y >> 16));
  hi = make_uint4(e4m3x2_to_f16x2(w.z), e4m3x2_to_f16x2(w.z >> 16), e4m3x2_to_f16x2(w.w),
                  e4m3x2_to_f16x2(w.w >> 16));
}

// bf16 values as f16 times 2^kPromptVShift: whether all of the warp's words w hold magnitudes from
// 2^-25, whose last bit is f16's smallest number then, to below 2^8, or 0.
template <int N>
__device__ __forceinline__ bool fits_f16(const uint4 (&w)[N]) {
  constexpr uint32_t kMost = (127 - kPromptVShift + 16) << 7;
  constexpr uint32_t kLeast = (127 - kPromptVShift - 17) << 7;
  uint32_t most[2] = {0u, 0u}, least[2] = {~0u, ~0u};     // less 1, so that 0 is the largest
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t mag = x[k] & 0x7FFF7FFFu;
      most[k & 1] = max_u16x2(most[k & 1], mag);
      least[k & 1] = min_u16x2(least[k & 1], add_u16x2(mag, ~0u));
    }
  }
  most[0] = max_u16x2(most[0], most[1]);
  least[0] = min_u16x2(least[0], least[1]);
  return __all_sync(0xffffffffu, max(most[0] & 0xFFFFu, most[0] >> 16) < kMost &&
                                     min(least[0] & 0xFFFFu, least[0] >> 16) >= kLeast - 1u);
}
__device__ __forceinline__ uint32_t scaled_f16x2(uint32_t w) {     // a 0 becomes one by rounding
  w += (kPromptVShift << 7) * 0x00010001u;
  return half2_bits(__floats2half2_rn(bf16_lo(w), bf16_hi(w)));
}

// 16 bytes of shared memory (the tiles' addresses are computed, and as generic ones a tile took
// three times as long to widen).
__device__ __forceinline__ uint4 load16(uint32_t at) {
  uint4 w;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
               : "r"(at)
               : "memory");
  return w;
}
__device__ __forceinline__ void store16(uint32_t at, uint4 w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w.x), "r"(w.y), "r"(w.z),
               "r"(w.w)
               : "memory");
}

__device__ __forceinline__ int load4(uint32_t at) {
  int x;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}

__device__ __forceinline__ PromptUnit load_unit(const PromptUnit& from) {
  union {
    uint4 w[3];
    PromptUnit un;
  } u;
  static_assert(sizeof(PromptUnit) == sizeof(u.w), "three pieces");
#pragma unroll
  for (int i = 0; i < 3; ++i) u.w[i] = load16(smem_u32(&from) + 16 * i);
  return u.un;
}

// The byte mask of the codes 0x7F and 0xFF (NaN) in a word.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return (((w & 0x7F7F7F7Fu) + 0x01010101u & 0x80808080u) >> 7) * 0xFFu;
}

// A K tile: keys x D codes, as TMA left them, to [half][key][64 dims] f16 with the 128-byte
// swizzle.  Consecutive lanes take what lies in different banks on both sides.
template <int D>
__device__ __forceinline__ void widen_keys(uint32_t dst, uint32_t raw, int lane, int worker,
                                           int workers) {
  constexpr int C = D / 16;                    // 16-dim pieces of a row
#pragma unroll 1
  for (int i = worker; i < kPromptTile * C / 32; i += workers) {
    int key, c;
    if constexpr (C == 8) {                    // 8 rows of one piece, four pieces
      key = (i >> 1) * 8 + (lane & 7);
      c = (i & 1) * 4 + (lane >> 3);
    } else {                                   // 8 rows of four pieces
      key = i * 8 + (lane >> 2);
      c = lane & 3;
    }
    const int at = C == 8 ? key * 128 + ((c ^ (key & 7)) << 4) : key * 64 + c * 16;
    uint4 lo, hi;
    widen16(load16(raw + at), lo, hi);
    const uint32_t row = dst + (c >> 2) * (kPromptTile * 128) + key * 128;
    const int ch = (c & 3) * 2;
    store16(row + ((ch ^ (key & 7)) << 4), lo);
    store16(row + (((ch + 1) ^ (key & 7)) << 4), hi);
  }
}

// A V tile: pages of D rows of 16 keys, to [half of 64 keys][dim][64 keys] f16.  At a border of
// the mask the codes from key `end` of the tile on and NaN become 0; whether there was a NaN.
template <int D>
__device__ __forceinline__ bool widen_values(uint32_t dst, uint32_t raw, int lane, int worker,
                                             int workers, bool border, int end) {
  bool found = false;
#pragma unroll 1
  for (int i = worker; i < kPromptTile / kBlockSize * D / 32; i += workers) {
    const int pg = i / (D / 32), d = i % (D / 32) * 32 + lane;
    uint4 w = load16(raw + (pg * D + d) * 16);
    if (__builtin_expect(border, 0)) {
      uint32_t* x = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int left = end - pg * kBlockSize - 4 * k;      // codes of this word that count
        if (left < 4) x[k] &= left <= 0 ? 0u : (1u << 8 * left) - 1u;
        const uint32_t bad = nan_codes(x[k]);
        found |= bad != 0;
        x[k] &= ~bad;
      }
    }
    uint4 lo, hi;
    widen16(w, lo, hi);
    const uint32_t row = dst + (pg >> 2) * (D * 128) + d * 128;
    const int ch = (pg & 3) * 2;
    store16(row + ((ch ^ (d & 7)) << 4), lo);
    store16(row + (((ch + 1) ^ (d & 7)) << 4), hi);
  }
  return found;
}

// A query row, D bf16 in halves of 128 swizzled bytes, to f16 times 2^-e; returns e.
template <int D>
__device__ __forceinline__ int widen_query(uint32_t tile, int row) {
  float most = 0.f;
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    const uint4 w =
        load16(tile + (c >> 3) * (kPromptTile * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4));
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      most = fmaxf(most, fmaxf(fabsf(bf16_lo(x[k])), fabsf(bf16_hi(x[k]))));
  }
  // the exponent of the largest element, and 7 less, while 2^e and 2^-e are normal numbers
  int e = most > 0.f && most < CUDART_INF_F
              ? static_cast<int>(__float_as_uint(most) >> 23) - 127 - 7 : 0;
  e = max(-126, e);
  const float up = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    const uint32_t at =
        tile + (c >> 3) * (kPromptTile * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
    uint4 w = load16(at);
    uint32_t* x = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      x[k] = half2_bits(__floats2half2_rn(bf16_lo(x[k]) * up, bf16_hi(x[k]) * up));
    store16(at, w);
  }
  return e;
}

template <int D, bool KV8>
__global__ void __launch_bounds__(PromptGeo<D, KV8>::kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tmv, const PromptParams p) {
  using Gm = PromptGeo<D, KV8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  auto& ms = *reinterpret_cast<PromptMisc<D, KV8>*>(smem + Gm::kMiscOff);
  static_assert(sizeof(PromptMisc<D, KV8>) <= Gm::kMiscBytes, "misc area");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ------------------------------------------------------------------ setup
  if (threadIdx.x == 0) {
    for (int i = 0; i < Gm::kKStages; ++i) {
      mbar_init(&ms.k_full[i], KV8 ? Gm::kAux : 1);
      mbar_init(&ms.k_empty[i], 1);
    }
    for (int i = 0; i < Gm::kVStages; ++i) {
      mbar_init(&ms.v_full[i], KV8 ? Gm::kAux : Gm::kPages);
      mbar_init(&ms.v_empty[i], 1);
    }
    for (int i = 0; i < Gm::kRawStages; ++i) {
      mbar_init(&ms.raw_full[i], 1);
      mbar_init(&ms.raw_empty[i], Gm::kAux);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms.q_full[i], 1);
      mbar_init(&ms.q_empty[i], 1);
      mbar_init(&ms.s_full[i], 1);
      mbar_init(&ms.p_half[i], 4);
      mbar_init(&ms.p_full[i], 4);
      mbar_init(&ms.o_full[i], 1);
      mbar_init(&ms.o_free[i], 4);
      mbar_init(&ms.unit_full[i], 1);
      mbar_init(&ms.unit_empty[i], 1 + Gm::kSoftmaxWarps + Gm::kAux);
      mbar_init(&ms.unit_checked[i], Gm::kAux);
      mbar_init(&ms.q_wide[i][0], Gm::kAux);
      mbar_init(&ms.q_wide[i][1], Gm::kAux);
    }
    mbar_init(&ms.fin, 1);
    fence_barrier_init();
  }
  if (warp == Gm::kSoftmaxWarps + 1) tc::tmem_alloc(&ms.tmem_base, Gm::kTmemCols);
  // rows of the Q tiles that hold no query row stay zero
  for (int i = threadIdx.x; i < 2 * Gm::kTileBytes / 16; i += Gm::kThreads)
    store16(smem_u32(smem) + i * 16, make_uint4(0, 0, 0, 0));
  tc::fence_proxy_async_smem();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = ms.tmem_base;
  if (p.max_parts > 1) grid_launch_dependents();       // the merge

  if (warp >= Gm::kSoftmaxWarps) {
    regs_fewer<Gm::kOtherRegs>();
    if (warp == Gm::kSoftmaxWarps) {
      // -------------------------------------------------------------- loads
      if (lane == 0) {
        tma_prefetch_map(&tmq);
        tma_prefetch_map(&tmk);
        if constexpr (KV8) tma_prefetch_map(&tmv);
      }
      // K tiles (K and V tiles of FP8 pages) into their ring
      constexpr int kRing = KV8 ? Gm::kRawStages : Gm::kKStages;
      uint64_t* full = KV8 ? ms.raw_full : ms.k_full;
      uint64_t* empty = KV8 ? ms.raw_empty : ms.k_empty;
      PromptWaits wait;
      int item = 0, ui = 0, u = blockIdx.x;
      uint32_t n_q[2] = {0, 0};                        // loads of each tile's query rows
      // the unit behind the present one: the next that no CTA has taken (asked for a few tiles
      // before it is needed, so that none is held for long), or every gridDim.x-th
      auto claim = [&]() {
        return p.counter == nullptr ? u + static_cast<int>(gridDim.x)
               : lane == 0          ? atomicAdd(p.counter, 1) + static_cast<int>(gridDim.x)
                                    : 0;
      };
      // the query rows, each tile's once its last unit's scores no longer need theirs: behind the
      // first K tile, but for FP8 pages in front of it, because the rows have to be widened
      auto load_query = [&](const PromptUnit& un) {
#pragma unroll 1
        for (int s = 0; s < 2 && wait.ok(); ++s) {
          const PromptSub sub = prompt_sub(p, un, s);
          if (sub.a == sub.e) continue;
          wait(&ms.q_empty[s], ((s ? n_q[1] : n_q[0]) & 1u) ^ 1u);
          if (!wait.all_ok()) break;
          ++(s ? n_q[1] : n_q[0]);
          if (lane == 0) {
            mbar_arrive_expect_tx(&ms.q_full[s], static_cast<uint32_t>(Gm::kHalves * p.sub_tokens *
                                                                       p.G * 128));
            for (int hh = 0; hh < Gm::kHalves; ++hh)
              tma_load_4d(smem + s * Gm::kTileBytes + hh * Gm::kHalfBytes, &tmq, &ms.q_full[s],
                          hh * 64, 0, un.head, un.row0 + s * p.sub_tokens);
          }
        }
      };
      int next = 0;
      while (true) {
        PromptUnit un;
        un.b = -1;
        while (u < p.num_units) {
          bool bad;
          if (prompt_unit(p, u, un, &bad)) break;
          if (bad && lane == 0) atomicOr(&g_pa_err, kErrBounds);
          un.b = -1;
          u = __shfl_sync(0xffffffffu, claim(), 0);
        }
        wait(&ms.unit_empty[ui & 1], (static_cast<uint32_t>(ui >> 1) & 1u) ^ 1u);
        if (!wait.all_ok()) break;
        if (lane == 0) {
          ms.unit[ui & 1] = un;
          mbar_arrive(&ms.unit_full[ui & 1]);
        }
        ++ui;
        if (un.b < 0) break;
        if (KV8) load_query(un);
        PromptPages pages;
        const int ask = max(un.t0, un.t1 - 4);
        for (int t = un.t0; t < un.t1 && wait.ok(); ++t) {
          if (t == ask) next = claim();
          // a bf16 page is one box of 16 keys per half, an FP8 page one box; a row past the pool
          // is filled with zeros
          constexpr int kBoxes = KV8 ? 1 : Gm::kHalves;
          const int box = lane & (Gm::kPages * kBoxes - 1);
          const int pg = box / kBoxes, h = box % kBoxes;
          const int first = (t - un.t0) * Gm::kPages;
          if (first % 32 == 0) pages.take(p, un, first, lane);
          const int id = __shfl_sync(0xffffffffu, pages.ids, (first & 31) + pg);
          const int page = id * p.Hkv + (id == p.num_blocks ? 0 : un.head);
          for (int kv = 0; kv < (KV8 ? 2 : 1); ++kv, ++item) {
            const int st = item % kRing;
            wait(&empty[st], (static_cast<uint32_t>(item / kRing) & 1u) ^ 1u);
            if (!wait.all_ok()) break;
            if (lane == 0)
              mbar_arrive_expect_tx(&full[st], KV8 ? Gm::kRawBytes : Gm::kTileBytes);
            __syncwarp();
            if (lane < Gm::kPages * kBoxes) {
              if constexpr (KV8)
                tma_load_2d(smem + Gm::kRawOff + st * Gm::kRawBytes + pg * kBlockSize * D,
                            kv ? &tmv : &tmk, &full[st], 0, page * (kv ? D / 8 : kBlockSize));
              else
                tma_load_2d(smem + Gm::kKOff + st * Gm::kTileBytes + h * Gm::kHalfBytes +
                                pg * kBlockSize * 128,
                            &tmk, &full[st], h * 64, page * kBlockSize);
            }
          }
          if (!KV8 && t == un.t0) load_query(un);
        }
        if (!wait.ok()) break;
        u = __shfl_sync(0xffffffffu, next, 0);
      }
      wait.report();
      // no copy may still be landing when the CTA ends
      if (lane == 0) {
        wait.tries = kPromptTries;
        for (int i = max(0, item - kRing); i < item; ++i)
          wait(&full[i % kRing], static_cast<uint32_t>(i / kRing) & 1u);
        for (int s = 0; s < 2; ++s)
          if (n_q[s] > 0) wait(&ms.q_full[s], (n_q[s] - 1) & 1u);
      }
      __syncwarp();
    } else if (warp == Gm::kSoftmaxWarps + 1) {
      // -------------------------------------------------------------- MMA issue
      const uint32_t leader = elect_one() ? 1u : 0u;
      // The whole warp goes through the steps, so that stages and descriptors are uniform
      // values, and one elected lane issues.
      constexpr uint32_t kIdS = tc::idesc_f16<128, kPromptTile, false, false, !KV8>();
      constexpr uint32_t kIdO = tc::idesc_f16<128, D, false, !KV8, false>();
      constexpr uint32_t kIdSplit = tc::idesc_f16<128, D, false, true, true>();
      const uint32_t kring = smem_u32(smem + Gm::kKOff), vring = smem_u32(smem + Gm::kVOff);
      const uint32_t qsm = smem_u32(smem);
      const uint32_t tm = uniform(tmem);
      // Lanes agree to go on once per tile; a wait that ran out in between leaves wrong products
      // behind an error that is reported.
      PromptWaits wait;
      int kst = 0, vst = 0;                            // stage and phase of the next K, V tile
      uint32_t kph = 0, vph = 0;
      auto k_done = [&]() {
        lead_commit(leader, &ms.k_empty[kst]);
        if (++kst == Gm::kKStages) {
          kst = 0;
          kph ^= 1u;
        }
      };
      uint32_t n_p[2] = {0, 0}, n_u[2] = {0, 0};       // P tiles taken, units of each tile begun
      uint32_t n_q[2] = {0, 0};                        // query rows of each tile taken
      // S of tile s from the K tile at `lo`
      auto scores = [&](int s, uint32_t lo) {
        const uint32_t a = desc_lo(qsm + s * Gm::kTileBytes, 16);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * Gm::kHalfBytes + (k & 3) * 32) >> 4;
          lead_mma_ss(leader, tm + s * kPromptTile, desc_of(a + off), desc_of(lo + off), kIdS,
                      k > 0 ? 1u : 0u);
        }
        lead_commit(leader, &ms.s_full[s]);
      };
      for (int ui = 0; wait.ok(); ++ui) {
        wait(&ms.unit_full[ui & 1], static_cast<uint32_t>(ui >> 1) & 1u);
        if (!wait.all_ok()) break;
        PromptUnit un = load_unit(ms.unit[ui & 1]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.unit_empty[ui & 1]);
        un.b = __shfl_sync(0xffffffffu, un.b, 0);
        if (un.b < 0) break;
        un.t0 = __shfl_sync(0xffffffffu, un.t0, 0);
        un.t1 = __shfl_sync(0xffffffffu, un.t1, 0);
        un.pos0 = __shfl_sync(0xffffffffu, un.pos0, 0);
        un.ntok = __shfl_sync(0xffffffffu, un.ntok, 0);
        const PromptSub sub[2] = {prompt_sub(p, un, 0), prompt_sub(p, un, 1)};
        // P.V of K/V tile t, then S of the next
        for (int t = un.t0 - 1; t < un.t1; ++t) {
          const bool more = t + 1 < un.t1;
          const uint32_t vlo =
              uniform(desc_lo(vring + vst * Gm::kTileBytes, KV8 ? 16 : Gm::kHalfBytes));
          const uint32_t klo = uniform(desc_lo(kring + kst * Gm::kTileBytes, 16));
          uint32_t split = 0u;
          if (t >= un.t0) {
            wait(&ms.v_full[vst], vph);
            if constexpr (!KV8) split = split_pages(smem_u32(ms.v_split[vst]));
          }
          bool k_here = false;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (sub[s].a <= t && t < sub[s].e) {
              if (t == sub[s].a) wait(&ms.o_free[s], (n_u[s]++ & 1u) ^ 1u);
#pragma unroll
              for (int half = 0; half < 2; ++half) {   // of the keys
                wait(half ? &ms.p_full[s] : &ms.p_half[s], n_p[s] & 1u);
                __syncwarp();
                tc::fence_after_sync();
                const uint32_t o = tm + Gm::kO + s * D, w = tm + s * kPromptTile;
                if (KV8 || __all_sync(0xffffffffu, split == 0u)) {
#pragma unroll
                  for (int i = 0; i < kPromptTile / 32; ++i) {
                    const int k = half * (kPromptTile / 32) + i;
                    const uint32_t off =
                        (KV8 ? (k >> 2) * (D * 128) + (k & 3) * 32 : k * 2048) >> 4;
                    lead_mma_ts(leader, o, w + k * 8, desc_of(vlo + off), kIdO,
                                k > 0 || t > sub[s].a ? 1u : 0u);
                  }
                } else {
#pragma unroll 1
                  for (int i = 0; i < kPromptTile / 32; ++i) {
                    const int k = half * (kPromptTile / 32) + i;
                    const bool two = (split & page_bit(k)) != 0u;
                    lead_mma_ts(leader, o, w + k * 8, desc_of(vlo + (k * 2048 >> 4)),
                                two ? kIdSplit : kIdO, k > 0 || t > sub[s].a ? 1u : 0u);
                    if (two)
                      lead_mma_ts(leader, o, w + kPromptTile / 2 + k * 8,
                                  desc_of(vlo + (k * 2048 >> 4)), kIdSplit, 1u);
                  }
                }
              }
              if (t + 1 == sub[s].e) lead_commit(leader, &ms.o_full[s]);
              ++n_p[s];
            }
            if (sub[s].a <= t + 1 && t + 1 < sub[s].e) {
              if (!k_here) wait(&ms.k_full[kst], kph);
              k_here = true;
              if (t + 1 == sub[s].a) {
                if constexpr (KV8)
                  wait(&ms.q_wide[ui & 1][s], static_cast<uint32_t>(ui >> 1) & 1u);
                else
                  wait(&ms.q_full[s], n_q[s]++ & 1u);
              }
              __syncwarp();
              tc::fence_after_sync();
              scores(s, klo);
              if (t + 2 == sub[s].e) lead_commit(leader, &ms.q_empty[s]);
            }
          }
          if (t >= un.t0) {
            lead_commit(leader, &ms.v_empty[vst]);
            if (++vst == Gm::kVStages) {
              vst = 0;
              vph ^= 1u;
            }
          }
          if (more) k_done();
          if (!wait.all_ok()) break;
        }
      }
      // every MMA has completed before the CTA gives its tensor memory back
      __syncwarp();
      lead_commit(leader, &ms.fin);
      wait.report();
      wait.tries = kPromptTries;
      wait(&ms.fin, 0);
      __syncwarp();
    } else {
      // -------------------------------------------------------------- V, or FP8 tiles widened
      const int aux = warp - Gm::kSoftmaxWarps - 2;
      PromptWaits wait;
      int item = 0, tiles = 0, turn = 0;               // FP8 tiles, V tiles so far; whose the next
                                                       //   page is
      uint32_t n_q[2] = {0, 0};
      for (int ui = 0; wait.ok(); ++ui) {
        wait(&ms.unit_full[ui & 1], static_cast<uint32_t>(ui >> 1) & 1u);
        if (!wait.all_ok()) break;
        const PromptUnit un = load_unit(ms.unit[ui & 1]);
        if (un.b < 0) break;
        const int last = un.pos0 + un.ntok - 1;
        auto taken_out = [&]() {
          if (lane == 0)
            asm volatile("st.shared.b32 [%0], 1;" ::"r"(smem_u32(&ms.unit[ui & 1].nonfinite))
                         : "memory");
        };
        if constexpr (KV8) {
#pragma unroll 1
          for (int s = 0; s < 2; ++s) {
            const PromptSub sub = prompt_sub(p, un, s);
            if (sub.a < sub.e) {
              wait(&ms.q_full[s], (s ? n_q[1]++ : n_q[0]++) & 1u);
              if (!wait.all_ok()) break;
              for (int r = aux * 32 + lane; r < p.sub_tokens * p.G; r += Gm::kAux * 32)
                ms.q_exp[ui & 1][s][r] =
                    static_cast<int8_t>(widen_query<D>(smem_u32(smem) + s * Gm::kTileBytes, r));
              tc::fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.q_wide[ui & 1][s]);
          }
          for (int t = un.t0; t < un.t1; ++t, ++tiles) {
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv, ++item) {
              const int rs = item % Gm::kRawStages;
              const int st = tiles % (kv ? Gm::kVStages : Gm::kKStages);
              const uint32_t use = static_cast<uint32_t>(tiles / (kv ? Gm::kVStages
                                                                     : Gm::kKStages));
              // (both asked for at once: each answer takes a while)
              uint64_t* in = &ms.raw_full[rs];
              uint64_t* to = kv ? &ms.v_empty[st] : &ms.k_empty[st];
              const uint32_t in_phase = static_cast<uint32_t>(item / Gm::kRawStages) & 1u;
              const uint32_t to_phase = (use & 1u) ^ 1u;
              const bool here = tc::mbar_test(in, in_phase), free = tc::mbar_test(to, to_phase);
              if (!here) wait(in, in_phase);
              if (!free) wait(to, to_phase);
              __syncwarp();
              const uint32_t base = smem_u32(smem), raw = base + Gm::kRawOff + rs * Gm::kRawBytes;
              if (kv) {
                const bool found = widen_values<D>(
                    base + Gm::kVOff + st * Gm::kTileBytes, raw, lane, aux, Gm::kAux,
                    prompt_masked(p, t, un.pos0, last), un.L - t * kPromptTile);
                if (__any_sync(0xffffffffu, found)) taken_out();
              } else {
                widen_keys<D>(base + Gm::kKOff + st * Gm::kTileBytes, raw, lane, aux, Gm::kAux);
              }
              tc::fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                mbar_arrive(kv ? &ms.v_full[st] : &ms.k_full[st]);
                mbar_arrive(&ms.raw_empty[rs]);
              }
            }
          }
        } else {
          // A TMA box of 16 keys costs its unit about 70 cycles, whatever the bytes, and K's are
          // as many as it can take; and shared memory has no time to be read and written once more
          // beside the products.  So V comes through registers and becomes f16 there, page by page
          // round the warps; a piece of a warp's next page is asked for as soon as one of the
          // present page is stored.
          constexpr int kRowChunks = D / 8;            // 16-byte chunks of a row
          constexpr int kRows = 32 / kRowChunks;       // rows of one warp-wide copy
          constexpr int kPieces = kBlockSize / kRows;
          const int c = lane % kRowChunks, r = lane / kRowChunks;
          constexpr int kPageBytes = kBlockSize * D * 2;
          const int count = (un.t1 - un.t0) * Gm::kPages;
          const uint8_t* const pool = static_cast<const uint8_t*>(p.v_pool) +
                                      static_cast<size_t>(un.head) * kPageBytes + lane * 16;
          auto page_at = [&](int id) {
            // (pages of the pool: below 2^27)
            return pool + static_cast<size_t>((id == p.num_blocks ? 0 : id) * p.Hkv) * kPageBytes;
          };
          PromptPages pages;
          // what is seldom needed of the unit, not kept in registers over the pages
          auto reload = [&]() {
            const uint32_t at = smem_u32(&ms.unit[ui & 1]);
            PromptUnit u;
            u.b = load4(at + offsetof(PromptUnit, b));
            u.ntok = load4(at + offsetof(PromptUnit, ntok));
            u.pos0 = load4(at + offsetof(PromptUnit, pos0));
            u.L = load4(at + offsetof(PromptUnit, L));
            u.t0 = load4(at + offsetof(PromptUnit, t0));
            u.t1 = load4(at + offsetof(PromptUnit, t1));
            return u;
          };
          // whether some query row must not see all of page i
          auto border = [&](int i) {
            const uint32_t at = smem_u32(&ms.unit[ui & 1]);
            const int first = load4(at + offsetof(PromptUnit, pos0)) -
                              load4(at + offsetof(PromptUnit, t0)) * kPromptTile - i * kBlockSize;
            return first < kBlockSize - 1 ||
                   (p.window > 0 && first + load4(at + offsetof(PromptUnit, ntok)) > p.window);
          };
          auto id_of = [&](int i) {
            if (i < Gm::kAux || ((i ^ (i - Gm::kAux)) & 32) != 0)
              pages.take(p, reload(), i & ~31, lane);
            return __shfl_sync(0xffffffffu, pages.ids, i & 31);
          };
          const uint32_t mine = smem_u32(smem) + Gm::kVOff + (c >> 3) * Gm::kHalfBytes + r * 128 +
                                (((c ^ r) & 7) << 4);
          int i = (aux + Gm::kAux - turn) % Gm::kAux;  // this warp's first page
          turn = (turn + count) % Gm::kAux;
          int next = id_of(i);
          uint4 w[kPieces];
#pragma unroll
          for (int k = 0; k < kPieces; ++k) w[k] = load_once(page_at(next) + k * 512);
#pragma unroll 1
          for (; i < count; i += Gm::kAux) {
            const int id = next;
            uint32_t kind = 0u;
            bool fits;
#pragma unroll 1
            for (bool again = true; !(fits = fits_f16(w)) && again; again = false) {
              // what no query row sees has weights of 0, so that any finite number does for it
              const PromptUnit u = reload();
              const int key = u.t0 * kPromptTile + i * kBlockSize + r;
              const int begin = p.window > 0 ? u.pos0 - p.window + 1 : 0, end = u.pos0 + u.ntok;
#pragma unroll
              for (int k = 0; k < kPieces; ++k)
                if (id == p.num_blocks || key + k * kRows < begin || key + k * kRows >= end)
                  w[k] = make_uint4(0u, 0u, 0u, 0u);
            }
            if (__builtin_expect(fits, 1)) {
#pragma unroll
              for (int k = 0; k < kPieces; ++k)
                w[k] = make_uint4(scaled_f16x2(w[k].x), scaled_f16x2(w[k].y), scaled_f16x2(w[k].z),
                                  scaled_f16x2(w[k].w));
            } else {
              // the page stays bf16; infinities and NaN stay where every query row sees it, else
              // they come out, and the rows that see them get them at the end
              const uint32_t mask = border(i) ? 0xFFFFu : 0u;
              uint32_t bad = 0u;
#pragma unroll
              for (int k = 0; k < kPieces; ++k) {
                bad |= nonfinite_bf16x2(w[k].x) | nonfinite_bf16x2(w[k].y) |
                       nonfinite_bf16x2(w[k].z) | nonfinite_bf16x2(w[k].w);
                w[k] = make_uint4(finite_bf16x2(w[k].x, mask), finite_bf16x2(w[k].y, mask),
                                  finite_bf16x2(w[k].z, mask), finite_bf16x2(w[k].w, mask));
              }
              const bool any = __any_sync(0xffffffffu, bad != 0u);
              kind = any && mask == 0u ? kOddPage : kSplitPage;
              if (any && mask != 0u) taken_out();
            }
            if (i + Gm::kAux < count) next = id_of(i + Gm::kAux);
            // (and the page behind it to L2, for contexts that come out of memory)
            const int ahead = i + 2 * Gm::kAux;
            if (ahead < count) {
              const bool later = ((ahead ^ (ahead - Gm::kAux)) & 32) != 0;
              const int far = __shfl_sync(0xffffffffu, later ? pages.next : pages.ids, ahead & 31);
              prefetch_l2(page_at(far) + lane * (kPageBytes / 32 - 16));
            }
            const int nth = tiles + i / Gm::kPages, st = nth % Gm::kVStages;
            wait(&ms.v_empty[st], (static_cast<uint32_t>(nth / Gm::kVStages) & 1u) ^ 1u);
            if (!wait.all_ok()) break;
            const uint32_t to = mine + st * Gm::kTileBytes + i % Gm::kPages * (kBlockSize * 128);
            auto place = [&](int k) {
              return (to ^ ((k * kRows & 7) << 4)) + k * kRows * 128;
            };
            const uint8_t* const from = page_at(next);
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
              store16(place(k), w[k]);
              w[k] = load_once(from + k * 512);
            }
            if (lane == 0) ms.v_split[st][i % Gm::kPages] = static_cast<uint8_t>(kind);
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.v_full[st]);
          }
          tiles += count / Gm::kPages;
        }
        if (!wait.all_ok()) break;
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ms.unit_checked[ui & 1]);
          mbar_arrive(&ms.unit_empty[ui & 1]);
        }
      }
      wait.report();
    }
  } else {
    // ---------------------------------------------------------------- softmax
    regs_more<Gm::kSoftmaxRegs>();
    const int s = warp >> 2;
    const int r = threadIdx.x & 127;                    // row of the tile
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + s * kPromptTile, to = tmem + lanes + Gm::kO + s * D;
    const int tok = r / p.G, g = r - tok * p.G;         // of this row
    PromptWaits wait;                                   // lanes agree to go on where they vote
    // with starts out of order a search may miss sequences without meeting the wrong ones
    if (blockIdx.x == 0) {
      for (int b = threadIdx.x; b < p.num_seqs; b += Gm::kSoftmaxWarps * 32)
        if (__ldg(p.query_starts + b) > __ldg(p.query_starts + b + 1))
          atomicOr(&g_pa_err, kErrBounds);
      __syncwarp();
    }
    uint32_t n_s = 0, n_o = 0;                          // S and O tiles taken
    int v_first = 0;                                    // place of the unit's first V tile: stage,
                                                        //   kVStages more in odd phases
    for (int ui = 0; wait.ok(); ++ui) {
      wait(&ms.unit_full[ui & 1], static_cast<uint32_t>(ui >> 1) & 1u);
      if (!wait.all_ok()) break;
      const PromptUnit un = load_unit(ms.unit[ui & 1]);
      if (un.b < 0) break;
      const PromptSub sub = prompt_sub(p, un, s);
      const bool live = tok < sub.n;                    // rows past the tile's end repeat the last
      const int pos = sub.first + min(tok, max(sub.n, 1) - 1);
      float c = p.scale_log2;
      if constexpr (KV8) {
        wait(&ms.q_wide[ui & 1][s], static_cast<uint32_t>(ui >> 1) & 1u);
        const int e = ms.q_exp[ui & 1][s][live ? r : 0];
        c *= __ldg(p.k_scale + un.head) *
             __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      }
      int v_at = (v_first + sub.a - un.t0) % (2 * Gm::kVStages);
      v_first = (v_first + un.t1 - un.t0) % (2 * Gm::kVStages);
      float ref = -CUDART_INF_F;                        // reference, log2 units
      float sum = 0.f;
      bool steady = false;                              // a reference that may stay
      for (int t = sub.a; t < sub.e; ++t) {
        wait(&ms.s_full[s], n_s++ & 1u);
        __syncwarp();
        tc::fence_after_sync();
        const bool masked = prompt_masked(p, t, sub.first, sub.first + sub.n - 1);
        bool look = !steady;                            // for the maximum
        PromptScores sc;
        // whether V has pages that stay bf16, nearly always known by now
        uint32_t split = 0u;
        const int st = v_at < Gm::kVStages ? v_at : v_at - Gm::kVStages;
        if constexpr (!KV8)
          split = tc::mbar_test(&ms.v_full[st], v_at >= Gm::kVStages)
                      ? split_pages(smem_u32(ms.v_split[st])) : kSplitUnknown;
        while (true) {
          sc.load(ts);
          // A score's factor is applied with the reference's subtraction, in one rounding; with
          // a factor that is not positive, or references that leave no bits behind the point, it
          // comes first.
          float cc = c, m = 0.f;
          // (unlikely, so that the code of most tiles is in one piece)
          if (__builtin_expect(look || masked, 0)) {
            bool first = !(c > 0.f), border = masked;
            while (true) {
              if (first) {
                sc.multiply(cc);
                cc = 1.f;
              }
              if (border) {
                const int hi = pos - t * kPromptTile;   // columns lo < i <= hi are visible
                sc.mask(p.window > 0 ? hi - p.window : -1, hi);
                border = false;
              }
              if (!look) break;
              m = sc.largest() * cc;
              if (first || !__any_sync(0xffffffffu, fabsf(m) > kPromptExact &&
                                                        fabsf(m) < CUDART_INF_F))
                break;
              first = true;
            }
            // by 8 at least, unless weights went past their limit, or 2^(8 + kShift) would be
            // rounded past it; the first finite score always
            const bool exact = fabsf(ref) <= kPromptExact;
            const bool move = look && m > ref + (steady || !exact ? 0.f : 8.f);
            if (__any_sync(0xffffffffu, move)) {
              const float f = move ? fmaxf(hw_exp2(ref - m), kPromptFaint) : 1.f;
              ref = move ? m : ref;
              sum *= f;
              if (t > sub.a) {
#pragma unroll 1
                for (int i = 0; i < D / 16; ++i) {
                  uint32_t o[16];
                  tc::tmem_ld16(to + i * 16, o);
                  tc::tmem_wait_ld();
                  tmem_wait_regs(o);
#pragma unroll
                  for (int k = 0; k < 16; ++k)
                    o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                  tc::tmem_st16(to + i * 16, o);
                }
              }
            }
            if (look) steady = __all_sync(0xffffffffu, c > 0.f && fabsf(ref) <= kPromptExact);
          }
          const float off = ref == -CUDART_INF_F ? 0.f : Gm::kShift - ref;
          sc.begin(cc, off);
          // beside the first half of the weights the largest of the other half's scores, so that
          // nothing is left to look at behind the test
          float most[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
          sc.template weights<0, 32>([&](int k) {
            most[k & 3] = max3(most[k & 3], sc.score(64 + 2 * k), sc.score(65 + 2 * k));
          });
          m = fmaxf(max3(most[0], most[1], most[2]), most[3]);
          const bool fine = sc.most_of_eight() <= kPromptLimit && fmaf(m, cc, off) <= 15.f;
          if (look || __all_sync(0xffffffffu, fine)) break;
          look = true;
        }
        if (!KV8 && __builtin_expect(__any_sync(0xffffffffu, split != 0u), 0)) {
          if (split == kSplitUnknown) {
            wait(&ms.v_full[st], v_at >= Gm::kVStages);
            split = split_pages(smem_u32(ms.v_split[st]));
          }
          split = uniform(split);
        }
        v_at = v_at + 1 == 2 * Gm::kVStages ? 0 : v_at + 1;
        sc.finish(ts, &ms.p_half[s], lane == 0 && split == 0u);
        sum += sc.total();
        tc::tmem_wait_st();
        if (!KV8 && __builtin_expect(split != 0u, 0)) {
          split_weights(ts, split);
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms.p_half[s]);
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms.p_full[s]);
        if (!wait.all_ok()) break;
      }
      if (!wait.all_ok()) break;

      // -------------------------------------------------------------- unit output
      wait(&ms.unit_checked[ui & 1], static_cast<uint32_t>(ui >> 1) & 1u);
      const bool special = *reinterpret_cast<volatile int*>(&ms.unit[ui & 1].nonfinite) != 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms.unit_empty[ui & 1]);
      const bool any = sub.e > sub.a;
      if (any) wait(&ms.o_full[s], n_o++ & 1u);
      if (!wait.all_ok()) break;
      tc::fence_after_sync();
      float vs = 1.f;
      if constexpr (KV8) vs = __ldg(p.v_scale + un.head);
      // (a partition without a key of this row, or with scores of -inf alone, has no weights)
      const float inv = (sum == 0.f && un.parts > 1 ? 1.f : __frcp_rn(sum)) *
                        (1.f / (1 << Gm::kVShift));
      // Four lanes exchange 16-byte pieces of their rows, so that they write 64 bytes of one row
      // at a time: a store that touches 32 rows takes 32 cycles, and there is nothing beside it.
      const bool whole = un.parts == 1;
      const size_t row0 =
          static_cast<size_t>(un.row0 + s * p.sub_tokens) * p.Hq + un.head * p.G;
      const size_t stride = whole ? D * 2 : static_cast<size_t>(p.max_parts) * D * 4;
      uint8_t* const dst = whole ? static_cast<uint8_t*>(p.out) + row0 * stride
                                 : reinterpret_cast<uint8_t*>(p.part_o) + row0 * stride +
                                       un.part * (D * 4);
      int ln = lane, rel = live ? tok * p.Hq + g : -1;  // this row, from row0
      // (what follows from the two is not to be kept in registers over the tiles)
      asm volatile("" : "+r"(ln), "+r"(rel));
      auto put = [&](int piece, const uint32_t* x) {    // 64 bytes of every lane's row
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          v[k] = make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
        swap_pieces<1>(v[0], v[1], ln);
        swap_pieces<1>(v[2], v[3], ln);
        swap_pieces<2>(v[0], v[2], ln);
        swap_pieces<2>(v[1], v[3], ln);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int to_row = __shfl_sync(0xffffffffu, rel, (ln & 28) + k);
          if (to_row >= 0)
            *reinterpret_cast<uint4*>(dst + to_row * stride + piece * 64 + (ln & 3) * 16) = v[k];
        }
      };
#pragma unroll 1
      for (int i = 0; i < D / 64; ++i) {
        uint32_t o[2][32];
        if (any) {
          tc::tmem_ld32(to + i * 64, o[0]);
          tc::tmem_ld32(to + i * 64 + 32, o[1]);
          tc::tmem_wait_ld();
          tmem_wait_regs(o[0]);
          tmem_wait_regs(o[1]);
          if (i + 1 == D / 64) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.o_free[s]);
          }
#pragma unroll
          for (int k = 0; k < 64; k += 2) {
            uint32_t* x = &o[k / 32][k % 32];
            uint64_t y = mul_f32x2(pack_f32x2(__uint_as_float(x[0]), __uint_as_float(x[1])),
                                   pack_f32x2(inv, inv));
            if constexpr (KV8) y = mul_f32x2(y, pack_f32x2(vs, vs));
            x[0] = static_cast<uint32_t>(y);
            x[1] = static_cast<uint32_t>(y >> 32);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 64; ++k) o[k / 32][k % 32] = 0u;
        }
        if (whole) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              o[h][k] = pack_bf16x2_rn(__uint_as_float(o[h][2 * k]),
                                       __uint_as_float(o[h][2 * k + 1]));
            put(2 * i + h, o[h]);
          }
        } else {
#pragma unroll
          for (int h = 0; h < 4; ++h) put(4 * i + h, o[h / 2] + h % 2 * 16);
          if (i == 0 && live)
            p.part_ml[(row0 + rel) * p.max_parts + un.part] = make_float2(ref - Gm::kShift, sum);
        }
      }
      // the infinities and NaN that were taken out of V, for the rows that see them: a row at a
      // time, its dims over the lanes
      if (__builtin_expect(special && any, 0)) {
        __syncwarp();
        float add[D / 32];
        int seen = -1;                                  // token that they are of
        for (int rr = (warp & 3) * 32; rr < (warp & 3) * 32 + 32; ++rr) {
          const int tk = rr / p.G;
          if (tk >= sub.n) break;
          if (tk != seen) {
            seen = tk;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) add[k] = 0.f;
            const int at = sub.first + tk, begin = p.window > 0 ? at - p.window + 1 : 0;
            for (int t = sub.a; t < sub.e; ++t) {
              if (!prompt_masked(p, t, un.pos0, un.pos0 + un.ntok - 1)) continue;
              const int stop = min(at, t * kPromptTile + kPromptTile - 1);
#pragma unroll 4
              for (int j = max(t * kPromptTile, begin); j <= stop; ++j) {
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                  const float v = prompt_value<D, KV8>(p, un, j, k * 32 + lane);
                  add[k] += fabsf(v) < CUDART_INF_F ? 0.f : v;
                }
              }
            }
          }
          const size_t out_row = row0 + static_cast<size_t>(tk) * p.Hq + rr % p.G;
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            const int d = k * 32 + lane;
            if (fabsf(add[k]) == 0.f) continue;
            if (un.parts == 1) {
              __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + out_row * D + d;
              *dst = __float2bfloat16_rn(__bfloat162float(*dst) + add[k]);
            } else {
              p.part_o[(out_row * p.max_parts + un.part) * D + d] += add[k];
            }
          }
        }
      }
    }
    wait.report();
  }

  // ------------------------------------------------------------------ teardown
  tc::fence_before_sync();
  __syncthreads();
  if (warp == Gm::kSoftmaxWarps + 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, Gm::kTmemCols);
    tc::tmem_relinquish();
  }
}

// ---------------------------------------------------------------- merge of partitions
// One warp per query row of a pair of tiles whose keys were cut: partition i holds O_i
// (normalised), the reference m_i (log2 units) and the sum l_i, and counts w_i = l_i 2^(m_i - M).
// It waits for memory three times at least (unit, statistics, values), so the first sixteen
// partitions' values are asked for with the statistics, before their weights are known: 19
// partitions of 1056 rows 8.5 us out of DRAM, against 12.3 with eight after the weights.
constexpr int kPromptMergeWarps = 4, kPromptMergeParts = 16;

template <int D>
__global__ void __launch_bounds__(kPromptMergeWarps * 32) prompt_merge_kernel(const PromptParams p) {
  constexpr int DL = D / 32;
  using Vec = std::conditional_t<DL == 4, float4, float2>;
  PromptUnit un;
  bool bad;
  const bool some = prompt_unit(p, blockIdx.x, un, &bad) && un.parts > 1;
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.y * kPromptMergeWarps + (threadIdx.x >> 5);
  if (!some || r >= un.ntok * p.G) return;
  const size_t row = static_cast<size_t>(un.row0 + r / p.G) * p.Hq + un.head * p.G + r % p.G;
  const float2* ml = p.part_ml + row * p.max_parts;
  const Vec* src = reinterpret_cast<const Vec*>(p.part_o + row * p.max_parts * D) + lane;
  // a partition without weights counts nothing, unless a value was infinite or NaN
  float M = -CUDART_INF_F;
  float acc[DL] = {}, total = 0.f;
  for (int i0 = 0; i0 < un.parts; i0 += kPromptMergeParts) {
    Vec v[kPromptMergeParts];
#pragma unroll
    for (int k = 0; k < kPromptMergeParts; ++k)
      v[k] = i0 + k < un.parts ? __ldcg(src + static_cast<size_t>(i0 + k) * 32) : Vec{};
    if (i0 == 0) {
      for (int i = lane; i < un.parts; i += 32) {
        const float2 x = __ldcg(ml + i);
        M = fmaxf(M, x.y == 0.f ? -CUDART_INF_F : x.x);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    }
    float w = 0.f;                                      // of partition i0 + lane
    if (lane < kPromptMergeParts && i0 + lane < un.parts) {
      const float2 x = __ldcg(ml + i0 + lane);
      if (x.y != 0.f) w = fmaxf(x.y * hw_exp2(x.x - M), kPromptFaint);
    }
#pragma unroll
    for (int k = 0; k < kPromptMergeParts; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      total += wk;
      const float* f = reinterpret_cast<const float*>(&v[k]);
#pragma unroll
      for (int d = 0; d < DL; ++d) acc[d] += wk * f[d];
    }
  }
  const float inv = __frcp_rn(total);
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + row * D + lane * DL;
#pragma unroll
  for (int k = 0; k < DL; k += 2)
    *reinterpret_cast<uint32_t*>(dst + k) = pack_bf16x2_rn(acc[k] * inv, acc[k + 1] * inv);
}

template <int D, bool KV8>
cudaError_t launch_prompt_as(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const PromptParams& p, cudaStream_t s) {
  using Gm = PromptGeo<D, KV8>;
  auto kern = prompt_kernel<D, KV8>;
  static std::atomic<unsigned long long> configured{0ull};
  static std::atomic<int> sm_count[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
  int sms = bit ? sm_count[dev].load(std::memory_order_relaxed) : 0;
  if (bit == 0 || (configured.load(std::memory_order_acquire) & bit) == 0 || sms == 0) {
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, kern);
    if (e != cudaSuccess) return e;
    // the softmax warps take their registers from what the launch holds
    if (at.numRegs < Gm::kRegs) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Gm::kAlloc);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (bit) {
      sm_count[dev].store(sms, std::memory_order_relaxed);
      configured.fetch_or(bit, std::memory_order_acq_rel);
    }
  }
  const int pairs = p.num_slots * p.Hkv;
  if (p.counter != nullptr) {
    e = cudaMemsetAsync(p.counter, 0, sizeof(int), s);
    if (e != cudaSuccess) return e;
  }
  kern<<<static_cast<unsigned>(std::min(p.num_units, sms)), Gm::kThreads, Gm::kAlloc, s>>>(tq, tk, tv,
                                                                                        p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.max_parts == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pairs),
                     static_cast<unsigned>((2 * p.sub_tokens * p.G + kPromptMergeWarps - 1) /
                                           kPromptMergeWarps), 1);
  cfg.blockDim = dim3(kPromptMergeWarps * 32, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prompt_merge_kernel<D>, p);
}

}  // namespace pa
