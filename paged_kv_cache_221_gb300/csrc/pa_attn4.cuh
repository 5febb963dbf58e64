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
// Balanced mode (kFlat): the pages of all (sequence, kv head) pairs form one list, cut
// into equal runs, one for each worker that is resident at once, so that ragged
// contexts neither leave a tail nor a second wave.  Each pair counts kSetup pages more
// than it has, for what starting on it costs.  A pair that lies in one run is
// written out directly; the others leave (m, l, O) partials, at most two per worker
// (the run's first and last pair), which attn4_merge_kernel joins.
// Unit mode: a worker takes whole (partition, sequence, kv head) units of a fixed size;
// the split-KV merge joins the partitions.  The result of a sequence then does not
// depend on the batch it is in.
#pragma once

#include "pa_pages.cuh"

namespace pa {

// NT n-tiles of 8 query rows per warp, NTW row columns (each a worker's job of its own), TP
// pages per softmax step, STAGES staged steps per warp, MINB CTAs of 4 warps per SM.
template <int NT_, int NTW_, int TP_, int STAGES_, int MINB_>
struct Cfg4 {
  static constexpr int NT = NT_, NTW = NTW_, TP = TP_, STAGES = STAGES_, MINB = MINB_;
  static constexpr int kWarps = 4, kThreads = 32 * kWarps, kRows = 8 * NT;
  static constexpr bool kQRegs = NT <= 2;
  static_assert(32 % TP == 0, "a step's pages come from one batch of block ids");
};

template <int D, class C>
struct Smem4 {
  using P = Page<kPageInt4, D>;
  static constexpr int kPairBytes = 2 * P::kBytes;          // a K page, then its V page
  static constexpr int kStageBytes = C::TP * kPairBytes;
  static constexpr int kRingBytes = C::STAGES * kStageBytes;
  static constexpr int kQBytes = C::kQRegs ? 0 : C::NT * QTileSmem<kPageInt4, D>::kBytes;
  static constexpr int kWarpBytes = kRingBytes + kQBytes;
  static constexpr int kBytes = C::kWarps * kWarpBytes;
  static_assert(kStageBytes % 16 == 0 && kWarpBytes % 16 == 0, "16-byte copies");
};

// Pages that sequence b's query tokens can see (0 if its length is out of range).
__device__ __forceinline__ int visible_pages(const AttnParams& p, int L, int* first) {
  *first = 0;
  if (L < p.T || L > p.max_ctx) return 0;
  if (p.window > 0) *first = max(0, L - p.T - p.window + 1) / kBlockSize;
  return (L + kBlockSize - 1) / kBlockSize - *first;
}

// What starting on a pair costs, in pages: block ids, query rows and the first pages are
// fetched one after the other.
constexpr int kSetup = 3;

// List entries of a pair with nb pages: its setup, then its pages.
__device__ __forceinline__ int pair_entries(int nb) { return nb > 0 ? nb + kSetup : 0; }

// The list over all sequences (one head): the entries of all, and of those before sequence
// `upto`.  A warp; kKeep chunks of 32 lengths are in flight at once.
constexpr int kKeep = 8;
__device__ __forceinline__ void count_entries(const AttnParams& p, int lane, int upto, int& all,
                                              int& before) {
  all = before = 0;
  for (int base = 0; base < p.num_seqs; base += 32 * kKeep) {
    int L[kKeep];
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
      const int b = base + 32 * k + lane;
      L[k] = b < p.num_seqs ? p.context_lens[b] : p.T - 1;   // no pages
    }
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
      int first;
      const int n = pair_entries(visible_pages(p, L[k], &first));
      all += n;
      if (base + 32 * k + lane < upto) before += n;
    }
  }
  all = __reduce_add_sync(0xffffffffu, all);
  before = __reduce_add_sync(0xffffffffu, before);
}

// Entries per run: everything split evenly over the workers, but at least min_share.
__device__ __forceinline__ int run_entries(const Attn4Params& p, int total) {
  return max(p.min_share, (total + p.workers - 1) / p.workers);
}

// base + page * stride in one wide multiply-add.
__device__ __forceinline__ const uint8_t* at_page(const uint8_t* base, uint32_t page,
                                                  uint32_t stride) {
  const uint8_t* r;
  asm("mad.wide.u32 %0, %1, %2, %3;" : "=l"(r) : "r"(page), "r"(stride), "l"(base));
  return r;
}

template <int D, class C, bool kFlat>
__global__ void __launch_bounds__(C::kThreads, C::MINB) paged_attn4_kernel(const Attn4Params p) {
  using P = Page<kPageInt4, D>;
  using Sm = Smem4<D, C>;
  constexpr int NT = C::NT, NTW = C::NTW, TP = C::TP, S = C::STAGES;
  constexpr int NG = P::kGroups;
  extern __shared__ __align__(128) uint8_t smem_all[];
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, q4 = lane & 3;
  uint8_t* smem = smem_all + warp * Sm::kWarpBytes;
  const int G = p.G, T = p.T, nrows = G * T;
  const int heads = p.Hkv * NTW;             // jobs per sequence
  const int worker = blockIdx.x * C::kWarps + warp;

  // Per lane: its chunks within a page (chunk `lane` of K and of V, and one of the scale
  // chunks) and their place in a stage.
  const uint32_t page_stride = static_cast<uint32_t>(p.Hkv) * P::kBytes;
  constexpr int SC = P::kScales / 16;        // scale chunks of a page
  const uint32_t ring = smem_u32(smem);
  const uint32_t swz = page_swizzle<kPageInt4, D>(lane / P::kChunks, lane % P::kChunks);
  const uint32_t sdst = P::kCodes + 16 * (lane % SC) + (lane < SC ? 0 : P::kBytes);
  const uint32_t koff = ldsm_offset<kPageInt4, D>(lane);

  // ---------------------------------------------------------------- this worker's work
  // Flat: entries [f, f_end) of the list; b is found by adding up the sequences before it,
  // `entry` counts from the pair's first entry.
  // Units: u, u + workers, ...
  int f = 0, f_end = 0, f0 = 0;
  int b = 0, job = 0, entry = 0, nb = 0, first = 0, L = 0;
  if constexpr (kFlat) {
    // The first 32 * kKeep lengths stay in registers between the sum and the search.
    int len[kKeep], sum = 0;
    bool invalid = false;
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
      len[k] = 32 * k + lane < p.num_seqs ? p.context_lens[32 * k + lane] : -1;
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
      int skip;
      sum += pair_entries(visible_pages(p, len[k], &skip));
      invalid |= 32 * k + lane < p.num_seqs && (len[k] < T || len[k] > p.max_ctx);
    }
    for (int i = 32 * kKeep + lane; i < p.num_seqs; i += 32) {
      int skip;
      const int x = p.context_lens[i];
      sum += pair_entries(visible_pages(p, x, &skip));
      invalid |= x < T || x > p.max_ctx;
    }
    if (invalid && worker == 0) atomicOr(&g_pa_err, kErrBounds);
    const int total = __reduce_add_sync(0xffffffffu, sum) * heads;
    const int share = run_entries(p, total);
    if (static_cast<long long>(worker) * share >= total) return;
    f = f0 = worker * share;
    f_end = min(total, f + share);
    int before = 0;                          // entries of the sequences before b, all heads
    bool found = false;
    auto search = [&](int base, int Ll) {
      int fl, mine = visible_pages(p, Ll, &fl);
      int run = pair_entries(mine);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
      }
      const int upto = before + run * heads;
      const unsigned past = __ballot_sync(0xffffffffu, upto > f);
      before = __shfl_sync(0xffffffffu, upto, 31);
      if (past == 0) return;
      found = true;
      const int at = __ffs(past) - 1;
      b = base + at;
      nb = __shfl_sync(0xffffffffu, mine, at);
      first = __shfl_sync(0xffffffffu, fl, at);
      L = __shfl_sync(0xffffffffu, Ll, at);
      const int ne = pair_entries(nb);
      const int from = f - (__shfl_sync(0xffffffffu, upto, at) - ne * heads);
      job = from / ne;
      entry = from % ne;
    };
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
      if (!found && 32 * k < p.num_seqs) search(32 * k, len[k]);
    for (int base = 32 * kKeep; !found; base += 32)   // f < total: some chunk ends past it
      search(base, base + lane < p.num_seqs ? p.context_lens[base + lane] : -1);
  }
  long long u = worker;

  while (true) {
    int page, n, part = 0;                   // pages of this segment; its partition
    int taken = 0;                           // list entries of this segment
    bool direct;
    if constexpr (kFlat) {
      taken = min(pair_entries(nb) - entry, f_end - f);
      page = max(0, entry - kSetup);
      n = max(0, entry + taken - kSetup) - page;
      direct = n == nb;
    } else {
      const long long units = static_cast<long long>(p.max_parts) * heads * p.num_seqs;
      if (u >= units) return;
      // partition-major: every sequence's first partition, then every second one, ...
      part = static_cast<int>(u / (heads * p.num_seqs));
      b = static_cast<int>(u / heads % p.num_seqs);
      job = static_cast<int>(u % heads);
      u += p.workers;
      L = p.context_lens[b];
      nb = visible_pages(p, L, &first);
      if (nb == 0 && part == 0 && lane == 0) atomicOr(&g_pa_err, kErrBounds);
      page = part * p.ppb;
      n = min(p.ppb, nb - page);
      if (n <= 0) continue;
      direct = nb <= p.ppb;
    }
    if (n > 0) {
    const int g = job / NTW, row0 = (job % NTW) * C::kRows;
    const int pg0 = first + page;

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
#pragma unroll
        for (int k = 0; k < TP; ++k) {
          // a step past the last page stages page 0 of the pool, masked below
          const uint32_t phys = __shfl_sync(0xffffffffu, ids, (it + k) & 31);
          const uint8_t* kp = at_page(ksrc, phys, page_stride);
          const uint8_t* vp = at_page(vsrc, phys, page_stride);
          const uint32_t to = st_in + k * Sm::kPairBytes;
#pragma unroll
          for (int c = 0; c < P::kCodes / 512; ++c) {   // 8 (16) rows on: the same swizzle
            cp_async_16(to + swz + 512 * c, kp + 512 * c, 16);
            cp_async_16(to + swz + P::kBytes + 512 * c, vp + 512 * c, 16);
          }
          if (lane < 2 * SC) cp_async_16(to + sdst, at_page(ssrc, phys, page_stride), 16);
        }
        it += TP;
        st_in = st_in + Sm::kStageBytes == ring + Sm::kRingBytes ? ring : st_in + Sm::kStageBytes;
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue();

    QOperand<kPageInt4, D, NT, C::kQRegs> qo;
    {
      const float k_scale = p.k_scale[g];
      uint8_t* qt = smem + Sm::kRingBytes;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if constexpr (C::kQRegs) {
          make_q_tile(qo.tile[j], raw[j], p.scale_log2, k_scale, lane);
          qo.rs0[j] = qo.tile[j].rs0;
          qo.rs1[j] = qo.tile[j].rs1;
        } else {
          QTile<kPageInt4, D> tile;
          make_q_tile(tile, raw[j], p.scale_log2, k_scale, lane);
          put_q_tile(qt + j * QTileSmem<kPageInt4, D>::kBytes, tile, lane);
          qo.rs0[j] = tile.rs0;
          qo.rs1[j] = tile.rs1;
        }
      }
      if constexpr (!C::kQRegs) qo.base = qt + lane * 8;   // each lane reads what it wrote
    }

    // Softmax state of rows 2q4, 2q4 + 1 of each n-tile: minus the reference m (log2
    // domain) and, in units of the raw scores, the value a score must pass to move m
    // (minus infinity until a score was seen).
    // z: rows 0 .. NG - 1 hold the groups' sums of weight * scale (what the codes' offset
    // adds to the output), rows 8 .. 15 the sum of the weights.
    float acc[NT][D / 16][4], z[NT][4], nm0[NT], nm1[NT], thr0[NT], thr1[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      nm0[j] = nm1[j] = 0.f;
      thr0[j] = thr1[j] = -CUDART_INF_F;
#pragma unroll
      for (int e = 0; e < 4; ++e) z[j][e] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][k][e] = 0.f;
    }
    // byte pair (token 2q, token 2q+1) of group gid % NG from two words of scales
    const uint32_t zsel = (gid & (NG - 1)) | ((gid & (NG - 1)) + 4) << 4;
    constexpr uint32_t kOnes = 0x3C003C00u;

    // Pages wholly visible to every row: first entry in [lo, hi]
    const int part_end = min(L, (pg0 + n) * kBlockSize);
    const int hi = min(L - T, part_end - 1) - (kBlockSize - 1);
    const int lo = max(0, L - p.wspan);
    int tok0 = pg0 * kBlockSize;
    uint32_t st = ring;

    for (int i = 0; i * TP < n; ++i) {
      cp_async_wait<S - 2>();
      __syncwarp();
      issue();                               // into the stage consumed last
      float t[TP][NT][4];
#pragma unroll
      for (int k = 0; k < TP; ++k)
        page_scores<kPageInt4, D>(t[k], st + k * Sm::kPairBytes, koff, qo, lane);

      const bool edge = tok0 < lo || tok0 + (TP - 1) * kBlockSize > hi || (bad | bad_before) != 0;
      // The end of page k's entries: none of a page that was not in the pool.  The batch of
      // ids that page i0 came from is the newest one unless `it` has passed on.
      auto end_of = [&](int k) {
        const int i0 = i * TP + k;
        const unsigned bits = (it - 1) >> 5 == i0 >> 5 ? bad : bad_before;
        return (bits >> (i0 & 31)) & 1u ? 0 : part_end;
      };
      if (edge) {
#pragma unroll
        for (int k = 0; k < TP; ++k) {
          const int end = end_of(k);
          const int j0 = tok0 + k * kBlockSize + gid, j1 = j0 + 8;
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const int r = row0 + 8 * j + 2 * q4;
            const int a = r < nrows ? L - T + r / G : L - 1;
            const int c = r + 1 < nrows ? L - T + (r + 1) / G : L - 1;
            const unsigned w = p.wcap;
            if (j0 >= end || static_cast<unsigned>(a - j0) >= w) t[k][j][0] = -CUDART_INF_F;
            if (j0 >= end || static_cast<unsigned>(c - j0) >= w) t[k][j][1] = -CUDART_INF_F;
            if (j1 >= end || static_cast<unsigned>(a - j1) >= w) t[k][j][2] = -CUDART_INF_F;
            if (j1 >= end || static_cast<unsigned>(c - j1) >= w) t[k][j][3] = -CUDART_INF_F;
          }
        }
      }

      // Online softmax: the reference m of a row moves only when a score passes it by
      // 7, so a weight is at most 2^7 and, times a V scale (at most 448), an f16 value.
      bool over = false;
      float x0[NT], x1[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        x0[j] = fmaxf(t[0][j][0], t[0][j][2]);
        x1[j] = fmaxf(t[0][j][1], t[0][j][3]);
#pragma unroll
        for (int k = 1; k < TP; ++k) {
          x0[j] = fmaxf(x0[j], fmaxf(t[k][j][0], t[k][j][2]));
          x1[j] = fmaxf(x1[j], fmaxf(t[k][j][1], t[k][j][3]));
        }
        over |= x0[j] > thr0[j] || x1[j] > thr1[j];
      }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            x0[j] = fmaxf(x0[j], __shfl_xor_sync(0xffffffffu, x0[j], o));
            x1[j] = fmaxf(x1[j], __shfl_xor_sync(0xffffffffu, x1[j], o));
          }
          float f0 = 1.f, f1 = 1.f;
          if (x0[j] > thr0[j]) {
            const float nm = -x0[j] * qo.rs0[j];
            f0 = thr0[j] == -CUDART_INF_F ? 0.f : hw_exp2(nm - nm0[j]);
            nm0[j] = nm;
            thr0[j] = x0[j] + 7.f / qo.rs0[j];
          }
          if (x1[j] > thr1[j]) {
            const float nm = -x1[j] * qo.rs1[j];
            f1 = thr1[j] == -CUDART_INF_F ? 0.f : hw_exp2(nm - nm1[j]);
            nm1[j] = nm;
            thr1[j] = x1[j] + 7.f / qo.rs1[j];
          }
          z[j][0] *= f0;
          z[j][1] *= f1;
          z[j][2] *= f0;
          z[j][3] *= f1;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            acc[j][k][0] *= f0;
            acc[j][k][1] *= f1;
            acc[j][k][2] *= f0;
            acc[j][k][3] *= f1;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < TP; ++k) {
        uint32_t ph0[NT], ph1[NT];             // P^T: tokens 2q, 2q+1 and 2q+8, 2q+9 of row gid
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const float p0 = hw_exp2(fmaf(t[k][j][0], qo.rs0[j], nm0[j]));
          const float p1 = hw_exp2(fmaf(t[k][j][1], qo.rs1[j], nm1[j]));
          const float p2 = hw_exp2(fmaf(t[k][j][2], qo.rs0[j], nm0[j]));
          const float p3 = hw_exp2(fmaf(t[k][j][3], qo.rs1[j], nm1[j]));
          ph0[j] = transpose_8x8(half2_bits(__floats2half2_rn(p0, p1)));
          ph1[j] = transpose_8x8(half2_bits(__floats2half2_rn(p2, p3)));
        }

        // V scales of tokens 2q, 2q+1 (w0, w1) and 2q+8, 2q+9 (w2, w3), a byte per group
        const uint32_t vp = st + k * Sm::kPairBytes + P::kBytes;
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
        if (edge) {                            // rows past the context may hold any scale, even NaN
          const int nv = end_of(k) - (tok0 + k * kBlockSize);
          w0 = 2 * q4 < nv ? w0 : 0u;
          w1 = 2 * q4 + 1 < nv ? w1 : 0u;
          w2 = 2 * q4 + 8 < nv ? w2 : 0u;
          w3 = 2 * q4 + 9 < nv ? w3 : 0u;
        }
        {
          uint32_t za, zb, none;
          e4m3x4_to_f16x4(__byte_perm(w0, w1, zsel), za, none);
          e4m3x4_to_f16x4(__byte_perm(w2, w3, zsel), zb, none);
#pragma unroll
          for (int j = 0; j < NT; ++j) mma_f16(z[j], za, kOnes, zb, kOnes, ph0[j], ph1[j]);
        }
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
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              const uint32_t b0 = f16x2_mul(ph0[j], fa), b1 = f16x2_mul(ph1[j], fb);
              // dims 32 gr + 4 gid + 0 and 2, then + 1 and 3 (times 16)
              mma_f16(acc[j][2 * gr], y0 & kNibLo, u0 & kNibLo, y1 & kNibLo, u1 & kNibLo, b0,
                            b1);
              mma_f16(acc[j][2 * gr + 1], y0 & kNibHi, u0 & kNibHi, y1 & kNibHi, u1 & kNibHi,
                            b0, b1);
            }
          }
        }
      }
      tok0 += TP * kBlockSize;
      st = st + Sm::kStageBytes == ring + Sm::kRingBytes ? ring : st + Sm::kStageBytes;
    }
    cp_async_wait<0>();
    __syncwarp();

    // -------------------------------------------------------------- result
    const float out_scale = p.v_scale[g];
    const size_t slot = kFlat ? static_cast<size_t>(worker) * 2 + (f == f0 ? 0 : 1) : 0;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float zz[2][NG];
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        zz[0][gr] = 8.f * __shfl_sync(0xffffffffu, z[j][0], gr * 4 + q4);
        zz[1][gr] = 8.f * __shfl_sync(0xffffffffu, z[j][1], gr * 4 + q4);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {          // rows 2q4 and 2q4 + 1
        const int r = row0 + 8 * j + 2 * q4 + h;
        if (r >= nrows) continue;
        const float l = z[j][2 + h];
        const bool none = (h ? thr1[j] : thr0[j]) == -CUDART_INF_F;
        const float inv = l > 0.f ? out_scale / l : 0.f;
        const size_t orow = (static_cast<size_t>(b) * T + r / G) * p.Hq + g * G + r % G;
        float* po = nullptr;
        if (!direct) {
          const size_t at = kFlat ? slot * C::kRows + (r - row0) : orow * p.max_parts + part;
          po = p.part_o + at * D;
          if (gid == 0)
            p.part_ml[at] = make_float2(none ? -CUDART_INF_F : -(h ? nm1[j] : nm0[j]), l);
        }
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          constexpr float A = 16777216.f, B = 1048576.f;   // 2^24, 2^20
          const float* a = acc[j][2 * gr] + h;
          const float* c = acc[j][2 * gr + 1] + h;
          const float z8 = zz[h][gr];
          const float4 o = make_float4(fmaf(a[0], A, -z8) * inv, fmaf(c[0], B, -z8) * inv,
                                       fmaf(a[2], A, -z8) * inv, fmaf(c[2], B, -z8) * inv);
          const int d = 32 * gr + 4 * gid;
          if (direct)
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + orow * D + d) =
                make_uint2(bf162_bits(__floats2bfloat162_rn(o.x, o.y)),
                           bf162_bits(__floats2bfloat162_rn(o.z, o.w)));
          else
            *reinterpret_cast<float4*>(po + d) = o;
        }
      }
    }

    }                                        // n > 0
    if constexpr (kFlat) {
      f += taken;
      if (f >= f_end) return;
      entry = 0;                             // the run goes on with the next pair
      if (++job == heads) {
        job = 0;
        do {
          L = p.context_lens[++b];
          nb = visible_pages(p, L, &first);
        } while (nb == 0);                   // f < total: a later sequence has pages
      }
    }
  }
}

// ---------------------------------------------------------------- merge of the runs
// One CTA of W warps per (job, query row).  Partial i of the job comes from worker w0 + i;
// warp k takes partials k, k + W, ...
template <int D, int W>
__global__ void __launch_bounds__(32 * W) attn4_merge_kernel(const Attn4Params p, int ntw,
                                                             int tile_rows, int live) {
  constexpr int DL = D / 32;
  __shared__ float s_acc[W][D];
  __shared__ float s_ml[W][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int heads = p.Hkv * ntw;
  const int r = static_cast<int>(blockIdx.x % live);
  const int job = static_cast<int>(blockIdx.x / live % heads);
  const int b = static_cast<int>(blockIdx.x / live / heads);
  const int row = job % ntw * tile_rows + r;
  int first, before, all;
  const int mine = p.context_lens[b];
  count_entries(p, lane, b, all, before);
  const int nb = visible_pages(p, mine, &first);
  const int share = run_entries(p, all * heads);
  const int ne = pair_entries(nb);
  const int f0 = before * heads + job * ne;
  // the workers of its first and its last page
  const int w0 = (f0 + kSetup) / share, w1 = (f0 + ne - 1) / share;
  // every CTA waits, so that this grid does not complete before the one it follows
  grid_dependency_wait();
  if (nb == 0 || w0 == w1 || row >= p.G * p.T) return;
  const int parts = w1 - w0 + 1;
  auto slot = [&](int i) {
    const bool second = i == 0 && f0 > w0 * share;       // the run's last pair, not its first
    return (static_cast<size_t>(w0 + i) * 2 + (second ? 1 : 0)) * tile_rows + r;
  };
  float M = -CUDART_INF_F, S = 0.f, acc[DL];
#pragma unroll
  for (int k = 0; k < DL; ++k) acc[k] = 0.f;
  for (int i = warp + W * lane; i < parts; i += 32 * W) M = fmaxf(M, p.part_ml[slot(i)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float u = M == -CUDART_INF_F ? 0.f : M;
#pragma unroll 4
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
  static_assert(tile.nt == C::NT && tile.ntw == C::NTW && tile.ctas == C::MINB, "the host's tile");
  const long long jobs = static_cast<long long>(p.num_seqs) * p.Hkv * C::NTW;
  auto fn = p.flat ? paged_attn4_kernel<D, C, true> : paged_attn4_kernel<D, C, false>;
  const cudaError_t e =
      cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>((p.workers + C::kWarps - 1) / C::kWarps);
  fn<<<grid, C::kThreads, bytes, s>>>(p);
  cudaError_t r = cudaGetLastError();
  if (r != cudaSuccess || !p.flat) return r;
  // the merge starts during the attention kernel's last wave
  cudaLaunchConfig_t cfg = {};
  const int live = std::min(C::kRows, p.G * p.T);   // rows of a tile that are used
  cfg.gridDim = dim3(static_cast<unsigned>(jobs * live), 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // more warps per row when a job has many runs
  if (p.workers >= 16 * jobs) {
    cfg.blockDim = dim3(256, 1, 1);
    return cudaLaunchKernelEx(&cfg, attn4_merge_kernel<D, 8>, p, C::NTW, C::kRows, live);
  }
  cfg.blockDim = dim3(32, 1, 1);
  return cudaLaunchKernelEx(&cfg, attn4_merge_kernel<D, 1>, p, C::NTW, C::kRows, live);
}

template <int D>
cudaError_t launch_attn4(const Attn4Params& p, int rows, cudaStream_t s) {
  if (rows <= 8) return launch_cfg4<D, Cfg4<1, 1, 2, 3, 4>>(p, s);
  if (rows <= 16) return launch_cfg4<D, Cfg4<2, 1, 1, 6, 2>>(p, s);
  if (rows <= 24) return launch_cfg4<D, Cfg4<3, 1, 1, 6, 2>>(p, s);
  if (rows <= 32) return launch_cfg4<D, Cfg4<4, 1, 1, 6, 2>>(p, s);
  return launch_cfg4<D, Cfg4<4, 2, 1, 6, 2>>(p, s);
}

}  // namespace pa
