// Eviction by accumulated attention weight (pa_evict_tokens), and the second launch
// of pa_accumulate_weights.
#include <algorithm>

#include "pa_runs.cuh"

namespace pa {

// ---------------------------------------------------------------- weights
// A CTA takes 1024 entries of one (sequence, kv head), four per thread: first every row's
// final (m, l) from the pieces of its job (a warp per row), then the sum over the rows, 16
// bytes of every row's scores per load.
constexpr int kSumThreads = 256, kSumEntries = 4 * kSumThreads;

__global__ void __launch_bounds__(kSumThreads) observe_sum_kernel(const ObserveParams p) {
  __shared__ float s_m[kMaxRows], s_f[kMaxRows];
  const int b = blockIdx.y / p.Hkv, g = blockIdx.y % p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const RunList list = observe_list(p, p.ntw);
  const int L = p.context_lens[b], T = p.T, nrows = p.G * p.T;
  const int e0 = blockIdx.x * kSumEntries;
  int first;
  const int nb = visible_pages(list, L, first);
  const bool work = nb > 0 && e0 < L;
  Pieces pc[2];                              // of the row columns
  if (work) {
    for (int c = 0; c < p.ntw; ++c) {
      if (p.flat)
        pc[c] = find_pieces(list, b, g * p.ntw + c, nb, lane);
      else
        pc[c] = Pieces{0, (nb + p.ppb - 1) / p.ppb, false};
    }
  }
  grid_dependency_wait();
  if (!work) return;
  for (int r = warp; r < nrows; r += kSumThreads / 32) {
    const int c = r / p.tile_rows, rl = r % p.tile_rows;
    const Pieces& x = c == 0 ? pc[0] : pc[1];
    const size_t unit0 = (static_cast<size_t>(b) * list.heads + g * p.ntw + c) * p.max_parts;
    float M = -CUDART_INF_F, l = 0.f;
    for (int i = lane; i < x.count; i += 32) {
      const float2 ml = p.ml[(p.flat ? x.slot(i) : unit0 + i) * p.tile_rows + rl];
      const float m = fmaxf(M, ml.x), u = m == -CUDART_INF_F ? 0.f : m;
      l = l * hw_exp2(M - u) + ml.y * hw_exp2(ml.x - u);
      M = m;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float a = __shfl_xor_sync(0xffffffffu, M, o), y = __shfl_xor_sync(0xffffffffu, l, o);
      const float m = fmaxf(M, a), u = m == -CUDART_INF_F ? 0.f : m;
      l = l * hw_exp2(M - u) + y * hw_exp2(a - u);
      M = m;
    }
    if (lane == 0) {
      s_m[r] = M == -CUDART_INF_F ? 0.f : M;
      s_f[r] = l > 0.f ? 1.f / l : 0.f;
    }
  }
  __syncthreads();
  const int j0 = e0 + 4 * threadIdx.x;
  if (j0 >= L) return;
  const size_t bg = static_cast<size_t>(b) * p.Hkv + g;
  const float* t = p.scores + bg * nrows * p.max_entries + j0;
  float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int r = 0; r < nrows; ++r) {
    const float4 x = *reinterpret_cast<const float4*>(t + static_cast<size_t>(r) * p.max_entries);
    const float m = s_m[r], f = s_f[r];
    w[0] = fmaf(hw_exp2(x.x - m), f, w[0]);
    w[1] = fmaf(hw_exp2(x.y - m), f, w[1]);
    w[2] = fmaf(hw_exp2(x.z - m), f, w[2]);
    w[3] = fmaf(hw_exp2(x.w - m), f, w[3]);
  }
  const size_t at = bg * p.weight_entries + j0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int j = j0 + e;
    if (j >= L) break;
    const bool fresh = j >= L - T;
    p.weights_out[at + e] = fresh ? w[e] : fmaf(p.decay, p.weights[at + e], w[e]);
    if (fresh && p.positions != nullptr)
      p.positions[at + e] = (p.seq_lens != nullptr ? p.seq_lens[b] : L) - L + j;
  }
}

cudaError_t launch_observe_sum(const ObserveParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.max_ctx + kSumEntries - 1) / kSumEntries),
                     static_cast<unsigned>(p.num_seqs * p.Hkv), 1);
  cfg.blockDim = dim3(kSumThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, observe_sum_kernel, p);
}

// ---------------------------------------------------------------- selection
// One CTA per (sequence, kv head).  The entries to keep are the `budget` first in the
// order (newest num_recent first, larger weight, lower index).  Either all protected
// (newest) entries stay and the threshold lies among the others, or it lies among the
// protected ones; a radix selection over the weights' order-preserving bits finds it
// in four passes, and a scan in index order settles ties, numbers the dropped
// entries below `budget` (the gaps) and the kept ones from `budget` on (the movers),
// and writes pair i = (i-th mover, i-th gap).
constexpr int kSelThreads = 512;

// Larger for larger weights; -0 equals +0; NaN is below every number.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sums of up to three small counts over the CTA, with the totals.
struct Count3 {
  int a, b, c;
};
__device__ __forceinline__ Count3 scan3(Count3 x, Count3& total, int3* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Count3 v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, v.a, o), b = __shfl_up_sync(0xffffffffu, v.b, o);
    const int c = __shfl_up_sync(0xffffffffu, v.c, o);
    if (lane >= o) {
      v.a += a;
      v.b += b;
      v.c += c;
    }
  }
  if (lane == 31) sh[warp] = make_int3(v.a, v.b, v.c);
  __syncthreads();
  Count3 before{0, 0, 0};
  total = Count3{0, 0, 0};
  for (int w = 0; w < kSelThreads / 32; ++w) {
    const int3 y = sh[w];
    if (w < warp) {
      before.a += y.x;
      before.b += y.y;
      before.c += y.z;
    }
    total.a += y.x;
    total.b += y.y;
    total.c += y.z;
  }
  __syncthreads();
  return Count3{before.a + v.a - x.a, before.b + v.b - x.b, before.c + v.c - x.c};
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  __shared__ int s_hist[256];
  __shared__ int3 s_scan[kSelThreads / 32];
  __shared__ int s_newest, s_protected, s_bad, s_digit, s_left;
  grid_launch_dependents();
  const int b = blockIdx.x / p.Hkv, g = blockIdx.x % p.Hkv;
  const int tid = threadIdx.x;
  const int L = p.context_lens[b];
  int* count = p.counts + blockIdx.x;
  if (L < 0 || L > p.max_ctx) {
    if (tid == 0) {
      *count = 0;
      if (g == 0) {
        p.new_lens[b] = L;
        atomicOr(&g_pa_err, kErrBounds);
      }
    }
    return;
  }
  if (L <= p.budget) {
    if (tid == 0) {
      *count = 0;
      if (g == 0) p.new_lens[b] = L;
    }
    return;
  }
  const size_t row = (static_cast<size_t>(b) * p.Hkv + g) * p.weight_entries;
  const float* w = p.weights + row;
  const int* pos = p.positions + row;
  if (tid == 0) {
    s_newest = -0x7fffffff - 1;
    s_protected = 0;
    s_bad = 0;
  }
  __syncthreads();
  // a block outside the pool: the sequence is left as it is (every head sees the same table)
  const int nblk = (L + kBlockSize - 1) / kBlockSize;
  for (int i = tid; i < nblk; i += kSelThreads)
    if (static_cast<unsigned>(p.block_tables[static_cast<size_t>(b) * p.mbs + i]) >=
        static_cast<unsigned>(p.num_blocks))
      s_bad = 1;
  int newest = -0x7fffffff - 1;
  for (int j = tid; j < L; j += kSelThreads) newest = max(newest, pos[j]);
  newest = __reduce_max_sync(0xffffffffu, newest);
  if ((tid & 31) == 0) atomicMax(&s_newest, newest);
  __syncthreads();
  if (s_bad) {
    if (tid == 0) {
      *count = 0;
      if (g == 0) {
        p.new_lens[b] = L;
        atomicOr(&g_pa_err, kErrBounds);
      }
    }
    return;
  }
  const long long bar = static_cast<long long>(s_newest) - p.num_recent;   // protected: pos > bar
  int mine = 0;
  for (int j = tid; j < L; j += kSelThreads) mine += pos[j] > bar ? 1 : 0;
  mine = __reduce_add_sync(0xffffffffu, mine);
  if ((tid & 31) == 0) atomicAdd(&s_protected, mine);
  __syncthreads();
  const bool among = s_protected >= p.budget;      // the threshold lies among the protected
  int k = among ? p.budget : p.budget - s_protected;   // entries of that class to keep

  // k-th largest key of the class, a byte at a time
  uint32_t prefix = 0, mask = 0;
  for (int shift = 24; shift >= 0 && k > 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelThreads) s_hist[i] = 0;
    __syncthreads();
    for (int j = tid; j < L; j += kSelThreads) {
      if ((pos[j] > bar) != among) continue;
      const uint32_t key = weight_key(w[j]);
      if ((key & mask) == prefix) atomicAdd(&s_hist[(key >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int left = k, d = 255;
      while (d > 0 && s_hist[d] < left) left -= s_hist[d--];
      s_digit = d;
      s_left = left;
    }
    __syncthreads();
    k = s_left;
    prefix |= static_cast<uint32_t>(s_digit) << shift;
    mask |= 255u << shift;
    __syncthreads();
  }
  // of the class: every key above `prefix` stays, and the first k that equal it (k = 0: none)
  const bool none = (among ? p.budget : p.budget - s_protected) == 0;

  int2* moves = p.moves + static_cast<size_t>(blockIdx.x) * p.max_moves;
  int ties = 0, gaps = 0, movers = 0;
  for (int j0 = 0; j0 < L; j0 += kSelThreads) {
    const int j = j0 + tid;
    bool keep = false, tie = false;
    if (j < L) {
      const bool prot = pos[j] > bar;
      if (prot != among) {
        keep = prot;                         // protected, or below a class that fills the budget
      } else if (!none) {
        const uint32_t key = weight_key(w[j]);
        keep = key > prefix;
        tie = key == prefix;
      }
    }
    Count3 total;
    const Count3 at = scan3(Count3{tie ? 1 : 0, 0, 0}, total, s_scan);
    if (tie && ties + at.a < k) keep = true;
    ties += total.a;
    const bool gap = j < L && !keep && j < p.budget, mover = keep && j >= p.budget;
    const Count3 to = scan3(Count3{0, gap ? 1 : 0, mover ? 1 : 0}, total, s_scan);
    if (gap) moves[gaps + to.b].y = j;
    if (mover) moves[movers + to.c].x = j;
    gaps += total.b;
    movers += total.c;
  }
  if (tid == 0) {
    *count = movers;
    if (g == 0) p.new_lens[b] = p.budget;
  }
}

// ---------------------------------------------------------------- moves
// A warp copies one entry at a time: its K and V rows, weight and position.  Gaps lie
// below `budget` and movers at or above it, so no copy reads what another writes.
constexpr int kMoveThreads = 256;

template <int F, int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
  using P = Page<F, D>;
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  const int bg = blockIdx.y;
  const int b = bg / p.Hkv, g = bg % p.Hkv;
  const int n = p.counts[bg];
  const int stride = gridDim.x * (kMoveThreads / 32);
  const int32_t* trow = p.block_tables + static_cast<size_t>(b) * p.mbs;
  uint8_t* kp = static_cast<uint8_t*>(p.k_pool);
  uint8_t* vp = static_cast<uint8_t*>(p.v_pool);
  for (int i = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5); i < n; i += stride) {
    const int2 mv = p.moves[static_cast<size_t>(bg) * p.max_moves + i];
    const size_t sp = (static_cast<size_t>(trow[mv.x / kBlockSize]) * p.Hkv + g) * P::kBytes;
    const size_t dp = (static_cast<size_t>(trow[mv.y / kBlockSize]) * p.Hkv + g) * P::kBytes;
    const int ts = mv.x % kBlockSize, td = mv.y % kBlockSize;
    if constexpr (F == kPageFp8) {
      for (int c = lane; c < P::kChunks; c += 32)
        reinterpret_cast<uint4*>(kp + dp + td * P::kRow)[c] =
            reinterpret_cast<const uint4*>(kp + sp + ts * P::kRow)[c];
      for (int d = lane; d < D; d += 32)     // V pages are transposed: a byte per dim
        vp[dp + d * kBlockSize + td] = vp[sp + d * kBlockSize + ts];
    } else {
      for (int c = lane; c < 2 * P::kChunks; c += 32) {
        uint8_t* pool = c < P::kChunks ? kp : vp;
        const int cc = c < P::kChunks ? c : c - P::kChunks;
        reinterpret_cast<uint4*>(pool + dp + td * P::kRow)[cc] =
            reinterpret_cast<const uint4*>(pool + sp + ts * P::kRow)[cc];
      }
      if constexpr (F == kPageInt4) {
        if (lane >= 32 - 2 * P::kGroups) {
          const int c = lane - (32 - 2 * P::kGroups);
          uint8_t* pool = c < P::kGroups ? kp : vp;
          const int cc = c < P::kGroups ? c : c - P::kGroups;
          pool[dp + P::kCodes + td * P::kGroups + cc] = pool[sp + P::kCodes + ts * P::kGroups + cc];
        }
      }
    }
    if (lane == 0) {
      const size_t row = static_cast<size_t>(bg) * p.weight_entries;
      p.weights[row + mv.y] = p.weights[row + mv.x];
      p.positions[row + mv.y] = p.positions[row + mv.x];
    }
  }
}

cudaError_t launch_evict(const EvictParams& p, int format, int head_dim, cudaStream_t s) {
  const int pairs = p.num_seqs * p.Hkv;
  evict_select_kernel<<<pairs, kSelThreads, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // about 8 CTAs per SM in all, at most one warp per move
  const int want = std::max(1, 8 * 152 / pairs);
  const int most = (p.max_moves + kMoveThreads / 32 - 1) / (kMoveThreads / 32);
  dim3 grid(static_cast<unsigned>(std::min(want, most)), static_cast<unsigned>(pairs));
  auto go = [&](auto fn) { fn<<<grid, kMoveThreads, 0, s>>>(p); };
  if (format == kPageBf16)
    head_dim == 64 ? go(evict_move_kernel<kPageBf16, 64>) : go(evict_move_kernel<kPageBf16, 128>);
  else if (format == kPageFp8)
    head_dim == 64 ? go(evict_move_kernel<kPageFp8, 64>) : go(evict_move_kernel<kPageFp8, 128>);
  else
    head_dim == 64 ? go(evict_move_kernel<kPageInt4, 64>) : go(evict_move_kernel<kPageInt4, 128>);
  return cudaGetLastError();
}

cudaError_t take_error_evict(unsigned* bits) { return read_error_word(bits); }

}  // namespace pa
