// Eviction by accumulated attention weight (pa_evict_tokens), and the second launch
// of pa_accumulate_weights.
#include <algorithm>

#include "pa_runs.cuh"

namespace pa {

// ---------------------------------------------------------------- weights
// A CTA joins the (m, l) of one (sequence, kv head)'s rows from the pieces of its job (a warp
// per row) and then takes every gridDim.x-th tile of 512 entries, four per thread: each
// thread copies its 16 bytes of every row's scores to shared memory, all rows in flight at
// once, and sums over them.  Twice as many CTAs as are resident at once: the jobs' lengths
// differ, and what a CTA does before its first tile costs (a call with 1 / 2 / 4 times as many:
// 115.2 / 113.3 / 117.4 us).  Bound by the scores' bytes on
// their way out of L2 and back: 189 MB of 20 rows (32 sequences of 2048-16384 tokens) take 37
// us; a second buffer per CTA (half the CTAs) took 8 us more, refilling each quarter of the
// rows as it is read 6.
constexpr int kSumThreads = 128, kSumEntries = 4 * kSumThreads;
constexpr int kSumRowBytes = kSumEntries * 4;

__global__ void __launch_bounds__(kSumThreads) observe_sum_kernel(const ObserveParams p) {
  __shared__ float s_m[kMaxRows], s_f[kMaxRows];
  __shared__ int s_undefined;                // a row's softmax is NaN
  extern __shared__ __align__(16) float s_scores[];   // [row][thread][4]
  const int b = blockIdx.y / p.Hkv, g = blockIdx.y % p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const RunList list = observe_list(p, p.ntw);
  const int L = p.context_lens[b], T = p.T, nrows = p.G * p.T;
  int first;
  const int nb = visible_pages(list, L, first);
  const bool work = nb > 0 && static_cast<int>(blockIdx.x) * kSumEntries < L;
  __shared__ Pieces pc[2];                   // of the row columns, a warp each
  if (work && warp < p.ntw) {
    Pieces x{0, (nb + p.ppb - 1) / p.ppb, false};
    if (p.flat) x = find_pieces(list, b, g * p.ntw + warp, nb, lane);
    if (lane == 0) pc[warp] = x;
  }
  grid_dependency_wait();
  if (!work) return;
  const size_t bg = static_cast<size_t>(b) * p.Hkv + g;
  const float* scores = p.scores + bg * nrows * p.max_entries + 4 * threadIdx.x;
  const uint32_t mine_at = smem_u32(s_scores) + 16 * threadIdx.x;
  const int stride = gridDim.x * kSumEntries;
  const uint64_t policy = read_policy(true);
  auto fetch = [&](int e0) {
    const bool mine = e0 + 4 * static_cast<int>(threadIdx.x) < L;
    for (int r = 0; mine && r < nrows; ++r)
      cp_async_16_hint(mine_at + r * kSumRowBytes,
                       scores + static_cast<size_t>(r) * p.max_entries + e0, policy);
    cp_async_commit();
  };
  int e0 = blockIdx.x * kSumEntries;
  fetch(e0);
  if (threadIdx.x == 0) s_undefined = 0;
  __syncthreads();
  for (int r = warp; r < nrows; r += kSumThreads / 32) {
    const int c = r / p.tile_rows, rl = r % p.tile_rows;
    const Pieces y = pc[c];
    const size_t job_slot = static_cast<size_t>(b) * list.heads + g * p.ntw + c;
    const bool whole = y.count == 1;
    float M = -CUDART_INF_F, l = 0.f;
    for (int i = lane; i < y.count; i += 32) {
      const size_t at = !p.flat ? job_slot * p.max_parts + i
                        : whole ? static_cast<size_t>(p.workers) * 2 + job_slot
                                : y.slot(i);
      const float2 ml = p.ml[at * p.tile_rows + rl];
      const float m = fmaxf(M, ml.x), u = m == -CUDART_INF_F ? 0.f : m;
      l = l * hw_exp2(M - u) + ml.y * hw_exp2(ml.x - u);
      M = m;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float a = __shfl_xor_sync(0xffffffffu, M, o), z = __shfl_xor_sync(0xffffffffu, l, o);
      const float m = fmaxf(M, a), u = m == -CUDART_INF_F ? 0.f : m;
      l = l * hw_exp2(M - u) + z * hw_exp2(a - u);
      M = m;
    }
    if (lane == 0) {
      // l is NaN behind a score of NaN or +inf, and 0 without a finite one
      s_m[r] = M == -CUDART_INF_F ? 0.f : M;
      s_f[r] = l > 0.f ? 1.f / l : CUDART_NAN_F;
      if (!(l > 0.f)) s_undefined = 1;
    }
  }
  __syncthreads();
  for (; e0 < L; e0 += stride) {
    const int j0 = e0 + 4 * threadIdx.x;
    const size_t at = bg * p.weight_entries + j0;
    float old[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) old[e] = j0 + e < L - T ? p.weights[at + e] : 0.f;
    cp_async_wait<0>();
    float w[4] = {0.f, 0.f, 0.f, 0.f};
    const float4* x4 = reinterpret_cast<const float4*>(s_scores);   // this thread's own copies
    if (!s_undefined) {
#pragma unroll 4
      for (int r = 0; r < nrows; ++r) {
        const float4 x = x4[r * kSumThreads + threadIdx.x];
        const float m = s_m[r], f = s_f[r];
        w[0] = fmaf(hw_exp2(x.x - m), f, w[0]);
        w[1] = fmaf(hw_exp2(x.y - m), f, w[1]);
        w[2] = fmaf(hw_exp2(x.z - m), f, w[2]);
        w[3] = fmaf(hw_exp2(x.w - m), f, w[3]);
      }
    } else if (j0 < L && static_cast<unsigned>(
                             p.block_tables[static_cast<size_t>(b) * p.mbs + j0 / kBlockSize]) <
                             static_cast<unsigned>(p.num_blocks)) {
      // a row adds to the entries that it sees alone (a NaN factor would reach the others): not to
      // later drafts, nor to entries of a block outside the pool
      for (int r = 0; r < nrows; ++r) {
        const float4 x = x4[r * kSumThreads + threadIdx.x];
        const float m = s_m[r], f = s_f[r], t[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j0 + e <= L - T + r / p.G) w[e] = fmaf(hw_exp2(t[e] - m), f, w[e]);
      }
    }
    if (e0 + stride < L) fetch(e0 + stride);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = j0 + e;
      if (j >= L) break;
      const bool fresh = j >= L - T;
      p.weights_out[at + e] = fresh ? w[e] : fmaf(p.decay, old[e], w[e]);
      if (fresh && p.positions != nullptr)
        p.positions[at + e] = (p.seq_lens != nullptr ? p.seq_lens[b] : L) - L + j;
    }
  }
}

cudaError_t launch_observe_sum(const ObserveParams& p, cudaStream_t s) {
  constexpr int kMost = kMaxRows * kSumRowBytes;
  const int pairs = p.num_seqs * p.Hkv, bytes = p.G * p.T * kSumRowBytes;
  const int resident = std::min(2048 / kSumThreads, 200 * 1024 / bytes);
  const int tiles = (p.max_ctx + kSumEntries - 1) / kSumEntries;
  const int wanted = (2 * kAttn4Sms * resident + pairs - 1) / pairs;
  const cudaError_t e = allow_smem<observe_sum_kernel>(kMost);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(std::max(1, std::min(tiles, wanted))),
                  static_cast<unsigned>(pairs));
  return launch_behind(observe_sum_kernel, grid, kSumThreads, bytes, s, true, p);
}

// ---------------------------------------------------------------- selection
// One CTA per (sequence, kv head).  The entries to keep are the `budget` first in the
// order (newest num_recent first, larger weight, lower index).  Either all protected
// (newest) entries stay and the threshold lies among the others, or it lies among the
// protected ones; a radix selection over the weights' order-preserving bits finds it
// in four passes.  Weights and positions are read once: a warp owns a run of consecutive
// entries and keeps them in registers; past 16384 entries keys and protected bits stay in
// shared memory, and what does not fit there is read again at every pass.  A ballot per 32
// entries and one exchange between the warps settle which ties stay (the lowest indices), a
// second exchange numbers the dropped entries below `budget` (the gaps) and the kept ones from
// `budget` on (the movers), and pair i becomes (i-th mover, i-th gap).  Bound by instructions
// and barriers: 16 rows x 8 heads of 4096-8192 entries, the whole eviction 55.0 us with the keys
// in shared memory (8 M instructions, most of them re-deriving what a register holds), 50.0 so.

// Up to this many dropped entries are found one after the other (a decode step drops one per new
// token).  64 x 8 rows of 2048 + n entries, the whole call: n = 1 / 4 / 8: 7.4 / 9.7 / 13.2 us,
// 18.7 by the radix passes (n = 12); 6000 + n entries: 13.2 / 17.1 / 23.0 and 38.4 us.
constexpr int kFewDropped = 8;

// Larger for larger weights; -0 equals +0; NaN is below every number.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix over the CTA's warps of two counts each warp holds, and the totals.
template <int W>
__device__ __forceinline__ int2 over_warps(int2 mine, int2& total, int2* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) sh[warp] = mine;
  __syncthreads();
  int2 v = lane < W ? sh[lane] : make_int2(0, 0);
  const int2 own = v;
#pragma unroll
  for (int o = 1; o < W; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, v.x, o), c = __shfl_up_sync(0xffffffffu, v.y, o);
    if (lane >= o) {
      v.x += a;
      v.y += c;
    }
  }
  total = make_int2(__shfl_sync(0xffffffffu, v.x, W - 1), __shfl_sync(0xffffffffu, v.y, W - 1));
  const int x = __shfl_sync(0xffffffffu, v.x - own.x, warp);
  const int y = __shfl_sync(0xffffffffu, v.y - own.y, warp);
  __syncthreads();
  return make_int2(x, y);
}

// One entry to its new place, a warp: its K and V rows, weight and position.  For the few moves
// of a decode step, which the selecting CTA makes itself (the bounded decode step 87.2 -> 85.9 us
// on the GPU and a launch less on the host).
__device__ __forceinline__ void move_entry(const EvictParams& p, int b, int g, int2 mv, size_t row,
                                           int lane) {
  const int D = p.head_dim;
  const int bytes = p.format == kPageBf16 ? 2 * D : p.format == kPageFp8 ? D : D / 2;
  const int groups = p.format == kPageInt4 ? D / 32 : 0;
  const int page = kBlockSize * (bytes + groups), ts = mv.x % kBlockSize, td = mv.y % kBlockSize;
  const int32_t* trow = p.block_tables + static_cast<size_t>(b) * p.mbs;
  const size_t from = (static_cast<size_t>(trow[mv.x / kBlockSize]) * p.Hkv + g) * page;
  const size_t to = (static_cast<size_t>(trow[mv.y / kBlockSize]) * p.Hkv + g) * page;
  uint8_t* kp = static_cast<uint8_t*>(p.k_pool);
  uint8_t* vp = static_cast<uint8_t*>(p.v_pool);
  const bool by_dim = p.format == kPageFp8;  // V pages are transposed
  for (int c = lane; c < (by_dim ? 1 : 2) * bytes / 16; c += 32) {
    uint8_t* pool = 16 * c < bytes ? kp : vp;
    const int at = 16 * c % bytes;
    *reinterpret_cast<uint4*>(pool + to + td * bytes + at) =
        *reinterpret_cast<const uint4*>(pool + from + ts * bytes + at);
  }
  for (int i = lane; by_dim && i < D; i += 32)
    vp[to + i * kBlockSize + td] = vp[from + i * kBlockSize + ts];
  if (lane < 2 * groups) {
    uint8_t* pool = lane < groups ? kp : vp;
    const int at = kBlockSize * bytes + lane % groups;
    pool[to + at + td * groups] = pool[from + at + ts * groups];
  }
  if (lane == 0) {
    p.weights[row + mv.y] = p.weights[row + mv.x];
    p.positions[row + mv.y] = p.positions[row + mv.x];
  }
}

// Sequences with nothing to drop, and lengths out of range, which are reported.
__device__ __forceinline__ bool left_alone(const EvictParams& p, int b, int g, int L) {
  const bool invalid = L < 0 || L > p.max_ctx;
  if (!invalid && L > p.budget) return false;
  if (threadIdx.x == 0) {
    p.counts[blockIdx.x] = 0;
    if (g == 0) {
      p.new_lens[b] = L;
      if (invalid) atomicOr(&g_pa_err, kErrBounds);
    }
  }
  return true;
}

// A block outside the pool: the sequence is left as it is (every head sees the same table).
__device__ __forceinline__ bool bad_block(const EvictParams& p, int b, int L, int threads) {
  bool bad = false;
  for (int i = threadIdx.x; i < (L + kBlockSize - 1) / kBlockSize; i += threads)
    bad |= static_cast<unsigned>(p.block_tables[static_cast<size_t>(b) * p.mbs + i]) >=
           static_cast<unsigned>(p.num_blocks);
  return bad;
}

__device__ __forceinline__ void leave_bad(const EvictParams& p, int b, int g, int L) {
  if (threadIdx.x != 0) return;
  p.counts[blockIdx.x] = 0;
  if (g == 0) {
    p.new_lens[b] = L;
    atomicOr(&g_pa_err, kErrBounds);
  }
}

// The digit at which a class's keys from the top reach k, and how many of that digit are among
// the k: from the counts of 256 digits.  A warp.
__device__ __forceinline__ void find_digit(const int* hist, int k, int lane, int& digit, int& left) {
  // bins 255 - 8 lane .. 248 - 8 lane
  int h[8], sum = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h[i] = hist[255 - 8 * lane - i];
    sum += h[i];
  }
  int above = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, above, o);
    if (lane >= o) above += a;
  }
  above -= sum;
  const bool here = above < k && above + sum >= k;
  int d = -1, l = k - above;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (d < 0 && h[i] >= l) d = 255 - 8 * lane - i;
    if (d < 0) l -= h[i];
  }
  const int at = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
  digit = __shfl_sync(0xffffffffu, d, at);
  left = __shfl_sync(0xffffffffu, l, at);
}

// The moves of a few dropped entries (lane i holds the i-th, -1 from `drop` on), in rising order
// of both their ends: the dropped ones below `budget` are the gaps, the kept ones from it on the
// movers.  Their number.
__device__ __forceinline__ int pair_few(int gone, int drop, int budget, int2* to, int lane) {
  const bool gap = gone >= 0 && gone < budget;
  bool mover = lane < drop;
  int before = 0;
  for (int i = 0; i < drop; ++i) {
    const int x = __shfl_sync(0xffffffffu, gone, i);
    before += x < gone;                      // all dropped entries below a gap are gaps
    if (x == budget + lane) mover = false;
  }
  const unsigned mb = __ballot_sync(0xffffffffu, mover);
  if (gap) to[before].y = gone;
  if (mover) to[__popc(mb & ((1u << lane) - 1u))].x = budget + lane;
  return __popc(mb);
}

// Up to E entries per thread, in registers: a warp owns up to 32 E consecutive ones.
template <int W, int E>
__global__ void __launch_bounds__(32 * W) evict_select_kernel(const EvictParams p) {
  constexpr int kThreads = 32 * W;
  static_assert(W >= kFewDropped, "a warp per move");
  __shared__ int s_hist[4][256];
  __shared__ int2 s_warp[W];
  __shared__ long long s_low[2][W];
  __shared__ int s_newest, s_protected, s_bad, s_count;
  grid_launch_dependents();
  const int b = blockIdx.x / p.Hkv, g = blockIdx.x % p.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int L = p.context_lens[b];
  if (left_alone(p, b, g, L)) return;
  const size_t row = (static_cast<size_t>(b) * p.Hkv + g) * p.weight_entries;
  const int per_warp = ((L + 31) / 32 + W - 1) / W;          // words of 32 entries, at most E
  const int j0 = 32 * warp * per_warp + lane;
  if (tid == 0) {
    s_newest = -0x7fffffff - 1;
    s_protected = s_bad = 0;
  }
  for (int i = tid; i < 4 * 256; i += kThreads) s_hist[i >> 8][i & 255] = 0;
  uint32_t key[E];
  int pos[E], newest = -0x7fffffff - 1;
  unsigned live = 0;                         // bit k: entry j0 + 32 k
#pragma unroll
  for (int k = 0; k < E; ++k) {
    const int j = j0 + 32 * k;
    const bool mine = k < per_warp && j < L;
    pos[k] = mine ? p.positions[row + j] : -0x7fffffff - 1;
    key[k] = mine ? __float_as_uint(p.weights[row + j]) : 0u;
    live |= mine ? 1u << k : 0u;
  }
  const bool bad = bad_block(p, b, L, kThreads);
  __syncthreads();
  if (bad) s_bad = 1;
#pragma unroll
  for (int k = 0; k < E; ++k) {
    newest = max(newest, pos[k]);
    key[k] = weight_key(__uint_as_float(key[k]));
  }
  newest = __reduce_max_sync(0xffffffffu, newest);
  if (lane == 0) atomicMax(&s_newest, newest);
  __syncthreads();
  if (s_bad) {
    leave_bad(p, b, g, L);
    return;
  }
  const long long bar = static_cast<long long>(s_newest) - p.num_recent;   // protected: pos > bar
  unsigned prot = 0;
#pragma unroll
  for (int k = 0; k < E; ++k) prot |= pos[k] > bar ? 1u << k : 0u;
  prot &= live;
  int2* moves = p.moves + static_cast<size_t>(blockIdx.x) * p.max_moves;

  const int drop = L - p.budget;
  if (drop <= kFewDropped) {
    // entry j as a number: the smallest ones go, an unprotected one before a protected one, then
    // the smaller weight, then the higher index
    long long low;                           // this thread's smallest one
    auto scan = [&]() {
      low = 0x7fffffffffffffffll;
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const long long x = static_cast<long long>(
            (static_cast<unsigned long long>((prot >> k) & 1u) << 62) |
            (static_cast<unsigned long long>(key[k]) << 30) |
            static_cast<unsigned>(0x3fffffff - j0 - 32 * k));
        if ((live >> k) & 1u) low = min(low, x);
      }
    };
    int gone = -1;                           // lane i: the i-th dropped entry
    scan();
    for (int i = 0; i < drop; ++i) {
      long long all = low;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) all = min(all, __shfl_xor_sync(0xffffffffu, all, o));
      if (lane == 0) s_low[i & 1][warp] = all;
      __syncthreads();
      all = s_low[i & 1][lane % W];
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) all = min(all, __shfl_xor_sync(0xffffffffu, all, o));
      const int j = 0x3fffffff - static_cast<int>(all & 0x3fffffff);
      if (low == all && i + 1 < drop) {
        live &= ~(1u << ((j - j0) / 32));
        scan();
      }
      if (lane == i) gone = j;
    }
    if (warp == 0) {
      const int n = pair_few(gone, drop, p.budget, p.move_here ? s_warp : moves, lane);
      if (lane == 0) {
        p.counts[blockIdx.x] = s_count = n;
        if (g == 0) p.new_lens[b] = p.budget;
      }
    }
    if (!p.move_here) return;
    __syncthreads();
    if (warp < s_count) move_entry(p, b, g, s_warp[warp], row, lane);
    return;
  }

  const int protects = __reduce_add_sync(0xffffffffu, __popc(prot));
  if (lane == 0 && protects > 0) atomicAdd(&s_protected, protects);
  __syncthreads();
  const bool among = s_protected >= p.budget;      // the threshold lies among the protected
  int left = among ? p.budget : p.budget - s_protected;   // entries of that class to keep
  const unsigned same = among ? prot : live & ~prot;      // the class
  unsigned tie = left == 0 ? 0u : same;      // of the class, equal to the threshold so far
  uint32_t threshold = 0;
  for (int pass = 0; pass < 4 && left > 0; ++pass) {
    const int shift = 24 - 8 * pass;
#pragma unroll
    for (int k = 0; k < E; ++k)
      if ((tie >> k) & 1u) atomicAdd(&s_hist[pass][(key[k] >> shift) & 255u], 1);
    __syncthreads();
    int digit;
    find_digit(s_hist[pass], left, lane, digit, left);
    threshold |= static_cast<uint32_t>(digit) << shift;
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (((key[k] >> shift) & 255u) != static_cast<uint32_t>(digit)) tie &= ~(1u << k);
  }
  // protected entries stay unless they are the class; of the class every key above the threshold
  // stays, and the first `left` that equal it
  unsigned keep = prot & ~same;
  if (left > 0) {
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (key[k] > threshold) keep |= same & (1u << k);
  }
  int2 total;
  int seen = over_warps<W>(make_int2(__reduce_add_sync(0xffffffffu, __popc(tie)), 0), total, s_warp).x;
  const unsigned below = (1u << lane) - 1u;
#pragma unroll
  for (int k = 0; k < E; ++k) {
    const unsigned tb = __ballot_sync(0xffffffffu, (tie >> k) & 1u);
    if (((tie >> k) & 1u) && seen + __popc(tb & below) < left) keep |= 1u << k;
    seen += __popc(tb);
  }
  unsigned low = 0;                          // entries below `budget`
#pragma unroll
  for (int k = 0; k < E; ++k) low |= j0 + 32 * k < p.budget ? 1u << k : 0u;
  const unsigned gap = live & ~keep & low, mover = keep & ~low;
  int2 at = over_warps<W>(make_int2(__reduce_add_sync(0xffffffffu, __popc(gap)),
                                    __reduce_add_sync(0xffffffffu, __popc(mover))),
                          total, s_warp);
#pragma unroll
  for (int k = 0; k < E; ++k) {
    const bool is_gap = (gap >> k) & 1u, is_mover = (mover >> k) & 1u;
    const unsigned gb = __ballot_sync(0xffffffffu, is_gap), mb = __ballot_sync(0xffffffffu, is_mover);
    if (is_gap) moves[at.x + __popc(gb & below)].y = j0 + 32 * k;
    if (is_mover) moves[at.y + __popc(mb & below)].x = j0 + 32 * k;
    at.x += __popc(gb);
    at.y += __popc(mb);
  }
  if (tid == 0) {
    p.counts[blockIdx.x] = total.y;
    if (g == 0) p.new_lens[b] = p.budget;
  }
}

// Longer contexts.  kStaged: keys and protected bits in shared memory.
template <int W, bool kStaged>
__global__ void __launch_bounds__(32 * W) evict_select_long_kernel(const EvictParams p) {
  constexpr int kThreads = 32 * W;
  extern __shared__ uint32_t s_dyn[];        // staged: protected bits, then keys
  __shared__ int s_hist[256];
  __shared__ int2 s_warp[W];
  __shared__ long long s_low[2][W];
  __shared__ int s_newest, s_protected, s_bad, s_digit, s_left;
  grid_launch_dependents();
  const int b = blockIdx.x / p.Hkv, g = blockIdx.x % p.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int L = p.context_lens[b];
  int* count = p.counts + blockIdx.x;
  if (left_alone(p, b, g, L)) return;
  const size_t row = (static_cast<size_t>(b) * p.Hkv + g) * p.weight_entries;
  const float* w = p.weights + row;
  const int* pos = p.positions + row;
  const int words = (L + 31) / 32;
  uint32_t* s_prot = s_dyn;
  uint32_t* s_key = s_dyn + (p.max_ctx + 31) / 32;
  if (tid == 0) {
    s_newest = -0x7fffffff - 1;
    s_protected = 0;
    s_bad = 0;
  }
  __syncthreads();
  if (bad_block(p, b, L, kThreads)) s_bad = 1;
  int newest = -0x7fffffff - 1;
#pragma unroll 4
  for (int j = tid; j < L; j += kThreads) {
    newest = max(newest, pos[j]);
    if constexpr (kStaged) s_key[j] = weight_key(w[j]);
  }
  newest = __reduce_max_sync(0xffffffffu, newest);
  if (lane == 0) atomicMax(&s_newest, newest);
  __syncthreads();
  if (s_bad) {
    leave_bad(p, b, g, L);
    return;
  }
  const long long bar = static_cast<long long>(s_newest) - p.num_recent;   // protected: pos > bar
  int mine = 0;
#pragma unroll 4
  for (int i = warp; i < words; i += W) {
    const int j = 32 * i + lane;
    const uint32_t bits = __ballot_sync(0xffffffffu, j < L && pos[j] > bar);
    if constexpr (kStaged) {
      if (lane == 0) s_prot[i] = bits;
    }
    mine += __popc(bits);
  }
  if (lane == 0 && mine > 0) atomicAdd(&s_protected, mine);
  __syncthreads();
  auto is_protected = [&](int j) {
    if constexpr (kStaged) return ((s_prot[j >> 5] >> (j & 31)) & 1u) != 0u;
    return pos[j] > bar;
  };
  auto key_of = [&](int j) {
    if constexpr (kStaged) return s_key[j];
    return weight_key(w[j]);
  };
  int2* moves = p.moves + static_cast<size_t>(blockIdx.x) * p.max_moves;

  const int drop = L - p.budget;
  if (drop <= kFewDropped && L < (1 << 30)) {
    // entry j as a number: the smallest ones go, an unprotected one before a protected one, then
    // the smaller weight, then the higher index
    constexpr long long kNone = 0x7fffffffffffffffll;
    long long low = kNone, last = -1;        // this thread's smallest one above `last`
    auto scan = [&]() {
      low = kNone;
#pragma unroll 4
      for (int j = tid; j < L; j += kThreads) {
        const long long x = static_cast<long long>(
            (is_protected(j) ? 1ull << 62 : 0ull) |
            (static_cast<unsigned long long>(key_of(j)) << 30) |
            static_cast<unsigned>(0x3fffffff - j));
        if (x > last) low = min(low, x);
      }
    };
    int gone = -1;                           // lane i: the i-th dropped entry
    scan();
    for (int i = 0; i < drop; ++i) {
      long long all = low;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) all = min(all, __shfl_xor_sync(0xffffffffu, all, o));
      if (lane == 0) s_low[i & 1][warp] = all;
      __syncthreads();
      all = s_low[i & 1][lane % W];
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) all = min(all, __shfl_xor_sync(0xffffffffu, all, o));
      last = all;
      if (low == last && i + 1 < drop) scan();
      if (lane == i) gone = 0x3fffffff - static_cast<int>(last & 0x3fffffff);
    }
    if (warp == 0) {
      const int n = pair_few(gone, drop, p.budget, p.move_here ? s_warp : moves, lane);
      if (lane == 0) {
        *count = s_left = n;
        if (g == 0) p.new_lens[b] = p.budget;
      }
    }
    if (!p.move_here) return;
    __syncthreads();
    if (warp < s_left) move_entry(p, b, g, s_warp[warp], row, lane);
    return;
  }

  const bool among = s_protected >= p.budget;      // the threshold lies among the protected
  int k = among ? p.budget : p.budget - s_protected;   // entries of that class to keep
  const bool none = k == 0;
  // k-th largest key of the class, a byte at a time
  uint32_t prefix = 0, mask = 0;
  for (int shift = 24; shift >= 0 && !none; shift -= 8) {
    for (int i = tid; i < 256; i += kThreads) s_hist[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (int j = tid; j < L; j += kThreads) {
      const uint32_t key = key_of(j);
      if (is_protected(j) == among && (key & mask) == prefix)
        atomicAdd(&s_hist[(key >> shift) & 255], 1);
    }
    __syncthreads();
    if (warp == 0) {
      int digit, left;
      find_digit(s_hist, k, lane, digit, left);
      if (lane == 0) {
        s_digit = digit;
        s_left = left;
      }
    }
    __syncthreads();
    k = s_left;
    prefix |= static_cast<uint32_t>(s_digit) << shift;
    mask |= 255u << shift;
  }
  // of the class: every key above `prefix` stays, and the first k that equal it
  const int per_warp = (words + W - 1) / W;
  const int i0 = min(words, warp * per_warp), i1 = min(words, i0 + per_warp);
  auto look = [&](int i, bool& keep, bool& tie) {
    const int j = 32 * i + lane;
    keep = tie = false;
    if (j >= L) return;
    const bool prot = is_protected(j);
    if (prot != among) {
      keep = prot;                           // protected, or below a class that fills the budget
    } else if (!none) {
      const uint32_t key = key_of(j);
      keep = key > prefix;
      tie = key == prefix;
    }
  };
  int ties = 0;
#pragma unroll 4
  for (int i = i0; i < i1; ++i) {
    bool keep, tie;
    look(i, keep, tie);
    ties += __popc(__ballot_sync(0xffffffffu, tie));
  }
  int2 total;
  const int ties_before = over_warps<W>(make_int2(ties, 0), total, s_warp).x;
  const unsigned below = (1u << lane) - 1u;
  int2 at = make_int2(0, 0);                 // gaps and movers before this warp's run
  for (int pass = 0; pass < 2; ++pass) {
    int seen = ties_before, gaps = 0, movers = 0;
#pragma unroll 4
    for (int i = i0; i < i1; ++i) {
      const int j = 32 * i + lane;
      bool keep, tie;
      look(i, keep, tie);
      const unsigned tb = __ballot_sync(0xffffffffu, tie);
      if (tie && seen + __popc(tb & below) < k) keep = true;
      seen += __popc(tb);
      const bool gap = j < L && !keep && j < p.budget, mover = keep && j >= p.budget;
      const unsigned gb = __ballot_sync(0xffffffffu, gap), mb = __ballot_sync(0xffffffffu, mover);
      if (pass == 1) {
        if (gap) moves[at.x + gaps + __popc(gb & below)].y = j;
        if (mover) moves[at.y + movers + __popc(mb & below)].x = j;
      }
      gaps += __popc(gb);
      movers += __popc(mb);
    }
    if (pass == 0) at = over_warps<W>(make_int2(gaps, movers), total, s_warp);
  }
  if (tid == 0) {
    *count = total.y;
    if (g == 0) p.new_lens[b] = p.budget;
  }
}

// ---------------------------------------------------------------- moves
// A warp copies kBatch entries at a time, all loads of a batch in flight before its first
// store: their K and V rows, weights and positions.  16 prompts of 4096-8192 tokens cut to 2048
// entries: 183 MB of bf16 rows in and out in 30 us (6.1 TB/s; 48 us with one move in flight).
// Gaps lie below `budget` and movers at or
// above it, so no copy reads what another writes.
constexpr int kMoveThreads = 128, kBatch = 4;

template <int F, int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p) {
  using P = Page<F, D>;
  // 16-byte chunks of a K and a V row; for FP8 the K row and, a byte per dim, the V row
  constexpr int kVec = F == kPageFp8 ? P::kChunks : 2 * P::kChunks;
  static_assert(kVec <= 32, "one chunk per lane");
  constexpr int kBytes = F == kPageFp8 ? D : (F == kPageInt4 ? 2 * P::kGroups : 0);
  constexpr int kB = (kBytes + 31) / 32;     // single bytes per lane
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  const int bg = blockIdx.y;
  const int b = bg / p.Hkv, g = bg % p.Hkv;
  const int n = p.counts[bg];
  const int stride = gridDim.x * (kMoveThreads / 32) * kBatch;
  const int32_t* trow = p.block_tables + static_cast<size_t>(b) * p.mbs;
  uint8_t* kp = static_cast<uint8_t*>(p.k_pool);
  uint8_t* vp = static_cast<uint8_t*>(p.v_pool);
  const size_t row = static_cast<size_t>(bg) * p.weight_entries;
  uint8_t* vpool = F != kPageFp8 && lane >= P::kChunks ? vp : kp;   // of this lane's chunk
  const int vchunk = 16 * (lane % P::kChunks);
  // byte i of an entry at token t of a page
  auto byte_at = [&](int i, size_t page, int t) -> uint8_t* {
    if constexpr (F == kPageFp8)
      return vp + page + i * kBlockSize + t;  // V pages are transposed
    else
      return (i < P::kGroups ? kp : vp) + page + P::kCodes + t * P::kGroups + i % P::kGroups;
  };
  for (int i = (blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5)) * kBatch; i < n;
       i += stride) {
    size_t sp[kBatch], dp[kBatch];
    int2 mv[kBatch];
    uint4 v[kBatch];
    uint8_t x[kBatch][kB > 0 ? kB : 1];
    float w[kBatch];
    int32_t ps[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e)
      mv[e] = p.moves[static_cast<size_t>(bg) * p.max_moves + min(i + e, n - 1)];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      sp[e] = (static_cast<size_t>(trow[mv[e].x / kBlockSize]) * p.Hkv + g) * P::kBytes;
      dp[e] = (static_cast<size_t>(trow[mv[e].y / kBlockSize]) * p.Hkv + g) * P::kBytes;
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int t = mv[e].x % kBlockSize;
      if (lane < kVec) v[e] = *reinterpret_cast<const uint4*>(vpool + sp[e] + t * P::kRow + vchunk);
#pragma unroll
      for (int c = 0; c < kB; ++c)
        if (lane + 32 * c < kBytes) x[e][c] = *byte_at(lane + 32 * c, sp[e], t);
      w[e] = p.weights[row + mv[e].x];
      ps[e] = p.positions[row + mv[e].x];
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      if (i + e >= n) break;
      const int t = mv[e].y % kBlockSize;
      if (lane < kVec) *reinterpret_cast<uint4*>(vpool + dp[e] + t * P::kRow + vchunk) = v[e];
#pragma unroll
      for (int c = 0; c < kB; ++c)
        if (lane + 32 * c < kBytes) *byte_at(lane + 32 * c, dp[e], t) = x[e][c];
      if (lane == 0) {
        p.weights[row + mv[e].y] = w[e];
        p.positions[row + mv[e].y] = ps[e];
      }
    }
  }
}

namespace {

cudaError_t launch_select(const EvictParams& p, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(p.num_seqs * p.Hkv);
  auto go = [&](auto fn, int warps, size_t bytes) {
    return launch_behind(fn, dim3(grid), 32 * warps, bytes, s, false, p);
  };
  // 16 entries per thread rather than 8 (twice the CTAs of half the warps per SM): 64 x 8 rows of
  // 2049 entries 9.3 -> 7.4 us, of 6001 18.5 -> 13.2; 32 entries gain no more
  if (p.max_ctx <= 4096) return go(evict_select_kernel<8, 16>, 8, 0);
  if (p.max_ctx <= 8192) return go(evict_select_kernel<16, 16>, 16, 0);
  if (p.max_ctx <= 16384) return go(evict_select_kernel<32, 16>, 32, 0);
  // keys and protected bits of the longest context, if they fit
  const size_t bytes = (static_cast<size_t>(p.max_ctx) + (p.max_ctx + 31) / 32) * 4;
  if (bytes > 200 * 1024) return go(evict_select_long_kernel<32, false>, 32, 0);
  const cudaError_t e = allow_smem<evict_select_long_kernel<32, true>>(200 * 1024);
  if (e != cudaSuccess) return e;
  return go(evict_select_long_kernel<32, true>, 32, bytes);
}

}  // namespace

cudaError_t launch_evict(const EvictParams& params, int format, int head_dim, cudaStream_t s) {
  EvictParams p = params;
  p.format = format;
  p.head_dim = head_dim;
  p.move_here = p.max_ctx - p.budget <= kFewDropped && p.max_ctx < (1 << 30);
  const int pairs = p.num_seqs * p.Hkv;
  const cudaError_t e = launch_select(p, s);
  if (e != cudaSuccess || p.move_here) return e;
  // At most one batch per warp, and about 40 CTAs per SM in all: 4 waves, so that rows with more
  // moves than others leave no tail (evicting from those 16 prompts, the whole call: 58.1 us with
  // 8 CTAs of 8 warps per SM, 55.0 so).
  const int want = std::max(1, 40 * kAttn4Sms / pairs);
  const int per_cta = kMoveThreads / 32 * kBatch;
  const int most = (p.max_moves + per_cta - 1) / per_cta;
  const dim3 grid(static_cast<unsigned>(std::min(want, most)), static_cast<unsigned>(pairs));
  auto go = [&](auto fn) { return launch_behind(fn, grid, kMoveThreads, 0, s, true, p); };
  if (format == kPageBf16)
    return head_dim == 64 ? go(evict_move_kernel<kPageBf16, 64>)
                          : go(evict_move_kernel<kPageBf16, 128>);
  if (format == kPageFp8)
    return head_dim == 64 ? go(evict_move_kernel<kPageFp8, 64>)
                          : go(evict_move_kernel<kPageFp8, 128>);
  return head_dim == 64 ? go(evict_move_kernel<kPageInt4, 64>)
                        : go(evict_move_kernel<kPageInt4, 128>);
}

cudaError_t take_error_evict(unsigned* bits) { return read_error_word(bits); }

}  // namespace pa
