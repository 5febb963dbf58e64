// Log probabilities of given tokens, entropy and the most probable alternatives of
// every row of logits.
//
// With y_i = (x_i - r) log2 e, r any reference, z = sum 2^(y_i), w = sum y_i 2^(y_i):
//   log p_i = x_i - r - log2 z ln 2,     entropy = (log2 z - w / z) ln 2,
// so one pass over the row gives everything, and neither needs the large log-sum-exp
// itself.  Every thread keeps (r, z, w) of its own elements, r following their maximum
// once an element passes it by 5.5 (2^8 in the sums); they are joined at the end.  The
// difference comes first, so that rows of one lowest value of the type are rows of equal
// probabilities.
//
// Alternatives.  The pass also keeps each thread's largest element.  If every one of the
// W warps has J threads at or above a value t, at least W J elements of the row are, so with
// W J >= k only elements >= t can be among the k largest; t is the least of the warps' J-th
// largest thread maxima, and then the k-th largest of the maxima that reach it.  A thread also
// remembers where its maximum came from (a step of two vectors) and the largest of its other
// steps: nearly always that one step, of the few threads that matter, is all that is read again.
// What is >= t goes to a list in shared memory, of which the k largest by (value, lower index)
// are found exactly.  A list that overflows (ties without end, as in rows that are masked to
// -inf) is made again from the elements above t and, in the order of the row, as many equal
// ones as are missing.
//
// The kernel is bound by reading the logits.  A cluster of CTAs shares a row when there are few
// and long ones.  2048 rows of 128256 bf16 with 20 alternatives 97 us (5.4 TB/s); 64 of 128256
// fp32 with 5 12.4 us, a launch and seven barriers on top of 5 us of reading; 1000 of 32003 fp16
// 18.5 us.  With CTAs of 512 threads the first took 157 us (with 256 others stream while one joins
// its row), of 128 threads 161, then 108 with 256; five or six CTAs per SM as four.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>
#include <stdint.h>

#include <algorithm>

#include "pa_pages.cuh"
#include "pa_ptx.cuh"

namespace cg = cooperative_groups;

namespace pa {

constexpr int kScoreThreads = 256;          // four CTAs per SM, so that rows are in different stages
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kScoreList = 2304;            // candidates a CTA holds; a row that leaves a thread
                                            // without an element has fewer in all
constexpr int kScoreSplit = 8;              // CTAs that share a row
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Order of values as unsigned integers; NaN above everything, the zeros equal, 0 = no value.
__device__ __forceinline__ uint32_t value_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
// Larger value first, then the lower index.
__device__ __forceinline__ unsigned long long entry_key(uint32_t value, uint32_t index) {
  return static_cast<unsigned long long>(value) << 32 | static_cast<uint32_t>(~index);
}

struct ScoreSums {
  float r, z, w;
};
__device__ __forceinline__ ScoreSums join(ScoreSums a, ScoreSums b) {
  const float r = fmaxf(a.r, b.r);
  if (r == -CUDART_INF_F) return ScoreSums{r, a.z + b.z, a.w + b.w};
  // 2^(y - d) (y - d) summed: 2^-d (w - d z); 2^-d is 0 long before d reaches its bound
  const float da = fminf((r - a.r) * kLog2e, 1000.f), db = fminf((r - b.r) * kLog2e, 1000.f);
  const float fa = a.r == -CUDART_INF_F ? 0.f : hw_exp2(-da);
  const float fb = b.r == -CUDART_INF_F ? 0.f : hw_exp2(-db);
  // sums without a reference hold no finite element: zeros, or NaN
  const float wa = a.r == -CUDART_INF_F ? a.w : fa * (a.w - da * a.z);
  const float wb = b.r == -CUDART_INF_F ? b.w : fb * (b.w - db * b.z);
  const float za = a.r == -CUDART_INF_F ? a.z : fa * a.z;
  const float zb = b.r == -CUDART_INF_F ? b.z : fb * b.z;
  return ScoreSums{r, za + zb, wa + wb};
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

template <typename T>
struct Vec;                                  // 16 bytes of logits
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void get(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void get(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(w[i]);
      x[2 * i + 1] = bf16_hi(w[i]);
    }
  }
};
template <>
struct Vec<__half> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void get(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
};
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

// The N elements x into the sums, and their maximum; elements of -inf add nothing.
template <int N>
__device__ __forceinline__ float add_elements(ScoreSums& s, const float (&x)[N]) {
  float m = fmaxf(x[0], x[1]), m2 = m;
#pragma unroll
  for (int i = 2; i + 1 < N; i += 4) {
    m = max3(m, x[i], x[i + 1]);
    if (i + 3 < N) m2 = max3(m2, x[i + 2], x[i + 3]);
  }
  m = fmaxf(m, m2);
  if (m > s.r + 5.5f) {                       // the first finite element always
    if (s.r != -CUDART_INF_F) {
      const float d = fminf((m - s.r) * kLog2e, 1000.f), f = hw_exp2(-d);
      s.w = f * (s.w - d * s.z);
      s.z *= f;
    }
    s.r = m;
  }
  const float off = s.r == -CUDART_INF_F ? 0.f : -s.r;
  const uint64_t c2 = pack_f32x2(kLog2e, kLog2e), off2 = pack_f32x2(off, off);
  uint64_t z2 = pack_f32x2(s.z, 0.f), w2 = pack_f32x2(s.w, 0.f);
  static_assert(N % 2 == 0, "pairs");
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const uint64_t t = mul_f32x2(add_f32x2(pack_f32x2(x[i], x[i + 1]), off2), c2);
    // 2^-150 is 0 in fp32: -inf times 0 is kept out of w, NaN is not
    const float t0 = max_nan(__uint_as_float(static_cast<uint32_t>(t)), -150.f);
    const float t1 = max_nan(__uint_as_float(static_cast<uint32_t>(t >> 32)), -150.f);
    const uint64_t e = pack_f32x2(hw_exp2(t0), hw_exp2(t1));
    z2 = add_f32x2(z2, e);
    w2 = fma_f32x2(e, pack_f32x2(t0, t1), w2);
  }
  s.z = __uint_as_float(static_cast<uint32_t>(z2)) + __uint_as_float(static_cast<uint32_t>(z2 >> 32));
  s.w = __uint_as_float(static_cast<uint32_t>(w2)) + __uint_as_float(static_cast<uint32_t>(w2 >> 32));
  return m;
}

constexpr int kScoreStep = 2;               // vectors of a thread's step
constexpr int kScoreRing = 4;               // steps on their way in a long row
constexpr int kScoreLong = 24 * kScoreThreads;  // vectors of a long row (of a CTA's part of it)

struct ScoreShared {
  union {
    uint4 ring[kScoreRing][kScoreStep * kScoreThreads];  // of every thread, in the pass
    unsigned long long list[kScoreList];                 // behind it
  };
  unsigned long long best[kScoreSplit * kMaxScoreTop];   // of every CTA of the row, in CTA 0
  unsigned long long red[kScoreWarps];
  ScoreSums sums[kScoreWarps];
  ScoreSums cta[kScoreSplit];                            // in CTA 0
  uint32_t warp_key[kScoreWarps];
  uint32_t maxima[kScoreThreads];
  int steps[kScoreWarps][32];
  uint32_t bound;
  int num_maxima;
  int count[kScoreWarps];
  int n;
};

// The k largest of `list` (n entries, distinct), in order, through put(rank, entry); every
// thread calls.  Ranks at or above n get nothing.
template <typename Put>
__device__ __forceinline__ void largest(const unsigned long long* list, int n, int k,
                                        ScoreShared& sh, Put put) {
  const int tid = threadIdx.x;
  if (n <= kScoreThreads) {                   // by counting the larger ones
    if (tid < n) {
      const unsigned long long mine = list[tid];
      int rank = 0;
      for (int i = 0; i < n; ++i) rank += list[i] > mine;
      if (rank < k) put(rank, mine);
    }
    __syncthreads();
    return;
  }
  unsigned long long below = ~0ull;           // one maximum after the other
  for (int r = 0; r < k; ++r) {
    unsigned long long m = 0;
    for (int i = tid; i < n; i += kScoreThreads) {
      const unsigned long long e = list[i];
      if (e < below && e > m) m = e;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long y = __shfl_xor_sync(0xffffffffu, m, o);
      m = y > m ? y : m;
    }
    if ((tid & 31) == 0) sh.red[tid >> 5] = m;
    __syncthreads();
    m = sh.red[0];
    for (int i = 1; i < kScoreWarps; ++i) m = sh.red[i] > m ? sh.red[i] : m;
    __syncthreads();
    below = m;
    if (tid == 0 && m != 0) put(r, m);
  }
}

// Every CTA of the cluster has started: its shared memory may be written.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// kSplit CTAs (a cluster) share a row.
template <typename T, int kSplit>
__global__ void __launch_bounds__(kScoreThreads, 4) score_kernel(const ScoreParams p) {
  constexpr int N = Vec<T>::kN;
  __shared__ ScoreShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int part = kSplit > 1 ? static_cast<int>(blockIdx.x % kSplit) : 0;
  const int row = blockIdx.x / kSplit;
  const T* x = static_cast<const T*>(p.logits) + static_cast<size_t>(row) * p.stride;
  const int V = p.vocab, K = p.top;
  // elements before the first 16-byte boundary, whole vectors, elements behind them
  const int head = min(V, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) /
                              static_cast<int>(sizeof(T)));
  const int nv = (V - head) / N, tail = head + nv * N;
  const uint4* vec = reinterpret_cast<const uint4*>(x + head);
  const int per = (nv + kSplit - 1) / kSplit, v0 = min(nv, part * per), v1 = min(nv, v0 + per);
  if (tid == 0) sh.n = sh.num_maxima = 0;
  if constexpr (kSplit > 1) cluster_arrive();

  float given = 0.f;
  int token = -1;
  if (part == 0 && tid == 0) {
    token = p.tokens[row];
    if (token >= V) {
      atomicOr(&g_pa_err, kErrBounds);
      given = CUDART_NAN_F;
    } else if (token >= 0) {
      given = to_float(x[token]);
    }
  }

  // ------------------------------------------------------------------ the pass
  ScoreSums s{-CUDART_INF_F, 0.f, 0.f};
  float most = -CUDART_INF_F, second = -CUDART_INF_F;   // maxima of the best and the other steps
  int best_at = v0;                                     // where the best step begins
  int v = v0 + tid;
  constexpr int U = kScoreStep;
  auto step = [&](const uint4 (&w)[U], int at) {
    float f[U * N];
#pragma unroll
    for (int i = 0; i < U; ++i) Vec<T>::get(w[i], *reinterpret_cast<float(*)[N]>(f + i * N));
    const float m = add_elements(s, f);
    second = fmaxf(second, fminf(m, most));
    best_at = m > most ? at : best_at;
    most = fmaxf(most, m);
  };
  if (v1 - v0 >= kScoreLong) {
    // Through shared memory, some steps ahead: the registers of four CTAs per SM hold too little
    // for memory to go on while a step is added up.  Measured, ahead / not, 1000 rows: 128256
    // bf16 49.4 / 53.5 us, 64000 29.5 / 31.0, 48000 22.7 / 22.3, 32003 18.5 / 17.0 (fp32 28.4 /
    // 28.8); two steps of four vectors ahead 102 against 97 us for the 2048 rows above.
    auto ask = [&](int stage, int from) {
      if (from + (U - 1) * kScoreThreads < v1) {
#pragma unroll
        for (int i = 0; i < U; ++i)
          cp_async_16(smem_u32(&sh.ring[stage][i * kScoreThreads + tid]),
                      vec + from + i * kScoreThreads, 16u);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kScoreRing; ++i) ask(i, v + i * U * kScoreThreads);
    for (int stage = 0; v + (U - 1) * kScoreThreads < v1; v += U * kScoreThreads) {
      cp_async_wait<kScoreRing - 1>();
      uint4 w[U];
#pragma unroll
      for (int i = 0; i < U; ++i) w[i] = sh.ring[stage][i * kScoreThreads + tid];
      step(w, v);
      ask(stage, v + kScoreRing * U * kScoreThreads);
      stage = stage + 1 == kScoreRing ? 0 : stage + 1;
    }
    cp_async_wait<0>();
  } else {
    for (; v + (2 * U - 1) * kScoreThreads < v1; v += 2 * U * kScoreThreads) {
      uint4 w[2][U];
#pragma unroll
      for (int i = 0; i < 2 * U; ++i) w[i / U][i % U] = __ldg(vec + v + i * kScoreThreads);
      step(w[0], v);
      step(w[1], v + U * kScoreThreads);
    }
  }
  for (; v < v1; v += kScoreThreads) {
    float f[N];
    Vec<T>::get(__ldg(vec + v), f);
    const float m = add_elements(s, f);
    second = fmaxf(second, fminf(m, most));
    best_at = m > most ? v : best_at;
    most = fmaxf(most, m);
  }
  // one element in front of or behind the vectors
  int extra = -1;
  if (part == 0) {
    if (tid < head)
      extra = tid;
    else if (tid - head < V - tail)
      extra = tail + tid - head;
  }
  float one = -CUDART_INF_F;
  if (extra >= 0) {
    one = to_float(x[extra]);
    const float f[2] = {one, -CUDART_INF_F};
    add_elements(s, f);
  }

  // ------------------------------------------------------------------ sums of the row
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    s = join(s, ScoreSums{__shfl_xor_sync(0xffffffffu, s.r, o), __shfl_xor_sync(0xffffffffu, s.z, o),
                          __shfl_xor_sync(0xffffffffu, s.w, o)});
  if (lane == 0) sh.sums[warp] = s;

  // ------------------------------------------------------------------ candidates
  if (K > 0) {
    const bool any = v0 + tid < v1 || extra >= 0;
    const uint32_t key = any ? value_key(fmaxf(most, one)) : 0u;
    // the J-th largest of the warp, W J >= K
    uint32_t kj = __reduce_max_sync(0xffffffffu, key), left = key;
    for (int j = kScoreWarps; j < K; j += kScoreWarps) {
      const unsigned who = __ballot_sync(0xffffffffu, left == kj);
      if (lane == __ffs(who) - 1) left = 0u;
      kj = __reduce_max_sync(0xffffffffu, left);
    }
    if (lane == 0) sh.warp_key[warp] = kj;
    __syncthreads();
    uint32_t least = sh.warp_key[0];
#pragma unroll
    for (int i = 1; i < kScoreWarps; ++i) least = min(least, sh.warp_key[i]);
    if (key >= least) sh.maxima[atomicAdd(&sh.num_maxima, 1)] = key;
    __syncthreads();
    const int maxima = sh.num_maxima;
    if (tid < maxima) {
      const uint32_t mine = sh.maxima[tid];
      int above = 0, equal = 0;
      for (int i = 0; i < maxima; ++i) {
        above += sh.maxima[i] > mine;
        equal += sh.maxima[i] == mine;
      }
      if (above < K && above + equal >= K) sh.bound = mine;
    }
    __syncthreads();
    least = sh.bound;
    const float bound = key_value(least);       // NaN where there is none
    auto offer = [&](float f, int index, bool above) {
      if (above ? f <= bound : f < bound) return;
      const uint32_t k = value_key(f);
      if (above ? k > least : k >= least) {
        const int at = atomicAdd(&sh.n, 1);
        if (at < kScoreList) sh.list[at] = entry_key(k, static_cast<uint32_t>(index));
      }
    };
    // (maxima pass over NaN, so a NaN may not be looked at; a row with one has NaN results, and
    // any of its tokens as alternatives)
    auto collect = [&](bool above) {
      const bool mine = v0 + tid < v1 && !(above ? most <= bound : most < bound);
      const bool all = mine && !(above ? second <= bound : second < bound);
      const unsigned step = __ballot_sync(0xffffffffu, mine && !all);
      if (mine && !all) sh.steps[warp][__popc(step & ((1u << lane) - 1))] = best_at;
      __syncwarp();
      for (int g = lane / U; g - lane / U < __popc(step); g += 32 / U) {
        if (g >= __popc(step)) continue;
        const int i = sh.steps[warp][g] + lane % U * kScoreThreads;
        if (i < v1) {
          float f[N];
          Vec<T>::get(__ldg(vec + i), f);
#pragma unroll
          for (int k = 0; k < N; ++k) offer(f[k], head + i * N + k, above);
        }
      }
      unsigned who = __ballot_sync(0xffffffffu, all);
      while (who) {
        const int t = (warp << 5) + __ffs(who) - 1;
        who &= who - 1;
        for (int i = v0 + t + lane * kScoreThreads; i < v1; i += 32 * kScoreThreads) {
          float f[N];
          Vec<T>::get(__ldg(vec + i), f);
#pragma unroll
          for (int k = 0; k < N; ++k) offer(f[k], head + i * N + k, above);
        }
      }
      __syncwarp();
      if (extra >= 0) offer(one, extra, above);
    };
    collect(false);
    __syncthreads();
    int n = sh.n;
    bool slow = false;
    if (n > kScoreList) {
      __syncthreads();
      if (tid == 0) sh.n = 0;
      __syncthreads();
      collect(true);
      __syncthreads();
      n = sh.n;
      slow = n > kScoreList;
      // equal ones in the order of the row: head, vectors, tail of this CTA's part
      const int lo = part == 0 ? 0 : head + v0 * N;
      const int hi = part == 0 && kSplit == 1 ? V : head + v1 * N;
      auto equal_from = [&](int from, int to) {
        for (int i0 = from; i0 < to && n < K; i0 += kScoreThreads) {
          const int i = i0 + tid;
          const bool is = i < to && value_key(to_float(x[i])) == least;
          const unsigned who = __ballot_sync(0xffffffffu, is);
          if (lane == 0) sh.count[warp] = __popc(who);
          __syncthreads();
          int before = n, total = n;
          for (int w = 0; w < kScoreWarps; ++w) {
            before += w < warp ? sh.count[w] : 0;
            total += sh.count[w];
          }
          const int at = before + __popc(who & ((1u << lane) - 1));
          if (is && at < kScoreList) sh.list[at] = entry_key(least, static_cast<uint32_t>(i));
          __syncthreads();
          n = min(total, kScoreList);
        }
      };
      if (!slow) {
        equal_from(lo, hi);
        if (part == 0 && kSplit > 1) equal_from(tail, V);
      }
    }
    unsigned long long* best = sh.best;
    if constexpr (kSplit > 1) {
      cg::cluster_group cluster = cg::this_cluster();
      cluster_wait();
      best = cluster.map_shared_rank(sh.best, 0) + part * kMaxScoreTop;
    }
    if (tid < K) best[tid] = 0;
    __syncthreads();
    if (!slow) {
      largest(sh.list, n, K, sh, [&](int r, unsigned long long e) { best[r] = e; });
    } else {
      // more than the list holds above t: one maximum of the part after the other
      unsigned long long below = ~0ull;
      for (int r = 0; r < K; ++r) {
        unsigned long long m = 0;
        auto look = [&](float f, int index) {
          const unsigned long long e = entry_key(value_key(f), static_cast<uint32_t>(index));
          if (e < below && e > m) m = e;
        };
        for (int i = v0 + tid; i < v1; i += kScoreThreads) {
          float f[N];
          Vec<T>::get(__ldg(vec + i), f);
#pragma unroll
          for (int k = 0; k < N; ++k) look(f[k], head + i * N + k);
        }
        if (extra >= 0) look(one, extra);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const unsigned long long y = __shfl_xor_sync(0xffffffffu, m, o);
          m = y > m ? y : m;
        }
        if (lane == 0) sh.red[warp] = m;
        __syncthreads();
        m = sh.red[0];
        for (int i = 1; i < kScoreWarps; ++i) m = sh.red[i] > m ? sh.red[i] : m;
        __syncthreads();
        below = m;
        if (tid == 0) best[r] = m;
      }
    }
  }
  __syncthreads();
  s = ScoreSums{-CUDART_INF_F, 0.f, 0.f};
  for (int i = 0; i < kScoreWarps; ++i) s = join(s, sh.sums[i]);
  if constexpr (kSplit > 1) {
    cg::cluster_group cluster = cg::this_cluster();
    if (K == 0) cluster_wait();
    if (tid == 0) cluster.map_shared_rank(sh.cta, 0)[part] = s;
    cluster.sync();                           // CTA 0 has every part's sums and candidates
    if (part != 0) return;
    s = sh.cta[0];
    for (int i = 1; i < kSplit; ++i) s = join(s, sh.cta[i]);
  }

  // ------------------------------------------------------------------ outputs
  const float lz = log2f(s.z);
  const float off = s.r == -CUDART_INF_F ? CUDART_NAN_F : -s.r;
  if (tid == 0) {
    p.logprobs[row] = token < 0 ? 0.f : given + off - lz * kLn2;
    p.entropy[row] = (lz - s.w / s.z) * kLn2;
  }
  if (K > 0) {
    auto put = [&](int r, unsigned long long e) {
      const float f = key_value(static_cast<uint32_t>(e >> 32));
      p.top_logprobs[static_cast<size_t>(row) * K + r] = f + off - lz * kLn2;
      p.top_tokens[static_cast<size_t>(row) * K + r] =
          static_cast<int32_t>(~static_cast<uint32_t>(e));
    };
    if constexpr (kSplit > 1) {
      // the parts' candidates, without the empty places
      if (tid == 0) sh.n = 0;
      __syncthreads();
      if (tid < kSplit * kMaxScoreTop && (tid & (kMaxScoreTop - 1)) < K && sh.best[tid] != 0)
        sh.list[atomicAdd(&sh.n, 1)] = sh.best[tid];
      __syncthreads();
      largest(sh.list, sh.n, K, sh, put);
    } else if (tid < K) {
      put(tid, sh.best[tid]);
    }
  }
}

template <typename T>
cudaError_t launch_score_as(const ScoreParams& p, cudaStream_t s) {
  // Eight CTAs for a row while they all run at once and the rows are long, since joining them
  // takes 3 us.  Measured, eight / one per row, bf16: 64 x 128256 10.2 / 11.7 us, 76 x 128256
  // 13.6 / 12.0, 32 x 64000 6.8 / 8.0, 64 x 64000 9.2 / 8.1, 16 x 32000 6.2 / 5.7.
  if (p.num_rows <= 64 && p.vocab >= std::max(48000, 1300 * p.num_rows)) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.num_rows) * kScoreSplit, 1, 1);
    cfg.blockDim = dim3(kScoreThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kScoreSplit;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, score_kernel<T, kScoreSplit>, p);
  }
  score_kernel<T, 1><<<static_cast<unsigned>(p.num_rows), kScoreThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_score(const ScoreParams& p, int dtype, cudaStream_t s) {
  return dtype == 0   ? launch_score_as<float>(p, s)
         : dtype == 1 ? launch_score_as<__nv_bfloat16>(p, s)
                      : launch_score_as<__half>(p, s);
}

cudaError_t take_error_score(unsigned* bits) { return read_error_word(bits); }

}  // namespace pa
