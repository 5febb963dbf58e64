// Block tables, reference counts, lengths and slots of a batch on the device: the
// new tokens of every sequence taken in, and sequences cut back.
//
// The state is that of the host block manager (pa_block_manager.cpp) and so is the
// order of allocation: the sequences in batch order, for each the copy of its partly
// filled last block first if another sequence still owns that block, then a block for
// every 16 tokens that do not fit; each time the lowest-numbered free block (reference
// count 0).  With have = ceil(L / 16), want = ceil((L + n) / 16):
//   copied_b = L % 16 and n > 0 and ref[last_b] - #{a < b appending into last_b} > 1
//   need_b   = want - have + copied_b,  at_b = need_0 + .. + need_(b-1)
//   the free block of rank r goes to the sequence b with at_b <= r < at_b + need_b.
//
// One cluster of CTAs does it all in one launch, because the work is a few dependent
// steps on little data: every CTA keeps the whole batch's prefix sums in shared memory,
// computed by itself, so that the only thing the CTAs exchange is the number of free
// blocks in each one's slice of the reference counts.  A thread counts the free blocks of a
// short run of the pool and, with the sums before it, hands out the same ones.  A call that
// cannot be met changes nothing.
//
// Bound by latency: a dozen dependent trips to L2 and barriers.  256 sequences that take in five
// tokens each, 32 of them sharing their last blocks, in a pool of 90000 blocks 12.4 us; 512
// sequences, 257256 tokens, in one of 262144 blocks 25.9 us with the slots' launch.  With runs of
// 32 blocks per thread, or one warp for all shared last blocks, 4 and 8 us more.
#include <cooperative_groups.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "pa_pages.cuh"
#include "pa_ptx.cuh"

namespace cg = cooperative_groups;

namespace pa {

constexpr int kStepCluster = 8;
constexpr int kStepThreads = 1024;
constexpr int kStepWarps = kStepThreads / 32;

struct StepShared {
  unsigned long long warp_sum[kStepWarps];
  unsigned long long many;              // new tokens of the sequences that take in over 2^21
  int free_blocks;                      // in this CTA's slice; read by the others
  unsigned fail;                        // error bits
  int num_shared;
};

// Inclusive sums over the CTA's threads of two 32-bit counts at once; `total` gets those of all.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, StepShared& sh,
                                                         unsigned long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) sh.warp_sum[warp] = v;
  __syncthreads();
  unsigned long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kStepWarps; ++w) {
    const unsigned long long x = sh.warp_sum[w];
    before += w < warp ? x : 0;
    all += x;
  }
  *total = all;
  __syncthreads();
  return before + v;
}

// Largest b in [0, n) with start[b] <= x (start ascending, start[0] <= x).
__device__ __forceinline__ int last_at_most(const int* start, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Slot and position of packed token i of sequence b, whose tokens start at `start`.
__device__ __forceinline__ void put_slot(const StepParams& p, int i, int b, int start, int len) {
  const int pos = len + i - start;
  const int id = p.block_tables[static_cast<size_t>(b) * p.mbs + pos / kBlockSize];
  p.slots[i] = static_cast<int64_t>(id) * kBlockSize + pos % kBlockSize;
  p.positions[i] = pos;
}

// Bit k: block first + k is free; for up to 32 blocks before `end`.
__device__ __forceinline__ uint32_t free_mask(const StepParams& p, int first, int end, bool wide) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 32; k += 4) {
    const int i = first + k;
    if (wide && i + 4 <= end) {
      const int4 r = *reinterpret_cast<const int4*>(p.ref_counts + i);
      m |= static_cast<uint32_t>((r.x == 0) | (r.y == 0) << 1 | (r.z == 0) << 2 | (r.w == 0) << 3)
           << k;
    } else {
      for (int j = i; j < min(i + 4, end); ++j)
        m |= static_cast<uint32_t>(p.ref_counts[j] == 0) << (j - first);
    }
  }
  return m;
}

__global__ void __cluster_dims__(kStepCluster, 1, 1) __launch_bounds__(kStepThreads, 1)
    extend_kernel(const StepParams p) {
  __shared__ StepShared sh;
  extern __shared__ int dyn[];
  const int B = p.num_seqs;
  int* at = dyn;                        // [B] blocks before this sequence's; bit 31: copied
  int* start = at + B;                  // [B] tokens before this sequence's
  int* last = start + B;                // [B] partly filled last block that it appends to, or -1
  int* len = last + B;                  // [B] tokens so far; bit 31 meanwhile: copied
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, lane = tid & 31;
  const int gid = rank * kStepThreads + tid, gsize = kStepCluster * kStepThreads;
  if (tid == 0) {
    sh.fail = 0;
    sh.many = 0;
    sh.num_shared = 0;
  }
  if (!p.slots_here) grid_launch_dependents();          // the slots' launch
  __syncthreads();

  // ------------------------------------------------- free blocks of this thread's run of the pool
  // (a multiple of 4 blocks, or of 32 where that is not enough)
  int run = (p.num_blocks + 4 * gsize - 1) / (4 * gsize) * 4;
  if (run > 32) run = (run + 31) / 32 * 32;
  const int first = static_cast<int>(min(static_cast<long long>(p.num_blocks),
                                         static_cast<long long>(gid) * run));
  const int end = min(p.num_blocks, first + run);
  const bool wide = (reinterpret_cast<uintptr_t>(p.ref_counts) & 15u) == 0;
  const uint32_t mask = first < end ? free_mask(p, first, min(end, first + 32), wide) : 0u;
  int mine = __popc(mask);
  for (int i = first + 32; i < end; i += 32) mine += __popc(free_mask(p, i, min(end, i + 32), wide));

  // ------------------------------------------------- what every sequence appends to
  for (int b = tid; b < B; b += kStepThreads) {
    const int L = p.context_lens[b], n = p.new_lens[b];
    int id = -1;
    if (L < 0 || n < 0 || static_cast<long long>(L) + n >
                              static_cast<long long>(p.mbs) * kBlockSize) {
      sh.fail = kErrBounds;
    } else if (n > 0 && L % kBlockSize != 0) {
      id = p.block_tables[static_cast<size_t>(b) * p.mbs + L / kBlockSize];
      if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_blocks)) {
        sh.fail = kErrBounds;
        id = -1;
      }
    }
    if (n >> 21) atomicAdd(&sh.many, static_cast<unsigned long long>(n));
    last[b] = id;
    len[b] = L;
    start[b] = n;
    const int owners = id >= 0 ? p.ref_counts[id] : 1;
    if (owners < 1) sh.fail = kErrBounds;               // it would be handed out as free
    if (owners > 1) at[atomicAdd(&sh.num_shared, 1)] = b;
  }
  __syncthreads();
  // Below, 1024 counts at a time are summed in 32 bits: those up to 2^21 cannot carry, and the
  // larger ones may not pass the call's limit, 2^30 at most, together.
  bool met = sh.fail == 0 && sh.many <= static_cast<unsigned long long>(p.num_tokens);
  // The shared last blocks, a warp for each: the batch's earlier sequences that append into the
  // same one have left it by then.
  for (int i = tid >> 5; i < sh.num_shared && met; i += kStepWarps) {
    const int b = at[i], block = last[b];
    int same = 0;
    for (int a = lane; a < b; a += 32) same += last[a] == block;
    same = __reduce_add_sync(0xffffffffu, same);
    if (lane == 0 && p.ref_counts[block] - same > 1) len[b] |= static_cast<int>(0x80000000u);
  }
  __syncthreads();

  // ------------------------------------------------- copies, and the sums over the batch
  unsigned long long sums = 0;          // blocks needed (high), tokens (low) so far
  for (int b0 = 0; b0 < B && met; b0 += kStepThreads) {
    const int b = b0 + tid;
    const bool here = b < B;
    const bool copied = here && len[b] < 0;
    const int n = here ? start[b] : 0, L = here ? len[b] & 0x7FFFFFFF : 0;
    const int need = (L + n + kBlockSize - 1) / kBlockSize - (L + kBlockSize - 1) / kBlockSize +
                     copied;
    unsigned long long total;
    const unsigned long long upto =
        sums + block_scan(static_cast<unsigned long long>(need) << 32 | static_cast<unsigned>(n),
                          sh, &total);
    if (here) {
      at[b] = (static_cast<int>(upto >> 32) - need) | (copied ? static_cast<int>(0x80000000u) : 0);
      start[b] = static_cast<int>(upto & 0xFFFFFFFFu) - n;
      len[b] = L;
    }
    sums += total;
    met = (sums & 0xFFFFFFFFu) <= static_cast<unsigned>(p.num_tokens);
  }
  if (!met && tid == 0 && sh.fail == 0) sh.fail = kErrBounds;
  unsigned long long here_free;
  const int upto_mine =
      static_cast<int>(block_scan(static_cast<unsigned long long>(mine), sh, &here_free));
  if (tid == 0) sh.free_blocks = static_cast<int>(here_free);
  cluster.sync();                       // nobody writes before everybody has read

  // ------------------------------------------------- can it be met
  unsigned fail = sh.fail;
  const int need_sum = static_cast<int>(sums >> 32), used = static_cast<int>(sums & 0xFFFFFFFFu);
  int before = 0, all = 0;
#pragma unroll
  for (int r = 0; r < kStepCluster; ++r) {
    const int f = cluster.map_shared_rank(&sh, r)->free_blocks;
    before += r < rank ? f : 0;
    all += f;
  }
  if (fail == 0 && need_sum > all) fail = kErrBlocks;
  if (gid == 0) {
    if (fail) atomicOr(&g_pa_err, fail);
    p.query_starts[0] = 0;
  }
  if (fail) {
    for (int b = gid; b < B; b += gsize) {
      p.query_starts[b + 1] = 0;
      p.copies[2 * b] = p.copies[2 * b + 1] = 0;
    }
    for (int i = gid; i < p.num_tokens; i += gsize) {
      p.slots[i] = -1;
      p.positions[i] = -1;
    }
    cluster.sync();                     // no CTA ends while its shared memory may be read
    return;
  }

  // ------------------------------------------------- free blocks to the sequences that need them
  int at_rank = before + upto_mine - mine;
  if (mine > 0 && at_rank < need_sum) {
    // the sequence of this thread's first rank: the last one whose blocks start at or before it
    int b = 0, hi = B;
    while (hi - b > 1) {
      const int mid = (b + hi) >> 1;
      if ((at[mid] & 0x7FFFFFFF) <= at_rank)
        b = mid;
      else
        hi = mid;
    }
    for (int i0 = first; i0 < end && at_rank < need_sum; i0 += 32) {
      uint32_t m = i0 == first ? mask : free_mask(p, i0, min(end, i0 + 32), wide);
      for (; m != 0 && at_rank < need_sum; m &= m - 1, ++at_rank) {
        const int i = i0 + __ffs(m) - 1;
        while (b + 1 < B && (at[b + 1] & 0x7FFFFFFF) <= at_rank) ++b;
        const int j = at_rank - (at[b] & 0x7FFFFFFF);
        const bool copied = at[b] < 0;
        const int have = (len[b] + kBlockSize - 1) / kBlockSize;
        int32_t* row = p.block_tables + static_cast<size_t>(b) * p.mbs;
        p.ref_counts[i] = 1;
        if (copied && j == 0) {
          row[have - 1] = i;
          atomicSub(p.ref_counts + last[b], 1);
          p.copies[2 * b] = last[b];
          p.copies[2 * b + 1] = i;
        } else {
          row[have + j - copied] = i;
        }
      }
    }
  }
  for (int b = gid; b < B; b += gsize) {
    const int n = (b + 1 < B ? start[b + 1] : used) - start[b];
    p.query_starts[b + 1] = start[b] + n;
    p.context_lens[b] = len[b] + n;
    if (at[b] >= 0) p.copies[2 * b] = p.copies[2 * b + 1] = 0;
  }
  cluster.sync();                       // the tables are written, and nobody reads another's sums

  // ------------------------------------------------- slots
  if (!p.slots_here) return;
  for (int i = gid; i < p.num_tokens; i += gsize) {
    if (i < used) {
      const int b = last_at_most(start, B, i);
      put_slot(p, i, b, start[b], len[b]);
    } else {
      p.slots[i] = -1;
      p.positions[i] = -1;
    }
  }
}

// Slots of many tokens, behind extend_kernel: one thread per token.
__global__ void __launch_bounds__(256) slots_kernel(const StepParams p) {
  grid_dependency_wait();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= p.num_tokens) return;
  if (i >= p.query_starts[p.num_seqs]) {
    p.slots[i] = -1;
    p.positions[i] = -1;
    return;
  }
  const int b = last_at_most(p.query_starts, p.num_seqs, i);
  put_slot(p, i, b, p.query_starts[b], p.context_lens[b] - p.new_lens[b]);
}

cudaError_t launch_extend(const StepParams& args, cudaStream_t s) {
  StepParams p = args;
  // up to two tokens per thread of the cluster, the launch that would spread them over the GPU
  // costs more than it saves.  Measured, here / by a launch: 8192 tokens 8.3 / 9.7 us, 16384
  // 9.1 / 9.7, 32768 11.0 / 10.3, 65536 14.8 / 11.4
  p.slots_here = p.num_tokens <= 2 * kStepCluster * kStepThreads;
  const int smem = 4 * p.num_seqs * static_cast<int>(sizeof(int));
  static std::atomic<unsigned long long> configured{0ull};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
  if (bit == 0 || (configured.load(std::memory_order_acquire) & bit) == 0) {
    e = cudaFuncSetAttribute(extend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             4 * kMaxStepSeqs * static_cast<int>(sizeof(int)));
    if (e != cudaSuccess) return e;
    if (bit) configured.fetch_or(bit, std::memory_order_acq_rel);
  }
  extend_kernel<<<kStepCluster, kStepThreads, smem, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.slots_here) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.num_tokens + 255) / 256), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, slots_kernel, p);
}

// Sequences cut back to keep[b] tokens: their blocks behind ceil(keep / 16) lose one owner.  Two
// dependent trips to L2 and the launch, 2.3 us for 256 sequences that drop a block at most.
__global__ void __launch_bounds__(128)
    truncate_kernel(int32_t* __restrict__ tables, int32_t* __restrict__ lens,
                    int32_t* __restrict__ refs, const int32_t* __restrict__ keep, int mbs,
                    int num_blocks) {
  const int b = blockIdx.x;
  const int L = lens[b], n = keep[b];
  if (n < 0 || n > L || static_cast<long long>(L) > static_cast<long long>(mbs) * kBlockSize) {
    if (threadIdx.x == 0) atomicOr(&g_pa_err, kErrBounds);
    return;
  }
  int32_t* row = tables + static_cast<size_t>(b) * mbs;
  const int end = (L + kBlockSize - 1) / kBlockSize;
  for (int j = (n + kBlockSize - 1) / kBlockSize + threadIdx.x; j < end; j += 128) {
    const int id = row[j];
    row[j] = -1;
    if (static_cast<unsigned>(id) >= static_cast<unsigned>(num_blocks)) {
      atomicOr(&g_pa_err, kErrBounds);
    } else if (atomicSub(refs + id, 1) < 1) {
      atomicAdd(refs + id, 1);                    // nobody owned it
      atomicOr(&g_pa_err, kErrBounds);
    }
  }
  __syncthreads();                                // every thread has read the length
  if (threadIdx.x == 0) lens[b] = n;
}

cudaError_t launch_truncate(int32_t* tables, int32_t* lens, int32_t* refs, const int32_t* keep,
                            int num_seqs, int mbs, int num_blocks, cudaStream_t s) {
  truncate_kernel<<<static_cast<unsigned>(num_seqs), 128, 0, s>>>(tables, lens, refs, keep, mbs,
                                                                  num_blocks);
  return cudaGetLastError();
}

cudaError_t take_error_step(unsigned* bits) { return read_error_word(bits); }

}  // namespace pa
