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
// blocks in each one's slice of the reference counts.  A call that cannot be met
// changes nothing.
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
  int warp_sum[kStepWarps];
  int carry;
  int free_blocks;                      // in this CTA's slice; read by the others
  unsigned fail;                        // error bits
};

// Inclusive sum over the CTA's threads; `total` gets the sum of all.
__device__ __forceinline__ int block_scan(int v, StepShared& sh, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) sh.warp_sum[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = sh.warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    sh.warp_sum[lane] = w;
  }
  __syncthreads();
  if (warp > 0) v += sh.warp_sum[warp - 1];
  *total = sh.warp_sum[kStepWarps - 1];
  __syncthreads();
  return v;
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

__global__ void __cluster_dims__(kStepCluster, 1, 1) __launch_bounds__(kStepThreads, 1)
    extend_kernel(const StepParams p) {
  __shared__ StepShared sh;
  extern __shared__ int dyn[];
  const int B = p.num_seqs;
  int* at = dyn;                        // [B] blocks before this sequence's; bit 31: copied
  int* start = at + B;                  // [B] tokens before this sequence's
  int* last = start + B;                // [B] partly filled last block that it appends to, or -1
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) {
    sh.fail = 0;
    sh.free_blocks = 0;
  }
  grid_launch_dependents();
  __syncthreads();

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
    last[b] = id;
  }
  // free blocks of this CTA's slice (a multiple of 4 blocks, so that slices start aligned)
  const int slice = (p.num_blocks + 4 * kStepCluster - 1) / (4 * kStepCluster) * 4;
  const int first = min(p.num_blocks, rank * slice), end = min(p.num_blocks, first + slice);
  const bool wide = (reinterpret_cast<uintptr_t>(p.ref_counts) & 15u) == 0;
  int mine = 0;
  for (int i = first + 4 * tid; i < end; i += 4 * kStepThreads) {
    if (wide && i + 4 <= end) {
      const int4 r = *reinterpret_cast<const int4*>(p.ref_counts + i);
      mine += (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
    } else {
      for (int k = i; k < min(i + 4, end); ++k) mine += p.ref_counts[k] == 0;
    }
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) atomicAdd(&sh.free_blocks, mine);
  __syncthreads();

  // ------------------------------------------------- copies, and the sums over the batch
  int need_sum = 0;
  unsigned long long new_sum = 0;
  for (int b0 = 0; b0 < B; b0 += kStepThreads) {
    const int b = b0 + tid;
    int n = 0, need = 0;
    bool copied = false;
    const bool here = b < B && sh.fail == 0;
    if (here) {
      const int L = p.context_lens[b];
      n = p.new_lens[b];
      need = (L + n + kBlockSize - 1) / kBlockSize - (L + kBlockSize - 1) / kBlockSize;
    }
    const int id = here ? last[b] : -1;
    const int owners = id >= 0 ? p.ref_counts[id] : 0;
    // the batch's earlier sequences that append into the same block have left it by then
    unsigned shared = __ballot_sync(0xffffffffu, owners > 1);
    while (shared) {
      const int src = __ffs(shared) - 1;
      shared &= shared - 1;
      const int block = __shfl_sync(0xffffffffu, id, src), before = b - lane + src;
      int same = 0;
      for (int a = lane; a < before; a += 32) same += last[a] == block;
      same = __reduce_add_sync(0xffffffffu, same);
      if (lane == src) copied = owners - same > 1;
    }
    need += copied;
    int total;
    const int upto = block_scan(need, sh, &total);
    int total_new;
    const int tokens = block_scan(n, sh, &total_new);
    if (b < B) {
      at[b] = (need_sum + upto - need) | (copied ? static_cast<int>(0x80000000u) : 0);
      start[b] = static_cast<int>(new_sum) + tokens - n;
    }
    need_sum += total;
    new_sum += static_cast<unsigned>(total_new);
    if (new_sum > static_cast<unsigned long long>(p.num_tokens)) break;   // uniform
  }
  if (new_sum > static_cast<unsigned long long>(p.num_tokens) && tid == 0) sh.fail = kErrBounds;
  cluster.sync();                       // nobody writes before everybody has read

  // ------------------------------------------------- can it be met
  unsigned fail = sh.fail;
  int before = 0, all = 0;
#pragma unroll
  for (int r = 0; r < kStepCluster; ++r) {
    const int f = cluster.map_shared_rank(&sh, r)->free_blocks;
    before += r < rank ? f : 0;
    all += f;
  }
  if (fail == 0 && need_sum > all) fail = kErrBlocks;
  const int gid = rank * kStepThreads + tid, gsize = kStepCluster * kStepThreads;
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
  for (int i0 = first; i0 < end && before < need_sum; i0 += 4 * kStepThreads) {
    const int i = i0 + 4 * tid;
    int r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = i + k < end ? p.ref_counts[i + k] : 1;
    const int own = (r[0] == 0) + (r[1] == 0) + (r[2] == 0) + (r[3] == 0);
    int total;
    int at_rank = before + block_scan(own, sh, &total) - own;
    before += total;
    if (own == 0 || at_rank >= need_sum) continue;
    // the sequences of this thread's ranks: the last one whose blocks start at or before them
    int lo = 0, hi = B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((at[mid] & 0x7FFFFFFF) <= at_rank)
        lo = mid;
      else
        hi = mid;
    }
    int b = lo;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (r[k] != 0 || at_rank >= need_sum) continue;
      while (b + 1 < B && (at[b + 1] & 0x7FFFFFFF) <= at_rank) ++b;
      const int j = at_rank - (at[b] & 0x7FFFFFFF);
      const bool copied = at[b] < 0;
      const int have = (p.context_lens[b] + kBlockSize - 1) / kBlockSize;
      int32_t* row = p.block_tables + static_cast<size_t>(b) * p.mbs;
      p.ref_counts[i + k] = 1;
      if (copied && j == 0) {
        row[have - 1] = i + k;
        atomicSub(p.ref_counts + last[b], 1);
        p.copies[2 * b] = last[b];
        p.copies[2 * b + 1] = i + k;
      } else {
        row[have + j - copied] = i + k;
      }
      ++at_rank;
    }
  }
  for (int b = gid; b < B; b += gsize) {
    p.query_starts[b + 1] = start[b] + p.new_lens[b];
    if (at[b] >= 0) p.copies[2 * b] = p.copies[2 * b + 1] = 0;
  }
  cluster.sync();                       // the tables are written

  // ------------------------------------------------- slots, and the new lengths behind them
  if (p.slots_here) {
    const int used = static_cast<int>(new_sum);
    for (int i = gid; i < p.num_tokens; i += gsize) {
      if (i < used) {
        const int b = last_at_most(start, B, i);
        put_slot(p, i, b, start[b], p.context_lens[b]);
      } else {
        p.slots[i] = -1;
        p.positions[i] = -1;
      }
    }
    cluster.sync();
  }
  for (int b = gid; b < B; b += gsize) p.context_lens[b] += p.new_lens[b];
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
  // up to two tokens per thread of the cluster, the launch that would spread them over the
  // GPU costs more than it saves
  p.slots_here = p.num_tokens <= 2 * kStepCluster * kStepThreads;
  const int smem = 3 * p.num_seqs * static_cast<int>(sizeof(int));
  static std::atomic<unsigned long long> configured{0ull};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
  if (bit == 0 || (configured.load(std::memory_order_acquire) & bit) == 0) {
    e = cudaFuncSetAttribute(extend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             3 * kMaxStepSeqs * static_cast<int>(sizeof(int)));
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

// Sequences cut back to keep[b] tokens: their blocks behind ceil(keep / 16) lose one owner.
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
