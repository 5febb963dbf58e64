// How the warp-streaming kernels split their work.
//
// Balanced runs: the pages of all jobs (a sequence's kv head, or one row column of it) form
// one list in the order (sequence, job, page), cut into equal runs, one for each worker (a
// warp) that is resident at once, so that ragged contexts neither leave a tail nor a second
// wave.  Each job counts kSetup entries more than it has pages, for what starting on it
// costs.  Every worker finds its own run from the lengths.  A job whose pages lie in one run
// is whole there, and a run may hold many of them; of the cut jobs a worker holds at most two
// pieces, its run's first and last.  A piece slot of a worker is therefore for cut jobs only.
// Units: a worker takes whole (partition, sequence, job) units of ppb pages, partition-major.
#pragma once

#include "pa_pages.cuh"

namespace pa {

struct RunList {
  const int32_t* lens;
  int num_seqs, T, max_ctx, window;
  int heads;                      // jobs per sequence
  int workers, min_share;         // balanced runs
  int ppb, max_parts;             // units
};

// Block ids and the first pages are fetched one after the other: about the time of five pages
// on a busy GPU.  256 sequences of 128-8192 tokens, whose short ones fall several to a run:
// 125.7 / 116.5 / 113.5 / 114.9 us with 1 / 3 / 5 / 7.
constexpr int kSetup = kRunSetup;

// Pages that a sequence's query tokens can see, from page `first` on (0 if its length is out of
// range).
__device__ __forceinline__ int visible_pages(const RunList& r, int L, int& first) {
  first = 0;
  if (L < r.T || L > r.max_ctx) return 0;
  if (r.window > 0) first = max(0, L - r.T - r.window + 1) / kBlockSize;
  return (L + kBlockSize - 1) / kBlockSize - first;
}

__device__ __forceinline__ int pair_entries(int nb) { return nb > 0 ? nb + kSetup : 0; }

// Entries per run: everything split evenly over the workers, but at least min_share.
__device__ __forceinline__ int run_entries(const RunList& r, int total) {
  return max(r.min_share, (total + r.workers - 1) / r.workers);
}

constexpr int kKeep = 8;                     // chunks of 32 lengths held in registers

// Pages [page, page + n) of job `job` of sequence b (whose length is L).
struct Segment {
  int b, job, L, first, page, n;
  int part;                                  // units: the partition
  bool whole;                                // all visible pages of the job
  bool second;                               // balanced: not the worker's first piece
};

template <bool kFlat>
struct Cursor {
  int b, job, entry, nb, first, L;           // balanced: the next piece
  int f, f_end, f0;
  long long u;                               // units

  // False if the worker has nothing to do.  `invalid`: a length is out of range (balanced).
  __device__ __forceinline__ bool start(const RunList& r, int worker, int lane, bool& invalid) {
    invalid = false;
    u = worker;
    if constexpr (!kFlat) return true;
    int len[kKeep], sum = 0;
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
      len[k] = 32 * k + lane < r.num_seqs ? r.lens[32 * k + lane] : -1;
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
      if (32 * k >= r.num_seqs) break;
      int skip;
      sum += pair_entries(visible_pages(r, len[k], skip));
      invalid |= 32 * k + lane < r.num_seqs && (len[k] < r.T || len[k] > r.max_ctx);
    }
    for (int i = 32 * kKeep + lane; i < r.num_seqs; i += 32) {
      int skip;
      const int x = r.lens[i];
      sum += pair_entries(visible_pages(r, x, skip));
      invalid |= x < r.T || x > r.max_ctx;
    }
    const int total = __reduce_add_sync(0xffffffffu, sum) * r.heads;
    const int share = run_entries(r, total);
    if (static_cast<long long>(worker) * share >= total) return false;
    f = f0 = worker * share;
    f_end = min(total, f + share);
    int before = 0;                          // entries of the sequences before b, all jobs
    bool found = false;
    auto search = [&](int base, int Ll) {
      int fl, mine = visible_pages(r, Ll, fl);
      int run = pair_entries(mine);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
      }
      const int upto = before + run * r.heads;
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
      const int from = f - (__shfl_sync(0xffffffffu, upto, at) - ne * r.heads);
      job = from / ne;
      entry = from % ne;
    };
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
      if (!found && 32 * k < r.num_seqs) search(32 * k, len[k]);
    for (int base = 32 * kKeep; !found; base += 32)   // f < total: some chunk ends past it
      search(base, base + lane < r.num_seqs ? r.lens[base + lane] : -1);
    return true;
  }

  // The next piece with pages; false at the end.  `invalid`: a length is out of range (units).
  __device__ __forceinline__ bool next(const RunList& r, Segment& s, bool& invalid) {
    if constexpr (kFlat) {
      while (f < f_end) {
        const int ne = pair_entries(nb);
        const int taken = min(ne - entry, f_end - f);
        const int page = max(0, entry - kSetup);
        const int n = max(0, entry + taken - kSetup) - page;
        s = Segment{b, job, L, first, page, n, 0, n == nb, f != f0};
        f += taken;
        entry = 0;
        if (f < f_end && ++job == r.heads) {
          job = 0;
          do {
            L = r.lens[++b];
            nb = visible_pages(r, L, first);
          } while (nb == 0);                 // f < total: a later sequence has pages
        }
        if (n > 0) return true;
      }
      return false;
    } else {
      const long long per_part = static_cast<long long>(r.heads) * r.num_seqs;
      while (u < per_part * r.max_parts) {
        const int part = static_cast<int>(u / per_part);
        const int in = static_cast<int>(u % per_part);
        u += r.workers;
        const int sb = in / r.heads, len = r.lens[sb];
        int fi;
        const int pages = visible_pages(r, len, fi);
        invalid |= pages == 0 && part == 0;
        const int n = min(r.ppb, pages - part * r.ppb);
        if (n <= 0) continue;
        s = Segment{sb, in % r.heads, len, fi, part * r.ppb, n, part, pages <= r.ppb, false};
        return true;
      }
      return false;
    }
  }
};

__device__ __forceinline__ RunList observe_list(const ObserveParams& p, int ntw) {
  return RunList{p.context_lens, p.num_seqs, p.T,         p.max_ctx, 0,
                 p.Hkv * ntw,    p.workers,  p.min_share, p.ppb,     p.max_parts};
}

// The pieces of job `job` of sequence b, in page order: piece i is held by worker w0 + i, as its
// second piece if `second` and i = 0, otherwise as its first.  One piece: the job is whole and
// has no slot here.  A warp.
struct Pieces {
  int w0, count;
  bool second;
  __device__ __forceinline__ size_t slot(int i) const {
    return static_cast<size_t>(w0 + i) * 2 + (i == 0 && second ? 1 : 0);
  }
};

__device__ __forceinline__ Pieces find_pieces(const RunList& r, int b, int job, int nb, int lane) {
  int all = 0, before = 0;
  for (int base = 0; base < r.num_seqs; base += 32 * kKeep) {
    int len[kKeep];
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
      len[k] = base + 32 * k + lane < r.num_seqs ? r.lens[base + 32 * k + lane] : -1;
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
      if (base + 32 * k >= r.num_seqs) break;
      int first;
      const int n = pair_entries(visible_pages(r, len[k], first));
      all += n;
      if (base + 32 * k + lane < b) before += n;
    }
  }
  all = __reduce_add_sync(0xffffffffu, all);
  before = __reduce_add_sync(0xffffffffu, before);
  const int share = run_entries(r, all * r.heads);
  const int ne = pair_entries(nb);
  const int f0 = before * r.heads + job * ne;
  // the workers of its first and its last page
  const int w0 = (f0 + kSetup) / share, w1 = (f0 + ne - 1) / share;
  return Pieces{w0, w1 - w0 + 1, f0 > w0 * share};
}

}  // namespace pa
