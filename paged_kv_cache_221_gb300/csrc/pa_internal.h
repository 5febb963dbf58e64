// Internal host/device interface between the C ABI (pa_api.cpp) and the
// kernel translation units.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

// Bits of the sticky device error word (one word per kernel translation unit).
enum : unsigned { kErrBounds = 1u, kErrTimeout = 2u };

constexpr int kBlockSize = 16;        // tokens per physical block (the only size built)
constexpr int kStages = 8;            // pages in flight per CTA (multiple of every PL)
constexpr int kMaxRows = 64;          // query rows per CTA (8 n-tiles of 8)
constexpr int kStreamMaxSeqs = 256;   // persistent decode kernel: sequences its unit list holds
constexpr int kStreamMaxPpb = 256;    // persistent decode kernel: pages per partition
constexpr int kMaxPartitions = 4096;  // split-KV partitions per sequence (merge smem bound)
constexpr unsigned long long kDefaultTimeoutNs = 2000000000ull;   // 2 s per wait
constexpr int kMaxSpecVocab = 1 << 19;  // speculative acceptance: largest vocabulary

// Everything an attention launch needs besides the two tensor maps.
struct AttnParams {
  const void* q;                  // bf16 [B, T, Hq, D]
  void* out;                      // bf16 [B, T, Hq, D]
  const int32_t* block_tables;    // [B, mbs]
  const int32_t* context_lens;    // [B]
  const void* new_k;              // bf16 [B, T, Hkv, D] or nullptr: K of the query tokens,
  const void* new_v;              //   written at positions L-T .. L-1 before they are read
  void* k_pool;                   // the pools again, for those writes
  void* v_pool;
  float* part_o;                  // [B*T*Hq, max_parts, D]   (split-KV partials)
  float2* part_ml;                // [B*T*Hq, max_parts]      (reference max in the log2
                                  //   domain, softmax denominator) per partition
  const int32_t* seq_group;       // [B] or nullptr
  const int32_t* group_prefix_blocks;  // [num_groups] or nullptr
  const float* k_scale;           // FP8 pages: [Hkv] dequantisation scales of K and V
  const float* v_scale;           //   (nullptr for bf16 pages)
  int mbs;                        // max_blocks_per_seq
  int max_ctx;                    // bound on context_lens
  int num_seqs, T, Hq, Hkv, G, num_blocks;
  int ppb;                        // pages (blocks) per partition
  int max_parts;                  // partition slots per query row
  int members_per_chunk;          // shared-prefix kernel: group members per CTA
  int num_chunks;                 // shared-prefix kernel: CTAs per group (per partition, head)
  int max_prefix_blocks;          // bound on group_prefix_blocks (launch sizing)
  float scale_log2;               // softmax scale * log2(e)
  int window;                     // sliding window (positions each query sees), 0 = none
  unsigned wcap;                  // window, or 2^31 without one (visibility: lim - j < wcap)
  int wspan;                      // window, or 2^30 without one (interior pages: tok0 +
                                  //   wspan >= context length)
  unsigned long long timeout_ns;  // limit of every pipeline wait
  int* unit_counter;              // tcgen05 kernel: next work unit to claim (zeroed before the
                                  //   launch), or nullptr for a fixed round-robin order
  void* stream_ctl;               // persistent decode kernel: its StreamCtl in the scratch,
                                  //   or nullptr (no scratch: fixed order)
};

// Claim state of the persistent decode kernel, kept in the split-KV scratch:
// a tag and the next unit-list position to hand out.  When the tag is present
// at launch, `next` is zero and CTAs claim positions from it; the split-KV merge
// that follows every such launch sets `next` back to zero and writes the tag.
// Without the tag (scratch not yet used by this kernel, or overwritten since)
// the launch takes positions in a fixed order and leaves `next` untouched.
struct StreamCtl {
  unsigned long long tag;
  int next;
  int pad;
};
constexpr unsigned long long kStreamTag = 0x70615F7374726D31ull;

// 4-bit pages.  flat: balanced runs, two partial slots of a tile's rows per worker in part_o /
// part_ml; otherwise units of ppb pages and the split-KV layout.
struct Attn4Params : AttnParams {
  bool flat;
  int workers;                    // warps that take part
  int min_share;                  // balanced mode: smallest run in list entries
  bool after_store;               // follows the launch that stores the call's new tokens
};
// Tile of a warp for `rows` query rows per kv head: n-tiles of 8 rows, row columns, and the
// groups of four warps that an SM holds.
struct Attn4Tile {
  int nt, ntw, ctas;
};
constexpr Attn4Tile attn4_tile(int rows) {
  return rows <= 8    ? Attn4Tile{1, 1, 3}
         : rows <= 16 ? Attn4Tile{2, 1, 2}
         : rows <= 24 ? Attn4Tile{3, 1, 2}
         : rows <= 32 ? Attn4Tile{4, 1, 2}
                      : Attn4Tile{4, 2, 2};
}
constexpr Attn4Tile observe_tile(int rows) {
  return rows <= 8    ? Attn4Tile{1, 1, 4}
         : rows <= 16 ? Attn4Tile{2, 1, 3}
         : rows <= 24 ? Attn4Tile{3, 1, 3}
         : rows <= 32 ? Attn4Tile{4, 1, 2}
                      : Attn4Tile{4, 2, 2};
}
constexpr int kAttn4Sms = 152;    // SMs the balanced mode fills
constexpr int kRunSetup = 5;      // list entries a job counts besides its pages (pa_runs.cuh)

// Accumulated attention weights: the first launch writes scores and the chunks' (m, l),
// the second adds the weights up.
struct ObserveParams {
  const void* q;                  // bf16 [B, T, Hq, D]
  const void* k_pool;
  const float* k_scale;           // [Hkv], FP8 and INT4 pages
  const int32_t* block_tables;    // [B, mbs]
  const int32_t* context_lens;    // [B]
  const int32_t* seq_lens;        // [B] or nullptr (= context_lens)
  const float* weights;           // [B, Hkv, weight_entries]
  float* weights_out;             // may be `weights`
  int32_t* positions;             // [B, Hkv, weight_entries] or nullptr
  float* scores;                  // scratch [B, Hkv, G * T, max_entries]
  // scratch [slot][rows of a tile]: (m, l) of every piece.  Balanced runs: two slots per worker
  // for pieces of cut jobs, then one per job that lies whole in a run; otherwise a slot per unit
  float2* ml;
  int mbs, max_ctx, num_seqs, T, Hq, Hkv, G, num_blocks;
  int max_entries;                // max_ctx in whole blocks
  int weight_entries;
  bool flat;                      // balanced runs, or units of ppb pages
  int workers, min_share, ppb, max_parts;
  int tile_rows, ntw;             // rows of a tile, row columns
  float scale_log2, decay;
};

// Eviction: the first launch selects and pairs movers with gaps, the second moves.
struct EvictParams {
  void* k_pool;
  void* v_pool;
  const int32_t* block_tables;    // [B, mbs]
  const int32_t* context_lens;    // [B]
  int32_t* new_lens;              // [B]
  float* weights;                 // [B, Hkv, weight_entries]
  int32_t* positions;             // [B, Hkv, weight_entries]
  int2* moves;                    // scratch [B, Hkv, max_moves] (from, to)
  int32_t* counts;                // scratch [B, Hkv]
  int mbs, max_ctx, num_seqs, Hkv, num_blocks, weight_entries, budget, num_recent, max_moves;
  int format, head_dim;           // of the pages
  bool move_here;                 // few entries to drop: one launch
};

// The partition size (tokens) a per-sequence call with partition_size 0 uses:
// the library default for this batch, with the FP8-page rule when fp8_pages.
int default_partition_for(int max_context_len, int num_seqs, int num_kv_heads, bool fp8_pages);

// Split-KV scratch bytes a call with these sizes needs (partition_size 0 = the
// library default for this kv-head count).
size_t workspace_for(int num_seqs, int num_q_heads, int num_kv_heads, int num_query_tokens,
                     int max_context_len, int head_dim, int partition_size,
                     int max_prefix_blocks);

// Kernel launchers (one translation unit per head_dim and mode); `rows` is the
// number of query rows one CTA carries (1 .. kMaxRows).
// overlap_previous: launch with programmatic stream serialisation so the kernel may
// run alongside the shared-prefix kernel launched just before it.
cudaError_t launch_attn_d64(const CUtensorMap& tk, const CUtensorMap& tv, const AttnParams& p,
                            int rows, dim3 grid, cudaStream_t s, bool overlap_previous);
cudaError_t launch_attn_d128(const CUtensorMap& tk, const CUtensorMap& tv, const AttnParams& p,
                             int rows, dim3 grid, cudaStream_t s, bool overlap_previous);
cudaError_t launch_attn_group_d64(const CUtensorMap& tk, const CUtensorMap& tv,
                                  const AttnParams& p, int rows, dim3 grid, cudaStream_t s);
cudaError_t launch_attn_group_d128(const CUtensorMap& tk, const CUtensorMap& tv,
                                   const AttnParams& p, int rows, dim3 grid, cudaStream_t s);
// FP8 (E4M3) pages: K [NB, Hkv, 16, D] token-major, V [NB, Hkv, D, 16] per-page transposed.
cudaError_t launch_attn8_d64(const CUtensorMap& tk, const CUtensorMap& tv, const AttnParams& p,
                             int rows, dim3 grid, cudaStream_t s, bool overlap_previous);
cudaError_t launch_attn8_d128(const CUtensorMap& tk, const CUtensorMap& tv, const AttnParams& p,
                              int rows, dim3 grid, cudaStream_t s, bool overlap_previous);
cudaError_t launch_attn_group8_d64(const CUtensorMap& tk, const CUtensorMap& tv,
                                   const AttnParams& p, int rows, dim3 grid, cudaStream_t s);
cudaError_t launch_attn_group8_d128(const CUtensorMap& tk, const CUtensorMap& tv,
                                    const AttnParams& p, int rows, dim3 grid, cudaStream_t s);
// Persistent decode kernel (pa_attn_stream.cuh): per-sequence mode, at most 8
// query rows per kv head, at most kStreamMaxSeqs sequences and kStreamMaxPpb
// pages per partition; `max_units` bounds the work units.  Unless `always`, it
// runs only where it measured faster than the one-CTA-per-unit kernel (FP8
// pages, or at least 4 units per resident CTA); *launched says whether it ran.
cudaError_t launch_stream_d64(const CUtensorMap& tk, const CUtensorMap& tv, const AttnParams& p,
                              int rows, long long max_units, bool kv8, bool always,
                              cudaStream_t s, bool* launched);
cudaError_t launch_stream_d128(const CUtensorMap& tk, const CUtensorMap& tv, const AttnParams& p,
                               int rows, long long max_units, bool kv8, bool always,
                               cudaStream_t s, bool* launched);
// tcgen05 kernel (head_dim 128, bf16 pages, 17-32 query rows per kv head).
cudaError_t launch_attn_tc_d128(const CUtensorMap& tk, const CUtensorMap& tv, const AttnParams& p,
                                int rows, dim3 grid, cudaStream_t s, bool overlap_previous);
cudaError_t launch_reshape_fp8(const void* key, const void* value, void* k_cache, void* v_cache,
                               const int64_t* slots, const float* k_scale, const float* v_scale,
                               int num_tokens, int num_blocks, int hkv, int head_dim,
                               cudaStream_t s);
// Speculative acceptance (pa_spec.cu): one CTA per sequence.
cudaError_t launch_spec_accept(const float* p, const float* q, const int32_t* drafts,
                               const uint32_t* a24, const uint32_t* s32, int num_seqs, int K,
                               int V, bool greedy, int32_t* out_tokens, int32_t* out_kept,
                               cudaStream_t s);
// Graph runner padding: rows [from, to) become a one-block sequence of `len` tokens
// in block `pad_block`.
cudaError_t launch_pad_rows(int32_t* block_tables, int32_t* context_lens, int from, int to,
                            int max_blocks_per_seq, int pad_block, int len, cudaStream_t s);
// Graph runner staging: `bytes` (a multiple of 16; both addresses 16-byte aligned and
// device-addressable) copied by a kernel.
cudaError_t launch_stage_copy(void* dst, const void* src, size_t bytes, cudaStream_t s);
// 4-bit pages: attention (k_pool / v_pool hold the pools), writes by slot or, with slots ==
// nullptr, by block table, and reads by slot.
cudaError_t launch_attn4_d64(const Attn4Params& p, int rows, cudaStream_t s);
cudaError_t launch_attn4_d128(const Attn4Params& p, int rows, cudaStream_t s);
cudaError_t launch_store_int4(const void* key, const void* value, void* k_cache, void* v_cache,
                              const int64_t* slots, const int32_t* tables, const int32_t* lens,
                              int T, int mbs, int max_ctx, const float* k_scale,
                              const float* v_scale, int num_tokens, int num_blocks, int hkv,
                              int head_dim, cudaStream_t s);
cudaError_t launch_gather_int4(void* key, void* value, const void* k_cache, const void* v_cache,
                               const int64_t* slots, const float* k_scale, const float* v_scale,
                               int num_tokens, int num_blocks, int hkv, int head_dim,
                               cudaStream_t s);
cudaError_t launch_observe_bf16(const ObserveParams& p, int head_dim, int rows, cudaStream_t s);
cudaError_t launch_observe_fp8(const ObserveParams& p, int head_dim, int rows, cudaStream_t s);
cudaError_t launch_observe_int4(const ObserveParams& p, int head_dim, int rows, cudaStream_t s);
cudaError_t launch_observe_sum(const ObserveParams& p, cudaStream_t s);
cudaError_t launch_evict(const EvictParams& p, int format, int head_dim, cudaStream_t s);
cudaError_t launch_reduce(const AttnParams& p, int head_dim, cudaStream_t s);
cudaError_t launch_reshape(const void* key, const void* value, void* k_cache, void* v_cache,
                           const int64_t* slots, int num_tokens, int num_blocks, int hkv,
                           int head_dim, int block_size, cudaStream_t s);
cudaError_t launch_copy_blocks(void* k_cache, void* v_cache, const int32_t* pairs, int num_pairs,
                               int num_blocks, int hkv, int head_dim, int block_size,
                               cudaStream_t s);
cudaError_t launch_selftest_wait(unsigned long long timeout_ns, cudaStream_t s);

// Read and clear the device error word of each translation unit (synchronous).
cudaError_t take_error_attn_d64(unsigned* bits);
cudaError_t take_error_attn_d128(unsigned* bits);
cudaError_t take_error_group_d64(unsigned* bits);
cudaError_t take_error_group_d128(unsigned* bits);
cudaError_t take_error_attn8_d64(unsigned* bits);
cudaError_t take_error_attn8_d128(unsigned* bits);
cudaError_t take_error_group8_d64(unsigned* bits);
cudaError_t take_error_group8_d128(unsigned* bits);
cudaError_t take_error_spec(unsigned* bits);
cudaError_t take_error_attn_tc_d128(unsigned* bits);
cudaError_t take_error_stream_d64(unsigned* bits);
cudaError_t take_error_stream_d128(unsigned* bits);
cudaError_t take_error_misc(unsigned* bits);
cudaError_t take_error_attn4_d64(unsigned* bits);
cudaError_t take_error_attn4_d128(unsigned* bits);
cudaError_t take_error_cache4(unsigned* bits);
cudaError_t take_error_observe_bf16(unsigned* bits);
cudaError_t take_error_observe_fp8(unsigned* bits);
cudaError_t take_error_observe_int4(unsigned* bits);
cudaError_t take_error_evict(unsigned* bits);

}  // namespace pa
