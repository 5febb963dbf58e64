// 4-bit pages: quantising writes by slot (pa_reshape_and_cache_int4) or by block table
// (the new tokens of pa_attention_int4), and reads by slot (pa_gather_cache_int4).
#include "pa_pages.cuh"

namespace pa {

// One thread per group of 32 head dims of one (token, kv head) of K or of V: no value is
// exchanged between threads, and a group's maximum, scale and reciprocal are worked out once.
// 16389 tokens, 8 heads of 128 dims, 85 MB in 19 us (4.4 TB/s); with one value at a time instead
// of two 20 us (ALU pipe 52 %); four threads per group, which each divide and round for eight
// values, 38 us.
// APPEND: token i = b * T + t goes to position context_lens[b] - T + t of sequence b; otherwise
// to slots[i].
template <int D, bool APPEND>
__global__ void __launch_bounds__(256)
    store_int4_kernel(const uint4* __restrict__ key, const uint4* __restrict__ value,
                      uint8_t* __restrict__ k_cache, uint8_t* __restrict__ v_cache,
                      const int64_t* __restrict__ slots, const int32_t* __restrict__ tables,
                      const int32_t* __restrict__ lens, int T, int mbs, int max_ctx,
                      const float* __restrict__ k_scale, const float* __restrict__ v_scale,
                      int num_tokens, int num_blocks, int hkv) {
  using P = Page<kPageInt4, D>;
  grid_launch_dependents();                    // the attention launch that follows an append
  const long long idx = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const long long half = static_cast<long long>(num_tokens) * hkv * P::kGroups;
  if (idx >= 2 * half) return;
  const bool is_v = idx >= half;
  const long long at = is_v ? idx - half : idx;
  const int gr = static_cast<int>(at % P::kGroups);
  const long long th = at / P::kGroups;
  // a 32-bit division where it will do
  const int i = static_cast<int>(
      th <= 0xffffffffll ? static_cast<uint32_t>(th) / static_cast<uint32_t>(hkv) : th / hkv);
  const int h = static_cast<int>(th - static_cast<long long>(i) * hkv);
  const uint4* src = (is_v ? value : key) + at * 4;
  const uint4 x[4] = {src[0], src[1], src[2], src[3]};
  long long s = -1;
  bool bad = false;
  if constexpr (APPEND) {
    const int b = i / T, L = lens[b];
    // a length out of range is reported by the attention kernel, which skips the sequence
    if (L >= T && L <= max_ctx) {
      const int pos = L - T + i % T;
      const int phys = tables[static_cast<size_t>(b) * mbs + pos / kBlockSize];
      s = static_cast<long long>(phys) * kBlockSize + pos % kBlockSize;
      bad = static_cast<unsigned>(phys) >= static_cast<unsigned>(num_blocks);
    }
  } else {
    s = slots[i];
    bad = s >= static_cast<long long>(num_blocks) * kBlockSize;
  }
  if (bad) {
    if (gr == 0) atomicOr(&g_pa_err, kErrBounds);
    return;
  }
  if (s < 0) return;                           // padding token
  const uint32_t w[16] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w,
                          x[2].x, x[2].y, x[2].z, x[2].w, x[3].x, x[3].y, x[3].z, x[3].w};
  uint32_t codes[4], scale;
  quantize_int4_32(w, (is_v ? v_scale : k_scale)[h], codes, scale);
  uint8_t* page = (is_v ? v_cache : k_cache) +
                  (static_cast<size_t>(s / kBlockSize) * hkv + h) * P::kBytes;
  const int t = static_cast<int>(s % kBlockSize);
  *reinterpret_cast<uint4*>(page + t * P::kRow + 16 * gr) =
      make_uint4(codes[0], codes[1], codes[2], codes[3]);
  page[P::kCodes + t * P::kGroups + gr] = static_cast<uint8_t>(scale);
}

// One thread per 8 head dims of kTokens (slot, kv head) rows a stride apart, K and V, all their
// loads in flight at once: bf16((u - 8) * (scale * head_scale)).  One row per thread while the
// threads fit on the GPU at once (256 tokens of 8 heads, 128 dims, written and read back: 4.9
// us, 6.2 with four), four otherwise (16389 tokens: 36.4 us, 37.6 with one).
template <int D, int kTokens>
__global__ void __launch_bounds__(256)
    gather_int4_kernel(uint4* __restrict__ key, uint4* __restrict__ value,
                       const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache,
                       const int64_t* __restrict__ slots, const float* __restrict__ k_scale,
                       const float* __restrict__ v_scale, int num_tokens, int num_blocks,
                       int hkv) {
  using P = Page<kPageInt4, D>;
  constexpr int VEC = D / 8;
  const int per_token = hkv * VEC;
  const int step = (num_tokens + kTokens - 1) / kTokens;   // tokens i, i + step, ...
  const long long idx = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (idx >= static_cast<long long>(step) * per_token) return;
  const int i0 = static_cast<int>(idx / per_token);
  const int hv = static_cast<int>(idx % per_token);
  const int v = hv % VEC, h = hv / VEC;
  long long s[kTokens];
#pragma unroll
  for (int k = 0; k < kTokens; ++k) s[k] = i0 + k * step < num_tokens ? slots[i0 + k * step] : -1;
  const long long limit = static_cast<long long>(num_blocks) * kBlockSize;
  uint32_t w[kTokens][2], sb[kTokens][2];
#pragma unroll
  for (int k = 0; k < kTokens; ++k) {
    w[k][0] = w[k][1] = 0x88888888u;           // zero, for rows without a slot
    sb[k][0] = sb[k][1] = 0u;
    if (s[k] >= limit) {
      if (v == 0) atomicOr(&g_pa_err, kErrBounds);
    } else if (s[k] >= 0) {
      const size_t page = (static_cast<size_t>(s[k] / kBlockSize) * hkv + h) * P::kBytes;
      const int t = static_cast<int>(s[k] % kBlockSize);
      const size_t code = page + t * P::kRow + 4 * v;
      const size_t scale = page + P::kCodes + t * P::kGroups + v / 4;
      w[k][0] = *reinterpret_cast<const uint32_t*>(k_cache + code);
      w[k][1] = *reinterpret_cast<const uint32_t*>(v_cache + code);
      sb[k][0] = k_cache[scale];
      sb[k][1] = v_cache[scale];
    }
  }
  const float hs[2] = {k_scale[h], v_scale[h]};
#pragma unroll
  for (int k = 0; k < kTokens; ++k) {
    if (i0 + k * step >= num_tokens) break;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint32_t sh = e4m3x2_to_f16x2(sb[k][kv]);
      const float unit =
          __half2float(__ushort_as_half(static_cast<unsigned short>(sh & 0xffffu))) * hs[kv];
      uint32_t r[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t x = w[k][kv] >> (8 * e);
        r[e] = bf162_bits(
            __floats2bfloat162_rn(static_cast<float>(static_cast<int>(x & 15u) - 8) * unit,
                                  static_cast<float>(static_cast<int>(x >> 4 & 15u) - 8) * unit));
      }
      (kv ? value : key)[(static_cast<long long>(i0) + k * step) * per_token + hv] =
          make_uint4(r[0], r[1], r[2], r[3]);
    }
  }
}

namespace {

unsigned blocks_for(long long threads) { return static_cast<unsigned>((threads + 255) / 256); }

}  // namespace

cudaError_t launch_store_int4(const void* key, const void* value, void* k_cache, void* v_cache,
                              const int64_t* slots, const int32_t* tables, const int32_t* lens,
                              int T, int mbs, int max_ctx, const float* k_scale,
                              const float* v_scale, int num_tokens, int num_blocks, int hkv,
                              int head_dim, cudaStream_t s) {
  if (num_tokens == 0) return cudaSuccess;
  const unsigned grid = blocks_for(2ll * num_tokens * hkv * (head_dim / kGroupDims));
  auto go = [&](auto fn) {
    fn<<<grid, 256, 0, s>>>(static_cast<const uint4*>(key), static_cast<const uint4*>(value),
                            static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache), slots,
                            tables, lens, T, mbs, max_ctx, k_scale, v_scale, num_tokens,
                            num_blocks, hkv);
  };
  if (slots != nullptr)
    head_dim == 64 ? go(store_int4_kernel<64, false>) : go(store_int4_kernel<128, false>);
  else
    head_dim == 64 ? go(store_int4_kernel<64, true>) : go(store_int4_kernel<128, true>);
  return cudaGetLastError();
}

cudaError_t launch_gather_int4(void* key, void* value, const void* k_cache, const void* v_cache,
                               const int64_t* slots, const float* k_scale, const float* v_scale,
                               int num_tokens, int num_blocks, int hkv, int head_dim,
                               cudaStream_t s) {
  if (num_tokens == 0) return cudaSuccess;
  const long long threads = static_cast<long long>(num_tokens) * hkv * (head_dim / 8);
  const bool one = threads <= 152ll * 2048;
  const long long tokens = one ? num_tokens : (static_cast<long long>(num_tokens) + 3) / 4;
  const unsigned grid = blocks_for(tokens * hkv * (head_dim / 8));
  auto go = [&](auto fn) {
    fn<<<grid, 256, 0, s>>>(static_cast<uint4*>(key), static_cast<uint4*>(value),
                            static_cast<const uint8_t*>(k_cache),
                            static_cast<const uint8_t*>(v_cache), slots, k_scale, v_scale,
                            num_tokens, num_blocks, hkv);
  };
  if (one)
    head_dim == 64 ? go(gather_int4_kernel<64, 1>) : go(gather_int4_kernel<128, 1>);
  else
    head_dim == 64 ? go(gather_int4_kernel<64, 4>) : go(gather_int4_kernel<128, 4>);
  return cudaGetLastError();
}

cudaError_t take_error_cache4(unsigned* bits) { return read_error_word(bits); }

}  // namespace pa
