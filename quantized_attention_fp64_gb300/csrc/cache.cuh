// The 8-bit paged key/value cache: its layout and the index arithmetic that
// every kernel on it shares (host and device, so the CPU tests run it too).
//
// A cache holds num_pages pages of page_size tokens (a multiple of 32) of H
// key/value heads. A page of one head is page_size / 32 blocks; a block is 32
// consecutive tokens with one fp32 scale for its keys and one for its values.
// Blocks are numbered (page * H + head) * blocks_per_page + block and lie in
// that order, 32 * D bytes each:
//  - keys:   int8 [D/64][32 tokens][64 channels]. Eight tokens of one
//    64-channel half are 512 contiguous bytes, which a warp reads with one
//    16-byte load per lane: lane 4n + t gets token n's channels 16t..16t+15,
//    the B fragments of four m16n8k16 products.
//  - values: int8 [D channels][32 positions], transposed, so that the products
//    over tokens read them as rows. Token 8j + 2t + e (j, t < 4, e < 2) of the
//    block lies at position 8t + 2j + e: the scores of those eight tokens
//    (j, e) sit in lane 4g + t of the key products' accumulators, and the
//    values that meet them are that lane's 8 consecutive bytes.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"

namespace sage {

constexpr int kCacheBlock = 32;  // tokens that share a scale

struct CacheView {
  int8_t* k;
  int8_t* v;
  float* ks;
  float* vs;
  int64_t num_pages;
  int32_t H;                // key/value heads
  int32_t blocks_per_page;  // page_size / 32
};

// Page table: sequence b's i-th page is row[i] of table + b * stride.
struct PageTable {
  const int32_t* table;
  int64_t stride;
  int64_t max_pages;
};

// Tokens that a row of the page table can name (lengths are 32-bit).
__host__ __device__ inline int64_t table_capacity(int64_t max_pages, int32_t blocks_per_page) {
  const int64_t most = (int64_t(1) << 31) - kCacheBlock;  // the last block's end still fits 32 bits
  const int64_t per_page = int64_t(blocks_per_page) * kCacheBlock;
  return max_pages > most / per_page ? most / per_page * per_page : max_pages * per_page;
}

// A length or count as the caller's array holds it, cut to what is there;
// *bad is set when it had to be cut.
__host__ __device__ inline int64_t checked_length(int64_t n, int64_t most, bool* bad) {
  if (n < 0) {
    *bad = true;
    return 0;
  }
  if (n > most) {
    *bad = true;
    return most;
  }
  return n;
}

__host__ __device__ inline bool page_ok(int64_t page, int64_t num_pages) { return page >= 0 && page < num_pages; }

// Number of the block that holds block `blk` of head `h` of `page`.
__host__ __device__ inline int64_t block_slot(int64_t page, int32_t h, int32_t H, int32_t blocks_per_page,
                                              int32_t blk) {
  return (page * H + h) * blocks_per_page + blk;
}

// The tensor-core attention goes by tiles of 64 keys and looks 32 tiles up at a
// time, past a sequence's end too. Lengths end at 2^31 - 32, where sums of a
// length or a key's number with what a tile holds leave 32 bits: none is formed.
constexpr int kTileKeys = 64;
// Key tiles of a row that sees `sees` keys.
__host__ __device__ inline int key_tiles(int sees) { return sees / kTileKeys + (sees % kTileKeys != 0 ? 1 : 0); }
// Whether block `blk` of a sequence of `len` tokens holds any.
__host__ __device__ inline bool block_has_tokens(int blk, int len) {
  return blk < len / kCacheBlock + (len % kCacheBlock != 0 ? 1 : 0);
}
// Whether the tile whose first key is `key0` has a key that a row which sees `sees` keys does not.
__host__ __device__ inline bool tile_hides_keys(int key0, int sees) { return sees - key0 < kTileKeys; }

// Position of token `i` (0..31) of a block in a row of the values.
__host__ __device__ inline int value_position(int i) { return ((i >> 1) & 3) * 8 + (i >> 3) * 2 + (i & 1); }
// The token at position `p` of a row of the values.
__host__ __device__ inline int value_token(int p) { return ((p >> 1) & 3) * 8 + (p >> 3) * 2 + (p & 1); }

// Value scales in the weights. Both attention kernels put a block's value scale
// into its weights: with y = z + log2 s_v (z: a logit times log2 e) and m about
// the largest y of the row, w = 2^(y - m) multiplies the codes, and the sum of
// 2^(z - m) is that of w over s_v. In m a scale counts as 2^kLogScaleMin at least
// (a scale of 0 everywhere: its codes are 0), so no 2^(z - m) is above
// 2^(8 - kLogScaleMin). Scales are at most 2^121, so a row's sum is 2^-121 at least.
// A weight that fp32 does not hold (below 2^-126) takes its part of the sum with
// it, although next to larger value scales that part may be all of the sum. Parts
// below 2^-45 of the sum do not matter. So while a row has met no scale above
// 2^kLogPlainMax (its sum is 2^-kLogPlainMax at least then), a block whose scale is
// 2^kLogPlainMin or more has a weight of 2^-96, 30 bits above what is lost, or does
// not matter. In other blocks ("odd") the sum is taken apart from the weights, of
// 2^(z - its largest in the block). Sums are taken to another maximum in two steps
// (rescale()), since the factor may leave fp32 where the sum does not.
constexpr float kLogScaleMin = -90.0f;
constexpr float kLogPlainMin = -31.0f, kLogPlainMax = 20.0f;

#ifdef __CUDACC__
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// log2 of a value scale.
__device__ __forceinline__ float log_scale(float vs) { return vs == 0.0f ? kLogScaleMin : __log2f(vs); }

// The factor from maximum m to `up` is the square of this.
__device__ __forceinline__ float half_step(float m, float up) { return ex2(0.5f * (m - up)); }
__device__ __forceinline__ float rescale(float l, float half) { return l * half * half; }
#endif

// Arguments of an attention call on the cache (checked on the host).
struct CacheAttentionArgs {
  CacheView c;
  PageTable pt;
  const int32_t* lengths;    // [B] tokens in the cache
  const int32_t* q_lengths;  // [B] query tokens, or null: T each
  Bf16In q;
  Out out;
  float* lse;                // [B][H][T] or null
  void* workspace;
  int64_t B, T;
  int32_t H;                 // query heads
  bool causal;
  bool zero_rest;            // rows past q_lengths become 0 and -inf
  float sm_log2;             // sm_scale * log2(e)
  int* dev_err;
};

// Launchers of the kernels on the cache (D: 64 or 128; B, T, heads > 0).
cudaError_t launch_cache_append(const CacheView& c, int64_t D, const PageTable& pt, const int32_t* starts,
                                const int32_t* counts, const Bf16In& k, const Bf16In& v, int64_t B, int64_t T,
                                int* dev_err, cudaStream_t stream);
cudaError_t launch_cache_read(const CacheView& c, int64_t D, const PageTable& pt, const int32_t* starts,
                              const int32_t* counts, const Out& k, const Out& v, int64_t B, int64_t T,
                              bool zero_rest, int* dev_err, cudaStream_t stream);
cudaError_t launch_cache_copy_pages(const CacheView& c, int64_t D, const int32_t* src, const int32_t* dst, int64_t n,
                                    int* dev_err, cudaStream_t stream);
size_t cache_attention_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Hkv, int64_t D);
// Many query rows (tensor cores), and its workspace.
cudaError_t launch_cache_attention_tc(const CacheAttentionArgs& a, int64_t D, cudaStream_t stream);
size_t cache_attention_tc_workspace_bytes(int64_t D);
// Joins the parts that the `ctas` CTAs of either attention kernel left in the
// workspace: one int4 per CTA (last CTA of the item that begins in this one and
// goes on, or -1; sequence; 2 x head + slot of the first part; first row), then,
// desc_bytes on, two slots per CTA of slot_rows rows of D floats and their
// (maximum, sum). rows: the most rows of a part.
cudaError_t launch_cache_join(const CacheAttentionArgs& a, int64_t D, int slot_rows, int rows, int ctas,
                              size_t desc_bytes, cudaStream_t stream);
cudaError_t launch_cache_attention(const CacheAttentionArgs& a, int64_t D, cudaStream_t stream);

// Arguments of adding the weights of a step's queries to scores (checked on the host).
struct CacheWeightsArgs {
  CacheView c;
  PageTable pt;
  const int32_t* lengths;    // [B] tokens in the cache
  const int32_t* q_lengths;  // [B] query tokens, or null: T each
  Bf16In q;
  const float* lse;          // [B][H][T]
  float* scores;             // element (b, hkv, j) at b * scores_b + hkv * scores_h + j, j < scores_n
  int64_t scores_b, scores_h, scores_n;
  int64_t B, T;
  int32_t H;                 // query heads
  bool causal;
  float sm_log2;             // sm_scale * log2(e)
  int* dev_err;
};
cudaError_t launch_cache_weights(const CacheWeightsArgs& a, int64_t D, cudaStream_t stream);
// Many query rows (tensor cores).
cudaError_t launch_cache_weights_tc(const CacheWeightsArgs& a, int64_t D, cudaStream_t stream);

// Arguments of an eviction (checked on the host).
struct CacheEvictArgs {
  CacheView c;
  PageTable from, to;
  const int32_t* lengths;    // [B]
  const float* scores;       // element (b, h, j) at b * scores_b + h * scores_h + j, j < scores_n
  int64_t scores_b, scores_h;
  int32_t scores_n;
  int64_t B;
  int32_t keep, recent;      // keep <= scores_n
  int32_t* lengths_out;      // [B]
  int32_t* kept;             // [B][H][kept_n]
  int32_t kept_n;
  float* scores_out;         // [B][H][scores_n]
  void* workspace;
  int* dev_err;
};
cudaError_t launch_cache_evict(const CacheEvictArgs& a, int64_t D, cudaStream_t stream);
size_t cache_evict_workspace_bytes(int64_t B, int64_t H, int64_t keep, int64_t scores_n);

}  // namespace sage
