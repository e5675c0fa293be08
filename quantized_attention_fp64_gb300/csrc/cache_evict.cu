// Cutting cached sequences back: selection of the tokens that stay, and their
// moving together.
//
// Selection. Scores become integers of the same order (a NaN the lowest, -0 like
// 0). The last one that stays is found digit by digit, eight bits at a time from
// the top, each time from a histogram of the next digit of the scores that agree
// with what is known; then everything above it stays, and of those equal to it
// the first ones.
//
// Moving. Kept tokens never move to a later place, so a CTA that takes a
// head's blocks of 32 new places in order and reads a block's tokens before it
// writes any of them may write over the old ones.
#include "cache.cuh"
#include "launch.cuh"
#include "tc_ptx.cuh"

namespace sage {
namespace {

constexpr int kSelect = 1024;  // threads that select for one head
constexpr int kMove = 128;     // threads that move one head's tokens

// Integers in the order of the scores.
__device__ __forceinline__ uint32_t order_of(float x) {
  uint32_t u = __float_as_uint(x);
  if (x != x) return 0u;
  if (u == 0x80000000u) u = 0u;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int32_t length_of(const CacheEvictArgs& a, int b, bool* bad) {
  const int64_t most = table_capacity(a.from.max_pages, a.c.blocks_per_page);
  return static_cast<int32_t>(checked_length(a.lengths[b], most < a.scores_n ? most : a.scores_n, bad));
}

__global__ void __launch_bounds__(kSelect) select_kernel(const CacheEvictArgs a) {
  __shared__ uint32_t count[256];
  __shared__ uint32_t warp_sum[2][32];
  __shared__ uint32_t found_digit, found_need;
  tc::griddep_wait();
  const int b = static_cast<int>(blockIdx.y), h = static_cast<int>(blockIdx.x);
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  const int32_t len = length_of(a, b, &bad);
  if (bad && tid == 0) atomicExch(a.dev_err, kDevErrPage);
  const int32_t stay = min(len, a.keep);
  const int32_t decided = len - min(a.recent, stay);           // the scores decide on those before
  const int32_t need = stay - (len - decided);                 // and keep so many of them
  const float* x = a.scores + b * a.scores_b + h * a.scores_h;
  int32_t* kept = a.kept + (static_cast<int64_t>(b) * a.c.H + h) * a.kept_n;
  float* moved = a.scores_out + (static_cast<int64_t>(b) * a.c.H + h) * a.scores_n;
  if (h == 0 && tid == 0) a.lengths_out[b] = stay;
  uint32_t known = 0, left = static_cast<uint32_t>(need);      // of the scores equal to `known`, keep `left`
  if (need < decided && need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) count[tid] = 0;
      __syncthreads();
      for (int32_t i = tid; i < decided; i += kSelect) {
        const uint32_t u = order_of(x[i]);
        if (shift == 24 || (u ^ known) >> (shift + 8) == 0) atomicAdd(&count[(u >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        uint32_t above = 0, d = 255;
        while (above + count[d] < left) above += count[d--];
        found_digit = d;
        found_need = left - above;
      }
      __syncthreads();
      known |= found_digit << shift;
      left = found_need;
      __syncthreads();
    }
  }
  // places in order: a token's place is the number of kept ones before it
  uint32_t place = 0, equal = 0;
  for (int32_t i0 = 0; i0 < len; i0 += kSelect) {
    const int32_t i = i0 + tid;
    const float score = i < len ? x[i] : 0.0f;
    const uint32_t u = order_of(score);
    const bool open = i < decided && need < decided;           // the scores decide
    const bool same = open && need > 0 && u == known;
    const uint32_t same_mask = __ballot_sync(0xffffffffu, same);
    if (lane == 0) warp_sum[0][warp] = __popc(same_mask);
    __syncthreads();
    uint32_t before = equal, all_same = 0;
    for (int w = 0; w < kSelect / 32; ++w) {
      if (w < warp) before += warp_sum[0][w];
      all_same += warp_sum[0][w];
    }
    before += __popc(same_mask & ((1u << lane) - 1u));
    const bool stays = i < len && (!open || (need > 0 && (u > known || (same && before < left))));
    const uint32_t mask = __ballot_sync(0xffffffffu, stays);
    if (lane == 0) warp_sum[1][warp] = __popc(mask);
    __syncthreads();
    uint32_t at = place, all = 0;
    for (int w = 0; w < kSelect / 32; ++w) {
      if (w < warp) at += warp_sum[1][w];
      all += warp_sum[1][w];
    }
    at += __popc(mask & ((1u << lane) - 1u));
    if (stays) {
      kept[at] = i;
      moved[at] = score;
    }
    place += all;
    equal += all_same;
    __syncthreads();
  }
  for (int32_t i = stay + tid; i < a.kept_n; i += kSelect) kept[i] = -1;
  for (int32_t i = stay + tid; i < a.scores_n; i += kSelect) moved[i] = 0.0f;
}

template <int D>
__global__ void __launch_bounds__(kMove) move_kernel(const CacheEvictArgs a) {
  __shared__ int8_t out[2][kCacheBlock][D];
  __shared__ int64_t from[kCacheBlock];
  __shared__ float scale[2][kCacheBlock];
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int b = static_cast<int>(blockIdx.y), h = static_cast<int>(blockIdx.x), tid = static_cast<int>(threadIdx.x);
  bool bad = false;
  const int32_t stay = min(length_of(a, b, &bad), a.keep);
  const int32_t* kept = a.kept + (static_cast<int64_t>(b) * a.c.H + h) * a.kept_n;
  bad = false;
  for (int32_t m = 0; m * kCacheBlock < stay; ++m) {
    __syncthreads();
    if (tid < kCacheBlock) {
      const int32_t i = m * kCacheBlock + tid;
      int64_t slot = -1;
      int32_t src = 0;
      if (i < stay) {
        src = kept[i];
        const int32_t blk = src / kCacheBlock;
        const int64_t page = a.from.table[b * a.from.stride + blk / a.c.blocks_per_page];
        if (page_ok(page, a.c.num_pages)) slot = block_slot(page, h, a.c.H, a.c.blocks_per_page, blk % a.c.blocks_per_page);
        else bad = true;
      }
      from[tid] = slot < 0 ? -1 : slot * kCacheBlock + src % kCacheBlock;
      scale[0][tid] = slot < 0 ? 0.0f : a.c.ks[slot];
      scale[1][tid] = slot < 0 ? 0.0f : a.c.vs[slot];
    }
    __syncthreads();
    float top[2] = {0.0f, 0.0f};
    for (int i = 0; i < kCacheBlock; ++i)
      for (int w = 0; w < 2; ++w) top[w] = top[w] != top[w] || scale[w][i] <= top[w] ? top[w] : scale[w][i];
    for (int i = 0; i < kCacheBlock; ++i) {
      const int64_t at = from[i];
      if (tid < D) {
        int8_t c[2] = {0, 0};
        if (at >= 0) {
          const int64_t slot = at / kCacheBlock;
          const int t = static_cast<int>(at % kCacheBlock);
          c[0] = a.c.k[slot * kCacheBlock * D + (tid / 64) * 64 * kCacheBlock + t * 64 + tid % 64];
          c[1] = a.c.v[(slot * D + tid) * kCacheBlock + value_position(t)];
        }
        for (int w = 0; w < 2; ++w) {
          const float r = top[w] > 0.0f ? __fdiv_rn(scale[w][i], top[w]) : 0.0f;
          out[w][i][tid] = static_cast<int8_t>(static_cast<int>(rintf(c[w] * r)));
        }
      }
    }
    __syncthreads();
    const int32_t in_seq = m / a.c.blocks_per_page;
    const int64_t page = in_seq < a.to.max_pages ? a.to.table[b * a.to.stride + in_seq] : -1;
    if (!page_ok(page, a.c.num_pages)) {
      bad = true;
      continue;
    }
    const int64_t slot = block_slot(page, h, a.c.H, a.c.blocks_per_page, m % a.c.blocks_per_page);
    if (tid < D)
      for (int i = 0; i < kCacheBlock; ++i) {
        a.c.k[slot * kCacheBlock * D + (tid / 64) * 64 * kCacheBlock + i * 64 + tid % 64] = out[0][i][tid];
        a.c.v[(slot * D + tid) * kCacheBlock + value_position(i)] = out[1][i][tid];
      }
    if (tid == 0) {
      a.c.ks[slot] = top[0];
      a.c.vs[slot] = top[1];
    }
  }
  if (bad) atomicExch(a.dev_err, kDevErrPage);
}

}  // namespace

size_t cache_evict_workspace_bytes(int64_t, int64_t, int64_t, int64_t) { return 0; }

cudaError_t launch_cache_evict(const CacheEvictArgs& a, int64_t D, cudaStream_t stream) {
  if (a.c.H == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>(a.c.H), static_cast<unsigned>(a.B));
  const cudaError_t e = launch_dependent(select_kernel, grid, kSelect, 0, stream, a);
  if (e != cudaSuccess) return e;
  return launch_dependent(D == 128 ? move_kernel<128> : move_kernel<64>, grid, kMove, 0, stream, a);
}

}  // namespace sage
