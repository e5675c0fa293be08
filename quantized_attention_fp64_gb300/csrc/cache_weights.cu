// Attention weights that cached tokens get from a step's queries: a thread has
// one token of one key/value head, and sums exp(z - lse) over the query heads of
// the group and the query rows that see it.
#include "cache.cuh"
#include "launch.cuh"
#include "tc_ptx.cuh"

namespace sage {
namespace {

constexpr int kThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
__global__ void __launch_bounds__(kThreads) cache_weights_kernel(const CacheWeightsArgs a) {
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int b = static_cast<int>(blockIdx.z), hk = static_cast<int>(blockIdx.y);
  bool bad = false;
  const int32_t len = static_cast<int32_t>(
      checked_length(a.lengths[b], table_capacity(a.pt.max_pages, a.c.blocks_per_page), &bad));
  const int32_t rows =
      a.q_lengths != nullptr ? static_cast<int32_t>(checked_length(a.q_lengths[b], a.T, &bad)) : static_cast<int32_t>(a.T);
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int G = a.H / a.c.H;
  if (j < len && j < a.scores_n) {
    const int32_t blk = static_cast<int32_t>(j / kCacheBlock);
    const int64_t page = a.pt.table[b * a.pt.stride + blk / a.c.blocks_per_page];
    if (!page_ok(page, a.c.num_pages)) {
      bad = true;
    } else {
      const int64_t slot = block_slot(page, hk, a.c.H, a.c.blocks_per_page, blk % a.c.blocks_per_page);
      const int8_t* codes = a.c.k + slot * kCacheBlock * D + (j % kCacheBlock) * 64;
      const float scale = a.c.ks[slot] * a.sm_log2;
      const int64_t first = a.causal ? j - len + rows : 0;  // the first row that sees the token
      float sum = 0.0f;
      for (int64_t t = first < 0 ? 0 : first; t < rows; ++t)
        for (int g = 0; g < G; ++g) {
          const int h = hk * G + g;
          const uint16_t* q = a.q.p + b * a.q.sb + t * a.q.ss + h * a.q.sh;
          float z = 0.0f;
          for (int d = 0; d < D; ++d)
            z = fmaf(__uint_as_float(static_cast<uint32_t>(q[d]) << 16),
                     static_cast<float>(codes[(d / 64) * 64 * kCacheBlock + d % 64]), z);
          const float lse = a.lse[(static_cast<int64_t>(b) * a.H + h) * a.T + t];
          if (lse != -INFINITY) sum += exp2f(fmaf(z, scale, -lse * kLog2e));
        }
      if (first < rows) a.scores[b * a.scores_b + hk * a.scores_h + j] += sum;
    }
  }
  if (bad) atomicExch(a.dev_err, kDevErrPage);
}

}  // namespace

cudaError_t launch_cache_weights(const CacheWeightsArgs& a, int64_t D, cudaStream_t stream) {
  const int64_t most = table_capacity(a.pt.max_pages, a.c.blocks_per_page);
  const int64_t tokens = a.scores_n < most ? a.scores_n : most;
  if (tokens == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>(div_up(tokens, kThreads)), static_cast<unsigned>(a.c.H),
                  static_cast<unsigned>(a.B));
  return launch_dependent(D == 128 ? cache_weights_kernel<128> : cache_weights_kernel<64>, grid, kThreads, 0, stream, a);
}

}  // namespace sage
