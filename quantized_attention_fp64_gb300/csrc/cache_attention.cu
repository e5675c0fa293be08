// Attention of T new queries per sequence to an 8-bit paged cache.
//
// For row t of sequence b and query head h (key/value head h / (H / Hkv)),
//   z_j = sm_scale * s_k[block of j] * sum_d q_d kcode_jd,
//   o   = sum_j p_j s_v[block of j] vcode_j / sum_j p_j,  p_j = exp(z_j - max z),
//   lse = max z + ln sum_j exp(z_j - max z),
// over the keys j that the row sees: all of the sequence's length[b], or with
// the causal mask those up to length[b] - q_length[b] + t (the queries are the
// sequence's last tokens). A row that sees no key gets o = 0 and lse = -inf.
//
// One CTA per row: it goes over the blocks of 32 keys with a running maximum
// and sum, everything in fp32.
#include <cuda_bf16.h>

#include "cache.cuh"
#include "common.cuh"

namespace sage {
namespace {

constexpr int kThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
__global__ void __launch_bounds__(kThreads) cache_attention_kernel(CacheAttentionArgs a) {
  __shared__ float qs[D];
  __shared__ float ps[kCacheBlock];
  const int64_t t = blockIdx.x;
  const int h = static_cast<int>(blockIdx.y), b = static_cast<int>(blockIdx.z);
  const int hk = h / (a.H / a.c.H), i = threadIdx.x;
  bool bad = false;
  const int64_t len = checked_length(a.lengths[b], table_capacity(a.pt.max_pages, a.c.blocks_per_page), &bad);
  const int64_t q_len = a.q_lengths != nullptr ? checked_length(a.q_lengths[b], a.T, &bad) : a.T;
  if (bad && i == 0) atomicExch(a.dev_err, kDevErrPage);
  if (t >= q_len) return;
  int64_t sees = a.causal ? len - q_len + t + 1 : len;
  if (sees < 0) sees = 0;
  const uint16_t* q = a.q.p + b * a.q.sb + t * a.q.ss + h * a.q.sh;
  if (i < D) qs[i] = __uint_as_float(static_cast<uint32_t>(q[i]) << 16);
  __syncthreads();
  float m = -INFINITY, l = 0.0f, o = 0.0f;
  const int key = i >> 2, part = i & 3;
  for (int64_t blk = 0; blk * kCacheBlock < sees; ++blk) {
    const int64_t page = a.pt.table[b * a.pt.stride + blk / a.c.blocks_per_page];
    if (!page_ok(page, a.c.num_pages)) {
      if (i == 0) atomicExch(a.dev_err, kDevErrPage);
      continue;
    }
    const int64_t slot = block_slot(page, hk, a.c.H, a.c.blocks_per_page, static_cast<int32_t>(blk % a.c.blocks_per_page));
    const int8_t* k = a.c.k + slot * (kCacheBlock * D);
    const int8_t* v = a.c.v + slot * (kCacheBlock * D);
    float z = 0.0f;
    for (int d = part * (D / 4); d < (part + 1) * (D / 4); ++d)
      z = fmaf(qs[d], static_cast<float>(k[(d / 64) * (kCacheBlock * 64) + key * 64 + d % 64]), z);
    z += __shfl_xor_sync(0xffffffffu, z, 1);
    z += __shfl_xor_sync(0xffffffffu, z, 2);
    z *= a.c.ks[slot] * a.sm_log2;
    if (part == 0) ps[key] = blk * kCacheBlock + key < sees ? z : -INFINITY;
    __syncthreads();
    float mb = m;
    for (int j = 0; j < kCacheBlock; ++j) mb = fmaxf(mb, ps[j]);
    const float ref = mb == -INFINITY ? 0.0f : mb;
    const float alpha = exp2f(m - ref);
    float sum = 0.0f, acc = 0.0f;
    for (int j = 0; j < kCacheBlock; ++j) {
      if (blk * kCacheBlock + j >= sees) break;
      const float p = exp2f(ps[j] - ref);
      sum += p;
      if (i < D) acc = fmaf(p, static_cast<float>(v[i * kCacheBlock + value_position(j)]), acc);
    }
    l = l * alpha + sum;
    o = o * alpha + acc * a.c.vs[slot];
    m = mb;
    __syncthreads();
  }
  if (i < D) {
    const __nv_bfloat16 r = __float2bfloat16_rn(l > 0.0f || l != l ? o / l : 0.0f);
    a.out.p[b * a.out.sb + t * a.out.ss + h * a.out.sh + i] = *reinterpret_cast<const uint16_t*>(&r);
  }
  if (a.lse != nullptr && i == 0)
    a.lse[(static_cast<int64_t>(b) * a.H + h) * a.T + t] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

size_t cache_attention_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

cudaError_t launch_cache_attention(const CacheAttentionArgs& a, int64_t D, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.T), static_cast<unsigned>(a.H), static_cast<unsigned>(a.B));
  if (D == 128)
    cache_attention_kernel<128><<<grid, kThreads, 0, stream>>>(a);
  else
    cache_attention_kernel<64><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace sage
