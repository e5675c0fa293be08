// Writing, reading and moving the pages of the 8-bit key/value cache.
//
// Append (one block of 32 tokens and one head at a time): with x the new
// tokens that fall into the block, a = max |x| over them and all channels, and
// s the block's scale where it already holds older tokens (else 0),
//   s' = max(s, a / 127),  code(x) = rint(x / s') in [-127, 127],
//   older codes c become rint(c * (s / s')) where s' differs from s.
// All divisions are correctly rounded in fp32, so the codes are a function of
// the inputs alone. A block whose new tokens hold an infinity or a NaN gets the
// scale NaN (its tokens then read as NaN, as the inputs would have made them).
// s' = 0 (all zeros) gives codes 0.
//
// These kernels move bytes: each token is read once and written once, and the
// time is that of HBM (or, for a few tokens, of one dependent load and store).
#include <cuda_bf16.h>

#include "cache.cuh"
#include "common.cuh"

namespace sage {
namespace {

constexpr int kThreads = 256;  // 128 on the keys, 128 on the values

__device__ __forceinline__ void flag_pages(int* dev_err) { atomicExch(dev_err, kDevErrPage); }

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ int quantize_one(float x, float s) {
  const float c = rintf(__fdiv_rn(x, s));
  return static_cast<int>(fminf(fmaxf(c, -127.0f), 127.0f));
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
  return (a & 255) | ((b & 255) << 8) | ((c & 255) << 16) | (static_cast<uint32_t>(d) << 24);
}

// The block that blockIdx.x stands for in sequence blockIdx.z, and the tokens
// of the call that fall into it.
struct Span {
  int64_t slot;   // block number in the cache, -1: nothing to do
  int64_t t0;     // the call's token in the block's slot 0 (negative: older tokens come first)
  int first, end; // slots [first, end) hold the call's tokens
};

__device__ Span find_span(const CacheView& c, const PageTable& pt, const int32_t* starts, const int32_t* counts,
                          int64_t T, int* dev_err) {
  const int64_t b = blockIdx.z;
  const int32_t h = static_cast<int32_t>(blockIdx.y);
  Span s;
  s.slot = -1;
  bool bad = false;
  const int64_t capacity = table_capacity(pt.max_pages, c.blocks_per_page);
  const int64_t start = checked_length(starts[b], capacity, &bad);
  int64_t n = counts != nullptr ? checked_length(counts[b], T, &bad) : T;
  n = checked_length(n, capacity - start, &bad);
  const int64_t blk = start / kCacheBlock + blockIdx.x;
  s.t0 = blk * kCacheBlock - start;
  s.first = s.t0 < 0 ? static_cast<int>(-s.t0) : 0;
  s.end = static_cast<int>(min(n - s.t0, static_cast<int64_t>(kCacheBlock)));
  if (s.end > s.first) {
    const int64_t page = pt.table[b * pt.stride + blk / c.blocks_per_page];
    if (page_ok(page, c.num_pages))
      s.slot = block_slot(page, h, c.H, c.blocks_per_page, static_cast<int32_t>(blk % c.blocks_per_page));
    else
      bad = true;
  }
  if (bad && threadIdx.x == 0) flag_pages(dev_err);
  return s;
}

// ------------------------------------------------------------------ append --
// One CTA writes one block of one head: threads 0..127 its keys, 128..255 its
// values. Four threads share a token, D / 4 channels each.
template <int D>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(CacheView c, PageTable pt, const int32_t* starts,
                                                                const int32_t* counts, Bf16In k, Bf16In v, int64_t T,
                                                                int* dev_err) {
  constexpr int kCh = D / 4;  // channels per thread
  constexpr int kW = kCh / 2; // 32-bit words of them
  // value codes of the block, transposed through shared memory: 36-byte rows
  // so that the byte stores of one warp (8 tokens x 4 channel groups) spread
  __shared__ __align__(16) uint8_t vt[D * 36];
  __shared__ uint32_t amax_w[8];
  const Span s = find_span(c, pt, starts, counts, T, dev_err);
  if (s.slot < 0) return;
  const int half = threadIdx.x >> 7, i = threadIdx.x & 127;
  const int row = i >> 2, part = i & 3;  // token slot, channel group
  const bool mine = row >= s.first && row < s.end;
  const Bf16In& in = half ? v : k;
  float* scale_at = (half ? c.vs : c.ks) + s.slot;
  const float s_old = s.first > 0 ? *scale_at : 0.0f;
  uint32_t w[kW];
#pragma unroll
  for (int q = 0; q < kW; ++q) w[q] = 0u;
  if (mine) {
    const uint16_t* p = in.p + static_cast<int64_t>(blockIdx.z) * in.sb + (s.t0 + row) * in.ss +
                        static_cast<int64_t>(blockIdx.y) * in.sh + part * kCh;
#pragma unroll
    for (int q = 0; q < kW / 4; ++q) reinterpret_cast<uint4*>(w)[q] = reinterpret_cast<const uint4*>(p)[q];
  }
  // max |x| as bit patterns: those of infinities and NaN are the largest
  uint32_t a = 0;
#pragma unroll
  for (int q = 0; q < kW; ++q) a = max(a, max(w[q] & 0x7FFFu, (w[q] >> 16) & 0x7FFFu));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
  if ((threadIdx.x & 31) == 0) amax_w[threadIdx.x >> 5] = a;
  __syncthreads();  // also: every thread has read s_old
  a = max(max(amax_w[half * 4], amax_w[half * 4 + 1]), max(amax_w[half * 4 + 2], amax_w[half * 4 + 3]));
  float s_new = __fdiv_rn(__uint_as_float(a << 16), kInt8Max);
  if (a >= 0x7F80u || s_old != s_old) s_new = __uint_as_float(0x7FC00000u);
  else s_new = fmaxf(s_old, s_new);
  const bool usable = s_new > 0.0f;             // false for 0 and NaN
  const bool grew = s.first > 0 && !(s_new == s_old);
  const float shrink = (grew && usable) ? __fdiv_rn(s_old, s_new) : 0.0f;
  if (i == 0) *scale_at = s_new;
  int8_t* block = (half ? c.v : c.k) + s.slot * (kCacheBlock * D);
  uint32_t codes[kCh / 4];
#pragma unroll
  for (int q = 0; q < kCh / 4; ++q) {
    codes[q] = 0u;
    if (mine && usable)
      codes[q] = pack4(quantize_one(bf16_lo(w[2 * q]), s_new), quantize_one(bf16_hi(w[2 * q]), s_new),
                       quantize_one(bf16_lo(w[2 * q + 1]), s_new), quantize_one(bf16_hi(w[2 * q + 1]), s_new));
  }
  if (half == 0) {
    // keys: this thread's channels lie inside one 64-channel half
    int8_t* p = block + (part * kCh / 64) * (kCacheBlock * 64) + row * 64 + (part * kCh) % 64;
    if (row < s.first) {
      if (grew) {
#pragma unroll
        for (int q = 0; q < kCh / 16; ++q) {
          uint4 o = reinterpret_cast<uint4*>(p)[q];
          int8_t* ob = reinterpret_cast<int8_t*>(&o);
#pragma unroll
          for (int e = 0; e < 16; ++e) ob[e] = static_cast<int8_t>(rintf(ob[e] * shrink));
          reinterpret_cast<uint4*>(p)[q] = o;
        }
      }
    } else {
#pragma unroll
      for (int q = 0; q < kCh / 16; ++q)
        reinterpret_cast<uint4*>(p)[q] = make_uint4(codes[4 * q], codes[4 * q + 1], codes[4 * q + 2], codes[4 * q + 3]);
    }
  } else {
    const int pos = value_position(row);
#pragma unroll
    for (int e = 0; e < kCh; ++e) vt[(part * kCh + e) * 36 + pos] = static_cast<uint8_t>(codes[e / 4] >> (8 * (e % 4)));
  }
  __syncthreads();
  if (half == 1) {
    for (int ch = i; ch < D; ch += 128) {
      uint32_t o[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) o[q] = *reinterpret_cast<const uint32_t*>(vt + ch * 36 + 4 * q);
      int8_t* p = block + ch * kCacheBlock;
      if (s.first > 0) {
        // older tokens' codes stay in the block
        uint32_t was[8];
        *reinterpret_cast<uint4*>(was) = reinterpret_cast<const uint4*>(p)[0];
        *reinterpret_cast<uint4*>(was + 4) = reinterpret_cast<const uint4*>(p)[1];
        int8_t* ob = reinterpret_cast<int8_t*>(o);
        const int8_t* wb = reinterpret_cast<const int8_t*>(was);
#pragma unroll
        for (int e = 0; e < kCacheBlock; ++e)
          if (value_token(e) < s.first) ob[e] = grew ? static_cast<int8_t>(rintf(wb[e] * shrink)) : wb[e];
      }
      reinterpret_cast<uint4*>(p)[0] = make_uint4(o[0], o[1], o[2], o[3]);
      reinterpret_cast<uint4*>(p)[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

// -------------------------------------------------------------------- read --

__device__ __forceinline__ uint32_t to_bf16x2(float a, float b) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <int D>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(CacheView c, PageTable pt, const int32_t* starts,
                                                              const int32_t* counts, Out k, Out v, int64_t T,
                                                              bool zero_rest, int* dev_err) {
  constexpr int kCh = D / 4;
  __shared__ __align__(16) uint8_t vt[D * 36];
  const Span s = find_span(c, pt, starts, counts, T, dev_err);
  const int half = threadIdx.x >> 7, i = threadIdx.x & 127;
  const int row = i >> 2, part = i & 3;
  const Out& o = half ? v : k;
  uint16_t* dst = o.p + static_cast<int64_t>(blockIdx.z) * o.sb + (s.t0 + row) * o.ss +
                  static_cast<int64_t>(blockIdx.y) * o.sh + part * kCh;
  if (zero_rest && row >= s.first && s.t0 + row < T && (row >= s.end || s.slot < 0)) {
#pragma unroll
    for (int q = 0; q < kCh / 8; ++q) reinterpret_cast<uint4*>(dst)[q] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (s.slot < 0) return;
  const float scale = (half ? c.vs : c.ks)[s.slot];
  const int8_t* block = (half ? c.v : c.k) + s.slot * (kCacheBlock * D);
  uint32_t codes[kCh / 4];
  if (half == 1) {
    for (int ch = i; ch < D; ch += 128) {
      uint32_t o[8];
      *reinterpret_cast<uint4*>(o) = reinterpret_cast<const uint4*>(block + ch * kCacheBlock)[0];
      *reinterpret_cast<uint4*>(o + 4) = reinterpret_cast<const uint4*>(block + ch * kCacheBlock)[1];
#pragma unroll
      for (int q = 0; q < 8; ++q) *reinterpret_cast<uint32_t*>(vt + ch * 36 + 4 * q) = o[q];
    }
  } else {
    const int8_t* p = block + (part * kCh / 64) * (kCacheBlock * 64) + row * 64 + (part * kCh) % 64;
#pragma unroll
    for (int q = 0; q < kCh / 16; ++q) reinterpret_cast<uint4*>(codes)[q] = reinterpret_cast<const uint4*>(p)[q];
  }
  __syncthreads();
  if (row < s.first || row >= s.end) return;
  if (half == 1) {
    const int pos = value_position(row);
#pragma unroll
    for (int q = 0; q < kCh / 4; ++q) {
      const uint8_t* p = vt + (part * kCh + 4 * q) * 36 + pos;
      codes[q] = p[0] | (p[36] << 8) | (p[72] << 16) | (static_cast<uint32_t>(p[108]) << 24);
    }
  }
  const int8_t* cb = reinterpret_cast<const int8_t*>(codes);
#pragma unroll
  for (int q = 0; q < kCh / 8; ++q)
    reinterpret_cast<uint4*>(dst)[q] =
        make_uint4(to_bf16x2(cb[8 * q] * scale, cb[8 * q + 1] * scale),
                   to_bf16x2(cb[8 * q + 2] * scale, cb[8 * q + 3] * scale),
                   to_bf16x2(cb[8 * q + 4] * scale, cb[8 * q + 5] * scale),
                   to_bf16x2(cb[8 * q + 6] * scale, cb[8 * q + 7] * scale));
}

// -------------------------------------------------------------------- copy --
// Page dst[i] becomes a copy of page src[i]. An entry with a negative dst, or
// with src = dst, stands for nothing. No page may be named twice as dst, nor as
// dst of one entry and src of another: the copies would depend on their order.
// Every CTA checks the whole lists with one bit per page in shared memory
// before it copies anything, so a list that breaks the rule, or names a page
// that is not there, moves no byte and sets the device error word.
constexpr int kCopyThreads = 256;
constexpr int64_t kCopyChunk = 32768;  // bytes of codes that one CTA moves at a time

__global__ void __launch_bounds__(kCopyThreads) cache_copy_kernel(CacheView c, const int32_t* src, const int32_t* dst,
                                                                  int64_t n, int64_t codes_bytes, int64_t scales,
                                                                  int64_t chunks, int* dev_err) {
  extern __shared__ uint32_t taken[];
  const int64_t words = (c.num_pages + 31) / 32;
  for (int64_t i = threadIdx.x; i < words; i += kCopyThreads) taken[i] = 0u;
  __syncthreads();
  bool bad = false;
  for (int64_t i = threadIdx.x; i < n; i += kCopyThreads) {
    const int32_t d = dst[i], s = src[i];
    if (d < 0 || d == s) continue;
    if (!page_ok(d, c.num_pages) || !page_ok(s, c.num_pages)) bad = true;
    else if (atomicOr(&taken[d >> 5], 1u << (d & 31)) >> (d & 31) & 1u) bad = true;
  }
  __syncthreads();
  for (int64_t i = threadIdx.x; i < n; i += kCopyThreads) {
    const int32_t d = dst[i], s = src[i];
    if (d >= 0 && d != s && page_ok(s, c.num_pages) && (taken[s >> 5] >> (s & 31) & 1u)) bad = true;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) flag_pages(dev_err);
    return;
  }
  // work: n entries x (keys, values) x chunks of a page's codes
  const int64_t total = n * 2 * chunks;
  for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
    const int64_t entry = u / (2 * chunks), r = u % (2 * chunks);
    const int which = static_cast<int>(r / chunks);
    const int64_t chunk = r % chunks;
    const int32_t d = dst[entry], s = src[entry];
    if (d < 0 || d == s) continue;
    int8_t* base = which ? c.v : c.k;
    const int64_t lo = chunk * kCopyChunk, hi = min(lo + kCopyChunk, codes_bytes);
    const uint4* from = reinterpret_cast<const uint4*>(base + s * codes_bytes);
    uint4* to = reinterpret_cast<uint4*>(base + d * codes_bytes);
    for (int64_t q = lo / 16 + threadIdx.x; q < hi / 16; q += kCopyThreads) to[q] = from[q];
    if (chunk == 0) {
      float* sc = which ? c.vs : c.ks;
      for (int64_t q = threadIdx.x; q < scales; q += kCopyThreads) sc[d * scales + q] = sc[s * scales + q];
    }
  }
}

dim3 span_grid(const CacheView& c, int64_t B, int64_t T) {
  // T tokens from any start touch at most (T + 30) / 32 + 1 blocks
  return dim3(static_cast<unsigned>((T + kCacheBlock - 2) / kCacheBlock + 1), static_cast<unsigned>(c.H),
              static_cast<unsigned>(B));
}

}  // namespace

cudaError_t launch_cache_append(const CacheView& c, int64_t D, const PageTable& pt, const int32_t* starts,
                                const int32_t* counts, const Bf16In& k, const Bf16In& v, int64_t B, int64_t T,
                                int* dev_err, cudaStream_t stream) {
  if (D == 128)
    cache_append_kernel<128><<<span_grid(c, B, T), kThreads, 0, stream>>>(c, pt, starts, counts, k, v, T, dev_err);
  else
    cache_append_kernel<64><<<span_grid(c, B, T), kThreads, 0, stream>>>(c, pt, starts, counts, k, v, T, dev_err);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheView& c, int64_t D, const PageTable& pt, const int32_t* starts,
                              const int32_t* counts, const Out& k, const Out& v, int64_t B, int64_t T,
                              bool zero_rest, int* dev_err, cudaStream_t stream) {
  if (D == 128)
    cache_read_kernel<128><<<span_grid(c, B, T), kThreads, 0, stream>>>(c, pt, starts, counts, k, v, T, zero_rest, dev_err);
  else
    cache_read_kernel<64><<<span_grid(c, B, T), kThreads, 0, stream>>>(c, pt, starts, counts, k, v, T, zero_rest, dev_err);
  return cudaGetLastError();
}

cudaError_t launch_cache_copy_pages(const CacheView& c, int64_t D, const int32_t* src, const int32_t* dst, int64_t n,
                                    int* dev_err, cudaStream_t stream) {
  const int64_t scales = static_cast<int64_t>(c.H) * c.blocks_per_page;
  const int64_t bytes = scales * kCacheBlock * D;
  const int64_t chunks = div_up(bytes, kCopyChunk);
  const int smem = static_cast<int>((c.num_pages + 31) / 32 * 4);
  cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(cache_copy_kernel), smem);
  if (e != cudaSuccess) return e;
  const int64_t work = n * 2 * chunks, most = int64_t(8) * sm_count_current();
  cache_copy_kernel<<<static_cast<unsigned>(work < most ? work : most), kCopyThreads, smem, stream>>>(
      c, src, dst, n, bytes, scales, chunks, dev_err);
  return cudaGetLastError();
}

}  // namespace sage
