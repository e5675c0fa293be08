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
#include "tc_ptx.cuh"

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

// A token's D channels are D / 8 lanes wide, 16 bytes of BF16 and 8 codes a
// lane, so 128 threads cover kRows tokens at a time and every access to global
// memory is whole sectors. Value codes change between token rows and channel
// rows in shared memory, four channels by eight positions to a thread.
template <int D>
struct Tile {
  static constexpr int kLanes = D / 8;           // lanes of a token
  static constexpr int kRows = 128 / kLanes;     // tokens at a time
  static constexpr int kTimes = kCacheBlock / kRows;
  static constexpr int kPitch = D + 16;          // bytes of a token row in shared memory: no bank conflicts
  static constexpr int kQuads = D;               // units of 4 channels x 8 positions: D / 4 x 4
};

// Bytes 4 x 4: out[p] gets byte p of w0..w3.
__device__ __forceinline__ void transpose4(const uint32_t (&w)[4], uint32_t (&out)[4]) {
  const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[2], w[3], 0x5140);
  const uint32_t c = __byte_perm(w[0], w[1], 0x7362), d = __byte_perm(w[2], w[3], 0x7362);
  out[0] = __byte_perm(a, b, 0x5410);
  out[1] = __byte_perm(a, b, 0x7632);
  out[2] = __byte_perm(c, d, 0x5410);
  out[3] = __byte_perm(c, d, 0x7632);
}

__device__ __forceinline__ uint32_t shrink4(uint32_t w, float r) {
  uint32_t o = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    o |= (static_cast<uint32_t>(static_cast<int>(rintf(static_cast<int8_t>(w >> (8 * e)) * r))) & 255u) << (8 * e);
  return o;
}

// ------------------------------------------------------------------ append --
// One CTA writes one block of one head: threads 0..127 its keys, 128..255 its
// values.
template <int D>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(CacheView c, PageTable pt, const int32_t* starts,
                                                                const int32_t* counts, Bf16In k, Bf16In v, int64_t T,
                                                                int* dev_err) {
  using L = Tile<D>;
  __shared__ __align__(16) uint8_t vt[kCacheBlock * L::kPitch];
  __shared__ uint32_t amax_w[8];
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const Span s = find_span(c, pt, starts, counts, T, dev_err);
  if (s.slot < 0) return;
  const int half = threadIdx.x >> 7, i = threadIdx.x & 127;
  const int ch = (i % L::kLanes) * 8, row0 = i / L::kLanes;
  const Bf16In& in = half ? v : k;
  float* scale_at = (half ? c.vs : c.ks) + s.slot;
  const float s_old = s.first > 0 ? *scale_at : 0.0f;
  const uint16_t* src = in.p + static_cast<int64_t>(blockIdx.z) * in.sb + static_cast<int64_t>(blockIdx.y) * in.sh + ch;
  uint4 x[L::kTimes];
#pragma unroll
  for (int q = 0; q < L::kTimes; ++q) {
    const int row = q * L::kRows + row0;
    x[q] = make_uint4(0u, 0u, 0u, 0u);
    if (row >= s.first && row < s.end) x[q] = *reinterpret_cast<const uint4*>(src + (s.t0 + row) * in.ss);
  }
  // max |x| as bit patterns: those of infinities and NaN are the largest
  uint32_t a = 0;
#pragma unroll
  for (int q = 0; q < L::kTimes; ++q) {
    const uint32_t w[4] = {x[q].x, x[q].y, x[q].z, x[q].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) a = max(a, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
  }
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
#pragma unroll
  for (int q = 0; q < L::kTimes; ++q) {
    const int row = q * L::kRows + row0;
    uint2 codes = make_uint2(0u, 0u);
    if (usable && row >= s.first && row < s.end) {
      codes.x = pack4(quantize_one(bf16_lo(x[q].x), s_new), quantize_one(bf16_hi(x[q].x), s_new),
                      quantize_one(bf16_lo(x[q].y), s_new), quantize_one(bf16_hi(x[q].y), s_new));
      codes.y = pack4(quantize_one(bf16_lo(x[q].z), s_new), quantize_one(bf16_hi(x[q].z), s_new),
                      quantize_one(bf16_lo(x[q].w), s_new), quantize_one(bf16_hi(x[q].w), s_new));
    }
    if (half == 0) {
      uint2* p = reinterpret_cast<uint2*>(block + (ch / 64) * (kCacheBlock * 64) + row * 64 + ch % 64);
      if (row >= s.first) {
        *p = codes;
      } else if (grew) {
        const uint2 was = *p;
        *p = make_uint2(shrink4(was.x, shrink), shrink4(was.y, shrink));
      }
    } else {
      *reinterpret_cast<uint2*>(vt + row * L::kPitch + ch) = codes;
    }
  }
  __syncthreads();
  if (half == 1 && i < L::kQuads) {
    const int quad = i >> 2, g = i & 3;  // channels 4 quad .. + 3, positions 8 g .. + 7
    uint32_t lo[4], hi[4], w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = *reinterpret_cast<const uint32_t*>(vt + value_token(8 * g + e) * L::kPitch + 4 * quad);
    transpose4(w, lo);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = *reinterpret_cast<const uint32_t*>(vt + value_token(8 * g + 4 + e) * L::kPitch + 4 * quad);
    transpose4(w, hi);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint2* p = reinterpret_cast<uint2*>(block + (4 * quad + e) * kCacheBlock + 8 * g);
      uint2 o = make_uint2(lo[e], hi[e]);
      if (s.first > 0) {
        // older tokens' codes stay in the block
        uint2 was = *p;
        if (grew) was = make_uint2(shrink4(was.x, shrink), shrink4(was.y, shrink));
        uint32_t keep_lo = 0, keep_hi = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if (value_token(8 * g + b) < s.first) keep_lo |= 255u << (8 * b);
          if (value_token(8 * g + 4 + b) < s.first) keep_hi |= 255u << (8 * b);
        }
        o = make_uint2((was.x & keep_lo) | (o.x & ~keep_lo), (was.y & keep_hi) | (o.y & ~keep_hi));
      }
      *p = o;
    }
  }
}

// -------------------------------------------------------------------- read --

__device__ __forceinline__ uint32_t to_bf16x2(uint32_t codes, int at, float scale) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(static_cast<int8_t>(codes >> (8 * at)) * scale,
                                                 static_cast<int8_t>(codes >> (8 * at + 8)) * scale);
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <int D>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(CacheView c, PageTable pt, const int32_t* starts,
                                                              const int32_t* counts, Out k, Out v, int64_t T,
                                                              bool zero_rest, int* dev_err) {
  using L = Tile<D>;
  __shared__ __align__(16) uint8_t vt[kCacheBlock * L::kPitch];
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const Span s = find_span(c, pt, starts, counts, T, dev_err);
  const int half = threadIdx.x >> 7, i = threadIdx.x & 127;
  const int ch = (i % L::kLanes) * 8, row0 = i / L::kLanes;
  const Out& o = half ? v : k;
  uint16_t* dst = o.p + static_cast<int64_t>(blockIdx.z) * o.sb + static_cast<int64_t>(blockIdx.y) * o.sh + ch;
  if (zero_rest) {
#pragma unroll
    for (int q = 0; q < L::kTimes; ++q) {
      const int row = q * L::kRows + row0;
      if (row >= s.first && s.t0 + row < T && (row >= s.end || s.slot < 0))
        *reinterpret_cast<uint4*>(dst + (s.t0 + row) * o.ss) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (s.slot < 0) return;
  const float scale = (half ? c.vs : c.ks)[s.slot];
  const int8_t* block = (half ? c.v : c.k) + s.slot * (kCacheBlock * D);
  uint2 codes[L::kTimes];
  if (half == 0) {
#pragma unroll
    for (int q = 0; q < L::kTimes; ++q)
      codes[q] = *reinterpret_cast<const uint2*>(block + (ch / 64) * (kCacheBlock * 64) + (q * L::kRows + row0) * 64 + ch % 64);
  } else if (i < L::kQuads) {
    const int quad = i >> 2, g = i & 3;
    uint2 x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      x[e] = *reinterpret_cast<const uint2*>(block + (4 * quad + e) * kCacheBlock + 8 * g);
    uint32_t w[4], t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = x[e].x;
    transpose4(w, t);
#pragma unroll
    for (int e = 0; e < 4; ++e) *reinterpret_cast<uint32_t*>(vt + value_token(8 * g + e) * L::kPitch + 4 * quad) = t[e];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = x[e].y;
    transpose4(w, t);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<uint32_t*>(vt + value_token(8 * g + 4 + e) * L::kPitch + 4 * quad) = t[e];
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < L::kTimes; ++q) {
    const int row = q * L::kRows + row0;
    if (row < s.first || row >= s.end) continue;
    const uint2 w = half ? *reinterpret_cast<const uint2*>(vt + row * L::kPitch + ch) : codes[q];
    *reinterpret_cast<uint4*>(dst + (s.t0 + row) * o.ss) =
        make_uint4(to_bf16x2(w.x, 0, scale), to_bf16x2(w.x, 2, scale), to_bf16x2(w.y, 0, scale), to_bf16x2(w.y, 2, scale));
  }
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
  tc::griddep_wait();
  tc::griddep_launch_dependents();
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
    // a whole chunk is eight 16-byte pieces per thread, all in flight at once
    uint4 x[kCopyChunk / 16 / kCopyThreads];
#pragma unroll
    for (int y = 0; y < kCopyChunk / 16 / kCopyThreads; ++y) {
      const int64_t q = lo / 16 + threadIdx.x + y * kCopyThreads;
      if (q < hi / 16) x[y] = from[q];
    }
#pragma unroll
    for (int y = 0; y < kCopyChunk / 16 / kCopyThreads; ++y) {
      const int64_t q = lo / 16 + threadIdx.x + y * kCopyThreads;
      if (q < hi / 16) to[q] = x[y];
    }
    if (chunk == 0) {
      float* sc = which ? c.vs : c.ks;
      for (int64_t q = threadIdx.x; q < scales; q += kCopyThreads) sc[d * scales + q] = sc[s * scales + q];
    }
  }
}

// Launched as a programmatic dependent: the grid may come up while the stream's
// previous kernel still runs; it waits for it before it reads anything.
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
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
  return launch(D == 128 ? cache_append_kernel<128> : cache_append_kernel<64>, span_grid(c, B, T), kThreads, 0, stream, c,
                pt, starts, counts, k, v, T, dev_err);
}

cudaError_t launch_cache_read(const CacheView& c, int64_t D, const PageTable& pt, const int32_t* starts,
                              const int32_t* counts, const Out& k, const Out& v, int64_t B, int64_t T,
                              bool zero_rest, int* dev_err, cudaStream_t stream) {
  return launch(D == 128 ? cache_read_kernel<128> : cache_read_kernel<64>, span_grid(c, B, T), kThreads, 0, stream, c, pt,
                starts, counts, k, v, T, zero_rest, dev_err);
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
  return launch(cache_copy_kernel, dim3(static_cast<unsigned>(work < most ? work : most)), kCopyThreads,
                static_cast<size_t>(smem), stream, c, src, dst, n, bytes, scales, chunks, dev_err);
}

}  // namespace sage
