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

// Packed pairs of fp32.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  return static_cast<uint64_t>(__float_as_uint(hi)) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ float pair_lo(uint64_t p) { return __uint_as_float(static_cast<uint32_t>(p)); }
__device__ __forceinline__ float pair_hi(uint64_t p) { return __uint_as_float(static_cast<uint32_t>(p >> 32)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// Eight codes, rint(x / s) with the division correctly rounded, from eight
// BF16 values. Instead of dividing eight times: with inv = 1 / s rounded once,
// y = x * inv is within 2^-23 of x / s (relative), and y + (x - y s) inv rounds
// a number within 2^-46 of it; the same once more is x / s correctly rounded
// (Markstein's theorem: inv is correctly rounded, and the residual of a quotient
// within one step is exact under a fused multiply-add).
// Once is enough for the code unless s, a 24-bit integer times a power of two,
// is within 7 of a multiple of 2^17: codes turn at h = H / 2 plus or minus half
// a step of fp32 there (H odd, below 2^8), that is at (H 2^t +- 1) / 2^(t + 1),
// t >= 17. For x = X 2^a (X < 2^8) and s = S 2^b to fall within 2^-46 of that,
// |X 2^n - (H 2^t +- 1) S| < 2^-46 2^49 = 8 with X 2^n above 2^47, so a multiple
// of 2^39, hence S within 7 of a multiple of 2^t. (All scales of a block's
// values are one, so this is asked once.)
// The theorem wants no residual below the range: [kScaleLow, kScaleHigh] keeps
// it there; other scales divide. Adding 1.5 * 2^23 leaves the rounded integer in
// the low byte.
constexpr float kScaleLow = 0x1p-90f, kScaleHigh = 0x1p+100f;

__device__ __forceinline__ uint2 quantize8(const uint4& x, float s, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t m[8];
  if (s >= kScaleLow && s <= kScaleHigh) {
    const uint64_t magic = pair(12582912.0f, 12582912.0f), inv2 = pair(inv, inv), minus_s = pair(-s, -s);
    uint64_t y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint64_t v = pair(bf16_lo(w[e]), bf16_hi(w[e]));
      y[e] = mul2(v, inv2);
      y[e] = fma2(fma2(y[e], minus_s, v), inv2, y[e]);
    }
    if (((__float_as_uint(s) + 32u) & 0xFFFFu) < 64u) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        y[e] = fma2(fma2(y[e], minus_s, pair(bf16_lo(w[e]), bf16_hi(w[e]))), inv2, y[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y[e] = add2(y[e], magic);
      m[2 * e] = static_cast<uint32_t>(y[e]);
      m[2 * e + 1] = static_cast<uint32_t>(y[e] >> 32);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      m[2 * e] = static_cast<uint32_t>(quantize_one(bf16_lo(w[e]), s));
      m[2 * e + 1] = static_cast<uint32_t>(quantize_one(bf16_hi(w[e]), s));
    }
  }
  return make_uint2(__byte_perm(__byte_perm(m[0], m[1], 0x0040), __byte_perm(m[2], m[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(m[4], m[5], 0x0040), __byte_perm(m[6], m[7], 0x0040), 0x5410));
}

// The block that blockIdx.x stands for in sequence blockIdx.z, and the tokens
// of the call that fall into it.
struct Span {
  int64_t slot;   // block number in the cache, -1: nothing to do
  int t0;         // the call's token in the block's slot 0 (negative: older tokens come first)
  int first, end; // slots [first, end) hold the call's tokens
};

__device__ __forceinline__ Span find_span(const CacheView& c, const PageTable& pt, const int32_t* starts,
                                          const int32_t* counts, int32_t T, int* dev_err) {
  const int b = static_cast<int>(blockIdx.z);
  Span s;
  s.slot = -1;
  bool bad = false;
  // lengths are 32-bit, and so is every number of tokens and blocks below
  const int32_t capacity = static_cast<int32_t>(table_capacity(pt.max_pages, c.blocks_per_page));
  const int32_t start = static_cast<int32_t>(checked_length(starts[b], capacity, &bad));
  int32_t n = counts != nullptr ? static_cast<int32_t>(checked_length(counts[b], T, &bad)) : T;
  n = static_cast<int32_t>(checked_length(n, capacity - start, &bad));
  const uint32_t blk = static_cast<uint32_t>(start) / kCacheBlock + blockIdx.x;
  s.t0 = static_cast<int>(blk * kCacheBlock - static_cast<uint32_t>(start));
  s.first = s.t0 < 0 ? -s.t0 : 0;
  s.end = min(n - s.t0, kCacheBlock);
  if (s.end > s.first) {
    const uint32_t in_seq = blk / static_cast<uint32_t>(c.blocks_per_page);
    const int64_t page = pt.table[b * pt.stride + in_seq];
    if (page_ok(page, c.num_pages))
      s.slot = block_slot(page, static_cast<int32_t>(blockIdx.y), c.H, c.blocks_per_page,
                          static_cast<int32_t>(blk - in_seq * static_cast<uint32_t>(c.blocks_per_page)));
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
// values. A call of many tokens is bound by instructions more than by HBM: 69
// us for 16 sequences of up to 4096 tokens, 8 heads of 128, where the bytes
// alone take 45; with eight plain divisions a thread it was 118, and the
// numbers of tokens and blocks in 64 bits cost another 14. Five CTAs to an SM
// (48 registers): with six the same call is 1 us quicker, but 64 single tokens
// take 0.7 us longer; with eight the registers spill (+3 us).
// kFew: calls of at most a block's tokens, whose time is that of loads that
// wait for one another. The older tokens' codes, should the scale grow, are
// asked for before that is known: 64 single tokens, appended and read back,
// 10.1 -> 9.2 us; in a call of many tokens the registers cost 2 us of 69.
template <int D, bool kFew>
__global__ void __launch_bounds__(kThreads, kFew ? 4 : 5) cache_append_kernel(CacheView c, PageTable pt, const int32_t* starts,
                                                                const int32_t* counts, Bf16In k, Bf16In v, int32_t T,
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
  const uint16_t* src = in.p + static_cast<int64_t>(blockIdx.z) * in.sb + static_cast<int64_t>(blockIdx.y) * in.sh + ch +
                        (s.t0 + row0) * in.ss;
  const int64_t step = L::kRows * in.ss;
  uint4 x[L::kTimes];
#pragma unroll
  for (int q = 0; q < L::kTimes; ++q) {
    const int row = q * L::kRows + row0;
    x[q] = make_uint4(0u, 0u, 0u, 0u);
    if (row >= s.first && row < s.end) x[q] = *reinterpret_cast<const uint4*>(src + q * step);
  }
  int8_t* block = (half ? c.v : c.k) + s.slot * (kCacheBlock * D);
  const int quad = i >> 2, g = i & 3;  // values: channels 4 quad .. + 3, positions 8 g .. + 7
  // codes of the block's older tokens: of the keys of row e * kRows + row0, of the values of channel 4 quad + e
  const auto older = [&](int e) {
    return *reinterpret_cast<const uint2*>(
        half ? block + (4 * quad + e) * kCacheBlock + 8 * g
             : block + (ch / 64) * (kCacheBlock * 64) + (e * L::kRows + row0) * 64 + ch % 64);
  };
  uint2 was[4];
  if (kFew && s.first > 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (half ? i < L::kQuads : e < L::kTimes && e * L::kRows + row0 < s.first) was[e] = older(e);
  }
  // max |x| as bit patterns: those of infinities and NaN are the largest
  uint32_t a = 0;
#pragma unroll
  for (int q = 0; q < L::kTimes; ++q) {
    const uint32_t w[4] = {x[q].x, x[q].y, x[q].z, x[q].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) a = __vmaxu2(a, w[e] & 0x7FFF7FFFu);
  }
  a = __reduce_max_sync(0xffffffffu, max(a & 0xFFFFu, a >> 16));
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
  const float inv = __fdiv_rn(1.0f, s_new);
#pragma unroll
  for (int q = 0; q < L::kTimes; ++q) {
    const int row = q * L::kRows + row0;
    uint2 codes = make_uint2(0u, 0u);
    if (usable && row >= s.first && row < s.end) codes = quantize8(x[q], s_new, inv);
    if (half == 0) {
      uint2* p = reinterpret_cast<uint2*>(block + (ch / 64) * (kCacheBlock * 64) + row * 64 + ch % 64);
      if (row >= s.first) {
        *p = codes;
      } else if (grew) {
        const uint2 old = kFew ? was[q] : older(q);
        *p = make_uint2(shrink4(old.x, shrink), shrink4(old.y, shrink));
      }
    } else {
      *reinterpret_cast<uint2*>(vt + row * L::kPitch + ch) = codes;
    }
  }
  __syncthreads();
  if (half == 1 && i < L::kQuads) {
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
        uint2 old = kFew ? was[e] : older(e);
        if (grew) old = make_uint2(shrink4(old.x, shrink), shrink4(old.y, shrink));
        uint32_t keep_lo = 0, keep_hi = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if (value_token(8 * g + b) < s.first) keep_lo |= 255u << (8 * b);
          if (value_token(8 * g + 4 + b) < s.first) keep_hi |= 255u << (8 * b);
        }
        o = make_uint2((old.x & keep_lo) | (o.x & ~keep_lo), (old.y & keep_hi) | (o.y & ~keep_hi));
      }
      *p = o;
    }
  }
}

// -------------------------------------------------------------------- read --

// Two codes times the scale, rounded to BF16 once. u: the codes plus 128, as
// unsigned bytes; a byte under the exponent of 2^23 is the fp32 2^23 + u, whose
// difference with 2^23 + 128 is the code, exactly: two byte permutes and half
// an instruction in place of a conversion at a quarter of the rate.
__device__ __forceinline__ uint32_t to_bf16x2(uint32_t u, int at, uint64_t scale2) {
  const uint64_t bias = pair(-8388736.0f, -8388736.0f);
  const uint32_t lo = __byte_perm(u, 0x4B000000u, 0x7440 + at), hi = __byte_perm(u, 0x4B000000u, 0x7441 + at);
  const uint64_t x = mul2(add2(static_cast<uint64_t>(hi) << 32 | lo, bias), scale2);
  const __nv_bfloat162 r = __floats2bfloat162_rn(pair_lo(x), pair_hi(x));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The same blocks the other way. 8 sequences of 8000 tokens, 8 heads of 128:
// 61 us, 6.4 TB/s; with six CTAs to an SM in place of eight 65 us, and 68 with
// conversions of integers and numbers of tokens in 64 bits.
template <int D>
__global__ void __launch_bounds__(kThreads, 8) cache_read_kernel(CacheView c, PageTable pt, const int32_t* starts,
                                                              const int32_t* counts, Out k, Out v, int32_t T,
                                                              bool zero_rest, int* dev_err) {
  using L = Tile<D>;
  __shared__ __align__(16) uint8_t vt[kCacheBlock * L::kPitch];
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const Span s = find_span(c, pt, starts, counts, T, dev_err);
  const int half = threadIdx.x >> 7, i = threadIdx.x & 127;
  const int ch = (i % L::kLanes) * 8, row0 = i / L::kLanes;
  const Out& o = half ? v : k;
  uint16_t* dst = o.p + static_cast<int64_t>(blockIdx.z) * o.sb + static_cast<int64_t>(blockIdx.y) * o.sh + ch +
                  (s.t0 + row0) * o.ss;
  const int64_t step = L::kRows * o.ss;
  if (zero_rest) {
#pragma unroll
    for (int q = 0; q < L::kTimes; ++q) {
      const int row = q * L::kRows + row0;
      if (row >= s.first && s.t0 + row < T && (row >= s.end || s.slot < 0))
        *reinterpret_cast<uint4*>(dst + q * step) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (s.slot < 0) return;
  const float scale = (half ? c.vs : c.ks)[s.slot];
  const uint64_t scale2 = pair(scale, scale);
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
    uint2 w = half ? *reinterpret_cast<const uint2*>(vt + row * L::kPitch + ch) : codes[q];
    w.x ^= 0x80808080u;
    w.y ^= 0x80808080u;
    *reinterpret_cast<uint4*>(dst + q * step) =
        make_uint4(to_bf16x2(w.x, 0, scale2), to_bf16x2(w.x, 2, scale2), to_bf16x2(w.y, 0, scale2),
                   to_bf16x2(w.y, 2, scale2));
  }
}

// -------------------------------------------------------------------- copy --
// Page dst[i] becomes a copy of page src[i]. An entry with a negative dst, or
// with src = dst, stands for nothing. No page may be named twice as dst, nor as
// dst of one entry and src of another: the copies would depend on their order.
// Every CTA checks the whole lists with one bit per page in shared memory
// before it copies anything, so a list that breaks the rule, or names a page
// that is not there, moves no byte and sets the device error word.
// Each warp moves its chunks through shared memory with bulk copies, one after
// the other; kCopyWarps of them in flight per SM are what HBM needs, and no
// register holds a byte of them. The first is on its way while the lists are
// checked. 2000 pages of 64 tokens, 8 heads of 128: 87 us, 6.0 TB/s read and
// written (102 us through registers, with 64 KB in flight per SM); 16 pages of 4
// heads: 3.1 us (2.7). 6 warps of 32768 bytes, 12 of 16384 and 24 of 8192
// measure 88, 86 and 91.
constexpr int kCopyWarps = 8;
constexpr int kCopyThreads = 32 * kCopyWarps;
constexpr int kCopyChunk = 16384;        // bytes of codes that a warp moves at a time
constexpr int kCopySmall = 4096;       // where there are fewer of them than warps, or no room
constexpr int kCopyBits = 227 * 1024 - 256 - kCopyWarps * kCopyChunk;
static_assert(kCopyWarps * kCopySmall + (1 << 17) <= 227 * 1024 - 256, "a bit for each of 2^20 pages");
constexpr int kCheckAtOnce = 8;        // entries whose loads a thread has in flight
constexpr uint64_t kCopyTimeoutNs = 2000000000ull;

struct CopyUnit {
  const int8_t* from;  // null: nothing to move
  int8_t* to;
  uint32_t bytes;
  int32_t s, d;        // pages
  int which;           // 0 keys, 1 values
  bool first;          // the page's first chunk: its scales go with it
};

__device__ __forceinline__ CopyUnit copy_unit(const CacheView& c, const int32_t* src, const int32_t* dst,
                                              int64_t codes_bytes, int chunk, int64_t chunks, int64_t u) {
  const int64_t entry = u / (2 * chunks);
  const int64_t r = u - entry * 2 * chunks;
  CopyUnit m;
  m.s = src[entry];
  m.d = dst[entry];
  m.which = r >= chunks;
  const int64_t lo = (r - (m.which ? chunks : 0)) * chunk;
  m.first = lo == 0;
  m.bytes = static_cast<uint32_t>(min(codes_bytes - lo, static_cast<int64_t>(chunk)));
  int8_t* base = m.which ? c.v : c.k;
  const bool moves = m.d >= 0 && m.d != m.s && page_ok(m.s, c.num_pages);
  m.from = moves ? base + m.s * codes_bytes + lo : nullptr;
  m.to = base + m.d * codes_bytes + lo;
  return m;
}

__global__ void __launch_bounds__(kCopyThreads) cache_copy_kernel(CacheView c, const int32_t* src, const int32_t* dst,
                                                                  int64_t n, int64_t codes_bytes, int64_t scales,
                                                                  int chunk, int64_t chunks, int* dev_err) {
  extern __shared__ __align__(128) uint8_t buffers[];  // a chunk per warp, then a bit per page
  __shared__ uint64_t landed[kCopyWarps];
  uint32_t* taken = reinterpret_cast<uint32_t*>(buffers + kCopyWarps * chunk);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar = tc::smem_u32(&landed[warp]), buffer = tc::smem_u32(buffers) + static_cast<uint32_t>(warp * chunk);
  if (lane == 0) {
    tc::mbar_init(bar, 1);
    tc::fence_mbar_init();
  }
  __syncwarp();
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int64_t total = n * 2 * chunks, step = static_cast<int64_t>(gridDim.x) * kCopyWarps;
  int64_t u = blockIdx.x + static_cast<int64_t>(warp) * gridDim.x;
  const auto fetch = [&](const CopyUnit& m) {
    if (lane != 0 || m.from == nullptr) return;
    tc::fence_proxy_async_global();  // earlier kernels wrote the page
    tc::mbar_arrive_expect_tx(bar, m.bytes);
    tc::bulk_load(buffer, m.from, m.bytes, bar);
  };
  uint32_t phase = 0;
  const auto wait = [&]() {
    uint64_t t0 = 0;
    for (uint32_t it = 1; !tc::mbar_try_wait(bar, phase & 1u); ++it) {
      if ((it & 127u) != 0) continue;
      const uint64_t now = tc::global_timer_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > kCopyTimeoutNs) return false;
    }
    ++phase;
    return true;
  };
  CopyUnit m;
  m.from = nullptr;
  if (u < total) {
    m = copy_unit(c, src, dst, codes_bytes, chunk, chunks, u);
    fetch(m);
  }
  const int words = static_cast<int>((c.num_pages + 31) / 32);
  for (int i = threadIdx.x; i < words; i += kCopyThreads) taken[i] = 0u;
  __syncthreads();
  bool bad = false;
  for (int64_t i0 = threadIdx.x; i0 < n; i0 += kCheckAtOnce * kCopyThreads) {
    int32_t d[kCheckAtOnce], s[kCheckAtOnce];
#pragma unroll
    for (int y = 0; y < kCheckAtOnce; ++y) {
      const int64_t i = i0 + y * kCopyThreads;
      d[y] = i < n ? dst[i] : -1;
      s[y] = i < n ? src[i] : -1;
    }
#pragma unroll
    for (int y = 0; y < kCheckAtOnce; ++y) {
      if (d[y] < 0 || d[y] == s[y]) continue;
      if (!page_ok(d[y], c.num_pages) || !page_ok(s[y], c.num_pages)) bad = true;
      else if (atomicOr(&taken[d[y] >> 5], 1u << (d[y] & 31)) >> (d[y] & 31) & 1u) bad = true;
    }
  }
  __syncthreads();
  for (int64_t i0 = threadIdx.x; i0 < n; i0 += kCheckAtOnce * kCopyThreads) {
    int32_t d[kCheckAtOnce], s[kCheckAtOnce];
#pragma unroll
    for (int y = 0; y < kCheckAtOnce; ++y) {
      const int64_t i = i0 + y * kCopyThreads;
      d[y] = i < n ? dst[i] : -1;
      s[y] = i < n ? src[i] : -1;
    }
#pragma unroll
    for (int y = 0; y < kCheckAtOnce; ++y)
      if (d[y] >= 0 && d[y] != s[y] && page_ok(s[y], c.num_pages) && (taken[s[y] >> 5] >> (s[y] & 31) & 1u)) bad = true;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) flag_pages(dev_err);
    if (m.from != nullptr && !wait() && lane == 0) atomicExch(dev_err, kDevErrTimeout);
    return;  // with no copy in flight
  }
  while (u < total) {
    // where the next chunk is, looked up under this one's copy
    CopyUnit next;
    next.from = nullptr;
    if (u + step < total) next = copy_unit(c, src, dst, codes_bytes, chunk, chunks, u + step);
    if (m.from != nullptr) {
      if (m.first) {
        float* sc = m.which ? c.vs : c.ks;
        for (int64_t q = lane; q < scales; q += 32) sc[m.d * scales + q] = sc[m.s * scales + q];
      }
      if (!wait()) {
        if (lane == 0) atomicExch(dev_err, kDevErrTimeout);
        break;
      }
      if (lane == 0) {
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                         reinterpret_cast<uint64_t>(m.to)),
                     "r"(buffer), "r"(m.bytes)
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the buffer has been read
      }
      __syncwarp();
    }
    u += step;
    m = next;
    fetch(m);
  }
  if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
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
  const bool few = T <= kCacheBlock;
  const auto kernel = D == 128 ? (few ? cache_append_kernel<128, true> : cache_append_kernel<128, false>)
                               : (few ? cache_append_kernel<64, true> : cache_append_kernel<64, false>);
  return launch(kernel, span_grid(c, B, T), kThreads, 0, stream, c,
                pt, starts, counts, k, v, static_cast<int32_t>(T), dev_err);
}

cudaError_t launch_cache_read(const CacheView& c, int64_t D, const PageTable& pt, const int32_t* starts,
                              const int32_t* counts, const Out& k, const Out& v, int64_t B, int64_t T,
                              bool zero_rest, int* dev_err, cudaStream_t stream) {
  return launch(D == 128 ? cache_read_kernel<128> : cache_read_kernel<64>, span_grid(c, B, T), kThreads, 0, stream, c, pt,
                starts, counts, k, v, static_cast<int32_t>(T), zero_rest, dev_err);
}

cudaError_t launch_cache_copy_pages(const CacheView& c, int64_t D, const int32_t* src, const int32_t* dst, int64_t n,
                                    int* dev_err, cudaStream_t stream) {
  const int64_t scales = static_cast<int64_t>(c.H) * c.blocks_per_page;
  const int64_t bytes = scales * kCacheBlock * D;
  const int64_t warps = static_cast<int64_t>(sm_count_current()) * kCopyWarps;
  const int bits = static_cast<int>((c.num_pages + 31) / 32 * 4);
  const int chunk = n * 2 * div_up(bytes, kCopyChunk) < warps || bits > kCopyBits ? kCopySmall : kCopyChunk;
  const int64_t chunks = div_up(bytes, chunk);
  const int smem = kCopyWarps * chunk + bits;
  cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(cache_copy_kernel), smem);
  if (e != cudaSuccess) return e;
  const int64_t work = n * 2 * chunks, most = sm_count_current();
  return launch(cache_copy_kernel, dim3(static_cast<unsigned>(work < most ? work : most)), kCopyThreads,
                static_cast<size_t>(smem), stream, c, src, dst, n, bytes, scales, chunk, chunks, dev_err);
}

}  // namespace sage
