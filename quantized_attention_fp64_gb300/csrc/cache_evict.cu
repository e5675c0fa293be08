// Cutting cached sequences back: selection of the tokens that stay, and their
// moving together.
//
// Selection: a CTA has one head of a sequence. Scores become integers of the same
// order (a NaN the lowest, -0 like 0), in shared memory where they fit. The last
// one that stays is found digit by digit (11, 11 and 10 bits from the top), each
// time from a histogram of the next digit of the scores that agree with what is
// known; everything above it stays, and of those equal to it the first ones. Then
// every warp counts what stays of its part of the sequence, and writes it behind
// what stays before.
//
// Moving: a warp has 32 new places (a block) of one head's keys or values. It
// reads only blocks that hold a kept token: keys row by row, values (channels by
// tokens) a whole block at a time, a lane with all 32 bytes of a channel. What
// bounds it is HBM, and the instructions that pick single bytes out of the values
// and round the codes again. 16 sequences of 8 heads, D = 128, cut from up to 16001 to
// 4096 tokens: selection 21 us (one CTA a head: a chain of three digits), moves 81 us,
// of which 358 MB from and to HBM need 53 (4.4 TB/s); in place 86.
// In place, kept tokens never move to a later place: block m is written by the
// warp that has places 32 m .. 32 m + 31, and its old tokens are read by the
// warps whose places they go to, which are m or before. So a warp reads first,
// says so in a word of the workspace, and waits for the words of those at most 32
// blocks before it writes. Blocks are handed out in order, and no warp waits
// before it has read: the wait ends, whatever else runs on the GPU.
#include "cache.cuh"
#include "launch.cuh"
#include "tc_kernel.cuh"

namespace sage {
namespace {

constexpr int kBins = 2048;
constexpr int kMoveWarps = 4;
constexpr int kStaged = 48 * 1024;  // scores of a head that shared memory holds

// Integers in the order of the scores, and back (-0 comes back as 0).
__device__ __forceinline__ float score_of(uint32_t u) {
  return __uint_as_float(u == 0u ? 0x7FC00000u : u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
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

// The workspace: a ticket, then for each head of a sequence the kept tokens in
// front of each of its blocks, then a word for each new block of keys and values.
struct Work {
  uint32_t* ticket;
  int32_t* before;   // [B * H][old_blocks + 1]
  uint32_t* read;    // [B * H][2][new_blocks]
  int32_t old_blocks, new_blocks;
};

__host__ __device__ inline int32_t blocks_in(int32_t tokens) { return tokens / kCacheBlock + (tokens % kCacheBlock != 0 ? 1 : 0); }

Work work_of(const CacheEvictArgs& a) {
  Work w;
  w.old_blocks = blocks_in(a.scores_n);
  w.new_blocks = blocks_in(a.keep);
  w.ticket = static_cast<uint32_t*>(a.workspace);
  w.before = reinterpret_cast<int32_t*>(w.ticket + 64);
  w.read = reinterpret_cast<uint32_t*>(w.before + a.B * a.c.H * (static_cast<int64_t>(w.old_blocks) + 1));
  return w;
}

// An exclusive sum over the block's threads, of two values; `sums` [2][33].
template <int kThreads>
__device__ __forceinline__ void sum_before(uint32_t& x, uint32_t& y, uint32_t (&sums)[2][33]) {
  const int lane = static_cast<int>(threadIdx.x) & 31, warp = static_cast<int>(threadIdx.x) >> 5;
  uint32_t sx = x, sy = y;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const uint32_t px = __shfl_up_sync(0xffffffffu, sx, s), py = __shfl_up_sync(0xffffffffu, sy, s);
    if (lane >= s) sx += px, sy += py;
  }
  if (lane == 31) sums[0][warp] = sx, sums[1][warp] = sy;
  __syncthreads();
  uint32_t bx = 0, by = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w)
    if (w < warp) bx += sums[0][w], by += sums[1][w];
  x = bx + sx - x;
  y = by + sy - y;
  __syncthreads();
}

template <int kThreads, bool kStage>
__global__ void __launch_bounds__(kThreads) select_kernel(const CacheEvictArgs a, const Work work, bool in_place) {
  extern __shared__ uint32_t keys[];  // kStage: the scores as integers
  __shared__ uint32_t count[kBins];
  __shared__ uint32_t sums[2][33];
  __shared__ uint32_t found[2];
  tc::griddep_launch_dependents();
  tc::griddep_wait();
  const int b = static_cast<int>(blockIdx.y), h = static_cast<int>(blockIdx.x);
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  const int32_t len = length_of(a, b, &bad);
  if (bad && tid == 0) atomicExch(a.dev_err, kDevErrPage);
  const int32_t stay = min(len, a.keep);
  if (h == 0 && tid == 0) a.lengths_out[b] = stay;
  if (h == 0 && b == 0 && tid == 0) *work.ticket = 0;
  if (a.c.H == 0) return;
  const int32_t decided = len - min(a.recent, stay);  // the scores decide on those before
  const int32_t need = stay - (len - decided);        // and keep so many of them
  const bool open = need < decided;
  const int64_t head = static_cast<int64_t>(b) * a.c.H + h;
  const float* x = a.scores + b * a.scores_b + h * a.scores_h;
  int32_t* kept = a.kept + head * a.kept_n;
  float* moved = a.scores_out + head * a.scores_n;
  int32_t* before = work.before + head * (work.old_blocks + 1);
  if (in_place)
    for (int32_t i = tid; i < 2 * work.new_blocks; i += kThreads) work.read[head * 2 * work.new_blocks + i] = 0;
  if (kStage) {
#pragma unroll 8
    for (int32_t i = tid; i < len; i += kThreads) keys[i] = order_of(x[i]);
    // (each thread reads back what it wrote, until the barriers below)
  }
  const auto key = [&](int32_t i) { return kStage ? keys[i] : order_of(x[i]); };
  uint32_t known = 0, left = static_cast<uint32_t>(need);  // of the scores equal to `known`, keep `left`
  if (open && need > 0) {
    constexpr int kShift[3] = {21, 10, 0}, kBits[3] = {11, 11, 10};
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? kShift[0] : pass == 1 ? kShift[1] : kShift[2];
      const uint32_t mask = (1u << (pass == 2 ? kBits[2] : kBits[0])) - 1u;
      const int above = shift + (pass == 2 ? kBits[2] : kBits[0]);  // bits from here on are known
      for (int i = tid; i < kBins; i += kThreads) count[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int32_t i = tid; i < decided; i += kThreads) {
        const uint32_t u = key(i);
        if (pass == 0 || (u ^ known) >> above == 0) atomicAdd(&count[(u >> shift) & mask], 1u);
      }
      __syncthreads();
      // bins from the top: the one in which the left-th falls
      constexpr int kEach = kBins / kThreads;
      uint32_t own[kEach], sum = 0, none = 0;
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        own[e] = count[kBins - 1 - (tid * kEach + e)];
        sum += own[e];
      }
      sum_before<kThreads>(sum, none, sums);
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        if (sum < left && left <= sum + own[e]) {
          found[0] = static_cast<uint32_t>(kBins - 1 - (tid * kEach + e));
          found[1] = left - sum;
        }
        sum += own[e];
      }
      __syncthreads();
      known |= found[0] << shift;
      left = found[1];
    }
  }
  __syncthreads();
  // what stays of each warp's part: tokens surely, and those equal to the last one that stays
  const int32_t part = (blocks_in(len) + kThreads / 32 - 1) / (kThreads / 32) * kCacheBlock;
  const int32_t lo = min(len, warp * part), hi = min(len, lo + part);
  uint32_t sure = 0, same = 0;
#pragma unroll 4
  for (int32_t i = lo + lane; i < hi; i += 32) {
    const uint32_t u = open && i < decided ? key(i) : 0u;
    const bool s = !open || i >= decided || (need > 0 && u > known);
    sure += s ? 1u : 0u;
    same += !s && need > 0 && u == known ? 1u : 0u;
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    sure += __shfl_xor_sync(0xffffffffu, sure, s);
    same += __shfl_xor_sync(0xffffffffu, same, s);
  }
  if (lane == 0) sums[0][warp] = sure, sums[1][warp] = same;
  __syncthreads();
  // (of the equal ones before this warp's part, `left` at most stay)
  uint32_t place = lane < warp ? sums[0][lane] : 0u, equal = lane < warp ? sums[1][lane] : 0u;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    place += __shfl_xor_sync(0xffffffffu, place, s);
    equal += __shfl_xor_sync(0xffffffffu, equal, s);
  }
  place += min(left, equal);
  for (int32_t i0 = lo; i0 < hi; i0 += 32) {
    const int32_t i = i0 + lane;
    const uint32_t u = i < hi ? key(i) : 0u;
    const bool s = i < hi && (!open || i >= decided || (need > 0 && u > known));
    const bool e = i < hi && !s && need > 0 && u == known;
    const uint32_t equals = __ballot_sync(0xffffffffu, e);
    const bool stays = s || (e && equal + __popc(equals & ((1u << lane) - 1u)) < left);
    const uint32_t stay_mask = __ballot_sync(0xffffffffu, stays);
    if (lane == 0) before[i0 / kCacheBlock] = static_cast<int32_t>(place);
    if (stays) {
      const uint32_t at = place + __popc(stay_mask & ((1u << lane) - 1u));
      kept[at] = i;
      moved[at] = score_of(u);
    }
    place += __popc(stay_mask);
    equal += __popc(equals);
  }
  if (tid == 0) before[blocks_in(len)] = stay;
  for (int32_t i = stay + tid; i < a.kept_n; i += kThreads) kept[i] = -1;
  for (int32_t i = stay + tid; i < a.scores_n; i += kThreads) moved[i] = 0.0f;
}

// ------------------------------------------------------------------- moving --

// Four codes rounded again: rint(c * r), each product rounded to fp32 first.
// Adding 1.5 2^23 leaves the integer in the low byte; 2^23 + 128 + c is c with its
// sign bit turned over, behind the exponent of 2^23.
__device__ __forceinline__ uint32_t shrink4(uint32_t w, float r0, float r1, float r2, float r3) {
  const uint32_t u = w ^ 0x80808080u;
  const float2 off = make_float2(-8388736.0f, -8388736.0f), magic = make_float2(12582912.0f, 12582912.0f);
  float2 a = make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440)), __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441)));
  float2 b = make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7442)), __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7443)));
  a = __fadd2_rn(a, off);
  b = __fadd2_rn(b, off);
  // (single products: packed ones come out fused with the sum behind them)
  a = __fadd2_rn(make_float2(__fmul_rn(a.x, r0), __fmul_rn(a.y, r1)), magic);
  b = __fadd2_rn(make_float2(__fmul_rn(b.x, r2), __fmul_rn(b.y, r3)), magic);
  return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                     __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
}

__device__ __forceinline__ uint32_t load_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void store_release(uint32_t* p, uint32_t v) {
  asm volatile("st.release.gpu.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kMoveWarps * 32, 8) move_kernel(const CacheEvictArgs a, const Work work, bool in_place) {
  constexpr int kRows = D / 32;    // channels of a lane
  constexpr int kPitch = 36;       // bytes of a channel's row in shared memory: no bank conflicts
  __shared__ __align__(16) uint8_t tile[kMoveWarps][D * kPitch];
  __shared__ uint32_t ticket;
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  if (in_place) {
    if (threadIdx.x == 0) ticket = atomicAdd(work.ticket, 1u);
    __syncthreads();
  }
  // units: block by block of all heads, keys and values (counted in 32 bits)
  const uint32_t heads = static_cast<uint32_t>(a.B) * static_cast<uint32_t>(a.c.H);
  const uint32_t unit = (in_place ? ticket : blockIdx.x) * kMoveWarps + static_cast<uint32_t>(warp);
  if (unit >= heads * 2u * static_cast<uint32_t>(work.new_blocks)) return;
  const bool values = (unit & 1u) != 0;
  const uint32_t block = unit / 2u / heads, of_block = unit / 2u - block * heads;
  const int32_t m = static_cast<int32_t>(block);
  const int b = static_cast<int>(of_block / static_cast<uint32_t>(a.c.H)), h = static_cast<int>(of_block) - b * a.c.H;
  const int64_t head = of_block;
  bool bad = false;
  const int32_t len = length_of(a, b, &bad), stay = min(len, a.keep);
  bad = false;
  const int32_t m0 = m * kCacheBlock;
  if (m0 >= stay) return;
  const int32_t n = min(kCacheBlock, stay - m0);
  // lane i: the token that goes to place m0 + i
  const int32_t src = lane < n ? a.kept[head * a.kept_n + m0 + lane] : -1;
  if (in_place && len <= a.keep && n == kCacheBlock) return;  // nothing moves (slots behind the last token become 0)
  uint32_t* read = work.read + head * 2 * work.new_blocks + (values ? work.new_blocks : 0);
  int64_t slot = -1;
  float scale = 0.0f;
  if (src >= 0) {
    const int32_t blk = src / kCacheBlock, in_seq = blk / a.c.blocks_per_page;
    const int64_t page = a.from.table[b * a.from.stride + in_seq];
    if (page_ok(page, a.c.num_pages)) {
      slot = block_slot(page, h, a.c.H, a.c.blocks_per_page, blk - in_seq * a.c.blocks_per_page);
      scale = (values ? a.c.vs : a.c.ks)[slot];
    } else {
      bad = true;
    }
  }
  const int32_t to_page = m / a.c.blocks_per_page;
  const int64_t page = to_page < a.to.max_pages ? a.to.table[b * a.to.stride + to_page] : -1;
  const bool there = page_ok(page, a.c.num_pages);
  const int64_t to = block_slot(page, h, a.c.H, a.c.blocks_per_page, m - to_page * a.c.blocks_per_page);
  if (bad || !there) atomicExch(a.dev_err, kDevErrPage);
  float top = scale;
  const bool odd = __any_sync(0xffffffffu, scale != scale);
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
  if (odd) top = __uint_as_float(0x7FC00000u);
  const float ratio = top > 0.0f ? __fdiv_rn(scale, top) : 0.0f;

  // waits until the block's old tokens have been read, by whomever they go to
  const auto may_write = [&]() {
    if (!there) return false;
    if (!in_place) return true;
    const int32_t* before = work.before + head * (work.old_blocks + 1);
    // kept tokens of the old block m (it exists: the sequence was longer) go to places [p, q)
    const int32_t p = before[m], q = before[m + 1];
    const int32_t first = p / kCacheBlock, last = min((q - 1) / kCacheBlock, m - 1);
    if (q == p) return true;
    bool ok = true;
    if (first + lane <= last) {  // at most two blocks
      uint64_t t0 = 0;
      for (uint32_t it = 1; load_acquire(read + first + lane) == 0; ++it) {
        if ((it & 63u) != 0) continue;
        const uint64_t now = tc::global_timer_ns();
        if (t0 == 0) t0 = now;
        else if (now - t0 > tc::kWaitNs) {
          atomicExch(a.dev_err, kDevErrTimeout);
          ok = false;
          break;
        }
      }
    }
    return __all_sync(0xffffffffu, ok) != 0;
  };
  const auto have_read = [&]() {
    if (!in_place) return;
    __syncwarp();
    if (lane == 0) store_release(read + m, 1u);
  };

  if (!values) {
    // keys: 16 codes of token 8 i + lane / 4, of each 64 channels
    uint4 c[4 * (D / 64)];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 8 * i + (lane >> 2);
      const int64_t s = __shfl_sync(0xffffffffu, slot, t);
      const int32_t at = __shfl_sync(0xffffffffu, src, t);
      const int8_t* p = a.c.k + s * (kCacheBlock * D) + (at % kCacheBlock) * 64 + (lane & 3) * 16;
#pragma unroll
      for (int y = 0; y < D / 64; ++y)
        c[4 * y + i] = s >= 0 ? *reinterpret_cast<const uint4*>(p + y * 64 * kCacheBlock) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float r = __shfl_sync(0xffffffffu, ratio, 8 * i + (lane >> 2));
#pragma unroll
      for (int y = 0; y < D / 64; ++y) {
        uint4& x = c[4 * y + i];
        x = make_uint4(shrink4(x.x, r, r, r, r), shrink4(x.y, r, r, r, r), shrink4(x.z, r, r, r, r), shrink4(x.w, r, r, r, r));
      }
    }
    have_read();
    if (!may_write()) return;
    int8_t* p = a.c.k + to * (kCacheBlock * D) + lane * 16;
#pragma unroll
    for (int y = 0; y < 4 * (D / 64); ++y) *reinterpret_cast<uint4*>(p + y * 512) = c[y];
    if (lane == 0) a.c.ks[to] = top;
    return;
  }
  // values: the old blocks on their way to L2, a line for each lane
  const uint32_t all = n == 32 ? 0xffffffffu : (1u << n) - 1u;
  for (uint32_t rest = all; rest != 0;) {
    const int64_t s = __shfl_sync(0xffffffffu, slot, __ffs(rest) - 1);
    rest &= ~__ballot_sync(0xffffffffu, slot == s);
    if (s >= 0 && lane * 128 < D * kCacheBlock)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a.c.v + s * (D * kCacheBlock) + lane * 128));
  }
  // lane has channels lane, lane + 32, ...
  uint8_t* rows = tile[warp] + lane * kPitch;
#pragma unroll
  for (int y = 0; y < kRows; ++y)
#pragma unroll
    for (int e = 0; e < 8; ++e) *reinterpret_cast<uint32_t*>(rows + y * 32 * kPitch + 4 * e) = 0u;
  uint32_t w[kRows][8];
  // where a lane's token stands in its old block's rows (low byte), and goes to
  const int places = value_position(src & (kCacheBlock - 1)) | value_position(lane) << 8;
  uint32_t left = all;
  while (left != 0) {
    // the tokens of one old block
    const int64_t s = __shfl_sync(0xffffffffu, slot, __ffs(left) - 1);
    uint32_t here = __ballot_sync(0xffffffffu, slot == s) & left;
    left &= ~here;
    if (s < 0) continue;
    const int8_t* p = a.c.v + (s * D + lane) * kCacheBlock;
#pragma unroll
    for (int y = 0; y < kRows; ++y) {
      const uint4 u = *reinterpret_cast<const uint4*>(p + y * 32 * kCacheBlock);
      const uint4 v = *reinterpret_cast<const uint4*>(p + y * 32 * kCacheBlock + 16);
      w[y][0] = u.x, w[y][1] = u.y, w[y][2] = u.z, w[y][3] = u.w;
      w[y][4] = v.x, w[y][5] = v.y, w[y][6] = v.z, w[y][7] = v.w;
    }
#pragma unroll 1
    while (here != 0) {
      const int at = __shfl_sync(0xffffffffu, places, __ffs(here) - 1);
      here &= here - 1u;
      uint32_t word[kRows];
      switch ((at >> 2) & 7) {  // the same for the whole warp
#define SAGE_PICK(e)                                            \
  case e:                                                       \
    _Pragma("unroll") for (int y = 0; y < kRows; ++y) word[y] = w[y][e]; \
    break;
        SAGE_PICK(0)
        SAGE_PICK(1)
        SAGE_PICK(2)
        SAGE_PICK(3)
        SAGE_PICK(4)
        SAGE_PICK(5)
        SAGE_PICK(6)
        default:
#pragma unroll
          for (int y = 0; y < kRows; ++y) word[y] = w[y][7];
#undef SAGE_PICK
      }
      uint8_t* to_byte = rows + (at >> 8);
#pragma unroll
      for (int y = 0; y < kRows; ++y) to_byte[y * 32 * kPitch] = static_cast<uint8_t>(word[y] >> (8 * (at & 3)));
    }
  }
  have_read();
  // ratios in the order of the positions
  const float at_position = __shfl_sync(0xffffffffu, ratio, value_token(lane));
  const bool write = may_write();
#pragma unroll
  for (int y = 0; y < kRows; ++y)
#pragma unroll
    for (int e = 0; e < 8; ++e) w[y][e] = *reinterpret_cast<const uint32_t*>(rows + y * 32 * kPitch + 4 * e);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float r0 = __shfl_sync(0xffffffffu, at_position, 4 * e), r1 = __shfl_sync(0xffffffffu, at_position, 4 * e + 1);
    const float r2 = __shfl_sync(0xffffffffu, at_position, 4 * e + 2), r3 = __shfl_sync(0xffffffffu, at_position, 4 * e + 3);
#pragma unroll
    for (int y = 0; y < kRows; ++y) w[y][e] = shrink4(w[y][e], r0, r1, r2, r3);
  }
  if (!write) return;
  int8_t* p = a.c.v + (to * D + lane) * kCacheBlock;
#pragma unroll
  for (int y = 0; y < kRows; ++y) {
    *reinterpret_cast<uint4*>(p + y * 32 * kCacheBlock) = make_uint4(w[y][0], w[y][1], w[y][2], w[y][3]);
    *reinterpret_cast<uint4*>(p + y * 32 * kCacheBlock + 16) = make_uint4(w[y][4], w[y][5], w[y][6], w[y][7]);
  }
  if (lane == 0) a.c.vs[to] = top;
}

}  // namespace

size_t cache_evict_workspace_bytes(int64_t B, int64_t H, int64_t keep, int64_t scores_n) {
  const size_t heads = static_cast<size_t>(B) * static_cast<size_t>(H);
  const size_t words = 64 + heads * (static_cast<size_t>(div_up(scores_n, kCacheBlock)) + 1) +
                       heads * 2 * static_cast<size_t>(div_up(keep, kCacheBlock));
  return (words * 4 + 255) / 256 * 256;
}

cudaError_t launch_cache_evict(const CacheEvictArgs& a, int64_t D, cudaStream_t stream) {
  const Work work = work_of(a);
  const bool in_place = a.from.table == a.to.table;  // (one row, or rows equally far apart)
  const dim3 grid(static_cast<unsigned>(a.c.H > 0 ? a.c.H : 1), static_cast<unsigned>(a.B));
  // A sequence of some thousand tokens is too little for 1024 threads (16 sequences of
  // 8 heads, selection and moves: up to 1000 tokens 21.1 us with 512 threads, 25.0 with
  // 1024; 2 of 4 heads up to 4000: 16.7 and 17.4; 16 of 8 up to 8000: 66 with 1024,
  // 72 with 256). Scores that fit are read once and stay in shared memory (a
  // sequence of 40000 tokens, 4 heads: 41.8 us, 51.3 read from L2 for each digit).
  const bool few = a.scores_n <= 4096, stage = a.scores_n <= kStaged;
  const auto select = few ? select_kernel<512, true> : (stage ? select_kernel<1024, true> : select_kernel<1024, false>);
  const int bytes = stage ? static_cast<int>(a.scores_n) * 4 : 0;
  cudaError_t e;
  if (bytes > 32768 && (e = set_smem_limit_once(reinterpret_cast<const void*>(select), kStaged * 4)) != cudaSuccess) return e;
  if ((e = launch_dependent(select, grid, few ? 512 : 1024, static_cast<size_t>(bytes), stream, a, work, in_place)) != cudaSuccess)
    return e;
  const int64_t units = a.B * a.c.H * 2 * work.new_blocks;
  if (units == 0) return cudaSuccess;
  return launch_dependent(D == 128 ? move_kernel<128> : move_kernel<64>, dim3(static_cast<unsigned>(div_up(units, kMoveWarps))),
                          kMoveWarps * 32, 0, stream, a, work, in_place);
}

}  // namespace sage
