// Attention weights that cached tokens get from a step's queries, many query rows
// (formula: cache_weights.cu), on the sm_103a tensor cores (tcgen05, TMA, TMEM).
//
// The products are taken the other way round than in attention: S^T = K Q^T, 128
// keys by 128 query rows, so that a TMEM lane is a key and its thread's sum over
// the query rows needs no exchange with other threads, and no order but one.
// A CTA has one or two key tiles of a head at a time, whose codes are turned into
// BF16 once (exactly: 8 bits with their sign), and all query rows that see them
// pass by in tiles that TMA brings (tokens x the heads of the group), each
// multiplied with both key tiles. Tiles of 128 keys of all sequences and heads
// form one list that is cut into equal ranges, one per CTA. Roles of the 24 warps:
//   warp 0      TMA: query tiles
//   warps 1, 3  TMEM allocation; the products for two groups of sum warps each
//   warp 2      log-sum-exps of the query tiles
//   warps 4-7   keys: codes to BF16, in the 128-byte-swizzled layout, one pair of
//               tiles ahead
//   warps 8-23  four groups: exponentials and sums of every other query tile of key
//               tile 0 or 1 (TMEM lane = key); or, where there is one key tile, of
//               every fourth
// TMEM holds an S^T of 128 x 128 for each group: all 512 columns. The product of a
// tile (512 cycles at D = 128) and its 16384 exponentials (512 cycles) weigh alike, and
// either unit is busy 55 to 60% of the time; the operands of a product are 64 KB of shared
// memory, 512 cycles of reading too, which was not measured. A causal chunk of 2000 tokens over 16001, 32 heads on 8, D = 128: 203 us, 1210
// TFLOP/s (276 with two groups, whose latencies lay open; 325 before the
// log-sum-exps came in a ring of their own).
//
// Every wait on an mbarrier is bounded, as in prompt_attention.cu.
#include <cuda.h>

#include "cache.cuh"
#include "launch.cuh"
#include "tc_kernel.cuh"

namespace sage {
namespace {

constexpr int kThreads = 768;
constexpr int kTile = 128;        // keys of a tile, and query rows of one
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kTmemCols = 512;

template <int D>
struct Smem {
  static constexpr uint32_t kSub = 128 * 128;        // 64 channels of 128 rows
  static constexpr uint32_t kTileBytes = 128 * D * 2;
  static constexpr int kStages = 3;                  // query tiles
  static constexpr int kLse = 4;                     // log-sum-exps of query tiles
  static constexpr uint32_t kOffK = 0;               // two pairs of key tiles
  static constexpr uint32_t kOffQ = 4 * kTileBytes;
  static constexpr uint32_t kOffLse = kOffQ + kStages * kTileBytes;   // [stage][128] -log2(e) lse
  static constexpr uint32_t kOffScale = kOffLse + kLse * 512;         // [pair][8 blocks]
  static constexpr uint32_t kOffThere = kOffScale + 2 * 32;           // [pair][8 blocks]: on a page of the cache
  static constexpr uint32_t kOffOdd = kOffThere + 2 * 32;             // [stage]: whether a row is in one of these
  static constexpr uint32_t kOffNone = kOffOdd + 4 * kLse;            // [stage][128 bits]: rows that add nothing
  static constexpr uint32_t kOffNan = kOffNone + 16 * kLse;           // [stage][128 bits]: rows whose log-sum-exp is a NaN
  static constexpr uint32_t kOffBar = (kOffNan + 16 * kLse + 7) / 8 * 8;
  static constexpr int kQFull = 0, kQEmpty = kQFull + kStages, kKFull = kQEmpty + kStages, kKEmpty = kKFull + 2;
  static constexpr int kSFull = kKEmpty + 2, kSFree = kSFull + 4, kDrain = kSFree + 4, kJoin = kDrain + 2;
  static constexpr int kLFull = kJoin + 12, kLEmpty = kLFull + kLse, kBars = kLEmpty + kLse;
  static constexpr uint32_t kOffTmem = kOffBar + 8 * kBars;
  static constexpr uint32_t kOffAbort = kOffTmem + 4;
  static constexpr uint32_t kBytes = kOffAbort + 4;
};
static_assert(Smem<128>::kBytes <= 232448u, "shared memory of one CTA: at most 227 KB");

// Registers: 768 threads launched at 80. The sums are the ones that want more (with
// 80, 56 of the control warps and 104 of the keys' the chunk above takes 215 us).
constexpr uint32_t kCtlRegs = 40, kSumRegs = 96, kKeyRegs = 56;
static_assert(128 * kCtlRegs + 512 * kSumRegs + 128 * kKeyRegs <= kThreads * 80, "registers of one CTA");

struct Params {
  CacheWeightsArgs a;
  int32_t group;          // query heads of a key/value head
  int32_t heads, tokens;  // of a query tile: heads of the group, and tokens
  int32_t splits;         // query tiles for all heads of the group
  uint64_t wait_ns;       // limit of a wait
};

__device__ __forceinline__ int32_t tiles_of(int32_t keys) { return keys / kTile + (keys % kTile != 0 ? 1 : 0); }

// A walk over the CTA's range of key tiles, one or two at a time.
struct Walk {
  int32_t b, h, tile;      // the first key tile of the pair
  int32_t left;            // tiles of the range from here on
  int32_t len, rows;       // tokens and query tokens of the sequence
  int32_t shown;           // tokens that scores has a place for
  int32_t n;               // key tiles of the pair: 1 or 2

  __device__ __forceinline__ int32_t capacity(const CacheWeightsArgs& a) const {
    return static_cast<int32_t>(table_capacity(a.pt.max_pages, a.c.blocks_per_page));
  }
  __device__ __forceinline__ int32_t shown_of(const CacheWeightsArgs& a, int32_t i) const {
    const int32_t l = min(max(a.lengths[i], 0), capacity(a));
    return l < a.scores_n ? l : static_cast<int32_t>(a.scores_n);
  }
  __device__ __forceinline__ void sequence(const CacheWeightsArgs& a) {
    len = min(max(a.lengths[b], 0), capacity(a));
    shown = shown_of(a, b);
    rows = a.q_lengths != nullptr ? min(max(a.q_lengths[b], 0), static_cast<int32_t>(a.T)) : static_cast<int32_t>(a.T);
  }
  __device__ __forceinline__ void pair() { n = min(2, min(left, tiles_of(shown) - tile)); }

  // By a whole warp.
  __device__ __forceinline__ void begin(const CacheWeightsArgs& a) {
    const int lane = static_cast<int>(threadIdx.x) & 31, B = static_cast<int>(a.B);
    int64_t total = 0;
    for (int i = lane; i < B; i += 32) total += tiles_of(shown_of(a, i));
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) total += __shfl_xor_sync(0xffffffffu, total, s);
    total *= a.c.H;
    int64_t at = total * blockIdx.x / gridDim.x;
    left = static_cast<int32_t>(total * (blockIdx.x + 1) / gridDim.x - at);
    if (left <= 0) return;
    for (int b0 = 0; b0 < B; b0 += 32) {
      const int64_t own = b0 + lane < B ? int64_t(tiles_of(shown_of(a, b0 + lane))) * a.c.H : 0;
      int64_t sum = own;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, sum, s);
        if (lane >= s) sum += x;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, sum > at);
      if (past != 0) {
        const int first = __ffs(past) - 1;
        at -= __shfl_sync(0xffffffffu, sum - own, first);
        b = b0 + first;
        break;
      }
      at -= __shfl_sync(0xffffffffu, sum, 31);
    }
    sequence(a);
    const int32_t t = tiles_of(shown);
    h = static_cast<int32_t>(at / t);
    tile = static_cast<int32_t>(at % t);
    pair();
  }
  __device__ __forceinline__ void next(const CacheWeightsArgs& a) {
    left -= n;
    tile += n;
    if (left > 0 && tile == tiles_of(shown)) {
      tile = 0;
      if (++h == a.c.H) {
        h = 0;
        do {
          ++b;
          sequence(a);
        } while (shown == 0);
      }
    }
    pair();
  }
  // Query tiles that pass by: [first, end), splits of the heads innermost.
  __device__ __forceinline__ int32_t end(const Params& p) const {
    return (rows + p.tokens - 1) / p.tokens * p.splits;
  }
  __device__ __forceinline__ int32_t first(const Params& p) const {
    // row t sees key j when j <= len - rows + t
    const int32_t t = p.a.causal ? max(0, tile * kTile - (len - rows)) : 0;
    return min(t, rows) / p.tokens * p.splits;
  }
};

// 32 rows of a query tile for the thread's key: the sum of 2^(S scale + lse').
__device__ __forceinline__ float sum_rows(const uint32_t (&s)[32], float scale, const float* lse) {
  float2 sa = make_float2(0.f, 0.f), sb = make_float2(0.f, 0.f);
  const float2 c2 = make_float2(scale, scale);
#pragma unroll
  for (int k = 0; k < 32; k += 4) {
    const float4 l = *reinterpret_cast<const float4*>(lse + k);
    const float2 x01 = __ffma2_rn(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), c2, make_float2(l.x, l.y));
    const float2 x23 = __ffma2_rn(make_float2(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3])), c2, make_float2(l.z, l.w));
    sa = __fadd2_rn(sa, make_float2(tc::exp2_approx(x01.x), tc::exp2_approx(x01.y)));
    sb = __fadd2_rn(sb, make_float2(tc::exp2_approx(x23.x), tc::exp2_approx(x23.y)));
  }
  return (sa.x + sa.y) + (sb.x + sb.y);
}

// S of rows that do not count becomes minus infinity in TMEM, so that their weights
// are 0: those of tokens before `since` or from `rows` on, and those of `none` (S may
// be a NaN). That of the other rows of `nan` becomes a NaN: their lse' is finite, so
// that keys which they do not see get nothing of it. Rows of the tile: `heads` heads,
// token by token; a bit each in none and nan, which are there where `marked`.
__device__ __forceinline__ void hide_rows(uint32_t tS, bool marked, const uint32_t* none, const uint32_t* nan, int32_t since,
                                          int32_t t, int32_t heads, int32_t rows) {
  int32_t g = 0;
#pragma unroll 1
  for (int b = 0; b < 4; ++b) {
    const uint32_t off = marked ? none[b] : 0u, odd = marked ? nan[b] : 0u;
    uint32_t s[32];
    tc::tmem_ld32(tS + 32u * static_cast<uint32_t>(b), s);
    tc::tmem_wait_ld();
    if (odd != 0u) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if ((odd >> k & 1u) != 0) s[k] = 0x7FC00000u;
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const bool out = (t < since) | (t >= rows) | ((off >> k & 1u) != 0);
      s[k] = out ? 0xFF800000u : s[k];
      const bool wrap = ++g == heads;
      g = wrap ? 0 : g;
      t += wrap ? 1 : 0;
    }
    tc::tmem_st32(tS + 32u * static_cast<uint32_t>(b), s);
  }
  tc::tmem_wait_st();
}

// The rows of a query tile that add nothing (log-sum-exp x of minus infinity), and those
// where it is a NaN, whose lse' becomes 0. By a whole warp; row 32 e + lane.
__device__ __forceinline__ void mark_rows(const float (&x)[4], float (&l)[4], uint32_t* none, uint32_t* nan) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t off = __ballot_sync(0xffffffffu, x[e] == -INFINITY), odd = __ballot_sync(0xffffffffu, x[e] != x[e]);
    if ((threadIdx.x & 31u) == 0) {
      none[e] = off;
      nan[e] = odd;
    }
    if (x[e] != x[e]) l[e] = 0.0f;
  }
}

// Whether a row of tokens [since, rows) of a key/value head adds to the keys it sees.
__device__ __forceinline__ bool is_weighed(const CacheWeightsArgs& a, int32_t b, int32_t h, int32_t group, int32_t since,
                                           int32_t rows) {
  const float* lse = a.lse + (static_cast<int64_t>(b) * a.H + h * group) * a.T;
  for (int32_t t = since; t < rows; ++t)
#pragma unroll 1
    for (int32_t g = 0; g < group; ++g)
      if (lse[static_cast<int64_t>(g) * a.T + t] != -INFINITY) return true;
  return false;
}

// Which of the four groups of sum warps (and S) takes the q-th query tile of a unit
// with n key tiles, key tile x: two of them share a key tile, or four the only one.
__device__ __forceinline__ int group_of(int n, int x, uint32_t q) {
  return n == 1 ? static_cast<int>(q & 3u) : 2 * x + static_cast<int>(q & 1u);
}

// Four codes to two BF16 pairs: 128 + the low seven bits, less 128 or (negative) 256.
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t low = w & 0x7F7F7F7Fu, sign = w & 0x80808080u;
  const uint32_t v0 = __byte_perm(low, 0x43434343u, 0x4140), v1 = __byte_perm(low, 0x43434343u, 0x4342);
  const uint32_t s0 = __byte_perm(sign, 0x43434343u, 0x4140), s1 = __byte_perm(sign, 0x43434343u, 0x4342);
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(v0), "r"(s0));
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(v1), "r"(s1));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    cache_weights_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ Params prm) {
  using L = Smem<D>;
  const CacheWeightsArgs& a = prm.a;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((tc::smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicExch(a.dev_err, kDevErrSmemAlign);
    return;
  }
  const uint32_t sbase = tc::smem_u32(smem);
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  const tc::Waits w{sbase + L::kOffBar, reinterpret_cast<volatile int*>(smem + L::kOffAbort), a.dev_err, prm.wait_ns};
  float* lse_ring = reinterpret_cast<float*>(smem + L::kOffLse);
  float* scale_ring = reinterpret_cast<float*>(smem + L::kOffScale);
  int32_t* there_ring = reinterpret_cast<int32_t*>(smem + L::kOffThere);
  int32_t* odd_ring = reinterpret_cast<int32_t*>(smem + L::kOffOdd);
  uint32_t* none_ring = reinterpret_cast<uint32_t*>(smem + L::kOffNone);
  uint32_t* nan_ring = reinterpret_cast<uint32_t*>(smem + L::kOffNan);
  if (threadIdx.x == 0) {
    *w.abort_flag = 0;
    for (int i = 0; i < L::kStages; ++i) {
      tc::mbar_init(w.bar(L::kQFull + i), 1);
      tc::mbar_init(w.bar(L::kQEmpty + i), 2);
    }
    for (int i = 0; i < L::kLse; ++i) {
      tc::mbar_init(w.bar(L::kLFull + i), 1);
      tc::mbar_init(w.bar(L::kLEmpty + i), 8);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(w.bar(L::kKFull + i), 128);
      tc::mbar_init(w.bar(L::kKEmpty + i), 18);  // both issuers, 16 warps
    }
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(w.bar(L::kSFull + i), 1);
      tc::mbar_init(w.bar(L::kSFree + i), 4);
    }
    tc::mbar_init(w.bar(L::kDrain), 1);
    tc::mbar_init(w.bar(L::kDrain + 1), 1);
    for (int i = 0; i < 12; ++i) tc::mbar_init(w.bar(L::kJoin + i), 4);
    tc::fence_mbar_init();
  }
  const int32_t rows_there = prm.heads * prm.tokens;  // rows that a query tile's copy fills
  if (rows_there < kTile) {
    // the others stay 0
    for (uint32_t i = threadIdx.x; i < L::kStages * L::kTileBytes / 16; i += kThreads)
      reinterpret_cast<uint4*>(smem + L::kOffQ)[i] = make_uint4(0, 0, 0, 0);
    tc::fence_proxy_async_smem();
  }
  if (warp == 1) {
    tc::tmem_alloc(sbase + L::kOffTmem, kTmemCols);
    tc::tmem_relinquish();
  }
  if (warp == 0 && lane == 0) tc::prefetch_tmap(&tm_q);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::kOffTmem);
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  bool ok = true;

  if (warp < 4) {
    tc::regs_dec<kCtlRegs>();
    if (warp == 0) {
      // ---------------------------------------------------------- query tiles --
      Walk k;
      k.begin(a);
      if (lane == 0) {
        uint32_t at = 0;
        for (; ok && k.left > 0; k.next(a))
          for (int32_t i = k.first(prm), n = k.end(prm); ok && i < n; ++i) {
            const uint32_t st = at % L::kStages;
            if (!(ok = tc::wait_bar(w, w.bar(L::kQEmpty + static_cast<int>(st)), ((at / L::kStages) & 1u) ^ 1u))) break;
            ++at;
            const uint32_t full = w.bar(L::kQFull + static_cast<int>(st));
            tc::mbar_arrive_expect_tx(full, static_cast<uint32_t>(rows_there) * D * 2);
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
              tc::tma_load_4d(sbase + L::kOffQ + st * L::kTileBytes + x * L::kSub, &tm_q, 64 * x,
                              k.h * prm.group + i % prm.splits * prm.heads, i / prm.splits * prm.tokens, k.b, full);
          }
        if (!ok) {
          // copies land before the CTA exits
          const tc::Waits d = w.draining();
          for (uint32_t p = at < L::kStages ? 0 : at - L::kStages; p < at; ++p)
            tc::wait_bar(d, w.bar(L::kQFull + static_cast<int>(p % L::kStages)), (p / L::kStages) & 1u);
        }
      }
    } else if (warp == 1 || warp == 3) {
      // ------------------------------------------------------------- products --
      // One warp for the first two groups of sum warps, one for the others: a single one
      // is not done with its waits in a product's time.
      const int x = warp >> 1;
      const bool leader = tc::elect_one();
      const uint64_t dk0 = tc::sw128_desc(sbase + L::kOffK), dq0 = tc::sw128_desc(sbase + L::kOffQ);
      uint32_t at = 0, unit = 0, freed = 0;  // freed: a bit for each S, its phase
      Walk k;
      for (k.begin(a); ok && k.left > 0; k.next(a), ++unit) {
        if (!(ok = tc::wait_bar_warp(w, w.bar(L::kKFull + static_cast<int>(unit & 1u)), (unit >> 1) & 1u))) break;
        const uint32_t at0 = at;
        for (int32_t i = k.first(prm), n = k.end(prm); i < n; ++i, ++at) {
          const uint32_t st = at % L::kStages, ls = at % L::kLse;
          // (the log-sum-exps as well: who waits for S then finds them, and misses no phase of theirs)
          if (!(ok = tc::wait_bar_warp(w, w.bar(L::kLFull + static_cast<int>(ls)), (at / L::kLse) & 1u)) ||
              !(ok = tc::wait_bar_warp(w, w.bar(L::kQFull + static_cast<int>(st)), (at / L::kStages) & 1u)))
            break;
          if (k.n == 2 || (((at - at0) >> 1) & 1u) == static_cast<uint32_t>(x)) {
            const int tile = k.n == 2 ? x : 0, buf = group_of(k.n, tile, at - at0);
            if (!(ok = tc::wait_bar_warp(w, w.bar(L::kSFree + buf), ((freed >> buf) & 1u) ^ 1u))) break;
            freed ^= 1u << buf;
            tc::tc_fence_after();
            if (leader) {
              const uint64_t dk = tc::desc_at(dk0, (2u * (unit & 1u) + static_cast<uint32_t>(tile)) * L::kTileBytes);
              const uint64_t dq = tc::desc_at(dq0, st * L::kTileBytes);
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t off = static_cast<uint32_t>(ks >> 2) * L::kSub + static_cast<uint32_t>(ks & 3) * 32u;
                tc::mma_f16_ss(tmem + 128u * static_cast<uint32_t>(buf), tc::desc_at(dk, off), tc::desc_at(dq, off),
                               tc::IdescBf16<kTile>::value, ks > 0 ? 1u : 0u);
              }
              tc::mma_commit(w.bar(L::kSFull + buf));
            }
          }
          if (leader) tc::mma_commit(w.bar(L::kQEmpty + static_cast<int>(st)));
          __syncwarp();
        }
        if (!ok) break;
        if (leader) tc::mma_commit(w.bar(L::kKEmpty + static_cast<int>(unit & 1u)));
        __syncwarp();
      }
      if (leader) tc::mma_commit(w.bar(L::kDrain + x));
      __syncwarp();
      tc::wait_bar(w.draining(), w.bar(L::kDrain + x), 0);
    } else if (warp == 2) {
      // ------------------------------------------------------ log-sum-exps --
      // (those of the next tile are on their way while this one's are written)
      uint32_t at = 0;
      int32_t t_off[4], g_off[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 32 * e + lane;
        t_off[e] = r < rows_there ? r / prm.heads : 1 << 30;
        g_off[e] = r % prm.heads;
      }
      const auto fetch = [&](const Walk& k, int32_t i, float (&x)[4], bool (&zero)[4]) {
        const int32_t q = prm.splits == 1 ? i : i / prm.splits, g0 = (i - q * prm.splits) * prm.heads, t0 = q * prm.tokens;
        const float* lse = a.lse + (static_cast<int64_t>(k.b) * a.H + k.h * prm.group) * a.T;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int32_t t = t0 + t_off[e], g = g0 + g_off[e];
          x[e] = t_off[e] < (1 << 30) && t < k.rows && g < prm.group ? lse[static_cast<int64_t>(g) * a.T + t] : -INFINITY;
          // (rows that no copy fills, or that lie behind the last token, have S = 0)
          zero[e] = t_off[e] == 1 << 30 || t >= a.T;
        }
      };
      Walk k;
      for (k.begin(a); ok && k.left > 0; k.next(a)) {
        const int32_t first = k.first(prm), n = k.end(prm);
        float x[4];
        bool zero[4];
        if (first < n) fetch(k, first, x, zero);
        for (int32_t i = first; i < n; ++i, ++at) {
          const uint32_t st = at % L::kLse;
          float l[4];
          bool odd = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            odd |= !(x[e] > -INFINITY) && !zero[e];
            l[e] = x[e] == -INFINITY ? -INFINITY : -x[e] * kLog2e;
          }
          odd = __any_sync(0xffffffffu, odd);
          const auto empty = [&]() {
            return tc::wait_bar_warp(w, w.bar(L::kLEmpty + static_cast<int>(st)), ((at / L::kLse) & 1u) ^ 1u);
          };
          if (odd) {
            if (!(ok = empty())) break;
            mark_rows(x, l, none_ring + 4 * st, nan_ring + 4 * st);
          }
          if (i + 1 < n) fetch(k, i + 1, x, zero);
          if (!(ok = empty())) break;
#pragma unroll
          for (int e = 0; e < 4; ++e) lse_ring[st * kTile + 32 * e + lane] = l[e];
          if (lane == 0) odd_ring[st] = odd ? 1 : 0;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(w.bar(L::kLFull + static_cast<int>(st)));
        }
      }
    }
    __syncwarp();
  } else if (warp >= 8) {
    // --------------------------------------------------------------------- sums --
    tc::regs_inc<kSumRegs>();
    const int group = (warp - 8) >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t tS = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 128u * static_cast<uint32_t>(group);
    uint32_t at = 0, unit = 0, s_cnt = 0;
    Walk k;
    for (k.begin(a); ok && k.left > 0; k.next(a), ++unit) {
      if (!(ok = tc::wait_bar_warp(w, w.bar(L::kKFull + static_cast<int>(unit & 1u)), (unit >> 1) & 1u))) break;
      const bool alone = k.n == 1;  // one key tile for all four groups
      const int tile = alone ? 0 : group >> 1, blk = 4 * tile + (row >> 5);
      // A scale of 0 or NaN counts as the smallest number, so that what is hidden
      // (minus infinity) stays that; a NaN becomes the sum's if a row sees the key.
      float scale = scale_ring[8 * (unit & 1u) + blk];
      const bool odd_scale = scale != scale;
      if (odd_scale || scale == 0.0f) scale = 0x1p-126f;
      const bool there = there_ring[8 * (unit & 1u) + blk] != 0;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(w.bar(L::kKEmpty + static_cast<int>(unit & 1u)));
      const int32_t j0 = (k.tile + tile) * kTile, j = j0 + row;
      const int32_t since = a.causal ? j - (k.len - k.rows) : 0;                    // the first row token that sees the key
      const int32_t all_since = a.causal ? j0 + kTile - 1 - (k.len - k.rows) : 0;   // and all keys of the tile
      const int32_t first = k.first(prm), n = k.end(prm), step = alone ? 4 : 2;
      // who adds to a key's score first reads it now, not at the end
      const float before = there && j < k.shown && group == 0
                               ? *static_cast<volatile float*>(a.scores + k.b * a.scores_b + k.h * a.scores_h + j)
                               : 0.0f;
      float sum = 0.0f;
      for (int32_t q = alone ? group : group & 1; q < n - first; q += step) {
        const uint32_t ls = (at + static_cast<uint32_t>(q)) % L::kLse, phase = (at + static_cast<uint32_t>(q)) / L::kLse;
        if (!(ok = tc::wait_bar_warp(w, w.bar(L::kSFull + group), s_cnt & 1u)) ||
            !(ok = tc::wait_bar_warp(w, w.bar(L::kLFull + static_cast<int>(ls)), phase & 1u)))
          break;
        ++s_cnt;
        tc::tc_fence_after();
        const float* lse = lse_ring + ls * kTile;
        const int32_t t0 = (prm.splits == 1 ? first + q : (first + q) / prm.splits) * prm.tokens;
        const bool marked = odd_ring[ls] != 0;
        if (t0 < all_since || marked)
          hide_rows(tS, marked, none_ring + 4 * ls, nan_ring + 4 * ls, since, t0, prm.heads, k.rows);
        // S is read 32 columns at a time, the next ones under this one's exponentials
        uint32_t s0[32], s1[32];
        tc::tmem_ld32(tS, s0);
        tc::tmem_wait_ld();
        tc::tmem_ld32(tS + 32u, s1);
        float part = sum_rows(s0, scale, lse);
        tc::tmem_wait_ld();
        tc::tmem_ld32(tS + 64u, s0);
        part += sum_rows(s1, scale, lse + 32);
        tc::tmem_wait_ld();
        tc::tmem_ld32(tS + 96u, s1);
        part += sum_rows(s0, scale, lse + 64);
        tc::tmem_wait_ld();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(w.bar(L::kSFree + group));
        part += sum_rows(s1, scale, lse + 96);
        sum += part;
        __syncwarp();
        if (lane == 0) {
          // eight arrivals: two groups of four warps, or one that arrives twice
          tc::mbar_arrive(w.bar(L::kLEmpty + static_cast<int>(ls)));
          if (alone) tc::mbar_arrive(w.bar(L::kLEmpty + static_cast<int>(ls)));
        }
      }
      if (!ok) break;
      at += static_cast<uint32_t>(max(n - first, 0));
      if (odd_scale && j < k.shown && is_weighed(a, k.b, k.h, prm.group, max(since, 0), k.rows)) sum = __uint_as_float(0x7FC00000u);
      // The groups add their sums one after another, so that they always come in this
      // order. (Four barriers for each, unit by unit: a group may be three units ahead of
      // the next one, which has to begin a unit before the keys of the one after the
      // next are brought.)
      const int turn = 4 * group + static_cast<int>(unit & 3u);
      if (group > 0 && !(ok = tc::wait_bar_warp(w, w.bar(L::kJoin + turn - 4), (unit >> 2) & 1u))) break;
      if (there && j < k.shown && !(sum == 0.0f)) {
        volatile float* p = a.scores + k.b * a.scores_b + k.h * a.scores_h + j;
        *p = (group == 0 ? before : *p) + sum;
      }
      __syncwarp();
      if (lane == 0 && group < 3) tc::mbar_arrive(w.bar(L::kJoin + turn));
    }
    tc::regs_dec<kCtlRegs>();
  } else {
    // --------------------------------------------------------------------- keys --
    tc::regs_dec<kKeyRegs>();
    const int g = lane >> 2, t4 = lane & 3;
    uint32_t unit = 0;
    bool bad = false;
    Walk k;
    for (k.begin(a); ok && k.left > 0; k.next(a), ++unit) {
      const uint32_t buf = unit & 1u;
      if (!(ok = tc::wait_bar_warp(w, w.bar(L::kKEmpty + static_cast<int>(buf)), ((unit >> 1) & 1u) ^ 1u))) break;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int local = 2 * (warp - 4) + y;             // block of the pair
        const int32_t blk = k.tile * 4 + local;
        if (local >= 4 * k.n) continue;
        int64_t slot = -1;
        if (block_has_tokens(blk, k.shown)) {
          const int32_t in_seq = blk / a.c.blocks_per_page;
          const int64_t page = a.pt.table[k.b * a.pt.stride + in_seq];
          if (page_ok(page, a.c.num_pages)) slot = block_slot(page, k.h, a.c.H, a.c.blocks_per_page, blk - in_seq * a.c.blocks_per_page);
          else bad = true;
        }
        if (lane == 0) {
          scale_ring[8 * buf + local] = slot < 0 ? 0.0f : a.c.ks[slot] * a.sm_log2;
          there_ring[8 * buf + local] = slot < 0 ? 0 : 1;
        }
        // key 8 n + g of the block, channels 16 t4 .. 16 t4 + 15 of each half
        uint8_t* tile = smem + L::kOffK + (2u * buf + static_cast<uint32_t>(local >> 2)) * L::kTileBytes;
#pragma unroll 1
        for (int x = 0; x < D / 64; ++x) {  // (half at a time, for few registers)
          uint4 c[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            c[i] = slot < 0 ? make_uint4(0, 0, 0, 0)
                            : *reinterpret_cast<const uint4*>(a.c.k + slot * (kCacheBlock * D) + (4 * x + i) * 512 + lane * 16);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = 32 * (local & 3) + 8 * i + g;
            uint32_t o[8];
            codes_to_bf16(c[i].x, o[0], o[1]);
            codes_to_bf16(c[i].y, o[2], o[3]);
            codes_to_bf16(c[i].z, o[4], o[5]);
            codes_to_bf16(c[i].w, o[6], o[7]);
            uint8_t* p = tile + x * L::kSub + key * 128;
            *reinterpret_cast<uint4*>(p + (((2 * t4) ^ (key & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(p + (((2 * t4 + 1) ^ (key & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
      }
      tc::fence_proxy_async_smem();
      tc::mbar_arrive(w.bar(L::kKFull + static_cast<int>(buf)));
    }
    if (bad) atomicExch(a.dev_err, kDevErrPage);
    tc::regs_dec<kCtlRegs>();
  }

  // lengths that had to be cut
  if (blockIdx.x == 0 && warp == 2) {
    bool bad = false;
    const int32_t capacity = static_cast<int32_t>(table_capacity(a.pt.max_pages, a.c.blocks_per_page));
    for (int b = lane; b < a.B; b += 32) {
      const int32_t n = a.lengths[b], r = a.q_lengths != nullptr ? a.q_lengths[b] : 0;
      bad |= n < 0 || n > capacity || r < 0 || r > a.T;
    }
    if (bad) atomicExch(a.dev_err, kDevErrPage);
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
cudaError_t launch(const CacheWeightsArgs& a, cudaStream_t stream) {
  Params p;
  p.a = a;
  p.group = a.H / a.c.H;
  p.heads = p.group < kTile ? p.group : kTile;
  p.tokens = kTile / p.heads;
  p.splits = static_cast<int32_t>(div_up(p.group, p.heads));
  p.wait_ns = tc::wait_limit_ns(div_up(a.T, p.tokens) * p.splits);
  CUtensorMap tq;
  const uint64_t dims[4] = {D, static_cast<uint64_t>(a.H), static_cast<uint64_t>(a.T), static_cast<uint64_t>(a.B)};
  // (strides of one head, token or sequence are not used; the tensor map wants valid ones)
  const uint64_t strides[3] = {static_cast<uint64_t>(a.H > 1 ? a.q.sh : D) * 2, static_cast<uint64_t>(a.T > 1 ? a.q.ss : D) * 2,
                               static_cast<uint64_t>(a.B > 1 ? a.q.sb : D) * 2};
  const uint32_t box[4] = {64, static_cast<uint32_t>(p.heads), static_cast<uint32_t>(p.tokens), 1};
  if (!make_tmap(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, a.q.p, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const int64_t most = table_capacity(a.pt.max_pages, a.c.blocks_per_page);
  const int64_t tiles = div_up(a.scores_n < most ? a.scores_n : most, kTile) * a.c.H * a.B, sms = sm_count_current();
  const int bytes = static_cast<int>(Smem<D>::kBytes);
  const cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(cache_weights_tc_kernel<D>), bytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(cache_weights_tc_kernel<D>, dim3(static_cast<unsigned>(tiles < sms ? tiles : sms)), kThreads,
                          static_cast<size_t>(bytes), stream, tq, p);
}

}  // namespace

cudaError_t launch_cache_weights_tc(const CacheWeightsArgs& a, int64_t D, cudaStream_t stream) {
  return D == 128 ? launch<128>(a, stream) : launch<64>(a, stream);
}

}  // namespace sage
