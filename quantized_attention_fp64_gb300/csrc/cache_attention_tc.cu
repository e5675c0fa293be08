// Attention of many query rows to an 8-bit paged cache (prompt chunks, cross
// attention): the tensor-core form of cache_attention.cu's formulas.
//
// A work unit is one key/value head of one sequence and a pair of tiles of 128
// query rows (query tokens x the heads that share the key/value head, token
// major), so the codes of a key tile are converted once for 256 rows. One CTA
// per unit, 16 warps:
//   warps 0, 1    one MMA-issuing thread per query tile
//   warp 2        TMEM allocation
//   warps 4-7, 8-11  softmax of query tile 0, 1 (TMEM lane = row)
//   warps 12-15   converters: read the int8 codes of 128 keys (a warp per
//                 32-key block, 16 bytes per lane and load, the next tile's
//                 loads in flight in registers), turn them into fp16 and store
//                 them in the 128-byte-swizzled layout that the MMA reads
// Per tile and step j (64 keys at D = 128, 128 at D = 64): S = Q K_j^T
// (tcgen05 kind::f16, fp32 in TMEM); the softmax reads S into registers and
// releases it, so the next step's QK runs under the exponentials; p goes to
// TMEM as fp16, and O += P V_j reads it there (P in shared memory would double
// what the products read from it). At D = 128 the 512 columns hold, per tile,
// 128 of O, 64 of S and two P of 32, written in turns; at D = 64 64 of O, 128
// of S and one P of 64.
// Numbers. Queries become fp16 times a power of two per row (their largest
// value in [1, 4)); key codes are exact in fp16. Values become
// fp16(code * fp16(s_v / R)), R the largest value scale of the unit's blocks:
// two roundings of 2^-12 relative; p is rounded to fp16, 2^-12 relative. A block
// whose scale is below 2^-14 R loses bits of that (its values are then held to
// 2^-25 R absolutely).
// The keys of a block stand in the order in which the values are stored
// (value_position), so V^T needs no reordering on the way.
//
// Every wait on an mbarrier is bounded, as in attention_tc.cu.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.cuh"
#include "common.cuh"
#include "tc_ptx.cuh"

namespace sage {
namespace {

constexpr int kThreads = 512;
constexpr int kRows = 128;      // rows of a query tile
constexpr int kKeys = 128;      // keys of a key tile
constexpr int kStages = 2;      // key and value tiles in shared memory
constexpr int kScaleSlots = 4;  // key tiles whose scales are kept
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.0f;   // p may reach 2^8 before the running maximum follows
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr uint32_t kTmemCols = 512;

// registers per thread of the control, converter and softmax warps
constexpr uint32_t kRegCtl = 56, kRegConv = 104, kRegSoftmax = 176;
static_assert(128 * (kRegCtl + kRegConv) + 256 * kRegSoftmax <= 65536, "register file of one SM");

template <int D>
struct Smem {
  static constexpr uint32_t kSub = 128 * 128;             // 64 channels of 128 rows, fp16
  static constexpr uint32_t kTile = (D / 64) * kSub;      // a query or key tile
  static constexpr uint32_t kSubV = D * 128;              // 64 keys of D channels, fp16
  static constexpr uint32_t kTileV = 2 * kSubV;
  static constexpr uint32_t kOffQ = 0;                    // 2 tiles
  static constexpr uint32_t kOffK = kOffQ + 2 * kTile;
  static constexpr uint32_t kOffV = kOffK + kStages * kTile;
  static constexpr uint32_t kOffBar = kOffV + kStages * kTileV;
};
constexpr int kBarQFull = 0, kBarKFull = kBarQFull + 2, kBarKEmpty = kBarKFull + kStages;
constexpr int kBarVFull = kBarKEmpty + kStages, kBarVEmpty = kBarVFull + kStages;
constexpr int kBarSFull = kBarVEmpty + kStages, kBarSFree = kBarSFull + 2, kBarPFull = kBarSFree + 2;
constexpr int kBarPVDone = kBarPFull + 2, kBarDrain = kBarPVDone + 4, kBarScale = kBarDrain + 2;  // PVDone: [tile][P buffer]
constexpr int kNumBars = kBarScale + kScaleSlots;
template <int D>
struct SmemTail {
  static constexpr uint32_t kOffTmem = Smem<D>::kOffBar + kNumBars * 8;
  static constexpr uint32_t kOffAbort = kOffTmem + 4;
  static constexpr uint32_t kOffTop = kOffAbort + 4;                    // [converter warp] largest value scale
  static constexpr uint32_t kOffScale = (kOffTop + 16 + 15) / 16 * 16;  // [slot][block] key scales
  static_assert(kOffScale % 16 == 0 && kOffTop % 4 == 0, "a slot is read as one float4");
  static constexpr uint32_t kBytes = kOffScale + kScaleSlots * 16;
};
static_assert(SmemTail<128>::kBytes <= 232448u, "shared memory of one CTA");

// Steps of a tile and its TMEM columns.
template <int D>
struct Step {
  static constexpr int kKeysPerStep = D == 128 ? 64 : 128;
  static constexpr int kPer = kKeys / kKeysPerStep;    // steps per key tile
  static constexpr int kP = D == 128 ? 2 : 1;          // buffers of P
  static constexpr uint32_t kIdescQK = D == 128 ? tc::kIdescM128N64 : tc::kIdescM128N128;
  __host__ __device__ static constexpr uint32_t col_o(int i) { return static_cast<uint32_t>(D * i); }
  __host__ __device__ static constexpr uint32_t col_s(int i) { return static_cast<uint32_t>(2 * D + (256 - D) * i); }
  __host__ __device__ static constexpr uint32_t col_p(int i, int buf) {
    return col_s(i) + static_cast<uint32_t>(kKeysPerStep + buf * (kKeysPerStep / 2));
  }
  static_assert(col_p(1, kP - 1) + kKeysPerStep / 2 <= kTmemCols, "tensor memory");
};

struct Ctx {
  uint32_t bar0;
  volatile int* abort_flag;
  int* dev_err;
  __device__ uint32_t bar(int i) const { return bar0 + 8u * static_cast<uint32_t>(i); }
};

__device__ __forceinline__ bool wait_bar(const Ctx& cx, uint32_t bar, uint32_t parity) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if ((it & 127u) == 0) {
      if (*cx.abort_flag) return false;
      const uint64_t now = tc::global_timer_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > kTimeoutNs) {
        *cx.abort_flag = 1;
        atomicExch(cx.dev_err, kDevErrTimeout);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait_bar_warp(const Ctx& cx, uint32_t bar, uint32_t parity) {
  const bool ok = wait_bar(cx, bar, parity);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <uint32_t N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <uint32_t N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ bool elect_one() {
  uint32_t pred;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(pred));
  return pred != 0;
}
__device__ __forceinline__ uint64_t desc_at(uint64_t base, uint32_t offset) { return base + (offset >> 4); }

// D(tmem) (+)= A(tmem) * B(smem)^T, f16 x f16 -> f32, K = 16.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Four int8 codes to four fp16, exactly (see cache_attention.cu).
__device__ __forceinline__ void codes_to_half(uint32_t x, __half2& lo, __half2& hi) {
  x ^= 0x80808080u;
  const uint32_t bias = 0x64806480u;
  const uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
  lo = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&bias));
  hi = __hsub2(*reinterpret_cast<const __half2*>(&b), *reinterpret_cast<const __half2*>(&bias));
}
__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// The work of a CTA, the same in every thread.
struct Unit {
  int b, h, len, q_len, R, G;
  int row0, tiles;  // first row, query tiles with rows
  int n[2], n_max;  // key tiles of each query tile
};

// Keys that a row sees (any row; a row past the last counts as the last).
__device__ __forceinline__ int row_sees(const CacheAttentionArgs& a, const Unit& u, int r) {
  if (!a.causal) return u.len;
  const int tok = min(r, u.R - 1) / u.G;
  return max(u.len - u.q_len + tok + 1, 0);
}

__device__ __forceinline__ Unit find_unit(const CacheAttentionArgs& a, int pairs, bool* bad) {
  Unit u;
  // the last rows of a causal chunk see the most keys: first
  const int heads = static_cast<int>(a.B) * a.c.H;
  const int pair = pairs - 1 - static_cast<int>(blockIdx.x) / heads, bh = static_cast<int>(blockIdx.x) % heads;
  u.b = bh / a.c.H;
  u.h = bh - u.b * a.c.H;
  u.len = static_cast<int>(checked_length(a.lengths[u.b], table_capacity(a.pt.max_pages, a.c.blocks_per_page), bad));
  u.q_len = static_cast<int>(a.q_lengths != nullptr ? checked_length(a.q_lengths[u.b], a.T, bad) : a.T);
  u.G = a.H / a.c.H;
  u.R = u.q_len * u.G;
  u.row0 = pair * 2 * kRows;
  u.tiles = u.row0 >= u.R ? 0 : (u.row0 + kRows >= u.R ? 1 : 2);
  u.n_max = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    u.n[i] = i < u.tiles ? (row_sees(a, u, u.row0 + i * kRows + kRows - 1) + kKeys - 1) / kKeys : 0;
    u.n_max = max(u.n_max, u.n[i]);
  }
  return u;
}

// dk: the step's first key of the key tile
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint64_t dq, uint64_t dk) {
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const uint32_t off = static_cast<uint32_t>(ks >> 2) * Smem<D>::kSub + static_cast<uint32_t>(ks & 3) * 32u;
    tc::mma_f16_ss(d_tmem, desc_at(dq, off), desc_at(dk, off), Step<D>::kIdescQK, ks > 0 ? 1u : 0u);
  }
}
// dv: the step's first 64 keys of the value tile
template <int D>
__device__ __forceinline__ void issue_pv(uint32_t d_tmem, uint32_t tp, uint64_t dv, bool acc) {
  constexpr uint32_t idesc = D == 128 ? tc::kIdescM128N128 : tc::kIdescM128N64;
#pragma unroll
  for (int ks = 0; ks < Step<D>::kKeysPerStep / 16; ++ks) {
    const uint32_t off = static_cast<uint32_t>(ks >> 2) * Smem<D>::kSubV + static_cast<uint32_t>(ks & 3) * 32u;
    mma_f16_ts(d_tmem, tp + 8u * static_cast<uint32_t>(ks), desc_at(dv, off), idesc, (acc || ks > 0) ? 1u : 0u);
  }
}

// The next 32 key tiles' blocks of a converter warp, one per lane.
struct Window {
  int64_t slot;  // block number in the cache, -1: none
  float ks, vs;
};
__device__ __forceinline__ Window load_window(const CacheAttentionArgs& a, const Unit& u, int blk, bool* bad) {
  Window w;
  w.slot = -1;
  w.ks = -1.0f;  // no tokens
  w.vs = 0.0f;
  if (blk * kCacheBlock < u.len) {
    const int pg = blk / a.c.blocks_per_page;
    const int page = a.pt.table[u.b * a.pt.stride + pg];
    if (page_ok(page, a.c.num_pages)) {
      w.slot = block_slot(page, u.h, a.c.H, a.c.blocks_per_page, blk - pg * a.c.blocks_per_page);
      w.ks = a.c.ks[w.slot];
      w.vs = a.c.vs[w.slot];
    } else {
      *bad = true;
    }
  }
  return w;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) cache_attention_tc_kernel(const CacheAttentionArgs a, int pairs) {
  using L = Smem<D>;
  using T = SmemTail<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((tc::smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicExch(a.dev_err, kDevErrSmemAlign);
    return;
  }
  const uint32_t sbase = tc::smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Ctx cx;
  cx.bar0 = sbase + L::kOffBar;
  cx.abort_flag = reinterpret_cast<volatile int*>(smem + T::kOffAbort);
  cx.dev_err = a.dev_err;
  tc::griddep_wait();
  bool bad = false;
  const Unit u = find_unit(a, pairs, &bad);
  if (threadIdx.x == 0) {
    if (bad) atomicExch(a.dev_err, kDevErrPage);
    *cx.abort_flag = 0;
    const uint32_t tiles = static_cast<uint32_t>(max(u.tiles, 1));
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(cx.bar(kBarQFull + s), kRows);
      tc::mbar_init(cx.bar(kBarSFull + s), 1);
      tc::mbar_init(cx.bar(kBarPFull + s), kRows);
      tc::mbar_init(cx.bar(kBarSFree + s), kRows);
      tc::mbar_init(cx.bar(kBarPVDone + 2 * s), 1);
      tc::mbar_init(cx.bar(kBarPVDone + 2 * s + 1), 1);
      tc::mbar_init(cx.bar(kBarDrain + s), 1);
    }
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(cx.bar(kBarKFull + s), 128);
      tc::mbar_init(cx.bar(kBarKEmpty + s), tiles);
      tc::mbar_init(cx.bar(kBarVFull + s), 128);
      tc::mbar_init(cx.bar(kBarVEmpty + s), tiles);
    }
    for (int s = 0; s < kScaleSlots; ++s) tc::mbar_init(cx.bar(kBarScale + s), 4);
    tc::fence_mbar_init();
  }
  if (warp == 2) {
    tc::tmem_alloc(sbase + T::kOffTmem, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + T::kOffTmem);

  if (warp < 4) {
    regs_dec<kRegCtl>();
    if (warp < 2) {
      // ------------------------------------------------ MMA issuer of tile i --
      const int i = warp;
      const bool leader = elect_one();
      using S = Step<D>;
      const uint32_t d_s = tmem + S::col_s(i), d_o = tmem + S::col_o(i);
      const uint64_t dq = tc::sw128_desc(sbase + L::kOffQ + static_cast<uint32_t>(i) * L::kTile);
      const uint64_t dk0 = tc::sw128_desc(sbase + L::kOffK), dv0 = tc::sw128_desc(sbase + L::kOffV);
      const int n = u.n[i] * S::kPer, n_all = u.n_max * S::kPer;  // steps of this tile, and of the CTA
      bool ok = i < u.tiles;
      if (ok && n > 0) ok = wait_bar_warp(cx, cx.bar(kBarQFull + i), 0);
      for (int j = 0; ok && j <= n_all; ++j) {
        if (j < n_all) {
          // QK_j once its keys are there and the softmax has read S_{j-1}
          const int tile = j / S::kPer, in = j % S::kPer;
          const uint32_t s = static_cast<uint32_t>(tile) % kStages, ph = (static_cast<uint32_t>(tile) / kStages) & 1u;
          if (in == 0 && !(ok = wait_bar_warp(cx, cx.bar(kBarKFull + s), ph))) break;
          if (j < n) {
            if (j > 0 && !(ok = wait_bar_warp(cx, cx.bar(kBarSFree + i), static_cast<uint32_t>(j - 1) & 1u))) break;
            tc::tc_fence_after();
            if (leader) {
              issue_qk<D>(d_s, dq, desc_at(dk0, s * L::kTile + static_cast<uint32_t>(in * S::kKeysPerStep) * 128u));
              tc::mma_commit(cx.bar(kBarSFull + i));
              if (in == S::kPer - 1) tc::mma_commit(cx.bar(kBarKEmpty + s));
            }
          } else if (leader && in == S::kPer - 1) {
            tc::mbar_arrive(cx.bar(kBarKEmpty + s));  // no row of this tile sees the keys
          }
          __syncwarp();
        }
        if (j >= 1) {
          // PV_{j-1} once its values and P_{j-1} are there
          const int jj = j - 1, tile = jj / S::kPer, in = jj % S::kPer;
          const uint32_t s = static_cast<uint32_t>(tile) % kStages, ph = (static_cast<uint32_t>(tile) / kStages) & 1u;
          if (in == 0 && !(ok = wait_bar_warp(cx, cx.bar(kBarVFull + s), ph))) break;
          if (jj < n) {
            if (!(ok = wait_bar_warp(cx, cx.bar(kBarPFull + i), static_cast<uint32_t>(jj) & 1u))) break;
            tc::tc_fence_after();
            if (leader) {
              issue_pv<D>(d_o, tmem + S::col_p(i, jj % S::kP),
                          desc_at(dv0, s * L::kTileV + static_cast<uint32_t>(in) * (S::kKeysPerStep / 64) * L::kSubV),
                          jj > 0);
              tc::mma_commit(cx.bar(kBarPVDone + 2 * i + jj % S::kP));
              if (in == S::kPer - 1) tc::mma_commit(cx.bar(kBarVEmpty + s));
            }
          } else if (leader && in == S::kPer - 1) {
            tc::mbar_arrive(cx.bar(kBarVEmpty + s));
          }
          __syncwarp();
        }
      }
      // all MMAs of this warp complete before TMEM is freed
      if (leader) tc::mma_commit(cx.bar(kBarDrain + i));
      __syncwarp();
      Ctx drain = cx;
      volatile int no_abort = 0;
      drain.abort_flag = &no_abort;
      wait_bar(drain, cx.bar(kBarDrain + i), 0);
    }
    __syncwarp();
  } else if (warp >= 12) {
    // ------------------------------------------------------------ converters --
    regs_dec<kRegConv>();
    const int w = warp - 12;  // block of each key tile
    // the largest value scale of the unit's blocks (NaN passes)
    float top = 0.0f;
    bool bad_page = false;
    for (int t = lane; t < u.n_max; t += 32) top = fmaxf(top, load_window(a, u, t * 4 + w, &bad_page).vs);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float* tops = reinterpret_cast<float*>(smem + T::kOffTop);
    if (lane == 0) tops[w] = top;
    asm volatile("bar.sync 1, 128;" ::: "memory");
    top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    const float inv_top = top > 0.0f ? 1.0f / top : 0.0f;
    // Load x of the warp. Keys: tokens 8 (x mod 4) + lane / 4 of 64-channel half
    // x / 4, channels 16 (lane mod 4) and up. Values: channel 16 x + v_ch,
    // positions 16 (lane mod 2) and up, where v_ch is lane / 2 with its bits 1
    // and 2 exchanged: the 8 lanes of a store phase then write channels c, c + 1,
    // c + 4, c + 5, whose swizzled chunks are all different.
    const int v_ch = ((lane >> 1) & 9) | ((lane >> 1) & 2) << 1 | ((lane >> 1) & 4) >> 1;
    const int v_at = 2 * v_ch + (lane & 1);
    Window win{-1, -1.0f, 0.0f};
    uint4 kr[D / 16], vr[D / 16];  // raw codes of the block: 512 bytes per load of the warp
    // window lane t holds key tile t mod 32; loads of a block that is not there read nothing
    const auto fetch = [&](int j, const int8_t* base, int at, uint4 (&r)[D / 16]) {
      const int64_t slot = __shfl_sync(0xffffffffu, win.slot, j & 31);
      const uint4* p = reinterpret_cast<const uint4*>(base + slot * (kCacheBlock * D)) + at;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) r[x] = slot >= 0 ? p[x * 32] : make_uint4(0u, 0u, 0u, 0u);
    };
    if (u.n_max > 0) {
      win = load_window(a, u, lane * 4 + w, &bad_page);
      fetch(0, a.c.k, lane, kr);
      fetch(0, a.c.v, v_at, vr);
    }
    bool ok = true;
    for (int j = 0; ok && j < u.n_max; ++j) {
      const uint32_t s = static_cast<uint32_t>(j) % kStages, ph = (static_cast<uint32_t>(j) / kStages) & 1u;
      const float ks = __shfl_sync(0xffffffffu, win.ks, j & 31);
      const float vs = __shfl_sync(0xffffffffu, win.vs, j & 31);
      if (!(ok = wait_bar_warp(cx, cx.bar(kBarKEmpty + s), ph ^ 1u))) break;
      const uint32_t k_row = sbase + L::kOffK + s * L::kTile;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const int n = lane >> 2, row = w * 32 + 8 * (n >> 1) + 2 * (x & 3) + (n & 1);  // value_position of token 8x + n
          const uint32_t cw[4] = {kr[x].x, kr[x].y, kr[x].z, kr[x].w};
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            __half2 lo, hi;
            codes_to_half(cw[e], lo, hi);
            o[2 * e] = bits(lo);
            o[2 * e + 1] = bits(hi);
          }
          const uint32_t at = k_row + static_cast<uint32_t>(x >> 2) * L::kSub + static_cast<uint32_t>(row) * 128u;
          const uint32_t c = static_cast<uint32_t>(lane & 3) * 2u, sw = static_cast<uint32_t>(row) & 7u;
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + ((c ^ sw) << 4)), "r"(o[0]), "r"(o[1]),
                       "r"(o[2]), "r"(o[3])
                       : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + (((c + 1u) ^ sw) << 4)), "r"(o[4]), "r"(o[5]),
                       "r"(o[6]), "r"(o[7])
                       : "memory");
        }
      if (lane == 0) {
        // a value scale that is NaN makes the rows that see the block NaN through their logits
        reinterpret_cast<float*>(smem + T::kOffScale)[(j % kScaleSlots) * 4 + w] = vs != vs ? vs : ks;
        tc::mbar_arrive(cx.bar(kBarScale + j % kScaleSlots));
      }
      tc::fence_proxy_async_smem();
      tc::mbar_arrive(cx.bar(kBarKFull + s));
      // the next tile's window and keys
      if (j + 1 < u.n_max) {
        if (((j + 1) & 31) == 0) win = load_window(a, u, (j + 1 + lane) * 4 + w, &bad_page);
        fetch(j + 1, a.c.k, lane, kr);
      }
      if (!(ok = wait_bar_warp(cx, cx.bar(kBarVEmpty + s), ph ^ 1u))) break;
      // fp16(s_v / R) below 2^-14 would lose bits: the power of two comes off after the product then
      float h = vs == vs ? vs * inv_top : 0.0f, shift = 1.0f;
      if (h < 6.1035156e-05f) {
        h *= 16384.0f;
        shift = 6.1035156e-05f;
      }
      const __half2 h2 = __float2half2_rn(h), shift2 = __float2half2_rn(shift);
      const uint32_t v_row = sbase + L::kOffV + s * L::kTileV + static_cast<uint32_t>(w >> 1) * L::kSubV;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        const int ch = 16 * x + v_ch;
        const uint32_t cw[4] = {vr[x].x, vr[x].y, vr[x].z, vr[x].w};
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          __half2 lo, hi;
          codes_to_half(cw[e], lo, hi);
          lo = __hmul2(lo, h2);
          hi = __hmul2(hi, h2);
          if (shift != 1.0f) {
            lo = __hmul2(lo, shift2);
            hi = __hmul2(hi, shift2);
          }
          o[2 * e] = bits(lo);
          o[2 * e + 1] = bits(hi);
        }
        const uint32_t at = v_row + static_cast<uint32_t>(ch) * 128u;
        const uint32_t c = static_cast<uint32_t>(w & 1) * 4u + static_cast<uint32_t>(lane & 1) * 2u;
        const uint32_t sw = static_cast<uint32_t>(ch) & 7u;
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + ((c ^ sw) << 4)), "r"(o[0]), "r"(o[1]),
                     "r"(o[2]), "r"(o[3])
                     : "memory");
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + (((c + 1u) ^ sw) << 4)), "r"(o[4]), "r"(o[5]),
                     "r"(o[6]), "r"(o[7])
                     : "memory");
      }
      tc::fence_proxy_async_smem();
      tc::mbar_arrive(cx.bar(kBarVFull + s));
      if (j + 1 < u.n_max) fetch(j + 1, a.c.v, v_at, vr);
    }
    if (bad_page) atomicExch(a.dev_err, kDevErrPage);
    __syncwarp();
    regs_dec<kRegCtl>();
  } else {
    // --------------------------------------------------------------- softmax --
    regs_inc<kRegSoftmax>();
    const int i = (warp - 4) >> 2, wq = warp & 3;
    const int r = u.row0 + i * kRows + wq * 32 + lane;  // this thread's row
    const uint32_t lane_addr = static_cast<uint32_t>(wq * 32) << 16;
    using S = Step<D>;
    const uint32_t tS = tmem + lane_addr + S::col_s(i), tO = tmem + lane_addr + S::col_o(i);
    const bool real = r < u.R;
    const int tok = r / u.G, head = u.h * u.G + r - tok * u.G;
    const int sees = real ? row_sees(a, u, r) : 0;
    bool ok = i < u.tiles;
    float m = -INFINITY, l = 0.0f, f = 0.0f;
    if (ok && u.n[i] > 0) {
      // the row's queries to fp16, times a power of two, in the swizzled layout
      const uint32_t q_row = sbase + L::kOffQ + static_cast<uint32_t>(i) * L::kTile + static_cast<uint32_t>(wq * 32 + lane) * 128u;
      uint4 x[D / 8];
      uint32_t amax = 0;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        x[c] = make_uint4(0u, 0u, 0u, 0u);
        if (real) x[c] = reinterpret_cast<const uint4*>(a.q.p + u.b * a.q.sb + tok * a.q.ss + head * a.q.sh)[c];
        const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = max(amax, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
      }
      uint32_t ex = amax >> 7;
      ex = ex == 255u ? 127u : min(max(ex, 1u), 253u);
      const float down = __uint_as_float((254u - ex) << 23);
      f = __uint_as_float(ex << 23) * a.sm_log2;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = pack_half2(__uint_as_float(w[e] << 16) * down, __uint_as_float(w[e] & 0xFFFF0000u) * down);
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(
                         q_row + static_cast<uint32_t>(c >> 3) * L::kSub + (((c & 7) ^ (lane & 7)) << 4)),
                     "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                     : "memory");
      }
      tc::fence_proxy_async_smem();
      tc::mbar_arrive(cx.bar(kBarQFull + i));
    }
    // the smallest limit in the warp decides, for all its lanes, whether a tile is masked
    const int all_see = __reduce_min_sync(0xffffffffu, real ? sees : 0x7fffffff);
    const float* scale_ring = reinterpret_cast<const float*>(smem + T::kOffScale);
    constexpr int kB = S::kKeysPerStep / kCacheBlock;  // blocks of a step
    const int n = u.n[i] * S::kPer;
    float k4[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // scales of the key tile
    // waits for the PV of step x (its P buffer and O are then free)
    const auto wait_pv = [&](int x) {
      return wait_bar_warp(cx, cx.bar(kBarPVDone + 2 * i + x % S::kP), static_cast<uint32_t>(x / S::kP) & 1u);
    };
    for (int j = 0; ok && j < n; ++j) {
      const int tile = j / S::kPer, in = j % S::kPer;
      if (in == 0) {
        if (!(ok = wait_bar_warp(cx, cx.bar(kBarScale + tile % kScaleSlots), static_cast<uint32_t>(tile / kScaleSlots) & 1u)))
          break;
        const float4 ks = *reinterpret_cast<const float4*>(scale_ring + (tile % kScaleSlots) * 4);
        k4[0] = ks.x;
        k4[1] = ks.y;
        k4[2] = ks.z;
        k4[3] = ks.w;
      }
      if (!(ok = wait_bar_warp(cx, cx.bar(kBarSFull + i), static_cast<uint32_t>(j) & 1u))) break;
      tc::tc_fence_after();
      uint32_t sr[kB][32];
#pragma unroll
      for (int b = 0; b < kB; ++b) tc::tmem_ld32(tS + 32u * b, sr[b]);
      tc::tmem_wait_ld();
      tc::tc_fence_before();
      tc::mbar_arrive(cx.bar(kBarSFree + i));  // the next QK may overwrite S
      float cb[kB];
      int lim[kB];  // tokens of each block that the row sees
      bool masked = (j + 1) * S::kKeysPerStep > all_see;
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        const float k = kB == 4 || in == 0 ? k4[b] : k4[(b + 2) & 3];
        cb[b] = f * k;
        lim[b] = k < 0.0f ? 0 : sees - j * S::kKeysPerStep - 32 * b;
        masked |= k < 0.0f;
      }
      float mt = -INFINITY;
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        if (masked) {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (value_token(c) >= lim[b]) sr[b][c] = 0xFF800000u;
        }
        float m0 = __uint_as_float(sr[b][0]), m1 = __uint_as_float(sr[b][1]);
#pragma unroll
        for (int c = 2; c < 30; c += 4) {
          m0 = max3(m0, __uint_as_float(sr[b][c]), __uint_as_float(sr[b][c + 1]));
          m1 = max3(m1, __uint_as_float(sr[b][c + 2]), __uint_as_float(sr[b][c + 3]));
        }
        m0 = max3(m0, __uint_as_float(sr[b][30]), __uint_as_float(sr[b][31]));
        m0 = fmaxf(m0, m1);
        mt = fmaxf(mt, m0 == -INFINITY ? m0 : m0 * cb[b]);
      }
      if (__any_sync(0xffffffffu, mt > m + kLazy)) {
        const float up = fmaxf(m, mt);
        const float alpha = up == -INFINITY ? 1.0f : ex2(m - up);
        m = up;
        l *= alpha;
        if (j > 0) {
          if (!(ok = wait_pv(j - 1))) break;  // O is at rest
          tc::tc_fence_after();
          const float2 a2 = make_float2(alpha, alpha);
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tc::tmem_ld32(tO + 32u * c, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const float2 y = __fmul2_rn(make_float2(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), a2);
              o[k] = __float_as_uint(y.x);
              o[k + 1] = __float_as_uint(y.y);
            }
            tc::tmem_st32(tO + 32u * c, o);
          }
        }
      }
      const float ref = m == -INFINITY ? 0.0f : m;
      const float2 n2 = make_float2(-ref, -ref);
      float2 sa = make_float2(0.0f, 0.0f), sb = make_float2(0.0f, 0.0f);
      uint32_t pw[kB / 2][32];
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        const float2 c2 = make_float2(cb[b], cb[b]);
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const float2 y = __ffma2_rn(make_float2(__uint_as_float(sr[b][c]), __uint_as_float(sr[b][c + 1])), c2, n2);
          float2 p = make_float2(ex2(y.x), ex2(y.y));
          if (masked) {
            if (value_token(c) >= lim[b]) p.x = 0.0f;
            if (value_token(c + 1) >= lim[b]) p.y = 0.0f;
          }
          if (c & 2) sb = __fadd2_rn(sb, p);
          else sa = __fadd2_rn(sa, p);
          pw[b / 2][16 * (b & 1) + c / 2] = pack_half2(p.x, p.y);
        }
      }
      l += (sa.x + sa.y) + (sb.x + sb.y);
      if (j >= S::kP) {
        if (!(ok = wait_pv(j - S::kP))) break;  // the buffer's last PV has read it
        tc::tc_fence_after();
      }
      const uint32_t tP = tmem + lane_addr + S::col_p(i, j % S::kP);
#pragma unroll
      for (int x = 0; x < kB / 2; ++x) tc::tmem_st32(tP + 32u * x, pw[x]);
      tc::tmem_wait_st();
      tc::tc_fence_before();
      tc::mbar_arrive(cx.bar(kBarPFull + i));
    }
    // epilogue
    if (ok && n > 0) {
      ok = wait_pv(n - 1);
      tc::tc_fence_after();
    }
    const float* tops = reinterpret_cast<const float*>(smem + T::kOffTop);
    if (!real) l = 0.0f;
    if (ok || i >= u.tiles) {
      const bool empty = i >= u.tiles || u.n[i] == 0;
      const bool pad = !real && a.zero_rest && r < static_cast<int>(a.T) * u.G;
      const float top = empty ? 0.0f : fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
      const float inv = l == 0.0f ? 0.0f : top / l;
      uint16_t* dst = a.out.p + u.b * a.out.sb + tok * a.out.ss + head * a.out.sh;
      if (a.lse != nullptr && (real || pad))
        a.lse[(static_cast<int64_t>(u.b) * a.H + head) * a.T + tok] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (!empty) {
          tc::tmem_ld32(tO + 32u * c, o);
          tc::tmem_wait_ld();
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = (empty || l == 0.0f) ? 0.0f : __uint_as_float(o[8 * k + 2 * e]) * inv;
            const float y = (empty || l == 0.0f) ? 0.0f : __uint_as_float(o[8 * k + 2 * e + 1]) * inv;
            const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
            w[e] = *reinterpret_cast<const uint32_t*>(&v);
          }
          if (real || pad) *reinterpret_cast<uint4*>(dst + 32 * c + 8 * k) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    tc::tc_fence_before();
    __syncwarp();
    regs_dec<kRegCtl>();
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t launch_cache_attention_tc(const CacheAttentionArgs& a, int64_t D, cudaStream_t stream) {
  const int64_t rows = a.T * (a.H / a.c.H);
  const int64_t pairs = div_up(rows, 2 * kRows);
  const int64_t units = pairs * a.B * a.c.H;
  if (units > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const auto kernel = D == 128 ? cache_attention_tc_kernel<128> : cache_attention_tc_kernel<64>;
  const int bytes = static_cast<int>(D == 128 ? SmemTail<128>::kBytes : SmemTail<64>::kBytes);
  cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(kernel), bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(bytes);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, static_cast<int>(pairs));
}

}  // namespace sage
