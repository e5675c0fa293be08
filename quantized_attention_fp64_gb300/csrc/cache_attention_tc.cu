// Attention of many query rows to an 8-bit paged cache (prompt chunks, cross
// attention): the tensor-core form of cache_attention.cu's formulas.
//
// A work unit is one key/value head of one sequence and a pair of tiles of 128
// query rows (query tokens x the heads that share the key/value head, token
// major), so the codes of a key tile (64 keys) are converted once for 256 rows.
// The key tiles of all units form one list (pair, head, tile) that is cut into
// equal ranges, one per CTA and SM, whatever the lengths and the mask; a unit
// that several CTAs share leaves its parts in the workspace (at most two per
// CTA, as in cache_attention.cu), and a second kernel joins them. 16 warps:
//   warps 0, 1    one MMA-issuing thread per query tile
//   warp 2        TMEM allocation
//   warps 4-7, 8-11  softmax of query tile 0, 1 (TMEM lane = row)
//   warp 3        where there is one query tile only (kOne, below): brings the codes
//   warps 12-15   converters: read the int8 codes of a key tile (two warps per
//                 32-key block, 16 bytes per lane and load, the next tile's
//                 loads in flight in registers), turn them into fp16 and store
//                 them in the 128-byte-swizzled layout that the MMA reads, four
//                 tiles ahead (eight at D = 64); they also bring the queries
//                 and run ahead into the next unit
// Per query tile and key tile j: S = Q K_j^T (tcgen05 kind::f16, fp32 in TMEM)
// into one of two buffers; the softmax reads S into registers and writes p as
// fp16 over it, and O += P V_j reads it there (P in shared memory would double
// what the products read from it). QK_{j+1} fills the other buffer meanwhile,
// and QK_{j+2} waits for PV_j. The columns hold, per query tile, D of O and two
// times 64 of S.
// Numbers. Queries become fp16 times a power of two per row (their largest
// value in [1, 4)); key and value codes are exact in fp16. The value scales go
// into the weights: with m a row's running maximum of z + log2 s_v (z: the
// logits times log2 e), P holds fp16(2^(z + log2 s_v - m)), a rounding of 2^-11
// of the weight (where it is below 2^-14 of the largest, of 2^-25 of that),
// O = sum P vcode, and the sum of 2^(z - m) is taken in fp32, block by block,
// from the weights before they are rounded, over s_v (or apart from them, see
// cache.cuh). So what a row does not see, whatever its scale, does not touch it.
// The keys of a block stand in the order in which the values are stored
// (value_position), so V^T needs no reordering on the way.
//
// Every wait on an mbarrier is bounded, as in attention_tc.cu.
// Measured (GB300): a causal chunk of 2000 tokens over 16001, 32 heads on 8 of
// 128: 396 us, 1240 TFLOP/s, 65% of cuBLAS's bf16 rate; the tensor pipe is busy
// 71% of the cycles (QK with 64 keys is bound by shared memory, which reads Q
// again for every key tile), and the chain of a key tile's softmax takes the
// rest. 2 x 4097 queries over up to 1500 states, 16 heads of 64: 96 us, 446
// TFLOP/s, of which the softmax's chain is 1300 cycles per 64 keys and beginning
// and ending a unit 4 us of every 20. What was slower: key tiles of 128 without a
// second buffer of S; S and P apart (404 us); four softmax warpgroups, and eight
// converter warps (both spill); waiting for keys and P by polling (410).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "cache.cuh"
#include "common.cuh"
#include "tc_ptx.cuh"

namespace sage {
namespace {

constexpr int kConv = 4;        // converter warps
constexpr int kThreads = 384 + 32 * kConv;
constexpr int kRows = 128;      // rows of a query tile
constexpr int kKeys = kTileKeys; // keys of a key tile
constexpr int kB = kKeys / kCacheBlock;  // blocks of a key tile
constexpr int kMaxSms = 160;
// Key tiles that are worth a CTA of their own: with n to a unit and p CTAs the
// tiles cost n / p and the join p, so p goes as the root of n (64 rows over 5000
// tokens, 4 heads, 20 us, 22 with two tiles each; 256 rows 27 and 34; over 1000 tokens
// 22, 21 with two and 26 with six).
__host__ __device__ inline int least_tiles(int64_t n) {
  const int least = static_cast<int>(sqrtf(0.4f * static_cast<float>(n)) + 0.5f);
  return least > 2 ? least : 2;
}
constexpr int kWindow = 32;     // key tiles whose pages and scales are looked up together
constexpr int kWindows = 16;    // lookups that are kept (more than the stages and what lies between)
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 6.0f;     // where the maximum is looked for: a weight may reach 2^6 before the running one follows
constexpr float kMost = 4096.0f;  // elsewhere: the sum of a block's weights may (then some weight is above 2^7)
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr uint32_t kTmemCols = 512;

// registers per thread of the control, converter and softmax warps
constexpr uint32_t kRegCtl = 56, kRegConv = 104, kRegSoftmax = 176;
constexpr uint32_t kRegLaunch = 65536 / kThreads / 8 * 8;
static_assert(128 * kRegCtl + 32 * kConv * kRegConv + 256 * kRegSoftmax <= kThreads * kRegLaunch,
              "registers that the CTA is launched with");

template <int D, bool kOne>
struct Smem {
  static constexpr uint32_t kSub = 128 * 128;             // 64 channels of 128 rows, fp16
  static constexpr uint32_t kTile = (D / 64) * kSub;      // a query tile
  static constexpr int kQTiles = kOne ? 1 : 2;            // of a unit
  static constexpr uint32_t kSubK = kKeys * 128;          // 64 channels of a key tile
  static constexpr uint32_t kTileKV = (D / 64) * kSubK;   // keys; values are D rows of 64 keys
  static constexpr int kStages = D == 128 ? 4 : 8;        // key and value tiles
  static constexpr int kQ = D == 128 ? 1 : 2;             // units whose queries are kept
  // key and value tiles as codes, where they wait in shared memory
  static constexpr int kRaw = !kOne ? 1 : (D == 128 ? 3 : 6);
  static constexpr uint32_t kRawBlock = kCacheBlock * D;  // bytes of a block's keys or values
  static constexpr uint32_t kOffQ = 0;                    // [unit][tile]
  static constexpr uint32_t kOffK = kOffQ + kQ * kQTiles * kTile;
  static constexpr uint32_t kOffV = kOffK + kStages * kTileKV;
  static constexpr uint32_t kOffRaw = kOffV + kStages * kTileKV;         // [stage] keys of the blocks, values of the blocks
  static constexpr uint32_t kOffBar = kOffRaw + (kOne ? kRaw * 2 * kB * kRawBlock : 0);
};
constexpr int kMaxStages = 8, kMaxRaw = 6;
constexpr int kBarQFull = 0, kBarQEmpty = 2, kBarFull = kBarQEmpty + 2, kBarEmpty = kBarFull + kMaxStages;
constexpr int kBarSFull = kBarEmpty + kMaxStages, kBarPFull = kBarSFull + 4;
constexpr int kBarPVDone = kBarPFull + 4, kBarDrain = kBarPVDone + 4;  // SFull, PFull, PVDone: [tile][buffer]
constexpr int kBarFold = kBarDrain + 2;  // the second half of a folded part is in the workspace; it has been read
constexpr int kBarRaw = kBarFold + 2, kBarRawFree = kBarRaw + kMaxRaw;
constexpr int kNumBars = kBarRawFree + kMaxRaw;
template <int D, bool kOne>
struct SmemTail {
  static constexpr uint32_t kOffAbort = Smem<D, kOne>::kOffBar + kNumBars * 8;  // as Ctx::abort_at has it
  static constexpr uint32_t kOffTmem = kOffAbort + 4;
  // [window][tile] two key scales, two log2 s_v
  static constexpr uint32_t kOffScale = (kOffTmem + 4 + 15) / 16 * 16;
  static_assert(kOffScale % 16 == 0, "a tile's scales are read as one float4");
  // a sum per warp, then where the CTA's range begins and how the list is cut
  static constexpr uint32_t kOffPlan = kOffScale + kWindows * kWindow * 16;
  static constexpr uint32_t kOffRow = kOffPlan + (kThreads / 32 + 8) * 4;                // [unit][256 rows] powers of two of the queries
  // one unit more than of the queries themselves: those are free once the
  // unit's last QK is done, when a softmax thread may still have to read its
  // factor; an issuer goes on to the next unit only after the softmax did
  static constexpr int kRowUnits = Smem<D, kOne>::kQ + 1;
  static constexpr uint32_t kBytes = kOffRow + kRowUnits * 2 * kRows * 4;
  // workspace: a descriptor of each CTA's last unit, then two slots per CTA
  static constexpr size_t kDesc = size_t(kMaxSms) * sizeof(int4);
  static constexpr size_t kSlot = size_t(2) * kRows * (D + 2);          // floats
  static constexpr size_t kWorkspace = kDesc + size_t(kMaxSms) * 2 * kSlot * 4;
};
static_assert(SmemTail<128, false>::kBytes <= 232448u && SmemTail<128, true>::kBytes <= 232448u &&
                  SmemTail<64, false>::kBytes <= 232448u && SmemTail<64, true>::kBytes <= 232448u,
              "shared memory of one CTA");
static_assert(SmemTail<128, true>::kWorkspace == SmemTail<128, false>::kWorkspace &&
                  SmemTail<64, true>::kWorkspace == SmemTail<64, false>::kWorkspace,
              "one workspace");

constexpr int kS = 2;                    // buffers of S and P
// TMEM columns of the query tiles
template <int D>
struct Cols {
  __host__ __device__ static constexpr uint32_t o(int i) { return 128u * static_cast<uint32_t>(i); }
  __host__ __device__ static constexpr uint32_t s(int i, int buf) {
    return 256u + 128u * static_cast<uint32_t>(i) + 64u * static_cast<uint32_t>(buf);
  }
};

// One arrival for the warp, after what its lanes did (an arrival per lane would
// be 32 atomics on one word).
__device__ __forceinline__ void arrive_warp(uint32_t bar, int lane) {
  __syncwarp();
  if (lane == 0) tc::mbar_arrive(bar);
}

// Barriers and the abort flag by their shared-memory addresses.
struct Ctx {
  uint32_t bar0;
  __device__ uint32_t abort_at() const { return bar0 + 8u * kNumBars; }
  __device__ uint32_t bar(int i) const { return bar0 + 8u * static_cast<uint32_t>(i); }
};
__device__ __forceinline__ uint32_t load_flag(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void store_flag(uint32_t addr, uint32_t v) {
  asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Bounded wait: when it runs out it raises the abort flag, which ends every
// other wait of the CTA; the error word is set at the CTA's end.
template <bool kHeedAbort = true>
__device__ __forceinline__ bool wait_bar(const Ctx& cx, uint32_t bar, uint32_t parity) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if ((it & 127u) == 0) {
      if (kHeedAbort && load_flag(cx.abort_at()) != 0) return false;
      const uint64_t now = tc::global_timer_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > kTimeoutNs) {
        store_flag(cx.abort_at(), 1u);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait_bar_warp(const Ctx& cx, uint32_t bar, uint32_t parity) {
  const bool ok = wait_bar(cx, bar, parity);
  return __all_sync(0xffffffffu, ok);
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

// 32 lanes x 16 columns (as tc::tmem_ld32).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
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
__device__ __forceinline__ void store16(uint32_t addr, const uint32_t* o) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
               : "memory");
}
__device__ __forceinline__ uint4 load16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
// A whole sector of global memory (32-byte aligned). A thread writes its own
// row, so two halves would be two writes to L2: 110 -> 106 us there.
__device__ __forceinline__ void store32(void* to, const uint32_t* o) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]),
               "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
               : "memory");
}
__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// A pair of query tiles of one key/value head.
struct Unit {
  int b, h, len, q_len, R, G;
  int row0, tiles;  // first row, query tiles with rows
  int n[2], n_max;  // key tiles of each query tile
};

// Keys that a row sees (a row past the last counts as the last).
__device__ __forceinline__ int row_sees(const CacheAttentionArgs& a, const Unit& u, int r) {
  if (!a.causal) return u.len;
  const int tok = min(r, u.R - 1) / u.G;
  return max(u.len - u.q_len + tok + 1, 0);
}

// Entry e of the list of (sequence, pair), without its head.
__device__ __forceinline__ Unit find_entry(const CacheAttentionArgs& a, int pairs, int e, bool* bad) {
  Unit u;
  u.b = e / pairs;
  u.h = 0;
  u.len = static_cast<int>(checked_length(a.lengths[u.b], table_capacity(a.pt.max_pages, a.c.blocks_per_page), bad));
  u.q_len = static_cast<int>(a.q_lengths != nullptr ? checked_length(a.q_lengths[u.b], a.T, bad) : a.T);
  u.G = a.H / a.c.H;
  u.R = u.q_len * u.G;
  u.row0 = (e - u.b * pairs) * 2 * kRows;
  u.tiles = u.row0 >= u.R ? 0 : (u.row0 + kRows >= u.R ? 1 : 2);
  u.n_max = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    u.n[i] = i < u.tiles ? key_tiles(row_sees(a, u, u.row0 + i * kRows + kRows - 1)) : 0;
    u.n_max = max(u.n_max, u.n[i]);
  }
  return u;
}

__device__ __forceinline__ int unit_size(const Unit& u) { return max(u.n_max, 1); }

// The list counts a unit's key tiles and, before them, kBegin more: what
// beginning a unit and bringing its rows out costs (2 x 4097 rows of 16 heads
// of 64 over up to 1500 keys: 106 us without, 96 with; between 3 and 11 both
// head dimensions measure within 2%).
template <int D>
constexpr int kBegin = D == 128 ? 8 : 6;

// A CTA's place in the list, `at` entries of the list into head h of entry e,
// with `todo` left in its range. The part of the range that lies in this unit
// is its next n, key tiles [t, t + tiles); a unit that sees no key or has no
// rows counts as one tile (its rows still have outputs). A part without tiles
// (the range ends where the unit begins) stands for nothing. The unit is found
// anew where it is needed: that costs less than the registers to keep it.
struct Place {
  int e, h, at, todo;
};
struct Part {
  Unit u;
  int n;                // of the list
  int t, tiles, size;   // key tiles: first of the part, of the part, of the unit
};
template <int D>
__device__ __forceinline__ Part part_at(const CacheAttentionArgs& a, int pairs, const Place& p) {
  bool bad = false;
  Part x;
  x.u = find_entry(a, pairs, p.e, &bad);
  x.u.h = p.h;
  x.size = unit_size(x.u);
  x.n = min(x.size + kBegin<D> - p.at, p.todo);
  x.t = max(p.at - kBegin<D>, 0);
  x.tiles = max(p.at + x.n - kBegin<D>, 0) - x.t;
  return x;
}
__device__ __forceinline__ Place first_place(const int* found) { return Place{found[0], found[1], found[2], found[3]}; }
// Past a part of n tiles.
__device__ __forceinline__ void place_next(const CacheAttentionArgs& a, Place& p, int n) {
  p.todo -= n;
  p.at = 0;
  if (++p.h == a.c.H) {
    p.h = 0;
    ++p.e;
  }
}
// Key tiles of query tile i in the part.
__device__ __forceinline__ int part_tiles(const Part& x, int i) {
  return max(min(x.t + x.tiles, i == 0 ? x.u.n[0] : x.u.n[1]) - x.t, 0);
}

// kOne (at most 128 query rows of a key/value head, so one query tile). A part
// of kFold key tiles or more is folded: tile slot i takes its key tiles i,
// i + 2, ..., both slots with the same queries, and slot 0 joins the two at the
// part's end, through rows of the workspace that the part leaves free. Shorter
// parts do not pay for the join. And warp 3 sends for the codes with bulk
// copies, where the second query tile's room lets some wait in shared memory.
// 40 rows over 14 x 20000 tokens, 8 heads of 128: 231 us as the form for more
// rows does it, 241 with folding alone, 215 with the copies alone, 176 with
// both (now 171); what bounds it is the conversion of the codes, which takes no
// less for fewer rows (32 rows, without tensor memory: 137 us).
constexpr int kFold = 8;
static_assert(kWindow % 2 == 0, "a folded query tile begins a window at its own first tile of it");
__device__ __forceinline__ bool folds(const Part& x) { return x.u.tiles == 1 && x.tiles >= kFold; }

template <int D>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint64_t dq, uint64_t dk) {
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks) {
    const uint32_t sub = static_cast<uint32_t>(ks >> 2), off = static_cast<uint32_t>(ks & 3) * 32u;
    tc::mma_f16_ss(d_tmem, desc_at(dq, sub * Smem<D, false>::kSub + off), desc_at(dk, sub * Smem<D, false>::kSubK + off),
                   tc::kIdescM128N64, ks > 0 ? 1u : 0u);
  }
}
template <int D>
__device__ __forceinline__ void issue_pv(uint32_t d_tmem, uint32_t tp, uint64_t dv, bool acc) {
  constexpr uint32_t idesc = D == 128 ? tc::kIdescM128N128 : tc::kIdescM128N64;
#pragma unroll
  for (int ks = 0; ks < kKeys / 16; ++ks)
    mma_f16_ts(d_tmem, tp + 8u * static_cast<uint32_t>(ks), desc_at(dv, 32u * static_cast<uint32_t>(ks)), idesc,
               (acc || ks > 0) ? 1u : 0u);
}

// 16 codes to fp16, into chunks c and c + 1 of a 128-byte row in the swizzled layout (sw: the row mod 8).
__device__ __forceinline__ void store_codes(uint32_t row, uint32_t c, uint32_t sw, const uint4& codes) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  uint32_t o[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    __half2 lo, hi;
    codes_to_half(w[e], lo, hi);
    o[2 * e] = bits(lo);
    o[2 * e + 1] = bits(hi);
  }
  store16(row + ((c ^ sw) << 4), o);
  store16(row + (((c + 1u) ^ sw) << 4), o + 4);
}

// A block of the cache as a converter lane keeps it. One that is not there
// (bad page, or past the sequence) stands at the cache's start: its codes are
// read and get the weight 0.
struct Window {
  int64_t at;  // first byte in the codes
  float ks, vs;
};
// The key scale as the softmax reads it, of the block that the lane looked up for
// its tile: below 0 (its sign bit is set) where the tile is not a plain one. That is
// because the block has no tokens, because its value scale is an odd one, or because
// it follows a large one in its half of the part's tiles (*large: in an earlier
// window). The other block of the tile may be the only one that has tokens, so one
// that has none says whether it follows a large one, too.
constexpr float kNoTokens = -INFINITY, kNoTokensOdd = -3e38f;  // (no scale is as large)
__device__ __forceinline__ bool marked(float ks) { return __float_as_int(ks) < 0; }
__device__ __forceinline__ bool has_tokens(float ks) { return !(ks <= kNoTokensOdd); }
__device__ __forceinline__ bool marked_odd(float ks) { return marked(ks) && ks != kNoTokens; }
__device__ __forceinline__ float mark(const Window& w, int lane, bool* large) {
  const float lv = log_scale(w.vs);
  const uint32_t above = __ballot_sync(0xffffffffu, lv > kLogPlainMax);
  const bool follows = *large || (above << (31 - lane)) != 0u;  // (or is one)
  *large |= above != 0u;
  if (w.ks < 0.0f) return follows ? kNoTokensOdd : kNoTokens;
  return follows || lv < kLogPlainMin ? -fabsf(w.ks) : fabsf(w.ks);
}
template <int D>
__device__ __forceinline__ Window load_window(const CacheAttentionArgs& a, int64_t row_of_table, int h, int len, int blk,
                                              bool* bad) {
  Window w;
  w.at = 0;
  w.ks = kNoTokens;
  w.vs = 0.0f;
  if (block_has_tokens(blk, len)) {
    const int pg = blk / a.c.blocks_per_page;
    const int page = a.pt.table[row_of_table + pg];
    if (page_ok(page, a.c.num_pages)) {
      const int64_t slot = block_slot(page, h, a.c.H, a.c.blocks_per_page, blk - pg * a.c.blocks_per_page);
      w.at = slot * (kCacheBlock * D);
      w.ks = a.c.ks[slot];
      w.vs = a.c.vs[slot];
    } else {
      *bad = true;
    }
  }
  return w;
}

// One block of a row: the weights 2^(s c + n) of its 32 scores, in fp16, and
// their sum. kMasked: from token lim on they are 0, whatever s and c are.
template <bool kMasked>
__device__ __forceinline__ float exp_block(const uint32_t (&s)[32], float c, float n, int lim, uint32_t (&pw)[16]) {
  const float2 c2 = make_float2(c, c), n2 = make_float2(n, n);
  float2 sa = make_float2(0.0f, 0.0f), sb = sa;
#pragma unroll
  for (int k = 0; k < 32; k += 2) {
    const float2 y = __ffma2_rn(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), c2, n2);
    float2 p = make_float2(ex2(y.x), ex2(y.y));
    if (kMasked) {
      if (value_token(k) >= lim) p.x = 0.0f;
      if (value_token(k + 1) >= lim) p.y = 0.0f;
    }
    if (k & 2) sb = __fadd2_rn(sb, p);
    else sa = __fadd2_rn(sa, p);
    pw[k / 2] = pack_half2(p.x, p.y);
  }
  return (sa.x + sa.y) + (sb.x + sb.y);
}

// What 16 keys (positions 16 h and up of a block, h = 0 or 1) of which the row sees
// those of the block's first lim tokens add to its sum, apart from their weights:
// 2^(s c - m), with s from tensor memory.
__device__ __forceinline__ float part_of_sum(uint32_t taddr, int h, float c, float m, int lim) {
  uint32_t s[16];
  tmem_ld16(taddr, s);
  tc::tmem_wait_ld();
  float top = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; ++k)
    if (value_token(k) + 4 * h < lim) top = fmaxf(top, __uint_as_float(s[k]) * c);
#pragma unroll
  for (int k = 0; k < 16; ++k)
    if (value_token(k) + 4 * h < lim) sum += ex2(fmaf(__uint_as_float(s[k]), c, -top));
  return sum == 0.0f ? 0.0f : rescale(sum, half_step(top, m));
}

template <int D, bool kOne>
__global__ void __launch_bounds__(kThreads, 1) cache_attention_tc_kernel(const CacheAttentionArgs a, int pairs) {
  using L = Smem<D, kOne>;
  using T = SmemTail<D, kOne>;
  using C = Cols<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((tc::smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicExch(a.dev_err, kDevErrSmemAlign);
    return;
  }
  const uint32_t sbase = tc::smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Ctx cx;
  cx.bar0 = sbase + L::kOffBar;
  if (threadIdx.x == 0) {
    store_flag(cx.abort_at(), 0u);
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(cx.bar(kBarQFull + s), kConv);
      tc::mbar_init(cx.bar(kBarQEmpty + s), 2);
      tc::mbar_init(cx.bar(kBarSFull + 2 * s), 2);
      tc::mbar_init(cx.bar(kBarSFull + 2 * s + 1), 2);
      tc::mbar_init(cx.bar(kBarPFull + 2 * s), kRows);
      tc::mbar_init(cx.bar(kBarPFull + 2 * s + 1), kRows);
      tc::mbar_init(cx.bar(kBarPVDone + 2 * s), 1);
      tc::mbar_init(cx.bar(kBarPVDone + 2 * s + 1), 1);
      tc::mbar_init(cx.bar(kBarDrain + s), 1);
    }
    for (int s = 0; s < L::kStages; ++s) {
      tc::mbar_init(cx.bar(kBarFull + s), kConv);
      tc::mbar_init(cx.bar(kBarEmpty + s), 2);
    }
    for (int s = 0; s < L::kRaw; ++s) {
      tc::mbar_init(cx.bar(kBarRaw + s), 1);
      tc::mbar_init(cx.bar(kBarRawFree + s), kConv);
    }
    tc::mbar_init(cx.bar(kBarFold), kRows);
    tc::mbar_init(cx.bar(kBarFold + 1), kRows);
    tc::fence_mbar_init();
  }
  if (warp == 2) {
    tc::tmem_alloc(sbase + T::kOffTmem, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::griddep_wait();
  tc::griddep_launch_dependents();

  // this CTA's range of the list: each thread sums a run of entries, a scan over
  // the threads finds whose run the range begins in
  int* plan = reinterpret_cast<int*>(smem + T::kOffPlan);
  int* found = plan + kThreads / 32;  // entry, head, tile, tiles; end of the range; how the list is cut
  bool bad = false;
  const int entries = static_cast<int>(a.B) * pairs, run = (entries + kThreads - 1) / kThreads;
  const int e_lo = min(run * static_cast<int>(threadIdx.x), entries), e_hi = min(e_lo + run, entries);
  int mine = 0;
  for (int e = e_lo; e < e_hi; ++e) mine += unit_size(find_entry(a, pairs, e, &bad)) + kBegin<D>;
  if (bad && blockIdx.x == 0) atomicExch(a.dev_err, kDevErrPage);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) plan[warp] = incl;
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + T::kOffTmem);
  int before = incl - mine, W = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += plan[w];
    W += plan[w];
  }
  W *= a.c.H;
  before *= a.c.H;
  const int units = entries * a.c.H;
  // no more CTAs than units, unless each still gets a few key tiles
  const int tiles = W - units * kBegin<D>;
  const int ctas = min(static_cast<int>(gridDim.x), max(units, tiles / least_tiles(tiles / units)));
  const int each = W / ctas, extra = W - each * ctas, c = static_cast<int>(blockIdx.x);
  const int lo = c < ctas ? c * each + min(c, extra) : 0, hi = c < ctas ? lo + each + (c < extra ? 1 : 0) : 0;
  if (lo < hi && before <= lo && lo < before + mine * a.c.H) {
    int e = e_lo;
    for (;; ++e) {
      const int x = (unit_size(find_entry(a, pairs, e, &bad)) + kBegin<D>) * a.c.H;
      if (lo < before + x) break;
      before += x;
    }
    const int size = unit_size(find_entry(a, pairs, e, &bad)) + kBegin<D>, h = (lo - before) / size;
    found[0] = e;
    found[1] = h;
    found[2] = lo - before - h * size;
  }
  if (threadIdx.x == 0) {
    found[3] = hi - lo;
    found[4] = hi;
    found[5] = each;
    found[6] = extra;
    // what stands if a wait runs out, or without work
    static_cast<int4*>(a.workspace)[blockIdx.x] = make_int4(-1, 0, 0, 0);
  }
  __syncthreads();

  if (warp < 4) {
    regs_dec<kRegCtl>();
    if (warp < 2) {
      // ------------------------------------------------ MMA issuer of tile i --
      const int i = warp;
      const bool leader = elect_one();
      const uint32_t d_o = tmem + C::o(i);
      const uint64_t dq0 = tc::sw128_desc(sbase + L::kOffQ);
      const uint64_t dk0 = tc::sw128_desc(sbase + L::kOffK), dv0 = tc::sw128_desc(sbase + L::kOffV);
      // key tiles (of the converters, of this query tile) and parts so far
      uint32_t cnt = 0, steps = 0, q_cnt = 0;
      bool ok = true;
      Place p = first_place(found);
      while (ok && p.todo > 0) {
        const Part x = part_at<D>(a, pairs, p);
        const int n_all = max(part_tiles(x, 0), part_tiles(x, 1));  // of the converters
        const int fold = kOne && folds(x) ? 1 : 0;
        const int n = fold ? (n_all + 1 - i) >> 1 : part_tiles(x, i);  // of this query tile
        const auto mine = [&](int j) { return fold ? (j & 1) == i : j < n; };
        place_next(a, p, x.n);
        if (n_all == 0) continue;
        const uint32_t qb = q_cnt % L::kQ;
        if (!(ok = wait_bar_warp(cx, cx.bar(kBarQFull + static_cast<int>(qb)), (q_cnt / L::kQ) & 1u))) break;
        ++q_cnt;
        if (n == 0 && leader) tc::mbar_arrive(cx.bar(kBarQEmpty + static_cast<int>(qb)));
        const uint64_t dq = desc_at(dq0, (qb * L::kQTiles + (kOne ? 0u : static_cast<uint32_t>(i))) * L::kTile);
        // PV_j once P_j is there (its values came with its keys)
        const auto pv = [&](int j) {
          const int s = static_cast<int>((cnt + static_cast<uint32_t>(j)) % L::kStages);
          if (mine(j)) {
            const uint32_t st = steps + static_cast<uint32_t>(j >> fold);
            const int buf = static_cast<int>(st % kS);
            if (!wait_bar_warp(cx, cx.bar(kBarPFull + 2 * i + buf), (st / kS) & 1u)) return false;
            tc::tc_fence_after();
            if (leader) {
              issue_pv<D>(d_o, tmem + C::s(i, buf), desc_at(dv0, static_cast<uint32_t>(s) * L::kTileKV), j > fold);
              tc::mma_commit(cx.bar(kBarPVDone + 2 * i + buf));
              tc::mma_commit(cx.bar(kBarEmpty + s));
            }
          } else if (leader) {
            tc::mbar_arrive(cx.bar(kBarEmpty + s));  // no row of this query tile sees the keys
          }
          __syncwarp();
          return true;
        };
        // PV_j follows this query tile's next QK
        for (int j = 0; ok && j <= n_all + fold; ++j) {
          bool pending = j > fold;
          if (j < n_all) {
            const uint32_t at = cnt + static_cast<uint32_t>(j), s = at % L::kStages, ph = (at / L::kStages) & 1u;
            const uint32_t full = cx.bar(kBarFull + static_cast<int>(s));
            // keys that are late do not hold up the last tile's PV
            if (pending && !__any_sync(0xffffffffu, tc::mbar_try_wait(full, ph))) {
              if (!(ok = pv(j - 1 - fold))) break;
              pending = false;
            }
            // QK_j once its keys are there and PV_{j-2} has read P in its buffer
            if (!(ok = wait_bar_warp(cx, full, ph))) break;
            if (mine(j)) {
              const uint32_t st = steps + static_cast<uint32_t>(j >> fold);
              const int buf = static_cast<int>(st % kS);
              if (st >= kS && !(ok = wait_bar_warp(cx, cx.bar(kBarPVDone + 2 * i + buf), (st / kS - 1u) & 1u))) break;
              tc::tc_fence_after();
              if (leader) {
                // S is there when the MMAs are done; the plain arrival passes on what the
                // converters wrote: scales, powers of two
                tc::mbar_arrive(cx.bar(kBarSFull + 2 * i + buf));
                issue_qk<D>(tmem + C::s(i, buf), dq, desc_at(dk0, s * L::kTileKV));
                tc::mma_commit(cx.bar(kBarSFull + 2 * i + buf));
                if ((j >> fold) == n - 1) tc::mma_commit(cx.bar(kBarQEmpty + static_cast<int>(qb)));
              }
              __syncwarp();
            }
          }
          if (pending && !(ok = pv(j - 1 - fold))) break;
        }
        cnt += static_cast<uint32_t>(n_all);
        steps += static_cast<uint32_t>(n);
      }
      // all MMAs of this warp complete before TMEM is freed
      if (leader) tc::mma_commit(cx.bar(kBarDrain + i));
      __syncwarp();
      wait_bar<false>(cx, cx.bar(kBarDrain + i), 0);
    } else if (kOne && warp == 3) {
      // ----------------------------------------------------- codes in advance --
      // Looks 32 key tiles up at a time, two blocks a lane, and sends for them
      // with bulk copies, kRaw tiles ahead of the converters.
      uint32_t sent = 0, windows = 0;
      bool ok = true, bad_page = false;
      Place p = first_place(found);
      while (ok && p.todo > 0) {
        const Part x = part_at<D>(a, pairs, p);
        place_next(a, p, x.n);
        const int tiles = part_tiles(x, 0);
        Window win[kB];
        bool large[kB] = {};
        for (int j = 0; ok && j < tiles; ++j, ++sent) {
          if (j % kWindow == 0) {
#pragma unroll
            for (int b = 0; b < kB; ++b)
              win[b] = load_window<D>(a, x.u.b * a.pt.stride, x.u.h, x.u.len, (x.t + j + lane) * kB + b, &bad_page);
            const float k0 = mark(win[0], lane, &large[0]), k1 = mark(win[1], lane, &large[1]);
            reinterpret_cast<float4*>(smem + T::kOffScale)[windows % kWindows * kWindow + lane] =
                make_float4(k0, k1, log_scale(win[0].vs), log_scale(win[1].vs));
            ++windows;
          }
          const int64_t at0 = __shfl_sync(0xffffffffu, win[0].at, j % kWindow);
          const int64_t at1 = __shfl_sync(0xffffffffu, win[1].at, j % kWindow);
          const uint32_t r = sent % L::kRaw;
          const uint32_t bar = cx.bar(kBarRaw + static_cast<int>(r));
          if (!(ok = wait_bar_warp(cx, cx.bar(kBarRawFree + static_cast<int>(r)), ((sent / L::kRaw) & 1u) ^ 1u))) break;
          if (lane == 0) tc::mbar_arrive_expect_tx(bar, 2 * kB * L::kRawBlock);
          __syncwarp();
          if (lane < 2 * kB)  // keys of block 0, 1, values of block 0, 1
            tc::bulk_load(sbase + L::kOffRaw + (r * 2 * kB + static_cast<uint32_t>(lane)) * L::kRawBlock,
                          (lane < kB ? a.c.k : a.c.v) + ((lane & 1) ? at1 : at0), L::kRawBlock, bar);
        }
      }
      if (bad_page) atomicExch(a.dev_err, kDevErrPage);
      // copies in flight land before the CTA ends (some are left where a wait ran out)
      for (uint32_t k = sent < L::kRaw ? 0u : sent - L::kRaw; k < sent; ++k)
        wait_bar<false>(cx, cx.bar(kBarRaw + static_cast<int>(k % L::kRaw)), (k / L::kRaw) & 1u);
    }
    __syncwarp();
  } else if (warp >= 12) {
    // ------------------------------------------------------------ converters --
    regs_dec<kRegConv>();
    const int w = warp - 12, blk = w & 1, share = w >> 1;  // block of each key tile, share of its codes
    // Load x of the warp, of kLoads. Keys: 8 tokens of one 64-channel half,
    // channels 16 (lane mod 4) and up of token lane / 4. Values: 16 channels,
    // positions 16 (lane mod 2) and up of channel v_ch, which is lane / 2 with
    // its bits 1 and 2 exchanged: the 8 lanes of a store phase then write
    // channels c, c + 1, c + 4, c + 5, whose swizzled chunks are all different.
    constexpr int kLoads = 2 * D / 16 / kConv;
    const int v_ch = ((lane >> 1) & 9) | ((lane >> 1) & 2) << 1 | ((lane >> 1) & 4) >> 1;
    const int v_at = 2 * v_ch + (lane & 1);
    bool bad_page = false, ok = true;
    // the tile that is fetched next: tile t of t_end of the unit at `p`
    Place p = first_place(found);
    int t = 0, t_end = 0, n = 0, len = 0;
    int64_t row_of_table = 0;
    uint32_t windows = 0, parts = 0;
    Window win{0, kNoTokens, 0.0f};
    int64_t at = 0;  // the block's first byte in the codes
    int in_window = 0, head = 0;
    bool large = false;  // a large value scale in the part's earlier windows
    // looks the next 32 tiles up; the softmax's view: key scales, marked, and log2 s_v
    const auto open_window = [&]() {
      win = load_window<D>(a, row_of_table, head, len, (t + lane) * kB + blk, &bad_page);
      const float ks = mark(win, lane, &large);
      reinterpret_cast<float*>(smem + T::kOffScale)[(windows % kWindows * kWindow + lane) * 4 + 2 * share + blk] =
          share == 0 ? ks : log_scale(win.vs);
      ++windows;
      in_window = 0;
    };
    const auto pick = [&]() { at = __shfl_sync(0xffffffffu, win.at, in_window); };
    // The queries of a unit to fp16, times a power of two per row, in the
    // swizzled layout: four lanes share a row, 8 rows of a warp at a time.
    const auto bring_queries = [&](const Unit& u) {
      const uint32_t qb = parts % L::kQ;
      if (!wait_bar_warp(cx, cx.bar(kBarQEmpty + static_cast<int>(qb)), ((parts / L::kQ) & 1u) ^ 1u)) {
        ok = false;
        return;
      }
      float* rows = reinterpret_cast<float*>(smem + T::kOffRow) + (parts % T::kRowUnits) * 2 * kRows;
      ++parts;
      const int g = lane >> 2, c4 = lane & 3;
      const uint16_t* base = a.q.p + u.b * a.q.sb + c4 * 16;
      constexpr int kTimes = L::kQTiles * kRows / (8 * kConv), kAhead = 256 / D;  // rows per lane, of which so many load together
#pragma unroll 1
      for (int it0 = 0; it0 < kTimes; it0 += kAhead) {
        uint4 x[kAhead][D / 32];
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
          const int r = u.row0 + ((it0 + y) * kConv + w) * 8 + g;
#pragma unroll
          for (int e = 0; e < D / 32; ++e) x[y][e] = make_uint4(0u, 0u, 0u, 0u);
          if (r < u.R) {
            const int tok = r / u.G;
            const uint4* src = reinterpret_cast<const uint4*>(base + tok * a.q.ss + (u.h * u.G + r - tok * u.G) * a.q.sh);
#pragma unroll
            for (int e = 0; e < D / 32; ++e) x[y][e] = src[(e >> 1) * 8 + (e & 1)];
          }
        }
#pragma unroll
        for (int y = 0; y < kAhead; ++y) {
          const int rr = ((it0 + y) * kConv + w) * 8 + g;
          uint32_t amax = 0;
#pragma unroll
          for (int e = 0; e < D / 32; ++e) {
            const uint32_t v[4] = {x[y][e].x, x[y][e].y, x[y][e].z, x[y][e].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) amax = max(amax, max(v[k] & 0x7FFFu, (v[k] >> 16) & 0x7FFFu));
          }
          amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
          amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
          uint32_t ex = amax >> 7;
          ex = ex == 255u ? 127u : min(max(ex, 1u), 253u);
          const float down = __uint_as_float((254u - ex) << 23);
          if (c4 == 0) rows[rr] = __uint_as_float(ex << 23);
          const uint32_t to = sbase + L::kOffQ + (qb * L::kQTiles + static_cast<uint32_t>(rr >> 7)) * L::kTile +
                              static_cast<uint32_t>(rr & 127) * 128u;
#pragma unroll
          for (int e = 0; e < D / 32; ++e) {
            const uint32_t v[4] = {x[y][e].x, x[y][e].y, x[y][e].z, x[y][e].w};
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              o[k] = pack_half2(__uint_as_float(v[k] << 16) * down, __uint_as_float(v[k] & 0xFFFF0000u) * down);
            const uint32_t ch = static_cast<uint32_t>(c4) * 2u + static_cast<uint32_t>(e & 1), sw = static_cast<uint32_t>(rr) & 7u;
            store16(to + static_cast<uint32_t>(e >> 1) * L::kSub + ((ch ^ sw) << 4), o);
          }
        }
      }
      tc::fence_proxy_async_smem();
      arrive_warp(cx.bar(kBarQFull + static_cast<int>(qb)), lane);
    };
    // the warp's share of a tile's codes, into stage s
    const auto put_keys = [&](uint32_t s, const uint4 (&kr)[kLoads]) {
      const uint32_t k_row = sbase + L::kOffK + s * L::kTileKV;
#pragma unroll
      for (int x = 0; x < kLoads; ++x) {
        const int at8 = share * kLoads + x, j8 = at8 & 3, hf = at8 >> 2;  // eight tokens of a 64-channel half
        const int n8 = lane >> 2, row = blk * 32 + 8 * (n8 >> 1) + 2 * j8 + (n8 & 1);  // value_position of token 8 j8 + n8
        store_codes(k_row + static_cast<uint32_t>(hf) * L::kSubK + static_cast<uint32_t>(row) * 128u,
                    static_cast<uint32_t>(lane & 3) * 2u, static_cast<uint32_t>(row) & 7u, kr[x]);
      }
    };
    const auto put_values = [&](uint32_t s, const uint4 (&vr)[kLoads]) {
      const uint32_t v_row = sbase + L::kOffV + s * L::kTileKV;
#pragma unroll
      for (int x = 0; x < kLoads; ++x) {
        const int ch = 16 * (share * kLoads + x) + v_ch;
        store_codes(v_row + static_cast<uint32_t>(ch) * 128u,
                    static_cast<uint32_t>(blk) * 4u + static_cast<uint32_t>(lane & 1) * 2u, static_cast<uint32_t>(ch) & 7u,
                    vr[x]);
      }
    };
    // opens the first unit from p on that has tiles; false at the end of the range
    const auto open_part = [&]() {
      while (p.todo > 0) {
        const Part x = part_at<D>(a, pairs, p);
        n = x.n;
        const int tiles = max(part_tiles(x, 0), part_tiles(x, 1));
        if (tiles > 0) {
          t = x.t;
          t_end = x.t + tiles;
          len = x.u.len;
          head = x.u.h;
          row_of_table = x.u.b * a.pt.stride;
          large = false;
          open_window();
          pick();
          // on their way while the queries are brought
          if (!kOne && ok) bring_queries(x.u);
          return true;
        }
        place_next(a, p, n);
      }
      return false;
    };
    const auto advance = [&]() {
      if (++t < t_end) {
        if (++in_window == kWindow) open_window();
        pick();
        return true;
      }
      place_next(a, p, n);
      return open_part();
    };
    if constexpr (kOne) {
      // warp 3 brings the codes: they wait in shared memory
      Place q = first_place(found);
      uint32_t cnt = 0;
      while (ok && q.todo > 0) {
        const Part x = part_at<D>(a, pairs, q);
        place_next(a, q, x.n);
        const int tiles = part_tiles(x, 0);
        if (tiles > 0) bring_queries(x.u);
        for (int j = 0; ok && j < tiles; ++j, ++cnt) {
          const uint32_t s = cnt % L::kStages, r = cnt % L::kRaw;
          if (!(ok = wait_bar_warp(cx, cx.bar(kBarRaw + static_cast<int>(r)), (cnt / L::kRaw) & 1u))) break;
          uint4 kr[kLoads], vr[kLoads];
          const uint32_t from = sbase + L::kOffRaw + (r * 2 * kB + static_cast<uint32_t>(blk)) * L::kRawBlock +
                                static_cast<uint32_t>(share * kLoads) * 512u;
#pragma unroll
          for (int y = 0; y < kLoads; ++y) {
            kr[y] = load16(from + static_cast<uint32_t>(y * 32 + lane) * 16u);
            vr[y] = load16(from + kB * L::kRawBlock + static_cast<uint32_t>(y * 32 + v_at) * 16u);
          }
          arrive_warp(cx.bar(kBarRawFree + static_cast<int>(r)), lane);
          if (!(ok = wait_bar_warp(cx, cx.bar(kBarEmpty + static_cast<int>(s)), ((cnt / L::kStages) & 1u) ^ 1u))) break;
          put_keys(s, kr);
          put_values(s, vr);
          tc::fence_proxy_async_smem();
          arrive_warp(cx.bar(kBarFull + static_cast<int>(s)), lane);
        }
      }
    } else {
      uint4 kr[kLoads], vr[kLoads];  // raw codes: 512 bytes per load of the warp
      const auto fetch = [&](const int8_t* codes, int lane_at, uint4 (&r)[kLoads]) {
        const uint4* src = reinterpret_cast<const uint4*>(codes + at) + share * kLoads * 32 + lane_at;
#pragma unroll
        for (int x = 0; x < kLoads; ++x) r[x] = src[x * 32];
      };
      bool more = open_part();
      if (more) {
        fetch(a.c.k, lane, kr);
        fetch(a.c.v, v_at, vr);
      }
      for (uint32_t cnt = 0; ok && more; ++cnt) {
        const uint32_t s = cnt % L::kStages;
        if (!(ok = wait_bar_warp(cx, cx.bar(kBarEmpty + static_cast<int>(s)), ((cnt / L::kStages) & 1u) ^ 1u))) break;
        put_keys(s, kr);
        // the next tile of the unit; the next unit only once this one's values are out
        const bool last = t + 1 >= t_end;
        if (!last) {
          advance();
          if (!ok) break;
          fetch(a.c.k, lane, kr);
        }
        put_values(s, vr);
        if (!last) fetch(a.c.v, v_at, vr);
        tc::fence_proxy_async_smem();
        arrive_warp(cx.bar(kBarFull + static_cast<int>(s)), lane);
        if (last) {
          more = advance();
          if (!ok) break;
          if (more) {
            fetch(a.c.k, lane, kr);
            fetch(a.c.v, v_at, vr);
          }
        }
      }
    }
    if (bad_page) atomicExch(a.dev_err, kDevErrPage);
    __syncwarp();
    regs_dec<kRegCtl>();
  } else {
    // --------------------------------------------------------------- softmax --
    regs_inc<kRegSoftmax>();
    const int i = (warp - 4) >> 2, wq = warp & 3;
    const uint32_t lane_addr = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tO = tmem + lane_addr + C::o(i);
    const float4* scales = reinterpret_cast<const float4*>(smem + T::kOffScale);
    const int rr = i * kRows + wq * 32 + lane;  // this thread's row of a pair
    bool ok = true;
    uint32_t steps = 0, windows = 0, parts = 0;  // key tiles of this query tile; the converters' windows and units
    uint32_t folded = 0;  // folded parts
    // waits for the PV of step x (its P buffer and O are then free)
    const auto wait_pv = [&](uint32_t x) {
      return wait_bar_warp(cx, cx.bar(kBarPVDone + 2 * i + static_cast<int>(x % kS)), (x / kS) & 1u);
    };
    Place p = first_place(found);
    while (p.todo > 0) {
      int n, sees, all_see, fold;
      {
        const Part x = part_at<D>(a, pairs, p);
        if (x.tiles == 0) {
          place_next(a, p, x.n);
          continue;
        }
        fold = kOne && folds(x) ? 1 : 0;
        const int r = x.u.row0 + (fold ? rr & (kRows - 1) : rr);
        const bool real = r < x.u.R;
        sees = real ? row_sees(a, x.u, r) : 0;
        // the smallest limit in the warp decides, for all its lanes, whether a tile is masked
        all_see = __reduce_min_sync(0xffffffffu, real ? sees : 0x7fffffff);
        n = fold ? (part_tiles(x, 0) + 1 - i) >> 1 : part_tiles(x, i);
      }
      float m = -INFINITY, l = 0.0f, f = 0.0f;
      const float* rows = reinterpret_cast<const float*>(smem + T::kOffRow) + (parts % T::kRowUnits) * 2 * kRows;
      for (int j = 0; ok && j < n; ++j) {
        const uint32_t st = steps + static_cast<uint32_t>(j);
        const uint32_t buf = st % kS, tS = tO + (C::s(0, 0) - C::o(0)) + (C::s(0, 1) - C::s(0, 0)) * buf;
        if (!(ok = wait_bar_warp(cx, cx.bar(kBarSFull + 2 * i + static_cast<int>(buf)), (st / kS) & 1u))) break;
        tc::tc_fence_after();
        uint32_t sr[kB][32];
#pragma unroll
        for (int b = 0; b < kB; ++b) tc::tmem_ld32(tS + 32u * b, sr[b]);
        const int jj = fold ? 2 * j + i : j;  // key tile of the part
        const uint32_t win = (windows + static_cast<uint32_t>(jj) / kWindow) % kWindows;
        const float4 sc = scales[win * kWindow + static_cast<uint32_t>(jj) % kWindow];
        if (j == 0) f = rows[fold ? rr & (kRows - 1) : rr] * a.sm_log2;
        tc::tmem_wait_ld();
        const int key0 = (max(p.at - kBegin<D>, 0) + jj) * kKeys;
        float cb[kB];
        int lim[kB];  // tokens of each block that the row sees
        bool masked = tile_hides_keys(key0, all_see);
#pragma unroll
        for (int b = 0; b < kB; ++b) {
          const float k = b == 0 ? sc.x : sc.y;
          cb[b] = f * k;
          lim[b] = !has_tokens(k) ? 0 : sees - key0 - 32 * b;
          masked |= marked(k);
        }
        if (masked) {
#pragma unroll
          for (int b = 0; b < kB; ++b) {
            cb[b] = f * fabsf(b == 0 ? sc.x : sc.y);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (value_token(c) >= lim[b]) sr[b][c] = 0xFF800000u;
          }
        }
        // The weights, whose sum over a block is taken back to that of p. First
        // with the running maximum as it is; that stands unless some row's sum
        // shows a weight above 2^7 (or a row has seen no key yet). The search
        // for the maximum, 34 instructions on a busy pipe, is left to the tiles
        // where it does not stand, and to masked ones: 419 us for a causal chunk
        // of 2000 tokens over 16001, 32 heads on 8, with it in every tile, 402
        // without.
        uint32_t pw[kB][16];
        float sum[kB];
        const bool plain = j > 0 && !masked;
        if (plain) {
#pragma unroll
          for (int b = 0; b < kB; ++b)
            sum[b] = exp_block<false>(sr[b], cb[b], (b == 0 ? sc.z : sc.w) - (m == -INFINITY ? 0.0f : m), 32, pw[b]);
        }
        if (!plain || __any_sync(0xffffffffu, fmaxf(sum[0], sum[1]) > kMost || m == -INFINITY)) {
          float mt = -INFINITY;
#pragma unroll
          for (int b = 0; b < kB; ++b) {
            float m0 = __uint_as_float(sr[b][0]), m1 = __uint_as_float(sr[b][1]);
#pragma unroll
            for (int c = 2; c < 30; c += 4) {
              m0 = max3(m0, __uint_as_float(sr[b][c]), __uint_as_float(sr[b][c + 1]));
              m1 = max3(m1, __uint_as_float(sr[b][c + 2]), __uint_as_float(sr[b][c + 3]));
            }
            m0 = max3(m0, __uint_as_float(sr[b][30]), __uint_as_float(sr[b][31]));
            m0 = fmaxf(m0, m1);
            mt = fmaxf(mt, m0 == -INFINITY ? m0 : fmaf(m0, cb[b], fmaxf(b == 0 ? sc.z : sc.w, kLogScaleMin)));
          }
          if (__any_sync(0xffffffffu, mt > m + kLazy)) {
            const float up = fmaxf(m, mt);
            const float half = up == -INFINITY ? 1.0f : half_step(m, up), alpha = half * half;
            m = up;
            l = rescale(l, half);
            if (j > 0) {
              if (!(ok = wait_pv(st - 1u))) break;  // O is at rest
              tc::tc_fence_after();
              const float2 a2 = make_float2(alpha, alpha);
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                tmem_ld16(tO + 16u * c, o);
                tc::tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                  const float2 y2 = __fmul2_rn(make_float2(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), a2);
                  o[k] = __float_as_uint(y2.x);
                  o[k + 1] = __float_as_uint(y2.y);
                }
                tmem_st16(tO + 16u * c, o);
              }
            }
          }
          const bool odd = marked_odd(sc.x) || marked_odd(sc.y);  // (the same for the warp)
          if (odd) {
#pragma unroll 1
            for (int q = 0; q < 2 * kB; ++q)
              l += part_of_sum(tS + 16u * q, q & 1, q < 2 ? cb[0] : cb[1], m, q < 2 ? lim[0] : lim[1]);
          }
#pragma unroll
          for (int b = 0; b < kB; ++b) {
            sum[b] = exp_block<true>(sr[b], cb[b], (b == 0 ? sc.z : sc.w) - (m == -INFINITY ? 0.0f : m), lim[b], pw[b]);
            if (odd) lim[b] = 0;  // l has the block's part
          }
        }
        // P goes over this row's S, which is in registers
#pragma unroll
        for (int b = 0; b < kB; ++b) {
          tmem_st16(tS + 16u * b, pw[b]);
          // (a block that the row does not reach adds nothing, whatever its scale is)
          l = fmaf(sum[b], lim[b] > 0 ? ex2(-(b == 0 ? sc.z : sc.w)) : 0.0f, l);
        }
        tc::tmem_wait_st();
        tc::tc_fence_before();
        tc::mbar_arrive(cx.bar(kBarPFull + 2 * i + static_cast<int>(buf)));
      }
      if (!ok) break;
      steps += static_cast<uint32_t>(n);

      // the part's rows: to the output, or to the workspace
      const Part x = part_at<D>(a, pairs, p);
      const Unit& u = x.u;
      const int all = max(part_tiles(x, 0), part_tiles(x, 1));
      windows += static_cast<uint32_t>((all + kWindow - 1) / kWindow);
      parts += all > 0 ? 1u : 0u;
      const int r = u.row0 + rr, tok = r / u.G, head = u.h * u.G + r - tok * u.G;
      const bool real = r < u.R;
      if (n > 0) {
        if (!(ok = wait_pv(steps - 1u))) break;
        tc::tc_fence_after();
      }
      const bool whole = x.tiles == x.size;
      const int which = p.todo == found[3] ? 0 : 1;
      if (p.todo == x.n && threadIdx.x == 128 && x.t == 0 && !whole) {
        // the last unit begins here and goes on in other CTAs: up to which one, and whose rows
        const int end = found[4] + x.size - x.tiles - 1, each = found[5], extra = found[6], head_units = extra * (each + 1);
        static_cast<int4*>(a.workspace)[blockIdx.x] =
            make_int4(end < head_units ? end / (each + 1) : extra + (end - head_units) / each, u.b, 2 * u.h + which,
                      u.row0);
      }
      const bool pad = !real && a.zero_rest && x.t == 0 && r < static_cast<int>(a.T) * u.G;
      const bool to_out = whole ? real || pad : pad;
      float* part = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + T::kDesc) +
                    (static_cast<size_t>(blockIdx.x) * 2 + which) * T::kSlot;
      float2 other = make_float2(-INFINITY, 0.0f);  // the second half's maximum and sum
      float s_own = 1.0f, s_other = 0.0f;
      if (fold) {
        // slot 1's half through the rows of the workspace that the part leaves free
        float* half = part + (kRows + (rr & (kRows - 1))) * D;
        float2* half_ml = reinterpret_cast<float2*>(part + 2 * kRows * D + 2 * (kRows + (rr & (kRows - 1))));
        if (i == 1) {
          if (!(ok = wait_bar_warp(cx, cx.bar(kBarFold + 1), (folded & 1u) ^ 1u))) break;
          *half_ml = make_float2(m, l);
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            tc::tmem_ld32(tO + 32u * cc, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 4; ++k) store32(half + 32 * cc + 8 * k, o + 8 * k);
          }
          __threadfence_block();
          tc::mbar_arrive(cx.bar(kBarFold));
        } else {
          if (!(ok = wait_bar_warp(cx, cx.bar(kBarFold), folded & 1u))) break;
          other = __ldcg(half_ml);
          if (other.y != 0.0f) {
            const float up = fmaxf(m, other.x);
            const float own = l == 0.0f ? 0.0f : half_step(m, up), its = half_step(other.x, up);
            s_own = own * own;
            s_other = its * its;
            l = rescale(l, own) + rescale(other.y, its);
            m = up;
          }
        }
        ++folded;
      }
      if (!real) l = s_other = 0.0f;
      const bool none = n == 0 || !real;
      // l = 0: no key was seen
      const float scale = none || l == 0.0f || s_own == 0.0f ? 0.0f : (whole ? 1.0f / l : 1.0f) * s_own;
      if (s_other != 0.0f && whole) s_other /= l;
      const bool wide = ((reinterpret_cast<uintptr_t>(a.out.p) | ((a.out.sb | a.out.ss | a.out.sh) << 1)) & 31) == 0;
      uint16_t* dst = a.out.p + u.b * a.out.sb + tok * a.out.ss + head * a.out.sh;
      if (to_out && a.lse != nullptr)
        a.lse[(static_cast<int64_t>(u.b) * a.H + head) * a.T + tok] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
      if (!whole && real) *reinterpret_cast<float2*>(part + 2 * kRows * D + 2 * rr) = make_float2(m, l);
      const int chunks = __any_sync(0xffffffffu, real || to_out) ? D / 32 : 0;
#pragma unroll 1
      for (int cc = 0; cc < chunks; ++cc) {
        uint32_t o[32];
        if (n > 0) {
          tc::tmem_ld32(tO + 32u * cc, o);
          tc::tmem_wait_ld();
        }
#pragma unroll
        for (int k = 0; k < 32; ++k)
          o[k] = (none || l == 0.0f || s_own == 0.0f) ? 0u : __float_as_uint(__uint_as_float(o[k]) * scale);
        if (s_other != 0.0f) {
          const float4* half = reinterpret_cast<const float4*>(part + (kRows + rr) * D + 32 * cc);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 y = __ldcg(half + k);
            o[4 * k] = __float_as_uint(fmaf(y.x, s_other, __uint_as_float(o[4 * k])));
            o[4 * k + 1] = __float_as_uint(fmaf(y.y, s_other, __uint_as_float(o[4 * k + 1])));
            o[4 * k + 2] = __float_as_uint(fmaf(y.z, s_other, __uint_as_float(o[4 * k + 2])));
            o[4 * k + 3] = __float_as_uint(fmaf(y.w, s_other, __uint_as_float(o[4 * k + 3])));
          }
        }
        if (to_out) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(o[16 * k + 2 * e]),
                                                             __uint_as_float(o[16 * k + 2 * e + 1]));
              w[e] = *reinterpret_cast<const uint32_t*>(&v);
            }
            uint16_t* to = dst + 32 * cc + 16 * k;
            if (wide) {
              store32(to, w);
            } else {
              *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
              *reinterpret_cast<uint4*>(to + 8) = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        } else if (real) {
#pragma unroll
          for (int k = 0; k < 4; ++k) store32(part + rr * D + 32 * cc + 8 * k, o + 8 * k);
        }
      }
      if (fold && i == 0) tc::mbar_arrive(cx.bar(kBarFold + 1));
      tc::tc_fence_before();
      place_next(a, p, x.n);
    }
    __syncwarp();
    regs_dec<kRegCtl>();
  }
  tc::tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && load_flag(cx.abort_at()) != 0) atomicExch(a.dev_err, kDevErrTimeout);
  if (warp == 2) {
    tc::tc_fence_after();
    tc::tmem_dealloc(*reinterpret_cast<volatile uint32_t*>(smem + T::kOffTmem), kTmemCols);
  }
}

}  // namespace

size_t cache_attention_tc_workspace_bytes(int64_t D) {
  return D == 128 ? SmemTail<128, false>::kWorkspace : SmemTail<64, false>::kWorkspace;
}

cudaError_t launch_cache_attention_tc(const CacheAttentionArgs& a, int64_t D, cudaStream_t stream) {
  const int64_t rows = a.T * (a.H / a.c.H);
  const int64_t pairs = div_up(rows, 2 * kRows);
  const int64_t tiles = table_capacity(a.pt.max_pages, a.c.blocks_per_page) / kKeys + 1;
  const int64_t units = pairs * a.B * a.c.H;
  const int sms = sm_count_current() < kMaxSms ? sm_count_current() : kMaxSms;
  // what the tables can name bounds the work: no CTA without any
  const int64_t most = tiles * units / least_tiles(tiles), want = units > most ? units : most;
  const unsigned ctas = static_cast<unsigned>(want < sms ? want : sms);
  const bool one = rows <= kRows;
  const auto kernel = D == 128 ? (one ? cache_attention_tc_kernel<128, true> : cache_attention_tc_kernel<128, false>)
                               : (one ? cache_attention_tc_kernel<64, true> : cache_attention_tc_kernel<64, false>);
  const int bytes = static_cast<int>(D == 128 ? (one ? SmemTail<128, true>::kBytes : SmemTail<128, false>::kBytes)
                                              : (one ? SmemTail<64, true>::kBytes : SmemTail<64, false>::kBytes));
  cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(kernel), bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(bytes);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, kernel, a, static_cast<int>(pairs))) != cudaSuccess || ctas == 1) return e;
  return launch_cache_join(a, D, 2 * kRows, static_cast<int>(rows < 2 * kRows ? rows : 2 * kRows),
                           static_cast<int>(ctas), D == 128 ? SmemTail<128, false>::kDesc : SmemTail<64, false>::kDesc, stream);
}

}  // namespace sage
