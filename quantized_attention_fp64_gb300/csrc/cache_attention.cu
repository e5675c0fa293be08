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
// Few rows per key/value head (decoding, checking drafts): the call reads the
// cache once and is bound by HBM.
//
// Work. A block of 32 keys of one key/value head is the unit; all blocks of all
// sequences and heads form one list (sequence, head, block) that is cut into as
// many equal ranges as there are CTAs, whatever the lengths. A range covers
// whole (sequence, head) items and at most two partial ones, its first and its
// last; partial items leave their running maximum, sum and unnormalised output
// in the workspace, two slots per CTA, and a second kernel joins them in the
// order of the keys.
// Warps. Each of a CTA's 8 warps takes every 8th block of the range through a
// ring of its own: lane 0 copies a block's keys and values (contiguous in the
// cache) into shared memory with bulk copies that complete on an mbarrier,
// kStages blocks ahead, so loads never wait for another warp. The warps' parts
// of an item are joined in shared memory where the item ends.
// Products. The item's rows (query tokens x heads that share the key/value
// head) are the 16 rows of m16n8k16 products. Queries become fp16 times a power
// of two per row (their largest value lies in [1, 4), so a bf16 value keeps its
// 8 bits down to 2^-16 of it, and errs by 2^-25 of it below), key codes are
// exact in fp16, sums are fp32. p is rounded to fp16 (2^-11 relative) and
// multiplied with the exact codes of the values; the block's value scale
// multiplies the fp32 products.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.cuh"
#include "common.cuh"
#include "tc_ptx.cuh"

namespace sage {
namespace {

constexpr int kRowThreads = 128;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCtas = 160;                  // one per SM
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s per wait
constexpr float kLazy = 8.0f;                   // p may reach 2^8 before the running maximum follows

// ---------------------------------------------------------------- the plan --

struct Seq {
  int64_t len, q_len;
};

__device__ __forceinline__ Seq load_seq(const CacheAttentionArgs& a, int64_t b, bool* bad) {
  Seq s;
  s.len = checked_length(a.lengths[b], table_capacity(a.pt.max_pages, a.c.blocks_per_page), bad);
  s.q_len = a.q_lengths != nullptr ? checked_length(a.q_lengths[b], a.T, bad) : a.T;
  return s;
}

// Units of one head of a sequence: its blocks, or one that is empty (a row
// without keys still has an output). A sequence without queries has one, too.
__device__ __forceinline__ int64_t seq_units(const Seq& s) {
  const int64_t n = (s.len + kCacheBlock - 1) / kCacheBlock;
  return (n == 0 || s.q_len == 0) ? 1 : n;
}

// Unit u of total W belongs to CTA owner(u); CTA c has [first(c), first(c + 1)).
struct Split {
  int64_t each, extra;  // W = each * ctas + extra: the first `extra` CTAs have one more
  __device__ Split(int64_t W, int ctas) : each(W / ctas), extra(W % ctas) {}
  __device__ int64_t first(int64_t c) const { return c * each + (c < extra ? c : extra); }
  __device__ int64_t owner(int64_t u) const {
    const int64_t head = extra * (each + 1);
    return u < head ? u / (each + 1) : extra + (u - head) / each;
  }
};

__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Sum of seq_units over sequences [0, n); every thread of the CTA gets it.
// buf: kWarps values of shared memory.
__device__ int64_t units_before(const CacheAttentionArgs& a, int64_t n, int64_t* buf) {
  int64_t x = 0;
  bool bad = false;
  for (int64_t b = threadIdx.x; b < n; b += kThreads) x += seq_units(load_seq(a, b, &bad));
  x = warp_sum(x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) x += buf[w];
  return x;
}

// ------------------------------------------------------------- arithmetic --

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Four int8 codes to two pairs of fp16: with the sign bit flipped a code is
// code + 128 in 0..255, and the half 0x6400 + that is 1024 + 128 + code exactly.
__device__ __forceinline__ void codes_to_half(uint32_t x, uint32_t& lo, uint32_t& hi) {
  x ^= 0x80808080u;
  const uint32_t bias = 0x64806480u;  // 1152, twice
  uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
  const __half2 ra = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&bias));
  const __half2 rb = __hsub2(*reinterpret_cast<const __half2*>(&b), *reinterpret_cast<const __half2*>(&bias));
  lo = *reinterpret_cast<const uint32_t*>(&ra);
  hi = *reinterpret_cast<const uint32_t*>(&rb);
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, int* dev_err) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if ((it & 127u) == 0) {
      const uint64_t now = tc::global_timer_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > kTimeoutNs) {
        atomicExch(dev_err, kDevErrTimeout);
        return false;
      }
    }
  }
}

// 4-byte asynchronous copy whose completion counts as one arrival on `bar`
// (together with the thread's earlier ones).
__device__ __forceinline__ void cp_async4_only(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// ------------------------------------------------------------------ decode --

template <int D, int MT>
struct Dec {
  static constexpr uint32_t kBlockBytes = kCacheBlock * D;     // keys or values of a block
  static constexpr int kStages = D == 128 ? 3 : 5;             // blocks in flight per warp
  static constexpr uint32_t kRing = kWarps * kStages * 2 * kBlockBytes;
  static constexpr uint32_t kOffMerge = kRing;                 // [warp][16 rows][64 channels] fp32
  static constexpr uint32_t kOffMl = kOffMerge + kWarps * 16 * 64 * 4;  // [warp][16 MT rows] (m, l)
  static constexpr uint32_t kOffScale = kOffMl + kWarps * 16 * MT * 8;  // [warp][stage] (key, value) scale
  static constexpr uint32_t kOffValid = kOffScale + kWarps * kStages * 8;
  static constexpr uint32_t kOffBar = kOffValid + kWarps * kStages * 4;
  static constexpr uint32_t kOffPlan = kOffBar + kWarps * kStages * 8;
  static constexpr uint32_t kBytes = kOffPlan + 128;
  static constexpr size_t kSlot = size_t(16) * MT * (D + 2);   // floats of a partial item
  static_assert(kBytes <= 232448u && kOffBar % 8 == 0 && kOffPlan % 8 == 0, "shared memory of one CTA");
};

// A position in the list of units.
struct Cursor {
  int64_t b, blk, units;  // sequence, block of the head, units of the head
  int32_t h;
  Seq s;
};

__device__ __forceinline__ void cursor_settle(const CacheAttentionArgs& a, Cursor& c) {
  while (c.blk >= c.units) {
    c.blk -= c.units;
    if (++c.h == a.c.H) {
      c.h = 0;
      if (++c.b >= a.B) return;  // the end of the list
      bool bad = false;
      c.s = load_seq(a, c.b, &bad);
      c.units = seq_units(c.s);
    }
  }
}

template <int D, int MT>
__global__ void __launch_bounds__(kThreads, 1) cache_decode_kernel(const CacheAttentionArgs a) {
  using L = Dec<D, MT>;
  constexpr int kHalves = D / 64;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sbase = tc::smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  if (threadIdx.x < kWarps * L::kStages) tc::mbar_init(sbase + L::kOffBar + 8 * threadIdx.x, 2);
  tc::fence_mbar_init();
  __syncthreads();
  // the previous kernel of the stream may still run up to here
  tc::griddep_wait();
  tc::griddep_launch_dependents();

  // this CTA's range of units and where it begins
  int64_t* plan = reinterpret_cast<int64_t*>(smem + L::kOffPlan);  // kWarps values, then (b, unit of b's first head)
  const int64_t W = units_before(a, a.B, plan) * a.c.H;
  const Split split(W, static_cast<int>(gridDim.x));
  const int64_t lo = split.first(blockIdx.x), hi = split.first(blockIdx.x + 1);
  if (lo == hi) return;
  for (int64_t base = 0, before = 0; base < a.B; base += kThreads) {
    const int64_t b = base + threadIdx.x;
    bool bad = false;
    const int64_t mine = b < a.B ? seq_units(load_seq(a, b, &bad)) : 0;
    if (bad && blockIdx.x == 0) atomicExch(a.dev_err, kDevErrPage);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) plan[warp] = incl;
    __syncthreads();
    int64_t start = before, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) start += plan[w];
      all += plan[w];
    }
    start += incl - mine;  // units of one head before sequence b
    if (b < a.B && start * a.c.H <= lo && lo < (start + mine) * a.c.H) {
      plan[kWarps] = b;
      plan[kWarps + 1] = lo - start * a.c.H;
    }
    before += all;
    if (before * a.c.H > lo && blockIdx.x != 0) break;  // CTA 0 looks at every length once
  }
  __syncthreads();
  Cursor seg;
  {
    bool bad = false;
    seg.b = plan[kWarps];
    seg.s = load_seq(a, seg.b, &bad);
    seg.units = seq_units(seg.s);
    seg.h = static_cast<int32_t>(plan[kWarps + 1] / seg.units);
    seg.blk = plan[kWarps + 1] % seg.units;
  }
  const int64_t n_cta = hi - lo;
  const int64_t n_mine = n_cta > warp ? (n_cta - warp + kWarps - 1) / kWarps : 0;  // this warp's blocks

  // the warp's next 32 blocks, one per lane: lane i of the window has blocks i, i + 32, ...
  Cursor ahead = seg;
  ahead.blk += warp + static_cast<int64_t>(lane) * kWarps;
  if (lane < n_mine) cursor_settle(a, ahead);
  int64_t window = -1;  // its block number in the cache, -1: no tokens
  const auto fill_window = [&](int64_t k0) {
    window = -1;
    if (k0 + lane < n_mine) {
      if (k0 > 0) {
        ahead.blk += 32 * kWarps;
        cursor_settle(a, ahead);
      }
      if (ahead.s.q_len > 0 && ahead.blk * kCacheBlock < ahead.s.len) {
        const int64_t page = a.pt.table[ahead.b * a.pt.stride + ahead.blk / a.c.blocks_per_page];
        if (page_ok(page, a.c.num_pages))
          window = block_slot(page, ahead.h, a.c.H, a.c.blocks_per_page,
                              static_cast<int32_t>(ahead.blk % a.c.blocks_per_page));
        else
          atomicExch(a.dev_err, kDevErrPage);
      }
    }
  };
  const uint32_t ring = sbase + static_cast<uint32_t>(warp) * L::kStages * 2 * L::kBlockBytes;
  const uint32_t bars = sbase + L::kOffBar + static_cast<uint32_t>(warp) * L::kStages * 8;
  const uint32_t scales = sbase + L::kOffScale + static_cast<uint32_t>(warp) * L::kStages * 8;
  volatile int* valid = reinterpret_cast<volatile int*>(smem + L::kOffValid) + warp * L::kStages;
  int64_t issued = 0;
  const auto issue = [&]() {  // whole warp
    if (issued >= n_mine) return;
    if ((issued & 31) == 0) fill_window(issued);
    const int64_t slot = __shfl_sync(0xffffffffu, window, static_cast<int>(issued & 31));
    if (lane == 0) {
      const uint32_t s = static_cast<uint32_t>(issued % L::kStages);
      const uint32_t bar = bars + 8 * s, dst = ring + s * 2 * L::kBlockBytes;
      valid[s] = slot >= 0;
      if (slot >= 0) {
        tc::mbar_arrive_expect_tx(bar, 2 * L::kBlockBytes);
        tc::bulk_load(dst, a.c.k + slot * L::kBlockBytes, L::kBlockBytes, bar);
        tc::bulk_load(dst + L::kBlockBytes, a.c.v + slot * L::kBlockBytes, L::kBlockBytes, bar);
        cp_async4_only(scales + 8 * s, a.c.ks + slot);
        cp_async4_only(scales + 8 * s + 4, a.c.vs + slot);
        cp_async_arrive(bar);
      } else {
        tc::mbar_arrive(bar);
        tc::mbar_arrive(bar);
      }
    }
    ++issued;
  };
#pragma unroll 1
  for (int s = 0; s < L::kStages; ++s) issue();

  int64_t taken = 0;  // blocks of this warp done
  bool alive = true;
  const int G = a.H / a.c.H;
#pragma unroll 1
  for (int64_t at = 0; at < n_cta;) {
    // the segment: units [at, at + n) of the CTA, blocks [seg.blk, seg.blk + n) of one item
    const int64_t n = min(seg.units - seg.blk, n_cta - at);
    const int64_t R = seg.s.q_len * G;
    const int64_t min_sees = a.causal ? seg.s.len - seg.s.q_len + 1 : seg.s.len;  // of the item's first token
    // queries: A fragments of the key products, rows g and g + 8 of each 16
    uint32_t qf[MT][kHalves][4][4];
    float f[MT][2];
    int64_t sees[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = mt * 16 + e * 8 + g;
        uint32_t w[kHalves][8];
        sees[mt][e] = 0;
        if (r < R) {
          const int64_t tok = r / G;
          sees[mt][e] = a.causal ? seg.s.len - seg.s.q_len + 1 + tok : seg.s.len;
          const uint16_t* p = a.q.p + seg.b * a.q.sb + tok * a.q.ss + (static_cast<int64_t>(seg.h) * G + r % G) * a.q.sh + 16 * t;
#pragma unroll
          for (int i = 0; i < kHalves; ++i) {
            *reinterpret_cast<uint4*>(w[i]) = *reinterpret_cast<const uint4*>(p + 64 * i);
            *reinterpret_cast<uint4*>(w[i] + 4) = *reinterpret_cast<const uint4*>(p + 64 * i + 8);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kHalves; ++i)
#pragma unroll
            for (int x = 0; x < 8; ++x) w[i][x] = 0u;
        }
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < kHalves; ++i)
#pragma unroll
          for (int x = 0; x < 8; ++x) amax = max(amax, max(w[i][x] & 0x7FFFu, (w[i][x] >> 16) & 0x7FFFu));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // the power of two below the largest value; infinities and NaN stay what they are
        uint32_t ex = amax >> 7;
        ex = ex == 255u ? 127u : min(max(ex, 1u), 253u);
        const float down = __uint_as_float((254u - ex) << 23);
        f[mt][e] = __uint_as_float(ex << 23) * a.sm_log2;
#pragma unroll
        for (int i = 0; i < kHalves; ++i)
#pragma unroll
          for (int x = 0; x < 8; ++x)
            qf[mt][i][x >> 1][(x & 1) * 2 + e] =
                pack_half2(__uint_as_float(w[i][x] << 16) * down, __uint_as_float(w[i][x] & 0xFFFF0000u) * down);
      }
    }
    float o[MT][D / 8][4];
    float m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int x = 0; x < D / 8; ++x) o[mt][x][0] = o[mt][x][1] = o[mt][x][2] = o[mt][x][3] = 0.0f;
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.0f;
    }
    // this warp's blocks of the segment: CTA units that are warp mod 8
    const int64_t first = at + (warp - at % kWarps + kWarps) % kWarps;
#pragma unroll 1
    for (int64_t u = first; u < at + n && alive; u += kWarps) {
      const uint32_t s = static_cast<uint32_t>(taken % L::kStages);
      const uint32_t parity = static_cast<uint32_t>(taken / L::kStages) & 1u;
      alive = __all_sync(0xffffffffu, wait_bounded(bars + 8 * s, parity, a.dev_err));
      if (!alive) break;
      if (valid[s] != 0) {
        const uint8_t* kb = smem + (ring - sbase) + s * 2 * L::kBlockBytes;
        const uint8_t* vb = kb + L::kBlockBytes;
        const float2 sc = *reinterpret_cast<const float2*>(smem + (scales - sbase) + 8 * s);
        const int64_t key0 = (seg.blk + (u - at)) * kCacheBlock;
        const bool masked = key0 + kCacheBlock > min_sees;
        float z[MT][4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) z[mt][j][0] = z[mt][j][1] = z[mt][j][2] = z[mt][j][3] = 0.0f;
#pragma unroll
          for (int i = 0; i < kHalves; ++i) {
            const uint4 c = *reinterpret_cast<const uint4*>(kb + i * 2048 + j * 512 + lane * 16);
            const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t b0, b1;
              codes_to_half(cw[x], b0, b1);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) mma16816(z[mt][j], qf[mt][i][x], b0, b1);
            }
          }
        }
        uint32_t pf[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              float y = z[mt][j][x] * (f[mt][x >> 1] * sc.x);
              if (masked && key0 + 8 * j + 2 * t + (x & 1) >= sees[mt][x >> 1]) y = -INFINITY;
              z[mt][j][x] = y;
              mx[x >> 1] = fmaxf(mx[x >> 1], y);
            }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
          }
          if (__any_sync(0xffffffffu, mx[0] > m[mt][0] + kLazy || mx[1] > m[mt][1] + kLazy)) {
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float up = fmaxf(m[mt][e], mx[e]);
              alpha[e] = up == -INFINITY ? 1.0f : ex2(m[mt][e] - up);
              m[mt][e] = up;
              l[mt][e] *= alpha[e];
            }
#pragma unroll
            for (int x = 0; x < D / 8; ++x) {
              o[mt][x][0] *= alpha[0];
              o[mt][x][1] *= alpha[0];
              o[mt][x][2] *= alpha[1];
              o[mt][x][3] *= alpha[1];
            }
          }
          const float ref[2] = {m[mt][0] == -INFINITY ? 0.0f : m[mt][0], m[mt][1] == -INFINITY ? 0.0f : m[mt][1]};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int x = 0; x < 4; ++x) z[mt][j][x] = ex2(z[mt][j][x] - ref[x >> 1]);
            l[mt][0] += z[mt][j][0] + z[mt][j][1];
            l[mt][1] += z[mt][j][2] + z[mt][j][3];
            pf[mt][j >> 1][(j & 1) * 2] = pack_half2(z[mt][j][0], z[mt][j][1]);
            pf[mt][j >> 1][(j & 1) * 2 + 1] = pack_half2(z[mt][j][2], z[mt][j][3]);
          }
        }
        // a block that a row does not reach adds nothing to it, whatever its scale is
        float vs[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e) vs[mt][e] = key0 < sees[mt][e] ? sc.y : 0.0f;
#pragma unroll
        for (int x = 0; x < D / 8; ++x) {
          const uint2 c = *reinterpret_cast<const uint2*>(vb + x * 256 + lane * 8);
          uint32_t b[4];
          codes_to_half(c.x, b[0], b[1]);
          codes_to_half(c.y, b[2], b[3]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma16816(d, pf[mt][0], b[0], b[1]);
            mma16816(d, pf[mt][1], b[2], b[3]);
            o[mt][x][0] = fmaf(d[0], vs[mt][0], o[mt][x][0]);
            o[mt][x][1] = fmaf(d[1], vs[mt][0], o[mt][x][1]);
            o[mt][x][2] = fmaf(d[2], vs[mt][1], o[mt][x][2]);
            o[mt][x][3] = fmaf(d[3], vs[mt][1], o[mt][x][3]);
          }
        }
      }
      ++taken;
      __syncwarp();  // every lane is done with the stage
      issue();
    }

    // join the warps' parts of the item
    float2* ml = reinterpret_cast<float2*>(smem + L::kOffMl);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[mt][e] += __shfl_xor_sync(0xffffffffu, l[mt][e], 1);
        l[mt][e] += __shfl_xor_sync(0xffffffffu, l[mt][e], 2);
        if (t == 0) ml[warp * 16 * MT + mt * 16 + e * 8 + g] = make_float2(m[mt][e], l[mt][e]);
      }
    const bool whole = n == seg.units;
    const int which = at == 0 ? 0 : 1;  // a partial item is the range's first or its last
    float* part = static_cast<float*>(a.workspace) + (static_cast<size_t>(blockIdx.x) * 2 + which) * L::kSlot;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt * 16 >= R) break;
#pragma unroll
      for (int half = 0; half < kHalves; ++half) {
        // rows of 64 channels as 32 pairs, pair u of row r at u ^ 4 (r mod 4): no bank conflicts
        float2* buf = reinterpret_cast<float2*>(smem + L::kOffMerge) + warp * 16 * 32;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int u = (4 * x + t) ^ ((g & 3) * 4);
          buf[g * 32 + u] = make_float2(o[mt][half * 8 + x][0], o[mt][half * 8 + x][1]);
          buf[(g + 8) * 32 + u] = make_float2(o[mt][half * 8 + x][2], o[mt][half * 8 + x][3]);
        }
        __syncthreads();
        const int row = threadIdx.x >> 4, c4 = threadIdx.x & 15;
        const int r = mt * 16 + row;
        if (r < R) {
          float top = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * 16 * MT + r].x);
          const float ref = top == -INFINITY ? 0.0f : top;
          float sum = 0.0f;
          float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 x = ml[w * 16 * MT + r];
            const float wt = ex2(x.x - ref);
            const float4 y = *reinterpret_cast<const float4*>(reinterpret_cast<const float2*>(smem + L::kOffMerge) +
                                                              (w * 16 + row) * 32 + ((2 * c4) ^ ((row & 3) * 4)));
            sum = fmaf(x.y, wt, sum);
            acc.x = fmaf(y.x, wt, acc.x);
            acc.y = fmaf(y.y, wt, acc.y);
            acc.z = fmaf(y.z, wt, acc.z);
            acc.w = fmaf(y.w, wt, acc.w);
          }
          if (whole) {
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            const int64_t tok = r / G, head = static_cast<int64_t>(seg.h) * G + r % G;
            uint16_t* p = a.out.p + seg.b * a.out.sb + tok * a.out.ss + head * a.out.sh + half * 64 + 4 * c4;
            const __nv_bfloat162 lo2 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
            const __nv_bfloat162 hi2 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
            *reinterpret_cast<uint2*>(p) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&lo2), *reinterpret_cast<const uint32_t*>(&hi2));
            if (a.lse != nullptr && half == 0 && c4 == 0)
              a.lse[(seg.b * a.H + head) * a.T + tok] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
          } else {
            *reinterpret_cast<float4*>(part + static_cast<size_t>(r) * D + half * 64 + 4 * c4) = acc;
            if (half == 0 && c4 == 0)
              *reinterpret_cast<float2*>(part + static_cast<size_t>(16) * MT * D + 2 * r) = make_float2(top, sum);
          }
        }
        __syncthreads();
      }
    }
    if (R == 0) __syncthreads();
    at += n;
    seg.blk += n;
    if (at < n_cta) cursor_settle(a, seg);
  }
  if (!alive) {
    // copies in flight land before the CTA ends
    for (; taken < issued; ++taken)
      wait_bounded(bars + 8 * static_cast<uint32_t>(taken % L::kStages),
                   static_cast<uint32_t>(taken / L::kStages) & 1u, a.dev_err);
  }
}

// Joins the partial items: one CTA per (sequence, key/value head); a warp per row.
template <int D, int MT>
__global__ void __launch_bounds__(kThreads) cache_join_kernel(const CacheAttentionArgs a, int ctas) {
  constexpr int kV = D / 32;  // channels per lane
  using L = Dec<D, MT>;
  __shared__ int64_t buf[kWarps];
  tc::griddep_wait();
  const int64_t b = blockIdx.y;
  const int32_t h = static_cast<int32_t>(blockIdx.x);
  const int64_t W = units_before(a, a.B, buf) * a.c.H;
  const int64_t before = units_before(a, b, buf) * a.c.H;
  bool bad = false;
  const Seq s = load_seq(a, b, &bad);
  const int64_t n = seq_units(s), u0 = before + h * n;
  const Split split(W, ctas);
  const int64_t c0 = split.owner(u0), c1 = split.owner(u0 + n - 1);
  if (c0 == c1) return;  // one CTA had the whole item
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.H / a.c.H;
  const float* ws = static_cast<const float*>(a.workspace);
  // CTA c0's part is its first one if its range begins with the item, else its last; the others' their first
  const size_t slot0 = (static_cast<size_t>(c0) * 2 + (split.first(c0) < u0 ? 1 : 0)) * L::kSlot;
  for (int64_t r = warp; r < s.q_len * G; r += kWarps) {
    float top = -INFINITY;
    for (int64_t c = c0 + lane; c <= c1; c += 32) {
      const float* p = ws + (c == c0 ? slot0 : static_cast<size_t>(c) * 2 * L::kSlot);
      top = fmaxf(top, p[static_cast<size_t>(16) * MT * D + 2 * r]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f, acc[kV];
#pragma unroll
    for (int x = 0; x < kV; ++x) acc[x] = 0.0f;
#pragma unroll 4
    for (int64_t c = c0; c <= c1; ++c) {
      const float* p = ws + (c == c0 ? slot0 : static_cast<size_t>(c) * 2 * L::kSlot);
      const float2 x = *reinterpret_cast<const float2*>(p + static_cast<size_t>(16) * MT * D + 2 * r);
      const float wt = ex2(x.x - ref);
      sum = fmaf(x.y, wt, sum);
#pragma unroll
      for (int i = 0; i < kV; ++i) acc[i] = fmaf(p[r * D + kV * lane + i], wt, acc[i]);
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int64_t tok = r / G, head = static_cast<int64_t>(h) * G + r % G;
    uint16_t* p = a.out.p + b * a.out.sb + tok * a.out.ss + head * a.out.sh + kV * lane;
#pragma unroll
    for (int i = 0; i < kV; i += 2) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(acc[i] * inv, acc[i + 1] * inv);
      *reinterpret_cast<uint32_t*>(p + i) = *reinterpret_cast<const uint32_t*>(&v);
    }
    if (a.lse != nullptr && lane == 0)
      a.lse[(b * a.H + head) * a.T + tok] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
  }
}

// -------------------------------------------------------------- many rows --
// One CTA per row: it goes over the blocks of 32 keys with a running maximum
// and sum, everything in fp32.
template <int D>
__global__ void __launch_bounds__(kRowThreads) cache_attention_kernel(CacheAttentionArgs a) {
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

int decode_ctas(const CacheAttentionArgs& a) {
  // a CTA for every 8 blocks that the tables can name (one per warp), at most one per SM
  const int64_t blocks = a.B * a.c.H * (table_capacity(a.pt.max_pages, a.c.blocks_per_page) / kCacheBlock);
  const int sms = sm_count_current();
  const int64_t most = sms < kMaxCtas ? sms : kMaxCtas, want = div_up(blocks, kWarps);
  return static_cast<int>(want < 1 ? 1 : (want < most ? want : most));
}

template <int D, int MT>
cudaError_t launch_decode(const CacheAttentionArgs& a, cudaStream_t stream) {
  using L = Dec<D, MT>;
  const int ctas = decode_ctas(a);
  cudaError_t e = set_smem_limit_once(reinterpret_cast<const void*>(cache_decode_kernel<D, MT>), L::kBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::kBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, cache_decode_kernel<D, MT>, a)) != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(a.c.H), static_cast<unsigned>(a.B));
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, cache_join_kernel<D, MT>, a, ctas);
}

}  // namespace

size_t cache_attention_workspace_bytes(int64_t, int64_t T, int64_t H, int64_t Hkv, int64_t D) {
  const int64_t rows = T * (H / Hkv);
  if (rows <= 16) return size_t(kMaxCtas) * 2 * (D == 128 ? Dec<128, 1>::kSlot : Dec<64, 1>::kSlot) * 4;
  if (rows <= 32) return size_t(kMaxCtas) * 2 * (D == 128 ? Dec<128, 2>::kSlot : Dec<64, 2>::kSlot) * 4;
  return 0;
}

cudaError_t launch_cache_attention(const CacheAttentionArgs& a, int64_t D, cudaStream_t stream) {
  const int64_t rows = a.T * (a.H / a.c.H);
  if (rows <= 16) return D == 128 ? launch_decode<128, 1>(a, stream) : launch_decode<64, 1>(a, stream);
  if (rows <= 32) return D == 128 ? launch_decode<128, 2>(a, stream) : launch_decode<64, 2>(a, stream);
  const dim3 grid(static_cast<unsigned>(a.T), static_cast<unsigned>(a.H), static_cast<unsigned>(a.B));
  if (D == 128)
    cache_attention_kernel<128><<<grid, kRowThreads, 0, stream>>>(a);
  else
    cache_attention_kernel<64><<<grid, kRowThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace sage
