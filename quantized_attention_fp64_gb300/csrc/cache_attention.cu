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
// Warps. Each of a CTA's 4 warps takes every 4th block of the range through a
// ring of its own: a lane copies a block's keys and values (contiguous in the
// cache) into shared memory with bulk copies that complete on an mbarrier,
// kStages blocks ahead, so loads never wait for another warp. The warps' parts
// of an item are joined in shared memory where the item ends; two or three CTAs
// share an SM, so that one streams while another joins.
// Products. The item's rows (query tokens x heads that share the key/value
// head) are the 16 rows of m16n8k16 products. Queries become fp16 times a power
// of two per row (their largest value lies in [1, 4), so a bf16 value keeps its
// 8 bits down to 2^-16 of it, and errs by 2^-25 of it below), key codes are
// exact in fp16, sums are fp32. The value scale of a block goes into its
// weights: with m a row's running maximum of z + log2 s_v (z: the logits times
// log2 e), the weights 2^(z + log2 s_v - m) are rounded to fp16 (by 2^-11 of
// themselves, or of what is below 2^-14 of the largest by 2^-25 of that) and
// multiplied with the exact codes; the sum of 2^(z - m) is taken in fp32, block
// by block, from the weights before they are rounded, over s_v (or apart from
// them, see cache.cuh). So a key of little weight and large values keeps its
// share, and one of small values its part of the sum.
// Measured (GB300, head dimension 128): one token each of 64 sequences of 900 to
// 8192, 32 heads on 8: 105 us, 5.7 TB/s of 6.8; two of about 131000 tokens, 28
// heads on 4: 51 us, 4.9 TB/s (the start, the uneven ends of the CTAs and the
// join take 10 us there); one of 1000: 6.6 us, a chain of dependent loads. 17 to
// 32 rows of a head over 14 x 20000 tokens: 137 us, 4.2 TB/s; no pipe is full
// there (issue slots 41%, tensor 47%, HBM 53%): with two warps to a scheduler the
// latencies of a warp's own instructions add up.
// Ranges cut two to four times finer than what the SMs hold are slower.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "cache.cuh"
#include "common.cuh"
#include "tc_ptx.cuh"

namespace sage {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s per wait
constexpr float kLazy = 8.0f;                   // a weight may reach 2^8 before the running maximum follows

// ---------------------------------------------------------------- the plan --

struct Seq {
  int len, q_len;
};

__device__ __forceinline__ Seq load_seq(const CacheAttentionArgs& a, int b, bool* bad) {
  Seq s;
  s.len = static_cast<int>(checked_length(a.lengths[b], table_capacity(a.pt.max_pages, a.c.blocks_per_page), bad));
  s.q_len = static_cast<int>(a.q_lengths != nullptr ? checked_length(a.q_lengths[b], a.T, bad) : a.T);
  return s;
}

// Units of one head of a sequence: its blocks, or one that is empty (a row
// without keys still has an output). A sequence without queries has one, too.
// All units of a call together are fewer than 2^31 (checked on the host).
__device__ __forceinline__ int seq_units(const Seq& s) {
  const int n = (s.len + kCacheBlock - 1) / kCacheBlock;
  return (n == 0 || s.q_len == 0) ? 1 : n;
}

// CTA c of `ctas` has the units [first(c), first(c + 1)) of W, unit u belongs to owner(u).
struct Split {
  int each, extra;  // W = each * ctas + extra: the first `extra` CTAs have one more
  __device__ Split(int W, int ctas) : each(W / ctas), extra(W % ctas) {}
  __device__ int first(int c) const { return c * each + (c < extra ? c : extra); }
  __device__ int owner(int u) const {
    const int head = extra * (each + 1);
    return u < head ? u / (each + 1) : extra + (u - head) / each;
  }
};

// ------------------------------------------------------------- arithmetic --

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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

// d = a b + c, m16n8k16, fp16 with fp32 sums
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                         float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  mma16816(d, a, b0, b1, d[0], d[1], d[2], d[3]);
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

// ------------------------------------------------------------------ decode --

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxSms = 160;
constexpr int kClusterBlocks = 8;  // blocks per warp up to which a cluster takes an item

template <int D, int MT>
struct Dec {
  // CTAs of an SM: what the accumulators' registers allow (168 or 255 a
  // thread); stages: blocks in flight per warp, 192 KB of an SM's in all
  static constexpr int kCtasPerSm = MT == 1 ? 3 : 2;
  static constexpr int kStages = (MT == 1 ? 2 : 3) * (128 / D);
  static constexpr uint32_t kBlockBytes = kCacheBlock * D;     // keys or values of a block
  static constexpr uint32_t kRing = kWarps * kStages * 2 * kBlockBytes;
  static constexpr uint32_t kOffMerge = kRing;                 // [warp][16 rows][32 channels] fp32, or the queries
  static_assert(16 * MT * D * 2 <= kWarps * 16 * 32 * 4, "the queries fit");
  static constexpr uint32_t kOffMl = kOffMerge + kWarps * 16 * 32 * 4;  // [warp][16 MT rows] (m, l)
  static constexpr uint32_t kOffScale = kOffMl + kWarps * 16 * MT * 8;  // [warp][stage] (key, value) scale
  static constexpr uint32_t kOffBar = kOffScale + kWarps * kStages * 8;
  static constexpr uint32_t kOffPlan = kOffBar + kWarps * kStages * 8;  // kWarps sums, then where the range begins
  static constexpr uint32_t kBytes = kOffPlan + (kWarps + 6) * 4;
  static_assert(kCtasPerSm * (kBytes + 1024) <= 233472u && kOffBar % 8 == 0, "shared memory of one SM");
  // workspace: a descriptor of each CTA's last item, then two slots per CTA
  static constexpr size_t kDesc = size_t(kMaxSms) * kCtasPerSm * sizeof(int4);
  static constexpr size_t kSlot = size_t(16) * MT * (D + 2);   // floats of a partial item
  static constexpr size_t kWorkspace = kDesc + size_t(kMaxSms) * kCtasPerSm * 2 * kSlot * 4;
};

// A position in the list of units.
struct Cursor {
  int b, h, blk, units;  // sequence, head, block of the head, units of the head
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

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// The rows rank, rank + parts, ... of an item from the parts that the cluster's
// CTAs hold at the start of their shared memory (as in a workspace slot).
template <int D, int MT>
__device__ __forceinline__ void join_cluster(const CacheAttentionArgs& a, uint32_t sbase, int rank, int parts, int b,
                                             int h, int R) {
  constexpr int kRows = kThreads / D;  // rows at a time, a thread per channel
  const int G = a.H / a.c.H, ch = static_cast<int>(threadIdx.x) % D;
  for (int r = rank + parts * (static_cast<int>(threadIdx.x) / D); r < R; r += parts * kRows) {
    const uint32_t at = sbase + (r * D + ch) * 4, at_ml = sbase + (16 * MT * D + 2 * r) * 4;
    float m[8], l[8], o[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      m[c] = -INFINITY;
      l[c] = o[c] = 0.0f;
      if (c < parts) {
        m[c] = ld_cluster_f32(tc::mapa_shared(at_ml, c));
        l[c] = ld_cluster_f32(tc::mapa_shared(at_ml + 4, c));
        o[c] = ld_cluster_f32(tc::mapa_shared(at, c));
      }
    }
    float top = m[0];
#pragma unroll
    for (int c = 1; c < 8; ++c) top = fmaxf(top, m[c]);
    const float ref = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f, acc = 0.0f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float half = half_step(m[c], ref);
      sum += rescale(l[c], half);
      acc = fmaf(o[c], half * half, acc);
    }
    const int tok = r / G, head = h * G + r - tok * G;
    const __nv_bfloat16 v = __float2bfloat16_rn(sum == 0.0f ? 0.0f : acc / sum);
    a.out.p[b * a.out.sb + tok * a.out.ss + head * a.out.sh + ch] = *reinterpret_cast<const uint16_t*>(&v);
    if (a.lse != nullptr && ch == 0)
      a.lse[(static_cast<int64_t>(b) * a.H + head) * a.T + tok] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
  }
}

// The queries of rows g and g + 8 of row tile mt of an item, this lane's channels; 0 past the last row.
template <int D>
__device__ __forceinline__ void load_queries(const CacheAttentionArgs& a, const Cursor& c, int mt, int g, int t,
                                             uint4 (&raw)[2][D / 32]) {
  const int G = a.H / a.c.H;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = mt * 16 + e * 8 + g;
#pragma unroll
    for (int x = 0; x < D / 32; ++x) raw[e][x] = make_uint4(0u, 0u, 0u, 0u);
    if (r < c.s.q_len * G) {
      const int tok = r / G;
      const uint4* p = reinterpret_cast<const uint4*>(a.q.p + c.b * a.q.sb + tok * a.q.ss + (c.h * G + r - tok * G) * a.q.sh + 16 * t);
#pragma unroll
      for (int x = 0; x < D / 32; ++x) raw[e][x] = p[(x >> 1) * 8 + (x & 1)];
    }
  }
}

// kCluster: small calls. A cluster of CTAs has one item each, cut into equal
// parts; the parts are joined through distributed shared memory and nothing
// goes through the workspace.
template <int D, int MT, bool kCluster>
__global__ void __launch_bounds__(kThreads, Dec<D, MT>::kCtasPerSm) cache_decode_kernel(const CacheAttentionArgs a) {
  using L = Dec<D, MT>;
  constexpr int kHalves = D / 64;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sbase = tc::smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  if (threadIdx.x < kWarps * L::kStages) tc::mbar_init(sbase + L::kOffBar + 8 * threadIdx.x, 1);
  tc::fence_mbar_init();
  // the previous kernel of the stream may still run up to here
  tc::griddep_wait();
  tc::griddep_launch_dependents();

  Cursor seg;
  int lo = 0, hi, rank = 0, parts = 1;
  int4* desc = static_cast<int4*>(a.workspace);
  Split split(0, 1);
  bool bad = false;
  if constexpr (kCluster) {
    rank = static_cast<int>(tc::cluster_ctarank());
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(parts));
    const int item = static_cast<int>(blockIdx.x) / parts;
    seg.b = item / a.c.H;
    seg.h = item - seg.b * a.c.H;
    seg.s = load_seq(a, seg.b, &bad);
    if (bad && rank == 0 && threadIdx.x == 0) atomicExch(a.dev_err, kDevErrPage);
    seg.units = seq_units(seg.s);
    split = Split(seg.units, parts);
    lo = split.first(rank);
    hi = split.first(rank + 1);
    seg.blk = lo;
    __syncthreads();  // the barriers are set up
  } else {
    // this CTA's range of units and where it begins: each thread sums a run of
    // sequences, a scan over the threads finds whose run the range begins in
    int* plan = reinterpret_cast<int*>(smem + L::kOffPlan);
    const int run = (static_cast<int>(a.B) + kThreads - 1) / kThreads;
    const int b_lo = min(run * static_cast<int>(threadIdx.x), static_cast<int>(a.B));
    const int b_hi = min(b_lo + run, static_cast<int>(a.B));
    int mine = 0;
    for (int b = b_lo; b < b_hi; ++b) mine += seq_units(load_seq(a, b, &bad));
    if (bad && blockIdx.x == 0) atomicExch(a.dev_err, kDevErrPage);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) plan[warp] = incl;
    __syncthreads();
    int before = incl - mine, W = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += plan[w];
      W += plan[w];
    }
    W *= a.c.H;
    split = Split(W, static_cast<int>(gridDim.x));
    lo = split.first(static_cast<int>(blockIdx.x));
    hi = split.first(static_cast<int>(blockIdx.x) + 1);
    before *= a.c.H;
    if (lo < hi && before <= lo && lo < before + mine * a.c.H) {
      int b = b_lo;
      Seq x;
      int units;
      for (;; ++b) {
        x = load_seq(a, b, &bad);
        units = seq_units(x);
        if (lo < before + units * a.c.H) break;
        before += units * a.c.H;
      }
      const int h = (lo - before) / units;
      plan[kWarps] = b;
      plan[kWarps + 1] = h;
      plan[kWarps + 2] = lo - before - h * units;
      plan[kWarps + 3] = units;
      plan[kWarps + 4] = x.len;
      plan[kWarps + 5] = x.q_len;
    }
    __syncthreads();
    if (lo == hi) {
      if (threadIdx.x == 0) desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
      return;
    }
    seg.b = plan[kWarps];
    seg.h = plan[kWarps + 1];
    seg.blk = plan[kWarps + 2];
    seg.units = plan[kWarps + 3];
    seg.s.len = plan[kWarps + 4];
    seg.s.q_len = plan[kWarps + 5];
  }
  const int n_cta = hi - lo;
  const int n_mine = n_cta > warp ? (n_cta - warp + kWarps - 1) / kWarps : 0;  // this warp's blocks

  // the warp's next 32 blocks, one per lane: lane i of the window has blocks i, i + 32, ...
  Cursor ahead = seg;
  ahead.blk += warp + lane * kWarps;
  if (lane < n_mine) cursor_settle(a, ahead);
  int64_t at_codes = -1;               // first byte in the codes, -1: no tokens
  float2 at_scales = make_float2(-1.0f, 0.0f);  // key scale (-1: no tokens), value scale
  const auto fill_window = [&](int k0) {
    at_codes = -1;
    at_scales.x = -1.0f;
    if (k0 + lane < n_mine) {
      if (k0 > 0) {
        ahead.blk += 32 * kWarps;
        cursor_settle(a, ahead);
      }
      if (ahead.s.q_len > 0 && ahead.blk * kCacheBlock < ahead.s.len) {
        const int pg = ahead.blk / a.c.blocks_per_page;
        const int page = a.pt.table[ahead.b * a.pt.stride + pg];
        if (page_ok(page, a.c.num_pages)) {
          const int64_t slot = block_slot(page, ahead.h, a.c.H, a.c.blocks_per_page, ahead.blk - pg * a.c.blocks_per_page);
          at_codes = slot * L::kBlockBytes;
          at_scales = make_float2(a.c.ks[slot], a.c.vs[slot]);
        } else {
          atomicExch(a.dev_err, kDevErrPage);
        }
      }
    }
  };
  const uint32_t ring = sbase + static_cast<uint32_t>(warp) * L::kStages * 2 * L::kBlockBytes;
  const uint32_t bars = sbase + L::kOffBar + static_cast<uint32_t>(warp) * L::kStages * 8;
  float2* scales = reinterpret_cast<float2*>(smem + L::kOffScale) + warp * L::kStages;
  int issued = 0;
  uint32_t into = 0;  // stage of the next issue
  const auto issue = [&]() {  // whole warp; the lane that has the block sends for it
    if (issued >= n_mine) return;
    if ((issued & 31) == 0) fill_window(issued);
    if (lane == (issued & 31)) {
      const uint32_t bar = bars + 8 * into, dst = ring + into * 2 * L::kBlockBytes;
      if (at_codes >= 0) {
        // (the copies do not wait for the scales; the phase ends after the arrival)
        tc::bulk_load(dst, a.c.k + at_codes, L::kBlockBytes, bar);
        tc::bulk_load(dst + L::kBlockBytes, a.c.v + at_codes, L::kBlockBytes, bar);
      }
      scales[into] = make_float2(at_scales.x, log_scale(at_scales.y));
      if (at_codes >= 0) tc::mbar_arrive_expect_tx(bar, 2 * L::kBlockBytes);
      else tc::mbar_arrive(bar);
    }
    ++issued;
    into = into + 1 == L::kStages ? 0 : into + 1;
  };
  // the first copies: a lane each
  if (n_mine > 0) {
    fill_window(0);
    issued = min(n_mine, L::kStages);
    into = issued == L::kStages ? 0 : static_cast<uint32_t>(issued);
    if (lane < issued) {
      const uint32_t bar = bars + 8 * lane, dst = ring + lane * 2 * L::kBlockBytes;
      if (at_codes >= 0) {
        tc::bulk_load(dst, a.c.k + at_codes, L::kBlockBytes, bar);
        tc::bulk_load(dst + L::kBlockBytes, a.c.v + at_codes, L::kBlockBytes, bar);
      }
      scales[lane] = make_float2(at_scales.x, log_scale(at_scales.y));
      if (at_codes >= 0) tc::mbar_arrive_expect_tx(bar, 2 * L::kBlockBytes);
      else tc::mbar_arrive(bar);
    }
    __syncwarp();
  }

  int taken = 0;  // blocks of this warp done
  uint32_t from = 0, parity = 0;  // stage and phase of the next one
  bool alive = true;
  const int G = a.H / a.c.H;
#pragma unroll 1
  for (int at = 0; at < n_cta || (kCluster && at == 0);) {
    // the segment: units [at, at + n) of the CTA, blocks [seg.blk, seg.blk + n) of one item
    const int n = min(seg.units - seg.blk, n_cta - at);
    const int R = seg.s.q_len * G;
    const int min_sees = a.causal ? seg.s.len - seg.s.q_len + 1 : seg.s.len;  // of the first token
    // Queries: A fragments of the key products, rows g and g + 8 of each 16. All
    // warps make them (each needs the rows' powers of two) and put a part of them
    // into shared memory, where the joins' buffer lies idle: a lane's four
    // registers of a product are one 16-byte load, and 32 registers stay free.
    uint4* qs = reinterpret_cast<uint4*>(smem + L::kOffMerge) + lane;
    float f[MT][2];
    int sees[MT][2];  // keys that the row sees (a length fits 31 bits)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      uint4 raw[2][D / 32];  // channels 64 i + 16 t and up
      load_queries<D>(a, seg, mt, g, t, raw);
      uint32_t qf[kHalves][4][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = mt * 16 + e * 8 + g;
        sees[mt][e] = r >= R ? 0 : (a.causal ? seg.s.len - seg.s.q_len + 1 + r / G : seg.s.len);
        uint32_t amax = 0;
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
          const uint32_t w[4] = {raw[e][x].x, raw[e][x].y, raw[e][x].z, raw[e][x].w};
#pragma unroll
          for (int y = 0; y < 4; ++y) amax = max(amax, max(w[y] & 0x7FFFu, (w[y] >> 16) & 0x7FFFu));
        }
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // the power of two below the largest value; infinities and NaN stay what they are
        uint32_t ex = amax >> 7;
        ex = ex == 255u ? 127u : min(max(ex, 1u), 253u);
        const float down = __uint_as_float((254u - ex) << 23);
        f[mt][e] = __uint_as_float(ex << 23) * a.sm_log2;
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
          const uint32_t w[4] = {raw[e][x].x, raw[e][x].y, raw[e][x].z, raw[e][x].w};
#pragma unroll
          for (int y = 0; y < 4; ++y)
            qf[x >> 1][(x & 1) * 2 + (y >> 1)][(y & 1) * 2 + e] =
                pack_half2(__uint_as_float(w[y] << 16) * down, __uint_as_float(w[y] & 0xFFFF0000u) * down);
        }
      }
#pragma unroll
      for (int i = 0; i < kHalves; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (x == warp)
            qs[((mt * kHalves + i) * 4 + x) * 32] = make_uint4(qf[i][x][0], qf[i][x][1], qf[i][x][2], qf[i][x][3]);
    }
    __syncthreads();
    float2 o[MT][D / 8][2];  // rows g and g + 8: channels 8x + 2t, + 1
    float l[MT][2];          // and the sum of this lane's keys
    bool large = false;      // a value scale above 2^kLogPlainMax has been met
    float m[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 0; x < D / 8; ++x) o[mt][x][e] = make_float2(0.0f, 0.0f);
        l[mt][e] = 0.0f;
        m[mt][e] = -INFINITY;
      }
    // this warp's blocks of the segment: CTA units that are warp mod kWarps
    const int first = at + (warp - at % kWarps + kWarps) % kWarps;
#pragma unroll 1
    for (int u = first; u < at + n && alive; u += kWarps) {
      const uint32_t s = from;
      alive = __all_sync(0xffffffffu, wait_bounded(bars + 8 * s, parity, a.dev_err));
      if (!alive) break;
      const float2 sc = scales[s];
      // one block of keys; `odd` takes its part of the sums apart from the weights
      const auto block = [&](auto odd) {
        const uint8_t* kb = smem + (ring - sbase) + s * 2 * L::kBlockBytes;
        const uint8_t* vb = kb + L::kBlockBytes;
        const int key0 = (seg.blk + (u - at)) * kCacheBlock;
        float z[MT][4][4];
#pragma unroll
        for (int i = 0; i < kHalves; ++i) {
          uint32_t cw[4][4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(cw[j]) = *reinterpret_cast<const uint4*>(kb + i * 2048 + j * 512 + lane * 16);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t qa[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) *reinterpret_cast<uint4*>(qa[mt]) = qs[((mt * kHalves + i) * 4 + x) * 32];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t b0, b1;
              codes_to_half(cw[j][x], b0, b1);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                if (i == 0 && x == 0) mma16816(z[mt][j], qa[mt], b0, b1, 0.0f, 0.0f, 0.0f, 0.0f);
                else mma16816(z[mt][j], qa[mt], b0, b1);
              }
            }
          }
        }
        const bool masked = key0 + kCacheBlock > min_sees;
        if (masked) {
          // keys behind what the row sees: below every number here, and p = 0 below
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (key0 + 8 * j + 2 * t + (x & 1) >= sees[mt][x >> 1]) z[mt][j][x] = -INFINITY;
        }
        uint32_t pf[MT][2][4];
        // a number in any case: where the scale is NaN so are the weights of the rows that see the block
        const float log_min = fmaxf(sc.y, kLogScaleMin), unscale = ex2(-log_min);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          // logits are z * c with c >= 0, so the largest z gives the largest of a block
          float c[2], zm[2], mx[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            c[e] = f[mt][e] * sc.x;
            float y = max3(z[mt][0][2 * e], z[mt][0][2 * e + 1], z[mt][1][2 * e]);
            y = max3(y, z[mt][1][2 * e + 1], z[mt][2][2 * e]);
            y = max3(y, z[mt][2][2 * e + 1], z[mt][3][2 * e]);
            y = fmaxf(y, z[mt][3][2 * e + 1]);
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 1));
            zm[e] = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
            mx[e] = zm[e] == -INFINITY ? -INFINITY : fmaf(zm[e], c[e], log_min);
          }
          if (__any_sync(0xffffffffu, mx[0] > m[mt][0] + kLazy || mx[1] > m[mt][1] + kLazy)) {
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float up = fmaxf(m[mt][e], mx[e]), half = up == -INFINITY ? 1.0f : half_step(m[mt][e], up);
              alpha[e] = half * half;
              m[mt][e] = up;
              l[mt][e] = rescale(l[mt][e], half);
            }
#pragma unroll
            for (int x = 0; x < D / 8; ++x)
#pragma unroll
              for (int e = 0; e < 2; ++e) o[mt][x][e] = __fmul2_rn(o[mt][x][e], make_float2(alpha[e], alpha[e]));
          }
          if constexpr (decltype(odd)::value) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float top = zm[e] * c[e];
              float part = 0.0f;
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                  if (key0 + 8 * j + 2 * t + x < sees[mt][e]) part += ex2(fmaf(z[mt][j][2 * e + x], c[e], -top));
              if (zm[e] != -INFINITY) l[mt][e] += rescale(part, half_step(top, m[mt][e]));
            }
          }
          const float add[2] = {sc.y - (m[mt][0] == -INFINITY ? 0.0f : m[mt][0]),
                                sc.y - (m[mt][1] == -INFINITY ? 0.0f : m[mt][1])};
          float2 p[4][2];
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 y = __ffma2_rn(make_float2(z[mt][j][2 * e], z[mt][j][2 * e + 1]), make_float2(c[e], c[e]),
                                          make_float2(add[e], add[e]));
              p[j][e] = make_float2(ex2(y.x), ex2(y.y));
            }
          if (masked) {
            // a scale of 0 or NaN would make a hidden key's logit NaN
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                if (key0 + 8 * j + 2 * t >= sees[mt][e]) p[j][e].x = 0.0f;
                if (key0 + 8 * j + 2 * t + 1 >= sees[mt][e]) p[j][e].y = 0.0f;
              }
          }
          float2 sum[2] = {p[0][0], p[0][1]};
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (j > 0) sum[e] = __fadd2_rn(sum[e], p[j][e]);
              pf[mt][j >> 1][(j & 1) * 2 + e] = pack_half2(p[j][e].x, p[j][e].y);
            }
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (!decltype(odd)::value) l[mt][e] = fmaf(sum[e].x + sum[e].y, unscale, l[mt][e]);
        }
#pragma unroll
        for (int x = 0; x < D / 8; ++x) {
          const uint2 c = *reinterpret_cast<const uint2*>(vb + x * 256 + lane * 8);
          uint32_t b[4];
          codes_to_half(c.x, b[0], b[1]);
          codes_to_half(c.y, b[2], b[3]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            float d[4];
            mma16816(d, pf[mt][0], b[0], b[1], 0.0f, 0.0f, 0.0f, 0.0f);
            mma16816(d, pf[mt][1], b[2], b[3]);
#pragma unroll
            for (int e = 0; e < 2; ++e)
              o[mt][x][e] = __fadd2_rn(o[mt][x][e], make_float2(d[2 * e], d[2 * e + 1]));
          }
        }
      };
      if (sc.x >= 0.0f || sc.x != sc.x) {
        large |= sc.y > kLogPlainMax;
        // (the same for all lanes)
        if (__builtin_expect(!large && !(sc.y < kLogPlainMin), 1)) block(std::false_type{});
        else block(std::true_type{});
      }
      ++taken;
      from = from + 1 == L::kStages ? 0 : from + 1;
      if (from == 0) parity ^= 1u;
      __syncwarp();  // every lane is done with the stage
      issue();
    }

    // the next item's queries are on their way to L1 during the join (its head
    // is the next one of the sequence, unless that was the last)
    if (!kCluster && at + n < n_cta && seg.h + 1 < a.c.H && threadIdx.x < R * (D / 64)) {
      const int r = threadIdx.x / (D / 64), tok = r / G;
      const uint16_t* p = a.q.p + seg.b * a.q.sb + tok * a.q.ss + ((seg.h + 1) * G + r - tok * G) * a.q.sh +
                          64 * (threadIdx.x % (D / 64));
      asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
    }

    // join the warps' parts of the item
    float2* ml = reinterpret_cast<float2*>(smem + L::kOffMl);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y = l[mt][e];
        y += __shfl_xor_sync(0xffffffffu, y, 1);
        y += __shfl_xor_sync(0xffffffffu, y, 2);
        if (t == 0) ml[warp * 16 * MT + mt * 16 + e * 8 + g] = make_float2(m[mt][e], y);
      }
    if (a.zero_rest && seg.blk == 0) {
      // padding rows, by the CTA that has the item's first block
      const int rest = (static_cast<int>(a.T) - seg.s.q_len) * G;
      for (int x = threadIdx.x; x < rest * (D / 8); x += kThreads) {
        const int r = R + x / (D / 8), tok = r / G, head = seg.h * G + r - tok * G;
        *reinterpret_cast<uint4*>(a.out.p + seg.b * a.out.sb + tok * a.out.ss + head * a.out.sh + x % (D / 8) * 8) =
            make_uint4(0u, 0u, 0u, 0u);
        if (a.lse != nullptr && x % (D / 8) == 0)
          a.lse[(static_cast<int64_t>(seg.b) * a.H + head) * a.T + tok] = -INFINITY;
      }
    }
    const bool whole = kCluster ? parts == 1 : n == seg.units;
    const int which = at == 0 ? 0 : 1;  // a partial item is the range's first or its last
    // a cluster's parts stay in shared memory, over the ring, whose blocks are used up
    float* part = kCluster ? reinterpret_cast<float*>(smem)
                           : reinterpret_cast<float*>(static_cast<char*>(a.workspace) + L::kDesc) +
                                 (static_cast<size_t>(blockIdx.x) * 2 + which) * L::kSlot;
    if (!kCluster && at + n == n_cta && threadIdx.x == 0) {
      // the last item, if it begins here and goes on in other CTAs: up to which one, and whose rows
      const int rest = seg.units - seg.blk - n;
      desc[blockIdx.x] = seg.blk == 0 && rest > 0 ? make_int4(split.owner(hi + rest - 1), seg.b, 2 * seg.h + which, 0)
                                                  : make_int4(-1, 0, 0, 0);
    }
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt * 16 >= R) break;
      // 16 rows x 32 channels of each warp at a time, or where there are no more
      // than 8 rows 8 x 64: pairs of channels, pair u of row r at u ^ 4 (r mod 4),
      // which is free of bank conflicts
      const bool few = R - mt * 16 <= 8;
      const int row = few ? threadIdx.x >> 4 : threadIdx.x >> 3, c4 = few ? threadIdx.x & 15 : threadIdx.x & 7;
      const int r = mt * 16 + row;
      float top = -INFINITY, sum = 0.0f, wt[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * 16 * MT + r].x);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 x = ml[w * 16 * MT + r];
        const float half = half_step(x.x, top == -INFINITY ? 0.0f : top);
        wt[w] = half * half;
        sum += rescale(x.y, half);
      }
      const int tok = r / G, head = seg.h * G + r - tok * G;
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      uint16_t* dst = a.out.p + seg.b * a.out.sb + tok * a.out.ss + head * a.out.sh + 4 * c4;
      if (r < R && c4 == 0) {
        if (!whole) *reinterpret_cast<float2*>(part + 16 * MT * D + 2 * r) = make_float2(top, sum);
        else if (a.lse != nullptr)
          a.lse[(static_cast<int64_t>(seg.b) * a.H + head) * a.T + tok] =
              sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
      }
      float2* buf = reinterpret_cast<float2*>(smem + L::kOffMerge);
      // sums the warps' channels 4 c4 .. + 3 of the row, `pitch` pairs a row and `rows` rows a warp, and puts them out
      const auto gather = [&](int first, int rows, int pitch) {
        if (r >= R) return;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 y = *reinterpret_cast<const float4*>(buf + (w * rows + row) * pitch + ((2 * c4) ^ ((row & 3) * 4)));
          acc.x = fmaf(y.x, wt[w], acc.x);
          acc.y = fmaf(y.y, wt[w], acc.y);
          acc.z = fmaf(y.z, wt[w], acc.z);
          acc.w = fmaf(y.w, wt[w], acc.w);
        }
        if (whole) {
          const __nv_bfloat162 lo2 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
          const __nv_bfloat162 hi2 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
          *reinterpret_cast<uint2*>(dst + first) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&lo2), *reinterpret_cast<const uint32_t*>(&hi2));
        } else {
          *reinterpret_cast<float4*>(part + r * D + first + 4 * c4) = acc;
        }
      };
      if (few) {
#pragma unroll
        for (int cut = 0; cut < D / 64; ++cut) {
#pragma unroll
          for (int x = 0; x < 8; ++x) buf[(warp * 8 + g) * 32 + ((4 * x + t) ^ ((g & 3) * 4))] = o[mt][cut * 8 + x][0];
          __syncthreads();
          gather(cut * 64, 8, 32);
          __syncthreads();
        }
      } else {
#pragma unroll
        for (int cut = 0; cut < D / 32; ++cut) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int u = (4 * x + t) ^ ((g & 3) * 4);
            buf[(warp * 16 + g) * 16 + u] = o[mt][cut * 4 + x][0];
            buf[(warp * 16 + g + 8) * 16 + u] = o[mt][cut * 4 + x][1];
          }
          __syncthreads();
          gather(cut * 32, 16, 16);
          __syncthreads();
        }
      }
    }
    if (R == 0) __syncthreads();
    if constexpr (kCluster) {
      if (parts > 1) {
        tc::cluster_arrive_release();
        tc::cluster_wait_acquire();
        join_cluster<D, MT>(a, sbase, rank, parts, seg.b, seg.h, R);
        __syncwarp();
        // no CTA ends while another reads its shared memory
        tc::cluster_arrive_release();
        tc::cluster_wait_acquire();
      }
      break;
    }
    at += n;
    seg.blk += n;
    if (at < n_cta) cursor_settle(a, seg);
  }
  if (!alive) {
    // copies in flight land before the CTA ends
    for (; taken < issued; ++taken) {
      wait_bounded(bars + 8 * from, parity, a.dev_err);
      from = from + 1 == L::kStages ? 0 : from + 1;
      if (from == 0) parity ^= 1u;
    }
  }
}

// Joins the items that several CTAs share. Block (c, y) serves the item that
// begins in CTA c and ends in a later one. kShare warps share a row, each with
// every kShare-th part; or a warp has kJoinRows rows, whose loads do not wait for
// one another.
constexpr int kJoinWarps = 8;
constexpr int kJoinRows = 2;
__host__ __device__ constexpr int join_rows(int share) { return share > 1 ? kJoinWarps / share : kJoinWarps * kJoinRows; }
template <int D, int kShare>
__global__ void __launch_bounds__(kJoinWarps * 32) cache_join_kernel(const CacheAttentionArgs a, int slot_rows,
                                                                     size_t desc_bytes) {
  constexpr int kV = D / 32;  // channels per lane
  __shared__ float acc_s[kJoinWarps][D];
  __shared__ float2 ml_s[kJoinWarps];
  tc::griddep_wait();
  const int c0 = static_cast<int>(blockIdx.x);
  const int4 item = static_cast<const int4*>(a.workspace)[c0];
  if (item.x < 0) return;
  const int G = a.H / a.c.H;
  bool bad = false;
  const int R = load_seq(a, item.y, &bad).q_len * G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kRows = kShare > 1 ? 1 : kJoinRows, kAhead = kShare > 1 ? 4 : 2;  // rows of a warp, parts in flight
  const int row0 = static_cast<int>(blockIdx.y) * join_rows(kShare) + warp / kShare * kRows;
  const size_t slot = static_cast<size_t>(slot_rows) * (D + 2);
  const float* ws = reinterpret_cast<const float*>(static_cast<const char*>(a.workspace) + desc_bytes);
  float top[kRows], sum[kRows], acc[kRows][kV];
  bool real[kRows];
#pragma unroll
  for (int y = 0; y < kRows; ++y) {
    real[y] = row0 + y < slot_rows && item.w + row0 + y < R;
    top[y] = -INFINITY;
    sum[y] = 0.0f;
#pragma unroll
    for (int v = 0; v < kV; ++v) acc[y][v] = 0.0f;
  }
  if (real[0]) {
    for (int c = c0 + warp % kShare; c <= item.x; c += kAhead * kShare) {
      float2 x[kRows][kAhead];
      float z[kRows][kAhead][kV];
#pragma unroll
      for (int y = 0; y < kRows; ++y)
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int ci = c + i * kShare;
          x[y][i] = make_float2(-INFINITY, 0.0f);
#pragma unroll
          for (int v = 0; v < kV; ++v) z[y][i][v] = 0.0f;
          if (ci <= item.x && real[y]) {
            const float* p = ws + (static_cast<size_t>(ci) * 2 + (ci == c0 ? item.z & 1 : 0)) * slot;
            x[y][i] = *reinterpret_cast<const float2*>(p + slot_rows * D + 2 * (row0 + y));
            if constexpr (kV == 4)
              *reinterpret_cast<float4*>(z[y][i]) = *reinterpret_cast<const float4*>(p + (row0 + y) * D + 4 * lane);
            else
              *reinterpret_cast<float2*>(z[y][i]) = *reinterpret_cast<const float2*>(p + (row0 + y) * D + 2 * lane);
          }
        }
#pragma unroll
      for (int y = 0; y < kRows; ++y) {
        float up = top[y];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) up = fmaxf(up, x[y][i].x);
        const float ref = up == -INFINITY ? 0.0f : up, step = half_step(top[y], ref), alpha = step * step;
        top[y] = up;
        sum[y] = rescale(sum[y], step);
#pragma unroll
        for (int v = 0; v < kV; ++v) acc[y][v] *= alpha;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const float half = half_step(x[y][i].x, ref), wt = half * half;
          sum[y] += rescale(x[y][i].y, half);
#pragma unroll
          for (int v = 0; v < kV; ++v) acc[y][v] = fmaf(z[y][i][v], wt, acc[y][v]);
        }
      }
    }
  }
  if constexpr (kShare > 1) {
#pragma unroll
    for (int v = 0; v < kV; ++v) acc_s[warp][kV * lane + v] = acc[0][v];
    if (lane == 0) ml_s[warp] = make_float2(top[0], sum[0]);
    __syncthreads();
    if (!real[0] || warp % kShare != 0) return;
#pragma unroll
    for (int w = 0; w < kShare; ++w) top[0] = fmaxf(top[0], ml_s[warp + w].x);
    const float ref = top[0] == -INFINITY ? 0.0f : top[0];
    sum[0] = 0.0f;
#pragma unroll
    for (int v = 0; v < kV; ++v) acc[0][v] = 0.0f;
#pragma unroll
    for (int w = 0; w < kShare; ++w) {
      const float half = half_step(ml_s[warp + w].x, ref), wt = half * half;
      sum[0] += rescale(ml_s[warp + w].y, half);
#pragma unroll
      for (int v = 0; v < kV; ++v) acc[0][v] = fmaf(acc_s[warp + w][kV * lane + v], wt, acc[0][v]);
    }
  }
#pragma unroll
  for (int y = 0; y < kRows; ++y) {
    if (!real[y]) break;
    const float inv = sum[y] == 0.0f ? 0.0f : 1.0f / sum[y];
    const int r = item.w + row0 + y, tok = r / G, head = (item.z >> 1) * G + r - tok * G;
    uint16_t* p = a.out.p + item.y * a.out.sb + tok * a.out.ss + head * a.out.sh + kV * lane;
#pragma unroll
    for (int v = 0; v < kV; v += 2) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(acc[y][v] * inv, acc[y][v + 1] * inv);
      *reinterpret_cast<uint32_t*>(p + v) = *reinterpret_cast<const uint32_t*>(&b);
    }
    if (a.lse != nullptr && lane == 0)
      a.lse[(static_cast<int64_t>(item.y) * a.H + head) * a.T + tok] =
          sum[y] == 0.0f ? -INFINITY : (top[y] + log2f(sum[y])) * kLn2;
  }
}

template <int D, int MT>
cudaError_t launch_decode(const CacheAttentionArgs& a, cudaStream_t stream) {
  using L = Dec<D, MT>;
  const int64_t items = a.B * a.c.H;
  const int64_t item_blocks = table_capacity(a.pt.max_pages, a.c.blocks_per_page) / kCacheBlock;
  const int sms = sm_count_current() < kMaxSms ? sm_count_current() : kMaxSms;
  const int64_t most = static_cast<int64_t>(sms) * L::kCtasPerSm;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::kBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  // one launch, a cluster per item, where the clusters fit the GPU at once and
  // a warp gets few blocks: one sequence of 1000 tokens 8.7 us through the list
  // and the second kernel, 6.7 so; one of 4000 11.7 and 9.9; 16 x 5 drafts over
  // 4001 tokens of 4 heads of 64 26 and 19. With more blocks a warp the clusters,
  // at most 8 CTAs an item, leave SMs idle that the list's even ranges use.
  // (The blocks are those that the tables can name, since the lengths are on the
  // device: a table for 131072 tokens sends 1000 through the list, 10.3 us where
  // rows of their own length take 7.1.)
  // Clusters leave some places of the SMs empty, so nine tenths are given out:
  // 16 sequences of 1000 tokens, 4 heads of 64, 7.6 us, 12.2 where all are and
  // some clusters wait; 4001 tokens 12.5 with 6 CTAs an item, 14.9 with 4
  int parts = 1;
  while (parts < 8 && parts * kWarps < item_blocks && items * (parts + 1) * 10 <= most * 9) ++parts;
  if (items <= most && item_blocks <= parts * kWarps * kClusterBlocks) {
    if ((e = set_smem_limit_once(reinterpret_cast<const void*>(cache_decode_kernel<D, MT, true>), L::kBytes)) !=
        cudaSuccess)
      return e;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(parts);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    cfg.gridDim = dim3(static_cast<unsigned>(items * parts));
    return cudaLaunchKernelEx(&cfg, cache_decode_kernel<D, MT, true>, a);
  }
  // else a CTA for every 4 blocks that the tables can name (one per warp), at most what the SMs hold
  const int64_t want = div_up(items * item_blocks, kWarps);
  const unsigned ctas = static_cast<unsigned>(want < 1 ? 1 : (want < most ? want : most));
  if ((e = set_smem_limit_once(reinterpret_cast<const void*>(cache_decode_kernel<D, MT, false>), L::kBytes)) !=
      cudaSuccess)
    return e;
  cfg.gridDim = dim3(ctas);
  if ((e = cudaLaunchKernelEx(&cfg, cache_decode_kernel<D, MT, false>, a)) != cudaSuccess || ctas == 1) return e;
  return launch_cache_join(a, D, 16 * MT, static_cast<int>(a.T * (a.H / a.c.H)), static_cast<int>(ctas), L::kDesc,
                           stream);
}

}  // namespace

cudaError_t launch_cache_join(const CacheAttentionArgs& a, int64_t D, int slot_rows, int rows, int ctas,
                              size_t desc_bytes, cudaStream_t stream) {
  // 8 warps to a row where an item has many parts and not too many rows (a
  // sequence of 131071 tokens, 28 heads on 4: 35 us, 60 with a warp per row; 64 rows
  // a head over 20000 tokens 27 and 32, 128 rows 35 and 37), else a warp (300 x 4
  // rows over 4000 tokens, few parts: 40 us, 64 with 8 warps per row; 256 rows over
  // 20000, many parts: 39 and 45)
  const int64_t items = a.B * a.c.H * div_up(a.T * (a.H / a.c.H), slot_rows);
  const int share = ctas > 8 * items && rows <= 128 ? 8 : 1;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(div_up(rows, join_rows(share))));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto kernel = D == 128 ? (share > 1 ? cache_join_kernel<128, 8> : cache_join_kernel<128, 1>)
                               : (share > 1 ? cache_join_kernel<64, 8> : cache_join_kernel<64, 1>);
  return cudaLaunchKernelEx(&cfg, kernel, a, slot_rows, desc_bytes);
}

size_t cache_attention_workspace_bytes(int64_t, int64_t T, int64_t H, int64_t Hkv, int64_t D) {
  const int64_t rows = T * (H / Hkv);
  if (rows <= 16) return D == 128 ? Dec<128, 1>::kWorkspace : Dec<64, 1>::kWorkspace;
  if (rows <= 32) return D == 128 ? Dec<128, 2>::kWorkspace : Dec<64, 2>::kWorkspace;
  return cache_attention_tc_workspace_bytes(D);
}

// By the rows of a key/value head (14 x 20000 tokens, 8 heads of 128, us): up to
// 16 one row tile, 98 (8 rows) and 100 (16); up to 32 two, 137; more on the tcgen05
// tensor cores, 171 (40 rows) to 181 (128) and 254 (256). Its 128-row tiles take
// as long for 20 rows as for 40, and four row tiles have no registers.
cudaError_t launch_cache_attention(const CacheAttentionArgs& a, int64_t D, cudaStream_t stream) {
  const int64_t rows = a.T * (a.H / a.c.H);
  if (rows <= 16) return D == 128 ? launch_decode<128, 1>(a, stream) : launch_decode<64, 1>(a, stream);
  if (rows <= 32) return D == 128 ? launch_decode<128, 2>(a, stream) : launch_decode<64, 2>(a, stream);
  return launch_cache_attention_tc(a, D, stream);
}

}  // namespace sage
