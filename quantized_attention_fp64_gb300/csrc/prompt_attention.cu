// Attention over packed prompts on the sm_103a tensor cores (tcgen05, TMA, TMEM).
//
//   out_t = sum_j p_tj v_j / sum_j p_tj,  p_tj = 2^(c (q_t . k_j - m_t)),  c = sm_scale log2 e
// over the keys that row t sees: all m of its sequence, or with the causal mask
// the first m - n + t + 1 (n queries). Both products are BF16 with fp32 sums; P
// is rounded to BF16, l_t = sum_j p_tj is taken in fp32 before that. (The tensor core
// wants P in the type of V. Outputs are off by 0.19 to 0.23% of their norm so, and by 0.16%
// with P in fp32, which is the outputs' own rounding; a second product for the rest of
// P would bring that for half as much tensor work again.)
//
// A unit of work is two query tiles of 128 rows that share the key tiles (128 keys)
// which pass through shared memory: the same rows of two query heads of a key/value
// head, or where the heads are odd, the last head's rows and the first one's next. So
// both have the same key tiles, or the second one more. (Two row tiles of one
// head, as it was, leave the first without work for the second's last key tile: 16
// prompts up to 2000 tokens, 32 heads on 8, took 200 us, and now 192.) Where there are
// fewer than SMs a unit is one tile.
// A first kernel lists the units' blocks of all sequences, those with the most key
// tiles first; the CTAs, one for each SM, take the units in that order forth and
// back (0 1 .. 151, 151 .. 1 0, ...), so that each gets about the same work whatever
// the lengths are. Calls of at most a unit for each SM do without. Roles of the 16 warps:
//   warp 0      TMA: the unit's queries, and a ring of key and value tiles in turn
//   warps 1, 2  TMEM allocation; the products of query tile 0, 1 (one thread issues)
//   warp 3      in the second pass (below): clears infinities and NaN in value tiles
//   warps 4-7, 8-11  softmax of query tile 0, 1 (TMEM lane = row)
//   warps 12-15 output: O of either tile, scaled and stored
// TMEM holds S0, S1, O0, O1: all 512 columns at D = 128. The softmax reads S of a
// key tile into registers and writes P over it, from where the product with V
// reads it; that product and the next S = Q K^T are issued together when P is
// there, so the tensor pipe works on one query tile while the other's softmax runs.
// The maximum m_t that the exponentials go by follows only when the true one has
// grown by 2^8: O is rescaled then, a few times at the beginning of a row. It is set
// 2^8 above the true one, so that no weight is above 1 and O overflows no sooner than
// the sum of a softmax by the true maximum (no bit is lost in floating point).
//
// Long rows. The tensor core cuts a product off at 2^-25 of the sum that it is added to or
// a little below, towards 0: one sum over 2^20 keys came out 0.5% too small, one over 2^24
// 10%. So O and l begin anew every 65536 keys (2^-10 at most is lost, 2^-12 measured); what
// they held goes to parts in the workspace, by fp32 additions, and comes back at the end
// of the unit.
//
// What a row does not see must not touch it, whatever stands there: its P is 0,
// but 0 times an infinity or a NaN of V is a NaN. And what it does see has a weight
// above 0, by the formula, though P may be 0 where the exponential leaves fp32. The
// output warps look for infinities and NaN in what they store, and a unit that has
// one is done again in a second pass. There warp 3 clears the rows of V behind the
// sequence's end and every infinity and NaN, before the product takes them. Those of
// tiles that all rows of the unit see are remembered by channel, and the output
// warps add them to every row; in the other tiles (the diagonal) they look the
// values up and add them to the rows that see them. Calls with finite values pay for the look at the outputs
// alone (2% of the prompts above); a look at all values beforehand took 23 us of
// them, one at the value tiles as they pass by 32.
//
// What bounds it. D = 128: the tensor pipe; 16384 causal tokens, 28 heads on 4, run at 1540
// to 1690 TFLOP/s (1250 to 1140 us, by what ran before; 79 to 86% of the measured peak of
// cuBLAS in a burst, which no kernel keeps up under the power limit: 1752 TFLOP/s for seconds).
// 16 prompts up to 2000 tokens, 1050 TFLOP/s (190 us): the masked halves of the diagonal tiles, ends of
// sequences, and a microsecond to begin and end a unit of 6 key tiles. D = 64: the
// softmax, whose exponentials are as many with half the products; 16384 tokens both
// ways 1060 TFLOP/s, 1.2 us for a step of two tiles. Code that runs once in a unit is kept short: it is fetched anew each
// time (the output warps' loop over 32 channels, three times as long, cost the
// prompts above 20 us).
//
// Every wait on an mbarrier is bounded; when one runs out the kernel sets the
// device error word, tells the other roles to stop, lets its copies and products
// drain, frees its TMEM and returns.
#include <cuda.h>

#include "launch.cuh"
#include "prompt.cuh"
#include "tc_kernel.cuh"

namespace sage {
namespace {

constexpr int kThreads = 512;
constexpr int kRows = 128;      // query rows of a tile
constexpr int kKeys = 128;      // keys of a tile
constexpr int kFixes = 8;       // more than the value tiles (at most 5 in the ring), and so the units, that warp 3 may be ahead
constexpr uint32_t kRedoWords = 8;
// What warp 3 has cleared in a unit: values that some of its rows see, and that all do.
constexpr uint32_t kBadSome = 1, kBadAll = 2;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kFold = 512;      // key tiles that O holds at most, a power of two
constexpr int kMostCtas = 160;  // for which the workspace has parts
constexpr float kGrowth = 8.0f; // the maximum follows when it has grown by 2^8, and is set that far above

// One or two query tiles of a key/value head, the same for each of them.
struct alignas(16) Block {
  int32_t q0, rows;   // first row of tile 0 in the tensor, rows of the sequence from there on
  int32_t kv0, keys;  // first key row, keys of the sequence
  int32_t sees;       // keys that row 0 sees with the causal mask, before it is cut to 0 .. keys
  int32_t g0, g1;     // query heads of tile 0 and 1 among those of the key/value head; g1 < 0: no tile 1
  int32_t down;       // rows that tile 1 begins behind tile 0: 0 or kRows
};

struct Header {
  int32_t blocks;            // entries of the list
  int32_t rest_lo, rest_hi;  // rows [0, rest_lo) and [rest_hi, N) belong to no sequence
};
constexpr size_t kHeaderBytes = 256;  // then the list

// Blocks of at most `pair` tiles that N rows in B sequences can make: of every
// sequence (rows / 128, rounded up) times the heads of a key/value head, in twos.
inline int64_t most_blocks(int64_t N, int64_t B, int64_t group, int pair) {
  const int64_t tiles = (N / kRows + B) * group;
  return pair == 1 ? tiles : (tiles + B) / 2;
}

// Tile i's first row and its rows, counted from the block's first.
__device__ __forceinline__ int32_t begin_of(const Block& b, int i) { return i == 0 ? 0 : b.down; }
__device__ __forceinline__ int32_t rows_of(const Block& b, int i) {
  return i == 1 && b.g1 < 0 ? 0 : min(kRows, b.rows - begin_of(b, i));
}
// Keys that row r of a block sees.
template <bool kCausal>
__device__ __forceinline__ int32_t sees(const Block& b, int32_t r) {
  return kCausal ? max(0, min(b.sees + r, b.keys)) : b.keys;
}
__device__ __forceinline__ int32_t tiles_of(int32_t keys) { return (keys + kKeys - 1) >> 7; }  // (keys are at most 2^30)
static_assert(kKeys == 128, "key tiles are counted by shifts");
// Key tiles of query tile i of a block.
template <bool kCausal>
__device__ __forceinline__ int32_t key_tiles(const Block& b, int i) {
  const int32_t rows = rows_of(b, i);
  return rows <= 0 ? 0 : tiles_of(sees<kCausal>(b, begin_of(b, i) + rows - 1));
}

// u / d for u below 2^31, by a multiplication.
struct Divisor {
  int32_t d;
  uint32_t mul;
  int shift;
  explicit Divisor(int32_t x) : d(x), mul(0), shift(0) {
    while ((int64_t(1) << shift) < x) ++shift;  // 2^shift >= d
    if (x > 1) mul = static_cast<uint32_t>((uint64_t(1) << (31 + shift)) / static_cast<uint64_t>(x) + 1), --shift;
  }
  __device__ __forceinline__ int32_t of(int32_t u) const {
    return d == 1 ? u : static_cast<int32_t>(__umulhi(static_cast<uint32_t>(u), mul) >> shift);
  }
};

// ------------------------------------------------------------------ planning --

__device__ __forceinline__ bool bad_offsets(const int32_t* offsets, const int32_t* kv_offsets, int32_t b, int32_t N,
                                            int32_t M) {
  const int32_t o = offsets[b], k = kv_offsets[b];
  return o < 0 || o > N || k < 0 || k > M || (b > 0 && (offsets[b - 1] > o || kv_offsets[b - 1] > k));
}

// The p-th block of sequence b: its tiles are numbered head by head of a
// key/value head, and then row tile by row tile, so that the two of a block have
// the same key tiles, or the second has one more.
__device__ __forceinline__ int32_t blocks_of(const int32_t* offsets, int32_t b, int32_t group, int pair) {
  const int32_t tiles = (offsets[b + 1] - offsets[b] + kRows - 1) / kRows * group;
  return (tiles + pair - 1) / pair;
}
__device__ __forceinline__ Block block_of(const int32_t* offsets, const int32_t* kv_offsets, int32_t b, int32_t p,
                                          const Divisor& group, int pair) {
  const int32_t q0 = offsets[b], n = offsets[b + 1] - q0, kv0 = kv_offsets[b], m = kv_offsets[b + 1] - kv0;
  const int32_t tile = p * pair, at = group.of(tile), g = tile - at * group.d;
  const bool next = g + 1 == group.d;  // tile 1 is of the next rows
  Block e;
  e.q0 = q0 + at * kRows;
  e.rows = n - at * kRows;
  e.kv0 = kv0;
  e.keys = m;
  e.sees = m - n + at * kRows + 1;
  e.g0 = g;
  e.g1 = pair == 1 || (next && e.rows <= kRows) ? -1 : next ? 0 : g + 1;
  e.down = next ? kRows : 0;
  return e;
}

constexpr int kPlanThreads = 512;
constexpr int kBins = kPlanThreads;

// acc stays (0, 0) as long as no BF16 of the pairs is an infinity or a NaN.
__device__ __forceinline__ uint32_t collect(uint32_t pair, uint32_t acc) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(pair), "r"(0u), "r"(acc));
  return d;
}
// Those are the sign bits of this.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7FFF7FFFu) + 0x00800080u) & 0x80008000u; }
__device__ __forceinline__ uint32_t not_finite(const uint4& u) {
  return not_finite(u.x) | not_finite(u.y) | not_finite(u.z) | not_finite(u.w);
}
// Eight channels with infinities or NaN: a bit for each that holds +inf goes to `up`, for
// -inf to `down`, for a NaN to both, and those become 0.
__device__ __forceinline__ void take_odd(uint4& u, uint32_t& up, uint32_t& down) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t odd = not_finite(w[k]), low = odd >> 15 & 1u, high = odd >> 31;
    const uint32_t nan_low = (w[k] & 0x7Fu) != 0u, nan_high = (w[k] & 0x7F0000u) != 0u;
    const uint32_t neg_low = w[k] >> 15 & 1u, neg_high = w[k] >> 31;
    up |= ((low & (nan_low | (neg_low ^ 1u))) | (high & (nan_high | (neg_high ^ 1u))) << 1) << (2 * k);
    down |= ((low & (nan_low | neg_low)) | (high & (nan_high | neg_high)) << 1) << (2 * k);
    w[k] &= ~(odd | (odd - (odd >> 15)));
  }
}
// And into the eight channels at p.
__device__ __forceinline__ void add_odd(uint16_t* p, uint32_t up, uint32_t down) {
  if ((up | down) == 0u) return;
#pragma unroll 1
  for (int k = 0; k < 8; ++k) {
    float x = __uint_as_float(static_cast<uint32_t>(p[k]) << 16);
    if (up >> k & 1u) x += INFINITY;
    if (down >> k & 1u) x -= INFINITY;
    p[k] = static_cast<uint16_t>(tc::bf16x2(x, 0.0f));
  }
}

// Lists the blocks of all sequences by their key tiles, the most first (in 512
// classes). Most of its time is a launch, barriers and code that is fetched: with
// 1024 threads calls of some units take 0.8 us more. Offsets that decrease or leave
// the tensors: no block, all rows are rest.
template <bool kCausal>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const int32_t* offsets, const int32_t* kv_offsets, int32_t B,
                                                            int32_t N, int32_t M, const Divisor group, Header* header,
                                                            Block* list, int* dev_err) {
  __shared__ int32_t count[kBins];
  __shared__ int32_t most;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  count[tid] = 0;
  if (tid == 0) most = 0;
  tc::griddep_launch_dependents();
  tc::griddep_wait();
  bool bad = false;
  for (int32_t b = tid; b <= B; b += kPlanThreads) bad |= bad_offsets(offsets, kv_offsets, b, N, M);
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      *header = Header{0, 0, 0};
      atomicExch(dev_err, kDevErrOffsets);
    }
    return;
  }
  const auto block = [&](int32_t b, int32_t p) { return block_of(offsets, kv_offsets, b, p, group, 2); };
  const auto blocks = [&](int32_t b) { return blocks_of(offsets, b, group.d, 2); };
  const auto cost = [&](const Block& e) { return max(key_tiles<kCausal>(e, 0), key_tiles<kCausal>(e, 1)); };
  for (int32_t b = tid; b < B; b += kPlanThreads) {
    const int32_t n = blocks(b);
    if (n > 0) atomicMax(&most, cost(block(b, n - 1)));
  }
  __syncthreads();
  const float scale = static_cast<float>(kBins - 1) / static_cast<float>(max(most, 1));
  const auto bin = [&](const Block& e) { return max(0, kBins - 1 - static_cast<int>(static_cast<float>(cost(e)) * scale)); };
  // threads of a sequence: a power of two, at least a warp
  const int shift = B <= 1 ? 9 : max(5, __clz(B - 1) - 23);
  const int32_t own_b = tid >> shift, own_p = tid & ((1 << shift) - 1);
  for (int32_t b = own_b; b < B; b += kPlanThreads >> shift)
    for (int32_t p = own_p, n = blocks(b); p < n; p += 1 << shift) atomicAdd(&count[bin(block(b, p))], 1);
  __syncthreads();
  // where each class begins: a sum over the classes before it
  const int32_t own = count[tid];
  int32_t sum = own;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int32_t x = __shfl_up_sync(0xffffffffu, sum, s);
    if (lane >= s) sum += x;
  }
  __shared__ int32_t warps[32];
  if (lane == 31) warps[warp] = sum;
  __syncthreads();
  int32_t before = 0;
  for (int w = 0; w < warp; ++w) before += warps[w];
  count[tid] = before + sum - own;
  if (tid == kPlanThreads - 1) *header = Header{before + sum, offsets[0], offsets[B]};
  __syncthreads();
  for (int32_t b = own_b; b < B; b += kPlanThreads >> shift)
    for (int32_t p = own_p, n = blocks(b); p < n; p += 1 << shift) {
      const Block e = block(b, p);
      list[atomicAdd(&count[bin(e)], 1)] = e;
    }
}

// ----------------------------------------------------------------- attention --

template <int D>
struct Smem {
  static constexpr uint32_t kSub = 128 * 128;          // 64 channels of 128 rows
  static constexpr uint32_t kTile = 128 * D * 2;       // 128 rows
  static constexpr int kStages = D == 128 ? 5 : 10;    // key and value tiles in the ring
  static constexpr uint32_t kOffQ = 0;
  static constexpr uint32_t kOffRing = 2 * kTile;
  static constexpr uint32_t kOffBar = kOffRing + kStages * kTile;
  // barriers
  static constexpr int kQFull = 0, kQEmpty = 2, kSFull = 4, kPFull = 6, kOFull = 8, kOEmpty = 10, kDrain = 12;
  static constexpr int kSFree = 14, kPFree = 16;         // P apart from S
  static constexpr int kStat = 18;                       // a tile's sums and maxima are there
  static constexpr int kRaw = 20, kFix = kRaw + kFixes;  // value tiles for warp 3, and units done by it
  static constexpr int kFull = kFix + kFixes, kEmpty = kFull + kStages, kTurn = kEmpty + kStages, kBars = kTurn + 2;
  static constexpr uint32_t kOffTmem = kOffBar + 8 * kBars;
  static constexpr uint32_t kOffAbort = kOffTmem + 4;
  static constexpr uint32_t kOffBad = kOffAbort + 4;   // [kFixes]: kBadSome, kBadAll
  static constexpr uint32_t kOffOdd = kOffBad + 4 * kFixes;  // [kFixes][2][D bits]: channels with +inf, -inf (NaN: both) of all rows
  static constexpr uint32_t kOffStat = (kOffOdd + kFixes * 2 * D / 8 + 7) / 8 * 8;  // [2][128]: l, -c m - 8
  static constexpr uint32_t kOffRedo = kOffStat + 2 * 128 * 8;  // units to do again, and whether there are any
  static constexpr uint32_t kOffBlock = (kOffRedo + 4 * (kRedoWords + 1) + 15) / 16 * 16;  // the CTA's block, and the header, without a list
  static constexpr uint32_t kBytes = kOffBlock + sizeof(Block) + 16;
};
static_assert(Smem<128>::kBytes <= 232448u && Smem<64>::kBytes <= 232448u, "shared memory of one CTA: at most 227 KB");

constexpr uint32_t kTmemCols = 512;
__device__ __forceinline__ uint32_t col_s(int i) { return 128u * static_cast<uint32_t>(i); }
template <int D>
__device__ __forceinline__ uint32_t col_o(int i) { return 256u + static_cast<uint32_t>(D) * static_cast<uint32_t>(i); }
// At D = 64 there are columns left for P beside S: the next S = Q K^T then runs
// under this one's exponentials. At D = 128 P takes the place of S.
template <int D>
constexpr bool kApart = D == 64;
template <int D>
__device__ __forceinline__ uint32_t col_p(int i) { return kApart<D> ? 384u + 64u * static_cast<uint32_t>(i) : col_s(i); }

constexpr uint32_t kCtlRegs = 72, kSoftmaxRegs = 184, kOutRegs = 72;  // 512 threads launched at 128
static_assert(128 * kCtlRegs + 256 * kSoftmaxRegs + 128 * kOutRegs <= kThreads * 128, "registers of one CTA");
static_assert(kOutRegs == kCtlRegs, "every warp runs the teardown with the control registers");

struct Params {
  Divisor Hkv, group;   // key/value heads, and the query heads of one
  const Header* header;
  const Block* list;    // null: no list, a unit for each CTA
  int pair;             // tiles of a block
  const int32_t *offsets, *kv_offsets;
  int32_t B, M;
  float* parts;         // [CTA][2][128][kPart], for units of more than kFold key tiles
  Out out;
  const uint16_t* v;
  int64_t v_ss, v_sh;
  float* lse;
  int64_t N;
  bool zero_rest;
  bool wide_out;        // rows of out begin at whole sectors (32 bytes)
  float scale;          // c
  int* dev_err;
  uint64_t wait_ns;     // limit of a wait
};

__device__ __forceinline__ Block load_block(const Block* list, int32_t e) {
  const int4* p = reinterpret_cast<const int4*>(list + e);
  const int4 x = p[0], y = p[1];
  return Block{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
}

// The CTA's units one after another; the next one's block is brought to L1 a unit ahead.
// Unit u is one of the list's blocks and a head, heads innermost; the CTAs take
// them in that order forth and back.
struct Units {
  const Params& prm;
  const Block* list;
  int32_t units, u, step, other;
  Block e;
  int32_t hk;            // key/value head
  uint32_t number;       // of the unit among the CTA's
  const uint32_t* redo;  // the units to take (a bit for each number modulo 32 kRedoWords), or null: all
  __device__ __forceinline__ Units(const Params& p, const Block* l, int32_t n, const uint32_t* r)
      : prm(p), list(l), units(n), number(0), redo(r) {
    const int32_t g = static_cast<int32_t>(gridDim.x), c = static_cast<int32_t>(blockIdx.x);
    u = c;
    step = 2 * (g - 1 - c) + 1;
    other = 2 * c + 1;
    if (!taken()) advance();
    else load();
  }
  __device__ __forceinline__ bool taken() const {
    return redo == nullptr || (redo[number / 32u % kRedoWords] >> (number & 31u) & 1u) != 0;
  }
  __device__ __forceinline__ bool valid() const { return u < units; }
  __device__ __forceinline__ int32_t head(int t) const { return hk * prm.group.d + (t == 0 ? e.g0 : e.g1); }
  __device__ __forceinline__ void load() {
    if (u >= units) return;
    const int32_t b = prm.Hkv.of(u);
    e = load_block(list, b);
    hk = u - b * prm.Hkv.d;
    const int32_t next = u + step;
    if (next < units) asm volatile("prefetch.global.L1 [%0];" ::"l"(list + prm.Hkv.of(next)));
  }
  __device__ __forceinline__ void advance() {
    do {
      u += step;
      const int32_t s = step;
      step = other;
      other = s;
      ++number;
    } while (u < units && !taken());
    load();
  }
};

// One key tile of the softmax for the thread's query row of tile t: S into
// registers, the maximum, P. lim: keys of the tile that the row sees. pv: products
// with V of the query tile before this one. (One copy of the code for tiles with
// and without hidden keys, and everything that runs once in a unit in small loops:
// code that has not run for a while comes from far, 5000 cycles a time as it was.)
template <int D>
__device__ __forceinline__ bool softmax_tile(const tc::Waits& w, int t, uint32_t tS, uint32_t tP, uint32_t tO, float c,
                                             int lim, bool first, uint32_t pv, float& m, float& neg, float& l) {
  using L = Smem<D>;
  uint32_t s[4][32];
#pragma unroll
  for (int b = 0; b < 4; ++b) tc::tmem_ld32(tS + 32u * b, s[b]);
  tc::tmem_wait_ld();
  if (kApart<D>) {
    tc::tc_fence_before();
    tc::mbar_arrive(w.bar(L::kSFree + t));
  }
  if (__any_sync(0xffffffffu, lim < kKeys)) {
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (32 * b + k >= lim) s[b][k] = 0xFF800000u;  // -inf
  }
  float mx[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    mx[b] = __uint_as_float(s[b][0]);
#pragma unroll
    for (int k = 1; k < 31; k += 2) mx[b] = tc::max3(mx[b], __uint_as_float(s[b][k]), __uint_as_float(s[b][k + 1]));
    mx[b] = fmaxf(mx[b], __uint_as_float(s[b][31]));
  }
  const float up = fmaxf(tc::max3(mx[0], mx[1], mx[2]), mx[3]);
  if (kApart<D> && pv > 0) {
    if (!tc::wait_bar_warp(w, w.bar(L::kPFree + t), (pv - 1) & 1u)) return false;
    tc::tc_fence_after();
  }
  // neg = -m c - 8: a weight would be above 1; with m = -inf whenever the row has seen a key
  if (__any_sync(0xffffffffu, fmaf(up, c, neg) > 0.0f || (m == -INFINITY && up != -INFINITY))) {
    const float m_new = fmaxf(m, up);
    const float neg_new = m_new == -INFINITY ? 0.0f : fmaf(-m_new, c, -kGrowth);
    if (!first) {
      // a row that had seen nothing has O = 0 and l = 0 (as they are in a new part)
      const float alpha = m == -INFINITY ? 0.0f : tc::exp2_approx(neg_new - neg);
      l *= alpha;
      const float2 a2 = make_float2(alpha, alpha);
#pragma unroll 1
      for (int x = 0; x < D / 16; ++x) {
        uint32_t o[16];
        tc::tmem_ld16(tO + 16u * x, o);
        tc::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          const float2 r = __fmul2_rn(make_float2(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), a2);
          o[k] = __float_as_uint(r.x);
          o[k + 1] = __float_as_uint(r.y);
        }
        tc::tmem_st16(tO + 16u * x, o);
      }
    }
    m = m_new;
    neg = neg_new;
  }
  const float2 c2 = make_float2(c, c), n2 = make_float2(neg, neg);
  float2 sa = make_float2(0.f, 0.f), sb = make_float2(0.f, 0.f);
  uint32_t p[4][16];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      const float2 x01 = __ffma2_rn(make_float2(__uint_as_float(s[b][k]), __uint_as_float(s[b][k + 1])), c2, n2);
      const float2 x23 = __ffma2_rn(make_float2(__uint_as_float(s[b][k + 2]), __uint_as_float(s[b][k + 3])), c2, n2);
      const float2 p01 = make_float2(tc::exp2_approx(x01.x), tc::exp2_approx(x01.y));
      const float2 p23 = make_float2(tc::exp2_approx(x23.x), tc::exp2_approx(x23.y));
      sa = __fadd2_rn(sa, p01);
      sb = __fadd2_rn(sb, p23);
      p[b][k / 2] = tc::bf16x2(p01.x, p01.y);
      p[b][k / 2 + 1] = tc::bf16x2(p23.x, p23.y);
    }
    tc::tmem_st16(tP + 16u * b, p[b]);
  }
  l += (sa.x + sa.y) + (sb.x + sb.y);
  tc::tmem_wait_st();
  tc::tc_fence_before();
  tc::mbar_arrive(w.bar(L::kPFull + t));
  return true;
}

// A row's parts in the workspace: sums of values [D], of weights, and what they are
// taken to (neg of that time; inf: the row had seen nothing, the factor to any later one is 0).
template <int D>
constexpr int kPart = D + 4;
// O goes to the parts (`none`: the unit's first time), and l.
template <int D>
__device__ __forceinline__ void fold(float* part, uint32_t tO, bool none, float m, float neg, float l) {
  const float scale = none ? 0.0f : tc::exp2_approx(neg - part[D + 1]);
  part[D] = none ? l : fmaf(part[D], scale, l);
  part[D + 1] = m == -INFINITY ? INFINITY : neg;
#pragma unroll 1
  for (int x = 0; x < D / 16; ++x) {
    uint32_t o[16];
    tc::tmem_ld16(tO + 16u * x, o);
    tc::tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      float* at = part + 16 * x + k;
      *at = none ? __uint_as_float(o[k]) : fmaf(*at, scale, __uint_as_float(o[k]));
    }
  }
}
// And back, on top of what O holds by now; returns l.
template <int D>
__device__ __forceinline__ float unfold(const float* part, uint32_t tO, float neg, float l) {
  const float scale = tc::exp2_approx(neg - part[D + 1]);
#pragma unroll 1
  for (int x = 0; x < D / 16; ++x) {
    uint32_t o[16];
    tc::tmem_ld16(tO + 16u * x, o);
    tc::tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(fmaf(part[16 * x + k], scale, __uint_as_float(o[k])));
    tc::tmem_st16(tO + 16u * x, o);
  }
  tc::tmem_wait_st();
  return fmaf(part[D], scale, l);
}

// kLong: units may have more than kFold key tiles.
template <int D, bool kCausal, bool kLong>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const Params prm) {
  using L = Smem<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((tc::smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicExch(prm.dev_err, kDevErrSmemAlign);
    return;
  }
  const uint32_t sbase = tc::smem_u32(smem);
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  const tc::Waits w{sbase + L::kOffBar, reinterpret_cast<volatile int*>(smem + L::kOffAbort), prm.dev_err, prm.wait_ns};
  volatile uint32_t* bad_units = reinterpret_cast<volatile uint32_t*>(smem + L::kOffBad);
  uint32_t* odd_channels = reinterpret_cast<uint32_t*>(smem + L::kOffOdd);
  uint32_t* redo = reinterpret_cast<uint32_t*>(smem + L::kOffRedo);
  if (threadIdx.x == 0) {
    *w.abort_flag = 0;
    for (uint32_t i = 0; i <= kRedoWords; ++i) redo[i] = 0;
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(w.bar(L::kQFull + i), 1);
      tc::mbar_init(w.bar(L::kQEmpty + i), 1);
      tc::mbar_init(w.bar(L::kSFull + i), 1);
      tc::mbar_init(w.bar(L::kPFull + i), 128);
      tc::mbar_init(w.bar(L::kOFull + i), 1);
      tc::mbar_init(w.bar(L::kOEmpty + i), 128);
      tc::mbar_init(w.bar(L::kDrain + i), 1);
      tc::mbar_init(w.bar(L::kSFree + i), 128);
      tc::mbar_init(w.bar(L::kPFree + i), 1);
      tc::mbar_init(w.bar(L::kStat + i), 128);
    }
    for (int i = 0; i < 2; ++i) tc::mbar_init(w.bar(L::kTurn + i), 1);
    for (int i = 0; i < 2 * kFixes; ++i) tc::mbar_init(w.bar(L::kRaw + i), 1);
    for (int i = 0; i < L::kStages; ++i) {
      tc::mbar_init(w.bar(L::kFull + i), 1);
      tc::mbar_init(w.bar(L::kEmpty + i), 2);
    }
    tc::fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(sbase + L::kOffTmem, kTmemCols);
    tc::tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tc::prefetch_tmap(&tm_q);
    tc::prefetch_tmap(&tm_k);
    tc::prefetch_tmap(&tm_v);
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::kOffTmem);
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  // Few units: no list is made beforehand, each CTA looks its own up.
  Block* own_block = reinterpret_cast<Block*>(smem + L::kOffBlock);
  Header* own_header = reinterpret_cast<Header*>(own_block + 1);
  const bool direct = prm.list == nullptr;
  if (direct) {
    if (warp == 0) {
      const int32_t N = static_cast<int32_t>(prm.N), B = prm.B;
      bool bad = false;
      for (int32_t b = lane; b <= B; b += 32) bad |= bad_offsets(prm.offsets, prm.kv_offsets, b, N, prm.M);
      bad = __any_sync(0xffffffffu, bad);
      if (bad && lane == 0 && blockIdx.x == 0) atomicExch(prm.dev_err, kDevErrOffsets);
      if (lane == 0) *own_header = bad ? Header{0, 0, 0} : Header{0, prm.offsets[0], prm.offsets[B]};
      __syncwarp();
      int32_t before = 0;
      const int32_t mine = prm.Hkv.of(static_cast<int32_t>(blockIdx.x));
      for (int32_t b0 = 0; !bad && b0 < B && before <= mine; b0 += 32) {
        const int32_t b = b0 + lane, n = b < B ? blocks_of(prm.offsets, b, prm.group.d, prm.pair) : 0;
        int32_t sum = n;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
          const int32_t x = __shfl_up_sync(0xffffffffu, sum, s);
          if (lane >= s) sum += x;
        }
        const int32_t p = mine - (before + sum - n);
        if (p >= 0 && p < n) {
          *own_block = block_of(prm.offsets, prm.kv_offsets, b, p, prm.group, prm.pair);
          own_header->blocks = 1;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
      }
    }
    __syncthreads();
  }
  const Block* list = direct ? own_block - prm.Hkv.of(static_cast<int32_t>(blockIdx.x)) : prm.list;
  const Header* header = direct ? own_header : prm.header;
  const int32_t units = direct ? (header->blocks != 0 ? static_cast<int32_t>(blockIdx.x) + 1 : 0) : header->blocks * prm.Hkv.d;

  // After the units: whether some have to be done again. All warps meet here once.
  const auto again = [&]() {
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
    return reinterpret_cast<volatile uint32_t*>(redo)[kRedoWords] != 0;
  };
  if (warp < 4) {
    tc::regs_dec<kCtlRegs>();
    if (warp == 0) {
      // -------------------------------------------------------------- copies --
      uint32_t at = 0, q_cnt[2] = {0, 0}, fixes = 0;  // ring position, queries loaded, tiles for warp 3
      int32_t raw[L::kStages];                          // of the stage's tile: its number among those, or -1
      bool ok = true;
      for (int pass = 0; pass < 2; ++pass) {
        if (pass > 0 && !again()) break;
        for (Units it(prm, list, lane == 0 ? units : 0, pass > 0 ? redo : nullptr); ok && it.valid(); it.advance()) {
          const Block& e = it.e;
          const int32_t hk = it.hk;
          const int32_t n0 = key_tiles<kCausal>(e, 0), n1 = key_tiles<kCausal>(e, 1), n = max(n0, n1);
          const auto queries = [&](int t) {
            if (!(ok = wait_bar(w, w.bar(L::kQEmpty + t), (q_cnt[t] & 1u) ^ 1u))) return;
            ++q_cnt[t];
            tc::mbar_arrive_expect_tx(w.bar(L::kQFull + t), L::kTile);
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
              tc::tma_load_3d(sbase + L::kOffQ + t * L::kTile + x * L::kSub, &tm_q, 64 * x, it.head(t), e.q0 + begin_of(e, t),
                              w.bar(L::kQFull + t));
          };
          const auto tile = [&](const void* map, int32_t j, bool through) {
            const uint32_t st = at % L::kStages;
            if (!(ok = wait_bar(w, w.bar(L::kEmpty + static_cast<int>(st)), ((at / L::kStages) & 1u) ^ 1u))) return;
            ++at;
            raw[st] = through ? static_cast<int32_t>(fixes % (2 * kFixes)) : -1;
            const uint32_t full = w.bar(through ? L::kRaw + static_cast<int>(fixes++ % kFixes) : L::kFull + static_cast<int>(st));
            tc::mbar_arrive_expect_tx(full, L::kTile);
#pragma unroll
            for (int x = 0; x < D / 64; ++x)
              tc::tma_load_3d(sbase + L::kOffRing + st * L::kTile + x * L::kSub, map, 64 * x, hk, e.kv0 + j * kKeys, full);
          };
          // the first keys and values come before the queries, for which the unit
          // before has to be through with its own
          for (int32_t j = 0; ok && j < n; ++j) {
            tile(&tm_k, j, false);
            if (ok) tile(&tm_v, j, pass > 0);  // (in the second pass through warp 3)
            if (j == 0) {
              if (ok && n0 > 0) queries(0);
              if (ok && n1 > 0) queries(1);
              // the next unit's queries on their way to L2
              const int32_t next = it.u + it.step;
              if (next < units) {
                const int32_t b = prm.Hkv.of(next);
                const Block f = load_block(list, b);
                const int32_t h = (next - b * prm.Hkv.d) * prm.group.d;
                for (int t = 0; t < 2 && rows_of(f, t) > 0; ++t)
#pragma unroll
                  for (int x = 0; x < D / 64; ++x)
                    tc::tma_prefetch_3d(&tm_q, 64 * x, h + (t == 0 ? f.g0 : f.g1), f.q0 + begin_of(f, t));
              }
            }
          }
        }
      }
      if (lane == 0) {
        if (!ok) {
          // every copy that this thread issued lands before the CTA exits
          const tc::Waits d = w.draining();
          for (int t = 0; t < 2; ++t)
            if (q_cnt[t] > 0) wait_bar(d, w.bar(L::kQFull + t), (q_cnt[t] - 1) & 1u);
          for (uint32_t p = at < L::kStages ? 0 : at - L::kStages; p < at; ++p) {
            const int32_t f = raw[p % L::kStages];
            if (f < 0) wait_bar(d, w.bar(L::kFull + static_cast<int>(p % L::kStages)), (p / L::kStages) & 1u);
            else wait_bar(d, w.bar(L::kRaw + f % kFixes), static_cast<uint32_t>(f / kFixes) & 1u);
          }
        }
      }
    } else if (warp <= 2) {
      // ------------------------------------------------ products of tile t --
      // The two query tiles' products take turns: issued side by side, they share the
      // tensor pipe and end together, and then both softmaxes run at once and the pipe
      // stands still. Tile 1's product with value tile j (and S of the next key tile)
      // comes after tile 0's with j, and tile 0's next one, of this unit or the next with
      // two tiles, after it. (Tile 1 has as many key tiles as tile 0, or one more, or
      // none at all.) So each of the two barriers is never more than a phase ahead of
      // who waits for it.
      const int t = warp - 1;
      const bool leader = tc::elect_one();
      const uint32_t d_s = tmem + col_s(t), d_p = tmem + col_p<D>(t), d_o = tmem + col_o<D>(t);
      const uint64_t dq = tc::sw128_desc(sbase + L::kOffQ + static_cast<uint32_t>(t) * L::kTile);
      const uint64_t dk0 = tc::sw128_desc(sbase + L::kOffRing), dv0 = tc::sw128_mn_desc(sbase + L::kOffRing, L::kSub);
      // ring position of the unit's first tile; queries, S, P, units with keys, the other tile's turns so far
      uint32_t base = 0, q_cnt = 0, s_cnt = 0, p_cnt = 0, done = 0, turns = 0;
      const auto full = [&](uint32_t p) {
        return wait_bar_warp(w, w.bar(L::kFull + static_cast<int>(p % L::kStages)), (p / L::kStages) & 1u);
      };
      const auto empty = [&](uint32_t p) { return w.bar(L::kEmpty + static_cast<int>(p % L::kStages)); };
      // S of the key tile at ring position p
      const auto wait_s = [&](uint32_t p) {
        if (!full(p)) return false;
        if (kApart<D> && s_cnt > 0 && !wait_bar_warp(w, w.bar(L::kSFree + t), (s_cnt - 1) & 1u)) return false;
        ++s_cnt;
        return true;
      };
      const auto product_s = [&](uint32_t p, bool last) {
        const uint64_t dk = tc::desc_at(dk0, (p % L::kStages) * L::kTile);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = static_cast<uint32_t>(ks >> 2) * L::kSub + static_cast<uint32_t>(ks & 3) * 32u;
          tc::mma_f16_ss(d_s, tc::desc_at(dq, off), tc::desc_at(dk, off), tc::IdescBf16<kKeys>::value, ks > 0 ? 1u : 0u);
        }
        tc::mma_commit(w.bar(L::kSFull + t));
        tc::mma_commit(empty(p));
        if (last) tc::mma_commit(w.bar(L::kQEmpty + t));
      };
      bool ok = true;
      int pass = 0;
    units_of_tile:
      for (Units it(prm, list, units, pass > 0 ? redo : nullptr); ok && it.valid(); it.advance()) {
        const Block& e = it.e;
        const int32_t own = key_tiles<kCausal>(e, t), theirs = key_tiles<kCausal>(e, 1 - t), n = max(own, theirs);
        if (own > 0) {
          if (!(ok = wait_bar_warp(w, w.bar(L::kQFull + t), q_cnt & 1u)) || !(ok = wait_s(base))) break;
          ++q_cnt;
          tc::tc_fence_after();
          if (leader) product_s(base, own == 1);
          __syncwarp();
        }
        for (int32_t j = 0; j < n; ++j) {
          const uint32_t pk = base + 2u * static_cast<uint32_t>(j), pv = pk + 1u;
          const bool more = j + 1 < own;
          if (kApart<D> && more) {
            if (!(ok = wait_s(pk + 2u))) break;
            tc::tc_fence_after();
            if (leader) product_s(pk + 2u, j + 2 == own);
            __syncwarp();
          }
          if (!(ok = full(pv))) break;
          // the output warps are through with the unit before
          if (j == 0 && !(ok = wait_bar_warp(w, w.bar(L::kOEmpty + t), (done & 1u) ^ 1u))) break;
          if (j < own) {
            if (!kApart<D> && more && !(ok = wait_s(pk + 2u))) break;
            // the keys' part of the tile, in steps of 16
            const int steps = (min(kKeys, e.keys - j * kKeys) + 15) >> 4;
            const uint64_t dv = tc::desc_at(dv0, (pv % L::kStages) * L::kTile);
            if (!(ok = wait_bar_warp(w, w.bar(L::kPFull + t), p_cnt & 1u))) break;
            ++p_cnt;
            const bool turn = j < theirs;
            if (turn) {
              const uint32_t before = turns++ + static_cast<uint32_t>(t);  // the other's turns that this one comes after
              if (before > 0 && !(ok = wait_bar_warp(w, w.bar(L::kTurn + 1 - t), (before - 1) & 1u))) break;
            }
            tc::tc_fence_after();
            if (leader) {
#pragma unroll
              for (int ks = 0; ks < kKeys / 16; ++ks)
                if (ks < steps)
                  tc::mma_f16_ts(d_o, d_p + 8u * ks, tc::desc_at(dv, 2048u * ks), tc::IdescBf16<D, true>::value,
                                 ((kLong ? (j & (kFold - 1)) != 0 : j > 0) || ks > 0) ? 1u : 0u);
              if (!kApart<D> && more) product_s(pk + 2u, j + 2 == own);
              tc::mma_commit(empty(pv));
              if (kApart<D>) tc::mma_commit(w.bar(L::kPFree + t));
              if (turn) {
                if (kApart<D>) tc::mbar_arrive(w.bar(L::kTurn + t));  // issued
                else tc::mma_commit(w.bar(L::kTurn + t));             // done
              }
              if (!more) tc::mma_commit(w.bar(L::kOFull + t));
            }
          } else {
            // a key tile that only the other query tile sees
            if (!(ok = full(pk))) break;
            if (leader) {
              tc::mbar_arrive(empty(pk));
              tc::mbar_arrive(empty(pv));
              if (own == 0 && j == 0) tc::mbar_arrive(w.bar(L::kOFull + t));
            }
          }
          __syncwarp();
        }
        if (n > 0) ++done;
        base += 2u * static_cast<uint32_t>(n);
      }
      if (pass++ == 0 && again()) goto units_of_tile;
      // all products are done before TMEM is freed
      if (leader) tc::mma_commit(w.bar(L::kDrain + t));
      __syncwarp();
      wait_bar(w.draining(), w.bar(L::kDrain + t), 0);
    } else {
      // ------------------------------------------ value tiles of the second pass --
      // (the ring goes on from the first)
      uint32_t base = 0, fixes = 0, done = 0;
      bool ok = true;
      const int32_t second = again() ? units : 0;
      for (Units it(prm, list, second, nullptr); it.valid(); it.advance())
        base += 2u * static_cast<uint32_t>(max(key_tiles<kCausal>(it.e, 0), key_tiles<kCausal>(it.e, 1)));
      for (Units it(prm, list, second, redo); ok && it.valid(); it.advance()) {
        const Block& e = it.e;
        const int32_t n = max(key_tiles<kCausal>(e, 0), key_tiles<kCausal>(e, 1));
        const int32_t whole = kCausal ? sees<kCausal>(e, 0) >> 7 : n;  // tiles whose keys all rows see
        uint32_t* odd = odd_channels + done % kFixes * (2 * D / 32);
        uint32_t bad = 0;
        for (int32_t j = 0; j < n; ++j) {
          const uint32_t p = base + 2u * static_cast<uint32_t>(j) + 1u;
          if (!(ok = wait_bar_warp(w, w.bar(L::kRaw + static_cast<int>(fixes % kFixes)), (fixes / kFixes) & 1u))) break;
          // (this tile is there, so the output warps are done with the unit eight before)
          if (j == 0 && lane < 2 * D / 32) odd[lane] = 0;
          __syncwarp();
          uint8_t* tile = smem + L::kOffRing + (p % L::kStages) * L::kTile;
          const int32_t there = min(kKeys, e.keys - j * kKeys);
          // rows of 128 bytes: row r of the 64 channels x at r * 128 + x * kSub
          for (int x = 0; x < D / 64; ++x) {
            uint4* chunk = reinterpret_cast<uint4*>(tile + x * L::kSub);
            uint32_t acc[4] = {0u, 0u, 0u, 0u};
#pragma unroll 8
            for (int q = lane; q < there * 8; q += 32) {
              const uint4 v = chunk[q];
              acc[0] = collect(v.x, acc[0]);
              acc[1] = collect(v.y, acc[1]);
              acc[2] = collect(v.z, acc[2]);
              acc[3] = collect(v.w, acc[3]);
            }
            if (__any_sync(0xffffffffu, not_finite(acc[0]) | not_finite(acc[1]) | not_finite(acc[2]) | not_finite(acc[3]))) {
              bad |= j < whole ? kBadAll : kBadSome;
              // (swizzled: the chunk q & 7 of a row has channels 8 ((q ^ row) & 7) on, which are two
              // places for a lane, whose rows are 4 apart)
              uint32_t up[2] = {0u, 0u}, down[2] = {0u, 0u};
#pragma unroll 1
              for (int q = lane; q < there * 8; q += 64) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  if (q + 32 * y >= there * 8) continue;
                  uint4 u = chunk[q + 32 * y];
                  take_odd(u, up[y], down[y]);
                  chunk[q + 32 * y] = u;
                }
              }
              if (j < whole) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const int c0 = 64 * x + 8 * ((lane ^ ((lane >> 3) + 4 * y)) & 7);
                  if (up[y] != 0u) atomicOr(odd + c0 / 32, up[y] << (c0 & 31));
                  if (down[y] != 0u) atomicOr(odd + D / 32 + c0 / 32, down[y] << (c0 & 31));
                }
              }
            }
            for (int q = there * 8 + lane; q < kKeys * 8; q += 32) chunk[q] = make_uint4(0, 0, 0, 0);
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(w.bar(L::kFull + static_cast<int>(p % L::kStages)));
          ++fixes;
        }
        if (ok && n > 0) {
          if (lane == 0) {
            bad_units[done % kFixes] = bad;
            tc::mbar_arrive(w.bar(L::kFix + static_cast<int>(done % kFixes)));
          }
          __syncwarp();
          ++done;
        }
        base += 2u * static_cast<uint32_t>(n);
      }
    }
    __syncwarp();
  } else if (warp < 12) {
    // ----------------------------------------------------------------- softmax --
    tc::regs_inc<kSoftmaxRegs>();
    const int t = (warp - 4) >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + col_s(t), tP = tmem + lanes + col_p<D>(t), tO = tmem + lanes + col_o<D>(t);
    uint32_t s_cnt = 0, done = 0;
    float2* stat = reinterpret_cast<float2*>(smem + L::kOffStat) + 128 * t + row;
    const auto part = [&]() { return prm.parts + ((static_cast<int64_t>(blockIdx.x) * 2 + t) * kRows + row) * kPart<D>; };
    bool ok = true;
    int pass = 0;
  units_of_rows:
    for (Units it(prm, list, units, pass > 0 ? redo : nullptr); ok && it.valid(); it.advance()) {
      const Block& e = it.e;
      const int32_t own = key_tiles<kCausal>(e, t), n = max(own, key_tiles<kCausal>(e, 1 - t));
      const int32_t mine = sees<kCausal>(e, begin_of(e, t) + row);
      float m = -INFINITY, neg = 0.0f, l = 0.0f;
      for (int32_t j = 0, end = kLong ? min(own, kFold) : own;;) {
        for (const int32_t first = j; j < end; ++j) {
          if (!(ok = wait_bar_warp(w, w.bar(L::kSFull + t), s_cnt & 1u))) break;
          tc::tc_fence_after();
          if (!(ok = softmax_tile<D>(w, t, tS, tP, tO, prm.scale, mine - j * kKeys, j == first, s_cnt, m, neg, l))) break;
          ++s_cnt;
        }
        if (!kLong || !ok || end == own) break;
        // O begins anew, once the products with V so far are done (at D = 128 the next S comes after them)
        if (!(ok = kApart<D> ? wait_bar_warp(w, w.bar(L::kPFree + t), (s_cnt - 1) & 1u)
                             : wait_bar_warp(w, w.bar(L::kSFull + t), s_cnt & 1u)))
          break;
        tc::tc_fence_after();
        fold<D>(part(), tO, j == kFold, m, neg, l);
        l = 0.0f;
        end = min(own, end + kFold);
      }
      if (kLong && ok && own > kFold) {
        if (!(ok = wait_bar_warp(w, w.bar(L::kOFull + t), done & 1u))) break;
        tc::tc_fence_after();
        l = unfold<D>(part(), tO, neg, l);
        tc::tc_fence_before();
      }
      if (ok && n > 0) {
        // the unit before has been stored (waited for in every unit: no phase is skipped)
        if (!(ok = wait_bar_warp(w, w.bar(L::kOEmpty + t), (done & 1u) ^ 1u))) break;
        ++done;
        if (own > 0) {
          *stat = make_float2(l, neg);
          tc::mbar_arrive(w.bar(L::kStat + t));
        }
      }
    }
    if (pass++ == 0 && again()) goto units_of_rows;
    tc::regs_dec<kCtlRegs>();
  } else {
    // ------------------------------------------------------------------ output --
    // O is read, scaled and stored by warps of its own: the softmax goes on with the
    // next unit.
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    tc::regs_dec<kOutRegs>();
    if (prm.zero_rest) {
      const int32_t lo = header->rest_lo, hi = header->rest_hi;
      // a row's head at a time for D / 8 threads
      const int at = static_cast<int>(threadIdx.x) - 384, c = at % (D / 8);
      const int64_t rest = lo + (prm.N - hi), heads = prm.Hkv.d * prm.group.d, items = rest * heads, step = static_cast<int64_t>(gridDim.x) * (128 / (D / 8));
      for (int64_t x = static_cast<int64_t>(blockIdx.x) * (128 / (D / 8)) + at / (D / 8); x < items; x += step) {
        const int64_t i = x / heads, h = x - i * heads, r = i < lo ? i : hi + (i - lo);
        *reinterpret_cast<uint4*>(prm.out.p + r * prm.out.ss + h * prm.out.sh + 8 * c) = make_uint4(0, 0, 0, 0);
        if (c == 0 && prm.lse != nullptr) prm.lse[h * prm.N + r] = -INFINITY;
      }
    }
    uint32_t fixed = 0, done = 0, stats[2] = {0, 0};  // (fixed: units of the second pass with keys)
    bool ok = true;
    int pass = 0;
  units_of_output:
    for (Units it(prm, list, units, pass > 0 ? redo : nullptr); ok && it.valid(); it.advance()) {
      const Block& e = it.e;
      const int32_t n0 = key_tiles<kCausal>(e, 0), n1 = key_tiles<kCausal>(e, 1), n = max(n0, n1);
      uint32_t bad = 0;  // infinities and NaN that warp 3 has cleared
      if (pass > 0 && n > 0) {
        if (!(ok = wait_bar_warp(w, w.bar(L::kFix + static_cast<int>(fixed % kFixes)), (fixed / kFixes) & 1u))) break;
        bad = bad_units[fixed % kFixes];
      }
      uint32_t met = 0;  // infinities and NaN among the outputs
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        const int32_t own = t == 0 ? n0 : n1, r = begin_of(e, t) + row, h = it.head(t);
        float2 st = make_float2(0.0f, 0.0f);
        if (own > 0) {
          uint32_t& c = stats[t];
          if (!(ok = wait_bar_warp(w, w.bar(L::kStat + t), c & 1u))) break;
          ++c;
          st = reinterpret_cast<const float2*>(smem + L::kOffStat)[128 * t + row];
        }
        if (n > 0 && !(ok = wait_bar_warp(w, w.bar(L::kOFull + t), done & 1u))) break;
        tc::tc_fence_after();
        if (rows_of(e, t) <= 0) {
          if (n > 0) tc::mbar_arrive(w.bar(L::kOEmpty + t));
          continue;
        }
        const float inv = st.x == 0.0f ? 0.0f : 1.0f / st.x;
        const bool there = row < rows_of(e, t);
        if (prm.lse != nullptr && there)
          prm.lse[static_cast<int64_t>(h) * prm.N + e.q0 + r] = st.x == 0.0f ? -INFINITY : (log2f(st.x) - st.y) * kLn2;
        uint16_t* dst = prm.out.p + (static_cast<int64_t>(e.q0) + r) * prm.out.ss + h * prm.out.sh;
        // 16 channels at a time, a whole sector for each lane's store: little code
#pragma unroll 1
        for (int x = 0; x < D / 16; ++x) {
          uint32_t o[16], c[8], acc[2] = {0u, 0u};
          tc::tmem_ld16(tmem + lanes + col_o<D>(t) + 16u * static_cast<uint32_t>(x), o);
          tc::tmem_wait_ld();
          if (x == D / 16 - 1 && n > 0) {
            tc::tc_fence_before();
            tc::mbar_arrive(w.bar(L::kOEmpty + t));
          }
          const float2 inv2 = make_float2(inv, inv);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 y = __fmul2_rn(make_float2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1])), inv2);
            c[k] = tc::bf16x2(y.x, y.y);
            acc[k & 1] = collect(c[k], acc[k & 1]);
          }
          if (own == 0) {  // (O is not this unit's)
#pragma unroll
            for (int k = 0; k < 8; ++k) c[k] = 0u;
          }
          if (there) {
            if (own > 0) met |= not_finite(acc[0]) | not_finite(acc[1]);
            if (prm.wide_out) {
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 16 * x), "r"(c[0]), "r"(c[1]),
                           "r"(c[2]), "r"(c[3]), "r"(c[4]), "r"(c[5]), "r"(c[6]), "r"(c[7])
                           : "memory");
            } else {
              *reinterpret_cast<uint4*>(dst + 16 * x) = make_uint4(c[0], c[1], c[2], c[3]);
              *reinterpret_cast<uint4*>(dst + 16 * x + 8) = make_uint4(c[4], c[5], c[6], c[7]);
            }
          }
        }
        if (__builtin_expect(bad != 0 && there, 0)) {
          const uint32_t* odd = odd_channels + fixed % kFixes * (2 * D / 32);
          const uint16_t* v = prm.v + static_cast<int64_t>(e.kv0) * prm.v_ss + it.hk * prm.v_sh;
          const int32_t from = (sees<kCausal>(e, 0) >> 7) * kKeys, mine = sees<kCausal>(e, r);
#pragma unroll 1
          for (int c = 0; c < D; c += 8) {
            uint32_t up = 0u, down = 0u;
            if (bad & kBadAll) {
              up = odd[c / 32] >> (c & 31) & 0xFFu;
              down = odd[D / 32 + c / 32] >> (c & 31) & 0xFFu;
            }
            if (kCausal && (bad & kBadSome)) {
#pragma unroll 1
              for (int32_t k = from; k < mine; ++k) {
                uint4 u = *reinterpret_cast<const uint4*>(v + k * prm.v_ss + c);
                if (not_finite(u) != 0u) take_odd(u, up, down);
              }
            }
            add_odd(dst + c, up, down);
          }
        }
      }
      if (pass == 0 && __any_sync(0xffffffffu, met != 0u)) {
        if (lane == 0) {
          atomicOr(redo + it.number / 32u % kRedoWords, 1u << (it.number & 31u));
          reinterpret_cast<volatile uint32_t*>(redo)[kRedoWords] = 1u;
        }
        __syncwarp();
      }
      if (n > 0) {
        ++done;
        if (pass > 0) ++fixed;
      }
    }
    if (pass++ == 0 && again()) goto units_of_output;
    tc::regs_dec<kCtlRegs>();
  }

  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// Rows of one head of a packed tensor: boxes of 64 channels x 128 rows, 128-byte swizzle.
bool make_map(CUtensorMap* map, const Bf16In& x, int64_t rows, int64_t heads, int64_t D) {
  const uint64_t dims[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(heads), static_cast<uint64_t>(rows)};
  // (strides of one head or row are not used; the tensor map wants valid ones)
  const uint64_t strides[2] = {static_cast<uint64_t>(heads > 1 ? x.sh : D) * 2, static_cast<uint64_t>(rows > 1 ? x.ss : D) * 2};
  const uint32_t box[3] = {64, 1, 128};
  return make_tmap(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, x.p, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

size_t list_bytes(int64_t N, int64_t B, int64_t group) {
  return (kHeaderBytes + static_cast<size_t>(most_blocks(N, B, group, 2)) * sizeof(Block) + 255) / 256 * 256;
}
// Whether a sequence may have more key tiles than O holds.
bool has_parts(int64_t M) { return M > int64_t(kFold) * kKeys; }
// CTAs of a call at most.
int64_t most_ctas(int64_t N, int64_t H, int64_t Hkv, int64_t B) {
  const int64_t units = most_blocks(N, B, H / Hkv, 1) * Hkv;
  return units < kMostCtas ? units : kMostCtas;
}

template <int D>
cudaError_t launch(const PromptArgs& a, cudaStream_t stream) {
  const int64_t rows = a.M > 0 ? a.M : 1;  // a tensor without rows is not read
  CUtensorMap tq, tk, tv;
  if (!make_map(&tq, a.q, a.N, a.H, D) || !make_map(&tk, a.k, rows, a.Hkv, D) || !make_map(&tv, a.v, rows, a.Hkv, D))
    return cudaErrorInvalidValue;
  Header* header = static_cast<Header*>(a.workspace);
  Block* list = reinterpret_cast<Block*>(static_cast<char*>(a.workspace) + kHeaderBytes);
  const int64_t group = a.H / a.Hkv, sms = sm_count_current() < kMostCtas ? sm_count_current() : kMostCtas;
  // (100 tokens, 28 heads: 7.8 us with a tile for each SM, 8.5 with two for 14 of them)
  const int pair = most_blocks(a.N, a.B, group, 1) * a.Hkv <= sms ? 1 : 2;
  const int64_t units = most_blocks(a.N, a.B, group, pair) * a.Hkv;
  // A unit for each CTA at most: no first kernel, which costs more than its list saves
  // then. 100 tokens, 28 heads: 7.8 us, 11.1 with it; 1230 tokens (140 units): 22.6 us, 24.0 with it.
  const bool direct = units <= sms;
  cudaError_t e;
  if (!direct && (e = launch_dependent(a.causal ? plan_kernel<true> : plan_kernel<false>, dim3(1), kPlanThreads, 0, stream,
                                       a.offsets, a.kv_offsets, a.B, static_cast<int32_t>(a.N),
                                       static_cast<int32_t>(a.M), Divisor(static_cast<int32_t>(group)), header, list, a.dev_err)) != cudaSuccess)
    return e;
  Params p{Divisor(a.Hkv), Divisor(static_cast<int32_t>(group))};
  p.pair = pair;
  p.header = header;
  p.list = direct ? nullptr : list;
  p.offsets = a.offsets;
  p.kv_offsets = a.kv_offsets;
  p.B = a.B;
  p.M = static_cast<int32_t>(a.M);
  p.parts = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + list_bytes(a.N, a.B, group));
  p.out = a.out;
  p.v = a.v.p;
  p.v_ss = a.v.ss;
  p.v_sh = a.v.sh;
  p.lse = a.lse;
  p.N = a.N;
  p.zero_rest = a.zero_rest;
  p.wide_out = reinterpret_cast<uintptr_t>(a.out.p) % 32 == 0 && a.out.ss % 16 == 0 && a.out.sh % 16 == 0;
  p.scale = a.sm_log2;
  p.dev_err = a.dev_err;
  p.wait_ns = tc::wait_limit_ns(div_up(a.M, kKeys));
  // The code for parts costs calls that need none 2 to 5% (16 prompts of 1500 tokens 265 -> 270 us, at D = 64 48.6 -> 51):
  // calls with few rows have a kernel without. (48 such prompts, 72000 rows: 811 us with, 782 without.)
  const bool parts = has_parts(a.M);
  const auto kernel = parts ? (a.causal ? prompt_attention_kernel<D, true, true> : prompt_attention_kernel<D, false, true>)
                            : (a.causal ? prompt_attention_kernel<D, true, false> : prompt_attention_kernel<D, false, false>);
  const int bytes = static_cast<int>(Smem<D>::kBytes);
  if ((e = set_smem_limit_once(reinterpret_cast<const void*>(kernel), bytes)) != cudaSuccess) return e;
  const int64_t grid = units < 1 ? 1 : units < sms ? units : sms;
  return launch_dependent(kernel, dim3(static_cast<unsigned>(grid)), kThreads,
                          static_cast<size_t>(bytes), stream, tq, tk, tv, p);
}

}  // namespace

size_t prompt_attention_workspace_bytes(int64_t N, int64_t M, int64_t H, int64_t Hkv, int64_t D, int64_t B) {
  const size_t parts = has_parts(M) ? static_cast<size_t>(most_ctas(N, H, Hkv, B) * 2 * kRows * (D + 4)) * sizeof(float) : 0;
  return list_bytes(N, B, H / Hkv) + parts;
}

cudaError_t launch_prompt_attention(const PromptArgs& a, int64_t D, cudaStream_t stream) {
  return D == 128 ? launch<128>(a, stream) : launch<64>(a, stream);
}

}  // namespace sage
