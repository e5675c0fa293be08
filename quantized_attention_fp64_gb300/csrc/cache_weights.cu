// Attention weights that cached tokens get from a step's queries, few query rows:
//   scores_j += sum over the R = G q_length rows of a key/value head of
//               2^(c s_j (q_r . code_j) - log2(e) lse_r),  c = sm_scale log2 e.
// (Many rows: cache_weights_tc.cu.)
//
// The keys' codes are read once, and with few rows nothing else counts. All
// blocks of 32 keys, of all sequences and heads, form one list that is cut into
// equal ranges, one per warp, whatever the lengths. A warp takes a block with
// 16-byte loads, 512 contiguous bytes each, the next block's in flight under this
// one's products. m16n8k16 in BF16, keys as rows: a lane's 16 codes of a key
// are its share of four products, since the channels may be taken in any order as
// long as the queries are; queries are BF16 already and codes (8 bits with their
// sign) are exact in it. The products' rows are keys, so a key's sum over the
// query rows is one in a lane and two exchanges between four lanes, always in the
// same order. 64 sequences of up to 8192 tokens, 8 key/value heads, D = 128, 4 rows
// each: 51 us, 6.2 TB/s (93% of a copy's rate); 16 rows 64 us, 32 rows 82 us, bound by the
// exponentials' and products' instructions.
#include "cache.cuh"
#include "launch.cuh"
#include "tc_kernel.cuh"

namespace sage {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

// The blocks of a sequence that scores has a place for.
__device__ __forceinline__ int32_t blocks_of(const CacheWeightsArgs& a, int32_t capacity, int b) {
  int32_t n = min(max(a.lengths[b], 0), capacity);
  if (n > a.scores_n) n = static_cast<int32_t>(a.scores_n);
  return n / kCacheBlock + (n % kCacheBlock != 0 ? 1 : 0);
}

// Four codes to two BF16 pairs: 128 + the low seven bits, less 128 or (negative) 256.
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t low = w & 0x7F7F7F7Fu, sign = w & 0x80808080u;
  const uint32_t v0 = __byte_perm(low, 0x43434343u, 0x4140), v1 = __byte_perm(low, 0x43434343u, 0x4342);
  const uint32_t s0 = __byte_perm(sign, 0x43434343u, 0x4140), s1 = __byte_perm(sign, 0x43434343u, 0x4342);
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(v0), "r"(s0));
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(v1), "r"(s1));
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load_codes(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// N: query rows in eights (1, 2, 4).
template <int D, int N>
__global__ void __launch_bounds__(kThreads, N == 4 ? 1 : 2) cache_weights_kernel(const CacheWeightsArgs a) {
  constexpr int kHalves = D / 64, kLoads = 4 * kHalves;
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x) & 31, g = lane >> 2, t4 = lane & 3;
  const int32_t capacity = static_cast<int32_t>(table_capacity(a.pt.max_pages, a.c.blocks_per_page));
  const int B = static_cast<int>(a.B), H = a.c.H, G = a.H / H;
  // all sequences' blocks, and where this warp's range begins
  int64_t total = 0;
  bool bad = false;
  for (int b = lane; b < B; b += 32) {
    total += blocks_of(a, capacity, b);
    const int32_t n = a.lengths[b], r = a.q_lengths != nullptr ? a.q_lengths[b] : 0;
    bad |= n < 0 || n > capacity || r < 0 || r > a.T;
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) total += __shfl_xor_sync(0xffffffffu, total, s);
  total *= H;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  const int64_t me = static_cast<int64_t>(threadIdx.x >> 5) * gridDim.x + blockIdx.x;
  int64_t at = total * me / warps;
  int64_t left = total * (me + 1) / warps - at;
  if (bad && me == 0) atomicExch(a.dev_err, kDevErrPage);
  if (left <= 0) return;
  int b = 0;
  for (int b0 = 0;; b0 += 32) {  // the sequence: the first whose blocks end behind `at`
    const int64_t own = b0 + lane < B ? static_cast<int64_t>(blocks_of(a, capacity, b0 + lane)) * H : 0;
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
    if (b0 + 32 >= B) return;  // (not reached: at < total)
  }
  int32_t blocks = blocks_of(a, capacity, b);
  int h = static_cast<int>(at / blocks);
  int32_t blk = static_cast<int32_t>(at % blocks);

  while (left > 0) {
    // a run of blocks of one head
    const int32_t run = static_cast<int32_t>(left < blocks - blk ? left : blocks - blk);
    const int32_t len = min(min(max(a.lengths[b], 0), capacity), static_cast<int32_t>(min(a.scores_n, int64_t(capacity))));
    const int32_t full_len = min(max(a.lengths[b], 0), capacity);
    const int32_t rows = a.q_lengths != nullptr ? min(max(a.q_lengths[b], 0), static_cast<int32_t>(a.T))
                                                : static_cast<int32_t>(a.T);
    const int R = rows * G;
    if (R > 0) {
      // query row 8n + g: channels 16 t4 .. 16 t4 + 15 of each half
      uint32_t q[N][kHalves][8];
      float lse[N][2];
      int32_t sees[N][2];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int r = 8 * n + g;
#pragma unroll
        for (int x = 0; x < kHalves; ++x) {
          uint4 u = make_uint4(0, 0, 0, 0), v = u;
          if (r < R) {
            const uint16_t* p =
                a.q.p + b * a.q.sb + (r / G) * a.q.ss + static_cast<int64_t>(h * G + r % G) * a.q.sh + 64 * x + 16 * t4;
            u = *reinterpret_cast<const uint4*>(p);
            v = *reinterpret_cast<const uint4*>(p + 8);
          }
          q[n][x][0] = u.x, q[n][x][1] = u.y, q[n][x][2] = u.z, q[n][x][3] = u.w;
          q[n][x][4] = v.x, q[n][x][5] = v.y, q[n][x][6] = v.z, q[n][x][7] = v.w;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = 8 * n + 2 * t4 + e;
          float l = -INFINITY;
          if (c < R) l = a.lse[(static_cast<int64_t>(b) * a.H + h * G + c % G) * a.T + c / G];
          lse[n][e] = -l * kLog2e;
          sees[n][e] = l == -INFINITY ? 0 : (a.causal ? full_len - rows + c / G + 1 : full_len);
        }
      }
      float* scores = a.scores + b * a.scores_b + h * a.scores_h;
      // 32 blocks are looked up at a time, one by each lane
      int64_t slots = -1;
      float scales = 0.0f;
      const auto look_up = [&](int32_t first) {
        const int32_t x = first + lane;
        slots = -1;
        if (x < blk + run) {
          const int32_t in_seq = x / a.c.blocks_per_page;
          const int64_t page = a.pt.table[b * a.pt.stride + in_seq];
          if (page_ok(page, a.c.num_pages)) {
            slots = block_slot(page, h, H, a.c.blocks_per_page, x - in_seq * a.c.blocks_per_page);
            scales = a.c.ks[slots] * a.sm_log2;
          } else {
            atomicExch(a.dev_err, kDevErrPage);
          }
        }
      };
      uint4 next[kLoads];
      int64_t next_slot;
      float next_scale, next_score = 0.0f;
      const int mine = (t4 >> 1) * 16 + (t4 & 1) * 8 + g;  // the key whose sum this lane writes
      const auto fetch = [&](int32_t i) {  // block blk + i
        if ((i & 31) == 0) look_up(blk + i);
        next_slot = __shfl_sync(0xffffffffu, slots, i & 31);
        next_scale = __shfl_sync(0xffffffffu, scales, i & 31);
        if (next_slot >= 0) {
          const int8_t* p = a.c.k + next_slot * (kCacheBlock * D) + lane * 16;
#pragma unroll
          for (int y = 0; y < kLoads; ++y) next[y] = load_codes(p + y * 512);
          const int32_t j = (blk + i) * kCacheBlock + mine;
          if (j < len) next_score = scores[j];
        }
      };
      fetch(0);
      for (int32_t i = 0; i < run; ++i) {
        uint4 code[kLoads];
#pragma unroll
        for (int y = 0; y < kLoads; ++y) code[y] = next[y];
        const int64_t slot = next_slot;
        const float scale = next_scale, score = next_score;
        if (i + 1 < run) fetch(i + 1);
        if (slot < 0) continue;
        const int32_t j0 = (blk + i) * kCacheBlock;
        float sum[4];
#pragma unroll
        for (int m = 0; m < 2; ++m) {  // keys 16 m + g, 16 m + g + 8
          float d[N][4];
#pragma unroll
          for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) d[n][e] = 0.0f;
#pragma unroll
          for (int x = 0; x < kHalves; ++x) {
            const uint4 u = code[4 * x + 2 * m], v = code[4 * x + 2 * m + 1];
            const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              uint32_t f[4];
              codes_to_bf16(uw[s], f[0], f[2]);
              codes_to_bf16(vw[s], f[1], f[3]);
#pragma unroll
              for (int n = 0; n < N; ++n) mma_bf16(d[n], f, q[n][x][2 * s], q[n][x][2 * s + 1]);
            }
          }
          float w0 = 0.0f, w1 = 0.0f;
          const int32_t key = j0 + 16 * m + g;
#pragma unroll
          for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float p0 = tc::exp2_approx(fmaf(d[n][e], scale, lse[n][e]));
              const float p1 = tc::exp2_approx(fmaf(d[n][2 + e], scale, lse[n][e]));
              w0 += key < sees[n][e] ? p0 : 0.0f;
              w1 += key + 8 < sees[n][e] ? p1 : 0.0f;
            }
          sum[2 * m] = w0;
          sum[2 * m + 1] = w1;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
          sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
        }
        const float add = (t4 & 2) ? ((t4 & 1) ? sum[3] : sum[2]) : ((t4 & 1) ? sum[1] : sum[0]);
        if (j0 + mine < len && !(add == 0.0f)) scores[j0 + mine] = score + add;
      }
    }
    left -= run;
    blk += run;
    if (blk == blocks) {
      blk = 0;
      if (++h == H) {
        h = 0;
        do {
          if (++b == B) return;
          blocks = blocks_of(a, capacity, b);
        } while (blocks == 0);
      }
    }
  }
}

}  // namespace

cudaError_t launch_cache_weights(const CacheWeightsArgs& a, int64_t D, cudaStream_t stream) {
  const int64_t most = table_capacity(a.pt.max_pages, a.c.blocks_per_page);
  const int64_t tokens = a.scores_n < most ? a.scores_n : most;
  if (tokens == 0) return cudaSuccess;
  const int64_t rows = a.T * (a.H / a.c.H);
  // Up to 32 rows here, more in cache_weights_tc.cu, which has the products of 128 rows
  // whatever there are: one sequence of 16001 tokens, 8 heads, 32 rows: 12.3 us here,
  // 21 there; 64 sequences up to 8192: 82 us here, 273 there.
  if (rows > 32) return launch_cache_weights_tc(a, D, stream);
  const int64_t blocks = div_up(tokens, kCacheBlock) * a.c.H * a.B;
  const int64_t ctas = div_up(blocks, kThreads / 32), fit = int64_t(sm_count_current()) * (rows > 16 ? 1 : 2);
  const dim3 grid(static_cast<unsigned>(ctas < fit ? ctas : fit));
  const auto kernel = D == 128 ? (rows <= 8 ? cache_weights_kernel<128, 1> : rows <= 16 ? cache_weights_kernel<128, 2> : cache_weights_kernel<128, 4>)
                               : (rows <= 8 ? cache_weights_kernel<64, 1> : rows <= 16 ? cache_weights_kernel<64, 2> : cache_weights_kernel<64, 4>);
  return launch_dependent(kernel, grid, kThreads, 0, stream, a);
}

}  // namespace sage
