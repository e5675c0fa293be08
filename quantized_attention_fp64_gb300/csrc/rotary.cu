// Rotary positions: each pair (a, b) of channels of a token at position p becomes
//   f (a cos x - b sin x, b cos x + a sin x),  x = p w_i.
//
// Angles. w_i comes as the part of a turn that one position adds, in units of
// 2^-64. The product with the position modulo 2^64 is the angle's part of a turn,
// without any rounding, however far the position and however fast the pair; its
// upper 32 bits, as a signed number, are the angle within half a turn. So the
// fast sine and cosine, whose error is absolute (2^-21 within that range),
// are enough before a rounding to BF16 (2^-8).
//
// The kernel moves bytes. A thread has 16 channels of a token, 8 pairs, in heads
// hl, hl + lanes, ...: one set of sines and cosines for all of them, and four
// heads' loads (two of 16 bytes each) in flight. A warp reads whole sectors, and
// whole lines where the head is 128 channels wide. HBM bounds it: 16001 tokens of
// 40 heads, D = 128, take 50 us, 6.5 TB/s (98% of a copy's rate); a step's 64 tokens 2.8 us,
// the latency of a launch, a load of the position, the sines and a store.
#include <cuda_bf16.h>

#include "launch.cuh"
#include "prompt.cuh"
#include "tc_ptx.cuh"

namespace sage {
namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 4;  // heads of a thread whose loads are in flight together

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Pairs (first[i], second[i]) with kInterleaved = false, (word's low, high half) otherwise.
template <bool kInterleaved>
__device__ __forceinline__ void turn(uint4& x, uint4& y, const float (&c)[8], const float (&s)[8]) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&x);
  uint32_t* b = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kInterleaved) {
      const float a0 = lo(a[i]), b0 = hi(a[i]), a1 = lo(b[i]), b1 = hi(b[i]);
      a[i] = pack(a0 * c[i] - b0 * s[i], b0 * c[i] + a0 * s[i]);
      b[i] = pack(a1 * c[4 + i] - b1 * s[4 + i], b1 * c[4 + i] + a1 * s[4 + i]);
    } else {
      const float a0 = lo(a[i]), a1 = hi(a[i]), b0 = lo(b[i]), b1 = hi(b[i]);
      a[i] = pack(a0 * c[2 * i] - b0 * s[2 * i], a1 * c[2 * i + 1] - b1 * s[2 * i + 1]);
      b[i] = pack(b0 * c[2 * i] + a0 * s[2 * i], b1 * c[2 * i + 1] + a1 * s[2 * i + 1]);
    }
  }
}

// lanes: threads (times D / 16) that share a token, a power of two.
template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a, uint32_t tokens, int lanes) {
  constexpr int kUnits = D / 16;
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int u = static_cast<int>(threadIdx.x) % kUnits, slot = static_cast<int>(threadIdx.x) / kUnits;
  const uint32_t n = blockIdx.x * static_cast<uint32_t>(kThreads / kUnits / lanes) + static_cast<uint32_t>(slot / lanes);
  if (n >= tokens) return;
  const int64_t b = n / static_cast<uint32_t>(a.T), t = n % static_cast<uint32_t>(a.T);
  const bool turned = 8 * u < a.pairs;
  const int c0 = turned && !kInterleaved ? 8 * u : 16 * u, c1 = turned && !kInterleaved ? a.pairs + 8 * u : 16 * u + 8;
  const int heads = a.H + a.Hkv;
  const uint16_t* q = a.q.p + b * a.q.sb + t * a.q.ss;
  const uint16_t* k = a.k.p + b * a.k.sb + t * a.k.ss;
  uint16_t* q_out = a.q_out.p + b * a.q_out.sb + t * a.q_out.ss;
  uint16_t* k_out = a.k_out.p + b * a.k_out.sb + t * a.k_out.ss;
  float c[8], s[8];
  bool ready = !turned;
  for (int h0 = slot % lanes; h0 < heads; h0 += kAtOnce * lanes) {
    uint4 x[kAtOnce], y[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int h = h0 + i * lanes;
      if (h < heads) {
        const uint16_t* p = h < a.H ? q + h * a.q.sh : k + (h - a.H) * a.k.sh;
        x[i] = *reinterpret_cast<const uint4*>(p + c0);
        y[i] = *reinterpret_cast<const uint4*>(p + c1);
      }
    }
    if (!ready) {  // under the first loads
      ready = true;
      const int64_t at = a.positions[b * a.pos_b + t * a.pos_t];
      const ulonglong2* w = reinterpret_cast<const ulonglong2*>(a.turns + 8 * u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const ulonglong2 v = w[i];
        const uint64_t turns[2] = {static_cast<uint64_t>(at) * v.x, static_cast<uint64_t>(at) * v.y};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float angle = static_cast<float>(static_cast<int32_t>(turns[e] >> 32)) * 1.4629180792671596e-09f;  // 2 pi / 2^32
          float sn, cs;
          __sincosf(angle, &sn, &cs);
          c[2 * i + e] = cs * a.magnitude;
          s[2 * i + e] = (a.inverse ? -sn : sn) * a.magnitude;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int h = h0 + i * lanes;
      if (h < heads) {
        if (turned) turn<kInterleaved>(x[i], y[i], c, s);
        uint16_t* p = h < a.H ? q_out + h * a.q_out.sh : k_out + (h - a.H) * a.k_out.sh;
        *reinterpret_cast<uint4*>(p + c0) = x[i];
        *reinterpret_cast<uint4*>(p + c1) = y[i];
      }
    }
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int64_t D, cudaStream_t stream) {
  const uint32_t tokens = static_cast<uint32_t>(a.B * a.T);
  const int slots = kThreads / static_cast<int>(D / 16);
  // One set of sines for many heads where there are tokens enough (16001 tokens, 40
  // heads: 50 us, 55 with lanes for all heads), else all heads at once (64 tokens: 2.8
  // us, 4.7 with four lanes; 500 tokens: 4.2 and 4.8).
  int lanes = 4;
  while (lanes < slots && lanes * kAtOnce < a.H + a.Hkv && div_up(tokens, slots / lanes) < 2 * sm_count_current())
    lanes *= 2;
  const dim3 grid(static_cast<unsigned>(div_up(tokens, slots / lanes)));
  const auto kernel = D == 128 ? (a.interleaved ? rotary_kernel<128, true> : rotary_kernel<128, false>)
                               : (a.interleaved ? rotary_kernel<64, true> : rotary_kernel<64, false>);
  return launch_dependent(kernel, grid, kThreads, 0, stream, a, tokens, lanes);
}

}  // namespace sage
