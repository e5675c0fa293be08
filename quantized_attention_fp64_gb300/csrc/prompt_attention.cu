// Attention over packed prompts: a warp has one query row of one head and takes
// the keys one after another, with the running maximum and sum of the softmax.
#include <cuda_bf16.h>

#include "launch.cuh"
#include "prompt.cuh"
#include "tc_ptx.cuh"

namespace sage {
namespace {

constexpr int kThreads = 256;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float value(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

template <int D>
__global__ void __launch_bounds__(kThreads) prompt_attention_kernel(const PromptArgs a) {
  constexpr int C = D / 32;
  tc::griddep_wait();
  tc::griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int h = static_cast<int>(blockIdx.y);
  if (row >= a.N) return;
  int32_t first = 0, end = 0, kv_first = 0, kv_end = 0;
  bool bad = false, found = false;
  for (int b = 0; b < a.B && !found; ++b) {
    packed_rows(a.offsets[b], a.offsets[b + 1], a.N, &bad, &first, &end);
    packed_rows(a.kv_offsets[b], a.kv_offsets[b + 1], a.M, &bad, &kv_first, &kv_end);
    found = row >= first && row < end;
  }
  if (bad && lane == 0) atomicExch(a.dev_err, kDevErrOffsets);
  uint16_t* out = a.out.p + row * a.out.ss + h * a.out.sh;
  float* lse = a.lse != nullptr ? a.lse + h * a.N + row : nullptr;
  if (!found) {
    if (!a.zero_rest) return;
    for (int c = 0; c < C; ++c) out[lane * C + c] = 0;
    if (lse != nullptr && lane == 0) *lse = -INFINITY;
    return;
  }
  const int64_t keys = kv_end - kv_first, last = a.causal ? keys - (end - row) : keys - 1;
  const int hk = h / (a.H / a.Hkv);
  float q[C], o[C], m = -INFINITY, l = 0.0f;
  for (int c = 0; c < C; ++c) {
    q[c] = value(a.q.p[row * a.q.ss + h * a.q.sh + lane * C + c]) * a.sm_log2;
    o[c] = 0.0f;
  }
  for (int64_t j = 0; j <= last; ++j) {
    const uint16_t* k = a.k.p + (kv_first + j) * a.k.ss + hk * a.k.sh + lane * C;
    const uint16_t* v = a.v.p + (kv_first + j) * a.v.ss + hk * a.v.sh + lane * C;
    float z = 0.0f;
    for (int c = 0; c < C; ++c) z = fmaf(q[c], value(k[c]), z);
    for (int s = 16; s > 0; s >>= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
    const float up = fmaxf(m, z);
    const float alpha = exp2f(m - up), p = exp2f(z - up);
    m = up;
    l = l * alpha + p;
    for (int c = 0; c < C; ++c) o[c] = fmaf(p, value(v[c]), o[c] * alpha);
  }
  for (int c = 0; c < C; ++c) {
    const __nv_bfloat16 r = __float2bfloat16_rn(last >= 0 ? o[c] / l : 0.0f);
    out[lane * C + c] = *reinterpret_cast<const uint16_t*>(&r);
  }
  if (lse != nullptr && lane == 0) *lse = last >= 0 ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

size_t prompt_attention_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

cudaError_t launch_prompt_attention(const PromptArgs& a, int64_t D, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(div_up(a.N, kThreads / 32)), static_cast<unsigned>(a.H));
  return launch_dependent(D == 128 ? prompt_attention_kernel<128> : prompt_attention_kernel<64>, grid, kThreads, 0,
                          stream, a);
}

}  // namespace sage
