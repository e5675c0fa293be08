// Checks of arguments that the entry points on BF16 tensors and device vectors share.
#pragma once

#include <cmath>
#include <cstdint>

#include "../../include/sage.h"
#include "common.cuh"

namespace sage {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool stride_ok(int64_t s) { return s % 8 == 0; }
inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }
inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA; }

inline int check_ints(const int32_t* p, bool needed) {
  if (p == nullptr) return needed ? SAGE_ERR_NULLPTR : SAGE_OK;
  return aligned(p, 4) ? SAGE_OK : SAGE_ERR_ALIGN;
}

inline int check_floats(const float* p, bool needed) {
  if (p == nullptr) return needed ? SAGE_ERR_NULLPTR : SAGE_OK;
  return aligned(p, 4) ? SAGE_OK : SAGE_ERR_ALIGN;
}

inline int check_tensor(const sage_bf16_tensor& t) {
  if (t.ptr_dev == nullptr) return SAGE_ERR_NULLPTR;
  return aligned(t.ptr_dev, 16) && stride_ok(t.stride_b) && stride_ok(t.stride_s) && stride_ok(t.stride_h)
             ? SAGE_OK
             : SAGE_ERR_ALIGN;
}

inline Bf16In to_in(const sage_bf16_tensor& t) {
  return Bf16In{static_cast<const uint16_t*>(t.ptr_dev), t.stride_b, t.stride_s, t.stride_h};
}

inline Out to_out(const sage_bf16_tensor& t) {
  return Out{static_cast<uint16_t*>(const_cast<void*>(t.ptr_dev)), t.stride_b, t.stride_s, t.stride_h};
}

// sm_scale as the entries take it: NaN (1 / sqrt(D)), or finite and positive.
inline bool scale_ok(float sm) { return std::isnan(sm) || (std::isfinite(sm) && sm > 0.0f); }
// sm_scale * log2(e)
inline float scale_log2(float sm, int64_t D) {
  const double scale = std::isnan(sm) ? 1.0 / std::sqrt(static_cast<double>(D)) : sm;
  return static_cast<float>(scale * 1.4426950408889634);
}

}  // namespace sage
