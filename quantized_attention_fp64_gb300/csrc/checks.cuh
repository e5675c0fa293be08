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

// Tensors that a tensor map describes: the strides of dimensions with more than
// one entry are positive and below 2^40 bytes (an expanded dimension has stride 0).
inline bool mapped_stride_ok(int64_t n, int64_t s) { return n <= 1 || (s > 0 && s < int64_t(1) << 39); }
inline int check_mapped(const sage_bf16_tensor& t, int64_t B, int64_t S, int64_t H) {
  const int rc = check_tensor(t);
  if (rc != SAGE_OK) return rc;
  return mapped_stride_ok(B, t.stride_b) && mapped_stride_ok(S, t.stride_s) && mapped_stride_ok(H, t.stride_h)
             ? SAGE_OK
             : SAGE_ERR_LAYOUT;
}

// Rows of n entries, B by H of them, that are written: none may overlap another
// (strides in entries, either one the larger).
inline bool rows_apart(int64_t B, int64_t stride_b, int64_t H, int64_t stride_h, int64_t n) {
  int64_t sb = stride_b < 0 ? -stride_b : stride_b, sh = stride_h < 0 ? -stride_h : stride_h;
  if (n <= 0 || B <= 0 || H <= 0 || (B == 1 && H == 1)) return true;
  if (B == 1) return sh >= n;
  if (H == 1) return sb >= n;
  if (sb < sh) {
    int64_t x = sb;
    sb = sh;
    sh = x;
    x = B;
    B = H;
    H = x;
  }
  return sh >= n && sb - n >= 0 && (sb - n) / sh >= H - 1;
}

// A tensor that is written: none of its rows of D channels may overlap another
// (the dimensions nested in one another, in any order; an expanded one has stride 0).
inline bool tensor_apart(const sage_bf16_tensor& t, int64_t B, int64_t S, int64_t H, int64_t D) {
  int64_t n[3] = {B, S, H}, s[3] = {t.stride_b, t.stride_s, t.stride_h};
  int64_t span = D;  // of what is nested so far
  if (B <= 0 || S <= 0 || H <= 0) return true;
  for (int done = 0; done < 3; ++done) {
    int64_t least = INT64_MAX, entries = 1;
    int at = -1;
    for (int i = 0; i < 3; ++i) {
      const int64_t x = s[i] == INT64_MIN ? INT64_MAX : s[i] < 0 ? -s[i] : s[i];
      if (n[i] > 1 && (at < 0 || x < least)) at = i, least = x, entries = n[i];
    }
    if (at < 0) return true;
    if (least < span) return false;
    span = entries - 1 > (INT64_MAX - span) / least ? INT64_MAX : span + (entries - 1) * least;
    n[at] = 1;
  }
  return true;
}

// Whether two tensors at one address have the same rows there.
inline bool same_rows(const sage_bf16_tensor& x, const sage_bf16_tensor& y, int64_t B, int64_t S, int64_t H) {
  return (B <= 1 || x.stride_b == y.stride_b) && (S <= 1 || x.stride_s == y.stride_s) && (H <= 1 || x.stride_h == y.stride_h);
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
