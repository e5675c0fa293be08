// C ABI of the operators on prompts: argument validation and dispatch.
// Everything is checked on the host before any work is enqueued, except what
// only the device holds (offsets), which the kernels check before they use it.
#include <cmath>

#include "../../include/sage.h"
#include "checks.cuh"
#include "prompt.cuh"

namespace sage {
namespace {

constexpr int64_t kMaxDim = 65535;                // sequences and heads
constexpr int64_t kMaxTokens = int64_t(1) << 30;  // rows of one tensor

int check_head_dim(int64_t D) { return D == 128 || D == 64 ? SAGE_OK : SAGE_ERR_HEAD_DIM; }

int check_prompt_sizes(int64_t N, int64_t M, int64_t H, int64_t Hkv, int64_t D, int64_t B) {
  if (N < 0 || M < 0 || H < 0 || Hkv < 0 || B < 0 || D < 0) return SAGE_ERR_SHAPE;
  const int rc = check_head_dim(D);
  if (rc != SAGE_OK) return rc;
  if (Hkv == 0 ? H != 0 : H % Hkv != 0) return SAGE_ERR_SHAPE;
  if (N > kMaxTokens || M > kMaxTokens || H > kMaxDim || B > kMaxDim) return SAGE_ERR_TOO_LARGE;
  // units of 128 rows of a head are counted in 32 bits
  if (H > 0 && N / 128 + B + 1 > (int64_t(1) << 30) / H) return SAGE_ERR_TOO_LARGE;
  return SAGE_OK;
}

}  // namespace
}  // namespace sage

using namespace sage;

extern "C" {

int sage_rotary_turns(const double* inv_freq, int64_t n, uint64_t* turns) {
  if (n < 0) return SAGE_ERR_SHAPE;
  if (n > 0 && (inv_freq == nullptr || turns == nullptr)) return SAGE_ERR_NULLPTR;
  for (int64_t i = 0; i < n; ++i)
    if (!std::isfinite(inv_freq[i])) return SAGE_ERR_ARG;
  for (int64_t i = 0; i < n; ++i) {
    // the part of a turn in [0, 1), then its first 64 binary places (a double
    // below 1/2 has places behind them, which are cut off)
    double t = inv_freq[i] * 0.15915494309189533577;
    t -= std::floor(t);
    if (t >= 1.0) t = 0.0;
    const double high = std::floor(t * 0x1p32);
    const double low = std::floor((t * 0x1p32 - high) * 0x1p32);
    turns[i] = static_cast<uint64_t>(high) << 32 | static_cast<uint64_t>(low);
  }
  return SAGE_OK;
}

int sage_rotary(const sage_rotary_args* args) {
  if (args == nullptr) return SAGE_ERR_NULLPTR;
  int rc;
  const int64_t B = args->B, T = args->T, H = args->H, Hkv = args->Hkv, D = args->D;
  if (B < 0 || T < 0 || H < 0 || Hkv < 0 || D < 0) return SAGE_ERR_SHAPE;
  if ((rc = check_head_dim(D)) != SAGE_OK) return rc;
  if (args->rotary_dim <= 0 || args->rotary_dim > D || args->rotary_dim % 16 != 0) return SAGE_ERR_ARG;
  if (!std::isfinite(args->magnitude)) return SAGE_ERR_ARG;
  if (B > kMaxTokens || T > kMaxTokens || H > kMaxDim || Hkv > kMaxDim || (T > 0 && B > kMaxTokens / T))
    return SAGE_ERR_TOO_LARGE;
  if ((rc = check_tensor(args->q)) != SAGE_OK || (rc = check_tensor(args->q_out)) != SAGE_OK) return rc;
  if (Hkv > 0 && ((rc = check_tensor(args->k)) != SAGE_OK || (rc = check_tensor(args->k_out)) != SAGE_OK)) return rc;
  if ((rc = check_ints(args->positions_dev, true)) != SAGE_OK) return rc;
  if (args->turns_dev == nullptr) return SAGE_ERR_NULLPTR;
  if (!aligned(args->turns_dev, 16)) return SAGE_ERR_ALIGN;
  if (!tensor_apart(args->q_out, B, T, H, D) || !tensor_apart(args->k_out, B, T, Hkv, D)) return SAGE_ERR_LAYOUT;
  if (B > 0 && T > 0) {
    // in place a thread writes what it has read, if that is where it belongs
    const void *q = args->q.ptr_dev, *k = args->k.ptr_dev, *q_out = args->q_out.ptr_dev, *k_out = args->k_out.ptr_dev;
    if (H > 0 && q_out == q && !same_rows(args->q_out, args->q, B, T, H)) return SAGE_ERR_LAYOUT;
    if (Hkv > 0 && k_out == k && !same_rows(args->k_out, args->k, B, T, Hkv)) return SAGE_ERR_LAYOUT;
    if (H > 0 && Hkv > 0 && (q_out == k_out || q_out == k || k_out == q)) return SAGE_ERR_ARG;
  }
  int* dev_err = nullptr;
  if ((rc = device_error_word(&dev_err)) != SAGE_OK) return rc;
  if (B == 0 || T == 0 || H + Hkv == 0) return SAGE_OK;
  RotaryArgs a;
  a.q = to_in(args->q);
  a.k = to_in(args->k);
  a.q_out = to_out(args->q_out);
  a.k_out = to_out(args->k_out);
  a.B = B;
  a.T = T;
  a.H = static_cast<int32_t>(H);
  a.Hkv = static_cast<int32_t>(Hkv);
  a.pairs = static_cast<int32_t>(args->rotary_dim / 2);
  a.turns = args->turns_dev;
  a.positions = args->positions_dev;
  a.pos_b = args->positions_stride_b;
  a.pos_t = args->positions_stride_t;
  a.magnitude = args->magnitude;
  a.interleaved = args->interleaved != 0;
  a.inverse = args->inverse != 0;
  return cuda_status(launch_rotary(a, D, static_cast<cudaStream_t>(args->cuda_stream)));
}

int sage_prompt_attention_workspace_size(int64_t N, int64_t M, int64_t H, int64_t Hkv, int64_t D, int64_t B,
                                         size_t* bytes) {
  if (bytes == nullptr) return SAGE_ERR_NULLPTR;
  const int rc = check_prompt_sizes(N, M, H, Hkv, D, B);
  if (rc != SAGE_OK) return rc;
  *bytes = N == 0 || H == 0 ? 0 : prompt_attention_workspace_bytes(N, M, H, Hkv, D, B);
  return SAGE_OK;
}

int sage_prompt_attention(const sage_prompt_attention_args* args) {
  if (args == nullptr) return SAGE_ERR_NULLPTR;
  int rc;
  const int64_t N = args->N, M = args->M, H = args->H, D = args->D, B = args->B;
  if ((rc = check_prompt_sizes(N, M, H, args->Hkv, D, B)) != SAGE_OK || (rc = check_mapped(args->q, 1, N, H)) != SAGE_OK ||
      (rc = check_mapped(args->k, 1, M, args->Hkv)) != SAGE_OK ||
      (rc = check_mapped(args->v, 1, M, args->Hkv)) != SAGE_OK ||
      (rc = check_tensor(args->out)) != SAGE_OK || (rc = check_ints(args->offsets_dev, true)) != SAGE_OK ||
      (rc = check_ints(args->kv_offsets_dev, false)) != SAGE_OK || (rc = check_floats(args->lse_dev, false)) != SAGE_OK)
    return rc;
  if (!scale_ok(args->sm_scale)) return SAGE_ERR_ARG;
  const void* out = args->out.ptr_dev;  // (a unit may be done twice: its queries have to be there still)
  if (N > 0 && H > 0 && (out == args->q.ptr_dev || (M > 0 && (out == args->k.ptr_dev || out == args->v.ptr_dev)))) return SAGE_ERR_ARG;
  if (!tensor_apart(args->out, 1, N, H, D)) return SAGE_ERR_LAYOUT;
  const size_t need = N == 0 || H == 0 ? 0 : prompt_attention_workspace_bytes(N, M, H, args->Hkv, D, B);
  if (need > 0) {
    if (args->workspace_dev == nullptr) return SAGE_ERR_NULLPTR;
    if (!aligned(args->workspace_dev, 256)) return SAGE_ERR_ALIGN;
    if (args->workspace_bytes < need) return SAGE_ERR_WORKSPACE;
  }
  PromptArgs a;
  if ((rc = device_error_word(&a.dev_err)) != SAGE_OK) return rc;
  if (N == 0 || H == 0) return SAGE_OK;
  a.q = to_in(args->q);
  a.k = to_in(args->k);
  a.v = to_in(args->v);
  a.out = to_out(args->out);
  a.N = N;
  a.M = M;
  a.H = static_cast<int32_t>(H);
  a.Hkv = static_cast<int32_t>(args->Hkv);
  a.B = static_cast<int32_t>(B);
  a.offsets = args->offsets_dev;
  a.kv_offsets = args->kv_offsets_dev != nullptr ? args->kv_offsets_dev : args->offsets_dev;
  a.lse = args->lse_dev;
  a.workspace = args->workspace_dev;
  a.causal = args->is_causal != 0;
  a.zero_rest = args->zero_rest != 0;
  a.sm_log2 = scale_log2(args->sm_scale, D);
  return cuda_status(launch_prompt_attention(a, D, static_cast<cudaStream_t>(args->cuda_stream)));
}

}  // extern "C"
