// C ABI of the 8-bit paged key/value cache: argument validation, buffer
// layout, dispatch. Everything is checked on the host before any work is
// enqueued, except what only the device holds (lengths, page numbers), which
// the kernels check before they use it.
#include <cmath>

#include "../../include/sage.h"
#include "cache.cuh"

namespace sage {
namespace {

constexpr int64_t kMaxPages = int64_t(1) << 20;  // the page lists' check keeps one bit per page in shared memory
constexpr int64_t kMaxPageSize = 4096;
constexpr int64_t kMaxDim = 65535;               // sequences and heads are grid dimensions
constexpr int64_t kMaxTokens = int64_t(1) << 30; // tokens of one call

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool stride_ok(int64_t s) { return s % 8 == 0; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA; }

int check_cache_sizes(int64_t num_pages, int64_t page_size, int64_t H, int64_t D) {
  if (num_pages < 0 || page_size < 0 || H < 0 || D < 0) return SAGE_ERR_SHAPE;
  if (D != 128 && D != 64) return SAGE_ERR_HEAD_DIM;
  if (page_size == 0 || page_size % kCacheBlock != 0) return SAGE_ERR_SHAPE;
  if (num_pages > kMaxPages || page_size > kMaxPageSize || H > kMaxDim) return SAGE_ERR_TOO_LARGE;
  // block numbers and byte offsets stay far inside int64; a block number fits 40 bits
  return SAGE_OK;
}

int check_cache(const sage_cache* c, CacheView* view) {
  if (c == nullptr) return SAGE_ERR_NULLPTR;
  const int rc = check_cache_sizes(c->num_pages, c->page_size, c->H, c->D);
  if (rc != SAGE_OK) return rc;
  const void* ptrs[4] = {c->k_codes_dev, c->v_codes_dev, c->k_scale_dev, c->v_scale_dev};
  for (const void* p : ptrs) {
    if (p == nullptr) return SAGE_ERR_NULLPTR;
    if (!aligned(p, 16)) return SAGE_ERR_ALIGN;
  }
  *view = CacheView{c->k_codes_dev, c->v_codes_dev, c->k_scale_dev, c->v_scale_dev, c->num_pages,
                    static_cast<int32_t>(c->H), static_cast<int32_t>(c->page_size / kCacheBlock)};
  return SAGE_OK;
}

int check_table(const int32_t* table, int64_t stride, int64_t max_pages, PageTable* out) {
  if (table == nullptr) return SAGE_ERR_NULLPTR;
  if (!aligned(table, 4)) return SAGE_ERR_ALIGN;
  if (max_pages < 0 || stride < 0) return SAGE_ERR_SHAPE;
  *out = PageTable{table, stride, max_pages};
  return SAGE_OK;
}

int check_ints(const int32_t* p, bool needed) {
  if (p == nullptr) return needed ? SAGE_ERR_NULLPTR : SAGE_OK;
  return aligned(p, 4) ? SAGE_OK : SAGE_ERR_ALIGN;
}

int check_tensor(const sage_bf16_tensor& t) {
  if (t.ptr_dev == nullptr) return SAGE_ERR_NULLPTR;
  return aligned(t.ptr_dev, 16) && stride_ok(t.stride_b) && stride_ok(t.stride_s) && stride_ok(t.stride_h)
             ? SAGE_OK
             : SAGE_ERR_ALIGN;
}

Bf16In to_in(const sage_bf16_tensor& t) {
  return Bf16In{static_cast<const uint16_t*>(t.ptr_dev), t.stride_b, t.stride_s, t.stride_h};
}

Out to_out(const sage_bf16_tensor& t) {
  return Out{static_cast<uint16_t*>(const_cast<void*>(t.ptr_dev)), t.stride_b, t.stride_s, t.stride_h};
}

int check_batch(int64_t B, int64_t T) {
  if (B < 0 || T < 0) return SAGE_ERR_SHAPE;
  if (B > kMaxDim || T > kMaxTokens) return SAGE_ERR_TOO_LARGE;
  return SAGE_OK;
}

int check_heads(int64_t H, int64_t Hkv) {
  if (H < 0 || (Hkv == 0 ? H != 0 : H % Hkv != 0)) return SAGE_ERR_SHAPE;
  return H > kMaxDim ? SAGE_ERR_TOO_LARGE : SAGE_OK;
}

}  // namespace
}  // namespace sage

using namespace sage;

extern "C" {

int sage_cache_size(int64_t num_pages, int64_t page_size, int64_t H, int64_t D, size_t* bytes, void* base_dev,
                    sage_cache* cache) {
  if (bytes == nullptr) return SAGE_ERR_NULLPTR;
  const int rc = check_cache_sizes(num_pages, page_size, H, D);
  if (rc != SAGE_OK) return rc;
  const size_t blocks = static_cast<size_t>(num_pages) * static_cast<size_t>(H) *
                        static_cast<size_t>(page_size / kCacheBlock);
  const size_t codes = round256(blocks * kCacheBlock * static_cast<size_t>(D)), scales = round256(blocks * 4);
  *bytes = 2 * codes + 2 * scales;
  if (base_dev != nullptr) {
    if (cache == nullptr) return SAGE_ERR_NULLPTR;
    if (!aligned(base_dev, 256)) return SAGE_ERR_ALIGN;
    char* p = static_cast<char*>(base_dev);
    cache->k_codes_dev = reinterpret_cast<int8_t*>(p);
    cache->v_codes_dev = reinterpret_cast<int8_t*>(p + codes);
    cache->k_scale_dev = reinterpret_cast<float*>(p + 2 * codes);
    cache->v_scale_dev = reinterpret_cast<float*>(p + 2 * codes + scales);
    cache->num_pages = num_pages;
    cache->page_size = page_size;
    cache->H = H;
    cache->D = D;
  }
  return SAGE_OK;
}

int sage_cache_append(const sage_cache_append_args* args) {
  if (args == nullptr) return SAGE_ERR_NULLPTR;
  CacheView c;
  PageTable pt;
  int rc;
  if ((rc = check_cache(args->cache, &c)) != SAGE_OK || (rc = check_batch(args->B, args->T)) != SAGE_OK ||
      (rc = check_table(args->table_dev, args->table_stride, args->max_pages, &pt)) != SAGE_OK ||
      (rc = check_ints(args->starts_dev, true)) != SAGE_OK || (rc = check_ints(args->counts_dev, false)) != SAGE_OK ||
      (rc = check_tensor(args->k)) != SAGE_OK || (rc = check_tensor(args->v)) != SAGE_OK)
    return rc;
  int* dev_err = nullptr;
  if ((rc = device_error_word(&dev_err)) != SAGE_OK) return rc;
  if (args->B == 0 || args->T == 0 || c.H == 0) return SAGE_OK;
  return cuda_status(launch_cache_append(c, args->cache->D, pt, args->starts_dev, args->counts_dev, to_in(args->k),
                                         to_in(args->v), args->B, args->T, dev_err,
                                         static_cast<cudaStream_t>(args->cuda_stream)));
}

int sage_cache_read(const sage_cache_read_args* args) {
  if (args == nullptr) return SAGE_ERR_NULLPTR;
  CacheView c;
  PageTable pt;
  int rc;
  if ((rc = check_cache(args->cache, &c)) != SAGE_OK || (rc = check_batch(args->B, args->T)) != SAGE_OK ||
      (rc = check_table(args->table_dev, args->table_stride, args->max_pages, &pt)) != SAGE_OK ||
      (rc = check_ints(args->starts_dev, true)) != SAGE_OK || (rc = check_ints(args->counts_dev, false)) != SAGE_OK ||
      (rc = check_tensor(args->k_out)) != SAGE_OK || (rc = check_tensor(args->v_out)) != SAGE_OK)
    return rc;
  int* dev_err = nullptr;
  if ((rc = device_error_word(&dev_err)) != SAGE_OK) return rc;
  if (args->B == 0 || args->T == 0 || c.H == 0) return SAGE_OK;
  return cuda_status(launch_cache_read(c, args->cache->D, pt, args->starts_dev, args->counts_dev, to_out(args->k_out),
                                       to_out(args->v_out), args->B, args->T, args->zero_rest != 0, dev_err,
                                       static_cast<cudaStream_t>(args->cuda_stream)));
}

int sage_cache_copy_pages(const sage_cache* cache, const int32_t* src_dev, const int32_t* dst_dev, int64_t n,
                          void* cuda_stream) {
  CacheView c;
  int rc;
  if ((rc = check_cache(cache, &c)) != SAGE_OK) return rc;
  if (n < 0) return SAGE_ERR_SHAPE;
  if (n > kMaxPages) return SAGE_ERR_TOO_LARGE;
  if ((rc = check_ints(src_dev, true)) != SAGE_OK || (rc = check_ints(dst_dev, true)) != SAGE_OK) return rc;
  int* dev_err = nullptr;
  if ((rc = device_error_word(&dev_err)) != SAGE_OK) return rc;
  if (n == 0 || c.H == 0 || c.num_pages == 0) return SAGE_OK;
  return cuda_status(launch_cache_copy_pages(c, cache->D, src_dev, dst_dev, n, dev_err,
                                             static_cast<cudaStream_t>(cuda_stream)));
}

int sage_cache_attention_workspace_size(int64_t B, int64_t T, int64_t H, int64_t Hkv, int64_t D, size_t* bytes) {
  if (bytes == nullptr) return SAGE_ERR_NULLPTR;
  int rc;
  if (Hkv < 0) return SAGE_ERR_SHAPE;
  if ((rc = check_batch(B, T)) != SAGE_OK || (rc = check_heads(H, Hkv)) != SAGE_OK) return rc;
  if (D != 128 && D != 64) return SAGE_ERR_HEAD_DIM;
  if (H > 0 && T > kMaxTokens / (H / Hkv)) return SAGE_ERR_TOO_LARGE;
  *bytes = (B == 0 || T == 0 || H == 0) ? 0 : cache_attention_workspace_bytes(B, T, H, Hkv, D);
  return SAGE_OK;
}

int sage_cache_attention(const sage_cache_attention_args* args) {
  if (args == nullptr) return SAGE_ERR_NULLPTR;
  CacheAttentionArgs a;
  int rc;
  const int64_t B = args->B, T = args->T, H = args->H;
  if ((rc = check_cache(args->cache, &a.c)) != SAGE_OK || (rc = check_batch(B, T)) != SAGE_OK ||
      (rc = check_heads(H, a.c.H)) != SAGE_OK ||
      (rc = check_table(args->table_dev, args->table_stride, args->max_pages, &a.pt)) != SAGE_OK ||
      (rc = check_ints(args->lengths_dev, true)) != SAGE_OK ||
      (rc = check_ints(args->q_lengths_dev, false)) != SAGE_OK || (rc = check_tensor(args->q)) != SAGE_OK ||
      (rc = check_tensor(args->out)) != SAGE_OK)
    return rc;
  if (a.c.num_pages == 0) a.pt.max_pages = 0;  // without pages there are no tokens, whatever the table says
  // the call's blocks, all sequences and heads, are counted in 32 bits
  // (once for every 256 query rows that share a key/value head, with 16 more
  // for what beginning a unit counts)
  const int64_t seq_blocks = table_capacity(a.pt.max_pages, a.c.blocks_per_page) / kCacheBlock + 16;
  constexpr int64_t kMost = (int64_t(1) << 31) - 1;
  if (H > 0 && T > kMaxTokens / (H / a.c.H)) return SAGE_ERR_TOO_LARGE;  // rows of a key/value head, too
  const int64_t pairs = H > 0 ? div_up(T * (H / a.c.H), 256) : 0;
  if (B > 0 && pairs > 0 && (pairs > kMost / (B * a.c.H) || seq_blocks > kMost / (B * a.c.H * pairs)))
    return SAGE_ERR_TOO_LARGE;
  if (args->lse_dev != nullptr && !aligned(args->lse_dev, 4)) return SAGE_ERR_ALIGN;
  const float sm = args->sm_scale;
  if (!(std::isnan(sm) || (std::isfinite(sm) && sm > 0.0f))) return SAGE_ERR_ARG;
  const int64_t D = args->cache->D;
  const size_t need = (B == 0 || T == 0 || H == 0) ? 0 : cache_attention_workspace_bytes(B, T, H, a.c.H, D);
  if (need > 0) {
    if (args->workspace_dev == nullptr) return SAGE_ERR_NULLPTR;
    if (!aligned(args->workspace_dev, 256)) return SAGE_ERR_ALIGN;
    if (args->workspace_bytes < need) return SAGE_ERR_WORKSPACE;
  }
  if ((rc = device_error_word(&a.dev_err)) != SAGE_OK) return rc;
  if (B == 0 || T == 0 || H == 0) return SAGE_OK;
  const double scale = std::isnan(sm) ? 1.0 / std::sqrt(static_cast<double>(D)) : sm;
  a.lengths = args->lengths_dev;
  a.q_lengths = args->q_lengths_dev;
  a.q = to_in(args->q);
  a.out = to_out(args->out);
  a.lse = args->lse_dev;
  a.workspace = args->workspace_dev;
  a.B = B;
  a.T = T;
  a.H = static_cast<int32_t>(H);
  a.causal = args->is_causal != 0;
  a.zero_rest = args->zero_rest != 0 && args->q_lengths_dev != nullptr;
  a.sm_log2 = static_cast<float>(scale * 1.4426950408889634);
  return cuda_status(launch_cache_attention(a, D, static_cast<cudaStream_t>(args->cuda_stream)));
}

}  // extern "C"
