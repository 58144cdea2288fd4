// The extern "C" boundary of the cache in 4 bits: argument checks and dispatch.
// No exception leaves this file; no allocation, free or synchronisation happens
// here.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "internal.h"

namespace qpkv {
namespace {

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

qpkv_status launched(cudaError_t e) { return e == cudaSuccess ? QPKV_OK : QPKV_ERR_CUDA; }

qpkv_status check_cache(int D, int ps, int P, int bt_stride, int Hkv, int dtype) {
  if (Hkv < 1 || P < 1 || bt_stride < 1 || ps < 1) return QPKV_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || ps % 16 != 0) return QPKV_ERR_UNSUPPORTED;
  if (dtype != QPKV_DTYPE_BF16 && dtype != QPKV_DTYPE_F16) return QPKV_ERR_UNSUPPORTED;
  if (Hkv > 65535 || static_cast<int64_t>(bt_stride) * ps > INT32_MAX - 64) return QPKV_ERR_UNSUPPORTED;
  return QPKV_OK;
}

bool strides_fit(int64_t t, int64_t h) { return t % 8 == 0 && h % 8 == 0; }

// Query heads over kv heads, and rows that an int counts.
bool heads_fit(int Hq, int Hkv, int T) {
  return Hq % Hkv == 0 && static_cast<int64_t>(T) * (Hq / Hkv) <= INT32_MAX - 64 &&
         static_cast<int64_t>(T) * Hq <= 4ll * INT32_MAX;
}

}  // namespace
}  // namespace qpkv

using namespace qpkv;

extern "C" {

qpkv_status qpkv_write_group4(const qpkv_write_group4_params* p, void* stream) {
  if (p == nullptr || p->num_seqs < 0 || p->num_tokens < 0) return QPKV_ERR_INVALID_ARG;
  const qpkv_status st = check_cache(p->head_dim, p->page_size, p->num_pages, p->bt_stride, p->num_heads_kv, p->dtype);
  if (st != QPKV_OK) return st;
  const bool turns = p->rope_cos != nullptr;
  if (turns != (p->rope_sin != nullptr) || (p->k_bounds != nullptr) != (p->bound_scale != nullptr) ||
      (turns && (p->rope_max_pos < 1 || p->rot_dim < 1)) ||
      (p->q != nullptr && (!turns || p->q_out == nullptr || p->num_heads_q < 1)))
    return QPKV_ERR_INVALID_ARG;
  if (turns && (p->rot_dim % 32 != 0 || p->rot_dim > p->head_dim)) return QPKV_ERR_UNSUPPORTED;
  if (p->q != nullptr && p->num_heads_q > 65535) return QPKV_ERR_UNSUPPORTED;
  if (p->num_seqs == 0 || p->num_tokens == 0) return QPKV_OK;
  // blocks: two at most for a (piece, head), one for 16 tokens of a query head
  const int64_t pieces = (static_cast<int64_t>(p->num_tokens) / p->page_size + 2ll * p->num_seqs) * 2 * p->num_heads_kv;
  const int64_t tiles = p->q != nullptr ? (static_cast<int64_t>(p->num_tokens) / 16 + 1) * p->num_heads_q : 0;
  if (pieces + tiles > INT32_MAX) return QPKV_ERR_UNSUPPORTED;
  if (p->cu_seqlens_q == nullptr || p->block_table == nullptr || p->k == nullptr || p->v == nullptr ||
      p->k_pool == nullptr || p->v_pool == nullptr)
    return QPKV_ERR_INVALID_ARG;
  if (!aligned(p->k, 16) || !aligned(p->v, 16) || !aligned(p->q, 16) || !aligned(p->q_out, 16) ||
      !aligned(p->k_pool, 16) || !aligned(p->v_pool, 16) || !aligned(p->k_bounds, 16) || !aligned(p->rope_cos, 16) ||
      !aligned(p->rope_sin, 16) || !aligned(p->bound_scale, 4) || !aligned(p->k_mul, 4) || !aligned(p->v_mul, 4) ||
      !strides_fit(p->k_stride_t, p->k_stride_h) || !strides_fit(p->v_stride_t, p->v_stride_h) ||
      (p->q != nullptr && (!strides_fit(p->q_stride_t, p->q_stride_h) || !strides_fit(p->q_out_stride_t, p->q_out_stride_h))))
    return QPKV_ERR_INVALID_ARG;
  qpkv_write_group4_params w = *p;
  if (w.error_word == nullptr && (w.error_word = default_error_word()) == nullptr) return QPKV_ERR_CUDA;
  return launched(launch_write_group4(w, static_cast<cudaStream_t>(stream)));
}

qpkv_status qpkv_read_group4(const qpkv_read_group4_params* p, void* stream) {
  if (p == nullptr || p->num_seqs < 0 || p->num_tokens < 0) return QPKV_ERR_INVALID_ARG;
  const qpkv_status st = check_cache(p->head_dim, p->page_size, p->num_pages, p->bt_stride, p->num_heads_kv, p->dtype);
  if (st != QPKV_OK) return st;
  if ((static_cast<int64_t>(p->num_tokens) / 16 + 1) * 2 * p->num_heads_kv > INT32_MAX) return QPKV_ERR_UNSUPPORTED;
  if (p->num_seqs == 0 || p->num_tokens == 0 || (p->k_out == nullptr && p->v_out == nullptr)) return QPKV_OK;
  if (p->cu_seqlens_q == nullptr || p->block_table == nullptr || (p->k_out != nullptr && p->k_pool == nullptr) ||
      (p->v_out != nullptr && p->v_pool == nullptr))
    return QPKV_ERR_INVALID_ARG;
  if (!aligned(p->k_pool, 16) || !aligned(p->v_pool, 16) || !aligned(p->k_out, 16) || !aligned(p->v_out, 16) ||
      !aligned(p->k_mul, 4) || !aligned(p->v_mul, 4))
    return QPKV_ERR_INVALID_ARG;
  qpkv_read_group4_params w = *p;
  if (w.error_word == nullptr && (w.error_word = default_error_word()) == nullptr) return QPKV_ERR_CUDA;
  return launched(launch_read_group4(w, static_cast<cudaStream_t>(stream)));
}

qpkv_status qpkv_select_pages(const qpkv_select_pages_params* p, void* stream) {
  if (p == nullptr || p->num_seqs < 0 || p->num_tokens < 0 || p->num_heads_q < 1 || p->window < 0 || p->first < 0 ||
      p->last < 1 || p->num_selected < 1 || static_cast<int64_t>(p->first) + p->last > p->num_selected)
    return QPKV_ERR_INVALID_ARG;
  const qpkv_status st = check_cache(p->head_dim, p->page_size, p->num_pages, p->bt_stride, p->num_heads_kv, p->dtype);
  if (st != QPKV_OK) return st;
  if (!heads_fit(p->num_heads_q, p->num_heads_kv, p->num_tokens) || p->num_heads_q / p->num_heads_kv > 128 ||
      p->bt_stride > kSelectMaxPages || static_cast<int64_t>(p->num_tokens) * p->num_heads_kv * 8 > INT32_MAX ||
      static_cast<int64_t>(p->num_tokens) * p->num_heads_kv * p->num_selected > INT32_MAX)
    return QPKV_ERR_UNSUPPORTED;
  if (p->num_seqs == 0 || p->num_tokens == 0) return QPKV_OK;
  if (p->cu_seqlens_q == nullptr || p->seqlens_kv == nullptr || p->block_table == nullptr || p->q == nullptr ||
      p->k_bounds == nullptr || p->bound_scale == nullptr || p->selected == nullptr)
    return QPKV_ERR_INVALID_ARG;
  if (!aligned(p->q, 16) || !aligned(p->k_bounds, 16) || !aligned(p->bound_scale, 4) || !aligned(p->selected, 4))
    return QPKV_ERR_INVALID_ARG;
  qpkv_select_pages_params w = *p;
  if (w.error_word == nullptr && (w.error_word = default_error_word()) == nullptr) return QPKV_ERR_CUDA;
  return launched(launch_select_pages(w, static_cast<cudaStream_t>(stream)));
}

size_t qpkv_attend_group4_workspace_bytes(int32_t num_seqs, int32_t num_tokens, int32_t num_heads_q,
                                          int32_t num_heads_kv, int32_t head_dim) {
  if (num_seqs < 0 || num_tokens < 0 || num_heads_q < 1 || num_heads_kv < 1 ||
      num_heads_q % num_heads_kv != 0 || (head_dim != 64 && head_dim != 128))
    return 0;
  return attend_group4_workspace_bytes(num_seqs, num_tokens, num_heads_q, num_heads_kv, head_dim);
}

qpkv_status qpkv_attend_group4(const qpkv_attend_group4_params* p, void* stream) {
  if (p == nullptr || p->num_seqs < 0 || p->num_tokens < 0 || p->num_heads_q < 1 || p->window < 0 ||
      !(p->logit_cap >= 0.f) || !std::isfinite(p->sm_scale) ||
      // its reciprocal times a score must stay finite.  At the other end the products' factor over the
      // cap falls below float32's normal numbers; its error of 2^-150, times a product below 2^34,
      // times this cap is 2^-49 of a score, and at 1e38, beside an infinite cap * log2(e), 2^10
      (p->logit_cap > 0.f && p->logit_cap < 1e-20f) || p->logit_cap > 1e20f ||
      (p->selected != nullptr && p->num_selected < 1))
    return QPKV_ERR_INVALID_ARG;
  const qpkv_status st = check_cache(p->head_dim, p->page_size, p->num_pages, p->bt_stride, p->num_heads_kv, p->dtype);
  if (st != QPKV_OK) return st;
  if (!heads_fit(p->num_heads_q, p->num_heads_kv, p->num_tokens)) return QPKV_ERR_UNSUPPORTED;
  // blocks of 16 tokens of the pools, and units of a listed task
  if (static_cast<int64_t>(p->num_pages) * p->num_heads_kv > INT32_MAX / (p->page_size / 16)) return QPKV_ERR_UNSUPPORTED;
  if (p->selected != nullptr &&
      (static_cast<int64_t>(p->num_selected) * p->page_size > INT32_MAX - 64 ||
       static_cast<int64_t>(p->num_tokens) * p->num_heads_q > INT32_MAX))
    return QPKV_ERR_UNSUPPORTED;
  if (p->num_seqs == 0 || p->num_tokens == 0) return QPKV_OK;
  if (p->cu_seqlens_q == nullptr || p->seqlens_kv == nullptr || p->block_table == nullptr || p->q == nullptr ||
      p->k_pool == nullptr || p->v_pool == nullptr || p->o == nullptr)
    return QPKV_ERR_INVALID_ARG;
  if (!aligned(p->q, 16) || !aligned(p->k_pool, 16) || !aligned(p->v_pool, 16) || !aligned(p->o, 16) ||
      !aligned(p->workspace, 16) || !aligned(p->k_mul, 4) || !aligned(p->v_mul, 4) || !aligned(p->lse, 4) ||
      !aligned(p->selected, 4) || !aligned(p->alibi_slopes, 4) || !aligned(p->prefix_lens, 4))
    return QPKV_ERR_INVALID_ARG;
  if (attend_group4_needs_workspace(*p) &&
      (p->workspace == nullptr ||
       p->workspace_bytes < qpkv_attend_group4_workspace_bytes(p->num_seqs, p->num_tokens, p->num_heads_q,
                                                               p->num_heads_kv, p->head_dim)))
    return QPKV_ERR_WORKSPACE_TOO_SMALL;
  qpkv_attend_group4_params w = *p;
  if (w.error_word == nullptr && (w.error_word = default_error_word()) == nullptr) return QPKV_ERR_CUDA;
  if (!(w.sm_scale > 0.f)) w.sm_scale = 1.f / std::sqrt(static_cast<float>(w.head_dim));
  return launched(launch_attend_group4(w, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
