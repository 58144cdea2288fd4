// The extern "C" boundary of the serving step on the device: argument checks
// and dispatch.  No exception leaves this file; no allocation, free or
// synchronisation happens here.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "internal.h"

namespace qpkv {
namespace {

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

qpkv_status launched(cudaError_t e) { return e == cudaSuccess ? QPKV_OK : QPKV_ERR_CUDA; }

// What the write and the attention ask of the pools.
qpkv_status check_pools(int D, int ps, int P, int bt_stride, int Hkv, int dtype, int format, int layout) {
  if (Hkv < 1 || P < 1 || bt_stride < 1 || ps < 1) return QPKV_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || ps % 16 != 0) return QPKV_ERR_UNSUPPORTED;
  if (dtype != QPKV_DTYPE_BF16 && dtype != QPKV_DTYPE_F16) return QPKV_ERR_UNSUPPORTED;
  if (format != QPKV_FORMAT_E4M3 && format != QPKV_FORMAT_INT8) return QPKV_ERR_UNSUPPORTED;
  if (layout != QPKV_KV_LAYOUT_NHD && layout != QPKV_KV_LAYOUT_HND) return QPKV_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(bt_stride) * ps > INT32_MAX - 64) return QPKV_ERR_UNSUPPORTED;
  return QPKV_OK;
}

}  // namespace
}  // namespace qpkv

using namespace qpkv;

extern "C" {

qpkv_status qpkv_assign_pages(const qpkv_assign_params* p, void* stream) {
  if (p == nullptr || p->num_seqs < 1 || p->num_tokens < 0 || p->page_size < 1 || p->num_pages < 1 ||
      p->bt_stride < 1 || p->num_free < 0)
    return QPKV_ERR_INVALID_ARG;
  if (p->new_lens == nullptr || p->seqlens == nullptr || p->block_table == nullptr ||
      p->free_count == nullptr || p->block_table_out == nullptr || p->seqlens_out == nullptr ||
      p->free_count_out == nullptr || p->cu_seqlens == nullptr ||
      (p->num_free > 0 && p->free_pages == nullptr) ||
      (p->num_tokens > 0 && (p->slot_mapping == nullptr || p->positions == nullptr)))
    return QPKV_ERR_INVALID_ARG;
  const int64_t most = static_cast<int64_t>(INT32_MAX) - p->page_size;
  if (p->num_seqs > kAssignMaxSeqs || static_cast<int64_t>(p->bt_stride) * p->page_size > most ||
      static_cast<int64_t>(p->num_pages) * p->page_size > most)
    return QPKV_ERR_UNSUPPORTED;
  qpkv_assign_params w = *p;
  if (w.error_word == nullptr && (w.error_word = default_error_word()) == nullptr)
    return QPKV_ERR_CUDA;
  return launched(launch_assign_pages(w, static_cast<cudaStream_t>(stream)));
}

qpkv_status qpkv_rope_axes(const qpkv_rope_axes_params* p, void* stream) {
  if (p == nullptr || p->num_tokens < 0 || p->num_heads_q < 1 || p->head_dim < 1 || p->rot_dim < 1 ||
      p->rope_max_pos < 1 || (p->k != nullptr && p->num_heads_kv < 1))
    return QPKV_ERR_INVALID_ARG;
  if (p->num_axes < 1 || p->num_axes > 4 || p->rot_dim % 2 != 0 || p->rot_dim > p->head_dim ||
      p->rot_dim > 256 || p->dtype < QPKV_DTYPE_BF16 || p->dtype > QPKV_DTYPE_F32)
    return QPKV_ERR_UNSUPPORTED;
  if (p->pair_axis == nullptr) return QPKV_ERR_INVALID_ARG;
  for (int i = 0; i < p->rot_dim / 2; ++i)
    if (p->pair_axis[i] >= p->num_axes) return QPKV_ERR_INVALID_ARG;
  if (p->num_tokens == 0) return QPKV_OK;
  if (p->positions == nullptr || p->rope_cos == nullptr || p->rope_sin == nullptr || p->q == nullptr ||
      p->q_out == nullptr || (p->k != nullptr && p->k_out == nullptr))
    return QPKV_ERR_INVALID_ARG;
  const uintptr_t es = p->dtype == QPKV_DTYPE_F32 ? 4 : 2;
  if (!aligned(p->q, es) || !aligned(p->q_out, es) || !aligned(p->k, es) || !aligned(p->k_out, es) ||
      !aligned(p->rope_cos, 4) || !aligned(p->rope_sin, 4) || !aligned(p->positions, 4))
    return QPKV_ERR_INVALID_ARG;
  qpkv_rope_axes_params w = *p;
  if (w.error_word == nullptr && (w.error_word = default_error_word()) == nullptr)
    return QPKV_ERR_CUDA;
  return launched(launch_rope_axes(w, static_cast<cudaStream_t>(stream)));
}

qpkv_status qpkv_write_page8(const qpkv_write_page8_params* p, void* stream) {
  if (p == nullptr || p->num_seqs < 0 || p->num_tokens < 0) return QPKV_ERR_INVALID_ARG;
  const qpkv_status st = check_pools(p->head_dim, p->page_size, p->num_pages, p->bt_stride,
                                     p->num_heads_kv, p->dtype, p->format, p->kv_layout);
  if (st != QPKV_OK) return st;
  if (p->num_heads_kv > 65535) return QPKV_ERR_UNSUPPORTED;
  if (p->num_seqs == 0 || p->num_tokens == 0) return QPKV_OK;
  // two blocks at most for a (piece, head)
  if ((static_cast<int64_t>(p->num_tokens) / p->page_size + 2ll * p->num_seqs) * 2 * p->num_heads_kv > INT32_MAX)
    return QPKV_ERR_UNSUPPORTED;
  if (p->cu_seqlens_q == nullptr || p->block_table == nullptr || p->k == nullptr || p->v == nullptr ||
      p->k_pool == nullptr || p->v_pool == nullptr || p->k_scale == nullptr || p->v_scale == nullptr)
    return QPKV_ERR_INVALID_ARG;
  if (!aligned(p->k, 16) || !aligned(p->v, 16) || !aligned(p->k_pool, 16) || !aligned(p->v_pool, 16) ||
      !aligned(p->k_scale, 4) || !aligned(p->v_scale, 4) || p->k_stride_t % 8 || p->k_stride_h % 8 ||
      p->v_stride_t % 8 || p->v_stride_h % 8)
    return QPKV_ERR_INVALID_ARG;
  qpkv_write_page8_params w = *p;
  if (w.error_word == nullptr && (w.error_word = default_error_word()) == nullptr)
    return QPKV_ERR_CUDA;
  return launched(launch_write_page8(w, static_cast<cudaStream_t>(stream)));
}

size_t qpkv_attend_page8_workspace_bytes(int32_t num_seqs, int32_t num_tokens, int32_t num_heads_q,
                                         int32_t num_heads_kv, int32_t head_dim) {
  if (num_seqs < 0 || num_tokens < 0 || num_heads_q < 1 || num_heads_kv < 1 ||
      num_heads_q % num_heads_kv != 0 || (head_dim != 64 && head_dim != 128))
    return 0;
  return attend_page8_workspace_bytes(num_seqs, num_tokens, num_heads_q, num_heads_kv, head_dim);
}

qpkv_status qpkv_attend_page8(const qpkv_attend_page8_params* p, void* stream) {
  if (p == nullptr || p->num_seqs < 0 || p->num_tokens < 0 || p->num_heads_q < 1 || p->window < 0 ||
      !(p->logit_cap >= 0.f) || p->logit_cap > 2.3e38f || !std::isfinite(p->sm_scale) ||
      (p->logit_cap > 0.f && p->logit_cap < 1e-20f))   // its reciprocal times a score, and it times log2(e), must stay finite
    return QPKV_ERR_INVALID_ARG;
  const qpkv_status st = check_pools(p->head_dim, p->page_size, p->num_pages, p->bt_stride,
                                     p->num_heads_kv, p->dtype, p->format, p->kv_layout);
  if (st != QPKV_OK) return st;
  if (p->num_heads_q % p->num_heads_kv != 0 ||
      static_cast<int64_t>(p->num_tokens) * (p->num_heads_q / p->num_heads_kv) > INT32_MAX - 64 ||
      static_cast<int64_t>(p->num_tokens) * p->num_heads_q > 4ll * INT32_MAX)
    return QPKV_ERR_UNSUPPORTED;
  const int64_t rows = static_cast<int64_t>(p->num_pages) * p->page_size;   // of a pool, as TMA counts them
  if (rows > (p->kv_layout == QPKV_KV_LAYOUT_HND ? INT32_MAX / p->num_heads_kv : INT32_MAX))
    return QPKV_ERR_UNSUPPORTED;
  if (p->num_seqs == 0 || p->num_tokens == 0) return QPKV_OK;
  if (p->cu_seqlens_q == nullptr || p->seqlens_kv == nullptr || p->block_table == nullptr ||
      p->q == nullptr || p->k_pool == nullptr || p->v_pool == nullptr || p->k_scale == nullptr ||
      p->v_scale == nullptr || p->o == nullptr || p->workspace == nullptr)
    return QPKV_ERR_INVALID_ARG;
  if (!aligned(p->q, 16) || !aligned(p->k_pool, 16) || !aligned(p->v_pool, 16) || !aligned(p->o, 16) ||
      !aligned(p->workspace, 16) || !aligned(p->k_scale, 4) || !aligned(p->v_scale, 4) || !aligned(p->lse, 4))
    return QPKV_ERR_INVALID_ARG;
  if (p->workspace_bytes < qpkv_attend_page8_workspace_bytes(p->num_seqs, p->num_tokens, p->num_heads_q,
                                                             p->num_heads_kv, p->head_dim))
    return QPKV_ERR_WORKSPACE_TOO_SMALL;
  qpkv_attend_page8_params w = *p;
  if (w.error_word == nullptr && (w.error_word = default_error_word()) == nullptr)
    return QPKV_ERR_CUDA;
  if (!(w.sm_scale > 0.f)) w.sm_scale = 1.f / std::sqrt(static_cast<float>(w.head_dim));
  return launched(launch_attend_page8(w, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
