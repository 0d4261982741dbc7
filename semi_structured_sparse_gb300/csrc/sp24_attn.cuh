// sp24_attn.cuh -- what the attention entry points share: the checks of a
// paged cache, the part of its description that kernels take, and which keys
// a query sees.
#pragma once
#include <cmath>
#include <cstdint>
#include "sp24_internal.cuh"

namespace sp24 {

// The cache as kernels see it.  Offsets are 64-bit: a cache may well hold more
// than 2^31 elements.
struct CacheView {
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  int64_t page_stride, head_stride, token_stride;  // bytes
  int num_pages;
  int page_shift;  // page_size = 1 << page_shift
};

inline sp24_status check_cache(const sp24_kv_cache* c, CacheView* out) {
  if (!c || !c->k || !c->v) return SP24_ERR_INVALID_ARG;
  if (c->heads < 1 || c->num_pages < 1 || c->num_pages > INT32_MAX) return SP24_ERR_INVALID_ARG;
  if (c->dtype != SP24_BF16 && c->dtype != SP24_E4M3) return SP24_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128) return SP24_ERR_UNSUPPORTED;
  int shift = 4;
  while (shift < 7 && (1 << shift) != c->page_size) ++shift;
  if ((1 << shift) != c->page_size) return SP24_ERR_UNSUPPORTED;
  const bool e4m3 = c->dtype == SP24_E4M3;
  if (e4m3 != (c->k_scale != nullptr) || e4m3 != (c->v_scale != nullptr)) return SP24_ERR_INVALID_ARG;
  const int64_t e = e4m3 ? 1 : 2, most = int64_t(1) << 40;
  for (int64_t s : {c->page_stride, c->head_stride, c->token_stride}) {
    if (s <= 0 || s >= most / e) return SP24_ERR_INVALID_ARG;
    if (s * e % 16 != 0) return SP24_ERR_ALIGNMENT;
  }
  if (c->token_stride < c->head_dim) return SP24_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v)) return SP24_ERR_ALIGNMENT;
  out->k = static_cast<const uint8_t*>(c->k);
  out->v = static_cast<const uint8_t*>(c->v);
  out->k_scale = c->k_scale;
  out->v_scale = c->v_scale;
  out->page_stride = c->page_stride * e;
  out->head_stride = c->head_stride * e;
  out->token_stride = c->token_stride * e;
  out->num_pages = static_cast<int>(c->num_pages);
  out->page_shift = shift;
  return SP24_OK;
}

// Tokens of a sequence, and rows of a call, at most: positions, and their
// differences, stay within 32 bits.
constexpr int kMostTokens = (1 << 30) - 1;
// A window that no sequence fills is none.
inline int effective_window(int window) { return window > kMostTokens ? 0 : window; }

// What decode and prompt calls have in common.
inline sp24_status check_attention(const void* q, int64_t rows, int64_t ldq, int q_heads, const sp24_kv_cache* c,
                                   const int32_t* page_table, int64_t table_width, int64_t ld_table,
                                   const int32_t* seq_lens, int64_t B, float scale, int window, int sinks,
                                   const void* Y, int64_t ldy, CacheView* out) {
  if (rows < 0 || rows > kMostTokens || B < 0 || B > kMostTokens) return SP24_ERR_INVALID_ARG;
  if (sp24_status st = check_cache(c, out)) return st;
  if (q_heads < 1 || q_heads % c->heads != 0) return SP24_ERR_INVALID_ARG;
  if (q_heads / c->heads > 128) return SP24_ERR_UNSUPPORTED;
  const int64_t width = int64_t(q_heads) * c->head_dim;
  if (!(scale > 0.0f) || !std::isfinite(scale) || window < 0 || sinks < 0) return SP24_ERR_INVALID_ARG;
  if (rows > 0 && B > 0) {
    if (!q || !Y || !page_table || !seq_lens) return SP24_ERR_INVALID_ARG;
    if (ldq < width || ldy < width || ldq >= (int64_t(1) << 39) || ldy >= (int64_t(1) << 39))
      return SP24_ERR_INVALID_ARG;
    if (table_width < 1 || ld_table < table_width || table_width > (kMostTokens >> out->page_shift))
      return SP24_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(Y) || ldq % 8 || ldy % 8) return SP24_ERR_ALIGNMENT;
    if ((reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(seq_lens)) & 3u)
      return SP24_ERR_ALIGNMENT;
  }
  return SP24_OK;
}

}  // namespace sp24
