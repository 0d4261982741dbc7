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

// ---------------------------------------------------------- shared first tokens
// sp24_attention_decode_shared in three launches: the prompt kernel attends the
// shared tokens of each group for all of its sequences' queries at once, the
// decode kernel each sequence's own tokens; both leave maxima, sums and weighted values
// in the workspace, which the third launch adds up.  What they know of the groups:
struct SharedGroups {
  const int32_t* cu;    // [G + 1]
  const int32_t* lens;  // [G]
  int G;
  int2* where;          // [sequences][kv heads] {row of its first head in the first piece, how many pieces}
  float* part;          // [parts][2 kTileRows][D] weighted values, then [parts][2 kTileRows][2] maxima and sums
  int pairs, parts;     // how many there is room for
  int window, sinks;    // of the call
  float* own;           // [sequences][query heads][D] and then [2]: the same of a sequence's own tokens, with
                        // kNotShared for the sum of weights where there is nothing to add
};
constexpr float kNotShared = -1.0f;
constexpr int kTileRows = 128;          // query rows of a tile of the prompt kernel; two tiles are a block
constexpr int kKeyTile = 128;           // keys of one of its tiles
// Weights of an e4m3 cache are 2^this times exp2(c S - m) in the kernels for prompts and for decoding.
constexpr float kPromptUp = 7.0f, kDecodeUp = 15.0f;

// The tokens that a group [lo, hi) of sequences reads together: none if it is
// one sequence, or if its first, through whose pages they are read, does not see all of its
// own (the entries of pages before its window may be anything); and no more than that one has.
__device__ __forceinline__ int shared_tokens(const SharedGroups& s, int lo, int hi, int shared, const int32_t* seq_lens,
                                             int most) {
  if (hi - lo < 2) return 0;
  const int n = min(__ldg(seq_lens + lo), most);
  return s.window > 0 && n > s.window && n - s.window > s.sinks ? 0 : max(0, min(shared, n));
}
// How many first tokens sequence b of B reads together with its group.
__device__ __forceinline__ int shared_of(const SharedGroups& s, int b, int B, const int32_t* seq_lens, int most) {
  int g = 0, end = s.G;
  while (end - g > 1) {  // the last group that begins at b or before
    const int mid = (g + end) / 2;
    if (__ldg(s.cu + mid) <= b) g = mid; else end = mid;
  }
  const int lo = max(__ldg(s.cu + g), 0), hi = min(__ldg(s.cu + g + 1), B);
  return b < lo || b >= hi ? 0 : shared_tokens(s, lo, hi, __ldg(s.lens + g), seq_lens, most);
}
// Tokens that sequence b reads one by one, as far as they take a share of the SMs.  Without a window those that its group
// reads together are among them: they are taken off for a group at once, which takes fewer loads (and only a sequence
// shorter than them does not share them).  Under a window some of a group may see all of them and others not: what the
// latter read of them is in L2, at 76 bytes per ns and SM (attention_decode of 64 sequences behind the same 16000 tokens,
// 363 us), and counts 7/16.  (Window 16384, of those 64 2 share: 373 us, 716 with a count of 1, 520 without any; 32 share:
// 219, 485, 330; 62: 54, 60, 86.)
__device__ __forceinline__ int counted_tokens(const SharedGroups& s, int b, int B, const int32_t* seq_lens, int most) {
  const int n = max(0, min(__ldg(seq_lens + b), most));
  if (s.window == 0) return n;
  const int shared = shared_of(s, b, B, seq_lens, most);
  if (n <= s.window || n - s.window <= s.sinks) return shared <= n ? n - shared : n;
  const int near = max(0, shared - (n - s.window)) + min(s.sinks, shared);
  return s.window + s.sinks - near + near / 16 * 7;  // (less than n)
}

// How many of the SMs should do the shared tokens: the others begin with the
// sequences' own at once, so that one's idle memory is the other's.  Both launches
// ask, and get the same answer: shares of the SMs as those of the work, of units
// (key tiles of up to 256 query rows), which the chain of products and
// exponentials bounds, and of the bytes of own keys and values.  `tokens`: the counted ones of all sequences, without a
// window less those that their groups read together.
// Fewer, and the shared tokens take them all first.  (200 sequences behind 20000 tokens, 28/4 heads of 64, e4m3: up to 1000
// of their own 74 us, 81 with 25; up to 100 59 us, 289 with 1.  64 behind 16000, up to 130, 32/8 heads of 128: 36.6 us, 42.5 with 60.)
constexpr unsigned int kLeastOwnSms = 40;
template <int D, bool E4M3>
__device__ __forceinline__ unsigned int shared_sms(unsigned int units, long long tokens, int kv_heads, unsigned int sms) {
  // (e4m3, heads of 64: those 200 with up to 1000 and 3000 of their own 73.9 and 84.2 us, with 1150 69.5 and 86.0, with 1700
  // 74.1 and 90.6.)
  constexpr float UNIT_NS = D == 128 ? (E4M3 ? 1650.0f : 1350.0f) : (E4M3 ? 1400.0f : 1150.0f);
  // That an SM's decode CTAs read.  (64 sequences behind 16000 tokens with up to 512 and 250 of their own, 96 in 6 groups with an
  // e4m3 cache: 44.3, 38.1 and 89.0 us; with 28 45.5, 38.3 and 93.0, with 36 43.6, 41.3 and 89.1, with 40 44.4, 41.3 and 92.9.)
  constexpr float BYTES_PER_NS = 32.0f;
  if (units == 0) return 0;
  const float bytes = static_cast<float>(max(tokens, 0ll)) * (kv_heads * D * (E4M3 ? 2 : 4));
  const float shared = units * UNIT_NS, own = bytes / BYTES_PER_NS;
  const unsigned int busy = max(1u, min(sms, static_cast<unsigned int>(sms * (shared / (shared + own)) + 0.999f)));
  return sms - busy < kLeastOwnSms ? sms : busy;
}

// A call, as the entry point hands it to both launches.
struct SharedCall {
  const void* q;
  int64_t ldq;
  int B, q_heads;
  const sp24_kv_cache* cache;
  CacheView view;
  const int32_t* page_table;
  int table_width;
  int64_t ld_table;
  const int32_t* seq_lens;
  float scale;
  int window, sinks;
  void* y;
  int64_t ldy;
  SharedGroups groups;
  void* decode_workspace;
};
sp24_status launch_shared_tokens(const SharedCall& c, const DeviceInfo& dev, cudaStream_t s);  // sp24_attn_prompt.cu
sp24_status launch_own_tokens(const SharedCall& c, const DeviceInfo& dev, cudaStream_t s);     // sp24_attn_decode.cu
size_t decode_workspace_bytes(const DeviceInfo& dev, int q_heads, int heads, int head_dim);    // sp24_attn_decode.cu

}  // namespace sp24
