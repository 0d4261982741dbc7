// sp24_attn_shared.cu -- sp24_attention_decode_shared: one new token per
// sequence over the paged cache, where groups of sequences have their first
// tokens in common.
//
//   Y[h] = sum_j p_j v_j / sum_j p_j,  p_j = exp2(c (q_h . k_j) - m_h),
//   c = scale log2(e) (times the cache's scale), m_h the running maximum
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "sp24_attn.cuh"
#include "sp24_ptx.cuh"

namespace sp24 {
namespace {

struct SharedParams {
  const __nv_bfloat16* q;
  int64_t ldq;
  int B, G;
  CacheView cache;
  const int32_t* page_table;
  int table_width;
  int64_t ld_table;
  const int32_t* seq_lens;
  const int32_t* cu_shared;
  const int32_t* shared_lens;
  float scale;
  int window, sinks;
  __nv_bfloat16* y;
  int64_t ldy;
  int q_heads, group;
  unsigned int* err;
};

// A warp per sequence and query head.
template <int D, bool E4M3>
__global__ void __launch_bounds__(32) attention_decode_shared_kernel(const __grid_constant__ SharedParams p) {
  constexpr int PL = D / 32;  // dims per lane
  const int lane = threadIdx.x, b = blockIdx.x, h = blockIdx.y, hk = h / p.group;
  pdl_wait();
  int n = p.seq_lens[b];
  const int most = p.table_width << p.cache.page_shift;
  if (n < 0 || n > most) {
    if (lane == 0) atomicOr(p.err, DEVERR_INDEX);
    n = n < 0 ? 0 : most;
  }
  // the group's first sequence, whose pages the shared tokens are read through, and their number
  int leader = b, shared = 0;
  if (lane == 0 && (p.cu_shared[0] < 0 || p.cu_shared[0] > p.B)) atomicOr(p.err, DEVERR_INDEX);
  for (int g = 0, end = min(max(p.cu_shared[0], 0), p.B); g < p.G; ++g) {
    const int lo = end, z = p.cu_shared[g + 1];
    end = min(max(z, lo), p.B);
    int s = p.shared_lens[g];
    if (s < 0 || s > most || z != end) {
      if (lane == 0) atomicOr(p.err, DEVERR_INDEX);
      s = s < 0 ? 0 : min(s, most);
    }
    if (b >= lo && b < end) leader = lo, shared = s;
  }
  const int from = p.window > 0 ? max(0, n - p.window) : 0, sinks = min(p.sinks, from);
  if (n < shared || from > 0) shared = 0;
  float q[PL], o[PL], m = -INFINITY, l = 0.0f;
  for (int i = 0; i < PL; ++i) {
    q[i] = __bfloat162float(p.q[b * p.ldq + int64_t(h) * D + lane * PL + i]);
    o[i] = 0.0f;
  }
  const float c = p.scale * 1.4426950408889634f * (E4M3 ? p.cache.k_scale[hk] : 1.0f);
  auto value = [&](const uint8_t* base, int64_t at, float (&x)[PL]) {
    for (int i = 0; i < PL; ++i) {
      if (E4M3) {
        const uint32_t two = e4m3x2_f16x2(base[at + lane * PL + i]);
        x[i] = __half2float(__ushort_as_half(static_cast<unsigned short>(two & 0xFFFF)));
      } else {
        x[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base + at)[lane * PL + i]);
      }
    }
  };
  for (int j = 0; j < n; ++j) {
    if (j >= sinks && j < from) j = from;
    int page = p.page_table[int64_t(j < shared ? leader : b) * p.ld_table + (j >> p.cache.page_shift)];
    if (page < 0 || page >= p.cache.num_pages) {
      if (lane == 0) atomicOr(p.err, DEVERR_INDEX);
      page = 0;
    }
    const int64_t at = page * p.cache.page_stride + hk * p.cache.head_stride +
                       (j & ((1 << p.cache.page_shift) - 1)) * p.cache.token_stride;
    float x[PL], s = 0.0f;
    value(p.cache.k, at, x);
    for (int i = 0; i < PL; ++i) s = fmaf(x[i], q[i], s);
    for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, k);
    s *= c;
    const float now = fmaxf(m, s), keep = ex2(m - now), w = ex2(s - now);
    m = now;
    l = fmaf(l, keep, w);
    value(p.cache.v, at, x);
    for (int i = 0; i < PL; ++i) o[i] = fmaf(x[i], w, o[i] * keep);
  }
  const float f = l == 0.0f ? 0.0f : (E4M3 ? p.cache.v_scale[hk] : 1.0f) / l;
  for (int i = 0; i < PL; ++i) p.y[b * p.ldy + int64_t(h) * D + lane * PL + i] = __float2bfloat16(o[i] * f);
  pdl_trigger();
}

}  // namespace
}  // namespace sp24

extern "C" size_t sp24_attention_decode_shared_workspace_size(int64_t B, int64_t G, int q_heads, int heads,
                                                              int head_dim) {
  using namespace sp24;
  if (B < 0 || B > kMostTokens || G < 0 || G > kMostTokens || q_heads < 1 || heads < 1 || q_heads % heads ||
      q_heads / heads > 128 || (head_dim != 64 && head_dim != 128))
    return 0;
  return 256;
}

extern "C" sp24_status sp24_attention_decode_shared(const void* q, int64_t B, int64_t ldq, int q_heads,
                                                    const sp24_kv_cache* cache, const int32_t* page_table,
                                                    int64_t table_width, int64_t ld_table, const int32_t* seq_lens,
                                                    const int32_t* cu_shared, const int32_t* shared_lens, int64_t G,
                                                    float scale, int window, int sinks, void* Y, int64_t ldy,
                                                    void* workspace, size_t workspace_bytes, void* stream) {
  using namespace sp24;
  SharedParams p = {};
  if (sp24_status st = check_attention(q, B, ldq, q_heads, cache, page_table, table_width, ld_table, seq_lens, B, scale,
                                       window, sinks, Y, ldy, &p.cache))
    return st;
  if (G < 0 || G > kMostTokens || !cu_shared || (G > 0 && !shared_lens)) return SP24_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(cu_shared) | reinterpret_cast<uintptr_t>(shared_lens)) & 3u) return SP24_ERR_ALIGNMENT;
  const DeviceInfo* dev = nullptr;
  if (sp24_status st = current_device(&dev)) return st;
  const size_t need = sp24_attention_decode_shared_workspace_size(B, G, q_heads, cache->heads, cache->head_dim);
  if (!workspace || workspace_bytes < need) return SP24_ERR_WORKSPACE;
  if (!aligned16(workspace)) return SP24_ERR_ALIGNMENT;
  if (B == 0) return SP24_OK;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.ldq = ldq;
  p.B = static_cast<int>(B);
  p.G = static_cast<int>(G);
  p.page_table = page_table;
  p.table_width = static_cast<int>(table_width);
  p.ld_table = ld_table;
  p.seq_lens = seq_lens;
  p.cu_shared = cu_shared;
  p.shared_lens = shared_lens;
  p.scale = scale;
  p.window = effective_window(window);
  p.sinks = sinks;
  p.y = static_cast<__nv_bfloat16*>(Y);
  p.ldy = ldy;
  p.q_heads = q_heads;
  p.group = q_heads / cache->heads;
  p.err = dev->err_word;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(B), static_cast<unsigned>(q_heads));
  const bool e4m3 = cache->dtype == SP24_E4M3;
  auto kern = cache->head_dim == 128
                  ? (e4m3 ? attention_decode_shared_kernel<128, true> : attention_decode_shared_kernel<128, false>)
                  : (e4m3 ? attention_decode_shared_kernel<64, true> : attention_decode_shared_kernel<64, false>);
  return launch_pdl(kern, grid, dim3(32), 0, s, p) == cudaSuccess ? SP24_OK : SP24_ERR_CUDA;
}
