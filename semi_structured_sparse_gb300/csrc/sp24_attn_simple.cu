// sp24_attn_simple.cu -- sp24_attention_prompt the plain
// way: one warp per query row and head, one key at a time.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include "sp24_attn.cuh"
#include "sp24_ptx.cuh"

namespace sp24 {
namespace {

struct SimpleParams {
  const __nv_bfloat16* q;
  int64_t ldq;
  const int32_t* cu_q;  // NULL: one row per sequence
  int B, T;
  CacheView cache;
  const int32_t* page_table;
  int table_width;
  int64_t ld_table;
  const int32_t* seq_lens;
  float scale;
  int window, sinks;
  __nv_bfloat16* y;
  int64_t ldy;
  int q_heads, group, D;
  bool e4m3;
  unsigned int* err;
};

__device__ float load_value(const uint8_t* p, int i, bool e4m3) {
  if (e4m3) {
    __nv_fp8_e4m3 v;
    v.__x = p[i];
    return float(v);
  }
  return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}

__global__ void simple_attention_kernel(const __grid_constant__ SimpleParams p) {
  pdl_wait();
  const int row = blockIdx.x, lane = threadIdx.x;
  int b = row, i = 0, m = 1;
  if (p.cu_q) {
    for (b = 0; b < p.B && p.cu_q[b + 1] <= row; ++b) {
    }
    if (b == p.B || row < p.cu_q[b]) return;
    i = row - p.cu_q[b];
    m = p.cu_q[b + 1] - p.cu_q[b];
  }
  const int page_size = 1 << p.cache.page_shift;
  int n = p.seq_lens[b];
  if (n < 0 || n > p.table_width * page_size) {
    if (lane == 0) atomicOr(p.err, DEVERR_INDEX);
    n = n < 0 ? 0 : p.table_width * page_size;
  }
  const int pos = n - m + i;
  const int per = p.D / 32;
  for (int h = blockIdx.y; h < p.q_heads; h += gridDim.y) {
    const int hk = h / p.group;
    const float ks = p.e4m3 ? p.cache.k_scale[hk] : 1.0f, vs = p.e4m3 ? p.cache.v_scale[hk] : 1.0f;
    float q[4], acc[4] = {0, 0, 0, 0}, top = -INFINITY, sum = 0.0f;
    for (int d = 0; d < per; ++d) q[d] = __bfloat162float(p.q[row * p.ldq + h * p.D + lane + 32 * d]);
    for (int j = 0; j <= pos; ++j) {
      if (p.window && j <= pos - p.window && j >= p.sinks) {
        j = pos - p.window;  // the next visible key is the window's first
        continue;
      }
      int page = p.page_table[b * p.ld_table + (j >> p.cache.page_shift)];
      if (page < 0 || page >= p.cache.num_pages) {
        if (lane == 0) atomicOr(p.err, DEVERR_INDEX);
        page = 0;
      }
      const int64_t at = page * p.cache.page_stride + hk * p.cache.head_stride +
                         (j & (page_size - 1)) * p.cache.token_stride;
      float s = 0.0f;
      for (int d = 0; d < per; ++d) s = fmaf(q[d], load_value(p.cache.k + at, lane + 32 * d, p.e4m3), s);
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      s *= p.scale * ks;
      const float now = fmaxf(top, s), keep = expf(top - now), e = expf(s - now);
      sum = fmaf(sum, keep, e);
      for (int d = 0; d < per; ++d)
        acc[d] = fmaf(acc[d], keep, e * load_value(p.cache.v + at, lane + 32 * d, p.e4m3));
      top = now;
    }
    for (int d = 0; d < per; ++d)
      p.y[row * p.ldy + h * p.D + lane + 32 * d] = __float2bfloat16(sum == 0.0f ? 0.0f : acc[d] * vs / sum);
  }
}

sp24_status run_simple(const SimpleParams& p, int rows, cudaStream_t s) {
  const dim3 grid(rows, p.q_heads < 65535 ? p.q_heads : 65535);
  return launch_pdl(simple_attention_kernel, grid, dim3(32), 0, s, p) == cudaSuccess ? SP24_OK : SP24_ERR_CUDA;
}

}  // namespace
}  // namespace sp24

extern "C" sp24_status sp24_attention_prompt(const void* q, int64_t T, int64_t ldq, int q_heads, const int32_t* cu_q,
                                             int64_t B, const sp24_kv_cache* cache, const int32_t* page_table,
                                             int64_t table_width, int64_t ld_table, const int32_t* seq_lens,
                                             float scale, int window, int sinks, void* Y, int64_t ldy, void* stream) {
  using namespace sp24;
  SimpleParams p = {};
  if (sp24_status st = check_attention(q, T, ldq, q_heads, cache, page_table, table_width, ld_table, seq_lens, B, scale,
                                       window, sinks, Y, ldy, &p.cache))
    return st;
  if (T > 0 && B > 0 && !cu_q) return SP24_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(cu_q) & 3u) return SP24_ERR_ALIGNMENT;
  const DeviceInfo* dev = nullptr;
  if (sp24_status st = current_device(&dev)) return st;
  if (T == 0 || B == 0) return SP24_OK;
  p.q = static_cast<const __nv_bfloat16*>(q), p.ldq = ldq, p.cu_q = cu_q, p.B = int(B), p.T = int(T);
  p.page_table = page_table, p.table_width = int(table_width), p.ld_table = ld_table, p.seq_lens = seq_lens;
  p.scale = scale, p.window = window, p.sinks = sinks, p.y = static_cast<__nv_bfloat16*>(Y), p.ldy = ldy;
  p.q_heads = q_heads, p.group = q_heads / cache->heads, p.D = cache->head_dim, p.e4m3 = cache->dtype == SP24_E4M3;
  p.err = dev->err_word;
  return run_simple(p, int(T), static_cast<cudaStream_t>(stream));
}
