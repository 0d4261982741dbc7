// sp24_attn_shared.cu -- sp24_attention_decode_shared: one new token per
// sequence over the paged cache, where groups of sequences have their first
// tokens in common.
//
// A softmax over shared and own keys is joined from the maxima, sums and
// weighted values of both.  The shared keys of a group are one matrix for the
// queries of all its sequences, so that part is a product of matrices: the
// prompt kernel's tensor-core tiles, with (sequence, head) pairs as rows, each
// pair of keys' and values' tiles read once for up to 256 of them.  The keys that are
// a sequence's own have one query per head: the decode kernel streams them.  It
// needs nothing of the first launch, so it begins on the SMs that this leaves
// idle and as it gets done.  A third launch adds a row's parts up, all loads of
// a row in one go.  (Added by the decode kernel's CTAs as their rows were complete, 64
// sequences behind 16000 tokens took 65 us: a chain of four latencies per item.)
//
// Measured (GB300, in a graph; 32/8 heads of 128): 64 sequences behind 16000 tokens, up to 512 of their
// own, bf16 43.9 us (132 MB: 3.0 TB/s; one by one 363 us); 96 in 6 groups behind up to 16000, e4m3 88.8 us;
// 200 behind 50001, 28/4 heads of 64 100.5 us.  Bound by the softmax warps of the shared tokens' launch, and by
// the own tokens' latencies on the other SMs.
#include <algorithm>
#include <cuda_bf16.h>
#include "sp24_attn.cuh"
#include "sp24_ptx.cuh"

namespace sp24 {
namespace {

// Blocks of rows that groups of B sequences have at most (each group's last may be partly
// filled), times the kv heads: pairs; a pair's keys are cut at most once per CTA.
struct Room {
  int64_t pairs, parts;
  size_t where, own, part, total;  // offsets behind the decode kernel's workspace
};
constexpr int64_t kLeastSaved = 32 << 20;  // bytes

// Sums of the prompt kernel times this are at the decode kernel's scale.
constexpr float kFromPrompt = 256.0f;
static_assert(kDecodeUp - kPromptUp == 8.0f, "");

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
Room room_for(int64_t B, int64_t G, int q_heads, int heads, int D, const DeviceInfo& dev) {
  Room r;
  const int64_t tokens = 2 * (kTileRows / (q_heads / heads));
  r.pairs = (B / tokens + std::min(B, G)) * heads;
  r.parts = r.pairs + dev.sm_count;
  r.where = up256(decode_workspace_bytes(dev, q_heads, heads, D));
  r.own = r.where + up256(static_cast<size_t>(B) * heads * sizeof(int2));
  r.part = r.own + up256(static_cast<size_t>(B) * q_heads * (D + 2) * sizeof(float));
  r.total = r.part + static_cast<size_t>(r.parts) * (2 * kTileRows) * (D + 2) * sizeof(float);
  return r;
}

// A row (a sequence's query head) per D / 4 lanes.
struct JoinParams {
  SharedGroups sh;
  int rows, q_heads, group, kv_heads;
  const float* v_scale;
  __nv_bfloat16* y;
  int64_t ldy;
};
constexpr int kJoinThreads = 128;
constexpr int kAhead = 8;  // pieces whose loads are in flight together
template <int D, bool E4M3>
__global__ void __launch_bounds__(kJoinThreads) attention_shared_join_kernel(const __grid_constant__ JoinParams p) {
  constexpr int LPR = D / 4;
  const int row = blockIdx.x * (kJoinThreads / LPR) + threadIdx.x / LPR, d = threadIdx.x % LPR * 4;
  pdl_wait();
  if (row < p.rows) {
    const int b = row / p.q_heads, h = row - b * p.q_heads, hk = h / p.group;
    const int2 at = __ldcg(p.sh.where + int64_t(b) * p.kv_heads + hk);
    float4 acc = __ldcg(reinterpret_cast<const float4*>(p.sh.own + int64_t(row) * D + d));
    const float2 own = __ldcg(reinterpret_cast<const float2*>(p.sh.own + int64_t(p.rows) * D + 2 * int64_t(row)));
    if (own.y != kNotShared) {
      float top = own.x, sum = own.y;
      // (Out of range is only what a first launch that gave up has not written.)
      const bool ok = at.x >= 0 && at.y > 0 && int64_t(at.x) + p.group + int64_t(at.y - 1) * (2 * kTileRows) <=
                                                   int64_t(p.sh.parts) * (2 * kTileRows);
      const int pieces = ok ? at.y : 0;
      const float* ml = p.sh.part + int64_t(p.sh.parts) * (2 * kTileRows * D);
      for (int i0 = 0; i0 < pieces; i0 += kAhead) {
        float4 v[kAhead];
        float2 w[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          v[i] = make_float4(0, 0, 0, 0);
          w[i] = make_float2(-INFINITY, 0.0f);
          if (i0 + i < pieces) {
            const int64_t r = at.x + h - hk * p.group + int64_t(i0 + i) * (2 * kTileRows);
            w[i] = __ldcg(reinterpret_cast<const float2*>(ml + 2 * r));
            v[i] = __ldcg(reinterpret_cast<const float4*>(p.sh.part + r * D + d));
          }
        }
        float now = top;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) now = fmaxf(now, w[i].x);
        const float use = now == -INFINITY ? 0.0f : now, keep = ex2(top - use);
        top = now;
        sum *= keep;
        acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const float f = ex2(w[i].x - use) * (E4M3 ? kFromPrompt : 1.0f);
          sum = fmaf(w[i].y, f, sum);
          acc.x = fmaf(v[i].x, f, acc.x), acc.y = fmaf(v[i].y, f, acc.y);
          acc.z = fmaf(v[i].z, f, acc.z), acc.w = fmaf(v[i].w, f, acc.w);
        }
      }
      const float f = sum == 0.0f ? 0.0f : (E4M3 ? p.v_scale[hk] : 1.0f) / sum;
      *reinterpret_cast<uint2*>(p.y + b * p.ldy + int64_t(h) * D + d) =
          make_uint2(bf16x2_rn(acc.x * f, acc.y * f), bf16x2_rn(acc.z * f, acc.w * f));
    }
  }
  pdl_trigger();
}

sp24_status launch_join(const SharedCall& c, cudaStream_t s) {
  JoinParams p;
  p.sh = c.groups;
  p.rows = c.B * c.q_heads;
  p.q_heads = c.q_heads;
  p.kv_heads = c.cache->heads;
  p.group = c.q_heads / c.cache->heads;
  p.v_scale = c.view.v_scale;
  p.y = static_cast<__nv_bfloat16*>(c.y);
  p.ldy = c.ldy;
  const bool e4m3 = c.cache->dtype == SP24_E4M3;
  const int per = kJoinThreads / (c.cache->head_dim / 4);
  auto kern = c.cache->head_dim == 128
                  ? (e4m3 ? attention_shared_join_kernel<128, true> : attention_shared_join_kernel<128, false>)
                  : (e4m3 ? attention_shared_join_kernel<64, true> : attention_shared_join_kernel<64, false>);
  return launch_pdl(kern, dim3((p.rows + per - 1) / per), dim3(kJoinThreads), 0, s, p) == cudaSuccess ? SP24_OK
                                                                                                   : SP24_ERR_CUDA;
}

}  // namespace
}  // namespace sp24

extern "C" size_t sp24_attention_decode_shared_workspace_size(int64_t B, int64_t G, int q_heads, int heads,
                                                              int head_dim) {
  using namespace sp24;
  const DeviceInfo* dev = nullptr;
  if (B < 0 || B > kMostTokens || G < 0 || G > kMostTokens || q_heads < 1 || heads < 1 || q_heads % heads ||
      q_heads / heads > 128 || (head_dim != 64 && head_dim != 128) || current_device(&dev))
    return 0;
  return room_for(B, G, q_heads, heads, head_dim, *dev).total;
}

extern "C" sp24_status sp24_attention_decode_shared(const void* q, int64_t B, int64_t ldq, int q_heads,
                                                    const sp24_kv_cache* cache, const int32_t* page_table,
                                                    int64_t table_width, int64_t ld_table, const int32_t* seq_lens,
                                                    const int32_t* cu_shared, const int32_t* shared_lens, int64_t G,
                                                    float scale, int window, int sinks, void* Y, int64_t ldy,
                                                    void* workspace, size_t workspace_bytes, void* stream) {
  using namespace sp24;
  SharedCall c = {};
  if (sp24_status st = check_attention(q, B, ldq, q_heads, cache, page_table, table_width, ld_table, seq_lens, B, scale,
                                       window, sinks, Y, ldy, &c.view))
    return st;
  if (G < 0 || G > kMostTokens || !cu_shared || (G > 0 && !shared_lens)) return SP24_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(cu_shared) | reinterpret_cast<uintptr_t>(shared_lens)) & 3u) return SP24_ERR_ALIGNMENT;
  const DeviceInfo* dev = nullptr;
  if (sp24_status st = current_device(&dev)) return st;
  const Room room = room_for(B, G, q_heads, cache->heads, cache->head_dim, *dev);
  if (!workspace || workspace_bytes < room.total) return SP24_ERR_WORKSPACE;
  if (!aligned16(workspace)) return SP24_ERR_ALIGNMENT;
  if (B == 0) return SP24_OK;
  // Sharing saves at most the groups' tokens but for one time each.  Where that takes less time than the two launches
  // more, the sequences are attended one by one.  (In wide tables, shared and one by one: 2 sequences behind 1000 tokens, 4 MB,
  // 14.4 and 7.5 us; 2 behind 4000, 16 MB, 16.1 and 11.3; 8 behind 1000, 29 MB, 14.6 and 11.1; 8 behind 4000, 115 MB, 16.5 and
  // 19.2; 32 behind 1000, 127 MB, 15.1 and 19.7.)
  const int64_t e = cache->dtype == SP24_E4M3 ? 1 : 2;
  const double saved = double(table_width << c.view.page_shift) * (B - 1) * cache->heads * (2 * cache->head_dim * e);
  if (G == 0 || saved < kLeastSaved)
    return sp24_attention_decode(q, B, ldq, q_heads, cache, page_table, table_width, ld_table, seq_lens, scale, window, sinks,
                                 Y, ldy, workspace, workspace_bytes, stream);
  // Numbers of rows, of all pieces' rows, and of key tiles over all pairs, are 32-bit.
  const int64_t tiles = ((table_width << c.view.page_shift) + 127) / 128;
  if (room.parts > INT32_MAX / (2 * kTileRows) || tiles > INT32_MAX / room.pairs || B > INT32_MAX / 128 / q_heads)
    return SP24_ERR_UNSUPPORTED;
  c.q = q;
  c.ldq = ldq;
  c.B = static_cast<int>(B);
  c.q_heads = q_heads;
  c.cache = cache;
  c.page_table = page_table;
  c.table_width = static_cast<int>(table_width);
  c.ld_table = ld_table;
  c.seq_lens = seq_lens;
  c.scale = scale;
  c.window = effective_window(window);
  c.sinks = sinks;
  c.y = Y;
  c.ldy = ldy;
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  c.decode_workspace = ws;
  c.groups.cu = cu_shared;
  c.groups.lens = shared_lens;
  c.groups.G = static_cast<int>(G);
  c.groups.where = reinterpret_cast<int2*>(ws + room.where);
  c.groups.own = reinterpret_cast<float*>(ws + room.own);
  c.groups.part = reinterpret_cast<float*>(ws + room.part);
  c.groups.pairs = static_cast<int>(room.pairs);
  c.groups.parts = static_cast<int>(room.parts);
  c.groups.window = c.window;
  c.groups.sinks = sinks;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (sp24_status st = launch_shared_tokens(c, *dev, s)) return st;
  if (sp24_status st = launch_own_tokens(c, *dev, s)) return st;
  return launch_join(c, s);
}
