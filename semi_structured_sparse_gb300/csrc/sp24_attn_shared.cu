// sp24_attn_shared.cu -- sp24_attention_decode_shared: one new token per
// sequence over the paged cache, where groups of sequences have their first
// tokens in common.
//
// A softmax over shared and own keys is joined from the maxima, sums and
// weighted values of both.  The shared keys of a group are one matrix for the
// queries of all its sequences, so that part is a product of matrices: the
// prompt kernel's tensor-core tiles, with (sequence, head) pairs as rows, each
// pair of keys' and values' tiles read once for up to 256 of them.  The keys that are
// a sequence's own have one query per head: the decode kernel streams them, and
// adds the shared part where a row's own is complete.  The second launch begins
// on the SMs that the first leaves idle and as it gets done.
#include <algorithm>
#include "sp24_attn.cuh"

namespace sp24 {
namespace {

// Blocks of rows that groups of B sequences have at most (each group's last may be partly
// filled), times the kv heads: pairs; a pair's keys are cut at most once per CTA.
struct Room {
  int64_t pairs, parts;
  size_t where, pieces, part, total;  // offsets behind the decode kernel's workspace
};
inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
Room room_for(int64_t B, int64_t G, int q_heads, int heads, int D, const DeviceInfo& dev) {
  Room r;
  const int64_t tokens = 2 * (kTileRows / (q_heads / heads));
  r.pairs = (B / tokens + std::min(B, G)) * heads;
  r.parts = r.pairs + dev.sm_count;
  r.where = up256(decode_workspace_bytes(dev, q_heads, heads, D));
  r.pieces = r.where + up256(static_cast<size_t>(B) * sizeof(int2));
  r.part = r.pieces + up256(static_cast<size_t>(r.pairs) * sizeof(int2));
  r.total = r.part + static_cast<size_t>(r.parts) * (2 * kTileRows) * (D + 2) * sizeof(float);
  return r;
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
  if (G == 0)
    return sp24_attention_decode(q, B, ldq, q_heads, cache, page_table, table_width, ld_table, seq_lens, scale, window, sinks,
                                 Y, ldy, workspace, workspace_bytes, stream);
  // Numbers of pieces' rows, and of key tiles over all pairs, are 32-bit.
  const int64_t tiles = ((table_width << c.view.page_shift) + 127) / 128;
  if (room.parts > INT32_MAX / (2 * kTileRows) || tiles > INT32_MAX / room.pairs) return SP24_ERR_UNSUPPORTED;
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
  c.groups.pieces = reinterpret_cast<int2*>(ws + room.pieces);
  c.groups.part = reinterpret_cast<float*>(ws + room.part);
  c.groups.pairs = static_cast<int>(room.pairs);
  c.groups.parts = static_cast<int>(room.parts);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (sp24_status st = launch_shared_tokens(c, *dev, s)) return st;
  return launch_own_tokens(c, *dev, s);
}
