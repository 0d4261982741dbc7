// sp24_attn_prompt.cu -- sp24_attention_prompt: causal attention of a ragged
// batch of new tokens over the paged cache, with an optional sliding window
// and sinks.
//
//   S = Q K^T,  P = exp2(c S - m),  O = P V / sum(P),  c = scale log2(e)
//   (times the cache's scale), m a row maximum that follows the true one
//
// Bound by the tensor core (4 D operations per visible key and query row) with
// heads of 128, by the softmax warps with heads of 64.  A block is 256 query
// rows of one kv head, as two tiles of 128: the rows of a tile are (token, head
// of the group) pairs, so a short prompt fills tiles too and all heads of a
// group share the keys' copies.  Keys and values come in tiles of 128 tokens, one TMA box per
// page and 64 dims, through a ring of shared memory.  Per key tile and query
// tile, S (128 x 128 fp32) and O (128 x D fp32) are in tensor memory, all 512
// columns of it; P goes back into the columns of S (into columns of its own with
// heads of 64) as bf16 (f16 for an e4m3 cache) and is the A operand of P V
// straight from there.
//
// Two softmax warpgroups (a thread per query row: maxima and sums need no
// shuffles) alternate with the tensor core: while one works on its tile, the
// MMAs run on the other's.  P V of key tile i and Q K^T of tile i + 1 are issued
// back to back for a query tile; the tensor core runs them in order, so S may
// overwrite P.  A row's O is rescaled only when its maximum has grown by more
// than 2^8 (P then stays below 256, which bf16 and fp32 sums hold as well as 1;
// f16 has its own room for it, Cfg::UP); that is rare after the first tiles, so
// the softmax warps do it themselves.
//
// One CTA per SM works through blocks: the first is its own, the others it
// takes from the part of the grid that no SM has begun (cluster launch
// control), so that copies of the next block's queries and keys, and its first
// Q K^T, overlap the end of this one, and SMs that are done early take more.
// Blocks that see many keys come first.  (With a launch per block, setting up
// and draining took 16,000 cycles of a block's 92,000 at 8192 tokens.)
//
// Measured (GB300, in a CUDA graph of a few calls): 8192 tokens, 32/8 heads of
// 128, 325 us, 1690 TFLOP/s of visible products (86 % of the measured bf16
// rate); 16001 tokens under a window of 4096 and 4 sinks, 28/4 heads of 64, 450
// us, 911 TFLOP/s; pieces of 1839 and 1629 tokens over 14000 in an e4m3 cache
// 554 us, 1525 TFLOP/s.  Calls back to back for 0.15 s, where the clock falls:
// 352 us, 448 and 570.  With heads of 128 a query tile's chain (S read 52
// cycles, the first half's exponentials beside the search for the maximum 450,
// the second half's 350, P written and seen 200, the rest of P V and Q K^T 768
// plus what the other tile's MMAs take) is 2600 cycles per key tile, against
// 2048 of MMAs for both tiles: tensor memory has no room for a second S.
//
// Where a call's blocks leave SMs idle and its page tables are long, a block's
// key tiles are cut into parts, each a block of the grid; a second, small launch
// adds their O up.
//
// Places of a key tile that no row of the CTA sees are not loaded by whole
// pages, and zeroed in V otherwise: 0 x NaN is not 0.  In S they are
// overwritten with -inf.
//
// With an e4m3 cache a further warpgroup turns the tiles' codes into f16
// (exactly) between the copy and the MMA; the softmax warps scale each query
// row by a power of two, so that bf16 queries fit f16's range.
#include <algorithm>
#include <cuda_bf16.h>
#include "sp24_attn.cuh"
#include "sp24_ptx.cuh"

namespace sp24 {
namespace {

constexpr int BM = kTileRows;  // query rows per tile, two tiles per CTA
constexpr int BN = kKeyTile;   // keys per tile
constexpr int kLeastTiles = 4;  // key tiles of a part, at least, where a block's keys are cut

struct PromptParams {
  int T, B;
  const int32_t* cu_q;
  CacheView cache;
  const int32_t* page_table;
  int table_width;
  int64_t ld_table;
  const int32_t* seq_lens;
  float scale;
  int window, sinks;
  __nv_bfloat16* y;
  int64_t ldy;
  int kv_heads, group, tile_tokens;  // tile_tokens = BM / group
  unsigned int inv_group;            // ceil(2^16 / group)
  int splits;      // parts that a block's key tiles are cut into
  float* part;     // splits > 1: of each part, O [2 BM][D], and then of all parts, maxima and sums [2 BM][2]
  int parts;       // how many `part` holds
  unsigned int* err;
  SharedGroups sh;  // shared first tokens: rows are sequences, of which each has one
};

template <int D_, bool E4M3_>
struct Cfg {
  static constexpr int D = D_;
  static constexpr bool E4M3 = E4M3_;
  static constexpr int THREADS = E4M3 ? 512 : 384;
  static constexpr int Q_TILE = BM * D * 2;
  static constexpr int KV_TILE = BN * D * 2;              // as the MMA reads it
  static constexpr int RAW_TILE = BN * D;                 // e4m3 codes
  static constexpr int RAW = E4M3 ? (D == 128 ? 2 : 4) : 0;
  static constexpr int SLOTS = D == 128 ? (E4M3 ? 4 : 5) : 8;
  static constexpr int BARS = 23 + 2 * SLOTS + 2 * RAW;
  static constexpr int SMEM = 1024 + 2 * Q_TILE + SLOTS * KV_TILE + RAW * RAW_TILE + BARS * 8;
  // Registers after the split: the warpgroups' shares stay within the launch's
  // (168 x 384 or 128 x 512).
  static constexpr int REG_SOFTMAX = E4M3 ? 208 : 216;
  static constexpr int REG_ISSUE = E4M3 ? 48 : 64;
  static constexpr int REG_CONVERT = 48;
  // Whether P V begins when half of P is there.  It shortens the chain S -> P ->
  // O -> next S of a query tile (8192 tokens: 350 us against 354, when it was
  // added), but costs beside the e4m3 conversion (576 us against 555) and with P
  // apart (460 against 454).
  static constexpr bool EARLY = !E4M3 && D == 128;
  // Whether P has columns of its own in tensor memory (heads of 64 leave room
  // for it).  Then Q K^T of the next key tile runs while the softmax warps are
  // busy with this one, as soon as they have read S.
  static constexpr bool APART = D == 64;
  // Whether P of a key tile's first half is formed with the maximum so far,
  // beside the search for the new one (and formed again in the rare tile where
  // the maximum has grown): 8192 tokens 329 us against 339.  Not with an e4m3
  // cache (579 us against 555: the registers do not reach), nor with P apart
  // (P V of the last key tile is still reading P then).
  static constexpr bool AHEAD = D == 128 && !E4M3;
  // (Shared tokens, few key tiles per block) whether the query tiles take turns at their exponentials from the first key
  // tile on, as they come to do in long blocks: a key tile of both takes 1.43 us instead of 1.75.  Not with heads of 64
  // (200 sequences behind 50001 tokens 129 us against 100), and no gain with an e4m3 cache.
  static constexpr bool TURNS = D == 128 && !E4M3;
  // With an e4m3 cache P, and its sums, are 2^UP times exp2(c S - m): up to 2^8
  // times that where the maximum has grown by less, so up to 2^15, near f16's end.
  // The row's largest weight is 2^7 at least; f16's smallest step, 2^-24, rounds
  // the smallest weights by 2^-32 of it at most.
  static constexpr float UP = kPromptUp;
  static constexpr uint32_t P_COL = APART ? 2 * BN : 0, P_STEP = APART ? BN / 2 : BN;  // P of query tile x
  static constexpr uint32_t O_COL = APART ? 3 * BN : 2 * BN;                           // O of query tile x: + x D
};
static_assert(2 * 128 * 216 + 128 * 64 <= 168 * 384, "register split, bf16");
static_assert(2 * 128 * 208 + 128 * 48 + 128 * 48 <= 128 * 512, "register split, e4m3");

// One lane of the warp, the same every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t x;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(x));
  return x != 0;
}
template <int N>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// Tensor memory <-> registers: this warp's 32 lanes, 32 consecutive columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// D (128 x N, fp32) (+)= A (tensor memory, 16-bit, 128 x 16) B (shared memory)
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
// kind::f16, fp32 accumulator; 16-bit type: 0 f16, 1 bf16; b_mn: B's rows (its N) are contiguous.
__host__ __device__ constexpr uint32_t idesc_16(int M, int N, uint32_t type, bool b_mn) {
  return (1u << 4) | (type << 7) | (type << 10) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// The next block of the grid that no SM has begun, if any, to this CTA: its
// index arrives in `response` (16 bytes of shared memory) and completes 16
// bytes on `bar`.
__device__ __forceinline__ void steal_block(void* response, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          smem_u32(response)),
      "r"(smem_u32(bar))
      : "memory");
}
// Its index along x, or -1.
__device__ __forceinline__ int stolen_block(const void* response) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t.reg .b32 y, z, w;\n\t"
      "ld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, r;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(smem_u32(response))
      : "memory");
  return ok ? static_cast<int>(x) : -1;
}

// Token of a tile's row r < BM: r / group.  r (inv_group - 2^16 / group) is below 128, so the quotient is off by less
// than 128 / 2^16 < 1 / group.
__device__ __forceinline__ int token_of(const PromptParams& p, int r) {
  return static_cast<int>(static_cast<unsigned int>(r) * p.inv_group >> 16);
}

// What a CTA works on.
struct Work {
  int b;             // sequence, or -1: nothing
  int hk;            // kv head
  int row0, rows;    // its first query row (in q), and how many tokens from there on are the sequence's
  int p0;            // position of that row's token
  int p_hi;          // the last position (the last visible key) of the CTA's rows
  int wlo, send;     // keys that some row sees: [0, send) and [wlo, p_hi]
  int first, nst;    // key tiles: 0 .. nst - 1 (sinks), then first, first + 1, ...
  int t0, nt;        // which of them: nt from number t0 on
  int part;          // where this part's sums go (splits > 1)
};
struct Pieces {      // shared tokens: all the parts that a pair's keys are cut into
  int first, count;
};

__device__ __forceinline__ int tile_of(const Work& w, int i) {
  return w.t0 + i < w.nst ? w.t0 + i : w.first + w.t0 + i - w.nst;
}

// Rows [lo, hi) of q of a sequence, and the tokens in its cache.
struct Rows {
  int lo, hi, n;
};
__device__ __forceinline__ Rows rows_of(const PromptParams& p, int b, bool report) {
  Rows s = {0, 0, 0};
  if (b < p.B) {
    const int a = __ldg(p.cu_q + b), z = __ldg(p.cu_q + b + 1);
    s.n = __ldg(p.seq_lens + b);
    s.lo = min(max(a, 0), p.T), s.hi = min(max(z, s.lo), p.T);
    const int most = p.table_width << p.cache.page_shift;
    const bool bad = s.n < 0 || s.n > most;
    if (bad) s.n = s.n < 0 ? 0 : most;
    if (report && (bad || s.lo != a || s.hi != z)) atomicOr(p.err, DEVERR_INDEX);
  }
  return s;
}
// Blocks of all sequences, over the warp; `mine`: sequence `lane`'s rows.
__device__ __forceinline__ int count_blocks(const PromptParams& p, int lane, bool report, Rows& mine) {
  const int tok = 2 * p.tile_tokens;
  mine = rows_of(p, lane, report);
  int total = (mine.hi - mine.lo + tok - 1) / tok;
  for (int b = lane + 32; b < p.B; b += 32) {
    const Rows s = rows_of(p, b, report);
    total += (s.hi - s.lo + tok - 1) / tok;
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, m);
  return total;
}

// Block `block` of the grid, as the warp sees it; `total`: blocks of 2
// tile_tokens tokens in all sequences; `mine`: sequence `lane`'s rows, where
// they are at hand.  The last block of the last sequence comes first, since late
// blocks of a prompt see the most keys; all parts and kv heads of a block come
// together.
__device__ __forceinline__ void find_work(const PromptParams& p, int block, int total, const Rows* mine, int lane,
                                          Work* out) {
  const int tok = 2 * p.tile_tokens;
  const int group = block / p.kv_heads;  // of blocks that differ in the kv head alone
  const int rank = p.splits > 1 ? group / p.splits : group, split = group - rank * p.splits;
  const int want = block < 0 ? -1 : total - 1 - rank;
  if (lane == 0) out->b = -1;
  __syncwarp();
  int seen = 0;
  for (int b0 = 0; want >= 0 && b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    const Rows s = b0 == 0 && mine ? *mine : rows_of(p, b, false);
    const int own = (s.hi - s.lo + tok - 1) / tok;
    int incl = own;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, incl, m);
      if (lane >= m) incl += x;
    }
    incl += seen;
    if (want < incl && want >= incl - own) {
      Work w;
      w.b = b;
      w.hk = block - group * p.kv_heads;
      const int i0 = (want - (incl - own)) * tok, m = s.hi - s.lo;
      w.row0 = s.lo + i0;
      w.rows = m - i0;
      w.p0 = s.n - m + i0;
      w.p_hi = w.p0 + min(tok, w.rows) - 1;
      w.wlo = p.window > 0 ? max(0, w.p0 - p.window + 1) : 0;
      w.send = min(p.sinks, w.wlo);
      w.first = w.wlo / BN;
      w.nst = min((w.send + BN - 1) / BN, w.first);
      const int tiles = w.p_hi < 0 ? 0 : w.nst + w.p_hi / BN + 1 - w.first;
      w.t0 = 0, w.nt = tiles;
      if (p.splits > 1) {  // (tiles: below 2^24; splits: at most 32)
        w.t0 = tiles * split / p.splits;
        w.nt = tiles * (split + 1) / p.splits - w.t0;
      }
      w.part = (rank * p.kv_heads + w.hk) * p.splits + split;
      *out = w;
    }
    seen = __shfl_sync(0xFFFFFFFFu, incl, 31);
    if (want < seen) break;
  }
  __syncwarp();
}

// The same for shared first tokens.  A pair is a block of a group's sequences and
// a kv head, a unit a key tile of it; the units of all pairs are dealt out to the
// CTAs in equal contiguous ranges, so that groups of any sizes and lengths keep
// all SMs busy alike.
struct Deal {
  unsigned int units, ctas, per, extra;  // the first `extra` CTAs take a unit more
  __device__ __forceinline__ unsigned int begin(unsigned int cta) const { return cta * per + min(cta, extra); }
  __device__ __forceinline__ unsigned int cta_of(unsigned int u) const {
    return u < extra * (per + 1) ? u / (per + 1) : extra + (u - extra * (per + 1)) / per;
  }
};
constexpr int kLeastUnits = 4;  // per CTA

// 32 groups, one per lane, with the units and pairs up to and with each.
struct Groups {
  int lo, end, n;                    // sequences, and the tokens that they read together
  bool in_order;                     // each begins where the one before it ends, within the batch
  unsigned int tiles, units, pairs;  // of this one
  unsigned int units_to, pairs_to;
};
__device__ __forceinline__ Groups load_groups(const PromptParams& p, int g, int lane, bool report, int before,
                                              unsigned int units_before, unsigned int pairs_before) {
  const int tok = 2 * p.tile_tokens, most = p.table_width << p.cache.page_shift;
  Groups s;
  int raw = 0, shared = 0;
  if (g < p.sh.G) raw = __ldg(p.sh.cu + g + 1), shared = __ldg(p.sh.lens + g);
  s.end = max(min(raw, p.T), before);
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, s.end, m);
    if (lane >= m) s.end = max(s.end, x);
  }
  s.lo = __shfl_up_sync(0xFFFFFFFFu, s.end, 1);
  if (lane == 0) s.lo = before;
  s.in_order = g >= p.sh.G || raw == s.end;
  if (report && g < p.sh.G && (!s.in_order || shared < 0 || shared > most)) atomicOr(p.err, DEVERR_INDEX);
  s.n = g < p.sh.G ? shared_tokens(p.sh, s.lo, s.end, shared, p.seq_lens, most) : 0;
  s.tiles = (s.n + BN - 1) / BN;
  s.pairs = s.tiles ? (s.end - s.lo + tok - 1) / tok * p.kv_heads : 0;
  s.units = s.pairs * s.tiles;
  s.units_to = s.units, s.pairs_to = s.pairs;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const unsigned int x = __shfl_up_sync(0xFFFFFFFFu, s.units_to, m), y = __shfl_up_sync(0xFFFFFFFFu, s.pairs_to, m);
    if (lane >= m) s.units_to += x, s.pairs_to += y;
  }
  s.units_to += units_before, s.pairs_to += pairs_before;
  return s;
}
// The work that begins with unit u, if it is one of these groups'.
__device__ __forceinline__ void place_unit(const PromptParams& p, const Groups& s, const Deal& deal, unsigned int u,
                                           unsigned int u_end, unsigned int cta, Work* out, Pieces* pieces) {
  if (u >= u_end || u >= s.units_to || u < s.units_to - s.units) return;
  Work w;
  const unsigned int local = u - (s.units_to - s.units), pair = local / s.tiles;
  const int block = pair / p.kv_heads;
  w.b = s.lo;
  w.hk = pair - block * p.kv_heads;
  w.row0 = s.lo + block * 2 * p.tile_tokens;
  w.rows = s.end - w.row0;
  w.p0 = w.p_hi = s.n - 1;
  w.wlo = w.send = w.first = w.nst = 0;
  w.t0 = local - pair * s.tiles;
  w.nt = min(s.tiles - w.t0, u_end - u);
  const int number = s.pairs_to - s.pairs + pair;
  w.part = number + cta;  // (either grows from one piece to the next)
  const unsigned int u0 = u - w.t0, first = deal.cta_of(u0);
  pieces->first = number + first;
  pieces->count = deal.cta_of(u0 + s.tiles - 1) - first + 1;
  if (number >= p.sh.pairs || w.part >= p.sh.parts) w.b = -1;  // (there is room for all that the host expects)
  *out = w;
}
// Goes through the groups: the units of all (none if groups are out of order: the
// launch for sequences' own tokens sees that as well, and attends all of them one by one),
// and how often their tokens would be read one by one; or (`out`) the work that begins with unit u.  `few`: the groups,
// where they are 32 at most and known.
__device__ __forceinline__ unsigned int scan_groups(const PromptParams& p, int lane, bool report, const Deal& deal,
                                                    unsigned int u, unsigned int u_end, unsigned int cta, Work* out,
                                                    Pieces* pieces, Groups* few, long long* times) {
  if (out && lane == 0) out->b = -1;
  __syncwarp();
  unsigned int units = 0, pairs = 0;
  if (out && p.sh.G <= 32) {
    place_unit(p, *few, deal, u, u_end, cta, out, pieces);
  } else {
    const int first = __ldg(p.sh.cu);
    int before = min(max(first, 0), p.T);
    if (report && lane == 0 && first != before) atomicOr(p.err, DEVERR_INDEX);
    long long sum = 0;
    bool in_order = first == before;
    for (int g0 = 0; g0 < p.sh.G; g0 += 32) {
      const Groups s = load_groups(p, g0 + lane, lane, report, before, units, pairs);
      if (out)
        place_unit(p, s, deal, u, u_end, cta, out, pieces);
      else
        *few = s, sum += static_cast<long long>(s.end - s.lo) * s.n;
      in_order &= s.in_order;
      units = __shfl_sync(0xFFFFFFFFu, s.units_to, 31), pairs = __shfl_sync(0xFFFFFFFFu, s.pairs_to, 31);
      before = __shfl_sync(0xFFFFFFFFu, s.end, 31);
      if (out && u < units) break;
    }
    if (times) *times = sum;
    if (!__all_sync(0xFFFFFFFFu, in_order)) units = 0;
  }
  __syncwarp();
  return units;
}
// SHARED: the shared first tokens of groups of sequences, for one query per
// sequence; every row sees all of them, and sums go to the workspace.
template <class C, bool SHARED = false>
__global__ void __launch_bounds__(C::THREADS, 1)
    attention_prompt_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap, const __grid_constant__ PromptParams p) {
  constexpr int D = C::D, SLOTS = C::SLOTS, RAW = C::RAW;
  constexpr bool E4M3 = C::E4M3;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Work s_work[2];
  __shared__ Pieces s_pieces[2];   // (shared tokens)
  __shared__ uint64_t turn[2];     // (TURNS) the other query tile has formed its P
  __shared__ __align__(16) uint4 s_response;
  __shared__ uint32_t s_tmem;
  __shared__ int s_last[2];  // position in the ring of the last copy of keys, and of values

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_s = smem;
  uint8_t* kv_s = q_s + 2 * C::Q_TILE;
  uint8_t* raw_s = kv_s + SLOTS * C::KV_TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(raw_s + RAW * C::RAW_TILE);
  uint64_t* q_full = bars;            // [2] the query tile has landed
  uint64_t* q_ready = bars + 2;       // [2] ... and is f16 (e4m3 caches)
  uint64_t* q_empty = bars + 4;       // [2] its last Q K^T is done
  uint64_t* s_full = bars + 6;        // [2] S of the next key tile is there, and P V of the last one done
  uint64_t* p_half = bars + 8;        // [2] P of the first 64 keys is there, and O at its scale
  uint64_t* p_full = bars + 10;       // [2] P is there
  uint64_t* o_full = bars + 12;       // [2] O is complete (APART: O of this key tile)
  uint64_t* drain = bars + 14;        // [2]
  uint64_t* work_full = bars + 16;    // [2]
  uint64_t* work_empty = bars + 18;   // [2]
  uint64_t* stolen = bars + 20;
  uint64_t* s_read = bars + 21;       // [2] S is in the softmax warps' registers (APART)
  uint64_t* kv_full = bars + 23;      // [SLOTS]
  uint64_t* kv_empty = kv_full + SLOTS;
  uint64_t* raw_full = kv_empty + SLOTS;  // [RAW]
  uint64_t* raw_empty = raw_full + RAW;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // known to be uniform

  if (warp == 8) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  } else if (warp == 10 && lane == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 1);
      mbar_init(&q_ready[x], 4);
      mbar_init(&q_empty[x], 1);
      mbar_init(&s_full[x], 1);
      mbar_init(&s_read[x], 4);
      mbar_init(&p_half[x], 4);
      mbar_init(&p_full[x], 4);
      mbar_init(&o_full[x], 1);
      mbar_init(&drain[x], 1);
      if (SHARED && C::TURNS) mbar_init(&turn[x], 4);
      mbar_init(&work_full[x], 1);
      mbar_init(&work_empty[x], E4M3 ? 15 : 11);  // the warps that read the work
    }
    mbar_init(stolen, 1);
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&kv_full[i], E4M3 ? 4 : 1);
      mbar_init(&kv_empty[i], 2);
    }
    for (int i = 0; i < RAW; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    fence_mbar_init();
  } else if (warp == 9 && lane == 0) {
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (SHARED) pdl_trigger();  // sequences' own tokens on SMs that have none of this, and as they get done
  const uint32_t tmem = s_tmem;
  // The work of this CTA's next block, for every role but the one that finds
  // it; done_with says that this warp will not read it again.
  auto wait_work = [&](int item) { return mbar_wait(&work_full[item & 1], (item >> 1) & 1); };
  auto done_with = [&](int item) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&work_empty[item & 1]);
  };
  auto tiles_of = [&](const Work& w) { return w.rows > p.tile_tokens ? 2 : 1; };

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<C::REG_SOFTMAX>();
    const int x = warp >> 2, r = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + x * BN, tp = tmem + lanes + C::P_COL + x * C::P_STEP;
    const uint32_t to = tmem + lanes + C::O_COL + x * D;
    uint32_t sn = 0, on = 0;  // key tiles and blocks so far, for the barriers' parities
    uint32_t tn = 0;          // turns so far
    bool ok = true;
    for (int item = 0; ok; ++item) {
      ok = wait_work(item);
      const Work& w = s_work[item & 1];
      if (!ok || w.b < 0) break;
      if (x >= tiles_of(w)) {
        done_with(item);
        continue;
      }
      float l = 0.0f, m = -INFINITY;
      if (w.nt > 0) {
        float c = p.scale * 1.4426950408889634f;
        if (E4M3) {
          ok = mbar_wait(&q_full[x], on & 1);
          if (!ok) break;
          // this row to f16, scaled by a power of two to at most 2
          uint8_t* q = q_s + x * C::Q_TILE + r * 128;
          float top = 0.0f;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(q + (i / 8) * (BM * 128) + (((i & 7) ^ (r & 7)) << 4));
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[j] << 16)), fabsf(__uint_as_float(u[j] & 0xFFFF0000u))));
          }
          uint32_t e = __float_as_uint(top) >> 23;  // as in the decode kernel
          e = e == 255 ? 127u : min(max(e, 64u), 253u);
          const float down = __uint_as_float((254u - e) << 23);
          c *= p.cache.k_scale[w.hk] * __uint_as_float(e << 23);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            uint4* at16 = reinterpret_cast<uint4*>(q + (i / 8) * (BM * 128) + (((i & 7) ^ (r & 7)) << 4));
            uint4 v = *at16;
            uint32_t* u = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              u[j] = f16x2_rn(__uint_as_float(u[j] << 16) * down, __uint_as_float(u[j] & 0xFFFF0000u) * down);
            *at16 = v;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_ready[x]);
        }
        // What the loop needs of the block, in registers: shared memory is busy with the MMAs' operands, and a read
        // would take some hundred cycles.
        const int nt = w.nt, nst = w.nst - w.t0, first = w.first * BN;  // nst: sink tiles from here on
        const int p_min = SHARED ? w.p_hi : w.p0 + x * p.tile_tokens, p_max = min(w.p_hi, p_min + p.tile_tokens - 1);
        int base = tile_of(w, 0) * BN;
        const bool turns = SHARED && C::TURNS && tiles_of(w) == 2;
        for (int i = 0; i < nt; ++i, ++sn, base = i == nst && nst > 0 ? first : base + BN) {
          ok = mbar_wait(&s_full[x], sn & 1);
          if (turns && ok && (x == 1 || tn > 0)) ok = mbar_wait(&turn[x], (x == 1 ? tn : tn - 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const int end = base + BN - 1;
          // Columns that this row does not see: past its own position, or before its window and after the sinks.
          const bool cut_hi = end > p_min, cut_lo = !SHARED && p.window > 0 && base <= p_max - p.window && end >= p.sinks;
          uint32_t su[BN];
#pragma unroll
          for (int j = 0; j < BN / 32; ++j) tmem_ld32(ts + 32 * j, su + 32 * j);
          tmem_ld_wait();
          if (C::APART) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_read[x]);
          }
          float* s = reinterpret_cast<float*>(su);
          if (cut_hi || cut_lo) {
            // (The position is worked out here, once or twice per block, to leave the registers to S.)
            int rr = r;
            asm volatile("" : "+r"(rr));  // here, not ahead of the loop
            const int token = SHARED ? 0 : token_of(p, rr);
            // (rows past the tile's tokens are no one's)
            const int hi = token < p.tile_tokens ? p_min + token - base : BN, lo = hi - p.window, sk = p.sinks - base;
            // Each 32 columns only where some row of the warp does not see them all.
            if (cut_lo) {
              const int last = __reduce_max_sync(0xFFFFFFFFu, lo);
#pragma unroll
              for (int j0 = 0; j0 < BN; j0 += 32) {
                if (last < j0 || j0 + 31 < sk) continue;
#pragma unroll
                for (int j = j0; j < j0 + 32; ++j)
                  if (!(j > lo || j < sk)) s[j] = -INFINITY;
              }
            }
            if (cut_hi) {
              const int least = __reduce_min_sync(0xFFFFFFFFu, hi);
#pragma unroll
              for (int j0 = 0; j0 < BN; j0 += 32) {
                if (least >= j0 + 31) continue;
#pragma unroll
                for (int j = j0; j < j0 + 32; ++j)
                  if (j > hi) s[j] = -INFINITY;
              }
            }
          }
          // P of 32 keys, and its sum.
          auto chunk = [&](int h, float less, float2 (&sum)[2]) {
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float2 e = __ffma2_rn(make_float2(s[32 * h + 2 * j], s[32 * h + 2 * j + 1]), make_float2(c, c),
                                    make_float2(less, less));
              e.x = ex2(e.x);
              e.y = ex2(e.y);
              sum[j & 1] = __fadd2_rn(sum[j & 1], e);
              pk[j] = E4M3 ? f16x2_rn(e.x, e.y) : bf16x2_rn(e.x, e.y);
            }
            tmem_st16(tp + 16 * h, pk);
          };
          float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
          // P of the first half with the maximum so far, beside the search for the new one: it is nearly always good.
          const bool ahead = C::AHEAD && i > 0;
          if (ahead) {
#pragma unroll
            for (int h = 0; h < 2; ++h) chunk(h, m == -INFINITY ? 0.0f : -m, sum);
          }
          float top[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) top[j] = max3(s[3 * j], s[3 * j + 1], s[3 * j + 2]);
#pragma unroll
          for (int j = 12; j < BN; j += 2) top[(j >> 1) & 3] = max3(top[(j >> 1) & 3], s[j], s[j + 1]);
          const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
          const bool grow = now > m + 8.0f;  // also from -inf
          if (C::APART && i > 0) {  // P V of the last key tile is done with P and O
            ok = mbar_wait(&o_full[x], (sn - 1) & 1);
            if (!ok) break;
            tc_fence_after();
          }
          const bool any = __any_sync(0xFFFFFFFFu, grow);
          if (any) {
            const float to_m = grow ? now : m;
            const float keep = m == to_m ? 1.0f : ex2(m - to_m);
            m = to_m;
            l *= keep;
            if (i > 0) {
#pragma unroll 1
              for (int j = 0; j < D; j += 16) {  // 16 columns at a time: S takes 128 registers
                uint32_t o[16];
                tmem_ld16(to + j, o);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * keep);
                tmem_st16(to + j, o);
              }
            }
          }
          const float less = m == -INFINITY ? 0.0f : E4M3 ? C::UP - m : -m;
          if (!ahead || any) {
            sum[0] = sum[1] = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int h = 0; h < 2; ++h) chunk(h, less, sum);
          }
          if (C::EARLY) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_half[x]);
          }
          chunk(2, less, sum);
          chunk(3, less, sum);
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&p_full[x]);
            if (turns) mbar_arrive(&turn[1 - x]);
          }
          if (turns) ++tn;
        }
        if (ok) ok = mbar_wait(&o_full[x], (C::APART ? sn - 1 : on) & 1);
        if (!ok) break;
        ++on;
        tc_fence_after();
      }
      // Out, a few dims at a time: a lane's 64 bytes of its row change places with those of its three neighbours, so that
      // four lanes write 64 bytes of one row together.
      auto exchange = [&](uint32_t (&v)[4][4]) {
#pragma unroll
        for (int bit = 1; bit < 4; bit <<= 1)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k & bit) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool upper = lane & bit;
              const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, upper ? v[k][e] : v[k | bit][e], bit);
              (upper ? v[k][e] : v[k | bit][e]) = got;
            }
          }
      };
      int rr = r;
      asm volatile("" : "+r"(rr));  // worked out here, not ahead of the loop: S takes the registers there
      if (SHARED) {
        // As below, but only the rows that are some sequence's; and where the joining launch finds them.
        float* const o_part = p.sh.part + static_cast<int64_t>(w.part) * (2 * BM * D) + x * (BM * D);
        float* const ml = p.sh.part + static_cast<int64_t>(p.sh.parts) * (2 * BM * D) +
                          static_cast<int64_t>(w.part) * (2 * BM * 2) + x * (BM * 2);
        const int token = token_of(p, rr), at = x * p.tile_tokens + token;
        const bool mine = token < p.tile_tokens && at < w.rows;
        if (mine) *reinterpret_cast<float2*>(ml + 2 * rr) = make_float2(m, l);
        if (w.t0 == 0 && mine && rr == token * p.group)
          p.sh.where[static_cast<int64_t>(w.row0 + at) * p.kv_heads + w.hk] =
              make_int2(s_pieces[item & 1].first * (2 * BM) + x * BM + rr, s_pieces[item & 1].count);
        const unsigned int some = __ballot_sync(0xFFFFFFFFu, mine);
#pragma unroll 1
        for (int j = 0; j < D && some; j += 16) {
          uint32_t v[4][4];
          tmem_ld16(to + j, reinterpret_cast<uint32_t(&)[16]>(v));
          tmem_ld_wait();
          exchange(v);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (some >> ((lane & ~3) + k) & 1)
              *reinterpret_cast<uint4*>(o_part + ((rr & ~3) + k) * D + j + (lane & 3) * 4) =
                  make_uint4(v[k][0], v[k][1], v[k][2], v[k][3]);
        }
      } else if (p.splits > 1) {
        // This part's O as it is, and its maximum and sum; attention_join_kernel adds the parts up.
        float* const o_part = p.part + static_cast<int64_t>(w.part) * (2 * BM * D) + x * (BM * D);
        float* const ml = p.part + static_cast<int64_t>(p.parts) * (2 * BM * D) + w.part * (2 * BM * 2) + x * (BM * 2);
        *reinterpret_cast<float2*>(ml + 2 * rr) = make_float2(m, l);
#pragma unroll 1
        for (int j = 0; j < D && w.nt > 0; j += 16) {
          uint32_t v[4][4];
          tmem_ld16(to + j, reinterpret_cast<uint32_t(&)[16]>(v));
          tmem_ld_wait();
          exchange(v);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(o_part + ((rr & ~3) + k) * D + j + (lane & 3) * 4) =
                make_uint4(v[k][0], v[k][1], v[k][2], v[k][3]);
        }
      } else {
        const float f = l == 0.0f ? 0.0f : (E4M3 ? p.cache.v_scale[w.hk] : 1.0f) / l;
        __nv_bfloat16* rows[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int rk = (rr & ~3) + k, tk = token_of(p, rk), ak = x * p.tile_tokens + tk;
          rows[k] = tk < p.tile_tokens && ak < w.rows
                        ? p.y + static_cast<int64_t>(w.row0 + ak) * p.ldy +
                              static_cast<int64_t>(w.hk * p.group + rk - tk * p.group) * D + (lane & 3) * 8
                        : nullptr;
        }
#pragma unroll 1
        for (int j = 0; j < D; j += 32) {
          uint32_t o[32];
          if (w.nt > 0) {
            tmem_ld32(to + j, o);
            tmem_ld_wait();
          }
          uint32_t v[4][4];
#pragma unroll
          for (int k = 0; k < 16; ++k)
            v[k >> 2][k & 3] =
                f == 0.0f ? 0u : bf16x2_rn(__uint_as_float(o[2 * k]) * f, __uint_as_float(o[2 * k + 1]) * f);
          exchange(v);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (rows[k]) *reinterpret_cast<uint4*>(rows[k] + j) = make_uint4(v[k][0], v[k][1], v[k][2], v[k][3]);
        }
      }
      tc_fence_before();  // O is read before this warp lets the next block's P V begin
      done_with(item);
    }
    if (!ok && lane == 0) atomicOr(p.err, DEVERR_TIMEOUT_EPILOGUE);
  } else if (warp < 12) {
    setmaxnreg_dec<C::REG_ISSUE>();
    if (warp == 8 || warp == 10) {
      // ------------------------------------------------------------ MMA
      // Each query tile has a warp of its own: a commit holds its thread back
      // until the MMAs that it tracks are done, and the other tile's MMAs fill
      // that time.
      const int x = (warp - 8) / 2;
      const uint32_t id_qk = idesc_16(BM, BN, E4M3 ? 0 : 1, false), id_pv = idesc_16(BM, D, E4M3 ? 0 : 1, true);
      const uint64_t q_d = smem_desc(smem_u32(q_s) + x * C::Q_TILE, 16, 1024, SWZ_128B);
      const uint64_t k_d = smem_desc(smem_u32(kv_s), 16, 1024, SWZ_128B);
      const uint64_t v_d = smem_desc(smem_u32(kv_s), BN * 128, 1024, SWZ_128B);
      const uint32_t t_s = tmem + x * BN, t_p = tmem + C::P_COL + x * C::P_STEP, t_o = tmem + C::O_COL + x * D;
      auto qk = [&](int slot) {
        const uint64_t kd = k_d + slot * (C::KV_TILE >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int off = ((k / 4) * (BM * 128) + (k % 4) * 32) >> 4;
          mma_bf16(t_s, q_d + off, kd + off, id_qk, k > 0);
        }
      };
      auto pv = [&](int slot, int half, bool add) {
        const uint64_t vd = v_d + slot * (C::KV_TILE >> 4);
#pragma unroll
        for (int j = 0; j < BN / 32; ++j) {
          const int k = half * (BN / 32) + j;
          mma_f16_ts(t_o, t_p + 8 * k, vd + k * (2048 >> 4), id_pv, add || j > 0);
        }
      };
      bool ok = true;
      int ring = 0;               // tiles of the ring so far: K, V, K, V, ...
      uint32_t pn = 0, qn = 0;    // key tiles and blocks so far
      auto wait_kv = [&](int n) { return mbar_wait(&kv_full[n % SLOTS], (n / SLOTS) & 1); };
      for (int item = 0; ok; ++item) {
        ok = wait_work(item);
        const Work w = s_work[item & 1];
        if (!ok || w.b < 0) break;
        const int tiles = tiles_of(w), nt = w.nt;
        // A slot is free when both warps have said so: each when its tile's MMAs have read it, or, for a tile without
        // rows, when the copy has landed.  That warp must not leave positions out: a parity tells a phase from the one
        // before it only, and copies may land in any order, so its wait in the next block could take a copy that is
        // still on its way for one that has landed.  With an e4m3 cache it may, and the other warp speaks for both: the
        // converting warps fill the ring in order, so a position that is filled says that all before it are.  (Going
        // along there too makes the compiler spill: pieces in an e4m3 cache 583 us against 554.)
        if (nt == 0 || x >= tiles) {
          if (E4M3) {
            ring += 2 * nt;
          } else {
            for (const int end = ring + 2 * nt; ring < end && ok; ++ring) {
              ok = wait_kv(ring);
              __syncwarp();  // the slot's next copy may land as soon as lane 0 has arrived
              if (ok && lane == 0) mbar_arrive(&kv_empty[ring % SLOTS]);
            }
          }
          done_with(item);
          continue;
        }
        auto release = [&](int n) {
          mma_commit(&kv_empty[n % SLOTS]);
          if (E4M3 && tiles == 1) mma_commit(&kv_empty[n % SLOTS]);
        };
        ok = mbar_wait(E4M3 ? &q_ready[x] : &q_full[x], qn & 1) && wait_kv(ring);
        ++qn;
        tc_fence_after();
        if (ok && elect_one()) {
          qk(ring % SLOTS);
          mma_commit(&s_full[x]);
          release(ring);
          if (nt == 1) mma_commit(&q_empty[x]);
        }
        __syncwarp();
        for (int i = 0; i < nt && ok; ++i, ++pn) {
          const bool more = i + 1 < nt;
          const int vn = ring + 1, kn = ring + 2;
          ring += 2;
          if (C::APART && more) {
            ok = wait_kv(kn) && mbar_wait(&s_read[x], pn & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              qk(kn % SLOTS);
              mma_commit(&s_full[x]);
              release(kn);
              if (i + 2 == w.nt) mma_commit(&q_empty[x]);
            }
            __syncwarp();
          }
          ok = wait_kv(vn);
          if (!ok) break;
          if (!E4M3) {
            // Rows of V that no row of the CTA sees: zeros, from both tiles' warps, each before its own MMAs (where the
            // other's MMAs already read the same zeros).
            const int base = tile_of(w, i) * BN;
            auto clear = [&](int lo, int hi) {
              uint8_t* v = kv_s + (vn % SLOTS) * C::KV_TILE;
              for (int j = lo * (D / 8) + lane; j < hi * (D / 8); j += 32) {
                const int r = j / (D / 8), ch = j % (D / 8);
                *reinterpret_cast<uint4*>(v + (ch / 8) * (BN * 128) + r * 128 + (ch & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
              }
            };
            if (base + BN - 1 > w.p_hi || (base < w.wlo && base + BN > w.send)) {
              clear(max(0, w.send - base), min(BN, w.wlo - base));
              clear(max(0, w.p_hi + 1 - base), BN);
              fence_proxy_async_smem();
              __syncwarp();
            }
          }
          if (C::EARLY) {
            ok = mbar_wait(&p_half[x], pn & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) pv(vn % SLOTS, 0, i > 0);
            __syncwarp();
          }
          ok = (C::APART || !more || wait_kv(kn)) && mbar_wait(&p_full[x], pn & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            if (!C::EARLY) pv(vn % SLOTS, 0, i > 0);
            pv(vn % SLOTS, 1, true);
            if (C::APART) {
              mma_commit(&o_full[x]);
              release(vn);
            } else if (more) {
              qk(kn % SLOTS);
              mma_commit(&s_full[x]);
              release(vn);
              release(kn);
              if (i + 2 == nt) mma_commit(&q_empty[x]);
            } else {
              mma_commit(&o_full[x]);
              release(vn);
            }
          }
          __syncwarp();
        }
        done_with(item);
      }
      if (!ok && lane == 0) atomicOr(p.err, DEVERR_TIMEOUT_MMA);
      if (elect_one()) mma_commit(&drain[x]);  // every MMA issued must finish before tensor memory is freed
      __syncwarp();
      mbar_wait(&drain[x], 0);
    } else {
      // ------------------------------------------------------------ copies
      // Warp 9 finds the CTA's work and copies K; warp 11 copies Q and V.
      const bool keys = warp == 9;
      constexpr int BOX_D = E4M3 ? D : 64;                 // dims per box
      constexpr int BOX_STRIDE = BN * 128;                 // between a tile's halves
      constexpr int RING = E4M3 ? RAW : SLOTS;
      uint64_t* full = E4M3 ? raw_full : kv_full;
      uint64_t* empty = E4M3 ? raw_empty : kv_empty;
      const int page_size = 1 << p.cache.page_shift, pages = BN >> p.cache.page_shift;
      bool ok = true, asked = false;
      int ring = 0, last = -1, block = blockIdx.x, total = 0;
      uint32_t qn[2] = {0, 0};
      Rows mine = {0, 0, 0};
      Deal deal = {};
      Groups groups = {};
      unsigned int unit = 0, unit_end = 0;
      if (SHARED && keys) {
        long long tokens = 0, times = 0;
        const int most = p.table_width << p.cache.page_shift;
        for (int b = lane; b < p.T; b += 32) tokens += counted_tokens(p.sh, b, p.T, p.seq_lens, most);
        deal.units = scan_groups(p, lane, blockIdx.x == 0, deal, 0, 0, 0, nullptr, nullptr, &groups, &times);
        if (p.sh.window == 0) tokens -= times;
#pragma unroll
        for (int m = 16; m; m >>= 1) tokens += __shfl_xor_sync(0xFFFFFFFFu, tokens, m);
        deal.ctas = max(1u, min(shared_sms<D, E4M3>(deal.units, tokens, p.kv_heads, gridDim.x), deal.units / kLeastUnits));
        deal.per = deal.units / deal.ctas, deal.extra = deal.units % deal.ctas;
        if (blockIdx.x < deal.ctas) unit = deal.begin(blockIdx.x), unit_end = deal.begin(blockIdx.x + 1);
      }
      if (!SHARED && keys) total = count_blocks(p, lane, blockIdx.x == 0, mine);
      int item = 0;
      for (; ok; ++item) {
        Work w;
        if (keys) {
          if (item >= 2) ok = mbar_wait(&work_empty[item & 1], ((item >> 1) - 1) & 1);
          if (!ok) break;
          if (SHARED)
            scan_groups(p, lane, false, deal, unit, unit_end, blockIdx.x, &s_work[item & 1], &s_pieces[item & 1], &groups,
                        nullptr);
          else
            find_work(p, block, total, item == 0 ? &mine : nullptr, lane, &s_work[item & 1]);
          w = s_work[item & 1];
          if (lane == 0) mbar_arrive(&work_full[item & 1]);
          if (w.b < 0) break;
          if (!SHARED) {
            if (lane == 0) {
              mbar_arrive_expect_tx(stolen, 16);
              steal_block(&s_response, stolen);
            }
            asked = true;
          }
        } else {
          ok = wait_work(item);
          if (!ok) break;
          w = s_work[item & 1];
          done_with(item);
          if (w.b < 0) break;
          if (w.nt > 0) {
            for (int x = 0; x < tiles_of(w) && ok; ++x) {
              if (qn[x] > 0) ok = mbar_wait(&q_empty[x], (qn[x] - 1) & 1);
              if (!ok) break;
              ++qn[x];
              if (lane == 0) {
                mbar_arrive_expect_tx(&q_full[x], p.tile_tokens * p.group * D * 2);
                for (int h = 0; h < D / 64; ++h)
                  tma_load_3d(q_s + x * C::Q_TILE + h * (BM * 128), &qmap, &q_full[x], 64 * h, w.hk * p.group,
                              w.row0 + x * p.tile_tokens);
              }
              __syncwarp();
            }
          }
        }
        const int32_t* table = p.page_table + int64_t(w.b) * p.ld_table;
        const CUtensorMap* map = keys ? &kmap : &vmap;
        for (int i = 0; i < w.nt && ok; ++i) {
          // lane j < pages: page j of the tile, if some row sees a token of it
          const int a = tile_of(w, i) * BN + lane * page_size, z = a + page_size - 1;
          const bool need = lane < pages && a <= w.p_hi && (z >= w.wlo || a < w.send);
          int page = 0;
          if (need) {
            page = __ldg(table + (a >> p.cache.page_shift));
            if (page < 0 || page >= p.cache.num_pages) {
              atomicOr(p.err, DEVERR_INDEX);
              page = 0;
            }
          }
          const int boxes = __popc(__ballot_sync(0xFFFFFFFFu, need));
          const int c = ring + 2 * i + (keys ? 0 : 1), slot = c % RING;
#ifdef SP24_FAULT_WITHHOLD_FIRST_STAGE
          if (c == 0) continue;  // the fault-test build: each CTA's first keys never come
#endif
          if (c >= RING) ok = mbar_wait(&empty[slot], (c / RING - 1) & 1);
          if (!ok) break;
          last = c;
          if (lane == 0) mbar_arrive_expect_tx(&full[slot], boxes * page_size * D * (E4M3 ? 1 : 2));
          __syncwarp();
          if (need) {
            uint8_t* dst = (E4M3 ? raw_s + slot * C::RAW_TILE : kv_s + slot * C::KV_TILE) +
                           lane * page_size * (E4M3 ? D : 128);
#pragma unroll
            for (int h = 0; h < D / BOX_D; ++h)
              tma_load_4d(dst + h * BOX_STRIDE, map, &full[slot], BOX_D * h, 0, w.hk, page);
          }
          __syncwarp();
        }
        ring += 2 * w.nt;
        if (SHARED && keys) unit += w.nt;
        if (!SHARED && keys && ok) {
          ok = mbar_wait(stolen, item & 1);
          if (!ok) break;
          asked = false;
          block = stolen_block(&s_response);
          fence_proxy_async_smem();  // read before the next answer is written
          __syncwarp();
        }
      }
      if (!ok && lane == 0) atomicOr(p.err, DEVERR_TIMEOUT_PRODUCER);
      // Copies in flight have to land before this CTA's shared memory goes, also where only other warps gave up on them:
      // of each slot the last copy, whichever warp's it is (a parity cannot tell a copy that has been overtaken from one
      // that has not landed, so both warps have to be done first).
      if (lane == 0) s_last[keys ? 0 : 1] = last;
      __syncwarp();
      asm volatile("bar.sync 1, 64;" ::: "memory");  // the two copying warps
      if (keys) {
        const int top = max(s_last[0], s_last[1]);
#pragma unroll 1
        for (int n = top; n > top - RING; --n) {
          const int c = n <= s_last[n & 1] ? n : n - RING;
          if (c >= 0) mbar_wait(&full[c % RING], (c / RING) & 1);
        }
      } else {
#pragma unroll 1
        for (int x = 0; x < 2; ++x)
          if (qn[x] > 0) mbar_wait(&q_full[x], (qn[x] - 1) & 1);
      }
      if (asked) mbar_wait(stolen, item & 1);
    }
  } else if (E4M3) {
    // -------------------------------------------------------------- e4m3 -> f16
    setmaxnreg_dec<C::REG_CONVERT>();
    constexpr int R = RAW ? RAW : 1;
    const int r = tid & 127;  // this thread's token of each tile
    bool ok = true;
    int ring = 0;
    for (int item = 0; ok; ++item) {
      ok = wait_work(item);
      const Work w = s_work[item & 1];
      if (!ok || w.b < 0) break;
      for (int i = 0; i < 2 * w.nt && ok; ++i, ++ring) {
        const int from = ring % R, slot = ring % SLOTS;
        ok = mbar_wait(&raw_full[from], (ring / R) & 1);
        if (ok && ring >= SLOTS) ok = mbar_wait(&kv_empty[slot], (ring / SLOTS - 1) & 1);
        if (!ok) break;
        const int j = tile_of(w, i >> 1) * BN + r;
        const bool seen = j <= w.p_hi && (j >= w.wlo || j < w.send);
        const uint8_t* src = raw_s + from * C::RAW_TILE + r * D;
        uint8_t* dst = kv_s + slot * C::KV_TILE + r * 128;
        const int sw = D == 128 ? (r & 7) : ((r >> 1) & 3);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint4 v = *reinterpret_cast<const uint4*>(src + ((i ^ sw) << 4));
          if (!seen) v = make_uint4(0, 0, 0, 0);
          uint8_t* to = dst + (i / 4) * (BN * 128);
          const int c0 = (2 * i) & 7;
          *reinterpret_cast<uint4*>(to + ((c0 ^ (r & 7)) << 4)) =
              make_uint4(e4m3x2_f16x2(v.x), e4m3x2_f16x2(v.x >> 16), e4m3x2_f16x2(v.y), e4m3x2_f16x2(v.y >> 16));
          *reinterpret_cast<uint4*>(to + (((c0 + 1) ^ (r & 7)) << 4)) =
              make_uint4(e4m3x2_f16x2(v.z), e4m3x2_f16x2(v.z >> 16), e4m3x2_f16x2(v.w), e4m3x2_f16x2(v.w >> 16));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&raw_empty[from]);
          mbar_arrive(&kv_full[slot]);
        }
      }
      done_with(item);
    }
    if (!ok && lane == 0) atomicOr(p.err, DEVERR_TIMEOUT_PRODUCER);
  }
  tc_fence_before();
  __syncthreads();
  pdl_trigger();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Adds up the parts of the blocks' rows (splits > 1): a warp per row (two rows
// with heads of 64), whose lanes first look at a part's maximum and sum each.
// Always in the same order: the result does not depend on timing.
constexpr int kJoinWarps = 4;
constexpr int kMostSplits = 32;
template <int D>
constexpr int kJoinRows = kJoinWarps * (128 / D);  // rows per CTA
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) attention_join_kernel(const __grid_constant__ PromptParams p) {
  __shared__ Work s_work;
  constexpr int LPR = D / 4, RPW = 32 / LPR, CHUNKS = BM / kJoinRows<D>;  // lanes per row, rows per warp
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int item = blockIdx.x / (2 * CHUNKS);  // rank * kv_heads + kv head
  const int x = blockIdx.x / CHUNKS % 2, r = blockIdx.x % CHUNKS * kJoinRows<D> + warp * RPW + lane / LPR;
  pdl_wait();
  if (warp == 0) {
    Rows mine;
    const int total = count_blocks(p, lane, false, mine);
    find_work(p, (item / p.kv_heads) * p.splits * p.kv_heads + item % p.kv_heads, total, &mine, lane,
              &s_work);
  }
  __syncthreads();
  const Work w = s_work;
  const int token = token_of(p, r), at = x * p.tile_tokens + token;
  const bool mine = w.b >= 0 && token < p.tile_tokens && at < w.rows;
  if (__any_sync(0xFFFFFFFFu, mine)) {
    // (Rows of another token's, or of no one's, go along: their parts are there, too, or not a number.)
    const int64_t row = static_cast<int64_t>(w.part) * (2 * BM) + x * BM + r;
    const float* ml = p.part + static_cast<int64_t>(p.parts) * (2 * BM * D) + 2 * row;
    const float* o = p.part + row * D + lane % LPR * 4;
    float2 v[kMostSplits / LPR];  // parts lane % LPR and, with heads of 64, 16 more
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kMostSplits / LPR; ++k) {
      const int s = k * LPR + lane % LPR;
      v[k] = s < p.splits ? __ldcg(reinterpret_cast<const float2*>(ml + s * (2 * BM * 2))) : make_float2(-INFINITY, 0.0f);
      top = fmaxf(top, v[k].x);
    }
#pragma unroll
    for (int m = LPR / 2; m; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
    const float use = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int k = 0; k < kMostSplits / LPR; ++k) {
      v[k].x = ex2(v[k].x - use);
      sum = fmaf(v[k].y, v[k].x, sum);
    }
#pragma unroll
    for (int m = LPR / 2; m; m >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, m);
    float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < kMostSplits / LPR; ++k) {
#pragma unroll 8
      for (int i = 0; i < LPR; ++i) {
        const int s = k * LPR + i;
        if (s >= p.splits) break;  // uniform
        const float f = __shfl_sync(0xFFFFFFFFu, v[k].x, (lane & ~(LPR - 1)) + i);
        if (f != 0.0f) {  // (a part without keys has written no O)
          const float4 y = __ldcg(reinterpret_cast<const float4*>(o + static_cast<int64_t>(s) * (2 * BM * D)));
          acc.x = fmaf(y.x, f, acc.x), acc.y = fmaf(y.y, f, acc.y);
          acc.z = fmaf(y.z, f, acc.z), acc.w = fmaf(y.w, f, acc.w);
        }
      }
    }
    if (mine) {
      const float f = sum == 0.0f ? 0.0f : (p.cache.v_scale ? p.cache.v_scale[w.hk] : 1.0f) / sum;
      __nv_bfloat16* y = p.y + static_cast<int64_t>(w.row0 + at) * p.ldy +
                         static_cast<int64_t>(w.hk * p.group + r - token * p.group) * D + (lane % LPR) * 4;
      *reinterpret_cast<uint2*>(y) = make_uint2(bf16x2_rn(acc.x * f, acc.y * f), bf16x2_rn(acc.z * f, acc.w * f));
    }
  }
  pdl_trigger();
}

// Blocks of query rows of a call, at most (every sequence's last may be partly
// filled), and into how many parts each is cut: where the blocks leave SMs idle
// and the cache may be long, one part per SM, of at least kLeastTiles key tiles.
// (32/8 heads of 128, cut against whole: 16 rows over 100000 keys 74 us and
// 900, 200 over 10000 41 and 121, 64 over 4000 19 and 48, 64 over 1000 19 and
// 21.  With 6 tiles per part 64 over 4000 takes 22 us, with 8 23.)
struct Shape {
  int64_t blocks;
  int splits;
};
inline Shape shape_of(int64_t T, int64_t B, int q_heads, const sp24_kv_cache& c, int64_t table_width, int window,
                      int sinks, int sms) {
  const int64_t tokens = 2 * (BM / (q_heads / c.heads));
  Shape s = {T / tokens + B, 1};
  int64_t keys = table_width * c.page_size;
  if (window > 0) keys = std::min(keys, int64_t(window) + tokens + std::min(sinks, kMostTokens) + 2 * BN);
  const int64_t idle = sms / std::max<int64_t>(1, s.blocks * c.heads);
  const int64_t most = std::min<int64_t>({idle, keys / (kLeastTiles * BN), kMostSplits});
  if (most > 1) s.splits = static_cast<int>(most);
  return s;
}
inline size_t part_bytes(const Shape& s, int heads, int D) {
  return s.splits > 1 ? static_cast<size_t>(s.blocks) * heads * s.splits * (2 * BM) * (D + 2) * 4 : 0;
}

template <int D, bool E4M3>
sp24_status make_maps(const PromptParams& p, const void* q, int64_t ldq, int q_heads, const sp24_kv_cache& cache,
                      CUtensorMap& qmap, CUtensorMap& kmap, CUtensorMap& vmap) {
  {
    const uint64_t dims[3] = {uint64_t(D), uint64_t(q_heads), uint64_t(p.T)};
    const uint64_t strides[2] = {uint64_t(D) * 2, uint64_t(ldq) * 2};
    const uint32_t box[3] = {64, uint32_t(p.group), uint32_t(p.tile_tokens)};
    if (sp24_status st = make_tmap_nd(&qmap, q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, dims, strides, box,
                                      CU_TENSOR_MAP_SWIZZLE_128B))
      return st;
  }
  const uint64_t dims[4] = {uint64_t(D), uint64_t(cache.page_size), uint64_t(cache.heads), uint64_t(cache.num_pages)};
  const uint64_t strides[3] = {uint64_t(p.cache.token_stride), uint64_t(p.cache.head_stride),
                               uint64_t(p.cache.page_stride)};
  const uint32_t box[4] = {uint32_t(E4M3 ? D : 64), uint32_t(cache.page_size), 1, 1};
  const auto type = E4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto swizzle = E4M3 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  if (sp24_status st = make_tmap_nd(&kmap, cache.k, type, 4, dims, strides, box, swizzle)) return st;
  return make_tmap_nd(&vmap, cache.v, type, 4, dims, strides, box, swizzle);
}

template <int D, bool E4M3>
sp24_status launch(const PromptParams& p, const void* q, int64_t ldq, int q_heads, const sp24_kv_cache& cache,
                   const DeviceInfo& dev, int64_t blocks, cudaStream_t s) {
  using C = Cfg<D, E4M3>;
  CUtensorMap qmap, kmap, vmap;
  if (sp24_status st = make_maps<D, E4M3>(p, q, ldq, q_heads, cache, qmap, kmap, vmap)) return st;
  if (launch_pdl_smem<attention_prompt_kernel<C>>(dev, dim3(static_cast<unsigned>(blocks * p.splits * p.kv_heads)),
                                                  dim3(C::THREADS), C::SMEM, s, qmap, kmap, vmap, p) != cudaSuccess)
    return SP24_ERR_CUDA;
  if (p.splits > 1 &&
      launch_pdl(attention_join_kernel<D>, dim3(static_cast<unsigned>(blocks * p.kv_heads * 2 * (BM / kJoinRows<D>))),
                 dim3(kJoinWarps * 32), 0, s, p) != cudaSuccess)
    return SP24_ERR_CUDA;
  return SP24_OK;
}

template <int D, bool E4M3>
sp24_status launch_shared(const PromptParams& p, const SharedCall& c, const DeviceInfo& dev, cudaStream_t s) {
  using C = Cfg<D, E4M3>;
  CUtensorMap qmap, kmap, vmap;
  if (sp24_status st = make_maps<D, E4M3>(p, c.q, c.ldq, c.q_heads, *c.cache, qmap, kmap, vmap)) return st;
  const cudaError_t r = launch_pdl_smem<attention_prompt_kernel<C, true>>(dev, dim3(dev.sm_count), dim3(C::THREADS), C::SMEM, s,
                                                                          qmap, kmap, vmap, p);
  return r == cudaSuccess ? SP24_OK : SP24_ERR_CUDA;
}

}  // namespace

sp24_status launch_shared_tokens(const SharedCall& c, const DeviceInfo& dev, cudaStream_t s) {
  PromptParams p = {};
  p.T = c.B;
  p.cache = c.view;
  p.page_table = c.page_table;
  p.table_width = c.table_width;
  p.ld_table = c.ld_table;
  p.seq_lens = c.seq_lens;
  p.scale = c.scale;
  p.kv_heads = c.cache->heads;
  p.group = c.q_heads / c.cache->heads;
  p.tile_tokens = BM / p.group;
  p.inv_group = (65536u + p.group - 1) / p.group;
  p.splits = 1;
  p.err = dev.err_word;
  p.sh = c.groups;
  if (c.cache->head_dim == 128)
    return c.cache->dtype == SP24_E4M3 ? launch_shared<128, true>(p, c, dev, s) : launch_shared<128, false>(p, c, dev, s);
  return c.cache->dtype == SP24_E4M3 ? launch_shared<64, true>(p, c, dev, s) : launch_shared<64, false>(p, c, dev, s);
}
}  // namespace sp24

extern "C" size_t sp24_attention_prompt_workspace_size(int64_t T, int64_t B, int q_heads, const sp24_kv_cache* cache,
                                                       int64_t table_width, int window, int sinks) {
  using namespace sp24;
  CacheView view;
  const DeviceInfo* dev = nullptr;
  if (check_cache(cache, &view) || T <= 0 || T > kMostTokens || B <= 0 || B > kMostTokens || q_heads < 1 ||
      q_heads % cache->heads || q_heads / cache->heads > BM || table_width < 1 ||
      table_width > (kMostTokens >> view.page_shift) || window < 0 || sinks < 0 || current_device(&dev))
    return 0;
  return part_bytes(shape_of(T, B, q_heads, *cache, table_width, effective_window(window), sinks, dev->sm_count),
                    cache->heads, cache->head_dim);
}

extern "C" sp24_status sp24_attention_prompt(const void* q, int64_t T, int64_t ldq, int q_heads, const int32_t* cu_q,
                                             int64_t B, const sp24_kv_cache* cache, const int32_t* page_table,
                                             int64_t table_width, int64_t ld_table, const int32_t* seq_lens,
                                             float scale, int window, int sinks, void* Y, int64_t ldy,
                                             void* workspace, size_t workspace_bytes, void* stream) {
  using namespace sp24;
  PromptParams p = {};
  if (sp24_status st = check_attention(q, T, ldq, q_heads, cache, page_table, table_width, ld_table, seq_lens, B, scale,
                                       window, sinks, Y, ldy, &p.cache))
    return st;
  if (T > 0 && B > 0 && !cu_q) return SP24_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(cu_q) & 3u) return SP24_ERR_ALIGNMENT;
  const DeviceInfo* dev = nullptr;
  if (sp24_status st = current_device(&dev)) return st;
  if (T == 0 || B == 0) return SP24_OK;
  p.T = static_cast<int>(T);
  p.B = static_cast<int>(B);
  p.cu_q = cu_q;
  p.page_table = page_table;
  p.table_width = static_cast<int>(table_width);
  p.ld_table = ld_table;
  p.seq_lens = seq_lens;
  p.scale = scale;
  p.window = effective_window(window);
  p.sinks = sinks;
  p.y = static_cast<__nv_bfloat16*>(Y);
  p.ldy = ldy;
  p.kv_heads = cache->heads;
  p.group = q_heads / cache->heads;
  p.tile_tokens = BM / p.group;
  p.inv_group = (65536u + p.group - 1) / p.group;
  p.err = dev->err_word;
  Shape shape = shape_of(T, B, q_heads, *cache, table_width, p.window, sinks, dev->sm_count);
  if (!aligned16(workspace)) return SP24_ERR_ALIGNMENT;
  if (shape.splits > 1 && (!workspace || workspace_bytes < part_bytes(shape, cache->heads, cache->head_dim)))
    shape.splits = 1;
  if (shape.blocks * shape.splits > INT32_MAX / 2 / p.kv_heads) return SP24_ERR_UNSUPPORTED;
  p.splits = shape.splits;
  p.parts = static_cast<int>(shape.blocks * p.kv_heads * shape.splits);
  p.part = static_cast<float*>(workspace);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool e4m3 = cache->dtype == SP24_E4M3;
  if (cache->head_dim == 128)
    return e4m3 ? launch<128, true>(p, q, ldq, q_heads, *cache, *dev, shape.blocks, s) : launch<128, false>(p, q, ldq, q_heads, *cache, *dev, shape.blocks, s);
  return e4m3 ? launch<64, true>(p, q, ldq, q_heads, *cache, *dev, shape.blocks, s) : launch<64, false>(p, q, ldq, q_heads, *cache, *dev, shape.blocks, s);
}
