// sp24_attn_decode.cu -- sp24_attention_decode: one new token per sequence
// over the paged cache.
//
//   Y[h] = sum_j p_j v_j / sum_j p_j,  p_j = exp2(c (q_h . k_j) - m_h),
//   c = scale log2(e) (times the cache's scale), m_h the running maximum
//
// Bound by memory: every visible key and value is read once, for all query
// heads that share it.  What follows from that:
// - The visible keys of all (sequence, kv head) pairs are cut into tiles of
//   equal size and dealt out to the CTAs in equal contiguous ranges, whatever
//   the lengths (which only the device knows).  A pair that is cut between CTAs
//   is joined by the CTA that finishes last, from fp32 partials in the
//   workspace, in the order of the keys: the result does not depend on timing.
// - Within a CTA every warp streams its own chunks of a tile through its own
//   ring of shared memory (cp.async, no barrier in the loop), with a running
//   maximum and sum of its own; the warps are joined at the end of a pair, while
//   the next pair's first keys are on their way.
//   Keys outside [lo, hi) of a chunk are not read: zeros take their place, so
//   whatever the cache holds there (NaN too) cannot reach a sum.
// - The few query heads of a pair are the narrow side of the products: S^T =
//   K Q^T and O^T = V^T P^T with keys, then dims, on the 16-row side of
//   mma.sync m16n8k16 and 8 heads on the other, so 8 heads waste nothing (with
//   heads on the 16-row side, half the products and half the registers of O
//   would be padding).  tcgen05 would want 128 rows.
// - The weights enter the tensor core as bf16 (f16 with an e4m3 cache), which
//   moves a result by 2^-8 of the weighted mean of |v| at most and in the mean far
//   less; their sum is of the fp32 values.
// - e4m3 codes become f16 in registers (exactly), so the products of an e4m3
//   cache are f16 ones; each query head is scaled by a power of two, which
//   keeps bf16 queries within f16's range, and each weight by 2^15 (kUp).
//
// Measured (GB300, 32/8 heads of 128 but for the last): one sequence of 131071
// tokens 88 us, 6.1 TB/s (90 % of the measured copy rate); 64 of 1 to 16000
// in an e4m3 cache 171 us, 6.2 TB/s (92 %); one of 1000 tokens 7.3 us, of
// which the keys take 1: launch, lengths, pages, keys and the join of 16 pieces
// are a chain of seven memory latencies; 128 of up to 9000 tokens under a
// window of 2000 with 4 sinks, 28/4 heads of 64, 45.8 us, 5.1 TB/s (75 %).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "sp24_attn.cuh"
#include "sp24_ptx.cuh"

namespace sp24 {
namespace {

constexpr int kWarps = 4;           // per CTA (2, and twice the CTAs: 131071 tokens 95 us against 88; 8, and half: e4m3 178
                                    // us against 170)
constexpr int kThreads = kWarps * 32;
constexpr int kCtasPerSm = 2;
constexpr int kHalf = 4096;         // bytes of keys (and of values) per chunk and stage
constexpr int kStageBytes = 2 * kHalf;
constexpr int kPieces = 16;         // of a pair, that a thread joins in one round of loads

struct DecodeParams {
  const __nv_bfloat16* q;
  int64_t ldq;
  int B;
  CacheView cache;
  const int32_t* page_table;
  int table_width;
  int64_t ld_table;
  const int32_t* seq_lens;
  float scale;
  int window, sinks;
  __nv_bfloat16* y;
  int64_t ldy;
  int kv_heads, group, head_blocks;  // head_blocks: CTA-wide blocks of 8 NH query heads per kv head
  float* partials;                   // [2 slots per CTA][8 NH][D], then [2 slots][8 NH][2] maxima and sums
  unsigned int* counters;            // [CTAs] pieces that arrived, by the pair's first CTA
  unsigned int* err;
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A sequence's visible keys are those of its sinks, [0, sinks), and those of
// its window, [lo, n).  In chunks of CT: the sinks' from token 0, then the
// window's from `from`, a multiple of 16 (so that 16 tokens in a row never
// cross a page).  A tile is kWarps chunks in a row.
struct Span {
  int n;             // tokens
  int lo, sinks;
  int from;          // where the window's chunks begin
  int sink_chunks, tiles;
};

template <int CT>
__device__ __forceinline__ Span span_of(const DecodeParams& p, int n, bool report) {
  Span s;
  const int most = p.table_width << p.cache.page_shift;
  if (n < 0 || n > most) {
    if (report) atomicOr(p.err, DEVERR_INDEX);
    n = n < 0 ? 0 : most;
  }
  s.n = n;
  s.lo = p.window > 0 && n > p.window ? n - p.window : 0;
  s.sinks = min(p.sinks, s.lo);
  if (s.sinks == s.lo) s.lo = s.sinks = 0;
  s.from = s.lo & ~15;
  s.sink_chunks = (s.sinks + CT - 1) / CT;
  const int chunks = s.sink_chunks + (n - s.from + CT - 1) / CT;
  s.tiles = max(1, (chunks + kWarps - 1) / kWarps);  // an empty sequence has one, without keys
  return s;
}

// With an e4m3 cache weights, and their sums, are 2^kUp times p_j: the largest is
// 2^15, near f16's end, so that those down to 2^-29 of it keep all 11 bits, and
// one is off by 2^-40 of the largest at most.  (With the largest at 1 f16's
// smallest step is 2^-24 of it: of 131071 keys some 17 nats below one other, half
// a percent of the sum, each would be rounded by up to a half.)
constexpr float kUp = 15.0f;

// Stages of a warp's ring.  e4m3: 3 (64 ragged sequences 169.6 us, 172.2 with
// 2), but 2 where 16 heads' exchange buffer takes the room.  bf16: 2 (131071
// tokens 86.6 us against 87.5, 128 windowed sequences 45.7 against 47.2).
template <bool E4M3, int NH>
constexpr int kStages = E4M3 && NH == 1 ? 3 : 2;
template <int D, bool E4M3, int NH>
constexpr int kSmem = kWarps * (kStages<E4M3, NH> * kStageBytes + 8 * NH * (D + 4) * 4);

// What a CTA does in one go: tiles t0 .. t1 - 1 of a sequence, for one kv head
// and up to 8 NH of its query heads.
struct Item {
  int b, hh, t0, t1;
  Span sp;
};

template <int D, bool E4M3, int NH>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) attention_decode_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int ROWB = D * (E4M3 ? 1 : 2);   // bytes of a token's key
  constexpr int CT = kHalf / ROWB;           // tokens per chunk: 16, 32 or 64
  constexpr int MT = CT / 16;
  constexpr int PIECES = ROWB / 16;          // 16-byte pieces of a row
  constexpr int RPI = 32 / PIECES;           // rows that a warp's 32 pieces cover: 2, 4 or 8
  constexpr int LOADS = CT / RPI;            // loads per lane and chunk half: 8
  constexpr int HEADS = 8 * NH;
  constexpr int PAD = D + 4;                 // row of the exchange buffer, in floats
  constexpr int S = kStages<E4M3, NH>, RING = S * kStageBytes;
  static_assert(LOADS == 8, "");

  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_sum[2][kWarps];
  __shared__ int s_found[2];
  __shared__ float s_m[kWarps][HEADS], s_l[kWarps][HEADS];
  __shared__ unsigned int s_last;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t ring_a = smem_u32(smem + warp * RING);
  float* const exchange = reinterpret_cast<float*>(smem + kWarps * RING);  // [kWarps][HEADS][PAD]
  pdl_wait();

  // ---- this CTA's range of tiles
  const int HH = p.kv_heads * p.head_blocks;
  // Tiles of the sequences: a sum over all, and a running sum over the first kThreads.
  auto tiles_of = [&](int x, bool report) {
    return x < p.B ? span_of<CT>(p, __ldg(p.seq_lens + x), report).tiles : 0;
  };
  auto scan = [&](int x) {  // inclusive, over the warp
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, m);
      if (lane >= m) x += y;
    }
    return x;
  };
  int own = tiles_of(tid, blockIdx.x == 0), rest = 0;
  for (int x = tid + kThreads; x < p.B; x += kThreads) rest += tiles_of(x, blockIdx.x == 0);
  int incl = scan(own);
  if (p.B > kThreads) {
#pragma unroll
    for (int m = 16; m; m >>= 1) rest += __shfl_xor_sync(0xFFFFFFFFu, rest, m);
  }
  if (lane == 31) s_sum[0][warp] = incl, s_sum[1][warp] = rest;
  __syncthreads();
  unsigned int total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += s_sum[0][w] + s_sum[1][w];
  total *= HH;
  const unsigned int ctas = min(gridDim.x, total), cta = blockIdx.x;
  if (cta >= ctas) return;  // uniform
  const unsigned int per = total / ctas, extra = total % ctas;  // the first `extra` CTAs take a tile more
  unsigned int u = cta * per + min(cta, extra);
  const unsigned int u_end = u + per + (cta < extra ? 1u : 0u);
  auto cta_of = [&](unsigned int x) {
    return x < extra * (per + 1) ? x / (per + 1) : extra + (x - extra * (per + 1)) / per;
  };
  // The sequence that tile u belongs to, and the tiles (of one head) of those before it.
  int b = 0, before = 0;
  {
    const int want = static_cast<int>(u / HH);
    for (int b0 = 0, seen = 0;; b0 += kThreads) {
      int base = seen, all = seen;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) base += s_sum[0][w];
        all += s_sum[0][w];
      }
      incl += base;
      if (want < incl && want >= incl - own) {
        s_found[0] = b0 + tid;
        s_found[1] = incl - own;
      }
      __syncthreads();
      if (want < all || b0 + kThreads >= p.B) break;  // uniform
      seen = all;
      own = tiles_of(b0 + kThreads + tid, false);
      incl = scan(own);
      if (lane == 31) s_sum[0][warp] = incl;
      __syncthreads();
    }
    b = s_found[0];
    before = s_found[1];
  }

  Item it;
  it.b = b;
  it.sp = span_of<CT>(p, __ldg(p.seq_lens + b), false);
  // The item that tile u of the launch begins.
  auto place = [&](Item& x) {
    const unsigned int local = u - static_cast<unsigned int>(before) * HH;
    x.hh = local / x.sp.tiles;
    x.t0 = local % x.sp.tiles;
    x.t1 = min(x.sp.tiles, x.t0 + static_cast<int>(u_end - u));
  };
  place(it);

  // ---- loads of chunks into stages
  const int row0 = lane / PIECES;
  auto chunk_at = [&](const Item& x, int ti, int& tok, int& lo, int& hi) {
    const int q = ti * kWarps + warp;
    if (q < x.sp.sink_chunks) {
      tok = q * CT;
      lo = 0, hi = x.sp.sinks;
    } else {
      tok = x.sp.from + (q - x.sp.sink_chunks) * CT;
      lo = x.sp.lo, hi = x.sp.n;
    }
  };
  // Page of each 16 tokens of the chunks ahead: lane i holds chunk (batch + i)'s.
  int page_now[MT], page_next[MT], page_then[MT];
  auto fetch_pages = [&](const Item& x, int ti, int (&out)[MT]) {
    const int32_t* table = p.page_table + int64_t(x.b) * p.ld_table;
    int tok = 0, lo = 0, hi = 0;
    if (ti < x.t1) chunk_at(x, ti, tok, lo, hi);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int j = tok + 16 * i;
      out[i] = 0;
      if (ti < x.t1 && j < hi && j + 16 > lo) {
        int id = __ldg(table + (j >> p.cache.page_shift));
        if (id < 0 || id >= p.cache.num_pages) {
          atomicOr(p.err, DEVERR_INDEX);
          id = 0;
        }
        out[i] = id;
      }
    }
  };
  auto issue = [&](const Item& x, int ti, int stage) {
    if (ti < x.t1) {
      int tok, lo, hi;
      chunk_at(x, ti, tok, lo, hi);
      const bool whole = tok >= lo && tok + CT <= hi;
      if (whole || (tok < hi && tok + CT > lo)) {
        const int64_t head = (x.hh / p.head_blocks) * p.cache.head_stride + (lane % PIECES) * 16;
        const uint32_t dst = ring_a + stage * kStageBytes;
        const int in_page = tok & ((1 << p.cache.page_shift) - 1);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
          const int sub = i * RPI / 16, row = i * RPI + row0;
          const int page = __shfl_sync(0xFFFFFFFFu, page_now[sub], (ti - x.t0) & 31);
          const int64_t at = page * p.cache.page_stride + head +
                             (((in_page + sub * 16) & ((1 << p.cache.page_shift) - 1)) + (row & 15)) *
                                 p.cache.token_stride;
          const int sw = ROWB >= 128 ? (row & 7) : ((row >> 1) & 3);
          const uint32_t to = dst + row * ROWB + (((lane % PIECES) ^ sw) << 4);
          const bool ok = whole || (tok + row >= lo && tok + row < hi);
          cp_async_16(to, p.cache.k + (ok ? at : 0), ok ? 16u : 0u);
          cp_async_16(to + kHalf, p.cache.v + (ok ? at : 0), ok ? 16u : 0u);
        }
      }
    }
    cp_async_commit();
  };
  fetch_pages(it, it.t0 + lane, page_now);
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(it, it.t0 + i, i);
  int stage = 0;

  while (true) {
    fetch_pages(it, it.t0 + 32 + lane, page_next);
    // The item after this one, and the pages of its first chunks: their copies are issued as soon as this one's keys
    // are done, before the warps are joined.
    const int tile0 = before * HH + it.hh * it.sp.tiles;  // the pair's first tile in the launch
    u += it.t1 - it.t0;
    const bool more = u < u_end;
    Item nx = it;
    if (more) {
      if (it.hh == HH - 1) {
        before += it.sp.tiles;
        nx.b = it.b + 1;
        nx.sp = span_of<CT>(p, __ldg(p.seq_lens + nx.b), false);
      }
      place(nx);
      fetch_pages(nx, nx.t0 + lane, page_then);
    }
    const int b = it.b, hk = it.hh / p.head_blocks, hb = it.hh % p.head_blocks;
    const int h0 = hk * p.group + hb * HEADS;                // first query head
    const int heads = min(HEADS, p.group - hb * HEADS);

    // ---- the queries, as the B operand of S^T = K Q^T (column g: head h0 + 8 n + g)
    uint32_t qf[NH][D / 16][2];
    float c[NH][2];      // score factor of heads 2t, 2t + 1
    const float c0 = p.scale * 1.4426950408889634f * (E4M3 ? p.cache.k_scale[hk] : 1.0f);
#pragma unroll
    for (int n = 0; n < NH; ++n) {
      const bool ok = 8 * n + g < heads;
      const __nv_bfloat16* q = p.q + b * p.ldq + int64_t(h0 + 8 * n + g) * D;
      if (!E4M3) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          qf[n][k][0] = ok ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 2 * t) : 0u;
          qf[n][k][1] = ok ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 2 * t + 8) : 0u;
        }
        c[n][0] = c[n][1] = c0;
      } else {
        // dims 4t .. 4t + 3 of each 16: the order in which a key's bytes arrive
        float top = 0.0f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint2 w = ok ? *reinterpret_cast<const uint2*>(q + 16 * k + 4 * t) : make_uint2(0, 0);
          qf[n][k][0] = w.x;
          qf[n][k][1] = w.y;
          top = fmaxf(top, fmaxf(fmaxf(fabsf(__uint_as_float(w.x << 16)), fabsf(__uint_as_float(w.x & 0xFFFF0000u))),
                                 fmaxf(fabsf(__uint_as_float(w.y << 16)), fabsf(__uint_as_float(w.y & 0xFFFF0000u)))));
        }
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        // 2^(exponent of the largest value), and 1 / it, both normal numbers; 1 for an endless row.  (A row below
        // 2^-63 is scaled as one of that size: its scores are zero to fp32 beside any other.)
        uint32_t e = __float_as_uint(top) >> 23;
        e = e == 255 ? 127u : min(max(e, 64u), 253u);
        const float up = __uint_as_float(e << 23), down = __uint_as_float((254u - e) << 23);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = qf[n][k][i];
            qf[n][k][i] = f16x2_rn(__uint_as_float(w << 16) * down, __uint_as_float(w & 0xFFFF0000u) * down);
          }
        c[n][0] = c0 * __shfl_sync(0xFFFFFFFFu, up, 8 * t);      // lane 4 * head holds that head's factor
        c[n][1] = c0 * __shfl_sync(0xFFFFFFFFu, up, 8 * t + 4);
      }
    }

    float o[NH][D / 16][4], m[NH][2], l[NH][2];
#pragma unroll
    for (int n = 0; n < NH; ++n) {
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][d][i] = 0.0f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
    }

    // ---- this warp's chunk of each tile
    for (int ti = it.t0; ti < it.t1; ++ti) {
      cp_async_wait<S - 2>();
      __syncwarp();
      {
        const int ahead = ti + S - 1;
        if (((ahead - it.t0) & 31) == 0) {
#pragma unroll
          for (int i = 0; i < MT; ++i) page_now[i] = page_next[i];
          fetch_pages(it, ahead + 32 + lane, page_next);
        }
        issue(it, ahead, stage == 0 ? S - 1 : stage - 1);
      }
      int tok, lo, hi;
      chunk_at(it, ti, tok, lo, hi);
      const uint32_t ks = ring_a + stage * kStageBytes, vs = ks + kHalf;
      stage = stage + 1 == S ? 0 : stage + 1;
      if (tok >= hi || tok + CT <= lo) continue;  // nothing visible: uniform over the warp

      float s[MT][NH][4];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
#pragma unroll
        for (int n = 0; n < NH; ++n) s[i][n][0] = s[i][n][1] = s[i][n][2] = s[i][n][3] = 0.0f;
        const int row = i * 16 + (lane & 15);
        const int sw = ROWB >= 128 ? (row & 7) : ((row >> 1) & 3);
        const uint32_t at = ks + row * ROWB;
        if (!E4M3) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            uint32_t a[4];
            ldmatrix4(a, at + (((2 * k + (lane >> 4)) ^ sw) << 4));
#pragma unroll
            for (int n = 0; n < NH; ++n) mma16816<false>(s[i][n], a[0], a[1], a[2], a[3], qf[n][k][0], qf[n][k][1]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < D / 16; k += 2) {
            uint32_t a[4];
            ldmatrix4(a, at + (((k + (lane >> 4)) ^ sw) << 4));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t a0 = e4m3x2_f16x2(a[2 * j]), a2 = e4m3x2_f16x2(a[2 * j] >> 16);
              const uint32_t a1 = e4m3x2_f16x2(a[2 * j + 1]), a3 = e4m3x2_f16x2(a[2 * j + 1] >> 16);
#pragma unroll
              for (int n = 0; n < NH; ++n) mma16816<true>(s[i][n], a0, a1, a2, a3, qf[n][k + j][0], qf[n][k + j][1]);
            }
          }
        }
      }
      if (tok < lo || tok + CT > hi) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const int j = tok + i * 16 + g;
          const bool a = j >= lo && j < hi, bb = j + 8 >= lo && j + 8 < hi;
#pragma unroll
          for (int n = 0; n < NH; ++n) {
            if (!a) s[i][n][0] = s[i][n][1] = -INFINITY;
            if (!bb) s[i][n][2] = s[i][n][3] = -INFINITY;
          }
        }
      }
      uint32_t pf[MT][NH][2];
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        float top[2] = {-INFINITY, -INFINITY}, less[2];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          top[0] = fmaxf(top[0], fmaxf(s[i][n][0], s[i][n][2]));
          top[1] = fmaxf(top[1], fmaxf(s[i][n][1], s[i][n][3]));
        }
        bool moved = false;
        float keep[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
          for (int mask = 4; mask < 32; mask <<= 1) top[x] = fmaxf(top[x], __shfl_xor_sync(0xFFFFFFFFu, top[x], mask));
          const float now = fmaxf(m[n][x], top[x] * c[n][x]);
          const float use = now == -INFINITY ? 0.0f : now;
          less[x] = E4M3 ? kUp - use : -use;
          keep[x] = ex2(m[n][x] - use);
          moved |= now > m[n][x];
          m[n][x] = now;
        }
        if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            l[n][x] *= keep[x];
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
              o[n][d][x] *= keep[x];
              o[n][d][2 + x] *= keep[x];
            }
          }
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          float e[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            e[x] = ex2(fmaf(s[i][n][x], c[n][x & 1], less[x & 1]));
            l[n][x & 1] += e[x];
          }
          // P^T with keys along k: [key g][heads 2t, 2t + 1] -> [head g][keys 2t, 2t + 1]
          pf[i][n][0] = movmatrix_trans(E4M3 ? f16x2_rn(e[0], e[1]) : bf16x2_rn(e[0], e[1]));
          pf[i][n][1] = movmatrix_trans(E4M3 ? f16x2_rn(e[2], e[3]) : bf16x2_rn(e[2], e[3]));
        }
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if (!E4M3) {
          const int row = i * 16 + ((lane >> 4) << 3) + (lane & 7);
          const uint32_t at = vs + row * ROWB;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            uint32_t a[4];
            ldmatrix4_trans(a, at + (((2 * d + ((lane >> 3) & 1)) ^ (row & 7)) << 4));
#pragma unroll
            for (int n = 0; n < NH; ++n) mma16816<false>(o[n][d], a[0], a[1], a[2], a[3], pf[i][n][0], pf[i][n][1]);
          }
        } else {
          // matrices: (keys 0-7, dims d), (keys 8-15, dims d), (keys 0-7, dims d + 1), (keys 8-15, dims d + 1);
          // a word holds dims 2g, 2g + 1 of keys 2t and 2t + 1: row g of O^T is dim 2g, row g + 8 dim 2g + 1
          const int row = i * 16 + (lane & 15);
          const int sw = ROWB >= 128 ? (row & 7) : ((row >> 1) & 3);
          const uint32_t at = vs + row * ROWB;
#pragma unroll
          for (int d = 0; d < D / 16; d += 2) {
            uint32_t a[4];
            ldmatrix4_trans(a, at + (((d + (lane >> 4)) ^ sw) << 4));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t x = __byte_perm(a[2 * j], 0, 0x3120), y = __byte_perm(a[2 * j + 1], 0, 0x3120);
              const uint32_t a0 = e4m3x2_f16x2(x), a1 = e4m3x2_f16x2(x >> 16);
              const uint32_t a2 = e4m3x2_f16x2(y), a3 = e4m3x2_f16x2(y >> 16);
#pragma unroll
              for (int n = 0; n < NH; ++n) mma16816<true>(o[n][d + j], a0, a1, a2, a3, pf[i][n][0], pf[i][n][1]);
            }
          }
        }
      }
    }

    if (more) {
#pragma unroll
      for (int i = 0; i < MT; ++i) page_now[i] = page_then[i];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < S - 1; ++i) issue(nx, nx.t0 + i, (stage + i) % S);
    }

    // ---- join the warps
    float* ex = exchange + warp * (HEADS * PAD);
#pragma unroll
    for (int n = 0; n < NH; ++n) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int mask = 4; mask < 32; mask <<= 1) l[n][x] += __shfl_xor_sync(0xFFFFFFFFu, l[n][x], mask);
        const int h = 8 * n + 2 * t + x;
        if (g == 0) {
          s_m[warp][h] = m[n][x];
          s_l[warp][h] = l[n][x];
        }
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          const int dim0 = E4M3 ? 16 * d + 2 * g : 16 * d + g, dim1 = E4M3 ? dim0 + 1 : dim0 + 8;
          ex[h * PAD + dim0] = o[n][d][x];
          ex[h * PAD + dim1] = o[n][d][2 + x];
        }
      }
    }
    __syncthreads();

    const bool cut = it.t0 > 0 || it.t1 < it.sp.tiles;
    const int slot = 2 * cta + (it.t0 == 0 ? 1 : 0);
    float* part = p.partials + int64_t(slot) * (HEADS * D);
    float* part_ml = p.partials + int64_t(2) * gridDim.x * (HEADS * D) + int64_t(slot) * (HEADS * 2);
    const float vscale = E4M3 ? p.cache.v_scale[hk] : 1.0f;
    for (int i = tid; i < heads * (D / 4); i += kThreads) {
      const int h = i / (D / 4), d = (i % (D / 4)) * 4;
      float top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][h]);
      const float use = top == -INFINITY ? 0.0f : top;
      float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(s_m[w][h] - use);
        const float4 v = *reinterpret_cast<const float4*>(exchange + (w * HEADS + h) * PAD + d);
        sum = fmaf(s_l[w][h], f, sum);
        acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
      }
      if (cut) {
        __stcg(reinterpret_cast<float4*>(part + h * D + d), acc);
        if (d == 0) __stcg(reinterpret_cast<float2*>(part_ml + 2 * h), make_float2(top, sum));
      } else {
        const float f = sum == 0.0f ? 0.0f : vscale / sum;
        *reinterpret_cast<uint2*>(p.y + b * p.ldy + int64_t(h0 + h) * D + d) =
            make_uint2(bf16x2_rn(acc.x * f, acc.y * f), bf16x2_rn(acc.z * f, acc.w * f));
      }
    }
    __syncthreads();  // the exchange buffer is free again; the partial is written

    if (cut) {
      // The pair's pieces are those of CTAs first .. last: the first in its second
      // slot, the others in their first.
      const unsigned int first = cta_of(tile0), last = cta_of(tile0 + it.sp.tiles - 1);
      const int pieces = static_cast<int>(last - first + 1);
      if (tid == 0) {
        __threadfence();
        s_last = atomicAdd(p.counters + first, 1u) + 1 == static_cast<unsigned int>(pieces);
        if (s_last) {
          __threadfence();
          p.counters[first] = 0;  // for the next launch
        }
      }
      __syncthreads();
      if (s_last) {
        // Each thread by itself, kPieces pieces at a time: their maxima, sums and values in one round of loads.
        const float* ml = p.partials + int64_t(2) * gridDim.x * (HEADS * D);
        for (int vec = tid; vec < heads * (D / 4); vec += kThreads) {
          const int h = vec / (D / 4), d = (vec % (D / 4)) * 4;
          float top = -INFINITY, sum = 0.0f;
          float4 acc = make_float4(0, 0, 0, 0);
          for (int i0 = 0; i0 < pieces; i0 += kPieces) {
            float4 v[kPieces];
            float2 w[kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
              v[i] = make_float4(0, 0, 0, 0);
              w[i] = make_float2(-INFINITY, 0.0f);
              if (i0 + i < pieces) {
                const int64_t sl = int64_t(2) * (first + i0 + i) + (i0 + i == 0 ? 1 : 0);
                w[i] = __ldcg(reinterpret_cast<const float2*>(ml + sl * (HEADS * 2) + 2 * h));
                v[i] = __ldcg(reinterpret_cast<const float4*>(p.partials + sl * (HEADS * D)) + vec);
              }
            }
            float now = top;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) now = fmaxf(now, w[i].x);
            const float use = now == -INFINITY ? 0.0f : now, keep = ex2(top - use);
            top = now;
            sum *= keep;
            acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
              const float f = ex2(w[i].x - use);
              sum = fmaf(w[i].y, f, sum);
              acc.x = fmaf(v[i].x, f, acc.x), acc.y = fmaf(v[i].y, f, acc.y);
              acc.z = fmaf(v[i].z, f, acc.z), acc.w = fmaf(v[i].w, f, acc.w);
            }
          }
          const float f = sum == 0.0f ? 0.0f : vscale / sum;
          *reinterpret_cast<uint2*>(p.y + b * p.ldy + int64_t(h0 + h) * D + d) =
              make_uint2(bf16x2_rn(acc.x * f, acc.y * f), bf16x2_rn(acc.z * f, acc.w * f));
        }
      }
    }

    if (!more) break;
    it = nx;
  }
  pdl_trigger();
}

int heads_per_cta(int group) { return group <= 8 ? 8 : 16; }
size_t control_bytes(int ctas) { return (static_cast<size_t>(ctas) * 4 + 255) / 256 * 256; }
size_t workspace_bytes_for(int ctas, int heads, int D) {
  return control_bytes(ctas) + static_cast<size_t>(2) * ctas * heads * (D + 2) * 4;
}

template <int D, bool E4M3, int NH>
sp24_status launch(const DecodeParams& p, const DeviceInfo& dev, int ctas, cudaStream_t s) {
  constexpr int TT = kHalf / (D * (E4M3 ? 1 : 2)) * kWarps;
  // Tile numbers are 32-bit: the host refuses what could pass them.
  const int64_t most = (int64_t(p.table_width) << p.cache.page_shift) / TT + 3;
  if (most * p.B > INT32_MAX / (int64_t(p.kv_heads) * p.head_blocks)) return SP24_ERR_UNSUPPORTED;
  const int smem = kSmem<D, E4M3, NH>;
  const cudaError_t r = launch_pdl_smem<attention_decode_kernel<D, E4M3, NH>>(dev, dim3(ctas), dim3(kThreads), smem, s, p);
  return r == cudaSuccess ? SP24_OK : SP24_ERR_CUDA;
}

}  // namespace
}  // namespace sp24

extern "C" size_t sp24_attention_decode_workspace_size(int q_heads, int heads, int head_dim) {
  using namespace sp24;
  if (q_heads < 1 || heads < 1 || q_heads % heads || q_heads / heads > 128 || (head_dim != 64 && head_dim != 128))
    return 0;
  const DeviceInfo* dev = nullptr;
  if (current_device(&dev)) return 0;
  return workspace_bytes_for(dev->sm_count * kCtasPerSm, heads_per_cta(q_heads / heads), head_dim);
}

extern "C" sp24_status sp24_attention_decode(const void* q, int64_t B, int64_t ldq, int q_heads,
                                             const sp24_kv_cache* cache, const int32_t* page_table,
                                             int64_t table_width, int64_t ld_table, const int32_t* seq_lens,
                                             float scale, int window, int sinks, void* Y, int64_t ldy,
                                             void* workspace, size_t workspace_bytes, void* stream) {
  using namespace sp24;
  DecodeParams p = {};
  if (sp24_status st = check_attention(q, B, ldq, q_heads, cache, page_table, table_width, ld_table, seq_lens, B, scale,
                                       window, sinks, Y, ldy, &p.cache))
    return st;
  const DeviceInfo* dev = nullptr;
  if (sp24_status st = current_device(&dev)) return st;
  const int ctas = dev->sm_count * kCtasPerSm, group = q_heads / cache->heads, hpc = heads_per_cta(group);
  const int D = cache->head_dim;
  if (!workspace || workspace_bytes < workspace_bytes_for(ctas, hpc, D)) return SP24_ERR_WORKSPACE;
  if (!aligned16(workspace)) return SP24_ERR_ALIGNMENT;
  if (B == 0) return SP24_OK;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.ldq = ldq;
  p.B = static_cast<int>(B);
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
  p.group = group;
  p.head_blocks = (group + hpc - 1) / hpc;
  p.counters = static_cast<unsigned int*>(workspace);
  p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + control_bytes(ctas));
  p.err = dev->err_word;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool e4m3 = cache->dtype == SP24_E4M3;
  if (D == 128) {
    if (hpc == 8) return e4m3 ? launch<128, true, 1>(p, *dev, ctas, s) : launch<128, false, 1>(p, *dev, ctas, s);
    return e4m3 ? launch<128, true, 2>(p, *dev, ctas, s) : launch<128, false, 2>(p, *dev, ctas, s);
  }
  if (hpc == 8) return e4m3 ? launch<64, true, 1>(p, *dev, ctas, s) : launch<64, false, 1>(p, *dev, ctas, s);
  return e4m3 ? launch<64, true, 2>(p, *dev, ctas, s) : launch<64, false, 2>(p, *dev, ctas, s);
}
