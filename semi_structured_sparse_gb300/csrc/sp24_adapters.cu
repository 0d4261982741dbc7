// sp24_adapters.cu -- sp24_add_adapters: to every row of a projection's output
// the product of its request's low-rank adapter,
//
//   out[t] = y[t] + scale_i B_i (A_i x[t]),  i = ids[t]
//
// Bound by memory: rows and the adapters in use are read once, and 2 r
// operations per value of x and y are few; with few rows, by a chain of
// latencies (ids; x and A; the meeting of all who have a part of A x; the results).
//
// Two forms.  Few rows: the rows of one adapter, wherever they are, to a cluster of
// CTAs, by mma.sync.  Many rows: tiles of 128 rows by tcgen05.mma, in two launches.
//
// Measured (GB300, in a graph): 1 row of 4096 values, rank 16, N 4096 4.4 us; 64 rows with an
// adapter each, N 6144 8.9 us; 200 rows of 20 adapters in no order, K 14336, rank 64,
// N 4096 16.8 us; 512 rows of 4 adapters, rank 64, K = N = 4096 12.0 us; 3000 rows of 16 adapters in runs, rank 32, N 14336 48 us (60 % of the measured
// copy rate); 8192 rows of 8 in runs, rank 64, K = N = 4096 53 to 55 us, as the runs end, of one 44 us (57 and 70 %).  Rank 128:
// 37.5 us for those 64 rows, 30 for the 200, 95 for the 3000, 84 for the 8192.
#include <cuda_bf16.h>
#include <algorithm>
#include <cmath>
#include "sp24_internal.cuh"
#include "sp24_ptx.cuh"

namespace sp24 {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMostCluster = 8;    // CTAs that share a few rows' work, at most
constexpr int kMostRank = 128;
constexpr int kNobody = -3;        // (ids are -1 and up, -2 behind the last row)
constexpr int kSlots = 1024, kBitsRow = 20;  // (words; 16 are used, 20 keep banks apart)
constexpr int kFewRows = 512;      // rows that are brought together by adapter
constexpr int kFew = 1024;         // rows up to which the form for few takes all, in blocks of kFewRows (4096 values, rank 16, 8
                                   // adapters in runs: 1024 rows 11.5 us, in tiles 17.4; 2048 rows 22 and 20)

struct AdapterParams {
  const __nv_bfloat16* y;
  const __nv_bfloat16* x;
  const __nv_bfloat16* a;
  const __nv_bfloat16* b;
  const int32_t* ids;
  const float* scales;
  __nv_bfloat16* out;
  int64_t ldy, ldx, ldo, stride_a, stride_b;
  int T, K, N, r, count;
  unsigned int* err;
};

__device__ __forceinline__ void cp_async_16(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Few rows.  An item is one adapter and up to R = 8 NT rows that have it, wherever they
// are in the batch; a cluster of 1 to 8 CTAs works on it.  Their warps cut K for
// A x, a warp's sums meet in shared memory and the CTAs' in all CTAs of the cluster
// (distributed shared memory, always added in the same order), and the warps
// cut N for B (A x).
//
// Both products are mma.sync m16n8k16 (8 rows leave tcgen05's 128 idle, and the
// bytes bound this): the rank on the 16-row side in the first, tokens in the
// second.  Along the axis that is summed over, the order is free as long as both
// operands have the same: so a lane takes 16 bytes in a row of each, as it finds
// them in memory, and no operand is rearranged.  In the second product the columns are
// numbered so that a lane's results are 8 columns in a row.
template <int MT, int NT>
struct FewCfg {
  static constexpr int R = 8 * NT, RP = 16 * MT;         // rows and rank, padded
  static constexpr int KS = MT < 2 ? 1 : MT / 2;         // 32s of the rank
  static constexpr int LOADS = 2 * MT + NT;              // 16-byte pieces per lane and 32 of K
  // (Items of 8 rows are the form for many adapters, of which an SM holds two up to rank 64: 512 rows of 100 adapters, rank
  // 64, K = N = 4096 29.5 us; with three stages and one CTA 6 us more.)
  static constexpr int STAGES = LOADS <= 5 ? 4 : NT == 1 || LOADS > 10 ? 2 : 3;
  // 32s of N whose operands are under way.  (512 rows with an adapter each, rank 16, K = N = 4096: 42 us with two, 47 with
  // one or four, 44 with three; with B sent for to L2 beside A, 49.)
  static constexpr int AHEAD = KS <= 2 ? 2 : 1;
  static constexpr int HLD = 32 * KS + 8;                // row of A x, in bf16
  static constexpr int RING = kWarps * STAGES * LOADS * 512, PART = kWarps * R * RP * 4;
  static constexpr int FIRST = RING > PART ? RING : PART;  // the ring, and then the warps' sums
  static constexpr int RECV = kMostCluster * R * RP * 4, H = 2 * R * HLD * 2;
  static constexpr int SMEM = FIRST + RECV + H;
  static constexpr int CTAS = NT == 1 && 2 * (SMEM + 2048) <= 227 * 1024 ? 2 : 1;  // per SM, that registers are to allow
};
template <int MT, int NT>
__global__ void __launch_bounds__(kThreads, FewCfg<MT, NT>::CTAS) add_adapters_few_kernel(
    const __grid_constant__ AdapterParams p, int items) {
  using C = FewCfg<MT, NT>;
  constexpr int R = C::R, RP = C::RP, KS = C::KS, ST = C::STAGES, MH = (NT + 1) / 2;  // 16-row tiles of tokens
  extern __shared__ __align__(128) uint8_t smem[];
  float* const part = reinterpret_cast<float*>(smem);                       // [kWarps][R][RP]
  float* const recv = reinterpret_cast<float*>(smem + C::FIRST);            // [CTAs][R][RP]
  uint8_t* const h_s = smem + C::FIRST + C::RECV;                           // [2][R][HLD] bf16
  __shared__ int s_count[kFewRows / 32], s_item[2], s_row[R];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t rank = cluster_rank(), ctas = cluster_nrank();
  const int gw = rank * kWarps + warp, GW = ctas * kWarps, block = blockIdx.x / ctas / items;
  const int item = blockIdx.x / ctas - block * items, t0 = block * kFewRows, T = min(kFewRows, p.T - t0);
  pdl_wait();

  // ---- this cluster's item: rows are numbered within their adapter; every R-th begins one
  constexpr int MINE = kFewRows / kThreads;
  int id[MINE], nth[MINE];
  unsigned int same[MINE];
  bool first[MINE];
#pragma unroll
  for (int i = 0; i < MINE; ++i) {
    const int x = tid + i * kThreads;
    id[i] = -2;
    if (x < T) {
      id[i] = __ldg(p.ids + t0 + x);
      if (id[i] >= p.count) {
        if (item == 0) atomicOr(p.err, DEVERR_INDEX);
        id[i] = -1;
      }
      id[i] = max(id[i], -1);
    }
  }
#pragma unroll
  for (int i = 0; i < MINE; ++i) {  // how many rows of these 32 before this one have its adapter
    same[i] = __match_any_sync(0xFFFFFFFFu, id[i]);
    nth[i] = __popc(same[i] & ((1u << lane) - 1));
  }
  // ... and of those before them.
  if (T > 32) {
    // Each adapter has a slot in a table, there its first row, and at that row the bits of all its rows.
    // (Slots depend on who comes first, the rest on the ids alone: all CTAs find the same.)
    int* const key = reinterpret_cast<int*>(smem);
    int* const head = key + kSlots;
    unsigned int* const bits = reinterpret_cast<unsigned int*>(head + kSlots);  // [rows][kBitsRow]
    static_assert(C::FIRST >= (2 * kSlots + kFewRows * kBitsRow) * 4, "the table is where the ring will be");
    const int slot_bits = T <= kSlots / 8 ? 8 : 10, slots = 1 << slot_bits;
    for (int j = tid; j < slots; j += kThreads) key[j] = kNobody, head[j] = kFewRows;
    for (int j = tid; j < T * (kBitsRow / 4); j += kThreads) reinterpret_cast<uint4*>(bits)[j] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    int slot[MINE];
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      slot[i] = 0;
      if (nth[i] || id[i] < -1) continue;  // (the first of its 32 speaks for the others)
      slot[i] = (static_cast<unsigned int>(id[i]) * 2654435769u) >> (32 - slot_bits);
      while (true) {  // at most half of the slots are taken
        const int who = atomicCAS(&key[slot[i]], kNobody, id[i]);
        if (who == kNobody || who == id[i]) break;
        slot[i] = (slot[i] + 1) & (slots - 1);
      }
      atomicMin(&head[slot[i]], tid + i * kThreads);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MINE; ++i)
      if (!nth[i] && id[i] >= -1) bits[head[slot[i]] * kBitsRow + i * kWarps + warp] = same[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      int before = 0;
      if (!nth[i] && id[i] >= -1) {
        const unsigned int* const mine = bits + head[slot[i]] * kBitsRow;
        const int upto = i * kWarps + warp;
#pragma unroll
        for (int w = 0; w < kFewRows / 32; w += 4) {
          if (w >= upto) break;
          const uint4 v = *reinterpret_cast<const uint4*>(mine + w);
          before += __popc(v.x);
          if (w + 1 < upto) before += __popc(v.y);
          if (w + 2 < upto) before += __popc(v.z);
          if (w + 3 < upto) before += __popc(v.w);
        }
      }
      nth[i] += __shfl_sync(0xFFFFFFFFu, before, __ffs(same[i]) - 1);
    }
  }
  if (tid < R) s_row[tid] = -1;
  if (tid == 0) s_item[0] = -1;
  unsigned int votes[MINE];
#pragma unroll
  for (int i = 0; i < MINE; ++i) {
    first[i] = id[i] > -2 && nth[i] % R == 0;
    votes[i] = __ballot_sync(0xFFFFFFFFu, first[i]);
    if (lane == 0) s_count[i * kWarps + warp] = __popc(votes[i]);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MINE; ++i) {
    if (!first[i]) continue;
    int before = __popc(votes[i] & ((1u << lane) - 1));
    for (int w = 0; w < i * kWarps + warp; ++w) before += s_count[w];
    if (before == item) s_item[0] = id[i], s_item[1] = nth[i];
  }
  __syncthreads();
  // (ids are -1 and up; "none" is told from an item of rows without an adapter by its rows)
  int total = 0;
#pragma unroll
  for (int w = 0; w < kFewRows / 32; ++w) total += s_count[w];
  if (item >= total) {  // the whole cluster
    pdl_trigger();
    return;
  }
  const int adapter = s_item[0], from = s_item[1];
#pragma unroll
  for (int i = 0; i < MINE; ++i)
    if (id[i] == adapter && nth[i] >= from && nth[i] < from + R) s_row[nth[i] - from] = t0 + tid + i * kThreads;
  __syncthreads();
  if (adapter < 0) {
    for (int i = gw; i < R * ((p.N + 255) / 256); i += GW) {
      const int row = s_row[i % R], n = i / R * 256 + lane * 8;
      if (row >= 0 && n < p.N)
        *reinterpret_cast<uint4*>(p.out + row * p.ldo + n) = *reinterpret_cast<const uint4*>(p.y + row * p.ldy + n);
    }
    pdl_trigger();
    return;
  }
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this CTA has begun

  // ---- A x, this warp's part of K
  const __nv_bfloat16* const a = p.a + adapter * p.stride_a;
  const int steps = (p.K + 31) / 32;
  const int k0 = static_cast<int>(int64_t(steps) * gw / GW), k1 = static_cast<int>(int64_t(steps) * (gw + 1) / GW);
  uint8_t* const ring = smem + warp * (ST * C::LOADS * 512) + lane * 16;
  const __nv_bfloat16* xr[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int row = s_row[8 * n + g];
    xr[n] = row < 0 ? nullptr : p.x + row * p.ldx;
  }
  auto issue = [&](int k) {
    if (k < k1) {
      const int at = 32 * k + 8 * t;
      const bool in = at < p.K;
      uint8_t* dst = ring + (k - k0) % ST * (C::LOADS * 512);
#pragma unroll
      for (int n = 0; n < NT; ++n) cp_async_16(dst + n * 512, xr[n] && in ? xr[n] + at : p.x, xr[n] && in);
#pragma unroll
      for (int m = 0; m < 2 * MT; ++m) {
        const bool ok = in && 8 * m + g < p.r;
        cp_async_16(dst + (NT + m) * 512, ok ? a + int64_t(8 * m + g) * p.K + at : a, ok);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) issue(k0 + i);
  const int blocks = (p.N + 31) / 32;
  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.0f;
  for (int k = k0; k < k1; ++k) {
    cp_async_wait<ST - 2>();
    const uint8_t* src = ring + (k - k0) % ST * (C::LOADS * 512);  // what this lane has copied itself
    uint4 xv[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) xv[n] = *reinterpret_cast<const uint4*>(src + n * 512);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint4 lo = *reinterpret_cast<const uint4*>(src + (NT + 2 * m) * 512);
      const uint4 hi = *reinterpret_cast<const uint4*>(src + (NT + 2 * m + 1) * 512);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma16816(acc[m][n], lo.x, hi.x, lo.y, hi.y, xv[n].x, xv[n].y);
        mma16816(acc[m][n], lo.z, hi.z, lo.w, hi.w, xv[n].z, xv[n].w);
      }
    }
    issue(k + ST - 1);
  }
  cp_async_wait<0>();

  // ---- the first columns' operands of B (A x), ahead of the wait for A x
  const int n0 = static_cast<int>(int64_t(blocks) * gw / GW), n1 = static_cast<int>(int64_t(blocks) * (gw + 1) / GW);
  const __nv_bfloat16* const b = p.b + adapter * p.stride_b;
  int row[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) row[i] = s_row[8 * i + g];
  uint4 bv[C::AHEAD][KS][4], yv[C::AHEAD][NT];
  const __nv_bfloat16* const b_lane = b + (8 * (g >> 1) + (g & 1)) * p.r + 8 * t;
  const __nv_bfloat16* y_row[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) y_row[i] = p.y + max(row[i], 0) * p.ldy + 8 * t;
  auto load = [&](int block, uint4 (&bv)[KS][4], uint4 (&yv)[NT]) {
    const __nv_bfloat16* from = b_lane + int64_t(32 * block) * p.r;
    const int left = block < n1 ? p.N - 32 * block : 0;  // columns from here on
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        bv[s][j] = make_uint4(0, 0, 0, 0);
        if (8 * (g >> 1) + 2 * j + (g & 1) < left && 32 * s + 8 * t < p.r)
          bv[s][j] = *reinterpret_cast<const uint4*>(from + 2 * j * p.r + 32 * s);
      }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      yv[i] = make_uint4(0, 0, 0, 0);
      if (row[i] >= 0 && 8 * t < left) yv[i] = *reinterpret_cast<const uint4*>(y_row[i] + 32 * block);
    }
  };
#pragma unroll
  for (int a = 0; a < C::AHEAD; ++a) load(n0 + a, bv[a], yv[a]);

  // ---- the warps' sums, then the CTAs'
  __syncthreads();  // the ring has been read
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        part[(warp * R + 8 * n + 2 * t + (i & 1)) * RP + 16 * m + g + 8 * (i >> 1)] = acc[m][n][i];
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // all CTAs have begun
  for (int e = tid; e < R * RP; e += kThreads) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += part[w * (R * RP) + e];
#pragma unroll
    for (uint32_t c = 0; c < kMostCluster; ++c)
      if (c < ctas) st_cluster(cluster_addr(recv + rank * (R * RP) + e, c), sum);
  }
  cluster_sync();
  const float scale = p.scales ? p.scales[adapter] : 1.0f;
  __nv_bfloat16* const h_hi = reinterpret_cast<__nv_bfloat16*>(h_s);
  __nv_bfloat16* const h_lo = h_hi + R * C::HLD;
  // A x in two bf16 parts, which hold it to 2^-16: one alone would move the product by 2^-8 of it.
  for (int e = tid; e < R * 32 * KS; e += kThreads) {
    const int i = e / (32 * KS), j = e % (32 * KS);
    float sum = 0.0f;
    if (j < p.r) {  // (behind the rank, an infinite x has made zeros into what is not a number)
#pragma unroll
      for (int c = 0; c < kMostCluster; ++c)
        if (c < static_cast<int>(ctas)) sum += recv[c * (R * RP) + i * RP + j];
      sum *= scale;
    }
    const __nv_bfloat16 hi = __float2bfloat16(sum);
    const float rest = sum - __bfloat162float(hi);
    h_hi[i * C::HLD + j] = hi;
    h_lo[i * C::HLD + j] = __float2bfloat16(isfinite(rest) ? rest : 0.0f);
  }
  __syncthreads();

  // ---- B (A x), this warp's columns, 32 at a time
  for (int block0 = n0; block0 < n1; block0 += C::AHEAD) {
#pragma unroll
    for (int a = 0; a < C::AHEAD; ++a) {
      const int block = block0 + a;
      if (block >= n1) break;
      float o[MH][4][4];
#pragma unroll
      for (int m = 0; m < MH; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[m][j][0] = o[m][j][1] = o[m][j][2] = o[m][j][3] = 0.0f;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
#pragma unroll
        for (int m = 0; m < MH; ++m) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const __nv_bfloat16* h = (x ? h_lo : h_hi) + 32 * s + 8 * t;
            const uint4 lo = *reinterpret_cast<const uint4*>(h + (16 * m + g) * C::HLD);
            uint4 hi = make_uint4(0, 0, 0, 0);
            if (2 * m + 1 < NT) hi = *reinterpret_cast<const uint4*>(h + (16 * m + 8 + g) * C::HLD);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              mma16816(o[m][j], lo.x, hi.x, lo.y, hi.y, bv[a][s][j].x, bv[a][s][j].y);
              mma16816(o[m][j], lo.z, hi.z, lo.w, hi.w, bv[a][s][j].z, bv[a][s][j].w);
            }
          }
        }
      }
      uint4 y[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) y[i] = yv[a][i];
      load(block + C::AHEAD, bv[a], yv[a]);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if (row[i] < 0 || 32 * block + 8 * t >= p.N) continue;
        const uint32_t w[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
        uint32_t r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          r[j] = bf16x2_rn(__uint_as_float(w[j] << 16) + o[i / 2][j][2 * (i & 1)],
                           __uint_as_float(w[j] & 0xFFFF0000u) + o[i / 2][j][2 * (i & 1) + 1]);
        *reinterpret_cast<uint4*>(p.out + row[i] * p.ldo + 32 * block + 8 * t) = make_uint4(r[0], r[1], r[2], r[3]);
      }
    }
  }
  pdl_trigger();
}

// Many rows, in two launches of tcgen05.mma with operands by TMA.  Rows come in tiles of
// 128 in a row.  The first launch forms D1 = A x (128 rows x rank), the second D2 =
// B (A x), 64 columns at a time, and adds y.  A unit of the first is 64 of a tile's
// K, of the second 64 of its N; each launch deals all units out to one CTA per SM in equal
// contiguous ranges.  A tile whose K is cut between CTAs has a piece of fp32 sums in the
// workspace from each, which the second launch adds up in order and takes apart
// into two bf16 operands.  It needs nothing else of the first launch, so that its
// CTAs begin as SMs get done with that one, and their first copies run meanwhile.
//
// A tile's rows may have several adapters: each is a product of its own, of which a row
// takes that of its own adapter (what another adapter makes of it reaches nothing).
// A result is formed in y's tile in shared memory, and stored from there.
constexpr int kTile = 128;          // rows
constexpr int kCols = 64;           // of K, or N, per unit
constexpr int kRowTile = kTile * kCols * 2;
// Warps that issue MMAs, every other unit each: a commit holds its thread back until they are done.  Each has stages of
// its own in every ring that it reads (as the two groups of warps that take the results have).  A wait tells a phase
// from the one before it only, so whoever waits on a stage has to see all its phases; with stages that change hands, a
// warp that is ahead would take a use that it has not waited for, and is not there yet, for its own.
constexpr int kIssue = 2;
constexpr int kLeastK = 8, kLeastN = 4;  // units per CTA

struct Deal {
  unsigned int ctas, per, extra;  // the first `extra` CTAs take a unit more
  __host__ __device__ static Deal of(unsigned int units, unsigned int sms, unsigned int least) {
    Deal d;
    d.ctas = units / least < 1 ? 1 : units / least < sms ? units / least : sms;
    d.per = units / d.ctas, d.extra = units % d.ctas;
    return d;
  }
  __device__ unsigned int begin(unsigned int cta) const { return cta * per + min(cta, extra); }
  __device__ unsigned int cta_of(unsigned int u) const {
    return u < extra * (per + 1) ? u / (per + 1) : extra + (u - extra * (per + 1)) / per;
  }
};

struct ManyParams {
  AdapterParams p;
  int32_t* order;     // the rows, sorted by adapter in windows of kWindow (null: as they are)
  int32_t* sorted;    // of each window: whether it has been (otherwise its rows stay as they are)
  int kbs, nbs, rp;   // units of a tile, and the rank padded to the MMA's multiple of 16
  Deal k, n;
  float* part;        // [pieces][kTile][rp]; the piece of a tile that CTA c of the first launch forms is tile + c
};

// Rows whose adapters are in no order would make every tile a tile of many adapters, so a launch before the two
// sorts them by adapter in windows, unless an adapter's rows mostly stand in runs.  A tile is then 128 rows in that
// order, fetched and stored four rows per copy where they are apart.  A radix sort that counts a digit's rows by
// warp, each warp's in order, keeps equal ones as they were and needs no atomics, so the results are the same
// every time.  (4096 rows of 4096 values, rank 16, 64 adapters, in no order: 74 us, 555 without the sort, 45 if each
// adapter's rows stand together.  Fetching all tiles row by row: 8192 rows with one adapter 116 us instead of 45, all
// copies issued by one thread.)
constexpr int kWindow = 8192, kSortThreads = 1024, kDigits = 256, kSortWarps = kSortThreads / 32;
constexpr int kEach = kWindow / kSortThreads, kHistRow = kSortWarps + 1;
constexpr int kLongRuns = 2;  // changes of adapter per tile up to which rows stay as they are
struct SortSmem {
  unsigned int key[kWindow];
  unsigned int count[kDigits * kHistRow];  // of a digit: of each warp's rows, and then where they go
  unsigned short at[kWindow];
  unsigned int warp_sum[kSortWarps], changes;
};
__global__ void __launch_bounds__(kSortThreads) adapters_sort_kernel(const __grid_constant__ ManyParams q, int bits) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SortSmem& sm = *reinterpret_cast<SortSmem*>(smem_raw);
  const AdapterParams& p = q.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int x0 = blockIdx.x * kWindow, n = min(kWindow, p.T - x0);
  if (tid == 0) sm.changes = 0;
  pdl_wait();
  pdl_trigger();
  const int mine = warp * (32 * kEach) + lane;  // and every 32nd behind it
  unsigned int key[kEach], at[kEach], rank[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int x = mine + 32 * i;
    at[i] = x;
    key[i] = 0xFFFFFFFFu;  // behind the last row: stays there
    if (x < n) {
      const int id = __ldg(p.ids + x0 + x);
      key[i] = id < 0 || id >= p.count ? 0 : id + 1;
    }
  }
  __syncthreads();
  int changes = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const unsigned int before = __shfl_up_sync(0xFFFFFFFFu, key[i], 1);
    changes += __popc(__ballot_sync(0xFFFFFFFFu, lane > 0 && mine + 32 * i < n && key[i] != before));
  }
  if (lane == 0 && changes) atomicAdd(&sm.changes, changes);
  __syncthreads();
  const bool sort = sm.changes > kLongRuns * ((n + kTile - 1) / kTile);
  if (tid == 0) q.sorted[blockIdx.x] = sort;
  if (!sort) return;
  for (int shift = 0; shift < bits; shift += 8) {
    for (int i = tid; i < kDigits * kHistRow; i += kSortThreads) sm.count[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const unsigned int digit = key[i] >> shift & (kDigits - 1);
      const unsigned int same = __match_any_sync(0xFFFFFFFFu, digit);
      const unsigned int before = __popc(same & ((1u << lane) - 1));
      unsigned int* const c = &sm.count[digit * kHistRow + warp];
      const unsigned int base = *c;
      rank[i] = base + before;
      __syncwarp();
      if (before == 0) *c = base + __popc(same);
      __syncwarp();
    }
    __syncthreads();
    {  // sums of what comes before, digits first, warps in order
      constexpr int PER = kDigits * kSortWarps / kSortThreads;
      static_assert(kSortWarps % PER == 0, "a thread's counts are of one digit");
      unsigned int* const c = &sm.count[tid * PER / kSortWarps * kHistRow + tid * PER % kSortWarps];
      unsigned int v[PER], sum = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = sum, sum += c[i];
      unsigned int upto = sum;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const unsigned int x = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (lane >= d) upto += x;
      }
      if (lane == 31) sm.warp_sum[warp] = upto;
      __syncthreads();
      unsigned int base = upto - sum;
      for (int w = 0; w < warp; ++w) base += sm.warp_sum[w];
#pragma unroll
      for (int i = 0; i < PER; ++i) c[i] = base + v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const unsigned int to = sm.count[(key[i] >> shift & (kDigits - 1)) * kHistRow + warp] + rank[i];
      sm.key[to] = key[i];
      sm.at[to] = static_cast<unsigned short>(at[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) key[i] = sm.key[mine + 32 * i], at[i] = sm.at[mine + 32 * i];
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (mine + 32 * i < n) q.order[x0 + mine + 32 * i] = x0 + at[i];
}

// What a CTA does in one go: units of one tile.
struct Segment {
  int tile, first, count;     // count 0: nothing more
  int adapters;
  int apart;                  // whether its rows are not in a row
  int adapter[kTile];         // the tile's adapters
  __align__(16) int row[kTile];
  int which[kTile];           // of each row: which of them, or -1
  float scale[kTile];         // of each row
};
// The segment that begins with unit u, by one warp.
__device__ __forceinline__ void find_segment(const ManyParams& q, unsigned int u, unsigned int u_end, int per_tile,
                                             bool report, bool scales, Segment* out) {
  const AdapterParams& p = q.p;
  const int lane = threadIdx.x & 31;
  if (u >= u_end) {
    if (lane == 0) out->count = 0;
    __syncwarp();
    return;
  }
  const int tile = u / per_tile, first = u - tile * per_tile;
  const int sorted = q.order ? __ldcg(q.sorted + tile / (kWindow / kTile)) : 0;
  int id[kTile / 32], which[kTile / 32];
  bool apart = false;
  int x[kTile / 32];
#pragma unroll
  for (int i = 0; i < kTile / 32; ++i) {
    x[i] = min(tile * kTile + 32 * i + lane, p.T - 1);  // (behind the last row: that row again, with the same result)
    id[i] = __ldg(p.ids + x[i]);                        // (on its way together with whether rows have been sorted)
    which[i] = -1;
  }
  if (sorted) {
#pragma unroll
    for (int i = 0; i < kTile / 32; ++i) {
      const int from = __ldcg(q.order + x[i]);
      apart |= from != x[i];
      x[i] = from;
      id[i] = __ldg(p.ids + from);
    }
  }
#pragma unroll
  for (int i = 0; i < kTile / 32; ++i) out->row[32 * i + lane] = x[i];
  apart = __any_sync(0xFFFFFFFFu, apart);
#pragma unroll
  for (int i = 0; i < kTile / 32; ++i)
    if (id[i] >= p.count) {
      if (report) atomicOr(p.err, DEVERR_INDEX);
      id[i] = -1;
    }
  int n = 0;
#pragma unroll
  for (int i = 0; i < kTile / 32; ++i) {
    while (true) {  // the first row whose adapter is not on the list yet
      const unsigned int left = __ballot_sync(0xFFFFFFFFu, id[i] >= 0 && which[i] < 0);
      if (!left) break;
      const int now = __shfl_sync(0xFFFFFFFFu, id[i], __ffs(left) - 1);
#pragma unroll
      for (int j = 0; j < kTile / 32; ++j)
        if (id[j] == now) which[j] = n;
      if (lane == 0) out->adapter[n] = now;
      ++n;
    }
  }
#pragma unroll
  for (int i = 0; i < kTile / 32; ++i) {
    out->which[32 * i + lane] = which[i];
    if (scales) out->scale[32 * i + lane] = p.scales && id[i] >= 0 ? __ldg(p.scales + id[i]) : 1.0f;
  }
  if (lane == 0) {
    out->tile = tile;
    out->first = first;
    out->apart = apart;
    out->count = min(per_tile - first, static_cast<int>(u_end - u));
    out->adapters = n;
  }
  __syncwarp();
}

__device__ __forceinline__ bool all_of(bool x) { return __all_sync(0xFFFFFFFFu, x); }
// A tile's rows, 64 columns of them, by a warp: four rows per lane where they are apart (by one lane, 4096 rows of 64
// adapters in no order took 89 us, 74 so).  `rows` is the same matrix in boxes of one row.
__device__ __forceinline__ void load_rows(uint8_t* dst, const CUtensorMap* tiles, const CUtensorMap* rows, uint64_t* bar,
                                          int col, const Segment& s) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) mbar_arrive_expect_tx(bar, kRowTile);
  __syncwarp();
  if (s.apart) {
    tma_gather4(dst + lane * (4 * kCols * 2), rows, bar, col, *reinterpret_cast<const int4*>(s.row + 4 * lane));
  } else if (lane == 0) {
    tma_load_2d(dst, tiles, bar, col, s.tile * kTile);
  }
}
__device__ __forceinline__ void store_rows(const uint8_t* src, const CUtensorMap* tiles, const CUtensorMap* rows, int col,
                                           const Segment& s) {
  const int lane = threadIdx.x & 31;
  if (s.apart) {
    tma_scatter4(rows, src + lane * (4 * kCols * 2), col, *reinterpret_cast<const int4*>(s.row + 4 * lane));
  } else if (lane == 0) {
    tma_store_2d(tiles, src, col, s.tile * kTile);
  }
}

// ------------------------------------------------------------------ A x
template <int KB>  // 64s of the rank
struct DownCfg {
  static constexpr int ROWS = 6, ADS = KB == 1 ? 14 : 6;  // stages
  static constexpr int R = ROWS / kIssue, A = ADS / kIssue;              // of each issuing warp
  static constexpr int AD_TILE = KB * 64 * 128;
  static constexpr int D1 = 64 * KB;                  // columns of an adapter's sums
  static constexpr int PASS = 512 / (kIssue * D1);    // adapters per pass over K
  static constexpr int BARS = 2 * ROWS + 2 * ADS + 2 + 4 + kIssue;
  static constexpr int SMEM = 1024 + ROWS * kRowTile + ADS * AD_TILE + BARS * 8;
  static_assert(SMEM + 2 * sizeof(Segment) + 64 <= 227 * 1024, "shared memory");
};
constexpr int kDownThreads = (4 + 2 + kIssue) * 32;  // sums, segments, copies, MMAs

template <int KB>
__global__ void __launch_bounds__(kDownThreads, 1)
    adapters_down_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap xrows,
                         const __grid_constant__ CUtensorMap amap,
                         const __grid_constant__ ManyParams q) {
  using C = DownCfg<KB>;
  constexpr int ROWS = C::ROWS, ADS = C::ADS;
  const AdapterParams& p = q.p;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ Segment s_seg[2];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const row_s = smem;
  uint8_t* const ad_s = row_s + ROWS * kRowTile;
  uint64_t* const row_full = reinterpret_cast<uint64_t*>(ad_s + ADS * C::AD_TILE);  // [ROWS]
  uint64_t* const row_empty = row_full + ROWS;
  uint64_t* const ad_full = row_empty + ROWS;     // [ADS]
  uint64_t* const ad_empty = ad_full + ADS;
  uint64_t* const d1_full = ad_empty + ADS;
  uint64_t* const d1_empty = d1_full + 1;
  uint64_t* const seg_full = d1_empty + 1;        // [2]
  uint64_t* const seg_empty = seg_full + 2;       // [2]
  uint64_t* const drain = seg_empty + 2;          // [kIssue]

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  if (warp == 4) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  } else if (warp == 5 && lane == 0) {
    for (int i = 0; i < ROWS; ++i) mbar_init(&row_full[i], 1), mbar_init(&row_empty[i], 1);
    for (int i = 0; i < ADS; ++i) mbar_init(&ad_full[i], 1), mbar_init(&ad_empty[i], 1);
    mbar_init(d1_full, kIssue);
    mbar_init(d1_empty, 4);
    for (int i = 0; i < 2; ++i) mbar_init(&seg_full[i], 1), mbar_init(&seg_empty[i], 5 + kIssue);
    for (int i = 0; i < kIssue; ++i) mbar_init(&drain[i], 1);
    fence_mbar_init();
    tma_prefetch_desc(&xmap), tma_prefetch_desc(&amap);
  }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = s_tmem;
  bool ok = true;
  auto wait_segment = [&](int i) { return mbar_wait(&seg_full[i & 1], (i >> 1) & 1); };
  auto done_with = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&seg_empty[i & 1]);
  };

  if (warp < 4) {
    // ------------------------------------------------------------------ sums
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    int passes = 0;  // so far
    for (int i = 0; ok; ++i) {
      ok = wait_segment(i);
      const Segment& s = s_seg[i & 1];
      if (!ok || s.count == 0) break;
      const int which = s.which[tid];
      float* const to = q.part + (int64_t(s.tile + blockIdx.x) * kTile + tid) * q.rp;
      for (int w0 = 0; w0 < s.adapters && ok; w0 += C::PASS, ++passes) {
        ok = mbar_wait(d1_full, passes & 1);
        if (!ok) break;
        tc_fence_after();
        for (int w = w0; w < min(s.adapters, w0 + C::PASS); ++w) {
          if (!__any_sync(0xFFFFFFFFu, which == w)) continue;
          for (int c = 0; c < q.rp; c += 8) {
            uint32_t u[2][8];
            float v[8];
            tmem_ld8(tmem + lanes + (w - w0) * kIssue * C::D1 + c, u[0]);
            if (s.count > 1) tmem_ld8(tmem + lanes + ((w - w0) * kIssue + 1) * C::D1 + c, u[1]);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 8; ++e)
              v[e] = s.count > 1 ? __uint_as_float(u[0][e]) + __uint_as_float(u[1][e]) : __uint_as_float(u[0][e]);
            if (which == w) {
              __stcg(reinterpret_cast<float4*>(to + c), make_float4(v[0], v[1], v[2], v[3]));
              __stcg(reinterpret_cast<float4*>(to + c + 4), make_float4(v[4], v[5], v[6], v[7]));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(d1_empty);
      }
      done_with(i);
    }
    if (!ok && lane == 0) atomicOr(p.err, DEVERR_TIMEOUT_EPILOGUE);
  } else if (warp == 4) {
    // -------------------------------------------------------------- segments
    unsigned int u = q.k.begin(blockIdx.x);
    const unsigned int end = q.k.begin(blockIdx.x + 1);
    for (int i = 0; ok; ++i) {
      if (i >= 2) ok = mbar_wait(&seg_empty[i & 1], ((i >> 1) - 1) & 1);
      if (!ok) break;
      find_segment(q, u, end, q.kbs, u % q.kbs == 0, false, &s_seg[i & 1]);
      const int count = s_seg[i & 1].count;
      if (lane == 0) mbar_arrive(&seg_full[i & 1]);
      __syncwarp();
      if (count == 0) break;
      u += count;
    }
    if (!ok && lane == 0) atomicOr(p.err, DEVERR_TIMEOUT_PRODUCER);
  } else if (warp == 5) {
    // ---------------------------------------------------------------- copies
    int rows[kIssue] = {}, ads[kIssue] = {};  // so far, of each issuing warp's
    for (int i = 0; ok; ++i) {
      ok = all_of(wait_segment(i));
      const Segment& s = s_seg[i & 1];
      if (!ok || s.count == 0) break;
      auto load = [&](int w0, int k, int x, int& row, int& ad) {
        const int col = (s.first + k) * kCols, at = x * C::R + row % C::R;
#ifdef SP24_FAULT_WITHHOLD_FIRST_STAGE
        if (x == 0 && row == 0) {  // the fault-test build: each CTA's first tile never comes
          ++row;
          return;
        }
#endif
        if (row >= C::R) ok = all_of(mbar_wait(&row_empty[at], (row / C::R - 1) & 1));
        if (!ok) return;
        load_rows(row_s + at * kRowTile, &xmap, &xrows, &row_full[at], col, s);
        ++row;
        for (int w = w0; w < min(s.adapters, w0 + C::PASS); ++w, ++ad) {
          const int to = x * C::A + ad % C::A;
          if (ad >= C::A) ok = all_of(mbar_wait(&ad_empty[to], (ad / C::A - 1) & 1));
          if (!ok) return;
          if (lane == 0) {
            mbar_arrive_expect_tx(&ad_full[to], q.rp * 128);
            tma_load_3d(ad_s + to * C::AD_TILE, &amap, &ad_full[to], col, 0, s.adapter[w]);
          }
        }
      };
      for (int w0 = 0; w0 < s.adapters && ok; w0 += C::PASS)
        for (int k = 0; k < s.count && ok; k += kIssue) {
#pragma unroll
          for (int x = 0; x < kIssue; ++x)
            if (k + x < s.count && ok) load(w0, k + x, x, rows[x], ads[x]);
        }
      done_with(i);
    }
    if (lane == 0) {
      if (!ok) atomicOr(p.err, DEVERR_TIMEOUT_PRODUCER);
      // Copies in flight have to land before this CTA's shared memory goes.
#pragma unroll
      for (int x = 0; x < kIssue; ++x) {
        for (int i = max(0, rows[x] - C::R); i < rows[x]; ++i) mbar_wait(&row_full[x * C::R + i % C::R], (i / C::R) & 1);
        for (int i = max(0, ads[x] - C::A); i < ads[x]; ++i) mbar_wait(&ad_full[x * C::A + i % C::A], (i / C::A) & 1);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------- MMA
    const int x = warp - 6;  // every other unit is this warp's
    const uint32_t id = idesc_bf16(kTile, q.rp);
    const uint64_t row_d = smem_desc(smem_u32(row_s), 16, 1024, SWZ_128B);
    const uint64_t ad_d = smem_desc(smem_u32(ad_s), 16, 1024, SWZ_128B);
    int row = 0, ad = 0, passes = 0;  // so far, of this warp's
    for (int i = 0; ok; ++i) {
      ok = wait_segment(i);
      const Segment& s = s_seg[i & 1];
      if (!ok || s.count == 0) break;
      const int count = s.count, adapters = s.adapters;
      if (lane == 0) {
        for (int w0 = 0; w0 < adapters && ok; w0 += C::PASS, ++passes) {
          const int some = min(adapters - w0, C::PASS);
          if (passes > 0) ok = mbar_wait(d1_empty, (passes - 1) & 1);
          tc_fence_after();
          for (int k = x; k < count && ok; k += kIssue, ++row) {
            const int at = x * C::R + row % C::R;
            ok = mbar_wait(&row_full[at], (row / C::R) & 1);
            for (int w = 0; w < some && ok; ++w, ++ad) {
              const int from = x * C::A + ad % C::A;
              ok = mbar_wait(&ad_full[from], (ad / C::A) & 1);
              if (!ok) break;
              tc_fence_after();
              const uint64_t a = row_d + at * (kRowTile >> 4), b = ad_d + from * (C::AD_TILE >> 4);
#pragma unroll
              for (int e = 0; e < kCols / 16; ++e)
                mma_bf16(tmem + (w * kIssue + x) * C::D1, a + 2 * e, b + 2 * e, id, k >= kIssue || e > 0);
              mma_commit(&ad_empty[from]);
              if (w + 1 == some) mma_commit(&row_empty[at]);
            }
          }
          if (ok) mma_commit(d1_full);
        }
      }
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      done_with(i);
    }
    if (lane == 0) {
      if (!ok) atomicOr(p.err, DEVERR_TIMEOUT_MMA);
      mma_commit(&drain[x]);  // every MMA issued must finish before tensor memory is freed
      mbar_wait(&drain[x], 0);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- y + B (A x)
template <int KB>
struct UpCfg {
  static constexpr int ROWS = KB == 1 ? 6 : 4, ADS = KB == 1 ? 6 : 4, HS = KB == 1 ? 2 : 1;  // stages
  static constexpr int AD_TILE = KB * 64 * 128;
  static constexpr int H = 2 * KB * kRowTile;  // A x of a tile, in two parts
  static constexpr int D2S = 512 / kCols;
  static constexpr int A = ADS / kIssue, D2 = D2S / kIssue;  // of each issuing warp, and group of those for results
  static_assert(ROWS % kIssue == 0, "a row tile's stage is always the same warp's");
  static constexpr int BARS = 3 * ROWS + 2 * ADS + 2 * HS + 2 * D2S + 4 + kIssue;
  static constexpr int SMEM = 1024 + ROWS * kRowTile + ADS * AD_TILE + HS * H + BARS * 8;
  static_assert(SMEM + 2 * sizeof(Segment) + 64 <= 227 * 1024, "shared memory");
};
constexpr int kGroups = kIssue, kSumWarps = 4 * kGroups;  // groups of warps that take every other unit's results
constexpr int kHWarps = 8;
constexpr int kUpThreads = (kSumWarps + kHWarps + 3 + kIssue) * 32;  // ..., segments, copies, stores, MMAs

template <int KB>
__global__ void __launch_bounds__(kUpThreads, 1)
    adapters_up_kernel(const __grid_constant__ CUtensorMap bmap, const __grid_constant__ CUtensorMap ymap,
                       const __grid_constant__ CUtensorMap yrows, const __grid_constant__ CUtensorMap omap,
                       const __grid_constant__ CUtensorMap orows, const __grid_constant__ ManyParams q) {
  using C = UpCfg<KB>;
  constexpr int ROWS = C::ROWS, ADS = C::ADS, HS = C::HS, D2S = C::D2S;
  constexpr int H0 = kSumWarps, SEG = H0 + kHWarps, COPY = SEG + 1, STORE = COPY + 1, ISSUE = STORE + 1;  // warps
  const AdapterParams& p = q.p;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ Segment s_seg[2];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const row_s = smem;
  uint8_t* const ad_s = row_s + ROWS * kRowTile;
  uint8_t* const h_s = ad_s + ADS * C::AD_TILE;
  uint64_t* const row_full = reinterpret_cast<uint64_t*>(h_s + HS * C::H);  // [ROWS]
  uint64_t* const row_empty = row_full + ROWS;
  uint64_t* const out_full = row_empty + ROWS;    // [ROWS] the tile holds results
  uint64_t* const ad_full = out_full + ROWS;      // [ADS]
  uint64_t* const ad_empty = ad_full + ADS;
  uint64_t* const h_full = ad_empty + ADS;        // [HS]
  uint64_t* const h_empty = h_full + HS;
  uint64_t* const d2_full = h_empty + HS;         // [D2S]
  uint64_t* const d2_empty = d2_full + D2S;
  uint64_t* const seg_full = d2_empty + D2S;      // [2]
  uint64_t* const seg_empty = seg_full + 2;       // [2]
  uint64_t* const drain = seg_empty + 2;          // [kIssue]

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  if (warp == SEG) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  } else if (warp == COPY && lane == 0) {
    for (int i = 0; i < ROWS; ++i) {
      mbar_init(&row_full[i], 1);
      mbar_init(&row_empty[i], 1);
      mbar_init(&out_full[i], 4);
    }
    for (int i = 0; i < ADS; ++i) mbar_init(&ad_full[i], 1), mbar_init(&ad_empty[i], 1);
    for (int i = 0; i < HS; ++i) mbar_init(&h_full[i], kHWarps), mbar_init(&h_empty[i], kIssue);
    for (int i = 0; i < D2S; ++i) mbar_init(&d2_full[i], 1), mbar_init(&d2_empty[i], 4);
    for (int i = 0; i < 2; ++i) mbar_init(&seg_full[i], 1), mbar_init(&seg_empty[i], kSumWarps + kHWarps + 2 + kIssue);
    for (int i = 0; i < kIssue; ++i) mbar_init(&drain[i], 1);
    fence_mbar_init();
    tma_prefetch_desc(&bmap), tma_prefetch_desc(&ymap), tma_prefetch_desc(&omap);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // (The launch before has waited for those that write what this one reads ahead of its own wait: all but the sums.)
  const uint32_t tmem = s_tmem;
  bool ok = true;
  auto wait_segment = [&](int i) { return mbar_wait(&seg_full[i & 1], (i >> 1) & 1); };
  auto done_with = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&seg_empty[i & 1]);
  };

  if (warp < kSumWarps) {
    // --------------------------------------------------------------- results
    const int r = tid & (kTile - 1), group = tid / kTile;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int unit = 0, row0 = 0;  // products of this group so far, and units of all before this segment
    for (int i = 0; ok; ++i) {
      ok = wait_segment(i);
      const Segment& s = s_seg[i & 1];
      if (!ok || s.count == 0) break;
      const int count = s.count, adapters = s.adapters, which = s.which[r];
      done_with(i);
      for (int n = (row0 + group) % kGroups; n < count && ok; n += kGroups) {
        const int row = row0 + n, stage = row % ROWS;
        ok = mbar_wait(&row_full[stage], (row / ROWS) & 1);
        if (!ok) break;
        uint8_t* const y = row_s + stage * kRowTile + r * 128;
        for (int w = 0; w < adapters; ++w, ++unit) {
          const int at = group * C::D2 + unit % C::D2;
          ok = mbar_wait(&d2_full[at], (unit / C::D2) & 1);
          if (!ok) break;
          if (r == 0) mbar_arrive(&ad_empty[group * C::A + unit % C::A]);  // the product has been formed
          tc_fence_after();
          if (__any_sync(0xFFFFFFFFu, which == w)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t u[2][16];
              uint4 v[4];
              tmem_ld16(tmem + lanes + at * kCols + 32 * h, u[0]);
              tmem_ld16(tmem + lanes + at * kCols + 32 * h + 16, u[1]);
#pragma unroll
              for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const uint4*>(y + (((h * 4 + k) ^ (r & 7)) << 4));
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t* a = &u[k / 2][8 * (k & 1)];
                auto add = [&](uint32_t two, int e) {
                  return bf16x2_rn(__uint_as_float(two << 16) + __uint_as_float(a[2 * e]),
                                   __uint_as_float(two & 0xFFFF0000u) + __uint_as_float(a[2 * e + 1]));
                };
                v[k] = make_uint4(add(v[k].x, 0), add(v[k].y, 1), add(v[k].z, 2), add(v[k].w, 3));
              }
              if (which == w) {
#pragma unroll
                for (int k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(y + (((h * 4 + k) ^ (r & 7)) << 4)) = v[k];
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&d2_empty[at]);
        }
        if (!ok) break;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&out_full[stage]);
      }
      row0 += count;
    }
    if (!ok && lane == 0) atomicOr(p.err, DEVERR_TIMEOUT_EPILOGUE);
  } else if (warp < SEG) {
    // ------------------------------------------------- A x as two bf16 operands
    pdl_wait();
    const int me = tid - H0 * 32, pieces8 = q.rp / 8;
    int n = 0;  // tiles with adapters so far
    for (int i = 0; ok; ++i) {
      ok = wait_segment(i);
      const Segment& s = s_seg[i & 1];
      if (!ok || s.count == 0) break;
      if (s.adapters > 0) {
        if (n >= HS) ok = mbar_wait(&h_empty[n % HS], (n / HS - 1) & 1);
        if (!ok) break;
        const unsigned int u0 = static_cast<unsigned int>(s.tile) * q.kbs;
        const int c0 = q.k.cta_of(u0), c1 = q.k.cta_of(u0 + q.kbs - 1);
        const float* from = q.part + int64_t(s.tile + c0) * kTile * q.rp;
        uint8_t* const h = h_s + n % HS * C::H;
        // Two tasks of 8 values at a time, and four pieces of each: their loads are under way together.  (A row without
        // an adapter has whatever is there: it reaches no other row, and is not used.)
        constexpr int STEP = kHWarps * 32;
        for (int e0 = me; e0 < kTile * pieces8; e0 += 2 * STEP) {
          float sum[2][8];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < 8; ++k) sum[j][k] = 0.0f;
          for (int k0 = c0; k0 <= c1; k0 += 4) {
            float4 v[2][4][2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                v[j][k][0] = v[j][k][1] = make_float4(0, 0, 0, 0);
                if (e0 + j * STEP < kTile * pieces8 && k0 + k <= c1) {  // (8 values: a task's place is its number's)
                  const float4* f = reinterpret_cast<const float4*>(from + int64_t(k0 + k - c0) * kTile * q.rp) + 2 * (e0 + j * STEP);
                  v[j][k][0] = __ldcg(f), v[j][k][1] = __ldcg(f + 1);
                }
              }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                sum[j][0] += v[j][k][0].x, sum[j][1] += v[j][k][0].y, sum[j][2] += v[j][k][0].z, sum[j][3] += v[j][k][0].w;
                sum[j][4] += v[j][k][1].x, sum[j][5] += v[j][k][1].y, sum[j][6] += v[j][k][1].z, sum[j][7] += v[j][k][1].w;
              }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int e = e0 + j * STEP, x = e / pieces8, c = e - x * pieces8;
            if (x >= kTile) break;
            const float scale = s.scale[x];
            if (8 * c >= p.r) {  // (behind the rank, an infinite x has made zeros into what is not a number)
#pragma unroll
              for (int k = 0; k < 8; ++k) sum[j][k] = 0.0f;
            }
            uint32_t big[4], rest[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float a = sum[j][2 * k] * scale, b = sum[j][2 * k + 1] * scale;
              big[k] = bf16x2_rn(a, b);
              const float ra = a - __uint_as_float(big[k] << 16), rb = b - __uint_as_float(big[k] & 0xFFFF0000u);
              rest[k] = bf16x2_rn(isfinite(ra) ? ra : 0.0f, isfinite(rb) ? rb : 0.0f);
            }
            uint8_t* to = h + (c / 8) * kRowTile + x * 128 + (((c & 7) ^ (x & 7)) << 4);
            *reinterpret_cast<uint4*>(to) = make_uint4(big[0], big[1], big[2], big[3]);
            *reinterpret_cast<uint4*>(to + KB * kRowTile) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&h_full[n % HS]);
        ++n;
      }
      done_with(i);
    }
    if (!ok && lane == 0) atomicOr(p.err, DEVERR_TIMEOUT_EPILOGUE);
  } else if (warp == SEG) {
    // -------------------------------------------------------------- segments
    unsigned int u = q.n.begin(blockIdx.x);
    const unsigned int end = q.n.begin(blockIdx.x + 1);
    for (int i = 0; ok; ++i) {
      if (i >= 2) ok = mbar_wait(&seg_empty[i & 1], ((i >> 1) - 1) & 1);
      if (!ok) break;
      find_segment(q, u, end, q.nbs, false, true, &s_seg[i & 1]);
      const int count = s_seg[i & 1].count;
      if (lane == 0) mbar_arrive(&seg_full[i & 1]);
      __syncwarp();
      if (count == 0) break;
      u += count;
    }
    if (!ok && lane == 0) atomicOr(p.err, DEVERR_TIMEOUT_PRODUCER);
  } else if (warp == COPY) {
    // ---------------------------------------------------------------- copies
    int row = 0, ads[kIssue] = {};  // so far: tiles of y, and of B for each issuing warp
    for (int i = 0; ok; ++i) {
      ok = all_of(wait_segment(i));
      const Segment& s = s_seg[i & 1];
      if (!ok || s.count == 0) break;
      for (int n = 0; n < s.count && ok; ++n) {
        const int col = (s.first + n) * kCols, at = row % ROWS, x = row % kIssue;
#ifdef SP24_FAULT_WITHHOLD_FIRST_STAGE
        if (row == 0) {
          ++row;
          continue;
        }
#endif
        if (row >= ROWS) ok = all_of(mbar_wait(&row_empty[at], (row / ROWS - 1) & 1));
        if (!ok) break;
        load_rows(row_s + at * kRowTile, &ymap, &yrows, &row_full[at], col, s);
        ++row;
        int ad = x ? ads[1] : ads[0];
        for (int w = 0; w < s.adapters; ++w, ++ad) {
          const int to = x * C::A + ad % C::A;
          if (ad >= C::A) ok = all_of(mbar_wait(&ad_empty[to], (ad / C::A - 1) & 1));
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&ad_full[to], KB * 64 * 128);
#pragma unroll
            for (int k = 0; k < KB; ++k)
              tma_load_3d(ad_s + to * C::AD_TILE + k * 64 * 128, &bmap, &ad_full[to], 64 * k, col, s.adapter[w]);
          }
        }
        (x ? ads[1] : ads[0]) = ad;
      }
      done_with(i);
    }
    if (lane == 0) {
      if (!ok) atomicOr(p.err, DEVERR_TIMEOUT_PRODUCER);
      // Copies in flight have to land before this CTA's shared memory goes.
      for (int i = max(0, row - ROWS); i < row; ++i) mbar_wait(&row_full[i % ROWS], (i / ROWS) & 1);
#pragma unroll
      for (int x = 0; x < kIssue; ++x)
        for (int i = max(0, ads[x] - C::A); i < ads[x]; ++i) mbar_wait(&ad_full[x * C::A + i % C::A], (i / C::A) & 1);
    }
    __syncwarp();
  } else if (warp == STORE) {
    // ---------------------------------------------------------------- stores
    int row = 0;
    for (int i = 0; ok; ++i) {
      ok = all_of(wait_segment(i));
      const Segment& s = s_seg[i & 1];
      if (!ok || s.count == 0) break;
      for (int n = 0; n < s.count && ok; ++n, ++row) {
        const int stage = row % ROWS;
        ok = all_of(mbar_wait(&out_full[stage], (row / ROWS) & 1));
        if (!ok) break;
        store_rows(row_s + stage * kRowTile, &omap, &orows, (s.first + n) * kCols, s);
        bulk_commit();
        if (row > 0) {  // the store before this one has read its tile
          asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&row_empty[(row - 1) % ROWS]);
        }
      }
      done_with(i);
    }
    bulk_wait_all();
    if (lane == 0) {
      if (!ok) atomicOr(p.err, DEVERR_TIMEOUT_EPILOGUE);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------- MMA
    const int x = warp - ISSUE;  // every other product is this warp's
    const uint32_t id = idesc_bf16(kTile, kCols);
    const uint64_t ad_d = smem_desc(smem_u32(ad_s), 16, 1024, SWZ_128B);
    const uint64_t h_d = smem_desc(smem_u32(h_s), 16, 1024, SWZ_128B);
    int unit = 0, row0 = 0, tiles = 0;  // products of this warp so far, units before this segment, tiles with adapters
    for (int i = 0; ok; ++i) {
      ok = wait_segment(i);
      const Segment& s = s_seg[i & 1];
      if (!ok || s.count == 0) break;
      const int count = s.count, adapters = s.adapters;
      done_with(i);
      if (lane == 0 && adapters > 0) {
        ok = mbar_wait(&h_full[tiles % HS], (tiles / HS) & 1);
        const uint64_t h = h_d + tiles % HS * (C::H >> 4);
        for (int n = (row0 + x) % kIssue; n < count && ok; n += kIssue) {
          for (int w = 0; w < adapters && ok; ++w, ++unit) {
            const int from = x * C::A + unit % C::A, at = x * C::D2 + unit % C::D2;
            ok = mbar_wait(&ad_full[from], (unit / C::A) & 1) &&
                 (unit < C::D2 || mbar_wait(&d2_empty[at], (unit / C::D2 - 1) & 1));
            if (!ok) break;
            tc_fence_after();
            const uint64_t b = ad_d + from * (C::AD_TILE >> 4);
            for (int part = 0; part < 2; ++part)
              for (int e = 0; e < q.rp / 16; ++e)
                mma_bf16(tmem + at * kCols, h + part * (KB * kRowTile >> 4) + (e / 4) * (kRowTile >> 4) + 2 * (e & 3),
                         b + (e / 4) * (64 * 128 >> 4) + 2 * (e & 3), id, part > 0 || e > 0);
            mma_commit(&d2_full[at]);
          }
        }
        if (ok) mma_commit(&h_empty[tiles % HS]);
      }
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      row0 += count;
      if (adapters > 0) ++tiles;
    }
    if (lane == 0) {
      if (!ok) atomicOr(p.err, DEVERR_TIMEOUT_MMA);
      mma_commit(&drain[x]);  // every MMA issued must finish before tensor memory is freed
      mbar_wait(&drain[x], 0);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  pdl_trigger();
  if (warp == SEG) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

inline Deal deal_k(int64_t T, int64_t K, int sms) {
  return Deal::of(static_cast<unsigned int>((T + kTile - 1) / kTile * ((K + kCols - 1) / kCols)), sms, kLeastK);
}
inline size_t part_bytes(int64_t T, int64_t K, int64_t r, int sms) {
  return static_cast<size_t>((T + kTile - 1) / kTile + deal_k(T, K, sms).ctas) * kTile *
         static_cast<size_t>((r + 15) / 16 * 16) * sizeof(float);
}
inline size_t many_bytes(int64_t T, int64_t K, int64_t r, int sms) {  // sums, whether sorted, the rows
  return T <= kFew ? 0 : part_bytes(T, K, r, sms) + static_cast<size_t>((T + kWindow - 1) / kWindow + T) * sizeof(int32_t);
}

template <int KB>
sp24_status launch_many(const AdapterParams& p, float* part, const DeviceInfo& dev, cudaStream_t s) {
  CUtensorMap x, a, b, y, o, x1, y1, o1;
  const auto type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto swizzle = CU_TENSOR_MAP_SWIZZLE_128B;
  ManyParams q;
  q.p = p;
  q.kbs = (p.K + kCols - 1) / kCols, q.nbs = (p.N + kCols - 1) / kCols;
  q.rp = (p.r + 15) / 16 * 16;
  q.k = deal_k(p.T, p.K, dev.sm_count);
  q.n = Deal::of(static_cast<unsigned int>((p.T + kTile - 1) / kTile) * q.nbs, dev.sm_count, kLeastN);
  q.part = part;
  q.order = q.sorted = nullptr;
  const unsigned windows = static_cast<unsigned>((p.T + kWindow - 1) / kWindow);
  if (p.count > 1) {
    q.sorted = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(part) + part_bytes(p.T, p.K, p.r, dev.sm_count));
    q.order = q.sorted + windows;
  }
  sp24_status st = make_tmap_2d(&x, p.x, type, p.K, p.T, p.ldx * 2, kCols, kTile, swizzle);
  if (!st) st = make_tmap_2d(&y, p.y, type, p.N, p.T, p.ldy * 2, kCols, kTile, swizzle);
  if (!st) st = make_tmap_2d(&o, p.out, type, p.N, p.T, p.ldo * 2, kCols, kTile, swizzle);
  if (!st) st = make_tmap_2d(&x1, p.x, type, p.K, p.T, p.ldx * 2, kCols, 1, swizzle);
  if (!st) st = make_tmap_2d(&y1, p.y, type, p.N, p.T, p.ldy * 2, kCols, 1, swizzle);
  if (!st) st = make_tmap_2d(&o1, p.out, type, p.N, p.T, p.ldo * 2, kCols, 1, swizzle);
  if (!st) st = make_tmap_3d(&a, p.a, type, p.K, p.r, p.count, uint64_t(p.K) * 2, p.stride_a * 2, kCols, q.rp, swizzle);
  if (!st) st = make_tmap_3d(&b, p.b, type, p.r, p.N, p.count, uint64_t(p.r) * 2, p.stride_b * 2, 64, kCols, swizzle);
  if (st) return st;
  int bits = 0;
  while (int64_t(p.count) >> bits) ++bits;  // of ids + 1
  if ((q.order && launch_pdl_smem<adapters_sort_kernel>(dev, dim3(windows), dim3(kSortThreads), sizeof(SortSmem), s, q,
                                                        bits) != cudaSuccess) ||
      launch_pdl_smem<adapters_down_kernel<KB>>(dev, dim3(q.k.ctas), dim3(kDownThreads), DownCfg<KB>::SMEM, s, x, x1, a, q) !=
          cudaSuccess ||
      launch_pdl_smem<adapters_up_kernel<KB>>(dev, dim3(q.n.ctas), dim3(kUpThreads), UpCfg<KB>::SMEM, s, b, y, y1, o, o1, q) !=
          cudaSuccess)
    return SP24_ERR_CUDA;
  return SP24_OK;
}

template <int MT, int NT>
cudaError_t launch_few(const AdapterParams& p, const DeviceInfo& dev, cudaStream_t s) {
  using C = FewCfg<MT, NT>;
  constexpr auto kern = add_adapters_few_kernel<MT, NT>;
  // Each adapter's last item may be partly filled; rows without an adapter count as one more.
  const int64_t T = std::min(p.T, kFewRows), blocks = (p.T + kFewRows - 1) / kFewRows;
  const int64_t adapters = std::min<int64_t>(T, p.count), items = std::min<int64_t>(T, T / C::R + adapters + 1);
  // As many CTAs per item as run at once, for as many items as rows spread over the adapters come to, evenly or by chance
  // (each adapter's last item is half full then).  More items than that take a second wave: 512 rows of 8 adapters by chance,
  // rank 64, N 14336 23 us, 32 with clusters for rows spread evenly (which take 19 for rows of one adapter, and these 23).  (200 rows
  // of 20 adapters, rank 64, K 14336, 1 CTA per SM: 14 clusters of 8 fit, 24 of 6; 26 us with 8 and 17 with 6.  512 rows with an
  // adapter each, rank 16, K = N = 1024: 30 us in twos, 18 with one CTA for each.)
  auto expect = [&](int64_t rows) {
    const int64_t some = std::min<int64_t>(rows, p.count);
    return std::min(items, std::max(some * ((rows / some + C::R - 1) / C::R), rows / C::R + some / 2) + 1);
  };
  const int64_t likely = expect(T) + (p.T > kFewRows ? expect(p.T - kFewRows) : 0);
  static_assert(kFew <= 2 * kFewRows, "two blocks");
  static std::atomic<int> most[64][kMostCluster + 1];  // clusters of each size that fit at once, + 1
  unsigned cluster = kMostCluster;
  for (; cluster > 1; --cluster) {
    std::atomic<int>& known = most[dev.ordinal & 63][cluster];
    int n = known.load(std::memory_order_relaxed);
    if (n == 0) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = cluster;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(cluster);
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = C::SMEM;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int fit = 0;
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess ||
          cudaOccupancyMaxActiveClusters(&fit, kern, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        fit = 0;
      }
      n = fit + 1;
      known.store(n, std::memory_order_relaxed);
    }
    if (likely <= n - 1) break;
  }
  return launch_pdl_clusters_smem<kern>(dev, cluster, dim3(static_cast<unsigned>(blocks * items * cluster)), dim3(kThreads),
                                        C::SMEM, s, p, static_cast<int>(items));
}
// Rows per item: 8 or 16, so that an adapter is rarely read more than once if its rows are few.  (200 rows of 20, K 14336,
// rank 64: 21 us with 8, 17.6 with 16; 40 rows of 8, K 4096, rank 16: 5.4 and 6.2, all at the time.  With 32, fewer CTAs have more to do:
// 512 rows in runs, K = N = 4096, rank 64 14.6 us, 12.6 with 16.)
template <int MT>
cudaError_t launch_few(const AdapterParams& p, const DeviceInfo& dev, cudaStream_t s) {
  const int64_t T = std::min(p.T, kFewRows), each = T / std::min<int64_t>(T, p.count);
  return each > 7 ? launch_few<MT, 2>(p, dev, s) : launch_few<MT, 1>(p, dev, s);
}

}  // namespace
}  // namespace sp24

extern "C" size_t sp24_add_adapters_workspace_size(int64_t T, int64_t K, int64_t r) {
  using namespace sp24;
  const int64_t most = int64_t(1) << 24;
  const DeviceInfo* dev = nullptr;
  if (T <= kFew || T > INT32_MAX / 2 || K < 8 || K > most || r < 1 || r > kMostRank || current_device(&dev)) return 0;
  return many_bytes(T, K, r, dev->sm_count);
}

extern "C" sp24_status sp24_add_adapters(const void* Y, int64_t ldy, const void* X, int64_t ldx, int64_t T, int64_t K,
                                         int64_t N, const void* A, int64_t stride_a, const void* B, int64_t stride_b,
                                         int64_t r, int64_t count, const int32_t* ids, const float* scales, void* out,
                                         int64_t ldo, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace sp24;
  const int64_t most = int64_t(1) << 24;
  if (T < 0 || T > INT32_MAX / 2 || K < 8 || N < 8 || K > most || N > most || r < 1 || count < 1 || count > INT32_MAX)
    return SP24_ERR_INVALID_ARG;
  if (K % 8 || N % 8 || r % 8 || r > kMostRank) return SP24_ERR_UNSUPPORTED;
  if (T > 0) {
    if (!Y || !X || !A || !B || !ids || !out) return SP24_ERR_INVALID_ARG;
    const int64_t far = int64_t(1) << 39;
    if (ldy < N || ldo < N || ldx < K || ldy >= far || ldo >= far || ldx >= far) return SP24_ERR_INVALID_ARG;
    if (stride_a < r * K || stride_b < N * r || stride_a >= far || stride_b >= far) return SP24_ERR_INVALID_ARG;
    if (!aligned16(Y) || !aligned16(X) || !aligned16(A) || !aligned16(B) || !aligned16(out) ||
        (ldy | ldx | ldo | stride_a | stride_b) % 8)
      return SP24_ERR_ALIGNMENT;
    if ((reinterpret_cast<uintptr_t>(ids) | reinterpret_cast<uintptr_t>(scales)) & 3u) return SP24_ERR_ALIGNMENT;
  }
  const DeviceInfo* dev = nullptr;
  if (sp24_status st = current_device(&dev)) return st;
  if (T == 0) return SP24_OK;
  if (const size_t need = many_bytes(T, K, r, dev->sm_count)) {
    if (!workspace || workspace_bytes < need) return SP24_ERR_WORKSPACE;
    if (!aligned16(workspace)) return SP24_ERR_ALIGNMENT;
    const int64_t tiles = (T + kTile - 1) / kTile, most = INT32_MAX / tiles;
    if ((K + kCols - 1) / kCols > most || (N + kCols - 1) / kCols > most) return SP24_ERR_UNSUPPORTED;  // 32-bit units
  }
  AdapterParams p;
  p.y = static_cast<const __nv_bfloat16*>(Y);
  p.x = static_cast<const __nv_bfloat16*>(X);
  p.a = static_cast<const __nv_bfloat16*>(A);
  p.b = static_cast<const __nv_bfloat16*>(B);
  p.ids = ids;
  p.scales = scales;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.ldy = ldy, p.ldx = ldx, p.ldo = ldo, p.stride_a = stride_a, p.stride_b = stride_b;
  p.T = static_cast<int>(T), p.K = static_cast<int>(K), p.N = static_cast<int>(N);
  p.r = static_cast<int>(r), p.count = static_cast<int>(count);
  p.err = dev->err_word;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (T > kFew)
    return r <= 64 ? launch_many<1>(p, static_cast<float*>(workspace), *dev, s)
                   : launch_many<2>(p, static_cast<float*>(workspace), *dev, s);
  if (r <= 16)
    e = launch_few<1>(p, *dev, s);
  else if (r <= 32)
    e = launch_few<2>(p, *dev, s);
  else if (r <= 64)
    e = launch_few<4>(p, *dev, s);
  else
    e = launch_few<8>(p, *dev, s);
  return e == cudaSuccess ? SP24_OK : SP24_ERR_CUDA;
}
