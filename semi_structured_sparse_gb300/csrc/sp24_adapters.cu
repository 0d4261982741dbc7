// sp24_adapters.cu -- sp24_add_adapters: to every row of a projection's output
// the product of its request's low-rank adapter,
//
//   out[t] = y[t] + scale_i B_i (A_i x[t]),  i = ids[t]
//
// Bound by memory: rows and the adapters in use are read once, and 2 r
// operations per value of x and y are few.
#include <cuda_bf16.h>
#include <algorithm>
#include <cmath>
#include "sp24_internal.cuh"
#include "sp24_ptx.cuh"

namespace sp24 {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCluster = 8;        // CTAs that share a few rows' work
constexpr int kMostRank = 128;
constexpr int kFewRows = 512;      // rows of a call that are sorted by adapter

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
// are in the batch; a cluster of 8 CTAs works on it.  Their 64 warps cut K for
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
  static constexpr int STAGES = MT <= 2 ? 4 : 2;
  static constexpr int HLD = 32 * KS + 8;                // row of A x, in bf16
  static constexpr int RING = kWarps * STAGES * LOADS * 512, PART = kWarps * R * RP * 4;
  static constexpr int FIRST = RING > PART ? RING : PART;  // the ring, and then the warps' sums
  static constexpr int RECV = kCluster * R * RP * 4, H = 2 * R * HLD * 2;
  static constexpr int SMEM = FIRST + RECV + H;
};
template <int MT, int NT>
__global__ void __launch_bounds__(kThreads) add_adapters_few_kernel(const __grid_constant__ AdapterParams p) {
  using C = FewCfg<MT, NT>;
  constexpr int R = C::R, RP = C::RP, KS = C::KS, ST = C::STAGES, MH = (NT + 1) / 2;  // 16-row tiles of tokens
  extern __shared__ __align__(128) uint8_t smem[];
  float* const part = reinterpret_cast<float*>(smem);                       // [kWarps][R][RP]
  float* const recv = reinterpret_cast<float*>(smem + C::FIRST);            // [kCluster][R][RP]
  uint8_t* const h_s = smem + C::FIRST + C::RECV;                           // [2][R][HLD] bf16
  __shared__ __align__(16) int s_id[kFewRows];
  __shared__ int s_count[kFewRows / 32], s_item[2], s_row[R];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t rank = cluster_rank();
  const int item = blockIdx.x / kCluster, gw = rank * kWarps + warp;
  constexpr int GW = kCluster * kWarps;
  pdl_wait();

  // ---- this cluster's item: rows are numbered within their adapter; every R-th begins one
  constexpr int MINE = kFewRows / kThreads;
  int id[MINE], nth[MINE];
  bool first[MINE];
#pragma unroll
  for (int i = 0; i < MINE; ++i) {
    const int x = tid + i * kThreads;
    id[i] = -2;
    if (x < p.T) {
      id[i] = p.ids[x];
      if (id[i] >= p.count) {
        if (blockIdx.x == 0) atomicOr(p.err, DEVERR_INDEX);
        id[i] = -1;
      }
      id[i] = max(id[i], -1);
    }
    s_id[x] = id[i];
    nth[i] = 0;
  }
  if (tid < R) s_row[tid] = -1;
  if (tid == 0) s_item[0] = -1;
  __syncthreads();
  const int scan = min(p.T, kFewRows);
  for (int x = 0; x < scan; x += 4) {
    const int4 v = *reinterpret_cast<const int4*>(s_id + x);
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      const int me = tid + i * kThreads;
      nth[i] += (v.x == id[i] && x < me) + (v.y == id[i] && x + 1 < me) + (v.z == id[i] && x + 2 < me) +
                (v.w == id[i] && x + 3 < me);
    }
  }
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
    if (id[i] == adapter && nth[i] >= from && nth[i] < from + R) s_row[nth[i] - from] = tid + i * kThreads;
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
  // this CTA's rows of B on their way to L2 meanwhile
  const int blocks = (p.N + 31) / 32;
  {
    const int b0 = static_cast<int>(int64_t(blocks) * (rank * kWarps) / GW) * 32;
    const int b1 = min(p.N, static_cast<int>(int64_t(blocks) * ((rank + 1) * kWarps) / GW) * 32);
    const __nv_bfloat16* b = p.b + adapter * p.stride_b;
    constexpr int PIECE = 8192;
    const int64_t bytes = int64_t(b1 - b0) * p.r * 2;
    for (int64_t i = int64_t(tid) * PIECE; i < bytes; i += int64_t(kThreads) * PIECE)
      bulk_prefetch_l2(reinterpret_cast<const uint8_t*>(b + int64_t(b0) * p.r) + i,
                       static_cast<uint32_t>(min(int64_t(PIECE), bytes - i)));
  }
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
  int row[2 * MH];
#pragma unroll
  for (int i = 0; i < 2 * MH; ++i) row[i] = i < NT ? s_row[8 * i + g] : -1;
  uint4 bv[KS][4], yv[2 * MH];
  auto load = [&](int block) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = 32 * block + 8 * (g >> 1) + 2 * j + (g & 1);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        bv[s][j] = make_uint4(0, 0, 0, 0);
        if (n < p.N && 32 * s + 8 * t < p.r)
          bv[s][j] = *reinterpret_cast<const uint4*>(b + int64_t(n) * p.r + 32 * s + 8 * t);
      }
    }
#pragma unroll
    for (int i = 0; i < 2 * MH; ++i) {
      yv[i] = make_uint4(0, 0, 0, 0);
      if (row[i] >= 0 && 32 * block + 8 * t < p.N)
        yv[i] = *reinterpret_cast<const uint4*>(p.y + row[i] * p.ldy + 32 * block + 8 * t);
    }
  };
  if (n0 < n1) load(n0);

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
    for (uint32_t c = 0; c < kCluster; ++c) st_cluster(cluster_addr(recv + rank * (R * RP) + e, c), sum);
  }
  cluster_sync();
  const float scale = p.scales ? p.scales[adapter] : 1.0f;
  __nv_bfloat16* const h_hi = reinterpret_cast<__nv_bfloat16*>(h_s);
  __nv_bfloat16* const h_lo = h_hi + R * C::HLD;
  // A x in two bf16 parts, which hold it to 2^-16: one alone would move the product by 2^-8 of it.
  for (int e = tid; e < R * 32 * KS; e += kThreads) {
    const int i = e / (32 * KS), j = e % (32 * KS);
    float sum = 0.0f;
    if (j < RP) {
#pragma unroll
      for (int c = 0; c < kCluster; ++c) sum += recv[c * (R * RP) + i * RP + j];
      sum *= scale;
    }
    const __nv_bfloat16 hi = __float2bfloat16(sum);
    const float rest = sum - __bfloat162float(hi);
    h_hi[i * C::HLD + j] = hi;
    h_lo[i * C::HLD + j] = __float2bfloat16(isfinite(rest) ? rest : 0.0f);
  }
  __syncthreads();

  // ---- B (A x), this warp's columns, 32 at a time
  for (int block = n0; block < n1; ++block) {
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
            mma16816(o[m][j], lo.x, hi.x, lo.y, hi.y, bv[s][j].x, bv[s][j].y);
            mma16816(o[m][j], lo.z, hi.z, lo.w, hi.w, bv[s][j].z, bv[s][j].w);
          }
        }
      }
    }
    uint4 y[2 * MH];
#pragma unroll
    for (int i = 0; i < 2 * MH; ++i) y[i] = yv[i];
    if (block + 1 < n1) load(block + 1);
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
  pdl_trigger();
}

// Many rows.  A tile of 128 rows in a row is a cluster's, whose CTAs cut K and then N
// among themselves, as above.  Both products are tcgen05.mma with operands by TMA:
// A x as D1 (128 rows x rank, in tensor memory), whose partial sums each CTA
// sends to the CTA that owns the row (distributed shared memory); the owner adds
// them up in order and sends the row's two bf16 parts to all, which is the A
// operand of D2 = (A x) B^T, 64 columns at a time.  A tile's rows may have
// several adapters: each is a pass over K, and a product per 64 columns, of
// which a row takes those of its own (a row's products are its own, so what
// another adapter makes of it reaches nothing).
//
// y's tiles come into the ring that x's came through, beside which the two
// matrices' tiles have one; the copies run ahead of the products, and so through the
// exchange.  The sum is formed in y's tile in shared memory, and stored from
// there.
constexpr int kTile = 128;          // rows
constexpr int kCols = 64;           // K, or N, per stage
constexpr int kRowTile = kTile * kCols * 2;
constexpr int kMostCluster = 8;
constexpr int kSumWarps = 8;
constexpr int kIssue = 2;           // warps that issue MMAs: a commit holds its thread back until they are done
constexpr int kManyThreads = (kSumWarps + 2 + kIssue) * 32;
template <int KB>  // 64s of the rank
struct ManyCfg {
  static constexpr int ROWS = KB == 1 ? 6 : 3, ADS = KB == 1 ? 6 : 2;  // stages
  static constexpr int D1 = 64 * KB;                   // columns of an adapter's D1
  static constexpr int PASS = 256 / (kIssue * D1);     // adapters per pass over K
  static constexpr int AD_TILE = KB * 64 * 128;
  static constexpr int RP4 = KB * 64 + 4;  // row of the sums' exchange, in floats
  static constexpr int RECV = (kTile + kMostCluster) * RP4 * 4;
  static constexpr int H = 2 * KB * kRowTile;  // two parts
  static constexpr int BARS = 3 * ROWS + 2 * ADS + 2 + 2 * 4 + 2 + kIssue;
  static constexpr int SMEM = 1024 + ROWS * kRowTile + ADS * AD_TILE + H + RECV + BARS * 8;
};

// Arrive, with release, on the mbarrier at p's offset in CTA `rank` of the cluster.
__device__ __forceinline__ void mbar_arrive_cluster(uint64_t* bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr(bar, rank)) : "memory");
}
// mbar_wait for what other CTAs of the cluster have written before they arrived.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i) {
      uint32_t ok;
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(smem_u32(bar)), "r"(parity)
          : "memory");
      if (ok) return true;
    }
    if (globaltimer_ns() - t0 > SP24_WAIT_TIMEOUT_NS) return false;
  }
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

template <int KB>
__global__ void __launch_bounds__(kManyThreads, 1)
    add_adapters_many_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap amap,
                             const __grid_constant__ CUtensorMap bmap, const __grid_constant__ CUtensorMap ymap,
                             const __grid_constant__ CUtensorMap omap, const __grid_constant__ AdapterParams p) {
  using C = ManyCfg<KB>;
  constexpr int ROWS = C::ROWS, ADS = C::ADS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ int s_which[kTile];    // of each row: which of the tile's adapters, or -1
  __shared__ int s_adapter[kTile];  // the tile's adapters
  __shared__ int s_adapters;
  __shared__ float s_scale[kTile];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const row_s = smem;
  uint8_t* const ad_s = row_s + ROWS * kRowTile;
  uint8_t* const h_s = ad_s + ADS * C::AD_TILE;
  float* const recv = reinterpret_cast<float*>(h_s + C::H);
  uint64_t* const bars = reinterpret_cast<uint64_t*>(h_s + C::H + C::RECV);
  uint64_t* const row_full = bars;                // [ROWS]
  uint64_t* const row_empty = row_full + ROWS;
  uint64_t* const out_full = row_empty + ROWS;    // [ROWS] the tile holds results
  uint64_t* const ad_full = out_full + ROWS;      // [ADS]
  uint64_t* const ad_empty = ad_full + ADS;
  uint64_t* const d1_full = ad_empty + ADS;
  uint64_t* const d1_empty = d1_full + 1;
  uint64_t* const d2_full = d1_empty + 1;         // [4]
  uint64_t* const d2_empty = d2_full + 4;
  uint64_t* const recv_full = d2_empty + 4;       // all CTAs' sums of this one's rows are there
  uint64_t* const h_full = recv_full + 1;         // all rows of A x are there
  uint64_t* const drain = h_full + 1;             // [kIssue]

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const uint32_t rank = cluster_rank(), ctas = cluster_nrank();
  const int row0 = blockIdx.x / ctas * kTile;
  if (warp == kSumWarps) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  } else if (warp == kSumWarps + 1 && lane == 0) {
    for (int i = 0; i < ROWS; ++i) {
      mbar_init(&row_full[i], 1);
      mbar_init(&row_empty[i], 1);
      mbar_init(&out_full[i], kSumWarps);
    }
    for (int i = 0; i < ADS; ++i) mbar_init(&ad_full[i], 1), mbar_init(&ad_empty[i], 1);
    mbar_init(d1_full, kIssue);
    mbar_init(d1_empty, kSumWarps);
    for (int i = 0; i < 4; ++i) mbar_init(&d2_full[i], 1), mbar_init(&d2_empty[i], kSumWarps);
    mbar_init(recv_full, kSumWarps * ctas);
    mbar_init(h_full, kSumWarps * ctas);
    for (int i = 0; i < kIssue; ++i) mbar_init(&drain[i], 1);
    fence_mbar_init();
    tma_prefetch_desc(&xmap), tma_prefetch_desc(&amap), tma_prefetch_desc(&bmap);
    tma_prefetch_desc(&ymap), tma_prefetch_desc(&omap);
  }
  cluster_sync();  // the other CTAs have begun, and their barriers are there
  pdl_wait();
  const int kbs = (p.K + kCols - 1) / kCols, nbs = (p.N + kCols - 1) / kCols;
  const int k0 = static_cast<int>(int64_t(kbs) * rank / ctas), nk = static_cast<int>(int64_t(kbs) * (rank + 1) / ctas) - k0;
  const int n0 = static_cast<int>(int64_t(nbs) * rank / ctas), nn = static_cast<int>(int64_t(nbs) * (rank + 1) / ctas) - n0;
  const int ahead = min(ROWS, nk);  // tiles of x that come before it is known which rows have an adapter
  if (warp == kSumWarps && lane == 0) {
    for (int i = 0; i < ahead; ++i) {
      mbar_arrive_expect_tx(&row_full[i], kRowTile);
      tma_load_2d(row_s + i * kRowTile, &xmap, &row_full[i], (k0 + i) * kCols, row0);
    }
  }
  if (warp == 0) {
    int id[kTile / 32], which[kTile / 32];
#pragma unroll
    for (int i = 0; i < kTile / 32; ++i) {
      const int x = row0 + 32 * i + lane;
      id[i] = x < p.T ? p.ids[x] : -1;
      if (id[i] >= p.count) {
        if (rank == 0) atomicOr(p.err, DEVERR_INDEX);
        id[i] = -1;
      }
      which[i] = -1;
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
        if (lane == 0) s_adapter[n] = now;
        ++n;
      }
    }
#pragma unroll
    for (int i = 0; i < kTile / 32; ++i) s_which[32 * i + lane] = which[i];
    if (lane == 0) s_adapters = n;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem, d1 = tmem, d2 = tmem + 256;
  const int adapters = s_adapters, passes = (adapters + C::PASS - 1) / C::PASS;
  const int rp = (p.r + 15) / 16 * 16;
  const int rows1 = max(passes * nk, ahead);  // tiles of x that come through the ring
  bool ok = true;

  if (warp < kSumWarps) {
    // ------------------------------------------------------------------ sums
    const int r = tid & (kTile - 1), half = tid / kTile, which = s_which[r];
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int own = (kTile + ctas - 1) / ctas;  // rows that a CTA adds up
    if (tid < adapters) s_scale[tid] = p.scales ? p.scales[s_adapter[tid]] : 1.0f;  // (seen by all after recv_full)
    const uint32_t to = cluster_addr(recv + (rank * own + r % own) * C::RP4, r / own);
    for (int pass = 0; pass < passes && ok; ++pass) {
      if (nk > 0) ok = mbar_wait(d1_full, pass & 1);
      if (!ok) break;
      tc_fence_after();
      for (int w = pass * C::PASS; w < min(adapters, (pass + 1) * C::PASS); ++w) {
        if (!__any_sync(0xFFFFFFFFu, which == w)) continue;
        for (int c = half * (rp / 2); c < (half + 1) * (rp / 2); c += 8) {
          uint32_t v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = 0;
          for (int x = 0; x < min(kIssue, nk); ++x) {  // what each issuing warp's stages came to
            uint32_t u[8];
            tmem_ld8(d1 + lanes + ((w - pass * C::PASS) * kIssue + x) * C::D1 + c, u);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(u[i]));
          }
          if (which == w) {
            st_cluster_v4(to + 4 * c, v[0], v[1], v[2], v[3]);
            st_cluster_v4(to + 4 * c + 16, v[4], v[5], v[6], v[7]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(d1_empty);
    }
    if (passes > 0 && ok) {
      __syncwarp();
      if (lane < static_cast<int>(ctas)) mbar_arrive_cluster(recv_full, lane);
      ok = mbar_wait_cluster(recv_full, 0);
      if (ok) {
        const int pieces = rp / 8;
        for (int e = tid; e < own * pieces; e += kSumWarps * 32) {
          const int i = e / pieces, c = e - i * pieces, x = rank * own + i;
          const int w = x < kTile ? s_which[x] : -1;
          if (w < 0) continue;
          float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
          for (uint32_t k = 0; k < ctas; ++k) {
            const float4* v = reinterpret_cast<const float4*>(recv + (k * own + i) * C::RP4 + 8 * c);
            const float4 lo = v[0], hi = v[1];
            sum[0] += lo.x, sum[1] += lo.y, sum[2] += lo.z, sum[3] += lo.w;
            sum[4] += hi.x, sum[5] += hi.y, sum[6] += hi.z, sum[7] += hi.w;
          }
          const float scale = s_scale[w];
          uint32_t big[4], rest[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a = sum[2 * k] * scale, b = sum[2 * k + 1] * scale;
            big[k] = bf16x2_rn(a, b);
            const float ra = a - __uint_as_float(big[k] << 16), rb = b - __uint_as_float(big[k] & 0xFFFF0000u);
            rest[k] = bf16x2_rn(isfinite(ra) ? ra : 0.0f, isfinite(rb) ? rb : 0.0f);
          }
          uint8_t* to = h_s + (c / 8) * kRowTile + x * 128 + (((c & 7) ^ (x & 7)) << 4);
          for (uint32_t k = 0; k < ctas; ++k) {
            st_cluster_v4(cluster_addr(to, k), big[0], big[1], big[2], big[3]);
            st_cluster_v4(cluster_addr(to + KB * kRowTile, k), rest[0], rest[1], rest[2], rest[3]);
          }
        }
        fence_proxy_async_all();
        __syncwarp();
        if (lane < static_cast<int>(ctas)) mbar_arrive_cluster(h_full, lane);
      }
    }
    int unit = 0, ring = rows1, ad = adapters * nk;
    for (int n = 0; n < nn && ok; ++n, ++ring) {
      uint32_t v[32];
      for (int w = 0; w < adapters; ++w, ++unit, ++ad) {
        ok = mbar_wait(&d2_full[unit & 3], (unit >> 2) & 1);
        if (!ok) break;
        if (tid == 0) mbar_arrive(&ad_empty[ad % ADS]);  // the product has been formed
        tc_fence_after();
        if (__any_sync(0xFFFFFFFFu, which == w)) {
          uint32_t u[16];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            tmem_ld16(d2 + lanes + (unit & 3) * kCols + half * 32 + 16 * k, u);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (which == w) v[16 * k + i] = u[i];
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&d2_empty[unit & 3]);
      }
      const int stage = ring % ROWS;
      if (ok) ok = mbar_wait(&row_full[stage], (ring / ROWS) & 1);
      if (!ok) break;
      if (which >= 0) {
        uint8_t* y = row_s + stage * kRowTile + r * 128;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint4* at = reinterpret_cast<uint4*>(y + (((half * 4 + k) ^ (r & 7)) << 4));
          const uint4 w = *at;
          auto add = [&](uint32_t two, int i) {
            return bf16x2_rn(__uint_as_float(two << 16) + __uint_as_float(v[8 * k + 2 * i]),
                             __uint_as_float(two & 0xFFFF0000u) + __uint_as_float(v[8 * k + 2 * i + 1]));
          };
          *at = make_uint4(add(w.x, 0), add(w.y, 1), add(w.z, 2), add(w.w, 3));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&out_full[stage]);
    }
    if (!ok && lane == 0) atomicOr(p.err, DEVERR_TIMEOUT_EPILOGUE);
  } else if (warp == kSumWarps) {
    // ---------------------------------------------------------------- copies
    if (lane == 0) {
      int row = ahead, ad = 0;
      // An adapter's tile, when the one before it in its place has been used.
      auto ad_free = [&](int use) {  // (a place that has been filled again since has been waited for)
        return use < 0 || use + ADS < ad || mbar_wait(&ad_empty[use % ADS], (use / ADS) & 1);
      };
      auto ad_stage = [&](uint32_t bytes) {
        ok = ad_free(ad - ADS);
        if (ok) mbar_arrive_expect_tx(&ad_full[ad % ADS], bytes);
        return ok;
      };
      auto row_tile = [&](const CUtensorMap* map, int x) {
        mbar_arrive_expect_tx(&row_full[row % ROWS], kRowTile);
        tma_load_2d(row_s + (row % ROWS) * kRowTile, map, &row_full[row % ROWS], x, row0);
        ++row;
      };
      // A tile of x has been used when the last of its pass's adapters has.
      int last[ROWS];
#pragma unroll
      for (int i = 0; i < ROWS; ++i) last[i] = -1;
      for (int pass = 0; pass < passes && ok; ++pass) {
        const int w0 = pass * C::PASS, w1 = min(adapters, w0 + C::PASS);
        for (int k = 0; k < nk && ok; ++k) {
          const int use = pass * nk + k;
          if (use >= ahead) {
            ok = ad_free(last[use % ROWS]);
            if (!ok) break;
            row_tile(&xmap, (k0 + k) * kCols);
          }
          for (int w = w0; w < w1 && ok; ++w) {
            if (!ad_stage(rp * 128)) break;
            tma_load_3d(ad_s + (ad % ADS) * C::AD_TILE, &amap, &ad_full[ad % ADS], (k0 + k) * kCols, 0, s_adapter[w]);
            ++ad;
          }
          last[use % ROWS] = ad - 1;
        }
      }
      for (int n = 0; n < nn && ok; ++n) {
        const int use = row;
        if (n >= ROWS)
          ok = mbar_wait(&row_empty[use % ROWS], (n / ROWS - 1) & 1);
        else if (passes > 0)
          ok = ad_free(last[use % ROWS]);
        else if (use >= ROWS || use % ROWS < ahead)  // no row has an adapter: x's tiles have landed, that is all
          ok = mbar_wait(&row_full[use % ROWS], 0);
        if (!ok) break;
        row_tile(&ymap, (n0 + n) * kCols);
        for (int w = 0; w < adapters && ok; ++w) {
          if (!ad_stage(KB * 64 * 128)) break;
#pragma unroll
          for (int k = 0; k < KB; ++k)
            tma_load_3d(ad_s + (ad % ADS) * C::AD_TILE + k * 64 * 128, &bmap, &ad_full[ad % ADS], 64 * k, (n0 + n) * kCols,
                        s_adapter[w]);
          ++ad;
        }
      }
      if (!ok) atomicOr(p.err, DEVERR_TIMEOUT_PRODUCER);
      // Copies in flight have to land before this CTA's shared memory goes.
      for (int i = max(0, row - ROWS); i < row; ++i) mbar_wait(&row_full[i % ROWS], (i / ROWS) & 1);
      for (int i = max(0, ad - ADS); i < ad; ++i) mbar_wait(&ad_full[i % ADS], (i / ADS) & 1);
    }
    __syncwarp();
  } else if (warp == kSumWarps + 2) {
    // ---------------------------------------------------------------- stores
    if (lane == 0) {
      const int ring = rows1;
      for (int n = 0; n < nn && ok; ++n) {
        const int stage = (ring + n) % ROWS;
        ok = mbar_wait(&out_full[stage], (n / ROWS) & 1);
        if (!ok) break;
        tma_store_2d(&omap, row_s + stage * kRowTile, (n0 + n) * kCols, row0);
        bulk_commit();
        if (n > 0) {  // the store before this one has read its tile
          asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          mbar_arrive(&row_empty[(ring + n - 1) % ROWS]);
        }
      }
      bulk_wait_all();
      if (!ok) atomicOr(p.err, DEVERR_TIMEOUT_EPILOGUE);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------- MMA
    if (lane == 0) {
      const int x = warp == kSumWarps + 1 ? 0 : 1;  // every other stage and product
      const uint32_t id1 = idesc_bf16(kTile, rp), id2 = idesc_bf16(kTile, kCols);
      const uint64_t row_d = smem_desc(smem_u32(row_s), 16, 1024, SWZ_128B);
      const uint64_t ad_d = smem_desc(smem_u32(ad_s), 16, 1024, SWZ_128B);
      const uint64_t h_d = smem_desc(smem_u32(h_s), 16, 1024, SWZ_128B);
      for (int pass = 0; pass < passes && ok; ++pass) {
        const int w0 = pass * C::PASS, w1 = min(adapters, w0 + C::PASS);
        if (nk > 0 && pass > 0) ok = mbar_wait(d1_empty, (pass - 1) & 1);
        for (int k = x; k < nk && ok; k += kIssue) {
          const int row = pass * nk + k;
          ok = mbar_wait(&row_full[row % ROWS], (row / ROWS) & 1);
          const uint64_t a = row_d + (row % ROWS) * (kRowTile >> 4);
          for (int w = w0; w < w1 && ok; ++w) {
            const int ad = w0 * nk + k * (w1 - w0) + w - w0;
            ok = mbar_wait(&ad_full[ad % ADS], (ad / ADS) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t b = ad_d + (ad % ADS) * (C::AD_TILE >> 4);
#pragma unroll
            for (int i = 0; i < kCols / 16; ++i)
              mma_bf16(d1 + ((w - w0) * kIssue + x) * C::D1, a + 2 * i, b + 2 * i, id1, k >= kIssue || i > 0);
            mma_commit(&ad_empty[ad % ADS]);
          }
        }
        if (nk > 0 && ok) mma_commit(d1_full);
      }
      if (passes > 0 && ok) ok = mbar_wait_cluster(h_full, 0);
      fence_proxy_async_all();
      for (int unit = x; unit < nn * adapters && ok; unit += kIssue) {
        const int ad = adapters * nk + unit;
        ok = mbar_wait(&ad_full[ad % ADS], (ad / ADS) & 1) &&
             (unit < 4 || mbar_wait(&d2_empty[unit & 3], ((unit >> 2) - 1) & 1));
        if (!ok) break;
        tc_fence_after();
        const uint64_t b = ad_d + (ad % ADS) * (C::AD_TILE >> 4);
        for (int part = 0; part < 2; ++part)
          for (int i = 0; i < rp / 16; ++i) {
            const uint64_t at = h_d + part * (KB * kRowTile >> 4) + (i / 4) * (kRowTile >> 4) + 2 * (i & 3);
            mma_bf16(d2 + (unit & 3) * kCols, at, b + (i / 4) * (64 * 128 >> 4) + 2 * (i & 3), id2, part > 0 || i > 0);
          }
        mma_commit(&d2_full[unit & 3]);
      }
      if (!ok) atomicOr(p.err, DEVERR_TIMEOUT_MMA);
      mma_commit(&drain[x]);  // every MMA issued must finish before tensor memory is freed
      mbar_wait(&drain[x], 0);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  pdl_trigger();
  if (warp == kSumWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  cluster_sync();  // no CTA writes to another's shared memory any more
}

// CTAs per cluster for so many tiles: as many as all of them still run at once with.
template <int KB>
unsigned many_cluster(const DeviceInfo& dev, int64_t tiles) {
  static std::atomic<int> most[64][kMostCluster + 1];  // clusters of each size that fit at once, + 1
  for (unsigned c = kMostCluster; c > 1; --c) {
    if (tiles * c > dev.sm_count) continue;
    std::atomic<int>& known = most[dev.ordinal & 63][c];
    int n = known.load(std::memory_order_relaxed);
    if (n == 0) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = c;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(c);
      cfg.blockDim = dim3(kManyThreads);
      cfg.dynamicSmemBytes = ManyCfg<KB>::SMEM;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int fit = 0;
      if (cudaFuncSetAttribute(add_adapters_many_kernel<KB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               ManyCfg<KB>::SMEM) != cudaSuccess ||
          cudaOccupancyMaxActiveClusters(&fit, add_adapters_many_kernel<KB>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        fit = 0;
      }
      n = fit + 1;
      known.store(n, std::memory_order_relaxed);
    }
    if (tiles <= n - 1) return c;
  }
  return 1;
}

template <int KB>
sp24_status launch_many(const AdapterParams& p, const DeviceInfo& dev, cudaStream_t s) {
  using C = ManyCfg<KB>;
  CUtensorMap x, a, b, y, o;
  const auto type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto swizzle = CU_TENSOR_MAP_SWIZZLE_128B;
  const uint32_t rp = (p.r + 15) / 16 * 16;
  sp24_status st = make_tmap_2d(&x, p.x, type, p.K, p.T, p.ldx * 2, kCols, kTile, swizzle);
  if (!st) st = make_tmap_2d(&y, p.y, type, p.N, p.T, p.ldy * 2, kCols, kTile, swizzle);
  if (!st) st = make_tmap_2d(&o, p.out, type, p.N, p.T, p.ldo * 2, kCols, kTile, swizzle);
  if (!st) st = make_tmap_3d(&a, p.a, type, p.K, p.r, p.count, uint64_t(p.K) * 2, p.stride_a * 2, kCols, rp, swizzle);
  if (!st) st = make_tmap_3d(&b, p.b, type, p.r, p.N, p.count, uint64_t(p.r) * 2, p.stride_b * 2, 64, kCols, swizzle);
  if (st) return st;
  const int64_t tiles = (p.T + kTile - 1) / kTile;
  const unsigned c = many_cluster<KB>(dev, tiles);
  return launch_pdl_clusters_smem<add_adapters_many_kernel<KB>>(dev, c, dim3(static_cast<unsigned>(tiles * c)),
                                                                dim3(kManyThreads), C::SMEM, s, x, a, b, y, o,
                                                                p) == cudaSuccess
             ? SP24_OK
             : SP24_ERR_CUDA;
}

template <int MT, int NT>
cudaError_t launch_few(const AdapterParams& p, const DeviceInfo& dev, cudaStream_t s) {
  using C = FewCfg<MT, NT>;
  // Each adapter's last item may be partly filled; rows without an adapter count as one more.
  const int items = std::min<int64_t>(p.T, p.T / C::R + std::min<int64_t>(p.T, int64_t(p.count) + 1));
  return launch_pdl_clusters_smem<add_adapters_few_kernel<MT, NT>>(dev, kCluster, dim3(items * kCluster), dim3(kThreads),
                                                                   C::SMEM, s, p);
}

}  // namespace
}  // namespace sp24

extern "C" sp24_status sp24_add_adapters(const void* Y, int64_t ldy, const void* X, int64_t ldx, int64_t T, int64_t K,
                                         int64_t N, const void* A, int64_t stride_a, const void* B, int64_t stride_b,
                                         int64_t r, int64_t count, const int32_t* ids, const float* scales, void* out,
                                         int64_t ldo, void* stream) {
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
  if (T > kFewRows) return r <= 64 ? launch_many<1>(p, *dev, s) : launch_many<2>(p, *dev, s);
  if (r <= 16)
    e = launch_few<1, 1>(p, *dev, s);
  else if (r <= 32)
    e = launch_few<2, 1>(p, *dev, s);
  else if (r <= 64)
    e = launch_few<4, 1>(p, *dev, s);
  else
    e = launch_few<8, 1>(p, *dev, s);
  return e == cudaSuccess ? SP24_OK : SP24_ERR_CUDA;
}
