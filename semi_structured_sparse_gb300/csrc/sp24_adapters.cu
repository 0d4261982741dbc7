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

// Many rows, one block each (to be replaced).
__global__ void __launch_bounds__(kThreads) add_adapters_kernel(const __grid_constant__ AdapterParams p) {
  __shared__ float h[kMostRank];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x;
  pdl_wait();
  int id = p.ids[t];
  if (id >= p.count) {
    if (threadIdx.x == 0) atomicOr(p.err, DEVERR_INDEX);
    id = -1;
  }
  if (id >= 0) {
    const __nv_bfloat16* x = p.x + t * p.ldx;
    for (int j = warp; j < p.r; j += kThreads / 32) {
      const __nv_bfloat16* a = p.a + id * p.stride_a + int64_t(j) * p.K;
      float sum = 0.0f;
      for (int k = lane; k < p.K; k += 32) sum = fmaf(__bfloat162float(a[k]), __bfloat162float(x[k]), sum);
#pragma unroll
      for (int m = 16; m; m >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, m);
      if (lane == 0) h[j] = sum * (p.scales ? p.scales[id] : 1.0f);
    }
  }
  __syncthreads();
  for (int n = threadIdx.x; n < p.N; n += kThreads) {
    float sum = __bfloat162float(p.y[t * p.ldy + n]);
    if (id >= 0) {
      const __nv_bfloat16* b = p.b + id * p.stride_b + int64_t(n) * p.r;
      float add = 0.0f;
      for (int j = 0; j < p.r; ++j) add = fmaf(__bfloat162float(b[j]), h[j], add);
      sum += add;
    }
    p.out[t * p.ldo + n] = __float2bfloat16(sum);
  }
  pdl_trigger();
}

template <int MT, int NT>
cudaError_t launch_few(const AdapterParams& p, const DeviceInfo& dev, cudaStream_t s) {
  using C = FewCfg<MT, NT>;
  // Each adapter's last item may be partly filled; rows without an adapter count as one more.
  const int items = std::min<int64_t>(p.T, p.T / C::R + std::min<int64_t>(p.T, int64_t(p.count) + 1));
  return launch_pdl_smem<add_adapters_few_kernel<MT, NT>, kCluster>(dev, dim3(items * kCluster), dim3(kThreads), C::SMEM, s, p);
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
  if (T > kFewRows)
    e = launch_pdl(add_adapters_kernel, dim3(static_cast<unsigned>(T)), dim3(kThreads), 0, s, p);
  else if (r <= 16)
    e = launch_few<1, 1>(p, *dev, s);
  else if (r <= 32)
    e = launch_few<2, 1>(p, *dev, s);
  else if (r <= 64)
    e = launch_few<4, 1>(p, *dev, s);
  else
    e = launch_few<8, 1>(p, *dev, s);
  return e == cudaSuccess ? SP24_OK : SP24_ERR_CUDA;
}
