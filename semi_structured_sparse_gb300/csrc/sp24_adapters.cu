// sp24_adapters.cu -- sp24_add_adapters: to every row of a projection's output
// the product of its request's low-rank adapter,
//
//   out[t] = y[t] + scale_i B_i (A_i x[t]),  i = ids[t]
//
// Bound by memory: rows and the adapters in use are read once, and 2 r
// operations per value of x and y are few.
#include <cuda_bf16.h>
#include <cmath>
#include "sp24_internal.cuh"
#include "sp24_ptx.cuh"

namespace sp24 {
namespace {

constexpr int kThreads = 256;
constexpr int kMostRank = 128;

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
  const cudaError_t e = launch_pdl(add_adapters_kernel, dim3(static_cast<unsigned>(T)), dim3(kThreads), 0,
                                   static_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? SP24_OK : SP24_ERR_CUDA;
}
