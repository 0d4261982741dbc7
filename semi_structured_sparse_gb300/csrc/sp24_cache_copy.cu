// sp24_cache_copy.cu -- sp24_cache_copy: keys and values of tokens from places
// of one paged cache to places of another (or of the same), quantised to e4m3 or
// read back from it on the way.
//
//   dst = round(x),  x = src (bf16) or code * scale[head] (e4m3);
//   round: to bf16, or e4m3_rn_satfinite(x / scale[head])
//
// Bound by memory: every byte of a token's rows is read and written once, 16 bytes
// per thread and access, a thread's keys and values on their way together.  A CTA
// takes 8 or 16 tokens of a few heads, whose rows a cache keeps together; many
// small CTAs keep more bytes in flight than fewer with more each (16000 tokens to e4m3, at the
// time: one unit per thread 19.6 us, two 22.8, four 31.6).
//
// Measured (GB300): 16000 tokens of 8 heads of 128 to e4m3 17.2 us, 5.7 TB/s (86 % of
// the measured copy rate), bf16 to bf16 21.1 us, 6.2 TB/s (93 %), e4m3 to e4m3 14.2 us;
// 50001 tokens of 4 heads of 64 back from e4m3 15.0 us, 5.2 TB/s (77 %); 64 tokens 1.5 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include "sp24_attn.cuh"
#include "sp24_ptx.cuh"

namespace sp24 {
namespace {

constexpr int kThreads = 256;
constexpr int kMostHeads = 65535;  // CTAs along a grid's y axis, at a head each
template <int D>
constexpr int kTokens = D / 8;  // per CTA (heads of 64, 50001 tokens read back: 15.0 us with 8, 16.7 with 16)

struct CopyParams {
  CacheView src, dst;
  const int64_t* src_slots;
  const int64_t* dst_slots;
  int64_t T, src_total, dst_total;  // slots of the caches
  int heads;
  unsigned int* err;
};

// x / d, correctly rounded, in three operations: with r the correctly rounded
// reciprocal of d and q = RN(x r), RN(q + RN(x - q d) r) is the correctly rounded
// quotient, unless d's significand is all ones (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990), as long as nothing
// leaves the range: quotients too small for that are far below e4m3's smallest
// step, and other divisors and larger values are divided plainly.  (16000 tokens of
// 8 heads of 128 to e4m3: 19.6 us with divisions throughout.)
template <int N>
__device__ __forceinline__ void divide(float2 (&f)[N], float d) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, fmaxf(fabsf(f[i].x), fabsf(f[i].y)));  // (not a number: stays one below)
  const uint32_t bits = __float_as_uint(d);
  if (d > 1e-25f && d < 1e25f && top < 1e10f && (bits & 0x7FFFFFu) != 0x7FFFFFu) {
    const float r = __frcp_rn(d);
    const float2 rr = make_float2(r, r), less = make_float2(-r, -r), dd = make_float2(d, d);
#pragma unroll
    for (int i = 0; i < N; ++i) {  // (with these signs -0 stays -0)
      const float2 q = __fmul2_rn(f[i], rr);
      f[i] = __ffma2_rn(__ffma2_rn(q, dd, make_float2(-f[i].x, -f[i].y)), less, q);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = make_float2(__fdiv_rn(f[i].x, d), __fdiv_rn(f[i].y, d));
  }
}

// A thread has 8 or 16 values of a head of a token, of the keys and of the values.
template <int D, bool FROM8, bool TO8>
__global__ void __launch_bounds__(kThreads) cache_copy_kernel(const __grid_constant__ CopyParams p) {
  constexpr int UNIT = FROM8 || TO8 ? 16 : 8;           // values
  constexpr int LPR = D / UNIT;                         // threads per row
  constexpr int HPP = kThreads / LPR / kTokens<D>;         // heads per CTA
  constexpr int IN = UNIT * (FROM8 ? 1 : 2) / 16;       // 16-byte pieces of a unit
  static_assert(HPP >= 1, "");
  const int piece = threadIdx.x % LPR, token = threadIdx.x / LPR % kTokens<D>;
  const int h = blockIdx.y * HPP + threadIdx.x / LPR / kTokens<D>;
  const int64_t t = int64_t(blockIdx.x) * kTokens<D> + token;
  pdl_wait();
  int64_t from = -1, to = -1;
  if (t < p.T && h < p.heads) from = p.src_slots[t], to = p.dst_slots[t];
  if (from >= p.src_total || to >= p.dst_total) {
    if (piece == 0) atomicOr(p.err, DEVERR_INDEX);
    from = -1;
  }
  if (from >= 0 && to >= 0) {
    const int64_t at = (from >> p.src.page_shift) * p.src.page_stride +
                       (from & ((1 << p.src.page_shift) - 1)) * p.src.token_stride + piece * (UNIT * (FROM8 ? 1 : 2));
    const int64_t dt = (to >> p.dst.page_shift) * p.dst.page_stride +
                       (to & ((1 << p.dst.page_shift) - 1)) * p.dst.token_stride + piece * (UNIT * (TO8 ? 1 : 2));
    uint4 v[2][IN];
#pragma unroll
    for (int i = 0; i < IN; ++i) {
      v[0][i] = *reinterpret_cast<const uint4*>(p.src.k + at + h * p.src.head_stride + 16 * i);
      v[1][i] = *reinterpret_cast<const uint4*>(p.src.v + at + h * p.src.head_stride + 16 * i);
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint8_t* out = const_cast<uint8_t*>(x ? p.dst.v : p.dst.k) + dt + h * p.dst.head_stride;
      if (!FROM8 && !TO8) {
        *reinterpret_cast<uint4*>(out) = v[x][0];
        continue;
      }
      float2 f[UNIT / 2];
      const uint32_t* w = reinterpret_cast<const uint32_t*>(v[x]);
      if (FROM8) {
        const float scale = (x ? p.src.v_scale : p.src.k_scale)[h];
#pragma unroll
        for (int i = 0; i < UNIT / 2; ++i) {
          const uint32_t two = e4m3x2_f16x2(w[i / 2] >> (16 * (i & 1)));
          f[i] = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2*>(&two)), make_float2(scale, scale));
        }
      } else {
#pragma unroll
        for (int i = 0; i < UNIT / 2; ++i)
          f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
      }
      if (TO8) {
        divide(f, (x ? p.dst.v_scale : p.dst.k_scale)[h]);
        uint32_t c[UNIT / 4];
#pragma unroll
        for (int i = 0; i < UNIT / 4; ++i)
          c[i] = __nv_cvt_float2_to_fp8x2(f[2 * i], __NV_SATFINITE, __NV_E4M3) |
                 static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(f[2 * i + 1], __NV_SATFINITE, __NV_E4M3)) << 16;
        *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(c);
      } else {
#pragma unroll
        for (int i = 0; i < UNIT / 8; ++i) {
          const float2* g = f + 4 * i;
          *reinterpret_cast<uint4*>(out + 16 * i) = make_uint4(bf16x2_rn(g[0].x, g[0].y), bf16x2_rn(g[1].x, g[1].y),
                                                               bf16x2_rn(g[2].x, g[2].y), bf16x2_rn(g[3].x, g[3].y));
        }
      }
    }
  }
  pdl_trigger();
}

template <int D, bool FROM8, bool TO8>
cudaError_t launch(const CopyParams& p, cudaStream_t s) {
  constexpr int HPP = kThreads / (D / (FROM8 || TO8 ? 16 : 8)) / kTokens<D>;
  const unsigned x = static_cast<unsigned>((p.T + kTokens<D> - 1) / kTokens<D>);
  return launch_pdl(cache_copy_kernel<D, FROM8, TO8>, dim3(x, (p.heads + HPP - 1) / HPP), dim3(kThreads), 0, s, p);
}
template <int D>
cudaError_t launch(const CopyParams& p, bool from8, bool to8, cudaStream_t s) {
  if (from8) return to8 ? launch<D, true, true>(p, s) : launch<D, true, false>(p, s);
  return to8 ? launch<D, false, true>(p, s) : launch<D, false, false>(p, s);
}

}  // namespace
}  // namespace sp24

extern "C" sp24_status sp24_cache_copy(const sp24_kv_cache* src, const int64_t* src_slots, const sp24_kv_cache* dst,
                                       const int64_t* dst_slots, int64_t T, void* stream) {
  using namespace sp24;
  CopyParams p = {};
  if (sp24_status st = check_cache(src, &p.src)) return st;
  if (sp24_status st = check_cache(dst, &p.dst)) return st;
  if (T < 0 || T > INT32_MAX || src->heads != dst->heads || src->head_dim != dst->head_dim || src->heads > kMostHeads)
    return SP24_ERR_INVALID_ARG;
  if (T > 0) {
    if (!src_slots || !dst_slots) return SP24_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(src_slots) | reinterpret_cast<uintptr_t>(dst_slots)) & 7u) return SP24_ERR_ALIGNMENT;
  }
  const DeviceInfo* dev = nullptr;
  if (sp24_status st = current_device(&dev)) return st;
  if (T == 0) return SP24_OK;
  p.src_slots = src_slots;
  p.dst_slots = dst_slots;
  p.T = T;
  p.src_total = int64_t(p.src.num_pages) << p.src.page_shift;
  p.dst_total = int64_t(p.dst.num_pages) << p.dst.page_shift;
  p.heads = src->heads;
  p.err = dev->err_word;
  const bool from8 = src->dtype == SP24_E4M3, to8 = dst->dtype == SP24_E4M3;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t r = src->head_dim == 128 ? launch<128>(p, from8, to8, s) : launch<64>(p, from8, to8, s);
  return r == cudaSuccess ? SP24_OK : SP24_ERR_CUDA;
}
