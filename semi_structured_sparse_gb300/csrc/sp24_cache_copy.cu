// sp24_cache_copy.cu -- sp24_cache_copy: keys and values of tokens from places
// of one paged cache to places of another (or of the same), quantised to e4m3 or
// read back from it on the way.
//
//   dst = round(x),  x = src (bf16) or code * scale[head] (e4m3);
//   round: to bf16, or e4m3_rn_satfinite(x / scale[head])
//
// Bound by memory: every byte of a token's rows is read and written once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include "sp24_attn.cuh"
#include "sp24_ptx.cuh"

namespace sp24 {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 16;  // per CTA

struct CopyParams {
  CacheView src, dst;
  const int64_t* src_slots;
  const int64_t* dst_slots;
  int64_t T, src_total, dst_total;  // slots of the caches
  int heads;
  unsigned int* err;
};

// U units (16 or 32 bytes of a head of a token) per thread, of keys and of values.
template <int D, bool FROM8, bool TO8, int U>
__global__ void __launch_bounds__(kThreads) cache_copy_kernel(const __grid_constant__ CopyParams p) {
  constexpr int UNIT = FROM8 || TO8 ? 16 : 8;           // values
  constexpr int LPR = D / UNIT;                         // threads per row
  constexpr int HPP = kThreads / LPR / kTokens;         // heads per pass of the CTA
  constexpr int IN = UNIT * (FROM8 ? 1 : 2) / 16;       // 16-byte pieces of a unit
  const int piece = threadIdx.x % LPR, token = threadIdx.x / LPR % kTokens;
  const int h0 = blockIdx.y * (U * HPP) + threadIdx.x / LPR / kTokens;
  const int64_t t = int64_t(blockIdx.x) * kTokens + token;
  pdl_wait();
  int64_t from = -1, to = -1;
  if (t < p.T) from = p.src_slots[t], to = p.dst_slots[t];
  if (from >= p.src_total || to >= p.dst_total) {
    if (piece == 0) atomicOr(p.err, DEVERR_INDEX);
    from = -1;
  }
  if (from >= 0 && to >= 0) {
    const int64_t at = (from >> p.src.page_shift) * p.src.page_stride +
                       (from & ((1 << p.src.page_shift) - 1)) * p.src.token_stride + piece * (UNIT * (FROM8 ? 1 : 2));
    const int64_t dt = (to >> p.dst.page_shift) * p.dst.page_stride +
                       (to & ((1 << p.dst.page_shift) - 1)) * p.dst.token_stride + piece * (UNIT * (TO8 ? 1 : 2));
    uint4 v[2][U][IN];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * HPP;
      if (h < p.heads) {
#pragma unroll
        for (int i = 0; i < IN; ++i) {
          v[0][u][i] = *reinterpret_cast<const uint4*>(p.src.k + at + h * p.src.head_stride + 16 * i);
          v[1][u][i] = *reinterpret_cast<const uint4*>(p.src.v + at + h * p.src.head_stride + 16 * i);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = h0 + u * HPP;
      if (h < p.heads) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint8_t* out = const_cast<uint8_t*>(x ? p.dst.v : p.dst.k) + dt + h * p.dst.head_stride;
          if (!FROM8 && !TO8) {
            *reinterpret_cast<uint4*>(out) = v[x][u][0];
            continue;
          }
          float f[UNIT];
          const uint32_t* w = reinterpret_cast<const uint32_t*>(v[x][u]);
          if (FROM8) {
            const float scale = (x ? p.src.v_scale : p.src.k_scale)[h];
#pragma unroll
            for (int i = 0; i < UNIT / 2; ++i) {
              const uint32_t two = e4m3x2_f16x2(w[i / 2] >> (16 * (i & 1)));
              const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&two));
              f[2 * i] = y.x * scale, f[2 * i + 1] = y.y * scale;
            }
          } else {
#pragma unroll
            for (int i = 0; i < UNIT / 2; ++i) {
              f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
          }
          if (TO8) {
            const float scale = (x ? p.dst.v_scale : p.dst.k_scale)[h];
            uint32_t c[UNIT / 4];
#pragma unroll
            for (int i = 0; i < UNIT / 4; ++i) {
              const float* g = f + 4 * i;
              const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(g[0], scale), __fdiv_rn(g[1], scale)),
                                                           __NV_SATFINITE, __NV_E4M3);
              const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(g[2], scale), __fdiv_rn(g[3], scale)),
                                                           __NV_SATFINITE, __NV_E4M3);
              c[i] = lo | (hi << 16);
            }
            *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(c);
          } else {
#pragma unroll
            for (int i = 0; i < UNIT / 8; ++i) {
              const float* g = f + 8 * i;
              *reinterpret_cast<uint4*>(out + 16 * i) = make_uint4(bf16x2_rn(g[0], g[1]), bf16x2_rn(g[2], g[3]),
                                                                   bf16x2_rn(g[4], g[5]), bf16x2_rn(g[6], g[7]));
            }
          }
        }
      }
    }
  }
  pdl_trigger();
}

template <int D, bool FROM8, bool TO8>
cudaError_t launch(const CopyParams& p, cudaStream_t s) {
  constexpr int HPP = kThreads / (D / (FROM8 || TO8 ? 16 : 8)) / kTokens;
  const unsigned x = static_cast<unsigned>((p.T + kTokens - 1) / kTokens);
  return launch_pdl(cache_copy_kernel<D, FROM8, TO8, 1>, dim3(x, (p.heads + HPP - 1) / HPP), dim3(kThreads), 0, s, p);
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
  if (T < 0 || T > INT32_MAX || src->heads != dst->heads || src->head_dim != dst->head_dim || src->heads > (1 << 16))
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
