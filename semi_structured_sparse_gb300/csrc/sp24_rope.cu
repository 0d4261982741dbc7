// sp24_rope.cu -- sp24_qk_norm_rope: per-head RMS norm and position rotation
// of queries and keys, keys and values appended to the paged cache, in one
// pass over the QKV projection's rows.
//
//   y = x / sqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos - b sin, b cos + a sin)
//
// Bound by memory: 2 bytes read and 2 (1 in an e4m3 cache) written per
// element.  A row's heads are independent, and the cosines and sines of its
// position are the same for all of them, so a warp stays with one token: lane
// l holds the cosines and sines of its 8 elements in registers and walks the
// token's heads, 32 / (D / 8) of them at a time, one 16-byte load and store
// per lane and head.  A rotated pair's other half comes from another lane by
// shuffle (half-split pairs) or sits in the same lane (neighbouring pairs).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include "sp24_attn.cuh"
#include "sp24_ptx.cuh"

namespace sp24 {
namespace {

constexpr int kWarps = 4;

struct RopeParams {
  const __nv_bfloat16* qkv;
  int64_t ldqkv;
  const __nv_bfloat16* q_weight;
  const __nv_bfloat16* k_weight;
  float eps;
  const float* cos_sin;
  int64_t max_pos;
  int rot;
  const int32_t* positions;
  const int64_t* slots;
  __nv_bfloat16* q_out;
  int64_t ldq;
  CacheView cache;
  int64_t num_slots;
  int q_heads, kv_heads;
  unsigned int* err;
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(bf16x2_rn(x[0], x[1]), bf16x2_rn(x[2], x[3]), bf16x2_rn(x[4], x[5]), bf16x2_rn(x[6], x[7]));
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// U head groups per step: their loads are issued together.
template <int D, bool E4M3, bool INTERLEAVED, int U>
__global__ void __launch_bounds__(kWarps * 32) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LPH = D / 8;           // lanes per head
  constexpr int HPW = 32 / LPH;        // heads per warp and step
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x;
  const int e0 = (lane % LPH) * 8;     // this lane's first element within a head
  const int heads = p.q_heads + 2 * p.kv_heads;
  const int groups = (heads + HPW - 1) / HPW;
  const int gstep = kWarps * gridDim.y;
  const __nv_bfloat16* row = p.qkv + t * p.ldqkv + e0;
  pdl_wait();

  const int64_t slot = p.slots[t];
  if (slot >= p.num_slots && lane == 0) atomicOr(p.err, DEVERR_INDEX);
  const bool store = slot >= 0 && slot < p.num_slots;
  const int64_t page = slot >> p.cache.page_shift;
  const int64_t place = slot & ((1 << p.cache.page_shift) - 1);
  const int64_t at = page * p.cache.page_stride + place * p.cache.token_stride + e0 * (E4M3 ? 1 : 2);

  // This lane's cosines and sines.  Elements past rot keep (1, 0).  half-split:
  // element i < rot/2 has the partner i + rot/2 and a sine of -sin, the others
  // the partner i - rot/2 and +sin.  Neighbouring: c[j], s[j] for pair j.
  float c[8], s[8];
  int partner = lane;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] = 1.0f;
    s[i] = 0.0f;
  }
  if (p.rot > 0) {
    const int64_t pos = p.positions[t];
    if (pos < 0 || pos >= p.max_pos) {  // the whole CTA works on this token
      if (lane == 0) atomicOr(p.err, DEVERR_INDEX);
      pdl_trigger();
      return;
    }
    const float* table = p.cos_sin + pos * p.rot;
    const int half = p.rot / 2;
    if (e0 < p.rot) {
      if (INTERLEAVED) {
        const float4 cv = *reinterpret_cast<const float4*>(table + e0 / 2);
        const float4 sv = *reinterpret_cast<const float4*>(table + half + e0 / 2);
        c[0] = cv.x, c[1] = cv.y, c[2] = cv.z, c[3] = cv.w;
        s[0] = sv.x, s[1] = sv.y, s[2] = sv.z, s[3] = sv.w;
      } else {
        const bool first = e0 < half;
        const int i0 = first ? e0 : e0 - half;
        partner = first ? lane + half / 8 : lane - half / 8;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 cv = *reinterpret_cast<const float4*>(table + i0 + i);
          const float4 sv = *reinterpret_cast<const float4*>(table + half + i0 + i);
          c[i] = cv.x, c[i + 1] = cv.y, c[i + 2] = cv.z, c[i + 3] = cv.w;
          s[i] = first ? -sv.x : sv.x, s[i + 1] = first ? -sv.y : sv.y;
          s[i + 2] = first ? -sv.z : sv.z, s[i + 3] = first ? -sv.w : sv.w;
        }
      }
    }
  }

  for (int g0 = blockIdx.y * kWarps + warp; g0 < groups; g0 += gstep * U) {
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = (g0 + u * gstep) * HPW + lane / LPH;
      raw[u] = h < heads ? *reinterpret_cast<const uint4*>(row + int64_t(h) * D) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if ((g0 + u * gstep) * HPW >= heads) break;  // uniform over the warp
      const int h = (g0 + u * gstep) * HPW + lane / LPH;
      float x[8];
      unpack8(raw[u], x);
      const bool turned = h < p.q_heads + p.kv_heads;  // queries and keys
      if (p.q_weight != nullptr) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int m = 1; m < LPH; m <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, m);
        if (turned) {
          const float r = rsqrtf(fmaf(ss, 1.0f / D, p.eps));
          float w[8];
          unpack8(*reinterpret_cast<const uint4*>((h < p.q_heads ? p.q_weight : p.k_weight) + e0), w);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
        }
      }
      if (INTERLEAVED) {
        if (turned && e0 < p.rot) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * c[i] - b * s[i];
            x[2 * i + 1] = b * c[i] + a * s[i];
          }
        }
      } else if (p.rot > 0) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xFFFFFFFFu, x[i], partner);
        if (turned && e0 < p.rot) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * c[i] + y[i] * s[i];
        }
      }
      if (h < p.q_heads) {
        *reinterpret_cast<uint4*>(p.q_out + t * p.ldq + int64_t(h) * D + e0) = pack8(x);
      } else if (h < heads && store) {
        const bool key = h < p.q_heads + p.kv_heads;
        const int hk = h - p.q_heads - (key ? 0 : p.kv_heads);
        uint8_t* dst = const_cast<uint8_t*>(key ? p.cache.k : p.cache.v) + at + hk * p.cache.head_stride;
        if (E4M3) {
          const float d = (key ? p.cache.k_scale : p.cache.v_scale)[hk];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = __fdiv_rn(x[i], d);
          *reinterpret_cast<uint2*>(dst) = make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
        } else {
          *reinterpret_cast<uint4*>(dst) = pack8(x);
        }
      }
    }
  }
  pdl_trigger();
}

template <int D, bool E4M3, bool INTERLEAVED>
cudaError_t launch(const RopeParams& p, int64_t T, const DeviceInfo& dev, cudaStream_t s) {
  const int groups = (p.q_heads + 2 * p.kv_heads + 32 / (D / 8) - 1) / (32 / (D / 8));
  // Few tokens: a warp per head group, so that one row's latency is one load's.
  // Many: a CTA per token, whose warps load 3 groups at a time.
  const bool few = T < 4 * dev.sm_count;
  const dim3 grid(static_cast<unsigned>(T), few ? static_cast<unsigned>((groups + kWarps - 1) / kWarps) : 1u);
  if (few) return launch_pdl(qk_norm_rope_kernel<D, E4M3, INTERLEAVED, 1>, grid, dim3(kWarps * 32), 0, s, p);
  return launch_pdl(qk_norm_rope_kernel<D, E4M3, INTERLEAVED, 3>, grid, dim3(kWarps * 32), 0, s, p);
}

}  // namespace
}  // namespace sp24

extern "C" sp24_status sp24_qk_norm_rope(const void* qkv, int64_t T, int64_t ldqkv, int q_heads, const void* q_weight,
                                         const void* k_weight, float eps, const float* cos_sin, int64_t max_pos,
                                         int rot, int interleaved, const int32_t* positions, const int64_t* slots,
                                         void* q_out, int64_t ldq, const sp24_kv_cache* cache, void* stream) {
  using namespace sp24;
  RopeParams p;
  if (T < 0 || T > INT32_MAX) return SP24_ERR_INVALID_ARG;
  if (sp24_status st = check_cache(cache, &p.cache)) return st;
  const int D = cache->head_dim;
  if (q_heads < 1 || q_heads > (1 << 20) || cache->heads > (1 << 20)) return SP24_ERR_INVALID_ARG;
  if (rot < 0 || rot > D) return SP24_ERR_INVALID_ARG;
  if (rot % 16 != 0) return SP24_ERR_UNSUPPORTED;
  if ((q_weight != nullptr) != (k_weight != nullptr)) return SP24_ERR_INVALID_ARG;
  if (q_weight && !(eps >= 0.0f && std::isfinite(eps))) return SP24_ERR_INVALID_ARG;
  if (T > 0) {
    if (!qkv || !q_out || !slots || (rot > 0 && (!cos_sin || !positions || max_pos < 1))) return SP24_ERR_INVALID_ARG;
    if (ldqkv < (int64_t(q_heads) + 2 * cache->heads) * D || ldq < int64_t(q_heads) * D) return SP24_ERR_INVALID_ARG;
    if (!aligned16(qkv) || !aligned16(q_out) || ldqkv % 8 || ldq % 8) return SP24_ERR_ALIGNMENT;
    if (!aligned16(q_weight) || !aligned16(k_weight) || (rot > 0 && !aligned16(cos_sin))) return SP24_ERR_ALIGNMENT;
    if ((reinterpret_cast<uintptr_t>(slots) & 7u) || (reinterpret_cast<uintptr_t>(positions) & 3u))
      return SP24_ERR_ALIGNMENT;
  }
  const DeviceInfo* dev = nullptr;
  if (sp24_status st = current_device(&dev)) return st;
  if (T == 0) return SP24_OK;
  p.qkv = static_cast<const __nv_bfloat16*>(qkv);
  p.ldqkv = ldqkv;
  p.q_weight = static_cast<const __nv_bfloat16*>(q_weight);
  p.k_weight = static_cast<const __nv_bfloat16*>(k_weight);
  p.eps = eps;
  p.cos_sin = cos_sin;
  p.max_pos = max_pos;
  p.rot = rot;
  p.positions = positions;
  p.slots = slots;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.ldq = ldq;
  p.num_slots = int64_t(p.cache.num_pages) << p.cache.page_shift;
  p.q_heads = q_heads;
  p.kv_heads = cache->heads;
  p.err = dev->err_word;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool e4m3 = cache->dtype == SP24_E4M3;
  cudaError_t r;
  if (D == 128)
    r = e4m3 ? (interleaved ? launch<128, true, true>(p, T, *dev, s) : launch<128, true, false>(p, T, *dev, s))
             : (interleaved ? launch<128, false, true>(p, T, *dev, s) : launch<128, false, false>(p, T, *dev, s));
  else
    r = e4m3 ? (interleaved ? launch<64, true, true>(p, T, *dev, s) : launch<64, true, false>(p, T, *dev, s))
             : (interleaved ? launch<64, false, true>(p, T, *dev, s) : launch<64, false, false>(p, T, *dev, s));
  return r == cudaSuccess ? SP24_OK : SP24_ERR_CUDA;
}
