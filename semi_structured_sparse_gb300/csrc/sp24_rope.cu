// sp24_rope.cu -- sp24_qk_norm_rope: per-head RMS norm and position rotation
// of queries and keys, keys and values appended to the paged cache, in one
// pass over the QKV projection's rows.
//
//   y = x / sqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos - b sin, b cos + a sin)
//
// Bound by memory: 2 bytes read and 2 (1 in an e4m3 cache) written per
// element.  A row's heads are independent, and the cosines and sines of its
// position are the same for all of them, so a warp stays with one token and
// walks its heads, 32 / (D / 8) of them at a time.  Of each head a lane has 4
// values and, for half-split pairs, the 4 values that they are rotated with: a
// rotation needs no other lane, and 4 cosines and 4 sines per lane do for all
// heads.  All of a warp's loads are issued before the position is known.
//
// Measured (GB300): 8192 tokens of 32 + 8 + 8 heads of 128 33.7 us, 6.1 TB/s
// (90 % of the measured copy rate); 3000 of 28 + 4 + 4 of 64 7.6 us; one token
// 1.6 us.  What it took at 8192 tokens: one 16-byte piece per lane with the
// partners fetched by shuffles, 49.7 us, 155 instructions per step; rotated
// pairs within a lane and packed fp32 arithmetic, 40.8; a warp's heads all of
// one kind and at fixed distances (no selects, no address arithmetic), 35.5; two
// warps with 6 groups' loads each instead of four with 3, 33.7.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include "sp24_attn.cuh"
#include "sp24_ptx.cuh"

namespace sp24 {
namespace {

constexpr int kWarps = 2;
constexpr int kMany = 6;  // head groups whose loads a warp issues together in long calls

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

// Four bf16 values as two pairs of fp32.
__device__ __forceinline__ void unpack4(const uint2& v, float2 (&x)[2]) {
  x[0] = make_float2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u));
  x[1] = make_float2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
}
__device__ __forceinline__ uint2 pack4(const float2 (&x)[2]) {
  return make_uint2(bf16x2_rn(x[0].x, x[0].y), bf16x2_rn(x[1].x, x[1].y));
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// U head groups at a time: their loads are issued together.  FEW: the token's
// groups are spread over gridDim.y CTAs, one per warp.  EVEN: no group holds heads
// of two kinds (queries, keys, values), so that a warp's lanes all do the same.
template <int D, bool E4M3, bool INTERLEAVED, int U, bool FEW, bool EVEN>
__global__ void __launch_bounds__(kWarps * 32) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LPH = D / 8;           // lanes per head
  constexpr int HPW = 32 / LPH;        // heads per group
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x;
  const int heads = p.q_heads + 2 * p.kv_heads, turned = p.q_heads + p.kv_heads;  // queries and keys
  // This lane's elements of a head: four from ea, four from eb.  Half-split
  // pairs: (ea + i, eb + i), for the first rot / 8 lanes; neighbours otherwise.
  const int l = lane % LPH, pairs = INTERLEAVED ? 0 : p.rot / 8;
  const int ea = l < pairs ? 4 * l : 8 * l, eb = l < pairs ? p.rot / 2 + 4 * l : 8 * l + 4;
  const bool rotates = INTERLEAVED ? ea < p.rot : l < pairs;
  const int sub = lane / LPH;
  pdl_wait();

  // Loads of the groups at g0, g0 + kWarps, ...; a lane past the last head reads that head.
  int hfirst = (FEW ? static_cast<int>(blockIdx.y) * kWarps + warp : warp) * HPW;  // uniform over the warp
  const __nv_bfloat16* row = p.qkv + t * p.ldqkv;
  uint2 ra[U], rb[U];
  auto load = [&]() {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = min(hfirst + u * (kWarps * HPW) + sub, heads - 1);
      ra[u] = *reinterpret_cast<const uint2*>(row + h * D + ea);
      rb[u] = *reinterpret_cast<const uint2*>(row + h * D + eb);
    }
  };
  load();

  const bool norm = p.q_weight != nullptr;
  float2 wq[4], wk[4];
  if (norm) {
    auto weights = [&](const __nv_bfloat16* w, float2 (&x)[4]) {
      float2 y[2];
      unpack4(*reinterpret_cast<const uint2*>(w + ea), y);
      x[0] = y[0], x[1] = y[1];
      unpack4(*reinterpret_cast<const uint2*>(w + eb), y);
      x[2] = y[0], x[3] = y[1];
    };
    weights(p.q_weight, wq);
    weights(p.k_weight, wk);
  }
  const int64_t slot = p.slots[t];
  const int64_t pos = p.rot > 0 ? p.positions[t] : 0;
  if (slot >= p.num_slots && threadIdx.x == 0) atomicOr(p.err, DEVERR_INDEX);
  const bool store = slot >= 0 && slot < p.num_slots;
  const int64_t at = (slot >> p.cache.page_shift) * p.cache.page_stride +
                     (slot & ((1 << p.cache.page_shift) - 1)) * p.cache.token_stride;
  if (p.rot > 0 && (pos < 0 || pos >= p.max_pos)) {  // the whole CTA works on this token
    if (threadIdx.x == 0) atomicOr(p.err, DEVERR_INDEX);
    pdl_trigger();
    return;
  }
  // Half-split: pair i turns by (c[i], s[i]), i < 4.  Neighbours: the pairs of
  // ea turn by (c0.x, s0.x) and (c0.y, s0.y), those of eb by (c1, s1).
  float2 c[2], s[2], ns[2];
  c[0] = c[1] = make_float2(1.0f, 1.0f);
  s[0] = s[1] = make_float2(0.0f, 0.0f);
  if (rotates) {
    const float* table = p.cos_sin + pos * p.rot + (INTERLEAVED ? ea / 2 : ea);
    const float4 cv = *reinterpret_cast<const float4*>(table);
    const float4 sv = *reinterpret_cast<const float4*>(table + p.rot / 2);
    c[0] = make_float2(cv.x, cv.y), c[1] = make_float2(cv.z, cv.w);
    s[0] = make_float2(sv.x, sv.y), s[1] = make_float2(sv.z, sv.w);
  }
  ns[0] = make_float2(-s[0].x, -s[0].y), ns[1] = make_float2(-s[1].x, -s[1].y);
  __nv_bfloat16* const q_row = p.q_out + t * p.ldq;

  // Norm (weights w) and rotation of one head's values.
  auto turn = [&](float2 (&a)[2], float2 (&b)[2], const float2 (&w)[4]) {
    if (norm) {
      float2 q = __fmul2_rn(a[0], a[0]);
      q = __ffma2_rn(a[1], a[1], q);
      q = __ffma2_rn(b[0], b[0], q);
      q = __ffma2_rn(b[1], b[1], q);
      float ss = q.x + q.y;
#pragma unroll
      for (int m = 1; m < LPH; m <<= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, m);
      const float r = rsqrtf(fmaf(ss, 1.0f / D, p.eps));
      const float2 rr = make_float2(r, r);
      a[0] = __fmul2_rn(a[0], __fmul2_rn(w[0], rr)), a[1] = __fmul2_rn(a[1], __fmul2_rn(w[1], rr));
      b[0] = __fmul2_rn(b[0], __fmul2_rn(w[2], rr)), b[1] = __fmul2_rn(b[1], __fmul2_rn(w[3], rr));
    }
    if (!rotates) return;
    if (INTERLEAVED) {
      auto pair = [](float2 x, float cc, float ss) {
        return make_float2(x.x * cc - x.y * ss, x.y * cc + x.x * ss);
      };
      a[0] = pair(a[0], c[0].x, s[0].x), a[1] = pair(a[1], c[0].y, s[0].y);
      b[0] = pair(b[0], c[1].x, s[1].x), b[1] = pair(b[1], c[1].y, s[1].y);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 x = a[i], y = b[i];
        a[i] = __ffma2_rn(y, ns[i], __fmul2_rn(x, c[i]));
        b[i] = __ffma2_rn(x, s[i], __fmul2_rn(y, c[i]));
      }
    }
  };
  auto put_query = [&](int h, const float2 (&a)[2], const float2 (&b)[2]) {
    *reinterpret_cast<uint2*>(q_row + h * D + ea) = pack4(a);
    *reinterpret_cast<uint2*>(q_row + h * D + eb) = pack4(b);
  };
  auto put_cache = [&](const uint8_t* base, const float* scale, int hk, const float2 (&a)[2], const float2 (&b)[2]) {
    if (!store) return;
    uint8_t* dst = const_cast<uint8_t*>(base) + at + hk * p.cache.head_stride;
    if (E4M3) {
      const float d = scale[hk];
      *reinterpret_cast<uint32_t*>(dst + ea) =
          e4m3x4(__fdiv_rn(a[0].x, d), __fdiv_rn(a[0].y, d), __fdiv_rn(a[1].x, d), __fdiv_rn(a[1].y, d));
      *reinterpret_cast<uint32_t*>(dst + eb) =
          e4m3x4(__fdiv_rn(b[0].x, d), __fdiv_rn(b[0].y, d), __fdiv_rn(b[1].x, d), __fdiv_rn(b[1].y, d));
    } else {
      *reinterpret_cast<uint2*>(dst + 2 * ea) = pack4(a);
      *reinterpret_cast<uint2*>(dst + 2 * eb) = pack4(b);
    }
  };

  while (true) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int hu = hfirst + u * (kWarps * HPW), h = hu + sub;
      if (hu >= heads) break;  // uniform
      float2 a[2], b[2];
      unpack4(ra[u], a);
      unpack4(rb[u], b);
      if (EVEN) {
        if (hu < p.q_heads) {
          turn(a, b, wq);
          put_query(h, a, b);
        } else if (hu < turned) {
          turn(a, b, wk);
          put_cache(p.cache.k, p.cache.k_scale, h - p.q_heads, a, b);
        } else {
          put_cache(p.cache.v, p.cache.v_scale, h - turned, a, b);
        }
      } else {
        const bool query = h < p.q_heads, key = !query && h < turned;
        const float2 va[2] = {a[0], a[1]}, vb[2] = {b[0], b[1]};
        float2 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = query ? wq[i] : wk[i];
        turn(a, b, w);
        if (query)
          put_query(h, a, b);
        else if (key)
          put_cache(p.cache.k, p.cache.k_scale, h - p.q_heads, a, b);
        else if (h < heads)
          put_cache(p.cache.v, p.cache.v_scale, h - turned, va, vb);
      }
    }
    if (FEW) break;
    hfirst += U * kWarps * HPW;
    if (hfirst >= heads) break;  // uniform
    load();
  }
  pdl_trigger();
}

template <int D, bool E4M3, bool INTERLEAVED>
cudaError_t launch(const RopeParams& p, int64_t T, const DeviceInfo& dev, cudaStream_t s) {
  const int groups = (p.q_heads + 2 * p.kv_heads + 32 / (D / 8) - 1) / (32 / (D / 8));
  // Few tokens: a warp per head group, so that a call takes one load's latency.
  // Many: a CTA per token (with 8192 tokens, a warp per group would read the
  // table and the weights 24 times per token).
  const bool few = T < 4 * dev.sm_count, even = p.q_heads % (32 / (D / 8)) == 0 && p.kv_heads % (32 / (D / 8)) == 0;
  const dim3 grid(static_cast<unsigned>(T), few ? static_cast<unsigned>((groups + kWarps - 1) / kWarps) : 1u);
  auto kern = few ? (even ? qk_norm_rope_kernel<D, E4M3, INTERLEAVED, 1, true, true>
                          : qk_norm_rope_kernel<D, E4M3, INTERLEAVED, 1, true, false>)
                  : (even ? qk_norm_rope_kernel<D, E4M3, INTERLEAVED, kMany, false, true>
                          : qk_norm_rope_kernel<D, E4M3, INTERLEAVED, kMany, false, false>);
  return launch_pdl(kern, grid, dim3(kWarps * 32), 0, s, p);
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
  if (q_heads < 1 || q_heads > (1 << 16) || cache->heads > (1 << 16)) return SP24_ERR_INVALID_ARG;
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
