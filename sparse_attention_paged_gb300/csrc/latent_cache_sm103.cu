// latent_cache_sm103.cu -- the latent cache's two ends.
//
// Store: a token's latent vector (512 values) is normalised
// (c * rsqrt(mean(c^2) + eps) * weight), its rotated part (64 values) turned
// by its position, and both written to the token's slot; with an fp8 cache
// the latent is quantised on the way.  Each group of 128 values gets the
// scale
//
//   s = 2^e, e the smallest with max|c| <= 448 * 2^e   (finite values; 1 for zeros)
//   code = e4m3(c / s), nearest even, infinities to +-448
//
// A power of two keeps c / s and code * s exact in fp32, and code * s exact
// in bf16 (four significant bits), so reading the cache back in bf16 loses
// nothing that the codes hold; e4m3 being a floating format, a scale up to
// twice the tightest one costs no relative precision above the subnormals.
//
// Load: a range of each request's tokens as packed bf16 rows.
//
// One warp per token in both, all of a token's loads at once; HBM-bound for
// many tokens, by latency for few.  In the store lane l holds values
// 16l .. 16l+15 and a group's maximum is a shuffle over eight lanes; in the
// load it holds 8l .. 8l+7 and 256 + 8l .., so that a warp writes 512
// adjacent bytes an instruction (4% faster than 32 bytes a lane).  Measured
// out of HBM, one call after another: storing 65,536 tokens with the norm
// and the rotation 29.1 us (fp8, 4.1 TB/s) and 28.9 us (bf16, 5.2 TB/s),
// loading them 21.3 us (fp8, 5.6 TB/s) and 25.0 us (bf16, 6.0 TB/s); 1,024
// tokens 2.5 us either way.  The store's work, about 250 instructions
// a token and 64 passes of L1 for the weights, is what keeps it from the
// load's rate.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "latent_common.cuh"
#include "sm100_ptx.cuh"

namespace dsa {

namespace {

constexpr int kWarps = 8;  // warps per block

__device__ __forceinline__ void unpack2(uint32_t u, float& a, float& b) {
  a = __uint_as_float(u << 16);
  b = __uint_as_float(u & 0xffff0000u);
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The exponent of the group's scale for its largest finite magnitude.
__device__ __forceinline__ int scale_exponent(float top) {
  if (!(top > 0.f)) return 0;
  // top = m * 2^x with m in [1, 2); 448 = 1.75 * 2^8
  const uint32_t bits = __float_as_uint(top);
  const int x = (int)(bits >> 23) - 127;                       // subnormal: -127, clamped below
  const int e = (bits & 0x7fffffu) <= 0x600000u ? x - 8 : x - 7;
  return max(e, -126);
}

// One token's latent (r0, r1: this lane's 16 values; w: their weights) and
// rotated part (rr: its two) into their place.
template <int KV>
__device__ __forceinline__ void store_token(const LatentStoreParams& p, int page, int slot, int pos, uint4 r0,
                                            uint4 r1, uint32_t rr, const float (&w)[16], int lane) {
  uint8_t* pg = p.cache + (long long)page * p.page_stride;

  // the rotated part
  float a, b;
  unpack2(rr, a, b);
  if (p.positions != nullptr) {
    if (pos < 0 || pos >= p.max_pos) {
      if (lane == 0) raise_status(p.status, DSA_ERR_BAD_POSITION);
      a = b = CUDART_NAN_F;
    } else {
      const float* row = p.table + (long long)pos * kRope;
      if (p.interleaved) {
        const float c = __ldg(row + lane), s = __ldg(row + kRope / 2 + lane);
        const float a0 = a;
        a = a0 * c - b * s;
        b = b * c + a0 * s;
      } else {
        // values 2l, 2l+1 pair with those 32 further on, 16 lanes away
        const int f = (2 * lane) % (kRope / 2);
        const float2 c = __ldg(reinterpret_cast<const float2*>(row + f));
        const float2 s = __ldg(reinterpret_cast<const float2*>(row + kRope / 2 + f));
        const float oa = __shfl_xor_sync(0xffffffffu, a, 16), ob = __shfl_xor_sync(0xffffffffu, b, 16);
        const float sign = lane < 16 ? -1.f : 1.f;
        a = a * c.x + sign * oa * s.x;
        b = b * c.y + sign * ob * s.y;
      }
    }
  }
  uint8_t* rope_at = KV == DSA_KV_BF16 ? pg + slot * kTokenBytesBf16 + kLatent * 2
                                       : pg + kRopeOffsetFp8 + slot * (kRope * 2);
  reinterpret_cast<uint32_t*>(rope_at)[lane] = pack2(a, b);

  // the latent
  float x[16];
  {
    const uint32_t u[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) unpack2(u[j], x[2 * j], x[2 * j + 1]);
  }
  if (p.weight != nullptr) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) s = fmaf(x[j], x[j], s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float r = rsqrtf(s * (1.f / kLatent) + p.eps);
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = x[j] * r * w[j];
  }
  if (KV == DSA_KV_BF16) {
    uint4* dst = reinterpret_cast<uint4*>(pg + slot * kTokenBytesBf16) + lane * 2;
    dst[0] = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
    dst[1] = make_uint4(pack2(x[8], x[9]), pack2(x[10], x[11]), pack2(x[12], x[13]),
                        pack2(x[14], x[15]));
    return;
  }
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float m = fabsf(x[j]);
    if (m < CUDART_INF_F) top = fmaxf(top, m);                 // false for infinities and NaN
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const int e = scale_exponent(top);
  const float inv = pow2(-e);                                  // -e <= 126
  uint32_t codes[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_fp8x2_storage_t lo =
        __nv_cvt_float2_to_fp8x2(make_float2(x[4 * j] * inv, x[4 * j + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t hi =
        __nv_cvt_float2_to_fp8x2(make_float2(x[4 * j + 2] * inv, x[4 * j + 3] * inv), __NV_SATFINITE, __NV_E4M3);
    codes[j] = (uint32_t)lo | ((uint32_t)hi << 16);
  }
  reinterpret_cast<uint4*>(pg + slot * kLatent)[lane] =
      make_uint4(codes[0], codes[1], codes[2], codes[3]);
  if ((lane & 7) == 0)
    reinterpret_cast<float*>(pg + kScaleOffsetFp8)[slot * kLatentGroups + lane / 8] = pow2(e);
}

template <int KV, int TOK>
__global__ void __launch_bounds__(kWarps * 32) latent_store_kernel(const LatentStoreParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long i0 = ((long long)blockIdx.x * kWarps + warp) * TOK;
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  int at[TOK], pos[TOK];
  uint4 r0[TOK], r1[TOK];
  uint32_t rr[TOK];
#pragma unroll
  for (int u = 0; u < TOK; ++u) {
    const long long i = i0 + u;
    at[u] = -1, pos[u] = 0;
    if (i >= p.n) continue;
    at[u] = __ldg(p.slots + i);
    if (p.positions != nullptr) pos[u] = __ldg(p.positions + i);
    const uint4* src = reinterpret_cast<const uint4*>(p.latent + i * p.latent_stride) + lane * 2;
    r0[u] = __ldg(src), r1[u] = __ldg(src + 1);
    rr[u] = __ldg(reinterpret_cast<const uint32_t*>(p.rope + i * p.rope_stride) + lane);
  }
  float w[16];
  if (p.weight != nullptr) {
    const float4* src = reinterpret_cast<const float4*>(p.weight) + lane * 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 f = __ldg(src + j);
      w[4 * j] = f.x, w[4 * j + 1] = f.y, w[4 * j + 2] = f.z, w[4 * j + 3] = f.w;
    }
  }
#pragma unroll
  for (int u = 0; u < TOK; ++u) {
    if (at[u] < 0) continue;                                   // warp-uniform, as all below
    const int page = at[u] / kPage;
    if (page >= p.num_pages) {
      if (lane == 0) raise_status(p.status, DSA_ERR_BAD_PAGE);
      continue;
    }
    store_token<KV>(p, page, at[u] % kPage, pos[u], r0[u], r1[u], rr[u], w, lane);
  }
}

// The request of output row i: the last r < n_req with cu[r] <= i (0 if
// none), a 32-way search with one load a level.  Any values of cu give an r
// in range.
__device__ __forceinline__ int find_request(const int* cu, int n_req, int i, int lane) {
  int lo = 0, len = n_req;
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int j = lane * step;
    const uint32_t below = __ballot_sync(0xffffffffu, j < len && __ldg(cu + lo + min(j, len - 1)) <= i);
    const int hit = below ? 31 - __clz(below) : 0;
    lo += hit * step;
    len = min(step, len - hit * step);
  }
  return lo;
}

template <int KV>
__global__ void __launch_bounds__(kWarps * 32) latent_load_kernel(const LatentLoadParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long i = (long long)blockIdx.x * kWarps + warp;
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  if (i >= p.n) return;
  const int r = find_request(p.cu, p.n_req, (int)i, lane);
  const int first = __ldg(p.cu + r), end = __ldg(p.cu + r + 1);
  const int start = p.starts ? __ldg(p.starts + r) : 0;
  uint4 o0 = make_uint4(0u, 0u, 0u, 0u), o1 = o0;
  uint32_t orope = 0;
  if (i >= first && i < end) {                                 // else a row of no request: zeros
    const long long pos = (long long)start + (i - first);
    int page = -1;
    const bool in = pos >= 0 && pos < (long long)p.W * kPage;
    if (in) page = __ldg(p.block_table + r * p.bt_stride + pos / kPage);
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) raise_status(p.status, in ? DSA_ERR_BAD_PAGE : DSA_ERR_BAD_SEQLEN);
      o0 = o1 = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);  // bf16 NaN
      orope = 0x7fff7fffu;
    } else {
      const uint8_t* pg = p.cache + (long long)page * p.page_stride;
      const int slot = (int)(pos % kPage);
      if (KV == DSA_KV_BF16) {
        const uint4* src = reinterpret_cast<const uint4*>(pg + slot * kTokenBytesBf16) + lane;
        o0 = src[0], o1 = src[32];
        orope = reinterpret_cast<const uint32_t*>(pg + slot * kTokenBytesBf16 + kLatent * 2)[lane];
      } else {
        const uint2* src = reinterpret_cast<const uint2*>(pg + slot * kLatent) + lane;
        const uint2 c0 = src[0], c1 = src[32];
        const float* scale = reinterpret_cast<const float*>(pg + kScaleOffsetFp8) + slot * kLatentGroups + lane / 16;
        const float s0 = scale[0], s1 = scale[2];
        orope = reinterpret_cast<const uint32_t*>(pg + kRopeOffsetFp8 + slot * (kRope * 2))[lane];
        const uint32_t u[4] = {c0.x, c0.y, c1.x, c1.y};
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const __half2_raw f = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u[j] >> (16 * h)), __NV_E4M3);
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f));
            const float s = j < 2 ? s0 : s1;
            o[2 * j + h] = pack2(v.x * s, v.y * s);
          }
        o0 = make_uint4(o[0], o[1], o[2], o[3]);
        o1 = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }
  uint16_t* out = p.out + i * p.out_stride;
  reinterpret_cast<uint4*>(out)[lane] = o0;
  reinterpret_cast<uint4*>(out)[lane + 32] = o1;
  reinterpret_cast<uint32_t*>(out + kLatent)[lane] = orope;
}

// From this many tokens on a warp stores kManyTok of them and loads their
// weights once: 4,096 tokens 4.3 us for 4.8, 22,528 12.3 for 13.0, 65,536
// 29.1 for 33.3 (fp8).  Below, latency counts: 1,024 tokens 3.2 us for 2.5.
// Four or eight a warp are slower than two at 22,528 tokens.
constexpr int kMany = 4096, kManyTok = 2;

template <typename P>
cudaError_t launch(void (*kernel)(P), const P& p, int tok, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)p.n + kWarps * tok - 1) / (kWarps * tok)));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_latent_store(const LatentStoreParams& p, int kv_dtype, cudaStream_t stream) {
  if (p.n >= kMany)
    return kv_dtype == DSA_KV_BF16 ? launch(latent_store_kernel<DSA_KV_BF16, kManyTok>, p, kManyTok, stream)
                                   : launch(latent_store_kernel<DSA_KV_FP8_E4M3, kManyTok>, p, kManyTok, stream);
  return kv_dtype == DSA_KV_BF16 ? launch(latent_store_kernel<DSA_KV_BF16, 1>, p, 1, stream)
                                 : launch(latent_store_kernel<DSA_KV_FP8_E4M3, 1>, p, 1, stream);
}

cudaError_t launch_latent_load(const LatentLoadParams& p, int kv_dtype, cudaStream_t stream) {
  return kv_dtype == DSA_KV_BF16 ? launch(latent_load_kernel<DSA_KV_BF16>, p, 1, stream)
                                 : launch(latent_load_kernel<DSA_KV_FP8_E4M3>, p, 1, stream);
}

}  // namespace dsa
