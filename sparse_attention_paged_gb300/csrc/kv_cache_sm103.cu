// kv_cache_sm103.cu -- the paged cache of keys and values with grouped heads:
// the store of new tokens into their slots, and the boxes around a page's keys.
//
// Store.  16-bit caches: the values as they are.  fp8: per token and head
//   s = 2^e, the smallest e >= -126 with max |x| <= 448 * 2^e (finite values)
//   code = e4m3(x / s), round to nearest even, infinities +-448, NaN NaN
// A power of two costs a floating format no precision and keeps code * s exact
// in 16 bits.  A row of zeros has the smallest scale, so that the attention
// never takes it for the largest of its weights.
//
// Boxes.  Per page, key head and channel the largest and smallest key:
//   e = the smallest e >= -126 with max(|high|, |low|) <= 127 * 2^e
//   bounds = ceil(high / 2^e), floor(low / 2^e)          int8, scale 2^e
// so that every key of the page lies in the box.  NaN keys are passed over, and
// infinities count as the largest finite number.  All of it is exact.
//
// Measured, bf16, 22,528 tokens, 8 heads of 128: the store 24 to 28 us (185 MB, the copy
// rate), into fp8 21; the boxes of its 352 pages 13.8 out of HBM (46 MB; a block's lengths, table, keys
// and sums follow one another) and some 10 behind the store; a decode step of 64
// requests 8.3 us for both, which is latency.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math_constants.h>
#include <stdint.h>

#include "paged_common.cuh"
#include "sm100_ptx.cuh"

namespace dsa {

namespace {

constexpr unsigned kAll = 0xffffffffu;

// 2^e, -126 <= e <= 127
__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Two 16-bit values as floats.
template <bool FP16>
__device__ __forceinline__ float2 wide(uint32_t u) {
  if (FP16) return __half22float2(*reinterpret_cast<const __half2*>(&u));
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// ---- store --------------------------------------------------------------------

constexpr int kStoreThreads = 256;
// Units of eight values of a key and a value that a thread has: two share a row's scale
// and addresses (fp8, 8 heads: 131,072 tokens of 128 values 115 us, 138 with one; 65,536 of 64
// values 30.6, 36.5 with one, 34.4 with four).  A copy has one: HBM bounds it.
constexpr int store_units(bool fp8) { return fp8 ? 2 : 1; }

// The largest finite magnitude of a row's 16-bit values, of its key in the low and of
// its value in the high half: magnitudes' bits are in their order.
template <bool FP16, int LANES, int UNITS>
__device__ __forceinline__ uint32_t largest(const uint4 (&raw)[2][UNITS]) {
  constexpr uint32_t kInf = FP16 ? 0x7c007c00u : 0x7f807f80u;
  auto reduce = [&](auto magnitude) {
    uint32_t top[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint32_t x = 0;
#pragma unroll
      for (int i = 0; i < UNITS; ++i)
        x = __vmaxu2(x, __vmaxu2(__vmaxu2(magnitude(raw[s][i].x), magnitude(raw[s][i].y)),
                                 __vmaxu2(magnitude(raw[s][i].z), magnitude(raw[s][i].w))));
      top[s] = max(x & 0xffffu, x >> 16);
    }
    uint32_t both = top[0] | top[1] << 16;
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) both = __vmaxu2(both, __shfl_xor_sync(kAll, both, o));
    return both;
  };
  uint32_t top = reduce([](uint32_t u) { return u & 0x7fff7fffu; });
  if (__any_sync(kAll, __vcmpgeu2(top, kInf)))
    top = reduce([](uint32_t u) { return u & 0x7fff7fffu & __vcmpltu2(u & 0x7fff7fffu, kInf); });
  return top;
}

// A thread has UNITS times eight values of one token and head, of its key and its value.
template <bool FP8, bool FP16, int D, int UNITS>
__global__ void __launch_bounds__(kStoreThreads) kv_store_kernel(const KvStoreParams p) {
  constexpr int lanes = D / 8 / UNITS;               // of a head
  const uint32_t row = blockIdx.x * (kStoreThreads / lanes) + threadIdx.x / lanes;
  const int c = threadIdx.x % lanes;
  const uint32_t token = row / (uint32_t)p.heads;
  const int head = (int)(row - token * p.heads);
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  const bool there = token < (uint32_t)p.n;
  const int at = there ? __ldg(p.slots + token) : -1;
  uint4 raw[2][UNITS];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x[s]) +
                                                       (long long)token * p.token[s] + head * p.head[s]) + c;
#pragma unroll
    for (int i = 0; i < UNITS; ++i) raw[s][i] = there ? __ldg(from + i * lanes) : make_uint4(0u, 0u, 0u, 0u);
  }
  const int page = at / kPage, slot = at % kPage;
  const bool good = at >= 0 && page < p.num_pages;
  if (at >= 0 && !good) raise_status(p.status, DSA_ERR_BAD_PAGE);
  const uint32_t top = FP8 ? largest<FP16, lanes, UNITS>(raw) : 0u;
  if (!good) return;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const long long to = (long long)page * p.at[s].page + (long long)slot * p.at[s].slot + head * p.at[s].head;
    if (!FP8) {
      uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.pool[s]) + to) + c;
#pragma unroll
      for (int i = 0; i < UNITS; ++i) out[i * lanes] = raw[s][i];
      continue;
    }
    // big = 1.m * 2^(E - 127): at most 448 * 2^e = 1.75 * 2^(e + 8)
    const float big = s ? wide<FP16>(top).y : wide<FP16>(top).x;
    const uint32_t bits = __float_as_uint(big);
    const int e = max((int)(bits >> 23) - 135 + ((bits & 0x7fffffu) > 0x600000u), -126);
    const float inverse = power(-e);
    uint2* out = reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.pool[s]) + to) + c;
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const uint32_t u[4] = {raw[s][i].x, raw[s][i].y, raw[s][i].z, raw[s][i].w};
      uint32_t codes[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 x = wide<FP16>(u[2 * j]), y = wide<FP16>(u[2 * j + 1]);
        const uint32_t a =
            __nv_cvt_float2_to_fp8x2(make_float2(x.x * inverse, x.y * inverse), __NV_SATFINITE, __NV_E4M3);
        const uint32_t b =
            __nv_cvt_float2_to_fp8x2(make_float2(y.x * inverse, y.y * inverse), __NV_SATFINITE, __NV_E4M3);
        codes[j] = a | b << 16;
      }
      out[i * lanes] = make_uint2(codes[0], codes[1]);
    }
    if (c == 0) p.scale[s][((long long)page * p.heads + head) * kPage + slot] = power(e);
  }
}

// ---- boxes --------------------------------------------------------------------

constexpr int kBoxThreads = 128;

template <bool FP16>
__device__ __forceinline__ uint32_t pick2(uint32_t a, uint32_t b, bool larger) {
  if (FP16) {
    const __half2 x = *reinterpret_cast<const __half2*>(&a), y = *reinterpret_cast<const __half2*>(&b);
    const __half2 r = larger ? __hmax2(x, y) : __hmin2(x, y);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&a);
  const __nv_bfloat162 y = *reinterpret_cast<const __nv_bfloat162*>(&b);
  const __nv_bfloat162 r = larger ? __hmax2(x, y) : __hmin2(x, y);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// A block has one page of one head: a thread 16 bytes of every few tokens.  Ten
// blocks an SM where the registers do (fp8 has 16 values a load, and takes more):
// 352 pages, 8 heads 13.8 us, 14.4 with eight.
template <int KV, int D>
__global__ void __launch_bounds__(kBoxThreads, KV == DSA_KV_FP8_E4M3 ? 8 : 10) block_bounds_kernel(const BlockBoundsParams p) {
  constexpr bool kFp8 = KV == DSA_KV_FP8_E4M3, kHalf = KV == DSA_KV_FP16;
  constexpr int kBytes = kFp8 ? 1 : 2, kUnits = D * kBytes / 16;
  constexpr int kGroups = kBoxThreads / kUnits, kLoads = kPage / kGroups;
  __shared__ float high[kGroups][D], low[kGroups][D];
  __shared__ float tops[kBoxThreads / 32];
  const int head = blockIdx.x % p.heads;
  const int turn = blockIdx.x / p.heads % p.pages, req = blockIdx.x / p.heads / p.pages;
  const int unit = threadIdx.x % kUnits, group = threadIdx.x / kUnits;
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  const int len = __ldg(p.seqlens + req), start = p.starts ? max(__ldg(p.starts + req), 0) : 0;
  if (len <= start) return;
  if ((long long)len > (long long)p.W * kPage) {
    if (threadIdx.x == 0) raise_status(p.status, DSA_ERR_BAD_SEQLEN);
    return;
  }
  for (int block = start / kPage + turn; block <= (len - 1) / kPage; block += p.pages) {
    const int page = __ldg(p.block_table + (long long)req * p.bt_stride + block);
    if (page < 0 || page >= p.num_pages) {
      if (threadIdx.x == 0) raise_status(p.status, DSA_ERR_BAD_PAGE);
      continue;
    }
    const int tokens = min(kPage, len - block * kPage);
    const uint8_t* base = static_cast<const uint8_t*>(p.pool) +
                          ((long long)page * p.at.page + head * p.at.head) * kBytes + unit * 16;
    const long long record = (long long)page * p.heads + head;
    uint4 raw[kLoads];
    float scale[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int token = i * kGroups + group;
      if (token < tokens) {
        raw[i] = __ldg(reinterpret_cast<const uint4*>(base + (long long)token * p.at.slot * kBytes));
        scale[i] = kFp8 ? __ldg(p.scale + record * kPage + token) : 1.f;
      }
    }
    if (!kFp8) {
      constexpr uint32_t kInf = kHalf ? 0x7c007c00u : 0x7f807f80u, kLess = kInf | 0x80008000u;
      uint32_t h[4] = {kLess, kLess, kLess, kLess}, l[4] = {kInf, kInf, kInf, kInf};
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        if (i * kGroups + group < tokens) {
          const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) h[j] = pick2<kHalf>(h[j], u[j], true), l[j] = pick2<kHalf>(l[j], u[j], false);
        }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        *reinterpret_cast<float2*>(&high[group][unit * 8 + 2 * j]) = wide<kHalf>(h[j]);
        *reinterpret_cast<float2*>(&low[group][unit * 8 + 2 * j]) = wide<kHalf>(l[j]);
      }
    } else {
      float h[16], l[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) h[j] = -CUDART_INF_F, l[j] = CUDART_INF_F;
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        if (i * kGroups + group < tokens) {
          const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const __half2_raw r =
                __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u[j >> 1] >> (16 * (j & 1))), __NV_E4M3);
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&r));
            const float x = v.x * scale[i], y = v.y * scale[i];
            h[2 * j] = fmaxf(h[2 * j], x), l[2 * j] = fminf(l[2 * j], x);
            h[2 * j + 1] = fmaxf(h[2 * j + 1], y), l[2 * j + 1] = fminf(l[2 * j + 1], y);
          }
        }
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        *reinterpret_cast<float4*>(&high[group][unit * 16 + j]) = make_float4(h[j], h[j + 1], h[j + 2], h[j + 3]);
        *reinterpret_cast<float4*>(&low[group][unit * 16 + j]) = make_float4(l[j], l[j + 1], l[j + 2], l[j + 3]);
      }
    }
    __syncthreads();
    float h = -CUDART_INF_F, l = CUDART_INF_F;
    const int d = threadIdx.x;
    if (d < D) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) h = fmaxf(h, high[g][d]), l = fminf(l, low[g][d]);
    }
    if (l > h) l = h = 0.f;                        // no number among the keys, or no channel
    h = fminf(fmaxf(h, -FLT_MAX), FLT_MAX), l = fminf(fmaxf(l, -FLT_MAX), FLT_MAX);
    float top = fmaxf(fabsf(h), fabsf(l));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kBoxThreads / 32; ++w) top = fmaxf(top, tops[w]);
    // top = 1.m * 2^(E - 127): at most 127 * 2^e = 1.984375 * 2^(e + 6)
    const uint32_t bits = __float_as_uint(top);
    const int e = max((int)(bits >> 23) - 133 + ((bits & 0x7fffffu) > 0x7e0000u), -126);
    const float inverse = power(-e);
    if (d < D) {
      p.bounds[(record * 2 + 0) * D + d] = (int8_t)(int)ceilf(h * inverse);
      p.bounds[(record * 2 + 1) * D + d] = (int8_t)(int)floorf(l * inverse);
      if (d == 0) p.bound_scale[record] = power(e);
    }
    __syncthreads();                               // the sums before the next page's
  }
}

template <typename K, typename P>
cudaError_t launch(K kernel, long long blocks, int threads, const P& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int KV>
cudaError_t launch_bounds_t(const BlockBoundsParams& p, cudaStream_t stream) {
  const long long blocks = (long long)p.n_req * p.pages * p.heads;
  return p.dim == 128 ? launch(block_bounds_kernel<KV, 128>, blocks, kBoxThreads, p, stream)
                      : launch(block_bounds_kernel<KV, 64>, blocks, kBoxThreads, p, stream);
}

template <bool FP8, bool FP16, int D, int UNITS>
cudaError_t launch_store_u(const KvStoreParams& p, cudaStream_t stream) {
  const long long rows = (long long)p.n * p.heads, per = (long long)UNITS * kStoreThreads / (D / 8);
  return launch(kv_store_kernel<FP8, FP16, D, UNITS>, (rows + per - 1) / per, kStoreThreads, p, stream);
}

template <bool FP8, bool FP16>
cudaError_t launch_store_t(const KvStoreParams& p, cudaStream_t stream) {
  constexpr int units = store_units(FP8);
  return p.dim == 128 ? launch_store_u<FP8, FP16, 128, units>(p, stream) : launch_store_u<FP8, FP16, 64, units>(p, stream);
}

}  // namespace

cudaError_t launch_kv_store(const KvStoreParams& p, int kv_dtype, cudaStream_t stream) {
  if (kv_dtype != DSA_KV_FP8_E4M3) return launch_store_t<false, false>(p, stream);
  return p.dtype == DSA_FP16 ? launch_store_t<true, true>(p, stream) : launch_store_t<true, false>(p, stream);
}

cudaError_t launch_block_bounds(const BlockBoundsParams& p, int kv_dtype, cudaStream_t stream) {
  if (kv_dtype == DSA_KV_BF16) return launch_bounds_t<DSA_KV_BF16>(p, stream);
  if (kv_dtype == DSA_KV_FP16) return launch_bounds_t<DSA_KV_FP16>(p, stream);
  return launch_bounds_t<DSA_KV_FP8_E4M3>(p, stream);
}

}  // namespace dsa
