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
// Measured, 22,528 tokens, 8 heads of 128: the bf16 store 24 to 28 us (185 MB, the copy
// rate), into fp8 21; the boxes of its 352 pages 8 us behind the store (46 MB, from L2), 65,536
// tokens' 24 (HBM at 80 % of the copy rate), fp8 131,072 tokens' 50 (instructions: a code is
// widened and scaled in fp32); a decode step of 64 requests 4.8 us for both, which is latency
// (8.9 in a graph's replay by itself, 10 to 12 as calls).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math_constants.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

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

constexpr int kBoxThreads = 128, kBoxBlocks = 8;  // threads of a block, blocks of an SM

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

// The lanes of a warp whose indexes agree below UNITS have the same N elements each: the
// largest (smallest) of all, N / 2 of them after each step, and so on.
template <int UNITS, int N, typename T, typename F>
__device__ __forceinline__ void share_out(T (&x)[N], int lane, F pick) {
  int n = N;
#pragma unroll
  for (int m = UNITS; m < 32; m <<= 1) {
    n >>= 1;
#pragma unroll
    for (int j = 0; j < N / 2; ++j)
      if (j < n) {
        const T keep = lane & m ? x[j + n] : x[j], give = lane & m ? x[j] : x[j + n];
        x[j] = pick(keep, __shfl_xor_sync(kAll, give, m));
      }
  }
}

// A page of one head is a block's at a time: a thread 16 bytes of every few tokens, the
// warp shares out their extremes, and the warps meet in shared memory (all lanes'
// extremes there, in banks that eight lanes have in common, took 62 us for 51 at 131,072 fp8
// tokens, 8 heads of 128).  The grid covers max_tokens for every request, and where they are of
// many lengths most of it is no page: a block looks 32 places up at a time (23 prompts of
// 300 to 9,000 tokens 7 us, 28 with a block for each place).
template <int KV, int D>
__global__ void __launch_bounds__(kBoxThreads, kBoxBlocks) block_bounds_kernel(const BlockBoundsParams p) {
  constexpr bool kFp8 = KV == DSA_KV_FP8_E4M3, kHalf = KV == DSA_KV_FP16;
  constexpr int kBytes = kFp8 ? 1 : 2, kUnits = D * kBytes / 16;
  constexpr int kUnitBits = kUnits == 4 ? 2 : kUnits == 8 ? 3 : 4;
  constexpr int kGroups = kBoxThreads / kUnits, kLoads = kPage / kGroups;
  // a 16-byte unit's extremes (values, or pairs of 16 bits), and those that a lane ends with
  constexpr int kHave = kFp8 ? 16 : 4, kLeft = kHave * kUnits / 32, kPair = kFp8 ? 1 : 2;
  using Extreme = std::conditional_t<kFp8, float, uint32_t>;
  __shared__ alignas(16) Extreme high[kBoxThreads / 32][D / kPair], low[kBoxThreads / 32][D / kPair];
  __shared__ float tops[kBoxThreads / 32];
  __shared__ int4 found[32];
  __shared__ int2 counts;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int unit = threadIdx.x % kUnits, group = threadIdx.x / kUnits;
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  auto box = [&](int at) {
    const int4 item = found[at];
    const int page = item.x, head = item.y, tokens = item.z;
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
    Extreme h[kHave], l[kHave];
    if constexpr (!kFp8) {
      constexpr uint32_t kInf = kHalf ? 0x7c007c00u : 0x7f807f80u, kLess = kInf | 0x80008000u;
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = kLess, l[j] = kInf;
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        if (i * kGroups + group < tokens) {
          const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) h[j] = pick2<kHalf>(h[j], u[j], true), l[j] = pick2<kHalf>(l[j], u[j], false);
        }
      share_out<kUnits>(h, lane, [](uint32_t x, uint32_t y) { return pick2<kHalf>(x, y, true); });
      share_out<kUnits>(l, lane, [](uint32_t x, uint32_t y) { return pick2<kHalf>(x, y, false); });
    } else {
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
      share_out<kUnits>(h, lane, [](float x, float y) { return fmaxf(x, y); });
      share_out<kUnits>(l, lane, [](float x, float y) { return fminf(x, y); });
    }
    // places: parts of the units (by the lane's upper bits, the first one largest), units, kLeft
    const int part = __brev((unsigned)lane / kUnits) >> (27 + kUnitBits);
#pragma unroll
    for (int j = 0; j < kLeft; ++j) {
      high[warp][(part * kUnits + lane % kUnits) * kLeft + j] = h[j];
      low[warp][(part * kUnits + lane % kUnits) * kLeft + j] = l[j];
    }
    __syncthreads();
    // a thread has a channel: d, at place `at` of the extremes
    float h1 = -CUDART_INF_F, l1 = CUDART_INF_F;
    const int t = threadIdx.x, place = t / kPair, of = place / kLeft;
    const int d = (of % kUnits * kHave + of / kUnits * kLeft + place % kLeft) * kPair + t % kPair;
    if (t < D) {
#pragma unroll
      for (int w = 0; w < kBoxThreads / 32; ++w) {
        if constexpr (kFp8) {
          h1 = fmaxf(h1, high[w][place]), l1 = fminf(l1, low[w][place]);
        } else {
          const float2 a = wide<kHalf>(high[w][place]), b = wide<kHalf>(low[w][place]);
          h1 = fmaxf(h1, t & 1 ? a.y : a.x), l1 = fminf(l1, t & 1 ? b.y : b.x);
        }
      }
    }
    if (l1 > h1) l1 = h1 = 0.f;                    // no number among the keys, or no channel
    h1 = fminf(fmaxf(h1, -FLT_MAX), FLT_MAX), l1 = fminf(fmaxf(l1, -FLT_MAX), FLT_MAX);
    float top = fmaxf(fabsf(h1), fabsf(l1));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kBoxThreads / 32; ++w) top = fmaxf(top, tops[w]);
    // top = 1.m * 2^(E - 127): at most 127 * 2^e = 1.984375 * 2^(e + 6)
    const uint32_t bits = __float_as_uint(top);
    const int e = max((int)(bits >> 23) - 133 + ((bits & 0x7fffffu) > 0x7e0000u), -126);
    const float inverse = power(-e);
    if (t < D) {
      // a quotient below 2^-149 is 0 here, and its key is not: 1 and -1 are the least codes around it
      const int up = (int)ceilf(h1 * inverse), down = (int)floorf(l1 * inverse);
      p.bounds[(record * 2 + 0) * D + d] = (int8_t)(h1 > 0.f ? max(up, 1) : up);
      p.bounds[(record * 2 + 1) * D + d] = (int8_t)(l1 < 0.f ? min(down, -1) : down);
      if (t == 0) p.bound_scale[record] = power(e);
    }
  };
  // 32 items at a time, a lane of the first warp each; those with a page into a list.
  // The last ones first: a store just before has left their keys in L2 (16 requests of
  // 4,096 tokens, both calls 103.8 us for 106.1).
  const uint32_t items = (uint32_t)p.n_req * p.pages * p.heads;
  for (uint32_t i0 = blockIdx.x; i0 < items; i0 += 32 * gridDim.x) {
    // (turns past the first where requests have more than max_tokens)
    for (int turn = 0;; ++turn) {
      if (threadIdx.x < 32) {
        const uint32_t from_end = i0 + lane * gridDim.x, item = items - 1 - from_end;
        int head = 0, page = -1, tokens = 0;
        bool more = false;
        if (from_end < items) {
          const uint32_t place = item / p.heads, req = place / p.pages;
          head = (int)(item - place * p.heads);
          const int start = p.starts ? max(__ldg(p.starts + req), 0) : 0, len = __ldg(p.seqlens + req);
          if (len > start) {
            const long long block = start / kPage + (long long)(place - req * p.pages) + (long long)turn * p.pages;
            const int end = (len - 1) / kPage;
            if ((long long)len > (long long)p.W * kPage) {
              raise_status(p.status, DSA_ERR_BAD_SEQLEN);
            } else if (block <= end) {
              page = __ldg(p.block_table + (long long)req * p.bt_stride + block);
              tokens = min(kPage, len - (int)block * kPage);
              more = block + p.pages <= end;
              if (page < 0 || page >= p.num_pages) {
                raise_status(p.status, DSA_ERR_BAD_PAGE);
                page = -1;
              }
            }
          }
        }
        const uint32_t there = __ballot_sync(kAll, page >= 0), again = __ballot_sync(kAll, more);
        if (page >= 0) found[__popc(there & ((1u << lane) - 1u))] = make_int4(page, head, tokens, 0);
        if (lane == 0) counts = make_int2(__popc(there), again != 0);
      }
      __syncthreads();
      const int2 n = counts;
      for (int i = 0; i < n.x; ++i) box(i);
      __syncthreads();                             // the list before the next one's
      if (!n.y) break;
    }
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
cudaError_t launch_bounds_t(const BlockBoundsParams& p, int sms, cudaStream_t stream) {
  const long long blocks = std::min((long long)p.n_req * p.pages * p.heads, (long long)sms * kBoxBlocks);
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

cudaError_t launch_block_bounds(const BlockBoundsParams& p, int kv_dtype, int sms, cudaStream_t stream) {
  if (kv_dtype == DSA_KV_BF16) return launch_bounds_t<DSA_KV_BF16>(p, sms, stream);
  if (kv_dtype == DSA_KV_FP16) return launch_bounds_t<DSA_KV_FP16>(p, sms, stream);
  return launch_bounds_t<DSA_KV_FP8_E4M3>(p, sms, stream);
}

}  // namespace dsa
