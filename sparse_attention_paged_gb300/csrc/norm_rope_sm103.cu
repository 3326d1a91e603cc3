// norm_rope_sm103.cu -- per-head normalisation of queries and keys with the
// position rotation in the same pass:
//
//   y = norm(x) * weight (+ bias),   rms:   x * rsqrt(mean(x^2) + eps)
//                                    layer: (x - mean) * rsqrt(var + eps)
//   (a, b) -> (a cos - b sin, b cos + a sin) for the rotated pairs
//
// with every step in fp32 and one rounding to the output type.  A row (one
// head of one token) stays in the registers of a group of 8, 16 or 32
// lanes, eight values a lane, from its one load to its one store, so the
// kernel moves each value once in each direction; the sums are shuffles
// within the group.  A group takes up to four heads of one token, so that
// four loads are in flight and the token's cosines and sines are read once
// for them.  Both values of a pair lie in one lane: where the half layout
// pairs values that are rot/2 apart, a lane takes four from either end.
// HBM-bound.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "latent_common.cuh"
#include "sm100_ptx.cuh"

namespace dsa {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8;  // values a lane holds

// Four values as they lie in memory, and as floats.
template <typename T>
struct Raw4 {
  uint2 r;
  __device__ __forceinline__ void load(const T* p) { r = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void zero() { r = make_uint2(0u, 0u); }
};

template <>
struct Raw4<float> {
  float4 r;
  __device__ __forceinline__ void load(const float* p) { r = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void zero() { r = make_float4(0.f, 0.f, 0.f, 0.f); }
};

__device__ __forceinline__ void unpack(const Raw4<__nv_bfloat16>& x, float* v) {
  v[0] = __uint_as_float(x.r.x << 16), v[1] = __uint_as_float(x.r.x & 0xffff0000u);
  v[2] = __uint_as_float(x.r.y << 16), v[3] = __uint_as_float(x.r.y & 0xffff0000u);
}

__device__ __forceinline__ void unpack(const Raw4<__half>& x, float* v) {
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&x.r.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&x.r.y));
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}

__device__ __forceinline__ void unpack(const Raw4<float>& x, float* v) {
  v[0] = x.r.x, v[1] = x.r.y, v[2] = x.r.z, v[3] = x.r.w;
}

__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

__device__ __forceinline__ void store4(__half* p, const float* v) {
  const __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

__device__ __forceinline__ void store4(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// Four floats of a vector that every row shares; `wide`: 16-byte aligned.
__device__ __forceinline__ void load_shared4(const float* p, bool wide, float* v) {
  if (wide) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __ldg(p + i);
}

__device__ __forceinline__ bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// LANES: lanes per row (8 * LANES >= dim); HEADS: heads a group takes.  The
// loads stay packed until their head's turn, so that three blocks fit an SM.
template <typename T, int LANES, int HEADS, bool INTER>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 2 : 3) norm_rope_kernel(const NormRopeParams p) {
  const long long unit = ((long long)blockIdx.x * kThreads + threadIdx.x) / LANES;
  const int c = threadIdx.x % LANES;
  const int units_q = (p.heads[0] + HEADS - 1) / HEADS;
  const int per_token = units_q + (p.heads[1] + HEADS - 1) / HEADS;
  const bool small = unit <= 0x7fffffff;         // spares the 64-bit division
  const long long token = small ? (unsigned)unit / (unsigned)per_token : unit / per_token;
  int j = (int)(unit - token * per_token);
  const int side = j >= units_q;
  j = (side ? j - units_q : j) * HEADS;
  const bool row_ok = token < p.tokens;
  const bool mine = row_ok && c * kChunk < p.dim;
  const int heads = row_ok ? min(HEADS, p.heads[side] - j) : 0;

  sm100::griddep_wait();
  sm100::griddep_launch_dependents();

  // Where this lane's two times four values lie: next to one another, or, in
  // a part that is rotated in the half layout, at both ends of four pairs
  const int at = c * kChunk - p.rot_offset;
  const bool turned = mine && p.positions != nullptr && at >= 0 && at < p.rot;
  const bool split = turned && !INTER;
  const int lo = split ? p.rot_offset + at / 2 : c * kChunk;
  const int hi = split ? lo + p.rot / 2 : lo + 4;

  Raw4<T> raw[HEADS][2];
  {
    const T* x = static_cast<const T*>(p.x[side]) + token * p.xt[side] + j * p.xh[side];
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
      raw[h][0].zero(), raw[h][1].zero();
      if (mine && h < heads) raw[h][0].load(x + lo), raw[h][1].load(x + hi);
      x += p.xh[side];
    }
  }

  // the angles of this lane's four pairs
  float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
  bool bad = false;
  if (row_ok && p.positions != nullptr) {
    const int pos = __ldg(p.positions + token);
    bad = pos < 0 || pos >= p.max_pos;
    if (turned && !bad) {
      const float* row = p.table + (long long)pos * p.rot + at / 2;
      load_shared4(row, true, cs);
      load_shared4(row + p.rot / 2, true, sn);
    }
  }
  float w[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.f, b[i] = 0.f;
  if (mine && p.norm != DSA_NORM_NONE) {
    const float *pw = p.weight[side], *pb = p.bias[side];
    if (pw) load_shared4(pw + lo, aligned16(pw), w), load_shared4(pw + hi, aligned16(pw), w + 4);
    if (pb) load_shared4(pb + lo, aligned16(pb), b), load_shared4(pb + hi, aligned16(pb), b + 4);
  }
  if (bad && c == 0) raise_status(p.status, DSA_ERR_BAD_POSITION);

  const float inv_dim = 1.f / (float)p.dim;
  T* y = static_cast<T*>(p.y[side]) + token * p.yt[side] + j * p.yh[side];
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    float v[8];
    unpack(raw[h][0], v);
    unpack(raw[h][1], v + 4);
    if (p.norm == DSA_NORM_LAYER) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
      const float mean = group_sum<LANES>(s) * inv_dim;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = mine ? v[i] - mean : 0.f;
    }
    if (p.norm != DSA_NORM_NONE) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(v[i], v[i], s);
      const float r = rsqrtf(group_sum<LANES>(s) * inv_dim + p.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fmaf(v[i] * r, w[i], b[i]);
    }
    if (turned) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a0 = INTER ? v[2 * i] : v[i], a1 = INTER ? v[2 * i + 1] : v[4 + i];
        v[INTER ? 2 * i : i] = a0 * cs[i] - a1 * sn[i];
        v[INTER ? 2 * i + 1 : 4 + i] = a1 * cs[i] + a0 * sn[i];
      }
    }
    if (bad) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = CUDART_NAN_F;
    }
    if (mine && h < heads) store4(y + lo, v), store4(y + hi, v + 4);
    y += p.yh[side];
  }
}

template <typename T, int LANES, int HEADS, bool INTER>
cudaError_t launch_t(const NormRopeParams& p, cudaStream_t stream) {
  const long long units = (long long)p.tokens * ((p.heads[0] + HEADS - 1) / HEADS +
                                                 (p.heads[1] + HEADS - 1) / HEADS);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((units * LANES + kThreads - 1) / kThreads));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_rope_kernel<T, LANES, HEADS, INTER>, p);
}

template <typename T, bool INTER>
cudaError_t launch_dim(const NormRopeParams& p, cudaStream_t stream) {
  if (p.dim <= 64) return launch_t<T, 8, 4, INTER>(p, stream);
  if (p.dim <= 128) return launch_t<T, 16, 4, INTER>(p, stream);
  return launch_t<T, 32, 4, INTER>(p, stream);
}

template <typename T>
cudaError_t launch_dtype(const NormRopeParams& p, cudaStream_t stream) {
  return p.interleaved ? launch_dim<T, true>(p, stream) : launch_dim<T, false>(p, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, int dtype, cudaStream_t stream) {
  if (dtype == DSA_BF16) return launch_dtype<__nv_bfloat16>(p, stream);
  if (dtype == DSA_FP16) return launch_dtype<__half>(p, stream);
  return launch_dtype<float>(p, stream);
}

}  // namespace dsa
