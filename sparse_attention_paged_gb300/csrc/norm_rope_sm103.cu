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
// for them.  In the half layout the partner of a value lies rot/2 values
// away in another lane and comes by shuffle; interleaved pairs lie in one
// lane.  HBM-bound.
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

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ void load8(const __half* p, float (&v)[8]) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Eight floats of a 4-byte aligned vector that every row shares.
__device__ __forceinline__ void load_shared8(const float* p, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __ldg(p + i);
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// LANES: lanes per row (8 * LANES >= dim); HEADS: heads a group takes.
template <typename T, int LANES, int HEADS>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeParams p) {
  const long long unit = ((long long)blockIdx.x * kThreads + threadIdx.x) / LANES;
  const int lane = threadIdx.x % 32, c = threadIdx.x % LANES;
  const int units_q = (p.heads[0] + HEADS - 1) / HEADS;
  const int per_token = units_q + (p.heads[1] + HEADS - 1) / HEADS;
  const long long token = unit / per_token;
  int j = (int)(unit % per_token);
  const int side = j >= units_q;
  j = (side ? j - units_q : j) * HEADS;
  const bool row_ok = token < p.tokens;
  const bool mine = row_ok && c * kChunk < p.dim;
  const int heads = row_ok ? min(HEADS, p.heads[side] - j) : 0;

  sm100::griddep_wait();
  sm100::griddep_launch_dependents();

  float v[HEADS][8];
  {
    const T* x = static_cast<const T*>(p.x[side]) + token * p.xt[side] + j * p.xh[side] + c * kChunk;
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[h][i] = 0.f;
      if (mine && h < heads) load8(x + h * p.xh[side], v[h]);
    }
  }

  // the token's angles: this lane's pairs
  float cs[8], sn[8];
  const int at = c * kChunk - p.rot_offset;      // this lane's first value in the rotated part
  const bool turned = mine && p.positions != nullptr && at >= 0 && at < p.rot;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
  if (row_ok && p.positions != nullptr) {
    const int pos = __ldg(p.positions + token);
    bad = pos < 0 || pos >= p.max_pos;
    if (turned && !bad) {
      const int half = p.rot / 2;
      const float* row = p.table + (long long)pos * p.rot;
      const int first = p.interleaved ? at / 2 : at % half;
      const float4* rc = reinterpret_cast<const float4*>(row + first);
      const float4* rs = reinterpret_cast<const float4*>(row + half + first);
      const float4 c0 = __ldg(rc), s0 = __ldg(rs);
      cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w;
      sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w;
      if (!p.interleaved) {
        const float4 c1 = __ldg(rc + 1), s1 = __ldg(rs + 1);
        cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
        sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
      }
    }
  }
  float w[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.f, b[i] = 0.f;
  if (mine && p.norm != DSA_NORM_NONE) {
    if (p.weight[side]) load_shared8(p.weight[side] + c * kChunk, w);
    if (p.bias[side]) load_shared8(p.bias[side] + c * kChunk, b);
  }

  const float inv_dim = 1.f / (float)p.dim;
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    if (p.norm == DSA_NORM_LAYER) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[h][i];
      const float mean = group_sum<LANES>(s) * inv_dim;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[h][i] = mine ? v[h][i] - mean : 0.f;
    }
    if (p.norm != DSA_NORM_NONE) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(v[h][i], v[h][i], s);
      const float r = rsqrtf(group_sum<LANES>(s) * inv_dim + p.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[h][i] = fmaf(v[h][i] * r, w[i], b[i]);
    }
  }

  if (p.positions != nullptr) {
    if (p.interleaved) {
#pragma unroll
      for (int h = 0; h < HEADS; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a0 = v[h][2 * i], a1 = v[h][2 * i + 1];
          if (turned) {
            v[h][2 * i] = a0 * cs[i] - a1 * sn[i];
            v[h][2 * i + 1] = a1 * cs[i] + a0 * sn[i];
          }
        }
    } else {
      // the partner's lane is rot/16 lanes away; lanes outside the rotated
      // part shuffle with themselves
      const int hop = p.rot / 16;
      const bool low = at < p.rot / 2;
      const int from = turned ? (low ? lane + hop : lane - hop) : lane;
#pragma unroll
      for (int h = 0; h < HEADS; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float o = __shfl_sync(0xffffffffu, v[h][i], from);
          if (turned) v[h][i] = v[h][i] * cs[i] + (low ? -o : o) * sn[i];
        }
    }
    if (bad) {
      if (c == 0) raise_status(p.status, DSA_ERR_BAD_POSITION);
#pragma unroll
      for (int h = 0; h < HEADS; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[h][i] = CUDART_NAN_F;
    }
  }

  T* y = static_cast<T*>(p.y[side]) + token * p.yt[side] + j * p.yh[side] + c * kChunk;
#pragma unroll
  for (int h = 0; h < HEADS; ++h)
    if (mine && h < heads) store8(y + h * p.yh[side], v[h]);
}

template <typename T, int LANES, int HEADS>
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
  return cudaLaunchKernelEx(&cfg, norm_rope_kernel<T, LANES, HEADS>, p);
}

template <typename T>
cudaError_t launch_dtype(const NormRopeParams& p, cudaStream_t stream) {
  if (p.dim <= 64) return launch_t<T, 8, 4>(p, stream);
  if (p.dim <= 128) return launch_t<T, 16, 4>(p, stream);
  return launch_t<T, 32, 4>(p, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, int dtype, cudaStream_t stream) {
  if (dtype == DSA_BF16) return launch_dtype<__nv_bfloat16>(p, stream);
  if (dtype == DSA_FP16) return launch_dtype<__half>(p, stream);
  return launch_dtype<float>(p, stream);
}

}  // namespace dsa
