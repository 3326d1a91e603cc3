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
// Values are read evict-first, as nothing else reads them.  Writing them so as
// well takes another 5 to 10% off this kernel's time and adds it to that of
// the next one, which reads them.
// Measured: 4,096 tokens of 64 + 1 heads of 128 bf16 values 31 us (4.4 TB/s
// of 136 MB, 0.64 of a copy's rate, with 61% of the issue slots taken: neither
// is full).  What holds it: a block has no loads in flight while it computes and
// stores, and an access is 8 bytes a lane (16 for fp32), which fills whole
// sectors in a part rotated by halves only; elsewhere neighbouring lanes are 16
// bytes apart, and an instruction takes half of each sector.  1,337 tokens of 24 + 8 heads of 192 fp16 values 7.6 us
// (4.3 TB/s) in a graph; 64 tokens 2.6 us, one DRAM round trip and the launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "latent_common.cuh"
#include "sm100_ptx.cuh"

namespace dsa {

namespace {

// Blocks of 128: 4,096 tokens of 65 heads 31.5 us for 32.2 with 256 (a wave's
// end is cut finer).
constexpr int kThreads = 128;
constexpr int kChunk = 8;  // values a lane holds

// Two floats in one 64-bit register pair: half the instructions of the sums
// and products, which bound this kernel once its loads are wide.
using F2 = unsigned long long;

__device__ __forceinline__ F2 pack(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(F2 x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float sum2(F2 a) {
  float x, y;
  unpair(a, x, y);
  return x + y;
}

// Four values as they lie in memory, and as floats.
template <typename T>
struct Raw4 {
  uint2 r;
  __device__ __forceinline__ void load(const T* p) { r = __ldcs(reinterpret_cast<const uint2*>(p)); }
  __device__ __forceinline__ void zero() { r = make_uint2(0u, 0u); }
};

template <>
struct Raw4<float> {
  float4 r;
  __device__ __forceinline__ void load(const float* p) { r = __ldcs(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void zero() { r = make_float4(0.f, 0.f, 0.f, 0.f); }
};

__device__ __forceinline__ void unpack(const Raw4<__nv_bfloat16>& x, F2* v) {
  v[0] = pack(__uint_as_float(x.r.x << 16), __uint_as_float(x.r.x & 0xffff0000u));
  v[1] = pack(__uint_as_float(x.r.y << 16), __uint_as_float(x.r.y & 0xffff0000u));
}

__device__ __forceinline__ void unpack(const Raw4<__half>& x, F2* v) {
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&x.r.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&x.r.y));
  v[0] = pack(a.x, a.y), v[1] = pack(b.x, b.y);
}

__device__ __forceinline__ void unpack(const Raw4<float>& x, F2* v) {
  v[0] = pack(x.r.x, x.r.y), v[1] = pack(x.r.z, x.r.w);
}

__device__ __forceinline__ void store4(__nv_bfloat16* p, const F2* v) {
  float a, b, c, d;
  unpair(v[0], a, b), unpair(v[1], c, d);
  const __nv_bfloat162 lo = __floats2bfloat162_rn(a, b), hi = __floats2bfloat162_rn(c, d);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

__device__ __forceinline__ void store4(__half* p, const F2* v) {
  float a, b, c, d;
  unpair(v[0], a, b), unpair(v[1], c, d);
  const __half2 lo = __floats2half2_rn(a, b), hi = __floats2half2_rn(c, d);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

__device__ __forceinline__ void store4(float* p, const F2* v) {
  float a, b, c, d;
  unpair(v[0], a, b), unpair(v[1], c, d);
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}

// Four floats of a vector that every row shares.
__device__ __forceinline__ void load_shared4(const float* p, float* v) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// LANES: lanes per row (8 * LANES >= dim; FULL: equal); HEADS: heads a group
// takes; INTER: interleaved pairs.  The loads stay packed until their head's turn, so that
// 32 warps fit an SM (16-bit types).
template <typename T, int LANES, int HEADS, bool INTER, bool FULL>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 6 : 8) norm_rope_kernel(const NormRopeParams p) {
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
      load_shared4(row, cs);
      load_shared4(row + p.rot / 2, sn);
    }
  }
  float w[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.f, b[i] = 0.f;
  if (mine && p.norm != DSA_NORM_NONE) {
    const float *pw = p.weight[side], *pb = p.bias[side];
    if (pw) load_shared4(pw + lo, w), load_shared4(pw + hi, w + 4);
    if (pb) load_shared4(pb + lo, b), load_shared4(pb + hi, b + 4);
  }
  if (bad && c == 0) raise_status(p.status, DSA_ERR_BAD_POSITION);

  F2 w2[4], b2[4], cs2[4], sn2[4], ms2[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) w2[i] = pack(w[2 * i], w[2 * i + 1]), b2[i] = pack(b[2 * i], b[2 * i + 1]);
  // half layout: cosines and sines of two pairs; interleaved: of one, twice
#pragma unroll
  for (int i = 0; i < (INTER ? 4 : 2); ++i) {
    cs2[i] = INTER ? pack(cs[i], cs[i]) : pack(cs[2 * i], cs[2 * i + 1]);
    sn2[i] = INTER ? pack(-sn[i], sn[i]) : pack(sn[2 * i], sn[2 * i + 1]);
    if (!INTER) ms2[i] = pack(-sn[2 * i], -sn[2 * i + 1]);
  }
  const float inv_dim = 1.f / (float)p.dim;
  const float poison = bad ? CUDART_NAN_F : 1.f;
  T* y = static_cast<T*>(p.y[side]) + token * p.yt[side] + j * p.yh[side];
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    F2 v[4];
    unpack(raw[h][0], v);
    unpack(raw[h][1], v + 2);
    if (p.norm == DSA_NORM_LAYER) {
      const float s = sum2(add2(add2(v[0], v[1]), add2(v[2], v[3])));
      const float mean = group_sum<LANES>(s) * inv_dim;
      const F2 off = pack(-mean, -mean);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = FULL || mine ? add2(v[i], off) : pack(0.f, 0.f);
    }
    if (p.norm != DSA_NORM_NONE) {
      const F2 s = fma2(v[3], v[3], fma2(v[2], v[2], fma2(v[1], v[1], mul2(v[0], v[0]))));
      const float r = rsqrtf(group_sum<LANES>(sum2(s)) * inv_dim + p.eps) * poison;
      const F2 r2 = pack(r, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = fma2(mul2(v[i], r2), w2[i], b2[i]);
    } else if (bad) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = pack(poison, poison);
    }
    if (turned) {
      if (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float a0, a1;
          unpair(v[i], a0, a1);
          v[i] = fma2(v[i], cs2[i], mul2(pack(a1, a0), sn2[i]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const F2 a0 = v[i], a1 = v[2 + i];
          v[i] = fma2(a0, cs2[i], mul2(a1, ms2[i]));
          v[2 + i] = fma2(a1, cs2[i], mul2(a0, sn2[i]));
        }
      }
    }
    if (mine && h < heads) store4(y + lo, v), store4(y + hi, v + 2);
    y += p.yh[side];
  }
}

template <typename T, int LANES, int HEADS, bool INTER, bool FULL>
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
  return cudaLaunchKernelEx(&cfg, norm_rope_kernel<T, LANES, HEADS, INTER, FULL>, p);
}

template <typename T, int LANES, bool INTER>
cudaError_t launch_lanes(const NormRopeParams& p, cudaStream_t stream) {
  if (p.dim == kChunk * LANES) return launch_t<T, LANES, 4, INTER, true>(p, stream);
  return launch_t<T, LANES, 4, INTER, false>(p, stream);
}

template <typename T, bool INTER>
cudaError_t launch_dim(const NormRopeParams& p, cudaStream_t stream) {
  if (p.dim <= 64) return launch_lanes<T, 8, INTER>(p, stream);
  if (p.dim <= 128) return launch_lanes<T, 16, INTER>(p, stream);
  return launch_lanes<T, 32, INTER>(p, stream);
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
