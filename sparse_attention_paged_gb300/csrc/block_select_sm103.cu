// block_select_sm103.cu -- the k pages of every row and key head that may hold
// the largest scores, judged by the boxes around the pages' keys.
//
// For one query q the largest score that a key in a page's box could have is
//   sum_d max(q_d high_d, q_d low_d) = sum_d (q_d)+ high_d - (q_d)- low_d,
// linear in the positive and negative parts of q, so that the sum over a
// group's query heads is one dot product with P = sum_h (q_h)+ and
// N = sum_h (q_h)-.  In whole numbers:
//   i = round(q * 2^(20 - x)), 2^x above the group's largest |q|;  P, N sums of i
//   p = ceil(P / 2^s), n = ceil(N / 2^s), s the smallest with max(P, N) <= 127 * 2^s
//   score = (sum_d p_d high_d - n_d low_d) * scale        int8 products, below 2^24
// The score is exact, and with it the order and the choice: the result does
// not depend on how the work is split.  Scores past the largest float count as
// that.  NaN queries count as 0, infinities as the largest float.
//
// A block per row and key head.  8 lanes have a page: 2 D bytes of codes, four
// products an instruction.  The k-th largest score is found by its bits, 8 at
// a time (histograms in shared memory), then each thread takes its run of
// pages in order.  Bound by HBM at long rows (2 D + 4 bytes a page and head),
// by latency at short ones.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "paged_common.cuh"
#include "sm100_ptx.cuh"

namespace dsa {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kGridBits = 20;

struct Shared {
  int parts[kThreads / 64][2][128];  // partial sums of P and N
  alignas(16) uint32_t codes[64];    // p (D bytes), then -n
  float tops[kWarps];
  int sizes[kWarps];
  uint32_t hist[256];
  uint32_t sums[kWarps];
  int bad, digit, rank;
};

// Floats in the order of unsigned numbers.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float value(uint16_t u, int dtype) {
  float x = dtype == DSA_FP16 ? __half2float(__ushort_as_half(u)) : __uint_as_float((uint32_t)u << 16);
  if (x != x) x = 0.f;
  return fminf(fmaxf(x, -FLT_MAX), FLT_MAX);
}

template <int D>
__global__ void __launch_bounds__(kThreads) block_select_kernel(const BlockSelectParams p) {
  extern __shared__ uint32_t keys[];     // [W] page ids, then scores
  __shared__ Shared s;
  const int row = blockIdx.x / p.heads, head = blockIdx.x % p.heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  const int len = __ldg(p.seqlens + row);
  int* out = p.blocks + ((long long)row * p.heads + head) * p.k;
  const bool past = (long long)len > (long long)p.W * kPage;
  const int n = len <= 0 || past ? 0 : (len - 1) / kPage + 1;
  if (past && threadIdx.x == 0) raise_status(p.status, DSA_ERR_BAD_SEQLEN);
  if (threadIdx.x == 0) s.bad = 0;
  __syncthreads();
  const int* table = p.block_table + (long long)row * p.bt_stride;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int page = __ldg(table + i);
    keys[i] = (uint32_t)page;
    if (page < 0 || page >= p.num_pages) s.bad = 1;
  }
  if (n <= p.k) {                        // every page
    __syncthreads();
    const bool bad = s.bad;
    if (bad && threadIdx.x == 0) raise_status(p.status, DSA_ERR_BAD_PAGE);
    for (int i = threadIdx.x; i < p.k; i += kThreads) out[i] = i < n && !bad ? i : -1;
    return;
  }

  // the group's queries
  const uint16_t* q = p.q + (long long)row * p.q_row + (long long)head * p.group * p.q_head;
  const int d = threadIdx.x % D, part = threadIdx.x / D;
  constexpr int kParts = kThreads / D;
  float top = 0.f;
  for (int h = part; h < p.group; h += kParts) top = fmaxf(top, fabsf(value(__ldg(q + h * p.q_head + d), p.dtype)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
  if (lane == 0) s.tops[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s.tops[w]);
  int x;
  frexpf(top, &x);                       // top < 2^x
  int above = 0, below = 0;
  for (int h = part; h < p.group; h += kParts) {
    const int i = (int)rintf(scalbnf(value(__ldg(q + h * p.q_head + d), p.dtype), kGridBits - x));
    above += max(i, 0), below += max(-i, 0);
  }
  s.parts[part][0][d] = above, s.parts[part][1][d] = below;
  __syncthreads();
  int sum = 0;
  if (threadIdx.x < 2 * D) {
#pragma unroll
    for (int k = 0; k < kParts; ++k) sum += s.parts[k][threadIdx.x / D][d];
  }
  int size = sum;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) size = max(size, __shfl_xor_sync(kAll, size, o));
  if (lane == 0) s.sizes[warp] = size;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) size = max(size, s.sizes[w]);
  int shift = max(0, 25 - __clz(size | 1));  // size < 128 * 2^shift
  if (size > 127 << shift) ++shift;
  if (threadIdx.x < 2 * D) {
    const int code = (sum + (1 << shift) - 1) >> shift;
    reinterpret_cast<int8_t*>(s.codes)[threadIdx.x] = (int8_t)(threadIdx.x < D ? code : -code);
  }
  __syncthreads();
  if (s.bad) {
    if (threadIdx.x == 0) raise_status(p.status, DSA_ERR_BAD_PAGE);
    for (int i = threadIdx.x; i < p.k; i += kThreads) out[i] = -1;
    return;
  }

  // scores: 8 lanes a page, 16 bytes at a time
  constexpr int kLoads = 2 * D / 128, kTeams = kThreads / 8, kAhead = 4;
  const int team = lane / 8, l = lane % 8;
  int4 code[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) code[j] = reinterpret_cast<const int4*>(s.codes)[j * 8 + l];
  for (int first = warp * 4; first < n; first += kTeams * kAhead) {  // by the warp together
    const int i0 = first + team;
    int4 box[kAhead][kLoads];
    float scale[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int i = i0 + a * kTeams;
      // a page's id is read by its own lanes only, before they put the score there
      const long long record = (long long)(i < n ? keys[i] : 0u) * p.heads + head;
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        box[a][j] = __ldg(reinterpret_cast<const int4*>(p.bounds + record * (2 * D)) + j * 8 + l);
      scale[a] = __ldg(p.bound_scale + record);
    }
    __syncwarp();
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int i = i0 + a * kTeams;
      int dot = 0;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        dot = __dp4a(box[a][j].x, code[j].x, dot);
        dot = __dp4a(box[a][j].y, code[j].y, dot);
        dot = __dp4a(box[a][j].z, code[j].z, dot);
        dot = __dp4a(box[a][j].w, code[j].w, dot);
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);
      if (i < n && l == 0) {
        const float score = fminf(fmaxf((float)dot * scale[a], -FLT_MAX), FLT_MAX);
        keys[i] = i < p.first || i >= n - p.last ? 0xffffffffu : ordered(score + 0.f);
      }
    }
  }
  __syncthreads();

  // the k-th largest key, 8 bits at a time; `rank` of those with its upper bits are taken
  uint32_t prefix = 0;
  int rank = p.k;
#pragma unroll
  for (int at = 24; at >= 0; at -= 8) {
    for (int i = threadIdx.x; i < 256; i += kThreads) s.hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const uint32_t key = keys[i];
      if (at == 24 || key >> (at + 8) == prefix) atomicAdd(&s.hist[key >> at & 255u], 1u);
    }
    __syncthreads();
    if (warp == 0) {
      // lane: 8 digits, the largest ones first
      uint32_t c[8], mine = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) mine += c[j] = s.hist[255 - (lane * 8 + j)];
      uint32_t before = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(kAll, before, o);
        if (lane >= o) before += v;
      }
      before -= mine;
      if (before < (uint32_t)rank && (uint32_t)rank <= before + mine) {
        int j = 0;
        while (before + c[j] < (uint32_t)rank) before += c[j++];
        s.digit = 255 - (lane * 8 + j), s.rank = rank - (int)before;
      }
    }
    __syncthreads();
    prefix = prefix << 8 | (uint32_t)s.digit;
    rank = s.rank;
  }

  // a thread takes its run of pages: larger keys, and the first `rank` equal ones
  const int run = (n + kThreads - 1) / kThreads;
  const int i0 = min((int)threadIdx.x * run, n), i1 = min(i0 + run, n);
  uint32_t found = 0;                      // larger ones in the low half, equal ones in the high half
  for (int i = i0; i < i1; ++i) {
    const uint32_t key = keys[i];
    found += key > prefix ? 1u : key == prefix ? 0x10000u : 0u;
  }
  uint32_t before = found;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(kAll, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) s.sums[warp] = before;
  before -= found;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (w < warp) before += s.sums[w];
  int larger = (int)(before & 0xffffu), equal = (int)(before >> 16);
  for (int i = i0; i < i1; ++i) {
    const uint32_t key = keys[i];
    if (key > prefix) {
      out[larger + min(equal, rank)] = i;
      ++larger;
    } else if (key == prefix) {
      if (equal < rank) out[larger + equal] = i;
      ++equal;
    }
  }
}

template <int D>
cudaError_t launch_t(const BlockSelectParams& p, cudaStream_t stream) {
  static bool ready[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !ready[dev]) {
    e = cudaFuncSetAttribute(block_select_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectMaxPages * 4);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) ready[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)p.rows * p.heads));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)p.W * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_select_kernel<D>, p);
}

}  // namespace

cudaError_t launch_block_select(const BlockSelectParams& p, cudaStream_t stream) {
  return p.dim == 128 ? launch_t<128>(p, stream) : launch_t<64>(p, stream);
}

}  // namespace dsa
