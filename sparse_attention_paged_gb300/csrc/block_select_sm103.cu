// block_select_sm103.cu -- the k pages of every row and key head that may hold
// the largest scores, as the boxes around the pages' keys have it.
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
// not depend on how the work is split.  As a bound it favours boxes of a coarse scale,
// whose codes are rounded outwards by larger steps.  Scores past the largest float count as
// that.  NaN queries count as 0, infinities as the largest float.
//
// Rows with tables of their own: a cluster of up to eight blocks per row and
// key head, each with a run of the row's pages.  8 lanes have a page: 2 D bytes
// of codes, four products an instruction.  Every block finds the best k of its
// run, and the first one the best k of those.  The k-th largest by bins of equal
// width, the keys of its bin ranked by all pairs.  Bound by latency, and by HBM at
// long rows, whose later pages are few blocks' work.  Measured: 64 rows
// of 64 to 2,048 pages, 8 heads of 128, 22 us with the boxes (78.6 MB) in L2 and 27 with
// boxes that come from HBM; one row of 64 pages 5.4, of 2,048 10.3.
//
// Rows that share a table (a prompt): a block per 16 or 32 rows and key head reads the
// boxes once, multiplies them on the tensor cores, and a warp selects for a row.
// Bound by its instructions: 1,024 rows of 352 pages, 8 heads of 128 31 us with the boxes
// (9.2 MB) in L2, some 3 more with an L2 that holds nothing of them.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <limits.h>
#include <stdint.h>

#include <algorithm>

#include "paged_common.cuh"
#include "sm100_ptx.cuh"

namespace dsa {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBlocksPerSm = 2;
constexpr int kOrdered = 128;        // rows that are started by their lengths, at most
constexpr int kWarpPages = 256;      // a row of so many is one warp's to choose from: of 64 pages 5.3 us, 6.4 by the block
constexpr int kRunFull = 1024;       // pages that a block has before another one joins it, where the GPU is half full
constexpr int kGridBits = 20;
constexpr uint32_t kAlways = 0xffffffffu;  // key of a page that is taken whatever its score

// Floats in the order of unsigned numbers.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A page's key: its score's place in the order.
__device__ __forceinline__ uint32_t key_of(float dot, float scale, int i, int n, const BlockSelectParams& p) {
  const float score = fminf(fmaxf(dot * scale, -FLT_MAX), FLT_MAX);
  return i < p.first || i >= n - p.last ? kAlways : ordered(score + 0.f);
}

__device__ __forceinline__ float value(uint32_t u, int dtype) {
  float x = dtype == DSA_FP16 ? __half2float(__ushort_as_half((unsigned short)u)) : __uint_as_float(u << 16);
  if (x != x) x = 0.f;
  return fminf(fmaxf(x, -FLT_MAX), FLT_MAX);
}

// A query value on its group's grid: 2^20 times itself over the power of two
// above the group's largest magnitude.  Two factors, as one can be past 2^127;
// a product that is not exact is below 1/2.
struct Grid {
  float a, b;
  __device__ __forceinline__ explicit Grid(float top) {
    int x;
    frexpf(top, &x);                     // top < 2^x, -148 <= x <= 128
    const int e = kGridBits - x;
    a = __uint_as_float((uint32_t)(min(e, 127) + 127) << 23), b = __uint_as_float((uint32_t)(max(e - 127, 0) + 127) << 23);
  }
  __device__ __forceinline__ int operator()(float v) const { return __float2int_rn(v * a * b); }
};

// The smallest s with size <= 127 * 2^s.
__device__ __forceinline__ int code_shift(int size) {
  int shift = max(0, 25 - __clz(size | 1));  // size < 128 * 2^shift
  if (size > 127 << shift) ++shift;
  return shift;
}
__device__ __forceinline__ int code_of(int sum, int shift) { return (sum + (1 << shift) - 1) >> shift; }

__device__ __forceinline__ int dot16(int4 a, int4 b, int sum) {
  sum = __dp4a(a.x, b.x, sum);
  sum = __dp4a(a.y, b.y, sum);
  sum = __dp4a(a.z, b.z, sum);
  return __dp4a(a.w, b.w, sum);
}

// Pages of a row; 0 where its length is past the table.
__device__ __forceinline__ int row_pages(const BlockSelectParams& p, int row, bool* past) {
  const int len = __ldg(p.seqlens + row);
  *past = (long long)len > (long long)p.W * kPage;
  return len <= 0 || *past ? 0 : (len - 1) / kPage + 1;
}

// ---- the choice by one warp ------------------------------------------------------

constexpr int kWarpBins = 256;

// One warp: the best k of n > k keys in shared memory, equal ones from the front,
// in order.  Bins of equal width between the smallest and the largest score; the
// keys of the bin with the k-th largest are ranked by all pairs (those that are
// not taken fall to 0), or, where they are too many (equal scores), it is found
// bit by bit.
__device__ __forceinline__ void warp_select(uint32_t* keys, int n, int k, int lane, uint32_t* bins, int* out) {
  uint32_t low = kAlways, high = 0;
#pragma unroll 4
  for (int i = lane; i < n; i += 32) {
    const uint32_t key = keys[i];
    low = min(low, key);
    if (key != kAlways) high = max(high, key);
  }
  low = __reduce_min_sync(kAll, low), high = __reduce_max_sync(kAll, high);
  constexpr int kEach = kWarpBins / 32;
#pragma unroll
  for (int j = 0; j < kEach; ++j) bins[j * 32 + lane] = 0;
  __syncwarp();
  const int shift = high > low ? max(0, 32 - 8 - __clz(high - low)) : 0;
  static_assert(kWarpBins == 1 << 8, "the bits of a bin");
  auto bin_of = [&](uint32_t key) { return (key - low) >> shift; };
  int above = 0;
#pragma unroll 4
  for (int i = lane; i < n; i += 32) {
    const uint32_t key = keys[i];
    if (key == kAlways) ++above;
    else atomicAdd(&bins[bin_of(key)], 1u);
  }
  above = __reduce_add_sync(kAll, above);
  __syncwarp();
  // lane: bins from the top
  int c[kEach], mine = 0;
#pragma unroll
  for (int j = 0; j < kEach; ++j) mine += c[j] = (int)bins[kWarpBins - 1 - (lane * kEach + j)];
  int before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kAll, before, o);
    if (lane >= o) before += v;
  }
  above += before - mine;
  int bin = -1, rest = 0, inside = 0;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    if (above < k && k <= above + c[j]) bin = kWarpBins - 1 - (lane * kEach + j), rest = k - above, inside = c[j];
    above += c[j];
  }
  const uint32_t owner = __ballot_sync(kAll, bin >= 0);
  uint32_t least = kAlways;                // no bin: pages that are always taken are all
  int equal = n;
  if (owner) {
    const int from = __ffs(owner) - 1;
    bin = __shfl_sync(kAll, bin, from), rest = __shfl_sync(kAll, rest, from), inside = __shfl_sync(kAll, inside, from);
    least = low + ((uint32_t)bin << shift);
    if (inside > rest && inside <= 32) {
      // its keys and places beside each other, then each against all
      int count = 0;
      for (int i0 = 0; i0 < n; i0 += 32) {
        const uint32_t key = i0 + lane < n ? keys[i0 + lane] : kAlways;
        const bool in = key != kAlways && bin_of(key) == (uint32_t)bin;
        const uint32_t who = __ballot_sync(kAll, in);
        if (in) {
          const int at = count + __popc(who & ((1u << lane) - 1));
          bins[at] = key, bins[32 + at] = i0 + lane;
        }
        count += __popc(who);
      }
      __syncwarp();
      const uint32_t key = bins[lane];
      int better = 0;
      for (int j = 0; j < inside; ++j) {
        const uint32_t other = __shfl_sync(kAll, key, j);
        better += other > key || (other == key && j < lane);  // places are in order
      }
      if (lane < inside && better >= rest) keys[bins[32 + lane]] = 0u;
      __syncwarp();
    } else if (inside > rest) {
      auto count = [&](uint32_t from) {
        int sum = 0;
#pragma unroll 4
        for (int i = lane; i < n; i += 32) sum += keys[i] >= from;
        return __reduce_add_sync(kAll, sum);
      };
      for (int bit = shift - 1; bit >= 0; --bit)
        if (count(least + (1u << bit)) >= k) least += 1u << bit;
      equal = k - count(least + 1);
    }
  }
  int larger = 0, same = 0;
  const uint32_t left = (1u << lane) - 1;
  if (equal == n) {                        // all from `least` on
#pragma unroll 4
    for (int i = lane; i - lane < n; i += 32) {
      const bool take = i < n && keys[i] >= least;
      const uint32_t who = __ballot_sync(kAll, take);
      if (take) out[larger + __popc(who & left)] = i;
      larger += __popc(who);
    }
    return;
  }
  for (int i0 = 0; i0 < n; i0 += 32) {
    const bool in = i0 + lane < n;
    const uint32_t key = in ? keys[i0 + lane] : 0u;
    const uint32_t more = __ballot_sync(kAll, in && key > least), alike = __ballot_sync(kAll, in && key == least);
    const int l = larger + __popc(more & left), e = same + __popc(alike & left);
    if (in && (key > least || (key == least && e < equal))) out[l + min(e, equal)] = i0 + lane;
    larger += __popc(more), same += __popc(alike);
  }
}

// ---- rows with tables of their own ---------------------------------------------

constexpr int kBinBits = 10, kBins = 1 << kBinBits;
constexpr int kBinned = 256;         // keys of a bin that are ranked by all pairs

struct Shared {
  union {
    struct {
      int length[kOrdered], row;
    } order;
    int parts[kThreads / 64][2][128];  // partial sums of P and N
    struct {
      uint32_t bins[kBins];
      uint32_t key[kBinned];
      int index[kBinned];
    } sort;
  };
  alignas(16) uint32_t codes[64];    // p (D bytes), then -n
  float tops[kWarps];
  int sizes[kWarps > 8 ? kWarps : 8];  // of queries; then the runs' best ones, summed up
  uint32_t low[kWarps], high[kWarps], always[kWarps], sums[kWarps];
  uint32_t bin, rest, inside, listed;  // the k-th largest's bin: keys of it that are taken, keys in it
  int bad, count;                    // of this block's run: a page outside the pool, pages for the choice
};

// Sums before this thread's over the block, the threads in order; a barrier inside.
__device__ __forceinline__ uint32_t sum_before(uint32_t mine, Shared& s) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(kAll, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) s.sums[warp] = before;
  before -= mine;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (w < warp) before += s.sums[w];
  return before;
}

// Takes the k largest of n >= k keys in shared memory, equal ones from the front:
// emit(place among them, index), in the order of the indices.  As the warp does it.
template <typename F>
__device__ void block_select(uint32_t* keys, int n, int k, Shared& s, F emit) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t low = kAlways, high = 0;
  for (int i = threadIdx.x; i < kBins; i += kThreads) s.sort.bins[i] = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint32_t key = keys[i];
    low = min(low, key);
    if (key != kAlways) high = max(high, key);
  }
  low = __reduce_min_sync(kAll, low), high = __reduce_max_sync(kAll, high);
  if (lane == 0) s.low[warp] = low, s.high[warp] = high;
  if (threadIdx.x == 0) s.bin = kBins, s.rest = s.inside = s.listed = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) low = min(low, s.low[w]), high = max(high, s.high[w]);
  const int shift = high > low ? max(0, 32 - kBinBits - __clz(high - low)) : 0;
  auto bin_of = [&](uint32_t key) { return (key - low) >> shift; };
  uint32_t always = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint32_t key = keys[i];
    if (key == kAlways) ++always;
    else atomicAdd(&s.sort.bins[bin_of(key)], 1u);
  }
  always = __reduce_add_sync(kAll, always);
  if (lane == 0) s.always[warp] = always;
  __syncthreads();
  // the bin with the k-th largest, counted from the top: a few bins a thread
  constexpr int kEach = kBins / kThreads;
  uint32_t c[kEach], mine = 0;
#pragma unroll
  for (int j = 0; j < kEach; ++j) mine += c[j] = s.sort.bins[kBins - 1 - (threadIdx.x * kEach + j)];
  uint32_t above = sum_before(mine, s);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) above += s.always[w];
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    if (above < (uint32_t)k && (uint32_t)k <= above + c[j])
      s.bin = kBins - 1 - (threadIdx.x * kEach + j), s.rest = k - above, s.inside = c[j];
    above += c[j];
  }
  __syncthreads();
  const uint32_t bin = s.bin, rest = s.rest, inside = s.inside;
  // taken: keys above `least`, and the first `equal` ones that equal it
  uint32_t least = bin < kBins ? low + (bin << shift) : kAlways, equal = n;
  if (inside > rest && inside <= kBinned) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const uint32_t key = keys[i];
      if (key != kAlways && bin_of(key) == bin) {
        const uint32_t at = atomicAdd(&s.listed, 1u);
        s.sort.key[at] = key, s.sort.index[at] = i;
      }
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < inside; i += kThreads) {
      const uint32_t key = s.sort.key[i];
      const int index = s.sort.index[i];
      uint32_t better = 0;
      for (uint32_t j = 0; j < inside; ++j)
        better += s.sort.key[j] > key || (s.sort.key[j] == key && s.sort.index[j] < index);
      if (better >= rest) keys[index] = 0u;  // below every score
    }
    __syncthreads();
  } else if (inside > rest) {
    auto count = [&](uint32_t from) {
      int sum = 0;
      for (int i = threadIdx.x; i < (n + kThreads - 1) / kThreads * kThreads; i += kThreads)
        sum += __syncthreads_count(i < n && keys[i] >= from);
      return sum;
    };
    for (int bit = shift - 1; bit >= 0; --bit)
      if (count(least + (1u << bit)) >= k) least += 1u << bit;
    equal = k - count(least + 1);
  }
  const int run = (n + kThreads - 1) / kThreads;
  const int i0 = min((int)threadIdx.x * run, n), i1 = min(i0 + run, n);
  uint32_t found = 0;                      // larger ones in the low half, equal ones in the high half
  for (int i = i0; i < i1; ++i) found += keys[i] > least ? 1u : keys[i] == least ? 0x10000u : 0u;
  const uint32_t before = sum_before(found, s);
  uint32_t larger = before & 0xffffu, same = before >> 16;
  for (int i = i0; i < i1; ++i) {
    const uint32_t key = keys[i];
    if (key > least) {
      emit((int)(larger + min(same, equal)), i);
      ++larger;
    } else if (key == least) {
      if (same < equal) emit((int)(larger + same), i);
      ++same;
    }
  }
}

// Another block's shared memory.
__device__ __forceinline__ uint32_t far_address(const void* p, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(sm100::smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t far_load(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    block_select_kernel(const BlockSelectParams p, int blocks, int run_max, bool by_length) {
  extern __shared__ uint32_t keys[];     // [run_max] page ids, then keys; for more blocks than one the best of
                                         // each run: [most] keys and [most] places, then those of all
  __shared__ Shared s;
  const int rank = blockIdx.x % blocks, head = blockIdx.x / blocks % p.heads;
  int row = blockIdx.x / blocks / p.heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int most = min(run_max, p.k);
  uint32_t *best = keys + run_max, *place = best + most;
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  if (by_length) {
    // the longest rows first: blocks start in the order of their numbers
    const int i = threadIdx.x;
    if (i < p.rows) s.order.length[i] = __ldg(p.seqlens + i);
    __syncthreads();
    if (i < p.rows) {
      const int mine = s.order.length[i];
      int before = 0;
      for (int j = 0; j < p.rows; ++j) before += s.order.length[j] > mine || (s.order.length[j] == mine && j < i);
      if (before == row) s.order.row = i;
    }
    __syncthreads();
    row = s.order.row;
    __syncthreads();
  }
  bool past;
  const int n = row_pages(p, row, &past);
  int* out = p.blocks + ((long long)row * p.heads + head) * p.k;
  if (past && rank == 0 && threadIdx.x == 0) raise_status(p.status, DSA_ERR_BAD_SEQLEN);
  if (threadIdx.x == 0) s.bad = 0, s.count = 0;
  __syncthreads();
  const int run = select_run(n, blocks), begin = min(rank * run, n), mine = min(run, n - begin);
  const bool all = n <= p.k;             // every page is taken: no scores
  if (rank > 0 && mine == 0) return;     // (the cluster's barrier goes by the threads that are there)
  const int active = select_active(n, run);
  const int* table = p.block_table + (long long)row * p.bt_stride + begin;
  for (int i = threadIdx.x; i < mine; i += kThreads) {
    int page = __ldg(table + i);
    if (page < 0 || page >= p.num_pages) s.bad = 1, page = 0;
    keys[i] = (uint32_t)page;
  }
  if (mine > 0 && !all) {
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
    const Grid grid(top);
    int above = 0, below = 0;
    for (int h = part; h < p.group; h += kParts) {
      const int i = grid(value(__ldg(q + h * p.q_head + d), p.dtype));
      above += max(i, 0), below += max(-i, 0);
    }
    s.parts[part][0][d] = above, s.parts[part][1][d] = below;
    __syncthreads();
    int sum = 0;
    if (threadIdx.x < 2 * D) {
#pragma unroll
      for (int k = 0; k < kParts; ++k) sum += s.parts[k][threadIdx.x / D][d];
    }
    const int size = __reduce_max_sync(kAll, sum);
    if (lane == 0) s.sizes[warp] = size;
    __syncthreads();
    int largest = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) largest = max(largest, s.sizes[w]);
    if (threadIdx.x < 2 * D) {
      const int code = code_of(sum, code_shift(largest));
      reinterpret_cast<int8_t*>(s.codes)[threadIdx.x] = (int8_t)(threadIdx.x < D ? code : -code);
    }
    __syncthreads();

    // scores: 8 lanes a page, 16 bytes at a time
    constexpr int kLoads = 2 * D / 128, kTeams = kThreads / 8, kAhead = 4;
    const int team = lane / 8, l = lane % 8;
    int4 code[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) code[j] = reinterpret_cast<const int4*>(s.codes)[j * 8 + l];
    for (int first = warp * 4; first < mine; first += kTeams * kAhead) {  // by the warp together
      const int i0 = first + team;
      int4 box[kAhead][kLoads];
      float scale[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int i = i0 + a * kTeams;
        // a page's id is read by its own lanes only, before they put the key there
        const long long record = (long long)(i < mine ? keys[i] : 0u) * p.heads + head;
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
        for (int j = 0; j < kLoads; ++j) dot = dot16(box[a][j], code[j], dot);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);
        if (i < mine && l == 0) keys[i] = key_of((float)dot, scale[a], begin + i, n, p);
      }
    }
    __syncthreads();
    if (run < n) {
      // the best of the run
      if (mine <= p.k) {
        for (int i = threadIdx.x; i < mine; i += kThreads) best[i] = keys[i], place[i] = begin + i;
      } else {
        block_select(keys, mine, p.k, s, [&](int at, int i) { best[at] = keys[i], place[at] = begin + i; });
      }
      if (threadIdx.x == 0) s.count = min(mine, p.k);
    }
  }
  if (active > 1) {
    cluster_sync();
    if (rank == 0) {
      // where each run's best go among all, and whether a page was bad
      uint32_t *all_keys = place + most, *all_places = all_keys + blocks * most;
      if (warp == 0) {
        const bool other = lane < active;
        const int count = other ? (int)far_load(far_address(&s.count, lane)) : 0;
        const bool bad = __any_sync(kAll, other && far_load(far_address(&s.bad, lane)));
        int before = count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(kAll, before, o);
          if (lane >= o) before += v;
        }
        if (other) s.sizes[lane] = before;
        __syncwarp();
        if (lane == 0) s.bad = bad;
      }
      __syncthreads();
      const int total = s.sizes[active - 1];
      for (int i = threadIdx.x; i < total; i += kThreads) {
        int r = 0;
        while (i >= s.sizes[r]) ++r;
        const int at = r ? i - s.sizes[r - 1] : i;
        all_keys[i] = far_load(far_address(best + at, r)), all_places[i] = far_load(far_address(place + at, r));
      }
      __syncthreads();
      if (!s.bad && !all && run < n) {
        // no more than k candidates only where the row has no more pages
        block_select(all_keys, total, p.k, s, [&](int at, int i) { out[at] = (int)all_places[i]; });
      }
    }
    cluster_sync();                      // nobody leaves while its memory is read
    if (rank > 0) return;
  } else {
    __syncthreads();
  }
  if (s.bad) {
    if (threadIdx.x == 0) raise_status(p.status, DSA_ERR_BAD_PAGE);
    for (int i = threadIdx.x; i < p.k; i += kThreads) out[i] = -1;
  } else if (all) {
    for (int i = threadIdx.x; i < p.k; i += kThreads) out[i] = i < n ? i : -1;
  } else if (run >= n && n <= kWarpPages) {
    if (warp == 0) warp_select(keys, n, p.k, lane, s.sort.bins, out);
  } else if (run >= n) {
    block_select(keys, n, p.k, s, [&](int at, int i) { out[at] = i; });
  }
}

// ---- rows that share a table ------------------------------------------------------

constexpr int kTileThreads = 512, kTileWarps = kTileThreads / 32;
constexpr int kTileMorePages = 512;     // keys of 32 rows: two such blocks are on an SM
constexpr int kTileMaxPages = 2048;      // keys of 16 rows in shared memory: 130 KB

// Keys of a row in shared memory: eight rows' pairs of keys are in 32 banks.
constexpr int tile_stride(int W) { return (W + 31) / 32 * 32 + 8; }
constexpr int tile_smem(int rows, int W) { return (rows * tile_stride(W) + W) * 4; }

// D += A * B, 16 rows x 16 values (fp16), 8 columns, fp32.
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four 8-bit whole numbers as fp16: the byte plus 128 under the exponent of 1024.
__device__ __forceinline__ void halves(uint32_t x, uint32_t& low, uint32_t& high) {
  x ^= 0x80808080u;
  const uint32_t u[2] = {__byte_perm(x, 0x64646464u, 0x4140), __byte_perm(x, 0x64646464u, 0x4342)};
  const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
  const __half2 l = __hsub2(*reinterpret_cast<const __half2*>(&u[0]), off);
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u[1]), off);
  low = *reinterpret_cast<const uint32_t*>(&l), high = *reinterpret_cast<const uint32_t*>(&h);
}

// kRows, 16 or 32, rows a block.
template <int D, int kRows>
__global__ void __launch_bounds__(kTileThreads, 2) block_select_tile_kernel(const BlockSelectParams p) {
  extern __shared__ uint32_t keys[];     // [kRows][stride], then the table's page ids
  const int stride = tile_stride(p.W);
  int* ids = reinterpret_cast<int*>(keys + kRows * stride);
  __shared__ alignas(16) uint16_t codes[kRows][2 * D + 8];  // p, then -n, as fp16; rows in other banks
  __shared__ uint32_t bins[kTileWarps][kWarpBins];
  __shared__ int pages[kRows];
  __shared__ int bad_at;                 // the first page of the table that is not in the pool
  const int row0 = blockIdx.x / p.heads * kRows, head = blockIdx.x % p.heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  if (threadIdx.x == 0) bad_at = INT_MAX;
  if (threadIdx.x < kRows) {
    bool past = false;
    pages[threadIdx.x] = row0 + threadIdx.x < p.rows ? row_pages(p, row0 + threadIdx.x, &past) : 0;
    if (past) raise_status(p.status, DSA_ERR_BAD_SEQLEN);
  }
  __syncthreads();
  int n_max = 0;
  uint32_t scored = 0;                   // rows that need scores
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    n_max = max(n_max, pages[r]);
    if (pages[r] > p.k) scored |= 1u << r;
  }
  for (int i = threadIdx.x; i < n_max; i += kTileThreads) {
    int page = __ldg(p.block_table + i);
    if (page < 0 || page >= p.num_pages) atomicMin(&bad_at, i), page = 0;
    ids[i] = page;
  }
  // a warp's rows' codes: D / 32 values a lane
  constexpr int kEach = D / 32;
  for (int r = warp; r < kRows; r += kTileWarps) {
    if (!(scored >> r & 1)) continue;
    const uint16_t* q =
        p.q + (long long)(row0 + r) * p.q_row + (long long)head * p.group * p.q_head + lane * kEach;
    auto load = [&](int h, float (&v)[kEach]) {
      uint32_t u[kEach / 2];
      if (kEach == 4) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(q + h * p.q_head));
        u[0] = w.x, u[kEach / 2 - 1] = w.y;
      } else {
        u[0] = __ldg(reinterpret_cast<const uint32_t*>(q + h * p.q_head));
      }
#pragma unroll
      for (int j = 0; j < kEach; ++j) v[j] = value(j & 1 ? u[j / 2] >> 16 : u[j / 2] & 0xffffu, p.dtype);
    };
    // The first eight heads' values stay in registers for the second pass: 1,024 rows of
    // 352 pages, 8 groups of 4 heads, 27.1 us for 28.4.
    constexpr int kKept = 8;
    float top = 0.f, v[kEach], kept[kKept][kEach];
    auto largest = [&](const float (&x)[kEach]) {
#pragma unroll
      for (int j = 0; j < kEach; ++j) top = fmaxf(top, fabsf(x[j]));
    };
#pragma unroll
    for (int h = 0; h < kKept; ++h)
      if (h < p.group) load(h, kept[h]), largest(kept[h]);
    for (int h = kKept; h < p.group; ++h) load(h, v), largest(v);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    const Grid grid(top);
    int above[kEach] = {}, below[kEach] = {}, size = 0;
    auto add = [&](const float (&x)[kEach]) {
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int i = grid(x[j]);
        above[j] += max(i, 0), below[j] += max(-i, 0);
      }
    };
#pragma unroll
    for (int h = 0; h < kKept; ++h)
      if (h < p.group) add(kept[h]);
    for (int h = kKept; h < p.group; ++h) load(h, v), add(v);
#pragma unroll
    for (int j = 0; j < kEach; ++j) size = max(size, max(above[j], below[j]));
    const int shift = code_shift(__reduce_max_sync(kAll, size));
    uint16_t* to = codes[r] + lane * kEach;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      to[j] = __half_as_ushort(__int2half_rn(code_of(above[j], shift)));
      to[D + j] = __half_as_ushort(__int2half_rn(-code_of(below[j], shift)));
    }
  }
  __syncthreads();
  if (scored) {
    // Products of the rows and 16 pages, whole numbers below 2^24 in fp32: exact.  A
    // dot product may take its values in any order, so that lane t of four reads
    // units t, t + 4, ... of 16 codes of a page as they lie, and rows likewise.
    constexpr int kUnits = 2 * D / 64, kTiles = kRows / 16;  // units of a lane, tiles of 16 rows
    const int g = lane >> 2, t = lane & 3;
    auto record = [&](int i) { return (long long)(i < n_max ? ids[i] : 0) * p.heads + head; };
    for (int first = warp * 16; first < n_max; first += kTileWarps * 16) {
      int4 box[2][kUnits];
      float scale[2][2];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int4* from = reinterpret_cast<const int4*>(p.bounds + record(first + 8 * w + g) * (2 * D)) + t;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) box[w][u] = __ldg(from + 4 * u);
#pragma unroll
        for (int j = 0; j < 2; ++j) scale[w][j] = __ldg(p.bound_scale + record(first + 8 * w + 2 * t + j));
      }
      float c[kTiles][2][4] = {};
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
#pragma unroll
        for (int v = 0; v < 2; ++v) {      // halves of a unit: 8 codes
          uint32_t x[2][4];
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            halves(v ? box[w][u].z : box[w][u].x, x[w][0], x[w][1]);
            halves(v ? box[w][u].w : box[w][u].y, x[w][2], x[w][3]);
          }
#pragma unroll
          for (int m = 0; m < kTiles; ++m) {
            const uint4 a = *reinterpret_cast<const uint4*>(codes[16 * m + g] + (t + 4 * u) * 16 + v * 8);
            const uint4 b = *reinterpret_cast<const uint4*>(codes[16 * m + g + 8] + (t + 4 * u) * 16 + v * 8);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              mma16816(c[m][w], a.x, b.x, a.y, b.y, x[w][0], x[w][1]);
              mma16816(c[m][w], a.z, b.z, a.w, b.w, x[w][2], x[w][3]);
            }
          }
        }
#pragma unroll
      for (int m = 0; m < kTiles; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 16 * m + g + 8 * h, n = pages[r];
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int i = first + 8 * w + 2 * t + j;
              if (i < n) keys[r * stride + i] = key_of(c[m][w][2 * h + j], scale[w][j], i, n, p);
            }
        }
    }
  }
  __syncthreads();
  for (int r = warp; r < kRows; r += kTileWarps) {
    if (row0 + r >= p.rows) continue;
    int* out = p.blocks + ((long long)(row0 + r) * p.heads + head) * p.k;
    const int n = pages[r];
    if (bad_at < n) {
      if (lane == 0) raise_status(p.status, DSA_ERR_BAD_PAGE);
      for (int i = lane; i < p.k; i += 32) out[i] = -1;
    } else if (n <= p.k) {
      for (int i = lane; i < p.k; i += 32) out[i] = i < n ? i : -1;
    } else {
      warp_select(keys + r * stride, n, p.k, lane, bins[warp], out);
    }
  }
}

template <typename K, typename... A>
cudaError_t launch(K kernel, long long grid, int threads, size_t smem, int cluster, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D>
cudaError_t launch_t(const BlockSelectParams& p, int sms, cudaStream_t stream) {
  static bool ready[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !ready[dev]) {
    e = cudaFuncSetAttribute(block_select_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelectMaxPages * 4);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(block_select_tile_kernel<D, 16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             tile_smem(16, kTileMaxPages));
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(block_select_tile_kernel<D, 32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             tile_smem(32, kTileMorePages));
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) ready[dev] = true;
  }
  const long long items = (long long)p.rows * p.heads, slots = (long long)sms * kBlocksPerSm;
  // Rows of a shared table by 16 once they fill the GPU: 352 pages, 8 heads, 32
  // rows 11.0 us and 17.4 by 16, 64 rows 21.2 and 17.5, 256 rows 62.9 and 17.7; 2,048
  // pages, 32 rows 25.4 and 52.6, 64 rows 47.6 and 52.8, 256 rows 147 and 53.
  // 32 rows a block read and unpack a box once for two products and take 1.73 times as
  // long as 16: where the SM with most blocks has less to do that way, and not with one on
  // an SM (608 rows 19.2 us and 15.7 by 16).  8 heads, rows that end at
  // 352 pages: 700 rows 27.0 us and 24.4 by 16, 1,024 rows 27.1 and 30.0, 2,048 rows
  // 51.5 and 51.9, 4,096 rows 87.8 and 97.3; at 128 pages 1,024 rows 18.0 and 19.7.
  if (p.bt_stride == 0 && items > slots && p.W <= kTileMaxPages) {
    const long long few = ((long long)p.rows + 15) / 16 * p.heads, more = ((long long)p.rows + 31) / 32 * p.heads;
    const long long deep = (more + sms - 1) / sms;
    if (p.W <= kTileMorePages && deep > 1 && 7 * deep < 4 * ((few + sms - 1) / sms))
      return launch(block_select_tile_kernel<D, 32>, more, kTileThreads, tile_smem(32, p.W), 1, stream, p);
    return launch(block_select_tile_kernel<D, 16>, few, kTileThreads, tile_smem(16, p.W), 1, stream, p);
  }
  // More blocks than one for a row while all of them are on the GPU together (the
  // blocks of a cluster start and end together, and with more of them than fit
  // the cluster's idle ones keep others out): past 512 pages, from 256 a block on, and
  // where they fill half of the GPU from 1,024 on.  8 heads, one row of 512 pages 10.8
  // us and 10.2 by one block, of 2,048 11.2 and 19.3, of 8,192 16.7 and 51.4; 16 rows of
  // 1,024 pages 16.3 and 14.0, of 4,096 29.7 and 34.6.  A list of many entries leaves no room
  // for all blocks' best ones beside each other.
  int blocks = 1;
  while (blocks < 8 && 2 * blocks * items <= slots && p.k <= kSelectMaxList && p.W > 2 * kSelectRun &&
         blocks * (4 * blocks * items > slots ? kRunFull : kSelectRun) < p.W)
    blocks *= 2;
  const int run = select_run(p.W, blocks), most = std::min(run, p.k);
  const size_t smem = 4 * (size_t)(blocks > 1 ? run + 2 * most + 2 * blocks * most : run);
  return launch(block_select_kernel<D>, items * blocks, kThreads, smem, blocks, stream, p, blocks, run,
                items > slots && p.rows <= kOrdered);
}

}  // namespace

cudaError_t launch_block_select(const BlockSelectParams& p, int sms, cudaStream_t stream) {
  return p.dim == 128 ? launch_t<128>(p, sms, stream) : launch_t<64>(p, sms, stream);
}

}  // namespace dsa
