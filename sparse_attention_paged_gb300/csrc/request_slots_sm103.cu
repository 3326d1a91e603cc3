// request_slots_sm103.cu -- block tables and slot maps from the requests'
// lengths: request b holds c_b tokens and gets n_b new ones, for which it
// takes the next ceil((c_b + n_b) / 64) - ceil(c_b / 64) pages of the free list,
// requests in order.  One that wants more pages than are left takes none, and
// those behind it go on from the same place of the list.
//
//   pages   o_b = sum of the pages taken before b; while the list is long enough for
//           all, those wanted; else a warp walks the requests, 32 at a time
//   tokens  cu_b = sum of n before b; token i, cu_b <= i < cu_{b+1}, has position
//           c_b + i - cu_b and the slot page * 64 + position % 64
//
// A token of a fresh page knows its place in the free list, and the one at the
// page's start enters the page into the table: no thread waits for another's
// store.  Every block takes the sums over all requests for itself (8 bytes a
// request, from L2) and then looks its tokens' requests up in shared memory.
// Bound by latency: the lengths, then the table or the free list, then stores.
// Measured: 3.2 us a call for a decode step of 64 requests, 3.4 for 23 prompts of
// 23,400 tokens.  Lists that end: 1,024 requests that each want a page, 500 left,
// 10.3 us (3.5 with enough; 52 with one thread that walks them).
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "paged_common.cuh"
#include "sm100_ptx.cuh"

namespace dsa {

namespace {

constexpr int kThreads = 256, kChunk = 1024;   // threads of a block, requests at a time
constexpr int kPer = kChunk / kThreads;
constexpr int kMaxPage = INT_MAX / kPage;      // past it a slot does not fit 32 bits

struct Shared {
  long long tokens[kThreads / 32], pages[kThreads / 32];
  long long cu[kChunk + 1];      // tokens before each request
  long long take[kChunk];        // pages before it; -1: it gets none
  int cached[kChunk], want[kChunk];
  long long given;               // pages that requests up to the chunk's end got
};

__global__ void __launch_bounds__(kThreads) request_slots_kernel(const RequestSlotsParams p) {
  __shared__ Shared s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  const long long t0 = (long long)blockIdx.x * kThreads, t1 = min(t0 + kThreads, (long long)p.n);
  const long long token = t0 + threadIdx.x;
  const bool first = blockIdx.x == 0;
  long long tokens = 0, pages = 0, taken = 0;  // before the chunk; up to the last request that got pages
  bool found = false;
  for (int r0 = 0; r0 < p.n_req; r0 += kChunk) {
    int c[kPer], n[kPer], want[kPer];
    long long my_tokens = 0, my_pages = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int r = r0 + threadIdx.x * kPer + j;
      c[j] = r < p.n_req ? __ldg(p.lengths + r) : 0;
      n[j] = r < p.n_req ? __ldg(p.fresh + r) : 0;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool bad = c[j] < 0 || n[j] < 0 || (long long)c[j] + n[j] > (long long)p.W * kPage;
      want[j] = bad ? -1 : ((c[j] + n[j] + kPage - 1) / kPage - (c[j] + kPage - 1) / kPage);
      n[j] = max(n[j], 0);
      my_tokens += n[j], my_pages += max(want[j], 0);
    }
    // sums over the block
    long long a = my_tokens, b = my_pages;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
      if (lane >= o) a += x, b += y;
    }
    if (lane == 31) s.tokens[warp] = a, s.pages[warp] = b;
    const long long given = pages;
    a += tokens - my_tokens, b += pages - my_pages;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) a += s.tokens[w], b += s.pages[w];
      tokens += s.tokens[w], pages += s.pages[w];
    }
    const bool enough = pages <= p.n_free;      // for all up to the chunk's end
    if (!enough) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) s.want[threadIdx.x * kPer + j] = want[j];
      __syncthreads();
      if (warp == 0) {
        int at = (int)given;                    // (at most n_free)
        for (int i0 = 0; i0 < min(kChunk, p.n_req - r0); i0 += 32) {
          const int w = s.want[i0 + lane];
          bool open = w > 0;                    // not decided yet
          int mine = w == 0 ? at : -1;
          while (true) {
            // whoever wants more than is left has lost; among the others, whoever does with
            // those before it
            const int left = p.n_free - at;
            open = open && w <= left;
            const int v = open ? w : 0;
            int before = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int x = __shfl_up_sync(0xffffffffu, before, o);
              if (lane >= o) before += x;
            }
            before -= v;
            const uint32_t over = __ballot_sync(0xffffffffu, open && before + v > left);
            const int end = over ? __ffs(over) - 1 : 32;
            if (open && lane < end) mine = at + before;
            open = open && lane > end;
            at += __shfl_sync(0xffffffffu, end < 32 ? before : before + v, min(end, 31));
            if (!over) break;
          }
          s.take[i0 + lane] = mine;
        }
        if (lane == 0) s.given = at;
      }
      __syncthreads();
      pages = s.given;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = threadIdx.x * kPer + j, r = r0 + i;
      if (!enough) b = r < p.n_req ? s.take[i] : 0;
      const bool got = want[j] >= 0 && b >= 0;
      s.cu[i] = a, s.take[i] = got ? b : -1, s.cached[i] = c[j];
      if (first && r < p.n_req) {
        if (p.seqlens) p.seqlens[r] = got ? c[j] + n[j] : 0;
        if (p.cu) p.cu[r] = (int)min(a, (long long)INT_MAX);
        if (!got) raise_status(p.status, want[j] < 0 ? DSA_ERR_BAD_SEQLEN : DSA_ERR_BAD_PAGE);
        else if (want[j] > 0) taken = b + want[j];
      }
      a += n[j], b += max(want[j], 0);
    }
    if (threadIdx.x == kThreads - 1) s.cu[kChunk] = a;
    __syncthreads();
    if (!found && token < t1 && token >= s.cu[0] && token < s.cu[kChunk]) {
      found = true;
      int low = 0, high = kChunk;              // cu[low] <= token < cu[high]
      while (high - low > 1) {
        const int mid = (low + high) / 2;
        if (s.cu[mid] <= token) low = mid;
        else high = mid;
      }
      int slot = -1, pos = 0;
      if (s.take[low] >= 0) {
        const int held = s.cached[low];
        pos = held + (int)(token - s.cu[low]);
        const int block = pos / kPage, have = (held + kPage - 1) / kPage;
        int* entry = p.block_table + (long long)(r0 + low) * p.bt_stride + block;
        int page;
        if (block < have) {
          page = *entry;
        } else {
          page = __ldg(p.free_pages + s.take[low] + (block - have));
          if (pos % kPage == 0) *entry = page;
        }
        if (page >= 0 && page < kMaxPage) slot = page * kPage + pos % kPage;
        else raise_status(p.status, DSA_ERR_BAD_PAGE);
      }
      p.slots[token] = slot;
      if (p.positions) p.positions[token] = pos;
    }
    __syncthreads();                            // the sums before the next chunk's
  }
  if (!found && token < t1) {
    p.slots[token] = -1;
    if (p.positions) p.positions[token] = 0;
  }
  if (!first) return;
  if (threadIdx.x == 0) {
    if (p.cu) p.cu[p.n_req] = (int)min(tokens, (long long)INT_MAX);
    if (tokens > p.n) raise_status(p.status, DSA_ERR_BAD_SEQLEN);
  }
  if (p.used) {
    // pages are given in order, so that the last one given counts them
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
    if (lane == 0) s.pages[warp] = taken;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kThreads / 32; ++w) taken = max(taken, s.pages[w]);
      *p.used = (int)taken;
    }
  }
}

}  // namespace

cudaError_t launch_request_slots(const RequestSlotsParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n > 0 ? (unsigned)(((long long)p.n + kThreads - 1) / kThreads) : 1);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, request_slots_kernel, p);
}

}  // namespace dsa
