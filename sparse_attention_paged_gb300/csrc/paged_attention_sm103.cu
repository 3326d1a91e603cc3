// paged_attention_sm103.cu -- attention of one query token per row over a
// paged cache of keys and values with grouped heads (Hq query heads share Hkv
// key and value heads):
//
//   s[t]   = scale * q[r, h] . k[t, h / group]        t < seqlens[r], or the
//   out    = sum_t softmax(s)[t] v[t, h / group]      tokens of the listed pages
//   lse    = log sum_t exp(s[t])
//
// One pass over the tokens with a running maximum and sum per head.  A page of
// 64 tokens of one key head, keys and values, is a stage of a ring in shared
// memory that TMA fills through the pools' own strides; four warps take 16 of
// its tokens each, with the tokens (and then the values) on the M side of the
// products and eight heads a column tile on the N side:
//
//   S^T [16 tokens x 8 heads] = K (A) * Q^T (B)       m16n8k16, fp32 sums
//   O^T [D x 8 heads]        += V^T (A) * P^T (B)
//
// Q's fragments stay in registers, and so does O^T; P^T is S^T's fragments
// after one 8 x 8 transpose in registers.  The order of the values in a dot
// product is free: lane t of four takes the 16-byte units 2t and 2t + 1 of a
// key's 128 bytes as they lie, with the queries in the same order, so that keys
// are read 16 bytes at a time without a bank conflict.  The reference of the
// running softmax is raised only when a score passes it by 2^8, which one vote
// finds out: sums are fp32, so that it changes no relative precision.  Each warp
// has its own; the four meet once a row, in the row's last stage.
//
// Decode reads 2 D values per token for 4 D * group operations: 16 operations
// a byte at 8 heads a group, where 285 would balance HBM and tensor cores.
// Warp-level products leave S and P in registers; through tensor memory they
// would take two more trips and barriers a page for tensor time that is not
// missed.
//
// fp8 cache: codes become fp16, which holds e4m3 exactly.  A head's queries are
// scaled to a largest magnitude below 2^14 by a power of two; scores take the
// token's key scale; the weights take its value scale before they are rounded
// to fp16, under a reference of their own that follows the largest weight *
// scale: that lies between 2^6 and 2^15, and a token's weight is rounded by
// 2^-11 of itself down to 2^-20 of it, and by 2^-31 of it below.  That reference is
// held as its distance from the scores': a score past 2^24 has no room for a scale's
// exponent beside it.
// 16-bit caches: the weights are rounded to the cache's type (2^-8 of
// themselves for bf16, 2^-11 for fp16, 2^-25 of the largest where it is below
// fp16's normal numbers), independently from token to token.
//
// Work: pages of one key head (a group of more than 32 query heads is several),
// rows in order, cut into equal slices, one per CTA.  A row that a
// slice cuts leaves partial sums in the workspace, joined by a second kernel in
// the order of the slices: the same bits every time.  Few short rows are not cut
// by slices but shared by the CTAs of a cluster, in one launch.
//
// Measured: 64 rows of 512 to 32,768 bf16 tokens, 32 heads on 8, 128 values, 300 us
// (6.9 TB/s, a little above the rate of a copy, half of which are writes); one row of
// 131,072 fp8 tokens, 64 heads, 52 (277 MB: 41 at that rate, start 5, last results and
// join 6); 64 rows of 32 listed fp8 pages 55; 1,024 prefill rows of 16 listed bf16 pages
// 141 back to back in a graph, 145 as calls (2.1 GB through L2, 15 TB/s); one row of
// 1,024 tokens 6.5 (32 heads on 8).
//
// Warps: the last one walks the slice (lengths, list, table; 32 pages at a
// time) and issues TMA, the others compute.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "paged_common.cuh"
#include "sm100_ptx.cuh"
#include "tensor_maps.cuh"

#ifndef DSA_WAIT_LIMIT_CYCLES
#define DSA_WAIT_LIMIT_CYCLES 4000000000ll
#endif

namespace dsa {

namespace {

using namespace sm100;

// at most about a second: the clock's low 32 bits are compared
constexpr uint32_t kWaitLimit = DSA_WAIT_LIMIT_CYCLES < 2000000000ll ? DSA_WAIT_LIMIT_CYCLES : 2000000000ll;
constexpr unsigned kAll = 0xffffffffu;

// What a row's (a head tile's) beginning and end cost beside its pages, in pages of
// so many bytes: the split counts them, so that a slice of short rows has fewer
// pages.  19 rows of 1 to 9,001 tokens, 35 heads on 5, 64 values: 18.6 us without,
// 14.4 with 32 to 128 KB; rows that are alike take the same time.
constexpr int row_start(int page_bytes) { return 65536 / page_bytes; }

// Shapes of one instance: cache type, values per head, column tiles of 8 query
// heads per warp, sets of four warps with heads of their own, and whether a
// cluster's CTAs share a row.
template <int KV, int D, int NT, int MT, bool CL>
struct Shape {
  static constexpr bool kFp8 = KV == DSA_KV_FP8_E4M3;
  static constexpr int kRowBytes = D * (kFp8 ? 1 : 2);
  static constexpr int kBoxBytes = kRowBytes < 128 ? kRowBytes : 128;
  static constexpr int kBoxes = kRowBytes / kBoxBytes;
  static constexpr int kBox = kPage * kBoxBytes;               // bytes of one box in shared memory
  static constexpr int kSide = kPage * kRowBytes;              // keys or values of a page
  static constexpr int kHeadsMax = 8 * NT * MT;
  static constexpr int kScaleBytes = kFp8 ? kPage * 4 : 0;
  static constexpr int kOffScale = 2 * kSide;
  static constexpr int kOffQ = kOffScale + 2 * kScaleBytes;
  static constexpr int kStage = (kOffQ + kHeadsMax * D * 2 + 1023) / 1024 * 1024;
  static constexpr int kCtas = MT == 1 ? 2 : 1;                // per SM
  static constexpr int kStart = row_start(2 * kSide);
  static constexpr int kConsumers = 4 * MT;                    // warps
  static constexpr int kThreads = (kConsumers + 1) * 32;
  static constexpr int kMisc = 4096;
  static constexpr int kRoom = (233472 / kCtas - 1024 - 1024 - kMisc) / kStage;
  static constexpr int kStages = (kRoom < 8 ? kRoom : 8) - CL;  // a cluster's CTAs exchange results in the last one
  static constexpr int kOffSums = kStages * kStage;            // [heads][D] sums, then [heads][4] statistics
  static constexpr int kOffMisc = (kStages + CL) * kStage;
  static constexpr int kSmem = kOffMisc + kMisc + 1024;
  // the four token slices of a row meet in a stage's keys and values, some columns at a time
  static constexpr int kWant = 4 * kHeadsMax * D * 4 / (2 * kSide), kPasses = kWant < 1 ? 1 : kWant;
  static constexpr int kCols = D / kPasses;
  static_assert(kStages >= 2 && kSmem <= 232448 && kCols >= 8 && kPasses * kCols == D, "shape");
  static_assert(kHeadsMax * (D + 4) * 4 <= kStage, "results of a cluster's CTA");
};

struct Misc {
  uint64_t full[8], empty[8];
  uint64_t meet;                 // the consumer warps' own barrier
  int4 meta[8];                  // per stage: row, tile, tokens | flags, last CTA of a row that is cut
  int scan[16];
  int begin, end, share, total;  // the slice, places per CTA, places in all
  int row, tile, place;          // where it begins, in its row's tile
  int rank;                      // in a cluster
  // per consumer warp and head: reference of the scores, distance to that of the sums, total.  Two of
  // them in turn: a warp may reach the end of the next row while another still
  // reads those of this one.
  float stat[2][8][16][3];
};
static_assert(sizeof(Misc) <= 4096, "misc");
// flags of a stage beside its tokens (0 to 64)
constexpr int kBegin = 1 << 8;   // a row (or a piece of it) begins: reset, and queries come with it
constexpr int kEnd = 1 << 9;     // ... ends
constexpr int kWhole = 1 << 10;  // the piece is the whole row
constexpr int kFirst = 1 << 11;  // the piece has the row's first unit
constexpr int kBad = 1 << 12;    // a page that it needs is not in the pool
constexpr int kDone = 1 << 13;   // the slice ends here: no unit

// A reference is raised to the largest score when one is this far above it
// (log2 units), and fp8's weights * value scales are 2^kBelow at theirs.
constexpr float kAbove = 8.f, kBelow = 6.f, kSmallest = 1.f / 64.f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// With results below 2^-126, down to 2^-149.
__device__ __forceinline__ float ex2_small(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// References before any token: of the scores, and (fp8) the distance to that of the weights *
// value scales.  fp8's are finite, so that differences of two of them are no NaN.
template <bool FP8>
__device__ __forceinline__ float no_top() {
  return FP8 ? -3e38f : -CUDART_INF_F;
}
template <bool FP8>
__device__ __forceinline__ float no_distance() {
  return FP8 ? -1e30f : 0.f;
}
// A partial result's distance from a reference of the scores above its own, and the factor from
// its sums to the largest distance of all.
template <bool FP8>
__device__ __forceinline__ float distance(float top, float ref, float above) {
  return FP8 ? (top - above) + ref : 0.f;
}
template <bool FP8>
__device__ __forceinline__ float factor(float top, float ref, float above, float high) {
  if (FP8) return ex2((top - above) + ref - high);
  return top == -CUDART_INF_F ? 0.f : ex2(top - above);
}

template <bool FP16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (FP16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The transpose of 8 x 8 values of 16 bits: lane 4 g + t has row g, columns 2 t and 2 t + 1.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t at, float4 v) {
  asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(at), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}
__device__ __forceinline__ void ldmatrix_t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}

// Four e4m3 codes as two pairs of fp16 values.
__device__ __forceinline__ void widen4(uint32_t codes, uint32_t& low, uint32_t& high) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(low), "=r"(high)
      : "r"(codes));
}

template <bool FP16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (FP16) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1,
                                            int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// `bytes` (a multiple of 16, both addresses 16-byte aligned) to shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint64_t* bar, uint32_t bytes) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// A wait of a whole warp (every lane asks and gets the same answer).  After
// one that ran out the rest return at once.
struct Waiter {
  int* status;
  bool ok;
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) {
    if (!ok) return false;
    if (__all_sync(kAll, mbar_try_wait(bar, parity))) return true;
    const uint32_t t0 = (uint32_t)clock();
#pragma unroll 1
    do {
      if (__all_sync(kAll, mbar_try_wait(bar, parity))) return true;
      ok = !__any_sync(kAll, (uint32_t)clock() - t0 > kWaitLimit);
    } while (ok);
    raise_status(status, DSA_ERR_TIMEOUT);
    return false;
  }
};

// Units of a row: its pages, or its list's entries (those that name no page of
// the row are passed over).  None for a row without tokens, or with more than
// its table has room for.
__device__ __forceinline__ int row_units(const PagedAttnParams& p, int len) {
  if (len <= 0 || (long long)len > (long long)p.W * kPage) return 0;
  return p.blocks ? p.k : (len - 1) / kPage + 1;
}

// The call's pages lie on a line, rows and their head tiles in order, with `start`
// places without a page before each tile's first; it is cut into equal slices.
// Where the CTA's slice begins and ends.  All threads.
template <int THREADS>
__device__ void find_slice(const PagedAttnParams& p, Misc* m, int start) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_row = p.heads * p.tiles, each = (p.rows + THREADS - 1) / THREADS;
  const int r0 = min((int)threadIdx.x * each, p.rows), r1 = min(r0 + each, p.rows);
  auto places = [&](int r) {
    const int n = row_units(p, __ldg(p.seqlens + r));
    return n ? n + start : 0;
  };
  int mine = 0;
  for (int r = r0; r < r1; ++r) mine += places(r) * per_row;
  int before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kAll, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) m->scan[warp] = before;
  before -= mine;
  __syncthreads();
  int total = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += m->scan[w];
    total += m->scan[w];
  }
  const int share = max(1, (int)(((long long)total + gridDim.x - 1) / gridDim.x));
  const int begin = (int)min((long long)blockIdx.x * share, (long long)total);
  const int end = (int)min((long long)begin + share, (long long)total);
  if (threadIdx.x == 0) m->begin = begin, m->end = end, m->share = share, m->total = total;
  if (begin >= before && begin < before + mine) {
    int at = before;
    for (int r = r0; r < r1; ++r) {
      const int n = places(r), all = n * per_row;
      if (begin < at + all) {
        m->row = r, m->tile = (begin - at) / n, m->place = (begin - at) % n;
        break;
      }
      at += all;
    }
  }
  __syncthreads();
}

// The same for a CTA of a cluster, which shares the pages of one row and head tile.
__device__ void cluster_slice(const PagedAttnParams& p, Misc* m, int ctas, int start) {
  if (threadIdx.x == 0) {
    const int rank = blockIdx.x % ctas, item = blockIdx.x / ctas, per_row = p.heads * p.tiles;
    const int n = row_units(p, __ldg(p.seqlens + item / per_row)), share = max(1, (n + ctas - 1) / ctas);
    m->row = item / per_row, m->tile = item % per_row, m->rank = rank, m->total = n, m->share = share;
    m->place = m->begin = start + min(rank * share, n), m->end = min(m->begin + share, start + n);
  }
  __syncthreads();
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// 16 bytes of another CTA's shared memory; `at` is the address in this one's.
__device__ __forceinline__ float4 far_load(uint32_t at, int rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// ---- the warp that loads ------------------------------------------------------

template <int KV, int D, int NT, int MT, bool CL>
__device__ void produce(const PagedAttnParams& p, const CUtensorMap* kmap, const CUtensorMap* vmap, Misc* m,
                        uint32_t stages) {
  using S = Shape<KV, D, NT, MT, CL>;
  const int lane = threadIdx.x & 31;
  Waiter wait{p.status, true};
  int stage = 0, issued = 0;
  uint32_t phase = 1;                       // of the next empty wait: the first round passes
  int left = m->end - m->begin;
  if (left > 0) {
    int row = m->row, tile = m->tile, place = m->place;
    int len = __ldg(p.seqlens + row), n = row_units(p, len);
    int at = m->begin;                      // index of `place` among all
    bool fresh = true;                      // the piece has had no stage yet
    int bad = 0;
    while (left > 0 && wait.ok) {
      const int head = tile / p.tiles, skip = min(max(S::kStart - place, 0), left);
      place += skip, at += skip, left -= skip;
      if (left == 0) break;
      const int unit = place - S::kStart;
      const int count = min(min(32, n - unit), left);
      // 32 pages' places in the row, and their ids
      int tokens = 0, page = -1;
      if (lane < count) {
        const int block = p.blocks ? __ldg(p.blocks + (long long)row * p.b_row + (long long)head * p.b_head + unit + lane)
                                   : unit + lane;
        if (block >= 0 && block <= (len - 1) / kPage) {
          tokens = min(kPage, len - block * kPage);
          page = __ldg(p.block_table + (long long)row * p.bt_stride + block);
          if (page < 0 || page >= p.num_pages) page = -1;
        }
      }
      if (__any_sync(kAll, tokens > 0 && page < 0)) bad = kBad;
      const bool piece_ends = unit + count == n || count == left;
      for (int i = 0; i < count; ++i) {
        const int t = __shfl_sync(kAll, tokens, i), id = __shfl_sync(kAll, page, i);
        const bool last = piece_ends && i + 1 == count, load = t > 0 && id >= 0;
        if (!load && !last) continue;
        if (!wait(&m->empty[stage], phase)) break;
        if (lane == 0) {
          int flags = (load ? t : 0) | (fresh ? kBegin : 0);
          int last_cta = 0;
          if (last) {
            flags |= kEnd | bad;
            const int first_unit = at - unit, end_unit = first_unit + n;
            const bool begins = m->begin <= first_unit, ends = m->end >= end_unit;
            if (begins) flags |= kFirst;
            if (begins && ends) flags |= kWhole;
            last_cta = (end_unit - 1) / m->share;
          }
          m->meta[stage] = make_int4(row, tile, flags, last_cta);
          const uint32_t dst = stages + stage * S::kStage;
          const int group0 = (tile % p.tiles) * S::kHeadsMax;
          const int heads = min(S::kHeadsMax, p.group - group0);
#ifdef DSA_TEST_SKIP_FIRST_TILE
          const bool deliver = issued > 0;
#else
          constexpr bool deliver = true;
#endif
          uint32_t bytes = load ? 2 * S::kSide + 2 * S::kScaleBytes : 0;
          if (load && fresh) bytes += heads * D * 2;
          if (bytes && deliver) {
            mbar_arrive_expect_tx(&m->full[stage], bytes);
#pragma unroll
            for (int b = 0; b < S::kBoxes; ++b) {
              tma_load_4d(dst + b * S::kBox, kmap, &m->full[stage], b * 32, 0, head, id);
              tma_load_4d(dst + S::kSide + b * S::kBox, vmap, &m->full[stage], b * 32, 0, head, id);
            }
            if (S::kFp8) {
              const long long s = ((long long)id * p.heads + head) * kPage;
              bulk_load(dst + S::kOffScale, p.k_scale + s, &m->full[stage], S::kScaleBytes);
              bulk_load(dst + S::kOffScale + S::kScaleBytes, p.v_scale + s, &m->full[stage], S::kScaleBytes);
            }
            if (fresh) {
              const uint16_t* q = p.q + (long long)row * p.q_row + (long long)(head * p.group + group0) * p.q_head;
              if (p.q_head == D) {
                bulk_load(dst + S::kOffQ, q, &m->full[stage], heads * D * 2);
              } else {
                for (int h = 0; h < heads; ++h)
                  bulk_load(dst + S::kOffQ + h * D * 2, q + (long long)h * p.q_head, &m->full[stage], D * 2);
              }
            }
          } else if (deliver) {
            mbar_arrive(&m->full[stage]);
          }
        }
        __syncwarp();
        ++issued;
        fresh = false;
        if (++stage == S::kStages) stage = 0, phase ^= 1;
      }
      place += count, at += count, left -= count;
      if (piece_ends && left > 0) {
        place = 0, fresh = true, bad = 0;
        if (++tile == p.heads * p.tiles) {
          tile = 0;
          do {
            len = __ldg(p.seqlens + ++row), n = row_units(p, len);
          } while (n == 0 && row + 1 < p.rows);
        }
      }
    }
  }
  // the end, for the consumers, in a stage that they have given back
  const bool told = wait(&m->empty[stage], phase);
  if (told && lane == 0) {
    m->meta[stage] = make_int4(0, 0, kDone, 0);
    mbar_arrive(&m->full[stage]);
  }
  // every copy has landed before the CTA's memory goes to another
  Waiter landed{p.status, true};
#ifdef DSA_TEST_SKIP_FIRST_TILE
  const int first = 1;
#else
  const int first = 0;
#endif
  for (int i = max(first, issued - S::kStages + told); i < issued; ++i)
    landed(&m->full[i % S::kStages], (i / S::kStages) & 1);
}

// ---- the warps that compute -----------------------------------------------------

template <int KV, int D, int NT, int MT, bool CL>
struct Consumer {
  using S = Shape<KV, D, NT, MT, CL>;
  static constexpr bool kFp8 = S::kFp8;
  static constexpr bool kHalf = KV != DSA_KV_BF16;    // the products' operands are fp16
  static constexpr int kSteps = D / 16;               // k steps of S^T, and row tiles of O^T
  static constexpr int kWarpHeads = 8 * NT;

  const PagedAttnParams& p;
  Misc* m;
  int warp, lane, g, t, slice, mt, heads;             // heads: of this warp's column tiles
  uint32_t qb[NT][kSteps][2];
  float o[kSteps][NT][4];
  // heads 2 t and 2 t + 1 of each column tile: reference of the scores, distance to that
  // of the weights * value scales (fp8), this lane's part of the total, and the
  // factor from a product to log2 units (fp8: the queries' power of two)
  float top[NT][2], ref[NT][2], sum[NT][2], qf[NT][2];
  Waiter wait;
  uint32_t meet_phase, turn, smem;

  __device__ Consumer(const PagedAttnParams& params, Misc* misc, int w, int l, uint32_t shared)
      : p(params), m(misc), warp(w), lane(l), g(l >> 2), t(l & 3), slice(w & 3), mt(w >> 2), heads(0),
        wait{params.status, true}, meet_phase(0), turn(0), smem(shared) {}

  // Where a cluster's CTA leaves its sums (head h of its tile) and statistics.
  __device__ __forceinline__ uint32_t sums_at(int h) const { return smem + S::kOffSums + h * D * 4; }
  __device__ __forceinline__ uint32_t stat_at(int h) const { return smem + S::kOffSums + (S::kHeadsMax * D + h * 4) * 4; }

  // All consumer warps.
  __device__ __forceinline__ bool meet() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&m->meet);
    const bool r = wait(&m->meet, meet_phase);
    meet_phase ^= 1;
    return r;
  }

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
#pragma unroll
      for (int n = 0; n < NT; ++n) o[j][n][0] = o[j][n][1] = o[j][n][2] = o[j][n][3] = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      top[n][0] = top[n][1] = no_top<kFp8>(), ref[n][0] = ref[n][1] = no_distance<kFp8>();
      sum[n][0] = sum[n][1] = 0.f;
    }
  }

  // Queries of head g of each column tile, in the order in which the keys are read.
  __device__ __forceinline__ void load_queries(uint32_t q) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint32_t at = q + (mt * kWarpHeads + 8 * n + g) * (D * 2);
      const bool there = 8 * n + g < heads;
      qf[n][0] = qf[n][1] = p.scale_log2;
      if (!kFp8) {
        // unit u = 2t + i of each 64 values: two steps
#pragma unroll
        for (int b = 0; b < D / 64; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 v = there ? lds128(at + b * 128 + (2 * t + i) * 16) : make_uint4(0, 0, 0, 0);
            const int s = b * 4 + i * 2;
            qb[n][s][0] = v.x, qb[n][s][1] = v.y, qb[n][s + 1][0] = v.z, qb[n][s + 1][1] = v.w;
          }
        continue;
      }
      // fp8: unit u of 16 values (2t + i of 8, or t of 4): four steps
      constexpr int kUnits = D / 64;
      uint32_t w[kUnits * 8];
      float big = 0.f;
#pragma unroll
      for (int i = 0; i < 2 * kUnits; ++i) {
        const uint4 v = there ? lds128(at + (2 * kUnits * t + i) * 16) : make_uint4(0, 0, 0, 0);
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
      auto low = [&](uint32_t u) {
        return p.dtype == DSA_FP16 ? __half2float(__ushort_as_half((unsigned short)u)) : __uint_as_float(u << 16);
      };
      auto high = [&](uint32_t u) {
        return p.dtype == DSA_FP16 ? __half2float(__ushort_as_half((unsigned short)(u >> 16)))
                                   : __uint_as_float(u & 0xffff0000u);
      };
#pragma unroll
      for (int k = 0; k < kUnits * 8; ++k) big = fmaxf(big, fmaxf(fabsf(low(w[k])), fabsf(high(w[k]))));
      big = fmaxf(big, __shfl_xor_sync(kAll, big, 1));
      big = fmaxf(big, __shfl_xor_sync(kAll, big, 2));
      // big < 2^x; queries times 2^(14 - x)
      const int x = max((int)(__float_as_uint(big) >> 23) - 126, -100);
      const float up = __uint_as_float((uint32_t)(127 + 14 - x) << 23);
      const float down = __uint_as_float((uint32_t)(127 - 14 + x) << 23);
#pragma unroll
      for (int c = 0; c < 2; ++c) qf[n][c] = __shfl_sync(kAll, down, (2 * t + c) * 4);  // heads 2t + c
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int c = 0; c < 2; ++c) qb[n][s][c] = pack2<true>(low(w[2 * s + c]) * up, high(w[2 * s + c]) * up);
    }
  }

  // S^T of the warp's 16 tokens: rows g and g + 8, heads 2t and 2t + 1.
  __device__ __forceinline__ void scores(uint32_t k, float (&s)[NT][4]) {
    float odd[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[n][c] = odd[n][c] = 0.f;
    const int token = slice * 16 + g;
    if (!kFp8) {
#pragma unroll
      for (int b = 0; b < D / 64; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t at = k + b * S::kBox + token * 128 + (((2 * t + i) ^ (token & 7)) << 4);
          const uint4 v = lds128(at), w = lds128(at + 8 * 128);
          const uint32_t a0[4] = {v.x, w.x, v.y, w.y}, a1[4] = {v.z, w.z, v.w, w.w};
          const int st = b * 4 + i * 2;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma16816<kHalf>(s[n], a0, qb[n][st][0], qb[n][st][1]);
            mma16816<kHalf>(odd[n], a1, qb[n][st + 1][0], qb[n][st + 1][1]);
          }
        }
    } else {
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const uint32_t at = k + (D == 128 ? token * 128 + (((2 * t + i) ^ (token & 7)) << 4)
                                          : token * 64 + ((t ^ ((token >> 1) & 3)) << 4));
        const uint4 v = lds128(at), w = lds128(at + 8 * S::kBoxBytes);
        const uint32_t x[4] = {v.x, v.y, v.z, v.w}, y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t a[4];
          widen4(x[c], a[0], a[2]);
          widen4(y[c], a[1], a[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float(&into)[4] = (c & 1) ? odd[n] : s[n];
            mma16816<true>(into, a, qb[n][i * 4 + c][0], qb[n][i * 4 + c][1]);
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[n][c] += odd[n][c];
  }

  // O^T += V^T * P^T; `keep`: masks of the tokens 2t, 2t + 1 (low and high half)
  // and + 8 of a page that ends inside the warp's tokens.
  template <bool CUT>
  __device__ __forceinline__ void values(uint32_t v, const uint32_t (&pb)[NT][2], uint32_t keep0, uint32_t keep1) {
    if (!kFp8) {
      // matrices of 8 tokens x 8 values: two of the values' units, tokens 0-7 and 8-15
      const int token = slice * 16 + (lane & 7) + 8 * (lane >> 4);
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        const int unit = 2 * j + (lane >> 3 & 1);        // of 16 bytes
        uint32_t a[4];
        ldmatrix_t(a, v + (unit >> 3) * S::kBox + token * 128 + (((unit & 7) ^ (token & 7)) << 4));
        if (CUT) a[0] &= keep0, a[1] &= keep0, a[2] &= keep1, a[3] &= keep1;
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816<kHalf>(o[j][n], a, pb[n][0], pb[n][1]);
      }
      return;
    }
    // row g of all tiles holds the D / 8 values from D / 8 * g on: two per tile, rows g and g + 8
    constexpr int kWords = D / 32;
    uint32_t w[4][kWords];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int token = slice * 16 + 2 * t + (i & 1) + 8 * (i >> 1);
      if (D == 128) {
        const uint4 x = lds128(v + token * 128 + ((g ^ (token & 7)) << 4));
        w[i][0] = x.x, w[i][1] = x.y, w[i][kWords - 2] = x.z, w[i][kWords - 1] = x.w;
      } else {
        const uint2 x = lds64(v + token * 64 + (((g >> 1) ^ ((token >> 1) & 3)) << 4) + (g & 1) * 8);
        w[i][0] = x.x, w[i][1] = x.y;
      }
    }
#pragma unroll
    for (int c = 0; c < kWords; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // codes of two tokens side by side: (2t, 2t + 1) and (2t + 8, 2t + 9), two values each
        uint32_t a[4];
        widen4(__byte_perm(w[0][c], w[1][c], h ? 0x7362 : 0x5140), a[0], a[1]);
        widen4(__byte_perm(w[2][c], w[3][c], h ? 0x7362 : 0x5140), a[2], a[3]);
        if (CUT) a[0] &= keep0, a[1] &= keep0, a[2] &= keep1, a[3] &= keep1;
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816<true>(o[c * 2 + h][n], a, pb[n][0], pb[n][1]);
      }
  }

  // The largest value of a head over the lanes that have its tokens.
  static __device__ __forceinline__ float over_tokens(float x) {
    x = fmaxf(x, __shfl_xor_sync(kAll, x, 4));
    x = fmaxf(x, __shfl_xor_sync(kAll, x, 8));
    return fmaxf(x, __shfl_xor_sync(kAll, x, 16));
  }

  __device__ __forceinline__ void page(uint32_t stage, int tokens) {
    if (tokens <= slice * 16) return;
    float s[NT][4];
    scores(stage, s);
    const int valid = tokens - slice * 16;               // of the warp's 16
    float e[2], f[2];                                    // fp8: exponent and mantissa of the tokens' value scales
    if (kFp8) {
      const uint32_t at = stage + S::kOffScale + (slice * 16 + g) * 4;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float ks = __uint_as_float(lds32(at + h * 32));
        const uint32_t bits = lds32(at + S::kScaleBytes + h * 32);
        const int x = (int)(bits >> 23 & 255u);
        e[h] = (float)(x - 127);
        f[h] = x == 255 ? __uint_as_float(bits)                      // not a number: the weight is none
               : x      ? __uint_as_float((bits & 0x807fffffu) | 0x3f800000u)
                        : __uint_as_float(bits) * 1.7014118346046923e38f;  // 2^127
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            // what makes a product smaller before the key scale, what makes it larger behind it: queries
            // and keys of any sizes pass no infinity on the way to a score that is none
            const float small = fminf(qf[n][c], 1.f), large = fmaxf(qf[n][c], 1.f) * p.scale_log2;
            s[n][2 * h + c] = s[n][2 * h + c] * small * ks * large;
          }
      }
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[n][c] *= qf[n][c & 1];
    }
    if (valid < 16) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (g + 8 * h >= valid) {
#pragma unroll
          for (int n = 0; n < NT; ++n) s[n][2 * h] = s[n][2 * h + 1] = -CUDART_INF_F;
          if (kFp8) f[h] = 0.f;                          // whatever its scale
        }
    }
    bool over = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        over |= s[n][c] > top[n][c & 1] + kAbove;
        if (kFp8) over |= s[n][c] - top[n][c & 1] + e[c >> 1] > ref[n][c & 1] + kAbove;
      }
    if (__any_sync(kAll, over)) raise(s, e);
    uint32_t pb[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float x[4];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float base = !kFp8 && top[n][c] == -CUDART_INF_F ? 0.f : top[n][c];
        const float y0 = s[n][c] - base, y1 = s[n][2 + c] - base;
        x[c] = ex2(y0), x[2 + c] = ex2(y1);
        sum[n][c] += x[c] + x[2 + c];
        if (kFp8) {
          const float from = ref[n][c] - kBelow;
          x[c] = ex2(y0 + e[0] - from) * f[0], x[2 + c] = ex2(y1 + e[1] - from) * f[1];
        }
      }
      pb[n][0] = transpose8(pack2<kHalf>(x[0], x[1]));
      pb[n][1] = transpose8(pack2<kHalf>(x[2], x[3]));
    }
    if (valid >= 16) {
      values<false>(stage + S::kSide, pb, 0, 0);
    } else {
      // masked tokens may hold anything, and 0 * NaN is NaN
      auto mask = [&](int token) {
        return (token < valid ? 0xffffu : 0u) | (token + 1 < valid ? 0xffff0000u : 0u);
      };
      values<true>(stage + S::kSide, pb, mask(2 * t), mask(2 * t + 8));
    }
  }

  // New references where a score is too far above the old one: the largest.
  __device__ __forceinline__ void raise(const float (&s)[NT][4], const float (&e)[2]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float big = over_tokens(fmaxf(s[n][c], s[n][2 + c]));
        float less = 1.f;
        if (big > top[n][c] + kAbove) {
          less = ex2(top[n][c] - big);
          if (kFp8) ref[n][c] += top[n][c] - big;
          top[n][c] = big;
        }
        sum[n][c] *= less;
        if (kFp8) {
          const float high = over_tokens(fmaxf(s[n][c] - top[n][c] + e[0], s[n][2 + c] - top[n][c] + e[1]));
          less = 1.f;
          if (high > ref[n][c] + kAbove) less = ex2(ref[n][c] - high), ref[n][c] = high;
        }
#pragma unroll
        for (int j = 0; j < kSteps; ++j) o[j][n][c] *= less, o[j][n][2 + c] *= less;
      }
  }

  // Value of O^T's row tile j that register c (rows g and g + 8) holds.
  __device__ __forceinline__ int column(int j, int c) const {
    return kFp8 ? (D / 8) * g + 2 * j + c : 16 * j + 8 * c + g;
  }

  // A row's four slices of tokens meet in the stage; results or partial sums go out.
  __device__ __forceinline__ void finish(uint8_t* stage, int4 meta) {
    float(*stats)[16][3] = m->stat[turn];
    turn ^= 1;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        sum[n][c] += __shfl_xor_sync(kAll, sum[n][c], 4);
        sum[n][c] += __shfl_xor_sync(kAll, sum[n][c], 8);
        sum[n][c] += __shfl_xor_sync(kAll, sum[n][c], 16);
        if (g == 0) {
          float* s = stats[warp][8 * n + 2 * t + c];
          s[0] = top[n][c], s[1] = ref[n][c], s[2] = sum[n][c];
        }
      }
    if (!meet()) return;
    const int group0 = (meta.y % p.tiles) * S::kHeadsMax, key_head = meta.y / p.tiles;
    const int all = min(S::kHeadsMax, p.group - group0);  // of the CTA
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int h = 8 * n + 2 * t + c;
        float big = -CUDART_INF_F, high = -CUDART_INF_F;
#pragma unroll
        for (int w = 0; w < 4; ++w) big = fmaxf(big, stats[mt * 4 + w][h][0]);
#pragma unroll
        for (int w = 0; w < 4; ++w)
          high = fmaxf(high, distance<kFp8>(stats[mt * 4 + w][h][0], stats[mt * 4 + w][h][1], big));
        const float f = factor<kFp8>(top[n][c], ref[n][c], big, high);
#pragma unroll
        for (int j = 0; j < kSteps; ++j) o[j][n][c] *= f, o[j][n][2 + c] *= f;
      }
    const bool whole = meta.z & kWhole;
    const int piece = (meta.z & kFirst) ? 1 : 0;
    const int hv = paged_cta_heads(p.group);
    float* part = p.ws + ((long long)blockIdx.x * 2 + piece) * hv * (D + 4);
    float* parts = reinterpret_cast<float*>(stage);
#pragma unroll 1
    for (int pass = 0; pass < S::kPasses; ++pass) {
      // slices of a column chunk; groups of 8 columns are permuted by row against bank conflicts
      auto place = [&](int col, int row) {
        return col ^ ((((row >> 1 & 3) ^ ((col >> 5) & 3)) << 3) & (S::kCols - 1));
      };
#pragma unroll
      for (int j = 0; j < kSteps; ++j)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int col = column(j, c >> 1) - pass * S::kCols, row = mt * kWarpHeads + 8 * n + 2 * t + (c & 1);
            if (col >= 0 && col < S::kCols)
              parts[(slice * S::kHeadsMax + row) * S::kCols + place(col, row)] = o[j][n][c];
          }
      if (!meet()) return;
      constexpr int kGroups = S::kCols / 8;
      for (int i = warp * 32 + lane; i < all * kGroups; i += S::kConsumers * 32) {
        const int row = i / kGroups, col = (i % kGroups) * 8;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float4* from =
              reinterpret_cast<const float4*>(parts + (w * S::kHeadsMax + row) * S::kCols + place(col, row));
          const float4 a = from[0], b = from[1];
          x[0] += a.x, x[1] += a.y, x[2] += a.z, x[3] += a.w, x[4] += b.x, x[5] += b.y, x[6] += b.z, x[7] += b.w;
        }
        const float(*st)[16][3] = stats + (row / kWarpHeads) * 4;
        const int h = row % kWarpHeads;
        float big = -CUDART_INF_F, high = -CUDART_INF_F, total = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) big = fmaxf(big, st[w][h][0]);
#pragma unroll
        for (int w = 0; w < 4; ++w) high = fmaxf(high, distance<kFp8>(st[w][h][0], st[w][h][1], big));
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float l = st[w][h][2];
          // a slice without tokens has no reference; a NaN total stays one
          total += st[w][h][0] == -CUDART_INF_F ? l : l * ex2(st[w][h][0] - big);
        }
        if (meta.z & kBad) total = CUDART_NAN_F;
        const int c0 = pass * S::kCols + col;
        if (CL && !whole) {
          sts128(sums_at(row) + c0 * 4, make_float4(x[0], x[1], x[2], x[3]));
          sts128(sums_at(row) + c0 * 4 + 16, make_float4(x[4], x[5], x[6], x[7]));
          if (c0 == 0) sts128(stat_at(row), make_float4(big, high, total, 0.f));
          continue;
        }
        if (!whole) {
          float4* to = reinterpret_cast<float4*>(part + (long long)row * D + c0);
          to[0] = make_float4(x[0], x[1], x[2], x[3]), to[1] = make_float4(x[4], x[5], x[6], x[7]);
          if (c0 == 0)
            *reinterpret_cast<float4*>(part + (long long)hv * D + row * 4) = make_float4(big, high, total, 0.f);
          continue;
        }
        write_out(p, meta.x, key_head * p.group + group0 + row, c0, x, big, high, total);
      }
      if (pass + 1 < S::kPasses && !meet()) return;
    }
    if ((meta.z & kBad) && warp == 0 && lane == 0) raise_status(p.status, DSA_ERR_BAD_PAGE);
    if (!CL && !whole && piece == 1 && warp == 0 && lane == 0) {
      int4* record = reinterpret_cast<int4*>(p.ws + (long long)gridDim.x * 2 * hv * (D + 4)) + blockIdx.x;
      *record = make_int4(meta.x, meta.y, meta.w, 0);
    }
  }

  // Eight values of a head's result: the total under `big`, the sums x under that and `high` above it.
  static __device__ __forceinline__ void write_out(const PagedAttnParams& p, int row, int head, int c0, float (&x)[8],
                                                   float big, float high, float total) {
    // no visible token: zeros, -inf
    const float f = total == 0.f ? 0.f : (kFp8 ? kSmallest : 1.f) / total;
    // of the size of the value scales, and 2^8 above them where the references of the scores and
    // of the weights have been raised apart: past 2^100 a second factor
    const float unit = kFp8 ? ex2_small(fminf(high, 100.f)) : 1.f, more = kFp8 ? ex2(fmaxf(high - 100.f, 0.f)) : 1.f;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = total == 0.f ? 0.f : x[2 * i] * f * unit * more;
      const float b = total == 0.f ? 0.f : x[2 * i + 1] * f * unit * more;
      w[i] = p.dtype == DSA_FP16 ? pack2<true>(a, b) : pack2<false>(a, b);
    }
    *reinterpret_cast<uint4*>(p.out + (long long)row * p.out_row + (long long)head * p.out_head + c0) =
        make_uint4(w[0], w[1], w[2], w[3]);
    if (c0 == 0 && p.lse)
      p.lse[(long long)row * p.heads * p.group + head] =
          total == 0.f ? -CUDART_INF_F : (big + log2f(total)) * 0.69314718055994531f;
  }

  // NaN or zeros into a row's heads [h0, h1), by `count` threads of which this one is `me`.
  __device__ void fill(int row, int h0, int h1, bool nan, int me, int count) {
    const uint32_t v = nan ? 0x7fff7fffu : 0u;           // NaN in either type
    for (int i = h0 * (D / 8) + me; i < h1 * (D / 8); i += count) {
      const int h = i / (D / 8), c0 = i % (D / 8) * 8;
      *reinterpret_cast<uint4*>(p.out + (long long)row * p.out_row + (long long)h * p.out_head + c0) =
          make_uint4(v, v, v, v);
      if (c0 == 0 && p.lse) p.lse[(long long)row * p.heads * p.group + h] = nan ? CUDART_NAN_F : -CUDART_INF_F;
    }
  }

  // Rows without units: zeros, or NaN where the length is past the table.
  __device__ void empty_rows() {
    if (CL) {
      // the cluster's row and heads, by its first CTA
      if (m->total > 0 || m->rank > 0) return;
      const bool bad = __ldg(p.seqlens + m->row) > 0;
      if (bad && warp == 0 && lane == 0) raise_status(p.status, DSA_ERR_BAD_SEQLEN);
      const int group0 = (m->tile % p.tiles) * S::kHeadsMax, h0 = (m->tile / p.tiles) * p.group + group0;
      fill(m->row, h0, h0 + min(S::kHeadsMax, p.group - group0), bad, warp * 32 + lane, S::kConsumers * 32);
      return;
    }
    for (int row = blockIdx.x; row < p.rows; row += gridDim.x) {
      const int len = __ldg(p.seqlens + row);
      if (row_units(p, len) > 0) continue;
      const bool bad = len > 0;
      if (bad && warp == 0 && lane == 0) raise_status(p.status, DSA_ERR_BAD_SEQLEN);
      fill(row, 0, p.heads * p.group, bad, warp * 32 + lane, S::kConsumers * 32);
    }
  }

  // After a wait that ran out: NaN for every row of the slice, and for its partial results.
  __device__ void poison() {
    if (CL) {
      for (int h = lane; h < S::kHeadsMax; h += 32) sts128(stat_at(h), make_float4(0.f, 0.f, CUDART_NAN_F, 0.f));
      if (m->share < m->total) return;     // (one CTA's row: below)
    }
    const int hv = paged_cta_heads(p.group);
    float* part = p.ws + (long long)blockIdx.x * 2 * hv * (D + 4);
    for (int i = lane; !CL && i < 2 * hv; i += 32)
      *reinterpret_cast<float4*>(part + (long long)(i / hv) * hv * (D + 4) + (long long)hv * D + (i % hv) * 4) =
          make_float4(0.f, 0.f, CUDART_NAN_F, 0.f);
    int left = m->end - m->begin, row = m->row, tile = m->tile, place = m->place;
    while (left > 0) {
      const int n = row_units(p, __ldg(p.seqlens + row));
      if (n == 0) {
        ++row;
        continue;
      }
      const int group0 = (tile % p.tiles) * S::kHeadsMax, h0 = (tile / p.tiles) * p.group + group0;
      const int count = min(left, S::kStart + n - place);
      if (place + count > S::kStart) fill(row, h0, h0 + min(S::kHeadsMax, p.group - group0), true, lane, 32);
      left -= count;
      place = 0;
      if (++tile == p.heads * p.tiles) tile = 0, ++row;
    }
  }

  __device__ void run(uint8_t* stages) {
    if (!CL && warp == 0 && lane == 0) {
      const int hv = paged_cta_heads(p.group);
      reinterpret_cast<int4*>(p.ws + (long long)gridDim.x * 2 * hv * (D + 4))[blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
    empty_rows();
    int stage = 0;
    uint32_t phase = 0;
    reset();
    while (wait(&m->full[stage], phase)) {
      const int4 meta = m->meta[stage];
      if (meta.z & kDone) return;
      uint8_t* at = stages + stage * S::kStage;
      const uint32_t base = smem_u32(at);
      const int tokens = meta.z & 127;
      if (meta.z & kBegin) {
        reset();
        heads = min(max(p.group - (meta.y % p.tiles) * S::kHeadsMax - mt * kWarpHeads, 0), kWarpHeads);
        if (tokens) load_queries(base + S::kOffQ);
      }
      if (heads > 0) page(base, tokens);
      if (meta.z & kEnd) {
        finish(at, meta);
        if (!wait.ok) break;
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&m->empty[stage]);
      if (++stage == S::kStages) stage = 0, phase ^= 1;
    }
    poison();
  }

  // After the cluster's barrier: the row's results from all its CTAs' sums, some
  // heads and columns by each CTA.
  __device__ void join_cluster(int ctas) {
    const int active = (m->total + m->share - 1) / m->share;
    if (active < 2) return;
    const int group0 = (m->tile % p.tiles) * S::kHeadsMax, h0 = (m->tile / p.tiles) * p.group + group0;
    const int all = min(S::kHeadsMax, p.group - group0) * (D / 8);
    for (int i = m->rank * S::kConsumers * 32 + warp * 32 + lane; i < all; i += ctas * S::kConsumers * 32) {
      const int h = i / (D / 8), c0 = i % (D / 8) * 8;
      float4 st[8], a[8], b[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < active)
          st[r] = far_load(stat_at(h), r), a[r] = far_load(sums_at(h) + c0 * 4, r), b[r] = far_load(sums_at(h) + c0 * 4 + 16, r);
      float big = -CUDART_INF_F, high = -CUDART_INF_F, total = 0.f;
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < active) big = fmaxf(big, st[r].x);
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < active) high = fmaxf(high, distance<kFp8>(st[r].x, st[r].y, big));
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < active) {
          total += st[r].x == -CUDART_INF_F ? st[r].z : st[r].z * ex2(st[r].x - big);
          const float w = factor<kFp8>(st[r].x, st[r].y, big, high);
          x[0] += w * a[r].x, x[1] += w * a[r].y, x[2] += w * a[r].z, x[3] += w * a[r].w;
          x[4] += w * b[r].x, x[5] += w * b[r].y, x[6] += w * b[r].z, x[7] += w * b[r].w;
        }
      write_out(p, m->row, h0 + h, c0, x, big, high, total);
    }
  }
};

template <int KV, int D, int NT, int MT, bool CL>
__global__ void __launch_bounds__(Shape<KV, D, NT, MT, CL>::kThreads, Shape<KV, D, NT, MT, CL>::kCtas)
    paged_attention_kernel(const __grid_constant__ PagedAttnParams p, const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap, int cluster) {
  using S = Shape<KV, D, NT, MT, CL>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  Misc* m = reinterpret_cast<Misc*>(smem + S::kOffMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&m->full[i], 1);
      mbar_init(&m->empty[i], S::kConsumers);
    }
    mbar_init(&m->meet, S::kConsumers);
    fence_barrier_init();
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  griddep_wait();
  griddep_launch_dependents();
  // (the barriers in these also publish the mbarriers)
  if (CL) cluster_slice(p, m, cluster, S::kStart);
  else find_slice<S::kThreads>(p, m, S::kStart);
  if (warp == S::kConsumers) {
    produce<KV, D, NT, MT, CL>(p, &kmap, &vmap, m, smem_u32(smem));
  } else {
    Consumer<KV, D, NT, MT, CL> c(p, m, warp, lane, smem_u32(smem));
    c.run(smem);
  }
  if (CL) {
    __syncwarp();
    cluster_sync();
    if (warp < S::kConsumers) {
      Consumer<KV, D, NT, MT, CL> c(p, m, warp, lane, smem_u32(smem));
      c.join_cluster(cluster);
    }
    __syncwarp();
    cluster_sync();                          // nobody leaves while its memory is read
  }
}

// ---- the join -------------------------------------------------------------------

constexpr int kJoinThreads = 128;

// Block (c, h): head h of the row whose units CTA c begins and does not end.
template <int KV, int D>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ PagedAttnParams p, int ctas,
                                                                  int heads_max) {
  constexpr int kLanes = D / 4, kGroups = kJoinThreads / kLanes;
  __shared__ float weight[kJoinThreads];
  __shared__ float4 stat[kJoinThreads / 32];
  __shared__ alignas(16) float sums[kGroups][D];
  const int hv = paged_cta_heads(p.group), h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  griddep_launch_dependents();
  const int4 record = *(reinterpret_cast<const int4*>(p.ws + (long long)ctas * 2 * hv * (D + 4)) + blockIdx.x);
  const int first = blockIdx.x, row = record.x, tile = record.y, last = record.z;
  // addresses come from it, and the workspace is the caller's
  if (row < 0 || row >= p.rows || tile < 0 || tile >= p.heads * p.tiles || last <= first || last >= ctas) return;
  const int group0 = (tile % p.tiles) * heads_max;
  if (h >= p.group - group0) return;
  const int pieces = last - first + 1;
  auto part = [&](int i) { return p.ws + ((long long)(first + i) * 2 + (i == 0)) * hv * (D + 4); };
  // the largest references
  constexpr bool kFp8 = KV == DSA_KV_FP8_E4M3;
  float big = no_top<kFp8>(), high = no_distance<kFp8>();
  auto larger = [&](float top, float ref) {
    const float above = fmaxf(big, top);
    high = fmaxf(distance<kFp8>(big, high, above), distance<kFp8>(top, ref, above)), big = above;
  };
  for (int i = threadIdx.x; i < pieces; i += kJoinThreads) {
    const float4 s = *reinterpret_cast<const float4*>(part(i) + (long long)hv * D + h * 4);
    larger(s.x, s.y);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float x = __shfl_xor_sync(kAll, big, o), y = kFp8 ? __shfl_xor_sync(kAll, high, o) : 0.f;
    larger(x, y);
  }
  if (lane == 0) stat[warp] = make_float4(big, high, 0.f, 0.f);
  __syncthreads();
  big = no_top<kFp8>(), high = no_distance<kFp8>();  // in one order, so that all threads have the same
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) larger(stat[w].x, stat[w].y);
  // four columns a thread, several groups of pieces
  const int col = threadIdx.x % kLanes * 4, group = threadIdx.x / kLanes;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  float total = 0.f;
  for (int i0 = 0; i0 < pieces; i0 += kJoinThreads) {
    const int n = min(kJoinThreads, pieces - i0);
    __syncthreads();
    if (threadIdx.x < n) {
      const float4 s = *reinterpret_cast<const float4*>(part(i0 + threadIdx.x) + (long long)hv * D + h * 4);
      weight[threadIdx.x] = factor<kFp8>(s.x, s.y, big, high);
      total += s.x == -CUDART_INF_F ? s.z : s.z * ex2(s.x - big);
    }
    __syncthreads();
#pragma unroll 4
    for (int i = group; i < n; i += kGroups) {
      const float4 v = *reinterpret_cast<const float4*>(part(i0 + i) + (long long)h * D + col);
      const float w = weight[i];
      x.x += w * v.x, x.y += w * v.y, x.z += w * v.z, x.w += w * v.w;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
  *reinterpret_cast<float4*>(&sums[group][col]) = x;
  __syncthreads();
  if (lane == 0) stat[warp].z = total;
  __syncthreads();
  total = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) total += stat[w].z;
  if (threadIdx.x < D / 8) {
    float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const int c0 = threadIdx.x * 8;
#pragma unroll
    for (int k = 0; k < kGroups; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] += sums[k][c0 + i];
    Consumer<KV, D, 1, 1, false>::write_out(p, row, (tile / p.tiles) * p.group + group0 + h, c0, y, big, high, total);
  }
}

template <typename K, typename... A>
cudaError_t launch(K kernel, dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
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

// The kernel's shared memory, allowed once per device.
template <int KV, int D, int NT, int MT, bool CL>
cudaError_t set_up() {
  static bool ready[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < kMaxDevices && ready[dev])) return e;
  e = cudaFuncSetAttribute(paged_attention_kernel<KV, D, NT, MT, CL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Shape<KV, D, NT, MT, CL>::kSmem);
  if (e == cudaSuccess && dev < kMaxDevices) ready[dev] = true;
  return e;
}

// Few short rows: a cluster of CTAs for each row and head tile, which join their
// results in their own memory; one launch where the balanced split takes two.  Up
// to so many pages a CTA, by the table's width (rows may be of any lengths) or by
// the lists (rows mostly are alike).  Measured, 32 heads on 8, 128 values, bf16,
// a cluster and the split: one row of 1,024 tokens 6.3 us and 8.5, of 4,096 9.2
// and 9.8, of 8,192 13.0 and 10.8; 16 rows of 1,024 10.7 and 13.0; fp8, lists of 32
// pages, one row 8.8 and 10.6, 16 rows 17.7 and 20.5.
constexpr int kClusterPages = 8, kClusterEntries = 16;

template <int KV, int D, int NT, int MT>
cudaError_t launch_t(const PagedAttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int sms,
                     cudaStream_t stream) {
  using S = Shape<KV, D, NT, MT, false>;
  const int ctas = sms * S::kCtas;
  const long long items = (long long)p.rows * p.heads * p.tiles, most = p.blocks ? p.k : p.W;
  int cluster = 1;
  while (cluster < 8 && 2 * cluster * items <= ctas && cluster < most) cluster *= 2;
  if (cluster > 1 && most <= (long long)cluster * (p.blocks ? kClusterEntries : kClusterPages)) {
    using C = Shape<KV, D, NT, MT, true>;
    const cudaError_t e = set_up<KV, D, NT, MT, true>();
    if (e != cudaSuccess) return e;
    return launch(paged_attention_kernel<KV, D, NT, MT, true>, dim3((unsigned)items * cluster), C::kThreads, C::kSmem,
                  cluster, stream, p, kmap, vmap, cluster);
  }
  cudaError_t e = set_up<KV, D, NT, MT, false>();
  if (e != cudaSuccess) return e;
  e = launch(paged_attention_kernel<KV, D, NT, MT, false>, dim3(ctas), S::kThreads, S::kSmem, 1, stream, p, kmap, vmap, 1);
  if (e != cudaSuccess) return e;
  return launch(paged_join_kernel<KV, D>, dim3(ctas, paged_cta_heads(p.group)), kJoinThreads, 0, 1, stream, p, ctas,
                S::kHeadsMax);
}

template <int KV, int D>
cudaError_t launch_d(const PagedAttnParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int sms,
                     cudaStream_t stream) {
  switch (paged_heads_max(p.group)) {
    case 8: return launch_t<KV, D, 1, 1>(p, kmap, vmap, sms, stream);
    case 16: return launch_t<KV, D, 2, 1>(p, kmap, vmap, sms, stream);
    default: return launch_t<KV, D, 2, 2>(p, kmap, vmap, sms, stream);
  }
}

}  // namespace

cudaError_t launch_paged_attention(const PagedAttnParams& p, int dim, int kv_dtype, const CUtensorMap& kmap,
                                   const CUtensorMap& vmap, int sms, cudaStream_t stream) {
  if (kv_dtype == DSA_KV_BF16)
    return dim == 128 ? launch_d<DSA_KV_BF16, 128>(p, kmap, vmap, sms, stream)
                      : launch_d<DSA_KV_BF16, 64>(p, kmap, vmap, sms, stream);
  if (kv_dtype == DSA_KV_FP16)
    return dim == 128 ? launch_d<DSA_KV_FP16, 128>(p, kmap, vmap, sms, stream)
                      : launch_d<DSA_KV_FP16, 64>(p, kmap, vmap, sms, stream);
  return dim == 128 ? launch_d<DSA_KV_FP8_E4M3, 128>(p, kmap, vmap, sms, stream)
                    : launch_d<DSA_KV_FP8_E4M3, 64>(p, kmap, vmap, sms, stream);
}

}  // namespace dsa
