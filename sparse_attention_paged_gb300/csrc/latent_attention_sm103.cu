// latent_attention_sm103.cu -- attention of H query heads over the cached
// latent tokens of a row, in the absorbed form:
//
//   s[h, t] = scale * (ql[h] . c[t] + qr[h] . r[t])      c: 512 values, r: 64
//   p[h, :] = softmax(s[h, :]) over the row's visible tokens
//   out[h]  = sum_t p[h, t] c[t],   lse[h] = log sum_t exp(s[h, t])
//
// One token serves as key and value of every head, so a tile of 64 tokens is
// brought into shared memory once (bf16, nine blocks of 64 values, 128-byte
// swizzle) and feeds both products as it lies there:
//
//   S^T [64 tokens x 64 heads]  = tile [64 x 576] (A, K-major) * Q^T (B, K-major)
//   O^T [512 values x 64 heads] += tile^T (A, MN-major) * P^T (B, MN-major)
//
// Keeping the heads on the N side leaves O^T at 4 x 64 TMEM columns, beside
// two S^T buffers, and a token's mask is a whole row of S^T.  The softmax
// warps read S^T, keep a maximum per head that is raised only when a score
// passes it by 2^8 (then O^T is rescaled in TMEM; the sums are fp32, so the
// reference point does not change their relative precision), and write P as
// bf16, rounded to nearest: its rounding is independent from token to token
// and below that of the bf16 result.
//
// Persistent: the call's tiles (per head group of 64) are cut into equal
// slices, one per CTA, rows in order.  A row that a slice cuts leaves
// unnormalised partial sums in the workspace, and a second kernel joins
// them, so one long row or a few short ones spread over every SM, and a
// batch of any lengths is balanced.
//
// Warps: 0-3 softmax and output, 4 MMA issue, 5-12 loaders in two groups of
// four, one per tile buffer.  A selected token is 1,152 contiguous bytes (fp8:
// 512 + 128 + 16), gathered with 16-byte loads per token through the block
// table; masked tokens are not read, their rows are zeros.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "latent_common.cuh"
#include "sm100_ptx.cuh"

#ifndef DSA_WAIT_LIMIT_CYCLES
#define DSA_WAIT_LIMIT_CYCLES 4000000000ll
#endif

namespace dsa {

namespace {

using namespace sm100;

constexpr int kTile = 64;                       // tokens per tile
constexpr int kBlocks = (kLatent + kRope) / 64; // 64-value blocks of a token
constexpr int kBlockBytes = kTile * 128;        // one block of a tile (or of Q)
constexpr int kTileBytes = kBlocks * kBlockBytes;
constexpr int kSoftmaxWarps = 4, kMmaWarp = 4, kLoadWarp0 = 5, kLoadWarps = 8;
constexpr int kAttnThreads = (kLoadWarp0 + kLoadWarps) * 32;
constexpr int kGroupThreads = kLoadWarps / 2 * 32;
constexpr int kKeysPerWarp = kTile / (kLoadWarps / 2);  // 16
constexpr float kSlack = 8.f;                   // log2 of how far a score may pass the kept maximum

// Shared memory, from a 1,024-byte boundary.
constexpr int kOffQ = 2 * kTileBytes;
constexpr int kOffP = kOffQ + kTileBytes;
constexpr int kOffMisc = kOffP + kBlockBytes;
struct Misc {
  uint64_t full[2], empty[2], sfull[2], pfull, qfree, ofull, ofree, done;
  uint32_t tmem;
  int abort;
  int start_row, start_tile, total;
  int nzero;
  uint32_t keymask[2][4];   // per tile buffer and loader warp: 16 valid bits, bad data in bit 16
  int scan[16];
  float red[4][kAttnHeads]; // per softmax warp and head
  float fac[kAttnHeads];
  int zero[64];
};
constexpr int kSmemBytes = kOffMisc + 2048 + 1024;
static_assert(sizeof(Misc) <= 2048, "misc");
static_assert(kSmemBytes <= 232448, "227 KB");

// TMEM columns: O^T 4 x 64, S^T 2 x 64.
constexpr uint32_t kTmemS = 256, kTmemCols = 512;

constexpr long long kWaitLimit = DSA_WAIT_LIMIT_CYCLES;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ bool bar_any(int id, int threads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// tcgen05.wait::ld tied to a 32-register destination
__device__ __forceinline__ void tmem_ld_wait32(uint32_t (&a)[32]) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]),
        "+r"(a[8]), "+r"(a[9]), "+r"(a[10]), "+r"(a[11]), "+r"(a[12]), "+r"(a[13]), "+r"(a[14]),
        "+r"(a[15]), "+r"(a[16]), "+r"(a[17]), "+r"(a[18]), "+r"(a[19]), "+r"(a[20]), "+r"(a[21]),
        "+r"(a[22]), "+r"(a[23]), "+r"(a[24]), "+r"(a[25]), "+r"(a[26]), "+r"(a[27]), "+r"(a[28]),
        "+r"(a[29]), "+r"(a[30]), "+r"(a[31])
      :
      : "memory");
}

// Descriptor of an MN-major operand in the 128-byte swizzle: 64 M/N values of
// one K index are a 128-byte row, eight K rows an atom; `k_bytes` from one
// atom to the next along K, `mn_bytes` to the next 64 M/N values.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t mn_bytes, uint32_t k_bytes) {
  uint64_t d = smem_desc_sw128(saddr, k_bytes);
  d &= ~((uint64_t)0x3FFFu << 16);
  d |= (uint64_t)((mn_bytes >> 4) & 0x3FFFu) << 16;
  return d;
}

constexpr uint32_t kIdescS = instr_desc(1, 1, kTile, kAttnHeads);
constexpr uint32_t kIdescO = instr_desc(1, 1, 128, kAttnHeads) | (1u << 15) | (1u << 16);  // A, B MN-major

// A row's visible entries: its length, or the part of its selection list that
// is read.  A length past the block table is an error: no entries.
__device__ __forceinline__ int row_entries(const LatentAttnParams& p, int row, int* len) {
  const int L = __ldg(p.seqlens + row);
  *len = L;
  if (L <= 0 || (long long)L > (long long)p.W * kPage) return 0;
  return p.idx ? min(L, p.k) : L;
}

// Walks the tiles of a CTA's slice, row by row; rows without tiles are passed.
struct TileWalk {
  int row, t, n, len, left, piece;
  bool first;
  __device__ __forceinline__ int tiles() const { return (n + kTile - 1) / kTile; }
  __device__ __forceinline__ bool last() const { return left == 1 || t + 1 == tiles(); }
  __device__ __forceinline__ void start(const LatentAttnParams& p, int row0, int tile0, int count) {
    row = row0, t = tile0, left = count, piece = 0, first = true, n = 0, len = 0;
    if (left > 0) n = row_entries(p, row, &len);
  }
  __device__ __forceinline__ void step(const LatentAttnParams& p) {
    if (--left <= 0) return;
    if (++t < tiles()) {
      first = false;
      return;
    }
    do {
      n = row_entries(p, ++row, &len);
    } while (n == 0 && row + 1 < p.rows);
    t = 0, first = true, ++piece;
  }
};

struct Waiter {
  Misc* m;
  int* status;
  bool ok;
  // Wait for phase `parity` of `bar`; after a wait that ran out (here or in
  // another warp) every wait returns at once.
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) {
    if (!ok) return false;
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t i = 1;; ++i) {
      if (mbar_try_wait(bar, parity)) return true;
      if ((i & 15u) == 0) {
        if (*reinterpret_cast<volatile int*>(&m->abort)) break;
        if (clock64() - t0 > kWaitLimit) {
          *reinterpret_cast<volatile int*>(&m->abort) = 1;
          raise_status(status, DSA_ERR_TIMEOUT);
          break;
        }
      }
    }
    ok = false;
    return false;
  }
};

// The byte offset in the cache of entry j of a tile's row, -1 when it is
// masked; *bad when a valid entry has no page.
__device__ __forceinline__ long long token_offset(const LatentAttnParams& p, const TileWalk& w, int j,
                                                  int kv_token_bytes, bool* bad, int* slot) {
  *bad = false;
  *slot = 0;
  if (j >= w.n) return -1;
  int pos = j;
  if (p.idx) {
    pos = __ldg(p.idx + w.row * p.idx_stride + j);
    if (pos < 0 || pos >= w.len) return -1;
  }
  const int page = __ldg(p.block_table + w.row * p.bt_stride + pos / kPage);
  if (page < 0 || page >= p.num_pages) {
    *bad = true;
    return -1;
  }
  *slot = pos % kPage;
  return (long long)page * p.page_stride + (long long)(pos % kPage) * kv_token_bytes;
}

// Bytes `chunk` (16 bytes each, 8 per block) of row r of a tile in the swizzled layout.
__device__ __forceinline__ uint32_t swz(int r, int chunk) {
  return (uint32_t)((chunk >> 3) * kBlockBytes + r * 128 + (((chunk & 7) ^ (r & 7)) << 4));
}

// 16 e4m3 codes times their scale as bf16, 32 bytes.
__device__ __forceinline__ void dequant16(const uint4& c, float s, uint4& a, uint4& b) {
  const uint32_t u[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __half2_raw f = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u[j] >> (16 * h)), __NV_E4M3);
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f));
      const __nv_bfloat162 r = __floats2bfloat162_rn(v.x * s, v.y * s);
      o[2 * j + h] = *reinterpret_cast<const uint32_t*>(&r);
    }
  a = make_uint4(o[0], o[1], o[2], o[3]);
  b = make_uint4(o[4], o[5], o[6], o[7]);
}

template <int KV>
__global__ void __launch_bounds__(kAttnThreads, 1) latent_attention_kernel(const LatentAttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Misc* m = reinterpret_cast<Misc*>(smem + kOffMisc);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x / p.groups, grp = blockIdx.x % p.groups;
  const int head0 = grp * kAttnHeads, heads = min(kAttnHeads, p.H - head0);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&m->full[i], kGroupThreads);
      mbar_init(&m->empty[i], 1);
      mbar_init(&m->sfull[i], 1);
    }
    mbar_init(&m->pfull, kSoftmaxWarps * 32);
    mbar_init(&m->qfree, 1);
    mbar_init(&m->ofull, 1);
    mbar_init(&m->ofree, kSoftmaxWarps * 32);
    mbar_init(&m->done, 1);
    fence_barrier_init();
    m->abort = 0;
    m->start_row = m->start_tile = m->total = 0;
    m->nzero = 0;
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&m->tmem, kTmemCols);
    tmem_relinquish();
  }
  griddep_wait();
  griddep_launch_dependents();

  // ---- the slice -----------------------------------------------------------
  // thread i owns a run of rows; an exclusive scan of the runs' tile counts
  // finds the row in which this CTA's slice begins
  const int per = (p.rows + kAttnThreads - 1) / kAttnThreads;
  const int r0 = min(p.rows, tid * per), r1 = min(p.rows, r0 + per);
  int mine = 0, len;
  for (int r = r0; r < r1; ++r) mine += (row_entries(p, r, &len) + kTile - 1) / kTile;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) m->scan[warp] = incl;
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = m->tmem;
  int base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kAttnThreads / 32; ++w) {
    if (w < warp) base += m->scan[w];
    total += m->scan[w];
  }
  const int ctas = min(p.ctas, total);            // every slice has a tile
  int begin = 0, end = 0;
  if (cta < ctas) {
    begin = (int)((long long)cta * total / ctas);
    end = (int)((long long)(cta + 1) * total / ctas);
  }
  {
    int at = base + incl - mine;
    if (end > begin && at <= begin && begin < at + mine) {
      int r = r0;
      for (;; ++r) {
        const int t = (row_entries(p, r, &len) + kTile - 1) / kTile;
        if (begin < at + t) break;
        at += t;
      }
      m->start_row = r;
      m->start_tile = begin - at;
    }
  }
  // rows without a visible token: zeros (a length past the table: NaN)
  for (long long r = cta; r - cta < p.rows; r += (long long)p.ctas * 64) {
    __syncthreads();
    if (tid == 0) m->nzero = 0;
    __syncthreads();
    if (tid < 64) {
      const long long row = r + (long long)tid * p.ctas;
      if (row < p.rows && row_entries(p, (int)row, &len) == 0) m->zero[atomicAdd(&m->nzero, 1)] = (int)row;
    }
    __syncthreads();
    for (int i = 0; i < m->nzero; ++i) {
      const int row = m->zero[i];
      const bool bad = __ldg(p.seqlens + row) > 0 && (p.idx == nullptr || p.k > 0);
      if (bad && tid == 0) raise_status(p.status, DSA_ERR_BAD_SEQLEN);
      const uint32_t v = bad ? 0x7fff7fffu : 0u;
      for (int j = tid; j < heads * (kLatent / 8); j += kAttnThreads) {
        const int h = head0 + j / (kLatent / 8);
        *reinterpret_cast<uint4*>(p.out + row * p.out_row + h * p.out_head + (j % (kLatent / 8)) * 8) =
            make_uint4(v, v, v, v);
      }
      if (p.lse && tid < heads) p.lse[(long long)row * p.H + head0 + tid] = bad ? CUDART_NAN_F : -CUDART_INF_F;
    }
  }
  __syncthreads();

  TileWalk walk;
  walk.start(p, m->start_row, m->start_tile, end - begin);
  Waiter wait{m, p.status, true};

  if (warp >= kLoadWarp0) {
    // ---- loaders -------------------------------------------------------------
    const int g = (warp - kLoadWarp0) / 4, w = (warp - kLoadWarp0) % 4;
    const uint32_t tile = sbase + g * kTileBytes;
    const int token_bytes = KV == DSA_KV_BF16 ? kTokenBytesBf16 : kLatent;
    if (g == 1) walk.step(p);
    for (int it = g; walk.left > 0; it += 2) {
      bool bad;
      int slot;
      const long long off =
          token_offset(p, walk, walk.t * kTile + w * kKeysPerWarp + (lane & 15), token_bytes, &bad, &slot);
      const uint32_t mask = __ballot_sync(0xffffffffu, off >= 0) & 0xffffu;
      const uint32_t badmask = __ballot_sync(0xffffffffu, bad);
      if (KV == DSA_KV_BF16) {
        if (it >= 2) wait(&m->empty[g], ((it >> 1) - 1) & 1);
        if (wait.ok) {
#pragma unroll
          for (int k = 0; k < kKeysPerWarp; ++k) {
            const long long o = __shfl_sync(0xffffffffu, off, k);
            const uint8_t* src = p.cache + (o < 0 ? 0 : o) + lane * 16;
            const int r = w * kKeysPerWarp + k;
            cp_async16(tile + swz(r, lane), src, o < 0 ? 0u : 16u);
            cp_async16(tile + swz(r, lane + 32), src + 512, o < 0 ? 0u : 16u);
          }
#pragma unroll
          for (int k4 = 0; k4 < kKeysPerWarp; k4 += 4) {
            const int k = k4 + lane / 8;
            const long long o = __shfl_sync(0xffffffffu, off, k);
            cp_async16(tile + swz(w * kKeysPerWarp + k, 64 + lane % 8),
                       p.cache + (o < 0 ? 0 : o) + kLatent * 2 + (lane % 8) * 16, o < 0 ? 0u : 16u);
          }
        }
      } else {
        // codes and scales into registers before the buffer is free
        uint4 codes[kKeysPerWarp];
        float scale[kKeysPerWarp];
        const int my_slot = slot;
#pragma unroll
        for (int k = 0; k < kKeysPerWarp; ++k) {
          const long long o = __shfl_sync(0xffffffffu, off, k);
          const int sl = __shfl_sync(0xffffffffu, my_slot, k);
          codes[k] = make_uint4(0u, 0u, 0u, 0u);
          scale[k] = 0.f;
          if (o >= 0) {
            codes[k] = __ldg(reinterpret_cast<const uint4*>(p.cache + o) + lane);
            // the page's start is o - slot * 512
            scale[k] = __ldg(reinterpret_cast<const float*>(p.cache + o - sl * kLatent + kScaleOffsetFp8) +
                             sl * kLatentGroups + lane / 8);
          }
        }
        if (it >= 2) wait(&m->empty[g], ((it >> 1) - 1) & 1);
        if (wait.ok) {
#pragma unroll
          for (int k4 = 0; k4 < kKeysPerWarp; k4 += 4) {
            const int k = k4 + lane / 8;
            const long long o = __shfl_sync(0xffffffffu, off, k);
            const int sl = __shfl_sync(0xffffffffu, my_slot, k);
            const uint8_t* src = p.cache + (o < 0 ? 0 : o - sl * kLatent + kRopeOffsetFp8 + sl * (kRope * 2));
            cp_async16(tile + swz(w * kKeysPerWarp + k, 64 + lane % 8), src + (lane % 8) * 16, o < 0 ? 0u : 16u);
          }
#pragma unroll
          for (int k = 0; k < kKeysPerWarp; ++k) {
            uint4 a, b;
            dequant16(codes[k], scale[k], a, b);
            const int r = w * kKeysPerWarp + k;
            // lanes 4-7 of each eight write their halves in the other order:
            // no two lanes of a store meet in a bank
            const int flip = (lane >> 2) & 1;
            st_shared_v4(tile + swz(r, 2 * lane + flip), flip ? b : a);
            st_shared_v4(tile + swz(r, 2 * lane + 1 - flip), flip ? a : b);
          }
        }
      }
      if (wait.ok) {
        if (lane == 0) m->keymask[g][w] = mask | (badmask ? 0x10000u : 0u);
        if (badmask && lane == 0) raise_status(p.status, DSA_ERR_BAD_PAGE);
        if (walk.first) {
          // this row's queries, by the group that brings the row's first tile
          if (walk.piece > 0) wait(&m->qfree, (walk.piece - 1) & 1);
          if (wait.ok) {
            for (int h = w * 16; h < w * 16 + 16; ++h) {
              const bool in = h < heads;
              const uint32_t n = in ? 16u : 0u;
              const long long hh = in ? head0 + h : head0;
              const uint16_t* ql = p.ql + walk.row * p.ql_row + hh * p.ql_head;
              const uint16_t* qr = p.qr + walk.row * p.qr_row + hh * p.qr_head;
              cp_async16(sbase + kOffQ + swz(h, lane), ql + lane * 8, n);
              cp_async16(sbase + kOffQ + swz(h, lane + 32), ql + 256 + lane * 8, n);
              if (lane < 8) cp_async16(sbase + kOffQ + swz(h, 64 + lane), qr + lane * 8, n);
            }
          }
        }
      }
      cp_async_wait_all();
      fence_proxy_async_smem();
#ifdef DSA_TEST_SKIP_FIRST_TILE
      // test builds only: never deliver the first tile, so that the waits for
      // it run out
      if (it == 0) {
        walk.step(p);
        if (walk.left > 0) walk.step(p);
        continue;
      }
#endif
      if (wait.ok) mbar_arrive(&m->full[g]);
      walk.step(p);
      if (walk.left > 0) walk.step(p);
    }
  } else if (warp == kMmaWarp) {
    // ---- MMA issue -----------------------------------------------------------
    if (lane == 0) {
      const uint32_t q = sbase + kOffQ, pt = sbase + kOffP;
      auto scores = [&](int it, bool last) {
        wait(&m->full[it & 1], (it >> 1) & 1);
        if (!wait.ok) return;
        tc_fence_after();
        fence_proxy_async_smem();
        const uint32_t a = sbase + (it & 1) * kTileBytes;
        const uint32_t d = tmem + kTmemS + (it & 1) * kAttnHeads;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16(d, smem_desc_sw128(a + b * kBlockBytes + k * 32, 1024),
                    smem_desc_sw128(q + b * kBlockBytes + k * 32, 1024), kIdescS, b + k > 0);
        mma_commit(&m->sfull[it & 1]);
        if (last) mma_commit(&m->qfree);
      };
      TileWalk ahead = walk;
      int it = 0;
      if (walk.left > 0) scores(0, walk.last());
      while (walk.left > 0) {
        ahead.step(p);
        const bool more = ahead.left > 0;
        // the next tile's scores go before this tile's values, except across
        // rows, where they wait for the next row's queries
        if (more && !ahead.first) scores(it + 1, ahead.last());
        wait(&m->pfull, it & 1);
        if (walk.first && walk.piece > 0) wait(&m->ofree, (walk.piece - 1) & 1);
        if (wait.ok) {
          tc_fence_after();
          const uint32_t a = sbase + (it & 1) * kTileBytes;
#pragma unroll
          for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f16(tmem + mt * kAttnHeads,
                      smem_desc_mn_sw128(a + mt * 2 * kBlockBytes + k * 2048, kBlockBytes, 1024),
                      smem_desc_mn_sw128(pt + k * 2048, kBlockBytes, 1024), kIdescO,
                      (k > 0 || !walk.first) ? 1u : 0u);
          mma_commit(&m->empty[it & 1]);
          if (walk.last()) mma_commit(&m->ofull);
        }
        if (more && ahead.first) scores(it + 1, ahead.last());
        walk = ahead;
        ++it;
      }
      if (!wait.ok) {
        // what was issued still runs: wait for it before TMEM is given back
        mma_commit(&m->done);
        mbar_wait_bounded(&m->done, 0, kWaitLimit);
      }
    }
    __syncwarp();
  } else {
    // ---- softmax and output --------------------------------------------------
    // this thread: keys 16 warp + gq and + 8, heads 8j + 2c and + 1
    const int gq = lane >> 2, c = lane & 3;
    const uint32_t my_lanes = (uint32_t)(warp * 32) << 16;
    const uint32_t prow = sbase + kOffP + (warp * 16 + gq) * 128;
    float mx[16], sum[16];
    bool bad = false;
    int split_row = -1, split_last = 0;
    long long tile_at = begin;                 // global index of the current tile
    for (int it = 0; walk.left > 0; ++it) {
      if (walk.first) {
#pragma unroll
        for (int j = 0; j < 16; ++j) mx[j] = -CUDART_INF_F, sum[j] = 0.f;
        bad = false;
      }
      wait(&m->sfull[it & 1], (it >> 1) & 1);
      wait(&m->full[it & 1], (it >> 1) & 1);   // the loaders' key mask
      __syncwarp();
      tc_fence_after();
      uint32_t r[32];
      tmem_ld_16x256b_x8(tmem + my_lanes + kTmemS + (it & 1) * kAttnHeads, r);
      const uint32_t km = *reinterpret_cast<volatile uint32_t*>(&m->keymask[it & 1][warp]);
      const bool v0 = (km >> gq) & 1, v1 = (km >> (gq + 8)) & 1;
      bad |= (km >> 16) & 1;
      tmem_ld_wait32(r);
      float s[32];
      bool over = false;
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float a = v0 ? __uint_as_float(r[4 * j + e]) * p.scale_log2 : -CUDART_INF_F;
          const float b = v1 ? __uint_as_float(r[4 * j + 2 + e]) * p.scale_log2 : -CUDART_INF_F;
          s[4 * j + e] = a, s[4 * j + 2 + e] = b;
          const float lim = mx[2 * j + e] + kSlack;
          over |= a > lim || b > lim;
        }
      // P's buffer and O^T are free once the previous tile's values are added
      if (it > 0) wait(&m->empty[(it - 1) & 1], ((it - 1) >> 1) & 1);
      if (bar_any(1, 128, over)) {
        float top[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float v = fmaxf(s[4 * (j / 2) + j % 2], s[4 * (j / 2) + 2 + j % 2]);
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
          top[j] = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        }
        if (gq == 0)
#pragma unroll
          for (int j = 0; j < 16; ++j) m->red[warp][8 * (j / 2) + 2 * c + j % 2] = top[j];
        bar_sync(1, 128);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int h = 8 * (j / 2) + 2 * c + j % 2;
          const float v = fmaxf(fmaxf(m->red[0][h], m->red[1][h]), fmaxf(m->red[2][h], m->red[3][h]));
          const float now = fmaxf(mx[j], v);
          const float f = now == mx[j] ? 1.f : ex2(mx[j] - now);
          mx[j] = now;
          sum[j] *= f;
          if (warp == 0 && gq == 0) m->fac[h] = f;
        }
        if (!walk.first) {
          bar_sync(1, 128);
          tc_fence_after();
#pragma unroll 1
          for (int col = 0; col < 4 * kAttnHeads; col += 32) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(tmem + my_lanes + col, o);
            tmem_ld_wait32(o);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              o[j] = __float_as_uint(__uint_as_float(o[j]) * m->fac[(col & 32) + j]);
            tmem_st_32x32b_x32(tmem + my_lanes + col, o);
          }
          tmem_st_wait();
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float pr[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float ref = mx[2 * j + e] == -CUDART_INF_F ? 0.f : mx[2 * j + e];
          pr[e] = ex2(s[4 * j + e] - ref);
          pr[2 + e] = ex2(s[4 * j + 2 + e] - ref);
          sum[2 * j + e] += pr[e] + pr[2 + e];
        }
        const __nv_bfloat162 lo = __floats2bfloat162_rn(pr[0], pr[1]), hi = __floats2bfloat162_rn(pr[2], pr[3]);
        // rows gq and gq + 8 swizzle alike
        const uint32_t at = prow + ((j ^ gq) << 4) + c * 4;
        st_shared_u32(at, *reinterpret_cast<const uint32_t*>(&lo));
        st_shared_u32(at + 8 * 128, *reinterpret_cast<const uint32_t*>(&hi));
      }
      fence_proxy_async_smem();
      tc_fence_before();
      if (wait.ok) mbar_arrive(&m->pfull);
      ++tile_at;

      if (walk.last()) {
        // ---- the piece's result ------------------------------------------------
        const bool whole = walk.t + 1 == walk.tiles() && tile_at - begin >= walk.tiles();
        const bool begins = tile_at - begin > walk.t;   // the piece holds the row's first tile
        bar_sync(1, 128);                               // every use of red and fac is over
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 4);
          sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 8);
          sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 16);
        }
        if (gq == 0)
#pragma unroll
          for (int j = 0; j < 16; ++j) m->red[warp][8 * (j / 2) + 2 * c + j % 2] = sum[j];
        if (warp == 0 && gq == 0)
#pragma unroll
          for (int j = 0; j < 16; ++j) m->fac[8 * (j / 2) + 2 * c + j % 2] = mx[j];
        wait(&m->ofull, walk.piece & 1);
        bad = bar_any(1, 128, bad || !wait.ok);
        float* slot = p.ws + ((long long)blockIdx.x * 2 + (begins ? 1 : 0)) * kPartialFloats;
        float total_h = 0.f, max_h = 0.f;
        if (warp < 2) {
          const int h = warp * 32 + lane;
          total_h = m->red[0][h] + m->red[1][h] + m->red[2][h] + m->red[3][h];
          max_h = m->fac[h];
          if (bad) total_h = CUDART_NAN_F, max_h = 0.f;
        }
        bar_sync(1, 128);
        if (warp < 2) {
          const int h = warp * 32 + lane;
          if (whole) {
            m->fac[h] = bad ? CUDART_NAN_F : total_h == 0.f ? 0.f : 1.f / total_h;
            if (p.lse && h < heads)
              p.lse[(long long)walk.row * p.H + head0 + h] = (max_h + log2f(total_h)) * 0.69314718055994531f;
          } else {
            m->fac[h] = bad ? CUDART_NAN_F : 1.f;
            slot[kAttnHeads * kLatent + h] = max_h;
            slot[kAttnHeads * kLatent + kAttnHeads + h] = total_h;
          }
        }
        bar_sync(1, 128);
        tc_fence_after();
#pragma unroll 1
        for (int col = 0; col < 4 * kAttnHeads; col += 32) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(tmem + my_lanes + col, o);
          tmem_ld_wait32(o);
          const int h0 = col & 32, dim = (col / kAttnHeads) * 128 + warp * 32 + lane;
          if (col == 4 * kAttnHeads - 32) {
            tc_fence_before();
            if (wait.ok) mbar_arrive(&m->ofree);
          }
          if (whole) {
            // two heads of a lane pair: each lane writes two values of one head
            uint16_t* dst = p.out + walk.row * p.out_row + (dim & ~1);
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float a = __uint_as_float(o[j]) * m->fac[h0 + j];
              const float b = __uint_as_float(o[j + 1]) * m->fac[h0 + j + 1];
              const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? a : b, 1);
              const __nv_bfloat162 v =
                  lane & 1 ? __floats2bfloat162_rn(other, b) : __floats2bfloat162_rn(a, other);
              const int h = h0 + j + (lane & 1);
              if (h < heads)
                *reinterpret_cast<__nv_bfloat162*>(dst + (long long)(head0 + h) * p.out_head) = v;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (h0 + j < heads) slot[(h0 + j) * kLatent + dim] = __uint_as_float(o[j]) * m->fac[h0 + j];
          }
        }
        bar_sync(1, 128);   // fac and red are free again
        if (!whole && begins) {
          // the row goes on in later CTAs: the one that holds its last tile
          const long long last_tile = tile_at - 1 + (walk.tiles() - 1 - walk.t);
          split_row = walk.row;
          split_last = (int)(((last_tile + 1) * ctas - 1) / total);
        }
      }
      walk.step(p);
    }
    if (tid == 0) {
      int* rec = reinterpret_cast<int*>(p.ws + (long long)gridDim.x * 2 * kPartialFloats) +
                 (long long)blockIdx.x * kSplitInts;
      rec[0] = split_row;
      rec[1] = split_last;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// Joins the partial sums of one row that slices cut: grid (CTA whose piece
// begins the row, four heads), a head per 128 threads.
constexpr int kJoinHeads = 4;
__global__ void __launch_bounds__(kJoinHeads * 128) latent_join_kernel(const LatentAttnParams p, int main_ctas) {
  griddep_wait();
  griddep_launch_dependents();
  const int* rec = reinterpret_cast<const int*>(p.ws + (long long)main_ctas * 2 * kPartialFloats) +
                   (long long)blockIdx.x * kSplitInts;
  const int row = rec[0], last = rec[1];
  if (row < 0) return;
  const int cta = blockIdx.x / p.groups, grp = blockIdx.x % p.groups;
  const int h = blockIdx.y * kJoinHeads + threadIdx.x / 128, d = (threadIdx.x % 128) * 4;
  const int head = grp * kAttnHeads + h;
  if (head >= p.H) return;
  const long long step = (long long)p.groups * 2 * kPartialFloats;
  const float* first = p.ws + ((long long)blockIdx.x * 2 + 1) * kPartialFloats;
  // the later pieces lie in slot 0 of their CTAs
  const float* rest = p.ws + (long long)blockIdx.x * 2 * kPartialFloats + step;
  const int n = last - cta;
  float top = first[kAttnHeads * kLatent + h];
  for (int i = 0; i < n; ++i) top = fmaxf(top, rest[i * step + kAttnHeads * kLatent + h]);
  const float ref = top == -CUDART_INF_F ? 0.f : top;
  float wgt = ex2(first[kAttnHeads * kLatent + h] - ref);
  float total = first[kAttnHeads * kLatent + kAttnHeads + h] * wgt;
  float4 v = *reinterpret_cast<const float4*>(first + h * kLatent + d);
  float4 acc = make_float4(v.x * wgt, v.y * wgt, v.z * wgt, v.w * wgt);
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float* s = rest + i * step;
    wgt = ex2(s[kAttnHeads * kLatent + h] - ref);
    total = fmaf(s[kAttnHeads * kLatent + kAttnHeads + h], wgt, total);
    v = *reinterpret_cast<const float4*>(s + h * kLatent + d);
    acc.x = fmaf(v.x, wgt, acc.x);
    acc.y = fmaf(v.y, wgt, acc.y);
    acc.z = fmaf(v.z, wgt, acc.z);
    acc.w = fmaf(v.w, wgt, acc.w);
  }
  const float inv = total == 0.f ? 0.f : 1.f / total;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(p.out + row * p.out_row + head * p.out_head + d) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  if (p.lse && threadIdx.x % 128 == 0)
    p.lse[(long long)row * p.H + head] = (top + log2f(total)) * 0.69314718055994531f;
}

template <int KV>
cudaError_t launch_t(LatentAttnParams p, int sms, cudaStream_t stream) {
  p.ctas = sms / p.groups;
  cudaError_t e = cudaFuncSetAttribute(latent_attention_kernel<KV>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.ctas * p.groups);
  cfg.blockDim = dim3(kAttnThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, latent_attention_kernel<KV>, p);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t join = cfg;
  join.gridDim = dim3(p.ctas * p.groups, (min(p.H, kAttnHeads) + kJoinHeads - 1) / kJoinHeads);
  join.blockDim = dim3(kJoinHeads * 128);
  join.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&join, latent_join_kernel, p, (int)(p.ctas * p.groups));
}

}  // namespace

cudaError_t launch_latent_attention(const LatentAttnParams& p, int kv_dtype, int sms, cudaStream_t stream) {
  if (kv_dtype == DSA_KV_BF16) return launch_t<DSA_KV_BF16>(p, sms, stream);
  return launch_t<DSA_KV_FP8_E4M3>(p, sms, stream);
}

}  // namespace dsa
