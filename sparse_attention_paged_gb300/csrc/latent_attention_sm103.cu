// latent_attention_sm103.cu -- attention of H query heads over the cached
// latent tokens of a row, in the absorbed form:
//
//   s[h, t] = scale * (ql[h] . c[t] + qr[h] . r[t])      c: 512 values, r: 64
//   p[h, :] = softmax(s[h, :]) over the row's visible tokens
//   out[h]  = sum_t p[h, t] c[t],   lse[h] = log sum_t exp(s[h, t])
//
// One token serves as key and value of every head, so a tile of 128 tokens is
// brought into shared memory once (16-bit, nine blocks of 64 values, 128-byte
// swizzle) and feeds both products as it lies there:
//
//   S^T [128 tokens x 64 heads] = tile [128 x 576] (A, K-major) * Q^T (B, K-major)
//   O^T [512 values x 64 heads] += tile^T (A, MN-major) * P^T (B, MN-major)
//
// Keeping the heads on the N side leaves O^T at 4 x 64 TMEM columns, gives
// every softmax thread one token, and makes a token's mask a whole row.  The
// softmax warps keep a reference per head that is raised only when a weight
// passes it by 2^8 (fp8: 2^9), and then O^T is rescaled in TMEM; the sums are
// fp32, so the reference does not change their relative precision.
//
// bf16 cache: tile, queries and weights are bf16.  The weights' rounding
// (nearest, 2^-8) is independent from token to token and below that of the
// bf16 result.
//
// fp8 cache: tile, latent queries and weights are fp16, which holds e4m3
// exactly and takes one conversion where bf16 takes four instructions.  With
// s(t) a power of two times one of token t's four scales, the tile holds code *
// s_g / s(t), the scores are multiplied by s(t) and the weights written as w *
// s(t).  s(t) is 2^4 of the smallest scale, which leaves the tile the smallest
// codes in full and gives small tokens beside large ones more of the weights'
// range, but at least 2^-7 of the largest, as 448 * 2^7 is still an fp16 number.
// For scales that are powers of two the tile is exact down to 2^-22 of the
// token's largest scale, rounded to 2^-32 of it below, and a group of 2^-32 of it
// or less counts as zeros; a group that does hold zeros has no say in s(t).  A
// head's queries are scaled by a power of two that brings the largest of the
// latent part below 2^15 and of the rotated part below 2^61, so that any finite
// bf16 values fit; the rotated part stays bf16 in an accumulator of its own.  The reference is kept on w * s(t): the largest lie
// between 2^6 and 2^15, what is 2^-20 of them is still a normal number, and
// what is below is rounded to 2^-31 of them.
//
// Shared memory holds one tile (144 KB) and the row's queries (72 KB); the
// tile is refilled part by part: the value product takes the latent parts of
// 128 values in order and gives each back as soon as it is used, the score
// product of the next tile takes them in the same order as they arrive.  P
// lies where the rotated part was, which only the score product reads.
//
// Persistent: the call's 128-token units (per head group of 64; 64-token where
// a few short rows have no more than one for each CTA) are cut into
// equal slices, one per CTA, rows in order.  A row that a slice cuts leaves
// unnormalised partial sums in the workspace, and a second kernel joins
// them, so one long row or a few short ones spread over every SM, and a
// batch of any lengths is balanced.
//
// Warps: 0-7 softmax and output, 8 MMA issue, 9-11 token lookup, 12-19
// loaders.  The lookup warps go through selection list and block table up to
// three tiles ahead and ask L2 for a tile's bytes when the tile before it
// arrives, which keeps HBM busy whatever the tile buffer does (152 rows of
// 8,192 fp8 tokens 264 us, 335 without).  The loaders copy (bf16) or convert (fp8) 16
// bytes at a time; masked tokens are not read, their rows are zeros.
//
// Measured (both kernels; 64 heads where not said otherwise; in a captured graph
// with warm inputs, and as single calls with inputs out of L2): 64 rows of 2,048
// selected tokens each, bf16, 49 and 53 us; 64 rows of 512 to 32,768 tokens, fp8,
// 138 both; one row of 131,072 bf16 tokens and 128 heads 58 and 63; 1,024 fp8
// prefill rows of 2,048 selected tokens 478 and 485 (610 TFLOP/s); one row of 512
// and 16 heads 11.4 and 11.6; 152 rows of 8,192 tokens 262 in either type (5.5
// and 3.1 TB/s).
// What bounds it: a tile's chain.  Value product (1,536 cycles of operand
// reads), the next tile's scores (1,728) and softmax (1,150 to 1,600) follow
// one another, since only one tile fits: 5,750 cycles a bf16 tile, 6,000 to
// 7,000 an fp8 tile, whose conversion stores share shared memory with the
// products.  Few rows: 6 us from the launch to the first tokens' addresses
// (lengths, list and table, one DRAM trip each), the first tile, the join.
// Tiles of 64 tokens in two buffers overlapped more but ran their products at
// half rate: the prefill took 1,316 us, the ragged rows 366.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stddef.h>
#include <stdint.h>

#include "latent_common.cuh"
#include "sm100_ptx.cuh"

#ifndef DSA_WAIT_LIMIT_CYCLES
#define DSA_WAIT_LIMIT_CYCLES 4000000000ll
#endif

namespace dsa {

namespace {

using namespace sm100;

constexpr int kTileShift = 7, kTile = 1 << kTileShift;  // tokens per tile, and per unit of the split
// Few rows that have no more than half tiles enough for every CTA are cut
// into those: one row of 512 tokens then runs on eight CTAs.
constexpr int kFewRows = 32;
constexpr int kParts = 4;                       // latent parts of 128 values; the rotated part follows
constexpr int kBlockBytes = kTile * 128;        // 64 values of a tile's tokens
constexpr int kPartBytes = 2 * kBlockBytes;
constexpr int kRopeBlock = 8;                   // index of the rotated part's block
constexpr int kQBlockBytes = kAttnHeads * 128;  // 64 values of the queries
constexpr int kSoftmaxWarps = 8, kMmaWarp = 8, kLookWarp0 = 9, kLookWarps = 3, kLoadWarp0 = 12, kLoadWarps = 8;
constexpr int kAttnThreads = (kLoadWarp0 + kLoadWarps) * 32;
// Tiles of looked-up tokens: one slot per lookup warp, so that no warp can be
// two phases of a slot's barrier ahead of another.
constexpr int kRing = kLookWarps;
constexpr int kKeysPerWarp = kTile / kLoadWarps;  // 16
constexpr int kHeadsPerWarp = kAttnHeads / kLoadWarps;  // 8
// Registers per thread: at launch (65,536 / 640 in steps of 8), then per role.
constexpr int kRegsLaunch = 96, kRegsSoftmax = 104, kRegsMisc = 72, kRegsLoad = 96;
static_assert(kSoftmaxWarps * kRegsSoftmax + 4 * kRegsMisc + kLoadWarps * kRegsLoad <=
                  kAttnThreads / 32 * kRegsLaunch,
              "the roles' registers are those of the launch");
static_assert(kSoftmaxWarps % 4 == 0 && kMmaWarp % 4 == 0 && kLoadWarp0 % 4 == 0 && kLoadWarps % 4 == 0,
              "a register count holds for a warpgroup of four warps");
// The reference (log2 units): a new one is set ref_below under the largest
// weight, and holds until a weight is ref_limit above it.
constexpr float ref_below(int kv) { return kv == DSA_KV_BF16 ? 0.f : 6.f; }
constexpr float ref_limit(int kv) { return kv == DSA_KV_BF16 ? 8.f : 15.f; }
constexpr uint32_t kUnset = 0x80000000u;        // bits of -reference (-0) before the first visible token
// s(t) over the largest of a token's scales at least, and over the smallest
constexpr float kScaleBelowTop = 1.f / 128, kScaleAboveLow = 16.f;
// A head's rotated queries may be up to 2^46 of its latent ones under the power
// of two that suits those: 2^61, far from bf16's limit and that of the sums.
constexpr float kRopeRoom = 1.4210854715202004e-14f;  // 2^-46
constexpr float kSmallestScale = 7.8886090522101181e-31f;  // 2^-100: keeps 1 / s and the sums in range

// Shared memory, from a 1,024-byte boundary.
constexpr int kOffQ = 9 * kBlockBytes;
constexpr int kOffMisc = kOffQ + 9 * kQBlockBytes;
constexpr int kOffP = kRopeBlock * kBlockBytes;
struct Misc {
  uint64_t full[kParts + 1];   // a part of the tile is in place (rotated part last; part 0: the queries too)
  uint64_t empty[kParts];      // the value product is done with the part; the last: with the tile
  uint64_t sfull;              // S^T is there
  uint64_t pfull;              // P is there
  uint64_t ofree;              // O^T has been read
  uint64_t qfirst;             // the first row's queries are there
  uint64_t look_full[kRing], look_empty[kRing], scale_full[kRing];
  uint64_t done;
  uint32_t tmem;
  int start_row, start_unit, nzero, shift;
  int begin, end, total, ctas; // the slice's units, the call's units, the CTAs that have one
  int scan[kAttnThreads / 32];
  alignas(16) uint2 ratio[kRing][kTile];  // fp8: each part's scale over s(t), fp16
  int token[kRing][kTile];     // page * 64 + slot, -1 when masked
  float key_scale[kRing][kTile];  // fp8: s(t)
  uint32_t mask[kRing][4];     // valid tokens
  int4 tile[kRing];            // row, tokens, flags, piece; flags: kFirst: a row or a part of one begins;
                               // kLast: it ends; kEnd: so does the slice; kBad: a visible token has no page
  int4 piece[8];               // of the rows or parts under way: row, kBegins | kWhole
  alignas(16) float red[4][kAttnHeads];  // per quarter of the tokens and head
  float nref[kAttnHeads];      // -reference, in log2 units; nref, mul, fac are read as float4
  float mul[2][kAttnHeads];    // fp8: from a head's score sums to log2 units, this row's and the next one's
  float fac[kAttnHeads], keep[kAttnHeads];
};
constexpr int kFirst = 1, kLast = 2, kEnd = 4, kBad = 8;
constexpr int kBegins = 1, kWhole = 2;          // a part holds its row's first unit / all of them
constexpr int kMiscBytes = 9 * 1024;
constexpr int kSmemBytes = kOffMisc + kMiscBytes + 1024;
static_assert(sizeof(Misc) <= kMiscBytes, "misc");
static_assert(kSmemBytes <= 232448, "227 KB");
static_assert(offsetof(Misc, nref) % 16 == 0 && offsetof(Misc, mul) % 16 == 0 && offsetof(Misc, fac) % 16 == 0 &&
                  offsetof(Misc, ratio) % 8 == 0 && kOffMisc % 16 == 0,
              "vector reads");

// TMEM columns: O^T 4 x 64, S^T 64, the rotated part's S^T (fp8) 64.
constexpr uint32_t kTmemS = 256, kTmemR = 320, kTmemCols = 512;

// at most about a second: the clock's low 32 bits are compared
constexpr uint32_t kWaitLimit = DSA_WAIT_LIMIT_CYCLES < 2000000000ll ? DSA_WAIT_LIMIT_CYCLES : 2000000000ll;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// The same for bytes of the cache.  Without the hint a line that has been
// prefetched and read outlives in L2 those that were prefetched after it, and
// they are fetched twice: 152 rows of 8,192 bf16 tokens read 2.3 GB of 1.43
// and took 398 us, with it 264.  Rows that share their tokens keep them all
// the same: 1,024 prefill rows of 2,048 out of 131,072 take 391 us and 393.
__device__ __forceinline__ uint64_t evict_first() {
  uint64_t r;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(r));
  return r;
}
__device__ __forceinline__ void cp_async16_once(uint32_t dst, const void* src, uint32_t bytes, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes),
               "l"(policy)
               : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// All but the last N groups of this thread.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Every copy of this thread, committed to a group or not.
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// 16 bytes that are read once: not kept in L1
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Ask L2 for a line / for `bytes` (a multiple of 16, 16-byte aligned).
__device__ __forceinline__ void l2_prefetch(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

__device__ __forceinline__ void l2_prefetch_bulk(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Whether phase `parity` of `bar` is complete, without waiting.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

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

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 32 lanes x 8 columns of TMEM, and the waits for them
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_wait8(uint32_t (&a)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_ld_wait8(uint32_t (&a)[8], uint32_t (&b)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]),
                 "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]), "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Descriptor of an MN-major operand in the 128-byte swizzle: 64 M/N values of
// one K index are a 128-byte row, eight K rows an atom; `k_bytes` from one
// atom to the next along K, `mn_bytes` to the next 64 M/N values.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t mn_bytes, uint32_t k_bytes) {
  uint64_t d = smem_desc_sw128(saddr, k_bytes);
  d &= ~((uint64_t)0x3FFFu << 16);
  d |= (uint64_t)((mn_bytes >> 4) & 0x3FFFu) << 16;
  return d;
}

// Instruction descriptors: formats 0 = fp16, 1 = bf16; O^T with A and B MN-major.
constexpr uint32_t format(int kv) { return kv == DSA_KV_BF16 ? 1u : 0u; }
constexpr uint32_t idesc_s(int kv) { return instr_desc(format(kv), format(kv), kTile, kAttnHeads); }
constexpr uint32_t idesc_o(int kv) {
  return instr_desc(format(kv), format(kv), 128, kAttnHeads) | (1u << 15) | (1u << 16);
}
constexpr uint32_t kIdescRope = instr_desc(1, 1, kTile, kAttnHeads);

// A row's visible entries: its length, or the part of its selection list that
// is read.  A length past the block table is an error: no entries.
__device__ __forceinline__ int row_entries(const LatentAttnParams& p, int row, int* len) {
  const int L = __ldg(p.seqlens + row);
  *len = L;
  if (L <= 0 || (long long)L > (long long)p.W * kPage) return 0;
  return p.idx ? min(L, p.k) : L;
}

// Units of 2^shift tokens; entries >= 0.
__device__ __forceinline__ int units_of(int entries, int shift) { return ((entries - 1) >> shift) + 1; }

__device__ __forceinline__ int row_units(const LatentAttnParams& p, int row) {
  int len;
  return units_of(row_entries(p, row, &len), kTileShift);
}

// Walks the tiles of a CTA's slice, row by row; rows without units are passed.
// A tile is a unit of one row: kTile tokens or half of that.
struct TileWalk {
  int row, u, n, len, left, piece, shift = kTileShift;
  bool first;
  __device__ __forceinline__ int units() const { return units_of(n, shift); }
  __device__ __forceinline__ int tokens() const { return min(n - (u << shift), 1 << shift); }
  __device__ __forceinline__ bool last() const { return left == 1 || u + 1 == units(); }
  __device__ __forceinline__ void start(const LatentAttnParams& p, int row0, int unit0, int units) {
    row = row0, u = unit0, left = units, piece = 0, first = true, n = 0, len = 0;
    if (left > 0) n = row_entries(p, row, &len);
  }
  __device__ __forceinline__ void step(const LatentAttnParams& p) {
    if (--left <= 0) return;
    ++u;
    first = false;
    if (u < units()) return;
    do {
      n = row_entries(p, ++row, &len);
    } while (n == 0 && row + 1 < p.rows);
    u = 0, first = true, ++piece;
  }
};

// Waits, by a whole warp together (every lane asks, and all get the same
// answer: the hardware then puts the warp to sleep, which it does not when
// one lane asks for the others) or by one lane.  After one that ran out the
// rest return at once.
template <bool WARP>
struct Waiter {
  int* status;
  bool ok;
  __device__ __forceinline__ bool reached(uint64_t* bar, uint32_t parity) {
    const bool r = mbar_try_wait(bar, parity);
    return WARP ? __all_sync(0xffffffffu, r) : r;
  }
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) {
    if (!ok) return false;
    if (reached(bar, parity)) return true;
    const uint32_t t0 = (uint32_t)clock();
#pragma unroll 1
    do {
      if (reached(bar, parity)) return true;
      const bool late = (uint32_t)clock() - t0 > kWaitLimit;
      ok = WARP ? !__any_sync(0xffffffffu, late) : !late;
    } while (ok);
    raise_status(status, DSA_ERR_TIMEOUT);
    return false;
  }
};

// Every lane's writes to shared memory, made visible to the MMA, before one
// lane arrives for the warp.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Which of the groups in `ask` (bits 0-3) of a token's codes are zeros, of either
// sign.  Those that are not show it in their first 16 codes almost always.
__device__ __forceinline__ uint32_t zero_groups(const uint8_t* codes, uint32_t ask) {
  auto value = [&](int group, int j) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(codes + group * kLatentGroup) + j);
    return ((v.x | v.y | v.z | v.w) & 0x7f7f7f7fu) != 0;
  };
#pragma unroll
  for (int g = 0; g < kLatentGroups; ++g)
    if (value(g, 0)) ask &= ~(1u << g);
  uint32_t zeros = 0;
#pragma unroll 1
  for (; ask; ask &= ask - 1) {
    const int g = __ffs(ask) - 1;
    bool any = false;
#pragma unroll
    for (int j = 1; j < kLatentGroup / 16; ++j) any |= value(g, j);
    if (!any) zeros |= 1u << g;
  }
  return zeros;
}

// Eight e4m3 codes times `f` (a factor twice, fp16), 16 bytes of fp16.
__device__ __forceinline__ uint4 widen8(uint32_t lo, uint32_t hi, uint32_t f) {
  const uint32_t u[2] = {lo, hi};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u[j >> 1] >> (16 * (j & 1))), __NV_E4M3);
    const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&r), *reinterpret_cast<const __half2*>(&f));
    o[j] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Eight bf16 values (16 bytes) as floats.
__device__ __forceinline__ void unpack8(const uint4& r, float (&v)[8]) {
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

// The largest magnitude of eight bf16 values; NaN does not count.
__device__ __forceinline__ float largest8(const uint4& r) {
  auto size = [](uint32_t u) {
    u &= 0x7fff7fffu;
    return *reinterpret_cast<const __nv_bfloat162*>(&u);
  };
  const __nv_bfloat162 m = __hmax2(__hmax2(size(r.x), size(r.y)), __hmax2(size(r.z), size(r.w)));
  return fmaxf(__low2float(m), __high2float(m));
}

// The largest value of a warp's lanes; NaN does not count.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Two floats in one register pair: half the instructions.
using F2 = unsigned long long;

__device__ __forceinline__ F2 pair(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 pair(uint32_t a, uint32_t b) { return pair(__uint_as_float(a), __uint_as_float(b)); }
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

// Sums 32 values per lane (16 pairs) over the warp's lanes: lane l gets sum l.
__device__ __forceinline__ float sum_columns(const F2 (&pairs)[16], int lane) {
  float v[32];
#pragma unroll
  for (int j = 0; j < 16; ++j) unpair(pairs[j], v[2 * j], v[2 * j + 1]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const bool up = lane & o;
      const float give = up ? v[j] : v[j + o], keep = up ? v[j + o] : v[j];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  return v[0];
}

// The split records, {row or -1, CTA with its last unit, CTA with its first, 0}:
// one per row where there are no more rows than CTAs (-1: nothing to join),
// else one per CTA, for the row that its slice begins and does not end.
__device__ __forceinline__ bool records_by_row(const LatentAttnParams& p) { return p.rows <= p.ctas; }

__device__ __forceinline__ void record_split(const LatentAttnParams& p, int row, bool split, int last) {
  const int grp = blockIdx.x % p.groups, cta = blockIdx.x / p.groups;
  if (!split && !records_by_row(p)) return;       // the CTA's -1 is there from the start
  reinterpret_cast<int4*>(p.ws + (long long)gridDim.x * 2 * kPartialFloats)[(records_by_row(p) ? row : cta) * p.groups +
                                                                            grp] =
      make_int4(split ? row : -1, last, cta, 0);
}

// What a masked token's codes are read from.
__device__ const uint4 g_zeros[kLatent / 16] = {};

// Brings `count` heads' queries of a row to their place, head by head, UNROLL
// heads' loads at a time.  bf16: as they are (cp.async; the caller waits for
// them).  fp8: the latent part as fp16, both parts times a power of two that
// brings the head's largest into [2^14, 2^15) (the rotated part counted as
// kRopeRoom of itself; values below 2^-86 times 2^100), and the factor that takes the
// scores back into `mul`.  Heads past `heads` are zeros.
template <int KV, int UNROLL>
__device__ __forceinline__ void load_queries(const LatentAttnParams& p, int row, int head0, int heads, int first,
                                             int count, uint32_t sbase, int lane, float* mul) {
  const int sub = lane >> 3, col = lane & 7;
  const uint16_t* ql = p.ql + row * p.ql_row + head0 * p.ql_head;
  const uint16_t* qr = p.qr + row * p.qr_row + head0 * p.qr_head;
  if constexpr (KV == DSA_KV_BF16) {
#pragma unroll 2
    for (int h = first; h < first + count; ++h) {
      const uint32_t n = h < heads ? 16u : 0u;
      const uint16_t* src = ql + (h < heads ? h : 0) * p.ql_head + lane * 8;
      const uint32_t dst = sbase + kOffQ + sub * kQBlockBytes + h * 128 + ((col ^ (h & 7)) << 4);
      cp_async16(dst, src, n);
      cp_async16(dst + 4 * kQBlockBytes, src + 256, n);
    }
#pragma unroll 1
    for (int h = first + sub; h < first + count; h += 4)
      cp_async16(sbase + kOffQ + kRopeBlock * kQBlockBytes + h * 128 + ((col ^ (h & 7)) << 4),
                 qr + (h < heads ? h : 0) * p.qr_head + col * 8, h < heads ? 16u : 0u);
  } else {
#pragma unroll 1
    for (int h0 = first; h0 < first + count; h0 += UNROLL) {
      uint4 a[UNROLL], b[UNROLL], r[UNROLL];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int h = h0 + u;
        a[u] = b[u] = r[u] = make_uint4(0u, 0u, 0u, 0u);
        if (h < heads) {
          const uint4* src = reinterpret_cast<const uint4*>(ql + h * p.ql_head) + lane;
          a[u] = __ldg(src);
          b[u] = __ldg(src + 32);
          if (lane < 8) r[u] = __ldg(reinterpret_cast<const uint4*>(qr + h * p.qr_head) + lane);
        }
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int h = h0 + u;
        float x[8], y[8];
        unpack8(a[u], x);
        unpack8(b[u], y);
        float top = largest8(r[u]) * kRopeRoom;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, fmaxf(fabsf(x[j]), fabsf(y[j])));
        top = warp_max(top);
        const int n = top > 0.f ? min(127 + 14 - (int)(__float_as_uint(top) >> 23), 100) : 0;
        const float f = __uint_as_float((uint32_t)(n + 127) << 23);
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __half2 lo = __floats2half2_rn(x[2 * j] * f, x[2 * j + 1] * f);
          const __half2 hi = __floats2half2_rn(y[2 * j] * f, y[2 * j + 1] * f);
          o[j] = *reinterpret_cast<const uint32_t*>(&lo);
          o[4 + j] = *reinterpret_cast<const uint32_t*>(&hi);
        }
        const uint32_t dst = sbase + kOffQ + h * 128 + ((col ^ (h & 7)) << 4);
        st_shared_v4(dst + sub * kQBlockBytes, make_uint4(o[0], o[1], o[2], o[3]));
        st_shared_v4(dst + (4 + sub) * kQBlockBytes, make_uint4(o[4], o[5], o[6], o[7]));
        if (lane < 8) {
          unpack8(r[u], x);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * j] * f, x[2 * j + 1] * f);
            o[j] = *reinterpret_cast<const uint32_t*>(&v);
          }
          st_shared_v4(dst + kRopeBlock * kQBlockBytes, make_uint4(o[0], o[1], o[2], o[3]));
        }
        if (lane == 0) mul[h] = p.scale_log2 * __uint_as_float((uint32_t)(127 - n) << 23);
      }
    }
  }
}

template <int KV>
__global__ void __launch_bounds__(kAttnThreads, 1) latent_attention_kernel(const LatentAttnParams p) {
  constexpr bool kFp8 = KV != DSA_KV_BF16;
  extern __shared__ uint8_t smem_raw[];
  // an offset, not a rounded address: the compiler keeps seeing shared memory
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Misc* m = reinterpret_cast<Misc*>(smem + kOffMisc);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int cta = blockIdx.x / p.groups, grp = blockIdx.x % p.groups;
  const int head0 = grp * kAttnHeads, heads = min(kAttnHeads, p.H - head0);

  if (tid == 0) {
    for (int i = 0; i <= kParts; ++i) mbar_init(&m->full[i], kLoadWarps);
    for (int i = 0; i < kParts; ++i) mbar_init(&m->empty[i], 1);
    mbar_init(&m->sfull, 1);
    mbar_init(&m->pfull, kSoftmaxWarps);
    mbar_init(&m->ofree, kSoftmaxWarps);
    mbar_init(&m->qfirst, kSoftmaxWarps);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&m->look_full[i], 1);
      mbar_init(&m->scale_full[i], 1);
      mbar_init(&m->look_empty[i], kLoadWarps + kSoftmaxWarps);
    }
    mbar_init(&m->done, 1);
    fence_barrier_init();
    m->start_row = m->start_unit = m->nzero = 0;
  }
  if (tid < kAttnHeads) m->nref[tid] = __uint_as_float(kUnset);
  if (warp == kMmaWarp) {
    tmem_alloc(&m->tmem, kTmemCols);
    tmem_relinquish();
  }
  griddep_wait();
  griddep_launch_dependents();

  // ---- the slice -----------------------------------------------------------
  // thread i owns a run of rows; an exclusive scan of the runs' unit counts
  // finds the row in which this CTA's slice begins
  TileWalk walk;
  {
    int begin = 0, end = 0, total = 0, ctas = 0, start_row = 0, start_unit = 0;
    // the equal part of `total` units that this CTA takes
    auto take = [&] {
      ctas = min(p.ctas, total);                    // every slice has a unit
      if (cta >= ctas) return;
      if (total < (1 << 22)) {                      // p.ctas < 512
        begin = (int)((unsigned)(cta * total) / (unsigned)ctas);
        end = (int)((unsigned)((cta + 1) * total) / (unsigned)ctas);
      } else {
        begin = (int)((long long)cta * total / ctas);
        end = (int)((long long)(cta + 1) * total / ctas);
      }
    };
    // a row without a visible token: zeros (a length past the table: NaN), by
    // threads `first`, `first` + `step`, ..
    auto clear = [&](int row, int first, int step) {
      const bool bad = __ldg(p.seqlens + row) > 0;
      if (bad && first == 0) raise_status(p.status, DSA_ERR_BAD_SEQLEN);
      if (first == 0) record_split(p, row, false, 0);
      const uint32_t v = bad ? 0x7fff7fffu : 0u;
#pragma unroll 1
      for (int j = first; j < heads * (kLatent / 8); j += step)
        *reinterpret_cast<uint4*>(p.out + row * p.out_row + (long long)(head0 + j / (kLatent / 8)) * p.out_head +
                                  (j % (kLatent / 8)) * 8) = make_uint4(v, v, v, v);
      for (int h = first; p.lse && h < heads; h += step)
        p.lse[(long long)row * p.H + head0 + h] = bad ? CUDART_NAN_F : -CUDART_INF_F;
    };
    if (p.rows <= kFewRows) {
      // few rows: every warp scans them for itself
      int len;
      const int entries = lane < p.rows ? row_entries(p, lane, &len) : 0;
      // (the bound keeps the sum from wrapping)
      const uint32_t halves = __reduce_add_sync(0xffffffffu, (uint32_t)min(units_of(entries, kTileShift - 1), 1 << 20));
      if (halves <= (uint32_t)p.ctas) walk.shift = kTileShift - 1;
      const int mine = units_of(entries, walk.shift);
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      total = __shfl_sync(0xffffffffu, incl, 31);
      take();
      const uint32_t here = __ballot_sync(0xffffffffu, end > begin && incl - mine <= begin && begin < incl);
      start_row = here ? __ffs(here) - 1 : 0;
      start_unit = begin - __shfl_sync(0xffffffffu, incl - mine, start_row);
      uint32_t empty = __ballot_sync(0xffffffffu, lane < p.rows && mine == 0 && lane % p.ctas == cta);
      for (; empty; empty &= empty - 1) clear(__ffs(empty) - 1, tid, kAttnThreads);
      if (tid == 0) m->start_row = start_row, m->start_unit = start_unit;
    } else {
      // thread i owns a run of rows; an exclusive scan of the runs' unit counts
      // finds the row in which this CTA's slice begins
      const int per = (p.rows + kAttnThreads - 1) / kAttnThreads;
      const int r0 = min(p.rows, tid * per), r1 = min(p.rows, r0 + per);
      int mine = 0;
      bool zero = false;
      for (int r = r0; r < r1; ++r) {
        const int t = row_units(p, r);
        mine += t;
        zero |= t == 0 && r % p.ctas == cta;
      }
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) m->scan[warp] = incl;
      const bool zeros = __syncthreads_or(zero);
      // the warps' totals: one per lane, scanned once more
      int sums = lane < kAttnThreads / 32 ? m->scan[lane] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sums, o);
        if (lane >= o) sums += v;
      }
      total = __shfl_sync(0xffffffffu, sums, 31);
      const int base = __shfl_sync(0xffffffffu, sums, warp > 0 ? warp - 1 : 0);
      take();
      int at = (warp > 0 ? base : 0) + incl - mine;
      if (end > begin && at <= begin && begin < at + mine) {
        int r = r0;
        for (;; ++r) {
          const int t = row_units(p, r);
          if (begin < at + t) break;
          at += t;
        }
        m->start_row = r;
        m->start_unit = begin - at;
      }
      if (zeros) {
        // the list of empty rows lies where the tile will
        int* list = reinterpret_cast<int*>(smem);
        for (int i = 0; i < per; ++i) {
          if (r0 + i < r1 && (r0 + i) % p.ctas == cta && row_units(p, r0 + i) == 0)
            list[atomicAdd(&m->nzero, 1)] = r0 + i;
          __syncthreads();
          const int n = m->nzero;
          __syncthreads();
          if (tid == 0) m->nzero = 0;
          for (int z = 0; z < n; ++z) clear(list[z], tid, kAttnThreads);
          __syncthreads();
        }
      }
    }
    if (tid == 0) {
      m->begin = begin, m->end = end, m->total = total, m->ctas = ctas, m->shift = walk.shift;
      if (!records_by_row(p))
        reinterpret_cast<int4*>(p.ws + (long long)gridDim.x * 2 * kPartialFloats)[blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
    __syncthreads();
    walk.start(p, m->start_row, m->start_unit, end - begin);
  }
  tc_fence_after();
  const uint32_t tmem = m->tmem;
  Waiter<true> wait{p.status, true};

  if (warp >= kLoadWarp0) {
    // ---- loaders -------------------------------------------------------------
    more_registers<kRegsLoad>();
    // warp w brings tokens 16w .. 16w+15 of every tile
    const int w = warp - kLoadWarp0;
    const int sub = lane >> 3, col = lane & 7;     // rotated part and fp8: 4 tokens x 8 lanes
    auto token_at = [&](int slot, int j) { return m->token[slot][w * kKeysPerWarp + j]; };
    auto page_of = [&](int t) { return p.cache + (long long)(t >> 6) * p.page_stride; };

    // fp8: four lanes take 64 codes of a token (one block of a part), the four
    // next to them the other block of the token's neighbour: even and odd rows
    // swizzle apart, so that the eight meet in no bank.  Step i: tokens 2p, 2p+1
    // with p = sub + 4 (i / 2), changed over for odd i.  The codes of a tile's
    // first two parts are in registers when the buffer falls free; the other
    // two parts' follow into their place.
    constexpr int kSteps = kKeysPerWarp / 4;
    const int other = col >> 2;
    auto step_token = [&](int i) { return 2 * (sub + 4 * (i >> 1)) + (other ^ (i & 1)); };
    const uint64_t once = evict_first();
    uint4 codes[2][kSteps];
    const uint8_t* row[kSteps];
    int rope_tok[kSteps];                          // rotated parts: tokens 4i + sub
    int4 tile = make_int4(0, 0, kEnd, 0);          // as the lookup warps found it
    auto fetch = [&](int it) {
      const int slot = it % kRing;
      wait(&m->look_full[slot], (it / kRing) & 1);
      tile = m->tile[slot];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int t = wait.ok ? token_at(slot, step_token(i)) : -1;
        row[i] = (t >= 0 ? page_of(t) + (t & 63) * kLatent : reinterpret_cast<const uint8_t*>(g_zeros)) + col * 16;
        codes[0][i] = ld_stream(row[i]);
        codes[1][i] = ld_stream(row[i] + 128);
        rope_tok[i] = wait.ok ? token_at(slot, 4 * i + sub) : -1;
      }
    };
    bool more = m->end > m->begin;
    if (kFp8 && more) fetch(0);

    // a wait that ran out ends the loop
    for (int it = 0; more && wait.ok; ++it) {
#ifdef DSA_TEST_SKIP_FIRST_TILE
      // test builds only: never deliver the first tile, so that the waits for
      // it run out
      const bool deliver = it != 0;
#else
      constexpr bool deliver = true;
#endif
      const int slot = it % kRing;
      if (!kFp8) {
        wait(&m->look_full[slot], (it / kRing) & 1);
        tile = m->tile[slot];
      }
      // no product reads further than the tokens' last 16 rows
      const bool mine_used = (w * kKeysPerWarp & ~15) < tile.y;
      more = !(tile.z & kEnd);
      const uint32_t prev = (it - 1) & 1;
      if (tile.z & kFirst) {
        // the row's queries; their place is free once the last scores are done
        if (it > 0) wait(&m->sfull, prev);
        // the first row's are the softmax warps' to bring: they have nothing
        // else to do then
        if (it > 0 && wait.ok)
          load_queries<KV, 2>(p, tile.x, head0, heads, w * kHeadsPerWarp, kHeadsPerWarp, sbase, lane,
                              m->mul[tile.w & 1]);
      }
      if (!kFp8) {
        // every address before the first part falls free
        const uint8_t* src[kKeysPerWarp / 2];
        const uint8_t* rsrc[kSteps];
        uint32_t valid = 0, rvalid = 0;
#pragma unroll
        for (int i = 0; i < kKeysPerWarp / 2; ++i) {
          const int t = wait.ok ? token_at(slot, 2 * i + (lane >> 4)) : -1;
          valid |= (t >= 0 ? 1u : 0u) << i;
          src[i] = page_of(max(t, 0)) + (max(t, 0) & 63) * kTokenBytesBf16 + (lane & 15) * 16;
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const int t = wait.ok ? token_at(slot, 4 * i + sub) : -1;
          rvalid |= (t >= 0 ? 1u : 0u) << i;
          rsrc[i] = page_of(max(t, 0)) + (max(t, 0) & 63) * kTokenBytesBf16 + kLatent * 2 + col * 16;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&m->look_empty[slot]);
        const uint32_t dst = sbase + ((lane >> 3) & 1) * kBlockBytes + (w * kKeysPerWarp + (lane >> 4)) * 128;
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          if (it > 0) wait(&m->empty[part], prev);
          if (wait.ok && mine_used) {
#pragma unroll
            for (int i = 0; i < kKeysPerWarp / 2; ++i)
              cp_async16_once(dst + part * kPartBytes + i * 256 + ((col ^ ((2 * i + (lane >> 4)) & 7)) << 4),
                              src[i] + part * 256, (valid >> i) & 1 ? 16u : 0u, once);
          }
          cp_async_commit();
        }
        if (wait.ok && mine_used) {
#pragma unroll
          for (int i = 0; i < kSteps; ++i)
            cp_async16_once(sbase + kOffP + (w * kKeysPerWarp + 4 * i + sub) * 128 + ((col ^ ((4 * i + sub) & 7)) << 4),
                            rsrc[i], (rvalid >> i) & 1 ? 16u : 0u, once);
        }
        cp_async_commit();
        cp_async_wait<4>();
        if (wait.ok && deliver) warp_arrive(&m->full[0], lane);
        cp_async_wait<3>();
        if (wait.ok && deliver) warp_arrive(&m->full[1], lane);
        cp_async_wait<2>();
        if (wait.ok && deliver) warp_arrive(&m->full[2], lane);
        cp_async_wait<1>();
        if (wait.ok && deliver) warp_arrive(&m->full[3], lane);
        cp_async_wait<0>();
        if (wait.ok && deliver) warp_arrive(&m->full[kParts], lane);
      } else {
        uint2 ratio[kSteps];
        uint32_t dst[kSteps];
        wait(&m->scale_full[slot], (it / kRing) & 1);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const int r = w * kKeysPerWarp + step_token(i);
          ratio[i] = m->ratio[slot][r];
          dst[i] = sbase + other * kBlockBytes + r * 128 + (((2 * (col & 3)) ^ (r & 7)) << 4);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&m->look_empty[slot]);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int odd = 0; odd < 2; ++odd) {
            const int part = 2 * half + odd;
            if (it > 0) wait(&m->empty[part], prev);
            if (wait.ok && mine_used) {
#pragma unroll
              for (int i = 0; i < kSteps; ++i) {
                const uint32_t two = half ? ratio[i].y : ratio[i].x;
                const uint32_t f = __byte_perm(two, two, odd ? 0x3232 : 0x1010);
                st_shared_v4(dst[i] + part * kPartBytes, widen8(codes[odd][i].x, codes[odd][i].y, f));
                st_shared_v4((dst[i] ^ 16) + part * kPartBytes, widen8(codes[odd][i].z, codes[odd][i].w, f));
              }
            }
            if (half == 0) {
#pragma unroll
              for (int i = 0; i < kSteps; ++i) codes[odd][i] = ld_stream(row[i] + (odd + 2) * 128);
            }
            if (wait.ok && deliver) warp_arrive(&m->full[part], lane);
          }
        }
        if (wait.ok && mine_used) {
#pragma unroll
          for (int i = 0; i < kSteps; ++i) {
            const int t = max(rope_tok[i], 0);
            cp_async16(sbase + kOffP + (w * kKeysPerWarp + 4 * i + sub) * 128 + ((col ^ ((4 * i + sub) & 7)) << 4),
                       page_of(t) + kRopeOffsetFp8 + (t & 63) * (kRope * 2) + col * 16, rope_tok[i] < 0 ? 0u : 16u);
          }
        }
        cp_async_wait_all();
        if (wait.ok && deliver) warp_arrive(&m->full[kParts], lane);
        if (more) fetch(it + 1);
      }
    }
    cp_async_wait_all();
  } else if (warp >= kMmaWarp) {
    // warps 8-11 are one warpgroup, and all of a warpgroup have to run the same
    // setmaxnreg: before its roles part
    fewer_registers<kRegsMisc>();
    if (warp >= kLookWarp0) {
      // ---- token lookup ----------------------------------------------------------
      // tile i by warp i % 3: list and block table to token, and L2 asked for it
      const int slot = warp - kLookWarp0;
      for (int it = 0; walk.left > 0; ++it) {
        if (it % kLookWarps == slot) {
          const int n = walk.tokens();
          const int flags = (walk.first ? kFirst : 0) | (walk.last() ? kLast : 0) | (walk.left == 1 ? kEnd : 0);
          int tok[4];
          bool bad = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = i * 32 + lane;
            tok[i] = -1;                             // first the position
            if (j < n) {
              const int e = (walk.u << walk.shift) + j;
              tok[i] = p.idx ? __ldg(p.idx + walk.row * p.idx_stride + e) : e;
            }
            if (tok[i] >= walk.len) tok[i] = -1;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (tok[i] < 0) {
              tok[i] = -1;
              continue;
            }
            const int page = __ldg(p.block_table + walk.row * p.bt_stride + tok[i] / kPage);
            const bool in = page >= 0 && page < p.num_pages;
            tok[i] = in ? page * kPage + tok[i] % kPage : -1;
            bad |= !in;
          }
          if (it >= kRing) wait(&m->look_empty[slot], (it / kRing - 1) & 1);
          const bool any_bad = __any_sync(0xffffffffu, bad);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t v = __ballot_sync(0xffffffffu, tok[i] >= 0);
            if (wait.ok) {
              m->token[slot][i * 32 + lane] = tok[i];
              if (lane == 0) m->mask[slot][i] = v;
            }
          }
          if (wait.ok && lane == 0) {
            m->tile[slot] = make_int4(walk.row, n, flags | (any_bad ? kBad : 0), walk.piece);
            if (walk.first) {
              const bool begins = walk.u == 0, whole = begins && walk.left >= walk.units();
              m->piece[walk.piece & 7] = make_int4(walk.row, (begins ? kBegins : 0) | (whole ? kWhole : 0), 0, 0);
              if (begins) {
                // where the row ends, should it go on in later CTAs
                const long long last_unit = (long long)m->end - walk.left + walk.units() - 1;
                record_split(p, walk.row, !whole, whole ? 0 : (int)(((last_unit + 1) * m->ctas - 1) / m->total));
              }
            }
          }
          if (any_bad && lane == 0) raise_status(p.status, DSA_ERR_BAD_PAGE);
          __syncwarp();
          if (wait.ok && lane == 0) mbar_arrive(&m->look_full[slot]);
          if (kFp8) {
            float4 sc[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int t = max(tok[i], 0);
              sc[i] = __ldg(reinterpret_cast<const float4*>(p.cache + (long long)(t >> 6) * p.page_stride +
                                                            kScaleOffsetFp8) + (t & 63));
            }
            // A group of scale 1 holds zeros (latent_store gives those 1) or values
            // up to 448.  Where 1 is a token's largest, zeros must not count, or
            // they would push groups of far smaller scales out of fp16.  (Where
            // every scale is 1 the look at the codes takes up to 10%: the prefill 533
            // us for 484.)
            float top[4];
            bool ones = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              top[i] = fmaxf(fmaxf(sc[i].x, sc[i].y), fmaxf(sc[i].z, sc[i].w));
              ones |= tok[i] >= 0 && top[i] == 1.f;
            }
            if (__any_sync(0xffffffffu, ones)) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int t = tok[i];
                if (t < 0 || top[i] != 1.f) continue;
                const uint32_t zeros = zero_groups(
                    p.cache + (long long)(t >> 6) * p.page_stride + (t & 63) * kLatent,
                    (sc[i].x == 1.f ? 1u : 0u) | (sc[i].y == 1.f ? 2u : 0u) | (sc[i].z == 1.f ? 4u : 0u) |
                        (sc[i].w == 1.f ? 8u : 0u));
                if (zeros & 1u) sc[i].x = 0.f;
                if (zeros & 2u) sc[i].y = 0.f;
                if (zeros & 4u) sc[i].z = 0.f;
                if (zeros & 8u) sc[i].w = 0.f;
                top[i] = fmaxf(fmaxf(sc[i].x, sc[i].y), fmaxf(sc[i].z, sc[i].w));
              }
              __syncwarp();
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 c = sc[i];
              const float low = fminf(fminf(c.x > 0.f ? c.x : top[i], c.y > 0.f ? c.y : top[i]),
                                      fminf(c.z > 0.f ? c.z : top[i], c.w > 0.f ? c.w : top[i]));
              const float most = fmaxf(fmaxf(kScaleBelowTop * top[i], kScaleAboveLow * low), kSmallestScale);
              const float inv = __frcp_rn(most);
              const __half2 a = __floats2half2_rn(sc[i].x * inv, sc[i].y * inv);
              const __half2 b = __floats2half2_rn(sc[i].z * inv, sc[i].w * inv);
              const bool in = tok[i] >= 0;           // a masked token: zeros times zero
              if (wait.ok) {
                m->ratio[slot][i * 32 + lane] = make_uint2(in ? *reinterpret_cast<const uint32_t*>(&a) : 0u,
                                                           in ? *reinterpret_cast<const uint32_t*>(&b) : 0u);
                m->key_scale[slot][i * 32 + lane] = in ? most : 1.f;
              }
            }
            __syncwarp();
            if (wait.ok && lane == 0) mbar_arrive(&m->scale_full[slot]);
          }
          if (it > 0) {
            // The first tile is loaded at once; the later ones wait for its place.
            // Asked for when the tile before has begun to arrive: earlier costs
            // 2 to 5% (the place in L2).  Late, or after a whole phase that was
            // missed, it would hold up the next tiles' lookup: the wait is short.
            for (int n = 0; n < 100 && !mbar_test_wait(&m->full[0], (it - 1) & 1); ++n) __nanosleep(40);
            if (p.idx == nullptr) {
              // whole pages: the first tokens of both
              const int t0 = __shfl_sync(0xffffffffu, tok[0], 0), t1 = __shfl_sync(0xffffffffu, tok[2], 0);
              const int t = lane == 0 ? t0 : lane == 1 ? t1 : -1;
              if (t >= 0)
                l2_prefetch_bulk(p.cache + (long long)(t >> 6) * p.page_stride,
                                 (uint32_t)(kFp8 ? kPageBytesFp8 : kPageBytesBf16));
            } else {
#pragma unroll 1
              for (int i = 0; i < 4; ++i) {
                const int t = i == 0 ? tok[0] : i == 1 ? tok[1] : i == 2 ? tok[2] : tok[3];
                if (t < 0) continue;
                const uint8_t* pg = p.cache + (long long)(t >> 6) * p.page_stride;
                const int s = t & 63;
                const uint8_t* row = pg + s * (kFp8 ? kLatent : kTokenBytesBf16);
                l2_prefetch_bulk(row, kFp8 ? kLatent : kTokenBytesBf16);
                if (kFp8) l2_prefetch(pg + kRopeOffsetFp8 + s * (kRope * 2));
              }
            }
            if (walk.first)
#pragma unroll 1
              for (int h = lane; h < heads; h += 32) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  l2_prefetch(p.ql + walk.row * p.ql_row + (head0 + h) * p.ql_head + j * 64);
                l2_prefetch(p.qr + walk.row * p.qr_row + (head0 + h) * p.qr_head);
              }
          }
        }
        walk.step(p);
      }
    } else {
      // ---- MMA issue -----------------------------------------------------------
      if (elect_one()) {
        Waiter<false> wait{p.status, true};
        if (walk.left > 0) wait(&m->qfirst, 0);
        for (int it = 0; walk.left > 0; ++it) {
          // eight MMAs to a step of these loops: all 68 in a row push the other
          // roles out of the instruction cache, four leave the tensor pipe idle
          uint64_t a_d = smem_desc_sw128(sbase, 1024), b_d = smem_desc_sw128(sbase + kOffQ, 1024);
#pragma unroll 1
          for (int part = 0; part < kParts; ++part) {
            wait(&m->full[part], it & 1);
            tc_fence_after();
            if (wait.ok)
#pragma unroll
              for (int k = 0; k < 8; ++k)
                mma_f16(tmem + kTmemS, a_d + (((k / 4) * kBlockBytes + (k % 4) * 32) >> 4),
                        b_d + (((k / 4) * kQBlockBytes + (k % 4) * 32) >> 4), idesc_s(KV), k > 0 || part > 0);
            a_d += kPartBytes >> 4;
            b_d += 2 * kQBlockBytes >> 4;
          }
          wait(&m->full[kParts], it & 1);
          tc_fence_after();
          if (wait.ok)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f16(tmem + (kFp8 ? kTmemR : kTmemS), a_d + (k * 32 >> 4), b_d + (k * 32 >> 4),
                      kFp8 ? kIdescRope : idesc_s(KV), !kFp8 || k > 0);
          if (wait.ok) mma_commit(&m->sfull);
          const int steps = (walk.tokens() + 15) / 16;
          const uint32_t keep = walk.first ? 0u : 1u;
          wait(&m->pfull, it & 1);
          if (walk.first && walk.piece > 0) wait(&m->ofree, (walk.piece - 1) & 1);
          tc_fence_after();
          if (wait.ok) {
            a_d = smem_desc_mn_sw128(sbase, kBlockBytes, 1024);
            b_d = smem_desc_mn_sw128(sbase + kOffP, kBlockBytes, 1024);
#pragma unroll 1
            for (int part = 0; part < kParts; ++part) {
#pragma unroll
              for (int k = 0; k < kTile / 16; ++k)
                if (k < steps)
                  mma_f16(tmem + part * kAttnHeads, a_d + (k * 2048 >> 4), b_d + (k * 2048 >> 4), idesc_o(KV),
                          k > 0 ? 1u : keep);
              mma_commit(&m->empty[part]);
              a_d += kPartBytes >> 4;
            }
          }
          walk.step(p);
        }
        if (!wait.ok) {
          // what was issued still runs: wait for it before TMEM is given back
          mma_commit(&m->done);
          mbar_wait_bounded(&m->done, 0, kWaitLimit);
        }
      }
      __syncwarp();
    }
  } else {
    // ---- softmax and output --------------------------------------------------
    more_registers<kRegsSoftmax>();
    // this thread: token 32 quarter + lane, heads 32 half .. 32 half + 31
    const int quarter = warp & 3, half = warp >> 2;
    const int hbase = half * 32, bar_half = 2 + half;
    const uint32_t my_tmem = tmem + ((uint32_t)(quarter * 32) << 16) + hbase;
    const int key = quarter * 32 + lane;
    F2 sum[16];
    // rows and parts come as the lookup warps found them: no walk of its own
    bool bad = false, fresh = true, more = m->end > m->begin;  // fresh: some head has no reference yet
    uint32_t piece = 0;
    if (more) {
      load_queries<KV, 4>(p, walk.row, head0, heads, warp * 8, 8, sbase, lane, m->mul[0]);
      cp_async_wait_all();
      warp_arrive(&m->qfirst, lane);
    }
    for (int it = 0; more; ++it) {
      const int slot = it % kRing;
      wait(&m->look_full[slot], (it / kRing) & 1);
      // a wait that ran out (here, or for the last tile) ends the loop, for the
      // four warps together: they meet at barriers
      if (bar_any(bar_half, 128, !wait.ok)) break;
      const bool valid = (*reinterpret_cast<volatile uint32_t*>(&m->mask[slot][quarter]) >> lane) & 1;
      const int flags = m->tile[slot].z;
      more = !(flags & kEnd);
      if (flags & kFirst) {
#pragma unroll
        for (int j = 0; j < 16; ++j) sum[j] = 0ull;
        bad = false;
        fresh = true;
      }
      bad |= (flags & kBad) != 0;
      if (kFp8) wait(&m->scale_full[slot], (it / kRing) & 1);
      const float key_scale = kFp8 ? m->key_scale[slot][key] : 1.f;
      __syncwarp();
      if (lane == 0) mbar_arrive(&m->look_empty[slot]);
      wait(&m->sfull, it & 1);
      __syncwarp();
      tc_fence_after();
      // weights in log2 units over the reference, e = score - reference
      float e[32];
      const float key_log = kFp8 ? __log2f(key_scale) : 0.f;
      const F2 ks2 = pair(key_scale, key_scale), sl2 = pair(p.scale_log2, p.scale_log2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t x[8], y[8];
        tmem_ld_32x32b_x8(my_tmem + kTmemS + 8 * i, x);
        if (kFp8) {
          tmem_ld_32x32b_x8(my_tmem + kTmemR + 8 * i, y);
          tmem_ld_wait8(x, y);
        } else {
          tmem_ld_wait8(x);
        }
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          const ulonglong2 n2 = *reinterpret_cast<const ulonglong2*>(&m->nref[hbase + 8 * i + j]);
          F2 u0 = pair(x[j], x[j + 1]), u1 = pair(x[j + 2], x[j + 3]);
          if (kFp8) {
            const ulonglong2 m2 = *reinterpret_cast<const ulonglong2*>(&m->mul[piece & 1][hbase + 8 * i + j]);
            u0 = fma2(fma2(u0, ks2, pair(y[j], y[j + 1])), m2.x, n2.x);
            u1 = fma2(fma2(u1, ks2, pair(y[j + 2], y[j + 3])), m2.y, n2.y);
          } else {
            u0 = fma2(u0, sl2, n2.x);
            u1 = fma2(u1, sl2, n2.y);
          }
          unpair(u0, e[8 * i + j], e[8 * i + j + 1]);
          unpair(u1, e[8 * i + j + 2], e[8 * i + j + 3]);
        }
      }
      if (!valid)
#pragma unroll
        for (int j = 0; j < 32; ++j) e[j] = -CUDART_INF_F;
      float most = e[0];
#pragma unroll
      for (int j = 1; j < 32; ++j) most = fmaxf(most, e[j]);
      if (bar_any(bar_half, 128, fresh || most + key_log > ref_limit(KV))) {
        // the tile's largest weight of each head, and the reference raised
        // where it has to be
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float v = warp_max(e[j] + key_log);
          top = lane == j ? v : top;
        }
        const int h = hbase + lane;
        m->red[quarter][h] = top;
        bar_sync(bar_half, 128);
        const float v = fmaxf(fmaxf(m->red[0][h], m->red[1][h]), fmaxf(m->red[2][h], m->red[3][h]));
        const float old = m->nref[h];
        const bool unset = __float_as_uint(old) == kUnset, seen = v > -CUDART_INF_F;
        fresh = __any_sync(0xffffffffu, unset && !seen);
        bar_sync(bar_half, 128);
        if (quarter == 0) {
          const float up = seen && (unset || v > ref_limit(KV)) ? v - ref_below(KV) : 0.f;
          if (seen) m->nref[h] = (unset ? 0.f : old) - up;
          m->fac[h] = up;
          m->keep[h] = unset ? 1.f : ex2(-up);            // sums of an unset head are zero
        }
        bar_sync(bar_half, 128);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 f = *reinterpret_cast<const float4*>(&m->fac[hbase + j]);
          e[j] -= f.x, e[j + 1] -= f.y, e[j + 2] -= f.z, e[j + 3] -= f.w;
        }
        if (!(flags & kFirst)) {
          // the scores' commit covers the last value product: O^T is at rest
#pragma unroll
          for (int j = 0; j < 16; ++j)
            sum[j] = mul2(sum[j], *reinterpret_cast<const F2*>(&m->keep[hbase + 2 * j]));
#pragma unroll 1
          for (int i = 0; i < 4 * kParts; ++i) {
            uint32_t o[8];
            const int c = (i & 3) * 8;
            if (__all_sync(0xffffffffu, m->keep[hbase + c + (lane & 7)] == 1.f)) continue;
            const uint32_t at = my_tmem + (i >> 2) * kAttnHeads + c;
            tmem_ld_32x32b_x8(at, o);
            tmem_ld_wait8(o);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * m->keep[hbase + c + j]);
            tmem_st_32x32b_x8(at, o);
          }
          tmem_st_wait();
        }
      }
#pragma unroll
      for (int j8 = 0; j8 < 32; j8 += 8) {
        uint32_t w[4];
#pragma unroll
        for (int u = 0; u < 8; u += 2) {
          float a = ex2(e[j8 + u]), b = ex2(e[j8 + u + 1]);
          const F2 ab = pair(a, b);
          sum[(j8 + u) / 2] = add2(sum[(j8 + u) / 2], ab);
          if (kFp8) {
            unpair(mul2(ab, ks2), a, b);
            const __half2 v = __floats2half2_rn(a, b);
            w[u / 2] = *reinterpret_cast<const uint32_t*>(&v);
          } else {
            const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
            w[u / 2] = *reinterpret_cast<const uint32_t*>(&v);
          }
        }
        st_shared_v4(sbase + kOffP + key * 128 + (((hbase + j8) / 8 ^ (key & 7)) << 4),
                     make_uint4(w[0], w[1], w[2], w[3]));
      }
      tc_fence_before();
      if (wait.ok) warp_arrive(&m->pfull, lane);

      if (flags & kLast) {
        // ---- the piece's result ------------------------------------------------
        bar_sync(bar_half, 128);                          // every use of red and fac is over
        m->red[quarter][hbase + lane] = sum_columns(sum, lane);
        wait(&m->empty[kParts - 1], it & 1);              // the last value product
        bad = bar_any(bar_half, 128, bad || !wait.ok);
        const int4 what = m->piece[piece & 7];
        const bool begins = what.y & kBegins, whole = what.y & kWhole;
        float* part_at = p.ws + ((long long)blockIdx.x * 2 + (begins ? 1 : 0)) * kPartialFloats;
        if (quarter == 0) {
          const int h = hbase + lane;
          float total_h = m->red[0][h] + m->red[1][h] + m->red[2][h] + m->red[3][h];
          const float nref = m->nref[h];
          const float max_h = bad ? 0.f : __float_as_uint(nref) == kUnset ? -CUDART_INF_F : -nref;
          if (bad) total_h = CUDART_NAN_F;
          if (whole) {
            m->fac[h] = total_h == 0.f ? 0.f : 1.f / total_h;
            if (p.lse && h < heads)
              p.lse[(long long)what.x * p.H + head0 + h] = (max_h + log2f(total_h)) * 0.69314718055994531f;
          } else {
            part_at[kAttnHeads * kLatent + h] = max_h;
            part_at[kAttnHeads * kLatent + kAttnHeads + h] = total_h;
          }
          m->nref[h] = __uint_as_float(kUnset);
        }
        bar_sync(bar_half, 128);
        tc_fence_after();
        // sixteen heads of a part at a time.  A warp's instructions come one in
        // about eight cycles here, so the loop is short rather than wide: bf16
        // pairs change lanes as one word, and pointers only move on
        const int odd = lane & 1, mine = heads - hbase;   // this half's heads
        uint16_t* row = p.out + what.x * p.out_row + (long long)(head0 + hbase + odd) * p.out_head + (key & ~1);
        const uint32_t pick = odd ? 0x3276 : 0x5410;
#pragma unroll 1
        for (int part = 0; part < kParts; ++part) {
          uint16_t* dst = row + part * 128;
          float* sum_at = part_at + hbase * kLatent + part * 128 + key;
#pragma unroll 1
          for (int h0 = 0; h0 < min(32, mine); h0 += 16) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(my_tmem + part * kAttnHeads + h0, o);
            tmem_ld_wait(o);
            if (whole) {
              // two heads of a lane pair: each lane writes two values of one head
#pragma unroll
              for (int j = 0; j < 16; j += 2) {
                const float2 f = *reinterpret_cast<const float2*>(&m->fac[hbase + h0 + j]);
                const __nv_bfloat162 two =
                    __floats2bfloat162_rn(__uint_as_float(o[j]) * f.x, __uint_as_float(o[j + 1]) * f.y);
                const uint32_t a = *reinterpret_cast<const uint32_t*>(&two);
                const uint32_t c = __byte_perm(a, __shfl_xor_sync(0xffffffffu, a, 1), pick);
                if (h0 + j + odd < mine) *reinterpret_cast<uint32_t*>(dst) = c;
                dst += 2 * p.out_head;
              }
            } else {
              // a part that went wrong has a total that is NaN: that is enough
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (h0 + j < mine) sum_at[j * kLatent] = __uint_as_float(o[j]);
              sum_at += 16 * kLatent;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (wait.ok && lane == 0) mbar_arrive(&m->ofree);
        bar_sync(bar_half, 128);                          // fac and red are free again
        ++piece;
      }
    }
    if (more) {
      // a wait ran out: the rows and parts from this one on are NaN
      walk.shift = m->shift;
      walk.start(p, m->start_row, m->start_unit, m->end - m->begin);
      for (uint32_t i = 0; walk.left > 0; walk.step(p)) {
        if (!walk.first) continue;
        if (i++ < piece) continue;
        const bool begins = walk.u == 0, whole = begins && walk.left >= walk.units();
        float* part_at = p.ws + ((long long)blockIdx.x * 2 + (begins ? 1 : 0)) * kPartialFloats;
        for (int h = hbase; h < min(heads, hbase + 32); ++h) {
          for (int d = key; whole && d < kLatent; d += 128)
            p.out[walk.row * p.out_row + (long long)(head0 + h) * p.out_head + d] = 0x7fff;
          if (key != 0) continue;
          if (whole && p.lse) p.lse[(long long)walk.row * p.H + head0 + h] = CUDART_NAN_F;
          if (!whole) {
            part_at[kAttnHeads * kLatent + h] = 0.f;
            part_at[kAttnHeads * kLatent + kAttnHeads + h] = CUDART_NAN_F;
          }
        }
        if (begins && tid == 0) {
          const long long last_unit = (long long)m->end - walk.left + walk.units() - 1;
          record_split(p, walk.row, !whole, whole ? 0 : (int)(((last_unit + 1) * m->ctas - 1) / m->total));
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// Joins the partial sums of the rows that slices cut, a block (record, heads).
// A thread has four values of a head; the pieces are read four at a time,
// their loads together.  WIDE (few rows, so each may have
// many pieces): a block has one head, and its four groups of 128 threads a
// quarter of the pieces each.  Otherwise it has four heads.
constexpr int kJoinThreads = 512;
template <bool WIDE>
__global__ void __launch_bounds__(kJoinThreads, WIDE ? 2 : 3) latent_join_kernel(const LatentAttnParams p,
                                                                                     int main_ctas) {
  __shared__ float4 sums[4][128];
  __shared__ float2 stats[4][128];
  griddep_wait();
  griddep_launch_dependents();
  const int grp = blockIdx.x % p.groups;
  const int4 rec = reinterpret_cast<const int4*>(p.ws + (long long)main_ctas * 2 * kPartialFloats)[blockIdx.x];
  const int row = rec.x, n = rec.y - rec.z;      // n pieces after the first
  if (row == -1) return;
  if (!split_record_ok(row, rec.y, rec.z, p.rows, p.ctas)) {  // another call wrote to this workspace
    if (threadIdx.x == 0) raise_status(p.status, DSA_ERR_INVALID_ARG);
    return;
  }
  const int part = threadIdx.x / 128, d = (threadIdx.x % 128) * 4;
  const int h = WIDE ? blockIdx.y : blockIdx.y * 4 + part;
  const int head = grp * kAttnHeads + h;
  if (head >= p.H) return;                       // WIDE: the whole block
  const long long step = (long long)p.groups * 2 * kPartialFloats;
  // the first piece lies in slot 1 of its CTA, the later ones in slot 0 of theirs
  const float* rest = p.ws + ((long long)rec.z * p.groups + grp) * 2 * kPartialFloats + step;
  const float* first = rest - step + kPartialFloats;
  float top = -CUDART_INF_F, total = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int i0 = -1 + (WIDE ? part : 0); i0 < n; i0 += WIDE ? 16 : 4) {
    float mx[4], sm[4];
    float4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * (WIDE ? 4 : 1);
      mx[u] = -CUDART_INF_F, sm[u] = 0.f, v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        const float* s = i < 0 ? first : rest + i * step;
        mx[u] = s[kAttnHeads * kLatent + h];
        sm[u] = s[kAttnHeads * kLatent + kAttnHeads + h];
        v[u] = *reinterpret_cast<const float4*>(s + h * kLatent + d);
      }
    }
    float now = top;
#pragma unroll
    for (int u = 0; u < 4; ++u) now = fmaxf(now, mx[u]);
    const float ref = now == -CUDART_INF_F ? 0.f : now;
    float wgt = ex2(top - ref);
    total *= wgt;
    acc.x *= wgt, acc.y *= wgt, acc.z *= wgt, acc.w *= wgt;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      wgt = ex2(mx[u] - ref);
      total = fmaf(sm[u], wgt, total);
      acc.x = fmaf(v[u].x, wgt, acc.x);
      acc.y = fmaf(v[u].y, wgt, acc.y);
      acc.z = fmaf(v[u].z, wgt, acc.z);
      acc.w = fmaf(v[u].w, wgt, acc.w);
    }
    top = now;
  }
  if (WIDE) {
    sums[part][threadIdx.x % 128] = acc;
    stats[part][threadIdx.x % 128] = make_float2(top, total);
    __syncthreads();
    if (part > 0) return;
    float now = top;
#pragma unroll
    for (int u = 1; u < 4; ++u) now = fmaxf(now, stats[u][threadIdx.x].x);
    const float ref = now == -CUDART_INF_F ? 0.f : now;
    float wgt = ex2(top - ref);
    total *= wgt;
    acc.x *= wgt, acc.y *= wgt, acc.z *= wgt, acc.w *= wgt;
#pragma unroll
    for (int u = 1; u < 4; ++u) {
      const float2 st = stats[u][threadIdx.x];
      const float4 v = sums[u][threadIdx.x];
      wgt = ex2(st.x - ref);
      total = fmaf(st.y, wgt, total);
      acc.x = fmaf(v.x, wgt, acc.x);
      acc.y = fmaf(v.y, wgt, acc.y);
      acc.z = fmaf(v.z, wgt, acc.z);
      acc.w = fmaf(v.w, wgt, acc.w);
    }
    top = now;
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
  const int records = p.rows < p.ctas ? p.rows : p.ctas, heads = p.H < kAttnHeads ? p.H : kAttnHeads;
  // The wide join, a block per head, while that is no more than five blocks an
  // SM.  fp8 calls of 64 heads over 2,048 tokens, wide and not: 2 rows 15.1 and
  // 22.8 us, 8 rows 17.6 and 20.4, 16 rows (1,024 blocks) 25.1 and 24.1, 48
  // rows 50.2 and 40.9; one row of 131,072 bf16 tokens and 128 heads 58 and 77.
  const bool wide = (long long)records * p.groups * heads <= 5LL * sms;
  cudaLaunchConfig_t join = cfg;
  join.gridDim = dim3(records * p.groups, wide ? heads : (heads + 3) / 4);
  join.blockDim = dim3(kJoinThreads);
  join.dynamicSmemBytes = 0;
  const int main_ctas = p.ctas * p.groups;
  return wide ? cudaLaunchKernelEx(&join, latent_join_kernel<true>, p, main_ctas)
              : cudaLaunchKernelEx(&join, latent_join_kernel<false>, p, main_ctas);
}

}  // namespace

cudaError_t launch_latent_attention(const LatentAttnParams& p, int kv_dtype, int sms, cudaStream_t stream) {
  if (kv_dtype == DSA_KV_BF16) return launch_t<DSA_KV_BF16>(p, sms, stream);
  return launch_t<DSA_KV_FP8_E4M3>(p, sms, stream);
}

}  // namespace dsa
