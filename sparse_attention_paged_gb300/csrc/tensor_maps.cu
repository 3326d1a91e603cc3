// tensor_maps.cu -- TMA tensor-map encoding for the key pool and the queries.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <string.h>

#include <mutex>

#include "tensor_maps.cuh"

namespace dsa {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (fn == nullptr) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                         cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }
  return fn;
}

// A small cache of encoded maps: a serving loop calls with the same pool
// and query buffers every step, and encoding is pure host work.  Keyed by
// everything the encoding reads; direct-mapped, guarded by a mutex.
struct MapKey {
  const void* base;
  unsigned long long dims[4], strides[3];
  unsigned box[4];
  int rank, swizzle;
  bool operator==(const MapKey& o) const { return memcmp(this, &o, sizeof o) == 0; }
};

struct MapCacheEntry {
  bool used;
  MapKey key;
  CUtensorMap map;
};

constexpr int kMapCacheSize = 32;
MapCacheEntry g_cache[kMapCacheSize];
std::mutex g_cache_mutex;

int cache_slot(const MapKey& k) {
  unsigned long long h = reinterpret_cast<unsigned long long>(k.base) >> 4;
  h ^= k.dims[0] * 0x9E3779B97F4A7C15ull ^ k.dims[1] * 0xC2B2AE3D27D4EB4Full ^ k.dims[2] ^
       k.strides[1] * 0x165667B19E3779F9ull ^ k.box[1];
  return (int)(h % kMapCacheSize);
}

// Encode (or fetch) a 4-byte-unit tiled map, 128-byte swizzle unless given.
bool encode_cached(CUtensorMap* m, int rank, const void* base, const cuuint64_t* dims,
                   const cuuint64_t* strides, const cuuint32_t* box,
                   CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  MapKey k;
  memset(&k, 0, sizeof k);
  k.base = base;
  k.rank = rank;
  k.swizzle = (int)swizzle;
  for (int i = 0; i < rank; ++i) {
    k.dims[i] = dims[i];
    k.box[i] = box[i];
  }
  for (int i = 0; i < rank - 1; ++i) k.strides[i] = strides[i];
  const int slot = cache_slot(k);
  {
    std::lock_guard<std::mutex> g(g_cache_mutex);
    if (g_cache[slot].used && g_cache[slot].key == k) {
      *m = g_cache[slot].map;
      return true;
    }
  }
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, rank, const_cast<void*>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return false;
  std::lock_guard<std::mutex> g(g_cache_mutex);
  g_cache[slot].used = true;
  g_cache[slot].key = k;
  g_cache[slot].map = *m;
  return true;
}

}  // namespace

// TMA moves a bounded number of elements per clock, so every map describes
// the data in 4-byte units (the bytes and the 128-byte-swizzled shared-memory
// image are the same as with the native element type): a 128-byte row of
// either dtype is 32 units.

// Key pool: dims {row bytes / 4, 64 slots, num_pages}, box = one page's
// 128-byte column block (fp8: the whole row; bf16: half a row, the second
// half at unit coordinate kHalfRowUnits).
bool encode_kcache_map(CUtensorMap* m, const RowsParams& p) {
  const bool bf16 = p.kv_dtype == DSA_KV_BF16;
  const cuuint64_t row_bytes = (cuuint64_t)kDim * (bf16 ? 2 : 1);
  cuuint64_t dims[3] = {row_bytes / 4, (cuuint64_t)kPage, (cuuint64_t)p.num_pages};
  cuuint64_t strides[2] = {row_bytes, (cuuint64_t)p.page_stride};
#ifndef DSA_FP8_BOX_ROWS
#define DSA_FP8_BOX_ROWS 64
#endif
  const cuuint32_t rows = bf16 ? (cuuint32_t)kPage : (cuuint32_t)DSA_FP8_BOX_ROWS;
  cuuint32_t box[3] = {32u, rows, 1u};
  return encode_cached(m, 3, p.kcache, dims, strides, box);
}

// Queries viewed as [rows * 64, 64 units] (a bf16 row of 128 values is 256
// bytes = 64 units), box {32 units, box_rows}; the second half-row at unit
// coordinate kHalfRowUnits.
bool encode_q_map(CUtensorMap* m, const RowsParams& p, int box_rows) {
  cuuint64_t dims[2] = {(cuuint64_t)kDim * 2 / 4, (cuuint64_t)p.rows * kHeads};
  cuuint64_t strides[1] = {(cuuint64_t)kDim * 2};
  cuuint32_t box[2] = {32u, (cuuint32_t)box_rows};
  return encode_cached(m, 2, p.q, dims, strides, box);
}

// Pool of a key/value cache: dims {row bytes / 4, 64 slots, heads, pages}
// through its strides, box = one head's 64 slots, 128 bytes of each (64 where
// a row has no more, in the 64-byte swizzle).
bool encode_kv_pool_map(CUtensorMap* m, const void* base, int row_bytes, long long slot_bytes,
                        long long head_bytes, long long page_bytes, int heads, int num_pages) {
  const int box_bytes = row_bytes < 128 ? row_bytes : 128;
  cuuint64_t dims[4] = {(cuuint64_t)row_bytes / 4, (cuuint64_t)kPage, (cuuint64_t)heads,
                        (cuuint64_t)num_pages};
  cuuint64_t strides[3] = {(cuuint64_t)slot_bytes, (cuuint64_t)head_bytes, (cuuint64_t)page_bytes};
  cuuint32_t box[4] = {(cuuint32_t)box_bytes / 4, (cuuint32_t)kPage, 1u, 1u};
  return encode_cached(m, 4, base, dims, strides, box,
                       box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

}  // namespace dsa
