// paged_api.cu -- the C ABI of the paged cache of keys and values
// (include/dsa_indexer.h): argument checks, parameter packing and launches.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dsa_indexer.h"
#include "paged_common.cuh"
#include "tensor_maps.cuh"

namespace dsa {
cudaError_t launch_request_slots(const RequestSlotsParams& p, cudaStream_t stream);
cudaError_t launch_kv_store(const KvStoreParams& p, int kv_dtype, cudaStream_t stream);
cudaError_t launch_block_bounds(const BlockBoundsParams& p, int kv_dtype, int sms, cudaStream_t stream);
cudaError_t launch_block_select(const BlockSelectParams& p, int sms, cudaStream_t stream);
cudaError_t launch_paged_attention(const PagedAttnParams& p, int dim, int kv_dtype, const CUtensorMap& kmap,
                                   const CUtensorMap& vmap, int sms, cudaStream_t stream);
}  // namespace dsa

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int launched(cudaError_t e) { return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA; }

// The current device's SM count, asked for once per device; 0 on failure.
int sm_count() {
  static int known[dsa::kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < dsa::kMaxDevices && known[dev] > 0) return known[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < dsa::kMaxDevices) known[dev] = n;
  return n;
}

constexpr long long k2G = 1LL << 31;

bool is16(int dtype) { return dtype == DSA_BF16 || dtype == DSA_FP16; }

// The cache's type beside that of the values that go in or come out.
int check_types(int dtype, int kv_dtype) {
  if (!is16(dtype)) return DSA_ERR_INVALID_ARG;
  if (kv_dtype == DSA_KV_FP8_E4M3) return DSA_OK;
  if (kv_dtype != DSA_KV_BF16 && kv_dtype != DSA_KV_FP16) return DSA_ERR_INVALID_ARG;
  return (kv_dtype == DSA_KV_FP16) == (dtype == DSA_FP16) ? DSA_OK : DSA_ERR_UNSUPPORTED;
}

int check_heads(int heads, int D, int page_size) {
  if (heads <= 0) return DSA_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || page_size != dsa::kPage) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

// A pool's address and strides (elements); everything on 16 bytes.
int check_pool(const void* pool, const dsa::PoolLayout& at, const float* scale, int heads, int D, int num_pages,
               int kv_dtype) {
  const bool fp8 = kv_dtype == DSA_KV_FP8_E4M3;
  if (!pool || num_pages <= 0 || (fp8 && !scale)) return DSA_ERR_INVALID_ARG;
  if (at.slot < D || (heads > 1 && at.head < D) || (num_pages > 1 && at.page < D)) return DSA_ERR_INVALID_ARG;
  if ((long long)num_pages * dsa::kPage >= k2G) return DSA_ERR_UNSUPPORTED;
  const long long unit = fp8 ? 16 : 8;
  if (!aligned(pool, 16) || at.slot % unit || (heads > 1 && at.head % unit) || (num_pages > 1 && at.page % unit) ||
      (fp8 && !aligned(scale, 16)))
    return DSA_ERR_MISALIGNED;
  return DSA_OK;
}

int check_table(const int* table, long long bt_stride, int W) {
  if (W <= 0 || bt_stride < 0 || (bt_stride != 0 && bt_stride < W)) return DSA_ERR_INVALID_ARG;
  if ((long long)W * dsa::kPage + dsa::kPage >= k2G) return DSA_ERR_UNSUPPORTED;
  return aligned(table, 4) ? DSA_OK : DSA_ERR_MISALIGNED;
}

#define DSA_CHECK(call)            \
  do {                             \
    const int st_ = (call);        \
    if (st_ != DSA_OK) return st_; \
  } while (0)

}  // namespace

extern "C" {

int dsa_request_slots(const int* lengths, const int* new_tokens, int n_req, const int* free_pages, int n_free,
                      int* block_table, long long bt_stride, int W, int page_size, int n, int* slots,
                      int* positions, int* seqlens, int* cu_rows, int* used, int* dev_status, void* stream) {
  if (n_req < 0 || n < 0 || n_free < 0) return DSA_ERR_INVALID_ARG;
  if (page_size != dsa::kPage) return DSA_ERR_UNSUPPORTED;
  DSA_CHECK(check_table(block_table, bt_stride, W));
  // requests have rows of their own here: their pages go into them
  if (n_req > 1 && bt_stride == 0) return DSA_ERR_INVALID_ARG;
  if (n_req > 0 && (!lengths || !new_tokens || !block_table)) return DSA_ERR_INVALID_ARG;
  if ((n > 0 && !slots) || (n_free > 0 && !free_pages)) return DSA_ERR_INVALID_ARG;
  // the blocks read the lengths while one of them writes these
  if (n_req > 0 && seqlens && (seqlens == lengths || seqlens == new_tokens)) return DSA_ERR_INVALID_ARG;
  if (!aligned(lengths, 4) || !aligned(new_tokens, 4) || !aligned(free_pages, 4) || !aligned(slots, 4) ||
      !aligned(positions, 4) || !aligned(seqlens, 4) || !aligned(cu_rows, 4) || !aligned(used, 4))
    return DSA_ERR_MISALIGNED;
  if (n == 0 && n_req == 0 && !cu_rows && !used) return DSA_OK;
  const dsa::RequestSlotsParams p{lengths, new_tokens, n_req, free_pages, n_free, block_table, bt_stride, W, n,
                                  slots, positions, seqlens, cu_rows, used, dev_status};
  return launched(dsa::launch_request_slots(p, static_cast<cudaStream_t>(stream)));
}

int dsa_kv_store(const void* k, long long k_token_stride, long long k_head_stride, const void* v,
                 long long v_token_stride, long long v_head_stride, int n, int Hkv, int D, int dtype,
                 const int* slot_mapping, void* k_cache, long long kc_page_stride, long long kc_slot_stride,
                 long long kc_head_stride, void* v_cache, long long vc_page_stride, long long vc_slot_stride,
                 long long vc_head_stride, float* k_scale, float* v_scale, int num_pages, int kv_dtype,
                 int page_size, int* dev_status, void* stream) {
  if (n < 0) return DSA_ERR_INVALID_ARG;
  DSA_CHECK(check_heads(Hkv, D, page_size));
  DSA_CHECK(check_types(dtype, kv_dtype));
  dsa::KvStoreParams p = {};
  p.at[0] = {kc_page_stride, kc_slot_stride, kc_head_stride};
  p.at[1] = {vc_page_stride, vc_slot_stride, vc_head_stride};
  DSA_CHECK(check_pool(k_cache, p.at[0], k_scale, Hkv, D, num_pages, kv_dtype));
  DSA_CHECK(check_pool(v_cache, p.at[1], v_scale, Hkv, D, num_pages, kv_dtype));
  if (n > 0 && (!k || !v || !slot_mapping)) return DSA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || k_token_stride % 8 || k_head_stride % 8 || v_token_stride % 8 ||
      v_head_stride % 8 || !aligned(slot_mapping, 4))
    return DSA_ERR_MISALIGNED;
  if ((long long)n * Hkv >= k2G) return DSA_ERR_UNSUPPORTED;
  if (n == 0) return DSA_OK;
  p.x[0] = k, p.x[1] = v;
  p.token[0] = k_token_stride, p.token[1] = v_token_stride;
  p.head[0] = k_head_stride, p.head[1] = v_head_stride;
  p.n = n, p.heads = Hkv, p.dim = D, p.dtype = dtype, p.slots = slot_mapping;
  p.pool[0] = k_cache, p.pool[1] = v_cache, p.scale[0] = k_scale, p.scale[1] = v_scale;
  p.num_pages = num_pages, p.status = dev_status;
  return launched(dsa::launch_kv_store(p, kv_dtype, static_cast<cudaStream_t>(stream)));
}

int dsa_block_bounds(const void* k_cache, long long kc_page_stride, long long kc_slot_stride,
                     long long kc_head_stride, const float* k_scale, int num_pages, int kv_dtype, int Hkv, int D,
                     int page_size, const int* block_table, long long bt_stride, int W, const int* starts,
                     const int* seqlens, int n_req, int max_tokens, signed char* bounds, float* bound_scale,
                     int* dev_status, void* stream) {
  if (n_req < 0 || max_tokens < 0) return DSA_ERR_INVALID_ARG;
  DSA_CHECK(check_heads(Hkv, D, page_size));
  if (kv_dtype != DSA_KV_FP8_E4M3 && kv_dtype != DSA_KV_BF16 && kv_dtype != DSA_KV_FP16) return DSA_ERR_INVALID_ARG;
  const dsa::PoolLayout at{kc_page_stride, kc_slot_stride, kc_head_stride};
  DSA_CHECK(check_pool(k_cache, at, k_scale, Hkv, D, num_pages, kv_dtype));
  DSA_CHECK(check_table(block_table, bt_stride, W));
  if (n_req > 0 && (!block_table || !seqlens || !bounds || !bound_scale)) return DSA_ERR_INVALID_ARG;
  if (!aligned(starts, 4) || !aligned(seqlens, 4) || !aligned(bounds, 16) || !aligned(bound_scale, 4))
    return DSA_ERR_MISALIGNED;
  if (n_req == 0 || max_tokens == 0) return DSA_OK;
  // pages that max_tokens tokens touch at most; more are taken in turns
  const long long touched = ((long long)max_tokens + 2 * dsa::kPage - 2) / dsa::kPage;
  const int pages = (int)(touched < W ? touched : W);
  if ((double)n_req * pages * Hkv >= (double)k2G) return DSA_ERR_UNSUPPORTED;
  const dsa::BlockBoundsParams p{k_cache, at, k_scale, Hkv, D, num_pages, block_table, bt_stride, W, starts, seqlens,
                                 n_req, pages, reinterpret_cast<int8_t*>(bounds), bound_scale, dev_status};
  const int sms = sm_count();
  if (sms <= 0) return DSA_ERR_CUDA;
  return launched(dsa::launch_block_bounds(p, kv_dtype, sms, static_cast<cudaStream_t>(stream)));
}

int dsa_block_select(const void* q, long long q_row_stride, long long q_head_stride, int rows, int Hq, int Hkv,
                     int D, int dtype, const signed char* bounds, const float* bound_scale, int num_pages,
                     const int* block_table, long long bt_stride, int W, int page_size, const int* seqlens, int k,
                     int first, int last, int* blocks, int* dev_status, void* stream) {
  if (rows < 0 || Hq <= 0 || !is16(dtype)) return DSA_ERR_INVALID_ARG;
  DSA_CHECK(check_heads(Hkv, D, page_size));
  if (Hq % Hkv) return DSA_ERR_INVALID_ARG;
  if (k <= 0 || first < 0 || last < 0 || (long long)first + last > k || num_pages <= 0) return DSA_ERR_INVALID_ARG;
  DSA_CHECK(check_table(block_table, bt_stride, W));
  // scores in shared memory; sums of a group's queries in 32 bits
  if (W > dsa::kSelectMaxPages || Hq / Hkv > 1024 || (long long)rows * Hkv * 8 >= k2G ||
      (long long)num_pages * dsa::kPage >= k2G)
    return DSA_ERR_UNSUPPORTED;
  if (rows > 0 && (!q || !bounds || !bound_scale || !block_table || !seqlens || !blocks)) return DSA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || q_row_stride % 8 || q_head_stride % 8 || !aligned(bounds, 16) || !aligned(bound_scale, 4) ||
      !aligned(seqlens, 4) || !aligned(blocks, 4))
    return DSA_ERR_MISALIGNED;
  if (rows == 0) return DSA_OK;
  const dsa::BlockSelectParams p{static_cast<const uint16_t*>(q), q_row_stride, q_head_stride, rows, Hkv, Hq / Hkv, D,
                                 dtype, reinterpret_cast<const int8_t*>(bounds), bound_scale, num_pages, block_table,
                                 bt_stride, W, seqlens, k, first, last, blocks, dev_status};
  const int sms = sm_count();
  if (sms <= 0) return DSA_ERR_CUDA;
  return launched(dsa::launch_block_select(p, sms, static_cast<cudaStream_t>(stream)));
}

long long dsa_paged_attention_workspace(int Hq, int Hkv, int D) {
  if (Hq <= 0 || Hkv <= 0 || Hq % Hkv || (D != 64 && D != 128)) return -1;
  const int sms = sm_count();
  return sms > 0 ? dsa::paged_ws_floats(sms, Hq / Hkv, D) : -1;
}

int dsa_paged_attention(const void* q, long long q_row_stride, long long q_head_stride, int rows, int Hq, int Hkv,
                        int D, int dtype, float scale, const void* k_cache, long long kc_page_stride,
                        long long kc_slot_stride, long long kc_head_stride, const void* v_cache,
                        long long vc_page_stride, long long vc_slot_stride, long long vc_head_stride,
                        const float* k_scale, const float* v_scale, int num_pages, int kv_dtype, int page_size,
                        const int* block_table, long long bt_stride, int W, const int* seqlens, const int* blocks,
                        long long blocks_row_stride, long long blocks_head_stride, int k, void* out,
                        long long out_row_stride, long long out_head_stride, float* lse, float* workspace,
                        long long workspace_floats, int* dev_status, void* stream) {
  if (rows < 0 || Hq <= 0) return DSA_ERR_INVALID_ARG;
  DSA_CHECK(check_heads(Hkv, D, page_size));
  if (Hq % Hkv) return DSA_ERR_INVALID_ARG;
  DSA_CHECK(check_types(dtype, kv_dtype));
  if (!(scale - scale == 0.f)) return DSA_ERR_INVALID_ARG;  // not finite
  const dsa::PoolLayout ka{kc_page_stride, kc_slot_stride, kc_head_stride};
  const dsa::PoolLayout va{vc_page_stride, vc_slot_stride, vc_head_stride};
  DSA_CHECK(check_pool(k_cache, ka, k_scale, Hkv, D, num_pages, kv_dtype));
  DSA_CHECK(check_pool(v_cache, va, v_scale, Hkv, D, num_pages, kv_dtype));
  DSA_CHECK(check_table(block_table, bt_stride, W));
  if (blocks && (k <= 0 || blocks_row_stride < 0 || blocks_head_stride < 0)) return DSA_ERR_INVALID_ARG;
  if (rows > 0 && (!q || !block_table || !seqlens || !out || !workspace)) return DSA_ERR_INVALID_ARG;
  const int group = Hq / Hkv, per_cta = dsa::paged_heads_max(group), tiles = (group + per_cta - 1) / per_cta;
  if ((double)rows * Hkv * tiles * ((blocks ? k : W) + 8.0) >= (double)k2G) return DSA_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || q_row_stride % 8 || q_head_stride % 8 || !aligned(out, 16) || out_row_stride % 8 ||
      out_head_stride % 8 || !aligned(workspace, 16) || !aligned(seqlens, 4) || !aligned(blocks, 4) ||
      !aligned(lse, 4))
    return DSA_ERR_MISALIGNED;
  if (rows == 0) return DSA_OK;
  const int sms = sm_count();
  if (sms <= 0) return DSA_ERR_CUDA;
  if (workspace_floats < dsa::paged_ws_floats(sms, group, D)) return DSA_ERR_INVALID_ARG;
  const int size = kv_dtype == DSA_KV_FP8_E4M3 ? 1 : 2;
  CUtensorMap kmap, vmap;
  // a dimension of one has any stride; the map wants a valid one
  auto encode = [&](CUtensorMap* m, const void* at, const dsa::PoolLayout& s) {
    return dsa::encode_kv_pool_map(m, at, D * size, s.slot * size, (Hkv > 1 ? s.head : s.slot) * size,
                                   (num_pages > 1 ? s.page : s.slot) * size, Hkv, num_pages);
  };
  if (!encode(&kmap, k_cache, ka) || !encode(&vmap, v_cache, va)) return DSA_ERR_UNSUPPORTED;
  dsa::PagedAttnParams p = {};
  p.q = static_cast<const uint16_t*>(q), p.q_row = q_row_stride, p.q_head = q_head_stride;
  p.rows = rows, p.heads = Hkv, p.group = group, p.tiles = tiles, p.dtype = dtype;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.k_scale = k_scale, p.v_scale = v_scale, p.num_pages = num_pages;
  p.block_table = block_table, p.bt_stride = bt_stride, p.W = W, p.seqlens = seqlens;
  p.blocks = blocks, p.b_row = blocks_row_stride, p.b_head = blocks_head_stride, p.k = k;
  p.out = static_cast<uint16_t*>(out), p.out_row = out_row_stride, p.out_head = out_head_stride;
  p.lse = lse, p.ws = workspace, p.status = dev_status;
  return launched(dsa::launch_paged_attention(p, D, kv_dtype, kmap, vmap, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
