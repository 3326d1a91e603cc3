// latent_api.cu -- the C ABI of the calls around the sparse attention
// (include/dsa_indexer.h): argument checks, parameter packing and launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include "dsa_indexer.h"
#include "latent_common.cuh"

namespace dsa {
cudaError_t launch_norm_rope(const NormRopeParams& p, int dtype, cudaStream_t stream);
cudaError_t launch_latent_store(const LatentStoreParams& p, int kv_dtype, cudaStream_t stream);
cudaError_t launch_latent_load(const LatentLoadParams& p, int kv_dtype, cudaStream_t stream);
cudaError_t launch_latent_attention(const LatentAttnParams& p, int kv_dtype, int sms,
                                    cudaStream_t stream);
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

// The pool's arguments, shared by the cache calls.
int check_cache(const void* cache, long long page_stride, int num_pages, int kv_dtype,
                int page_size, int latent_dim, int rope_dim) {
  if (latent_dim != dsa::kLatent || rope_dim != dsa::kRope || page_size != dsa::kPage)
    return DSA_ERR_UNSUPPORTED;
  if (kv_dtype != DSA_KV_FP8_E4M3 && kv_dtype != DSA_KV_BF16) return DSA_ERR_INVALID_ARG;
  if (!cache || num_pages <= 0) return DSA_ERR_INVALID_ARG;
  if (page_stride < (kv_dtype == DSA_KV_BF16 ? dsa::kPageBytesBf16 : dsa::kPageBytesFp8))
    return DSA_ERR_INVALID_ARG;
  if (page_stride % 16 != 0 || !aligned(cache, 16)) return DSA_ERR_MISALIGNED;
  return DSA_OK;
}

int check_rotation(const int* positions, const float* table, int max_pos) {
  if (!positions) return DSA_OK;
  if (!table || max_pos <= 0) return DSA_ERR_INVALID_ARG;
  if (!aligned(positions, 4) || !aligned(table, 16)) return DSA_ERR_MISALIGNED;
  return DSA_OK;
}

}  // namespace

extern "C" {

int dsa_qk_norm_rope(const void* q, long long q_token_stride, long long q_head_stride, int Hq,
                     const void* k, long long k_token_stride, long long k_head_stride, int Hk,
                     int T, int D, int dtype, int norm, const float* q_weight,
                     const float* k_weight, const float* q_bias, const float* k_bias, float eps,
                     const int* positions, const float* rope_table, int max_pos, int rot_dims,
                     int rot_offset, int interleaved, void* q_out, long long qo_token_stride,
                     long long qo_head_stride, void* k_out, long long ko_token_stride,
                     long long ko_head_stride, int* dev_status, void* stream) {
  if (T < 0 || Hq < 0 || Hk < 0) return DSA_ERR_INVALID_ARG;
  if (dtype != DSA_BF16 && dtype != DSA_FP16 && dtype != DSA_FP32) return DSA_ERR_INVALID_ARG;
  if (norm != DSA_NORM_NONE && norm != DSA_NORM_RMS && norm != DSA_NORM_LAYER)
    return DSA_ERR_INVALID_ARG;
  if (!(eps >= 0.f)) return DSA_ERR_INVALID_ARG;
  if (D < 8 || D > 256 || D % 8 != 0) return DSA_ERR_UNSUPPORTED;
  if (positions) {
    if (rot_dims <= 0 || rot_offset < 0 || rot_dims > D || rot_offset > D - rot_dims)
      return DSA_ERR_INVALID_ARG;
    if (rot_offset % 8 != 0 || rot_dims % (interleaved ? 8 : 16) != 0) return DSA_ERR_UNSUPPORTED;
  }
  if (T > 0 && Hq > 0 && (!q || !q_out)) return DSA_ERR_INVALID_ARG;
  if (T > 0 && Hk > 0 && (!k || !k_out)) return DSA_ERR_INVALID_ARG;
  int st = check_rotation(positions, rope_table, max_pos);
  if (st != DSA_OK) return st;
  const long long unit = dtype == DSA_FP32 ? 4 : 8;  // elements in 16 bytes
  if (Hq > 0 && (!aligned(q, 16) || !aligned(q_out, 16) || q_token_stride % unit ||
                 q_head_stride % unit || qo_token_stride % unit || qo_head_stride % unit))
    return DSA_ERR_MISALIGNED;
  if (Hk > 0 && (!aligned(k, 16) || !aligned(k_out, 16) || k_token_stride % unit ||
                 k_head_stride % unit || ko_token_stride % unit || ko_head_stride % unit))
    return DSA_ERR_MISALIGNED;
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(q_bias, 16) || !aligned(k_bias, 16))
    return DSA_ERR_MISALIGNED;
  if (T == 0 || Hq + (long long)Hk == 0) return DSA_OK;
  // at most one unit of 32 lanes per head: the grid stays below 2^31 blocks
  if ((double)T * ((double)Hq + Hk) >= 8e9) return DSA_ERR_UNSUPPORTED;
  dsa::NormRopeParams p = {};
  p.x[0] = q, p.x[1] = k, p.y[0] = q_out, p.y[1] = k_out;
  p.xt[0] = q_token_stride, p.xt[1] = k_token_stride;
  p.xh[0] = q_head_stride, p.xh[1] = k_head_stride;
  p.yt[0] = qo_token_stride, p.yt[1] = ko_token_stride;
  p.yh[0] = qo_head_stride, p.yh[1] = ko_head_stride;
  p.heads[0] = Hq, p.heads[1] = Hk;
  p.weight[0] = q_weight, p.weight[1] = k_weight;
  p.bias[0] = q_bias, p.bias[1] = k_bias;
  p.tokens = T, p.dim = D, p.norm = norm, p.eps = eps;
  p.positions = positions, p.table = rope_table, p.max_pos = max_pos;
  p.rot = positions ? rot_dims : 0, p.rot_offset = positions ? rot_offset : 0;
  p.interleaved = interleaved != 0, p.status = dev_status;
  return launched(dsa::launch_norm_rope(p, dtype, static_cast<cudaStream_t>(stream)));
}

int dsa_latent_store(const void* latent, long long latent_stride, const void* rope,
                     long long rope_stride, int n, int latent_dim, int rope_dim,
                     const float* norm_weight, float eps, const int* positions,
                     const float* rope_table, int max_pos, int interleaved,
                     const int* slot_mapping, void* cache, long long page_stride_bytes,
                     int num_pages, int kv_dtype, int page_size, int* dev_status, void* stream) {
  if (n < 0 || !(eps >= 0.f)) return DSA_ERR_INVALID_ARG;
  int st = check_cache(cache, page_stride_bytes, num_pages, kv_dtype, page_size, latent_dim, rope_dim);
  if (st != DSA_OK) return st;
  if (n > 0 && (!latent || !rope || !slot_mapping)) return DSA_ERR_INVALID_ARG;
  st = check_rotation(positions, rope_table, max_pos);
  if (st != DSA_OK) return st;
  if (!aligned(latent, 16) || latent_stride % 8 != 0 || !aligned(rope, 4) || rope_stride % 2 != 0 ||
      !aligned(norm_weight, 16) || !aligned(slot_mapping, 4))
    return DSA_ERR_MISALIGNED;
  if (n == 0) return DSA_OK;
  const dsa::LatentStoreParams p{static_cast<const uint16_t*>(latent),
                                 static_cast<const uint16_t*>(rope),
                                 latent_stride, rope_stride, n, norm_weight, eps, positions,
                                 rope_table, max_pos, interleaved != 0, slot_mapping,
                                 static_cast<uint8_t*>(cache), page_stride_bytes, num_pages,
                                 dev_status};
  return launched(dsa::launch_latent_store(p, kv_dtype, static_cast<cudaStream_t>(stream)));
}

int dsa_latent_load(const void* cache, long long page_stride_bytes, int num_pages, int kv_dtype,
                    int page_size, const int* block_table, long long bt_stride, int W,
                    const int* starts, const int* cu_rows, int n_req, int n, int latent_dim,
                    int rope_dim, void* out, long long out_stride, int* dev_status, void* stream) {
  if (n < 0 || n_req < 0 || W <= 0) return DSA_ERR_INVALID_ARG;
  int st = check_cache(cache, page_stride_bytes, num_pages, kv_dtype, page_size, latent_dim, rope_dim);
  if (st != DSA_OK) return st;
  if (bt_stride < 0 || (bt_stride != 0 && bt_stride < W)) return DSA_ERR_INVALID_ARG;
  if (n > 0 && (n_req == 0 || !block_table || !cu_rows || !out)) return DSA_ERR_INVALID_ARG;
  if (out_stride < dsa::kLatent + dsa::kRope) return DSA_ERR_INVALID_ARG;
  if (!aligned(out, 16) || out_stride % 8 != 0 || !aligned(block_table, 4) || !aligned(cu_rows, 4) ||
      !aligned(starts, 4))
    return DSA_ERR_MISALIGNED;
  if (n == 0) return DSA_OK;
  const dsa::LatentLoadParams p{static_cast<const uint8_t*>(cache), page_stride_bytes, num_pages,
                                block_table, bt_stride, W, starts, cu_rows, n_req, n,
                                static_cast<uint16_t*>(out), out_stride, dev_status};
  return launched(dsa::launch_latent_load(p, kv_dtype, static_cast<cudaStream_t>(stream)));
}

long long dsa_latent_attention_workspace(void) {
  const int sms = sm_count();
  return sms > 0 ? dsa::latent_ws_floats(sms) : -1;
}

int dsa_latent_attention(const void* q_latent, long long ql_row_stride, long long ql_head_stride,
                         const void* q_rope, long long qr_row_stride, long long qr_head_stride,
                         int rows, int H, int latent_dim, int rope_dim, float scale,
                         const void* cache, long long page_stride_bytes, int num_pages,
                         int kv_dtype, int page_size, const int* block_table, long long bt_stride,
                         int W, const int* seqlens, const int* idx, long long idx_stride, int k,
                         void* out, long long out_row_stride, long long out_head_stride,
                         float* lse, float* workspace, long long workspace_floats,
                         int* dev_status, void* stream) {
  if (rows < 0 || W <= 0 || H <= 0) return DSA_ERR_INVALID_ARG;
  int st = check_cache(cache, page_stride_bytes, num_pages, kv_dtype, page_size, latent_dim, rope_dim);
  if (st != DSA_OK) return st;
  if (H > 2 * dsa::kAttnHeads) return DSA_ERR_UNSUPPORTED;
  if (!(scale - scale == 0.f)) return DSA_ERR_INVALID_ARG;  // not finite
  if (bt_stride < 0 || (bt_stride != 0 && bt_stride < W)) return DSA_ERR_INVALID_ARG;
  if (idx && (k <= 0 || idx_stride < k)) return DSA_ERR_INVALID_ARG;
  if (rows > 0 && (!q_latent || !q_rope || !block_table || !seqlens || !out || !workspace))
    return DSA_ERR_INVALID_ARG;
  const long long tiles = idx ? (k + 63LL) / 64 : W;
  if ((long long)rows * tiles >= (1LL << 31) || (long long)W * dsa::kPage >= (1LL << 31) ||
      (long long)num_pages * dsa::kPage >= (1LL << 31))
    return DSA_ERR_UNSUPPORTED;
  if (!aligned(q_latent, 16) || !aligned(q_rope, 16) || ql_row_stride % 8 || ql_head_stride % 8 ||
      qr_row_stride % 8 || qr_head_stride % 8 || !aligned(out, 16) || out_row_stride % 8 ||
      out_head_stride % 8 || !aligned(workspace, 16) || !aligned(block_table, 4) ||
      !aligned(seqlens, 4) || !aligned(idx, 4) || !aligned(lse, 4))
    return DSA_ERR_MISALIGNED;
  if (rows == 0) return DSA_OK;
  const int sms = sm_count();
  if (sms <= 0) return DSA_ERR_CUDA;
  if (workspace_floats < dsa::latent_ws_floats(sms)) return DSA_ERR_INVALID_ARG;
  dsa::LatentAttnParams p = {};
  p.ql = static_cast<const uint16_t*>(q_latent), p.qr = static_cast<const uint16_t*>(q_rope);
  p.ql_row = ql_row_stride, p.ql_head = ql_head_stride;
  p.qr_row = qr_row_stride, p.qr_head = qr_head_stride;
  p.rows = rows, p.H = H, p.groups = (H + dsa::kAttnHeads - 1) / dsa::kAttnHeads;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.cache = static_cast<const uint8_t*>(cache), p.page_stride = page_stride_bytes;
  p.num_pages = num_pages, p.block_table = block_table, p.bt_stride = bt_stride, p.W = W;
  p.seqlens = seqlens, p.idx = idx, p.idx_stride = idx_stride, p.k = k;
  p.out = static_cast<uint16_t*>(out), p.out_row = out_row_stride, p.out_head = out_head_stride;
  p.lse = lse, p.ws = workspace, p.status = dev_status;
  return launched(dsa::launch_latent_attention(p, kv_dtype, sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
