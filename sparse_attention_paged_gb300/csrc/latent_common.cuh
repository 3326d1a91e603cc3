// latent_common.cuh -- parameters and layouts shared by the kernels around
// latent attention: the per-head norm + rotation, the latent cache's store
// and load, and the attention over it.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dsa_common.cuh"

namespace dsa {

constexpr int kLatent = 512;      // latent values per token
constexpr int kRope = 64;         // rotated values per token
constexpr int kLatentGroup = 128; // latent values that share one scale (fp8 cache)
constexpr int kLatentGroups = kLatent / kLatentGroup;

// bf16 page: 64 tokens of 576 values.  fp8 page: the 64 tokens' codes, then
// their rotated parts (bf16), then their scales (fp32).
constexpr int kTokenBytesBf16 = (kLatent + kRope) * 2;                         // 1,152
constexpr long long kPageBytesBf16 = (long long)kPage * kTokenBytesBf16;       // 73,728
constexpr int kRopeOffsetFp8 = kPage * kLatent;                                // 32,768
constexpr int kScaleOffsetFp8 = kRopeOffsetFp8 + kPage * kRope * 2;            // 40,960
constexpr long long kPageBytesFp8 = kScaleOffsetFp8 + kPage * kLatentGroups * 4;  // 41,984

struct NormRopeParams {
  const void* x[2];            // queries, keys
  void* y[2];
  long long xt[2], xh[2];      // token and head strides, elements
  long long yt[2], yh[2];
  int heads[2];
  const float* weight[2];      // nullable
  const float* bias[2];        // nullable
  int tokens, dim, norm;
  float eps;
  const int* positions;        // null: no rotation
  const float* table;          // [max_pos, rot]: rot/2 cosines, rot/2 sines
  int max_pos, rot, rot_offset, interleaved;
  int* status;
};

struct LatentStoreParams {
  const uint16_t* latent;      // bf16 bits, row i at latent + i * latent_stride
  const uint16_t* rope;
  long long latent_stride, rope_stride;
  int n;
  const float* weight;         // null: no norm
  float eps;
  const int* positions;        // null: no rotation
  const float* table;
  int max_pos, interleaved;
  const int* slots;
  uint8_t* cache;
  long long page_stride;
  int num_pages;
  int* status;
};

struct LatentLoadParams {
  const uint8_t* cache;
  long long page_stride;
  int num_pages;
  const int* block_table;
  long long bt_stride;
  int W;
  const int* starts;           // null: 0
  const int* cu;               // [n_req + 1]
  int n_req, n;
  uint16_t* out;
  long long out_stride;
  int* status;
};

struct LatentAttnParams {
  const uint16_t* ql;          // bf16 bits, [rows, H, 512] through the strides
  const uint16_t* qr;          // [rows, H, 64]
  long long ql_row, ql_head, qr_row, qr_head;
  int rows, H, groups;         // groups = ceil(H / 64)
  float scale_log2;            // scale * log2(e)
  const uint8_t* cache;
  long long page_stride;
  int num_pages;
  const int* block_table;
  long long bt_stride;
  int W;
  const int* seqlens;
  const int* idx;              // null: every position below the length
  long long idx_stride;
  int k;
  uint16_t* out;
  long long out_row, out_head;
  float* lse;                  // nullable, [rows, H]
  float* ws;
  int* status;
  int ctas;                    // CTAs per head group
};

// The attention's workspace: per CTA two partial rows (the sums of 64 heads
// x 512 values, their maxima and their totals), then the split records.
constexpr int kAttnHeads = 64;
constexpr int kPartialFloats = kAttnHeads * kLatent + 2 * kAttnHeads;
constexpr int kSplitInts = 4;
constexpr long long latent_ws_floats(long long sms) { return sms * (2LL * kPartialFloats + kSplitInts); }

// A split record {row, CTA with its last unit, CTA with its first, 0} that names rows and CTAs of
// this call.  The join takes addresses from it, and the workspace is the caller's memory.
__host__ __device__ constexpr bool split_record_ok(int row, int last, int first, int rows, int ctas) {
  return row >= 0 && row < rows && first >= 0 && first <= last && last < ctas;
}

}  // namespace dsa
