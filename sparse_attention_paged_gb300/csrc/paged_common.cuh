// paged_common.cuh -- parameters shared by the kernels of the paged cache of
// keys and values: slots from request lengths, the cache's store, the pages'
// boxes, the selection of pages and the attention over them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dsa_common.cuh"

namespace dsa {

struct RequestSlotsParams {
  const int* lengths;          // [n_req] cached tokens
  const int* fresh;            // [n_req] new tokens
  int n_req;
  const int* free_pages;
  int n_free;
  int* block_table;
  long long bt_stride;
  int W;
  int n;                       // rows of slots and positions
  int* slots;
  int* positions;              // nullable
  int* seqlens;                // nullable, [n_req]
  int* cu;                     // nullable, [n_req + 1]
  int* used;                   // nullable
  int* status;
};

// One pool of keys or values: token s of head h in page p starts at
// at + p * page + s * slot + h * head (elements).
struct PoolLayout {
  long long page, slot, head;
};

struct KvStoreParams {
  const void* x[2];            // keys, values: [n, heads, dim], 16-bit
  long long token[2], head[2]; // strides, elements
  int n, heads, dim, dtype;
  const int* slots;
  void* pool[2];
  PoolLayout at[2];
  float* scale[2];             // fp8: [pages, heads, 64]
  int num_pages;
  int* status;
};

struct BlockBoundsParams {
  const void* pool;
  PoolLayout at;
  const float* scale;          // fp8: [pages, heads, 64]
  int heads, dim, num_pages;
  const int* block_table;
  long long bt_stride;
  int W;
  const int* starts;           // null: 0
  const int* seqlens;
  int n_req;
  int pages;                   // pages of a request that the grid covers at once
  int8_t* bounds;              // [pages, heads, 2, dim]
  float* bound_scale;          // [pages, heads]
  int* status;
};

// The selection keeps a row's scores in shared memory, and up to a list's
// length also the best of several blocks.
constexpr int kSelectMaxPages = 32768, kSelectMaxList = 1024;

// A row's n pages among the blocks that share it: pages of a block's run, at least
// kSelectRun where there are as many (a row of few pages is one block's), and blocks that
// have one.  A row without pages is one block's too: neither is ever 0.
constexpr int kSelectRun = 256;
constexpr int select_run(int n, int blocks) {
  const int even = (n + blocks - 1) / blocks, least = n < kSelectRun ? n : kSelectRun;
  return even > least ? even : least > 1 ? least : 1;
}
constexpr int select_active(int n, int run) { return n > run ? (n + run - 1) / run : 1; }

struct BlockSelectParams {
  const uint16_t* q;           // bf16 or fp16 bits, [rows, Hq, dim] through the strides
  long long q_row, q_head;
  int rows, heads, group, dim, dtype;  // heads: of the keys
  const int8_t* bounds;
  const float* bound_scale;
  int num_pages;
  const int* block_table;
  long long bt_stride;
  int W;
  const int* seqlens;
  int k, first, last;
  int* blocks;                 // [rows, heads, k]
  int* status;
};

struct PagedAttnParams {
  const uint16_t* q;           // bf16 or fp16 bits, [rows, Hq, dim] through the strides
  long long q_row, q_head;
  int rows, heads, group;      // heads: of the keys; group: query heads of each
  int tiles;                   // work items of a key head: ceil(group / heads that a CTA takes)
  int dtype;
  float scale_log2;            // scale * log2(e)
  const float* k_scale;        // fp8: [pages, heads, 64]
  const float* v_scale;
  int num_pages;
  const int* block_table;
  long long bt_stride;
  int W;
  const int* seqlens;
  const int* blocks;           // null: every page below the length
  long long b_row, b_head;
  int k;
  uint16_t* out;
  long long out_row, out_head;
  float* lse;                  // nullable, [rows, Hq]
  float* ws;
  int* status;
};

// The attention's launch, by the query heads of a key head: heads that a CTA
// takes (one or two column tiles of 8 per warp, one or two sets of warps), and
// CTAs per SM.
constexpr int paged_heads_max(int group) { return group > 16 ? 32 : group > 8 ? 16 : 8; }
constexpr int paged_ctas_per_sm(int group) { return group > 16 ? 1 : 2; }
constexpr int paged_cta_heads(int group) { return group < paged_heads_max(group) ? group : paged_heads_max(group); }

// Its workspace: two partial results per CTA (sums of the CTA's heads, then
// their statistics, four floats a head), then a split record of four ints per CTA.
constexpr long long paged_ws_floats(long long sms, int group, int dim) {
  return sms * paged_ctas_per_sm(group) * (2LL * paged_cta_heads(group) * (dim + 4) + 4);
}

}  // namespace dsa
