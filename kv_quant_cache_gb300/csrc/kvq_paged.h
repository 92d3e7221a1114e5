// kvq_paged.h -- internal host-side interface of the paged grouped-query
// operators (kvq_paged_api.cu validates and dispatches, the kernels' files
// launch).  Not installed; callers use include/kvq.h.
//
// The cache is bf16 [num_pages, 2, num_heads_kv, page_size, head_dim]: of each
// page the keys of every kv head, then the values.  Token slot s is offset
// s % page_size of page s / page_size.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq_launch.h"

namespace kvq {

struct AppendArgs {
  void* qkv;
  void* q_out;  // == qkv: q rows rotated in place
  const float* cos_sin;  // nullptr: no rotation (rotary_dim 0)
  const int64_t* positions;
  const int64_t* slot_mapping;
  void* kv_cache;
  int num_tokens;
  int num_heads_q, num_heads_kv;
  int head_dim, rotary_dim, is_neox;
  int64_t max_pos, num_pages;
  int page_size;
  int* errors;
};

struct PageBoundsArgs {
  const void* kv_cache;
  const int64_t* pages;
  const int* lens;
  void* bounds;
  int num_listed;
  int num_heads_kv, head_dim, page_size;
  int64_t num_pages;
  int* errors;
};

// What the block selection and both attentions share: queries, the request
// each of them belongs to, and the requests' pages.
struct PagedQuery {
  const void* q;
  int64_t q_stride;  // elements between tokens
  int num_tokens;
  int num_heads_q, num_heads_kv, head_dim;
  int64_t num_pages;
  int page_size;
  const int* page_table;  // [num_requests, table_width]
  int num_requests, table_width;
  const int* requests;  // request of each token; nullptr: token t is request t
  const int* lens;      // keys of the request that each token sees
  int* errors;
};

struct BlockSelectArgs {
  PagedQuery x;
  const void* bounds;
  int topk, keep_first, keep_last;
  int* blocks;
};

struct SparseAttnArgs {
  PagedQuery x;
  const void* kv_cache;
  const int* blocks;
  int topk;
  float scale;
  void* out;
  void* workspace;
};

struct PrefixAttnArgs {
  PagedQuery x;
  const void* kv_cache;
  const int* prefix_pages;
  int64_t prefix_len;
  int config;  // prefix_config() as it was when the workspace was checked
  float scale;
  void* out;
  void* workspace;
};

// The paged cache held in 4 bits (kvq_kv4.cuh); its append takes AppendArgs.
struct Kv4GatherArgs {
  const void* kv_cache;
  const int64_t* slots;
  int64_t num_listed;
  void* k;
  void* v;
  int num_heads_kv, head_dim, page_size;
  int64_t num_pages;
  int* errors;
};

struct Kv4AttnArgs {
  PagedQuery x;  // (requests is not used)
  const void* kv_cache;
  int per_request;  // tokens of a request
  float scale;
  void* out;
  void* workspace;
};

// Attention over listed 584-byte latent entries.
struct LatentAttnArgs {
  const void* q;
  int64_t q_stride;  // elements between tokens
  int num_tokens, num_heads;
  const uint8_t* kv_cache;
  int64_t num_slots;
  const int* slots;  // [num_tokens, list_width]
  int list_width;
  const int* lens;
  float scale;
  void* out;
  void* workspace;
  int* errors;
};

// Pages of one request (or of the block selection) that a call may list.
constexpr int kMaxSelectBlocks = 16384;

cudaError_t launch_paged_append(const AppendArgs& a, cudaStream_t stream);
cudaError_t launch_page_bounds(const PageBoundsArgs& a, cudaStream_t stream);
cudaError_t launch_block_select(const BlockSelectArgs& a, cudaStream_t stream);
cudaError_t launch_sparse_attn(const SparseAttnArgs& a, cudaStream_t stream);
cudaError_t launch_prefix_attn(const PrefixAttnArgs& a, cudaStream_t stream);

cudaError_t launch_kv4_append(const AppendArgs& a, cudaStream_t stream);
cudaError_t launch_kv4_gather(const Kv4GatherArgs& a, cudaStream_t stream);
cudaError_t launch_kv4_attn(const Kv4AttnArgs& a, cudaStream_t stream);
cudaError_t launch_latent_attn(const LatentAttnArgs& a, cudaStream_t stream);

// Row tiles of the attention over the 4-bit cache (CTAs at least), and the bytes of
// workspace that it and the latent attention need.
int64_t kv4_attn_units(int64_t num_tokens, int per_request, int num_heads_q, int num_heads_kv);
int64_t kv4_attn_workspace(int64_t num_tokens, int per_request, int num_heads_q,
                           int num_heads_kv, int head_dim, int page_size, int table_width);
int64_t latent_attn_workspace(int64_t num_tokens, int num_heads, int list_width);

// The ways the prefix can be taken (kvq_set_prefix_config).
extern const LaunchConfig kPrefixConfigs[];
extern const int kPrefixNumConfigs;
int set_prefix_config(int id);  // -1: by the sizes; returns the previous one
int prefix_config();
uint32_t set_tile_wait_limit(uint32_t polls);  // kvq_set_tile_wait_limit
uint32_t tile_wait_limit();

// Bytes of workspace the two attentions need (0: none).
// Depends on the sizes (and a forced configuration) alone, so that it can be
// asked for without a device.  A call reads prefix_config() once and hands it
// on: one that changes meanwhile may not change what the workspace is for.
int64_t sparse_attn_workspace(int64_t num_tokens, int num_heads_q, int num_heads_kv,
                              int head_dim, int page_size, int topk);
int64_t prefix_attn_workspace(int64_t num_tokens, int num_heads_q, int num_heads_kv,
                              int head_dim, int page_size, int64_t prefix_len, int table_width,
                              int config);

}  // namespace kvq
