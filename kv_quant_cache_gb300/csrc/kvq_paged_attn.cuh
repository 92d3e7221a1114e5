// kvq_paged_attn.cuh -- what the paged attention kernels share: the partial
// results of a split key range, and their join.
//
// A row is one query head of one token.  Softmax over a key range split into
// parts needs of each part its normalised output o_i and
// l_i = log2(sum over its keys of 2^(s log2 e)); then
//   out = sum_i w_i o_i / sum_i w_i,   w_i = 2^(l_i - max l).
// A part without a key has l_i = -inf and weight 0; a row without any part
// left is zero.  o_i and l_i are fp32.
#pragma once

#include <cuda.h>

#include "kvq_device.cuh"
#include "kvq_paged.h"

namespace kvq {

constexpr float kLog2e = 1.4426950408889634f;

// Partials of `slots` parts: [slots][rows][D] fp32, then [slots][rows] fp32.
struct Partials {
  float* o;
  float* lse;
  int64_t rows;
};

inline int64_t partials_bytes(int64_t slots, int64_t rows, int head_dim) {
  return slots * rows * ((int64_t)head_dim + 1) * 4;
}

inline Partials partials_at(void* workspace, int64_t slots, int64_t rows, int head_dim) {
  Partials p;
  p.o = static_cast<float*>(workspace);
  p.lse = p.o + slots * rows * head_dim;
  p.rows = rows;
  return p;
}

// Joins the parts into out bf16 [rows][D].
cudaError_t launch_attn_join(const Partials& parts, int slots, int head_dim, void* out,
                             cudaStream_t stream);

// The prefix on the tensor cores (kvq_paged_prefix.cu): sizes it takes, the
// parts it makes of the prefix, the tensor map of the cache (false where it
// cannot be copied that way: not memory of the current device, no pages), and
// the launch (partials slots 0 .. parts - 1).
struct PrefixTilesPlan {
  int row_tiles;  // items of 256 query rows of a kv head (128: heads of 256)
  int blocks;     // of 128 keys, of the prefix
  int lanes, teams;  // CTAs that keep in step, and how many times so many
  int parts;      // partials of an item, at most
};
bool prefix_tiles_fit(int64_t num_tokens, int num_heads_q, int num_heads_kv, int head_dim,
                      int page_size, int64_t prefix_len, int config);
PrefixTilesPlan prefix_tiles_plan(int64_t num_tokens, int num_heads_q, int num_heads_kv,
                                  int head_dim, int64_t prefix_len);
bool prefix_tiles_map(const PrefixAttnArgs& a, CUtensorMap* map);
cudaError_t launch_prefix_tiles(const PrefixAttnArgs& a, const CUtensorMap& map,
                                const Partials& parts, cudaStream_t stream);

}  // namespace kvq
