// kvq_kv4_api.cu -- the C ABI of the operators on quantised caches (include/kvq.h):
// host-side validation and launch on the caller's stream.  No allocation, no sync.
#include <climits>
#include <cmath>

#include "kvq.h"
#include "kvq_dsv4_entry.cuh"
#include "kvq_launch.h"
#include "kvq_paged.h"

namespace {

using kvq::report_launch;

constexpr int64_t kIndexLimit = (int64_t)1 << 31;
constexpr int kMaxPageSize = 1 << 16;
constexpr int kMaxHeads = 1 << 16;
constexpr int64_t kMaxListed = 1 << 22;  // pages of a request
constexpr int64_t kMaxEntries = 1 << 30;  // latent entries listed for a token
constexpr int kMaxCluster = 8;           // CTAs of a row tile along the grid's x

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// (infinite in units of log2 it would make NaN of a score of zero)
bool scale_ok(float scale) { return std::isfinite(scale * 1.4426950408889634f); }

bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}

kvq_status check_cache4(int num_heads_kv, int head_dim, int64_t num_pages, int page_size) {
  if (num_heads_kv < 1 || num_heads_kv > kMaxHeads || num_pages < 0 ||
      num_pages > (int64_t)INT_MAX || page_size < 1 || page_size > kMaxPageSize)
    return KVQ_ERR_SHAPE;
  return (head_dim == 64 || head_dim == 128 || head_dim == 256) && page_size % 16 == 0
             ? KVQ_OK
             : KVQ_ERR_UNSUPPORTED;
}

kvq_status check_rows(int64_t num_tokens, int num_heads, int64_t q_stride, int dim) {
  if (num_tokens < 0 || num_tokens >= kIndexLimit || num_heads < 1 || num_heads > kMaxHeads ||
      num_tokens * num_heads >= kIndexLimit || q_stride < (int64_t)num_heads * dim ||
      q_stride >= kIndexLimit)
    return KVQ_ERR_SHAPE;
  return q_stride % 8 == 0 ? KVQ_OK : KVQ_ERR_ALIGN;
}

}  // namespace

extern "C" {

kvq_status paged_kv4_rope_append(void* qkv, void* q_out, int64_t num_tokens, int num_heads_q,
                                 int num_heads_kv, int head_dim, const float* cos_sin_cache,
                                 int64_t max_pos, int rotary_dim, int is_neox,
                                 const int64_t* positions, const int64_t* slot_mapping,
                                 void* kv_cache, int64_t num_pages, int page_size,
                                 int32_t* error_count, kvq_stream_t stream) {
  const kvq_status c = check_cache4(num_heads_kv, head_dim, num_pages, page_size);
  if (c != KVQ_OK) return c;
  if (num_tokens < 0 || num_heads_q < 0 || num_heads_q > kMaxHeads || max_pos < 0)
    return KVQ_ERR_SHAPE;
  if (is_neox != 0 && is_neox != 1) return KVQ_ERR_UNSUPPORTED;
  if (rotary_dim != 0 && (rotary_dim < 16 || rotary_dim > head_dim || rotary_dim % 16 != 0))
    return KVQ_ERR_UNSUPPORTED;
  const int64_t rows = (int64_t)num_heads_q + 2 * (int64_t)num_heads_kv;
  if (num_tokens >= kIndexLimit || num_tokens * rows >= kIndexLimit) return KVQ_ERR_SHAPE;
  if (num_tokens == 0) return KVQ_OK;
  if (!qkv || !slot_mapping || !kv_cache) return KVQ_ERR_NULL;
  if (rotary_dim != 0 && (!cos_sin_cache || !positions)) return KVQ_ERR_NULL;
  if (!aligned(qkv, 16) || !aligned(q_out, 16) || !aligned(kv_cache, 16) ||
      !aligned(slot_mapping, 8) || !aligned(error_count, 4) ||
      (rotary_dim != 0 && (!aligned(cos_sin_cache, 16) || !aligned(positions, 8))))
    return KVQ_ERR_ALIGN;
  if (q_out && overlap(q_out, num_tokens * num_heads_q * head_dim * 2, qkv,
                       num_tokens * rows * head_dim * 2))
    return KVQ_ERR_VALUE;
  kvq::AppendArgs a;
  a.qkv = qkv;
  a.q_out = q_out ? q_out : qkv;
  a.cos_sin = cos_sin_cache;
  a.positions = positions;
  a.slot_mapping = slot_mapping;
  a.kv_cache = kv_cache;
  a.num_tokens = (int)num_tokens;
  a.num_heads_q = num_heads_q;
  a.num_heads_kv = num_heads_kv;
  a.head_dim = head_dim;
  a.rotary_dim = rotary_dim;
  a.is_neox = is_neox;
  a.max_pos = max_pos;
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.errors = error_count;
  return report_launch(kvq::launch_kv4_append(a, reinterpret_cast<cudaStream_t>(stream)));
}

kvq_status paged_kv4_gather(const void* kv_cache, int64_t num_pages, int num_heads_kv,
                            int page_size, int head_dim, const int64_t* slots,
                            int64_t num_listed, void* k, void* v, int32_t* error_count,
                            kvq_stream_t stream) {
  const kvq_status c = check_cache4(num_heads_kv, head_dim, num_pages, page_size);
  if (c != KVQ_OK) return c;
  if (num_listed < 0 || num_listed >= kIndexLimit || num_listed * 2 * num_heads_kv >= kIndexLimit)
    return KVQ_ERR_SHAPE;
  if (num_listed == 0) return KVQ_OK;
  if (!kv_cache || !slots || !k || !v) return KVQ_ERR_NULL;
  if (!aligned(kv_cache, 16) || !aligned(slots, 8) || !aligned(k, 16) || !aligned(v, 16) ||
      !aligned(error_count, 4))
    return KVQ_ERR_ALIGN;
  const int64_t bytes = num_listed * num_heads_kv * head_dim * 2;
  if (overlap(k, bytes, v, bytes)) return KVQ_ERR_VALUE;
  kvq::Kv4GatherArgs a;
  a.kv_cache = kv_cache;
  a.slots = slots;
  a.num_listed = num_listed;
  a.k = k;
  a.v = v;
  a.num_heads_kv = num_heads_kv;
  a.head_dim = head_dim;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.errors = error_count;
  return report_launch(kvq::launch_kv4_gather(a, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t paged_kv4_attention_workspace(int64_t num_tokens, int64_t tokens_per_request,
                                      int num_heads_q, int num_heads_kv, int head_dim,
                                      int page_size, int64_t table_width) {
  if (num_tokens < 1 || tokens_per_request < 1 || num_tokens % tokens_per_request != 0 ||
      num_heads_q < 1 || num_heads_q > kMaxHeads || num_heads_kv < 1 ||
      num_heads_q % num_heads_kv != 0 || check_cache4(num_heads_kv, head_dim, 0, page_size) ||
      table_width < 0 || table_width > kMaxListed || num_tokens >= kIndexLimit ||
      num_tokens * num_heads_q >= kIndexLimit)
    return 0;
  return kvq::kv4_attn_workspace(num_tokens, (int)tokens_per_request, num_heads_q, num_heads_kv,
                                 head_dim, page_size, (int)table_width);
}

kvq_status paged_kv4_attention(const void* q, int64_t q_stride, int64_t num_tokens,
                               int64_t tokens_per_request, int num_heads_q, int num_heads_kv,
                               int head_dim, const void* kv_cache, int64_t num_pages,
                               int page_size, const int32_t* page_table, int64_t table_width,
                               const int32_t* lens, float scale, void* out, void* workspace,
                               int64_t workspace_bytes, int32_t* error_count,
                               kvq_stream_t stream) {
  kvq_status c = check_cache4(num_heads_kv, head_dim, num_pages, page_size);
  if (c == KVQ_OK) c = check_rows(num_tokens, num_heads_q, q_stride, head_dim);
  if (c != KVQ_OK) return c;
  if (num_heads_q % num_heads_kv != 0 || tokens_per_request < 1 ||
      num_tokens % tokens_per_request != 0 || table_width < 0 || table_width > kMaxListed)
    return KVQ_ERR_SHAPE;
  if (!scale_ok(scale)) return KVQ_ERR_VALUE;
  if (num_tokens == 0) return KVQ_OK;
  if (kvq::kv4_attn_units(num_tokens, (int)tokens_per_request, num_heads_q, num_heads_kv) *
          kMaxCluster >= kIndexLimit)  // CTAs of the grid
    return KVQ_ERR_SHAPE;
  if (!q || !kv_cache || !lens || !out || (table_width > 0 && !page_table)) return KVQ_ERR_NULL;
  const int64_t need =
      kvq::kv4_attn_workspace(num_tokens, (int)tokens_per_request, num_heads_q, num_heads_kv,
                              head_dim, page_size, (int)table_width);
  if (need > 0 && !workspace) return KVQ_ERR_NULL;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(page_table, 4) || !aligned(lens, 4) ||
      !aligned(out, 16) || !aligned(error_count, 4) || (need > 0 && !aligned(workspace, 16)))
    return KVQ_ERR_ALIGN;
  if (workspace_bytes < need) return KVQ_ERR_SHAPE;
  const int64_t q_bytes = ((num_tokens - 1) * q_stride + (int64_t)num_heads_q * head_dim) * 2;
  if (overlap(q, q_bytes, out, num_tokens * num_heads_q * head_dim * 2)) return KVQ_ERR_VALUE;
  kvq::Kv4AttnArgs a;
  a.x.q = q;
  a.x.q_stride = q_stride;
  a.x.num_tokens = (int)num_tokens;
  a.x.num_heads_q = num_heads_q;
  a.x.num_heads_kv = num_heads_kv;
  a.x.head_dim = head_dim;
  a.x.num_pages = num_pages;
  a.x.page_size = page_size;
  a.x.page_table = page_table;
  a.x.num_requests = (int)(num_tokens / tokens_per_request);
  a.x.table_width = (int)table_width;
  a.x.requests = nullptr;
  a.x.lens = lens;
  a.x.errors = error_count;
  a.kv_cache = kv_cache;
  a.per_request = (int)tokens_per_request;
  a.scale = scale;
  a.out = out;
  a.workspace = workspace;
  return report_launch(kvq::launch_kv4_attn(a, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t dsv4_latent_attention_workspace(int64_t num_tokens, int num_heads, int64_t list_width) {
  if (num_tokens < 1 || num_tokens >= kIndexLimit || num_heads < 1 || num_heads > kMaxHeads ||
      num_tokens * num_heads >= kIndexLimit || list_width < 0 || list_width > kMaxEntries)
    return 0;
  return kvq::latent_attn_workspace(num_tokens, num_heads, (int)list_width);
}

kvq_status dsv4_latent_attention(const void* q, int64_t q_stride, int64_t num_tokens,
                                 int num_heads, const uint8_t* kv_cache, int64_t num_blocks,
                                 int block_size, const int32_t* slots, int64_t list_width,
                                 const int32_t* lens, float scale, void* out, void* workspace,
                                 int64_t workspace_bytes, int32_t* error_count,
                                 kvq_stream_t stream) {
  const kvq_status c = check_rows(num_tokens, num_heads, q_stride, kvq::dsv4::kDim);
  if (c != KVQ_OK) return c;
  if (num_blocks < 0 || num_blocks >= kIndexLimit || block_size < 1 || list_width < 0 ||
      list_width > kMaxEntries)
    return KVQ_ERR_SHAPE;
  if (!scale_ok(scale)) return KVQ_ERR_VALUE;
  if (num_tokens == 0) return KVQ_OK;
  if (!q || !kv_cache || !lens || !out || (list_width > 0 && !slots)) return KVQ_ERR_NULL;
  const int64_t need = kvq::latent_attn_workspace(num_tokens, num_heads, (int)list_width);
  if (need > 0 && !workspace) return KVQ_ERR_NULL;
  if (!aligned(q, 16) || !aligned(kv_cache, 8) || !aligned(slots, 4) || !aligned(lens, 4) ||
      !aligned(out, 16) || !aligned(error_count, 4) || (need > 0 && !aligned(workspace, 16)))
    return KVQ_ERR_ALIGN;
  if (workspace_bytes < need) return KVQ_ERR_SHAPE;
  const int64_t row = (int64_t)num_heads * kvq::dsv4::kDim;
  if (overlap(q, ((num_tokens - 1) * q_stride + row) * 2, out, num_tokens * row * 2))
    return KVQ_ERR_VALUE;
  kvq::LatentAttnArgs a;
  a.q = q;
  a.q_stride = q_stride;
  a.num_tokens = (int)num_tokens;
  a.num_heads = num_heads;
  a.kv_cache = kv_cache;
  a.num_slots = num_blocks * block_size;
  a.slots = slots;
  a.list_width = (int)list_width;
  a.lens = lens;
  a.scale = scale;
  a.out = out;
  a.workspace = workspace;
  a.errors = error_count;
  return report_launch(kvq::launch_latent_attn(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
