// kvq_paged_api.cu -- the C ABI of the paged grouped-query operators
// (include/kvq.h): host-side validation and launch on the caller's stream.
// No allocation, no sync.
#include <climits>
#include <cmath>

#include "kvq.h"
#include "kvq_launch.h"
#include "kvq_paged.h"

namespace {

using kvq::report_launch;

constexpr int64_t kIndexLimit = (int64_t)1 << 31;
constexpr int kMaxPageSize = 1 << 16;
constexpr int kMaxHeads = 1 << 16;
constexpr int64_t kMaxListed = 1 << 22;  // pages of a request, a prefix or a selection

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

bool prefix_ok(int64_t prefix_len, int page_size) {
  return prefix_len >= 0 && prefix_len < kIndexLimit &&
         (prefix_len + page_size - 1) / page_size <= kMaxListed;
}

// The kernels take the scale in units of log2: infinite there, it would make
// NaN of a score of zero.
bool scale_ok(float scale) { return std::isfinite(scale * 1.4426950408889634f); }

// Sizes that every operator takes.
kvq_status check_cache(int num_heads_kv, int head_dim, int64_t num_pages, int page_size) {
  if (num_heads_kv < 1 || num_heads_kv > kMaxHeads || num_pages < 0 ||
      num_pages > (int64_t)INT_MAX || page_size < 1 || page_size > kMaxPageSize)
    return KVQ_ERR_SHAPE;
  return head_dim_ok(head_dim) ? KVQ_OK : KVQ_ERR_UNSUPPORTED;
}

kvq_status check_query(int64_t num_tokens, int num_heads_q, int num_heads_kv, int64_t q_stride,
                       int head_dim, int64_t num_requests, int64_t table_width) {
  if (num_tokens < 0 || num_heads_q < 1 || num_heads_q > kMaxHeads ||
      num_heads_q % num_heads_kv != 0)
    return KVQ_ERR_SHAPE;
  // CTAs, rows of partials and table entries are counted in 32 bits
  if (num_tokens >= kIndexLimit || num_tokens * num_heads_q >= kIndexLimit ||
      num_requests < 0 || num_requests >= kIndexLimit || table_width < 0 ||
      table_width > kMaxListed)
    return KVQ_ERR_SHAPE;
  if (q_stride < (int64_t)num_heads_q * head_dim || q_stride >= kIndexLimit)
    return KVQ_ERR_SHAPE;
  return q_stride % 8 == 0 ? KVQ_OK : KVQ_ERR_ALIGN;
}

// The request arrays of a call with tokens; NULL `requests` stands for the
// tokens' own indices.
kvq_status check_requests(const void* q, const void* kv_cache, const int32_t* page_table,
                          int64_t num_requests, int64_t table_width, const int32_t* requests,
                          const int32_t* lens, int64_t num_tokens, const int32_t* errors) {
  if (!q || !kv_cache || !lens) return KVQ_ERR_NULL;
  if (!page_table && num_requests * table_width > 0) return KVQ_ERR_NULL;
  if (!requests && num_requests < num_tokens) return KVQ_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(page_table, 4) ||
      !aligned(requests, 4) || !aligned(lens, 4) || !aligned(errors, 4))
    return KVQ_ERR_ALIGN;
  return KVQ_OK;
}

bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}

kvq::PagedQuery query(const void* q, int64_t q_stride, int64_t num_tokens, int num_heads_q,
                      int num_heads_kv, int head_dim, int64_t num_pages, int page_size,
                      const int32_t* page_table, int64_t num_requests, int64_t table_width,
                      const int32_t* requests, const int32_t* lens, int32_t* errors) {
  kvq::PagedQuery x;
  x.q = q;
  x.q_stride = q_stride;
  x.num_tokens = (int)num_tokens;
  x.num_heads_q = num_heads_q;
  x.num_heads_kv = num_heads_kv;
  x.head_dim = head_dim;
  x.num_pages = num_pages;
  x.page_size = page_size;
  x.page_table = page_table;
  x.num_requests = (int)num_requests;
  x.table_width = (int)table_width;
  x.requests = requests;
  x.lens = lens;
  x.errors = errors;
  return x;
}

}  // namespace

extern "C" {

kvq_status paged_kv_rope_append(void* qkv, void* q_out, int64_t num_tokens, int num_heads_q,
                                int num_heads_kv, int head_dim, const float* cos_sin_cache,
                                int64_t max_pos, int rotary_dim, int is_neox,
                                const int64_t* positions, const int64_t* slot_mapping,
                                void* kv_cache, int64_t num_pages, int page_size,
                                int32_t* error_count, kvq_stream_t stream) {
  kvq_status c = check_cache(num_heads_kv, head_dim, num_pages, page_size);
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
  return report_launch(kvq::launch_paged_append(a, reinterpret_cast<cudaStream_t>(stream)));
}

kvq_status paged_kv_page_bounds(const void* kv_cache, int64_t num_pages, int num_heads_kv,
                                int page_size, int head_dim, const int64_t* pages,
                                const int32_t* lens, int64_t num_listed, void* bounds,
                                int32_t* error_count, kvq_stream_t stream) {
  const kvq_status c = check_cache(num_heads_kv, head_dim, num_pages, page_size);
  if (c != KVQ_OK) return c;
  if (num_listed < 0 || num_listed >= kIndexLimit || num_listed * num_heads_kv >= kIndexLimit)
    return KVQ_ERR_SHAPE;
  if (num_listed == 0) return KVQ_OK;
  if (!kv_cache || !pages || !lens || !bounds) return KVQ_ERR_NULL;
  if (!aligned(kv_cache, 16) || !aligned(pages, 8) || !aligned(lens, 4) || !aligned(bounds, 16) ||
      !aligned(error_count, 4))
    return KVQ_ERR_ALIGN;
  kvq::PageBoundsArgs a;
  a.kv_cache = kv_cache;
  a.pages = pages;
  a.lens = lens;
  a.bounds = bounds;
  a.num_listed = (int)num_listed;
  a.num_heads_kv = num_heads_kv;
  a.head_dim = head_dim;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.errors = error_count;
  return report_launch(kvq::launch_page_bounds(a, reinterpret_cast<cudaStream_t>(stream)));
}

kvq_status paged_kv_block_select(const void* q, int64_t q_stride, int64_t num_tokens,
                                 int num_heads_q, int num_heads_kv, int head_dim,
                                 const void* bounds, int64_t num_pages, int page_size,
                                 const int32_t* page_table, int64_t num_requests,
                                 int64_t table_width, const int32_t* requests,
                                 const int32_t* lens, int topk, int keep_first, int keep_last,
                                 int32_t* blocks, int32_t* error_count, kvq_stream_t stream) {
  kvq_status c = check_cache(num_heads_kv, head_dim, num_pages, page_size);
  if (c == KVQ_OK)
    c = check_query(num_tokens, num_heads_q, num_heads_kv, q_stride, head_dim, num_requests,
                    table_width);
  if (c != KVQ_OK) return c;
  if (topk < 1 || topk > kMaxListed || keep_first < 0 || keep_last < 0) return KVQ_ERR_SHAPE;
  if (table_width > kvq::kMaxSelectBlocks) return KVQ_ERR_UNSUPPORTED;
  if (num_tokens * num_heads_kv * 8 >= kIndexLimit) return KVQ_ERR_SHAPE;  // CTAs of the grid
  if (num_tokens == 0) return KVQ_OK;
  c = check_requests(q, bounds, page_table, num_requests, table_width, requests, lens, num_tokens,
                     error_count);
  if (c != KVQ_OK) return c;
  if (!blocks) return KVQ_ERR_NULL;
  if (!aligned(blocks, 4)) return KVQ_ERR_ALIGN;
  kvq::BlockSelectArgs a;
  a.x = query(q, q_stride, num_tokens, num_heads_q, num_heads_kv, head_dim, num_pages, page_size,
              page_table, num_requests, table_width, requests, lens, error_count);
  a.bounds = bounds;
  a.topk = topk;
  a.keep_first = keep_first;
  a.keep_last = keep_last;
  a.blocks = blocks;
  return report_launch(kvq::launch_block_select(a, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t paged_block_sparse_attention_workspace(int64_t num_tokens, int num_heads_q,
                                               int num_heads_kv, int head_dim, int page_size,
                                               int topk) {
  if (num_tokens < 1 || num_heads_kv < 1 || num_heads_q < 1 || num_heads_q > kMaxHeads ||
      num_heads_q % num_heads_kv != 0 || !head_dim_ok(head_dim) || page_size < 1 ||
      page_size > kMaxPageSize || topk < 1 || topk > kMaxListed || num_tokens >= kIndexLimit ||
      num_tokens * num_heads_q >= kIndexLimit)
    return 0;
  return kvq::sparse_attn_workspace(num_tokens, num_heads_q, num_heads_kv, head_dim, page_size,
                                    topk);
}

kvq_status paged_block_sparse_attention(const void* q, int64_t q_stride, int64_t num_tokens,
                                        int num_heads_q, int num_heads_kv, int head_dim,
                                        const void* kv_cache, int64_t num_pages, int page_size,
                                        const int32_t* page_table, int64_t num_requests,
                                        int64_t table_width, const int32_t* requests,
                                        const int32_t* lens, const int32_t* blocks, int topk,
                                        float scale, void* out, void* workspace,
                                        int64_t workspace_bytes, int32_t* error_count,
                                        kvq_stream_t stream) {
  kvq_status c = check_cache(num_heads_kv, head_dim, num_pages, page_size);
  if (c == KVQ_OK)
    c = check_query(num_tokens, num_heads_q, num_heads_kv, q_stride, head_dim, num_requests,
                    table_width);
  if (c != KVQ_OK) return c;
  if (topk < 1 || topk > kMaxListed) return KVQ_ERR_SHAPE;
  if (!scale_ok(scale)) return KVQ_ERR_VALUE;
  if (num_tokens == 0) return KVQ_OK;
  c = check_requests(q, kv_cache, page_table, num_requests, table_width, requests, lens,
                     num_tokens, error_count);
  if (c != KVQ_OK) return c;
  const int64_t need = kvq::sparse_attn_workspace(num_tokens, num_heads_q, num_heads_kv, head_dim,
                                                  page_size, topk);
  if (!blocks || !out || (need > 0 && !workspace)) return KVQ_ERR_NULL;
  if (!aligned(blocks, 4) || !aligned(out, 16) || (need > 0 && !aligned(workspace, 16)))
    return KVQ_ERR_ALIGN;
  if (workspace_bytes < need) return KVQ_ERR_SHAPE;
  const int64_t q_bytes = ((num_tokens - 1) * q_stride + (int64_t)num_heads_q * head_dim) * 2;
  const int64_t out_bytes = num_tokens * num_heads_q * head_dim * 2;
  if (overlap(q, q_bytes, out, out_bytes)) return KVQ_ERR_VALUE;
  kvq::SparseAttnArgs a;
  a.x = query(q, q_stride, num_tokens, num_heads_q, num_heads_kv, head_dim, num_pages, page_size,
              page_table, num_requests, table_width, requests, lens, error_count);
  a.kv_cache = kv_cache;
  a.blocks = blocks;
  a.topk = topk;
  a.scale = scale;
  a.out = out;
  a.workspace = workspace;
  return report_launch(kvq::launch_sparse_attn(a, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t paged_shared_prefix_attention_workspace(int64_t num_tokens, int num_heads_q,
                                                int num_heads_kv, int head_dim, int page_size,
                                                int64_t prefix_len, int64_t table_width) {
  if (num_tokens < 1 || num_heads_kv < 1 || num_heads_q < 1 || num_heads_q > kMaxHeads ||
      num_heads_q % num_heads_kv != 0 || !head_dim_ok(head_dim) || page_size < 1 ||
      page_size > kMaxPageSize || !prefix_ok(prefix_len, page_size) || table_width < 0 ||
      table_width > kMaxListed || num_tokens >= kIndexLimit ||
      num_tokens * num_heads_q >= kIndexLimit)
    return 0;
  return kvq::prefix_attn_workspace(num_tokens, num_heads_q, num_heads_kv, head_dim, page_size,
                                    prefix_len, (int)table_width, kvq::prefix_config());
}

kvq_status paged_shared_prefix_attention(const void* q, int64_t q_stride, int64_t num_tokens,
                                         int num_heads_q, int num_heads_kv, int head_dim,
                                         const void* kv_cache, int64_t num_pages, int page_size,
                                         const int32_t* prefix_pages, int64_t prefix_len,
                                         const int32_t* page_table, int64_t num_requests,
                                         int64_t table_width, const int32_t* requests,
                                         const int32_t* lens, float scale, void* out,
                                         void* workspace, int64_t workspace_bytes,
                                         int32_t* error_count, kvq_stream_t stream) {
  kvq_status c = check_cache(num_heads_kv, head_dim, num_pages, page_size);
  if (c == KVQ_OK)
    c = check_query(num_tokens, num_heads_q, num_heads_kv, q_stride, head_dim, num_requests,
                    table_width);
  if (c != KVQ_OK) return c;
  if (!prefix_ok(prefix_len, page_size)) return KVQ_ERR_SHAPE;
  if (!scale_ok(scale)) return KVQ_ERR_VALUE;
  if (num_tokens == 0) return KVQ_OK;
  c = check_requests(q, kv_cache, page_table, num_requests, table_width, requests, lens,
                     num_tokens, error_count);
  if (c != KVQ_OK) return c;
  const int config = kvq::prefix_config();
  const int64_t need = kvq::prefix_attn_workspace(num_tokens, num_heads_q, num_heads_kv, head_dim,
                                                  page_size, prefix_len, (int)table_width, config);
  if (!out || (prefix_len > 0 && !prefix_pages) || (need > 0 && !workspace)) return KVQ_ERR_NULL;
  if (!aligned(prefix_pages, 4) || !aligned(out, 16) || (need > 0 && !aligned(workspace, 16)))
    return KVQ_ERR_ALIGN;
  if (workspace_bytes < need) return KVQ_ERR_SHAPE;
  const int64_t q_bytes = ((num_tokens - 1) * q_stride + (int64_t)num_heads_q * head_dim) * 2;
  const int64_t out_bytes = num_tokens * num_heads_q * head_dim * 2;
  if (overlap(q, q_bytes, out, out_bytes)) return KVQ_ERR_VALUE;
  kvq::PrefixAttnArgs a;
  a.x = query(q, q_stride, num_tokens, num_heads_q, num_heads_kv, head_dim, num_pages, page_size,
              page_table, num_requests, table_width, requests, lens, error_count);
  a.kv_cache = kv_cache;
  a.prefix_pages = prefix_pages;
  a.prefix_len = prefix_len;
  a.config = config;
  a.scale = scale;
  a.out = out;
  a.workspace = workspace;
  return report_launch(kvq::launch_prefix_attn(a, reinterpret_cast<cudaStream_t>(stream)));
}

int kvq_prefix_num_configs(void) { return kvq::kPrefixNumConfigs; }

const char* kvq_prefix_config_name(int id) {
  return (id >= 0 && id < kvq::kPrefixNumConfigs) ? kvq::kPrefixConfigs[id].name : nullptr;
}

int kvq_set_prefix_config(int id) {
  if (id >= kvq::kPrefixNumConfigs) return -2;
  return kvq::set_prefix_config(id < 0 ? -1 : id);
}

uint32_t kvq_set_tile_wait_limit(uint32_t polls) { return kvq::set_tile_wait_limit(polls); }

}  // extern "C"
