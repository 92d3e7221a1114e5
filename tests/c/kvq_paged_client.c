/*
 * kvq_paged_client.c -- a plain C99 caller of the paged grouped-query
 * operators (include/kvq.h), on a case whose results are exact by
 * construction:
 *
 *   append:    T tokens, rotation by position 0 (cos 1, sin 0): keys, values
 *              and query rows come out bit for bit; one token without a slot.
 *   bounds:    the keys of token t are all t + 1: a page's bounds are the
 *              smallest and largest t + 1 of its tokens.
 *   selection: positive queries rank the pages by their largest key.
 *   attention: zero queries weigh every key 1, all values are 2: the output
 *              is 2, over the selected blocks as over the shared prefix; a
 *              token without keys gets zeros.
 *
 * Exit status 0 when every check holds.
 */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <cuda_runtime.h>

#include "kvq.h"

static int failures = 0;

#define CHECK(cond, ...)                     \
  do {                                       \
    if (!(cond)) {                           \
      fprintf(stderr, "FAIL: " __VA_ARGS__); \
      fprintf(stderr, "\n");                 \
      ++failures;                            \
    }                                        \
  } while (0)

#define CUDA(call)                                                        \
  do {                                                                    \
    cudaError_t e_ = (call);                                              \
    if (e_ != cudaSuccess) {                                              \
      fprintf(stderr, "CUDA error %s at %s:%d\n", cudaGetErrorString(e_), \
              __FILE__, __LINE__);                                        \
      exit(2);                                                            \
    }                                                                     \
  } while (0)

enum { T = 11, HQ = 4, HKV = 2, D = 64, PAGE = 4, PAGES = 4, TOPK = 2, ROWS = HQ + 2 * HKV };
#define ONE 0x3F80u
#define TWO 0x4000u

static void* dev_copy(const void* host, size_t bytes) {
  void* d = NULL;
  CUDA(cudaMalloc(&d, bytes));
  CUDA(cudaMemcpy(d, host, bytes, cudaMemcpyHostToDevice));
  return d;
}

static void* dev_fill(size_t bytes, int byte) {
  void* d = NULL;
  CUDA(cudaMalloc(&d, bytes));
  CUDA(cudaMemset(d, byte, bytes));
  return d;
}

/* bf16 of a small whole number (exact). */
static uint16_t bf16(float v) {
  uint32_t u;
  memcpy(&u, &v, 4);
  return (uint16_t)(u >> 16);
}

int main(void) {
  uint16_t qkv[T * ROWS * D];
  int64_t pos[T], slots[T], all_pages[PAGES];
  float table[2 * D];
  for (int t = 0; t < T; ++t) {
    pos[t] = 0;
    slots[t] = t == 5 ? -1 : t;
    for (int r = 0; r < ROWS; ++r)
      for (int d = 0; d < D; ++d)
        qkv[(t * ROWS + r) * D + d] =
            r < HQ ? ONE : r < HQ + HKV ? bf16((float)(t + 1)) : TWO;
  }
  for (int d = 0; d < 2 * D; ++d) table[d] = d < D / 2 ? 1.0f : 0.0f;
  for (int i = 0; i < PAGES; ++i) all_pages[i] = i;

  const size_t cache_values = (size_t)PAGES * 2 * HKV * PAGE * D;
  void* d_qkv = dev_copy(qkv, sizeof qkv);
  void* d_q = dev_fill(sizeof(uint16_t) * T * HQ * D, 0xA5);
  float* d_table = (float*)dev_copy(table, sizeof table);
  int64_t* d_pos = (int64_t*)dev_copy(pos, sizeof pos);
  int64_t* d_slots = (int64_t*)dev_copy(slots, sizeof slots);
  void* d_cache = dev_fill(cache_values * 2, 0);
  int32_t* d_err = (int32_t*)dev_fill(4, 0);
  kvq_status s = paged_kv_rope_append(d_qkv, d_q, T, HQ, HKV, D, d_table, 2, D, 1, d_pos, d_slots,
                                      d_cache, PAGES, PAGE, d_err, NULL);
  CHECK(s == KVQ_OK, "append: %s", kvq_status_string(s));
  uint16_t q[T * HQ * D], *cache = (uint16_t*)malloc(cache_values * 2);
  CUDA(cudaMemcpy(q, d_q, sizeof q, cudaMemcpyDeviceToHost));
  CUDA(cudaMemcpy(cache, d_cache, cache_values * 2, cudaMemcpyDeviceToHost));
  int bad = 0;
  for (int i = 0; i < T * HQ * D; ++i) bad += q[i] != ONE;
  for (int p = 0; p < PAGES; ++p)
    for (int kv = 0; kv < 2; ++kv)
      for (int h = 0; h < HKV; ++h)
        for (int o = 0; o < PAGE; ++o)
          for (int d = 0; d < D; ++d) {
            const int t = p * PAGE + o, there = t < T && t != 5;
            const uint16_t want = !there ? 0 : kv ? TWO : bf16((float)(t + 1));
            bad += cache[(((p * 2 + kv) * HKV + h) * PAGE + o) * D + d] != want;
          }
  CHECK(bad == 0, "append: %d values differ", bad);

  /* token 5 has no entry: its place (slot 5) still holds zeros */
  const int32_t fill[PAGES] = {4, 4, 3, 0};
  int32_t* d_fill = (int32_t*)dev_copy(fill, sizeof fill);
  int64_t* d_ids = (int64_t*)dev_copy(all_pages, sizeof all_pages);
  uint16_t bounds[PAGES * HKV * 2 * D];
  void* d_bounds = dev_fill(sizeof bounds, 0);
  s = paged_kv_page_bounds(d_cache, PAGES, HKV, PAGE, D, d_ids, d_fill, PAGES, d_bounds, d_err,
                           NULL);
  CHECK(s == KVQ_OK, "bounds: %s", kvq_status_string(s));
  CUDA(cudaMemcpy(bounds, d_bounds, sizeof bounds, cudaMemcpyDeviceToHost));
  const float lo[PAGES] = {1, 0, 9, 0}, hi[PAGES] = {4, 8, 11, 0};
  bad = 0;
  for (int p = 0; p < PAGES; ++p)
    for (int h = 0; h < HKV; ++h)
      for (int d = 0; d < D; ++d) {
        const uint16_t* b = bounds + (p * HKV + h) * 2 * D;
        bad += b[d] != bf16(lo[p]) || b[D + d] != bf16(hi[p]);
      }
  CHECK(bad == 0, "bounds: %d differ", bad);

  /* two tokens of one request: the first sees all keys, the second none */
  const int32_t pages[PAGES] = {0, 1, 2, 3}, lens[2] = {T, 0}, request[2] = {0, 0};
  int32_t* d_pages = (int32_t*)dev_copy(pages, sizeof pages);
  int32_t* d_lens = (int32_t*)dev_copy(lens, sizeof lens);
  int32_t* d_request = (int32_t*)dev_copy(request, sizeof request);
  int32_t blocks[2 * HKV * TOPK];
  int32_t* d_blocks = (int32_t*)dev_fill(sizeof blocks, 0x55);
  s = paged_kv_block_select(d_q, HQ * D, 2, HQ, HKV, D, d_bounds, PAGES, PAGE, d_pages, 1, PAGES,
                            d_request, d_lens, TOPK, 0, 0, d_blocks, d_err, NULL);
  CHECK(s == KVQ_OK, "select: %s", kvq_status_string(s));
  CUDA(cudaMemcpy(blocks, d_blocks, sizeof blocks, cudaMemcpyDeviceToHost));
  for (int h = 0; h < HKV; ++h) {
    CHECK(blocks[h * TOPK] == 1 && blocks[h * TOPK + 1] == 2, "select: head %d has %d, %d", h,
          blocks[h * TOPK], blocks[h * TOPK + 1]);
    CHECK(blocks[(HKV + h) * TOPK] == -1 && blocks[(HKV + h) * TOPK + 1] == -1,
          "select: a token without keys has blocks");
  }

  /* the selected blocks hold token 5's empty place too: fill its values */
  for (int h = 0; h < HKV; ++h)
    for (int d = 0; d < D; ++d) cache[(((1 * 2 + 1) * HKV + h) * PAGE + 1) * D + d] = TWO;
  CUDA(cudaMemcpy(d_cache, cache, cache_values * 2, cudaMemcpyHostToDevice));
  void* d_zero = dev_fill(sizeof(uint16_t) * 2 * HQ * D, 0);
  uint16_t out[2 * HQ * D];
  void* d_out = dev_fill(sizeof out, 0xA5);
  for (int which = 0; which < 2; ++which) {
    const int64_t need =
        which ? paged_shared_prefix_attention_workspace(2, HQ, HKV, D, PAGE, 7, PAGES)
              : paged_block_sparse_attention_workspace(2, HQ, HKV, D, PAGE, TOPK);
    void* ws = dev_fill((size_t)need + 16, 0xFF);
    CUDA(cudaMemset(d_out, 0xA5, sizeof out));
    s = which ? paged_shared_prefix_attention(d_zero, HQ * D, 2, HQ, HKV, D, d_cache, PAGES, PAGE,
                                              d_pages, 7, d_pages, 1, PAGES, d_request, d_lens,
                                              0.125f, d_out, ws, need, d_err, NULL)
              : paged_block_sparse_attention(d_zero, HQ * D, 2, HQ, HKV, D, d_cache, PAGES, PAGE,
                                             d_pages, 1, PAGES, d_request, d_lens, d_blocks, TOPK,
                                             0.125f, d_out, ws, need, d_err, NULL);
    CHECK(s == KVQ_OK, "attention %d: %s", which, kvq_status_string(s));
    CUDA(cudaMemcpy(out, d_out, sizeof out, cudaMemcpyDeviceToHost));
    bad = 0;
    for (int i = 0; i < 2 * HQ * D; ++i)
      bad += out[i] != (i < HQ * D || which ? TWO : 0); /* the second token has the prefix alone */
    CHECK(bad == 0, "attention %d: %d values differ", which, bad);
  }
  int32_t err = -1;
  CUDA(cudaMemcpy(&err, d_err, 4, cudaMemcpyDeviceToHost));
  CHECK(err == 0, "%d indices were rejected", err);

  /* host-side validation: nothing is launched on an error */
  CHECK(paged_kv_rope_append(d_qkv, d_qkv, T, HQ, HKV, D, NULL, 0, 0, 1, NULL, d_slots, d_cache,
                             PAGES, PAGE, NULL, NULL) == KVQ_ERR_VALUE, "q_out over qkv");
  CHECK(paged_block_sparse_attention(d_zero, HQ * D, 2, HQ, 3, D, d_cache, PAGES, PAGE, d_pages, 1,
                                     PAGES, d_request, d_lens, d_blocks, TOPK, 0.125f, d_out, NULL,
                                     0, NULL, NULL) == KVQ_ERR_SHAPE, "4 heads over 3");
  CUDA(cudaDeviceSynchronize());
  if (failures) return 1;
  printf("paged c client ok\n");
  return 0;
}
