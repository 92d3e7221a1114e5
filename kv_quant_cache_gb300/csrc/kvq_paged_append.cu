// kvq_paged_append.cu -- the cache side of grouped-query attention: keys and
// values of new tokens into the paged cache with the rotary embedding applied
// on the way (the query heads rotated in the same pass), and the per-page
// bounds of the keys that the block selection reads.
//
// Append.  A row (one head of one token) of D dims is D/16 lanes of two
// 16-byte fragments.  For NeoX pairs the fragments of a rotated lane are the
// two halves of its pairs (dims 8l.. and 8l + rot/2..), otherwise adjacent;
// either way the partner is in the same lane and no shuffle is needed:
//   out_a = x_a cos - x_b sin,   out_b = x_b cos + x_a sin     (fp32)
// rounded once to bf16.  A warp takes STEPS groups of 32/(D/16) rows of one
// token; its cos/sin values are loaded once for all of them, and all its row
// loads are in flight before any is used.  V rows and rows past rotary_dim
// pass through unchanged.  Memory bound: every row is read once and written
// once; 32768 tokens x (32 + 2 x 8) heads of 128, 823 MB: 119-122 us,
// 6.8 TB/s, the rate of a plain copy.
//
// Bounds.  One warp per (page, kv head): the head's keys of a page are
// contiguous, so a warp reads 512 bytes a step and keeps 8 running minima and
// maxima a lane in packed bf16 (exact: the result is one of the keys; NaN
// propagates), then joins the lanes that hold the same dims.  Memory bound:
// 8192 pages x 8 heads x 64 keys of 128, 1.1 GB: 157 us, 7.0 TB/s (reads
// alone run a little above the rate of a copy); 64 pages: 3.8 us, three
// dependent latencies.
#include "kvq_device.cuh"
#include "kvq_paged.h"

namespace kvq {
namespace {

constexpr int kWarps = 4;

struct AppendParams {
  __nv_bfloat16* qkv;
  __nv_bfloat16* q_out;
  const float* cos_sin;
  const int64_t* positions;
  const int64_t* slots;
  __nv_bfloat16* cache;
  int num_q, num_kv, num_rows, first_row;
  int rot;
  int chunks, chunk_rows;  // warps per token, rows each of them takes
  int64_t items;
  int64_t max_pos, num_slots;
  int page_size;
  int64_t q_token_stride;  // elements between tokens of q_out
  int* errors;
  int trigger_from;
};

template <int D, bool NEOX, int STEPS>
__global__ void __launch_bounds__(kWarps * 32)
paged_append_kernel(const AppendParams p) {
  constexpr int LPR = D / 16;    // lanes per row
  constexpr int RPW = 32 / LPR;  // rows per warp step
  grid_dependency_sync(p.trigger_from);
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (item >= p.items) return;
  const int lane = threadIdx.x & 31;
  const int l = lane % LPR;
  const int64_t t = item / p.chunks;
  const int chunk = (int)(item - t * p.chunks);
  const int r0 = p.first_row + chunk * p.chunk_rows;
  const int r1 = min(r0 + p.chunk_rows, p.num_rows);
  const int64_t slot = __ldg(p.slots + t);
  const int64_t pos = p.rot ? __ldg(p.positions + t) : 0;

  // the lane's two fragments: NeoX pair halves while rotated, else adjacent
  const bool rotated = 16 * l < p.rot;
  const bool halves = NEOX && rotated;
  const int oa = halves ? 8 * l : 16 * l;
  const int ob = halves ? 8 * l + (p.rot >> 1) : 16 * l + 8;

  const __nv_bfloat16* src = p.qkv + t * (int64_t)p.num_rows * D;
  uint4 xa[STEPS], xb[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int r = r0 + s * RPW + lane / LPR;
    if (r < r1) {
      xa[s] = load_stream(src + (size_t)r * D + oa);
      xb[s] = load_stream(src + (size_t)r * D + ob);
    }
  }
  if (p.rot && (pos < 0 || pos >= p.max_pos)) {  // warp-uniform: leave the token as it is
    if (p.errors && chunk == 0 && lane == 0) atomicAdd(p.errors, 1);
    return;
  }
  const bool bad_slot = slot < -1 || slot >= p.num_slots;
  if (bad_slot && p.errors && chunk == 0 && lane == 0) atomicAdd(p.errors, 1);
  const bool store_kv = slot >= 0 && !bad_slot;
  float cs[8], sn[8];
  if (rotated) {
    // frequencies of the pairs: NeoX 8l..8l+7 (8 pairs over both fragments);
    // GPT-J 8l..8l+3 in the first fragment and 8l+4..8l+7 in the second
    const float* row = p.cos_sin + pos * p.rot + 8 * l;
    const float4 c0 = __ldg(reinterpret_cast<const float4*>(row));
    const float4 c1 = __ldg(reinterpret_cast<const float4*>(row + 4));
    const float4 s0 = __ldg(reinterpret_cast<const float4*>(row + (p.rot >> 1)));
    const float4 s1 = __ldg(reinterpret_cast<const float4*>(row + (p.rot >> 1) + 4));
    cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w;
    cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
    sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w;
    sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
  }
  int64_t kv_row = 0;  // first cache row of the token: head 0 of the page's keys
  if (store_kv) {
    const int64_t page = slot / p.page_size;
    kv_row = page * 2 * p.num_kv * p.page_size + (slot - page * p.page_size);
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int r = r0 + s * RPW + lane / LPR;
    if (r >= r1) continue;
    if (rotated && r < p.num_q + p.num_kv) {
      float a[8], b[8];
      unpack_bf16x8(xa[s], a);
      unpack_bf16x8(xb[s], b);
      if (NEOX) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float u = a[i], v = b[i];
          a[i] = fmaf(-v, sn[i], u * cs[i]);
          b[i] = fmaf(u, sn[i], v * cs[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float u = a[2 * i], v = a[2 * i + 1];
          a[2 * i] = fmaf(-v, sn[i], u * cs[i]);
          a[2 * i + 1] = fmaf(u, sn[i], v * cs[i]);
          const float w = b[2 * i], z = b[2 * i + 1];
          b[2 * i] = fmaf(-z, sn[4 + i], w * cs[4 + i]);
          b[2 * i + 1] = fmaf(w, sn[4 + i], z * cs[4 + i]);
        }
      }
      xa[s] = pack_bf16x8(a);
      xb[s] = pack_bf16x8(b);
    }
    __nv_bfloat16* dst;
    if (r < p.num_q) {
      dst = p.q_out + t * p.q_token_stride + (size_t)r * D;
    } else {
      if (!store_kv) continue;
      // key heads, then value heads, as the page holds them
      dst = p.cache + (kv_row + (int64_t)(r - p.num_q) * p.page_size) * D;
    }
    // evict first: 32768 tokens 120 us, with plain stores 124 us
    store_stream(dst + oa, xa[s]);
    store_stream(dst + ob, xb[s]);
  }
}

template <int D, bool NEOX, int STEPS>
cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream) {
  constexpr int RPW = 32 / (D / 16);
  AppendParams p;
  p.qkv = static_cast<__nv_bfloat16*>(a.qkv);
  p.q_out = static_cast<__nv_bfloat16*>(a.q_out);
  p.cos_sin = a.cos_sin;
  p.positions = a.positions;
  p.slots = a.slot_mapping;
  p.cache = static_cast<__nv_bfloat16*>(a.kv_cache);
  p.num_q = a.num_heads_q;
  p.num_kv = a.num_heads_kv;
  p.num_rows = a.num_heads_q + 2 * a.num_heads_kv;
  const bool in_place = a.q_out == a.qkv;
  // in place without a rotation the query rows stay as they are
  p.first_row = in_place && a.rotary_dim == 0 ? a.num_heads_q : 0;
  p.q_token_stride = (int64_t)(in_place ? p.num_rows : p.num_q) * D;
  p.rot = a.rotary_dim;
  p.max_pos = a.max_pos;
  p.num_slots = a.num_pages * a.page_size;
  p.page_size = a.page_size;
  p.errors = a.errors;
  const int rows = p.num_rows - p.first_row;
  const int groups = (rows + RPW - 1) / RPW;
  p.chunks = (groups + STEPS - 1) / STEPS;
  p.chunk_rows = (groups + p.chunks - 1) / p.chunks * RPW;
  p.items = (int64_t)a.num_tokens * p.chunks;
  if (p.items == 0) return cudaSuccess;
  const int64_t grid = (p.items + kWarps - 1) / kWarps;
  static std::atomic<int> cache[kMaxDevices];
  const auto kernel = paged_append_kernel<D, NEOX, STEPS>;
  p.trigger_from = last_wave_start(kernel, kWarps * 32, grid, cache);
  return launch_kernel(kernel, dim3((unsigned)grid), dim3(kWarps * 32), 0, stream, p);
}

template <int D, bool NEOX>
cudaError_t append_shape(const AppendArgs& a, cudaStream_t stream) {
  // Rows of one warp: a decode step is spread as wide as it goes (17 tokens:
  // 2.5 us against 2.6 us); from about one warp step for every resident warp
  // of a quarter of the GPU on, three steps a warp keep six loads a lane in
  // flight (32768 tokens x 48 heads: 120 us, 1 step 142 us, 2 steps 121 us,
  // 4 steps 120 us; 32768 x 20 heads of 64: 27, 36, 33 and 30 us).
  const int64_t rows = (int64_t)a.num_tokens * (a.num_heads_q + 2 * a.num_heads_kv);
  return rows < 152 * 32 ? launch_append<D, NEOX, 1>(a, stream)
                         : launch_append<D, NEOX, 3>(a, stream);
}

template <int D>
cudaError_t append_dim(const AppendArgs& a, cudaStream_t stream) {
  return a.is_neox ? append_shape<D, true>(a, stream) : append_shape<D, false>(a, stream);
}

// ---- page bounds ---------------------------------------------------------------

struct BoundsParams {
  const __nv_bfloat16* cache;
  const int64_t* pages;
  const int* lens;
  __nv_bfloat16* bounds;
  int num_kv, page_size;
  int64_t num_pages, items;
  int* errors;
  int trigger_from;
};

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ void take(uint32_t lo[4], uint32_t hi[4], const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    lo[k] = min2(lo[k], w[k]);
    hi[k] = max2(hi[k], w[k]);
  }
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) page_bounds_kernel(const BoundsParams p) {
  constexpr int LPR = D / 8;     // lanes per key
  constexpr int KPW = 32 / LPR;  // keys per warp step
  constexpr int UNROLL = 8;
  grid_dependency_sync(p.trigger_from);
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (item >= p.items) return;
  const int lane = threadIdx.x & 31;
  const int64_t i = item / p.num_kv;
  const int h = (int)(item - i * p.num_kv);
  const int64_t page = __ldg(p.pages + i);
  const int len = __ldg(p.lens + i);
  const bool none = page == -1 || len == 0;
  if (page < -1 || page >= p.num_pages || len < 0 || len > p.page_size) {
    if (p.errors && h == 0 && lane == 0) atomicAdd(p.errors, 1);
    return;
  }
  if (none) return;
  const __nv_bfloat16* keys =
      p.cache + (page * 2 * p.num_kv + h) * (int64_t)p.page_size * D + 8 * (lane % LPR);
  uint32_t lo[4], hi[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) lo[k] = 0x7f807f80u, hi[k] = 0xff80ff80u;  // +inf, -inf
  for (int r = lane / LPR; r < len; r += KPW * UNROLL) {
    uint4 v[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      v[u] = __ldg(reinterpret_cast<const uint4*>(
          keys + (size_t)min(r + u * KPW, len - 1) * D));  // past the end: the last key again
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) take(lo, hi, v[u]);
  }
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      lo[k] = min2(lo[k], __shfl_xor_sync(kFullMask, lo[k], o));
      hi[k] = max2(hi[k], __shfl_xor_sync(kFullMask, hi[k], o));
    }
  }
  if (lane < LPR) {
    __nv_bfloat16* out = p.bounds + (page * p.num_kv + h) * 2 * D + 8 * lane;
    *reinterpret_cast<uint4*>(out) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<uint4*>(out + D) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
}

template <int D>
cudaError_t launch_bounds(const PageBoundsArgs& a, cudaStream_t stream) {
  BoundsParams p;
  p.cache = static_cast<const __nv_bfloat16*>(a.kv_cache);
  p.pages = a.pages;
  p.lens = a.lens;
  p.bounds = static_cast<__nv_bfloat16*>(a.bounds);
  p.num_kv = a.num_heads_kv;
  p.page_size = a.page_size;
  p.num_pages = a.num_pages;
  p.items = (int64_t)a.num_listed * a.num_heads_kv;
  p.errors = a.errors;
  const int64_t grid = (p.items + kWarps - 1) / kWarps;
  static std::atomic<int> cache[kMaxDevices];
  p.trigger_from = last_wave_start(page_bounds_kernel<D>, kWarps * 32, grid, cache);
  return launch_kernel(page_bounds_kernel<D>, dim3((unsigned)grid), dim3(kWarps * 32), 0, stream,
                       p);
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 64: return append_dim<64>(a, stream);
    case 128: return append_dim<128>(a, stream);
    case 256: return append_dim<256>(a, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_page_bounds(const PageBoundsArgs& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 64: return launch_bounds<64>(a, stream);
    case 128: return launch_bounds<128>(a, stream);
    case 256: return launch_bounds<256>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kvq
