// kvq_paged_attn.cu -- attention of few query rows over keys and values read
// from the paged cache: the selected blocks of block-sparse attention, the
// own keys of each token of shared-prefix attention, and the prefix itself
// where few rows share it.
//
// One CTA takes up to 16 query rows that see the same keys (the heads of one
// kv head's group) and one part of their key range.  It first lists the
// part's pages in shared memory ({page, valid keys}), so that no table lookup
// stands between a page and its loads.  Then each of its warps works alone,
// on every kWarps-th group of 16 keys, with an online softmax of its own:
//   * K and V rows of the group come in by 16-byte asynchronous copies,
//     kStages groups deep, into a shared-memory ring that only this warp
//     uses, so there is no CTA barrier in the loop; a 16-byte fragment c of
//     row r is stored at c ^ (r & 7), which keeps the matrix loads free of
//     bank conflicts;
//   * S = Q K^T and O += P V are 16x8x16 matrix instructions, fp32
//     accumulators; the P fragments are the S fragments, rounded once to
//     bf16 (the row sum adds the unrounded fp32 values);
//   * keys past a page's valid count are neither read nor weighted: their
//     rows are filled with zeros and their scores set to -inf.
// The warps' states are joined in shared memory at the end.  With one part
// per row the CTA writes the output, otherwise a partial for the join kernel.
//
// Bound by the reading of K and V: 16 rows of products per key row are a few
// per cent of the tensor pipes, which is why the small matrix instruction is
// enough here and one tile of 16 rows is as cheap as one row.
#include "kvq_paged_attn.cuh"
#include "kvq_tma.cuh"

namespace kvq {
namespace {

constexpr int kWarps = 4;
constexpr int kRows = 16;         // query rows of a CTA
constexpr int kGroup = 16;        // keys of one step of a warp
constexpr int kMaxPages = 2048;   // pages a CTA can list

enum KeySource { kSparse = 0, kOwn = 1, kPrefix = 2 };

struct AttnParams {
  const __nv_bfloat16* q;
  int64_t q_stride;
  const __nv_bfloat16* cache;
  int num_q, num_kv, group;  // group = num_q / num_kv
  int chunks;                // CTAs a group of heads takes (ceil(group / 16))
  int num_tokens;
  int64_t num_pages;
  int page_size;
  // kSparse, kOwn: the request's pages
  const int* table;
  int num_requests, table_width;
  const int* requests;
  const int* lens;
  // kSparse
  const int* blocks;
  int topk;
  // kPrefix
  const int* prefix_pages;
  int64_t prefix_len;
  int row_tiles;  // tiles of 16 rows of one kv head
  float scale_log2;
  int splits;
  int first_slot;      // partials slot of split 0
  Partials parts;      // used unless direct
  __nv_bfloat16* out;  // direct
  bool direct;
  int* errors;
  int trigger_from;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int bytes = valid ? 16 : 0;  // 0: the 16 bytes are filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(__cvta_generic_to_global(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
struct Shape {
  static constexpr int kStages = D == 256 ? 2 : 3;
  static constexpr int kTile = kGroup * D * 2;        // bytes of 16 K (or V) rows
  static constexpr int kStage = 2 * kTile;            // K, then V
  static constexpr int kRing = kStages * kStage;      // of one warp
  static constexpr int kList = kMaxPages * 8;         // {page, valid keys}
  static constexpr int kState = kWarps * kRows * 8;   // {m, l} per warp and row
  static constexpr int kSmem = kWarps * kRing + kList + kState;
  static_assert(kRing >= kRows * D * 4, "a warp's output fits in its ring");
};

template <int D, int SOURCE>
__global__ void __launch_bounds__(kWarps * 32) paged_attn_kernel(const AttnParams p) {
  using S = Shape<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  grid_dependency_sync(p.trigger_from);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int2* list = reinterpret_cast<int2*>(smem + kWarps * S::kRing);
  float2* state = reinterpret_cast<float2*>(smem + kWarps * S::kRing + S::kList);

  // ---- which rows, which keys --------------------------------------------------
  // rows of this CTA: row r is head head0 + r of token t (kSparse, kOwn), or
  // row tile * 16 + r of the (token, head of the group) pairs (kPrefix)
  int kv_head, t = 0, head0 = 0, rows;
  int64_t flat0 = 0;
  if (SOURCE == kPrefix) {
    kv_head = blockIdx.x / p.row_tiles;
    flat0 = (int64_t)(blockIdx.x % p.row_tiles) * kRows;
    const int64_t left = (int64_t)p.num_tokens * p.group - flat0;
    rows = left < kRows ? (int)left : kRows;
  } else {
    const int chunk = blockIdx.x % p.chunks;
    const int tg = blockIdx.x / p.chunks;
    kv_head = tg % p.num_kv;
    t = tg / p.num_kv;
    head0 = kv_head * p.group + chunk * kRows;
    rows = min(kRows, p.group - chunk * kRows);
  }
  // keys of the whole range (a page or a selected block counts page_size)
  int64_t keys;
  int req = 0, len = 0;
  bool rejected = false;
  if (SOURCE == kPrefix) {
    keys = p.prefix_len;
  } else {
    req = p.requests ? __ldg(p.requests + t) : t;
    len = __ldg(p.lens + t);
    const int64_t room = (int64_t)p.table_width * p.page_size;
    if (req < 0 || req >= p.num_requests || len < 0 || len > room) {
      rejected = true;
      if (len > room) len = (int)room;
      if (req < 0 || req >= p.num_requests || len < 0) len = 0;
    }
    keys = SOURCE == kSparse ? (len > 0 ? (int64_t)p.topk * p.page_size : 0) : len;
  }
  // this split's share, in whole pages
  const int64_t pages = (keys + p.page_size - 1) / p.page_size;
  const int64_t share = (pages + p.splits - 1) / p.splits;
  const int64_t page0 = share * blockIdx.y;
  const int listed = (int)max((int64_t)0, min(share, pages - page0));
  for (int i = threadIdx.x; i < listed; i += kWarps * 32) {
    int2 e = make_int2(0, 0);
    const int64_t at = page0 + i;
    if (SOURCE == kPrefix) {
      e.x = __ldg(p.prefix_pages + at);
      e.y = (int)min((int64_t)p.page_size, keys - at * p.page_size);
    } else if (SOURCE == kOwn) {
      e.x = __ldg(p.table + (int64_t)req * p.table_width + at);
      e.y = (int)min((int64_t)p.page_size, keys - at * p.page_size);
    } else {
      const int b = __ldg(p.blocks + ((int64_t)t * p.num_kv + kv_head) * p.topk + at);
      if (b >= 0 && (int64_t)b * p.page_size < len) {
        e.x = __ldg(p.table + (int64_t)req * p.table_width + b);
        e.y = min(p.page_size, len - b * p.page_size);
      } else if (b != -1) {
        rejected = true;
      }
    }
    if (e.y > 0 && (e.x < 0 || e.x >= p.num_pages)) {
      rejected = true;
      e = make_int2(0, 0);
    }
    list[i] = e;
  }
  if (rejected && p.errors && (SOURCE == kPrefix || threadIdx.x < listed || threadIdx.x == 0))
    atomicAdd(p.errors, 1);

  // ---- Q fragments ---------------------------------------------------------------
  // a lane holds rows lane/4 and lane/4 + 8, dims 16k + 2(lane%4) + {0, 1, 8, 9}
  uint32_t qf[D / 16][4];
  int64_t out_row[2];  // token * num_q + head of the lane's two rows, -1: no row
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = (lane >> 2) + 8 * i;
    out_row[i] = -1;
    const __nv_bfloat16* src = nullptr;
    if (r < rows) {
      int64_t tok = t;
      int head = head0 + r;
      if (SOURCE == kPrefix) {
        tok = (flat0 + r) / p.group;
        head = kv_head * p.group + (int)(flat0 + r - tok * p.group);
      }
      out_row[i] = tok * p.num_q + head;
      src = p.q + tok * p.q_stride + (int64_t)head * D + 2 * (lane & 3);
    }
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      qf[k][i] = src ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * k)) : 0u;
      qf[k][2 + i] = src ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * k + 8)) : 0u;
    }
  }
  __syncthreads();

  // ---- the warp's groups of keys ---------------------------------------------------
  const int total = listed * p.page_size;  // at most kMaxPages * page_size: checked at launch
  const int steps = (total + kGroup * kWarps - 1) / (kGroup * kWarps);
  const uint32_t ring = tma::smem_addr(smem) + warp * S::kRing;
  const int64_t head_elems = (int64_t)p.page_size * D;

  // Starts the copies of step i's 16 keys: lane r < 16 finds row r's place.
  auto issue = [&](int i) {
    const int k0 = (i * kWarps + warp) * kGroup;
    int64_t row = -1;
    if (lane < kGroup && i < steps && k0 + lane < total) {
      const int at = (k0 + lane) / p.page_size;
      const int off = k0 + lane - at * p.page_size;
      const int2 e = list[at];
      if (off < e.y) row = ((int64_t)e.x * 2 * p.num_kv + kv_head) * head_elems + (int64_t)off * D;
    }
    const uint32_t stage = ring + (i % S::kStages) * S::kStage;
    constexpr int FRAGS = D / 8;          // 16-byte fragments of a row
    constexpr int RPI = 32 / FRAGS > 0 ? 32 / FRAGS : 1;  // rows of one warp-wide copy
#pragma unroll
    for (int j = 0; j < kGroup / RPI; ++j) {
      const int r = j * RPI + lane / FRAGS, c = lane % FRAGS;
      const int64_t from = __shfl_sync(kFullMask, row, r);
      const __nv_bfloat16* src = p.cache + (from < 0 ? 0 : from) + 8 * c;
      const uint32_t dst = stage + r * (2 * D) + ((c ^ (r & 7)) << 4);
      cp_async16(dst, src, from >= 0);
      cp_async16(dst + S::kTile, src + (from < 0 ? 0 : p.num_kv * head_elems), from >= 0);
    }
    cp_commit();
  };

  float o[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int k = 0; k < 4; ++k) o[n][k] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

#pragma unroll
  for (int i = 0; i < S::kStages - 1; ++i) issue(i);
  for (int i = 0; i < steps; ++i) {
    issue(i + S::kStages - 1);
    cp_wait<S::kStages - 1>();
    __syncwarp();
    // which of the step's keys exist: bit r of the warp's ballot
    const int k0 = (i * kWarps + warp) * kGroup;
    bool there = false;
    if (lane < kGroup && k0 + lane < total) {
      const int at = (k0 + lane) / p.page_size;
      there = k0 + lane - at * p.page_size < list[at].y;
    }
    const uint32_t mask = __ballot_sync(kFullMask, there);
    if (mask == 0) {
      __syncwarp();
      continue;
    }
    const uint32_t kt = ring + (i % S::kStages) * S::kStage, vt = kt + S::kTile;
    float s[2][4] = {};
    {
      const int r = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t b[4];
        ldmatrix4(b, kt + r * (2 * D) + (((2 * k + half) ^ (r & 7)) << 4));
        mma16816(s[0], qf[k], b[0], b[1]);
        mma16816(s[1], qf[k], b[2], b[3]);
      }
    }
    // scores in units of log2: s * scale * log2(e); keys that do not exist -inf
    float top[2] = {m[0], m[1]};
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = 8 * n + 2 * (lane & 3) + (k & 1);
        s[n][k] = (mask >> key) & 1 ? s[n][k] * p.scale_log2 : -INFINITY;
        top[k >> 1] = fmaxf(top[k >> 1], s[n][k]);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      top[h] = fmaxf(top[h], __shfl_xor_sync(kFullMask, top[h], 1));
      top[h] = fmaxf(top[h], __shfl_xor_sync(kFullMask, top[h], 2));
    }
    if (__any_sync(kFullMask, top[0] != m[0] || top[1] != m[1])) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // (-inf) - (-inf): no key yet, nothing accumulated, any factor does
        const float f = top[h] == m[h] ? 1.f : exp2f(m[h] - top[h]);
        l[h] *= f;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) o[n][2 * h] *= f, o[n][2 * h + 1] *= f;
        m[h] = top[h];
      }
    }
    uint32_t pf[4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      float e[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float ref = m[k >> 1] == -INFINITY ? 0.f : m[k >> 1];
        e[k] = exp2f(s[n][k] - ref);
      }
      l[0] += e[0] + e[1];
      l[1] += e[2] + e[3];
      pf[2 * n] = pack_bf16x2(e[0], e[1]);
      pf[2 * n + 1] = pack_bf16x2(e[2], e[3]);
    }
    {
      const int r = (lane & 7) + (((lane >> 3) & 1) << 3), half = lane >> 4;
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        uint32_t b[4];
        ldmatrix4_trans(b, vt + r * (2 * D) + (((2 * n + half) ^ (r & 7)) << 4));
        mma16816(o[2 * n], pf, b[0], b[1]);
        mma16816(o[2 * n + 1], pf, b[2], b[3]);
      }
    }
    __syncwarp();  // the stage is read before its next copies start
  }
  cp_wait<0>();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(kFullMask, l[h], 1);
    l[h] += __shfl_xor_sync(kFullMask, l[h], 2);
    if ((lane & 3) == 0) state[warp * kRows + (lane >> 2) + 8 * h] = make_float2(m[h], l[h]);
  }
  __syncthreads();

  // ---- join the warps ------------------------------------------------------------------
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = (lane >> 2) + 8 * h;
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, state[w * kRows + r].x);
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      sum += state[w * kRows + r].y * exp2f(state[w * kRows + r].x - ref);
    const float f = sum == 0.f ? 0.f : exp2f(m[h] - ref) / sum;  // 0: the row has no key
    float* dst = reinterpret_cast<float*>(smem + warp * S::kRing) + r * D + 2 * (lane & 3);
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
      *reinterpret_cast<float2*>(dst + 8 * n) = make_float2(o[n][2 * h] * f, o[n][2 * h + 1] * f);
    if (!p.direct && warp == 0 && (lane & 3) == 0 && out_row[h] >= 0)
      p.parts.lse[(int64_t)(p.first_slot + blockIdx.y) * p.parts.rows + out_row[h]] =
          sum == 0.f ? -INFINITY : ref + log2f(sum);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (D / 4); i += kWarps * 32) {
    const int r = i / (D / 4), c = 4 * (i % (D / 4));
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 u = *reinterpret_cast<const float4*>(
          reinterpret_cast<const float*>(smem + w * S::kRing) + r * D + c);
      v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
    int64_t tok = t;
    int head = head0 + r;
    if (SOURCE == kPrefix) {
      tok = (flat0 + r) / p.group;
      head = kv_head * p.group + (int)(flat0 + r - tok * p.group);
    }
    const int64_t row = tok * p.num_q + head;
    if (p.direct) {
      *reinterpret_cast<uint2*>(p.out + row * D + c) =
          make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    } else {
      const int64_t slot = p.first_slot + blockIdx.y;
      *reinterpret_cast<float4*>(p.parts.o + (slot * p.parts.rows + row) * D + c) = v;
    }
  }
}

// ---- the join of the parts -------------------------------------------------------------

struct JoinParams {
  Partials parts;
  int slots;
  __nv_bfloat16* out;
  int trigger_from;
};

// One warp per row; the row's weights are found by the lanes together.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) attn_join_kernel(const JoinParams p) {
  grid_dependency_sync(p.trigger_from);
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= p.parts.rows) return;
  const int lane = threadIdx.x & 31;
  float top = -INFINITY;
  for (int s = lane; s < p.slots; s += 32) top = fmaxf(top, p.parts.lse[s * p.parts.rows + row]);
  top = group_max<32>(top);
  constexpr int V = D / 32;  // dims of a lane
  const float ref = top == -INFINITY ? 0.f : top;
  float acc[V] = {};
  float sum = 0.f;
  for (int s = 0; s < p.slots; ++s) {
    const float lse = p.parts.lse[s * p.parts.rows + row];
    if (lse == -INFINITY) continue;  // a part without a key
    const float w = exp2f(lse - ref);  // may be 0; a NaN output still counts
    sum += w;
    const float* o = p.parts.o + (s * p.parts.rows + row) * D + V * lane;
#pragma unroll
    for (int k = 0; k < V; k += 2) {
      const float2 v = *reinterpret_cast<const float2*>(o + k);
      acc[k] = fmaf(w, v.x, acc[k]);
      acc[k + 1] = fmaf(w, v.y, acc[k + 1]);
    }
  }
  const float f = sum == 0.f ? 0.f : 1.f / sum;
  __nv_bfloat16* out = p.out + row * D + V * lane;
#pragma unroll
  for (int k = 0; k < V; k += 2)
    *reinterpret_cast<uint32_t*>(out + k) = pack_bf16x2(acc[k] * f, acc[k + 1] * f);
}

template <int D>
cudaError_t launch_join(const JoinParams& in, cudaStream_t stream) {
  JoinParams p = in;
  const int64_t grid = (p.parts.rows + kWarps - 1) / kWarps;
  static std::atomic<int> cache[kMaxDevices];
  p.trigger_from = last_wave_start(attn_join_kernel<D>, kWarps * 32, grid, cache);
  return launch_kernel(attn_join_kernel<D>, dim3((unsigned)grid), dim3(kWarps * 32), 0, stream, p);
}

// ---- launch ------------------------------------------------------------------------------

// Parts a range of up to `pages` pages is split into when `ctas` CTAs would
// each take a whole one: enough CTAs for two on each of the 152 SMs, none
// with less than 4 groups of keys a warp, and none with more pages than fit
// its list.
int splits_for(int64_t ctas, int64_t pages, int page_size) {
  const int64_t least = (pages + kMaxPages - 1) / kMaxPages;
  const int64_t most = pages * page_size / (kGroup * kWarps * 4);
  int64_t s = (2 * 152 + ctas - 1) / ctas;
  if (s > most) s = most;
  if (s < least) s = least;
  if (s > pages) s = pages;
  return s < 1 ? 1 : (int)s;
}

template <int D, int SOURCE>
cudaError_t launch_attn(AttnParams p, int64_t ctas, cudaStream_t stream) {
  static std::atomic<int> cache[kMaxDevices];
  int per_sm = 0;
  const cudaError_t e = tma::prepare(paged_attn_kernel<D, SOURCE>, kWarps * 32, Shape<D>::kSmem,
                                     cache, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t wave = (int64_t)per_sm * device_sm_count();
  p.trigger_from = 0;
  if (ctas > wave) p.trigger_from = (int)(ctas - wave);
  return launch_kernel(paged_attn_kernel<D, SOURCE>, dim3((unsigned)ctas, (unsigned)p.splits),
                       dim3(kWarps * 32), Shape<D>::kSmem, stream, p);
}

template <int SOURCE>
cudaError_t launch_attn_dim(const AttnParams& p, int head_dim, int64_t ctas,
                            cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_attn<64, SOURCE>(p, ctas, stream);
    case 128: return launch_attn<128, SOURCE>(p, ctas, stream);
    case 256: return launch_attn<256, SOURCE>(p, ctas, stream);
  }
  return cudaErrorInvalidValue;
}

AttnParams common(const PagedQuery& x, const void* kv_cache, float scale) {
  AttnParams p = {};
  p.q = static_cast<const __nv_bfloat16*>(x.q);
  p.q_stride = x.q_stride;
  p.cache = static_cast<const __nv_bfloat16*>(kv_cache);
  p.num_q = x.num_heads_q;
  p.num_kv = x.num_heads_kv;
  p.group = x.num_heads_q / x.num_heads_kv;
  p.chunks = (p.group + kRows - 1) / kRows;
  p.num_tokens = x.num_tokens;
  p.num_pages = x.num_pages;
  p.page_size = x.page_size;
  p.table = x.page_table;
  p.num_requests = x.num_requests;
  p.table_width = x.table_width;
  p.requests = x.requests;
  p.lens = x.lens;
  p.scale_log2 = scale * kLog2e;
  p.errors = x.errors;
  return p;
}

int64_t own_ctas(int64_t num_tokens, int num_q, int num_kv) {
  const int group = num_q / num_kv;
  return num_tokens * num_kv * ((group + kRows - 1) / kRows);
}

int64_t prefix_tiles(int64_t num_tokens, int num_q, int num_kv) {
  return (num_tokens * (num_q / num_kv) + kRows - 1) / kRows;
}

// Parts of the prefix on the small matrix instruction, and of the tokens' own
// keys (0: there are none).
int prefix_slots(int64_t num_tokens, int num_q, int num_kv, int page_size, int64_t prefix_len) {
  if (prefix_len == 0) return 0;
  return splits_for(prefix_tiles(num_tokens, num_q, num_kv) * num_kv,
                    (prefix_len + page_size - 1) / page_size, page_size);
}

int own_slots(int64_t num_tokens, int num_q, int num_kv, int page_size, int table_width) {
  if (table_width == 0) return 0;
  return splits_for(own_ctas(num_tokens, num_q, num_kv), table_width, page_size);
}

}  // namespace

cudaError_t launch_attn_join(const Partials& parts, int slots, int head_dim, void* out,
                             cudaStream_t stream) {
  JoinParams p;
  p.parts = parts;
  p.slots = slots;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.trigger_from = 0;
  switch (head_dim) {
    case 64: return launch_join<64>(p, stream);
    case 128: return launch_join<128>(p, stream);
    case 256: return launch_join<256>(p, stream);
  }
  return cudaErrorInvalidValue;
}

int64_t sparse_attn_workspace(int64_t num_tokens, int num_heads_q, int num_heads_kv,
                              int head_dim, int page_size, int topk) {
  const int s = splits_for(own_ctas(num_tokens, num_heads_q, num_heads_kv), topk, page_size);
  return s == 1 ? 0 : partials_bytes(s, num_tokens * num_heads_q, head_dim);
}

cudaError_t launch_sparse_attn(const SparseAttnArgs& a, cudaStream_t stream) {
  const PagedQuery& x = a.x;
  AttnParams p = common(x, a.kv_cache, a.scale);
  p.blocks = a.blocks;
  p.topk = a.topk;
  const int64_t ctas = own_ctas(x.num_tokens, x.num_heads_q, x.num_heads_kv);
  p.splits = splits_for(ctas, a.topk, x.page_size);
  p.direct = p.splits == 1;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  const int64_t rows = (int64_t)x.num_tokens * x.num_heads_q;
  if (!p.direct) p.parts = partials_at(a.workspace, p.splits, rows, x.head_dim);
  const cudaError_t e = launch_attn_dim<kSparse>(p, x.head_dim, ctas, stream);
  if (e != cudaSuccess || p.direct) return e;
  return launch_attn_join(p.parts, p.splits, x.head_dim, a.out, stream);
}

int64_t prefix_attn_workspace(int64_t num_tokens, int num_heads_q, int num_heads_kv,
                              int head_dim, int page_size, int64_t prefix_len,
                              int table_width) {
  const int64_t slots =
      prefix_slots(num_tokens, num_heads_q, num_heads_kv, page_size, prefix_len);
  int64_t tiles = 0;
  if (prefix_tiles_fit(num_tokens, num_heads_q, num_heads_kv, head_dim, page_size, prefix_len))
    tiles = prefix_tiles_plan(num_tokens, num_heads_q, num_heads_kv, head_dim, page_size,
                              prefix_len).parts;
  // either kernel may run: which one depends on where the cache lies
  return partials_bytes((slots > tiles ? slots : tiles) +
                            own_slots(num_tokens, num_heads_q, num_heads_kv, page_size,
                                      table_width),
                        num_tokens * num_heads_q, head_dim);
}

cudaError_t launch_prefix_attn(const PrefixAttnArgs& a, cudaStream_t stream) {
  const PagedQuery& x = a.x;
  AttnParams p = common(x, a.kv_cache, a.scale);
  p.prefix_pages = a.prefix_pages;
  p.prefix_len = a.prefix_len;
  const int64_t rows = (int64_t)x.num_tokens * x.num_heads_q;
  CUtensorMap map;
  const bool tiles = prefix_tiles_fit(x.num_tokens, x.num_heads_q, x.num_heads_kv, x.head_dim,
                                      x.page_size, a.prefix_len) &&
                     prefix_tiles_map(a, &map);
  const int s1 = tiles ? prefix_tiles_plan(x.num_tokens, x.num_heads_q, x.num_heads_kv,
                                           x.head_dim, x.page_size, a.prefix_len).parts
                       : prefix_slots(x.num_tokens, x.num_heads_q, x.num_heads_kv, x.page_size,
                                      a.prefix_len);
  const int s2 = own_slots(x.num_tokens, x.num_heads_q, x.num_heads_kv, x.page_size,
                           x.table_width);
  p.parts = partials_at(a.workspace, s1 + s2, rows, x.head_dim);
  cudaError_t e = cudaSuccess;
  if (tiles) {
    e = launch_prefix_tiles(a, map, p.parts, stream);
  } else if (s1) {
    p.row_tiles = (int)prefix_tiles(x.num_tokens, x.num_heads_q, x.num_heads_kv);
    p.splits = s1;
    p.first_slot = 0;
    e = launch_attn_dim<kPrefix>(p, x.head_dim, (int64_t)p.row_tiles * x.num_heads_kv, stream);
  }
  if (e == cudaSuccess && s2) {
    p.splits = s2;
    p.first_slot = s1;
    e = launch_attn_dim<kOwn>(p, x.head_dim, own_ctas(x.num_tokens, x.num_heads_q, x.num_heads_kv),
                              stream);
  }
  if (e != cudaSuccess) return e;
  return launch_attn_join(p.parts, s1 + s2, x.head_dim, a.out, stream);
}

}  // namespace kvq
