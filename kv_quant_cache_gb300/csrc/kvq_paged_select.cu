// kvq_paged_select.cu -- which cache blocks (pages) a token attends to: a
// cheap score of every block from the bounds of its keys, and the top-k.
//
// Score of block j for a token and kv head, with the group's query heads h
// and the bounds lo <= key <= hi of the block's keys, dim by dim:
//   sum_h sum_d max(q_hd lo_jd, q_hd hi_jd)
//     = sum_d [ up_d hi_jd + down_d lo_jd ],
//   up_d = sum_h max(q_hd, 0),  down_d = sum_h min(q_hd, 0),
// an upper bound of the group's summed logits on any key of the block.  The
// group's sums are taken once, so a block costs 2 D products whatever the
// group's size: bound by reading the bounds once.
//
// One cluster of 1..8 CTAs per (token, kv head) (more CTAs where few tokens
// would leave SMs idle).  Every CTA scores a share of the blocks in fp32 and
// writes the scores into the first CTA's shared memory; that CTA selects.
//
// Which block is k-th must not depend on fp32 rounding: the set a token
// attends to is an integer result.  The scoring warps carry the largest
// sum of |products| along, which bounds every fp32 score's error by E.  With
// T the k-th largest fp32 score, blocks above T + 2E are in and below T - 2E
// out whatever the rounding; if more blocks lie between than there are
// places left, those few are scored again in fp64 (products of an fp64 sum
// of bf16 values with a bf16 value) and the places go to the largest, the
// lower index first where equal.
#include <cooperative_groups.h>

#include "kvq_device.cuh"
#include "kvq_paged.h"
#include "kvq_tma.cuh"

namespace cg = cooperative_groups;

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

struct SelectParams {
  const __nv_bfloat16* q;
  int64_t q_stride;
  const __nv_bfloat16* bounds;
  int num_kv, group;
  int64_t num_pages;
  int page_size;
  const int* table;
  int num_requests, table_width;
  const int* requests;
  const int* lens;
  int topk, keep_first, keep_last;
  int* blocks;
  int* errors;
  int cluster;
};

// Order-preserving keys: a larger score has a larger key; NaN (and a page
// outside the cache) ranks with -inf, kept blocks above everything.
constexpr uint32_t kKeep32 = 0xffffffffu;
__device__ __forceinline__ uint32_t key32(float s) {
  if (!(s > -INFINITY)) return 0x007fffffu;  // the key of -inf
  const uint32_t b = __float_as_uint(s);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value32(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t key64(double s) {
  if (!(s > -(double)INFINITY)) return 0x000fffffffffffffull;
  const uint64_t b = (uint64_t)__double_as_longlong(s);
  return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

// Shared memory of a CTA (the selecting one uses all of it).
template <int D>
struct Shared {
  float up[D], down[D];
  double up64[D], down64[D];
  float err[kMaxCluster * kWarps];
  unsigned hist[256];
  unsigned warp_a[kWarps], warp_b[kWarps];
  unsigned long long pick;
  unsigned place;
};

// The `place`-th largest (1 = largest) of the keys that `get(i, &key)` gives
// for i < n, found one byte at a time from the top; *equal becomes how many
// of the keys equal to it belong to the `place` largest.  All threads call.
template <typename Key, typename Get, typename Sh>
__device__ Key radix_select(int n, unsigned place, Sh& sh, const Get& get, unsigned* equal) {
  Key prefix = 0;
  const int tid = threadIdx.x;
  for (int shift = (int)sizeof(Key) * 8 - 8; shift >= 0; shift -= 8) {
    for (int b = tid; b < 256; b += kThreads) sh.hist[b] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      Key k;
      if (!get(i, &k)) continue;
      const bool same = shift + 8 >= (int)sizeof(Key) * 8 || (k >> (shift + 8)) == (prefix >> (shift + 8));
      if (same) atomicAdd(&sh.hist[(unsigned)(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid < 32) {
      // lane l owns bins 255 - 8l .. 248 - 8l: counts from the top
      unsigned c[8], sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = sh.hist[255 - 8 * tid - j], sum += c[j];
      unsigned above = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned v = __shfl_up_sync(kFullMask, above, o);
        if (tid >= o) above += v;
      }
      above -= sum;  // keys in higher bins than this lane's
      if (above < place && place <= above + sum) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (above < place && place <= above + c[j]) {
            sh.pick = 255 - 8 * tid - j;
            sh.place = place - above;
          }
          above += c[j];
        }
      }
    }
    __syncthreads();
    prefix |= (Key)sh.pick << shift;
    place = sh.place;
    __syncthreads();
  }
  *equal = place;
  return prefix;
}

template <int D>
__global__ void __launch_bounds__(kThreads) block_select_kernel(const SelectParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared<D>& sh = *reinterpret_cast<Shared<D>*>(smem);
  // scores of the first CTA: fp32 keys, then fp64 keys, one of each per block
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem + ((sizeof(Shared<D>) + 15) & ~size_t(15)));
  unsigned long long* wide =
      reinterpret_cast<unsigned long long*>(keys + ((p.table_width + 1) & ~1));
  cg::cluster_group cluster = cg::this_cluster();
  grid_dependency_sync(0);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = p.cluster > 1 ? (int)cluster.block_rank() : 0;
  const int64_t tg = blockIdx.x / p.cluster;
  const int64_t t = tg / p.num_kv;
  const int h = (int)(tg - t * p.num_kv);
  int* out = p.blocks + tg * p.topk;

  // ---- the token's blocks ---------------------------------------------------------
  int req = p.requests ? __ldg(p.requests + t) : (int)t;
  int len = __ldg(p.lens + t);
  const int64_t room = (int64_t)p.table_width * p.page_size;
  bool rejected = false;
  if (req < 0 || req >= p.num_requests || len < 0) {
    rejected = true;
    req = 0;
    len = 0;
  } else if (len > room) {
    rejected = true;
    len = (int)room;
  }
  if (rejected && p.errors && rank == 0 && tid == 0) atomicAdd(p.errors, 1);
  const int n = (int)(((int64_t)len + p.page_size - 1) / p.page_size);
  if (n <= p.topk) {  // all of them: no score decides anything (cluster-uniform)
    if (rank == 0)
      for (int i = tid; i < p.topk; i += kThreads) out[i] = i < n ? i : -1;
    return;
  }

  // ---- the group's query sums ------------------------------------------------------
  for (int d = tid; d < D; d += kThreads) {
    double up = 0., down = 0.;
    const __nv_bfloat16* q = p.q + t * p.q_stride + (int64_t)h * p.group * D + d;
    for (int g = 0; g < p.group; ++g) {
      const float v = __bfloat162float(q[(int64_t)g * D]);
      up += v > 0.f ? v : v == v ? 0.f : v;  // a NaN stays one
      down += v < 0.f ? v : v == v ? 0.f : v;
    }
    sh.up64[d] = up, sh.down64[d] = down;
    sh.up[d] = (float)up, sh.down[d] = (float)down;
  }
  __syncthreads();
  // the selecting CTA's shared memory has to exist before scores go there
  if (p.cluster > 1) cluster.sync();

  // ---- scores ------------------------------------------------------------------------
  // A block's bounds are 2 D contiguous values (lo, then hi): lane l of a
  // block's LPB lanes takes values 8l.. of each run of 8 LPB.
  constexpr int LPB = D / 4 < 32 ? D / 4 : 32;
  constexpr int VECS = 2 * D / (8 * LPB);
  constexpr int BPW = 32 / LPB;  // blocks of one warp step
  constexpr int UNROLL = 4;
  uint32_t* to_keys = p.cluster > 1 ? cluster.map_shared_rank(keys, 0) : keys;
  float* to_err = p.cluster > 1 ? cluster.map_shared_rank(sh.err, 0) : sh.err;
  const int bl = lane % LPB;
  float w[VECS][8];
#pragma unroll
  for (int v = 0; v < VECS; ++v) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int at = 8 * (v * LPB + bl) + k;
      w[v][k] = at < D ? sh.down[at] : sh.up[at - D];
    }
  }
  const int* row = p.table + (int64_t)req * p.table_width;
  const int64_t head_elems = 2 * D;
  float worst = 0.f;  // of this lane: the largest sum of |products| it saw
  bool odd = false;
  const int per_step = BPW * UNROLL;
  for (int j0 = (rank * kWarps + warp) * per_step; j0 < n; j0 += p.cluster * kWarps * per_step) {
    uint4 x[UNROLL][VECS];
    bool fine[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int j = j0 + u * BPW + lane / LPB;
      const int page = j < n ? __ldg(row + j) : -1;
      fine[u] = page >= 0 && page < p.num_pages;
      if (j < n && !fine[u] && p.errors && bl == 0) atomicAdd(p.errors, 1);
      const __nv_bfloat16* src =
          p.bounds + ((int64_t)(fine[u] ? page : 0) * p.num_kv + h) * head_elems + 8 * bl;
#pragma unroll
      for (int v = 0; v < VECS; ++v)
        x[u][v] = fine[u] ? __ldg(reinterpret_cast<const uint4*>(src + 8 * LPB * v))
                          : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      float s = 0.f, a = 0.f;
#pragma unroll
      for (int v = 0; v < VECS; ++v) {
        float b[8];
        unpack_bf16x8(x[u][v], b);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          s = fmaf(w[v][k], b[k], s);
          a = fmaf(fabsf(w[v][k]), fabsf(b[k]), a);
        }
      }
      odd |= !(a <= 3.0e38f);  // infinite or NaN: fp32 says nothing
      worst = fmaxf(worst, a);
      s = group_sum<LPB>(s);
      const int j = j0 + u * BPW + lane / LPB;
      if (bl == 0 && j < n) {
        const bool keep = j < p.keep_first || j >= n - p.keep_last;
        to_keys[j] = keep ? kKeep32 : fine[u] ? key32(s) : key32(-INFINITY);
      }
    }
  }
  // sum over the lanes of their largest: at least every block's sum.  The
  // fp32 score takes at most 8 VECS + 5 additions and one rounding of the
  // query sums on any path, so it is off by less than 32 * 2^-24 of it (and
  // by a few steps of the smallest binary32 where products underflow).
  worst = group_sum<LPB>(worst);
  worst = BPW > 1 ? fmaxf(worst, __shfl_xor_sync(kFullMask, worst, 16)) : worst;
  odd = __any_sync(kFullMask, odd || !(worst <= 3.0e38f));
  if (lane == 0)
    to_err[rank * kWarps + warp] =
        odd ? INFINITY : worst > 0.f ? worst * (32.f / 16777216.f) + 1.0e-42f : 0.f;
  if (p.cluster > 1) {
    cluster.sync();  // every score has arrived; no CTA is needed any longer but the first
    if (rank != 0) return;
  } else {
    __syncthreads();
  }

  // ---- the k-th largest, its doubtful neighbours ---------------------------------------
  float E = 0.f;
  for (int i = 0; i < p.cluster * kWarps; ++i) E = fmaxf(E, sh.err[i]);
  unsigned ties;
  const uint32_t kth = radix_select<uint32_t>(
      n, (unsigned)p.topk, sh, [&](int i, uint32_t* k) { *k = keys[i]; return true; }, &ties);
  // keys from `in` up are selected, below `maybe` are not
  uint32_t in = kth, maybe = kth;
  if (kth != kKeep32 && E > 0.f) {
    const float T = value32(kth);
    if (E == INFINITY || !(fabsf(T) <= 3.0e38f)) {
      in = kKeep32;
      maybe = 0;
    } else {
      const float up = T + 2.f * E, down = T - 2.f * E;
      // one step outward covers the rounding of the two sums
      in = min(key32(up) + 2u, kKeep32);
      maybe = key32(down) - 2u;
    }
  }
  unsigned places = ties;  // places left for the keys in [maybe, in)
  bool exact = in == maybe;
  if (!exact) {
    unsigned above = 0, between = 0;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
      const int i = i0 + tid;
      const uint32_t k = i < n ? keys[i] : 0u;
      above += i < n && k >= in;
      between += i < n && k < in && k >= maybe;
    }
    above = __reduce_add_sync(kFullMask, above);
    between = __reduce_add_sync(kFullMask, between);
    if (lane == 0) sh.warp_a[warp] = above, sh.warp_b[warp] = between;
    __syncthreads();
    above = between = 0;
    for (int i = 0; i < kWarps; ++i) above += sh.warp_a[i], between += sh.warp_b[i];
    __syncthreads();
    places = (unsigned)p.topk - above;
    if (between == places) {
      in = maybe;  // all of them
      places = 0;
      exact = true;
    }
  } else {
    // equal fp32 scores are equal scores: no product was other than zero, or
    // only kept blocks compete; `ties` of the blocks at kth, lowest first
  }
  unsigned long long kth64 = 0;
  unsigned ties64 = 0;
  const bool only_ties = exact && places > 0;
  if (!exact) {
    // the doubtful ones again, one per warp, in fp64 and in one fixed order
    for (int i = warp; i < n; i += kWarps) {
      if (!(keys[i] < in && keys[i] >= maybe)) continue;
      const int page = __ldg(row + i);
      double s = 0.;
      if (page >= 0 && page < p.num_pages) {
        const __nv_bfloat16* b = p.bounds + ((int64_t)page * p.num_kv + h) * head_elems;
        for (int d = lane; d < D; d += 32) {
          s = fma(sh.down64[d], (double)__bfloat162float(b[d]), s);
          s = fma(sh.up64[d], (double)__bfloat162float(b[D + d]), s);
        }
      } else {
        s = -(double)INFINITY;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFullMask, s, o);
      if (lane == 0) wide[i] = key64(s);
    }
    __syncthreads();
    kth64 = radix_select<unsigned long long>(
        n, places, sh,
        [&](int i, unsigned long long* k) {
          if (!(keys[i] < in && keys[i] >= maybe)) return false;
          *k = wide[i];
          return true;
        },
        &ties64);
  }

  // ---- the selected blocks, ascending -----------------------------------------------------
  const unsigned ties_to_take = exact ? places : ties64;
  unsigned taken = 0, tied = 0;
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const int i = i0 + tid;
    bool sure = false, tie = false;
    if (i < n) {
      const uint32_t k = keys[i];
      if (exact) {
        sure = only_ties ? k > kth : k >= in;
        tie = only_ties && k == kth;
      } else {
        sure = k >= in;
        if (!sure && k >= maybe) {
          sure = wide[i] > kth64;
          tie = wide[i] == kth64;
        }
      }
    }
    const unsigned tm = __ballot_sync(kFullMask, tie);
    if (lane == 0) sh.warp_a[warp] = __popc(tm);
    __syncthreads();
    unsigned before = tied + __popc(tm & ((1u << lane) - 1u));
    for (int j = 0; j < kWarps; ++j) {
      const unsigned c = sh.warp_a[j];
      if (j < warp) before += c;
      tied += c;
    }
    const bool sel = sure || (tie && before < ties_to_take);
    const unsigned sm = __ballot_sync(kFullMask, sel);
    if (lane == 0) sh.warp_b[warp] = __popc(sm);
    __syncthreads();
    unsigned at = taken + __popc(sm & ((1u << lane) - 1u));
    for (int j = 0; j < kWarps; ++j) {
      const unsigned c = sh.warp_b[j];
      if (j < warp) at += c;
      taken += c;
    }
    if (sel && at < (unsigned)p.topk) out[at] = i;
  }
}

template <int D>
size_t smem_bytes(int width) {
  return ((sizeof(Shared<D>) + 15) & ~size_t(15)) + (size_t)((width + 1) & ~1) * 4 +
         (size_t)width * 8;
}

// CTAs of a cluster: more while the whole grid would leave SMs idle and a CTA
// would still have a step of blocks for each of its warps.
int cluster_for(int64_t items, int width) {
  int c = 1;
  while (c < kMaxCluster && items * c < 152 && width > c * 2 * kWarps * 8) c *= 2;
  return c;
}

template <int D>
cudaError_t launch_select(const BlockSelectArgs& a, cudaStream_t stream) {
  const PagedQuery& x = a.x;
  static std::atomic<int> cache[kMaxDevices];
  int per_sm = 0;
  // one opt-in for the largest size that the validation lets through
  const cudaError_t e = tma::prepare(block_select_kernel<D>, kThreads, smem_bytes<D>(kMaxSelectBlocks),
                               cache, &per_sm);
  if (e != cudaSuccess) return e;
  SelectParams p;
  p.q = static_cast<const __nv_bfloat16*>(x.q);
  p.q_stride = x.q_stride;
  p.bounds = static_cast<const __nv_bfloat16*>(a.bounds);
  p.num_kv = x.num_heads_kv;
  p.group = x.num_heads_q / x.num_heads_kv;
  p.num_pages = x.num_pages;
  p.page_size = x.page_size;
  p.table = x.page_table;
  p.num_requests = x.num_requests;
  p.table_width = x.table_width;
  p.requests = x.requests;
  p.lens = x.lens;
  p.topk = a.topk;
  p.keep_first = a.keep_first;
  p.keep_last = a.keep_last;
  p.blocks = a.blocks;
  p.errors = x.errors;
  const int64_t items = (int64_t)x.num_tokens * x.num_heads_kv;
  p.cluster = cluster_for(items, x.table_width);
  return launch_clusters(block_select_kernel<D>, dim3((unsigned)(items * p.cluster)),
                         dim3(kThreads), smem_bytes<D>(x.table_width), p.cluster, stream, p);
}

}  // namespace

cudaError_t launch_block_select(const BlockSelectArgs& a, cudaStream_t stream) {
  switch (a.x.head_dim) {
    case 64: return launch_select<64>(a, stream);
    case 128: return launch_select<128>(a, stream);
    case 256: return launch_select<256>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kvq
