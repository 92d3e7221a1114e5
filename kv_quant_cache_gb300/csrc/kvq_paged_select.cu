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
// One cluster of 1..8 CTAs takes a token and kv head.  Its CTAs score a share
// of the blocks each, their fp32 scores go into the first CTA's shared memory,
// and that CTA selects.
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
#include "kvq_mma.cuh"
#include "kvq_paged.h"
#include "kvq_tma.cuh"

namespace cg = cooperative_groups;

namespace kvq {
namespace {

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
  int cluster;  // CTAs of a cluster
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

constexpr int kBins = 512;  // 64 tokens x 256 blocks 14.5 us, with 2048 bins 15.0

// Shared memory of a CTA of T threads (the selecting one uses all of it).
template <int D, int T>
struct Shared {
  static constexpr int kThreads = T, kWarps = T / 32;
  static constexpr int kFew = T;  // candidates that are ranked against each other directly
  double up64[D], down64[D];
  // of every scoring warp: its error bound, its smallest and largest key (of
  // blocks that are not kept anyway)
  float err[kMaxCluster * kWarps];
  uint32_t least[kMaxCluster * kWarps], most[kMaxCluster * kWarps];
  unsigned hist[kBins];
  int few[kFew];  // candidates by index
  unsigned warp_sum[kWarps];
  unsigned count;
  unsigned pick, place, bin_count;
  unsigned long long kth64;
};

// While scoring, the place of the fp64 keys has the query sums (down, then up,
// as a block's bounds are lo, then hi) in three bf16 parts, and their sizes
// rounded up.
template <int D>
struct QueryParts {
  __nv_bfloat16 part[4][2 * D];
};

// Inclusive prefix sum over the CTA of one value a thread; *total: all of it.
template <typename Sh>
__device__ unsigned block_scan(unsigned v, Sh& sh, unsigned* total) {
  constexpr int kWarps = Sh::kWarps;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned u = __shfl_up_sync(kFullMask, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) sh.warp_sum[warp] = v;
  __syncthreads();
  unsigned sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) v += sum;
    sum += sh.warp_sum[w];
  }
  *total = sum;
  __syncthreads();
  return v;
}

// Finds the bin that holds the `place`-th largest key (1 = largest) from the
// counts in sh.hist: sh.pick the bin, sh.place its place within the bin,
// sh.bin_count the bin's keys.  All threads call, after a barrier.
template <typename Sh>
__device__ void find_bin(unsigned place, Sh& sh) {
  constexpr int PER = kBins / Sh::kThreads;
  const int first = kBins - 1 - PER * (int)threadIdx.x;  // this thread's highest bin
  unsigned c[PER], sum = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) c[j] = sh.hist[first - j], sum += c[j];
  unsigned total;
  unsigned above = block_scan(sum, sh, &total) - sum;
  if (above < place && place <= above + sum) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (above < place && place <= above + c[j]) {
        sh.pick = first - j;
        sh.place = place - above;
        sh.bin_count = c[j];
      }
      above += c[j];
    }
  }
  __syncthreads();
}

// The `place`-th largest of the keys that `get(i, &key)` gives for i < n (all
// keys between lo and hi); *equal becomes how many of the keys equal to it
// belong to the `place` largest.  One linear split of [lo, hi] into bins
// usually leaves a few candidates, which are ranked directly; otherwise the
// bin's own range is split again (each time by 2^9).  All threads call.
template <typename Key, typename Get, typename Sh>
__device__ Key select_largest(int n, unsigned place, Key lo, Key hi, Sh& sh, const Get& get,
                              unsigned* equal) {
  constexpr int kThreads = Sh::kThreads, kFew = Sh::kFew;
  const int tid = threadIdx.x;
  while (true) {
    int shift = 0;
    while (((hi - lo) >> shift) >= (Key)kBins) ++shift;
    for (int b = tid; b < kBins; b += kThreads) sh.hist[b] = 0;
    if (tid == 0) sh.count = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      Key k;
      if (get(i, &k) && k >= lo && k <= hi) atomicAdd(&sh.hist[(unsigned)((k - lo) >> shift)], 1u);
    }
    __syncthreads();
    find_bin(place, sh);
    place = sh.place;
    lo += (Key)sh.pick << shift;
    const Key last = lo + (((Key)1 << shift) - 1);
    if (last < hi) hi = last;
    const unsigned c = sh.bin_count;
    if (shift == 0 || lo == hi) {  // one value is left
      *equal = place;
      __syncthreads();
      return lo;
    }
    if (c <= (unsigned)kFew) {
      for (int i = tid; i < n; i += kThreads) {
        Key k;
        if (get(i, &k) && k >= lo && k <= hi) sh.few[atomicAdd(&sh.count, 1u)] = i;
      }
      __syncthreads();
      if (tid < (int)c) {
        Key mine, other;
        get(sh.few[tid], &mine);
        unsigned larger = 0, same = 0;
        for (unsigned j = 0; j < c; ++j) {
          get(sh.few[j], &other);
          larger += other > mine;
          same += other == mine;
        }
        if (larger < place && place <= larger + same) {  // every such thread writes the same
          sh.kth64 = (unsigned long long)mine;
          sh.place = place - larger;
        }
      }
      __syncthreads();
      const Key k = (Key)sh.kth64;
      *equal = sh.place;
      __syncthreads();
      return k;
    }
    __syncthreads();
  }
}

// Selects from the scores (all threads of the CTA): `keys` of n > topk blocks,
// `scorers` entries of err, least and most; the group's queries, the request's
// pages and the bounds of the head on page 0 for scores that have to be taken
// again.
template <int D, typename Sh>
__device__ void select_blocks(const SelectParams& p, Sh& sh, uint32_t* keys,
                              unsigned long long* wide, int scorers, int n,
                              const __nv_bfloat16* queries, const int* row,
                              const __nv_bfloat16* bounds, int* out) {
  constexpr int kThreads = Sh::kThreads, kWarps = Sh::kWarps, kFew = Sh::kFew;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t page_elems = (int64_t)p.num_kv * 2 * D;
  // ---- the k-th largest, its doubtful neighbours ---------------------------------------
  float E = 0.f;
  uint32_t least = 0xffffffffu, most = 0;
  for (int i = lane; i < scorers; i += 32) {
    E = fmaxf(E, sh.err[i]);
    least = min(least, sh.least[i]);
    most = max(most, sh.most[i]);
  }
  E = group_max<32>(E);
  least = __reduce_min_sync(kFullMask, least);
  most = __reduce_max_sync(kFullMask, most);
  unsigned ties;
  // the kept blocks are selected anyway; the others compete for what is left
  const int kept = min(n, min(n, p.keep_first) + min(n, p.keep_last));
  uint32_t kth;
  if (kept >= p.topk) {
    kth = kKeep32;
    ties = p.topk;
  } else {
    kth = select_largest<uint32_t>(
        n, (unsigned)(p.topk - kept), least, most, sh,
        [&](int i, uint32_t* k) { *k = keys[i]; return *k != kKeep32; }, &ties);
  }
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
  // a thread's blocks from here on: `each` consecutive ones
  const int each = (n + kThreads - 1) / kThreads;
  const int mine0 = min(n, tid * each), mine1 = min(n, mine0 + each);
  unsigned places = ties;  // places left for the keys in [maybe, in)
  bool exact = in == maybe;
  const bool only_ties = exact;  // equal fp32 scores are equal scores: no product was other
                                 // than zero, or only kept blocks compete
  unsigned long long kth64 = 0;
  unsigned total;
  if (!exact) {
    unsigned above = 0, between = 0;
    if (tid == 0) sh.count = 0;
    for (int i = mine0; i < mine1; ++i) {
      above += keys[i] >= in;
      between += keys[i] < in && keys[i] >= maybe;
    }
    block_scan(above | between << 16, sh, &total);  // at most 16384 each
    places = (unsigned)p.topk - (total & 0xffffu);
    const unsigned doubtful = total >> 16;
    if (doubtful == places) {
      in = maybe;  // all of them
      exact = true;
    } else {
      // the doubtful ones again, one per warp, in fp64 and in one fixed order
      for (int d = tid; d < D; d += kThreads) {
        double up = 0., down = 0.;
        const __nv_bfloat16* q = queries + d;
        for (int g = 0; g < p.group; ++g) {
          const float v = __bfloat162float(q[(int64_t)g * D]);
          up += v > 0.f ? v : v == v ? 0.f : v;
          down += v < 0.f ? v : v == v ? 0.f : v;
        }
        sh.up64[d] = up, sh.down64[d] = down;
      }
      const bool few = doubtful <= (unsigned)kFew;
      if (few) {
        for (int i = mine0; i < mine1; ++i)
          if (keys[i] < in && keys[i] >= maybe) sh.few[atomicAdd(&sh.count, 1u)] = i;
      }
      __syncthreads();
      for (int c = warp; c < (few ? (int)doubtful : n); c += kWarps) {
        const int i = few ? sh.few[c] : c;
        if (!few && !(keys[i] < in && keys[i] >= maybe)) continue;
        const int page = __ldg(row + i);
        double s = 0.;
        if (page >= 0 && page < p.num_pages) {
          const __nv_bfloat16* b = bounds + page * page_elems;
#pragma unroll
          for (int d = 0; d < D; d += 32) {
            s = fma(sh.down64[d + lane], (double)__bfloat162float(b[d + lane]), s);
            s = fma(sh.up64[d + lane], (double)__bfloat162float(b[D + d + lane]), s);
          }
        } else {
          s = -(double)INFINITY;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFullMask, s, o);
        if (lane == 0) wide[i] = key64(s);
      }
      __syncthreads();
      if (few) {
        // each against the others: larger first, then the lower index; the
        // places go to the first of them
        bool sel = false;
        int i = 0;
        if (tid < (int)doubtful) {
          i = sh.few[tid];
          unsigned ahead = 0;
          for (unsigned c = 0; c < doubtful; ++c) {
            const int k = sh.few[c];
            ahead += wide[k] > wide[i] || (wide[k] == wide[i] && k < i);
          }
          sel = ahead < places;
        }
        __syncthreads();
        if (tid < (int)doubtful) keys[i] = sel ? kKeep32 : 0u;
        __syncthreads();
        exact = true;
      } else {
        kth64 = select_largest<unsigned long long>(
            n, places, 0ull, ~0ull, sh,
            [&](int i, unsigned long long* k) {
              if (!(keys[i] < in && keys[i] >= maybe)) return false;
              *k = wide[i];
              return true;
            },
            &places);
      }
    }
  }

  // ---- the selected blocks, ascending -----------------------------------------------------
  // `places` of the ties are selected, the lowest indices.  A thread keeps
  // which of its blocks (at most 64) are in, and which are ties, in two words.
  const uint64_t from = only_ties ? (uint64_t)kth + 1 : in;
  uint64_t sures = 0, tied = 0;
  for (int i = mine0; i < mine1; ++i) {
    const uint32_t k = keys[i];
    bool sure = k >= from, tie = only_ties && k == kth;
    if (!exact && !sure && k >= maybe) {
      sure = wide[i] > kth64;
      tie = wide[i] == kth64;
    }
    sures |= (uint64_t)sure << (i - mine0);
    tied |= (uint64_t)tie << (i - mine0);
  }
  const unsigned has = __popcll(sures) | __popcll(tied) << 16;
  const unsigned before = block_scan(has, sh, &total) - has;
  unsigned at = before & 0xffffu;  // places taken before this thread's blocks
  int left = (int)places - (int)(before >> 16);  // ties that still have a place
  at += min(before >> 16, places);
  for (uint64_t todo = sures | tied; todo; todo &= todo - 1) {
    const int bit = __ffsll((long long)todo) - 1;
    if (tied >> bit & 1) {
      if (left-- <= 0) continue;
    }
    if (at < (unsigned)p.topk) out[at] = mine0 + bit;
    ++at;
  }
}

template <int D, int kThreads>
__global__ void __launch_bounds__(kThreads, (D == 256 ? 1 : 2) * 256 / kThreads)
block_select_kernel(const SelectParams p) {
  using Sh = Shared<D, kThreads>;
  constexpr int kWarps = kThreads / 32;
  extern __shared__ __align__(16) uint8_t smem[];
  Sh& sh = *reinterpret_cast<Sh*>(smem);
  // scores of the first CTA: fp32 keys, then fp64 keys, one of each per block
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem + ((sizeof(Sh) + 15) & ~size_t(15)));
  unsigned long long* wide =
      reinterpret_cast<unsigned long long*>(keys + ((p.table_width + 3) & ~3));
  QueryParts<D>& queries_in = *reinterpret_cast<QueryParts<D>*>(wide);
  cg::cluster_group cluster = cg::this_cluster();
  if (p.cluster > 1) cluster.barrier_arrive();
  grid_dependency_sync(0);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = p.cluster > 1 ? (int)(blockIdx.x % p.cluster) : 0;
  const uint32_t unit = blockIdx.x / p.cluster;
  const int t = unit / (uint32_t)p.num_kv;
  const int h = (int)(unit - (uint32_t)t * p.num_kv);
  int* out = p.blocks + (int64_t)unit * p.topk;

  // ---- the token's blocks, and the groups' query sums -----------------------------
  int req = p.requests ? __ldg(p.requests + t) : t;
  int len = __ldg(p.lens + t);
  const __nv_bfloat16* queries = p.q + t * p.q_stride + (int64_t)h * p.group * D;
  bool any_weight = false;
  for (int d = 2 * tid; d < D; d += 2 * kThreads) {  // two dims a thread
    const __nv_bfloat16* q = queries + d;
    float sums[2][2] = {};  // down, up
    for (int g0 = 0; g0 < p.group; g0 += 8) {  // eight loads in flight
      uint32_t v[8];
#pragma unroll
      for (int g = 0; g < 8; ++g)
        v[g] = g0 + g < p.group
                   ? __ldg(reinterpret_cast<const uint32_t*>(q + (int64_t)(g0 + g) * D))
                   : 0u;
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        const float f[2] = {__uint_as_float(v[g] << 16), __uint_as_float(v[g] & 0xffff0000u)};
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // a NaN stays one
          sums[0][k] += f[k] < 0.f ? f[k] : f[k] == f[k] ? 0.f : f[k];
          sums[1][k] += f[k] > 0.f ? f[k] : f[k] == f[k] ? 0.f : f[k];
        }
      }
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const float a = sums[half][0], b = sums[half][1];
      any_weight |= a != 0.f || b != 0.f;
      uint32_t* to = reinterpret_cast<uint32_t*>(&queries_in.part[0][half * D + d]);
      constexpr int COLUMN = D;  // 4-byte words of one part
      const uint32_t hi = pack_bf16x2(a, b);
      const float a1 = a - __uint_as_float(hi << 16), b1 = b - __uint_as_float(hi & 0xffff0000u);
      const uint32_t mid = pack_bf16x2(a1, b1);
      to[0] = hi;
      to[COLUMN] = mid;
      to[2 * COLUMN] =
          pack_bf16x2(a1 - __uint_as_float(mid << 16), b1 - __uint_as_float(mid & 0xffff0000u));
      const __nv_bfloat162 size = __halves2bfloat162(__float2bfloat16_ru(fabsf(a)),
                                                     __float2bfloat16_ru(fabsf(b)));
      to[3 * COLUMN] = *reinterpret_cast<const uint32_t*>(&size);
    }
  }
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
  const int n = (int)(((uint32_t)len + (uint32_t)p.page_size - 1) / (uint32_t)p.page_size);
  if (n <= p.topk) {  // all of them: no score decides anything (cluster-uniform)
    if (rank == 0)
      for (int i = tid; i < p.topk; i += kThreads) out[i] = i < n ? i : -1;
    if (p.cluster > 1) cluster.barrier_wait();
    return;
  }
  // zero queries have zero scores, exactly
  any_weight = __syncthreads_or(any_weight);

  // ---- scores ------------------------------------------------------------------------
  // A warp takes 16 blocks at a time, as the 16 rows of the small matrix
  // instruction: 2 D / 16 steps of bounds (row major, 8 lanes apart a row)
  // against three columns that hold the query sums, split into three bf16
  // parts.  Products of bf16 values are exact; four accumulators keep the
  // running sums, and with them the rounding, small.  A second product, with
  // the signs dropped, and a fourth column give each block's sum of
  // |products|.  Lane l holds
  // values 8(l%4).. of every 32 of rows l/4 and l/4 + 8: the order of the
  // inner dimension does not matter as long as both operands have it.
  // (As fp32 multiply-adds by 32 lanes a block this took 82 instructions a
  // block, with too few loads in flight: 64 tokens x 8 heads of up to 1024
  // blocks 77 us, now 50 us, 202 MB at 4.0 TB/s; one token of 1563 blocks
  // 16 us, now 10 us.)
  constexpr int STEPS = 2 * D / 32;  // of 32 values: two matrix instructions
  uint32_t* to_keys = p.cluster > 1 ? cluster.map_shared_rank(keys, 0) : keys;
  const int g = lane >> 2, c = lane & 3;
  uint4 wb[STEPS];  // column g: a part of the query sums (0-2), their sizes (3), nothing
#pragma unroll
  for (int k = 0; k < STEPS; ++k)
    wb[k] = g < 4 ? *reinterpret_cast<const uint4*>(&queries_in.part[g & 3][32 * k + 8 * c])
                  : make_uint4(0, 0, 0, 0);
  const int* row = p.table + (int64_t)req * p.table_width;
  const __nv_bfloat16* bounds = p.bounds + (int64_t)h * 2 * D + 8 * c;
  const int64_t page_elems = (int64_t)p.num_kv * 2 * D;
  float worst = 0.f;  // the largest sum of |products| seen
  bool odd = false;
  uint32_t least = 0xffffffffu, most = 0;
  const int first = (rank * kWarps + warp) * 16, stride = p.cluster * kWarps * 16;
  int next[2];  // the pages of rows g and g + 8 of the coming blocks
#pragma unroll
  for (int r = 0; r < 2; ++r) next[r] = first + g + 8 * r < n ? __ldg(row + first + g + 8 * r) : -1;
  // the selecting CTA's shared memory has to exist before scores go there
  if (p.cluster > 1) cluster.barrier_wait();
  for (int j0 = first; j0 < n; j0 += stride) {
    int page[2];
    uint4 x[STEPS][2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int j = j0 + g + 8 * r;
      page[r] = next[r];
      next[r] = j + stride < n ? __ldg(row + j + stride) : -1;
      if (page[r] < 0 || page[r] >= p.num_pages) {
        if (j < n && p.errors && c == 0) atomicAdd(p.errors, 1);
        page[r] = -1;
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const __nv_bfloat16* src = bounds + (int64_t)max(page[r], 0) * page_elems;
#pragma unroll
      for (int k = 0; k < STEPS; ++k)
        x[k][r] = page[r] >= 0 ? __ldg(reinterpret_cast<const uint4*>(src + 32 * k))
                               : make_uint4(0, 0, 0, 0);
    }
    float acc[4][4] = {}, size[4] = {};
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
      const uint32_t a0[4] = {x[k][0].x, x[k][1].x, x[k][0].y, x[k][1].y};
      const uint32_t a1[4] = {x[k][0].z, x[k][1].z, x[k][0].w, x[k][1].w};
      uint32_t b0[4], b1[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) b0[i] = a0[i] & 0x7fff7fffu, b1[i] = a1[i] & 0x7fff7fffu;
      mma16816(acc[(2 * k) & 3], a0, wb[k].x, wb[k].y);
      mma16816(acc[(2 * k + 1) & 3], a1, wb[k].z, wb[k].w);
      mma16816(size, b0, wb[k].x, wb[k].y);
      mma16816(size, b1, wb[k].z, wb[k].w);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      // columns 0 and 1 are with c == 0, 2 and 3 with c == 1
      const float left = (acc[0][2 * r] + acc[1][2 * r]) + (acc[2][2 * r] + acc[3][2 * r]);
      const float second =
          (acc[0][2 * r + 1] + acc[1][2 * r + 1]) + (acc[2][2 * r + 1] + acc[3][2 * r + 1]);
      const float upper = __shfl_up_sync(kFullMask, left + second, 1);
      const int j = j0 + g + 8 * r;
      if (c == 1 && j < n) {
        const float s = upper + left, total = size[2 * r + 1];
        odd |= !(total <= 3.0e38f);  // infinite or NaN: fp32 says nothing
        worst = fmaxf(worst, total);
        const bool keep = j < p.keep_first || j >= n - p.keep_last;
        const uint32_t k = keep ? kKeep32 : page[r] >= 0 ? key32(s) : key32(-INFINITY);
        to_keys[j] = k;
        if (!keep) {
          least = min(least, k);
          most = max(most, k);
        }
      }
    }
  }
  // A fp32 score's error, as a share of the sum of |products| S: a matrix
  // instruction adds 16 exact products to a sum of at most S/4 (each of four
  // accumulators has a quarter of the steps); even if every one of them were
  // cut off at 2^-24 of that sum, the 2 D / 16 steps (at most 32) would lose
  // less than 32 * 16 * 2^-24 / 8 = 2^-18 S; taken twice over, and `group`
  // roundings of the query sums and a few of the final sums besides (and
  // products may underflow).
  worst = group_max<32>(worst);
  odd = __any_sync(kFullMask, odd);
  least = __reduce_min_sync(kFullMask, least);
  most = __reduce_max_sync(kFullMask, most);
  if (lane == 0) {
    Sh& to = p.cluster > 1 ? *cluster.map_shared_rank(&sh, 0) : sh;
    const int at = rank * kWarps + warp;
    const float bound = 0x1p-17f + (float)(8 + p.group) * 0x1p-24f;
    to.err[at] = odd ? INFINITY : any_weight ? worst * bound + 1.0e-35f : 0.f;
    to.least[at] = least;
    to.most[at] = most;
  }
  if (p.cluster > 1) {
    cluster.sync();  // every score has arrived; no CTA is needed any longer but the first
    if (rank != 0) return;
  } else {
    __syncthreads();
  }
  select_blocks<D>(p, sh, keys, wide, p.cluster * kWarps, n, queries, row,
                   p.bounds + (int64_t)h * 2 * D, out);
}

template <int D, int kThreads>
size_t smem_bytes(int width) {
  const size_t wide = (size_t)width * 8;
  return ((sizeof(Shared<D, kThreads>) + 15) & ~size_t(15)) + (size_t)((width + 3) & ~3) * 4 +
         (wide > sizeof(QueryParts<D>) ? wide : sizeof(QueryParts<D>));
}

// CTAs of a cluster: more while all of them are resident at once, two to an SM
// (one with heads of 256, and for clusters of eight, which find room later),
// and have more than a tile of blocks for each warp.  4 tokens x 8 kv heads x
// 1024 blocks of 128 dims take 8.7 us in clusters of four, 10.7 in eights; 16
// tokens, 17.2 us in one CTA each, 16.0 in pairs; 8 tokens of 256 dims 16.9 us in
// pairs, 23.3 in fours.  (Several heads to a cluster, warps side by side on a
// page's neighbouring heads, was not faster: of 256 dims and 64 tokens 116 us
// against 99 us, of 128 as fast.)
int cluster_for(int64_t items, int width, int head_dim) {
  int c = 1;
  while (c < kMaxCluster && width > c * 16 * 2 &&
         items * c * 2 <= (head_dim == 256 || c * 2 == 8 ? 152 : 2 * 152))
    c *= 2;
  return c;
}

template <int D, int kThreads>
cudaError_t launch_select(const BlockSelectArgs& a, int cluster, cudaStream_t stream) {
  const PagedQuery& x = a.x;
  static std::atomic<int> cache[kMaxDevices];
  int per_sm = 0;
  // one opt-in for the largest size that the validation lets through
  const cudaError_t e =
      tma::prepare(block_select_kernel<D, kThreads>, kThreads,
                   smem_bytes<D, kThreads>(kMaxSelectBlocks), cache, &per_sm);
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
  p.cluster = cluster;
  return launch_clusters(block_select_kernel<D, kThreads>, dim3((unsigned)(items * cluster)),
                         dim3(kThreads), smem_bytes<D, kThreads>(x.table_width), cluster, stream,
                         p);
}

// More items than CTAs that are resident at once: CTAs of half the threads, of
// which twice as many are, so that some select while others score.  256 tokens
// x 8 heads of 128 dims, 64 blocks 28 us against 46, 256 blocks 60 against 76;
// 64 tokens, 1024 blocks 49.8 / 51.3 (of 64 dims 27.5 / 30.0, of 256 91 / 99),
// 2048 blocks, which therefore keep the larger, 128 / 99.
template <int D>
cudaError_t launch_select(const BlockSelectArgs& a, cudaStream_t stream) {
  const int64_t items = (int64_t)a.x.num_tokens * a.x.num_heads_kv;
  if (items > (D == 256 ? 152 : 2 * 152) && a.x.table_width <= 1024)
    return launch_select<D, 128>(a, 1, stream);
  return launch_select<D, 256>(a, cluster_for(items, a.x.table_width, D), stream);
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
