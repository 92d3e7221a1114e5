// kvq_paged_attn.cu -- attention of few query rows over keys and values read
// from the paged cache: the selected blocks of block-sparse attention, the
// own keys of each token of shared-prefix attention, and the prefix itself
// where few rows share it.
//
// One cluster of 1..8 CTAs takes up to 16 query rows of one kv head and the
// pages that any of them sees, its CTAs a part each.  The rows are either the
// heads of one token's group (block-sparse), or 16 consecutive (token, head of
// the group) pairs: then the prefix's pages are seen by all rows and a token's
// own pages by its rows alone, in one sweep and one softmax.  A CTA first
// lists its part's pages in shared memory ({page, valid keys, whose}), so that
// no table lookup stands between a page and its loads.  Then each of its warps
// works alone, on every kWarps-th group of 16 keys, with an online softmax of
// its own:
//   * K and V rows of the group come in by 16-byte asynchronous copies, three
//     groups deep (heads of 256: one and a half), into a shared-memory ring
//     that only this warp uses, so there is no CTA barrier in the loop; a
//     16-byte fragment c of row r is stored at c ^ (r & 7), which keeps the
//     matrix loads free of bank conflicts;
//   * S = Q K^T and O += P V are 16x8x16 matrix instructions, fp32
//     accumulators; the P fragments are the S fragments, rounded once to
//     bf16 (the row sum adds the unrounded fp32 values);
//   * keys past a page's valid count are neither read nor weighted: their
//     rows are filled with zeros and their scores set to -inf.
// The warps' states are joined in shared memory, the CTAs' through the
// cluster's shared memory (one launch, no workspace).  Only where a cluster
// per 16 rows would leave most of the GPU idle on a long range is the range
// split further, into partials for the join kernel.  Where the prefix was
// taken by the tensor-core tiles, this kernel runs behind theirs for the own
// keys and joins their partials to its rows as it writes them.
//
// Bound by the reading of K and V: 16 rows of products per key row keep the
// tensor pipes a fifth busy, which is why the small matrix instruction is
// enough here and one tile of 16 rows is as cheap as one row.  64 sequences x 8
// kv heads x 4096 selected keys of 128 dims, 1.07 GB: 158-163 us, 6.6-6.8 TB/s;
// of 256 dims, 2.15 GB: 300 us (one CTA an SM with two whole groups a warp, 347
// us; three CTAs of two warps, 399 us).
// Short ranges are bound by latency instead: about 5 us from a CTA's start to
// its end (length, page table, keys: three dependent reads; two joins).  Two
// warps a CTA, two or four stages, three CTAs to an SM and an L2 prefetch of
// the first pages each lost 5-40 % on one of the sizes and won on few.
#include <cooperative_groups.h>

#include "kvq_mma.cuh"
#include "kvq_paged_attn.cuh"
#include "kvq_tma.cuh"

namespace cg = cooperative_groups;

namespace kvq {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxCluster = 8;
constexpr int kRows = 16;         // query rows of a CTA
constexpr int kGroup = 16;        // keys of one step of a warp
constexpr int kFlight = 8;        // parts of the prefix that a thread loads together
constexpr int kSoloPages = 512;   // .. where it is a single warp

// Whose a listed page is: of all rows, or of the rows of one token of the tile.
constexpr int kAllRows = 31;
constexpr int kValidBits = 20;  // valid keys of a page: at most 2^16

struct AttnParams {
  const __nv_bfloat16* q;
  int64_t q_stride;
  const __nv_bfloat16* cache;
  int num_q, num_kv, group;  // group = num_q / num_kv
  int tiles;                 // row tiles of a kv head (of a token and kv head: block-sparse)
  int units;                 // row tiles in all
  int num_tokens;
  int64_t num_pages;
  int page_size;
  int page_shift;            // log2 of page_size, -1: not a power of two
  const int* table;
  int num_requests, table_width;
  const int* requests;
  const int* lens;
  // block-sparse
  const int* blocks;
  int topk;
  // shared prefix
  const int* prefix_pages;
  int prefix_len;
  float scale_log2;
  int cluster, splits;
  // The result goes to `out`, joined with `prefix_parts` partials of the
  // prefix (0: none); with several splits it goes to partials itself.
  __nv_bfloat16* out;
  int prefix_parts;
  int prefix_ctas;  // .. from so many CTAs
  Partials parts;
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

// Clears the values of keys outside `keep` in a V fragment: registers 0 and 2
// hold keys 2(lane%4) and the next, registers 1 and 3 those 8 further.
__device__ __forceinline__ void keep_keys(uint32_t b[4], uint32_t keep, int lane) {
  const uint32_t k = keep >> (2 * (lane & 3));
  const uint32_t lo = (k & 1 ? 0xffffu : 0u) | (k & 2 ? 0xffff0000u : 0u);
  const uint32_t hi = (k & 0x100 ? 0xffffu : 0u) | (k & 0x200 ? 0xffff0000u : 0u);
  b[0] &= lo, b[2] &= lo;
  b[1] &= hi, b[3] &= hi;
}

// How many 16-key groups or rows fit, and where they lie.
template <int D>
struct Shape {
  // CTAs of an SM: four of 64 dims (a shorter list; three with one of 2048 pages:
  // 64 sequences x 8 kv heads x 4096 keys 114 us against 89)
  static constexpr int kCtas = D == 64 ? 4 : 2;
  static constexpr int kMaxPages = D == 64 ? 512 : 2048;  // pages a CTA lists at a time
  // A warp's ring holds K and V of three steps; with heads of 256 a step and a
  // half, three tiles that keys and values take in turn, so that two CTAs fit.
  static constexpr bool kHalf = D == 256;
  static constexpr int kStages = 3;
  static constexpr int kPad = D + 8;                  // fp32 values of an output row: rows
                                                      // 32 bytes apart in the banks
  static constexpr int kTile = kGroup * D * 2;        // bytes of 16 K (or V) rows
  static constexpr int kStage = 2 * kTile;            // K, then V
  static constexpr int kRing = kStages * (kHalf ? kTile : kStage);
  static constexpr int kList = kMaxPages * 8;         // {page, valid keys}
  static constexpr int kState = kWarps * kRows * 8;   // {m, l} per warp and row
  static constexpr int kLse = kRows * 4;              // of the CTA's part, per row
  static constexpr int kSmem = kWarps * kRing + kList + kState + kLse;
  static constexpr int kSoloSmem = kRing + kSoloPages * 8;
  static_assert(kRing >= kRows * kPad * 4, "a warp's output fits in its ring");
  static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
};

// The reference of a row's join with the prefix's parts, and the sum of all
// weights; `lse` is the row's own part.
__device__ __forceinline__ float parts_top(const AttnParams& p, int64_t row, float lse,
                                           float* sum) {
  float top = lse;
  for (int s = 0; s < p.prefix_parts; ++s) top = fmaxf(top, p.parts.lse[s * p.parts.rows + row]);
  const float ref = top == -INFINITY ? 0.f : top;
  *sum = exp2f(lse - ref);
  for (int s = 0; s < p.prefix_parts; ++s)
    *sum += exp2f(p.parts.lse[s * p.parts.rows + row] - ref);
  return ref;
}

// Joins four dims of a row (its own part's, normalised, in *v) with the
// prefix's parts; they lie at p.parts.o[at + s * part_stride].  A part without
// a key (its output may be unwritten) stays out.  One sweep with a running
// reference, so that the sums and outputs of several parts are in flight
// together (with four instead of eight, 20 to 40 parts take 2-4 us longer).
__device__ __forceinline__ void add_parts(const AttnParams& p, int64_t row, int64_t at,
                                          int64_t part_stride, float lse, float4* v) {
  float top = lse, sum = lse == -INFINITY ? 0.f : 1.f;
  float4 a = *v;  // zeros where there is no own key
  for (int s0 = 0; s0 < p.prefix_parts; s0 += kFlight) {
    float w[kFlight];
    float4 x[kFlight];
    const float old = top;
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      w[u] = -INFINITY;
      if (s0 + u < p.prefix_parts) {
        w[u] = p.parts.lse[(s0 + u) * p.parts.rows + row];
        x[u] = *reinterpret_cast<const float4*>(p.parts.o + at + (s0 + u) * part_stride);
      }
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u) top = fmaxf(top, w[u]);
    const float ref = top == -INFINITY ? 0.f : top;
    const float f = old == top ? 1.f : exp2f(old - ref);
    sum *= f;
    a.x *= f, a.y *= f, a.z *= f, a.w *= f;
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      if (w[u] == -INFINITY) continue;
      const float g = exp2f(w[u] - ref);
      sum += g;
      a.x = fmaf(g, x[u].x, a.x), a.y = fmaf(g, x[u].y, a.y);
      a.z = fmaf(g, x[u].z, a.z), a.w = fmaf(g, x[u].w, a.w);
    }
  }
  const float f = sum == 0.f ? 0.f : 1.f / sum;
  *v = make_float4(a.x * f, a.y * f, a.z * f, a.w * f);
}

// SPARSE: the rows of one token's group and the blocks selected for them;
// otherwise a tile of (token, head) pairs, the prefix and their own keys.
// WHOLE: page_size is a multiple of 16, so a group of keys lies in one page.
// SOLO: every warp has a row tile to itself (no cluster, no parts).
template <int D, bool SPARSE, bool WHOLE, bool SOLO>
__global__ void __launch_bounds__((SOLO ? 1 : kWarps) * 32) paged_attn_kernel(const AttnParams p) {
  using S = Shape<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  // After the prefix's tiles: they let this kernel be scheduled only when what
  // came before both is done, and it needs their partials at its end alone.
  const bool late = !SPARSE && p.prefix_parts > 0;
  if (!late) grid_dependency_sync(p.trigger_from);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kTeam = SOLO ? 1 : kWarps;  // warps on a row tile
  int2* list = reinterpret_cast<int2*>(smem + kTeam * S::kRing);
  float2* state = reinterpret_cast<float2*>(smem + kWarps * S::kRing + S::kList);
  float* part_lse = reinterpret_cast<float*>(smem + kWarps * S::kRing + S::kList + S::kState);
  const int rank = !SOLO && p.cluster > 1 ? (int)(blockIdx.x % p.cluster) : 0;
  const int unit = SOLO ? (int)blockIdx.x : (int)blockIdx.x / p.cluster;

  // ---- which rows -----------------------------------------------------------------
  // row r is row flat0 + r of the kv head's (token, head of the group) pairs
  const uint32_t group = p.group;
  const int tile = unit % p.tiles, per = unit / p.tiles;
  const int kv_head = SPARSE ? per % p.num_kv : per;
  const uint32_t flat0 = SPARSE ? (uint32_t)(per / p.num_kv) * group + tile * kRows
                                : (uint32_t)tile * kRows;
  const uint32_t flat_end = SPARSE ? (uint32_t)(per / p.num_kv + 1) * group
                                   : (uint32_t)p.num_tokens * group;
  const int rows = (int)min((uint32_t)kRows, flat_end - flat0);
  const int t0 = SPARSE ? per / p.num_kv : (int)(flat0 / group);  // the first row's token
  const int in0 = (int)(flat0 - (uint32_t)t0 * group);            // and its place in the group
  // row r's token, less t0 (block-sparse: one token), and its output row
  auto token_of = [&](int r) { return SPARSE ? 0 : (int)((uint32_t)(in0 + r) / group); };
  auto row_of = [&](int r) {  // token * num_q + head
    const int u = token_of(r);
    return (int64_t)(t0 + u) * p.num_q + kv_head * (int)group + (in0 + r - u * (int)group);
  };

  // ---- whose pages: lane i has token t0 + i of the tile --------------------------------
  const int tokens = token_of(rows - 1) + 1;
  int req = 0, len = 0;
  if (lane < tokens) {
    req = p.requests ? __ldg(p.requests + t0 + lane) : t0 + lane;
    len = __ldg(p.lens + t0 + lane);
  }

  // ---- Q fragments ---------------------------------------------------------------
  // a lane holds rows lane/4 and lane/4 + 8, dims 16k + 2(lane%4) + {0, 1, 8, 9}
  uint32_t qf[D / 16][4];
  int mine[2];  // the row's token, less t0; -1: no row
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = (lane >> 2) + 8 * i;
    const int u = token_of(r);
    mine[i] = r < rows ? u : -1;
    const __nv_bfloat16* src =
        p.q + (int64_t)(t0 + u) * p.q_stride +
        (int64_t)(kv_head * (int)group + in0 + r - u * (int)group) * D + 2 * (lane & 3);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      qf[k][i] = r < rows ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * k)) : 0u;
      qf[k][2 + i] = r < rows ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * k + 8)) : 0u;
    }
  }

  // ---- which pages -----------------------------------------------------------------
  // a page index and a place in it (the quotient fits 32 bits: checked at launch)
  const uint32_t page_size = p.page_size;
  const int shift = p.page_shift;
  auto pages_of = [&](uint32_t keys) {  // pages that hold `keys` keys
    const uint32_t up = keys + page_size - 1;
    return (int)(shift >= 0 ? up >> shift : up / page_size);
  };
  bool rejected = false;
  {
    const int64_t room = (int64_t)p.table_width * p.page_size;
    if (lane < tokens && (req < 0 || req >= p.num_requests || len < 0)) {
      rejected = true;
      req = len = 0;
    } else if (len > room) {
      rejected = true;
      len = (int)room;
    }
  }
  // pages of the lane's token, and where they end in the tile's list
  int end = SPARSE ? (lane == 0 && len > 0 ? p.topk : 0) : pages_of(len);
  if (!SPARSE) {
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
      const int v = __shfl_up_sync(kFullMask, end, o);
      if (lane >= o) end += v;
    }
  }
  const int prefix = SPARSE ? 0 : pages_of(p.prefix_len);
  const int pages = prefix + __shfl_sync(kFullMask, end, SPARSE ? 0 : 15);
  const int parts = p.cluster * p.splits;
  const int share = parts == 1 ? pages : (int)(((uint32_t)pages + parts - 1) / (uint32_t)parts);
  const int64_t begin = (int64_t)share * (blockIdx.y * p.cluster + rank);
  const int page0 = (int)min(begin, (int64_t)pages);
  const int page_end = page0 + min(share, pages - page0);

  float o[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int k = 0; k < 4; ++k) o[n][k] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  // as many pages at a time as the list holds: usually all of them
  constexpr int kCapacity = SOLO ? kSoloPages : S::kMaxPages;
  for (int page_lo = page0; page_lo < page_end; page_lo += kCapacity) {
    const int listed = min(kCapacity, page_end - page_lo);
    if (page_lo != page0) {  // the list is no longer read
      if (SOLO) __syncwarp(); else __syncthreads();
    }
    for (int i0 = 0; i0 < listed; i0 += kTeam * 32) {
      const int i = i0 + (SOLO ? lane : (int)threadIdx.x);
      const int at = page_lo + i - prefix;  // among the tokens' own pages
      // the token whose pages hold `at`: the number of tokens that end before
      int tok = 0, skip = 0;
      if (!SPARSE) {
        for (int k = 0; k + 1 < tokens; ++k) tok += at >= __shfl_sync(kFullMask, end, k);
        skip = __shfl_sync(kFullMask, end, max(tok - 1, 0));
        if (tok == 0) skip = 0;
      }
      const int r = __shfl_sync(kFullMask, req, tok), n = __shfl_sync(kFullMask, len, tok);
      int page = 0, valid = 0, whose = kAllRows;
      if (i < listed) {
        if (SPARSE) {
          const int b = __ldg(p.blocks + ((int64_t)t0 * p.num_kv + kv_head) * p.topk + page_lo + i);
          if (b >= 0 && (int64_t)b * p.page_size < n) {
            page = __ldg(p.table + (int64_t)r * p.table_width + b);
            valid = min(p.page_size, n - b * p.page_size);
          } else if (b != -1) {
            rejected = true;
          }
        } else if (at < 0) {
          page = __ldg(p.prefix_pages + page_lo + i);
          valid = (int)min((int64_t)p.page_size,
                           p.prefix_len - (int64_t)(page_lo + i) * p.page_size);
        } else {
          page = __ldg(p.table + (int64_t)r * p.table_width + (at - skip));
          valid = (int)min((int64_t)p.page_size, n - (int64_t)(at - skip) * p.page_size);
          whose = tok;
        }
        if (valid > 0 && (page < 0 || page >= p.num_pages)) {
          rejected = true;
          valid = 0;
        }
        list[i] = make_int2(page, valid | whose << kValidBits);
      }
    }
    if (SOLO) __syncwarp(); else __syncthreads();

    // ---- the warp's groups of keys ---------------------------------------------------
    const uint32_t total = (uint32_t)listed * page_size;  // below 2^31
    const int steps = (int)((total + kGroup * kTeam - 1) / (kGroup * kTeam));
    const int member = SOLO ? 0 : warp;  // of the team
    const uint32_t ring = tma::smem_addr(smem) + warp * S::kRing;
    const int64_t head_elems = (int64_t)p.page_size * D;
    const int64_t v_from_k = p.num_kv * head_elems;
    auto entry_of = [&](uint32_t key, int* off) {
      const uint32_t at = shift >= 0 ? key >> shift : key / page_size;
      *off = (int)(key - at * page_size);
      return list[at];
    };

    // Where step i's keys and values lie.
    auto k_tile = [&](int i) {
      return ring + (S::kHalf ? 2 * i % S::kStages * S::kTile : i % S::kStages * S::kStage);
    };
    auto v_tile = [&](int i) {
      return S::kHalf ? ring + (2 * i + 1) % S::kStages * S::kTile : k_tile(i) + S::kTile;
    };
    // Starts the copies of step i's 16 keys, their values, or both.
    auto issue = [&](int i, bool keys, bool values) {
      const uint32_t k0 = (uint32_t)(i * kTeam + member) * kGroup;
      const uint32_t kt = k_tile(i), vt = v_tile(i);
      constexpr int FRAGS = D / 8;                          // 16-byte fragments of a row
      constexpr int RPI = 32 / FRAGS > 0 ? 32 / FRAGS : 1;  // rows of one warp-wide copy
      const int r0 = lane / FRAGS, c = lane % FRAGS;
      if (WHOLE) {
        int there = 0;  // keys of the group that exist
        const __nv_bfloat16* src = p.cache + 8 * c;
        if (i < steps && k0 < total) {
          int off;
          const int2 e = entry_of(k0, &off);
          there = (e.y & ((1 << kValidBits) - 1)) - off;
          if (there > 0)
            src += ((int64_t)e.x * 2 * p.num_kv + kv_head) * head_elems + (int64_t)(off + r0) * D;
        }
#pragma unroll
        for (int j = 0; j < kGroup / RPI; ++j) {
          const int r = j * RPI + r0;
          const bool ok = r < there;
          const __nv_bfloat16* from = ok ? src + j * RPI * D : p.cache;
          const uint32_t at = r * (2 * D) + ((c ^ (r & 7)) << 4);
          if (keys) cp_async16(kt + at, from, ok);
          if (values) cp_async16(vt + at, ok ? from + v_from_k : from, ok);
        }
      } else {
        int64_t row = -1;  // lane r < 16 finds row r's place
        if (lane < kGroup && i < steps && k0 + lane < total) {
          int off;
          const int2 e = entry_of(k0 + lane, &off);
          if (off < (e.y & ((1 << kValidBits) - 1)))
            row = ((int64_t)e.x * 2 * p.num_kv + kv_head) * head_elems + (int64_t)off * D;
        }
#pragma unroll
        for (int j = 0; j < kGroup / RPI; ++j) {
          const int r = j * RPI + r0;
          const int64_t from = __shfl_sync(kFullMask, row, r);
          const __nv_bfloat16* src = p.cache + (from < 0 ? 0 : from + 8 * c);
          const uint32_t at = r * (2 * D) + ((c ^ (r & 7)) << 4);
          if (keys) cp_async16(kt + at, src, from >= 0);
          if (values) cp_async16(vt + at, from >= 0 ? src + v_from_k : src, from >= 0);
        }
      }
      cp_commit();
    };

#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i) {
      if (S::kHalf) issue(0, i == 0, i == 1);
      else issue(i, true, true);
    }
    // heads of 256: the next step's values take the place of the keys
    auto next_values = [&](int i) {
      __syncwarp();
      issue(i + 1, false, true);
      cp_wait<S::kStages - 1>();
      __syncwarp();
    };
    for (int i = 0; i < steps; ++i) {
      if (S::kHalf) issue(i + 1, true, false);
      else issue(i + S::kStages - 1, true, true);
      cp_wait<S::kStages - 1>();
      __syncwarp();
      // whose the step's keys are: lane r < 16 for key r, -2 where there is none
      const uint32_t k0 = (uint32_t)(i * kTeam + member) * kGroup;
      int whose = -2;
      uint32_t todo;  // the keys that exist
      if (WHOLE) {
        int there = 0;
        if (k0 < total) {
          int off;
          const int e = entry_of(k0, &off).y;
          there = (e & ((1 << kValidBits) - 1)) - off;
          whose = e >> kValidBits;
        }
        todo = there >= kGroup ? 0xffffu : there > 0 ? (1u << there) - 1u : 0u;
      } else {
        if (lane < kGroup && k0 + lane < total) {
          int off;
          const int e = entry_of(k0 + lane, &off).y;
          if (off < (e & ((1 << kValidBits) - 1))) whose = e >> kValidBits;
        }
        todo = __ballot_sync(kFullMask, whose != -2);
      }
      if (todo == 0) {
        if (S::kHalf) next_values(i);
        else __syncwarp();
        continue;
      }
      const uint32_t kt = k_tile(i), vt = v_tile(i);
      float raw[2][4] = {};
      {
        const int r = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t b[4];
          ldmatrix4(b, kt + r * (2 * D) + (((2 * k + half) ^ (r & 7)) << 4));
          mma16816(raw[0], qf[k], b[0], b[1]);
          mma16816(raw[1], qf[k], b[2], b[3]);
        }
      }
      if (S::kHalf) next_values(i);
      // one round for all keys that the same rows see: a single one but where
      // small pages of several tokens share the step
      constexpr bool kMayMix = !SPARSE && !WHOLE;
      const int first_seen_by = kMayMix ? __shfl_sync(kFullMask, whose, __ffs(todo) - 1) : 0;
      const bool mixed =
          kMayMix && __any_sync(kFullMask, whose != -2 && whose != first_seen_by);
      while (todo) {
        const int seen_by = SPARSE ? kAllRows
                            : WHOLE ? whose : __shfl_sync(kFullMask, whose, __ffs(todo) - 1);
        const uint32_t mask = kMayMix ? __ballot_sync(kFullMask, whose == seen_by) : todo;
        todo &= ~mask;
        bool sees[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) sees[h] = SPARSE || seen_by == kAllRows || seen_by == mine[h];
        // scores in units of log2: s * scale * log2(e); keys not seen -inf
        float s[2][4];
        float top[2] = {m[0], m[1]};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int key = 8 * n + 2 * (lane & 3) + (k & 1);
            s[n][k] = sees[k >> 1] && ((mask >> key) & 1) ? raw[n][k] * p.scale_log2 : -INFINITY;
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
        const int r = (lane & 7) + (((lane >> 3) & 1) << 3), half = lane >> 4;
        if (SPARSE || seen_by == kAllRows) {
          // zeros in V where there is no key, and every row sees the others
          // (in a mixed step the others' keys have weight 0 here, but a NaN
          // value of theirs would not stay out: they are cleared)
          const uint32_t keep = mixed ? mask : 0xffffu;
#pragma unroll
          for (int n = 0; n < D / 16; ++n) {
            uint32_t b[4];
            ldmatrix4_trans(b, vt + r * (2 * D) + (((2 * n + half) ^ (r & 7)) << 4));
            if (kMayMix && mixed) keep_keys(b, keep, lane);
            mma16816(o[2 * n], pf, b[0], b[1]);
            mma16816(o[2 * n + 1], pf, b[2], b[3]);
          }
        } else {
          // other tokens' rows keep their sums whatever these values are (a
          // zero weight times an infinite or NaN value would reach them)
#pragma unroll
          for (int n = 0; n < D / 16; ++n) {
            uint32_t b[4];
            ldmatrix4_trans(b, vt + r * (2 * D) + (((2 * n + half) ^ (r & 7)) << 4));
            if (kMayMix && mixed) keep_keys(b, mask, lane);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              float x[4] = {o[2 * n + u][0], o[2 * n + u][1], o[2 * n + u][2], o[2 * n + u][3]};
              mma16816(x, pf, b[2 * u], b[2 * u + 1]);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (sees[k >> 1]) o[2 * n + u][k] = x[k];
            }
          }
        }
      }
      __syncwarp();  // the stage is read before its next copies start
    }
    cp_wait<0>();
  }
  if (rejected && p.errors) atomicAdd(p.errors, 1);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(kFullMask, l[h], 1);
    l[h] += __shfl_xor_sync(kFullMask, l[h], 2);
    if (!SOLO && (lane & 3) == 0)
      state[warp * kRows + (lane >> 2) + 8 * h] = make_float2(m[h], l[h]);
  }
  if (late) {
    grid_dependency_wait();
    if ((int)blockIdx.x >= p.trigger_from) launch_dependents();
  }
  if (SOLO) {  // the rows are this warp's: straight from its registers
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = (lane >> 2) + 8 * h;
      if (r >= rows) continue;
      const int64_t row = row_of(r);
      float f = l[h] == 0.f ? 0.f : 1.f / l[h];  // 0: the row has no key
      if (late) {
        const float lse =
            l[h] == 0.f ? -INFINITY : (m[h] == -INFINITY ? 0.f : m[h]) + log2f(l[h]);
        float sum;
        const float ref = parts_top(p, row, lse, &sum);
        f = lse == -INFINITY ? 0.f : f * exp2f(lse - ref);
#pragma unroll
        for (int n = 0; n < D / 8; ++n) o[n][2 * h] *= f, o[n][2 * h + 1] *= f;
        for (int s = 0; s < p.prefix_parts; ++s) {
          const float part = p.parts.lse[s * p.parts.rows + row];
          if (part == -INFINITY) continue;
          const float w = exp2f(part - ref);
          const float* from = p.parts.o + (s * p.parts.rows + row) * D + 2 * (lane & 3);
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            const float2 x = *reinterpret_cast<const float2*>(from + 8 * n);
            o[n][2 * h] = fmaf(w, x.x, o[n][2 * h]);
            o[n][2 * h + 1] = fmaf(w, x.y, o[n][2 * h + 1]);
          }
        }
        f = sum == 0.f ? 0.f : 1.f / sum;
      }
      __nv_bfloat16* dst = p.out + row * D + 2 * (lane & 3);
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<uint32_t*>(dst + 8 * n) =
            pack_bf16x2(o[n][2 * h] * f, o[n][2 * h + 1] * f);
    }
    return;
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
    float* dst = reinterpret_cast<float*>(smem + warp * S::kRing) + r * S::kPad + 2 * (lane & 3);
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
      *reinterpret_cast<float2*>(dst + 8 * n) = make_float2(o[n][2 * h] * f, o[n][2 * h + 1] * f);
    if (warp == 0 && (lane & 3) == 0)
      part_lse[r] = sum == 0.f ? -INFINITY : ref + log2f(sum);
  }
  __syncthreads();
  // the CTA's part: the sum of its warps', which are scaled to one reference
  const bool joined = p.cluster > 1;
  float* own_o = reinterpret_cast<float*>(smem);
  auto warps_sum = [&](int at) {
    float4 v = *reinterpret_cast<const float4*>(own_o + at);
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 u = *reinterpret_cast<const float4*>(smem + w * S::kRing + 4 * at);
      v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
    return v;
  };
  const int all = rows * (D / 4);  // 16-byte pieces of the rows
  if (joined) {
#pragma unroll 4
    for (int i = threadIdx.x; i < all; i += kWarps * 32) {
      const int at = i / (D / 4) * S::kPad + 4 * (i % (D / 4));
      *reinterpret_cast<float4*>(own_o + at) = warps_sum(at);
    }
    cluster.sync();
  }
  // each CTA of the cluster writes a slice of the rows
  const int slice = joined ? (all + p.cluster - 1) / p.cluster : all;
  const int last = min((rank + 1) * slice, all);
#pragma unroll 2
  for (int i = rank * slice + threadIdx.x; i < last; i += kWarps * 32) {
    const int r = i / (D / 4), c = 4 * (i % (D / 4)), at = r * S::kPad + c;
    float4 v;
    float lse;
    if (joined) {
      float part[kMaxCluster], top = -INFINITY, sum = 0.f;
      float4 u[kMaxCluster];
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        part[k] = -INFINITY;
        if (k < p.cluster) {
          part[k] = cluster.map_shared_rank(part_lse, k)[r];
          u[k] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(own_o, k) + at);
        }
        top = fmaxf(top, part[k]);
      }
      const float ref = top == -INFINITY ? 0.f : top;
      v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        if (part[k] == -INFINITY) continue;  // a part without a key
        const float w = exp2f(part[k] - ref);
        sum += w;
        v.x = fmaf(w, u[k].x, v.x), v.y = fmaf(w, u[k].y, v.y);
        v.z = fmaf(w, u[k].z, v.z), v.w = fmaf(w, u[k].w, v.w);
      }
      const float f = sum == 0.f ? 0.f : 1.f / sum;
      v.x *= f, v.y *= f, v.z *= f, v.w *= f;
      lse = sum == 0.f ? -INFINITY : ref + log2f(sum);
    } else {
      v = warps_sum(at);
      lse = part_lse[r];
    }
    const int64_t row = row_of(r);
    if (p.splits == 1) {
      if (late) add_parts(p, row, row * D + c, (int64_t)D * p.parts.rows, lse, &v);
      *reinterpret_cast<uint2*>(p.out + row * D + c) =
          make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    } else {
      const int64_t slot = blockIdx.y;
      *reinterpret_cast<float4*>(p.parts.o + (slot * p.parts.rows + row) * D + c) = v;
      if (c == 0) p.parts.lse[slot * p.parts.rows + row] = lse;
    }
  }
  if (joined) cluster.sync();  // no CTA ends while its part is being read
}

// ---- the join of the parts -------------------------------------------------------------

struct JoinParams {
  Partials parts;
  int slots;
  __nv_bfloat16* out;
  int trigger_from;
};

// One warp per row.  The lanes fetch the parts' sums together, 32 parts at a
// time, and then the outputs, eight parts in flight.
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
  for (int s0 = 0; s0 < p.slots; s0 += 32) {
    const float lse =
        s0 + lane < p.slots ? p.parts.lse[(s0 + lane) * p.parts.rows + row] : -INFINITY;
    // a part without a key (its output may be unwritten) stays out; a weight of
    // 0 does not: a NaN output still counts
    const uint32_t full = __ballot_sync(kFullMask, lse != -INFINITY);
    const float weight = exp2f(lse - ref);
    const float* from = p.parts.o + (s0 * p.parts.rows + row) * D + V * lane;
    const int count = min(32, p.slots - s0);
    for (int s = 0; s < count; s += 8) {
      float v[8][V];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const bool there = s + u < count && (full >> (s + u) & 1);
#pragma unroll
        for (int k = 0; k < V; k += 2) {
          const float2 x = there ? *reinterpret_cast<const float2*>(
                                       from + (int64_t)(s + u) * p.parts.rows * D + k)
                                 : make_float2(0.f, 0.f);
          v[u][k] = x.x, v[u][k + 1] = x.y;
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float w = __shfl_sync(kFullMask, weight, (s + u) & 31);
        if (s + u < count && (full >> (s + u) & 1)) {
          sum += w;
#pragma unroll
          for (int k = 0; k < V; ++k) acc[k] = fmaf(w, v[u][k], acc[k]);
        }
      }
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

// How a launch of `units` row tiles over up to `pages` pages each is spread.
struct Spread {
  int cluster, splits;
  bool solo;  // a warp per row tile
};

// CTAs are added while all of them are resident at once, two to an SM of the
// part's 152 (heads of 64 have four, but these numbers; with half as many again
// in a second wave the same range took 20-30 % longer, with twice as many, 24 us
// against 10.4) and each keeps at least two steps of 16
// keys for every warp: first within a cluster of up to 8 (joined in place);
// beyond that, as partials that a second launch joins, only where a CTA would
// be left with more than 2048 keys (below, the second launch costs more than it
// saves).  Behind the prefix's tiles (`late`) the SMs come free one by one, and
// eight seats of a cluster late: there four serve up to 8192 keys (16 tokens of
// 32 heads of 128 after 2048 keys, own keys 64: 14.2 us against 19.4; 640: 17.2
// / 22.4; 2048, more than that: 34.8 / 29.2).
Spread spread_for(int64_t units, int64_t pages, int page_size, bool late) {
  Spread s = {1, 1, false};
  const int64_t keys = pages * page_size;
  const int most = late && keys < 8192 ? kMaxCluster / 2 : kMaxCluster;
  // clusters resident at once: larger ones do not fill the SMs evenly
  auto fit = [](int cluster) { return cluster == 8 ? 36 : cluster == 4 ? 74 : 2 * 152 / cluster; };
  while (s.cluster < most && units <= fit(s.cluster * 2) &&
         keys >= (int64_t)s.cluster * 2 * kGroup * kWarps)
    s.cluster *= 2;
  int64_t splits = 1;
  while (!late && units * s.cluster * (splits + 1) <= 2 * 152 &&
         keys > s.cluster * splits * 2048)
    ++splits;
  s.splits = (int)splits;
  // With many tiles of short ranges, a CTA of one warp each: no joins between
  // warps, and four times as many tiles in flight (640 tiles of 512 keys 32 us
  // against 38 us, of 1024 keys 58 against 66; 1024 tiles of up to 200 keys 38
  // against 51).  Longer ranges keep the four warps: the last tiles of a wave
  // take four times as long on one (1280 tiles of 1024 keys 127 us against
  // 108; 1024 tiles of 2 to 1152 keys 91 against 82).
  s.solo = units >= 4 * 152 && keys <= 512;
  return s;
}

template <int D, bool SPARSE, bool WHOLE, bool SOLO>
cudaError_t launch_attn(AttnParams p, cudaStream_t stream) {
  static std::atomic<int> cache[kMaxDevices];
  int per_sm = 0;
  constexpr int threads = SOLO ? 32 : kWarps * 32;
  constexpr int most = 110 * 1024;
  int smem = SOLO ? Shape<D>::kSoloSmem : Shape<D>::kSmem;
  const cudaError_t e = tma::prepare(paged_attn_kernel<D, SPARSE, WHOLE, SOLO>, threads, smem,
                                     cache, &per_sm, most);
  if (e != cudaSuccess) return e;
  const int64_t ctas = (int64_t)p.units * p.cluster, wave = (int64_t)per_sm * device_sm_count();
  p.trigger_from = ctas > wave ? (int)(ctas - wave) : 0;
  // Behind the prefix's tiles, where these have most SMs, the SMs come free one
  // by one: the first shall not take four CTAs if two on each are enough (33 x 3
  // tokens of 64 dims 27.6 us against 32.3; where the tiles leave SMs free, 64
  // tokens of 32 heads after 2048 keys, 17.7 us against 14.2).
  if (p.prefix_ctas > 76 && ctas <= 2 * 152 && smem < most) smem = most;
  return launch_clusters(paged_attn_kernel<D, SPARSE, WHOLE, SOLO>,
                         dim3((unsigned)ctas, (unsigned)p.splits), dim3(threads), smem, p.cluster,
                         stream, p);
}

template <int D, bool SPARSE>
cudaError_t launch_attn_page(const AttnParams& p, bool solo, cudaStream_t stream) {
  if (p.page_size % kGroup != 0) return launch_attn<D, SPARSE, false, false>(p, stream);
  return solo ? launch_attn<D, SPARSE, true, true>(p, stream)
              : launch_attn<D, SPARSE, true, false>(p, stream);
}

template <bool SPARSE>
cudaError_t launch_attn_dim(AttnParams p, int head_dim, int64_t units, const Spread& s,
                            cudaStream_t stream) {
  p.units = (int)units;
  p.cluster = s.cluster;
  p.splits = s.splits;
  switch (head_dim) {
    case 64: return launch_attn_page<64, SPARSE>(p, s.solo, stream);
    case 128: return launch_attn_page<128, SPARSE>(p, s.solo, stream);
    case 256: return launch_attn_page<256, SPARSE>(p, s.solo, stream);
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
  p.num_tokens = x.num_tokens;
  p.num_pages = x.num_pages;
  p.page_size = x.page_size;
  p.page_shift = -1;
  for (int s = 0; s < 31; ++s)
    if (x.page_size == 1 << s) p.page_shift = s;
  p.table = x.page_table;
  p.num_requests = x.num_requests;
  p.table_width = x.table_width;
  p.requests = x.requests;
  p.lens = x.lens;
  p.scale_log2 = scale * kLog2e;
  p.errors = x.errors;
  return p;
}

// Row tiles: block-sparse, of a token and kv head; shared prefix, of a kv head.
int sparse_tiles(int num_q, int num_kv) { return (num_q / num_kv + kRows - 1) / kRows; }

int64_t shared_tiles(int64_t num_tokens, int num_q, int num_kv) {
  return (num_tokens * (num_q / num_kv) + kRows - 1) / kRows;
}

Spread sparse_spread(int64_t num_tokens, int num_q, int num_kv, int page_size, int topk) {
  return spread_for(num_tokens * num_kv * sparse_tiles(num_q, num_kv), topk, page_size, false);
}

// The tokens' own keys, with the prefix's or behind its tiles (`late`).  The
// own pages that a tile can have: those of every token that has a row in it.
Spread shared_spread(int64_t num_tokens, int num_q, int num_kv, int page_size,
                     int64_t prefix_len, int table_width, bool late) {
  const int group = num_q / num_kv;
  const int64_t tokens = group >= kRows ? 2 : (kRows + group - 2) / group + 1;
  const int64_t own = (tokens < num_tokens ? tokens : num_tokens) * table_width;
  return spread_for(shared_tiles(num_tokens, num_q, num_kv) * num_kv,
                    (prefix_len + page_size - 1) / page_size + own, page_size, late);
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
  const int s = sparse_spread(num_tokens, num_heads_q, num_heads_kv, page_size, topk).splits;
  return s == 1 ? 0 : partials_bytes(s, num_tokens * num_heads_q, head_dim);
}

cudaError_t launch_sparse_attn(const SparseAttnArgs& a, cudaStream_t stream) {
  const PagedQuery& x = a.x;
  AttnParams p = common(x, a.kv_cache, a.scale);
  p.blocks = a.blocks;
  p.topk = a.topk;
  p.tiles = sparse_tiles(x.num_heads_q, x.num_heads_kv);
  const Spread s = sparse_spread(x.num_tokens, x.num_heads_q, x.num_heads_kv, x.page_size, a.topk);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  if (s.splits > 1)
    p.parts = partials_at(a.workspace, s.splits, (int64_t)x.num_tokens * x.num_heads_q, x.head_dim);
  const cudaError_t e = launch_attn_dim<true>(
      p, x.head_dim, (int64_t)x.num_tokens * x.num_heads_kv * p.tiles, s, stream);
  if (e != cudaSuccess || s.splits == 1) return e;
  return launch_attn_join(p.parts, s.splits, x.head_dim, a.out, stream);
}

int64_t prefix_attn_workspace(int64_t num_tokens, int num_heads_q, int num_heads_kv,
                              int head_dim, int page_size, int64_t prefix_len,
                              int table_width, int config) {
  const int64_t rows = num_tokens * num_heads_q;
  const int s = shared_spread(num_tokens, num_heads_q, num_heads_kv, page_size, prefix_len,
                              table_width, false).splits;
  int64_t slots = s == 1 ? 0 : s;
  if (prefix_tiles_fit(num_tokens, num_heads_q, num_heads_kv, head_dim, page_size, prefix_len,
                       config)) {
    // either way may be taken: which one depends on where the cache lies
    const int64_t parts =
        prefix_tiles_plan(num_tokens, num_heads_q, num_heads_kv, head_dim, prefix_len).parts;
    if (parts > slots) slots = parts;
  }
  return partials_bytes(slots, rows, head_dim);
}

cudaError_t launch_prefix_attn(const PrefixAttnArgs& a, cudaStream_t stream) {
  const PagedQuery& x = a.x;
  AttnParams p = common(x, a.kv_cache, a.scale);
  p.tiles = (int)shared_tiles(x.num_tokens, x.num_heads_q, x.num_heads_kv);
  p.prefix_pages = a.prefix_pages;
  const int64_t rows = (int64_t)x.num_tokens * x.num_heads_q;
  const int64_t units = (int64_t)p.tiles * x.num_heads_kv;
  CUtensorMap map;
  // (the tiles scale their masked scores, -inf, too: a scale of zero is not theirs)
  const bool tiles = a.scale != 0.f &&
                     prefix_tiles_fit(x.num_tokens, x.num_heads_q, x.num_heads_kv, x.head_dim,
                                      x.page_size, a.prefix_len, a.config) &&
                     prefix_tiles_map(a, &map);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.prefix_len = tiles ? 0 : (int)a.prefix_len;
  const Spread s = shared_spread(x.num_tokens, x.num_heads_q, x.num_heads_kv, x.page_size,
                                 p.prefix_len, x.table_width, tiles);
  if (!tiles) {
    if (s.splits > 1) p.parts = partials_at(a.workspace, s.splits, rows, x.head_dim);
    const cudaError_t e = launch_attn_dim<false>(p, x.head_dim, units, s, stream);
    if (e != cudaSuccess || s.splits == 1) return e;
    return launch_attn_join(p.parts, s.splits, x.head_dim, a.out, stream);
  }
  // The tiles, and then the tokens' own keys, whose kernel joins both: its CTAs
  // start as the tiles' run out, and need their partials at the end alone.
  const PrefixTilesPlan plan = prefix_tiles_plan(x.num_tokens, x.num_heads_q, x.num_heads_kv,
                                                 x.head_dim, a.prefix_len);
  p.prefix_parts = plan.parts;
  p.prefix_ctas = plan.lanes * plan.teams;
  p.parts = partials_at(a.workspace, p.prefix_parts, rows, x.head_dim);
  const cudaError_t e = launch_prefix_tiles(a, map, p.parts, stream);
  if (e != cudaSuccess) return e;
  return launch_attn_dim<false>(p, x.head_dim, units, s, stream);
}

}  // namespace kvq
