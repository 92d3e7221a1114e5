// kvq_paged_prefix.cu -- the shared prefix of a batch on the tensor cores: all
// query rows of a kv head (every token, every head of its group) against the
// prefix's keys and values.
//
// The work is items of up to 256 query rows of one kv head (two tiles of 128)
// times the prefix in blocks of 128 keys.  One CTA to an SM takes an equal
// share of the blocks; the part of an item that falls to it is a segment.  The
// CTAs that have the same blocks of a head, for different rows, keep in step,
// so that keys and values come from memory once (each CTA on its own way
// through 134 MB of them: 3300 cycles a block instead of 2500).  Per tile and
// key block
//   S = Q K^T   [128 x 128], fp32 in tensor memory,
//   P = 2^(S scale log2(e) - m), rounded once to bf16, over S's columns,
//   O += P V    [128 x D], fp32 in tensor memory, P read from there.
// With heads of 256, O of one tile takes half of the tensor memory: an item is
// one tile, and its blocks take S's two places in turn instead.
// Warps have one role each:
//   * warps 0-7 and 8-15: the softmax of tile 0 and of tile 1 (the warps
//     behind these are 8 lower where there is no tile 1).  Two threads own
//     a row (its tensor-memory lane), 64 keys each, and exchange only their
//     maxima (1250 cycles from scores to weights; one thread a row: 1500).
//     The reference m of a row only moves when a score exceeds it by more than
//     2^8; until then weights above 1 are as exact as those below, and O is
//     seldom rescaled;
//   * warp 16, one lane: issues the matrix instructions.  While one tile's
//     (or block's) softmax runs, the other's products do;
//   * warps 17 and 18: load K and V, two blocks ahead (heads of 256: the two
//     halves of a block's dims), by tensor-map copies (a page, or 128 keys of
//     one, at a time; 128-byte swizzle).  A block that
//     ends past the prefix, or that lists a page outside the cache, is copied
//     by the warp's own copies instead, all in flight at once, with zeros in V
//     where there is no key (3000 keys of 256 dims: 40 us with loads of four at
//     a time, 29); the softmax gives those places weight 0.
// A segment's result is a partial (normalised O and log2 of the weight sum).
// The kernel of the tokens' own keys, launched behind this one, joins them.
//
// Bound by the tensor cores, and by the power they may draw: 2048 rows x 8 kv
// heads x 32768 keys of 128 dims, 275 GFLOP, take 160 us (1720 TFLOP/s, tensor
// pipe active 77 % of the time, 141 MB read for 134 MB of keys and values);
// run back to back the clock settles at 1.75 of 2.07 GHz at the power limit.
// With heads of 64 the softmax bounds it: half the products for the same
// exponentials (949 TFLOP/s with the own keys' kernel); of 256, 1690 TFLOP/s (a
// prefetch of the next block into the L2 gained 3 % there and lost 20 % with
// 16-token pages).  On a short prefix half of the time is a CTA's start and
// end, 5 us: Q comes in by asynchronous copies, all at once, and the partials
// leave line by line through shared memory (with loads of four at a time and a
// row's pieces stored by one lane, 9 us; of 256 dims 7 instead of 13).
#include <string.h>

#include "kvq_paged_attn.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

constexpr int kTileRows = 128;
constexpr int kKeys = 128;            // keys of a block
// Registers of a thread where there are 640: 96 at launch; the softmax groups
// take 104, the last group keeps 56 (512 x 104 + 128 x 56 = 60416 of 61440).
constexpr int kSoftmaxRegs = 104, kOtherRegs = 56;
constexpr float kRescaleAt = 8.f;     // log2 by which a score may exceed m

struct PrefixParams {
  CUtensorMap map;  // the cache as [pages][2 Hkv][page_size][D]
  const __nv_bfloat16* q;
  int64_t q_stride;
  const __nv_bfloat16* cache;
  int num_q, num_kv, group;
  int64_t rows;  // tokens * group
  int64_t num_pages;
  int page_shift;
  const int* prefix_pages;
  int prefix_len;
  float scale_log2;  // >= 0
  uint32_t q_flip;   // sign bits flipped in Q where the scale is negative
  int row_tiles;     // items of one kv head
  int lanes;         // CTAs in step: the row tiles of a head, or 1
  int teams;         // .. and how many times so many there are
  int64_t items;     // of a lane
  int blocks;        // of 128 keys, of an item
  int slots;         // partials of an item, at most
  Partials parts;
  int* errors;
  uint32_t wait_polls;  // of a barrier, before the waiter gives up
};

// Row tiles of an item: two, or one of heads of 256, whose O takes half of the
// tensor memory.
constexpr int row_tiles_of(int head_dim) { return head_dim == 256 ? 1 : 2; }

template <int D>
struct Layout {
  static constexpr int kTiles = row_tiles_of(D);
  static constexpr int kMmaWarp = 8 * kTiles, kLoadWarp = kMmaWarp + 1;  // .. K, and V the next
  static constexpr int kThreads = 32 * kMmaWarp + 128;
  // K and V have two slots each, for two blocks, or for the two halves of a
  // block's dims.
  static constexpr int kSplit = D == 256 ? 2 : 1;
  static constexpr int kWidth = D / kSplit;          // dims of a slot
  static constexpr int kTile = kTileRows * D * 2;    // bytes of a tile of Q
  static constexpr int kSlot = kKeys * kWidth * 2;
  static constexpr int kQ = 0;
  static constexpr int kK = kTiles * kTile;
  static constexpr int kV = kK + 2 * kSlot;
  static constexpr int kTops = kV + 2 * kSlot;  // [2 blocks, and the sums][2 halves][256 rows]
  static constexpr int kBars = kTops + 3 * 2048;
  static constexpr int kEnd = kBars + 24 * 8 + 32;
  static constexpr int kSmem = kEnd + 1024;          // room to align the base
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
};

// mbarriers, by index
enum { kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kQFull = 8, kSFull = 10, kPFull = 12,
       kPvDone = 16, kDrain = 18, kBarriers = 19 };  // kPFull + 2 buffer + part

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Two fp32 values at a time: (a.x, a.y) * m + c and a + b.
union Pair {
  float f[2];
  unsigned long long u;
};
__device__ __forceinline__ Pair pair(float x, float y) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.u) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair m, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.u) : "l"(a.u), "l"(m.u), "l"(c.u));
  return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
  return r;
}

// Barrier of the two warps that share 32 rows.
__device__ __forceinline__ void pair_sync(int id) {
  asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
}

// What a warp that gives up hands its partner in place of a maximum or a sum (a
// NaN that no instruction makes).  It does so at the pair's next barrier, which
// the partner reaches as well, and both leave there: a barrier is always met by
// both, and no warp waits at one alone.
constexpr uint32_t kGaveUp = 0x7fc0deadu;
__device__ __forceinline__ bool gave_up(float x) { return __float_as_uint(x) == kGaveUp; }

// Where 16-byte fragment c of row r lies in a swizzled 128-row tile.
__device__ __forceinline__ uint32_t tile_offset(int r, int c) {
  return (uint32_t)((c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
  const int bytes = there ? 16 : 0;  // 0: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(__cvta_generic_to_global(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The share of a CTA, walked segment by segment: of the blocks of its lane's
// items, one item after the other, an equal part for each team.
struct Segments {
  int64_t at, stop;
  int64_t item;
  int first, n;       // the segment: blocks first .. first + n - 1 of the item
  int kv_head;
  int64_t row0;       // the item's first row
  int64_t rows_left;  // rows of the kv head from there on
  int tiles, rows;    // row tiles of the segment, rows of a whole item
  int lane, team;

  __device__ __forceinline__ Segments(const PrefixParams& p, int rows) : rows(rows) {
    team = (int)blockIdx.x / p.lanes;
    lane = (int)blockIdx.x - team * p.lanes;
    const int64_t all = p.items * p.blocks;
    at = team * all / p.teams;
    stop = (team + 1) * all / p.teams;
    n = 0;
  }
  __device__ __forceinline__ bool next(const PrefixParams& p) {
    at += n;
    if (at >= stop) return false;
    item = at / p.blocks;
    first = (int)(at - item * p.blocks);
    n = (int)min((int64_t)(p.blocks - first), stop - at);
    int tile = lane;
    kv_head = (int)item;
    if (p.lanes != p.row_tiles) {  // one lane: a head's row tiles one after the other
      kv_head = (int)(item / p.row_tiles);
      tile = (int)(item - (int64_t)kv_head * p.row_tiles);
    }
    row0 = (int64_t)tile * rows;
    rows_left = p.rows - row0;
    tiles = rows > kTileRows && rows_left > kTileRows ? 2 : 1;
    return true;
  }
  // The item's segments are numbered from the team that has its first block.
  __device__ __forceinline__ int slot(const PrefixParams& p) const {
    return team - (int)(((item * p.blocks + 1) * p.teams - 1) / (p.items * p.blocks));
  }
};

template <int D>
__global__ void __launch_bounds__(Layout<D>::kThreads, 1)
prefix_tiles_kernel(const __grid_constant__ PrefixParams p) {
  using L = Layout<D>;
  constexpr int kMmaWarp = L::kMmaWarp, kLoadWarp = L::kLoadWarp;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (tma::smem_addr(raw) + 1023u) & ~1023u;
  uint8_t* smem = raw + (base - tma::smem_addr(raw));
  volatile float* tops = reinterpret_cast<float*>(smem + L::kTops);
  const uint32_t bars = base + L::kBars;
  int* shared_state = reinterpret_cast<int*>(smem + L::kBars + 24 * 8);
  volatile int* dead = shared_state;  // a wait ran out
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(shared_state + 1);
  auto bar = [&](int i) { return bars + 8u * i; };
  auto await = [&](int i, uint32_t parity) {
    return tc::wait_warp(bar(i), parity, dead, p.wait_polls);
  };

  const int warp = __shfl_sync(kFullMask, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // a block comes in pieces: a page, or 128 keys of one; lane i has piece i
  const int piece_shift = min(p.page_shift, 7), pieces = kKeys >> piece_shift;
  const int page_mask = (1 << p.page_shift) - 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBarriers; ++i) {
      const bool by_warps = (i >= kQFull && i < kQFull + 2) || (i >= kPFull && i < kPFull + 4);
      tma::mbar_init(bar(i), by_warps ? 8 : 1);
    }
    tma::mbar_init_fence();
    *dead = 0;
  }
  if (warp == kMmaWarp) tc::alloc512(tma::smem_addr(tmem_slot));
  // All CTAs are resident at once: the kernel of the tokens' own keys may take
  // up the SMs that have none, or are done.  Not before the wait: that kernel
  // reads its inputs without one.
  grid_dependency_wait();
  launch_dependents();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = __shfl_sync(kFullMask, *tmem_slot, 0);
  Segments seg(p, L::kTiles * kTileRows);

  if (warp < kMmaWarp) {
    if constexpr (L::kTiles == 2)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---- softmax ---------------------------------------------------------------------
    const int tile = warp >> 3, half = (warp >> 2) & 1;
    const int r = tile * kTileRows + (warp & 3) * 32 + lane;  // the thread's row
    const int pair_bar = 1 + tile * 4 + (warp & 3);           // its two warps' barrier
    const uint32_t at = tmem + ((uint32_t)(warp & 3) << 21);  // the warp's 32 lanes
    const uint32_t o_at = at + 256 + 128 * tile + (D / 2) * half;
    // The warp's slice of its tile of Q, which it fills, and, when the products
    // that read Q are done, passes the results through.
    constexpr int kSlice = L::kTile / 8;
    uint8_t* slice = smem + L::kQ + tile * L::kTile + (warp & 7) * kSlice;
    uint32_t done = 0;  // blocks of this tile so far: the phase of its barriers
    bool ok = true;
    auto pv_done = [&](uint32_t block) {
      const int buf = L::kTiles == 2 ? tile : block & 1;
      const uint32_t phase = L::kTiles == 2 ? block & 1 : (block >> 1) & 1;
      return await(kPvDone + buf, phase);
    };
    auto row_of = [&](const Segments& seg) {  // of the thread's row: token * num_q + head
      const uint32_t flat = (uint32_t)(seg.row0 + r), t = flat / (uint32_t)p.group;
      return (int64_t)t * p.num_q + seg.kv_head * p.group + (int)(flat - t * p.group);
    };
    auto put_sum = [&](const Segments& seg, int64_t row, int slot, float lse) {
      if (half != 0 || r >= seg.rows_left) return;
      p.parts.lse[slot * p.parts.rows + row] = lse;
      // an item has fewer segments than others: the slots left over are empty
      if (seg.first + seg.n == p.blocks)
        for (int k = slot + 1; k < p.slots; ++k) p.parts.lse[k * p.parts.rows + row] = -INFINITY;
    };
    // Meets the partner at the pair's next barrier, whose values lie at `slot`.
    auto give_up = [&](int slot) {
      tops[slot + half * 256 + r] = __uint_as_float(kGaveUp);
      pair_sync(pair_bar);
    };
    while (seg.next(p)) {
      if (tile >= seg.tiles) continue;
      // Q comes in, to each warp's slice of the tile; the products that read the
      // previous segment's have all been seen to be done
#pragma unroll
      for (int i = 0; i < kSlice / 512; ++i) {
        const int at = (warp & 7) * kSlice + i * 512 + lane * 16;
        const int qr = (at & (128 * 128 - 1)) >> 7;
        const int d = (at >> 14) * 64 + ((((at >> 4) ^ qr) & 7) << 3);
        const int64_t from = tile * kTileRows + qr;
        const bool here = from < seg.rows_left;
        const uint32_t flat = (uint32_t)(seg.row0 + (here ? from : 0));
        const uint32_t t = flat / (uint32_t)p.group;
        const int h = seg.kv_head * p.group + (int)(flat - t * p.group);
        cp_async16(base + L::kQ + tile * L::kTile + at,
                   p.q + (int64_t)t * p.q_stride + (int64_t)h * D + d, here);
      }
      cp_wait_all();
      if (p.q_flip) {
        for (int i = 0; i < kSlice / 512; ++i) {
          uint4* at = reinterpret_cast<uint4*>(slice + i * 512 + lane * 16);
          const uint4 v = *at;
          *at = make_uint4(v.x ^ p.q_flip, v.y ^ p.q_flip, v.z ^ p.q_flip, v.w ^ p.q_flip);
        }
      }
      tma::fence_proxy_async();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(kQFull + tile));
      if (p.wait_polls == 0) {  // (not looked at in every wait: heads of 256 3 % slower)
        *dead = 1;
        ok = false;
        break;
      }

      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < seg.n; ++j, ++done) {
        // pages of the block outside the cache: their keys are not there
        const int key0 = (seg.first + j) * kKeys;
        bool outside = false;
        if (lane < pieces && key0 + (lane << piece_shift) < p.prefix_len) {
          const int page =
              __ldg(p.prefix_pages + ((key0 + (lane << piece_shift)) >> p.page_shift));
          outside = page < 0 || page >= p.num_pages;
        }
        const uint32_t bad = __ballot_sync(kFullMask, outside);
        // S has two buffers: one a tile, or the blocks of one tile in turn
        const int buf = L::kTiles == 2 ? tile : done & 1;
        const uint32_t phase = L::kTiles == 2 ? done & 1 : (done >> 1) & 1;
        const uint32_t s_at = at + 128 * buf + 64 * half, p_at = at + 128 * buf + 32 * half;
        if (!await(kSFull + buf, phase)) {
          give_up((done & 1) * 512);
          ok = false;
          break;
        }
        tc::fence_after();
        uint32_t s[2][32];
        tc::ld32(s[0], s_at);
        tc::ld32(s[1], s_at + 32);
        tc::wait_ld();
        if (bad != 0 || p.prefix_len - key0 < kKeys) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const int key = 64 * half + 32 * c + k;
              if (key0 + key >= p.prefix_len || (bad >> (key >> piece_shift) & 1))
                s[c][k] = 0xff800000u;  // -inf
            }
        }
        float top4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t* x = s[c >> 1] + 16 * (c & 1);
          top4[c] = __uint_as_float(x[0]);
#pragma unroll
          for (int k = 1; k < 15; k += 2)
            top4[c] = max3(top4[c], __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
        }
        float top = max3(top4[0], top4[1], max3(top4[2], top4[3], __uint_as_float(s[0][15])));
        top = max3(top, __uint_as_float(s[0][31]),
                   fmaxf(__uint_as_float(s[1][15]), __uint_as_float(s[1][31])));
        // the row's maximum over both halves; from here on both have read S
        tops[(done & 1) * 512 + half * 256 + r] = top;
        pair_sync(pair_bar);
        const float other = tops[(done & 1) * 512 + (half ^ 1) * 256 + r];
        top = fmaxf(m, fmaxf(top, other));
        // one vote for both that are rare (32768 keys x 2048 rows x 8 heads: 171.6 us
        // with the own keys' kernel; a vote each: 173.4)
        if (__any_sync(kFullMask,
                       (top - m) * p.scale_log2 > kRescaleAt || gave_up(other))) {
          if (__any_sync(kFullMask, gave_up(other))) {
            ok = false;
            break;
          }
          const float f = top == m ? 1.f : ex2((m - top) * p.scale_log2);
          l *= f;
          m = top;
          if (j > 0) {
            // O is at rest once the previous block's product is done
            if (!pv_done(done - 1)) {
              give_up(j + 1 < seg.n ? ((done + 1) & 1) * 512 : 1024);
              ok = false;
              break;
            }
            tc::fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c) {
              uint32_t o[32];
              tc::ld32(o, o_at + 32 * c);
              tc::wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tc::st32(o_at + 32 * c, o);
            }
          }
        }
        const float shift = m == -INFINITY ? 0.f : -m * p.scale_log2;
        const Pair scale2 = pair(p.scale_log2, p.scale_log2), shift2 = pair(shift, shift);
        Pair sum0 = pair(0.f, 0.f), sum1 = sum0;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            Pair a = fma2(pair(__uint_as_float(s[c][2 * k]), __uint_as_float(s[c][2 * k + 1])),
                          scale2, shift2);
            Pair b = fma2(pair(__uint_as_float(s[c][2 * k + 2]), __uint_as_float(s[c][2 * k + 3])),
                          scale2, shift2);
            a = pair(ex2(a.f[0]), ex2(a.f[1]));
            b = pair(ex2(b.f[0]), ex2(b.f[1]));
            sum0 = add2(sum0, a);
            sum1 = add2(sum1, b);
            w[k] = pack_bf16x2(a.f[0], a.f[1]);
            w[k + 1] = pack_bf16x2(b.f[0], b.f[1]);
          }
          tc::st16(p_at + 16 * c, w);
          // each half's first 32 keys are handed over before the others are done
          tc::wait_st();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar(kPFull + 2 * buf + c));
        }
        sum0 = add2(sum0, sum1);
        l += sum0.f[0] + sum0.f[1];
      }
      // ---- the partial -----------------------------------------------------------------
      if (ok) {
        const bool last = pv_done(done - 1);
        tops[1024 + half * 256 + r] = last ? l : __uint_as_float(kGaveUp);
        pair_sync(pair_bar);
        const float other = tops[1024 + (half ^ 1) * 256 + r];
        l += other;
        ok = last && !__any_sync(kFullMask, gave_up(other));
      }
      if (!ok) break;
      tc::fence_after();
      const int64_t row = row_of(seg);
      const int slot = seg.slot(p);
      const float f = l == 0.f ? 0.f : 1.f / l;
      // Through shared memory, so that lanes side by side write a row's values
      // side by side: 32 rows x kWide values at a time, fragments of four
      // exchanged by row against bank conflicts.
      constexpr int kWide = D == 64 ? 16 : 32, kFrags = kWide / 4;
      auto place = [&](int of, int frag) {
        return reinterpret_cast<float4*>(
            slice + (of * kFrags + (frag ^ ((kFrags == 8 ? of : of >> 1) & (kFrags - 1)))) * 16);
      };
      float* out = p.parts.o + slot * p.parts.rows * D + (D / 2) * half;
#pragma unroll 1
      for (int c = 0; c < D / 64; ++c) {
        uint32_t o[32];
        tc::ld32(o, o_at + 32 * c);
        tc::wait_ld();
#pragma unroll
        for (int k0 = 0; k0 < 32; k0 += kWide) {
#pragma unroll
          for (int k = 0; k < kFrags; ++k) {
            const uint32_t* x = o + k0 + 4 * k;
            *place(lane, k) =
                make_float4(__uint_as_float(x[0]) * f, __uint_as_float(x[1]) * f,
                            __uint_as_float(x[2]) * f, __uint_as_float(x[3]) * f);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < kFrags; ++i) {
            const int of = i * (32 / kFrags) + lane / kFrags, k = lane % kFrags;
            const int64_t to = __shfl_sync(kFullMask, (int)row, of);
            if (r - lane + of < seg.rows_left)
              *reinterpret_cast<float4*>(out + to * D + 32 * c + k0 + 4 * k) = *place(of, k);
          }
          __syncwarp();
        }
      }
      put_sum(seg, row, slot,
              l == 0.f ? -INFINITY : log2f(l) + (m == -INFINITY ? 0.f : m * p.scale_log2));
      tc::fence_before();
    }
    // The warp has given up: what this segment and those still to come should
    // have held is marked, whatever the workspace had there before.
    if (!ok) {
      do {
        if (tile < seg.tiles) put_sum(seg, row_of(seg), seg.slot(p), NAN);
      } while (seg.next(p));
    }
  } else if constexpr (L::kTiles == 2) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  }
  if (warp == kMmaWarp) {
    // ---- the matrix instructions -------------------------------------------------------
    constexpr uint32_t qk = tc::instr_desc(kKeys, false), pv = tc::instr_desc(L::kWidth, true);
    const uint64_t q_desc = tc::smem_desc(base + L::kQ, 16);
    const uint64_t k_desc = tc::smem_desc(base + L::kK, 16);
    const uint64_t v_desc = tc::smem_desc(base + L::kV, 128 * 128);
    uint32_t block = 0;
    bool ok = true;
    if constexpr (L::kTiles == 2) {
      auto scores = [&](int tile, int stage) {
        const uint64_t a = q_desc + (uint32_t)(tile * (L::kTile >> 4));
        const uint64_t b = k_desc + (uint32_t)(stage * (L::kSlot >> 4));
  #pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
          tc::mma_ss(tmem + 128 * tile, a + off, b + off, qk, k > 0);
        }
        tc::commit(bar(kSFull + tile));
      };
      uint32_t done[2] = {0, 0}, segs[2] = {0, 0};  // phases of the barriers
      while (ok && seg.next(p)) {
        ok = await(kKFull + (block & 1), (block >> 1) & 1);
        for (int t = 0; ok && t < seg.tiles; ++t) {
          ok = await(kQFull + t, segs[t]++ & 1);
          if (!ok) break;
          tc::fence_after();
          scores(t, block & 1);
        }
        if (!ok) break;
        tc::commit(bar(kKEmpty + (block & 1)));
        for (int j = 0; ok && j < seg.n; ++j, ++block) {
          const int stage = block & 1, next = stage ^ 1;
          const bool more = j + 1 < seg.n;
          ok = await(kVFull + stage, (block >> 1) & 1) &&
               (!more || await(kKFull + next, ((block + 1) >> 1) & 1));
          for (int t = 0; ok && t < seg.tiles; ++t) {
            const uint64_t v = v_desc + (uint32_t)(stage * (L::kSlot >> 4));
            for (int c = 0; ok && c < 2; ++c) {  // keys 0-31 and 64-95, then the others
              ok = await(kPFull + 2 * t + c, done[t] & 1);
              if (!ok) break;
              tc::fence_after();
  #pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int k = 4 * (i >> 1) + 2 * c + (i & 1);
                tc::mma_ts(tmem + 256 + 128 * t, tmem + 128 * t + 8 * k, v + k * (16 * 128 >> 4),
                           pv, j > 0 || c > 0 || i > 0);
              }
            }
            if (!ok) break;
            ++done[t];
            tc::commit(bar(kPvDone + t));
            // the next scores go over P, which the products above read first:
            // matrix instructions of one thread run in order
            if (more) scores(t, next);
          }
          if (!ok) break;
          tc::commit(bar(kVEmpty + stage));
          if (more) tc::commit(bar(kKEmpty + next));
        }
      }
    } else {
      // One tile: the scores of a block go before the products with the values of
      // the one before it, into S's other buffer (its weights have been read
      // then), and its softmax runs meanwhile.
      uint32_t segs = 0;
      auto scores = [&](uint32_t block) {
        for (int h = 0; ok && h < 2; ++h) {
          ok = await(kKFull + h, block & 1);
          if (!ok) break;
          tc::fence_after();
#pragma unroll
          for (int k = 0; k < L::kWidth / 16; ++k) {
            const uint32_t off = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
            tc::mma_ss(tmem + 128 * (block & 1),
                       q_desc + off + (uint32_t)(h * ((L::kWidth / 64) * (128 * 128) >> 4)),
                       k_desc + off + (uint32_t)(h * (L::kSlot >> 4)), qk, h > 0 || k > 0);
          }
          tc::commit(bar(kKEmpty + h));
        }
        if (ok) tc::commit(bar(kSFull + (block & 1)));
      };
      while (ok && seg.next(p)) {
        ok = await(kQFull, segs++ & 1);
        if (!ok) break;
        tc::fence_after();
        scores(block);
        for (int j = 0; ok && j < seg.n; ++j, ++block) {
          if (j + 1 < seg.n) scores(block + 1);
          const int buf = block & 1;
          for (int h = 0; ok && h < 2; ++h) {
            ok = await(kVFull + h, block & 1);
            const uint64_t v = v_desc + (uint32_t)(h * (L::kSlot >> 4));
            for (int c = 0; ok && c < 2; ++c) {  // keys 0-31 and 64-95, then the others
              if (h == 0) ok = await(kPFull + 2 * buf + c, (block >> 1) & 1);
              if (!ok) break;
              tc::fence_after();
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int k = 4 * (i >> 1) + 2 * c + (i & 1);
                tc::mma_ts(tmem + 256 + L::kWidth * h, tmem + 128 * buf + 8 * k,
                           v + k * (16 * 128 >> 4), pv, j > 0 || c > 0 || i > 0);
              }
            }
            if (ok) tc::commit(bar(kVEmpty + h));
          }
          if (ok) tc::commit(bar(kPvDone + buf));
        }
      }
    }
    if (!ok) {  // nothing may be in flight when the tensor memory goes
      tc::commit(bar(kDrain));
      tc::drain(bar(kDrain), 0);
      __syncwarp();
    }
  } else if (warp == kLoadWarp || warp == kLoadWarp + 1) {
    // ---- the loads: one warp for K, one for V --------------------------------------------
    const int kv = warp - kLoadWarp;
    const int64_t head_elems = ((int64_t)D) << p.page_shift;
    uint32_t turn = 0;  // slots filled so far
    int last[2] = {-1, -1};  // of each slot: its latest turn, if that is the copy engine's
    bool ok = true;
    while (ok && seg.next(p)) {
      const int head = kv * p.num_kv + seg.kv_head;
      for (int j = 0; ok && j < seg.n; ++j) {
        const int first = (seg.first + j) * kKeys;
        const int key = first + (lane << piece_shift);
        int page = -1;
        if (lane < pieces && key < p.prefix_len) {
          page = __ldg(p.prefix_pages + (key >> p.page_shift));
          if (page < 0 || page >= p.num_pages) {
            page = -1;
            if (p.errors && kv == 0) atomicAdd(p.errors, 1);
          }
        }
        const bool here = __all_sync(kFullMask, lane >= pieces || page >= 0);
        const bool whole = here && p.prefix_len - first >= kKeys;
        for (int h = 0; h < L::kSplit; ++h, ++turn) {
          const int slot = turn & 1;
          const uint32_t full = bar((kv ? kVFull : kKFull) + slot);
          const uint32_t dst = base + (kv ? L::kV : L::kK) + slot * L::kSlot;
          if (turn >= 2) {
            ok = await((kv ? kVEmpty : kKEmpty) + slot, ((turn >> 1) - 1) & 1);
            if (!ok) break;
          }
          if (whole) {
            if (lane == 0) tma::mbar_arrive_expect_tx(full, L::kSlot);
            __syncwarp();
            if (lane < pieces) {
#pragma unroll
              for (int b = 0; b < L::kWidth / 64; ++b)
                tma::tile_load_4d(dst + b * (128 * 128) + (lane << (piece_shift + 7)), &p.map,
                                  L::kWidth * h + 64 * b, key & page_mask, head, page, full);
            }
            (slot ? last[1] : last[0]) = (int)turn;
          } else {
            constexpr int FRAGS = L::kWidth / 8, RPW = 32 / FRAGS;
#pragma unroll 8
            for (int i = 0; i < kKeys / RPW; ++i) {
              const int r = i * RPW + lane / FRAGS, c = lane % FRAGS, k = first + r;
              const int from = __shfl_sync(kFullMask, page, r >> piece_shift);
              const bool there = from >= 0 && k < p.prefix_len;
              const __nv_bfloat16* src =
                  p.cache + ((int64_t)from * 2 * p.num_kv + head) * head_elems +
                  (int64_t)(k & page_mask) * D + L::kWidth * h + 8 * c;
              cp_async16(dst + tile_offset(r, c), there ? src : p.cache, there);
            }
            cp_wait_all();
            tma::fence_proxy_async();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(full);
            // the copies of the slot's turn before have been read: none is in flight
            (slot ? last[1] : last[0]) = -1;
          }
          __syncwarp();
        }
      }
    }
    if (!ok) {  // let the copies in flight land before the CTA may end
      for (int slot = 0; slot < 2; ++slot) {
        const int turn = slot ? last[1] : last[0];
        if (turn >= 0) tc::drain(bar((kv ? kVFull : kKFull) + slot), (turn >> 1) & 1);
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && p.errors && *dead) atomicAdd(p.errors, 1);
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::dealloc512(tmem);
  }
}

std::atomic<uint32_t> g_tile_wait_limit{tc::kPolls};

template <int D>
cudaError_t launch(const PrefixAttnArgs& a, const CUtensorMap& map, const Partials& parts,
                   cudaStream_t stream) {
  const PagedQuery& x = a.x;
  using L = Layout<D>;
  static std::atomic<int> cache[kMaxDevices];
  int per_sm = 0;
  const cudaError_t e = tma::prepare(prefix_tiles_kernel<D>, L::kThreads, L::kSmem, cache, &per_sm);
  if (e != cudaSuccess) return e;
  PrefixParams p;
  memset(&p, 0, sizeof p);
  p.map = map;
  p.q = static_cast<const __nv_bfloat16*>(x.q);
  p.q_stride = x.q_stride;
  p.cache = static_cast<const __nv_bfloat16*>(a.kv_cache);
  p.num_q = x.num_heads_q;
  p.num_kv = x.num_heads_kv;
  p.group = x.num_heads_q / x.num_heads_kv;
  p.rows = (int64_t)x.num_tokens * p.group;
  p.num_pages = x.num_pages;
  while ((1 << p.page_shift) < x.page_size) ++p.page_shift;
  p.prefix_pages = a.prefix_pages;
  p.prefix_len = (int)a.prefix_len;
  p.scale_log2 = fabsf(a.scale) * kLog2e;
  p.q_flip = a.scale < 0.f ? 0x80008000u : 0u;
  const PrefixTilesPlan plan =
      prefix_tiles_plan(x.num_tokens, x.num_heads_q, x.num_heads_kv, D, a.prefix_len);
  p.row_tiles = plan.row_tiles;
  p.lanes = plan.lanes;
  p.teams = plan.teams;
  p.items = (int64_t)plan.row_tiles / plan.lanes * x.num_heads_kv;
  p.blocks = plan.blocks;
  p.slots = plan.parts;
  p.parts = parts;
  p.errors = x.errors;
  p.wait_polls = g_tile_wait_limit.load(std::memory_order_relaxed);
  return launch_kernel(prefix_tiles_kernel<D>, dim3((unsigned)(plan.lanes * plan.teams)),
                       dim3(L::kThreads), L::kSmem, stream, p);
}

}  // namespace

namespace {
std::atomic<int> g_prefix_config{-1};
}  // namespace

const LaunchConfig kPrefixConfigs[] = {{"rows<4w>"}, {"tiles<20w,128x128>"}};
const int kPrefixNumConfigs = 2;

int set_prefix_config(int id) { return g_prefix_config.exchange(id, std::memory_order_relaxed); }
uint32_t set_tile_wait_limit(uint32_t polls) {
  return g_tile_wait_limit.exchange(polls, std::memory_order_relaxed);
}
int prefix_config() { return g_prefix_config.load(std::memory_order_relaxed); }

// Sizes the tiles can take, and where they pay.  Up to 16 rows of a kv head are
// one row tile of the other kernel, which reads the prefix once.  Beyond, each
// of its row tiles reads it again, but it is one launch without partials: by
// the products' size, GB300, us of the rows / the tiles (32 query heads, 8 kv
// heads of 128, own keys up to 64): 2^20 (16 tokens x 2048 keys) 13.0 / 12.6,
// (64 x 512) 14.1 / 15.8, 2^21 (32 x 2048) 16.8 / 17.2, (64 x 1024) 18.2 / 19.9,
// 2^22 (16 x 8192) 25 / 20, (64 x 2048) 26 / 22, 2^23 (16 x 16384) 41 / 25; heads
// of 64, 2^21 (32 x 2048) 12.6 / 11.3, (16 x 4096) 12.6 / 14.5, 2^22 (32 x 4096)
// 18 / 15; heads of 256, 2^20 (64 x 512) 23 / 26, 2^21 (32 x 2048) 28 / 24, 2^22
// (32 x 4096) 43 / 27, 2^28 (256 tokens x 64 heads x 16384) 1760 / 190.  (In a
// graph; outside one the second launch costs the host 5 us, which is why heads
// of 64 stay with one at 2^21.)
bool prefix_tiles_fit(int64_t num_tokens, int num_heads_q, int num_heads_kv, int head_dim,
                      int page_size, int64_t prefix_len, int config) {
  const int64_t rows = num_tokens * (num_heads_q / num_heads_kv);
  const bool can = page_size >= 8 && (page_size & (page_size - 1)) == 0 && prefix_len > 0;
  if (!can || config >= 0) return can && config == 1;
  const int64_t least = (head_dim == 64 ? 6 : head_dim == 128 ? 4 : 3) << 19;
  return rows > 16 && rows * num_heads_kv > least / prefix_len;
}

bool prefix_tiles_map(const PrefixAttnArgs& a, CUtensorMap* map) {
  const PagedQuery& x = a.x;
  if (x.num_pages == 0 || !tma::device_memory(a.kv_cache)) return false;
  const cuuint64_t row = (cuuint64_t)x.head_dim * 2;
  const cuuint64_t head = row * x.page_size, page = head * 2 * x.num_heads_kv;
  if (page >= ((cuuint64_t)1 << 40)) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)x.head_dim, (cuuint64_t)x.page_size,
                              (cuuint64_t)2 * x.num_heads_kv, (cuuint64_t)x.num_pages};
  const cuuint64_t strides[3] = {row, head, page};
  const cuuint32_t box[4] = {64, (cuuint32_t)(x.page_size < kKeys ? x.page_size : kKeys), 1, 1};
  return tma::encode_bf16_4d_swizzled(map, a.kv_cache, dims, strides, box);
}

PrefixTilesPlan prefix_tiles_plan(int64_t num_tokens, int num_heads_q, int num_heads_kv,
                                  int head_dim, int64_t prefix_len) {
  const int64_t rows = num_tokens * (num_heads_q / num_heads_kv);
  PrefixTilesPlan plan;
  const int of_item = row_tiles_of(head_dim) * kTileRows;
  plan.row_tiles = (int)((rows + of_item - 1) / of_item);
  plan.blocks = (int)((prefix_len + kKeys - 1) / kKeys);
  // The part has 152 SMs (with fewer, some CTAs form a second wave).  In step, if
  // that leaves at most a fifth of the SMs without a CTA (which
  // costs as much as reading out of step); every CTA has an item or two blocks.
  const int fit = 152 / (plan.row_tiles < 152 ? plan.row_tiles : 152);
  plan.lanes = plan.row_tiles <= 152 && fit * plan.row_tiles * 5 >= 152 * 4 ? plan.row_tiles : 1;
  const int64_t items = (int64_t)plan.row_tiles / plan.lanes * num_heads_kv;
  const int64_t all = items * plan.blocks, most = all / 2 > items ? all / 2 : items;
  plan.teams = (int)(most < 152 / plan.lanes ? most : 152 / plan.lanes);
  // an item's blocks fall to so many teams at most
  plan.parts = (int)((plan.blocks - 1) * (int64_t)plan.teams / all) + 2;
  return plan;
}

cudaError_t launch_prefix_tiles(const PrefixAttnArgs& a, const CUtensorMap& map,
                                const Partials& parts, cudaStream_t stream) {
  switch (a.x.head_dim) {
    case 64: return launch<64>(a, map, parts, stream);
    case 128: return launch<128>(a, map, parts, stream);
    case 256: return launch<256>(a, map, parts, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kvq
