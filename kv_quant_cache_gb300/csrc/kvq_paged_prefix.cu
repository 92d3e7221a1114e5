// kvq_paged_prefix.cu -- the shared prefix of a batch on the tensor cores: all
// query rows of a kv head (every token, every head of its group) against the
// prefix's keys and values.
//
// One CTA takes up to 256 query rows (two tiles of 128) and one part of the
// prefix, 128 keys at a time.  Per tile and key block
//   S = Q K^T   [128 x 128], fp32 in tensor memory,
//   P = 2^(S scale log2(e) - m), rounded once to bf16, over S's columns,
//   O += P V    [128 x D], fp32 in tensor memory, P read from there.
// Warps have one role each:
//   * warps 0-7 and 8-15: the softmax of tile 0 and tile 1.  Two threads own
//     a row (its tensor-memory lane), 64 keys each, and exchange only their
//     maxima.  (One thread a row: 1500 cycles a block instead of about half,
//     and the tensor cores waited.)  The reference m of a row only moves when
//     a score exceeds it by more than 2^8; until then weights above 1 are as
//     exact as those below, and O is seldom rescaled;
//   * warp 16, one lane: issues the matrix instructions.  While one tile's
//     softmax runs, the other tile's products do;
//   * warps 17 and 18: load K and V, two blocks ahead, by tensor-map copies (a
//     page, or 128 keys of one, at a time; 128-byte swizzle).  A block that
//     ends past the prefix, or that lists a page outside the cache, is copied
//     by the warp's own loads instead, with zeros in V where there is no key;
//     the softmax gives those places weight 0.
// The result is a partial (normalised O and log2 of the weight sum) for the
// join with the other parts and with each token's own keys.
//
// Bound by the tensor cores: 4 * 256 * 128 * D operations per 2 * 128 * D * 2
// bytes of keys and values, which the L2 serves to the CTAs that share them.
#include <string.h>

#include "kvq_paged_attn.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

constexpr int kTileRows = 128;
constexpr int kKeys = 128;            // keys of a block
constexpr int kThreads = 640;         // five groups of four warps
constexpr int kMmaWarp = 16, kLoadWarp = 17;  // 17: K, 18: V
// Registers of a thread: 640 x 96 at launch; the softmax groups take 104, the
// last group keeps 56 (512 x 104 + 128 x 56 = 60416 of 61440).
constexpr int kSoftmaxRegs = 104, kOtherRegs = 56;
constexpr int kMaxPages = 2048;       // pages of a part
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
  int row_tiles;     // CTAs over the rows of one kv head
  int share;         // blocks of a part
  int first_slot;
  Partials parts;
  int* errors;
};

template <int D>
struct Layout {
  static constexpr int kBlocks = D / 64;             // 128-byte wide column blocks
  static constexpr int kTile = kKeys * D * 2;        // bytes of 128 rows
  static constexpr int kQ = 0;
  static constexpr int kK = 2 * kTile;
  static constexpr int kV = kK + 2 * kTile;
  static constexpr int kList = kV + 2 * kTile;
  static constexpr int kTops = kList + kMaxPages * 4;  // [2 blocks][2 halves][256 rows]
  static constexpr int kBars = kTops + 4096;
  static constexpr int kEnd = kBars + 24 * 8 + 32;
  static constexpr int kSmem = kEnd + 1024;          // room to align the base
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
};

// mbarriers, by index
enum { kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kQFull = 8, kSFull = 9, kPFull = 11,
       kPvDone = 15, kDrain = 17, kBarriers = 18 };  // kPFull + 2 tile + part

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

// Its arrival alone, by a warp that gives up (`dead` is set): the other one's
// next pair_sync, its last before it fails in a wait of its own, passes.
__device__ __forceinline__ void pair_leave(int id) {
  __threadfence_block();
  asm volatile("bar.arrive %0, 64;" ::"r"(id) : "memory");
}

// Where 16-byte fragment c of row r lies in a swizzled 128-row tile.
__device__ __forceinline__ uint32_t tile_offset(int r, int c) {
  return (uint32_t)((c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void st_shared16(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
prefix_tiles_kernel(const __grid_constant__ PrefixParams p) {
  using L = Layout<D>;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (tma::smem_addr(raw) + 1023u) & ~1023u;
  uint8_t* smem = raw + (base - tma::smem_addr(raw));
  int* list = reinterpret_cast<int*>(smem + L::kList);
  volatile float* tops = reinterpret_cast<float*>(smem + L::kTops);
  const uint32_t bars = base + L::kBars;
  int* shared_state = reinterpret_cast<int*>(smem + L::kBars + 24 * 8);
  volatile int* dead = shared_state;      // a wait ran out
  int* any_bad = shared_state + 1;        // a listed page lies outside the cache
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(shared_state + 2);
  auto bar = [&](int i) { return bars + 8u * i; };

  const int warp = __shfl_sync(kFullMask, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int kv_head = blockIdx.x / p.row_tiles;
  const int64_t row0 = (int64_t)(blockIdx.x % p.row_tiles) * (2 * kTileRows);
  const int64_t rows_left = p.rows - row0;
  const int tiles = rows_left > kTileRows ? 2 : 1;
  const int key0 = (int)blockIdx.y * p.share * kKeys;
  const int key1 = (int)min((int64_t)p.prefix_len, (int64_t)key0 + (int64_t)p.share * kKeys);
  const int n = (key1 - key0 + kKeys - 1) / kKeys;  // at least 1
  const int page0 = key0 >> p.page_shift;
  const int listed = ((key1 - 1) >> p.page_shift) - page0 + 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBarriers; ++i) {
      tma::mbar_init(bar(i), i == kQFull ? 16 : i >= kPFull && i < kPFull + 4 ? 8 : 1);
    }
    tma::mbar_init_fence();
    *dead = 0;
    *any_bad = 0;
  }
  if (warp == kMmaWarp) tc::alloc512(tma::smem_addr(tmem_slot));
  __syncthreads();
  grid_dependency_wait();
  for (int i = threadIdx.x; i < listed; i += kThreads) {
    int page = __ldg(p.prefix_pages + page0 + i);
    if (page < 0 || page >= p.num_pages) {
      page = -1;
      *any_bad = 1;
      if (p.errors) atomicAdd(p.errors, 1);
    }
    list[i] = page;
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = __shfl_sync(kFullMask, *tmem_slot, 0);

  if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---- softmax ---------------------------------------------------------------------
    // all 512 threads bring in Q, tile after tile
    constexpr int FRAGS = D / 8;
    for (int i = threadIdx.x; i < tiles * kTileRows * FRAGS; i += 512) {
      const int r = i / FRAGS, c = i % FRAGS;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < rows_left) {
        const int64_t t = (row0 + r) / p.group;
        const int h = kv_head * p.group + (int)(row0 + r - t * p.group);
        v = __ldg(reinterpret_cast<const uint4*>(p.q + t * p.q_stride + (int64_t)h * D + 8 * c));
        v.x ^= p.q_flip, v.y ^= p.q_flip, v.z ^= p.q_flip, v.w ^= p.q_flip;
      }
      st_shared16(base + L::kQ + (r >> 7) * L::kTile + tile_offset(r & 127, c), v);
    }
    tma::fence_proxy_async();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar(kQFull));

    const int tile = warp >> 3, half = (warp >> 2) & 1;
    const int r = tile * kTileRows + (warp & 3) * 32 + lane;  // the thread's row
    const int pair_bar = 1 + tile * 4 + (warp & 3);           // its two warps' barrier
    const uint32_t at = tmem + ((uint32_t)(warp & 3) << 21);  // the warp's 32 lanes
    const uint32_t s_at = at + 128 * tile + 64 * half, p_at = at + 128 * tile + 32 * half;
    const uint32_t o_at = at + 256 + 128 * tile + (D / 2) * half;
    const bool ragged_end = ((key1 - key0) & (kKeys - 1)) != 0;
    const bool bad = *any_bad != 0;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    if (tile < tiles) {
      for (int j = 0; j < n; ++j) {
        ok = tc::wait_warp(bar(kSFull + tile), j & 1, dead);
        if (!ok) break;
        tc::fence_after();
        uint32_t s[2][32];
        tc::ld32(s[0], s_at);
        tc::ld32(s[1], s_at + 32);
        tc::wait_ld();
        if (bad || (ragged_end && j == n - 1)) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const int key = key0 + j * kKeys + 64 * half + 32 * c + k;
              if (key >= key1 || list[(key >> p.page_shift) - page0] < 0)
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
        tops[(j & 1) * 512 + half * 256 + r] = top;
        pair_sync(pair_bar);
        top = fmaxf(m, fmaxf(top, tops[(j & 1) * 512 + (half ^ 1) * 256 + r]));
        if (__any_sync(kFullMask, (top - m) * p.scale_log2 > kRescaleAt)) {
          const float f = top == m ? 1.f : ex2((m - top) * p.scale_log2);
          l *= f;
          m = top;
          if (j > 0) {
            // O is at rest once the previous block's product is done
            ok = tc::wait_warp(bar(kPvDone + tile), (j - 1) & 1, dead);
            if (!ok) break;
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
          if (lane == 0) tc::mbar_arrive(bar(kPFull + 2 * tile + c));
        }
        sum0 = add2(sum0, sum1);
        l += sum0.f[0] + sum0.f[1];
      }
      // ---- the partial -----------------------------------------------------------------
      if (ok) ok = tc::wait_warp(bar(kPvDone + tile), (n - 1) & 1, dead);
      tc::fence_after();
      // the halves' sums; not the slots of the last block's maxima
      if (ok) {
        tops[(n & 1) * 512 + half * 256 + r] = l;
        pair_sync(pair_bar);
        l += tops[(n & 1) * 512 + (half ^ 1) * 256 + r];
        ok = *dead == 0;
      } else {
        pair_leave(pair_bar);
      }
      const int64_t t = (row0 + r) / p.group;
      const int64_t row = t * p.num_q + kv_head * p.group + (row0 + r - t * p.group);
      const int64_t slot = p.first_slot + blockIdx.y;
      const float f = l == 0.f ? 0.f : 1.f / l;
      float* out = p.parts.o + (slot * p.parts.rows + row) * D + (D / 2) * half;
#pragma unroll 1
      for (int c = 0; c < D / 64; ++c) {
        uint32_t o[32];
        tc::ld32(o, o_at + 32 * c);
        tc::wait_ld();
        if (r < rows_left) {
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            *reinterpret_cast<float4*>(out + 32 * c + k) =
                make_float4(__uint_as_float(o[k]) * f, __uint_as_float(o[k + 1]) * f,
                            __uint_as_float(o[k + 2]) * f, __uint_as_float(o[k + 3]) * f);
        }
      }
      if (half == 0 && r < rows_left)
        p.parts.lse[slot * p.parts.rows + row] =
            !ok ? NAN : l == 0.f ? -INFINITY : log2f(l) + (m == -INFINITY ? 0.f : m * p.scale_log2);
    }
    tc::fence_before();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  }
  if (warp == kMmaWarp) {
    // ---- the matrix instructions -------------------------------------------------------
    constexpr uint32_t qk = tc::instr_desc(kKeys, false), pv = tc::instr_desc(D, true);
    const uint64_t q_desc = tc::smem_desc(base + L::kQ, 16);
    const uint64_t k_desc = tc::smem_desc(base + L::kK, 16);
    const uint64_t v_desc = tc::smem_desc(base + L::kV, 128 * 128);
    auto scores = [&](int tile, int stage) {
      const uint64_t a = q_desc + (uint32_t)(tile * (L::kTile >> 4));
      const uint64_t b = k_desc + (uint32_t)(stage * (L::kTile >> 4));
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
        tc::mma_ss(tmem + 128 * tile, a + off, b + off, qk, k > 0);
      }
      tc::commit(bar(kSFull + tile));
    };
    bool ok = tc::wait_warp(bar(kQFull), 0, dead) && tc::wait_warp(bar(kKFull), 0, dead);
    if (ok) {
      tc::fence_after();
      for (int t = 0; t < tiles; ++t) scores(t, 0);
      tc::commit(bar(kKEmpty));
    }
    for (int j = 0; ok && j < n; ++j) {
      const int stage = j & 1, next = (j + 1) & 1;
      const bool more = j + 1 < n;
      ok = tc::wait_warp(bar(kVFull + stage), (j >> 1) & 1, dead) &&
           (!more || tc::wait_warp(bar(kKFull + next), ((j + 1) >> 1) & 1, dead));
      for (int t = 0; ok && t < tiles; ++t) {
        const uint64_t v = v_desc + (uint32_t)(stage * (L::kTile >> 4));
        for (int c = 0; ok && c < 2; ++c) {  // keys 0-31 and 64-95, then the others
          ok = tc::wait_warp(bar(kPFull + 2 * t + c), j & 1, dead);
          if (!ok) break;
          tc::fence_after();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int k = 4 * (i >> 1) + 2 * c + (i & 1);
            tc::mma_ts(tmem + 256 + 128 * t, tmem + 128 * t + 8 * k, v + k * (16 * 128 >> 4), pv,
                       j > 0 || c > 0 || i > 0);
          }
        }
        if (!ok) break;
        tc::commit(bar(kPvDone + t));
        // the next scores go over P, which the products above read first:
        // matrix instructions of one thread run in order
        if (more) scores(t, next);
      }
      if (!ok) break;
      tc::commit(bar(kVEmpty + stage));
      if (more) tc::commit(bar(kKEmpty + next));
    }
    if (!ok) {  // nothing may be in flight when the tensor memory goes
      tc::commit(bar(kDrain));
      for (uint32_t i = 0; i < (1u << 22) && !tma::mbar_test(bar(kDrain), 0); ++i) {
      }
      __syncwarp();
    }
  } else if (warp == kLoadWarp || warp == kLoadWarp + 1) {
    // ---- the loads: one warp for K, one for V --------------------------------------------
    const int kv = warp - kLoadWarp;
    const int page_size = 1 << p.page_shift;
    const int box = min(page_size, kKeys), pieces = kKeys / box;
    const int head = kv * p.num_kv + kv_head;
    const int64_t head_elems = (int64_t)page_size * D;
    int last = -1;  // latest block whose copies were started
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int stage = j & 1, first = key0 + j * kKeys;
      const uint32_t full = bar((kv ? kVFull : kKFull) + stage);
      const uint32_t dst = base + (kv ? L::kV : L::kK) + stage * L::kTile;
      // lane i has piece i of the block
      const int key = first + lane * box;
      const int page = lane < pieces && key < key1 ? list[(key >> p.page_shift) - page0] : -1;
      const bool whole = first + kKeys <= key1 &&
                         __all_sync(kFullMask, lane >= pieces || page >= 0);
      if (j >= 2) {
        ok = tc::wait_warp(bar((kv ? kVEmpty : kKEmpty) + stage), ((j >> 1) - 1) & 1, dead);
        if (!ok) break;
      }
      if (whole) {
        if (lane == 0) tma::mbar_arrive_expect_tx(full, L::kTile);
        __syncwarp();
        if (lane < pieces) {
#pragma unroll
          for (int b = 0; b < L::kBlocks; ++b)
            tma::tile_load_4d(dst + b * (128 * 128) + lane * box * 128, &p.map, 64 * b,
                              key & (page_size - 1), head, page, full);
        }
        last = j;
      } else {
        constexpr int FRAGS = D / 8, RPW = 32 / FRAGS;
#pragma unroll 4
        for (int r = lane / FRAGS; r < kKeys; r += RPW) {
          const int k = first + r, c = lane % FRAGS;
          const int from = k < key1 ? list[(k >> p.page_shift) - page0] : -1;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (from >= 0)
            v = __ldg(reinterpret_cast<const uint4*>(
                p.cache + ((int64_t)from * 2 * p.num_kv + head) * head_elems +
                (int64_t)(k & (page_size - 1)) * D + 8 * c));
          st_shared16(dst + tile_offset(r, c), v);
        }
        tma::fence_proxy_async();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(full);
      }
      __syncwarp();
    }
    if (!ok && last >= 0) {  // let the copies in flight land before the CTA may end
      const uint32_t full = bar((kv ? kVFull : kKFull) + (last & 1));
      for (uint32_t i = 0; i < (1u << 22) && !tma::mbar_test(full, (last >> 1) & 1); ++i) {
      }
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::dealloc512(tmem);
  }
}

// Blocks of a part.  `items` CTAs each have `blocks` blocks to share among
// `splits` of them, one CTA to an SM: the time of a plan is its waves times
// (blocks of a part + the start and end of a CTA, about 3 blocks' time), and
// each part's rows go through memory once more.
int share_for(int64_t items, int64_t blocks, int64_t out_rows, int head_dim, int page_size) {
  const int64_t room = (int64_t)kMaxPages * page_size / kKeys;  // blocks a list can hold
  const double per_part = (double)out_rows * head_dim * 8 / 8e12 / 1.1e-6;
  int64_t best = 1;
  double best_cost = 1e300;
  for (int64_t s = 1; s <= blocks && s <= 1024; ++s) {
    const int64_t share = (blocks + s - 1) / s;
    if (share > room) continue;
    const int64_t parts = (blocks + share - 1) / share;
    const int64_t waves = (items * parts + 151) / 152;
    const double cost = (double)waves * (share + 3) + per_part * parts;
    if (cost < best_cost) best_cost = cost, best = share;
    if (items * s > 152 * 16) break;
  }
  if (best_cost == 1e300) best = room;
  return (int)best;
}

template <int D>
cudaError_t launch(const PrefixAttnArgs& a, const CUtensorMap& map, const Partials& parts,
                   cudaStream_t stream) {
  const PagedQuery& x = a.x;
  using L = Layout<D>;
  static std::atomic<int> cache[kMaxDevices];
  int per_sm = 0;
  const cudaError_t e = tma::prepare(prefix_tiles_kernel<D>, kThreads, L::kSmem, cache, &per_sm);
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
  p.row_tiles = (int)((p.rows + 2 * kTileRows - 1) / (2 * kTileRows));
  const PrefixTilesPlan plan = prefix_tiles_plan(x.num_tokens, x.num_heads_q, x.num_heads_kv, D,
                                                 x.page_size, a.prefix_len);
  p.share = plan.share;
  p.first_slot = 0;
  p.parts = parts;
  p.errors = x.errors;
  return launch_kernel(prefix_tiles_kernel<D>,
                             dim3((unsigned)(p.row_tiles * x.num_heads_kv), (unsigned)plan.parts),
                             dim3(kThreads), L::kSmem, stream, p);
}

}  // namespace

bool prefix_tiles_fit(int64_t num_tokens, int num_heads_q, int num_heads_kv, int head_dim,
                      int page_size, int64_t prefix_len) {
  return (head_dim == 64 || head_dim == 128) && page_size >= 8 &&
         (page_size & (page_size - 1)) == 0 && prefix_len > 0 &&
         num_tokens * (num_heads_q / num_heads_kv) > 16;
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
                                  int head_dim, int page_size, int64_t prefix_len) {
  const int64_t rows = num_tokens * (num_heads_q / num_heads_kv);
  const int64_t blocks = (prefix_len + kKeys - 1) / kKeys;
  const int64_t items = (rows + 2 * kTileRows - 1) / (2 * kTileRows) * num_heads_kv;
  PrefixTilesPlan plan;
  plan.share = share_for(items, blocks, num_tokens * num_heads_q, head_dim, page_size);
  plan.parts = (int)((blocks + plan.share - 1) / plan.share);
  return plan;
}

cudaError_t launch_prefix_tiles(const PrefixAttnArgs& a, const CUtensorMap& map,
                                const Partials& parts, cudaStream_t stream) {
  return a.x.head_dim == 64 ? launch<64>(a, map, parts, stream)
                            : launch<128>(a, map, parts, stream);
}

}  // namespace kvq
