// kvq_latent_attn.cu -- attention of each token's heads over the latent entries
// listed for it, on the tensor cores: keys and values are the same 512-dim vectors
// of the FP8 cache.
//
// Up to 64 heads of a token and its list are a unit, the list in tiles of 128
// entries.  The entries are the first operand of both products,
//   S^T = X Q^T   [128 entries x heads],  O^T = X^T P^T   [4 x 128 dims x heads],
// fp32 in tensor memory: the 128 rows of an instruction are always filled, whatever
// the number of heads, and O^T of 64 heads takes half of the tensor memory, where
// O of 128 rows would take all of it.  X is decoded once, to bf16 in shared memory,
// and read by both products (by the second one transposed).
// Warps have one role each:
//   * warps 0-7: the softmax.  A thread has one entry (its tensor-memory lane) and half
//     of the heads.  The reference of a head moves only when a score exceeds it by
//     more than 30 in units of log2, a weight of 2^30, so that the exchange of maxima
//     between lanes, and the rescaling of O^T, are rare; weights, rounded to bf16 for the
//     product (the sums take them unrounded), go to shared memory as rows of heads;
//   * warps 8-23: read entries (8 bytes a lane, a whole tile ahead in registers) and
//     decode them, four warps to a quarter of the dims: as soon as the second product
//     of the tile before is done with a quarter, the next tile's takes its place;
//   * warp 24: issues the matrix instructions;
//   * warp 25: looks the lists up, up to four tiles ahead;
//   * warps 26 and 27: copy the queries of a unit as soon as the last scores of the unit
//     before are done, while its outputs are still to come.
//
// What bounds it: X has room for one tile, so that its products, the softmax between them
// and the next tile's decoding follow one another, and shared memory, which all of them
// use.  Of the 9600 cycles of a tile of 64 heads (16 tokens x 128 heads x 16384 entries)
// its pipe is busy for 6900 at most, by the counters: 3000 of operands that the matrix
// instructions read (A of 128 KB twice, of 64 heads as B), 3900 of loads and stores (X
// written, entries and scores, partials).  The next busiest are issue slots, 38 %, and
// the tensor cores, 21 %.
// 16 tokens x 128 heads x 16384 entries 112 us (460 TFLOP/s), 64 x 64 x 2048 48 us.
//
// With few units a CTA to an SM takes an equal share of all tiles of all lists, from
// the lists' actual lengths; a unit that falls to several CTAs goes to partials,
// which a second launch joins.  With many units a CTA takes one.
#include <climits>
#include <cstring>
#include <type_traits>

#include "kvq_dsv4_entry.cuh"
#include "kvq_paged_attn.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

constexpr int kDim = dsv4::kDim;
constexpr int kKeys = 128;          // entries of a tile
constexpr int kQuarters = 4;        // of the dims
constexpr int kSoftmaxWarps = 8, kLoadWarps = 16;
constexpr int kMmaWarp = kSoftmaxWarps + kLoadWarps, kListWarp = kMmaWarp + 1;
constexpr int kQueryWarp = kListWarp + 1, kQueryWarps = 2;
constexpr int kThreads = 32 * (kQueryWarp + kQueryWarps);
constexpr int kAhead = 4;  // tiles whose slots are in shared memory
// (28 warps of 72 registers each.  A softmax warp reads its scores twice, half of its
// heads at a time, to make do with them.)
// Up to so many units the tiles are shared out.  Both ways measured, lists of half to all of
// 2048 entries, 64 heads: 76 tokens 54 us (74 as a CTA to a unit), 228 121 (136), 608 281
// (287), 1024 451 (457): sharing out fills the last wave, and wins little once there are
// many.  Not so where units fill whole waves (152 tokens 90 (80); 152 of 128 heads 158
// (145)) and where lists are of few tiles, as partials and their join cost more than they
// bring (608 tokens of 150 to 300 entries 97 (79)): the host does not know the lengths.
constexpr int kSharedUnits = 4 * 152;
constexpr int kCtas = 152;             // .. to so many CTAs
// log2 by which a score may exceed its reference: weights are as exact above 1 as below
constexpr float kRescaleAt = 30.f;
constexpr float kNone = -3.402823466e38f;  // the reference of a head with scores of -inf alone

struct LatentParams {
  const __nv_bfloat16* q;
  int64_t q_stride;
  int num_tokens, num_heads;
  int blocks;                // of heads, of a token
  const uint8_t* cache;
  int64_t num_slots;
  const int* slots;
  int list_width;
  const int* lens;
  float scale_log2;
  bool shared_out;           // the tiles are shared out
  __nv_bfloat16* out;
  float* part_o;             // [CTAs][2][heads of a unit][512]
  float2* part_sums;         // [CTAs][2][heads of a unit]: reference, sum of the weights
  int* errors;
  uint32_t wait_polls;       // of a barrier, before the waiter gives up
};

// mbarriers, by index
enum { kXFull = 0, kXEmpty = 4, kListFull = 8, kListEmpty = 12, kQFull = 16, kSFull = 17,
       kPFull = 18, kODone = 19, kQEmpty = 20, kDrain = 21, kBarriers = 22 };

template <int NH>
struct Layout {
  static constexpr int kChunk = kKeys * 128;            // 64 dims of a tile
  static constexpr int kX = 0;                          // 8 chunks
  static constexpr int kP = 8 * kChunk;                 // 128 rows of up to 64 heads
  static constexpr int kQChunk = NH * 128;              // 64 dims of Q
  static constexpr int kQ = kP + kChunk;
  static constexpr int kTops = kQ + 8 * kQChunk;        // [4 quadrants of lanes][NH]
  static constexpr int kRef = kTops + 4 * 64 * 4;       // [NH] references, [NH] factors
  static constexpr int kStart = kRef + 2 * 64 * 4;      // [tokens + 1] first tiles
  static constexpr int kLens = kStart + (kSharedUnits + 8) * 4;  // [tokens] lengths of lists
  static constexpr int kLists = kLens + (kSharedUnits + 8) * 4;  // [kAhead][128] slots
  static constexpr int kBars = kLists + kAhead * kKeys * 4;
  static constexpr int kEnd = kBars + 24 * 8 + 48;
  static constexpr int kSmem = kEnd + 1024;             // room to align the base
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  const int bytes = there ? 16 : 0;  // 0: zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(__cvta_generic_to_global(src)), "r"(bytes)
               : "memory");
}

// Barriers of the softmax warps; vote: whether any thread's flag is set.
__device__ __forceinline__ void softmax_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kSoftmaxWarps) : "memory");
}
__device__ __forceinline__ bool softmax_vote(bool flag) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)flag), "n"(32 * kSoftmaxWarps)
      : "memory");
  return any != 0;
}

// Joins v[c] of the 32 lanes: afterwards v[0] of lane l is column l / (32 / N)'s.
template <int N, typename Op>
__device__ __forceinline__ float columns(float (&v)[N], int lane, Op op) {
  int n = N;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (n > 1) {
      n >>= 1;
#pragma unroll
      for (int k = 0; k < N / 2; ++k) {
        if (k < n) {
          const bool up = lane & o;
          const float mine = up ? v[k + n] : v[k], other = up ? v[k] : v[k + n];
          v[k] = op(mine, __shfl_xor_sync(kFullMask, other, o));
        }
      }
    } else {
      v[0] = op(v[0], __shfl_xor_sync(kFullMask, v[0], o));
    }
  }
  return v[0];
}

// Multiplication and addition where a shift or a sum would do: those share a pipe of half
// the rate with the logic below, this one does not.  (The factors come from registers
// that the compiler does not know, or it would make shifts and sums of them.)
struct Factors {
  uint32_t one, sixteen;
};
__device__ __forceinline__ Factors factors() {
  Factors f;
  asm volatile("mov.b32 %0, 1;" : "=r"(f.one));
  asm volatile("mov.b32 %0, 16;" : "=r"(f.sixteen));
  return f;
}
__device__ __forceinline__ uint32_t mad(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("mad.lo.u32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t which) {
  uint32_t d;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(d) : "r"(a), "r"(which));
  return d;
}

// Eight e4m3 codes, none of them NaN, times 2^(byte - 127), byte up to 134, as bf16.
// Sign and magnitude are put where a bf16 has them, with the exponent's bias short by
// 120: one product mends that and applies the scale, subnormal codes included.
__device__ __forceinline__ uint4 decode8(const uint2& codes, uint32_t byte, const Factors& f) {
  const uint32_t pair = mad(byte, 0x00800080u, 0x3c003c00u);  // 2^(byte - 7), twice
  const __nv_bfloat162 scale = *reinterpret_cast<const __nv_bfloat162*>(&pair);
  auto two = [&](uint32_t word, uint32_t which) {
    // (code, its sign bit eight times), twice
    uint32_t x = mad(prmt(word, which), f.sixteen, 0) & 0x87f087f0u;
    const __nv_bfloat162 v = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&x), scale);
    return *reinterpret_cast<const uint32_t*>(&v);
  };
  return make_uint4(two(codes.x, 0x9180), two(codes.x, 0xb3a2), two(codes.y, 0x9180),
                    two(codes.y, 0xb3a2));
}

// Collects in bits 7 of the bytes whether a code is NaN, a magnitude of 127: adding one
// then changes its sign bit.  (Only behind a NaN may a carry reach the next byte.)
__device__ __forceinline__ uint32_t nan_bits(uint32_t so_far, uint32_t codes, const Factors& f) {
  return so_far | (mad(codes, f.one, 0x01010101u) ^ codes);
}

// How many entries of its list a token has; a length outside the list is cut.
__device__ __forceinline__ int list_len(const LatentParams& p, int len) {
  return max(0, min(len, p.list_width));
}
__device__ __forceinline__ int list_tiles(int len) {  // (an empty list is one empty tile)
  return max(1, len / kKeys + (len % kKeys != 0));
}

// The segments of a CTA: parts of a unit's tiles.
struct Segments {
  int64_t at, stop;
  int n;              // the segment: tiles first .. first + n - 1 of the unit's `tiles`
  int first, tiles;
  int token, block;   // the unit
  int len;            // entries of its list
  int count;          // segments so far

  // CTAs that have tiles, so that each of them has one at least, and the first tile of
  // CTA b (past the last: all)
  __device__ __forceinline__ static int busy(int64_t all, int ctas) {
    return (int)min(all, (int64_t)ctas);
  }
  __device__ __forceinline__ static int64_t border(int64_t all, int b, int ctas) {
    return all * min(b, ctas) / ctas;
  }
  __device__ __forceinline__ Segments(const LatentParams& p, const int* start) {
    n = 0, count = 0;
    if (p.shared_out) {
      const int64_t all = (int64_t)start[p.num_tokens] * p.blocks;
      const int ctas = busy(all, (int)gridDim.x);
      at = border(all, (int)blockIdx.x, ctas);
      stop = border(all, (int)blockIdx.x + 1, ctas);
    } else {
      at = 0, stop = 1;
    }
  }
  __device__ __forceinline__ bool next(const LatentParams& p, const int* start,
                                       const int* lens) {
    at += n;
    if (at >= stop) return false;
    ++count;
    if (p.shared_out) {
      int lo = 0, hi = p.num_tokens;  // the last token that starts at or before `at`
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)start[mid] * p.blocks <= at) lo = mid;
        else hi = mid;
      }
      token = lo;
      tiles = start[lo + 1] - start[lo];
      const int rest = (int)(at - (int64_t)start[lo] * p.blocks);
      block = rest / tiles;
      first = rest - block * tiles;
      n = (int)min((int64_t)(tiles - first), stop - at);
      len = lens[token];
    } else {
      token = (int)blockIdx.x / p.blocks;
      block = (int)blockIdx.x - token * p.blocks;
      len = list_len(p, __ldg(p.lens + token));
      first = 0;
      n = tiles = list_tiles(len);
      stop = n;
    }
    return true;
  }
  __device__ __forceinline__ bool whole() const { return n == tiles; }
};

template <int K>
using I = std::integral_constant<int, K>;

template <int NH>
__global__ void __launch_bounds__(kThreads, 1)
latent_tiles_kernel(const __grid_constant__ LatentParams p) {
  using L = Layout<NH>;
  constexpr int COLS = NH / 2;  // heads of a softmax thread
  extern __shared__ uint8_t raw[];
  const uint32_t base = (tma::smem_addr(raw) + 1023u) & ~1023u;
  uint8_t* smem = raw + (base - tma::smem_addr(raw));
  volatile float* tops = reinterpret_cast<float*>(smem + L::kTops);
  float* refs = reinterpret_cast<float*>(smem + L::kRef);
  float* moves = refs + 64;  // factors of the heads
  int* start = reinterpret_cast<int*>(smem + L::kStart);
  int* lens = reinterpret_cast<int*>(smem + L::kLens);
  const uint32_t bars = base + L::kBars;
  volatile int* lists = reinterpret_cast<int*>(smem + L::kLists);
  int* shared_state = reinterpret_cast<int*>(smem + L::kBars + 24 * 8);
  volatile int* dead = shared_state;      // a wait ran out
  volatile int* quit = shared_state + 1;  // .. of a softmax warp
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(shared_state + 2);
  volatile int* place = shared_state + 4;  // [kAhead] of a tile in its segment: first 1, last 2
  auto bar = [&](int i) { return bars + 8u * i; };
  auto await = [&](int i, uint32_t parity) {
    return tc::wait_warp(bar(i), parity, dead, p.wait_polls);
  };
  const int warp = __shfl_sync(kFullMask, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBarriers; ++i)
      tma::mbar_init(bar(i), i < kXEmpty ? kLoadWarps / kQuarters
                             : i >= kListEmpty && i < kQFull ? kLoadWarps + kSoftmaxWarps + 1
                             : i == kQFull ? kQueryWarps : i == kPFull ? kSoftmaxWarps : 1);
    tma::mbar_init_fence();
    *dead = *quit = 0;
  }
  if (warp == kMmaWarp) tc::alloc512(tma::smem_addr(tmem_slot));
  grid_dependency_wait();
  if (p.shared_out) {
    // the first tile of each token, of one block of heads
    for (int t = threadIdx.x; t < p.num_tokens; t += kThreads) {
      const int len = __ldg(p.lens + t);
      lens[t] = list_len(p, len);
      start[t + 1] = list_tiles(lens[t]);
      if (blockIdx.x == 0 && len != list_len(p, len) && p.errors) atomicAdd(p.errors, 1);
    }
    __syncthreads();
    if (warp == 0) {
      int sum = 0;
      for (int t0 = 0; t0 < p.num_tokens; t0 += 32) {
        int v = t0 + lane < p.num_tokens ? start[t0 + lane + 1] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(kFullMask, v, o);
          if (lane >= o) v += u;
        }
        if (t0 + lane < p.num_tokens) start[t0 + lane + 1] = sum + v;
        sum += __shfl_sync(kFullMask, v, 31);
      }
      if (lane == 0) start[0] = 0;
    }
  } else if (threadIdx.x == 0 && blockIdx.x % p.blocks == 0 && p.errors) {
    const int len = __ldg(p.lens + blockIdx.x / p.blocks);
    if (len != list_len(p, len)) atomicAdd(p.errors, 1);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = __shfl_sync(kFullMask, *tmem_slot, 0);
  const uint32_t s_tmem = tmem, o_tmem = tmem + 128;  // S^T; O^T, NH columns a quarter
  Segments seg(p, start);
  // tiles of the CTA, and the barrier phase of the list of tile i
  int left = (int)(seg.stop - seg.at);
  if (!p.shared_out) left = list_tiles(list_len(p, __ldg(p.lens + blockIdx.x / p.blocks)));
  auto list_phase = [](uint32_t i) { return i / kAhead & 1; };

  if (warp < kSoftmaxWarps) {
    // ---- softmax ---------------------------------------------------------------------
    const int quad = warp & 3, half = warp >> 2;
    const int r = 32 * quad + lane;  // the thread's entry of a tile
    const uint32_t lanes = (uint32_t)quad << 21;
    const int col0 = half * COLS;  // .. and its first head
    uint32_t done = 0, segs = 0;  // phases of the barriers
    bool ok = true;
    while (ok && seg.next(p, start, lens)) {
      const int head0 = seg.block * NH, rows = min(NH, p.num_heads - head0);
      if (threadIdx.x < NH) refs[threadIdx.x] = 0.f;
      softmax_sync();

      bool fresh = true;  // no entry so far: the references mean nothing
      float l[COLS];
#pragma unroll
      for (int c = 0; c < COLS; ++c) l[c] = 0.f;
      for (int j = 0; j < seg.n; ++j, ++done) {
        const bool ready = p.wait_polls != 0 &&
                           await(kListFull + done % kAhead, list_phase(done)) &&
                           await(kSFull, done & 1);
        if (!ready) *dead = *quit = 1;
        const bool there = ready && lists[done % kAhead * kKeys + r] >= 0;
        // scores in units of log2, less their heads' references if asked for; PART heads
        // at a time. (The product is rounded before the reference, one of its kind, is
        // taken off: the entry that it is from has weight 1 however large the scores, and
        // so have those of the same score in all tiles and parts.)
        constexpr int PART = COLS < 16 ? COLS : 16;
        const float none = there ? 0.f : -INFINITY;
        auto scores = [&](int c0, float (&x)[PART], bool less) {
          uint32_t s[PART];
          __syncwarp();
          tc::ld(s, s_tmem + lanes + col0 + c0);
          tc::wait_ld();
          auto score = [&](uint32_t y, float ref) {
            return __fadd_rn(__fmul_rn(__uint_as_float(y), p.scale_log2), less ? none - ref : none);
          };
#pragma unroll
          for (int c = 0; c < PART; c += 4) {
            const float4 ref = *reinterpret_cast<const float4*>(refs + col0 + c0 + c);
            x[c] = score(s[c], ref.x);
            x[c + 1] = score(s[c + 1], ref.y);
            x[c + 2] = score(s[c + 2], ref.z);
            x[c + 3] = score(s[c + 3], ref.w);
          }
        };
        // The weights of PART heads, added to (taken off) the sums and handed over; not
        // those of a thread with a score far above its reference.
        auto weigh = [&](int c0, float sign) {
          float x[PART], top = -INFINITY;
          scores(c0, x, true);
#pragma unroll
          for (int c = 0; c < PART; c += 2) top = fmaxf(top, fmaxf(x[c], x[c + 1]));
          if (top > kRescaleAt) return true;
#pragma unroll
          for (int c1 = 0; c1 < PART; c1 += 8) {
            uint32_t w[4];
#pragma unroll
            for (int c = c1; c < c1 + 8; c += 2) {
              const float a = ex2(x[c]), b = ex2(x[c + 1]);
              l[c0 + c] = fmaf(a, sign, l[c0 + c]);
              l[c0 + c + 1] = fmaf(b, sign, l[c0 + c + 1]);
              w[(c - c1) >> 1] = pack_bf16x2(a, b);
            }
            *reinterpret_cast<uint4*>(smem + L::kP + r * 128 +
                                      ((((col0 + c0 + c1) >> 3) ^ (r & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
          return false;
        };
        bool moved = !ready || (fresh && there);
        if (ready) {
          tc::fence_after();
          if (!fresh) {
#pragma unroll
            for (int c0 = 0; c0 < COLS; c0 += PART) moved |= weigh(c0, 1.f);
          }
        }
        if (softmax_vote(moved)) {  // rare
          if (*quit) {
            ok = false;
            break;
          }
#pragma unroll
          for (int c0 = 0; c0 < COLS; c0 += PART) {
            // (what is lost in taking off what was added is lost against larger weights)
            if (!fresh) weigh(c0, -1.f);
            float x[PART];
            scores(c0, x, false);
            const float mine = columns(x, lane, [](float a, float b) { return fmaxf(a, b); });
            if (lane % (32 / PART) == 0) tops[quad * 64 + col0 + c0 + lane / (32 / PART)] = mine;
          }
          softmax_sync();
          if (threadIdx.x < NH) {  // each head's reference becomes the maximum
            const float old = refs[threadIdx.x];
            float top = fresh ? -INFINITY : old;
            for (int k = 0; k < 4; ++k) top = fmaxf(top, tops[k * 64 + threadIdx.x]);
            top = fmaxf(top, kNone);  // (as -inf less itself is NaN)
            moves[threadIdx.x] = ex2(old - top);
            refs[threadIdx.x] = top;
          }
          const bool rescale = !fresh;
          fresh = false;
          softmax_sync();
          if (rescale) {
#pragma unroll
            for (int c = 0; c < COLS; ++c) l[c] *= moves[col0 + c];
            // O^T is at rest: the scores came after the products before them
#pragma unroll 1
            for (int k = 0; k < kQuarters * COLS / 8; ++k) {
              const int c0 = col0 + 8 * (k % (COLS / 8));
              const uint32_t at = o_tmem + lanes + k / (COLS / 8) * NH + c0;
              uint32_t o[8];
              tc::ld8(o, at);
              tc::wait_ld();
#pragma unroll
              for (int c = 0; c < 8; ++c)
                o[c] = __float_as_uint(__uint_as_float(o[c]) * moves[c0 + c]);
              tc::st8(at, o);
            }
            tc::wait_st();
          }
#pragma unroll
          for (int c0 = 0; c0 < COLS; c0 += PART) weigh(c0, 1.f);
        } else if (fresh) {  // a tile without an entry: no weights
          uint4* const row = reinterpret_cast<uint4*>(smem + L::kP + r * 128);
          for (int c = 0; c < 8; ++c) row[c] = make_uint4(0, 0, 0, 0);
        }
        tma::fence_proxy_async();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(bar(kPFull));
          tc::mbar_arrive(bar(kListEmpty + done % kAhead));
        }
      }
      // ---- the unit's output, or a partial -------------------------------------------------
      const int slot_at = 2 * (int)blockIdx.x + (seg.count > 1);
      if (ok) {
        const float mine = columns(l, lane, [](float a, float b) { return a + b; });
        if (lane % (32 / COLS) == 0) tops[quad * 64 + col0 + lane / (32 / COLS)] = mine;
        if (!await(kODone, segs++ & 1)) *dead = *quit = 1;
        softmax_sync();
        ok = !*quit;
      }
      if (!ok) break;
      tc::fence_after();
      if (threadIdx.x < NH) {
        float sum = 0.f;
        for (int k = 0; k < 4; ++k) sum += tops[k * 64 + threadIdx.x];
        moves[threadIdx.x] = sum == 0.f ? 0.f : 1.f / sum;  // 0: no entry
        if (!seg.whole())
          p.part_sums[slot_at * NH + threadIdx.x] =
              make_float2(sum == 0.f ? -INFINITY : refs[threadIdx.x], sum);
      }
      softmax_sync();
      const bool whole = seg.whole();
      const int64_t row0 = whole ? (int64_t)seg.token * p.num_heads + head0 : (int64_t)slot_at * NH;
#pragma unroll 1
      for (int k = 0; k < kQuarters; ++k) {
        uint32_t o[COLS];
        tc::ld(o, o_tmem + lanes + k * NH + col0);
        tc::wait_ld();
        const int64_t at = (row0 + col0) * kDim + 128 * k + r;
        if (whole) {
          __nv_bfloat16* to = p.out + at;
#pragma unroll
          for (int c = 0; c < COLS; ++c)
            if (col0 + c < rows)
              to[c * kDim] = __float2bfloat16_rn(__uint_as_float(o[c]) * moves[col0 + c]);
        } else {
          float* to = p.part_o + at;
#pragma unroll
          for (int c = 0; c < COLS; ++c) to[c * kDim] = __uint_as_float(o[c]) * moves[col0 + c];
        }
      }
      tc::fence_before();
      softmax_sync();  // tops, moves and refs may be written again
    }
    // Given up: what this segment and those still to come should have held is marked.
    if (!ok) {
      do {
        const int rows = min(NH, p.num_heads - seg.block * NH);
        for (int i = threadIdx.x; i < NH * kDim; i += 32 * kSoftmaxWarps) {
          const int h = i / kDim;
          if (!seg.whole()) {
            if (i < NH)
              p.part_sums[(2 * (int)blockIdx.x + (seg.count > 1)) * NH + i] = make_float2(0.f, NAN);
          } else if (h < rows) {
            p.out[((int64_t)seg.token * p.num_heads + seg.block * NH) * kDim + i] =
                __float2bfloat16_rn(NAN);
          }
        }
      } while (seg.next(p, start, lens));
    }
  } else if (warp < kMmaWarp) {
    // ---- entries: four warps to a quarter of the dims ------------------------------------
    const int quarter = (warp - kSoftmaxWarps) >> 2;
    // The thread has fragment i of the quarter (8 dims; of the last one four coded dims and
    // four rotary ones) of 16 entries, 8 apart: the same place in the swizzle.
    const int i = lane & 15, key0 = 2 * (warp & 3) + (lane >> 4);
    // EARLY of them are decoded before their place is free, as far as registers go; with
    // many heads as many of the next tile's are read then too: the loads, a burst that
    // shared memory accesses wait behind, are then not all under way while the softmax is
    // (16 x 128 heads x 16384 entries 129 -> 115 us; few heads wait for the loads instead,
    // and with 32 all of it was 2 % slower).
    constexpr bool AHEAD = NH > 32;
    constexpr int N = 16, STRIDE = kKeys / N, EARLY = AHEAD ? 4 : 8;
    // of entry i of the half warp's: its slot (-1: none) and the exponents of the quarter,
    // those of the next tile as soon as its list is looked up
    int slot = -1;
    uint32_t ex = 0, next_ex = 0;
    bool listed = true;  // (a tile whose list did not come is not handed over)
    auto next_slots = [&](uint32_t tile) {
      slot = -1;
      if (tile >= (uint32_t)left) return;
      listed = await(kListFull + tile % kAhead, list_phase(tile));
      if (!listed) return;
      slot = lists[tile % kAhead * kKeys + key0 + STRIDE * i];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(kListEmpty + tile % kAhead));
    };
    auto slot_of = [&](int k) { return __shfl_sync(kFullMask, slot, (lane & 16) + k); };
    auto read_scales = [&]() {
      const uint8_t* e =
          p.cache + (int64_t)slot * dsv4::kEntry + dsv4::kScaleAt + 4 * (quarter >> 1);
      next_ex = slot < 0 ? 0 : __ldg(reinterpret_cast<const uint32_t*>(e));
    };
    // bytes over 134, or a NaN code: the whole warp decodes the long way
    auto large = [&]() { return ((ex & 0x7f7f7f7fu) + 0x79797979u) & ex; };
    const Factors f = factors();
    auto hand_over = [&]() {
      tma::fence_proxy_async();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(kXFull + quarter));
    };
    next_slots(0);
    read_scales();
    ex = next_ex;
    if (quarter < 3) {
      uint8_t* x_at = smem + L::kX + (2 * quarter + (i >> 3)) * L::kChunk + key0 * 128 +
                      (((i & 7) ^ (key0 & 7)) << 4);
      const uint32_t which = 0x4440 + 2 * (quarter & 1) + (i >> 3);  // the fragment's exponent
      uint2 code[N];
      auto read = [&](auto from, auto to) {  // the codes of entries from .. to - 1
#pragma unroll
        for (int k = from.value; k < to.value; ++k) {
          const int of = slot_of(k);
          const uint8_t* e = p.cache + (int64_t)of * dsv4::kEntry + 128 * quarter + 8 * i;
          code[k] = make_uint2(0, 0);
          if (of >= 0) code[k] = __ldg(reinterpret_cast<const uint2*>(e));
        }
      };
      read(I<0>(), I<N>());
      for (int tile = 0; listed && tile < left; ++tile) {
        uint32_t strange = large();
#pragma unroll
        for (int k = 0; k < N; ++k)
          strange = nan_bits(nan_bits(strange, code[k].x, f), code[k].y, f);
        const bool odd = __any_sync(kFullMask, (strange & 0x80808080u) != 0);
        auto byte_of = [&](int k) {
          return prmt(__shfl_sync(kFullMask, ex, (lane & 16) + k), which);
        };
        // not before the last tile's weights are there: the softmax, which everything
        // waits for, would share its issue slots with all this
        if (tile > 0 && !await(kPFull, (tile - 1) & 1)) break;
        if (AHEAD) {
          next_slots(tile + 1);
          read_scales();
        }
        // (two ways with a branch around each: with the choice made entry by entry both
        // were gone for every one, and a quarter took 2850 cycles instead of 1100)
        uint4 early[EARLY];
        if (!odd) {
#pragma unroll
          for (int k = 0; k < EARLY; ++k) early[k] = decode8(code[k], byte_of(k), f);
        } else {
#pragma unroll
          for (int k = 0; k < EARLY; ++k)
            early[k] = dsv4::dequant8(code[k], dsv4::ue8m0_scale(byte_of(k)));
        }
        if (AHEAD) read(I<0>(), I<EARLY>());
        if (tile > 0 && !await(kXEmpty + quarter, (tile - 1) & 1)) break;
#pragma unroll
        for (int k = 0; k < EARLY; ++k)
          *reinterpret_cast<uint4*>(x_at + STRIDE * k * 128) = early[k];
        if (!odd) {
#pragma unroll
          for (int k = EARLY; k < N; ++k)
            *reinterpret_cast<uint4*>(x_at + STRIDE * k * 128) = decode8(code[k], byte_of(k), f);
        } else {
#pragma unroll
          for (int k = EARLY; k < N; ++k)
            *reinterpret_cast<uint4*>(x_at + STRIDE * k * 128) =
                dsv4::dequant8(code[k], dsv4::ue8m0_scale(byte_of(k)));
        }
        hand_over();
        if (!AHEAD) {
          next_slots(tile + 1);
          read_scales();
          read(I<0>(), I<EARLY>());
        }
        read(I<EARLY>(), I<N>());
        ex = next_ex;
      }
    } else {
      uint8_t* x_at =
          smem + L::kX + 6 * L::kChunk + key0 * 128 + (((i >> 1) ^ (key0 & 7)) << 4) + 8 * (i & 1);
      uint32_t code[N];
      uint2 rope[N];
      auto read = [&](auto from, auto to) {  // the codes of entries from .. to - 1
#pragma unroll
        for (int k = from.value; k < to.value; ++k) {
          const int of = slot_of(k);
          const uint8_t* e = p.cache + (int64_t)of * dsv4::kEntry;
          code[k] = 0, rope[k] = make_uint2(0, 0);
          if (of >= 0) {
            code[k] = __ldg(reinterpret_cast<const uint32_t*>(e + 384 + 4 * i));
            rope[k] = __ldg(reinterpret_cast<const uint2*>(e + dsv4::kRopeAt + 8 * i));
          }
        }
      };
      read(I<0>(), I<N>());
      for (int tile = 0; listed && tile < left; ++tile) {
        uint32_t strange = large();
#pragma unroll
        for (int k = 0; k < N; ++k) strange = nan_bits(strange, code[k], f);
        const bool odd = __any_sync(kFullMask, (strange & 0x80808080u) != 0);
        auto byte_of = [&](int k) {
          return prmt(__shfl_sync(kFullMask, ex, (lane & 16) + k), 0x4442);
        };
        auto decoded = [&](int k) {
          const uint4 v = decode8(make_uint2(code[k], 0), byte_of(k), f);
          return make_uint2(v.x, v.y);
        };
        auto decoded_odd = [&](int k) {
          const uint4 v = dsv4::dequant8(make_uint2(code[k], 0), dsv4::ue8m0_scale(byte_of(k)));
          return make_uint2(v.x, v.y);
        };
        auto put = [&](int k, const uint2& v) {
          *reinterpret_cast<uint2*>(x_at + STRIDE * k * 128) = v;
          *reinterpret_cast<uint2*>(x_at + STRIDE * k * 128 + L::kChunk) = rope[k];
        };
        if (tile > 0 && !await(kPFull, (tile - 1) & 1)) break;
        if (AHEAD) {
          next_slots(tile + 1);
          read_scales();
        }
        uint2 early[EARLY];
        if (!odd) {
#pragma unroll
          for (int k = 0; k < EARLY; ++k) early[k] = decoded(k);
        } else {
#pragma unroll
          for (int k = 0; k < EARLY; ++k) early[k] = decoded_odd(k);
        }
        if (tile > 0 && !await(kXEmpty + quarter, (tile - 1) & 1)) break;
#pragma unroll
        for (int k = 0; k < EARLY; ++k) put(k, early[k]);
        if (AHEAD) read(I<0>(), I<EARLY>());
        if (!odd) {
#pragma unroll
          for (int k = EARLY; k < N; ++k) put(k, decoded(k));
        } else {
#pragma unroll
          for (int k = EARLY; k < N; ++k) put(k, decoded_odd(k));
        }
        hand_over();
        if (!AHEAD) {
          next_slots(tile + 1);
          read_scales();
          read(I<0>(), I<EARLY>());
        }
        read(I<EARLY>(), I<N>());
        ex = next_ex;
      }
    }
  } else if (warp == kMmaWarp) {
    // ---- the matrix instructions -------------------------------------------------------
    constexpr uint32_t qk = tc::instr_desc(NH, false), pv = tc::instr_desc(NH, true, true);
    const uint64_t x_desc = tc::smem_desc(base + L::kX, 16);
    const uint64_t q_desc = tc::smem_desc(base + L::kQ, 16);
    const uint64_t xt_desc = tc::smem_desc(base + L::kX, L::kChunk);
    const uint64_t p_desc = tc::smem_desc(base + L::kP, L::kChunk);
    uint32_t segs = 0;
    bool ok = true;
    for (uint32_t tile = 0; ok && tile < (uint32_t)left; ++tile) {
      ok = await(kListFull + tile % kAhead, list_phase(tile));
      const int where = place[tile % kAhead];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(kListEmpty + tile % kAhead));
      if (where & 1) ok = ok && await(kQFull, segs++ & 1);
#pragma unroll 1
      for (int q = 0; ok && q < kQuarters; ++q) {
        ok = await(kXFull + q, tile & 1);
        if (!ok) break;
        tc::fence_after();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t chunk = 2 * q + (k >> 2), off = (k & 3) * 32;
          tc::mma_ss(s_tmem, x_desc + ((chunk * L::kChunk + off) >> 4),
                     q_desc + ((chunk * L::kQChunk + off) >> 4), qk, q > 0 || k > 0);
        }
      }
      if (!ok) break;
      tc::commit(bar(kSFull));
      if (where & 2) tc::commit(bar(kQEmpty));
      ok = await(kPFull, tile & 1);
      if (!ok) break;
      tc::fence_after();
#pragma unroll 1
      for (int q = 0; q < kQuarters; ++q) {
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          tc::mma_ss(o_tmem + q * NH, xt_desc + ((2 * q * L::kChunk + k * 2048) >> 4),
                     p_desc + (k * 2048 >> 4), pv, !(where & 1) || k > 0);
        tc::commit(bar(kXEmpty + q));
      }
      if (where & 2) tc::commit(bar(kODone));
    }
    // Nothing may be in flight when the tensor memory goes: not the last products either,
    // which nobody waits for where a softmax warp gave up on them.
    tc::commit(bar(kDrain));
    tc::drain(bar(kDrain), 0);
    __syncwarp();
  } else if (warp == kListWarp) {
    // ---- the lists ------------------------------------------------------------------------
    bool ok = true, rejected = false;
    uint32_t tile = 0;
    while (ok && seg.next(p, start, lens)) {
      const int* list = p.slots + (int64_t)seg.token * p.list_width;
      for (int j = 0; ok && j < seg.n; ++j, ++tile) {
        int slot[kKeys / 32];
#pragma unroll
        for (int u = 0; u < kKeys / 32; ++u) {
          const int at = (seg.first + j) * kKeys + 32 * u + lane;
          slot[u] = at < seg.len ? __ldg(list + at) : -1;
          if (slot[u] < -1 || slot[u] >= p.num_slots) rejected = true, slot[u] = -1;
        }
        // into the L2 meanwhile: the loads behind the last tile's are a burst, which from
        // memory takes as long as the whole tile
#pragma unroll
        for (int u = 0; u < kKeys / 32; ++u) {
          if (slot[u] < 0) continue;
          const uint8_t* e = p.cache + (int64_t)slot[u] * dsv4::kEntry;
#pragma unroll
          for (int b = 0; b < dsv4::kEntry; b += 128) prefetch_l2(e + b);
          prefetch_l2(e + dsv4::kEntry - 1);
        }
        if (tile >= kAhead) ok = await(kListEmpty + tile % kAhead, list_phase(tile - kAhead));
        if (!ok) break;
#pragma unroll
        for (int u = 0; u < kKeys / 32; ++u)
          lists[tile % kAhead * kKeys + 32 * u + lane] = slot[u];
        if (lane == 0) place[tile % kAhead] = (j == 0 ? 1 : 0) | (j + 1 == seg.n ? 2 : 0);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(kListFull + tile % kAhead));
      }
    }
    if (rejected && p.errors) atomicAdd(p.errors, 1);
  } else if (warp >= kQueryWarp) {
    // ---- the queries, swizzled -------------------------------------------------------------
    for (uint32_t segs = 0; seg.next(p, start, lens); ++segs) {
      if (segs > 0 && !await(kQEmpty, (segs - 1) & 1)) break;
      const int head0 = seg.block * NH, rows = min(NH, p.num_heads - head0);
      const __nv_bfloat16* q = p.q + (int64_t)seg.token * p.q_stride + (int64_t)head0 * kDim;
      const int c = threadIdx.x & 63;  // the thread's fragment of every row
      const uint32_t to = base + L::kQ + (c >> 3) * L::kQChunk;
#pragma unroll 4
      for (int h = 0; h < NH; ++h)
        copy16(to + h * 128 + (((c & 7) ^ (h & 7)) << 4), h < rows ? q + h * kDim + 8 * c : p.q,
               h < rows);
      asm volatile("cp.async.wait_all;" ::: "memory");
      tma::fence_proxy_async();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(kQFull));
    }
  }
  tc::fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && p.errors && *dead) atomicAdd(p.errors, 1);
  if (warp == kMmaWarp) {
    tc::fence_after();
    tc::dealloc512(tmem);
  }
}

// ---- the join of the parts -------------------------------------------------------------

struct JoinParams {
  LatentParams x;
  int ctas;   // of the tiles' grid
  int heads;  // of a unit
};

constexpr int kJoinWarps = 4;

// One warp per row, the rows of one token to a CTA.  Which CTAs had the row's unit
// follows from the lists' lengths, as it did for them.
template <int FLIGHT>
__global__ void __launch_bounds__(kJoinWarps * 32) latent_join_kernel(const JoinParams p) {
  grid_dependency_wait();
  __shared__ int sums[2][kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_token = (p.x.num_heads + kJoinWarps - 1) / kJoinWarps;
  const int token = (int)blockIdx.x / per_token;
  const int head = ((int)blockIdx.x - token * per_token) * kJoinWarps + warp;
  int before = 0, all = 0;  // tiles (of a block of heads) of the tokens before, of all
  for (int t = threadIdx.x; t < p.x.num_tokens; t += kJoinWarps * 32) {
    const int n = list_tiles(list_len(p.x, __ldg(p.x.lens + t)));
    all += n;
    before += t < token ? n : 0;
  }
  before = __reduce_add_sync(kFullMask, before);
  all = __reduce_add_sync(kFullMask, all);
  if (lane == 0) sums[0][warp] = before, sums[1][warp] = all;
  __syncthreads();
  if (head >= p.x.num_heads) return;
  before = all = 0;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) before += sums[0][w], all += sums[1][w];
  const int n = list_tiles(list_len(p.x, __ldg(p.x.lens + token)));
  const int block = head / p.heads;
  const int64_t total = (int64_t)all * p.x.blocks;
  const int64_t a = (int64_t)before * p.x.blocks + (int64_t)block * n;
  const int ctas = Segments::busy(total, p.ctas);
  const int b0 = (int)(((a + 1) * ctas - 1) / total);  // the CTAs of tiles a and a + n - 1
  const int b1 = (int)(((a + n) * ctas - 1) / total);
  if (b0 == b1) return;  // one had them all
  const int parts = b1 - b0 + 1;
  auto at = [&](int s) {  // row of the part
    const bool second = s == 0 && Segments::border(total, b0, ctas) < a;
    return (int64_t)(2 * (b0 + s) + second) * p.heads + (head - block * p.heads);
  };
  float top = -INFINITY;
  for (int s = lane; s < parts; s += 32) top = fmaxf(top, p.x.part_sums[at(s)].x);
  top = group_max<32>(top);
  const float ref = top == -INFINITY ? 0.f : top;
  constexpr int V = kDim / 32;  // dims of a lane, four at a time
  float acc[V] = {};
  float sum = 0.f;
  for (int s0 = 0; s0 < parts; s0 += FLIGHT) {
    float2 w[FLIGHT];
    float4 v[FLIGHT][V / 4];
#pragma unroll
    for (int u = 0; u < FLIGHT; ++u) {
      w[u].x = -INFINITY;
      if (s0 + u >= parts) continue;
      w[u] = p.x.part_sums[at(s0 + u)];
      const float4* from = reinterpret_cast<const float4*>(p.x.part_o + at(s0 + u) * kDim) + lane;
#pragma unroll
      for (int k = 0; k < V / 4; ++k) v[u][k] = from[32 * k];
    }
#pragma unroll
    for (int u = 0; u < FLIGHT; ++u) {
      if (w[u].x == -INFINITY) continue;  // a part without an entry
      const float g = exp2f(w[u].x - ref) * w[u].y;
      sum += g;
#pragma unroll
      for (int k = 0; k < V / 4; ++k) {
        acc[4 * k] = fmaf(g, v[u][k].x, acc[4 * k]);
        acc[4 * k + 1] = fmaf(g, v[u][k].y, acc[4 * k + 1]);
        acc[4 * k + 2] = fmaf(g, v[u][k].z, acc[4 * k + 2]);
        acc[4 * k + 3] = fmaf(g, v[u][k].w, acc[4 * k + 3]);
      }
    }
  }
  const float f = sum == 0.f ? 0.f : 1.f / sum;
  uint2* out =
      reinterpret_cast<uint2*>(p.x.out + ((int64_t)token * p.x.num_heads + head) * kDim) + lane;
#pragma unroll
  for (int k = 0; k < V; k += 4)
    out[8 * k] = make_uint2(pack_bf16x2(acc[k] * f, acc[k + 1] * f),
                            pack_bf16x2(acc[k + 2] * f, acc[k + 3] * f));
}

// ---- launch ------------------------------------------------------------------------------

struct Plan {
  int heads, blocks;  // of a unit; units of a token
  bool shared_out;
  int64_t ctas;
  bool parts;         // units may fall to several CTAs
};

Plan plan_for(int64_t num_tokens, int num_heads, int list_width) {
  Plan s;
  const int64_t tiles = list_width > kKeys ? (list_width + kKeys - 1) / kKeys : 1;
  // As many heads to a unit as there are, up to 64, while that leaves less than half of
  // the SMs idle: fewer are more units, each quicker through its tile's steps (one token of
  // 64 heads x 2051 entries 18.0 us in 17 tiles, 14.5 in 68 of 16 heads).
  s.heads = num_heads <= 16 ? 16 : num_heads <= 32 ? 32 : 64;
  while (s.heads > 16 &&
         num_tokens * ((num_heads + s.heads - 1) / s.heads) * tiles * 2 <= kCtas)
    s.heads /= 2;
  s.blocks = (num_heads + s.heads - 1) / s.heads;
  const int64_t units = num_tokens * s.blocks;
  // (the tiles that are shared out are counted in 32 bits: past them a CTA would take heads that
  // are not there.  So many tiles keep all SMs busy as a CTA to a unit too, and a 64-bit count
  // costs registers that are not left: 112 -> 131 us at 16 x 128 heads x 16384 entries.)
  s.parts = s.shared_out = units <= kSharedUnits && tiles > 1 && units * tiles <= INT_MAX;
  s.ctas = !s.shared_out ? units : units * tiles < kCtas ? units * tiles : kCtas;
  return s;
}

template <int NH>
cudaError_t launch(const LatentParams& p, const Plan& s, cudaStream_t stream) {
  static std::atomic<int> cache[kMaxDevices];
  int per_sm = 0;
  cudaError_t e =
      tma::prepare(latent_tiles_kernel<NH>, kThreads, Layout<NH>::kSmem, cache, &per_sm);
  if (e != cudaSuccess) return e;
  return launch_kernel(latent_tiles_kernel<NH>, dim3((unsigned)s.ctas), dim3(kThreads),
                       Layout<NH>::kSmem, stream, p);
}

}  // namespace

int64_t latent_attn_workspace(int64_t num_tokens, int num_heads, int list_width) {
  const Plan s = plan_for(num_tokens, num_heads, list_width);
  return s.parts ? s.ctas * 2 * s.heads * (kDim + 2) * 4 : 0;
}

cudaError_t launch_latent_attn(const LatentAttnArgs& a, cudaStream_t stream) {
  const Plan s = plan_for(a.num_tokens, a.num_heads, a.list_width);
  LatentParams p;
  memset(&p, 0, sizeof p);
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.q_stride = a.q_stride;
  p.num_tokens = a.num_tokens;
  p.num_heads = a.num_heads;
  p.blocks = s.blocks;
  p.cache = a.kv_cache;
  p.num_slots = a.num_slots;
  p.slots = a.slots;
  p.list_width = a.list_width;
  p.lens = a.lens;
  p.scale_log2 = a.scale * kLog2e;
  p.shared_out = s.shared_out;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  if (s.parts) {
    p.part_o = static_cast<float*>(a.workspace);
    p.part_sums = reinterpret_cast<float2*>(p.part_o + s.ctas * 2 * s.heads * kDim);
  }
  p.errors = a.errors;
  p.wait_polls = tile_wait_limit();
  cudaError_t e = cudaErrorInvalidValue;
  switch (s.heads) {
    case 16: e = launch<16>(p, s, stream); break;
    case 32: e = launch<32>(p, s, stream); break;
    case 64: e = launch<64>(p, s, stream); break;
  }
  if (e != cudaSuccess || !s.parts) return e;
  JoinParams j;
  j.x = p;
  j.ctas = (int)s.ctas;
  j.heads = s.heads;
  const int64_t grid = (int64_t)a.num_tokens * ((a.num_heads + kJoinWarps - 1) / kJoinWarps);
  // Few rows wait for their loads, many for the SMs' registers: 2 x 64 rows 23.8 us with two
  // parts in flight and 19.9 with eight, 152 x 64 rows 96.3 and 108.1.
  return launch_kernel((int64_t)a.num_tokens * a.num_heads <= 512 ? latent_join_kernel<8>
                                                                  : latent_join_kernel<2>,
                       dim3((unsigned)grid), dim3(kJoinWarps * 32), 0, stream, j);
}

}  // namespace kvq
