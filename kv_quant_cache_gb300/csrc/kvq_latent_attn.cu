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
//     more than 2^8, so that the exchange of maxima between lanes, and the
//     rescaling of O^T, are rare; weights go to shared memory as rows of heads;
//   * warps 8-15: read entries (8 bytes a lane, a whole tile ahead in registers) and
//     decode them, a quarter of the dims at a time: as soon as the second product of the
//     tile before is done with a quarter, the next tile's takes its place;
//   * warp 16: issues the matrix instructions.
//
// With few units a CTA to an SM takes an equal share of all tiles of all lists, from
// the lists' actual lengths; a unit that falls to several CTAs goes to partials,
// which a second launch joins.  With many units a CTA takes one.
#include <cstring>

#include "kvq_dsv4_entry.cuh"
#include "kvq_paged_attn.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

constexpr int kDim = dsv4::kDim;
constexpr int kKeys = 128;          // entries of a tile
constexpr int kQuarters = 4;        // of the dims
constexpr int kSoftmaxWarps = 8, kLoadWarps = 8;
constexpr int kMmaWarp = kSoftmaxWarps + kLoadWarps;
constexpr int kThreads = 32 * (kMmaWarp + 4);  // (three warps of that group have no work)
// Registers of the softmax, loading and other warps: of the 96 each that a CTA of 20
// warps is launched with.
constexpr int kSoftmaxRegs = 104, kLoadRegs = 120, kOtherRegs = 32;
static_assert(2 * kSoftmaxRegs + 2 * kLoadRegs + kOtherRegs <= 5 * 96, "registers of an SM's part");
constexpr int kSharedUnits = 4 * 152;  // up to so many units the tiles are shared out
constexpr int kCtas = 152;             // .. to so many CTAs
constexpr float kRescaleAt = 8.f;      // log2 by which a score may exceed the reference

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
  float* part_lse;           // [CTAs][2][heads of a unit]
  int* errors;
  uint32_t wait_polls;       // of a barrier, before the waiter gives up
};

// mbarriers, by index
enum { kXFull = 0, kXEmpty = 4, kQFull = 8, kSFull = 9, kPFull = 10, kODone = 11, kDrain = 12,
       kBarriers = 13 };

template <int NH>
struct Layout {
  static constexpr int kChunk = kKeys * 128;            // 64 dims of a tile
  static constexpr int kX = 0;                          // 8 chunks
  static constexpr int kP = 8 * kChunk;                 // 128 rows of up to 64 heads
  static constexpr int kQChunk = NH * 128;              // 64 dims of Q
  static constexpr int kQ = kP + kChunk;
  static constexpr int kTops = kQ + 8 * kQChunk;        // [4 quadrants of lanes][NH]
  static constexpr int kRef = kTops + 4 * 64 * 4;       // [NH] references
  static constexpr int kStart = kRef + 64 * 4;          // [tokens + 1] first tiles
  static constexpr int kBars = kStart + (kSharedUnits + 8) * 4;
  static constexpr int kEnd = kBars + 16 * 8 + 32;
  static constexpr int kSmem = kEnd + 1024;             // room to align the base
  static_assert(kSmem <= 227 * 1024, "shared memory per CTA");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
  __device__ __forceinline__ bool next(const LatentParams& p, const int* start) {
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
      len = list_len(p, __ldg(p.lens + token));
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
  int* start = reinterpret_cast<int*>(smem + L::kStart);
  const uint32_t bars = base + L::kBars;
  int* shared_state = reinterpret_cast<int*>(smem + L::kBars + 16 * 8);
  volatile int* dead = shared_state;      // a wait ran out
  volatile int* quit = shared_state + 1;  // .. of a softmax warp
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(shared_state + 2);
  auto bar = [&](int i) { return bars + 8u * i; };
  auto await = [&](int i, uint32_t parity) {
    return tc::wait_warp(bar(i), parity, dead, p.wait_polls);
  };
  const int warp = __shfl_sync(kFullMask, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBarriers; ++i)
      tma::mbar_init(bar(i), i < kXEmpty ? kLoadWarps
                             : i == kQFull || i == kPFull ? kSoftmaxWarps : 1);
    tma::mbar_init_fence();
    *dead = *quit = 0;
  }
  if (warp == kMmaWarp) tc::alloc512(tma::smem_addr(tmem_slot));
  grid_dependency_wait();
  if (p.shared_out) {
    // the first tile of each token, of one block of heads
    for (int t = threadIdx.x; t < p.num_tokens; t += kThreads) {
      const int len = __ldg(p.lens + t);
      start[t + 1] = list_tiles(list_len(p, len));
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

  if (warp < kSoftmaxWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---- softmax ---------------------------------------------------------------------
    const int quad = warp & 3, half = warp >> 2;
    const int r = 32 * quad + lane;  // the thread's entry of a tile
    const uint32_t lanes = (uint32_t)quad << 21;
    const int col0 = half * COLS;  // .. and its first head
    uint32_t done = 0, segs = 0;  // phases of the barriers
    bool ok = true, rejected = false;
    while (ok && seg.next(p, start)) {
      const int head0 = seg.block * NH, rows = min(NH, p.num_heads - head0);
      // Q, swizzled; the products that read the last segment's are done
      for (int i = threadIdx.x; i < NH * 64; i += 32 * kSoftmaxWarps) {
        const int h = i >> 6, c = i & 63;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (h < rows)
          v = __ldg(reinterpret_cast<const uint4*>(p.q + (int64_t)seg.token * p.q_stride +
                                                   (int64_t)(head0 + h) * kDim) + c);
        *reinterpret_cast<uint4*>(smem + L::kQ + (c >> 3) * L::kQChunk + h * 128 +
                                  (((c & 7) ^ (h & 7)) << 4)) = v;
      }
      tma::fence_proxy_async();
      if (threadIdx.x < NH) refs[threadIdx.x] = -INFINITY;
      softmax_sync();
      if (lane == 0) tc::mbar_arrive(bar(kQFull));

      const int* list = p.slots + (int64_t)seg.token * p.list_width;
      auto listed = [&](int tile) {  // the thread's slot of a tile, -1: none
        const int at = tile * kKeys + r;
        return at < seg.len ? __ldg(list + at) : -1;
      };
      int slot = listed(seg.first);
      float l[COLS];
#pragma unroll
      for (int c = 0; c < COLS; ++c) l[c] = 0.f;
      for (int j = 0; j < seg.n; ++j, ++done) {
        const bool there = slot >= 0 && slot < p.num_slots;
        rejected |= !there && slot != -1;
        if (j + 1 < seg.n) slot = listed(seg.first + j + 1);
        const bool ready = p.wait_polls != 0 && await(kSFull, done & 1);
        if (!ready) *dead = *quit = 1;
        bool moved = !ready;
        float x[COLS];
        auto scores = [&]() {  // in units of log2
          uint32_t s[COLS];
          tc::ld(s, s_tmem + lanes + col0);
          tc::wait_ld();
#pragma unroll
          for (int c = 0; c < COLS; ++c)
            x[c] = there ? __uint_as_float(s[c]) * p.scale_log2 : -INFINITY;
        };
        if (ready) {
          tc::fence_after();
          scores();
#pragma unroll
          for (int c = 0; c < COLS; ++c) moved |= x[c] > refs[col0 + c] + kRescaleAt;
        }
        if (softmax_vote(moved)) {  // rare
          if (*quit) {
            ok = false;
            break;
          }
          const float mine = columns(x, lane, [](float a, float b) { return fmaxf(a, b); });
          if (lane % (32 / COLS) == 0) tops[quad * 64 + col0 + lane / (32 / COLS)] = mine;
          softmax_sync();
#pragma unroll
          for (int c0 = 0; c0 < COLS; c0 += 8) {
            float f[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float old = refs[col0 + c0 + c];
              float to = old;
#pragma unroll
              for (int k = 0; k < 4; ++k) to = fmaxf(to, tops[k * 64 + col0 + c0 + c]);
              f[c] = to == old ? 1.f : ex2(old - to);
              l[c0 + c] *= f[c];
            }
            if (j == 0) continue;
            // O^T is at rest: the scores came after the products before them
#pragma unroll 1
            for (int k = 0; k < kQuarters; ++k) {
              const uint32_t at = o_tmem + lanes + k * NH + col0 + c0;
              uint32_t o[8];
              tc::ld8(o, at);
              tc::wait_ld();
#pragma unroll
              for (int c = 0; c < 8; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f[c]);
              tc::st8(at, o);
            }
          }
          tc::wait_st();
          softmax_sync();
          if (threadIdx.x < NH) {
            float to = refs[threadIdx.x];
            for (int k = 0; k < 4; ++k) to = fmaxf(to, tops[k * 64 + threadIdx.x]);
            refs[threadIdx.x] = to;
          }
          softmax_sync();
          scores();
        }
#pragma unroll
        for (int c0 = 0; c0 < COLS; c0 += 8) {
          uint32_t w[4];
#pragma unroll
          for (int c = c0; c < c0 + 8; c += 2) {
            const float ra = refs[col0 + c], rb = refs[col0 + c + 1];
            const float a = ex2(x[c] - (ra == -INFINITY ? 0.f : ra));
            const float b = ex2(x[c + 1] - (rb == -INFINITY ? 0.f : rb));
            l[c] += a, l[c + 1] += b;
            w[(c - c0) >> 1] = pack_bf16x2(a, b);
          }
          *reinterpret_cast<uint4*>(smem + L::kP + r * 128 +
                                    ((((col0 + c0) >> 3) ^ (r & 7)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
        tma::fence_proxy_async();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(kPFull));
      }
      // ---- the unit's output, or a partial -------------------------------------------------
      if (ok) {
        const bool last = await(kODone, segs++ & 1);
        if (!last) *dead = *quit = 1;
        const float mine = columns(l, lane, [](float a, float b) { return a + b; });
        if (lane % (32 / COLS) == 0) tops[quad * 64 + col0 + lane / (32 / COLS)] = mine;
        softmax_sync();
        ok = !*quit;
      }
      if (!ok) break;
      tc::fence_after();
      const int slot_at = 2 * (int)blockIdx.x + (seg.count > 1);
      float f[COLS];
#pragma unroll
      for (int c = 0; c < COLS; ++c) {
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) sum += tops[k * 64 + col0 + c];
        f[c] = sum == 0.f ? 0.f : 1.f / sum;  // 0: no entry
        if (!seg.whole() && r == 0) {
          const float ref = refs[col0 + c];
          p.part_lse[slot_at * NH + col0 + c] =
              sum == 0.f ? -INFINITY : (ref == -INFINITY ? 0.f : ref) + log2f(sum);
        }
      }
#pragma unroll 1
      for (int k = 0; k < kQuarters; ++k) {
        uint32_t o[COLS];
        tc::ld(o, o_tmem + lanes + k * NH + col0);
        tc::wait_ld();
        const int d = 128 * k + r;
#pragma unroll
        for (int c = 0; c < COLS; ++c) {
          const float v = __uint_as_float(o[c]) * f[c];
          if (seg.whole()) {
            if (col0 + c < rows)
              p.out[((int64_t)seg.token * p.num_heads + head0 + col0 + c) * kDim + d] =
                  __float2bfloat16_rn(v);
          } else {
            p.part_o[((int64_t)slot_at * NH + col0 + c) * kDim + d] = v;
          }
        }
      }
      tc::fence_before();
      softmax_sync();  // tops, refs and Q may be written again
    }
    // Given up: what this segment and those still to come should have held is marked.
    if (!ok) {
      do {
        const int rows = min(NH, p.num_heads - seg.block * NH);
        for (int i = threadIdx.x; i < NH * kDim; i += 32 * kSoftmaxWarps) {
          const int h = i / kDim;
          if (!seg.whole()) {
            if (i < NH) p.part_lse[(2 * (int)blockIdx.x + (seg.count > 1)) * NH + i] = NAN;
          } else if (h < rows) {
            p.out[((int64_t)seg.token * p.num_heads + seg.block * NH) * kDim + i] =
                __float2bfloat16_rn(NAN);
          }
        }
      } while (seg.next(p, start));
    }
    if (rejected && half == 0 && p.errors) atomicAdd(p.errors, 1);
  } else if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
    // ---- entries: a quarter of the dims at a time -------------------------------------------
    // The thread has fragment i (8 dims) of each quarter, of 8 entries 16 apart.
    const int lw = warp - kSoftmaxWarps, i = lane & 15;
    const int key0 = 2 * lw + (lane >> 4);
    constexpr int N = kKeys / 16;
    uint2 code[kQuarters][N], more[N];
    uint32_t ex;  // four exponents of entry i / 2 of the thread's half warp
    int slot[N];
    Segments ahead = seg;
    int ahead_j = 0;
    bool any = ahead.next(p, start);
    // the slots of the next tile that is to be read (-1: none)
    auto slots_of_next = [&]() {
#pragma unroll
      for (int k = 0; k < N; ++k) slot[k] = -1;
      if (!any) return;
      const int* list = p.slots + (int64_t)ahead.token * p.list_width;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int at = (ahead.first + ahead_j) * kKeys + key0 + 16 * k;
        if (at < ahead.len) slot[k] = __ldg(list + at);
        if (slot[k] >= p.num_slots) slot[k] = -1;
      }
      if (++ahead_j == ahead.n) {
        any = ahead.next(p, start);
        ahead_j = 0;
      }
    };
    auto entry = [&](int k) { return p.cache + (int64_t)slot[k] * dsv4::kEntry; };
    auto read = [&](int q) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        code[q][k] = make_uint2(0, 0);
        if (q == 3) more[k] = make_uint2(0, 0);
        if (slot[k] < 0) continue;
        if (q < 3 || i < 8) {
          code[q][k] = __ldg(reinterpret_cast<const uint2*>(entry(k) + 128 * q + 8 * i));
        } else {
          const uint2* rope =
              reinterpret_cast<const uint2*>(entry(k) + dsv4::kRopeAt + 16 * (i - 8));
          code[q][k] = __ldg(rope);
          more[k] = __ldg(rope + 1);
        }
      }
    };
    auto read_scales = [&]() {
      int of = -1;
#pragma unroll
      for (int k = 0; k < N; ++k) of = i >> 1 == k ? slot[k] : of;
      ex = of < 0 ? 0
                  : __ldg(reinterpret_cast<const uint32_t*>(p.cache + (int64_t)of * dsv4::kEntry +
                                                            dsv4::kScaleAt + 4 * (i & 1)));
    };
    slots_of_next();
#pragma unroll
    for (int q = 0; q < kQuarters; ++q) read(q);
    read_scales();
    uint32_t tile = 0;
    bool ok = true;
    while (ok && seg.next(p, start)) {
      for (int j = 0; ok && j < seg.n; ++j, ++tile) {
        slots_of_next();
#pragma unroll
        for (int q = 0; q < kQuarters; ++q) {
          if (tile > 0) ok = ok && await(kXEmpty + q, (tile - 1) & 1);
          if (!ok) break;
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const int r = key0 + 16 * k;
            const uint32_t four = __shfl_sync(kFullMask, ex, (lane & 16) + 2 * k + (q >> 1));
            uint4 v;
            if (q < 3 || i < 8) {
              const uint32_t byte = four >> (16 * (q & 1) + (i & 8)) & 0xffu;
              v = dsv4::dequant8(code[q][k], dsv4::ue8m0_scale(byte));
            } else {
              v = make_uint4(code[q][k].x, code[q][k].y, more[k].x, more[k].y);
            }
            *reinterpret_cast<uint4*>(smem + L::kX + (2 * q + (i >> 3)) * L::kChunk + r * 128 +
                                      (((i & 7) ^ (r & 7)) << 4)) = v;
          }
          tma::fence_proxy_async();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar(kXFull + q));
          read(q);
        }
        read_scales();
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  }
  if (warp == kMmaWarp) {
    // ---- the matrix instructions -------------------------------------------------------
    constexpr uint32_t qk = tc::instr_desc(NH, false), pv = tc::instr_desc(NH, true, true);
    const uint64_t x_desc = tc::smem_desc(base + L::kX, 16);
    const uint64_t q_desc = tc::smem_desc(base + L::kQ, 16);
    const uint64_t xt_desc = tc::smem_desc(base + L::kX, L::kChunk);
    const uint64_t p_desc = tc::smem_desc(base + L::kP, L::kChunk);
    uint32_t tile = 0, segs = 0;
    bool ok = true;
    while (ok && seg.next(p, start)) {
      ok = await(kQFull, segs & 1);
      for (int j = 0; ok && j < seg.n; ++j, ++tile) {
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
        ok = await(kPFull, tile & 1);
        if (!ok) break;
        tc::fence_after();
        for (int q = 0; q < kQuarters; ++q) {
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            tc::mma_ss(o_tmem + q * NH, xt_desc + ((2 * q * L::kChunk + k * 2048) >> 4),
                       p_desc + (k * 2048 >> 4), pv, j > 0 || k > 0);
          tc::commit(bar(kXEmpty + q));
        }
      }
      if (ok) {
        tc::commit(bar(kODone));
        ++segs;
      }
    }
    if (!ok) {  // nothing may be in flight when the tensor memory goes
      tc::commit(bar(kDrain));
      tc::drain(bar(kDrain), 0);
      __syncwarp();
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
  for (int s = lane; s < parts; s += 32) top = fmaxf(top, p.x.part_lse[at(s)]);
  top = group_max<32>(top);
  const float ref = top == -INFINITY ? 0.f : top;
  constexpr int V = kDim / 32;  // dims of a lane, four at a time
  float acc[V] = {};
  float sum = 0.f;
  for (int s = 0; s < parts; ++s) {
    const float lse = p.x.part_lse[at(s)];
    if (lse == -INFINITY) continue;  // a part without an entry
    const float w = exp2f(lse - ref);
    sum += w;
    const float4* from = reinterpret_cast<const float4*>(p.x.part_o + at(s) * kDim) + lane;
#pragma unroll
    for (int k = 0; k < V; k += 4) {
      const float4 v = from[8 * k];
      acc[k] = fmaf(w, v.x, acc[k]), acc[k + 1] = fmaf(w, v.y, acc[k + 1]);
      acc[k + 2] = fmaf(w, v.z, acc[k + 2]), acc[k + 3] = fmaf(w, v.w, acc[k + 3]);
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
  s.heads = num_heads <= 16 ? 16 : num_heads <= 32 ? 32 : 64;
  s.blocks = (num_heads + s.heads - 1) / s.heads;
  const int64_t units = num_tokens * s.blocks;
  const int64_t tiles = list_width > kKeys ? (list_width + kKeys - 1) / kKeys : 1;
  s.parts = s.shared_out = units <= kSharedUnits && tiles > 1;
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
  return s.parts ? s.ctas * 2 * s.heads * (kDim + 1) * 4 : 0;
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
    p.part_lse = p.part_o + s.ctas * 2 * s.heads * kDim;
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
  return launch_kernel(latent_join_kernel, dim3((unsigned)grid), dim3(kJoinWarps * 32), 0, stream,
                       j);
}

}  // namespace kvq
