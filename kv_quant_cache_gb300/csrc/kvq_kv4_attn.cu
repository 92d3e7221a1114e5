// kvq_kv4_attn.cu -- attention over the paged cache held in 4 bits, for the few
// query rows of a decode step or a short chunk.
//
// One cluster of 1..8 CTAs takes up to 8, 16, 24 or 32 query rows of one request and kv
// head (tokens x heads of the group) and the request's keys, its CTAs a part each.
// A warp works alone on every kWarps-th group of 16 keys, with an online softmax of
// its own.  With q_j the row's dims of group j of 64, and n = c - 8 the codes:
//   S   = scale sum_j ( s_kj (q_j n_kj) + z_kj sum(q_j) )
//   O_j = sum_k (P_k s_kj) n_kj + sum_k P_k z_kj
// so no code is ever multiplied by its scale: codes become bf16 integers by a
// mask and a product, two at a time, and go straight into 16x8x16
// matrix instructions.  K's scales (times `scale`) are applied to S in fp32; K's zeros,
// bf16 as they are, meet scale sum(q_j) in three bf16 values (24 bits of it) in one more
// matrix instruction; V's scales are applied to the weights P, whose product is rounded
// once to bf16 (the row sum adds the unrounded P), V's zeros to P in fp32.  Every second
// code comes out as a quarter of n: the other dims of Q are divided by 4 (exact), S
// multiplied by it, and so are those dims of O.
//
// The codes are the first operand of both products, S^T = K Q^T and O^T = V^T P^T:
// 16 keys (or dims) against 8 rows, so that the 1 to 8 rows that most models have to
// a kv head fill the instruction, and what is done per score is done on no
// padding.  More rows are more second operands to the same codes.  The transposed
// P takes one matrix transposition in registers.
//
// The reference of a row's softmax moves only when a score exceeds it by more than 8 in
// units of log2, a weight of 2^8, which spares the exchange of maxima: until then weights
// above 1 are as exact as those below.  It starts at the least finite number, so that a score
// of -inf weighs nothing wherever it comes.
//
// A group's codes come in by 16-byte asynchronous copies, three groups ahead, into
// a ring that only this warp uses, so that there is no CTA barrier in the loop.
// 32-byte pieces (a group of dims of one key) are exchanged so that the four
// keys that a load touches lie in different banks; the matrix instructions may take
// the keys in any order, and key_of() is one that does for the loads of K and of V.
//
// What bounds it: instructions, and their latencies.  A step of 16 keys of 128 dims and up to
// 8 rows is 359 of a warp (150 decode the codes, 17 are matrix instructions), for 2.3 KB: 64
// sequences x 32768 keys x 8 heads take 363 us, 5.0 TB/s.  Nothing is full there: issue slots
// are 66 % busy, memory 53 %, and the 16 warps to an SM that registers allow wait for results
// and for the ALU pipe.  With 24 and more rows of 64 dims, 16 of 128 and 8 of 256 they are 8,
// and latencies weigh more.
#include <cooperative_groups.h>

#include <type_traits>

#include "kvq_kv4.cuh"
#include "kvq_paged_attn.cuh"
#include "kvq_tma.cuh"

namespace cg = cooperative_groups;

namespace kvq {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxCluster = 8;
constexpr int kStep = 16;   // keys of one step of a warp
constexpr int kStages = 4;
constexpr int kWaves = 16;  // of CTAs, into which long ranges are cut at most
constexpr float kRescaleAt = 8.f;  // log2 by which a score may exceed the reference
constexpr float kNone = -3.402823466e38f;  // the reference before the first score

struct Attn4Params {
  const __nv_bfloat16* q;
  int64_t q_stride;
  const uint8_t* cache;
  int num_q, num_kv, group;  // group = num_q / num_kv
  int per_request;           // tokens of a request
  int tiles;                 // row tiles of a request and kv head
  int64_t num_pages;
  int page_size;
  int page_shift;            // log2 of page_size, -1: not a power of two
  const int* table;
  int table_width;
  const int* lens;
  float scale_log2;
  int cluster, splits;
  int part_steps;            // steps of a CTA's part, at least; 0: an equal share
  __nv_bfloat16* out;
  Partials parts;            // with several splits
  int* errors;
  int trigger_from;
};

// CTAs of an SM, by the registers of D dims and NT times 8 query rows
constexpr int ctas_of(int D, int NT) {
  // (three to an SM, of fewer registers each, were slower at 64 dims and 32 rows, 46 us
  // for 31, and at 128 and 24, 148 for 91)
  return D * NT <= 64 ? 5 : D * NT <= 128 ? 4 : 2;
}

// D dims, NT times 8 query rows.
template <int D, int NT>
struct Shape4 {
  static constexpr int kRows = 8 * NT;
  static constexpr int kCtas = ctas_of(D, NT);
  // Steps of the loop's body: four make places in the ring constants (64 sequences x 32768
  // keys 392 -> 384 us, 40 x 8 heads of 64 dims x 8192 keys 60 -> 53), where registers are
  // left for it (24 rows of 128 dims 71 -> 73, 16 of 256 61 -> 63).
  static constexpr int kUnroll = D * NT <= 256 && D < 256 ? 4 : D == 256 ? 2 : 1;
  // Two steps at a time where there are few warps to hide a step's latencies, and registers
  // for it (16 rows of 128 dims 51.5 -> 49.2 us, 24 of 64 24.7 -> 24.0, 8 of 256 105 ->
  // 104; 32 of 64 the same, 24 of 128 71 -> 74, 32 of 128 111 -> 160).
  static constexpr bool kPair = D * NT > 128 && D * NT <= 256 && NT < 4;
  static constexpr int kGroups = D / kv4::kGroup;
  static constexpr int kCodes = kStep * D / 2;           // bytes of 16 keys' codes
  static constexpr int kMeta = kStep * kGroups * 4;      // .. scales and zeros
  static constexpr int kStage = 2 * (kCodes + kMeta);    // K codes, V codes, K meta, V meta
  static constexpr int kRing = kStages * kStage;
  static constexpr int kPad = D + 8;                     // fp32 values of an output row
  static constexpr int kOut = kRows * kPad * 4;          // a warp's output takes its ring's place
  static constexpr int kWarp = kRing > kOut ? kRing : kOut;
  static constexpr int kState = kWarps * kRows * 8;      // {m, l} per warp and row
  static constexpr int kLse = kRows * 4;
  static constexpr int kSmem = kWarps * kWarp + kState + kLse;
  static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "shared memory of an SM");
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst),
               "l"(__cvta_generic_to_global(src))
               : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// (not volatile: the compiler may move these about, as loads and products of a step
// have nothing to do with each other)
__device__ __forceinline__ void mma(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The key of a step that stands at row (or column) n of half h of the matrix
// instructions: keys that one load touches differ in their lowest two bits.
__device__ __forceinline__ int key_of(int h, int n) { return 8 * h + (n ^ (n >> 2)); }

// Where the 32-byte piece of key r, group j lies.
template <int GROUPS>
__device__ __forceinline__ uint32_t piece_at(int r, int j) {
  if (GROUPS == 1) return r * 32;
  if (GROUPS == 2) return r * 64 + ((j ^ (r >> 1 & 1)) << 5);
  return r * 128 + ((j ^ (r & 3)) << 5);
}

__device__ __forceinline__ uint32_t fma2(uint32_t x, uint32_t a, uint32_t b) {
  uint32_t y;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(x), "r"(a), "r"(b));
  return y;
}

// The codes in the low four bits of each half, less 8; and those in the next four, less
// 8, a quarter of that.  128 + c is a mask away; the number whose bits are 16 c is 16 c
// times the smallest there is, up to 8 bits, and one product with 2^127 mends that.
// Neither takes a shift.  (`big` is 0x43004300 from a register: an instruction takes one
// constant, and with two the mask and the bits would be two of them.)
__device__ __forceinline__ uint32_t low_codes(uint32_t w, uint32_t big) {
  uint32_t x;
  asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(x) : "r"(w), "r"(big));
  return fma2(x, 0x3f803f80u, 0xc308c308u);  // 1, -136
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w) {
  return fma2(w & 0x00f000f0u, 0x7f007f00u, 0xc000c000u);  // 2^127, -2
}

// Transposes an 8x8 matrix of 16-bit values, two neighbours of a row to a lane.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The upper halves of two words.
__device__ __forceinline__ uint32_t highs(uint32_t a, uint32_t b) {
  return __byte_perm(a, b, 0x7632);
}

// N words at once
template <int N>
__device__ __forceinline__ void words(uint32_t (&w)[N], const uint32_t* from) {
  if (N == 1) {
    w[0] = *from;
  } else if (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(from);
    w[0] = x.x, w[N > 1] = x.y;
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(from);
    w[0] = x.x, w[N > 1] = x.y, w[N > 2 ? 2 : 0] = x.z, w[N > 2 ? 3 : 0] = x.w;
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, Shape4<D, NT>::kCtas)
attn4_kernel(const Attn4Params p) {
  using S = Shape4<D, NT>;
  constexpr int GROUPS = S::kGroups, kRows = S::kRows;
  extern __shared__ __align__(128) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  grid_dependency_sync(p.trigger_from);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;  // the lane's place in a matrix fragment
  float2* state = reinterpret_cast<float2*>(smem + kWarps * S::kWarp);
  float* part_lse = reinterpret_cast<float*>(smem + kWarps * S::kWarp + S::kState);
  const int rank = p.cluster > 1 ? (int)(blockIdx.x % p.cluster) : 0;
  const int unit = (int)blockIdx.x / p.cluster;

  // ---- which rows: of request `req`, rows row0 .. of its (token, head) pairs ---------
  const int tile = unit % p.tiles, per = unit / p.tiles;
  const int kv_head = per % p.num_kv, req = per / p.num_kv;
  const int row0 = tile * kRows;
  const int rows = min(kRows, p.per_request * p.group - row0);
  const int64_t t0 = (int64_t)req * p.per_request;
  auto row_of = [&](int r) {  // token * num_q + head
    const int u = (row0 + r) / p.group;
    return (t0 + u) * p.num_q + kv_head * p.group + (row0 + r - u * p.group);
  };

  // ---- what each row sees -----------------------------------------------------------
  bool rejected = false;
  int len = 0;  // of lane r's row
  if (lane < rows) {
    len = __ldg(p.lens + t0 + (row0 + lane) / p.group);
    const int64_t room = (int64_t)p.table_width * p.page_size;
    if (len < 0) rejected = true, len = 0;
    if (len > room) rejected = true, len = (int)room;
  }
  const int most = __reduce_max_sync(kFullMask, len);
  const int least = __reduce_min_sync(kFullMask, lane < rows ? len : most);

  // ---- which keys: an equal share of the request's groups of 16, or parts of a given size,
  // of a larger one where so many parts would not reach the end -----------------------------
  const int parts = p.cluster * p.splits;
  const int all_steps = most / kStep + (most % kStep != 0);
  const int share = max(p.part_steps, (all_steps + parts - 1) / parts);
  const int64_t begin = (int64_t)share * (blockIdx.y * p.cluster + rank);
  // A part past the request's end, for all CTAs of the cluster (the first part, where there is
  // no key): its sums say so, and the join reads no more of it.  Tables are as wide as the
  // longest request may get, so most parts may be like this.
  if (p.splits > 1 && (int64_t)share * blockIdx.y * p.cluster >= all_steps) {
    if (rank == 0 && threadIdx.x < rows)
      p.parts.lse[blockIdx.y * p.parts.rows + row_of(threadIdx.x)] = -INFINITY;
    if (rejected && p.errors) atomicAdd(p.errors, 1);
    return;
  }
  const int first = (int)min(begin, (int64_t)all_steps) + warp;
  const int last = (int)min(begin + share, (int64_t)all_steps);
  const int steps = first < last ? (last - first + kWarps - 1) / kWarps : 0;
  const int* table = p.table + (int64_t)req * p.table_width;
  const int64_t head_block = (int64_t)p.page_size * kv4::row_bytes(D);
  const uint8_t* cache = p.cache + kv_head * head_block;
  const int64_t v_from_k = p.num_kv * head_block;
  const uint32_t ring = tma::smem_addr(smem) + warp * S::kWarp;

  // The pages of 32 steps at a time, one a lane, looked up a window ahead: where the
  // step's codes and scales lie in the cache (-1: outside it).
  int64_t codes_at = 0, next_codes;
  int64_t meta_at = 0, next_meta;
  auto look_up = [&](int i, int64_t* codes, int64_t* meta) {
    *codes = -1, *meta = 0;
    if (i >= steps) return;
    const uint32_t key = (uint32_t)(first + i * kWarps) * kStep;
    const uint32_t at = p.page_shift >= 0 ? key >> p.page_shift : key / (uint32_t)p.page_size;
    const int off = (int)(key - at * (uint32_t)p.page_size);
    const int id = __ldg(table + at);
    if (id >= 0 && id < p.num_pages) {
      const int64_t page = (int64_t)id * 2 * v_from_k;
      *codes = page + off * (D / 2);
      *meta = page + (int64_t)p.page_size * (D / 2) + off * (GROUPS * 4);
    } else {
      rejected = true;
    }
  };
  look_up(lane, &next_codes, &next_meta);
  uint32_t outside = 0;  // of the steps in the ring: bit i % kStages, the page is not there

  // where the lane's fragments of a step go
  uint32_t place[S::kCodes / 512];
#pragma unroll
  for (int k = 0; k < S::kCodes / 512; ++k) {
    const int f = lane + 32 * k;
    place[k] = piece_at<GROUPS>((f >> 1) / GROUPS, (f >> 1) % GROUPS) + ((f & 1) << 4);
  }
  const int meta_from = 16 * (lane & 15);
  const bool meta_v = lane >= 16, meta_mine = (lane & 15) < S::kMeta / 16;
  auto issue = [&](int i) {
    if ((i & 31) == 0) {
      codes_at = next_codes, meta_at = next_meta;
      look_up(i + 32 + lane, &next_codes, &next_meta);
    }
    const int64_t codes = __shfl_sync(kFullMask, codes_at, i & 31);
    const int64_t meta = __shfl_sync(kFullMask, meta_at, i & 31);
    outside = (outside & ~(1u << i % kStages)) | (codes < 0 ? 1u << i % kStages : 0u);
    if (codes >= 0) {
      const uint8_t* k = cache + codes + 16 * lane;
      const uint8_t* v = k + v_from_k;
      const uint32_t to = ring + i % kStages * S::kStage;
#pragma unroll
      for (int f = 0; f < S::kCodes / 512; ++f) {
        copy16(to + place[f], k + 512 * f);
        copy16(to + S::kCodes + place[f], v + 512 * f);
      }
      if (meta_mine)
        copy16(to + 2 * S::kCodes + (meta_v ? S::kMeta : 0) + meta_from,
               cache + meta + (meta_v ? v_from_k : 0) + meta_from);
    }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);

  // ---- Q fragments --------------------------------------------------------------------
  // row 8 n + g; step s of group j: dims 64 j + 16 t + 2 s + {0, 1} and those 8 further
  uint32_t qf[NT][D / 16][2];
  // sum(q_j) scale / 4 of row 8 n + g in three bf16 values, at the columns of z below (of
  // one group: values 0 to 2 at columns 0 to 2; of more: value t at 2 t + {0, 1} + {0, 8})
  uint32_t qz[NT][GROUPS == 4 ? 2 : 1];
  int sees[NT][2];            // .. and the keys they see
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = 8 * n + g;
    const int u = (row0 + r) / p.group;
    const __nv_bfloat16* src =
        p.q + (t0 + u) * p.q_stride + (int64_t)(kv_head * p.group + row0 + r - u * p.group) * D;
    qz[n][0] = qz[n][GROUPS / 4] = 0;
#pragma unroll
    for (int j = 0; j < GROUPS; ++j) {
      uint4 a = make_uint4(0, 0, 0, 0), b = a;
      if (r < rows) {
        a = __ldg(reinterpret_cast<const uint4*>(src + 64 * j + 16 * t));
        b = __ldg(reinterpret_cast<const uint4*>(src + 64 * j + 16 * t + 8));
      }
      const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
      float sum = 0.f;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        // (even steps take whole codes)
        qf[n][4 * j + s][0] = s & 1 ? x[s] : fma2(x[s], 0x3e803e80u, 0x80008000u);
        qf[n][4 * j + s][1] = s & 1 ? y[s] : fma2(y[s], 0x3e803e80u, 0x80008000u);
        sum += (low(x[s]) + high(x[s])) + (low(y[s]) + high(y[s]));
      }
      sum += __shfl_xor_sync(kFullMask, sum, 1);
      sum += __shfl_xor_sync(kFullMask, sum, 2);
      sum *= 0.25f * p.scale_log2;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const __nv_bfloat16 x = __float2bfloat16_rn(sum);
        sum -= __bfloat162float(x);
        const uint32_t bits = __bfloat16_as_ushort(x);
        if (GROUPS == 1) {
          if (t == k / 2) qz[n][0] |= bits << (16 * (k % 2));
        } else {
          if (t == k) qz[n][j / 2] |= bits << (16 * (j % 2));
        }
      }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) sees[n][c] = __shfl_sync(kFullMask, len, 8 * n + 2 * t + c);
  }

  uint32_t big;
  asm volatile("mov.b32 %0, 0x43004300;" : "=r"(big));
  // tile 4 j + e of O^T: its row g is dim 64 j + 8 g + 2 e, row g + 8 the next; columns 2 t
  // and 2 t + 1 are those rows of Q
  float o[NT][D / 16][4];
  float zeros[NT][GROUPS][2];  // sum of P z over this lane's keys
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[n][i][k] = 0.f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      m[n][c] = kNone, l[n][c] = 0.f;
#pragma unroll
      for (int j = 0; j < GROUPS; ++j) zeros[n][j][c] = 0.f;
    }
  }

  const float q_scale = p.scale_log2;
  // P steps of 16 keys together; all: every row sees every one of them.
  auto step = [&](int i, auto all_seen, auto together) {
    constexpr bool ALL = decltype(all_seen)::value;
    constexpr int P = decltype(together)::value;
    auto stage = [&](int p) { return smem + warp * S::kWarp + (i + p) % kStages * S::kStage; };
    auto seen = [&](int p, int h, int n, int c) {
      return ALL || (first + (i + p) * kWarps) * kStep + key_of(h, g) < sees[n][c];
    };

    // ---- S^T: keys g and g + 8 (of key_of), rows 2 t and 2 t + 1 ---------------------------
    // in quarters, of units of log2; first the zeros' part
    float s[P][NT][4];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint8_t* kc = stage(p);
      const uint32_t* km = reinterpret_cast<const uint32_t*>(kc + 2 * S::kCodes);
      uint32_t meta[2][GROUPS];
#pragma unroll
      for (int h = 0; h < 2; ++h) words(meta[h], km + key_of(h, g) * GROUPS);
      const uint32_t z[4] = {highs(meta[0][0], meta[0][GROUPS > 1]),
                             highs(meta[1][0], meta[1][GROUPS > 1]),
                             GROUPS == 4 ? highs(meta[0][GROUPS / 2], meta[0][GROUPS - 1]) : 0,
                             GROUPS == 4 ? highs(meta[1][GROUPS / 2], meta[1][GROUPS - 1]) : 0};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int k = 0; k < 4; ++k) s[p][n][k] = 0.f;
        mma(s[p][n], z, qz[n][0], GROUPS == 4 ? qz[n][GROUPS / 4] : 0);
      }
#pragma unroll
      for (int j = 0; j < GROUPS; ++j) {
        uint2 w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[h] = *reinterpret_cast<const uint2*>(kc + piece_at<GROUPS>(key_of(h, g), j) + 8 * t);
        float raw[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) raw[n][k] = 0.f;
        auto part = [&](int i, auto pair) {
          const uint32_t a[4] = {pair(w[0].x), pair(w[1].x), pair(w[0].y), pair(w[1].y)};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma(raw[n], a, qf[n][4 * j + i][0], qf[n][4 * j + i][1]);
        };
        part(0, [&](uint32_t x) { return low_codes(x, big); });
        part(1, [&](uint32_t x) { return high_codes(x); });
        part(2, [&](uint32_t x) { return low_codes(x >> 8, big); });
        part(3, [&](uint32_t x) { return high_codes(x >> 8); });
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float sk = low(meta[h][j]) * q_scale;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              s[p][n][2 * h + c] = fmaf(sk, raw[n][2 * h + c], s[p][n][2 * h + c]);
        }
      }
    }

    // ---- softmax, in units of log2 ----------------------------------------------------------
    float y[P][NT][4], above = -INFINITY;  // less the references
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float& x = s[p][n][2 * h + c];
            if (!seen(p, h, n, c)) x = -INFINITY;
            y[p][n][2 * h + c] = fmaf(4.f, x, -m[n][c]);
          }
          // (from kNone on every score exceeds it; -inf does not)
          above = fmaxf(above, fmaxf(y[p][n][c], y[p][n][2 + c]));
        }
    if (__any_sync(kFullMask, above > kRescaleAt)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float top = m[n][c];
#pragma unroll
          for (int p = 0; p < P; ++p) top = fmaxf(top, 4.f * fmaxf(s[p][n][c], s[p][n][2 + c]));
          top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 4));
          top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 8));
          top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 16));
          const float f = top == m[n][c] ? 1.f : ex2(m[n][c] - top);
          m[n][c] = top;
          l[n][c] *= f;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) o[n][k][c] *= f, o[n][k][2 + c] *= f;
#pragma unroll
          for (int j = 0; j < GROUPS; ++j) zeros[n][j][c] *= f;
#pragma unroll
          for (int p = 0; p < P; ++p)
#pragma unroll
            for (int h = 0; h < 2; ++h) y[p][n][2 * h + c] = fmaf(4.f, s[p][n][2 * h + c], -top);
        }
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            s[p][n][2 * h + c] = ex2(y[p][n][2 * h + c]);
            if (!seen(p, h, n, c)) s[p][n][2 * h + c] = 0.f;
          }
          l[n][c] += s[p][n][c] + s[p][n][2 + c];
        }

    // ---- O^T --------------------------------------------------------------------------------
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint8_t* vc = stage(p) + S::kCodes;
      const uint32_t* vm =
          reinterpret_cast<const uint32_t*>(vc + S::kCodes) + kStep * GROUPS;
      uint32_t meta[2][GROUPS];
#pragma unroll
      for (int h = 0; h < 2; ++h) words(meta[h], vm + key_of(h, g) * GROUPS);
#pragma unroll
      for (int j = 0; j < GROUPS; ++j) {
        uint32_t b[NT][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float sv = low(meta[h][j]), zv = high(meta[h][j]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float e[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              // (a key that a row does not see may hold anything)
              e[c] = seen(p, h, n, c) ? s[p][n][2 * h + c] * sv : 0.f;
              if (seen(p, h, n, c))
                zeros[n][j][c] = fmaf(s[p][n][2 * h + c], zv, zeros[n][j][c]);
            }
            b[n][h] = transposed(pack_bf16x2(e[0], e[1]));
          }
        }
        uint2 word[2];  // of keys 2 t and the next, of both halves
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          auto of = [&](int c) {
            return *reinterpret_cast<const uint32_t*>(
                vc + piece_at<GROUPS>(key_of(h, 2 * t + c), j) + 4 * g);
          };
          word[h] = make_uint2(of(0), of(1));
        }
        // bytes of the two keys, a code each of dims 2 i (bytes 0, 1) or 2 i + 1 (2, 3)
        auto both = [&](int h, uint32_t which) { return __byte_perm(word[h].x, word[h].y, which); };
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t even0 = both(0, 0x0400 + 0x0101 * i), even1 = both(1, 0x0400 + 0x0101 * i);
          const uint32_t odd0 = both(0, 0x0602 + 0x0101 * i), odd1 = both(1, 0x0602 + 0x0101 * i);
          const uint32_t lo[4] = {low_codes(even0, big), low_codes(odd0, big),
                                  low_codes(even1, big), low_codes(odd1, big)};
          const uint32_t hi[4] = {high_codes(even0), high_codes(odd0), high_codes(even1),
                                  high_codes(odd1)};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma(o[n][4 * j + 2 * i], lo, b[n][0], b[n][1]);
            mma(o[n][4 * j + 2 * i + 1], hi, b[n][0], b[n][1]);
          }
        }
      }
    }
  };
  auto out_of_cache = [&](int i) { return (outside & 1u << i % kStages) != 0; };
  constexpr std::integral_constant<int, 1> kOne{};
  auto turn = [&](int i, auto all_seen) {
    issue(i + kStages - 1);
    copy_wait<kStages - 1>();
    __syncwarp();
    if (!out_of_cache(i)) step(i, all_seen, kOne);  // (else nothing was copied)
    __syncwarp();  // the stage is read before its next copies start
  };
  auto turn2 = [&](int i) {  // two steps together
    issue(i + kStages - 1);
    copy_wait<kStages - 2>();
    __syncwarp();
    if (!out_of_cache(i) && !out_of_cache(i + 1)) {
      step(i, std::true_type(), std::integral_constant<int, 2>());
    } else {
#pragma unroll 1
      for (int k = i; k < i + 2; ++k)
        if (!out_of_cache(k)) step(k, std::false_type(), kOne);
    }
    __syncwarp();
    issue(i + kStages);
  };
  // the steps of keys that every row sees, then the others
  const int seen_by_all = max(0, min(steps, (least / kStep - first + kWarps - 1) / kWarps));
  int i = 0;
#pragma unroll 1
  for (; i + S::kUnroll <= seen_by_all; i += S::kUnroll) {
    if (S::kPair) {
#pragma unroll
      for (int k = 0; k < S::kUnroll; k += 2) turn2(i + k);
    } else {
#pragma unroll
      for (int k = 0; k < S::kUnroll; ++k) turn(i + k, std::true_type());
    }
  }
#pragma unroll 1
  for (; i < steps; ++i) turn(i, std::false_type());
  copy_wait<0>();
  if (rejected && p.errors) atomicAdd(p.errors, 1);
  auto all_keys = [](float x) {  // the sum over the lanes that hold the same rows
    x += __shfl_xor_sync(kFullMask, x, 4);
    x += __shfl_xor_sync(kFullMask, x, 8);
    return x + __shfl_xor_sync(kFullMask, x, 16);
  };
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      l[n][c] = all_keys(l[n][c]);
      if (g == 0) state[warp * kRows + 8 * n + 2 * t + c] = make_float2(m[n][c], l[n][c]);
#pragma unroll
      for (int j = 0; j < GROUPS; ++j) zeros[n][j][c] = all_keys(zeros[n][j][c]);
    }
  __syncthreads();

  // ---- join the warps ------------------------------------------------------------------
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = 8 * n + 2 * t + c;
      float ref = kNone, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) ref = fmaxf(ref, state[w * kRows + r].x);
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        sum += state[w * kRows + r].y * exp2f(state[w * kRows + r].x - ref);
      const float f = sum == 0.f ? 0.f : exp2f(m[n][c] - ref) / sum;  // 0: the row has no key
      float* dst = reinterpret_cast<float*>(smem + warp * S::kWarp) + r * S::kPad + 8 * g;
#pragma unroll
      for (int j = 0; j < GROUPS; ++j) {
        const float z = zeros[n][j][c];
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const float *x = o[n][4 * j + e], *y = o[n][4 * j + e + 1];
          *reinterpret_cast<float4*>(dst + 64 * j + 2 * e) =
              make_float4((x[c] + z) * f, (x[2 + c] + z) * f, fmaf(4.f, y[c], z) * f,
                          fmaf(4.f, y[2 + c], z) * f);
        }
      }
      if (warp == 0 && g == 0) part_lse[r] = sum == 0.f ? -INFINITY : ref + log2f(sum);
    }
  __syncthreads();
  // the CTA's part: the sum of its warps', which are scaled to one reference
  const bool joined = p.cluster > 1;
  float* own_o = reinterpret_cast<float*>(smem);
  auto warps_sum = [&](int at) {
    float4 v = *reinterpret_cast<const float4*>(own_o + at);
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 u = *reinterpret_cast<const float4*>(smem + w * S::kWarp + 4 * at);
      v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
    return v;
  };
  const int all = rows * (D / 4);  // 16-byte pieces of the rows
  if (joined) {
    for (int i = threadIdx.x; i < all; i += kWarps * 32) {
      const int at = i / (D / 4) * S::kPad + 4 * (i % (D / 4));
      *reinterpret_cast<float4*>(own_o + at) = warps_sum(at);
    }
    cluster.sync();
  }
  // each CTA of the cluster writes a slice of the rows
  const int slice = joined ? (all + p.cluster - 1) / p.cluster : all;
  const int stop = min((rank + 1) * slice, all);
  for (int i = rank * slice + threadIdx.x; i < stop; i += kWarps * 32) {
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

// ---- launch ------------------------------------------------------------------------------

struct Spread4 {
  int rows;  // of a tile: 8, 16, 24 or 32
  int tiles;
  int64_t units;
  int cluster, splits;
  int part_steps;
};

// CTAs are added while all of them are resident at once and each keeps at least two
// steps for every warp: first within a cluster, joined in place; beyond that as partials
// that a second launch joins.  Where no more fit, a long range is cut in parts of 2048
// keys instead (of 4096 where that is six waves of CTAs all the same): lengths differ,
// and the last tiles of a wave would keep a few SMs busy alone.  The range is the table's,
// since lengths are known on the device alone.  So that a table much wider than the requests are
// long costs little, parts are 16 waves of CTAs at most (up to 80 MB of partials), and of more
// keys in those requests that they would not reach the end of (64 and 256 sequences of 2048
// keys, 64 query heads, a table for 131072: 52 and 138 us, without a limit and with empty parts
// that write zeros 120 and 455; with a table for 2048 41 and 128).  What a cluster holds at
// once is not cut if its CTAs have about as little as that (16 x 8 heads of 16 rows, 8192
// keys: 56 us in clusters of 2, 67 in parts), unless they leave many places empty (20 x 8
// heads of 8 rows: 52 us in clusters of 2, 48 in parts).
Spread4 spread4(int64_t num_tokens, int per_request, int num_heads_q, int num_heads_kv,
                int head_dim, int page_size, int table_width) {
  Spread4 s;
  const int64_t rows = (int64_t)num_heads_q / num_heads_kv * per_request;
  const int limit = head_dim == 256 ? 16 : 32;
  s.tiles = (int)((rows + limit - 1) / limit);
  s.rows = (int)((rows + s.tiles * 8 - 1) / (s.tiles * 8)) * 8;
  s.units = num_tokens / per_request * num_heads_kv * s.tiles;
  const int64_t keys = (int64_t)table_width * page_size;
  const int64_t resident = 152 * ctas_of(head_dim, s.rows / 8);
  s.cluster = 1, s.part_steps = 0;
  while (s.cluster < kMaxCluster && s.units * s.cluster * 2 <= resident &&
         keys >= (int64_t)s.cluster * 2 * 2 * kStep * kWarps)
    s.cluster *= 2;
  const bool full = s.units * s.cluster * 4 >= resident * 3;
  int64_t splits = 1;
  if (s.units * s.cluster * 2 <= resident) {
    while (s.units * s.cluster * (splits + 1) <= resident && keys > s.cluster * splits * 1024)
      ++splits;
  } else if (keys >= 4096 && (keys + 2047) / 2048 > s.cluster * (full && s.cluster > 1 ? 2 : 1)) {
    s.cluster = 1;
    const int part = s.units * (keys / 4096) >= 6 * resident ? 4096 : 2048;
    s.part_steps = part / kStep;
    splits = (keys + part - 1) / part;
    const int64_t most = kWaves * resident / s.units;
    if (splits > most) splits = most > 1 ? most : 1;
  }
  s.splits = (int)splits;
  return s;
}

template <int D, int NT>
cudaError_t launch4(Attn4Params p, int64_t units, cudaStream_t stream) {
  using S = Shape4<D, NT>;
  static std::atomic<int> cache[kMaxDevices];
  int per_sm = 0;
  const cudaError_t e =
      tma::prepare(attn4_kernel<D, NT>, kWarps * 32, S::kSmem, cache, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t ctas = units * p.cluster, wave = (int64_t)per_sm * device_sm_count();
  p.trigger_from = ctas > wave ? (int)(ctas - wave) : 0;
  return launch_clusters(attn4_kernel<D, NT>, dim3((unsigned)ctas, (unsigned)p.splits),
                         dim3(kWarps * 32), S::kSmem, p.cluster, stream, p);
}

}  // namespace

int64_t kv4_attn_units(int64_t num_tokens, int per_request, int num_heads_q, int num_heads_kv) {
  // (the smallest tiles there are)
  const int64_t rows = (int64_t)num_heads_q / num_heads_kv * per_request;
  return num_tokens / per_request * num_heads_kv * ((rows + 7) / 8);
}

int64_t kv4_attn_workspace(int64_t num_tokens, int per_request, int num_heads_q,
                           int num_heads_kv, int head_dim, int page_size, int table_width) {
  const int s = spread4(num_tokens, per_request, num_heads_q, num_heads_kv, head_dim, page_size,
                        table_width).splits;
  return s == 1 ? 0 : partials_bytes(s, num_tokens * num_heads_q, head_dim);
}

cudaError_t launch_kv4_attn(const Kv4AttnArgs& a, cudaStream_t stream) {
  const PagedQuery& x = a.x;
  const Spread4 s = spread4(x.num_tokens, a.per_request, x.num_heads_q, x.num_heads_kv,
                            x.head_dim, x.page_size, x.table_width);
  Attn4Params p = {};
  p.q = static_cast<const __nv_bfloat16*>(x.q);
  p.q_stride = x.q_stride;
  p.cache = static_cast<const uint8_t*>(a.kv_cache);
  p.num_q = x.num_heads_q;
  p.num_kv = x.num_heads_kv;
  p.group = x.num_heads_q / x.num_heads_kv;
  p.per_request = a.per_request;
  p.tiles = s.tiles;
  p.num_pages = x.num_pages;
  p.page_size = x.page_size;
  p.page_shift = -1;
  for (int k = 0; k < 31; ++k)
    if (x.page_size == 1 << k) p.page_shift = k;
  p.table = x.page_table;
  p.table_width = x.table_width;
  p.lens = x.lens;
  p.scale_log2 = a.scale * kLog2e;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.errors = x.errors;
  p.cluster = s.cluster;
  p.splits = s.splits;
  p.part_steps = s.part_steps;
  if (s.splits > 1)
    p.parts = partials_at(a.workspace, s.splits, (int64_t)x.num_tokens * x.num_heads_q, x.head_dim);
  cudaError_t e = cudaErrorInvalidValue;
  switch (x.head_dim + s.rows) {
    case 64 + 8: e = launch4<64, 1>(p, s.units, stream); break;
    case 64 + 16: e = launch4<64, 2>(p, s.units, stream); break;
    case 64 + 24: e = launch4<64, 3>(p, s.units, stream); break;
    case 64 + 32: e = launch4<64, 4>(p, s.units, stream); break;
    case 128 + 8: e = launch4<128, 1>(p, s.units, stream); break;
    case 128 + 16: e = launch4<128, 2>(p, s.units, stream); break;
    case 128 + 24: e = launch4<128, 3>(p, s.units, stream); break;
    case 128 + 32: e = launch4<128, 4>(p, s.units, stream); break;
    case 256 + 8: e = launch4<256, 1>(p, s.units, stream); break;
    case 256 + 16: e = launch4<256, 2>(p, s.units, stream); break;
  }
  if (e != cudaSuccess || s.splits == 1) return e;
  return launch_attn_join(p.parts, s.splits, x.head_dim, a.out, stream);
}

}  // namespace kvq
