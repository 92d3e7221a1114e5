// kvq_kv4_attn.cu -- attention over the paged cache held in 4 bits, for the few
// query rows of a decode step.
//
// One cluster of 1..8 CTAs takes up to 16 query rows of one request and kv head
// (tokens x heads of the group) and the request's keys, its CTAs a part each.  A
// warp works alone on every kWarps-th group of 16 keys, with an online softmax of
// its own.  With q_j the row's dims of group j of 64, and n = c - 8 the codes:
//   S   = scale sum_j ( s_kj (q_j n_kj) + z_kj sum(q_j) )
//   O_j = sum_k (P_k s_kj) n_kj + sum_k P_k z_kj
// so no code is ever multiplied by its scale: codes become bf16 integers by a
// shift, a mask and a subtraction, two at a time, and go straight into 16x8x16
// matrix instructions; K's scales and zeros are applied to S in fp32, V's scales
// to the weights P, whose product is rounded once to bf16 (the row sum adds the
// unrounded P), V's zeros to P in fp32.  K's codes keep the 16 that the mask leaves
// in them, which S takes back with the zero: (z - 24 s) sum(q).  (V's must not:
// the sum over a long range would lose in the offset what it is to keep.)
//
// A group's codes come in by 16-byte asynchronous copies, three groups ahead, into
// a ring that only this warp uses, so that there is no CTA barrier in the loop.
// 32-byte pieces (a group of dims of one key) are exchanged so that the four
// keys that a load touches lie in different banks.  The matrix instructions may take
// the keys in any order: key_of() lists the one that does for the loads of K and of V.
#include <cooperative_groups.h>

#include "kvq_kv4.cuh"
#include "kvq_mma.cuh"
#include "kvq_paged_attn.cuh"
#include "kvq_tma.cuh"

namespace cg = cooperative_groups;

namespace kvq {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxCluster = 8;
constexpr int kRows = 16;   // query rows of a CTA
constexpr int kStep = 16;   // keys of one step of a warp
constexpr int kStages = 4;

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
  __nv_bfloat16* out;
  Partials parts;            // with several splits
  int* errors;
  int trigger_from;
};

template <int D>
struct Shape4 {
  static constexpr int kCtas = D == 256 ? 2 : 3;         // of an SM, by their registers
  static constexpr int kGroups = D / kv4::kGroup;
  static constexpr int kCodes = kStep * D / 2;           // bytes of 16 keys' codes
  static constexpr int kMeta = kStep * kGroups * 4;      // .. scales and zeros
  static constexpr int kStage = 2 * (kCodes + kMeta);    // K codes, V codes, K meta, V meta
  static constexpr int kRing = kStages * kStage;
  static constexpr int kPad = D + 8;                     // fp32 values of an output row
  static constexpr int kState = kWarps * kRows * 8;      // {m, l} per warp and row
  static constexpr int kLse = kRows * 4;
  static constexpr int kSmem = kWarps * kRing + kState + kLse;
  static_assert(kRing >= kRows * kPad * 4, "a warp's output fits in its ring");
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
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
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

__device__ __forceinline__ uint32_t less24(uint32_t pair) {  // 16 + c -> c - 8, twice, exact
  const __nv_bfloat162 v = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&pair),
                                   __floats2bfloat162_rn(24.f, 24.f));
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <int D>
__global__ void __launch_bounds__(kWarps * 32, Shape4<D>::kCtas)
attn4_kernel(const Attn4Params p) {
  using S = Shape4<D>;
  constexpr int GROUPS = S::kGroups;
  extern __shared__ __align__(128) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  grid_dependency_sync(p.trigger_from);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;  // the lane's place in a matrix fragment
  float2* state = reinterpret_cast<float2*>(smem + kWarps * S::kRing);
  float* part_lse = reinterpret_cast<float*>(smem + kWarps * S::kRing + S::kState);
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
  int sees[2];  // keys that rows g and g + 8 see
  sees[0] = __shfl_sync(kFullMask, len, g);
  sees[1] = __shfl_sync(kFullMask, len, g + 8);

  // ---- Q fragments --------------------------------------------------------------------
  // step s of group j: dims 64 j + 16 t + 2 s + {0, 1} and those 8 further, rows g, g + 8
  uint32_t qf[D / 16][4];
  float qsum[2][GROUPS];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = g + 8 * i;
    const int u = (row0 + r) / p.group;
    const __nv_bfloat16* src =
        p.q + (t0 + u) * p.q_stride + (int64_t)(kv_head * p.group + row0 + r - u * p.group) * D;
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
        qf[4 * j + s][i] = x[s];
        qf[4 * j + s][2 + i] = y[s];
        sum += (low(x[s]) + high(x[s])) + (low(y[s]) + high(y[s]));
      }
      sum += __shfl_xor_sync(kFullMask, sum, 1);
      sum += __shfl_xor_sync(kFullMask, sum, 2);
      qsum[i][j] = sum;
    }
  }

  // ---- which keys: of the request's groups of 16 an equal share ------------------------
  const int parts = p.cluster * p.splits;
  const int all_steps = most / kStep + (most % kStep != 0);
  const int share = (int)(((int64_t)all_steps + parts - 1) / parts);
  const int64_t begin = (int64_t)share * (blockIdx.y * p.cluster + rank);
  const int first = (int)min(begin, (int64_t)all_steps) + warp;
  const int last = (int)min(begin + share, (int64_t)all_steps);
  const int steps = first < last ? (last - first + kWarps - 1) / kWarps : 0;
  const int* table = p.table + (int64_t)req * p.table_width;
  const int64_t head_block = (int64_t)p.page_size * kv4::row_bytes(D);
  const uint32_t ring = tma::smem_addr(smem) + warp * S::kRing;

  // The pages of 32 steps at a time, one a lane, looked up a window ahead: page (-1:
  // outside the cache) and the step's first key in it.
  int page = 0, off = 0, next_page, next_off;
  auto look_up = [&](int i, int* page, int* off) {
    *page = -1, *off = 0;
    if (i >= steps) return;
    const uint32_t key = (uint32_t)(first + i * kWarps) * kStep;
    const uint32_t at = p.page_shift >= 0 ? key >> p.page_shift : key / (uint32_t)p.page_size;
    *off = (int)(key - at * (uint32_t)p.page_size);
    const int id = __ldg(table + at);
    if (id >= 0 && id < p.num_pages) *page = id;
    else rejected = true;
  };
  look_up(lane, &next_page, &next_off);
  uint32_t outside = 0;  // of the last 32 steps issued: bit i % 32, the page is not there

  auto issue = [&](int i) {
    if ((i & 31) == 0) {
      page = next_page, off = next_off;
      look_up(i + 32 + lane, &next_page, &next_off);
    }
    const int id = __shfl_sync(kFullMask, page, i & 31);
    const int key = __shfl_sync(kFullMask, off, i & 31);
    outside = (outside & ~(1u << (i & 31))) | ((id < 0 ? 1u : 0u) << (i & 31));
    if (i < steps && id >= 0) {
      const uint8_t* k = p.cache + ((int64_t)id * 2 * p.num_kv + kv_head) * head_block;
      const uint8_t* v = k + p.num_kv * head_block;
      const int64_t codes = (int64_t)key * (D / 2);
      const int64_t meta = (int64_t)p.page_size * (D / 2) + key * (GROUPS * 4);
      const uint32_t to = ring + i % kStages * S::kStage;
#pragma unroll
      for (int f = lane; f < S::kCodes / 16; f += 32) {
        const uint32_t at = piece_at<GROUPS>((f >> 1) / GROUPS, (f >> 1) % GROUPS) + ((f & 1) << 4);
        copy16(to + at, k + codes + 16 * f);
        copy16(to + S::kCodes + at, v + codes + 16 * f);
      }
      const int f = lane & 15;
      if (f < S::kMeta / 16)
        copy16(to + 2 * S::kCodes + (lane >> 4) * S::kMeta + 16 * f,
               (lane >> 4 ? v : k) + meta + 16 * f);
    }
    copy_commit();
  };

  float o[D / 8][4];  // tile 8 j + e: dims 64 j + 8 n + e of its columns n
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int k = 0; k < 4; ++k) o[n][k] = 0.f;
  float zeros[2][GROUPS] = {};  // sum of P z over this lane's keys
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);
  for (int i = 0; i < steps; ++i) {
    issue(i + kStages - 1);
    copy_wait<kStages - 1>();
    __syncwarp();
    if (outside >> (i & 31) & 1) continue;  // (nothing was copied)
    const uint32_t kc = ring + i % kStages * S::kStage, vc = kc + S::kCodes;
    const uint32_t km = vc + S::kCodes, vm = km + S::kMeta;
    const int key0 = (first + i * kWarps) * kStep;
    const bool whole = key0 <= least - kStep;  // every row sees every key

    // ---- S ------------------------------------------------------------------------------
    float s[2][4] = {};
#pragma unroll
    for (int j = 0; j < GROUPS; ++j) {
      float raw[2][4] = {};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint2 w = lds64(kc + piece_at<GROUPS>(key_of(h, g), j) + 8 * t);
        mma16816(raw[h], qf[4 * j], kv4::pair16<0>(w.x), kv4::pair16<0>(w.y));
        mma16816(raw[h], qf[4 * j + 1], kv4::pair16<1>(w.x), kv4::pair16<1>(w.y));
        mma16816(raw[h], qf[4 * j + 2], kv4::pair16<2>(w.x), kv4::pair16<2>(w.y));
        mma16816(raw[h], qf[4 * j + 3], kv4::pair16<3>(w.x), kv4::pair16<3>(w.y));
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t w = lds32(km + (key_of(h, 2 * t + c) * GROUPS + j) * 4);
          const float sk = low(w), zk = fmaf(-24.f, sk, high(w));
#pragma unroll
          for (int r = 0; r < 2; ++r)
            s[h][2 * r + c] += fmaf(sk, raw[h][2 * r + c], zk * qsum[r][j]);
        }
    }

    // ---- softmax: rows g (r = 0) and g + 8 ------------------------------------------------
    bool seen[2][4];
    float top[2] = {m[0], m[1]};
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        seen[h][k] = whole || key0 + key_of(h, 2 * t + (k & 1)) < sees[k >> 1];
        s[h][k] = seen[h][k] ? s[h][k] * p.scale_log2 : -INFINITY;
        top[k >> 1] = fmaxf(top[k >> 1], s[h][k]);
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(kFullMask, top[r], 1));
      top[r] = fmaxf(top[r], __shfl_xor_sync(kFullMask, top[r], 2));
    }
    if (__any_sync(kFullMask, top[0] != m[0] || top[1] != m[1])) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        // (-inf) - (-inf): no key yet, nothing accumulated, any factor does
        const float f = top[r] == m[r] ? 1.f : exp2f(m[r] - top[r]);
        l[r] *= f;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) o[n][2 * r] *= f, o[n][2 * r + 1] *= f;
#pragma unroll
        for (int j = 0; j < GROUPS; ++j) zeros[r][j] *= f;
        m[r] = top[r];
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float ref = m[k >> 1] == -INFINITY ? 0.f : m[k >> 1];
        s[h][k] = exp2f(s[h][k] - ref);
        l[k >> 1] += s[h][k];
      }

    // ---- O --------------------------------------------------------------------------------
#pragma unroll
    for (int j = 0; j < GROUPS; ++j) {
      float e[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t w = lds32(vm + (key_of(h, 2 * t + c) * GROUPS + j) * 4);
          const float sv = low(w), zv = high(w);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int k = 2 * r + c;
            // (a key that a row does not see may hold anything)
            e[h][k] = seen[h][k] ? s[h][k] * sv : 0.f;
            zeros[r][j] = seen[h][k] ? fmaf(s[h][k], zv, zeros[r][j]) : zeros[r][j];
          }
        }
      const uint32_t pf[4] = {pack_bf16x2(e[0][0], e[0][1]), pack_bf16x2(e[0][2], e[0][3]),
                              pack_bf16x2(e[1][0], e[1][1]), pack_bf16x2(e[1][2], e[1][3])};
      uint32_t even[2], odd[2];  // codes of two keys each: dims 2 i, dims 2 i + 1 of the word
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t a = lds32(vc + piece_at<GROUPS>(key_of(h, 2 * t), j) + 4 * g);
        const uint32_t b = lds32(vc + piece_at<GROUPS>(key_of(h, 2 * t + 1), j) + 4 * g);
        even[h] = __byte_perm(a, b, 0x5410);
        odd[h] = __byte_perm(a, b, 0x7632);
      }
      float(*to)[4] = o + 8 * j;
      mma16816(to[0], pf, less24(kv4::pair16<0>(even[0])), less24(kv4::pair16<0>(even[1])));
      mma16816(to[1], pf, less24(kv4::pair16<0>(odd[0])), less24(kv4::pair16<0>(odd[1])));
      mma16816(to[2], pf, less24(kv4::pair16<1>(even[0])), less24(kv4::pair16<1>(even[1])));
      mma16816(to[3], pf, less24(kv4::pair16<1>(odd[0])), less24(kv4::pair16<1>(odd[1])));
      mma16816(to[4], pf, less24(kv4::pair16<2>(even[0])), less24(kv4::pair16<2>(even[1])));
      mma16816(to[5], pf, less24(kv4::pair16<2>(odd[0])), less24(kv4::pair16<2>(odd[1])));
      mma16816(to[6], pf, less24(kv4::pair16<3>(even[0])), less24(kv4::pair16<3>(even[1])));
      mma16816(to[7], pf, less24(kv4::pair16<3>(odd[0])), less24(kv4::pair16<3>(odd[1])));
    }
    __syncwarp();  // the stage is read before its next copies start
  }
  copy_wait<0>();
  if (rejected && p.errors) atomicAdd(p.errors, 1);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(kFullMask, l[r], 1);
    l[r] += __shfl_xor_sync(kFullMask, l[r], 2);
    if (t == 0) state[warp * kRows + g + 8 * r] = make_float2(m[r], l[r]);
#pragma unroll
    for (int j = 0; j < GROUPS; ++j) {
      zeros[r][j] += __shfl_xor_sync(kFullMask, zeros[r][j], 1);
      zeros[r][j] += __shfl_xor_sync(kFullMask, zeros[r][j], 2);
    }
  }
  __syncthreads();

  // ---- join the warps ------------------------------------------------------------------
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = g + 8 * h;
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, state[w * kRows + r].x);
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      sum += state[w * kRows + r].y * exp2f(state[w * kRows + r].x - ref);
    const float f = sum == 0.f ? 0.f : exp2f(m[h] - ref) / sum;  // 0: the row has no key
    float* dst = reinterpret_cast<float*>(smem + warp * S::kRing) + r * S::kPad + 16 * t;
#pragma unroll
    for (int j = 0; j < GROUPS; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c)  // dims 64 j + 16 t + 8 c + e
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float z = zeros[h][j];
          const int k = 2 * h + c;
          *reinterpret_cast<float4*>(dst + 64 * j + 8 * c + e) = make_float4(
              (o[8 * j + e][k] + z) * f, (o[8 * j + e + 1][k] + z) * f,
              (o[8 * j + e + 2][k] + z) * f, (o[8 * j + e + 3][k] + z) * f);
        }
    if (warp == 0 && t == 0) part_lse[r] = sum == 0.f ? -INFINITY : ref + log2f(sum);
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
  int cluster, splits;
};

// CTAs are added while all of them are resident at once and each keeps at least
// two steps for every warp: first within a cluster, joined in place; beyond that as
// partials that a second launch joins.
Spread4 spread4_for(int64_t units, int64_t keys, int head_dim) {
  const int per_sm = head_dim == 256 ? 2 : 3;
  Spread4 s = {1, 1};
  while (s.cluster < kMaxCluster && units * s.cluster * 2 <= 152 * per_sm &&
         keys >= (int64_t)s.cluster * 2 * 2 * kStep * kWarps)
    s.cluster *= 2;
  while (units * s.cluster * (s.splits + 1) <= 152 * per_sm && keys > s.cluster * s.splits * 2048)
    ++s.splits;
  return s;
}

int tiles4(int num_heads_q, int num_heads_kv, int per_request) {
  return (int)(((int64_t)num_heads_q / num_heads_kv * per_request + kRows - 1) / kRows);
}

Spread4 spread4(int64_t num_tokens, int per_request, int num_heads_q, int num_heads_kv,
                int head_dim, int page_size, int table_width) {
  const int64_t units = num_tokens / per_request * num_heads_kv *
                        tiles4(num_heads_q, num_heads_kv, per_request);
  return spread4_for(units, (int64_t)table_width * page_size, head_dim);
}

template <int D>
cudaError_t launch4(Attn4Params p, int64_t units, cudaStream_t stream) {
  static std::atomic<int> cache[kMaxDevices];
  int per_sm = 0;
  const cudaError_t e =
      tma::prepare(attn4_kernel<D>, kWarps * 32, Shape4<D>::kSmem, cache, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t ctas = units * p.cluster, wave = (int64_t)per_sm * device_sm_count();
  p.trigger_from = ctas > wave ? (int)(ctas - wave) : 0;
  return launch_clusters(attn4_kernel<D>, dim3((unsigned)ctas, (unsigned)p.splits),
                         dim3(kWarps * 32), Shape4<D>::kSmem, p.cluster, stream, p);
}

}  // namespace

int64_t kv4_attn_units(int64_t num_tokens, int per_request, int num_heads_q, int num_heads_kv) {
  return num_tokens / per_request * num_heads_kv * tiles4(num_heads_q, num_heads_kv, per_request);
}

int64_t kv4_attn_workspace(int64_t num_tokens, int per_request, int num_heads_q,
                           int num_heads_kv, int head_dim, int page_size, int table_width) {
  const int s = spread4(num_tokens, per_request, num_heads_q, num_heads_kv, head_dim, page_size,
                        table_width).splits;
  return s == 1 ? 0 : partials_bytes(s, num_tokens * num_heads_q, head_dim);
}

cudaError_t launch_kv4_attn(const Kv4AttnArgs& a, cudaStream_t stream) {
  const PagedQuery& x = a.x;
  Attn4Params p = {};
  p.q = static_cast<const __nv_bfloat16*>(x.q);
  p.q_stride = x.q_stride;
  p.cache = static_cast<const uint8_t*>(a.kv_cache);
  p.num_q = x.num_heads_q;
  p.num_kv = x.num_heads_kv;
  p.group = x.num_heads_q / x.num_heads_kv;
  p.per_request = a.per_request;
  p.tiles = tiles4(x.num_heads_q, x.num_heads_kv, a.per_request);
  p.num_pages = x.num_pages;
  p.page_size = x.page_size;
  p.page_shift = -1;
  for (int s = 0; s < 31; ++s)
    if (x.page_size == 1 << s) p.page_shift = s;
  p.table = x.page_table;
  p.table_width = x.table_width;
  p.lens = x.lens;
  p.scale_log2 = a.scale * kLog2e;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.errors = x.errors;
  const Spread4 s = spread4(x.num_tokens, a.per_request, x.num_heads_q, x.num_heads_kv,
                            x.head_dim, x.page_size, x.table_width);
  p.cluster = s.cluster;
  p.splits = s.splits;
  if (s.splits > 1)
    p.parts = partials_at(a.workspace, s.splits, (int64_t)x.num_tokens * x.num_heads_q, x.head_dim);
  const int64_t units = kv4_attn_units(x.num_tokens, a.per_request, x.num_heads_q, x.num_heads_kv);
  cudaError_t e = cudaErrorInvalidValue;
  switch (x.head_dim) {
    case 64: e = launch4<64>(p, units, stream); break;
    case 128: e = launch4<128>(p, units, stream); break;
    case 256: e = launch4<256>(p, units, stream); break;
  }
  if (e != cudaSuccess || s.splits == 1) return e;
  return launch_attn_join(p.parts, s.splits, x.head_dim, a.out, stream);
}

}  // namespace kvq
