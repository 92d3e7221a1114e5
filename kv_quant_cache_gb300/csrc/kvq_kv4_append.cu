// kvq_kv4_append.cu -- keys and values of new tokens into the paged cache held in
// 4 bits, with the rotary embedding applied on the way, and listed tokens read
// back as bf16.
//
// Append.  Lanes, rows and steps are those of the bf16 append: a row of D dims
// is D/16 lanes of two fragments of 8 dims, which hold both members of every
// rotated pair.  A fragment is one word of codes.  Per group of 64 dims
//   scale = bf16((hi - lo) / 15),   zero = bf16(lo + 8 scale),
//   code  = round((x - zero) / scale) + 8, held to 0 .. 15,
// of the bf16 values x.  A code is a decision, so that it shall not hang on
// the order of fp32 operations: the rotated keys are the exact a c - b s rounded
// to fp32 (products split into value and error, the sum's error added back) and
// then to bf16, and the quotient's rounding is decided on the exact remainder.
// Minimum and maximum of a group travel together in one register, (lo, -hi) as a
// bf16 pair.
// Every row is read once, q rows are written as they came, key and value rows in 9/32 of
// their bytes.  32768 tokens of 32 + 16 heads of 128: 143 us, 4.9 TB/s.  Neither memory (59 %)
// nor the issue slots (70 %, with rotation, extrema and rounding) are full: loads, arithmetic
// and stores of a warp follow one another, and registers allow 28 warps to an SM.
//
// Read back.  A lane takes words l and l + D/16 of a row, so that a row's
// stores are contiguous; all loads of a warp's rows are in flight together.  65536
// tokens of 8 heads of 128: 56 us, 6.2 TB/s.
#include "kvq_device.cuh"
#include "kvq_kv4.cuh"
#include "kvq_paged.h"

namespace kvq {
namespace {

constexpr int kWarps = 4;
constexpr int kCtas = 7;                            // of an SM, append
constexpr int64_t kLater = 152 * kCtas / 2 * kWarps;  // warps: half a wave of CTAs

struct Append4Params {
  __nv_bfloat16* qkv;
  __nv_bfloat16* q_out;
  const float* cos_sin;
  const int64_t* positions;
  const int64_t* slots;
  uint8_t* cache;
  int num_q, num_kv, num_rows, first_row;
  int rot;
  int chunks;  // warps per token; they take its groups of rows in turn
  int64_t items;
  int64_t max_pos, num_slots;
  int page_size;
  int64_t q_token_stride;  // elements between tokens of q_out
  int* errors;
  int trigger_from;
};

// a c - b s, rounded once to fp32 (but for results that lie within 2^-45 or so of
// the middle of two).
__device__ __forceinline__ float exact_rotation(float a, float c, float b, float s) {
  const float p = __fmul_rn(a, c), q = __fmul_rn(b, s);
  const float pe = __fmaf_rn(a, c, -p), qe = __fmaf_rn(b, s, -q);
  const float d = __fsub_rn(p, q);
  const float v = __fsub_rn(d, p);                                         // the part of -q in d
  const float e = __fsub_rn(__fsub_rn(p, __fsub_rn(d, v)), __fadd_rn(q, v));  // lost in d
  return __fadd_rn(d, __fadd_rn(e, __fsub_rn(pe, qe)));
}

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// (min, -max) of the eight values of a fragment.
__device__ __forceinline__ uint32_t span(const uint4& v) {
  constexpr uint32_t neg = 0x80008000u;
  const uint32_t lo = min2(min2(v.x, v.y), min2(v.z, v.w));
  const uint32_t hi = min2(min2(v.x ^ neg, v.y ^ neg), min2(v.z ^ neg, v.w ^ neg));
  const uint32_t lo2 = min2(lo, lo >> 16), hi2 = min2(hi, hi >> 16);
  return __byte_perm(lo2, hi2, 0x5410);
}

// Scale and zero of a group from its (lo, -hi), as the cache holds them.
__device__ __forceinline__ uint32_t group_meta(uint32_t lohi) {
  const float lo = __uint_as_float(lohi << 16), hi = -__uint_as_float(lohi & 0xffff0000u);
  const float width = __fsub_rn(hi, lo);
  if (!(width < INFINITY)) return 0x7fc07fc0u;  // NaN, an infinity: the group reads back as NaN
  // width / 15, correctly rounded: a product, and the exact remainder's share of it
  // (Markstein's correction)
  float q = __fmul_rn(width, 1.f / 15.f);
  q = __fmaf_rn(__fmaf_rn(-15.f, q, width), 1.f / 15.f, q);
  if (width < 0x1p-100f) q = __fdiv_rn(width, 15.f);  // (where the remainder may not be exact)
  const float scale = __bfloat162float(__float2bfloat16_rn(q));
  return pack_bf16x2(scale, __fadd_rn(lo, __fmul_rn(8.f, scale)));
}

// Whether the ends of a group may come out past the codes at the ends: only where the
// roundings of scale and zero make up half a step.
__device__ __forceinline__ bool past_ends(uint32_t lohi, uint32_t meta) {
  const float lo = __uint_as_float(lohi << 16), hi = -__uint_as_float(lohi & 0xffff0000u);
  const float scale = __uint_as_float(meta << 16), zero = __uint_as_float(meta & 0xffff0000u);
  return scale > 0.f && (hi - zero > 7.49f * scale || lo - zero < -8.49f * scale);
}

// The word of codes of a fragment's eight values; cut: codes may lie past the ends.
// Rounding to a whole number is adding 1.5 2^23; the remainder t - c scale is exact, and
// shows where the product of t and the reciprocal has rounded across the middle of two
// codes, or from it to the odd one (values of 8 bits lie in the middle often: 3 in
// 1000).  Four codes are put together as one number, c_0 + 16 c_1 + .., which is exact
// and keeps to the pipe that the rest of the work leaves free.
__device__ __forceinline__ uint32_t codes_of(const uint4& v, uint32_t meta, bool cut) {
  const float scale = __uint_as_float(meta << 16), zero = __uint_as_float(meta & 0xffff0000u);
  if (!(scale > 0.f)) return 0x88888888u;  // one value (or NaN): zero alone
  constexpr float kWhole = 12582912.f;
  float x[8], u[8];  // u: the codes, negative, between -7 and 8
  unpack_bf16x8(v, x);
  if (scale < 0x1p-100f) {  // its reciprocal may overflow
    for (int i = 0; i < 8; ++i) u[i] = -rintf(__fdiv_rn(__fsub_rn(x[i], zero), scale));
    cut = true;
  } else {
    float inv;  // (what it is off by, the remainder shows)
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
    const float half = 0.5f * scale;
    float r[8];
    bool middle = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = __fsub_rn(x[i], zero);
      u[i] = __fsub_rn(kWhole, __fmaf_rn(t, inv, kWhole));
      r[i] = __fmaf_rn(u[i], scale, t);
      middle |= fabsf(r[i]) >= half;
    }
    if (middle) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // above half a step by its bits, less the lowest of the whole number: at half, odd
        const uint32_t odd = __float_as_uint(__fadd_rn(u[i], kWhole)) & 1u;
        if ((__float_as_uint(r[i]) & 0x7fffffffu) > __float_as_uint(half) - odd)
          u[i] -= copysignf(1.f, r[i]);
      }
    }
  }
  if (cut) {
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = fminf(fmaxf(u[i], -7.f), 8.f);
  }
  constexpr float kBase = 8388608.f + 8.f * (1 + 16 + 256 + 4096);  // 2^23, and 8 to each code
  uint32_t half_word[2];  // dims of even place, of odd place
#pragma unroll
  for (int h = 0; h < 2; ++h)
    half_word[h] = __float_as_uint(fmaf(
        u[6 + h], -4096.f, fmaf(u[4 + h], -256.f, fmaf(u[2 + h], -16.f, kBase - u[h]))));
  return __byte_perm(half_word[0], half_word[1], 0x5410);
}

template <int D, bool NEOX, int STEPS>
// (seven CTAs an SM: 32768 tokens 151 us, as many as registers allowed without, 161)
__global__ void __launch_bounds__(kWarps * 32, kCtas) append4_kernel(const Append4Params p) {
  constexpr int LPR = D / 16;    // lanes per row
  constexpr int RPW = 32 / LPR;  // rows per warp step
  constexpr int GROUPS = D / kv4::kGroup;
  grid_dependency_sync(p.trigger_from);
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (item >= p.items) return;
  const int lane = threadIdx.x & 31;
  const int l = lane % LPR;
  const int64_t t = item / p.chunks;
  const int chunk = (int)(item - t * p.chunks);
  // In turn: key and value rows, which take most of the work, are a token's last (a
  // stretch of rows to each warp: the last one of a CTA at work alone, 235 us at 32768
  // tokens).
  auto first_of = [&](int s) { return p.first_row + (s * p.chunks + chunk) * RPW; };
  const int64_t slot = __ldg(p.slots + t);
  const int64_t pos = p.rot ? __ldg(p.positions + t) : 0;

  // the lane's two fragments: NeoX pair halves while rotated, else adjacent
  const bool rotated = 16 * l < p.rot;
  const bool halves = NEOX && rotated;
  const int oa = halves ? 8 * l : 16 * l;
  const int ob = halves ? 8 * l + (p.rot >> 1) : 16 * l + 8;

  const __nv_bfloat16* src = p.qkv + t * (int64_t)p.num_rows * D;
  uint4 xa[STEPS], xb[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int r = first_of(s) + lane / LPR;
    if (r < p.num_rows) {
      xa[s] = load_stream(src + (size_t)r * D + oa);
      xb[s] = load_stream(src + (size_t)r * D + ob);
    } else {
      xa[s] = xb[s] = make_uint4(0, 0, 0, 0);
    }
  }
  if (STEPS > 1 && item + kLater < p.items) {
    // rows of a warp that comes later, into the L2: without, a CTA's loads, all issued at
    // once, take their time from memory before anything can be done (32768 tokens 143
    // us, 150 without, 144 a whole wave ahead)
    constexpr int LINES = RPW * D * 2 / 128, PER_ROW = D * 2 / 128;
    const int64_t later = (item + kLater) / p.chunks;
    const int its = (int)(item + kLater - later * p.chunks);
    const int s = lane / LINES, line = lane % LINES;
    const int r = p.first_row + (s * p.chunks + its) * RPW + line / PER_ROW;
    if (s < STEPS && r < p.num_rows)
      prefetch_l2(p.qkv + (later * p.num_rows + r) * D + line % PER_ROW * 64);
  }
  if (p.rot && (pos < 0 || pos >= p.max_pos)) {  // warp-uniform: leave the token as it is
    if (p.errors && chunk == 0 && lane == 0) atomicAdd(p.errors, 1);
    return;
  }
  const bool bad_slot = slot < -1 || slot >= p.num_slots;
  if (bad_slot && p.errors && chunk == 0 && lane == 0) atomicAdd(p.errors, 1);
  const bool store_kv = slot >= 0 && !bad_slot;
  float cs[8], sn[8];
  if (rotated) {
    // frequencies of the pairs: NeoX 8l..8l+7 (8 pairs over both fragments);
    // GPT-J 8l..8l+3 in the first fragment and 8l+4..8l+7 in the second
    const float* row = p.cos_sin + pos * p.rot + 8 * l;
    const float4 c0 = __ldg(reinterpret_cast<const float4*>(row));
    const float4 c1 = __ldg(reinterpret_cast<const float4*>(row + 4));
    const float4 s0 = __ldg(reinterpret_cast<const float4*>(row + (p.rot >> 1)));
    const float4 s1 = __ldg(reinterpret_cast<const float4*>(row + (p.rot >> 1) + 4));
    cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w;
    cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
    sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w;
    sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
  }
  const int64_t page = store_kv ? slot / p.page_size : 0;
  const int off = store_kv ? (int)(slot - page * p.page_size) : 0;
  const int64_t block = (int64_t)p.page_size * kv4::row_bytes(D);
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int r = first_of(s) + lane / LPR;
    if (first_of(s) >= p.num_rows) break;  // warp-uniform
    if (rotated && r < p.num_q + p.num_kv) {
      float a[8], b[8];
      unpack_bf16x8(xa[s], a);
      unpack_bf16x8(xb[s], b);
      auto turn_all = [&](auto turn) {
        if (NEOX) {
#pragma unroll
          for (int i = 0; i < 8; ++i) turn(a[i], b[i], cs[i], sn[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            turn(a[2 * i], a[2 * i + 1], cs[i], sn[i]);
            turn(b[2 * i], b[2 * i + 1], cs[4 + i], sn[4 + i]);
          }
        }
      };
      // (one branch around all pairs: with the choice made pair by pair every row went
      // both ways)
      if (r < p.num_q) {
        turn_all([](float& u, float& v, float c, float n) {
          const float x = u, y = v;
          u = fmaf(-y, n, x * c);
          v = fmaf(x, n, y * c);
        });
      } else {
        turn_all([](float& u, float& v, float c, float n) {
          const float x = u, y = v;
          u = exact_rotation(x, c, y, n);
          v = exact_rotation(y, c, -x, n);
        });
      }
      xa[s] = pack_bf16x8(a);
      xb[s] = pack_bf16x8(b);
    }
    if (r < p.num_q) {
      __nv_bfloat16* dst = p.q_out + t * p.q_token_stride + (size_t)r * D;
      store_stream(dst + oa, xa[s]);
      store_stream(dst + ob, xb[s]);
    }
    if (!store_kv || first_of(s) + RPW <= p.num_q) continue;  // warp-uniform: no key or value
    const uint32_t sa = span(xa[s]), sb = span(xb[s]);
    const int ga = oa / kv4::kGroup, gb = ob / kv4::kGroup;
    uint32_t own = 0;  // of group l % GROUPS
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      constexpr uint32_t none = 0x7f807f80u;  // (+inf, +inf)
      uint32_t m = min2(ga == g ? sa : none, gb == g ? sb : none);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) m = min2(m, __shfl_xor_sync(kFullMask, m, o));
      if (l % GROUPS == g) own = m;
    }
    const uint32_t ends = own;
    own = group_meta(own);
    const bool cut = __any_sync(kFullMask, past_ends(ends, own));
    const uint32_t ma = __shfl_sync(kFullMask, own, lane - l + ga);
    const uint32_t mb = __shfl_sync(kFullMask, own, lane - l + gb);
    if (r < p.num_q || r >= p.num_rows) continue;
    // key heads, then value heads, as the page holds them
    uint8_t* to = p.cache + (page * 2 * p.num_kv + (r - p.num_q)) * block;
    uint32_t* codes = reinterpret_cast<uint32_t*>(to + (int64_t)off * (D / 2));
    codes[oa / 8] = codes_of(xa[s], ma, cut);
    codes[ob / 8] = codes_of(xb[s], mb, cut);
    uint32_t* words =
        reinterpret_cast<uint32_t*>(to + (int64_t)p.page_size * (D / 2)) + off * GROUPS;
    if (l < GROUPS) words[l] = own;
  }
}

template <int D, bool NEOX, int STEPS>
cudaError_t launch_append4(const AppendArgs& a, cudaStream_t stream) {
  constexpr int RPW = 32 / (D / 16);
  Append4Params p;
  p.qkv = static_cast<__nv_bfloat16*>(a.qkv);
  p.q_out = static_cast<__nv_bfloat16*>(a.q_out);
  p.cos_sin = a.cos_sin;
  p.positions = a.positions;
  p.slots = a.slot_mapping;
  p.cache = static_cast<uint8_t*>(a.kv_cache);
  p.num_q = a.num_heads_q;
  p.num_kv = a.num_heads_kv;
  p.num_rows = a.num_heads_q + 2 * a.num_heads_kv;
  const bool in_place = a.q_out == a.qkv;
  // in place without a rotation the query rows stay as they are
  p.first_row = in_place && a.rotary_dim == 0 ? a.num_heads_q : 0;
  p.q_token_stride = (int64_t)(in_place ? p.num_rows : p.num_q) * D;
  p.rot = a.rotary_dim;
  p.max_pos = a.max_pos;
  p.num_slots = a.num_pages * a.page_size;
  p.page_size = a.page_size;
  p.errors = a.errors;
  const int rows = p.num_rows - p.first_row;
  const int groups = (rows + RPW - 1) / RPW;
  p.chunks = (groups + STEPS - 1) / STEPS;
  p.items = (int64_t)a.num_tokens * p.chunks;
  const int64_t grid = (p.items + kWarps - 1) / kWarps;
  static std::atomic<int> cache[kMaxDevices];
  const auto kernel = append4_kernel<D, NEOX, STEPS>;
  p.trigger_from = last_wave_start(kernel, kWarps * 32, grid, cache);
  return launch_kernel(kernel, dim3((unsigned)grid), dim3(kWarps * 32), 0, stream, p);
}

template <int D, bool NEOX>
cudaError_t append4_shape(const AppendArgs& a, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.num_tokens * (a.num_heads_q + 2 * a.num_heads_kv);
  return rows < 152 * 32 ? launch_append4<D, NEOX, 1>(a, stream)
                         : launch_append4<D, NEOX, 3>(a, stream);
}

template <int D>
cudaError_t append4_dim(const AppendArgs& a, cudaStream_t stream) {
  return a.is_neox ? append4_shape<D, true>(a, stream) : append4_shape<D, false>(a, stream);
}

// ---- reading back -----------------------------------------------------------------

struct Gather4Params {
  const uint8_t* cache;
  const int64_t* slots;
  __nv_bfloat16* k;
  __nv_bfloat16* v;
  int num_kv, page_size;
  int chunks, chunk_rows;  // warps per slot, rows (key heads, then value heads) of each
  int64_t items;
  int64_t num_slots;
  int* errors;
  int trigger_from;
};

// Eight codes -> bf16, packed.  scale (c - 8) is exact in fp32; the sum is rounded
// there and then to bf16.
__device__ __forceinline__ uint4 values_of(uint32_t w, uint32_t meta) {
  const float scale = __uint_as_float(meta << 16), zero = __uint_as_float(meta & 0xffff0000u);
  auto pair = [&](uint32_t x) {  // 16 + c, twice
    const float a = __uint_as_float(x << 16) - 24.f, b = __uint_as_float(x & 0xffff0000u) - 24.f;
    return pack_bf16x2(fmaf(scale, a, zero), fmaf(scale, b, zero));
  };
  return make_uint4(pair(kv4::pair16<0>(w)), pair(kv4::pair16<1>(w)),
                    pair(kv4::pair16<2>(w)), pair(kv4::pair16<3>(w)));
}

template <int D, int STEPS>
__global__ void __launch_bounds__(kWarps * 32) gather4_kernel(const Gather4Params p) {
  constexpr int LPR = D / 16;
  constexpr int RPW = 32 / LPR;
  constexpr int GROUPS = D / kv4::kGroup;
  grid_dependency_sync(p.trigger_from);
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (item >= p.items) return;
  const int lane = threadIdx.x & 31;
  const int l = lane % LPR;
  const int64_t i = item / p.chunks;
  const int chunk = (int)(item - i * p.chunks);
  const int r0 = chunk * p.chunk_rows, r1 = min(r0 + p.chunk_rows, 2 * p.num_kv);
  const int64_t slot = __ldg(p.slots + i);
  const bool bad = slot < -1 || slot >= p.num_slots;
  if (bad && p.errors && chunk == 0 && lane == 0) atomicAdd(p.errors, 1);
  const bool there = slot >= 0 && !bad;
  uint32_t w[STEPS][2], m[STEPS][2];
  if (there) {
    const int64_t page = slot / p.page_size;
    const int off = (int)(slot - page * p.page_size);
    const int64_t block = (int64_t)p.page_size * kv4::row_bytes(D);
    const uint8_t* base = p.cache + page * 2 * p.num_kv * block;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int r = r0 + s * RPW + lane / LPR;
      if (r >= r1) continue;
      const uint8_t* from = base + r * block;
      const uint32_t* codes = reinterpret_cast<const uint32_t*>(from + (int64_t)off * (D / 2));
      const uint32_t* meta =
          reinterpret_cast<const uint32_t*>(from + (int64_t)p.page_size * (D / 2)) + off * GROUPS;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        w[s][h] = __ldg(codes + l + h * LPR);
        m[s][h] = __ldg(meta + (l + h * LPR) / 8);
      }
    }
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int r = r0 + s * RPW + lane / LPR;
    if (r >= r1) continue;
    __nv_bfloat16* to = (r < p.num_kv ? p.k : p.v) +
                        (i * p.num_kv + (r < p.num_kv ? r : r - p.num_kv)) * D;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      store_stream(to + 8 * (l + h * LPR),
                   there ? values_of(w[s][h], m[s][h]) : make_uint4(0, 0, 0, 0));
  }
}

template <int D, int STEPS>
cudaError_t launch_gather4(const Kv4GatherArgs& a, cudaStream_t stream) {
  constexpr int RPW = 32 / (D / 16);
  Gather4Params p;
  p.cache = static_cast<const uint8_t*>(a.kv_cache);
  p.slots = a.slots;
  p.k = static_cast<__nv_bfloat16*>(a.k);
  p.v = static_cast<__nv_bfloat16*>(a.v);
  p.num_kv = a.num_heads_kv;
  p.page_size = a.page_size;
  const int groups = (2 * a.num_heads_kv + RPW - 1) / RPW;
  p.chunks = (groups + STEPS - 1) / STEPS;
  p.chunk_rows = (groups + p.chunks - 1) / p.chunks * RPW;
  p.items = a.num_listed * p.chunks;
  p.num_slots = a.num_pages * a.page_size;
  p.errors = a.errors;
  const int64_t grid = (p.items + kWarps - 1) / kWarps;
  static std::atomic<int> cache[kMaxDevices];
  p.trigger_from = last_wave_start(gather4_kernel<D, STEPS>, kWarps * 32, grid, cache);
  return launch_kernel(gather4_kernel<D, STEPS>, dim3((unsigned)grid), dim3(kWarps * 32), 0,
                       stream, p);
}

template <int D>
cudaError_t gather4_shape(const Kv4GatherArgs& a, cudaStream_t stream) {
  return a.num_listed * 2 * a.num_heads_kv < 152 * 32 ? launch_gather4<D, 1>(a, stream)
                                                      : launch_gather4<D, 4>(a, stream);
}

}  // namespace

cudaError_t launch_kv4_append(const AppendArgs& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 64: return append4_dim<64>(a, stream);
    case 128: return append4_dim<128>(a, stream);
    case 256: return append4_dim<256>(a, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_kv4_gather(const Kv4GatherArgs& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 64: return gather4_shape<64>(a, stream);
    case 128: return gather4_shape<128>(a, stream);
    case 256: return gather4_shape<256>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kvq
