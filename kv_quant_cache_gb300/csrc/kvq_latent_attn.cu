// kvq_latent_attn.cu -- attention of each token's heads over the latent entries
// listed for it: keys and values are the same 512-dim vectors of the FP8 cache.
//
// A CTA takes 16 heads of one token and a part of its list, 64 entries at a time.
// Its warps read 16 entries each, as the gather does, and leave them as bf16 rows
// in shared memory (16-byte fragment c of row r at c ^ (r & 7)); each then takes the
// scores of its 16 keys, and after the row maxima have been exchanged, 128 dims of
// the output over all 64.  Where the list is split, the parts are joined by a second
// launch.
#include "kvq_dsv4_entry.cuh"
#include "kvq_mma.cuh"
#include "kvq_paged_attn.cuh"
#include "kvq_tma.cuh"

namespace kvq {
namespace {

constexpr int kWarps = 4;
constexpr int kRows = 16;  // heads of a CTA
constexpr int kKeys = 64;  // entries of a step
constexpr int kDim = dsv4::kDim;

struct LatentParams {
  const __nv_bfloat16* q;
  int64_t q_stride;
  int num_heads, tiles;  // tiles of 16 heads
  const uint8_t* cache;
  int64_t num_slots;
  const int* slots;
  int list_width;
  const int* lens;
  float scale_log2;
  int splits;
  __nv_bfloat16* out;
  Partials parts;  // with several splits
  int* errors;
  int trigger_from;
};

constexpr int kTile = kKeys * kDim * 2;              // bytes of the entries of a step
constexpr int kQAt = kTile;                          // Q, 16 rows of 1024 bytes
constexpr int kPAt = kQAt + kRows * kDim * 2;        // P, 16 rows of 64, 144 bytes apart
constexpr int kPStride = 144;
constexpr int kTopAt = kPAt + kRows * kPStride;      // [4 warps][16] maxima, then sums
constexpr int kSmem = kTopAt + kWarps * kRows * 4;

__device__ __forceinline__ uint32_t row_at(int r, int c) {  // fragment c of a row of 512
  return r * 1024 + ((c ^ (r & 7)) << 4);
}

__global__ void __launch_bounds__(kWarps * 32, 2) latent_rows_kernel(const LatentParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  grid_dependency_sync(p.trigger_from);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int64_t token = blockIdx.x / p.tiles;
  const int head0 = (int)(blockIdx.x - token * p.tiles) * kRows;
  const int rows = min(kRows, p.num_heads - head0);
  const uint32_t base = tma::smem_addr(smem);
  volatile float* tops = reinterpret_cast<float*>(smem + kTopAt);

  bool rejected = false;
  int len = __ldg(p.lens + token);
  if (len < 0 || len > p.list_width) {
    rejected = threadIdx.x == 0;
    len = len < 0 ? 0 : p.list_width;
  }
  const int steps = len / kKeys + (len % kKeys != 0);
  const int share = (steps + p.splits - 1) / p.splits;
  const int first = min((int)blockIdx.y * share, steps), last = min(first + share, steps);

  for (int i = threadIdx.x; i < kRows * 64; i += kWarps * 32) {
    const int r = i >> 6, c = i & 63;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r < rows)
      v = __ldg(reinterpret_cast<const uint4*>(p.q + token * p.q_stride +
                                               (int64_t)(head0 + r) * kDim) + c);
    *reinterpret_cast<uint4*>(smem + kQAt + row_at(r, c)) = v;
  }

  float o[16][4] = {};
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  for (int step = first; step < last; ++step) {
    // ---- the warp's 16 entries -------------------------------------------------------
    int slot = -1;
    {
      const int at = step * kKeys + warp * 16 + (lane & 15);
      if (at < len) {
        slot = __ldg(p.slots + token * p.list_width + at);
        if (slot < -1 || slot >= p.num_slots) {
          if (lane < 16) rejected = true;
          slot = -1;
        }
      }
    }
    const uint32_t there = __ballot_sync(kFullMask, slot >= 0);
    __syncthreads();  // the step before has been read
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
      const int s = __shfl_sync(kFullMask, slot, i);
      const int r = warp * 16 + i;
      uint4 a = make_uint4(0, 0, 0, 0), b = a;
      if (s >= 0) {
        const uint8_t* e = p.cache + (int64_t)s * dsv4::kEntry;
        const uint2 sc = __ldg(reinterpret_cast<const uint2*>(e + dsv4::kScaleAt));
        const uint2 c0 = __ldg(reinterpret_cast<const uint2*>(e + 8 * lane));
        a = dsv4::dequant8(c0, dsv4::ue8m0_scale(sc.x >> (8 * (lane >> 3)) & 0xffu));
        if (lane < 24) {
          const uint2 c1 = __ldg(reinterpret_cast<const uint2*>(e + 256 + 8 * lane));
          b = dsv4::dequant8(c1, dsv4::ue8m0_scale(sc.y >> (8 * (lane >> 3)) & 0xffu));
        } else {
          const uint2* rope =
              reinterpret_cast<const uint2*>(e + dsv4::kRopeAt + 16 * (lane - 24));
          const uint2 x = __ldg(rope), y = __ldg(rope + 1);
          b = make_uint4(x.x, x.y, y.x, y.y);
        }
      }
      *reinterpret_cast<uint4*>(smem + row_at(r, lane)) = a;
      *reinterpret_cast<uint4*>(smem + row_at(r, 32 + lane)) = b;
    }
    __syncwarp();
    if (step == first) __syncthreads();  // Q is there

    // ---- scores of the warp's keys ------------------------------------------------------
    float s[2][4] = {};
    {
      const int qr = (lane & 7) + ((lane >> 3 & 1) << 3), qc = lane >> 4;
      const int kr = warp * 16 + (lane & 7) + (lane >> 4 << 3), kc = lane >> 3 & 1;
#pragma unroll 8
      for (int k = 0; k < kDim / 16; ++k) {
        uint32_t a[4], b[4];
        ldmatrix4(a, base + kQAt + row_at(qr, 2 * k + qc));
        ldmatrix4(b, base + row_at(kr, 2 * k + kc));
        mma16816(s[0], a, b[0], b[1]);
        mma16816(s[1], a, b[2], b[3]);
      }
    }
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = 8 * h + 2 * t4 + (k & 1);
        s[h][k] = there >> key & 1 ? s[h][k] * p.scale_log2 : -INFINITY;
        top[k >> 1] = fmaxf(top[k >> 1], s[h][k]);
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(kFullMask, top[r], 1));
      top[r] = fmaxf(top[r], __shfl_xor_sync(kFullMask, top[r], 2));
      if (t4 == 0) tops[warp * kRows + g + 8 * r] = top[r];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float to = m[r];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) to = fmaxf(to, tops[w * kRows + g + 8 * r]);
      const float f = to == m[r] ? 1.f : exp2f(m[r] - to);
      l[r] *= f;
#pragma unroll
      for (int n = 0; n < 16; ++n) o[n][2 * r] *= f, o[n][2 * r + 1] *= f;
      m[r] = to;
      const float ref = to == -INFINITY ? 0.f : to;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float x = exp2f(s[h][2 * r] - ref), y = exp2f(s[h][2 * r + 1] - ref);
        l[r] += x + y;
        *reinterpret_cast<uint32_t*>(smem + kPAt + (g + 8 * r) * kPStride +
                                     (warp * 16 + 8 * h + 2 * t4) * 2) = pack_bf16x2(x, y);
      }
    }
    __syncthreads();

    // ---- the warp's 128 dims -------------------------------------------------------------
#pragma unroll
    for (int k = 0; k < kKeys / 16; ++k) {
      uint32_t a[4];
      ldmatrix4(a, base + kPAt + ((lane & 7) + ((lane >> 3 & 1) << 3)) * kPStride +
                       (16 * k + 8 * (lane >> 4)) * 2);
      const int r = 16 * k + (lane & 7) + ((lane >> 3 & 1) << 3);
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        uint32_t b[4];
        ldmatrix4_trans(b, base + row_at(r, 16 * warp + 2 * n + (lane >> 4)));
        mma16816(o[2 * n], a, b[0], b[1]);
        mma16816(o[2 * n + 1], a, b[2], b[3]);
      }
    }
  }
  if (rejected && p.errors) atomicAdd(p.errors, 1);
  // the sums of the warps' keys
  __syncthreads();
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(kFullMask, l[r], 1);
    l[r] += __shfl_xor_sync(kFullMask, l[r], 2);
    if (t4 == 0) tops[warp * kRows + g + 8 * r] = l[r];
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = g + 8 * h;
    if (r >= rows) continue;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += tops[w * kRows + r];
    const float f = sum == 0.f ? 0.f : 1.f / sum;  // 0: the row has no key
    const int64_t row = token * p.num_heads + head0 + r;
    const int d = 128 * warp + 2 * t4;
    if (p.splits == 1) {
#pragma unroll
      for (int n = 0; n < 16; ++n)
        *reinterpret_cast<uint32_t*>(p.out + row * kDim + d + 8 * n) =
            pack_bf16x2(o[n][2 * h] * f, o[n][2 * h + 1] * f);
    } else {
      const int64_t slot = blockIdx.y;
#pragma unroll
      for (int n = 0; n < 16; ++n)
        *reinterpret_cast<float2*>(p.parts.o + (slot * p.parts.rows + row) * kDim + d + 8 * n) =
            make_float2(o[n][2 * h] * f, o[n][2 * h + 1] * f);
      if (warp == 0 && t4 == 0)
        p.parts.lse[slot * p.parts.rows + row] =
            sum == 0.f ? -INFINITY : (m[h] == -INFINITY ? 0.f : m[h]) + log2f(sum);
    }
  }
}

int latent_splits(int64_t num_tokens, int num_heads, int list_width) {
  const int64_t units = num_tokens * ((num_heads + kRows - 1) / kRows);
  const int64_t steps = ((int64_t)list_width + kKeys - 1) / kKeys;
  int64_t splits = 1;
  while (units * (splits + 1) <= 2 * 152 && steps >= (splits + 1) * 2) ++splits;
  return (int)splits;
}

}  // namespace

int64_t latent_attn_workspace(int64_t num_tokens, int num_heads, int list_width) {
  const int s = latent_splits(num_tokens, num_heads, list_width);
  return s == 1 ? 0 : partials_bytes(s, num_tokens * num_heads, kDim);
}

cudaError_t launch_latent_attn(const LatentAttnArgs& a, cudaStream_t stream) {
  LatentParams p = {};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.q_stride = a.q_stride;
  p.num_heads = a.num_heads;
  p.tiles = (a.num_heads + kRows - 1) / kRows;
  p.cache = a.kv_cache;
  p.num_slots = a.num_slots;
  p.slots = a.slots;
  p.list_width = a.list_width;
  p.lens = a.lens;
  p.scale_log2 = a.scale * kLog2e;
  p.splits = latent_splits(a.num_tokens, a.num_heads, a.list_width);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.errors = a.errors;
  const int64_t rows = (int64_t)a.num_tokens * a.num_heads;
  if (p.splits > 1) p.parts = partials_at(a.workspace, p.splits, rows, kDim);
  static std::atomic<int> cache[kMaxDevices];
  int per_sm = 0;
  cudaError_t e = tma::prepare(latent_rows_kernel, kWarps * 32, kSmem, cache, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t ctas = (int64_t)a.num_tokens * p.tiles;
  const int64_t wave = (int64_t)per_sm * device_sm_count();
  p.trigger_from = ctas > wave ? (int)(ctas - wave) : 0;
  e = launch_kernel(latent_rows_kernel, dim3((unsigned)ctas, (unsigned)p.splits),
                    dim3(kWarps * 32), kSmem, stream, p);
  if (e != cudaSuccess || p.splits == 1) return e;
  return launch_attn_join(p.parts, p.splits, kDim, a.out, stream);
}

}  // namespace kvq
