// kvq_dsv4_entry.cuh -- the 584-byte cache entry of one token's shared vector of 512
// dims, and its codes as bf16:
//   bytes [0, 448)    e4m3 codes of dims 0 .. 447, blocks b of 64
//   bytes [448, 576)  dims 448 .. 511 in bf16
//   bytes [576, 583)  UE8M0 exponent bytes of the blocks; byte 583 a pad
#pragma once

#include "kvq_device.cuh"

namespace kvq {
namespace dsv4 {

constexpr int kDim = 512;
constexpr int kEntry = 584;
constexpr int kRopeAt = 448;
constexpr int kScaleAt = 576;

// 2^(byte - 127) as a binary32 (byte 0 gives the subnormal 2^-127).
__device__ __forceinline__ float ue8m0_scale(uint32_t byte) {
  return byte ? __uint_as_float(byte << 23) : __uint_as_float(0x00400000u);
}

// Eight e4m3 codes (element 0 in the lowest byte) times a power of two ->
// eight bf16, packed.
__device__ __forceinline__ uint4 dequant8(const uint2 codes, float scale) {
  const uint32_t w[2] = {codes.x, codes.y};
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_fp8x2_storage_t pair = (__nv_fp8x2_storage_t)(w[k >> 1] >> (16 * (k & 1)));
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(pair, __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    o[k] = pack_bf16x2(f.x * scale, f.y * scale);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace dsv4
}  // namespace kvq
