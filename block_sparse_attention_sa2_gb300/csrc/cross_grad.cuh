// Device helpers that the backward kernels of attention share: products, and LSE and D as channels of them.
#pragma once

#include "sa2_device.cuh"

namespace sa2 {

__device__ __forceinline__ void store32_bf16(uint16_t* dst, const float (&v)[32]) {
  uint4* p = reinterpret_cast<uint4*>(dst);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    p[i] = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                      pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
}

// One product with A and B K-major in shared memory (128 rows per panel each).
template <int D>
__device__ __forceinline__ void issue_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    umma_ss(d, a + kmajor_kstep(kk, 128), b + kmajor_kstep(kk, 128), idesc, kk > 0 ? 1u : 0u);
}
// D (+)= A B with A in TMEM, 16 rows of B per k-step; A's k-steps 2 i and 2 i + 1 lie in the first 16 of
// the columns 32 i .. 32 i + 31 (over the scores that they were made from).
__device__ __forceinline__ constexpr uint32_t a_kstep(int kk) { return 32u * (kk >> 1) + 8u * (kk & 1); }
__device__ __forceinline__ void issue_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, int steps, bool fresh) {
  umma_ts(d, a, b, idesc, fresh ? 0u : 1u);
#pragma unroll
  for (int kk = 1; kk < 8; ++kk)
    if (kk < steps) umma_ts(d, a + a_kstep(kk), b + (uint64_t)(kk * 128), idesc, 1u);
}

// 16 more channels of 128 rows: 16-byte rows of 8 channels in groups of 8, the groups of channels 0..7
// and 8..15 next to each other.
constexpr int kXTile = 4096;
// LSE is divided by the scale; below this one q . k counts for nothing beside it, and is left to.
constexpr float kMinScale = 0x1p-100f;
__device__ __forceinline__ uint32_t x_row(int r) { return (uint32_t)(r >> 3) * 256 + (r & 7) * 16; }
__device__ __forceinline__ uint64_t x_desc(uint32_t saddr) { return smem_desc(saddr, 128, 256, 0); }
// x as the sum of three bf16 numbers, exact to 2^-24 of x (an infinity or NaN: the first alone).
__device__ __forceinline__ uint2 split3(float x) {
  const uint32_t hi = pack_bf16x2(x, 0.f) & 0xFFFFu;
  const float r1 = x - __uint_as_float(hi << 16);
  if (!(fabsf(r1) < INFINITY)) return make_uint2(hi, 0u);
  const uint32_t mid = pack_bf16x2(r1, 0.f) & 0xFFFFu;
  const uint32_t lo = pack_bf16x2(r1 - __uint_as_float(mid << 16), 0.f) & 0xFFFFu;
  return make_uint2(hi | mid << 16, lo);
}

}  // namespace sa2
