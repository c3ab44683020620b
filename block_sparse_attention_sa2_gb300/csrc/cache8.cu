// The 8-bit key/value cache: append (quantise) and read (the held values back).
//
// A block of 64 tokens of one head is held as e4m3 values x8 and one scale 2^e, x ~ x8 * 2^e,
// with e the least integer for which the block's largest magnitude is at most 448 * 2^e (448 is
// the largest e4m3 value), kept within [-100, 119].  e4m3 is a floating-point format, so a scale
// that is a power of two costs no precision against an arbitrary one, and it makes everything
// around the values exact: x * 2^-e, the read-back x8 * 2^e in bf16, and the growth of a block's
// scale, which is a shift of the held exponents (rounded again only where that leaves the normal
// range).  The limits keep every factor 2^e, 2^-e a normal fp32 number.
#include <cuda_fp8.h>

#include "cross_internal.h"

namespace sa2 {
namespace {

constexpr int kScaleBlock = 64;
constexpr int kThreads = 256;
constexpr int kEMin = -100, kEMax = 119;
constexpr float kMaxHeld = 448.f * 6.646139978924579e35f;  // 448 * 2^119

// Least e with amax <= 448 * 2^e (448 = 1.75 * 2^8), clamped.  amax >= 0.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, kEMin), kEMax);
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

__device__ __forceinline__ float2 from_e4m3x2(uint32_t x) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x & 0xFFFFu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// One CTA per block of 64 tokens, head and tensor (K or V): the block's new tokens and the tokens
// that it already holds are loaded once into registers (8 channels of 2 or 4 tokens per thread),
// the largest new magnitude is reduced over the CTA, and the block is written once.
// Bound by the bytes: 2 in and 1 out per new value, 1 in and 1 out per held one (8 x 40 heads, 8192 new tokens,
// d = 128: 358 us, 5.6 TB/s).
template <int D, bool F16>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(CacheRef c, int n, TokenRef k, TokenRef v,
                                                               const int32_t* __restrict__ pos,
                                                               const int32_t* __restrict__ n_new, unsigned* status) {
  constexpr int kLanes = D / 8;             // threads per token
  constexpr int kRows = kThreads / kLanes;  // tokens per pass
  constexpr int kPasses = kScaleBlock / kRows;
  __shared__ float warp_max[kThreads / 32];
  const int b = blockIdx.z >> 1, h = blockIdx.y;
  const bool is_v = (blockIdx.z & 1) != 0;
  const int tid = threadIdx.x;
  int p = pos[b], m = n_new ? n_new[b] : n;
  bool bad = p < 0 || p > c.C || m < 0 || m > n;
  p = min(max(p, 0), c.C);
  m = min(max(m, 0), n);
  if (m > c.C - p) {
    bad = true;
    m = c.C - p;
  }
  if (bad && tid == 0) report_error(status, kDevErrBounds);
  const int j = p / kScaleBlock + blockIdx.x;  // block of the cache
  const int t0 = j * kScaleBlock;
  if (m == 0 || t0 >= p + m) return;  // the same for the whole CTA
  const TokenRef& src = is_v ? v : k;
  const uint16_t* x = static_cast<const uint16_t*>(src.p) + b * src.sb + h * src.sh;
  uint8_t* x8 = (is_v ? c.v : c.k) + b * c.sb + h * c.sh;
  float* scale = (is_v ? c.vs : c.ks) + ((int64_t)b * gridDim.y + h) * c.nsb + j;
  const bool held = t0 < p;  // the block keeps tokens
  const int ch = (tid % kLanes) * 8, r0 = tid / kLanes;

  uint4 in[kPasses];
  uint2 old[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int t = t0 + r0 + i * kRows;
    in[i] = make_uint4(0, 0, 0, 0);
    old[i] = make_uint2(0, 0);
    if (t >= p && t < p + m)
      in[i] = *reinterpret_cast<const uint4*>(x + (int64_t)(t - p) * src.sn + ch);
    else if (t < p)
      old[i] = *reinterpret_cast<const uint2*>(x8 + (int64_t)t * c.sn + ch);
  }
  const float was = held ? *scale : 0.f;
  float amax = 0.f;
  bool odd = false;  // an infinity, a NaN or a value that is saturated
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const uint32_t w[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 f = unpack2<F16>(w[q]);
      amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
      odd |= !(fabsf(f.x) <= kMaxHeld) || !(fabsf(f.y) <= kMaxHeld);
    }
  }
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((tid & 31) == 0) warp_max[tid >> 5] = amax;
  if (odd) report_error(status, kDevErrRange);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) amax = fmaxf(amax, warp_max[w]);

  int e = scale_exponent(amax);
  const int e_was = (int)(__float_as_uint(was) >> 23) - 127;
  if (held) e = min(max(e, e_was), kEMax);
  const float mul = pow2(-e);
  // 2^(e_was - e) takes a held value to the new scale; below 2^-126 every one of them rounds to 0
  const float shift = held ? (e_was - e < -126 ? 0.f : pow2(e_was - e)) : 0.f;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int t = t0 + r0 + i * kRows;
    if (t >= p + m) continue;
    uint2 out;
    if (t >= p) {
      const float2 f0 = unpack2<F16>(in[i].x), f1 = unpack2<F16>(in[i].y), f2 = unpack2<F16>(in[i].z),
                   f3 = unpack2<F16>(in[i].w);
      out.x = to_e4m3x4(f0.x * mul, f0.y * mul, f1.x * mul, f1.y * mul);
      out.y = to_e4m3x4(f2.x * mul, f2.y * mul, f3.x * mul, f3.y * mul);
    } else {
      if (shift == 1.f) continue;  // held as it is
      const float2 f0 = from_e4m3x2(old[i].x), f1 = from_e4m3x2(old[i].x >> 16), f2 = from_e4m3x2(old[i].y),
                   f3 = from_e4m3x2(old[i].y >> 16);
      out.x = to_e4m3x4(f0.x * shift, f0.y * shift, f1.x * shift, f1.y * shift);
      out.y = to_e4m3x4(f2.x * shift, f2.y * shift, f3.x * shift, f3.y * shift);
    }
    *reinterpret_cast<uint2*>(x8 + (int64_t)t * c.sn + ch) = out;
  }
  if (tid == 0) *scale = pow2(e);  // every thread read the old scale before the barrier above
}

// Tokens [pos[b], pos[b] + n) back at 16 bits: 16 channels per thread, K and V in one launch.
// e4m3 * 2^e is exact in bf16; in fp16 it is rounded, and infinite beyond the fp16 range.  Bound by the bytes
// (8 x 40 heads, 8192 tokens, d = 128: 324 us, 6.2 TB/s).
template <int D, bool F16>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(CacheRef c, int n, TokenRef k, TokenRef v,
                                                             const int32_t* __restrict__ pos, unsigned* status) {
  constexpr int kLanes = D / 16;
  const int b = blockIdx.z >> 1, h = blockIdx.y;
  const bool is_v = (blockIdx.z & 1) != 0;
  const int i = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  if (i >= n) return;
  const int ch = (threadIdx.x % kLanes) * 16;
  const int64_t t = (int64_t)pos[b] + i;
  const TokenRef& dst = is_v ? v : k;
  uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (t < 0 || t >= c.C) {
    report_error(status, kDevErrBounds);
  } else {
    const uint8_t* x8 = (is_v ? c.v : c.k) + b * c.sb + h * c.sh + t * c.sn + ch;
    const float s = (is_v ? c.vs : c.ks)[((int64_t)b * gridDim.y + h) * c.nsb + t / kScaleBlock];
    const uint4 u = *reinterpret_cast<const uint4*>(x8);
    const uint32_t in[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 f0 = from_e4m3x2(in[q]), f1 = from_e4m3x2(in[q] >> 16);
      w[2 * q] = F16 ? pack_f16x2(f0.x * s, f0.y * s) : pack_bf16x2(f0.x * s, f0.y * s);
      w[2 * q + 1] = F16 ? pack_f16x2(f1.x * s, f1.y * s) : pack_bf16x2(f1.x * s, f1.y * s);
    }
  }
  uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst.p) + b * dst.sb + h * dst.sh +
                                        (int64_t)i * dst.sn + ch);
  out[0] = make_uint4(w[0], w[1], w[2], w[3]);
  out[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

}  // namespace

cudaError_t launch_cache_append(const CacheRef& c, int B, int Hkv, int d, int n, bool f16, const TokenRef& k,
                                const TokenRef& v, const int32_t* pos, const int32_t* n_new, unsigned* status,
                                cudaStream_t st) {
  const dim3 grid((unsigned)((n + kScaleBlock - 2) / kScaleBlock + 1), (unsigned)Hkv, (unsigned)(2 * B));
  prof_start(st, kToF16);
  if (d == 128)
    f16 ? cache_append_kernel<128, true><<<grid, kThreads, 0, st>>>(c, n, k, v, pos, n_new, status)
        : cache_append_kernel<128, false><<<grid, kThreads, 0, st>>>(c, n, k, v, pos, n_new, status);
  else
    f16 ? cache_append_kernel<64, true><<<grid, kThreads, 0, st>>>(c, n, k, v, pos, n_new, status)
        : cache_append_kernel<64, false><<<grid, kThreads, 0, st>>>(c, n, k, v, pos, n_new, status);
  prof_stop(st, kToF16);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheRef& c, int B, int Hkv, int d, int n, bool f16, const TokenRef& k,
                              const TokenRef& v, const int32_t* pos, unsigned* status, cudaStream_t st) {
  const int per = kThreads / (d / 16);
  const dim3 grid((unsigned)((n + per - 1) / per), (unsigned)Hkv, (unsigned)(2 * B));
  prof_start(st, kToF16);
  if (d == 128)
    f16 ? cache_read_kernel<128, true><<<grid, kThreads, 0, st>>>(c, n, k, v, pos, status)
        : cache_read_kernel<128, false><<<grid, kThreads, 0, st>>>(c, n, k, v, pos, status);
  else
    f16 ? cache_read_kernel<64, true><<<grid, kThreads, 0, st>>>(c, n, k, v, pos, status)
        : cache_read_kernel<64, false><<<grid, kThreads, 0, st>>>(c, n, k, v, pos, status);
  prof_stop(st, kToF16);
  return cudaGetLastError();
}

}  // namespace sa2
