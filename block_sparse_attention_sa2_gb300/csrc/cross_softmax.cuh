// Device helpers that the attention kernels with one row per thread share: exponentials, scores from TMEM,
// their maximum and P, and the product P V.
#pragma once

#include "sa2_device.cuh"

namespace sa2 {

constexpr float kRescaleThreshold = 8.0f;  // log2 units: O and l are rescaled only past 2^8

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 32 scores of a row; those behind the last key (whatever they are) as -inf.
__device__ __forceinline__ void load_scores(uint32_t taddr, float (&x)[32], int valid) {
  uint32_t u[32];
  tmem_ld32(taddr, u);
  tmem_ld_wait(u);
#pragma unroll
  for (int c = 0; c < 32; ++c) x[c] = __uint_as_float(u[c]);
  if (valid < 32) {
#pragma unroll
    for (int c = 0; c < 32; ++c) x[c] = c < valid ? x[c] : -INFINITY;
  }
}

// Maximum of three in one instruction.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

__device__ __forceinline__ float max32(const float (&x)[32]) {
  float m[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) m[c] = max3(x[c], x[c + 4], x[c + 8]);
#pragma unroll
  for (int c = 12; c < 28; c += 8)
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = max3(m[i], x[c + i], x[c + 4 + i]);
  return max3(max3(m[0], x[28], x[29]), max3(m[1], x[30], x[31]), fmaxf(m[2], m[3]));
}

// Two fp32 operations in one instruction (the results are those of two single ones).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 y;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return y;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 y;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 y;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}

// p = exp2(x * mul + add) as 16-bit pairs, and their sum (before rounding) added to l.
template <bool F16>
__device__ __forceinline__ void exp32(const float (&x)[32], float mul, float add, uint32_t* pk, float2 (&l)[2]) {
  const float2 mul2{mul, mul}, addv{add, add};
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    const float2 y = fma2(make_float2(x[2 * c], x[2 * c + 1]), mul2, addv);
    const float2 p{ex2(y.x), ex2(y.y)};
    l[c & 1] = add2(l[c & 1], p);
    pk[c] = F16 ? pack_f16x2(p.x, p.y) : pack_bf16x2(p.x, p.y);
  }
}

// 32 channels of a row, rounded to the call's type.
__device__ __forceinline__ void store32(uint16_t* dst, const float (&v)[32], bool f16) {
  uint4* p = reinterpret_cast<uint4*>(dst);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      w[q] = f16 ? pack_f16x2(v[8 * i + 2 * q], v[8 * i + 2 * q + 1])
                 : pack_bf16x2(v[8 * i + 2 * q], v[8 * i + 2 * q + 1]);
    p[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// O (+)= P V over up to 64 keys: A = P in TMEM (16 keys in 8 columns), B = V, 16 rows per k-step.
__device__ __forceinline__ void issue_pv(uint32_t o, uint32_t p, uint64_t v, uint32_t idesc, int steps, bool fresh) {
  umma_ts(o, p, v, idesc, fresh ? 0u : 1u);
  if (steps == 4) {
#pragma unroll
    for (int kk = 1; kk < 4; ++kk) umma_ts(o, p + kk * 8, v + (uint64_t)(kk * 128), idesc, 1u);
  } else {
    for (int kk = 1; kk < steps; ++kk) umma_ts(o, p + kk * 8, v + (uint64_t)(kk * 128), idesc, 1u);
  }
}

}  // namespace sa2
