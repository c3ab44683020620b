// Attention of few query rows (at most 16 per key head: tokens x the heads that share it) to many
// keys, 16-bit or from the 8-bit cache, on sm_103a.
//
// Every key and value is used for 16 rows at most, so the bytes bound it: the kernel is built to keep
// them coming.  One CTA of 8 warps per SM; each warp takes its own steps of keys (4 KB of K and 4 KB
// of V), copied into a ring of its own in shared memory by cp.async, three steps deep: 192 KB under
// way per SM, and no barrier between warps until the end of a piece (8 x 40 heads, 32760 keys, d = 128: one
// query 376 us over cached keys, 7.1 TB/s, and 796 over 16-bit ones, 6.7 TB/s; 16 queries 388 and 792; 17, which
// the kernel of 128-row tiles takes, 895 and 798).  The products are the warp's own
// mma.sync m16n8k16: tcgen05 works on 128 rows, of which 112 would be empty, and needs its operands in
// the layouts that TMA writes, while here the bytes go from the ring straight into fragments:
//   S = Q K^T   A = Q (16 rows), B = K: thread (g, t) = (lane / 4, lane % 4) holds key g's channels
//               from its own 16-byte chunks, in any order, as Q's fragments have the same one
//   O += P V    A = P = the fragments that S came out in; B = V: thread (g, t) holds its four keys'
//               values of channels in chunk g (+ 8 i), pairs of keys interleaved byte by byte
// 8-bit values become fp16 with one conversion per pair.  V's scale enters the exponent (see
// include/sa2.h), K's and the query row's multiply the score.
// A piece's warps are joined in shared memory, pieces of a split segment by cross_join_kernel.
#include <cuda_fp8.h>

#include "cross_few.cuh"
#include "cross_sched.cuh"
#include "cross_softmax.cuh"

namespace sa2 {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kStages = 3;
constexpr int kTileBytes = kFewTileBytes;
constexpr int kStageBytes = 2 * kTileBytes;

__device__ __forceinline__ uint32_t f16x2_of(uint32_t e4m3x2) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(e4m3x2 & 0xFFFFu), __NV_E4M3);
  return *reinterpret_cast<const uint32_t*>(&h);
}

struct KvRef {
  const uint8_t *k, *v;
  int64_t k_sb, k_sh, k_sn, v_sb, v_sh, v_sn;  // in bytes
  const float *ks, *vs;
  int nsb;
};

// F16: the type of Q and O (and of K, V when they are 16-bit).
template <int D, bool KV8, bool F16>
__global__ void __launch_bounds__(kThreads, 1) cross_few_kernel(CrossShape s, FwdPlan plan, KvRef kv, CrossFwdArgs a) {
  using T = FewTile<D, KV8>;
  constexpr bool kMmaF16 = KV8 || F16;
  constexpr int kNT = T::kKeys / 8;   // 8-key tiles of S per step
  constexpr int kCT = D / 8;          // 8-channel tiles of O
  constexpr int kKS = D / 16;         // k-steps of S
  constexpr int kKC = T::kChunks / 4 > 0 ? T::kChunks / 4 : 1;  // K chunks per thread and key
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float warp_m[kWarps][kFewRows], warp_l[kWarps][kFewRows], warp_r[kWarps][kFewRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * kStages * kStageBytes;
  const uint32_t ring_u = smem_u32(ring);
  const int rows = s.N * s.G;
  if (a.kv_len && blockIdx.x == 0)
    for (int b = tid; b < s.B; b += kThreads)
      if (a.kv_len[b] < 0 || a.kv_len[b] > s.M) report_error(a.status, kDevErrBounds);

  if (plan.split) kernel_trigger();
  PieceIter it(s, plan, a.kv_len);
  Piece x;
  while (it.next(x)) {
    const int key0 = x.k0 << 6, key1 = min(x.keys, (x.k0 + x.nb) << 6);
    const uint8_t* kp = kv.k + x.b * kv.k_sb + x.hk * kv.k_sh;
    const uint8_t* vp = kv.v + x.b * kv.v_sb + x.hk * kv.v_sh;
    const float *ksp = kv.ks, *vsp = kv.vs;
    if constexpr (KV8) {
      const int64_t off = ((int64_t)x.b * s.Hkv + x.hk) * kv.nsb;
      ksp += off;
      vsp += off;
    }
    // step i of this warp: keys from key0 + (i * kWarps + warp) * kKeys on
    const int steps_all = (key1 - key0 + T::kKeys - 1) / T::kKeys;
    const int steps = steps_all > warp ? (steps_all - warp + kWarps - 1) / kWarps : 0;
    auto copy_step = [&](int i) {
      if (i < steps) {
        const uint32_t dst = ring_u + (i % kStages) * kStageBytes;
        const int base = key0 + (i * kWarps + warp) * T::kKeys;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int c = (q * 32 + lane) % T::kChunks, r = (q * 32 + lane) / T::kChunks;
          const bool live = base + r < key1;
          const int64_t key = live ? base + r : key0;
          copy16(dst + T::at(r, c), kp + key * kv.k_sn + c * 16, live);
          copy16(dst + kTileBytes + T::at(r, c), vp + key * kv.v_sn + c * 16, live);
        }
      }
      copy_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) copy_step(i);
    float nks = 1.f, nvs = 1.f;  // the next step's scales
    auto load_scales = [&](int i) {
      if (KV8 && i < steps) {  // (a step lies within one block of 64 tokens)
        const int block = (key0 + (i * kWarps + warp) * T::kKeys) >> 6;
        nks = __ldg(ksp + block);
        nvs = __ldg(vsp + block);
      }
    };
    load_scales(0);

    // Q's fragments: rows g and g + 8; of each, this thread's channels in the order of its K chunks
    uint32_t qf[kKS][4];
    float row_scale[2] = {a.scale_log2, a.scale_log2};
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int r = g + 8 * hf, n = r / s.G, h = x.hk * s.G + r - n * s.G;
      const bool live = r < rows;
      const uint16_t* qp = static_cast<const uint16_t*>(a.q.p) + x.b * a.q.sb + h * a.q.sh + (int64_t)n * a.q.sn;
      uint32_t w[2 * kKS];
#pragma unroll
      for (int i = 0; i < 2 * kKS; ++i) {  // pair i: values 2 i, 2 i + 1 of the thread's list
        const int pos = 2 * i, ci = pos / T::kPer;
        const int c = T::kChunks >= 8 ? 2 * t + (ci & 1) + 8 * (ci >> 1) : t;
        w[i] = live ? *reinterpret_cast<const uint32_t*>(qp + c * T::kPer + pos % T::kPer) : 0u;
      }
      if constexpr (KV8 && !F16) {
        // bf16 rows to fp16 under a power of two that takes the largest magnitude to [2^14, 2^15)
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < 2 * kKS; ++i) mx = max(mx, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        int e = 0;
        // a row of zeros, or with an infinity or NaN, keeps its scale
        if (mx >= 0x0080u && mx < 0x7F80u) e = min(max((int)(mx >> 7) - 127 - 14, -112), 112);
        const float f = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < 2 * kKS; ++i)
          w[i] = pack_f16x2(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xFFFF0000u) * f);
        row_scale[hf] *= __uint_as_float((uint32_t)(127 + e) << 23);
      }
#pragma unroll
      for (int k = 0; k < kKS; ++k) {
        qf[k][hf] = w[2 * k];
        qf[k][2 + hf] = w[2 * k + 1];
      }
    }

    float o[kCT][4] = {};
    // reference of the exponentials; sum of exp2(s), relative to m_used, cache: to l_ref (see cross_fwd.cu)
    float m_used[2] = {0.f, 0.f}, l[2] = {0.f, 0.f}, l_ref[2] = {-INFINITY, -INFINITY};
    for (int i = 0; i < steps; ++i) {
      copy_step(i + kStages - 1);
      copy_wait<kStages - 1>();
      __syncwarp();
      const uint8_t* kt = ring + (i % kStages) * kStageBytes;
      const uint8_t* vt = kt + kTileBytes;
      const int base = key0 + (i * kWarps + warp) * T::kKeys;
      float mul[2] = {row_scale[0], row_scale[1]}, ev = 0.f;
      if constexpr (KV8) {
        mul[0] = score_factor(row_scale[0], nks);
        mul[1] = score_factor(row_scale[1], nks);
        ev = (float)((int)(__float_as_uint(nvs) >> 23) - 127);
        load_scales(i + 1);
      }
      // S: tile j has keys 8 j .. 8 j + 7; thread: rows g, g + 8, keys 8 j + 2 t, + 1
      float sc[kNT][4];
#pragma unroll
      for (int j = 0; j < kNT; ++j) {
        sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
        uint32_t w[4 * kKC];
#pragma unroll
        for (int c = 0; c < kKC; ++c) {
          const int ch = T::kChunks >= 8 ? 2 * t + (c & 1) + 8 * (c >> 1) : t;
          const uint4 u = *reinterpret_cast<const uint4*>(kt + T::at(8 * j + g, ch));
          w[4 * c] = u.x;
          w[4 * c + 1] = u.y;
          w[4 * c + 2] = u.z;
          w[4 * c + 3] = u.w;
        }
#pragma unroll
        for (int k = 0; k < kKS; ++k) {
          if constexpr (KV8)
            mma16816<true>(sc[j], qf[k], f16x2_of(w[k]), f16x2_of(w[k] >> 16));
          else
            mma16816<F16>(sc[j], qf[k], w[2 * k], w[2 * k + 1]);
        }
      }
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < kNT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (base + 8 * j + 2 * t + (q & 1) >= key1) sc[j][q] = -INFINITY;
          mx[q >> 1] = fmaxf(mx[q >> 1], sc[j][q]);
        }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        mx[hf] = fmaf(mx[hf], mul[hf], ev);
        mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(0xffffffffu, mx[hf], 1));
        mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(0xffffffffu, mx[hf], 2));
      }
      if (i == 0) {
        m_used[0] = fmaxf(mx[0], kLeastRef);
        m_used[1] = fmaxf(mx[1], kLeastRef);
      } else if (__any_sync(0xffffffffu, mx[0] > m_used[0] + kRescaleThreshold || mx[1] > m_used[1] + kRescaleThreshold)) {
        float al[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          // (a row's reference follows from its own scores only)
          const float m = mx[hf] > m_used[hf] + kRescaleThreshold ? mx[hf] : m_used[hf];
          al[hf] = m == m_used[hf] ? 1.f : ex2(m_used[hf] - m);
          if constexpr (!KV8) l[hf] *= al[hf];
          m_used[hf] = m;
        }
#pragma unroll
        for (int c = 0; c < kCT; ++c) {
          o[c][0] *= al[0];
          o[c][1] *= al[0];
          o[c][2] *= al[1];
          o[c][3] *= al[1];
        }
      }
      // P in the layout of an A operand: 16 keys (tiles 2 k, 2 k + 1) per k-step
      uint32_t pf[kNT / 2][4];
      float ls[2] = {0.f, 0.f};
      // cache: scores whose exponent is 2^-64 or less of the reference's are 0 in P, but count in the sum
      const bool low[2] = {KV8 && mx[0] < m_used[0] - 64.f, KV8 && mx[1] < m_used[1] - 64.f};
      const float ref[2] = {low[0] ? mx[0] : m_used[0], low[1] ? mx[1] : m_used[1]};
      const float add[2] = {ev - ref[0], ev - ref[1]};
#pragma unroll
      for (int j = 0; j < kNT; ++j) {
        float p[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          p[q] = ex2(fmaf(sc[j][q], mul[q >> 1], add[q >> 1]));
          ls[q >> 1] += p[q];
        }
        pf[j >> 1][2 * (j & 1)] = kMmaF16 ? pack_f16x2(p[0], p[1]) : pack_bf16x2(p[0], p[1]);
        pf[j >> 1][2 * (j & 1) + 1] = kMmaF16 ? pack_f16x2(p[2], p[3]) : pack_bf16x2(p[2], p[3]);
      }
      if constexpr (KV8) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float y = ref[hf] - ev;
          if (y > l_ref[hf] + 60.f) {  // (the first step too)
            l[hf] *= ex2(l_ref[hf] - y);
            l_ref[hf] = y;
          }
          l[hf] = fmaf(ls[hf], ex2(y - l_ref[hf]), l[hf]);
        }
        if (__any_sync(0xffffffffu, low[0] || low[1])) {
#pragma unroll
          for (int k = 0; k < kNT / 2; ++k)
#pragma unroll
            for (int q = 0; q < 4; ++q) pf[k][q] = low[q & 1] ? 0u : pf[k][q];
        }
      } else {
        l[0] += ls[0];
        l[1] += ls[1];
        l_ref[0] = m_used[0];
        l_ref[1] = m_used[1];
      }
      // O += P V: keys 16 k + 2 t, + 1 and 16 k + 8 + 2 t, + 1; channels of chunk g (+ 8 i)
#pragma unroll
      for (int k = 0; k < kNT / 2; ++k) {
        if constexpr (KV8) {
          constexpr int kWords = D / 32;  // words of a key per thread (16 or 8 bytes)
          uint32_t v[4][kWords];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = 16 * k + 2 * t + (q & 1) + 8 * (q >> 1);
            if constexpr (D == 128)
              *reinterpret_cast<uint4*>(v[q]) = *reinterpret_cast<const uint4*>(vt + T::at(r, g));
            else
              *reinterpret_cast<uint2*>(v[q]) = *reinterpret_cast<const uint2*>(vt + T::at(r, g >> 1) + (g & 1) * 8);
          }
#pragma unroll
          for (int w = 0; w < kWords; ++w)
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // bytes 2 e, 2 e + 1 of the word: channels 4 w + 2 e, + 1
              const uint32_t sel = e ? 0x7362u : 0x5140u;
              const uint32_t lo = __byte_perm(v[0][w], v[1][w], sel), hi = __byte_perm(v[2][w], v[3][w], sel);
              mma16816<true>(o[4 * w + 2 * e], pf[k], f16x2_of(lo), f16x2_of(hi));
              mma16816<true>(o[4 * w + 2 * e + 1], pf[k], f16x2_of(lo >> 16), f16x2_of(hi >> 16));
            }
        } else {
          constexpr int kVC = D / 64;  // chunks g + 8 i
#pragma unroll
          for (int i8 = 0; i8 < kVC; ++i8) {
            uint32_t v[4][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int r = 16 * k + 2 * t + (q & 1) + 8 * (q >> 1);
              *reinterpret_cast<uint4*>(v[q]) = *reinterpret_cast<const uint4*>(vt + T::at(r, g + 8 * i8));
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              mma16816<F16>(o[8 * i8 + 2 * w], pf[k], __byte_perm(v[0][w], v[1][w], 0x5410),
                            __byte_perm(v[2][w], v[3][w], 0x5410));
              mma16816<F16>(o[8 * i8 + 2 * w + 1], pf[k], __byte_perm(v[0][w], v[1][w], 0x7632),
                            __byte_perm(v[2][w], v[3][w], 0x7632));
            }
          }
        }
      }
      __syncwarp();  // the step's stage is read before its next copy
    }
    // ---- join the warps: O relative to the largest of their references
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 1);
      l[hf] += __shfl_xor_sync(0xffffffffu, l[hf], 2);
      if (t == 0) {
        warp_m[warp][g + 8 * hf] = steps > 0 ? m_used[hf] : -INFINITY;
        warp_l[warp][g + 8 * hf] = steps > 0 ? l[hf] : 0.f;
        warp_r[warp][g + 8 * hf] = steps > 0 ? l_ref[hf] : -INFINITY;
      }
    }
    copy_wait<0>();
    __syncthreads();  // every ring is read: it holds the warps' O now, [warp][row][channel]
    float* os = reinterpret_cast<float*>(smem);
    constexpr int kPitch = D + 4;
    if (steps > 0) {
#pragma unroll
      for (int c = 0; c < kCT; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = g + 8 * (q >> 1), n = 2 * t + (q & 1);
          // channel tile c: value c % kVal of chunk (or half chunk) n + 8 (c / kVal)
          constexpr int kVal = KV8 ? D / 8 : 8;
          os[(warp * kFewRows + r) * kPitch + (n + 8 * (c / kVal)) * kVal + c % kVal] = o[c][q];
        }
    }
    __syncthreads();
    for (int i = tid; i < rows * (D / 2); i += kThreads) {
      const int r = i / (D / 2), ch = i % (D / 2) * 2;
      float m = -INFINITY, lr = -INFINITY;
      bool nan = false;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        nan |= warp_m[w][r] != warp_m[w][r];
        m = fmaxf(m, warp_m[w][r]);
        lr = fmaxf(lr, warp_r[w][r]);
      }
      if (nan) m = NAN;
      float v0 = 0.f, v1 = 0.f, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (warp_m[w][r] == -INFINITY) continue;  // no keys
        const float f = ex2(warp_m[w][r] - m);
        const float2 u = *reinterpret_cast<const float2*>(os + (w * kFewRows + r) * kPitch + ch);
        v0 = fmaf(f, u.x, v0);
        v1 = fmaf(f, u.y, v1);
        sum = fmaf(ex2(warp_r[w][r] - lr), warp_l[w][r], sum);
      }
      const float root = ex2(0.5f * (m - lr));  // 2^(m - lr) alone may leave fp32's range
      const float inv = sum == 0.f ? 0.f : root / sum * root;  // (no keys, or no score above -inf)
      const float lse2 = (nan ? m : lr) + __log2f(sum);
      const int n = r / s.G, h = x.hk * s.G + r - n * s.G;
      if (plan.split) {
        const int64_t row = ((int64_t)blockIdx.x + x.seg) * kFewRows + r;
        *reinterpret_cast<float2*>(a.part_o + row * D + ch) = make_float2(v0 * inv, v1 * inv);
        if (ch == 0) a.part_l[row] = lse2;
      } else {
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o.p) + x.b * a.o.sb + h * a.o.sh + (int64_t)n * a.o.sn + ch) =
            F16 ? pack_f16x2(v0 * inv, v1 * inv) : pack_bf16x2(v0 * inv, v1 * inv);
        if (ch == 0) a.lse[((int64_t)x.b * s.H + h) * s.N + n] = lse2 * 0.69314718055994531f;
      }
    }
    __syncthreads();  // before the next piece's copies
  }
}

template <int D, bool KV8, bool F16>
cudaError_t launch_t(const CrossShape& s, const FwdPlan& p, const KvRef& kv, const CrossFwdArgs& a, cudaStream_t st) {
  constexpr int kBytes = kWarps * kStages * kStageBytes;
  static_assert(kWarps * kFewRows * (D + 4) * 4 <= kBytes && kBytes + 1024 <= (int)kMaxDynSmem, "shared memory");
  auto kern = cross_few_kernel<D, KV8, F16>;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = allow_smem(kern, kBytes, allowed);
  if (e != cudaSuccess) return e;
  prof_start(st, kAttnFwd);
  kern<<<(unsigned)p.grid, kThreads, kBytes, st>>>(s, p, kv, a);
  prof_stop(st, kAttnFwd);
  e = cudaGetLastError();
  return e == cudaSuccess && p.split ? launch_cross_join(s, p, a, st) : e;
}

}  // namespace

cudaError_t launch_few_rows(const CrossShape& s, const FwdPlan& p, const TokenRef& k, const TokenRef& v,
                            const CacheRef& c, bool cache, const CrossFwdArgs& a, cudaStream_t st) {
  KvRef kv{};
  if (cache) {
    kv = {c.k, c.v, c.sb, c.sh, c.sn, c.sb, c.sh, c.sn, c.ks, c.vs, c.nsb};
  } else {
    kv = {static_cast<const uint8_t*>(k.p), static_cast<const uint8_t*>(v.p), 2 * k.sb, 2 * k.sh, 2 * k.sn,
          2 * v.sb, 2 * v.sh, 2 * v.sn, nullptr, nullptr, 0};
  }
  const bool f16 = s.dtype == SA2_FP16;
  if (s.d == 128) {
    if (cache) return f16 ? launch_t<128, true, true>(s, p, kv, a, st) : launch_t<128, true, false>(s, p, kv, a, st);
    return f16 ? launch_t<128, false, true>(s, p, kv, a, st) : launch_t<128, false, false>(s, p, kv, a, st);
  }
  if (cache) return f16 ? launch_t<64, true, true>(s, p, kv, a, st) : launch_t<64, true, false>(s, p, kv, a, st);
  return f16 ? launch_t<64, false, true>(s, p, kv, a, st) : launch_t<64, false, false>(s, p, kv, a, st);
}

}  // namespace sa2
