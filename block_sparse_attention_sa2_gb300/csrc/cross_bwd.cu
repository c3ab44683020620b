// Backward of cross attention on sm_103a (tcgen05 + TMEM + TMA):
//   P = exp(s - LSE), dP = dO V^T, D = rowsum(dO * O), dS = P (dP - D),
//   dV = P^T dO, dK = scale dS^T Q, dQ = scale dS K.
// Two kernels, one that walks the keys of a query tile (dQ) and one that walks the queries of a key
// block (dK, dV): every sum is made in one order, in TMEM or in a fixed order of parts, so the
// result does not depend on scheduling.  S and dP are computed in both: 7 products where one
// kernel would do 5, but that one would have to add dQ up across CTAs, in fp32 in memory: for
// 512 keys four times the size of dQ, written and read again, which costs more than 2 products.
// P and dS are rounded to bf16 for their products.  A query tile's rows are tokens x the G heads
// that share the key head, so that dK and dV of shared heads need no other sum.
#include "cross_sched.cuh"

namespace sa2 {
namespace {

constexpr uint32_t kTmemCols = 512;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

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

// ------------------------------------------------------------------------- statistics
//
// D and log2(e) * LSE of every query row: D / 16 threads per row, one row each, grid (query tiles,
// 128 / rows of a CTA).  Bound by the bytes of dO and O: 12 heads x 32760, d = 128: 33 us, 6.1 TB/s (with
// a whole tile per CTA, four rows per thread, 44: too few CTAs on an SM to cover the others' ends).
template <int D>
constexpr int kStatsRows = 256 / (D / 16);
template <int D>
__global__ void __launch_bounds__(256) cross_stats_kernel(CrossShape s, BwdPlan plan, CrossBwdArgs a) {
  constexpr int kLanes = D / 16;
  kernel_trigger();
  if (a.kv_len && blockIdx.x == 0 && blockIdx.y == 0)
    for (int b = threadIdx.x; b < s.B; b += 256)
      if (a.kv_len[b] < 0 || a.kv_len[b] > s.M) report_error(a.status, kDevErrBounds);
  const int head = blockIdx.x / plan.tiles, tile = blockIdx.x - head * plan.tiles;
  const int b = head / s.Hkv, hk = head - b * s.Hkv;
  const int ch = (threadIdx.x % kLanes) * 16;
  const int r = threadIdx.x / kLanes + blockIdx.y * kStatsRows<D>;
  const int tok_r = r / s.G, g = r - tok_r * s.G;
  const int n = tile * plan.nb + tok_r;
  uint4 x[2], y[2];
  x[0] = x[1] = y[0] = y[1] = make_uint4(0, 0, 0, 0);
  float lse = INFINITY;
  if (tok_r < plan.nb && n < s.N) {
    const uint4* px = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.dO.p) + b * a.dO.sb +
                                                     (int64_t)(hk * s.G + g) * a.dO.sh + n * a.dO.sn + ch);
    const uint4* py = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.o.p) + b * a.o.sb +
                                                     (int64_t)(hk * s.G + g) * a.o.sh + n * a.o.sn + ch);
    x[0] = __ldg(px);
    x[1] = __ldg(px + 1);
    y[0] = __ldg(py);
    y[1] = __ldg(py + 1);
    if (ch == 0) lse = a.lse[((int64_t)b * s.H + hk * s.G + g) * s.N + n];
  }
  float acc = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t xs[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    const uint32_t ys[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      acc = fmaf(__uint_as_float(xs[q] << 16), __uint_as_float(ys[q] << 16), acc);
      acc = fmaf(__uint_as_float(xs[q] & 0xFFFF0000u), __uint_as_float(ys[q] & 0xFFFF0000u), acc);
    }
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (ch == 0) {
    float* rec = a.stats + (int64_t)blockIdx.x * 256;
    rec[r] = lse * 1.4426950408889634f;
    rec[128 + r] = acc;
  }
}

// ------------------------------------------------------------------------------- dQ
//
// A work item is a query tile; its CTA walks the key blocks.  Per block j:
//   S_j = Q K_j^T, dP_j = dO V_j^T  (M = 128 rows, N = 128 keys), dS_j = P (dP - D) in bf16 over
//   dP_j's columns in TMEM, dQ += dS_j K_j.
// S_{j+1} needs only that the row threads have read S_j (dQ_{j-1} runs meanwhile), dP_{j+1} that
// dQ_{j-1} has completed (S_{j+1} runs meanwhile; dP has two buffers), and dQ_j has a whole period of
// three products for dS_j to be made in.
// Roles: warp 0 TMA; warps 1, 3 and 2 issuers of S, dP and dQ; 8 (d = 128) or 16 (d = 64) warps of row threads,
// two or four per row (d = 64, 19 heads x 8192 x 4096: two 254 us, four 188); 4 warps epilogue.
// TMEM columns: S 0, dP 128 and 256, dQ 384.
template <int D>
struct DqSmem {
  static constexpr int kRowWarps = D == 128 ? 8 : 16;
  static constexpr int kThreads = 32 * (4 + kRowWarps + 4);
  static constexpr int kPanels = D / 64;
  static constexpr int kTile = 128 * 128 * kPanels;
  static constexpr int kKStages = 3, kVStages = 2;
  static constexpr int kOffQ = 0, kOffDO = kTile;
  static constexpr int kOffK = 2 * kTile;
  static constexpr int kOffV = kOffK + kKStages * kTile;
  static constexpr int kOffBar = kOffV + kVStages * kTile;
  // at least 120 KB, so that one CTA (512 TMEM columns) has an SM to itself
  static constexpr int kBytes = (kOffBar + 512 + 1024) > 120 * 1024 ? (kOffBar + 512 + 1024) : 120 * 1024;
  static_assert(kBytes <= (int)kMaxDynSmem, "shared memory");
};

template <int D>
__global__ void __launch_bounds__(DqSmem<D>::kThreads, 1)
    cross_dq_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo, CrossShape s,
                    BwdPlan plan, CrossBwdArgs a) {
  using L = DqSmem<D>;
  constexpr int kKSt = L::kKStages, kVSt = L::kVStages;
  constexpr uint32_t kS = 0, kDP = 128, kDQ = 384;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  auto bar_kfull = [&](int st) { return smem_u32(&bars[st]); };
  auto bar_kempty = [&](int st) { return smem_u32(&bars[3 + st]); };
  auto bar_vfull = [&](int st) { return smem_u32(&bars[6 + st]); };
  auto bar_vempty = [&](int st) { return smem_u32(&bars[8 + st]); };
  const uint32_t bar_q = smem_u32(&bars[10]), bar_qfree = smem_u32(&bars[11]);    // Q landed / read
  const uint32_t bar_do = smem_u32(&bars[12]), bar_dofree = smem_u32(&bars[13]);  // dO
  const uint32_t bar_s = smem_u32(&bars[14]), bar_sfree = smem_u32(&bars[15]);    // S in TMEM / read out
  auto bar_dp = [&](int i) { return smem_u32(&bars[16 + i]); };    // dP buffer i in TMEM
  auto bar_ds = [&](int i) { return smem_u32(&bars[18 + i]); };    // dS written over it
  auto bar_dqm = [&](int i) { return smem_u32(&bars[20 + i]); };   // dQ += dS K from it completed
  const uint32_t bar_dq = smem_u32(&bars[22]), bar_dqfree = smem_u32(&bars[23]);  // dQ of the item complete / read
  const uint32_t bar_drain = smem_u32(&bars[24]), bar_gdrain = smem_u32(&bars[25]), bar_pdrain = smem_u32(&bars[26]);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffBar + 384);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffBar + 392);
  const WaitCtl wc{abort_flag, s.wait_ns};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < kKSt; ++i) {
      mbar_init(bar_kfull(i), 1);
      mbar_init(bar_kempty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_vfull(i), 1);
      mbar_init(bar_vempty(i), 1);
      mbar_init(bar_dp(i), 1);
      mbar_init(bar_ds(i), 32 * L::kRowWarps);
      mbar_init(bar_dqm(i), 1);
    }
    mbar_init(bar_q, 1);
    mbar_init(bar_qfree, 1);
    mbar_init(bar_do, 1);
    mbar_init(bar_dofree, 1);
    mbar_init(bar_s, 1);
    mbar_init(bar_sfree, 32 * L::kRowWarps);
    mbar_init(bar_dq, 1);
    mbar_init(bar_dqfree, 128);
    mbar_init(bar_drain, 1);
    mbar_init(bar_gdrain, 1);
    mbar_init(bar_pdrain, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  kernel_wait();
  const int64_t items = (int64_t)s.B * s.Hkv * plan.tiles;
  struct Item {
    int b, hk, tile, keys, nk;
  };
  auto item_at = [&](int64_t i) {
    Item x;
    const int64_t head = i / plan.tiles;
    x.tile = (int)(i - head * plan.tiles);
    x.b = (int)(head / s.Hkv);
    x.hk = (int)(head - (int64_t)x.b * s.Hkv);
    x.keys = key_count(a.kv_len, x.b, s.M);
    x.nk = key_blocks(x.keys);
    return x;
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint32_t q_bytes = (uint32_t)(L::kPanels * 128 * plan.nb * s.G);
      uint32_t J = 0, nv = 0, qn = 0, don = 0;  // K, V, Q and dO tiles loaded
      bool ok = true;
      for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
        const Item x = item_at(i);
        for (int j = 0; j < x.nk; ++j) {
          const int ks = J % kKSt, vs = nv % kVSt;
          if (J >= (uint32_t)kKSt && !mbar_wait(bar_kempty(ks), ((J / kKSt) - 1) & 1, wc)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar_kfull(ks), L::kTile);
          for (int p = 0; p < L::kPanels; ++p)
            tma_load_5d(sbase + L::kOffK + ks * L::kTile + p * 16384, &mk, bar_kfull(ks), p * 64, 0, j * kKeyBlock,
                        x.hk, x.b);
          ++J;
          if (j == 0) {
            if (qn >= 1 && !mbar_wait(bar_qfree, (qn - 1) & 1, wc)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(bar_q, q_bytes);
            for (int p = 0; p < L::kPanels; ++p)
              tma_load_5d(sbase + L::kOffQ + p * 16384, &mq, bar_q, p * 64, 0, x.tile * plan.nb, x.hk, x.b);
            ++qn;
            if (don >= 1 && !mbar_wait(bar_dofree, (don - 1) & 1, wc)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(bar_do, q_bytes);
            for (int p = 0; p < L::kPanels; ++p)
              tma_load_5d(sbase + L::kOffDO + p * 16384, &mdo, bar_do, p * 64, 0, x.tile * plan.nb, x.hk, x.b);
            ++don;
          }
          if (nv >= (uint32_t)kVSt && !mbar_wait(bar_vempty(vs), ((nv / kVSt) - 1) & 1, wc)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar_vfull(vs), L::kTile);
          for (int p = 0; p < L::kPanels; ++p)
            tma_load_5d(sbase + L::kOffV + vs * L::kTile + p * 16384, &mv, bar_vfull(vs), p * 64, 0, j * kKeyBlock,
                        x.hk, x.b);
          ++nv;
        }
      }
      for (uint32_t v = J > (uint32_t)kKSt ? J - kKSt : 0; v < J; ++v)
        mbar_drain(bar_kfull(v % kKSt), (v / kKSt) & 1, abort_flag);
      for (uint32_t v = nv > (uint32_t)kVSt ? nv - kVSt : 0; v < nv; ++v)
        mbar_drain(bar_vfull(v % kVSt), (v / kVSt) & 1, abort_flag);
      if (qn) mbar_drain(bar_q, (qn - 1) & 1, abort_flag);
      if (don) mbar_drain(bar_do, (don - 1) & 1, abort_flag);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ issuer of S
    const uint64_t qd = smem_desc(sbase + L::kOffQ, 16, 1024);
    bool ok = true;
    uint32_t J = 0, n = 0;  // blocks, items
    for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
      const Item x = item_at(i);
      for (int j = 0; j < x.nk; ++j, ++J) {
        const int ks = J % kKSt;
        const int steps = (min(kKeyBlock, x.keys - j * kKeyBlock) + 15) >> 4;
        const uint32_t idS = idesc_bf16_f32(128, steps * 16, false, false);
        ok = __all_sync(0xffffffffu, mbar_wait(bar_kfull(ks), (J / kKSt) & 1, wc) &&
                                         (j > 0 || mbar_wait(bar_q, n & 1, wc)) &&
                                         (J == 0 || mbar_wait(bar_sfree, (J - 1) & 1, wc)));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          issue_ss<D>(tmem + kS, qd, smem_desc(sbase + L::kOffK + ks * L::kTile, 16, 1024), idS);
          umma_commit(bar_s);
          if (j + 1 == x.nk) umma_commit(bar_qfree);
        }
        __syncwarp();
      }
      if (x.nk > 0) ++n;
    }
    if (elect_one()) umma_commit(bar_drain);
    __syncwarp();
    mbar_drain(bar_drain, 0, abort_flag);
  } else if (warp == 3) {
    // ------------------------------------------------------------------ issuer of dP
    const uint64_t dod = smem_desc(sbase + L::kOffDO, 16, 1024);
    bool ok = true;
    uint32_t J = 0, n = 0;
    for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
      const Item x = item_at(i);
      for (int j = 0; j < x.nk; ++j, ++J) {
        const int vs = J % kVSt, bb = J & 1;
        const int steps = (min(kKeyBlock, x.keys - j * kKeyBlock) + 15) >> 4;
        const uint32_t idS = idesc_bf16_f32(128, steps * 16, false, false);
        ok = __all_sync(0xffffffffu, mbar_wait(bar_vfull(vs), (J / kVSt) & 1, wc) &&
                                         (j > 0 || mbar_wait(bar_do, n & 1, wc)) &&
                                         (J < 2 || mbar_wait(bar_dqm(bb), ((J >> 1) - 1) & 1, wc)));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          issue_ss<D>(tmem + kDP + bb * 128, dod, smem_desc(sbase + L::kOffV + vs * L::kTile, 16, 1024), idS);
          umma_commit(bar_dp(bb));
          umma_commit(bar_vempty(vs));
          if (j + 1 == x.nk) umma_commit(bar_dofree);
        }
        __syncwarp();
      }
      if (x.nk > 0) ++n;
    }
    if (elect_one()) umma_commit(bar_pdrain);
    __syncwarp();
    mbar_drain(bar_pdrain, 0, abort_flag);
  } else if (warp == 2) {
    // ------------------------------------------------------------------ issuer of dQ
    constexpr uint32_t idQ = idesc_bf16_f32(128, D, false, true);
    bool ok = true;
    uint32_t J = 0, n = 0;
    for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
      const Item x = item_at(i);
      for (int j = 0; j < x.nk; ++j, ++J) {
        const int ks = J % kKSt, bb = J & 1;
        const int valid = min(kKeyBlock, x.keys - j * kKeyBlock), steps = (valid + 15) >> 4;
        ok = __all_sync(0xffffffffu, (j > 0 || n == 0 || mbar_wait(bar_dqfree, (n - 1) & 1, wc)) &&
                                         mbar_wait(bar_kfull(ks), (J / kKSt) & 1, wc) &&
                                         mbar_wait(bar_ds(bb), (J >> 1) & 1, wc));
        if (!ok) break;
        if (valid & 15) {
          // rows of K behind the last key, up to the next multiple of 16, as zeros: dS is 0 there, but
          // 0 * NaN is NaN.  S_j, which read them before, has completed (dS_j was made from it).
          const int rows = 16 * steps - valid, nz = rows * 8 * L::kPanels;
          uint8_t* kt = smem + L::kOffK + ks * L::kTile;
          for (int q = lane; q < nz; q += 32) {
            const int row = valid + (q >> 3) % rows, p = (q >> 3) / rows;
            *reinterpret_cast<uint4*>(kt + p * 16384 + row * 128 + (q & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async();
          __syncwarp();
        }
        tc_fence_after();
        const uint64_t kmn = smem_desc(sbase + L::kOffK + ks * L::kTile, 16384, 1024);
        if (elect_one()) {
          issue_ts(tmem + kDQ, tmem + kDP + bb * 128, kmn, idQ, steps, j == 0);
          umma_commit(bar_dqm(bb));
          umma_commit(bar_kempty(ks));
          if (j + 1 == x.nk) umma_commit(bar_dq);
        }
        __syncwarp();
      }
      if (x.nk > 0) ++n;
    }
    if (elect_one()) umma_commit(bar_gdrain);
    __syncwarp();
    mbar_drain(bar_gdrain, 0, abort_flag);
  } else if (warp >= 4 && warp < 4 + L::kRowWarps) {
    // ------------------------------------------------------------------ row threads
    if (s.stall_ns && blockIdx.x == 0) stall_for(s.stall_ns);  // failure-path test hook
    constexpr int kKeys = 512 / L::kRowWarps;  // of each block, for this thread
    const int k0 = kKeys * ((warp - 4) >> 2);
    const int r = 32 * (warp & 3) + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    bool ok = true;
    uint32_t J = 0;
    for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
      const Item x = item_at(i);
      if (x.nk == 0) continue;
      const float lse2 = a.stats[i * 256 + r], Dr = a.stats[i * 256 + 128 + r];
      for (int j = 0; j < x.nk; ++j, ++J) {
        const int bb = J & 1;
        const int valid = x.keys - j * kKeyBlock - k0;  // of this thread's keys
        if (!__all_sync(0xffffffffu, mbar_wait(bar_s, J & 1, wc))) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t u[kKeys / 32][32];
        float p[kKeys];
#pragma unroll
        for (int h = 0; h < kKeys / 32; ++h) tmem_ld32(trow + kS + k0 + 32 * h, u[h]);
#pragma unroll
        for (int h = 0; h < kKeys / 32; ++h) tmem_ld_wait(u[h]);
        tc_fence_before();
        mbar_arrive(bar_sfree);
#pragma unroll
        for (int c = 0; c < kKeys; ++c) p[c] = ex2(fmaf(__uint_as_float(u[c >> 5][c & 31]), a.scale_log2, -lse2));
        if (!__all_sync(0xffffffffu, mbar_wait(bar_dp(bb), (J >> 1) & 1, wc))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t tdp = trow + kDP + bb * 128 + k0;
#pragma unroll
        for (int h = 0; h < kKeys / 32; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t v[16];
            tmem_ld16(tdp + 32 * h + 16 * q, v);
            tmem_ld_wait16(v);
#pragma unroll
            for (int c = 0; c < 16; c += 2) {
              const int k = 32 * h + 16 * q + c;
              const float d0 = p[k] * (__uint_as_float(v[c]) - Dr), d1 = p[k + 1] * (__uint_as_float(v[c + 1]) - Dr);
              pk[(16 * q + c) / 2] = pack_bf16x2(d0, d1);
            }
          }
          if (valid < 32 * (h + 1)) {  // behind the last key dP may be anything
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const int left = valid - 32 * h - 2 * c;
              pk[c] = left > 1 ? pk[c] : (left > 0 ? pk[c] & 0xFFFFu : 0u);
            }
          }
          tmem_st16(tdp + 32 * h, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar_ds(bb));
      }
    }
  } else if (warp >= 4 + L::kRowWarps) {
    // ------------------------------------------------------------------ epilogue
    const int r = 32 * (warp & 3) + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const int tok_r = r / s.G, gq = r - tok_r * s.G;
    bool ok = true;
    uint32_t n = 0;
    for (int64_t i = blockIdx.x; ok && i < items; i += gridDim.x) {
      const Item x = item_at(i);
      const int tok = x.tile * plan.nb + tok_r;
      const bool row_valid = tok_r < plan.nb && tok < s.N;
      uint16_t* row = static_cast<uint16_t*>(a.dq.p) + x.b * a.dq.sb + (int64_t)(x.hk * s.G + gq) * a.dq.sh +
                      (int64_t)tok * a.dq.sn;
      if (x.nk == 0) {
        if (row_valid)
          for (int c = 0; c < D / 8; ++c) reinterpret_cast<uint4*>(row)[c] = make_uint4(0, 0, 0, 0);
        continue;
      }
      if (!__all_sync(0xffffffffu, mbar_wait(bar_dq, n & 1, wc))) {
        ok = false;
        break;
      }
      ++n;
      tc_fence_after();
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t u[32];
        tmem_ld32(trow + kDQ + c0, u);
        tmem_ld_wait(u);
        if (c0 + 32 >= D) {
          tc_fence_before();
          mbar_arrive(bar_dqfree);
        }
        float v[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c] = __uint_as_float(u[c]) * a.scale;
        if (row_valid) store32_bf16(row + c0, v);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) report_error(a.status, kDevErrTimeout);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// --------------------------------------------------------------------------- dK, dV
//
// A CTA holds a block of 128 keys and walks query tiles, a half tile of 64 rows at a time.  The products
// are formed transposed, keys along the TMEM lanes, so that P^T and dS^T go from the element-wise threads
// to the next product through TMEM.  Per half tile, in its buffer (two at d = 128, three at d = 64):
//   S^T = K Q^T, dP^T = V dO^T  (M = 128 keys, N = 64 rows),  dV += P^T dO, dK += dS^T Q  (K = 64).
// P^T is written over S^T and dS^T over dP^T; S^T and dP^T of a half tile wait for dV and dK of the one that
// had the buffer, those between are made meanwhile.  (With whole tiles TMEM has room for one S^T and dP^T,
// and S, P, dV, S are one chain: 19 heads x 8192 x 4096, d = 128: 485 us, half tiles 441.)
// LSE and D belong to TMEM columns here, and every element-wise thread needs all of them: from shared memory
// 32 cycles of its 128 bytes per clock for each warp and 32 values, 1000 cycles per tile beside the products'
// reads.  At d = 64 they come through the products instead: 16 more channels, K and V with ones in three of
// them, Q with -LSE / scale and dO with -D as three bf16 each, so that S^T is s - LSE (in units of the
// scale) and dP^T is dP - D, in fp32, for one more step of 48 cycles: the same shape at d = 64 takes 269
// us, 314 with loads.  At d = 128, where the products take three quarters of the time, 488 against 441.
// Roles: warp 0 TMA; warps 1, 3 and 2 issuers of S, of dP, and of dV and dK (a wait and its bookkeeping take
// an issuer 200 to 400 cycles beside the element-wise warps); warps 4..19 element-wise: two sets of 8 warps
// take half tiles in turn, so that one's latencies fall into the other's work; thread = key, two per key:
// rows 0..31 and 32..63; warp 20 (d = 64) writes the 16 channels.
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

template <int D>
struct DkvSmem {
  static constexpr bool kX = D == 64;  // LSE and D through the products
  static constexpr int kThreads = kX ? 672 : 640;
  static constexpr int kPanels = D / 64;
  static constexpr int kTile = 128 * 128 * kPanels;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kOffK = 0, kOffV = kTile;
  static constexpr int kOffStage = 2 * kTile;  // Q, dO, statistics
  static constexpr int kStageQ = 0, kStageDO = kTile, kStageX = 2 * kTile;
  static constexpr int kStageStats = kStageX + (kX ? 2 * kXTile : 0);
  static constexpr int kStage = kStageStats + 1024;
  static constexpr int kOffOnes = kOffStage + kStages * kStage;
  static constexpr int kOffBar = kOffOnes + (kX ? kXTile : 0);
  static constexpr int kBytes = kOffBar + 512 + 1024;
  static_assert(kBytes <= (int)kMaxDynSmem && kBytes > 114 * 1024, "shared memory: one CTA per SM");
};

// The pieces of a CTA's run: key block kb of head (b, hk), query tiles [t0, t0 + nt).
struct DkvPiece {
  int b, hk, kb, keys, t0, nt;
  bool whole;
  int slot;
};
// Parts that every key block's tiles are cut into, one per CTA, where that leaves less than a tenth of
// the CTAs without work; 0: equal runs.  With parts, the key blocks of a head read the same tiles at
// the same time, and all but the first find them in L2 (512 keys, 12 heads of 32760 queries: DRAM
// traffic 805 -> 201 MB).
__device__ __forceinline__ int dkv_parts(int64_t segs, int tiles, int grid) {
  if (segs == 0 || segs > grid) return 0;
  const int64_t parts = min((int64_t)tiles, grid / segs);
  return parts * segs * 10 >= (int64_t)grid * 9 ? (int)parts : 0;
}

struct DkvIter {
  const CrossShape& s;
  const BwdPlan& p;
  const int32_t* kv_len;
  int64_t g, g_begin, g_end, base;
  int b;
  // (whole warps)
  __device__ __forceinline__ DkvIter(const CrossShape& s_, const BwdPlan& p_, const int32_t* l)
      : s(s_), p(p_), kv_len(l), base(0), b(0) {
    const int64_t segs = total_key_blocks(s, kv_len, 1), total = segs * p.tiles;
    const int parts = dkv_parts(segs, p.tiles, p.grid);
    if (parts) {
      // part i of segment blockIdx.x % segs, so that a head's key blocks are neighbours
      const int64_t seg = blockIdx.x % segs;
      const int i = (int)(blockIdx.x / segs);
      g = seg * p.tiles + (int64_t)i * p.tiles / parts;
      g_end = i < parts ? seg * p.tiles + (int64_t)(i + 1) * p.tiles / parts : g;
    } else {
      const int64_t run = run_length(total, p.grid);
      g = run * blockIdx.x;
      g_end = g + run < total ? g + run : total;
    }
    g_begin = g;
  }
  __device__ __forceinline__ bool next(DkvPiece& x) {
    if (g >= g_end) return false;
    int64_t nk = key_blocks(key_count(kv_len, b, s.M));
    while (g >= base + nk * s.Hkv * p.tiles) {
      base += nk * s.Hkv * p.tiles;
      ++b;
      nk = key_blocks(key_count(kv_len, b, s.M));
    }
    const int64_t off = g - base, seg = off / p.tiles;
    x.b = b;
    x.keys = key_count(kv_len, b, s.M);
    x.hk = (int)(seg / nk);
    x.kb = (int)(seg - x.hk * nk);
    x.t0 = (int)(off - seg * p.tiles);
    const int64_t left = g_end - g;
    x.nt = p.tiles - x.t0 < left ? p.tiles - x.t0 : (int)left;
    x.whole = x.nt == p.tiles;
    x.slot = 2 * blockIdx.x + (g == g_begin ? 0 : 1);
    g += x.nt;
    return true;
  }
};

template <int D>
__global__ void __launch_bounds__(DkvSmem<D>::kThreads, 1)
    cross_dkdv_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo, CrossShape s,
                      BwdPlan plan, CrossBwdArgs a) {
  using L = DkvSmem<D>;
  constexpr int kStages = L::kStages;
  constexpr uint32_t kBufs = D == 128 ? 2 : 3;  // of S^T and dP^T, 64 columns each
  constexpr uint32_t kS = 0, kDP = 64 * kBufs, kDV = 2 * kDP, kDK = kDV + D;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  auto bar_full = [&](int st) { return smem_u32(&bars[st]); };
  auto bar_empty = [&](int st) { return smem_u32(&bars[4 + st]); };
  const uint32_t bar_kv = smem_u32(&bars[8]), bar_kvfree = smem_u32(&bars[9]);
  auto bar_s = [&](uint32_t b) { return smem_u32(&bars[10 + b]); };    // S^T, dP^T in TMEM buffer b
  auto bar_dp = [&](uint32_t b) { return smem_u32(&bars[13 + b]); };
  auto bar_p = [&](uint32_t b) { return smem_u32(&bars[16 + b]); };    // P^T, dS^T written over them
  auto bar_ds = [&](uint32_t b) { return smem_u32(&bars[19 + b]); };
  auto bar_dvm = [&](uint32_t b) { return smem_u32(&bars[22 + b]); };  // dV, dK products from them completed
  auto bar_dkm = [&](uint32_t b) { return smem_u32(&bars[25 + b]); };
  const uint32_t bar_acc = smem_u32(&bars[28]), bar_accfree = smem_u32(&bars[29]);  // the piece's sums complete / read
  const uint32_t bar_drain = smem_u32(&bars[30]), bar_gdrain = smem_u32(&bars[31]), bar_pdrain = smem_u32(&bars[32]);
  auto bar_x = [&](int st) { return smem_u32(&bars[33 + st]); };  // the 16 channels written
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffBar + 384);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffBar + 392);
  const WaitCtl wc{abort_flag, s.wait_ns};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // Tile rows that hold no query (128 is not a multiple of G) are never loaded: zeros, since their
  // P and dS are 0 but 0 * NaN is NaN.
  const int used = plan.nb * s.G;
  if (used < 128) {
    const int n = (128 - used) * 8 * L::kPanels * 2 * kStages;
    for (int i = tid; i < n; i += L::kThreads) {
      const int row = used + (i >> 3) % (128 - used);
      int x = (i >> 3) / (128 - used);
      const int p = x % L::kPanels;
      x /= L::kPanels;
      uint8_t* t = smem + L::kOffStage + (x >> 1) * L::kStage + ((x & 1) ? L::kStageDO : L::kStageQ);
      *reinterpret_cast<uint4*>(t + p * 16384 + row * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
  }
  for (int i = tid; L::kX && i < (2 * kStages + 1) * (kXTile / 16); i += L::kThreads) {
    const int x = i / (kXTile / 16), at = (i % (kXTile / 16)) * 16;
    const bool ones = x == 2 * kStages && !(at & 128);
    uint8_t* tile = x == 2 * kStages ? smem + L::kOffOnes
                                     : smem + L::kOffStage + (x >> 1) * L::kStage + L::kStageX + (x & 1) * kXTile;
    *reinterpret_cast<uint4*>(tile + at) = ones ? make_uint4(0x3F803F80u, 0x3F80u, 0, 0) : make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async();
  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar_full(i), 1);
      mbar_init(bar_empty(i), 1);
      mbar_init(bar_x(i), 1);
    }
    mbar_init(bar_kv, 1);
    mbar_init(bar_kvfree, 2);
    for (uint32_t b = 0; b < kBufs; ++b) {
      mbar_init(bar_s(b), 1);
      mbar_init(bar_dp(b), 1);
      mbar_init(bar_p(b), 256);
      mbar_init(bar_ds(b), 256);
      mbar_init(bar_dvm(b), 1);
      mbar_init(bar_dkm(b), 1);
    }
    mbar_init(bar_acc, 1);
    mbar_init(bar_accfree, 512);
    mbar_init(bar_drain, 1);
    mbar_init(bar_gdrain, 1);
    mbar_init(bar_pdrain, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  kernel_trigger();
  kernel_wait();

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    DkvIter it(s, plan, a.kv_len);
    if (lane == 0) {
      const uint32_t q_bytes = (uint32_t)(L::kPanels * 128 * used);
      uint32_t U = 0, n = 0;
      bool ok = true;
      DkvPiece x;
      while (ok && it.next(x)) {
        if (n >= 1 && !mbar_wait(bar_kvfree, (n - 1) & 1, wc)) break;
        mbar_arrive_expect_tx(bar_kv, 2 * L::kTile);
        for (int p = 0; p < L::kPanels; ++p) {
          tma_load_5d(sbase + L::kOffK + p * 16384, &mk, bar_kv, p * 64, 0, x.kb * kKeyBlock, x.hk, x.b);
          tma_load_5d(sbase + L::kOffV + p * 16384, &mv, bar_kv, p * 64, 0, x.kb * kKeyBlock, x.hk, x.b);
        }
        ++n;
        for (int t = x.t0; t < x.t0 + x.nt; ++t, ++U) {
          const int st = U % kStages;
          if (U >= (uint32_t)kStages && !mbar_wait(bar_empty(st), ((U / kStages) - 1) & 1, wc)) {
            ok = false;
            break;
          }
          const uint32_t stg = sbase + L::kOffStage + st * L::kStage;
          mbar_arrive_expect_tx(bar_full(st), 2 * q_bytes + 1024);
          for (int p = 0; p < L::kPanels; ++p) {
            tma_load_5d(stg + L::kStageQ + p * 16384, &mq, bar_full(st), p * 64, 0, t * plan.nb, x.hk, x.b);
            tma_load_5d(stg + L::kStageDO + p * 16384, &mdo, bar_full(st), p * 64, 0, t * plan.nb, x.hk, x.b);
          }
          bulk_load(stg + L::kStageStats, a.stats + (((int64_t)x.b * s.Hkv + x.hk) * plan.tiles + t) * 256, 1024,
                    bar_full(st));
        }
      }
      for (uint32_t v = U > (uint32_t)kStages ? U - kStages : 0; v < U; ++v)
        mbar_drain(bar_full(v % kStages), (v / kStages) & 1, abort_flag);
      if (n) mbar_drain(bar_kv, (n - 1) & 1, abort_flag);
    }
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------------------ issuers of S^T and of dP^T
    DkvIter it(s, plan, a.kv_len);
    constexpr uint32_t idS = idesc_bf16_f32(128, 64, false, false);
    const bool dp = warp == 3;
    const uint64_t akd = smem_desc(sbase + (dp ? L::kOffV : L::kOffK), 16, 1024);
    const uint32_t bst = sbase + L::kOffStage + (dp ? L::kStageDO : L::kStageQ);
    const uint32_t xst = sbase + L::kOffStage + L::kStageX + (dp ? kXTile : 0);
    const uint32_t dst = tmem + (dp ? kDP : kS), done = dp ? bar_dp(0) : bar_s(0), freed = dp ? bar_dkm(0) : bar_dvm(0);
    bool ok = true;
    uint32_t u = 0, n = 0;  // half tiles, pieces
    DkvPiece x;
    while (ok && it.next(x)) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar_kv, n & 1, wc));
      for (int i = 0; ok && i < 2 * x.nt; ++i, ++u) {
        const uint32_t U = u >> 1, st = U % kStages, half = u & 1, b = u % kBufs;
        ok = __all_sync(0xffffffffu, (half || (mbar_wait(bar_full(st), (U / kStages) & 1, wc) &&
                                                   (!L::kX || mbar_wait(bar_x(st), (U / kStages) & 1, wc)))) &&
                                         (u < kBufs || mbar_wait(freed + 8 * b, (u / kBufs - 1) & 1, wc)));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          issue_ss<D>(dst + 64 * b, akd, smem_desc(bst + st * L::kStage + half * 8192, 16, 1024), idS);
          if constexpr (L::kX)
            umma_ss(dst + 64 * b, x_desc(sbase + L::kOffOnes), x_desc(xst + st * L::kStage + half * (kXTile / 2)), idS, 1u);
          umma_commit(done + 8 * b);
          if (i + 1 == 2 * x.nt) umma_commit(bar_kvfree);
        }
        __syncwarp();
      }
      ++n;
    }
    if (elect_one()) umma_commit(dp ? bar_pdrain : bar_drain);
    __syncwarp();
    mbar_drain(dp ? bar_pdrain : bar_drain, 0, abort_flag);
  } else if (warp == 2) {
    // ------------------------------------------------------------------ issuer of dV and dK
    DkvIter it(s, plan, a.kv_len);
    constexpr uint32_t idG = idesc_bf16_f32(128, D, false, true);
    bool ok = true;
    uint32_t u = 0, n = 0;
    DkvPiece x;
    while (ok && it.next(x)) {
      for (int i = 0; ok && i < 2 * x.nt; ++i, ++u) {
        const uint32_t U = u >> 1, st = U % kStages, half = u & 1, b = u % kBufs, use = (u / kBufs) & 1;
        const uint32_t stg = sbase + L::kOffStage + st * L::kStage + half * 8192;  // rows 64 .. of each panel
        ok = __all_sync(0xffffffffu, (i > 0 || n == 0 || mbar_wait(bar_accfree, (n - 1) & 1, wc)) &&
                                         (half || mbar_wait(bar_full(st), (U / kStages) & 1, wc)) &&
                                         mbar_wait(bar_p(b), use, wc));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          issue_ts(tmem + kDV, tmem + kS + 64 * b, smem_desc(stg + L::kStageDO, 16384, 1024), idG, 4, i == 0);
          umma_commit(bar_dvm(b));
        }
        __syncwarp();
        ok = __all_sync(0xffffffffu, mbar_wait(bar_ds(b), use, wc));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          issue_ts(tmem + kDK, tmem + kDP + 64 * b, smem_desc(stg + L::kStageQ, 16384, 1024), idG, 4, i == 0);
          umma_commit(bar_dkm(b));
          if (half) umma_commit(bar_empty(st));
          if (i + 1 == 2 * x.nt) umma_commit(bar_acc);
        }
        __syncwarp();
      }
      ++n;
    }
    if (elect_one()) umma_commit(bar_gdrain);
    __syncwarp();
    mbar_drain(bar_gdrain, 0, abort_flag);
  } else if (L::kX && warp == 20) {
    // ------------------------------------------------------------- the 16 channels of LSE and D
    DkvIter it(s, plan, a.kv_len);
    const float inv = -1.f / fmaxf(a.scale_log2, kMinScale);
    uint32_t U = 0;
    bool ok = true;
    DkvPiece x;
    while (ok && it.next(x)) {
      for (int t = 0; t < x.nt; ++t, ++U) {
        const int st = U % kStages;
        uint8_t* stg = smem + L::kOffStage + st * L::kStage;
        ok = __all_sync(0xffffffffu, mbar_wait(bar_full(st), (U / kStages) & 1, wc));
        if (!ok) break;
        const float* rec = reinterpret_cast<const float*>(stg + L::kStageStats);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 32 * i + lane;
          *reinterpret_cast<uint2*>(stg + L::kStageX + x_row(r)) = split3(rec[r] * inv);
          *reinterpret_cast<uint2*>(stg + L::kStageX + kXTile + x_row(r)) = split3(-rec[128 + r]);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_x(st));
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------- element-wise threads
    if (s.stall_ns && blockIdx.x == 0) stall_for(s.stall_ns);  // failure-path test hook
    DkvIter it(s, plan, a.kv_len);
    const uint32_t half = (uint32_t)(warp - 4) >> 3;  // of every tile
    const int g = ((warp - 4) >> 2) & 1;           // rows 32 g .. 32 g + 31 of the half tile
    const int r = 32 * (warp & 3) + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const float mul = L::kX ? fmaxf(a.scale_log2, kMinScale) : a.scale_log2;
    const uint32_t ts0 = trow + kS + 32 * g + (kBufs == 2 ? 64 * half : 0);
    bool ok = true;
    uint32_t U = 0, n = 0;  // tiles, pieces
    DkvPiece x;
    while (ok && it.next(x)) {
      for (int t = 0; t < x.nt; ++t, ++U) {
        const uint32_t u = 2 * U + half, b = kBufs == 2 ? half : u % kBufs, use = (kBufs == 2 ? U : u / kBufs) & 1;
        const uint32_t ts = kBufs == 2 ? ts0 : ts0 + 64 * b, tdp = ts + kDP - kS;
        const int st = U % kStages;
        const float4* l4 = reinterpret_cast<const float4*>(smem + L::kOffStage + st * L::kStage + L::kStageStats) +
                           16 * half + 8 * g;
        const float4* d4 = l4 + 32;
        if (!__all_sync(0xffffffffu, (L::kX || mbar_wait(bar_full(st), (U / kStages) & 1, wc)) && mbar_wait(bar_s(b), use, wc))) {
          ok = false;
          break;
        }
        tc_fence_after();
        float p[32];
        uint32_t v[32], pk[16];
        tmem_ld32(ts, v);
        tmem_ld_wait(v);
        if constexpr (L::kX) {
#pragma unroll
          for (int c = 0; c < 32; ++c) p[c] = ex2(__uint_as_float(v[c]) * mul);
#pragma unroll
          for (int c = 0; c < 16; ++c) pk[c] = pack_bf16x2(p[2 * c], p[2 * c + 1]);
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float4 l = l4[q];
            float* pp = p + 4 * q;
            pp[0] = ex2(fmaf(__uint_as_float(v[4 * q]), mul, -l.x));
            pp[1] = ex2(fmaf(__uint_as_float(v[4 * q + 1]), mul, -l.y));
            pp[2] = ex2(fmaf(__uint_as_float(v[4 * q + 2]), mul, -l.z));
            pp[3] = ex2(fmaf(__uint_as_float(v[4 * q + 3]), mul, -l.w));
            pk[2 * q] = pack_bf16x2(pp[0], pp[1]);
            pk[2 * q + 1] = pack_bf16x2(pp[2], pp[3]);
          }
        }
        tmem_st16(ts, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar_p(b));
        if (!__all_sync(0xffffffffu, mbar_wait(bar_dp(b), use, wc))) {
          ok = false;
          break;
        }
        tc_fence_after();
        tmem_ld32(tdp, v);
        tmem_ld_wait(v);
        if constexpr (L::kX) {
#pragma unroll
          for (int c = 0; c < 16; ++c)
            pk[c] = pack_bf16x2(p[2 * c] * __uint_as_float(v[2 * c]), p[2 * c + 1] * __uint_as_float(v[2 * c + 1]));
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float4 d = d4[q];
            const float* pp = p + 4 * q;
            pk[2 * q] = pack_bf16x2(pp[0] * (__uint_as_float(v[4 * q]) - d.x), pp[1] * (__uint_as_float(v[4 * q + 1]) - d.y));
            pk[2 * q + 1] =
                pack_bf16x2(pp[2] * (__uint_as_float(v[4 * q + 2]) - d.z), pp[3] * (__uint_as_float(v[4 * q + 3]) - d.w));
          }
        }
        tmem_st16(tdp, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar_ds(b));
      }
      if (!ok) break;
      // ---- the piece's sums: thread = key, a quarter of the channels
      if (!__all_sync(0xffffffffu, mbar_wait(bar_acc, n & 1, wc))) {
        ok = false;
        break;
      }
      ++n;
      tc_fence_after();
      const int key = x.kb * kKeyBlock + r, quarter = 2 * (int)half + g;
      const bool live = key < x.keys, store = key < s.M;
#pragma unroll 1
      for (int w = 0; w < 2; ++w) {  // dK, dV
        const TokenRef& out = w ? a.dv : a.dk;
        const float mul = w ? 1.f : a.scale;
        uint16_t* row = static_cast<uint16_t*>(out.p) + x.b * out.sb + (int64_t)x.hk * out.sh + (int64_t)key * out.sn;
        float* part = a.part + (((int64_t)x.slot * 2 + w) * 128 + r) * D;
#pragma unroll
        for (int c0 = 0; c0 < D / 4; c0 += 16) {
          const int ch = quarter * (D / 4) + c0;
          uint32_t z[16];
          tmem_ld16(trow + (w ? kDV : kDK) + ch, z);
          tmem_ld_wait16(z);
          float f[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) f[c] = live ? __uint_as_float(z[c]) * mul : 0.f;
          if (!x.whole) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              reinterpret_cast<float4*>(part + ch)[c] = make_float4(f[4 * c], f[4 * c + 1], f[4 * c + 2], f[4 * c + 3]);
          } else if (store) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
              reinterpret_cast<uint4*>(row + ch)[c] =
                  make_uint4(pack_bf16x2(f[8 * c], f[8 * c + 1]), pack_bf16x2(f[8 * c + 2], f[8 * c + 3]),
                             pack_bf16x2(f[8 * c + 4], f[8 * c + 5]), pack_bf16x2(f[8 * c + 6], f[8 * c + 7]));
          }
        }
      }
      tc_fence_before();
      mbar_arrive(bar_accfree);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) report_error(a.status, kDevErrTimeout);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Adds the parts of key blocks whose tiles several runs shared, in run order, and writes zeros
// behind the last key block of each sequence.  Grid (B * Hkv * key blocks of M, 8): an eighth of a block
// each, since a head has few (12 heads x 32760 x 512: the whole backward 314 us, with one CTA per block 322).
constexpr int kJoinParts = 8;
template <int D>
__global__ void __launch_bounds__(256) cross_dkdv_join_kernel(CrossShape s, BwdPlan plan, CrossBwdArgs a) {
  kernel_trigger();
  const int head = blockIdx.x / plan.kblocks, kb = blockIdx.x - head * plan.kblocks, lane = threadIdx.x & 31;
  const int b = head / s.Hkv, hk = head - b * s.Hkv;
  const int keys = key_count(a.kv_len, b, s.M), nk = key_blocks(keys);
  // the parts: slots first, first + step, ... of CTAs; the part that a run begins with is in 2 * CTA
  int c0 = 0, count = 0, step = 1;
  int64_t g0 = 0, run = 0;
  if (kb < nk) {
    const int64_t segs = total_key_blocks(s, a.kv_len, 1);
    int64_t before = 0;
    for (int i = lane; i < b; i += 32) before += key_blocks(key_count(a.kv_len, i, s.M));
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    const int64_t seg = before * s.Hkv + (int64_t)hk * nk + kb;
    const int parts = dkv_parts(segs, plan.tiles, plan.grid);
    if (parts) {
      c0 = (int)seg;
      count = parts;
      step = (int)segs;
    } else {
      run = run_length(segs * plan.tiles, plan.grid);
      g0 = seg * plan.tiles;
      c0 = (int)(g0 / run);
      count = (int)((g0 + plan.tiles - 1) / run) - c0 + 1;
    }
  }
  kernel_wait();  // (by every CTA: the dQ kernel waits for this one alone)
  if (count == 1) return;  // one CTA had all of its tiles
  constexpr int kItems = 2 * 128 * (D / 8) / kJoinParts;
  for (int j = threadIdx.x; j < kItems; j += 256) {
    const int i = blockIdx.y * kItems + j;
    const int w = i / (128 * (D / 8)), r = i / (D / 8) % 128, ch = i % (D / 8) * 8;
    const int key = kb * kKeyBlock + r;
    if (key >= s.M) continue;
    float v[8] = {};
    if (key < keys) {
      for (int k = 0; k < count; ++k) {
        const int c = c0 + k * step;
        const int slot = 2 * c + (run * c >= g0 ? 0 : 1);  // the part begins with the run, or inside it
        const float4* p = reinterpret_cast<const float4*>(a.part + (((int64_t)slot * 2 + w) * 128 + r) * D + ch);
        const float4 x = p[0], y = p[1];
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
      }
    }
    const TokenRef& out = w ? a.dv : a.dk;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out.p) + b * out.sb + hk * out.sh + key * out.sn + ch) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}

template <int D>
cudaError_t launch_t(const CrossShape& s, const BwdPlan& p, const CUtensorMap& mq, const CUtensorMap& mk,
                     const CUtensorMap& mv, const CUtensorMap& mdo, const CrossBwdArgs& a, cudaStream_t st) {
  auto dq = cross_dq_kernel<D>;
  auto dkv = cross_dkdv_kernel<D>;
  static std::atomic<unsigned long long> dq_allowed{0}, dkv_allowed{0};
  cudaError_t e = allow_smem(dq, DqSmem<D>::kBytes, dq_allowed);
  if (e == cudaSuccess) e = allow_smem(dkv, DkvSmem<D>::kBytes, dkv_allowed);
  if (e != cudaSuccess) return e;
  prof_start(st, kBwdPre);
  cross_stats_kernel<D><<<dim3((unsigned)((int64_t)s.B * s.Hkv * p.tiles), 128 / kStatsRows<D>), 256, 0, st>>>(s, p, a);
  prof_stop(st, kBwdPre);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  prof_start(st, kAttnBwd);
  e = launch_early(dkv, dim3((unsigned)p.grid), DkvSmem<D>::kThreads, DkvSmem<D>::kBytes, st, mq, mk, mv, mdo, s, p, a);
  if (e == cudaSuccess)
    e = launch_early(cross_dkdv_join_kernel<D>, dim3((unsigned)((int64_t)s.B * s.Hkv * p.kblocks), kJoinParts), 256,
                     0, st, s, p, a);
  prof_stop(st, kAttnBwd);
  if (e != cudaSuccess) return e;
  prof_start(st, kAttnBwdDq);
  e = launch_early(dq, dim3((unsigned)p.dq_grid), DqSmem<D>::kThreads, DqSmem<D>::kBytes, st, mq, mk, mv, mdo, s, p, a);
  prof_stop(st, kAttnBwdDq);
  return e;
}

}  // namespace

BwdPlan cross_bwd_plan(const CrossShape& s, int sms) {
  BwdPlan p;
  p.nb = 128 / s.G;
  p.tiles = (s.N + p.nb - 1) / p.nb;
  p.kblocks = (s.M + kKeyBlock - 1) / kKeyBlock;
  const int64_t heads = (int64_t)s.B * s.Hkv;
  p.dq_grid = (int)(heads * p.tiles < sms ? heads * p.tiles : sms);
  const int64_t work = heads * p.kblocks * p.tiles;
  p.grid = (int)(work < sms ? work : sms);
  return p;
}

size_t cross_bwd_floats(const CrossShape& s, const BwdPlan& p, size_t* stats) {
  *stats = (size_t)s.B * s.Hkv * p.tiles * 256;
  return *stats + (size_t)2 * p.grid * 2 * 128 * s.d;
}

cudaError_t launch_cross_bwd(const CrossShape& s, const BwdPlan& p, const CUtensorMap& mq, const CUtensorMap& mk,
                             const CUtensorMap& mv, const CUtensorMap& mdo, const CrossBwdArgs& a, cudaStream_t st) {
  return s.d == 128 ? launch_t<128>(s, p, mq, mk, mv, mdo, a, st) : launch_t<64>(s, p, mq, mk, mv, mdo, a, st);
}

}  // namespace sa2
