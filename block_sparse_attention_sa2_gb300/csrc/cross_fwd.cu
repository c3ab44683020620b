// Attention of queries to keys of another length, forward, on sm_103a (tcgen05 + TMEM): over
// 16-bit keys and values (cross attention) and over the 8-bit cache.
//
//   s = scale * q k^T,  O = softmax(s) V,  LSE = log sum exp(s)
//
// One CTA per SM works on a pair of query tiles (2 x 128 rows) at a time, so that each key block
// that reaches shared memory feeds twice the matrix work and one tile's softmax runs beside the
// other's products.  A tile's rows are the tokens of all G query heads that share the key head
// (row = token * G + head), which lets few tokens of many heads fill a tile.
//
// Roles (544 threads): warp 0 TMA producer (Q tiles, a ring of K and V blocks of 128 keys); warps 1 and
// 2 issuers of S of tile 0 and 1, warps 3 and 16 of their P V (an issuer's waits and bookkeeping take 200
// to 400 cycles beside the softmax warps: with S and P V of a tile in one warp they were the bound, 12
// heads x 32760 x 512, d = 128: 106 us, apart 98); warps 4..7 epilogue (16-bit keys) or converters
// (8-bit keys: from blocks as they lie in the cache to fp16 in the ring, and Q to fp16); warps 8..11 and
// 12..15 the softmax of tile 0 and 1, one row per thread.
// A tile goes through its keys in half blocks of 64, with two S buffers:
//   S_t(i) = Q_t K_i^T   M = 128, N = 64, K = d   (shared memory, K-major)
//   O_t   += P_t(i) V_i  M = 128, N = d, K = 64   (A = P from TMEM, written over S_t(i); V MN-major)
// S_t(i+1) is made while the softmax of S_t(i) runs, once P_t(i-1) V, which read its columns, has
// completed.  With blocks of 128 keys TMEM has room for one S per tile only, and S, softmax and P V
// are one chain: 3300 to 5000 cycles per 128 keys and tile pair, by how the two tiles happened to fall
// in step, against 2560 of shared-memory reads for the products here.
// Bound now: d = 128 by the products and, in long runs, the power limit (24 heads x 8192 x 4096: 313 us, 1310
// TFLOP/s at 1350 W); d = 64 by the softmax threads (1370 cycles per half block, two of them per scheduler,
// most of it latency; the exponentials are 512 of them: without them it is no faster).
//
// The last block of a sequence may be partial.  Its products run over the valid keys rounded up
// to 16; scores behind the last key are replaced by -inf (whatever they are: NaN too), and up to
// 15 rows of V behind it are zeroed in shared memory, since 0 * NaN is NaN.
#include <algorithm>
#include <cuda_fp8.h>

#include "cross_sched.cuh"
#include "cross_softmax.cuh"

namespace sa2 {
namespace {

constexpr int kThreads = 544;
constexpr uint32_t kTmemCols = 512;
// TMEM columns: the two S buffers of tile t at 128 t and 128 t + 64 (P as 16-bit pairs over the first
// 32 columns of its S), O at 256 + 128 t.
__device__ __forceinline__ uint32_t col_s(int t, uint32_t buf) { return 128u * t + 64u * buf; }
__device__ __forceinline__ uint32_t col_o(int t) { return 256u + 128u * t; }

template <int D, bool KV8>
struct XSmem {
  static constexpr int kPanels = D / 64;
  static constexpr int kTile = 128 * 128 * kPanels;  // 128 rows x 128 B per panel
  static constexpr int kStages = D == 64 ? 8 : 4;
  static constexpr int kOffKV = 2 * kTile;
  static constexpr int kRaw = kTile / 2;                  // 8-bit keys: a block as it lies in the cache
  static constexpr int kRawStages = D == 64 ? 4 : 2;
  static constexpr int kOffRaw = kOffKV + kStages * kTile;
  static constexpr int kOffO = kOffRaw;                   // 16-bit keys: a tile of O on its way out
  static constexpr int kOffBar = kOffRaw + (KV8 ? kRawStages * kRaw : kTile);
  // [2][128], for each row 1 / l (16-bit keys) or the scale of its converted query (8-bit keys)
  static constexpr int kOffRow = kOffBar + 512;
  static constexpr int kBytes = kOffRow + 1024 + 1024;
  static_assert(kBytes <= (int)kMaxDynSmem, "shared memory");
};

__device__ __forceinline__ uint2 e4m3x4_to_f16x4(uint32_t w) {
  const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
  const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// F16: the type of Q and O (and of K, V when they are 16-bit).
template <int D, bool KV8, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    cross_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo, CrossShape s,
                     FwdPlan plan, CacheRef cache,
                     CrossFwdArgs a) {
  using L = XSmem<D, KV8>;
  constexpr int kStages = L::kStages;
  constexpr bool kMmaF16 = KV8 || F16;  // the cache's products run in fp16
  // How far (log2) a block's maximum may lead the reference.  fp16 P holds 2^15; bf16 P could hold far more, but P V
  // is summed in fp32 before O and l follow: V would be left what the lead does not take of 2^128.
  constexpr float kMaxLead = 14.f;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  auto bar_full = [&](int st) { return smem_u32(&bars[st]); };        // ring stage filled
  auto bar_empty = [&](int st) { return smem_u32(&bars[8 + st]); };   // ... and read by its MMAs
  auto bar_qfull = [&](int t) { return smem_u32(&bars[16 + t]); };    // Q of tile t in shared memory
  auto bar_qempty = [&](int t) { return smem_u32(&bars[18 + t]); };   // ... and read (by its last S; cache: and its row scales)
  auto bar_s = [&](int t, uint32_t u) { return smem_u32(&bars[20 + 2 * t + u]); };   // S buffer u of tile t in TMEM
  auto bar_p = [&](int t, uint32_t u) { return smem_u32(&bars[24 + 2 * t + u]); };   // P written over it
  auto bar_pv = [&](int t, uint32_t u) { return smem_u32(&bars[48 + 2 * t + u]); };  // P V from it completed
  auto bar_o = [&](int t) { return smem_u32(&bars[28 + t]); };        // O_t of the piece complete
  auto bar_ofree = [&](int t) { return smem_u32(&bars[30 + t]); };    // ... and read out
  auto bar_l = [&](int t) { return smem_u32(&bars[32 + t]); };        // 1 / l of the piece written
  auto bar_drain = [&](int t) { return smem_u32(&bars[34 + t]); };
  auto bar_pdrain = [&](int t) { return smem_u32(&bars[36 + t]); };
  const uint32_t bar_st = smem_u32(&bars[38]), bar_stfree = smem_u32(&bars[39]);  // O tile staged / copied out
  auto bar_rfull = [&](int i) { return smem_u32(&bars[40 + i]); };    // 8-bit block landed
  auto bar_rempty = [&](int i) { return smem_u32(&bars[44 + i]); };   // ... and converted
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffBar + 448);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffBar + 456);
  float* row_s = reinterpret_cast<float*>(smem + L::kOffRow);
  const WaitCtl wc{abort_flag, s.wait_ns};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    *abort_flag = 0;
    for (int st = 0; st < kStages; ++st) {
      mbar_init(bar_full(st), KV8 ? 128 : 1);
      mbar_init(bar_empty(st), 2);  // both issuers
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar_qfull(t), KV8 ? 128 : 1);
      mbar_init(bar_qempty(t), KV8 ? 129 : 1);
      for (uint32_t u = 0; u < 2; ++u) {
        mbar_init(bar_s(t, u), 1);
        mbar_init(bar_p(t, u), 128);
        mbar_init(bar_pv(t, u), 1);
      }
      mbar_init(bar_o(t), 1);
      mbar_init(bar_ofree(t), 128);
      mbar_init(bar_l(t), 128);
      mbar_init(bar_drain(t), 1);
      mbar_init(bar_pdrain(t), 1);
    }
    for (int i = 0; i < L::kRawStages; ++i) {
      mbar_init(bar_rfull(i), 1);
      mbar_init(bar_rempty(i), 128);
    }
    mbar_init(bar_st, 128);
    mbar_init(bar_stfree, 1);
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
  if (plan.split) kernel_trigger();
  const int tp = plan.tp;  // tiles per segment
  auto active = [&](const Piece& x, int t) { return (x.mask >> t) & 1; };
  // K's or V's stages of a piece, free as far as a tile without rows goes.  Every phase of bar_full is
  // waited for: a warp that skipped one would take the phase before it for its own.
  auto pass_stages = [&](uint32_t r, int nb) {
    for (int i = 0; i < nb; ++i, r += 2) {
      if (!__all_sync(0xffffffffu, mbar_wait(bar_full(r % kStages), (r / kStages) & 1, wc))) return false;
      if (lane == 0) mbar_arrive(bar_empty(r % kStages));
    }
    return true;
  };
  if (a.kv_len && blockIdx.x == 0 && warp == 3) {
    for (int b = lane; b < s.B; b += 32)
      if (a.kv_len[b] < 0 || a.kv_len[b] > s.M) report_error(a.status, kDevErrBounds);
  }

  if (warp == 0 && !KV8) {
    // ------------------------------------------------------------------ TMA producer
    PieceIter it(s, plan, a.kv_len);  // (whole warps)
    if (lane == 0) {
      tma_prefetch_map(&mq);
      tma_prefetch_map(&mk);
      tma_prefetch_map(&mv);
      const uint32_t q_bytes = (uint32_t)(L::kPanels * 128 * plan.nb * s.G);
      uint32_t r = 0, qn[2] = {0, 0};  // ring loads and Q tiles issued
      bool ok = true;
      Piece x;
      while (ok && it.next(x)) {
        auto load = [&](const CUtensorMap* map, int kb) {
          const int st = r % kStages;
          if (r >= (uint32_t)kStages && !mbar_wait(bar_empty(st), ((r / kStages) - 1) & 1, wc)) return false;
          mbar_arrive_expect_tx(bar_full(st), L::kTile);
          for (int pn = 0; pn < L::kPanels; ++pn)
            tma_load_5d(sbase + L::kOffKV + st * L::kTile + pn * 16384, map, bar_full(st), pn * 64, 0, kb * kKeyBlock,
                        x.hk, x.b);
          ++r;
          return true;
        };
        for (int j = 0; ok && j < x.nb; ++j) {
          ok = load(&mk, x.k0 + j);
          if (j == 0) {
            for (int t = 0; ok && t < 2; ++t) {
              if (!active(x, t)) continue;
              if (qn[t] >= 1 && !mbar_wait(bar_qempty(t), (qn[t] - 1) & 1, wc)) {
                ok = false;
                break;
              }
              mbar_arrive_expect_tx(bar_qfull(t), q_bytes);
              for (int pn = 0; pn < L::kPanels; ++pn)
                tma_load_5d(sbase + t * L::kTile + pn * 16384, &mq, bar_qfull(t), pn * 64, 0,
                            (x.pair * tp + t) * plan.nb, x.hk, x.b);
              ++qn[t];
            }
          }
          if (ok) ok = load(&mv, x.k0 + j);
        }
      }
      // No copy may still be in flight when the CTA exits: each stage's last load, each tile's Q.
      for (uint32_t v = r > (uint32_t)kStages ? r - kStages : 0; v < r; ++v)
        mbar_drain(bar_full(v % kStages), (v / kStages) & 1, abort_flag);
      for (int t = 0; t < 2; ++t)
        if (qn[t]) mbar_drain(bar_qfull(t), (qn[t] - 1) & 1, abort_flag);
    }
  } else if (warp == 0) {
    // ---------------------------------------------------- TMA producer of the 8-bit blocks
    PieceIter it(s, plan, a.kv_len);  // (whole warps)
    if (lane == 0) {
      tma_prefetch_map(&mk);
      tma_prefetch_map(&mv);
      uint32_t r = 0;
      bool ok = true;
      Piece x;
      while (ok && it.next(x)) {
        for (int i = 0; i < 2 * x.nb; ++i, ++r) {
          const int st = r % L::kRawStages;
          if (r >= (uint32_t)L::kRawStages && !mbar_wait(bar_rempty(st), ((r / L::kRawStages) - 1) & 1, wc)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar_rfull(st), L::kRaw);
          tma_load_5d(sbase + L::kOffRaw + st * L::kRaw, (i & 1) ? &mv : &mk, bar_rfull(st), 0, 0,
                      (x.k0 + (i >> 1)) * kKeyBlock, x.hk, x.b);
        }
      }
      for (uint32_t v = r > (uint32_t)L::kRawStages ? r - L::kRawStages : 0; v < r; ++v)
        mbar_drain(bar_rfull(v % L::kRawStages), (v / L::kRawStages) & 1, abort_flag);
    }
  } else if (warp == 1 || warp == 2) {
    // ------------------------------------------------------------------ issuer of S of tile t
    PieceIter it(s, plan, a.kv_len);
    const int t = warp - 1;
    const uint64_t qd = smem_desc(sbase + t * L::kTile, 16, 1024);
    bool ok = true;
    uint32_t r = 0, c = 0, pc = 0;  // ring loads of earlier pieces; half blocks and pieces done
    Piece x;
    while (ok && it.next(x)) {
      if (!active(x, t)) {
        ok = pass_stages(r, x.nb);
        r += 2 * x.nb;
        continue;
      }
      const int keys = min(x.nb * kKeyBlock, x.keys - x.k0 * kKeyBlock);
      const int halves = (keys + 63) >> 6;
      // into buffer c & 1, whose P V two half blocks ago has completed
      for (int i = 0; i < halves; ++i, ++c) {
        const uint32_t rk = r + (i & ~1), u = c & 1;
        const int ks = rk % kStages;
        const bool last = i + 1 == halves;
        ok = __all_sync(0xffffffffu, ((i & 1) || mbar_wait(bar_full(ks), (rk / kStages) & 1, wc)) &&
                                         (i > 0 || mbar_wait(bar_qfull(t), pc & 1, wc)) &&
                                         (c < 2 || mbar_wait(bar_pv(t, u), ((c >> 1) - 1) & 1, wc)));
        if (!ok) break;
        tc_fence_after();
        const uint32_t idS = idesc_f32acc(128, min(64, (keys - 64 * i + 15) & ~15), false, false, !kMmaF16);
        const uint64_t kd = smem_desc(sbase + L::kOffKV + ks * L::kTile + (i & 1) * 8192, 16, 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_ss(tmem + col_s(t, u), qd + kmajor_kstep(kk, 128), kd + kmajor_kstep(kk, 128), idS, kk > 0 ? 1u : 0u);
          umma_commit(bar_s(t, u));
          if ((i & 1) || last) umma_commit(bar_empty(ks));
          if (last) umma_commit(bar_qempty(t));
        }
        __syncwarp();
      }
      if (x.nb > 0) ++pc;
      r += 2 * x.nb;
    }
    // no MMA may still run when TMEM is released, on the abort path too
    if (elect_one()) umma_commit(bar_drain(t));
    __syncwarp();
    mbar_drain(bar_drain(t), 0, abort_flag);
  } else if (warp == 3 || warp == 16) {
    // ------------------------------------------------------------------ issuer of P V of tile t
    PieceIter it(s, plan, a.kv_len);
    constexpr uint32_t idO = idesc_f32acc(128, D, false, true, !kMmaF16);
    const int t = warp >> 4;
    bool ok = true;
    uint32_t r = 0, c = 0, pc = 0;
    Piece x;
    while (ok && it.next(x)) {
      if (!active(x, t)) {
        ok = pass_stages(r + 1, x.nb);
        r += 2 * x.nb;
        continue;
      }
      const int keys = min(x.nb * kKeyBlock, x.keys - x.k0 * kKeyBlock);
      const int halves = (keys + 63) >> 6;
      for (int i = 0; i < halves; ++i, ++c) {
        const uint32_t rv = r + (i & ~1) + 1, u = c & 1;
        const int vs = rv % kStages, valid = min(64, keys - 64 * i), steps = (valid + 15) >> 4;
        const bool last = i + 1 == halves;
        ok = __all_sync(0xffffffffu, (i & 1) || mbar_wait(bar_full(vs), (rv / kStages) & 1, wc));
        if (!ok) break;
        const int rows = 16 * steps - valid;
        if (!KV8 && rows > 0) {
          // `rows` rows of V behind the last key (both issuers write the same zeros): a row is 128 bytes
          // in each panel
          uint8_t* vt = smem + L::kOffKV + vs * L::kTile + (i & 1) * 8192;
          const int nz = rows * 8 * L::kPanels;
          for (int q = lane; q < nz; q += 32) {
            const int row = valid + (q >> 3) % rows, pn = (q >> 3) / rows;
            *reinterpret_cast<uint4*>(vt + pn * 16384 + row * 128 + (q & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async();
          __syncwarp();
        }
        ok = __all_sync(0xffffffffu, (i > 0 || pc == 0 || mbar_wait(bar_ofree(t), (pc - 1) & 1, wc)) &&
                                         mbar_wait(bar_p(t, u), (c >> 1) & 1, wc));
        if (!ok) break;
        tc_fence_after();
        const uint64_t vd = smem_desc(sbase + L::kOffKV + vs * L::kTile + (i & 1) * 8192, 16384, 1024);
        if (elect_one()) {
          issue_pv(tmem + col_o(t), tmem + col_s(t, u), vd, idO, steps, i == 0);
          umma_commit(bar_pv(t, u));
          if ((i & 1) || last) umma_commit(bar_empty(vs));
          if (last) umma_commit(bar_o(t));
        }
        __syncwarp();
      }
      if (x.nb > 0) ++pc;
      r += 2 * x.nb;
    }
    if (elect_one()) umma_commit(bar_pdrain(t));
    __syncwarp();
    mbar_drain(bar_pdrain(t), 0, abort_flag);
  } else if (warp >= 8) {
    // ------------------------------------------------------------------ softmax rows
    if (s.stall_ns && blockIdx.x == 0) stall_for(s.stall_ns);  // failure-path test hook
    PieceIter it(s, plan, a.kv_len);
    const int t = (warp - 8) >> 2;
    const int r = 32 * (warp & 3) + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const uint32_t to = trow + col_o(t);
    bool ok = true;
    uint32_t c = 0, pc = 0;
    Piece x;
    while (ok && it.next(x)) {
      if (!active(x, t)) continue;
      // (found again behind the keys, for the registers of the loop between)
      auto row_of = [&](int& h, int& n) {
        const int tok_r = r / s.G;
        n = (x.pair * tp + t) * plan.nb + tok_r;
        h = x.hk * s.G + r - tok_r * s.G;
        return tok_r < plan.nb && n < s.N;
      };
      if (x.nb == 0) {  // (direct mode) no keys
        int h, n;
        const bool row_valid = row_of(h, n);
        const int64_t row = ((int64_t)x.b * s.H + h) * s.N + n;
        if (row_valid) {
          a.lse[row] = -INFINITY;
          if constexpr (KV8) {
            uint4* op = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o.p) + x.b * a.o.sb + h * a.o.sh + n * a.o.sn);
            for (int i = 0; i < D / 8; ++i) op[i] = make_uint4(0, 0, 0, 0);
          }
        }
        continue;
      }
      // cache: scores are q8 scale * k8 scale * (q . k) and V's scale enters as an exponent
      float qscale = a.scale_log2;
      int64_t sc = 0;  // of the piece's first half block
      float nks = 1.f, nvs = 1.f;  // of the next half block, loaded one ahead
      if constexpr (KV8) {
        sc = ((int64_t)x.b * s.Hkv + x.hk) * cache.nsb + 2 * x.k0;
        nks = cache.ks[sc];
        nvs = cache.vs[sc];
        if (!__all_sync(0xffffffffu, mbar_wait(bar_qfull(t), pc & 1, wc))) {
          ok = false;
          break;
        }
        qscale *= row_s[t * 128 + r];
        mbar_arrive(bar_qempty(t));
      }
      float m_used = 0.f, m_run = 0.f;  // reference of the exponentials, largest so far
      // sum of exp2(s) relative to m_used; cache: to l_ref, since s + log2(V's scale), which m_used follows,
      // can be any distance from s
      float l = 0.f, l_ref = -INFINITY;
      // O and l to another reference.  O holds the half blocks before this one once their P V has
      // completed: the last one's, from the other buffer, is waited for.
      auto rescale = [&](float m_new) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar_pv(t, (c & 1) ^ 1), ((c - 1) >> 1) & 1, wc))) return false;
        tc_fence_after();
        const float alpha = m_new == m_used ? 1.f : ex2(m_used - m_new);
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 16) {
          uint32_t o[16];
          tmem_ld16(to + c0, o);
          tmem_ld_wait16(o);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st16(to + c0, o);
        }
        tmem_st_wait();
        if constexpr (!KV8) l *= alpha;
        m_used = m_new;
        return true;
      };
      const int keys = min(x.nb * kKeyBlock, x.keys - x.k0 * kKeyBlock);
      for (int i = 0; 64 * i < keys; ++i, ++c) {
        const uint32_t u = c & 1, ts = trow + col_s(t, u);
        const int valid = keys - 64 * i;
        float mul = qscale, ev = 0.f;
        if constexpr (KV8) {
          mul = score_factor(qscale, nks);
          ev = (float)((int)(__float_as_uint(nvs) >> 23) - 127);
          if (valid > 64) {
            nks = cache.ks[sc + i + 1];
            nvs = cache.vs[sc + i + 1];
          }
        }
        if (!__all_sync(0xffffffffu, mbar_wait(bar_s(t, u), (c >> 1) & 1, wc))) {
          ok = false;
          break;
        }
        tc_fence_after();
        // The exponentials are taken against a maximum of the half blocks before this one, so that they
        // need not wait for this one's: the first uses its own, then O and l follow when the maximum
        // has grown past 2^8.  Only where P would lead by more than 2^14 does a half block's own maximum
        // come first (the loop below runs twice).
        if (i == 0) {
          float y[32];
          load_scores(ts, y, valid);
          const float m0 = max32(y);
          load_scores(ts + 32, y, valid - 32);
          m_used = m_run = fmaxf(fmaf(fmaxf(m0, max32(y)), mul, ev), kLeastRef);
        } else if (__any_sync(0xffffffffu, m_run > m_used + kRescaleThreshold)) {
          ok = rescale(m_run > m_used + kRescaleThreshold ? m_run : m_used);
        }
        uint32_t pk[32];
        float sum, ref = m_used;
        // cache: scores whose exponent is 2^-64 or less of the reference's (small values beside large
        // ones) are 0 in P, but count in the sum: relative to their own maximum
        bool low = false;
        for (bool again = false;;) {
          float2 part[2] = {{0.f, 0.f}, {0.f, 0.f}};
          float mx;
          {
            float y[32];
            load_scores(ts, y, valid);
            mx = max32(y);
            exp32<kMmaF16>(y, mul, ev - ref, pk, part);
            load_scores(ts + 32, y, valid - 32);
            mx = fmaxf(mx, max32(y));
            exp32<kMmaF16>(y, mul, ev - ref, pk + 16, part);
          }
          const float2 both = add2(part[0], part[1]);
          sum = both.x + both.y;
          mx = fmaf(mx, mul, ev);
          m_run = fmaxf(m_run, mx);
          if (again || !ok) break;
          low = KV8 && mx < m_used - 64.f;
          if (!__any_sync(0xffffffffu, low || mx > m_used + kMaxLead)) break;
          // (a row's reference follows from its own scores only: neighbours, and rows of the tile that are no
          // query's, must not change its roundings)
          if (__any_sync(0xffffffffu, mx > m_used + kMaxLead)) ok = rescale(mx > m_used + kMaxLead ? mx : m_used);
          low = KV8 && mx < m_used - 64.f;
          ref = low ? mx : m_used;
          again = true;
        }
        if (!ok) break;
        if (KV8 && low) {
#pragma unroll
          for (int q = 0; q < 32; ++q) pk[q] = 0u;
        }
        tmem_st32(ts, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar_p(t, u));
        if constexpr (KV8) {
          const float x = ref - ev;
          if (x > l_ref + 60.f) {  // (the first half block too)
            l *= ex2(l_ref - x);
            l_ref = x;
          }
          l = fmaf(sum, ex2(x - l_ref), l);
        } else {
          l += sum;
        }
      }
      if (!ok) break;
      int h, n;
      const bool row_valid = row_of(h, n);
      const int64_t row = ((int64_t)x.b * s.H + h) * s.N + n;
      const int64_t slot_row = ((int64_t)blockIdx.x + x.seg) * 256 + t * 128 + r;
      const float lse2 = (KV8 ? l_ref : m_used) + __log2f(l);
      if (row_valid) {
        if (plan.split)
          a.part_l[slot_row] = lse2;
        else
          a.lse[row] = lse2 * 0.69314718055994531f;
      }
      if constexpr (!KV8) {
        // the epilogue warps read the previous piece's 1 / l before they released its O
        if (pc > 0 && !__all_sync(0xffffffffu, mbar_wait(bar_ofree(t), (pc - 1) & 1, wc))) {
          ok = false;
          break;
        }
        row_s[t * 128 + r] = inverse_sum(l);
        mbar_arrive(bar_l(t));
      } else {
        if (!__all_sync(0xffffffffu, mbar_wait(bar_o(t), pc & 1, wc))) {
          ok = false;
          break;
        }
        tc_fence_after();
        // 2^(m_used - l_ref) / l; the power alone may leave fp32's range, where l makes up for it
        const float root = ex2(0.5f * (m_used - l_ref)), inv_l = root / l * root;
        uint16_t* op = static_cast<uint16_t*>(a.o.p) + x.b * a.o.sb + h * a.o.sh + n * a.o.sn;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t u[32];
          tmem_ld32(to + c0, u);
          tmem_ld_wait(u);
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]) * inv_l;
          if (row_valid && plan.split) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              reinterpret_cast<float4*>(a.part_o + slot_row * D + c0)[i] =
                  make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          } else if (row_valid) {
            store32(op + c0, v, F16);
          }
        }
        tc_fence_before();
        mbar_arrive(bar_ofree(t));
      }
      ++pc;
    }
  } else if (warp >= 4 && !KV8) {
    // ------------------------------------------------------------------ epilogue: O / l
    // A tile goes out through shared memory with one TMA store: stored row by row, 16 bytes per
    // thread, it kept the load/store unit busy for 3000 cycles, which the softmax threads' tcgen05.ld
    // waited for (M = 512: a fifth of the time).
    PieceIter it(s, plan, a.kv_len);
    const int r = 32 * (warp & 3) + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const int tok_r = r / s.G, g = r - tok_r * s.G;
    bool ok = true;
    uint32_t pc[2] = {0, 0}, staged = 0;
    Piece x;
    while (ok && it.next(x)) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (!ok || !active(x, t)) continue;
        const int n = (x.pair * tp + t) * plan.nb + tok_r;
        const bool row_valid = tok_r < plan.nb && n < s.N;
        const int h = x.hk * s.G + g;
        if (x.nb == 0) {
          uint16_t* op = static_cast<uint16_t*>(a.o.p) + x.b * a.o.sb + h * a.o.sh + n * a.o.sn;
          if (row_valid)
            for (int i = 0; i < D / 8; ++i) reinterpret_cast<uint4*>(op)[i] = make_uint4(0, 0, 0, 0);
          continue;
        }
        ok = __all_sync(0xffffffffu, mbar_wait(bar_l(t), pc[t] & 1, wc) && mbar_wait(bar_o(t), pc[t] & 1, wc) &&
                                         (plan.split || staged == 0 || mbar_wait(bar_stfree, (staged - 1) & 1, wc)));
        if (!ok) break;
        ++pc[t];
        tc_fence_after();
        const float inv_l = row_s[t * 128 + r];
        const int64_t slot_row = ((int64_t)blockIdx.x + x.seg) * 256 + t * 128 + r;
        uint8_t* st_row = smem + L::kOffO + r * 128;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t u[32];
          tmem_ld32(trow + col_o(t) + c0, u);
          tmem_ld_wait(u);
          if (c0 + 32 >= D) {
            tc_fence_before();
            mbar_arrive(bar_ofree(t));
          }
          if (plan.split) {
            if (row_valid) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                reinterpret_cast<float4*>(a.part_o + slot_row * D + c0)[i] =
                    make_float4(__uint_as_float(u[4 * i]) * inv_l, __uint_as_float(u[4 * i + 1]) * inv_l,
                                __uint_as_float(u[4 * i + 2]) * inv_l, __uint_as_float(u[4 * i + 3]) * inv_l);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float v0 = __uint_as_float(u[8 * i + 2 * q]) * inv_l, v1 = __uint_as_float(u[8 * i + 2 * q + 1]) * inv_l;
                w[q] = F16 ? pack_f16x2(v0, v1) : pack_bf16x2(v0, v1);
              }
              // 16-byte chunk k of the row's 128 bytes in panel c0 / 64, swizzled
              const int k = (c0 & 32) / 8 + i;
              *reinterpret_cast<uint4*>(st_row + (c0 >> 6) * 16384 + ((k ^ (r & 7)) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        if (!plan.split) {
          fence_proxy_async();
          mbar_arrive(bar_st);
          if (warp == 4) {
            ok = __all_sync(0xffffffffu, mbar_wait(bar_st, staged & 1, wc));
            if (!ok) break;
            if (lane == 0) {
              for (int pn = 0; pn < L::kPanels; ++pn)  // tokens past the end are not written
                tma_store_5d(&mo, sbase + L::kOffO + pn * 16384, pn * 64, 0, (x.pair * tp + t) * plan.nb, x.hk, x.b);
              bulk_commit();
              bulk_wait_read();
              mbar_arrive(bar_stfree);
            }
            __syncwarp();
          }
          ++staged;
        }
      }
    }
  } else if (warp >= 4 && KV8) {
    // --------------------------------------------------- converters: Q, K, V to fp16
    PieceIter it(s, plan, a.kv_len);
    constexpr int kChunks = D / 16;       // 16-byte chunks of an 8-bit row
    constexpr int kRows = 128 / kChunks;  // rows per pass of the 128 threads
    const int ct = tid - 128;
    const int ch = ct % kChunks, r0 = ct / kChunks;
    bool ok = true;
    uint32_t r = 0, qn[2] = {0, 0};
    Piece x;
    while (ok && it.next(x)) {
      if (x.nb == 0) continue;
      // Q: thread = row, scaled by a power of two so that its largest magnitude is in [2^14, 2^15)
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        if (!active(x, t)) continue;
        if (qn[t] >= 1 && !__all_sync(0xffffffffu, mbar_wait(bar_qempty(t), (qn[t] - 1) & 1, wc))) {
          ok = false;
          break;
        }
        ++qn[t];
        const int tok_r = ct / s.G, g = ct - tok_r * s.G;
        const int n = (x.pair * tp + t) * plan.nb + tok_r;
        const bool row_valid = tok_r < plan.nb && n < s.N;
        const uint4* qp = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q.p) + x.b * a.q.sb +
                                                         (int64_t)(x.hk * s.G + g) * a.q.sh + (int64_t)n * a.q.sn);
        int e = 0;
        if constexpr (!F16) {
          // the largest magnitude: bf16 magnitudes compare as integers
          uint32_t mx = 0;
#pragma unroll 4
          for (int i = 0; i < D / 8; ++i) {
            const uint4 u = row_valid ? __ldg(qp + i) : make_uint4(0, 0, 0, 0);
            mx = max(max(mx, max(u.x & 0x7FFFu, (u.x >> 16) & 0x7FFFu)), max(u.y & 0x7FFFu, (u.y >> 16) & 0x7FFFu));
            mx = max(max(mx, max(u.z & 0x7FFFu, (u.z >> 16) & 0x7FFFu)), max(u.w & 0x7FFFu, (u.w >> 16) & 0x7FFFu));
          }
          // a row of zeros, or with an infinity or NaN, keeps its scale
          if (mx >= 0x0080u && mx < 0x7F80u) e = min(max((int)(mx >> 7) - 127 - 14, -112), 112);
        }
        row_s[t * 128 + ct] = __uint_as_float((uint32_t)(127 + e) << 23);
        const float f = __uint_as_float((uint32_t)(127 - e) << 23);
        uint8_t* dst = smem + t * L::kTile + ct * 128;
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
          uint4 u = row_valid ? __ldg(qp + i) : make_uint4(0, 0, 0, 0);
          if constexpr (!F16) {
            u.x = pack_f16x2(__uint_as_float(u.x << 16) * f, __uint_as_float(u.x & 0xFFFF0000u) * f);
            u.y = pack_f16x2(__uint_as_float(u.y << 16) * f, __uint_as_float(u.y & 0xFFFF0000u) * f);
            u.z = pack_f16x2(__uint_as_float(u.z << 16) * f, __uint_as_float(u.z & 0xFFFF0000u) * f);
            u.w = pack_f16x2(__uint_as_float(u.w << 16) * f, __uint_as_float(u.w & 0xFFFF0000u) * f);
          }
          *reinterpret_cast<uint4*>(dst + (i >> 3) * 16384 + (((i & 7) ^ (ct & 7)) << 4)) = u;
        }
        fence_proxy_async();
        mbar_arrive(bar_qfull(t));
      }
      if (!ok) break;
      // K_0, V_0, K_1, ... as they land, into the ring, swizzled: a key's 16 values of chunk ch are 32
      // bytes of panel ch / 4; behind the last key zeros
      for (int i = 0; i < 2 * x.nb; ++i, ++r) {
        const int st = r % kStages, rs = r % L::kRawStages;
        if (!__all_sync(0xffffffffu,
                        mbar_wait(bar_rfull(rs), (r / L::kRawStages) & 1, wc) &&
                            (r < (uint32_t)kStages || mbar_wait(bar_empty(st), ((r / kStages) - 1) & 1, wc)))) {
          ok = false;
          break;
        }
        const int valid = x.keys - (x.k0 + (i >> 1)) * kKeyBlock;
        const uint8_t* src = smem + L::kOffRaw + rs * L::kRaw + r0 * D + ch * 16;
        uint8_t* dst = smem + L::kOffKV + st * L::kTile + (ch >> 2) * 16384;
#pragma unroll
        for (int q = 0; q < kChunks; ++q) {
          const int row = r0 + q * kRows;
          const uint4 u = row < valid ? *reinterpret_cast<const uint4*>(src + q * kRows * D) : make_uint4(0, 0, 0, 0);
          const uint2 w0 = e4m3x4_to_f16x4(u.x), w1 = e4m3x4_to_f16x4(u.y), w2 = e4m3x4_to_f16x4(u.z),
                      w3 = e4m3x4_to_f16x4(u.w);
          const uint4 lo = make_uint4(w0.x, w0.y, w1.x, w1.y), hi = make_uint4(w2.x, w2.y, w3.x, w3.y);
          // the two panels' lanes store opposite halves first, so that a quarter warp's 16-byte
          // stores fall into different banks
          const int odd = (ch >> 2) & 1, k16 = (ch & 3) * 2;
          *reinterpret_cast<uint4*>(dst + row * 128 + (((k16 + odd) ^ (row & 7)) << 4)) = odd ? hi : lo;
          *reinterpret_cast<uint4*>(dst + row * 128 + (((k16 + 1 - odd) ^ (row & 7)) << 4)) = odd ? lo : hi;
        }
        fence_proxy_async();
        mbar_arrive(bar_full(st));
        mbar_arrive(bar_rempty(rs));
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

// Joins the parts of split segments: O = sum_i 2^(l_i - m) O_i / sum_i 2^(l_i - m) over a segment's
// parts in key order, l_i their log2 sums and m the largest; LSE = ln 2 (m + log2 sum).  Rows of
// sequences without keys get 0 and -inf.  One warp per row; grid (segments, parts of their rows).
template <int D, bool F16>
__global__ void __launch_bounds__(256) cross_join_kernel(CrossShape s, FwdPlan plan, CrossFwdArgs a) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int seg = blockIdx.x;
  const int per_b = s.Hkv * plan.pairs;
  const int b = seg / per_b, hk = (seg - b * per_b) / plan.pairs, pair = seg - b * per_b - hk * plan.pairs;
  const int64_t run = run_length(total_key_blocks(s, a.kv_len, plan.pairs, plan.shift), plan.grid);
  int64_t base = 0;
  for (int i = lane; i < b; i += 32) base += key_blocks(key_count(a.kv_len, i, s.M), plan.shift);
  for (int o = 16; o > 0; o >>= 1) base += __shfl_xor_sync(0xffffffffu, base, o);
  const int nk = key_blocks(key_count(a.kv_len, b, s.M), plan.shift);
  const int64_t g0 = base * per_b + (int64_t)(seg - b * per_b) * nk;
  const int c0 = (int)(g0 / run), c1 = nk > 0 ? (int)((g0 + nk - 1) / run) : c0 - 1;
  const int rows = min(plan.tp * 128, plan.rows) / gridDim.y;
  kernel_wait();
  for (int i = warp; i < rows; i += 8) {
    const int rr = blockIdx.y * rows + i, t = rr >> 7, r = rr & 127;
    const int tile = pair * plan.tp + t;
    if (t >= plan.tp || tile >= plan.tiles) return;
    const int tok_r = r / s.G, g = r - tok_r * s.G, n = tile * plan.nb + tok_r, h = hk * s.G + g;
    if (tok_r >= plan.nb || n >= s.N) continue;
    // lane i has part c0 + i's sum; 32 parts at a time (more are rare), eight of their rows in flight
    float m = kLeastRef, acc[kPer] = {}, l = 0.f;
    for (int base = c0; base <= c1; base += 32) {
      const int n32 = min(32, c1 + 1 - base);
      const float mine = lane < n32 ? a.part_l[((int64_t)base + lane + seg) * plan.rows + rr] : -INFINITY;
      float mx = mine;
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      if (__any_sync(0xffffffffu, mine != mine)) mx = NAN;
      const float m_new = m != m ? m : (mx > m || mx != mx ? mx : m);
      const float keep = base == c0 ? 0.f : ex2(m - m_new);
      m = m_new;
      l *= keep;
#pragma unroll
      for (int q = 0; q < kPer; ++q) acc[q] *= keep;
      const float wl = lane < n32 ? ex2(mine - m) : 0.f;
      for (int k = 0; k < n32; k += 8) {
        float v[8][kPer];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (k + u >= n32) break;
          const float* src = a.part_o + (((int64_t)base + k + u + seg) * plan.rows + rr) * D;
          if constexpr (kPer == 4)
            *reinterpret_cast<float4*>(v[u]) = *reinterpret_cast<const float4*>(src + lane * 4);
          else
            *reinterpret_cast<float2*>(v[u]) = *reinterpret_cast<const float2*>(src + lane * 2);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float w = __shfl_sync(0xffffffffu, wl, (k + u) & 31);
          if (k + u < n32) {
            l += w;
#pragma unroll
            for (int q = 0; q < kPer; ++q) acc[q] = fmaf(w, v[u][q], acc[q]);
          }
        }
      }
    }
    const float inv = inverse_sum(l);
    uint32_t w[kPer / 2];
#pragma unroll
    for (int q = 0; q < kPer / 2; ++q)
      w[q] = F16 ? pack_f16x2(acc[2 * q] * inv, acc[2 * q + 1] * inv) : pack_bf16x2(acc[2 * q] * inv, acc[2 * q + 1] * inv);
    uint16_t* op = static_cast<uint16_t*>(a.o.p) + b * a.o.sb + h * a.o.sh + (int64_t)n * a.o.sn + lane * kPer;
    if constexpr (kPer == 4)
      *reinterpret_cast<uint2*>(op) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(op) = w[0];
    if (lane == 0)
      a.lse[((int64_t)b * s.H + h) * s.N + n] = (m + __log2f(l)) * 0.69314718055994531f;
  }
}

template <int D, bool KV8, bool F16>
cudaError_t launch_t(const CrossShape& s, const FwdPlan& p, const CUtensorMap& mq, const CUtensorMap& mk,
                     const CUtensorMap& mv, const CUtensorMap& mo, const CacheRef& c, const CrossFwdArgs& a, cudaStream_t st) {
  auto kern = cross_fwd_kernel<D, KV8, F16>;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = allow_smem(kern, XSmem<D, KV8>::kBytes, allowed);
  if (e != cudaSuccess) return e;
  prof_start(st, kAttnFwd);
  kern<<<(unsigned)p.grid, kThreads, XSmem<D, KV8>::kBytes, st>>>(mq, mk, mv, mo, s, p, c, a);
  prof_stop(st, kAttnFwd);
  e = cudaGetLastError();
  return e == cudaSuccess && p.split ? launch_cross_join(s, p, a, st) : e;
}

template <bool KV8>
cudaError_t launch_any(const CrossShape& s, const FwdPlan& p, const CUtensorMap& mq, const CUtensorMap& mk,
                       const CUtensorMap& mv, const CUtensorMap& mo, const CacheRef& c, const CrossFwdArgs& a,
                       cudaStream_t st) {
  const bool f16 = s.dtype == SA2_FP16;
  if (s.d == 128)
    return f16 ? launch_t<128, KV8, true>(s, p, mq, mk, mv, mo, c, a, st)
               : launch_t<128, KV8, false>(s, p, mq, mk, mv, mo, c, a, st);
  return f16 ? launch_t<64, KV8, true>(s, p, mq, mk, mv, mo, c, a, st)
             : launch_t<64, KV8, false>(s, p, mq, mk, mv, mo, c, a, st);
}

}  // namespace

// Segments are whole where they fill the SMs at least four times over (their sizes then even
// out) or where a sequence has fewer than eight key blocks (the second kernel would cost what
// the split gains).
FwdPlan cross_fwd_plan(const CrossShape& s, int sms) {
  FwdPlan p;
  if (s.N * (int64_t)s.G <= kFewRows) {
    // One tile of all rows.  Whole segments where a CTA's warps have at most four steps each, or
    // where there are CTAs enough to even out the lengths.
    p.few = true;
    p.nb = s.N;
    p.tiles = p.tp = p.pairs = 1;
    p.shift = 6;
    p.rows = kFewRows;
    const int64_t segs = (int64_t)s.B * s.Hkv;
    p.segs = segs > INT32_MAX ? -1 : (int)segs;
    p.split = s.M > 1024 && segs < 8 * (int64_t)sms;
    p.grid = p.split ? (int)std::min<int64_t>(sms, segs * ((s.M + 63) / 64)) : p.segs;
    p.join_rows = kFewRows;
    return p;
  }
  p.few = false;
  p.shift = kKeyBlockShift;
  p.rows = 256;
  p.nb = 128 / s.G;
  p.tiles = (s.N + p.nb - 1) / p.nb;
  const int64_t heads = (int64_t)s.B * s.Hkv;
  const int blocks = (s.M + kKeyBlock - 1) / kKeyBlock;
  const int64_t paired = heads * ((p.tiles + 1) / 2);
  p.split = blocks >= 8 && paired < 4 * (int64_t)sms;
  // one tile per CTA while each finds an SM of its own
  p.tp = !p.split && heads * p.tiles <= sms ? 1 : 2;
  p.pairs = (p.tiles + p.tp - 1) / p.tp;
  const int64_t segs = heads * p.pairs;
  p.segs = segs > INT32_MAX ? -1 : (int)segs;
  const int64_t items = p.split ? segs * blocks : segs;
  p.grid = (int)(items < sms ? items : sms);
  // 16 rows per CTA while that is needed to fill the SMs, eight CTAs on each, then 64 (finding a segment's
  // parts takes a warp as long as two rows)
  p.join_rows = segs * (p.tp * 8) > 8 * (int64_t)sms ? 64 : 16;
  return p;
}

cudaError_t launch_cross_join(const CrossShape& s, const FwdPlan& p, const CrossFwdArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)p.segs, (unsigned)(std::min(p.tp * 128, p.rows) / p.join_rows));
  const bool f16 = s.dtype == SA2_FP16;
  prof_start(st, kAttnFwd);
  const auto kern = s.d == 128 ? (f16 ? cross_join_kernel<128, true> : cross_join_kernel<128, false>)
                               : (f16 ? cross_join_kernel<64, true> : cross_join_kernel<64, false>);
  const cudaError_t e = launch_early(kern, grid, 256, 0, st, s, p, a);
  prof_stop(st, kAttnFwd);
  return e;
}

size_t cross_fwd_partials(const CrossShape& s, const FwdPlan& p) {
  return p.split ? (size_t)(p.grid + p.segs) * p.rows * (s.d + 1) : 0;
}

cudaError_t launch_cross_fwd(const CrossShape& s, const FwdPlan& p, const CUtensorMap& mq, const CUtensorMap& mk,
                             const CUtensorMap& mv, const CUtensorMap& mo, const CrossFwdArgs& a, cudaStream_t st) {
  return launch_any<false>(s, p, mq, mk, mv, mo, CacheRef{}, a, st);
}

cudaError_t launch_cache_fwd(const CrossShape& s, const FwdPlan& p, const CUtensorMap& mk, const CUtensorMap& mv,
                             const CacheRef& c, const CrossFwdArgs& a, cudaStream_t st) {
  const CUtensorMap none{};
  return launch_any<true>(s, p, none, mk, mv, none, c, a, st);
}

}  // namespace sa2
