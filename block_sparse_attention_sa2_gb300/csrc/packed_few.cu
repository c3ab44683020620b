// Attention of few new tokens' rows (at most 16 per key head of a sequence: a single token of up to 16 heads that share
// a key head, or several of fewer) to the keys and values that a paged cache holds of their sequence, on sm_103a.
//
// Every key and value is used for 16 rows at most, so the bytes bound it.  The products, rings and roundings are those of
// cross_decode.cu: a CTA of 8 warps per SM, each with its own steps of 4 KB of K and of V, copied three steps deep by
// cp.async, on mma.sync m16n8k16 (a tcgen05 tile would be an eighth full at most).  Here a step's place comes from the
// table: each lane holds the page of one of the warp's next 32 steps, read a whole round ahead.  A row sees the keys
// up to its token's position.
//
// Measured: 16 single tokens over up to 32760 keys (264450 in all), 40/8 heads of d = 128: 169 us with the parts' join,
// 6.4 TB/s, 96 % of the copy rate.  Short ones are bound by the chain place - page - keys - steps - result of a piece (one
// token over 512 keys, 12 heads: 7.4 us; over 16 keys 4.1).
#include <algorithm>

#include "cross_few.cuh"
#include "cross_softmax.cuh"
#include "packed_sched.cuh"

namespace sa2 {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kStages = 3;
constexpr int kStageBytes = 2 * kFewTileBytes;

// A piece of work takes as long as this many 64-key blocks more than it has: its pages are looked up, the first keys come,
// warps are joined.  Runs count them as blocks that lie before a segment's own; without them some CTAs have ten times the
// others' pieces.  (100 sequences of 64 to 1351 keys, 8 key heads of d = 128: without 120 us, 2 blocks 74, 3 68, 4 63, 5
// 58, 6 58, 8 59; 11 of 1 to 16001, 4 key heads of d = 64: 2 blocks 24.2 us, 4 21.0, 8 18.4, 10 18.4, 16 18.7.)
__host__ __device__ constexpr int piece_blocks(int d) { return 5 * 128 / d; }

// Two numbers rounded to the call's type, the first in the lower half, and back.
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  return F16 ? pack_f16x2(x, y) : pack_bf16x2(x, y);
}
template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&u));
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}

struct FewPiece {
  int b, qtok, pos, n;  // sequence, its first new token, that token's position, new tokens
  int keys, k0, nb;     // of the sequence; 64-key blocks [k0, k0 + nb)
  int hk, slot;         // key head (-1: no work left), slot of the partial results (-1: whole)
};

// The order of work, walked by one warp: segments (sequence, key head) of sequences with few tokens; see PackedPlan.
struct FewWalk {
  const PackedShape& s;
  const PackedSeqs& q;
  const int lane, piece;
  bool whole;
  int64_t g, g_end, run;  // whole: the next segment and their number; else blocks
  int at, nblk, hk, cut;  // cut: from the segment's begin, the first `piece` lie before its blocks
  int chunk, before;  // whole: the 32 sequences looked at last, and how many of this kernel lie before them
  int mine;           // blocks of sequence `lane`

  // Blocks of a sequence of n new tokens; 0: not one of this kernel.
  __device__ __forceinline__ int blocks_of(int n, int held) const {
    if (n < 1 || n > s.few) return 0;
    return max(keys_in_range(s, held, n) ? key_blocks(held, 6) : 0, 1);
  }
  __device__ __forceinline__ int blocks(int b) const {
    return b < s.B ? blocks_of(q.seq[b + 1] - q.seq[b], q.kv_len[b]) : 0;
  }
  __device__ __forceinline__ FewWalk(const PackedShape& s_, const PackedSeqs& q_, bool may_split, unsigned* status)
      : s(s_), q(q_), lane(threadIdx.x & 31), piece(piece_blocks(s_.d)), whole(false), g(0), g_end(0), run(1), at(0), nblk(0), hk(0), cut(0),
        chunk(0), before(0), mine(0) {
    if (threadIdx.x >= 32) return;
    int64_t total = 0;
    int segs = 0, most = 0;
    Faults f;
    for (int b = lane; b < s.B; b += 32) {
      const int lo = q.seq[b], hi = q.seq[b + 1], held = q.kv_len[b];  // (loads that do not wait for each other)
      const int k = f.add(s, lo, hi, true, held) ? 0 : blocks_of(hi - lo, held);
      if (b == lane) mine = k;
      total += k;
      segs += k > 0;
      most = max(most, k);
    }
    if (!f.none_bad(blockIdx.x == 0, status)) return;
    const unsigned all = __reduce_add_sync(kFull, (unsigned)segs) * s.Hkv;  // (the host has seen to it: below 2^31)
    whole = !may_split;
    if (may_split) {
      total = warp_total(total) * s.Hkv;
      most = __reduce_max_sync(kFull, most);
      // Few short segments are never cut: their CTAs share the bandwidth with no others.  Else the kernel that joins parts
      // takes as long as kJoin blocks, and segments' own lengths leave CTAs half a longest one's excess apart.  (12 key
      // heads of d = 128, 32 sequences of up to 300 keys: 15.6 us whole, 19.1 us in runs; 8 key heads, 64 sequences of 700
      // keys: 46.6 us whole, 43.7 us in runs; 16 of up to 32760: 167 us in runs, where the longest segment alone is 17 MB,
      // 420 us at a CTA's share of the bandwidth.)
      constexpr float kJoin = 4.5f;
      const float share = __fdividef(1.f, gridDim.x), mean = all > 0 ? __fdividef(total, all) : 0.f;
      const float in_whole = fmaxf(ceilf(all * share) * (mean + piece) + .5f * (most - mean), most + piece);
      total += (int64_t)piece * all;
      const float in_runs = total * share + piece + kJoin;
      whole = (all <= gridDim.x && most <= kFewWhole) || in_whole <= in_runs;
    }
    if (whole) {
      g = blockIdx.x;
      g_end = all;
      return;
    }
    run = run_length(total, gridDim.x);
    g = run * blockIdx.x;
    g_end = g + run < total ? g + run : total;
    if (g >= g_end) return;
    // the segment of block g
    int64_t off = g;
    for (int c = 0;; c += 32) {  // (found)
      const int k = c == 0 ? mine : blocks(c + lane);
      const int64_t here = k > 0 ? (int64_t)(k + piece) * s.Hkv : 0, to = warp_scan(here);
      const unsigned in = __ballot_sync(kFull, off < to);
      if (in) {
        const int src = __ffs(in) - 1;
        at = c + src;
        nblk = __shfl_sync(kFull, k, src);
        off -= __shfl_sync(kFull, to - here, src);
        break;
      }
      off -= __shfl_sync(kFull, to, 31);
    }
    const int len = nblk + piece;
    hk = off < (1 << 30) ? (int)off / len : (int)(off / len);
    cut = (int)(off - (int64_t)hk * len);
  }
  __device__ __forceinline__ bool next(FewPiece& y, CutRecord& rec) {
    if (g >= g_end) return false;
    if (whole) {  // segment g: the key head of a sequence of this kernel, in order
      const int seg = (int)((unsigned)g / (unsigned)s.Hkv);
      hk = (int)g - seg * s.Hkv;
      for (;; chunk += 32) {  // (found)
        const int k = chunk == 0 ? mine : blocks(chunk + lane);
        const unsigned some = __ballot_sync(kFull, k > 0);
        const unsigned in = __ballot_sync(kFull, k > 0 && before + __popc(some & ((1u << lane) - 1)) == seg);
        if (in) {
          at = chunk + __ffs(in) - 1;
          nblk = __shfl_sync(kFull, k, __ffs(in) - 1);
          break;
        }
        before += __popc(some);
      }
    }
    const SeqInfo x = seq_info(s, q, at);
    y.b = at;
    y.qtok = x.lo;
    y.pos = x.pos;
    y.n = x.n;
    y.keys = x.keys;
    y.hk = hk;
    if (whole) {
      y.k0 = 0;
      y.nb = nblk;
      y.slot = -1;
      g += gridDim.x;
      return true;
    }
    const int64_t left = g_end - g;
    const int len = nblk + piece, end = len - cut < left ? len : cut + (int)left;
    y.k0 = max(cut - piece, 0);
    y.nb = end - piece - y.k0;
    if (y.nb <= 0) return false;  // the run ends before the segment's first block
    y.slot = y.nb == nblk ? -1 : 2 * (int)blockIdx.x + (y.k0 == 0);
    if (y.k0 == 0 && y.nb < nblk)
      rec = {(int)((g - cut + len - 1) / run) - (int)blockIdx.x + 1, y.slot, y.qtok, y.n, hk, 0, 0, 0};
    g += end - cut;
    cut = 0;
    if (g < g_end && ++hk == s.Hkv) {
      hk = 0;
      do ++at; while (blocks(at) == 0);  // g < total: there is one
      nblk = blocks(at);
    }
    return true;
  }
};

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    packed_few_kernel(const __grid_constant__ PackedShape s, const __grid_constant__ PackedPlan plan,
                      const __grid_constant__ PackedFwdArgs a) {
  using T = FewTile<D, false>;
  constexpr int kNT = T::kKeys / 8;   // 8-key tiles of S per step
  constexpr int kCT = D / 8;          // 8-channel tiles of O
  constexpr int kKS = D / 16;         // k-steps of S
  constexpr int kKC = T::kChunks / 4;  // K chunks per thread and key
  constexpr int kIds = T::kKeys / 16;  // places in the table that a step can touch
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float warp_m[kWarps][kFewRows], warp_l[kWarps][kFewRows];
  __shared__ FewPiece piece;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * kStages * kStageBytes;
  const uint32_t ring_u = smem_u32(ring);
  kernel_wait();
  kernel_trigger();
  const int page_shift = __ffs(s.page) - 1;

  FewWalk walk(s, a.seqs, plan.few_split, a.status);  // (walked on by warp 0)
  CutRecord rec{0, 0, 0, 0, 0, 0, 0, 0};
  for (;;) {
    if (warp == 0) {
      FewPiece y;
      if (!walk.next(y, rec)) y.hk = -1;
      if (lane == 0) piece = y;
    }
    __syncthreads();
    const FewPiece x = piece;
    if (x.hk < 0) break;
    const int rows = x.n * s.G;
    const int key0 = x.k0 << 6, key1 = min(x.keys, (x.k0 + x.nb) << 6);
    const uint16_t* kp = static_cast<const uint16_t*>(a.k.p) + x.hk * a.k.sh;
    const uint16_t* vp = static_cast<const uint16_t*>(a.v.p) + x.hk * a.v.sh;
    const int32_t* row = a.seqs.table + x.b * s.table_stride;
    // Q's fragments: rows g and g + 8; of each, this thread's channels in the order of its K chunks (asked for first:
    // they are back when the pages' numbers are)
    uint32_t w[2][2 * kKS];
    int lim[2];  // keys before which a row's keys end
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int r = g + 8 * hf, n = r / s.G, h = x.hk * s.G + r - n * s.G;
      const bool live = r < rows;
      lim[hf] = s.causal && live ? min(key1, x.pos + n + 1) : key1;
      const uint16_t* qp = static_cast<const uint16_t*>(a.q.p) + h * a.q.sh + (int64_t)(x.qtok + n) * a.q.sn;
#pragma unroll
      for (int i = 0; i < 2 * kKS; i += 4) {  // a chunk: values 2 i .. 2 i + 7 of the thread's list
        const int ci = 2 * i / T::kPer, c = 2 * t + (ci & 1) + 8 * (ci >> 1);
        const uint4 u = live ? *reinterpret_cast<const uint4*>(qp + c * T::kPer) : make_uint4(0, 0, 0, 0);
        w[hf][i] = u.x;
        w[hf][i + 1] = u.y;
        w[hf][i + 2] = u.z;
        w[hf][i + 3] = u.w;
      }
    }
    // step i of this warp: keys from key0 + (i * kWarps + warp) * kKeys on
    const int steps_all = (key1 - key0 + T::kKeys - 1) / T::kKeys;
    const int steps = steps_all > warp ? (steps_all - warp + kWarps - 1) / kWarps : 0;
    // the pages of steps 32 j + lane: of their first 16 keys, and of their second (d = 64), -1 where there are none
    int ids[2], next_ids[2];
    auto look_up = [&](int i, int (&id)[2]) {
#pragma unroll
      for (int p = 0; p < kIds; ++p) {
        const int key = key0 + (i * kWarps + warp) * T::kKeys + 16 * p;
        id[p] = -1;
        if (i < steps && key < key1) {
          id[p] = row[key >> page_shift];
          if (id[p] < 0 || id[p] >= s.pages) {
            report_error(a.status, kDevErrBounds);
            id[p] = -1;  // reads as zeros
          }
        }
      }
    };
    look_up(lane, next_ids);
    auto copy_step = [&](int i) {
      if ((i & 31) == 0) {  // (every warp comes here for each of its steps in turn)
#pragma unroll
        for (int p = 0; p < kIds; ++p) ids[p] = next_ids[p];
        look_up(i + 32 + lane, next_ids);
      }
      int id[kIds];
#pragma unroll
      for (int p = 0; p < kIds; ++p) id[p] = __shfl_sync(kFull, ids[p], i & 31);
      if (i < steps) {
        const uint32_t dst = ring_u + (i % kStages) * kStageBytes;
        constexpr int kRows = 32 / T::kChunks, kPer = 8 / kIds;  // keys of a warp's copy; copies of 16 keys
        const int r0 = lane / T::kChunks, c = lane % T::kChunks;
#pragma unroll
        for (int p = 0; p < kIds; ++p) {  // 16 keys from a multiple of 16 on lie in one page
          const int key = key0 + (i * kWarps + warp) * T::kKeys + 16 * p;
          const int64_t off = (id[p] >= 0 ? id[p] : 0) * a.k.sb + ((key & (s.page - 1)) + r0) * a.k.sn + c * 8;
          const int left = id[p] >= 0 ? key1 - key - r0 : 0;
#pragma unroll
          for (int q = 0; q < kPer; ++q) {
            const int64_t at = off + (int64_t)(q * kRows) * a.k.sn;  // (V's pages have K's strides)
            copy16(dst + T::at(16 * p + q * kRows + r0, c), kp + at, q * kRows < left);
            copy16(dst + kFewTileBytes + T::at(16 * p + q * kRows + r0, c), vp + at, q * kRows < left);
          }
        }
      }
      copy_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) copy_step(i);

    uint32_t qf[kKS][4];
#pragma unroll
    for (int k = 0; k < kKS; ++k)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        qf[k][hf] = w[hf][2 * k];
        qf[k][2 + hf] = w[hf][2 * k + 1];
      }

    float o[kCT][4] = {};
    float m_used[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};  // reference of the exponentials; sum of exp2(s) relative to it
    const float mul = a.scale_log2;
    for (int i = 0; i < steps; ++i) {
      copy_step(i + kStages - 1);
      copy_wait<kStages - 1>();
      __syncwarp();
      const uint8_t* kt = ring + (i % kStages) * kStageBytes;
      const uint8_t* vt = kt + kFewTileBytes;
      const int base = key0 + (i * kWarps + warp) * T::kKeys;
      // S: tile j has keys 8 j .. 8 j + 7; thread: rows g, g + 8, keys 8 j + 2 t, + 1
      float sc[kNT][4];
#pragma unroll
      for (int j = 0; j < kNT; ++j) {
        sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
        uint32_t w[4 * kKC];
#pragma unroll
        for (int c = 0; c < kKC; ++c) {
          const int ch = 2 * t + (c & 1) + 8 * (c >> 1);
          const uint4 u = *reinterpret_cast<const uint4*>(kt + T::at(8 * j + g, ch));
          w[4 * c] = u.x;
          w[4 * c + 1] = u.y;
          w[4 * c + 2] = u.z;
          w[4 * c + 3] = u.w;
        }
#pragma unroll
        for (int k = 0; k < kKS; ++k) mma16816<F16>(sc[j], qf[k], w[2 * k], w[2 * k + 1]);
      }
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < kNT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (base + 8 * j + 2 * t + (q & 1) >= lim[q >> 1]) sc[j][q] = -INFINITY;
          mx[q >> 1] = fmaxf(mx[q >> 1], sc[j][q]);
        }
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        mx[hf] *= mul;
        mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(kFull, mx[hf], 1));
        mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(kFull, mx[hf], 2));
      }
      if (i == 0) {
        m_used[0] = fmaxf(mx[0], kLeastRef);
        m_used[1] = fmaxf(mx[1], kLeastRef);
      } else if (__any_sync(kFull, mx[0] > m_used[0] + kRescaleThreshold || mx[1] > m_used[1] + kRescaleThreshold)) {
        float al[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          // (a row's reference follows from its own scores only)
          const float m = mx[hf] > m_used[hf] + kRescaleThreshold ? mx[hf] : m_used[hf];
          al[hf] = m == m_used[hf] ? 1.f : ex2(m_used[hf] - m);
          l[hf] *= al[hf];
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
      // P in the layout of an A operand: 16 keys (tiles 2 k, 2 k + 1) per k-step; rounded, and what the rounding left.
      // (O is then as exact as its own type; with P rounded alone a token's O over 512 keys was 1.4 to 1.55 times as far
      // off as its own rounding.  The second products take 1 to 3 % at d = 128, up to 9 % at d = 64.)
      uint32_t pf[kNT / 2][4], pr[kNT / 2][4];
#pragma unroll
      for (int j = 0; j < kNT; ++j) {
        float p[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          p[q] = ex2(fmaf(sc[j][q], mul, -m_used[q >> 1]));
          l[q >> 1] += p[q];
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint32_t u = pack2<F16>(p[2 * hf], p[2 * hf + 1]);
          const float2 r = unpack2<F16>(u);
          pf[j >> 1][2 * (j & 1) + hf] = u;
          pr[j >> 1][2 * (j & 1) + hf] = pack2<F16>(p[2 * hf] - r.x, p[2 * hf + 1] - r.y);
        }
      }
      // O += P V: keys 16 k + 2 t, + 1 and 16 k + 8 + 2 t, + 1; channels of chunk g (+ 8 i)
#pragma unroll
      for (int k = 0; k < kNT / 2; ++k) {
#pragma unroll
        for (int i8 = 0; i8 < D / 64; ++i8) {
          uint32_t v[4][4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = 16 * k + 2 * t + (q & 1) + 8 * (q >> 1);
            *reinterpret_cast<uint4*>(v[q]) = *reinterpret_cast<const uint4*>(vt + T::at(r, g + 8 * i8));
          }
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t e0 = __byte_perm(v[0][w], v[1][w], 0x5410), e1 = __byte_perm(v[2][w], v[3][w], 0x5410);
            const uint32_t f0 = __byte_perm(v[0][w], v[1][w], 0x7632), f1 = __byte_perm(v[2][w], v[3][w], 0x7632);
            mma16816<F16>(o[8 * i8 + 2 * w], pr[k], e0, e1);
            mma16816<F16>(o[8 * i8 + 2 * w + 1], pr[k], f0, f1);
            mma16816<F16>(o[8 * i8 + 2 * w], pf[k], e0, e1);
            mma16816<F16>(o[8 * i8 + 2 * w + 1], pf[k], f0, f1);
          }
        }
      }
      __syncwarp();  // the step's stage is read before its next copy
    }
    // ---- join the warps: O relative to the largest of their references
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      l[hf] += __shfl_xor_sync(kFull, l[hf], 1);
      l[hf] += __shfl_xor_sync(kFull, l[hf], 2);
      if (t == 0) {
        warp_m[warp][g + 8 * hf] = steps > 0 ? m_used[hf] : -INFINITY;
        warp_l[warp][g + 8 * hf] = steps > 0 ? l[hf] : 0.f;
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
          // channel tile c: value c % 8 of chunk n + 8 (c / 8)
          os[(warp * kFewRows + r) * kPitch + (n + 8 * (c / 8)) * 8 + c % 8] = o[c][q];
        }
    }
    __syncthreads();
    for (int i = tid; i < rows * (D / 2); i += kThreads) {
      const int r = i / (D / 2), ch = i % (D / 2) * 2;
      float m = -INFINITY;
      bool nan = false;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        nan |= warp_m[w][r] != warp_m[w][r];
        m = fmaxf(m, warp_m[w][r]);
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
        sum = fmaf(f, warp_l[w][r], sum);
      }
      const float inv = inverse_sum(sum);  // (0: no keys, or no score above -inf)
      const float lse2 = sum == 0.f ? -INFINITY : m + __log2f(sum);
      const int n = r / s.G, h = x.hk * s.G + r - n * s.G;
      if (x.slot >= 0) {
        const int64_t pr = (int64_t)x.slot * kFewRows + r;
        *reinterpret_cast<float2*>(a.few.o + pr * D + ch) = make_float2(v0 * inv, v1 * inv);
        if (ch == 0) a.few.l[pr] = lse2;
      } else {
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o.p) + h * a.o.sh + (int64_t)(x.qtok + n) * a.o.sn + ch) =
            F16 ? pack_f16x2(v0 * inv, v1 * inv) : pack_bf16x2(v0 * inv, v1 * inv);
        if (ch == 0) a.lse[(int64_t)h * s.T + x.qtok + n] = lse2 * 0.69314718055994531f;
      }
    }
    __syncthreads();  // before the next piece's copies
  }
  if (plan.few_split && tid == 0) a.few.rec[blockIdx.x] = rec;
}

template <int D, bool F16>
cudaError_t launch_t(const PackedShape& s, const PackedPlan& p, const PackedFwdArgs& a, cudaStream_t st) {
  constexpr int kBytes = kWarps * kStages * kStageBytes;
  static_assert(kWarps * kFewRows * (D + 4) * 4 <= kBytes && kBytes + 2048 <= (int)kMaxDynSmem, "shared memory");
  auto kern = packed_few_kernel<D, F16>;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = allow_smem(kern, kBytes, allowed);
  if (e != cudaSuccess) return e;
  return launch_early(kern, dim3((unsigned)p.few_grid), kThreads, kBytes, st, s, p, a);
}

}  // namespace

cudaError_t launch_packed_few(const PackedShape& s, const PackedPlan& p, const PackedFwdArgs& a, cudaStream_t st) {
  const bool f16 = s.dtype == SA2_FP16;
  if (s.d == 128) return f16 ? launch_t<128, true>(s, p, a, st) : launch_t<128, false>(s, p, a, st);
  return f16 ? launch_t<64, true>(s, p, a, st) : launch_t<64, false>(s, p, a, st);
}

}  // namespace sa2
