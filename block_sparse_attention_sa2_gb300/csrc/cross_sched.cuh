// The order of work of the cross- and cache-attention forward kernels (FwdPlan): every role of a
// CTA, and the kernel that joins split segments, walks the same sequence of pieces.
#pragma once

#include "cross_internal.h"

namespace sa2 {

// See launch_early.
__device__ __forceinline__ void kernel_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void kernel_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The least reference of a row's exponentials: finite, so that scores of -inf (an infinite key) count as 0 against it
// even where a block, a warp's step or a part has no other.
constexpr float kLeastRef = -3.4028234663852886e38f;
// 1 / l; 0 for a row without any score above -inf, whose O is then 0 and whose LSE is -inf.
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.f ? 0.f : 1.f / l; }

// The factor from products to scores of a block of cached keys.  It is a product of three numbers, of which two are
// powers of two as small as 2^-112 and 2^-100: kept above 0, where every score is 0 all the same (the products are
// below 2^32), since scores behind the last key are -inf and 0 times that is NaN.
__device__ __forceinline__ float score_factor(float row, float key_scale) {
  const float x = row * key_scale;
  return x < 0x1p-126f ? 0x1p-126f : x;
}

// Keys of sequence b, clamped to [0, M].
__device__ __forceinline__ int key_count(const int32_t* kv_len, int b, int M) {
  const int n = kv_len ? kv_len[b] : M;
  return n < 0 ? 0 : (n > M ? M : n);
}
// Blocks of 2^shift keys.
__device__ __forceinline__ int key_blocks(int keys, int shift = kKeyBlockShift) {
  return (keys + (1 << shift) - 1) >> shift;
}

// Key blocks of all segments together; called by whole warps.
__device__ __forceinline__ int64_t total_key_blocks(const CrossShape& s, const int32_t* kv_len, int pairs,
                                                    int shift = kKeyBlockShift) {
  int64_t n = 0;
  for (int b = (int)(threadIdx.x & 31); b < s.B; b += 32) n += key_blocks(key_count(kv_len, b, s.M), shift);
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n * s.Hkv * pairs;
}
// Key blocks of one CTA's run in split mode.
__device__ __forceinline__ int64_t run_length(int64_t total, int grid) {
  const int64_t n = (total + grid - 1) / grid;
  return n > 0 ? n : 1;
}

// A part of a segment: blocks [k0, k0 + nb) of the keys of key head hk of sequence b, for the
// tile pair `pair`.
struct Piece {
  int b, hk, pair, seg;
  int k0, nb;
  int keys;  // of the sequence
  int mask;  // tiles of the pair that the piece is for: 1, 2 or 3 (0: none left of its pair)
};

// Direct mode: segments that do not fill a last round of the grid, and whose tiles can go one by one
// without another round, are taken so, since a single tile takes less time than a pair (24 heads x 8192 x
// 4096, d = 128: 324 us with pairs alone, 313).
__device__ __forceinline__ int single_segs(const FwdPlan& p) {
  const int rest = p.segs % p.grid;
  return !p.split && p.tp == 2 && 2 * rest <= p.grid ? rest : 0;
}

struct PieceIter {
  const CrossShape& s;
  const FwdPlan& p;
  const int32_t* kv_len;
  int64_t g, g_end;  // split: the CTA's run of blocks; direct: the next segment in g
  int paired;        // direct: segments taken whole
  int b;             // split: sequence of block g, and the blocks before it
  int64_t base;

  __device__ __forceinline__ PieceIter(const CrossShape& s_, const FwdPlan& p_, const int32_t* kv_len_)
      : s(s_), p(p_), kv_len(kv_len_), paired(0), b(0), base(0) {
    if (p.split) {
      const int64_t total = total_key_blocks(s, kv_len, p.pairs, p.shift);
      const int64_t run = run_length(total, p.grid);
      g = run * blockIdx.x;
      g_end = g + run < total ? g + run : total;
    } else {
      g = blockIdx.x;
      const int single = single_segs(p);
      paired = p.segs - single;
      g_end = p.segs + single;
    }
  }
  __device__ __forceinline__ bool next(Piece& x) {
    if (g >= g_end) return false;
    const int per_b = s.Hkv * p.pairs;
    if (!p.split) {
      const int k = (int)g - paired;
      x.seg = k < 0 ? (int)g : paired + (k >> 1);
      x.mask = k < 0 ? 3 : 1 << (k & 1);
      x.b = x.seg / per_b;
      x.keys = key_count(kv_len, x.b, s.M);
      x.k0 = 0;
      x.nb = key_blocks(x.keys, p.shift);
      g += p.grid;
    } else {
      int nk = key_blocks(key_count(kv_len, b, s.M), p.shift);
      while (g >= base + (int64_t)nk * per_b) {  // g < total: ends at a sequence with keys
        base += (int64_t)nk * per_b;
        ++b;
        nk = key_blocks(key_count(kv_len, b, s.M), p.shift);
      }
      x.b = b;
      x.keys = key_count(kv_len, b, s.M);
      const int64_t off = g - base;
      x.seg = b * per_b + (int)(off / nk);
      x.k0 = (int)(off % nk);
      const int64_t left = g_end - g;
      x.nb = nk - x.k0 < left ? nk - x.k0 : (int)left;
      g += x.nb;
      x.mask = 3;
    }
    const int in_b = x.seg - x.b * per_b;
    x.hk = in_b / p.pairs;
    x.pair = in_b - x.hk * p.pairs;
    if (p.tp == 1 || 2 * x.pair + 1 == p.tiles) x.mask &= 1;
    return true;
  }
};

}  // namespace sa2
