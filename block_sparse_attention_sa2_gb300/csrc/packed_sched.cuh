// Where packed sequences lie, and the order in which the CTAs of the packed kernels work on them.
// The functions here are called by whole warps; one warp of a CTA walks the work and hands it to the
// others through slots in shared memory.
#pragma once

#include "cross_sched.cuh"
#include "packed_internal.h"

namespace sa2 {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ int64_t warp_sum(int64_t x) {
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}
__device__ __forceinline__ int64_t warp_scan(int64_t x) {  // inclusive
  const int lane = threadIdx.x & 31;
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Sequence b: its first token, its tokens, its keys, and the position of its first token among them.
// A number of keys that the table has no room for, or that leaves out new tokens, counts as none.
struct SeqInfo {
  int lo, n, keys, pos;
};
__device__ __forceinline__ bool keys_in_range(const PackedShape& s, int keys, int n) {
  return keys >= n && keys <= (int64_t)s.width * s.page;
}
__device__ __forceinline__ SeqInfo seq_info(const PackedShape& s, const PackedSeqs& q, int b) {
  SeqInfo x;
  x.lo = q.seq[b];
  x.n = q.seq[b + 1] - x.lo;
  x.keys = x.n;
  x.pos = 0;
  if (q.kv_len) {
    const int k = q.kv_len[b];
    const bool ok = keys_in_range(s, k, x.n);
    x.keys = ok ? k : 0;
    x.pos = ok ? k - x.n : 0;
  }
  return x;
}

// True where the sequences' places are in order and within [0, T]; nothing is done in a call where they are
// not.  `report`: one CTA's warp reports that, and lengths out of range.
__device__ __forceinline__ bool seqs_in_order(const PackedShape& s, const PackedSeqs& q, bool report, unsigned* status) {
  bool bad = false, odd = false;
  for (int b = (int)(threadIdx.x & 31); b < s.B; b += 32) {
    const int lo = q.seq[b], hi = q.seq[b + 1];
    const bool out = lo < 0 || hi < lo || hi > s.T;
    bad |= out;
    if (!out) odd |= hi - lo > s.max_new || (q.kv_len && !keys_in_range(s, q.kv_len[b], hi - lo));
  }
  if (report && (bad || odd)) report_error(status, kDevErrBounds);
  return !__any_sync(kFull, bad);
}

// sum over i < n of floor((a i + b) / m), a, b >= 0: whole parts out, then the lattice points under the
// line counted along the other axis.
__device__ __forceinline__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t sum = 0;
  while (n > 0) {
    sum += n * (n - 1) / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const int64_t top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top % m;
    const int64_t t = m;
    m = a;
    a = t;
  }
  return sum;
}

// Key blocks of segment p (of `segs`) of a sequence, at least one, and of its segments 0 .. p - 1.
__device__ __forceinline__ int segment_blocks(const PackedShape& s, const SeqInfo& x, int w, int p) {
  const int64_t to = s.causal ? (int64_t)x.pos + (int64_t)(p + 1) * w : x.keys;
  const int n = key_blocks(to < x.keys ? (int)to : x.keys);
  return n > 0 ? n : 1;
}
__device__ __forceinline__ int64_t blocks_before(const PackedShape& s, const SeqInfo& x, int w, int segs, int p) {
  if (!s.causal || x.keys == 0) return (int64_t)p * segment_blocks(s, x, w, 0);
  const int whole = p < segs ? p : segs - 1;  // all but the last reach w tokens further than the one before
  int64_t n = floor_sum(whole, kKeyBlock, w, (int64_t)x.pos + w + kKeyBlock - 1);
  if (p >= segs && segs > 0) n += segment_blocks(s, x, w, segs - 1);
  return n;
}

// A piece of work of a forward CTA: key blocks [k0, k0 + nb) for the tokens of a segment.
struct Piece2 {
  int qtok;  // its first token in the packed axis,
  int pos;   // that token's position,
  int ntok;  // and the sequence's tokens from there on
  int keys;  // of the sequence
  int k0, nb;
  int hk;    // key head; -1: no work left
  int slot;  // of the partial results; -1: the segment is whole
};

struct PackedWalk {
  const PackedShape& s;
  const PackedPlan& p;
  const PackedFwdArgs& a;
  int b, lo;  // of the piece given out last: its sequence, and that one's first token
  // direct
  int64_t segs, ticket;  // segments of one key head; the next item
  unsigned drawn;        // of the counter, for the item after it (lane 0)
  int section, level, most;
  int64_t at_level, above;  // segments of at least `level`, of more
  // split
  int64_t g, g_end, run, begin;
  SeqInfo x;
  int at, nseg, hk, pr, cut;  // the run's next piece: sequence, its segments, key head, segment, block in it

  __device__ __forceinline__ int segments(int b_) const {
    const int n = b_ < s.B ? a.seqs.seq[b_ + 1] - a.seqs.seq[b_] : 0;
    return n > 0 ? (n + p.w - 1) / p.w : 0;
  }
  // segments with at least `l` before them in their sequence
  __device__ __forceinline__ int64_t segments_from(int l) const {
    int64_t n = 0;
    for (int i = (int)(threadIdx.x & 31); i < s.B; i += 32) {
      const int k = segments(i);
      n += k > l ? k - l : 0;
    }
    return warp_sum(n);
  }

  __device__ __forceinline__ PackedWalk(const PackedShape& s_, const PackedPlan& p_, const PackedFwdArgs& a_)
      : s(s_), p(p_), a(a_), b(0), lo(0), segs(0), ticket(blockIdx.x), drawn(0), section(-1), level(0), most(0),
        at_level(0), above(0), g(0), g_end(0), run(1), begin(0), at(0), nseg(0), hk(0), pr(0), cut(0) {
    if (!seqs_in_order(s, a.seqs, blockIdx.x == 0, a.status)) return;
    const int lane = threadIdx.x & 31;
    if (!p.split) {
      int64_t n = 0;
      for (int i = lane; i < s.B; i += 32) {
        const int k = segments(i);
        n += k;
        most = max(most, k);
      }
      segs = warp_sum(n);
      most = __reduce_max_sync(kFull, most);
      if (p.tickets) draw();
      return;
    }
    int64_t total = 0;
    for (int i = lane; i < s.B; i += 32) total += blocks_of(i);
    total = warp_sum(total);
    run = run_length(total, p.grid);
    begin = g = run * blockIdx.x;
    g_end = g + run < total ? g + run : total;
    if (g >= g_end) return;
    // the run's first sequence, key head, segment and block
    int64_t off = g;
    for (int c = 0;; c += 32) {  // g < total: found
      const int64_t mine = c + lane < s.B ? blocks_of(c + lane) : 0;
      const int64_t to = warp_scan(mine);
      const unsigned in = __ballot_sync(kFull, off < to);
      if (in) {
        const int src = __ffs(in) - 1;
        at = c + src;
        off -= __shfl_sync(kFull, to - mine, src);
        break;
      }
      off -= __shfl_sync(kFull, to, 31);
    }
    x = seq_info(s, a.seqs, at);
    nseg = segments(at);
    const int64_t per = blocks_before(s, x, p.w, nseg, nseg);
    hk = (int)(off / per);
    off -= hk * per;
    int l = 0, h = nseg - 1;  // last segment that begins at or before off
    while (l < h) {
      const int m = (l + h + 1) >> 1;
      if (blocks_before(s, x, p.w, nseg, m) <= off) l = m; else h = m - 1;
    }
    pr = l;
    cut = (int)(off - blocks_before(s, x, p.w, nseg, pr));
  }
  __device__ __forceinline__ int64_t blocks_of(int b_) const {
    const int n = segments(b_);
    return n == 0 ? 0 : s.Hkv * blocks_before(s, seq_info(s, a.seqs, b_), p.w, n, n);
  }
  __device__ __forceinline__ void draw() {
    if ((threadIdx.x & 31) == 0) drawn = atomicAdd(a.counter, 1u);
  }

  __device__ __forceinline__ bool next(Piece2& y, CutRecord& rec) {
    return p.split ? next_of_run(y, rec) : next_item(y);
  }

  __device__ __forceinline__ bool next_item(Piece2& y) {
    const int lane = threadIdx.x & 31;
    if (ticket >= segs * s.Hkv) return false;
    const int sec = (int)(ticket / (segs * p.heads));
    const int64_t in = ticket - sec * segs * p.heads;
    const int heads = min(p.heads, s.Hkv - sec * p.heads);
    const int64_t rank = in / heads;  // segments of a section by falling level, then by sequence
    y.hk = sec * p.heads + (int)(in - rank * heads);
    if (p.tickets) {
      ticket = (int64_t)p.grid + __shfl_sync(kFull, drawn, 0);
      draw();  // (back before it is needed)
    } else {
      ticket = segs * s.Hkv;
    }
    if (sec != section) {
      section = sec;
      level = most - 1;
      above = 0;
      at_level = segments_from(level);
    }
    if (rank >= at_level) {
      int l = 0, h = level - 1;  // the highest level with more than `rank` segments from it on
      while (l < h) {
        const int m = (l + h + 1) >> 1;
        if (segments_from(m) > rank) l = m; else h = m - 1;
      }
      level = l;
      at_level = segments_from(l);
      above = segments_from(l + 1);
    }
    int r = (int)(rank - above);  // of the sequences that reach this level
    for (int c = 0; c < s.B; c += 32) {
      const bool mine = segments(c + lane) > level;
      const unsigned in_c = __ballot_sync(kFull, mine);
      const int n = __popc(in_c);
      if (r < n) {
        const bool it = mine && __popc(in_c & ((1u << lane) - 1)) == r;
        b = c + __ffs(__ballot_sync(kFull, it)) - 1;
        break;
      }
      r -= n;
    }
    const SeqInfo z = seq_info(s, a.seqs, b);
    fill(y, z, level);
    y.k0 = 0;
    y.nb = segment_blocks(s, z, p.w, level);
    y.slot = -1;
    return true;
  }
  __device__ __forceinline__ void fill(Piece2& y, const SeqInfo& z, int seg) {
    lo = z.lo;
    y.qtok = z.lo + seg * p.w;
    y.pos = z.pos + seg * p.w;
    y.ntok = z.n - seg * p.w;
    y.keys = z.keys;
  }

  __device__ __forceinline__ bool next_of_run(Piece2& y, CutRecord& rec) {
    if (g >= g_end) return false;
    const int n = segment_blocks(s, x, p.w, pr);
    const int64_t left = g_end - g;
    fill(y, x, pr);
    y.hk = hk;
    y.k0 = cut;
    y.nb = n - cut < left ? n - cut : (int)left;
    y.slot = y.nb == n ? -1 : 2 * (int)blockIdx.x + (g == begin ? 0 : 1);
    if (cut == 0 && y.nb < n)
      rec = {(int)((g + n - 1) / run) - (int)blockIdx.x + 1, y.slot, y.qtok, y.ntok, hk, 0, 0, 0};
    b = at;
    g += y.nb;
    cut = 0;  // (a run that ends inside the segment has no further piece)
    if (g < g_end && ++pr == nseg) {
      pr = 0;
      if (++hk == s.Hkv) {
        hk = 0;
        do ++at; while (segments(at) == 0);  // g < total: there is one
        x = seq_info(s, a.seqs, at);
        nseg = segments(at);
      }
    }
    return true;
  }
};

}  // namespace sa2
