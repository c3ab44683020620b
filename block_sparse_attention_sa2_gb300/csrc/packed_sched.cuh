// Where packed sequences lie, and the order in which the CTAs of the packed kernels work on them.
// The functions here are called by whole warps; one warp of a CTA walks the work and hands it to the
// others through slots in shared memory.
#pragma once

#include "cross_sched.cuh"
#include "packed_internal.h"

namespace sa2 {

constexpr unsigned kFull = 0xffffffffu;

// The thread's index, read again: what is made of it is not kept in registers over other loops.
__device__ __forceinline__ int thread_anew() {
  int x;
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(x));
  return x;
}

__device__ __forceinline__ int64_t warp_sum(int64_t x) {
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}
// The same of numbers below 2^52, none negative, in two instructions (and more registers).
__device__ __forceinline__ int64_t warp_total(int64_t x) {
  const unsigned lo = __reduce_add_sync(kFull, (unsigned)x & 0x3FFFFFFu), hi = __reduce_add_sync(kFull, (unsigned)(x >> 26));
  return (int64_t)lo + ((int64_t)hi << 26);
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

// What is wrong with the sequences that it has been shown: places out of order or outside of [0, T], lengths out of range.
struct Faults {
  bool bad = false, odd = false;
  __device__ __forceinline__ bool add(const PackedShape& s, int lo, int hi, bool paged, int held) {
    const bool out = lo < 0 || hi < lo || hi > s.T;
    bad |= out;
    if (!out) odd |= hi - lo > s.max_new || (paged && !keys_in_range(s, held, hi - lo));
    return out;
  }
  // For a whole warp: whether the places are in order; `report`: it reports what it has found.
  __device__ __forceinline__ bool none_bad(bool report, unsigned* status) const {
    if (report && (bad || odd)) report_error(status, kDevErrBounds);
    return !__any_sync(kFull, bad);
  }
};
// True where the sequences' places are in order and within [0, T]; nothing is done in a call where they are
// not.  `report`: one CTA's warp reports that, and lengths out of range.
__device__ __forceinline__ bool seqs_in_order(const PackedShape& s, const PackedSeqs& q, bool report, unsigned* status) {
  Faults f;
  for (int b = (int)(threadIdx.x & 31); b < s.B; b += 32) {
    const int lo = q.seq[b], hi = q.seq[b + 1], held = q.kv_len ? q.kv_len[b] : 0;  // (loads that do not wait for each other)
    f.add(s, lo, hi, q.kv_len, held);
  }
  return f.none_bad(report, status);
}

// sum over i < n of floor((a i + b) / m), a, b >= 0: whole parts out, then the lattice points under the line
// counted along the other axis.  In 32 bits but for the sums: with a <= m or n a < 2^31 and b < 2^31 no
// number passes 2^31 (a n + b is below m n + m after the first step, and shrinks).
__device__ __forceinline__ int64_t floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
  int64_t sum = 0;
  while (n > 0) {
    sum += (int64_t)n * (n - 1) / 2 * (a / m) + (int64_t)n * (b / m);
    a %= m;
    b %= m;
    const unsigned top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top % m;
    const unsigned t = m;
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
  int64_t n = floor_sum(whole, kKeyBlock, w, (unsigned)x.pos + w + kKeyBlock - 1);
  if (p >= segs && segs > 0) n += segment_blocks(s, x, w, segs - 1);
  return n;
}

__device__ __forceinline__ int segments_of(const PackedShape& s, const PackedSeqs& q, int w, int b) {
  const int n = b < s.B ? q.seq[b + 1] - q.seq[b] : 0;
  return n > s.few ? (n + w - 1) / w : 0;
}

// Work items, `parts` of every segment of w tokens of every key head, taken from a counter by the CTAs (the
// first by their own numbers): in sections of `heads` key heads; in a section by the segment's place in its
// sequence, the last ones first (rising: the first ones first), then by sequence, head and part.
struct ItemQueue {
  const PackedShape& s;
  const PackedSeqs& q;
  const int w, parts, heads, grid;
  const bool rising;
  unsigned* counter;   // null: no more items than CTAs
  bool first;
  bool in_order;   // see seqs_in_order; where not, there are no items
  int mine;        // segments of sequence `lane`
  int segs;        // of one key head (below 2^29)
  int section, level, most;
  int before, upto;  // segments that come before this level, and with it

  __device__ __forceinline__ ItemQueue(const PackedShape& s_, const PackedSeqs& q_, int w_, int parts_, int heads_,
                                       int grid_, bool rising_, unsigned* counter_, bool report, unsigned* status)
      : s(s_), q(q_), w(w_), parts(parts_), heads(heads_), grid(grid_), rising(rising_), counter(counter_),
        first(true), in_order(false), mine(0), segs(0), section(-1), level(0), most(0), before(0), upto(0) {
    const int lane = threadIdx.x & 31;
    Faults f;
    int n = 0;
    for (int i = lane; i < s.B; i += 32) {
      const int lo = q.seq[i], hi = q.seq[i + 1], held = q.kv_len ? q.kv_len[i] : 0;  // (loads that do not wait for each other)
      const int k = !f.add(s, lo, hi, q.kv_len, held) && hi - lo > s.few ? (hi - lo + w - 1) / w : 0;
      if (i == lane) mine = k;
      n += k;
      most = max(most, k);
    }
    in_order = f.none_bad(report, status);
    if (!in_order) return;
    segs = __reduce_add_sync(kFull, n);
    most = __reduce_max_sync(kFull, most);
  }
  __device__ __forceinline__ int segments(int b) const { return b < 32 ? mine : segments_of(s, q, w, b); }  // b % 32 = lane
  // Segments that come in order before those of place l.
  __device__ __forceinline__ int ahead_of(int l) const {
    int n = 0;
    for (int i = (int)(threadIdx.x & 31); i < s.B; i += 32) {
      const int k = segments(i);
      n += rising ? min(k, l) : max(k - l - 1, 0);
    }
    return __reduce_add_sync(kFull, n);
  }
  __device__ __forceinline__ bool next(int& b, int& seg, int& hk, int& part) {
    const int lane = threadIdx.x & 31;
    // (the host has seen to it that all items together are below 2^31)
    const unsigned per_head = (unsigned)segs * parts;
    // An item is taken only when the CTA is about to need it (its loads for the one before are all issued): taken one
    // ahead, with three or four items to a CTA, the long ones stayed where they had been given out (5 sequences of
    // 514 to 3314 tokens, 8 key heads: CTAs of 187 to 376 us in the dK, dV kernel).
    unsigned item = blockIdx.x;
    if (!first) {
      if (!counter) return false;
      unsigned t = 0;
      if (lane == 0) t = atomicAdd(counter, 1u);
      item = (unsigned)grid + __shfl_sync(kFull, t, 0);
    }
    first = false;
    if (item >= per_head * (unsigned)s.Hkv) return false;
    const unsigned per_section = per_head * (unsigned)heads;  // (of a full one)
    const int sec = (int)(item / per_section);
    const unsigned in = item - (unsigned)sec * per_section, width = (unsigned)(min(heads, s.Hkv - sec * heads) * parts);
    const int rank = (int)(in / width), rest = (int)(in - (unsigned)rank * width);
    hk = sec * heads + rest / parts;
    part = rest % parts;
    if (sec != section) {
      section = sec;
      set_level(rising ? 0 : most - 1);
    }
    if (rank >= upto) {
      // places are looked through in their order, d steps behind this one: the last with no more than `rank` ahead
      int l = 1, h = rising ? most - 1 - level : level;
      while (l < h) {
        const int m = (l + h + 1) >> 1;
        if (ahead_of(rising ? level + m : level - m) <= rank) l = m; else h = m - 1;
      }
      set_level(rising ? level + l : level - l);
    }
    seg = level;
    int r = rank - before;  // of the sequences that have this place
    for (int c = 0; c < s.B; c += 32) {
      const bool has = segments(c + lane) > level;
      const unsigned in_c = __ballot_sync(kFull, has);
      const int n = __popc(in_c);
      if (r < n) {
        const bool it = has && __popc(in_c & ((1u << lane) - 1)) == r;
        b = c + __ffs(__ballot_sync(kFull, it)) - 1;
        break;
      }
      r -= n;
    }
    return true;
  }
  __device__ __forceinline__ void set_level(int l) {
    level = l;
    before = ahead_of(l);
    upto = rising ? ahead_of(l + 1) : (l > 0 ? ahead_of(l - 1) : segs);
  }
};

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
  const PackedSeqs& q;
  ItemQueue queue;  // direct
  int b, lo;        // of the piece given out last: its sequence, and that one's first token
  // split: the run's blocks, and its next piece: sequence, its segments, key head, segment, block in it
  int64_t g, g_end, run, begin;
  SeqInfo x;
  int at, nseg, hk, pr, cut;

  __device__ __forceinline__ PackedWalk(const PackedShape& s_, const PackedPlan& p_, const PackedFwdArgs& a)
      : s(s_), p(p_), q(a.seqs),
        queue(s_, a.seqs, p_.w, 1, p_.heads, p_.grid, false, p_.tickets ? a.counter : nullptr, blockIdx.x == 0, a.status),
        b(0), lo(0), g(0), g_end(0), run(1), begin(0), at(0), nseg(0), hk(0), pr(0), cut(0) {
    if (!queue.in_order || !p.split) return;
    const int lane = threadIdx.x & 31;
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
    x = seq_info(s, q, at);
    nseg = segments_of(s, q, p.w, at);
    const int64_t per = blocks_before(s, x, p.w, nseg, nseg);
    hk = (int)(off / per);
    off -= hk * per;
    int h = nseg;  // the last segment that begins at or before off, 32 of them looked at per step
    while (h - pr > 1) {
      const int step = (h - pr + 31) >> 5, c = pr + lane * step;
      pr += (31 - __clz(__ballot_sync(kFull, c < h && blocks_before(s, x, p.w, nseg, c) <= off))) * step;
      h = min(h, pr + step);
    }
    cut = (int)(off - blocks_before(s, x, p.w, nseg, pr));
  }
  __device__ __forceinline__ int64_t blocks_of(int b_) const {
    const int n = segments_of(s, q, p.w, b_);
    return n == 0 ? 0 : s.Hkv * blocks_before(s, seq_info(s, q, b_), p.w, n, n);
  }

  __device__ __forceinline__ bool next(Piece2& y, CutRecord& rec) {
    return p.split ? next_of_run(y, rec) : next_item(y);
  }
  __device__ __forceinline__ bool next_item(Piece2& y) {
    int seg, part;
    if (!queue.next(b, seg, y.hk, part)) return false;
    const SeqInfo z = seq_info(s, q, b);
    fill(y, z, seg);
    y.k0 = 0;
    y.nb = segment_blocks(s, z, p.w, seg);
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
        do ++at; while (segments_of(s, q, p.w, at) == 0);  // g < total: there is one
        x = seq_info(s, q, at);
        nseg = segments_of(s, q, p.w, at);
      }
    }
    return true;
  }
};

// Where a sequence's query tiles have their records: tile t of sequence b has record first_record + t of its
// key head.  No two sequences share one, since lo / nb + b grows by at least the tiles of what lies between.
__device__ __forceinline__ int first_record(int lo, int nb, int b) { return lo / nb + b; }
// The last sequence whose first record (of runs of nb tokens) is at or before i; 32 of them looked at per step.
__device__ __forceinline__ int sequence_of_record(const PackedShape& s, const PackedSeqs& q, int nb, int i) {
  const int lane = threadIdx.x & 31;
  int l = 0, h = s.B;
  while (h - l > 1) {
    const int step = (h - l + 31) >> 5, c = l + lane * step;
    const unsigned m = __ballot_sync(kFull, c < h && first_record(q.seq[c], nb, c) <= i);
    const int n = m ? 32 - __clz(m) : 1;  // (places in order: the lowest lanes)
    l += (n - 1) * step;
    h = min(h, l + step);
  }
  return l;
}

}  // namespace sa2
