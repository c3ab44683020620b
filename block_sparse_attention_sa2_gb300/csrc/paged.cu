// The paged cache: new tokens' keys and values into the pages of their sequences.
#include "packed_sched.cuh"
#include "paged.h"

namespace sa2 {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;  // of a token per thread, all of their loads in flight

// A thread moves 16 bytes of one token for up to kHeads key heads; the token's sequence (the last that
// begins at or before it, by bisection), page and place in it are found once.  K and V in one launch (grid z).
// Bound by the bytes, one read and one write of each (3600 tokens of 40 key heads, d = 128: 23 us, 6.4 TB/s), and few
// tokens by the chain place - page - token (one token 2.0 us of a stream of calls, 2.15 where its keys are read last).
__global__ void __launch_bounds__(kThreads) paged_append_kernel(PagedAppendArgs a) {
  kernel_wait();
  kernel_trigger();
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int tok = (int)(i / a.words), word = (int)(i % a.words);
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
    for (int b = threadIdx.x; b < a.B; b += kThreads) {
      const int lo = a.seqs.seq[b], hi = a.seqs.seq[b + 1], held = a.seqs.kv_len[b];
      if (lo < 0 || hi < lo || hi > a.T || held < hi - lo || held > (int64_t)a.width * a.page)
        report_error(a.status, kDevErrBounds);
    }
  if (i >= (int64_t)a.T * a.words) return;
  const TokenRef &src = blockIdx.z ? a.v : a.k, &dst = blockIdx.z ? a.v_pages : a.k_pages;
  const int h0 = blockIdx.y * kHeads;
  const uint16_t* x = static_cast<const uint16_t*>(src.p) + (int64_t)tok * src.sn + h0 * src.sh + word * 8;
  uint4 u[kHeads];  // (on their way while the place is looked up)
#pragma unroll
  for (int q = 0; q < kHeads; ++q)
    if (h0 + q < a.Hkv) u[q] = *reinterpret_cast<const uint4*>(x + q * src.sh);
  int l = 0, h = a.B;
  while (l < h) {  // first b with seq[b + 1] > tok
    const int m = (l + h) >> 1;
    if (a.seqs.seq[m + 1] > tok) h = m; else l = m + 1;
  }
  if (l == a.B || a.seqs.seq[l] > tok) return;  // a token of no sequence
  const int64_t held = a.seqs.kv_len[l], end = a.seqs.seq[l + 1];
  if (held < end - a.seqs.seq[l] || held > (int64_t)a.width * a.page) return;
  const int64_t pos = held - end + tok;
  const int id = a.seqs.table[l * a.table_stride + pos / a.page];
  if (id < 0 || id >= a.pages) {
    report_error(a.status, kDevErrBounds);
    return;
  }
  uint16_t* y = static_cast<uint16_t*>(dst.p) + id * dst.sb + (pos % a.page) * dst.sn + h0 * dst.sh + word * 8;
#pragma unroll
  for (int q = 0; q < kHeads; ++q)
    if (h0 + q < a.Hkv) *reinterpret_cast<uint4*>(y + q * dst.sh) = u[q];
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t st) {
  const int64_t blocks = ((int64_t)a.T * a.words + kThreads - 1) / kThreads;
  const dim3 grid((unsigned)blocks, (unsigned)((a.Hkv + kHeads - 1) / kHeads), 2);
  prof_start(st, kToF16);
  const cudaError_t e = launch_early(paged_append_kernel, grid, kThreads, 0, st, a);
  prof_stop(st, kToF16);
  return e;
}

}  // namespace sa2
