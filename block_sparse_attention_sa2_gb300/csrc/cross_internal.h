// Declarations shared by the cross- and cache-attention sources (cross_*.cu, cache8.cu).
#pragma once

#include <atomic>
#include <utility>

#include "sa2_internal.h"

namespace sa2 {

// Shape of a cross- or cache-attention call.  M is the key capacity: sequence b attends to its
// first kv_len[b] keys.  Query heads h = hk * G + g share key head hk.
struct CrossShape {
  int B, H, Hkv, G, N, M, d;
  int dtype;  // SA2_BF16 or SA2_FP16
  unsigned long long wait_ns, stall_ns;
};

// A token tensor [B, heads, tokens, d], strides in elements.
struct TokenRef {
  void* p;
  int64_t sb, sh, sn;
};

// The 8-bit cache: e4m3 keys and values and one power-of-two scale per head and 64 tokens.
struct CacheRef {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int64_t sb, sh, sn;  // of k and v
  int C, nsb;          // capacity in tokens, scales per head
};

constexpr int kKeyBlock = 128, kKeyBlockShift = 7;  // keys per step of the kernels on query tiles

// How the work of a forward call is split over CTAs.  A segment is one pair of query tiles of
// one key head; a tile holds nb tokens of all G heads of the group, row = token * G + g.
//   direct (split = 0): a work item is a whole segment, items go round robin over the CTAs;
//   split:              the 128-key blocks of all segments are cut into `grid` equal runs, one
//                       per CTA.  A run may begin or end inside a segment; each part of a
//                       segment leaves its own O and log2 sum exp in slot CTA + segment, and a
//                       second kernel joins a segment's parts in the order of its keys.
struct FwdPlan {
  int nb, tiles;
  int tp, pairs;  // tiles per segment (1 or 2), segments per key head
  int segs;
  int grid;
  int split;
  int shift;  // log2 of the keys per block
  int rows;   // of a slot of the split's partial results
  int join_rows;  // split: rows of a segment per CTA of the kernel that joins the parts
  bool few;   // at most kFewRows query rows per key head: the kernel of cross_decode.cu
};
constexpr int kFewRows = 16;

struct CrossFwdArgs {
  const int32_t* kv_len;  // [B] or null
  TokenRef q;             // read by the cache kernel only (the other one has a tensor map)
  TokenRef o;
  float* lse;     // [B, H, N]
  float* part_o;  // split: [grid + segs][rows][d]
  float* part_l;  // split: [grid + segs][rows], log2 units
  float scale_log2;
  unsigned* status;
};

FwdPlan cross_fwd_plan(const CrossShape& s, int sms);
size_t cross_fwd_partials(const CrossShape& s, const FwdPlan& p);  // floats of part_o + part_l

// The backward's query tiles are those of the forward (nb tokens of all G heads, row = token * G +
// g); its statistics are kept per tile: stats[(head * tiles + tile) * 256 + r] = log2(e) * LSE of
// row r (+inf for rows that hold no query: their P is 0) and [... + 128 + r] = D, head = b * Hkv + hk.
// The dK / dV kernel's work, (key block, query tile) pairs ordered by key head, key block and tile,
// is cut into equal runs, one per CTA (dkv_parts in cross_bwd.cu).  A run that holds a key block's tiles whole writes
// its dK, dV; of the others each run leaves fp32 sums, slot 2 * CTA for the part that the run
// begins with and 2 * CTA + 1 for one that begins inside it, which a second kernel adds in order.
struct BwdPlan {
  int nb, tiles;
  int kblocks;  // 128-key blocks of M
  int dq_grid, grid;
};

struct CrossBwdArgs {
  const int32_t* kv_len;
  TokenRef o, dO, dq, dk, dv;
  const float* lse;
  float* stats;
  float* part;  // [2 * grid][2][128][d]: dK, dV
  float scale, scale_log2;
  unsigned* status;
};

BwdPlan cross_bwd_plan(const CrossShape& s, int sms);
size_t cross_bwd_floats(const CrossShape& s, const BwdPlan& p, size_t* stats);
cudaError_t launch_cross_bwd(const CrossShape& s, const BwdPlan& p, const CUtensorMap& mq, const CUtensorMap& mk,
                             const CUtensorMap& mv, const CUtensorMap& mdo, const CrossBwdArgs& a, cudaStream_t st);

// Allows a kernel its dynamic shared memory, once per device (`done` has a bit for each).
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// A launch that may begin while the kernel before it on the stream, once all of that one's CTAs have
// called kernel_trigger(), still runs: it calls kernel_wait() before it touches what that kernel (or
// one before it) writes.  The cross and cache calls use it between the kernels of one call only (the first is launched
// as usual); of the packed, paged and rotary calls every kernel is launched so, and all of its threads wait before they
// touch memory, so that a grid ends after all before it and the next may trust that.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t st, A&&... args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = (size_t)smem;
  c.stream = st;
  c.attrs = &early;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, std::forward<A>(args)...);
}

// Argument checks that the entry points share (cross_api.cu): limits, the SMs of the current device (152 where
// there is none), a status for a CUDA error, and a token tensor's pointer and strides.
constexpr int kMaxTokens = 1 << 28;
constexpr int kMaxGroup = 64;
int sm_count();
sa2_status cuda_status(cudaError_t e);
sa2_status check_tensor(const sa2_tensor* t, int B, int heads, int G, int tokens, int d, int esz, TokenRef* r);
bool misaligned4(const void* p);

// The device's status word, and the wait settings of the calling thread's next launches
// (sa2_api.cu).
unsigned* status_word();
void wait_settings(unsigned long long* wait_ns, unsigned long long* stall_ns);

// Tensor map of a 16-bit token tensor [B, heads, tokens, d] seen as (d, G, tokens, heads / G,
// B), boxes of 64 channels x box_g heads x box_n tokens with the 128-byte swizzle; tokens past
// the end read as zero (attn_common.cu).
bool make_group_map(CUtensorMap* map, const TokenRef& t, int B, int heads, int G, int tokens, int d, int box_g,
                    int box_n, bool f16);

// Tensor map of the cache's keys or values, boxes of d channels x box_n tokens as they lie.
bool make_cache_map(CUtensorMap* map, const uint8_t* base, const CacheRef& c, int B, int Hkv, int d, int box_n);

cudaError_t launch_cross_fwd(const CrossShape& s, const FwdPlan& p, const CUtensorMap& mq, const CUtensorMap& mk,
                             const CUtensorMap& mv, const CUtensorMap& mo, const CrossFwdArgs& a, cudaStream_t st);
cudaError_t launch_cache_fwd(const CrossShape& s, const FwdPlan& p, const CUtensorMap& mk, const CUtensorMap& mv,
                             const CacheRef& c, const CrossFwdArgs& a, cudaStream_t st);
cudaError_t launch_cross_join(const CrossShape& s, const FwdPlan& p, const CrossFwdArgs& a, cudaStream_t st);
// Few query rows: over 16-bit keys and values (cache = false) or the cache.
cudaError_t launch_few_rows(const CrossShape& s, const FwdPlan& p, const TokenRef& k, const TokenRef& v,
                            const CacheRef& c, bool cache, const CrossFwdArgs& a, cudaStream_t st);
cudaError_t launch_cache_append(const CacheRef& c, int B, int Hkv, int d, int n, bool f16, const TokenRef& k,
                                const TokenRef& v, const int32_t* pos, const int32_t* n_new, unsigned* status,
                                cudaStream_t st);
cudaError_t launch_cache_read(const CacheRef& c, int B, int Hkv, int d, int n, bool f16, const TokenRef& k,
                              const TokenRef& v, const int32_t* pos, unsigned* status, cudaStream_t st);

}  // namespace sa2
