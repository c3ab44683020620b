// Declarations of the paged cache's append (paged.cu).
#pragma once

#include "packed_internal.h"

namespace sa2 {

struct PagedAppendArgs {
  PackedSeqs seqs;
  TokenRef k, v, k_pages, v_pages;  // (the pages' sb is the stride of pages)
  int B, T, Hkv, words;             // words of 16 bytes of a token and head
  int page, pages, width;
  int64_t table_stride;
  unsigned* status;
};

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t st);

}  // namespace sa2
