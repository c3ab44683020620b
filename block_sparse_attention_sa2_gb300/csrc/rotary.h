// Declarations of the rotary positions (rotary.cu).
#pragma once

#include "cross_internal.h"

namespace sa2 {

struct RotaryTensor {
  TokenRef x, y;  // from, to
  int heads;
};

struct RotaryArgs {
  RotaryTensor t[2];    // the second may have no heads
  int N;                // tokens of a sequence
  int64_t tokens;       // of all
  const int64_t* pairs;  // [half][2]: turns per position (64 bits behind the point), axis
  const int32_t* pos;   // [axes][B][N]
  int64_t pos_axis, pos_b;
  int half, axes;       // pairs, axes of the positions
  float gain;
  unsigned* status;
  int inverse, in_place;
  // words of 16 bytes that hold turned channels, of both kinds; heads per thread; runs of heads of the first tensor
  int turned, words, per, chunks;
  int toks;  // tokens of a CTA
};

cudaError_t launch_rotary(const RotaryArgs& a, int d, int dtype, bool half_layout, int sms, cudaStream_t st);

}  // namespace sa2
