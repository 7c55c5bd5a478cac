// Internal declarations of the operators on prompts' rows: rotary positions and
// the attention of packed prompts.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "bsa.h"
#include "bsa_launch.h"

namespace bsa {

// Rows [batch][heads][tokens][d] of 2-byte elements; strides in elements.
struct RopeRows {
  const uint16_t* p;
  uint16_t* o;
  long long sb, sh, st, ob, oh, ot;
};

struct RopeParams {
  RopeRows q, k;
  const uint64_t* steps;
  const int32_t* positions;  // [B][T] or nullptr: 0 .. T-1
  float amp;
  int fp16, neighbours, inverse;
  int B, T, Hq, H;           // H: heads of q and k together
  int d, rot;
  int per, parts;            // rounds of heads per warp; warps per token
  int tail;                  // the elements past rot are copied (not in place)
};

cudaError_t launch_rope(const RopeParams& p, cudaStream_t s);
int rope_heads_per_round(int d);

}  // namespace bsa
