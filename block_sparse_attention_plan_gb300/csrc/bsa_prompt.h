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

// Attention of packed prompts (bsa_prompt_attn.cu).
constexpr int kPromptRows = 256;   // query rows of a work item: two tiles of 128
// Up to so many prompts of so many tokens together find their items without the
// schedule kernel.  The kernels with it and without it, us, at 32/8 heads of 128 and 8/2 of 64:
//   24 of 1 to 59 tokens  21.8 / 18.5, 14.5 / 12.0    16 of 512  67.6 / 64.6, 24.4 / 20.5
//   64 of 64              37.1 / 34.3, 16.4 / 12.3    64 of 512   221 / 211,  56.7 / 53.6
//   one of 4096            105 / 101,  45.1 / 43.1    one of 8192 343 / 341,  78.0 / 76.0
//   3500 behind 63 of 9   98.9 / 96.8, 41.5 / 39.0
//   3500 ahead of 63 of 9 98.1 / 102,  41.5 / 59.6    8000 ahead of 63 of 20  341 / 361, 82.5 / 133
// The schedule is 3 to 4 us, and past these limits less than what dealing the items out as
// they lie may cost; below them a long prompt listed ahead of short ones is the one order
// that it costs more (the lengths are on the device: no rule on them can choose).
constexpr int kPromptFew = 64, kPromptFewTokens = 4096;
constexpr int kPromptCtlTiles = 3; // control word: work items of a group of heads (0-2: as a plan's)
constexpr int kPromptCtlCtas = 4;  // control word: CTAs of the attention kernel
// Behind the 16 control words, status and detail of each CTA, which it writes as it ends.
constexpr int kPromptCtlOwn = 16;
constexpr int kPromptMaxCtas = 512;
constexpr int kPromptCtlWords = kPromptCtlOwn + 2 * kPromptMaxCtas;
struct PromptParams {
  CUtensorMap tmQ;         // q as [halves][T][Hq][64], box {64, gp, 128 / gp, halves}: 128 rows, a token's heads together
  CUtensorMap tmK, tmV;    // k, v as [halves][T][Hkv][64], box {64, 1, 128, halves}
  const uint16_t* v;       // (values that are no numbers are looked up again)
  long long v_st, v_sh;
  uint16_t* o;
  long long o_st, o_sh;
  float* lse;              // [T][Hq] or nullptr
  const int32_t* offsets;  // [n + 1]
  int32_t* control;        // [kPromptCtlWords]
  int32_t* tile_ptr;       // [n + 1]: work items ahead of each prompt
  int4* tiles;             // {first row, length, first token, 0}, longest first
  int n, T, Hq, Hkv, g;
  int gp_shift;            // log2 of the heads of a tile
  int causal, fp16, o_v8;
  int few;                 // no schedule: n <= kPromptFew, T <= kPromptFewTokens
  float scale_log2;
  long long watchdog_ns;
};
cudaError_t launch_prompt(const PromptParams& p, int d, int sms, cudaStream_t s);

cudaError_t launch_rope(const RopeParams& p, cudaStream_t s);
int rope_heads_per_round(int d);

}  // namespace bsa
