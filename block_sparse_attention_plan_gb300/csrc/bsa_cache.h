// Internal declarations of the 8-bit K/V cache: device views, the control
// words and the kernels' launchers.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "bsa.h"
#include "bsa_launch.h"

namespace bsa {

constexpr int kCacheListMax = 4096;  // sequences in one resize or fork
// Control words of a cache; the scratch lists follow at kCacheScratch.
constexpr int kCacheStatus = 0;
constexpr int kCacheDetail = 1;
constexpr int kCacheLive = 2;    // held pages the last compaction found
constexpr int kCachePairs = 3;   // page copies queued for the copy kernel
constexpr int kCacheTaken = 4;   // pages that the last resize took: entries of list_a
constexpr int kCacheScratch = 16;

// Device view of a cache, by value to every kernel.
struct CacheDev {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int32_t* table;
  int32_t* lens;
  int32_t* refs;
  int32_t* control;
  int kind, num_pages, Hkv, page, d, sb, max_seqs, max_pages;
  // Scratch: free pages found / page map / marks; copy pairs.
  __host__ __device__ int32_t* list_a() const { return control + kCacheScratch; }
  __host__ __device__ int32_t* pair_src() const { return control + kCacheScratch + num_pages; }
  __host__ __device__ int32_t* pair_dst() const { return control + kCacheScratch + 2 * (size_t)num_pages; }
};
inline size_t cache_control_ints(int num_pages) { return kCacheScratch + 3 * (size_t)num_pages; }

#ifdef __CUDACC__
// First error of its cache since the last report.
__device__ __forceinline__ void cache_error(int32_t* control, int code, int detail) {
  if (atomicCAS(control + kCacheStatus, 0, code) == 0) atomicExch(control + kCacheDetail, detail);
}
#endif

// Token tensor [n][Hkv][T][d] of bf16 or fp16 elements.
struct CacheRows {
  const uint16_t* p;
  long long sb, sh, st;  // strides in elements
};

struct CacheAppendParams {
  CacheDev c;
  CacheRows k, v;
  int fp16, n, T, blocks;  // blocks: most scale blocks one row can touch
  const int32_t* seqs;
  const int32_t* counts;
  const int32_t* start;
};

// Queries per unit of work at most: four row tiles of 24.
constexpr int kCacheUnitRows = 96;
// What a unit's beginning (queries, joining the warps) costs a CTA, in tiles.  Measured for 0, 4, 8, 12,
// 16, 24: 32 sequences of up to 32768 tokens 176, 170, 170, 170, 170, 172 us; 5 draft tokens of 16
// sequences, INT8, d 64: 70, 67, 63, 62, 63, 65 us; 64 sequences of up to 700 tokens 34, 26, 25, 25, 24, 25 us.
constexpr int kCacheUnitHead = 12;
// Keys per tile: 4 KB of K and of V.
constexpr int cache_tile_keys(int d) { return 4096 / d; }
constexpr int kCacheMaxGrid = 320;   // most CTAs of the attention kernel (workspace bound)

struct CacheAttnParams {
  CUtensorMap tmK, tmV;  // pools as lines of 128 bytes (128 / d tokens), box: min(page, tile) tokens
  CacheDev c;
  CacheRows q;
  uint16_t* o;
  long long o_sb, o_sh, o_st;
  float* lse;
  const int32_t* seqs;
  const uint8_t* mask;  // [B][Hq][NKB]
  int32_t* list;        // active tiles of each (b, kv head) [B*Hkv][max_tiles] (with a mask)
  int32_t* counts;      // how many [B*Hkv]
  float* part;          // partial O and (m, l): see bsa_cache_attn.cu
  int32_t* desc;        // rows split over CTAs, for the combine kernel [grid][4]
  int fp16, B, Hq, g, nq, M, groups, NKB, bk, tile, max_tiles, causal;
  int rows_cap;         // query rows of a partial's slot
  int head;             // places of the line that a unit's beginning counts for
  float scale_log2;
  long long watchdog_ns;
};

// K and V of sequences seqs[0 .. B) as bf16 [B][Hkv][Nk][d] (zero at and past
// the length), their lengths [B], and what the forward's key-norm pass gives:
// the largest key norm and value of every unit of ku keys, rows' flags cleared.
struct CacheLoadParams {
  CacheDev c;
  const int32_t* seqs;
  int B, Nk;
  uint16_t* k;
  uint16_t* v;
  int32_t* lens;
  float* kmax;  // [B*Hkv][NKU]
  float* vmax;
  int32_t* fb_flag;  // [rows]
  int32_t* control;  // the forward's control words
  int control_words;
  int rows, ku, NKU;
  int device;  // the plan's
};

cudaError_t launch_cache_resize(const CacheDev& c, const int32_t* seqs, const int32_t* new_lens, int n,
                                cudaStream_t s);
cudaError_t launch_cache_fork(const CacheDev& c, const int32_t* src, const int32_t* dst, int n, cudaStream_t s);
cudaError_t launch_cache_compact(const CacheDev& c, int sms, cudaStream_t s);
cudaError_t launch_cache_copy(const CacheDev& dst, const CacheDev& src, const int32_t* dst_pages,
                              const int32_t* src_pages, int n, cudaStream_t s);
cudaError_t launch_cache_append(const CacheAppendParams& p, int sms, cudaStream_t s);
cudaError_t launch_cache_attention(const CacheAttnParams& p, int grid, cudaStream_t s);
cudaError_t launch_cache_load(const CacheLoadParams& p, cudaStream_t s);
// The arrays of a plan's forward that its key-norm pass writes, and that forward
// without the pass, the causal offset of each sequence taken from its key length
// (bsa_api.cu).
bsa_status key_norm_views(const bsa_plan* plan, CacheLoadParams* p);
bsa_status forward_after_load(const bsa_plan* plan, const void* Q, const CacheLoadParams& p, int flags, void* O,
                              float* LSE, float scale, cudaStream_t stream);

}  // namespace bsa
