// Keys and values of a cache's sequences as bf16 [B][Hkv][Nk][d], for the
// block-sparse forward, with the bounds its key-norm pass would read them for.
//
// The forward's products are bound by the tensor pipe and read each K/V tile
// once per query tile that selects it, so the codes are converted once, by a
// pass of its own (1 byte read and 2 written per element), and not again in
// every tile's inner loop.  Issue bounds it, at 76 %: what it writes stays in
// L2, and DRAM is at 28 %.  The largest key norm and
// the largest value of every K/V unit (see bsa_prep.cu) are taken while the
// elements are in registers: a pass over the 2-byte copies costs as much again
// (16384 keys of 8 heads, d 128: 18.7 us, 5.4 TB/s of what it reads and writes
// together, against 20 + 18 us in two passes).  Positions at and past a sequence's length
// become zero: the forward masks them but multiplies what they hold.
#include "bsa_cache.h"
#include "bsa_cache_codes.cuh"
#include "bsa_device.cuh"

namespace bsa {
namespace {

using namespace dev;

constexpr int kThreads = 256;
constexpr int kItems = 4;  // chunks of 16 codes per thread: 128 tokens (d = 128) or 256 of a head per CTA

template <int D, int KIND>
__global__ void __launch_bounds__(kThreads) load_kernel(const __grid_constant__ CacheLoadParams p) {
  constexpr int kCols = D / 16;                          // chunks of a token
  constexpr int kTokens = kThreads * kItems / kCols;     // of a CTA
  constexpr int kBlocks = kTokens / 32;                  // of 32 tokens
  constexpr int kBlockThreads = 32 * kCols;              // threads that hold one of a step's blocks
  __shared__ float s_max[kBlocks];
  next_may_launch();
  wait_for_previous();
  const CacheDev& c = p.c;
  const int tid = threadIdx.x;
  const int bh = blockIdx.y, b = bh / c.Hkv, h = bh % c.Hkv;
  const int seq = p.seqs ? load_written(p.seqs + b) : b;
  // (a sequence or a length out of range: an empty one, recorded)
  int len = seq >= 0 && seq < c.max_seqs ? load_written(c.lens + seq) : (seq == -1 ? 0 : -1);
  const bool known = len >= 0 && len <= c.max_pages * c.page;
  if (!known) len = 0;
  const bool isv = blockIdx.z != 0;
  if (blockIdx.x == 0 && h == 0 && !isv) {
    // A sequence with a token in no page is skipped: the forward masks keys by
    // their number alone, so it gets a length of 0.
    const int pages = (min(len, p.Nk) + c.page - 1) / c.page;
    bool gap = false;
    for (int j = tid; j < pages; j += kThreads) {
      const int ph = load_written(c.table + (size_t)seq * c.max_pages + j);
      gap |= ph < 0 || ph >= c.num_pages;
    }
    gap = __syncthreads_or(gap);
    if (tid == 0) {
      p.lens[b] = gap ? 0 : len;  // (whole: the queries are the last tokens, of which Nk may leave out some)
      if (!known) cache_error(c.control, BSA_ERR_INVALID_ARG, b);
    }
  }
  // What a forward resets ahead of its passes.
  const long long at = ((long long)(blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x) * kThreads + tid;
  const long long all = (long long)gridDim.x * gridDim.y * gridDim.z * kThreads;
  for (long long i = at; i < p.rows; i += all) p.fb_flag[i] = 0;
  if (at < p.control_words) p.control[at] = 0;
  len = min(len, p.Nk);
  const uint8_t* codes = isv ? c.v : c.k;
  const float* scales = isv ? c.vs : c.ks;
  uint16_t* out = (isv ? p.v : p.k) + (size_t)bh * p.Nk * D;
  const int t0 = blockIdx.x * kTokens;
  const int lpage = 31 - __clz(c.page), lsb = 31 - __clz(c.sb);
  if (tid < kBlocks) s_max[tid] = 0.f;
  const int col = tid % kCols;
  uint4 x[kItems];
  float sc[kItems];
  int ph[kItems];
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    const int key = t0 + (j * kThreads + tid) / kCols;
    ph[j] = key < len ? load_written(c.table + (size_t)seq * c.max_pages + (key >> lpage)) : 0;
    if (ph[j] < 0 || ph[j] >= c.num_pages) {
      cache_error(c.control, BSA_ERR_PLAN_MISMATCH, seq);
      ph[j] = -1;
    }
  }
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    const int key = t0 + (j * kThreads + tid) / kCols;
    x[j] = make_uint4(0u, 0u, 0u, 0u);  // (codes 0)
    sc[j] = 0.f;
    if (key < len && ph[j] >= 0) {
      const unsigned row = ((unsigned)(ph[j] * c.Hkv + h) << lpage) + (key & (c.page - 1));  // (below 2^31)
      x[j] = __ldcs(reinterpret_cast<const uint4*>(codes + (size_t)row * D + col * 16));
      sc[j] = load_written(scales + (row >> lsb));
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    const int token = (j * kThreads + tid) / kCols;
    const uint32_t cw[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
    uint32_t w[8];
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint2 hh = codes_to_half4<KIND>(cw[e]);
      const float2 f0 = half2_to_float2(hh.x), f1 = half2_to_float2(hh.y);
      w[2 * e] = pack_bf16x2(f0.x * sc[j], f0.y * sc[j]);
      w[2 * e + 1] = pack_bf16x2(f1.x * sc[j], f1.y * sc[j]);
    }
    // The bounds are those of the bf16 elements, as the key-norm pass takes them.
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float lo = __uint_as_float(w[e] << 16), hi = __uint_as_float(w[e] & 0xffff0000u);
      m = isv ? fmaxf(m, fmaxf(fabsf(lo), fabsf(hi))) : fmaf(hi, hi, fmaf(lo, lo, m));
    }
    if (t0 + token < p.Nk) st_global_v8(out + (size_t)(t0 + token) * D + col * 16, w);
#pragma unroll
    for (int o = 1; o < kCols; o <<= 1) {  // the chunks of a token: neighbouring lanes
      const float y = __shfl_xor_sync(0xffffffffu, m, o);
      m = isv ? fmaxf(m, y) : m + y;
    }
#pragma unroll
    for (int o = kCols; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // (bounds are not negative, or NaN, which compares above every number)
    if ((tid & 31) == 0)
      atomicMax(reinterpret_cast<int*>(s_max) + (j * kThreads + tid) / kBlockThreads, __float_as_int(m));
  }
  __syncthreads();
  // Units of ku tokens: the largest of their blocks of 32.
  const int units = kTokens / p.ku;
  if (tid < units) {
    const int unit = t0 / p.ku + tid;
    if (unit < p.NKU) {
      float m = 0.f;
      for (int q = tid * (p.ku / 32); q < (tid + 1) * (p.ku / 32); ++q) m = fmaxf(m, s_max[q]);
      const size_t to = (size_t)bh * p.NKU + unit;
      if (isv) p.vmax[to] = m;
      else p.kmax[to] = sqrtf(m);
    }
  }
}

template <int D>
cudaError_t launch_d(const CacheLoadParams& p, cudaStream_t s) {
  constexpr int kTokens = kThreads * kItems / (D / 16);
  const dim3 grid((unsigned)((p.Nk + kTokens - 1) / kTokens), (unsigned)(p.B * p.c.Hkv), 2);
  return launch_after(p.c.kind == BSA_CACHE_INT8 ? load_kernel<D, BSA_CACHE_INT8> : load_kernel<D, BSA_CACHE_E4M3>, grid,
                      dim3(kThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_cache_load(const CacheLoadParams& p, cudaStream_t s) {
  return p.c.d == 64 ? launch_d<64>(p, s) : launch_d<128>(p, s);
}

}  // namespace bsa
