// Appending tokens to the 8-bit cache: quantise a block of new tokens with one
// scale and scatter the codes into their page.
//
// A unit is one scale block (sb tokens of a page) of one head of K or V.  Its
// new elements are read once and stay in registers (32 per thread) between the
// maximum and the rounding; what bounds a long append is the 2 bytes read and
// the byte written per element, what bounds one token per sequence is the
// latency of the chain sequence -> length -> page -> scale -> store, so
// everything that does not depend on the page is loaded before it is needed.
// With power-of-two scales x / scale is exact, codes move to a larger scale
// without a second rounding (subnormal codes excepted), and both code types
// times their scale are exact in bf16 and fp16 products.
#include "bsa_cache.h"
#include "bsa_cache_codes.cuh"

namespace bsa {
namespace {

using namespace dev;

constexpr int kVec = 4;  // 16-byte chunks (8 elements) per thread

template <int KIND>
__global__ void __launch_bounds__(1024) append_kernel(const CacheAppendParams p, int tpu) {
  __shared__ float s_max[32];
  const CacheDev& c = p.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit_in = tid / tpu, ut = tid - unit_in * tpu;
  // Units in the order (row, block, K/V, head): heads of a token together.
  const long long unit = (long long)blockIdx.x * (blockDim.x / tpu) + unit_in;
  const int h = (int)(unit % c.Hkv);
  long long rest = unit / c.Hkv;
  const int isv = (int)(rest & 1);
  rest >>= 1;
  const int blk = (int)(rest % p.blocks);
  const long long row_l = rest / p.blocks;
  const bool in_grid = row_l < p.n;
  const int row = in_grid ? (int)row_l : 0;

  const int seq = !in_grid ? -1 : (p.seqs ? __ldg(p.seqs + row) : row);
  int count = p.counts ? __ldg(p.counts + row) : p.T;
  const int given = p.start ? __ldg(p.start + row) : 0;
  const bool known = seq >= 0 && seq < c.max_seqs;
  const int len = known ? __ldg(c.lens + seq) : 0;
  const int pos = p.start ? given : len - count;
  // Counts out of [0, T], tokens out of [0, len) or a sequence out of range.
  bool good = known && count >= 0 && count <= p.T && len <= c.max_pages * c.page;
  if (good && count > 0) good = pos >= 0 && pos <= len - count;
  if (in_grid && !good && seq != -1 && blk == 0 && h == 0 && isv == 0 && ut == 0)
    cache_error(c.control, BSA_ERR_INVALID_ARG, row);
  if (!good) count = 0;
  const int b0 = count > 0 ? (pos / c.sb + blk) * c.sb : 0;  // first position of the block
  const int lo = max(b0, pos), hi = min(b0 + c.sb, pos + count);
  bool active = count > 0 && lo < hi;
  int phys = 0;
  if (active) {
    phys = __ldg(c.table + (size_t)seq * c.max_pages + b0 / c.page);
    if (phys < 0 || phys >= c.num_pages) {
      if (h == 0 && isv == 0 && ut == 0) cache_error(c.control, BSA_ERR_PLAN_MISMATCH, seq);
      active = false;
    }
  }
  // Other tokens of the sequence in this block: below lo, or from hi on.
  const int held = min(b0 + c.sb, len);
  const bool others = active && (lo > b0 || hi < held);
  const size_t head = (size_t)phys * c.Hkv + h;
  float* scale_p = (isv ? c.vs : c.ks) + head * (c.page / c.sb) + (b0 % c.page) / c.sb;
  const float was = others ? *scale_p : 0.f;
  uint8_t* codes = (isv ? c.v : c.k) + (head * c.page + b0 % c.page) * (size_t)c.d;

  const CacheRows& src = isv ? p.v : p.k;
  const int cols = c.d / 8;
  uint4 x[kVec];
  float amax = 0.f;
  bool fresh[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int ch = j * tpu + ut, r = ch / cols, col = ch - r * cols;
    fresh[j] = active && b0 + r >= lo && b0 + r < hi;
    x[j] = make_uint4(0u, 0u, 0u, 0u);
    if (fresh[j])
      x[j] = __ldg(reinterpret_cast<const uint4*>(src.p + (long long)row * src.sb + (long long)h * src.sh +
                                                  (long long)(b0 + r - pos) * src.st + col * 8));
  }
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = elems_to_float2(w[e], p.fp16);
      const float a = fabsf(f.x), b = fabsf(f.y);
      if (a < INFINITY) amax = fmaxf(amax, a);  // finite elements only
      if (b < INFINITY) amax = fmaxf(amax, b);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (tpu > 32) {
    if (lane == 0) s_max[warp] = amax;
    __syncthreads();
    const int w0 = unit_in * (tpu / 32);
    for (int w = 0; w < tpu / 32; ++w) amax = fmaxf(amax, s_max[w0 + w]);
  }
  __syncwarp();  // every thread of the unit has read its scale before one writes it
  if (!active) return;  // (no barrier follows)
  float scale = scale_for<KIND>(amax);
  if (others) scale = fmaxf(scale, was);
  const float inv = 1.f / scale;  // exact for a power of two
  const bool pow2 = (__float_as_uint(scale) & 0x7fffffu) == 0;
  const bool grown = others && scale != was;
  if (ut == 0 && (!others || grown)) *scale_p = scale;
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int ch = j * tpu + ut, r = ch / cols, col = ch - r * cols;
    if (fresh[j]) {
      const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
      uint32_t q[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = elems_to_float2(w[e], p.fp16);
        q[e] = pow2 ? encode2<KIND>(f.x * inv, f.y * inv) : encode2<KIND>(f.x / scale, f.y / scale);
      }
      *reinterpret_cast<uint2*>(codes + (size_t)r * c.d + col * 8) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
    } else if (grown && b0 + r < held) {
      // Another token of the sequence: its codes move to the larger scale.
      uint2* at = reinterpret_cast<uint2*>(codes + (size_t)r * c.d + col * 8);
      const uint2 old = *at;
      const float ratio = was / scale;
      uint32_t q[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint2 hh = codes_to_half4<KIND>(e ? old.y : old.x);
        const float2 f0 = half2_to_float2(hh.x), f1 = half2_to_float2(hh.y);
        q[2 * e] = encode2<KIND>(f0.x * ratio, f0.y * ratio);
        q[2 * e + 1] = encode2<KIND>(f1.x * ratio, f1.y * ratio);
      }
      *at = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
    }
  }
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendParams& p, cudaStream_t s) {
  const int tpu = p.c.sb * p.c.d / (8 * kVec);  // threads of a unit: 32 .. 1024
  const int threads = tpu < 256 ? 256 : tpu;
  const long long units = (long long)p.n * p.blocks * 2 * p.c.Hkv;
  const long long per = threads / tpu, grid = (units + per - 1) / per;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  if (p.c.kind == BSA_CACHE_INT8) append_kernel<BSA_CACHE_INT8><<<(unsigned)grid, threads, 0, s>>>(p, tpu);
  else append_kernel<BSA_CACHE_E4M3><<<(unsigned)grid, threads, 0, s>>>(p, tpu);
  return cudaGetLastError();
}

}  // namespace bsa
