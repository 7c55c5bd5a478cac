// Appending tokens to the 8-bit cache: quantise a block of new tokens with one
// scale and scatter the codes into their page.
//
// A unit is one scale block (sb tokens of a page) of one head of K or V.  Its
// new elements are read once and stay in registers (32 per thread) between the
// maximum and the rounding.  A CTA takes units of one (row, block): what leads
// to the page (sequence -> length -> table entry) is read once for all of
// them, and a unit's elements are loaded while the one before is rounded.
// Bound by the 2 bytes read and the byte written per element for a long
// append, by that chain of reads for a token per sequence.
//
// With power-of-two scales x / scale is exact, codes move to a larger scale
// without a second rounding (subnormal codes excepted), and both code types
// times their scale are exact in bf16 and fp16 products.
#include "bsa_cache.h"
#include "bsa_cache_codes.cuh"

namespace bsa {
namespace {

using namespace dev;

constexpr int kVec = 4;  // 16-byte chunks (8 elements) per thread and unit

// Larger of the magnitudes of two pairs of elements (a NaN never wins).
template <bool FP16>
__device__ __forceinline__ uint32_t max_magnitude2(uint32_t m, uint32_t x) {
  uint32_t r;
  if constexpr (FP16) asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(x & 0x7fff7fffu));
  else asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(x & 0x7fff7fffu));
  return r;
}

// Codes of 8 elements, x / scale rounded.  `inv`: 1 / scale where scale is a
// power of two (then the product is exact), else 0.  `finite`: no infinity and
// no NaN among them.
template <int KIND, bool FP16>
__device__ __forceinline__ uint2 encode8(const uint4& x, float scale, float inv, bool finite) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t q[4];
  if (KIND == BSA_CACHE_INT8 && inv != 0.f && finite) {
    // x / scale + 1.5 * 2^23: the sum's last byte is the integer, rounded to
    // nearest even (|x / scale| <= 127 by the scale's choice).
    uint32_t b[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = elems_to_float2(w[e], FP16);
      b[2 * e] = __float_as_uint(fmaf(f.x, inv, 12582912.f));
      b[2 * e + 1] = __float_as_uint(fmaf(f.y, inv, 12582912.f));
    }
    return make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = elems_to_float2(w[e], FP16);
    q[e] = inv != 0.f ? encode2<KIND>(f.x * inv, f.y * inv) : encode2<KIND>(f.x / scale, f.y / scale);
  }
  return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
}

// Grid: (rows x blocks, parts); a CTA takes the units [part U / parts,
// (part + 1) U / parts) of its (row, block), U = 2 Hkv, blockDim / tpu at once.
template <int KIND, bool FP16>
__global__ void __launch_bounds__(1024) append_kernel(const __grid_constant__ CacheAppendParams p, int tpu) {
  __shared__ float s_max[2][32];
  next_may_launch();
  wait_for_previous();
  const CacheDev& c = p.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit_in = tid / tpu, ut = tid - unit_in * tpu;
  const int row = blockIdx.x / p.blocks, blk = blockIdx.x - row * p.blocks;
  const int seq = p.seqs ? __ldg(p.seqs + row) : row;
  const int count = p.counts ? __ldg(p.counts + row) : p.T;
  const int given = p.start ? __ldg(p.start + row) : 0;
  const bool known = seq >= 0 && seq < c.max_seqs;
  const int len = known ? __ldg(c.lens + seq) : 0;
  const int pos = p.start ? given : len - count;
  const bool first = blk == 0 && blockIdx.y == 0 && tid == 0;
  // Counts out of [0, T], tokens out of [0, len) or a sequence out of range.
  bool good = known && count >= 0 && count <= p.T && len <= c.max_pages * c.page;
  if (good && count > 0) good = pos >= 0 && pos <= len - count;
  if (first && !good && seq != -1) cache_error(c.control, BSA_ERR_INVALID_ARG, row);
  if (!good || count == 0) return;
  const int b0 = (pos / c.sb + blk) * c.sb;  // first position of the block
  const int lo = max(b0, pos), hi = min(b0 + c.sb, pos + count);
  if (lo >= hi) return;
  const int U = 2 * c.Hkv, upi = blockDim.x / tpu;
  const int u1 = (int)((long long)(blockIdx.y + 1) * U / gridDim.y);
  int u = (int)((long long)blockIdx.y * U / gridDim.y) + unit_in;
  const int steps = (u1 - (u - unit_in) + upi - 1) / upi;

  // This thread's chunks: row of the block and column, the same in every unit.
  const int cols = c.d / 8;
  int r[kVec];
  const int col = ut % cols;  // (tpu is a multiple of d / 8 or d / 8 a multiple of it: see below)
#pragma unroll
  for (int j = 0; j < kVec; ++j) r[j] = (j * tpu + ut) / cols;
  auto load = [&](int unit, uint4 (&x)[kVec]) {
    const CacheRows& src = unit < c.Hkv ? p.k : p.v;
    const uint16_t* base = src.p + (long long)row * src.sb + (long long)(unit < c.Hkv ? unit : unit - c.Hkv) * src.sh +
                           (long long)(b0 - pos) * src.st + col * 8;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      x[j] = make_uint4(0u, 0u, 0u, 0u);
      if (unit < u1 && b0 + r[j] >= lo && b0 + r[j] < hi)
        x[j] = __ldcs(reinterpret_cast<const uint4*>(base + (long long)r[j] * src.st));
    }
  };
  uint4 x[kVec];
  load(u, x);  // (does not need the page)
  const int phys = __ldg(c.table + (size_t)seq * c.max_pages + b0 / c.page);
  if (phys < 0 || phys >= c.num_pages) {
    if (blockIdx.y == 0 && tid == 0) cache_error(c.control, BSA_ERR_PLAN_MISMATCH, seq);
    return;
  }
  // Other tokens of the sequence in this block: below lo, or from hi on.
  const int held = min(b0 + c.sb, len);
  const bool others = lo > b0 || hi < held;

  for (int step = 0; step < steps; ++step, u += upi) {
    const bool active = u < u1;
    const bool isv = u >= c.Hkv;
    const size_t head = (size_t)phys * c.Hkv + (isv ? u - c.Hkv : u);
    float* scale_p = (isv ? c.vs : c.ks) + head * (c.page / c.sb) + (b0 & (c.page - 1)) / c.sb;
    const float was = active && others ? *scale_p : 0.f;
    uint4 next[kVec];
    load(u + upi, next);
    uint32_t m2 = 0u;
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      m2 = max_magnitude2<FP16>(max_magnitude2<FP16>(max_magnitude2<FP16>(max_magnitude2<FP16>(m2, x[j].x), x[j].y), x[j].z), x[j].w);
    const float2 mm = elems_to_float2(m2, FP16);
    float amax = fmaxf(mm.x, mm.y);
    if (amax == INFINITY) {  // rare: the finite elements alone decide
      amax = 0.f;
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = elems_to_float2(w[e], FP16);
          if (fabsf(f.x) < INFINITY) amax = fmaxf(amax, fabsf(f.x));
          if (fabsf(f.y) < INFINITY) amax = fmaxf(amax, fabsf(f.y));
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (tpu > 32) {
      // (the other half of s_max may still be read by a warp one step behind)
      if (lane == 0) s_max[step & 1][warp] = amax;
      __syncthreads();
      const int w0 = unit_in * (tpu / 32);
      for (int w = 0; w < tpu / 32; ++w) amax = fmaxf(amax, s_max[step & 1][w0 + w]);
    } else {
      __syncwarp();  // every thread of the unit has read its scale before one writes it
    }
    if (active) {
      float scale = scale_for<KIND>(amax);
      if (others) scale = fmaxf(scale, was);
      const float inv = (__float_as_uint(scale) & 0x7fffffu) == 0 ? 1.f / scale : 0.f;
      const bool grown = others && scale != was;
      if (ut == 0 && (!others || grown)) *scale_p = scale;
      uint8_t* codes = (isv ? c.v : c.k) + (head * c.page + (b0 & (c.page - 1))) * (size_t)c.d + col * 8;
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        uint2* at = reinterpret_cast<uint2*>(codes + (size_t)r[j] * c.d);
        if (b0 + r[j] >= lo && b0 + r[j] < hi) {
          // Infinities and NaN have all exponent bits set.
          bool finite = true;
          if (KIND == BSA_CACHE_INT8) {
            const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
            constexpr uint32_t ex = FP16 ? 0x7c00u : 0x7f80u;
#pragma unroll
            for (int e = 0; e < 4; ++e) finite = finite && (w[e] & ex) != ex && (w[e] & ex << 16) != ex << 16;
          }
          *at = encode8<KIND, FP16>(x[j], scale, inv, finite);
        } else if (grown && b0 + r[j] < held) {
          // Another token of the sequence: its codes move to the larger scale.
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
#pragma unroll
    for (int j = 0; j < kVec; ++j) x[j] = next[j];
  }
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendParams& p, int sms, cudaStream_t s) {
  // Threads of a unit: 32 .. 1024, a multiple of the d / 8 chunks of a token.
  const int tpu = p.c.sb * p.c.d / (8 * kVec);
  const int threads = tpu < 256 ? 256 : tpu;
  const long long gx = (long long)p.n * p.blocks;
  if (gx > 0x7fffffffll) return cudaErrorInvalidValue;
  // Units of a (row, block) are spread over CTAs until there are about eight
  // CTAs' worth of threads for each SM.
  const int most = (2 * p.c.Hkv + threads / tpu - 1) / (threads / tpu);
  const long long want = (8ll * sms * 256 / threads + gx - 1) / gx;
  const int parts = (int)(want < 1 ? 1 : (want < most ? want : most));
  const dim3 grid((unsigned)gx, (unsigned)parts);
  if (p.c.kind == BSA_CACHE_INT8)
    return launch_after(p.fp16 ? append_kernel<BSA_CACHE_INT8, true> : append_kernel<BSA_CACHE_INT8, false>, grid,
                        dim3(threads), 0, s, p, tpu);
  return launch_after(p.fp16 ? append_kernel<BSA_CACHE_E4M3, true> : append_kernel<BSA_CACHE_E4M3, false>, grid,
                      dim3(threads), 0, s, p, tpu);
}

}  // namespace bsa
