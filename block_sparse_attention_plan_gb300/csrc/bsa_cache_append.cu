// Appending tokens to the 8-bit cache: quantise a block of new tokens with one
// scale and scatter the codes into their page.
//
// A unit is one scale block (sb tokens of a page) of one head of K or V.  Its
// new elements are read once and stay in registers (32 per thread) between the
// maximum and the rounding.  A CTA takes units of one (row, block): what leads
// to the page (sequence -> length -> table entry) is read once for all of
// them, and a unit's elements are loaded while the one before is rounded.
// A long append would be bound by the 2 bytes read and the byte written per
// element but for the instructions, which are counted here (about five per
// element: maxima of pairs as integers, the scale's reciprocal from its bits,
// what depends on the thread alone kept out of the units' loop): 113 MB for 6
// sequences of up to 4001 tokens, 16 heads of 64, in 22.2 us, 5.1 TB/s.  A token
// per sequence is bound by that chain of reads: 7.3 us for 64 sequences, 8 heads
// of 128.
//
// With power-of-two scales x / scale is exact, codes move to a larger scale
// without a second rounding (subnormal codes excepted), and both code types
// times their scale are exact in bf16 and fp16 products.
#include <type_traits>

#include "bsa_cache.h"
#include "bsa_cache_codes.cuh"

namespace bsa {
namespace {

using namespace dev;

constexpr int kVec = 4;  // 16-byte chunks (8 elements) per thread and unit
constexpr float kInvertible = 0x1p127f;  // scales below it have a normal reciprocal (a cache filled by others may hold it)

// Larger of each two elements' magnitudes, as integers: of elements of one sign
// these compare like the numbers, with infinity and then NaN above all others.
__device__ __forceinline__ uint32_t max_magnitude2(uint32_t m, uint32_t x) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(x & 0x7fff7fffu));
  return r;
}

// Codes of 8 elements, rounded from x * inv (scale = 1 / inv a power of two: the
// product is exact).  `finite`: no infinity and no NaN among them.
template <int KIND, bool FP16>
__device__ __forceinline__ uint2 encode8(const uint4& x, float inv, bool finite) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  if (KIND == BSA_CACHE_INT8 && finite) {
    // x * inv + 1.5 * 2^23: the sum's last byte is the integer, rounded to
    // nearest even (|x * inv| <= 127 by the scale's choice).
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
  uint32_t q[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = elems_to_float2(w[e], FP16);
    q[e] = encode2<KIND>(f.x * inv, f.y * inv);
  }
  return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
}

// a * b and a / b rounded to odd (towards zero, the last bit set if anything was
// cut off): a rounding to the codes' few bits then gives what it would of the
// exact value, ties included.
__device__ __forceinline__ float odd_if(float x, float rest) {
  return rest != 0.f && fabsf(x) < INFINITY ? __uint_as_float(__float_as_uint(x) | 1u) : x;
}
__device__ __forceinline__ float mul_odd(float a, float b) {
  const float p = __fmul_rz(a, b);
  return odd_if(p, fmaf(a, b, -p));
}
__device__ __forceinline__ float div_odd(float a, float b) {
  const float q = __fdiv_rz(a, b);
  return odd_if(q, fmaf(-q, b, a));
}

// The same for a scale that is no power of two (a cache filled by others).
template <int KIND, bool FP16>
__device__ __noinline__ uint2 encode8_div(uint4 x, float scale) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t q[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = elems_to_float2(w[e], FP16);
    q[e] = encode2<KIND>(div_odd(f.x, scale), div_odd(f.y, scale));
  }
  return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
}

// 8 codes moved from scale `was` to `scale`.
template <int KIND>
__device__ __noinline__ uint2 recode8(uint2 old, float ratio) {
  uint32_t q[4];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const uint2 hh = codes_to_half4<KIND>(e ? old.y : old.x);
    const float2 f0 = half2_to_float2(hh.x), f1 = half2_to_float2(hh.y);
    q[2 * e] = encode2<KIND>(mul_odd(f0.x, ratio), mul_odd(f0.y, ratio));
    q[2 * e + 1] = encode2<KIND>(mul_odd(f1.x, ratio), mul_odd(f1.y, ratio));
  }
  return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
}

// Largest finite magnitude of a thread's elements where some are not finite.
template <bool FP16>
__device__ __noinline__ float finite_max(uint4 x0, uint4 x1, uint4 x2, uint4 x3) {
  const uint32_t w[16] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w,
                          x2.x, x2.y, x2.z, x2.w, x3.x, x3.y, x3.z, x3.w};
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float2 f = elems_to_float2(w[e], FP16);
    if (fabsf(f.x) < INFINITY) m = fmaxf(m, fabsf(f.x));
    if (fabsf(f.y) < INFINITY) m = fmaxf(m, fabsf(f.y));
  }
  return m;
}

// Grid: (rows x blocks, parts); a CTA takes the units [part U / parts,
// (part + 1) U / parts) of its (row, block), U = 2 Hkv, blockDim / tpu at once.
// LIST: the sequences are given in a list, in which none may appear twice (an
// instantiation of its own: the search costs the others a microsecond).
template <int KIND, bool FP16, bool LIST>
__global__ void __launch_bounds__(1024) append_kernel(const __grid_constant__ CacheAppendParams p, int tpu) {
  __shared__ float s_max[2][32];
  next_may_launch();
  wait_for_previous();
  const CacheDev& c = p.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit_in = tid / tpu, ut = tid - unit_in * tpu;
  const int row = blockIdx.x / p.blocks, blk = blockIdx.x - row * p.blocks;
  const int seq = LIST ? load_written(p.seqs + row) : row;
  if constexpr (LIST) {
    bool twice = false;  // named by an earlier row: both would write one block
    for (int j = tid; j < row; j += blockDim.x) twice |= load_written(p.seqs + j) == seq;
    if (__syncthreads_or(twice && seq != -1)) {
      if (blk == 0 && blockIdx.y == 0 && tid == 0) cache_error(c.control, BSA_ERR_INVALID_ARG, row);
      return;
    }
  }
  const int count = p.counts ? load_written(p.counts + row) : p.T;
  const int given = p.start ? load_written(p.start + row) : 0;
  const bool known = seq >= 0 && seq < c.max_seqs;
  const int len = known ? load_written(c.lens + seq) : 0;
  const int pos = p.start ? given : len - count;
  const bool first = blk == 0 && blockIdx.y == 0 && tid == 0;
  // Counts out of [0, T], tokens out of [0, len) or a sequence out of range.
  bool good = known && count >= 0 && count <= p.T && len <= c.max_pages * c.page;
  if (good && count > 0) good = pos >= 0 && pos <= len - count;
  if (first && !good && seq != -1) cache_error(c.control, BSA_ERR_INVALID_ARG, row);
  if (!good || count == 0) return;
  const int b0 = ((pos >> (31 - __clz(c.sb))) + blk) * c.sb;  // first position of the block
  const int lo = max(b0, pos), hi = min(b0 + c.sb, pos + count);
  if (lo >= hi) return;
  const int U = 2 * c.Hkv, upi = blockDim.x / tpu;
  const int u1 = (int)((long long)(blockIdx.y + 1) * U / gridDim.y);
  int u = (int)((long long)blockIdx.y * U / gridDim.y) + unit_in;
  const int steps = (u1 - (u - unit_in) + upi - 1) / upi;

  // This thread's chunks, the same in every unit: chunk j is row (j tpu + ut) /
  // (d / 8) of the block (tpu is a multiple of d / 8, so all have one column).
  const int cols = c.d / 8, row0 = ut / cols, rows_j = tpu / cols;
  unsigned fresh = 0, old = 0;  // bit j: a new token, another token of the sequence
  const int held = min(b0 + c.sb, len);
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int t = b0 + row0 + j * rows_j;
    if (t >= lo && t < hi) fresh |= 1u << j;
    else if (t < held) old |= 1u << j;
  }
  const int first_row = b0 - pos + row0;  // (of the tensor; below 0 where the tokens begin in the block)
  const int col = (ut - row0 * cols) * 8;
  // (addresses are built anew for each unit: kept, they cost the registers that
  // let four CTAs share an SM without spills)
  auto load = [&](int unit, uint4 (&x)[kVec]) {
    const bool isv = unit >= c.Hkv;
    const CacheRows& src = isv ? p.v : p.k;
    const uint16_t* at = src.p + (long long)row * src.sb + (long long)(isv ? unit - c.Hkv : unit) * src.sh +
                         (long long)first_row * src.st + col;
    const long long step = (long long)rows_j * src.st;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      x[j] = make_uint4(0u, 0u, 0u, 0u);
      if (unit < u1 && (fresh >> j & 1u)) x[j] = __ldcs(reinterpret_cast<const uint4*>(at));
      at += step;
    }
  };
  uint4 x[kVec];
  load(u, x);  // (does not need the page)
  const int phys = load_written(c.table + (size_t)seq * c.max_pages + (b0 >> (31 - __clz(c.page))));
  if (phys < 0 || phys >= c.num_pages) {
    if (blockIdx.y == 0 && tid == 0) cache_error(c.control, BSA_ERR_PLAN_MISMATCH, seq);
    return;
  }
  const int refs = load_written(c.refs + phys);  // (arrives while the first units' maxima are taken)
  // Other tokens of the sequence in this block: below lo, or from hi on.
  const bool others = lo > b0 || hi < held;
  const int lsb = 31 - __clz(c.sb), in_page = b0 & (c.page - 1);

  for (int step = 0; step < steps; ++step, u += upi) {
    const bool active = u < u1, isv = u >= c.Hkv;
    const size_t first = ((size_t)phys * c.Hkv + (isv ? u - c.Hkv : u)) * c.page + in_page;  // row of the pool
    float* scale_p = (isv ? c.vs : c.ks) + (first >> lsb);
    const float was = active && others ? *scale_p : 0.f;
    uint4 next[kVec];
    load(u + upi, next);
    uint32_t m2 = 0u;
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      m2 = max_magnitude2(max_magnitude2(max_magnitude2(max_magnitude2(m2, x[j].x), x[j].y), x[j].z), x[j].w);
    constexpr uint32_t inf = FP16 ? 0x7c00u : 0x7f80u;
    m2 = max(m2 & 0xffffu, m2 >> 16);
    const bool finite = m2 < inf;
    float mine = elems_to_float2(m2, FP16).x;
    if (!finite) mine = finite_max<FP16>(x[0], x[1], x[2], x[3]);  // rare
    float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mine)));  // (not negative)
    if (tpu > 32) {
      // (the other half of s_max may still be read by a warp one step behind)
      if (lane == 0) s_max[step & 1][warp] = amax;
      __syncthreads();
      const int w0 = unit_in * (tpu / 32);
      for (int w = 0; w < tpu / 32; ++w) amax = fmaxf(amax, s_max[step & 1][w0 + w]);
    } else {
      __syncwarp();  // every thread of the unit has read its scale before one writes it
    }
    if (active && refs <= 1) {
      float scale = scale_for<KIND>(amax);
      // 0: nothing has been stored in the block since the sequence entered it
      // (the same for what no scale is: memory that was never written).
      const bool stored = was > 0.f && was < INFINITY;
      if (stored) scale = fmaxf(scale, was);
      const bool grown = others && scale != was;
      if (ut == 0 && (!others || grown)) *scale_p = scale;
      uint8_t* at = (isv ? c.v : c.k) + first * c.d + ut * 8;
      if ((__float_as_uint(scale) & 0x7fffffu) == 0 && scale < kInvertible) {
        const float inv = __uint_as_float((254u << 23) - __float_as_uint(scale));  // 2^-e of 2^e
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          if (fresh >> j & 1u) *reinterpret_cast<uint2*>(at + j * tpu * 8) = encode8<KIND, FP16>(x[j], inv, finite);
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          if (fresh >> j & 1u) *reinterpret_cast<uint2*>(at + j * tpu * 8) = encode8_div<KIND, FP16>(x[j], scale);
      }
      if (grown && old) {  // the codes of the other tokens move to the larger scale, or become 0
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          if (old >> j & 1u) {
            uint2* o = reinterpret_cast<uint2*>(at + j * tpu * 8);
            *o = stored ? recode8<KIND>(*o, was / scale) : make_uint2(0u, 0u);
          }
      }
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) x[j] = next[j];
  }
  // A page that other sequences hold is theirs too.
  if (refs > 1 && blockIdx.y == 0 && tid == 0) cache_error(c.control, BSA_ERR_INVALID_ARG, row);
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendParams& p, int sms, cudaStream_t s) {
  // Threads of a unit: 32 .. 1024, a multiple of the d / 8 chunks of a token.
  const int tpu = p.c.sb * p.c.d / (8 * kVec);
  const int threads = tpu < 256 ? 256 : tpu;
  const long long gx = (long long)p.n * p.blocks;
  if (gx > 0x7fffffffll) return cudaErrorInvalidValue;
  // Units of a (row, block) are spread over CTAs until there are about four CTAs
  // of 256 threads for each SM, which is what fits: more only repeat the way to
  // the page (eight: 23.7 us, four: 21.9 us for 6 x 4001 tokens of 16 heads).
  const int most = (2 * p.c.Hkv + threads / tpu - 1) / (threads / tpu);
  const long long want = (4ll * sms * 256 / threads + gx - 1) / gx;
  const int parts = (int)(want < 1 ? 1 : (want < most ? want : most));
  const dim3 grid((unsigned)gx, (unsigned)parts);
  auto kernel = [&](auto kind, auto fp16) {
    constexpr int K = decltype(kind)::value;
    constexpr bool F = decltype(fp16)::value;
    return p.seqs ? append_kernel<K, F, true> : append_kernel<K, F, false>;
  };
  using std::integral_constant;
  auto of_kind = [&](auto kind) {
    return p.fp16 ? kernel(kind, std::true_type{}) : kernel(kind, std::false_type{});
  };
  return launch_after(p.c.kind == BSA_CACHE_INT8 ? of_kind(integral_constant<int, BSA_CACHE_INT8>{})
                                                 : of_kind(integral_constant<int, BSA_CACHE_E4M3>{}),
                      grid, dim3(threads), 0, s, p, tpu);
}

}  // namespace bsa
