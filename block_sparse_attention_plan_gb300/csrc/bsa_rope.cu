// Rotary positions of queries and keys.
//
// Mathematics.  Pair i of a row at position t is turned by the angle t f_i and
// scaled by amp:
//   y_a = amp (x_a cos - x_b sin),  y_b = amp (x_b cos + x_a sin).
// The angle is held in turns as a 64-bit fraction: steps[i] = f_i / (2 pi) 2^64,
// so that t * steps[i] modulo 2^64, one integer product, is the exact remainder
// of a whole number of turns at any position (as a product in fp32 the angle is
// off by 2^-24 of itself: 0.06 radians at position 10^6).  Its upper 32 bits
// become the argument of sincospif, within 2^-25 half turns.
//
// What bounds it: every element is read and written once.  A lane holds eight
// pairs, as two vectors of 16 bytes, and their sines and cosines, which serve
// all heads of a token: a warp goes over the heads of q and then of k in rounds
// of 32 / (d / 16) heads, kUnroll rounds of loads in flight.  With few tokens
// (a decoding step) a token's rounds are spread over several warps, which then
// compute the sines anew.  (16001 tokens of 32 + 8 heads of 128: 55 us, 5.9 TB/s, 0.87 of a
// copy's rate; a token of each of 64 sequences: 3 to 5 us.)
#include "bsa_prompt.h"

namespace bsa {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kUnroll = 4;

template <bool FP16>
__device__ __forceinline__ float2 unpack(uint32_t w) {
  if constexpr (FP16) {
    float2 f;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(w));
    return f;
  }
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <bool FP16>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  uint32_t r;
  if constexpr (FP16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Turns the eight pairs of vectors a and b: (a[e], b[e]) where halves are paired,
// else neighbours, four of a and then four of b.
template <bool FP16, bool NEIGHBOURS>
__device__ __forceinline__ void turn(uint4& a, uint4& b, const float (&co)[8], const float (&si)[8]) {
  uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 x = unpack<FP16>(wa[e]), y = unpack<FP16>(wb[e]);
    if constexpr (NEIGHBOURS) {
      wa[e] = pack<FP16>(fmaf(x.x, co[e], -x.y * si[e]), fmaf(x.y, co[e], x.x * si[e]));
      wb[e] = pack<FP16>(fmaf(y.x, co[4 + e], -y.y * si[4 + e]), fmaf(y.y, co[4 + e], y.x * si[4 + e]));
    } else {
      wa[e] = pack<FP16>(fmaf(x.x, co[2 * e], -y.x * si[2 * e]), fmaf(x.y, co[2 * e + 1], -y.y * si[2 * e + 1]));
      wb[e] = pack<FP16>(fmaf(y.x, co[2 * e], x.x * si[2 * e]), fmaf(y.y, co[2 * e + 1], x.y * si[2 * e + 1]));
    }
  }
  a = make_uint4(wa[0], wa[1], wa[2], wa[3]);
  b = make_uint4(wb[0], wb[1], wb[2], wb[3]);
}

template <bool FP16, bool NEIGHBOURS>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  next_may_launch();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const long long token = w / p.parts;
  if (token >= (long long)p.B * p.T) return;
  const int part = (int)(w - token * p.parts);
  const int bi = (int)(token / p.T), t = (int)(token - (long long)bi * p.T);
  const int lanes = p.d / 16;  // of a head
  const int c = lane % lanes, per_round = 32 / lanes;
  const int turning = p.rot / 16;
  const bool turns = c < turning;
  if (!turns && !p.tail) return;
  // Elements of this lane's two vectors.
  const int ea = turns ? 8 * c : p.rot + 16 * (c - turning);
  const int eb = turns ? ea + p.rot / 2 : ea + 8;
  const int h0 = part * p.per * per_round + lane / lanes;
  const int h1 = min(p.H, (part + 1) * p.per * per_round);
  auto in = [&](int h) {
    const RopeRows& r = h < p.Hq ? p.q : p.k;
    return r.p + bi * r.sb + (h < p.Hq ? h : h - p.Hq) * r.sh + t * r.st;
  };
  auto out = [&](int h) {
    const RopeRows& r = h < p.Hq ? p.q : p.k;
    return r.o + bi * r.ob + (h < p.Hq ? h : h - p.Hq) * r.oh + t * r.ot;
  };
  uint4 a[kUnroll], b[kUnroll];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (h + u * per_round < h1) {
        const uint16_t* at = in(h + u * per_round);
        a[u] = load_written(reinterpret_cast<const uint4*>(at + ea));
        b[u] = load_written(reinterpret_cast<const uint4*>(at + eb));
      }
  };
  load(h0);  // (on their way while the sines are computed)
  float co[8], si[8];
  if (turns) {
    const long long pos = p.positions ? load_written(p.positions + token) : t;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = NEIGHBOURS ? (e < 4 ? 4 * c + e : 4 * c + p.rot / 4 + e - 4) : 8 * c + e;
      const uint64_t x = (uint64_t)pos * load_written(p.steps + i);
      sincospif((float)(int32_t)(x >> 32) * 0x1p-31f, &si[e], &co[e]);
      co[e] *= p.amp;
      si[e] *= p.inverse ? -p.amp : p.amp;
    }
  }
  for (int h = h0; h < h1; h += kUnroll * per_round) {
    if (h != h0) load(h);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (h + u * per_round < h1) {
        if (turns) turn<FP16, NEIGHBOURS>(a[u], b[u], co, si);
        uint16_t* at = out(h + u * per_round);
        *reinterpret_cast<uint4*>(at + ea) = a[u];
        *reinterpret_cast<uint4*>(at + eb) = b[u];
      }
  }
}

}  // namespace

int rope_heads_per_round(int d) { return 32 / (d / 16); }

cudaError_t launch_rope(const RopeParams& p, cudaStream_t s) {
  const long long warps = (long long)p.B * p.T * p.parts;
  const long long grid = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  auto kernel = p.fp16 ? (p.neighbours ? rope_kernel<true, true> : rope_kernel<true, false>)
                       : (p.neighbours ? rope_kernel<false, true> : rope_kernel<false, false>);
  return launch_after(kernel, dim3((unsigned)grid), dim3(kRopeThreads), 0, s, p);
}

}  // namespace bsa
