// Keys and values of a cache's sequences as bf16 [B][Hkv][Nk][d], for the
// block-sparse forward.
//
// The forward's products are bound by the tensor pipe and read each K/V tile
// once per query tile that selects it, so the codes are converted once, by a
// pass that the memory bounds (1 byte read and 2 written per element), and not
// again in every tile's inner loop.  Positions at and past a sequence's length
// become zero: the forward masks them but multiplies what they hold.
#include "bsa_cache.h"
#include "bsa_cache_codes.cuh"
#include "bsa_device.cuh"

namespace bsa {
namespace {

using namespace dev;

constexpr int kThreads = 256;

template <int KIND>
__global__ void __launch_bounds__(kThreads) load_kernel(const CacheDev c, const int32_t* seqs, int B, int Nk,
                                                        uint16_t* k_out, uint16_t* v_out, int32_t* lens_out) {
  next_may_launch();
  wait_for_previous();
  // Work item: 16 codes of a token.
  const int cols = c.d / 16;
  const long long per = (long long)Nk * cols;              // of one (batch row, head)
  const int bh = blockIdx.y, b = bh / c.Hkv, h = bh % c.Hkv;
  const int seq = seqs ? __ldg(seqs + b) : b;
  const bool known = seq >= 0 && seq < c.max_seqs;
  int len = known ? __ldg(c.lens + seq) : 0;
  len = min(max(len, 0), min(Nk, c.max_pages * c.page));
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0 && blockIdx.z == 0) {
    lens_out[b] = len;
    if (!known && seq != -1) cache_error(c.control, BSA_ERR_INVALID_ARG, b);
  }
  const bool isv = blockIdx.z != 0;
  const uint8_t* codes = isv ? c.v : c.k;
  const float* scales = isv ? c.vs : c.ks;
  uint16_t* out = (isv ? v_out : k_out) + (size_t)bh * Nk * c.d;
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < per; i += (long long)gridDim.x * kThreads) {
    const int key = (int)(i / cols), col = (int)(i % cols);
    uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    if (key < len) {
      int ph = __ldg(c.table + (size_t)seq * c.max_pages + key / c.page);
      if (ph < 0 || ph >= c.num_pages) {
        cache_error(c.control, BSA_ERR_PLAN_MISMATCH, seq);
      } else {
        const size_t row = ((size_t)ph * c.Hkv + h) * c.page + key % c.page;
        const uint4 x = __ldcs(reinterpret_cast<const uint4*>(codes + row * c.d + col * 16));
        const float s = __ldg(scales + row / c.sb);
        const uint32_t cw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint2 hh = codes_to_half4<KIND>(cw[e]);
          const float2 f0 = half2_to_float2(hh.x), f1 = half2_to_float2(hh.y);
          w[2 * e] = pack_bf16x2(f0.x * s, f0.y * s);
          w[2 * e + 1] = pack_bf16x2(f1.x * s, f1.y * s);
        }
      }
    }
    st_global_v8(out + (size_t)key * c.d + col * 16, w);
  }
}

}  // namespace

cudaError_t launch_cache_load(const CacheDev& c, const int32_t* seqs, int B, int Nk, uint16_t* k, uint16_t* v,
                              int32_t* lens, cudaStream_t s) {
  const long long items = (long long)Nk * (c.d / 16);
  long long gx = (items + 4 * kThreads - 1) / (4 * kThreads);
  if (gx < 1) gx = 1;
  const dim3 grid((unsigned)gx, (unsigned)(B * c.Hkv), 2);
  return launch_after(c.kind == BSA_CACHE_INT8 ? load_kernel<BSA_CACHE_INT8> : load_kernel<BSA_CACHE_E4M3>, grid,
                      dim3(kThreads), 0, s, c, seqs, B, Nk, k, v, lens);
}

}  // namespace bsa
