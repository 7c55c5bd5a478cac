// Attention weight that cached tokens gather.
//
// Mathematics.  For the M = g nq query rows that share a K/V head, with the
// logarithm of each row's sum from the attention that was run:
//   w[key] (+)= sum over rows of exp(scale <q, K_key> - lse(row))
// Scores as in bsa_cache_attn.cu: S^T = K Q^T by mma.m16n8k16 with the codes as
// the 16-row operand, exact in fp16, and rows divided by a power of two that
// brings their largest element into [1, 2) (fp16 to 2^-25 of that element); the
// score is one fused product and difference, fma(S, S_k qs, -lse), so that what
// is rounded is the small exponent and not two large terms of it.
//
// What bounds it: d bytes per key and K/V head at the memory's rate, and the 8
// of its weight.  Tokens' sums are independent of each other, so there is
// nothing to join: the tiles (32 keys at d = 128, 64 at d = 64: 4 KB) of all
// (sequence, K/V head) pairs form one line that the CTAs cut evenly, and in a
// CTA's piece of a pair the warps take tiles in turn (a window of selected
// blocks is spread over them).  Keys go from global memory to registers, 16
// bytes a lane: the order of a row's elements in the product is free, so a lane
// takes the words it has loaded; a tile's registers are refilled for the next
// tile as soon as they are converted, which keeps 4 KB a warp and 64 KB an SM
// on their way.  The rows wait in shared memory, prepared once per pair; with
// more than kWeighRows of them a piece is gone over again for the next ones.
#include "bsa_cache.h"
#include "bsa_cache_codes.cuh"
#include "bsa_device.cuh"

namespace bsa {
namespace {

using namespace dev;

constexpr int kWeighWarps = 8;
constexpr int kWeighThreads = 32 * kWeighWarps;
constexpr int kWeighRows = 128;  // query rows in shared memory at a time

template <int D>
struct WeighCfg {
  static constexpr int TK = 4096 / D;          // keys of a tile
  static constexpr int kGroups = TK / 16;      // keys of one matrix instruction, one scale each
  static constexpr int kVecs = D / 64;         // 16-byte vectors of a lane in a row of codes
  static constexpr int kRowBytes = 2 * D + 16; // of a prepared query row (16: no bank conflicts)
  static constexpr int kOffConst = kWeighRows * kRowBytes;       // {qs, lse} of each row
  static constexpr int kOffLim = kOffConst + kWeighRows * 8;     // last key position of each row (causal)
  static constexpr int kOffHead = kOffLim + kWeighRows * 4;      // head in the group
  static constexpr int kOffScan = kOffHead + kWeighRows * 4;     // prefix of the threads' tiles
  static constexpr int kSmem = kOffScan + (kWeighThreads + kWeighWarps + 1) * 4;
  static_assert(kSmem <= 48 * 1024, "no attribute needed");
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Sequence of batch row b (-1: none, or out of range), and its length (0 where
// the sequence, its length or the room for its weights is out of range).
__device__ __forceinline__ int weigh_seq(const CacheWeighParams& p, int b) {
  const int s = p.seqs ? load_written(p.seqs + b) : b;
  return s >= 0 && s < p.c.max_seqs ? s : -1;
}
__device__ __forceinline__ int weigh_len(const CacheWeighParams& p, int b) {
  const int s = weigh_seq(p, b);
  if (s < 0) return 0;
  const int n = load_written(p.c.lens + s);
  if (n < 0 || n > p.c.max_pages * p.c.page || n > p.stride) return 0;
  return n;
}

template <int D, int KIND>
__global__ void __launch_bounds__(kWeighThreads, 2) weigh_kernel(const __grid_constant__ CacheWeighParams p) {
  using C = WeighCfg<D>;
  constexpr int TK = C::TK, G = C::kGroups, NV = C::kVecs;
  extern __shared__ __align__(16) uint8_t smem[];
  const CacheDev& c = p.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int l4 = lane & 3, r8 = lane >> 2;
  float* s_const = reinterpret_cast<float*>(smem + C::kOffConst);
  int* s_lim = reinterpret_cast<int*>(smem + C::kOffLim);
  int* s_head = reinterpret_cast<int*>(smem + C::kOffHead);
  int* s_scan = reinterpret_cast<int*>(smem + C::kOffScan);
  const int lpage = 31 - __clz(c.page), lsb = 31 - __clz(c.sb), lbk = p.mask ? 31 - __clz(p.bk) : 0;
  next_may_launch();
  wait_for_previous();

  // Sequences and lengths out of range are recorded by the first CTA.
  if (blockIdx.x == 0) {
    for (int b = tid; b < p.B; b += kWeighThreads) {
      const int s = p.seqs ? load_written(p.seqs + b) : b;
      if (s == -1) continue;
      bool bad = s < 0 || s >= c.max_seqs;
      if (!bad) {
        const int n = load_written(c.lens + s);
        bad = n < 0 || n > c.max_pages * c.page || n > p.stride;
      }
      if (bad) cache_error(c.control, BSA_ERR_INVALID_ARG, b);
    }
  }
  // This CTA's piece of the line of tiles.
  const int per = (p.B + kWeighThreads - 1) / kWeighThreads;
  int sum = 0;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b < p.B) sum += (weigh_len(p, b) + TK - 1) / TK;
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) s_scan[kWeighThreads + warp] = inc;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWeighWarps; ++w) {
    const int x = s_scan[kWeighThreads + w];
    if (w < warp) before += x;
    total += x;
  }
  s_scan[tid] = before + inc - sum;  // tiles of a head ahead of this thread's rows
  __syncthreads();
  const long long line = (long long)total * c.Hkv;
  const long long lo = line * blockIdx.x / gridDim.x, hi = line * (blockIdx.x + 1) / gridDim.x;
  if (lo >= hi) return;
  // Batch row that holds place lo: the last thread whose rows begin at or before it.
  int first = 0;
  for (int step = kWeighThreads / 2; step; step >>= 1)
    if ((long long)s_scan[first + step] * c.Hkv <= lo) first += step;
  int b = first * per;
  long long base = (long long)s_scan[first] * c.Hkv;  // place where row b begins
  int len = b < p.B ? weigh_len(p, b) : 0;
  int tiles = (len + TK - 1) / TK;
  while (base + (long long)tiles * c.Hkv <= lo) {
    base += (long long)tiles * c.Hkv;
    len = weigh_len(p, ++b);
    tiles = (len + TK - 1) / TK;
  }
  int h = (int)((lo - base) / tiles);
  base += (long long)h * tiles;  // place where the pair (b, h) begins

  for (; base < hi;) {
    // Tiles [t0, t1) of the pair.
    const int t0 = (int)(lo > base ? lo - base : 0), t1 = (int)(hi - base < tiles ? hi - base : tiles);
    const int seq = weigh_seq(p, b);
    bool twice = false;
    if (p.seqs) {
      for (int a = tid; a < b; a += kWeighThreads) twice |= load_written(p.seqs + a) == seq;
      twice = __syncthreads_or(twice);
      if (twice && t0 == 0 && h == 0 && tid == 0) cache_error(c.control, BSA_ERR_INVALID_ARG, b);
    }
    if (!twice) {
      const int32_t* table = c.table + (size_t)seq * c.max_pages;
      float* weights = p.weights + ((size_t)seq * c.Hkv + h) * p.stride;
      const uint8_t* mask = p.mask ? p.mask + ((size_t)b * p.Hq + (size_t)h * p.g) * p.NKB : nullptr;
      const int fresh0 = len > p.fresh ? len - p.fresh : 0;  // weights from here on begin at 0
      const int free_end = p.causal ? len - p.nq + 1 : len;  // keys below it are seen by every query
      for (int m0 = 0; m0 < p.M; m0 += kWeighRows) {
        const int rows = min(p.M - m0, kWeighRows);
        // ------------------------------------------------------------ a tile's keys
        uint4 kv[G][2][NV];
        float sc[G];
        bool held[G];
        // Keys of group gr of tile t into its registers (nothing of no page).
        auto load_group = [&](int t, int gr) {
          const int j = t * TK + gr * 16;
          const int pg = j < len ? load_written(table + (j >> lpage)) : -1;
          held[gr] = pg >= 0 && pg < c.num_pages;
          sc[gr] = 0.f;
          if (!held[gr]) {
            if (j < len && lane == 0) cache_error(c.control, BSA_ERR_PLAN_MISMATCH, seq);
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int v = 0; v < NV; ++v) kv[gr][x][v] = make_uint4(0u, 0u, 0u, 0u);
            return;
          }
          const size_t row = ((size_t)pg * c.Hkv + h) * c.page + (j & (c.page - 1));
          sc[gr] = load_written(c.ks + (row >> lsb));
          const uint8_t* at = c.k + (row + r8) * D + 16 * l4;
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int v = 0; v < NV; ++v)
              kv[gr][x][v] = load_written(reinterpret_cast<const uint4*>(at + (size_t)x * 8 * D + 64 * v));
        };
        // The next tile at or past t that has something to do; bit x of `active`:
        // tile t32 + x kWeighWarps.
        int t32 = t0 + warp;
        uint32_t active = 0u;
        auto look = [&]() {
          const int t = t32 + lane * kWeighWarps;
          bool some = t < t1;
          if (some && p.mask && !(m0 == 0 && (t + 1) * TK > fresh0)) {
            some = false;
            for (int x = 0; x < p.g && !some; ++x)
#pragma unroll
              for (int q = 0; q < TK / 32; ++q) {
                const int kb = (t * TK + 32 * q) >> lbk;
                if (kb < p.NKB) some |= load_written(mask + (size_t)x * p.NKB + kb) != 0;
              }
          }
          active = __ballot_sync(0xffffffffu, some);
        };
        look();
        auto next_tile = [&]() -> int {  // -1: none is left
          while (!active) {
            t32 += 32 * kWeighWarps;
            if (t32 >= t1) return -1;
            look();
          }
          const int x = __ffs(active) - 1;
          active &= active - 1;
          return t32 + x * kWeighWarps;
        };
        int t = next_tile();
        if (t >= 0) {
#pragma unroll
          for (int gr = 0; gr < G; ++gr) load_group(t, gr);
        }
        // ------------------------------------------------------------ the rows
        __syncthreads();  // (those before them are used up)
        for (int m = warp * 8 + r8; m < ((rows + 7) & ~7); m += 8 * kWeighWarps) {
          // Four lanes a row: lane l4 has elements 64 v + 16 l4 .. + 15.
          uint32_t w[NV][8];
          const bool real = m < rows;
          const int hd = real ? (m0 + m) / p.nq : 0, i = real ? (m0 + m) - hd * p.nq : 0;
          const uint16_t* at = p.q.p + (long long)b * p.q.sb + (long long)(h * p.g + hd) * p.q.sh + (long long)i * p.q.st + 16 * l4;
          uint32_t top = 0u;
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
            if (real) {
              x = load_written(reinterpret_cast<const uint4*>(at + 64 * v));
              y = load_written(reinterpret_cast<const uint4*>(at + 64 * v + 8));
            }
            const uint32_t u[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              w[v][e] = u[e];
              const float2 f = elems_to_float2(u[e], p.fp16);
              top = max(top, max(__float_as_uint(f.x) & 0x7fffffffu, __float_as_uint(f.y) & 0x7fffffffu));
            }
          }
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          // 2^e <= largest < 2^(e+1); below 2^-126 e stays there (elements then are
          // at least 2^-133 and keep their bits).
          const int e = max(min((int)(top >> 23), 254), 1) - 127;
          const float inv = e == 127 ? 0x1p-127f : __uint_as_float((uint32_t)(127 - e) << 23);
          uint8_t* dst = smem + m * C::kRowBytes + 32 * l4;
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            uint32_t o[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const float2 f = elems_to_float2(w[v][x], p.fp16);
              asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o[x]) : "f"(f.y * inv), "f"(f.x * inv));
            }
            *reinterpret_cast<uint4*>(dst + 128 * v) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(dst + 128 * v + 16) = make_uint4(o[4], o[5], o[6], o[7]);
          }
          if (l4 == 0) {
            const float z = real ? load_written(p.lse + ((size_t)b * p.Hq + h * p.g + hd) * p.nq + i) : INFINITY;
            s_const[2 * m] = real ? p.scale * __uint_as_float((uint32_t)(e + 127) << 23) : 0.f;
            s_const[2 * m + 1] = z == -INFINITY ? INFINITY : z;  // a row that attends nothing gives nothing
            s_lim[m] = p.causal ? len - p.nq + i : 0x7fffffff;
            s_head[m] = hd;
          }
        }
        __syncthreads();
        // ------------------------------------------------------------ the tiles
        while (t >= 0) {
          const int key0 = t * TK;
          const int tn = next_tile();
          // Heads of the group that select the tile, for each 32 keys.
          uint32_t sel[TK / 32];
#pragma unroll
          for (int q = 0; q < TK / 32; ++q) {
            sel[q] = 0xffffffffu;
            if (p.mask) {
              const int kb = (key0 + 32 * q) >> lbk;
              bool on = false;
              if (kb < p.NKB)
                for (int x = lane; x < p.g; x += 32) on |= load_written(mask + (size_t)x * p.NKB + kb) != 0;
              sel[q] = __ballot_sync(0xffffffffu, on);
            }
          }
          // Weights so far of the tokens that this lane writes: token 8 (l4 + 4 x) + r8.
          float w[TK / 32];
#pragma unroll
          for (int x = 0; x < TK / 32; ++x) {
            const int j = key0 + 8 * (l4 + 4 * x) + r8;
            w[x] = j < len && (m0 > 0 || j < fresh0) ? weights[j] : 0.f;
          }
#pragma unroll
          for (int gr = 0; gr < G; ++gr) {
            uint32_t a[NV][4][4];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              const uint32_t lo4[4] = {kv[gr][0][v].x, kv[gr][0][v].y, kv[gr][0][v].z, kv[gr][0][v].w};
              const uint32_t hi4[4] = {kv[gr][1][v].x, kv[gr][1][v].y, kv[gr][1][v].z, kv[gr][1][v].w};
#pragma unroll
              for (int s = 0; s < 4; ++s) {
                const uint2 x = codes_to_half4<KIND>(lo4[s]), y = codes_to_half4<KIND>(hi4[s]);
                a[v][s][0] = x.x;
                a[v][s][1] = y.x;
                a[v][s][2] = x.y;
                a[v][s][3] = y.y;
              }
            }
            const float scale = sc[gr];
            const bool there = held[gr];
            if (tn >= 0) load_group(tn, gr);
            const int j0 = key0 + gr * 16 + r8;  // this lane's keys: j0, j0 + 8
            float acc0 = 0.f, acc1 = 0.f;
            if (there && sel[gr / 2]) {
              for (int n = 0; n < rows; n += 8) {
                float s[4] = {0.f, 0.f, 0.f, 0.f};
                const uint8_t* br = smem + (n + r8) * C::kRowBytes + 32 * l4;
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                  for (int x = 0; x < 2; ++x) {
                    const uint4 bw = *reinterpret_cast<const uint4*>(br + 128 * v + 16 * x);
                    mma16816(s, a[v][2 * x][0], a[v][2 * x][1], a[v][2 * x][2], a[v][2 * x][3], bw.x, bw.y);
                    mma16816(s, a[v][2 * x + 1][0], a[v][2 * x + 1][1], a[v][2 * x + 1][2], a[v][2 * x + 1][3], bw.z,
                             bw.w);
                  }
                const float4 cst = *reinterpret_cast<const float4*>(s_const + 2 * (n + 2 * l4));
                constexpr float kLog2e = 1.4426950408889634f;
                float p00 = ex2_approx(fmaf(s[0], scale * cst.x, -cst.y) * kLog2e);
                float p01 = ex2_approx(fmaf(s[1], scale * cst.z, -cst.w) * kLog2e);
                float p10 = ex2_approx(fmaf(s[2], scale * cst.x, -cst.y) * kLog2e);
                float p11 = ex2_approx(fmaf(s[3], scale * cst.z, -cst.w) * kLog2e);
                if (p.mask) {
                  const int h0 = s_head[n + 2 * l4], h1 = s_head[n + 2 * l4 + 1];
                  bool on0, on1;
                  if (p.g <= 32) {
                    on0 = sel[gr / 2] >> h0 & 1u;
                    on1 = sel[gr / 2] >> h1 & 1u;
                  } else {
                    const int kb = j0 >> lbk;
                    on0 = kb < p.NKB && load_written(mask + (size_t)h0 * p.NKB + kb) != 0;
                    on1 = kb < p.NKB && load_written(mask + (size_t)h1 * p.NKB + kb) != 0;
                  }
                  if (!on0) p00 = p10 = 0.f;
                  if (!on1) p01 = p11 = 0.f;
                }
                if (j0 + 8 >= free_end) {  // (also keys past the length: their sums are not stored)
                  const int2 lim = *reinterpret_cast<const int2*>(s_lim + n + 2 * l4);
                  if (j0 > lim.x) p00 = 0.f;
                  if (j0 > lim.y) p01 = 0.f;
                  if (j0 + 8 > lim.x) p10 = 0.f;
                  if (j0 + 8 > lim.y) p11 = 0.f;
                }
                if (n + 2 * l4 >= rows) p00 = p10 = 0.f;
                if (n + 2 * l4 + 1 >= rows) p01 = p11 = 0.f;
                acc0 += p00 + p01;
                acc1 += p10 + p11;
              }
              acc0 += __shfl_xor_sync(0xffffffffu, acc0, 1);
              acc1 += __shfl_xor_sync(0xffffffffu, acc1, 1);
              acc0 += __shfl_xor_sync(0xffffffffu, acc0, 2);
              acc1 += __shfl_xor_sync(0xffffffffu, acc1, 2);
            }
            // Keys 0-7 of group gr are column 2 gr of the tile's eights, keys 8-15 the next.
            if ((2 * gr & 3) == l4) w[gr / 2] += acc0;
            if (((2 * gr + 1) & 3) == l4) w[gr / 2] += acc1;
          }
#pragma unroll
          for (int x = 0; x < TK / 32; ++x) {
            const int j = key0 + 8 * (l4 + 4 * x) + r8;
            if (j < len) weights[j] = w[x];
          }
          t = tn;
        }
      }
    }
    // To the next pair with tiles.
    base += tiles;
    if (++h == c.Hkv) {
      h = 0;
      do {
        if (++b >= p.B) return;
        len = weigh_len(p, b);
        tiles = (len + TK - 1) / TK;
      } while (tiles == 0);
    }
  }
}

}  // namespace

cudaError_t launch_cache_weigh(const CacheWeighParams& p, int sms, cudaStream_t s) {
  auto go = [&](auto kernel, int smem) { return launch_after(kernel, dim3(2 * sms), dim3(kWeighThreads), smem, s, p); };
  const bool i8 = p.c.kind == BSA_CACHE_INT8;
  if (p.c.d == 64)
    return i8 ? go(weigh_kernel<64, BSA_CACHE_INT8>, WeighCfg<64>::kSmem)
              : go(weigh_kernel<64, BSA_CACHE_E4M3>, WeighCfg<64>::kSmem);
  return i8 ? go(weigh_kernel<128, BSA_CACHE_INT8>, WeighCfg<128>::kSmem)
            : go(weigh_kernel<128, BSA_CACHE_E4M3>, WeighCfg<128>::kSmem);
}

}  // namespace bsa
