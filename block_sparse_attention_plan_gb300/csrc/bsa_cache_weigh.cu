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
// nothing to join: the tiles (4 KB: 32 keys at d = 128, 64 at d = 64) of all
// (sequence, K/V head) pairs form one line that the CTAs cut evenly, and in a
// CTA's piece of a pair the warps take tiles in turn (a window of selected
// blocks is spread over them).  Each warp feeds itself: a ring of three tiles in shared
// memory, filled by bulk copies of a page's rows, the next one requested as soon as a
// tile is in registers.  The order of a row's elements in the product is free, so a
// lane takes 16-byte vectors as they lie (at d = 128 with two lanes to a bank, which
// costs less than turning halves about).  Pages, scales and weights are read a tile ahead.  The rows wait in shared memory, prepared once per
// pair.  From 33 rows on the products are what costs (128 rows a pass, pieces are gone
// over again for more): tiles of 16 keys, so that few tokens spread over all warps.
//
// Measured: 32 sequences of 500 to 32768 tokens, a query of 32 heads over 8 of 128, E4M3:
// 103 us, 5.7 TB/s (operands read from global memory by their lanes 153, through the ring
// 131, with up to 8 rows in registers 119, pieces cut with kHead 105: 12, 6, 20 or 32
// places 105, 113, 104, 105).  4 of 3000 to 12001, 32 queries of 32 heads over 8 of 64, INT8:
// 28 us (tiles of 64 keys 46).  With masks the line is still cut by tokens, selected or not:
// the first case with blocks of 64, of a head the first, the last 16 and 16 others: 101 us for a
// quarter of the bytes (CTAs are busy 44 % of that time; those with a sequence's last blocks go on
// the longest), with 64 others 110; 16 sequences, 8 queries: 109 (96 without the mask).
#include "bsa_cache.h"
#include "bsa_cache_codes.cuh"
#include "bsa_device.cuh"

namespace bsa {
namespace {

using namespace dev;

constexpr int kWeighWarps = 8;
constexpr int kWeighThreads = 32 * kWeighWarps;
// What a pair's beginning (its rows, the first tiles' way) costs a CTA, in tiles.
constexpr int kHead = 16;

// ROWS: query rows in shared memory at a time.
template <int D, int ROWS>
struct WeighCfg {
  static constexpr int kGroups = ROWS <= 32 ? 256 / D : 1;  // of 16 keys: one matrix instruction, one scale each
  static constexpr int TK = 16 * kGroups;      // keys of a tile
  static constexpr int kTileBytes = TK * D;
  static constexpr int kStages = 3;            // of a warp
  static constexpr int kVecs = D / 64;         // 16-byte vectors of a lane in a row of codes
  static constexpr int kCols = (TK + 31) / 32; // tokens that a lane writes
  static constexpr int kRowBytes = 2 * D + 16; // of a prepared query row (16: no bank conflicts)
  static constexpr int kOffRows = kWeighWarps * kStages * kTileBytes;
  static constexpr int kOffConst = kOffRows + ROWS * kRowBytes;  // {qs, lse} of each row
  static constexpr int kOffLim = kOffConst + ROWS * 8;           // last key position of each row (causal; -1: it has no sum)
  static constexpr int kOffHead = kOffLim + ROWS * 4;            // head in the group
  static constexpr int kOffBar = kOffHead + ROWS * 4;            // full [warps][stages]
  static constexpr int kOffTile = kOffBar + kWeighWarps * kStages * 8;  // [warps][stages][8]: tile, pool rows of its groups
  static constexpr int kOffScan = kOffTile + kWeighWarps * kStages * 32;  // prefix of the threads' tiles
  static constexpr int kOffAbort = kOffScan + (kWeighThreads + kWeighWarps) * 4;
  static constexpr int kSmem = kOffAbort + 16;
  static_assert(kSmem <= 113 * 1024, "two CTAs an SM");
};
enum WeighSite : int { kSiteWeighTile = 0x58 };

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Bulk copy of `bytes` (a multiple of 16) into shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
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

template <int D, int KIND, int ROWS>
__global__ void __launch_bounds__(kWeighThreads, 2) weigh_kernel(const __grid_constant__ CacheWeighParams p) {
  using C = WeighCfg<D, ROWS>;
  constexpr int TK = C::TK, G = C::kGroups, NV = C::kVecs;
  extern __shared__ __align__(128) uint8_t smem[];
  const CacheDev& c = p.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int l4 = lane & 3, r8 = lane >> 2;
  uint8_t* s_rows = smem + C::kOffRows;
  float* s_const = reinterpret_cast<float*>(smem + C::kOffConst);
  int* s_lim = reinterpret_cast<int*>(smem + C::kOffLim);
  int* s_head = reinterpret_cast<int*>(smem + C::kOffHead);
  int* s_tile = reinterpret_cast<int*>(smem + C::kOffTile) + warp * C::kStages * 8;
  int* s_scan = reinterpret_cast<int*>(smem + C::kOffScan);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::kOffAbort);
  const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * C::kStages * C::kTileBytes);
  const uint32_t bars = smem_u32(smem) + C::kOffBar + (uint32_t)(warp * C::kStages * 8);
  const Watchdog wd{s_abort, c.control + kCacheStatus, c.control + kCacheDetail, p.watchdog_ns};
  const int lpage = 31 - __clz(c.page), lsb = 31 - __clz(c.sb), lbk = p.mask ? 31 - __clz(p.bk) : 0;
  if (tid == 0) {
    *s_abort = 0;
    for (int i = 0; i < kWeighWarps * C::kStages; ++i) mbar_init(smem_u32(smem) + C::kOffBar + 8 * i, 1);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
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
  // This CTA's piece of the line: kHead places and the tiles of every pair that has some.
  const int per = (p.B + kWeighThreads - 1) / kWeighThreads;
  auto places_of = [&](int row) {
    const int t = (weigh_len(p, row) + TK - 1) / TK;
    return t > 0 ? t + kHead : 0;
  };
  int sum = 0;
  for (int i = 0; i < per; ++i) {
    const int row = tid * per + i;
    if (row < p.B) sum += places_of(row);
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
  s_scan[tid] = before + inc - sum;  // places of a head ahead of this thread's rows
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
  int places = b < p.B ? places_of(b) : 0;
  while (base + (long long)places * c.Hkv <= lo) {
    base += (long long)places * c.Hkv;
    places = places_of(++b);
  }
  int h = (int)((lo - base) / places);
  base += (long long)h * places;  // place where the pair (b, h) begins
  int len = weigh_len(p, b);

  uint32_t asked = 0, used = 0;  // tiles requested and taken by this warp
  bool gave_up = false;          // a wait of this warp ran out: it requests nothing more
  for (; base < hi;) {
    // Tiles [t0, t1) of the pair.
    const long long row0 = base + kHead;
    const int t0 = (int)(lo > row0 ? lo - row0 : 0), t1 = (int)(hi - row0 < places - kHead ? hi - row0 : places - kHead);
    const int seq = weigh_seq(p, b);
    bool twice = false;
    if (p.seqs) {
      for (int a = tid; a < b; a += kWeighThreads) twice |= load_written(p.seqs + a) == seq;
      twice = __syncthreads_or(twice);
      if (twice && lo <= base && h == 0 && tid == 0) cache_error(c.control, BSA_ERR_INVALID_ARG, b);
    }
    if (!twice && t0 < t1) {
      const int32_t* table = c.table + (size_t)seq * c.max_pages;
      float* weights = p.weights + ((size_t)seq * c.Hkv + h) * p.stride;
      const uint8_t* mask = p.mask ? p.mask + ((size_t)b * p.Hq + (size_t)h * p.g) * p.NKB : nullptr;
      const int fresh0 = len > p.fresh ? len - p.fresh : 0;  // weights from here on begin at 0
      const int free_end = p.causal ? len - p.nq + 1 : len;  // keys below it are seen by every query that has a sum
      for (int m0 = 0; m0 < p.M; m0 += ROWS) {
        const int rows = min(p.M - m0, ROWS);
        // ------------------------------------------------------------ requests
        // The next tile that has something to do; bit x of `active`: tile
        // t32 + x kWeighWarps.
        int t32 = t0 + warp;
        uint32_t active = 0u;
        auto look = [&]() {
          const int t = t32 + lane * kWeighWarps;
          bool some = t < t1;
          if (some && p.mask && !(m0 == 0 && (t + 1) * TK > fresh0)) {
            some = false;
            for (int x = 0; x < p.g && !some; ++x)
#pragma unroll
              for (int q = 0; q < C::kCols; ++q) {
                const int kb = (t * TK + 32 * q) >> lbk;
                if (kb < p.NKB) some |= load_written(mask + (size_t)x * p.NKB + kb) != 0;
              }
          }
          active = __ballot_sync(0xffffffffu, some);
        };
        look();
        // The tile to request next (-1: none is left) and, in lane g, the page of its
        // group g, read a request ahead.
        int t_next, pg_next;
        auto advance = [&]() {
          t_next = -1;
          while (!active) {
            t32 += 32 * kWeighWarps;
            if (t32 >= t1) return;
            look();
          }
          const int x = __ffs(active) - 1;
          active &= active - 1;
          t_next = t32 + x * kWeighWarps;
          const int j = t_next * TK + 16 * lane;
          pg_next = lane < G && j < len ? load_written(table + (j >> lpage)) : -1;
        };
        int waiting = 0;  // tiles on their way
        // Requests the next tile into the stage after the last one's; the first lane of a
        // page's groups copies them.
        const int run = min(c.page, TK);
        auto request = [&]() {
          if (t_next < 0 || gave_up) return;
          const uint32_t s = asked % C::kStages, bar = bars + 8 * s;
          int row = -1;
          if (lane < G) {
            const int j = t_next * TK + 16 * lane;
            if (j < len) {
              if (pg_next >= 0 && pg_next < c.num_pages) row = (pg_next * c.Hkv + h) * c.page + (j & (c.page - 1));
              else cache_error(c.control, BSA_ERR_PLAN_MISMATCH, seq);
            }
            s_tile[s * 8 + 1 + lane] = row;
          }
          const bool copies = row >= 0 && ((16 * lane) & (run - 1)) == 0;
          const int parts = __popc(__ballot_sync(0xffffffffu, copies));
          if (lane == 0) {
            s_tile[s * 8] = t_next;
            if (parts) mbar_arrive_expect_tx(bar, (uint32_t)(parts * run * D));
            else mbar_arrive(bar);
          }
          __syncwarp();
          if (copies)
            bulk_load(ring + s * C::kTileBytes + (uint32_t)(16 * lane * D), c.k + (size_t)row * D, (uint32_t)(run * D), bar);
          ++asked;
          ++waiting;
          advance();
        };
        advance();
#pragma unroll 1
        for (int i = 0; i < C::kStages; ++i) request();
        // Of the next tile, read a tile ahead: the scales of its groups, and the weights so far of
        // the tokens that this lane writes (token 8 (l4 + 4 x) + r8).
        float sc_next[G], w_next[C::kCols];
        auto ahead = [&]() {
          const int* e = s_tile + (used % C::kStages) * 8;
#pragma unroll
          for (int gr = 0; gr < G; ++gr) {
            const int row = e[1 + gr];
            sc_next[gr] = row >= 0 ? load_written(c.ks + (row >> lsb)) : 0.f;
          }
#pragma unroll
          for (int x = 0; x < C::kCols; ++x) {
            const int to = 8 * (l4 + 4 * x) + r8, j = e[0] * TK + to;
            w_next[x] = to < TK && j < len && (m0 > 0 || j < fresh0) ? weights[j] : 0.f;
          }
        };
        __syncwarp();
        if (waiting) ahead();
        // ------------------------------------------------------------ the rows
        __syncthreads();  // (those before them are used up)
        bool some_none = false;
        for (int m = warp * 8 + r8; m < ((rows + 7) & ~7); m += 8 * kWeighWarps) {
          // Four lanes a row: lane l4 has elements 64 v + 16 l4 .. + 15.
          uint32_t w[NV][8];
          const bool real = m < rows;
          const int hd = (m0 + min(m, rows - 1)) / p.nq, i = real ? (m0 + m) - hd * p.nq : 0;
          // A row of no sum, and one that is none, give nothing: zeros, and e^-inf.
          const float z = real ? load_written(p.lse + ((size_t)b * p.Hq + h * p.g + hd) * p.nq + i) : -INFINITY;
          const uint16_t* at = p.q.p + (long long)b * p.q.sb + (long long)(h * p.g + hd) * p.q.sh + (long long)i * p.q.st + 16 * l4;
          uint32_t top = 0u;
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
            if (real) {
              x = load_written(reinterpret_cast<const uint4*>(at + 64 * v));
              y = load_written(reinterpret_cast<const uint4*>(at + 64 * v + 8));
            }
            if (z == -INFINITY) x = y = make_uint4(0u, 0u, 0u, 0u);  // (whatever the row holds)
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
          uint8_t* dst = s_rows + m * C::kRowBytes + 32 * l4;
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
            s_const[2 * m] = real ? p.scale * __uint_as_float((uint32_t)(e + 127) << 23) : 0.f;
            s_const[2 * m + 1] = z == -INFINITY ? INFINITY : z;
            s_lim[m] = z == -INFINITY ? -1 : p.causal ? len - p.nq + i : 0x7fffffff;
            s_head[m] = hd;
          }
          some_none |= real && z == -INFINITY;
        }
        // Rows of no sum see no key: one that is no number would make NaN even of their zeros.
        // (Those that only fill up an eight have the last row's head and see no other key than it:
        // their NaN is one that the row gives itself.)
        const int late_from = __syncthreads_or(some_none) ? 0 : free_end;
        // Up to 8 rows stay in registers: this lane's elements of row r8, and what rows
        // 2 l4 and 2 l4 + 1 are finished with.
        uint4 rb[ROWS == 8 ? 2 * NV : 1];
        float4 rc = make_float4(0.f, 0.f, 0.f, 0.f);
        int2 rl = make_int2(0, 0), rh = make_int2(0, 0);
        if constexpr (ROWS == 8) {
#pragma unroll
          for (int v = 0; v < 2 * NV; ++v)
            rb[v] = *reinterpret_cast<const uint4*>(s_rows + r8 * C::kRowBytes + 32 * l4 + 128 * (v >> 1) + 16 * (v & 1));
          rc = *reinterpret_cast<const float4*>(s_const + 4 * l4);
          rl = *reinterpret_cast<const int2*>(s_lim + 2 * l4);
          rh = *reinterpret_cast<const int2*>(s_head + 2 * l4);
        }
        // Weights of keys j0, j0 + 8 for two rows, from their products x4; their sums.
        auto weigh2 = [&](const float (&x4)[4], float scale, const float4& cst, const int2& lim, const int2& hd, int j0,
                          uint32_t sel, bool late, float& s0, float& s1) {
          constexpr float kLog2e = 1.4426950408889634f;
          const float q0 = scale * cst.x, q1 = scale * cst.z;
          float p00 = ex2_approx(fmaf(x4[0], q0, -cst.y) * kLog2e);
          float p01 = ex2_approx(fmaf(x4[1], q1, -cst.w) * kLog2e);
          float p10 = ex2_approx(fmaf(x4[2], q0, -cst.y) * kLog2e);
          float p11 = ex2_approx(fmaf(x4[3], q1, -cst.w) * kLog2e);
          if (p.mask) {
            bool on0, on1;
            if (p.g <= 32) {
              on0 = sel >> hd.x & 1u;
              on1 = sel >> hd.y & 1u;
            } else {
              const int kb = j0 >> lbk;
              on0 = kb < p.NKB && load_written(mask + (size_t)hd.x * p.NKB + kb) != 0;
              on1 = kb < p.NKB && load_written(mask + (size_t)hd.y * p.NKB + kb) != 0;
            }
            if (!on0) p00 = p10 = 0.f;
            if (!on1) p01 = p11 = 0.f;
          }
          if (late) {  // (also keys past the length: their sums are not stored)
            if (j0 > lim.x) p00 = 0.f;
            if (j0 > lim.y) p01 = 0.f;
            if (j0 + 8 > lim.x) p10 = 0.f;
            if (j0 + 8 > lim.y) p11 = 0.f;
          }
          s0 += p00 + p01;
          s1 += p10 + p11;
        };
        // ------------------------------------------------------------ the tiles
        for (; waiting; --waiting) {
          const uint32_t s = used % C::kStages;
          const int key0 = s_tile[s * 8] * TK;
          float w[C::kCols];
#pragma unroll
          for (int x = 0; x < C::kCols; ++x) w[x] = w_next[x];
          // Heads of the group that select the tile, for each 32 keys.
          uint32_t sel[C::kCols];
#pragma unroll
          for (int q = 0; q < C::kCols; ++q) {
            sel[q] = 0xffffffffu;
            if (p.mask) {
              const int kb = (key0 + 32 * q) >> lbk;
              bool on = false;
              if (kb < p.NKB)
                for (int x = lane; x < p.g; x += 32) on |= load_written(mask + (size_t)x * p.NKB + kb) != 0;
              sel[q] = __ballot_sync(0xffffffffu, on);
            }
          }
          if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * s, (used / C::kStages) & 1u, wd, kSiteWeighTile))) break;
          uint4 kv[G][2][NV];
          float sc[G];
          bool held[G];
#pragma unroll
          for (int gr = 0; gr < G; ++gr) {
            sc[gr] = sc_next[gr];
            held[gr] = s_tile[s * 8 + 1 + gr] >= 0;
            const uint32_t at = ring + s * C::kTileBytes + (uint32_t)((16 * gr + r8) * D + 16 * l4);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
              for (int v = 0; v < NV; ++v) kv[gr][x][v] = ld_shared_v4(at + x * 8 * D + 64 * v);
            }
          }
          ++used;
          __syncwarp();  // the stage has been read: refill it
          request();
          __syncwarp();
          if (waiting > 1) ahead();
          // Sums of the tile's eights of keys: 2 gr and 2 gr + 1 are those of group gr.
          float eights[2 * G];
#pragma unroll
          for (int gr = 0; gr < G; ++gr) {
            const float scale = sc[gr];
            const int j0 = key0 + gr * 16 + r8;  // this lane's keys: j0, j0 + 8
            const bool late = key0 + gr * 16 + 15 >= late_from;
            float acc0 = 0.f, acc1 = 0.f;
            // This lane's word s4 of vector v as operand registers.
            auto operand = [&](int v, int s4, uint32_t (&a)[4]) {
              const uint4 lo = kv[gr][0][v], hi = kv[gr][1][v];
              const uint2 x = codes_to_half4<KIND>(s4 == 0 ? lo.x : s4 == 1 ? lo.y : s4 == 2 ? lo.z : lo.w);
              const uint2 y = codes_to_half4<KIND>(s4 == 0 ? hi.x : s4 == 1 ? hi.y : s4 == 2 ? hi.z : hi.w);
              a[0] = x.x;
              a[1] = y.x;
              a[2] = x.y;
              a[3] = y.y;
            };
            if constexpr (ROWS == 8) {
              float x4[4] = {0.f, 0.f, 0.f, 0.f}, y4[4] = {0.f, 0.f, 0.f, 0.f};  // (two chains of products)
#pragma unroll
              for (int v = 0; v < 2 * NV; ++v) {
                uint32_t a[4];
                operand(v >> 1, 2 * (v & 1), a);
                mma16816(x4, a[0], a[1], a[2], a[3], rb[v].x, rb[v].y);
                operand(v >> 1, 2 * (v & 1) + 1, a);
                mma16816(y4, a[0], a[1], a[2], a[3], rb[v].z, rb[v].w);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) x4[e] += y4[e];
              weigh2(x4, scale, rc, rl, rh, j0, sel[gr / 2], late, acc0, acc1);
              if (!held[gr]) acc0 = acc1 = 0.f;
            } else if (held[gr] && sel[gr / 2]) {
              uint32_t a[NV][4][4];
#pragma unroll
              for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int s4 = 0; s4 < 4; ++s4) operand(v, s4, a[v][s4]);
              auto products = [&](int n, float (&x4)[4]) {
                float y4[4] = {0.f, 0.f, 0.f, 0.f};
                const uint8_t* br = s_rows + (n + r8) * C::kRowBytes + 32 * l4;
#pragma unroll
                for (int e = 0; e < 4; ++e) x4[e] = 0.f;
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                  for (int x = 0; x < 2; ++x) {
                    const uint4 bw = *reinterpret_cast<const uint4*>(br + 128 * v + 16 * x);
                    mma16816(x4, a[v][2 * x][0], a[v][2 * x][1], a[v][2 * x][2], a[v][2 * x][3], bw.x, bw.y);
                    mma16816(y4, a[v][2 * x + 1][0], a[v][2 * x + 1][1], a[v][2 * x + 1][2], a[v][2 * x + 1][3], bw.z,
                             bw.w);
                  }
#pragma unroll
                for (int e = 0; e < 4; ++e) x4[e] += y4[e];
              };
              if (!p.mask && !late) {  // every row sees these keys
#pragma unroll(ROWS > 32 ? 256 / D : 1)
                for (int n = 0; n < rows; n += 8) {
                  float x4[4];
                  products(n, x4);
                  const float4 cst = *reinterpret_cast<const float4*>(s_const + 2 * (n + 2 * l4));
                  constexpr float kLog2e = 1.4426950408889634f;
                  const float q0 = scale * cst.x, q1 = scale * cst.z;
                  acc0 += ex2_approx(fmaf(x4[0], q0, -cst.y) * kLog2e) + ex2_approx(fmaf(x4[1], q1, -cst.w) * kLog2e);
                  acc1 += ex2_approx(fmaf(x4[2], q0, -cst.y) * kLog2e) + ex2_approx(fmaf(x4[3], q1, -cst.w) * kLog2e);
                }
              } else {
#pragma unroll 1
                for (int n = 0; n < rows; n += 8) {
                  float x4[4];
                  products(n, x4);
                  weigh2(x4, scale, *reinterpret_cast<const float4*>(s_const + 2 * (n + 2 * l4)),
                         *reinterpret_cast<const int2*>(s_lim + n + 2 * l4), *reinterpret_cast<const int2*>(s_head + n + 2 * l4),
                         j0, sel[gr / 2], late, acc0, acc1);
                }
              }
            }
            eights[2 * gr] = acc0;
            eights[2 * gr + 1] = acc1;
          }
          // Over the four lanes of a key: lane l4 gets the sum of eight l4 (+ 4 x).
          if constexpr (G == 1) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              eights[e] += __shfl_xor_sync(0xffffffffu, eights[e], 1);
              eights[e] += __shfl_xor_sync(0xffffffffu, eights[e], 2);
            }
            w[0] += l4 & 1 ? eights[1] : eights[0];
          } else {
#pragma unroll
            for (int x = 0; x < C::kCols; ++x) {
              const bool odd = l4 & 1, high = l4 & 2;
              const float* e = eights + 4 * x;
              const float a = (odd ? e[1] : e[0]) + __shfl_xor_sync(0xffffffffu, odd ? e[0] : e[1], 1);
              const float c2 = (odd ? e[3] : e[2]) + __shfl_xor_sync(0xffffffffu, odd ? e[2] : e[3], 1);
              w[x] += (high ? c2 : a) + __shfl_xor_sync(0xffffffffu, high ? a : c2, 2);
            }
          }
#pragma unroll
          for (int x = 0; x < C::kCols; ++x) {
            const int to = 8 * (l4 + 4 * x) + r8, j = key0 + to;
            if (to < TK && j < len) weights[j] = w[x];
          }
        }
        if (waiting) {  // what was requested lands
          gave_up = true;
          for (; used < asked; ++used) {
            volatile int no_abort = 0;
            mbar_wait(bars + 8 * (used % C::kStages), (used / C::kStages) & 1u,
                      Watchdog{&no_abort, wd.status, wd.detail, 100000000ll}, kSiteWeighTile);
          }
          waiting = 0;
        }
      }
    }
    // To the next pair with tiles.
    base += places;
    if (++h == c.Hkv) {
      h = 0;
      do {
        if (++b >= p.B) return;
        places = places_of(b);
      } while (places == 0);
      len = weigh_len(p, b);
    }
  }
}

template <int D, int ROWS>
cudaError_t launch(const CacheWeighParams& p, int sms, cudaStream_t s) {
  constexpr int kSmem = WeighCfg<D, ROWS>::kSmem;
  auto go = [&](auto kernel) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    return e != cudaSuccess ? e : launch_after(kernel, dim3(2 * sms), dim3(kWeighThreads), kSmem, s, p);
  };
  return p.c.kind == BSA_CACHE_INT8 ? go(weigh_kernel<D, BSA_CACHE_INT8, ROWS>) : go(weigh_kernel<D, BSA_CACHE_E4M3, ROWS>);
}

}  // namespace

cudaError_t launch_cache_weigh(const CacheWeighParams& p, int sms, cudaStream_t s) {
  if (p.M <= 8) return p.c.d == 64 ? launch<64, 8>(p, sms, s) : launch<128, 8>(p, sms, s);
  if (p.c.d == 64) return p.M <= 32 ? launch<64, 32>(p, sms, s) : launch<64, 128>(p, sms, s);
  return p.M <= 32 ? launch<128, 32>(p, sms, s) : launch<128, 128>(p, sms, s);
}

}  // namespace bsa
