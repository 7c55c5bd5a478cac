// Attention of a few queries per sequence over the 8-bit paged cache.
//
// Mathematics.  For the M = g * nq query rows that share a K/V head (g heads
// of the group, nq queries each):
//   x[key][row] = S_k(key) * qs(row) * sum_d kcode[key][d] * q16[row][d]
// with q16 the row divided by a power of two that brings its largest element
// into [1, 2) (exact in fp16 to 2^-25 of that element) and qs that power times
// scale * log2(e); p = 2^(x - m + 7) rounded to fp16, and
//   O[d][row] += S_v * sum over 16 keys of vcode[key][d] * p[key][row]
// where the 16 keys of one matrix instruction lie in one scale block.  Both
// products are mma.m16n8k16 with the codes as the 16-row operand (S^T = K Q^T
// and O^T = V^T P^T): with 1 to 8 rows nothing of the instruction is wasted on
// the codes' side, codes convert to fp16 exactly, and S^T's accumulators become
// P^T's operand by one movmatrix per 8 keys.  m is a running reference that is
// moved only when a score passes it by more than 8 (then O and the sums are
// rescaled), so fp16 weights keep 11 bits.  The 7 puts the largest of them, 2^15,
// under fp16's 2^16, and what becomes 0 in the products (below 2^-25) at 2^-32 of
// the reference: a tail of n keys just below that loses n 2^-32 of O.  m is a
// whole number, so that 7 - m and the differences of references are exact.
//
// What bounds it: 2 d bytes per key and K/V head at the memory's rate (32
// sequences of up to 32768 tokens, 8 heads of 128, 4 rows: 1.11 GB in 170 to
// 173 us, 6.5 TB/s) up to about 16 rows, the warps' issue and latency above (16
// sequences of up to 16000, 8 heads of 64, 20 rows: 63 us, 2.4 TB/s); an SM's
// share is 23 bytes per cycle, against which a tile of 8 KB costs 250 to 800 warp
// instructions (8 to 24 rows) of the 1400 that the SM can issue meanwhile.
// mma.sync and not tcgen05: at the memory's rate the products are 2 flops per row
// and byte, 6 % of the tensor pipe's measured rate at 8 rows and 17 % at 24, and
// the codes have to pass through registers to be converted anyway.  That holds
// for the rows of one row tile.  With more, every row tile reads and converts a
// tile again, and at 96 rows the products alone are two thirds of the pipe's
// rate: there converting once and tcgen05 would be the faster way, which this
// kernel does not take (24 queries of 16 sequences, 4 heads a group: 329 us).
//
// Work split: the tiles (8 KB: 32 keys at d = 128, 64 at d = 64) of all (sequence, K/V head) pairs form one line
// which the CTAs cut into equal pieces, so that ragged lengths and few long
// sequences both fill the machine.  A row whose tiles lie in several CTAs
// leaves partial sums in the workspace; the combine kernel joins them in the
// order of the CTAs (results do not depend on timing).  It is launched ahead of
// this kernel's end and waits for it.  (Joining by the CTA that is last, behind
// a flag per part, saves the launch but puts fences and reads of L2 that is
// busy with the others' tiles at the end of every CTA: 193 us against 183 us
// for 32 sequences of up to 32768 tokens.)  Inside a CTA the tiles
// go round the warps, each with its own sums, joined when the piece of a row
// ends.  Each warp feeds itself: a ring of tiles of its own, filled by TMA (a
// page's rows of a head are one box; the copy engine takes a line of the box at
// a time whatever its length, so at d = 64 a line is two tokens; 128-byte
// swizzled so that the products read with few conflicts), the next tile requested as soon as one is used up.
// (A warp that feeds all others issues a tile every 700 cycles, too slow for
// tiles of 8 KB, and tiles of 16 KB leave room for six warps' rings at most.)
#include <type_traits>

#include "bsa_cache.h"
#include "bsa_cache_codes.cuh"
#include "bsa_device.cuh"

namespace bsa {
namespace {

using namespace dev;

constexpr int kWarps = 4;
constexpr int kAttnThreads = 32 * kWarps;
constexpr int kMaxNT = 3;  // 8-row column tiles per warp at most
static_assert(kCacheUnitRows == 8 * kMaxNT * kWarps, "24 query rows for each warp of a full unit");
constexpr float kMoveReference = 8.f;  // log2: weights stay <= 2^(8 + kShift)
constexpr float kShift = 7.f;          // log2 of the weight of a score at the reference
constexpr float kUnshift = 0x1p-7f;    // taken out of the sums: values may be as large as ever

enum CacheSite : int { kSiteTileFull = 0x50 };

template <int D>
struct AttnCfg {
  static constexpr int TK = cache_tile_keys(D);      // keys of a tile
  static constexpr int kGroups = TK / 16;            // keys of one matrix instruction, one scale each for K and V
  static constexpr int kTileBytes = TK * D;          // K or V of a tile
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = 3;                  // per warp
  static constexpr int kMergeBytes = kWarps * 8 * D * 4;  // 8 rows a warp at a time (the tile counts' prefix uses it first)
  static constexpr int kOffMerge = kWarps * kStages * kStageBytes;
  static constexpr int kOffMl = kOffMerge + kMergeBytes;      // float [warps][8][2]
  static constexpr int kOffBar = kOffMl + kWarps * 8 * 8;     // full [warps][stages]
  static constexpr int kOffAbort = kOffBar + kWarps * kStages * 8;
  static constexpr int kSmem = kOffAbort + 16;
  static_assert(kSmem <= 113 * 1024, "two CTAs per SM");
  static_assert(kMergeBytes >= 4 * (kAttnThreads + kWarps), "prefix");
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with an accumulator that starts at zero.
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint64_t policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(addr) : "memory");
  return r;
}

// Lists and masks of the caller: coherent loads like load_written's, which the
// compiler leaves where they are (moved about, they cost the kernel 2 %).
template <class T>
__device__ __forceinline__ T load_given(const T* p) {
  return __ldca(p);
}

// Length of batch row b's sequence (0 for a padded row, and where the sequence or
// its length is out of range: recorded with the empty rows).
__device__ __forceinline__ int seq_of(const CacheAttnParams& p, int b) {
  const int s = p.seqs ? load_given(p.seqs + b) : b;
  return s >= 0 && s < p.c.max_seqs ? s : -1;
}
__device__ __forceinline__ int len_of(const CacheAttnParams& p, int b) {
  const int s = seq_of(p, b);
  if (s < 0) return 0;
  const int n = load_written(p.c.lens + s);
  return n >= 0 && n <= p.c.max_pages * p.c.page ? n : 0;
}

// The line of tiles: entry e is a batch row with its Hkv heads (no mask) or one
// (batch row, head) with its list (mask); each entry's tiles are repeated for
// its heads and for the groups of kCacheUnitRows query rows.
__device__ __forceinline__ int entry_tiles(const CacheAttnParams& p, int e) {
  if (p.mask) return load_written(p.counts + e);
  return (len_of(p, e) + p.tile - 1) / p.tile;
}

// Walks the pieces of units in places [lo, hi) of the line (fewer than 2^31
// places: checked on the host).  A unit has `head` places that hold no tile ahead
// of those of its tiles: what beginning it costs a CTA, so that CTAs with few
// beginnings get more tiles.
struct Walk {
  int e, sub, cnt;   // entry, unit within it, its tiles
  int t0, t1;        // this piece: tiles [t0, t1) of the unit
  int row0;          // place of the unit's first tile
  int lo, hi;
};
__device__ __forceinline__ void walk_piece(Walk& w) {
  w.t0 = max(w.lo - w.row0, 0);
  w.t1 = min(w.cnt, w.hi - w.row0);
}
// To the next unit with tiles in the piece; false when the piece ends.
__device__ __forceinline__ bool walk_next(const CacheAttnParams& p, Walk& w, int mult, int head) {
  w.row0 += w.cnt;
  if (w.row0 + head >= w.hi) return false;
  if (++w.sub == mult) {
    w.sub = 0;
    do w.cnt = entry_tiles(p, ++w.e);
    while (w.cnt == 0);
  }
  w.row0 += head;
  walk_piece(w);
  return true;
}
// To the first unit of the piece.  `base`: place where entry e begins; it, or one
// behind it, holds place lo.
__device__ __forceinline__ bool walk_start(const CacheAttnParams& p, Walk& w, int mult, int head, int e, int base, int lo,
                                           int hi) {
  w.lo = lo;
  w.hi = hi;
  w.cnt = entry_tiles(p, e);
  while (w.cnt == 0 || lo >= base + (w.cnt + head) * mult) {
    if (w.cnt > 0) base += (w.cnt + head) * mult;
    w.cnt = entry_tiles(p, ++e);
  }
  w.e = e;
  w.sub = (lo - base) / (w.cnt + head);
  w.row0 = base + w.sub * (w.cnt + head) + head;
  walk_piece(w);
  return w.t1 > w.t0 || walk_next(p, w, mult, head);  // (the piece may end in the head)
}

// Batch row, K/V head and group of query rows of a unit.
struct Unit {
  int b, h, grp;
};
__device__ __forceinline__ Unit unit_of(const CacheAttnParams& p, int e, int sub) {
  Unit u;
  u.grp = sub % p.groups;
  const int x = sub / p.groups;
  if (p.mask) {
    u.b = e / p.c.Hkv;
    u.h = e % p.c.Hkv;
  } else {
    u.b = e;
    u.h = x;
  }
  return u;
}

__device__ __forceinline__ void store2(const CacheAttnParams& p, uint16_t* at, float4 f) {
  uint2 w;
  if (p.fp16) w = make_uint2(pack_half2(f.x, f.y), pack_half2(f.z, f.w));
  else w = make_uint2(pack_bf16x2(f.x, f.y), pack_bf16x2(f.z, f.w));
  *reinterpret_cast<uint2*>(at) = w;
}
// Query row m of a unit (within its K/V head's M rows): head and query.
__device__ __forceinline__ uint16_t* o_row(const CacheAttnParams& p, int b, int h, int m) {
  const int hq = h * p.g + m / p.nq, i = m % p.nq;
  return p.o + b * p.o_sb + hq * p.o_sh + i * p.o_st;
}
__device__ __forceinline__ float* lse_row(const CacheAttnParams& p, int b, int h, int m) {
  const int hq = h * p.g + m / p.nq, i = m % p.nq;
  return p.lse + ((size_t)b * p.Hq + hq) * p.nq + i;
}

// NaN codes among 16 keys' values (v, as loaded for O^T += V^T P^T) where some
// row does not attend some key: a weight of 0 would not keep them out of that
// row.  They are taken out of v, and the rows that do attend them (counted by a
// product of indicators) become NaN.  Nothing to do for a tile without any.
template <int NT, int DV, int MT>
__device__ __forceinline__ void take_nans(uint32_t (&v)[4][DV / 4], float (&o)[NT][MT][4], uint32_t kept, int kg) {
  uint32_t any = 0u;
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll
    for (int q = 0; q < DV / 4; ++q) any |= (v[e][q] & 0x7f7f7f7fu) + 0x01010101u;  // 0x80 in a byte: NaN
  if (!__any_sync(0xffffffffu, (any & 0x80808080u) != 0u)) return;
  uint32_t kf[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const uint32_t b = kept >> ((kg * NT + nt) * 4);
    kf[nt][0] = movmatrix((b & 1u ? 0x3c00u : 0u) | (b & 2u ? 0x3c000000u : 0u));
    kf[nt][1] = movmatrix((b & 4u ? 0x3c00u : 0u) | (b & 8u ? 0x3c000000u : 0u));
  }
#pragma unroll
  for (int q = 0; q < DV / 4; ++q) {
    uint32_t ind[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t n = (((v[e][q] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;  // 1 in a byte: NaN
      v[e][q] &= ~(n * 0xffu);
      ind[e] = n * 0x38u;  // 1.0
    }
    const uint2 ab0 = codes_to_half4<BSA_CACHE_E4M3>(__byte_perm(ind[0], ind[1], 0x5140));
    const uint2 cd0 = codes_to_half4<BSA_CACHE_E4M3>(__byte_perm(ind[2], ind[3], 0x5140));
    const uint2 ab1 = codes_to_half4<BSA_CACHE_E4M3>(__byte_perm(ind[0], ind[1], 0x7362));
    const uint2 cd1 = codes_to_half4<BSA_CACHE_E4M3>(__byte_perm(ind[2], ind[3], 0x7362));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float y[4], z[4];
      mma16816_first(y, ab0.x, ab0.y, cd0.x, cd0.y, kf[nt][0], kf[nt][1]);
      mma16816_first(z, ab1.x, ab1.y, cd1.x, cd1.y, kf[nt][0], kf[nt][1]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (y[e] > 0.f) o[nt][2 * q][e] = __uint_as_float(0x7fffffffu);
        if (z[e] > 0.f) o[nt][2 * q + 1][e] = __uint_as_float(0x7fffffffu);
      }
    }
  }
}

// A warp's requests for tiles: where it is in the line, and for the next (up to)
// 32 tiles of the piece a lane each with the tile's number (bits from kNoBox on:
// its boxes that are not read) and the pool row of each of its boxes (-1: no
// token in it, or the table has no page for them).
constexpr int kNoBox = 25;  // (tiles are below 2^25: sequences end at 2^30 tokens)
constexpr int kTileMask = (1 << kNoBox) - 1;
struct Feed {
  Walk w;
  int pos, n, i;    // first tile of the batch (within the unit), its size, the next one to request
  int tile, pr[4];  // this lane's tile
  int len;          // of the piece's sequence
  const uint8_t* mask;  // of query row `lane` of the warp (with a mask)
  bool more;
};

template <int D, int KIND, int NT>
__global__ void __launch_bounds__(kAttnThreads, 2) attn_kernel(const __grid_constant__ CacheAttnParams p) {
  using C = AttnCfg<D>;
  constexpr int TK = C::TK;
  // Groups of 16 keys whose scores are held at once, as registers allow (16 rows
  // of 16 sequences, one and two groups, E4M3 / INT8: d = 128 70.8 / 73.1 and 69.7
  // / 71.7 us, d = 64 48.1 / 50.9 and 45.0 / 47.5 us).
  constexpr int KG = NT * D <= 64 ? 4 : (NT < 3 ? 2 : 1);
  extern __shared__ __align__(1024) uint8_t smem[];
  int* s_prefix = reinterpret_cast<int*>(smem + C::kOffMerge);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::kOffAbort);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = blockIdx.x;
  const uint32_t base = smem_u32(smem);
  const uint32_t bars = base + C::kOffBar + warp * C::kStages * 8;  // this warp's
  const uint32_t ring = base + warp * C::kStages * C::kStageBytes;
  const Watchdog wd{s_abort, p.c.control + kCacheStatus, p.c.control + kCacheDetail, p.watchdog_ns};
  // Row tiles of 8 NT query rows: a warp each.  Warps of the same row tile take
  // tiles in turn (KL of them); those of other row tiles read the same tiles
  // again, from L2.
  const int rows_unit = min(p.M, kCacheUnitRows);
  const int R = rows_unit <= 8 * NT ? 1 : (rows_unit <= 16 * NT ? 2 : 4);
  const int KL = kWarps / R, rt = warp % R, kl = warp / R;
  if (tid == 0) {
    *s_abort = 0;
    if (base & 1023u) record_failure(wd, BSA_ERR_CUDA, 0);  // the swizzle's layout needs it
    for (int s = 0; s < kWarps * C::kStages; ++s) mbar_init(base + C::kOffBar + 8 * s, 1);
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&p.tmK);
    tma_prefetch_desc(&p.tmV);
  }
  next_may_launch();  // the combine kernel may queue up
  wait_for_previous();
  // This CTA's piece of the line: sums of the entries' tiles by thread, then a
  // prefix over the threads.
  const int E = p.mask ? p.B * p.c.Hkv : p.B;
  const int mult = p.mask ? p.groups : p.c.Hkv * p.groups;
  const int per = (E + kAttnThreads - 1) / kAttnThreads;
  int sum = 0;
  int units = 0;
  for (int e = tid * per; e < min(E, (tid + 1) * per); ++e) {
    const int cnt = entry_tiles(p, e);
    sum += cnt;
    units += cnt > 0 ? 1 : 0;
  }
  sum *= mult;
  units *= mult;
  const int head = p.head;
  sum += head * units;
  int x = sum;  // inclusive prefix over the warp, then over the warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_prefix[kAttnThreads + warp] = x;
  __syncthreads();
  int T = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i == warp) x += T;
    T += s_prefix[kAttnThreads + i];
  }
  s_prefix[tid] = x - sum;  // tiles before this thread's entries
  __syncthreads();
  // A few places at least for each CTA, so that short lines leave few parts to
  // join; the first `more_of` CTAs have one more.  The CTAs that hold tiles of a
  // unit are consecutive ones.
  const int G = min((T + KL - 1) / KL, (int)gridDim.x);
  const int share = G > 0 ? T / G : 0, more_of = T - share * G;
  const int lo = cta < G ? cta * share + min(cta, more_of) : 0;
  const int hi = cta < G ? lo + share + (cta < more_of ? 1 : 0) : 0;
  // Empty entries' rows: O = 0, LSE = -inf.
  for (int e = cta; e < E; e += (int)gridDim.x) {
    if (entry_tiles(p, e) != 0) continue;
    const int b = p.mask ? e / p.c.Hkv : e;
    const int h0 = p.mask ? e % p.c.Hkv : 0, h1 = p.mask ? h0 + 1 : p.c.Hkv;
    if (tid == 0) {
      const int s = p.seqs ? load_given(p.seqs + b) : b;
      const int n = s >= 0 && s < p.c.max_seqs ? load_written(p.c.lens + s) : (s == -1 ? 0 : -1);
      if (n < 0 || n > p.c.max_pages * p.c.page) cache_error(p.c.control, BSA_ERR_INVALID_ARG, b);
    }
    const int c4 = tid % (D / 4);
    for (int r = tid / (D / 4); r < (h1 - h0) * p.M; r += kAttnThreads / (D / 4)) {
      const int m = r % p.M, h = h0 + r / p.M;
      store2(p, o_row(p, b, h, m) + 4 * c4, make_float4(0.f, 0.f, 0.f, 0.f));
      if (c4 == 0 && p.lse) *lse_row(p, b, h, m) = -INFINITY;
    }
  }
  if (tid == 0) p.desc[4 * cta] = 0;  // no row of this CTA goes on in the next one (so far)
  if (lo >= hi || *s_abort) return;   // (the same for every thread: barriers above)
  // The thread whose entries hold tile lo (the last that does not start past it).
  int a = 0, z = kAttnThreads;
  while (z - a > 1) {
    const int m = (a + z) >> 1;
    if (s_prefix[m] <= lo) a = m;
    else z = m;
  }
  Walk w;
  bool more = walk_start(p, w, mult, head, a * per, s_prefix[a], lo, hi);
  __syncthreads();  // the prefix gives way to the merge buffer
  if (!more) return;

  // ------------------------------------------------------------- computation
  const int g = lane >> 2, t4 = lane & 3;
  constexpr int KS = D / 16;    // 16-element steps of q . k
  constexpr int MT = D / 16;    // 16-row tiles of O^T
  constexpr int DV = D / 8;     // consecutive elements of O a thread holds
  // This warp's query rows as they are: read ahead of the first tiles, which the
  // memory is then busy with.
  uint32_t q_raw[NT][KS][2];
  auto load_q = [&](const Unit& u) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int m = u.grp * kCacheUnitRows + rt * 8 * NT + 8 * nt + g;
#pragma unroll
      for (int k = 0; k < KS; ++k) q_raw[nt][k][0] = q_raw[nt][k][1] = 0u;
      if (m < p.M) {
        const uint16_t* qr = p.q.p + u.b * p.q.sb + (u.h * p.g + m / p.nq) * p.q.sh + (m % p.nq) * p.q.st;
        // Word s of 16-byte chunk (D == 128: 2 t4 + i; D == 64: t4) of a row of
        // codes are elements 16 chunk + 4 s ..: the same of q.
#pragma unroll
        for (int k2 = 0; k2 < KS / 2; ++k2) {
          const uint4 x = load_written(reinterpret_cast<const uint4*>(qr + t4 * (D / 4) + k2 * 8));
          q_raw[nt][2 * k2][0] = x.x;
          q_raw[nt][2 * k2][1] = x.y;
          q_raw[nt][2 * k2 + 1][0] = x.z;
          q_raw[nt][2 * k2 + 1][1] = x.w;
        }
      }
    }
  };
  load_q(unit_of(p, w.e, w.sub));

  // ---------------------------------------------------------------- requests
  const int lpage = 31 - __clz(p.c.page), lsb = 31 - __clz(p.c.sb);
  const int lbk = p.mask ? 31 - __clz(p.bk) : 0;
  const int cs = min(p.c.page, TK);  // keys per box
  const int lcs = 31 - __clz(cs), nc = TK >> lcs;
  // Read once, unless other row tiles or groups of rows come back for it.
  const uint64_t pol = R == 1 && p.groups == 1 ? policy_evict_first() : policy_evict_normal();
  // First tile of a piece that is this warp's: the tile at place t of the line is
  // taken by the warps with kl = t mod KL.
  auto first_of = [&](const Walk& x) { return x.t0 + ((kl - (x.row0 + x.t0)) & (KL - 1)); };  // (KL is 1, 2 or 4)
  Feed f;
  f.w = w;
  f.pos = first_of(w);
  f.n = f.i = 0;
  f.more = true;
  f.len = 0;
  f.tile = 0;
  // The batch at f.pos (of the next piece that has a tile for this warp).
  auto refill = [&]() {
    f.pos += f.n * KL;
    while (f.pos >= f.w.t1) {
      if (!walk_next(p, f.w, mult, head)) {
        f.more = false;
        return;
      }
      f.pos = first_of(f.w);
    }
    const Unit u = unit_of(p, f.w.e, f.w.sub);
    const int seq = seq_of(p, u.b);
    f.len = len_of(p, u.b);
    f.n = min(32, (f.w.t1 - f.pos + KL - 1) / KL);
    f.i = 0;
    const int32_t* row = p.c.table + (size_t)seq * p.c.max_pages;
    if (p.mask) {
      const int m = min(u.grp * kCacheUnitRows + rt * 8 * NT + lane, p.M - 1);
      f.mask = p.mask + ((size_t)u.b * p.Hq + u.h * p.g + m / p.nq) * p.NKB;
    }
    f.tile = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) f.pr[j] = -1;
    if (lane < f.n) {
      const int t = f.pos + lane * KL;
      const int tile = p.mask ? load_written(p.list + (size_t)f.w.e * p.max_tiles + t) : t;
      f.tile = tile;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = tile * TK + (j << lcs);
        if (j < nc && key < f.len) {
          const int ph = load_written(row + (key >> lpage));
          if (ph >= 0 && ph < p.c.num_pages) f.pr[j] = (ph * p.c.Hkv + u.h) * p.c.page + (key & (p.c.page - 1));
          else cache_error(p.c.control, BSA_ERR_PLAN_MISMATCH, seq);  // not attended
        }
        if (j < nc && f.pr[j] < 0) f.tile |= 1 << (kNoBox + j);
      }
    }
  };
  // Request the warp's next tile into stage s.  Returns its number with the bits
  // of boxes that are not read (-1: there is none); `scale` gets this lane's
  // scale of it: lanes 0 .. kGroups - 1 K's of 16 keys each, the next kGroups V's
  // (0 where no key is read); `sel` the mask's bytes of query row `lane` for the
  // tile's halves of 32 keys.
  auto request = [&](int s, float& scale, uchar2& sel) -> int {
    scale = 0.f;
    sel = make_uchar2(0, 0);
    if (f.more && f.i == f.n) refill();
    if (!f.more) return -1;
    int box[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) box[j] = __shfl_sync(0xffffffffu, f.pr[j], f.i);
    const int tagged = __shfl_sync(0xffffffffu, f.tile, f.i), tile = tagged & kTileMask;
    ++f.i;
    if (lane == 0) {
      uint32_t bytes = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) bytes += box[j] >= 0 ? 2u * cs * D : 0u;
      mbar_arrive_expect_tx(bars + 8 * s, bytes);
    }
    __syncwarp();
    const int j = lane & 3;
    const int mybox = j == 0 ? box[0] : (j == 1 ? box[1] : (j == 2 ? box[2] : box[3]));
    if (lane < 8 && mybox >= 0)
      tma_load_2d(ring + s * C::kStageBytes + (lane >> 2) * C::kTileBytes + j * cs * D, lane < 4 ? &p.tmK : &p.tmV, 0,
                  mybox / (128 / D), bars + 8 * s, pol);
    if (lane < 2 * C::kGroups) {
      const int gr = lane % C::kGroups, jb = (16 * gr) >> lcs;
      const int sbox = jb == 0 ? box[0] : (jb == 1 ? box[1] : (jb == 2 ? box[2] : box[3]));
      if (tile * TK + 16 * gr < f.len && sbox >= 0)
        scale = load_written((lane < C::kGroups ? p.c.ks : p.c.vs) + ((size_t)(unsigned)(sbox + ((16 * gr) & (cs - 1))) >> lsb));
    }
    if (p.mask && lane < 8 * NT) {
      const int k0 = tile * TK >> lbk;
      if (k0 < p.NKB) sel.x = load_given(f.mask + k0);
      if (TK > 32) {
        const int k1 = (tile * TK + 32) >> lbk;
        if (k1 < p.NKB) sel.y = load_given(f.mask + k1);
      }
    }
    return tagged;
  };
  // Tiles and scales of the stages, the one to be used next first.
  int tq[C::kStages];
  float sq[C::kStages];
  uchar2 mq[C::kStages];
#pragma unroll
  for (int s = 0; s < C::kStages; ++s) tq[s] = request(s, sq[s], mq[s]);
  int stage = 0;
  uint32_t phase = 0;

  float* merge = reinterpret_cast<float*>(smem + C::kOffMerge);
  float* ml = reinterpret_cast<float*>(smem + C::kOffMl);
  bool ok = true;
  while (more) {
    const Unit u = unit_of(p, w.e, w.sub);
    const int len = len_of(p, u.b);
    const int m0 = u.grp * kCacheUnitRows + rt * 8 * NT;  // first query row of this warp
    // Query fragments: lane (g, t4) holds row 8 nt + g, elements 4 a word of codes.
    uint32_t qf[NT][KS][2];
    float qs[NT][2];  // scale of rows 8 nt + 2 t4, + 1
    int lim;          // keys below it are visible to row `lane` of the warp
    {
      const int m = m0 + lane;
      lim = m < p.M ? (p.causal ? min(len, len - p.nq + m % p.nq + 1) : len) : 0;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      auto& raw = q_raw[nt];
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 f = elems_to_float2(raw[k][e], p.fp16);
          amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // 2^e with amax in [2^e, 2^(e+1)); rows of zeros and of infinities keep 1.
      int e = (int)(__float_as_uint(amax) >> 23) - 127;
      if (!(amax > 0.f) || amax == INFINITY) e = 0;
      e = max(e, -126);  // (the least power that is normal)
      const float down = __uint_as_float((uint32_t)(127 - min(e, 126)) << 23);
      const float up = __uint_as_float((uint32_t)(127 + min(e, 126)) << 23);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float2 f = elems_to_float2(raw[k][x], p.fp16);
          qf[nt][k][x] = pack_half2(f.x * down, f.y * down);
        }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        qs[nt][x] = __shfl_sync(0xffffffffu, up, (2 * t4 + x) * 4) * p.scale_log2;
      }
    }
    float o[NT][MT][4];
    float m_ref[NT][2], l_sum[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        m_ref[nt][x] = -INFINITY;
        l_sum[nt][x] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < MT; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[nt][k][x] = 0.f;
    }
    const int first_limit = p.causal ? len - p.nq + 1 : len;  // keys below it are visible to every row

    int t = first_of(w);
    for (; t < w.t1 && ok; t += KL) {
      const int key0 = (tq[0] & kTileMask) * TK;
      if (!__all_sync(0xffffffffu, mbar_wait(bars + 8 * stage, phase, wd, kSiteTileFull))) {
        ok = false;  // recorded; these rows' results are void, the walk goes on so that no barrier is missed
        break;
      }
      const uint32_t ks = ring + stage * C::kStageBytes, vs = ks + C::kTileBytes;
      const bool tail = key0 + TK > len;
      const uint32_t unread = (uint32_t)tq[0] >> kNoBox;  // boxes of the tile
      auto box_read = [&](int r) { return (unread >> (r >> lcs) & 1u) == 0u; };  // that of the tile's key r
      // The tile's computation, for tiles that every row attends wholly and for
      // the others: the code of the masks, in the loop that most tiles take,
      // would cost those a tenth (registers, and the loop outgrows the
      // instruction cache).
      auto compute = [&](auto masked_c) {
      constexpr bool kMasked = decltype(masked_c)::value;
#pragma unroll 1
      for (int kb16 = 0; kb16 < TK; kb16 += 16 * KG) {
        // ---- S^T = K Q^T: 16 keys a time
        float x[KG][NT][4];
#pragma unroll
        for (int kg = 0; kg < KG; ++kg) {
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            const int r0 = kb16 + 16 * kg + g, r1 = r0 + 8;
            uint4 a, b;
            if constexpr (D == 128) {
              a = ld_shared_v4(ks + r0 * 128 + (((2 * t4 + i) ^ (r0 & 7)) << 4));
              b = ld_shared_v4(ks + r1 * 128 + (((2 * t4 + i) ^ (r1 & 7)) << 4));
            } else {
              a = ld_shared_v4(ks + (r0 >> 1) * 128 + (((r0 & 1) * 4 + t4) ^ ((r0 >> 1) & 7)) * 16);
              b = ld_shared_v4(ks + (r1 >> 1) * 128 + (((r1 & 1) * 4 + t4) ^ ((r1 >> 1) & 7)) * 16);
            }
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint2 ha = codes_to_half4<KIND>(aw[q]), hb = codes_to_half4<KIND>(bw[q]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if (i == 0 && q == 0)
                  mma16816_first(x[kg][nt], ha.x, hb.x, ha.y, hb.y, qf[nt][0][0], qf[nt][0][1]);
                else
                  mma16816(x[kg][nt], ha.x, hb.x, ha.y, hb.y, qf[nt][4 * i + q][0], qf[nt][4 * i + q][1]);
              }
            }
          }
        }
        // ---- scores (log2), masks, reference
#pragma unroll
        for (int kg = 0; kg < KG; ++kg) {
          const float sk = __shfl_sync(0xffffffffu, sq[0], kb16 / 16 + kg);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint64_t f = fmul2(f2_make(sk, sk), f2_make(qs[nt][0], qs[nt][1]));
            f2_split(fmul2(f2_make(x[kg][nt][0], x[kg][nt][1]), f), x[kg][nt][0], x[kg][nt][1]);
            f2_split(fmul2(f2_make(x[kg][nt][2], x[kg][nt][3]), f), x[kg][nt][2], x[kg][nt][3]);
          }
        }
        uint32_t kept = 0xffffffffu;  // bit (kg NT + nt) 4 + e: this thread's score is one that is attended
        if constexpr (kMasked) {
          // Rows whose heads select the tile's halves of 32 keys.
          uint32_t sel[2] = {0xffffffffu, 0xffffffffu};
          if (p.mask) {
            sel[0] = __ballot_sync(0xffffffffu, mq[0].x != 0);
            sel[1] = __ballot_sync(0xffffffffu, mq[0].y != 0);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int row = 8 * nt + 2 * t4 + c;
              const int end = __shfl_sync(0xffffffffu, lim, row) - key0 - kb16;
#pragma unroll
              for (int kg = 0; kg < KG; ++kg)
#pragma unroll
                for (int hi8 = 0; hi8 < 2; ++hi8) {
                  const bool keep = 16 * kg + g + 8 * hi8 < end && (sel[(kb16 + 16 * kg) >> 5] >> row & 1u) &&
                                      box_read(kb16 + 16 * kg);
                  if (!keep) {
                    x[kg][nt][2 * hi8 + c] = -INFINITY;
                    kept &= ~(1u << ((kg * NT + nt) * 4 + 2 * hi8 + c));
                  }
                }
            }
        }
        bool move = false;
        float mx[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v = fmaxf(x[0][nt][c], x[0][nt][c + 2]);
#pragma unroll
            for (int kg = 1; kg < KG; ++kg) v = fmax3(v, x[kg][nt][c], x[kg][nt][c + 2]);
            mx[nt][c] = v;
            move |= v > m_ref[nt][c] + kMoveReference;
          }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float f[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float v = mx[nt][c];
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
              f[c] = 1.f;
              v = floorf(v);
              if (v > m_ref[nt][c]) {
                f[c] = ex2_approx(m_ref[nt][c] - v);  // 0 from -inf
                m_ref[nt][c] = v;
              }
              l_sum[nt][c] *= f[c];
            }
#pragma unroll
            for (int k = 0; k < MT; ++k)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[nt][k][e] *= f[e & 1];
          }
        }
        // ---- weights and P^T fragments
        uint32_t pf[KG][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint64_t ref = f2_make(m_ref[nt][0] == -INFINITY ? 0.f : kShift - m_ref[nt][0],
                                       m_ref[nt][1] == -INFINITY ? 0.f : kShift - m_ref[nt][1]);
          uint64_t l2 = f2_make(l_sum[nt][0], l_sum[nt][1]);
#pragma unroll
          for (int kg = 0; kg < KG; ++kg) {
            float y0, y1, y2, y3;
            f2_split(fadd2(f2_make(x[kg][nt][0], x[kg][nt][1]), ref), y0, y1);
            f2_split(fadd2(f2_make(x[kg][nt][2], x[kg][nt][3]), ref), y2, y3);
            const float p0 = ex2_approx(y0), p1 = ex2_approx(y1), p2 = ex2_approx(y2), p3 = ex2_approx(y3);
            l2 = fadd2(l2, fadd2(f2_make(p0, p1), f2_make(p2, p3)));
            pf[kg][nt][0] = movmatrix(pack_half2(p0, p1));
            pf[kg][nt][1] = movmatrix(pack_half2(p2, p3));
          }
          f2_split(l2, l_sum[nt][0], l_sum[nt][1]);
        }
        // ---- O^T += S_v V^T P^T: the 16 keys of a group lie in one scale block
        // (One addition for groups that have the same scale would save a tenth of
        // the instructions, but the second path's code costs more than that.)
        float sv[KG];
        uint32_t v[KG][4][DV / 4];
#pragma unroll
        for (int kg = 0; kg < KG; ++kg) {
          sv[kg] = __shfl_sync(0xffffffffu, sq[0], C::kGroups + kb16 / 16 + kg) * kUnshift;
          const int ra = kb16 + 16 * kg + 2 * t4;  // keys 2 t4, + 1, + 8, + 9 of the 16
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = ra + (e & 1) + (e >> 1) * 8;
            if constexpr (D == 128) {
              const uint4 y = ld_shared_v4(vs + r * 128 + ((g ^ (r & 7)) << 4));
              v[kg][e][0] = y.x;
              v[kg][e][1] = y.y;
              v[kg][e][2] = y.z;
              v[kg][e][3] = y.w;
            } else {
              const uint2 y = ld_shared_v2(vs + (r >> 1) * 128 + (((r & 1) * 4 + (g >> 1)) ^ ((r >> 1) & 7)) * 16 + (g & 1) * 8);
              v[kg][e][0] = y.x;
              v[kg][e][1] = y.y;
            }
            // Rows past the sequence, and of boxes that were not read, hold
            // anything: weight 0 would not stop a NaN.
            if (kMasked && ((tail && key0 + r >= len) || !box_read(kb16 + 16 * kg))) {
#pragma unroll
              for (int q = 0; q < DV / 4; ++q) v[kg][e][q] = 0u;
            }
          }
          if constexpr (KIND == BSA_CACHE_E4M3 && kMasked) take_nans<NT, DV, MT>(v[kg], o, kept, kg);
        }
        // Pairs of keys of one element: {a0 b0 a1 b1}, {a2 b2 a3 b3}.
#pragma unroll
        for (int q = 0; q < DV / 4; ++q) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
            for (int kg = 0; kg < KG; ++kg) {
              const uint32_t pick = hh ? 0x7362 : 0x5140;
              const uint2 ab = codes_to_half4<KIND>(__byte_perm(v[kg][0][q], v[kg][1][q], pick));
              const uint2 cd = codes_to_half4<KIND>(__byte_perm(v[kg][2][q], v[kg][3][q], pick));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float y[4];
                mma16816_first(y, ab.x, ab.y, cd.x, cd.y, pf[kg][nt][0], pf[kg][nt][1]);
                float (&acc)[4] = o[nt][2 * q + hh];
                if constexpr (NT * D < 384) {
                  const uint64_t f = f2_make(sv[kg], sv[kg]);
                  f2_split(ffma2(f, f2_make(y[0], y[1]), f2_make(acc[0], acc[1])), acc[0], acc[1]);
                  f2_split(ffma2(f, f2_make(y[2], y[3]), f2_make(acc[2], acc[3])), acc[2], acc[3]);
                } else {  // (pairs cost the fullest variant registers: 335 against 329 us for 96 rows)
#pragma unroll
                  for (int e = 0; e < 4; ++e) acc[e] = fmaf(sv[kg], y[e], acc[e]);
                }
              }
            }
          }
        }
      }
      };
      if (key0 + TK > first_limit || p.mask != nullptr || unread != 0u) {
        if (__any_sync(0xffffffffu, !(fabsf(sq[0]) < INFINITY))) {
          // A scale of values that is no number reaches the rows that attend a key
          // of its 16 (times a weight of 0 it would reach the others too).
          const uint32_t sel0 = p.mask ? __ballot_sync(0xffffffffu, mq[0].x != 0) : 0xffffffffu;
          const uint32_t sel1 = p.mask ? __ballot_sync(0xffffffffu, mq[0].y != 0) : 0xffffffffu;
#pragma unroll 1
          for (int gr = 0; gr < C::kGroups; ++gr) {
            const float sv = __shfl_sync(0xffffffffu, sq[0], C::kGroups + gr);
            if (fabsf(sv) < INFINITY || !box_read(16 * gr)) continue;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const int row = 8 * nt + 2 * t4 + c;
                const bool attends = key0 + 16 * gr < __shfl_sync(0xffffffffu, lim, row) &&
                                     ((16 * gr < 32 ? sel0 : sel1) >> row & 1u);
                if (attends) {
#pragma unroll
                  for (int k = 0; k < MT; ++k) o[nt][k][c] = o[nt][k][c + 2] = __uint_as_float(0x7fffffffu);
                }
              }
          }
          if (lane >= C::kGroups && !(fabsf(sq[0]) < INFINITY)) sq[0] = 0.f;
        }
        compute(std::true_type{});
      } else {
        compute(std::false_type{});
      }
      __syncwarp();  // every lane has read the stage
#pragma unroll
      for (int s = 0; s + 1 < C::kStages; ++s) {
        tq[s] = tq[s + 1];
        sq[s] = sq[s + 1];
        mq[s] = mq[s + 1];
      }
      tq[C::kStages - 1] = request(stage, sq[C::kStages - 1], mq[C::kStages - 1]);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }

    // ---- end of the piece: join the warps that took its tiles, 8 rows of each
    // warp at a time
    const bool starts = w.t0 == 0, whole = starts && w.t1 == w.cnt;
    Walk after = w;
    more = walk_next(p, after, mult, head);
    if (more) load_q(unit_of(p, after.e, after.sub));  // the next piece's queries, ahead of the barriers
    const int rows = min(p.M - u.grp * kCacheUnitRows, kCacheUnitRows);
    float* part = p.part + (size_t)(2 * cta + (starts ? 1 : 0)) * p.rows_cap * (D + 2);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (nt > 0) named_bar_sync(1, 32 * kWarps);  // the rows before have been read
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float l = l_sum[nt][c];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int row = warp * 8 + 2 * t4 + c;
        if (g == 0) {
          ml[row * 2] = m_ref[nt][c];
          ml[row * 2 + 1] = l * kUnshift;
        }
        float* mr = merge + (size_t)row * D + g * DV;
#pragma unroll
        for (int k = 0; k < MT; k += 2)
          *reinterpret_cast<float4*>(mr + 2 * k) =
              make_float4(o[nt][k][c], o[nt][k][c + 2], o[nt][k + 1][c], o[nt][k + 1][c + 2]);
      }
      named_bar_sync(1, 32 * kWarps);
      // A thread per (row, 4 elements).
      for (int i = tid; i < R * 8 * (D / 4); i += 32 * kWarps) {
        const int c4 = i % (D / 4), rr = i / (D / 4) % 8, rtile = i / (D / 4) / 8;
        const int r = rtile * 8 * NT + 8 * nt + rr;  // row of the unit
        if (r >= rows) continue;
        float M = -INFINITY;
        for (int k = 0; k < KL; ++k) M = fmaxf(M, ml[((k * R + rtile) * 8 + rr) * 2]);
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < KL; ++k) {
          const int at = (k * R + rtile) * 8 + rr;
          const float f = M == -INFINITY ? 1.f : ex2_approx(ml[at * 2] - M);
          const float4 y = *reinterpret_cast<const float4*>(merge + (size_t)at * D + 4 * c4);
          L = fmaf(f, ml[at * 2 + 1], L);
          acc.x = fmaf(f, y.x, acc.x);
          acc.y = fmaf(f, y.y, acc.y);
          acc.z = fmaf(f, y.z, acc.z);
          acc.w = fmaf(f, y.w, acc.w);
        }
        if (whole) {
          const int m = u.grp * kCacheUnitRows + r;
          const bool some = L > 0.f || L != L;
          const float inv = some ? 1.f / L : 0.f;
          store2(p, o_row(p, u.b, u.h, m) + 4 * c4, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
          if (c4 == 0 && p.lse)
            *lse_row(p, u.b, u.h, m) = some ? (M + __log2f(L)) * 0.69314718055994531f : -INFINITY;
        } else {
          float* pr = part + (size_t)r * (D + 2);
          *reinterpret_cast<float2*>(pr + 4 * c4) = make_float2(acc.x, acc.y);
          *reinterpret_cast<float2*>(pr + 4 * c4 + 2) = make_float2(acc.z, acc.w);
          if (c4 == 0) *reinterpret_cast<float2*>(pr + D) = make_float2(M, L);
        }
      }
    }
    if (tid == 0 && starts && !whole) {
      // CTAs up to the one that holds the unit's last tile.
      const int last = w.row0 + w.cnt - 1, longer = more_of * (share + 1);
      const int c1 = last < longer ? last / (share + 1) : more_of + (last - longer) / share;
      *reinterpret_cast<int4*>(p.desc + 4 * cta) = make_int4(c1 - cta + 1, u.b, u.h, u.grp);
    }
    named_bar_sync(1, 32 * kWarps);
    w = after;
  }
  if (!ok) {
    // Let the tiles in flight land before the CTA's shared memory goes away.
    volatile int no_abort = 0;
    const Watchdog quick{&no_abort, wd.status, wd.detail, 100000000ll};
#pragma unroll 1
    for (int k = 0; k < C::kStages; ++k) {
      if (tq[0] >= 0) mbar_wait(bars + 8 * stage, phase, quick, kSiteTileFull);
      tq[0] = k + 1 < C::kStages ? (k == 0 ? tq[1] : tq[2]) : -1;
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
}

// Joins the parts of a row that several CTAs worked on, in the CTAs' order.
// One CTA per (first CTA of the row, query row and every kCombineRows-th after
// it); its warps take every fourth part each.
constexpr int kCombineRows = 12;

template <int D>
__global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ CacheAttnParams p) {
  __shared__ float s_l[4];
  __shared__ float s_o[4][D];
  next_may_launch();
  wait_for_previous();
  const int c0 = blockIdx.x;
  const int4 ds = *reinterpret_cast<const int4*>(p.desc + 4 * c0);
  const int n = ds.x;
  if (n <= 0) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rows = min(p.M - ds.w * kCacheUnitRows, kCacheUnitRows);
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    auto slot = [&](int k) { return p.part + ((size_t)(2 * (c0 + k) + (k == 0 ? 1 : 0)) * p.rows_cap + r) * (D + 2); };
    float M = -INFINITY;
    for (int k = lane; k < n; k += 32) M = fmaxf(M, slot(k)[D]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f;
    constexpr int E = D / 32;
    float acc[E] = {};
#pragma unroll 4
    for (int k = warp; k < n; k += 4) {
      const float* s = slot(k);
      const float2 ml = *reinterpret_cast<const float2*>(s + D);
      const float f = M == -INFINITY ? 1.f : ex2_approx(ml.x - M);
      L = fmaf(f, ml.y, L);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        const float2 y = *reinterpret_cast<const float2*>(s + lane * E + 2 * e);
        acc[2 * e] = fmaf(f, y.x, acc[2 * e]);
        acc[2 * e + 1] = fmaf(f, y.y, acc[2 * e + 1]);
      }
    }
    __syncthreads();  // the row before has been read
    if (lane == 0) s_l[warp] = L;
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[e];
    __syncthreads();
    L = s_l[0] + s_l[1] + s_l[2] + s_l[3];
    const bool some = L > 0.f || L != L;
    const int m = ds.w * kCacheUnitRows + r;
    if (tid < D / 4) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = 4 * tid + e;
        v[e] = s_o[0][d] + s_o[1][d] + s_o[2][d] + s_o[3][d];
        v[e] = some ? v[e] / L : 0.f;
      }
      store2(p, o_row(p, ds.y, ds.z, m) + 4 * tid, make_float4(v[0], v[1], v[2], v[3]));
      if (tid == 0 && p.lse) *lse_row(p, ds.y, ds.z, m) = some ? (M + __log2f(L)) * 0.69314718055994531f : -INFINITY;
    }
  }
}

// Tiles that some head of the group selects, below the length:
// one CTA per (batch row, K/V head).
constexpr int kTilesThreads = 1024;
static_assert(kTilesThreads / 32 == 32, "a lane per warp");

__global__ void __launch_bounds__(kTilesThreads) tiles_kernel(const __grid_constant__ CacheAttnParams p) {
  __shared__ int warp_s[kTilesThreads / 32];
  next_may_launch();
  wait_for_previous();
  const int e = blockIdx.x, b = e / p.c.Hkv, h = e % p.c.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = len_of(p, b);
  const int tiles = min((len + p.tile - 1) / p.tile, p.max_tiles);
  const uint8_t* mrow = p.mask + ((size_t)b * p.Hq + (size_t)h * p.g) * p.NKB;
  int32_t* out = p.list + (size_t)e * p.max_tiles;
  const int lbk = 31 - __clz(p.bk);
  int done = 0;
  for (int base = 0; base < tiles; base += kTilesThreads) {
    const int t = base + tid;
    unsigned on = 0u;
    if (t < tiles) {
      const int k0 = t * p.tile >> lbk, k1 = p.bk < p.tile ? min(k0 + 1, p.NKB - 1) : k0;
#pragma unroll 8
      for (int i = 0; i < p.g; ++i) on |= load_written(mrow + (size_t)i * p.NKB + k0) | load_written(mrow + (size_t)i * p.NKB + k1);
    }
    const unsigned bal = __ballot_sync(0xffffffffu, on != 0u);
    if (lane == 0) warp_s[warp] = __popc(bal);
    __syncthreads();
    // A lane per warp: the tiles of the warps below this one, and of all.
    const int cnt = warp_s[lane];
    int below = lane < warp ? cnt : 0, all = cnt;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      below += __shfl_xor_sync(0xffffffffu, below, o);
      all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    if (on) out[done + below + __popc(bal & ((1u << lane) - 1u))] = t;
    done += all;
    __syncthreads();
  }
  if (tid == 0) p.counts[e] = done;
}

template <int D, int KIND, int NT>
cudaError_t launch_t(const CacheAttnParams& p, int grid, cudaStream_t s) {
  const int smem = AttnCfg<D>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(attn_kernel<D, KIND, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_after(attn_kernel<D, KIND, NT>, dim3(grid), dim3(kAttnThreads), smem, s, p);
}
template <int D, int KIND>
cudaError_t launch_k(const CacheAttnParams& p, int grid, cudaStream_t s) {
  // As few row tiles as hold the rows (1, 2 or 4 of at most 24), for each
  // converts the codes again, and as few columns in them.
  const int rows = p.M < kCacheUnitRows ? p.M : kCacheUnitRows;
  const int per = rows <= 24 ? rows : (rows <= 48 ? (rows + 1) / 2 : (rows + 3) / 4);
  if (per <= 8) return launch_t<D, KIND, 1>(p, grid, s);
  return per <= 16 ? launch_t<D, KIND, 2>(p, grid, s) : launch_t<D, KIND, 3>(p, grid, s);
}
template <int D>
cudaError_t launch_d(const CacheAttnParams& p, int grid, cudaStream_t s) {
  cudaError_t e = p.c.kind == BSA_CACHE_INT8 ? launch_k<D, BSA_CACHE_INT8>(p, grid, s)
                                             : launch_k<D, BSA_CACHE_E4M3>(p, grid, s);
  if (e != cudaSuccess) return e;
  const int rows = p.rows_cap < kCombineRows ? p.rows_cap : kCombineRows;
  return launch_after(combine_kernel<D>, dim3(grid, rows), dim3(128), 0, s, p);
}

}  // namespace

cudaError_t launch_cache_attention(const CacheAttnParams& p, int grid, cudaStream_t s) {
  if (p.mask) {
    const cudaError_t e = launch_after(tiles_kernel, dim3(p.B * p.c.Hkv), dim3(kTilesThreads), 0, s, p);
    if (e != cudaSuccess) return e;
  }
  return p.c.d == 64 ? launch_d<64>(p, grid, s) : launch_d<128>(p, grid, s);
}

}  // namespace bsa
