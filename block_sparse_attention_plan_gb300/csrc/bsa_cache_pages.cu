// Page operations of the 8-bit K/V cache: resize (with copy on write), fork,
// compact and copy.  The whole state is the page table, the lengths and a
// reference count per page; "free" means a count of 0 and pages are taken
// lowest first, so every result is a function of the state and the arguments.
//
// The bookkeeping is a few thousand integers: one CTA of 1024 threads does it
// with block scans (no grid synchronisation, no host), and a second, wide
// kernel moves the page contents it queued.  The copies are what costs: a page
// of 64 tokens and 8 heads is 131 KB.  Compacting 5280 held pages of 8000 moves
// 471 MB in 91 us, of which the copy takes 74 (6.4 TB/s); a step of a few pages
// is the bookkeeping's chain of reads and scans, 6 us to compact 600 pages, 13 and
// 22 us to grow 16 and 256 forked sequences by a token.
#include "bsa_cache.h"

namespace bsa {
namespace {

constexpr int kThreads = 1024;

// Exclusive block scan of one int per thread; `total` gets the sum.  `warp_s`
// is shared scratch of 33 ints.
__device__ __forceinline__ int block_scan(int x, int* warp_s, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_s[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int w = warp_s[lane], s = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_s[lane] = s - w;
    if (lane == 31) warp_s[32] = s;
  }
  __syncthreads();
  total = warp_s[32];
  const int r = warp_s[warp] + inc - x;
  __syncthreads();  // warp_s may be reused
  return r;
}

__device__ __forceinline__ int pages_of(int len, int page) { return (len + page - 1) / page; }

// Bit q of the result: page p0 + q is held (16 pages, a multiple of 16 first).
__device__ __forceinline__ unsigned held_pages(const CacheDev& c, int p0) {
  unsigned bits = 0;
  if (p0 + 16 <= c.num_pages && (reinterpret_cast<uintptr_t>(c.refs) & 15) == 0) {
    int4 r[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) r[q] = __ldcg(reinterpret_cast<const int4*>(c.refs + p0) + q);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      bits |= ((r[q].x > 0) | (r[q].y > 0) << 1 | (r[q].z > 0) << 2 | (r[q].w > 0) << 3) << (4 * q);
  } else {
    for (int q = 0; q < 16; ++q)
      if (p0 + q < c.num_pages && __ldcg(c.refs + p0 + q) > 0) bits |= 1u << q;
  }
  return bits;
}

// A block that a sequence enters (one wholly past its old length) gets scale 0,
// "nothing stored": what the page's last holder left there is no scale of the
// tokens to come.  A growth by one token, a step of decoding, writes none: the
// token is alone in such a block, so storing it sets the scale.
//
// One CTA.  Everything the decisions need is read once, into shared memory, so
// that a step of a serving loop (a token more for each sequence, no page more)
// is a chain of four reads: list, length, last page, its count.
//   s_seq: the sequence (-1: skipped)  s_have, s_want: lengths
//   s_page: its partly filled last page where that is shared (else -1); then
//           whether it takes a page in its place; then where its pages start in
//           the list of free ones
constexpr int kItems = kCacheListMax / kThreads;  // consecutive items per thread

__global__ void __launch_bounds__(kThreads) resize_kernel(const CacheDev c, const int32_t* seqs,
                                                          const int32_t* new_lens, int n) {
  next_may_launch();
  wait_for_previous();
  extern __shared__ int resize_s[];
  int* s_seq = resize_s;
  int* s_have = resize_s + n;
  int* s_want = resize_s + 2 * n;
  int* s_page = resize_s + 3 * n;
  __shared__ int warp_s[33];
  __shared__ int s_pairs;
  __shared__ unsigned long long s_need;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cap = c.max_pages * c.page;
  if (tid == 0) {
    s_pairs = 0;
    s_need = 0;
  }
  for (int i = tid; i < n; i += kThreads) {
    const int s = seqs ? load_written(seqs + i) : i, want = load_written(new_lens + i);
    const bool known = s >= 0 && s < c.max_seqs;
    const int have = known ? __ldcg(c.lens + s) : -1;
    const bool ok = known && want >= 0 && want <= cap && have >= 0 && have <= cap;
    if (!ok && s != -1) cache_error(c.control, BSA_ERR_INVALID_ARG, i);
    s_seq[i] = s;
    s_have[i] = ok ? have : -1;
    s_want[i] = want;
  }
  __syncthreads();
  // A sequence may appear once, its first item counts.
  if (seqs) {
    bool twice[kItems];
    for (int u = 0, i = tid; i < n; i += kThreads, ++u) {
      twice[u] = false;
      const int s = s_seq[i];
      for (int j = 0; j < i; ++j) twice[u] |= s_seq[j] == s;
      if (s < 0) twice[u] = false;
    }
    __syncthreads();
    for (int u = 0, i = tid; i < n; i += kThreads, ++u)
      if (twice[u]) {
        cache_error(c.control, BSA_ERR_INVALID_ARG, i);
        s_have[i] = -1;
      }
  }
  for (int i = tid; i < n; i += kThreads) {
    if (s_have[i] < 0) s_seq[i] = -1;  // (a skipped item's own entry only: no other thread reads it before the barrier)
    s_page[i] = 0;
  }
  bool shrinks = false;
  for (int i = tid; i < n; i += kThreads)
    shrinks |= s_seq[i] >= 0 && pages_of(s_want[i], c.page) < pages_of(s_have[i], c.page);
  // Releases (`sign` -1; +1 takes them back): eight lanes per item, four pages
  // per lane and step.
  auto release = [&](int sign) {
    const int sub = tid & 7;
    for (int i = tid >> 3; i < n; i += kThreads / 8) {
      const int s = s_seq[i];
      if (s < 0) continue;
      const int hp = pages_of(s_have[i], c.page), wp = pages_of(s_want[i], c.page);
      const int32_t* row = c.table + (size_t)s * c.max_pages;
      for (int j = wp + sub; j < hp; j += 32) {
        int pg[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) pg[q] = j + 8 * q < hp ? __ldcg(row + j + 8 * q) : -1;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (j + 8 * q >= hp) continue;
          if (pg[q] >= 0 && pg[q] < c.num_pages) atomicAdd(c.refs + pg[q], sign);
          else cache_error(c.control, BSA_ERR_PLAN_MISMATCH, s);
        }
      }
    }
  };
  shrinks = __syncthreads_or(shrinks);
  if (shrinks) {
    // An item with an entry among them that is no page is skipped; a sequence that
    // is freed gives back those that are.
    for (int i = tid >> 3; i < n; i += kThreads / 8) {
      const int s = s_seq[i];
      if (s < 0 || s_want[i] == 0) continue;
      const int hp = pages_of(s_have[i], c.page);
      for (int j = pages_of(s_want[i], c.page) + (tid & 7); j < hp; j += 8) {
        const int p = __ldcg(c.table + (size_t)s * c.max_pages + j);
        if (p < 0 || p >= c.num_pages) s_page[i] = 1;
      }
    }
    __syncthreads();
    for (int i = tid; i < n; i += kThreads)
      if (s_page[i]) {
        cache_error(c.control, BSA_ERR_PLAN_MISMATCH, s_seq[i]);
        s_seq[i] = -1;
      }
    __syncthreads();
    release(-1);
    __syncthreads();
  }
  // Growth into a partly filled last page that others hold too.
  bool cow = false, enters = false;  // enters: blocks past the old length, in a page held already
  for (int i = tid; i < n; i += kThreads) {
    int shared_page = -1;
    const int s = s_seq[i], have = s_have[i];
    enters |= s >= 0 && s_want[i] > have + 1 && (have & (c.page - 1)) != 0;
    if (s >= 0 && s_want[i] > have && have % c.page) {
      const int p = __ldcg(c.table + (size_t)s * c.max_pages + have / c.page);
      if (p < 0 || p >= c.num_pages) {
        cache_error(c.control, BSA_ERR_PLAN_MISMATCH, s);
        s_seq[i] = -1;  // skipped
      } else if (__ldcg(c.refs + p) > 1) {
        shared_page = p;
      }
    }
    s_page[i] = shared_page;
    cow |= shared_page >= 0;
  }
  cow = __syncthreads_or(cow);
  if (cow) {
    bool own[kItems];
    for (int u = 0, i = tid; i < n; i += kThreads, ++u) {
      const int p = s_page[i];
      own[u] = false;
      if (p < 0) continue;
      int rank = 0;  // earlier items of this call that grow into the same page
      for (int j = 0; j < i; ++j) rank += s_page[j] == p;
      own[u] = __ldcg(c.refs + p) - rank > 1;
    }
    __syncthreads();
    for (int u = 0, i = tid; i < n; i += kThreads, ++u) s_page[i] = own[u] ? 1 : -1;
    __syncthreads();
  }
  // s_page is now 1 for an item that replaces its last page.
  int mine[kItems], sum = 0;
#pragma unroll
  for (int u = 0; u < kItems; ++u) {
    const int i = tid * kItems + u;
    mine[u] = 0;
    if (i < n && s_seq[i] >= 0)
      mine[u] = max(0, pages_of(s_want[i], c.page) - pages_of(s_have[i], c.page)) + (s_page[i] > 0 ? 1 : 0);
    sum += mine[u];
  }
  int total;
  int off = block_scan(sum, warp_s, total);
  if (__syncthreads_or(sum > (1 << 20))) {  // (4096 tables of 2^26 entries: the sum may pass 32 bits)
    atomicAdd(&s_need, (unsigned long long)sum);
    __syncthreads();
    total = (int)min(s_need, 0x7fffffffull);
  }
  // From here on s_page: where an item's pages start in the list, and in the
  // sign bit whether the first of them replaces the shared page.
#pragma unroll
  for (int u = 0; u < kItems; ++u) {
    const int i = tid * kItems + u;
    if (i < n) {
      s_page[i] = off | (s_page[i] > 0 ? (int)0x80000000 : 0);
      off += mine[u];
    }
  }
  // The lowest `total` free pages, in order: 16 pages per thread and step.
  int found = 0;
  for (int base = 0; base < c.num_pages && found < total; base += kThreads * 16) {
    const int p0 = base + tid * 16;
    const unsigned exist = p0 + 16 <= c.num_pages ? 0xffffu : (p0 >= c.num_pages ? 0u : (1u << (c.num_pages - p0)) - 1u);
    unsigned free_bits = ~held_pages(c, p0) & exist;
    int here;
    int at = found + block_scan(__popc(free_bits), warp_s, here);
    while (free_bits && at < total) {
      const int q = __ffs(free_bits) - 1;
      free_bits &= free_bits - 1;
      c.list_a()[at++] = p0 + q;
    }
    found += here;
  }
  __syncthreads();
  if (found < total) {  // nothing changes: take the releases back
    if (shrinks) release(1);
    if (tid == 0) {
      cache_error(c.control, BSA_ERR_WORKSPACE, total - found);
      c.control[kCachePairs] = 0;
      c.control[kCacheTaken] = 0;
    }
    return;
  }
  for (int i = warp; i < n; i += kThreads / 32) {
    const int s = s_seq[i];
    if (s < 0) continue;
    const int want = s_want[i], hp = pages_of(s_have[i], c.page), wp = pages_of(want, c.page);
    int32_t* row = c.table + (size_t)s * c.max_pages;
    int32_t* list = c.list_a() + (s_page[i] & 0x7fffffff);
    const int replaced = s_page[i] < 0 ? 1 : 0;
    if (replaced && lane == 0) {
      const int old = __ldcg(row + hp - 1), fresh = __ldcg(list);
      const int at = atomicAdd(&s_pairs, 1);
      c.pair_src()[at] = old;
      c.pair_dst()[at] = fresh;
      atomicSub(c.refs + old, 1);
      c.refs[fresh] = 1;
      row[hp - 1] = fresh;
    }
    for (int j = hp + lane; j < wp; j += 32) {
      const int p = __ldcg(list + replaced + j - hp);
      c.refs[p] = 1;
      row[j] = p;
    }
    for (int j = wp + lane; j < hp; j += 32) row[j] = -1;
    if (lane == 0) {
      c.lens[s] = want;
      // Left in the list are the pages whose scales the copy kernel clears: not a
      // copied one, and not that of a growth by one token (lane 0 has read it).
      if (replaced || (wp > hp && want == s_have[i] + 1)) list[0] = -1;
    }
  }
  __syncthreads();
  // Scales of the copied pages, then (others may be copying from the page that
  // one keeps) 0 for the blocks past the old length of pages that were held.
  const int lsb = 31 - __clz(c.sb), blocks = c.page >> lsb, scales = c.Hkv * blocks;
  for (int x = tid; x < s_pairs * scales; x += kThreads) {  // (below 2^31: pool rows are)
    const int pr = x / scales, q = x - pr * scales;
    const size_t from = (size_t)__ldcg(c.pair_src() + pr) * scales + q, to = (size_t)__ldcg(c.pair_dst() + pr) * scales + q;
    const float k = c.ks[from], v = c.vs[from];
    c.ks[to] = k;
    c.vs[to] = v;
  }
  if (__syncthreads_or(enters)) {
    for (int i = warp; i < n; i += kThreads / 32) {
      const int s = s_seq[i], have = s_have[i], kept = ((have & (c.page - 1)) + c.sb - 1) >> lsb;
      if (s < 0 || s_want[i] <= have + 1 || kept == 0 || kept == blocks) continue;
      const int p = __ldcg(c.table + (size_t)s * c.max_pages + have / c.page);
      if (p < 0 || p >= c.num_pages) continue;
      for (int x = lane; x < c.Hkv * (blocks - kept); x += 32) {
        const size_t at = ((size_t)p * c.Hkv + x / (blocks - kept)) * blocks + kept + x % (blocks - kept);
        c.ks[at] = 0.f;
        c.vs[at] = 0.f;
      }
    }
  }
  if (tid == 0) {
    c.control[kCachePairs] = s_pairs;
    c.control[kCacheTaken] = total;
  }
}

// Freeing sequences needs no order: one CTA per item, which is skipped if an
// earlier item names its sequence.
__global__ void __launch_bounds__(256) free_kernel(const CacheDev c, const int32_t* seqs, int n) {
  next_may_launch();
  wait_for_previous();
  const int i = blockIdx.x, tid = threadIdx.x;
  const int s = seqs ? load_written(seqs + i) : i;
  if (s == -1) return;
  bool ok = s >= 0 && s < c.max_seqs;
  if (seqs && ok)
    for (int j = tid; j < i; j += 256) ok = ok && load_written(seqs + j) != s;
  const int len = s >= 0 && s < c.max_seqs ? c.lens[s] : 0;
  ok = ok && len >= 0 && len <= c.max_pages * c.page;
  if (!__syncthreads_and(ok)) {
    if (tid == 0) cache_error(c.control, BSA_ERR_INVALID_ARG, i);
    return;
  }
  const int held = pages_of(len, c.page);
  int32_t* row = c.table + (size_t)s * c.max_pages;
  for (int j = tid; j < held; j += 256) {
    const int p = row[j];
    if (p >= 0 && p < c.num_pages) atomicSub(c.refs + p, 1);
    else cache_error(c.control, BSA_ERR_PLAN_MISMATCH, s);
    row[j] = -1;
  }
  if (tid == 0) c.lens[s] = 0;  // (every thread has read it)
}

// One CTA per pair; each checks its own pair against the whole list.  A length
// that a pair reads is written by no other one: a source is no destination.
__global__ void __launch_bounds__(256) fork_kernel(const CacheDev c, const int32_t* src, const int32_t* dst, int n) {
  next_may_launch();
  wait_for_previous();
  const int i = blockIdx.x, tid = threadIdx.x;
  const int a = load_written(src + i), b = load_written(dst + i);
  if (a == -1 || b == -1) return;
  bool ok = a >= 0 && a < c.max_seqs && b >= 0 && b < c.max_seqs;
  for (int j = tid; ok && j < n; j += 256) {
    const int sj = load_written(src + j), dj = load_written(dst + j);
    if (sj == -1 || dj == -1) continue;
    if ((dj == b && j < i) || sj == b) ok = false;
  }
  int len = 0;
  if (ok) {
    len = c.lens[a];
    ok = len >= 0 && len <= c.max_pages * c.page && c.lens[b] == 0;
  }
  if (!__syncthreads_and(ok)) {
    if (tid == 0) cache_error(c.control, BSA_ERR_INVALID_ARG, i);
    return;
  }
  const int held = pages_of(len, c.page);
  const int32_t* from = c.table + (size_t)a * c.max_pages;
  int32_t* to = c.table + (size_t)b * c.max_pages;
  bool whole = true;
  for (int j = tid; j < held; j += 256) whole &= from[j] >= 0 && from[j] < c.num_pages;
  if (!__syncthreads_and(whole)) {
    if (tid == 0) cache_error(c.control, BSA_ERR_PLAN_MISMATCH, a);
    return;
  }
  for (int j = tid; j < held; j += 256) {
    const int p = from[j];
    to[j] = p;
    atomicAdd(c.refs + p, 1);
  }
  if (tid == 0) c.lens[b] = len;  // (every thread has read lens[b]: the barrier above)
}

// One CTA.  The i-th held page at or past L goes to the i-th free page below
// L; list_a gets the map of the moved pages (indexed by page), the pairs what
// the copy kernel moves.  16 pages per thread and step; a pool of up to 16384
// pages is read once, held in registers between the count and the lists.
__global__ void __launch_bounds__(kThreads) compact_kernel(const CacheDev c) {
  next_may_launch();
  wait_for_previous();
  __shared__ int warp_s[33];
  const int tid = threadIdx.x;
  constexpr int kStep = kThreads * 16;
  const unsigned first = held_pages(c, tid * 16);
  int live = __popc(first);
  for (int base = kStep; base < c.num_pages; base += kStep) live += __popc(held_pages(c, base + tid * 16));
  int L;
  block_scan(live, warp_s, L);
  int holes = 0, moved = 0;
  for (int base = 0; base < c.num_pages; base += kStep) {
    const int p0 = base + tid * 16;
    const unsigned held = base == 0 ? first : held_pages(c, p0);
    // Pages of these 16 below L, and that exist.
    const unsigned below = p0 + 16 <= L ? 0xffffu : (p0 >= L ? 0u : (1u << (L - p0)) - 1u);
    unsigned hole = ~held & below, mover = held & ~below;
    // Holes lie below L and movers at or past it: one scan of both counts.
    int both;
    const int at = block_scan(__popc(hole) | __popc(mover) << 16, warp_s, both);
    int ha = holes + (at & 0xffff), ma = moved + (at >> 16);
    while (hole) {
      c.pair_dst()[ha++] = p0 + __ffs(hole) - 1;
      hole &= hole - 1;
    }
    while (mover) {
      c.pair_src()[ma++] = p0 + __ffs(mover) - 1;
      mover &= mover - 1;
    }
    holes += both & 0xffff;
    moved += both >> 16;
  }
  __syncthreads();
#pragma unroll 4
  for (int i = tid; i < moved; i += kThreads) {
    const int p = __ldcg(c.pair_src() + i), to = __ldcg(c.pair_dst() + i);
    c.list_a()[p] = to;
    c.refs[to] = __ldcg(c.refs + p);
    c.refs[p] = 0;
  }
  if (tid == 0) {
    c.control[kCacheLive] = L;
    c.control[kCachePairs] = moved;
  }
}

// The pairs a caller asks for: those that are in range, whose destination no
// earlier pair has and (within one cache) no pair reads.
__global__ void __launch_bounds__(kThreads) check_pairs_kernel(const CacheDev dst, const CacheDev src, int same,
                                                               const int32_t* dp, const int32_t* sp, int n) {
  next_may_launch();
  wait_for_previous();
  __shared__ int s_pairs;
  const int tid = threadIdx.x;
  int32_t* mark = dst.list_a();
  if (tid == 0) s_pairs = 0;
  for (int i = tid; i < n; i += kThreads) {
    const int d = dp[i], s = sp[i];
    if (d >= 0 && d < dst.num_pages) mark[d] = 0x7fffffff;
    if (same && s >= 0 && s < dst.num_pages) mark[s] = 0x7fffffff;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const int d = dp[i];
    if (d >= 0 && d < dst.num_pages) atomicMin(mark + d, i);
  }
  __syncthreads();
  if (same) {  // a source: negative from here on
    for (int i = tid; i < n; i += kThreads) {
      const int s = sp[i];
      if (s >= 0 && s < dst.num_pages) atomicOr(mark + s, (int)0x80000000);
    }
  }
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const int d = dp[i], s = sp[i];
    const bool ok = d >= 0 && d < dst.num_pages && s >= 0 && s < src.num_pages && __ldcg(mark + d) == i;
    if (!ok) {
      cache_error(dst.control, BSA_ERR_INVALID_ARG, i);
      continue;
    }
    const int at = atomicAdd(&s_pairs, 1);
    dst.pair_src()[at] = s;
    dst.pair_dst()[at] = d;
  }
  __syncthreads();
  if (tid == 0) dst.control[kCachePairs] = s_pairs;
}

// Moves the contents of the queued pairs (and, after a compaction, rewrites the
// table; after a resize, which has copied the pairs' scales, clears those of the
// pages taken).  Work items of 16 KB of codes: 256 threads x 4 independent
// 16-byte copies, so that eight CTAs keep 128 KB in flight per SM; a pair's
// scales are one more item.
constexpr int kCopyThreads = 256;
constexpr int kCopyBytes = kCopyThreads * 16 * 4;
enum class CopyFor { kPages, kResize, kCompact };

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const CacheDev dst, const CacheDev src, CopyFor what) {
  next_may_launch();
  wait_for_previous();
  const int tid = threadIdx.x;
  const int pairs = __ldcg(dst.control + kCachePairs);
  const long long bytes = (long long)dst.Hkv * dst.page * dst.d;  // of a page of K or V: a multiple of 1 KB
  const int chunks = (int)((bytes + kCopyBytes - 1) / kCopyBytes);
  const int per = 2 * chunks + (what == CopyFor::kResize ? 0 : 1);
  const int scales = dst.Hkv * (dst.page / dst.sb);
  const long long items = (long long)pairs * per;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int pr = (int)(it / per), w = (int)(it % per);
    const int a = __ldcg(dst.pair_src() + pr), b = __ldcg(dst.pair_dst() + pr);
    if (w < 2 * chunks) {
      const uint8_t* from = (w < chunks ? src.k : src.v) + (size_t)a * bytes;
      uint8_t* to = (w < chunks ? dst.k : dst.v) + (size_t)b * bytes;
      const long long o = (long long)(w < chunks ? w : w - chunks) * kCopyBytes + tid * 16;
      uint4 x[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (o + q * (kCopyThreads * 16) < bytes) x[q] = __ldcs(reinterpret_cast<const uint4*>(from + o + q * (kCopyThreads * 16)));
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (o + q * (kCopyThreads * 16) < bytes) *reinterpret_cast<uint4*>(to + o + q * (kCopyThreads * 16)) = x[q];
    } else {
      for (int i = tid; i < scales; i += kCopyThreads) {
        dst.ks[(size_t)b * scales + i] = src.ks[(size_t)a * scales + i];
        dst.vs[(size_t)b * scales + i] = src.vs[(size_t)a * scales + i];
      }
    }
  }
  if (what == CopyFor::kResize) {
    const int all = __ldcg(dst.control + kCacheTaken) * scales;  // (below 2^31: pool rows are)
    for (int x = blockIdx.x * kCopyThreads + tid; x < all; x += gridDim.x * kCopyThreads) {
      const int p = __ldcg(dst.list_a() + x / scales);
      if (p < 0) continue;
      dst.ks[(size_t)p * scales + x % scales] = 0.f;
      dst.vs[(size_t)p * scales + x % scales] = 0.f;
    }
  }
  if (what == CopyFor::kCompact && pairs > 0) {
    const int L = __ldcg(dst.control + kCacheLive);
    const long long entries = (long long)dst.max_seqs * dst.max_pages;
    for (long long e = (long long)blockIdx.x * kCopyThreads + tid; e < entries; e += (long long)gridDim.x * kCopyThreads) {
      const int p = dst.table[e];
      if (p >= L && p < dst.num_pages) dst.table[e] = __ldcg(dst.list_a() + p);
    }
  }
}

// CTAs of the copy kernel for at most `pairs` pairs: eight per SM at most.
int copy_grid(const CacheDev& c, long long pairs, int sms) {
  const long long per = 2 * (((long long)c.Hkv * c.page * c.d + kCopyBytes - 1) / kCopyBytes) + 1;
  const long long want = pairs * per;
  const long long most = 8ll * (sms > 0 ? sms : 1);
  return (int)(want < 1 ? 1 : (want < most ? want : most));
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 1;
  return sms;
}

}  // namespace

cudaError_t launch_cache_resize(const CacheDev& c, const int32_t* seqs, const int32_t* new_lens, int n,
                                cudaStream_t s) {
  if (!new_lens) {
    return launch_after(free_kernel, dim3(n), dim3(256), 0, s, c, seqs, n);
  }
  const int smem = 4 * n * (int)sizeof(int);
  cudaError_t e = cudaSuccess;
  // (one limit for every call: the attribute is the kernel's, shared by host threads)
  if (smem > 48 * 1024 - 256)
    e = cudaFuncSetAttribute(resize_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             4 * kCacheListMax * (int)sizeof(int));
  if (e != cudaSuccess) return e;
  e = launch_after(resize_kernel, dim3(1), dim3(kThreads), smem, s, c, seqs, new_lens, n);
  if (e != cudaSuccess) return e;
  return launch_after(copy_kernel, dim3(copy_grid(c, n, sm_count())), dim3(kCopyThreads), 0, s, c, c, CopyFor::kResize);
}

cudaError_t launch_cache_fork(const CacheDev& c, const int32_t* src, const int32_t* dst, int n, cudaStream_t s) {
  return launch_after(fork_kernel, dim3(n), dim3(256), 0, s, c, src, dst, n);
}

cudaError_t launch_cache_compact(const CacheDev& c, int sms, cudaStream_t s) {
  const cudaError_t e = launch_after(compact_kernel, dim3(1), dim3(kThreads), 0, s, c);
  if (e != cudaSuccess) return e;
  return launch_after(copy_kernel, dim3(copy_grid(c, c.num_pages / 2 + 1, sms)), dim3(kCopyThreads), 0, s, c, c, CopyFor::kCompact);
}

cudaError_t launch_cache_copy(const CacheDev& dst, const CacheDev& src, const int32_t* dst_pages,
                              const int32_t* src_pages, int n, cudaStream_t s) {
  const int same = dst.k == src.k ? 1 : 0;
  const cudaError_t e =
      launch_after(check_pairs_kernel, dim3(1), dim3(kThreads), 0, s, dst, src, same, dst_pages, src_pages, n);
  if (e != cudaSuccess) return e;
  return launch_after(copy_kernel, dim3(copy_grid(dst, n, sm_count())), dim3(kCopyThreads), 0, s, dst, src, CopyFor::kPages);
}

}  // namespace bsa
