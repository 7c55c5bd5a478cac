// Eviction from the 8-bit cache: the tokens of a sequence that gathered the least
// attention weight leave, the others move together.
//
// What is computed.  Of the n tokens of a sequence that is cut to k, each K/V head
// keeps the last r = min(recent, k), the first s = min(sink, k - r) and, of those
// between, the k - r - s of largest weight (of equal ones the first); they move, in
// their order, to places 0 .. k - 1.  A block's scale becomes the largest of the
// scales of the tokens that come to lie in it, codes of a smaller one are rounded
// to it.
//
// Two kernels.  select: a cluster of CTAs per (sequence, head), each with a share of
// consecutive tokens, whose weights it holds in shared memory (longer shares are read
// again).  The weight of the last token to be kept is found digit by digit: a histogram
// of 11 bits over all weights, then of those in the digit's bin alone (a few percent),
// the CTAs' histograms added up through distributed shared memory.  The list of kept
// tokens is written in order, and their weights move.  move: a cluster per (sequence,
// head, K or V) moves codes and scales in rounds; the CTA that is the last of its
// sequence sets the length and gives back the pages behind it (a third kernel would
// cost its launch and the drain ahead of it).
//
// Why rounds of a cluster: kept tokens only move towards the front (token i of the
// list comes from a place >= i), so once the sources of places [0, x) have been
// read, writing them harms no source of a later place.  A round's places are read by
// all CTAs of the cluster into registers, the cluster meets, then they are written;
// no second meeting is needed, and nothing is copied twice or waits on a flag.
//
// What bounds them: the selection, short phases between barriers; the move, the bytes
// of kept tokens there and back.  Measured, selection and move: 32 sequences of 2177 to
// 2304 tokens to 2048, 8 heads of 128, E4M3: 14 + 45 us (the move 0.9 of a copy's rate); 48 of
// 700 to 12000 to 1000, 8 heads of 64, INT8, pages of 16: 33 + 34; one of 64001 to 8000: 24 + 19.
//
// Lengths are on the device; threads, shared memory and clusters of the selection go by the
// table's width (or the weights', where that is less) and by the number of pairs.  The first of
// these cases in tables of 2304, 8192, 12288, 16384, 32768 and 131072 tokens a sequence: 56, 58, 57,
// 61, 59 and 72 us in all.  Two sequences of 192 tokens, 8 heads, in clusters of eight: 29 us.
#include "bsa_cache.h"
#include "bsa_cache_codes.cuh"
#include "bsa_device.cuh"

namespace bsa {
namespace {

using namespace dev;

constexpr int kDigit = 11;
constexpr int kBins = 1 << kDigit;

// Keys in the order of weights: NaN below all, both zeros alike.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);  // (-0 becomes +0)
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// What becomes of list item i: its sequence, length and new length; false where it
// is left out (`code`: what is recorded, 0: nothing).
struct Cut {
  int seq, have, want;
};
__device__ __forceinline__ bool cut_of(const CacheEvictParams& p, int i, Cut& x, int& code) {
  const CacheDev& c = p.c;
  x.seq = p.seqs ? load_written(p.seqs + i) : i;
  code = 0;
  if (x.seq == -1) return false;
  code = BSA_ERR_INVALID_ARG;
  if (x.seq < 0 || x.seq >= c.max_seqs) return false;
  x.have = load_written(c.lens + x.seq);
  x.want = load_written(p.keep + i);
  if (x.have < 0 || x.have > c.max_pages * c.page || x.have > p.stride || x.want < 0) return false;
  if (x.want < x.have && x.want > p.keep_max) return false;
  code = 0;
  return true;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Word of another CTA's shared memory (`addr`: this CTA's address of it).
__device__ __forceinline__ int ld_cluster(uint32_t addr, int rank) {
  uint32_t at;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ int2 ld_cluster2(uint32_t addr, int rank) {
  uint32_t at;
  int2 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}

// Tokens of a CTA whose weights are held in shared memory, at most.
constexpr int kHeld = 49152;
constexpr int kList = 128;        // tokens of a bin that are ranked one against another
// Tokens of a CTA on its own, by its table, for which 512 threads do (fewer warps meet sooner; 32
// sequences of 2304 tokens, 8 heads: 256, 512, 1024 threads 78, 67, 80 us in all; up to this
// width two CTAs of 512 fit an SM with all weights held).
constexpr int kFewTokens = 12288;

template <int kSelectThreads>
__global__ void __launch_bounds__(kSelectThreads, 1024 / kSelectThreads) evict_select_kernel(const __grid_constant__ CacheEvictParams p, int cluster,
                                                                      int hold) {
  constexpr int kWarps = kSelectThreads / 32, kMine = kBins / kSelectThreads;  // bins of a thread
  static_assert(kMine % 2 == 0, "bins are read in pairs");
  constexpr bool kJoined = kSelectThreads == 1024;  // (512 threads: a CTA on its own)
  extern __shared__ float s_w[];  // [hold]
  __shared__ int s_hist[2][kBins];  // the digits in turn: others may still read the last one's
  __shared__ int s_warp[2][33];
  __shared__ int s_pick[3];         // bin, how many of it are to be taken, how many there are
  __shared__ uint2 s_list[kList];   // keys and places of a bin's tokens, all CTAs'
  __shared__ uint2 s_other[kList];
  __shared__ int s_listed;
  __shared__ int s_count[2];        // tokens of this CTA that stay in any case, that tie
  const CacheDev& c = p.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit = blockIdx.x / cluster, rank = blockIdx.x - unit * cluster;
  const int i = unit / c.Hkv, h = unit - i * c.Hkv;
  next_may_launch();
  wait_for_previous();
  Cut x;
  int code;
  bool good = cut_of(p, i, x, code);
  bool twice = false;
  if (good && p.seqs) {
    for (int a = tid; a < i; a += kSelectThreads) twice |= load_written(p.seqs + a) == x.seq;
  }
  const bool cuts = good && x.want < x.have;
  bool missing = false, shared = false;
  if (cuts) {
    // Every page is one, and those that are written are the sequence's alone (the first ones, of
    // sinks alone, are not).
    const int32_t* row = c.table + (size_t)x.seq * c.max_pages;
    const int lpage = 31 - __clz(c.page);
    const int hp = (x.have + c.page - 1) >> lpage, wp = (x.want + c.page - 1) >> lpage;
    const int sp = min(p.sink, x.want - min(p.recent, x.want)) >> lpage;
    for (int j = tid; j < hp; j += kSelectThreads) {
      const int pg = load_written(row + j);
      if (pg < 0 || pg >= c.num_pages) missing = true;
      else if (j >= sp && j < wp && load_written(c.refs + pg) > 1) shared = true;
    }
  }
  // This CTA's tokens: consecutive, the shares of warps' sizes.
  const int n = cuts ? x.have : 0, k = x.want;
  const int share = ((n + cluster - 1) / cluster + 31) & ~31, first = min(n, rank * share), count = min(n, first + share) - first;
  const float* w = p.weights + ((size_t)(good ? x.seq : 0) * c.Hkv + h) * p.stride + first;
  const int r = min(p.recent, k), s = min(p.sink, k - r), need = cuts ? k - r - s : 0;
  // Candidates of this CTA: [lo, hi) of its tokens; the others stay.
  const int lo = min(max(s - first, 0), count), hi = max(min(n - r - first, count), lo);
  for (int q = tid; q < kBins; q += kSelectThreads) s_hist[0][q] = 0;
  if (tid == 0) s_listed = 0;
  __syncthreads();
  // Weights into shared memory, and the first digit's histogram.
#pragma unroll 4
  for (int j = tid; j < count; j += kSelectThreads) {
    const float v = load_written(w + j);
    if (j < hold) s_w[j] = v;
    if (j >= lo && j < hi) atomicAdd(&s_hist[0][order_key(v) >> (32 - kDigit)], 1);
  }
  int detail = i;
  const int wrong = __syncthreads_or((twice ? 1 : 0) | (missing ? 2 : 0) | (shared ? 4 : 0));  // (zero or not)
  if (wrong) {
    good = false;
    const bool any_twice = __syncthreads_or(twice), any_missing = __syncthreads_or(missing);
    code = any_twice || !any_missing ? BSA_ERR_INVALID_ARG : BSA_ERR_PLAN_MISMATCH;
    if (!any_twice && any_missing) detail = x.seq;
  }
  if (h == 0 && rank == 0 && tid == 0) {
    p.cut[i] = good && cuts ? x.want : -1;
    p.done[i] = 0;
    if (code != 0) cache_error(c.control, code, detail);
  }
  if (!good) return;  // (the whole cluster)
  int32_t* kept = p.kept + ((size_t)i * c.Hkv + h) * p.keep_max;
  if (!cuts) {
    for (int j = rank * kSelectThreads + tid; j < min(x.have, p.keep_max); j += cluster * kSelectThreads) kept[j] = j;
    return;
  }
  auto weight = [&](int j) { return j < hold ? s_w[j] : load_written(w + j); };  // of token first + j
  // The key of the last of `need` candidates (larger ones are all kept), digit by
  // digit from the top: bits of the key found so far, how many of those that have
  // them are still to be taken.
  uint32_t found = 0u;
  int left = need;
  if (need > 0) {
    int turn = 0;
    for (int shift = 32 - kDigit, bits = kDigit;; turn ^= 1) {
      int* hist = s_hist[turn];
      const uint32_t digit = (1u << bits) - 1u;
      if (shift < 32 - kDigit) {  // (the first one's has been taken with the loads)
        for (int q = tid; q < kBins; q += kSelectThreads) hist[q] = 0;
        __syncthreads();
        const uint32_t above = ~0u << (shift + bits);
        for (int j = lo + tid; j < hi; j += kSelectThreads) {
          const uint32_t key = order_key(weight(j));
          if (((key ^ found) & above) == 0u) atomicAdd(&hist[key >> shift & digit], 1);
        }
      }
      // Sums from the top: thread t has the kMine bins below kBins - kMine t.
      int mine[kMine], sum = 0;
      const int bin0 = kBins - kMine * (tid + 1);
      if (kJoined && cluster > 1) {
        cluster_arrive();
        cluster_wait();
        const uint32_t at = smem_u32(hist + bin0);
#pragma unroll
        for (int e = 0; e < kMine; e += 2) {
          int2 got[8];  // (all on their way at once)
#pragma unroll
          for (int q = 0; q < 8; ++q) got[q] = q < cluster ? ld_cluster2(at + 4 * e, q) : make_int2(0, 0);
          mine[e] = mine[e + 1] = 0;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            mine[e] += got[q].x;
            mine[e + 1] += got[q].y;
          }
        }
      } else {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kMine; ++e) mine[e] = hist[bin0 + e];
      }
#pragma unroll
      for (int e = 0; e < kMine; ++e) sum += mine[e];
      int inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 31) s_warp[0][warp] = inc;
      __syncthreads();
      int before = inc - sum + __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[0][lane] : 0);
      if (before < left && before + sum >= left) {  // (one thread)
#pragma unroll
        for (int e = kMine - 1; e >= 0; --e) {
          if (before < left && before + mine[e] >= left) {
            s_pick[0] = bin0 + e;
            s_pick[1] = left - before;
            s_pick[2] = mine[e];
          }
          before += mine[e];
        }
      }
      __syncthreads();
      found |= (uint32_t)s_pick[0] << shift;
      left = s_pick[1];
      if (shift == 0) break;
      const int members = s_pick[2];
      if (members <= kList) {
        // Few enough to be ranked one against another: the last to be taken is the one
        // that left - 1 of them come before.  CTAs put theirs into each other's lists.
        const uint32_t same = ~0u << shift;
        for (int j = lo + tid; j < hi; j += kSelectThreads) {
          const uint32_t key = order_key(weight(j));
          if (((key ^ found) & same) == 0u) {
            const int at = atomicAdd(&s_listed, 1);
            s_list[at] = make_uint2(key, (uint32_t)(first + j));
          }
        }
        if (kJoined && cluster > 1) {
          cluster_arrive();
          cluster_wait();
          int filled = s_listed;  // (this CTA's own lie in front)
          const int own = filled;
          for (int q = 0; q < cluster; ++q) {
            if (q == rank) continue;
            const int theirs = ld_cluster(smem_u32(&s_listed), q);
            for (int e = tid; e < theirs; e += kSelectThreads) {
              const int2 v = ld_cluster2(smem_u32(s_list + e), q);
              s_other[filled - own + e] = make_uint2((uint32_t)v.x, (uint32_t)v.y);
            }
            filled += theirs;
          }
          __syncthreads();
          for (int e = tid; e < members; e += kSelectThreads) {
            const uint2 me = e < own ? s_list[e] : s_other[e - own];
            int ahead = 0, equal = 0;
            for (int o = 0; o < members; ++o) {
              const uint2 y = o < own ? s_list[o] : s_other[o - own];
              const bool tie = y.x == me.x && y.y < me.y;
              ahead += y.x > me.x || tie;
              equal += tie;
            }
            if (ahead == left - 1) {
              s_pick[0] = (int)me.x;
              s_pick[1] = equal + 1;
            }
          }
        } else {
          __syncthreads();
          for (int e = tid; e < members; e += kSelectThreads) {
            const uint2 me = s_list[e];
            int ahead = 0, equal = 0;
            for (int o = 0; o < members; ++o) {
              const uint2 y = s_list[o];
              const bool tie = y.x == me.x && y.y < me.y;
              ahead += y.x > me.x || tie;
              equal += tie;
            }
            if (ahead == left - 1) {
              s_pick[0] = (int)me.x;
              s_pick[1] = equal + 1;
            }
          }
        }
        __syncthreads();
        found = (uint32_t)s_pick[0];
        left = s_pick[1];
        break;
      }
      bits = min(kDigit, shift);
      shift -= bits;
    }
  }
  // The list: a warp goes over consecutive tokens; counts first, then places.
  // `left` tokens of the found key are kept, the first ones.
  const int span = ((count + kWarps - 1) / kWarps + 31) & ~31, j0 = min(count, warp * span), j1 = min(count, j0 + span);
  auto kind_of = [&](int j, bool& stays, bool& tie) {
    stays = j < lo || j >= hi;
    tie = false;
    if (!stays && need > 0) {
      const uint32_t key = order_key(weight(j));
      stays = key > found;
      tie = key == found;
    }
  };
  int stay = 0, ties = 0;
#pragma unroll 4
  for (int j = j0 + lane; j < j1; j += 32) {
    bool a, b;
    kind_of(j, a, b);
    stay += a;
    ties += b;
  }
  stay = __reduce_add_sync(0xffffffffu, stay);
  ties = __reduce_add_sync(0xffffffffu, ties);
  if (lane == 0) {
    s_warp[0][warp] = stay;
    s_warp[1][warp] = ties;
  }
  __syncthreads();
  const int stay_w = lane < kWarps ? s_warp[0][lane] : 0, ties_w = lane < kWarps ? s_warp[1][lane] : 0;
  int at = __reduce_add_sync(0xffffffffu, lane < warp ? stay_w : 0), tied = __reduce_add_sync(0xffffffffu, lane < warp ? ties_w : 0);
  if (kJoined && cluster > 1) {  // those of the CTAs ahead
    if (warp == 0) {
      const int a = __reduce_add_sync(0xffffffffu, stay_w), b = __reduce_add_sync(0xffffffffu, ties_w);
      if (lane == 0) {
        s_count[0] = a;
        s_count[1] = b;
      }
    }
    cluster_arrive();
    cluster_wait();
    for (int q = 0; q < rank; ++q) {
      at += ld_cluster(smem_u32(s_count), q);
      tied += ld_cluster(smem_u32(s_count + 1), q);
    }
  }
  at += min(tied, left);
  const bool held = share <= hold;  // by every CTA: weights may be written where they belong
  float* wk = p.weights + ((size_t)x.seq * c.Hkv + h) * p.stride;
  auto put = [&](int j, bool a) {
    const uint32_t all = __ballot_sync(0xffffffffu, a);
    if (a) {
      const int to = at + __popc(all & ((1u << lane) - 1u));
      kept[to] = first + j;
      if (held) wk[to] = s_w[j];
    }
    at += __popc(all);
  };
  if (tied >= left || tied + ties <= left) {  // none of this warp's ties are kept, or all
    const uint32_t least = tied >= left ? found + 1u : found;
#pragma unroll 8
    for (int j = j0 + lane; j - lane < j1; j += 32) {
      bool a = j < j1;
      if (a && j >= lo && j < hi) a = need > 0 && order_key(weight(j)) >= least;
      put(j, a);
    }
  } else {
    for (int j = j0 + lane; j - lane < j1; j += 32) {
      bool a = false, b = false;
      if (j < j1) kind_of(j, a, b);
      const uint32_t all_b = __ballot_sync(0xffffffffu, b);
      if (b && tied + __popc(all_b & ((1u << lane) - 1u)) < left) a = true;
      tied += __popc(all_b);
      put(j, a);
    }
  }
  // No CTA leaves while others may read its shared memory, nor (the weights' second
  // way) goes on before the list is there.
  if (kJoined && cluster > 1) {
    if (!held) __threadfence();
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (held || rank > 0) return;
  // Weights of longer shares, by one CTA: read, meet, write; a later chunk's come from
  // places that this one does not write.
  for (int b0 = 0; b0 < k; b0 += 8 * kSelectThreads) {
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int j = b0 + q * kSelectThreads + tid;
      v[q] = j < k ? load_written(wk + __ldcg(kept + j)) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int j = b0 + q * kSelectThreads + tid;
      if (j < k) wk[j] = v[q];
    }
  }
}

// ------------------------------------------------------------------ codes and scales
constexpr int kMoveThreads = 256;
constexpr int kMoveTable = 1024;  // entries of the page table in shared memory

// Codes of a block's smaller scale at its new one: rounded to nearest, ties to even.
template <int KIND>
__device__ __forceinline__ uint4 recode16(uint4 x, float ratio) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (KIND == BSA_CACHE_INT8) {
      // A byte u under 0x4b0000 is fp32 2^23 + u; 1.5 2^23 + y holds y, rounded to a whole
      // number, in its low byte.  ratio is at most 1: nothing to saturate.
      const uint32_t u = w[e] ^ 0x80808080u;  // code + 128
      float f[4];
      f[0] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7650));
      f[1] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7651));
      f[2] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7652));
      f[3] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7653));
#pragma unroll
      for (int q = 0; q < 4; ++q) f[q] = fmaf(f[q] - (8388608.f + 128.f), ratio, 12582912.f);
      const uint32_t a = __byte_perm(__float_as_uint(f[0]), __float_as_uint(f[1]), 0x0040);
      const uint32_t b = __byte_perm(__float_as_uint(f[2]), __float_as_uint(f[3]), 0x0040);
      w[e] = __byte_perm(a, b, 0x5410);
    } else {
      const uint2 hh = codes_to_half4<KIND>(w[e]);
      const float2 a = half2_to_float2(hh.x), b = half2_to_float2(hh.y);
      w[e] = encode2<KIND>(a.x * ratio, a.y * ratio) | encode2<KIND>(b.x * ratio, b.y * ratio) << 16;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D, int KIND>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ CacheEvictParams p, int cluster) {
  constexpr int kTokens = 32768 / D;                   // of a CTA in a round: 32 KB
  constexpr int kPer = kTokens / kMoveThreads;         // a thread looks up
  constexpr int kVec = kTokens * D / 16 / kMoveThreads;  // 16-byte vectors of a thread
  constexpr int kLanes = D / 16;                       // threads of a token
  // Rounds in turn.
  __shared__ int s_from[2][kTokens], s_to[2][kTokens];  // pool rows; -1: no token
  __shared__ float s_scale[2][kTokens];                 // of a token, then over the largest; < 0: nothing stored
  __shared__ uint32_t s_top[2][kTokens / 16];           // bits of the largest of a block
  __shared__ int s_moves[2][kTokens / 16];              // a token of the block moves
  __shared__ int s_table[kMoveTable];
  const CacheDev& c = p.c;
  const int tid = threadIdx.x;
  const int unit = blockIdx.x / cluster, rank = blockIdx.x - unit * cluster;
  const int i = unit / (2 * c.Hkv), x = unit - i * 2 * c.Hkv, h = x >> 1;
  uint8_t* pool = x & 1 ? c.v : c.k;
  float* scales = x & 1 ? c.vs : c.ks;
  const int lpage = 31 - __clz(c.page), lsb = 31 - __clz(c.sb);
  if (tid < 2 * (kTokens / 16)) {
    s_top[0][tid] = 0u;
    s_moves[0][tid] = 0;
  }
  next_may_launch();
  wait_for_previous();
  const int k = load_written(p.cut + i);
  if (k < 0) return;  // (the whole cluster)
  const int seq = p.seqs ? load_written(p.seqs + i) : i;
  const int n = load_written(c.lens + seq);
  const int hp = (n + c.page - 1) >> lpage, wp = (k + c.page - 1) >> lpage;
  int32_t* table = c.table + (size_t)seq * c.max_pages;
  const int32_t* kept = p.kept + ((size_t)i * c.Hkv + h) * p.keep_max;
  const int rounds = (k + kTokens * cluster - 1) / (kTokens * cluster);
  if (rounds > 0)
    for (int j = tid; j < min(hp, kMoveTable); j += kMoveThreads) s_table[j] = load_written(table + j);
  // Where this thread's tokens of a round come from and go to, and their scales.
  int src[kPer], from[kPer], to[kPer];
  float sc[kPer];
  auto list = [&](int round) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int j = (round * cluster + rank) * kTokens + e * kMoveThreads + tid;
      src[e] = j < k ? load_written(kept + j) : -1;
    }
  };
  auto row_of = [&](int j) {
    const int pg = j >> lpage;
    return ((pg < kMoveTable ? s_table[pg] : load_written(table + pg)) * c.Hkv + h) * c.page + (j & (c.page - 1));
  };
  auto find = [&](int round) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int j = (round * cluster + rank) * kTokens + e * kMoveThreads + tid;
      from[e] = src[e] >= 0 ? row_of(src[e]) : -1;
      to[e] = src[e] >= 0 ? row_of(j) : 0;
      sc[e] = src[e] >= 0 ? load_written(scales + (from[e] >> lsb)) : 0.f;
    }
  };
  auto note = [&](int side) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int t = e * kMoveThreads + tid;
      const bool stored = sc[e] > 0.f && sc[e] < INFINITY;
      s_from[side][t] = from[e];
      s_to[side][t] = to[e];
      s_scale[side][t] = stored ? sc[e] : -1.f;
      if (stored) atomicMax(&s_top[side][t >> lsb], __float_as_uint(sc[e]));
      if (from[e] >= 0 && from[e] != to[e]) s_moves[side][t >> lsb] = 1;
    }
  };
  if (rounds > 0) {
    list(0);
    __syncthreads();
    find(0);
    list(1);
    note(0);
  }
  for (int round = 0; round < rounds; ++round) {
    const int side = round & 1, j0 = (round * cluster + rank) * kTokens;
    __syncthreads();  // the round's places are there, the last one's are used up
    if (tid < kTokens / 16) {
      s_top[side ^ 1][tid] = 0u;
      s_moves[side ^ 1][tid] = 0;
    }
    uint4 v[kVec];
#pragma unroll
    for (int q = 0; q < kVec; ++q) {
      const int t = q * (kMoveThreads / kLanes) + tid / kLanes;
      v[q] = make_uint4(0u, 0u, 0u, 0u);
      if (s_from[side][t] >= 0 && s_moves[side][t >> lsb])
        v[q] = load_written(reinterpret_cast<const uint4*>(pool + (size_t)s_from[side][t] * D + 16 * (tid % kLanes)));
    }
    // What becomes of a token's codes, for all threads that hold some of them.
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int t = e * kMoveThreads + tid;
      const float was = s_scale[side][t];
      if (was > 0.f) s_scale[side][t] = was / __uint_as_float(s_top[side][t >> lsb]);
    }
    // (The next rounds' tokens, lists and scales lie behind every place that this one writes.)
    find(round + 1);
    list(round + 2);
    if (cluster > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
#pragma unroll
    for (int q = 0; q < kVec; ++q) {
      const int t = q * (kMoveThreads / kLanes) + tid / kLanes;
      if (s_from[side][t] < 0 || !s_moves[side][t >> lsb]) continue;
      const float ratio = s_scale[side][t];
      uint4 y = v[q];
      if (ratio < 0.f) y = make_uint4(0u, 0u, 0u, 0u);
      else if (ratio != 1.f) y = recode16<KIND>(y, ratio);
      *reinterpret_cast<uint4*>(pool + (size_t)s_to[side][t] * D + 16 * (tid % kLanes)) = y;
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int t = e * kMoveThreads + tid;
      if ((t & (c.sb - 1)) == 0 && j0 + t < k && s_moves[side][t >> lsb])
        scales[s_to[side][t] >> lsb] = __uint_as_float(s_top[side][t >> lsb]);
    }
    note(side ^ 1);
  }
  // The last CTA of the sequence to get here: nobody reads its table any more.
  __shared__ bool s_last;
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    s_last = atomicAdd(p.done + i, 1) == 2 * c.Hkv * cluster - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  for (int j = wp + tid; j < hp; j += kMoveThreads) {
    atomicSub(c.refs + load_written(table + j), 1);
    table[j] = -1;
  }
  __syncthreads();
  if (tid == 0) c.lens[seq] = k;
}

// Launch of clusters that may begin before the kernel ahead has ended.
template <class... Params, class... Args>
cudaError_t launch_clusters(void (*kernel)(Params...), unsigned grid, int threads, int cluster, int smem, cudaStream_t s,
                            const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
// CTAs of a cluster, 1 to `most`: as many as keep `places` CTAs busy.
int cluster_of(long long units, long long places, int most) {
  int x = most;
  while (x > 1 && units * x > places) x >>= 1;
  return x;
}

}  // namespace

cudaError_t launch_cache_evict(const CacheEvictParams& p, int sms, cudaStream_t s) {
  const long long units = (long long)p.n * p.c.Hkv;
  const long long room = (long long)p.c.max_pages * p.c.page < p.stride ? (long long)p.c.max_pages * p.c.page : p.stride;
  const int select = cluster_of(units, 2ll * sms, 8);
  // (no more than its share can be)
  const long long share = (room + 32ll * select - 1) / (32ll * select) * 32;
  const int hold = (int)(share < kHeld ? share : kHeld);
  auto choose = [&](auto kernel, int threads) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeld * 4);
    return e != cudaSuccess ? e : launch_clusters(kernel, (unsigned)(units * select), threads, select, hold * 4, s, p, select, hold);
  };
  cudaError_t e = select == 1 && room <= kFewTokens ? choose(evict_select_kernel<512>, 512)
                                                    : choose(evict_select_kernel<1024>, 1024);
  if (e != cudaSuccess) return e;
  const int move = cluster_of(2 * units, 4ll * sms, 16);
  const unsigned grid = (unsigned)(2 * units * move);
  auto go = [&](auto kernel) {  // (16 CTAs of this size find their places in every GPC)
    const cudaError_t x = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return x != cudaSuccess ? x : launch_clusters(kernel, grid, kMoveThreads, move, 0, s, p, move);
  };
  const bool i8 = p.c.kind == BSA_CACHE_INT8;
  if (p.c.d == 64) return i8 ? go(evict_move_kernel<64, BSA_CACHE_INT8>) : go(evict_move_kernel<64, BSA_CACHE_E4M3>);
  return i8 ? go(evict_move_kernel<128, BSA_CACHE_INT8>) : go(evict_move_kernel<128, BSA_CACHE_E4M3>);
}

}  // namespace bsa
