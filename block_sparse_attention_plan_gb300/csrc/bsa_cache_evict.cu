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
#include "bsa_cache.h"
#include "bsa_cache_codes.cuh"
#include "bsa_device.cuh"

namespace bsa {
namespace {

using namespace dev;

constexpr int kSelectThreads = 1024;
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

// Tokens of a CTA whose weights are held in shared memory: two sizes, the smaller one
// lets two CTAs share an SM.
constexpr int kHeldSmall = 12288, kHeldLarge = 49152;

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const __grid_constant__ CacheEvictParams p, int cluster,
                                                                      int hold) {
  extern __shared__ float s_w[];  // [hold]
  __shared__ int s_hist[2][kBins];  // the digits in turn: others may still read the last one's
  __shared__ int s_warp[2][33];
  __shared__ int s_pick[2];
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
    // Every page is one, and those that are written are the sequence's alone.
    const int32_t* row = c.table + (size_t)x.seq * c.max_pages;
    const int lpage = 31 - __clz(c.page);
    const int hp = (x.have + c.page - 1) >> lpage, wp = (x.want + c.page - 1) >> lpage;
    for (int j = tid; j < hp; j += kSelectThreads) {
      const int pg = load_written(row + j);
      if (pg < 0 || pg >= c.num_pages) missing = true;
      else if (j < wp && load_written(c.refs + pg) > 1) shared = true;
    }
  }
  // This CTA's tokens: consecutive, the shares of warps' sizes.
  const int n = cuts ? x.have : 0, k = x.want;
  const int share = ((n + cluster - 1) / cluster + 31) & ~31, first = min(n, rank * share), count = min(n, first + share) - first;
  const float* w = p.weights + ((size_t)(good ? x.seq : 0) * c.Hkv + h) * p.stride + first;
  for (int j = tid; j < min(count, hold); j += kSelectThreads) s_w[j] = load_written(w + j);
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
  const int r = min(p.recent, k), s = min(p.sink, k - r), need = k - r - s;
  // Candidates of this CTA: [lo, hi) of its tokens; the others stay.
  const int lo = min(max(s - first, 0), count), hi = max(min(n - r - first, count), lo);
  // The key of the last of `need` candidates (larger ones are all kept), digit by
  // digit from the top: bits of the key found so far, how many of those that have
  // them are still to be taken.
  uint32_t found = 0u;
  int left = need;
  if (need > 0) {
    int turn = 0;
    for (int shift = 32 - kDigit, bits = kDigit;; turn ^= 1) {
      int* hist = s_hist[turn];
      for (int q = tid; q < kBins; q += kSelectThreads) hist[q] = 0;
      __syncthreads();
      const uint32_t above = shift + bits == 32 ? 0u : ~0u << (shift + bits);
      const uint32_t digit = (1u << bits) - 1u;
      for (int j = lo + tid; j < hi; j += kSelectThreads) {
        const uint32_t key = order_key(weight(j));
        if (((key ^ found) & above) == 0u) atomicAdd(&hist[key >> shift & digit], 1);
      }
      // Sums from the top: thread t has bins kBins - 1 - 2 t and the one below.
      int top, low;
      if (cluster > 1) {
        cluster_arrive();
        cluster_wait();
        const uint32_t at = smem_u32(hist + kBins - 2 - 2 * tid);
        top = low = 0;
        for (int q = 0; q < cluster; ++q) {
          low += ld_cluster(at, q);
          top += ld_cluster(at + 4, q);
        }
      } else {
        __syncthreads();
        top = hist[kBins - 1 - 2 * tid];
        low = hist[kBins - 2 - 2 * tid];
      }
      int inc = top + low;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 31) s_warp[0][warp] = inc;
      __syncthreads();
      int before = inc - top - low;
      {
        const int y = s_warp[0][lane];
        before += __reduce_add_sync(0xffffffffu, lane < warp ? y : 0);
      }
      if (before < left && before + top >= left) {
        s_pick[0] = kBins - 1 - 2 * tid;
        s_pick[1] = left - before;
      } else if (before + top < left && before + top + low >= left) {
        s_pick[0] = kBins - 2 - 2 * tid;
        s_pick[1] = left - before - top;
      }
      __syncthreads();
      found |= (uint32_t)s_pick[0] << shift;
      left = s_pick[1];
      if (shift == 0) break;
      bits = min(kDigit, shift);
      shift -= bits;
    }
  }
  // The list: a warp goes over consecutive tokens; counts first, then places.
  // `left` tokens of the found key are kept, the first ones.
  const int span = ((count + 31) / 32 + 31) & ~31, j0 = min(count, warp * span), j1 = min(count, j0 + span);
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
  const int stay_w = s_warp[0][lane], ties_w = s_warp[1][lane];
  int at = __reduce_add_sync(0xffffffffu, lane < warp ? stay_w : 0), tied = __reduce_add_sync(0xffffffffu, lane < warp ? ties_w : 0);
  if (cluster > 1) {  // those of the CTAs ahead
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
#pragma unroll 4
  for (int j = j0 + lane; j - lane < j1; j += 32) {
    bool a = false, b = false;
    if (j < j1) kind_of(j, a, b);
    const uint32_t all_b = __ballot_sync(0xffffffffu, b);
    const uint32_t under = (1u << lane) - 1u;
    if (b && tied + __popc(all_b & under) < left) a = true;
    const uint32_t all_a = __ballot_sync(0xffffffffu, a);
    if (a) {
      const int to = at + __popc(all_a & under);
      kept[to] = first + j;
      if (held) wk[to] = s_w[j];
    }
    at += __popc(all_a);
    tied += __popc(all_b);
  }
  // No CTA leaves while others may read its shared memory, nor (the weights' second
  // way) goes on before the list is there.
  if (cluster > 1) {
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
constexpr int kMoveTokens = 256;  // of a CTA in a round: a thread finds one, 32 KB at d = 128

template <int D, int KIND>
__device__ __forceinline__ uint4 recode16(uint4 x, float ratio) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint2 hh = codes_to_half4<KIND>(w[e]);
    const float2 a = half2_to_float2(hh.x), b = half2_to_float2(hh.y);
    w[e] = encode2<KIND>(a.x * ratio, a.y * ratio) | encode2<KIND>(b.x * ratio, b.y * ratio) << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D, int KIND>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ CacheEvictParams p, int cluster) {
  constexpr int kVec = kMoveTokens * D / 16 / kMoveThreads;  // 16-byte vectors of a thread
  constexpr int kLanes = D / 16;                             // threads of a token
  __shared__ long long s_from[kMoveTokens];  // pool rows
  __shared__ long long s_to[kMoveTokens];
  __shared__ float s_scale[kMoveTokens];     // of a token; 0: nothing stored
  __shared__ uint32_t s_tops[2][kMoveTokens / 16];  // bits of the largest of a block; rounds in turn
  __shared__ int s_moved[2][kMoveTokens / 16];      // a token of the block moves
  const CacheDev& c = p.c;
  const int tid = threadIdx.x;
  const int unit = blockIdx.x / cluster, rank = blockIdx.x - unit * cluster;
  const int i = unit / (2 * c.Hkv), x = unit - i * 2 * c.Hkv, h = x >> 1;
  uint8_t* pool = x & 1 ? c.v : c.k;
  float* scales = x & 1 ? c.vs : c.ks;
  const int lpage = 31 - __clz(c.page), lsb = 31 - __clz(c.sb);
  next_may_launch();
  wait_for_previous();
  const int k = load_written(p.cut + i);
  if (k < 0) return;  // (the whole cluster)
  const int seq = p.seqs ? load_written(p.seqs + i) : i;
  const int32_t* table = c.table + (size_t)seq * c.max_pages;
  const int32_t* kept = p.kept + ((size_t)i * c.Hkv + h) * p.keep_max;
  const int rounds = (k + kMoveTokens * cluster - 1) / (kMoveTokens * cluster);
  for (int round = 0; round < rounds; ++round) {
    const int j0 = (round * cluster + rank) * kMoveTokens;
    uint32_t* s_top = s_tops[round & 1];
    int* s_moves = s_moved[round & 1];
    // Where this thread's token comes from and goes to.
    if (tid < kMoveTokens / 16) {
      s_top[tid] = 0u;
      s_moves[tid] = 0;
    }
    __syncthreads();  // (also: the last round's places are used up)
    {
      const int j = j0 + tid;
      long long from = -1, to = 0;
      float sc = 0.f;
      if (j < k) {
        const int src = load_written(kept + j);
        from = ((long long)load_written(table + (src >> lpage)) * c.Hkv + h) * c.page + (src & (c.page - 1));
        to = ((long long)load_written(table + (j >> lpage)) * c.Hkv + h) * c.page + (j & (c.page - 1));
        sc = load_written(scales + (from >> lsb));
        if (!(sc > 0.f && sc < INFINITY)) sc = 0.f;
        if (sc > 0.f) atomicMax(&s_top[tid >> lsb], __float_as_uint(sc));
        if (from != to) s_moves[tid >> lsb] = 1;
      }
      s_from[tid] = from;
      s_to[tid] = to;
      s_scale[tid] = sc;
    }
    __syncthreads();
    uint4 v[kVec];
#pragma unroll
    for (int q = 0; q < kVec; ++q) {
      const int t = q * (kMoveThreads / kLanes) + tid / kLanes;
      v[q] = make_uint4(0u, 0u, 0u, 0u);
      if (s_from[t] >= 0 && s_moves[t >> lsb])
        v[q] = load_written(reinterpret_cast<const uint4*>(pool + s_from[t] * D + 16 * (tid % kLanes)));
    }
    cluster_arrive();
    cluster_wait();
#pragma unroll
    for (int q = 0; q < kVec; ++q) {
      const int t = q * (kMoveThreads / kLanes) + tid / kLanes;
      if (s_from[t] < 0 || !s_moves[t >> lsb]) continue;
      const float was = s_scale[t], now = __uint_as_float(s_top[t >> lsb]);
      uint4 y = v[q];
      if (!(was > 0.f)) y = make_uint4(0u, 0u, 0u, 0u);
      else if (was != now) y = recode16<D, KIND>(y, was / now);
      *reinterpret_cast<uint4*>(pool + s_to[t] * D + 16 * (tid % kLanes)) = y;
    }
    if ((tid & (c.sb - 1)) == 0 && j0 + tid < k && s_moves[tid >> lsb])
      scales[s_to[tid] >> lsb] = __uint_as_float(s_top[tid >> lsb]);
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
  const int n = load_written(c.lens + seq);
  int32_t* row = c.table + (size_t)seq * c.max_pages;
  const int hp = (n + c.page - 1) >> lpage, wp = (k + c.page - 1) >> lpage;
  for (int j = wp + tid; j < hp; j += kMoveThreads) {
    atomicSub(c.refs + load_written(row + j), 1);
    row[j] = -1;
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
// CTAs of a cluster, 1 to 8: as many as keep `places` CTAs busy.
int cluster_of(long long units, long long places) {
  int x = 8;
  while (x > 1 && units * x > places) x >>= 1;
  return x;
}

}  // namespace

cudaError_t launch_cache_evict(const CacheEvictParams& p, int sms, cudaStream_t s) {
  const long long units = (long long)p.n * p.c.Hkv;
  const long long room = (long long)p.c.max_pages * p.c.page < p.stride ? (long long)p.c.max_pages * p.c.page : p.stride;
  const int select = cluster_of(units, 2ll * sms);  // two CTAs of 1024 threads an SM
  const int hold = room <= (long long)select * kHeldSmall ? kHeldSmall : kHeldLarge;
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeldLarge * 4);
  if (e != cudaSuccess) return e;
  e = launch_clusters(evict_select_kernel, (unsigned)(units * select), kSelectThreads, select, hold * 4, s, p, select, hold);
  if (e != cudaSuccess) return e;
  const int move = cluster_of(2 * units, 8ll * sms);  // (twice the four CTAs an SM that registers allow)
  const unsigned grid = (unsigned)(2 * units * move);
  auto go = [&](auto kernel) { return launch_clusters(kernel, grid, kMoveThreads, move, 0, s, p, move); };
  const bool i8 = p.c.kind == BSA_CACHE_INT8;
  if (p.c.d == 64) return i8 ? go(evict_move_kernel<64, BSA_CACHE_INT8>) : go(evict_move_kernel<64, BSA_CACHE_E4M3>);
  return i8 ? go(evict_move_kernel<128, BSA_CACHE_INT8>) : go(evict_move_kernel<128, BSA_CACHE_E4M3>);
}

}  // namespace bsa
