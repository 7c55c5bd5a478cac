// Attention of packed prompts: softmax(scale Q K^T) V within each prompt, causal
// or not, heads grouped over K/V heads.
//
// Work items are 256 query rows of one prompt: two 128-row tiles, whose rows are
// 256 / gp tokens of gp heads that share a K/V head (gp: the largest power of two
// in the group, at most 16).  A schedule kernel lists the items of all prompts,
// those with the most key blocks first; the attention kernel's CTAs (one per SM) take
// them, for one group of heads after the other, from a counter.  For few prompts of few
// tokens the schedule kernel would be up to a quarter of the time: there each CTA finds its
// own items in the line of all prompts', from its end on.  That puts a prompt's longest
// items first, but not those of a long prompt ahead of short ones (figures beside
// kPromptFew).
//
// One CTA (384 threads):
//   warp 0    takes work items, publishes them, loads both Q tiles and the K and
//             V blocks (128 keys) into one ring, in the order they are used;
//   warps 1, 2  issue the products.  At d = 128, where they are what takes the time:
//             S = Q K^T and O += P V of tile A and of tile B, in turns:
//               PV_A(j) S_A(j+1) | PV_B(j) S_B(j+1) | PV_A(j+1) ...,
//             so that one tile's products run while the other tile's softmax does.
//             Each has done its waiting when its turn comes, while the other's products
//             keep the tensor cores busy.  (One thread for both: 350 to 1000 cycles of
//             waits with nothing queued, a prompt of 12007 tokens, 32 / 8 heads of 128,
//             859 us, and 953 with descriptors in one thread's registers; two without
//             turns fall into step, products and softmax of both tiles by turns: 994;
//             in turns: 749.)
//             At d = 64, where a tile waits longer for its products' way (P's arrival, the
//             issue, S's arrival: half of a block's time) than for the products: tensor
//             memory has room for three buffers of scores, so warp 1 issues S up to three
//             steps (A, B, A ..) ahead, warp 2 P V.  (A prompt of 8192 tokens, 32 / 8 heads of
//             64: 256 us, 288 in turns; one warp for both: 382, a step's waits, commits and
//             descriptors are some 1700 cycles of its instructions; blocks of 64 keys with
//             two buffers a tile: 360; four tiles of them: 607, spilled registers.)
//   warp 3    looks over the values of every block that some row of the item does not
//             attend as a whole (below);
//   warps 4-7, 8-11  the softmax of tile A and of tile B, a thread per row, against a
//             reference that is the first block's maximum and moves (O is rescaled) only when
//             a block's weights come to more than 2^15: no maximum is taken of the others, a
//             quarter of the time from S to P, which is what the two tiles wait for.  And the
//             epilogue.
//
// Tensor memory (512 columns): S_A, S_B (128 each; three of them at d = 64), O_A, O_B (d
// each).  P takes the
// first 64 columns of its tile's S: a warp has read its rows' scores before it writes
// their weights, and S_x(j+1) is issued behind PV_x(j), which reads them: the
// instructions of one thread run in their order (at d = 64 S of step i + 3 waits for P V
// of step i).  For the same reason the arrival of S_x(j+1) tells the softmax that PV_x(j) is
// done with O (at d = 64 a softmax that rescales O waits for that).
//
// Keys that a row does not attend get weight 0, which keeps a score of any kind out,
// but 0 times a value that is infinite or NaN is NaN: a later token's, or (past the
// prompt's end) another prompt's.  So in blocks that some row attends in part such
// values are replaced by 0 in shared memory before the product, and an item that had
// any adds them to the rows that do attend them at its end, from global memory.
//
// Weights are rounded to the inputs' type, which is what the tensor cores take beside such
// values; their sum is of the unrounded ones.  O is 2e-3 (bf16) or 3e-4 (fp16) of its norm
// off a result whose weights stay in 32 bits, and 1.2 to 1.3 times as far from the exact one
// as that (rounding O is most of both).  Two products with P in two parts would take that away
// for half as much work again.
//
// What bounds it: the tensor cores, 2 * 2 * 128 * 128 d flops a block and tile (d = 128:
// 72 % busy; 12007 tokens, 32 / 8 heads: 694 to 713 us for the kernel alone, 1660 to 1700
// TFLOP/s, 725 to 767 for a call among others, where the power limit comes in; not causal
// 1399 to 1421, 1661 to 1689), and the exponentials, 128 * 128, with what a step costs the issuing
// warps (d = 64, 8192 tokens: 255 to 260 us, 1057 to 1077 TFLOP/s, not causal 469, 1171).
#include <cstdint>

#include "bsa_device.cuh"
#include "bsa_internal.h"
#include "bsa_prompt.h"

namespace bsa {
namespace {

using namespace dev;

constexpr int kThreads = 384;
// 128 x kRegsControl + 256 x kRegsSoftmax within the 384 x 168 of the launch.
constexpr int kRegsControl = 72;
constexpr int kRegsSoftmax = 208;
static_assert(128 * kRegsControl + 256 * kRegsSoftmax <= kThreads * 168, "register split");
constexpr int kSlots = 4;                   // work items published ahead
constexpr int kConsumers = 2 + 1 + 8;       // issuing warps, scanning warp, eight softmax warps
// A block's weights of a row that sum to more than 2^kMostLog move the row's reference.
// fp16 weights are kept at 2^6 of their size, and none of them is past fp16's range of 2^16
// then: 128 at the reference sum to 2^13, and what falls below the range is 2^-30 of the
// reference.  bf16 weights have fp32's range: they are kept at 2^-kMostLog over the number of a
// row's blocks, so that all of its weights sum to less than 1 and no finite value, however
// large, takes O out of range.  (At the other end values below 2^-100 lose bits to fp32's
// smallest numbers: weights at the reference are 2^-16 for one block, 2^-22 for 12007 tokens.)
constexpr int kMostLog = 15;

enum PromptSite : int { kSitePromptOffsets = 0x60, kSiteTurn };

template <int D_>
struct Cfg {
  static constexpr int D = D_;
  // Three buffers of scores between both tiles, one warp that fills and one that uses them
  // (below); otherwise a buffer and a warp of its own for each tile.
  static constexpr bool kThree = D == 64;
  static constexpr int kAhead = kThree ? 2 : 1;      // blocks that the ring has keys ahead of values
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kChunkBytes = 128 * 128;
  static constexpr int kQBufs = D == 128 ? 1 : 2;  // of both tiles
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kOffKV = kQBufs * 2 * kTileBytes;
  static constexpr int kOffBar = kOffKV + kStages * kTileBytes;
  static constexpr int kQFull = 0, kQEmpty = 2;
  static constexpr int kFull = 4;
  static constexpr int kClean = kFull + kStages;
  // Both tiles are done with block b (of the CTA's): its values and the next keys.
  // kBlocks: more than the ring's entries belong to.
  static constexpr int kBlocks = 16;
  static constexpr int kDone = kClean + kBlocks;
  static constexpr int kSFull = kDone + kBlocks;         // [2]; kThree: [2][3], of a tile and a buffer
  static constexpr int kPFull = kSFull + (kThree ? 6 : 2); // [2]; kThree: [3], of a buffer
  static constexpr int kFree = kPFull + 3;               // kThree: [3], P V is done with a buffer
  static constexpr int kKeysIn = kFree + 3;              // kThree: [kBlocks], the keys of a block are there
  static constexpr int kOFull = kKeysIn + (kThree ? kBlocks : 0);  // [2]
  static constexpr int kOFree = kOFull + 2;              // [2]
  static constexpr int kTurn = kOFree + 2;               // [2]
  static constexpr int kDrain = kTurn + 2;               // [2]
  static constexpr int kSchedFull = kDrain + 2;
  static constexpr int kSchedEmpty = kSchedFull + kSlots;
  static constexpr int kNumBars = kSchedEmpty + kSlots;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;   // tmem base, abort flag, copies requested of K/V and of Q, status and detail
  static constexpr int kOffSched = kOffMisc + 32;           // int [kSlots][8]
  static constexpr int kOffDirty = kOffSched + 32 * kSlots; // int [2 kSlots]
  static constexpr int kOffPtr = kOffDirty + 8 * kSlots;    // int [2][kPromptFew + 1]: items ahead of each prompt, offsets
  static constexpr int kSmem = kOffPtr + 8 * (kPromptFew + 1);
  static_assert(kSmem <= 232448, "shared memory");
  // Tensor memory: S of tile x (kThree: buffer x) at 128 x, O of tile x at kColO + kStepO x.
  static constexpr uint32_t kColO = kThree ? 384 : 256, kStepO = kThree ? 64 : 128;
  // The ring holds an item's blocks (nb) in the order of their use: K_0 .. K_(kAhead - 1),
  // then V_0, K_kAhead, V_1, K_(kAhead + 1), ...
  __device__ static __forceinline__ int key_entry(int nb, int i) {
    const int n0 = min(kAhead, nb);
    return i < n0 ? i : 2 * i - n0 + 1;
  }
  __device__ static __forceinline__ int value_entry(int nb, int j) {
    const int n0 = min(kAhead, nb);
    return j < nb - n0 ? n0 + 2 * j : nb + j;
  }
  // Blocks of `keys` keys; matrix instructions of P V (16 keys each) for block j of them
  // (values behind are not read).
  __host__ __device__ static constexpr int blocks(int keys) { return (keys + 127) >> 7; }
  __device__ static __forceinline__ int steps(int keys, int j) { return min(8, (keys - 128 * j + 15) >> 4); }
};

template <class C>
struct Smem {
  uint32_t base;
  __device__ __forceinline__ uint32_t bar(int i) const { return base + C::kOffBar + 8u * (uint32_t)i; }
  __device__ __forceinline__ uint32_t q(int buf, int x) const { return base + (uint32_t)((buf * 2 + x) * C::kTileBytes); }
  __device__ __forceinline__ uint32_t kv(uint32_t s) const { return base + C::kOffKV + s * (uint32_t)C::kTileBytes; }
};

struct Item {
  int it;        // < 0: no more
  int row0;      // first row of the prompt
  int len;       // its tokens
  int t0;        // first token of the item
  int unit;      // group of gp heads
};
// Keys that some row of tile x of an item attends (0: the tile has no token), and those
// of the item.
__device__ __forceinline__ int keys_of(const PromptParams& p, const Item& m, int x) {
  const int half = 128 >> p.gp_shift, first = m.t0 + x * half;
  if (first >= m.len) return 0;
  return p.causal ? min(m.len, first + half) : m.len;
}
__device__ __forceinline__ int item_keys(const PromptParams& p, const Item& m) {
  return p.causal ? min(m.len, m.t0 + (kPromptRows >> p.gp_shift)) : m.len;
}
// The first key that some row of the item does not attend.
__device__ __forceinline__ int masked_from(const PromptParams& p, const Item& m) {
  return p.causal ? min(m.t0 + 1, m.len) : m.len;
}

template <class C>
__device__ __forceinline__ Item take(const Smem<C>& sm, const uint8_t* smem, uint32_t t, bool arrives, bool warp_sync,
                                     const Watchdog& wd) {
  Item m{-2, 0, 0, 0, 0};
  const int slot = (int)(t % kSlots);
  bool ok = mbar_wait(sm.bar(C::kSchedFull + slot), (t / kSlots) & 1u, wd, kSiteSched);
  if (warp_sync) ok = __all_sync(0xffffffffu, ok);
  if (!ok) return m;
  const volatile int* e = reinterpret_cast<const volatile int*>(smem + C::kOffSched) + slot * 8;
  m.it = e[0];
  m.row0 = e[1];
  m.len = e[2];
  m.t0 = e[3];
  m.unit = e[4];
  if (warp_sync) __syncwarp();
  if (arrives) mbar_arrive(sm.bar(C::kSchedEmpty + slot));
  return m;
}

// Bounded wait of the teardown: goes by no abort flag.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, const Watchdog& wd) {
  volatile int no_abort = 0;
  Watchdog quick{&no_abort, wd.status, wd.detail, 100000000ll};
  mbar_wait(bar, parity, quick, kSiteDrain);
}

// ------------------------------------------------------------------ producer
// The prompt of item e of the line: the last that begins at or before it.
__device__ __forceinline__ int prompt_of(const int* ptr, int n, int e) {
  int lo = 0, hi = n;  // ptr[lo] <= e < ptr[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (ptr[mid] <= e) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The items ahead of each of up to kPromptFew prompts and the offsets, by one warp; returns how many
// there are (0 where the offsets do not ascend within [0, T]).
__device__ __forceinline__ int few_items(const PromptParams& p, int* ptr) {
  const int lane = threadIdx.x & 31, tq = kPromptRows >> p.gp_shift;
  int* off = ptr + kPromptFew + 1;
  bool bad = false;
  int base = 0;
  for (int i0 = 0; i0 < p.n; i0 += 32) {
    const int i = i0 + lane;
    int x = 0, a = 0, b = 0;
    if (i < p.n) {
      a = load_written(p.offsets + i);
      b = load_written(p.offsets + i + 1);
      if (a < 0 || b < a || b > p.T) bad = true;
      else x = (b - a + tq - 1) / tq;
    }
    int inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (i < p.n) {
      ptr[i] = base + inc - x;
      off[i] = a;
      off[i + 1] = b;  // (the next lane's own, the same)
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) ptr[p.n] = base;
  __syncwarp();
  bad = __any_sync(0xffffffffu, bad);
  if (blockIdx.x == 0 && lane == 0) {  // (what CTAs record of their waits has words of its own)
    p.control[kCtlStatus] = bad ? BSA_ERR_INVALID_ARG : BSA_OK;
    p.control[kCtlDetail] = bad ? kSitePromptOffsets : 0;
  }
  return bad ? 0 : base;
}

template <int D>
__device__ __noinline__ void producer(const PromptParams& p, uint8_t* smem, const Smem<Cfg<D>> sm, const Watchdog wd,
                                      int few) {
  using C = Cfg<D>;
  tma_prefetch_desc(&p.tmQ);
  tma_prefetch_desc(&p.tmK);
  tma_prefetch_desc(&p.tmV);
  const uint64_t pol_q = policy_evict_first(), pol_kv = policy_evict_last();
  const int units = p.Hq >> p.gp_shift, half = 128 >> p.gp_shift;
  const int tiles = p.few ? few : *reinterpret_cast<const volatile int32_t*>(p.control + kPromptCtlTiles);
  const int work = tiles * units;
  const int* ptr = reinterpret_cast<const int*>(smem + C::kOffPtr);
  uint32_t q_it = 0, kv_it = 0, block = 0;
  // Blocks that the entries of the ring belong to, four bits each, the oldest lowest: an
  // entry holds keys or values until both tiles are done with that block.
  uint64_t belongs = 0;
  static_assert(4 * C::kStages <= 64 && C::kBlocks <= 16, "four bits");
  bool ok = true;
  for (uint32_t t = 0; ok; ++t) {
    const int slot = (int)(t % kSlots);
    if (!mbar_wait(sm.bar(C::kSchedEmpty + slot), ((t / kSlots) & 1u) ^ 1u, wd, kSiteSched)) break;
    Item m{-1, 0, 0, 0, 0};
    // (few: there and back over the CTAs, so that the longest item's gets the shortest next)
    const int it = p.few ? (int)(t * gridDim.x + (t & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x))
                         : atomicAdd(p.control + kCtlWorkCounter, 1);
    if (it < work) {
      if (p.few) {
        const int x = tiles - 1 - it / units, i = prompt_of(ptr, p.n, x);
        const int* off = ptr + kPromptFew + 1;
        m = Item{it, off[i], off[i + 1] - off[i], (x - ptr[i]) * (2 * half), it % units};
      } else {
        const int4 e = load_written(p.tiles + it / units);
        m = Item{it, e.x, e.y, e.z, it % units};
      }
    }
    volatile int* e = reinterpret_cast<volatile int*>(smem + C::kOffSched) + slot * 8;
    e[0] = m.it;
    e[1] = m.row0;
    e[2] = m.len;
    e[3] = m.t0;
    e[4] = m.unit;
    mbar_arrive(sm.bar(C::kSchedFull + slot));
    if (m.it < 0) break;
    const int nb = C::blocks(item_keys(p, m));
    const bool two = m.t0 + half < m.len;
    const int h0 = m.unit << p.gp_shift, kvh = h0 / p.g;
    const int qb = (int)(q_it % C::kQBufs);
    if (!mbar_wait(sm.bar(C::kQEmpty + qb), ((q_it / C::kQBufs) & 1u) ^ 1u, wd, kSiteQEmpty)) break;
    const uint32_t qf = sm.bar(C::kQFull + qb);
    mbar_arrive_expect_tx(qf, two ? 2 * C::kTileBytes : C::kTileBytes);
    tma_load_4d(sm.q(qb, 0), &p.tmQ, 0, h0, m.row0 + m.t0, 0, qf, pol_q);
    if (two) tma_load_4d(sm.q(qb, 1), &p.tmQ, 0, h0, m.row0 + m.t0 + half, 0, qf, pol_q);
    ++q_it;
    for (int j = 0; j < 2 * nb; ++j) {
      const uint32_t s = kv_it % C::kStages;
      // Entry j: the first keys, then values and keys in turn, then the last values.
      const int n0 = min(C::kAhead, nb), e = j - n0, pairs = nb - n0;
      const bool value = e >= 2 * pairs || (e >= 0 && !(e & 1));
      const int of = e < 0 ? j : (e >= 2 * pairs ? e - pairs : (e & 1 ? n0 : 0) + (e >> 1));
      const uint32_t mine = block + (uint32_t)(value ? of : max(0, of - 1));
      if (kv_it >= (uint32_t)C::kStages) {
        // (blocks differ by less than 16: the low bits tell which of them it was)
        const uint32_t was = mine - ((mine - (uint32_t)(belongs & 15)) & 15u);
        if (!mbar_wait(sm.bar(C::kDone + (int)(was % C::kBlocks)), (was / C::kBlocks) & 1u, wd, kSiteKvEmpty)) {
          ok = false;
          break;
        }
      }
      belongs = (belongs >> 4 & ~(15ull << 4 * (C::kStages - 1))) | (uint64_t)(mine & 15u) << 4 * (C::kStages - 1);
      const uint32_t full = sm.bar(C::kFull + (int)s);
      mbar_arrive_expect_tx(full, C::kTileBytes);
      tma_load_4d(sm.kv(s), value ? &p.tmV : &p.tmK, 0, kvh, m.row0 + of * 128, 0, full, pol_kv);
      ++kv_it;
    }
    block += (uint32_t)nb;
  }
  volatile uint32_t* asked = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc) + 2;
  asked[0] = kv_it;
  asked[1] = q_it;
}
// Copies that were requested land before the shared memory goes away.  For the CTA's end:
// a wait may give up when the requests have long been made.
template <class C>
__device__ __noinline__ void drain_copies(const uint8_t* smem, const Smem<C> sm, const Watchdog wd) {
  const volatile uint32_t* asked = reinterpret_cast<const volatile uint32_t*>(smem + C::kOffMisc) + 2;
  const uint32_t kv_it = asked[0], q_it = asked[1];
  const uint32_t nk = kv_it < (uint32_t)C::kStages ? kv_it : (uint32_t)C::kStages;
  for (uint32_t t = kv_it - nk; t < kv_it; ++t)
    drain_wait(sm.bar(C::kFull + (int)(t % C::kStages)), (t / C::kStages) & 1u, wd);
  const uint32_t nq = q_it < (uint32_t)C::kQBufs ? q_it : (uint32_t)C::kQBufs;
  for (uint32_t t = q_it - nq; t < q_it; ++t)
    drain_wait(sm.bar(C::kQFull + (int)(t % C::kQBufs)), (t / C::kQBufs) & 1u, wd);
}

// ------------------------------------------------------------------ matrix products
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// What the issuing warps have in common.  A whole warp runs them, so that the descriptors
// are uniform values; one lane issues.
template <int D, bool FP16>
struct Products {
  using C = Cfg<D>;
  static constexpr uint32_t kIdescS = FP16 ? idesc_f16_f32(128, 128, false) : idesc_bf16_f32(128, 128, false);
  static constexpr uint32_t kIdescO = FP16 ? idesc_f16_f32(128, D, true) : idesc_bf16_f32(128, D, true);
  const Smem<C>& sm;
  const Watchdog& wd;
  bool ok = true;

  __device__ static __forceinline__ uint32_t stage(uint32_t r) { return r % (uint32_t)C::kStages; }
  __device__ __forceinline__ uint64_t q(int qb, int x) const { return smem_desc_sw128(sm.q(qb, x), 16, 1024); }
  __device__ __forceinline__ uint64_t k(uint32_t r) const { return smem_desc_sw128(sm.kv(stage(r)), 16, 1024); }
  __device__ __forceinline__ uint64_t v(uint32_t r) const { return smem_desc_sw128(sm.kv(stage(r)), C::kChunkBytes, 1024); }
  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, int site) {
    ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, wd, site));
    return ok;
  }
  // A wait that polls: a suspended try_wait is about 100 cycles later.  (64 or 256 polls
  // are the same within 1 %.)
  __device__ __forceinline__ bool wait_spinning(uint32_t bar, uint32_t parity, int site) {
    bool there = false;
    for (int i = 0; i < 256 && !there; ++i) there = mbar_test_wait(bar, parity);
    if (__all_sync(0xffffffffu, there)) return true;
    return wait(bar, parity, site);
  }
  __device__ __forceinline__ bool full(uint32_t r) {
    return wait(sm.bar(C::kFull + (int)stage(r)), (r / C::kStages) & 1u, kSiteKvFull);
  }
  __device__ __forceinline__ bool clean(uint32_t block) {
    return wait(sm.bar(C::kClean + (int)(block % C::kBlocks)), (block / C::kBlocks) & 1u, kSiteKvFull);
  }
  // By one lane:
  __device__ static __forceinline__ void scores(uint32_t scol, uint64_t qd, uint64_t kd) {
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint64_t off = (uint64_t)(((kk / 4) * C::kChunkBytes + (kk % 4) * 32) >> 4);
      mma_ss(scol, qd + off, kd + off, kIdescS, kk > 0 ? 1u : 0u);
    }
  }
  __device__ static __forceinline__ void values(uint32_t ocol, uint32_t pcol, uint64_t vd, int steps, bool more) {
    if (steps == 8) {
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mma_ts(ocol, pcol + 8u * (uint32_t)kk, vd + (uint64_t)(kk * (2048 >> 4)), kIdescO, (more || kk > 0) ? 1u : 0u);
    } else {
#pragma unroll 1
      for (int kk = 0; kk < steps; ++kk)
        mma_ts(ocol, pcol + 8u * (uint32_t)kk, vd + (uint64_t)(kk * (2048 >> 4)), kIdescO, (more || kk > 0) ? 1u : 0u);
    }
  }
  // Everything issued is done.
  __device__ __forceinline__ void drain(int x) {
    if (elect_one()) {
      mma_commit(sm.bar(C::kDrain + x));
      drain_wait(sm.bar(C::kDrain + x), 0, wd);
    }
    __syncwarp();
  }
};

// d = 128: the products of tile x, in turns with the other's.
template <int D, bool FP16>
__device__ __forceinline__ void issuer(const PromptParams& p, const uint8_t* smem, const Smem<Cfg<D>>& sm, uint32_t tmem_,
                                       const Watchdog& wd, int x) {
  using C = Cfg<D>;
  Products<D, FP16> w{sm, wd};
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_, 0);
  const uint32_t scol = tmem + 128u * (uint32_t)x, ocol = tmem + C::kColO + C::kStepO * (uint32_t)x;
  // Items, ring entries and blocks so far; blocks (P V) and items of tile x; turns.
  uint32_t q_it = 0, ring = 0, block = 0, pc = 0, oc = 0, turn = 0;
  while (w.ok) {
    const Item got = take<C>(sm, smem, q_it, (threadIdx.x & 31) == 0, true, wd);
    if (__shfl_sync(0xffffffffu, got.it, 0) < 0) break;
    const int nb = __shfl_sync(0xffffffffu, C::blocks(item_keys(p, got)), 0);
    const int keys = __shfl_sync(0xffffffffu, keys_of(p, got, x), 0), nx = C::blocks(keys);
    const int qb = (int)(q_it % C::kQBufs);
    const uint64_t qd = w.q(qb, x);
    // (Also where the tile has no token.  A wait by parity is one for this phase only if
    // the phase before it is known to be over: whoever waits on a barrier at all waits for
    // each of its phases, in order.)
    if (!w.wait(sm.bar(C::kQFull + qb), (q_it / C::kQBufs) & 1u, kSiteQFull) || !w.full(ring)) break;
    tc_fence_after();
    if (elect_one()) {
      if (nx > 0) {
        w.scores(scol, qd, w.k(ring));
        mma_commit(sm.bar(C::kSFull + x));
        if (nx == 1) mma_commit(sm.bar(C::kQEmpty + qb));
      } else {
        mbar_arrive(sm.bar(C::kQEmpty + qb));
      }
    }
    __syncwarp();
    for (int j = 0; j < nb; ++j, ++block, ++turn) {
      const uint32_t rv = ring + (uint32_t)C::value_entry(nb, j), rk = ring + (uint32_t)C::key_entry(nb, j + 1);
      const bool mine = j < nx, more = j + 1 < nx;
      // (What the products take, ahead of the waits: behind the last one nothing but them.)
      const uint64_t vd = w.v(rv), kd = w.k(rk);
      const uint32_t done = sm.bar(C::kDone + (int)(block % C::kBlocks));
      const int steps = C::steps(keys, j);
      if (!w.full(rv) || (j + 1 < nb && !w.full(rk)) || !w.clean(block)) break;
      if (mine && j == 0 && oc > 0 && !w.wait(sm.bar(C::kOFree + x), (oc - 1) & 1u, kSiteODone)) break;
      if (!w.wait(sm.bar(C::kTurn + x), (turn & 1u) ^ (x ? 0u : 1u), kSiteTurn)) break;
      if (mine) {  // (last: what the softmax has written is awaited most)
        if (!w.wait_spinning(sm.bar(C::kPFull + x), pc & 1u, kSitePFull)) break;
        ++pc;
      }
      tc_fence_after();
      if (elect_one()) {
        if (mine) w.values(ocol, scol, vd, steps, j > 0);
        if (more) w.scores(scol, qd, kd);
        mbar_arrive(sm.bar(C::kTurn + (x ^ 1)));
        if (mine) {
          mma_commit(sm.bar(more ? C::kSFull + x : C::kOFull + x));
          mma_commit(done);
          if (j + 2 == nx) mma_commit(sm.bar(C::kQEmpty + qb));
        } else {
          mbar_arrive(done);
        }
      }
      __syncwarp();
      if (mine && !more) ++oc;
    }
    ring += 2 * (uint32_t)nb;
    ++q_it;
  }
  w.drain(x);
}

// d = 64: steps go by blocks, of a block tile A's and then tile B's; step i's scores are in
// buffer i % 3.  One warp issues S, up to three steps ahead, one P V.
template <int D, bool FP16>
__device__ __forceinline__ void issuer_of_scores(const PromptParams& p, const uint8_t* smem, const Smem<Cfg<D>>& sm,
                                                 uint32_t tmem_, const Watchdog& wd) {
  using C = Cfg<D>;
  Products<D, FP16> w{sm, wd};
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_, 0);
  // Items, ring entries and blocks so far; the buffer, its phase, and whether it was used before.
  uint32_t q_it = 0, ring = 0, block = 0, s3 = 0, phase = 1;
  bool used = false;
  while (w.ok) {
    const Item got = take<C>(sm, smem, q_it, (threadIdx.x & 31) == 0, true, wd);
    if (__shfl_sync(0xffffffffu, got.it, 0) < 0) break;
    const int nb = __shfl_sync(0xffffffffu, C::blocks(item_keys(p, got)), 0);
    const int n0 = __shfl_sync(0xffffffffu, C::blocks(keys_of(p, got, 0)), 0);
    const int n1 = __shfl_sync(0xffffffffu, C::blocks(keys_of(p, got, 1)), 0);
    const int qb = (int)(q_it % C::kQBufs);
    const uint64_t q0 = w.q(qb, 0), q1 = w.q(qb, 1);
    if (!w.wait(sm.bar(C::kQFull + qb), (q_it / C::kQBufs) & 1u, kSiteQFull)) break;
    for (int j = 0; j < nb && w.ok; ++j, ++block) {
      const uint64_t kd = w.k(ring + (uint32_t)C::key_entry(nb, j));
      if (!w.wait(sm.bar(C::kKeysIn + (int)(block % C::kBlocks)), (block / C::kBlocks) & 1u, kSiteKvFull)) break;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (j >= (x ? n1 : n0)) continue;
        if (used && !w.wait_spinning(sm.bar(C::kFree + (int)s3), phase, kSitePFull)) break;
        tc_fence_after();
        if (elect_one()) {
          w.scores(tmem + 128u * s3, x ? q1 : q0, kd);
          mma_commit(sm.bar(C::kSFull + 3 * x + (int)s3));
        }
        __syncwarp();
        if (s3 == 2) {
          s3 = 0;
          phase ^= 1u;
          used = true;
        } else {
          ++s3;
        }
      }
      if (elect_one()) {
        if (j > 0) mma_commit(sm.bar(C::kDone + (int)((block - 1) % C::kBlocks)));
        if (j + 1 == nb) {
          mma_commit(sm.bar(C::kDone + (int)(block % C::kBlocks)));
          mma_commit(sm.bar(C::kQEmpty + qb));
        }
      }
      __syncwarp();
    }
    ring += 2 * (uint32_t)nb;
    ++q_it;
  }
  w.drain(0);
}

template <int D, bool FP16>
__device__ __forceinline__ void issuer_of_outputs(const PromptParams& p, const uint8_t* smem, const Smem<Cfg<D>>& sm,
                                                  uint32_t tmem_, const Watchdog& wd) {
  using C = Cfg<D>;
  Products<D, FP16> w{sm, wd};
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_, 0);
  // Items, ring entries and blocks so far; the buffer and its phase; the tiles' outputs.
  uint32_t t = 0, ring = 0, block = 0, p3 = 0, phase = 0, oc[2] = {0, 0};
  while (w.ok) {
    const Item got = take<C>(sm, smem, t, (threadIdx.x & 31) == 0, true, wd);
    if (__shfl_sync(0xffffffffu, got.it, 0) < 0) break;
    const int nb = __shfl_sync(0xffffffffu, C::blocks(item_keys(p, got)), 0);
    const int keys0 = __shfl_sync(0xffffffffu, keys_of(p, got, 0), 0);
    const int keys1 = __shfl_sync(0xffffffffu, keys_of(p, got, 1), 0);
    for (int j = 0; j < nb && w.ok; ++j, ++block) {
      const uint64_t vd = w.v(ring + (uint32_t)C::value_entry(nb, j));
      if (!w.clean(block)) break;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int keys = x ? keys1 : keys0, steps = C::steps(keys, j);
        if (steps <= 0) continue;
        const bool ends = 128 * (j + 1) >= keys;
        if (j == 0 && oc[x] > 0 && !w.wait(sm.bar(C::kOFree + x), (oc[x] - 1) & 1u, kSiteODone)) break;
        if (!w.wait_spinning(sm.bar(C::kPFull + (int)p3), phase, kSitePFull)) break;
        tc_fence_after();
        if (elect_one()) {
          w.values(tmem + C::kColO + C::kStepO * (uint32_t)x, tmem + 128u * p3, vd, steps, j > 0);
          mma_commit(sm.bar(C::kFree + (int)p3));
          if (ends) mma_commit(sm.bar(C::kOFull + x));
        }
        __syncwarp();
        if (ends) ++oc[x];
        if (p3 == 2) {
          p3 = 0;
          phase ^= 1u;
        } else {
          ++p3;
        }
      }
      if (elect_one()) mma_commit(sm.bar(C::kDone + (int)(block % C::kBlocks)));
      __syncwarp();
    }
    ring += 2 * (uint32_t)nb;
    ++t;
  }
  w.drain(1);
}

// ------------------------------------------------------------------ values
// 0xffff in the halves of w that are infinite or NaN.
template <bool FP16>
__device__ __forceinline__ uint32_t no_numbers(uint32_t w) {
  constexpr uint32_t kExp = FP16 ? 0x7c007c00u : 0x7f807f80u;
  return __vcmpeq2(w & kExp, kExp);
}

template <int D, bool FP16>
__device__ __forceinline__ void scanner(const PromptParams& p, uint8_t* smem, const Smem<Cfg<D>>& sm, const Watchdog& wd,
                                        int lane) {
  using C = Cfg<D>;
  volatile int* dirty = reinterpret_cast<volatile int*>(smem + C::kOffDirty);
  uint32_t ring = 0, block = 0;
  for (uint32_t t = 0;; ++t) {
    const Item m = take<C>(sm, smem, t, lane == 0, true, wd);
    if (m.it < 0) return;
    const int keys = item_keys(p, m), nb = C::blocks(keys), from = masked_from(p, m);
    if (lane == 0) dirty[t % (2 * kSlots)] = 0;
    auto full = [&](uint32_t r) {
      return __all_sync(0xffffffffu,
                        mbar_wait(sm.bar(C::kFull + (int)(r % C::kStages)), (r / C::kStages) & 1u, wd, kSiteKvFull));
    };
    // (The keys, too: a stage may alternate between keys and values, and a wait that
    // skipped a phase would pass before the values are there.  Each wait comes ahead of the
    // arrival that the stage's next use goes by.)
    // kThree: the issuing warps go by this warp's waits, two arrivals a block.
    const uint32_t block0 = block;
    auto keys_in = [&](int j) {
      if (!full(ring + (uint32_t)C::key_entry(nb, j))) return false;
      if (C::kThree && lane == 0) mbar_arrive(sm.bar(C::kKeysIn + (int)((block0 + (uint32_t)j) % C::kBlocks)));
      return true;
    };
    for (int j = 0; j < min(C::kAhead, nb); ++j)
      if (!keys_in(j)) return;
    for (int j = 0; j < nb; ++j, ++block) {
      const uint32_t r = ring + (uint32_t)C::value_entry(nb, j), s = r % C::kStages;
      if (!full(r)) return;
      if ((j + 1) * 128 > from) {
        // Of the rows that are read, those that every row of the item attends can stay.
        bool here = false;
        const int lo = max(0, from - 128 * j), end = 16 * C::steps(keys, j);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const uint32_t at = sm.kv(s) + (uint32_t)(c * C::kChunkBytes + lane * 16);
#pragma unroll 4
          for (int q = (lo & ~3) * 128; q < end * 128; q += 512) {
            const uint4 x = ld_shared_v4(at + q);
            const uint32_t a = no_numbers<FP16>(x.x), b = no_numbers<FP16>(x.y), e = no_numbers<FP16>(x.z),
                           f = no_numbers<FP16>(x.w);
            if (a | b | e | f) {
              st_shared_v4(at + q, x.x & ~a, x.y & ~b, x.z & ~e, x.w & ~f);
              here = true;
            }
          }
        }
        if (__any_sync(0xffffffffu, here)) {
          fence_proxy_async_smem();  // the product reads what was written
          if (lane == 0) dirty[t % (2 * kSlots)] = 1;
        }
      }
      if (!C::kThree && j + C::kAhead < nb && !keys_in(j + C::kAhead)) return;
      __syncwarp();
      if (lane == 0) mbar_arrive(sm.bar(C::kClean + (int)(block % C::kBlocks)));
      if (C::kThree && j + C::kAhead < nb && !keys_in(j + C::kAhead)) return;
    }
    ring += 2 * (uint32_t)nb;
  }
}

// ------------------------------------------------------------------ softmax
// Values that were replaced by 0, to the rows of the item that attend them: an
// infinity or NaN among a row's values is one in its output, whatever its weight.  A
// warp mends its own 32 rows (of tokens tok0 .. ), a lane D / 32 columns.
template <int D, bool FP16>
__device__ __noinline__ void add_no_numbers(const PromptParams& p, const Item m, int tok0, int row0) {
  constexpr int kCols = D / 32;
  constexpr uint32_t kExp = FP16 ? 0x7c00u : 0x7f80u;
  const int c0 = (int)(threadIdx.x & 31) * kCols;
  const int h0 = m.unit << p.gp_shift, gp = 1 << p.gp_shift, rows = gp < 32 ? gp : 32;
  const int end = min(m.len, tok0 + (32 >> p.gp_shift)), from = masked_from(p, m) & ~127;
  const uint16_t* v = p.v + (long long)(h0 / p.g) * p.v_sh + c0;
  uint32_t seen[kCols];  // +inf 1, -inf 2, NaN 4
#pragma unroll
  for (int c = 0; c < kCols; ++c) seen[c] = 0u;
  auto what = [](uint32_t w) -> uint32_t {
    return (w & kExp) != kExp ? 0u : ((w & 0x7fffu) == kExp ? 1u << (w >> 15) : 4u);
  };
  auto look = [&](int t) {
#pragma unroll
    for (int c = 0; c < kCols; ++c) seen[c] |= what(load_written(v + (long long)(m.row0 + t) * p.v_st + c));
  };
  auto add = [&](int t) {
    for (int h = 0; h < rows; ++h) {
      uint16_t* o = p.o + (long long)(m.row0 + t) * p.o_st + (long long)(h0 + (row0 & (gp - 1)) + h) * p.o_sh + c0;
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        if (!seen[c]) continue;
        const uint32_t s = seen[c] | what(o[c]);
        o[c] = (uint16_t)(s == 1u ? kExp : (s == 2u ? kExp | 0x8000u : 0x7fffu));
      }
    }
  };
  __syncwarp();  // the rows are written
  if (p.causal) {
    for (int t = from; t < end; ++t) {
      look(t);
      if (t >= tok0) add(t);
    }
  } else {
    for (int t = from; t < m.len; ++t) look(t);
    for (int t = tok0; t < end; ++t) add(t);
  }
  __syncwarp();
}

template <int D, bool FP16>
__device__ __forceinline__ void softmax(const PromptParams& p, uint8_t* smem, const Smem<Cfg<D>>& sm, uint32_t tmem,
                                        const Watchdog& wd) {
  using C = Cfg<D>;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int x = (warp - 4) >> 2, quad = warp & 3;
  const int row = quad * 32 + lane;
  const uint32_t tl = (uint32_t)(quad * 32) << 16;
  const uint32_t ocol = tmem + tl + C::kColO + C::kStepO * (uint32_t)x;
  const int half = 128 >> p.gp_shift, gp = 1 << p.gp_shift;
  const volatile int* dirty = reinterpret_cast<const volatile int*>(smem + C::kOffDirty);
  const float sl2 = p.scale_log2;
  const uint64_t sl2x2 = f2_make(sl2, sl2);
  // Blocks and outputs of this tile; kThree: steps of both ahead of the item's, phases of the
  // buffers' next scores.
  uint32_t sc = 0, oc = 0, steps = 0, phases = 0;
  for (uint32_t t = 0;; ++t) {
    const Item m = take<C>(sm, smem, t, lane == 0, true, wd);
    if (m.it < 0) return;
    const int n0 = C::blocks(keys_of(p, m, 0)), n1 = C::blocks(keys_of(p, m, 1)), n = x ? n1 : n0;
    const uint32_t base = steps;
    steps += (uint32_t)(n0 + n1);
    if (n == 0) continue;
    const int first = m.t0 + x * half, tok = first + (row >> p.gp_shift);
    // Last key of this row, and the key below which all rows of the tile attend.
    const int lim = p.causal ? min(tok, m.len - 1) : m.len - 1;
    const int lim_warp = p.causal ? min(first + ((quad * 32) >> p.gp_shift), m.len - 1) : m.len - 1;  // its first row's
    const int whole = p.causal ? min(first + 1, m.len) : m.len;
    // Rows of the warp that are the prompt's: those behind its end may hold anything, and move no
    // reference.
    const uint32_t own_rows = __ballot_sync(0xffffffffu, tok < m.len);
    // Weights are kept at 2^shift of their size and, in a block, summed to no more than `most`.
    const int log_n = 32 - __clz(n);
    const float shift = FP16 ? 6.f : (float)(-kMostLog - log_n);
    const float most = FP16 ? (float)(1 << kMostLog) : __uint_as_float((uint32_t)(127 - log_n) << 23);
    float m_ref = -INFINITY, l = 0.f;
    for (int j = 0; j < n; ++j) {
      // Where its scores are, and the phase that says so.
      int buf = x, full = C::kSFull + x;
      uint32_t parity = sc & 1u;
      if constexpr (C::kThree) {
        buf = (int)((base + (uint32_t)(min(n0, j + x) + min(n1, j))) % 3u);
        full = C::kSFull + 3 * x + buf;
        parity = phases >> buf & 1u;
        phases ^= 1u << buf;
      }
      if (!__all_sync(0xffffffffu, mbar_wait(sm.bar(full), parity, wd, kSiteSFull))) return;
      const uint32_t scol = tmem + tl + 128u * (uint32_t)buf;
      tc_fence_after();
      uint32_t v[128], pk[64];
      float sum, factor = 1.f;
      // The first block sets the reference, m.  Later ones are weighed against it as it is:
      // only where a row's weights come to more than `most` has a score passed it by so much
      // that it has to move, and the scores (the weights are not stored yet) are read again.
      for (bool move = j == 0;; move = true) {
        tmem_ld32_at<0>(scol, v);
        tmem_ld32_at<32>(scol + 32u, v);
        tmem_ld32_at<64>(scol + 64u, v);
        tmem_ld32_at<96>(scol + 96u, v);
        tmem_wait_ld();
        if ((j + 1) * 128 > whole) {
          const int rel = lim - j * 128;  // the last element that counts
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (lim_warp >= j * 128 + 32 * c + 31) continue;  // all of the warp's rows attend these
#pragma unroll
            for (int e = 32 * c; e < 32 * c + 32; ++e)
              if (e > rel) v[e] = __float_as_uint(-INFINITY);
          }
        }
        if (move) {
          float mx4[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) mx4[c] = fmaxf(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1]));
#pragma unroll
          for (int e = 8; e < 128; e += 8) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              mx4[c] = fmax3(mx4[c], __uint_as_float(v[e + 2 * c]), __uint_as_float(v[e + 2 * c + 1]));
          }
          const float m_new = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sl2;
          if (j == 0) {
            m_ref = m_new;
          } else {
            if (m_new > m_ref) {
              factor = ex2_approx(m_ref - m_new);
              m_ref = m_new;
            }
            // The products before this block's have to be done with O.  One buffer a tile: this
            // block's scores have arrived, so they are.
            if constexpr (C::kThree) {
              const uint32_t i = base + (uint32_t)(min(n0, j - 1 + x) + min(n1, j - 1));
              if (!__all_sync(0xffffffffu, mbar_wait(sm.bar(C::kFree + (int)(i % 3u)), i / 3u & 1u, wd, kSiteODone))) return;
            }
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(ocol + 32u * (uint32_t)c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
              tmem_st32(ocol + 32u * (uint32_t)c, o);
            }
          }
        }
        const float mb = shift - (m_ref == -INFINITY ? 0.f : m_ref);
        const uint64_t mbx2 = f2_make(mb, mb);
        uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int e = 0; e < 64; ++e) {
          float x0, x1;
          f2_split(ffma2(f2_make(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), sl2x2, mbx2), x0, x1);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          pk[e] = FP16 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
          acc2[e & 3] = fadd2(acc2[e & 3], f2_make(p0, p1));
        }
        float s0, s1;
        f2_split(fadd2(fadd2(acc2[0], acc2[1]), fadd2(acc2[2], acc2[3])), s0, s1);
        sum = s0 + s1;
        if (move || !(__ballot_sync(0xffffffffu, sum > most || m_ref == -INFINITY) & own_rows)) break;
      }
      tmem_st32_at<0>(scol, pk);
      tmem_st32_at<32>(scol + 32u, pk);
      l = l * factor + sum;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sm.bar(C::kPFull + buf));
      ++sc;
    }
    // ------------------------------------------------------------ epilogue
    if (!__all_sync(0xffffffffu, mbar_wait(sm.bar(C::kOFull + x), oc & 1u, wd, kSiteODone))) return;
    ++oc;
    tc_fence_after();
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // (NaN stays)
    const int head = (m.unit << p.gp_shift) + (row & (gp - 1));
    const bool real = tok < m.len;
    uint16_t* out = p.o + (long long)(m.row0 + tok) * p.o_st + (long long)head * p.o_sh;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint32_t o[32], pk[16];
      tmem_ld32(ocol + 32u * (uint32_t)c, o);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float a = __uint_as_float(o[2 * e]) * inv, b = __uint_as_float(o[2 * e + 1]) * inv;
        pk[e] = FP16 ? pack_f16x2(a, b) : pack_bf16x2(a, b);
      }
      if (real && p.o_v8) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t w8[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w8[e] = pk[8 * q + e];
          st_global_v8(out + 32 * c + 16 * q, w8);
        }
      } else if (real) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint4*>(out + 32 * c + 8 * q) = make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
      }
      __syncwarp();
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(sm.bar(C::kOFree + x));
    if (real && p.lse)
      p.lse[(long long)(m.row0 + tok) * p.Hq + head] =
          l == 0.f ? -INFINITY : (m_ref - shift + __log2f(l)) * 0.69314718055994531f;
    if (dirty[t % (2 * kSlots)]) add_no_numbers<D, FP16>(p, m, first + ((quad * 32) >> p.gp_shift), quad * 32);
  }
}

template <int D, bool FP16>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ PromptParams p) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Smem<C> sm{smem_u32(smem)};
  volatile uint32_t* tmem_holder = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  // (Status words in shared memory until the end: pointers of the CTA's own into global memory
  // are registers that every wait would hold, d = 64: 256 -> 264 us for the six documents.)
  int32_t* found = reinterpret_cast<int32_t*>(smem + C::kOffMisc + 16);
  const Watchdog wd{abort_flag, found, found + 1, p.watchdog_ns};
  next_may_launch();
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    tmem_holder[2] = tmem_holder[3] = 0u;
    found[0] = BSA_OK;
    found[1] = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(sm.bar(C::kQFull + i), 1);
      mbar_init(sm.bar(C::kQEmpty + i), C::kThree ? 1 : 2);
      mbar_init(sm.bar(C::kTurn + i), 1);
      mbar_init(sm.bar(C::kDrain + i), 1);
    }
    for (int i = C::kSFull; i < C::kPFull; ++i) mbar_init(sm.bar(i), 1);
    for (int i = C::kPFull; i < C::kFree; ++i) mbar_init(sm.bar(i), 4);
    for (int i = C::kFree; i < C::kOFree; ++i) mbar_init(sm.bar(i), 1);
    for (int i = C::kOFree; i < C::kTurn; ++i) mbar_init(sm.bar(i), 4);
    for (int i = 0; i < C::kStages; ++i) mbar_init(sm.bar(C::kFull + i), 1);
    for (int i = 0; i < C::kBlocks; ++i) {
      mbar_init(sm.bar(C::kClean + i), 1);
      mbar_init(sm.bar(C::kDone + i), 2);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(sm.bar(C::kSchedFull + i), 1);
      mbar_init(sm.bar(C::kSchedEmpty + i), kConsumers);
    }
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 2) {
    tmem_alloc(sm.base + C::kOffMisc, 512);
    tmem_relinquish();
  }
  wait_for_previous();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  if (threadIdx.x == 0 && (sm.base & 1023u)) record_failure(wd, BSA_ERR_CUDA, 0);  // the swizzle's layout needs it
  __syncthreads();
  if (warp >= 4) {
    regs_inc<kRegsSoftmax>();
    if (!*abort_flag) softmax<D, FP16>(p, smem, sm, tmem, wd);
  } else {
    regs_dec<kRegsControl>();
    if (!*abort_flag) {
      if (warp == 3) scanner<D, FP16>(p, smem, sm, wd, lane);
      else if (warp >= 1) {
        if constexpr (!C::kThree) issuer<D, FP16>(p, smem, sm, tmem, wd, warp - 1);
        else if (warp == 1) issuer_of_scores<D, FP16>(p, smem, sm, tmem, wd);
        else issuer_of_outputs<D, FP16>(p, smem, sm, tmem, wd);
      } else {
        const int few = p.few ? few_items(p, reinterpret_cast<int*>(smem + C::kOffPtr)) : 0;
        if (lane == 0) producer<D>(p, smem, sm, wd, few);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {
    if (*abort_flag) drain_copies<C>(smem, sm, wd);
    int32_t* own = p.control + kPromptCtlOwn + 2 * blockIdx.x;
    own[0] = *const_cast<volatile int32_t*>(found);
    own[1] = *const_cast<volatile int32_t*>(found + 1);
    if (blockIdx.x == 0) p.control[kPromptCtlCtas] = (int)gridDim.x;
  }
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ schedule
// The work items of all prompts, those with the most key blocks first (a counting
// sort by blocks).  Offsets that do not ascend within [0, T] leave no item: prompts
// would overlap.
constexpr int kScheduleThreads = 1024;
constexpr int kBuckets = 1024;

__global__ void __launch_bounds__(kScheduleThreads) prompt_schedule_kernel(const __grid_constant__ PromptParams p) {
  __shared__ int s_warp[32];
  __shared__ int s_bucket[kBuckets];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  next_may_launch();
  wait_for_previous();
  const int tq = kPromptRows >> p.gp_shift;  // tokens of an item
  // Exclusive scan of one int per thread; returns the total too.
  auto scan = [&](int x, int& total) {
    int inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < 32; ++w) {
      const int y = s_warp[w];
      before += w < warp ? y : 0;
      all += y;
    }
    __syncthreads();
    total = all;
    return before + inc - x;
  };
  bool bad = false;
  int base = 0, longest = 0;
  for (int i0 = 0; i0 < p.n; i0 += kScheduleThreads) {
    const int i = i0 + tid;
    int tiles = 0;
    if (i < p.n) {
      const int a = load_written(p.offsets + i), b = load_written(p.offsets + i + 1);
      if (a < 0 || b < a || b > p.T) {
        bad = true;
      } else {
        tiles = (b - a + tq - 1) / tq;
        longest = max(longest, b - a);
      }
    }
    int total;
    const int at = scan(tiles, total);
    if (i < p.n) p.tile_ptr[i] = base + at;
    base += total;
  }
  s_bucket[tid] = 0;
  bad = __syncthreads_or(bad);
  if (tid == 0) {
    p.control[kCtlWorkCounter] = 0;
    p.control[kCtlStatus] = bad ? BSA_ERR_INVALID_ARG : BSA_OK;
    p.control[kCtlDetail] = bad ? kSitePromptOffsets : 0;
    p.control[kPromptCtlTiles] = bad ? 0 : base;
    p.tile_ptr[p.n] = base;
  }
  if (bad) return;
  // Blocks of a bucket: so many that the longest prompt's fit.
#pragma unroll
  for (int o = 16; o; o >>= 1) longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
  if (lane == 0) s_warp[warp] = longest;
  __syncthreads();
  for (int w = 0; w < 32; ++w) longest = max(longest, s_warp[w]);
  int shift = 0;
  while (((longest + 127) >> 7) >> shift >= kBuckets) ++shift;
  // Item e of the line, and its bucket.
  auto item = [&](int e, int& bucket) {
    const int lo = prompt_of(p.tile_ptr, p.n, e);
    const int a = load_written(p.offsets + lo), len = load_written(p.offsets + lo + 1) - a;
    const int t0 = (e - p.tile_ptr[lo]) * tq;
    const int keys = p.causal ? min(len, t0 + tq) : len;
    bucket = kBuckets - 1 - (((keys + 127) >> 7) >> shift);
    return make_int4(a, len, t0, 0);
  };
  for (int e = tid; e < base; e += kScheduleThreads) {
    int b;
    item(e, b);
    atomicAdd(&s_bucket[b], 1);
  }
  __syncthreads();
  int total;
  const int at = scan(s_bucket[tid], total);
  s_bucket[tid] = at;
  __syncthreads();
  for (int e = tid; e < base; e += kScheduleThreads) {
    int b;
    const int4 x = item(e, b);
    p.tiles[atomicAdd(&s_bucket[b], 1)] = x;
  }
}

template <int D, bool FP16>
cudaError_t launch(const PromptParams& p, int sms, cudaStream_t s) {
  constexpr int kSmem = Cfg<D>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(prompt_kernel<D, FP16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  long long ctas = ((long long)p.T / (kPromptRows >> p.gp_shift) + p.n) * (p.Hq >> p.gp_shift);
  if (ctas > sms) ctas = sms;
  if (ctas > kPromptMaxCtas) ctas = kPromptMaxCtas;
  return launch_after(prompt_kernel<D, FP16>, dim3((unsigned)ctas), dim3(kThreads), kSmem, s, p);
}

}  // namespace

cudaError_t launch_prompt(const PromptParams& p, int d, int sms, cudaStream_t s) {
  if (!p.few) {
    const cudaError_t e = launch_after(prompt_schedule_kernel, dim3(1), dim3(kScheduleThreads), 0, s, p);
    if (e != cudaSuccess) return e;
  }
  if (d == 64) return p.fp16 ? launch<64, true>(p, sms, s) : launch<64, false>(p, sms, s);
  return p.fp16 ? launch<128, true>(p, sms, s) : launch<128, false>(p, sms, s);
}

}  // namespace bsa
