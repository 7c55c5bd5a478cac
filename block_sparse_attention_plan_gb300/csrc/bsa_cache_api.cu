// Host side of the 8-bit cache's entry points: argument checks, workspace
// layout and launches.  See include/bsa.h for the contract of each.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "bsa_cache.h"
#include "bsa_internal.h"

using namespace bsa;

namespace {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool pow2_between(int x, int lo, int hi) { return x >= lo && x <= hi && (x & (x - 1)) == 0; }

// The struct's own checks; *out gets the kernels' view.
bsa_status check_cache(const bsa_cache* c, CacheDev* out) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !c->block_table || !c->seq_lens || !c->page_refs ||
      !c->control)
    return BSA_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
      !aligned(c->block_table, 4) || !aligned(c->seq_lens, 4) || !aligned(c->page_refs, 4) || !aligned(c->control, 4))
    return BSA_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->Hkv < 1 || c->max_seqs < 1 || c->max_pages < 1) return BSA_ERR_INVALID_ARG;
  if (c->kind != BSA_CACHE_E4M3 && c->kind != BSA_CACHE_INT8) return BSA_ERR_UNSUPPORTED;
  if (c->d != 64 && c->d != 128) return BSA_ERR_UNSUPPORTED;
  if (!pow2_between(c->page_size, 16, 256) || !pow2_between(c->scale_block, 16, c->page_size))
    return BSA_ERR_UNSUPPORTED;
  // Pool rows and positions in a sequence are 32-bit; control lists too.
  if ((long long)c->num_pages * c->Hkv > ((1ll << 31) - 1) / c->page_size) return BSA_ERR_UNSUPPORTED;
  if ((long long)c->max_pages * c->page_size > (1ll << 30)) return BSA_ERR_UNSUPPORTED;
  out->k = static_cast<uint8_t*>(c->k);
  out->v = static_cast<uint8_t*>(c->v);
  out->ks = c->k_scale;
  out->vs = c->v_scale;
  out->table = c->block_table;
  out->lens = c->seq_lens;
  out->refs = c->page_refs;
  out->control = c->control;
  out->kind = c->kind;
  out->num_pages = c->num_pages;
  out->Hkv = c->Hkv;
  out->page = c->page_size;
  out->d = c->d;
  out->sb = c->scale_block;
  out->max_seqs = c->max_seqs;
  out->max_pages = c->max_pages;
  return BSA_OK;
}

// A [batch][heads][tokens][d] tensor: `heads` and `tokens` > 1 need their strides.
bool good_rows(const bsa_rows* r) {
  return r && r->data && aligned(r->data, 16) && r->stride_b >= 0 && r->stride_h >= 0 && r->stride_t >= 0 &&
         r->stride_b % 8 == 0 && r->stride_h % 8 == 0 && r->stride_t % 8 == 0;
}
CacheRows rows_of(const bsa_rows* r) {
  return CacheRows{static_cast<const uint16_t*>(r->data), r->stride_b, r->stride_h, r->stride_t};
}

bsa_status sms_of(int dev, int* sms) {
  return cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

inline bool list_ok(const int32_t* p) { return !p || aligned(p, 4); }

// Workspace of an attention call (byte offsets).
struct AttnLayout {
  int rows_cap, max_tiles;
  size_t off_part, off_desc, off_counts, off_list, bytes;
};
bsa_status attn_layout(const CacheDev& c, int B, int Hq, int nq, int NKB, int bk, bool masked, AttnLayout* out) {
  if (B < 1 || Hq < 1 || nq < 1 || Hq % c.Hkv) return BSA_ERR_INVALID_ARG;
  const long long M = (long long)(Hq / c.Hkv) * nq;
  const int tile = cache_tile_keys(c.d);
  long long tiles = ((long long)c.max_pages * c.page + tile - 1) / tile;
  if (masked) {
    if (bk != 32 && bk != 64 && bk != 128 && bk != 256) return BSA_ERR_UNSUPPORTED;
    if (NKB < 1) return BSA_ERR_INVALID_ARG;
    const long long mt = ((long long)NKB * bk + tile - 1) / tile;
    if (mt < tiles) tiles = mt;
  }
  const long long groups = (M + kCacheUnitRows - 1) / kCacheUnitRows;
  if (M >= (1ll << 30) || (long long)B * Hq * nq >= (1ll << 31) ||
      (double)B * c.Hkv * groups * (tiles + kCacheUnitHead) >= 2147483648.0 || (long long)B * c.Hkv > (1ll << 24))
    return BSA_ERR_UNSUPPORTED;
  AttnLayout l;
  l.rows_cap = (int)(M < kCacheUnitRows ? M : kCacheUnitRows);
  l.max_tiles = (int)tiles;
  size_t off = 0;
  l.off_part = off;   off = align256(off + 4ull * 2 * kCacheMaxGrid * l.rows_cap * (c.d + 2));
  l.off_desc = off;   off = align256(off + 16ull * kCacheMaxGrid);
  l.off_counts = off; off = align256(off + (masked ? 4ull * B * c.Hkv : 0));
  l.off_list = off;   off = align256(off + (masked ? 4ull * B * c.Hkv * (uint64_t)tiles : 0));
  l.bytes = off;
  *out = l;
  return BSA_OK;
}

}  // namespace

extern "C" {

size_t bsa_cache_control_bytes(int num_pages) { return num_pages < 1 ? 0 : 4 * cache_control_ints(num_pages); }

bsa_status bsa_cache_init(const bsa_cache* cache, void* stream) {
  CacheDev c;
  bsa_status st = check_cache(cache, &c);
  if (st != BSA_OK) return st;
  if ((st = check_device(nullptr)) != BSA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(c.table, 0xff, 4ull * c.max_seqs * c.max_pages, s) != cudaSuccess ||
      cudaMemsetAsync(c.lens, 0, 4ull * c.max_seqs, s) != cudaSuccess ||
      cudaMemsetAsync(c.refs, 0, 4ull * c.num_pages, s) != cudaSuccess ||
      cudaMemsetAsync(c.control, 0, 4ull * kCacheScratch, s) != cudaSuccess)
    return BSA_ERR_CUDA;
  return BSA_OK;
}

bsa_status bsa_cache_status(const bsa_cache* cache, void* stream, int32_t* detail) {
  CacheDev c;
  bsa_status st = check_cache(cache, &c);
  if (st != BSA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t word[2] = {0, 0};
  if (cudaMemcpyAsync(word, c.control, sizeof(word), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaMemsetAsync(c.control, 0, sizeof(word), s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
    return BSA_ERR_CUDA;
  if (detail) *detail = word[1];
  return static_cast<bsa_status>(word[0]);
}

bsa_status bsa_cache_resize(const bsa_cache* cache, const int32_t* seqs, const int32_t* new_lens, int n,
                            void* stream) {
  CacheDev c;
  bsa_status st = check_cache(cache, &c);
  if (st != BSA_OK) return st;
  if (n < 1 || !list_ok(seqs) || !list_ok(new_lens) || (!seqs && n > c.max_seqs)) return BSA_ERR_INVALID_ARG;
  if (n > kCacheListMax && (seqs || new_lens)) return BSA_ERR_UNSUPPORTED;
  if ((st = check_device(nullptr)) != BSA_OK) return st;
  return launch_cache_resize(c, seqs, new_lens, n, static_cast<cudaStream_t>(stream)) == cudaSuccess ? BSA_OK
                                                                                                     : BSA_ERR_CUDA;
}

bsa_status bsa_cache_fork(const bsa_cache* cache, const int32_t* src, const int32_t* dst, int n, void* stream) {
  CacheDev c;
  bsa_status st = check_cache(cache, &c);
  if (st != BSA_OK) return st;
  if (n < 1 || !src || !dst || !list_ok(src) || !list_ok(dst)) return BSA_ERR_INVALID_ARG;
  if (n > kCacheListMax) return BSA_ERR_UNSUPPORTED;
  if ((st = check_device(nullptr)) != BSA_OK) return st;
  return launch_cache_fork(c, src, dst, n, static_cast<cudaStream_t>(stream)) == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

bsa_status bsa_cache_compact(const bsa_cache* cache, void* stream) {
  CacheDev c;
  bsa_status st = check_cache(cache, &c);
  if (st != BSA_OK) return st;
  int dev = 0, sms = 0;
  if ((st = check_device(&dev)) != BSA_OK || (st = sms_of(dev, &sms)) != BSA_OK) return st;
  return launch_cache_compact(c, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

bsa_status bsa_cache_copy_pages(const bsa_cache* dst, const bsa_cache* src, const int32_t* dst_pages,
                                const int32_t* src_pages, int n, void* stream) {
  CacheDev d, s;
  bsa_status st = check_cache(dst, &d);
  if (st != BSA_OK || (st = check_cache(src, &s)) != BSA_OK) return st;
  if (n < 1 || n > d.num_pages || !dst_pages || !src_pages || !list_ok(dst_pages) || !list_ok(src_pages))
    return BSA_ERR_INVALID_ARG;
  if (d.kind != s.kind || d.Hkv != s.Hkv || d.page != s.page || d.d != s.d || d.sb != s.sb) return BSA_ERR_INVALID_ARG;
  if ((d.k == s.k) != (d.v == s.v) || (d.k == s.k && d.num_pages != s.num_pages)) return BSA_ERR_INVALID_ARG;
  if ((st = check_device(nullptr)) != BSA_OK) return st;
  return launch_cache_copy(d, s, dst_pages, src_pages, n, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? BSA_OK
             : BSA_ERR_CUDA;
}

bsa_status bsa_cache_append(const bsa_cache* cache, const bsa_rows* k, const bsa_rows* v, int dtype,
                            const int32_t* seqs, const int32_t* counts, const int32_t* start, int n, int T,
                            void* stream) {
  CacheAppendParams p;
  bsa_status st = check_cache(cache, &p.c);
  if (st != BSA_OK) return st;
  if (n < 1 || T < 1 || !good_rows(k) || !good_rows(v)) return BSA_ERR_INVALID_ARG;
  if (!list_ok(seqs) || !list_ok(counts) || !list_ok(start) || (!seqs && n > p.c.max_seqs)) return BSA_ERR_INVALID_ARG;
  if (dtype != BSA_BF16 && dtype != BSA_FP16) return BSA_ERR_UNSUPPORTED;
  if ((long long)T > (long long)p.c.max_pages * p.c.page) return BSA_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  if ((st = check_device(&dev)) != BSA_OK || (st = sms_of(dev, &sms)) != BSA_OK) return st;
  p.k = rows_of(k);
  p.v = rows_of(v);
  p.fp16 = dtype == BSA_FP16;
  p.n = n;
  p.T = T;
  p.blocks = (T + p.c.sb - 2) / p.c.sb + 1;
  p.seqs = seqs;
  p.counts = counts;
  p.start = start;
  return launch_cache_append(p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

size_t bsa_cache_attention_workspace_bytes(const bsa_cache* cache, int B, int Hq, int nq, int NKB, int bk) {
  CacheDev c;
  AttnLayout l;
  if (check_cache(cache, &c) != BSA_OK || attn_layout(c, B, Hq, nq, NKB, bk, NKB > 0, &l) != BSA_OK) return 0;
  return l.bytes;
}

bsa_status bsa_cache_attention(const bsa_cache* cache, const bsa_rows* q, const bsa_rows* o, float* LSE, int dtype,
                               const int32_t* seqs, const uint8_t* mask, int NKB, int bk, int B, int Hq, int nq,
                               int flags, float scale, void* workspace, size_t workspace_bytes, void* stream) {
  CacheAttnParams p;
  std::memset(&p, 0, sizeof(p));
  bsa_status st = check_cache(cache, &p.c);
  if (st != BSA_OK) return st;
  if (!good_rows(q) || !good_rows(o) || !workspace || !aligned(workspace, 16) || !aligned(LSE, 4) || !list_ok(seqs))
    return BSA_ERR_INVALID_ARG;
  if (flags & ~BSA_CACHE_CAUSAL) return BSA_ERR_INVALID_ARG;
  if (dtype != BSA_BF16 && dtype != BSA_FP16) return BSA_ERR_UNSUPPORTED;
  if (!(scale == scale) || std::isinf(scale)) return BSA_ERR_INVALID_ARG;
  AttnLayout l;
  if ((st = attn_layout(p.c, B, Hq, nq, NKB, bk, mask != nullptr, &l)) != BSA_OK) return st;
  if (!seqs && B > p.c.max_seqs) return BSA_ERR_INVALID_ARG;
  // Rows that several CTAs write must not be one.
  if ((B > 1 && !o->stride_b) || (Hq > 1 && !o->stride_h) || (nq > 1 && !o->stride_t)) return BSA_ERR_INVALID_ARG;
  if (workspace_bytes < l.bytes) return BSA_ERR_WORKSPACE;
  int dev = 0, sms = 0;
  if ((st = check_device(&dev)) != BSA_OK || (st = sms_of(dev, &sms)) != BSA_OK) return st;
  const int tokens = 128 / p.c.d;  // of a line
  const uint64_t lines = (uint64_t)p.c.num_pages * p.c.Hkv * p.c.page / tokens;
  p.tile = cache_tile_keys(p.c.d);
  const int box = (p.c.page < p.tile ? p.c.page : p.tile) / tokens;
  if (!encode_lines_map(&p.tmK, p.c.k, lines, box) || !encode_lines_map(&p.tmV, p.c.v, lines, box))
    return BSA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.q = rows_of(q);
  p.o = static_cast<uint16_t*>(o->data);
  p.o_sb = o->stride_b;
  p.o_sh = o->stride_h;
  p.o_st = o->stride_t;
  p.lse = LSE;
  p.seqs = seqs;
  p.mask = mask;
  p.part = reinterpret_cast<float*>(ws + l.off_part);
  p.desc = reinterpret_cast<int32_t*>(ws + l.off_desc);
  p.counts = reinterpret_cast<int32_t*>(ws + l.off_counts);
  p.list = reinterpret_cast<int32_t*>(ws + l.off_list);
  p.fp16 = dtype == BSA_FP16;
  p.B = B;
  p.Hq = Hq;
  p.g = Hq / p.c.Hkv;
  p.nq = nq;
  p.M = p.g * nq;
  p.groups = (p.M + kCacheUnitRows - 1) / kCacheUnitRows;
  p.NKB = NKB;
  p.bk = bk;
  p.max_tiles = l.max_tiles;
  p.causal = flags & BSA_CACHE_CAUSAL ? 1 : 0;
  p.rows_cap = l.rows_cap;
  p.head = kCacheUnitHead;
  const double sc = scale > 0.f ? (double)scale : 1.0 / std::sqrt((double)p.c.d);
  p.scale_log2 = (float)(sc * 1.4426950408889634);
  p.watchdog_ns = watchdog_limit_ns();
  const int grid = 2 * sms < kCacheMaxGrid ? 2 * sms : kCacheMaxGrid;  // two CTAs per SM
  return launch_cache_attention(p, grid, static_cast<cudaStream_t>(stream)) == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

bsa_status bsa_cache_weigh(const bsa_cache* cache, const bsa_rows* q, const float* LSE, int dtype, const int32_t* seqs,
                           const uint8_t* mask, int NKB, int bk, int B, int Hq, int nq, int flags, float scale,
                           int fresh, float* weights, int weights_tokens, void* stream) {
  CacheWeighParams p;
  std::memset(&p, 0, sizeof(p));
  bsa_status st = check_cache(cache, &p.c);
  if (st != BSA_OK) return st;
  if (!good_rows(q) || !LSE || !aligned(LSE, 4) || !weights || !aligned(weights, 4) || weights_tokens < 1 ||
      !list_ok(seqs))
    return BSA_ERR_INVALID_ARG;
  if ((flags & ~BSA_CACHE_CAUSAL) || fresh < 0) return BSA_ERR_INVALID_ARG;
  if (dtype != BSA_BF16 && dtype != BSA_FP16) return BSA_ERR_UNSUPPORTED;
  if (!(scale == scale) || std::isinf(scale)) return BSA_ERR_INVALID_ARG;
  AttnLayout l;  // (the same limits on sizes; and the line of tiles of 16 keys is 32-bit)
  if ((st = attn_layout(p.c, B, Hq, nq, NKB, bk, mask != nullptr, &l)) != BSA_OK) return st;
  if ((double)B * ((double)p.c.max_pages * p.c.page / 16 + 32) >= 2147483648.0) return BSA_ERR_UNSUPPORTED;
  if (!seqs && B > p.c.max_seqs) return BSA_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  if ((st = check_device(&dev)) != BSA_OK || (st = sms_of(dev, &sms)) != BSA_OK) return st;
  p.q = rows_of(q);
  p.lse = LSE;
  p.weights = weights;
  p.stride = weights_tokens;
  p.seqs = seqs;
  p.mask = mask;
  p.fp16 = dtype == BSA_FP16;
  p.B = B;
  p.Hq = Hq;
  p.g = Hq / p.c.Hkv;
  p.nq = nq;
  p.M = p.g * nq;
  p.NKB = NKB;
  p.bk = bk;
  p.causal = flags & BSA_CACHE_CAUSAL ? 1 : 0;
  p.fresh = fresh;
  p.watchdog_ns = watchdog_limit_ns();
  p.scale = scale > 0.f ? scale : (float)(1.0 / std::sqrt((double)p.c.d));
  return launch_cache_weigh(p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

size_t bsa_cache_evict_workspace_bytes(int n) { return n < 1 || n > kCacheListMax ? 0 : align256(8ull * n); }

bsa_status bsa_cache_evict(const bsa_cache* cache, float* weights, int weights_tokens, const int32_t* seqs,
                           const int32_t* keep, int sink, int recent, int32_t* kept, int keep_max, int n,
                           void* workspace, size_t workspace_bytes, void* stream) {
  CacheEvictParams p;
  std::memset(&p, 0, sizeof(p));
  bsa_status st = check_cache(cache, &p.c);
  if (st != BSA_OK) return st;
  if (!weights || !aligned(weights, 4) || weights_tokens < 1 || !keep || !list_ok(keep) || !list_ok(seqs) || !kept ||
      !list_ok(kept) || keep_max < 1 || n < 1 || sink < 0 || recent < 0 || (!seqs && n > p.c.max_seqs) || !workspace ||
      !aligned(workspace, 4))
    return BSA_ERR_INVALID_ARG;
  if (n > kCacheListMax || (long long)n * p.c.Hkv > (1ll << 24)) return BSA_ERR_UNSUPPORTED;
  if (workspace_bytes < bsa_cache_evict_workspace_bytes(n)) return BSA_ERR_WORKSPACE;
  int dev = 0, sms = 0;
  if ((st = check_device(&dev)) != BSA_OK || (st = sms_of(dev, &sms)) != BSA_OK) return st;
  p.weights = weights;
  p.stride = weights_tokens;
  p.seqs = seqs;
  p.keep = keep;
  p.kept = kept;
  p.cut = static_cast<int32_t*>(workspace);
  p.done = p.cut + n;
  p.n = n;
  p.sink = sink;
  p.recent = recent;
  p.keep_max = keep_max;
  return launch_cache_evict(p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

size_t bsa_cache_forward_workspace_bytes(const bsa_plan* plan, const bsa_cache* cache) {
  bsa_plan_layout L;
  CacheDev c;
  if (bsa_plan_get_layout(plan, &L) != BSA_OK || check_cache(cache, &c) != BSA_OK) return 0;
  const uint64_t kv = 2ull * L.B * c.Hkv * L.NKB * L.bk * c.d;
  return 2 * align256(kv) + align256(4ull * L.B);
}

bsa_status bsa_cache_forward(const bsa_plan* plan, const bsa_cache* cache, const int32_t* seqs, const void* Q,
                             int flags, void* O, float* LSE, float scale, void* workspace, size_t workspace_bytes,
                             void* stream) {
  CacheLoadParams p;
  std::memset(&p, 0, sizeof(p));
  CacheDev& c = p.c;
  bsa_status st = check_cache(cache, &c);
  if (st != BSA_OK) return st;
  bsa_plan_layout L;
  if (!plan) return BSA_ERR_INVALID_ARG;
  if (bsa_plan_get_layout(plan, &L) != BSA_OK) return BSA_ERR_PLAN_MISMATCH;
  if (L.Hkv != c.Hkv) return BSA_ERR_PLAN_MISMATCH;
  if (!Q || !O || !LSE || !workspace || !aligned(workspace, 256) || !list_ok(seqs) || (!seqs && L.B > c.max_seqs))
    return BSA_ERR_INVALID_ARG;
  if (!aligned(Q, 16) || !aligned(O, 16) || !aligned(LSE, 16)) return BSA_ERR_INVALID_ARG;
  if (flags & ~(BSA_FWD_CAUSAL | BSA_FWD_SPLIT_P)) return BSA_ERR_INVALID_ARG;
  if (!(scale == scale) || std::isinf(scale)) return BSA_ERR_INVALID_ARG;
  if (L.qu * L.rq == 64) return BSA_ERR_UNSUPPORTED;  // 64-row q-tiles take no key lengths
  const long long Nk = (long long)L.NKB * L.bk;
  if ((long long)L.B * L.Hkv * Nk >= (1ll << 31) || (long long)L.B * L.Hkv > 65535) return BSA_ERR_UNSUPPORTED;
  if (workspace_bytes < bsa_cache_forward_workspace_bytes(plan, cache)) return BSA_ERR_WORKSPACE;
  int dev = 0;
  if ((st = check_device(&dev)) != BSA_OK) return st;
  if ((st = key_norm_views(plan, &p)) != BSA_OK) return st;
  if (p.device != dev) return BSA_ERR_PLAN_MISMATCH;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const uint64_t kv = align256(2ull * L.B * c.Hkv * (uint64_t)Nk * c.d);
  p.seqs = seqs;
  p.B = L.B;
  p.Nk = (int)Nk;
  p.k = reinterpret_cast<uint16_t*>(ws);
  p.v = reinterpret_cast<uint16_t*>(ws + kv);
  p.lens = reinterpret_cast<int32_t*>(ws + 2 * kv);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (launch_cache_load(p, s) != cudaSuccess) return BSA_ERR_CUDA;
  return forward_after_load(plan, Q, p, flags, O, LSE, scale, s);
}

}  // extern "C"
