// Host side of the operators on prompts' rows: argument checks, workspace
// layout and launches.  See include/bsa.h for the contract of each.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "bsa_internal.h"
#include "bsa_prompt.h"

using namespace bsa;

namespace {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool good_rows(const bsa_rows* r) {
  return r && r->data && aligned(r->data, 16) && r->stride_b >= 0 && r->stride_h >= 0 && r->stride_t >= 0 &&
         r->stride_b % 8 == 0 && r->stride_h % 8 == 0 && r->stride_t % 8 == 0;
}

// Rows in and out of bsa_rope_apply; false where they are no such rows, or where
// several rows that are written are one.
bool rope_rows(const bsa_rows* in, const bsa_rows* out, int B, int H, int T, RopeRows* r) {
  if (!good_rows(in) || !good_rows(out)) return false;
  if ((B > 1 && !out->stride_b) || (H > 1 && !out->stride_h) || (T > 1 && !out->stride_t)) return false;
  *r = RopeRows{static_cast<const uint16_t*>(in->data), static_cast<uint16_t*>(out->data),
                in->stride_b, in->stride_h, in->stride_t, out->stride_b, out->stride_h, out->stride_t};
  return true;
}
// Every row of the output is the input's own.
bool in_place(const RopeRows& r, int B, int H, int T) {
  return r.p == r.o && (B == 1 || r.sb == r.ob) && (H == 1 || r.sh == r.oh) && (T == 1 || r.st == r.ot);
}

// Packed rows [T][H][d]: rows of their own.
bool good_packed(const bsa_rows* r, int T, int H) {
  return good_rows(r) && (T == 1 || (r->stride_t && r->stride_t < (1ll << 38))) &&
         (H == 1 || (r->stride_h && r->stride_h < (1ll << 38)));
}

struct PromptLayout {
  size_t off_ptr, off_tiles, bytes;
  int gp_shift;
};
bsa_status prompt_layout(int n, int T, int Hq, int Hkv, PromptLayout* out) {
  if (n < 1 || T < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv) return BSA_ERR_INVALID_ARG;
  PromptLayout l;
  const int g = Hq / Hkv;
  l.gp_shift = 0;
  while (l.gp_shift < 4 && !(g >> l.gp_shift & 1)) ++l.gp_shift;
  const long long tiles = (long long)T / (kPromptRows >> l.gp_shift) + n;
  if (T > (1 << 30) || Hq > 65536 || tiles * (Hq >> l.gp_shift) >= (1ll << 31)) return BSA_ERR_UNSUPPORTED;
  size_t off = align256(4 * kPromptCtlWords);
  l.off_ptr = off;   off = align256(off + 4ull * ((uint64_t)n + 1));
  l.off_tiles = off; off = align256(off + 16ull * (uint64_t)tiles);
  l.bytes = off;
  *out = l;
  return BSA_OK;
}

}  // namespace

extern "C" {

size_t bsa_prompt_workspace_bytes(int n, int T, int Hq, int Hkv) {
  PromptLayout l;
  return prompt_layout(n, T, Hq, Hkv, &l) == BSA_OK ? l.bytes : 0;
}

bsa_status bsa_prompt_attention(const bsa_rows* q, const bsa_rows* k, const bsa_rows* v, const bsa_rows* o, float* LSE,
                                int dtype, const int32_t* offsets, int n, int T, int Hq, int Hkv, int d, int flags,
                                float scale, void* workspace, size_t workspace_bytes, void* stream) {
  PromptParams p;
  std::memset(&p, 0, sizeof(p));
  PromptLayout l;
  bsa_status st = prompt_layout(n, T, Hq, Hkv, &l);
  if (st != BSA_OK) return st;
  if (!good_packed(q, T, Hq) || !good_packed(k, T, Hkv) || !good_packed(v, T, Hkv) || !good_packed(o, T, Hq) ||
      !offsets || !aligned(offsets, 4) || !aligned(LSE, 4) || !workspace || !aligned(workspace, 16))
    return BSA_ERR_INVALID_ARG;
  if (flags & ~BSA_PROMPT_CAUSAL) return BSA_ERR_INVALID_ARG;
  if (!(scale == scale) || std::isinf(scale)) return BSA_ERR_INVALID_ARG;
  if (dtype != BSA_BF16 && dtype != BSA_FP16) return BSA_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return BSA_ERR_UNSUPPORTED;
  if (workspace_bytes < l.bytes) return BSA_ERR_WORKSPACE;
  int dev = 0, sms = 0;
  if ((st = check_device(&dev)) != BSA_OK) return st;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return BSA_ERR_CUDA;
  if (!encode_packed_map(&p.tmQ, *q, T, Hq, d, 1 << l.gp_shift, 128 >> l.gp_shift) ||
      !encode_packed_map(&p.tmK, *k, T, Hkv, d, 1, 128) || !encode_packed_map(&p.tmV, *v, T, Hkv, d, 1, 128))
    return BSA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.v = static_cast<const uint16_t*>(v->data);
  p.v_st = v->stride_t;
  p.v_sh = v->stride_h;
  p.o = static_cast<uint16_t*>(o->data);
  p.o_st = o->stride_t;
  p.o_sh = o->stride_h;
  p.o_v8 = aligned(o->data, 32) && o->stride_t % 16 == 0 && o->stride_h % 16 == 0;
  p.lse = LSE;
  p.offsets = offsets;
  p.control = reinterpret_cast<int32_t*>(ws);
  p.tile_ptr = reinterpret_cast<int32_t*>(ws + l.off_ptr);
  p.tiles = reinterpret_cast<int4*>(ws + l.off_tiles);
  p.n = n;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.g = Hq / Hkv;
  p.gp_shift = l.gp_shift;
  p.causal = flags & BSA_PROMPT_CAUSAL ? 1 : 0;
  p.fp16 = dtype == BSA_FP16;
  p.few = n <= kPromptFew && T <= kPromptFewTokens ? 1 : 0;
  const double sc = scale > 0.f ? (double)scale : 1.0 / std::sqrt((double)d);
  p.scale_log2 = (float)(sc * 1.4426950408889634);
  p.watchdog_ns = watchdog_limit_ns();
  return launch_prompt(p, d, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

bsa_status bsa_prompt_status(const void* workspace, void* stream, int32_t* detail) {
  if (!workspace || !aligned(workspace, 16)) return BSA_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t words[kPromptCtlWords];
  if (cudaMemcpyAsync(words, workspace, sizeof(words), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return BSA_ERR_CUDA;
  // What was found of the offsets, then what the CTAs' waits recorded, the first CTA's first.
  const int32_t* word = words + kCtlStatus;
  const int32_t ctas = words[kPromptCtlCtas];
  for (int32_t i = 0; word[0] == BSA_OK && i < ctas && i < kPromptMaxCtas; ++i) word = words + kPromptCtlOwn + 2 * i;
  if (detail) *detail = word[1];
  return static_cast<bsa_status>(word[0]);
}

bsa_status bsa_rope_steps(int rot, double base, int scaling, double factor, double original, uint64_t* steps,
                          float* amplitude) {
  if (!steps || !amplitude || rot < 16 || rot > 128 || rot % 16) return BSA_ERR_INVALID_ARG;
  if (!(base > 1.0) || std::isinf(base)) return BSA_ERR_INVALID_ARG;
  if (scaling < BSA_ROPE_NONE || scaling > BSA_ROPE_PARTS) return BSA_ERR_UNSUPPORTED;
  if (scaling != BSA_ROPE_NONE && (!(factor >= 1.0) || std::isinf(factor))) return BSA_ERR_INVALID_ARG;
  if (scaling == BSA_ROPE_PARTS && (!(original >= 1.0) || std::isinf(original))) return BSA_ERR_INVALID_ARG;
  const double turn = 6.283185307179586;
  double b = base;
  if (scaling == BSA_ROPE_BASE) b *= std::pow(factor, (double)rot / (rot - 2));
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(b, -2.0 * i / rot);
    if (scaling == BSA_ROPE_LINEAR) f /= factor;
    if (scaling == BSA_ROPE_PARTS) {
      double stay = (original * f / turn - 1.0) / 31.0;
      stay = stay < 0.0 ? 0.0 : (stay > 1.0 ? 1.0 : stay);
      f = f / factor * (1.0 - stay) + f * stay;
    }
    steps[i] = (uint64_t)(f / turn * 0x1p64);  // (at most 1 / (2 pi) turns a position)
  }
  *amplitude = scaling == BSA_ROPE_PARTS ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  return BSA_OK;
}

bsa_status bsa_rope_apply(const bsa_rope* rope, const bsa_rows* q, const bsa_rows* q_out, int Hq, const bsa_rows* k,
                          const bsa_rows* k_out, int Hk, int dtype, const int32_t* positions, int B, int T, int d,
                          int flags, void* stream) {
  RopeParams p;
  std::memset(&p, 0, sizeof(p));
  if (!rope || !rope->steps || !aligned(rope->steps, 8) || !aligned(positions, 4)) return BSA_ERR_INVALID_ARG;
  if (B < 1 || T < 1 || Hq < 1 || Hk < 0 || (flags & ~BSA_ROPE_INVERSE)) return BSA_ERR_INVALID_ARG;
  if (dtype != BSA_BF16 && dtype != BSA_FP16) return BSA_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return BSA_ERR_UNSUPPORTED;
  if (rope->rot < 16 || rope->rot > d || rope->rot % 16) return BSA_ERR_UNSUPPORTED;
  if (rope->pairs != BSA_ROPE_HALF && rope->pairs != BSA_ROPE_NEIGHBOURS) return BSA_ERR_UNSUPPORTED;
  if (!(rope->amplitude == rope->amplitude) || std::isinf(rope->amplitude)) return BSA_ERR_INVALID_ARG;
  if (!rope_rows(q, q_out, B, Hq, T, &p.q) || (Hk > 0 && !rope_rows(k, k_out, B, Hk, T, &p.k)))
    return BSA_ERR_INVALID_ARG;
  if (Hq > 65536 || Hk > 65536 || (long long)B * T > (1ll << 30)) return BSA_ERR_UNSUPPORTED;
  int dev = 0, sms = 0;
  bsa_status st = check_device(&dev);
  if (st != BSA_OK) return st;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return BSA_ERR_CUDA;
  p.steps = rope->steps;
  p.positions = positions;
  p.amp = rope->amplitude;
  p.fp16 = dtype == BSA_FP16;
  p.neighbours = rope->pairs == BSA_ROPE_NEIGHBOURS;
  p.inverse = flags & BSA_ROPE_INVERSE ? 1 : 0;
  p.B = B;
  p.T = T;
  p.Hq = Hq;
  p.H = Hq + Hk;
  p.d = d;
  p.rot = rope->rot;
  p.tail = rope->rot < d && !(in_place(p.q, B, Hq, T) && (Hk == 0 || in_place(p.k, B, Hk, T)));
  // Rounds of heads per warp: all of a token's where the tokens alone give every
  // SM 16 warps, fewer where they do not.
  const int rounds = (p.H + rope_heads_per_round(d) - 1) / rope_heads_per_round(d);
  const long long tokens = (long long)B * T, want = 16ll * sms;
  long long parts = (want + tokens - 1) / tokens;
  if (parts > rounds) parts = rounds;
  p.per = (int)((rounds + parts - 1) / parts);
  p.parts = (rounds + p.per - 1) / p.per;
  return launch_rope(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // extern "C"
