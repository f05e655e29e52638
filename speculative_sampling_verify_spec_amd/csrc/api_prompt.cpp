// Host side of whole prompts: argument checks and launches of
// spec_prompt_attention and spec_prompt_weights.  Nothing here allocates, synchronises or keeps state.
#include <cmath>
#include <cstdint>

#include "specverify.h"
#include "sv_host.h"
#include "sv_prompt.h"

namespace sv {
namespace {

// Checks that the prompts' calls share; fills `s` when they pass.
int check_packed(const void* q, int64_t q_stride, const void* k, const void* v, int64_t kv_stride,
                 const int32_t* starts, float scale, int B, int T, int heads, int Hq, int dim, int dtype, Packed* s) {
  if (dtype != SPECV_F32 && dtype != SPECV_BF16) return SPECV_E_DTYPE;
  if (!q || !k || !starts) return SPECV_E_NULL;
  if (B < 1 || B > kMaxSeqs || T < 1 || T > SPECV_KV_MAX_APPEND || !valid_dim(dim)) return SPECV_E_SHAPE;
  if (heads < 1 || heads > kMaxHeads || Hq < 1 || Hq > kMaxHeads || Hq % heads || Hq / heads > SPECV_KV_MAX_GROUP)
    return SPECV_E_SHAPE;
  // a sequence's rows are counted in 32 bits, a grid's threads too
  if (static_cast<long>(T) * (Hq / heads) >= (1L << 30)) return SPECV_E_SHAPE;
  if (prompt_slots(T, Hq / heads, B, kPromptRows) * heads >= (1L << 24)) return SPECV_E_SHAPE;
  if (!std::isfinite(scale * 1.5f)) return SPECV_E_SHAPE;  // times log2(e), as the kernels use it
  if (const int rc = check_row(&q_stride, Hq, dim, dtype)) return rc;
  if (const int rc = check_row(&kv_stride, heads, dim, dtype)) return rc;
  if (q_stride >= (1 << 24) || kv_stride >= (1 << 24)) return SPECV_E_SHAPE;  // a tile's rows are reached in 32 bits
  if (!aligned16(q) || !aligned16(k) || !aligned16(v)) return SPECV_E_ALIGN;
  s->q = q;
  s->k = k;
  s->v = v;
  s->q_row = q_stride;
  s->kv_row = kv_stride;
  s->starts = starts;
  s->scale = scale;
  s->B = B;
  s->T = T;
  s->H = heads;
  s->Hq = Hq;
  s->G = Hq / heads;
  // r / G for r < 2^31 is mulhi(r, m) >> (l - 1) with 2^l >= G and m = floor(2^(31 + l) / G) + 1 < 2^32:
  // r m / 2^(31 + l) exceeds r / G by r (m G - 2^(31 + l)) / (G 2^(31 + l)) < 2^31 G / (G 2^31 2^l) <= 1 / G
  int l = 1;
  while ((1 << l) < s->G) ++l;
  s->magic = s->G > 1 ? static_cast<uint32_t>((uint64_t(1) << (31 + l)) / s->G + 1) : 0;
  s->shift = l - 1;
  return SPECV_OK;
}

}  // namespace
}  // namespace sv

extern "C" {

int spec_prompt_attention(const void* q, int64_t q_stride, const void* k, const void* v, int64_t kv_stride,
                          const int32_t* starts, float scale, int B, int T, int heads, int Hq, int dim, void* out,
                          float* out_lse, int dtype, void* stream) {
  using namespace sv;
  PromptAttn p{};
  if (const int rc = check_packed(q, q_stride, k, v, kv_stride, starts, scale, B, T, heads, Hq, dim, dtype, &p.s))
    return rc;
  if (!v || !out) return SPECV_E_NULL;
  if (!aligned16(out)) return SPECV_E_ALIGN;
  p.out = out;
  p.lse = out_lse;
  p.slots = static_cast<unsigned>(prompt_slots(T, p.s.G, B, kPromptRows));
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const hipError_t e = dim == 64    ? launch_prompt_64(p, dtype, st)
                       : dim == 96  ? launch_prompt_96(p, dtype, st)
                       : dim == 128 ? launch_prompt_128(p, dtype, st)
                                    : launch_prompt_256(p, dtype, st);
  return e == hipSuccess ? SPECV_OK : SPECV_E_HIP;
}

int spec_prompt_weights(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const float* lse,
                        const int32_t* starts, float scale, int B, int T, int heads, int Hq, int dim,
                        float* out_weights, int64_t capacity, int dtype, void* stream) {
  using namespace sv;
  PromptWeights p{};
  if (const int rc = check_packed(q, q_stride, k, nullptr, k_stride, starts, scale, B, T, heads, Hq, dim, dtype, &p.s))
    return rc;
  if (!lse || !out_weights) return SPECV_E_NULL;
  if (capacity < 1 || capacity > INT32_MAX) return SPECV_E_SHAPE;
  if (prompt_slots(T, 1, B, kWeightKeys) * heads >= (1L << 24)) return SPECV_E_SHAPE;
  p.lse = lse;
  p.w = out_weights;
  p.capacity = static_cast<int>(capacity);
  p.slots = static_cast<unsigned>(prompt_slots(T, 1, B, kWeightKeys));
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const hipError_t e = dim == 64    ? launch_prompt_weights_64(p, dtype, st)
                       : dim == 96  ? launch_prompt_weights_96(p, dtype, st)
                       : dim == 128 ? launch_prompt_weights_128(p, dtype, st)
                                    : launch_prompt_weights_256(p, dtype, st);
  return e == hipSuccess ? SPECV_OK : SPECV_E_HIP;
}

}  // extern "C"
