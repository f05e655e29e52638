// Argument checks shared by the host side of the cache's and the prompts' calls.
#pragma once

#include <cstddef>
#include <cstdint>

#include "specverify.h"
#include "sv_kv.h"

namespace sv {

constexpr size_t kAlign = 256;
constexpr int kMaxSeqs = 65535;  // a grid's second and third dimension
constexpr int kMaxHeads = 32767;

inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

inline bool valid_dim(int d) { return d == 64 || d == 96 || d == 128 || d == 256; }

// Checks of the cache descriptor; fills `v` when they pass.
inline int check_cache(const specv_kv_t* kv, KvView* v) {
  if (!kv) return SPECV_E_NULL;
  if (kv->type != SPECV_E4M3 && kv->type != SPECV_I8) return SPECV_E_DTYPE;
  if (!kv->k_pages || !kv->v_pages || !kv->k_scales || !kv->v_scales || !kv->page_table) return SPECV_E_NULL;
  const int P = kv->page_size;
  if (P != 16 && P != 32 && P != 64 && P != 128) return SPECV_E_SHAPE;
  if (kv->num_pages < 1 || kv->max_pages < 1 || kv->heads < 1 || kv->heads > kMaxHeads || !valid_dim(kv->dim))
    return SPECV_E_SHAPE;
  if (static_cast<long>(kv->max_pages) * P > INT32_MAX) return SPECV_E_SHAPE;
  if (!aligned16(kv->k_pages) || !aligned16(kv->v_pages)) return SPECV_E_ALIGN;
  if (reinterpret_cast<uintptr_t>(kv->k_scales) % 4 || reinterpret_cast<uintptr_t>(kv->v_scales) % 4)
    return SPECV_E_ALIGN;
  v->kp = static_cast<uint8_t*>(kv->k_pages);
  v->vp = static_cast<uint8_t*>(kv->v_pages);
  v->ks = kv->k_scales;
  v->vs = kv->v_scales;
  v->table = kv->page_table;
  v->pages = kv->num_pages;
  v->width = kv->max_pages;
  v->P = P;
  v->pshift = P == 16 ? 4 : P == 32 ? 5 : P == 64 ? 6 : 7;
  v->H = kv->heads;
  v->D = kv->dim;
  return SPECV_OK;
}

// A token row of `heads` heads: 0 stands for contiguous rows.  Rows keep the
// 16-byte alignment of the vector loads and do not overlap.
inline int check_row(int64_t* row, long heads, int D, int dtype) {
  if (*row == 0) *row = heads * D;
  if (*row < heads * D || *row > (int64_t(1) << 40)) return SPECV_E_SHAPE;
  return *row * (dtype == SPECV_F32 ? 4 : 2) % 16 ? SPECV_E_ALIGN : SPECV_OK;
}

// Whether a[0 .. na) and b[0 .. nb) share bytes; null arrays share none.
inline bool overlap(const int32_t* a, long na, const int32_t* b, long nb) {
  const auto x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + 4 * static_cast<uintptr_t>(nb) && y < x + 4 * static_cast<uintptr_t>(na);
}

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

}  // namespace sv
