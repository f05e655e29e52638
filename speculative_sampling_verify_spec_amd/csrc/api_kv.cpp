// Host side of the 8-bit paged cache: argument checks and launches of
// spec_kv_append, spec_kv_read and spec_kv_attention.  Nothing here
// allocates, synchronises or keeps state.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "specverify.h"
#include "sv_kv.h"

namespace sv {
namespace {

constexpr size_t kAlign = 256;
constexpr int kMaxSeqs = 65535;  // a grid's second and third dimension
constexpr int kMaxHeads = 32767;

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

bool valid_dim(int d) { return d == 64 || d == 96 || d == 128 || d == 256; }

// Checks of the cache descriptor; fills `v` when they pass.
int check_cache(const specv_kv_t* kv, KvView* v) {
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
int check_row(int64_t* row, long heads, int D, int dtype) {
  if (*row == 0) *row = heads * D;
  if (*row < heads * D || *row > (int64_t(1) << 40)) return SPECV_E_SHAPE;
  return *row * (dtype == SPECV_F32 ? 4 : 2) % 16 ? SPECV_E_ALIGN : SPECV_OK;
}

// Whether a[0 .. na) and b[0 .. nb) share bytes; null arrays share none.
bool overlap(const int32_t* a, long na, const int32_t* b, long nb) {
  const auto x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + 4 * static_cast<uintptr_t>(nb) && y < x + 4 * static_cast<uintptr_t>(na);
}

// How an attention call is cut into workgroups; from sizes alone (the lengths
// are on the device), so that the workspace's size is known before.
struct KvPlan {
  int mt, mb, granule, splits;
};

// Workgroups to aim at.  Fewer leave CUs idle, more mean more of the parts'
// own cost, their queries and their sums (us, at 256 / 512 / 1024 / 2048): 2 x
// 5 positions over 131072 tokens 125, 111, 121, 137; 64 x 6 over 301-2111
// 41, 41, 54, 50; 16 x 9 in fp32 over 65-2900 29.2, 27.1, 26.8, 26.7; 512 x 1
// with heads of 256 223, 222, 224, 276.
constexpr long kTargetGroups = 512;
// Tiles per part: four for each wave.  Fewer would need a second launch for
// the join: 1 x 1 over 1000 tokens takes 12.4 us in one part of 16 tiles and
// 11.5 us in four of 4, but 14.8 and 18.5 us a call with the launches' cost.
constexpr int kMinGranule = 16;

KvPlan kv_plan(const KvView& c, int B, int N, int Hq, int dtype) {
  KvPlan pl;
  const int rows = N * (Hq / c.H), most = 16 * kv_max_mt(dtype, c.D);
  pl.mb = (rows + most - 1) / most;
  pl.mt = ((rows + pl.mb - 1) / pl.mb + 15) / 16;
  const long tiles = ((static_cast<long>(c.width) << c.pshift) + 63) / 64;
  const long groups = static_cast<long>(B) * c.H * pl.mb;
  const long per = std::max(1L, kTargetGroups / groups);  // parts a longest sequence should have
  pl.granule = static_cast<int>(std::max<long>(kMinGranule, (tiles + per - 1) / per));
  pl.splits = static_cast<int>(std::max(1L, (tiles + pl.granule - 1) / pl.granule));
  return pl;
}

bool valid_attention(const KvView& c, int B, int N, int Hq) {
  if (B < 1 || B > kMaxSeqs || N < 1 || N > SPECV_MAX_TREE || Hq < 1 || Hq > kMaxHeads || Hq % c.H || Hq / c.H > SPECV_KV_MAX_GROUP)
    return false;
  for (int dt : {SPECV_F32, SPECV_BF16}) {  // a grid's workgroups times their threads stay below 2^32
    const KvPlan pl = kv_plan(c, B, N, Hq, dt);
    if ((static_cast<long>(B) * c.H * pl.splits + 7) * pl.mb * 256 >= (1L << 32)) return false;
  }
  return static_cast<long>(B) * N * Hq * 64 < (1L << 32);
}

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

size_t part_rows(int B, int N, int Hq, const KvPlan& pl) { return static_cast<size_t>(B) * N * Hq * pl.splits; }

}  // namespace
}  // namespace sv

extern "C" {

int spec_kv_append(const specv_kv_t* kv, const void* k, const void* v, int64_t row_stride, const int32_t* lengths,
                   const int32_t* counts, const int32_t* index, int B, int N, int32_t* out_lengths, int dtype,
                   void* stream) {
  using namespace sv;
  KvAppend p{};
  if (dtype != SPECV_F32 && dtype != SPECV_BF16) return SPECV_E_DTYPE;
  if (const int rc = check_cache(kv, &p.c)) return rc;
  if (!k || !v || !lengths) return SPECV_E_NULL;
  if (B < 1 || B > kMaxSeqs || N < 1 || N > SPECV_KV_MAX_APPEND) return SPECV_E_SHAPE;
  if (const int rc = check_row(&row_stride, p.c.H, p.c.D, dtype)) return rc;
  if (!aligned16(k) || !aligned16(v)) return SPECV_E_ALIGN;
  // one workgroup writes a sequence's new length while others still read these
  if (overlap(out_lengths, B, lengths, B) || overlap(out_lengths, B, counts, B) ||
      overlap(out_lengths, B, index, static_cast<long>(B) * N) ||
      overlap(out_lengths, B, p.c.table, static_cast<long>(B) * p.c.width))
    return SPECV_E_OVERLAP;
  p.k = k;
  p.v = v;
  p.row = row_stride;
  p.lengths = lengths;
  p.counts = counts;
  p.index = index;
  p.B = B;
  p.N = N;
  p.out_lengths = out_lengths;
  p.groups = kv_append_groups(N, p.c.P);
  return launch_kv_append(p, dtype, kv->type, static_cast<hipStream_t>(stream)) == hipSuccess ? SPECV_OK
                                                                                             : SPECV_E_HIP;
}

int spec_kv_read(const specv_kv_t* kv, const int32_t* starts, const int32_t* lengths, int B, int T, void* out_k,
                 void* out_v, int dtype, void* stream) {
  using namespace sv;
  KvRead p{};
  if (dtype != SPECV_F32 && dtype != SPECV_BF16) return SPECV_E_DTYPE;
  if (const int rc = check_cache(kv, &p.c)) return rc;
  if (!lengths || (!out_k && !out_v)) return SPECV_E_NULL;
  if (B < 1 || B > kMaxSeqs || T < 1 || T > SPECV_KV_MAX_APPEND) return SPECV_E_SHAPE;
  if (!aligned16(out_k) || !aligned16(out_v)) return SPECV_E_ALIGN;
  p.starts = starts;
  p.lengths = lengths;
  p.B = B;
  p.T = T;
  p.out_k = out_k;
  p.out_v = out_v;
  return launch_kv_read(p, dtype, kv->type, static_cast<hipStream_t>(stream)) == hipSuccess ? SPECV_OK : SPECV_E_HIP;
}

size_t spec_kv_attention_workspace_size(const specv_kv_t* kv, int B, int N, int Hq) {
  using namespace sv;
  KvView c{};
  if (check_cache(kv, &c) != SPECV_OK) return 0;
  if (!valid_attention(c, B, N, Hq)) return 0;
  size_t most = kAlign;  // a call in one part per sequence uses none of it
  for (int dt : {SPECV_F32, SPECV_BF16}) {
    const KvPlan pl = kv_plan(c, B, N, Hq, dt);
    const size_t rows = part_rows(B, N, Hq, pl);
    if (pl.splits > 1) most = std::max(most, align_up(rows * c.D * sizeof(float)) + align_up(rows * sizeof(float2)));
  }
  return most;
}

int spec_kv_attention(const specv_kv_t* kv, const void* q, int64_t q_stride, const void* k_new, const void* v_new,
                      int64_t kv_stride, const int32_t* lengths, const int32_t* num_nodes, const int32_t* parents,
                      float scale, int B, int N, int Hq, void* out, float* out_lse, int dtype, void* workspace,
                      size_t workspace_bytes, void* stream) {
  using namespace sv;
  KvAttn p{};
  if (dtype != SPECV_F32 && dtype != SPECV_BF16) return SPECV_E_DTYPE;
  if (const int rc = check_cache(kv, &p.c)) return rc;
  if (!q || !lengths || !out || !k_new != !v_new) return SPECV_E_NULL;
  if (!valid_attention(p.c, B, N, Hq)) return SPECV_E_SHAPE;
  if (!std::isfinite(scale * 1.5f)) return SPECV_E_SHAPE;  // times log2(e), as the kernels use it
  if (const int rc = check_row(&q_stride, Hq, p.c.D, dtype)) return rc;
  if (k_new)
    if (const int rc = check_row(&kv_stride, p.c.H, p.c.D, dtype)) return rc;
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(out)) return SPECV_E_ALIGN;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % kAlign ||
      workspace_bytes < spec_kv_attention_workspace_size(kv, B, N, Hq))
    return SPECV_E_WORKSPACE;
  p.q = q;
  p.kn = k_new;
  p.vn = v_new;
  p.q_row = q_stride;
  p.kv_row = kv_stride;
  p.lengths = lengths;
  p.nodes = num_nodes;
  p.parents = parents;
  p.scale = scale;
  p.B = B;
  p.N = N;
  p.Hq = Hq;
  p.G = Hq / p.c.H;
  p.inv_g = 1.f / static_cast<float>(p.G);
  p.out = out;
  p.lse = out_lse;
  const KvPlan pl = kv_plan(p.c, B, N, Hq, dtype);
  p.mt = pl.mt;
  p.mb = pl.mb;
  p.granule = pl.granule;
  p.splits = pl.splits;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) +
                                        align_up(part_rows(B, N, Hq, pl) * p.c.D * sizeof(float)));
  return launch_kv_attention(p, dtype, kv->type, static_cast<hipStream_t>(stream)) == hipSuccess ? SPECV_OK
                                                                                                : SPECV_E_HIP;
}

}  // extern "C"
