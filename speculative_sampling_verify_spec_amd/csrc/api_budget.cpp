// Host side of the cache under a budget: argument checks and launches of
// spec_kv_weights and spec_kv_evict.  Nothing here allocates, synchronises or
// keeps state.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "specverify.h"
#include "sv_budget.h"
#include "sv_host.h"

namespace sv {
namespace {

bool apart(const void* a, long na, const void* b, long nb) {
  return !overlap(static_cast<const int32_t*>(a), na, static_cast<const int32_t*>(b), nb);
}

// Words from the first to the last of `rows` token rows `stride` elements
// apart, of `row` elements each (strides that no memory has are cut short).
long row_words(long rows, int64_t stride, long row, int dtype) {
  const long n = (rows - 1) * std::min<int64_t>(stride, int64_t(1) << 36) + row;
  return dtype == SPECV_F32 ? n : n / 2;
}

// Positions are rounded up to a workgroup's in 32 bits.
constexpr int64_t kMostPositions = (int64_t(1) << 31) - 2 * kEvictTile;
int64_t positions(const KvView& c) { return static_cast<int64_t>(c.width) << c.pshift; }

// Weights cover every position that the table can hold.
bool covers(const KvView& c, int64_t capacity) {
  return capacity >= positions(c) && positions(c) <= kMostPositions && capacity <= INT32_MAX;
}

// Workgroups that share a head's tokens, for `pairs` sequences' heads of up to
// `turns` times 256 tokens: two a CU where that fills them, and up to eight as
// long as each has eight turns, so that the longest sequence does not end alone;
// eight a CU for so many pairs that its length alone would decide.  512, 2048
// and this many (us; heads of 8): 1 sequence of 131072 tokens 23.7, 26.7, 23.6; 16 of
// up to 4096 13.7, 16.2, 13.7; 64 of up to 2111 22.4, 24.4, 22.5; 32 of up to 32768 170,
// 140, 140, 33 of them 278, 146, 145, 64 of them 327, 262, 262; 40 of 8192 88, 73, 73.
// 40 of up to 2111 tokens take 20.5 so, with six workgroups a head 17.5.
long weight_splits(long pairs, long turns) {
  const long most = std::max(1L, 2048 / pairs);
  return pairs > 512 ? most : std::max(512 / pairs, std::min(most, turns / 8));
}

}  // namespace
}  // namespace sv

extern "C" {

int spec_kv_weights(const specv_kv_t* kv, const void* q, int64_t q_stride, const float* lse, const void* k_new,
                    int64_t k_stride, const int32_t* lengths, const int32_t* counts, const int32_t* index,
                    float scale, int B, int N, int Hq, const float* weights, float* out_weights, int64_t capacity,
                    int dtype, void* stream) {
  using namespace sv;
  KvWeights p{};
  if (dtype != SPECV_F32 && dtype != SPECV_BF16) return SPECV_E_DTYPE;
  if (const int rc = check_cache(kv, &p.c)) return rc;
  if (!q || !lse || !lengths || !weights || !out_weights) return SPECV_E_NULL;
  if (B < 1 || B > kMaxSeqs || N < 1 || N > SPECV_MAX_TREE || Hq < 1 || Hq > kMaxHeads || Hq % p.c.H ||
      Hq / p.c.H > SPECV_KV_MAX_GROUP || static_cast<long>(B) * p.c.H >= (1L << 24))
    return SPECV_E_SHAPE;
  if (!covers(p.c, capacity) || !std::isfinite(scale * 1.5f)) return SPECV_E_SHAPE;
  if (const int rc = check_row(&q_stride, Hq, p.c.D, dtype)) return rc;
  if (k_new)
    if (const int rc = check_row(&k_stride, p.c.H, p.c.D, dtype)) return rc;
  if (!aligned16(q) || !aligned16(k_new)) return SPECV_E_ALIGN;
  const long all = static_cast<long>(B) * p.c.H * capacity;
  if (weights != out_weights && !apart(weights, all, out_weights, all)) return SPECV_E_OVERLAP;
  // workgroups write a head's weights while others still read these
  const long nodes = static_cast<long>(B) * N, blocks = static_cast<long>(p.c.pages) * p.c.H;
  const struct { const void* at; long n; } in[] = {{q, row_words(nodes, q_stride, Hq * p.c.D, dtype)},
      {k_new, row_words(nodes, k_stride, p.c.H * p.c.D, dtype)}, {lse, nodes * Hq}, {lengths, B}, {counts, B}, {index, nodes},
      {p.c.table, static_cast<long>(B) * p.c.width}, {p.c.kp, blocks * p.c.P * p.c.D / 4}, {p.c.ks, blocks}};
  for (const auto& x : in)
    if (!apart(x.at, x.n, out_weights, all)) return SPECV_E_OVERLAP;
  p.q = q;
  p.kn = k_new;
  p.q_row = q_stride;
  p.k_row = k_stride;
  p.lse = lse;
  p.lengths = lengths;
  p.counts = counts;
  p.index = index;
  p.scale = scale;
  p.B = B;
  p.N = N;
  p.Hq = Hq;
  p.G = Hq / p.c.H;
  p.w = weights;
  p.out = out_weights;
  p.capacity = capacity;
  const long turns = ((static_cast<long>(p.c.width) << p.c.pshift) + 255) / 256, pairs = static_cast<long>(B) * p.c.H;
  p.splits = static_cast<unsigned>(std::min(turns, weight_splits(pairs, turns)));
  return launch_kv_weights(p, dtype, kv->type, static_cast<hipStream_t>(stream)) == hipSuccess ? SPECV_OK : SPECV_E_HIP;
}

size_t spec_kv_evict_workspace_size(const specv_kv_t* kv, int B) {
  using namespace sv;
  KvView c{};
  if (check_cache(kv, &c) != SPECV_OK || B < 1 || B > kMaxSeqs || positions(c) > kMostPositions) return 0;
  const long rows = static_cast<long>(B) * c.H, tiles = kv_evict_tiles(c);
  if (rows * tiles >= (1L << 22)) return 0;  // a grid's threads stay below 2^32
  return std::max(kAlign, tiles > 1 ? align_up(static_cast<size_t>(rows) * tiles * kEvictWords * sizeof(uint32_t)) : 0);
}

int spec_kv_evict(const specv_kv_t* kv, const int32_t* lengths, const float* weights, int64_t capacity,
                  const int32_t* new_pages, int budget, int recent, int limit, int B, int32_t* out_table,
                  int32_t* out_lengths, float* out_weights, int32_t* kept, void* workspace, size_t workspace_bytes,
                  void* stream) {
  using namespace sv;
  KvEvict p{};
  if (const int rc = check_cache(kv, &p.c)) return rc;
  if (!lengths || !weights || !new_pages || !out_table || !out_lengths || !out_weights || !kept) return SPECV_E_NULL;
  const long most = static_cast<long>(p.c.width) << p.c.pshift;
  if (B < 1 || B > kMaxSeqs || p.c.H > kMaxHeads || budget < 1 || budget > most || recent < 0 || recent > budget ||
      limit < budget || !covers(p.c, capacity))
    return SPECV_E_SHAPE;
  const long width = (budget + p.c.P - 1) / p.c.P, table = static_cast<long>(B) * p.c.width;
  const long pages = B * width, heads = static_cast<long>(B) * p.c.H, all = heads * capacity, keep = heads * budget;
  const size_t need = spec_kv_evict_workspace_size(kv, B);
  if (!need || heads * width >= (1L << 23)) return SPECV_E_SHAPE;  // a grid's threads stay below 2^32
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % kAlign || workspace_bytes < need) return SPECV_E_WORKSPACE;
  // workgroups write these while others still read those
  const struct Words { const void* at; long n; } in[] = {{lengths, B}, {p.c.table, table}, {new_pages, pages}, {weights, all}},
      out[] = {{out_table, table}, {out_lengths, B}, {out_weights, all}, {kept, keep}};
  for (int i = 0; i < 4; ++i) {
    for (const auto& x : in)
      if (!apart(x.at, x.n, out[i].at, out[i].n)) return SPECV_E_OVERLAP;
    for (int j = 0; j < i; ++j)
      if (!apart(out[j].at, out[j].n, out[i].at, out[i].n)) return SPECV_E_OVERLAP;
  }
  // the workspace too; the cache's own arrays, the page table among them, are not compared with it
  for (const auto& x : {in[0], in[2], in[3], out[0], out[1], out[2], out[3]})
    if (!apart(x.at, x.n, workspace, static_cast<long>(need / 4))) return SPECV_E_OVERLAP;
  p.lengths = lengths;
  p.w = weights;
  p.capacity = capacity;
  p.new_pages = new_pages;
  p.new_width = static_cast<int>(width);
  p.budget = budget;
  p.recent = recent;
  p.limit = limit;
  p.B = B;
  p.out_table = out_table;
  p.out_lengths = out_lengths;
  p.out_w = out_weights;
  p.kept = kept;
  p.tiles = static_cast<int>(kv_evict_tiles(p.c));
  p.scratch = static_cast<uint32_t*>(workspace);
  return launch_kv_evict(p, kv->type, static_cast<hipStream_t>(stream)) == hipSuccess ? SPECV_OK : SPECV_E_HIP;
}

}  // extern "C"
