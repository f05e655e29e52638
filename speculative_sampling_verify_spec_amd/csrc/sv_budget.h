// The cache under a budget: parameters shared by the host code and kernels of
// the gathered weights and of the eviction.
#pragma once

#include "sv_kv.h"

namespace sv {

struct KvWeights {
  KvView c;
  const void* q;          // [B][N] rows of Hq*D elements, q_row elements apart
  const void* kn;         // [B][N] rows of H*D elements, k_row elements apart, or null
  long q_row, k_row;
  const float* lse;       // [B][N][Hq]
  const int32_t* lengths;
  const int32_t* counts;  // or null
  const int32_t* index;   // or null
  float scale;
  int B, N, Hq, G;
  const float* w;         // [B][H][capacity]
  float* out;             // as w; may be w
  long capacity;
  unsigned splits;        // workgroups that share a head's tokens
};

struct KvEvict {
  KvView c;
  const int32_t* lengths;
  const float* w;           // [B][H][capacity]
  long capacity;
  const int32_t* new_pages; // [B][new_width]
  int new_width, budget, recent, limit, B;
  int32_t* out_table;       // [B][width]
  int32_t* out_lengths;     // [B]
  float* out_w;             // [B][H][capacity]
  int32_t* kept;            // [B][H][budget]
  int tiles;                // workgroups that share a head's choice (kv_evict_tiles)
  uint32_t* scratch;        // [B][H][tiles][kEvictWords] if there are several
};

// The weights that a workgroup of the choice holds; the counts by the first 11
// bits and the list of those weights that workgroups of the same row tell each
// other, and with two more counts and two findings what that takes.
constexpr int kEvictTile = 16384, kEvictBins = 2048, kEvictList = 2044;
constexpr int kEvictWords = kEvictBins + kEvictList + 4;
inline long kv_evict_tiles(const KvView& c) { return ((static_cast<long>(c.width) << c.pshift) + kEvictTile - 1) / kEvictTile; }

hipError_t launch_kv_weights(const KvWeights& p, int dtype, int fmt, hipStream_t s);
hipError_t launch_kv_evict(const KvEvict& p, int fmt, hipStream_t s);

}  // namespace sv
