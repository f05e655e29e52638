// Eviction of the cached tokens that gathered the least weight: choosing what
// stays, and moving it to new pages.
#include <type_traits>

#include "sv_budget.h"
#include "sv_device.h"
#include "sv_mfma.h"

namespace sv {

namespace {

using frag::lds_barrier;

constexpr int kSBlock = 1024, kSWaves = kSBlock / kWave;
constexpr int kGroups = 4, kTile = kEvictTile;  // groups of four weights a thread holds; weights of a workgroup
static_assert(kTile == kGroups * 4 * kSBlock, "a workgroup's weights are in its registers");
constexpr int kBins = kEvictBins, kList = kEvictList;

// Weights as integers that order as they do (0 has one sign); NaN is below all.
__device__ inline uint32_t weight_key(float w) {
  const uint32_t u = w == 0.f ? 0u : __float_as_uint(w);
  if (w != w) return 0;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Inclusive prefix sum over the lanes of a wave: in rows of 16 lanes, then + the rows' totals.
__device__ inline uint32_t lanes_upto(uint32_t v) {
  int s = static_cast<int>(v);
  s += dpp_i32<0x111, 0xf>(static_cast<int>(v));
  s += dpp_i32<0x112, 0xf>(static_cast<int>(v));
  s += dpp_i32<0x113, 0xf>(static_cast<int>(v));
  s += dpp_i32<0x114, 0xf, 0xe>(s);
  s += dpp_i32<0x118, 0xf, 0xc>(s);
  s += dpp_i32<0x142, 0xa>(s);
  s += dpp_i32<0x143, 0xc>(s);
  return static_cast<uint32_t>(s);
}

__device__ inline uint32_t lane_of(uint32_t v, int lane) { return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), lane)); }

// How many of the lanes before this one, added to `sum`.
__device__ inline uint32_t lanes_before(uint64_t m, uint32_t sum) {
  return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(m >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(m), sum));
}

// A sequence's head in the choice: its weights, and what is to be chosen.
struct Choice {
  const float* row;
  float* out_row;
  int32_t* kept;
  int len, n;     // positions, and the first n of them to choose among
  int need;       // how many
  bool cut;
  long pair;
};
__device__ inline Choice choice(const KvEvict& p, long b, int h) {
  Choice x;
  x.len = kv_len(p.c, p.lengths, b);
  x.cut = x.len > p.limit;
  x.n = x.len - p.recent;
  x.need = p.budget - p.recent;
  x.pair = b * p.c.H + h;
  x.row = p.w + x.pair * p.capacity;
  x.out_row = p.out_w + x.pair * p.capacity;
  x.kept = p.kept + x.pair * static_cast<long>(p.budget);
  return x;
}

// A workgroup's weights: a thread has 4 (tid + 1024 j) .. + 3 of a tile.  What
// is behind the row, or behind its capacity, is any number.
struct Held {
  struct __attribute__((packed, aligned(4))) Four { float x[4]; };
  Four v[kGroups];
  int at0;
  __device__ void load(const float* row, int len, long capacity, int tile) {
    at0 = tile * kTile;
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      if (at0 + 4 * j * kSBlock >= len) break;
      const int at = place(j);
      if (at0 + 4 * (j + 1L) * kSBlock <= capacity) {
        v[j] = *reinterpret_cast<const Four*>(row + at);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[j].x[k] = row[min(static_cast<long>(at + k), capacity - 1)];
      }
    }
  }
  __device__ int place(int j) const { return at0 + 4 * (static_cast<int>(threadIdx.x) + j * kSBlock); }
  // use(position, weight), by all lanes of a wave at once
  template <class F>
  __device__ void each(int len, F&& use) const {
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      if (at0 + 4 * j * kSBlock >= len) break;
#pragma unroll
      for (int k = 0; k < 4; ++k) use(place(j) + k, v[j].x[k]);
    }
  }
};

// What the workgroups of a long row tell each other (KvEvict.scratch): their
// counts by the first digit; then how many of their weights are above that
// digit, and those that have it (if they are not too many).
struct Told {
  uint32_t over, same, digit, need;
};
__device__ inline uint32_t* bins_of(const KvEvict& p, long pair, int tile) {
  return p.scratch + (pair * p.tiles + tile) * kEvictWords;
}
__device__ inline uint32_t* list_of(const KvEvict& p, long pair, int tile) { return bins_of(p, pair, tile) + kBins; }
__device__ inline Told* told_of(const KvEvict& p, long pair, int tile) {
  return reinterpret_cast<Told*>(list_of(p, pair, tile) + kList);
}

// Long rows, first: a workgroup per 16384 weights counts them by their highest 11 bits.
__global__ __launch_bounds__(kSBlock) void k_kv_count(KvEvict p) {
  const Choice x = choice(p, blockIdx.z, blockIdx.y);
  const int tile = blockIdx.x, tid = threadIdx.x;
  if (!x.cut || tile * kTile >= x.len) return;
  Held v;
  v.load(x.row, x.len, p.capacity, tile);
  __shared__ uint32_t hist[kBins][2];  // even and odd lanes: fewer of a wave at the same place
  static_assert(kBins == 2 * kSBlock, "two bins a thread");
#pragma unroll
  for (int i = 0; i < 4; ++i) (&hist[0][0])[tid + i * kSBlock] = 0;
  __syncthreads();
  v.each(x.len, [&](int at, float w) {
    if (at < x.n) atomicAdd(&hist[weight_key(w) >> 21][tid & 1], 1u);
  });
  __syncthreads();
  uint32_t* const bins = bins_of(p, x.pair, tile);
#pragma unroll
  for (int i = 0; i < 2; ++i) bins[tid + i * kSBlock] = hist[tid + i * kSBlock][0] + hist[tid + i * kSBlock][1];
}

// Long rows, second: every workgroup of a row finds the digit that the last
// weight to stay has, and lists its own weights that have it.
__global__ __launch_bounds__(kSBlock) void k_kv_list(KvEvict p) {
  const Choice x = choice(p, blockIdx.z, blockIdx.y);
  const int tile = blockIdx.x, tid = threadIdx.x, lane = tid % kWave, w = __builtin_amdgcn_readfirstlane(tid / kWave);
  if (!x.cut || tile * kTile >= x.len) return;
  Held v;
  v.load(x.row, x.len, p.capacity, tile);
  const int ntile = (x.len + kTile - 1) / kTile, top = kBins - 1 - 2 * tid;
  uint32_t x0 = 0, x1 = 0;  // a thread's two bins, counted from the top
#pragma unroll 8
  for (int t = 0; t < ntile; ++t) {
    const uint2 y = *reinterpret_cast<const uint2*>(bins_of(p, x.pair, t) + top - 1);
    x0 += y.y;
    x1 += y.x;
  }
  __shared__ uint32_t wave_at[kSWaves], digit, need, over, same;
  uint32_t upto = lanes_upto(x0 + x1);
  if (lane == kWave - 1) wave_at[w] = upto;
  if (tid == 0) {
    digit = kBins;  // nothing to choose: none has it
    need = over = same = 0;
  }
  __syncthreads();
  for (int i = 0; i < w; ++i) upto += wave_at[i];
  const uint32_t above = upto - x0 - x1, want = static_cast<uint32_t>(x.need);
  if (above < want && upto >= want) {
    const bool first = above + x0 >= want;
    digit = first ? top : top - 1;
    need = want - (first ? above : above + x0);
  }
  __syncthreads();
  uint32_t* const list = list_of(p, x.pair, tile);
  const uint32_t found = digit;
  uint32_t more = 0;
  v.each(x.len, [&](int at, float y) {
    const uint32_t key = weight_key(y);
    const bool chosen = at < x.n, agrees = chosen && key >> 21 == found;
    more += at < x.len && (!chosen || key >> 21 > found) ? 1u : 0u;
    const uint64_t m = __ballot(agrees);
    if (!m) return;
    uint32_t first = 0;
    if (lane == 0) first = atomicAdd(&same, static_cast<uint32_t>(__popcll(m)));  // in any order: they are only counted
    const uint32_t i = lanes_before(m, __builtin_amdgcn_readfirstlane(first));
    if (agrees && i < kList) list[i] = key;
  });
  more = lane_of(lanes_upto(more), kWave - 1);
  if (lane == 0 && more) atomicAdd(&over, more);
  __syncthreads();
  if (tid == 0) *told_of(p, x.pair, tile) = Told{over, same, found, need};
}

// One workgroup per sequence, head and 16384 positions: which of them stay.
// The weight of the last one to stay is found by its digits, from the highest:
// a pass counts the weights by their next 8 bits among those that agree with
// the digits found, in a table of its own, which every wave then looks through
// for itself.  What is above that weight stays, and of those equal to it the
// first ones.  Rows of up to 16384 weights are in the workgroup's registers
// (MANY false); 512 rows of up to 4096 take 15 us, the passes' chain, as 32 rows
// of 700 take 9.  Of longer ones the first 11 bits are known, and the weights
// that have them are listed by the workgroups of the row (or read again, where
// a workgroup has more of them than its list takes: where all weights are the same,
// every workgroup reads the whole row in every pass.  A call of 2 rows of up to
// 131072 takes 176 us then, of 1 of 278528 314 and of 1 of 2^20 1911, with weights
// spread over many powers of two 117, 129 and 385, with weights that decay as the
// logarithm of the position 85, 98 and 329).
template <bool MANY>
__global__ __launch_bounds__(kSBlock) void k_kv_select(KvEvict p) {
  const KvView& c = p.c;
  const int tile = MANY ? blockIdx.x : 0, h = blockIdx.y, tid = threadIdx.x, lane = tid % kWave;
  const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
  const long b = blockIdx.z;
  const Choice x = choice(p, b, h);
  const int after = x.cut ? p.budget : x.len, ntile = (x.len + kTile - 1) / kTile;
  Held v;
  v.load(x.row, x.len, p.capacity, tile);
  __shared__ uint32_t hist[4][256][4];  // a pass's counts, four lanes' apart: fewer of a wave at the same place
#pragma unroll
  for (int i = 0; i < 4; ++i) (&hist[i][0][0])[tid] = 0;
  if (h == 0 && tile == 0) {
    if (tid == 0) p.out_lengths[b] = after;
    for (int i = tid; i < c.width; i += kSBlock)
      p.out_table[b * c.width + i] = !x.cut ? c.table[b * c.width + i] : i < p.new_width ? p.new_pages[b * p.new_width + i] : -1;
  }
  const long end = MANY && tile + 1 < p.tiles ? (tile + 1L) * kTile : p.capacity;
  for (long i = max(static_cast<long>(after), static_cast<long>(tile) * kTile) + tid; i < end; i += kSBlock) x.out_row[i] = 0.f;
  if (!x.cut) {
    v.each(x.len, [&](int at, float y) {
      if (at < x.len) x.out_row[at] = y;
    });
    if (tile == 0)
      for (int i = tid; i < p.budget; i += kSBlock) x.kept[i] = -1;
    return;
  }
  if (tile >= ntile) return;

  uint32_t found = 0, need = static_cast<uint32_t>(x.need);
  const bool some = x.need > 0;
  uint32_t out = 0, ties = 0;  // what stays above, and the equal weights, before the tile
  if constexpr (MANY) {
    const Told mine = *told_of(p, x.pair, tile);
    found = mine.digit << 21;
    need = mine.need;
  }
  // the weights of the row's first tiles that may be the last to stay: use(key).
  // Lists are read eight at a time, a thread's two places of each: loads that
  // do not wait for each other; eight stay in registers for all passes.
  uint32_t same[8], key[8][2];
  auto read = [&](int t0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) same[i] = t0 + i < ntile ? told_of(p, x.pair, t0 + i)->same : 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t at = tid + j * kSBlock;
        key[i][j] = same[i] <= kList && at < same[i] ? list_of(p, x.pair, t0 + i)[at] : 0u;
      }
  };
  if (MANY && some) read(0);
  auto candidates = [&](int tiles, uint32_t mask, auto&& use) {
    if constexpr (MANY) {
      for (int t0 = 0; t0 < tiles; t0 += 8) {
        if (ntile > 8) read(t0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (t0 + i >= tiles) break;
          if (same[i] <= kList) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (static_cast<uint32_t>(tid + j * kSBlock) < same[i] && (key[i][j] & mask) == (found & mask)) use(key[i][j]);
            continue;
          }
          Held other;
          other.load(x.row, x.len, p.capacity, t0 + i);
          other.each(x.len, [&](int at, float y) {
            const uint32_t k = weight_key(y);
            if (at < x.n && (k & mask) == (found & mask)) use(k);
          });
        }
      }
    } else {
      v.each(x.len, [&](int at, float y) {
        const uint32_t key = weight_key(y);
        if (at < x.n && (key & mask) == (found & mask)) use(key);
      });
    }
  };
  static_assert(kList <= 2 * kSBlock, "two places a thread");
  __syncthreads();
  if (some) {
    constexpr int kPasses = MANY ? 3 : 4;
#pragma unroll MANY ? 1 : kPasses
    for (int pass = 0; pass < kPasses; ++pass) {
      const int upper = MANY ? 21 - 8 * pass : 32 - 8 * pass, shift = upper > 8 ? upper - 8 : 0;  // bits below those found
      const uint32_t mask = upper == 32 ? 0u : ~0u << upper;
      candidates(ntile, mask, [&](uint32_t key) { atomicAdd(&hist[pass][(key >> shift) & 255u & ~(mask >> shift)][lane & 3], 1u); });
      __syncthreads();
      // the highest digit with `need` weights at and above it: a lane has four, counted from the top
      uint32_t n[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 y = *reinterpret_cast<const uint4*>(&hist[pass][255 - 4 * lane - i][0]);
        n[i] = y.x + y.y + y.z + y.w;
        sum += n[i];
      }
      const uint32_t upto = lanes_upto(sum);
      const int at = __builtin_ctzll(__ballot(upto >= need));  // need is at most the count of all
      uint32_t above = lane_of(upto - sum, at);
      int digit = 255 - 4 * at;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const uint32_t y = lane_of(n[i], at);
        const bool next = above + y < need && digit == 255 - 4 * at - i;
        above += next ? y : 0u;
        digit -= next ? 1 : 0;
      }
      need -= above;
      found |= static_cast<uint32_t>(digit) << shift;
    }
  }
  // `need` of the weights equal to `found` stay, the first ones, and all above
  if constexpr (MANY) {
    __shared__ uint32_t before[2];
    if (tid < 2) before[tid] = 0;
    __syncthreads();
    uint32_t more = 0, equal = 0;
    for (int t = tid; t < tile; t += kSBlock) more += told_of(p, x.pair, t)->over;
    if (some)
      candidates(tile, ~0u << 21, [&](uint32_t key) {
        more += key > found ? 1u : 0u;
        equal += key == found ? 1u : 0u;
      });
    more = lane_of(lanes_upto(more), kWave - 1);
    equal = lane_of(lanes_upto(equal), kWave - 1);
    if (lane == 0) {
      atomicAdd(&before[0], more);
      atomicAdd(&before[1], equal);
    }
    __syncthreads();
    out = before[0];
    ties = before[1];
  }
  // Positions go up with the group, the wave, the lane and the place in the
  // four: a count for each group and wave, scanned by every wave.
  __shared__ uint32_t counts[kGroups * kSWaves];
  static_assert(kGroups * kSWaves == kWave, "a lane per group and wave");
  uint32_t over = 0, tie = 0;  // bit 4 j + k
#pragma unroll
  for (int j = 0; j < kGroups; ++j) {
    uint32_t mine = 0;  // counts of the group's four: above, and equal in the upper half
    if (v.at0 + 4 * j * kSBlock < x.len) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int at = v.place(j) + k;
        const uint32_t key = weight_key(v.v[j].x[k]);
        const bool chosen = at < x.n, o = at < x.len && (!chosen || (some && key > found)), e = chosen && some && key == found;
        over |= o ? 1u << (4 * j + k) : 0u;
        tie |= e ? 1u << (4 * j + k) : 0u;
        mine += static_cast<uint32_t>(__popcll(__ballot(o))) + (static_cast<uint32_t>(__popcll(__ballot(e))) << 16);
      }
    }
    if (lane == 0) counts[j * kSWaves + w] = mine;
  }
  __syncthreads();
  const uint32_t own = counts[lane], before = lanes_upto(own) - own;  // at most 16384 in all: the halves do not meet
#pragma unroll
  for (int j = 0; j < kGroups; ++j) {
    if (v.at0 + 4 * j * kSBlock >= x.len) break;
    const uint32_t y = lane_of(before, j * kSWaves + w), o = over >> (4 * j) & 15u, e = tie >> (4 * j) & 15u;
    uint32_t equal = ties + (y >> 16), rank = out + (y & 0xffffu);  // before this lane's
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      equal = lanes_before(__ballot(e >> k & 1u), equal);
      rank = lanes_before(__ballot(o >> k & 1u), rank);
    }
    rank += min(equal, need);  // of the equal ones, the first `need` stay
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool eq = e >> k & 1u, stays = (o >> k & 1u) || (eq && equal < need);
      equal += eq ? 1u : 0u;
      if (stays) {
        x.kept[rank] = v.place(j) + k;
        x.out_row[rank] = v.v[j].x[k];
        ++rank;
      }
    }
  }
}

constexpr int kMBlock = 256, kMWaves = kMBlock / kWave;

// Four codes' largest finite magnitude in units of their scale.
template <int FMT>
__device__ inline float largest4(uint32_t w) {
  float f[4];
  kv_decode4<FMT>(w, f);
  return fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));  // NaN does not count
}
template <int FMT>
__device__ inline float largest16(const uint4& v) {
  return fmaxf(fmaxf(largest4<FMT>(v.x), largest4<FMT>(v.y)), fmaxf(largest4<FMT>(v.z), largest4<FMT>(v.w)));
}

// What a token's codes are multiplied by, from its scale and the new one's
// reciprocal (a power of two too); finite, so that a code of 0 stays 0.
__device__ inline float code_ratio(float from, float per_to) { return fminf(from * per_to, kLargest<SPECV_F32>); }

// 1 / s of a power of two 2^-126 .. 2^126, exactly.
__device__ inline float reciprocal(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

// Bytes of a channel's row of V codes in LDS: whole words, an odd number of
// them, so that 64 channels' same token falls into 64 different banks.
__host__ __device__ inline int v_row(int P) { return P + 4; }

// One workgroup per sequence, head and new page: gathers the tokens that stay,
// finds the blocks' new scales (as an append of them would) and writes their
// codes in their units.  A workgroup's time is that of the loads that wait for
// each other, so there are three: the kept positions, their pages, and then
// codes and scales together.
//
// K rows are copied 16 bytes a thread and stay in its registers between the
// two.  V pages have a channel's tokens side by side.  Where many of them stay, a
// lane takes a channel and loads 16 tokens of it, of which it puts those that stay
// into LDS one after the other; which ones they are is the same for all lanes, so
// that this costs one LDS write for a token and 64 channels.  Where few stay, the
// loads are what counts: four lanes take a channel's 64 tokens, so that a request
// is of whole 64 bytes, and each puts its own into LDS.  Sequences cut the first
// and the second way (us a call; heads of 128): in pages of 128 tokens to a
// quarter 161 and 140, to an eighth 145 and 113, to a sixteenth (2 of up to
// 131072) 134 and 118; in pages of 64 lengths of 900 to 4096 to 1024 107 and 114,
// to a quarter 132 and 131, to an eighth 108 and 103, to a sixteenth 88 and 88.
//
// Bound by the lines of V that the kept tokens lie in, nearly all of them even
// if one token in 16 stays: 64 sequences of up to 4096 tokens to 1024 (8 heads
// of 128) 88 us, 4.1 TB/s; 2 of up to 131072 to 8192 74 us, 3.9 TB/s.
template <int FMT, int kMost>  // kMost: pieces of 16 K codes of a block that a thread has at most
__global__ __launch_bounds__(kMBlock) void k_kv_move(KvEvict p) {
  const KvView& c = p.c;
  const int col = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid % kWave;
  const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
  const long b = blockIdx.z;
  const int D = c.D, P = c.P, n = min(p.budget - col * P, P);
  const int32_t* const kept = p.kept + (b * c.H + h) * static_cast<long>(p.budget) + col * P;
  // a thread per token, and the tokens of a wave's share of V one a lane
  const int per = (n + kMWaves - 1) / kMWaves, t0 = min(w * per, n), own = min(per, n - t0);
  const int to = p.new_pages[b * p.new_width + col], first = kept[0], last = kept[n - 1];
  const int at_k = tid < n ? kept[tid] : -1, at_v = lane < own ? kept[t0 + lane] : -1;
  if (first < 0 || to < 0 || to >= c.pages) return;  // not cut, or no page to move to
  const int page_k = at_k < 0 ? -1 : kv_page(c, b, at_k >> c.pshift), page_v = at_v < 0 ? -1 : kv_page(c, b, at_v >> c.pshift);
  __shared__ size_t row_at[128];    // start of a token's row of K codes, ~0: no page
  __shared__ __align__(16) float unit_k[128], unit_v[128];  // the scales
  __shared__ float waves[2][kMWaves];
  extern __shared__ __align__(16) uint8_t codes[];  // V: [D][v_row(P)]
  const size_t bytes = static_cast<size_t>(P) * D;
  const size_t dst = (static_cast<size_t>(to) * c.H + h) * bytes;
  const size_t blk_k = static_cast<size_t>(max(page_k, 0)) * c.H + h;
  if (tid < P) row_at[tid] = page_k < 0 ? ~size_t(0) : blk_k * bytes + static_cast<size_t>(at_k & (P - 1)) * D;
  const float ks = tid < P && page_k >= 0 ? c.ks[blk_k] : 0.f, vs = tid < P && page_k >= 0 ? c.vs[blk_k] : 0.f;
  lds_barrier();
  // ---- K: into registers ----
  const int pieces = D / 16, all = n * pieces;
  const unsigned inv = 65536u / pieces + 1;  // e / pieces is e * inv >> 16 for e < 2048
  uint4 x[kMost];
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int e = tid + i * kMBlock, t = static_cast<int>(e * inv >> 16);
    x[i] = make_uint4(0, 0, 0, 0);
    if (e < all && row_at[t] != ~size_t(0)) x[i] = *reinterpret_cast<const uint4*>(c.kp + row_at[t] + 16 * (e - t * pieces));
  }
  // ---- V: into LDS; the wave's tokens in runs that lie in the same 16 tokens of a
  // page, or in the same 64 (or all of a smaller page) where few stay; some runs
  // are loaded before the first is needed ----
  constexpr int kFew = kMost > 2 ? 3 : 5;  // larger blocks gain from a third on, smaller ones from a fifth
  const bool few = P > 16 && last - first >= kFew * n;
  const int row = v_row(P), sshift = few ? min(c.pshift, 6) - 4 : 0, seg = 16 << sshift;
  const int mine = page_v < 0 ? -1 : at_v & (P - 1);
  const uint64_t mine_at = mine < 0 ? 0 : (static_cast<size_t>(page_v) * c.H + h) * bytes + (mine & ~(seg - 1));
  const uint32_t at_lo = static_cast<uint32_t>(mine_at), at_hi = static_cast<uint32_t>(mine_at >> 32);
  const int prev = __shfl_up(mine, 1, kWave);
  const uint32_t prev_lo = __shfl_up(at_lo, 1, kWave), prev_hi = __shfl_up(at_hi, 1, kWave);
  // places do not go up where a table holds a page more than once
  uint64_t left = __ballot(lane < own && (lane == 0 || mine < 0 || prev < 0 || mine <= prev || prev_lo != at_lo || prev_hi != at_hi));
  if (!few) {
    // a lane has a channel; the tokens that stay are the same for all lanes
    const int run = (D + kWave - 1) / kWave;  // blocks of 64 channels, at most 4
    constexpr int kRuns = 4;
    while (left) {
      uint64_t lo[kRuns][2], hi[kRuns][2];
      for (int half = 0; half < run; half += 2) {  // two blocks of channels at a time
        uint64_t rest = left;
#pragma unroll
        for (int k = 0; k < kRuns; ++k) {
#pragma unroll
          for (int i = 0; i < 2; ++i) lo[k][i] = hi[k][i] = 0;
          if (!rest) continue;
          const int s = __builtin_ctzll(rest);
          rest &= rest - 1;
          if (__builtin_amdgcn_readlane(mine, s) < 0) continue;
          const uint64_t from = static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(at_hi, s))) << 32 |
                                static_cast<uint32_t>(__builtin_amdgcn_readlane(at_lo, s));
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (half + i < run) {
              const int d = min((half + i) * kWave + lane, D - 1);
              const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(c.vp + from + static_cast<size_t>(d) * P);
              lo[k][i] = y.x;
              hi[k][i] = y.y;
            }
        }
        rest = left;
#pragma unroll
        for (int k = 0; k < kRuns; ++k) {
          if (!rest) continue;
          int t = __builtin_ctzll(rest);
          rest &= rest - 1;
          const int end = rest ? __builtin_ctzll(rest) : own;
          for (; t < end; ++t) {
            const int at = __builtin_amdgcn_readlane(mine, t);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (half + i < run) {
                const int d = (half + i) * kWave + lane;
                const uint64_t y = at & 8 ? hi[k][i] : lo[k][i];
                if (d < D) codes[d * row + t0 + t] = static_cast<uint8_t>(y >> (8 * (at & 7)));
              }
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kRuns; ++k) left &= left - 1;
    }
  } else {
    // lanes side by side have 16 tokens each of a channel, of which every lane puts its own into LDS
    const int part = lane & ((1 << sshift) - 1), chan = lane >> sshift;
    const int per_chunk = kWave >> sshift, chunks = (D + per_chunk - 1) / per_chunk;  // channels of a load, and loads
    constexpr int kRuns = 2, kChunks = kMost > 2 ? 4 : 2;
    while (left) {
      uint64_t from[kRuns], stay[kRuns];  // a run's place, and its tokens among those of the place
      int begin[kRuns];
      uint64_t rest = left;
#pragma unroll
      for (int k = 0; k < kRuns; ++k) {
        from[k] = stay[k] = 0;
        begin[k] = 0;
        if (!rest) continue;
        int t = __builtin_ctzll(rest);
        rest &= rest - 1;
        const int end = rest ? __builtin_ctzll(rest) : own;
        begin[k] = t0 + t;
        if (__builtin_amdgcn_readlane(mine, t) < 0) {  // no page: a zero
          for (int d = lane; d < D; d += kWave) codes[d * row + t0 + t] = 0;
          continue;
        }
        from[k] = static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(at_hi, t))) << 32 |
                  static_cast<uint32_t>(__builtin_amdgcn_readlane(at_lo, t));
        for (; t < end; ++t) stay[k] |= uint64_t(1) << (__builtin_amdgcn_readlane(mine, t) & (seg - 1));
      }
      for (int first = 0; first < chunks; first += kChunks) {
        uint64_t lo[kRuns][kChunks], hi[kRuns][kChunks];
#pragma unroll
        for (int k = 0; k < kRuns; ++k) {
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            lo[k][i] = hi[k][i] = 0;
            if (stay[k] && first + i < chunks) {
              const int d = min((first + i) * per_chunk + chan, D - 1);
              const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(c.vp + from[k] + static_cast<size_t>(d) * P + 16 * part);
              lo[k][i] = y.x;
              hi[k][i] = y.y;
            }
          }
        }
        auto keep = [&](auto run) {
          constexpr int k = decltype(run)::value;
          if (!stay[k]) return;
          uint32_t own16 = static_cast<uint32_t>(stay[k] >> (16 * part)) & 0xffffu;
          uint8_t* to = &codes[begin[k] + __popcll(stay[k] & ((uint64_t(1) << (16 * part)) - 1))];
          int most = 0;  // of a lane's
#pragma unroll
          for (int i = 0; i < 4; ++i) most = max(most, __popc(static_cast<uint32_t>(stay[k] >> (16 * i)) & 0xffffu));
          for (int n16 = 0; n16 < most; ++n16, ++to) {
            if (own16) {
              const int at = __builtin_ctz(own16);
#pragma unroll
              for (int i = 0; i < kChunks; ++i) {
                const int d = (first + i) * per_chunk + chan;
                const uint64_t y = at & 8 ? hi[k][i] : lo[k][i];
                const uint32_t z = static_cast<uint32_t>(at & 4 ? y >> 32 : y);
                if (first + i < chunks && d < D) to[d * row] = static_cast<uint8_t>(z >> (8 * (at & 3)));
              }
            }
            own16 &= own16 - 1;
          }
        };
        keep(std::integral_constant<int, 0>{});
        keep(std::integral_constant<int, 1>{});
      }
#pragma unroll
      for (int k = 0; k < kRuns; ++k) left &= left - 1;
    }
  }
  if (tid < P) {
    unit_k[tid] = ks;
    unit_v[tid] = vs;
  }
  lds_barrier();
  // ---- the new scales ----
  // A thread's words of four V codes, kMost * 4 at most, are a workgroup's
  // threads apart: of different channels, but always of the same four tokens.
  const int wshift = c.pshift - 2, vt = 4 * (tid & ((1 << wshift) - 1)), vall = D << wshift;
  auto word = [&](int e) {
    return e < vall && vt < n ? *reinterpret_cast<const uint32_t*>(&codes[(e >> wshift) * row + vt]) : 0u;
  };
  float most[4] = {0.f, 0.f, 0.f, 0.f};
  float top_k = 0.f, u[kMost];
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int e = tid + i * kMBlock;
    u[i] = e < all ? unit_k[e * inv >> 16] : 0.f;
    top_k = fmaxf(top_k, largest16<FMT>(x[i]) * u[i]);
  }
#pragma unroll
  for (int i = 0; i < 4 * kMost; ++i) {
    float f[4];
    kv_decode4<FMT>(word(tid + i * kMBlock), f);
#pragma unroll
    for (int k = 0; k < 4; ++k) most[k] = fmaxf(most[k], fabsf(f[k]));  // NaN does not count
  }
  const float4 uv = *reinterpret_cast<const float4*>(&unit_v[vt]);  // 0 behind the last token
  float top_v = fmaxf(fmaxf(most[0] * uv.x, most[1] * uv.y), fmaxf(most[2] * uv.z, most[3] * uv.w));
  top_k = wave_max(top_k);
  top_v = wave_max(top_v);
  if (lane == 0) {
    waves[0][w] = top_k;
    waves[1][w] = top_v;
  }
  lds_barrier();
#pragma unroll
  for (int i = 0; i < kMWaves; ++i) {
    top_k = fmaxf(top_k, waves[0][i]);
    top_v = fmaxf(top_v, waves[1][i]);
  }
  const float sk = kv_scale<FMT>(fminf(top_k, kLargest<SPECV_F32>)), sv = kv_scale<FMT>(fminf(top_v, kLargest<SPECV_F32>));
  if (tid == 0) {
    c.ks[static_cast<size_t>(to) * c.H + h] = sk;
    c.vs[static_cast<size_t>(to) * c.H + h] = sv;
  }
  // ---- the codes in their units: all in the format's range, unless a value passed that of 32 bits ----
  const float per_sk = reciprocal(sk), per_sv = reciprocal(sv);
  const float rv[4] = {code_ratio(uv.x, per_sv), code_ratio(uv.y, per_sv), code_ratio(uv.z, per_sv), code_ratio(uv.w, per_sv)};
  auto write = [&](auto encode) {
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      const int e = tid + i * kMBlock;
      const float r = code_ratio(u[i], per_sk), rk[4] = {r, r, r, r};
      if (e < all)
        *reinterpret_cast<uint4*>(c.kp + dst + 16 * static_cast<size_t>(e)) =
            make_uint4(encode(x[i].x, rk), encode(x[i].y, rk), encode(x[i].z, rk), encode(x[i].w, rk));
    }
#pragma unroll
    for (int i = 0; i < 4 * kMost; ++i) {
      const int e = tid + i * kMBlock;
      const uint32_t v = encode(word(e), rv);
      uint8_t* const out = c.vp + dst + static_cast<size_t>(e >> wshift) * P + vt;
      if (e < vall && vt + 4 <= n) *reinterpret_cast<uint32_t*>(out) = v;
      else if (e < vall)
        for (int k = 0; vt + k < n; ++k) out[k] = static_cast<uint8_t>(v >> (8 * k));
    }
  };
  auto product = [](uint32_t code, const float* r, float* f) {
    kv_decode4<FMT>(code, f);
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] *= r[k];
  };
  if (fmaxf(top_k, top_v) <= kLargest<SPECV_F32>) {
    write([&](uint32_t code, const float* r) {
      float f[4];
      product(code, r, f);
      return kv_encode4_finite<FMT>(f);  // NaN stays NaN in e4m3, and int8 has none
    });
  } else {
    write([&](uint32_t code, const float* r) {
      float f[4];
      product(code, r, f);
      return kv_encode4<FMT>(f);
    });
  }
}

template <int FMT, int M>
hipError_t launch_move_of(const KvEvict& p, hipStream_t st) {
  const size_t lds = static_cast<size_t>(p.c.D) * v_row(p.c.P);
  hipLaunchKernelGGL((k_kv_move<FMT, M>), dim3(p.new_width, p.c.H, p.B), dim3(kMBlock), lds, st, p);
  return hipGetLastError();
}

template <int FMT>
hipError_t launch_move(const KvEvict& p, hipStream_t st) {
  const int pieces = (p.c.P * p.c.D + 16 * kMBlock - 1) / (16 * kMBlock);  // 1 .. 8
  return pieces > 4   ? launch_move_of<FMT, 8>(p, st)
         : pieces > 2 ? launch_move_of<FMT, 4>(p, st)
         : pieces > 1 ? launch_move_of<FMT, 2>(p, st)
                      : launch_move_of<FMT, 1>(p, st);
}

}  // namespace

hipError_t launch_kv_evict(const KvEvict& p, int fmt, hipStream_t st) {
  const dim3 grid(p.tiles, p.c.H, p.B);
  if (p.tiles > 1) {
    hipLaunchKernelGGL(k_kv_count, grid, dim3(kSBlock), 0, st, p);
    hipLaunchKernelGGL(k_kv_list, grid, dim3(kSBlock), 0, st, p);
    hipLaunchKernelGGL((k_kv_select<true>), grid, dim3(kSBlock), 0, st, p);
  } else {
    hipLaunchKernelGGL((k_kv_select<false>), grid, dim3(kSBlock), 0, st, p);
  }
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  return fmt == SPECV_E4M3 ? launch_move<SPECV_E4M3>(p, st) : launch_move<SPECV_I8>(p, st);
}

}  // namespace sv
