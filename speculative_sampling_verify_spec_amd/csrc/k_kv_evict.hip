// Eviction of the cached tokens that gathered the least weight: choosing what
// stays, and moving it to new pages.
#include "sv_budget.h"
#include "sv_device.h"
#include "sv_mfma.h"

namespace sv {

namespace {

using frag::lds_barrier;

constexpr int kSBlock = 1024, kSWaves = kSBlock / kWave;
constexpr int kBins = 2048;
constexpr int kGroups = 4, kTile = kGroups * 4 * kSBlock;  // groups of four weights a thread holds; weights of a tile
constexpr int kList = 8192;                                // weights kept in LDS for the last digit

// Weights as integers that order as they do (0 has one sign); NaN is below all.
__device__ inline uint32_t weight_key(float w) {
  const uint32_t u = w == 0.f ? 0u : __float_as_uint(w);
  if (w != w) return 0;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One workgroup per sequence and head: which positions stay.  The weight of
// the last one to stay is found by its digits (11, 11 and 10 bits, from the
// highest): a pass counts the weights by their next digit among those that
// agree with the digits found.  What is above that weight stays, and of those
// equal to it the first ones.  A thread holds 16 weights; up to 16384 stay in
// registers from the first pass to the last, longer rows are read again for
// the second digit and at the end (for the third if more than 8192 weights
// agree in the first).
__global__ __launch_bounds__(kSBlock) void k_kv_select(KvEvict p) {
  const KvView& c = p.c;
  const int h = blockIdx.x, tid = threadIdx.x, lane = tid % kWave, w = __builtin_amdgcn_readfirstlane(tid / kWave);
  const long b = blockIdx.y;
  const int len = kv_len(c, p.lengths, b);
  const bool cut = len > p.limit;
  const long base = (b * c.H + h) * p.capacity;
  const float* const row = p.w + base;
  float* const out_row = p.out_w + base;
  int32_t* const kept = p.kept + (b * c.H + h) * static_cast<long>(p.budget);
  const int after = cut ? p.budget : len;

  // weights 4 (tid + 1024 j) .. of a tile; behind the row 0
  struct __attribute__((packed, aligned(4))) Four { float x[4]; };
  Four v[kGroups];
  auto load = [&](int tile) {
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      const int at = tile * kTile + 4 * (tid + j * kSBlock);
      if (at + 4 <= len) v[j] = *reinterpret_cast<const Four*>(row + at);
      else
#pragma unroll
        for (int k = 0; k < 4; ++k) v[j].x[k] = at + k < len ? row[at + k] : 0.f;
    }
  };
  // use(position, weight): of a tile's existing weights
  auto each = [&](int tile, auto&& use) {
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      if (tile * kTile + 4 * j * kSBlock >= len) break;
      const int at = tile * kTile + 4 * (tid + j * kSBlock);
#pragma unroll
      for (int k = 0; k < 4; ++k) use(at + k, v[j].x[k]);
    }
  };
  const int ntile = (len + kTile - 1) / kTile;
  if (ntile) load(0);

  if (h == 0) {
    if (tid == 0) p.out_lengths[b] = after;
    for (int i = tid; i < c.width; i += kSBlock)
      p.out_table[b * c.width + i] = !cut ? c.table[b * c.width + i] : i < p.new_width ? p.new_pages[b * p.new_width + i] : -1;
  }
  for (long i = after + tid; i < p.capacity; i += kSBlock) out_row[i] = 0.f;
  if (!cut) {
    for (int t = 0; t < ntile; ++t) {
      if (t) load(t);
      each(t, [&](int at, float x) {
        if (at < len) out_row[at] = x;
      });
    }
    for (int i = tid; i < p.budget; i += kSBlock) kept[i] = -1;
    return;
  }

  const int n = len - p.recent;  // the positions to choose among
  int need = p.budget - p.recent;
  const bool some = need > 0;
  __shared__ uint32_t hist[kBins], list[kList];
  __shared__ uint32_t wave_at[kSWaves], digit_found, rest_found, listed;
  uint32_t found = 0;  // the digits found
  if (some) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t mask = pass == 0 ? 0u : pass == 1 ? ~0u << 21 : ~0u << 10, digit = pass == 2 ? 1023u : 2047u;
      hist[tid] = hist[tid + kSBlock] = 0;
      if (tid == 0 && pass < 2) listed = 0;
      __syncthreads();
      auto count = [&](uint32_t key) { atomicAdd(&hist[(key >> shift) & digit], 1u); };
      if (pass == 2 && ntile > 1 && listed <= kList) {
        for (uint32_t i = tid; i < listed; i += kSBlock)
          if ((list[i] & mask) == found) count(list[i]);
      } else {
#pragma unroll 1
        for (int t = 0; t < ntile; ++t) {
          if (ntile > 1) load(t);
          each(t, [&](int at, float x) {
            const uint32_t key = weight_key(x);
            const bool agrees = at < n && (key & mask) == found;
            if (agrees) count(key);
            if (pass == 1 && ntile > 1) {
              const uint64_t m = __ballot(agrees);
              if (!m) return;
              uint32_t first = 0;
              if (lane == 0) first = atomicAdd(&listed, static_cast<uint32_t>(__popcll(m)));
              const uint32_t i = __builtin_amdgcn_readfirstlane(first) +
                                 __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(m >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(m), 0u));
              if (agrees && i < kList) list[i] = key;
            }
          });
        }
      }
      __syncthreads();
      // the highest digit with `need` weights at and above it: a thread has two bins, counted from the top
      const int top = kBins - 1 - 2 * tid;
      const uint32_t x0 = hist[top], x1 = hist[top - 1];
      uint32_t sum = x0 + x1;
#pragma unroll
      for (int d = 1; d < kWave; d *= 2) {
        const uint32_t y = __shfl_up(sum, d, kWave);
        if (lane >= d) sum += y;
      }
      if (lane == kWave - 1) wave_at[w] = sum;
      __syncthreads();
      for (int i = 0; i < w; ++i) sum += wave_at[i];
      const uint32_t above = sum - x0 - x1;  // weights with a higher digit than this thread's
      if (above < static_cast<uint32_t>(need) && sum >= static_cast<uint32_t>(need)) {
        const bool first = above + x0 >= static_cast<uint32_t>(need);
        digit_found = first ? top : top - 1;
        rest_found = first ? above : above + x0;
      }
      __syncthreads();
      found |= digit_found << shift;
      need -= static_cast<int>(rest_found);
    }
  }

  // `need` of the weights equal to `found` stay, the first ones, and all above.
  // Positions of a tile go up with the group, the wave, the lane and the place
  // in the four: a count for each group and wave, scanned by every wave.
  const uint32_t last = static_cast<uint32_t>(need);
  uint32_t out = 0, ties = 0;  // what stays above, and the equal weights, before the tile
  __shared__ uint32_t counts[2][kGroups * kSWaves];
  static_assert(kGroups * kSWaves == kWave, "a lane per group and wave");
#pragma unroll 1
  for (int t = 0; t < ntile; ++t) {
    if (ntile > 1) load(t);
    uint32_t over = 0, tie = 0;  // bit 4 j + k
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      const int at = t * kTile + 4 * (tid + j * kSBlock);
      uint32_t mine = 0;  // counts of the group's four: above, and equal in the upper half
      if (t * kTile + 4 * j * kSBlock < len) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t key = weight_key(v[j].x[k]);
          const bool chosen = at + k < n;
          const bool o = at + k < len && (!chosen || (some && key > found)), e = chosen && some && key == found;
          over |= o ? 1u << (4 * j + k) : 0u;
          tie |= e ? 1u << (4 * j + k) : 0u;
          mine += static_cast<uint32_t>(__popcll(__ballot(o))) + (static_cast<uint32_t>(__popcll(__ballot(e))) << 16);
        }
      }
      if (lane == 0) counts[t & 1][j * kSWaves + w] = mine;
    }
    __syncthreads();
    const uint32_t own = counts[t & 1][lane];  // at most 16384 in all: the halves do not meet
    uint32_t upto = own;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
      const uint32_t y = __shfl_up(upto, d, kWave);
      if (lane >= d) upto += y;
    }
    const uint32_t before = upto - own;
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      if (t * kTile + 4 * j * kSBlock >= len) break;
      const int at = t * kTile + 4 * (tid + j * kSBlock);
      const uint32_t x = __builtin_amdgcn_readlane(before, j * kSWaves + w);
      uint32_t equal = ties + (x >> 16);  // equal weights before this lane's
      uint32_t rank = out + (x & 0xffffu);
      const uint32_t o = over >> (4 * j) & 15u, e = tie >> (4 * j) & 15u;
      auto lanes_before = [&](uint32_t bits) {
        uint32_t sum = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint64_t m = __ballot(bits >> k & 1u);
          sum = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(m >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(m), sum));
        }
        return sum;
      };
      equal += lanes_before(e);
      rank += lanes_before(o) + min(equal, last);  // of the equal ones, the first `last` stay
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool eq = e >> k & 1u, stays = (o >> k & 1u) || (eq && equal < last);
        equal += eq ? 1u : 0u;
        if (stays) {
          kept[rank] = at + k;
          out_row[rank] = v[j].x[k];
          ++rank;
        }
      }
    }
    const uint32_t all = __builtin_amdgcn_readlane(upto, kWave - 1);
    out += all & 0xffffu;
    ties += all >> 16;
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

// What a token's codes are multiplied by; finite, so that a code of 0 stays 0.
__device__ inline float code_ratio(float from, float to) { return fminf(from / to, 0x1.fffffep127f); }

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
// two.  V pages have a channel's tokens side by side: a lane takes a channel
// and loads 16 tokens of it, of which it puts those that stay into LDS one
// after the other; which ones they are is the same for all lanes, so that this
// costs one LDS write for a token and 64 channels.
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
  const int to = p.new_pages[b * p.new_width + col], first = kept[0];
  const int at_k = tid < n ? kept[tid] : -1, at_v = lane < own ? kept[t0 + lane] : -1;
  if (first < 0 || to < 0 || to >= c.pages) return;  // not cut, or no page to move to
  const int page_k = at_k < 0 ? -1 : kv_page(c, b, at_k >> c.pshift), page_v = at_v < 0 ? -1 : kv_page(c, b, at_v >> c.pshift);
  __shared__ size_t row_at[128];    // start of a token's row of K codes, ~0: no page
  __shared__ __align__(16) float unit_k[128], unit_v[128];  // the scales
  __shared__ float waves[2][kMWaves];
  extern __shared__ __align__(16) uint8_t codes[];  // V: [D][v_row(P)]
  const size_t bytes = static_cast<size_t>(P) * D, dst = (static_cast<size_t>(to) * c.H + h) * bytes;
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
  // ---- V: into LDS; the wave's tokens in runs that lie in the same 16 tokens
  // of a page, four of which are loaded before the first is needed ----
  const int row = v_row(P);
  const int mine = page_v < 0 ? -1 : at_v & (P - 1);
  const uint64_t mine_at = mine < 0 ? 0 : (static_cast<size_t>(page_v) * c.H + h) * bytes + (mine & ~15);
  const uint32_t at_lo = static_cast<uint32_t>(mine_at), at_hi = static_cast<uint32_t>(mine_at >> 32);
  const int prev = __shfl_up(mine, 1, kWave);
  const uint32_t prev_lo = __shfl_up(at_lo, 1, kWave), prev_hi = __shfl_up(at_hi, 1, kWave);
  uint64_t left = __ballot(lane < own && (lane == 0 || mine < 0 || prev < 0 || prev_lo != at_lo || prev_hi != at_hi));
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
  if (tid < P) {
    unit_k[tid] = ks;
    unit_v[tid] = vs;
  }
  __syncthreads();
  // ---- the new scales ----
  float top_k = 0.f, top_v = 0.f, u[kMost];
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int e = tid + i * kMBlock;
    u[i] = e < all ? unit_k[e * inv >> 16] : 0.f;
    top_k = fmaxf(top_k, largest16<FMT>(x[i]) * u[i]);
  }
  // words of four codes; of a row's, the last ones may be behind the last token
  const int wshift = c.pshift - 2, words = 1 << wshift;
  for (int e = tid; e < D << wshift; e += kMBlock) {
    const int d = e >> wshift, t = 4 * (e & (words - 1));
    if (t >= n) continue;
    float f[4];
    kv_decode4<FMT>(*reinterpret_cast<const uint32_t*>(&codes[d * row + t]), f);
    const float4 y = *reinterpret_cast<const float4*>(&unit_v[t]);  // 0 behind the last token
    top_v = fmaxf(fmaxf(top_v, fmaxf(fabsf(f[0]) * y.x, fabsf(f[1]) * y.y)), fmaxf(fabsf(f[2]) * y.z, fabsf(f[3]) * y.w));
  }
#pragma unroll
  for (int d = 32; d > 0; d /= 2) {
    top_k = fmaxf(top_k, __shfl_xor(top_k, d, kWave));
    top_v = fmaxf(top_v, __shfl_xor(top_v, d, kWave));
  }
  if (lane == 0) {
    waves[0][w] = top_k;
    waves[1][w] = top_v;
  }
  __syncthreads();
  auto scale_of = [&](const float* m) {
    return kv_scale<FMT>(fminf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), 0x1.fffffep127f));
  };
  const float sk = scale_of(waves[0]), sv = scale_of(waves[1]);
  if (tid == 0) {
    c.ks[static_cast<size_t>(to) * c.H + h] = sk;
    c.vs[static_cast<size_t>(to) * c.H + h] = sv;
  }
  if (tid < P) unit_v[tid] = code_ratio(unit_v[tid], sv);
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int e = tid + i * kMBlock;
    if (e < all) {
      const float r = code_ratio(u[i], sk);
      *reinterpret_cast<uint4*>(c.kp + dst + 16 * static_cast<size_t>(e)) =
          make_uint4(kv_rescale4<FMT>(x[i].x, r), kv_rescale4<FMT>(x[i].y, r), kv_rescale4<FMT>(x[i].z, r),
                     kv_rescale4<FMT>(x[i].w, r));
    }
  }
  lds_barrier();
  for (int e = tid; e < D << wshift; e += kMBlock) {
    const int d = e >> wshift, t = 4 * (e & (words - 1));
    if (t >= n) continue;
    float f[4];
    kv_decode4<FMT>(*reinterpret_cast<const uint32_t*>(&codes[d * row + t]), f);
    const float4 y = *reinterpret_cast<const float4*>(&unit_v[t]);
    f[0] *= y.x;
    f[1] *= y.y;
    f[2] *= y.z;
    f[3] *= y.w;
    const uint32_t v = kv_encode4<FMT>(f);
    uint8_t* const out = c.vp + dst + static_cast<size_t>(d) * P + t;
    if (t + 4 <= n) *reinterpret_cast<uint32_t*>(out) = v;
    else
      for (int i = 0; t + i < n; ++i) out[i] = static_cast<uint8_t>(v >> (8 * i));
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
  hipLaunchKernelGGL(k_kv_select, dim3(p.c.H, p.B), dim3(kSBlock), 0, st, p);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  return fmt == SPECV_E4M3 ? launch_move<SPECV_E4M3>(p, st) : launch_move<SPECV_I8>(p, st);
}

}  // namespace sv
