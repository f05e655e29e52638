// Eviction of the cached tokens that gathered the least weight: choosing what
// stays, and moving it to new pages.
#include "sv_budget.h"
#include "sv_device.h"

namespace sv {

namespace {

constexpr int kSBlock = 1024, kSWaves = kSBlock / kWave;
constexpr int kBins = 2048;

// Weights as integers that order as they do (0 has one sign); NaN is below all.
__device__ inline uint32_t weight_key(float w) {
  const uint32_t u = w == 0.f ? 0u : __float_as_uint(w);
  if (w != w) return 0;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One workgroup per sequence and head: which positions stay.  The weight that
// the last one to stay has is found by its digits (11, 11 and 10 bits, from the
// highest): a pass counts the weights by their next digit among those that
// agree with the digits found.  Then every wave goes through a range of
// positions of its own, first counting and then writing what stays, in order.
__global__ __launch_bounds__(kSBlock) void k_kv_select(KvEvict p) {
  const KvView& c = p.c;
  const int h = blockIdx.x, tid = threadIdx.x, lane = tid % kWave, w = tid / kWave;
  const long b = blockIdx.y;
  const int len = kv_len(c, p.lengths, b);
  const bool cut = len > p.limit;
  const long base = (b * c.H + h) * p.capacity;
  int32_t* const kept = p.kept + (b * c.H + h) * static_cast<long>(p.budget);
  const int after = cut ? p.budget : len;
  if (h == 0) {
    if (tid == 0) p.out_lengths[b] = after;
    for (int i = tid; i < c.width; i += kSBlock)
      p.out_table[b * c.width + i] = !cut ? c.table[b * c.width + i] : i < p.new_width ? p.new_pages[b * p.new_width + i] : -1;
  }
  for (long i = after + tid; i < p.capacity; i += kSBlock) p.out_w[base + i] = 0.f;
  if (!cut) {
    for (int i = tid; i < len; i += kSBlock) p.out_w[base + i] = p.w[base + i];
    for (int i = tid; i < p.budget; i += kSBlock) kept[i] = -1;
    return;
  }
  const int n = len - p.recent;  // the positions to choose among
  int need = p.budget - p.recent;
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t wave_at[kSWaves], digit_found, rest_found;
  uint32_t found = 0, mask = 0;  // the digits found
  if (need > 0) {
    int shift = 21, bits = 11;
    for (int pass = 0; pass < 3; ++pass) {
      for (int i = tid; i < kBins; i += kSBlock) hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < n; i += kSBlock) {
        const uint32_t k = weight_key(p.w[base + i]);
        if ((k & mask) == found) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1u);
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
      mask |= ((1u << bits) - 1) << shift;
      need -= static_cast<int>(rest_found);
      shift -= pass == 0 ? 11 : 10;
      bits = pass == 0 ? 11 : 10;
      __syncthreads();
    }
  }
  // `need` of the weights equal to `found` stay, the first ones, and all above
  const bool some = p.budget > p.recent;
  const int per = ((len + kSWaves - 1) / kSWaves + kWave - 1) / kWave * kWave;
  const int i0 = min(w * per, len), i1 = min(i0 + per, len);
  uint32_t more = 0, equal = 0;
  for (int i = i0; i < i1; i += kWave) {
    const int at = i + lane;
    const uint32_t k = at < n ? weight_key(p.w[base + at]) : 0u;
    more += __popcll(__ballot(at < i1 && (at >= n || (some && k > found))));
    equal += __popcll(__ballot(at < n && at < i1 && some && k == found));
  }
  __shared__ uint32_t more_of[kSWaves], equal_of[kSWaves];
  if (lane == 0) {
    more_of[w] = more;
    equal_of[w] = equal;
  }
  __syncthreads();
  uint32_t out = 0, ties = 0;  // what stays before, and the equal weights before
  for (int i = 0; i < w; ++i) {
    out += more_of[i];
    ties += equal_of[i];
  }
  out += min(ties, static_cast<uint32_t>(need));
  const uint64_t below = (1ull << lane) - 1;
  for (int i = i0; i < i1; i += kWave) {
    const int at = i + lane;
    const float x = at < i1 ? p.w[base + at] : 0.f;
    const uint32_t k = weight_key(x);
    const bool over = at < i1 && (at >= n || (some && k > found)), tie = at < n && at < i1 && some && k == found;
    const uint64_t tied = __ballot(tie);
    const bool stays = over || (tie && ties + __popcll(tied & below) < static_cast<uint32_t>(need));
    const uint64_t staying = __ballot(stays);
    if (stays) {
      const uint32_t r = out + __popcll(staying & below);
      kept[r] = at;
      p.out_w[base + r] = x;
    }
    out += __popcll(staying);
    ties += __popcll(tied);
  }
}

constexpr int kMBlock = 256;

// Sixteen codes' largest finite magnitude, as a value in units of their scale.
template <int FMT>
__device__ inline float largest16(const uint4& v) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[4];
    kv_decode4<FMT>(u[i], f);
#pragma unroll
    for (int j = 0; j < 4; ++j) m = fmaxf(m, fabsf(f[j]));  // NaN does not count
  }
  return m;
}

__device__ inline float block_max(float x, float* at) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) x = fmaxf(x, __shfl_xor(x, d, kWave));
  if (threadIdx.x % kWave == 0) at[threadIdx.x / kWave] = x;
  __syncthreads();
  return fmaxf(fmaxf(at[0], at[1]), fmaxf(at[2], at[3]));
}

// What a token's codes are multiplied by; finite, so that a code of 0 stays 0.
__device__ inline float code_ratio(float from, float to) { return fminf(from / to, 0x1.fffffep127f); }

// One workgroup per sequence, head, new page and K or V: gathers the tokens
// that stay, finds the block's new scale (as an append of them would) and
// writes their codes in its units.
template <int FMT>
__global__ __launch_bounds__(kMBlock) void k_kv_move(KvEvict p) {
  const KvView& c = p.c;
  const int col = blockIdx.x % static_cast<unsigned>(p.new_width), is_v = blockIdx.x / static_cast<unsigned>(p.new_width);
  const int h = blockIdx.y, tid = threadIdx.x;
  const long b = blockIdx.z;
  if (kv_len(c, p.lengths, b) <= p.limit) return;
  const int to = p.new_pages[b * p.new_width + col];
  if (to < 0 || to >= c.pages) return;
  const int n = min(p.budget - col * c.P, c.P), D = c.D, P = c.P;
  __shared__ int from[128];      // page of a token, -1: none
  __shared__ int slot[128];      // its place there
  __shared__ float unit[128];    // its scale
  __shared__ float waves[kMBlock / kWave];
  __shared__ __align__(16) uint8_t codes[128 * 256];
  if (tid < P) {
    int page = -1, at = 0;
    if (tid < n) {
      at = p.kept[(b * c.H + h) * static_cast<long>(p.budget) + col * P + tid];
      page = at < 0 ? -1 : kv_page(c, b, at >> c.pshift);
    }
    from[tid] = page;
    slot[tid] = at & (P - 1);
    unit[tid] = page < 0 ? 0.f : (is_v ? c.vs : c.ks)[static_cast<size_t>(page) * c.H + h];
  }
  __syncthreads();
  const size_t blk = static_cast<size_t>(P) * D, dst = (static_cast<size_t>(to) * c.H + h) * blk;
  float top = 0.f;
  if (!is_v) {
    const int per = D / 16;  // pieces of 16 codes of a token
    for (int e = tid; e < n * per; e += kMBlock) {
      const int t = e / per, d = e - t * per;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (from[t] >= 0)
        x = *reinterpret_cast<const uint4*>(c.kp + (static_cast<size_t>(from[t]) * c.H + h) * blk + static_cast<size_t>(slot[t]) * D + 16 * d);
      *reinterpret_cast<uint4*>(&codes[16 * e]) = x;
      top = fmaxf(top, largest16<FMT>(x) * unit[t]);
    }
    top = block_max(top, waves);
    const float s = kv_scale<FMT>(fminf(top, 0x1.fffffep127f));
    if (tid == 0) c.ks[static_cast<size_t>(to) * c.H + h] = s;
    for (int e = tid; e < n * per; e += kMBlock) {
      uint4 x = *reinterpret_cast<const uint4*>(&codes[16 * e]);
      const float r = code_ratio(unit[e / per], s);
      x = make_uint4(kv_rescale4<FMT>(x.x, r), kv_rescale4<FMT>(x.y, r), kv_rescale4<FMT>(x.z, r), kv_rescale4<FMT>(x.w, r));
      *reinterpret_cast<uint4*>(c.kp + dst + 16 * e) = x;
    }
  } else {
    // [D][P]: a lane takes a token, whose codes are P bytes apart
    for (int e = tid; e < P * D; e += kMBlock) {
      const int t = e & (P - 1), d = e >> c.pshift;
      uint8_t x = 0;
      if (from[t] >= 0) x = c.vp[(static_cast<size_t>(from[t]) * c.H + h) * blk + static_cast<size_t>(d) * P + slot[t]];
      codes[e] = x;
      float f[4];
      kv_decode4<FMT>(x, f);
      top = fmaxf(top, fabsf(f[0]) * unit[t]);
    }
    top = block_max(top, waves);
    const float s = kv_scale<FMT>(fminf(top, 0x1.fffffep127f));
    if (tid == 0) c.vs[static_cast<size_t>(to) * c.H + h] = s;
    for (int e = tid; e < P * D / 4; e += kMBlock) {
      const int t = 4 * e & (P - 1);
      if (t >= n) continue;
      float f[4];
      kv_decode4<FMT>(*reinterpret_cast<const uint32_t*>(&codes[4 * e]), f);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] *= code_ratio(unit[t + i], s);
      const uint32_t x = kv_encode4<FMT>(f);
      if (t + 4 <= n) *reinterpret_cast<uint32_t*>(c.vp + dst + 4 * e) = x;
      else
        for (int i = 0; t + i < n; ++i) c.vp[dst + 4 * e + i] = static_cast<uint8_t>(x >> (8 * i));
    }
  }
}

}  // namespace

hipError_t launch_kv_evict(const KvEvict& p, int fmt, hipStream_t st) {
  hipLaunchKernelGGL(k_kv_select, dim3(p.c.H, p.B), dim3(kSBlock), 0, st, p);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  const dim3 grid(2 * p.new_width, p.c.H, p.B);
  if (fmt == SPECV_E4M3) hipLaunchKernelGGL((k_kv_move<SPECV_E4M3>), grid, dim3(kMBlock), 0, st, p);
  else hipLaunchKernelGGL((k_kv_move<SPECV_I8>), grid, dim3(kMBlock), 0, st, p);
  return hipGetLastError();
}

}  // namespace sv
