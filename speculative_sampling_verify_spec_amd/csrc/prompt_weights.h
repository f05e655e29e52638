// The attention weight that a prompt's tokens gather from the prompt itself
// (the kernel template; k_prompt_<dim>.hip instantiate it):
//   w[j] = sum over the queries i >= j, and the query heads that share a key
//          head, of e^(scale q_i . k_j - lse_i).
//
// A workgroup takes 128 tokens of one sequence and key head as keys, a wave 32
// of them, whose fragments stay in registers, and goes through the rows (query
// head r % G of token r / G) from its first key's token on:
//   S = Q K^T         A = 32 rows x 16 channels,  B = 16 channels x 32 keys
// A lane then has one key, so that the sum over rows stays in its registers and
// no atomics join anything.  The rows pass through LDS, 64 at a time and for
// all waves, from memory without registers between.
//
// A score costs one quarter-rate instruction and two of full rate, 24 cycles of a
// SIMD for 64, against 16 of its products: about 400 of the 645-667 us that 2 prompts
// of 8000 and 8191 tokens (32 heads on 8 of 128) take, 0.81-0.84 PFLOP/s.  Vector
// instructions are issued in 67 % of the cycles and the matrix cores busy in 48 %:
// neither is full, and the barrier of every tile and the reads of the rows from LDS
// stand between.  48 prompts of 25 to 1405 tokens 217-225 us.  Tiles of 128 rows: 6
// and 26 % more; four waves a SIMD: 45 %.  32-bit inputs: 16 prompts of 3 to 600
// tokens (16 heads of 64) 29 us, 2 of 4000 and 4095 (32 heads on 8 of 128) 1080 us.
#pragma once

#include <type_traits>

#include "sv_device.h"
#include "sv_mfma.h"
#include "sv_prompt.h"

namespace sv {

namespace {

using namespace frag;

constexpr int kWBlock = 256;

// Rows of a tile and waves a SIMD.
template <int DT, int D> struct WeightShape {
  static constexpr int tile = DT == SPECV_F32 ? 32 : 64;
  static constexpr int buffers = DT == SPECV_F32 ? 1 : 2;
  static constexpr int waves = DT == SPECV_F32 && D == 256 ? 1 : 2;
};

template <int DT, int D>
__global__ __launch_bounds__(kWBlock, (WeightShape<DT, D>::waves)) void k_prompt_weights(PromptWeights p) {
  using Shape = WeightShape<DT, D>;
  constexpr int NP = kPieces<DT>, NF = D / 16, BM = Shape::tile, NB = BM / 32, NC = D / 8;
  constexpr int kPlane = BM * D, kAll = BM * NC, kLoads = (kAll + kWBlock - 1) / kWBlock;
  static_assert(DT == SPECV_F32 || kAll % kWBlock == 0, "whole loads");
  static_assert(kWeightKeys == 32 * (kWBlock / kWave), "32 keys a wave");
  const Packed& s = p.s;
  const int h = static_cast<int>(blockIdx.x % static_cast<unsigned>(s.H));
  const unsigned place = blockIdx.x / static_cast<unsigned>(s.H);
  const PromptBlock at = prompt_block<kWBlock, true>(s, place, 1, kWeightKeys);
  const int tid = threadIdx.x, lane = tid % kWave, w = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int col = lane % 32, half = lane / 32;
  if (at.block < 0) {
    // sequences without tokens: a wave clears one at a time
    const unsigned free = p.slots - at.used;
    for (long b = (place - at.used) * (kWBlock / kWave) + w; b < s.B; b += static_cast<long>(free) * (kWBlock / kWave)) {
      int first, last;
      prompt_range(s, static_cast<int>(b), first, last);
      if (first < last) continue;
      for (long j = lane; j < p.capacity; j += kWave) p.w[(b * s.H + h) * p.capacity + j] = 0.f;
    }
    return;
  }
  const int len = at.last - at.first, rows = len * s.G;
  const int nblock = (len + kWeightKeys - 1) / kWeightKeys, block = at.block;
  const int key0 = block * kWeightKeys, wkey = key0 + 32 * w, key = wkey + col;
  float* const wrow = p.w + (static_cast<long>(at.seq) * s.H + h) * p.capacity;
  if (block == nblock - 1)  // behind the prompt
    for (long j = static_cast<long>(len) + tid; j < p.capacity; j += kWBlock) wrow[j] = 0.f;

  __shared__ __align__(16) __bf16 lq[Shape::buffers][NP * kPlane];
  __shared__ __align__(16) float ll[Shape::buffers][BM];  // lse in log2; +infinity where a row weighs nothing

  const float kscale = s.scale * kLog2e;
  bf16x8 k[NF][NP];
  {
    const long base = (static_cast<long>(at.first) + min(key, len - 1)) * s.kv_row + static_cast<long>(h) * D + 8 * half;
    Raw8<DT> x[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) x[f].load(s.k, base + 16 * f);
#pragma unroll
    for (int f = 0; f < NF; ++f) x[f].pieces(k[f]);
  }

  // A tile has `step` rows, a multiple of G where G is small, so that a lane's
  // rows are the same heads in every tile and their places the same from the
  // tile's first token on; further rows of the tile weigh nothing.
  const bool even = s.G <= 32;
  const int step = even ? BM / s.G * s.G : BM;
  const int row_first = key0 * s.G, ntile = (rows - row_first + step - 1) / step;
  const long qbase = static_cast<long>(at.first) * s.q_row + static_cast<long>(h) * s.G * D;
  auto offset = [&](int tile, int e) {
    const int t = e / NC, r = min(row_first + tile * step + t, rows - 1), tok = s.token_of(r);
    return qbase + static_cast<long>(tok) * s.q_row + static_cast<long>(r - tok * s.G) * D + 8 * swizzle<D>(t, e % NC);
  };
  // bf16: a lane's places from the tile's first token on, in bytes: below 2^32, as rows are below 2^24 elements
  auto place_in = [&](int e, int r0, int most) {
    const int t = e / NC, tok0 = s.token_of(r0), r = min(r0 + t, most), tok = s.token_of(r);
    return 2 * (static_cast<uint32_t>(tok - tok0) * static_cast<uint32_t>(s.q_row) + static_cast<uint32_t>(r - tok * s.G) * D +
                8 * swizzle<D>(t, e % NC));
  };
  const uint32_t lq_at = lds_address(&lq[0][0]);
  uint32_t place_at[DT == SPECV_BF16 ? kLoads : 1];
  if constexpr (DT == SPECV_BF16) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) place_at[i] = place_in(tid + i * kWBlock, row_first, row_first + step - 1);
  }
  auto request = [&](int tile, int buf) {
    if constexpr (DT == SPECV_BF16) {
      const int r0 = row_first + tile * step;
      const uint16_t* const from = static_cast<const uint16_t*>(s.q) + qbase + static_cast<long>(__builtin_amdgcn_readfirstlane(s.token_of(r0))) * s.q_row;
      const bool whole = even && r0 + step <= rows;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t a = whole ? place_at[i] : place_in(tid + i * kWBlock, r0, rows - 1);
        load_lds(from, a, lq_at + 2 * (buf * NP * kPlane) + 16 * (i * kWBlock + w * kWave));
      }
    }
  };
  auto fill = [&](int tile) {
    if constexpr (DT == SPECV_F32) {
#pragma unroll D == 256 ? 1 : kLoads
      for (int i = 0; i < kLoads; ++i) {
        const int e = tid + i * kWBlock;
        if (kAll % kWBlock && e >= kAll) break;
        Raw8<DT> x;
        x.load(s.q, offset(tile, e));
        bf16x8 f[NP];
        x.pieces(f);
#pragma unroll
        for (int j = 0; j < NP; ++j) *reinterpret_cast<bf16x8*>(&lq[0][j * kPlane + 8 * e]) = f[j];
      }
    }
  };
  // the statistics of a tile's rows, by its first threads: loaded, and later put into LDS
  auto stat = [&](int tile) {
    float x = INFINITY;
    const int r = row_first + tile * step + tid;
    if (tid < step && r < rows) {
      const int tok = s.token_of(r);
      x = p.lse[(static_cast<long>(at.first) + tok) * s.Hq + h * s.G + (r - tok * s.G)];
    }
    return x;
  };
  auto put_stat = [&](int buf, float x) {
    asm volatile("" : "+v"(x));  // not looked at before: the wait for it would be one for the tile requested after it
    if (tid < BM) ll[buf][tid] = x == -INFINITY ? INFINITY : x * kLog2e;
  };

  // From the last tile on: all workgroups of a head begin with the same rows
  // and go on together, so that they find them in the cache (2 x 8191: 795 us,
  // from each one's own first rows on 814 us, at an earlier build).
  //
  // A query that weighs nothing (lse infinite) makes e^(s - lse) 0 by itself,
  // unless its score is not finite: then the sums are NaN, and are made again
  // with every statistic looked at (done at once, in the tiles that have such
  // queries: 48 prompts 230 us from 217, 2 x 8191 690 from 649; so 211 from 209
  // and 645.5 from 644.6, both sides in turn).
  float sum;
  for (bool careful = false;; careful = true) {
    request(ntile - 1, 0);
    float next = stat(ntile - 1), lost = 0.f;  // the tiles' sums are added with what each addition rounds away
    sum = 0.f;
    if constexpr (DT == SPECV_BF16) {
      put_stat(0, next);
      landed_barrier();
    }
    for (int tile = ntile - 1; tile >= 0; --tile) {
      const int buf = Shape::buffers == 2 ? (ntile - 1 - tile) & 1 : 0;
      const bool more = tile > 0;
      if constexpr (DT == SPECV_F32) {
        fill(tile);
        put_stat(0, next);
        if (more) next = stat(tile - 1);
        __syncthreads();
      } else if (more) {
        next = stat(tile - 1);
        request(tile - 1, buf ^ 1);
      }
      const int r0 = row_first + tile * step;
      if (wkey < len && r0 + BM > wkey * s.G) {  // a row sees a key of the wave
        float part = 0.f;
        // The products of a block of 32 rows are under way while the exponentials
        // of the block before are taken: the matrix unit and the vector unit work
        // at the same time, and a product's result is not waited for.
        auto scores = [&](int n, f32x16& sc) {
#pragma unroll
          for (int i = 0; i < 16; ++i) sc[i] = 0.f;
#pragma unroll
          for (int f = 0; f < NF; ++f) {
            bf16x8 a[NP];
            const int t = 32 * n + col;
#pragma unroll
            for (int j = 0; j < NP; ++j)
              a[j] = *reinterpret_cast<const bf16x8*>(&lq[buf][j * kPlane + t * D + 8 * swizzle<D>(t, 2 * f + half)]);
#pragma unroll
            for (int z = NP - 1; z >= 0; --z)
#pragma unroll
              for (int i = 0; i <= z; ++i) sc = mfma32(a[z - i], k[f][i], sc);
          }
        };
        // mixed: some rows do not see some of the wave's keys; wild: some that weigh nothing have scores that are not finite
        auto blocks = [&](auto mixed, auto wild) {
          f32x16 sc[2];
          scores(0, sc[0]);
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            if (n + 1 < NB) scores(n + 1, sc[(n + 1) & 1]);
            // rows from `first` on see the lane's key; from `past` on they are others' copies
            const int first = key * s.G - (r0 + 32 * n + 4 * half), past = step - (32 * n + 4 * half);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const f32x4 l4 = *reinterpret_cast<const f32x4*>(&ll[buf][32 * n + 8 * j + 4 * half]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float e = ex2(fmaf(sc[n & 1][4 * j + i], kscale, -l4[i]));
                const bool none = (decltype(mixed)::value && (8 * j + i < first || 8 * j + i >= past)) || (decltype(wild)::value && l4[i] == INFINITY);
                part += none ? 0.f : e;  // whatever an unseen score is
              }
            }
          }
        };
        if (careful) blocks(std::true_type{}, std::true_type{});
        else if (r0 >= (wkey + 31) * s.G) blocks(std::false_type{}, std::false_type{});
        else blocks(std::true_type{}, std::false_type{});
        const float y = part - lost, z = sum + y;
        lost = (z - sum) - y;
        sum = z;
      }
      if constexpr (DT == SPECV_BF16) {
        if (more) put_stat(buf ^ 1, next);
      }
      landed_barrier();
    }
    if (careful || !__syncthreads_or(sum != sum)) break;
  }
  sum = halves_sum(sum);
  if (half == 0 && key < len && key < p.capacity) wrow[key] = sum;
}

template <int D>
hipError_t launch_weights(const PromptWeights& p, int dtype, hipStream_t st) {
  const dim3 grid(p.slots * static_cast<unsigned>(p.s.H));
  if (dtype == SPECV_F32) hipLaunchKernelGGL((k_prompt_weights<SPECV_F32, D>), grid, dim3(kWBlock), 0, st, p);
  else hipLaunchKernelGGL((k_prompt_weights<SPECV_BF16, D>), grid, dim3(kWBlock), 0, st, p);
  return hipGetLastError();
}

}  // namespace

}  // namespace sv
