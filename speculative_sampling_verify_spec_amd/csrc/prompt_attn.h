// Causal attention of whole prompts (the kernel template; k_prompt_<dim>.hip
// instantiate it).
//
// A workgroup takes 128 rows of one sequence and one key head; row r is query
// head r % G of token r / G, so the G query heads that share a key head also
// share its tiles, and a short prompt fills a block with all its heads.  A
// wave has 32 of the rows as the columns of both products:
//   S^T = K Q^T       A = 32 tokens x 16 channels,  B = 16 channels x 32 rows
//   O^T += V^T P^T    A = 32 channels x 16 tokens,  B = 16 tokens x 32 rows
// with v_mfma_f32_32x32x16_bf16.  A lane then has one row's scores, so that
// the softmax needs one exchange between two lanes; and its scores of a tile
// are, as they come, the B operand of the second product, for the order of
// tokens in which the A operand is read.  That operand is V transposed, which
// the transposing LDS read gives.
//
// The tiles of K and V pass through LDS, swizzled by 16 bytes so that neither
// read meets bank conflicts; bf16 goes from memory to LDS without registers
// between, the next tile while this one is worked on.
//
// Softmax: the running maximum is held per row and only moved when a tile
// exceeds it by more than 2^8 (the weights then stay below 2^8, and the sums
// are in 32 bits), so most tiles rescale nothing.  The weights are rounded to
// bf16 for the product with the values, as the output is.
//
// 32-bit inputs: every operand is split into three bf16 pieces whose sum has
// 24 bits; products take the six largest of nine pieces' products.
#pragma once

#include <cfloat>
#include <type_traits>

#include "sv_device.h"
#include "sv_kv.h"
#include "sv_mfma.h"
#include "sv_prompt.h"

namespace sv {

namespace {

using namespace frag;

constexpr int kPBlock = 256;

// Tokens of a tile, LDS buffers of tiles and waves a SIMD.
template <int DT, int D> struct PromptShape {
  static constexpr int tile = DT == SPECV_F32 || D == 256 ? 32 : 64;
  static constexpr int buffers = DT == SPECV_F32 ? 1 : 2;
  static constexpr int waves = DT == SPECV_F32 || D == 256 ? 1 : 2;
};

template <int DT, int D>
__global__ __launch_bounds__(kPBlock, (PromptShape<DT, D>::waves)) void k_prompt_attn(PromptAttn p) {
  using Shape = PromptShape<DT, D>;
  constexpr int NP = kPieces<DT>, NF = D / 16, ND = D / 32, BN = Shape::tile, NB = BN / 32, NC = D / 8;
  constexpr int kPlane = BN * D;                 // elements of a tile's piece
  constexpr int kAll = BN * NC, kLoads = (kAll + kPBlock - 1) / kPBlock;  // pieces of 8 elements of K (and of V): of the tile, of a thread
  static_assert(DT == SPECV_F32 || kAll % kPBlock == 0, "whole loads");
  const Packed& s = p.s;
  const int h = static_cast<int>(blockIdx.x % static_cast<unsigned>(s.H));
  const unsigned place = blockIdx.x / static_cast<unsigned>(s.H);
  const PromptBlock at = prompt_block<kPBlock, false>(s, place, s.G, kPromptRows);
  const int tid = threadIdx.x, lane = tid % kWave, w = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int col = lane % 32, half = lane / 32;
  if (at.block < 0) {
    // tokens of no sequence (before the first and behind the last) see nothing
    const int lead = min(max(s.starts[0], 0), s.T), tail = min(max(s.starts[s.B], lead), s.T);
    const int gone = lead + s.T - tail;
    const unsigned free = p.slots - at.used;
    float zero[4] = {0.f, 0.f, 0.f, 0.f};
    for (long i = place - at.used; i < gone; i += free) {
      const long tok = i < lead ? i : tail + (i - lead);
      const long row = tok * s.Hq + static_cast<long>(h) * s.G;
      for (int e = tid; e < s.G * D / 4; e += kPBlock) kv_store4<DT>(p.out, row * D + 4 * e, zero);
      if (p.lse)
        for (int e = tid; e < s.G; e += kPBlock) p.lse[row + e] = -INFINITY;
    }
    return;
  }
  const int len = at.last - at.first, rows = len * s.G;
  const int row0 = at.block * kPromptRows, wrow = row0 + 32 * w;
  const int r = min(wrow + col, rows - 1);  // a row that exists
  const int tok = s.token_of(r), hq = h * s.G + (r - tok * s.G);

  __shared__ __align__(16) __bf16 lk[Shape::buffers][NP * kPlane], lv[Shape::buffers][NP * kPlane];
  __shared__ int wild;  // a value that is not finite was cleared

  // ---- queries, negated where the scale is ----
  const float kscale = fmaxf(fabsf(s.scale) * kLog2e, 0x1p-149f);  // > 0: a masked score stays -infinity
  // fp32 with D = 256 keeps them whole and splits them in every tile: their
  // pieces would take 192 registers
  constexpr bool kWhole = DT == SPECV_F32 && D == 256;
  bf16x8 q[kWhole ? 1 : NF][NP];
  Raw8<DT> xq[NF];
  f32x16 o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  float m = -FLT_MAX, l = 0.f;

  // tokens seen by the workgroup's last and first row
  const int last_tok = s.token_of(min(row0 + kPromptRows - 1, rows - 1)), first_tok = s.token_of(row0);
  const int ntile = last_tok / BN + 1;
  const long kbase = static_cast<long>(at.first) * s.kv_row + static_cast<long>(h) * D;

  auto offset = [&](int tile, int e) {
    const int t = e / NC;
    return kbase + static_cast<long>(min(tile * BN + t, len - 1)) * s.kv_row + 8 * swizzle<D>(t, e % NC);
  };
  // bf16: memory to LDS, whose rows hold the pieces in the swizzled order.  A
  // lane's places in a tile are below 2^32 bytes: rows are below 2^24 elements.
  const uint32_t lk_at = lds_address(&lk[0][0]), lv_at = lds_address(&lv[0][0]);
  uint32_t place_at[kLoads];
  const uint32_t row_bytes = 2 * static_cast<uint32_t>(s.kv_row);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int e = tid + i * kPBlock, t = e / NC;
    place_at[i] = t * row_bytes + 16 * swizzle<D>(t, e % NC);
  }
  auto request = [&](int tile, int buf) {
    if constexpr (DT == SPECV_BF16) {
      const long first = kbase + static_cast<long>(tile) * BN * s.kv_row;
      const uint16_t *k = static_cast<const uint16_t*>(s.k) + first, *v = static_cast<const uint16_t*>(s.v) + first;
      const int rest = len - tile * BN;  // tokens from the tile's first on; its further rows are the last one's again
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        uint32_t at = place_at[i];
        if (rest < BN) at -= static_cast<uint32_t>(max((tid + i * kPBlock) / NC - (rest - 1), 0)) * row_bytes;
        const uint32_t to = 2 * (buf * NP * kPlane) + 16 * (i * kPBlock + w * kWave);
        load_lds(k, at, lk_at + to);
        load_lds(v, at, lv_at + to);
      }
    }
  };
  // fp32: through registers, where an element becomes its pieces; a tile is
  // loaded a tile ahead where there are registers for it
  constexpr bool kAhead = DT == SPECV_F32 && D <= 128;
  Raw8<DT> xk[kAhead ? kLoads : 1], xv[kAhead ? kLoads : 1];
  auto load = [&](int tile) {
    if constexpr (kAhead) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const long a = offset(tile, min(tid + i * kPBlock, kAll - 1));
        xk[i].load(s.k, a);
        xv[i].load(s.v, a);
      }
    }
  };
  auto put = [&](__bf16* to, int e, const Raw8<DT>& x) {
    bf16x8 f[NP];
    x.pieces(f);
#pragma unroll
    for (int j = 0; j < NP; ++j) *reinterpret_cast<bf16x8*>(&to[j * kPlane + 8 * e]) = f[j];
  };
  auto fill = [&](int tile) {
    if constexpr (DT == SPECV_F32) {
      int thread = tid;
      if constexpr (kWhole) asm volatile("" : "+v"(thread));
#pragma unroll kAhead ? kLoads : 1
      for (int i = 0; i < kLoads; ++i) {
        const int e = thread + i * kPBlock;
        if (kAll % kPBlock && e >= kAll) break;
        if constexpr (!kAhead) {
          const long a = offset(tile, e);
          xk[0].load(s.k, a);
          xv[0].load(s.v, a);
        }
        put(lk[0], e, xk[kAhead ? i : 0]);
        put(lv[0], e, xv[kAhead ? i : 0]);
      }
    }
  };
  // clears what is not finite among a tile's values in LDS
  auto tame = [&](int buf) {
    bool odd = false;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int e = tid + i * kPBlock;
      if (kAll % kPBlock && e >= kAll) break;
      Raw8<SPECV_BF16> x;  // an element that is not finite is its own first piece
      uint4* at = reinterpret_cast<uint4*>(&lv[buf][8 * e]);
      x.w[0] = *at;
      if (x.wild()) {
        odd = true;
        x.tame();
        *at = x.w[0];
      }
    }
    if (odd) wild = 1;
  };
  // The queries' rows come the way a tile does, in whole lines, into the buffers
  // that the second tile will take, where these hold them; else from memory into
  // registers (48 prompts of 1 to 1500 tokens 403 us, with rows read and written
  // by lanes 421).
  constexpr bool kQueriesInLds = DT == SPECV_BF16 && 2 * BN >= kPromptRows;
  if (tid == 0) wild = 0;
  request(0, 0);
  load(0);
  if constexpr (kQueriesInLds) {
    const int tok0 = s.token_of(row0);
    const uint16_t* const from = static_cast<const uint16_t*>(s.q) + (static_cast<long>(at.first) + tok0) * s.q_row + static_cast<long>(h) * s.G * D;
#pragma unroll
    for (int i = 0; i < 2 * kLoads; ++i) {
      const int e = tid + i * kPBlock, t = e / NC, x = min(row0 + t, rows - 1), y = s.token_of(x);  // the last row again behind it
      const uint32_t a = 2 * (static_cast<uint32_t>(y - tok0) * static_cast<uint32_t>(s.q_row) + static_cast<uint32_t>(x - y * s.G) * D +
                              8 * swizzle<D>(t % BN, e % NC));
      load_lds(from, a, (i < kLoads ? lk_at : lv_at) + 2 * kPlane + 16 * (i % kLoads * kPBlock + w * kWave));
    }
    landed_barrier();
    const __bf16* const rows_at = w < 2 ? lk[1] : lv[1];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int t = 32 * (w % 2) + col;
      xq[f].w[0] = *reinterpret_cast<const uint4*>(&rows_at[t * D + 8 * swizzle<D>(t, 2 * f + half)]);
    }
    lds_barrier();  // before the second tile is requested
  } else {
    const long base = (static_cast<long>(at.first) + tok) * s.q_row + static_cast<long>(hq) * D + 8 * half;
#pragma unroll
    for (int f = 0; f < NF; ++f) xq[f].load(s.q, base + 16 * f);
    if constexpr (DT == SPECV_BF16) landed_barrier();
  }
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    xq[f].hide();
    xq[f].negate(s.scale < 0.f);
    if constexpr (!kWhole) xq[f].pieces(q[f]);
  }

  // a tile's part in the rows; mixed: some rows of the workgroup do not see all of it
  auto step = [&](int tile, auto mixed) {
    const int buf = Shape::buffers == 2 ? tile & 1 : 0;
    if constexpr (DT == SPECV_F32) {
      fill(tile);
      if (tile + 1 < ntile) load(tile + 1);
      lds_barrier();
    } else if (tile + 1 < ntile) {
      request(tile + 1, buf ^ 1);
    }
    if constexpr (decltype(mixed)::value) {
      tame(buf);
      lds_barrier();
    }
    const int t0 = tile * BN;
    // waves whose rows see nothing of the tile wait for the others
    if (!decltype(mixed)::value || (t0 * s.G < wrow + 32 && wrow < rows)) {
      // the lane's places in LDS are computed in every tile where registers are short
      int own = lane;
      if constexpr (kWhole) asm volatile("" : "+v"(own));
      // ---- scores: token 32 n + 8 (i / 4) + 4 half + i % 4 of the tile in register i ----
      f32x16 sc[NB];
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) sc[n][i] = 0.f;
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        constexpr int kStep = kWhole ? 0 : 1;
        if constexpr (kWhole) {
          __builtin_amdgcn_sched_barrier(0);  // reads far ahead would not leave registers for the pieces
          xq[f].hide();
          xq[f].pieces(q[0]);
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          bf16x8 a[NP];
          const int t = 32 * n + own % 32;
#pragma unroll
          for (int j = 0; j < NP; ++j)
            a[j] = *reinterpret_cast<const bf16x8*>(&lk[buf][j * kPlane + t * D + 8 * swizzle<D>(t, 2 * f + own / 32)]);
#pragma unroll
          for (int z = NP - 1; z >= 0; --z)
#pragma unroll
            for (int i = 0; i <= z; ++i) sc[n] = mfma32(a[z - i], q[f * kStep][i], sc[n]);
        }
      }
      if constexpr (decltype(mixed)::value) {
        const int sees = tok - t0 - 4 * half;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (32 * n + 8 * (i / 4) + i % 4 > sees) sc[n][i] = -INFINITY;
      }
      float x = sc[0][0];
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) x = fmaxf(x, sc[n][i]);
      x *= kscale;
      if (__any(x > m + 8.f)) {
        x = halves_max(x);
        const bool need = x > m + 8.f;  // each row decides for itself, so that its bits do not depend on its neighbours
        const float a = need ? ex2(m - x) : 1.f;
        m = need ? x : m;
        l *= a;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[d][i] *= a;
      }
      bf16x8 pf[NB * 2][NP];
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const f32x2 e = {ex2(fmaf(sc[n][i], kscale, -m)), ex2(fmaf(sc[n][i + 1], kscale, -m))};
          sum += e[0];
          sum += e[1];
          split2<NP>(e, &pf[2 * n + i / 8][0], i % 8);
        }
      l += sum;
      // ---- values: slots 0..3 of half h hold tokens 16 c + 4 h .., 4..7 those 8 further ----
#pragma unroll
      for (int c = 0; c < 2 * NB; ++c)
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          bf16x8 a[NP];
          const int t = 4 * (own / 32) + (own % 16) / 4, piece = 4 * d + 2 * ((own / 16) % 2) + (own % 4) / 2;
#pragma unroll
          for (int j = 0; j < NP; ++j)
            a[j] = read_transposed(&lv[buf][j * kPlane + (16 * c + t) * D + 8 * swizzle<D>(16 * c + t, piece) + 4 * (own % 2)],
                                   &lv[buf][j * kPlane + (16 * c + t + 8) * D + 8 * swizzle<D>(16 * c + t + 8, piece) + 4 * (own % 2)]);
#pragma unroll
          for (int z = NP - 1; z >= 0; --z)
#pragma unroll
            for (int i = 0; i <= z; ++i) o[d] = mfma32(a[z - i], pf[c][i], o[d]);
        }
      if constexpr (decltype(mixed)::value)
        if (wild) {
          // values that are not finite must not meet a weight of 0: they were
          // left out, and are added where they are seen
#pragma unroll 1
          for (int j = 0; j < BN && t0 + j < len; ++j) {
            float e = 0.f;
#pragma unroll
            for (int c = 0; c < 2 * NB; ++c)
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (16 * c + 8 * (i / 4) + 4 * half + i % 4 == j) e = static_cast<float>(pf[c][0][i]);
            e = halves_sum(e);
            const long a = kbase + static_cast<long>(t0 + j) * s.kv_row + 4 * half;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                // few loads at a time: this rare part's registers count for the whole kernel
                if (i % 4 == 0) __builtin_amdgcn_sched_barrier(0);
                const long k = a + 32 * d + 8 * (i / 4) + i % 4;
                float y;
                if constexpr (DT == SPECV_F32) y = static_cast<const float*>(s.v)[k];
                else y = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(s.v)[k]) << 16);
                if (!isfinite(y) && t0 + j <= tok) o[d][i] += e * y;
              }
          }
        }
    }
    if constexpr (DT == SPECV_F32) lds_barrier();
    else landed_barrier();
  };
  const int whole = min((first_tok + 1) / BN, ntile);  // tiles that every row sees all of
  for (int tile = 0; tile < whole; ++tile) step(tile, std::false_type{});
  for (int tile = whole; tile < ntile; ++tile) step(tile, std::true_type{});

  l = halves_sum(l);
  const bool there = wrow + col < rows, some = !(l == 0.f);
  const float inv = some ? 1.f / l : 0.f;
  const long orow = (static_cast<long>(at.first) + tok) * s.Hq + hq;
  if (p.lse && half == 0 && there) p.lse[orow] = kv_lse(m, l, some);
  auto value = [&](int d, int i) { return some ? o[d][i] * inv : 0.f; };
  if constexpr (DT == SPECV_F32) {
    if (!there) return;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const float y[4] = {value(d, i), value(d, i + 1), value(d, i + 2), value(d, i + 3)};
        kv_store4<DT>(p.out, orow * D + 32 * d + 2 * i + 4 * half, y);
      }
  } else {
    // Through LDS, where a wave has 32 rows for itself by now, to whole lines:
    // a lane has 4 channels of each 8 and its partner the others; they exchange
    // what makes 16 bytes for each.
    __bf16* const out = (w < 2 ? lk[0] : lv[0]) + w % 2 * 32 * D;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 8) {
        uint32_t a[2], b[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          a[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{value(d, i + 2 * k), value(d, i + 2 * k + 1)}), bf16x2));
          b[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{value(d, i + 4 + 2 * k), value(d, i + 4 + 2 * k + 1)}), bf16x2));
        }
        const auto x = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false), y = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
        *reinterpret_cast<uint4*>(&out[col * D + 8 * swizzle<D>(col, 4 * d + i / 4 + half)]) = make_uint4(x[0], y[0], x[1], y[1]);
      }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 32 * NC / kWave; ++i) {
      const int e = i * kWave + lane, t = e / NC, x = wrow + t, y = s.token_of(min(x, rows - 1));
      if (x < rows)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + ((static_cast<long>(at.first) + y) * s.Hq + h * s.G + (x - y * s.G)) * D + 8 * (e % NC)) =
            *reinterpret_cast<const uint4*>(&out[t * D + 8 * swizzle<D>(t, e % NC)]);
    }
  }
}

template <int D>
hipError_t launch_prompt(const PromptAttn& p, int dtype, hipStream_t st) {
  const dim3 grid(p.slots * static_cast<unsigned>(p.s.H));
  if (dtype == SPECV_F32) hipLaunchKernelGGL((k_prompt_attn<SPECV_F32, D>), grid, dim3(kPBlock), 0, st, p);
  else hipLaunchKernelGGL((k_prompt_attn<SPECV_BF16, D>), grid, dim3(kPBlock), 0, st, p);
  return hipGetLastError();
}

}  // namespace

}  // namespace sv
