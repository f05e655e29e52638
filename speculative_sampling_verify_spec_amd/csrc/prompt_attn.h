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
// Measured (32 heads on 8 of 128): a prompt of 16384 tokens 2045-2085 us, 1.05-1.08
// PFLOP/s, nine tenths of what a large matrix product reaches on the same card,
// bound by the matrix cores at the clock that they leave; 48 prompts of 25 to 1405
// tokens 410-418 us, the matrix cores busy for 41 % of the cycles: a block of 8 tiles
// on average has its queries, first tile and results to wait for.
//
// 32-bit inputs: every operand is split into three bf16 pieces whose sum has
// 24 bits; products take the six largest of nine pieces' products.
#pragma once

#include <cfloat>
#include <type_traits>
#include <utility>

#include "sv_device.h"
#include "sv_kv.h"
#include "sv_mfma.h"
#include "sv_prompt.h"

namespace sv {

namespace {

using namespace frag;

constexpr int kPBlock = 256;

// f(0), f(1) .. with numbers that the compiler knows.
template <class F, int... I>
__device__ __forceinline__ void in_order(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}

constexpr float kHeld = 8.f;  // how far, in powers of two, scores may exceed the held maximum

// Tokens of a tile, LDS buffers of tiles and waves a SIMD.
template <int DT, int D> struct PromptShape {
  static constexpr int tile = DT == SPECV_F32 || D == 256 ? 32 : 64;
  static constexpr bool piped = DT == SPECV_BF16 && D == 256;
  static constexpr int buffers = DT == SPECV_F32 ? 1 : piped ? 4 : 2;
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
    // Tokens of no sequence see nothing: those before and behind all that one
    // holds, wherever it stands among starts, so that no row has two writers
    // unless sequences share it.
    __shared__ int held[2];
    if (tid == 0) {
      held[0] = s.T;
      held[1] = 0;
    }
    __syncthreads();
    for (int b = tid; b < s.B; b += kPBlock) {
      int first, last;
      prompt_range(s, b, first, last);
      if (first < last) {
        atomicMin(&held[0], first);
        atomicMax(&held[1], last);
      }
    }
    __syncthreads();
    const int lead = held[0], tail = max(held[1], lead);
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
  auto buffer = [](int tile) { return tile & (Shape::buffers - 1); };
  auto request = [&](const void* base, uint32_t to, int tile, int from_load, int to_load, bool inside = false) {
    if constexpr (DT == SPECV_BF16) {
      const uint16_t* const from = static_cast<const uint16_t*>(base) + kbase + static_cast<long>(tile) * BN * s.kv_row;
      const int rest = len - tile * BN;  // tokens from the tile's first on; its further rows are the last one's again
      to += buffer(tile) * 2 * kPlane + 16 * w * kWave;
#pragma unroll
      for (int i = from_load; i < to_load; ++i) {
        uint32_t at = place_at[i];
        if (!inside && rest < BN) at -= static_cast<uint32_t>(max((tid + i * kPBlock) / NC - (rest - 1), 0)) * row_bytes;
        load_lds(from, at, to + 16 * i * kPBlock);
      }
    }
  };
  auto request_k = [&](int tile) { request(s.k, lk_at, tile, 0, kLoads); };
  auto request_v = [&](int tile) { request(s.v, lv_at, tile, 0, kLoads); };
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
      if constexpr (kAhead) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int e = thread + i * kPBlock;
          if (kAll % kPBlock && e >= kAll) break;
          put(lk[0], e, xk[i]);
          put(lv[0], e, xv[i]);
        }
      } else {
        // two places of K and of V at a time, as the registers allow: each such turn
        // waits for memory once (a head of 256 channels over 5000 tokens 1265 us, one
        // place at a time 1307)
        static_assert(kAll % kPBlock == 0 && kLoads % 2 == 0, "whole loads");
#pragma unroll 1
        for (int e = thread; e < kAll; e += 2 * kPBlock) {
          const long a = offset(tile, e), b = offset(tile, e + kPBlock);
          Raw8<DT> k0, v0, k1, v1;
          k0.load(s.k, a);
          k1.load(s.k, b);
          v0.load(s.v, a);
          v1.load(s.v, b);
          put(lk[0], e, k0);
          put(lk[0], e + kPBlock, k1);
          put(lv[0], e, v0);
          put(lv[0], e + kPBlock, v1);
        }
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
  // that a later tile will take (48 prompts of 1 to 1500 tokens 403 us, with rows read and written
  // by lanes 421).
  constexpr int kSpare = Shape::buffers / 2, kQueryLoads = kPromptRows * NC / kPBlock;
  static_assert(DT == SPECV_F32 || 2 * kSpare * BN >= kPromptRows, "room for the queries");
  if (tid == 0) wild = 0;
  load(0);
  if constexpr (DT == SPECV_BF16) {
    request_k(0);
    if constexpr (!Shape::piped) request_v(0);
    const int tok0 = s.token_of(row0);
    const uint16_t* const from = static_cast<const uint16_t*>(s.q) + (static_cast<long>(at.first) + tok0) * s.q_row + static_cast<long>(h) * s.G * D;
#pragma unroll
    for (int i = 0; i < kQueryLoads; ++i) {
      const int e = tid + i * kPBlock, t = e / NC, x = min(row0 + t, rows - 1), y = s.token_of(x);  // the last row again behind it
      const uint32_t a = 2 * (static_cast<uint32_t>(y - tok0) * static_cast<uint32_t>(s.q_row) + static_cast<uint32_t>(x - y * s.G) * D +
                              8 * swizzle<D>(t, e % NC));
      load_lds(from, a, (i < kQueryLoads / 2 ? lk_at : lv_at) + kSpare * 2 * kPlane + 16 * (i % (kQueryLoads / 2) * kPBlock + w * kWave));
    }
    if constexpr (Shape::piped) {
      request_v(0);
      if (ntile > 1) {
        request_k(1);
        request_v(1);
        landed_barrier<3 * kLoads>();
      } else {
        landed_barrier<kLoads>();
      }
    } else {
      landed_barrier();
    }
    const __bf16* const rows_at = w < 2 ? lk[kSpare] : lv[kSpare];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int t = 32 * (w % 2) + col;
      xq[f].w[0] = *reinterpret_cast<const uint4*>(&rows_at[t * D + 8 * swizzle<D>(t, 2 * f + half)]);
    }
    lds_barrier();  // before the next tile is requested there
  } else {
    const long base = (static_cast<long>(at.first) + tok) * s.q_row + static_cast<long>(hq) * D + 8 * half;
#pragma unroll
    for (int f = 0; f < NF; ++f) xq[f].load(s.q, base + 16 * f);
  }
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    xq[f].hide();
    xq[f].negate(s.scale < 0.f);
    if constexpr (!kWhole) xq[f].pieces(q[f]);
  }

  // The lane's places in a tile.  With D = 256 the compiler works all of them out
  // again in every tile; a swizzle changes the low 4 bits of a piece's number
  // alone, so that 8 places of K and 8 of V make all others by constant steps.
  typedef const __attribute__((address_space(3))) __bf16* LdsPtr;
  LdsPtr kat[8], vat[8];
  if constexpr (Shape::piped) {
    const int t = 4 * half + (lane % 16) / 4, piece = 2 * ((lane / 16) % 2) + (lane % 4) / 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int x = t + i % 2 * 8;
      kat[i] = (LdsPtr)(&lk[0][0]) + (col * D + 8 * swizzle<D>(col, 2 * i + half));
      vat[i] = (LdsPtr)(&lv[0][0]) + (x * D + 8 * swizzle<D>(x, 4 * (i / 2) + piece) + 4 * (lane % 2));
      asm volatile("" : "+v"(kat[i]), "+v"(vat[i]));
    }
  }

  auto fragment_k = [&](int tile, int f) {
    return *(const __attribute__((address_space(3))) bf16x8*)(kat[f % 8] + buffer(tile) * kPlane + f / 8 * 128);
  };
  auto fragment_v = [&](int tile, int c, int d) {
    const int from = buffer(tile) * kPlane + 16 * c * D + d / 4 * 128;
    return read_transposed(vat[d % 4 * 2] + from, vat[d % 4 * 2 + 1] + from);
  };

  // mixed: some rows of the workgroup do not see all of the tile
  // ---- scores: token 32 n + 8 (i / 4) + 4 half + i % 4 of the tile in register i ----
  auto mask = [&](int tile, f32x16* sc) {
    const int sees = tok - tile * BN - 4 * half;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (32 * n + 8 * (i / 4) + i % 4 > sees) sc[n][i] = -INFINITY;
  };
  auto scores = [&](int tile, f32x16* sc, auto mixed) {
    const int buf = buffer(tile);
    // the lane's places in LDS are computed in every tile where registers are short
    int own = lane;
    if constexpr (kWhole) asm volatile("" : "+v"(own));
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
          if constexpr (Shape::piped) a[j] = fragment_k(tile, f);
          else a[j] = *reinterpret_cast<const bf16x8*>(&lk[buf][j * kPlane + t * D + 8 * swizzle<D>(t, 2 * f + own / 32)]);
#pragma unroll
        for (int z = NP - 1; z >= 0; --z)
#pragma unroll
          for (int i = 0; i <= z; ++i) sc[n] = mfma32(a[z - i], q[f * kStep][i], sc[n]);
      }
    }
    if constexpr (decltype(mixed)::value) mask(tile, sc);
  };
  // moves the held maximum to the scores' where they exceed it by too much
  auto highest = [&](const f32x16* sc) {
    float x = sc[0][0];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) x = fmaxf(x, sc[n][i]);
    return x;
  };
  auto raise = [&](float x, bool first) {
    x *= kscale;
    if (__any(x > m + kHeld)) {
      x = halves_max(x);
      const bool need = x > m + kHeld;  // each row decides for itself, so that its bits do not depend on its neighbours
      const float a = need ? ex2(m - x) : 1.f;
      m = need ? x : m;
      if (first) return;  // nothing is summed yet
      l *= a;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= a;
    }
  };
  auto weights = [&](const f32x16* sc, bf16x8 (*pf)[NP]) {
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
  };
  // ---- values: slots 0..3 of half h hold tokens 16 c + 4 h .., 4..7 those 8 further ----
  auto values = [&](int tile, bf16x8 (*pf)[NP]) {
    const int buf = buffer(tile);
    int own = lane;
    if constexpr (kWhole) asm volatile("" : "+v"(own));
#pragma unroll
    for (int c = 0; c < 2 * NB; ++c)
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        bf16x8 a[NP];
        const int t = 4 * (own / 32) + (own % 16) / 4, piece = 4 * d + 2 * ((own / 16) % 2) + (own % 4) / 2;
#pragma unroll
        for (int j = 0; j < NP; ++j)
          if constexpr (Shape::piped) a[j] = fragment_v(tile, c, d);
          else a[j] = read_transposed(&lv[buf][j * kPlane + (16 * c + t) * D + 8 * swizzle<D>(16 * c + t, piece) + 4 * (own % 2)],
                                 &lv[buf][j * kPlane + (16 * c + t + 8) * D + 8 * swizzle<D>(16 * c + t + 8, piece) + 4 * (own % 2)]);
#pragma unroll
        for (int z = NP - 1; z >= 0; --z)
#pragma unroll
          for (int i = 0; i <= z; ++i) o[d] = mfma32(a[z - i], pf[c][i], o[d]);
      }
  };
  // values that are not finite must not meet a weight of 0: they were left out
  // of the tile, and are added where they are seen
  auto add_wild = [&](int tile, bf16x8 (*pf)[NP]) {
    const int t0 = tile * BN;
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
  };

  const int whole = min((first_tok + 1) / BN, ntile);  // tiles that every row sees all of
  if constexpr (Shape::piped) {
    // One wave a SIMD: its own products of the next tile's scores are under way
    // while it takes this one's exponentials, and its requests are spread among
    // the products (6 prompts of 660 to 1040 tokens, 16 heads on 2: 67 us, a tile's
    // parts one after the other 82).  K is requested four tiles ahead, V three.
    constexpr int kFirst = 4, kTotal = NF + 2 * ND;
    static_assert(NB == 1 && NF == 16 && ND == 8 && NP == 1 && kLoads == 4, "a tile of 32 tokens");
    // what of the requests made until a tile is done may be under way behind it: those
    // after K of two tiles further and V of the next
    auto arrive = [&](int rest) {
      if (rest >= 4) landed_barrier<4 * kLoads>();
      else if (rest == 3) landed_barrier<3 * kLoads>();
      else if (rest == 2) landed_barrier<kLoads>();
      else landed_barrier();
    };
    if (ntile > 2) {
      request_k(2);
      request_v(2);
    }
    if (ntile > 3) request_k(3);
    f32x16 sc;
    scores(0, &sc, std::false_type{});
    if (whole == 0) mask(0, &sc);
    raise(highest(&sc), true);
    arrive(ntile);
    // steady: every row sees this and the next tile whole, and four more whole ones follow
    auto step = [&](int tile, auto steady) {
      constexpr bool kSteady = decltype(steady)::value;
      const int rest = ntile - 1 - tile;  // tiles behind this one
      if (!kSteady && tile >= whole) {
        tame(buffer(tile));
        lds_barrier();
      }
      // The order is written out (the compiler's takes the exponentials first): a
      // product, the read for the one four further on, a part of the softmax or of
      // the requests, which else wait for one another.  Behind the last tile the
      // scores are of what is left in LDS, and not used.
      bf16x8 pf[2][NP], ring[kFirst];
      f32x16 even, odd;  // two sums, for products that need not wait for the one before
      auto read = [&](int i) {
        if (i < NF) return fragment_k(tile + 1, i);
        return fragment_v(tile, (i - NF) / ND, (i - NF) % ND);
      };
#pragma unroll
      for (int i = 0; i < kFirst; ++i) ring[i] = read(i);
#pragma unroll
      for (int i = 0; i < 16; ++i) even[i] = odd[i] = 0.f;
      float sum = 0.f, x = -INFINITY;
      in_order([&](auto number) {
        constexpr int i = decltype(number)::value;
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (i < NF) {
          if constexpr (i % 2 == 0) even = mfma32(ring[i % kFirst], q[i][0], even);
          else odd = mfma32(ring[i % kFirst], q[i][0], odd);
          if constexpr (i % 2 == 0) {
            const f32x2 e = {ex2(fmaf(sc[i], kscale, -m)), ex2(fmaf(sc[i + 1], kscale, -m))};
            sum += e[0];
            sum += e[1];
            split2<NP>(e, &pf[i / 8][0], i % 8);
          }
        } else {
          constexpr int j = i - NF;
          o[j % ND] = mfma32(ring[i % kFirst], pf[j / ND][0], o[j % ND]);
          if constexpr (j == 3) {
            sc = even + odd;
            if (!kSteady && tile + 1 >= whole) mask(tile + 1, &sc);
          }
          if constexpr (j >= 4 && j < 12) x = fmaxf(fmaxf(x, sc[2 * (j - 4)]), sc[2 * (j - 4) + 1]);
        }
        if constexpr (i + kFirst < kTotal) ring[i % kFirst] = read(i + kFirst);
        if constexpr (i % 4 == 1) {
          constexpr int part = i / 4;
          if constexpr (part < kLoads) {
            if (kSteady || rest >= 4) request(s.k, lk_at, tile + 4, part, part + 1, kSteady);
          } else if (kSteady || rest >= 3) {
            request(s.v, lv_at, tile + 3, part - kLoads, part - kLoads + 1, kSteady);
          }
        }
      }, std::make_integer_sequence<int, kTotal>{});
      __builtin_amdgcn_sched_barrier(0);
      l += sum;
      if (!kSteady && tile >= whole && wild) add_wild(tile, pf);
      if (kSteady || rest > 0) raise(x, false);
      if constexpr (kSteady) landed_barrier<4 * kLoads>();
      else arrive(rest);
    };
    const int steady = max(min(whole - 1, min(ntile, len / BN) - 4), 0);
    for (int tile = 0; tile < steady; ++tile) step(tile, std::true_type{});
    for (int tile = steady; tile < ntile; ++tile) step(tile, std::false_type{});
  } else {
    auto step = [&](int tile, auto mixed) {
      if constexpr (DT == SPECV_F32) {
        fill(tile);
        if (tile + 1 < ntile) load(tile + 1);
        lds_barrier();
      } else if (tile + 1 < ntile) {
        request_k(tile + 1);
        request_v(tile + 1);
      }
      if constexpr (decltype(mixed)::value) {
        tame(buffer(tile));
        lds_barrier();
      }
      // waves whose rows see nothing of the tile wait for the others
      if (!decltype(mixed)::value || (tile * BN * s.G < wrow + 32 && wrow < rows)) {
        f32x16 sc[NB];
        bf16x8 pf[NB * 2][NP];
        scores(tile, sc, mixed);
        raise(highest(sc), false);
        weights(sc, pf);
        values(tile, pf);
        if constexpr (decltype(mixed)::value)
          if (wild) add_wild(tile, pf);
      }
      if constexpr (DT == SPECV_F32) lds_barrier();
      else landed_barrier();
    };
    for (int tile = 0; tile < whole; ++tile) step(tile, std::false_type{});
    for (int tile = whole; tile < ntile; ++tile) step(tile, std::true_type{});
  }

  l = halves_sum(l);
  const bool there = wrow + col < rows, some = !(l == 0.f);
  const float inv = some ? 1.f / l : 0.f;
  const long orow = (static_cast<long>(at.first) + tok) * s.Hq + hq;
  if (p.lse && half == 0 && there) p.lse[orow] = kv_lse(m, l, some);
  if (__any(!some))  // a row of no weight (rare) is 0, whatever the values
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] = some ? o[d][i] : 0.f;
  auto value = [&](int d, int i) { return o[d][i] * inv; };
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
