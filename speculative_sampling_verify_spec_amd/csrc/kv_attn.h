// Attention of a draft's nodes over the 8-bit paged cache and over the nodes
// themselves (the kernel template; k_kv_attn_<dim>.hip instantiate it).
//
// The R = N G queries that share a cached head (N nodes, G query heads per
// cached head) are the columns of every product, so a cached byte is read
// once for all of them:
//   S^T = K Q^T       A = 16 tokens x 32 channels,  B = 32 channels x 16 queries
//   O^T += V^T P^T    A = 16 channels x 32 tokens,  B = 32 tokens x 16 queries
// with v_mfma_f32_16x16x32_bf16.  Codes become bf16 exactly (4 or 7
// significant bits); a block's K scale multiplies the scores of its tokens,
// its V scale their weights.
//
// A wave takes 64 tokens at a time.  Tile t (0..3) of S^T has token 16 (i/4)
// + 4 t + i%4 in its row i, so that the four results a lane gets from each of
// the four tiles belong to 16 consecutive tokens: the softmax's weights are
// then already the B operand of the second product, and the matching A
// operand is 16 consecutive bytes of a transposed V page.  No cached byte
// passes through LDS (the queries' fragments do, where they would cost too
// many registers), there is no barrier in the loop, and every load is 16 bytes
// a lane.  The channels of Q are permuted the way 16-byte loads of K deliver
// them.
//
// Bound by reading the cache once: 256 x 9 positions (G = 4, D = 128, e4m3)
// over 1001-4097 tokens take 280 us, 5.0 TB/s; 512 x 1 (G = 8, D = 256, int8)
// 215 us, 4.8 TB/s; equal lengths of 2560 with one position 6.1 TB/s.  Many
// queries are bound by instruction issue instead: 128 trees of 32 nodes 223 us
// for 90 GFLOP, 61 % of it VALU (conversions, exponentials) and 21 % MFMA.
//
// Softmax: the running maximum is held per query and only moved when a tile
// exceeds it by more than 2^8 (the weights then stay below 2^8, and the sums
// are in 32 bits), so most tiles rescale nothing.
//
// 32-bit inputs: q, the weights, and the nodes' k and v are split into three
// bf16 pieces whose sum has 24 bits; products with codes take three matrix
// instructions, products of two split operands the six largest of nine.
#pragma once

#include <cfloat>

#include "sv_device.h"
#include "sv_kv.h"
#include "sv_mfma.h"
#include "sv_tree.h"

namespace sv {

namespace {

using namespace frag;

constexpr float kLazyMax = 8.f;  // log2: how far a score may exceed the held maximum

// V scales below this count as 0 with bf16 weights: the values are below
// 2^-77, and weights down to 2^-40 stay in the sums beside scales above it.
constexpr float kFlatScale = 0x1p-86f;

// The bytes of a word of codes that are NaN.
template <int FMT>
__device__ inline uint32_t nan_bytes(uint32_t w) {
  if constexpr (FMT == SPECV_E4M3) return ((((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xffu;
  else return 0;
}

// Eight consecutive elements as NP operand fragments.
template <int DT>
__device__ inline void load8(const void* base, long i, bf16x8* frag) {
  if constexpr (DT == SPECV_BF16) {
    frag[0] = *reinterpret_cast<const bf16x8*>(static_cast<const uint16_t*>(base) + i);
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    const float4 x = p[0], y = p[1];
    const float f[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      __bf16 s[3];
      split<3>(f[j], s);
      frag[0][j] = s[0];
      frag[1][j] = s[1];
      frag[2][j] = s[2];
    }
  }
}

template <int DT>
__device__ inline float load1(const void* base, long i) {
  if constexpr (DT == SPECV_F32) return static_cast<const float*>(base)[i];
  else return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(base)[i]) << 16);
}

constexpr int kAWaves = 4, kABlock = kAWaves * kWave;  // waves and threads per workgroup
constexpr int kTile = 64;                       // cached tokens a wave takes at a time

// The queries' fragments stay in registers if they take at most 16: 2 x 8
// positions (G = 4, D = 64) over 900 tokens take 12.7 us, through LDS 13.2; 2 x 2
// with D = 96 11.7 and 12.1; long caches differ by 1 %.  24 would spill
// (32-bit, D = 64: 128 registers for four waves; 36.0 us against 37.8).
constexpr bool q_in_lds(int dt, int D, int MT) { return MT * (dt == SPECV_F32 ? 3 : 1) * D / 8 > 16; }

// Waves a SIMD should hold, which bounds the registers of each to 512 /
// waves: the most that fit without spilling (the build refuses spills).
constexpr int waves_per(int dt, int D, int MT) {
  if (D == 256) return dt == SPECV_F32 ? 1 : 2;
  if (MT == 1) return D == 64 ? 4 : dt == SPECV_F32 ? 2 : 3;
  if (MT == 2) return D == 64 && dt == SPECV_BF16 ? 3 : 2;
  return 2;
}

// One workgroup: MT x 16 queries of one (sequence, cached head) over one of
// the parts of the sequence's tokens; its waves take the part's tiles in turn.
template <int DT, int FMT, int D, int MT>
__global__ __launch_bounds__(kABlock, waves_per(DT, D, MT)) void k_kv_attn(KvAttn p) {
  constexpr int NP = kPieces<DT>, NF = D / 32, ND = D / 16, NC = D / 64;
  const KvView& c = p.c;
  // workgroups of one part and head that differ only in their queries read
  // the same cache: eight apart, they run on the same XCD and share its L2
  const unsigned per = 8 * p.mb, outer = blockIdx.x / per * 8 + blockIdx.x % 8;
  const int mblk = blockIdx.x % per / 8;
  const unsigned pair = outer / static_cast<unsigned>(p.splits);
  const int part = static_cast<int>(outer - pair * p.splits);
  const unsigned seq = pair / static_cast<unsigned>(c.H);
  if (seq >= static_cast<unsigned>(p.B)) return;
  const int h = static_cast<int>(pair - seq * c.H);
  const long b = seq;
  const int lane = threadIdx.x % kWave, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int col = lane % 16, g = lane / 16;
  // page of this lane's 16 tokens (group g) of a tile, -1: none
  auto page_of = [&](int tile) {
    const unsigned tok = static_cast<unsigned>(tile) * kTile + 16 * g;
    return kv_page(c, b, tok >> c.pshift);
  };
  // the first pages are looked up beside the length, not after it
  int tile = part * p.granule + w;
  int pid = page_of(tile), pid_next = page_of(tile + kAWaves);
  const int len = kv_len(c, p.lengths, b);
  const int ntile = (len >> 6) + ((len & 63) != 0);
  const int parts = kv_parts(ntile, p.granule);
  if (part >= parts) return;
  const int nn = p.nodes ? min(max(p.nodes[b], 0), p.N) : p.N;
  const int rows = nn * p.G;           // queries that exist
  const int row0 = mblk * MT * 16;
  // r / G: exact, (r + 1/2) / G is at least 2^-11 from an integer and off by 2^-17 at most
  auto node_of = [&](int r) { return static_cast<int>((r + 0.5f) * p.inv_g); };

  // one buffer in LDS: the queries' fragments during the loop (where they
  // would take too many registers), the waves' sums at the join
  constexpr bool QL = q_in_lds(DT, D, MT);
  constexpr int TV = (ND + kAWaves - 1) / kAWaves;  // blocks of 16 channels that a wave finishes
  constexpr int kJoinBytes = kAWaves * (kAWaves - 1) * MT * TV * kWave * 16, kQBytes = QL ? MT * NF * NP * kWave * 16 : 0;
  __shared__ __align__(16) char lds[kJoinBytes > kQBytes ? kJoinBytes : kQBytes];
  bf16x8* const lq = reinterpret_cast<bf16x8*>(lds);

  // ---- queries: B operands, negated where the scale is (kept >= 0) ----
  const float kscale = fabsf(p.scale) * kLog2e;
  constexpr int QF = QL ? (NF + kAWaves - 1) / kAWaves : NF;  // fragments this wave loads
  bf16x8 qreg[MT][QF][NP];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int r = min(row0 + mt * 16 + col, p.N * p.G - 1);  // a row that exists; what others give is not written
    const int n = node_of(r);
    const long base = (b * p.N + n) * p.q_row + static_cast<long>(h * p.G + (r - n * p.G)) * D;
#pragma unroll
    for (int f = 0; f < QF; ++f) {
      const int frag = QL ? min(f * kAWaves + w, NF - 1) : f;
      load8<DT>(p.q, base + chan<D>(frag, g), qreg[mt][f]);
    }
  }
  auto query = [&](int mt, int f, int i) -> bf16x8 {
    if constexpr (QL) return lq[((mt * NF + f) * NP + i) * kWave + lane];
    else return qreg[mt][f][i];
  };

  f32x4 o[MT][ND];
  float m[MT], l[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    m[mt] = -INFINITY;
    l[mt] = 0.f;
#pragma unroll
    for (int d = 0; d < ND; ++d) o[mt][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  // moves the held maximum of a query to the largest x of its four lanes where
  // one exceeds it by too much; each query decides for itself, so that its
  // bits do not depend on what the queries beside it see
  auto raise = [&](int mt, float x) {
    if (!__any(x > m[mt] + kLazyMax)) return;  // true for the first finite x
    x = groups_max(x);
    const bool need = x > m[mt] + kLazyMax;
    const float a = need ? ex2(m[mt] - x) : 1.f;
    m[mt] = need ? x : m[mt];
    l[mt] *= a;
#pragma unroll
    for (int d = 0; d < ND; ++d) o[mt][d] *= a;
  };

  // ---- cached tokens ----
  const int tile1 = min((part + 1) * p.granule, ntile);
  // K is kept a tile ahead, or half a tile where registers are short
  // (D = 256: two waves a SIMD instead of one, 263 us against 319 at B = 512, N = 1)
  constexpr int KB = D == 256 ? 2 : 4;
  uint4 kraw[KB][NC], vraw[ND];
  uint2 ktail[KB];
  const size_t blkbytes = static_cast<size_t>(c.P) * D;
  // this lane's row of K: token 16 (col / 4) + col % 4 of a tile
  auto k_rows = [&](int tile, int pid) -> const uint8_t* {
    const int grp = col >> 2;
    const int id = max(__shfl(pid, grp * 16, kWave), 0);
    const int off = ((tile % 2 * kTile + 16 * grp) & (c.P - 1)) + (col & 3);  // pages of at most two tiles
    return c.kp + (static_cast<size_t>(id) * c.H + h) * blkbytes + static_cast<size_t>(off) * D;
  };
  auto load_k = [&](const uint8_t* a, int t) {
#pragma unroll
    for (int i = 0; i < NC; ++i) kraw[t % KB][i] = *reinterpret_cast<const uint4*>(a + 4 * t * D + 64 * i + 16 * g);
    if constexpr (NF % 2) ktail[t % KB] = *reinterpret_cast<const uint2*>(a + 4 * t * D + 64 * NC + 8 * g);
  };
  float ks = 0.f, vs = 0.f;
  auto load_v = [&](int tile, int pid) {
    const size_t blk = static_cast<size_t>(max(pid, 0)) * c.H + h;
    const uint8_t* a = c.vp + blk * blkbytes + static_cast<size_t>(col) * c.P + ((tile % 2 * kTile + 16 * g) & (c.P - 1));
    const size_t step = static_cast<size_t>(16) * c.P;
    // four addresses at a time: all of them at once would cost registers at
    // the loop's fullest point.  Pages of up to 64 tokens are read in whole
    // lines and past the caches (B = 256, N = 1, 2560 tokens: 217 us against
    // 240); a tile of a 128-token page has half of each line, and the other
    // half should be found in the cache (238 us against 279); so should what
    // other workgroups of the same head read again (tree 240 us against 248).
    if (c.P < 128 && p.mb == 1) {
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        if (d % 4 == 0) __builtin_amdgcn_sched_barrier(0);
        vraw[d] = load16_nt(a + d * step, 0);
      }
    } else {
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        if (d % 4 == 0) __builtin_amdgcn_sched_barrier(0);
        vraw[d] = load16(a + d * step, 0);
      }
    }
    ks = c.ks[blk];
    vs = c.vs[blk];
  };
  const uint8_t* this_k = nullptr;
  if (tile < tile1) {
    this_k = k_rows(tile, pid);
#pragma unroll
    for (int t = 0; t < KB; ++t) load_k(this_k, t);
    load_v(tile, pid);
  }
  // the queries, requested first, are here before the cached bytes
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int f = 0; f < QF; ++f)
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        if (p.scale < 0.f) qreg[mt][f][i] = -qreg[mt][f][i];
        if constexpr (QL)
          if (f * kAWaves + w < NF) lq[((mt * NF + f * kAWaves + w) * NP + i) * kWave + lane] = qreg[mt][f][i];
      }
  if constexpr (QL) lds_barrier();
  // ---- the nodes, 16 a wave, with the last part: while the first tile is
  // on its way, and with every load requested before the first is needed ----
  static_assert(SPECV_MAX_TREE <= 16 * kAWaves, "a wave has one block of 16 nodes");
  const int j0 = 16 * w;
  if (p.kn && part == parts - 1 && j0 < nn) {
    constexpr int VG = ND < 8 ? ND : 8;  // blocks of 16 channels of V at a time
    const long at0 = b * p.N * p.kv_row + static_cast<long>(h) * D;
    float vn[VG][4];
    auto load_vn = [&](int d0) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const long at = at0 + min(j0 + 4 * g + r, p.N - 1) * p.kv_row + col;
#pragma unroll
        for (int d = 0; d < VG; ++d) vn[d][r] = load1<DT>(p.vn, at + 16 * (d0 + d));
      }
    };
    bf16x8 kf[NF][NP];
#pragma unroll
    for (int f = 0; f < NF; ++f) load8<DT>(p.kn, at0 + min(j0 + col, p.N - 1) * p.kv_row + chan<D>(f, g), kf[f]);
    load_vn(0);
    uint64_t set = 0;
    if (p.parents) {
      bool valid;
      int depth;
      ancestor_sets(p.parents + b * p.N, p.N, set, valid, depth);
    } else {
      set = ~0ull >> (63 - lane);
    }
    uint32_t sees[MT];  // bit i: the query sees node j0 + i
    f32x4 s[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int r = row0 + mt * 16 + col;
      const uint32_t x = static_cast<uint32_t>(__shfl(static_cast<int>(set >> j0), r < rows ? node_of(r) : 0, kWave));
      sees[mt] = r < rows ? x & 0xffffu : 0u;
      s[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int z = NP - 1; z >= 0; --z)
#pragma unroll
          for (int i = 0; i <= z; ++i) s[mt] = mfma(kf[f][z - i], query(mt, f, i), s[mt]);
    bf16x8 pf[MT][NP];
    float keep[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float x = -INFINITY;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool ok = (sees[mt] >> (4 * g + r)) & 1;
        s[mt][r] = ok ? s[mt][r] * kscale : -INFINITY;
        x = fmaxf(x, s[mt][r]);
      }
      m[mt] = fmaxf(m[mt], -FLT_MAX);  // finite: a node's score can be -infinity where it is seen, too
      raise(mt, x);
#pragma unroll
      for (int i = 0; i < NP; ++i) pf[mt][i] = bf16x8{};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool ok = (sees[mt] >> (4 * g + r)) & 1;
        const float e = ok ? ex2(s[mt][r] - m[mt]) : 0.f;
        l[mt] += e;
        keep[mt][r] = e;
        __bf16 piece[3];
        split<NP>(e, piece);
#pragma unroll
        for (int i = 0; i < NP; ++i) pf[mt][i][r] = piece[i];
      }
    }
    // values that are not finite must not meet a weight of 0: they stay out
    // of the products and are added where they are seen
    bool wild = false;
#pragma unroll
    for (int d0 = 0; d0 < ND; d0 += VG) {
      if (d0) load_vn(d0);
#pragma unroll
      for (int d = 0; d < VG; ++d) {
        if (d0 + d >= ND) break;
        bf16x8 vf[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) vf[i] = bf16x8{};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float x = j0 + 4 * g + r < nn ? vn[d][r] : 0.f;
          if (!isfinite(x)) {
            wild = true;
            x = 0.f;
          }
          __bf16 piece[3];
          split<NP>(x, piece);
#pragma unroll
          for (int i = 0; i < NP; ++i) vf[i][r] = piece[i];
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int z = NP - 1; z >= 0; --z)
#pragma unroll
            for (int i = 0; i <= z; ++i) o[mt][d0 + d] = mfma(vf[z - i], pf[mt][i], o[mt][d0 + d]);
      }
    }
    if (__any(wild)) {
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {  // nodes j0 + 4 k + i: lane group k holds their weights
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = j0 + 4 * k + i;
          const long at = at0 + min(j, p.N - 1) * p.kv_row + 4 * g;
          float e[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) e[mt] = __shfl(keep[mt][i], col + 16 * k, kWave);
#pragma unroll
          for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              // few loads at a time: this rare part's registers count for the whole kernel's occupancy
              if (r == 0) __builtin_amdgcn_sched_barrier(0);
              const float x = load1<DT>(p.vn, at + 16 * d + r);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
                if (!isfinite(x) && ((sees[mt] >> (4 * k + i)) & 1) && j < nn) o[mt][d][r] += e[mt] * x;
            }
        }
      }
    }
  }

  for (; tile < tile1; tile += kAWaves) {
    const bool more = tile + kAWaves < tile1;
    // tokens of this lane's 16 that exist; the bytes behind them, and scales
    // of no page, may be anything (NaN too) and are cleared.  So are values
    // whose block has next to no magnitude (blocks of zeros have the smallest
    // scale): a weight times such a scale could vanish from the weights' sum.
    // NaN has no magnitude, and stays.
    const int have = pid < 0 ? 0 : min(max(len - tile * kTile - 16 * g, 0), 16);
    const bool flat = NP == 1 && !(vs >= kFlatScale);
    const bool whole = __all(have == 16 && !flat);
    if (!whole) {
      if (have == 0) ks = 1.f;
      if (have == 0 || flat) vs = 1.f;
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        uint32_t* x = reinterpret_cast<uint32_t*>(&vraw[d]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = have - 4 * i;
          x[i] &= n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
        }
      }
      if (__any(flat))
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          uint32_t* x = reinterpret_cast<uint32_t*>(&vraw[d]);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] &= flat ? nan_bytes<FMT>(x[i]) : ~0u;
        }
    }
    // > 0 also for a scale of 0, so that a masked score of -inf stays -inf; the
    // smallest number there is, which leaves the other scores below 2^-33
    const float kc = fmaxf(ks * kscale, 0x1p-149f);
    // bf16: the V scale enters as its logarithm (exact for a power of two)
    const float lvs = NP == 1 ? __builtin_amdgcn_logf(vs) : 0.f, per_vs = NP == 1 ? 1.f / vs : 1.f;
    const uint8_t* next_k = more ? k_rows(tile + kAWaves, pid_next) : nullptr;
#pragma unroll
    for (int j = 0; j < 2; ++j) {  // halves of the tile: 8 of each lane's 16 tokens
      // the queries' fragments are read from LDS here, not kept across the loop
      if constexpr (QL) asm volatile("" ::: "memory");
      f32x4 s[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) s[mt][0] = s[mt][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        bf16x8 kf[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint4 x = kraw[(2 * j + t) % KB][f / 2 < NC ? f / 2 : 0];
          kf[t] = f >= 2 * NC ? codes8<FMT>(ktail[(2 * j + t) % KB].x, ktail[(2 * j + t) % KB].y)
                  : f % 2     ? codes8<FMT>(x.z, x.w)
                              : codes8<FMT>(x.x, x.y);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = NP - 1; i >= 0; --i) {
            const bf16x8 q = query(mt, f, i);
            s[mt][0] = mfma(kf[0], q, s[mt][0]);
            s[mt][1] = mfma(kf[1], q, s[mt][1]);
          }
      }
      // weights as the B operand: bf16 (half a step of 2^-8 relative, as the
      // output's own type has), or their three pieces
      bf16x8 pf[MT][NP];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (!whole) {
          m[mt] = fmaxf(m[mt], -FLT_MAX);  // finite, also while the query has seen nothing
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (8 * j + e >= have) s[mt][e / 4][e % 4] = -INFINITY;
        }
        float x = s[mt][0][0];
#pragma unroll
        for (int e = 1; e < 8; ++e) x = fmaxf(x, s[mt][e / 4][e % 4]);
        raise(mt, x * kc);
        const float shift = lvs - m[mt];
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float y = ex2(fmaf(s[mt][e / 4][e % 4], kc, shift));
          sum += y;
          __bf16 piece[3];
          split<NP>(NP == 1 ? y : y * vs, piece);
#pragma unroll
          for (int i = 0; i < NP; ++i) pf[mt][i][e] = piece[i];
        }
        l[mt] += sum * per_vs;
      }
      if (KB == 2 && j == 0) {
        load_k(this_k, 2);
        load_k(this_k, 3);
      } else if (more) {
        load_k(next_k, KB == 2 ? 0 : 2 * j);
        load_k(next_k, KB == 2 ? 1 : 2 * j + 1);
      }
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const bf16x8 vf = j ? codes8<FMT>(vraw[d].z, vraw[d].w) : codes8<FMT>(vraw[d].x, vraw[d].y);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = NP - 1; i >= 0; --i) o[mt][d] = mfma(vf, pf[mt][i], o[mt][d]);
      }
    }
    if (more) load_v(tile + kAWaves, pid_next);
    this_k = next_k;
    pid = pid_next;
    pid_next = page_of(tile + 2 * kAWaves);
  }

  // ---- join the waves: each finishes TV blocks of channels, to which the
  // others hand their sums, all scaled to the queries' largest maximum ----
  // the lane's number again, so that nothing of it is kept across the loop
  const int jl = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u)), jc = jl % 16, jg = jl / 16;
  __shared__ float sm[kAWaves][MT * 16], sl[kAWaves][MT * 16];
  f32x4* const so = reinterpret_cast<f32x4*>(lds);
  auto slot = [&](int to, int from, int mt, int t) {
    return (((to * (kAWaves - 1) + from - (from > to)) * MT + mt) * TV + t) * kWave + jl;
  };
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    l[mt] = groups_sum(l[mt]);
    if (jg == 0) {
      sm[w][mt * 16 + jc] = m[mt];
      sl[w][mt * 16 + jc] = l[mt];
    }
  }
  lds_barrier();  // also: the queries' fragments are no longer read
  float scale[MT], inv[MT];  // what this wave's sums, and the whole sums, are multiplied by
  long orow[MT];             // the queries' output rows, -1: no such row
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    float mk[kAWaves], lk[kAWaves];
#pragma unroll
    for (int k = 0; k < kAWaves; ++k) {
      mk[k] = sm[k][mt * 16 + jc];
      lk[k] = sl[k][mt * 16 + jc];
    }
    float top = mk[0], lt = 0.f;
#pragma unroll
    for (int k = 1; k < kAWaves; ++k) top = fmaxf(top, mk[k]);
#pragma unroll
    for (int k = 0; k < kAWaves; ++k)
      lt += mk[k] == -INFINITY ? lk[k] : lk[k] * ex2(mk[k] - top);  // 0, or NaN of a wave that saw only NaN
    scale[mt] = m[mt] == -INFINITY ? 0.f : ex2(m[mt] - top);
    const int r = row0 + mt * 16 + jc;
    const int n = node_of(r);
    const bool there = r < p.N * p.G;
    orow[mt] = there ? (b * p.N + n) * p.Hq + h * p.G + (r - n * p.G) : -1;
    const bool some = r < rows && !(lt == 0.f);  // a query that exists and sees something
    inv[mt] = parts > 1 ? 1.f : some ? 1.f / lt : 0.f;
    if (there && w == 0 && jg == 0) {
      if (parts > 1) p.part_ml[orow[mt] * p.splits + part] = make_float2(top, lt);
      else if (p.lse) p.lse[orow[mt]] = kv_lse(top, lt, some);
    }
  }
#pragma unroll
  for (int d = 0; d < ND; ++d)
    if (d / TV != w)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) so[slot(d / TV, w, mt, d % TV)] = o[mt][d] * scale[mt];
  lds_barrier();
  if (w * TV >= ND) return;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int t = 0; t < TV; ++t) {
      f32x4 mine = o[mt][t];  // o[mt][w * TV + t]
#pragma unroll
      for (int k = 1; k < kAWaves; ++k)
        if (k * TV + t < ND) mine = w == k ? o[mt][k * TV + t] : mine;
      mine *= scale[mt];
      f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < kAWaves; ++k) {  // in the waves' order
        const f32x4 x = so[slot(w, k == w ? (w ? 0 : 1) : k, mt, t)];
        acc += k == w ? mine : x;
      }
      if (orow[mt] < 0) continue;
      const int d = 16 * (w * TV + t) + 4 * jg;
      if (parts > 1) {
        *reinterpret_cast<f32x4*>(p.part_o + (orow[mt] * p.splits + part) * D + d) = acc;
      } else {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = inv[mt] == 0.f ? 0.f : acc[e] * inv[mt];  // 0 whatever the sums are
        kv_store4<DT>(p.out, orow[mt] * D + d, y);
      }
    }
}

template <int DT, int FMT, int D, int MT>
hipError_t launch_one(const KvAttn& p, hipStream_t st) {
  const long outer = (static_cast<long>(p.B) * p.c.H * p.splits + 7) / 8 * 8;
  hipLaunchKernelGGL((k_kv_attn<DT, FMT, D, MT>), dim3(static_cast<unsigned>(outer * p.mb)), dim3(kABlock), 0, st, p);
  return hipGetLastError();
}

// The kernel for p.mt blocks of 16 queries (at most kv_max_mt).
template <int DT, int FMT, int D>
hipError_t launch_mt(const KvAttn& p, hipStream_t st) {
  constexpr int most = kv_max_mt(DT, D);
  if (p.mt == 1) return launch_one<DT, FMT, D, 1>(p, st);
  if constexpr (most >= 2)
    if (p.mt == 2) return launch_one<DT, FMT, D, 2>(p, st);
  if constexpr (most >= 3)
    if (p.mt == 3) return launch_one<DT, FMT, D, 3>(p, st);
  if constexpr (most >= 4)
    if (p.mt == 4) return launch_one<DT, FMT, D, 4>(p, st);
  return hipErrorInvalidValue;
}

template <int D>
hipError_t launch_dim(const KvAttn& p, int dtype, int fmt, hipStream_t st) {
  if (dtype == SPECV_F32)
    return fmt == SPECV_E4M3 ? launch_mt<SPECV_F32, SPECV_E4M3, D>(p, st) : launch_mt<SPECV_F32, SPECV_I8, D>(p, st);
  return fmt == SPECV_E4M3 ? launch_mt<SPECV_BF16, SPECV_E4M3, D>(p, st) : launch_mt<SPECV_BF16, SPECV_I8, D>(p, st);
}

}  // namespace

}  // namespace sv
