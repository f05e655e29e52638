// The attention weight that cached tokens gather from the nodes a round keeps:
//   w[j] += sum over the kept nodes i, and the query heads that share the
//           cached head, of e^(scale q_i . k_j - lse_i),
// and, for the kept nodes themselves, that behind the cached ones the weights
// from the nodes of the path that see them.
//
// The rows (query head r % G of path node r / G) are put into LDS once as A
// operands of v_mfma_f32_16x16x32_bf16, 16 rows x 32 channels each, with their
// statistics.  A wave then takes 64 tokens at a time, whose K codes become
// bf16 exactly and are the B operands (32 channels x 16 tokens).  A lane has
// one token of each of the four groups of 16, and the sum over rows stays in
// its registers until the four lanes of a token join it at the end.  More rows
// than LDS takes are gone through in turns, which add to each other's sums.
//
// Bound by reading K, every page once a turn: 256 paths of trees over 97-2500
// tokens (8 heads of 128, int8) 89 us, 4.0 TB/s; 64 single tokens over 301-2111
// 23 us, of which the chain length - page - codes at the beginning and the join
// are 10.  Turns of 32 instead of 64 KiB of rows take the same there.  With 32-bit
// queries the paths take 119 us, the single tokens 27.
#include <algorithm>

#include "sv_budget.h"
#include "sv_device.h"
#include "sv_mfma.h"

namespace sv {

namespace {

using namespace frag;

constexpr int kGWaves = 4, kGBlock = kGWaves * kWave;
constexpr int kGTile = 64;
constexpr int kGMostLds = 64 << 10;  // bytes of row fragments: two workgroups a CU at least

// A row's weight of a token; a row of lse +infinity weighs nothing, whatever its
// score is (256 paths 88.9 us, without that 87.9).
__device__ inline float weight(float score, float scale, float lse) {
  return lse == INFINITY ? 0.f : ex2(fmaf(score, scale, -lse));
}

// Bytes of 16 rows in LDS.
template <int DT, int D>
constexpr int kRowBlock = D / 32 * kPieces<DT> * kWave * 16 + 64;

template <int DT, int FMT, int D>
__global__ __launch_bounds__(kGBlock, D == 256 ? 2 : D == 128 ? 3 : 4) void k_kv_weights(KvWeights p, int turn) {
  constexpr int NP = kPieces<DT>, NF = D / 32, NC = D / 64, NT = kGTile / 16;
  extern __shared__ __align__(16) char lds[];
  bf16x8* const lq = reinterpret_cast<bf16x8*>(lds);                                         // [turn / 16][NF][NP][kWave]
  float* const ll = reinterpret_cast<float*>(lds + turn / 16 * (NF * NP * kWave * 16));      // [turn], log2; +infinity: none
  const KvView& c = p.c;
  const unsigned pair = blockIdx.x / p.splits, split_no = blockIdx.x - pair * p.splits;
  const unsigned seq = pair / static_cast<unsigned>(c.H);
  const long b = seq;
  const int h = static_cast<int>(pair - seq * c.H);
  const int lane = threadIdx.x % kWave, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int col = lane % 16, g = lane / 16;

  const int stride = static_cast<int>(p.splits) * kGWaves;
  const int tile0 = static_cast<int>(split_no) * kGWaves + w;
  // page of this lane's token of a tile, -1: none; the first ones are looked up beside the length
  auto page_of = [&](int tile) { return kv_page(c, b, (static_cast<unsigned>(tile) * kGTile + lane) >> c.pshift); };
  const int pid_first = page_of(tile0);
  const int len = kv_len(c, p.lengths, b);
  const int ntile = (len + kGTile - 1) / kGTile;
  if (static_cast<int>(split_no) * kGWaves >= ntile && split_no != 0) return;

  // the path: every wave finds it for itself, a lane per node
  int want = p.N;
  if (p.counts) want = min(max(p.counts[b], 0), p.N);
  int node = lane;
  if (p.index && lane < p.N) node = p.index[b * p.N + lane];
  const uint64_t bad = __ballot(lane >= want || node < 0 || node >= p.N);
  const int count = bad ? __builtin_ctzll(bad) : kWave;
  const int rows = count * p.G;
  const float* const wrow = p.w + (b * c.H + h) * p.capacity;
  float* const orow = p.out + (b * c.H + h) * p.capacity;
  const float kscale = p.scale * kLog2e;
  const size_t blkbytes = static_cast<size_t>(c.P) * D;

  for (int row_at = 0; row_at == 0 || row_at < rows; row_at += turn) {
    const int have = min(rows - row_at, turn), nblock = (have + 15) / 16;  // rows and blocks of rows of this turn
    if (row_at) __syncthreads();
    // a block's fragments are loaded by one wave, statistics by a thread a row
    for (int k = w; k < nblock; k += kGWaves) {
      const int r = min(row_at + 16 * k + col, rows - 1), slot = r / p.G;
      const long n = __shfl(node, slot, kWave);
      const long base = (b * p.N + n) * p.q_row + static_cast<long>(h * p.G + (r - slot * p.G)) * D;
      Raw8<DT> x[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f) x[f].load(p.q, base + chan<D>(f, g));
      if (lane < 16) {
        const float l = p.lse[(b * p.N + n) * p.Hq + h * p.G + (r - slot * p.G)];
        ll[16 * k + lane] = 16 * k + lane >= have || l == -INFINITY ? INFINITY : l * kLog2e;  // rows that weigh nothing
      }
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        bf16x8 q[NP];
        x[f].pieces(q);
#pragma unroll
        for (int i = 0; i < NP; ++i) lq[((k * NF + f) * NP + i) * kWave + lane] = q[i];
      }
    }
    const float* const before = row_at ? orow : wrow;
    // ---- cached tokens ----
    int pid = pid_first;
    bool ready = false;
    for (int tile = tile0; tile < ntile; tile += stride) {
      uint4 raw[NT][NC > 0 ? NC : 1];
      uint2 tail[NT];
      float kc[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        // a group of 16 tokens lies in one page
        const int page = max(__builtin_amdgcn_readlane(pid, 16 * t), 0);
        const size_t blk = static_cast<size_t>(page) * c.H + h;
        const int off = (tile * kGTile + 16 * t) & (c.P - 1);
        const uint8_t* a = c.kp + blk * blkbytes + static_cast<size_t>(off + col) * D;
#pragma unroll
        for (int i = 0; i < NC; ++i) raw[t][i] = *reinterpret_cast<const uint4*>(a + 64 * i + 16 * g);
        if constexpr (NF % 2) tail[t] = *reinterpret_cast<const uint2*>(a + 64 * NC + 8 * g);
        kc[t] = c.ks[blk];
      }
      const int tok = tile * kGTile + lane;
      const float old = tok < len ? before[tok] : 0.f;
      const bool seen = pid >= 0;
      pid = page_of(tile + stride);
      if (!ready) __syncthreads();  // the rows are in LDS
      ready = true;
      float sum[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        sum[t] = 0.f;
        kc[t] *= kscale;
      }
      for (int k = 0; k < nblock; ++k) {
        const f32x4 l4 = *reinterpret_cast<const f32x4*>(&ll[16 * k + 4 * g]);
        f32x4 s[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) s[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          bf16x8 kf[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint4 x = raw[t][f / 2 < NC ? f / 2 : 0];
            kf[t] = f >= 2 * NC ? codes8<FMT>(tail[t].x, tail[t].y) : f % 2 ? codes8<FMT>(x.z, x.w) : codes8<FMT>(x.x, x.y);
          }
#pragma unroll
          for (int i = NP - 1; i >= 0; --i) {
            const bf16x8 q = lq[((k * NF + f) * NP + i) * kWave + lane];
#pragma unroll
            for (int t = 0; t < NT; ++t) s[t] = mfma(q, kf[t], s[t]);
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[t] += weight(s[t][i], kc[t], l4[i]);
      }
      // lane 16 t + col gets its token's sum
      float mine = 0.f;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float x = groups_sum(sum[t]);
        mine = g == t ? x : mine;
      }
      if (tok < len) orow[tok] = seen ? old + mine : old;
    }
    if (!ready) __syncthreads();
    // ---- the path's own tokens: one group of 16 a wave, by the first workgroup ----
    if (split_no == 0 && p.kn && 16 * w < count) {
      const int mine = 16 * w + col;  // path node, as a key
      const long n = __shfl(node, min(mine, count - 1), kWave);
      const long base = (b * p.N + n) * p.k_row + static_cast<long>(h) * D;
      const long pos = static_cast<long>(len) + mine;
      float sum = 0.f;
      for (int k = 0; k < nblock; ++k) {
        const int row0 = row_at + 16 * k;
        if (row0 + 15 < 16 * w * p.G) continue;  // before the group's first node
        const f32x4 l4 = *reinterpret_cast<const f32x4*>(&ll[16 * k + 4 * g]);
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          Raw8<DT> x;
          bf16x8 kf[NP];
          x.load(p.kn, base + chan<D>(f, g));
          x.pieces(kf);
#pragma unroll
          for (int z = NP - 1; z >= 0; --z)
#pragma unroll
            for (int i = 0; i <= z; ++i) s = mfma(lq[((k * NF + f) * NP + i) * kWave + lane], kf[z - i], s);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (row0 + 4 * g + i >= mine * p.G) sum += weight(s[i], kscale, l4[i]);
      }
      sum = groups_sum(sum);
      if (g == 0 && mine < count && pos < p.capacity) orow[pos] = row_at ? orow[pos] + sum : sum;
    }
  }
}

template <int DT, int FMT, int D>
hipError_t launch_one(const KvWeights& p, hipStream_t st) {
  const unsigned grid = static_cast<unsigned>(p.B) * static_cast<unsigned>(p.c.H) * p.splits;
  const int blocks = std::min(kGMostLds / (kRowBlock<DT, D>), (p.N * p.G + 15) / 16);
  const size_t bytes = static_cast<size_t>(blocks) * (kRowBlock<DT, D>);
  hipLaunchKernelGGL((k_kv_weights<DT, FMT, D>), dim3(grid), dim3(kGBlock), bytes, st, p, 16 * blocks);
  return hipGetLastError();
}

template <int DT, int FMT>
hipError_t launch_dims(const KvWeights& p, hipStream_t st) {
  return p.c.D == 64    ? launch_one<DT, FMT, 64>(p, st)
         : p.c.D == 96  ? launch_one<DT, FMT, 96>(p, st)
         : p.c.D == 128 ? launch_one<DT, FMT, 128>(p, st)
                        : launch_one<DT, FMT, 256>(p, st);
}

}  // namespace

hipError_t launch_kv_weights(const KvWeights& p, int dtype, int fmt, hipStream_t st) {
  if (dtype == SPECV_F32)
    return fmt == SPECV_E4M3 ? launch_dims<SPECV_F32, SPECV_E4M3>(p, st) : launch_dims<SPECV_F32, SPECV_I8>(p, st);
  return fmt == SPECV_E4M3 ? launch_dims<SPECV_BF16, SPECV_E4M3>(p, st) : launch_dims<SPECV_BF16, SPECV_I8>(p, st);
}

}  // namespace sv
