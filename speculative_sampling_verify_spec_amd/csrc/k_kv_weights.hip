// The attention weight that cached tokens gather from the nodes a round keeps:
//   w[j] += sum over the kept nodes i, and the query heads that share the
//           cached head, of e^(scale q_i . k_j - lse_i),
// and, for the kept nodes themselves, that behind the cached ones the weights
// from the nodes of the path that see them.
//
// A wave takes 64 tokens at a time: their K codes become bf16 exactly and are
// the B operand (32 channels x 16 tokens) of v_mfma_f32_16x16x32_bf16, 16 rows
// (query head r % G of path node r / G) the A operand.  A lane then has one
// token of each of the four groups of 16, and the sum over rows stays in its
// registers until the four lanes of a token join it at the end.
#include "sv_budget.h"
#include "sv_device.h"
#include "sv_mfma.h"

namespace sv {

namespace {

using namespace frag;

constexpr int kGWaves = 4, kGBlock = kGWaves * kWave;
constexpr int kGTile = 64;

// Eight codes to bf16, exact.
template <int FMT>
__device__ inline bf16x8 code_frag(uint32_t a, uint32_t b) {
  float f[8];
  kv_decode4<FMT>(a, f);
  kv_decode4<FMT>(b, f + 4);
  bf16x8 v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __builtin_bit_cast(__bf16, static_cast<uint16_t>(__float_as_uint(f[i]) >> 16));
  return v;
}

__device__ inline f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// First channel of the 8 that lane group g holds of fragment f: fragments 2c
// and 2c + 1 are the halves of the 16 codes a lane loads of 64 channels; a
// last odd fragment is an 8-byte load of 32.
template <int D>
__device__ inline int channel(int f, int g) {
  return f < D / 64 * 2 ? f / 2 * 64 + 16 * g + f % 2 * 8 : D / 64 * 64 + 8 * g;
}

template <int DT, int FMT, int D>
__global__ __launch_bounds__(kGBlock) void k_kv_weights(KvWeights p) {
  constexpr int NP = kPieces<DT>, NF = D / 32, NC = D / 64, NT = kGTile / 16;
  const KvView& c = p.c;
  const unsigned pair = blockIdx.x / p.splits, split_no = blockIdx.x - pair * p.splits;
  const long b = pair / static_cast<unsigned>(c.H);
  const int h = static_cast<int>(pair - b * c.H);
  const int lane = threadIdx.x % kWave, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int col = lane % 16, g = lane / 16;

  // the path: every wave finds it for itself, a lane per node
  int want = p.N;
  if (p.counts) want = min(max(p.counts[b], 0), p.N);
  int node = lane;
  if (p.index && lane < p.N) node = p.index[b * p.N + lane];
  const uint64_t bad = __ballot(lane >= want || node < 0 || node >= p.N);
  const int count = bad ? __builtin_ctzll(bad) : kWave;
  const int rows = count * p.G;
  const int len = kv_len(c, p.lengths, b);
  const float* const wrow = p.w + (b * c.H + h) * p.capacity;
  float* const orow = p.out + (b * c.H + h) * p.capacity;
  const float kscale = p.scale * kLog2e;

  // a row's query fragments and the statistics of this lane's four rows
  auto query = [&](int row0, bf16x8 (*q)[NP], float* l2) {
    {
      const int r = max(min(row0 + col, rows - 1), 0), slot = r / p.G;
      const long n = __shfl(node, slot, kWave);
      const long base = (b * p.N + n) * p.q_row + static_cast<long>(h * p.G + (r - slot * p.G)) * D;
      Raw8<DT> x[NF];
#pragma unroll
      for (int f = 0; f < NF; ++f) x[f].load(p.q, base + channel<D>(f, g));
#pragma unroll
      for (int f = 0; f < NF; ++f) x[f].pieces(q[f]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = row0 + 4 * g + i, rr = max(min(r, rows - 1), 0), slot = rr / p.G;
      const long n = __shfl(node, slot, kWave);
      const float x = p.lse[(b * p.N + n) * p.Hq + h * p.G + (rr - slot * p.G)];
      l2[i] = r >= rows || x == -INFINITY ? INFINITY : x * kLog2e;  // rows that weigh nothing
    }
  };

  const int ntile = (len + kGTile - 1) / kGTile;
  const int stride = static_cast<int>(p.splits) * kGWaves;
  for (int tile = static_cast<int>(split_no) * kGWaves + w; tile < ntile; tile += stride) {
    bf16x8 k[NT][NF];
    float kc[NT], sum[NT];
    bool seen[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int tok = tile * kGTile + 16 * t + col;
      const int page = tok < len ? kv_page(c, b, tok >> c.pshift) : -1;
      seen[t] = page >= 0;
      const size_t blk = static_cast<size_t>(max(page, 0)) * c.H + h;
      kc[t] = c.ks[blk] * kscale;
      const uint8_t* a = c.kp + (blk * c.P + (tok & (c.P - 1))) * D;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(a + 64 * i + 16 * g);
        k[t][2 * i] = code_frag<FMT>(x.x, x.y);
        k[t][2 * i + 1] = code_frag<FMT>(x.z, x.w);
      }
      if constexpr (NF % 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(a + 64 * NC + 8 * g);
        k[t][NF - 1] = code_frag<FMT>(x.x, x.y);
      }
      sum[t] = 0.f;
    }
    for (int row0 = 0; row0 < rows; row0 += 16) {
      bf16x8 q[NF][NP];
      float l2[4];
      query(row0, q, l2);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
          for (int i = NP - 1; i >= 0; --i) s = mfma16(q[f][i], k[t][f], s);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[t] += ex2(fmaf(s[i], kc[t], -l2[i]));
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float x = sum[t];
      x += __shfl_xor(x, 16, kWave);
      x += __shfl_xor(x, 32, kWave);
      const int tok = tile * kGTile + 16 * t + col;
      if (g == 0 && tok < len) orow[tok] = seen[t] ? wrow[tok] + x : wrow[tok];
    }
  }

  // the path's own tokens: one group of 16 a wave, by the first workgroup
  if (split_no != 0 || !p.kn) return;
  if (16 * w >= count) return;
  const int mine = 16 * w + col;  // path node, as a key
  bf16x8 k[NF][NP];
  {
    const long n = __shfl(node, min(mine, count - 1), kWave);
    const long base = (b * p.N + n) * p.k_row + static_cast<long>(h) * D;
    Raw8<DT> x[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) x[f].load(p.kn, base + channel<D>(f, g));
#pragma unroll
    for (int f = 0; f < NF; ++f) x[f].pieces(k[f]);
  }
  float sum = 0.f;
  for (int row0 = 16 * w * p.G; row0 < rows; row0 += 16) {
    bf16x8 q[NF][NP];
    float l2[4];
    query(row0, q, l2);
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int z = NP - 1; z >= 0; --z)
#pragma unroll
        for (int i = 0; i <= z; ++i) s = mfma16(q[f][i], k[f][z - i], s);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (row0 + 4 * g + i >= mine * p.G) sum += ex2(fmaf(s[i], kscale, -l2[i]));
  }
  sum += __shfl_xor(sum, 16, kWave);
  sum += __shfl_xor(sum, 32, kWave);
  const long pos = static_cast<long>(len) + mine;
  if (g == 0 && mine < count && pos < p.capacity) orow[pos] = sum;
}

template <int DT, int FMT, int D>
hipError_t launch_one(const KvWeights& p, hipStream_t st) {
  const unsigned grid = static_cast<unsigned>(p.B) * static_cast<unsigned>(p.c.H) * p.splits;
  hipLaunchKernelGGL((k_kv_weights<DT, FMT, D>), dim3(grid), dim3(kGBlock), 0, st, p);
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
