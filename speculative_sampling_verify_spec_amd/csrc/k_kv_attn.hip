// Attention of a draft's nodes over the 8-bit paged cache and over the nodes
// themselves.  One wave per (sequence, node, query head): 64 cached tokens at
// a time, one score per lane, with the running maximum and sum of the
// softmax; then every lane adds p v to its own channels.
#include "sv_device.h"
#include "sv_kv.h"

namespace sv {

namespace {

template <int DT>
__device__ inline float elt(const void* p, long i) {
  if constexpr (DT == SPECV_F32) return static_cast<const float*>(p)[i];
  else return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
}

constexpr int kMaxDim = 256;

template <int DT, int FMT>
__global__ __launch_bounds__(kWave) void k_kv_attn(KvAttn p) {
  const KvView& c = p.c;
  const int hq = blockIdx.x % p.Hq, n = blockIdx.x / p.Hq, lane = threadIdx.x;
  const long b = blockIdx.y;
  const int h = hq / p.G;
  __shared__ float sq[kMaxDim];
  __shared__ float sp[kWave];
  const long orow = (b * p.N + n) * p.Hq + hq;
  const int nn = p.nodes ? min(max(p.nodes[b], 0), p.N) : p.N;
  constexpr int kPer = kMaxDim / kWave;
  float o[kPer] = {0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;
  if (n < nn) {
    const float c2 = p.scale * 1.44269504088896f;
    for (int d = lane; d < c.D; d += kWave)
      sq[d] = elt<DT>(p.q, (b * p.N + n) * p.q_row + static_cast<long>(hq) * c.D + d) * c2;
    __syncthreads();
    const int len = kv_len(c, p.lengths, b);
    uint64_t set = 0;
    if (p.kn) {
      if (p.parents) {
        uint64_t mine;
        bool valid;
        int depth;
        ancestor_sets(p.parents + b * p.N, p.N, mine, valid, depth);
        set = __shfl(mine, n, kWave);
      } else {
        set = ~0ull >> (63 - n);
      }
    }
    for (int t0 = 0; t0 < len; t0 += kWave) {
      const int t = t0 + lane;
      const int id = t < len ? kv_page(c, b, t >> c.pshift) : -1;
      const int off = t & (c.P - 1);
      float s = -INFINITY, vs = 0.f;
      if (id >= 0) {
        const long blk = static_cast<long>(id) * c.H + h;
        const uint32_t* kr = reinterpret_cast<const uint32_t*>(c.kp + (blk * c.P + off) * c.D);
        s = 0.f;
        for (int d = 0; d < c.D; d += 4) {
          float f[4];
          kv_decode4<FMT>(kr[d / 4], f);
          for (int j = 0; j < 4; ++j) s += f[j] * sq[d + j];
        }
        s *= c.ks[blk];
        vs = c.vs[blk];
      }
      const float mn = fmaxf(m, wave_max(s));
      if (mn == -INFINITY) continue;  // uniform
      const float r = ex2(m - mn), e = ex2(s - mn);
      m = mn;
      l = l * r + wave_sum_f32(e);
      __syncthreads();
      sp[lane] = e * vs;
      __syncthreads();
      for (int i = 0; i < kPer; ++i) o[i] *= r;
      for (int j = 0; j < kWave && t0 + j < len; ++j) {
        const int idj = kv_page(c, b, (t0 + j) >> c.pshift);
        if (idj < 0) continue;
        const long blk = static_cast<long>(idj) * c.H + h;
        const uint8_t* vb = c.vp + blk * c.P * c.D + ((t0 + j) & (c.P - 1));
        for (int i = 0, d = lane; d < c.D; ++i, d += kWave) {
          float f[4];
          kv_decode4<FMT>(vb[static_cast<long>(d) * c.P], f);
          o[i] += sp[j] * f[0];
        }
      }
    }
    for (int j = 0; j < p.N; ++j) {
      if (!((set >> j) & 1)) continue;  // uniform
      const long at = (b * p.N + j) * p.kv_row + static_cast<long>(h) * c.D;
      float s = 0.f;
      for (int d = lane; d < c.D; d += kWave) s += elt<DT>(p.kn, at + d) * sq[d];
      s = wave_sum_f32(s);
      const float mn = fmaxf(m, s);
      if (mn == -INFINITY) continue;
      const float r = ex2(m - mn), e = ex2(s - mn);
      m = mn;
      l = l * r + e;
      for (int i = 0, d = lane; d < c.D; ++i, d += kWave) o[i] = o[i] * r + e * elt<DT>(p.vn, at + d);
    }
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  for (int i = 0, d = lane; d < c.D; ++i, d += kWave) {
    const float y = o[i] * inv;
    if constexpr (DT == SPECV_F32) static_cast<float*>(p.out)[orow * c.D + d] = y;
    else static_cast<__bf16*>(p.out)[orow * c.D + d] = static_cast<__bf16>(y);
  }
  if (p.lse && lane == 0)
    p.lse[orow] = l == 0.f ? -INFINITY : static_cast<float>(0.693147180559945 * (m + static_cast<double>(__builtin_amdgcn_logf(l))));
}

}  // namespace

hipError_t launch_kv_attention(const KvAttn& p, int dtype, int fmt, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(p.N) * p.Hq, static_cast<unsigned>(p.B)), block(kWave);
  if (dtype == SPECV_F32) {
    if (fmt == SPECV_E4M3) hipLaunchKernelGGL((k_kv_attn<SPECV_F32, SPECV_E4M3>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((k_kv_attn<SPECV_F32, SPECV_I8>), grid, block, 0, st, p);
  } else {
    if (fmt == SPECV_E4M3) hipLaunchKernelGGL((k_kv_attn<SPECV_BF16, SPECV_E4M3>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((k_kv_attn<SPECV_BF16, SPECV_I8>), grid, block, 0, st, p);
  }
  return hipGetLastError();
}

}  // namespace sv
