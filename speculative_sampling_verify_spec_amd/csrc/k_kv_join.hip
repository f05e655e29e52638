// Cache attention: the launch, and the join of a sequence's parts.
#include "sv_device.h"
#include "sv_kv.h"

namespace sv {

namespace {

// An output row's parts, each scaled to the largest maximum, summed by GR
// groups of D / 4 threads: group i takes parts i, i + GR, ...; the groups'
// sums meet in LDS in their order, so the same call gives the same bits.
// WIDE: a workgroup per row, GR = 1024 / D; else GR = 1 and several rows per
// workgroup, for few parts.  Rows of sequences in one part are already written.
// Bound by the latency of length, maxima and sums in turn, all from the caches
// the attention just wrote: 640 rows of up to 121 parts take 6 us.
template <int DT, bool WIDE>
__global__ __launch_bounds__(kBlock) void k_kv_join(KvAttn p) {
  __shared__ float4 sy[kBlock];
  __shared__ float sl[kBlock];
  const int tpr = p.c.D / 4, groups = kBlock / tpr;  // 16, 10, 8 or 4
  const int grp = threadIdx.x / tpr, d = threadIdx.x % tpr * 4;
  const long row = WIDE ? blockIdx.x : static_cast<long>(blockIdx.x) * groups + grp;
  if (grp >= groups && !WIDE) return;
  if (row >= static_cast<long>(p.B) * p.N * p.Hq) return;
  const long b = row / (static_cast<long>(p.N) * p.Hq);
  const int len = kv_len(p.c, p.lengths, b);
  const int parts = kv_parts((len >> 6) + ((len & 63) != 0), p.granule);
  if (parts == 1) return;
  const int n = static_cast<int>(row / p.Hq % p.N);
  const bool exists = n < (p.nodes ? min(max(p.nodes[b], 0), p.N) : p.N);
  const long at = row * p.splits;
  const int first = WIDE ? grp : 0, step = WIDE ? groups : 1;
  float top = -INFINITY;
  if (WIDE) {
    for (int i = threadIdx.x % kWave; i < parts; i += kWave) top = fmaxf(top, p.part_ml[at + i].x);
    top = wave_max(top);
  } else {
    for (int i = 0; i < parts; ++i) top = fmaxf(top, p.part_ml[at + i].x);
  }
  float y[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f;
  if (grp < groups)
#pragma unroll 4
    for (int i = first; i < parts; i += step) {
      const float2 ml = p.part_ml[at + i];
      const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
      const float4 v = *reinterpret_cast<const float4*>(p.part_o + (at + i) * p.c.D + d);
      y[0] += v.x * f;
      y[1] += v.y * f;
      y[2] += v.z * f;
      y[3] += v.w * f;
      l += ml.x == -INFINITY ? ml.y : ml.y * f;  // 0, or NaN of a part that saw only NaN
    }
  if (WIDE) {
    sy[threadIdx.x] = make_float4(y[0], y[1], y[2], y[3]);
    sl[threadIdx.x] = l;
    __syncthreads();
    if (grp > 0) return;
    for (int i = 1; i < groups; ++i) {
      const float4 v = sy[threadIdx.x + i * tpr];
      y[0] += v.x;
      y[1] += v.y;
      y[2] += v.z;
      y[3] += v.w;
      l += sl[threadIdx.x + i * tpr];
    }
  }
  const bool some = exists && !(l == 0.f);  // a query that exists and sees something
  const float inv = 1.f / l;
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] = some ? y[j] * inv : 0.f;
  kv_store4<DT>(p.out, row * p.c.D + d, y);
  if (d == 0 && p.lse) p.lse[row] = kv_lse(top, l, some);
}

// More parts than this: a workgroup per row.  A whole call of 2 x 5 positions
// (G = 4, D = 128) over 20000 tokens, 20 parts, takes 29.1 us wide and 31.4
// with a row's parts in series (121 parts: the join alone 6 us and 74); 8 x 5 over
// 8000, 8 parts, 33.7 either way; 16 x 5 over 8000, 4 parts, 54.0 and 52.1.
constexpr int kWideParts = 8;

template <int DT>
hipError_t launch_join(const KvAttn& p, hipStream_t st) {
  const long rows = static_cast<long>(p.B) * p.N * p.Hq, per = kBlock / (p.c.D / 4);
  if (p.splits > kWideParts)
    hipLaunchKernelGGL((k_kv_join<DT, true>), dim3(static_cast<unsigned>(rows)), dim3(kBlock), 0, st, p);
  else
    hipLaunchKernelGGL((k_kv_join<DT, false>), dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(kBlock), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_attention(const KvAttn& p, int dtype, int fmt, hipStream_t st) {
  hipError_t rc = hipErrorInvalidValue;
  switch (p.c.D) {
    case 64: rc = launch_kv_attn_64(p, dtype, fmt, st); break;
    case 96: rc = launch_kv_attn_96(p, dtype, fmt, st); break;
    case 128: rc = launch_kv_attn_128(p, dtype, fmt, st); break;
    case 256: rc = launch_kv_attn_256(p, dtype, fmt, st); break;
  }
  if (rc != hipSuccess || p.splits == 1) return rc;
  return dtype == SPECV_F32 ? launch_join<SPECV_F32>(p, st) : launch_join<SPECV_BF16>(p, st);
}

}  // namespace sv
