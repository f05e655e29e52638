// Cache attention: the launch, and the join of a sequence's parts.
#include "sv_device.h"
#include "sv_kv.h"

namespace sv {

namespace {

// D / 4 threads per output row: the parts' sums, each scaled to the largest
// maximum, in the parts' order.  Rows of sequences in one part are already
// written.
template <int DT>
__global__ __launch_bounds__(kBlock) void k_kv_join(KvAttn p) {
  const int tpr = p.c.D / 4, rows_per = kBlock / tpr;
  const int sub = threadIdx.x / tpr, d = threadIdx.x % tpr * 4;
  const long row = static_cast<long>(blockIdx.x) * rows_per + sub;
  if (sub >= rows_per || row >= static_cast<long>(p.B) * p.N * p.Hq) return;
  const long b = row / (static_cast<long>(p.N) * p.Hq);
  const int len = kv_len(p.c, p.lengths, b);
  const int parts = kv_parts((len >> 6) + ((len & 63) != 0), p.granule);
  if (parts == 1) return;
  const int n = static_cast<int>(row / p.Hq % p.N);
  const bool exists = n < (p.nodes ? min(max(p.nodes[b], 0), p.N) : p.N);
  const long at = row * p.splits;
  float top = -INFINITY;
  for (int i = 0; i < parts; ++i) top = fmaxf(top, p.part_ml[at + i].x);
  float y[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f;
  for (int i = 0; i < parts; ++i) {
    const float2 ml = p.part_ml[at + i];
    const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
    const float4 v = *reinterpret_cast<const float4*>(p.part_o + (at + i) * p.c.D + d);
    y[0] += v.x * f;
    y[1] += v.y * f;
    y[2] += v.z * f;
    y[3] += v.w * f;
    l += ml.x == -INFINITY ? ml.y : ml.y * f;  // 0, or NaN of a part that saw only NaN
  }
  kv_finish<DT>(p, row, d, y, top, l, exists);
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
  const long rows = static_cast<long>(p.B) * p.N * p.Hq, per = kBlock / (p.c.D / 4);
  const dim3 grid(static_cast<unsigned>((rows + per - 1) / per)), block(kBlock);
  if (dtype == SPECV_F32) hipLaunchKernelGGL(k_kv_join<SPECV_F32>, grid, block, 0, st, p);
  else hipLaunchKernelGGL(k_kv_join<SPECV_BF16>, grid, block, 0, st, p);
  return hipGetLastError();
}

}  // namespace sv
