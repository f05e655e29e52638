// The 8-bit paged cache: appending tokens (quantised as they are written) and
// reading a range back.
//
// A page holds P tokens of every head; the block of one page and one head has
// one scale s, a power of two, for K and one for V.  A value x is kept as
// code = rnd(clamp(x / s)) and stands for code * s.  Because s is a power of
// two, x / s, code * s and the ratio of two scales are exact: the only
// rounding is the format's own, and any order of the same calls gives the
// same bits.  Appending to a block begun by an earlier call may need a larger
// scale: then its codes are rounded again to the grown scale (exact in e4m3,
// but for codes that become subnormal).
//
// K pages are [P][D], V pages are [D][P]: the attention's second product
// reads V along the tokens.
#include "sv_device.h"
#include "sv_kv.h"

namespace sv {

namespace {

// Four elements of a row, at element i (a multiple of 4).
template <int DT>
__device__ inline void load4(const void* row, long i, float* f) {
  if constexpr (DT == SPECV_F32) {
    const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(row) + i);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(row) + i);
    f[0] = __uint_as_float(v.x << 16); f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16); f[3] = __uint_as_float(v.y & 0xffff0000u);
  }
}

__device__ inline int block_min_i32(int v, int* lds /* >= kWaves */) {
  v = wave_min_i32(v);
  __syncthreads();
  if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = v;
  __syncthreads();
  int t = lds[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) t = min(t, lds[i]);
  return t;
}

// One workgroup per (page the call may touch, K or V of a head, sequence).
template <int DT, int FMT>
__global__ __launch_bounds__(kBlock) void k_kv_append(KvAppend p) {
  const KvView& c = p.c;
  const int slot = blockIdx.x, h = blockIdx.y >> 1, isv = blockIdx.y & 1;
  const long b = blockIdx.z;
  const int tid = threadIdx.x;
  __shared__ float ldsf[kWaves];
  __shared__ int ldsi[kWaves];

  const int len = kv_len(c, p.lengths, b);
  const int room = (c.width << c.pshift) - len;
  int n = min(p.counts ? min(max(p.counts[b], 0), p.N) : p.N, room);
  // the tokens end at the first index outside [0, N), and at the first page
  // the table does not have; every page before this workgroup's counts (and
  // every page, where the new length is written)
  const bool reports = slot == 0 && blockIdx.y == 0 && p.out_lengths;
  const int col0 = len >> c.pshift;
  int stop = n;
  if (p.index)
    for (int i = tid; i < n; i += kBlock) {
      const int ix = p.index[b * p.N + i];
      if (ix < 0 || ix >= p.N) stop = min(stop, i);
    }
  if (n > 0) {
    const int end = (len + n - 1) >> c.pshift;
    const int last = reports || slot > end - col0 ? end : col0 + slot;
    for (int col = col0 + tid; col <= last; col += kBlock)
      if (kv_page(c, b, col) < 0) stop = min(stop, max((col << c.pshift) - len, 0));
  }
  n = block_min_i32(stop, ldsi);
  if (reports && tid == 0) p.out_lengths[b] = len + n;

  const long p0 = (static_cast<long>(col0) + slot) << c.pshift;               // the page's first position
  const int t0 = static_cast<int>(max(len - p0, 0L));                         // tokens of it cached before
  const int t1 = static_cast<int>(min(len + n - p0, static_cast<long>(c.P)));  // and after
  if (t1 <= t0) return;
  const int id = kv_page(c, b, p0 >> c.pshift);      // a page: n ends before the first that is not
  const long blk = static_cast<long>(id) * c.H + h;
  float* sp = (isv ? c.vs : c.ks) + blk;
  const float s_old = *sp;
  const void* src = isv ? p.v : p.k;
  constexpr int eb = DT == SPECV_F32 ? 4 : 2;
  auto row = [&](int t) -> const void* {  // token t of the page
    const long i = p0 + t - len;
    const long r = b * p.N + (p.index ? p.index[b * p.N + i] : i);
    return static_cast<const char*>(src) + (r * p.row + static_cast<long>(h) * c.D) * eb;
  };
  const int nv = c.D / 4, work = (t1 - t0) * nv;
  float amax = 0.f;
  for (int i = tid; i < work; i += kBlock) {
    float f[4];
    load4<DT>(row(t0 + i / nv), (i % nv) * 4, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) amax = fmaxf(amax, isfinite(f[j]) ? fabsf(f[j]) : 0.f);
  }
  amax = block_max(amax, ldsf);
  float s = kv_scale<FMT>(amax);
  if (t0 > 0) s = fmaxf(s, s_old);
  const float inv = 1.f / s;
  uint8_t* page = (isv ? c.vp : c.kp) + blk * c.P * c.D;
  for (int i = tid; i < work; i += kBlock) {
    const int t = t0 + i / nv, d = (i % nv) * 4;
    float f[4];
    load4<DT>(row(t), d, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] *= inv;
    const uint32_t w = kv_encode4<FMT>(f);
    if (!isv) {
      *reinterpret_cast<uint32_t*>(page + static_cast<long>(t) * c.D + d) = w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) page[static_cast<long>(d + j) * c.P + t] = static_cast<uint8_t>(w >> (8 * j));
    }
  }
  if (t0 > 0 && s > s_old) {  // the tokens that were there, to the grown scale
    const float ratio = s_old * inv;
    for (int i = tid; i < t0 * c.D; i += kBlock) {
      const long at = isv ? static_cast<long>(i / t0) * c.P + i % t0 : i;
      float f[4];
      kv_decode4<FMT>(page[at], f);
      f[0] *= ratio;
      f[1] = f[2] = f[3] = 0.f;
      page[at] = static_cast<uint8_t>(kv_encode4<FMT>(f));
    }
  }
  if (tid == 0) *sp = s;
}

// One workgroup per (page the range may touch, K or V of a head, sequence).
template <int DT, int FMT>
__global__ __launch_bounds__(kBlock) void k_kv_read(KvRead p) {
  const KvView& c = p.c;
  const int slot = blockIdx.x, h = blockIdx.y >> 1, isv = blockIdx.y & 1;
  const long b = blockIdx.z;
  void* out = isv ? p.out_v : p.out_k;
  if (!out) return;
  const int len = kv_len(c, p.lengths, b);
  const long start = p.starts ? max(p.starts[b], 0) : 0;
  const long p0 = ((start >> c.pshift) + slot) << c.pshift;
  const long a = max(start, p0), z = min(start + p.T, p0 + c.P);  // positions this workgroup writes
  if (z <= a) return;
  const int id = kv_page(c, b, p0 >> c.pshift);
  const long blk = static_cast<long>(max(id, 0)) * c.H + h;
  const float s = id >= 0 ? (isv ? c.vs : c.ks)[blk] : 0.f;
  const uint8_t* page = (isv ? c.vp : c.kp) + blk * c.P * c.D;
  const int nv = c.D / 4;
  const int work = static_cast<int>(z - a) * nv;
  for (int i = threadIdx.x; i < work; i += kBlock) {
    const long pos = a + i / nv;
    const int t = static_cast<int>(pos - p0), d = (i % nv) * 4;
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    if (id >= 0 && pos < len) {
      uint32_t w = 0;
      if (!isv) {
        w = *reinterpret_cast<const uint32_t*>(page + static_cast<long>(t) * c.D + d);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) w |= static_cast<uint32_t>(page[static_cast<long>(d + j) * c.P + t]) << (8 * j);
      }
      kv_decode4<FMT>(w, f);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] *= s;
    }
    kv_store4<DT>(out, ((b * p.T + (pos - start)) * c.H + h) * c.D + d, f);
  }
}

}  // namespace

// Pages that n consecutive tokens can touch, whatever position they start at.
static unsigned kv_slots(long n, int P) { return static_cast<unsigned>((n + P - 2) / P + 1); }

hipError_t launch_kv_append(const KvAppend& p, int dtype, int fmt, hipStream_t st) {
  const dim3 grid(kv_slots(p.N, p.c.P), static_cast<unsigned>(2 * p.c.H), static_cast<unsigned>(p.B)), block(kBlock);
  if (dtype == SPECV_F32) {
    if (fmt == SPECV_E4M3) hipLaunchKernelGGL((k_kv_append<SPECV_F32, SPECV_E4M3>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((k_kv_append<SPECV_F32, SPECV_I8>), grid, block, 0, st, p);
  } else {
    if (fmt == SPECV_E4M3) hipLaunchKernelGGL((k_kv_append<SPECV_BF16, SPECV_E4M3>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((k_kv_append<SPECV_BF16, SPECV_I8>), grid, block, 0, st, p);
  }
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvRead& p, int dtype, int fmt, hipStream_t st) {
  const dim3 grid(kv_slots(p.T, p.c.P), static_cast<unsigned>(2 * p.c.H), static_cast<unsigned>(p.B)), block(kBlock);
  if (dtype == SPECV_F32) {
    if (fmt == SPECV_E4M3) hipLaunchKernelGGL((k_kv_read<SPECV_F32, SPECV_E4M3>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((k_kv_read<SPECV_F32, SPECV_I8>), grid, block, 0, st, p);
  } else {
    if (fmt == SPECV_E4M3) hipLaunchKernelGGL((k_kv_read<SPECV_BF16, SPECV_E4M3>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((k_kv_read<SPECV_BF16, SPECV_I8>), grid, block, 0, st, p);
  }
  return hipGetLastError();
}

}  // namespace sv
