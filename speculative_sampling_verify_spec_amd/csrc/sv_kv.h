// The 8-bit paged cache: parameters shared by its host code and kernels, and
// the device helpers for its formats.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "specverify.h"

namespace sv {

// The cache as the kernels see it (see specv_kv_t).
struct KvView {
  uint8_t* kp;           // K pages [pages][H][P][D]
  uint8_t* vp;           // V pages [pages][H][D][P]
  float* ks;             // scales [pages][H]
  float* vs;
  const int32_t* table;  // [B][width] page ids
  int pages, width;
  int P, pshift;         // tokens per page, log2
  int H, D;
};

struct KvAppend {
  KvView c;
  const void* k;         // [B][N] token rows of H*D elements, row elements apart
  const void* v;
  long row;
  const int32_t* lengths;
  const int32_t* counts;  // or null
  const int32_t* index;   // or null
  int B, N;
  int32_t* out_lengths;   // or null
  unsigned groups;        // workgroups that share a head's pages (kv_append_groups)
};

struct KvRead {
  KvView c;
  const int32_t* starts;  // or null
  const int32_t* lengths;
  int B, T;
  void* out_k;            // [B][T][H][D], or null
  void* out_v;
  int chunks;             // workgroups that share a page (the launcher sets it)
};

struct KvAttn {
  KvView c;
  const void* q;          // [B][N] rows of Hq*D elements, q_row elements apart
  const void* kn;         // [B][N] rows of H*D elements, kv_row elements apart, or null
  const void* vn;
  long q_row, kv_row;
  const int32_t* lengths;
  const int32_t* nodes;   // or null
  const int32_t* parents; // or null: a chain
  float scale;
  int B, N, Hq, G;        // G = Hq / H query heads share a cached head
  float inv_g;            // 1 / G
  void* out;              // [B][N][Hq][D]
  float* lse;             // [B][N][Hq] or null
  // plan (kv_plan) and workspace
  int mt, mb;             // blocks of 16 queries per workgroup, workgroups per (sequence, head, part)
  int granule, splits;    // a part has at most `granule` tiles; no sequence has more than `splits` parts
  float* part_o;          // [B][N][Hq][splits][D] sums of weight * value
  float2* part_ml;        // [B][N][Hq][splits] (maximum, sum of weights), scores in log2
};

// Largest number of 16-query blocks a workgroup's registers hold at two waves
// a SIMD (32-bit, D = 256: one).  A fourth block at D = 128 leaves one wave:
// 128 trees of 32 nodes (128 queries a cached head) took 395 us so, against 267
// in workgroups of 48, though those read the cache three times and not twice.
constexpr int kv_max_mt(int dtype, int D) {
  if (D == 256) return 1;
  return dtype == SPECV_F32 ? 2 : D == 64 ? 4 : 3;
}

// Parts of a sequence of `ntile` tiles.
__host__ __device__ inline int kv_parts(int ntile, int granule) {
  return ntile <= granule ? 1 : (ntile + granule - 1) / granule;
}

// Pages that n consecutive tokens can touch, whatever position they start at.
inline unsigned kv_slots(long n, int P) { return static_cast<unsigned>((n + P - 2) / P + 1); }

// Workgroups of one head of one sequence in an append.  Each looks through
// the call's pages and indexes up to its own last one, so their number bounds
// the entries looked at for a token (131072 tokens of 8 heads of 64 in pages of
// 16: 130 us, with a workgroup for each of the 8193 pages 186; by index, every
// workgroup to the end of it, 362 and 1458).  A few tokens rarely cross into a
// second page: one workgroup takes both (256 x 6 tokens by four waves: 13.9 us,
// with one per page 21.6).
constexpr unsigned kMaxAppendGroups = 1024;
inline unsigned kv_append_groups(int N, int P) {
  const unsigned slots = kv_slots(N, P);
  return slots <= 2 ? 1 : slots < kMaxAppendGroups ? slots : kMaxAppendGroups;
}

// Launchers, next to their kernels.  dtype: SPECV_F32 or SPECV_BF16; fmt:
// SPECV_E4M3 or SPECV_I8.
hipError_t launch_kv_append(const KvAppend& p, int dtype, int fmt, hipStream_t s);
hipError_t launch_kv_read(const KvRead& p, int dtype, int fmt, hipStream_t s);
hipError_t launch_kv_attention(const KvAttn& p, int dtype, int fmt, hipStream_t s);
hipError_t launch_kv_attn_64(const KvAttn& p, int dtype, int fmt, hipStream_t s);
hipError_t launch_kv_attn_96(const KvAttn& p, int dtype, int fmt, hipStream_t s);
hipError_t launch_kv_attn_128(const KvAttn& p, int dtype, int fmt, hipStream_t s);
hipError_t launch_kv_attn_256(const KvAttn& p, int dtype, int fmt, hipStream_t s);

#ifdef __HIPCC__

constexpr float kE4m3Max = 448.f;  // largest e4m3 value: 0.875 * 2^9
constexpr float kI8Max = 127.f;    // largest int8 code used (symmetric): 0.9921875 * 2^7

// Largest finite value of an element type.
template <int DT>
constexpr float kLargest = DT == SPECV_F32 ? 0x1.fffffep127f : 0x1.fep127f;

// Four codes of a word to float; exact for both formats.
template <int FMT>
__device__ inline void kv_decode4(uint32_t w, float* f) {
  if constexpr (FMT == SPECV_E4M3) {
    f[0] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(w), 0);
    f[1] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(w), 1);
    f[2] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(w), 2);
    f[3] = __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(w), 3);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
  }
}

// Four values, in units of the scale, to codes: round to nearest, ties to
// even (the formats' own 8-bit rounding: the cache's one deliberate loss).
// Infinite values saturate; NaN stays NaN in e4m3 and becomes 0 in int8.
template <int FMT>
__device__ inline uint32_t kv_encode4(const float* x) {
  constexpr float top = FMT == SPECV_E4M3 ? kE4m3Max : kI8Max;
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float c = fminf(fmaxf(x[i], -top), top);
    y[i] = x[i] == x[i] ? c : (FMT == SPECV_E4M3 ? x[i] : 0.f);
  }
  if constexpr (FMT == SPECV_E4M3) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true));
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= (static_cast<uint32_t>(static_cast<int>(rintf(y[i]))) & 0xffu) << (8 * i);
    return w;
  }
}

// As kv_encode4 for values known to be finite and in the format's range.  int8:
// adding 1.5 * 2^23 leaves the value, rounded to the nearest integer (ties to
// even), in the low byte.
template <int FMT>
__device__ inline uint32_t kv_encode4_finite(const float* x) {
  if constexpr (FMT == SPECV_E4M3) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], w, true));
  } else {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(x[i] + 12582912.f);
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400), __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400),
                                 0x05040100);
  }
}

// Running maximum of the finite magnitudes of 16-byte vectors, on their bits:
// magnitudes order like integers, and adding the smallest exponent step makes
// infinities and NaN negative.
template <int DT> struct MaxBits;
template <> struct MaxBits<SPECV_F32> {
  int m = 0x00800000, any = 0;
  __device__ void add(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = static_cast<int>((w[i] & 0x7fffffffu) + 0x00800000u);
      any |= t;
      m = max(m, t);
    }
  }
  __device__ float value() const { return __int_as_float(m - 0x00800000); }
  __device__ bool wild() const { return any < 0; }  // an infinity or a NaN was among them
};
template <> struct MaxBits<SPECV_BF16> {
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  s16x2 m = {0x0080, 0x0080};
  uint32_t any = 0;
  __device__ void add(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const s16x2 t = __builtin_bit_cast(s16x2, w[i] & 0x7fff7fffu) + s16x2{0x0080, 0x0080};
      any |= __builtin_bit_cast(uint32_t, t);
      m = __builtin_elementwise_max(m, t);
    }
  }
  __device__ float value() const {
    const int top = max(static_cast<int>(m.x), static_cast<int>(m.y)) - 0x0080;
    return __int_as_float(top << 16);
  }
  __device__ bool wild() const { return (any & 0x80008000u) != 0; }
};

// Four codes to the codes of ratio times their values.
template <int FMT>
__device__ inline uint32_t kv_rescale4(uint32_t w, float ratio) {
  float f[4];
  kv_decode4<FMT>(w, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] *= ratio;
  return kv_encode4<FMT>(f);
}

// The smallest power of two s with amax <= top * s, at least 2^-126 (the
// smallest normal number, also for amax = 0).  amax is finite, so s <= 2^120
// (e4m3) or 2^122 (int8), and the code of a value past 248 or 63.5 times that
// stands for 2^128, which spec_kv_read gives as the largest finite value.
template <int FMT>
__device__ inline float kv_scale(float amax) {
  constexpr int bits = FMT == SPECV_E4M3 ? 9 : 7;
  constexpr float top = FMT == SPECV_E4M3 ? 0.875f : 0.9921875f;
  int e;
  const float m = frexpf(amax, &e);  // amax = m 2^e, m in [1/2, 1)
  int k = e - bits + (m > top ? 1 : 0);
  if (!(amax > 0.f) || k < -126) k = -126;
  return __int_as_float((k + 127) << 23);
}

// The page id in the table's column c of sequence b, or -1 when there is no
// such column or its id names no page.
__device__ inline int kv_page(const KvView& c, long b, long col) {
  if (col >= c.width) return -1;
  const int id = c.table[b * c.width + col];
  return id >= 0 && id < c.pages ? id : -1;
}

// Cached tokens of sequence b: its length, clamped to what the table holds.
__device__ inline int kv_len(const KvView& c, const int32_t* lengths, long b) {
  return min(max(lengths[b], 0), c.width << c.pshift);
}

// Four elements to a row; bf16 by round to nearest even (the type's own
// rounding; what a cache holds under power-of-two scales is exact in bf16).
template <int DT>
__device__ inline void kv_store4(void* base, long i, const float* f) {
  if constexpr (DT == SPECV_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(base) + i) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    bf16x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = static_cast<__bf16>(f[j]);
    *reinterpret_cast<bf16x4*>(static_cast<uint16_t*>(base) + i) = v;
  }
}

// A row's 16 bytes, as kv_store4.
template <int DT>
__device__ inline void kv_store16(void* base, long i, const float* f) {
  if constexpr (DT == SPECV_F32) {
    kv_store4<DT>(base, i, f);
  } else {
    typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
    bf16x8 v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = static_cast<__bf16>(f[j]);
    *reinterpret_cast<bf16x8*>(static_cast<uint16_t*>(base) + i) = v;
  }
}

// ln of a row's sum of weights from its statistics (scores in log2).
__device__ inline float kv_lse(float m, float l, bool some) {
  return some ? static_cast<float>(0.6931471805599453 * (static_cast<double>(m) + __builtin_amdgcn_logf(l))) : -INFINITY;
}

#endif  // __HIPCC__

}  // namespace sv
