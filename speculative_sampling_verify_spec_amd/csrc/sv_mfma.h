// Operand fragments of the bf16 matrix instructions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "specverify.h"

namespace sv {

namespace frag {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.44269504088896f;

// Number of bf16 pieces of an element: 32 bits are the sum of three.
template <int DT>
constexpr int kPieces = DT == SPECV_F32 ? 3 : 1;

// x as a sum of NP bf16 pieces.  One piece: round to nearest.  Three: the
// leading 8 bits, the next 8 and the last 8 of the 24, an exact sum (by
// truncation, so that the largest floats stay finite); x that is not finite
// is its own first piece.
template <int NP>
__device__ inline void split(float x, __bf16* piece) {
  if constexpr (NP == 1) {
    piece[0] = static_cast<__bf16>(x);
  } else {
    auto lead = [](float f) { return __uint_as_float(__float_as_uint(f) & 0xffff0000u); };
    auto bits = [](float f) { return __builtin_bit_cast(__bf16, static_cast<uint16_t>(__float_as_uint(f) >> 16)); };
    piece[0] = bits(x);
    const float r = isfinite(x) ? x - lead(x) : 0.f;
    piece[1] = bits(r);
    piece[2] = bits(r - lead(r));
  }
}

// Two values' pieces into elements at, at + 1 of NP fragments.
template <int NP>
__device__ inline void split2(f32x2 x, bf16x8* f, int at) {
  if constexpr (NP == 1) {
    const bf16x2 y = __builtin_convertvector(x, bf16x2);
    f[0][at] = y[0];
    f[0][at + 1] = y[1];
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      __bf16 s[3];
      split<3>(x[k], s);
#pragma unroll
      for (int j = 0; j < 3; ++j) f[j][at + k] = s[j];
    }
  }
}

// Eight consecutive elements, as they are loaded: 16 bytes of bf16, 32 of fp32.
template <int DT>
struct Raw8 {
  uint4 w[DT == SPECV_F32 ? 2 : 1];
  __device__ void load(const void* base, long i) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + i * (DT == SPECV_F32 ? 4 : 2));
    w[0] = p[0];
    if constexpr (DT == SPECV_F32) w[1] = p[1];
  }
  __device__ void clear() {
    w[0] = make_uint4(0, 0, 0, 0);
    if constexpr (DT == SPECV_F32) w[1] = w[0];
  }
  __device__ void negate(bool yes) {
    const uint32_t signs = yes ? (DT == SPECV_F32 ? 0x80000000u : 0x80008000u) : 0u;
    uint32_t* u = reinterpret_cast<uint32_t*>(w);
#pragma unroll
    for (int i = 0; i < (DT == SPECV_F32 ? 8 : 4); ++i) u[i] ^= signs;
  }
  // Makes the compiler take the elements as new here, so that what is computed
  // from them is not kept across a loop.
  __device__ void hide() {
    uint32_t* u = reinterpret_cast<uint32_t*>(w);
#pragma unroll
    for (int i = 0; i < (DT == SPECV_F32 ? 8 : 4); ++i) asm volatile("" : "+v"(u[i]));
  }
  __device__ float at(int j) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
    if constexpr (DT == SPECV_F32) return __uint_as_float(u[j]);
    else return __uint_as_float(j % 2 ? u[j / 2] & 0xffff0000u : u[j / 2] << 16);
  }
  // Whether an element is infinite or NaN.
  __device__ bool wild() const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < (DT == SPECV_F32 ? 8 : 4); ++i) {
      if constexpr (DT == SPECV_F32) any |= ((u[i] & 0x7fffffffu) + 0x00800000u) & 0x80000000u;
      else any |= ((u[i] & 0x7fff7fffu) + 0x00800080u) & 0x80008000u;
    }
    return any != 0;
  }
  // 0 in place of what is infinite or NaN.
  __device__ void tame() {
    uint32_t* u = reinterpret_cast<uint32_t*>(w);
#pragma unroll
    for (int i = 0; i < (DT == SPECV_F32 ? 8 : 4); ++i) {
      if constexpr (DT == SPECV_F32) {
        if (!isfinite(__uint_as_float(u[i]))) u[i] = 0;
      } else {
        if ((u[i] & 0x7f80u) == 0x7f80u) u[i] &= 0xffff0000u;
        if ((u[i] & 0x7f800000u) == 0x7f800000u) u[i] &= 0xffffu;
      }
    }
  }
  __device__ void pieces(bf16x8* f) const {
    if constexpr (DT == SPECV_BF16) {
      f[0] = __builtin_bit_cast(bf16x8, w[0]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        __bf16 s[3];
        split<3>(at(j), s);
        f[0][j] = s[0];
        f[1][j] = s[1];
        f[2][j] = s[2];
      }
    }
  }
};

// Eight codes to bf16, exact.
template <int FMT>
__device__ inline bf16x8 codes8(uint32_t a, uint32_t b) {
  union { uint32_t w[4]; bf16x2 h[4]; bf16x8 v; } u;
  if constexpr (FMT == SPECV_E4M3) {
    u.h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, false);
    u.h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, true);
    u.h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, false);
    u.h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, true);
  } else {
    // integers up to 127 have at most 7 significant bits: their floats' upper halves are their bf16
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = i < 2 ? a : b;
      const int s = 16 * (i & 1);
      const uint32_t lo = __float_as_uint(static_cast<float>(static_cast<int8_t>(w >> s)));
      const uint32_t hi = __float_as_uint(static_cast<float>(static_cast<int8_t>(w >> (s + 8))));
      u.w[i] = __builtin_amdgcn_perm(hi, lo, 0x07060302);
    }
  }
  return u.v;
}

// D[16][16] += A[16][32] B[32][16].  A: lane l has row l % 16 and columns 8
// (l / 16) .. + 7; B: column l % 16 and rows 8 (l / 16) .. + 7; D: column l %
// 16, and register i row 4 (l / 16) + i.
__device__ inline f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// D[32][32] += A[32][16] B[16][32].  A: lane l has row l % 32 and columns 8
// (l / 32) .. + 7; B: column l % 32 and rows 8 (l / 32) .. + 7; D: column l %
// 32, and register i row 8 (i / 4) + 4 (l / 32) + i % 4.
__device__ inline f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// First channel of the 8 that lane group g holds of fragment f: fragments 2c
// and 2c + 1 are the halves of the 16 bytes a lane loads of 64 channels; a
// last odd fragment is an 8-byte load of 32.
template <int D>
__device__ inline int chan(int f, int g) {
  return f < D / 64 * 2 ? f / 2 * 64 + 16 * g + f % 2 * 8 : D / 64 * 64 + 8 * g;
}

// Maximum and sum over the four lanes that hold the same query (lane % 16).
__device__ inline float groups_max(float v) {
  const unsigned u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const unsigned w = __float_as_uint(v);
  const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ inline float groups_sum(float v) {
  const unsigned u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const unsigned w = __float_as_uint(v);
  const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Maximum and sum over the two lanes l and l + 32.
__device__ inline float halves_max(float v) {
  const unsigned u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ inline float halves_sum(float v) {
  const unsigned u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// Where the 16-byte piece c of row t stands in a row of D elements in LDS, so
// that sixteen rows' same piece, and four rows' same four pieces (a transposing
// read), fall into different banks.
template <int D>
__device__ inline int swizzle(int t, int c) {
  if constexpr (D == 96) return c ^ ((t >> 2) & 3);  // rows begin in four different places of the banks
  else if constexpr (D == 64) return c ^ (4 * ((t >> 1) & 1) + 2 * ((t >> 2) & 1) + ((t >> 3) & 1));  // two rows a round of banks
  else return c ^ (4 * (t & 3) + 2 * ((t >> 2) & 1) + ((t >> 3) & 1));
}

// Eight k of one column for an A operand, from rows of LDS: the 16 lanes of a
// group give the addresses of 4 rows x 16 columns (lane j row j / 4, columns 4
// (j % 4) .. + 3) twice, and lane j gets column j of both.
template <class P>
__device__ inline bf16x8 read_transposed(P lo, P hi) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4* lds_ptr;
  const s16x4 u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(lo));
  const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(hi));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Where an array of shared memory begins in LDS.
template <class T>
__device__ inline uint32_t lds_address(T* shared) {
  typedef __attribute__((address_space(3))) T* lds_ptr;
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_ptr)shared));
}

// 16 bytes a lane from memory (the wave's `base`, `offset` bytes further)
// straight to LDS: the wave's 1024 bytes from address `to` on.  The load takes
// that address from M0, a wait state after it was written; the compiler, which
// else sees to that, does not look into the string.
__device__ inline void load_lds(const void* base, uint32_t offset, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(__builtin_amdgcn_readfirstlane(to)), "v"(offset),
               "s"(base)
               : "memory", "m0");
}

// A barrier that orders LDS only: __syncthreads would also wait for every
// global load in flight, the next tile's among them.
__device__ inline void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// A barrier after which what load_lds requested before it is in LDS, but for the
// kLeft youngest requests.  The wait is one that the compiler knows of (vmcnt,
// and lgkmcnt 0): it would else wait for its own loads from before again, and so
// for the next tile's requests, wherever their results are used.
template <int kLeft = 0>
__device__ inline void landed_barrier() {
  static_assert(kLeft < 64, "6 bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (kLeft & 15) | (kLeft >> 4) << 14);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace frag

}  // namespace sv
