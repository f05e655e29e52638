// Whole prompts, packed: parameters shared by their host code and kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "specverify.h"

namespace sv {

// Token rows of B packed sequences.
struct Packed {
  const void* q;          // [T] rows of Hq*D elements, q_row elements apart
  const void* k;          // [T] rows of H*D elements, kv_row elements apart
  const void* v;          // as k, or null
  long q_row, kv_row;
  const int32_t* starts;  // [B + 1]
  float scale;
  int B, T, H, Hq, G;     // G = Hq / H query heads share a key head
};

struct PromptAttn {
  Packed s;
  void* out;              // [T][Hq][D]
  float* lse;             // [T][Hq] or null
  unsigned slots;         // places for blocks of kPromptRows rows of a head (prompt_slots)
};

struct PromptWeights {
  Packed s;               // no v
  const float* lse;       // [T][Hq]
  float* w;               // [B][H][capacity]
  int capacity;
  unsigned slots;         // places for blocks of kWeightKeys tokens of a head
  uint32_t magic;         // r / G is mulhi(r, magic) >> shift for r < 2^31 (G > 1)
  int shift;
};

constexpr int kWeightKeys = 128;  // tokens of one workgroup, as keys
constexpr int kPromptRows = 128;  // rows (a token's query head each) of one workgroup

// Places for the blocks of all sequences of one head, whatever their lengths:
// the sum over sequences of ceil(rows / size) is below rows / size + B, so at
// least one place stays free (whose workgroup clears what no sequence holds).
inline long prompt_slots(long T, int per_token, int B, int size) { return (T * per_token + size - 1) / size + B; }

hipError_t launch_prompt_64(const PromptAttn& p, int dtype, hipStream_t s);
hipError_t launch_prompt_96(const PromptAttn& p, int dtype, hipStream_t s);
hipError_t launch_prompt_128(const PromptAttn& p, int dtype, hipStream_t s);
hipError_t launch_prompt_256(const PromptAttn& p, int dtype, hipStream_t s);
hipError_t launch_prompt_weights_64(const PromptWeights& p, int dtype, hipStream_t s);
hipError_t launch_prompt_weights_96(const PromptWeights& p, int dtype, hipStream_t s);
hipError_t launch_prompt_weights_128(const PromptWeights& p, int dtype, hipStream_t s);
hipError_t launch_prompt_weights_256(const PromptWeights& p, int dtype, hipStream_t s);

#ifdef __HIPCC__

// A block of a sequence's rows: the sequence's token range and the block's number.
struct PromptBlock {
  int first, last;  // the sequence's tokens first .. last-1
  int seq;          // the sequence
  int block;        // -1: none
  int used;         // blocks of all sequences (valid when block < 0)
};

// Sequence b's tokens, whatever starts holds.
__device__ inline void prompt_range(const Packed& s, int b, int& first, int& last) {
  first = min(max(s.starts[b], 0), s.T);
  last = min(max(s.starts[b + 1], first), s.T);
}

// The block in a place: sequences in order, a sequence's blocks (of `size`
// rows, per_token rows a token) from the last to the first, whose rows see
// most.  Every thread of a workgroup of THREADS calls it.
template <int THREADS>
__device__ inline PromptBlock prompt_block(const Packed& s, unsigned place, int per_token, int size) {
  __shared__ long wave_sum[THREADS / 64 + 1];
  __shared__ int found[4];
  PromptBlock r;
  r.block = -1;
  r.used = 0;
  const int lane = threadIdx.x % 64, w = threadIdx.x / 64;
  long before = 0;
  for (int b0 = 0; b0 < s.B; b0 += THREADS) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    int first = 0, last = 0;
    if (b < s.B) prompt_range(s, b, first, last);
    const long n = (static_cast<long>(last - first) * per_token + size - 1) / size;
    long sum = n;  // blocks up to and with this thread's sequence
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const long x = __shfl_up(sum, d, 64);
      if (lane >= d) sum += x;
    }
    if (lane == 63) wave_sum[w] = sum;
    if (threadIdx.x == 0) found[2] = -1;
    __syncthreads();
    for (int i = 0; i < w; ++i) sum += wave_sum[i];
    sum += before;
    if (static_cast<long>(place) >= sum - n && static_cast<long>(place) < sum) {
      found[0] = first;
      found[1] = last;
      found[2] = static_cast<int>(sum - 1 - place);
      found[3] = b;
    }
    long total = 0;
    for (int i = 0; i < THREADS / 64; ++i) total += wave_sum[i];
    before += total;
    __syncthreads();
    if (found[2] >= 0) {
      r.first = found[0];
      r.last = found[1];
      r.block = found[2];
      r.seq = found[3];
      return r;
    }
    __syncthreads();
  }
  r.used = static_cast<int>(min(before, static_cast<long>(INT32_MAX)));
  return r;
}

#endif  // __HIPCC__

}  // namespace sv
