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
  uint32_t magic;         // r / G is mulhi(r, magic) >> shift for r < 2^31 (G > 1)
  int shift;
#ifdef __HIPCC__
  __device__ int token_of(int r) const {
    return G == 1 ? r : static_cast<int>(__umulhi(static_cast<uint32_t>(r), magic) >> shift);
  }
#endif
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

// Lanes' sum up to and with each lane, for a whole wave: rows of 16 lanes, then
// + the rows' totals.
__device__ inline int lanes_sum_upto(int v) {
  int x = v;
  x += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, v, 0x113, 0xf, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xe, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xc, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, true);
  return x;
}

// The block in a place, for up to 64 sequences: a lane has a sequence, and
// every wave finds the block for itself.  A sequence's blocks begin with the
// last one, whose rows see most (with FROM_START with the first, which most
// rows see).  Where the chip has work for several turns (places from kInOrder
// on), sequences come one after the other, so that blocks that read the same
// keys do so together; else the highest blocks of all sequences come first,
// so that no long one begins late.  In order and highest first (us, places):
// attention of 48 prompts of 25 to 1405 tokens 411 and 448 (9648), of 16 of up to
// 4000 890 and 920 (9424), of 64 of up to 300 54 and 64 (2976), of 16 of up to 1500 143
// and 146 (3280), of 6 with heads of 256 71 and 66 (618); weights of 64 prompts of up to
// 2000 with a head of their own 165 and 168 (5048), of 32 of up to 1500 60 and 57
// (3488), of 48 of 25 to 1405 234 and 211 (2704), of 2 of 8000 and 8191 749 and 640
// (1032).  So the attention would take the order from fewer places on than the
// weights; one number serves both.
constexpr unsigned kInOrder = 4096;

template <bool FROM_START>
__device__ inline PromptBlock prompt_block_of_few(const Packed& s, int place, int per_token, int size) {
  const int lane = threadIdx.x % 64;
  int first = 0, last = 0;
  if (lane < s.B) prompt_range(s, lane, first, last);
  const int n = static_cast<int>((static_cast<long>(last - first) * per_token + size - 1) / size);
  const int upto = lanes_sum_upto(n);
  PromptBlock r;
  r.block = -1;
  r.used = __builtin_amdgcn_readlane(upto, 63);
  if (place >= r.used) return r;
  uint64_t here;
  int mine;  // of each lane, the block that the place would be of its sequence
  if (gridDim.x >= kInOrder) {
    here = __ballot(place < upto);
    mine = FROM_START ? place - (upto - n) : upto - 1 - place;
  } else {
    // levels: a sequence's n blocks stand on 0 .. n - 1, the first to come highest.  The highest level with
    // more blocks on and above it than `place`
    int top = n;
    top = max(top, __builtin_amdgcn_update_dpp(top, top, 0xb1, 0xf, 0xf, false));
    top = max(top, __builtin_amdgcn_update_dpp(top, top, 0x4e, 0xf, 0xf, false));
    top = max(top, __builtin_amdgcn_update_dpp(top, top, 0x141, 0xf, 0xf, false));
    top = max(top, __builtin_amdgcn_update_dpp(top, top, 0x140, 0xf, 0xf, false));
    top = max(top, __builtin_amdgcn_update_dpp(top, top, 0x142, 0xa, 0xf, false));
    top = max(top, __builtin_amdgcn_update_dpp(top, top, 0x143, 0xc, 0xf, false));
    int lo = 0, hi = __builtin_amdgcn_readlane(top, 63), above = 0;
    while (hi - lo > 1) {
      const int mid = lo + (hi - lo) / 2, count = __builtin_amdgcn_readlane(lanes_sum_upto(max(n - mid, 0)), 63);
      if (count > place) {
        lo = mid;
      } else {
        hi = mid;
        above = count;
      }
    }
    here = __ballot(n > lo);  // the sequences that reach this level, in order
    for (int i = place - above; i > 0; --i) here &= here - 1;
    mine = FROM_START ? n - 1 - lo : lo;
  }
  const int b = __builtin_ctzll(here);
  r.seq = b;
  r.first = __builtin_amdgcn_readlane(first, b);
  r.last = __builtin_amdgcn_readlane(last, b);
  r.block = __builtin_amdgcn_readlane(mine, b);
  return r;
}

// The block in a place, for any number of sequences: in their order, a
// sequence's blocks as above.  Every thread of a workgroup of THREADS calls it.
// Every workgroup looks through all starts up to its own sequence, so that the
// cost grows with the square of their number: prompts of 4 tokens (32 heads on 8
// of 64), 65 of them 12 us, 1000 107, 4000 918, 16000 12 ms.
template <int THREADS, bool FROM_START>
__device__ inline PromptBlock prompt_block(const Packed& s, unsigned place, int per_token, int size) {
  if (s.B <= 64) return prompt_block_of_few<FROM_START>(s, static_cast<int>(place), per_token, size);
  __shared__ long wave_sum[THREADS / 64];
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
      found[2] = static_cast<int>(FROM_START ? place - (sum - n) : sum - 1 - place);
      found[3] = b;
    }
    long total = 0;
    for (int i = 0; i < THREADS / 64; ++i) total += wave_sum[i];
    before += total;
    __syncthreads();
    if (found[2] >= 0) {
      r.first = __builtin_amdgcn_readfirstlane(found[0]);
      r.last = __builtin_amdgcn_readfirstlane(found[1]);
      r.block = __builtin_amdgcn_readfirstlane(found[2]);
      r.seq = __builtin_amdgcn_readfirstlane(found[3]);
      return r;
    }
    __syncthreads();
  }
  r.used = static_cast<int>(min(before, static_cast<long>(INT32_MAX)));
  return r;
}

#endif  // __HIPCC__

}  // namespace sv
