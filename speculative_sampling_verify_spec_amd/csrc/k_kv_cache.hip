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
//
// A workgroup has the K or V of a block, or both, or a share of it.  Its items
// are 4 tokens x 16 bytes of a value row, of the tokens the call touches.  For K, neighbouring lanes take
// neighbouring channels (whole rows on both sides); for V neighbouring lanes
// take neighbouring tokens, so that the four codes of a channel, one word,
// meet their neighbours in the transposed page and the rows are still touched
// 64 bytes at a time: the transposition needs no LDS.
//
// Large calls are bound by HBM: appending 4 x 8191 bf16 tokens (8 heads of
// 128) moves 201 MB in 44 us, 4.6 TB/s, and reading 64 x 1500-4096 back as
// bf16 1.45 GB in 293 us, 4.9 TB/s; a large copy reaches 4.75 TB/s.  Short
// appends are a chain of dependent loads (length; table and index; rows; the
// words shared with older tokens): 256 paths of up to 32 nodes take 19 us, 256 x
// 9 tokens 10 us and one token of 8 sequences 6 us.
#include <algorithm>

#include "sv_device.h"
#include "sv_kv.h"

namespace sv {

namespace {

// The smallest v of a workgroup of NW waves.
template <int NW>
__device__ inline int block_min_i32(int v, int* lds /* >= NW */) {
  v = wave_min_i32(v);
  if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = v;
  __syncthreads();
  int t = lds[0];
#pragma unroll
  for (int i = 1; i < NW; ++i) t = min(t, lds[i]);
  return t;
}

// Item i of a block's tokens 4 a0 .. 4 (a0 + na) - 1: tokens 4 a .. 4 a + 3,
// vector v of their rows of vpr.
__device__ inline void item_of(int isv, unsigned i, int a0, unsigned na, unsigned vpr, int& a, int& v) {
  const unsigned per = isv ? na : vpr, q = i / per, r = i - q * per;
  a = a0 + static_cast<int>(isv ? r : q);
  v = static_cast<int>(isv ? q : r);
}

// A workgroup of NW waves takes one head of one sequence, in an equal share of
// consecutive pages of those that its tokens touch: its K and V with one item
// per thread, one of them with NI items.  The values stay in registers between
// the search for the largest magnitude and the quantisation.
//
// Five waves a SIMD with one item a thread: 95 registers; left to itself the
// compiler takes 120 (256 x 32 tokens 23.2 us against 24.5), six waves spill.
template <int DT, int FMT, int NI, int NW>
__global__ __launch_bounds__(NW * kWave, NI == 1 ? 5 : 1) void k_kv_append(KvAppend p) {
  constexpr bool BOTH = NI == 1;
  constexpr int E = Elt<DT>::kPerVec, NX = BOTH ? 2 : 1, kThreads = NW * kWave;
  const KvView& c = p.c;
  const int h = BOTH ? blockIdx.y : blockIdx.y >> 1;
  const long b = blockIdx.z;
  const int tid = threadIdx.x;
  __shared__ float ldsf[NX][NW];
  __shared__ int ldsi[NW];

  const int len = kv_len(c, p.lengths, b);
  const int room = (c.width << c.pshift) - len;
  int n = min(p.counts ? min(max(p.counts[b], 0), p.N) : p.N, room);
  // the tokens end at the first index outside [0, N), and at the first page
  // the table does not have; what counts is every page and token up to this
  // workgroup's last (all of them, where the new length is written)
  const bool reports = blockIdx.x == 0 && blockIdx.y == 0 && p.out_lengths;
  const int col0 = len >> c.pshift;
  int stop = n, first = 0, per = 1;  // this workgroup's first page, from col0 on, and how many
  if (n > 0) {
    // shares of the pages that this sequence's tokens can touch, not of the
    // call's: a call padded to many more keeps its workgroups busy (1000 tokens
    // of 131072, pages of 16: 9.4 us, in shares of the call's pages 30)
    const int end = (len + n - 1) >> c.pshift, groups = gridDim.x;
    if (end - col0 >= groups) per = (end - col0 + groups) / groups;
    first = static_cast<int>(blockIdx.x) * per;
    if (first > end - col0) return;
    const int last = reports ? end : min(end, col0 + first + per - 1);
    const int upto = last == end ? n : ((last + 1) << c.pshift) - len;  // tokens up to there
    const int i0 = min(tid, upto - 1), c0 = min(col0 + tid, last);  // both loads before either test
    const int ix0 = p.index ? p.index[b * p.N + i0] : 0, id0 = c.table[b * c.width + c0];
    if (ix0 < 0 || ix0 >= p.N) stop = min(stop, i0);
    if (id0 < 0 || id0 >= c.pages) stop = min(stop, max((c0 << c.pshift) - len, 0));
    // long calls: the loads of several turns go out together (131072 tokens
    // of 8 heads of 64 in pages of 16: 130 us, one by one 165; by index 362 and 928)
    if (p.index)
#pragma unroll 8
      for (int i = tid + kThreads; i < upto; i += kThreads) {
        const int ix = p.index[b * p.N + i];
        stop = ix < 0 || ix >= p.N ? min(stop, i) : stop;
      }
#pragma unroll 8
    for (int col = col0 + tid + kThreads; col <= last; col += kThreads) {
      const int id = c.table[b * c.width + col];
      stop = id < 0 || id >= c.pages ? min(stop, max((col << c.pshift) - len, 0)) : stop;
    }
  }
  n = block_min_i32<NW>(stop, ldsi);
  if (reports && tid == 0) p.out_lengths[b] = len + n;
  if (n <= 0) return;  // below, every page visited gets at least one token

  const int vpr = c.D / E;
  const int wave0 = __builtin_amdgcn_readfirstlane(tid) & ~(kWave - 1);  // the wave's first item
  // the tokens of its pages end here
  const long stop_at = min(static_cast<long>(len) + n, (static_cast<long>(col0) + first + per) << c.pshift);
  for (long col = static_cast<long>(col0) + first; (col << c.pshift) < stop_at; ++col) {
    const long p0 = col << c.pshift;                                            // the page's first position
    const int t0 = static_cast<int>(max(len - p0, 0L));                         // tokens of it cached before
    const int t1 = static_cast<int>(min(stop_at - p0, static_cast<long>(c.P)));  // and after
    const long blk = static_cast<long>(kv_page(c, b, col)) * c.H + h;  // a page: n ends before the first that is not
    // only the groups of four tokens that get new ones
    const int a0 = t0 / 4, na = (t1 + 3) / 4 - a0, items = na * vpr;
    // byte masks of a word of tokens 4 a .. 4 a + 3: those this call writes,
    // and those cached before
    auto fresh_mask = [&](int a) {
      uint32_t m = 0;
#pragma unroll
      for (int r = 0; r < 4; ++r) m |= 4 * a + r >= t0 && 4 * a + r < t1 ? 0xffu << (8 * r) : 0u;
      return m;
    };
    auto old_mask = [&](int a) {
      uint32_t m = 0;
#pragma unroll
      for (int r = 0; r < 4; ++r) m |= 4 * a + r < t0 ? 0xffu << (8 * r) : 0u;
      return m;
    };

    uint4 raw[NX][NI][4];
    uint32_t cur[NI][E];  // V: words that get some new bytes, as they are
    float s_old[NX], amax[NX];
    bool wild[NX];  // this lane holds a value that is not finite
#pragma unroll
    for (int x = 0; x < NX; ++x) {
      const int isv = BOTH ? x : blockIdx.y & 1;
      s_old[x] = (isv ? c.vs : c.ks)[blk];
      const char* src = static_cast<const char*>(isv ? p.v : p.k) + static_cast<long>(h) * c.D * Elt<DT>::kBytes;
      const uint8_t* page = c.vp + blk * c.P * c.D;
#pragma unroll
      for (int k = 0; k < NI; ++k) {
        const int i = tid + k * kThreads;
        int a, v;
        item_of(isv, i, a0, na, vpr, a, v);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = 4 * a + r;
          raw[x][k][r] = make_uint4(0, 0, 0, 0);
          if (i < items && t >= t0 && t < t1) {
            const long at = p0 + t - len;
            const long row = b * p.N + (p.index ? p.index[b * p.N + at] : at);
            raw[x][k][r] = load16(src + row * p.row * Elt<DT>::kBytes, v);
          }
        }
        if (isv && i < items) {
          const uint32_t fresh = fresh_mask(a);
          if (fresh && fresh != ~0u)
#pragma unroll
            for (int j = 0; j < E; ++j)
              cur[k][j] = *reinterpret_cast<const uint32_t*>(page + static_cast<long>(v * E + j) * c.P + 4 * a);
        }
      }
    }
#pragma unroll
    for (int x = 0; x < NX; ++x) {
      MaxBits<DT> top;
#pragma unroll
      for (int k = 0; k < NI; ++k)
        if (wave0 + k * kThreads < items)
#pragma unroll
          for (int r = 0; r < 4; ++r) top.add(raw[x][k][r]);
      wild[x] = top.wild();
      amax[x] = wave_max(top.value());
    }
    __syncthreads();  // also: nobody reads the LDS of the page before any more
    if (tid % kWave == 0)
#pragma unroll
      for (int x = 0; x < NX; ++x) ldsf[x][tid / kWave] = amax[x];
    __syncthreads();
#pragma unroll
    for (int x = 0; x < NX; ++x) {
      const int isv = BOTH ? x : blockIdx.y & 1;
      float top = ldsf[x][0];
#pragma unroll
      for (int i = 1; i < NW; ++i) top = fmaxf(top, ldsf[x][i]);
      float s = kv_scale<FMT>(top);
      if (t0 > 0) s = fmaxf(s, s_old[x]);
      const bool grow = t0 > 0 && s > s_old[x];  // the tokens that were there go to the grown scale
      const float inv = 1.f / s, ratio = s_old[x] * inv;
      uint8_t* page = (isv ? c.vp : c.kp) + blk * c.P * c.D;
#pragma unroll
      for (int k = 0; k < NI; ++k) {
        const int i = tid + k * kThreads;
        if (i >= items) break;
        int a, v;
        item_of(isv, i, a0, na, vpr, a, v);
        float f[4][E];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          Elt<DT>::unpack(raw[x][k][r], f[r]);
#pragma unroll
          for (int j = 0; j < E; ++j) f[r][j] *= inv;
        }
        if (!isv) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int t = 4 * a + r;
            uint32_t* at = reinterpret_cast<uint32_t*>(page + static_cast<long>(t) * c.D + v * E);
            const bool fresh = t >= t0 && t < t1;
            if (!fresh && !(grow && t < t0)) continue;
            uint32_t w[E / 4];
            if (fresh) {
#pragma unroll
              for (int j = 0; j < E / 4; ++j)
                w[j] = wild[x] ? kv_encode4<FMT>(&f[r][4 * j]) : kv_encode4_finite<FMT>(&f[r][4 * j]);
            } else {
              uint32_t had[E / 4];
#pragma unroll
              for (int j = 0; j < E / 4; ++j) had[j] = at[j];
#pragma unroll
              for (int j = 0; j < E / 4; ++j) w[j] = kv_rescale4<FMT>(had[j], ratio);
            }
            if constexpr (E == 8) *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
            else *at = w[0];
          }
        } else {
          const uint32_t fresh = fresh_mask(a), again = grow ? old_mask(a) : 0;
          uint32_t* at = reinterpret_cast<uint32_t*>(page + static_cast<long>(v * E) * c.P + 4 * a);
          const int step = c.P / 4;
#pragma unroll
          for (int j = 0; j < E; ++j) {
            const float y[4] = {f[0][j], f[1][j], f[2][j], f[3][j]};
            uint32_t w = wild[x] ? kv_encode4<FMT>(y) : kv_encode4_finite<FMT>(y);
            if (fresh != ~0u) {
              w = (w & fresh) | (cur[k][j] & ~fresh);
              if (again) w = (w & ~again) | (kv_rescale4<FMT>(cur[k][j], ratio) & again);
            }
            at[j * step] = w;
          }
        }
      }
      if (grow)  // the groups before, of old tokens only
        for (int i = tid; i < a0 * vpr; i += kThreads) {
          int a, v;
          item_of(isv, i, 0, a0, vpr, a, v);
          // K: 4 rows of E codes; V: E rows of 4
          uint32_t* at = reinterpret_cast<uint32_t*>(page + (isv ? static_cast<long>(v * E) * c.P + 4 * a
                                                                : static_cast<long>(4 * a) * c.D + v * E));
          const int step = (isv ? c.P : c.D) / 4;
          uint32_t had[E];
#pragma unroll
          for (int j = 0; j < E; ++j) had[j] = at[isv ? j * step : j / (E / 4) * step + j % (E / 4)];
#pragma unroll
          for (int j = 0; j < E; ++j)
            at[isv ? j * step : j / (E / 4) * step + j % (E / 4)] = kv_rescale4<FMT>(had[j], ratio);
        }
      if (tid == 0) (isv ? c.vs : c.ks)[blk] = s;
    }
  }
}

// One workgroup per (page the range may touch, K or V of a head, sequence),
// NI items per thread; SPREAD: one item per thread, p.chunks workgroups per
// page.
template <int DT, int FMT, int NI, bool SPREAD>
__global__ __launch_bounds__(kBlock) void k_kv_read(KvRead p) {
  constexpr int E = Elt<DT>::kPerVec;
  const KvView& c = p.c;
  const int slot = SPREAD ? blockIdx.x / p.chunks : blockIdx.x, first = SPREAD ? (blockIdx.x - slot * p.chunks) * kBlock : 0;
  const int h = blockIdx.y >> 1, isv = blockIdx.y & 1;
  const long b = blockIdx.z;
  void* out = isv ? p.out_v : p.out_k;
  if (!out) return;
  const int len = kv_len(c, p.lengths, b);
  const long start = p.starts ? max(p.starts[b], 0) : 0;
  const long p0 = ((start >> c.pshift) + slot) << c.pshift;
  // the page's tokens t0 .. t1 - 1 are written, those from `have` on as 0
  const int t0 = static_cast<int>(max(start - p0, 0L));
  const int t1 = static_cast<int>(min(start + p.T - p0, static_cast<long>(c.P)));
  if (t1 <= t0) return;
  const int id = kv_page(c, b, p0 >> c.pshift);
  const int have = id < 0 ? 0 : static_cast<int>(max(min(len - p0, static_cast<long>(c.P)), 0L));
  const long blk = static_cast<long>(max(id, 0)) * c.H + h;
  const float s = (isv ? c.vs : c.ks)[blk];
  const uint8_t* page = (isv ? c.vp : c.kp) + blk * c.P * c.D;
  const int a0 = t0 / 4, na = (t1 + 3) / 4 - a0, vpr = c.D / E, items = na * vpr;
  if (SPREAD && first + static_cast<int>(threadIdx.x) >= items) return;
  // row t's place in the output: token p0 + t - start
  const long row0 = b * p.T + (p0 - start);

  // Blocks next to the largest float: a code times the scale can pass the
  // output type's range where the value that was appended did not.
  constexpr float top = kLargest<DT>;
  const bool huge = s > 0x1p119f;

  uint32_t raw[NI][E];  // K: words of 4 channels, [token][E / 4]; V: words of 4 tokens, [channel]
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const int i = first + static_cast<int>(threadIdx.x) + k * kBlock;
    int a, v;
    item_of(isv, i < items ? i : 0, a0, na, vpr, a, v);
    if (!isv) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t* at = reinterpret_cast<const uint32_t*>(page + static_cast<long>(4 * a + r) * c.D + v * E);
        if constexpr (E == 8) {
          const uint2 w = *reinterpret_cast<const uint2*>(at);
          raw[k][2 * r] = w.x;
          raw[k][2 * r + 1] = w.y;
        } else {
          raw[k][r] = *at;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j)
        raw[k][j] = *reinterpret_cast<const uint32_t*>(page + static_cast<long>(v * E + j) * c.P + 4 * a);
    }
  }
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const int i = first + static_cast<int>(threadIdx.x) + k * kBlock;
    if (i >= items) break;
    int a, v;
    item_of(isv, i, a0, na, vpr, a, v);
    float f[4][E];
    if (!isv) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int j = 0; j < E / 4; ++j) kv_decode4<FMT>(raw[k][r * (E / 4) + j], &f[r][4 * j]);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) {
        float g[4];
        kv_decode4<FMT>(raw[k][j], g);
#pragma unroll
        for (int r = 0; r < 4; ++r) f[r][j] = g[r];
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 4 * a + r;
      if (t < t0 || t >= t1) continue;
#pragma unroll
      for (int j = 0; j < E; ++j) f[r][j] = t < have ? f[r][j] * s : 0.f;
      if (huge)
#pragma unroll
        for (int j = 0; j < E; ++j) f[r][j] = f[r][j] > top ? top : f[r][j] < -top ? -top : f[r][j];  // NaN stays
      kv_store16<DT>(out, ((row0 + t) * c.H + h) * c.D + v * E, f[r]);
    }
  }
}

template <int DT, int FMT>
hipError_t append(const KvAppend& p, hipStream_t st) {
  // items of a page that N tokens can touch, wherever they begin: at most 2048
  const int items = std::min(p.c.P / 4, (std::min(p.N, p.c.P) + 6) / 4) * (p.c.D / Elt<DT>::kPerVec);
  const unsigned H = static_cast<unsigned>(p.c.H), B = static_cast<unsigned>(p.B);
  // K and V in one workgroup share the table, index and length reads: 256 x 6
  // tokens by four waves 13.9 us, apart 17.3 (D = 128, P = 64).  With two items a
  // thread the registers count for more: 64 x 100 tokens (D = 128, P = 128) 16.0 us
  // together, 14.3 apart, 4 x 4096 23.8 and 22.4, but 256 x 64 34.2 and 37.0.
#define LAUNCH(ni, nw) \
  hipLaunchKernelGGL((k_kv_append<DT, FMT, ni, nw>), dim3(p.groups, ni == 1 ? H : 2 * H, B), dim3(nw * kWave), 0, st, p)
  // No more waves than items.  One wave: 256 x 9 tokens (P = 64, 8 heads of 128) 10.4 us, by
  // four waves 13.8; 256 x 1 9.7 and 13.2; 64 x 9 7.0 and 7.5, but 14.4 and 12.6
  // if every block's scale grows.  More in turns of one wave queue up: 256
  // paths of up to 32 nodes and their read 89 us against 70.  Three waves: the
  // same paths and read 40.4 us, by four 41.5.
  if (items <= kWave) LAUNCH(1, 1);
  else if (items <= 2 * kWave) LAUNCH(1, 2);
  else if (items <= 3 * kWave) LAUNCH(1, 3);
  else if (items <= kBlock) LAUNCH(1, kWaves);
  else if (items <= 2 * kBlock) LAUNCH(2, kWaves);
  else if (items <= 4 * kBlock) LAUNCH(4, kWaves);
  else if constexpr (DT == SPECV_F32) LAUNCH(8, kWaves);
#undef LAUNCH
  return hipGetLastError();
}

template <int DT, int FMT>
hipError_t read(KvRead p, hipStream_t st) {
  // items of a page that T tokens can touch, wherever they begin
  const int items = std::min(p.c.P / 4, (std::min(p.T, p.c.P) + 6) / 4) * (p.c.D / Elt<DT>::kPerVec);
  // Calls over whole pages spread a page's items over workgroups: 16 x 4096
  // tokens (P = 128) 98 us, with several items a thread 102 (bf16, D = 128), 173 and
  // 196 (fp32, D = 256).  In short calls the workgroups that find nothing to do
  // count: 256 x 33 tokens in fp32 (P = 64, D = 128) 43 us spread and 28 not.
  p.chunks = p.T >= 4 * p.c.P ? (items + kBlock - 1) / kBlock : 1;
  const dim3 grid(kv_slots(p.T, p.c.P) * p.chunks, static_cast<unsigned>(2 * p.c.H), static_cast<unsigned>(p.B));
  // no more waves than items: 64 x 100 tokens (P = 16, D = 64) 9.0 us, four waves each 12.4
  const dim3 block(std::min((items + kWave - 1) / kWave * kWave, kBlock));
#define LAUNCH(ni, spread) hipLaunchKernelGGL((k_kv_read<DT, FMT, ni, spread>), grid, block, 0, st, p)
  if (p.chunks > 1) LAUNCH(1, true);
  else if (items <= kBlock) LAUNCH(1, false);
  else if (items <= 2 * kBlock) LAUNCH(2, false);
  else if (items <= 4 * kBlock) LAUNCH(4, false);
  else if constexpr (DT == SPECV_F32) LAUNCH(8, false);
#undef LAUNCH
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const KvAppend& p, int dtype, int fmt, hipStream_t st) {
  if (dtype == SPECV_F32)
    return fmt == SPECV_E4M3 ? append<SPECV_F32, SPECV_E4M3>(p, st) : append<SPECV_F32, SPECV_I8>(p, st);
  return fmt == SPECV_E4M3 ? append<SPECV_BF16, SPECV_E4M3>(p, st) : append<SPECV_BF16, SPECV_I8>(p, st);
}

hipError_t launch_kv_read(const KvRead& p, int dtype, int fmt, hipStream_t st) {
  if (dtype == SPECV_F32)
    return fmt == SPECV_E4M3 ? read<SPECV_F32, SPECV_E4M3>(p, st) : read<SPECV_F32, SPECV_I8>(p, st);
  return fmt == SPECV_E4M3 ? read<SPECV_BF16, SPECV_E4M3>(p, st) : read<SPECV_BF16, SPECV_I8>(p, st);
}

}  // namespace sv
