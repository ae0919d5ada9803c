// Embedding table on the Adam path (include/muon_embed.h): lookup, gradient by
// sorted tokens, and the Adam step of the rows a batch has touched.
//
//   out_i = s E[t_i];   G[v] = s sum_{i: t_i = v} dout_i
//
// All of it is bound by HBM, or by the launches for small batches. The
// gradient takes three launches:
//  - sort: a block owns R consecutive vocabulary entries in one segment of the
//    batch. It reads all n tokens, counts those of its range before, in and
//    behind its segment and those below its range (which gives the place of
//    its first token without any other block's word), and writes its tokens'
//    records ordered by token, then by position. No atomics across blocks, no
//    sum that depends on how tokens are spread, any n.
//  - sum: the sorted records are cut into chunks of equal length, whatever
//    tokens they hold. A wave takes the columns of a slab through one chunk and
//    writes the sum of each token that lies within it; a token that crosses a
//    chunk's border leaves float32 partial sums, one per chunk.
//  - join: adds a crossing token's partial sums in order, in float64.
// Equal inputs give equal bits: no sum depends on which wave comes first.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>

#include "../../include/muon_embed.h"
#include "adam_elem.hpp"
#include "embed_grid.hpp"

namespace muon_embed {

using muon_adam::kVec;

constexpr int kSortThreads = 512;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortLoads = 8;      // tokens a lane has in flight
constexpr int kQueue = 64 * (kSortLoads + 1);  // of a wave: tokens found, not yet placed
constexpr int kMaxRange = 3000;    // vocabulary entries of a sort block, at most: ten counters each, 117 of the 160 KB of LDS (reached where vocab * segments exceeds 3000 * kSortBlocks)
constexpr int kSortBlocks = 256;   // sort blocks: one per CU
constexpr int kSegment = 4096;     // tokens of a segment of the batch, at least
constexpr int kSlab = 64 * kVec;   // columns of a wave in the sum
constexpr int64_t kSumWaves = 4096;  // waves of the sum aimed at: 16 on each CU
constexpr int64_t kMaxWaves = 1 << 23;  // of one launch (the join has a block for each)

// A sorted token.
struct Rec {
  int32_t pos;   // its position in the batch
  int32_t key;   // the token
  int32_t slot;  // the token's rank among the distinct tokens of its range
  int32_t end;   // index behind the token's last record
};

// Vectors at an element's alignment (the hardware takes any address).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4 __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {  // round to nearest even
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, b2));
}

// Eight consecutive elements, the first `n` of them if fewer are left.
__device__ __forceinline__ void load8(const uint16_t* p, int n, float (&x)[8]) {
  if (n >= 8) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      x[2 * q] = __uint_as_float(w[q] << 16);
      x[2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = q < n ? muon_adam::bf2f(p[q]) : 0.f;
  }
}
__device__ __forceinline__ void load8(const float* p, int n, float (&x)[8]) {
  if (n >= 8) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      x[q] = a[q];
      x[q + 4] = b[q];
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = q < n ? p[q] : 0.f;
  }
}
__device__ __forceinline__ void store8(uint16_t* p, int n, const float (&x)[8]) {
  if (n >= 8) {
    const u32x4 w = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
    *reinterpret_cast<u32x4*>(p) = w;
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < n) p[q] = static_cast<uint16_t>(pack_bf16(x[q], 0.f));
  }
}
__device__ __forceinline__ void store8(float* p, int n, const float (&x)[8]) {
  if (n >= 8) {
    *reinterpret_cast<f32x4*>(p) = f32x4{x[0], x[1], x[2], x[3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < n) p[q] = x[q];
  }
}
// The same for four.
template <typename T>
__device__ __forceinline__ void load4_of(const T* p, int n, float (&x)[kVec]) {
  if (n >= kVec) {
    muon_adam::load4<false>(p, x);
  } else {
#pragma unroll
    for (int q = 0; q < kVec; ++q) x[q] = q < n ? muon_adam::PElem<T>::load(p, q) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store4_of(T* p, int n, const float (&x)[kVec]) {
  if (n >= kVec) {
    muon_adam::store4<false>(p, x);
  } else {
#pragma unroll
    for (int q = 0; q < kVec; ++q)
      if (q < n) muon_adam::PElem<T>::store(p, q, x[q]);
  }
}

// A token as it was given, -1 where it is outside the vocabulary.
__device__ __forceinline__ int32_t narrow(int32_t t, int32_t vocab) {
  return static_cast<uint32_t>(t) < static_cast<uint32_t>(vocab) ? t : -1;
}
__device__ __forceinline__ int32_t narrow(int64_t t, int32_t vocab) {
  return (t >> 32) == 0 ? narrow(static_cast<int32_t>(t), vocab) : -1;
}
template <typename I>
__device__ __forceinline__ int32_t token(const I* tokens, int64_t i, int32_t vocab) {
  return narrow(tokens[i], vocab);
}

// A wave's tokens i0 + 64 u + lane, u < U; behind fin the last one again, so
// that no load is behind a branch.
template <int U, typename I>
__device__ __forceinline__ void load_tokens(const I* tokens, int64_t i0, int64_t fin, int lane, I (&t)[U]) {
  if (i0 + 64 * U <= fin) {
#pragma unroll
    for (int u = 0; u < U; ++u) t[u] = tokens[i0 + 64 * u + lane];
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) t[u] = tokens[min(i0 + 64 * u + lane, fin - 1)];
  }
}
// A token as 32 bits, all of them set for one that no vocabulary (at most 2^24
// entries) has. Both passes of the sort test each token's range in as few
// instructions as they can: every block reads the whole batch.
__device__ __forceinline__ uint32_t narrow(int32_t t) { return static_cast<uint32_t>(t); }
__device__ __forceinline__ uint32_t narrow(int64_t t) { return static_cast<uint64_t>(t) >> 32 ? ~0u : static_cast<uint32_t>(t); }
// The first `left` of a wave's batch; none of the others is in a range.
template <int U, typename I>
__device__ __forceinline__ void narrow_all(const I (&t)[U], int left, int lane, uint32_t (&v)[U]) {
#pragma unroll
  for (int u = 0; u < U; ++u) v[u] = narrow(t[u]);
  if (left < 64 * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = 64 * u + lane < left ? v[u] : ~0u;
  }
}

// k / d for magic = (2^32 - 1) / d: 2^32 - magic d lies in [1, d], so the
// product's high word is the quotient or one less.
__device__ __forceinline__ uint32_t div_by(uint32_t k, uint32_t d, uint32_t magic) {
  const uint32_t q = __umulhi(k, magic);
  return k - q * d >= d ? q + 1 : q;
}

// ----------------------------------------------------------------- lookup

struct LookArgs {
  const void* table;
  const void* tokens;
  void* out;
  int64_t ld, out_ld;
  int64_t n;
  int32_t vocab, cols;
  int32_t vpr;      // vectors in a row
  int32_t per;      // tokens of a block
  uint32_t magic;   // for divisions by vpr
  float scale;
};

// A row's last vector starts at cols - 8 where the row is no whole number of
// them: some elements are written twice, with the same value. Loads are
// without branches, so that all of a thread's are in flight at once: a token
// outside the vocabulary loads row 0 and stores zeros. 8192 tokens of 768 bf16
// elements 5.4 us; 65536 of 1021 fp32 ones to bf16 (145 MB read from HBM, 134
// written) 55.5 us, 5.0 TB/s (with 1, 2, 4 and 8 vectors in flight 58, 55, 55.5
// and 56.5 us).
template <typename E, typename O, typename I>
__global__ __launch_bounds__(kThreads) void embed_lookup_kernel(LookArgs A) {
  const int64_t first = int64_t(blockIdx.x) * A.per;
  const int64_t left = A.n - first;
  const uint32_t vpr = static_cast<uint32_t>(A.vpr);
  const uint32_t nv = vpr * static_cast<uint32_t>(left < A.per ? left : A.per);
  const E* const table = static_cast<const E*>(A.table);
  O* const out = static_cast<O*>(A.out) + first * A.out_ld;
  const I* const tokens = static_cast<const I*>(A.tokens) + first;
  if (A.cols < kLookVec) {  // narrow rows: one vector each
    for (uint32_t k = threadIdx.x; k < nv; k += kThreads) {
      const int32_t t = token(tokens, k, A.vocab);
      float x[8];
      load8(table + int64_t(max(t, 0)) * A.ld, A.cols, x);
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = t >= 0 ? x[q] * A.scale : 0.f;
      store8(out + k * A.out_ld, A.cols, x);
    }
    return;
  }
  for (uint32_t k0 = threadIdx.x; k0 < nv; k0 += kThreads * kLookRuns) {
    float x[kLookRuns][8];
    int32_t t[kLookRuns];
    int64_t at[kLookRuns];
    int c[kLookRuns];
#pragma unroll
    for (int j = 0; j < kLookRuns; ++j) {
      const uint32_t k = min(k0 + j * kThreads, nv - 1), r = div_by(k, vpr, A.magic);
      c[j] = min(static_cast<int>(k - r * vpr) * kLookVec, A.cols - kLookVec);
      at[j] = int64_t(r) * A.out_ld + c[j];
      t[j] = token(tokens, r, A.vocab);
    }
#pragma unroll
    for (int j = 0; j < kLookRuns; ++j) load8(table + int64_t(max(t[j], 0)) * A.ld + c[j], 8, x[j]);
#pragma unroll
    for (int j = 0; j < kLookRuns; ++j) {
      if (k0 + j * kThreads >= nv) break;
#pragma unroll
      for (int q = 0; q < 8; ++q) x[j][q] = t[j] >= 0 ? x[j][q] * A.scale : 0.f;
      store8(out + at[j], 8, x[j]);
    }
  }
}

// ------------------------------------------------------------------- sort

struct SortArgs {
  const void* tokens;
  Rec* recs;
  int32_t* distinct;  // per range: its distinct tokens
  int32_t* live;      // tokens inside the vocabulary
  uint8_t* present;   // dense form: whether a token occurs (nullptr: not wanted)
  int32_t n, vocab, range;
  int32_t segments, run;  // of the batch; tokens of a wave in its block's segment, a multiple of 64
  int32_t bits;           // of a token's place in the range
};

__device__ __forceinline__ int lanes_below(uint64_t mask, int lane) {
  return __popcll(mask & ((uint64_t(1) << lane) - 1));
}

// Bound by instructions and latency, not bytes: every block reads the whole
// batch, from its XCD's L2. 32768 int64 tokens 19 us (reading and counting 8,
// scan 3, placing 3 to 6), 65536 of a vocabulary of 100003 36 us, 8192 int32
// ones 11, 17 ones 5. Sixteen tokens of a lane in flight for eight: 25 us for
// 19, the longer body being read through the instruction cache by every block.
//
// A batch's frequent tokens fall into few ranges, whose blocks set the time:
// hence the segments. What else counts is the number of instructions a token
// takes in the blocks that it does not belong to, and their size (a long
// unrolled body takes as long to fetch as to run): tokens are compared as 32
// bits (21 -> 19 us against 64; one outside the vocabulary is in no range), and
// those of the range are queued and placed 64 at a time.
template <typename I>
__global__ __launch_bounds__(kSortThreads) void embed_sort_kernel(SortArgs A) {
  extern __shared__ __align__(16) int32_t lds[];
  constexpr int W = kSortWaves, U = kSortLoads;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int part = blockIdx.x / A.segments, segment = blockIdx.x - part * A.segments;
  const int lo = part * A.range;
  const int nk = min(A.range, A.vocab - lo);
  int32_t* const cnt = lds;              // [key][wave]: the wave's tokens, then where its next one goes
  int32_t* const before = lds + W * nk;  // [key]: tokens of earlier segments; then the end of the token's records
  int32_t* const behind = before + nk;   // [key]: of later segments; then the token's rank in the range
  __shared__ uint2 queues[W][kQueue];
  __shared__ int32_t below[W];
  __shared__ int64_t scan[W];
  for (int i = tid * 4; i < (W + 2) * nk; i += kSortThreads * 4) *reinterpret_cast<int4*>(lds + i) = int4{0, 0, 0, 0};
  __syncthreads();

  const I* const tokens = static_cast<const I*>(A.tokens);
  const int64_t seg0 = min(int64_t(A.n), segment * int64_t(A.run) * W), seg1 = min(int64_t(A.n), seg0 + int64_t(A.run) * W);
  const int64_t run0 = min(seg1, seg0 + int64_t(wave) * A.run), run1 = min(seg1, run0 + A.run);  // the wave's own
  int under = 0;
#pragma unroll 1
  for (int stage = 0; stage < 3; ++stage) {  // earlier segments, the block's, later ones
    int64_t beg = run0, fin = run1;
    int32_t* to = cnt + wave;
    if (stage != 1) {  // a share for every wave
      const int64_t from = stage == 0 ? 0 : seg1, till = stage == 0 ? seg0 : int64_t(A.n);
      const int64_t each = ((till - from + kSortThreads - 1) / kSortThreads) * 64;
      beg = min(till, from + wave * each);
      fin = min(till, beg + each);
      to = stage == 0 ? before : behind;
    }
    const int pitch = stage == 1 ? W : 1;
    I next[U];
    if (beg < fin) load_tokens(tokens, beg, fin, lane, next);
#pragma unroll 1
    for (int64_t i0 = beg; i0 < fin; i0 += 64 * U) {
      uint32_t v[U];
      narrow_all(next, static_cast<int>(min(fin - i0, int64_t(64 * U))), lane, v);
      load_tokens(tokens, min(i0 + 64 * U, fin - 1), fin, lane, next);  // in flight meanwhile
#pragma unroll
      for (int u = 0; u < U; ++u) {
        under += __popcll(__ballot(v[u] < static_cast<uint32_t>(lo)));
        const uint32_t k = v[u] - lo;
        if (k < static_cast<uint32_t>(nk)) atomicAdd(to + k * pitch, 1);
      }
    }
  }
  if (lane == 0) below[wave] = under;
  __syncthreads();

  I ahead[U];  // the wave's first tokens to place, on their way during the scan
  if (run0 < run1) load_tokens(tokens, run0, run1, lane, ahead);

  // Starts of the tokens: a scan over the keys of (count, is there any) in one 64-bit sum.
  int64_t carry = 0;
  for (int w = 0; w < W; ++w) carry += below[w];
  const int first = static_cast<int>(carry);
#pragma unroll 1
  for (int k0 = 0; k0 < nk; k0 += kSortThreads) {
    const int k = k0 + tid;
    int total = 0, early = 0, c[W] = {};
    if (k < nk) {
      static_assert(W == 8, "two vectors of four counters");
      const int4 x = *reinterpret_cast<const int4*>(cnt + W * k), y = *reinterpret_cast<const int4*>(cnt + W * k + 4);
      c[0] = x.x, c[1] = x.y, c[2] = x.z, c[3] = x.w, c[4] = y.x, c[5] = y.y, c[6] = y.z, c[7] = y.w;
      early = before[k];
      total = early + behind[k];
#pragma unroll
      for (int w = 0; w < W; ++w) total += c[w];
    }
    const int64_t own = int64_t(total) + (total > 0 ? int64_t(1) << 32 : 0);
    int64_t x = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t y = __shfl_up(x, o, 64);
      if (lane >= o) x += y;
    }
    if (lane == 63) scan[wave] = x;
    __syncthreads();
    int64_t base = carry;
    for (int w = 0; w < W; ++w) {
      if (w < wave) base += scan[w];
      carry += scan[w];
    }
    if (k < nk) {
      const int64_t at = base + x - own;
      int start = static_cast<int>(at) + early;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const int n = c[w];
        c[w] = start;
        start += n;
      }
      *reinterpret_cast<int4*>(cnt + W * k) = int4{c[0], c[1], c[2], c[3]};
      *reinterpret_cast<int4*>(cnt + W * k + 4) = int4{c[4], c[5], c[6], c[7]};
      before[k] = static_cast<int>(at) + total;
      behind[k] = static_cast<int>(at >> 32);
    }
    __syncthreads();
  }
  const int32_t* const end = before;
  const int32_t* const slot = behind;
  if (tid == 0 && segment == 0) {
    A.distinct[part] = static_cast<int>(carry >> 32);
    if (blockIdx.x + A.segments == gridDim.x) *A.live = static_cast<int>(carry);
  }

  if (static_cast<int>(carry) > first && run0 < run1) {
    // read by lanes other than the ones that wrote it
    volatile int32_t* const mine = cnt + wave;
    volatile uint2* const queue = queues[wave];
    int have = 0;
#pragma unroll 1
    for (int64_t i0 = run0; i0 < run1; i0 += 64 * U) {
      uint32_t v[U];
      narrow_all(ahead, static_cast<int>(min(run1 - i0, int64_t(64 * U))), lane, v);
      load_tokens(tokens, min(i0 + 64 * U, run1 - 1), run1, lane, ahead);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t k = v[u] - lo;
        const bool in = k < static_cast<uint32_t>(nk);
        const uint64_t found = __ballot(in);
        if (in) {
          const int at = have + lanes_below(found, lane);
          queue[at].x = k;
          queue[at].y = static_cast<uint32_t>(i0) + 64 * u + lane;
        }
        have += __popcll(found);
      }
      const bool last = i0 + 64 * U >= run1;
      int taken = 0;
#pragma unroll 1
      for (; have - taken >= 64 || (last && taken < have); taken += 64) {
        const bool in = lane < have - taken;
        const uint32_t k = queue[taken + (in ? lane : 0)].x, pos = queue[taken + (in ? lane : 0)].y;
        uint64_t same = __ballot(in);
        uint32_t same0 = static_cast<uint32_t>(same), same1 = static_cast<uint32_t>(same >> 32);
#pragma unroll 1
        for (int b = 0; b < A.bits; ++b) {  // the lanes with this lane's token
          const uint64_t with = __ballot((k >> b) & 1);
          const uint32_t flip = ((k >> b) & 1) - 1;  // lanes with the bit keep `with`, those without its complement
          same0 &= static_cast<uint32_t>(with) ^ flip;
          same1 &= static_cast<uint32_t>(with >> 32) ^ flip;
        }
        if (in) {
          same = static_cast<uint64_t>(same1) << 32 | same0;
          const int at = mine[W * k], earlier = lanes_below(same, lane);
          A.recs[at + earlier] = {static_cast<int32_t>(pos), lo + static_cast<int32_t>(k), slot[k], end[k]};
          if (earlier == 0) mine[W * k] = at + __popcll(same);
        }
      }
      if (taken < have && taken > 0) {  // fewer than 64 are left: to the front
        const bool in = lane < have - taken;
        const uint32_t k = queue[taken + (in ? lane : 0)].x, pos = queue[taken + (in ? lane : 0)].y;
        if (in) {
          queue[lane].x = k;
          queue[lane].y = pos;
        }
      }
      have = max(0, have - taken);
    }
  }

  if (A.present == nullptr || segment != 0) return;
  // all of a token's records end behind its first one, so an empty token's end is where the next one starts
  for (int k = tid; k < nk; k += kSortThreads) A.present[lo + k] = end[k] != (k > 0 ? end[k - 1] : first);
}

// -------------------------------------------------------------------- sum

enum Mode { kDense = 0, kAdd = 1, kRows = 2 };

struct SumArgs {
  const Rec* recs;
  const int32_t* distinct;
  const int32_t* live;
  const void* dout;
  int64_t dout_ld;
  void* grad;       // dense and add: the table's gradient; rows: the values
  int64_t grad_ld;
  int32_t* rows;    // rows: the tokens
  int32_t* count;   // rows: how many
  float* head;      // [chunk][ld_part]: the part of a token that began in an earlier chunk
  float* tail;      // [chunk][ld_part]: the first part of a token that goes on in the next chunk
  int64_t ld_part;
  int64_t n;        // records, live and not
  const uint8_t* present;  // dense form
  int32_t cols, slabs, chunks, chunk, range, ranges, vocab;
  int32_t sum_blocks;      // the blocks behind them clear rows
  float scale;
};

constexpr int kClearRows = 16;  // of a wave

__device__ __forceinline__ int wave_sum(int x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
  return x;
}

// Distinct tokens in ranges [b0, b1): the same for every lane.
__device__ __forceinline__ int distinct_in(const int32_t* distinct, int b0, int b1, int lane) {
  int s = 0;
  for (int b = b0 + lane; b < b1; b += 64) s += distinct[b];
  return __builtin_amdgcn_readfirstlane(wave_sum(s));
}

// A lane has columns [col, col + 4) and works on [from, from + 4), which differs
// where the row ends: its last lane then does some of the columns before its
// own once more (rows of under four columns aside).
struct Cols {
  int col, nc;  // nc: how many of them exist, at most zero for none
  int from;
};
__device__ __forceinline__ Cols cols_of(int slab, int lane, int cols) {
  const int col = slab * kSlab + lane * kVec;
  return {col, cols - col, cols >= kVec ? min(col, cols - kVec) : 0};
}

// A finished sum goes out. row: the token, or its place among the rows. A
// column that two lanes have gets the same value twice; an addition to what is
// there may happen once only, so there each lane keeps to its own columns.
template <typename G, int MODE>
__device__ __forceinline__ void put(const SumArgs& A, int64_t row, const Cols& l, const float (&acc)[kVec]) {
  if (l.nc <= 0) return;
  G* const p = static_cast<G*>(A.grad) + row * A.grad_ld + l.from;
  float x[kVec];
  if (MODE != kAdd) {
#pragma unroll
    for (int q = 0; q < kVec; ++q) x[q] = acc[q] * A.scale;
    store4_of(p, A.cols, x);
    return;
  }
  const int skip = l.col - l.from;
  if (skip == 0) {
    load4_of(p, A.cols, x);
#pragma unroll
    for (int q = 0; q < kVec; ++q) x[q] += acc[q] * A.scale;
    store4_of(p, A.cols, x);
    return;
  }
#pragma unroll
  for (int q = 0; q < kVec; ++q)
    if (q >= skip) muon_adam::PElem<G>::store(p, q, muon_adam::PElem<G>::load(p, q) + acc[q] * A.scale);
}

__device__ __forceinline__ void put_part(float* part, const SumArgs& A, int64_t chunk, const Cols& l, const float (&acc)[kVec]) {
  if (l.nc > 0) muon_adam::store4<false>(part + chunk * A.ld_part + l.from, acc);
}

// A row's four elements as they lie in memory.
template <typename D> struct Raw;
template <> struct Raw<float> {
  typedef muon_adam::f32x4 T;
  static constexpr int rows = 8;  // in one group of loads; two groups are in flight
  static __device__ __forceinline__ float get(const T& x, int q) { return x[q]; }
};
template <> struct Raw<uint16_t> {
  typedef muon_adam::u32x2 T;
  static constexpr int rows = 16;
  static __device__ __forceinline__ float get(const T& x, int q) {
    return __uint_as_float(q & 1 ? x[q >> 1] & 0xffff0000u : x[q >> 1] << 16);
  }
};

// Clears the rows of tokens that do not occur. They run beside the sums, not
// in the sort (which has the time that the batch's frequent tokens take, and
// no use for HBM).
template <typename G>
__device__ __forceinline__ void clear_rows(const SumArgs& A, int block, int lane) {
  const int r0 = (block * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * kClearRows;
  if (r0 >= A.vocab) return;
  const int r = min(r0 + lane, A.vocab - 1);
  const bool clear = lane < kClearRows && r0 + lane < A.vocab && A.present[r] == 0;
  const float zero[8] = {};
  for (uint64_t todo = __ballot(clear); todo; todo &= todo - 1) {
    G* const row = static_cast<G*>(A.grad) + int64_t(r0 + __builtin_ctzll(todo)) * A.grad_ld;
    for (int c = lane * 8; c < A.cols; c += 512) store8(row + c, A.cols - c, zero);
  }
}

// Bound by HBM where rows are whole cache lines: 32768 bf16 rows of 768 into a
// dense gradient (53 MB read, 78 written) 28 us, 4.7 TB/s; 65536 fp32 rows of
// 1024 (253 and 76 MB) 61 us, 5.4 TB/s. 15000 rows of 765 added to an fp32
// gradient (34 and 10 MB) take 26 us: rows of 1530 bytes at every alignment, and
// few tokens with many rows. dout is read once and past the caches (the two
// whole calls 61 -> 55 and 237 -> 225 us).
template <typename D, typename G, int MODE>
__global__ __launch_bounds__(kThreads) void embed_sum_kernel(SumArgs A) {
  const int lane = threadIdx.x & 63;
  if (MODE == kDense && int(blockIdx.x) >= A.sum_blocks) {
    clear_rows<G>(A, blockIdx.x - A.sum_blocks, lane);
    return;
  }
  const int64_t id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) + int64_t(blockIdx.x) * (kThreads / 64);
  if (MODE == kRows && id == 0) {  // (there is a block without tokens, too)
    const int total = distinct_in(A.distinct, 0, A.ranges, lane);
    if (lane == 0) *A.count = total;
  }
  const int64_t chunk = id / A.slabs;
  const int slab = static_cast<int>(id - chunk * A.slabs);
  const int64_t c0 = chunk * A.chunk;
  if (c0 >= A.n) return;
  // a chunk has at most 64 records: lane i has the i-th (those behind *live
  // are not set and not used; all are loaded at once)
  Rec mine = A.recs[min(c0 + lane, A.n - 1)];
  const int before = A.recs[c0 > 0 ? c0 - 1 : 0].key;
  const int live = __builtin_amdgcn_readfirstlane(*A.live);
  if (c0 >= live) return;
  const int len = static_cast<int>(min(int64_t(A.chunk), live - c0));
  const int c1 = static_cast<int>(c0) + len;
  const Cols l = cols_of(slab, lane, A.cols);
  if (lane >= len) {  // the last record again
    mine.pos = __builtin_amdgcn_readlane(mine.pos, len - 1);
    mine.key = __builtin_amdgcn_readlane(mine.key, len - 1);
    mine.slot = __builtin_amdgcn_readlane(mine.slot, len - 1);
  }
  int key = __builtin_amdgcn_readfirstlane(mine.key);
  // the first token's sum is a part if it began in an earlier chunk
  bool head = c0 > 0 && __builtin_amdgcn_readfirstlane(before) == key;
  int row = mine.key;  // where the lane's token goes
  if (MODE == kRows) {
    const int mine_in = mine.key / A.range;
    int base = 0, from = 0;
    for (uint64_t todo = ~uint64_t(0); todo;) {  // a range at a time
      const int r = __builtin_amdgcn_readlane(mine_in, __builtin_ctzll(todo));
      base += distinct_in(A.distinct, from, r, lane);
      from = r;
      if (mine_in == r) row = base + mine.slot;
      todo &= ~__ballot(mine_in == r);
    }
    // (the chunk that a token begins in)
    const int left = __shfl_up(mine.key, 1, 64);
    if (slab == 0 && lane < len && (lane > 0 ? left != mine.key : !head)) A.rows[row] = mine.key;
  }
  float acc[kVec] = {};
  int at = 0;  // a record of the current token
  auto flush = [&]() {
    if (head) put_part(A.head, A, chunk, l, acc);
    else put<G, MODE>(A, __builtin_amdgcn_readlane(row, at), l, acc);
    head = false;
#pragma unroll
    for (int q = 0; q < kVec; ++q) acc[q] = 0.f;
  };
  const D* const dout = static_cast<const D*>(A.dout) + l.from;
  typedef Raw<D> R;
  constexpr int U = R::rows;
  if (A.cols < kVec) {  // narrow rows
    for (int i = 0; i < len; ++i) {
      const int k = __builtin_amdgcn_readlane(mine.key, i);
      if (k != key) flush();
      key = k;
      at = i;
      float x[kVec];
      load4_of(dout + int64_t(__builtin_amdgcn_readlane(mine.pos, i)) * A.dout_ld, A.cols, x);
#pragma unroll
      for (int q = 0; q < kVec; ++q) acc[q] += x[q];
    }
  } else {
    // The next group of rows is fetched before the last one is added up, with
    // no branch around a load (behind the chunk's end the last row again), so
    // that the waits for a group need not count those of the next.
    auto fetch = [&](int i0, typename R::T (&x)[U]) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        x[u] = __builtin_nontemporal_load(reinterpret_cast<const typename R::T*>(dout + int64_t(__builtin_amdgcn_readlane(mine.pos, min(i0 + u, len - 1))) * A.dout_ld));
    };
    auto add = [&](int i0, const typename R::T (&x)[U]) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i0 + u >= len) break;
        const int k = __builtin_amdgcn_readlane(mine.key, i0 + u);
        if (k != key) flush();
        key = k;
        at = i0 + u;
#pragma unroll
        for (int q = 0; q < kVec; ++q) acc[q] += R::get(x[u], q);
      }
    };
    typename R::T x[U], y[U];
    fetch(0, x);
    if (A.chunk <= U) {
      add(0, x);
    } else for (int i0 = 0; i0 < len; i0 += 2 * U) {
      fetch(i0 + U, y);
      add(i0, x);
      fetch(i0 + 2 * U, x);
      add(i0 + U, y);
    }
  }
  if (!head && __builtin_amdgcn_readlane(mine.end, at) > c1) put_part(A.tail, A, chunk, l, acc);
  else flush();
}

// A token that crosses chunks: its first part, then one part of every later
// chunk it reaches. Block (chunk, slab); the waves take the later parts in
// turn, and their sums are added in order, in float64: a token may have 2^18
// parts, and a float32 sum that has outgrown them rounds each the same way (2^22
// equal rows: off by 1.5e-4, in float64 by 6e-7, which is the runs' own; whole
// calls 55.5 and 223 us with either). 5 to 8 us, most of it the latency of
// finding out which block has something to add and of its few loads.
template <typename G, int MODE>
__global__ __launch_bounds__(kThreads) void embed_join_kernel(SumArgs A) {
  __shared__ double red[kThreads / 64 - 1][kVec][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t chunk = blockIdx.x / A.slabs;
  const int slab = static_cast<int>(blockIdx.x - chunk * A.slabs);
  const int64_t c0 = chunk * A.chunk, c1 = c0 + A.chunk;
  if (c1 >= A.n) return;
  const Rec r = A.recs[c1 - 1];
  const int before = A.recs[c0 > 0 ? c0 - 1 : 0].key;
  if (c1 >= *A.live) return;  // the last chunk: nothing goes on behind it
  if (r.end <= c1) return;
  if (c0 > 0 && before == r.key) return;  // began before this chunk: another block's
  const Cols l = cols_of(slab, lane, A.cols);
  const int64_t stop = (r.end - 1) / A.chunk;  // the last chunk it reaches
  double acc[kVec] = {};
  constexpr int W = kThreads / 64, U = 8;
  if (l.nc > 0) {
    if (wave == 0) {
      float x[kVec];
      muon_adam::load4<false>(A.tail + chunk * A.ld_part + l.from, x);
#pragma unroll
      for (int q = 0; q < kVec; ++q) acc[q] = double(x[q]);
    }
    for (int64_t j0 = chunk + 1 + wave; j0 <= stop; j0 += W * U) {
      float x[U][kVec];
#pragma unroll
      for (int u = 0; u < U; ++u) muon_adam::load4<false>(A.head + min(j0 + u * W, stop) * A.ld_part + l.from, x[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (j0 + u * W > stop) break;
#pragma unroll
        for (int q = 0; q < kVec; ++q) acc[q] += double(x[u][q]);
      }
    }
  }
  if (wave > 0)
#pragma unroll
    for (int q = 0; q < kVec; ++q) red[wave - 1][q][lane] = acc[q];
  __syncthreads();
  if (wave > 0) return;
  float sum[kVec];
#pragma unroll
  for (int q = 0; q < kVec; ++q) {
#pragma unroll
    for (int w = 0; w < W - 1; ++w) acc[q] += red[w][q][lane];
    sum[q] = static_cast<float>(acc[q]);
  }
  int64_t row = r.key;
  if (MODE == kRows) row = distinct_in(A.distinct, 0, r.key / A.range, lane) + r.slot;
  put<G, MODE>(A, row, l, sum);
}

// ------------------------------------------------------------ Adam on rows

struct RowArgs {
  void* table;
  float* m;
  float* v;
  int64_t ld;
  const int32_t* rows;
  const void* values;
  const int32_t* count;
  const float* gscale;
  int64_t capacity;
  int32_t vocab, cols;
  int32_t vpr;      // vectors of four in a row
  uint32_t magic;   // for divisions by vpr
  int32_t per;      // rows of a block's turn
  muon_adam::Consts k;
};

// Bound by HBM: the fp32 rows of a batch of 65536 tokens, width 1024 (294 MB read,
// 220 written) 99 us, 5.2 TB/s; bf16 ones of 8192 tokens, width 768, 14 us.
template <typename T>
__global__ __launch_bounds__(kThreads) void embed_adam_kernel(RowArgs A) {
  muon_adam::Consts k = A.k;
  k.gs = A.gscale ? *A.gscale : 1.f;
  const int64_t count = min(int64_t(*A.count), A.capacity);
  const uint32_t vpr = static_cast<uint32_t>(A.vpr);
  for (int64_t r0 = int64_t(blockIdx.x) * A.per; r0 < count; r0 += int64_t(gridDim.x) * A.per) {
    const uint32_t nv = vpr * static_cast<uint32_t>(min(count - r0, int64_t(A.per)));
    for (uint32_t i = threadIdx.x; i < nv; i += kThreads) {
      const uint32_t r = div_by(i, vpr, A.magic);
      const int c = static_cast<int>(i - r * vpr) * kVec, nc = A.cols - c;
      const int32_t id = A.rows[r0 + r];
      if (static_cast<uint32_t>(id) >= static_cast<uint32_t>(A.vocab)) continue;
      T* const p = static_cast<T*>(A.table) + int64_t(id) * A.ld + c;
      float* const m = A.m + int64_t(id) * A.cols + c;
      float* const v = A.v + int64_t(id) * A.cols + c;
      muon_adam::Vec4 x;
      load4_of(p, nc, x.p);
      load4_of(static_cast<const T*>(A.values) + (r0 + r) * A.cols + c, nc, x.g);
      load4_of(m, nc, x.m);
      load4_of(v, nc, x.v);
#pragma unroll
      for (int q = 0; q < kVec; ++q) x.p[q] = muon_adam::adam_elem(x.p[q], x.g[q], x.m[q], x.v[q], k);
      store4_of(m, nc, x.m);
      store4_of(v, nc, x.v);
      store4_of(p, nc, x.p);
    }
  }
}

// ------------------------------------------------------------------- host

int64_t size_of(int32_t dtype) { return dtype == MUON_F32 ? 4 : 2; }

struct Sizes {
  int32_t range, ranges;  // sort: entries of a range, ranges
  int32_t segments, run;  // segments of the batch, tokens of a wave in one
  int32_t chunk, chunks;  // sum: records of a chunk, chunks
  int32_t slabs;
  int64_t ld_part;
  size_t recs, distinct, live, present, head, tail, total;  // byte offsets, and the whole
};

// Sort: a block per CU, ranges times segments of the batch. Segments split the
// work of ranges with many tokens (but all blocks read all tokens), so there
// are as many as leave each kSegment tokens and fit beside the ranges, whose
// length the counters in LDS limit (with segments of 2048, 4096 and 8192 tokens
// the gradient of 32768 tokens of 50257 takes 57, 55 and 59 us, that of 30011
// of 5003 47.5, 49 and 51, rows of 8192 47, 47 and 51). Sum: chunks short enough
// that chunks and slabs give every CU a few waves, of at least 4 and at most 64
// records (a lane each). With 2048, 4096 and 8192 waves the same three take 57,
// 55 and 55, 62, 49 and 43, and 47, 47 and 54 us, rows of 65536 223, 223 and 228:
// more waves suit a dense gradient of few, frequent tokens, and cost the row
// form, whose waves each look for their place among the distinct tokens. Both
// forms use the same number, and give the same bits.
Sizes sizes_of(int64_t vocab, int64_t cols, int64_t n) {
  Sizes s{};
  const int64_t least = (vocab + kMaxRange - 1) / kMaxRange;
  const int64_t segments = std::max<int64_t>(1, std::min(n / kSegment, kSortBlocks / least));
  const int64_t wanted = std::max<int64_t>(least, kSortBlocks / segments);
  s.range = static_cast<int32_t>((vocab + wanted - 1) / wanted);
  s.ranges = static_cast<int32_t>((vocab + s.range - 1) / s.range);
  const int64_t unit = segments * kSortThreads;  // a multiple of 64 tokens for every wave
  s.run = static_cast<int32_t>((n + unit - 1) / unit * 64);
  s.segments = static_cast<int32_t>(segments);
  s.slabs = static_cast<int32_t>((cols + kSlab - 1) / kSlab);
  int64_t chunk = 4;
  while (chunk < 64 && (n + chunk - 1) / chunk * s.slabs > kSumWaves) chunk *= 2;
  s.chunk = static_cast<int32_t>(chunk);
  s.chunks = static_cast<int32_t>((n + chunk - 1) / chunk);
  s.ld_part = (cols + kVec - 1) / kVec * kVec;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  // room for the chunks of any batch up to n (shorter batches may have more of them)
  const int64_t most = std::min((n + 3) / 4, std::max((n + 63) / 64, kSumWaves / s.slabs + int64_t(1)));
  const size_t part = up(size_t(most) * size_t(s.ld_part) * sizeof(float));
  s.recs = 0;
  s.distinct = s.recs + up(size_t(n) * sizeof(Rec));
  s.live = s.distinct + up(size_t(std::max<int64_t>(least, kSortBlocks)) * sizeof(int32_t));
  s.present = s.live + 256;
  s.head = s.present + up(size_t(vocab));
  s.tail = s.head + part;
  s.total = s.tail + part;
  return s;
}

uint32_t magic_of(int64_t d) { return static_cast<uint32_t>(UINT32_MAX / static_cast<uint64_t>(d)); }

// Byte ranges of a call; true if a written one meets another.
struct Spans {
  struct Span {
    uintptr_t lo, hi;
    bool write;
  } s[10];
  int n = 0;
  bool wraps = false;
  void add(const void* p, int64_t bytes, bool write) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (bytes <= 0 || p == nullptr) return;
    if (lo > UINTPTR_MAX - static_cast<uintptr_t>(bytes)) wraps = true;
    s[n++] = {lo, lo + static_cast<uintptr_t>(bytes), write};
  }
  bool meet() const {
    if (wraps) return true;
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < i; ++j)
        if ((s[i].write || s[j].write) && s[i].lo < s[j].hi && s[j].lo < s[i].hi) return true;
    return false;
  }
};

int64_t span_of(int64_t rows, int64_t ld, int64_t cols, int64_t es) { return rows > 0 ? ((rows - 1) * ld + cols) * es : 0; }

muon_status check_sizes(int64_t vocab, int64_t cols, int64_t max_tokens) {
  if (vocab < 1 || vocab > MUON_EMBED_MAX_VOCAB || cols < 1 || cols > MUON_EMBED_MAX_COLS || max_tokens < 0 ||
      max_tokens > MUON_EMBED_MAX_TOKENS)
    return MUON_E_SHAPE;
  if ((max_tokens + 63) / 64 * ((cols + kSlab - 1) / kSlab) > kMaxWaves) return MUON_E_SHAPE;
  return MUON_OK;
}

}  // namespace muon_embed

struct muon_embed_plan_s {
  int device = -1;
  muon_dtype dtype = MUON_BF16;
  muon_embed_table t{};
  int64_t max_tokens = 0;
  const float* gscale = nullptr;
};

namespace {

using namespace muon_embed;

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

muon_status check_tokens(const muon_embed_plan* p, const muon_embed_tokens* t) {
  if (t == nullptr) return MUON_E_INVALID;
  if (t->reserved != 0 || (t->wide != 0 && t->wide != 1)) return MUON_E_INVALID;
  if (t->n < 0 || t->n > p->max_tokens) return MUON_E_SHAPE;
  if (t->n > 0 && t->data == nullptr) return MUON_E_INVALID;
  return misaligned(t->data, t->wide ? 8 : 4) ? MUON_E_ALIGN : MUON_OK;
}

muon_status check_acts(const muon_embed_plan* p, const muon_embed_acts* a, int64_t n) {
  if (a == nullptr || a->reserved != 0) return MUON_E_INVALID;
  if (a->dtype != MUON_F32 && a->dtype != MUON_BF16) return MUON_E_DTYPE;
  if (n == 0) return MUON_OK;
  if (a->ld < p->t.cols || a->ld > MUON_EMBED_MAX_LD) return MUON_E_SHAPE;
  if (a->data == nullptr) return MUON_E_INVALID;
  return misaligned(a->data, size_t(size_of(a->dtype))) ? MUON_E_ALIGN : MUON_OK;
}

void add_table(const muon_embed_plan* p, Spans* s) {
  s->add(p->t.table, span_of(p->t.vocab, p->t.ld, p->t.cols, size_of(p->dtype)), false);
  s->add(p->t.exp_avg, p->t.vocab * p->t.cols * 4, false);
  s->add(p->t.exp_avg_sq, p->t.vocab * p->t.cols * 4, false);
}

bool on_device(const muon_embed_plan* p) {
  int dev = -1;
  return hipGetDevice(&dev) == hipSuccess && dev == p->device;
}

muon_status launched() { return hipGetLastError() == hipSuccess ? MUON_OK : MUON_E_LAUNCH; }

template <typename E, typename O>
void launch_lookup(const LookArgs& a, bool wide, unsigned grid, hipStream_t s) {
  if (wide) hipLaunchKernelGGL((embed_lookup_kernel<E, O, int64_t>), dim3(grid), dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((embed_lookup_kernel<E, O, int32_t>), dim3(grid), dim3(kThreads), 0, s, a);
}

template <typename D, typename G, int MODE>
muon_status launch_sum(const SumArgs& a, hipStream_t s) {
  const int64_t waves = int64_t(a.chunks) * a.slabs;
  constexpr int each = kThreads / 64, rows = each * kClearRows;
  SumArgs b = a;
  b.sum_blocks = static_cast<int32_t>(std::max<int64_t>(MODE == kRows ? 1 : 0, (waves + each - 1) / each));
  const int64_t clear = MODE == kDense ? (int64_t(a.vocab) + rows - 1) / rows : 0;
  hipLaunchKernelGGL((embed_sum_kernel<D, G, MODE>), dim3(unsigned(b.sum_blocks + clear)), dim3(kThreads), 0, s, b);
  muon_status st = launched();
  if (st != MUON_OK || a.chunks < 2) return st;
  hipLaunchKernelGGL((embed_join_kernel<G, MODE>), dim3(unsigned(waves)), dim3(kThreads), 0, s, a);
  return launched();
}

template <int MODE>
muon_status launch_sum(const SumArgs& a, int32_t dout, muon_dtype grad, hipStream_t s) {
  if (dout == MUON_F32) return grad == MUON_F32 ? launch_sum<float, float, MODE>(a, s) : launch_sum<float, uint16_t, MODE>(a, s);
  return grad == MUON_F32 ? launch_sum<uint16_t, float, MODE>(a, s) : launch_sum<uint16_t, uint16_t, MODE>(a, s);
}

muon_status run_gradient(muon_embed_plan* p, const muon_embed_tokens* tokens, const muon_embed_acts* dout, float scale,
                         void* grad, int64_t grad_ld, int mode, int32_t* rows, int32_t* count, void* ws, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const Sizes z = sizes_of(p->t.vocab, p->t.cols, tokens->n);
  char* const w = static_cast<char*>(ws);
  SortArgs a{};
  a.tokens = tokens->data;
  a.recs = reinterpret_cast<Rec*>(w + z.recs);
  a.distinct = reinterpret_cast<int32_t*>(w + z.distinct);
  a.live = reinterpret_cast<int32_t*>(w + z.live);
  a.present = mode == kDense ? reinterpret_cast<uint8_t*>(w + z.present) : nullptr;
  a.n = static_cast<int32_t>(tokens->n);
  a.vocab = static_cast<int32_t>(p->t.vocab);
  a.range = z.range;
  a.segments = z.segments;
  a.run = z.run;
  while ((1 << a.bits) < z.range) ++a.bits;
  const size_t lds = (size_t(kSortWaves + 2) * size_t(z.range) + 3) / 4 * 16;  // cleared 16 bytes at a time
  if (tokens->wide)
    hipLaunchKernelGGL(embed_sort_kernel<int64_t>, dim3(unsigned(z.ranges * z.segments)), dim3(kSortThreads), lds, s, a);
  else
    hipLaunchKernelGGL(embed_sort_kernel<int32_t>, dim3(unsigned(z.ranges * z.segments)), dim3(kSortThreads), lds, s, a);
  muon_status st = launched();
  if (st != MUON_OK) return st;
  SumArgs b{};
  b.recs = a.recs;
  b.distinct = a.distinct;
  b.live = a.live;
  b.dout = dout->data;
  b.dout_ld = dout->ld;
  b.grad = grad;
  b.grad_ld = grad_ld;
  b.rows = rows;
  b.count = count;
  b.head = reinterpret_cast<float*>(w + z.head);
  b.tail = reinterpret_cast<float*>(w + z.tail);
  b.ld_part = z.ld_part;
  b.n = tokens->n;
  b.present = a.present;
  b.vocab = a.vocab;
  b.cols = static_cast<int32_t>(p->t.cols);
  b.slabs = z.slabs;
  b.chunk = z.chunk;
  b.chunks = z.chunks;
  b.range = z.range;
  b.ranges = z.ranges;
  b.scale = scale;
  if (mode == kAdd && tokens->n == 0) return MUON_OK;
  if (mode == kDense) return launch_sum<kDense>(b, dout->dtype, p->dtype, s);
  if (mode == kAdd) return launch_sum<kAdd>(b, dout->dtype, p->dtype, s);
  return launch_sum<kRows>(b, dout->dtype, p->dtype, s);
}

}  // namespace

extern "C" {

muon_status muon_embed_workspace_bytes(int64_t vocab, int64_t cols, int64_t max_tokens, size_t* bytes) {
  if (bytes == nullptr) return MUON_E_INVALID;
  const muon_status st = check_sizes(vocab, cols, max_tokens);
  if (st != MUON_OK) return st;
  *bytes = sizes_of(vocab, cols, max_tokens).total;
  return MUON_OK;
}

muon_status muon_embed_plan_create(const muon_embed_table* table, muon_dtype dtype, int64_t max_tokens,
                                   muon_embed_plan** plan) {
  if (plan == nullptr) return MUON_E_INVALID;
  *plan = nullptr;
  if (table == nullptr) return MUON_E_INVALID;
  if (dtype != MUON_F32 && dtype != MUON_BF16) return MUON_E_DTYPE;
  muon_status st = check_sizes(table->vocab, table->cols, max_tokens);
  if (st != MUON_OK) return st;
  if (table->ld < table->cols || table->ld > MUON_EMBED_MAX_LD) return MUON_E_SHAPE;
  if (table->table == nullptr || (table->exp_avg == nullptr) != (table->exp_avg_sq == nullptr)) return MUON_E_INVALID;
  if (!std::isfinite(table->lr_mul) || !std::isfinite(table->wd_mul)) return MUON_E_INVALID;
  if (misaligned(table->table, size_t(size_of(dtype))) || misaligned(table->exp_avg, 4) ||
      misaligned(table->exp_avg_sq, 4))
    return MUON_E_ALIGN;
  Spans sp;
  sp.add(table->table, span_of(table->vocab, table->ld, table->cols, size_of(dtype)), true);
  sp.add(table->exp_avg, table->vocab * table->cols * 4, true);
  sp.add(table->exp_avg_sq, table->vocab * table->cols * 4, true);
  if (sp.meet()) return MUON_E_INVALID;
  int dev = 0;
  hipDeviceProp_t prop;
  if (hipGetDevice(&dev) != hipSuccess || hipGetDeviceProperties(&prop, dev) != hipSuccess ||
      std::strncmp(prop.gcnArchName, "gfx950", 6) != 0)
    return MUON_E_DEVICE;
  muon_embed_plan_s* p = new (std::nothrow) muon_embed_plan_s();
  if (!p) return MUON_E_ALLOC;
  p->device = dev;
  p->dtype = dtype;
  p->t = *table;
  p->max_tokens = max_tokens;
  *plan = p;
  return MUON_OK;
}

muon_status muon_embed_plan_lookup(muon_embed_plan* plan, const muon_embed_tokens* tokens, float scale,
                                   const muon_embed_acts* out, void* stream) {
  if (plan == nullptr || !std::isfinite(scale)) return MUON_E_INVALID;
  muon_status st = check_tokens(plan, tokens);
  if (st != MUON_OK) return st;
  const int64_t n = tokens->n;
  if ((st = check_acts(plan, out, n)) != MUON_OK) return st;
  if (n == 0) return MUON_OK;
  Spans sp;
  add_table(plan, &sp);
  sp.add(tokens->data, n * (tokens->wide ? 8 : 4), false);
  sp.add(out->data, span_of(n, out->ld, plan->t.cols, size_of(out->dtype)), true);
  if (sp.meet()) return MUON_E_INVALID;
  if (!on_device(plan)) return MUON_E_DEVICE;
  LookArgs a{};
  a.table = plan->t.table;
  a.tokens = tokens->data;
  a.out = out->data;
  a.ld = plan->t.ld;
  a.out_ld = out->ld;
  a.n = n;
  a.vocab = static_cast<int32_t>(plan->t.vocab);
  a.cols = static_cast<int32_t>(plan->t.cols);
  const LookGrid look = lookup_grid(plan->t.cols, n);
  a.vpr = static_cast<int32_t>(look.vpr);
  a.magic = magic_of(a.vpr);
  a.per = static_cast<int32_t>(look.per);
  a.scale = scale;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const unsigned grid = unsigned(look.blocks);
  const bool w = tokens->wide != 0, f = plan->dtype == MUON_F32, of = out->dtype == MUON_F32;
  if (f && of) launch_lookup<float, float>(a, w, grid, s);
  else if (f) launch_lookup<float, uint16_t>(a, w, grid, s);
  else if (of) launch_lookup<uint16_t, float>(a, w, grid, s);
  else launch_lookup<uint16_t, uint16_t>(a, w, grid, s);
  return launched();
}

muon_status muon_embed_plan_gradient(muon_embed_plan* plan, const muon_embed_tokens* tokens, const muon_embed_acts* dout,
                                     float scale, void* grad, int64_t grad_ld, int32_t accumulate, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  if (plan == nullptr || !std::isfinite(scale) || grad == nullptr || (accumulate != 0 && accumulate != 1))
    return MUON_E_INVALID;
  muon_status st = check_tokens(plan, tokens);
  if (st != MUON_OK) return st;
  const int64_t n = tokens->n, es = size_of(plan->dtype);
  if ((st = check_acts(plan, dout, n)) != MUON_OK) return st;
  if (grad_ld < plan->t.cols || grad_ld > MUON_EMBED_MAX_LD) return MUON_E_SHAPE;
  if (misaligned(grad, size_t(es))) return MUON_E_ALIGN;
  if (workspace == nullptr || misaligned(workspace, 256) ||
      workspace_bytes < sizes_of(plan->t.vocab, plan->t.cols, n).total)
    return MUON_E_WORKSPACE;
  Spans sp;
  add_table(plan, &sp);
  sp.add(tokens->data, n * (tokens->wide ? 8 : 4), false);
  sp.add(dout->data, span_of(n, dout->ld, plan->t.cols, size_of(dout->dtype)), false);
  sp.add(grad, span_of(plan->t.vocab, grad_ld, plan->t.cols, es), true);
  sp.add(workspace, int64_t(sizes_of(plan->t.vocab, plan->t.cols, n).total), true);
  if (sp.meet()) return MUON_E_INVALID;
  if (n == 0 && accumulate) return MUON_OK;
  if (!on_device(plan)) return MUON_E_DEVICE;
  return run_gradient(plan, tokens, dout, scale, grad, grad_ld, accumulate ? kAdd : kDense, nullptr, nullptr, workspace, stream);
}

muon_status muon_embed_plan_gradient_rows(muon_embed_plan* plan, const muon_embed_tokens* tokens,
                                          const muon_embed_acts* dout, float scale, int32_t* rows, void* values,
                                          int32_t* count, void* workspace, size_t workspace_bytes, void* stream) {
  if (plan == nullptr || !std::isfinite(scale) || count == nullptr) return MUON_E_INVALID;
  muon_status st = check_tokens(plan, tokens);
  if (st != MUON_OK) return st;
  const int64_t n = tokens->n, es = size_of(plan->dtype), cap = std::min(n, plan->t.vocab);
  if ((st = check_acts(plan, dout, n)) != MUON_OK) return st;
  if (n > 0 && (rows == nullptr || values == nullptr)) return MUON_E_INVALID;
  if (misaligned(rows, 4) || misaligned(count, 4) || misaligned(values, size_t(es))) return MUON_E_ALIGN;
  if (workspace == nullptr || misaligned(workspace, 256) ||
      workspace_bytes < sizes_of(plan->t.vocab, plan->t.cols, n).total)
    return MUON_E_WORKSPACE;
  Spans sp;
  add_table(plan, &sp);
  sp.add(tokens->data, n * (tokens->wide ? 8 : 4), false);
  sp.add(dout->data, span_of(n, dout->ld, plan->t.cols, size_of(dout->dtype)), false);
  sp.add(rows, cap * 4, true);
  sp.add(values, cap * plan->t.cols * es, true);
  sp.add(count, 4, true);
  sp.add(workspace, int64_t(sizes_of(plan->t.vocab, plan->t.cols, n).total), true);
  if (sp.meet()) return MUON_E_INVALID;
  if (!on_device(plan)) return MUON_E_DEVICE;
  return run_gradient(plan, tokens, dout, scale, values, plan->t.cols, kRows, rows, count, workspace, stream);
}

muon_status muon_embed_plan_adam_rows(muon_embed_plan* plan, const muon_adam_config* cfg, const int32_t* rows,
                                      const void* values, const int32_t* count, int64_t capacity, void* stream) {
  if (plan == nullptr || cfg == nullptr || count == nullptr) return MUON_E_INVALID;
  if (!std::isfinite(cfg->lr) || !std::isfinite(cfg->beta1) || !std::isfinite(cfg->beta2) || !std::isfinite(cfg->eps) ||
      !std::isfinite(cfg->wd))
    return MUON_E_INVALID;
  if (cfg->beta1 < 0.f || cfg->beta1 >= 1.f || cfg->beta2 < 0.f || cfg->beta2 >= 1.f || cfg->eps < 0.f || cfg->step < 1)
    return MUON_E_INVALID;
  if (plan->t.exp_avg == nullptr) return MUON_E_INVALID;
  if (capacity < 0 || capacity > plan->t.vocab) return MUON_E_SHAPE;
  const int64_t es = size_of(plan->dtype);
  if (capacity > 0 && (rows == nullptr || values == nullptr)) return MUON_E_INVALID;
  if (misaligned(rows, 4) || misaligned(count, 4) || misaligned(values, size_t(es))) return MUON_E_ALIGN;
  Spans sp;
  const muon_embed_table& t = plan->t;
  sp.add(t.table, span_of(t.vocab, t.ld, t.cols, es), true);
  sp.add(t.exp_avg, t.vocab * t.cols * 4, true);
  sp.add(t.exp_avg_sq, t.vocab * t.cols * 4, true);
  sp.add(rows, capacity * 4, false);
  sp.add(values, capacity * t.cols * es, false);
  sp.add(count, 4, false);
  if (sp.meet()) return MUON_E_INVALID;
  if (capacity == 0) return MUON_OK;
  if (!on_device(plan)) return MUON_E_DEVICE;
  RowArgs a{};
  a.table = t.table;
  a.m = t.exp_avg;
  a.v = t.exp_avg_sq;
  a.ld = t.ld;
  a.rows = rows;
  a.values = values;
  a.count = count;
  a.gscale = plan->gscale;
  a.capacity = capacity;
  a.vocab = static_cast<int32_t>(t.vocab);
  a.cols = static_cast<int32_t>(t.cols);
  a.vpr = static_cast<int32_t>((t.cols + kVec - 1) / kVec);
  a.magic = magic_of(a.vpr);
  a.per = std::max(1, 2 * kThreads / a.vpr);
  // the scalars of muon_adam_plan_step
  const float lr = cfg->lr * t.lr_mul;
  a.k.b1 = cfg->beta1;
  a.k.c1 = 1.f - cfg->beta1;
  a.k.b2 = cfg->beta2;
  a.k.c2 = 1.f - cfg->beta2;
  a.k.eps = cfg->eps;
  a.k.keep = 1.f - lr * (cfg->wd * t.wd_mul);
  a.k.step = lr * static_cast<float>(1.0 / (1.0 - std::pow(double(cfg->beta1), double(cfg->step))));
  a.k.isb2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(double(cfg->beta2), double(cfg->step))));
  a.k.gs = 1.f;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const unsigned grid = unsigned(std::min<int64_t>((capacity + a.per - 1) / a.per, 8192));
  if (plan->dtype == MUON_F32) hipLaunchKernelGGL(embed_adam_kernel<float>, dim3(grid), dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL(embed_adam_kernel<uint16_t>, dim3(grid), dim3(kThreads), 0, s, a);
  return launched();
}

muon_status muon_embed_plan_set_grad_scale(muon_embed_plan* plan, const float* scale) {
  if (plan == nullptr) return MUON_E_INVALID;
  if (misaligned(scale, 4)) return MUON_E_ALIGN;
  plan->gscale = scale;
  return MUON_OK;
}

void muon_embed_plan_destroy(muon_embed_plan* plan) { delete plan; }

}  // extern "C"
