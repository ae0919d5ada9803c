// Global gradient norm and clipping (include/muon_clip.h): the kernels, the
// plan (validated list split into work items in device memory) and the C ABI.
//
//   N = c sqrt(sum of squares of every element of every tensor)
//   factor = c min(1, max_norm / (N + eps));  out = g factor
//
// The norm reads every gradient once (2 or 4 bytes an element, two flops) and
// is bound by HBM, or by the launches for small lists. One wave takes one
// work item, a run of consecutive elements (or of rows of a strided tensor)
// of one tensor; squares are summed in float64, where a bf16 or fp32 square
// neither over- nor underflows, so no scaling by a maximum is needed.
// (Float32 sums would save next to nothing: 59.6 against 60.7 us on the 328 MB
// below when both were tried.) Partial sums go to fixed slots of the
// workspace and are added in a fixed order: no atomics, equal inputs give
// equal bits.
//
// Launches: one for lists of up to 64 KB; otherwise the norm's partial sums,
// then either their total (norm only) or the scaling, whose blocks each add
// the partials up for themselves.
//
// Measured on one MI355X: norm of the 124 M gradients of a GPT-2 (85 M bf16,
// 39.5 M fp32, 328 MB) with every tensor's norm 53 us (6.2 TB/s); of 2.15 GB
// 325 us (6.6 TB/s, the rate of the best plain copy kernel); norm and scaling
// of the 328 MB into other buffers 153 us (984 MB moved, 6.4 TB/s); 1.2 GB in
// place 194 us when not clipped, 643 us when clipped; 64 KB 3.6 and 5.6 us.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include "../../include/muon_clip.h"

namespace muon_clip {

constexpr int kWaves = 4;                 // work items (one per wave) of a block
constexpr int kThreads = 64 * kWaves;
constexpr int64_t kMinBytes = 4096;       // smallest work item
constexpr int64_t kMaxBytes = 1 << 28;    // largest (its element count fits an int32)
// 32 waves on each of the 256 CUs, all resident at once. Half as many: 1.2 GB
// in place 201 us for 192; twice as many: 328 MB norm 55.4 us for 53.6 (more
// partials to add up).
constexpr int64_t kTargetItems = 8192;
constexpr int kReduced = 1024;            // partials of a long list are first added up to this many
constexpr int kWide = 512;                // tensors of more items get a block for their norm, others a wave
constexpr int kSmall = 16;                // lists of at most this many items run in one block, a wave each
// A norm reads past the caches (non-temporal: 53 us for 328 MB, 60.6 with
// plain loads), except the last 256 MB of a clipping call, the size of the
// last-level cache, where the scaling finds some of them again (328 MB clipped: 152 us,
// 172 when all are read past the caches; 1.2 GB in place: 193 and 191 us).
constexpr int64_t kKeepBytes = 256 << 20;

// One wave's work: `rows` rows of `n` consecutive elements.
struct Item {
  const char* g;
  char* o;
  int64_t ld, out_ld;  // elements
  int32_t n, rows;
  int32_t dtype;       // muon_dtype
  uint32_t magic;      // rows > 1: (2^32 - 1) / vectors in a row, see div_row
};

struct Range {
  int32_t beg, end;  // work items of a tensor
};

struct Args {
  const Item* items;
  int32_t n_items;
  int32_t n_stream;    // the norm reads the first n_stream items past the caches
  int32_t n_part;      // block sums in `part`
  double* part;        // one sum per block of the norm kernel
  double* isum;        // one sum per item (nullptr: not wanted)
  const Range* ranges; // items of each tensor
  int32_t n_tensors;
  const int32_t* wide; // tensors of more than kWide items
  int32_t n_wide;
  float* norms;        // nullptr: not wanted
  muon_clip_result* res;
  float max_norm, eps, mul;
};

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
// 16-byte accesses at an element's alignment (the hardware takes any)
typedef f32x4 f32x4_u __attribute__((aligned(4)));
typedef u32x4 u32x4_u __attribute__((aligned(2)));

// Element types: V elements to a 16-byte vector.
struct F32 {
  typedef float T;
  typedef f32x4 Vec;
  typedef f32x4_u VecU;
  static constexpr int V = 4;
  static __device__ __forceinline__ float get(const Vec& x, int e) { return x[e]; }
  static __device__ __forceinline__ float load(const T* p) { return *p; }
  static __device__ __forceinline__ void store(T* p, float x) { *p = x; }
  static __device__ __forceinline__ Vec scale(const Vec& x, float s) { return x * s; }
};
struct Bf16 {
  typedef uint16_t T;
  typedef u32x4 Vec;
  typedef u32x4_u VecU;
  static constexpr int V = 8;
  static __device__ __forceinline__ float get(const Vec& x, int e) {
    return __uint_as_float(e & 1 ? x[e >> 1] & 0xffff0000u : x[e >> 1] << 16);
  }
  static __device__ __forceinline__ float load(const T* p) { return __uint_as_float(uint32_t(*p) << 16); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {  // round to nearest even
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
  }
  static __device__ __forceinline__ void store(T* p, float x) { *p = static_cast<T>(pack(x, 0.f)); }
  static __device__ __forceinline__ Vec scale(const Vec& x, float s) {
    Vec y;
#pragma unroll
    for (int q = 0; q < 4; ++q) y[q] = pack(get(x, 2 * q) * s, get(x, 2 * q + 1) * s);
    return y;
  }
};

// One vector at an element's alignment; NT: not kept in the caches. Clipped
// gradients are stored non-temporal (328 MB clipped: 153 us, 196 with plain
// stores; 57 MB of strided rows 37 and 43 us).
template <typename E, bool NT>
__device__ __forceinline__ typename E::Vec load_vec(const typename E::T* p) {
  const typename E::VecU* q = reinterpret_cast<const typename E::VecU*>(p);
  if constexpr (NT) return __builtin_nontemporal_load(q);
  else return *q;
}
template <typename E>
__device__ __forceinline__ void store_vec(typename E::T* p, const typename E::Vec& x) {
  const typename E::VecU y = x;
  __builtin_nontemporal_store(y, reinterpret_cast<typename E::VecU*>(p));
}

__device__ __forceinline__ double sq(float x) { return double(x) * double(x); }

// Adds one vector's squares. The barrier keeps the scheduler from converting
// several vectors ahead: 64 float64 values in flight would take 138 registers
// and leave room for three waves on a SIMD instead of eight (norm of 57 MB of
// strided rows: 23.9 us for 13.4).
template <typename E>
__device__ __forceinline__ void add_vec(const typename E::Vec& x, double& a, double& b) {
#pragma unroll
  for (int e = 0; e < E::V; e += 2) {
    a += sq(E::get(x, e));
    b += sq(E::get(x, e + 1));
  }
  __builtin_amdgcn_sched_barrier(0);
}

// Elements before the first 16-byte boundary at or after p, at most n.
template <typename E>
__device__ __forceinline__ int head_of(const typename E::T* p, int n) {
  const int h = static_cast<int>(-reinterpret_cast<uintptr_t>(p) & 15) / static_cast<int>(sizeof(typename E::T));
  return h < n ? h : n;
}

// A lane's share of the sum of squares of n consecutive elements.
template <typename E, bool NT>
__device__ __forceinline__ double ssq_run(const typename E::T* p, int n, int lane) {
  double a = 0.0, b = 0.0;
  const int head = head_of<E>(p, n);
  if (lane < head) a = sq(E::load(p + lane));
  p += head;
  n -= head;
  const int nv = n / E::V;
  constexpr int U = 8;
  int k = lane;
#pragma unroll 1
  for (; k + 64 * (U - 1) < nv; k += 64 * U) {
    typename E::Vec x[U];
#pragma unroll
    for (int j = 0; j < U; ++j) x[j] = load_vec<E, NT>(p + int64_t(k + 64 * j) * E::V);
#pragma unroll
    for (int j = 0; j < U; ++j) add_vec<E>(x[j], a, b);
  }
#pragma unroll 1
  for (; k < nv; k += 64) {
    const typename E::Vec x = load_vec<E, NT>(p + int64_t(k) * E::V);
    add_vec<E>(x, a, b);
  }
  const int t = nv * E::V + lane;
  if (t < n) b += sq(E::load(p + t));
  return a + b;
}

// k / d for magic = (2^32 - 1) / d: 2^32 - magic d lies in [1, d], so the
// product's high word is the quotient or one less.
__device__ __forceinline__ uint32_t div_row(uint32_t k, uint32_t d, uint32_t magic) {
  const uint32_t q = __umulhi(k, magic);
  return k - q * d >= d ? q + 1 : q;
}

// Strided rows: the vectors of all rows in one index space (rows may start
// at any element, so the accesses are those of an element's alignment), then
// the elements behind each row's last vector.
template <typename E, bool NT>
__device__ __forceinline__ double ssq_rows(const typename E::T* g, const Item& it, int lane) {
  const uint32_t vpr = static_cast<uint32_t>(it.n) / E::V, nv = vpr * static_cast<uint32_t>(it.rows);
  double a = 0.0, b = 0.0;
  auto at = [&](uint32_t k) {
    const uint32_t r = div_row(k, vpr, it.magic);
    return g + int64_t(r) * it.ld + (k - r * vpr) * E::V;
  };
  constexpr uint32_t U = 8;
  uint32_t k = lane;
#pragma unroll 1
  for (; k + 64 * (U - 1) < nv; k += 64 * U) {
    typename E::Vec x[U];
#pragma unroll
    for (uint32_t j = 0; j < U; ++j) x[j] = load_vec<E, NT>(at(k + 64 * j));
#pragma unroll
    for (uint32_t j = 0; j < U; ++j) add_vec<E>(x[j], a, b);
  }
#pragma unroll 1
  for (; k < nv; k += 64) {
    const typename E::Vec x = load_vec<E, NT>(at(k));
    add_vec<E>(x, a, b);
  }
  const uint32_t done = vpr * E::V, tail = static_cast<uint32_t>(it.n) - done;
#pragma unroll 1
  for (uint32_t e = lane; e < tail * static_cast<uint32_t>(it.rows); e += 64) {
    const uint32_t r = e / tail;
    a += sq(E::load(g + int64_t(r) * it.ld + done + (e - r * tail)));
  }
  return a + b;
}

template <typename E, bool NT>
__device__ __forceinline__ double ssq_item(const Item& it, int lane) {
  typedef typename E::T T;
  const T* g = reinterpret_cast<const T*>(it.g);
  return it.rows > 1 ? ssq_rows<E, NT>(g, it, lane) : ssq_run<E, NT>(g, it.n, lane);
}

template <bool NT>
__device__ __forceinline__ double ssq_any(const Item& it, int lane) {
  return it.dtype == MUON_F32 ? ssq_item<F32, NT>(it, lane) : ssq_item<Bf16, NT>(it, lane);
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
  return x;
}

template <int W = kWaves>
__device__ __forceinline__ double block_sum(double x, double* red) {
  x = wave_sum(x);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < W; ++w) s += red[w];
  return s;
}

// A thread's share (of T threads) of the sum of n partials, eight loads at once.
template <int T>
__device__ __forceinline__ double sum_share(const double* part, int n, int t) {
  double s = 0.0;
  for (int i = t; i < n; i += 8 * T) {
    double x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = i + j * T < n ? part[i + j * T] : 0.0;
    s += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
  }
  return s;
}

// Sum of n partials, the same for every thread of the block.
__device__ __forceinline__ double sum_partials(const double* part, int n, double* red) {
  return block_sum(sum_share<kThreads>(part, n, threadIdx.x), red);
}

__device__ __forceinline__ muon_clip_result result_of(double total, const Args& A) {
  const double n = sqrt(total) * double(A.mul), d = n + double(A.eps);
  const double c = d <= double(A.max_norm) ? 1.0 : double(A.max_norm) / d;  // NaN stays NaN
  return {static_cast<float>(n), static_cast<float>(c * double(A.mul))};
}

// Sums of squares: block b takes items 4 b .. 4 b + 3, a wave each.
__global__ __launch_bounds__(kThreads, 8) void clip_norm_kernel(Args A) {
  __shared__ double red[kWaves];
  const int lane = threadIdx.x & 63;
  const int i = __builtin_amdgcn_readfirstlane(blockIdx.x * kWaves + (threadIdx.x >> 6));
  double s = 0.0;
  if (i < A.n_items) {
    const Item it = A.items[i];
    s = wave_sum(i < A.n_stream ? ssq_any<true>(it, lane) : ssq_any<false>(it, lane));
    if (A.isum != nullptr && lane == 0) A.isum[i] = s;
  }
  if (lane == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) t += red[w];
    A.part[blockIdx.x] = t;
  }
}

// Long lists: block b adds up a run of consecutive partials.
__global__ __launch_bounds__(kThreads) void clip_reduce_kernel(const double* part, double* out, int n, int each) {
  __shared__ double red[kWaves];
  const int64_t beg = int64_t(blockIdx.x) * each;
  const int64_t m = beg < n ? (n - beg < each ? n - beg : each) : 0;
  const double s = sum_partials(part + beg, static_cast<int>(m), red);
  if (threadIdx.x == 0) out[blockIdx.x] = s;
}

__device__ __forceinline__ float tensor_norm(double s, const Args& A) {
  return static_cast<float>(sqrt(s) * double(A.mul));
}

// Norms of tensors from their items' sums: blocks 0 .. n_wide - 1 take a
// tensor of many items each, the others four tensors, a wave each.
__device__ __forceinline__ void tensor_norms(const Args& A, int b, double* red) {
  if (b < A.n_wide) {
    const int t = A.wide[b];
    const Range r = A.ranges[t];
    const double s = sum_partials(A.isum + r.beg, r.end - r.beg, red);
    if (threadIdx.x == 0) A.norms[t] = tensor_norm(s, A);
    return;
  }
  const int64_t t = int64_t(b - A.n_wide) * kWaves + (threadIdx.x >> 6);
  if (t >= A.n_tensors) return;
  const Range r = A.ranges[t];
  if (r.end - r.beg > kWide) return;
  const int lane = threadIdx.x & 63;
  const double s = wave_sum(sum_share<64>(A.isum + r.beg, r.end - r.beg, lane));
  if (lane == 0) A.norms[t] = tensor_norm(s, A);
}

// Block 0: the norm and the factor. The others: tensor norms.
__global__ __launch_bounds__(kThreads) void clip_finish_kernel(Args A) {
  __shared__ double red[kWaves];
  if (blockIdx.x > 0) {
    tensor_norms(A, blockIdx.x - 1, red);
    return;
  }
  const double s = sum_partials(A.part, A.n_part, red);
  if (threadIdx.x == 0) *A.res = result_of(s, A);
}

// o = g s for n consecutive elements, aligned on the output.
template <typename E>
__device__ __forceinline__ void scale_run(const typename E::T* g, typename E::T* o, int n, float s, int lane) {
  const int head = head_of<E>(o, n);
  if (lane < head) E::store(o + lane, E::load(g + lane) * s);
  g += head;
  o += head;
  n -= head;
  const int nv = n / E::V;
  constexpr int U = 4;
  int k = lane;
#pragma unroll 1
  for (; k + 64 * (U - 1) < nv; k += 64 * U) {
    typename E::Vec x[U];
#pragma unroll
    for (int j = 0; j < U; ++j) x[j] = load_vec<E, true>(g + int64_t(k + 64 * j) * E::V);
#pragma unroll
    for (int j = 0; j < U; ++j) store_vec<E>(o + int64_t(k + 64 * j) * E::V, E::scale(x[j], s));
  }
#pragma unroll 1
  for (; k < nv; k += 64) {
    const typename E::Vec x = load_vec<E, true>(g + int64_t(k) * E::V);
    store_vec<E>(o + int64_t(k) * E::V, E::scale(x, s));
  }
  const int t = nv * E::V + lane;
  if (t < n) E::store(o + t, E::load(g + t) * s);
}

// The same for strided rows (see ssq_rows).
template <typename E>
__device__ __forceinline__ void scale_rows(const typename E::T* g, typename E::T* o, const Item& it, float s, int lane) {
  const uint32_t vpr = static_cast<uint32_t>(it.n) / E::V, nv = vpr * static_cast<uint32_t>(it.rows);
  constexpr uint32_t U = 4;
  uint32_t k = lane;
#pragma unroll 1
  for (; k + 64 * (U - 1) < nv; k += 64 * U) {
    typename E::Vec x[U];
#pragma unroll
    for (uint32_t j = 0; j < U; ++j) {
      const uint32_t r = div_row(k + 64 * j, vpr, it.magic), c = (k + 64 * j - r * vpr) * E::V;
      x[j] = load_vec<E, true>(g + int64_t(r) * it.ld + c);
    }
    asm volatile("" : "+v"(k));  // the rows are worked out again: addresses kept take registers that waves need
#pragma unroll
    for (uint32_t j = 0; j < U; ++j) {
      const uint32_t r = div_row(k + 64 * j, vpr, it.magic), c = (k + 64 * j - r * vpr) * E::V;
      store_vec<E>(o + int64_t(r) * it.out_ld + c, E::scale(x[j], s));
    }
  }
#pragma unroll 1
  for (; k < nv; k += 64) {
    const uint32_t r = div_row(k, vpr, it.magic), c = (k - r * vpr) * E::V;
    const typename E::Vec x = load_vec<E, true>(g + int64_t(r) * it.ld + c);
    store_vec<E>(o + int64_t(r) * it.out_ld + c, E::scale(x, s));
  }
  const uint32_t done = vpr * E::V, tail = static_cast<uint32_t>(it.n) - done;
#pragma unroll 1
  for (uint32_t e = lane; e < tail * static_cast<uint32_t>(it.rows); e += 64) {
    const uint32_t r = e / tail, c = done + (e - r * tail);
    E::store(o + int64_t(r) * it.out_ld + c, E::load(g + int64_t(r) * it.ld + c) * s);
  }
}

template <typename E>
__device__ __forceinline__ void scale_item(const Item& it, float s, int lane) {
  typedef typename E::T T;
  const T* g = reinterpret_cast<const T*>(it.g);
  T* o = reinterpret_cast<T*>(it.o);
  if (it.rows > 1) scale_rows<E>(g, o, it, s, lane);
  else scale_run<E>(g, o, it.n, s, lane);
}

__device__ __forceinline__ void scale_any(const Item& it, float s, int lane) {
  if (it.g == it.o && s == 1.f) return;  // in place with a factor of one: nothing to do
  if (it.dtype == MUON_F32) scale_item<F32>(it, s, lane);
  else scale_item<Bf16>(it, s, lane);
}

// out = g factor, an item a wave. Every block adds the partials up itself (at
// most 32 KB, all blocks the same order), which takes no longer than a launch
// that does it once (two launches instead of three: 328 MB clipped 201 us for 203,
// 14 MB 12.3 for 13.6);
// block 0 leaves the result, the blocks behind the items the tensor norms.
__global__ __launch_bounds__(kThreads) void clip_scale_kernel(Args A, int item_blocks) {
  __shared__ double red[kWaves];
  if (int(blockIdx.x) >= item_blocks) {
    tensor_norms(A, blockIdx.x - item_blocks, red);
    return;
  }
  const int lane = threadIdx.x & 63;
  const int i = __builtin_amdgcn_readfirstlane(blockIdx.x * kWaves + (threadIdx.x >> 6));
  const muon_clip_result r = result_of(sum_partials(A.part, A.n_part, red), A);
  if (blockIdx.x == 0 && threadIdx.x == 0) *A.res = r;
  if (i < A.n_items) scale_any(A.items[i], r.scale, lane);
}

// Short lists, where launches are most of the time: one block does the whole
// call, norm and scaling, an item a wave. 64 KB (16 items) take 3.6 us for
// the norm and 5.6 us with the scaling, as long as the two launches of a list
// of 128 to 320 KB (4.4 and 5.6 us); 128 KB in one block took 5.0 and 8.4 us.
__global__ __launch_bounds__(64 * kSmall) void clip_small_kernel(Args A, int scale) {
  __shared__ double isum[kSmall];
  const int lane = threadIdx.x & 63, i = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (i < A.n_items) {
    const double s = wave_sum(ssq_any<false>(A.items[i], lane));
    if (lane == 0) isum[i] = s;
  }
  __syncthreads();
  const muon_clip_result r = result_of(wave_sum(lane < A.n_items ? isum[lane] : 0.0), A);
  if (threadIdx.x == 0) *A.res = r;
  if (A.norms != nullptr)
    for (int t = threadIdx.x; t < A.n_tensors; t += 64 * kSmall) {
      const Range q = A.ranges[t];
      double s = 0.0;
      for (int k = q.beg; k < q.end; ++k) s += isum[k];
      A.norms[t] = tensor_norm(s, A);
    }
  if (scale && i < A.n_items) scale_any(A.items[i], r.scale, lane);
}

// ------------------------------------------------------------------ host

// A tensor's place in memory: rows of `width` bytes, `stride` bytes apart
// (one row: stride 0), from the first byte to behind the last.
struct Interval {
  uintptr_t lo, hi;
  uintptr_t width, stride;
  bool write;
};

struct Host {
  std::vector<Item> items;
  std::vector<Range> ranges;
  std::vector<int32_t> wide;
  bool all_out = true;  // every non-empty tensor has an out
  int32_t n_stream = 0; // items before the last kKeepBytes
};

int64_t size_of(int32_t dtype) { return dtype == MUON_F32 ? 4 : 2; }

// Whether a written span meets another one (sorted by lo).
bool spans_meet(const Interval* beg, const Interval* end) {
  uintptr_t max_hi_any = 0, max_hi_w = 0;
  for (const Interval* x = beg; x < end; ++x) {
    if (x->lo < max_hi_w || (x->write && x->lo < max_hi_any)) return true;
    max_hi_any = std::max(max_hi_any, x->hi);
    if (x->write) max_hi_w = std::max(max_hi_w, x->hi);
  }
  return false;
}

// The same for tensors whose spans run into each other (sorted by lo), when
// they are column slices of one matrix: all rows one stride apart, so every
// byte of a tensor lies in its columns [c, c + width) modulo the stride, and
// tensors in separate groups of columns share none. True also where that
// cannot be told (other strides, columns across the end of the stride).
bool slices_meet(const Interval* beg, const Interval* end) {
  uintptr_t stride = 0;
  for (const Interval* x = beg; x < end; ++x) {
    if (x->stride != 0 && stride != 0 && x->stride != stride) return true;
    stride = std::max(stride, x->stride);
  }
  if (stride == 0) return true;
  auto column = [=](const Interval& x) { return (x.lo - beg->lo) % stride; };
  std::vector<Interval> by_column(beg, end);
  for (const Interval& x : by_column)
    if (x.width > stride - column(x)) return true;
  std::stable_sort(by_column.begin(), by_column.end(),
                   [&](const Interval& x, const Interval& y) { return column(x) < column(y); });
  for (size_t i = 0, j; i < by_column.size(); i = j) {
    uintptr_t right = 0;
    for (j = i; j < by_column.size() && (j == i || column(by_column[j]) < right); ++j)
      right = std::max(right, column(by_column[j]) + by_column[j].width);
    std::sort(by_column.begin() + i, by_column.begin() + j,
              [](const Interval& x, const Interval& y) { return x.lo < y.lo; });
    if (spans_meet(by_column.data() + i, by_column.data() + j)) return true;
  }
  return false;
}

// Whether a written tensor may share a byte with another one of the list.
bool overlaps(std::vector<Interval>& iv) {
  std::sort(iv.begin(), iv.end(), [](const Interval& x, const Interval& y) { return x.lo < y.lo; });
  const Interval* const p = iv.data();
  for (size_t i = 0, j; i < iv.size(); i = j) {  // runs of spans that meet
    uintptr_t hi = 0;
    for (j = i; j < iv.size() && (j == i || iv[j].lo < hi); ++j) hi = std::max(hi, iv[j].hi);
    if (spans_meet(p + i, p + j) && slices_meet(p + i, p + j)) return true;
  }
  return false;
}

muon_status build(const muon_clip_tensor* ts, int32_t n, Host* H) {
  if (n < 0 || n > MUON_CLIP_MAX_TENSORS) return MUON_E_SHAPE;
  if (n > 0 && ts == nullptr) return MUON_E_INVALID;
  std::vector<Interval> iv;
  double total = 0.0;  // bytes
  int64_t elems = 0;
  for (int32_t i = 0; i < n; ++i) {
    const muon_clip_tensor& T = ts[i];
    if (T.dtype != MUON_F32 && T.dtype != MUON_BF16) return MUON_E_DTYPE;
    if (T.reserved != 0) return MUON_E_INVALID;
    if (T.rows < 0 || T.cols < 0 || T.rows > MUON_CLIP_MAX_NUMEL || T.cols > MUON_CLIP_MAX_NUMEL) return MUON_E_SHAPE;
    if (T.rows == 0 || T.cols == 0) continue;
    if (T.rows > MUON_CLIP_MAX_NUMEL / T.cols) return MUON_E_SHAPE;
    if (T.ld < T.cols || T.ld > MUON_CLIP_MAX_NUMEL || T.rows - 1 > MUON_CLIP_MAX_NUMEL / T.ld) return MUON_E_SHAPE;
    if (T.grad == nullptr) return MUON_E_INVALID;
    const uintptr_t es = static_cast<uintptr_t>(size_of(T.dtype));
    const uintptr_t g = reinterpret_cast<uintptr_t>(T.grad), o = reinterpret_cast<uintptr_t>(T.out);
    if (g % es != 0 || o % es != 0) return MUON_E_ALIGN;
    const uintptr_t width = static_cast<uintptr_t>(T.cols) * es;
    const uintptr_t span = static_cast<uintptr_t>((T.rows - 1) * T.ld + T.cols) * es;
    if (g > UINTPTR_MAX - span) return MUON_E_SHAPE;
    if (o != 0) {
      if (T.out_ld < T.cols || T.out_ld > MUON_CLIP_MAX_NUMEL || T.rows - 1 > MUON_CLIP_MAX_NUMEL / T.out_ld)
        return MUON_E_SHAPE;
      const uintptr_t ospan = static_cast<uintptr_t>((T.rows - 1) * T.out_ld + T.cols) * es;
      if (o > UINTPTR_MAX - ospan) return MUON_E_SHAPE;
      if (g == o && T.rows > 1 && T.ld != T.out_ld) return MUON_E_INVALID;
      iv.push_back({o, o + ospan, width, T.rows > 1 ? static_cast<uintptr_t>(T.out_ld) * es : 0, true});
    } else {
      H->all_out = false;
    }
    if (g != o) iv.push_back({g, g + span, width, T.rows > 1 ? static_cast<uintptr_t>(T.ld) * es : 0, false});
    total += double(T.rows) * double(T.cols) * double(es);
    elems += T.rows * T.cols;
    if (elems > MUON_CLIP_MAX_NUMEL) return MUON_E_SHAPE;
  }
  if (overlaps(iv)) return MUON_E_INVALID;

  // Items of about equal bytes: at most twice kTargetItems of them (twice
  // 2^42 / kMaxBytes for the longest list) and one more per tensor.
  const double want = std::ceil(total / double(kTargetItems) / double(kMinBytes)) * double(kMinBytes);
  const int64_t bytes = static_cast<int64_t>(std::min(double(kMaxBytes), std::max(double(kMinBytes), want)));
  H->ranges.resize(static_cast<size_t>(n));
  for (int32_t i = 0; i < n; ++i) {
    const muon_clip_tensor& T = ts[i];
    Range& R = H->ranges[i];
    R.beg = static_cast<int32_t>(H->items.size());
    const int64_t es = size_of(T.dtype), chunk = bytes / es;
    int64_t rows = T.rows, cols = T.cols;
    if (rows > 0 && cols > 0) {
      const char* g = static_cast<const char*>(T.grad);
      char* o = static_cast<char*>(T.out);
      const bool flat = rows == 1 || (T.ld == cols && (o == nullptr || T.out_ld == cols));
      if (flat) {
        cols *= rows;
        rows = 1;
      }
      if (cols >= chunk) {  // pieces of rows
        for (int64_t r = 0; r < rows; ++r)
          for (int64_t c = 0; c < cols; c += chunk)
            H->items.push_back({g + (r * T.ld + c) * es, o ? o + (r * T.out_ld + c) * es : nullptr, 0, 0,
                                static_cast<int32_t>(std::min(chunk, cols - c)), 1, T.dtype, 0});
      } else {              // whole rows, at most about one item's bytes
        const int64_t each = std::max<int64_t>(1, chunk / cols), vpr = cols * es / 16;
        const uint32_t magic = static_cast<uint32_t>(UINT32_MAX / std::max<int64_t>(1, vpr));
        for (int64_t r = 0; r < rows; r += each)
          H->items.push_back({g + r * T.ld * es, o ? o + r * T.out_ld * es : nullptr, T.ld, T.out_ld,
                              static_cast<int32_t>(cols), static_cast<int32_t>(std::min(each, rows - r)), T.dtype, magic});
      }
    }
    R.end = static_cast<int32_t>(H->items.size());
    if (R.end - R.beg > kWide) H->wide.push_back(i);
  }
  int64_t kept = 0;
  size_t k = H->items.size();
  while (k > 0 && kept < kKeepBytes) {
    const Item& it = H->items[--k];
    kept += int64_t(it.n) * it.rows * size_of(it.dtype);
  }
  H->n_stream = static_cast<int32_t>(k);
  return MUON_OK;
}

int32_t blocks_of(size_t items) { return static_cast<int32_t>((items + kWaves - 1) / kWaves); }

// Workspace: item sums, block sums, reduced sums (float64 each).
size_t workspace_of(size_t items) { return 8 * (items + size_t(blocks_of(items)) + kReduced); }

}  // namespace muon_clip

struct muon_clip_plan_s {
  int device = -1;
  void* dmem = nullptr;
  const muon_clip::Item* d_items = nullptr;
  const muon_clip::Range* d_ranges = nullptr;
  const int32_t* d_wide = nullptr;
  int32_t n_items = 0, n_tensors = 0, n_wide = 0, n_stream = 0;
  bool all_out = true;
  size_t ws_bytes = 0;
};

namespace {

muon_status enqueue(muon_clip_plan* plan, const muon_clip_config* cfg, muon_clip_result* result, float* norms,
                    void* ws, size_t ws_bytes, void* stream, bool scale) {
  using namespace muon_clip;
  if (plan == nullptr || cfg == nullptr || result == nullptr) return MUON_E_INVALID;
  if (!(cfg->max_norm >= 0.f) || !std::isfinite(cfg->eps) || cfg->eps < 0.f || !std::isfinite(cfg->grad_mul) ||
      !(cfg->grad_mul > 0.f))
    return MUON_E_INVALID;
  if (scale && !plan->all_out) return MUON_E_INVALID;
  if (reinterpret_cast<uintptr_t>(result) % 4 != 0 || reinterpret_cast<uintptr_t>(norms) % 4 != 0) return MUON_E_ALIGN;
  if (ws == nullptr || ws_bytes < plan->ws_bytes || reinterpret_cast<uintptr_t>(ws) % 256 != 0)
    return MUON_E_WORKSPACE;
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev != plan->device) return MUON_E_DEVICE;
  const int32_t blocks = blocks_of(static_cast<size_t>(plan->n_items));
  Args a{};
  a.items = plan->d_items;
  a.n_items = plan->n_items;
  a.n_stream = scale ? plan->n_stream : plan->n_items;
  a.isum = norms ? static_cast<double*>(ws) : nullptr;
  a.part = static_cast<double*>(ws) + plan->n_items;
  a.n_part = blocks;
  a.ranges = plan->d_ranges;
  a.n_tensors = plan->n_tensors;
  a.wide = plan->d_wide;
  a.n_wide = plan->n_wide;
  a.norms = norms;
  a.res = result;
  a.max_norm = cfg->max_norm;
  a.eps = cfg->eps;
  a.mul = cfg->grad_mul;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 block(kThreads);
  if (plan->n_items <= kSmall) {
    hipLaunchKernelGGL(clip_small_kernel, dim3(1), dim3(64 * kSmall), 0, s, a, scale ? 1 : 0);
    return hipGetLastError() == hipSuccess ? MUON_OK : MUON_E_LAUNCH;
  }
  hipLaunchKernelGGL(clip_norm_kernel, dim3(unsigned(blocks)), block, 0, s, a);
  if (hipGetLastError() != hipSuccess) return MUON_E_LAUNCH;
  if (blocks > 4 * kReduced) {
    const int32_t each = (blocks + kReduced - 1) / kReduced;
    hipLaunchKernelGGL(clip_reduce_kernel, dim3(kReduced), block, 0, s, a.part, a.part + blocks, blocks, each);
    if (hipGetLastError() != hipSuccess) return MUON_E_LAUNCH;
    a.part += blocks;
    a.n_part = kReduced;
  }
  const unsigned extra = norms ? unsigned(plan->n_wide + (plan->n_tensors + kWaves - 1) / kWaves) : 0u;
  if (scale)
    hipLaunchKernelGGL(clip_scale_kernel, dim3(unsigned(blocks) + extra), block, 0, s, a, blocks);
  else
    hipLaunchKernelGGL(clip_finish_kernel, dim3(1u + extra), block, 0, s, a);
  return hipGetLastError() == hipSuccess ? MUON_OK : MUON_E_LAUNCH;
}

}  // namespace

extern "C" {

muon_status muon_clip_workspace_bytes(const muon_clip_tensor* ts, int32_t n, size_t* bytes) {
  if (bytes == nullptr) return MUON_E_INVALID;
  try {
    muon_clip::Host H;
    const muon_status st = muon_clip::build(ts, n, &H);
    if (st == MUON_OK) *bytes = muon_clip::workspace_of(H.items.size());
    return st;
  } catch (...) {
    return MUON_E_ALLOC;
  }
}

muon_status muon_clip_plan_create(const muon_clip_tensor* ts, int32_t n, muon_clip_plan** plan) {
  if (plan == nullptr) return MUON_E_INVALID;
  *plan = nullptr;
  try {
    muon_clip::Host H;
    const muon_status st = muon_clip::build(ts, n, &H);
    if (st != MUON_OK) return st;
    int dev = 0;
    hipDeviceProp_t prop;
    if (hipGetDevice(&dev) != hipSuccess || hipGetDeviceProperties(&prop, dev) != hipSuccess ||
        std::strncmp(prop.gcnArchName, "gfx950", 6) != 0)
      return MUON_E_DEVICE;
    const size_t ib = (sizeof(muon_clip::Item) * H.items.size() + 255) / 256 * 256;
    const size_t rb = ib + (sizeof(muon_clip::Range) * H.ranges.size() + 255) / 256 * 256;
    std::vector<char> h(std::max<size_t>(256, rb + sizeof(int32_t) * H.wide.size()), 0);
    if (!H.items.empty()) std::memcpy(h.data(), H.items.data(), sizeof(muon_clip::Item) * H.items.size());
    if (!H.ranges.empty()) std::memcpy(h.data() + ib, H.ranges.data(), sizeof(muon_clip::Range) * H.ranges.size());
    if (!H.wide.empty()) std::memcpy(h.data() + rb, H.wide.data(), sizeof(int32_t) * H.wide.size());
    muon_clip_plan_s* p = new (std::nothrow) muon_clip_plan_s();
    if (!p) return MUON_E_ALLOC;
    p->device = dev;
    p->n_items = static_cast<int32_t>(H.items.size());
    p->n_tensors = n;
    p->n_stream = H.n_stream;
    p->n_wide = static_cast<int32_t>(H.wide.size());
    p->all_out = H.all_out;
    p->ws_bytes = muon_clip::workspace_of(H.items.size());
    if (hipMalloc(&p->dmem, h.size()) != hipSuccess) {
      (void)hipGetLastError();
      delete p;
      return MUON_E_ALLOC;
    }
    if (hipMemcpy(p->dmem, h.data(), h.size(), hipMemcpyHostToDevice) != hipSuccess) {
      (void)hipGetLastError();
      (void)hipFree(p->dmem);
      delete p;
      return MUON_E_DEVICE;
    }
    p->d_items = static_cast<const muon_clip::Item*>(p->dmem);
    p->d_ranges = reinterpret_cast<const muon_clip::Range*>(static_cast<char*>(p->dmem) + ib);
    p->d_wide = reinterpret_cast<const int32_t*>(static_cast<char*>(p->dmem) + rb);
    *plan = p;
    return MUON_OK;
  } catch (...) {
    return MUON_E_ALLOC;
  }
}

muon_status muon_clip_plan_norm(muon_clip_plan* plan, const muon_clip_config* cfg, muon_clip_result* result,
                                float* norms, void* workspace, size_t workspace_bytes, void* stream) {
  return enqueue(plan, cfg, result, norms, workspace, workspace_bytes, stream, false);
}

muon_status muon_clip_plan_step(muon_clip_plan* plan, const muon_clip_config* cfg, muon_clip_result* result,
                                float* norms, void* workspace, size_t workspace_bytes, void* stream) {
  return enqueue(plan, cfg, result, norms, workspace, workspace_bytes, stream, true);
}

void muon_clip_plan_destroy(muon_clip_plan* plan) {
  if (!plan) return;
  (void)hipDeviceSynchronize();
  if (plan->dmem) (void)hipFree(plan->dmem);
  delete plan;
}

}  // extern "C"
