// The Muon step on stacks of matrices with a short side (include/muon_stack.h).
//
// With m = min(rows, cols) <= 128 the Newton-Schulz iteration runs on the
// m x m Gram matrix. Polynomials of one symmetric matrix commute, so from
// A_0 = X X^T
//
//   Q_i = a I + b A_i + c A_i^2,  A_{i+1} = Q_i A_i Q_i,  P = Q_{s-1} .. Q_0
//
// and s steps are X <- P X: X (n columns) is read for A_0 and read and
// written for P X, where the step-by-step form reads it twice and writes it
// once for each of the s steps. Rounding errors of A along small eigenvalues
// grow by the map's slope (a^2 at zero) in each of the s - 1 updates of A, so
// A is formed anew from X after s steps (run_length).
//
// Phases of a matrix, each over runs of columns ("parts") or as a whole:
//   gram    buf' and u from the gradient, A = sum of u u^T over the part
//   solve   one workgroup: the norm (the trace of A), s steps, P; in small sets
//           with mp = 32 every workgroup of the next phase for itself
//   update  X <- P X for the part's columns, and its sum of X X^T
//   last    X <- P X for the part's columns, out or the weights
// A tile of X is mp x kCols (mp = m padded to 32, 64 or 128), in LDS as two
// fp16 numbers hi + lo per element, rows along the product's inner dimension:
// [m][k] for X X^T, [k][m] for P X. Products are hi hi + hi lo + lo hi with
// v_mfma_f32_32x32x16_f16 (16x16x32 in the solve).
//
// What bounds it: gram and last move every element's 6 and 8 bytes (bf16) and
// are within 1.4 to 1.8 of a copy's time; without their products they take 38
// for 41 and 46 for 47 us on 576 matrices of 64 x 768, without any LDS 37 and 46. The solve is matrix instructions, LDS reads and barriers in turn,
// one workgroup for a matrix. In small sets the phases' chains of dependent
// steps count: launch, record, first tile, and the solve's steps one by one.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include "../../include/muon_stack.h"
#include "overlap.hpp"
#include "plan.hpp"

namespace muon_stack_ns {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
// accesses at an element's alignment (the hardware takes any address)
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));

// A matrix in the rows <= cols orientation.
struct Mat {
  const void* g;
  void* b;
  void* o;
  void* w;
  int64_t ld, wld;
  int32_t m, n;
  int32_t tall;        // rows > cols: the long side runs along memory rows
  int32_t parts;
  int64_t gram_off;    // workspace: per part an mp x mp partial Gram matrix (fp32, accumulator order)
  int64_t exp_off;     // per part the exponent its operands were scaled by (int32)
  int64_t rec_off;     // {sigma, exponent} of the first run of steps
  int64_t p_off;       // P: mp x mp hi, then lo (fp16, scaled by kPScale)
  int64_t x_off;       // X between runs of steps: n (padded to tiles) x mp, fp32
  float lr_mul, wd_mul;
};

// Part `index` of a matrix: columns [beg, end), in tiles. The workgroups' first
// parts come first, in their order; `next` leads to a workgroup's others (-1:
// none). The matrix stands in the record, so that a workgroup's first gradients
// are one read away from its launch arguments (with a table of its own for
// each, three reads: 1 us more of a workgroup's 6 on a small set).
struct Part {
  Mat M;
  int32_t beg, end, index, next;
};

struct Args {
  const Mat* mats;    // by class
  const Part* parts;  // of the class
  char* ws;
  const float* gscale;
  float a, b, c, mu, eps, lr, wd;
  int32_t nesterov, use_mom;
  int32_t runs, each, more;  // runs of steps: `each` steps, the first `more` of them one more
  int32_t run;               // the run this launch belongs to
};

constexpr int kXExp = 12;             // operands are scaled to at most 2^13 (X) and 2^14 (A)
constexpr float kAScale = 4096.f;     // A, Q A: entries at most 4
constexpr float kPScale = 8.f;        // Q, P: entries at most 4096

template <int MT> struct Cfg {
  static constexpr int mp = 32 * MT;
  static constexpr int cols = MT == 1 ? 128 : 64;      // kCols
  static constexpr int threads = MT == 4 ? 512 : 256;
  static constexpr int waves = threads / 64;
  static constexpr int tiles = MT == 4 ? 2 : 1;        // 32 x 32 tiles of an mp x mp product per wave
  static constexpr int ks = cols + 8;                  // row stride of [m][k], in halves: rows 16 bytes
  static constexpr int ms = mp + 8;                    // of [k][m]; apart modulo the banks
  static constexpr int lds_m = cols * ms * 4;          // bytes, hi and lo
  static constexpr int lds_k = mp * ks * 4;
  static constexpr int lds_stage = 4 * (mp * (cols + 4) > cols * (mp + 4) ? mp * (cols + 4) : cols * (mp + 4));
  static constexpr int lds_second = lds_k > lds_stage ? lds_k : lds_stage;
  static constexpr int lds_gram = MT == 1 && lds_k < waves * 4096 ? waves * 4096 : lds_k;
  static constexpr int square = 2 * mp * mp;           // halves of an mp x mp matrix in the solve, hi and lo
  static constexpr int lds_solve = (MT == 4 ? 2 : 3) * square * 2;
  static constexpr int lds_tile = lds_m + lds_second;  // (with mp = 32 the solve and P fit in, too)
  static_assert(MT > 1 || lds_tile >= lds_solve + mp * ms * 4);
};

// Waves on a SIMD that the registers have to allow for the workgroups of a launch to run at once (groups_of).
constexpr int per_simd(int mt, bool narrow) { return mt == 4 || narrow ? 2 : 3; }

// A barrier that orders LDS alone: __syncthreads() would also wait for the
// global loads on their way (no wave reads what another has stored to global
// memory in the same launch).
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// ------------------------------------------------------------- elementwise

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {  // round to nearest even
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, b2));
}

// The matrices' pointers come from a table in memory: unless told, the
// compiler takes them for flat ones, whose accesses count as LDS accesses, too,
// and are waited for with them.
#define MUON_GLOBAL __attribute__((address_space(1)))
template <typename T> using global = MUON_GLOBAL T;

// Eight consecutive elements as they lie in memory.
template <typename T> struct Raw;
template <> struct Raw<uint16_t> {
  u32x4_u v;
  __device__ __forceinline__ void load(const global<uint16_t>* p) { v = *reinterpret_cast<const global<u32x4_u>*>(p); }
  __device__ __forceinline__ float get(int q) const { return __uint_as_float(q & 1 ? v[q >> 1] & 0xffff0000u : v[q >> 1] << 16); }
  __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = pack_bf16(x[2 * q], x[2 * q + 1]);
  }
  __device__ __forceinline__ void store(global<uint16_t>* p) const { *reinterpret_cast<global<u32x4_u>*>(p) = v; }
};
template <> struct Raw<float> {
  f32x4_u v, w;
  __device__ __forceinline__ void load(const global<float>* p) {
    v = *reinterpret_cast<const global<f32x4_u>*>(p);
    w = *reinterpret_cast<const global<f32x4_u>*>(p + 4);
  }
  __device__ __forceinline__ float get(int q) const { return q < 4 ? v[q] : w[q - 4]; }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    v = f32x4_u{x[0], x[1], x[2], x[3]};
    w = f32x4_u{x[4], x[5], x[6], x[7]};
  }
  __device__ __forceinline__ void store(global<float>* p) const {
    *reinterpret_cast<global<f32x4_u>*>(p) = v;
    *reinterpret_cast<global<f32x4_u>*>(p + 4) = w;
  }
};
__device__ __forceinline__ void store1(global<uint16_t>* p, float x) { *p = static_cast<uint16_t>(pack_bf16(x, 0.f)); }
__device__ __forceinline__ void store1(global<float>* p, float x) { *p = x; }

// mu b + g rounded once to the buffer's type. fp32: the fused multiply-add.
// bf16: rounding the nearest float32 once more is wrong where it lies half way
// between two bf16 numbers and the exact value does not (one element in a
// hundred with mu = 0.95, so a wave always has one). Rounded to odd it is
// right: of the float32 numbers below and above an inexact value the odd one,
// which is never half way, and on the exact value's side of it. The two come
// from the rounding modes of the fused multiply-add; the mode is changed and
// restored within the asm, so no other instruction sees it.
__device__ __forceinline__ void fma_odd(float mu, const float (&b)[4], const float (&g)[4], float (&x)[4]) {
  float d[4], u[4];
  asm("s_setreg_imm32_b32 hwreg(HW_REG_MODE, 0, 2), 2\n\t"  // float32: toward -infinity
      "s_nop 1\n\t"
      "v_fma_f32 %0, %8, %9, %13\n\t"
      "v_fma_f32 %1, %8, %10, %14\n\t"
      "v_fma_f32 %2, %8, %11, %15\n\t"
      "v_fma_f32 %3, %8, %12, %16\n\t"
      "s_setreg_imm32_b32 hwreg(HW_REG_MODE, 0, 2), 1\n\t"  // toward +infinity
      "s_nop 1\n\t"
      "v_fma_f32 %4, %8, %9, %13\n\t"
      "v_fma_f32 %5, %8, %10, %14\n\t"
      "v_fma_f32 %6, %8, %11, %15\n\t"
      "v_fma_f32 %7, %8, %12, %16\n\t"
      "s_setreg_imm32_b32 hwreg(HW_REG_MODE, 0, 2), 0\n\t"  // to nearest
      "s_nop 1"
      : "=&v"(d[0]), "=&v"(d[1]), "=&v"(d[2]), "=&v"(d[3]), "=&v"(u[0]), "=&v"(u[1]), "=&v"(u[2]), "=&v"(u[3])
      : "v"(mu), "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]), "v"(g[0]), "v"(g[1]), "v"(g[2]), "v"(g[3]));
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t lo = __float_as_uint(d[q]), hi = __float_as_uint(u[q]);
    const uint32_t odd = 0u - (lo & 1u);
    x[q] = __uint_as_float((lo & odd) | (hi & ~odd));  // (equal where the value is exact; +0 for a sum of zero)
  }
}
// nb: as stored.
__device__ __forceinline__ void momentum(float mu, const Raw<float>& b, const float (&g)[8], Raw<float>& nb) {
  float s[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) s[q] = __fmaf_rn(mu, b.get(q), g[q]);
  nb.set(s);
}
__device__ __forceinline__ void momentum(float mu, const Raw<uint16_t>& b, const float (&g)[8], Raw<uint16_t>& nb) {
  float s[8];
#pragma unroll
  for (int h = 0; h < 8; h += 4) {
    const float x[4] = {b.get(h), b.get(h + 1), b.get(h + 2), b.get(h + 3)}, y[4] = {g[h], g[h + 1], g[h + 2], g[h + 3]};
    float z[4];
    fma_odd(mu, x, y, z);
#pragma unroll
    for (int q = 0; q < 4; ++q) s[h + q] = z[q];
  }
  nb.set(s);
}

// The exponent e of x >= 0 (its bits) in [2^e, 2^(e+1)), in [-126, 127].
__device__ __forceinline__ int exponent(int bits) { return min(max((bits >> 23) - 127, -126), 127); }

// The largest of the lanes' numbers (none negative), for all of them.
__device__ __forceinline__ int wave_max(int v) {
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true));  // row_shr:1, 2, 4, 8
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xf, 0xf, true));  // row_bcast:15, 31
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xf, 0xf, true));
  return __builtin_amdgcn_readlane(v, 63);
}

// x = hi + lo, two of them at once, as packed pairs.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  const f16x2 h = __builtin_convertvector((f2{x, y}), f16x2);
  // (x - h in one mixed-precision instruction; exact)
  const f16x2 l = __builtin_convertvector((f2{__builtin_fmaf(static_cast<float>(h[0]), -1.f, x), __builtin_fmaf(static_cast<float>(h[1]), -1.f, y)}), f16x2);
  hi = __builtin_bit_cast(uint32_t, h);
  lo = __builtin_bit_cast(uint32_t, l);
}

// ---------------------------------------------------------- tiles in memory

// The two vectors of eight consecutive elements a thread moves of a tile:
// vector c8 of rows ra and rb. Rows run along memory: the m rows of a wide
// matrix (eight columns each), the columns of a tall one (eight of its m).
struct Spot {
  int ra, rb, c;
};
template <int MT, bool ALONG_K, bool PAIRS>
__device__ __forceinline__ Spot spot(int tid) {
  typedef Cfg<MT> C;
  constexpr int vpr = (ALONG_K ? C::cols : C::mp) / 8;
  const int r = tid / vpr, c = tid % vpr * 8;
  if (PAIRS) return {2 * r, 2 * r + 1, c};
  return {r, r + C::threads / vpr, c};
}

// Where a thread's two vectors are in memory, in elements from the matrix's
// first. In a tile at the matrix's edge a vector that would reach over a row's
// end is moved back to end with it (`back` elements, eight or more: it has none
// of its own), and a row that does not exist is the last one: the loads need
// no branch, and fix() puts the values in their places. NARROW: memory rows of
// under eight elements, which are loaded one by one.
template <bool TALL, bool NARROW>
struct Frame {
  int64_t a, b;
  int c, back;  // first element in the row as loaded
  bool oka, okb;
  __device__ __forceinline__ Frame(const Mat& M, int64_t ld, int k0, const Spot& s, bool edge) {
    const int r0 = TALL ? k0 : 0, at = TALL ? s.c : k0 + s.c;
    c = at;
    back = 0;
    oka = okb = true;
    if (NARROW || edge) {
      const int rows = TALL ? M.n : M.m, len = TALL ? M.m : M.n;
      c = NARROW ? min(at, len - 1) : min(at, len - 8);
      back = at - c;
      oka = r0 + s.ra < rows;
      okb = r0 + s.rb < rows;
      a = int64_t(min(r0 + s.ra, rows - 1)) * ld + c;
      b = int64_t(min(r0 + s.rb, rows - 1)) * ld + c;
    } else {
      a = (r0 * ld + (TALL ? 0 : k0)) + (s.ra * ld + s.c);
      b = (r0 * ld + (TALL ? 0 : k0)) + (s.rb * ld + s.c);
    }
  }
};
// Whether a tile reaches over the matrix's sides.
template <int MT>
__device__ __forceinline__ bool at_edge(const Mat& M, int k0) {
  return M.m < Cfg<MT>::mp || k0 + Cfg<MT>::cols > M.n;
}

template <typename T, bool TALL, bool NARROW>
__device__ __forceinline__ void fetch(const void* base, const Mat& M, const Frame<TALL, NARROW>& f, Raw<T> (&x)[2]) {
  const global<T>* const a = (const global<T>*)base + f.a;
  const global<T>* const b = (const global<T>*)base + f.b;
  if constexpr (!NARROW) {
    x[0].load(a);
    x[1].load(b);
  } else {
    // the row's elements from c on, the last of them again behind its end
    const int left = (TALL ? M.m : M.n) - 1 - f.c;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int at = min(q, left);
      if constexpr (sizeof(T) == 2) {
        const uint32_t u = uint32_t(a[at]), v = uint32_t(b[at]);
        x[0].v[q >> 1] = q & 1 ? x[0].v[q >> 1] | u << 16 : u;
        x[1].v[q >> 1] = q & 1 ? x[1].v[q >> 1] | v << 16 : v;
      } else if (q < 4) {
        x[0].v[q] = a[at];
        x[1].v[q] = b[at];
      } else {
        x[0].w[q - 4] = a[at];
        x[1].w[q - 4] = b[at];
      }
    }
  }
}

// How many elements of the vector are the thread's own: [0, mine) once they
// are in their places (NARROW: they already are).
template <bool TALL, bool NARROW>
__device__ __forceinline__ int own(const Mat& M, const Frame<TALL, NARROW>& f, bool ok) {
  if (!ok) return 0;
  if (NARROW) return f.back > 0 ? 0 : min(8, (TALL ? M.m : M.n) - f.c);
  return max(0, 8 - f.back);
}
// Moves a vector's values `back` places to the front; zeros where nothing is the thread's own.
template <bool TALL, bool NARROW>
__device__ __forceinline__ void fix(const Mat& M, const Frame<TALL, NARROW>& f, bool ok, float (&x)[8]) {
  const int n = own(M, f, ok);
  if constexpr (!NARROW) {
#pragma unroll
    for (int s = 1; s < 8; s <<= 1)
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = f.back & s ? (q + s < 8 ? x[q + s] : 0.f) : x[q];
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) x[q] = q < n ? x[q] : 0.f;
}
// The other way: values in their places go to where the vector was loaded.
template <bool TALL, bool NARROW>
__device__ __forceinline__ void spread(const Frame<TALL, NARROW>& f, float (&x)[8]) {
  if constexpr (!NARROW) {
#pragma unroll
    for (int s = 1; s < 8; s <<= 1)
#pragma unroll
      for (int q = 7; q >= 0; --q) x[q] = f.back & s ? (q >= s ? x[q - s] : 0.f) : x[q];
  }
}
// Stores the thread's own elements of one of its rows (at: f.a or f.b). At an
// edge the values have not been put in their places yet.
template <typename T, bool TALL, bool NARROW>
__device__ __forceinline__ void put_row(void* base, const Mat& M, const Frame<TALL, NARROW>& f, int64_t at, bool ok, bool edge, Raw<T>& x) {
  if (!NARROW && !edge) {
    x.store((global<T>*)base + at);
    return;
  }
  float v[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = x.get(q);
  fix(M, f, ok, v);
  global<T>* const p = (global<T>*)base + at + f.back;
  const int n = own(M, f, ok);
  if (n == 8) {
    x.set(v);
    x.store(p);
  } else {
#pragma unroll
    for (int q = 0; q < 7; ++q)
      if (q < n) store1(p + q, v[q]);
  }
}

// Writes a thread's 2 x 8 values (scaled to fp16's range) as hi and lo.
// SAME: the tile's rows are memory rows, eight consecutive halves each; else
// the memory rows ra, rb = ra + 1 are columns of the tile, in pairs.
template <bool SAME>
__device__ __forceinline__ void put_tile(_Float16* hi, _Float16* lo, int stride, const Spot& s, const float (&x)[2][8]) {
  if constexpr (SAME) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint4 h, l;
      split2(x[j][0], x[j][1], h.x, l.x);
      split2(x[j][2], x[j][3], h.y, l.y);
      split2(x[j][4], x[j][5], h.z, l.z);
      split2(x[j][6], x[j][7], h.w, l.w);
      const int at = (j ? s.rb : s.ra) * stride + s.c;
      *reinterpret_cast<uint4*>(hi + at) = h;
      *reinterpret_cast<uint4*>(lo + at) = l;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      uint32_t h, l;
      split2(x[0][q], x[1][q], h, l);
      const int at = (s.c + q) * stride + s.ra;
      *reinterpret_cast<uint32_t*>(hi + at) = h;
      *reinterpret_cast<uint32_t*>(lo + at) = l;
    }
  }
}

// acc += X Y^T over K of the inner dimension, from K0: 32 rows of X from row
// xr, 32 of Y from row yr (rows `stride` halves apart). Accumulator i of a
// lane: row 8 (i / 4) + 4 (lane / 32) + i % 4, column lane % 32.
__device__ __forceinline__ f32x16 mul3(const f16x8& xh, const f16x8& xl, const f16x8& yh, const f16x8& yl, f32x16 acc) {
  acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(xh, yh, acc, 0, 0, 0);
  acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(xh, yl, acc, 0, 0, 0);
  acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(xl, yh, acc, 0, 0, 0);
  return acc;
}
__device__ __forceinline__ f16x8 frag(const _Float16* p, int row, int stride, int k, int lane) {
  return *reinterpret_cast<const f16x8*>(p + (row + (lane & 31)) * stride + k + (lane >> 5) * 8);
}

// The rows (of 4) and column of a lane's accumulators 4 g .. 4 g + 3.
__device__ __forceinline__ int acc_row(int g, int lane) { return 8 * g + 4 * (lane >> 5); }

// Writes the transpose of a 32 x 32 accumulator tile: element (row, col) goes
// to [c0 + col][r0 + row], four consecutive halves at a time.
__device__ __forceinline__ void put_acc(_Float16* hi, _Float16* lo, int stride, int r0, int c0, const f32x16& x, float scale, int lane) {
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    uint2 h, l;
    split2(x[4 * g] * scale, x[4 * g + 1] * scale, h.x, l.x);
    split2(x[4 * g + 2] * scale, x[4 * g + 3] * scale, h.y, l.y);
    const int at = (c0 + (lane & 31)) * stride + r0 + acc_row(g, lane);
    *reinterpret_cast<uint2*>(hi + at) = h;
    *reinterpret_cast<uint2*>(lo + at) = l;
  }
}

// Which 32 x 32 tiles of an mp x mp product a wave has: rows ti, columns tj + t.
template <int MT>
__device__ __forceinline__ void tile_of(int wave, int& ti, int& tj) {
  if (MT == 4) ti = wave >> 1, tj = 2 * (wave & 1);
  else if (MT == 2) ti = wave >> 1, tj = wave & 1;
  else ti = 0, tj = 0;
}

// acc += the tile's K K^T. MT = 1 has one tile of the product: each wave takes
// every fourth step of the inner dimension, and the sums are added at the end.
template <int MT>
__device__ __forceinline__ void gram_tile(const _Float16* hi, const _Float16* lo, f32x16 (&acc)[Cfg<MT>::tiles], int wave, int lane) {
  typedef Cfg<MT> C;
  int ti, tj;
  tile_of<MT>(wave, ti, tj);
  constexpr int step = MT == 1 ? C::waves : 1;
#pragma unroll
  for (int k = 0; k < C::cols / 16; k += step) {
    const int kk = 16 * (MT == 1 ? k + wave : k);
    const f16x8 xh = frag(hi, 32 * ti, C::ks, kk, lane), xl = frag(lo, 32 * ti, C::ks, kk, lane);
#pragma unroll
    for (int t = 0; t < C::tiles; ++t) {
      const f16x8 yh = frag(hi, 32 * (tj + t), C::ks, kk, lane), yl = frag(lo, 32 * (tj + t), C::ks, kk, lane);
      acc[t] = mul3(xh, xl, yh, yl, acc[t]);
    }
  }
}

// Where the partial Gram matrices of a run of steps are. With mp = 32 the
// workgroups of `update` may read them all before they write the next run's,
// each at its own time, so the runs take turns with two arrays.
template <int MT>
__device__ __forceinline__ int64_t gram_at(const Mat& M, int run) {
  return M.gram_off + (MT == 1 && run % 2 ? int64_t(M.parts) * (Cfg<MT>::mp * Cfg<MT>::mp * 4) : 0);
}

// The part's sum of X X^T, for a run, goes to the workspace, in accumulator order.
template <int MT>
__device__ __forceinline__ void put_gram(const Args& A, const Mat& M, int run, int part, f32x16 (&acc)[Cfg<MT>::tiles], char* lds, int wave, int lane) {
  typedef Cfg<MT> C;
  float4* const out = reinterpret_cast<float4*>(A.ws + gram_at<MT>(M, run)) + int64_t(part) * (C::mp * C::mp / 4);
  if constexpr (MT == 1) {
    float4* const red = reinterpret_cast<float4*>(lds);
    lds_barrier();
#pragma unroll
    for (int g = 0; g < 4; ++g) red[(wave * 4 + g) * 64 + lane] = make_float4(acc[0][4 * g], acc[0][4 * g + 1], acc[0][4 * g + 2], acc[0][4 * g + 3]);
    lds_barrier();
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < C::waves; ++w) {
      const float4 t = red[(w * 4 + wave) * 64 + lane];
      s.x += t.x, s.y += t.y, s.z += t.z, s.w += t.w;
    }
    out[wave * 64 + lane] = s;
    lds_barrier();
  } else {
#pragma unroll
    for (int t = 0; t < C::tiles; ++t)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        out[((wave * C::tiles + t) * 4 + g) * 64 + lane] = make_float4(acc[t][4 * g], acc[t][4 * g + 1], acc[t][4 * g + 2], acc[t][4 * g + 3]);
  }
}

// ------------------------------------------------------------------ phases

// What a launch's u depends on.
struct Step {
  float gs, mu;
  bool use_mom, nesterov;
  __device__ __forceinline__ Step(const Args& A) : gs(A.gscale ? *A.gscale : 1.f), mu(A.mu), use_mom(A.use_mom), nesterov(A.nesterov) {}
};
// u of a vector from the gradient and the momentum as loaded; FIRST: b becomes
// the momentum's new value. (Without momentum the second operand is the
// gradient again: it is loaded, and not used.)
template <typename T, bool FIRST>
__device__ __forceinline__ void form_u(const Step& S, const Raw<T>& g, Raw<T>& b, float (&u)[8]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) u[q] = g.get(q) * S.gs;
  if (!S.use_mom) return;
  if constexpr (FIRST) {
    const Raw<T> old = b;
    momentum(S.mu, old, u, b);
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) u[q] = S.nesterov ? __fmaf_rn(S.mu, b.get(q), u[q]) : b.get(q);
}

// A tile's gradient and momentum on their way.
template <typename T, int MT, bool TALL, bool NARROW>
struct Load {
  Raw<T> g[2], b[2];
  __device__ __forceinline__ void start(const Mat& M, const void* b2, int k0, const Spot& s) {
    const Frame<TALL, NARROW> f(M, M.ld, k0, s, at_edge<MT>(M, k0));
    fetch<T>(M.g, M, f, g);
    fetch<T>(b2, M, f, b);
  }
};

// Phase gram over the part's columns. The operands are scaled by a power of
// two that puts the largest |u| so far into [2^12, 2^13): when a tile raises
// it, the sums so far are rescaled, which is exact.
template <typename T, int MT, bool TALL, bool NARROW>
__device__ __forceinline__ void phase_gram(const Args& A, const Mat& M, const Part& p, char* lds) {
  typedef Cfg<MT> C;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  _Float16* const hi = reinterpret_cast<_Float16*>(lds);
  _Float16* const lo = hi + C::mp * C::ks;
  __shared__ int top[C::waves];
  const Step S(A);
  const void* const b2 = S.use_mom ? M.b : M.g;
  // a wide matrix's rows are the tile's; of a tall one they are its columns
  const Spot s = spot<MT, !TALL, TALL>(tid);
  f32x16 acc[C::tiles] = {};
  int e = -126;
  constexpr int kAhead = NARROW ? 1 : 2;  // tiles on their way while one is worked on
  Load<T, MT, TALL, NARROW> x, y;
  auto start = [&](Load<T, MT, TALL, NARROW>& l, int t) { l.start(M, b2, min(t, p.end - 1) * C::cols, s); };
  auto work = [&](Load<T, MT, TALL, NARROW>& l, int t) {
    const int k0 = t * C::cols;
    const bool edge = at_edge<MT>(M, k0);
    const Frame<TALL, NARROW> f(M, M.ld, k0, s, edge);
    float u[2][8];
    form_u<T, true>(S, l.g[0], l.b[0], u[0]);
    form_u<T, true>(S, l.g[1], l.b[1], u[1]);
    if (S.use_mom) {
      put_row<T>(M.b, M, f, f.a, f.oka, edge, l.b[0]);
      put_row<T>(M.b, M, f, f.b, f.okb, edge, l.b[1]);
    }
    if (NARROW || edge) {
      fix(M, f, f.oka, u[0]);
      fix(M, f, f.okb, u[1]);
    }
    start(l, t + kAhead);
    float big = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) big = fmaxf(big, fmaxf(fabsf(u[0][q]), fabsf(u[1][q])));
    const int most = wave_max(__float_as_int(big));
    if (lane == 0) top[wave] = exponent(most);
    lds_barrier();  // the tile of the pass before has been read, too
    int now = e;
#pragma unroll
    for (int w = 0; w < C::waves; ++w) now = max(now, top[w]);
    now = __builtin_amdgcn_readfirstlane(now);
    if (now > e) {
#pragma unroll
      for (int i = 0; i < C::tiles; ++i)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][q] = ldexpf(acc[i][q], 2 * (e - now));
      e = now;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 8; ++q) u[j][q] = ldexpf(u[j][q], kXExp - e);
    put_tile<!TALL>(hi, lo, C::ks, s, u);
    lds_barrier();
    gram_tile<MT>(hi, lo, acc, wave, lane);
  };
  start(x, p.beg);
  if constexpr (kAhead == 1) {
    for (int t = p.beg; t < p.end; ++t) work(x, t);
  } else {
    __builtin_amdgcn_sched_barrier(0);  // loads are waited for in the order they went out
    start(y, p.beg + 1);
    for (int t = p.beg; t < p.end; t += 2) {
      work(x, t);
      if (t + 1 >= p.end) break;
      work(y, t + 1);
    }
  }
  put_gram<MT>(A, M, 0, p.index, acc, lds, wave, lane);
  if (tid == 0) reinterpret_cast<int32_t*>(A.ws + M.exp_off)[p.index] = e;
}

// The solve's matrices. A wave has 16 whole columns of each (its own ones), one
// per lane % 16, as accumulators of v_mfma_f32_16x16x32_f16: element e of step
// s of a lane is row row_of(s, e). As an operand of a product over the rows the
// same registers hold that lane's part of the inner dimension, in an order that
// the LDS copy of a matrix (column by column, chunks of eight rows) follows: a
// wave's own operand never goes through LDS, and a step has two barriers (mp =
// 128: four). Against 32 x 32 tiles with both operands in LDS and six to eight
// barriers a step: 96 matrices of 16 x 765, four runs of steps, 58 -> 52 us; 48
// matrices of 64 x 768 16 -> 15 us; 256 of 128 x 2048 the same 61 us, for which
// four waves of 32 columns take 74.
template <int MT> struct Sq {
  static constexpr int mp = 32 * MT;
  static constexpr int waves = mp / 16, threads = 64 * waves;
  static constexpr int steps = mp / 32, tiles = mp / 16;
};
template <int MT> struct Acc {  // own columns in float32
  f32x4 t[Sq<MT>::tiles];
  __device__ __forceinline__ float get(int s, int e) const { return t[2 * s + (e >> 2)][e & 3]; }
  __device__ __forceinline__ void set(int s, int e, float x) { t[2 * s + (e >> 2)][e & 3] = x; }
};
template <int MT> struct Own {  // own columns as hi + lo
  f16x8 h[Sq<MT>::steps], l[Sq<MT>::steps];
  __device__ __forceinline__ float get(int s, int e) const { return static_cast<float>(h[s][e]) + static_cast<float>(l[s][e]); }
  __device__ __forceinline__ void set(const Acc<MT>& x, float scale) {
#pragma unroll
    for (int s = 0; s < Sq<MT>::steps; ++s) {
      uint4 a, b;
      split2(x.get(s, 0) * scale, x.get(s, 1) * scale, a.x, b.x);
      split2(x.get(s, 2) * scale, x.get(s, 3) * scale, a.y, b.y);
      split2(x.get(s, 4) * scale, x.get(s, 5) * scale, a.z, b.z);
      split2(x.get(s, 6) * scale, x.get(s, 7) * scale, a.w, b.w);
      h[s] = __builtin_bit_cast(f16x8, a);
      l[s] = __builtin_bit_cast(f16x8, b);
    }
  }
};
__device__ __forceinline__ int row_of(int s, int e, int lane) { return 32 * s + 16 * (e >> 2) + 4 * (lane >> 4) + (e & 3); }

// The LDS copy: hi, then lo, in rows of 2 mp bytes (a column each) without
// padding (three of 64 x 64 let three workgroups share a CU). The 16-byte
// chunks of a row are exchanged so that the same chunk of 16 rows in turn lies
// in all banks.
template <int MT>
__device__ __forceinline__ int chunk_at(int row, int c) {
  constexpr int n = 4 * MT;  // chunks of a row
  return row * (8 * n) + ((c ^ (MT == 1 ? row >> 2 : MT == 2 ? row >> 1 : row)) & (n - 1)) * 8;
}
template <int MT>
__device__ __forceinline__ void put_own(_Float16* x, const Own<MT>& v, int wave, int lane) {
  typedef Sq<MT> Q;
#pragma unroll
  for (int s = 0; s < Q::steps; ++s) {
    const int at = chunk_at<MT>(16 * wave + (lane & 15), 4 * s + (lane >> 4));
    *reinterpret_cast<f16x8*>(x + at) = v.h[s];
    *reinterpret_cast<f16x8*>(x + Q::mp * Q::mp + at) = v.l[s];
  }
}
// The own columns of Y^T X: Y from LDS, the own columns of X.
template <int MT>
__device__ __forceinline__ void mul_own(const _Float16* y, const Own<MT>& x, Acc<MT>& acc, int lane) {
  typedef Sq<MT> Q;
#pragma unroll
  for (int t = 0; t < Q::tiles; ++t) acc.t[t] = f32x4{};
#pragma unroll
  for (int s = 0; s < Q::steps; ++s) {
    // (128 rows: else the loads of all steps are hoisted, and registers spilled)
    if (MT == 4 && s % 2 == 0) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < Q::tiles; ++t) {
      const int at = chunk_at<MT>(16 * t + (lane & 15), 4 * s + (lane >> 4));
      const f16x8 yh = *reinterpret_cast<const f16x8*>(y + at), yl = *reinterpret_cast<const f16x8*>(y + Q::mp * Q::mp + at);
      acc.t[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(yh, x.h[s], acc.t[t], 0, 0, 0);
      acc.t[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(yh, x.l[s], acc.t[t], 0, 0, 0);
      acc.t[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(yl, x.h[s], acc.t[t], 0, 0, 0);
    }
  }
}

// What makes X of u: sigma, and the exponent it is scaled for.
struct Norm {
  float sigma;
  int e;
};

// Phase solve: A from its parts, the norm (first run), the run's steps on A
// and P. The matrices are symmetric but for rounding. The order of the factors
// matters for that rounding: T = A^T Q, A' = T^T Q = Q^T A Q and P' = P^T Q keep
// the antisymmetric part of A's errors from growing faster than the rest (with
// T = Q^T A it grew by 14 in every step of the quintic: X off by 4e-4 after five
// steps on full-rank 64 x 768, 1e-5 in this order). P goes to out: mp x mp hi,
// then lo, in rows of `stride` halves.
template <int MT>
__device__ __forceinline__ void phase_solve(const Args& A, const Mat& M, char* lds, _Float16* out, int stride, Norm& norm) {
  typedef Sq<MT> Q;
  const int run = A.run, tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  constexpr int kSquare = Cfg<MT>::square;
  _Float16* const la = reinterpret_cast<_Float16*>(lds);  // A
  _Float16* const lt = la + kSquare;                      // T
  _Float16* const lp = MT == 4 ? la : lt + kSquare;       // P (mp = 128: where A was, for its product)
  __shared__ float red[Q::waves];
  const bool mine = wave < Q::waves;  // (with mp = 32 a workgroup may have more)
  const int32_t* const exps = reinterpret_cast<const int32_t*>(A.ws + M.exp_off);
  int e = kXExp;
  if (run == 0) {
    int top = 0;
    for (int p = lane; p < M.parts; p += 64) top = max(top, exps[p] + 126);
    e = wave_max(top) - 126;
  }
  Acc<MT> acc;
#pragma unroll
  for (int t = 0; t < Q::tiles; ++t) acc.t[t] = f32x4{};
  const float4* const in = reinterpret_cast<const float4*>(A.ws + gram_at<MT>(M, run));
  constexpr int kJoin = MT == 4 ? 2 : 4;  // parts on their way at once
  // the four rows from row_of(s, 4 u): put_gram's tile (r / 32, column / 32), its g and lane
  auto place = [&](int s, int u) {
    const int r = row_of(s, 4 * u, lane), c = 16 * wave + (lane & 15);
    return ((MT * (r >> 5) + (c >> 5)) * 4 + (r >> 3 & 3)) * 64 + (r >> 2 & 1) * 32 + (c & 31);
  };
  if (mine)
    for (int p = 0; p < M.parts; p += kJoin) {
      float4 x[kJoin][Q::steps][2];
      int shift[kJoin];
#pragma unroll
      for (int j = 0; j < kJoin; ++j) {
        const int q = min(p + j, M.parts - 1);
        shift[j] = run == 0 ? 2 * (exps[q] - e) : 0;
#pragma unroll
        for (int s = 0; s < Q::steps; ++s)
#pragma unroll
          for (int u = 0; u < 2; ++u) x[j][s][u] = in[int64_t(q) * (Q::mp * Q::mp / 4) + place(s, u)];
      }
#pragma unroll
      for (int j = 0; j < kJoin; ++j)
        if (p + j < M.parts)
#pragma unroll
          for (int s = 0; s < Q::steps; ++s)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              acc.set(s, 4 * u, acc.get(s, 4 * u) + ldexpf(x[j][s][u].x, shift[j]));
              acc.set(s, 4 * u + 1, acc.get(s, 4 * u + 1) + ldexpf(x[j][s][u].y, shift[j]));
              acc.set(s, 4 * u + 2, acc.get(s, 4 * u + 2) + ldexpf(x[j][s][u].z, shift[j]));
              acc.set(s, 4 * u + 3, acc.get(s, 4 * u + 3) + ldexpf(x[j][s][u].w, shift[j]));
            }
    }
  auto diag = [&](int s, int k) { return row_of(s, k, lane) == 16 * wave + (lane & 15); };
  float scale = 1.f / (kAScale * kAScale);  // X was scaled by 2^kXExp
  if (run == 0) {
    // the trace is the sum of squares
    float d = 0.f;
#pragma unroll
    for (int s = 0; s < Q::steps; ++s)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (diag(s, k)) d += acc.get(s, k);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) d += __shfl_xor(d, o, 64);
    if (mine && lane == 0) red[wave] = d;
    lds_barrier();
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < Q::waves; ++w) sum += red[w];
    // sigma = 1 / ((norm + eps) 2^(kXExp - e)), whatever float32 makes of the norm; zeros give zeros
    const double size = ldexp(sqrt(double(sum)), e - kXExp);
    norm.sigma = sum == 0.f ? 0.f : static_cast<float>(1.0 / ldexp(size + double(A.eps), kXExp - e));
    norm.e = e;
    scale = norm.sigma * norm.sigma;
  }
#pragma unroll
  for (int t = 0; t < Q::tiles; ++t) acc.t[t] *= scale;
  Own<MT> x, q, pr;  // A, Q and P
  const int steps = A.each + (run < A.more ? 1 : 0);
  if (steps == 0) {
#pragma unroll
    for (int s = 0; s < Q::steps; ++s)
#pragma unroll
      for (int k = 0; k < 8; ++k) acc.set(s, k, diag(s, k) ? 1.f : 0.f);
    pr.set(acc, kPScale);
  } else {
    x.set(acc, kAScale);
    if (mine) put_own<MT>(la, x, wave, lane);
    lds_barrier();
  }
  constexpr float kAA = 1.f / (kAScale * kAScale), kAQ = 1.f / (kAScale * kPScale), kPQ = 1.f / (kPScale * kPScale);
#pragma unroll 1
  for (int i = 0; i < steps; ++i) {
    const bool more = i + 1 < steps;
    if (mine) {
      mul_own<MT>(la, x, acc, lane);
      const float b = A.b / kAScale, c = A.c * kAA;
#pragma unroll
      for (int s = 0; s < Q::steps; ++s)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc.set(s, k, __fmaf_rn(c, acc.get(s, k), __fmaf_rn(b, x.get(s, k), diag(s, k) ? A.a : 0.f)));
      q.set(acc, kPScale);
      if (i == 0) pr = q;
      if (more) {
        mul_own<MT>(la, q, acc, lane);
        x.set(acc, kAQ * kAScale);
        put_own<MT>(lt, x, wave, lane);
      }
    }
    if (i > 0) {
      if (MT == 4) lds_barrier();  // A has been read
      if (mine) put_own<MT>(lp, pr, wave, lane);
    }
    if (i > 0 || more) lds_barrier();
    if (mine) {
      if (i > 0) {
        mul_own<MT>(lp, q, acc, lane);
        pr.set(acc, kPQ * kPScale);
      }
      if (more) {
        mul_own<MT>(lt, q, acc, lane);
        x.set(acc, kAQ * kAScale);
      }
    }
    if (!more) break;
    if (MT == 4 && i > 0) lds_barrier();  // P has been read
    if (mine) put_own<MT>(la, x, wave, lane);
    lds_barrier();
  }
  if (mine) {
    const int c = 16 * wave + (lane & 15);
#pragma unroll
    for (int s = 0; s < Q::steps; ++s)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int at = c * stride + row_of(s, 4 * u, lane);
        *reinterpret_cast<f16x4*>(out + at) = f16x4{pr.h[s][4 * u], pr.h[s][4 * u + 1], pr.h[s][4 * u + 2], pr.h[s][4 * u + 3]};
        *reinterpret_cast<f16x4*>(out + Q::mp * stride + at) = f16x4{pr.l[s][4 * u], pr.l[s][4 * u + 1], pr.l[s][4 * u + 2], pr.l[s][4 * u + 3]};
      }
  }
}

// What a tile of P X needs on its way: the gradient and momentum, or X.
template <typename T, int MT, bool TALL, bool NARROW>
struct ApplyLoad {
  Load<T, MT, TALL, NARROW> u;
  Raw<float> x[2];
};

// P X for the part's columns: GRAD: X is sigma u, from the gradients, else what
// the run before left. LAST: out or the weights, else X and its X X^T.
template <typename T, int MT, bool TALL, bool NARROW, bool GRAD, bool LAST, bool WEIGHTS, bool SOLVE>
__device__ __forceinline__ void phase_apply(const Args& A, const Mat& M, const Part& p, Norm norm, char* lds) {
  typedef Cfg<MT> C;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  _Float16* const mh = reinterpret_cast<_Float16*>(lds);        // [k][m]
  _Float16* const ml = mh + C::cols * C::ms;
  _Float16* const kh = reinterpret_cast<_Float16*>(lds + C::lds_m);  // [m][k]
  _Float16* const kl = kh + C::mp * C::ks;
  float* const stage = reinterpret_cast<float*>(lds + C::lds_m);
  const int mi = wave % MT, ki = wave / MT;  // the wave's rows of X and columns of the tile, in 32s
  const Step S(A);
  const void* const b2 = S.use_mom ? M.b : M.g;
  const float keep = 1.f - (A.lr * M.lr_mul) * (A.wd * M.wd_mul), step = A.lr * M.lr_mul;
  global<float>* const xs = (global<float>*)(A.ws + M.x_off);
  constexpr bool kRowsAreK = TALL || !GRAD;  // memory rows are columns of X
  const Spot s = spot<MT, !kRowsAreK, !kRowsAreK>(tid);
  const Spot o = spot<MT, !TALL, false>(tid);
  f32x16 acc2[C::tiles] = {};
  // tiles on their way while one is worked on (a second one of fp32 numbers does not fit in the registers beside P's share)
  constexpr int kAhead = !GRAD || sizeof(T) == 4 || NARROW ? 1 : 2;
  typedef ApplyLoad<T, MT, TALL, NARROW> L;
  L x, y;
  Raw<T> wt[2];  // the weights, one tile ahead
  auto start = [&](L& l, int t) {
    const int k0 = min(t, p.end - 1) * C::cols;
    if constexpr (GRAD) {
      l.u.start(M, b2, k0, s);
    } else {
      l.x[0].load(xs + int64_t(k0 + s.ra) * C::mp + s.c);
      l.x[1].load(xs + int64_t(k0 + s.rb) * C::mp + s.c);
    }
  };
  auto start_w = [&](int t) {
    if constexpr (LAST && WEIGHTS) {
      const int k0 = min(t, p.end - 1) * C::cols;
      const Frame<TALL, NARROW> fr(M, M.wld, k0, o, at_edge<MT>(M, k0));
      fetch<T>(M.w, M, fr, wt);
    }
  };
  start(x, p.beg);
  start_w(p.beg);
  f16x8 ph[C::mp / 16], pl[C::mp / 16];
  if constexpr (SOLVE) {
    const _Float16* const pm = reinterpret_cast<const _Float16*>(lds + C::lds_solve);
#pragma unroll
    for (int k = 0; k < C::mp / 16; ++k) {
      ph[k] = frag(pm, 0, C::ms, 16 * k, lane);
      pl[k] = frag(pm + C::mp * C::ms, 0, C::ms, 16 * k, lane);
    }
    lds_barrier();
  } else {
    const _Float16* const pm = reinterpret_cast<const _Float16*>(A.ws + M.p_off);
#pragma unroll
    for (int k = 0; k < C::mp / 16; ++k) {
      ph[k] = frag(pm, 32 * mi, C::mp, 16 * k, lane);
      pl[k] = frag(pm + C::mp * C::mp, 32 * mi, C::mp, 16 * k, lane);
    }
    if (GRAD) norm = *reinterpret_cast<const Norm*>(A.ws + M.rec_off);
  }
  const float f = GRAD ? norm.sigma * (1.f / kPScale) : 1.f / (kAScale * kPScale);
  const int e = norm.e;
  auto work = [&](L& l, int t) {
    const int k0 = t * C::cols;
    const bool edge = at_edge<MT>(M, k0);
    float u[2][8];
    if constexpr (GRAD) {
      form_u<T, false>(S, l.u.g[0], l.u.b[0], u[0]);
      form_u<T, false>(S, l.u.g[1], l.u.b[1], u[1]);
      if (NARROW || edge) {
        const Frame<TALL, NARROW> fr(M, M.ld, k0, s, edge);
        fix(M, fr, fr.oka, u[0]);
        fix(M, fr, fr.okb, u[1]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 8; ++q) u[j][q] = l.x[j].get(q);
    }
    start(l, t + kAhead);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 8; ++q) u[j][q] = GRAD ? ldexpf(u[j][q], kXExp - e) : u[j][q] * kAScale;
    put_tile<kRowsAreK>(mh, ml, C::ms, s, u);
    lds_barrier();
    f32x16 acc = {};
#pragma unroll
    for (int k = 0; k < C::mp / 16; ++k)
      acc = mul3(frag(mh, 32 * ki, C::ms, 16 * k, lane), frag(ml, 32 * ki, C::ms, 16 * k, lane), ph[k], pl[k], acc);
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] *= f;
    const int col = 32 * mi + (lane & 31);
    if constexpr (!LAST) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        xs[int64_t(k0 + 32 * ki + acc_row(i >> 2, lane) + (i & 3)) * C::mp + col] = acc[i];
      put_acc(kh, kl, C::ks, 32 * ki, 32 * mi, acc, kAScale, lane);
      lds_barrier();
      gram_tile<MT>(kh, kl, acc2, wave, lane);
    } else {
      // through LDS, so that memory rows are written whole
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int row = 32 * ki + acc_row(g, lane);
        if constexpr (TALL) {
#pragma unroll
          for (int i = 0; i < 4; ++i) stage[(row + i) * (C::mp + 4) + col] = acc[4 * g + i];
        } else {
          *reinterpret_cast<f32x4*>(stage + col * (C::cols + 4) + row) = f32x4{acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]};
        }
      }
      lds_barrier();
      const Frame<TALL, NARROW> fr(M, WEIGHTS ? M.wld : M.ld, k0, o, edge);
      // values of weights at an edge are where they were loaded: those of X go there
      Raw<T> r[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const f32x4* const in = reinterpret_cast<const f32x4*>(stage + (j ? o.rb : o.ra) * ((TALL ? C::mp : C::cols) + 4) + o.c);
        const f32x4 a = in[0], b = in[1];
        float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
        if (NARROW || edge) spread<TALL, NARROW>(fr, v);
        if constexpr (WEIGHTS) {
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = __fmaf_rn(-step, v[q], wt[j].get(q) * keep);
        }
        r[j].set(v);
      }
      start_w(t + 1);
      put_row<T>(WEIGHTS ? M.w : M.o, M, fr, fr.a, fr.oka, edge, r[0]);
      put_row<T>(WEIGHTS ? M.w : M.o, M, fr, fr.b, fr.okb, edge, r[1]);
    }
  };
  if constexpr (kAhead == 1) {
    for (int t = p.beg; t < p.end; ++t) work(x, t);
  } else {
    __builtin_amdgcn_sched_barrier(0);  // loads are waited for in the order they went out
    start(y, p.beg + 1);
    for (int t = p.beg; t < p.end; t += 2) {
      work(x, t);
      if (t + 1 >= p.end) break;
      work(y, t + 1);
    }
  }
  if constexpr (!LAST) put_gram<MT>(A, M, A.run + 1, p.index, acc2, lds, wave, lane);
}

// The matrix's direction is the workgroup's own matter; the rest is the launch's.
template <typename T, int MT, bool NARROW, bool GRAD, bool LAST, bool WEIGHTS, bool SOLVE>
__device__ __forceinline__ void apply_any(const Args& A, const Mat& M, const Part& p, Norm norm, char* lds) {
  if (M.tall) phase_apply<T, MT, true, NARROW, GRAD, LAST, WEIGHTS, SOLVE>(A, M, p, norm, lds);
  else phase_apply<T, MT, false, NARROW, GRAD, LAST, WEIGHTS, SOLVE>(A, M, p, norm, lds);
}
template <typename T, int MT, bool NARROW>
__device__ __forceinline__ void gram_any(const Args& A, const Mat& M, const Part& p, char* lds) {
  if (M.tall) phase_gram<T, MT, true, NARROW>(A, M, p, lds);
  else phase_gram<T, MT, false, NARROW>(A, M, p, lds);
}

// ----------------------------------------------------------------- kernels

// Gradient and momentum read, the momentum written, parts' Gram matrices: 576
// bf16 matrices of 64 x 768 (170 MB and 19 MB of parts) 41 us, 4.6 TB/s; 192 of
// 128 x 2048 (302 MB and 25 MB) 85 us (80 to 88 by run), 3.9 TB/s; 48 of 64 x 768
// 9 us.
template <typename T, int MT, bool NARROW>
__global__ __launch_bounds__(Cfg<MT>::threads, per_simd(MT, NARROW)) void stack_gram_kernel(Args A) {
  extern __shared__ __align__(16) char lds[];
#pragma unroll 1
  for (int i = int(blockIdx.x); i >= 0;) {
    const Part p = A.parts[i];  // by value: a reference would be read again after every store
    gram_any<T, MT, NARROW>(A, p.M, p, lds);
    lds_barrier();
    i = p.next;
  }
}

// Five quintic steps: 48 matrices of 64 rows 14.5 us (parts 4, a step 2), 576 in
// two or three on each CU 28 us; 192 of 128 rows 58 to 63 us, a step 11, of which
// the matrix cores are busy for 5 and the LDS for 3.5, in turns.
template <int MT>
__global__ __launch_bounds__(Sq<MT>::threads) void stack_solve_kernel(Args A, int first) {
  extern __shared__ __align__(16) char lds[];
  const Mat M = A.mats[first + blockIdx.x];
  Norm norm = {};
  phase_solve<MT>(A, M, lds, reinterpret_cast<_Float16*>(A.ws + M.p_off), Cfg<MT>::mp, norm);
  if (A.run == 0 && threadIdx.x == 0) *reinterpret_cast<Norm*>(A.ws + M.rec_off) = norm;
}

// LAST with weights: 576 bf16 matrices of 64 x 768 (226 MB) 47 us, 4.9 TB/s; 192
// of 128 x 2048 (403 MB) 97 us (92 to 100 by run), 4.2 TB/s; 48 of 64 x 768, no
// weights, 8 us. With 172 registers, so that two workgroups shared a CU and a
// third of them waited, the first took 53. SOLVE: each part's workgroup solves
// for P itself.
template <typename T, int MT, bool NARROW, bool GRAD, bool LAST, bool WEIGHTS, bool SOLVE>
__global__ __launch_bounds__(Cfg<MT>::threads, per_simd(MT, NARROW || SOLVE)) void stack_apply_kernel(Args A) {
  extern __shared__ __align__(16) char lds[];
#pragma unroll 1
  for (int i = int(blockIdx.x); i >= 0;) {
    const Part p = A.parts[i];
    Norm norm = {};
    if constexpr (SOLVE) {  // P into the tile's LDS, behind what the solve uses itself
      phase_solve<MT>(A, p.M, lds, reinterpret_cast<_Float16*>(lds + Cfg<MT>::lds_solve), Cfg<MT>::ms, norm);
      lds_barrier();
    }
    apply_any<T, MT, NARROW, GRAD, LAST, WEIGHTS, SOLVE>(A, p.M, p, norm, lds);
    lds_barrier();
    i = p.next;
  }
}

// -------------------------------------------------------------------- host

constexpr int kClasses = 4;  // mp = 32 with memory rows of under eight elements, 32, 64, 128
int class_of(const muon_stack& s) {
  const int64_t m = std::min(s.rows, s.cols);
  return s.cols < 8 ? 0 : m <= 32 ? 1 : m <= 64 ? 2 : 3;
}
int mp_of(int cls) { return cls < 2 ? 32 : 16 << cls; }
int cols_of(int cls) { return cls < 2 ? 128 : 64; }

struct Host {
  muon_dtype dtype = MUON_BF16;
  std::vector<muon_stack> stacks;
  std::vector<Mat> mats;               // by class, then in the caller's order
  std::vector<int32_t> owner;          // the stack of each
  std::vector<int64_t> index;          // its place in it
  std::vector<Part> parts;             // by class, the matrices' records not filled in
  std::vector<int32_t> part_mat;       // the matrix of each
  int32_t mat_beg[kClasses + 1] = {}, part_beg[kClasses + 1] = {}, groups[kClasses] = {};
  bool solve_there[kClasses] = {};     // the parts' workgroups solve for P themselves
  size_t ws_bytes = 0;
};

bool empty(const muon_stack& s) { return s.count == 0 || s.rows == 0 || s.cols == 0; }

// Whether a stack's matrices are apart, and the place of each of them in
// memory. Those that follow each other without a gap, in rows or in columns,
// are one place; between others there may be matrices of another stack.
bool apart(const muon_stack& s, int64_t ld, int64_t stride, const void* p, bool write, int64_t es,
           std::vector<muon::tensor_overlap::Interval>* iv) {
  const int64_t span = (s.rows - 1) * ld + s.cols, all = (s.count - 1) * stride + span;
  const bool blocks = s.count == 1 || stride >= span;
  const bool side = !blocks && stride >= s.cols && (s.count - 1) * stride + s.cols <= ld;
  if (!blocks && !side) return false;
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  if (lo > UINTPTR_MAX - static_cast<uintptr_t>(all * es)) return false;
  int64_t count = s.count, rows = s.rows, cols = s.cols;
  if (blocks && (count == 1 || stride == rows * ld)) rows *= count, count = 1;
  else if (side && stride == cols) cols *= count, count = 1;
  const bool solid = rows == 1 || ld == cols;  // no gaps between the rows
  const int64_t size = (rows - 1) * ld + cols;
  for (int64_t t = 0; t < count; ++t) {
    const uintptr_t at = lo + static_cast<uintptr_t>(t * stride * es);
    iv->push_back({at, at + static_cast<uintptr_t>(size * es), static_cast<uintptr_t>((solid ? size : cols) * es),
                   static_cast<uintptr_t>((solid ? 0 : ld) * es), write});
  }
  return true;
}

constexpr int64_t kMaxStep = int64_t(1) << 40;  // elements of a stride

muon_status validate(const muon_stack* st, int32_t n, muon_dtype dtype, const muon_stack_weight* w, int64_t* total) {
  if (dtype != MUON_F32 && dtype != MUON_BF16) return MUON_E_DTYPE;
  if (n < 0 || n > MUON_STACK_MAX_MATRICES) return MUON_E_SHAPE;
  if (n > 0 && st == nullptr) return MUON_E_INVALID;
  const int64_t es = dtype == MUON_F32 ? 4 : 2;
  std::vector<muon::tensor_overlap::Interval> iv;
  *total = 0;
  for (int32_t i = 0; i < n; ++i) {
    const muon_stack& s = st[i];
    if (s.count < 0 || s.rows < 0 || s.cols < 0 || s.count > MUON_STACK_MAX_MATRICES || s.rows > MUON_STACK_MAX_LONG ||
        s.cols > MUON_STACK_MAX_LONG)
      return MUON_E_SHAPE;
    if (empty(s)) continue;
    if (std::min(s.rows, s.cols) > MUON_STACK_MAX_SHORT) return MUON_E_SHAPE;
    *total += s.count;
    if (*total > MUON_STACK_MAX_MATRICES) return MUON_E_SHAPE;
    if (s.ld < s.cols || s.ld > kMaxStep || s.stride < 0 || s.stride > kMaxStep) return MUON_E_SHAPE;
    if (s.grad == nullptr || s.out == nullptr) return MUON_E_INVALID;
    for (const void* p : {s.grad, static_cast<const void*>(s.momentum), static_cast<const void*>(s.out)})
      if (reinterpret_cast<uintptr_t>(p) % es != 0) return MUON_E_ALIGN;
    if (!apart(s, s.ld, s.stride, s.out, true, es, &iv)) return MUON_E_INVALID;
    if (s.momentum && !apart(s, s.ld, s.stride, s.momentum, true, es, &iv)) return MUON_E_INVALID;
    if (s.grad != s.out && !apart(s, s.ld, s.stride, s.grad, false, es, &iv)) return MUON_E_INVALID;
    if (w == nullptr) continue;
    const muon_stack_weight& v = w[i];
    if (v.weight == nullptr || !std::isfinite(v.lr_mul) || !std::isfinite(v.wd_mul)) return MUON_E_INVALID;
    if (v.ld < s.cols || v.ld > kMaxStep || v.stride < 0 || v.stride > kMaxStep) return MUON_E_SHAPE;
    if (reinterpret_cast<uintptr_t>(v.weight) % es != 0) return MUON_E_ALIGN;
    if (!apart(s, v.ld, v.stride, v.weight, true, es, &iv)) return MUON_E_INVALID;
  }
  return muon::tensor_overlap::overlaps(iv) ? MUON_E_INVALID : MUON_OK;
}

// The tiles of a class, one matrix after the other, are dealt out in equal runs
// to as many workgroups as run at once (three of 256 threads, two for narrow
// matrices, or one of 512 on each of 256 CUs), but none is given fewer than kLeast tiles, or so few that a
// matrix falls into more than kMaxParts parts. More workgroups than run at once
// mean more parts, whose Gram matrices are written and added up again: gram and
// update of 576 matrices of 64 x 768 take 41 + 47 us in 768 workgroups, 45 + 53
// in 1152, 47 + 57 in 2304; of 192 of 128 x 2048 83 + 95 in 256, 102 + 118 in
// 384, 92 + 108 in 768. kLeast 1, 2 and 4: 48 matrices of 64 x 768 31, 31 and 34
// us, 96 of 16 x 765 56, 52 and 76. kMaxParts 16, 64 and 128: two of 65536 x 64
// 208, 77 and 67 us, two of 128 x 65536 365, 171 and 174, eight of 32 x 32768 68,
// 58 and 47.
constexpr int64_t kMaxParts = 128, kLeast = 2;
int64_t groups_of(int cls) { return cls == 3 ? 256 : cls == 0 ? 512 : 768; }
// Matrices of mp = 32 that all run at once in two workgroups on each CU have
// their P solved for by the workgroups that use it: the launch that this saves
// costs more than one wave's solve does in each of them (96 fp32 matrices of 16
// x 765, four runs of steps: 58 us with, 53 us without it; 288 bf16 matrices of
// 32 x 768, which take turns: 37 us with, 41 us without).
constexpr int64_t kSolveThere = 512;

muon_status build(const muon_stack* st, int32_t n, muon_dtype dtype, Host* H) {
  int64_t total = 0;
  const muon_status status = validate(st, n, dtype, nullptr, &total);
  if (status != MUON_OK) return status;
  H->dtype = dtype;
  H->stacks.assign(st, st + n);
  const int64_t es = dtype == MUON_F32 ? 4 : 2;
  size_t off = 0;
  auto take = [&](int64_t bytes) {
    const size_t at = off;
    off += (static_cast<size_t>(bytes) + 255) / 256 * 256;
    return static_cast<int64_t>(at);
  };
  for (int cls = 0; cls < kClasses; ++cls) {
    H->mat_beg[cls] = static_cast<int32_t>(H->mats.size());
    const size_t part0 = H->parts.size();
    H->part_beg[cls] = static_cast<int32_t>(part0);
    int64_t tiles = 0, longest = 0;
    const int64_t cols = cols_of(cls), mp = mp_of(cls);
    auto tiles_of = [&](const muon_stack& s) { return (std::max(s.rows, s.cols) + cols - 1) / cols; };
    for (int32_t i = 0; i < n; ++i)
      if (!empty(st[i]) && class_of(st[i]) == cls) {
        tiles += st[i].count * tiles_of(st[i]);
        longest = std::max(longest, tiles_of(st[i]));
      }
    if (tiles == 0) continue;
    const int64_t least = std::max(kLeast, (longest + kMaxParts - 1) / kMaxParts);
    const int64_t groups = std::max<int64_t>(1, std::min(groups_of(cls), tiles / least));
    H->solve_there[cls] = mp == 32 && tiles / least <= kSolveThere;
    int64_t at = 0, group = 0;  // tiles dealt out, and the workgroup the next one goes to
    auto end_of = [&](int64_t g) { return (g + 1) * tiles / groups; };
    H->groups[cls] = static_cast<int32_t>(groups);
    H->parts.resize(part0 + groups);
    H->part_mat.resize(part0 + groups);
    int64_t of_group = -1;  // the part that the group's next one follows (-1: it has none)
    for (int32_t i = 0; i < n; ++i) {
      const muon_stack& s = st[i];
      if (empty(s) || class_of(s) != cls) continue;
      for (int64_t t = 0; t < s.count; ++t) {
        Mat M{};
        M.g = static_cast<const char*>(s.grad) + t * s.stride * es;
        M.b = s.momentum ? static_cast<char*>(s.momentum) + t * s.stride * es : nullptr;
        M.o = static_cast<char*>(s.out) + t * s.stride * es;
        M.ld = s.ld;
        M.m = static_cast<int32_t>(std::min(s.rows, s.cols));
        M.n = static_cast<int32_t>(std::max(s.rows, s.cols));
        M.tall = s.rows > s.cols;
        const int64_t nt = tiles_of(s);
        for (int64_t beg = 0; beg < nt;) {
          const int64_t end = std::min(nt, beg + end_of(group) - at);
          int64_t place = static_cast<int64_t>(part0) + group;
          if (of_group >= 0) {
            place = static_cast<int64_t>(H->parts.size());
            H->parts[of_group].next = static_cast<int32_t>(place - static_cast<int64_t>(part0));
            H->parts.emplace_back();
            H->part_mat.emplace_back();
          }
          Part& p = H->parts[place];
          p.beg = static_cast<int32_t>(beg);
          p.end = static_cast<int32_t>(end);
          p.index = M.parts++;
          p.next = -1;
          H->part_mat[place] = static_cast<int32_t>(H->mats.size());
          of_group = place;
          at += end - beg;
          beg = end;
          if (at == end_of(group)) {
            of_group = -1;
            ++group;
          }
        }
        M.gram_off = take((mp == 32 ? 2 : 1) * M.parts * mp * mp * 4);  // (gram_at)
        M.exp_off = take(M.parts * 4);
        M.rec_off = take(8);
        M.p_off = take(mp * mp * 4);
        M.x_off = take(nt * cols * mp * 4);
        H->mats.push_back(M);
        H->owner.push_back(i);
        H->index.push_back(t);
      }
    }
  }
  H->mat_beg[kClasses] = static_cast<int32_t>(H->mats.size());
  H->part_beg[kClasses] = static_cast<int32_t>(H->parts.size());
  H->ws_bytes = off;
  return MUON_OK;
}

// The plan's tables in device memory: the matrices, then the parts.
size_t parts_at(const Host& H) { return (sizeof(Mat) * H.mats.size() + 255) / 256 * 256; }
std::vector<char> tables(const Host& H, const std::vector<Mat>& mats) {
  const size_t at = parts_at(H);
  std::vector<char> h(std::max<size_t>(256, at + sizeof(Part) * H.parts.size()), 0);
  if (!mats.empty()) std::memcpy(h.data(), mats.data(), sizeof(Mat) * mats.size());
  for (size_t i = 0; i < H.parts.size(); ++i) {
    Part p = H.parts[i];
    p.M = mats[H.part_mat[i]];
    std::memcpy(h.data() + at + i * sizeof(Part), &p, sizeof(Part));
  }
  return h;
}

// The largest number of steps from one Gram matrix. Errors of A grow by at
// most the slope of lambda -> lambda q(lambda)^2 in each update of A, and move
// the last factor q by |b / a| of what they have become: with A rounded to 2^-23
// a run of five quintic steps leaves 1.39 11.86^4 2^-23 = 3.3e-3 of X for each
// such rounding that lies in directions of singular value near zero. That is
// what bf16 sets take (a median of up to 1.8e-3 on gradients of rank one, 3e-6
// on random ones; a bf16 output's rounding is 1.7e-3): with runs of three
// and two steps X is off by 5e-5 at most on the same gradients, and 48 matrices
// of 64 x 768 take 45 us for 31, 576 of them 175 for 115, 192 of 128 x 2048 332 for
// 217. fp32 sets form A anew before errors have grown by eight. The slope and
// |q| are taken over the values that 65 points of X0's range pass through (on
// the host in every call: 1 us; 4097 points took 50 and set the time of small
// sets). P's entries have to stay in fp16's range, too.
int run_length(const muon_config& c, muon_dtype dtype) {
  double slope = 0.0, top = 0.0;
  for (int i = 0; i <= 64; ++i) {
    double x = i / 64.0;
    for (int32_t t = 0; t < c.steps; ++t) {
      const double l = x * x, q = c.a + l * (c.b + c.c * l), dq = c.b + 2.0 * c.c * l;
      slope = std::max(slope, std::fabs(q * q + 2.0 * l * q * dq));
      top = std::max(top, std::fabs(q));
      x *= q;
    }
  }
  const double limit = dtype == MUON_F32 ? 8.0 : 32768.0;
  int s = 1;
  double grown = slope, size = top * top;
  while (s < c.steps && grown <= limit && size <= 4096.0) {
    ++s;
    grown *= slope;
    size *= top;
  }
  return s;
}

}  // namespace muon_stack_ns

struct muon_stack_plan_s {
  muon_stack_ns::Host host;
  int device = -1;
  void* dmem = nullptr;
  const muon_stack_ns::Mat* d_mats = nullptr;
  const muon_stack_ns::Part* d_parts = nullptr;
  bool has_weights = false;
  const float* gscale = nullptr;
};

namespace {

using namespace muon_stack_ns;

template <typename K>
muon_status go(K kernel, unsigned grid, int threads, int lds, hipStream_t s, const Args& a) {
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(unsigned(threads)), size_t(lds), s, a);
  return hipGetLastError() == hipSuccess ? MUON_OK : MUON_E_LAUNCH;
}

// The steps' phases, launch by launch. SOLVE: without a launch for the solve.
template <typename T, int MT, bool NARROW, bool WEIGHTS, bool SOLVE>
muon_status run_phases(unsigned groups, int mats, int first, Args a, hipStream_t s) {
  typedef Cfg<MT> C;
  muon_status st = go(stack_gram_kernel<T, MT, NARROW>, groups, C::threads, C::lds_gram, s, a);
  for (int run = 0; run < a.runs && st == MUON_OK; ++run) {
    a.run = run;
    if constexpr (!SOLVE) {
      hipLaunchKernelGGL(stack_solve_kernel<MT>, dim3(unsigned(mats)), dim3(Sq<MT>::threads), C::lds_solve, s, a, first);
      if (hipGetLastError() != hipSuccess) return MUON_E_LAUNCH;
    }
    const bool last = run + 1 == a.runs;
    if (run == 0)
      st = last ? go(stack_apply_kernel<T, MT, NARROW, true, true, WEIGHTS, SOLVE>, groups, C::threads, C::lds_tile, s, a)
                : go(stack_apply_kernel<T, MT, NARROW, true, false, false, SOLVE>, groups, C::threads, C::lds_tile, s, a);
    else
      st = last ? go(stack_apply_kernel<T, MT, NARROW, false, true, WEIGHTS, SOLVE>, groups, C::threads, C::lds_tile, s, a)
                : go(stack_apply_kernel<T, MT, NARROW, false, false, false, SOLVE>, groups, C::threads, C::lds_tile, s, a);
  }
  return st;
}

template <typename T, int MT, bool NARROW, bool WEIGHTS>
muon_status run_class(const muon_stack_plan_s* p, int cls, Args a, hipStream_t s) {
  const Host& H = p->host;
  const int first = H.mat_beg[cls], mats = H.mat_beg[cls + 1] - first;
  if (mats == 0) return MUON_OK;
  const unsigned groups = unsigned(H.groups[cls]);
  a.parts = p->d_parts + H.part_beg[cls];
  if constexpr (MT == 1)
    if (H.solve_there[cls]) return run_phases<T, MT, NARROW, WEIGHTS, true>(groups, mats, first, a, s);
  return run_phases<T, MT, NARROW, WEIGHTS, false>(groups, mats, first, a, s);
}

template <typename T, bool WEIGHTS>
muon_status run_all(const muon_stack_plan_s* p, const Args& a, hipStream_t s) {
  muon_status st = run_class<T, 1, true, WEIGHTS>(p, 0, a, s);
  if (st == MUON_OK) st = run_class<T, 1, false, WEIGHTS>(p, 1, a, s);
  if (st == MUON_OK) st = run_class<T, 2, false, WEIGHTS>(p, 2, a, s);
  if (st == MUON_OK) st = run_class<T, 4, false, WEIGHTS>(p, 3, a, s);
  return st;
}

muon_status step(muon_stack_plan_s* p, const muon_config* cfg, const muon_apply* ap, void* ws, size_t bytes, void* stream) {
  if (p == nullptr) return MUON_E_INVALID;
  const Host& H = p->host;
  // the range check of the 16-bit operands holds for both dtypes
  muon_status st = muon::validate_config(cfg, MUON_BF16);
  if (st != MUON_OK) return st;
  if (H.mats.empty()) return MUON_OK;
  if (ap != nullptr && !p->has_weights) return MUON_E_INVALID;
  if (ws == nullptr || bytes < H.ws_bytes || reinterpret_cast<uintptr_t>(ws) % 256 != 0) return MUON_E_WORKSPACE;
  if (cfg->momentum != 0.f)
    for (const Mat& M : H.mats)
      if (M.b == nullptr) return MUON_E_INVALID;
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev != p->device) return MUON_E_DEVICE;
  Args a{};
  a.mats = p->d_mats;
  a.ws = static_cast<char*>(ws);
  a.gscale = p->gscale;
  a.a = cfg->a;
  a.b = cfg->b;
  a.c = cfg->c;
  a.mu = cfg->momentum;
  a.eps = cfg->eps;
  a.nesterov = cfg->nesterov;
  a.use_mom = cfg->momentum != 0.f;
  if (ap != nullptr) {
    a.lr = ap->lr;
    a.wd = ap->wd;
  }
  const int len = run_length(*cfg, H.dtype);
  a.runs = std::max(1, (cfg->steps + len - 1) / len);
  a.each = cfg->steps / a.runs;
  a.more = cfg->steps % a.runs;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (H.dtype == MUON_F32) return ap ? run_all<float, true>(p, a, s) : run_all<float, false>(p, a, s);
  return ap ? run_all<uint16_t, true>(p, a, s) : run_all<uint16_t, false>(p, a, s);
}

}  // namespace

extern "C" {

muon_status muon_stack_workspace_bytes(const muon_stack* stacks, int32_t n, muon_dtype dtype, size_t* bytes) {
  if (bytes == nullptr) return MUON_E_INVALID;
  try {
    Host H;
    const muon_status st = build(stacks, n, dtype, &H);
    if (st == MUON_OK) *bytes = H.ws_bytes;
    return st;
  } catch (...) {
    return MUON_E_ALLOC;
  }
}

muon_status muon_stack_plan_create(const muon_stack* stacks, int32_t n, muon_dtype dtype, muon_stack_plan** plan) {
  if (plan == nullptr) return MUON_E_INVALID;
  *plan = nullptr;
  muon_stack_plan_s* p = nullptr;
  try {
    p = new muon_stack_plan_s();
    muon_status st = build(stacks, n, dtype, &p->host);
    if (st == MUON_OK) {
      hipDeviceProp_t prop;
      if (hipGetDevice(&p->device) != hipSuccess || hipGetDeviceProperties(&prop, p->device) != hipSuccess ||
          std::strncmp(prop.gcnArchName, "gfx950", 6) != 0)
        st = MUON_E_DEVICE;
    }
    if (st != MUON_OK) {
      delete p;
      return st;
    }
    const std::vector<char> h = tables(p->host, p->host.mats);
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
    p->d_mats = static_cast<const Mat*>(p->dmem);
    p->d_parts = reinterpret_cast<const Part*>(static_cast<char*>(p->dmem) + parts_at(p->host));
    *plan = p;
    return MUON_OK;
  } catch (...) {
    if (p != nullptr && p->dmem != nullptr) (void)hipFree(p->dmem);
    delete p;
    return MUON_E_ALLOC;
  }
}

muon_status muon_stack_plan_step(muon_stack_plan* plan, const muon_config* cfg, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  return step(plan, cfg, nullptr, workspace, workspace_bytes, stream);
}

muon_status muon_stack_plan_set_weights(muon_stack_plan* plan, const muon_stack_weight* w, int32_t n) {
  if (plan == nullptr) return MUON_E_INVALID;
  Host& H = plan->host;
  if (n != static_cast<int32_t>(H.stacks.size())) return MUON_E_SHAPE;
  if (n > 0 && w == nullptr) return MUON_E_INVALID;
  try {
    int64_t total = 0;
    muon_status st = validate(H.stacks.data(), n, H.dtype, w, &total);
    if (st != MUON_OK) return st;
    std::vector<Mat> mats = H.mats;
    const int64_t es = H.dtype == MUON_F32 ? 4 : 2;
    for (size_t i = 0; i < mats.size(); ++i) {
      const muon_stack_weight& v = w[H.owner[i]];
      mats[i].w = static_cast<char*>(v.weight) + H.index[i] * v.stride * es;
      mats[i].wld = v.ld;
      mats[i].lr_mul = v.lr_mul;
      mats[i].wd_mul = v.wd_mul;
    }
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev != plan->device) return MUON_E_DEVICE;
    const std::vector<char> h = tables(H, mats);
    if (hipDeviceSynchronize() != hipSuccess) return MUON_E_DEVICE;
    if (hipMemcpy(plan->dmem, h.data(), h.size(), hipMemcpyHostToDevice) != hipSuccess) return MUON_E_DEVICE;
    H.mats = std::move(mats);
    plan->has_weights = true;
    return MUON_OK;
  } catch (...) {
    return MUON_E_ALLOC;
  }
}

muon_status muon_stack_plan_step_apply(muon_stack_plan* plan, const muon_config* cfg, const muon_apply* ap, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  const muon_status st = muon::validate_apply(ap);
  if (st != MUON_OK) return st;
  return step(plan, cfg, ap, workspace, workspace_bytes, stream);
}

muon_status muon_stack_plan_set_grad_scale(muon_stack_plan* plan, const float* scale) {
  if (plan == nullptr) return MUON_E_INVALID;
  if (reinterpret_cast<uintptr_t>(scale) % 4 != 0) return MUON_E_ALIGN;
  plan->gscale = scale;
  return MUON_OK;
}

void muon_stack_plan_destroy(muon_stack_plan* plan) {
  if (!plan) return;
  (void)hipDeviceSynchronize();
  if (plan->dmem) (void)hipFree(plan->dmem);
  delete plan;
}

}  // extern "C"
