// One element of the Adam update and the vector accesses around it, shared by
// the step over whole tensors (adam.hip) and over rows of a table (embed.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace muon_adam {

constexpr int kVec = 4;        // consecutive elements per thread and access

__device__ __forceinline__ float bf2f(uint16_t h) { return __uint_as_float(uint32_t(h) << 16); }
__device__ __forceinline__ uint16_t f2bf(float f) {  // round to nearest even
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return static_cast<uint16_t>((u >> 16) | 0x40u);  // NaN
  return static_cast<uint16_t>((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}

template <typename T> struct PElem;
template <> struct PElem<float> {
  static __device__ __forceinline__ float load(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
  static __device__ __forceinline__ void store(void* p, int64_t i, float v) { static_cast<float*>(p)[i] = v; }
};
template <> struct PElem<uint16_t> {
  static __device__ __forceinline__ float load(const void* p, int64_t i) {
    return bf2f(static_cast<const uint16_t*>(p)[i]);
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, float v) {
    static_cast<uint16_t*>(p)[i] = f2bf(v);
  }
};

struct Consts {
  float b1, c1, b2, c2, eps, keep, step, isb2;
  float gs;  // the gradient's factor
};

// One element: updates m, v in place and returns the new parameter value.
__device__ __forceinline__ float adam_elem(float p, float g, float& m, float& v, const Consts& k) {
  g *= k.gs;  // exact for a factor of one
  m = __fmaf_rn(k.b1, m, k.c1 * g);
  v = __fmaf_rn(k.b2, v, k.c2 * (g * g));
  const float denom = __fsqrt_rn(v) * k.isb2 + k.eps;
  return __fmaf_rn(-k.step, __fdiv_rn(m, denom), p * k.keep);
}

// Vectors of four elements at an element's alignment (the hardware takes any
// address).
typedef float f32x4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2), aligned(2)));

// Four consecutive elements of one tensor in registers.
struct Vec4 {
  float p[kVec], g[kVec], m[kVec], v[kVec];
};

// NT: past the caches (blocks of whole kBlock elements). Part blocks take
// plain accesses: 300 tensors of 2000 fp32 elements 4.4 us, 5.4 with the hints
// (5000 of them, more than the caches hold, 58 and 53 us).
template <bool NT>
__device__ __forceinline__ void load4(const float* a, float (&x)[kVec]) {
  const f32x4* q4 = reinterpret_cast<const f32x4*>(a);
  f32x4 w;
  if constexpr (NT) w = __builtin_nontemporal_load(q4);
  else w = *q4;
#pragma unroll
  for (int q = 0; q < 4; ++q) x[q] = w[q];
}
template <bool NT>
__device__ __forceinline__ void load4(const uint16_t* a, float (&x)[kVec]) {
  const u32x2* q2 = reinterpret_cast<const u32x2*>(a);
  u32x2 w;
  if constexpr (NT) w = __builtin_nontemporal_load(q2);
  else w = *q2;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    x[2 * q] = __uint_as_float(w[q] << 16);
    x[2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
  }
}
template <bool NT>
__device__ __forceinline__ void store4(float* a, const float (&x)[kVec]) {
  const f32x4 w = {x[0], x[1], x[2], x[3]};
  if constexpr (NT) __builtin_nontemporal_store(w, reinterpret_cast<f32x4*>(a));
  else *reinterpret_cast<f32x4*>(a) = w;
}
template <bool NT>
__device__ __forceinline__ void store4(uint16_t* a, const float (&x)[kVec]) {
  const u32x2 w = {uint32_t(f2bf(x[0])) | (uint32_t(f2bf(x[1])) << 16),
                   uint32_t(f2bf(x[2])) | (uint32_t(f2bf(x[3])) << 16)};
  if constexpr (NT) __builtin_nontemporal_store(w, reinterpret_cast<u32x2*>(a));
  else *reinterpret_cast<u32x2*>(a) = w;
}

}  // namespace muon_adam
