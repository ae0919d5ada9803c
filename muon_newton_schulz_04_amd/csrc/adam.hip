// Adam branch of the optimizer step (include/muon_adam.h): one fused
// elementwise kernel over a whole list of parameter tensors, its plan
// (validated tensor table and work items in device memory) and the C ABI.
//
// The update (mhpq.cn, modded-nanogpt track_1_short technical guide, section
// 6.2: Adam with betas (0.9, 0.99) and per-group lr_mul / wd_mul for the
// parameters off the Muon path), per element, in fp32:
//   m = beta1 m + (1 - beta1) g;  v = beta2 v + (1 - beta2) g^2
//   p = p (1 - lr' wd') - (lr' / bc1) m / (sqrt(v) / sqrt(bc2) + eps)
// g times the plan's gradient factor where it has one (a clipped gradient, read
// from device memory: no pass of its own over the gradients), and
// with lr' = lr lr_mul, wd' = wd wd_mul, bc_i = 1 - beta_i^t (the bias-
// corrected form m/bc1 / (sqrt(v/bc2) + eps), rearranged so that the per-call
// factors 1/bc1 and 1/sqrt(bc2) are computed once on the host).
//
// HBM-bound: per element it reads p, g, m, v and writes p, m, v (22 bytes
// for bf16 parameters, 28 for fp32). What measured best on the 39.5 M
// elements of a GPT-2 124M's parameters off the Muon path (bf16, 869 MB;
// with the 79 MB read of their norm before it):
//  - a block takes 2048 consecutive elements, so that the blocks running at
//    one time sweep a compact range (16384 elements a block: 195 us, 4096:
//    181, 2048: 177);
//  - every access of a wave is one run of consecutive bytes (four elements a
//    lane: 8 bytes of bf16, 16 of float32), which alone changes nothing but
//    makes non-temporal loads and stores of whole lines possible: 159 us
//    (141 us of it this kernel, 6.2 TB/s). With eight elements a lane, whose
//    float32 accesses touch every other 16 bytes, the same hints took 210 us.
// Accesses are those of an element's alignment, whatever the tensor's.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include "../../include/muon_adam.h"
#include "adam_elem.hpp"

namespace muon_adam {

constexpr int kChunk = 16384;  // the unit of muon_adam_work_items; blocks are kBlock elements
constexpr int kThreads = 256;
constexpr int kRuns = 2;       // runs of kVec elements per thread, kThreads * kVec apart
constexpr int kBlock = kThreads * kVec * kRuns;
constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 1;  // a launch holds under 2^32 threads

struct Tensor {
  void* p;
  const void* g;
  float* m;
  float* v;
  int64_t numel;
  float lr_mul, wd_mul;
};

// A block's work.
struct Item {
  int32_t t;    // tensor index
  int32_t run;  // elements run * kBlock .. + kBlock - 1 of the tensor
};

struct Args {
  const Tensor* ts;
  const Item* items;
  float lr, b1, b2, eps, wd;
  float inv_bc1, inv_sqrt_bc2;  // 1 / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  const float* gscale;          // gradients are multiplied by *gscale (nullptr: by one)
};

// The four arrays of elements e .. e + 3, and back with their update.
// (The pointers by value: through a reference to Tensor they become flat
// accesses; Adam on one block's vectors 2.6 us for 2.3.)
template <bool NT, typename T>
__device__ __forceinline__ void load_vec4(const T* p, const T* g, const float* m, const float* v, Vec4& x) {
  load4<NT>(p, x.p);
  load4<NT>(g, x.g);
  load4<NT>(m, x.m);
  load4<NT>(v, x.v);
}
template <bool NT, typename T>
__device__ __forceinline__ void update_vec4(T* p, float* m, float* v, Vec4& x, const Consts& k) {
#pragma unroll
  for (int q = 0; q < kVec; ++q) x.p[q] = adam_elem(x.p[q], x.g[q], x.m[q], x.v[q], k);
  store4<NT>(m, x.m);
  store4<NT>(v, x.v);
  store4<NT>(p, x.p);
}

// One element.
template <typename T>
__device__ __forceinline__ void update1(T* p, const T* g, float* m, float* v, const Consts& k) {
  float mx = *m, vx = *v;
  const float px = adam_elem(PElem<T>::load(p, 0), PElem<T>::load(g, 0), mx, vx, k);
  *m = mx;
  *v = vx;
  PElem<T>::store(p, 0, px);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void adam_kernel(Args A) {
  const Item it = A.items[blockIdx.x];
  const Tensor t = A.ts[it.t];
  const int64_t base = int64_t(it.run) * kBlock;
  const float lr_e = A.lr * t.lr_mul;
  Consts k;
  k.b1 = A.b1;
  k.c1 = 1.f - A.b1;
  k.b2 = A.b2;
  k.c2 = 1.f - A.b2;
  k.eps = A.eps;
  k.keep = 1.f - lr_e * (A.wd * t.wd_mul);
  k.step = lr_e * A.inv_bc1;
  k.isb2 = A.inv_sqrt_bc2;
  k.gs = A.gscale ? *A.gscale : 1.f;
  T* const p = static_cast<T*>(t.p) + base;
  const T* const g = static_cast<const T*>(t.g) + base;
  float* const m = t.m + base;
  float* const v = t.v + base;
  const int64_t left = t.numel - base;
  Vec4 x[kRuns];
  if (left >= kBlock) {
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
      const int e = (r * kThreads + threadIdx.x) * kVec;
      load_vec4<true>(p + e, g + e, m + e, v + e, x[r]);
    }
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
      const int e = (r * kThreads + threadIdx.x) * kVec;
      update_vec4<true>(p + e, m + e, v + e, x[r], k);
    }
    return;
  }
  // A tensor's last elements: one a lane where that is enough (10000 tensors
  // of 100 elements 9.0 us, 9.8 in vectors), else whole vectors and one element
  // a lane for what is behind them, all loaded before the first store. A loop
  // of one element a lane, each round waited for, took 6.1 us for 4.5 on 300
  // tensors of 2000 bf16 elements and 3.6 for 2.7 on one.
  const int n = static_cast<int>(left), tid = threadIdx.x;
  if (n <= kThreads) {
    if (tid < n) update1(p + tid, g + tid, m + tid, v + tid, k);
    return;
  }
  const int nv = n / kVec * kVec, z = nv + tid;
#pragma unroll
  for (int r = 0; r < kRuns; ++r) {
    const int e = (r * kThreads + tid) * kVec;
    if (e < nv) load_vec4<false>(p + e, g + e, m + e, v + e, x[r]);
  }
  float zp = 0.f, zg = 0.f, zm = 0.f, zv = 0.f;
  if (z < n) {
    zp = PElem<T>::load(p, z);
    zg = PElem<T>::load(g, z);
    zm = m[z];
    zv = v[z];
  }
#pragma unroll
  for (int r = 0; r < kRuns; ++r) {
    const int e = (r * kThreads + tid) * kVec;
    if (e < nv) update_vec4<false>(p + e, m + e, v + e, x[r], k);
  }
  if (z < n) {
    zp = adam_elem(zp, zg, zm, zv, k);
    m[z] = zm;
    v[z] = zv;
    PElem<T>::store(p, z, zp);
  }
}

// ------------------------------------------------------------------ host

struct Interval {
  uintptr_t lo, hi;
  bool write;
};

// *blocks receives the kernel's blocks, *items what muon_adam_work_items counts.
muon_status build(const muon_adam_tensor* ts, int32_t n, muon_dtype dtype, std::vector<Tensor>* out,
                  int64_t* blocks, int64_t* items) {
  if (dtype != MUON_F32 && dtype != MUON_BF16) return MUON_E_DTYPE;
  if (n < 0 || n > MUON_ADAM_MAX_TENSORS) return MUON_E_SHAPE;
  if (n > 0 && ts == nullptr) return MUON_E_INVALID;
  const size_t es = dtype == MUON_F32 ? 4 : 2;
  std::vector<Interval> iv;
  out->assign(static_cast<size_t>(n), Tensor{});
  *blocks = *items = 0;
  for (int32_t i = 0; i < n; ++i) {
    const muon_adam_tensor& T = ts[i];
    if (T.numel < 0 || T.numel > MUON_ADAM_MAX_NUMEL) return MUON_E_SHAPE;
    if (T.numel == 0) continue;
    if (!T.param || !T.grad || !T.exp_avg || !T.exp_avg_sq) return MUON_E_INVALID;
    if (!std::isfinite(T.lr_mul) || !std::isfinite(T.wd_mul)) return MUON_E_INVALID;
    auto addr = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
    if (addr(T.param) % es || addr(T.grad) % es || addr(T.exp_avg) % 4 || addr(T.exp_avg_sq) % 4)
      return MUON_E_ALIGN;
    const uintptr_t pb = static_cast<uintptr_t>(T.numel) * es, sb = static_cast<uintptr_t>(T.numel) * 4;
    iv.push_back({addr(T.param), addr(T.param) + pb, true});
    iv.push_back({addr(T.grad), addr(T.grad) + pb, false});
    iv.push_back({addr(T.exp_avg), addr(T.exp_avg) + sb, true});
    iv.push_back({addr(T.exp_avg_sq), addr(T.exp_avg_sq) + sb, true});
    Tensor& D = (*out)[i];
    D.p = T.param;
    D.g = T.grad;
    D.m = T.exp_avg;
    D.v = T.exp_avg_sq;
    D.numel = T.numel;
    D.lr_mul = T.lr_mul;
    D.wd_mul = T.wd_mul;
    *items += (T.numel + kChunk - 1) / kChunk;
    *blocks += (T.numel + kBlock - 1) / kBlock;
  }
  std::sort(iv.begin(), iv.end(), [](const Interval& x, const Interval& y) { return x.lo < y.lo; });
  uintptr_t max_hi_any = 0, max_hi_w = 0;
  for (const Interval& x : iv) {
    if (x.lo < max_hi_w || (x.write && x.lo < max_hi_any)) return MUON_E_INVALID;
    max_hi_any = std::max(max_hi_any, x.hi);
    if (x.write) max_hi_w = std::max(max_hi_w, x.hi);
  }
  return MUON_OK;
}

}  // namespace muon_adam

struct muon_adam_plan_s {
  int device = -1;
  muon_dtype dtype = MUON_BF16;
  void* dmem = nullptr;
  const muon_adam::Tensor* d_ts = nullptr;
  const muon_adam::Item* d_items = nullptr;
  int64_t nblocks = 0;
  const float* gscale = nullptr;  // muon_adam_plan_set_grad_scale
};

extern "C" {

muon_status muon_adam_work_items(const muon_adam_tensor* ts, int32_t n, muon_dtype dtype,
                                 int64_t* items) {
  if (items == nullptr) return MUON_E_INVALID;
  try {
    std::vector<muon_adam::Tensor> t;
    int64_t blocks = 0, count = 0;
    const muon_status st = muon_adam::build(ts, n, dtype, &t, &blocks, &count);
    if (st == MUON_OK) *items = count;
    return st;
  } catch (...) {
    return MUON_E_ALLOC;
  }
}

muon_status muon_adam_plan_create(const muon_adam_tensor* ts, int32_t n, muon_dtype dtype,
                                  muon_adam_plan** plan) {
  if (plan == nullptr) return MUON_E_INVALID;
  *plan = nullptr;
  std::vector<muon_adam::Tensor> t;
  std::vector<char> h;  // the tensor table, then the blocks
  int64_t nblocks = 0;
  size_t tb = 0, bytes = 0;
  try {
    int64_t count = 0;
    const muon_status st = muon_adam::build(ts, n, dtype, &t, &nblocks, &count);
    if (st != MUON_OK) return st;
    if (nblocks > muon_adam::kMaxBlocks) return MUON_E_SHAPE;
    tb = (sizeof(muon_adam::Tensor) * std::max<size_t>(1, t.size()) + 255) / 256 * 256;
    bytes = tb + sizeof(muon_adam::Item) * static_cast<size_t>(std::max<int64_t>(1, nblocks));
    h.assign(bytes, 0);
  } catch (...) {
    return MUON_E_ALLOC;
  }
  int dev = 0;
  hipDeviceProp_t prop;
  if (hipGetDevice(&dev) != hipSuccess || hipGetDeviceProperties(&prop, dev) != hipSuccess ||
      std::strncmp(prop.gcnArchName, "gfx950", 6) != 0)
    return MUON_E_DEVICE;
  muon_adam_plan_s* p = new (std::nothrow) muon_adam_plan_s();
  if (!p) return MUON_E_ALLOC;
  p->device = dev;
  p->dtype = dtype;
  p->nblocks = nblocks;
  if (!t.empty()) std::memcpy(h.data(), t.data(), sizeof(muon_adam::Tensor) * t.size());
  char* at = h.data() + tb;
  for (int32_t i = 0; i < n; ++i)
    for (int64_t r = 0; r * muon_adam::kBlock < t[i].numel; ++r, at += sizeof(muon_adam::Item)) {
      const muon_adam::Item it = {i, static_cast<int32_t>(r)};
      std::memcpy(at, &it, sizeof(it));
    }
  if (hipMalloc(&p->dmem, bytes) != hipSuccess) {
    (void)hipGetLastError();
    delete p;
    return MUON_E_ALLOC;
  }
  if (hipMemcpy(p->dmem, h.data(), bytes, hipMemcpyHostToDevice) != hipSuccess) {
    (void)hipGetLastError();
    (void)hipFree(p->dmem);
    delete p;
    return MUON_E_DEVICE;
  }
  p->d_ts = static_cast<const muon_adam::Tensor*>(p->dmem);
  p->d_items = reinterpret_cast<const muon_adam::Item*>(static_cast<char*>(p->dmem) + tb);
  *plan = p;
  return MUON_OK;
}

muon_status muon_adam_plan_step(muon_adam_plan* plan, const muon_adam_config* cfg, void* stream) {
  if (plan == nullptr || cfg == nullptr) return MUON_E_INVALID;
  if (!std::isfinite(cfg->lr) || !std::isfinite(cfg->beta1) || !std::isfinite(cfg->beta2) ||
      !std::isfinite(cfg->eps) || !std::isfinite(cfg->wd))
    return MUON_E_INVALID;
  if (cfg->beta1 < 0.f || cfg->beta1 >= 1.f || cfg->beta2 < 0.f || cfg->beta2 >= 1.f ||
      cfg->eps < 0.f || cfg->step < 1)
    return MUON_E_INVALID;
  if (plan->nblocks == 0) return MUON_OK;
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev != plan->device) return MUON_E_DEVICE;
  muon_adam::Args a{};
  a.ts = plan->d_ts;
  a.items = plan->d_items;
  a.lr = cfg->lr;
  a.b1 = cfg->beta1;
  a.b2 = cfg->beta2;
  a.eps = cfg->eps;
  a.wd = cfg->wd;
  a.gscale = plan->gscale;
  a.inv_bc1 = static_cast<float>(1.0 / (1.0 - std::pow(double(cfg->beta1), double(cfg->step))));
  a.inv_sqrt_bc2 =
      static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(double(cfg->beta2), double(cfg->step))));
  hipStream_t s = static_cast<hipStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(plan->nblocks)), block(muon_adam::kThreads);
  if (plan->dtype == MUON_F32)
    hipLaunchKernelGGL(muon_adam::adam_kernel<float>, grid, block, 0, s, a);
  else
    hipLaunchKernelGGL(muon_adam::adam_kernel<uint16_t>, grid, block, 0, s, a);
  return hipGetLastError() == hipSuccess ? MUON_OK : MUON_E_LAUNCH;
}

muon_status muon_adam_plan_set_grad_scale(muon_adam_plan* plan, const float* scale) {
  if (plan == nullptr) return MUON_E_INVALID;
  if (reinterpret_cast<uintptr_t>(scale) % 4 != 0) return MUON_E_ALIGN;
  plan->gscale = scale;
  return MUON_OK;
}

void muon_adam_plan_destroy(muon_adam_plan* plan) {
  if (!plan) return;
  (void)hipDeviceSynchronize();
  if (plan->dmem) (void)hipFree(plan->dmem);
  delete plan;
}

}  // extern "C"
