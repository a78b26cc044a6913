// Global gradient norm over many tensors, and clipping.
//
// The tensors are cut into chunks of kChunk elements, numbered through; block
// b of the norm kernel sums the squares of chunks b, b + grid, ... and writes
// one fp64 partial sum, and every block of the scaling kernel adds the partial
// sums in one fixed order, so the norm does not depend on timing and all
// blocks use the same coefficient.  No atomics, no wait of one block on
// another.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <vector>

#include "kd_internal.h"

namespace kd {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 16384;     // elements a block takes at a time
constexpr int kMaxGrid = 608;     // partial sums a launch writes at most
constexpr int kTable = 256;       // tensors a launch takes (its kernel parameters hold them)

struct ClipTensor {
  const void* g;
  void* out;
  int64_t n;
};
struct ClipTable {
  ClipTensor t[kTable];
  uint32_t first[kTable + 1];  // first chunk of each tensor; [n]: number of chunks
  int n;
};

// The tensor chunk c belongs to.
__device__ __forceinline__ int clip_find(const ClipTable& tab, uint32_t c) {
  int lo = 0, hi = tab.n;  // first[lo] <= c < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tab.first[mid] <= c) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16& o) { o = __float2bfloat16(v); }

__device__ double block_sum(double v) {
  __shared__ double red[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  for (int w = 0; w < kThreads / 32; ++w) v += red[w];
  return v;
}

// sum of (scale g)^2 over this thread's elements of a chunk
template <class T>
__device__ __forceinline__ float chunk_squares(const T* g, int n, float scale, bool& any) {
  float s = 0.f;
  bool a = false;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const float v = to_f(g[i]) * scale;
    a |= v != 0.f;
    s = fmaf(v, v, s);
  }
  any = a;
  return s;
}

template <class T>
__global__ void __launch_bounds__(kThreads) k_clip_norm(const __grid_constant__ ClipTable tab,
                                                        double* partial) {
  double sum = 0.0;
  for (uint32_t c = blockIdx.x; c < tab.first[tab.n]; c += gridDim.x) {
    const ClipTensor& t = tab.t[clip_find(tab, c)];
    const int64_t at = (int64_t)(c - tab.first[clip_find(tab, c)]) * kChunk;
    const T* g = static_cast<const T*>(t.g) + at;
    const int n = (int)min((int64_t)kChunk, t.n - at);
    bool any;
    float s = chunk_squares(g, n, 1.f, any);
    double d = (double)s;
    // squares outside fp32's range: once more, scaled by a power of two
    if (!(s <= 3e38f)) {
      bool unused;
      d = (double)chunk_squares(g, n, 0x1p-72f, unused) * 0x1p144;
    } else if (s < 1e-30f && any) {
      bool unused;
      d = (double)chunk_squares(g, n, 0x1p72f, unused) * 0x1p-144;
    }
    sum += d;
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

template <class T>
__global__ void __launch_bounds__(kThreads) k_clip_scale(const __grid_constant__ ClipTable tab,
                                                         const double* partial, int n_partial,
                                                         float max_norm, float* norm_out,
                                                         uint32_t* status) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < n_partial; i += kThreads) sum += partial[i];
  sum = block_sum(sum);
  const double norm = sqrt(sum);
  const bool finite = norm <= 1.7976931348623157e308;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (norm_out) *norm_out = (float)norm;
    if (!finite) set_status(status, KD_DEV_NONFINITE);
  }
  const bool clip = finite && norm > (double)max_norm;
  const float coef = clip ? (float)((double)max_norm / norm) : 1.f;
  for (uint32_t c = blockIdx.x; c < tab.first[tab.n]; c += gridDim.x) {
    const int k = clip_find(tab, c);
    const ClipTensor& t = tab.t[k];
    if (!clip && t.out == t.g) continue;
    const int64_t at = (int64_t)(c - tab.first[k]) * kChunk;
    const T* g = static_cast<const T*>(t.g) + at;
    T* out = static_cast<T*>(t.out) + at;
    const int n = (int)min((int64_t)kChunk, t.n - at);
    for (int i = threadIdx.x; i < n; i += kThreads) {
      T v = g[i];
      if (clip) from_f(to_f(v) * coef, v);
      out[i] = v;
    }
  }
}

size_t clip_launches(int32_t n) { return n ? ((size_t)n + kTable - 1) / kTable : 1; }

// chunks are numbered in 32 bits within a launch
kd_status clip_check(const int64_t* numel, int32_t n) {
  if (n < 0 || (n > 0 && !numel)) return KD_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i)
    if (numel[i] < 0 || numel[i] > (int64_t)1 << 36) return KD_ERR_INVALID_ARG;
  return KD_OK;
}

// No out may overlap another tensor's gradient or out (the same tensor twice
// among them): it would be scaled twice, or read after it was written.
bool clip_disjoint(const void* const* grads, void* const* outs, const int64_t* numel, int32_t n,
                   size_t esz) {
  struct Span {
    uintptr_t lo, hi;
    bool out;
  };
  std::vector<Span> v;
  v.reserve(2 * (size_t)n);
  for (int32_t i = 0; i < n; ++i) {
    if (numel[i] == 0) continue;
    const uintptr_t b = (uintptr_t)numel[i] * esz;
    const uintptr_t o = reinterpret_cast<uintptr_t>(outs[i]);
    const uintptr_t g = reinterpret_cast<uintptr_t>(grads[i]);
    v.push_back(Span{o, o + b, true});
    if (g != o) v.push_back(Span{g, g + b, false});
  }
  std::sort(v.begin(), v.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
  uintptr_t end_out = 0, end_any = 0;
  for (const Span& x : v) {
    if (x.lo < (x.out ? end_any : end_out)) return false;
    end_any = std::max(end_any, x.hi);
    if (x.out) end_out = std::max(end_out, x.hi);
  }
  return true;
}

template <class T>
void clip_run(const void* const* grads, void* const* outs, const int64_t* numel, int32_t n,
              float max_norm, float* norm_out, uint32_t* status, double* partial,
              cudaStream_t s) {
  auto table = [&](int32_t t0, ClipTable& tab) {
    tab.n = (int)std::min<int32_t>(kTable, n - t0);
    uint32_t c = 0;
    for (int i = 0; i < tab.n; ++i) {
      tab.t[i] = ClipTensor{grads[t0 + i], outs ? outs[t0 + i] : nullptr, numel[t0 + i]};
      tab.first[i] = c;
      c += (uint32_t)((numel[t0 + i] + kChunk - 1) / kChunk);
    }
    tab.first[tab.n] = c;
    return c;
  };
  int used = 0;
  ClipTable tab;
  memset(&tab, 0, sizeof(tab));
  for (int32_t t0 = 0; t0 < n; t0 += kTable) {
    const uint32_t chunks = table(t0, tab);
    if (!chunks) continue;
    const int grid = (int)std::min<uint32_t>(chunks, kMaxGrid);
    note_launch();
    k_clip_norm<T><<<grid, kThreads, 0, s>>>(tab, partial + used);
    used += grid;
  }
  bool told = false;  // the norm has been written
  for (int32_t t0 = 0; t0 < n && outs; t0 += kTable) {
    const uint32_t chunks = table(t0, tab);
    if (!chunks) continue;
    note_launch();
    k_clip_scale<T><<<(int)std::min<uint32_t>(chunks, kMaxGrid), kThreads, 0, s>>>(
        tab, partial, used, max_norm, told ? nullptr : norm_out, status);
    told = true;
  }
  if (!told) {  // norm only, or nothing in the tensors
    tab.n = 0;
    tab.first[0] = 0;
    note_launch();
    k_clip_scale<T><<<1, kThreads, 0, s>>>(tab, partial, used, max_norm, norm_out, status);
  }
}

}  // namespace
}  // namespace kd

using namespace kd;

extern "C" kd_status kd_clip_grad_norm_workspace_size(const int64_t* numel, int32_t n_tensors,
                                                      size_t* bytes) {
  const kd_status st = clip_check(numel, n_tensors);
  if (st != KD_OK || !bytes) return KD_ERR_INVALID_ARG;
  *bytes = clip_launches(n_tensors) * kMaxGrid * sizeof(double);
  return KD_OK;
}

extern "C" kd_status kd_clip_grad_norm(const void* const* grads, void* const* outs,
                                       const int64_t* numel, int32_t n_tensors, int32_t dtype,
                                       float max_norm, float* norm_out, uint32_t* dev_status,
                                       void* workspace, size_t ws_bytes, void* stream) {
  size_t need = 0;
  if (kd_clip_grad_norm_workspace_size(numel, n_tensors, &need) != KD_OK)
    return KD_ERR_INVALID_ARG;
  if (dtype != KD_BF16 && dtype != KD_FP32) return KD_ERR_INVALID_ARG;
  if (!(std::isfinite(max_norm) && max_norm >= 0.f)) return KD_ERR_INVALID_ARG;
  const size_t esz = dtype == KD_BF16 ? 2 : 4;
  for (int32_t i = 0; i < n_tensors; ++i) {
    if (numel[i] == 0) continue;
    if (!grads || !grads[i] || (outs && !outs[i])) return KD_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(grads[i]) % esz) return KD_ERR_INVALID_ARG;
    if (outs && reinterpret_cast<uintptr_t>(outs[i]) % esz) return KD_ERR_INVALID_ARG;
  }
  try {
    if (outs && !clip_disjoint(grads, outs, numel, n_tensors, esz)) return KD_ERR_INVALID_ARG;
  } catch (...) {
    return KD_ERR_INVALID_ARG;  // no host memory for the list
  }
  if (!workspace || ws_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 256)
    return KD_ERR_WORKSPACE;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || !kd_device_supported(dev)) return KD_ERR_NO_DEVICE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* partial = static_cast<double*>(workspace);
  if (dtype == KD_BF16)
    clip_run<__nv_bfloat16>(grads, outs, numel, n_tensors, max_norm, norm_out, dev_status,
                            partial, s);
  else
    clip_run<float>(grads, outs, numel, n_tensors, max_norm, norm_out, dev_status, partial, s);
  return cudaGetLastError() == cudaSuccess ? KD_OK : KD_ERR_CUDA;
}
