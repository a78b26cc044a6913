// Global gradient norm over many tensors, and clipping.
//
// The tensors are cut into chunks of kChunk elements, numbered through; block
// b of the norm kernel sums the squares of chunks b, b + grid, ... and writes
// one fp64 partial sum, and every block of the scaling kernel adds the partial
// sums in one fixed order, so the norm does not depend on timing and all
// blocks use the same coefficient.  No atomics, no wait of one block on
// another.
//
// Bound by HBM: gradients larger than L2 have to be read twice, for the norm and
// to be scaled.  1.38 GB of bf16 into other tensors (2 reads, 1 write) 642 us,
// 6.5 TB/s; 54 tensors of 2.5 MB in all 19 us, most of it the two launches.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>
#include <vector>

#include "kd_internal.h"

namespace kd {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 16384;     // elements a block takes at a time
constexpr int kMaxGrid = 608;     // partial sums a launch writes at most
// tensors a launch takes: its kernel parameters hold them, and a short list costs
// less to launch
constexpr int kTable = 256, kShortTable = 64;

struct ClipTensor {
  const void* g;
  void* out;
  int64_t n;
};
template <int MOST>
struct ClipTable {
  ClipTensor t[MOST];
  uint32_t first[MOST + 1];  // first chunk of each tensor; [n]: number of chunks
  int n;
};

// The tensor chunk c belongs to.
template <int MOST>
__device__ __forceinline__ int clip_find(const ClipTable<MOST>& tab, uint32_t c) {
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

// A 16-byte vector of the tensor's elements.
template <class T>
struct Vec {
  static constexpr int N = 16 / (int)sizeof(T);
};
__device__ __forceinline__ void unpack(uint4 w, float* v, float) {
  v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y);
  v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void unpack(uint4 w, float* v, __nv_bfloat16) {
  v[0] = bf16lo(w.x), v[1] = bf16hi(w.x), v[2] = bf16lo(w.y), v[3] = bf16hi(w.y);
  v[4] = bf16lo(w.z), v[5] = bf16hi(w.z), v[6] = bf16lo(w.w), v[7] = bf16hi(w.w);
}
__device__ __forceinline__ uint4 pack(const float* v, float) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                    __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 pack(const float* v, __nv_bfloat16) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                    pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ bool aligned(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}
constexpr int kUnroll = 4;  // vectors a thread has in flight

// sum of (scale g)^2 over this thread's (at most 64) elements of a chunk
template <class T>
__device__ __forceinline__ float chunk_squares(const T* g, int n, float scale) {
  constexpr int N = Vec<T>::N;
  float s0 = 0.f, s1 = 0.f;
  int i0 = 0;
  if (aligned(g)) {
    const int vecs = n / N;
    i0 = vecs * N;
    const uint4* p = reinterpret_cast<const uint4*>(g);
    for (int j = threadIdx.x; j < vecs; j += kUnroll * kThreads) {
      uint4 w[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        w[u] = j + u * kThreads < vecs ? p[j + u * kThreads] : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        float v[N];
        unpack(w[u], v, T());
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          const float a = v[e] * scale, b = v[e + 1] * scale;
          s0 = fmaf(a, a, s0);
          s1 = fmaf(b, b, s1);
        }
      }
    }
  }
  for (int i = i0 + threadIdx.x; i < n; i += kThreads) {
    const float a = to_f(g[i]) * scale;
    s0 = fmaf(a, a, s0);
  }
  return s0 + s1;
}

// Bound by HBM: one read of everything.
template <class T, int MOST>
__global__ void __launch_bounds__(kThreads, 4)
    k_clip_norm(const __grid_constant__ ClipTable<MOST> tab, double* partial) {
  asm volatile("griddepcontrol.launch_dependents;");
  double sum = 0.0;
  for (uint32_t c = blockIdx.x; c < tab.first[tab.n]; c += gridDim.x) {
    const int k = clip_find(tab, c);
    const int64_t at = (int64_t)(c - tab.first[k]) * kChunk;
    const T* g = static_cast<const T*>(tab.t[k].g) + at;
    const int n = (int)min((int64_t)kChunk, tab.t[k].n - at);
    const float s = chunk_squares(g, n, 1.f);
    // squares at the ends of fp32's range: once more, scaled by a power of two
    // (elements below 2^-49 by 2^96: the least, 2^-149, squares to 2^-106)
    if (!(s <= 3e38f)) sum += (double)chunk_squares(g, n, 0x1p-72f) * 0x1p144;
    else if (s < 1e-30f) sum += (double)chunk_squares(g, n, 0x1p96f) * 0x1p-192;
    else sum += (double)s;
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// Launched to start while the norm kernel ends.  Takes the chunks backwards:
// the last ones it read are still in L2.
template <class T, int MOST>
__global__ void __launch_bounds__(kThreads, 4)
    k_clip_scale(const __grid_constant__ ClipTable<MOST> tab, const double* partial,
                 int n_partial, float max_norm, float* norm_out, uint32_t* status) {
  constexpr int N = Vec<T>::N;
  asm volatile("griddepcontrol.wait;" ::: "memory");
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
  const double ratio = clip ? (double)max_norm / norm : 1.0;
  float coef = (float)ratio, post = 1.f;
  // below fp32's normal numbers, where it would lose its bits: in two factors, the
  // second a power of two; the first is at most 1, and its product with an element
  // no smaller than the result
  const bool small = coef < 0x1p-126f;
  if (small) {
    post = ratio >= 0x1p-226 ? 0x1p-100f : 0x1p-149f;
    coef = (float)(ratio * (ratio >= 0x1p-226 ? 0x1p100 : 0x1p149));
  }
  const uint32_t chunks = tab.first[tab.n];
  for (uint32_t b = blockIdx.x; b < chunks; b += gridDim.x) {
    const uint32_t c = chunks - 1 - b;
    const int k = clip_find(tab, c);
    const ClipTensor& t = tab.t[k];
    if (!clip && t.out == t.g) continue;
    const int64_t at = (int64_t)(c - tab.first[k]) * kChunk;
    const T* g = static_cast<const T*>(t.g) + at;
    T* out = static_cast<T*>(t.out) + at;
    const int n = (int)min((int64_t)kChunk, t.n - at);
    int i0 = 0;
    if (aligned(g) && aligned(out)) {
      const int vecs = n / N;
      i0 = vecs * N;
      const uint4* p = reinterpret_cast<const uint4*>(g);
      uint4* o = reinterpret_cast<uint4*>(out);
      for (int j = threadIdx.x; j < vecs; j += kUnroll * kThreads) {
        uint4 w[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (j + u * kThreads < vecs) w[u] = p[j + u * kThreads];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          if (j + u * kThreads >= vecs) break;
          if (clip) {  // (not multiplied by 1: a NaN is passed on as it is)
            float v[N];
            unpack(w[u], v, T());
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] *= coef;
            if (small) {
#pragma unroll
              for (int e = 0; e < N; ++e) v[e] *= post;
            }
            w[u] = pack(v, T());
          }
          __stcs(&o[j + u * kThreads], w[u]);
        }
      }
    }
    for (int i = i0 + threadIdx.x; i < n; i += kThreads) {
      T v = g[i];
      if (clip) from_f(to_f(v) * coef * post, v);
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

template <class T, int MOST>
bool clip_run(const void* const* grads, void* const* outs, const int64_t* numel, int32_t n,
              float max_norm, float* norm_out, uint32_t* status, double* partial,
              cudaStream_t s) {
  auto table = [&](int32_t t0, ClipTable<MOST>& tab) {
    tab.n = (int)std::min<int32_t>(MOST, n - t0);
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
  bool told = false;  // the norm has been written
  ClipTable<MOST> tab;
  memset(&tab, 0, sizeof(tab));
  for (int32_t t0 = 0; t0 < n; t0 += MOST) {
    const uint32_t chunks = table(t0, tab);
    if (!chunks) continue;
    const int grid = (int)std::min<uint32_t>(chunks, kMaxGrid);
    note_launch();
    k_clip_norm<T, MOST><<<grid, kThreads, 0, s>>>(tab, partial + used);
    used += grid;
  }
  auto scale = [&](int grid, float* norm) {
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    // only right behind the norm kernel: a second scaling kernel (or one with
    // no norm kernel before it) follows in stream order
    cfg.numAttrs = used > 0 && !told ? 1 : 0;
    note_launch();
    return cudaLaunchKernelEx(&cfg, k_clip_scale<T, MOST>, tab, (const double*)partial, used, max_norm,
                              norm, status) == cudaSuccess;
  };
  for (int32_t t0 = 0; t0 < n && outs; t0 += MOST) {
    const uint32_t chunks = table(t0, tab);
    if (!chunks) continue;
    if (!scale((int)std::min<uint32_t>(chunks, kMaxGrid), told ? nullptr : norm_out)) return false;
    told = true;
  }
  if (!told) {  // norm only, or nothing in the tensors
    tab.n = 0;
    tab.first[0] = 0;
    if (!scale(1, norm_out)) return false;
  }
  return true;
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
  if ((reinterpret_cast<uintptr_t>(norm_out) | reinterpret_cast<uintptr_t>(dev_status)) % 4)
    return KD_ERR_INVALID_ARG;
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
  auto run = [&](auto few) {
    constexpr int MOST = decltype(few)::value ? kShortTable : kTable;
    return dtype == KD_BF16
               ? clip_run<__nv_bfloat16, MOST>(grads, outs, numel, n_tensors, max_norm, norm_out,
                                               dev_status, partial, s)
               : clip_run<float, MOST>(grads, outs, numel, n_tensors, max_norm, norm_out,
                                       dev_status, partial, s);
  };
  const bool ok = n_tensors <= kShortTable ? run(std::true_type{}) : run(std::false_type{});
  return ok && cudaGetLastError() == cudaSuccess ? KD_OK : KD_ERR_CUDA;
}
