// What the row kernels around the head share (kd_norm.cu, kd_embed.cu,
// kd_verify.cu): 16-byte vectors of either element type, and host-side checks
// and launches.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "kd_internal.h"
#include "kd_logprob.cuh"

namespace kd {

template <class T>
struct RowVec;
template <>
struct RowVec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(uint4 w, float* v) {
    v[0] = __uint_as_float(w.x), v[1] = __uint_as_float(w.y);
    v[2] = __uint_as_float(w.z), v[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 put(const float* v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  }
};
template <>
struct RowVec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(uint4 w, float* v) {
    v[0] = bf16lo(w.x), v[1] = bf16hi(w.x), v[2] = bf16lo(w.y), v[3] = bf16hi(w.y);
    v[4] = bf16lo(w.z), v[5] = bf16hi(w.z), v[6] = bf16lo(w.w), v[7] = bf16hi(w.w);
  }
  static __device__ __forceinline__ uint4 put(const float* v) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                      pack_bf16(v[6], v[7]));
  }
};

// A launch may start while the one before it on the stream ends (the kernel
// waits for it with chain_wait before it touches what that one wrote).
__device__ __forceinline__ void chain_next() {
  asm volatile("griddepcontrol.launch_dependents;");
}
__device__ __forceinline__ void chain_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------------ host side
template <class... P>
bool rows_launch(void (*kern)(P...), int64_t grid, int threads, size_t smem, bool chained,
                 cudaStream_t s, P... args) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = chained ? 1 : 0;
  note_launch();
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess;
}

inline int64_t rows_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
template <class... P>
bool rows_aligned(uintptr_t size, P... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ...) & (size - 1)) == 0;
}
inline bool rows_meet(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + nb && y < x + na;
}
// an output element by element over an input, or apart from it
inline bool rows_over(const void* out, const void* in, size_t bytes) {
  return out == in || !rows_meet(out, bytes, in, bytes);
}
inline bool rows_ws_ok(const void* ws, size_t have, size_t need) {
  return need == 0 || (ws && have >= need && reinterpret_cast<uintptr_t>(ws) % 256 == 0);
}
inline size_t rows_take(size_t& off, size_t bytes) {
  const size_t o = off;
  off = (off + bytes + 255) / 256 * 256;
  return o;
}
inline kd_status rows_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || !kd_device_supported(dev)) return KD_ERR_NO_DEVICE;
  return KD_OK;
}

}  // namespace kd
