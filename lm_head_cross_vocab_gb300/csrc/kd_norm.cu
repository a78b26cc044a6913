// Root-mean-square norm of rows with the residual's addition, and its backward.
//
//   s = x + residual,  r = (mean s^2 + eps)^-1/2,  h = s r w
//   d_x = r g - (s r) r m + d_sum,  g = d_h w,  m = r mean(g s);   d_w = sum_n d_h s r
//
// (s r is of size 1 and m of g's, whatever the row's; an r^3 would leave fp32's range
// from rows of 2^42 on.)
// TPR threads hold a row in registers, so every tensor is read once and the
// sums of a row (s^2; backward: also g s) are one reduction.  Rows of whole
// 16-byte vectors move as such; others (an odd width, a view at an odd offset)
// element by element, neighbouring threads on neighbouring elements.
// The backward's blocks take rows in turn and keep their share of d_w in
// registers; a second kernel adds the blocks' shares in a fixed order.
// Bound by HBM: 16384 x 4096 bf16 with a residual 78.5 us, 6.8 TB/s; its backward
// 69 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "kd_internal.h"
#include "kd_rows.cuh"

namespace kd {
namespace {

struct NormArgs {
  const void *x, *res, *w, *dh;  // backward: x is s, res is d_sum
  void *sum, *h;                 // backward: h is d_x
  float* part;                   // backward: [grid][d] shares of d_w, or NULL
  int64_t n;
  int d;
  float eps, off;
};

// A thread's elements of a row: VPT vectors, TPR apart, or VPT * N elements,
// TPR apart (held as they came: packed, each load would be waited for before the
// next).  Zero beyond the row.
template <class T, int TPR, int VPT, bool VEC>
struct RowPart {
  static constexpr int N = RowVec<T>::N, E = VPT * N;
  uint4 w[VEC ? VPT : 1];
  T x[VEC ? 1 : E];

  __device__ __forceinline__ void load(const T* p, int d, int t) {
    if constexpr (VEC) {
      const uint4* q = reinterpret_cast<const uint4*>(p);
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        w[i] = i * TPR + t < d / N ? q[i * TPR + t] : make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (e * TPR + t < d) x[e] = p[e * TPR + t];
        else from_f(0.f, x[e]);
      }
    }
  }
  __device__ __forceinline__ void get(int i, float* v) const {
    if constexpr (VEC) {
      RowVec<T>::get(w[i], v);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = to_f(x[i * N + e]);
    }
  }
  // the values of vector i
  static __device__ __forceinline__ void store(T* p, int d, int t, int i, const float* v) {
    if constexpr (VEC) {
      if (i * TPR + t < d / N) reinterpret_cast<uint4*>(p)[i * TPR + t] = RowVec<T>::put(v);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int at = (i * N + e) * TPR + t;
        if (at < d) from_f(v[e], p[at]);
      }
    }
  }
  // column of element e of vector i
  static __device__ __forceinline__ int column(int t, int i, int e) {
    return VEC ? (i * TPR + t) * N + e : (i * N + e) * TPR + t;
  }
};

constexpr int norm_block(int tpr) { return tpr < 128 ? 128 : tpr; }
// Blocks of the backward on an SM.  The rows on their way keep memory busy, not the
// threads, and each block leaves a share of d_w to add (16384 x 2048 bf16, 128 threads
// a row: 47.2 us with two blocks, 49.3 with three, 52.0 with four; short rows need
// the threads: 50000 x 256 27.1 us with four, 31.7 with two).  Threads of 20 and 24
// elements need more than 128 registers: three blocks of 128, one of 256 (8000 x 5120
// 58 us; two that spill 74).
constexpr int norm_per_sm(int tpr, int vpt) {
  const bool many = vpt == 3 || vpt == 5;
  return tpr <= 64 ? (many ? 3 : 4) : tpr <= 128 ? 2 : tpr <= 256 ? (many ? 1 : 2) : 1;
}

// Sums of a row over its TPR threads, in every one of them.  `red` holds
// TPR / 32 pairs; a block that calls it again passes the other of two buffers.
template <int TPR>
__device__ __forceinline__ float2 row_sums(float2 v, float2* red) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[threadIdx.x / TPR * (TPR / 32) + (threadIdx.x & (TPR / 32 - 1))];
#pragma unroll
    for (int o = TPR / 64; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
  }
  return v;
}

template <class T, int TPR, int VPT, bool VEC>
__global__ void __launch_bounds__(norm_block(TPR)) k_norm_fwd(NormArgs a) {
  using P = RowPart<T, TPR, VPT, VEC>;
  constexpr int N = P::N;
  __shared__ float2 red[32];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (norm_block(TPR) / TPR) + threadIdx.x / TPR;
  const bool on = row < a.n;
  const int64_t at = (on ? row : 0) * a.d;
  P x, r, w;
  x.load(static_cast<const T*>(a.x) + at, a.d, t);
  if (a.res) r.load(static_cast<const T*>(a.res) + at, a.d, t);
  w.load(static_cast<const T*>(a.w), a.d, t);
  float s[P::E], sq = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    x.get(i, s + i * N);
    if (a.res) {
      float v[N];
      r.get(i, v);
#pragma unroll
      for (int e = 0; e < N; ++e) s[i * N + e] += v[e];
    }
#pragma unroll
    for (int e = 0; e < N; ++e) sq = fmaf(s[i * N + e], s[i * N + e], sq);
    if (a.sum && on) P::store(static_cast<T*>(a.sum) + at, a.d, t, i, s + i * N);
  }
  sq = row_sums<TPR>(make_float2(sq, 0.f), red).x;
  const float scale = 1.f / sqrtf(sq / (float)a.d + a.eps);
  if (!on) return;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    float v[N];
    w.get(i, v);
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = s[i * N + e] * scale * (v[e] + a.off);
    P::store(static_cast<T*>(a.h) + at, a.d, t, i, v);
  }
}

// Backward.  With whole vectors (and rows that leave room for it) a thread's own
// vectors of the rows to come are on their way into shared memory, stages - 1 rows
// ahead: 8 or 16 warps an SM hold too few loads in their registers to keep memory
// busy (16384 x 4096 bf16, d_x alone: 89 us without, 64 us with them, 6.3 TB/s).  Each
// thread reads only what it copied itself, so the ring needs no barrier.
template <int TPR, int VPT, bool VEC>
constexpr bool norm_ring() {
  return VEC && TPR * VPT <= 2048;
}
template <class T, int TPR, int VPT, bool VEC>
__global__ void __launch_bounds__(norm_block(TPR), norm_per_sm(TPR, VPT)) k_norm_bwd(NormArgs a, int stages) {
  using P = RowPart<T, TPR, VPT, VEC>;
  constexpr int N = P::N, BLOCK = norm_block(TPR), ROWS = BLOCK / TPR;
  constexpr bool RING = norm_ring<TPR, VPT, VEC>();
  extern __shared__ uint4 ring[];  // [stages][2 or 3 tensors][VPT][BLOCK]
  __shared__ float2 red[2][32];
  chain_next();
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int64_t step = (int64_t)gridDim.x * ROWS, begin = (int64_t)blockIdx.x * ROWS;
  auto copy = [&](int slot, const void* tensor, int64_t row) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(tensor) + row * a.d);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (i * TPR + t < a.d / N) {
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(&ring[(slot * VPT + i) * BLOCK + threadIdx.x]);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src + i * TPR + t)
                     : "memory");
      }
  };
  const int tensors = a.res ? 3 : 2;
  auto ask = [&](int stage, int64_t first) {
    if (first + sub < a.n) {
      copy(stage * tensors, a.x, first + sub);
      copy(stage * tensors + 1, a.dh, first + sub);
      if (a.res) copy(stage * tensors + 2, a.res, first + sub);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto take = [&](int slot, P& p) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      p.w[i] = i * TPR + t < a.d / N ? ring[(slot * VPT + i) * BLOCK + threadIdx.x]
                                     : make_uint4(0, 0, 0, 0);
  };
  if constexpr (RING)
    for (int q = 0; q < stages; ++q) ask(q, begin + q * step);
  P w;
  w.load(static_cast<const T*>(a.w), a.d, t);
  float dw[P::E];
#pragma unroll
  for (int e = 0; e < P::E; ++e) dw[e] = 0.f;
  const float inv_d = 1.f / (float)a.d;
  int turn = 0, stage = 0;
  for (int64_t first = begin; first < a.n; first += step) {
    const bool on = first + sub < a.n;
    const int64_t at = (on ? first + sub : 0) * a.d;
    P s, g, up;
    if constexpr (RING) {
      if (stages == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
      else if (stages == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
      else if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
      else asm volatile("cp.async.wait_group 0;" ::: "memory");
      take(stage * tensors, s);
      take(stage * tensors + 1, g);
      if (a.res) take(stage * tensors + 2, up);
    } else {
      s.load(static_cast<const T*>(a.x) + at, a.d, t);
      g.load(static_cast<const T*>(a.dh) + at, a.d, t);
      if (a.res) up.load(static_cast<const T*>(a.res) + at, a.d, t);
    }
    float2 sums = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float sv[N], gv[N], wv[N];
      s.get(i, sv);
      g.get(i, gv);
      w.get(i, wv);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        sums.x = fmaf(sv[e], sv[e], sums.x);
        sums.y = fmaf(gv[e] * (wv[e] + a.off), sv[e], sums.y);
      }
    }
    sums = row_sums<TPR>(sums, red[turn]);
    turn ^= 1;
    if (on) {
      const float r = 1.f / sqrtf(sums.x * inv_d + a.eps);
      const float rm = r * (r * (sums.y * inv_d));
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float sv[N], gv[N], wv[N];
        s.get(i, sv);
        g.get(i, gv);
        w.get(i, wv);
        float o[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
          // (s r is in both gradients, or r g is: with 64 registers the latter spills
          // less, 2048 x 32768 bf16 223 us and 434; else the former is no slower, 8000 x
          // 5120 51.5 us and 54.0)
          if constexpr (TPR < 1024) {
            const float y = sv[e] * r;
            o[e] = fmaf(-y, rm, r * (gv[e] * (wv[e] + a.off)));
            dw[i * N + e] = fmaf(gv[e], y, dw[i * N + e]);
          } else {
            const float y = gv[e] * r;
            o[e] = fmaf(-(sv[e] * r), rm, y * (wv[e] + a.off));
            dw[i * N + e] = fmaf(y, sv[e], dw[i * N + e]);
          }
        }
        if (a.res) {
          float uv[N];
          up.get(i, uv);
#pragma unroll
          for (int e = 0; e < N; ++e) o[e] += uv[e];
        }
        if (a.h) P::store(static_cast<T*>(a.h) + at, a.d, t, i, o);
      }
    }
    if constexpr (RING) {  // (the slot's values have all been used)
      ask(stage, first + stages * step);
      stage = stage + 1 == stages ? 0 : stage + 1;
    }
  }
  if (!a.part) return;
  // the block's share: its row groups in order
  if constexpr (ROWS > 1) {
    __shared__ float share[TPR * P::E];
    for (int q = 0; q < ROWS; ++q) {
      if (sub == q) {
#pragma unroll
        for (int e = 0; e < P::E; ++e) {
          if (q) dw[e] += share[e * TPR + t];
          share[e * TPR + t] = dw[e];
        }
      }
      __syncthreads();
    }
    if (sub != ROWS - 1) return;
  }
  float* part = a.part + (int64_t)blockIdx.x * a.d;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int c = P::column(t, i, e);
      if (c < a.d) part[c] = dw[i * N + e];
    }
}

// d_w: 32 columns a block; a warp adds every 32nd share, then the warps' sums in
// order.
constexpr int kWeightThreads = 1024, kWeightAhead = 10;
template <class T>
__global__ void __launch_bounds__(kWeightThreads) k_norm_weight(const float* part, int parts, int d, T* dw) {
  constexpr int kWarps = kWeightThreads / 32;
  __shared__ float sum[kWarps][33];
  chain_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  for (int p = warp; p < parts; p += kWarps * kWeightAhead) {
    float x[kWeightAhead];
#pragma unroll
    for (int u = 0; u < kWeightAhead; ++u)
      x[u] = c < d && p + u * kWarps < parts ? part[(int64_t)(p + u * kWarps) * d + c] : 0.f;
#pragma unroll
    for (int u = 0; u < kWeightAhead; ++u) v += x[u];
  }
  sum[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < d) {
#pragma unroll
    for (int q = 1; q < kWarps; ++q) v += sum[q][lane];
    from_f(v, dw[c]);
  }
}

// Threads of a row and vectors of a thread, for rows of up to KD_RMSNORM_MAX_D
// elements.  The backward's shares of d_w stay in registers: 16 elements a thread, 20
// and 24 where a row lies between the powers of two.  Beyond 8192 elements a row takes
// 1024 threads of 64 registers each, and what those do not hold is spilled (bf16, 4096 x
// 8192 42 us, 4096 x 12288 118, 4096 x 16384 135, 2048 x 32768 223, for floors of 30,
// 45, 59 and 59 us).
template <class T, bool BACKWARD, class F>
auto norm_shape(int64_t d, F&& run) {
  const int64_t vecs = rows_div(d, RowVec<T>::N);
#define KD_SHAPE(TPR, VPT) \
  return run(std::integral_constant<int, TPR>(), std::integral_constant<int, VPT>())
  if (vecs <= 8) KD_SHAPE(8, 1);
  if constexpr (BACKWARD && RowVec<T>::N == 8) {
    if (vecs <= 16) KD_SHAPE(8, 2);
    if (vecs <= 64) KD_SHAPE(32, 2);
    if (vecs <= 96) KD_SHAPE(32, 3);
    if (vecs <= 128) KD_SHAPE(64, 2);
    if (vecs <= 256) KD_SHAPE(128, 2);
    if (vecs <= 384) KD_SHAPE(128, 3);
    if (vecs <= 512) KD_SHAPE(256, 2);
    if (vecs <= 768) KD_SHAPE(256, 3);
    if (vecs <= 1024) KD_SHAPE(512, 2);
    if (vecs <= 2048) KD_SHAPE(1024, 2);
    KD_SHAPE(1024, 4);
  } else {
    if (vecs <= 32) KD_SHAPE(8, 4);
    if (vecs <= 64) KD_SHAPE(32, 2);
    if (vecs <= 128) KD_SHAPE(32, 4);
    if (vecs <= 160) KD_SHAPE(32, 5);
    if (vecs <= 256) KD_SHAPE(128, 2);
    if (vecs <= 512) KD_SHAPE(128, 4);
    if (vecs <= 640) KD_SHAPE(128, 5);
    if (vecs <= 1024) KD_SHAPE(256, 4);
    if (vecs <= 2048) KD_SHAPE(512, 4);
    if constexpr (RowVec<T>::N == 8) {
      KD_SHAPE(1024, 4);
    } else {
      if (vecs <= 4096) KD_SHAPE(1024, 4);
      KD_SHAPE(1024, 8);
    }
  }
#undef KD_SHAPE
}

// Blocks of the backward: each writes a share of d_w, so that few rows take few
// blocks.
int norm_grid(int64_t n, int64_t d, bool bf16) {
  auto grid = [&](auto tpr, auto vpt) {
    constexpr int TPR = decltype(tpr)::value, VPT = decltype(vpt)::value;
    return (int)std::min<int64_t>(rows_div(n, 4 * (norm_block(TPR) / TPR)),
                                  (int64_t)std::max(1, tc_num_sms()) * norm_per_sm(TPR, VPT));
  };
  return bf16 ? norm_shape<__nv_bfloat16, true>(d, grid) : norm_shape<float, true>(d, grid);
}

template <class T, bool VEC>
bool norm_run(const NormArgs& a, void* d_w, int grid, cudaStream_t s) {
  if (!a.dh)
    return norm_shape<T, false>(a.d, [&](auto tpr, auto vpt) {
      constexpr int TPR = decltype(tpr)::value, VPT = decltype(vpt)::value;
      constexpr int block = norm_block(TPR);
      return rows_launch(k_norm_fwd<T, TPR, VPT, VEC>, rows_div(a.n, block / TPR), block, 0, false,
                         s, a);
    });
  return norm_shape<T, true>(a.d, [&](auto tpr, auto vpt) {
    constexpr int TPR = decltype(tpr)::value, VPT = decltype(vpt)::value;
    constexpr int block = norm_block(TPR);
    size_t smem = 0;
    int stages = 0;
    auto kern = k_norm_bwd<T, TPR, VPT, VEC>;
    if constexpr (norm_ring<TPR, VPT, VEC>()) {  // 220 KB for an SM's blocks: 2 stages or more
      constexpr size_t most = (size_t)220 * 1024 / norm_per_sm(TPR, VPT);
      const size_t row = (size_t)(a.res ? 3 : 2) * VPT * block * 16;
      stages = (int)std::min<size_t>(4, most / row);
      smem = stages * row;
      // (always the same limit: another thread may be about to launch with more)
      if (smem > 40000 && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)most) != cudaSuccess)
        return false;
    }
    if (!rows_launch(kern, grid, block, smem, false, s, a, stages)) return false;
    return !d_w || rows_launch(k_norm_weight<T>, rows_div(a.d, 32), kWeightThreads, 0, true, s,
                               (const float*)a.part, grid, a.d, static_cast<T*>(d_w));
  });
}

bool norm_dispatch(const NormArgs& a, bool bf16, bool vec, void* d_w, int grid, cudaStream_t s) {
  if (bf16)
    return vec ? norm_run<__nv_bfloat16, true>(a, d_w, grid, s)
               : norm_run<__nv_bfloat16, false>(a, d_w, grid, s);
  return vec ? norm_run<float, true>(a, d_w, grid, s) : norm_run<float, false>(a, d_w, grid, s);
}

kd_status norm_check(const kd_rmsnorm_problem* p) {
  if (!p || p->n_tokens < 0 || p->n_tokens > INT32_MAX || p->d_model < 1 ||
      p->d_model > KD_RMSNORM_MAX_D)
    return KD_ERR_INVALID_ARG;
  if (p->dtype != KD_BF16 && p->dtype != KD_FP32) return KD_ERR_INVALID_ARG;
  if (!(std::isfinite(p->eps) && p->eps >= 0.f) || !std::isfinite(p->weight_offset))
    return KD_ERR_INVALID_ARG;
  return KD_OK;
}

}  // namespace
}  // namespace kd

using namespace kd;

extern "C" kd_status kd_rmsnorm_workspace_size(const kd_rmsnorm_problem* p, size_t* bwd_bytes) {
  const kd_status st = norm_check(p);
  if (st != KD_OK) return st;
  if (bwd_bytes)
    *bwd_bytes = (size_t)norm_grid(p->n_tokens, p->d_model, p->dtype == KD_BF16) *
                 (size_t)p->d_model * 4;
  return KD_OK;
}

extern "C" kd_status kd_rmsnorm_fwd(const kd_rmsnorm_problem* p, const void* x,
                                    const void* residual, const void* weight, void* sum, void* h,
                                    void* stream) {
  kd_status st = norm_check(p);
  if (st != KD_OK) return st;
  const size_t esz = p->dtype == KD_BF16 ? 2 : 4, row = (size_t)p->d_model * esz;
  const size_t all = (size_t)p->n_tokens * row;
  if (p->n_tokens > 0 && (!x || !weight || !h)) return KD_ERR_INVALID_ARG;
  if (!rows_aligned(esz, x, residual, weight, sum, h)) return KD_ERR_INVALID_ARG;
  if (!rows_over(h, x, all) || !rows_over(h, residual, all) || !rows_over(sum, x, all) ||
      !rows_over(sum, residual, all) || rows_meet(sum, all, h, all) ||
      rows_meet(weight, row, h, all) || rows_meet(weight, row, sum, all))
    return KD_ERR_INVALID_ARG;
  if ((st = rows_device()) != KD_OK || p->n_tokens == 0) return st;
  NormArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x;
  a.res = residual;
  a.w = weight;
  a.sum = sum;
  a.h = h;
  a.n = p->n_tokens;
  a.d = (int)p->d_model;
  a.eps = p->eps;
  a.off = p->weight_offset;
  const bool vec = row % 16 == 0 && rows_aligned(16, x, residual, weight, sum, h);
  const bool ok = norm_dispatch(a, esz == 2, vec, nullptr, 0, static_cast<cudaStream_t>(stream));
  return ok && cudaGetLastError() == cudaSuccess ? KD_OK : KD_ERR_CUDA;
}

extern "C" kd_status kd_rmsnorm_bwd(const kd_rmsnorm_problem* p, const void* sum,
                                    const void* weight, const void* d_h, const void* d_sum,
                                    void* d_x, void* d_weight, void* workspace, size_t ws_bytes,
                                    void* stream) {
  size_t need = 0;
  kd_status st = kd_rmsnorm_workspace_size(p, &need);
  if (st != KD_OK) return st;
  const size_t esz = p->dtype == KD_BF16 ? 2 : 4, row = (size_t)p->d_model * esz;
  const size_t all = (size_t)p->n_tokens * row;
  if (p->n_tokens > 0 && (!sum || !weight || !d_h)) return KD_ERR_INVALID_ARG;
  if (!rows_aligned(esz, sum, weight, d_h, d_sum, d_x, d_weight)) return KD_ERR_INVALID_ARG;
  if (!rows_over(d_x, sum, all) || !rows_over(d_x, d_h, all) || !rows_over(d_x, d_sum, all) ||
      rows_meet(d_x, all, weight, row) || rows_meet(d_weight, row, sum, all) ||
      rows_meet(d_weight, row, weight, row) || rows_meet(d_weight, row, d_h, all) ||
      rows_meet(d_weight, row, d_sum, all) || rows_meet(d_weight, row, d_x, all))
    return KD_ERR_INVALID_ARG;
  if (d_weight && !rows_ws_ok(workspace, ws_bytes, need)) return KD_ERR_WORKSPACE;
  if ((st = rows_device()) != KD_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!d_x && !d_weight) return KD_OK;
  if (p->n_tokens == 0)
    return d_weight && cudaMemsetAsync(d_weight, 0, row, s) != cudaSuccess ? KD_ERR_CUDA : KD_OK;
  NormArgs a;
  memset(&a, 0, sizeof(a));
  a.x = sum;
  a.res = d_sum;
  a.w = weight;
  a.dh = d_h;
  a.h = d_x;
  a.part = d_weight ? static_cast<float*>(workspace) : nullptr;
  a.n = p->n_tokens;
  a.d = (int)p->d_model;
  a.eps = p->eps;
  a.off = p->weight_offset;
  const bool vec = row % 16 == 0 && rows_aligned(16, sum, weight, d_h, d_sum, d_x);
  const bool ok = norm_dispatch(a, esz == 2, vec, d_weight, norm_grid(a.n, a.d, esz == 2), s);
  return ok && cudaGetLastError() == cudaSuccess ? KD_OK : KD_ERR_CUDA;
}
