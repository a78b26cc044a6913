// Embedding lookup and its gradient.
//
//   h[n] = scale W[tokens[n]],   d_w[v] (+)= scale sum_{n : tokens[n] = v} d_h[n]
//
// The gradient is a segmented sum over the tokens sorted by id, in three
// launches:
//   k_embed_sort    a block owns a range of ids and reads all tokens twice: it
//                   counts its ids (and the tokens below them, which is where its
//                   part of the sorted list starts: no block waits for another),
//                   then writes its tokens' places.  A warp has its own run of
//                   the tokens and its own counters, so the list is stable: by id,
//                   and by n within an id.
//   k_embed_reduce  a block has kRun places of the sorted list and some columns,
//                   and adds up the pieces that start there.  An id with fewer than
//                   2 kPiece tokens is one piece and is written at once; more are
//                   cut into pieces of kPiece rows (the last one longer), so that
//                   a frequent token is not one block's work; their fp32 sums go
//                   to the workspace.
//   k_embed_join    adds the pieces of each such id in order.
// Each sum's order depends on the tokens alone.
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

// ------------------------------------------------------------------ lookup
struct LookupArgs {
  const int64_t* tokens;
  const void* w;
  void* h;
  int64_t n, vocab, ignore;
  int64_t d;
  int parts;  // of a row, kSpan vectors (or elements) a lane each
  float scale;
  uint32_t* status;
};
constexpr int kSpan = 4;
constexpr int kLookupThreads = 256;

// A warp copies 32 * kSpan vectors of a row.
template <class T, bool VEC>
__global__ void __launch_bounds__(kLookupThreads) k_embed_rows(LookupArgs a) {
  constexpr int N = RowVec<T>::N;
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * (kLookupThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = item / a.parts;
  const int part = (int)(item - row * a.parts);
  if (row >= a.n) return;
  const int64_t v = a.tokens[row];
  const bool in = v != a.ignore && v >= 0 && v < a.vocab;
  if (!in && v != a.ignore && part == 0 && lane == 0) set_status(a.status, KD_DEV_BAD_LABEL);
  const T* w = static_cast<const T*>(a.w) + (in ? v : 0) * a.d;
  T* h = static_cast<T*>(a.h) + row * a.d;
  const int64_t first = (int64_t)part * (32 * kSpan) + lane;
  if constexpr (VEC) {
    const uint4* src = reinterpret_cast<const uint4*>(w);
    uint4* dst = reinterpret_cast<uint4*>(h);
    const int64_t vecs = a.d / N;
    uint4 u[kSpan];
#pragma unroll
    for (int i = 0; i < kSpan; ++i)
      u[i] = in && first + i * 32 < vecs ? src[first + i * 32] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kSpan; ++i) {
      if (a.scale != 1.f) {
        float x[N];
        RowVec<T>::get(u[i], x);
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = in ? x[e] * a.scale : 0.f;
        u[i] = RowVec<T>::put(x);
      }
      if (first + i * 32 < vecs) __stcs(&dst[first + i * 32], u[i]);
    }
  } else {
    float x[kSpan];
#pragma unroll
    for (int i = 0; i < kSpan; ++i)
      x[i] = in && first + i * 32 < a.d ? to_f(w[first + i * 32]) : 0.f;
#pragma unroll
    for (int i = 0; i < kSpan; ++i)
      if (first + i * 32 < a.d) from_f(in ? x[i] * a.scale : 0.f, h[first + i * 32]);
  }
}

// ------------------------------------------------------------------ sort
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kMaxIds = 1024;  // ids of a block
constexpr int kAhead = 8;      // tokens a lane has in flight

// Places of one id in the sorted list.
struct Segment {
  int32_t first, count;
};

struct SortArgs {
  const int64_t* tokens;
  int64_t n, vocab, ignore;
  int ids;            // of a block
  Segment* seg;       // [vocab]
  int32_t *pos, *id;  // sorted: row, id
  uint32_t* status;
};

__device__ __forceinline__ int block_scan_1024(int v, int* warp_sum, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  int w = warp_sum[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
  return before + x - v;  // exclusive
}

__global__ void __launch_bounds__(kSortThreads) k_embed_sort(SortArgs a) {
  extern __shared__ int counter[];  // [kSortWarps][ids]
  __shared__ int warp_sum[32], below_sum;
  chain_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t lo = (int64_t)blockIdx.x * a.ids;
  for (int i = threadIdx.x; i < kSortWarps * a.ids; i += kSortThreads) counter[i] = 0;
  if (threadIdx.x == 0) below_sum = 0;
  __syncthreads();
  // this warp's run of the tokens, whole groups of 32
  const int64_t groups = (a.n + 31) / 32, each = (groups + kSortWarps - 1) / kSortWarps;
  const int64_t begin = warp * each * 32, end = min((warp + 1) * each * 32, a.n);
  int* mine = counter + warp * a.ids;
  auto fetch = [&](int64_t at) {  // an id, or -1
    if (at >= end) return (int64_t)-1;
    const int64_t t = a.tokens[at];
    if (t == a.ignore) return (int64_t)-1;
    if (t < 0 || t >= a.vocab) {
      if (blockIdx.x == 0) set_status(a.status, KD_DEV_BAD_LABEL);
      return (int64_t)-1;
    }
    return t;
  };
  int below = 0;
  // (each warp reads its run twice, and nobody writes it: no copy is kept)
  for (int64_t at = begin + lane; at - lane < end; at += 32 * kAhead) {
    int64_t t[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) t[u] = fetch(at + u * 32);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (t[u] >= 0 && t[u] < lo) ++below;
      else if (t[u] >= lo && t[u] < lo + a.ids) atomicAdd(&mine[t[u] - lo], 1);
    }
  }
  below = __reduce_add_sync(0xffffffffu, below);
  if (lane == 0 && below) atomicAdd(&below_sum, below);
  __syncthreads();
  // counts to places: by id, then by warp
  int count = 0, total;
  const int own = threadIdx.x;
  if (own < a.ids)
    for (int w = 0; w < kSortWarps; ++w) count += counter[w * a.ids + own];
  int place = below_sum + block_scan_1024(count, warp_sum, total);
  if (own < a.ids) {
    if (lo + own < a.vocab) a.seg[lo + own] = Segment{place, count};
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = counter[w * a.ids + own];
      counter[w * a.ids + own] = place;
      place += c;
    }
  }
  if (!total) return;  // (the whole block)
  __syncthreads();
  for (int64_t at = begin + lane; at - lane < end; at += 32 * kAhead) {
    int64_t t[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) t[u] = fetch(at + u * 32);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = t[u] >= lo && t[u] < lo + a.ids ? (int)(t[u] - lo) : -1;
      if (!__any_sync(0xffffffffu, k >= 0)) continue;
      const uint32_t same = __match_any_sync(0xffffffffu, k);
      int p = 0;
      if (k >= 0) p = mine[k] + __popc(same & ((1u << lane) - 1));
      __syncwarp();
      if (k >= 0) {
        if (lane == __ffs(same) - 1) mine[k] += __popc(same);
        a.pos[p] = (int32_t)(at + u * 32);
        a.id[p] = (int32_t)t[u];
      }
      __syncwarp();
    }
  }
}

// ------------------------------------------------------------------ reduce
constexpr int kRun = 32;     // places of the sorted list a block starts pieces in
constexpr int kPiece = 32;   // rows of a piece of a frequent id
constexpr int kReduceThreads = 128;
constexpr int kRowsAhead = 8;

struct ReduceGradArgs {
  const void* dh;
  void* dw;
  const Segment* seg;
  const int32_t *pos, *id;
  float* part;        // [n / kPiece + 1][d] sums of frequent ids' pieces
  int64_t n, vocab, d;
  int slices;         // of the columns
  int accumulate;
  float scale;
};

// A thread's columns of one row: a vector, or N elements kReduceThreads apart.
template <class T, bool VEC>
struct Columns {
  static constexpr int N = RowVec<T>::N;
  static constexpr int64_t kSlice = (int64_t)kReduceThreads * N;
  static __device__ __forceinline__ void load(const T* row, int64_t c0, int64_t d, float* v) {
    if constexpr (VEC) {
      const int64_t c = c0 + threadIdx.x * N;
      RowVec<T>::get(c < d ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0, 0, 0, 0), v);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int64_t c = c0 + e * kReduceThreads + threadIdx.x;
        v[e] = c < d ? to_f(row[c]) : 0.f;
      }
    }
  }
  static __device__ __forceinline__ void store(T* row, int64_t c0, int64_t d, const float* v) {
    if constexpr (VEC) {
      const int64_t c = c0 + threadIdx.x * N;
      if (c < d) __stcs(reinterpret_cast<uint4*>(row + c), RowVec<T>::put(v));
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int64_t c = c0 + e * kReduceThreads + threadIdx.x;
        if (c < d) from_f(v[e], row[c]);
      }
    }
  }
  static __device__ __forceinline__ void store_part(float* row, int64_t c0, int64_t d,
                                                    const float* v) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int64_t c = VEC ? c0 + threadIdx.x * N + e : c0 + e * kReduceThreads + threadIdx.x;
      if (c < d) row[c] = v[e];
    }
  }
};

template <class T, bool VEC>
__global__ void __launch_bounds__(kReduceThreads) k_embed_reduce(ReduceGradArgs a) {
  using C = Columns<T, VEC>;
  constexpr int N = C::N;
  // pieces that start here: first place, rows, id, and whether the sum goes to `part`
  __shared__ int p_first[kRun], p_rows[kRun], p_id[kRun], p_part[kRun], pieces;
  __shared__ int rows[kRun + 2 * kPiece];
  chain_wait();
  chain_next();
  const int64_t run = blockIdx.x / a.slices;
  const int64_t c0 = (blockIdx.x - run * a.slices) * C::kSlice;
  const int64_t at = run * kRun;
  const int live = a.seg[a.vocab - 1].first + a.seg[a.vocab - 1].count;  // places in all
  T* dw = static_cast<T*>(a.dw);
  const T* dh = static_cast<const T*>(a.dh);
  if (threadIdx.x < 32) {
    int len = 0, v = 0, part = 0;
    const int64_t p = at + threadIdx.x;
    if (p < live) {
      v = a.id[p];
      const Segment s = a.seg[v];
      const int off = (int)(p - s.first);
      if (s.count < 2 * kPiece) {
        len = off == 0 ? s.count : 0;
      } else {
        const int q = s.count / kPiece, j = off / kPiece;
        part = 1;
        if (off % kPiece == 0 && j < q) len = j < q - 1 ? kPiece : s.count - j * kPiece;
      }
    }
    const uint32_t starts = __ballot_sync(0xffffffffu, len > 0);
    if (len > 0) {
      const int k = __popc(starts & ((1u << threadIdx.x) - 1));
      p_first[k] = threadIdx.x;
      p_rows[k] = len;
      p_id[k] = v;
      p_part[k] = part;
    }
    if (threadIdx.x == 0) pieces = __popc(starts);
  }
  static_assert(kRun == 32, "a lane a place");
  for (int i = threadIdx.x; i < kRun + 2 * kPiece; i += kReduceThreads)
    rows[i] = at + i < live ? a.pos[at + i] : 0;
  // rows of ids that do not occur, dealt out to all runs
  if (!a.accumulate) {
    const int64_t runs = gridDim.x / a.slices;
    float zero[N];
#pragma unroll
    for (int e = 0; e < N; ++e) zero[e] = 0.f;
    for (int64_t v = run; v < a.vocab; v += runs)
      if (a.seg[v].count == 0) C::store(dw + v * a.d, c0, a.d, zero);
  }
  __syncthreads();
  for (int k = 0; k < pieces; ++k) {
    const int first = p_first[k], len = p_rows[k];
    float sum[N];
#pragma unroll
    for (int e = 0; e < N; ++e) sum[e] = 0.f;
    for (int r = 0; r < len; r += kRowsAhead) {
      float v[kRowsAhead][N];
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u)
        if (r + u < len) C::load(dh + (int64_t)rows[first + r + u] * a.d, c0, a.d, v[u]);
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u)
        if (r + u < len) {
#pragma unroll
          for (int e = 0; e < N; ++e) sum[e] += v[u][e];
        }
    }
    if (p_part[k]) {
      C::store_part(a.part + (at + first) / kPiece * a.d, c0, a.d, sum);
    } else {
      T* row = dw + (int64_t)p_id[k] * a.d;
      float old[N];
      if (a.accumulate) C::load(row, c0, a.d, old);
#pragma unroll
      for (int e = 0; e < N; ++e)
        sum[e] = a.accumulate ? fmaf(a.scale, sum[e], old[e]) : a.scale * sum[e];
      C::store(row, c0, a.d, sum);
    }
  }
}

// ------------------------------------------------------------------ join
constexpr int kJoinThreads = 256, kJoinCols = 32;
constexpr int kJoinPlaces = 8192;  // places a block looks for frequent ids in

template <class T>
__global__ void __launch_bounds__(kJoinThreads) k_embed_join(ReduceGradArgs a, int cols) {
  constexpr int kWarps = kJoinThreads / 32;
  __shared__ int heads[kJoinPlaces / (2 * kPiece) + 1], count;
  __shared__ float sums[kWarps][33];
  if (threadIdx.x == 0) count = 0;
  chain_wait();
  __syncthreads();
  const int64_t chunk = blockIdx.x / cols;
  const int64_t c = (blockIdx.x - chunk * cols) * kJoinCols + (threadIdx.x & 31);
  const int warp = threadIdx.x >> 5;
  const int64_t at = chunk * kJoinPlaces;
  const int live = a.seg[a.vocab - 1].first + a.seg[a.vocab - 1].count;
  for (int64_t p = at + threadIdx.x; p < at + kJoinPlaces && p < live; p += kJoinThreads) {
    const int v = a.id[p];
    const Segment s = a.seg[v];
    if (p == s.first && s.count >= 2 * kPiece) heads[atomicAdd(&count, 1)] = v;  // any order
  }
  __syncthreads();
  const int n = count;
  for (int k = 0; k < n; ++k) {
    const int v = heads[k];
    const Segment s = a.seg[v];
    const int q = s.count / kPiece;
    const float* part = a.part + (int64_t)(s.first / kPiece) * a.d + c;
    float x = 0.f;
    if (c < a.d)
      for (int j = warp; j < q; j += kWarps) x += part[(int64_t)j * a.d];
    sums[warp][threadIdx.x & 31] = x;
    __syncthreads();
    if (warp == 0 && c < a.d) {
      for (int w = 1; w < kWarps; ++w) x += sums[w][threadIdx.x];
      T& o = static_cast<T*>(a.dw)[(int64_t)v * a.d + c];
      from_f(a.accumulate ? fmaf(a.scale, x, to_f(o)) : a.scale * x, o);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ plan
struct EmbedPlan {
  int ids;             // of a sorting block
  size_t seg, pos, id, part, bytes;
};

kd_status embed_plan(const kd_embed_problem* p, EmbedPlan& P) {
  if (!p || p->n_tokens < 0 || p->n_tokens > (int64_t)1 << 30 || p->vocab < 1 ||
      p->vocab > (int64_t)1 << 30 || p->d_model < 1 || p->d_model > (int64_t)1 << 30)
    return KD_ERR_INVALID_ARG;
  if (p->dtype != KD_BF16 && p->dtype != KD_FP32) return KD_ERR_INVALID_ARG;
  if (!std::isfinite(p->scale)) return KD_ERR_INVALID_ARG;
  const int nsm = std::max(1, tc_num_sms());
  P.ids = 64;
  while (P.ids < kMaxIds && p->vocab > (int64_t)nsm * P.ids) P.ids *= 2;
  size_t off = 0;
  P.seg = rows_take(off, (size_t)p->vocab * sizeof(Segment));
  P.pos = rows_take(off, (size_t)p->n_tokens * 4);
  P.id = rows_take(off, (size_t)p->n_tokens * 4);
  P.part = rows_take(off, p->n_tokens >= 2 * kPiece
                              ? (size_t)(p->n_tokens / kPiece + 1) * p->d_model * 4 : 0);
  P.bytes = off;
  return KD_OK;
}

template <class T>
bool lookup_run(LookupArgs a, bool vec, cudaStream_t s) {
  const int64_t units = vec ? a.d / RowVec<T>::N : a.d;
  a.parts = (int)rows_div(units, 32 * kSpan);
  const int64_t grid = rows_div(a.n * a.parts, kLookupThreads / 32);
  if (grid > INT32_MAX) return false;
  return vec ? rows_launch(k_embed_rows<T, true>, grid, kLookupThreads, 0, false, s, a)
             : rows_launch(k_embed_rows<T, false>, grid, kLookupThreads, 0, false, s, a);
}

template <class T>
bool reduce_run(ReduceGradArgs a, bool vec, cudaStream_t s) {
  a.slices = (int)rows_div(a.d, Columns<T, true>::kSlice);
  // at least some blocks for the zero rows
  const int64_t runs = std::max<int64_t>(rows_div(a.n, kRun), a.accumulate ? 1 : 256);
  const int64_t grid = runs * a.slices;
  const int64_t cols = rows_div(a.d, kJoinCols), join = rows_div(a.n, kJoinPlaces) * cols;
  if (grid > INT32_MAX || join > INT32_MAX) return false;
  const bool ok = vec ? rows_launch(k_embed_reduce<T, true>, grid, kReduceThreads, 0, true, s, a)
                      : rows_launch(k_embed_reduce<T, false>, grid, kReduceThreads, 0, true, s, a);
  if (!ok || a.n < 2 * kPiece) return ok;
  return rows_launch(k_embed_join<T>, join, kJoinThreads, 0, true, s, a, (int)cols);
}

}  // namespace
}  // namespace kd

using namespace kd;

extern "C" kd_status kd_embed_workspace_size(const kd_embed_problem* p, size_t* bwd_bytes) {
  EmbedPlan P;
  const kd_status st = embed_plan(p, P);
  if (st != KD_OK) return st;
  if (bwd_bytes) *bwd_bytes = P.bytes;
  return KD_OK;
}

extern "C" kd_status kd_embed_fwd(const kd_embed_problem* p, const int64_t* tokens, const void* w,
                                  void* h, uint32_t* dev_status, void* stream) {
  EmbedPlan P;
  kd_status st = embed_plan(p, P);
  if (st != KD_OK) return st;
  const size_t esz = p->dtype == KD_BF16 ? 2 : 4, row = (size_t)p->d_model * esz;
  if (p->n_tokens > 0 && (!tokens || !w || !h)) return KD_ERR_INVALID_ARG;
  if (!rows_aligned(8, tokens) || !rows_aligned(esz, w, h) || !rows_aligned(4, dev_status))
    return KD_ERR_INVALID_ARG;
  const size_t all = (size_t)p->n_tokens * row;
  if (rows_meet(h, all, w, (size_t)p->vocab * row) ||
      rows_meet(h, all, tokens, (size_t)p->n_tokens * 8))
    return KD_ERR_INVALID_ARG;
  // (a launch has at most 2^31 - 1 blocks of 2048 16-byte vectors or 1024 elements)
  if ((p->n_tokens * rows_div(p->d_model, 32 * kSpan)) / 8 >= INT32_MAX) return KD_ERR_UNSUPPORTED;
  if ((st = rows_device()) != KD_OK || p->n_tokens == 0) return st;
  LookupArgs a;
  memset(&a, 0, sizeof(a));
  a.tokens = tokens;
  a.w = w;
  a.h = h;
  a.n = p->n_tokens;
  a.vocab = p->vocab;
  a.ignore = p->ignore_index;
  a.d = p->d_model;
  a.scale = p->scale;
  a.status = dev_status;
  const bool vec = row % 16 == 0 && rows_aligned(16, w, h);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool ok = esz == 2 ? lookup_run<__nv_bfloat16>(a, vec, s) : lookup_run<float>(a, vec, s);
  return ok && cudaGetLastError() == cudaSuccess ? KD_OK : KD_ERR_CUDA;
}

extern "C" kd_status kd_embed_bwd(const kd_embed_problem* p, const int64_t* tokens,
                                  const void* d_h, void* d_w, int32_t accumulate,
                                  uint32_t* dev_status, void* workspace, size_t ws_bytes,
                                  void* stream) {
  EmbedPlan P;
  kd_status st = embed_plan(p, P);
  if (st != KD_OK) return st;
  const size_t esz = p->dtype == KD_BF16 ? 2 : 4, row = (size_t)p->d_model * esz;
  const size_t table = (size_t)p->vocab * row;
  if (!d_w || (p->n_tokens > 0 && (!tokens || !d_h))) return KD_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return KD_ERR_INVALID_ARG;
  if (!rows_aligned(8, tokens) || !rows_aligned(esz, d_h, d_w) || !rows_aligned(4, dev_status))
    return KD_ERR_INVALID_ARG;
  if (rows_meet(d_w, table, d_h, (size_t)p->n_tokens * row) ||
      rows_meet(d_w, table, tokens, (size_t)p->n_tokens * 8))
    return KD_ERR_INVALID_ARG;
  if (rows_div(std::max<int64_t>(p->n_tokens, 8192), kRun) * rows_div(p->d_model, 512) >= INT32_MAX)
    return KD_ERR_UNSUPPORTED;
  if (!rows_ws_ok(workspace, ws_bytes, P.bytes)) return KD_ERR_WORKSPACE;
  if ((st = rows_device()) != KD_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p->n_tokens == 0)
    return !accumulate && cudaMemsetAsync(d_w, 0, table, s) != cudaSuccess ? KD_ERR_CUDA : KD_OK;
  char* ws = static_cast<char*>(workspace);
  SortArgs t;
  memset(&t, 0, sizeof(t));
  t.tokens = tokens;
  t.n = p->n_tokens;
  t.vocab = p->vocab;
  t.ignore = p->ignore_index;
  t.ids = P.ids;
  t.seg = reinterpret_cast<Segment*>(ws + P.seg);
  t.pos = reinterpret_cast<int32_t*>(ws + P.pos);
  t.id = reinterpret_cast<int32_t*>(ws + P.id);
  t.status = dev_status;
  const int smem = kSortWarps * P.ids * 4;
  if (smem > 40000 && cudaFuncSetAttribute(k_embed_sort, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           smem) != cudaSuccess)
    return KD_ERR_CUDA;
  if (!rows_launch(k_embed_sort, rows_div(p->vocab, P.ids), kSortThreads, (size_t)smem, false, s, t))
    return KD_ERR_CUDA;
  ReduceGradArgs a;
  memset(&a, 0, sizeof(a));
  a.dh = d_h;
  a.dw = d_w;
  a.seg = t.seg;
  a.pos = t.pos;
  a.id = t.id;
  a.part = reinterpret_cast<float*>(ws + P.part);
  a.n = p->n_tokens;
  a.vocab = p->vocab;
  a.d = p->d_model;
  a.accumulate = accumulate;
  a.scale = p->scale;
  const bool vec = row % 16 == 0 && rows_aligned(16, d_h, d_w);
  const bool ok = esz == 2 ? reduce_run<__nv_bfloat16>(a, vec, s) : reduce_run<float>(a, vec, s);
  return ok && cudaGetLastError() == cudaSuccess ? KD_OK : KD_ERR_CUDA;
}
