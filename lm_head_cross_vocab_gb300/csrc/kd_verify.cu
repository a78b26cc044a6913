// Verification of drafted tokens against a target's probabilities.
//
//   p = softmax(z_t / T_t), q = softmax(z_d / T_d) per row; draft i stands when
//   u_i q(x_i) < p(x_i); the token behind the last that stands is
//   argmax_v r_v / e_v, r = max(p - q, 0) at a rejected row, else p.
//
// Two launches.  k_verify_sums reads every row once and keeps its sum of
// exponentials (greedy: the largest logit's id too), a row in as many parts as
// give the GPU enough blocks.  k_verify_draw joins the parts, decides which drafts
// stand (a few values a sequence, so that each of its blocks decides for
// itself), and runs the race over the one row it ended at, that row in parts
// again; the block that comes last writes the sequence's outputs.
// A race needs one value an id: no running sum across blocks, and no order of
// summation.  r <= p, so that once a block has some id's score r / e, all others
// are held against it by their p alone, which costs an exponential and a compare;
// only the few that pass have their q read and their score formed.
// Exponentials are 2^((z - m) k), k = log2(e) / T, m an offset that trails the
// running maximum; a row's sum S goes with its m, so that p = 2^((z - m) k) / S
// never takes a difference of two log-sum-exps, and logits of any size keep their
// accuracy.
// Bound by HBM where rows are many (256 sequences of 7 drafts, 151936 bf16: sums 168 us,
// 6.95 TB/s, draw 55 us, 4.5 TB/s), by the draw's phases, each waited for, where they are
// few (one sequence of 4 drafts 10.6 us on the GPU).
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

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kUnroll = 4;
constexpr int kMaxParts = 64;       // of a row
constexpr int kMostDrafts = KD_VERIFY_MAX_DRAFTS;

// Sum s of one row's (or a part's) exponentials 2^((z - m) k); best: cand_word of
// the largest logit (greedy).
struct RowSum {
  float m, s;
  uint64_t best;
};

struct VerifyArgs {
  const void *zt, *zd;
  const int64_t* drafts;
  const int32_t* lengths;
  const float *u, *noise;
  int64_t b, vocab, ldt, ldd, ignore;
  int k;
  int greedy;
  float kt, kd, inv_t;        // log2(e) / T of both, 1 / T of the target
  int parts, race_parts;
  RowSum* sums;               // [rows][parts]: B (K + 1) target rows, then B K of the drafter
  uint64_t* leader;           // [B]: the largest score, and the complement of its id
  uint32_t* arrived;          // [B]
  int64_t* tokens;
  int32_t* accepted;
  float* logprob;
  uint32_t* status;
};

__device__ __forceinline__ int drafts_of(const VerifyArgs& a, int64_t b) {
  if (!a.lengths) return a.k;
  const int l = a.lengths[b];
  return l > a.k ? a.k : l;  // negative: takes no part
}

// One part of a row of V elements: whole 16-byte vectors, and the loose
// elements at either end of the row, which the first part takes.
template <class T>
struct Part {
  static constexpr int N = RowVec<T>::N;
  const T* z;
  int64_t vocab;
  int head, tail;             // loose elements
  int64_t v0, v1;             // vectors

  __device__ __forceinline__ Part(const T* z_, int64_t vocab_, int part, int parts)
      : z(z_), vocab(vocab_) {
    const int skew = (int)((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T));
    const int64_t lead = min((int64_t)(skew ? N - skew : 0), vocab);
    const int64_t vecs = (vocab - lead) / N;
    head = (int)lead;
    tail = (int)(vocab - lead - vecs * N);
    v0 = vecs * part / parts;
    v1 = vecs * (part + 1) / parts;
    if (part) head_in = 0, tail = 0;
    else head_in = head;
  }
  int head_in;
  __device__ __forceinline__ const uint4* vectors() const {
    return reinterpret_cast<const uint4*>(z + head);
  }
  __device__ __forceinline__ int loose() const { return head_in + tail; }
  __device__ __forceinline__ int64_t loose_at(int i) const {
    return i < head_in ? i : vocab - tail + (i - head_in);
  }
};

// largest of a vector, a NaN kept
__device__ __forceinline__ float vec_top(uint4 w, float) {
  return max_nan(max_nan(__uint_as_float(w.x), __uint_as_float(w.y)),
                 max_nan(__uint_as_float(w.z), __uint_as_float(w.w)));
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float vec_top(uint4 w, __nv_bfloat16) {
  const uint32_t m = max_nan_bf16x2(max_nan_bf16x2(w.x, w.y), max_nan_bf16x2(w.z, w.w));
  return max_nan(bf16lo(m), bf16hi(m));
}

struct Fold {
  float k, m, up;  // a logit above `up` moves the offset
  float2 s;
  __device__ __forceinline__ void init(float k_) {
    k = k_;
    m = up = neg_inf();
    s = make_float2(0.f, 0.f);
  }
  __device__ __forceinline__ void expect(float top) {
    if (top > up) {
      const float f = ex2((m - top) * k);
      s = make_float2(s.x * f, s.y * f);
      m = top;
      up = top + 8.f / k;
    }
  }
  __device__ __forceinline__ void pair(float z0, float z1) {
    const float2 x = mul2(sub2(make_float2(z0, z1), make_float2(m, m)), make_float2(k, k));
    s = add2(s, make_float2(ex2(x.x), ex2(x.y)));
  }
  __device__ __forceinline__ void one(float z) {
    if (z == neg_inf()) return;
    expect(z);
    s.x += ex2((z - m) * k);
  }
};
__device__ __forceinline__ void join_sum(float& m, float& s, float m2, float s2, float k) {
  const float to = fmaxf(m, m2);
  if (m != to) s *= ex2((m - to) * k);
  if (m2 != to) s2 *= ex2((m2 - to) * k);
  s += s2;
  m = to;
}
// all lanes' sums, in every lane: the largest offset first, then one rescale each
__device__ __forceinline__ void warp_sum(float& m, float& s, float k) {
  float to = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, o));
  if (m != to) s *= ex2((m - to) * k);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  m = to;
}
__device__ __forceinline__ uint64_t warp_best(uint64_t w) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t x = __shfl_xor_sync(0xffffffffu, w, o);
    w = x > w ? x : w;
  }
  return w;
}
// a row with a distribution: neither a NaN nor +infinity nor only -infinity
__device__ __forceinline__ bool sum_ok(const RowSum& r) {
  return r.s > 0.f && r.s < __int_as_float(0x7f800000) && fabsf(r.m) < __int_as_float(0x7f800000);
}

template <class T, bool GREEDY, int NT>
__global__ void __launch_bounds__(NT) k_verify_sums(VerifyArgs a) {
  constexpr int N = RowVec<T>::N, kWarps = NT / 32;
  __shared__ float wm[kWarps], ws[kWarps];
  __shared__ uint64_t wb[kWarps];
  chain_next();
  const int64_t row = blockIdx.x / a.parts;
  const int part = (int)(blockIdx.x - row * a.parts);
  const int64_t targets = a.b * (a.k + 1);
  const bool draft = row >= targets;
  const int64_t in = draft ? row - targets : row;
  const int per = draft ? a.k : a.k + 1;
  const int64_t b = in / per;
  const int i = (int)(in - b * per);
  if (!draft && i == 0 && part == 0 && threadIdx.x == 0) {
    a.arrived[b] = 0;
    a.leader[b] = 0;
  }
  if (i >= drafts_of(a, b) + (draft ? 0 : 1) || drafts_of(a, b) < 0) return;
  const T* z = static_cast<const T*>(draft ? a.zd : a.zt) + in * (draft ? a.ldd : a.ldt);
  const Part<T> p(z, a.vocab, part, a.parts);
  Fold f;
  f.init(draft ? a.kd : a.kt);
  // greedy: the largest logit and the step it came in; who has the block's largest
  // looks that step's vectors through once more
  float top = neg_inf();
  int64_t top_v = 0;
  int top_n = 0;
  const uint4* q = p.vectors();
  auto take = [&](const uint4* w, int64_t v, auto count) {
    constexpr int C = decltype(count)::value;
    float m = vec_top(w[0], T());
#pragma unroll
    for (int u = 1; u < C; ++u) m = max_nan(m, vec_top(w[u], T()));
    if (m == neg_inf()) return;
    f.expect(m);
    if (GREEDY && m > top) {
      top = m;
      top_v = v;
      top_n = C;
    }
#pragma unroll
    for (int u = 0; u < C; ++u) {
      float x[N];
      RowVec<T>::get(w[u], x);
#pragma unroll
      for (int e = 0; e < N; e += 2) f.pair(x[e], x[e + 1]);
    }
  };
  int64_t v = p.v0 + threadIdx.x;
  for (; v + (kUnroll - 1) * NT < p.v1; v += kUnroll * NT) {
    uint4 w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) w[u] = q[v + u * NT];
    take(w, v, std::integral_constant<int, kUnroll>());
  }
  for (; v < p.v1; v += NT) {
    const uint4 w = q[v];
    take(&w, v, std::integral_constant<int, 1>());
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t best = 0;
  float loose = neg_inf();
  int64_t loose_at = 0;
  if (threadIdx.x < p.loose()) {
    loose_at = p.loose_at(threadIdx.x);
    loose = to_f(z[loose_at]);
    f.one(loose);
  }
  if (GREEDY) {
    float most = fmaxf(top, loose);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (lane == 0) wm[warp] = most;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) most = fmaxf(most, wm[w]);
    __syncthreads();
    if (most > neg_inf()) {
      if (loose == most) best = cand_word(order_key(most), (uint32_t)loose_at);
      if (top == most) {
        int64_t at = -1;
        for (int u = 0; u < top_n && at < 0; ++u) {
          float x[N];
          RowVec<T>::get(q[top_v + u * NT], x);
#pragma unroll
          for (int e = N - 1; e >= 0; --e)
            if (x[e] == most) at = p.head + (top_v + u * NT) * N + e;
        }
        const uint64_t w = cand_word(order_key(most), (uint32_t)at);
        best = w > best ? w : best;
      }
    }
  }
  float off = f.m, s = f.s.x + f.s.y;
  warp_sum(off, s, f.k);
  if (GREEDY) best = warp_best(best);
  if (lane == 0) {
    wm[warp] = off;
    ws[warp] = s;
    wb[warp] = best;
  }
  __syncthreads();
  if (warp == 0) {
    off = lane < kWarps ? wm[lane] : neg_inf();
    s = lane < kWarps ? ws[lane] : 0.f;
    best = lane < kWarps ? wb[lane] : 0;
    warp_sum(off, s, f.k);
    if (GREEDY) best = warp_best(best);
    if (lane == 0) a.sums[row * a.parts + part] = RowSum{off, s, best};
  }
}

// 2^((z - m) k), the roundings of z - m and of the product made up for
__device__ __forceinline__ float power(float z, float m, float k) {
  const float d = __fsub_rn(z, m), y = __fsub_rn(z, d);
  const float lost = __fadd_rn(__fsub_rn(z, __fadd_rn(d, y)), __fsub_rn(y, m));
  const float x = __fmul_rn(d, k), rest = fmaf(lost, k, fmaf(d, k, -x));
  const float p = ex2(x) * fmaf(rest, kLn2, 1.f);
  return x < -150.f ? 0.f : p;  // (z = -inf among others: rest is NaN then)
}

// u a b < c d, to some 2^-46: with the products' own roundings a u just below 1
// would count as 1 where a b = c d, as in equal rows whose sums are equal.  (In fp64, a unit that this GPU has little of,
// the decisions of a block took 1.5 to 3 us.)
__device__ __forceinline__ bool below(float u, float a, float b, float c, float d) {
  const float x = __fmul_rn(a, b), xr = __fmaf_rn(a, b, -x);
  const float y = __fmul_rn(c, d), yr = __fmaf_rn(c, d, -y);
  const float z = __fmul_rn(u, x), zr = __fmaf_rn(u, x, -z);
  return __fadd_rn(__fsub_rn(z, y), __fsub_rn(__fmaf_rn(u, xr, zr), yr)) < 0.f;
}

// The race over ids of one row.  A score is 2^64 r / e: within fp32 for every r <= 1
// and every noise that takes part (r = 2^-100 behind noise of 2^60 is lost without the
// factor).  Its word: its bits above, the complement of
// the id below, so that a larger word is ahead and equal scores go to the lowest
// id; 0: nobody.  All blocks' words are compared as integers: no order matters.
struct Race {
  float kt, mt, inv_t;        // of the target's row
  float kd, md, inv_d;        // of the drafter's (q taken away), inv_d = 0: none
  int64_t out;                // this id has q = 1, -1: none

  __device__ __forceinline__ float weight(float zt, float zd, int64_t id) const {
    float r = __fmul_rn(power(zt, mt, kt), inv_t);
    if (inv_d > 0.f) r = __fsub_rn(r, __fmul_rn(power(zd, md, kd), inv_d));
    return id == out ? 0.f : r;
  }
  static __device__ __forceinline__ uint64_t score(float r, float e, int64_t id) {
    if (!(r > 0.f && e >= 0x1p-60f && e <= 0x1p60f)) return 0;
    const float s = __fdiv_rn(__fmul_rn(r, 0x1p64f), e);
    return s > 0.f ? (uint64_t)__float_as_uint(s) << 32 | (uint32_t)~(uint32_t)id : 0;
  }
};
constexpr int kList = 1024;  // ids that a block takes a closer look at
struct RaceShared {
  uint64_t best;
  int count;
  int rest;  // while best is 0: whether some id has a weight, whatever its noise
  int list[kList];
};
constexpr int kIds = 8;    // ids a thread takes at a time
constexpr int kAhead = 2;  // times that, on their way
// kIds neighbouring ids' logits and noise, as they come.
template <class T>
struct IdVec {
  static constexpr int Z = kIds / RowVec<T>::N;
  uint4 z[Z];
  float4 e[kIds / 4];
  __device__ __forceinline__ void load(const T* zt, const float* noise, int first) {
#pragma unroll
    for (int i = 0; i < Z; ++i) z[i] = reinterpret_cast<const uint4*>(zt + first)[i];
#pragma unroll
    for (int i = 0; i < kIds / 4; ++i) e[i] = __ldcs(&reinterpret_cast<const float4*>(noise + first)[i]);
  }
  __device__ __forceinline__ void get(float* x, float* y) const {
#pragma unroll
    for (int i = 0; i < Z; ++i) RowVec<T>::get(z[i], x + i * RowVec<T>::N);
#pragma unroll
    for (int i = 0; i < kIds / 4; ++i)
      y[4 * i] = e[i].x, y[4 * i + 1] = e[i].y, y[4 * i + 2] = e[i].z, y[4 * i + 3] = e[i].w;
  }
};
// The block's leader of ids [lo, hi), in every thread.
template <class T>
__device__ __forceinline__ uint64_t race_part(const Race& c, const T* zt, const T* zd,
                                              const float* noise, int64_t lo, int64_t hi,
                                              RaceShared& sh) {
  const int tid = threadIdx.x;
  if (tid == 0) {
    sh.best = 0;
    sh.count = 0;
    sh.rest = 0;
  }
  __syncthreads();
  const T* z0 = zt + lo;
  const float* e0 = noise + lo;
  const bool vec = ((reinterpret_cast<uintptr_t>(z0) | reinterpret_cast<uintptr_t>(e0)) & 15) == 0;
  const int n = (int)(hi - lo), whole = vec ? n / kIds * kIds : 0;
  constexpr int kStep = kThreads * kIds;
  auto exact = [&](int i) {
    const float r = c.weight(to_f(z0[i]), zd ? to_f(zd[lo + i]) : 0.f, lo + i);
    if (r > 0.f) sh.rest = 1;
    return c.score(r, e0[i], lo + i);
  };
  auto offer = [&](uint64_t w) {
    if (w) atomicMax((unsigned long long*)&sh.best, (unsigned long long)w);
  };
  // ids that are not in a vector: kIds of them kThreads apart, or nothing
  auto singles = [&](int at, float* z, float* e) {
#pragma unroll
    for (int j = 0; j < kIds; ++j) {
      const int i = at + j * kThreads + tid;
      z[j] = i < n ? to_f(z0[i]) : neg_inf();
      e[j] = i < n ? e0[i] : 1.f;
    }
  };
  float z[kIds], e[kIds];
  // some scores: of each thread's first ids the one that seems ahead
  {
    float d[kIds];
    const T* d0 = zd ? zd + lo : nullptr;
    const bool both = zd && (reinterpret_cast<uintptr_t>(d0) & 15) == 0;
    const int first = tid * kIds < whole ? tid * kIds : whole + tid;
    const int apart = tid * kIds < whole ? 1 : kThreads;
    if (tid * kIds < whole) {
      IdVec<T> w;
      w.load(z0, e0, first);
      if (both) {
        uint4 y[IdVec<T>::Z];
#pragma unroll
        for (int i = 0; i < IdVec<T>::Z; ++i) y[i] = reinterpret_cast<const uint4*>(d0 + first)[i];
#pragma unroll
        for (int i = 0; i < IdVec<T>::Z; ++i) RowVec<T>::get(y[i], d + i * RowVec<T>::N);
      }
      w.get(z, e);
    } else {
      singles(whole, z, e);
    }
    if (!both || apart > 1) {
#pragma unroll
      for (int j = 0; j < kIds; ++j)
        d[j] = zd && first + j * apart < n ? to_f(d0[first + j * apart]) : 0.f;
    }
    float most = 0.f, zb = 0.f, db = 0.f, eb = 1.f;
    int at = -1;
#pragma unroll
    for (int j = 0; j < kIds; ++j) {
      const float p = ex2((z[j] - c.mt) * c.kt) * c.inv_t;
      const float q = ex2((d[j] - c.md) * c.kd) * c.inv_d;  // (inv_d = 0 without a drafter)
      const float x = __fdividef(p - q, e[j]);
      if (x > most) {
        most = x;
        at = first + j * apart;
        zb = z[j], db = d[j], eb = e[j];
      }
    }
    uint64_t w = at >= 0 ? c.score(c.weight(zb, db, lo + at), eb, lo + at) : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t x = __shfl_xor_sync(0xffffffffu, w, o);
      w = x > w ? x : w;
    }
    if ((tid & 31) == 0) offer(w);
  }
  __syncthreads();
  // p = 2^x / S, x = (z - m) k: an id may be ahead if 2^x > score S e.  The factor
  // covers the roundings of this test: of x (|x| 2^-23, 2^x being 0 below x = -126),
  // of the power (2^-22) and of the products.  Without a score yet every id of some
  // p passes, that of infinite or NaN noise too (where 0 e is NaN), so that `rest`
  // is known where nobody arrives
  // (a ratio near fp32's lower end has lost bits: everything passes)
  const float ratio = __uint_as_float((uint32_t)(sh.best >> 32)) * 0x1p-64f;
  const float held = ratio < 0x1p-100f ? 0.f : ratio / c.inv_t * (1.f - 0x1p-14f);
  const float2 k2 = make_float2(c.kt, c.kt), m2 = make_float2(c.mt, c.mt), h2 = make_float2(held, held);
  __syncthreads();
  auto sift = [&](const float* z, const float* e, int first, int apart) {
    uint32_t pass = 0;
#pragma unroll
    for (int j = 0; j < kIds; j += 2) {
      const float2 x = mul2(sub2(make_float2(z[j], z[j + 1]), m2), k2);
      const float2 y = mul2(make_float2(e[j], e[j + 1]), h2);
      if (!(ex2(x.x) <= y.x)) pass |= 1u << j;
      if (!(ex2(x.y) <= y.y)) pass |= 2u << j;
    }
    for (; pass; pass &= pass - 1) {
      const int i = first + (__ffs(pass) - 1) * apart;
      const int k = atomicAdd(&sh.count, 1);
      if (k < kList) sh.list[k] = i;
      else offer(exact(i));
    }
  };
  for (int at = tid * kIds; at < whole; at += kAhead * kStep) {
    IdVec<T> w[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (at + u * kStep < whole) w[u].load(z0, e0, at + u * kStep);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (at + u * kStep < whole) {
        w[u].get(z, e);
        sift(z, e, at + u * kStep, 1);
      }
  }
  int at = whole;
  for (; at + kStep <= n; at += kStep) {  // (no id of these is beyond the end)
#pragma unroll
    for (int j = 0; j < kIds; ++j) {
      z[j] = to_f(z0[at + j * kThreads + tid]);
      e[j] = __ldcs(&e0[at + j * kThreads + tid]);
    }
    sift(z, e, at + tid, kThreads);
  }
  if (at < n) {
    singles(at, z, e);
    sift(z, e, at + tid, kThreads);
  }
  __syncthreads();
  const int count = min(sh.count, kList);
  for (int k = tid; k < count; k += kThreads) offer(exact(sh.list[k]));
  __syncthreads();
  return sh.best;
}

template <class T>
__global__ void __launch_bounds__(kThreads, 4) k_verify_draw(VerifyArgs a) {
  __shared__ RowSum tgt[kMostDrafts + 1], drf[kMostDrafts];
  __shared__ RaceShared race_shared;
  __shared__ int stands, last;
  __shared__ uint32_t trouble;
  const int64_t b = blockIdx.x / a.race_parts;
  const int part = (int)(blockIdx.x - b * a.race_parts);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = a.k + 1;
  chain_wait();
  // what the decisions need of each draft, a lane of the first warp each, on its
  // way while the sums are joined
  int64_t x = -1;
  float u = 0.f;
  if (warp == 0 && lane < a.k) {
    x = a.drafts[b * a.k + lane];
    if (!a.greedy) u = a.u[b * a.k + lane];
  }
  const int len = drafts_of(a, b);
  const bool over = a.lengths && a.lengths[b] > a.k;
  const T* zt = static_cast<const T*>(a.zt) + b * rows * a.ldt;
  const T* zd = static_cast<const T*>(a.zd) + b * a.k * a.ldd;
  if (len < 0) {
    if (part == 0) {
      for (int i = threadIdx.x; i < rows; i += kThreads) {
        if (a.tokens) a.tokens[b * rows + i] = a.ignore;
        if (a.logprob) a.logprob[b * rows + i] = 0.f;
      }
      if (a.accepted && threadIdx.x == 0) a.accepted[b] = 0;
    }
    return;
  }
  const bool has_q = a.zd != nullptr && !a.greedy;
  float zx = 0.f, qx = 0.f;
  if (warp == 0 && lane < len && x >= 0 && x < a.vocab) {
    zx = to_f(zt[lane * a.ldt + x]);
    if (has_q) qx = to_f(zd[lane * a.ldd + x]);
  }
  // ---- the rows' sums: two rows of a warp at a time, their parts a lane each
  const int sums = len + 1 + (has_q ? len : 0);
  for (int r0 = warp; r0 < sums; r0 += 2 * kWarps) {
    RowSum v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + h * kWarps;
      v[h] = RowSum{neg_inf(), 0.f, 0};
      if (r >= sums) continue;
      const int64_t row = r > len ? a.b * rows + b * a.k + (r - len - 1) : b * rows + r;
      const float k = r > len ? a.kd : a.kt;
      if (lane < a.parts) v[h] = a.sums[row * a.parts + lane];
      if (lane + 32 < a.parts) {
        const RowSum o = a.sums[row * a.parts + lane + 32];
        join_sum(v[h].m, v[h].s, o.m, o.s, k);
        v[h].best = o.best > v[h].best ? o.best : v[h].best;
      }
    }
    static_assert(kMaxParts <= 64, "two parts a lane");
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + h * kWarps;
      if (r >= sums) continue;
      warp_sum(v[h].m, v[h].s, r > len ? a.kd : a.kt);
      if (a.greedy) v[h].best = warp_best(v[h].best);
      if (lane == 0) (r > len ? drf[r - len - 1] : tgt[r]) = v[h];
    }
  }
  __syncthreads();
  // ---- the drafts that stand: a lane each
  if (warp == 0) {
    bool ok = false, bad = false, foreign = false;
    if (lane < len) {
      foreign = x < 0 || x >= a.vocab;
      const RowSum t = tgt[lane];
      bad = !sum_ok(t);
      if (a.greedy) {
        ok = !foreign && !bad && (int64_t)(uint32_t)~(uint32_t)t.best == x;
      } else {
        const bool bad_q = has_q && !sum_ok(drf[lane]);
        if (!foreign && !bad && !bad_q) {
          const float p = power(zx, t.m, a.kt);
          if (has_q) {
            const RowSum d = drf[lane];
            const float q = power(qx, d.m, a.kd);
            ok = below(u, q, t.s, p, d.s);
          } else {
            ok = below(u, 1.f, t.s, p, 1.f);
          }
        }
        bad = bad || bad_q;
      }
    }
    const uint32_t oks = __ballot_sync(0xffffffffu, ok), bads = __ballot_sync(0xffffffffu, bad);
    const uint32_t foreigns = __ballot_sync(0xffffffffu, foreign);
    const int n = oks == 0xffffffffu ? 32 : __ffs(~oks) - 1;
    // what lies behind the first that does not stand is not reported
    const uint32_t seen = n >= 31 ? 0xffffffffu : (2u << n) - 1;
    if (lane == 0) {
      stands = n;
      trouble = ((bads & seen) || !sum_ok(tgt[n]) ? KD_DEV_NONFINITE : 0) |
                ((foreigns & seen) || over ? KD_DEV_BAD_LABEL : 0);
    }
  }
  __syncthreads();
  const int n = stands;
  const RowSum row = tgt[n];
  const bool alive = sum_ok(row);
  // ---- the race
  uint64_t leader = 0;
  bool rest = false;  // nobody has arrived, but some id of this row might have with other noise
  const float* noise = a.noise + b * a.vocab;
  zt += n * a.ldt;
  if (!a.greedy) {
    Race race{a.kt, row.m, 1.f / row.s, a.kd, 0.f, 0.f, -1};
    const T* q = nullptr;
    if (n < len) {
      if (has_q && sum_ok(drf[n])) {
        q = zd + n * a.ldd;
        race.md = drf[n].m;
        race.inv_d = 1.f / drf[n].s;
      } else if (!has_q) {
        race.out = a.drafts[b * a.k + n];
      }
    }
    // parts of whole vectors of 16 logits
    const int64_t units = (a.vocab + 15) / 16;
    const int64_t lo = units * part / a.race_parts * 16;
    const int64_t hi = min(units * (part + 1) / a.race_parts * 16, a.vocab);
    if (alive) {
      leader = race_part<T>(race, zt, q, noise, lo, hi, race_shared);
      rest = race_shared.rest;
    }
    if (a.race_parts > 1) {
      if (threadIdx.x == 0) {
        // (release: the leader comes before the arrival; acquire: all of theirs)
        if (leader) atomicMax((unsigned long long*)&a.leader[b], (unsigned long long)leader);
        // the blocks that arrived, and above them those that found a weight
        const uint32_t here = 1u | (uint32_t)rest << 16;
        uint32_t before;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;"
                     : "=r"(before)
                     : "l"(&a.arrived[b]), "r"(here)
                     : "memory");
        last = (before & 0xffff) == (uint32_t)a.race_parts - 1;
        if (last) {
          race_shared.best = *(volatile uint64_t*)&a.leader[b];
          race_shared.rest = (before + here) >> 16;
        }
      }
      static_assert(kMaxParts < 1 << 16, "arrivals in 16 bits");
      __syncthreads();
      if (!last) return;
      leader = race_shared.best;
      rest = race_shared.rest;
      __syncthreads();
    }
    if (alive && !leader && !rest && n < len) {
      // p <= q everywhere: no residual to draw from.  (Where there is one whose ids all
      // have noise that takes no part, nothing is drawn.)
      race.inv_d = 0.f;
      race.out = -1;
      leader = race_part<T>(race, zt, (const T*)nullptr, noise, 0, a.vocab, race_shared);
    }
  }
  // ---- outputs
  const bool drawn = alive && (a.greedy || leader);
  const int64_t token = (int64_t)(uint32_t)~(uint32_t)(a.greedy ? row.best : leader);
  if (warp == 0) {
    auto put = [&](int i, int64_t x, float z) {  // place i: an accepted draft, the drawn one, none
      const bool there = i < n || (i == n && drawn);
      if (a.tokens) a.tokens[b * rows + i] = there ? x : a.ignore;
      if (a.logprob) {
        const RowSum t = tgt[min(i, n)];
        a.logprob[b * rows + i] = there ? fmaf(z - t.m, a.inv_t, -logf(t.s))
                                        : i == n ? __int_as_float(0x7fffffff) : 0.f;
      }
    };
    const float z = drawn ? to_f(zt[token]) : 0.f;
    if (lane < rows) put(lane, lane < n ? x : token, lane < n ? zx : z);
    if (lane == 0 && rows > 32) put(32, token, z);
  }
  if (threadIdx.x == 0) {
    if (a.accepted) a.accepted[b] = n;
    const uint32_t t = trouble | (drawn ? 0u : KD_DEV_NONFINITE);
    if (t) set_status(a.status, t);
  }
}

// ------------------------------------------------------------------ plan
struct VerifyPlan {
  int parts[2], race_parts;   // parts, rows: of the target alone, and with the drafter's
  int64_t rows[2];
  size_t sums, leader, arrived, bytes;
};

kd_status verify_plan(const kd_verify_problem* p, VerifyPlan& P) {
  if (!p || p->n_seqs < 0 || p->n_seqs > (int64_t)1 << 20 || p->vocab < 1 ||
      p->vocab > (int64_t)1 << 30 || p->n_drafts < 0 || p->n_drafts > KD_VERIFY_MAX_DRAFTS)
    return KD_ERR_INVALID_ARG;
  if (p->dtype != KD_BF16 && p->dtype != KD_FP32) return KD_ERR_INVALID_ARG;
  if (!(std::isfinite(p->t_target) && p->t_target >= 0.f) ||
      !(std::isfinite(p->t_draft) && p->t_draft > 0.f) || !std::isfinite(kL2E / p->t_draft) ||
      (p->t_target > 0.f && !std::isfinite(kL2E / p->t_target)))
    return KD_ERR_INVALID_ARG;
  if ((p->ld_target && p->ld_target < p->vocab) || (p->ld_draft && p->ld_draft < p->vocab))
    return KD_ERR_INVALID_ARG;
  const int nsm = std::max(1, tc_num_sms());
  const int64_t bytes = p->vocab * (p->dtype == KD_BF16 ? 2 : 4);
  const int64_t b = std::max<int64_t>(p->n_seqs, 1);
  // Parts of a row in the first launch: three blocks an SM where rows are few, else
  // some 96 KB each (72 rows of 304 KB: 15.6 us with 6 parts, 20.5 with 1, 22.4 with
  // 34; 3840 rows: 233.6 us with 3, 237.3 with 1, 249.9 with 8), 16 KB at least.  The
  // drafter's rows count where they are read.
  size_t off = 0, sums = 0;
  for (int i = 0; i < 2; ++i) {
    P.rows[i] = p->n_seqs * ((i ? 2 : 1) * (int64_t)p->n_drafts + 1);
    const int64_t r = std::max<int64_t>(P.rows[i], 1);
    const int64_t parts = std::max<int64_t>(
        1, std::min<int64_t>({std::max(rows_div((int64_t)nsm * 3, r), (bytes + 49152) / 98304),
                              bytes / 16384, kMaxParts}));
    // (a launch has at most 2^31 - 1 blocks; there are at most 2^27 rows)
    P.parts[i] = (int)std::min<int64_t>(parts, INT32_MAX / r);
    sums = std::max(sums, (size_t)r * P.parts[i] * sizeof(RowSum));
  }
  // and of the row that is drawn from: as many blocks as the SMs hold, four each, or
  // where that is one or two a row, four (48 rows of 128256: 31.7 us with 12 parts, 37.7
  // with 16; 256 rows of 151936: 227.8 us with 4, 247.3 with 2, 237 with 3); parts
  // below 8192 ids only up to two blocks an SM (16 rows of 151936: 12.5 us with 16,
  // 13.5 with 37), and of 2048 at least
  const int64_t most = (int64_t)nsm * 4 / b;
  P.race_parts = (int)std::max<int64_t>(
      1, std::min<int64_t>({most >= 3 ? most : 4, std::max(p->vocab / 8192, (int64_t)nsm * 2 / b),
                            p->vocab / 2048, kMaxParts}));
  P.sums = rows_take(off, sums);
  P.leader = rows_take(off, (size_t)b * 8);
  P.arrived = rows_take(off, (size_t)b * 4);
  P.bytes = off;
  return KD_OK;
}

// An output over an input, or over another output.
bool verify_overlaps(const kd_verify_problem* p, const kd_verify_inputs* in, const int64_t* tokens,
                     const int32_t* accepted, const float* logprob) {
  const size_t n = (size_t)p->n_seqs, k = (size_t)p->n_drafts, v = (size_t)p->vocab;
  const size_t esz = p->dtype == KD_BF16 ? 2 : 4;
  const size_t lt = p->ld_target ? p->ld_target : v, ld = p->ld_draft ? p->ld_draft : v;
  struct Span {
    const void* p;
    size_t bytes;
  };
  const Span outs[] = {{tokens, n * (k + 1) * 8}, {accepted, n * 4}, {logprob, n * (k + 1) * 4}};
  const Span ins[] = {{in->target_logits, ((n * (k + 1) - 1) * lt + v) * esz},
                      {k ? in->draft_logits : nullptr, k ? ((n * k - 1) * ld + v) * esz : 0},
                      {in->drafts, n * k * 8}, {in->lengths, n * 4}, {in->uniform, n * k * 4},
                      {in->noise, n * v * 4}};
  for (int i = 0; i < 3; ++i) {
    for (const Span& x : ins)
      if (rows_meet(outs[i].p, outs[i].bytes, x.p, x.bytes)) return true;
    for (int j = 0; j < i; ++j)
      if (rows_meet(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return true;
  }
  return false;
}

template <class T, int NT>
bool sums_run(const VerifyArgs& a, int64_t rows, cudaStream_t s) {
  return a.greedy ? rows_launch(k_verify_sums<T, true, NT>, rows * a.parts, NT, 0, false, s, a)
                  : rows_launch(k_verify_sums<T, false, NT>, rows * a.parts, NT, 0, false, s, a);
}
template <class T>
bool verify_run(const VerifyArgs& a, int64_t rows, cudaStream_t s) {
  // short parts take smaller blocks, more of them on an SM (349 sequences of 8 drafts, 8214
  // bf16: 20.1 us with 128 threads, 24.9 with 256; 194 of 5, 1174: 4.3 us with 32, 8.3 with 256)
  const int64_t bytes = a.vocab * (int64_t)sizeof(T) / a.parts;
  const bool ok = bytes <= 4096    ? sums_run<T, 32>(a, rows, s)
                  : bytes <= 32768 ? sums_run<T, 128>(a, rows, s)
                                   : sums_run<T, 256>(a, rows, s);
  return ok && rows_launch(k_verify_draw<T>, a.b * a.race_parts, kThreads, 0, true, s, a);
}

}  // namespace
}  // namespace kd

using namespace kd;

extern "C" kd_status kd_verify_workspace_size(const kd_verify_problem* p, size_t* bytes) {
  VerifyPlan P;
  const kd_status st = verify_plan(p, P);
  if (st != KD_OK) return st;
  if (bytes) *bytes = P.bytes;
  return KD_OK;
}

extern "C" kd_status kd_verify_drafts(const kd_verify_problem* p, const kd_verify_inputs* in,
                                      int64_t* tokens, int32_t* accepted, float* logprob,
                                      uint32_t* dev_status, void* workspace, size_t ws_bytes,
                                      void* stream) {
  VerifyPlan P;
  kd_status st = verify_plan(p, P);
  if (st != KD_OK) return st;
  if (!in) return KD_ERR_INVALID_ARG;
  const bool greedy = p->t_target == 0.f;
  const int64_t n = p->n_seqs, k = p->n_drafts, v = p->vocab;
  const size_t esz = p->dtype == KD_BF16 ? 2 : 4;
  if (n > 0 && (!in->target_logits || (k > 0 && !in->drafts) || (!greedy && !in->noise) ||
                (!greedy && k > 0 && !in->uniform)))
    return KD_ERR_INVALID_ARG;
  if (!rows_aligned(esz, in->target_logits, in->draft_logits) ||
      !rows_aligned(8, in->drafts, tokens) ||
      !rows_aligned(4, in->lengths, in->uniform, in->noise, accepted, logprob, dev_status))
    return KD_ERR_INVALID_ARG;
  if (n > 0 && verify_overlaps(p, in, tokens, accepted, logprob)) return KD_ERR_INVALID_ARG;
  if (!rows_ws_ok(workspace, ws_bytes, P.bytes)) return KD_ERR_WORKSPACE;
  if ((st = rows_device()) != KD_OK || n == 0) return st;
  char* ws = static_cast<char*>(workspace);
  VerifyArgs a;
  memset(&a, 0, sizeof(a));
  a.zt = in->target_logits;
  a.zd = k > 0 && !greedy ? in->draft_logits : nullptr;
  a.drafts = in->drafts;
  a.lengths = in->lengths;
  a.u = in->uniform;
  a.noise = in->noise;
  a.b = n;
  a.vocab = v;
  a.ldt = p->ld_target ? p->ld_target : v;
  a.ldd = p->ld_draft ? p->ld_draft : v;
  a.ignore = p->ignore_index;
  a.k = (int)k;
  a.greedy = greedy;
  a.kt = greedy ? kL2E : kL2E / p->t_target;
  a.kd = kL2E / p->t_draft;
  a.inv_t = greedy ? 1.f : 1.f / p->t_target;
  a.parts = P.parts[a.zd != nullptr];
  a.race_parts = greedy ? 1 : P.race_parts;
  a.sums = reinterpret_cast<RowSum*>(ws + P.sums);
  a.leader = reinterpret_cast<uint64_t*>(ws + P.leader);
  a.arrived = reinterpret_cast<uint32_t*>(ws + P.arrived);
  a.tokens = tokens;
  a.accepted = accepted;
  a.logprob = logprob;
  a.status = dev_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t rows = P.rows[a.zd != nullptr];
  const bool ok = esz == 2 ? verify_run<__nv_bfloat16>(a, rows, s) : verify_run<float>(a, rows, s);
  return ok && cudaGetLastError() == cudaSuccess ? KD_OK : KD_ERR_CUDA;
}
