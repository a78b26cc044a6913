// Per-row arithmetic of the token log-probabilities, shared by the kernels over
// materialised logits (kd_logprob.cu) and the tensor-core epilogues (kd_tc.cu).
//
// Per row, with k = log2(e) / T and m = max z, one sweep keeps
//   s = sum 2^x,  t = sum 2^x x,   x = (z - m) k
// (rescaled when the running maximum grows), and then
//   log S = ln s,  entropy = ln s - ln2 t / s,  log p_v = (z_v - m) / T - ln s.
// Nothing is taken as a difference of two large log-sum-exps, so rows of very
// large or very negative logits keep their absolute accuracy.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kd_common.cuh"
#include "kd_internal.h"

namespace kd {

constexpr int kMaxTopk = 1024;
constexpr float kLn2 = 0.6931471805599453f;
// Exponents below this give 2^x = 0 in fp32; x is held above it so that the
// product 2^x x of an id of probability 0 (z = -inf among others) is 0.
constexpr float kXMin = -160.f;

// ------------------------------------------------------------------ elements
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16& o) { o = __float2bfloat16(v); }

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Order of logits as unsigned integers: larger logit, larger key; -0 = +0; a
// NaN above every number.
__device__ __forceinline__ uint32_t order_key(float z) {
  if (z != z) return 0xffffffffu;
  const uint32_t b = __float_as_uint(z + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  if (key == 0xffffffffu) return __int_as_float(0x7fffffff);
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}
// Candidate: key above, complement of the id below, so that a larger word is
// an earlier alternative (ties to the lowest id) and no two are equal.
__device__ __forceinline__ uint64_t cand_word(uint32_t key, uint32_t id) {
  return ((uint64_t)key << 32) | (uint32_t)~id;
}

// ------------------------------------------------------------------ statistics
struct LpState {
  float m, s, t;
};
// 2^((z - m) k) and its exponent, for z <= m (NaN kept)
__device__ __forceinline__ float lp_x(float z, float m, float k) {
  return max_nan((z - m) * k, kXMin);
}
// Rescale of s and t when the maximum moves from a.m up to m.
__device__ __forceinline__ void lp_raise(LpState& a, float m, float k) {
  if (a.m == m) return;
  const float x = lp_x(a.m, m, k), f = ex2(x);
  a.t = f * fmaf(a.s, x, a.t);
  a.s = f * a.s;
  a.m = m;
}
__device__ __forceinline__ void lp_merge(LpState& a, LpState b, float k) {
  const float m = fmaxf(a.m, b.m);
  lp_raise(a, m, k);
  lp_raise(b, m, k);
  a.s += b.s;
  a.t += b.t;
}
__device__ __forceinline__ LpState lp_shfl_xor(const LpState& a, int o) {
  return {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o),
          __shfl_xor_sync(0xffffffffu, a.t, o)};
}

// Running sums of one thread, against an exponent offset that trails the
// running maximum by up to kRaise (terms of at most 2^kRaise), so that most
// chunks of a row need no rescale.  The caller raises before it adds.
constexpr float kRaise = 8.f;

struct LpFold {
  float off, off_up, k;  // offset; a logit above off_up asks for a raise
  float top;             // true maximum
  float2 s, t;

  __device__ __forceinline__ void init(float k_) {
    k = k_;
    off = off_up = top = neg_inf();
    s = t = make_float2(0.f, 0.f);
  }
  __device__ __forceinline__ void raise(float m) {
    const float x = lp_x(off, m, k), f = ex2(x);
    const float2 ff = make_float2(f, f);
    t = mul2(ff, fma2(s, make_float2(x, x), t));
    s = mul2(ff, s);
    off = m;
    off_up = m + kRaise / k;
  }
  // the maximum of the logits that follow (not -inf)
  __device__ __forceinline__ void expect(float m) {
    top = fmaxf(top, m);
    if (m > off_up) raise(m);
  }
  __device__ __forceinline__ void add_pair(float z0, float z1) {
    float2 x = mul2(sub2(make_float2(z0, z1), make_float2(off, off)), make_float2(k, k));
    x.x = max_nan(x.x, kXMin);
    x.y = max_nan(x.y, kXMin);
    const float2 e = make_float2(ex2(x.x), ex2(x.y));
    s = add2(s, e);
    t = fma2(e, x, t);
  }
  __device__ __forceinline__ void add_one(float z) {
    if (z == neg_inf()) return;
    expect(z);
    const float x = lp_x(z, off, k), e = ex2(x);
    s.x += e;
    t.x = fmaf(e, x, t.x);
  }
  // sums relative to the true maximum
  __device__ __forceinline__ LpState state() const {
    LpState a{off, s.x + s.y, t.x + t.y};
    lp_raise(a, top, k);
    return a;
  }
};

struct LpRow {
  float m, log_s, ent;
};
// m = -inf: no id has any probability (log S is 0 then, or NaN beside a NaN)
__device__ __forceinline__ LpRow lp_finish(const LpState& a) {
  LpRow r;
  r.m = a.m;
  if (a.m == neg_inf() && !(a.s != a.s)) {
    r.log_s = 0.f;
    r.ent = 0.f;
  } else {
    r.log_s = logf(a.s);
    const float h = r.log_s - kLn2 * (a.t / a.s);
    r.ent = h < 0.f ? 0.f : h;
  }
  return r;
}
__device__ __forceinline__ float lp_of(float z, const LpRow& r, float inv_t) {
  return r.m == neg_inf() && r.log_s == 0.f ? neg_inf() : fmaf(z - r.m, inv_t, -r.log_s);
}

struct LpGradArgs {
  const void* z;          // [n, cols] rows of pitch ld: columns col0 .. of the vocabulary
  int64_t n, cols, ld, col0, vocab;
  float inv_t, k2;
  const int64_t* tokens;
  int64_t ignore;
  const float *stats, *d_lp, *d_ent;
  void* g;                // [n, cols] rows of pitch ldg
  int64_t ldg;
  uint32_t* status;
};

// dz_v = p (c0 + c1 x) + [v = y] cy with x = log2 p:
//   c0 = -(g_l + g_H H) / T, c1 = -g_H ln2 / T, cy = g_l / T
struct LpGradRow {
  float m, off;          // x = (z - m) k - off, off = log2 S
  float c0, c1, cy;
  int64_t y;
  bool live;             // false: a zero row
};
__device__ __forceinline__ LpGradRow lp_grad_row(const LpGradArgs& a, int64_t r) {
  LpGradRow g;
  const int64_t y = a.tokens ? a.tokens[r] : -1;
  g.live = !(a.tokens && y == a.ignore);
  g.y = -1;
  g.m = g.off = g.c0 = g.c1 = g.cy = 0.f;
  if (!g.live) return g;
  const float4 st = reinterpret_cast<const float4*>(a.stats)[r];
  float gl = a.d_lp ? a.d_lp[r] : 0.f;
  const float gh = a.d_ent ? a.d_ent[r] : 0.f;
  const bool in = y >= 0 && y < a.vocab;
  if (!in) {
    if (a.tokens) set_status(a.status, KD_DEV_BAD_LABEL);
    gl = 0.f;
  }
  if (st.x == neg_inf() && st.y == 0.f) {
    g.live = false;
    return g;
  }
  g.y = in ? y : -1;
  g.m = st.x;
  g.off = st.y * kL2E;
  g.c0 = -(gl + gh * st.z) * a.inv_t;
  g.c1 = -gh * kLn2 * a.inv_t;
  g.cy = gl * a.inv_t;
  return g;
}
__device__ __forceinline__ void lp_grad_pair(float& z0, float& z1, const LpGradRow& g, float k) {
  float2 x = mul2(sub2(make_float2(z0, z1), make_float2(g.m, g.m)), make_float2(k, k));
  x = sub2(x, make_float2(g.off, g.off));
  x.x = max_nan(x.x, kXMin);
  x.y = max_nan(x.y, kXMin);
  x = mul2(make_float2(ex2(x.x), ex2(x.y)),
           fma2(make_float2(g.c1, g.c1), x, make_float2(g.c0, g.c0)));
  z0 = x.x;
  z1 = x.y;
}
__device__ __forceinline__ float lp_grad(float z, const LpGradRow& g, float k) {
  const float x = max_nan(fmaf(z - g.m, k, -g.off), kXMin);
  return ex2(x) * fmaf(g.c1, x, g.c0);
}

// The terms of one row of a product (kd_internal.h).
struct TermRow {
  int n;
  const __nv_bfloat16* src[kTermRows];
  float c[kTermRows];
};
__device__ __forceinline__ TermRow term_row(const TcTerms& t, int64_t o) {
  TermRow r;
  r.n = 0;
  int q[kTermRows];
#pragma unroll
  for (int i = 0; i < kTermRows; ++i) q[i] = INT32_MAX;
  if (t.one_q) {
    const int64_t y = t.one_q[o];
    if (y >= 0 && y < t.src_rows) {
      r.n = 1;
      r.src[0] = t.src + y * t.ld_src;
      r.c[0] = t.one_c[o];
    }
    return r;
  }
  const int n = t.count[o];
  if (n < 1 || n > kTermRows) return r;
  r.n = n;
#pragma unroll
  for (int i = 0; i < kTermRows; ++i)
    if (i < n) q[i] = t.list[o * kTermRows + i];
  // in ascending order, however they were listed
#pragma unroll
  for (int i = 0; i < kTermRows; ++i)
#pragma unroll
    for (int j = 0; j + 1 < kTermRows - i; ++j) {
      const int a = min(q[j], q[j + 1]), b = max(q[j], q[j + 1]);
      q[j] = a;
      q[j + 1] = b;
    }
#pragma unroll
  for (int i = 0; i < kTermRows; ++i)
    if (i < n) {
      r.src[i] = t.src + q[i] * t.ld_src;
      r.c[i] = t.one_c[q[i]];
    }
  return r;
}

}  // namespace kd
