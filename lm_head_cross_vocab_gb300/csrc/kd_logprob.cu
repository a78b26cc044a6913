// Token log-probabilities: log p of given tokens, the entropy and the top
// alternatives of every row, from materialised logits or from hidden states
// and the head weight, and their backward passes.
//
// Per row, with k = log2(e) / T and m = max z, one sweep keeps
//   s = sum 2^x,  t = sum 2^x x,   x = (z - m) k
// (rescaled when the running maximum grows), and then
//   log S = ln s,  entropy = ln s - ln2 t / s,  log p_v = (z_v - m) / T - ln s.
// Nothing is taken as a difference of two large log-sum-exps, so rows of very
// large or very negative logits keep their absolute accuracy.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "kd_internal.h"

namespace kd {
namespace {

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
__device__ __forceinline__ LpState lp_empty() { return {neg_inf(), 0.f, 0.f}; }
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
__device__ __forceinline__ void lp_add(LpState& a, float z, float k) {
  if (z > a.m) lp_raise(a, z, k);
  if (z == neg_inf()) return;
  const float x = lp_x(z, a.m, k), e = ex2(x);
  a.s += e;
  a.t = fmaf(e, x, a.t);
}
__device__ __forceinline__ LpState lp_shfl_xor(const LpState& a, int o) {
  return {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o),
          __shfl_xor_sync(0xffffffffu, a.t, o)};
}

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

struct LpArgs {
  const void* z;          // [n, vocab] rows of pitch ld
  int64_t n, vocab, ld;
  float inv_t, k2;        // 1 / T, log2(e) / T
  const int64_t* tokens;  // may be NULL
  int64_t ignore;
  int topk;
  float *logprob, *entropy, *topk_lp, *stats;
  int32_t* topk_idx;
  uint32_t* status;
};

// Per-token outputs but the alternatives (one thread).
__device__ __forceinline__ void lp_store(const LpArgs& a, int64_t r, const LpRow& row, int64_t y,
                                         float zy) {
  if (a.logprob) {
    float v = __int_as_float(0x7fffffff);
    if (y >= 0 && y < a.vocab) v = lp_of(zy, row, a.inv_t);
    a.logprob[r] = v;
  }
  if (a.entropy) a.entropy[r] = row.ent;
  if (a.stats)
    reinterpret_cast<float4*>(a.stats)[r] =
        make_float4(row.m, row.log_s, row.ent, fmaf(row.m, a.inv_t, row.log_s));
}
// Outputs of an ignored row (all threads of the block).
__device__ __forceinline__ void lp_store_ignored(const LpArgs& a, int64_t r) {
  if (threadIdx.x == 0) {
    if (a.logprob) a.logprob[r] = 0.f;
    if (a.entropy) a.entropy[r] = 0.f;
    if (a.stats) reinterpret_cast<float4*>(a.stats)[r] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int j = threadIdx.x; j < a.topk; j += blockDim.x) {
    if (a.topk_idx) a.topk_idx[r * a.topk + j] = j;
    if (a.topk_lp) a.topk_lp[r * a.topk + j] = neg_inf();
  }
}

// ------------------------------------------------------------------ selection
struct SelectShared {
  uint64_t cand[kMaxTopk];
  uint32_t hist[256];
  uint32_t prefix, want, count;
  uint32_t warp_ties[32];
};

// The K best of a row by radix selection on the order keys: eight bits a
// sweep, then one sweep that collects what lies above the K-th key and the
// lowest ids among those equal to it.  Exact for any row.
template <class T>
__device__ void select_exact(const T* z, int64_t v, int k, SelectShared& sh) {
  const int tid = threadIdx.x, nt = blockDim.x;
  if (tid == 0) {
    sh.prefix = 0;
    sh.want = (uint32_t)k;
    sh.count = 0;
  }
  uint32_t mask = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += nt) sh.hist[i] = 0;
    __syncthreads();
    const uint32_t prefix = sh.prefix;
    for (int64_t i = tid; i < v; i += nt) {
      const uint32_t key = order_key(to_f(z[i]));
      if ((key & mask) == prefix) atomicAdd(&sh.hist[(key >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t want = sh.want, b = 255;
      while (b > 0 && sh.hist[b] < want) want -= sh.hist[b--];
      sh.want = want;
      sh.prefix = prefix | (b << shift);
    }
    mask |= 255u << shift;
    __syncthreads();
  }
  const uint32_t kth = sh.prefix, ties = sh.want;
  uint32_t seen = 0;
  for (int64_t base = 0; base < v; base += nt) {
    const int64_t i = base + tid;
    const uint32_t key = i < v ? order_key(to_f(z[i])) : 0u;
    if (i < v && key > kth) sh.cand[atomicAdd(&sh.count, 1u)] = cand_word(key, (uint32_t)i);
    const bool tie = i < v && key == kth;
    if (__syncthreads_or(tie && seen < ties)) {
      const uint32_t b = __ballot_sync(0xffffffffu, tie);
      if ((tid & 31) == 0) sh.warp_ties[tid >> 5] = __popc(b);
      __syncthreads();
      uint32_t before = seen, total = 0;
      for (int w = 0; w < nt / 32; ++w) {
        if (w < (tid >> 5)) before += sh.warp_ties[w];
        total += sh.warp_ties[w];
      }
      before += __popc(b & ((1u << (tid & 31)) - 1u));
      if (tie && before < ties)
        sh.cand[atomicAdd(&sh.count, 1u)] = cand_word(key, (uint32_t)i);
      seen += total;
      __syncthreads();
    }
  }
  __syncthreads();
}

// Writes the K candidates in order: each one's place is the number of larger
// words.
__device__ void write_top(const LpArgs& a, int64_t r, const uint64_t* cand, const LpRow& row) {
  for (int j = threadIdx.x; j < a.topk; j += blockDim.x) {
    const uint64_t w = cand[j];
    int place = 0;
    for (int i = 0; i < a.topk; ++i) place += cand[i] > w;
    if (a.topk_idx) a.topk_idx[r * a.topk + place] = (int32_t)~(uint32_t)w;
    if (a.topk_lp)
      a.topk_lp[r * a.topk + place] = lp_of(key_value((uint32_t)(w >> 32)), row, a.inv_t);
  }
}

// ------------------------------------------------------------------ forward
constexpr int kRowThreads = 256;

// One block per row.
template <class T>
__global__ void __launch_bounds__(kRowThreads) k_logprob_rows(LpArgs a) {
  __shared__ SelectShared sh;
  __shared__ LpState warp_state[kRowThreads / 32];
  const int64_t r = blockIdx.x;
  const T* z = static_cast<const T*>(a.z) + r * a.ld;
  const int64_t y = a.tokens ? a.tokens[r] : -1;
  if (a.tokens && y == a.ignore) {
    lp_store_ignored(a, r);
    return;
  }
  LpState st = lp_empty();
  for (int64_t i = threadIdx.x; i < a.vocab; i += kRowThreads) lp_add(st, to_f(z[i]), a.k2);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) lp_merge(st, lp_shfl_xor(st, o), a.k2);
  if ((threadIdx.x & 31) == 0) warp_state[threadIdx.x >> 5] = st;
  __syncthreads();
  st = warp_state[0];
  for (int w = 1; w < kRowThreads / 32; ++w) lp_merge(st, warp_state[w], a.k2);
  const LpRow row = lp_finish(st);
  if (threadIdx.x == 0) {
    const bool in = y >= 0 && y < a.vocab;
    if (a.tokens && !in) set_status(a.status, KD_DEV_BAD_LABEL);
    lp_store(a, r, row, y, in ? to_f(z[y]) : 0.f);
  }
  if (a.topk) {
    select_exact(z, a.vocab, a.topk, sh);
    write_top(a, r, sh.cand, row);
  }
}

template <class T>
void launch_rows(const LpArgs& a, cudaStream_t s) {
  if (a.n <= 0) return;
  note_launch();
  k_logprob_rows<T><<<(unsigned)a.n, kRowThreads, 0, s>>>(a);
}

// ------------------------------------------------------------------ backward
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
__device__ __forceinline__ float lp_grad(float z, const LpGradRow& g, float k) {
  const float x = max_nan(fmaf(z - g.m, k, -g.off), kXMin);
  return ex2(x) * fmaf(g.c1, x, g.c0);
}

template <class T, class O>
__global__ void __launch_bounds__(kRowThreads) k_logprob_grad(LpGradArgs a) {
  const int64_t r = blockIdx.x;
  const T* z = static_cast<const T*>(a.z) + r * a.ld;
  O* out = static_cast<O*>(a.g) + r * a.ldg;
  const LpGradRow g = lp_grad_row(a, r);
  for (int64_t i = threadIdx.x; i < a.cols; i += kRowThreads) {
    float v = 0.f;
    if (g.live) {
      v = lp_grad(to_f(z[i]), g, a.k2);
      if (a.col0 + i == g.y) v += g.cy;
    }
    from_f(v, out[i]);
  }
}

template <class T, class O>
void launch_grad(const LpGradArgs& a, cudaStream_t s) {
  if (a.n <= 0) return;
  note_launch();
  k_logprob_grad<T, O><<<(unsigned)a.n, kRowThreads, 0, s>>>(a);
}

// Copy of the hidden states with the rows of ignored tokens zeroed: their
// gradient rows are 0, but 0 times what a padded row holds need not be.
template <class T>
__global__ void __launch_bounds__(kRowThreads) k_mask_rows(const T* __restrict__ h, int64_t d,
                                                           const int64_t* tokens, int64_t ignore,
                                                           T* __restrict__ out) {
  const int64_t r = blockIdx.x;
  const bool live = !(tokens && tokens[r] == ignore);
  for (int64_t i = threadIdx.x; i < d; i += kRowThreads) {
    T v;
    from_f(0.f, v);
    out[r * d + i] = live ? h[r * d + i] : v;
  }
}

// ------------------------------------------------------------------ plan
constexpr size_t kAlign = 256;
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

struct LpPlan {
  bool hidden, bf16;
  int64_t n, v, d, ld, ldg;
  int nsm;
  float inv_t, k2;
  int64_t fr;               // forward: rows of a logit chunk
  int64_t R, C;             // backward: chunk of G
  size_t f_z, f_bytes;
  size_t b_h, b_z, b_g, b_dh, b_dw, b_bytes;
};

size_t take(size_t& off, size_t bytes) {
  const size_t o = off;
  off = align_up(off + bytes);
  return o;
}
template <class T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

kd_status lp_plan(const kd_logprob_problem* p, LpPlan& P) {
  memset(&P, 0, sizeof(P));
  if (!p) return KD_ERR_INVALID_ARG;
  if (p->n_tokens < 0 || p->n_tokens > INT32_MAX || p->vocab < 1 || p->vocab > (int64_t)1 << 30)
    return KD_ERR_INVALID_ARG;
  if (p->dtype != KD_BF16 && p->dtype != KD_FP32) return KD_ERR_INVALID_ARG;
  if (p->source != KD_STUDENT_HIDDEN && p->source != KD_STUDENT_LOGITS) return KD_ERR_INVALID_ARG;
  if (!(std::isfinite(p->temperature) && p->temperature > 0.f) ||
      !std::isfinite(kL2E / p->temperature))
    return KD_ERR_INVALID_ARG;
  if (p->topk < 0 || p->topk > kMaxTopk || p->topk > p->vocab) return KD_ERR_INVALID_ARG;
  P.hidden = p->source == KD_STUDENT_HIDDEN;
  P.bf16 = p->dtype == KD_BF16;
  P.n = p->n_tokens;
  P.v = p->vocab;
  P.d = p->d_model;
  P.ld = p->ld_logits ? p->ld_logits : P.v;
  P.ldg = p->ld_d_logits ? p->ld_d_logits : P.v;
  P.inv_t = 1.f / p->temperature;
  P.k2 = kL2E / p->temperature;
  P.nsm = std::max(1, tc_num_sms());
  if (!P.hidden) return (P.ld < P.v || P.ldg < P.v) ? KD_ERR_INVALID_ARG : KD_OK;
  if (P.d < 1 || P.d > (int64_t)1 << 30) return KD_ERR_INVALID_ARG;
  if (P.bf16 && P.d % 8) return KD_ERR_UNSUPPORTED;  // TMA row pitch
  // the fp32 product's grid: 64 columns a block, at most 65535 blocks
  if (!P.bf16 && (P.v > (int64_t)65535 * 64 || P.d > (int64_t)65535 * 64))
    return KD_ERR_UNSUPPORTED;
  const int64_t n = std::max<int64_t>(P.n, 1);
  // forward: fp32 logits of fr rows, at most 128 MiB (or one block of rows)
  P.fr = std::min(n, std::max<int64_t>(256, ((int64_t)32 << 20) / P.v / 256 * 256));
  size_t off = 0;
  P.f_z = take(off, (size_t)P.fr * P.v * 4);
  P.f_bytes = off;
  // backward
  kd_problem q;
  memset(&q, 0, sizeof(q));
  q.n_tokens = n;
  q.vocab = P.v;
  q.d_student = P.d;
  q.student = KD_STUDENT_HIDDEN;
  if (P.bf16) choose_chunk(&q, (int64_t)64 << 20, 256, 4, P.R, P.C);
  else choose_chunk(&q, (int64_t)8 << 20, 64, 8, P.R, P.C);
  off = 0;
  const size_t esz = P.bf16 ? 2 : 4;
  P.b_h = take(off, (size_t)n * P.d * esz);
  P.b_z = take(off, (size_t)P.R * P.C * 4);
  P.b_g = P.bf16 ? take(off, (size_t)P.R * P.C * 2) : P.b_z;  // fp32: G in place of z
  if (P.bf16 && cdiv(P.v, P.C) > 1) P.b_dh = take(off, (size_t)n * P.d * 4);
  if (P.bf16 && cdiv(n, P.R) > 1) P.b_dw = take(off, (size_t)P.v * P.d * 4);
  P.b_bytes = off;
  return KD_OK;
}

kd_status lp_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || !kd_device_supported(dev)) return KD_ERR_NO_DEVICE;
  return KD_OK;
}

kd_status lp_inputs(const LpPlan& P, const kd_logprob_inputs* in) {
  if (!in) return KD_ERR_INVALID_ARG;
  if (P.n == 0) return KD_OK;
  if (!P.hidden) return in->logits ? KD_OK : KD_ERR_INVALID_ARG;
  if (!in->h || !in->w) return KD_ERR_INVALID_ARG;
  if (P.bf16 && (!aligned16(in->h) || !aligned16(in->w))) return KD_ERR_UNSUPPORTED;
  return KD_OK;
}

bool ws_ok(const void* ws, size_t have, size_t need) {
  return need == 0 || (ws && have >= need && reinterpret_cast<uintptr_t>(ws) % kAlign == 0);
}

// z[rows, cols] (fp32, pitch ldz) = H[r0.., :] W[c0.., :]^T
int lp_logits(const LpPlan& P, const kd_logprob_inputs* in, int64_t r0, int64_t rows, int64_t c0,
              int64_t cols, float* z, int64_t ldz, uint32_t* status, cudaStream_t s) {
  if (!P.bf16) {
    const float* h = static_cast<const float*>(in->h) + r0 * P.d;
    const float* w = static_cast<const float*>(in->w) + c0 * P.d;
    launch_simt_gemm(h, P.d, 1, w, 1, P.d, z, ldz, rows, cols, P.d, false, s);
    return 0;
  }
  TcGemmArgs g;
  memset(&g, 0, sizeof(g));
  g.a0 = static_cast<const __nv_bfloat16*>(in->h) + r0 * P.d;
  g.b0 = static_cast<const __nv_bfloat16*>(in->w) + c0 * P.d;
  g.lda0 = g.ldb0 = P.d;
  g.M = rows;
  g.N = cols;
  g.K0 = P.d;
  g.mode = TC_OUT_F32;
  g.c32 = z;
  g.ldc32 = ldz;
  g.status = status;
  return launch_tc_gemm(g, P.nsm, s);
}

}  // namespace
}  // namespace kd

using namespace kd;

extern "C" kd_status kd_logprob_workspace_size(const kd_logprob_problem* problem,
                                               size_t* fwd_bytes, size_t* bwd_bytes) {
  LpPlan P;
  const kd_status st = lp_plan(problem, P);
  if (st != KD_OK) return st;
  if (fwd_bytes) *fwd_bytes = P.f_bytes;
  if (bwd_bytes) *bwd_bytes = P.b_bytes;
  return KD_OK;
}

extern "C" kd_status kd_logprob_fwd(const kd_logprob_problem* p, const kd_logprob_inputs* in,
                                    float* logprob, float* entropy, int32_t* topk_idx,
                                    float* topk_logprob, float* stats, uint32_t* dev_status,
                                    void* workspace, size_t ws_bytes, void* stream) {
  LpPlan P;
  kd_status st = lp_plan(p, P);
  if (st == KD_OK) st = lp_inputs(P, in);
  if (st != KD_OK) return st;
  if (logprob && !in->tokens && P.n > 0) return KD_ERR_INVALID_ARG;
  if (stats && !aligned16(stats)) return KD_ERR_INVALID_ARG;
  if (!ws_ok(workspace, ws_bytes, P.f_bytes)) return KD_ERR_WORKSPACE;
  st = lp_device();
  if (st != KD_OK) return st;
  if (P.n == 0 || (!logprob && !entropy && !topk_idx && !topk_logprob && !stats)) return KD_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int k = (topk_idx || topk_logprob) ? p->topk : 0;
  LpArgs a;
  memset(&a, 0, sizeof(a));
  a.vocab = P.v;
  a.inv_t = P.inv_t;
  a.k2 = P.k2;
  a.ignore = p->ignore_index;
  a.topk = k;
  a.status = dev_status;
  auto rows_from = [&](int64_t r0, int64_t n) {
    a.n = n;
    a.tokens = in->tokens ? in->tokens + r0 : nullptr;
    a.logprob = logprob ? logprob + r0 : nullptr;
    a.entropy = entropy ? entropy + r0 : nullptr;
    a.stats = stats ? stats + r0 * KD_LOGPROB_STATS : nullptr;
    a.topk_idx = topk_idx ? topk_idx + r0 * k : nullptr;
    a.topk_lp = topk_logprob ? topk_logprob + r0 * k : nullptr;
  };
  if (!P.hidden) {
    rows_from(0, P.n);
    a.z = in->logits;
    a.ld = P.ld;
    if (P.bf16) launch_rows<__nv_bfloat16>(a, s);
    else launch_rows<float>(a, s);
  } else {
    float* z = at<float>(workspace, P.f_z);
    a.z = z;
    a.ld = P.v;
    for (int64_t r0 = 0; r0 < P.n; r0 += P.fr) {
      const int64_t rows = std::min(P.fr, P.n - r0);
      if (lp_logits(P, in, r0, rows, 0, P.v, z, P.v, dev_status, s)) return KD_ERR_CUDA;
      rows_from(r0, rows);
      launch_rows<float>(a, s);
    }
  }
  return cudaGetLastError() == cudaSuccess ? KD_OK : KD_ERR_CUDA;
}

extern "C" kd_status kd_logprob_bwd(const kd_logprob_problem* p, const kd_logprob_inputs* in,
                                    const float* stats, const float* d_logprob,
                                    const float* d_entropy, void* d_h, void* d_w, void* d_logits,
                                    uint32_t* dev_status, void* workspace, size_t ws_bytes,
                                    void* stream) {
  LpPlan P;
  kd_status st = lp_plan(p, P);
  if (st == KD_OK) st = lp_inputs(P, in);
  if (st != KD_OK) return st;
  if (P.hidden ? d_logits != nullptr : (d_h || d_w)) return KD_ERR_INVALID_ARG;
  if (P.n > 0 && (!stats || !aligned16(stats) || (d_logprob && !in->tokens)))
    return KD_ERR_INVALID_ARG;
  if (!ws_ok(workspace, ws_bytes, P.b_bytes)) return KD_ERR_WORKSPACE;
  st = lp_device();
  if (st != KD_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t esz = P.bf16 ? 2 : 4;
  if (P.n == 0) {
    if (d_w && cudaMemsetAsync(d_w, 0, (size_t)P.v * P.d * esz, s) != cudaSuccess)
      return KD_ERR_CUDA;
    return KD_OK;
  }
  LpGradArgs a;
  memset(&a, 0, sizeof(a));
  a.vocab = P.v;
  a.inv_t = P.inv_t;
  a.k2 = P.k2;
  a.ignore = p->ignore_index;
  a.status = dev_status;
  if (!P.hidden) {
    if (!d_logits) return KD_OK;
    a.z = in->logits;
    a.n = P.n;
    a.cols = P.v;
    a.ld = P.ld;
    a.tokens = in->tokens;
    a.stats = stats;
    a.d_lp = d_logprob;
    a.d_ent = d_entropy;
    a.g = d_logits;
    a.ldg = P.ldg;
    if (P.bf16) launch_grad<__nv_bfloat16, __nv_bfloat16>(a, s);
    else launch_grad<float, float>(a, s);
    return cudaGetLastError() == cudaSuccess ? KD_OK : KD_ERR_CUDA;
  }
  if (!d_h && !d_w) return KD_OK;
  const int64_t n = P.n, v = P.v, D = P.d, R = P.R, C = P.C;
  const int64_t nr = cdiv(n, R), nc = cdiv(v, C);
  float* z = at<float>(workspace, P.b_z);
  void* g = at<char>(workspace, P.b_g);
  void* hm = at<char>(workspace, P.b_h);
  if (d_w) {
    note_launch();
    if (P.bf16)
      k_mask_rows<__nv_bfloat16><<<(unsigned)n, kRowThreads, 0, s>>>(
          static_cast<const __nv_bfloat16*>(in->h), D, in->tokens, p->ignore_index,
          static_cast<__nv_bfloat16*>(hm));
    else
      k_mask_rows<float><<<(unsigned)n, kRowThreads, 0, s>>>(
          static_cast<const float*>(in->h), D, in->tokens, p->ignore_index,
          static_cast<float*>(hm));
  }
  for (int64_t ri = 0; ri < nr; ++ri) {
    const int64_t r0 = ri * R, rc = std::min(R, n - r0);
    for (int64_t ci = 0; ci < nc; ++ci) {
      const int64_t c0 = ci * C, cc = std::min(C, v - c0);
      if (lp_logits(P, in, r0, rc, c0, cc, z, C, dev_status, s)) return KD_ERR_CUDA;
      a.z = z;
      a.n = rc;
      a.cols = cc;
      a.col0 = c0;
      a.ld = a.ldg = C;
      a.tokens = in->tokens ? in->tokens + r0 : nullptr;
      a.stats = stats + r0 * KD_LOGPROB_STATS;
      a.d_lp = d_logprob ? d_logprob + r0 : nullptr;
      a.d_ent = d_entropy ? d_entropy + r0 : nullptr;
      a.g = g;
      if (!P.bf16) {
        launch_grad<float, float>(a, s);
        const float* gf = static_cast<const float*>(g);
        if (d_h)
          launch_simt_gemm(gf, C, 1, static_cast<const float*>(in->w) + c0 * D, D, 1,
                           static_cast<float*>(d_h) + r0 * D, D, rc, D, cc, ci > 0, s);
        if (d_w)
          launch_simt_gemm(gf, 1, C, static_cast<const float*>(hm) + r0 * D, D, 1,
                           static_cast<float*>(d_w) + c0 * D, D, cc, D, rc, ri > 0, s);
        continue;
      }
      launch_grad<float, __nv_bfloat16>(a, s);
      auto product = [&](const __nv_bfloat16* b, int64_t m, int64_t kk, bool a_mn, float* acc,
                         __nv_bfloat16* out, int64_t i, int64_t parts) {
        TcGemmArgs t;
        memset(&t, 0, sizeof(t));
        t.a0 = static_cast<const __nv_bfloat16*>(g);
        t.lda0 = C;
        t.a0_mn = a_mn;
        t.b0 = b;
        t.ldb0 = D;
        t.b0_mn = 1;
        t.M = m;
        t.N = D;
        t.K0 = kk;
        t.mode = parts == 1      ? TC_OUT_BF16
                 : i == 0        ? TC_OUT_F32
                 : i + 1 < parts ? TC_OUT_F32_ACC
                                 : TC_OUT_F32_ACC_BF16;
        t.c32 = acc;
        t.ldc32 = D;
        t.c16 = out;
        t.ldc16 = D;
        t.status = dev_status;
        return launch_tc_gemm(t, P.nsm, s);
      };
      if (d_h && product(static_cast<const __nv_bfloat16*>(in->w) + c0 * D, rc, cc, false,
                         nc > 1 ? at<float>(workspace, P.b_dh) + r0 * D : nullptr,
                         static_cast<__nv_bfloat16*>(d_h) + r0 * D, ci, nc))
        return KD_ERR_CUDA;
      if (d_w && product(static_cast<const __nv_bfloat16*>(hm) + r0 * D, cc, rc, true,
                         nr > 1 ? at<float>(workspace, P.b_dw) + c0 * D : nullptr,
                         static_cast<__nv_bfloat16*>(d_w) + c0 * D, ri, nr))
        return KD_ERR_CUDA;
    }
  }
  return cudaGetLastError() == cudaSuccess ? KD_OK : KD_ERR_CUDA;
}
