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
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "kd_internal.h"
#include "kd_logprob.cuh"

namespace cg = cooperative_groups;

namespace kd {
namespace {

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

// ------------------------------------------------------------------ rows
// One block of NT threads takes a row, or, when there are too few rows to fill
// the device, a cluster of blocks takes it in slices that are joined through
// distributed shared memory.  A slice is read once, 64 contiguous bytes a thread
// and step, the next step's in flight beside the one being folded into (offset, s,
// t); the offset trails the running maximum by up to 2^8, so that most steps need
// no rescale.  What the K best cost on top: each thread keeps the maximum of every
// slot (a step, or a run of them, at most kSlots) and of all; the K-th largest of
// the threads' maxima (of the slots' for many alternatives) bounds the K-th
// largest logit from below, so only the 64 bytes of the few slots above it are
// read again, and what lies above the bound in them, little more than K ids, is
// put in order.
//
// Without alternatives bound by HBM: 4096 x 151936 bf16 177-180 us (6.9-7.0 TB/s),
// fp32 333-340 us (7.4 TB/s), 16384 x 32000 bf16 155 us.  With them a block's
// selection follows its sweep, about 16000 of its 62000 cycles with 100, and the
// four blocks of an SM do not quite cover one another's: 199-204 us with 20,
// 219-222 us with 100 (5.6 TB/s), 375 us in fp32.  Nothing of a row is in local memory (the
// selection out of line, with what it needs spilled, 278 us: the sweeps push such
// lines out of L1), and its steps are few instructions, which wait their turn
// behind the other blocks' sweeps.  Few rows, bound by latency: one row of 151936
// 4.2-4.8 us, with 20 alternatives 7.6-8.0 us, with 100 9.8-10.1 us (8 blocks).
constexpr int kSlots = 32;
// slots above the bound the lists of a block's warps hold
constexpr int row_pairs(int nt) { return nt == 128 ? 1024 : 4096; }
constexpr int kMaxCap = 4096;  // candidates a block sorts at most
constexpr int kFewK = 128, kFewCap = 1024;  // with up to kFewK alternatives
constexpr int kUnroll = 4;
constexpr int kOwn = 256;      // maxima that bound few alternatives, one or two a thread

struct Words {
  uint32_t w[4];
};
__device__ __forceinline__ Words load16(const void* p) {
  Words v;
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3])
               : "l"(p));
  return v;
}
// 32 bytes (and a 32-byte boundary): one sector a lane.
__device__ __forceinline__ void load32(const void* p, Words& a, Words& b) {
  asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(a.w[0]), "=r"(a.w[1]), "=r"(a.w[2]), "=r"(a.w[3]), "=r"(b.w[0]),
                 "=r"(b.w[1]), "=r"(b.w[2]), "=r"(b.w[3])
               : "l"(p));
}
// A vector of the row: elements, and -inf in each.
template <class T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kNone = 0xff800000u;
  static __device__ __forceinline__ void get(const Words& v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v.w[i]);
  }
  static __device__ __forceinline__ float top(const Words& v) {
    return max_nan(max_nan(__uint_as_float(v.w[0]), __uint_as_float(v.w[1])),
                   max_nan(__uint_as_float(v.w[2]), __uint_as_float(v.w[3])));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t kNone = kNegInfX2;
  static __device__ __forceinline__ void get(const Words& v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16lo(v.w[i]);
      f[2 * i + 1] = bf16hi(v.w[i]);
    }
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ float top(const Words& v) {
    const uint32_t m = max2(max2(v.w[0], v.w[1]), max2(v.w[2], v.w[3]));
    return max_nan(bf16lo(m), bf16hi(m));
  }
};

// The part of a row one block takes: `nvec` vectors of 16 bytes, an even number,
// from the 32-byte boundary `head` elements into the row (those of all blocks of
// the cluster together cover the row's); block 0 takes the `loose` elements
// before and behind them as well.  A thread takes 64 bytes, the least that HBM
// gives, at a time: they are what it reads again.
template <class T>
struct Slice {
  const T* z;
  int nvec, chunks, rounds;  // vectors; runs of four; vectors of a thread
  int head, loose, base;     // base: element index of vector 0 of the slice
  int64_t vocab;

  // 1 << lb blocks
  __device__ __forceinline__ Slice(const T* row, int64_t vocab_, int rank, int lb, int nt) {
    constexpr int N = Vec<T>::N;
    z = row;
    vocab = vocab_;
    const int off = (int)((reinterpret_cast<uintptr_t>(row) & 31) / sizeof(T));
    head = off ? 2 * N - off : 0;
    if (head > vocab) head = (int)vocab;
    const int64_t all = (vocab - head) / (2 * N), v0 = all * rank >> lb;
    nvec = 2 * (int)((all * (rank + 1) >> lb) - v0);
    chunks = (nvec + 3) / 4;
    rounds = (chunks + nt - 1) / nt * 4;
    loose = rank == 0 ? (int)(vocab - all * 2 * N) : 0;
    base = head + (int)v0 * 2 * N;
  }
  __device__ __forceinline__ const T* at_vec(int i) const { return z + base + (int64_t)i * Vec<T>::N; }
  __device__ __forceinline__ Words vec(int i) const { return load16(at_vec(i)); }
  // step j of thread t of nt; -inf behind the vectors
  __device__ __forceinline__ void chunk(int j, int t, int nt, Words* w) const {
    const int c = j * nt + t;
    if (4 * (j + 1) * nt <= nvec) {
      load32(at_vec(4 * c), w[0], w[1]);
      load32(at_vec(4 * c + 2), w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i / 4].w[i % 4] = Vec<T>::kNone;
      if (4 * c < nvec) load32(at_vec(4 * c), w[0], w[1]);
      if (4 * c + 2 < nvec) load32(at_vec(4 * c + 2), w[2], w[3]);
    }
  }
  // asks L2 for the bytes of steps j and j + 1 of nt threads, if both are whole
  __device__ __forceinline__ void prefetch(int j, int nt) const {
    if (4 * (j + 2) * nt <= nvec)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at_vec(4 * j * nt)),
                   "r"(2 * 4 * nt * 16)
                   : "memory");
  }
  __device__ __forceinline__ int64_t loose_at(int i) const { return i < head ? i : vocab - loose + i; }
  // elements of the slice, in the order of their ids, for the exact selection
  __device__ __forceinline__ int64_t size() const { return (int64_t)nvec * Vec<T>::N + loose; }
  __device__ __forceinline__ int64_t at(int64_t i) const {
    if (loose == 0) return base + i;
    if (i < head) return i;
    i -= head;
    const int64_t body = (int64_t)nvec * Vec<T>::N;
    return i < body ? base + i : vocab - loose + head + (i - body);
  }
};

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Shared memory of the selection; cand has `cap` places.
struct SelectShared {
  uint32_t hist[256];
  uint32_t prefix, want, count, bound;
  uint32_t warp_sum[2][32];
};

// The K best of a slice by radix selection on the order keys: eight bits a
// sweep, then one sweep that collects what lies above the K-th key and the
// lowest ids among those equal to it.  Exact for any row; taken where too many
// ids lie at or above the bound (long runs of equal logits).
template <class T>
__device__ __noinline__ void select_exact(Slice<T> sl, int k, SelectShared& sh, uint64_t* cand) {
  const int tid = threadIdx.x, nt = blockDim.x;
  const int64_t v = sl.size();
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
      const uint32_t key = order_key(to_f(sl.z[sl.at(i)]));
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
    const int64_t id = i < v ? sl.at(i) : 0;
    const uint32_t key = i < v ? order_key(to_f(sl.z[id])) : 0u;
    if (i < v && key > kth) cand[atomicAdd(&sh.count, 1u)] = cand_word(key, (uint32_t)id);
    const bool tie = i < v && key == kth;
    if (__syncthreads_or(tie && seen < ties)) {
      const uint32_t b = __ballot_sync(0xffffffffu, tie);
      if ((tid & 31) == 0) sh.warp_sum[0][tid >> 5] = __popc(b);
      __syncthreads();
      uint32_t before = seen, total = 0;
      for (int w = 0; w < nt / 32; ++w) {
        if (w < (tid >> 5)) before += sh.warp_sum[0][w];
        total += sh.warp_sum[0][w];
      }
      before += __popc(b & ((1u << (tid & 31)) - 1u));
      if (tie && before < ties) cand[atomicAdd(&sh.count, 1u)] = cand_word(key, (uint32_t)id);
      seen += total;
      __syncthreads();
    }
  }
  __syncthreads();
}

// Largest 16-bit key that at least k of 32 P keys reach, k <= 32 P: one
// warp, two bits a step below the highest bit in which the keys differ, so that
// the other blocks of the SM keep the issue slots.
template <int P>
__device__ __forceinline__ void bound_key(const uint16_t* keys, int k, uint32_t* out) {
  uint32_t key[P], lo = 0xffffu, hi = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    key[i] = keys[i * 32 + threadIdx.x];
    lo = min(lo, key[i]);
    hi = max(hi, key[i]);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  int shift = (32 - __clz(lo ^ hi) + 1) & ~1;  // even; bits below it may differ
  lo = lo >> shift << shift;
#pragma unroll 1
  while ((shift -= 2) >= 0) {
    uint32_t c[3] = {0, 0, 0};
#pragma unroll
    for (int q = 0; q < 3; ++q) {
#pragma unroll
      for (int i = 0; i < P; ++i) c[q] += key[i] >= (lo | ((uint32_t)(q + 1) << shift));
      c[q] = __reduce_add_sync(0xffffffffu, c[q]);
    }
    lo |= (uint32_t)((c[0] >= (uint32_t)k) + (c[1] >= (uint32_t)k) + (c[2] >= (uint32_t)k))
          << shift;
  }
  if (threadIdx.x == 0) *out = lo;
}
// The same over all slots of all threads: block-wide counts.
template <int NT>
__device__ __forceinline__ uint32_t bound_key_slots(const uint16_t* keys, int slots, int k, SelectShared& sh) {
  constexpr int W = NT / 32;
  static_assert(2 * 3 * W <= 256, "counts of two steps");
  const int warp = threadIdx.x >> 5;
  const bool lane0 = (threadIdx.x & 31) == 0;
  uint32_t lo = 0xffffu, hi = 0;
#pragma unroll 8
  for (int i = 0; i < slots; ++i) {
    lo = min(lo, (uint32_t)keys[i * NT + threadIdx.x]);
    hi = max(hi, (uint32_t)keys[i * NT + threadIdx.x]);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane0) {
    sh.warp_sum[0][warp] = lo;
    sh.warp_sum[1][warp] = hi;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) {
    lo = min(lo, sh.warp_sum[0][w]);
    hi = max(hi, sh.warp_sum[1][w]);
  }
  int shift = (32 - __clz(lo ^ hi) + 1) & ~1;  // even; bits below it may differ
  lo = lo >> shift << shift;
  uint32_t* sum = sh.hist;
#pragma unroll 1
  while ((shift -= 2) >= 0) {
    const uint32_t t = 1u << shift;
    uint32_t c0 = 0, c1 = 0, c2 = 0;
#pragma unroll 4
    for (int i = 0; i < slots; ++i) {
      const uint32_t q = keys[i * NT + threadIdx.x];
      c0 += q >= (lo | t);
      c1 += q >= (lo | 2 * t);
      c2 += q >= (lo | 3 * t);
    }
    c0 = __reduce_add_sync(0xffffffffu, c0);
    c1 = __reduce_add_sync(0xffffffffu, c1);
    c2 = __reduce_add_sync(0xffffffffu, c2);
    if (lane0) {
      sum[warp] = c0;
      sum[W + warp] = c1;
      sum[2 * W + warp] = c2;
    }
    __syncthreads();
    c0 = c1 = c2 = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      c0 += sum[w];
      c1 += sum[W + w];
      c2 += sum[2 * W + w];
    }
    lo |= (uint32_t)((c0 >= (uint32_t)k) + (c1 >= (uint32_t)k) + (c2 >= (uint32_t)k)) << shift;
    sum = sh.hist + (sum == sh.hist ? 3 * W : 0);  // alternately: one barrier a step
  }
  return lo;
}

// One step of a bitonic sort, descending where `down`: of two words the one
// that belongs at the lower index.
__device__ __forceinline__ void exchange(uint64_t& a, uint64_t& b, bool down) {
  if ((a < b) == down) {
    const uint64_t t = a;
    a = b;
    b = t;
  }
}
// Descending bitonic sort of NT * E words, zeros behind the first n.  Thread t
// holds words t E .. t E + E - 1, so steps below E stay in its registers, steps
// below 32 E in its warp, and only the few above go through shared memory.
template <int NT, int E>
__device__ __forceinline__ void sort_bitonic(uint64_t* cand, int n) {
  const int t0 = threadIdx.x * E;
  uint64_t w[E];
#pragma unroll
  for (int i = 0; i < E; ++i) w[i] = t0 + i < n ? cand[t0 + i] : 0;
#pragma unroll 1
  for (int size = 2; size <= NT * E; size <<= 1) {
#pragma unroll 1
    for (int step = size >> 1; step >= E; step >>= 1) {
      const bool low = (t0 & step) == 0;         // this thread's words are the lower ones
      const bool keep_max = ((t0 & size) == 0) == low;
      if (step < 32 * E) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const uint64_t o = __shfl_xor_sync(0xffffffffu, w[i], step / E);
          w[i] = keep_max ? max(w[i], o) : min(w[i], o);
        }
      } else {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < E; ++i) cand[i * NT + threadIdx.x] = w[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const uint64_t o = cand[i * NT + (threadIdx.x ^ (step / E))];
          w[i] = keep_max ? max(w[i], o) : min(w[i], o);
        }
      }
    }
#pragma unroll
    for (int step = E / 2; step > 0; step >>= 1) {
      if (step > size >> 1) continue;
#pragma unroll
      for (int i = 0; i < E; ++i)
        if ((i & step) == 0) exchange(w[i], w[i + step], ((t0 + i) & size) == 0);
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < E; ++i) cand[t0 + i] = w[i];
  __syncthreads();
}
// More than 2 NT words, out of line: the sweep has no registers to spare for them.
// Of more than 8 NT only the first 4 NT in order, the best of two halves (with 16
// words a thread the kernel's registers do not suffice).
template <int NT, int CAP>
__device__ __noinline__ void sort_many(uint64_t* cand, int n) {
  static_assert(CAP <= 16 * NT, "");
  if (n <= 4 * NT) return sort_bitonic<NT, 4>(cand, n);
  if constexpr (CAP > 8 * NT) {
    static_assert(4 * NT >= kMaxTopk, "as many as are asked for");
    if (n > 8 * NT) {
      sort_bitonic<NT, 8>(cand + 8 * NT, n - 8 * NT);
      sort_bitonic<NT, 8>(cand, 8 * NT);
      for (int i = threadIdx.x; i < 4 * NT; i += NT) cand[4 * NT + i] = cand[8 * NT + i];
      __syncthreads();
      n = 8 * NT;
    }
  }
  sort_bitonic<NT, 8>(cand, n);
}
// How many of cand[i, end) are larger than w (i even).
__device__ __forceinline__ int larger(const uint64_t* cand, int i, int end, uint64_t w) {
  int n = 0;
#pragma unroll 1
  for (; i + 7 < end; i += 8) {
    ulonglong2 o[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) o[u] = *reinterpret_cast<const ulonglong2*>(cand + i + 2 * u);
#pragma unroll
    for (int u = 0; u < 4; ++u) n += (int)(o[u].x > w) + (int)(o[u].y > w);
  }
#pragma unroll 1
  for (; i < end; ++i) n += cand[i] > w;
  return n;
}

// emit(place, word) for each of the first n of cand[0, total), the place being the
// number of larger ones: 1 << lg threads a word.
template <int NT, class F>
__device__ __forceinline__ void rank_words(const uint64_t* cand, int n, int total, F&& emit) {
  constexpr int kBits = NT == 128 ? 7 : NT == 256 ? 8 : 10;
  static_assert(NT == 1 << kBits, "");
  const int lg = max(0, min(5, kBits - 32 + __clz(n - 1))), g = 1 << lg;
  const int seg = (((total + g - 1) >> lg) + 1) & ~1, from = ((int)threadIdx.x & (g - 1)) * seg;
  for (int j0 = 0; j0 < n; j0 += NT >> lg) {
    const int j = j0 + ((int)threadIdx.x >> lg);
    if (j - (((int)threadIdx.x & 31) >> lg) >= n) break;  // the whole warp
    const uint64_t w = j < n ? cand[j] : ~0ull;
    int place = larger(cand, from, min(total, from + seg), w);
    for (int o = 1; o < g; o <<= 1) place += __shfl_xor_sync(0xffffffffu, place, o);
    if (from == 0 && j < n) emit(place, w);
  }
}

// Words cand[0, n), n <= CAP, in descending order (of more than 8 NT the first
// 4 NT): emit(place, word) for each,
// which may write to cand[place] where in_place.  Few words go to the place that
// the number of larger ones gives, more through a bitonic sort.
template <int NT, int CAP, class F>
__device__ __forceinline__ void sort_words(uint64_t* cand, int n, bool in_place, F&& emit) {
  if (n <= NT) {
    int place = 0;
    uint64_t w = 0;
    rank_words<NT>(cand, n, n, [&](int p, uint64_t o) {
      place = p + 1;
      w = o;
    });
    if (in_place) __syncthreads();
    if (place) emit(place - 1, w);
    if (in_place) __syncthreads();
    return;
  }
  if (n <= 2 * NT) {  // two words a thread
    const int j = threadIdx.x + NT;
    const uint64_t w0 = cand[threadIdx.x], w1 = j < n ? cand[j] : ~0ull;
    const int p0 = larger(cand, 0, n, w0), p1 = larger(cand, 0, n, w1);
    if (in_place) __syncthreads();
    emit(p0, w0);
    if (j < n) emit(p1, w1);
    if (in_place) __syncthreads();
    return;
  }
  if constexpr (CAP > 2 * NT) {
    sort_many<NT, CAP>(cand, n);
    if (CAP > 8 * NT && n > 8 * NT) n = 4 * NT;
    if (!in_place)
      for (int i = threadIdx.x; i < n; i += NT) emit(i, cand[i]);
  }
}

// Dynamic shared memory: cand[cap] (u64), the upper halves of the slot keys
// [kSlots][NT] and of the threads' own maxima [kOwn] (u16), and the list of slots
// above the bound [row_pairs] (u16); in clusters, all blocks' lists [blocks][k] (u64).
__host__ __device__ constexpr int row_cap(int k) { return k <= kFewK ? kFewCap : kMaxCap; }
template <int NT>
__host__ __device__ constexpr int row_smem(int k, int blocks) {
  return k == 0 ? 0
                : row_cap(k) * 8 + (kSlots * NT + kOwn) * 2 + row_pairs(NT) * 2 +
                      (blocks > 1 ? blocks * k * 8 : 0);
}

// Words of the lanes before this one, and of all.
__device__ __forceinline__ uint32_t lanes_before(uint32_t n, int& all) {
  const int lane = threadIdx.x & 31;
  uint32_t sum = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t below = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += below;
  }
  all = (int)__shfl_sync(0xffffffffu, sum, 31);
  return sum - n;
}
// Places for them behind *count: one scan and one atomic a warp.
__device__ __forceinline__ uint32_t warp_places(uint32_t n, uint32_t* count) {
  int all;
  const uint32_t before = lanes_before(n, all);
  uint32_t at = 0;
  if ((threadIdx.x & 31) == 0 && all) at = atomicAdd(count, (uint32_t)all);
  return __shfl_sync(0xffffffffu, at, 0) + before;
}

// Own maxima of threads that have something.
__device__ __forceinline__ int own_keys(int chunks) { return min(kOwn, chunks); }

// The ids of the slice whose order keys reach bound << 16, into cand; their number
// (above cap: not all of them, and none is left out otherwise).  A slot is 1 << lg
// of a thread's vectors, its key an order key where of_slots, else the upper half
// of its largest logit; best: this thread's key.  Behind a barrier.
template <class T, int NT>
__device__ __forceinline__ int collect(const Slice<T>& sl, uint32_t bound, uint32_t best, bool of_slots,
                                       int cap, int slots, int lg, SelectShared& sh, uint64_t* cand) {
  constexpr int N = Vec<T>::N;
  static_assert(kSlots <= 32 && kUnroll * N <= 32, "a bit each");
  const int tid = threadIdx.x;
  const uint16_t* slot_key = reinterpret_cast<const uint16_t*>(cand + cap);
  uint16_t* list = reinterpret_cast<uint16_t*>(cand + cap) + kSlots * NT + kOwn;
  // not below the lowest value of that key; where the key is a NaN's or no
  // value's, every logit is let through
  const float low = key_value(bound << 16);
  // the slots above the bound, of the threads above it
  uint32_t bits = 0;
  if (of_slots) {
#pragma unroll 8
    for (int i = 0; i < slots; ++i) bits |= (uint32_t)(slot_key[i * NT + tid] >= bound) << i;
  } else if (best >= bound) {
#pragma unroll 8
    for (int i = 0; i < slots; ++i)
      bits |= (uint32_t)!(__uint_as_float((uint32_t)slot_key[i * NT + tid] << 16) < low) << i;
  }
  // listed and read again by their own warp
  constexpr int kWarpPairs = row_pairs(NT) / (NT / 32);
  uint16_t* mine = list + (tid >> 5) * kWarpPairs;
  int pairs;
  uint32_t p = lanes_before(__popc(bits), pairs);
  for (; bits; bits &= bits - 1, ++p)
    if (p < (uint32_t)kWarpPairs) mine[p] = (uint16_t)((__ffs(bits) - 1) * NT + tid);
  __syncwarp();
  if (pairs > kWarpPairs) {
    if ((tid & 31) == 0) atomicAdd(&sh.count, (uint32_t)cap + 1);  // the exact selection
    pairs = 0;
  }
  if (tid < sl.loose) {
    const int64_t id = sl.loose_at(tid);
    const float z = to_f(sl.z[id]);
    if (!(z < low)) {
      const uint32_t at = atomicAdd(&sh.count, 1u);
      if (at < (uint32_t)cap) cand[at] = cand_word(order_key(z), (uint32_t)id);
    }
  }
  const int items = pairs << lg;
  for (int i0 = tid & 31; (i0 & ~31) < items; i0 += kUnroll * 32) {
    Words w[kUnroll];
    int at[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * 32;
      at[u] = INT32_MAX;
      if (i < items) {
        const int pair = mine[i >> lg];
        const int q = (pair / NT << lg) + (i & ((1 << lg) - 1));
        at[u] = ((q / kUnroll) * NT + pair % NT) * kUnroll + q % kUnroll;
      }
      if (at[u] < sl.nvec) w[u] = sl.vec(at[u]);
    }
    uint32_t hits = 0;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (at[u] >= sl.nvec) continue;
      float z[N];
      Vec<T>::get(w[u], z);
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (!(z[e] < low)) hits |= 1u << (u * N + e);
    }
    uint32_t c = warp_places(__popc(hits), &sh.count);
    for (; hits; hits &= hits - 1, ++c) {
      if (c >= (uint32_t)cap) break;
      const int bit = __ffs(hits) - 1, u = bit / N;
      const int v = u < 2 ? (u == 0 ? at[0] : at[1]) : (u == 2 ? at[2] : at[3]);
      const int64_t id = sl.base + (int64_t)v * N + bit % N;
      cand[c] = cand_word(order_key(to_f(sl.z[id])), (uint32_t)id);
    }
  }
  __syncthreads();
  return (int)sh.count;
}

// The slice's best `want` ids, or some more, in order to emit (see sort_words).
// One warp does `side` while another finds the bound.  own: this
// thread's maxima, of its even and odd steps if two.
template <class T, int NT, class Side, class Emit>
__device__ __forceinline__ int select_top(const Slice<T>& sl, int want, int cap, int slots, int lg,
                           const float (&own)[kOwn / NT], SelectShared& sh, uint64_t* cand,
                           bool in_place, Side&& side, Emit&& emit) {
  const int tid = threadIdx.x;
  uint16_t* slot_key = reinterpret_cast<uint16_t*>(cand + cap);
  uint16_t* own_key = slot_key + kSlots * NT;
  uint32_t bound;  // upper half of an order key
  // few alternatives: the threads' own maxima bound them closely enough (k of
  // n leave about -n log(1 - k/n) ids above the bound); more: those of their even
  // and odd steps, or the slots
  const bool few = want <= min(NT, sl.chunks) / 2, of_slots = !few && want > own_keys(sl.chunks) / 2;
  uint32_t best = 0;
#pragma unroll
  for (int i = 0; i < kOwn / NT; ++i) {
    const uint32_t q = order_key(own[i]) >> 16;
    best = max(best, q);
    own_key[i * NT + tid] = (uint16_t)q;
  }
  if (few) own_key[tid] = (uint16_t)best;
  if (of_slots) {
    // (a lowest denormal's upper half reads as that of -0, which is kept as +0)
    for (int i = 0; i < slots; ++i) {
      const uint32_t q = slot_key[i * NT + tid];
      slot_key[i * NT + tid] =
          q == 0x8000u ? 0x7fffu : (uint16_t)(order_key(__uint_as_float(q << 16)) >> 16);
    }
  }
  __syncthreads();
  if ((tid >> 5) == 1) side();
  if (of_slots) {
    bound = bound_key_slots<NT>(slot_key, slots, want, sh);
  } else {
    if (tid < 32) {
      if (few) bound_key<NT / 32>(own_key, want, &sh.bound);
      else bound_key<kOwn / 32>(own_key, want, &sh.bound);
    }
    __syncthreads();
    bound = sh.bound;
  }
  int have = collect<T, NT>(sl, bound, best, of_slots, cap, slots, lg, sh, cand);
  if (have > cap) {
    __syncthreads();
    select_exact(sl, want, sh, cand);
    have = want;
  }
  // (128 threads: at most kFewK alternatives)
  sort_words<NT, NT == 128 ? kFewCap : kMaxCap>(cand, have, in_place, emit);
  return have;
}

// CL: a cluster of blocks a row, else one.
template <class T, int NT, bool TOPK, bool CL>
__global__ void __launch_bounds__(NT, 1024 / NT) k_logprob_rows(LpArgs a) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ SelectShared sh;
  __shared__ LpState warp_state[NT / 32];
  __shared__ LpState block_state;
  __shared__ LpRow block_row;
  __shared__ int block_count, counts[8];
  cg::cluster_group cluster = cg::this_cluster();
  const int blocks = CL ? (int)cluster.num_blocks() : 1, rank = CL ? (int)cluster.block_rank() : 0;
  const int tid = threadIdx.x;
  const int cap = row_cap(a.topk);
  uint64_t* cand = reinterpret_cast<uint64_t*>(dyn);
  uint16_t* slot_key = reinterpret_cast<uint16_t*>(cand + cap);
  Words even[kUnroll], odd[kUnroll];
  const int lb = __ffs(blocks) - 1;
  const int64_t r = blockIdx.x >> lb;
  const Slice<T> sl(static_cast<const T*>(a.z) + r * a.ld, a.vocab, rank, lb, NT);
  sl.chunk(0, tid, NT, even);
  const int64_t label = a.tokens ? a.tokens[r] : -1;
  if (a.tokens && label == a.ignore) {  // the whole cluster
    if (rank == 0) lp_store_ignored(a, r);
    return;
  }
  const bool in = label >= 0 && label < a.vocab;
  constexpr int kTeller = TOPK ? 32 : 0;  // the thread that writes the row's own values
  const float zy = (tid == kTeller && rank == 0 && in) ? to_f(sl.z[label]) : 0.f;

  // ---- one sweep
  int lg = 2;  // a slot: 2^lg vectors
  static_assert(kUnroll == 4, "a slot is a power of two of steps, or a vector");
  // where the slots bound the alternatives a slot of a short row is one vector
  if (a.topk > own_keys(sl.chunks) / 2 && sl.rounds <= kSlots) lg = 0;
  else while (((sl.rounds - 1) >> lg) >= kSlots) ++lg;
  const int slots = ((sl.rounds - 1) >> lg) + 1;
  uint16_t* slot = slot_key + tid;
  float own[kOwn / NT], slot_top = neg_inf();
#pragma unroll
  for (int i = 0; i < kOwn / NT; ++i) own[i] = neg_inf();
  auto close_slot = [&](float top) {
    *slot = (uint16_t)(__float_as_uint(top + 0.f) >> 16);
    slot += NT;
  };
  LpFold f;
  f.init(a.k2);
  if (tid < sl.loose) f.add_one(to_f(sl.z[sl.loose_at(tid)]));
  auto step = [&](int j, const Words* w, float& best) {
    float m[kUnroll], mm = neg_inf();
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      m[u] = Vec<T>::top(w[u]);
      mm = max_nan(mm, m[u]);
    }
    if (mm != neg_inf()) {
      f.expect(mm);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        float z[Vec<T>::N];
        Vec<T>::get(w[u], z);
#pragma unroll
        for (int e = 0; e < Vec<T>::N; e += 2) f.add_pair(z[e], z[e + 1]);
      }
    }
    if (TOPK) {
      best = max_nan(best, mm);
      if (lg == 0) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) close_slot(m[u]);
      } else {
        slot_top = max_nan(slot_top, mm);
        if ((((j + 1) * kUnroll) & ((1 << lg) - 1)) == 0) {
          close_slot(slot_top);
          slot_top = neg_inf();
        }
      }
    }
  };
  const int steps = sl.rounds / kUnroll;
  // Long rows: one thread asks L2 for the two steps to come, whose loads then find
  // them half on their way (8192 x 65536 with 20 alternatives 177 us, without it
  // 201 us; 4096 x 151936 220 and 225 us with 100).  Further ahead it only costs
  // (4 steps 227 us, 10 steps 255 us), as it does in rows of a few steps.
  for (int j = 0; j < steps; j += 2) {
    if (tid == 0) sl.prefetch(j + 2, NT);
    sl.chunk(j + 1, tid, NT, odd);
    step(j, even, own[0]);
    if (j + 1 >= steps) break;
    sl.chunk(j + 2, tid, NT, even);
    step(j + 1, odd, own[kOwn / NT - 1]);
  }
  if (TOPK && (sl.rounds & ((1 << lg) - 1))) close_slot(slot_top);

  // ---- the row's statistics
  LpState st = f.state();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) lp_merge(st, lp_shfl_xor(st, o), a.k2);
  if ((tid & 31) == 0) warp_state[tid >> 5] = st;
  if (TOPK && tid == 0) sh.count = 0;
  auto block_sums = [&]() {
    st = warp_state[tid & (NT / 32 - 1)];
#pragma unroll
    for (int o = NT / 64; o > 0; o >>= 1) lp_merge(st, lp_shfl_xor(st, o), a.k2);
  };
  auto join_states = [&]() {  // one a lane, of up to eight blocks
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) lp_merge(st, lp_shfl_xor(st, o), a.k2);
    st.m = __shfl_sync(0xffffffffu, st.m, 0);
    st.s = __shfl_sync(0xffffffffu, st.s, 0);
    st.t = __shfl_sync(0xffffffffu, st.t, 0);
  };
  auto finish = [&]() {
    const LpRow row = lp_finish(st);
    if (tid == kTeller) {
      if (a.tokens && !in) set_status(a.status, KD_DEV_BAD_LABEL);
      lp_store(a, r, row, label, zy);
    }
    return row;
  };
  auto store_top = [&](int p, uint64_t w, const LpRow& row) {
    if (a.topk_idx) a.topk_idx[r * a.topk + p] = (int32_t)~(uint32_t)w;
    if (a.topk_lp) a.topk_lp[r * a.topk + p] = lp_of(key_value((uint32_t)(w >> 32)), row, a.inv_t);
  };

  // ---- the slice's best
  int have = 0;
  if (!TOPK) {
    __syncthreads();
    block_sums();
    if (!CL) finish();
  } else {  // (with a barrier at its head)
    have = (int)min((int64_t)a.topk, sl.size());
    auto side = [&]() {
      block_sums();
      if (!CL) {
        const LpRow row = finish();
        if (tid == kTeller) block_row = row;
      } else if (tid == kTeller) {
        block_state = st;
      }
    };
    // few enough alternatives: each block fetches what the others collect and finds
    // the places of its own; under the bound of the whole row, from all blocks'
    // maxima, a block collects its share of little more than K ids
    if constexpr (CL) if (a.topk <= blocks * NT / 2) {
      static_assert(NT == kOwn, "a maximum a thread");
      uint16_t* own_key = slot_key + kSlots * NT;
      const uint32_t best = order_key(own[0]) >> 16;
      own_key[tid] = (uint16_t)best;
      __syncthreads();
      uint32_t bound;
      if (blocks * a.topk * 9 / 8 <= NT) {  // so few that each block's own bound will do
        if (tid < 32) bound_key<NT / 32>(own_key, a.topk, &sh.bound);
        if ((tid >> 5) == 1) side();
        __syncthreads();
        bound = sh.bound;
      } else {
        cluster_arrive();
        if ((tid >> 5) == 1) side();
        __syncwarp();
        cluster_wait();
        if (tid < blocks * (NT / 8))
          reinterpret_cast<uint4*>(cand)[tid] = reinterpret_cast<const uint4*>(
              cluster.map_shared_rank(own_key, tid / (NT / 8)))[tid % (NT / 8)];
        __syncthreads();
        bound = bound_key_slots<NT>(reinterpret_cast<const uint16_t*>(cand), blocks, a.topk, sh);
      }
      const int n = collect<T, NT>(sl, bound, best, false, cap, slots, lg, sh, cand);
      if (tid == 0) block_count = n;
      cluster.sync();
      const int b = tid & 31;
      const int c = b < blocks ? *cluster.map_shared_rank(&block_count, b) : 0;
      int others;
      const int first = (int)lanes_before(b == rank ? 0u : (uint32_t)c, others);
      const int total = n + others;
      if ((int)__reduce_max_sync(0xffffffffu, (uint32_t)c) <= cap && total <= cap) {
        // the others' words behind this block's
        for (int i0 = tid & ~31; i0 < others; i0 += NT) {
          const int i = i0 + b;
          int q = 0, at = 0;  // block q's word `at`
          for (int o = 0; o < blocks; ++o) {
            const int f = __shfl_sync(0xffffffffu, first, o);
            if (i >= f && o != rank) {
              q = o;
              at = i - f;
            }
          }
          if (i < others) cand[n + i] = cluster.map_shared_rank(cand, q)[at];
        }
        st = b < blocks ? *cluster.map_shared_rank(&block_state, b) : LpState{neg_inf(), 0.f, 0.f};
        __syncwarp();
        cluster_arrive();  // this block has read the others
        join_states();
        const LpRow row = rank == 0 ? finish() : lp_finish(st);
        __syncthreads();
        rank_words<NT>(cand, n, total, [&](int p, uint64_t w) {
          if (p < a.topk) store_top(p, w, row);
        });
        __syncwarp();
        cluster_wait();  // no block leaves while another reads its ids
        return;
      }
      // long runs of equal logits: block by block
      cluster.sync();
      if (tid == 0) sh.count = 0;
    }
    auto emit = [&](int p, uint64_t w) {
      if (CL) cand[p] = w;
      else if (p < have) store_top(p, w, block_row);
    };
    select_top<T, NT>(sl, have, cap, slots, lg, own, sh, cand, CL, side, emit);
  }
  if constexpr (CL) {
    // ---- join the slices: every block fetches all sums and lists
    uint64_t* all = reinterpret_cast<uint64_t*>(slot_key + kSlots * NT + kOwn + row_pairs(NT));
    if (tid == 0) {
      if (!TOPK) block_state = st;
      block_count = have;
    }
    cluster.sync();
    const int b = tid & 31;
    st = b < blocks ? *cluster.map_shared_rank(&block_state, b) : LpState{neg_inf(), 0.f, 0.f};
    if (tid < blocks) counts[tid] = *cluster.map_shared_rank(&block_count, tid);
    if (TOPK)
      for (int i = tid; i < blocks * a.topk; i += NT)
        all[i] = cluster.map_shared_rank(cand, i / a.topk)[i % a.topk];
    __syncwarp();
    cluster_arrive();  // this block has read the others
    join_states();
    const LpRow row = rank == 0 ? finish() : lp_finish(st);
    if (TOPK) {
      int* place = reinterpret_cast<int*>(slot_key);  // of each word (the keys are done with)
      // larger words here, and in the other slices' sorted lists: one thread
      // for each word and slice
      for (int j = tid; j < have; j += NT) place[j] = j;
      __syncthreads();
      for (int i = tid; i < have * blocks; i += NT) {
        const int j = i >> lb, b = i & (blocks - 1);
        if (b == rank) continue;
        const uint64_t w = cand[j];
        const uint64_t* other = all + b * a.topk;
        int lo = 0, hi = counts[b];
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (other[mid] > w) lo = mid + 1;
          else hi = mid;
        }
        if (lo) atomicAdd(&place[j], lo);
      }
      __syncthreads();
      for (int j = tid; j < have; j += NT)
        if (place[j] < a.topk) store_top(place[j], cand[j], row);
    }
    __syncwarp();
    cluster_wait();  // no block leaves while another reads its lists
  }
}

// ------------------------------------------------------------------ joining parts
// Hidden sources: the records of the tensor-core epilogue, one per part (half a
// tile of a vocabulary split) and row.
constexpr int kMaxSplits = 128;

struct LpJoin {
  LpArgs a;
  const float4* sums;      // [parts][n]
  const uint64_t* cand;    // [parts][n][kTokCap]
  const int32_t* count;    // [parts][n]
  int parts;
};

// One warp: the joined sums of row r and the logit of its token.
__device__ __forceinline__ LpState join_sums(const LpJoin& j, int64_t r, float& zy) {
  constexpr int P = 2 * kMaxSplits / 32;
  float4 q[P];
#pragma unroll
  for (int u = 0; u < P; ++u) {
    const int p = 32 * u + ((int)threadIdx.x & 31);
    q[u] = p < j.parts ? j.sums[(int64_t)p * j.a.n + r] : make_float4(neg_inf(), 0.f, 0.f, 0.f);
  }
  LpState st{neg_inf(), 0.f, 0.f};
#pragma unroll
  for (int u = 0; u < P; ++u) st.m = fmaxf(st.m, q[u].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) st.m = fmaxf(st.m, __shfl_xor_sync(0xffffffffu, st.m, o));
  zy = 0.f;
#pragma unroll
  for (int u = 0; u < P; ++u) {
    LpState a{q[u].x, q[u].y, q[u].z};
    lp_raise(a, st.m, j.a.k2);
    st.s += a.s;
    st.t += a.t;
    zy += q[u].w;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    st.s += __shfl_xor_sync(0xffffffffu, st.s, o);
    st.t += __shfl_xor_sync(0xffffffffu, st.t, o);
    zy += __shfl_xor_sync(0xffffffffu, zy, o);
  }
  return st;
}

__device__ __forceinline__ void join_store(const LpJoin& j, int64_t r, int64_t y,
                                           const LpRow& row, float zy) {
  if (j.a.tokens && !(y >= 0 && y < j.a.vocab)) set_status(j.a.status, KD_DEV_BAD_LABEL);
  lp_store(j.a, r, row, y, zy);
}

// Without alternatives: a warp per row.
__global__ void __launch_bounds__(256) k_logprob_join(LpJoin j) {
  const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (r >= j.a.n) return;
  const int64_t y = j.a.tokens ? j.a.tokens[r] : -1;
  const bool off = j.a.tokens && y == j.a.ignore;
  float zy = 0.f;
  LpState st{neg_inf(), 0.f, 0.f};
  if (!off) st = join_sums(j, r, zy);  // (the parts of an ignored row are not written)
  if (threadIdx.x & 31) return;
  if (off) {
    LpArgs a = j.a;
    if (a.logprob) a.logprob[r] = 0.f;
    if (a.entropy) a.entropy[r] = 0.f;
    if (a.stats) reinterpret_cast<float4*>(a.stats)[r] = make_float4(0.f, 0.f, 0.f, 0.f);
  } else {
    join_store(j, r, y, lp_finish(st), zy);
  }
}

// With alternatives: a block per row, the parts' lists dealt to its warps.  The
// K-th largest of kOwn best candidates bounds the K-th best from below; what lies
// above it is sorted.  Bound by the latency of its few dependent loads: with cold
// caches 11 us for one row (25 us where every thread searched all parts for its
// word's), 29 us for 2048 rows with 20 alternatives, 52 us with 100 (64 us with 4
// words held by a thread, 55 us with 12).
template <int NT>
__global__ void __launch_bounds__(NT) k_logprob_join_top(LpJoin j) {
  constexpr int W = NT / 32, kGroup = NT / kOwn, kHeld = 8;
  static_assert(2 * kMaxSplits <= 32 * W, "a lane for each part of a warp");
  __shared__ __align__(16) uint64_t cand[kMaxCap / 2];
  __shared__ uint16_t own_key[kOwn];
  __shared__ SelectShared sh;
  __shared__ LpRow row;
  __shared__ uint64_t last;
  const LpArgs& a = j.a;
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, k = a.topk, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t y = a.tokens ? a.tokens[r] : -1;
  if (a.tokens && y == a.ignore) {
    lp_store_ignored(a, r);
    return;
  }
  if (tid == 0) sh.count = 0;
  // lane i: the candidates of this warp's part i, part warp + W i of the row
  // (a part that a timed-out wait ended has written nothing)
  const int parts = (j.parts - warp + W - 1) / W;
  const int mine =
      lane < parts ? max(0, min(j.count[(int64_t)(warp + W * lane) * a.n + r], kTokCap)) : 0;
  int total;
  const int first = (int)lanes_before((uint32_t)mine, total);
  // word i of the warp's lists, one behind the other
  auto word = [&](int i) -> uint64_t {
    int part = 0, at = i;
    for (int o = 1; o < parts; ++o) {
      const int f = __shfl_sync(0xffffffffu, first, o);
      if (i >= f) {
        part = o;
        at = i - f;
      }
    }
    if (i >= total) return 0;
    const uint64_t w = j.cand[((int64_t)(warp + W * part) * a.n + r) * kTokCap + at];
    return cand_word(order_key(__uint_as_float((uint32_t)(w >> 32))), ~(uint32_t)w);
  };
  uint64_t held[kHeld];  // those behind are read again
#pragma unroll
  for (int u = 0; u < kHeld; ++u) held[u] = 32 * u < total ? word(32 * u + lane) : 0;
  auto each = [&](auto&& f) {
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
      if (held[u]) f(held[u]);
#pragma unroll 1
    for (int i = 32 * kHeld; i < total; i += 4 * 32) {
      uint64_t w[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) w[u] = word(i + 32 * u + lane);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (w[u]) f(w[u]);
    }
  };
  if (warp == W - 1) {
    float zy;
    const LpRow q = lp_finish(join_sums(j, r, zy));
    if (lane == 0) {
      row = q;
      join_store(j, r, y, q, zy);
    }
  }
  uint64_t best = 0;
  each([&](uint64_t w) { best = max(best, w); });
#pragma unroll
  for (int o = 1; o < kGroup; o <<= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (tid % kGroup == 0) own_key[tid / kGroup] = (uint16_t)(best >> 48);
  __syncthreads();
  if (tid < 32) bound_key<kOwn / 32>(own_key, k, &sh.bound);
  __syncthreads();
  const uint32_t bound = sh.bound;
  each([&](uint64_t w) {
    if ((uint32_t)(w >> 48) < bound) return;
    const uint32_t at = atomicAdd(&sh.count, 1u);
    if (at < kMaxCap / 2) cand[at] = w;
  });
  __syncthreads();
  auto store = [&](int i, uint64_t w) {
    if (i >= k) return;
    if (a.topk_idx) a.topk_idx[r * k + i] = (int32_t)~(uint32_t)w;
    if (a.topk_lp) a.topk_lp[r * k + i] = lp_of(key_value((uint32_t)(w >> 32)), row, a.inv_t);
  };
  const int have = (int)sh.count;
  if (have <= kMaxCap / 2) {
    sort_words<NT, kMaxCap / 2>(cand, have, false, store);
  } else {
    // many equal logits: one after the other
    if (tid == 0) last = 0;
    for (int i = 0; i < k; ++i) {
      __syncthreads();
      const uint64_t l = last;
      uint64_t w = 0;
      each([&](uint64_t q) {
        if (i == 0 || q < l) w = max(w, q);
      });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) w = max(w, __shfl_xor_sync(0xffffffffu, w, o));
      __shared__ uint64_t warp_best[W];
      if ((tid & 31) == 0) warp_best[tid >> 5] = w;
      __syncthreads();
      if (tid == 0) {
        for (int q = 1; q < W; ++q) w = max(w, warp_best[q]);
        cand[i] = last = w;
      }
    }
    __syncthreads();
    for (int i = tid; i < k; i += NT) store(i, cand[i]);
  }
}

// ------------------------------------------------------------------ launches
// Right behind the kernel that writes the parts: on the device when that ends.
int launch_join(void (*kern)(LpJoin), int64_t grid, int threads, const LpJoin& j, cudaStream_t s) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  note_launch();
  return (int)cudaLaunchKernelEx(&cfg, kern, j);
}

// Blocks of a cluster for each row: enough of them to give every SM work, as
// long as a slice keeps 16 KiB and no SM gets more than four blocks (with up to
// twice as many blocks 80 rows of 151936 bf16 with 20 alternatives took 24 us for
// 18 us, 333 fp32 rows of 32003 25 us for 16 us).
int row_blocks(int64_t n, int64_t row_bytes, int nsm) {
  int c = 1;
  while (c < 8 && n * c * 2 <= 4 * nsm && row_bytes / (2 * c) >= 16384) c *= 2;
  return c;
}

template <class T, int NT, bool TOPK, bool CL = false>
int launch_rows_nt(const LpArgs& a, int blocks, cudaStream_t s) {
  auto kern = k_logprob_rows<T, NT, TOPK, CL>;
  const int smem = row_smem<NT>(a.topk, blocks);
  if (smem > 40000 && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           smem) != cudaSuccess)
    return 1;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)blocks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(a.n * blocks));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = blocks > 1 ? 1 : 0;
  note_launch();
  return (int)cudaLaunchKernelEx(&cfg, kern, a);
}

template <class T>
int launch_rows(const LpArgs& a, int nsm, cudaStream_t s) {
  if (a.n <= 0) return 0;
  const int64_t bytes = a.vocab * (int64_t)sizeof(T);
  const int blocks = row_blocks(a.n, bytes, nsm);
  // short rows: more, smaller blocks on an SM (128 and 256 threads: 16384 x 32000
  // bf16 157 us and 181 us, with 20 alternatives 229 us and 305 us, with 100 350 us
  // and 386 us; 8192 x 65536 with 20 204 us and 225 us, 6000 x 98000 237 us and
  // 231 us, 4096 x 151936 245 us and 226 us)
  if (blocks == 1 && a.topk <= kFewK && bytes < 163840)
    return a.topk ? launch_rows_nt<T, 128, true>(a, 1, s) : launch_rows_nt<T, 128, false>(a, 1, s);
  if (blocks == 1)
    return a.topk ? launch_rows_nt<T, 256, true>(a, 1, s) : launch_rows_nt<T, 256, false>(a, 1, s);
  return a.topk ? launch_rows_nt<T, 256, true, true>(a, blocks, s)
                : launch_rows_nt<T, 256, false, true>(a, blocks, s);
}

// ------------------------------------------------------------------ backward
constexpr int kRowThreads = 256;

// dz of an fp32 logit chunk in its place (fp32 hidden sources), a block per row.
__global__ void __launch_bounds__(kRowThreads) k_logprob_grad_chunk(LpGradArgs a) {
  const int64_t r = blockIdx.x;
  float* z = static_cast<float*>(a.g) + r * a.ldg;
  const LpGradRow g = lp_grad_row(a, r);
  for (int64_t i = threadIdx.x; i < a.cols; i += kRowThreads) {
    float v = 0.f;
    if (g.live) {
      v = lp_grad(z[i], g, a.k2);
      if (a.col0 + i == g.y) v += g.cy;
    }
    z[i] = v;
  }
}

// dz of materialised logits: a block takes kSegVecs vectors of a row, each
// thread four 16-byte loads at a time, and stores what it loaded in place (so
// d_logits may be the logits).  Bound by HBM: one read and one write of every
// element, 8192 x 128256 bf16 in 575 us (7.3 TB/s).  Rows whose two sides differ
// in their offset from a 16-byte boundary go element by element.
constexpr int kSegVecs = 2048;

template <class T>
__device__ __forceinline__ void store_vec(T* p, const float* v);
template <>
__device__ __forceinline__ void store_vec(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                            pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

template <class T>
__global__ void __launch_bounds__(kRowThreads) k_logprob_grad(LpGradArgs a, int segs) {
  constexpr int N = Vec<T>::N;
  const int64_t r = blockIdx.x / segs;
  const int seg = (int)(blockIdx.x % segs), tid = threadIdx.x;
  const T* z = static_cast<const T*>(a.z) + r * a.ld;
  T* out = static_cast<T*>(a.g) + r * a.ldg;
  const LpGradRow g = lp_grad_row(a, r);
  auto one = [&](int64_t i) {
    float v = 0.f;
    if (g.live) {
      v = lp_grad(to_f(z[i]), g, a.k2);
      if (i == g.y) v += g.cy;
    }
    from_f(v, out[i]);
  };
  const int zo = (int)(reinterpret_cast<uintptr_t>(z) & 15);
  if (zo != (int)(reinterpret_cast<uintptr_t>(out) & 15)) {
    const int64_t e0 = (int64_t)seg * kSegVecs * N, e1 = min(a.cols, e0 + (int64_t)kSegVecs * N);
    for (int64_t i = e0 + tid; i < e1; i += kRowThreads) one(i);
    return;
  }
  const int64_t head = min(a.cols, (int64_t)(zo ? N - zo / (int)sizeof(T) : 0));
  const int64_t all = (a.cols - head) / N, tail0 = head + all * N;
  if (seg == 0) {
    const int loose = (int)(head + a.cols - tail0);
    if (tid < loose) one(tid < head ? tid : tail0 + (tid - head));
  }
  const int64_t v0 = (int64_t)seg * kSegVecs;
  const int n = (int)min((int64_t)kSegVecs, all - v0);  // may be < 0: no vector here
  z += head + v0 * N;
  out += head + v0 * N;
  const int64_t y = g.y < 0 ? -1 : g.y - (head + v0 * N);
  for (int i0 = tid; i0 < n; i0 += kUnroll * kRowThreads) {
    uint4 w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kRowThreads;
      if (g.live && i < n) w[u] = *reinterpret_cast<const uint4*>(z + (int64_t)i * N);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kRowThreads;
      if (i >= n) break;
      float v[N];
      if (g.live) {
        Words q;
        q.w[0] = w[u].x, q.w[1] = w[u].y, q.w[2] = w[u].z, q.w[3] = w[u].w;
        Vec<T>::get(q, v);
#pragma unroll
        for (int e = 0; e < N; e += 2) lp_grad_pair(v[e], v[e + 1], g, a.k2);
        if ((uint64_t)(y - (int64_t)i * N) < (uint64_t)N) {
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (y - (int64_t)i * N == e) v[e] += g.cy;
        }
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = 0.f;
      }
      store_vec<T>(out + (int64_t)i * N, v);
    }
  }
}

void launch_grad_chunk(const LpGradArgs& a, cudaStream_t s) {
  note_launch();
  k_logprob_grad_chunk<<<(unsigned)a.n, kRowThreads, 0, s>>>(a);
}
template <class T>
void launch_grad(const LpGradArgs& a, cudaStream_t s) {
  const int64_t per = (int64_t)kSegVecs * Vec<T>::N;
  const int64_t segs = (a.cols + per - 1) / per;
  // rows in as many launches as the grid's 2^31 - 1 blocks ask for
  const int64_t most = INT32_MAX / segs;
  for (int64_t r0 = 0; r0 < a.n; r0 += most) {
    LpGradArgs b = a;
    b.n = std::min(most, a.n - r0);
    b.z = static_cast<const T*>(a.z) + r0 * a.ld;
    b.g = static_cast<T*>(a.g) + r0 * a.ldg;
    if (a.tokens) b.tokens = a.tokens + r0;
    b.stats = a.stats + r0 * KD_LOGPROB_STATS;
    if (a.d_lp) b.d_lp = a.d_lp + r0;
    if (a.d_ent) b.d_ent = a.d_ent + r0;
    note_launch();
    k_logprob_grad<T><<<(unsigned)(b.n * segs), kRowThreads, 0, s>>>(b, (int)segs);
  }
}

// Copy of the hidden states with the rows of ignored tokens zeroed: their
// gradient rows are 0, but 0 times what a padded row holds need not be.  With
// `count`, also the tokens of each column: how many, and the first kTermRows
// that are counted.
template <class V>
__global__ void __launch_bounds__(kRowThreads) k_mask_rows(const V* __restrict__ h, int64_t d,
                                                           const int64_t* tokens, int64_t ignore,
                                                           V* __restrict__ out, int64_t vocab,
                                                           int32_t* count, int32_t* list) {
  const int64_t r = blockIdx.x;
  const int64_t y = tokens ? tokens[r] : -1;
  const bool live = !(tokens && y == ignore);
  if (count && threadIdx.x == 0 && live && y >= 0 && y < vocab) {
    const int at = atomicAdd(&count[y], 1);
    if (at < kTermRows) list[y * kTermRows + at] = (int32_t)r;
  }
  for (int64_t i = threadIdx.x; i < d; i += kRowThreads) out[r * d + i] = live ? h[r * d + i] : V();
}
// Sum of the parts of a product whose K was split, in their order, and of the
// terms of its rows (of d floats).
__global__ void __launch_bounds__(kRowThreads) k_sum_parts(const float4* __restrict__ part,
                                                           int64_t vecs, int parts, int64_t d,
                                                           const TcTerms terms,
                                                           const float4* __restrict__ add,
                                                           float4* __restrict__ o32,
                                                           uint2* __restrict__ o16) {
  const int64_t i = blockIdx.x * (int64_t)kRowThreads + threadIdx.x;
  if (i >= vecs) return;
  float4 s = add ? add[i] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    const float4 v = part[p * vecs + i];
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  if (terms.src) {
    const int64_t row = 4 * i / d, col = 4 * i % d;
    const TermRow t = term_row(terms, row);
    if (t.n) {
      const uint2 x = *reinterpret_cast<const uint2*>(t.src[0] + col);
      s.x = fmaf(t.c[0], bf16lo(x.x), s.x), s.y = fmaf(t.c[0], bf16hi(x.x), s.y);
      s.z = fmaf(t.c[0], bf16lo(x.y), s.z), s.w = fmaf(t.c[0], bf16hi(x.y), s.w);
    }
  }
  if (o32) o32[i] = s;
  if (o16) o16[i] = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
}

// rows >= n behind the first n: zeros
__global__ void __launch_bounds__(kRowThreads) k_pad_rows(const uint4* __restrict__ h, int64_t n,
                                                          int64_t vecs, uint4* __restrict__ out,
                                                          uint32_t* __restrict__ ones, int64_t words) {
  const int64_t r = blockIdx.x;
  for (int64_t i = r * kRowThreads + threadIdx.x; i < words; i += (int64_t)gridDim.x * kRowThreads)
    ones[i] = ~0u;
  for (int64_t i = threadIdx.x; i < vecs; i += kRowThreads)
    out[r * vecs + i] = r < n ? h[r * vecs + i] : make_uint4(0, 0, 0, 0);
}

// ------------------------------------------------------------------ plan
constexpr size_t kAlign = 256;
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
// Arrays of elements of `size` bytes, each at a multiple of that.
template <class... P>
bool aligned_to(uintptr_t size, P... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ...) & (size - 1)) == 0;
}

struct LpPlan {
  bool hidden, bf16;
  int64_t n, v, d, ld, ldg;
  int nsm;
  float inv_t, k2;
  bool fused;               // forward: sums and alternatives in the tensor-core epilogue
  int splits;               // its vocabulary splits
  int64_t fr;               // forward: rows a launch takes
  int64_t R, C;             // backward: chunk of G
  size_t f_z, f_h, f_sums, f_count, f_pub, f_cand, f_bytes;
  int bufs;                 // chunk buffers
  int ks;                   // parts of K in dH = G W, at most
  size_t b_h, b_g, b_dh, b_dw, b_part, b_done, b_rest, b_count, b_list, b_bytes;
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

// Rows of one fused launch: bounds the candidates' workspace.
constexpr int64_t kFusedRows = 8192;
// Fewer rows than kFewRows are copied into kPadRows, zeros behind them: with
// one row every SM fetches the same few lines of H at the same time, which
// halves the rate at which W arrives (one row of D 4096 against 151936 columns:
// 320 us as it is, 199 us from 16 rows on, whatever they hold).
constexpr int64_t kFewRows = 16, kPadRows = 64;
// Published values of the parts: a line each where there are few rows, so that
// all parts' reads of one row do not meet in a few lines (one row of 151936 x 4096
// with 20 alternatives 211 us, 222 us with the values of its 256 parts side by side).
int64_t pub_pitch(int64_t n) { return std::max<int64_t>(n, 32); }

// Vocabulary splits of the fused forward: the smallest makespan, in tiles, of
// m_tiles * s items on `workers` CTAs (pairs).  An item costs more than its
// tiles: its record, and with alternatives the first tile, of which nearly every
// logit is listed, and the parts' candidates in the join.
int tok_splits(int64_t m_tiles, int64_t n_tiles, int workers, bool topk) {
  int best = 1;
  double best_cost = 1e300;
  for (int64_t s = 1; s <= std::min<int64_t>(n_tiles, kMaxSplits); ++s) {
    const int64_t rounds = cdiv(m_tiles * s, workers);
    const double cost = (double)rounds * ((double)cdiv(n_tiles, s) + (topk ? 1.0 : 0.02));
    if (cost < best_cost - 1e-9) {
      best_cost = cost;
      best = (int)s;
    }
  }
  return best;
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
  size_t off = 0;
  P.fused = P.bf16 && p->topk <= kTokTopk;
  if (P.fused) {
    const bool pair = tc_use_pairs();
    P.fr = std::min<int64_t>(n, kFusedRows);
    P.splits = tok_splits(cdiv(P.fr, tc_tile_rows(pair)), cdiv(P.v, 256),
                          pair ? std::max(1, P.nsm / 2) : P.nsm, p->topk > 0);
    if (n < kFewRows) P.f_h = take(off, (size_t)kPadRows * P.d * 2);
    const size_t recs = (size_t)2 * P.splits * P.fr;
    P.f_sums = take(off, recs * sizeof(float4));
    if (p->topk > 0) {
      P.f_count = take(off, recs * 4);
      P.f_pub = take(off, (size_t)2 * P.splits * pub_pitch(P.fr) * 4);
      P.f_cand = take(off, recs * kTokCap * 8);
    }
  } else {
    // fp32 logits of fr rows, at most 128 MiB (or one block of rows)
    P.fr = std::min(n, std::max<int64_t>(256, ((int64_t)32 << 20) / P.v / 256 * 256));
    P.f_z = take(off, (size_t)P.fr * P.v * 4);
  }
  P.f_bytes = off;
  // backward
  kd_problem q;
  memset(&q, 0, sizeof(q));
  q.n_tokens = n;
  q.vocab = P.v;
  q.d_student = P.d;
  q.student = KD_STUDENT_HIDDEN;
  const int64_t quant = P.bf16 ? 256 : 64;
  // few rows: less of G than there is of W, in one chunk
  if (round_up(n, 128) * round_up(P.v, quant) <= (int64_t)(P.bf16 && n <= 256 ? 48 : 8) << 20) {
    P.R = round_up(n, 128);
    P.C = round_up(P.v, quant);
  } else if (P.bf16) {
    choose_chunk(&q, (int64_t)64 << 20, quant, 4, P.R, P.C);
  } else {
    choose_chunk(&q, (int64_t)8 << 20, quant, 8, P.R, P.C);
  }
  off = 0;
  const size_t esz = P.bf16 ? 2 : 4;
  P.b_h = take(off, (size_t)n * P.d * esz);
  // bf16: a chunk is made while the products read the last one and the tail of
  // the one before it still runs
  const int64_t chunks = cdiv(n, P.R) * cdiv(P.v, P.C);
  P.bufs = P.bf16 ? (int)std::min<int64_t>(chunks, 3) : 1;
  P.b_g = take(off, (size_t)P.bufs * P.R * P.C * esz);  // fp32: z, then G in its place
  P.ks = 1;
  if (P.bf16) {
    P.ks = tc_gemm_k_splits(std::min(n, P.R), P.d, std::min(P.v, P.C), P.nsm);
    if (P.ks > 1) P.b_part = take(off, (size_t)P.ks * std::min(n, P.R) * P.d * 4);
    P.b_done = take(off, 4);
    P.b_rest = take(off, (size_t)n * 4);
    P.b_count = take(off, (size_t)P.v * 4);
    P.b_list = take(off, (size_t)P.v * kTermRows * 4);
  }
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
  if (!aligned_to(8, in->tokens)) return KD_ERR_INVALID_ARG;
  if (!P.hidden)
    return in->logits && aligned_to(P.bf16 ? 2 : 4, in->logits) ? KD_OK : KD_ERR_INVALID_ARG;
  if (!in->h || !in->w || (!P.bf16 && !aligned_to(4, in->h, in->w))) return KD_ERR_INVALID_ARG;
  if (P.bf16 && (!aligned16(in->h) || !aligned16(in->w))) return KD_ERR_UNSUPPORTED;
  return KD_OK;
}

bool spans_meet(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + nb && y < x + na;
}
// A gradient that shares memory with what the backward still reads or writes
// otherwise.  d_logits may be the logits element by element, or lie between
// their rows.
bool bwd_overlaps(const LpPlan& P, const kd_logprob_inputs* in, const void* d_h, const void* d_w,
                  const void* d_logits) {
  const size_t esz = P.bf16 ? 2 : 4;
  if (P.hidden) {
    const size_t nh = (size_t)P.n * P.d * esz, nw = (size_t)P.v * P.d * esz;
    return spans_meet(d_h, nh, in->h, nh) || spans_meet(d_h, nh, in->w, nw) ||
           spans_meet(d_w, nw, in->h, nh) || spans_meet(d_w, nw, in->w, nw) ||
           spans_meet(d_h, nh, d_w, nw);
  }
  const size_t row = (size_t)P.v * esz, pz = (size_t)P.ld * esz, pg = (size_t)P.ldg * esz;
  if (!spans_meet(in->logits, (size_t)(P.n - 1) * pz + row, d_logits,
                  (size_t)(P.n - 1) * pg + row))
    return false;
  if (pz != pg) return true;
  const uintptr_t z = reinterpret_cast<uintptr_t>(in->logits);
  const uintptr_t g = reinterpret_cast<uintptr_t>(d_logits);
  const size_t off = (g > z ? g - z : z - g) % pz;
  return g != z && (off < row || pz - off < row);
}

// bf16: rows are stored in 16-byte vectors
bool grad_ok(const LpPlan& P, const void* g) { return !P.bf16 || aligned16(g); }

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
  if (!aligned_to(4, logprob, entropy, topk_idx, topk_logprob, dev_status))
    return KD_ERR_INVALID_ARG;
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
    if (P.bf16 ? launch_rows<__nv_bfloat16>(a, P.nsm, s) : launch_rows<float>(a, P.nsm, s))
      return KD_ERR_CUDA;
  } else if (P.fused) {
    for (int64_t r0 = 0; r0 < P.n; r0 += P.fr) {
      rows_from(r0, std::min(P.fr, P.n - r0));
      TcTokArgs t;
      memset(&t, 0, sizeof(t));
      t.h = static_cast<const __nv_bfloat16*>(in->h) + r0 * P.d;
      t.h_rows = a.n;
      t.pub = at<float>(workspace, P.f_pub);
      t.pub_ld = pub_pitch(a.n);
      const int64_t pubs = k ? 2 * P.splits * t.pub_ld : 0;  // all ones: nothing published
      if (a.n < kFewRows && P.n < kFewRows) {
        note_launch();
        k_pad_rows<<<(unsigned)kPadRows, kRowThreads, 0, s>>>(
            static_cast<const uint4*>(t.h), a.n, P.d / 8, at<uint4>(workspace, P.f_h),
            reinterpret_cast<uint32_t*>(t.pub), pubs);
        t.h = at<char>(workspace, P.f_h);
        t.h_rows = kPadRows;
      } else if (pubs && cudaMemsetAsync(t.pub, 0xff, (size_t)pubs * 4, s) != cudaSuccess) {
        return KD_ERR_CUDA;
      }
      t.w = in->w;
      t.n = a.n;
      t.vocab = P.v;
      t.d = P.d;
      t.tokens = a.tokens;
      t.ignore = a.ignore;
      t.k2 = P.k2;
      t.topk = k;
      t.n_splits = P.splits;
      t.sums = at<float4>(workspace, P.f_sums);
      t.cand = at<uint64_t>(workspace, P.f_cand);
      t.count = at<int32_t>(workspace, P.f_count);
      t.status = dev_status;
      if (launch_tc_tok(t, P.nsm, s)) return KD_ERR_CUDA;
      const LpJoin j{a, t.sums, t.cand, t.count, 2 * P.splits};
      // (few rows, or many lists: more of a row's lists at once)
      if (!k ? launch_join(k_logprob_join, cdiv(a.n, 8), 256, j, s)
          : a.n <= P.nsm || j.parts > 64 ? launch_join(k_logprob_join_top<1024>, a.n, 1024, j, s)
                         : launch_join(k_logprob_join_top<256>, a.n, 256, j, s))
        return KD_ERR_CUDA;
    }
  } else {
    float* z = at<float>(workspace, P.f_z);
    a.z = z;
    a.ld = P.v;
    for (int64_t r0 = 0; r0 < P.n; r0 += P.fr) {
      const int64_t rows = std::min(P.fr, P.n - r0);
      if (lp_logits(P, in, r0, rows, 0, P.v, z, P.v, dev_status, s)) return KD_ERR_CUDA;
      rows_from(r0, rows);
      if (launch_rows<float>(a, P.nsm, s)) return KD_ERR_CUDA;
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
  if (!aligned_to(4, d_logprob, d_entropy, dev_status) ||
      !aligned_to(P.bf16 ? 2 : 4, d_h, d_w, d_logits))
    return KD_ERR_INVALID_ARG;
  if (P.n > 0 && (!grad_ok(P, d_h) || !grad_ok(P, d_w))) return KD_ERR_UNSUPPORTED;
  if (!ws_ok(workspace, ws_bytes, P.b_bytes)) return KD_ERR_WORKSPACE;
  if (P.n > 0 && bwd_overlaps(P, in, d_h, d_w, d_logits)) return KD_ERR_INVALID_ARG;
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
    if (P.bf16) launch_grad<__nv_bfloat16>(a, s);
    else launch_grad<float>(a, s);
    return cudaGetLastError() == cudaSuccess ? KD_OK : KD_ERR_CUDA;
  }
  if (!d_h && !d_w) return KD_OK;
  const int64_t n = P.n, v = P.v, D = P.d, R = P.R, C = P.C;
  const int64_t nr = cdiv(n, R), nc = cdiv(v, C);
  void* g = at<char>(workspace, P.b_g);
  void* hm = at<char>(workspace, P.b_h);
  // What rounding the tokens' elements of G to bf16 took from them (fp32) goes
  // into both products at their end: into d_h[i] with W's row of token i, into
  // d_w[v] with the hidden states of the tokens v where they are few (the lists
  // hold kTermRows; of an id that more tokens share G's rounding stays).  Rows
  // without a token in range keep 0.
  float* rest = P.bf16 ? at<float>(workspace, P.b_rest) : nullptr;
  int32_t* count = P.bf16 ? at<int32_t>(workspace, P.b_count) : nullptr;
  int32_t* list = P.bf16 ? at<int32_t>(workspace, P.b_list) : nullptr;
  uint32_t* done = P.bf16 ? at<uint32_t>(workspace, P.b_done) : nullptr;
  if (P.bf16) {  // (rest lies behind the chain's word, count behind rest)
    const size_t bytes = !in->tokens ? 4
                         : d_w       ? P.b_count - P.b_done + (size_t)v * 4
                                     : P.b_rest - P.b_done + (size_t)n * 4;
    if (cudaMemsetAsync(done, 0, bytes, s) != cudaSuccess) return KD_ERR_CUDA;
  }
  if (d_w) {
    note_launch();
    if (P.bf16)
      k_mask_rows<uint4><<<(unsigned)n, kRowThreads, 0, s>>>(
          static_cast<const uint4*>(in->h), D / 8, in->tokens, p->ignore_index,
          static_cast<uint4*>(hm), v, in->tokens ? count : nullptr, list);
    else
      k_mask_rows<float><<<(unsigned)n, kRowThreads, 0, s>>>(
          static_cast<const float*>(in->h), D, in->tokens, p->ignore_index,
          static_cast<float*>(hm), v, nullptr, nullptr);
  }
  if (!P.bf16) {
    for (int64_t ri = 0; ri < nr; ++ri) {
      const int64_t r0 = ri * R, rc = std::min(R, n - r0);
      for (int64_t ci = 0; ci < nc; ++ci) {
        const int64_t c0 = ci * C, cc = std::min(C, v - c0);
        float* z = static_cast<float*>(g);
        if (lp_logits(P, in, r0, rc, c0, cc, z, C, dev_status, s)) return KD_ERR_CUDA;
        a.n = rc;
        a.cols = cc;
        a.col0 = c0;
        a.ld = a.ldg = C;
        a.tokens = in->tokens ? in->tokens + r0 : nullptr;
        a.stats = stats + r0 * KD_LOGPROB_STATS;
        a.d_lp = d_logprob ? d_logprob + r0 : nullptr;
        a.d_ent = d_entropy ? d_entropy + r0 : nullptr;
        a.g = g;
        launch_grad_chunk(a, s);
        if (d_h)
          launch_simt_gemm(z, C, 1, static_cast<const float*>(in->w) + c0 * D, D, 1,
                           static_cast<float*>(d_h) + r0 * D, D, rc, D, cc, ci > 0, s);
        if (d_w)
          launch_simt_gemm(z, 1, C, static_cast<const float*>(hm) + r0 * D, D, 1,
                           static_cast<float*>(d_w) + c0 * D, D, cc, D, rc, ri > 0, s);
      }
    }
    return cudaGetLastError() == cudaSuccess ? KD_OK : KD_ERR_CUDA;
  }
  // Chunk i is made before the products of chunk i - 1 are launched, into the
  // buffer after the one they read; with the launches chained, the next one
  // fills the SMs that the partial last wave of the one before leaves idle.
  struct Chunk {
    int64_t ri, ci, r0, rc, c0, cc;
    __nv_bfloat16* g;
  };
  const int64_t chunks = nr * nc;
  auto chunk = [&](int64_t i) {
    Chunk k;
    k.ri = i / nc;
    k.ci = i % nc;
    k.r0 = k.ri * R;
    k.rc = std::min(R, n - k.r0);
    k.c0 = k.ci * C;
    k.cc = std::min(C, v - k.c0);
    k.g = static_cast<__nv_bfloat16*>(g) + (size_t)(i % P.bufs) * R * C;
    return k;
  };
  auto terms = [&](const Chunk& k, bool of_w, bool last) {
    TcTerms t;
    memset(&t, 0, sizeof(t));
    if (!in->tokens || !last) return t;
    t.ld_src = D;
    t.one_c = rest;
    if (of_w) {
      t.src = static_cast<const __nv_bfloat16*>(hm);
      t.src_rows = n;
      t.count = count + k.c0;
      t.list = list + k.c0 * kTermRows;
    } else {
      t.src = static_cast<const __nv_bfloat16*>(in->w);
      t.src_rows = v;
      t.one_q = in->tokens + k.r0;
      t.one_c = rest + k.r0;
    }
    return t;
  };
  // a chain ends where a launch needs the one right before it: between a chunk
  // and its products when nothing is made between them, and at a sum of parts
  bool first = true;
  uint32_t launches = 0;
  auto link = [&]() {
    const TcLink l{first ? TC_CHAIN_FIRST : TC_CHAIN_NEXT, ++launches, done};
    first = false;
    return l;
  };
  auto make = [&](const Chunk& k) {
    TcTokGradArgs t;
    memset(&t, 0, sizeof(t));
    t.h = in->h;
    t.w = in->w;
    t.n = n;
    t.vocab = v;
    t.d = D;
    t.r0 = k.r0;
    t.rc = k.rc;
    t.c0 = k.c0;
    t.cc = k.cc;
    t.g = k.g;
    t.ldg = C;
    t.inv_t = P.inv_t;
    t.k2 = P.k2;
    t.tokens = in->tokens;
    t.ignore = p->ignore_index;
    t.stats = stats;
    t.d_lp = d_logprob;
    t.d_ent = d_entropy;
    t.rest = rest;
    t.link = link();
    t.status = dev_status;
    return launch_tc_tok_grad(t, P.nsm, s);
  };
  // parts of K in dH = G W over a chunk's columns: a narrow last chunk may have
  // fewer blocks than whole chunks have parts, and a part needs one
  auto k_parts = [&](const Chunk& k) { return (int)std::min<int64_t>(P.ks, cdiv(k.cc, 64)); };
  // C[m, D] (+)= A B over chunk part i of `parts`
  auto product = [&](const Chunk& k, const __nv_bfloat16* b, int64_t m, int64_t kk, bool a_mn,
                     float* acc, __nv_bfloat16* out, int64_t i, int64_t parts) {
    TcGemmArgs t;
    memset(&t, 0, sizeof(t));
    t.a0 = k.g;
    t.lda0 = C;
    t.a0_mn = a_mn;
    t.b0 = b;
    t.ldb0 = D;
    t.b0_mn = 1;
    t.M = m;
    t.N = D;
    t.K0 = kk;
    t.status = dev_status;
    t.ldc32 = D;
    t.ldc16 = D;
    t.link = link();
    const bool last = i + 1 == parts;
    if (!a_mn && P.ks > 1) {  // dH over few rows: K in parts; sum_parts below
      t.k_splits = k_parts(k);
      t.mode = TC_OUT_F32;
      t.c32 = at<float>(workspace, P.b_part);
      return launch_tc_gemm(t, P.nsm, s);
    }
    t.mode = parts == 1 ? TC_OUT_BF16
             : i == 0   ? TC_OUT_F32
             : !last    ? TC_OUT_F32_ACC
                        : TC_OUT_F32_ACC_BF16;
    t.terms = terms(k, a_mn, last);
    t.c32 = acc;
    t.c16 = out;
    return launch_tc_gemm(t, P.nsm, s);
  };
  auto sum_parts = [&](const Chunk& k, float* acc, __nv_bfloat16* out) {
    const int64_t vecs = k.rc * D / 4;
    const bool last = k.ci + 1 == nc;
    note_launch();
    k_sum_parts<<<(unsigned)cdiv(vecs, kRowThreads), kRowThreads, 0, s>>>(
        at<float4>(workspace, P.b_part), vecs, k_parts(k), D, terms(k, false, last),
        k.ci > 0 ? reinterpret_cast<const float4*>(acc) : nullptr,
        last ? nullptr : reinterpret_cast<float4*>(acc),
        last ? reinterpret_cast<uint2*>(out) : nullptr);
  };
  auto products = [&](const Chunk& k) {
    float* acc = nc > 1 ? at<float>(workspace, P.b_dh) + k.r0 * D : nullptr;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(d_h) + k.r0 * D;
    if (d_h && product(k, static_cast<const __nv_bfloat16*>(in->w) + k.c0 * D, k.rc, k.cc, false,
                       acc, out, k.ci, nc))
      return 1;
    if (d_w && product(k, static_cast<const __nv_bfloat16*>(hm) + k.r0 * D, k.cc, k.rc, true,
                       nr > 1 ? at<float>(workspace, P.b_dw) + k.c0 * D : nullptr,
                       static_cast<__nv_bfloat16*>(d_w) + k.c0 * D, k.ri, nr))
      return 1;
    if (d_h && P.ks > 1) sum_parts(k, acc, out);
    return 0;
  };
  if (make(chunk(0))) return KD_ERR_CUDA;
  for (int64_t i = 1; i < chunks; ++i) {
    if (P.ks > 1) first = true;
    if (make(chunk(i)) || products(chunk(i - 1))) return KD_ERR_CUDA;
  }
  first = true;
  if (products(chunk(chunks - 1))) return KD_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? KD_OK : KD_ERR_CUDA;
}
