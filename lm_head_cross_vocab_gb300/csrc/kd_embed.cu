// Embedding lookup and its gradient.
//
//   h[n] = scale W[tokens[n]],   d_w[v] (+)= scale sum_{n : tokens[n] = v} d_h[n]
//
// The gradient is a segmented sum over the tokens sorted into groups of one id,
// in three launches:
//   k_embed_sort    a block owns every G-th id and reads all tokens: it keeps and
//                   counts its own (and counts the tokens of the blocks before it,
//                   which is where its part of the list starts: no block waits for
//                   another), then writes its tokens' places, an id's rows in their
//                   order.  Every G-th id, since text's frequent ids are neighbours.
//   k_embed_reduce  a team of threads has a run of the list and some columns,
//                   and adds up the pieces that start there.  An id with fewer than
//                   2 kPiece tokens is one piece and is written at once; more are
//                   cut into pieces of kPiece rows (the last one longer), so that
//                   a frequent token is not one team's work; their fp32 sums go
//                   to the workspace.
//   k_embed_join    adds the pieces of each such id in order.
// Each sum's order depends on the tokens alone.
// The lookup is bound by its writes (16384 x 4096 bf16 32 us, 4.2 TB/s written and each
// id's row read once), the gradient of a whole table by the table's (16384 tokens of 4096
// into 151936 rows 206 us, a fill alone 164-170 us), that of few ids by the latency of
// three launches (4096 tokens of 2048 added to 32000 rows 17 us).
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
  int parts;  // of a row, kSpan vectors (or kSingles elements) a lane each
  float scale;
  uint32_t* status;
};
constexpr int kSpan = 4, kSingles = 16;
constexpr int kLookupThreads = 256;

// A warp copies 32 * kSpan vectors of a row, or 32 * kSingles elements.
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
  const int64_t first = (int64_t)part * (32 * (VEC ? kSpan : kSingles)) + lane;
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
    T x[kSingles];
#pragma unroll
    for (int i = 0; i < kSingles; ++i) {
      if (in && first + i * 32 < a.d) x[i] = w[first + i * 32];
      else from_f(0.f, x[i]);
    }
#pragma unroll
    for (int i = 0; i < kSingles; ++i) {
      if (first + i * 32 >= a.d) break;
      if (a.scale != 1.f && in) from_f(to_f(x[i]) * a.scale, x[i]);
      h[first + i * 32] = x[i];
    }
  }
}

// Short rows of whole vectors: a warp takes 32 * kSpan vectors of as many rows as
// they reach over.
template <class T>
__global__ void __launch_bounds__(kLookupThreads) k_embed_short(LookupArgs a) {
  constexpr int N = RowVec<T>::N;
  const int lane = threadIdx.x & 31;
  const int64_t first = ((int64_t)blockIdx.x * (kLookupThreads / 32) + (threadIdx.x >> 5)) * (32 * kSpan);
  const int vecs = (int)(a.d / N);
  const int64_t row0 = first / vecs;
  const int skip = (int)(first - row0 * vecs);
  int64_t v[kSpan];
  int col[kSpan];
  bool in[kSpan];
#pragma unroll
  for (int i = 0; i < kSpan; ++i) {
    const int at = skip + lane + i * 32, down = at / vecs;
    const int64_t row = row0 + down;
    col[i] = row < a.n ? at - down * vecs : -1;
    v[i] = row < a.n ? a.tokens[row] : a.ignore;
  }
  uint4 u[kSpan];
#pragma unroll
  for (int i = 0; i < kSpan; ++i) {
    in[i] = v[i] != a.ignore && v[i] >= 0 && v[i] < a.vocab;
    if (!in[i] && v[i] != a.ignore && col[i] == 0) set_status(a.status, KD_DEV_BAD_LABEL);
    u[i] = in[i] ? reinterpret_cast<const uint4*>(static_cast<const T*>(a.w) + v[i] * a.d)[col[i]]
                 : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kSpan; ++i) {
    if (col[i] < 0) break;
    if (a.scale != 1.f && in[i]) {
      float x[N];
      RowVec<T>::get(u[i], x);
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] *= a.scale;
      u[i] = RowVec<T>::put(x);
    }
    __stcs(&reinterpret_cast<uint4*>(a.h)[first + lane + i * 32], u[i]);
  }
}

// ------------------------------------------------------------------ sort
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kAhead = 8;      // tokens a lane has in flight
constexpr int kKept = 128;     // tokens a warp keeps, each as its place in the warp's
constexpr int kPlaceBits = 21; // run below and its id's number above
constexpr int kOneWarp = 512;  // tokens of a block that one warp puts in order

// Places of one id in the list.
struct Segment {
  int32_t first, count;
};
struct Place {
  int32_t row, id;
};
// A frequent id (id -1: none) whose places begin in a run.
struct Head {
  int32_t id;
  Segment seg;
};

struct SortArgs {
  const int64_t* tokens;
  int64_t n, vocab, ignore;
  int lg, ids;        // 2^lg blocks, ids of a block
  Segment* seg;       // [vocab]
  Place* place;       // [n]
  int32_t* live;      // places in all
  uint32_t* status;
};

// Sum over the threads before this one; `total` over all.
__device__ __forceinline__ int block_scan(int v, int* warp_sum, int& total) {
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
  return before + x - v;
}

// Dynamic shared memory: [ids] counters, the warps' lists of the tokens kept, and
// one list of them all or [kSortWarps][ids] counters.
constexpr int kListBytes = kSortWarps * kKept * 4;
__host__ __device__ constexpr int sort_smem(int ids) {
  const int many = kSortWarps * ids * 4, one = kOneWarp * (int)sizeof(Place);
  return (ids + 3) / 4 * 16 + kListBytes + (many > one ? many : one);
}
// Ids of a block: as many as shared memory holds (227 KB, 1 KB of it for the kernel's
// own).  Every block reads all tokens, and at this size an SM holds one: 128 blocks
// are one wave, 256 two (200019 ids, 60000 tokens of 256 47.5 us with 128 blocks, 53.7
// with 256; 4096 of 2048 23.3 and 24.0, 16384 of 2048 43.5 and 44.0).
constexpr int kMaxIds = (226 * 1024 - kListBytes) / ((1 + kSortWarps) * 4) / 4 * 4;
static_assert(sort_smem(kMaxIds) <= 226 * 1024, "shared memory of a block");
static_assert(kMaxIds <= 1 << (32 - kPlaceBits), "a token in 32 bits");
// The reduction may start while the sort ends, unless the sort's shared memory takes an
// SM's largest setting, 228 KB: the reduction's blocks that come to such an SM meanwhile
// have 28 KB of L1 to read through (16384 tokens of 2048, 200019 ids: 43.5 us, started
// early 47.2; 151936 ids, which need 196 KB: 42.6 and, early, 42.1).
constexpr int kChainedSmem = 194 * 1024;

__global__ void __launch_bounds__(kSortThreads) k_embed_sort(SortArgs a) {
  extern __shared__ __align__(16) int counter[];
  __shared__ int warp_sum[32], kept[32], below_sum, crowded;
  chain_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t block = blockIdx.x, mask = (1u << a.lg) - 1, before = (1u << lane) - 1;
  uint32_t* list = reinterpret_cast<uint32_t*>(counter + (a.ids + 3) / 4 * 4) + warp * kKept;
  int* more = counter + (a.ids + 3) / 4 * 4 + kSortWarps * kKept;
  int* run = more + warp * a.ids;  // this warp's own counters
  for (int i = threadIdx.x; i < a.ids; i += kSortThreads) counter[i] = 0;
  if (threadIdx.x == 0) below_sum = crowded = 0;
  // this warp's run of the tokens, whole groups of 32
  const int64_t groups = (a.n + 31) / 32, each = (groups + kSortWarps - 1) / kSortWarps;
  const int64_t begin = warp * each * 32, end = min((warp + 1) * each * 32, a.n);
  // a token's id modulo the blocks, ~0 where it has none
  const uint32_t vocab = (uint32_t)a.vocab;
  const bool inside = (uint64_t)a.ignore < (uint64_t)a.vocab;
  auto owner = [&](int64_t t) {
    const uint32_t id = (uint32_t)t;
    bool in = (uint32_t)((uint64_t)t >> 32) == 0 && id < vocab;
    if (!in && t != a.ignore && block == 0) set_status(a.status, KD_DEV_BAD_LABEL);
    if (inside) in = in && t != a.ignore;
    return in ? id & mask : 0xffffffffu;
  };
  auto row_of = [&](uint32_t x) { return (int)(begin + (x & ((1u << kPlaceBits) - 1))); };
  auto id_of = [&](uint32_t x) { return (int)(x >> kPlaceBits); };
  // the lanes' tokens (k -1: none) to their places, the next of each id in `next`
  auto rank = [&](int* next, int row, int k) {
    const uint32_t same = __match_any_sync(0xffffffffu, k);
    const int p = k >= 0 ? next[k] + __popc(same & before) : 0;
    __syncwarp();
    if (k >= 0) {
      if (lane == __ffs(same) - 1) next[k] += __popc(same);
      a.place[p] = Place{row, (int32_t)(((uint32_t)k << a.lg) + block)};
    }
    __syncwarp();
  };
  __syncthreads();
  // tokens of this warp's run that the block owns, in the list, and from `full` on
  // only counted; and tokens of the blocks before it
  int mine = 0, owned = 0, below = 0;
  int64_t full = -1;
  const bool may_fill = each * 32 > kKept;
  if (may_fill)
    for (int i = lane; i < a.ids; i += 32) run[i] = 0;
  __syncwarp();
  auto take = [&](int64_t at, int64_t t) {
    const uint32_t of = owner(t);
    below += of < block;
    const uint32_t in = __ballot_sync(0xffffffffu, of == block);
    if (!in) return;
    const int k = (int)((uint32_t)t >> a.lg), more = __popc(in);
    if (full < 0 && (mine + more > kKept || at - lane - begin >= (1 << kPlaceBits) - 32))
      full = at - lane;
    if (of == block) {
      atomicAdd(&counter[k], 1);
      if (full < 0) list[mine + __popc(in & before)] = (uint32_t)k << kPlaceBits | (uint32_t)(at - begin);
      else atomicAdd(&run[k], 1);
    }
    owned += more;
    if (full < 0) mine += more;
  };
  int64_t at = begin + lane;
  for (; at - lane + 32 * kAhead <= end; at += 32 * kAhead) {
    int64_t t[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) t[u] = a.tokens[at + u * 32];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) take(at + u * 32, t[u]);
  }
  if (at - lane < end) {
    int64_t t[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) t[u] = at + u * 32 < end ? a.tokens[at + u * 32] : a.ignore;
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (at - lane + u * 32 < end) take(at + u * 32, t[u]);
  }
  below = __reduce_add_sync(0xffffffffu, below);
  if (lane == 0) {
    if (below) atomicAdd(&below_sum, below);
    kept[warp] = owned;
    if (full >= 0) crowded = 1;
  }
  __syncthreads();
  // counts to places
  int first = below_sum;
  const int total = __reduce_add_sync(0xffffffffu, kept[lane]);
  if (block == mask && threadIdx.x == 0) *a.live = below_sum + total;
  for (int i0 = 0; i0 < a.ids; i0 += kSortThreads) {
    const int id = i0 + threadIdx.x, count = id < a.ids ? counter[id] : 0;
    int sum;
    const int place = first + block_scan(count, warp_sum, sum);
    if (id < a.ids) {
      const int64_t v = ((int64_t)id << a.lg) + block;
      if (v < a.vocab) a.seg[v] = Segment{place, count};
      counter[id] = place;
    }
    first += sum;
    __syncthreads();
  }
  if (total <= kOneWarp && !crowded) {
    // one list, which a warp goes through in order
    const int c = kept[lane];
    int x = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const int to = __shfl_sync(0xffffffffu, x - c, warp);
    Place* all = reinterpret_cast<Place*>(more);
    for (int i = lane; i < mine; i += 32) all[to + i] = Place{row_of(list[i]), id_of(list[i])};
    __syncthreads();
    if (warp) return;
    for (int i0 = 0; i0 < total; i0 += 32) {
      const Place x = i0 + lane < total ? all[i0 + lane] : Place{0, -1};
      rank(counter, x.row, x.id);
    }
    return;
  }
  // many tokens: each warp counts its own apart, and places them once it knows where
  // (16384 tokens, two in five the same: 9.8 us, by one warp 27).  Those that it has
  // not kept it reads again.
  if (!may_fill)
    for (int i = lane; i < a.ids; i += 32) run[i] = 0;
  __syncwarp();
  for (int i = lane; i < mine; i += 32) atomicAdd(&run[id_of(list[i])], 1);
  __syncthreads();
  for (int id = threadIdx.x; id < a.ids; id += kSortThreads) {
    int place = counter[id];
    for (int w = 0; w < kSortWarps; ++w) {
      int& c = more[w * a.ids + id];
      const int n = c;
      c = place;
      place += n;
    }
  }
  __syncthreads();
  for (int i0 = 0; i0 < mine; i0 += 32) {
    const bool on = i0 + lane < mine;
    const uint32_t x = on ? list[i0 + lane] : 0;
    rank(run, row_of(x), on ? id_of(x) : -1);
  }
  if (full < 0) return;
  for (int64_t at = full + lane; at - lane < end; at += 32 * kAhead) {
    int64_t t[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) t[u] = at + u * 32 < end ? a.tokens[at + u * 32] : a.ignore;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const bool in = owner(t[u]) == block;
      if (__any_sync(0xffffffffu, in))
        rank(run, (int)(at + u * 32), in ? (int)((uint32_t)t[u] >> a.lg) : -1);
    }
  }
}

// ------------------------------------------------------------------ reduce
constexpr int kPiece = 16;   // rows of a piece of a frequent id
constexpr int kMinRun = 4, kMostRun = kPiece;  // a run starts one piece of a frequent id at most
constexpr int kReduceThreads = 128;
constexpr int kReduceWarps = kReduceThreads / 32;
constexpr int kRowsAhead = 8;
constexpr int kMostRows = 2 * kMostRun + 2 * kPiece;  // rows a team reads, those added to among them
constexpr int kZeroBytes = 65536;  // of d_w that a block fills with zeros, about

struct ReduceGradArgs {
  const void* dh;
  void* dw;
  const Segment* seg;
  const Place* place;
  const int32_t* live;
  Head* head;         // [runs]
  float* part;        // [runs][d] sums of frequent ids' pieces, by the run they start in
  int64_t n, vocab, d;
  int run;            // places of the list a team starts pieces in, a power of two
  int slices;         // of the columns
  int64_t teams;      // blocks that add; the others write the rows of zeros
  int zeros;          // ids of each of those, a warp's up to 32
  int accumulate;
  float scale;
};

// A thread's columns of one row: a vector, or N elements TEAM apart (held as they
// came, so that nothing waits for them before they are added).
template <class T, int TEAM, bool VEC>
struct Columns {
  static constexpr int N = RowVec<T>::N;
  static constexpr int64_t kSlice = (int64_t)TEAM * N;
  uint4 w;
  T x[N];
  __device__ __forceinline__ void load(const T* row, int64_t c0, int64_t d, int t) {
    if constexpr (VEC) {
      const int64_t c = c0 + t * N;
      w = c < d ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int64_t c = c0 + e * TEAM + t;
        if (c < d) x[e] = row[c];
        else from_f(0.f, x[e]);
      }
    }
  }
  __device__ __forceinline__ void get(float* v) const {
    if constexpr (VEC) {
      RowVec<T>::get(w, v);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = to_f(x[e]);
    }
  }
  static __device__ __forceinline__ void store(T* row, int64_t c0, int64_t d, int t,
                                               const float* v) {
    if constexpr (VEC) {
      const int64_t c = c0 + t * N;
      if (c < d) __stcs(reinterpret_cast<uint4*>(row + c), RowVec<T>::put(v));
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int64_t c = c0 + e * TEAM + t;
        if (c < d) from_f(v[e], row[c]);
      }
    }
  }
  static __device__ __forceinline__ void store_part(float* row, int64_t c0, int64_t d, int t,
                                                    const float* v) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int64_t c = VEC ? c0 + t * N + e : c0 + e * TEAM + t;
      if (c < d) row[c] = v[e];
    }
  }
};

// A block's share of the ids: zeros where an id does not occur.  A warp has a
// quarter of them, one behind the other.
template <class T, bool VEC>
__device__ __forceinline__ void zero_rows(const ReduceGradArgs& a, int64_t share) {
  const int lane = threadIdx.x & 31, each = a.zeros / kReduceWarps;
  const int64_t v0 = share * a.zeros + (threadIdx.x >> 5) * each;
  uint32_t none = __ballot_sync(0xffffffffu, lane < each && v0 + lane < a.vocab &&
                                                 a.seg[v0 + lane].count == 0);
  T* rows = static_cast<T*>(a.dw) + v0 * a.d;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int64_t row_vecs = a.d / RowVec<T>::N;
  if (VEC && row_vecs < 32) {  // all its rows' vectors in one run
    const int vecs = (int)row_vecs;
    for (int i = lane; i < each * vecs; i += 32)
      if ((none >> (i / vecs)) & 1) __stcs(&reinterpret_cast<uint4*>(rows)[i], zero);
    return;
  }
  for (; none; none &= none - 1) {
    T* row = rows + (__ffs(none) - 1) * a.d;
    const int64_t lead = min((int64_t)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) /
                                 (int64_t)sizeof(T), a.d);
    const int64_t vecs = (a.d - lead) / RowVec<T>::N, tail = lead + vecs * RowVec<T>::N;
    if (lane < lead) from_f(0.f, row[lane]);
    uint4* p = reinterpret_cast<uint4*>(row + lead);
    for (int64_t i = lane; i < vecs; i += 32) __stcs(&p[i], zero);
    if (tail + lane < a.d) from_f(0.f, row[tail + lane]);
  }
}

// A team adds up the pieces that start in its run of places, over its columns.
// The rows it reads (the pieces', and behind each the row of d_w that the sum is
// added to) are one list, so that kRowsAhead of them are always on their way,
// wherever the pieces end: most ids occur once or twice.
template <class T, int TEAM, bool VEC>
__global__ void __launch_bounds__(kReduceThreads) k_embed_reduce(ReduceGradArgs a) {
  using C = Columns<T, TEAM, VEC>;
  constexpr int N = C::N, kTeams = kReduceThreads / TEAM;
  __shared__ int src_[kTeams][kMostRows], out_[kTeams][kMostRows], rows_[kTeams];
  constexpr int kAheadHere = VEC ? kRowsAhead : kRowsAhead / 2;
  chain_wait();
  chain_next();
  if (blockIdx.x >= a.teams) {
    zero_rows<T, VEC>(a, blockIdx.x - a.teams);
    return;
  }
  const int team = threadIdx.x / TEAM, t = threadIdx.x % TEAM;
  const int64_t item = (int64_t)blockIdx.x * kTeams + team;
  const int64_t run = item / a.slices, at = run * a.run;
  const int64_t c0 = (item - run * a.slices) * C::kSlice;
  T* dw = static_cast<T*>(a.dw);
  const T* dh = static_cast<const T*>(a.dh);
  // src: a row of d_h, or ~id of a row of d_w that is added to.  out: none (-1), the
  // row of d_w that ends here, or -2: part[run]
  int *src = src_[team], *out = out_[team];
  if (t < 32) {  // two places a lane: the run's, and as far as its last piece goes
    static_assert(kMostRun - 1 + 2 * kPiece - 1 < 64, "places of the last piece");
    const Place none{0, 0};
    const Place x0 = at + t < a.n ? a.place[at + t] : none;
    const Place x1 = at + t + 32 < a.n ? a.place[at + t + 32] : none;
    const int64_t live = *a.live;
    int len = 0, ends = -1;
    Head head{-1, Segment{0, 0}};
    if (t < a.run && at + t < live) {
      const Segment s = a.seg[x0.id];
      const int off = (int)(at + t - s.first);
      if (s.count < 2 * kPiece) {
        len = off == 0 ? s.count : 0;
        ends = x0.id;
      } else {
        const int q = s.count / kPiece, j = off / kPiece;
        if (off % kPiece == 0 && j < q) len = j < q - 1 ? kPiece : s.count - j * kPiece;
        ends = -2;
        if (off == 0) head = Head{x0.id, s};
      }
    }
    const uint32_t heads = __ballot_sync(0xffffffffu, head.id >= 0);
    if (t == (heads ? __ffs(heads) - 1 : 0) && c0 == 0 && at < a.n) a.head[run] = head;
    // the pieces lie one behind the other: a place's row is its distance from the
    // first one's start, and the rows added to that come before it
    const uint32_t starts = __ballot_sync(0xffffffffu, len > 0);
    const uint32_t added = __ballot_sync(0xffffffffu, len > 0 && ends >= 0 && a.accumulate);
    const int begin = __ffs(starts) - 1;
    auto list = [&](int i, int row) {
      const uint32_t upto = i < 31 ? (2u << i) - 1 : 0xffffffffu;
      const int from = max(31 - __clz(starts & upto), 0);  // its piece's start
      const int n = __shfl_sync(0xffffffffu, len, from), o = __shfl_sync(0xffffffffu, ends, from);
      if (!starts || i < begin || i >= from + n) return;
      const int to = i - begin + __popc(added & ((1u << from) - 1));
      const bool last = i == from + n - 1, old = (added >> from) & 1;
      src[to] = row;
      out[to] = last && !old ? o : -1;
      if (last && old) {
        src[to + 1] = ~o;
        out[to + 1] = o;
      }
    };
    list(t, x0.row);
    list(t + 32, x1.row);
    const int final = starts ? 31 - __clz(starts) : 0;
    const int n = __shfl_sync(0xffffffffu, len, final);
    if (t == 0) rows_[team] = starts ? final + n - begin + __popc(added) : 0;
  }
  if (TEAM > 32) __syncthreads();  // (of the block's teams)
  else __syncwarp();
  const int rows = rows_[team];
  float sum[N];
#pragma unroll
  for (int e = 0; e < N; ++e) sum[e] = 0.f;
  for (int r = 0; r < rows; r += kAheadHere) {
    C w[kAheadHere];
#pragma unroll
    for (int u = 0; u < kAheadHere; ++u) {
      if (r + u >= rows) break;
      const int i = src[r + u];
      w[u].load(i >= 0 ? dh + (int64_t)i * a.d : dw + (int64_t)~i * a.d, c0, a.d, t);
    }
#pragma unroll
    for (int u = 0; u < kAheadHere; ++u) {
      if (r + u >= rows) break;
      const int i = src[r + u], o = out[r + u];
      float v[N];
      w[u].get(v);
      if (i >= 0) {
#pragma unroll
        for (int e = 0; e < N; ++e) sum[e] += v[e];
        if (o == -1) continue;
      }
      if (o >= 0) {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = i >= 0 ? a.scale * sum[e] : fmaf(a.scale, sum[e], v[e]);
        C::store(dw + (int64_t)o * a.d, c0, a.d, t, v);
      } else {
        C::store_part(a.part + run * a.d, c0, a.d, t, sum);
      }
#pragma unroll
      for (int e = 0; e < N; ++e) sum[e] = 0.f;
    }
  }
}

// ------------------------------------------------------------------ join
constexpr int kJoinPlaces = 1024;  // places whose runs a block looks for frequent ids in
constexpr int kJoinCols = 4;     // columns of a lane, 32 apart
constexpr int kWarpParts = 64;   // pieces of an id that are one warp's work

struct Four {
  float v[kJoinCols];
};

// The sum of pieces first, first + step, ... of q, kRowsAhead of them on their way.
__device__ __forceinline__ Four join_parts(const float* part, int64_t apart, int64_t d, int64_t c,
                                           int first, int step, int q) {
  Four s{{0.f, 0.f, 0.f, 0.f}};
  for (int j = first; j < q; j += step * kRowsAhead) {
    float v[kRowsAhead][kJoinCols];
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u)
#pragma unroll
      for (int e = 0; e < kJoinCols; ++e)
        v[u][e] = j + u * step < q && c + 32 * e < d ? part[(j + u * step) * apart + c + 32 * e]
                                                     : 0.f;
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u)
#pragma unroll
      for (int e = 0; e < kJoinCols; ++e) s.v[e] += v[u][e];
  }
  return s;
}

template <class T, int THREADS>
__global__ void __launch_bounds__(THREADS) k_embed_join(ReduceGradArgs a, int cols) {
  constexpr int kWarps = THREADS / 32;
  __shared__ Head heads[kJoinPlaces / (2 * kPiece) + 1];
  __shared__ int count;
  __shared__ Four sums[kWarps][32];
  if (threadIdx.x == 0) count = 0;
  chain_wait();
  __syncthreads();
  const int64_t chunk = blockIdx.x / cols;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (blockIdx.x - chunk * cols) * (32 * kJoinCols) + lane;
  const int here = kJoinPlaces / a.run;  // runs, a thread each
  const int64_t run = chunk * here + threadIdx.x, runs = (a.n + a.run - 1) / a.run;
  if (threadIdx.x < here && run < runs) {
    const Head h = a.head[run];
    if (h.id >= 0) heads[atomicAdd(&count, 1)] = h;  // (in any order: each is summed by itself)
  }
  __syncthreads();
  const int n = count;
  // piece j begins kPiece j places behind the first: kPiece / run runs
  const int64_t apart = a.d * (kPiece / a.run);
  auto parts = [&](const Head& h) { return a.part + (int64_t)(h.seg.first / a.run) * a.d; };
  auto row = [&](const Head& h) { return static_cast<T*>(a.dw) + (int64_t)h.id * a.d + c; };
  auto old = [&](const Head& h) {  // what is added to
    Four o;
#pragma unroll
    for (int e = 0; e < kJoinCols; ++e) o.v[e] = a.accumulate && c + 32 * e < a.d ? to_f(row(h)[32 * e]) : 0.f;
    return o;
  };
  auto finish = [&](const Head& h, const Four& s, const Four& o) {
#pragma unroll
    for (int e = 0; e < kJoinCols; ++e)
      if (c + 32 * e < a.d)
        from_f(a.accumulate ? fmaf(a.scale, s.v[e], o.v[e]) : a.scale * s.v[e], row(h)[32 * e]);
  };
  for (int k = warp; k < n; k += kWarps) {
    const Head h = heads[k];
    const int q = h.seg.count / kPiece;
    if (q > kWarpParts) continue;
    const Four o = old(h);
    finish(h, join_parts(parts(h), apart, a.d, c, 0, 1, q), o);
  }
  for (int k = 0; k < n; ++k) {  // more pieces: all warps, their sums in order
    const Head h = heads[k];
    const int q = h.seg.count / kPiece;
    if (q <= kWarpParts) continue;
    sums[warp][lane] = join_parts(parts(h), apart, a.d, c, warp, kWarps, q);
    __syncthreads();
    if (warp == 0) {
      Four x = sums[0][lane];
      for (int w = 1; w < kWarps; ++w)
#pragma unroll
        for (int e = 0; e < kJoinCols; ++e) x.v[e] += sums[w][lane].v[e];
      finish(h, x, old(h));
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ plan
struct EmbedPlan {
  int lg, ids;         // sorting blocks and the ids of each
  int run;             // places a team starts pieces in
  size_t seg, place, live, head, part, bytes;
};

kd_status embed_plan(const kd_embed_problem* p, EmbedPlan& P) {
  if (!p || p->n_tokens < 0 || p->n_tokens > (int64_t)1 << 30 || p->vocab < 1 ||
      p->vocab > (int64_t)1 << 30 || p->d_model < 1 || p->d_model > (int64_t)1 << 30)
    return KD_ERR_INVALID_ARG;
  if (p->dtype != KD_BF16 && p->dtype != KD_FP32) return KD_ERR_INVALID_ARG;
  if (!std::isfinite(p->scale)) return KD_ERR_INVALID_ARG;
  P.lg = 7;  // 128 blocks, or as many as have kMaxIds ids at most
  while (rows_div(p->vocab, (int64_t)1 << P.lg) > kMaxIds) ++P.lg;
  P.ids = (int)rows_div(p->vocab, (int64_t)1 << P.lg);
  const int esz = p->dtype == KD_BF16 ? 2 : 4;
  // runs as short as leaves 16 teams an SM or, beyond that, kMostRun places: the
  // rows of a short run are one batch of loads
  const int64_t slices = rows_div(p->d_model * esz, 128 * 16);
  const int64_t teams = (int64_t)std::max(1, tc_num_sms()) * 16;
  P.run = kMinRun;
  while (P.run < kMostRun && p->n_tokens * slices > teams * P.run) P.run *= 2;
  const int64_t runs = rows_div(p->n_tokens, P.run);
  size_t off = 0;
  P.seg = rows_take(off, (size_t)p->vocab * sizeof(Segment));
  P.place = rows_take(off, (size_t)p->n_tokens * sizeof(Place));
  P.live = rows_take(off, 4);
  P.head = rows_take(off, (size_t)runs * sizeof(Head));
  P.part = rows_take(off, p->n_tokens >= 2 * kPiece ? (size_t)runs * p->d_model * 4 : 0);
  P.bytes = off;
  return KD_OK;
}

template <class T>
bool lookup_run(LookupArgs a, bool vec, cudaStream_t s) {
  a.parts = (int)(vec ? rows_div(a.d / RowVec<T>::N, 32 * kSpan) : rows_div(a.d, 32 * kSingles));
  // (60000 x 72 bf16, nine vectors: 9.8 us a warp a row; with rows behind one another
  // 4.2 us)
  if (vec && a.d / RowVec<T>::N <= 64) {
    const int64_t grid = rows_div(a.n * (a.d / RowVec<T>::N), 32 * kSpan * (kLookupThreads / 32));
    return grid <= INT32_MAX &&
           rows_launch(k_embed_short<T>, grid, kLookupThreads, 0, false, s, a);
  }
  const int64_t grid = rows_div(a.n * a.parts, kLookupThreads / 32);
  if (grid > INT32_MAX) return false;
  return vec ? rows_launch(k_embed_rows<T, true>, grid, kLookupThreads, 0, false, s, a)
             : rows_launch(k_embed_rows<T, false>, grid, kLookupThreads, 0, false, s, a);
}

// A team of as many warps as a row has vectors for, up to a block.
template <class T, int TEAM, bool VEC>
bool reduce_team(ReduceGradArgs a, bool chained, cudaStream_t s) {
  a.slices = (int)rows_div(a.d, Columns<T, TEAM, VEC>::kSlice);
  a.teams = rows_div(rows_div(a.n, a.run) * a.slices, kReduceThreads / TEAM);
  // Many small blocks, behind the ones that add: they fill the table from front to
  // back, which memory takes at 7.4 TB/s, and at 6.5 TB/s from everywhere at once.
  a.zeros = kReduceWarps * (int)std::min<int64_t>(
      32, std::max<int64_t>(1, kZeroBytes / kReduceWarps / (a.d * (int64_t)sizeof(T))));
  const int64_t grid = a.teams + (a.accumulate ? 0 : rows_div(a.vocab, a.zeros));
  return grid <= INT32_MAX &&
         rows_launch(k_embed_reduce<T, TEAM, VEC>, grid, kReduceThreads, 0, chained, s, a);
}
template <class T>
bool reduce_run(const ReduceGradArgs& a, bool vec, bool chained, cudaStream_t s) {
  auto team = [&](auto size) {
    constexpr int TEAM = decltype(size)::value;
    return vec ? reduce_team<T, TEAM, true>(a, chained, s)
               : reduce_team<T, TEAM, false>(a, chained, s);
  };
  const int64_t vecs = rows_div(a.d, RowVec<T>::N);
  const bool ok = vecs <= 32   ? team(std::integral_constant<int, 32>())
                  : vecs <= 64 ? team(std::integral_constant<int, 64>())
                               : team(std::integral_constant<int, 128>());
  if (!ok || a.n < 2 * kPiece) return ok;
  // few columns: larger blocks, for an id of many pieces (65536 tokens of 512, all the
  // same: 70 us with 1024 threads, 89 with 256; 16384 of 4096: 209 and 213 us the other way)
  const int64_t cols = rows_div(a.d, 32 * kJoinCols), join = rows_div(a.n, kJoinPlaces) * cols;
  if (join > INT32_MAX) return false;
  return cols < 16 ? rows_launch(k_embed_join<T, 1024>, join, 1024, 0, true, s, a, (int)cols)
                   : rows_launch(k_embed_join<T, 256>, join, 256, 0, true, s, a, (int)cols);
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
  // (a launch has at most 2^31 - 1 blocks)
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
  if (rows_div(p->n_tokens, kMostRun) * rows_div(p->d_model, 32) + p->vocab >= INT32_MAX)
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
  t.lg = P.lg;
  t.ids = P.ids;
  t.seg = reinterpret_cast<Segment*>(ws + P.seg);
  t.place = reinterpret_cast<Place*>(ws + P.place);
  t.live = reinterpret_cast<int32_t*>(ws + P.live);
  t.status = dev_status;
  const int smem = sort_smem(P.ids);
  // (always the same limit: another thread may be about to launch with more)
  if (smem > 40000 && cudaFuncSetAttribute(k_embed_sort, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           sort_smem(kMaxIds)) != cudaSuccess)
    return KD_ERR_CUDA;
  if (!rows_launch(k_embed_sort, (int64_t)1 << P.lg, kSortThreads, (size_t)smem, false, s, t))
    return KD_ERR_CUDA;
  ReduceGradArgs a;
  memset(&a, 0, sizeof(a));
  a.dh = d_h;
  a.dw = d_w;
  a.seg = t.seg;
  a.place = t.place;
  a.live = t.live;
  a.head = reinterpret_cast<Head*>(ws + P.head);
  a.part = reinterpret_cast<float*>(ws + P.part);
  a.n = p->n_tokens;
  a.vocab = p->vocab;
  a.d = p->d_model;
  a.run = P.run;
  a.accumulate = accumulate;
  a.scale = p->scale;
  const bool vec = row % 16 == 0 && rows_aligned(16, d_h, d_w);
  const bool chained = smem <= kChainedSmem;
  const bool ok = esz == 2 ? reduce_run<__nv_bfloat16>(a, vec, chained, s)
                           : reduce_run<float>(a, vec, chained, s);
  return ok && cudaGetLastError() == cudaSuccess ? KD_OK : KD_ERR_CUDA;
}
