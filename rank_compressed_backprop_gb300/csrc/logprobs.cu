// logprobs.cu -- log probabilities of given tokens from rows of logits, with the
// entropy and the largest alternatives, and the gradient of both.
//   m = max_j x_j,  d_j = x_j - m,  S = sum_j exp(scale d_j)
//   logp = scale d_t - log S,   H = log S - scale (sum_j d_j exp(scale d_j)) / S
//   p_j = exp(scale d_j - log S)
//   gx_j = scale (g (1[j = t] - p_j) - gH p_j (log p_j + H))
//
// Both are bound by HBM: the forward reads the logits once, a thread keeping the
// running maximum and sums of its vectors; the gradient reads them once and writes
// once.  Exponents are those of differences to the maximum, taken in one of two forms by
// its size (Part), so that a row of large logits keeps its accuracy and one that is masked
// whole, by whatever value, is a uniform one.
//
// A row belongs to one CTA, or to a cluster of up to kMaxShares when rows are few;
// its CTAs' results meet in shared memory of the first.
//
// Alternatives: no list is kept in order while the row streams by.  The k-th largest of the
// values that kSeen groups of threads have seen is a bound below which none of the k
// best lie; it is taken after the row's first batch of vectors and whenever the row read is
// four times as long (twice for many alternatives), and at the end if much has
// been kept.  Vectors that hold something above the bound are put by in shared memory, some
// 4 k of them a time, and what of them passes the last bound is ranked by counting.
// Larger comes first, NaN above everything, then the lower index: one 64-bit key an
// element, no two alike.
#include <algorithm>
#include <type_traits>

#include "ckpt.cuh"

namespace instant {

INSTANT_FAULT_READER(read_fault_logprobs)

namespace {

constexpr int kThreads = 256;    // of the gradient's CTAs
constexpr int kBatch = 4;        // 16-byte vectors a thread has under way
constexpr int kSeen = 64;        // groups of threads that a bound is taken from, twice INSTANT_TOP_MAX
constexpr int kGroups = 128;     // groups of slice_top
constexpr int kFewTop = 16;      // alternatives up to which bounds may be further apart
constexpr int kMaxCand = 512;    // elements at or above the bound that are ranked at once
constexpr int kFewKept = 256;    // vectors with one that are kept for up to kFewAsked alternatives
constexpr int kMaxKept = 512;    // and for more
constexpr int kFewAsked = 8;
constexpr int kManyKept = 64;    // of which a last bound sorts out
constexpr int kMaxShares = 8;    // CTAs of a row
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float inf_f() { return __uint_as_float(0x7f800000u); }

// maximum that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// over the warp
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// 16 bytes that no other CTA reads
__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <typename T>
constexpr int kPer = 16 / sizeof(T);  // elements of a vector

// a vector as pairs of fp32
__device__ __forceinline__ void to_pairs(const uint4& u, float2 (&v)[4]) {  // bf16
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void to_pairs(const uint4& u, float2 (&v)[2]) {  // fp32
  v[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
  v[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
}

// largest element of a vector, NaN if it holds one
__device__ __forceinline__ float vec_max(const uint4& u, uint16_t) {
  uint32_t a, b;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(u.x), "r"(u.y));
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(u.z), "r"(u.w));
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
  return max_nan(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
}
__device__ __forceinline__ float vec_max(const uint4& u, float) {
  return max_nan(max_nan(__uint_as_float(u.x), __uint_as_float(u.y)),
                 max_nan(__uint_as_float(u.z), __uint_as_float(u.w)));
}

// of a batch
__device__ __forceinline__ float batch_max(const uint4 (&u)[kBatch], uint16_t) {
  uint32_t a[kBatch];
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {
    uint32_t b;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a[j]) : "r"(u[j].x), "r"(u[j].y));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(u[j].z), "r"(u[j].w));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a[j]) : "r"(a[j]), "r"(b));
  }
#pragma unroll
  for (int j = 1; j < kBatch; ++j) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a[0]) : "r"(a[0]), "r"(a[j]));
  return max_nan(__uint_as_float(a[0] << 16), __uint_as_float(a[0] & 0xffff0000u));
}
__device__ __forceinline__ float batch_max(const uint4 (&u)[kBatch], float) {
  float m = vec_max(u[0], 0.f);
#pragma unroll
  for (int j = 1; j < kBatch; ++j) m = max_nan(m, vec_max(u[j], 0.f));
  return m;
}

// values below -1e37 as -1e37: their weight is 0 beside a maximum m with |m c| <= 2^20 (with
// c >= 1e-30, x c is -1e7), and the product with their exponent (at least -1e38) is no NaN
__device__ __forceinline__ uint4 not_below(const uint4& u, uint16_t) {
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(w[i]) : "r"(w[i]), "r"(0xfcf1fcf1u));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 not_below(const uint4& u, float) {
  auto f = [](uint32_t w) { return __float_as_uint(max_nan(__uint_as_float(w), -1e37f)); };
  return make_uint4(f(u.x), f(u.y), f(u.z), f(u.w));
}

template <typename T>
__device__ __forceinline__ uint4 no_vector() {  // of minus infinities
  const uint32_t w = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
  return make_uint4(w, w, w, w);
}

// order of the alternatives: value (minus zero like zero, NaN first), lower index first
__device__ __forceinline__ uint64_t element_key(float v, uint32_t index) {
  uint32_t b = __float_as_uint(v + 0.f);
  b = v != v ? 0xffffffffu : (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return (static_cast<uint64_t>(b) << 32) | (~index);
}
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t b = static_cast<uint32_t>(key >> 32);
  return __uint_as_float((b & 0x80000000u) ? b ^ 0x80000000u : ~b);
}
__device__ __forceinline__ uint32_t key_index(uint64_t key) { return ~static_cast<uint32_t>(key); }

// Running maximum and sums of a part of a row.  An exponent is taken as w = x c - mc with
// c = scale log2 e and mc = m c rounded, one FMA; rest = m c - mc, by which the rounding
// shifts all of them, is put right in the row's log S.  That is so while |m c| is at most
// 2^20, where the rest is below 2^-5; from 2^31 on 2^rest itself would leave the range of
// fp32.  Larger maxima (a row masked whole by some -1e10, one of the type's lowest values)
// and very large or small scales take w as (x - m) c instead.
struct Scale {
  float c, near;  // near: the largest |m| of the first form
};
struct Part {
  float m, s, a;  // max, sum 2^w, sum w 2^w
  __device__ __forceinline__ static bool careful(float m, const Scale& b) { return !(fabsf(m) <= b.near); }
  __device__ __forceinline__ static float ref(float m, const Scale& b) { return __fmul_rn(m, b.c); }  // mc, in no FMA
  __device__ __forceinline__ static float rest(float m, const Scale& b) {
    return careful(m, b) ? 0.f : fmaf(m, b.c, -ref(m, b));
  }
  // Moves the sums to another maximum (at least m, or a NaN), from the one form of an exponent
  // to the other where that changes.  s is finite, at most the number of its elements and 2^(2^-5).
  template <bool ENT>
  __device__ __forceinline__ void move(float m1, const Scale& b) {
    float t = ref(m, b) - ref(m1, b);
    if (careful(m, b) || careful(m1, b)) t = fmaf(m - m1, b.c, rest(m1, b) - rest(m, b));
    const float f = m == -inf_f() ? 0.f : ex2_approx(t);
    if (ENT) a = f == 0.f ? 0.f : f * fmaf(t, s, a);  // t may be huge where f is 0
    s = f * s;
    m = m1;
  }
  template <bool ENT>
  __device__ __forceinline__ void join(Part o, const Scale& b) {
    const float m1 = max_nan(m, o.m);
    if (!(m1 == m)) move<ENT>(m1, b);
    if (!(m1 == o.m)) o.move<ENT>(m1, b);
    s += o.s;
    a += o.a;
  }
  // log S from s: S = s 2^-rest
  __device__ __forceinline__ float log_sum(const Scale& b) const {
    return m == -inf_f() ? m : fmaf(-kLn2, rest(m, b), logf(s));
  }
};

// scale (x - m) - log S; halves, as the difference may pass the range of fp32 where the product does not
__device__ __forceinline__ float log_prob(float x, float m, float scale, float logs) {
  return fmaf(2.f * scale, 0.5f * x - 0.5f * m, -logs);
}

// the part of a row that one CTA reads: 16-byte vectors, and for the first CTA of
// the row the elements before the first boundary and after the last
template <typename T>
struct Slice {
  const T* row;
  int V, head, vecs, first, last;  // vectors [first, last) of `vecs` after `head` elements
  __device__ __forceinline__ Slice(const T* r, int V_, int rank, int shares) : row(r), V(V_) {
    constexpr int E = kPer<T>;
    const uintptr_t at = reinterpret_cast<uintptr_t>(r);
    head = min(V, static_cast<int>(((16 - (at & 15)) & 15) / sizeof(T)));
    vecs = (V - head) / E;
    const int per = (vecs + shares - 1) / shares;
    first = min(vecs, rank * per);
    last = min(vecs, first + per);
  }
  __device__ __forceinline__ const T* vec(int v) const { return row + head + static_cast<size_t>(v) * kPer<T>; }
  __device__ __forceinline__ int index(int v) const { return head + v * kPer<T>; }
  // elements outside the vectors: fewer than two vectors of them
  __device__ __forceinline__ int edges() const { return V - vecs * kPer<T>; }
  __device__ __forceinline__ int edge(int i) const { return i < head ? i : i + vecs * kPer<T>; }
};

// the largest key of the CTA (every thread gets it)
template <int NT>
__device__ uint64_t block_max_key(uint64_t k, uint64_t* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t p = __shfl_xor_sync(0xffffffffu, k, o);
    k = p > k ? p : k;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = k;
  __syncthreads();
  k = red[0];
#pragma unroll
  for (int w = 1; w < (NT / 32); ++w) k = red[w] > k ? red[w] : k;
  return k;
}

struct TopShared {
  float4 seen[kSeen / 4];    // the largest value of each group of threads
  uint32_t least[2];         // the bound, one in use and one for the next time
  int n_kept, n_cand, n_groups;
  uint64_t cand[kMaxCand];   // keys of the elements that are ranked
  uint64_t best[INSTANT_TOP_MAX];
  uint64_t bound, red[32];   // slice_top's
  int groups[INSTANT_TOP_MAX];
};

template <int ROOM>
struct TopKept : TopShared {
  uint4 kept[ROOM];  // vectors put by, and their numbers
  int kept_at[ROOM];
};
template <>
struct TopKept<0> {};  // no alternatives

// floats in the order of unsigned integers, and back
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t b) {
  return __uint_as_float((b & 0x80000000u) ? b ^ 0x80000000u : ~b);
}

__device__ __forceinline__ void top_start(TopShared& sh) {
  if (threadIdx.x < INSTANT_TOP_MAX) sh.best[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    sh.least[0] = 0xffffffffu;
    sh.n_kept = sh.n_cand = 0;
  }
}

// The k-th largest of what the groups of threads have seen (seen: a thread's largest value),
// or less where there is a NaN: at least k elements of the row so far are as large.  The
// CTA's threads together; turn: how many times before.
template <int NT>
__device__ __forceinline__ float top_bound(float seen, int k, int turn, TopShared& sh) {
  const int tid = threadIdx.x;
  constexpr int each = NT / kSeen;  // threads of a group
#pragma unroll
  for (int o = 1; o < each; o *= 2) seen = max_nan(seen, __shfl_xor_sync(0xffffffffu, seen, o));
  float* all = reinterpret_cast<float*>(sh.seen);
  if (tid % each == 0) all[tid / each] = seen;
  __syncthreads();
  if (tid < kSeen) {
    const float mine = all[tid];
    int above = 0;
#pragma unroll 8
    for (int i = 0; i < kSeen / 4; ++i) {
      const float4 v = sh.seen[i];
      above += (v.x > mine) + (v.y > mine) + (v.z > mine) + (v.w > mine);
    }
    const uint32_t m = __reduce_min_sync(0xffffffffu, above < k && mine == mine ? ordered(mine) : 0xffffffffu);
    if ((tid & 31) == 0) atomicMin(&sh.least[turn & 1], m);
  }
  if (tid == NT - 1) sh.least[(turn + 1) & 1] = 0xffffffffu;  // everyone has read the last one
  __syncthreads();
  const uint32_t least = sh.least[turn & 1];
  return least == 0xffffffffu ? -inf_f() : from_ordered(least);
}

// an element that may be one of the k best
__device__ __forceinline__ void offer(float v, int index, TopShared& sh) {
  const uint64_t key = element_key(v, index);
  const int at = atomicAdd(&sh.n_cand, 1);
  if (at < kMaxCand) sh.cand[at] = key;
}
template <typename T>
__device__ __forceinline__ void offer_vec(const uint4& u, int index, float least, TopShared& sh) {
  float2 x[kPer<T> / 2];
  to_pairs(u, x);
#pragma unroll
  for (int e = 0; e < kPer<T> / 2; ++e) {
    if (!(x[e].x < least)) offer(x[e].x, index + 2 * e, sh);  // a NaN too
    if (!(x[e].y < least)) offer(x[e].y, index + 2 * e + 1, sh);
  }
}

// the candidates in order into sh.best; false if there were too many
template <int NT>
__device__ __forceinline__ bool rank_candidates(int k, TopShared& sh) {
  __syncthreads();
  const int n = sh.n_cand;
  if (n > kMaxCand) return false;
  for (int i = threadIdx.x; i < n; i += NT) {
    const uint64_t mine = sh.cand[i];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) rank += sh.cand[j] > mine;
    if (rank < k) sh.best[rank] = mine;
  }
  __syncthreads();
  return true;
}

// a vector that may hold one
template <int ROOM>
__device__ __forceinline__ void keep_vec(const uint4& u, int v, TopKept<ROOM>& sh) {
  const int at = atomicAdd(&sh.n_kept, 1);
  if (at < ROOM) {
    sh.kept[at] = u;
    sh.kept_at[at] = v;
  }
}

// The k first elements of the slice that equal `value`, its largest, as candidates, found by
// one warp from the front: a row of one value (masked whole, or a head not yet trained) is
// done with its first vectors.  False if they lie further apart.
template <typename T>
__device__ __forceinline__ bool first_equal(const Slice<T>& sl, float value, int k, TopShared& sh) {
  __syncthreads();
  if (threadIdx.x < 32) {
    int v = sl.first + static_cast<int>(threadIdx.x);
    bool found = false;
    for (int i = 0; i < 32 && !found; ++i, v += 32) {
      if (v < sl.last) {
        float2 x[kPer<T> / 2];
        to_pairs(*reinterpret_cast<const uint4*>(sl.vec(v)), x);
#pragma unroll
        for (int e = 0; e < kPer<T> / 2; ++e) {
          if (x[e].x == value) offer(x[e].x, sl.index(v) + 2 * e, sh);
          if (x[e].y == value) offer(x[e].y, sl.index(v) + 2 * e + 1, sh);
        }
      }
      __syncwarp();
      found = *static_cast<volatile int*>(&sh.n_cand) >= k;  // 31 and one round's 256 at most
      __syncwarp();
    }
    if (threadIdx.x == 0) sh.n_groups = found;
  }
  __syncthreads();
  return sh.n_groups != 0;
}

// Keys of the k best elements of the slice, in order, into sh.best (0 where there are
// fewer), from the vectors put by and the row's edges (edge: this thread's, if edges);
// false if there were too many.  Behind a barrier that follows the last vector; seen and
// turn as in top_bound.
template <int NT, typename T, int ROOM>
__device__ __forceinline__ bool kept_top(const Slice<T>& sl, float least, float seen, int turn, int k, bool edges,
                                         float edge, TopKept<ROOM>& sh) {
  const int n = sh.n_kept;
  if (n > ROOM) {
    if (__syncthreads_or(!(seen <= least)) || !first_equal(sl, least, k, sh)) return false;
    if (edges && !(edge < least)) offer(edge, sl.edge(threadIdx.x), sh);
    return rank_candidates<NT>(k, sh);
  }
  if (n > kManyKept) least = top_bound<NT>(seen, k, turn, sh);
  for (int i = threadIdx.x; i < n; i += NT) offer_vec<T>(sh.kept[i], sl.index(sh.kept_at[i]), least, sh);
  if (edges && !(edge < least)) offer(edge, sl.edge(threadIdx.x), sh);
  return rank_candidates<NT>(k, sh);
}

// The same from the row itself, where too many of its elements are alike or its later parts
// hold most of the largest ones: the groups' best elements by their keys (the index rounded
// up to the last of a vector) give a bound that ties do not blur, and only the k best groups
// look at their vectors again; where most of the largest elements lie with a few threads,
// a pass an alternative.
template <int NT, typename T>
__device__ __noinline__ void slice_top(const Slice<T>& sl, int k, bool edges, TopShared& sh) {
  constexpr int E = kPer<T>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kG = NT < kGroups ? NT : kGroups, kEach = NT / kG;
  uint64_t best = 0;
  for (int v = sl.first + tid; v < sl.last; v += NT) {
    const uint64_t key = element_key(vec_max(*reinterpret_cast<const uint4*>(sl.vec(v)), T()), sl.index(v) + E - 1);
    best = key > best ? key : best;
  }
#pragma unroll
  for (int o = 1; o < kEach; o *= 2) {
    const uint64_t other = __shfl_xor_sync(0xffffffffu, best, o);
    best = other > best ? other : best;
  }
  __syncthreads();
  if (tid % kEach == 0) sh.cand[tid / kEach] = best;
  if (tid == 0) {
    sh.n_groups = 0;
    sh.bound = 0;
  }
  __syncthreads();
  const uint64_t mine = tid < kG ? sh.cand[tid] : 0;
  int rank = 0;
  for (int i = 0; i < kG; ++i) rank += sh.cand[i] > mine;
  if (mine != 0 && rank < k) {
    sh.groups[atomicAdd(&sh.n_groups, 1)] = tid;
    if (rank == k - 1) sh.bound = mine;
  }
  __syncthreads();
  if (tid == 0) sh.n_cand = 0;
  const uint64_t bound = sh.bound;
  __syncthreads();
  auto see = [&](float v, int index) {
    if (element_key(v, index) >= bound) offer(v, index, sh);
  };
  auto see_vec = [&](int v, auto f) {
    float2 x[E / 2];
    to_pairs(*reinterpret_cast<const uint4*>(sl.vec(v)), x);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      f(x[e].x, sl.index(v) + 2 * e);
      f(x[e].y, sl.index(v) + 2 * e + 1);
    }
  };
  const int rounds = (sl.last - sl.first + NT - 1) / NT;
  for (int g = warp; g < sh.n_groups; g += (NT / 32))
    for (int i = lane; i < rounds * kEach; i += 32) {
      const int v = sl.first + sh.groups[g] * kEach + i / kEach * NT + i % kEach;
      if (v < sl.last) see_vec(v, see);
    }
  const bool edge = edges && tid < sl.edges();
  if (edge) see(elem_to_f<T>(sl.row[sl.edge(tid)]), sl.edge(tid));
  if (rank_candidates<NT>(k, sh)) return;
  uint64_t below = ~0ull;
  for (int r = 0; r < k; ++r) {
    uint64_t top = 0;
    auto next = [&](float v, int index) {
      const uint64_t key = element_key(v, index);
      if (key < below && key > top) top = key;
    };
    for (int v = sl.first + tid; v < sl.last; v += NT) see_vec(v, next);
    if (edge) next(elem_to_f<T>(sl.row[sl.edge(tid)]), sl.edge(tid));
    below = block_max_key<NT>(top, sh.red);
    if (tid == 0) sh.best[r] = below;
  }
  __syncthreads();
}

__device__ __forceinline__ float dsmem_ld_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t dsmem_ld_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

// token of a row: negative (or past the vocabulary, which is reported) means none
__device__ __forceinline__ long long row_token(const void* t, int wide, int row, int V) {
  const long long v = wide ? static_cast<const long long*>(t)[row] : static_cast<const int*>(t)[row];
  if (v >= V) {
    raise_fault(FAULT_INDEX);
    return -1;
  }
  return v;
}

// NT threads, CTAS of them an SM; ROOM: vectors kept for alternatives, 0 without any.  With
// registers to spare the next batch's loads are under way while one is taken in, and while the
// CTA waits for its first bound (0.5 us of 16 at 513 x 30523 fp32)
template <typename T, int NT, int CTAS, bool ENT, int ROOM>
__global__ void __launch_bounds__(NT, CTAS) k_logprobs(const __grid_constant__ LogprobArgs a) {
  constexpr int E = kPer<T>;
  constexpr bool TOP = ROOM > 0;
  __shared__ Part red[(NT / 32)];
  __shared__ Part part;  // of this CTA
  __shared__ TopKept<ROOM> top;
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x, rank = blockIdx.z, shares = gridDim.z;
  const T* x = static_cast<const T*>(a.x) + static_cast<size_t>(row) * a.ld;
  const Slice<T> sl(x, a.V, rank, shares);
  const float c = a.scale * kLog2e;
  const Scale b{c, a.near};
  const bool first = rank == 0;

  long long token = -1;
  float xt = 0.f;
  if (first && tid == 0 && a.logp) {
    token = row_token(a.tokens, a.wide, row, a.V);
    if (token >= 0) xt = elem_to_f<T>(x[token]);
  }

  const bool edge = first && tid < sl.edges();
  const float xe = edge ? elem_to_f<T>(x[sl.edge(tid)]) : 0.f;

  Part p;
  p.m = -inf_f();
  p.s = p.a = 0.f;
  float2 s2 = both(0.f), a2 = both(0.f);
  float mc = 0.f, seen = -inf_f();  // seen: this thread's largest, for the alternatives
  bool careful = true;
  auto batch = [&](const uint4 (&u)[kBatch]) {  // returns the thread's largest
    const float own = batch_max(u, T());
    if (TOP) seen = max_nan(seen, own);
    // the warp's maximum, so that it moves some ln(batches) times: a thread's own moves in one lane or
    // another at almost every batch
    const float mb = warp_max(own);
    if (!(mb <= p.m)) {
      p.s = s2.x + s2.y;
      p.a = a2.x + a2.y;
      p.move<ENT>(max_nan(mb, p.m), b);
      s2 = make_float2(p.s, 0.f);
      a2 = make_float2(p.a, 0.f);
      mc = Part::ref(p.m, b);
      careful = Part::careful(p.m, b);
    }
    if (!careful) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        float2 w[E / 2];
        to_pairs(ENT ? not_below(u[j], T()) : u[j], w);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          w[e] = fma2(w[e], both(c), both(-mc));
          const float2 ex = make_float2(ex2_approx(w[e].x), ex2_approx(w[e].y));
          s2 = add2(s2, ex);
          if (ENT) a2 = fma2(w[e], ex, a2);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        float2 w[E / 2];
        to_pairs(u[j], w);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          const float2 d = p.m == -inf_f() ? w[e] : add2(w[e], both(-p.m));
          w[e] = mul2(d, both(c));
          const float2 ex = make_float2(ex2_approx(w[e].x), ex2_approx(w[e].y));
          s2 = add2(s2, ex);
          if (ENT) a2 = fma2(make_float2(fmaxf(w[e].x, -1e38f), fmaxf(w[e].y, -1e38f)), ex, a2);
        }
      }
    }
    return own;
  };
  constexpr int kStep = kBatch * NT;  // vectors of a batch
  int at = sl.first;                        // the batch's first, for all threads
  float least = 0.f;
  auto load = [&](uint4 (&u)[kBatch]) {  // minus infinities behind the last vector
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int v = at + j * NT + tid;
      u[j] = v < sl.last ? load_stream(sl.vec(v)) : no_vector<T>();
    }
  };
  constexpr bool kAhead = NT * CTAS <= 1024;
  uint4 ahead[kBatch];
  int turn = 0, next = 0;  // of the bound
  const int grow = a.top > kFewTop ? 2 : 4;
  if constexpr (TOP) {
    top_start(top);
    uint4 u[kBatch];
    load(u);
    const float own = batch(u);
    if constexpr (kAhead) {
      at += kStep;
      load(ahead);
      at -= kStep;
    }
    least = top_bound<NT>(seen, a.top, turn++, top);
    if (!(own < least)) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int v = at + j * NT + tid;
        if (!(vec_max(u[j], T()) < least) && v < sl.last) keep_vec(u[j], v, top);
      }
    }
    at += kStep;
    next = sl.first + grow * kStep;
  }
  auto later = [&](const uint4 (&u)[kBatch]) {
    const float own = batch(u);
    if constexpr (TOP) if (!(own <= least)) {  // what equals the bound comes after k others by now
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int v = at + j * NT + tid;
        if (!(vec_max(u[j], T()) <= least) && v < sl.last) keep_vec(u[j], v, top);
      }
    }
  };
  auto bound = [&] {  // before the batch at `at`
    if constexpr (TOP)
      if (at == next) {
        least = top_bound<NT>(seen, a.top, turn++, top);
        next = sl.first + grow * (at - sl.first);
      }
  };
  if constexpr (kAhead) {
    if (!TOP) load(ahead);
    while (at < sl.last) {
      uint4 u[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) u[j] = ahead[j];
      at += kStep;
      load(ahead);
      at -= kStep;
      bound();
      later(u);
      at += kStep;
    }
  } else {
    for (; at + kStep <= sl.last; at += kStep) {
      uint4 u[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) u[j] = load_stream(sl.vec(at + j * NT + tid));
      bound();
      later(u);
    }
    if (at < sl.last) {
      uint4 u[kBatch];
      load(u);
      bound();
      later(u);
    }
  }
  p.s = s2.x + s2.y;
  p.a = a2.x + a2.y;
  if (edge) {
    Part e;
    e.m = xe;
    const float w = Part::careful(e.m, b) ? e.m - e.m : Part::rest(e.m, b);  // NaN for an infinity
    e.s = e.m == -inf_f() ? 0.f : ex2_approx(w);
    e.a = e.m == -inf_f() ? 0.f : w * e.s;
    p.join<ENT>(e, b);
  }
  // over the warp, then over the CTA
  auto warp_join = [&](Part& q) {
    const float m1 = warp_max(q.m);
    if (!(m1 == q.m)) q.move<ENT>(m1, b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      q.s += __shfl_xor_sync(0xffffffffu, q.s, o);
      if (ENT) q.a += __shfl_xor_sync(0xffffffffu, q.a, o);
    }
  };
  warp_join(p);
  if (lane == 0) red[warp] = p;
  __syncthreads();
  if (warp == (TOP ? NT / 32 - 1 : 0)) {  // beside the other warps' work on the alternatives
    p = red[lane & (NT / 32 - 1)];
    if (lane >= NT / 32) {
      p.m = red[0].m;
      p.s = p.a = 0.f;
    }
    warp_join(p);
    if (lane == 0) part = p;
  }
  if constexpr (TOP)
    if (!kept_top<NT>(sl, least, seen, turn, a.top, edge, xe, top)) slice_top<NT>(sl, a.top, first, top);

  if (shares > 1) {
    cluster_sync();
    if (first && warp == 0) {
      if (lane < shares) {
        const uint32_t src = dsmem_addr(&part, lane);
        p.m = dsmem_ld_f32(src);
        p.s = dsmem_ld_f32(src + 4);
        p.a = dsmem_ld_f32(src + 8);
      } else {
        p.m = part.m;
        p.s = p.a = 0.f;
      }
      warp_join(p);
    }
    if constexpr (TOP) if (first) {
      // the CTAs' alternatives, ranked like one CTA's candidates (all distinct but for 0)
      __syncthreads();
      TopShared& sh = top;
      const int n = shares * a.top;
      static_assert(kMaxShares * INSTANT_TOP_MAX <= kMaxCand && kMaxShares * INSTANT_TOP_MAX <= 256, "one a thread");
      uint64_t mine = 0;
      if (tid < n) sh.cand[tid] = mine = dsmem_ld_u64(dsmem_addr(&sh.best[tid % a.top], tid / a.top));
      __syncthreads();
      int r = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) r += sh.cand[j] > mine;
      if (mine && r < a.top) sh.best[r] = mine;
    }
    __syncthreads();
    cluster_sync();  // no CTA leaves while its shared memory is read
    if (!first) return;
  }
  if (warp != 0) return;
  if (TOP && shares == 1) p = part;
  const bool none = p.m == -inf_f();
  const float logs = p.log_sum(b);
  if (lane == 0) {
    if (a.logp) a.logp[row] = token < 0 ? 0.f : none ? -inf_f() : log_prob(xt, p.m, a.scale, logs);
    if (a.stats) reinterpret_cast<float2*>(a.stats)[row] = make_float2(p.m, logs);
    if (ENT) a.entropy[row] = none ? 0.f : fmaf(-kLn2, p.a / p.s, logf(p.s));
  }
  if constexpr (TOP) if (lane < a.top) {
    const uint32_t id = key_index(top.best[lane]);
    const size_t o = static_cast<size_t>(row) * a.top + lane;
    if (a.top_ids) a.top_ids[o] = id;
    if (a.top_logp) a.top_logp[o] = none ? -inf_f() : log_prob(key_value(top.best[lane]), p.m, a.scale, logs);
  }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ uint4 from_pairs(const float2* v);
template <>
__device__ __forceinline__ uint4 from_pairs<uint16_t>(const float2* v) {
  return make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y),
                    pack_bf16x2(v[3].x, v[3].y));
}
template <>
__device__ __forceinline__ uint4 from_pairs<float>(const float2* v) {
  return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                    __float_as_uint(v[1].y));
}

template <typename T, bool ENT>
__global__ void __launch_bounds__(kThreads) k_logprobs_grad(const __grid_constant__ LogprobGradArgs a) {
  constexpr int E = kPer<T>;
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x;
  const int row = blockIdx.x, rank = blockIdx.y, shares = gridDim.y;
  const T* x = static_cast<const T*>(a.x) + static_cast<size_t>(row) * a.ld;
  T* gx = static_cast<T*>(a.gx) + static_cast<size_t>(row) * a.ld;
  const Slice<T> sl(x, a.V, rank, shares);
  T* body = gx + sl.head;

  const long long token = a.g_logp ? row_token(a.tokens, a.wide, row, a.V) : -1;
  const float2 st = reinterpret_cast<const float2*>(a.stats)[row];
  const bool none = st.x == -inf_f();
  const float g = token >= 0 ? a.scale * a.g_logp[row] : 0.f;
  const float gh = ENT ? a.scale * a.g_entropy[row] : 0.f;
  const float H = ENT ? a.entropy[row] : 0.f;
  const float c = a.scale * kLog2e;
  const float2 shift = both(-st.x), c2 = both(c), off = both(-st.y * kLog2e);

  // gradient of a pair but for the token's own 1
  auto grad2 = [&](float2 v) {
    float2 w = fma2(add2(v, shift), c2, off);  // log2 p
    if (ENT) w = make_float2(w.x < -16384.f ? -16384.f : w.x, w.y < -16384.f ? -16384.f : w.y);  // p = 0; keeps a NaN
    const float2 p = make_float2(ex2_approx(w.x), ex2_approx(w.y));
    float2 f = both(-g);
    if (ENT) f = fma2(both(-gh), fma2(w, both(kLn2), both(H)), f);
    return mul2(p, f);
  };

  const bool zero = none || (!ENT && token < 0);
  if (zero) {
    for (int v = sl.first + tid; v < sl.last; v += kThreads)
      reinterpret_cast<uint4*>(body)[v] = make_uint4(0, 0, 0, 0);
  } else {
    const long long tv = token - sl.head;
    const int hit = token >= sl.head && tv / E < sl.last ? static_cast<int>(tv / E) : -1;
    for (int v = sl.first + tid; v < sl.last; v += kBatch * kThreads) {
      uint4 u[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (v + j * kThreads < sl.last) u[j] = load_stream(sl.vec(v + j * kThreads));
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int vj = v + j * kThreads;
        if (vj >= sl.last) break;
        float2 o[E / 2];
        to_pairs(u[j], o);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) o[e] = grad2(o[e]);
        if (vj == hit) {
          const int k = static_cast<int>(tv % E);
#pragma unroll
          for (int e = 0; e < E / 2; ++e) {
            if (k == 2 * e) o[e].x += g;
            if (k == 2 * e + 1) o[e].y += g;
          }
        }
        reinterpret_cast<uint4*>(body)[vj] = from_pairs<T>(o);
      }
    }
  }
  if (rank) return;
  if (tid < sl.edges()) {
    const int i = sl.edge(tid);
    float o = 0.f;
    if (!zero) {
      o = grad2(both(elem_to_f<T>(x[i]))).x;
      if (i == token) o += g;
    }
    gx[i] = f_to_elem<T>(o);
  }
  for (int i = a.V + tid; i < a.ld; i += kThreads) gx[i] = f_to_elem<T>(0.f);
}

// Scale::near, below 0 where no maximum is near
float near_of(float c) { return c >= 1e-30f && c <= 10.f ? 1048576.f / c : -1.f; }

// CTAs of a row: enough for `per_sm` CTAs an SM, with a vector or more for every thread
int row_shares(int rows, int vecs, int threads, int per_sm, int most) {
  int n = 1;
  while (n < most && static_cast<long long>(rows) * n < static_cast<long long>(per_sm) * sm_count() &&
         vecs >= 2 * n * threads)
    n *= 2;
  return n;
}

}  // namespace

cudaError_t launch_logprobs(LogprobArgs a, bool bf16, cudaStream_t st) {
  a.near = near_of(a.scale * kLog2e);
  const int vecs = a.V / (bf16 ? 8 : 4);
  // Small CTAs hide one another's row ends, large ones are sooner done with a row when rows
  // are few.  us by shape, bf16, without / with five alternatives and entropy: 8192 x 6000
  // 0: 21.5 / 40.5, 1: 29.5 / 55; 1571 x 50001 0: 27 / 38.5, 1: 32 / 43; 1000 x 30000
  // 1: 13.5 / 20.7, 2: 13.0 / 20.9, 3: 16.2 / 26.5; 513 x 128000 1: 24 / 36, 2: 22 / 33,
  // 3: 23 / 37; 300 x 262144 1: 38 / 59, 2: 29 / 42, 3: 25 / 33; 8192 x 32768 0: 77.6 (0.99 of the bytes' rate)
  const long long sms = sm_count(), rows = a.rows;
  int shape = rows >= 8 * sms ? 0 : rows > 4 * sms ? 1 : rows > 2 * sms ? 2 : 3;
  if (vecs < 512) shape = 0;  // no batch for more threads
  // A cluster a row where rows leave SMs idle (one row of 128000 bf16, 512 threads, 1 / 2 / 4 / 8
  // CTAs: 5.8 / 4.5 / 3.4 / 3.0 us; but 160 x 30000 4.8 / 5.1 / 7.3 / 12.9)
  const int shares = shape == 3 ? row_shares(a.rows, vecs, 512, 1, kMaxShares) : 1;
  const dim3 grid(a.rows, 1, shares);
  auto go = [&](auto kernel, int nt) {
    return launch_ex(kernel, grid, dim3(nt), 0, st, shares, pdl_enabled(), a);
  };
  auto sized = [&](auto t, auto ent, auto top) {
    using T = decltype(t);
    constexpr bool E = decltype(ent)::value;
    constexpr int K = decltype(top)::value;
    switch (shape) {
      case 0: return go(k_logprobs<T, 128, 12, E, K>, 128);
      case 1: return go(k_logprobs<T, 256, 5, E, K>, 256);
      case 2: return go(k_logprobs<T, 256, 4, E, K>, 256);
      default: return go(k_logprobs<T, 512, 2, E, K>, 512);
    }
  };
  auto asked = [&](auto t) {
    auto with = [&](auto top) {
      return a.entropy ? sized(t, std::true_type(), top) : sized(t, std::false_type(), top);
    };
    // Shared memory that holds no vectors is L1's, for the loads that are under way: us at 1571 x
    // 50001, room for 512 / 256 / 128: five alternatives 36.2 / 35.2 / 35.2 (64: 38.9, overflows),
    // 32 alternatives 45.4 / 50 / 90
    if (a.top > kFewAsked) return with(std::integral_constant<int, kMaxKept>());
    if (a.top > 0) return with(std::integral_constant<int, kFewKept>());
    return with(std::integral_constant<int, 0>());
  };
  return bf16 ? asked(uint16_t()) : asked(0.f);
}

cudaError_t launch_logprobs_grad(const LogprobGradArgs& a, bool bf16, cudaStream_t st) {
  // few rows are shared out to some 16 CTAs an SM (513 x 30523 fp32 with the entropy's part,
  // one CTA a row 25.9 us, 2 23.9, 4 22.2, 8 21.9; 8192 x 32768 bf16 155.5, 154.3, 162, 181)
  const dim3 grid(a.rows, row_shares(a.rows, a.V / (bf16 ? 8 : 4), kThreads, 16, 64));
  const bool ent = a.g_entropy != nullptr;
  auto go = [&](auto kernel) { return launch_ex(kernel, grid, dim3(kThreads), 0, st, 1, pdl_enabled(), a); };
  if (bf16) return ent ? go(k_logprobs_grad<uint16_t, true>) : go(k_logprobs_grad<uint16_t, false>);
  return ent ? go(k_logprobs_grad<float, true>) : go(k_logprobs_grad<float, false>);
}

}  // namespace instant
