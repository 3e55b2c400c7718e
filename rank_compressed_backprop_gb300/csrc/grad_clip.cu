// grad_clip.cu -- the norm of many gradients together, and the gradients clipped by it.
//   N = scale sqrt(sum over all tensors of g^2),  f = min(1, max_norm / N),  out = g scale f
//
// Bound by HBM: each gradient is read once for the norm and once more to be scaled,
// the second time from L2 as far as it holds them, and written once.  The tensors are
// cut into chunks of kBytes that the CTAs take in turn, so the list may mix matrices with
// scalars.  k_grad_norm leaves a partial sum of squares a CTA (ClipPart); every CTA of
// k_grad_clip adds them in the same order and gets the same factor.
// The pointers travel in the launch's parameters: nothing is copied to the device, and
// a captured graph holds its own list.
//
// Squares are added in fp32 within a chunk (65 of a thread's at most) and in two fp32 words over
// a CTA's chunks and over the CTAs; vectors of very large or very small values in 64 bits
// throughout.  The two sums meet in 64 bits, before the root.
#include <algorithm>

#include "ckpt.cuh"

namespace instant {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 8;
constexpr int kBytes = kThreads * kUnroll * 16;  // a chunk: 16 bytes a thread and step
constexpr int kManyChunks = 2048;                // 64 MB

template <typename T>
constexpr int kPer = 16 / sizeof(T);

__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void values_of(const uint4& u, float (&v)[8], uint16_t) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void values_of(const uint4& u, float (&v)[4], float) {
  v[0] = __uint_as_float(u.x);
  v[1] = __uint_as_float(u.y);
  v[2] = __uint_as_float(u.z);
  v[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ uint4 packed(const float (&v)[8], uint16_t) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ uint4 packed(const float (&v)[4], float) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}

// Calls f(item, chunk within it) for the CTA's chunks, which lie gridDim.x apart, so that the
// CTAs together sweep over the tensors; from the last backwards when REVERSE.  The CTA's
// threads go together.  l.start has the items of the first (or last) gridDim.x chunks: a
// search took a chain of loads from the launch's parameters, each a miss in a long list.
template <bool REVERSE, typename List, typename F>
__device__ __forceinline__ void each_chunk(const List& l, F f) {
  int c = REVERSE ? l.chunks - 1 - static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x);
  int i = l.start[blockIdx.x];
  while (true) {
    f(l.item[i], c - l.item[i].chunk);
    c += REVERSE ? -static_cast<int>(gridDim.x) : static_cast<int>(gridDim.x);
    if (REVERSE ? c < 0 : c >= l.chunks) return;
    int lo = REVERSE ? 0 : i, hi = REVERSE ? i : l.count - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (l.item[mid].chunk <= c) lo = mid;
      else hi = mid - 1;
    }
    i = lo;
  }
}

// a thread's share of a chunk: up to kUnroll vectors, and for few threads an element
// before the first 16-byte boundary of the tensor or after the last
template <typename T>
struct ChunkAt {
  const T* g;
  T* out;
  long long vecs;    // of the tensor
  long long v0;      // the chunk's first vector
  int head, edges;
  bool aligned;      // out as g
  __device__ __forceinline__ ChunkAt(const ClipItem& it, int chunk) {
    g = static_cast<const T*>(it.g);
    out = static_cast<T*>(it.out);
    const uintptr_t at = reinterpret_cast<uintptr_t>(g);
    const long long h = ((16 - (at & 15)) & 15) / sizeof(T);
    head = static_cast<int>(h < it.n ? h : it.n);
    vecs = (it.n - head) / kPer<T>;
    v0 = static_cast<long long>(chunk) * (kThreads * kUnroll);
    edges = chunk == 0 ? static_cast<int>(it.n - vecs * kPer<T>) : 0;
    aligned = ((at ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
  }
  __device__ __forceinline__ long long edge(int i) const { return i < head ? i : i + vecs * kPer<T>; }
  __device__ __forceinline__ long long vec(int j) const { return v0 + j * kThreads + threadIdx.x; }
  __device__ __forceinline__ long long at(long long v) const { return head + v * kPer<T>; }
};

// Bounds of the values whose squares are added in fp32: 2^31 chunks of 2^14 values are 2^45 squares
// of at most 2^80, and their sum stays below 2^128
constexpr float kLarge = 1099511627776.f;          // 2^40
constexpr float kSmall = 8.8817841970012523e-16f;  // 2^-50

// Adds the squares of a thread's values to a sum in fp32 while the largest of them lies
// between the bounds (what a smaller one beside it may lose is below 2^-26 of the sum),
// else in 64 bits: of zeros nothing, a NaN or an infinity as it is.
template <int N>
__device__ __forceinline__ void add_squares(const float (&v)[N], float& mid, double& wide) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(v[i]));
  if (top <= kLarge && top >= kSmall) {
#pragma unroll
    for (int i = 0; i < N; ++i) mid = fmaf(v[i], v[i], mid);
    return;
  }
  float any = top;
#pragma unroll
  for (int i = 0; i < N; ++i) any = v[i] != v[i] ? v[i] : any;
  if (any == 0.f) return;
#pragma unroll
  for (int i = 0; i < N; ++i) wide = fma(static_cast<double>(v[i]), static_cast<double>(v[i]), wide);
}

// A sum in two fp32 words: what an addition rounds off goes to the second (Knuth's TwoSum).
// Sums in 64 bits by every thread took longer than the data here: the GPU adds two a cycle
// and SM.
struct Sum2 {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float t = __fadd_rn(hi, v), b = __fsub_rn(t, hi);
    lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(v, b));
    hi = t;
  }
  __device__ __forceinline__ void warp_sum() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float h = __shfl_xor_sync(0xffffffffu, hi, o), l = __shfl_xor_sync(0xffffffffu, lo, o);
      add(h);
      lo += l;
    }
  }
};

// the CTA's sums as one, for thread 0
__device__ __forceinline__ ClipPart block_sum(Sum2 sum, double wide, ClipPart* red) {
  sum.warp_sum();
  const bool any = __syncthreads_or(wide != 0.);  // a NaN too
  if (any) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) wide += __shfl_xor_sync(0xffffffffu, wide, o);
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = ClipPart{sum.hi, sum.lo, wide};
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      sum.add(red[w].hi);
      sum.lo += red[w].lo;
    }
    if (any)
      for (int w = 1; w < kWarps; ++w) wide += red[w].wide;
  }
  return ClipPart{sum.hi, sum.lo, wide};
}

template <typename T>
__device__ __forceinline__ void chunk_squares(const ClipItem& it, int chunk, float& mid, double& wide) {
  const ChunkAt<T> k(it, chunk);
  uint4 u[kUnroll];
#pragma unroll
  for (int j = 0; j < kUnroll; ++j)
    u[j] = k.vec(j) < k.vecs ? load_once(k.g + k.at(k.vec(j))) : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    float v[kPer<T>];
    values_of(u[j], v, T());
    add_squares(v, mid, wide);
  }
  if (static_cast<int>(threadIdx.x) < k.edges) {
    const float v[1] = {elem_to_f<T>(k.g[k.edge(threadIdx.x)])};
    add_squares(v, mid, wide);
  }
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const ClipItem& it, int chunk, float f) {
  const ChunkAt<T> k(it, chunk);
  uint4 u[kUnroll];
#pragma unroll
  for (int j = 0; j < kUnroll; ++j)
    if (k.vec(j) < k.vecs) u[j] = load_once(k.g + k.at(k.vec(j)));
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    if (k.vec(j) >= k.vecs) break;
    float v[kPer<T>];
    values_of(u[j], v, T());
#pragma unroll
    for (int i = 0; i < kPer<T>; ++i) v[i] *= f;
    T* o = k.out + k.at(k.vec(j));
    if (k.aligned) {
      *reinterpret_cast<uint4*>(o) = packed(v, T());
    } else {
#pragma unroll
      for (int i = 0; i < kPer<T>; ++i) o[i] = f_to_elem<T>(v[i]);
    }
  }
  if (static_cast<int>(threadIdx.x) < k.edges) {
    const long long i = k.edge(threadIdx.x);
    k.out[i] = f_to_elem<T>(elem_to_f<T>(k.g[i]) * f);
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads, kClipCtas) k_grad_norm(const __grid_constant__ ClipList<N> l) {
  __shared__ ClipPart red[kWarps];
  pdl_launch_dependents();
  pdl_wait();
  Sum2 sum;
  double wide = 0.;
  each_chunk<false>(l, [&](const ClipItem& it, int chunk) {
    float mid = 0.f;
    if (it.bf16) chunk_squares<uint16_t>(it, chunk, mid, wide);
    else chunk_squares<float>(it, chunk, mid, wide);
    sum.add(mid);
  });
  const ClipPart all = block_sum(sum, wide, red);
  if (threadIdx.x == 0) l.part[l.part0 + blockIdx.x] = all;
}

// a power of two in 64 bits, and the exponent of a positive normal number
__device__ __forceinline__ double pow2(int k) { return __hiloint2double((1023 + k) << 20, 0); }
__device__ __forceinline__ int exponent(double v) { return ((__double2hiint(v) >> 20) & 0x7ff) - 1023; }

// Square root of a sum of squares times scale: an fp32 root of a number in [1, 4), the power
// of two and the scale put back in 64 bits (a root and a quotient in 64 bits by every CTA
// took some microseconds)
__device__ __forceinline__ double norm_of(double all, float scale) {
  if (!(all > 1e-300 && all < 1e300)) return all;  // 0, infinity, NaN
  const int k = exponent(all) >> 1;
  return static_cast<double>(__fsqrt_rn(static_cast<float>(all * pow2(-2 * k)))) * pow2(k) * scale;
}
// max_norm / norm for a norm above max_norm, both with the norm's power of two taken out
__device__ __forceinline__ float factor_of(float max_norm, double norm) {
  const double p = pow2(-exponent(norm));
  return static_cast<float>(max_norm * p) / static_cast<float>(norm * p);
}

// The factor of all gradients from the CTAs' sums; out: where the norm and the factor go, or null
__device__ __forceinline__ float common_factor(const ClipPart* part, int parts, float max_norm, float scale, float* out) {
  __shared__ ClipPart red[kWarps];
  __shared__ float factor;
  Sum2 sum;
  double wide = 0.;
#pragma unroll 2
  for (int i = threadIdx.x; i < parts; i += kThreads) {
    const ClipPart p = part[i];
    sum.add(p.hi);
    sum.lo += p.lo;
    if (p.wide != 0.) wide += p.wide;
  }
  const ClipPart all = block_sum(sum, wide, red);
  if (threadIdx.x == 0) {
    const double norm = norm_of(static_cast<double>(all.hi) + all.lo + all.wide, scale);
    // a norm that is not finite in fp32 clips nothing
    const bool clips = static_cast<float>(norm) <= 3.4028235e38f && norm > max_norm;
    const float f = clips ? factor_of(max_norm, norm) : 1.f;
    if (out) {
      out[0] = static_cast<float>(norm);
      out[1] = f;
    }
    factor = f * scale;
  }
  __syncthreads();
  return factor;
}

template <int N>
__global__ void __launch_bounds__(kThreads, kClipCtas) k_grad_clip(const __grid_constant__ ClipList<N> l) {
  pdl_launch_dependents();
  pdl_wait();
  const float f = common_factor(l.part, l.parts, l.max_norm, l.scale, blockIdx.x == 0 ? l.norm : nullptr);
  if ((f == 1.f && l.in_place) || l.chunks == 0) return;
  // the other way round: what was read last is still in L2
  each_chunk<true>(l, [&](const ClipItem& it, int chunk) {
    if (it.bf16) chunk_scale<uint16_t>(it, chunk, f);
    else chunk_scale<float>(it, chunk, f);
  });
}

// Long lists: the factor by itself, and a CTA a chunk.
__global__ void __launch_bounds__(kThreads) k_grad_factor(ClipPart* part, int parts, float max_norm, float scale, float* norm) {
  pdl_launch_dependents();
  pdl_wait();
  const float f = common_factor(part, parts, max_norm, scale, norm);
  if (threadIdx.x == 0) part[parts].hi = f;
}
template <int N>
__global__ void __launch_bounds__(kThreads, kClipCtas) k_grad_scale(const __grid_constant__ ClipList<N> l) {
  pdl_launch_dependents();
  const int c = l.chunks - 1 - static_cast<int>(blockIdx.x);
  int lo = 0, hi = l.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (l.item[mid].chunk <= c) lo = mid;
    else hi = mid - 1;
  }
  const ClipItem& it = l.item[lo];
  pdl_wait();
  const float f = l.part[l.parts].hi;
  if (f == 1.f && l.in_place) return;
  if (it.bf16) chunk_scale<uint16_t>(it, c - it.chunk, f);
  else chunk_scale<float>(it, c - it.chunk, f);
}

}  // namespace

long long clip_chunks(long long n, bool bf16) {
  const long long per = kBytes / (bf16 ? 2 : 4);
  return (n + per - 1) / per;
}

template <int N>
cudaError_t launch_grad_norm(const ClipList<N>& l, cudaStream_t st) {
  return launch_ex(k_grad_norm<N>, dim3(l.ctas), dim3(kThreads), 0, st, 1, pdl_enabled(), l);
}
// A CTA a chunk writes long lists at 6.65 TB/s over the three passes where CTAs that stay
// reach 6.25 (90 million fp32 values into other buffers 162.6 us, not 173.3; 34 million
// 65.6, not 68.6), but costs a launch, and 10 us of CTAs that find nothing to do where the
// gradients are in place and not clipped.
template <int N>
cudaError_t launch_grad_clip(const ClipList<N>& l, cudaStream_t st) {
  if (l.chunks <= kManyChunks || (l.in_place && l.scale == 1.f))
    return launch_ex(k_grad_clip<N>, dim3(l.ctas), dim3(kThreads), 0, st, 1, pdl_enabled(), l);
  const cudaError_t e =
      launch_ex(k_grad_factor, dim3(1), dim3(kThreads), 0, st, 1, pdl_enabled(), l.part, l.parts, l.max_norm, l.scale, l.norm);
  if (e != cudaSuccess) return e;
  return launch_ex(k_grad_scale<N>, dim3(l.chunks), dim3(kThreads), 0, st, 1, pdl_enabled(), l);
}
#define INSTANT_CLIP_LIST(N)                                               \
  template cudaError_t launch_grad_norm(const ClipList<N>&, cudaStream_t); \
  template cudaError_t launch_grad_clip(const ClipList<N>&, cudaStream_t);
INSTANT_CLIP_LIST(kClipItems[0])
INSTANT_CLIP_LIST(kClipItems[1])
INSTANT_CLIP_LIST(kClipItems[2])
INSTANT_CLIP_LIST(kClipItems[3])

}  // namespace instant
