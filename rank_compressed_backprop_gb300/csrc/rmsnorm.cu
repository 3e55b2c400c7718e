// rmsnorm.cu -- root-mean-square norm with the residual's addition and an 8-bit
// checkpoint of its normalised rows, and the gradient from that checkpoint.
//   h = x + res,  r = (mean_j h_j^2 + eps)^(-1/2),  u = h r,  y = u gamma
//   d = gy gamma, c = mean_j(d_j u_j),  gx = r (d - u c) + res,  ggamma = sum_t gy u
// The backward reads u from its codes and r, so a training step keeps one byte
// an element of the norm and neither h nor y.
//
// Both directions are bound by HBM: a row stays in its threads' registers
// between the reduction and the outputs, so every tensor crosses the bus once.
// A thread holds V vectors of eight channels; W warps share a row, and a CTA
// takes several rows when rows are short.  Sixteen neighbouring lanes hold one
// checkpoint group.
#include "ckpt.cuh"

namespace instant {

namespace {

// sum over the W warps of a row; every thread gets it.  red: two buffers of 32
// floats used in turn, so one barrier a row is enough.  Rows of one warp need
// no barrier; with several the whole CTA meets (all its rows move in step).
template <int W>
__device__ __forceinline__ float row_sum(float v, float* red, int warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (W == 1) return v;
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  __syncthreads();
  float sum = 0.f;
  const int first = warp / W * W;
#pragma unroll
  for (int i = 0; i < W; ++i) sum += red[first + i];
  return sum;
}

template <typename T, int W, int V>
__global__ void __launch_bounds__(W > 8 ? 32 * W : 256)
    k_rms_norm(NormArgs a) {
  constexpr int kWarps = W > 8 ? W : 8;
  constexpr int kRows = kWarps / W;  // rows of a CTA
  __shared__ float red[32];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5;
  const int t = threadIdx.x % (32 * W);  // thread within its row
  const int row = blockIdx.x * kRows + warp / W;
  const bool on = row < a.rows;
  const size_t base = static_cast<size_t>(on ? row : 0) * a.C;
  const T* x = static_cast<const T*>(a.x) + base;
  const T* res = a.res ? static_cast<const T*>(a.res) + base : nullptr;
  float h[V][8];
  float ss = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = 8 * (v * 32 * W + t);
    load_part<8>(x + c, on ? a.C - c : 0, a.vec, h[v]);
    if (res) {
      float o[8];
      load_part<8>(res + c, on ? a.C - c : 0, a.vec, o);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[v][e] += o[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(h[v][e], h[v][e], ss);
  }
  const float r = rsqrtf(row_sum<W>(ss, red, warp) / static_cast<float>(a.C) + a.eps);
  if (!on) return;  // a whole warp at a time
  if (a.r && t == 0) a.r[row] = r;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = 8 * (v * 32 * W + t);
    const int n = a.C - c;
    if (a.h) store_part<8>(static_cast<T*>(a.h) + base + c, n, a.vec, h[v]);
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[v][e] *= r;
      m = max(m, abs_bits(h[v][e]));
    }
    if (a.k.q) {
      const uint32_t code = ckpt_scale_code(half_warp_max(m));
      const float inv = ckpt_inv_scale(code);
      if (n > 0)
        *reinterpret_cast<uint2*>(a.k.q + static_cast<size_t>(row) * a.ld + c) =
            make_uint2(ckpt_code4(h[v][0], h[v][1], h[v][2], h[v][3], inv),
                       ckpt_code4(h[v][4], h[v][5], h[v][6], h[v][7], inv));
      if (n > 0 && (threadIdx.x & 15) == 0)
        a.k.s[static_cast<size_t>(c / kCkptGroup) * a.rows + row] = static_cast<uint8_t>(code);
    }
    float g[8];
    load_part<8>(static_cast<const T*>(a.gamma) + c, n, a.vec, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] *= h[v][e];
    if (a.y) store_part<8>(static_cast<T*>(a.y) + base + c, n, a.vec, g);
  }
}

// Rows go round the CTAs; a thread keeps its columns' share of ggamma in
// registers over all its rows, the CTA's row slots add theirs in shared memory
// at the end, and a second kernel adds the CTAs' shares in a fixed order.
template <typename T, int W, int V>
__global__ void __launch_bounds__(W > 8 ? 32 * W : 256)
    k_rms_norm_back(NormBackArgs a) {
  constexpr int kWarps = W > 8 ? W : 8;
  constexpr int kRows = kWarps / W;
  extern __shared__ float gsum[];  // [kRows > 1][8 * 32 * W * V]
  __shared__ float red[2][32];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5;
  const int t = threadIdx.x % (32 * W);
  const int slot = warp / W;
  float acc[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[v][e] = 0.f;
  const float inv_c = 1.f / static_cast<float>(a.C);
  int it = 0;
  for (int row0 = blockIdx.x * kRows; row0 < a.rows; row0 += gridDim.x * kRows, ++it) {
    const int row = row0 + slot;
    const bool on = row < a.rows;
    const size_t base = static_cast<size_t>(on ? row : 0) * a.C;
    const float r = on ? a.r[row] : 0.f;
    float u[V][8], d[V][8];
    float dot = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 8 * (v * 32 * W + t);
      const int n = on ? a.C - c : 0;
      float gm[8];
      load_part<8>(static_cast<const T*>(a.gy) + base + c, n, a.vec, d[v]);
      load_part<8>(static_cast<const T*>(a.gamma) + c, n, a.vec, gm);
      uint2 w = make_uint2(0u, 0u);
      float scale = 0.f;
      if (n > 0) {
        w = *reinterpret_cast<const uint2*>(a.k.q + static_cast<size_t>(row) * a.ld + c);
        scale = ckpt_scale(a.k.s[static_cast<size_t>(c / kCkptGroup) * a.rows + row]);
      }
      ckpt_values4(w.x, scale, u[v]);
      ckpt_values4(w.y, scale, u[v] + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e >= n) u[v][e] = 0.f;  // padding codes are not defined
        acc[v][e] = fmaf(d[v][e], u[v][e], acc[v][e]);
        d[v][e] *= gm[e];
        dot = fmaf(d[v][e], u[v][e], dot);
      }
    }
    const float c1 = row_sum<W>(dot, red[it & 1], warp) * inv_c;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 8 * (v * 32 * W + t);
      const int n = on ? a.C - c : 0;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = r * (d[v][e] - u[v][e] * c1);
      if (a.res) {
        float q[8];
        load_part<8>(static_cast<const T*>(a.res) + base + c, n, a.vec, q);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += q[e];
      }
      store_part<8>(static_cast<T*>(a.gx) + base + c, n, a.vec, o);
    }
  }
  if (kRows > 1) {
    // the row slots' sums, slot 0 first
    for (int s = 0; s < kRows; ++s) {
      if (slot == s) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float* p = gsum + 8 * (v * 32 * W + t) + e;
            *p = s == 0 ? acc[v][e] : *p + acc[v][e];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.C; c += blockDim.x)
      a.part[static_cast<size_t>(blockIdx.x) * a.C + c] = gsum[c];
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 8 * (v * 32 * W + t);
      float* p = a.part + static_cast<size_t>(blockIdx.x) * a.C + c;
      store_part<8>(p, a.C - c, a.C % 4 == 0, acc[v]);
    }
  }
}

// warps a row and vectors a thread: the fewest threads that hold the row in two
// vectors each, and four vectors only for rows beyond 32 x 32 x 16 channels
#define INSTANT_NORM_DISPATCH(C, GO)                     \
  do {                                                   \
    if ((C) <= 256) GO(1, 1);                            \
    if ((C) <= 512) GO(1, 2);                            \
    if ((C) <= 1024) GO(2, 2);                           \
    if ((C) <= 2048) GO(4, 2);                           \
    if ((C) <= 4096) GO(8, 2);                           \
    if ((C) <= 8192) GO(16, 2);                          \
    if ((C) <= 16384) GO(32, 2);                         \
    GO(32, 4);                                           \
  } while (0)

template <typename T, int W, int V>
cudaError_t norm_go(const NormArgs& a, cudaStream_t st) {
  constexpr int kWarps = W > 8 ? W : 8;
  constexpr int kRows = kWarps / W;
  return launch_ex(k_rms_norm<T, W, V>, dim3((a.rows + kRows - 1) / kRows), dim3(32 * kWarps), 0, st, 1,
                   pdl_enabled(), a);
}

template <typename T>
cudaError_t norm_dispatch(const NormArgs& a, cudaStream_t st) {
#define GO(W, V) return norm_go<T, W, V>(a, st)
  INSTANT_NORM_DISPATCH(a.C, GO);
#undef GO
}

template <typename T, int W, int V>
cudaError_t back_go(const NormBackArgs& a, cudaStream_t st) {
  constexpr int kWarps = W > 8 ? W : 8;
  constexpr int kRows = kWarps / W;
  const size_t smem = kRows > 1 ? sizeof(float) * 8 * 32 * W * V : 0;
  const cudaError_t e =
      launch_ex(k_rms_norm_back<T, W, V>, dim3(norm_back_parts(a.rows, a.C)), dim3(32 * kWarps), smem, st,
                1, pdl_enabled(), a);
  if (e != cudaSuccess) return e;
  return launch_part_sum(a.part, a.ggamma, norm_back_parts(a.rows, a.C), a.C, a.accumulate, st);
}

template <typename T>
cudaError_t back_dispatch(const NormBackArgs& a, cudaStream_t st) {
#define GO(W, V) return back_go<T, W, V>(a, st)
  INSTANT_NORM_DISPATCH(a.C, GO);
#undef GO
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? norm_dispatch<uint16_t>(a, st) : norm_dispatch<float>(a, st);
}

// CTAs of the backward, each with one share of ggamma: two to eight per SM
// (about 2048 threads), no more than there are row slots
int norm_back_parts(int rows, int C) {
  int w = 1;
  while (w < 32 && 512 * w < C) w *= 2;
  const int slots = w > 8 ? 1 : 8 / w;
  const long long ctas = (static_cast<long long>(rows) + slots - 1) / slots;
  const long long most = static_cast<long long>(kColSumSMs) * (w > 8 ? 64 / w : 4);
  return static_cast<int>(ctas < most ? ctas : most);
}

cudaError_t launch_rms_norm_back(const NormBackArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? back_dispatch<uint16_t>(a, st) : back_dispatch<float>(a, st);
}

}  // namespace instant
