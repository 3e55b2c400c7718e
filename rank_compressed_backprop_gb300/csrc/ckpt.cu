// ckpt.cu -- 8-bit activation checkpoints of tensors that no other kernel
// here produced (pack), their values (unpack), and the column sums of a
// gradient (the bias gradient next to a weight gradient).
//
// All three are bound by HBM: pack reads each element once and writes one byte
// for it, unpack the reverse.  A half warp owns one group of 128 channels, eight
// channels a lane, so that the group's largest magnitude is four shuffles away.
#include "ckpt.cuh"

namespace instant {

namespace {

constexpr int kThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_ckpt_pack(const T* __restrict__ x, int8_t* __restrict__ q, uint8_t* __restrict__ s, int rows,
                int C, int ld, int groups, int vec) {
  pdl_launch_dependents();
  pdl_wait();
  const int hl = threadIdx.x & 15;
  const long long total = static_cast<long long>(rows) * groups;
  const long long stride = static_cast<long long>(gridDim.x) * (kThreads / 16);
  // whole warps stay in the loop together: the shuffles name all 32 lanes
  for (long long i0 = static_cast<long long>(blockIdx.x) * (kThreads / 16); i0 < total; i0 += stride) {
    const long long i = i0 + (threadIdx.x >> 4);
    const bool on = i < total;
    const int row = on ? static_cast<int>(i / groups) : 0;
    const int g = on ? static_cast<int>(i - static_cast<long long>(row) * groups) : 0;
    const int c = g * kCkptGroup + 8 * hl;
    float v[8];
    load_part<8>(x + static_cast<size_t>(row) * C + c, on ? C - c : 0, vec, v);
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, abs_bits(v[e]));
    const uint32_t code = ckpt_scale_code(half_warp_max(m));
    const float inv = ckpt_inv_scale(code);
    if (on && c < C)
      *reinterpret_cast<uint2*>(q + static_cast<size_t>(row) * ld + c) =
          make_uint2(ckpt_code4(v[0], v[1], v[2], v[3], inv), ckpt_code4(v[4], v[5], v[6], v[7], inv));
    if (on && hl == 0) s[static_cast<size_t>(g) * rows + row] = static_cast<uint8_t>(code);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_ckpt_unpack(const int8_t* __restrict__ q, const uint8_t* __restrict__ s, T* __restrict__ x,
                  int rows, int C, int ld, int chunks, int vec) {
  pdl_launch_dependents();
  pdl_wait();
  const long long total = static_cast<long long>(rows) * chunks;  // 16 channels each
  const long long stride = static_cast<long long>(gridDim.x) * kThreads;
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < total; i += stride) {
    const int row = static_cast<int>(i / chunks);
    const int c = 16 * static_cast<int>(i - static_cast<long long>(row) * chunks);
    const uint4 w = *reinterpret_cast<const uint4*>(q + static_cast<size_t>(row) * ld + c);
    const float scale = ckpt_scale(s[static_cast<size_t>(c / kCkptGroup) * rows + row]);
    float v[16];
    ckpt_values4(w.x, scale, v);
    ckpt_values4(w.y, scale, v + 4);
    ckpt_values4(w.z, scale, v + 8);
    ckpt_values4(w.w, scale, v + 12);
    T* dst = x + static_cast<size_t>(row) * C + c;
    store_part<8>(dst, C - c, vec, v);
    if (C - c > 8) store_part<8>(dst + 8, C - c - 8, vec, v + 8);
  }
}

// Column sums in two fixed-order stages (no atomics: the same bits on every
// call).  Stage 1: a CTA sums `per` rows of 8 x 32 columns, eight warps taking
// the rows in turn; stage 2 adds the row shares.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_col_sum(const T* __restrict__ x, float* __restrict__ part, int rows, int C, int per, int vec) {
  __shared__ float red[8][kThreads];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 256 + 8 * lane;
  const int r0 = blockIdx.y * per;
  const int r1 = min(rows, r0 + per);
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int r = r0 + warp; r < r1; r += 8) {
    float v[8];
    load_part<8>(x + static_cast<size_t>(r) * C + c, C - c, vec, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += v[e];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) red[warp][8 * lane + e] = acc[e];
  __syncthreads();
  float sum = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) sum += red[w][threadIdx.x];
  const int col = blockIdx.x * 256 + threadIdx.x;
  if (col < C) part[static_cast<size_t>(blockIdx.y) * C + col] = sum;
}

// out[c] (+)= sum_p part[p][c]: 32 columns a CTA, eight warps share the parts
__global__ void __launch_bounds__(kThreads)
    k_part_sum(const float* __restrict__ part, float* __restrict__ out, int parts, int C,
               int accumulate) {
  __shared__ float red[8][32];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float acc = 0.f;
  if (c < C) {
#pragma unroll 8
    for (int p = warp; p < parts; p += 8) acc += part[static_cast<size_t>(p) * C + c];
  }
  red[warp][lane] = acc;
  __syncthreads();
  if (warp == 0 && c < C) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) sum += red[w][lane];
    out[c] = accumulate ? out[c] + sum : sum;
  }
}

int grid_for(long long work, int per_cta, int per_sm) {
  const long long n = (work + per_cta - 1) / per_cta;
  const long long cap = static_cast<long long>(per_sm) * sm_count();
  return static_cast<int>(n < cap ? n : cap);
}

}  // namespace

cudaError_t launch_ckpt_pack(const void* x, const CkptRef& k, int rows, int C, bool bf16, bool vec,
                             cudaStream_t st) {
  const int groups = (C + kCkptGroup - 1) / kCkptGroup;
  const int grid = grid_for(static_cast<long long>(rows) * groups, kThreads / 16, 32);
  if (bf16)
    return launch_ex(k_ckpt_pack<uint16_t>, dim3(grid), dim3(kThreads), 0, st, 1, pdl_enabled(),
                     static_cast<const uint16_t*>(x), k.q, k.s, rows, C, ckpt_ld(C), groups, int(vec));
  return launch_ex(k_ckpt_pack<float>, dim3(grid), dim3(kThreads), 0, st, 1, pdl_enabled(),
                   static_cast<const float*>(x), k.q, k.s, rows, C, ckpt_ld(C), groups, int(vec));
}

cudaError_t launch_ckpt_unpack(const CkptRef& k, void* x, int rows, int C, bool bf16, bool vec,
                               cudaStream_t st) {
  const int chunks = (C + 15) / 16;
  const int grid = grid_for(static_cast<long long>(rows) * chunks, kThreads, 32);
  if (bf16)
    return launch_ex(k_ckpt_unpack<uint16_t>, dim3(grid), dim3(kThreads), 0, st, 1, pdl_enabled(),
                     static_cast<const int8_t*>(k.q), static_cast<const uint8_t*>(k.s),
                     static_cast<uint16_t*>(x), rows, C, ckpt_ld(C), chunks, int(vec));
  return launch_ex(k_ckpt_unpack<float>, dim3(grid), dim3(kThreads), 0, st, 1, pdl_enabled(),
                   static_cast<const int8_t*>(k.q), static_cast<const uint8_t*>(k.s),
                   static_cast<float*>(x), rows, C, ckpt_ld(C), chunks, int(vec));
}

// row shares of the column sums: enough CTAs for four per SM, at least 32 rows each
int col_sum_parts(int rows, int C) {
  const long long strips = (C + 255) / 256;
  const long long want = (4ll * kColSumSMs + strips - 1) / strips;
  const long long most = (rows + 31) / 32;
  return static_cast<int>(want < most ? want : most);
}

cudaError_t launch_part_sum(const float* part, float* out, int parts, int C, int accumulate,
                            cudaStream_t st) {
  return launch_ex(k_part_sum, dim3((C + 31) / 32), dim3(kThreads), 0, st, 1, pdl_enabled(), part, out,
                   parts, C, accumulate);
}

cudaError_t launch_col_sum(const void* x, float* out, float* part, int rows, int C, int accumulate,
                           bool bf16, bool vec, cudaStream_t st) {
  int parts = col_sum_parts(rows, C);
  const int per = (rows + parts - 1) / parts;
  parts = (rows + per - 1) / per;
  const dim3 grid((C + 255) / 256, parts);
  const cudaError_t e =
      bf16 ? launch_ex(k_col_sum<uint16_t>, grid, dim3(kThreads), 0, st, 1, pdl_enabled(),
                       static_cast<const uint16_t*>(x), part, rows, C, per, int(vec))
           : launch_ex(k_col_sum<float>, grid, dim3(kThreads), 0, st, 1, pdl_enabled(),
                       static_cast<const float*>(x), part, rows, C, per, int(vec));
  if (e != cudaSuccess) return e;
  return launch_part_sum(part, out, parts, C, accumulate, st);
}

}  // namespace instant
