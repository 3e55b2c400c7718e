// linear_simt.cu -- the three products of an MLP block's linear layers on plain
// FFMA: the fp32 path.
//   forward   z = x w^T + bias, y = act(z) + res, checkpoints of z and y
//   back      gx = (gy w) * act'(z) + res, z from its checkpoint
//   grad_w    gw (+)= (gy^T v) * col_scale, v the checkpoint's values
// One kernel: a 64 x 128 output tile, 16-deep slices of both operands staged in
// shared memory, 4 x 8 outputs a thread.  A tile is 128 columns wide so that the
// 16 threads of a half warp hold whole checkpoint groups of their rows.
#include "ckpt.cuh"

namespace instant {

namespace {

constexpr int BM = 64, BN = 128, BK = 16;
constexpr int kThreads = 256;
enum { FORWARD = 0, BACK = 1, GRAD_W = 2 };

// checkpoint of a row's 128 columns, eight in each lane of a half warp: four at
// c0 and four at c1
__device__ __forceinline__ void put_ckpt(const CkptRef& k, int ld, int rows, int row, bool on, int c0,
                                         int c1, int C, const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (c0 + e < C) m = max(m, abs_bits(v[e]));
    if (c1 + e < C) m = max(m, abs_bits(v[4 + e]));
  }
  const uint32_t code = ckpt_scale_code(half_warp_max(m));
  const float inv = ckpt_inv_scale(code);
  if (!on) return;
  int8_t* q = k.q + static_cast<size_t>(row) * ld;
  if (c0 < C) *reinterpret_cast<uint32_t*>(q + c0) = ckpt_code4(v[0], v[1], v[2], v[3], inv);
  if (c1 < C) *reinterpret_cast<uint32_t*>(q + c1) = ckpt_code4(v[4], v[5], v[6], v[7], inv);
  if ((threadIdx.x & 15) == 0 && c0 < C)
    k.s[static_cast<size_t>(c0 / kCkptGroup) * rows + row] = static_cast<uint8_t>(code);
}

template <typename T, int KIND>
__global__ void __launch_bounds__(kThreads) k_linear_simt(LinearArgs a) {
  __shared__ float As[BK][BM + 4];
  __shared__ float Bs[BK][BN + 4];
  pdl_launch_dependents();
  pdl_wait();
  const int nt = (a.N + BN - 1) / BN;
  const int m0 = blockIdx.x / nt * BM;
  const int n0 = blockIdx.x % nt * BN;
  const int tid = threadIdx.x;
  const int tx = tid & 15, ty = tid >> 4;
  const T* A = static_cast<const T*>(a.a);
  const T* B = static_cast<const T*>(a.b);
  float acc[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;

  float ra[4], rb[8];
  auto fetch = [&](int k0) {
    if (KIND == GRAD_W) {  // gy [K, M]
      const int k = k0 + (tid >> 4), m = m0 + 4 * (tid & 15);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        ra[e] = k < a.K && m + e < a.M ? elem_to_f<T>(A[static_cast<size_t>(k) * a.M + m + e]) : 0.f;
    } else {               // x or gy [M, K]
      const int m = m0 + (tid >> 2), k = k0 + 4 * (tid & 3);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        ra[e] = m < a.M && k + e < a.K ? elem_to_f<T>(A[static_cast<size_t>(m) * a.K + k + e]) : 0.f;
    }
    if (KIND == FORWARD) {  // w [N, K]
      const int n = n0 + (tid >> 1), k = k0 + 8 * (tid & 1);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        rb[e] = n < a.N && k + e < a.K ? elem_to_f<T>(B[static_cast<size_t>(n) * a.K + k + e]) : 0.f;
    } else if (KIND == BACK) {  // w [K, N]
      const int k = k0 + (tid >> 4), n = n0 + 8 * (tid & 15);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        rb[e] = k < a.K && n + e < a.N ? elem_to_f<T>(B[static_cast<size_t>(k) * a.N + n + e]) : 0.f;
    } else {                // codes [K, ld]
      const int k = k0 + (tid >> 4), n = n0 + 8 * (tid & 15);
      const bool on = k < a.K && n < a.N;
      uint2 w = make_uint2(0u, 0u);
      float scale = 0.f;
      if (on) {
        w = *reinterpret_cast<const uint2*>(a.ck.q + static_cast<size_t>(k) * a.ld + n);
        scale = ckpt_scale(a.ck.s[static_cast<size_t>(n / kCkptGroup) * a.K + k]);
      }
      ckpt_values4(w.x, scale, rb);
      ckpt_values4(w.y, scale, rb + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n + e >= a.N) rb[e] = 0.f;  // padding codes are not defined
    }
  };
  auto stage = [&]() {
    if (KIND == GRAD_W) {
#pragma unroll
      for (int e = 0; e < 4; ++e) As[tid >> 4][4 * (tid & 15) + e] = ra[e];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) As[4 * (tid & 3) + e][tid >> 2] = ra[e];
    }
    if (KIND == FORWARD) {
#pragma unroll
      for (int e = 0; e < 8; ++e) Bs[8 * (tid & 1) + e][tid >> 1] = rb[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) Bs[tid >> 4][8 * (tid & 15) + e] = rb[e];
    }
  };

  fetch(0);
  for (int k0 = 0; k0 < a.K; k0 += BK) {
    __syncthreads();
    stage();
    __syncthreads();
    if (k0 + BK < a.K) fetch(k0 + BK);  // in flight over the products of this slice
#pragma unroll
    for (int k = 0; k < BK; ++k) {
      const float4 av = *reinterpret_cast<const float4*>(&As[k][4 * ty]);
      const float4 b0 = *reinterpret_cast<const float4*>(&Bs[k][4 * tx]);
      const float4 b1 = *reinterpret_cast<const float4*>(&Bs[k][64 + 4 * tx]);
      const float am[4] = {av.x, av.y, av.z, av.w};
      const float bn[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(am[i], bn[j], acc[i][j]);
    }
  }

  const int c0 = n0 + 4 * tx, c1 = c0 + 64;
  const bool vec = a.vec;
  float bias[8];
  if (KIND != BACK && a.bias) {  // forward: bias; grad_w: column scale
    load_part<4>(static_cast<const T*>(a.bias) + c0, a.N - c0, vec, bias);
    load_part<4>(static_cast<const T*>(a.bias) + c1, a.N - c1, vec, bias + 4);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + 4 * ty + i;
    const bool on = m < a.M;
    const size_t base = static_cast<size_t>(on ? m : 0) * a.N;
    const int n_0 = on ? a.N - c0 : 0, n_1 = on ? a.N - c1 : 0;
    float* v = acc[i];
    if (KIND == GRAD_W) {
      float* out = static_cast<float*>(a.out) + base;
      if (a.bias) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= bias[j];
      }
      if (a.accumulate) {
        float o[8];
        load_part<4>(out + c0, n_0, vec, o);
        load_part<4>(out + c1, n_1, vec, o + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += o[j];
      }
      store_part<4>(out + c0, n_0, vec, v);
      store_part<4>(out + c1, n_1, vec, v + 4);
      continue;
    }
    if (KIND == FORWARD) {
      if (a.bias) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += bias[j];
      }
      if (a.zk.q) put_ckpt(a.zk, a.ld, a.M, m, on, c0, c1, a.N, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = act_f32(v[j], a.act);
    } else if (a.act != INSTANT_ACT_NONE) {
      uint32_t w0 = 0, w1 = 0;
      float scale = 0.f;
      if (on && c0 < a.N) {
        const int8_t* q = a.ck.q + static_cast<size_t>(m) * a.ld;
        w0 = *reinterpret_cast<const uint32_t*>(q + c0);
        if (c1 < a.N) w1 = *reinterpret_cast<const uint32_t*>(q + c1);
        scale = ckpt_scale(a.ck.s[static_cast<size_t>(c0 / kCkptGroup) * a.M + m]);
      }
      float z[8];
      ckpt_values4(w0, scale, z);
      ckpt_values4(w1, scale, z + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= act_slope_f32(z[j], a.act);
    }
    if (a.res) {
      float o[8];
      load_part<4>(static_cast<const T*>(a.res) + base + c0, n_0, vec, o);
      load_part<4>(static_cast<const T*>(a.res) + base + c1, n_1, vec, o + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += o[j];
    }
    if (KIND == FORWARD && a.yk.q) put_ckpt(a.yk, a.ld, a.M, m, on, c0, c1, a.N, v);
    if (a.out) {
      T* out = static_cast<T*>(a.out) + base;
      store_part<4>(out + c0, n_0, vec, v);
      store_part<4>(out + c1, n_1, vec, v + 4);
    }
  }
}

template <typename T, int KIND>
cudaError_t go(const LinearArgs& a, cudaStream_t st) {
  const long long tiles = static_cast<long long>((a.M + BM - 1) / BM) * ((a.N + BN - 1) / BN);
  if (tiles > 0x7fffffffll) return cudaErrorInvalidValue;
  return launch_ex(k_linear_simt<T, KIND>, dim3(static_cast<unsigned>(tiles)), dim3(kThreads), 0, st, 1,
                   pdl_enabled(), a);
}

}  // namespace

cudaError_t launch_linear_simt(const LinearArgs& a, bool bf16, cudaStream_t st) {
  switch (a.kind) {
    case FORWARD: return bf16 ? go<uint16_t, FORWARD>(a, st) : go<float, FORWARD>(a, st);
    case BACK: return bf16 ? go<uint16_t, BACK>(a, st) : go<float, BACK>(a, st);
    default: return bf16 ? go<uint16_t, GRAD_W>(a, st) : go<float, GRAD_W>(a, st);
  }
}

}  // namespace instant
