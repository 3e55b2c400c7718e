// ckpt.cu -- 8-bit activation checkpoints of tensors that no other kernel
// here produced (pack), their values (unpack), and the column sums of a
// gradient (the bias gradient next to a weight gradient).
//
// All three are bound by HBM: pack reads each element once and writes one byte
// for it, unpack the reverse.  A half warp owns one group of 128 channels, eight
// channels a lane, so that the group's largest magnitude is four shuffles away.
#include <algorithm>

#include "ckpt.cuh"

namespace instant {

namespace {

constexpr int kThreads = 256;

// A CTA takes `gp` neighbouring groups (a power of two up to 16) of 16 / gp rows
// at a time, two such steps under way together, and walks down its rows: no index
// needs a division.  8191 x 11008 bf16: 43 us, 0.92 of the copy rate (four steps, whose
// registers halve the CTAs of an SM, 50; one 49).
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads)
    k_ckpt_pack(const T* __restrict__ x, int8_t* __restrict__ q, uint8_t* __restrict__ s, int rows,
                int C, int ld, int gp, int per) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kUnroll = 2;
  const int hl = threadIdx.x & 15, h = threadIdx.x >> 4;
  const int g = blockIdx.x * gp + (h & (gp - 1));
  const int step = 16 / gp;
  const int c = g * kCkptGroup + 8 * hl;
  const int cc = VEC && c >= C ? 0 : c;
  const int r1 = min(rows, (static_cast<int>(blockIdx.y) + 1) * per);
  // whole warps stay in the loop together: the shuffles name all 32 lanes
  for (int r0 = blockIdx.y * per; r0 < r1; r0 += kUnroll * step) {
    float2 v[kUnroll][4];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      // past the last row the last one again, past the last column the row's first
      // (neither is stored, and the latter does not count for its group)
      const int row = min(r0 + j * step + h / gp, r1 - 1);
      load_pairs<VEC>(x + static_cast<size_t>(row) * C + cc, VEC ? 8 : C - c, v[j]);
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int row = r0 + j * step + h / gp;
      const bool on = row < r1 && c < C;
      const uint32_t code = ckpt_scale_code(half_warp_max(c < C ? max_bits8(v[j]) : 0u));
      const uint2 w = ckpt_code8(v[j], code);
      if (on) {
        *reinterpret_cast<uint2*>(q + static_cast<size_t>(row) * ld + c) = w;
        if (hl == 0) s[static_cast<size_t>(g) * rows + row] = static_cast<uint8_t>(code);
      }
    }
  }
}

// A thread takes eight channels of a row (8 bytes in, 16 out), four rows at once;
// a CTA `cp` neighbouring threads' channels of 256 / cp rows.
template <typename T, bool VEC>
__device__ __forceinline__ void unpack_rows(const int8_t* __restrict__ q, const uint8_t* __restrict__ s,
                                            T* __restrict__ x, int rows, int C, int ld, int cp, int per,
                                            int column, int share) {
  constexpr int kUnroll = 4;
  const int c = 8 * (column * cp + (threadIdx.x & (cp - 1)));
  if (c >= C) return;
  const int step = kThreads / cp;
  const uint8_t* sg = s + static_cast<size_t>(c / kCkptGroup) * rows;
  const int r1 = min(rows, (share + 1) * per);
  for (int r0 = share * per + static_cast<int>(threadIdx.x) / cp; r0 < r1; r0 += kUnroll * step) {
    uint2 w[kUnroll];
    float scale[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int row = r0 + j * step;
      if (row < r1) {
        w[j] = *reinterpret_cast<const uint2*>(q + static_cast<size_t>(row) * ld + c);
        scale[j] = ckpt_scale(sg[row]);
      }
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int row = r0 + j * step;
      if (row >= r1) break;
      float2 v[4];
      ckpt_pairs8(w[j], scale[j], v);
      store_pairs<VEC>(x + static_cast<size_t>(row) * C + c, C - c, v);
    }
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads)
    k_ckpt_unpack(const int8_t* __restrict__ q, const uint8_t* __restrict__ s, T* __restrict__ x,
                  int rows, int C, int ld, int cp, int per) {
  pdl_launch_dependents();
  pdl_wait();
  unpack_rows<T, VEC>(q, s, x, rows, C, ld, cp, per, blockIdx.x, blockIdx.y);
}

// Column sums in two fixed-order stages (no atomics: the same bits on every
// call).  Stage 1: a CTA sums `per` rows of 8 x 32 columns, eight warps taking
// the rows in turn; stage 2 adds the row shares.
template <typename T, bool VEC>
__device__ __forceinline__ void sum_rows(const T* __restrict__ x, float* __restrict__ part, int rows, int C, int per,
                                         int strip, int share) {
  __shared__ float red[8][kThreads];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = strip * 256 + 8 * lane;
  const int r0 = share * per;
  const int r1 = min(rows, r0 + per);
  float2 sum2[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) sum2[e] = both(0.f);
  if (c < C) {
    const T* p = x + static_cast<size_t>(r0 + warp) * C + c;
    const size_t step = 8 * static_cast<size_t>(C);
    // eight rows' loads under way together
    constexpr int kBatch = 8;
    int r = r0 + warp;
    for (; r + 8 * (kBatch - 1) < r1; r += 8 * kBatch, p += kBatch * step) {
      float2 v[kBatch][4];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) load_pairs<VEC>(p + j * step, VEC ? 8 : C - c, v[j]);
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum2[e] = add2(sum2[e], v[j][e]);
    }
    for (; r < r1; r += 8, p += step) {
      float2 v[4];
      load_pairs<VEC>(p, VEC ? 8 : C - c, v);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum2[e] = add2(sum2[e], v[e]);
    }
  }
  const float acc[8] = {sum2[0].x, sum2[0].y, sum2[1].x, sum2[1].y, sum2[2].x, sum2[2].y, sum2[3].x, sum2[3].y};
#pragma unroll
  for (int e = 0; e < 8; ++e) red[warp][8 * lane + e] = acc[e];
  __syncthreads();
  float sum = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) sum += red[w][threadIdx.x];
  const int col = strip * 256 + threadIdx.x;
  if (col < C) part[static_cast<size_t>(share) * C + col] = sum;
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads, 3)
    k_col_sum(const float* __restrict__ x, float* __restrict__ part, int rows, int C, int per) {
  pdl_launch_dependents();
  pdl_wait();
  sum_rows<float, VEC>(x, part, rows, C, per, blockIdx.x, blockIdx.y);
}

// Stage 1 of a bias gradient beside the checkpoint's values for the weight gradient,
// in one launch: the CTAs from `sums` on sum x, the others unpack
__global__ void __launch_bounds__(kThreads, 3)
    k_unpack_and_sum(const int8_t* __restrict__ q, const uint8_t* __restrict__ s, uint16_t* __restrict__ v, int C,
                     int ld, int cp, int per, int columns, const uint16_t* __restrict__ x, float* __restrict__ part,
                     int Cx, int sum_per, int strips, int sums, int rows) {
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.x;
  if (b < sums) unpack_rows<uint16_t, true>(q, s, v, rows, C, ld, cp, per, b % columns, b / columns);
  else sum_rows<uint16_t, true>(x, part, rows, Cx, sum_per, (b - sums) % strips, (b - sums) / strips);
}

// out[c] (+)= sum_p part[p][c]: eight columns a CTA (a 32-byte sector of each
// share), 64 threads of each column take the shares in turn
__global__ void __launch_bounds__(512)
    k_part_sum(const float* __restrict__ part, float* __restrict__ out, int parts, int C,
               int accumulate) {
  __shared__ float red[64][9];
  pdl_launch_dependents();
  pdl_wait();
  const int col = threadIdx.x & 7, row = threadIdx.x >> 3;
  const int c = blockIdx.x * 8 + col;
  float acc = 0.f;
  if (c < C) {
#pragma unroll 8
    for (int p = row; p < parts; p += 64) acc += part[static_cast<size_t>(p) * C + c];
  }
  red[row][col] = acc;
  __syncthreads();
  // warp w adds up column w
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp >= 8) return;
  float sum = red[lane][warp] + red[lane + 32][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const int cw = blockIdx.x * 8 + warp;
  if (lane == 0 && cw < C) out[cw] = accumulate ? out[cw] + sum : sum;
}

// the smallest power of two that is at least n, or `most`
int pow2_up(int n, int most) {
  int p = 1;
  while (p < n && p < most) p *= 2;
  return p;
}

// rows a CTA walks when a column of CTAs shares the rows: about `ctas` CTAs in
// all, a multiple of `pass` rows, and no more than 65535 CTAs a column
int rows_per_cta(int rows, int columns, int pass, int ctas) {
  const long long want = std::max(1ll, static_cast<long long>(ctas) / columns);
  const long long per = std::max((rows + want - 1) / want, (static_cast<long long>(rows) + 65534) / 65535);
  return static_cast<int>((per + pass - 1) / pass * pass);
}

// Sum of the partial products of a weight gradient, in the order of the shares of the
// rows; four columns a thread
__global__ void __launch_bounds__(kThreads)
    k_split_sum(const float* __restrict__ part, float* __restrict__ out, const uint16_t* __restrict__ scale,
                long long n, long long pitch, int N, int splits, int accumulate) {
  pdl_launch_dependents();
  pdl_wait();
  const long long i = 4 * (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x);
  if (i >= n) return;
  float4 v[kMaxSplits];
#pragma unroll
  for (int s = 0; s < kMaxSplits; ++s)
    if (s < splits) v[s] = *reinterpret_cast<const float4*>(part + s * pitch + i);
#pragma unroll
  for (int s = 1; s < kMaxSplits; ++s)
    if (s < splits) {
      v[0].x += v[s].x;
      v[0].y += v[s].y;
      v[0].z += v[s].z;
      v[0].w += v[s].w;
    }
  if (scale) {
    const uint2 w = *reinterpret_cast<const uint2*>(scale + i % N);
    v[0].x *= __uint_as_float(w.x << 16);
    v[0].y *= __uint_as_float(w.x & 0xffff0000u);
    v[0].z *= __uint_as_float(w.y << 16);
    v[0].w *= __uint_as_float(w.y & 0xffff0000u);
  }
  float4* dst = reinterpret_cast<float4*>(out + i);
  if (accumulate) {
    const float4 o = *dst;
    v[0].x += o.x;
    v[0].y += o.y;
    v[0].z += o.z;
    v[0].w += o.w;
  }
  *dst = v[0];
}

}  // namespace

cudaError_t launch_split_sum(const float* part, int splits, float* out, const void* scale, int M, int N,
                             int accumulate, cudaStream_t st) {
  const long long n = static_cast<long long>(M) * N;  // N is a multiple of 8
  const long long pitch = (static_cast<long long>(M) + 255) / 256 * 256 * N;
  const long long ctas = (n / 4 + kThreads - 1) / kThreads;
  if (ctas > 0x7fffffffll || splits > kMaxSplits) return cudaErrorInvalidValue;
  return launch_ex(k_split_sum, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, st, 1, pdl_enabled(), part, out,
                   static_cast<const uint16_t*>(scale), n, pitch, N, splits, accumulate);
}

cudaError_t launch_ckpt_pack(const void* x, const CkptRef& k, int rows, int C, bool bf16, bool vec,
                             cudaStream_t st) {
  const int groups = (C + kCkptGroup - 1) / kCkptGroup;
  const int gp = pow2_up(groups, 16);
  const int columns = (groups + gp - 1) / gp;
  const int per = rows_per_cta(rows, columns, 2 * 16 / gp, 16 * sm_count());
  const dim3 grid(columns, (rows + per - 1) / per);
  auto go = [&](auto kernel, auto* p) {
    return launch_ex(kernel, grid, dim3(kThreads), 0, st, 1, pdl_enabled(), p, k.q, k.s, rows, C, ckpt_ld(C), gp,
                     per);
  };
  if (bf16) return go(k_ckpt_pack<uint16_t, true>, static_cast<const uint16_t*>(x));
  return vec ? go(k_ckpt_pack<float, true>, static_cast<const float*>(x))
             : go(k_ckpt_pack<float, false>, static_cast<const float*>(x));
}

// how the CTAs of an unpacking divide [rows, C]
struct UnpackPlan {
  int cp, columns, per, shares;
  UnpackPlan(int rows, int C) {
    const int chunks = (C + 7) / 8;
    cp = pow2_up(chunks, kThreads);
    columns = (chunks + cp - 1) / cp;
    per = rows_per_cta(rows, columns, 4 * kThreads / cp, 16 * sm_count());
    shares = (rows + per - 1) / per;
  }
};

cudaError_t launch_ckpt_unpack(const CkptRef& k, void* x, int rows, int C, bool bf16, bool vec,
                               cudaStream_t st) {
  const UnpackPlan p(rows, C);
  auto go = [&](auto kernel, auto* dst) {
    return launch_ex(kernel, dim3(p.columns, p.shares), dim3(kThreads), 0, st, 1, pdl_enabled(),
                     static_cast<const int8_t*>(k.q), static_cast<const uint8_t*>(k.s), dst, rows, C, ckpt_ld(C), p.cp,
                     p.per);
  };
  if (bf16) return go(k_ckpt_unpack<uint16_t, true>, static_cast<uint16_t*>(x));
  return vec ? go(k_ckpt_unpack<float, true>, static_cast<float*>(x))
             : go(k_ckpt_unpack<float, false>, static_cast<float*>(x));
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
  return launch_ex(k_part_sum, dim3((C + 7) / 8), dim3(512), 0, st, 1, pdl_enabled(), part, out,
                   parts, C, accumulate);
}

cudaError_t launch_col_sum(const float* x, float* out, float* part, int rows, int C, int accumulate, bool vec,
                           cudaStream_t st) {
  int parts = col_sum_parts(rows, C);
  const int per = (rows + parts - 1) / parts;
  parts = (rows + per - 1) / per;
  const cudaError_t e = launch_ex(vec ? k_col_sum<true> : k_col_sum<false>, dim3((C + 255) / 256, parts),
                                  dim3(kThreads), 0, st, 1, pdl_enabled(), x, part, rows, C, per);
  return e != cudaSuccess ? e : launch_part_sum(part, out, parts, C, accumulate, st);
}

// bf16 values of a checkpoint of [rows, C] and the shares of the column sums of x
// [rows, Cx], whose number it returns; launch_part_sum adds them
cudaError_t launch_unpack_and_sum(const CkptRef& k, void* values, int rows, int C, const void* x, float* part, int Cx,
                                  int* parts, cudaStream_t st) {
  const UnpackPlan p(rows, C);
  const int per = (rows + col_sum_parts(rows, Cx) - 1) / col_sum_parts(rows, Cx);
  *parts = (rows + per - 1) / per;
  const int strips = (Cx + 255) / 256;
  const long long unpacks = static_cast<long long>(p.columns) * p.shares;
  const long long all = unpacks + static_cast<long long>(strips) * *parts;
  if (all > 0x7fffffffll) return cudaErrorInvalidValue;
  return launch_ex(k_unpack_and_sum, dim3(static_cast<unsigned>(all)), dim3(kThreads), 0, st, 1, pdl_enabled(),
                   static_cast<const int8_t*>(k.q), static_cast<const uint8_t*>(k.s), static_cast<uint16_t*>(values), C,
                   ckpt_ld(C), p.cp, p.per, p.columns, static_cast<const uint16_t*>(x), part, Cx, per, strips,
                   static_cast<int>(unpacks), rows);
}

}  // namespace instant
