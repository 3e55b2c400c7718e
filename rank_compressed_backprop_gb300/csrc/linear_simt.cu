// linear_simt.cu -- the three products of an MLP block's linear layers on plain
// FFMA: the fp32 path.
//   forward   z = x w^T + bias, y = act(z) + res, checkpoints of z and y
//   back      gx = (gy w) * act'(z) + res, z from its checkpoint
//   grad_w    gw (+)= (gy^T v) * col_scale, v the checkpoint's values
// A warp owns R rows and 128 columns of the output, each lane the columns lane,
// lane + 32, lane + 64 and lane + 96, so that it holds whole checkpoint groups of its
// rows.  16-deep slices of both operands go through three stages of shared memory
// by asynchronous copies: the operand of rows is read by broadcast (R values a
// step), the one of columns without bank conflicts, and 4 R products a lane follow
// from R + 4 values.  Few tiles leave too few warps on an SM to hide the latency of
// a slice, so K is then split across the CTAs of a cluster: each leaves its partial
// tile in shared memory, and a warp adds a row's partial sums in the order of the
// ranks through distributed shared memory and carries the row through the epilogue.
#include <algorithm>

#include "ckpt.cuh"

namespace instant {

namespace {

constexpr int BN = 128, BK = 16, NS = 3;
constexpr int LDK = BK + 4;   // floats of a staged row of K: eight rows 16 bytes apart cover all banks
enum { FORWARD = 0, BACK = 1, GRAD_W = 2 };

// 16 or 4 bytes global -> shared, asynchronous; zeros where `on` is false
template <int BYTES>
__device__ __forceinline__ void copy_async(float* dst, const float* src, bool on) {
  const int n = on ? BYTES : 0;
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ float dsmem_ld(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// a block of `rows` x `cols` floats at (r0, c0) of a row-major [nr, nc] tensor into
// shared memory with row pitch `ld`; zeros past the tensor's end
template <int ROWS, int COLS, int THREADS, bool VEC>
__device__ __forceinline__ void stage_block(float* dst, int ld, const float* src, int r0, int c0, int nr, int nc) {
  constexpr int W = VEC ? 4 : 1;
  for (int i = threadIdx.x; i < ROWS * COLS / W; i += THREADS) {
    const int r = i / (COLS / W), c = W * (i % (COLS / W));
    const bool on = r0 + r < nr && c0 + c < nc;
    const float* p = on ? src + static_cast<size_t>(r0 + r) * nc + c0 + c : src;
    copy_async<4 * W>(dst + r * ld + c, p, on);
  }
}

// the same transposed, an element a copy
template <int ROWS, int COLS, int THREADS>
__device__ __forceinline__ void stage_transposed(float* dst, int ld, const float* src, int r0, int c0, int nr, int nc) {
  for (int i = threadIdx.x; i < ROWS * COLS; i += THREADS) {
    const int r = i / COLS, c = i % COLS;
    const bool on = r0 + r < nr && c0 + c < nc;
    copy_async<4>(dst + c * ld + r, on ? src + static_cast<size_t>(r0 + r) * nc + c0 + c : src, on);
  }
}

// checkpoint of a row's 128 columns, four in each lane
__device__ __forceinline__ void put_ckpt(const CkptRef& k, int ld, int rows, int row, int n0, int C, const float* v) {
  const int lane = threadIdx.x & 31;
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (n0 + lane + 32 * j < C) m = max(m, abs_bits(v[j]));
  const uint32_t code = ckpt_scale_code(__reduce_max_sync(0xffffffffu, m));
  const float inv = ckpt_inv_scale(code);
  int8_t* q = k.q + static_cast<size_t>(row) * ld + n0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (n0 + lane + 32 * j < C) q[lane + 32 * j] = static_cast<int8_t>(ckpt_code(v[j], inv));
  if (lane == 0) k.s[static_cast<size_t>(n0 / kCkptGroup) * rows + row] = static_cast<uint8_t>(code);
}

// VEC: rows of both operands start on 16-byte boundaries
template <int KIND, int BM, int R, bool VEC>
__global__ void __launch_bounds__(32 * BM / R) k_linear_simt(LinearArgs a, int splits, int per) {
  constexpr int T = 32 * BM / R;
  constexpr bool K_IN = KIND == FORWARD;   // staged [m][k] and [n][k], else [k][m] and [k][n]
  constexpr int LDA = K_IN ? LDK : KIND == BACK ? BM + 4 : BM, LDB = K_IN ? LDK : BN;
  constexpr int A_FLOATS = K_IN ? BM * LDK : BK * LDA, B_FLOATS = K_IN ? BN * LDK : BK * BN;
  __shared__ __align__(16) float buf[NS * (A_FLOATS + B_FLOATS)];
  static_assert(BM * BN <= NS * (A_FLOATS + B_FLOATS), "the partial tile goes over the stages");
  auto As = [&](int s) { return buf + s * A_FLOATS; };
  auto Bs = [&](int s) { return buf + NS * A_FLOATS + s * B_FLOATS; };
  pdl_wait();
  const int nt = (a.N + BN - 1) / BN;
  const int m0 = blockIdx.x / nt * BM;
  const int n0 = blockIdx.x % nt * BN;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float* A = static_cast<const float*>(a.a);
  const float* B = static_cast<const float*>(a.b);

  auto stage = [&](int s, int k0) {
    if (KIND == GRAD_W) stage_block<BK, BM, T, VEC>(As(s), LDA, A, k0, m0, a.K, a.M);
    else if (KIND == BACK) stage_transposed<BM, BK, T>(As(s), LDA, A, m0, k0, a.M, a.K);
    else stage_block<BM, BK, T, VEC>(As(s), LDA, A, m0, k0, a.M, a.K);
    if (KIND == FORWARD) {
      stage_block<BN, BK, T, VEC>(Bs(s), LDB, B, n0, k0, a.N, a.K);
    } else if (KIND == BACK) {
      stage_block<BK, BN, T, VEC>(Bs(s), LDB, B, k0, n0, a.K, a.N);
    } else {
      // eight codes of a token a thread (rows of codes are padded to 16)
      for (int i = threadIdx.x; i < BK * BN / 8; i += T) {
        const int k = i / (BN / 8), c = 8 * (i % (BN / 8));
        const bool on = k0 + k < a.K && n0 + c < a.N;
        uint2 w = make_uint2(0u, 0u);
        float scale = 0.f;
        if (on) {
          w = *reinterpret_cast<const uint2*>(a.ck.q + static_cast<size_t>(k0 + k) * a.ld + n0 + c);
          scale = ckpt_scale(a.ck.s[static_cast<size_t>(n0 / kCkptGroup) * a.K + k0 + k]);
        }
        float2 v[4];
        ckpt_pairs8(w, scale, v);
        float* d = Bs(s) + k * LDB + c;
        *reinterpret_cast<float4*>(d) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
        *reinterpret_cast<float4*>(d + 4) = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
      }
    }
  };

  float2 acc[R / 2][4];  // rows 2 i and 2 i + 1
#pragma unroll
  for (int i = 0; i < R / 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = both(0.f);

  const int rank = blockIdx.z;  // == rank in the cluster (1 x 1 x splits)
  const int k_begin = rank * per * BK;
  const int nk = max(0, min(per, (a.K + BK - 1) / BK - rank * per));
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) {
    if (s < nk) stage(s, k_begin + s * BK);
    cp_async_commit();
  }
  int s = 0;
  for (int kc = 0; kc < nk; ++kc) {
    cp_async_wait<NS - 2>();
    __syncthreads();  // slice kc is there for all, and slot kc + NS - 1 was read by all
    {
      const int next = kc + NS - 1;
      if (next < nk) stage(next % NS, k_begin + next * BK);
      cp_async_commit();
    }
    const float* as = As(s) + warp * R * (K_IN ? LDA : 1);
    const float* bs = Bs(s);
    if (K_IN) {
#pragma unroll
      for (int k = 0; k < BK; k += 4) {
        float4 b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(bs + (lane + 32 * j) * LDB + k);
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float4 x = *reinterpret_cast<const float4*>(as + i * LDA + k);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float& d = i & 1 ? acc[i / 2][j].y : acc[i / 2][j].x;
            d = fmaf(x.w, b[j].w, fmaf(x.z, b[j].z, fmaf(x.y, b[j].y, fmaf(x.x, b[j].x, d))));
          }
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < BK; ++k) {
        float2 b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = both(bs[k * LDB + lane + 32 * j]);
#pragma unroll
        for (int i = 0; i < R; i += 4) {
          const float4 x = *reinterpret_cast<const float4*>(as + k * LDA + i);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[i / 2][j] = fma2(make_float2(x.x, x.y), b[j], acc[i / 2][j]);
            acc[i / 2 + 1][j] = fma2(make_float2(x.z, x.w), b[j], acc[i / 2 + 1][j]);
          }
        }
      }
    }
    if (++s == NS) s = 0;
  }

  // not before: the next launch's CTAs would take their places beside these wherever
  // there is room, and two would share an SM while others stood empty (1024 x 2048 ->
  // 2048 back to back 340 us instead of 286)
  pdl_launch_dependents();

  // partial tile [row][column] over the stages
  cp_async_wait<0>();
  __syncthreads();
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      buf[(warp * R + i) * BN + lane + 32 * j] = i & 1 ? acc[i / 2][j].y : acc[i / 2][j].x;
  if (splits > 1) cluster_sync(); else __syncwarp();  // one CTA: a warp finishes its own rows

  float bias[4];
  bool on[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = n0 + lane + 32 * j;
    on[j] = c < a.N;
    bias[j] = a.bias && on[j] ? static_cast<const float*>(a.bias)[c] : 0.f;  // grad_w: column scale
  }
  const int first = splits > 1 ? rank + splits * warp : warp * R;
  const int step = splits > 1 ? splits * (BM / R) : 1;
  const int last = min(splits > 1 ? BM : warp * R + R, a.M - m0);
#pragma unroll 1
  for (int i = first; i < last; i += step) {
    const int m = m0 + i;
    const size_t base = static_cast<size_t>(m) * a.N + n0 + lane;
    // global operands are asked for before the peers' partial sums
    const bool slopes = KIND == BACK && a.act != INSTANT_ACT_NONE;
    const int8_t* q = a.ck.q + static_cast<size_t>(m) * a.ld + n0 + lane;
    float scale = 0.f, z[4], res[4];
    if (slopes) scale = ckpt_scale(__ldg(a.ck.s + static_cast<size_t>(n0 / kCkptGroup) * a.M + m));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      z[j] = slopes && on[j] ? static_cast<float>(__ldg(q + 32 * j)) : 0.f;
      res[j] = KIND != GRAD_W && a.res && on[j] ? static_cast<const float*>(a.res)[base + 32 * j] : 0.f;
    }
    const float* src = buf + i * BN + lane;
    float v[4];
    if (splits == 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = src[32 * j];
    } else {
      float part[8][4];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < splits) {
          const uint32_t at = dsmem_addr(src, q);
#pragma unroll
          for (int j = 0; j < 4; ++j) part[q][j] = dsmem_ld(at + 128 * j);
        }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = part[0][j];
#pragma unroll
        for (int q = 1; q < 8; ++q)
          if (q < splits) v[j] += part[q][j];
      }
    }
    if (KIND == GRAD_W) {
      float* out = static_cast<float*>(a.out) + base;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (on[j]) {
          const float x = a.bias ? v[j] * bias[j] : v[j];
          out[32 * j] = a.accumulate ? out[32 * j] + x : x;
        }
      continue;
    }
    if (KIND == FORWARD) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += bias[j];
      if (a.zk.q) put_ckpt(a.zk, a.ld, a.M, m, n0, a.N, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = act_f32(v[j], a.act);
    } else if (slopes) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] *= act_slope_f32(z[j] * scale, a.act);
    }
    if (a.res) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += res[j];
    }
    if (KIND == FORWARD && a.yk.q) put_ckpt(a.yk, a.ld, a.M, m, n0, a.N, v);
    if (a.out) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (on[j]) static_cast<float*>(a.out)[base + 32 * j] = v[j];
    }
  }
  if (splits > 1) cluster_sync();  // peers may still read this CTA's tile
}

template <int KIND, int BM, int R>
cudaError_t go(const LinearArgs& a, cudaStream_t st) {
  const long long tiles = static_cast<long long>((a.M + BM - 1) / BM) * ((a.N + BN - 1) / BN);
  if (tiles > 0x7fffffffll) return cudaErrorInvalidValue;
  // 16-byte copies where every row of both operands starts on a 16-byte boundary
  const bool vec = (KIND == GRAD_W ? a.M : a.K) % 4 == 0 &&
                   (KIND == GRAD_W ? true : (KIND == BACK ? a.N : a.K) % 4 == 0);
  // shares of K: about two CTAs an SM, at least four slices each
  const int nk = (a.K + BK - 1) / BK;
  const int want = static_cast<int>(std::min<long long>(8, 2ll * sm_count() / tiles));
  int splits = std::max(1, std::min(want, nk / 4));
  const int per = (nk + splits - 1) / splits;
  splits = (nk + per - 1) / per;
  const dim3 grid(static_cast<unsigned>(tiles), 1, splits), block(32 * BM / R);
  return vec ? launch_ex(k_linear_simt<KIND, BM, R, true>, grid, block, 0, st, splits, pdl_enabled(), a, splits, per)
             : launch_ex(k_linear_simt<KIND, BM, R, false>, grid, block, 0, st, splits, pdl_enabled(), a, splits, per);
}

// row tiles of 64, or of 16 for short batches
template <int KIND>
cudaError_t go_rows(const LinearArgs& a, cudaStream_t st) {
  return a.M > 32 ? go<KIND, 64, 8>(a, st) : go<KIND, 16, 4>(a, st);
}

}  // namespace

cudaError_t launch_linear_simt(const LinearArgs& a, cudaStream_t st) {
  switch (a.kind) {
    case FORWARD: return go_rows<FORWARD>(a, st);
    case BACK: return go_rows<BACK>(a, st);
    default: return go_rows<GRAD_W>(a, st);
  }
}

}  // namespace instant
