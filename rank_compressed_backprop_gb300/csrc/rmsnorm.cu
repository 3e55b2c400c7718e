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
// takes several rows at a time when rows are short.  Sixteen neighbouring lanes
// hold one checkpoint group.
//
// The forward, and the backward of few or unaligned rows, start a CTA for a
// handful of rows.  The streaming backward keeps CTAs on the SMs; a thread of each
// copies blocks of whole rows (they are contiguous) into a ring in shared memory
// with bulk copies, so that an SM has up to 200 KB under way whatever its warps
// wait for, and the share of ggamma stays in registers over all rows of a CTA.
#include <algorithm>

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

// a row's outputs from its unnormalised values (all threads of the row; h is
// spent); gamma(v, g) gives the thread's vector v of gamma
template <typename T, int W, int V, bool VEC, typename Gamma>
__device__ __forceinline__ void norm_outputs(const NormArgs& a, float2 (&h)[V][4], float r, int row, int t,
                                             Gamma gamma) {
  const size_t base = static_cast<size_t>(row) * a.C;
  if (a.r && t == 0) a.r[row] = r;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = 8 * (v * 32 * W + t);
    const int n = a.C - c;
    if (a.h) store_pairs<VEC>(static_cast<T*>(a.h) + base + c, n, h[v]);
#pragma unroll
    for (int e = 0; e < 4; ++e) h[v][e] = mul2(h[v][e], both(r));
    if (a.k.q) {
      const uint32_t code = group_code(h[v]);
      const uint2 w = ckpt_code8(h[v], code);
      if (n > 0) {
        *reinterpret_cast<uint2*>(a.k.q + static_cast<size_t>(row) * a.ld + c) = w;
        if ((threadIdx.x & 15) == 0)
          a.k.s[static_cast<size_t>(c / kCkptGroup) * a.rows + row] = static_cast<uint8_t>(code);
      }
    }
    if (a.y) {
      float2 g[4];
      gamma(v, g);
#pragma unroll
      for (int e = 0; e < 4; ++e) g[e] = mul2(g[e], h[v][e]);
      store_pairs<VEC>(static_cast<T*>(a.y) + base + c, n, g);
    }
  }
}

// adds a vector's squares to ss
__device__ __forceinline__ void add_squares(const float2* h, float2& ss) {
#pragma unroll
  for (int e = 0; e < 4; ++e) ss = fma2(h[e], h[e], ss);
}

template <typename T, int W, int V, bool VEC>
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
  float2 h[V][4];
  float2 ss = both(0.f);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = 8 * (v * 32 * W + t);
    load_pairs<VEC>(x + c, on ? a.C - c : 0, h[v]);
    if (res) {
      float2 o[4];
      load_pairs<VEC>(res + c, on ? a.C - c : 0, o);
#pragma unroll
      for (int e = 0; e < 4; ++e) h[v][e] = add2(h[v][e], o[e]);
    }
    add_squares(h[v], ss);
  }
  // correctly rounded: an error of r shifts the whole row, and codes near the middle of two flip
  const float r = __frsqrt_rn(row_sum<W>(ss.x + ss.y, red, warp) / static_cast<float>(a.C) + a.eps);
  if (!on) return;  // a whole warp at a time
  norm_outputs<T, W, V, VEC>(a, h, r, row, t, [&](int v, float2* g) {
    const int c = 8 * (v * 32 * W + t);
    load_pairs<VEC>(static_cast<const T*>(a.gamma) + c, a.C - c, g);
  });
}

// one vector of the backward: u from its codes, the share of ggamma, d = gy gamma
// (in place of gy) and the share of the row's dot product.  n channels exist; the
// codes past them are not defined
template <bool VEC>
__device__ __forceinline__ void back_vector(uint2 w, float scale, int n, const float2* gamma, float2* d,
                                            float2* u, float2* acc, float2& dot) {
  ckpt_pairs8(w, scale, u);
  if (!VEC && n < 8) {
    float* f = reinterpret_cast<float*>(u);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e >= n) f[e] = 0.f;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    acc[e] = fma2(d[e], u[e], acc[e]);
    d[e] = mul2(d[e], gamma[e]);
    dot = fma2(d[e], u[e], dot);
  }
}

// r (d - u c) in place of d
__device__ __forceinline__ void back_result(float r, float c, const float2* u, float2* d) {
#pragma unroll
  for (int e = 0; e < 4; ++e) d[e] = mul2(both(r), fma2(u[e], both(-c), d[e]));
}

// Rows go round the CTAs; a thread keeps its columns' share of ggamma in
// registers over all its rows, the CTA's row slots add theirs in shared memory
// at the end, and a second kernel adds the CTAs' shares in a fixed order.
template <typename T, int W, int V, bool VEC>
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
  float2 acc[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[v][e] = both(0.f);
  const float inv_c = 1.f / static_cast<float>(a.C);
  int it = 0;
  for (int row0 = blockIdx.x * kRows; row0 < a.rows; row0 += gridDim.x * kRows, ++it) {
    const int row = row0 + slot;
    const bool on = row < a.rows;
    const size_t base = static_cast<size_t>(on ? row : 0) * a.C;
    const float r = on ? a.r[row] : 0.f;
    float2 u[V][4], d[V][4];
    float2 dot = both(0.f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 8 * (v * 32 * W + t);
      const int n = on ? a.C - c : 0;
      float2 gm[4];
      load_pairs<VEC>(static_cast<const T*>(a.gy) + base + c, n, d[v]);
      load_pairs<VEC>(static_cast<const T*>(a.gamma) + c, n, gm);
      uint2 w = make_uint2(0u, 0u);
      float scale = 0.f;
      if (n > 0) {
        w = *reinterpret_cast<const uint2*>(a.k.q + static_cast<size_t>(row) * a.ld + c);
        scale = ckpt_scale(a.k.s[static_cast<size_t>(c / kCkptGroup) * a.rows + row]);
      }
      back_vector<VEC>(w, scale, n, gm, d[v], u[v], acc[v], dot);
    }
    const float c1 = row_sum<W>(dot.x + dot.y, red[it & 1], warp) * inv_c;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 8 * (v * 32 * W + t);
      const int n = on ? a.C - c : 0;
      back_result(r, c1, u[v], d[v]);
      if (a.res) {
        float2 o[4];
        load_pairs<VEC>(static_cast<const T*>(a.res) + base + c, n, o);
#pragma unroll
        for (int e = 0; e < 4; ++e) d[v][e] = add2(d[v][e], o[e]);
      }
      store_pairs<VEC>(static_cast<T*>(a.gx) + base + c, n, d[v]);
    }
  }
  if (kRows > 1) {
    // the row slots' sums, slot 0 first
    for (int s = 0; s < kRows; ++s) {
      if (slot == s) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2* p = reinterpret_cast<float2*>(gsum + 8 * (v * 32 * W + t)) + e;
            *p = s == 0 ? acc[v][e] : add2(*p, acc[v][e]);
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
      store_pairs<VEC>(p, a.C - c, acc[v]);
    }
  }
}

// how a streaming CTA walks the rows: blocks of `block` whole rows, `stages` of
// them in its ring
struct StreamPlan {
  int block, blocks, stages, grid;
  int per_cta, chunk;                   // blocks of a CTA, rows whose factors and scales it holds
  uint32_t res_off, q_off;              // within a slot
  uint32_t stage_bytes, gamma_off, r_off, s_off, bar_off;
  size_t smem;
};

// ---------------------------------------------------------------------------
// streaming form
// ---------------------------------------------------------------------------
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// barrier of the W warps that share a row, which are row slot `slot` of eight warps
// (ids in the instructions: one in a register would reserve all of them)
template <int W>
__device__ __forceinline__ void row_barrier(int slot) {
  if (W >= 8 || slot == 0) named_barrier<2>(32 * W);
  else if (slot == 1) named_barrier<3>(32 * W);
  else if (slot == 2) named_barrier<4>(32 * W);
  else named_barrier<5>(32 * W);
}

// sum over the W warps of a row; `red` is a buffer of 32 floats, another one at
// the next call
template <int W>
__device__ __forceinline__ float row_sum_stream(float v, float* red, int warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (W == 1) return v;
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  row_barrier<W>(warp / W);
  const float* p = red + warp / W * W;
  if (W == 2) return p[0] + p[1];
  float4 sum = *reinterpret_cast<const float4*>(p);
#pragma unroll
  for (int i = 4; i < W; i += 4) {
    const float4 q = *reinterpret_cast<const float4*>(p + i);
    sum.x += q.x; sum.y += q.y; sum.z += q.z; sum.w += q.w;
  }
  return (sum.x + sum.y) + (sum.z + sum.w);
}

// The copies of a CTA's blocks lo .. hi - 1 into the ring, one thread.  A slot
// holds a block of rows: gy, residual, codes.
template <typename T>
__device__ __forceinline__ void produce(const NormBackArgs& a, const StreamPlan& p, uint8_t* ring,
                                        uint64_t* full, uint64_t* empty, int lo, int hi) {
  const uint32_t row_bytes = static_cast<uint32_t>(a.C * sizeof(T));
  int s = 0, par = 1, issued = 0;
  for (int b = lo; b < hi; ++b) {
    if (!mbar_wait(&empty[s], par)) {
      raise_fault(FAULT_WAIT_EMPTY);
      break;
    }
    const int row0 = b * p.block;
    const int n = min(p.block, a.rows - row0);
    uint8_t* dst = ring + static_cast<size_t>(s) * p.stage_bytes;
    mbar_arrive_expect_tx(&full[s], n * (row_bytes * (a.res ? 2 : 1) + a.ld));
    const size_t off = static_cast<size_t>(row0) * row_bytes;
    bulk_load(dst, static_cast<const uint8_t*>(a.gy) + off, n * row_bytes, &full[s]);
    if (a.res) bulk_load(dst + p.res_off, static_cast<const uint8_t*>(a.res) + off, n * row_bytes, &full[s]);
    bulk_load(dst + p.q_off, a.k.q + static_cast<size_t>(row0) * a.ld, n * a.ld, &full[s]);
    if (issued < p.stages) ++issued;
    if (++s == p.stages) {
      s = 0;
      par ^= 1;
    }
  }
  // the last copies have landed before the CTA goes
  par ^= 1;
  for (; issued > 0; --issued) {
    if (--s < 0) {
      s = p.stages - 1;
      par ^= 1;
    }
    if (!mbar_wait(&full[s], par)) raise_fault(FAULT_WAIT_FULL);
  }
}

// Streaming backward.  A CTA's rows are neighbours: their factors and scale bytes are
// fetched for `chunk` rows at once, and the copies start when the first chunk is there
// (a plain load waits behind the copies that are under way: 5 us).  A row's two passes
// read the ring, or what the registers hold.  The warps of a row meet at a barrier of
// their own.  Beyond the bytes' floor it takes about 10 us whatever the size: 3 for the
// second kernel, the rest launch, first loads and copies, and the sums at the end.
//
// What a consumer thread keeps in registers: its columns' shares of ggamma, gamma too,
// or the row's values too between its two passes
enum { HOLD_SUMS, HOLD_GAMMA, HOLD_ROW };

template <typename T, int W, int V, int CTAS, int HOLD>
__global__ void __launch_bounds__((W > 8 ? 32 * W : 256) + 32, CTAS)
    k_rms_norm_back_stream(NormBackArgs a, StreamPlan p) {
  constexpr int kWarps = W > 8 ? W : 8;
  constexpr int kSlots = kWarps / W;  // rows at a time
  constexpr int kCons = 32 * kWarps;  // consumer threads; one more warp produces
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float red[2][32];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.bar_off);
  uint64_t* empty = full + p.stages;
  T* gamma = reinterpret_cast<T*>(smem + p.gamma_off);
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    fence_barrier_init();
  }
  pdl_launch_dependents();
  __syncthreads();
  pdl_wait();
  const int warp = threadIdx.x >> 5;
  const int lo = min(p.blocks, static_cast<int>(blockIdx.x) * p.per_cta);
  const int hi = min(p.blocks, lo + p.per_cta);
  if (warp == kWarps) {
    if (lo < hi) named_barrier<6>(kCons + 32);  // the first chunk is there
    if ((threadIdx.x & 31) == 0) produce<T>(a, p, smem, full, empty, lo, hi);
    return;
  }
  const int t = threadIdx.x % (32 * W);  // thread within its row
  const int slot = warp / W;
  const float inv_c = 1.f / static_cast<float>(a.C);
  float2 acc[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[v][e] = both(0.f);
  int col[V];  // this thread's columns, and whether they exist
  bool in[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = 8 * (v * 32 * W + t);
    in[v] = c < a.C;
    col[v] = in[v] ? c : 0;
  }
  constexpr bool kGamma = HOLD != HOLD_SUMS, kHold = HOLD == HOLD_ROW;
  float2 gm[kGamma ? V : 1][4];
  if (kGamma) {
#pragma unroll
    for (int v = 0; v < V; ++v) load_pairs<true>(static_cast<const T*>(a.gamma) + col[v], 8, gm[v]);
  } else {  // into shared memory; the first chunk's barrier makes it visible
    for (int c = 8 * threadIdx.x; c < a.C; c += 8 * kCons) {
      float2 g[4];
      load_pairs<true>(static_cast<const T*>(a.gamma) + c, 8, g);
      store_pairs<true>(gamma + c, 8, g);
    }
  }
  int s = 0, par = 0, it = 0;
  bool ok = true;  // after a wait that ran out no more are made: the loops stay in step
  float* sr = reinterpret_cast<float*>(smem + p.r_off);  // factors of the chunk's rows
  uint8_t* ssc = smem + p.s_off;                         // scale bytes, [group][chunk]
  const int groups = (a.C + kCkptGroup - 1) / kCkptGroup;
  int chunk0 = lo * p.block;                             // first row of the chunk
  for (int b = lo; b < hi; ++b) {
    if (b == lo || b * p.block - chunk0 >= p.chunk) {
      if (b != lo) named_barrier<1>(kCons);
      chunk0 = b * p.block;
      const int n = min(p.chunk, min(a.rows, hi * p.block) - chunk0);
      for (int i = threadIdx.x; i < n; i += kCons) sr[i] = a.r[chunk0 + i];
      for (int g = warp; g < groups; g += kWarps)
        for (int i = threadIdx.x & 31; i < n; i += 32)
          ssc[g * p.chunk + i] = a.k.s[static_cast<size_t>(g) * a.rows + chunk0 + i];
      if (b == lo) named_barrier<6>(kCons + 32);
      else named_barrier<1>(kCons);
    }
    if (ok && !mbar_wait(&full[s], par)) {
      raise_fault(FAULT_WAIT_FULL);
      ok = false;
    }
    const uint8_t* base = smem + static_cast<size_t>(s) * p.stage_bytes;
    const T* sgy = reinterpret_cast<const T*>(base);
    const T* sres = reinterpret_cast<const T*>(base + p.res_off);
    const int8_t* sq = reinterpret_cast<const int8_t*>(base + p.q_off);
    const int row0 = b * p.block;
    const int in_chunk = row0 - chunk0;
    const int n_rows = min(p.block, a.rows - row0);
    for (int i0 = 0; i0 < n_rows; i0 += kSlots, ++it) {
      const int i = i0 + slot;
      const bool on = i < n_rows;  // the same for all warps of a row
      const T* gyr = sgy + i * a.C;
      const int8_t* qr = sq + i * a.ld;
      // a vector past the row's end repeats its first one with a scale of zero
      // (columns that are never written, terms of zero in the row's sum)
      float2 dot = both(0.f);
      float2 gy[kHold ? V : 1][4], q[kHold ? V : 1][4];
      float scale[kHold ? V : 1];
      auto fetch = [&](int v, int at) {
        scale[at] = in[v] ? ckpt_scale(ssc[(col[v] / kCkptGroup) * p.chunk + in_chunk + i]) : 0.f;
        load_pairs<true>(gyr + col[v], 8, gy[at]);
        code_pairs(*reinterpret_cast<const uint2*>(qr + col[v]), q[at]);
        if (!kGamma) load_pairs<true>(gamma + col[v], 8, gm[0]);
      };
      if (on) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int h = kHold ? v : 0;
          fetch(v, h);
          float2 part = both(0.f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = mul2(gy[h][e], q[h][e]);
            acc[v][e] = fma2(x, both(scale[h]), acc[v][e]);
            part = fma2(x, gm[kGamma ? v : 0][e], part);
          }
          dot = fma2(part, both(scale[h]), dot);
        }
      }
      const float c1 = row_sum_stream<W>(dot.x + dot.y, red[it & 1], warp) * -inv_c;
      if (on) {
        const float r = sr[in_chunk + i];
        const T* resr = sres + i * a.C;
        T* gxr = static_cast<T*>(a.gx) + static_cast<size_t>(row0 + i) * a.C;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          // r (gy gamma - u c) + residual
          const int h = kHold ? v : 0;
          if (!kHold) fetch(v, 0);
          const float2 uc = both(scale[h] * c1);
          float2 d[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) d[e] = fma2(q[h][e], uc, mul2(gy[h][e], gm[kGamma ? v : 0][e]));
          if (a.res) {
            float2 o[4];
            load_pairs<true>(resr + col[v], 8, o);
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = fma2(d[e], both(r), o[e]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = mul2(d[e], both(r));
          }
          store_pairs<true>(gxr + col[v], in[v] ? 8 : 0, d);
        }
      }
    }
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[s]);
    if (++s == p.stages) {
      s = 0;
      par ^= 1;
    }
  }
  // this CTA's share of ggamma: the row slots' sums, slot 0 first, over the ring
  // (every copy has been waited for and read)
  named_barrier<1>(kCons);
  float* gsum = reinterpret_cast<float*>(smem);
  for (int k = 0; k < kSlots; ++k) {
    if (slot == k) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float2* q = reinterpret_cast<float2*>(gsum + 8 * (v * 32 * W + t)) + e;
          *q = k == 0 ? acc[v][e] : add2(*q, acc[v][e]);
        }
    }
    named_barrier<1>(kCons);
  }
  for (int c = threadIdx.x; c < a.C; c += kCons) a.part[static_cast<size_t>(blockIdx.x) * a.C + c] = gsum[c];
}

// direct forms, warps a row and vectors a thread: two vectors a thread up to 16
// warps, then more vectors (1024 x 2 at 11008 channels took 181 us over 8191 rows,
// 512 x 3 139)
#define INSTANT_NORM_DISPATCH(C, GO)                     \
  do {                                                   \
    if ((C) <= 256) GO(1, 1);                            \
    if ((C) <= 512) GO(1, 2);                            \
    if ((C) <= 1024) GO(2, 2);                           \
    if ((C) <= 2048) GO(4, 2);                           \
    if ((C) <= 4096) GO(8, 2);                           \
    if ((C) <= 8192) GO(16, 2);                          \
    if ((C) <= 12288) GO(16, 3);                         \
    if ((C) <= 16384) GO(16, 4);                         \
    GO(32, 4);                                           \
  } while (0)

// Streaming backward: warps a row, vectors a thread, CTAs an SM, what a thread holds.
// Whatever the registers hold a thread needs no second time from the ring, but a
// spilled register waits behind the copies like any plain load: with the row held at
// 8192 x 4096 (spills) 131 us instead of 46, gamma held at 8191 x 11008 291 instead of
// 113.  Three CTAs an SM, whose registers hold only the sums, took 49 us at
// 8192 x 4096, 29 instead of 27.5 at 16384 x 1024 and 21.6 instead of 18.7 at
// 12544 x 448 fp32.
#define INSTANT_STREAM_DISPATCH(C, GO)                   \
  do {                                                   \
    if ((C) <= 256) GO(1, 1, 2, HOLD_ROW);               \
    if ((C) <= 512) GO(2, 1, 2, HOLD_ROW);               \
    if ((C) <= 1024) GO(4, 1, 2, HOLD_ROW);              \
    if ((C) <= 2048) GO(8, 1, 2, HOLD_ROW);              \
    if ((C) <= 4096) GO(8, 2, 2, HOLD_GAMMA);            \
    if ((C) <= 8192) GO(16, 2, 1, HOLD_GAMMA);           \
    GO(16, 3, 1, HOLD_SUMS);                             \
  } while (0)

// Streaming plan; false where the direct form runs: rows too wide for a ring of
// two, or fewer blocks than CTAs (us, streaming / direct, bf16: 8192 x 4096 45.8 / 95.3,
// 8191 x 11008 113 / 272, 16384 x 768 26.4 / 43, 1000 x 1024 6.8 / 7.6, 300 x 8192
// 10.4 / 13.6; 8192 x 64 7.4 / 6.3).  A slot holds about 16 KB, the CTAs of an SM about
// 220 KB.
bool stream_plan(StreamPlan& p, const NormBackArgs& a, size_t elem, int w, int v, int ctas, int most_ctas) {
  const int slots = w > 8 ? 1 : 8 / w;
  const int groups = (a.C + kCkptGroup - 1) / kCkptGroup;
  const size_t row = elem * a.C;
  const size_t pass = slots * (row * (a.res ? 2 : 1) + a.ld);
  const size_t passes = pass >= 16384 ? 1 : std::min<size_t>(8, 16384 / pass);
  p.block = static_cast<int>(slots * passes);
  p.blocks = (a.rows + p.block - 1) / p.block;
  const int full = ctas * std::min(sm_count(), kColSumSMs);
  if (p.blocks < most_ctas * sm_count()) return false;
  p.grid = std::min(full, norm_back_parts(a.rows, a.C));  // the workspace's shares
  p.per_cta = (p.blocks + p.grid - 1) / p.grid;
  p.grid = (p.blocks + p.per_cta - 1) / p.per_cta;
  // about 4 KB of factors and scales
  p.chunk = std::min(p.per_cta, std::max(1, 4096 / (groups + 4) / p.block)) * p.block;
  size_t at = p.block * row;
  p.res_off = static_cast<uint32_t>(at);
  if (a.res) at += p.block * row;
  p.q_off = static_cast<uint32_t>(at);
  at += static_cast<size_t>(p.block) * a.ld;
  const size_t stage = (at + 127) / 128 * 128;
  const size_t gamma = (row + 127) / 128 * 128;
  const size_t rest = gamma + (static_cast<size_t>(p.chunk) * (4 + groups) + 127) / 128 * 128 + 256;
  const size_t room = 220 * 1024 / ctas - 1024;
  if (rest + 2 * stage > room) return false;
  p.stage_bytes = static_cast<uint32_t>(stage);
  p.stages = static_cast<int>(std::min<size_t>(8, (room - rest) / stage));
  // the ring is also the place of a CTA's column sums
  const size_t ring = std::max<size_t>(p.stages * stage, sizeof(float) * 256 * w * v);
  p.gamma_off = static_cast<uint32_t>(ring);
  p.r_off = static_cast<uint32_t>(ring + gamma);
  p.s_off = static_cast<uint32_t>(p.r_off + 4 * p.chunk);
  p.bar_off = static_cast<uint32_t>(ring + rest - 256);
  p.smem = ring + rest;
  return p.smem <= room;
}

template <typename T, int W, int V, int CTAS, int HOLD>
cudaError_t back_stream_go(const NormBackArgs& a, bool* done, cudaStream_t st) {
  StreamPlan p;
  *done = false;
  for (int ctas = CTAS; ctas >= 1 && !*done; --ctas)  // fewer CTAs an SM have wider rings
    *done = stream_plan(p, a, sizeof(T), W, V, ctas, CTAS);
  if (!*done) return cudaSuccess;
  auto k = k_rms_norm_back_stream<T, W, V, CTAS, HOLD>;
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(k), p.smem, true);
  if (e == cudaSuccess)
    e = launch_ex(k, dim3(p.grid), dim3((W > 8 ? 32 * W : 256) + 32), p.smem, st, 1, pdl_enabled(), a, p);
  if (e != cudaSuccess) return e;
  return launch_part_sum(a.part, a.ggamma, p.grid, a.C, a.accumulate, st);
}

template <typename T>
cudaError_t back_stream_dispatch(const NormBackArgs& a, bool* done, cudaStream_t st) {
#define GO(W, V, CTAS, HOLD) return back_stream_go<T, W, V, CTAS, HOLD>(a, done, st)
  INSTANT_STREAM_DISPATCH(a.C, GO);
#undef GO
}

template <typename T, bool VEC, int W, int V>
cudaError_t norm_go(const NormArgs& a, cudaStream_t st) {
  constexpr int kWarps = W > 8 ? W : 8;
  constexpr int kRows = kWarps / W;
  return launch_ex(k_rms_norm<T, W, V, VEC>, dim3((a.rows + kRows - 1) / kRows), dim3(32 * kWarps), 0, st, 1,
                   pdl_enabled(), a);
}

template <typename T, bool VEC>
cudaError_t norm_dispatch(const NormArgs& a, cudaStream_t st) {
#define GO(W, V) return norm_go<T, VEC, W, V>(a, st)
  INSTANT_NORM_DISPATCH(a.C, GO);
#undef GO
}

template <typename T, bool VEC, int W, int V>
cudaError_t back_go(const NormBackArgs& a, cudaStream_t st) {
  constexpr int kWarps = W > 8 ? W : 8;
  constexpr int kRows = kWarps / W;
  const size_t smem = kRows > 1 ? sizeof(float) * 8 * 32 * W * V : 0;
  const cudaError_t e =
      launch_ex(k_rms_norm_back<T, W, V, VEC>, dim3(norm_back_parts(a.rows, a.C)), dim3(32 * kWarps), smem, st,
                1, pdl_enabled(), a);
  if (e != cudaSuccess) return e;
  return launch_part_sum(a.part, a.ggamma, norm_back_parts(a.rows, a.C), a.C, a.accumulate, st);
}

template <typename T, bool VEC>
cudaError_t back_dispatch(const NormBackArgs& a, cudaStream_t st) {
#define GO(W, V) return back_go<T, VEC, W, V>(a, st)
  INSTANT_NORM_DISPATCH(a.C, GO);
#undef GO
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, bool bf16, cudaStream_t st) {
  if (bf16) return norm_dispatch<uint16_t, true>(a, st);
  return a.vec ? norm_dispatch<float, true>(a, st) : norm_dispatch<float, false>(a, st);
}

// the most CTAs of the backward, each with one share of ggamma: four an SM, no
// more than there are row slots of the form with the fewest
int norm_back_parts(int rows, int C) {
  const int slots = C <= 256 ? 8 : C <= 512 ? 4 : C <= 1024 ? 2 : 1;
  const long long ctas = (static_cast<long long>(rows) + slots - 1) / slots;
  const long long most = static_cast<long long>(kColSumSMs) * 4;
  return static_cast<int>(ctas < most ? ctas : most);
}

cudaError_t launch_rms_norm_back(const NormBackArgs& a, bool bf16, cudaStream_t st) {
  if (a.vec && a.C <= 12288) {
    bool done;
    const cudaError_t e = bf16 ? back_stream_dispatch<uint16_t>(a, &done, st) : back_stream_dispatch<float>(a, &done, st);
    if (done) return e;
  }
  if (bf16) return back_dispatch<uint16_t, true>(a, st);
  return a.vec ? back_dispatch<float, true>(a, st) : back_dispatch<float, false>(a, st);
}

INSTANT_FAULT_READER(read_fault_norm)

}  // namespace instant
