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
// Two forms.  The direct one starts a CTA for a handful of rows and loads them
// into registers.  The streaming one keeps two CTAs on each SM; a thread of each
// copies blocks of whole rows (they are contiguous) into a ring in shared memory
// with bulk copies, so that an SM always has 100 KB and more under way whatever
// its warps wait for, and the backward's share of ggamma stays in registers over
// all rows of a CTA.  Which one runs, with both measured: see stream_plan.
#include <algorithm>
#include <cstdlib>

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
template <typename T, int W, int V, typename Gamma>
__device__ __forceinline__ void norm_outputs(const NormArgs& a, float2 (&h)[V][4], float r, int row, int t,
                                             Gamma gamma) {
  const size_t base = static_cast<size_t>(row) * a.C;
  if (a.r && t == 0) a.r[row] = r;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = 8 * (v * 32 * W + t);
    const int n = a.C - c;
    if (a.h) store_pairs(static_cast<T*>(a.h) + base + c, n, a.vec, h[v]);
#pragma unroll
    for (int e = 0; e < 4; ++e) h[v][e] = mul2(h[v][e], both(r));
    if (a.k.q) {
      const uint32_t code = group_code(h[v]);
      const float inv = ckpt_inv_scale(code);
      if (n > 0) {
        *reinterpret_cast<uint2*>(a.k.q + static_cast<size_t>(row) * a.ld + c) =
            make_uint2(ckpt_code4_any(h[v][0], h[v][1], code, inv), ckpt_code4_any(h[v][2], h[v][3], code, inv));
        if ((threadIdx.x & 15) == 0)
          a.k.s[static_cast<size_t>(c / kCkptGroup) * a.rows + row] = static_cast<uint8_t>(code);
      }
    }
    if (a.y) {
      float2 g[4];
      gamma(v, g);
#pragma unroll
      for (int e = 0; e < 4; ++e) g[e] = mul2(g[e], h[v][e]);
      store_pairs(static_cast<T*>(a.y) + base + c, n, a.vec, g);
    }
  }
}

// adds a vector's squares to ss
__device__ __forceinline__ void add_squares(const float2* h, float2& ss) {
#pragma unroll
  for (int e = 0; e < 4; ++e) ss = fma2(h[e], h[e], ss);
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
  float2 h[V][4];
  float2 ss = both(0.f);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = 8 * (v * 32 * W + t);
    load_pairs(x + c, on ? a.C - c : 0, a.vec, h[v]);
    if (res) {
      float2 o[4];
      load_pairs(res + c, on ? a.C - c : 0, a.vec, o);
#pragma unroll
      for (int e = 0; e < 4; ++e) h[v][e] = add2(h[v][e], o[e]);
    }
    add_squares(h[v], ss);
  }
  const float r = rsqrtf(row_sum<W>(ss.x + ss.y, red, warp) / static_cast<float>(a.C) + a.eps);
  if (!on) return;  // a whole warp at a time
  norm_outputs<T, W, V>(a, h, r, row, t, [&](int v, float2* g) {
    const int c = 8 * (v * 32 * W + t);
    load_pairs(static_cast<const T*>(a.gamma) + c, a.C - c, a.vec, g);
  });
}

// one vector of the backward: u from its codes, the share of ggamma, d = gy gamma
// (in place of gy) and the share of the row's dot product.  n channels exist; the
// codes past them are not defined
__device__ __forceinline__ void back_vector(uint2 w, float scale, int n, const float2* gamma, float2* d,
                                            float2* u, float2* acc, float2& dot) {
  ckpt_pairs4(w.x, scale, u);
  ckpt_pairs4(w.y, scale, u + 2);
  if (n < 8) {
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
      load_pairs(static_cast<const T*>(a.gy) + base + c, n, a.vec, d[v]);
      load_pairs(static_cast<const T*>(a.gamma) + c, n, a.vec, gm);
      uint2 w = make_uint2(0u, 0u);
      float scale = 0.f;
      if (n > 0) {
        w = *reinterpret_cast<const uint2*>(a.k.q + static_cast<size_t>(row) * a.ld + c);
        scale = ckpt_scale(a.k.s[static_cast<size_t>(c / kCkptGroup) * a.rows + row]);
      }
      back_vector(w, scale, n, gm, d[v], u[v], acc[v], dot);
    }
    const float c1 = row_sum<W>(dot.x + dot.y, red[it & 1], warp) * inv_c;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 8 * (v * 32 * W + t);
      const int n = on ? a.C - c : 0;
      back_result(r, c1, u[v], d[v]);
      if (a.res) {
        float2 o[4];
        load_pairs(static_cast<const T*>(a.res) + base + c, n, a.vec, o);
#pragma unroll
        for (int e = 0; e < 4; ++e) d[v][e] = add2(d[v][e], o[e]);
      }
      store_pairs(static_cast<T*>(a.gx) + base + c, n, a.vec, d[v]);
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
      store_pairs(p, a.C - c, a.C % 4 == 0, acc[v]);
    }
  }
}

// how a streaming CTA walks the rows: blocks of `block` whole rows, `stages` of
// them in its ring
struct StreamPlan {
  int block, blocks, stages, grid;
  uint32_t stage_bytes;
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

// sum over the W warps of a row; `red` is a buffer of 32 floats, another one at
// the next call
template <int W, int THREADS>
__device__ __forceinline__ float row_sum_stream(float v, float* red, int warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (W == 1) return v;
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  named_barrier<1>(THREADS);
  float sum = 0.f;
  const int first = warp / W * W;
#pragma unroll
  for (int i = 0; i < W; ++i) sum += red[first + i];
  return sum;
}

// The ring of a streaming CTA: `stages` slots, each a block of `block` rows of up
// to three tensors.  full: bytes of a slot's copies; empty: one arrival a warp.
struct Ring {
  uint8_t* base;
  uint64_t *full, *empty;
};

template <typename T>
__device__ __forceinline__ void produce(const StreamPlan& p, const Ring& g, const void* const (&src)[3],
                                        const uint32_t (&row_bytes)[3], int rows) {
  int s = 0, par = 1, issued = 0;
  for (int b = blockIdx.x; b < p.blocks; b += gridDim.x) {
    if (!mbar_wait(&g.empty[s], par)) {
      raise_fault(FAULT_WAIT_EMPTY);
      break;
    }
    const int row0 = b * p.block;
    const uint32_t n = static_cast<uint32_t>(min(p.block, rows - row0));
    uint32_t bytes = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (src[i]) bytes += n * row_bytes[i];
    mbar_arrive_expect_tx(&g.full[s], bytes);
    uint8_t* dst = g.base + static_cast<size_t>(s) * p.stage_bytes;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (src[i]) {
        bulk_load(dst, static_cast<const uint8_t*>(src[i]) + static_cast<size_t>(row0) * row_bytes[i],
                  n * row_bytes[i], &g.full[s]);
        dst += p.block * row_bytes[i];
      }
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
    if (!mbar_wait(&g.full[s], par)) raise_fault(FAULT_WAIT_FULL);
  }
}

template <int THREADS>
__device__ __forceinline__ Ring ring_init(uint8_t* smem, const StreamPlan& p) {
  Ring g;
  g.base = smem;
  g.full = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(p.stages) * p.stage_bytes);
  g.empty = g.full + p.stages;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&g.full[i], 1);
      mbar_init(&g.empty[i], THREADS / 32);
    }
    fence_barrier_init();
  }
  __syncthreads();
  return g;
}

// One answer for all consumer threads, which meet at a barrier in every row.
template <int THREADS>
__device__ __forceinline__ bool wait_block(uint64_t* bar, uint32_t parity) {
  const uint32_t mine = mbar_wait(bar, parity) ? 1u : 0u;
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 2, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(mine), "n"(THREADS)
      : "memory");
  return all != 0;
}

template <typename T, int W, int V>
__global__ void __launch_bounds__((W > 8 ? 32 * W : 256) + 32, W > 8 ? 1 : 2)
    k_rms_norm_stream(NormArgs a, StreamPlan p) {
  constexpr int kWarps = W > 8 ? W : 8;
  constexpr int kSlots = kWarps / W;  // rows at a time
  constexpr int kCons = 32 * kWarps;  // consumer threads; one more warp produces
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[2][32];
  const Ring g = ring_init<kCons>(smem, p);
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5;
  if (warp == kWarps) {
    if ((threadIdx.x & 31) == 0) {
      const void* const src[3] = {a.x, a.res, nullptr};
      const uint32_t bytes = static_cast<uint32_t>(a.C * sizeof(T));
      const uint32_t row_bytes[3] = {bytes, bytes, 0};
      produce<T>(p, g, src, row_bytes, a.rows);
    }
    return;
  }
  const int t = threadIdx.x % (32 * W);  // thread within its row
  const int slot = warp / W;
  const int res_off = p.block * a.C;     // elements from a block's x to its residual
  float2 gm[V][4];                       // this thread's columns of gamma
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = 8 * (v * 32 * W + t);
    load_pairs(static_cast<const T*>(a.gamma) + c, a.C - c, a.vec, gm[v]);
  }
  int s = 0, par = 0, it = 0;
  for (int b = blockIdx.x; b < p.blocks; b += gridDim.x) {
    if (!wait_block<kCons>(&g.full[s], par)) {
      raise_fault(FAULT_WAIT_FULL);
      return;
    }
    const T* sx = reinterpret_cast<const T*>(g.base + static_cast<size_t>(s) * p.stage_bytes);
    const int row0 = b * p.block;
    const int n_rows = min(p.block, a.rows - row0);
    for (int i0 = 0; i0 < n_rows; i0 += kSlots, ++it) {
      const int i = i0 + slot;
      const bool on = i < n_rows;
      const T* xr = sx + (on ? i : 0) * a.C;
      float2 h[V][4];
      float2 ss = both(0.f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = 8 * (v * 32 * W + t);
        const int n = on ? a.C - c : 0;
        load_pairs(xr + c, n, true, h[v]);
        if (a.res) {
          float2 o[4];
          load_pairs(xr + res_off + c, n, true, o);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[v][e] = add2(h[v][e], o[e]);
        }
        add_squares(h[v], ss);
      }
      if (i0 + kSlots >= n_rows) {  // the block is in registers: its slot may be refilled
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&g.empty[s]);
      }
      const float r =
          rsqrtf(row_sum_stream<W, kCons>(ss.x + ss.y, red[it & 1], warp) / static_cast<float>(a.C) + a.eps);
      if (on)
        norm_outputs<T, W, V>(a, h, r, row0 + i, t, [&](int v, float2* g) {
#pragma unroll
          for (int e = 0; e < 4; ++e) g[e] = gm[v][e];
        });
    }
    if (++s == p.stages) {
      s = 0;
      par ^= 1;
    }
  }
}

template <typename T, int W, int V>
__global__ void __launch_bounds__((W > 8 ? 32 * W : 256) + 32, W > 8 ? 1 : 2)
    k_rms_norm_back_stream(NormBackArgs a, StreamPlan p) {
  constexpr int kWarps = W > 8 ? W : 8;
  constexpr int kSlots = kWarps / W;
  constexpr int kCons = 32 * kWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[2][32];
  const Ring g = ring_init<kCons>(smem, p);
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5;
  if (warp == kWarps) {
    if ((threadIdx.x & 31) == 0) {
      const void* const src[3] = {a.gy, a.k.q, a.res};
      const uint32_t bytes = static_cast<uint32_t>(a.C * sizeof(T));
      const uint32_t row_bytes[3] = {bytes, static_cast<uint32_t>(a.ld), bytes};
      produce<T>(p, g, src, row_bytes, a.rows);
    }
    return;
  }
  const int t = threadIdx.x % (32 * W);
  const int slot = warp / W;
  const float inv_c = 1.f / static_cast<float>(a.C);
  float2 acc[V][4], gm[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = 8 * (v * 32 * W + t);
    load_pairs(static_cast<const T*>(a.gamma) + c, a.C - c, a.vec, gm[v]);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[v][e] = both(0.f);
  }
  // factor and scale bytes of the next row of this thread, asked for a row early:
  // they lie a row apart in memory, and nothing else waits for a plain load here
  float r_next = 0.f;
  uint32_t s_next[V];
  auto ask = [&](int row) {
    const bool in = row < a.rows;
    r_next = in ? a.r[row] : 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 8 * (v * 32 * W + t);
      s_next[v] = in && c < a.C ? a.k.s[static_cast<size_t>(c / kCkptGroup) * a.rows + row] : 0u;
    }
  };
  ask(blockIdx.x * p.block + slot);
  int s = 0, par = 0, it = 0;
  bool ok = true;
  for (int b = blockIdx.x; b < p.blocks; b += gridDim.x) {
    ok = wait_block<kCons>(&g.full[s], par);
    if (!ok) {
      raise_fault(FAULT_WAIT_FULL);
      break;
    }
    const uint8_t* base = g.base + static_cast<size_t>(s) * p.stage_bytes;
    const T* sgy = reinterpret_cast<const T*>(base);
    const int8_t* sq = reinterpret_cast<const int8_t*>(base + static_cast<size_t>(p.block) * a.C * sizeof(T));
    const T* sres = reinterpret_cast<const T*>(sq + static_cast<size_t>(p.block) * a.ld);
    const int row0 = b * p.block;
    const int n_rows = min(p.block, a.rows - row0);
    for (int i0 = 0; i0 < n_rows; i0 += kSlots, ++it) {
      const int i = i0 + slot;
      const bool on = i < n_rows;
      const float r = r_next;
      float scale[V];
#pragma unroll
      for (int v = 0; v < V; ++v) scale[v] = ckpt_scale(s_next[v]);
      // the row after this one: in this block, or the first of the CTA's next
      ask(i0 + kSlots < n_rows ? row0 + i + kSlots : row0 + static_cast<int>(gridDim.x) * p.block + slot);
      float2 u[V][4], d[V][4];
      float2 dot = both(0.f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = 8 * (v * 32 * W + t);
        const int n = on ? a.C - c : 0;
        load_pairs(sgy + (on ? i : 0) * a.C + c, n, true, d[v]);
        uint2 w = make_uint2(0u, 0u);
        if (n > 0) w = *reinterpret_cast<const uint2*>(sq + static_cast<size_t>(i) * a.ld + c);
        else scale[v] = 0.f;
        back_vector(w, scale[v], n, gm[v], d[v], u[v], acc[v], dot);
      }
      const float c1 = row_sum_stream<W, kCons>(dot.x + dot.y, red[it & 1], warp) * inv_c;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = 8 * (v * 32 * W + t);
        const int n = on ? a.C - c : 0;
        back_result(r, c1, u[v], d[v]);
        if (a.res) {
          float2 o[4];
          load_pairs(sres + (on ? i : 0) * a.C + c, n, true, o);
#pragma unroll
          for (int e = 0; e < 4; ++e) d[v][e] = add2(d[v][e], o[e]);
        }
        store_pairs(static_cast<T*>(a.gx) + static_cast<size_t>(row0 + (on ? i : 0)) * a.C + c, n, true, d[v]);
      }
    }
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&g.empty[s]);
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

// the same with the widest rows in three or four vectors of 16 warps
#define INSTANT_STREAM_DISPATCH(C, GO)                   \
  do {                                                   \
    if ((C) <= 256) GO(1, 1);                            \
    if ((C) <= 512) GO(1, 2);                            \
    if ((C) <= 1024) GO(2, 2);                           \
    if ((C) <= 2048) GO(4, 2);                           \
    if ((C) <= 4096) GO(8, 2);                           \
    if ((C) <= 8192) GO(16, 2);                          \
    if ((C) <= 12288) GO(16, 3);                         \
    GO(16, 4);                                           \
  } while (0)

// Streaming plan of `rows` rows that bring row_bytes each, W warps a row; false
// where the direct form runs: rows whose copies are not multiples of 16 bytes or
// do not fit a ring of two.  A slot holds about 16 KB, a CTA about 100 KB (two an
// SM; one of 16 warps with 200 KB).
bool stream_plan(StreamPlan& p, int rows, int C, size_t row_bytes, bool vec) {
  if (!vec || C > 16384) return false;
  if (const char* v = getenv("STREAM")) { if (atoi(v) == 0) return false; }
  int w = 1;
  while (w < 16 && 512 * w < C) w *= 2;
  const int slots = w > 8 ? 1 : 8 / w;
  const size_t pass = slots * row_bytes;
  const size_t passes = pass >= 16384 ? 1 : std::min<size_t>(16, 16384 / pass);
  p.block = static_cast<int>(slots * passes);
  p.blocks = (rows + p.block - 1) / p.block;
  p.stage_bytes = static_cast<uint32_t>((passes * pass + 127) / 128 * 128);
  p.stages = static_cast<int>(std::min<size_t>(8, (w > 8 ? 200 * 1024 : 100 * 1024) / p.stage_bytes));
  if (p.stages < 2) return false;
  const int sms = std::min(sm_count(), kColSumSMs);
  p.grid = std::min(p.blocks, w > 8 ? sms : 2 * sms);
  // the ring is also the place of a CTA's column sums (the backward)
  p.smem = std::max<size_t>(static_cast<size_t>(p.stages) * p.stage_bytes, sizeof(float) * 512 * 2 * w * 2) +
           16 * p.stages;
  return true;
}

template <typename T, int W, int V>
cudaError_t norm_stream_go(const NormArgs& a, const StreamPlan& p, cudaStream_t st) {
  auto k = k_rms_norm_stream<T, W, V>;
  const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(k), p.smem, true);
  if (e != cudaSuccess) return e;
  return launch_ex(k, dim3(p.grid), dim3((W > 8 ? 32 * W : 256) + 32), p.smem, st, 1, pdl_enabled(), a, p);
}

template <typename T>
cudaError_t norm_stream_dispatch(const NormArgs& a, const StreamPlan& p, cudaStream_t st) {
#define GO(W, V) return norm_stream_go<T, W, V>(a, p, st)
  INSTANT_STREAM_DISPATCH(a.C, GO);
#undef GO
}

template <typename T, int W, int V>
cudaError_t back_stream_go(const NormBackArgs& a, const StreamPlan& p, cudaStream_t st) {
  auto k = k_rms_norm_back_stream<T, W, V>;
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(k), p.smem, true);
  if (e == cudaSuccess)
    e = launch_ex(k, dim3(p.grid), dim3((W > 8 ? 32 * W : 256) + 32), p.smem, st, 1, pdl_enabled(), a, p);
  if (e != cudaSuccess) return e;
  return launch_part_sum(a.part, a.ggamma, p.grid, a.C, a.accumulate, st);
}

template <typename T>
cudaError_t back_stream_dispatch(const NormBackArgs& a, const StreamPlan& p, cudaStream_t st) {
#define GO(W, V) return back_stream_go<T, W, V>(a, p, st)
  INSTANT_STREAM_DISPATCH(a.C, GO);
#undef GO
}

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
  const size_t row = static_cast<size_t>(a.C) * (bf16 ? 2 : 4);
  StreamPlan p;
  if (stream_plan(p, a.rows, a.C, a.res ? 2 * row : row, a.vec))
    return bf16 ? norm_stream_dispatch<uint16_t>(a, p, st) : norm_stream_dispatch<float>(a, p, st);
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
  const size_t row = static_cast<size_t>(a.C) * (bf16 ? 2 : 4);
  StreamPlan p;
  if (stream_plan(p, a.rows, a.C, (a.res ? 2 * row : row) + a.ld, a.vec))
    return bf16 ? back_stream_dispatch<uint16_t>(a, p, st) : back_stream_dispatch<float>(a, p, st);
  return bf16 ? back_dispatch<uint16_t>(a, st) : back_dispatch<float>(a, st);
}

INSTANT_FAULT_READER(read_fault_norm)

}  // namespace instant
