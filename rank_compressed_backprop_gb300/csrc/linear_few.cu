// linear_few.cu -- the three products of an MLP block's linear layers (forward,
// back, grad_w; see linear_tc.cu) where the output has too few tiles to fill the
// GPU with CTA pairs: a single token of generation, short batches, narrow layers.
//
// With few rows the time is that of reading the weights, so the roles are
// swapped: the 128 lanes of the accumulator are output channels (of w, or of the
// checkpoint's values in grad_w) and its NT columns are rows, NT = 16, 32, 64 or
// 128, the fewest that hold the rows.  A 64-deep chunk of weights is 16 KB, and
// three (NT <= 32) or two CTAs share an SM, so an SM has 100 to 200 KB of loads
// under way.  K is split across the CTAs of a cluster until the grid is one full
// wave; each parks its fp32 partial tile in shared memory, and the rows are
// dealt out over the cluster: a warp adds the partial sums of a row's 128 channels
// in the order of the ranks (the same bits on every call) through distributed
// shared memory and carries the row through the epilogue, 4 channels a lane -- one
// checkpoint group a warp.
// One token, 4096 -> 11008: 15.8 us, the weights' 90 MB at 5.7 TB/s (a library matrix
// product 17.6); 64 rows 18.9.
#include <map>
#include <mutex>
#include <tuple>

#include "ckpt.cuh"

namespace instant {

namespace {

constexpr int BM = 128, BK = 64;              // channels of a tile, depth of a chunk
constexpr uint32_t A_BYTES = BM * BK * 2;     // 16 KB
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int LD = BM + 4;                    // floats of a row of the partial tile
enum { FORWARD = 0, BACK = 1, GRAD_W = 2 };

__host__ __device__ constexpr int stages_of(int nt) { return nt == 128 ? 3 : 4; }
__host__ __device__ constexpr uint32_t stage_of(int nt) { return A_BYTES + nt * BK * 2; }
__host__ __device__ constexpr uint32_t bar_of(int nt) {
  const uint32_t ring = stages_of(nt) * stage_of(nt), red = nt * LD * 4;
  return ring > red ? ring : red;
}
constexpr size_t smem_of(int nt) { return bar_of(nt) + 128 + 1024; }

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

// checkpoint of a row's 128 channels, four a lane from c
__device__ __forceinline__ void put_ckpt(uint8_t* s, int8_t* q, int ld, int rows, int row, int c, int C,
                                         const float (&v)[4]) {
  uint32_t m = 0;
  if (c < C) m = max(max(abs_bits(v[0]), abs_bits(v[1])), max(abs_bits(v[2]), abs_bits(v[3])));
  const uint32_t code = ckpt_scale_code(warp_max(m));
  if (c < C)
    *reinterpret_cast<uint32_t*>(q + static_cast<size_t>(row) * ld + c) =
        ckpt_code4(v[0], v[1], v[2], v[3], ckpt_inv_scale(code));
  if ((threadIdx.x & 31) == 0 && c < C)
    s[static_cast<size_t>(c / kCkptGroup) * rows + row] = static_cast<uint8_t>(code);
}

template <int ACT>
__device__ __forceinline__ void act4(float (&v)[4]) {
  const float2 a = act_fast<ACT>(make_float2(v[0], v[1])), b = act_fast<ACT>(make_float2(v[2], v[3]));
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}
template <int ACT>
__device__ __forceinline__ void slope4(float (&v)[4], const float (&z)[4]) {
  const float2 a = act_slope_fast<ACT>(make_float2(z[0], z[1])), b = act_slope_fast<ACT>(make_float2(z[2], z[3]));
  v[0] *= a.x; v[1] *= a.y; v[2] *= b.x; v[3] *= b.y;
}

// one row's epilogue, all 32 lanes: channels c .. c + 3 of output row `row`
template <int KIND>
__device__ __forceinline__ void finish_row(const FewArgs& a, float (&v)[4], int row, int c) {
  const bool on = c < a.N;
  const size_t off = static_cast<size_t>(row) * a.N + c;
  float t[4];
  if (KIND == GRAD_W) {
    if (!on) return;
    float* out = static_cast<float*>(a.out) + off;
    if (a.bias) {
      load_vec<4>(static_cast<const uint16_t*>(a.bias) + c, t);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= t[e];
    }
    if (a.accumulate) {
      load_vec<4>(out, t);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += t[e];
    }
    store_vec<4>(out, v);
    return;
  }
  if (KIND == FORWARD) {
    if (a.bias && on) {
      load_vec<4>(static_cast<const uint16_t*>(a.bias) + c, t);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += t[e];
    }
    if (a.zk.q) put_ckpt(a.zk.s, a.zk.q, a.ld, a.M, row, c, a.N, v);
    switch (a.act) {
      case INSTANT_ACT_RELU: act4<INSTANT_ACT_RELU>(v); break;
      case INSTANT_ACT_GELU: act4<INSTANT_ACT_GELU>(v); break;
      case INSTANT_ACT_SILU: act4<INSTANT_ACT_SILU>(v); break;
      default: break;
    }
  } else if (a.act != INSTANT_ACT_NONE && on) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(a.ck.q + static_cast<size_t>(row) * a.ld + c);
    float z[4];
    ckpt_values4(w, ckpt_scale(a.ck.s[static_cast<size_t>(c / kCkptGroup) * a.M + row]), z);
    switch (a.act) {
      case INSTANT_ACT_RELU: slope4<INSTANT_ACT_RELU>(v, z); break;
      case INSTANT_ACT_GELU: slope4<INSTANT_ACT_GELU>(v, z); break;
      default: slope4<INSTANT_ACT_SILU>(v, z); break;
    }
  }
  if (a.res && on) {
    load_vec<4>(static_cast<const uint16_t*>(a.res) + off, t);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += t[e];
  }
  if (KIND == FORWARD && a.yk.q) put_ckpt(a.yk.s, a.yk.q, a.ld, a.M, row, c, a.N, v);
  if (a.out && on) store_vec<4>(static_cast<uint16_t*>(a.out) + off, v);
}

// Rows of the tile, dealt out over the cluster's warps; a warp takes ROWS at a
// time, whose loads of up to SPLITS partial sums are under way together.
template <int KIND, int ROWS, int SPLITS>
__device__ __forceinline__ void finish_rows(const FewArgs& a, const float* red, int rank, int rows, int r0,
                                            int n0) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stride = kWarps * a.splits;
  for (int base = rank + a.splits * warp; base < rows; base += ROWS * stride) {
    float4 part[ROWS][SPLITS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const int i = base + j * stride;
      const float* src = red + i * LD + 4 * lane;
#pragma unroll
      for (int q = 0; q < SPLITS; ++q)
        if (i < rows && q < a.splits)
          part[j][q] = SPLITS == 1 ? *reinterpret_cast<const float4*>(src) : dsmem_ld_f4(dsmem_addr(src, q));
    }
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const int i = base + j * stride;
      if (i >= rows) break;
      float v[4] = {part[j][0].x, part[j][0].y, part[j][0].z, part[j][0].w};
#pragma unroll
      for (int q = 1; q < SPLITS; ++q)
        if (q < a.splits) {
          v[0] += part[j][q].x; v[1] += part[j][q].y; v[2] += part[j][q].z; v[3] += part[j][q].w;
        }
      finish_row<KIND>(a, v, r0 + i, n0 + 4 * lane);
    }
  }
}

template <int KIND, int NT>
__global__ void __launch_bounds__(kThreads)
    k_linear_few(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                 FewArgs a) {
  constexpr bool A_MN = KIND != FORWARD, B_MN = KIND == GRAD_W;
  constexpr int NS = stages_of(NT);
  constexpr uint32_t STAGE = stage_of(NT);
  constexpr int COLS = NT <= 16 ? 64 : 128;  // TMEM columns
  constexpr int ACCS = COLS / NT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* red = reinterpret_cast<float*>(smem);  // [NT][LD], over the ring after the K loop
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + bar_of(NT));
  uint64_t* empty = full + NS;
  uint64_t* done = empty + NS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * BM;   // first channel
  const int r0 = blockIdx.y * NT;   // first row
  const int rank = blockIdx.z;      // == rank in the cluster (1 x 1 x splits)
  const int k_begin = rank * a.per;
  const int nk = max(0, min(a.nk - k_begin, a.per));
  // segments of at least four chunks, each in an accumulator of its own: the tensor
  // cores' sums cut low bits at every step, and the segments are added in fp32
  const int seg = max(4, (nk + ACCS - 1) / ACCS);

  auto load_a = [&](uint8_t* dst, int k0, uint64_t* bar) {
    if (A_MN) {  // stored [K, N]: two boxes of 64 channels x 64 K rows
      tma_load_2d(dst, &map_a, bar, n0, k0);
      tma_load_2d(dst + A_BYTES / 2, &map_a, bar, n0 + 64, k0);
    } else {
      tma_load_2d(dst, &map_a, bar, k0, n0);
    }
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    fence_barrier_init();
    prefetch_tmap(&map_a);
    prefetch_tmap(&map_b);
    // the ring's first chunks of weights into L2 while the predecessor finishes
    // (L2 is the point of coherence: a line fetched early follows later writes)
    if (KIND != GRAD_W)
      for (int i = 0; i < nk && i < NS; ++i) {
        const int k0 = (k_begin + i) * BK;
        if (A_MN) {
          tma_prefetch_l2_2d(&map_a, n0, k0);
          tma_prefetch_l2_2d(&map_a, n0 + 64, k0);
        } else {
          tma_prefetch_l2_2d(&map_a, k0, n0);
        }
      }
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait();

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    int issued = 0, s = 0, par = 1;
    for (int i = 0; i < nk; ++i) {
      if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], par))) {
        raise_fault(FAULT_WAIT_EMPTY);
        break;
      }
      if (elect_one()) {
        const int k0 = (k_begin + i) * BK;
        uint8_t* sa = smem + s * STAGE;
        uint8_t* sb = sa + A_BYTES;
        mbar_arrive_expect_tx(&full[s], STAGE);
        load_a(sa, k0, &full[s]);
        if (B_MN) {
#pragma unroll
          for (int h = 0; h < NT / 64; ++h) tma_load_2d(sb + h * 64 * BK * 2, &map_b, &full[s], r0 + 64 * h, k0);
        } else {
          tma_load_2d(sb, &map_b, &full[s], k0, r0);
        }
      }
      __syncwarp();
      ++issued;
      if (++s == NS) {
        s = 0;
        par ^= 1;
      }
    }
    for (int i = issued - NS < 0 ? 0 : issued - NS; i < issued; ++i)
      if (!mbar_wait(&full[i % NS], (i / NS) & 1)) raise_fault(FAULT_WAIT_FULL);
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    constexpr uint32_t idesc = idesc_bf16_f32(BM, NT, A_MN, B_MN);
    const uint32_t base = smem_u32(smem);
    const uint64_t a_desc0 = A_MN ? sdesc_sw128(base, A_BYTES / 2, 1024) : sdesc_sw128(base, 16, 1024);
    const uint64_t b_desc0 =
        B_MN ? sdesc_sw128(base + A_BYTES, 64 * BK * 2, 1024) : sdesc_sw128(base + A_BYTES, 16, 1024);
    int s = 0, par = 0, acc = 0, left = seg;  // accumulator and what its segment lacks
    for (int i = 0; i < nk; ++i) {
      if (!__all_sync(0xffffffffu, mbar_wait(&full[s], par))) {
        raise_fault(FAULT_WAIT_FULL);
        break;
      }
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          umma_bf16(tmem + acc * NT, a_desc0 + s * (STAGE >> 4) + kk * (A_MN ? 2048 >> 4 : 32 >> 4),
                    b_desc0 + s * (STAGE >> 4) + kk * (B_MN ? 2048 >> 4 : 32 >> 4), idesc, left != seg || kk != 0);
        umma_commit(&empty[s]);
        if (i == nk - 1) umma_commit(done);
      }
      __syncwarp();
      if (--left == 0) {
        ++acc;
        left = seg;
      }
      if (++s == NS) {
        s = 0;
        par ^= 1;
      }
    }
  }
  __syncwarp();

  // ---------------- TMEM -> fp32 partial tile [row][channel] ----------------
  if (nk > 0 && !mbar_wait(done, 0)) raise_fault(FAULT_WAIT_DONE);
  tc_fence_after();
  __syncthreads();  // every stage is consumed: the ring becomes the partial tile
  {
    // warps 0-3 and 4-7 take every other 16 rows of the four lane quarters
    const int ch = (warp & 3) * 32 + lane;
    const uint32_t taddr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
#pragma unroll 1
    for (int j0 = 16 * (warp >> 2); j0 < NT; j0 += 32) {
      float v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = 0.f;
#pragma unroll 1
      for (int acc = 0; acc * seg < nk; ++acc) {
        float w[16];
        tmem_ld16(taddr + acc * NT + j0, w);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] += w[j];
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) red[(j0 + j) * LD + ch] = v[j];
    }
  }
  tc_fence_before();
  if (a.splits > 1) cluster_sync(); else __syncthreads();

  // ---------------- rows of the tile, dealt out over the cluster's warps ----------------
  const int rows = min(NT, a.M - r0);
  if (a.splits == 1) finish_rows<KIND, 4, 1>(a, red, rank, rows, r0, n0);
  else if (a.splits == 2) finish_rows<KIND, 4, 2>(a, red, rank, rows, r0, n0);
  else if (a.splits <= 4) finish_rows<KIND, 2, 4>(a, red, rank, rows, r0, n0);
  else finish_rows<KIND, 1, 8>(a, red, rank, rows, r0, n0);
  // peers may still read this CTA's tile: leave together
  if (a.splits > 1) cluster_sync(); else __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, COLS);
}

// Stand-in for the cluster occupancy query with this shared memory and block
// size (registers and TMEM never limit this kernel)
__global__ void __launch_bounds__(kThreads) k_few_fit(int* p) {
  extern __shared__ int fit_smem[];
  if (p) p[threadIdx.x] = fit_smem[threadIdx.x];
}

// clusters of `splits` CTAs with `bytes` of shared memory that the device holds at once
int clusters_at_once(size_t bytes, int splits) {
  static std::mutex mu;
  static std::map<std::tuple<int, size_t, int>, int> counts;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lock(mu);
  const auto key = std::make_tuple(dev, bytes, splits);
  const auto it = counts.find(key);
  if (it != counts.end()) return it->second;
  const void* k = reinterpret_cast<const void*>(k_few_fit);
  if (raise_smem_limit(k, bytes) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1024, 1, splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = splits;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;
  }
  counts[key] = n;
  return n;
}

template <int KIND, int NT>
cudaError_t go(const CUtensorMap& ma, const CUtensorMap& mb, FewArgs a, cudaStream_t st) {
  auto k = k_linear_few<KIND, NT>;
  const size_t bytes = smem_of(NT);
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(k), bytes, true);
  if (e != cudaSuccess) return e;
  const dim3 tiles((a.N + BM - 1) / BM, (a.M + NT - 1) / NT);
  const long long n = static_cast<long long>(tiles.x) * tiles.y;
  // the most shares of K whose clusters all fit the device at once
  a.splits = 1;
  for (int s = 2; s <= 8 && s <= a.nk; ++s)
    if (clusters_at_once(bytes, s) >= n) a.splits = s;
  a.per = (a.nk + a.splits - 1) / a.splits;
  return launch_ex(k, dim3(tiles.x, tiles.y, a.splits), dim3(kThreads), bytes, st, a.splits, pdl_enabled(), ma, mb,
                   a);
}

template <int KIND>
cudaError_t go_rows(int nt, const CUtensorMap& ma, const CUtensorMap& mb, const FewArgs& a, cudaStream_t st) {
  if (KIND != GRAD_W) {
    if (nt == 16) return go<KIND, KIND == GRAD_W ? 64 : 16>(ma, mb, a, st);
    if (nt == 32) return go<KIND, KIND == GRAD_W ? 64 : 32>(ma, mb, a, st);
  }
  return nt == 64 ? go<KIND, 64>(ma, mb, a, st) : go<KIND, 128>(ma, mb, a, st);
}

}  // namespace

int few_rows_tile(const LinearArgs& l) {
  int nt = l.kind == GRAD_W ? 64 : 16;  // an MN-major operand comes in 64-wide boxes
  // checkpoints, whose codes show the sums' low bits: two accumulators of 64 rows rather
  // than one of 128
  const int most = l.zk.q || l.yk.q ? 64 : 128;
  while (nt < most && nt < l.M) nt *= 2;
  return nt;
}

cudaError_t launch_linear_few(const LinearArgs& l, cudaStream_t st) {
  FewArgs a{};
  a.M = l.M;
  a.N = l.N;
  a.K = l.K;
  a.nk = (l.K + BK - 1) / BK;
  a.bias = l.bias;
  a.res = l.res;
  a.out = l.out;
  a.zk = l.zk;
  a.yk = l.yk;
  a.ck = l.ck;
  a.ld = l.ld;
  a.act = l.act;
  a.accumulate = l.accumulate;
  const int nt = few_rows_tile(l);
  if ((l.M + nt - 1) / nt > kFewMaxRowTiles) return cudaErrorInvalidValue;
  CUtensorMap ma, mb;
  auto map = [](CUtensorMap* m, const void* p, long long inner, long long outer, int box_outer) {
    const uint64_t d[2] = {static_cast<uint64_t>(inner), static_cast<uint64_t>(outer)};
    const uint64_t s[1] = {static_cast<uint64_t>(inner) * 2};
    const uint32_t b[2] = {64, static_cast<uint32_t>(box_outer)};
    return make_map(m, p, 2, d, s, b);
  };
  const bool ok = l.kind == FORWARD ? map(&ma, l.b, l.K, l.N, BM) && map(&mb, l.a, l.K, l.M, nt)
                  : l.kind == BACK ? map(&ma, l.b, l.N, l.K, BK) && map(&mb, l.a, l.K, l.M, nt)
                                   : map(&ma, l.b, l.N, l.K, BK) && map(&mb, l.a, l.M, l.K, BK);
  if (!ok) return cudaErrorInvalidValue;
  if (l.kind == FORWARD) return go_rows<FORWARD>(nt, ma, mb, a, st);
  if (l.kind == BACK) return go_rows<BACK>(nt, ma, mb, a, st);
  return go_rows<GRAD_W>(nt, ma, mb, a, st);
}

INSTANT_FAULT_READER(read_fault_few)

}  // namespace instant
