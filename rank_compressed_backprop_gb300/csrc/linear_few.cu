// linear_few.cu -- the three products of an MLP block's linear layers (forward,
// back, grad_w; see linear_tc.cu) where the output has too few tiles to fill the
// GPU with CTA pairs: a single token of generation, short batches, narrow layers.
//
// With few rows the time is that of reading the weights, so the roles are
// swapped: the 128 lanes of the accumulator are output channels (of w, or of the
// checkpoint's values in grad_w) and its NT columns are rows, NT = 16, 32, 64 or
// 128, the fewest that hold the rows.  A 64-deep chunk of weights is 16 KB, and
// three (NT = 16) or two CTAs share an SM, so an SM has 100 to 200 KB of loads
// under way.  K is split across the CTAs of a cluster until the grid is one full
// wave; each parks its fp32 partial tile in shared memory, and the rows are
// dealt out over the cluster: a warp adds the partial sums of a row's 128 channels
// in the order of the ranks (the same bits on every call) through distributed
// shared memory and carries the row through the epilogue, 4 channels a lane -- one
// checkpoint group a warp.
// The tensor cores' sums cut low bits at every step (linear_tc.cu), so an accumulator
// holds a segment of a few chunks only: warps of their own add it to registers in
// ordinary fp32 while the next segment's products run in another accumulator.  (With the
// whole share of K in one to four accumulators a weight gradient over 8192 rows was 2.5e-6
// from 64 bits, now 1.9e-7, and the checkpoints of 128 x 4096 -> 11008 2.2 times as far off
// as after fp32 sums in order, now 0.8 times, in the same time.)  128 rows in bf16, which
// hide those bits, have one segment.
// One token, 4096 -> 11008: 15.8 us, the weights' 90 MB at 5.7 TB/s (a library matrix
// product 17.6); 64 rows 18.9; 128 rows with z's and y's checkpoints 30.
#include <algorithm>
#include <cmath>
#include <map>
#include <mutex>
#include <tuple>

#include "ckpt.cuh"

namespace instant {

namespace {

constexpr int BM = 128, BK = 64;              // channels of a tile, depth of a chunk
constexpr uint32_t A_BYTES = BM * BK * 2;     // 16 KB
constexpr int LD = BM + 4;                    // floats of a row of the partial tile
enum { FORWARD = 0, BACK = 1, GRAD_W = 2 };

// The warps' roles.  Up to 64 rows warp 0 produces, warp 1 issues the products and warps 4
// to 7 take the segments over, a thread all rows of its channel.  A weight gradient of 128
// rows has eight warps for that, which have half of the rows each, beside a producer and an
// issuer, and one accumulator: while it is read, the products of the SM's other CTA run.
// (With ten warps for all sizes there was less room for the next launch to start in: 1571
// rows, 768 x 776 16.1 us instead of 12.7, 512 x 1024 -> 1024 10.7 instead of 9.5.)
template <int KIND, int NT>
struct Roles {
  static constexpr bool kWide = KIND == GRAD_W && NT == 128;
  static constexpr bool kSums = kWide || NT <= 64;  // else one segment, read by all warps at the end
  static constexpr int kWarps = kWide ? 10 : 8;
  static constexpr int kProducer = kWide ? 8 : 0, kIssuer = kWide ? 9 : 1;
  static constexpr int kReader = kWide ? 0 : 4;     // first of the warps that read
  static constexpr int kReaders = kWide ? 8 : 4;
  static constexpr int kRows = kSums ? NT * 4 / kReaders : 16;  // of a reader's channel at a time
  static constexpr int kSegment = KIND == GRAD_W ? 16 : 4;      // chunks, as in linear_tc.cu for gradients
};

__host__ __device__ constexpr int stages_of(int nt) { return nt == 128 ? 3 : 4; }
__host__ __device__ constexpr uint32_t stage_of(int nt) { return A_BYTES + nt * BK * 2; }
__host__ __device__ constexpr uint32_t bar_of(int nt) {
  const uint32_t ring = stages_of(nt) * stage_of(nt), red = nt * LD * 4;
  return ring > red ? ring : red;
}
constexpr size_t smem_of(int nt) { return bar_of(nt) + 192 + 1024; }

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
template <int KIND, int WARPS, int ROWS, int SPLITS>
__device__ __forceinline__ void finish_rows(const FewArgs& a, const float* red, int rank, int rows, int r0,
                                            int n0) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stride = WARPS * a.splits;
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
// (two CTAs of the wide form are to fit an SM; named for the others, a number of CTAs would
// only let the compiler take more registers, which the next launch then waits for)
__global__ void __launch_bounds__(32 * Roles<KIND, NT>::kWarps, Roles<KIND, NT>::kWide ? 2 : 0)
    k_linear_few(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                 FewArgs a) {
  constexpr bool A_MN = KIND != FORWARD, B_MN = KIND == GRAD_W;
  constexpr int NS = stages_of(NT);
  constexpr uint32_t STAGE = stage_of(NT);
  constexpr int COLS = NT <= 16 ? 64 : 128;  // TMEM columns
  constexpr int ACCS = COLS / NT;
  using R = Roles<KIND, NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* red = reinterpret_cast<float*>(smem);  // [NT][LD], over the ring after the K loop
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + bar_of(NT));
  uint64_t* empty = full + NS;
  uint64_t* t_full = empty + NS;     // [ACCS] a segment's products are done
  uint64_t* t_empty = t_full + ACCS; // [ACCS] its sums have been read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(t_empty + ACCS);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * BM;   // first channel
  const int r0 = blockIdx.y * NT;   // first row
  const int rank = blockIdx.z;      // == rank in the cluster (1 x 1 x splits)
  const int k_begin = rank * a.per;
  const int nk = max(0, min(a.nk - k_begin, a.per));
  const int seg = R::kSums ? R::kSegment : nk;

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
    for (int i = 0; i < ACCS; ++i) {
      mbar_init(&t_full[i], 1);
      mbar_init(&t_empty[i], R::kReaders);
    }
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

  const int ch = (warp & 3) * 32 + lane;  // a warp has the TMEM lanes of its quarter
  const uint32_t taddr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  const bool reads = warp >= R::kReader && warp < R::kReader + R::kReaders;
  const int j0 = (warp - R::kReader) / 4 * R::kRows;  // first of a reader's rows
  float v[R::kRows];                                  // their sums
  if (warp == R::kProducer) {
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
  } else if (warp == R::kIssuer) {
    // ---------------- MMA issuer ----------------
    constexpr uint32_t idesc = idesc_bf16_f32(BM, NT, A_MN, B_MN);
    const uint32_t base = smem_u32(smem);
    const uint64_t a_desc0 = A_MN ? sdesc_sw128(base, A_BYTES / 2, 1024) : sdesc_sw128(base, 16, 1024);
    const uint64_t b_desc0 =
        B_MN ? sdesc_sw128(base + A_BYTES, 64 * BK * 2, 1024) : sdesc_sw128(base + A_BYTES, 16, 1024);
    int s = 0, par = 0, acc = 0, turn = 0, left = 0;  // accumulator, turns through all, what its segment lacks
    for (int i = 0; i < nk; ++i) {
      const bool first = left == 0;
      if (first) {
        left = min(seg, nk - i);
        if (turn > 0 && !__all_sync(0xffffffffu, mbar_wait(&t_empty[acc], (turn - 1) & 1))) {
          raise_fault(FAULT_WAIT_EMPTY);
          break;
        }
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&full[s], par))) {
        raise_fault(FAULT_WAIT_FULL);
        break;
      }
      tc_fence_after();
      --left;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          umma_bf16(tmem + acc * NT, a_desc0 + s * (STAGE >> 4) + kk * (A_MN ? 2048 >> 4 : 32 >> 4),
                    b_desc0 + s * (STAGE >> 4) + kk * (B_MN ? 2048 >> 4 : 32 >> 4), idesc, !first || kk != 0);
        umma_commit(&empty[s]);
        if (left == 0) umma_commit(&t_full[acc]);
      }
      __syncwarp();
      if (left == 0 && ++acc == ACCS) {
        acc = 0;
        ++turn;
      }
      if (++s == NS) {
        s = 0;
        par ^= 1;
      }
    }
  } else if (R::kSums && reads) {
    // ---------------- segments out of TMEM ----------------
#pragma unroll
    for (int j = 0; j < R::kRows; ++j) v[j] = 0.f;
    int acc = 0, par = 0;
#pragma unroll 1
    for (int k0 = 0; k0 < nk; k0 += seg) {
      if (!__all_sync(0xffffffffu, mbar_wait(&t_full[acc], par))) {
        raise_fault(FAULT_WAIT_DONE);
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < R::kRows; j += 16) {
        float w[16];
        tmem_ld16(taddr + acc * NT + j0 + j, w);
#pragma unroll
        for (int e = 0; e < 16; ++e) v[j + e] += w[e];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&t_empty[acc]);
      if (++acc == ACCS) {
        acc = 0;
        par ^= 1;
      }
    }
  }
  __syncwarp();

  // ---------------- fp32 partial tile [row][channel] ----------------
  if (!R::kSums && nk > 0 && !mbar_wait(t_full, 0)) raise_fault(FAULT_WAIT_DONE);
  tc_fence_after();
  __syncthreads();  // every stage is consumed: the ring becomes the partial tile
  if constexpr (R::kSums) {
    if (reads) {
#pragma unroll
      for (int j = 0; j < R::kRows; ++j) red[(j0 + j) * LD + ch] = v[j];
    }
  } else {
    // warps 0-3 and 4-7 take every other 16 rows
#pragma unroll 1
    for (int j1 = 16 * (warp >> 2); j1 < NT; j1 += 32) {
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = 0.f;
      if (nk > 0) tmem_ld16(taddr + j1, v);
#pragma unroll
      for (int j = 0; j < 16; ++j) red[(j1 + j) * LD + ch] = v[j];
    }
  }
  tc_fence_before();
  if (a.splits > 1) cluster_sync(); else __syncthreads();

  // ---------------- rows of the tile, dealt out over the cluster's warps ----------------
  const int rows = min(NT, a.M - r0);
  if (a.splits == 1) finish_rows<KIND, R::kWarps, 4, 1>(a, red, rank, rows, r0, n0);
  else if (a.splits == 2) finish_rows<KIND, R::kWarps, 4, 2>(a, red, rank, rows, r0, n0);
  else if (a.splits <= 4) finish_rows<KIND, R::kWarps, 2, 4>(a, red, rank, rows, r0, n0);
  else finish_rows<KIND, R::kWarps, 1, 8>(a, red, rank, rows, r0, n0);
  // peers may still read this CTA's tile: leave together
  if (a.splits > 1) cluster_sync(); else __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, COLS);
}

// Stand-in for the cluster occupancy query with this shared memory and block
// size (registers, 102 a thread at most, and TMEM columns do not limit this kernel)
__global__ void k_few_fit(int* p) {
  extern __shared__ int fit_smem[];
  if (p) p[threadIdx.x] = fit_smem[threadIdx.x];
}

// clusters of `splits` CTAs with `bytes` of shared memory that the device holds at once
int clusters_at_once(size_t bytes, int threads, int splits) {
  static std::mutex mu;
  static std::map<std::tuple<int, size_t, int, int>, int> counts;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lock(mu);
  const auto key = std::make_tuple(dev, bytes, threads, splits);
  const auto it = counts.find(key);
  if (it != counts.end()) return it->second;
  const void* k = reinterpret_cast<const void*>(k_few_fit);
  if (raise_smem_limit(k, bytes) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1024, 1, splits);
  cfg.blockDim = dim3(threads);
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
  constexpr int kThreads = 32 * Roles<KIND, NT>::kWarps;
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(k), bytes, true);
  if (e != cudaSuccess) return e;
  const dim3 tiles((a.N + BM - 1) / BM, (a.M + NT - 1) / NT);
  const long long n = static_cast<long long>(tiles.x) * tiles.y;
  // the most shares of K whose clusters all fit the device at once
  a.splits = 1;
  for (int s = 2; s <= 8 && s <= a.nk; ++s)
    if (clusters_at_once(bytes, kThreads, s) >= n) a.splits = s;
  a.per = (a.nk + a.splits - 1) / a.splits;
  return launch_ex(k, dim3(tiles.x, tiles.y, a.splits), dim3(kThreads), bytes, st, a.splits, pdl_enabled(), ma, mb,
                   a);
}

template <int KIND>
cudaError_t go_rows(int nt, const CUtensorMap& ma, const CUtensorMap& mb, const FewArgs& a, cudaStream_t st) {
  if constexpr (KIND != GRAD_W) {
    if (nt == 16) return go<KIND, 16>(ma, mb, a, st);
    if (nt == 32) return go<KIND, 32>(ma, mb, a, st);
  }
  return nt == 64 ? go<KIND, 64>(ma, mb, a, st) : go<KIND, 128>(ma, mb, a, st);
}

}  // namespace

// Fitted to 29 weight gradients: chunks of a CTA, two of which share an SM, and waves of
// CTAs (us; without the unpacking, measured / estimate in tiles of 64 rows: 1571 rows, 768 x
// 776 8.9 / 10.2, 8192 x 2048 x 512 26 / 27, 2048 x 2048 x 2048 24 / 27, 8192 x 4096 x 1152
// 85 / 84)
double few_grad_w_us(const LinearArgs& l, int nt) {
  const int nk = (l.K + BK - 1) / BK, places = 2 * sm_count();
  const double tiles = static_cast<double>((l.M + nt - 1) / nt) * ((l.N + BM - 1) / BM);
  const int splits = static_cast<int>(std::max(1.0, std::min({8.0, static_cast<double>(nk), places / tiles})));
  return 7.5 + (nt == 128 ? 0.56 : 0.30) * ((nk + splits - 1) / splits) * std::ceil(tiles * splits / places);
}

int few_rows_tile(const LinearArgs& l) {
  // an MN-major operand comes in 64-wide boxes; 128 rows where 64 leave the last wave of
  // CTAs short (with the bias gradient 8192 x 4096 x 1152 79 us instead of 101, 32768 x 11008
  // x 128 236 instead of 294; but 768 x 776 over 1571 rows 16.1 instead of 12.7)
  if (l.kind == GRAD_W) return few_grad_w_us(l, 128) + 3.0 < few_grad_w_us(l, 64) ? 128 : 64;
  int nt = 16;
  // with checkpoints 64 rows at most, whose sums are taken over in segments
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
