// embed.cu -- the embedding table of a language model: lookup with scaling,
//   y_i = scale T[t_i],
// and the gradient of the table,
//   gT_v (+)= scale sum of g_i over the i with t_i = v.
// A token below zero is no token: its row of y is zero and it has no gradient.
//
// Both are bound by HBM.  The gradient's sums are taken in fp32 in a fixed order, the same
// bits on every call: the positions are sorted by token (stably), eight neighbours of them are
// added in order, then a CTA's eights in order; of a token that lies in many CTAs eight warps
// add every eighth CTA's share, and their sums are added in order.
//   k_embed_sort  up to kSortMax positions in one cluster, in shared memory; more go through
//                 k_sort_count, k_sort_scan (of many) and k_sort_move, eight bits of the
//                 token at a time
//   k_embed_zero  zeros over the table's gradient, while the cluster sorts; up to kSortAlone
//                 positions one CTA sorts, and others of its launch write the zeros
//   k_embed_sum   a warp sums kSegment neighbouring positions of the sorted order in its
//                 registers, all their loads under way at once, and writes each token's
//                 sum; the shares of a token that lies in several warps meet in shared
//                 memory, those of one that lies in several CTAs in the workspace
//   k_embed_join  adds the CTAs' shares, in order (of few positions the CTA of k_embed_sum
//                 whose share comes last)
#include <algorithm>

#include "ckpt.cuh"

namespace instant {

INSTANT_FAULT_READER(read_fault_embed)

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------
__device__ __forceinline__ long long load_token(const void* tokens, int wide, int i) {
  return wide ? static_cast<const long long*>(tokens)[i] : static_cast<const int*>(tokens)[i];
}
// a token's row, -1 for none; one past the table is reported and skipped
__device__ __forceinline__ int table_row(long long t, int V) {
  if (t >= V) {
    raise_fault(FAULT_INDEX);
    return -1;
  }
  return t < 0 ? -1 : static_cast<int>(t);
}

__device__ __forceinline__ uint4 scaled(uint4 u, float s, uint16_t) {
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = pack_bf16x2(__uint_as_float(w[i] << 16) * s, __uint_as_float(w[i] & 0xffff0000u) * s);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 scaled(uint4 u, float s, float) {
  return make_uint4(__float_as_uint(__uint_as_float(u.x) * s), __float_as_uint(__uint_as_float(u.y) * s),
                    __float_as_uint(__uint_as_float(u.z) * s), __float_as_uint(__uint_as_float(u.w) * s));
}

// A unit is a vector of 16 bytes, or one fp32 where rows start on no vector boundary.  A
// CTA takes `cp` neighbouring units (a power of two up to 256) of 256 / cp rows at a
// time, kUnroll such steps under way together, and walks down its rows.
template <typename U>
__device__ __forceinline__ U zero_unit();
template <>
__device__ __forceinline__ uint4 zero_unit<uint4>() { return make_uint4(0, 0, 0, 0); }
template <>
__device__ __forceinline__ float zero_unit<float>() { return 0.f; }

template <typename T>
__device__ __forceinline__ uint4 scaled_unit(uint4 u, float s) { return scaled(u, s, T()); }
template <typename T>
__device__ __forceinline__ float scaled_unit(float u, float s) { return u * s; }

template <typename T, typename U>
__global__ void __launch_bounds__(kThreads)
    k_embed(const void* __restrict__ tokens, int wide, const U* __restrict__ table, U* __restrict__ y, int rows,
            int V, int units, float scale, int cp, int per) {
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x * cp + (threadIdx.x & (cp - 1));
  if (c >= units) return;
  const int step = kThreads / cp;
  const int r1 = min(rows, (static_cast<int>(blockIdx.y) + 1) * per);
  for (int r0 = blockIdx.y * per + static_cast<int>(threadIdx.x) / cp; r0 < r1; r0 += kUnroll * step) {
    long long raw[kUnroll];
    int t[kUnroll];
    U u[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) raw[j] = r0 + j * step < r1 ? load_token(tokens, wide, r0 + j * step) : -1;
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) t[j] = table_row(raw[j], V);
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) u[j] = t[j] >= 0 ? table[static_cast<size_t>(t[j]) * units + c] : zero_unit<U>();
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
      if (r0 + j * step < r1)
        y[static_cast<size_t>(r0 + j * step) * units + c] = t[j] >= 0 ? scaled_unit<T>(u[j], scale) : zero_unit<U>();
  }
}

// ---------------------------------------------------------------------------
// positions sorted by token
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCtas = 8;                         // of the cluster
constexpr int kSortItems = 4;                        // positions a thread, at most
constexpr int kSortMax = kSortThreads * kSortItems * kSortCtas;  // positions it takes
constexpr int kSortAlone = 2 * kSortThreads;         // positions that one CTA sorts by itself
constexpr int kDigits = 256;

// the sort's key: the token, V for none (sorted last)
__device__ __forceinline__ uint32_t sort_key(long long token, int V) {
  const int t = table_row(token, V);
  return static_cast<uint32_t>(t < 0 ? V : t);
}

// How many lanes of the warp with the same digit come before this one, added to the
// warp's counter, which moves on.  Lanes that are not `on` take no part.  The lanes with
// the same digit come from a ballot a bit: with __match_any_sync a sort of 12543
// positions took 43 us instead of 31.
__device__ __forceinline__ int warp_rank(uint32_t digit, bool on, uint32_t* count) {
  const int lane = threadIdx.x & 31;
  unsigned same = __ballot_sync(0xffffffffu, on);
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const bool set = (digit >> b) & 1;
    const unsigned m = __ballot_sync(0xffffffffu, set);
    same &= set ? m : ~m;
  }
  const int leader = on ? __ffs(same) - 1 : lane;
  uint32_t base = 0;
  if (on && lane == leader) {
    base = count[digit];
    count[digit] = base + __popc(same);
  }
  base = __shfl_sync(0xffffffffu, base, leader);
  __syncwarp();
  return static_cast<int>(base) + __popc(same & ((1u << lane) - 1));
}

struct SortShared {
  uint32_t count[kSortWarps][kDigits];
  uint32_t quarter[4][kDigits];  // sums over eight warps each
  uint32_t total[kDigits];       // of this CTA, read by the cluster
  uint32_t base[kDigits];        // where this CTA's positions of a digit begin
  uint32_t red[kDigits / 32];
  uint2 item[kSortThreads * kSortItems];  // key and position, between two passes
};

__device__ __forceinline__ void clear_counts(SortShared& sh) {
  uint4* c = reinterpret_cast<uint4*>(&sh.count[0][0]);
#pragma unroll
  for (int d = 0; d < kSortWarps * kDigits / 4; d += kSortThreads) c[d + threadIdx.x] = make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// count[warp][digit] becomes the sum over the warps before it, total[digit] that over all
__device__ __forceinline__ void scan_warps(SortShared& sh) {
  const int digit = threadIdx.x & (kDigits - 1), q = threadIdx.x / kDigits;
  constexpr int kEach = kSortWarps / 4;
  uint32_t c[kEach], sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    c[i] = sh.count[q * kEach + i][digit];
    sum += c[i];
  }
  sh.quarter[q][digit] = sum;
  __syncthreads();
  uint32_t base = 0;
#pragma unroll
  for (int i = 0; i < 3; ++i) base += i < q ? sh.quarter[i][digit] : 0;
  if (q == 3) sh.total[digit] = base + sum;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    sh.count[q * kEach + i][digit] = base;
    base += c[i];
  }
}

__device__ __forceinline__ uint32_t dsmem_ld_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// CTA `cta` of `ctas` writes its share of zeros over the gradient, which go on beside the sort:
// in CTAs of the same launch where one CTA sorts, else by k_embed_zero, which starts when
// k_embed_sort has waited for everything before it, and whose last CTA's end waits for that one's.
// Short CTAs in the order of memory write 7.28 TB/s here, CTAs that stay on the SMs and take
// every 304th piece 6.4, or a run of their own 5.6 (537 MB).  Zeros that leave out the rows
// which a token names, written by CTAs of k_embed_sum, were slower (8192 tokens, 32768 x
// 4096: 112 us instead of 103; 12543 tokens, 30523 x 449: 34 instead of 28): the table's look-up,
// and reads among the writes.
constexpr int kZeroVecs = 4;  // 16-byte vectors a thread
__device__ __forceinline__ void write_zeros(float* p, size_t n, unsigned cta, unsigned ctas) {
  const size_t vecs = n / 4, step = static_cast<size_t>(ctas) * kSortThreads;
  size_t i = static_cast<size_t>(cta) * kSortThreads + threadIdx.x;
  if (i < n % 4) p[4 * vecs + i] = 0.f;
  for (; i < vecs; i += step) reinterpret_cast<uint4*>(p)[i] = make_uint4(0, 0, 0, 0);
}

// One cluster of up to kSortCtas CTAs (one for kSortAlone positions) sorts all tokens,
// eight bits a pass; keys and positions cross between the CTAs through their shared
// memory, and after the last pass go to a.key and a.pos.  Thread t of warp w of CTA r holds
// the positions (r << part) + w * 32 * items + 32 j + lane, 1 << part a CTA.
// Bound by the latency of its passes, some 2.5 us each (loads of the totals, ranks, two
// barriers of the cluster).
__global__ void __launch_bounds__(kSortThreads) k_embed_sort(const __grid_constant__ EmbedGradArgs a, int items, int part) {
  extern __shared__ __align__(16) uint8_t smem[];
  SortShared& sh = *reinterpret_cast<SortShared*>(smem);
  pdl_wait();
  pdl_launch_dependents();  // not before the wait: k_embed_zero does not wait before it writes
  if (blockIdx.x > 0) {
    write_zeros(a.gtable, static_cast<size_t>(a.V) * a.C, blockIdx.x - 1, gridDim.x - 1);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.z, ctas = gridDim.z;
  const int n = a.rows;
  const int own = warp * 32 * items + lane;
  const int i0 = (rank << part) + own;
  for (int i = tid; i < a.counts; i += kSortThreads) a.count[i] = 0;  // with one CTA only
  uint32_t key[kSortItems], pos[kSortItems];
  {
    long long t[kSortItems];
#pragma unroll
    for (int j = 0; j < kSortItems; ++j)
      t[j] = j < items && i0 + 32 * j < n ? load_token(a.tokens, a.wide, i0 + 32 * j) : -1;
    clear_counts(sh);  // while the tokens come
#pragma unroll
    for (int j = 0; j < kSortItems; ++j) {
      key[j] = sort_key(t[j], a.V);
      pos[j] = i0 + 32 * j;
    }
  }
  __syncthreads();
  for (int bit = 0;; bit += 8) {
    const bool last = (static_cast<uint32_t>(a.V) >> bit) < kDigits;
    int before[kSortItems];
#pragma unroll
    for (int j = 0; j < kSortItems; ++j)
      if (j < items) before[j] = warp_rank((key[j] >> bit) & (kDigits - 1), i0 + 32 * j < n, sh.count[warp]);
    __syncthreads();
    scan_warps(sh);
    cluster_sync();
    if (tid < kDigits) {
      uint32_t c[kSortCtas], all = 0, lower = 0;
#pragma unroll
      for (int r = 0; r < kSortCtas; ++r) c[r] = r < ctas ? dsmem_ld_u32(dsmem_addr(&sh.total[tid], r)) : 0;
#pragma unroll
      for (int r = 0; r < kSortCtas; ++r) {
        lower += r < rank ? c[r] : 0;
        all += c[r];
      }
      uint32_t inc = all;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const uint32_t p = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += p;
      }
      if (lane == 31) sh.red[warp] = inc;
      sh.base[tid] = inc - all + lower;
    }
    __syncthreads();
    if (last) cluster_arrive();  // the totals have been read: after the wait below a CTA may leave
    if (tid < kDigits) {
      uint32_t add = 0;
#pragma unroll
      for (int w = 0; w < kDigits / 32 - 1; ++w) add += w < warp ? sh.red[w] : 0;
      sh.base[tid] += add;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSortItems; ++j) {
      if (j >= items || i0 + 32 * j >= n) break;
      const uint32_t digit = (key[j] >> bit) & (kDigits - 1);
      const uint32_t to = sh.base[digit] + sh.count[warp][digit] + before[j];
      if (last) {
        a.key[to] = key[j];
        a.pos[to] = pos[j];
      } else {
        dsmem_st_u2(dsmem_addr(&sh.item[to & ((1u << part) - 1)], to >> part), make_uint2(key[j], pos[j]));
      }
    }
    __syncwarp();
    if (last) break;
    cluster_arrive();
    __syncthreads();   // count is free
    clear_counts(sh);
    cluster_wait();    // the items have arrived
#pragma unroll
    for (int j = 0; j < kSortItems; ++j)
      if (j < items && i0 + 32 * j < n) {
        const uint2 v = sh.item[own + 32 * j];
        key[j] = v.x;
        pos[j] = v.y;
      }
    __syncthreads();
  }
  cluster_wait();
}

__global__ void __launch_bounds__(kSortThreads) k_embed_zero(float* p, size_t n, int beside) {
  pdl_launch_dependents();
  if (!beside) pdl_wait();
  write_zeros(p, n, blockIdx.x, gridDim.x);
  if (beside && blockIdx.x == gridDim.x - 1) pdl_wait();  // the others make room for CTAs behind them
}

// --- more positions than a cluster holds: tiles of 1024 to 16384 positions, a CTA each, and
// eight bits in two launches: the tiles' counts of each digit, and the move to where they say.
// A CTA of the move adds up the counts of all tiles, work that grows with their square: from
// kScanTiles tiles on k_sort_scan does that between the two, for a launch (us without / with it over
// 50000 x 8: 128 tiles 35.6 / 39.0, 196 54 / 54, 256 64.0 / 58.4, 512 1375 / 1338; over 60000 x 8, 8192
// tiles 30.5 / 24.3 ms).
constexpr int kTileItems = 16;  // positions a thread, at most
constexpr int kScanTiles = 200;
struct SortPass {
  const void* tokens;       // first pass: the tokens, else null
  int wide, V, n, bit, tiles, items;
  const uint32_t *key0, *pos0;
  uint32_t *key, *pos;
  uint32_t* count;          // [tiles][kDigits], and of kScanTiles tiles or more another row
};

__device__ __forceinline__ uint32_t pass_key(const SortPass& p, int i) {
  return p.tokens ? sort_key(load_token(p.tokens, p.wide, i), p.V) : p.key0[i];
}

__global__ void __launch_bounds__(kSortThreads) k_sort_count(const __grid_constant__ SortPass p) {
  __shared__ uint32_t count[kDigits];
  pdl_launch_dependents();
  pdl_wait();
  if (threadIdx.x < kDigits) count[threadIdx.x] = 0;
  __syncthreads();
  const long long tile = static_cast<long long>(p.items) * kSortThreads;
  const int i1 = static_cast<int>(min(static_cast<long long>(p.n), (blockIdx.x + 1) * tile));
  for (int i = static_cast<int>(blockIdx.x * tile) + threadIdx.x; i < i1; i += kSortThreads)
    atomicAdd(&count[(pass_key(p, i) >> p.bit) & (kDigits - 1)], 1u);
  __syncthreads();
  if (threadIdx.x < kDigits) p.count[static_cast<size_t>(blockIdx.x) * kDigits + threadIdx.x] = count[threadIdx.x];
}

// The counts of a digit become the sums over the tiles before, and those over all go to a row
// behind them, so that k_sort_move reads two rows.  A CTA takes 32
// digits, a warp of it neighbouring tiles, each twice.
__global__ void __launch_bounds__(kSortThreads) k_sort_scan(const __grid_constant__ SortPass p) {
  __shared__ uint32_t sum[kSortWarps][32];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int each = (p.tiles + kSortWarps - 1) / kSortWarps;
  const int t0 = min(p.tiles, warp * each), t1 = min(p.tiles, t0 + each);
  uint32_t* count = p.count + blockIdx.x * 32 + lane;
  uint32_t at = 0;
#pragma unroll 8
  for (int t = t0; t < t1; ++t) at += count[static_cast<size_t>(t) * kDigits];
  sum[warp][lane] = at;
  __syncthreads();
  at = 0;
  for (int w = 0; w < warp; ++w) at += sum[w][lane];
  if (warp == kSortWarps - 1) count[static_cast<size_t>(p.tiles) * kDigits] = at + sum[warp][lane];
  for (int t = t0; t < t1; t += 8) {
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = t + i < t1 ? count[static_cast<size_t>(t + i) * kDigits] : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (t + i < t1) count[static_cast<size_t>(t + i) * kDigits] = at;
      at += c[i];
    }
  }
}

// SCANNED: k_sort_scan has been over the counts
template <bool SCANNED>
__global__ void __launch_bounds__(kSortThreads) k_sort_move(const __grid_constant__ SortPass p) {
  __shared__ uint32_t counts[kSortWarps][kDigits];
  __shared__ uint32_t lower[4][kDigits], total[4][kDigits], red[kDigits / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int d = tid; d < kSortWarps * kDigits; d += kSortThreads) (&counts[0][0])[d] = 0;
  // the tiles' counts of each digit, four threads a digit: all of them, and those before this one
  {
    const int digit = tid & (kDigits - 1), q = tid / kDigits;
    uint32_t low = 0, all = 0;
    if constexpr (SCANNED) {
      if (q == 0) {
        low = p.count[static_cast<size_t>(blockIdx.x) * kDigits + digit];
        all = p.count[static_cast<size_t>(p.tiles) * kDigits + digit];
      }
    } else {
#pragma unroll 8
      for (int t = q; t < p.tiles; t += 4) {
        const uint32_t c = p.count[static_cast<size_t>(t) * kDigits + digit];
        all += c;
        low += t < static_cast<int>(blockIdx.x) ? c : 0;
      }
    }
    lower[q][digit] = low;
    total[q][digit] = all;
  }
  __syncthreads();
  const long long i0 = static_cast<long long>(blockIdx.x) * p.items * kSortThreads + warp * 32 * p.items + lane;
  uint32_t key[kTileItems];
  int rank[kTileItems];
#pragma unroll
  for (int j = 0; j < kTileItems; ++j) {
    if (j >= p.items) break;
    const bool on = i0 + 32 * j < p.n;
    key[j] = on ? pass_key(p, static_cast<int>(i0 + 32 * j)) : 0;
    rank[j] = warp_rank((key[j] >> p.bit) & (kDigits - 1), on, counts[warp]);
  }
  // where the digit begins: behind all smaller ones
  uint32_t inc = 0, all = 0;
  if (tid < kDigits) {
    inc = all = total[0][tid] + total[1][tid] + total[2][tid] + total[3][tid];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t q = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += q;
    }
    if (lane == 31) red[warp] = inc;
  }
  __syncthreads();
  if (tid < kDigits) {  // and where the warps' shares of it do
    uint32_t at = inc - all + lower[0][tid] + lower[1][tid] + lower[2][tid] + lower[3][tid];
    for (int w = 0; w < warp; ++w) at += red[w];
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t c = counts[w][tid];
      counts[w][tid] = at;
      at += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kTileItems; ++j) {
    if (j >= p.items || i0 + 32 * j >= p.n) break;
    const int i = static_cast<int>(i0 + 32 * j);
    const uint32_t to = counts[warp][(key[j] >> p.bit) & (kDigits - 1)] + rank[j];
    p.key[to] = key[j];
    p.pos[to] = p.pos0 ? p.pos0[i] : i;
  }
}

// ---------------------------------------------------------------------------
// sums
// ---------------------------------------------------------------------------
constexpr int kSegment = 8;
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = kWarps * kSegment;

// the channels of a lane: W neighbouring ones (VEC), or W at a distance of 32
template <typename T, bool VEC>
struct Lane {
  static constexpr int W = sizeof(T) == 2 ? 8 : 4;
  static constexpr int kStrip = 32 * W;
  int c, C;
  __device__ __forceinline__ Lane(int strip, int C_) : C(C_) {
    c = strip * kStrip + (VEC ? W : 1) * static_cast<int>(threadIdx.x & 31);
  }
  __device__ __forceinline__ bool on(int j) const { return VEC ? c < C : c + 32 * j < C; }
  // row = v scale, or row += v scale with old
  __device__ __forceinline__ void add_to(const float* v, float* row, float scale, bool old) const {
    float q[W] = {};
    if (old) load32(row, q);
    if (VEC) {
      if (c >= C) return;
#pragma unroll
      for (int j = 0; j < W; j += 4) {
        const float4 o = make_float4(fmaf(v[j], scale, q[j]), fmaf(v[j + 1], scale, q[j + 1]),
                                     fmaf(v[j + 2], scale, q[j + 2]), fmaf(v[j + 3], scale, q[j + 3]));
        *reinterpret_cast<float4*>(row + c + j) = o;
      }
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j)
        if (on(j)) row[c + 32 * j] = fmaf(v[j], scale, q[j]);
    }
  }
  __device__ __forceinline__ void prefetch(const float* row) const {
#pragma unroll
    for (int j = 0; j < (VEC ? 1 : W); ++j)
      if (on(j)) asm volatile("prefetch.global.L1 [%0];" ::"l"(row + c + 32 * j));
  }
  __device__ __forceinline__ void load32(const float* row, float* v) const {
    if (VEC) {
      if (c >= C) return;
#pragma unroll
      for (int j = 0; j < W; j += 4) {
        const float4 q = *reinterpret_cast<const float4*>(row + c + j);
        v[j] = q.x, v[j + 1] = q.y, v[j + 2] = q.z, v[j + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] = on(j) ? row[c + 32 * j] : 0.f;
    }
  }
};

template <typename T, bool VEC>
struct Held;  // a lane's channels of one row as loaded
template <>
struct Held<uint16_t, true> {
  uint4 u;
  __device__ __forceinline__ void load(const Lane<uint16_t, true>& l, const uint16_t* row) {
    if (l.c < l.C) u = *reinterpret_cast<const uint4*>(row + l.c);
  }
  __device__ __forceinline__ void add(float* acc) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[2 * i] += __uint_as_float(w[i] << 16);
      acc[2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <bool VEC>
struct Held<float, VEC> {
  float v[4];
  __device__ __forceinline__ void load(const Lane<float, VEC>& l, const float* row) { l.load32(row, v); }
  __device__ __forceinline__ void add(float* acc) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] += v[i];
  }
};

// the last of the blocks that begin with token k, counted on from `block`, which precedes them
__device__ __forceinline__ int last_block(const uint32_t* key, uint32_t k, int block, int blocks) {
  while (true) {
    const int b = block + 1 + static_cast<int>(threadIdx.x & 31);
    const unsigned more = __ballot_sync(0xffffffffu, b < blocks && key[min(b, blocks - 1) * kBlock] == k);
    const int m = more == 0xffffffffu ? 32 : __ffs(~more) - 1;
    block += m;
    if (m < 32) return block;
  }
}

// The shares of token k, whose positions lie in the blocks first..last: eight warps take the
// blocks in turn, and what they add up is added in order.  red: kWarps rows
template <typename L>
__device__ __forceinline__ void add_shares(const EmbedGradArgs& a, const L& l, uint32_t k, int first, int last, int blocks,
                                           float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float acc[L::W] = {};
  if (warp == 0) l.load32(a.part + (static_cast<size_t>(blocks) + first) * a.C, acc);
#pragma unroll 4
  for (int b = first + 1 + warp; b <= last; b += kWarps) {
    float v[L::W] = {};
    l.load32(a.part + static_cast<size_t>(b) * a.C, v);
#pragma unroll
    for (int e = 0; e < L::W; ++e) acc[e] += v[e];
  }
#pragma unroll
  for (int e = 0; e < L::W; ++e) red[32 * (warp * L::W + e) + lane] = acc[e];
  __syncthreads();
  if (warp) return;
#pragma unroll
  for (int w = 1; w < kWarps; ++w)
#pragma unroll
    for (int e = 0; e < L::W; ++e) acc[e] += red[32 * (w * L::W + e) + lane];
  l.add_to(acc, a.gtable + static_cast<size_t>(k) * a.C, a.scale, a.accumulate);
}

// The CTA of `block` has left its share of token k, whose positions lie in several blocks (from
// this one on unless before).  The CTA that finds all the others' shares there adds them.
template <typename L>
__device__ __forceinline__ void join_blocks(const EmbedGradArgs& a, const L& l, uint32_t k, int block, int blocks,
                                            int strip, int strips, bool before, float* red) {
  __shared__ bool all;
  int first = block;
  while (before) {  // back to the block that the token began in
    const int b = first - 1 - static_cast<int>(threadIdx.x & 31);
    const unsigned more = __ballot_sync(0xffffffffu, b > 0 && a.key[max(b, 1) * kBlock - 1] == k);
    const int m = more == 0xffffffffu ? 32 : __ffs(~more) - 1;
    first -= m;
    if (m < 32) break;
  }
  if (before) --first;
  const int last = last_block(a.key, k, block, blocks);
  __syncthreads();  // red and all are free
  if (threadIdx.x == 0) {
    all = atomicAdd(&a.count[static_cast<size_t>(first) * strips + strip], 1u) == static_cast<uint32_t>(last - first);
    __threadfence();
  }
  __syncthreads();
  if (all) add_shares(a, l, k, first, last, blocks, red);
}

// A warp takes kSegment positions of the sorted order and a strip of channels, a CTA kBlock
// positions; a token's shares from several warps meet in shared memory.
// part: [2][blocks][C], the CTA's share of its first token where that began before it, and
// of its last where that began in it and goes on
// inside: those shares are added here, by the CTA that comes last, else by k_embed_join
template <typename T, bool VEC, bool INSIDE>
__global__ void __launch_bounds__(kThreads) k_embed_sum(const __grid_constant__ EmbedGradArgs a, int blocks, int strips) {
  using L = Lane<T, VEC>;
  // a warp's share of its first token, if that began before it, and of its last, if that
  // goes on behind it; the token of the latter
  __shared__ float head_sum[kWarps][32 * L::W], tail_sum[kWarps][32 * L::W];
  __shared__ uint32_t last_key[kWarps], open_key;
  __shared__ bool began[kWarps], through[kWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int block = blockIdx.x / strips;
  const int strip = blockIdx.x % strips;
  const L l(strip, a.C);
  const uint32_t V = a.V;
  if (threadIdx.x == 0) open_key = V;  // of a token that goes on behind the CTA
  const int i0 = block * kBlock + warp * kSegment, n = max(0, min(kSegment, a.rows - i0));
  // lanes 1..kSegment hold the segment's keys, lane 0 the one before it, the next the one after
  uint32_t key = V;
  int pos = 0;
  if (lane <= n + 1 && i0 + lane - 1 >= 0 && i0 + lane - 1 < a.rows) {
    key = a.key[i0 + lane - 1];
    if (lane >= 1 && lane <= n) pos = a.pos[i0 + lane - 1];
  }
  Held<T, VEC> g[kSegment];
#pragma unroll
  for (int j = 0; j < kSegment; ++j) {
    const uint32_t k = __shfl_sync(0xffffffffu, key, j + 1);
    const int p = __shfl_sync(0xffffffffu, pos, j + 1);
    if (j < n && k < V) g[j].load(l, static_cast<const T*>(a.gy) + static_cast<size_t>(p) * a.C);
  }
  if (a.accumulate) {  // the rows that are added to, before their turn comes one by one
#pragma unroll
    for (int j = 0; j < kSegment; ++j) {
      const uint32_t k = __shfl_sync(0xffffffffu, key, j + 1), next = __shfl_sync(0xffffffffu, key, j + 2);
      if (j < n && k < V && next != k) l.prefetch(a.gtable + static_cast<size_t>(k) * a.C);
    }
  }
  const uint32_t k0 = __shfl_sync(0xffffffffu, key, 1);
  const uint32_t before = __shfl_sync(0xffffffffu, key, 0);
  bool head = n > 0 && i0 > 0 && k0 < V && before == k0;  // the first token began before
  if (lane == 0) {
    began[warp] = head;
    through[warp] = false;
    last_key[warp] = V;
  }
  __syncwarp();
  float acc[L::W] = {};
#pragma unroll
  for (int j = 0; j < kSegment; ++j) {
    const uint32_t k = __shfl_sync(0xffffffffu, key, j + 1);
    const uint32_t next = __shfl_sync(0xffffffffu, key, j + 2);
    if (j >= n || k >= V) continue;
    g[j].add(acc);
    const bool goes_on = i0 + j + 1 < a.rows && next == k;
    if (j + 1 < n && goes_on) continue;
    if (head || goes_on) {
      float* to = head ? head_sum[warp] : tail_sum[warp];
#pragma unroll
      for (int e = 0; e < L::W; ++e) to[32 * e + lane] = acc[e];
      if (lane == 0) {
        if (head) through[warp] = goes_on;
        else last_key[warp] = k;
      }
    } else {
      l.add_to(acc, a.gtable + static_cast<size_t>(k) * a.C, a.scale, a.accumulate);
    }
    head = false;
#pragma unroll
    for (int e = 0; e < L::W; ++e) acc[e] = 0.f;
  }
  __syncthreads();
  // Tokens that lie in several warps: the warp that one began in adds the shares of
  // those behind it, and warp 0 those of one that began before the CTA
  auto follow = [&](int w, bool& open) {  // shares of warps w, w + 1, ... of the token that goes on into w
    open = true;
    for (; w < kWarps && open; ++w) {
#pragma unroll
      for (int e = 0; e < L::W; ++e) acc[e] += head_sum[w][32 * e + lane];
      open = through[w];
    }
  };
  if (warp == 0 && began[0]) {
    bool open;
    follow(0, open);
    l.add_to(acc, a.part + static_cast<size_t>(block) * a.C, 1.f, false);
#pragma unroll
    for (int e = 0; e < L::W; ++e) acc[e] = 0.f;
  }
  const uint32_t k = last_key[warp];
  if (k < V) {
#pragma unroll
    for (int e = 0; e < L::W; ++e) acc[e] = tail_sum[warp][32 * e + lane];
    bool open;
    follow(warp + 1, open);
    if (open) {
      l.add_to(acc, a.part + (static_cast<size_t>(blocks) + block) * a.C, 1.f, false);
      if (lane == 0) open_key = k;
    } else {
      l.add_to(acc, a.gtable + static_cast<size_t>(k) * a.C, a.scale, a.accumulate);
    }
  }
  if (!INSIDE) return;
  __syncthreads();
  if (!began[0] && open_key >= V) return;
  __threadfence();
  __syncthreads();
  if (began[0]) join_blocks(a, l, a.key[block * kBlock], block, blocks, strip, strips, true, &head_sum[0][0]);
  if (open_key < V) join_blocks(a, l, open_key, block, blocks, strip, strips, false, &head_sum[0][0]);
}

// the tokens whose positions lie in several CTAs of k_embed_sum
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) k_embed_join(const __grid_constant__ EmbedGradArgs a, int blocks) {
  using L = Lane<T, VEC>;
  __shared__ float red[kWarps * 32 * L::W];
  pdl_launch_dependents();
  pdl_wait();
  const int block = blockIdx.x;
  const int end = (block + 1) * kBlock;  // the next block's first position
  const uint32_t k = a.key[end - 1], k1 = a.key[end], k0 = block > 0 ? a.key[end - kBlock - 1] : a.V;
  if (k >= static_cast<uint32_t>(a.V) || k1 != k) return;  // ends here
  if (k0 == k) return;                                      // began before
  add_shares(a, L(blockIdx.y, a.C), k, block, last_block(a.key, k, block, blocks), blocks, red);
}

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// smallest power of two that is at least n, or `most`
int pow2_up(int n, int most) {
  int p = 1;
  while (p < n && p < most) p *= 2;
  return p;
}

int blocks_of(int rows) { return (rows + kBlock - 1) / kBlock; }
int strip_of(int C, bool bf16) {
  return bf16 ? Lane<uint16_t, true>::kStrip : C % 4 == 0 ? Lane<float, true>::kStrip : Lane<float, false>::kStrip;
}
// positions a thread of a tile, a power of two: two tiles an SM where there are enough (counted from the one
// device this library is built for, so that the workspace's size needs no device)
int tile_items(int rows) {
  int n = 1;
  while (n < kTileItems && static_cast<long long>(rows) > 2ll * kColSumSMs * n * kSortThreads) n *= 2;
  return n;
}
int tiles_of(int rows) {
  const long long tile = static_cast<long long>(tile_items(rows)) * kSortThreads;
  return static_cast<int>((rows + tile - 1) / tile);
}
size_t count_bytes(int rows) {  // a row of counts a tile, and one of sums
  const int tiles = tiles_of(rows);
  return up256(static_cast<size_t>(tiles + (tiles >= kScanTiles)) * kDigits * 4);
}

}  // namespace

size_t embed_grad_bytes(int rows, int C) {
  const size_t words = up256(static_cast<size_t>(rows) * 4);
  const size_t sort = rows <= kSortMax ? 2 * words : 4 * words + count_bytes(rows);
  const size_t strips = (C + strip_of(C, false) - 1) / strip_of(C, false);  // bf16 has half as many
  const size_t counts = rows <= kSortAlone ? up256(blocks_of(rows) * strips * 4) : 0;
  return sort + counts + static_cast<size_t>(2) * blocks_of(rows) * C * 4;
}

cudaError_t launch_embed(const void* tokens, int wide, const void* table, void* y, int rows, int V, int C, float scale,
                         bool bf16, cudaStream_t st) {
  const bool vec = bf16 || C % 4 == 0;
  const int units = bf16 ? C / 8 : vec ? C / 4 : C;
  const int cp = pow2_up(units, kThreads);
  const long long columns = (units + cp - 1) / cp;
  // about 16 CTAs an SM, whole batches of rows, no more CTAs a column than a grid has in y
  const int pass = kUnroll * kThreads / cp;
  const long long want = std::max(1ll, 16ll * sm_count() / columns);
  long long per = std::max((rows + want - 1) / want, (static_cast<long long>(rows) + 65534) / 65535);
  per = (per + pass - 1) / pass * pass;
  const dim3 grid(static_cast<unsigned>(columns), static_cast<unsigned>((rows + per - 1) / per));
  auto go = [&](auto kernel, auto* t, auto* o) {
    return launch_ex(kernel, grid, dim3(kThreads), 0, st, 1, pdl_enabled(), tokens, wide, t, o, rows, V, units, scale,
                     cp, static_cast<int>(per));
  };
  if (bf16) return go(k_embed<uint16_t, uint4>, static_cast<const uint4*>(table), static_cast<uint4*>(y));
  if (vec) return go(k_embed<float, uint4>, static_cast<const uint4*>(table), static_cast<uint4*>(y));
  return go(k_embed<float, float>, static_cast<const float*>(table), static_cast<float*>(y));
}

cudaError_t launch_embed_grad(EmbedGradArgs a, void* ws, bool bf16, cudaStream_t st) {
  const int n = a.rows;
  uint8_t* w = static_cast<uint8_t*>(ws);
  const size_t words = up256(static_cast<size_t>(n) * 4);
  auto take = [&](size_t bytes) {
    uint32_t* p = reinterpret_cast<uint32_t*>(w);
    w += bytes;
    return p;
  };
  a.key = take(words);
  a.pos = take(words);
  const int blocks = blocks_of(n), strips = (a.C + strip_of(a.C, bf16) - 1) / strip_of(a.C, bf16);
  const long long sums = static_cast<long long>(blocks) * strips;
  if (sums > 0x7fffffffll) return cudaErrorInvalidValue;
  // Few positions are two launches (one CTA sorts while others of its launch write the zeros;
  // tokens over several CTAs are added up by the last of them), more are four: a call for 300
  // positions takes 5 us less of the host, but the fences of such CTAs cost 8192 positions over
  // 32768 x 4096 103.8 us instead of 99.4, 12543 over 30523 x 449 26.6 instead of 23.8.
  const bool alone = n <= kSortAlone;
  a.counts = alone ? static_cast<int>(sums) : 0;
  a.count = take(alone ? up256(static_cast<size_t>(sums) * 4) : 0);
  const size_t values = static_cast<size_t>(a.V) * a.C, each = 4 * kZeroVecs * kSortThreads;
  const unsigned zeros = a.accumulate ? 0 : static_cast<unsigned>((values + each - 1) / each);
  const bool one = n <= kSortMax;
  cudaError_t e = cudaSuccess;
  if (one) {
    const int ctas = alone ? 1 : kSortCtas;
    int items = 1, part = 10;  // powers of two, so that a position's CTA is a shift away
    while (ctas * items * kSortThreads < n) items *= 2, ++part;
    e = raise_smem_limit(reinterpret_cast<const void*>(k_embed_sort), sizeof(SortShared));
    if (e == cudaSuccess)
      e = launch_ex(k_embed_sort, dim3(alone ? 1 + zeros : 1, 1, ctas), dim3(kSortThreads), sizeof(SortShared), st,
                    ctas, pdl_enabled(), a, items, part);
  }
  if (e == cudaSuccess && zeros > 0 && !alone)
    e = launch_ex(k_embed_zero, dim3(zeros), dim3(kSortThreads), 0, st, 1, pdl_enabled(), a.gtable, values, one ? 1 : 0);
  if (!one) {
    SortPass p{};
    p.tokens = a.tokens;
    p.wide = a.wide;
    p.V = a.V;
    p.n = n;
    p.tiles = tiles_of(n);
    p.items = tile_items(n);
    uint32_t* key1 = take(words);
    uint32_t* pos1 = take(words);
    p.count = take(count_bytes(n));
    const bool scan = p.tiles >= kScanTiles;
    int passes = 1;
    while (passes < 4 && (static_cast<uint32_t>(a.V) >> (8 * passes)) != 0) ++passes;
    // the last pass ends in a.key, a.pos
    for (int i = 0; i < passes && e == cudaSuccess; ++i) {
      const bool last = (passes - 1 - i) % 2 == 0;
      p.bit = 8 * i;
      p.key = last ? a.key : key1;
      p.pos = last ? a.pos : pos1;
      e = launch_ex(k_sort_count, dim3(p.tiles), dim3(kSortThreads), 0, st, 1, pdl_enabled(), p);
      if (e == cudaSuccess && scan)
        e = launch_ex(k_sort_scan, dim3(kDigits / 32), dim3(kSortThreads), 0, st, 1, pdl_enabled(), p);
      if (e == cudaSuccess)
        e = launch_ex(scan ? k_sort_move<true> : k_sort_move<false>, dim3(p.tiles), dim3(kSortThreads), 0, st, 1,
                      pdl_enabled(), p);
      p.tokens = nullptr;
      p.key0 = p.key;
      p.pos0 = p.pos;
    }
  }
  if (e != cudaSuccess) return e;
  a.part = reinterpret_cast<float*>(w);
  auto go = [&](auto inside, auto sum, auto join) {
    cudaError_t r = launch_ex(alone ? inside : sum, dim3(static_cast<unsigned>(sums)), dim3(kThreads), 0, st, 1,
                              pdl_enabled(), a, blocks, strips);
    if (r == cudaSuccess && !alone)
      r = launch_ex(join, dim3(blocks - 1, strips), dim3(kThreads), 0, st, 1, pdl_enabled(), a, blocks);
    return r;
  };
  if (bf16)
    return go(k_embed_sum<uint16_t, true, true>, k_embed_sum<uint16_t, true, false>, k_embed_join<uint16_t, true>);
  if (a.C % 4 == 0)
    return go(k_embed_sum<float, true, true>, k_embed_sum<float, true, false>, k_embed_join<float, true>);
  return go(k_embed_sum<float, false, true>, k_embed_sum<float, false, false>, k_embed_join<float, false>);
}

}  // namespace instant
