// linear_tc.cu -- the three products of an MLP block's linear layers on the
// tensor cores (bf16 operands, fp32 accumulation), each with its epilogue:
//   forward   z = x w^T + bias, y = act(z) + res, checkpoints of z and y
//   back      gx = (gy w) * act'(z) + res, z from its checkpoint
//   grad_w    gw (+)= (gy^T v) * col_scale, v a checkpoint's values in bf16 (exact)
//
// A persistent kernel of CTA pairs: the two CTAs of a cluster share one
// 256 x 256 output tile (tcgen05.mma cta_group::2, M = 256, N = 256, K = 16).
// Each holds 128 of the tile's rows as its A operand and 128 of its columns as
// its half of B, so an operand byte staged in shared memory feeds twice the
// products of a single CTA's 128 x 128 tile; the fp32 accumulator is 128 lanes x
// 256 columns of each CTA's TMEM, two of them, so that the epilogue of one tile
// runs under the products of the next.
//   warp 0     TMA producer (one elected lane issues): 64-deep chunks of this CTA's
//              A and B halves into a ring; the arrivals of both CTAs are counted on
//              the leader's barrier (the leader issues the products of both)
//   warp 1     MMA issuer (the leader's only); commits free the stage in both CTAs
//   warps 4-19  epilogue: four groups of four warps, each 64 columns of the
//              accumulator, a thread a row.  (Two groups of 128 columns a thread left
//              two warps on each scheduler, whose latencies showed: 12544 x 448 ->
//              1792 with gelu and both checkpoints 53 us.)  Two groups share the 128
//              columns of a checkpoint group and exchange the scale byte of their
//              halves' largest magnitudes: the larger byte is the group's
// The tensor cores' fp32 accumulation cuts low bits at every step, which adds
// up over a long contraction (6e-6 of a 8192-token weight gradient).  Where the
// output shows it (fp32 gradients: 16 chunks; and checkpoints, whose codes flip: see
// kShortK) the accumulator holds `seg` chunks at a time and the epilogue threads add the
// segments into registers in ordinary fp32, under the products of the next.
// Operands contracted over their rows (w in back, gy and v in grad_w) are MN-major
// operands read from their natural layout.  The residual comes by TMA into swizzled
// boxes while the products run -- a thread's own row by plain loads touches 32 lines an
// access and doubled the time of 12544 x 448 -> 1792 -- and the results leave through
// the same boxes by TMA stores, which also clip ragged edges; accumulation into gw is
// the TMA's own add (each element is added to once).
//
// Bound: at 8192 x 11008 -> 4096 the tensor cores (393 us, 1.88 PFLOP/s; sustained 444,
// 1.66 PFLOP/s, under the power limit, like a library matrix product of these sizes);
// at 12544 x 448 -> 1792 the epilogue's instructions (20 us plain, 35 with gelu, 42 with
// both checkpoints, for 11 us of products).
#include <utility>

#include "ckpt.cuh"

namespace instant {

namespace {

constexpr int BM = 256, BN = 256, BK = 64;   // tile of a CTA pair; each CTA: 128 rows of A, 128 of B
constexpr uint32_t A_BYTES = 128 * BK * 2;   // 16 KB
constexpr uint32_t B_BYTES = 128 * BK * 2;   // 16 KB
enum { FORWARD = 0, BACK = 1, GRAD_W = 2 };
constexpr uint32_t STAGE = A_BYTES + B_BYTES;
constexpr uint32_t BOX = 128 * 128;          // staging box: 128 rows x 128 bytes
constexpr int kThreads = 640;
// Chunks of a short contraction.  Its forward sums segments of three with or without
// checkpoints, in the same code, so that in this kernel both give the same bits (longer
// contractions and linear_few.cu promise no such thing), and as few of the checkpoints'
// codes differ from those of exact sums as after fp32 sums in order (of the 22 million of
// 12544 x 448 -> 1792 82 to 104, after fp32 sums 78 to 87; with fours 112 to 141).  That
// costs 4 us of 37 against fours there, and 8 of 26 without checkpoints against one
// segment.  Longer ones sum even segments of six at most, and only with checkpoints.
// Values are then 1.2 to 1.4 times (576 to 1024 channels) and 1.0 to 1.2 times (above) as far
// from those of exact sums as after fp32 sums, which is a hundredth of the codes' own
// rounding.  Fours up to 1024 channels, 1.0 to 1.3 times, took 74 us instead of 67 at
// 8192 x 1024 -> 4096 and 20.6 instead of 19.4 at 8192 x 576 -> 1024; eights above, up to 1.5
// times, 80 instead of 85 at 8192 x 1536 -> 4096.
constexpr int kShortK = 8;
// Over a long one the first two segments, whose products run under the epilogue of the
// tile before, are sixteens: with eights that epilogue (7 us) outlasted them and the
// tensor cores stood (8192 x 4096 -> 11008 with gelu and both checkpoints 510 us instead of
// 478, 4096 x 4096 -> 4096 103 instead of 99).
constexpr int kLongK = 64;
// Shared memory: the ring of chunks, the boxes through which epilogue operands
// come in and results go out (64 columns of 128 rows for each group, or of 32 rows
// for each warp that goes through on its own), the tile's bias or column scale, and
// where checkpoints are written, at the cost of a stage, a box of codes for each warp
// and scale bytes under exchange
template <bool KEEP>
struct Lay {
  static constexpr int ns = KEEP ? 4 : 5;
  static constexpr int ins = 16;
  static constexpr uint32_t box = ns * STAGE;
  static constexpr uint32_t vec = box + 4 * BOX;
  static constexpr uint32_t code = vec + (KEEP ? 16 * 32 * 64 : 4 * 64 * 4);
  static constexpr uint32_t bar = code + (KEEP ? 8 * 128 : 0);  // 8 pairs of warps x z, y x 2 halves x 32 bytes
  static constexpr uint32_t total = bar + 8 * (2 * ns + 4 + ins + 1);
};

// ---- cluster-scope barriers and pair-wide tensor-core operations ----------
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// waits for arrivals of both CTAs; gives up like mbar_wait
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  uint32_t n = 0;
  while (!mbar_try_wait_cluster(bar, parity)) {
    if (((++n) & 255u) == 0 && global_timer_ns() - t0 > kWaitLimitNs) return false;
  }
  return true;
}

// one answer for a converged warp
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity)) != 0;
}

// barrier among the `count` threads of an epilogue group or pair of groups.  (An
// id in a register reserves all barriers of the SM; this kernel has it to itself,
// and its epilogue is one piece of code for all groups.)
__device__ __forceinline__ void group_barrier(int id, int count) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// one answer for the threads of a group or pair, which meet at barriers
__device__ __forceinline__ bool mbar_wait_group(uint64_t* bar, uint32_t parity, int id, int count) {
  const uint32_t mine = mbar_wait_cluster(bar, parity) ? 1u : 0u;
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(mine), "r"(id), "r"(count)
      : "memory");
  return all != 0;
}

// Arrival on a barrier of either CTA.  It announces that a slot of TMEM has been
// read, which tcgen05.fence orders; no memory is handed over, so a release at
// CTA scope is enough (one at cluster scope waits for all that its thread has
// under way and took 0.9 us).
__device__ __forceinline__ void mbar_arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

// TMA load into this CTA, completion counted on a barrier of either CTA of the pair
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int c0,
                                                 int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(src)), "r"(c0), "r"(c1)
      : "memory");
}

__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, const void* src, int c0, int c1) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(src)), "r"(c0), "r"(c1)
      : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst_smem)),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}

__device__ __forceinline__ void umma_bf16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                               uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// arrives on the barrier at this offset in both CTAs once every product issued
// so far by this thread has completed
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// output tile t of the grouped order -> (m, n): groups of tiles share columns
// of the B operand in L2
__device__ __forceinline__ void tile_at(const TcArgs& a, int t, int& m, int& n) {
  const int per_group = a.group * a.nt;
  const int gid = t / per_group;
  const int first = gid * a.group;
  const int gsz = min(a.mt - first, a.group);
  const int r = t - gid * per_group;
  m = first + r % gsz;
  n = r / gsz;
}

// piece t of the work: an output tile, and in grad_w a share of its chunks
template <int KIND>
__device__ __forceinline__ void work_at(const TcArgs& a, int t, int& m, int& n, int& share, int& k_lo, int& nk) {
  share = 0;
  k_lo = 0;
  nk = a.nk;
  if (KIND == GRAD_W && a.splits > 1) {
    const int tiles = a.mt * a.nt;
    share = t / tiles;
    t -= share * tiles;
    k_lo = share * a.per;
    nk = min(a.per, a.nk - k_lo);
  }
  tile_at(a, t, m, n);
}

// chunks of a tile's i-th segment: the first two run under the epilogue of the tile before
__device__ __forceinline__ int segment(const TcArgs& a, int i) { return i < 2 ? a.seg01 : a.seg; }

// 32 columns of this warp's 32 lanes, no wait
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
      "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// N columns from taddr into v (N a multiple of 32), loads in flight together
template <int N>
__device__ __forceinline__ void tmem_read(uint32_t taddr, float2* v) {
  uint32_t r[N];
#pragma unroll
  for (int i = 0; i < N / 32; ++i) tmem_ld32_async(taddr + 32 * i, r + 32 * i);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < N / 2; ++i) v[i] = make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
}

// ---------------------------------------------------------------------------
// epilogues: 64 columns of the tile, a row a thread, values in pairs
// ---------------------------------------------------------------------------
// 2 N columns of a row vector of the tile (bias or column scale, fp32 in shared
// memory: one address for the whole warp)
template <int N, bool MUL>
__device__ __forceinline__ void with_row_vector(const float* vec, float2* v) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float4 b = *reinterpret_cast<const float4*>(vec + 2 * i);
    const float2 lo = make_float2(b.x, b.y), hi = make_float2(b.z, b.w);
    v[i] = MUL ? mul2(v[i], lo) : add2(v[i], lo);
    v[i + 1] = MUL ? mul2(v[i + 1], hi) : add2(v[i + 1], hi);
  }
}

// 16-byte piece c of row r of a staging box
__device__ __forceinline__ void put_piece(uint8_t* box, int r, int c, uint4 v) {
  *reinterpret_cast<uint4*>(box + r * 128 + ((c ^ (r & 7)) << 4)) = v;
}

__device__ __forceinline__ uint4 get_piece(const uint8_t* box, int r, int c) {
  return *reinterpret_cast<const uint4*>(box + r * 128 + ((c ^ (r & 7)) << 4));
}

// adds 2 N columns in bf16 from piece c0 of the box on
template <int N>
__device__ __forceinline__ void add_bf16(const uint8_t* box, int r, int c0, float2* v) {
#pragma unroll
  for (int c = 0; c < N / 4; ++c) {
    const uint4 u = get_piece(box, r, c0 + c);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[4 * c + e] = add2(v[4 * c + e], make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u)));
  }
}

// 2 N columns in bf16 from piece c0 of the box on
template <int N>
__device__ __forceinline__ void put_bf16(uint8_t* box, int r, int c0, const float2* v) {
#pragma unroll
  for (int c = 0; c < N / 4; ++c)
    put_piece(box, r, c0 + c,
              make_uint4(pack_bf16x2(v[4 * c].x, v[4 * c].y), pack_bf16x2(v[4 * c + 1].x, v[4 * c + 1].y),
                         pack_bf16x2(v[4 * c + 2].x, v[4 * c + 2].y), pack_bf16x2(v[4 * c + 3].x, v[4 * c + 3].y)));
}

// scale code of the largest of 64 magnitudes
__device__ __forceinline__ uint32_t half_code(const float2* v) {
  float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 32; ++j) m[j & 3] = max_abs3(m[j & 3], v[j].x, v[j].y);
  return ckpt_scale_code(__float_as_uint(max_abs3(max_abs3(m[0], m[1], m[2]), m[3], 0.f)));
}

// codes of 64 columns
__device__ __forceinline__ void make_codes(uint4 (&q)[4], uint32_t code, const float2* v) {
  const float inv = ckpt_inv_scale(code);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float2* w = v + 8 * c;
    if (code != 248u)
      q[c] = make_uint4(ckpt_code4_in_range(w[0], w[1], inv), ckpt_code4_in_range(w[2], w[3], inv),
                        ckpt_code4_in_range(w[4], w[5], inv), ckpt_code4_in_range(w[6], w[7], inv));
    else
      q[c] = make_uint4(ckpt_code4(w[0].x, w[0].y, w[1].x, w[1].y, inv), ckpt_code4(w[2].x, w[2].y, w[3].x, w[3].y, inv),
                        ckpt_code4(w[4].x, w[4].y, w[5].x, w[5].y, inv), ckpt_code4(w[6].x, w[6].y, w[7].x, w[7].y, inv));
  }
}

// One accumulator segment after the other into v, 64 columns of a row a thread.
// `release(acc)` hands the accumulator back; ids and count as in mbar_wait_group.
template <typename Release>
__device__ __forceinline__ bool sum_segments(const TcArgs& a, int nk, uint32_t tbase, uint64_t* t_full, int id,
                                             int count, int& q, float2* v, const Release& release) {
  for (int i = 0, k0 = 0; k0 < nk; k0 += segment(a, i), ++i, ++q) {
    const int acc = q & 1;
    if (!mbar_wait_group(&t_full[acc], (q >> 1) & 1, id, count)) return false;
    tc_fence_after();
    if (k0 == 0) {
      tmem_read<64>(tbase + acc * BN, v);
    } else {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        float w[16];
        tmem_ld16(tbase + acc * BN + 16 * h, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 * h + j] = add2(v[8 * h + j], make_float2(w[2 * j], w[2 * j + 1]));
      }
    }
    release(acc);
  }
  return true;
}

// Forward with checkpoints, or over a short contraction.  A warp takes 32 rows x 64 columns through on its own:
// its own box for the residual and y, its own TMA operations; the codes, 64 bytes of
// a row, through a second box (by plain stores, a row a thread, they took 4 us more at
// 12544 x 448 -> 1792).  It meets only the warp with the other half
// of its rows' checkpoint groups, twice, to exchange the bytes of their largest
// magnitudes.  (With a pair of groups, 256 threads, in step through boxes of 128
// rows the barriers were a third of the epilogue, and 12544 x 448 -> 1792 with gelu and
// both checkpoints took 43 us instead of 36.)
template <int ACT>
__device__ __forceinline__ void epilogue_keep(const TcArgs& a, const CUtensorMap* my, const CUtensorMap* mz,
                                              const CUtensorMap* mk, const CUtensorMap* mr, uint8_t* smem, uint32_t tmem,
                                              uint64_t* t_full, uint64_t* in_full, uint32_t t_empty_leader,
                                              uint32_t rank, int pair, int pairs) {
  using L = Lay<true>;
  const int warp = (threadIdx.x >> 5) - 4, lane = threadIdx.x & 31;
  const int group = warp >> 2, quarter = warp & 3;  // 64 columns, 32 TMEM lanes
  const int half = group & 1;
  const int mate = (group >> 1) * 4 + quarter;      // the two halves of 32 rows' groups
  const int id = 1 + mate, count = 64;
  uint8_t* box = smem + L::box + warp * (32 * 128);
  uint8_t* cbox = smem + L::vec + warp * (32 * 64);  // codes; before them the bias
  float* vec = reinterpret_cast<float*>(cbox);
  uint8_t* zcode = smem + L::code + 128 * mate;  // [half][32]
  uint8_t* ycode = zcode + 64;
  in_full += warp;
  int in_par = 0, q = 0;
  const int tiles = a.mt * a.nt;
  const uint32_t tbase = tmem + 64 * group + (static_cast<uint32_t>(quarter * 32) << 16);
  auto release = [&](int acc) {  // the accumulator may be overwritten
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_at(t_empty_leader + 8 * acc);
  };
  for (int t = pair; t < tiles; t += pairs) {
    int m, n;
    tile_at(a, t, m, n);
    const int row0 = m * BM + static_cast<int>(rank) * 128 + 32 * quarter;
    const int row = row0 + lane;
    const int col = n * BN + 64 * group;
    const bool on = row < a.M && col < a.N;
    const size_t scale_at = static_cast<size_t>(col / kCkptGroup) * a.M + row;
    if (lane == 0) {
      tma_store_wait_read<0>();  // the boxes are free
      if (a.res) {
        mbar_arrive_expect_tx(in_full, 32 * 128);
        tma_load_2d(box, mr, in_full, col, row0);
      }
    }
    __syncwarp();
    if (a.bias) {
      const int c = col + 2 * lane;  // N is even
      float2 b = both(0.f);
      if (c < a.N) {
        const uint32_t u = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.bias) + c);
        b = make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
      }
      *reinterpret_cast<float2*>(vec + 2 * lane) = b;
    }
    float2 v[32];
    if (!sum_segments(a, a.nk, tbase, t_full, id, count, q, v, release)) {
      raise_fault(FAULT_WAIT_DONE);
      break;
    }
    if (a.bias) {
      with_row_vector<32, false>(vec, v);
      __syncwarp();  // codes come over it
    }
    auto keep = [&](const CkptRef& k, const CUtensorMap* map, uint8_t* bytes, bool second) {
      uint32_t code = half_code(v);
      bytes[32 * half + lane] = static_cast<uint8_t>(code);
      group_barrier(id, count);
      code = max(code, static_cast<uint32_t>(bytes[32 * (half ^ 1) + lane]));
      uint4 codes[4];
      make_codes(codes, code, v);
      if (half == 0 && on) k.s[scale_at] = static_cast<uint8_t>(code);
      if (second) {
        // z's codes have left; y, whose store came after theirs, may not
        if (lane == 0) {
          if (a.out) tma_store_wait_read<1>();
          else tma_store_wait_read<0>();
        }
        __syncwarp();
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4*>(cbox + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = codes[c];
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (row0 < a.M && col < a.N) tma_store_2d(map, cbox, col, row0);
        tma_store_commit();
      }
    };
    if (a.zk.q) keep(a.zk, mz, zcode, false);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = act_fast<ACT>(v[j]);
    if (a.res) {
      if (!mbar_wait(in_full, in_par)) raise_fault(FAULT_WAIT_FULL);
      in_par ^= 1;
      add_bf16<32>(box, lane, 0, v);
    }
    if (a.out) {
      put_bf16<32>(box, lane, 0, v);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (row0 < a.M && col < a.N) tma_store_2d(my, box, col, row0);
        tma_store_commit();
      }
    }
    if (a.yk.q) keep(a.yk, mk, ycode, true);
  }
  if (lane == 0) tma_store_wait_all();
}

template <int KIND, int ACT>
__device__ __forceinline__ void epilogue(const TcArgs& a, const CUtensorMap* my, const CUtensorMap* mr, uint8_t* smem,
                                         uint32_t tmem, uint64_t* t_full, uint64_t* in_full,
                                         uint32_t t_empty_leader, uint32_t rank, int pair, int pairs) {
  constexpr bool CODES = KIND == BACK && ACT != INSTANT_ACT_NONE;
  // In back a warp takes its 32 rows through on its own, with its own box and TMA
  // operations (12544 x 448 -> 1792: 24 us instead of 29 with relu', 34 instead of 36
  // with gelu'); forward without checkpoints gains nothing by it and has its bias by group
  constexpr bool ALONE = KIND == BACK;
  using L = Lay<false>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = (warp - 4) >> 2;        // 64 columns each
  const int quarter = 32 * (warp & 3);      // first of the warp's TMEM lanes
  const int r = ALONE ? lane : quarter + lane;  // row of the box
  const int id = 1 + group, count = 128;
  const bool lead = r == 0;                 // issues loads and stores
  constexpr uint32_t kBox = ALONE ? BOX / 4 : BOX;
  const int boxes = ALONE ? warp - 4 : group;
  uint8_t* box = smem + L::box + boxes * kBox;
  in_full += boxes;                         // epilogue operands arrived
  int in_par = 0;
  float* vec = reinterpret_cast<float*>(smem + L::vec) + 64 * group;
  const int tiles = a.mt * a.nt * (KIND == GRAD_W ? a.splits : 1);
  const uint32_t tbase = tmem + 64 * group + (static_cast<uint32_t>(quarter) << 16);
  int q = 0;    // accumulators read so far
  auto release = [&](int acc) {  // the accumulator may be overwritten
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_at(t_empty_leader + 8 * acc);
  };
  for (int t = pair; t < tiles; t += pairs) {
    int m, n, share, k_lo, nk;
    work_at<KIND>(a, t, m, n, share, k_lo, nk);
    const int row0 = m * BM + static_cast<int>(rank) * 128 + (ALONE ? quarter : 0);
    const int col = n * BN + 64 * group;
    const bool on = row0 + r < a.M;
    const bool stores = col < a.N && row0 < a.M;
    if (lead) tma_store_wait_read<0>();  // the box is free
    if (lead && a.res) {
      mbar_arrive_expect_tx(in_full, kBox);
      tma_load_2d(box, mr, in_full, col, row0);
    }
    // the columns' bias or scale, read by the whole group before a barrier that all
    // pass before the next tile, and written before the wait below
    if (a.bias && KIND != BACK && r < 64)
      vec[r] = col + r < a.N ? bf16_to_f32(static_cast<const uint16_t*>(a.bias)[col + r]) : 0.f;
    if (KIND == GRAD_W) {
      float2 v[32];
      if (!sum_segments(a, nk, tbase, t_full, id, count, q, v, release)) {
        raise_fault(FAULT_WAIT_DONE);
        break;
      }
      if (a.bias) with_row_vector<32, true>(vec, v);
      // two boxes of 32 fp32 columns
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1) {
          if (lead) tma_store_wait_read<0>();
          group_barrier(id, count);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float2* w = v + 16 * h + 2 * c;
          put_piece(box, r, c, make_uint4(__float_as_uint(w[0].x), __float_as_uint(w[0].y),
                                          __float_as_uint(w[1].x), __float_as_uint(w[1].y)));
        }
        fence_proxy_async_smem();
        group_barrier(id, count);
        if (lead) {
          const int c0 = col + 32 * h;
          if (c0 < a.N && row0 < a.M) {
            // the shares' products lie one after the other, padded to whole tiles
            if (a.accumulate) tma_add_2d(my, box, c0, row0);
            else tma_store_2d(my, box, c0, share * a.mt * BM + row0);
          }
          tma_store_commit();
        }
      }
    } else {
      // the row's codes, asked for while the products run (by plain loads: half a
      // line a thread, 4% faster here than through a box by TMA)
      uint4 codes[4];
      float scale = 0.f;
      if (CODES) {
        const int8_t* p = a.ck.q + static_cast<size_t>(on ? row0 + r : 0) * a.ld + col;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          codes[c] = on && col + 16 * c < a.N ? *reinterpret_cast<const uint4*>(p + 16 * c)
                                              : make_uint4(0u, 0u, 0u, 0u);
        if (on && col < a.N)
          scale = ckpt_scale(a.ck.s[static_cast<size_t>(col / kCkptGroup) * a.M + row0 + r]);
      }
      const int acc = q & 1;
      const uint32_t par = (q >> 1) & 1;
      if (ALONE ? !mbar_wait_warp(&t_full[acc], par) : !mbar_wait_group(&t_full[acc], par, id, count)) {
        raise_fault(FAULT_WAIT_DONE);
        break;
      }
      if (a.res) {
        if (!mbar_wait(in_full, in_par)) raise_fault(FAULT_WAIT_FULL);
        in_par ^= 1;
      }
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // 32 columns at a time
        float2 v[16];
        tmem_read<32>(tbase + acc * BN + 32 * h, v);
        if (h == 1) release(acc);
        if (KIND == FORWARD) {
          if (a.bias) with_row_vector<16, false>(vec + 32 * h, v);
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = act_fast<ACT>(v[j]);
        } else if (CODES) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint4 w = codes[2 * h + c];
            float2 z[8];
            ckpt_pairs8(make_uint2(w.x, w.y), scale, z);
            ckpt_pairs8(make_uint2(w.z, w.w), scale, z + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[8 * c + e] = mul2(v[8 * c + e], act_slope_fast<ACT>(z[e]));
          }
        }
        if (a.res) add_bf16<16>(box, r, 4 * h, v);
        put_bf16<16>(box, r, 4 * h, v);
      }
      ++q;
      fence_proxy_async_smem();
      if (ALONE) __syncwarp(); else group_barrier(id, count);
      if (lead) {
        if (stores) tma_store_2d(my, box, col, row0);
        tma_store_commit();
      }
    }
  }
  if (lead) tma_store_wait_all();
}

// Column sums of gy on the side (grad_w's bias gradient): the pair kernel's two
// idle warps stream gy from L2 and HBM at a rate that a long product does not
// notice.  A share of the rows of 256 columns a warp, eight rows' loads under way.
__device__ __forceinline__ void side_sums(const TcArgs& a, int w, int warps) {
  const int lane = threadIdx.x & 31;
  const int strips = (a.M + 255) / 256;
  for (int task = w; task < strips * a.sum_parts; task += warps) {
    const int part = task / strips;
    const int c = (task - part * strips) * 256 + 8 * lane;
    if (c >= a.M) continue;
    const int r1 = min(a.K, (part + 1) * a.sum_per);
    const uint16_t* p = static_cast<const uint16_t*>(a.sum_src) + static_cast<size_t>(part) * a.sum_per * a.M + c;
    float2 sum[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = both(0.f);
    auto add = [&](uint4 u) {
      const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sum[e] = add2(sum[e], make_float2(__uint_as_float(x[e] << 16), __uint_as_float(x[e] & 0xffff0000u)));
    };
    int r = part * a.sum_per;
    for (; r + 8 <= r1; r += 8, p += 8 * static_cast<size_t>(a.M)) {
      uint4 u[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = *reinterpret_cast<const uint4*>(p + j * static_cast<size_t>(a.M));
#pragma unroll
      for (int j = 0; j < 8; ++j) add(u[j]);
    }
    for (; r < r1; ++r, p += a.M) add(*reinterpret_cast<const uint4*>(p));
    float* dst = a.sum_part + static_cast<size_t>(part) * a.M + c;
    *reinterpret_cast<float4*>(dst) = make_float4(sum[0].x, sum[0].y, sum[1].x, sum[1].y);
    *reinterpret_cast<float4*>(dst + 4) = make_float4(sum[2].x, sum[2].y, sum[3].x, sum[3].y);
  }
}

// ---------------------------------------------------------------------------
template <int KIND, int ACT, bool KEEP>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    k_linear_tc(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ CUtensorMap map_y, const __grid_constant__ CUtensorMap map_z,
                const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_r, TcArgs a) {
  using L = Lay<KEEP>;
  constexpr int NS = L::ns;
  constexpr bool A_MN = KIND == GRAD_W, B_MN = KIND != FORWARD;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::bar);  // leader's: both CTAs' TMA bytes
  uint64_t* empty = full + NS;       // each CTA's: products of a chunk done
  uint64_t* t_full = empty + NS;     // [2] each CTA's: accumulator done
  uint64_t* t_empty = t_full + 2;    // [2] leader's: accumulator read
  uint64_t* in_full = t_empty + 2;   // [L::ins] each CTA's: epilogue operands arrived
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(in_full + L::ins);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int tiles = a.mt * a.nt * (KIND == GRAD_W ? a.splits : 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&t_full[i], 1);
      mbar_init(&t_empty[i], 32);  // epilogue warps of both CTAs
    }
    for (int i = 0; i < L::ins; ++i) mbar_init(&in_full[i], 1);
    fence_barrier_init();
    prefetch_tmap(&map_a);
    prefetch_tmap(&map_b);
    prefetch_tmap(&map_y);
  }
  if (warp == 0) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait();

  if (warp == 0) {
    // ---------------- producer ----------------
    const uint32_t full_leader = dsmem_addr(full, 0);
    constexpr uint32_t kPairBytes = 2 * STAGE;
    int s = 0, par = 1, issued = 0;  // slot, and parity of its last release (1: never used)
    bool ok = true;
    for (int t = pair; ok && t < tiles; t += pairs) {
      int m, n, share, k_lo, nk;
      work_at<KIND>(a, t, m, n, share, k_lo, nk);
      const int m0 = m * BM + static_cast<int>(rank) * 128;
      const int n0 = n * BN + static_cast<int>(rank) * 128;
      for (int kc = 0; kc < nk; ++kc) {
        if (!mbar_wait_warp(&empty[s], par)) {
          raise_fault(FAULT_WAIT_EMPTY);
          ok = false;
          break;
        }
        if (elect_one()) {
          uint8_t* sa = smem + s * STAGE;
          uint8_t* sb = sa + A_BYTES;
          const uint32_t bar = full_leader + 8 * s;
          const int k0 = (k_lo + kc) * BK;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], kPairBytes);
          if (A_MN) {  // stored [K, M]: two boxes of 64 M x 64 K rows
            tma_load_2d_pair(sa, &map_a, bar, m0, k0);
            tma_load_2d_pair(sa + A_BYTES / 2, &map_a, bar, m0 + 64, k0);
          } else {
            tma_load_2d_pair(sa, &map_a, bar, k0, m0);
          }
          if (B_MN) {
            tma_load_2d_pair(sb, &map_b, bar, n0, k0);
            tma_load_2d_pair(sb + B_BYTES / 2, &map_b, bar, n0 + 64, k0);
          } else {
            tma_load_2d_pair(sb, &map_b, bar, k0, n0);
          }
        }
        __syncwarp();
        ++issued;
        if (++s == NS) {
          s = 0;
          par ^= 1;
        }
      }
    }
    // the last loads have landed before the CTA goes (the leader counts both CTAs')
    par ^= 1;
    for (int k = 0; k < NS && k < issued; ++k) {
      if (--s < 0) {
        s = NS - 1;
        par ^= 1;
      }
      if (rank == 0 && !mbar_wait_cluster(&full[s], par)) raise_fault(FAULT_WAIT_FULL);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer of the pair ----------------
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(BM, BN, A_MN, B_MN);
      // descriptors' address field counts 16 bytes: slots and steps are additions
      const uint32_t base = smem_u32(smem);
      const uint64_t a_desc0 = A_MN ? sdesc_sw128(base, A_BYTES / 2, 1024) : sdesc_sw128(base, 16, 1024);
      const uint64_t b_desc0 =
          B_MN ? sdesc_sw128(base + A_BYTES, B_BYTES / 2, 1024) : sdesc_sw128(base + A_BYTES, 16, 1024);
      int s = 0, par = 0, q = 0;
      bool ok = true;
      for (int t = pair; ok && t < tiles; t += pairs) {
        int m, n, share, k_lo, nk;
        work_at<KIND>(a, t, m, n, share, k_lo, nk);
        int left = 0, acc = 0, i = 0;  // chunks left of the accumulator's segment, segments begun
        for (int kc = 0; kc < nk; ++kc) {
          const bool first = left == 0;
          if (first) {
            acc = q & 1;
            left = min(segment(a, i++), nk - kc);
            if (q >= 2 && !mbar_wait_warp(&t_empty[acc], ((q >> 1) - 1) & 1)) {
              raise_fault(FAULT_WAIT_EMPTY);
              ok = false;
              break;
            }
            ++q;
          }
          if (!mbar_wait_warp(&full[s], par)) {
            raise_fault(FAULT_WAIT_FULL);
            ok = false;
            break;
          }
          tc_fence_after();
          --left;
          if (elect_one()) {
            const uint64_t a_desc = a_desc0 + s * (STAGE >> 4);
            const uint64_t b_desc = b_desc0 + s * (STAGE >> 4);
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              umma_bf16_pair(tmem + acc * BN, a_desc + kk * (A_MN ? 2048 >> 4 : 32 >> 4),
                             b_desc + kk * (B_MN ? 2048 >> 4 : 32 >> 4), idesc, kk == 0 ? !first : 1u);
            umma_commit_pair(&empty[s]);
            if (left == 0) umma_commit_pair(&t_full[acc]);
          }
          __syncwarp();
          if (++s == NS) {
            s = 0;
            par ^= 1;
          }
        }
      }
    }
  } else if (KIND == GRAD_W && warp < 4) {
    if (a.sum_part) side_sums(a, 2 * blockIdx.x + warp - 2, 2 * gridDim.x);
  } else if (warp >= 4) {
    const uint32_t t_empty_leader = dsmem_addr(t_empty, 0);
    if constexpr (KEEP)
      epilogue_keep<ACT>(a, &map_y, &map_z, &map_k, &map_r, smem, tmem, t_full, in_full, t_empty_leader, rank, pair,
                         pairs);
    else
      epilogue<KIND, ACT>(a, &map_y, &map_r, smem, tmem, t_full, in_full, t_empty_leader, rank, pair, pairs);
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // the peer's barriers, operands and accumulator stay until both are done
  if (warp == 0) tmem_dealloc_pair(tmem, 512);
}

template <int KIND, int ACT, bool KEEP>
cudaError_t go(const TcMaps& m, const TcArgs& a, cudaStream_t st) {
  constexpr size_t bytes = Lay<KEEP>::total + 1024;
  auto k = k_linear_tc<KIND, ACT, KEEP>;
  const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(k), bytes);
  if (e != cudaSuccess) return e;
  const long long tiles = static_cast<long long>(a.mt) * a.nt * (KIND == GRAD_W ? a.splits : 1);
  const int pairs = static_cast<int>(tiles < sm_count() / 2 ? tiles : sm_count() / 2);
  return launch_ex(k, dim3(2 * pairs), dim3(kThreads), bytes, st, 1, pdl_enabled(), m.a, m.b, m.y, m.z,
                   m.k, m.r, a);
}

template <int KIND, bool KEEP>
cudaError_t go_act(int act, const TcMaps& m, const TcArgs& a, cudaStream_t st) {
  switch (act) {
    case INSTANT_ACT_RELU: return go<KIND, INSTANT_ACT_RELU, KEEP>(m, a, st);
    case INSTANT_ACT_GELU: return go<KIND, INSTANT_ACT_GELU, KEEP>(m, a, st);
    case INSTANT_ACT_SILU: return go<KIND, INSTANT_ACT_SILU, KEEP>(m, a, st);
    default: return go<KIND, INSTANT_ACT_NONE, KEEP>(m, a, st);
  }
}

bool map2(CUtensorMap* m, const void* p, long long inner, long long outer, long long pitch_bytes,
          int box_inner, int box_outer, CUtensorMapDataType type,
          CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  const uint64_t d[2] = {static_cast<uint64_t>(inner), static_cast<uint64_t>(outer)};
  const uint64_t s[1] = {static_cast<uint64_t>(pitch_bytes)};
  const uint32_t b[2] = {static_cast<uint32_t>(box_inner), static_cast<uint32_t>(box_outer)};
  return make_map(m, p, 2, d, s, b, type, swizzle);
}

}  // namespace

// Every tensor map is encoded before the launch; the caller has checked extents
// and alignment.
cudaError_t launch_linear_tc(const LinearArgs& l, cudaStream_t st) {
  constexpr CUtensorMapDataType kBf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  TcArgs a{};
  a.M = l.M;
  a.N = l.N;
  a.K = l.K;
  a.mt = (l.M + BM - 1) / BM;
  a.nt = (l.N + BN - 1) / BN;
  a.nk = (l.K + BK - 1) / BK;
  a.group = 8;
  const bool keep = l.kind == FORWARD && (l.zk.q || l.yk.q || a.nk <= kShortK);
  const int most = a.nk <= kShortK ? 3 : 6;  // of a forward's segments, which are as even as that allows
  const int segments = (a.nk + most - 1) / most;
  a.seg = l.kind == GRAD_W ? 16 : !keep ? a.nk : (a.nk + segments - 1) / segments;
  a.seg01 = keep && a.nk >= kLongK ? 16 : a.seg;
  a.splits = l.kind == GRAD_W && l.splits > 1 ? l.splits : 1;
  a.per = (a.nk + a.splits - 1) / a.splits;
  if (static_cast<long long>(a.mt) * a.nt * a.splits > 0x7fffffffll - 4096) return cudaErrorInvalidValue;
  a.bias = l.bias;
  a.res = l.res;
  a.out = l.out;
  a.zk = l.zk;
  a.yk = l.yk;
  a.ck = l.ck;
  a.ld = l.ld;
  a.accumulate = l.accumulate;
  if (a.splits > 1) {  // launch_split_sum scales, and adds to gw
    a.bias = nullptr;
    a.out = l.split_part;
    a.accumulate = 0;
  }
  a.sum_src = l.a;
  a.sum_part = l.sum_part;
  a.sum_parts = l.sum_parts;
  a.sum_per = l.sum_per;
  TcMaps m{};
  const int box_rows = l.kind == BACK || keep ? 32 : 128;  // a warp's box or a group's
  bool ok;
  if (l.kind == FORWARD) {
    ok = map2(&m.a, l.a, l.K, l.M, 2ll * l.K, BK, 128, kBf) && map2(&m.b, l.b, l.K, l.N, 2ll * l.K, BK, 128, kBf);
  } else if (l.kind == BACK) {
    ok = map2(&m.a, l.a, l.K, l.M, 2ll * l.K, BK, 128, kBf) && map2(&m.b, l.b, l.N, l.K, 2ll * l.N, 64, BK, kBf);
  } else {
    ok = map2(&m.a, l.a, l.M, l.K, 2ll * l.M, 64, BK, kBf) && map2(&m.b, l.b, l.N, l.K, 2ll * l.N, 64, BK, kBf);
  }
  if (l.kind == GRAD_W)
    ok = ok && map2(&m.y, a.out, l.N, a.splits > 1 ? static_cast<long long>(a.splits) * a.mt * BM : l.M, 4ll * l.N, 32,
                    128, CU_TENSOR_MAP_DATA_TYPE_FLOAT32);
  else if (l.out)
    ok = ok && map2(&m.y, l.out, l.N, l.M, 2ll * l.N, 64, box_rows, kBf);
  for (const auto& [map, q] : {std::make_pair(&m.z, l.zk.q), std::make_pair(&m.k, l.yk.q)})
    if (q) ok = ok && map2(map, q, l.N, l.M, l.ld, 64, 32, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_64B);
  if (l.res) ok = ok && map2(&m.r, l.res, l.N, l.M, 2ll * l.N, 64, box_rows, kBf);
  if (!ok) return cudaErrorInvalidValue;
  if (l.kind == GRAD_W) return go<GRAD_W, INSTANT_ACT_NONE, false>(m, a, st);
  if (l.kind == BACK) return go_act<BACK, false>(l.act, m, a, st);
  return keep ? go_act<FORWARD, true>(l.act, m, a, st) : go_act<FORWARD, false>(l.act, m, a, st);
}

INSTANT_FAULT_READER(read_fault_linear)

}  // namespace instant
