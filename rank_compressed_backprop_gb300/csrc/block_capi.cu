// block_capi.cu -- the extern "C" boundary of the MLP-block operators declared
// in include/instant.h (norm, products with epilogues, 8-bit checkpoints):
// argument validation and launch planning.  No device memory is allocated here.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "instant.h"
#include "kernels.h"

using namespace instant;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int cdiv(int a, int b) { return (a + b - 1) / b; }
bool dtype_ok(instant_dtype dt) { return dt == INSTANT_F32 || dt == INSTANT_BF16; }
bool act_ok(int act) { return act >= INSTANT_ACT_NONE && act <= INSTANT_ACT_SILU; }
instant_status from_cuda(cudaError_t e) { return e == cudaSuccess ? INSTANT_OK : INSTANT_ERR_CUDA; }

// largest extents: row counts rounded up to a tile and padded rows stay within an int
bool extent_ok(int rows, int C) { return rows >= 1 && rows <= (1 << 30) && C >= 1 && C <= (1 << 24); }

// a checkpoint's two arrays come together
bool pair_ok(const void* q, const void* s) { return (q == nullptr) == (s == nullptr); }

CkptRef ref(const void* q, const void* s) {
  CkptRef r;
  r.q = static_cast<int8_t*>(const_cast<void*>(q));
  r.s = static_cast<uint8_t*>(const_cast<void*>(s));
  return r;
}

// bf16 rows are read and written in whole vectors of eight channels; fp32 rows
// may be any width and are where C allows it
bool align_ok(instant_dtype dt, int C) { return dt == INSTANT_F32 || C % 8 == 0; }
bool vec_ok(int C) { return C % 8 == 0; }

// pieces of 256 x 256 x 64 chunks on the CTA pairs
double pairs_us(double pieces, int chunks, int sms) {
  return 4.5 + 0.30 * chunks * std::ceil(pieces / std::max(1, sms / 2));
}

// the partial products' way to memory and back through launch_split_sum
double split_sum_us(int splits, int M, int N) {
  return splits > 1 ? 3.0 + 4e-6 * splits * M * N / 4.0 : 0.0;
}

// Shares of the rows into which the pair kernel cuts a weight gradient [M, N] over K
// rows: its tiles are few (14 at 1792 x 448) and its rows many, so that without them
// most pairs stand idle (us, without shares and the split-K kernel in their place / with:
// 12544 x 448 x 1792 33.7 / 24.3, 16384 x 768 x 768 28 / 25.3, 9728 x 448 x 2048 24.9 /
// 23).  A gain of less than a tenth is left: at 16384 x 4096 x 4096 the estimate saw 1 %
// in two shares and they took 348 instead of 340.  Counted from the SMs of the one device
// this library is built for: the workspace's size needs no device.
int grad_w_splits(int M, int N, int K) {
  const double tiles = static_cast<double>(cdiv(M, 256)) * cdiv(N, 256);
  const int chunks = cdiv(K, 64);
  int best = 1;
  double best_us = 0.9 * pairs_us(tiles, chunks, kColSumSMs);
  for (int n = 2; n <= kMaxSplits; ++n) {
    const int per = cdiv(chunks, n);
    if (cdiv(chunks, per) != n) continue;  // an empty share
    const double us = pairs_us(tiles * n, per, kColSumSMs) + split_sum_us(n, M, N);
    if (us < best_us) {
      best = n;
      best_us = us;
    }
  }
  return best;
}

// bf16 products run on the tensor cores, fp32 ones on FFMA.  Of the two tensor-core
// kernels the one with the smaller estimate runs:
//   CTA pairs, 256 x 256 tiles      4.5 us + 0.30 us a chunk of 64 and wave of 76 tiles
//   split K, 128 x NT tiles         8 us + 0.28 us (NT = 128), 0.15 (64) or 0.13 a
//                                   chunk, over the SMs; weight gradients: few_grad_w_us
// which are fits to both kernels timed over 21 shapes of forward and of back and 29 of the
// weight gradient.  Measured
// (rows x K -> N, split K against pairs, us): forward 1 x 4096 -> 11008 15.8 / 40.5,
// 128 x 4096 -> 11008 21.7 / 25.1, 256 x 4096 -> 11008 32.7 / 25.3, 512 x 1024 -> 1024
// 9.6 / 8.8, 2048 x 2048 -> 2048 19.3 / 14.8; back 33 x 11008 -> 4096 17.5 / 50.3,
// 1024 x 4096 -> 1024 14.4 / 21.6; weight gradient with the unpacking before it
// over 700 rows, 1792 x 448 8.4 / 9.8, over 8192, 256 x 256 11.4 / 13.7, 768 x 768 20 / 20,
// 4096 x 1024 84 / 48.
double pairs_us(const LinearArgs& a) {
  const int splits = std::max(1, a.splits);
  return pairs_us(static_cast<double>(cdiv(a.M, 256)) * cdiv(a.N, 256) * splits, cdiv(cdiv(a.K, 64), splits),
                  sm_count()) +
         split_sum_us(splits, a.M, a.N);
}

bool runs_on_pairs(const LinearArgs& a) {
  const int nt = few_rows_tile(a);
  if (cdiv(a.M, nt) > kFewMaxRowTiles) return true;  // narrow products of millions of rows
  if (a.kind == 2) return pairs_us(a) <= few_grad_w_us(a, nt);
  const double chunk_us = nt == 128 ? 0.28 : nt == 64 ? 0.15 : 0.13;
  return pairs_us(a) <= 8.0 + chunk_us * cdiv(a.K, 64) * cdiv(a.N, 128) * cdiv(a.M, nt) / sm_count();
}

cudaError_t launch_linear(const LinearArgs& a, bool bf16, cudaStream_t st) {
  if (!bf16) return launch_linear_simt(a, st);
  return runs_on_pairs(a) ? launch_linear_tc(a, st) : launch_linear_few(a, st);
}

}  // namespace

extern "C" {

instant_status instant_ckpt_pack(const void* x, void* q, void* s, int rows, int C, instant_dtype dt,
                                 void* stream) {
  if (!dtype_ok(dt)) return INSTANT_ERR_DTYPE;
  if (!x || !q || !s) return INSTANT_ERR_ARG;
  if (!extent_ok(rows, C)) return INSTANT_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(q) || !align_ok(dt, C)) return INSTANT_ERR_ALIGN;
  return from_cuda(launch_ckpt_pack(x, ref(q, s), rows, C, dt == INSTANT_BF16, vec_ok(C),
                                    static_cast<cudaStream_t>(stream)));
}

instant_status instant_ckpt_unpack(const void* q, const void* s, void* x, int rows, int C,
                                   instant_dtype dt, void* stream) {
  if (!dtype_ok(dt)) return INSTANT_ERR_DTYPE;
  if (!x || !q || !s) return INSTANT_ERR_ARG;
  if (!extent_ok(rows, C)) return INSTANT_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(q) || !align_ok(dt, C)) return INSTANT_ERR_ALIGN;
  return from_cuda(launch_ckpt_unpack(ref(q, s), x, rows, C, dt == INSTANT_BF16, vec_ok(C),
                                      static_cast<cudaStream_t>(stream)));
}

instant_status instant_rms_norm(const void* x, const void* residual, const void* gamma, void* h,
                                void* y, void* q, void* s, float* r, int rows, int C, float eps,
                                instant_dtype dt, void* stream) {
  if (!dtype_ok(dt)) return INSTANT_ERR_DTYPE;
  if (!x || !gamma || !(y || q) || !pair_ok(q, s) || !(eps >= 0.f)) return INSTANT_ERR_ARG;
  if (!extent_ok(rows, C) || C > INSTANT_RMS_NORM_MAX_C) return INSTANT_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(gamma) || !aligned16(h) || !aligned16(y) ||
      !aligned16(q) || !align_ok(dt, C))
    return INSTANT_ERR_ALIGN;
  NormArgs a;
  a.x = x;
  a.res = residual;
  a.gamma = gamma;
  a.h = h;
  a.y = y;
  a.k = ref(q, s);
  a.r = r;
  a.rows = rows;
  a.C = C;
  a.ld = ckpt_ld(C);
  a.vec = vec_ok(C);
  a.eps = eps;
  return from_cuda(launch_rms_norm(a, dt == INSTANT_BF16, static_cast<cudaStream_t>(stream)));
}

size_t instant_rms_norm_backward_workspace_bytes(int rows, int C) {
  if (!extent_ok(rows, C) || C > INSTANT_RMS_NORM_MAX_C) return 0;
  return static_cast<size_t>(norm_back_parts(rows, C)) * C * sizeof(float);
}

instant_status instant_rms_norm_backward(const void* gy, const void* q, const void* s, const float* r,
                                         const void* gamma, const void* residual, void* gx,
                                         float* ggamma, int accumulate, void* ws, size_t ws_bytes,
                                         int rows, int C, instant_dtype dt, void* stream) {
  if (!dtype_ok(dt)) return INSTANT_ERR_DTYPE;
  if (!gy || !q || !s || !r || !gamma || !gx || !ggamma) return INSTANT_ERR_ARG;
  if (!extent_ok(rows, C) || C > INSTANT_RMS_NORM_MAX_C) return INSTANT_ERR_SHAPE;
  if (!ws || ws_bytes < instant_rms_norm_backward_workspace_bytes(rows, C)) return INSTANT_ERR_WORKSPACE;
  if (!aligned16(gy) || !aligned16(q) || !aligned16(gamma) || !aligned16(residual) || !aligned16(gx) ||
      !aligned16(ggamma) || !aligned16(ws) || !align_ok(dt, C))
    return INSTANT_ERR_ALIGN;
  NormBackArgs a;
  a.gy = gy;
  a.gamma = gamma;
  a.res = residual;
  a.gx = gx;
  a.k = ref(q, s);
  a.r = r;
  a.part = static_cast<float*>(ws);
  a.ggamma = ggamma;
  a.rows = rows;
  a.C = C;
  a.ld = ckpt_ld(C);
  a.vec = vec_ok(C);
  a.accumulate = accumulate != 0;
  return from_cuda(launch_rms_norm_back(a, dt == INSTANT_BF16, static_cast<cudaStream_t>(stream)));
}

instant_status instant_linear_act(const void* x, const void* w, const void* bias, const void* residual,
                                  void* y, void* zq, void* zs, void* yq, void* ys, int rows, int Cx,
                                  int Cy, instant_act act, instant_dtype dt, void* stream) {
  if (!dtype_ok(dt)) return INSTANT_ERR_DTYPE;
  if (!x || !w || !(y || yq) || !pair_ok(zq, zs) || !pair_ok(yq, ys) || !act_ok(act))
    return INSTANT_ERR_ARG;
  if (!extent_ok(rows, Cx) || !extent_ok(rows, Cy)) return INSTANT_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(w) || !aligned16(bias) || !aligned16(residual) || !aligned16(y) ||
      !aligned16(zq) || !aligned16(yq) || !align_ok(dt, Cx) || !align_ok(dt, Cy))
    return INSTANT_ERR_ALIGN;
  LinearArgs a{};
  a.kind = 0;
  a.M = rows;
  a.N = Cy;
  a.K = Cx;
  a.a = x;
  a.b = w;
  a.bias = bias;
  a.res = residual;
  a.out = y;
  a.zk = ref(zq, zs);
  a.yk = ref(yq, ys);
  a.ld = ckpt_ld(Cy);
  a.act = act;
  return from_cuda(launch_linear(a, dt == INSTANT_BF16, static_cast<cudaStream_t>(stream)));
}

instant_status instant_linear_act_grad(const void* gy, const void* w, const void* zq, const void* zs,
                                       const void* residual, void* gx, int rows, int Cx, int Cy,
                                       instant_act act, instant_dtype dt, void* stream) {
  if (!dtype_ok(dt)) return INSTANT_ERR_DTYPE;
  if (!gy || !w || !gx || !pair_ok(zq, zs) || !act_ok(act) || (act != INSTANT_ACT_NONE && !zq))
    return INSTANT_ERR_ARG;
  if (!extent_ok(rows, Cx) || !extent_ok(rows, Cy)) return INSTANT_ERR_SHAPE;
  if (!aligned16(gy) || !aligned16(w) || !aligned16(zq) || !aligned16(residual) || !aligned16(gx) ||
      !align_ok(dt, Cx) || !align_ok(dt, Cy))
    return INSTANT_ERR_ALIGN;
  LinearArgs a{};
  a.kind = 1;
  a.M = rows;
  a.N = Cx;
  a.K = Cy;
  a.a = gy;
  a.b = w;
  a.res = residual;
  a.out = gx;
  a.ck = ref(zq, zs);
  a.ld = ckpt_ld(Cx);
  a.act = act;
  return from_cuda(launch_linear(a, dt == INSTANT_BF16, static_cast<cudaStream_t>(stream)));
}

// the checkpoint's values in bf16, then the row shares of gb
static size_t values_bytes(int rows, int Cx) {
  return (static_cast<size_t>(rows) * Cx * 2 + 255) & ~static_cast<size_t>(255);
}

static size_t sums_bytes(int rows, int Cy) {
  return (static_cast<size_t>(col_sum_parts(rows, Cy)) * Cy * sizeof(float) + 255) & ~static_cast<size_t>(255);
}
static size_t splits_bytes(int rows, int Cx, int Cy) {
  const int splits = grad_w_splits(Cy, Cx, rows);
  return splits > 1 ? static_cast<size_t>(splits) * cdiv(Cy, 256) * 256 * Cx * sizeof(float) : 0;
}

size_t instant_ckpt_grad_w_workspace_bytes(int rows, int Cx, int Cy) {
  if (!extent_ok(rows, Cx) || !extent_ok(rows, Cy)) return 0;
  return values_bytes(rows, Cx) + sums_bytes(rows, Cy) + splits_bytes(rows, Cx, Cy);
}

instant_status instant_ckpt_grad_w(const void* gy, const void* q, const void* s, const void* col_scale,
                                   float* gw, float* gb, int accumulate, void* ws, size_t ws_bytes,
                                   int rows, int Cx, int Cy, instant_dtype dt, void* stream) {
  if (!dtype_ok(dt)) return INSTANT_ERR_DTYPE;
  if (!gy || !q || !s || !gw) return INSTANT_ERR_ARG;
  if (!extent_ok(rows, Cx) || !extent_ok(rows, Cy)) return INSTANT_ERR_SHAPE;
  if ((gb || dt == INSTANT_BF16) && (!ws || ws_bytes < instant_ckpt_grad_w_workspace_bytes(rows, Cx, Cy)))
    return INSTANT_ERR_WORKSPACE;
  if (!aligned16(gy) || !aligned16(q) || !aligned16(col_scale) || !aligned16(gw) || !aligned16(gb) ||
      !aligned16(ws) || !align_ok(dt, Cx) || !align_ok(dt, Cy))
    return INSTANT_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf16 = dt == INSTANT_BF16;
  LinearArgs a{};
  a.kind = 2;
  a.M = Cy;
  a.N = Cx;
  a.K = rows;
  a.a = gy;
  a.bias = col_scale;
  a.out = gw;
  a.ck = ref(q, s);
  a.ld = ckpt_ld(Cx);
  a.accumulate = accumulate != 0;
  float* part = gb ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + values_bytes(rows, Cx)) : nullptr;
  if (!bf16) {
    cudaError_t e = launch_linear(a, bf16, st);
    if (e == cudaSuccess && gb)
      e = launch_col_sum(static_cast<const float*>(gy), gb, part, rows, Cy, accumulate != 0, vec_ok(Cy), st);
    return from_cuda(e);
  }
  // the values are exact in bf16 and every row tile of gw reads them: made once
  a.b = ws;
  a.splits = grad_w_splits(Cy, Cx, rows);
  a.split_part =
      reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + values_bytes(rows, Cx) + sums_bytes(rows, Cy));
  const bool pairs = runs_on_pairs(a);
  // gb's shares on the side of a product long enough for the pair kernel's idle warps
  // to read gy, which they do at about 0.8 TB/s over all pairs (32768 rows, 64 x 64, on 8 of
  // the 76: 45 us instead of 25); else in the launch that makes the values
  int parts = 0;
  cudaError_t e;
  const double busy = std::min(1.0, static_cast<double>(cdiv(Cy, 256)) * cdiv(Cx, 256) * a.splits / (kColSumSMs / 2));
  if (gb && !(pairs && 2e-6 * rows * Cy / (0.8 * busy) <= pairs_us(a))) {
    e = launch_unpack_and_sum(a.ck, ws, rows, Cx, gy, part, Cy, &parts, st);
  } else {
    e = launch_ckpt_unpack(a.ck, ws, rows, Cx, true, true, st);
    if (gb) {
      a.sum_part = part;
      a.sum_parts = std::min(col_sum_parts(rows, Cy), std::max(1, 2 * kColSumSMs / cdiv(Cy, 256)));
      a.sum_per = cdiv(rows, a.sum_parts);
      parts = a.sum_parts = cdiv(rows, a.sum_per);
    }
  }
  if (e == cudaSuccess) e = launch_linear(a, bf16, st);
  if (e == cudaSuccess && pairs && a.splits > 1)
    e = launch_split_sum(a.split_part, a.splits, gw, col_scale, Cy, Cx, accumulate != 0, st);
  if (e == cudaSuccess && gb) e = launch_part_sum(part, gb, parts, Cy, accumulate != 0, st);
  return from_cuda(e);
}

}  // extern "C"
