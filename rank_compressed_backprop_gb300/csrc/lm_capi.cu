// lm_capi.cu -- the extern "C" boundary of the operators at the ends of a language
// model declared in include/instant.h (embedding, token log probabilities, gradient
// norm): argument validation and launch planning.  No device memory is allocated here.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "instant.h"
#include "kernels.h"

using namespace instant;

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dtype_ok(instant_dtype dt) { return dt == INSTANT_F32 || dt == INSTANT_BF16; }
bool tokens_ok(int token_bytes) { return token_bytes == 4 || token_bytes == 8; }
instant_status from_cuda(cudaError_t e) { return e == cudaSuccess ? INSTANT_OK : INSTANT_ERR_CUDA; }

constexpr int kMaxRows = 1 << 30, kMaxV = 1 << 24;

bool embed_shape_ok(int rows, int V, int C) {
  return rows >= 1 && rows <= kMaxRows && V >= 1 && V <= kMaxV && C >= 1 && C <= INSTANT_EMBED_MAX_C;
}
// within 2^-120 .. 2^120: the scale times log2 e is finite, and a difference of two logits that passes the
// range of fp32 has a weight of 0 (beyond 2^128 2^-120 log2 e its exponent is -369)
bool logits_scale_ok(float scale) { return scale >= 0x1p-120f && scale <= 0x1p120f; }
bool logits_shape_ok(int rows, int V, int ld) {
  return rows >= 1 && rows <= kMaxRows && V >= 1 && V <= ld && ld <= kMaxV;
}

// one launch's list after another over the tensors that hold anything; f returns a CUDA error
template <int N, typename F>
cudaError_t each_list(const instant_grad_item* items, int count, ClipList<N>& l, bool backwards, F f) {
  cudaError_t e = cudaSuccess;
  l.count = l.chunks = 0;
  auto flush = [&] {
    if (l.count == 0) return;
    l.ctas = std::min(l.chunks, kClipGrid);
    for (int c = 0, i = backwards ? l.count - 1 : 0; c < l.ctas; ++c) {
      if (backwards)
        while (l.item[i].chunk > l.chunks - 1 - c) --i;
      else
        while (i + 1 < l.count && l.item[i + 1].chunk <= c) ++i;
      l.start[c] = static_cast<uint16_t>(i);
    }
    if (e == cudaSuccess) e = f(l);
    l.part0 += l.ctas;
    l.count = l.chunks = 0;
  };
  for (int i = 0; i < count; ++i) {
    const instant_grad_item& it = items[i];
    if (it.n == 0) continue;
    if (l.count == N) flush();
    ClipItem& c = l.item[l.count++];
    c.g = it.g;
    c.out = it.out;
    c.n = it.n;
    c.chunk = l.chunks;
    c.bf16 = it.dt == INSTANT_BF16;
    l.chunks += static_cast<int>(clip_chunks(it.n, c.bf16));
  }
  flush();
  return e;
}

// chunks of all tensors, counted in an int
instant_status check_items(const instant_grad_item* items, int count) {
  if (!items || count < 1) return INSTANT_ERR_ARG;
  long long chunks = 0;
  for (int i = 0; i < count; ++i) {
    const instant_grad_item& it = items[i];
    if (!dtype_ok(it.dt)) return INSTANT_ERR_DTYPE;
    if (it.n < 0 || it.n > (1ll << 45)) return INSTANT_ERR_SHAPE;
    chunks += clip_chunks(it.n, it.dt == INSTANT_BF16);
    if (chunks > 0x7fffffffll) return INSTANT_ERR_SHAPE;
    if (it.n > 0 && (!it.g || !it.out)) return INSTANT_ERR_ARG;
    const unsigned e = it.dt == INSTANT_BF16 ? 2 : 4;
    if (!aligned(it.g, e) || !aligned(it.out, e)) return INSTANT_ERR_ALIGN;
  }
  return INSTANT_OK;
}

// a partial sum for every CTA of every launch
size_t clip_bytes(int count) {
  const size_t launches = (static_cast<size_t>(count) + kClipItems[3] - 1) / kClipItems[3];
  return (launches * kClipGrid + 1) * sizeof(ClipPart);
}

template <int N>
cudaError_t clip(const instant_grad_item* items, int count, float max_norm, float scale, float* norm, ClipPart* part,
                 cudaStream_t st) {
  ClipList<N> l;
  l.part = part;
  l.norm = nullptr;
  l.max_norm = max_norm;
  l.scale = scale;
  l.in_place = 1;
  l.part0 = l.parts = 0;
  for (int i = 0; i < count; ++i) l.in_place &= items[i].out == items[i].g;
  cudaError_t e = each_list(items, count, l, false, [&](const ClipList<N>& b) { return launch_grad_norm(b, st); });
  if (e != cudaSuccess) return e;
  l.parts = l.part0;
  l.part0 = 0;
  l.norm = norm;
  if (l.parts == 0) {  // nothing to add up: a norm of 0
    l.count = l.chunks = 0;
    l.ctas = 1;
    return launch_grad_clip(l, st);
  }
  return each_list(items, count, l, true, [&](const ClipList<N>& b) { return launch_grad_clip(b, st); });
}

}  // namespace

extern "C" {

instant_status instant_embed(const void* tokens, int token_bytes, const void* table, void* y, int rows, int V,
                             int C, float scale, instant_dtype dt, void* stream) {
  if (!dtype_ok(dt) || !tokens_ok(token_bytes)) return INSTANT_ERR_DTYPE;
  if (!tokens || !table || !y || !std::isfinite(scale)) return INSTANT_ERR_ARG;
  if (!embed_shape_ok(rows, V, C)) return INSTANT_ERR_SHAPE;
  if (!aligned(tokens, token_bytes) || !aligned(table, 16) || !aligned(y, 16) || (dt == INSTANT_BF16 && C % 8))
    return INSTANT_ERR_ALIGN;
  return from_cuda(launch_embed(tokens, token_bytes == 8, table, y, rows, V, C, scale, dt == INSTANT_BF16,
                                static_cast<cudaStream_t>(stream)));
}

size_t instant_embed_grad_workspace_bytes(int rows, int V, int C) {
  return embed_shape_ok(rows, V, C) ? embed_grad_bytes(rows, C) : 0;
}

instant_status instant_embed_grad(const void* gy, const void* tokens, int token_bytes, float* gtable,
                                  int accumulate, void* ws, size_t ws_bytes, int rows, int V, int C, float scale,
                                  instant_dtype dt, void* stream) {
  if (!dtype_ok(dt) || !tokens_ok(token_bytes)) return INSTANT_ERR_DTYPE;
  if (!gy || !tokens || !gtable || !std::isfinite(scale)) return INSTANT_ERR_ARG;
  if (!embed_shape_ok(rows, V, C)) return INSTANT_ERR_SHAPE;
  if (!ws || ws_bytes < embed_grad_bytes(rows, C)) return INSTANT_ERR_WORKSPACE;
  if (!aligned(gy, 16) || !aligned(tokens, token_bytes) || !aligned(gtable, 16) || !aligned(ws, 16) ||
      (dt == INSTANT_BF16 && C % 8))
    return INSTANT_ERR_ALIGN;
  EmbedGradArgs a{};
  a.gy = gy;
  a.tokens = tokens;
  a.wide = token_bytes == 8;
  a.gtable = gtable;
  a.rows = rows;
  a.V = V;
  a.C = C;
  a.scale = scale;
  a.accumulate = accumulate != 0;
  return from_cuda(launch_embed_grad(a, ws, dt == INSTANT_BF16, static_cast<cudaStream_t>(stream)));
}

instant_status instant_token_logprobs(const void* x, const void* tokens, int token_bytes, float* logp, float* stats,
                                      float* entropy, long long* top_ids, float* top_logp, int rows, int V, int ld,
                                      int top, float scale, instant_dtype dt, void* stream) {
  if (!dtype_ok(dt) || !tokens_ok(token_bytes)) return INSTANT_ERR_DTYPE;
  if (!x || !(logp || stats || entropy || top_ids || top_logp) || (logp && !tokens) ||
      !logits_scale_ok(scale))
    return INSTANT_ERR_ARG;
  if ((top == 0) != !(top_ids || top_logp)) return INSTANT_ERR_ARG;
  if (!logits_shape_ok(rows, V, ld) || top < 0 || top > INSTANT_TOP_MAX || top > V) return INSTANT_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(tokens, token_bytes) || !aligned(logp, 4) || !aligned(stats, 8) ||
      !aligned(entropy, 4) || !aligned(top_ids, 8) || !aligned(top_logp, 4))
    return INSTANT_ERR_ALIGN;
  LogprobArgs a{};
  a.x = x;
  a.tokens = tokens;
  a.wide = token_bytes == 8;
  a.logp = logp;
  a.stats = stats;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_logp = top_logp;
  a.rows = rows;
  a.V = V;
  a.ld = ld;
  a.top = top;
  a.scale = scale;
  return from_cuda(launch_logprobs(a, dt == INSTANT_BF16, static_cast<cudaStream_t>(stream)));
}

instant_status instant_token_logprobs_grad(const void* x, const void* tokens, int token_bytes, const float* stats,
                                           const float* g_logp, const float* g_entropy, const float* entropy,
                                           void* gx, int rows, int V, int ld, float scale, instant_dtype dt,
                                           void* stream) {
  if (!dtype_ok(dt) || !tokens_ok(token_bytes)) return INSTANT_ERR_DTYPE;
  if (!x || !stats || !gx || !(g_logp || g_entropy) || (g_logp && !tokens) || (!g_entropy != !entropy) ||
      !logits_scale_ok(scale))
    return INSTANT_ERR_ARG;
  if (!logits_shape_ok(rows, V, ld)) return INSTANT_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(tokens, token_bytes) || !aligned(stats, 8) || !aligned(g_logp, 4) ||
      !aligned(g_entropy, 4) || !aligned(entropy, 4) || !aligned(gx, 16))
    return INSTANT_ERR_ALIGN;
  LogprobGradArgs a{};
  a.x = x;
  a.tokens = tokens;
  a.wide = token_bytes == 8;
  a.stats = stats;
  a.g_logp = g_logp;
  a.g_entropy = g_entropy;
  a.entropy = entropy;
  a.gx = gx;
  a.rows = rows;
  a.V = V;
  a.ld = ld;
  a.scale = scale;
  return from_cuda(launch_logprobs_grad(a, dt == INSTANT_BF16, static_cast<cudaStream_t>(stream)));
}

size_t instant_grad_clip_workspace_bytes(int count) { return count < 1 ? 0 : clip_bytes(count); }

instant_status instant_grad_clip(const instant_grad_item* items, int count, float max_norm, float scale, float* norm,
                                 void* ws, size_t ws_bytes, void* stream) {
  if (!norm || !(max_norm > 0.f) || !(std::isfinite(scale) && scale > 0.f)) return INSTANT_ERR_ARG;
  const instant_status bad = check_items(items, count);
  if (bad != INSTANT_OK) return bad;
  if (!ws || ws_bytes < clip_bytes(count)) return INSTANT_ERR_WORKSPACE;
  if (!aligned(ws, 16) || !aligned(norm, 8)) return INSTANT_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  ClipPart* part = static_cast<ClipPart*>(ws);
  auto go = [&](auto n) { return clip<decltype(n)::value>(items, count, max_norm, scale, norm, part, st); };
  using std::integral_constant;
  return from_cuda(count <= kClipItems[0]   ? go(integral_constant<int, kClipItems[0]>())
                   : count <= kClipItems[1] ? go(integral_constant<int, kClipItems[1]>())
                   : count <= kClipItems[2] ? go(integral_constant<int, kClipItems[2]>())
                                            : go(integral_constant<int, kClipItems[3]>()));
}

}  // extern "C"
