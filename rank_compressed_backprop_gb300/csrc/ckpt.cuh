// ckpt.cuh -- 8-bit activation checkpoints and activation functions, shared by
// the kernels of an MLP block.
//
// A checkpoint of t [rows, C] cuts each row into groups of 128 channels (the
// last one may be shorter).  A group with largest magnitude amax holds
//   2^k   the smallest power of two with amax / 2^k <= 127, k in [-120, 121]
//   q     = round(t / 2^k), ties to even, within [-127, 127]
// stored as int8 codes q [rows, ld] (ld = C rounded up to 16) and one byte
// s [groups, rows] = k + 127 per group, 255 when the group holds an infinity or
// a NaN (it then reads back as NaN).  The scale is a power of two so that
// q 2^k, at most seven significant bits, is exact in bf16: a gradient that reads
// a checkpoint feeds it to the tensor cores without a second rounding, and
// t / 2^k is exact, so the only rounding is that to the codes.  The lower clamp
// keeps q 2^k a normal number (what is below 2^-121 reads back as 0), the upper
// one keeps 127 * 2^k finite.
#pragma once

#include "kernels.h"
#include "tc.cuh"

namespace instant {

constexpr int kCkptGroup = 128;
constexpr uint32_t kCkptNaN = 255;

// magnitude bits: NaN > inf > every finite value, so an integer maximum keeps
// the non-finite ones (fmaxf would drop a NaN)
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// scale byte of a group from the bits of its largest magnitude: with amax =
// 1.f * 2^E, k = E - 6, one more when the significand 1.f is above 127 / 64
__device__ __forceinline__ uint32_t ckpt_scale_code(uint32_t amax) {
  if (amax >= 0x7f800000u) return kCkptNaN;
  int c = static_cast<int>(amax >> 23) - 6 + ((amax & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return static_cast<uint32_t>(min(max(c, 7), 248));
}

__device__ __forceinline__ float ckpt_scale(uint32_t code) {  // 2^k (NaN for 255)
  return code == kCkptNaN ? __uint_as_float(0x7fc00000u) : __uint_as_float(code << 23);
}

__device__ __forceinline__ float ckpt_inv_scale(uint32_t code) {  // 2^-k
  return code == kCkptNaN ? 0.f : __uint_as_float((254u - code) << 23);
}

// The code of v as the low byte of an integer.  Adding 1.5 * 2^23 rounds to an
// integer, ties to even, and leaves it in two's complement in the low bits of
// the sum; |v inv| <= 127 by the choice of the scale except at its upper
// clamp, where the minimum matters.
__device__ __forceinline__ uint32_t ckpt_code(float v, float inv) {
  const float t = fminf(fmaxf(v * inv, -127.f), 127.f);
  return __float_as_uint(t + 12582912.f);
}

__device__ __forceinline__ uint32_t ckpt_code4(float a, float b, float c, float d, float inv) {
  const uint32_t ab = __byte_perm(ckpt_code(a, inv), ckpt_code(b, inv), 0x0040);
  const uint32_t cd = __byte_perm(ckpt_code(c, inv), ckpt_code(d, inv), 0x0040);
  return __byte_perm(ab, cd, 0x5410);
}

// byte i of w as a float times the scale
template <int I>
__device__ __forceinline__ float ckpt_value(uint32_t w, float scale) {
  // q + 128 in the low mantissa bits of 2^23: one byte permute and a subtract
  const uint32_t m = __byte_perm(w ^ 0x80808080u, 0x4b000000u, 0x7440 | I);
  return (__uint_as_float(m) - 8388736.f) * scale;
}

__device__ __forceinline__ void ckpt_values4(uint32_t w, float scale, float* v) {
  v[0] = ckpt_value<0>(w, scale);
  v[1] = ckpt_value<1>(w, scale);
  v[2] = ckpt_value<2>(w, scale);
  v[3] = ckpt_value<3>(w, scale);
}

// maximum over the 16 lanes of a half warp
__device__ __forceinline__ uint32_t half_warp_max(uint32_t v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// ---------------------------------------------------------------------------
// element access: bf16 (as its 16 bits) and fp32
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ float elem_to_f(T v);
template <>
__device__ __forceinline__ float elem_to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float elem_to_f<uint16_t>(uint16_t v) { return bf16_to_f32(v); }

template <typename T>
__device__ __forceinline__ T f_to_elem(float v);
template <>
__device__ __forceinline__ float f_to_elem<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t f_to_elem<uint16_t>(float v) { return bf16_bits(v); }

// N consecutive elements (N = 4 or 8) from an address aligned to the access
template <int N>
__device__ __forceinline__ void load_vec(const uint16_t* p, float* v) {
  uint32_t w[N / 2];
  if (N == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x; w[1] = u.y; w[N / 2 - 2] = u.z; w[N / 2 - 1] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x; w[1] = u.y;
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <int N>
__device__ __forceinline__ void load_vec(const float* p, float* v) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const float4 u = *reinterpret_cast<const float4*>(p + 4 * i);
    v[4 * i] = u.x; v[4 * i + 1] = u.y; v[4 * i + 2] = u.z; v[4 * i + 3] = u.w;
  }
}
template <int N>
__device__ __forceinline__ void store_vec(uint16_t* p, const float* v) {
  if (N == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[N - 4], v[N - 3]), pack_bf16x2(v[N - 2], v[N - 1]));
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
template <int N>
__device__ __forceinline__ void store_vec(float* p, const float* v) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    *reinterpret_cast<float4*>(p + 4 * i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

// the same with `n` valid elements of N (the rest read as 0, are not written);
// vec: the address is aligned and, where all N are valid, may be used at once
template <int N, typename T>
__device__ __forceinline__ void load_part(const T* p, int n, bool vec, float* v) {
  if (vec && n >= N) {
    load_vec<N>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < n ? elem_to_f<T>(p[i]) : 0.f;
  }
}
template <int N, typename T>
__device__ __forceinline__ void store_part(T* p, int n, bool vec, const float* v) {
  if (vec && n >= N) {
    store_vec<N>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) p[i] = f_to_elem<T>(v[i]);
  }
}

// ---------------------------------------------------------------------------
// activations in fp32 with CUDA's own functions (the fp32 path; gelu in its erf
// form through erfc, which keeps its relative accuracy in the negative tail)
// ---------------------------------------------------------------------------
__device__ __forceinline__ float act_f32(float z, int act) {
  switch (act) {
    case INSTANT_ACT_RELU: return z < 0.f ? 0.f : z;  // keeps a NaN
    case INSTANT_ACT_GELU: return 0.5f * z * erfcf(-0.70710678f * z);
    case INSTANT_ACT_SILU: return z / (1.f + expf(-z));
    default: return z;
  }
}

__device__ __forceinline__ float act_slope_f32(float z, int act) {
  switch (act) {
    case INSTANT_ACT_RELU: return z > 0.f ? 1.f : (z <= 0.f ? 0.f : z);  // keeps a NaN
    case INSTANT_ACT_GELU:
      return 0.5f * erfcf(-0.70710678f * z) + z * 0.39894228f * expf(-0.5f * z * z);
    case INSTANT_ACT_SILU: {
      const float s = 1.f / (1.f + expf(-z));
      return s * (1.f + z * (1.f - s));
    }
    default: return 1.f;
  }
}

// ---------------------------------------------------------------------------
// The same for outputs in bf16, two values at a time: the epilogues of the
// tensor-core products spend most of their instructions here, and the packed
// fp32 operations halve those that are sums and products.
//   gelu(z) = max(z, 0) - |z| Phi(-|z|),  Phi(-t) = exp(-t^2 / 2) M(t), t >= 0
// with M(t) = erfcx(t / sqrt 2) / 2, which falls smoothly from 1/2 like 1 / t; M is
// a degree-8 polynomial in 1 / (1 + 0.235 t) without constant term, fitted by
// weighted least squares on [0, 16] to 1.2e-7 relative (5e-7 evaluated in fp32), so
// the negative tail keeps its relative accuracy.  Error with the approximate
// exponential and reciprocal: gelu 8e-6 relative at z = -13, where the roundings of
// z^2 / 2 count most, 1.5e-6 from -4 on; gelu' 6e-7, below -1 relative like gelu.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float ex2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint64_t f2_bits(float2 v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ float2 f2_of(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)), "l"(f2_bits(c)));
  return f2_of(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return f2_of(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return f2_of(r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Phi(-|z|), and e = exp(-z^2 / 2)
__device__ __forceinline__ float2 normal_tail(float2 z, float2& e) {
  const float2 s = make_float2(rcp_approx(fmaf(0.235f, fabsf(z.x), 1.f)), rcp_approx(fmaf(0.235f, fabsf(z.y), 1.f)));
  float2 m = fma2(both(-0.064109147f), s, both(0.21002914f));
  m = fma2(m, s, both(-0.14554477f));
  m = fma2(m, s, both(0.17967278f));
  m = fma2(m, s, both(0.035570811f));
  m = fma2(m, s, both(0.097954720f));
  m = fma2(m, s, both(0.092617162f));
  m = fma2(m, s, both(0.093809262f));
  const float2 x = mul2(mul2(z, z), both(-0.72134752f));  // -log2(e) / 2
  e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
  return mul2(e, mul2(m, s));
}

template <int ACT>
__device__ __forceinline__ float2 act_fast(float2 z) {
  if (ACT == INSTANT_ACT_RELU) return make_float2(z.x < 0.f ? 0.f : z.x, z.y < 0.f ? 0.f : z.y);
  if (ACT == INSTANT_ACT_GELU) {
    float2 e;
    const float2 p = normal_tail(z, e);
    // -|z|, cut at -40 above zero, where the tail is 0 in fp32: plus infinity then meets no
    // 0 * inf, and minus infinity does, as in the formula
    const float2 n = make_float2(fminf(z.x, fmaxf(-z.x, -40.f)), fminf(z.y, fmaxf(-z.y, -40.f)));
    return make_float2(fmaf(n.x, p.x, fmaxf(z.x, 0.f)), fmaf(n.y, p.y, fmaxf(z.y, 0.f)));
  }
  if (ACT == INSTANT_ACT_SILU) {
    const float2 x = mul2(z, both(-1.44269504f));
    const float2 d = add2(make_float2(ex2_approx(x.x), ex2_approx(x.y)), both(1.f));
    return mul2(z, make_float2(rcp_approx(d.x), rcp_approx(d.y)));
  }
  return z;
}

template <int ACT>
__device__ __forceinline__ float2 act_slope_fast(float2 z) {
  if (ACT == INSTANT_ACT_RELU)
    return make_float2(z.x > 0.f ? 1.f : (z.x <= 0.f ? 0.f : z.x), z.y > 0.f ? 1.f : (z.y <= 0.f ? 0.f : z.y));
  if (ACT == INSTANT_ACT_GELU) {
    // Phi(z) and z times the density.  Below zero Phi(z) is the tail itself: one minus
    // it and back would leave nothing of it (gelu'(-5.5) was 3 % off)
    float2 e;
    const float2 p = normal_tail(z, e);
    const float2 h = fma2(p, both(-1.f), both(1.f));
    const float2 c = make_float2(z.x < 0.f ? p.x : h.x, z.y < 0.f ? p.y : h.y);
    return fma2(mul2(z, both(0.39894228f)), e, c);
  }
  if (ACT == INSTANT_ACT_SILU) {
    const float2 x = mul2(z, both(-1.44269504f));
    const float2 d = add2(make_float2(ex2_approx(x.x), ex2_approx(x.y)), both(1.f));
    const float2 s = make_float2(rcp_approx(d.x), rcp_approx(d.y));
    return mul2(s, fma2(z, fma2(s, both(-1.f), both(1.f)), both(1.f)));
  }
  return both(1.f);
}

// the larger magnitude of three values, NaN if one of them is
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Codes of four values whose scale is not at its upper clamp: no value is above
// 127 steps then (of a NaN group the codes do not matter).
__device__ __forceinline__ uint32_t ckpt_code4_in_range(float2 ab, float2 cd, float inv) {
  const float2 p = fma2(ab, both(inv), both(12582912.f));
  const float2 q = fma2(cd, both(inv), both(12582912.f));
  const uint32_t lo = __byte_perm(__float_as_uint(p.x), __float_as_uint(p.y), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(q.x), __float_as_uint(q.y), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// the codes of eight values
__device__ __forceinline__ uint2 ckpt_code8(const float2* v, uint32_t code) {
  const float inv = ckpt_inv_scale(code);
  if (code == 248u)  // the upper clamp of the scale: a value may be up to 128 steps
    return make_uint2(ckpt_code4(v[0].x, v[0].y, v[1].x, v[1].y, inv), ckpt_code4(v[2].x, v[2].y, v[3].x, v[3].y, inv));
  return make_uint2(ckpt_code4_in_range(v[0], v[1], inv), ckpt_code4_in_range(v[2], v[3], inv));
}

// eight codes as numbers, in pairs (2^23 + 128 + q, less 2^23 + 128)
__device__ __forceinline__ void code_pairs(uint2 w, float2* v) {
  const uint32_t x[2] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u};
  const float2 o = both(-8388736.f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[2 * i] = add2(make_float2(__uint_as_float(__byte_perm(x[i], 0x4b000000u, 0x7440)),
                                __uint_as_float(__byte_perm(x[i], 0x4b000000u, 0x7441))), o);
    v[2 * i + 1] = add2(make_float2(__uint_as_float(__byte_perm(x[i], 0x4b000000u, 0x7442)),
                                    __uint_as_float(__byte_perm(x[i], 0x4b000000u, 0x7443))), o);
  }
}

// the values of eight codes (folding the offset and the scale into one operation
// would overflow at the largest scales)
__device__ __forceinline__ void ckpt_pairs8(uint2 w, float scale, float2* v) {
  code_pairs(w, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], both(scale));
}

// Eight elements as four pairs, n of which exist.  VEC: the address is aligned
// and rows are whole vectors, so it is all eight or none; otherwise any number.
template <bool VEC, typename T>
__device__ __forceinline__ void load_pairs(const T* p, int n, float2* v) {
  float t[8];
  if (VEC) {
    if (n > 0) {
      load_vec<8>(p, t);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = 0.f;
    }
  } else {
    load_part<8>(p, n, false, t);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = make_float2(t[2 * i], t[2 * i + 1]);
}
template <bool VEC, typename T>
__device__ __forceinline__ void store_pairs(T* p, int n, const float2* v) {
  const float t[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
  if (VEC) {
    if (n > 0) store_vec<8>(p, t);
  } else {
    store_part<8>(p, n, false, t);
  }
}

// bits of the largest of eight magnitudes, NaN's if one is a NaN
__device__ __forceinline__ uint32_t max_bits8(const float2* v) {
  return __float_as_uint(max_abs3(max_abs3(v[0].x, v[0].y, max_abs3(v[1].x, v[1].y, v[2].x)), v[2].y,
                                  max_abs3(v[3].x, v[3].y, 0.f)));
}

// the checkpoint of a group held by a half warp, eight channels a lane in pairs:
// its scale code, for ckpt_code8
__device__ __forceinline__ uint32_t group_code(const float2* v) {
  return ckpt_scale_code(half_warp_max(max_bits8(v)));
}

}  // namespace instant
