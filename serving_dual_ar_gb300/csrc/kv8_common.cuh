// Shared pieces of the 8-bit KV cache kernels.
//
// Cache: pages of 16 tokens, e4m3 bytes [2 (K, V)][Hkv][16][hd] and fp32
// scales [2][Hkv], powers of two.  A block is the 16 rows of one (page, K or
// V, head); its scale is 2^e with the smallest e in [-32, 32] whose 448 * 2^e
// covers the block's largest magnitude.  With scales that are powers of two a
// change of scale moves the exponents of the stored values and nothing else, so a
// block filled token by token holds the bytes that it would hold if filled at once
// -- but for values that become e4m3 subnormals when the scale grows behind them,
// which were rounded before and are rounded once more.
#pragma once

#include <cuda_fp16.h>

#include "s2_common.cuh"
#include "two_float.cuh"

namespace s2 {

constexpr int kKv8Page = 16;
constexpr int kKv8EMin = -32, kKv8EMax = 32;

// ---------------------------------------------------------------- workspace

inline int kv8_sms() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 1;
}
// Tickets come first in a workspace, partial sums behind them from the same
// place on in every call: what one call leaves there another of other sizes, or
// of the other kind, never takes for a ticket.  Tickets: two levels of two slots
// for up to eight warps an SM (decode), one an SM (prompts).
inline size_t kv8_ticket_bytes(int sms) { return (size_t)sms * 2 * 2 * 8 * 4; }

// ---------------------------------------------------------------- scales

S2_DEV float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // |e| <= 126
// Exponent of a stored scale: of the power of two next to it (one that a library
// function computed may lie a bit beside it), within the range that the
// kernels write.
S2_DEV int kv8_scale_exp(float s) {
  const int e = (int)(((__float_as_uint(s) & 0x7fffffffu) + 0x400000u) >> 23) - 127;
  return min(max(e, kKv8EMin), kKv8EMax);
}
// The smallest e in [-32, 32] with amax <= 448 * 2^e (448 = 1.75 * 2^8);
// infinity takes the largest, and saturates.
S2_DEV int kv8_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax) & 0x7fffffffu;
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kKv8EMin), kKv8EMax);
}

// ---------------------------------------------------------------- e4m3

// Two values to e4m3 (nearest, ties to even, saturating; NaN stays NaN), x in
// the low byte.
S2_DEV uint32_t e4m3x2(float x, float y) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
  return r;
}
// Two e4m3 bytes (low byte first) to f16x2; every e4m3 value is an f16 value.
S2_DEV uint32_t f16x2_of_e4m3(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
// The four bytes of a word times f (a power of two <= 1), rounded to e4m3.
S2_DEV uint32_t e4m3_rescale4(uint32_t w, float f) {
  uint32_t a = f16x2_of_e4m3((uint16_t)w), b = f16x2_of_e4m3((uint16_t)(w >> 16));
  const float2 x = __half22float2(*reinterpret_cast<__half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<__half2*>(&b));
  return e4m3x2(x.x * f, x.y * f) | (e4m3x2(y.x * f, y.y * f) << 16);
}

// ---------------------------------------------------------------- keys to about 2^-44

// One key row by one warp: RMSNorm, gain and rotation of x[0 .. HD), lane l
// taking dims l + 32 i, as values rounded to odd.  The sum of squares, its
// inverse root (one Newton step on the float one) and the rotation run in
// two-float arithmetic (about 44 bits), because the result is rounded to 8
// bits at once: whether a prompt or a single step appends a token, in
// whatever batch, it is rounded from the same value.  Everything else of the
// attention is fp32.
template <int HD>
S2_DEV void kv8_key_row(const float* __restrict__ x, const float* __restrict__ gain,
                        const float* __restrict__ cs, const float* __restrict__ sn, float eps, int lane,
                        float (&out)[HD / 32]) {
  constexpr int N = HD / 32;
  float v[N], g[N], c[N / 2], s[N / 2];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = x[lane + 32 * i];
    g[i] = gain[lane + 32 * i];
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    c[i] = cs[lane + 32 * i];
    s[i] = sn[lane + 32 * i];
  }
  Two ss = two_prod(v[0], v[0]);
#pragma unroll
  for (int i = 1; i < N; ++i) ss = add(ss, two_prod(v[i], v[i]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    ss = add(ss, Two{__shfl_xor_sync(0xffffffffu, ss.hi, o), __shfl_xor_sync(0xffffffffu, ss.lo, o)});
  ss = add(Two{ss.hi * (1.f / HD), ss.lo * (1.f / HD)}, Two{eps, 0.f});
  const float r0 = rsqrtf(ss.hi);
  const Two q = two_prod(r0, r0);
  Two t = mul(ss, q.hi);                        // ss r0^2
  t.lo = __fmaf_rn(ss.hi, q.lo, t.lo);
  const float d = __fsub_rn(__fsub_rn(1.f, t.hi), t.lo);
  const Two r = quick_two(r0, __fmul_rn(__fmul_rn(0.5f, r0), d));
  Two y[N];
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = mul(mul(r, v[i]), g[i]);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const Two a = y[i], b = y[i + N / 2];
    out[i] = round_odd(add(mul(a, c[i]), mul(b, -s[i])));
    out[i + N / 2] = round_odd(add(mul(b, c[i]), mul(a, s[i])));
  }
}

template <int N>
S2_DEV float abs_max(const float (&v)[N], float m) {   // NaN does not count
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

}  // namespace s2
