// Rounding of rows to 8-bit and 4-bit values with a power of two per 32 of
// them (mx_common.cuh): activations, the residual's addition with RMSNorm and
// such an output, weights, and weights back.
#include "mx_common.cuh"
#include "two_float.cuh"

namespace s2 {

namespace {

// Values k0 .. k0 + 7 of a row as floats, zeros from K on.  vec: rows start on
// 16-byte boundaries.  (No __restrict__: a row may be one that the kernel wrote.)
template <typename T>
S2_DEV void load_row8(const T* row, int k0, int K, bool vec, float (&v)[8]) {
  if (vec && k0 + 8 <= K) {
    load8(row + k0, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k0 + i < K ? to_f(row[k0 + i]) : 0.f;
  }
}
template <typename T>
S2_DEV void store_row8(T* row, int k0, int K, bool vec, const float (&v)[8]) {
  if (vec && k0 + 8 <= K) {
    if (sizeof(T) == 4) {
      float4* p = reinterpret_cast<float4*>(row + k0);
      p[0] = make_float4(v[0], v[1], v[2], v[3]);
      p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(row + k0) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k0 + i < K) row[k0 + i] = from_f<T>(v[i]);
  }
}

S2_DEV float max8(const float (&v)[8]) {   // NaN does not count
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}
// Over the four lanes of a group.
S2_DEV float max_of_group(float m) {
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
}
// The bytes of the four groups of a half-warp's 128 values as one word.
S2_DEV uint32_t scale_word(uint32_t byte, int lane) {
  uint32_t w = byte << (((lane >> 2) & 3) * 8);
  w |= __shfl_xor_sync(0xffffffffu, w, 4);
  return w | __shfl_xor_sync(0xffffffffu, w, 8);
}

// Eight values of a lane, 32 of four lanes, to e4m3 and their scale's byte.
// NaN and infinities are stored as NaN and do not count for the scale.
S2_DEV uint2 round8(float (&v)[8], bool group_in_row, uint32_t& byte) {
  float m = max_of_group(max8(v));
  if (__any_sync(0xffffffffu, m > 3.402823466e38f)) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (fabsf(v[i]) > 3.402823466e38f) v[i] = __uint_as_float(0x7fffffffu);
    m = max_of_group(max8(v));
  }
  const int e = mx8_exponent(m);
  const float f = mx_pow2(-e);
  byte = group_in_row ? (uint32_t)(e + 127) : 127u;
  return make_uint2(mx_e4m3x2(v[0] * f, v[1] * f) | (mx_e4m3x2(v[2] * f, v[3] * f) << 16),
                    mx_e4m3x2(v[4] * f, v[5] * f) | (mx_e4m3x2(v[6] * f, v[7] * f) << 16));
}
// Rows of y8 have a pitch of a multiple of 16 and start on 16 bytes.
S2_DEV void store_codes8(uint8_t* row, int k0, int K, uint2 c) {
  if (k0 + 8 <= K) {
    *reinterpret_cast<uint2*>(row + k0) = c;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k0 + i < K) row[k0 + i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
  }
}

// ---------------------------------------------------------------- two floats an instruction

using F2 = unsigned long long;
S2_DEV F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
S2_DEV void f2_split(F2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
S2_DEV F2 f2_add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
S2_DEV F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
S2_DEV F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
S2_DEV F2 f2_neg(F2 a) { return a ^ 0x8000000080000000ull; }
S2_DEV F2 f2_sub(F2 a, F2 b) { return f2_add(a, f2_neg(b)); }

// Eight values as they lie in memory, 16-byte aligned.
template <typename T> struct Raw8;
template <> struct Raw8<float> {
  uint4 a, b;
  S2_DEV void load(const float* p) {
    a = *reinterpret_cast<const uint4*>(p);
    b = *reinterpret_cast<const uint4*>(p + 4);
  }
  S2_DEV void zero() { a = b = make_uint4(0, 0, 0, 0); }
  // Bits of the largest magnitude of the four lanes' 32 values; infinity's or above
  // if there is an infinity or a NaN.
  S2_DEV uint32_t group_max() const {
    const uint32_t k = 0x7fffffffu;
    uint32_t m = max(max(max(a.x & k, a.y & k), max(a.z & k, a.w & k)), max(max(b.x & k, b.y & k), max(b.z & k, b.w & k)));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  }
  S2_DEV void get(F2 (&v)[4]) const {
    v[0] = f2(__uint_as_float(a.x), __uint_as_float(a.y));
    v[1] = f2(__uint_as_float(a.z), __uint_as_float(a.w));
    v[2] = f2(__uint_as_float(b.x), __uint_as_float(b.y));
    v[3] = f2(__uint_as_float(b.z), __uint_as_float(b.w));
  }
};
template <> struct Raw8<__nv_bfloat16> {
  uint4 a;
  S2_DEV void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  S2_DEV void zero() { a = make_uint4(0, 0, 0, 0); }
  S2_DEV uint32_t group_max() const {      // two at a time
    const uint32_t k = 0x7fff7fffu;
    uint32_t m = __vmaxu2(__vmaxu2(a.x & k, a.y & k), __vmaxu2(a.z & k, a.w & k));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    return max(m & 0xffff0000u, m << 16);
  }
  S2_DEV void get(F2 (&v)[4]) const {
    v[0] = f2(bf16lo(a.x), bf16hi(a.x));
    v[1] = f2(bf16lo(a.y), bf16hi(a.y));
    v[2] = f2(bf16lo(a.z), bf16hi(a.z));
    v[3] = f2(bf16lo(a.w), bf16hi(a.w));
  }
};

S2_DEV float f2_max8(const F2 (&v)[4]) {   // of the magnitudes; NaN does not count
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    f2_split(v[i], a, b);
    m = fmaxf(m, fmaxf(fabsf(a), fabsf(b)));
  }
  return m;
}
// mx8_exponent of finite magnitudes by its bits: 1.75 is 0x600000 of a mantissa.
S2_DEV int exponent_of_bits(uint32_t u) { return max((int)((u + 0x1fffffu) >> 23) - 135, kMxEMin); }
S2_DEV uint2 f2_e4m3(const F2 (&v)[4], float q) {   // v * q to e4m3
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    f2_split(f2_mul(v[i], f2(q, q)), a, b);
    c[i] = mx_e4m3x2(a, b);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// ---------------------------------------------------------------- rows to 8 bits

// Units (row, 128 values) of a half-warp, 16 apart, all loaded before the first
// is rounded; one division a thread finds the first.
constexpr int kUnits = 4;
struct Units {
  long long row;
  int kt;
  S2_DEV Units(int KT) {
    const long long u = (long long)blockIdx.x * (16 * kUnits) + (threadIdx.x >> 4);
    row = u <= 0x7fffffff ? (int)u / KT : u / KT;
    kt = (int)(u - row * KT);
  }
  S2_DEV void next(int KT, int rows, int kts) {      // 16 units: rows x KT + kts
    row += rows;
    kt += kts;
    if (kt >= KT) {
      kt -= KT;
      ++row;
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(256) mx8_pack_kernel(Mx8PackArgs p) {
  pdl_launch_next();
  pdl_wait();
  const int lane = threadIdx.x & 31, KT = (p.K + 127) / 128, rows = 16 / KT, kts = 16 % KT;
  const Units first(KT);
  Units u = first;
  float v[kUnits][8];
#pragma unroll
  for (int i = 0; i < kUnits; ++i, u.next(KT, rows, kts))
    load_row8(static_cast<const T*>(p.x) + u.row * p.ldx, u.kt * 128 + (lane & 15) * 8, u.row < p.T ? p.K : 0, p.vec,
              v[i]);
  u = first;
#pragma unroll
  for (int i = 0; i < kUnits; ++i, u.next(KT, rows, kts)) {
    const int k0 = u.kt * 128 + (lane & 15) * 8;
    uint32_t byte;
    const uint2 c = round8(v[i], (k0 & ~31) < p.K, byte);
    const uint32_t w = scale_word(byte, lane);
    if (u.row >= p.T) continue;
    store_codes8(p.y8 + u.row * p.ld8, k0, p.K, c);
    if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(p.scale + mx_scale_at(u.row, u.kt, KT)) = w;
  }
}

// The same where rows start on 16 bytes and K is a multiple of 8: a warp takes 256
// columns of consecutive rows, whose addresses lie a pitch apart, with two floats
// an instruction and in registers few enough that an SM has loads under way all the
// time.  8,000 x 4,096 bf16 values in 17.1 us (5.8 TB/s), 8,000 x 2,560 fp32 values in
// 16.7 us (6.2 TB/s); the first was 31.9 us as above, bound by its instructions, most of them for
// addresses.
template <typename T> constexpr int kVecRows = sizeof(T) == 2 ? 4 : 2;   // a power of two up to 32
struct Strip {
  int row0, kt, k0;      // first row, and this lane's column block and first column
  S2_DEV Strip(int KT, int rows) {
    const int segs = (KT + 1) / 2, w = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    row0 = w / segs * rows;
    kt = w % segs * 2 + (lane >> 4);
    k0 = kt * 128 + (lane & 15) * 8;
  }
};
template <typename T>
__global__ void __launch_bounds__(256, 5) mx8_pack_vec_kernel(Mx8PackArgs p) {
  constexpr int U = kVecRows<T>;
  pdl_launch_next();
  pdl_wait();
  const int lane = threadIdx.x & 31, KT = (p.K + 127) / 128;
  const Strip s(KT, U);
  const bool in = s.k0 < p.K;
  const T* x = static_cast<const T*>(p.x) + s.row0 * p.ldx + s.k0;
  Raw8<T> raw[U];
#pragma unroll
  for (int i = 0; i < U; ++i, x += p.ldx) {
    if (in && s.row0 + i < p.T) raw[i].load(x);
    else raw[i].zero();
  }
  uint8_t* y = p.y8 + s.row0 * p.ld8 + s.k0;
  uint8_t* scale = p.scale + mx_scale_at(s.row0, s.kt, KT);      // rows that share 32: 16 bytes apart
#pragma unroll
  for (int i = 0; i < U; ++i, y += p.ld8, scale += 16) {
    F2 v[4];
    raw[i].get(v);
    const uint32_t m = raw[i].group_max();
    const int e = exponent_of_bits(m);
    uint2 c = f2_e4m3(v, mx_pow2(-min(e, kMxEMax)));
    uint32_t byte = (s.k0 & ~31) < p.K ? (uint32_t)(e + 127) : 127u;
    if (__any_sync(0xffffffffu, m >= 0x7f800000u)) {
      float w[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) f2_split(v[j], w[2 * j], w[2 * j + 1]);
      c = round8(w, (s.k0 & ~31) < p.K, byte);
    }
    const uint32_t w = scale_word(byte, lane);
    if (s.row0 + i >= p.T) break;      // the whole warp
    if (in) *reinterpret_cast<uint2*>(y) = c;
    if ((lane & 15) == 0 && s.kt < KT) *reinterpret_cast<uint32_t*>(scale) = w;
  }
}

// ---------------------------------------------------------------- residual + RMSNorm to 8 bits

// One CTA per row: h = x + r (rounded to x's type and stored), then y = h /
// sqrt(mean h^2 + eps) * gain to e4m3 with scales.  The codes are those of the
// exact values, whatever the order of the sum: the sum of squares, its inverse
// root and the products are unevaluated sums of two floats (about 2^-44).  Rows of
// any length and alignment; h is read back for the rounding.  A row whose sum of
// squares, or eps, leaves fp32's range is taken once more scaled by 2^-80 or 2^64
// (2^120).  A row with a NaN or an infinity is NaN throughout.
// 1 / sqrt(s / K + eps): a Newton step on the float one.  NaN for a row with a
// NaN or an infinity, or with nothing at all and no eps.
S2_DEV Two inverse_root(Two s, Two inv_k, float eps) {
  Two m = two_prod(s.hi, inv_k.hi);
  m.lo = __fmaf_rn(s.hi, inv_k.lo, __fmaf_rn(s.lo, inv_k.hi, m.lo));
  m = add(quick_two(m.hi, m.lo), Two{eps, 0.f});
  if (!(m.hi < __uint_as_float(0x7f800000u) && m.hi > 0.f)) return {__uint_as_float(0x7fffffffu), 0.f};
  const float r0 = rsqrtf(m.hi);
  const Two q = two_prod(r0, r0);
  Two t = mul(m, q.hi);
  t.lo = __fmaf_rn(m.hi, q.lo, t.lo);
  const float d = __fsub_rn(__fsub_rn(1.f, t.hi), t.lo);
  return quick_two(r0, __fmul_rn(__fmul_rn(0.5f, r0), d));
}

template <typename TX, typename TR>
__global__ void __launch_bounds__(1024) add_rmsnorm_mx8_kernel(AddNormMx8Args p) {
  __shared__ float2 part[32];
  pdl_launch_next();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
  const int KT = (p.K + 127) / 128;
  const long long row = blockIdx.x;
  const TX* x = static_cast<const TX*>(p.x) + row * p.ldx;
  const TR* r = p.r ? static_cast<const TR*>(p.r) + row * p.ldr : nullptr;
  TX* h = static_cast<TX*>(p.h) + row * p.ldh;
  const int runs = KT * 16;               // runs of 8 values, the row's padding included
  float v[8];

  auto sum_up = [](const float (&a)[8], float f, Two& s) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = f == 1.f ? a[i] : a[i] * f;
      const Two q = two_prod(v, v);
      const Two t = two_sum(s.hi, q.hi);
      s = {t.hi, __fadd_rn(s.lo, __fadd_rn(t.lo, q.lo))};
    }
  };
  auto joined = [&](int k0, float (&a)[8]) {     // h of a run, stored
    float b[8];
    load_row8(x, k0, p.K, p.vec, a);
    if (r) {
      load_row8(r, k0, p.K, p.vec, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = to_f(from_f<TX>(__fadd_rn(a[i], b[i])));
    }
    if (h != x || r) store_row8(h, k0, p.K, p.vec, a);
  };
  auto join = [](Two a, Two b) {                 // their sum, lo not brought below hi's last bit
    const Two t = two_sum(a.hi, b.hi);
    return Two{t.hi, __fadd_rn(__fadd_rn(a.lo, b.lo), t.lo)};
  };
  auto total = [&](Two s) {                      // over the CTA, the same in every thread
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      s = join(s, Two{__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)});
    if (nt == 32) return quick_two(s.hi, s.lo);
    __syncthreads();                             // of the pass before
    if (lane == 0) part[warp] = make_float2(s.hi, s.lo);
    __syncthreads();
    float2 q = part[0];
    Two t = {q.x, q.y};
    if (nt <= 256) {
      for (int w = 1; w < nt / 32; ++w) {
        q = part[w];
        t = join(t, Two{q.x, q.y});
      }
    } else {
      q = lane < nt / 32 ? part[lane] : make_float2(0.f, 0.f);
      t = {q.x, q.y};
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        t = join(t, Two{__shfl_xor_sync(0xffffffffu, t.hi, o), __shfl_xor_sync(0xffffffffu, t.lo, o)});
    }
    return quick_two(t.hi, t.lo);
  };

  Two s;
  float f = 1.f, ef;
  for (int pass = 0;; ++pass) {
    s = {0.f, 0.f};
    for (int run = tid; run < runs; run += nt) {
      if (pass == 0) joined(run * 8, v);
      else load_row8(h, run * 8, p.K, p.vec, v);
      sum_up(v, f, s);
    }
    s = total(s);
    // fp32 holds the squares' sum to the last bits of two floats between about
    // 2^-79 a value and 2^120 in all
    ef = p.eps * f * f;
    if (pass == 0 && !(s.hi + ef < 1.329e36f)) f = 8.2718061255302767e-25f;                       // 2^-80
    else if (pass < 2 && f >= 1.f && s.hi * p.inv_k.hi + ef < 1.654e-24f) f = pass ? 1.3292279957849159e36f   // 2^120
                                                                                   : 1.8446744073709552e19f;  // 2^64
    else break;
  }
  const Two rs = inverse_root(s, p.inv_k, ef);
  for (int run0 = 0; run0 < runs; run0 += nt) {
    const int run = run0 + tid, k0 = run * 8;
    float y[8], g[8];
    load_row8(h, k0, run < runs ? p.K : 0, p.vec, v);
    load_row8(p.gain, k0, run < runs ? p.K : 0, p.gain_vec, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = v[i] * f;
      Two q = two_prod(a, rs.hi);
      q.lo = __fmaf_rn(a, rs.lo, q.lo);
      const Two z = two_prod(q.hi, g[i]);
      y[i] = k0 + i < p.K ? round_odd(quick_two(z.hi, __fmaf_rn(q.lo, g[i], z.lo))) : 0.f;
    }
    uint32_t byte;
    const uint2 c = round8(y, (k0 & ~31) < p.K, byte);
    const uint32_t w = scale_word(byte, lane);
    if (run >= runs) continue;
    store_codes8(p.y8 + row * p.ld8, k0, p.K, c);
    if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(p.scale + mx_scale_at(row, run >> 4, KT)) = w;
  }
}

// The same for aligned rows with K a multiple of 8 and up to 2,048 runs, C of them
// a thread, held in registers, with two floats an instruction.  y is taken in fp32
// first, and where that is too near the middle of two codes, or a group's largest
// value too near the end of a scale's reach, with the 44 bits.  8,000 x 2,560 fp32
// rows with a bf16 residual take 37.6 us (6.0 TB/s); with an instruction for each
// float it was bound by those, 62 a value, and took 50.9.
template <typename TX, typename TR, int C>
__global__ void __launch_bounds__(C == 1 ? 128 : C == 2 ? 256 : 512) add_rmsnorm_mx8_vec_kernel(AddNormMx8Args p) {
  __shared__ float2 part[32];
  // C = 1: a row each for four warps
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tid = C == 1 ? lane : threadIdx.x, nt = C == 1 ? 32 : blockDim.x;
  const int KT = (p.K + 127) / 128;
  const long long row = C == 1 ? blockIdx.x * 4LL + warp : blockIdx.x;
  if (row >= p.T) return;
  const TX* x = static_cast<const TX*>(p.x) + row * p.ldx;
  const TR* r = p.r ? static_cast<const TR*>(p.r) + row * p.ldr : nullptr;
  TX* h = static_cast<TX*>(p.h) + row * p.ldh;
  pdl_launch_next();
  pdl_wait();

  Raw8<TX> xs[C];
  Raw8<TR> rs8[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int k0 = (tid + c * nt) * 8;
    xs[c].zero();
    rs8[c].zero();
    if (k0 < p.K) {
      xs[c].load(x + k0);
      if (r) rs8[c].load(r + k0);
    }
  }
  F2 v[C][4];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int k0 = (tid + c * nt) * 8;
    xs[c].get(v[c]);
    if (r) {
      F2 b[4];
      rs8[c].get(b);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[c][i] = f2_add(v[c][i], b[i]);
        if (sizeof(TX) == 2) {
          float lo, hi;
          f2_split(v[c][i], lo, hi);
          const __nv_bfloat162 q = __floats2bfloat162_rn(lo, hi);
          w[i] = *reinterpret_cast<const uint32_t*>(&q);
          v[c][i] = f2(bf16lo(w[i]), bf16hi(w[i]));
        }
      }
      if (k0 < p.K) {
        if (sizeof(TX) == 2) {
          *reinterpret_cast<uint4*>(h + k0) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          reinterpret_cast<ulonglong2*>(h + k0)[0] = make_ulonglong2(v[c][0], v[c][1]);
          reinterpret_cast<ulonglong2*>(h + k0)[1] = make_ulonglong2(v[c][2], v[c][3]);
        }
      }
    } else if (h != x && k0 < p.K) {
      *reinterpret_cast<uint4*>(h + k0) = xs[c].a;
      if (sizeof(TX) == 4) reinterpret_cast<ulonglong2*>(h + k0)[sizeof(TX) == 4] = make_ulonglong2(v[c][2], v[c][3]);
    }
  }

  auto join = [](Two a, Two b) {                 // their sum, lo not brought below hi's last bit
    const Two t = two_sum(a.hi, b.hi);
    return Two{t.hi, __fadd_rn(__fadd_rn(a.lo, b.lo), t.lo)};
  };
  // The sum of (f v)^2 over the CTA, the same in every thread.
  auto sum_up = [&](float f) {
    F2 s = 0, lo = 0;
    const F2 ff = f2(f, f), minus = f2(-1.f, -1.f);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const F2 a = f == 1.f ? v[c][i] : f2_mul(v[c][i], ff);
        // q - a^2, exactly: nothing where the values have 8 bits
        const F2 q = f2_mul(a, a), miss = sizeof(TX) == 2 ? 0 : f2_fma(f2_mul(a, minus), a, q);
        const F2 t = f2_add(s, q), b = f2_sub(t, s);
        const F2 err = f2_add(f2_sub(s, f2_sub(t, b)), f2_sub(q, b));
        lo = f2_add(lo, sizeof(TX) == 2 ? err : f2_sub(err, miss));
        s = t;
      }
    float s0, s1, l0, l1;
    f2_split(s, s0, s1);
    f2_split(lo, l0, l1);
    Two t = join(Two{s0, l0}, Two{s1, l1});
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      t = join(t, Two{__shfl_xor_sync(0xffffffffu, t.hi, o), __shfl_xor_sync(0xffffffffu, t.lo, o)});
    if (C > 1) {
      __syncthreads();                           // of the pass before
      if (lane == 0) part[warp] = make_float2(t.hi, t.lo);
      __syncthreads();
      float2 q = part[0];
      t = {q.x, q.y};
      for (int w = 1; w < nt / 32; ++w) {
        q = part[w];
        t = join(t, Two{q.x, q.y});
      }
    }
    return quick_two(t.hi, t.lo);
  };
  float f = 1.f;
  Two s = sum_up(1.f);
  float ef = p.eps;
  // fp32 holds the squares' sum to the last bits of two floats between about
  // 2^-79 a value and 2^120 in all
  if (!(s.hi + ef < 1.329e36f && s.hi * p.inv_k.hi + ef >= 1.654e-24f))
    for (int pass = 0; pass < 3; ++pass) {
      if (pass == 0 && !(s.hi + ef < 1.329e36f)) f = 8.2718061255302767e-25f;                         // 2^-80
      else if (pass < 2 && f >= 1.f && s.hi * p.inv_k.hi + ef < 1.654e-24f) f = pass ? 1.3292279957849159e36f   // 2^120
                                                                                     : 1.8446744073709552e19f;  // 2^64
      else break;
      s = sum_up(f);
      ef = p.eps * f * f;
    }
  const Two rs = inverse_root(s, p.inv_k, ef);

#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int run = tid + c * nt, k0 = run * 8, kt = run >> 4;
    Raw8<float> graw;
    graw.zero();
    if (k0 < p.K) graw.load(p.gain + k0);
    F2 g[4], y[4];
    graw.get(g);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = f2_mul(f2_mul(v[c][i], f2(rs.hi, rs.hi)), g[i]);   // off by less than 2^-22
    const uint32_t m = __float_as_uint(max_of_group(f2_max8(y)));
    const int e = exponent_of_bits(m);
    const float q = mx_pow2(-min(e, kMxEMax));
    uint2 code = f2_e4m3(y, q * (1.f - 4.76837158203125e-7f));                            // 1 -+ 2^-21
    const uint2 above = f2_e4m3(y, q * (1.f + 4.76837158203125e-7f));
    // sure where both are the same, the group's largest is 16 steps from the end of a
    // scale's reach or more, and it is far from fp32's ends: 2^-100 to 2^127
    const bool sure = f == 1.f && code.x == above.x && code.y == above.y &&
                      (m == 0u || (((m + 0x20000fu) & 0x7fffffu) >= 0x20u && m - 0x0d800000u < 0x71800000u));
    uint32_t byte = (k0 & ~31) < p.K ? (uint32_t)(e + 127) : 127u;
    if (__any_sync(0xffffffffu, !sure)) {
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float a[2], b[2];
        f2_split(v[c][i / 2], a[0], a[1]);
        f2_split(g[i / 2], b[0], b[1]);
        const float af = a[i % 2] * f;
        Two z = two_prod(af, rs.hi);
        z.lo = __fmaf_rn(af, rs.lo, z.lo);
        const Two t = two_prod(z.hi, b[i % 2]);
        w[i] = k0 < p.K ? round_odd(quick_two(t.hi, __fmaf_rn(z.lo, b[i % 2], t.lo))) : 0.f;
      }
      code = round8(w, (k0 & ~31) < p.K, byte);
    }
    const uint32_t w = scale_word(byte, lane);
    if (kt >= KT) continue;
    if (k0 < p.K) *reinterpret_cast<uint2*>(p.y8 + row * p.ld8 + k0) = code;
    if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(p.scale + mx_scale_at(row, kt, KT)) = w;
  }
}

// ---------------------------------------------------------------- weights to 4 bits and back

// As mx8_pack_kernel, eight values to a word of codes.  A group that holds a
// NaN or an infinity gets the scale NaN.
template <typename T>
__global__ void __launch_bounds__(256) w4_pack_kernel(W4PackArgs p) {
  const int lane = threadIdx.x & 31, KT = (p.K + 127) / 128, rows = 16 / KT, kts = 16 % KT;
  const Units first(KT);
  Units u = first;
  float v[kUnits][8];
#pragma unroll
  for (int i = 0; i < kUnits; ++i, u.next(KT, rows, kts))
    load_row8(static_cast<const T*>(p.w) + u.row * p.ldw, u.kt * 128 + (lane & 15) * 8, u.row < p.N ? p.K : 0, p.vec,
              v[i]);
  u = first;
#pragma unroll
  for (int i = 0; i < kUnits; ++i, u.next(KT, rows, kts)) {
    const int k0 = u.kt * 128 + (lane & 15) * 8;
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) odd |= !(fabsf(v[i][j]) < __uint_as_float(0x7f800000u));
    const float m = max_of_group(odd ? __uint_as_float(0x7f800000u) : max8(v[i]));
    const bool nan = m == __uint_as_float(0x7f800000u);
    const int e = mx4_exponent(m);
    const float f = mx_pow2(-e);
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) c |= mx_e2m1x2(v[i][2 * j] * f, v[i][2 * j + 1] * f) << (8 * j);
    if (nan) c = 0;
    const uint32_t w = scale_word((k0 & ~31) >= p.K ? 127u : nan ? 255u : (uint32_t)(e + 127), lane);
    if (u.row >= p.N) continue;
    *reinterpret_cast<uint32_t*>(p.codes + (size_t)u.row * (KT * 64) + k0 / 2) = c;
    if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(p.scale + mx_scale_at(u.row, u.kt, KT)) = w;
  }
}

// Aligned rows with K a multiple of 8, as mx8_pack_vec_kernel.
template <typename T>
__global__ void __launch_bounds__(256, 5) w4_pack_vec_kernel(W4PackArgs p) {
  constexpr int U = kVecRows<T>;
  const int lane = threadIdx.x & 31, KT = (p.K + 127) / 128;
  const Strip s(KT, U);
  const bool in = s.k0 < p.K;
  const T* x = static_cast<const T*>(p.w) + s.row0 * p.ldw + s.k0;
  Raw8<T> raw[U];
#pragma unroll
  for (int i = 0; i < U; ++i, x += p.ldw) {
    if (in && s.row0 + i < p.N) raw[i].load(x);
    else raw[i].zero();
  }
  uint8_t* codes = p.codes + (size_t)s.row0 * (KT * 64) + s.k0 / 2;
  uint8_t* scale = p.scale + mx_scale_at(s.row0, s.kt, KT);
#pragma unroll
  for (int i = 0; i < U; ++i, codes += KT * 64, scale += 16) {
    F2 v[4];
    raw[i].get(v);
    const uint32_t m = raw[i].group_max();
    const bool nan = m >= 0x7f800000u;
    // 1.5 is 0x400000 of a mantissa
    const int e = min(max((int)((m + 0x3fffffu) >> 23) - 129, kMxEMin), kMxEMax);
    const float q = mx_pow2(-e);
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a, b;
      f2_split(f2_mul(v[j], f2(q, q)), a, b);
      c |= mx_e2m1x2(a, b) << (8 * j);
    }
    const uint32_t w = scale_word((s.k0 & ~31) >= p.K ? 127u : nan ? 255u : (uint32_t)(e + 127), lane);
    if (s.row0 + i >= p.N) break;      // the whole warp
    if (s.kt < KT) {
      *reinterpret_cast<uint32_t*>(codes) = nan ? 0u : c;
      if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(scale) = w;
    }
  }
}

// Two e2m1 codes (a byte's) as floats.
S2_DEV F2 f2_of_e2m1x2(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(byte));
  float a, b;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(a), "=f"(b) : "r"(h));
  return f2(a, b);
}

template <typename T>
__global__ void __launch_bounds__(256) w4_unpack_kernel(W4PackArgs p) {
  const int lane = threadIdx.x & 31, KT = (p.K + 127) / 128, rows = 16 / KT, kts = 16 % KT;
  const Units first(KT);
  Units u = first;
  uint32_t c[kUnits], w[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i, u.next(KT, rows, kts)) {
    c[i] = w[i] = 0;
    if (u.row < p.N) {
      c[i] = *reinterpret_cast<const uint32_t*>(p.codes + (size_t)u.row * (KT * 64) + u.kt * 64 + (lane & 15) * 4);
      w[i] = *reinterpret_cast<const uint32_t*>(p.scale + mx_scale_at(u.row, u.kt, KT));
    }
  }
  u = first;
#pragma unroll
  for (int i = 0; i < kUnits; ++i, u.next(KT, rows, kts)) {
    if (u.row >= p.N) continue;
    const float s = mx_scale((w[i] >> (((lane >> 2) & 3) * 8)) & 255u);
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) f2_split(f2_mul(f2_of_e2m1x2(c[i] >> (8 * j)), f2(s, s)), v[2 * j], v[2 * j + 1]);
    store_row8(static_cast<T*>(p.w) + u.row * p.ldw, u.kt * 128 + (lane & 15) * 8, p.K, p.vec, v);
  }
}

// Aligned rows with K a multiple of 8.
template <typename T>
__global__ void __launch_bounds__(256) w4_unpack_vec_kernel(W4PackArgs p) {
  constexpr int U = 4;
  const int lane = threadIdx.x & 31, KT = (p.K + 127) / 128;
  const Strip s(KT, U);
  if (s.k0 >= p.K) return;
  const uint8_t* codes = p.codes + (size_t)s.row0 * (KT * 64) + s.k0 / 2;
  const uint8_t* scale = p.scale + mx_scale_at(s.row0, s.kt, KT) + ((lane >> 2) & 3);
  uint32_t c[U], e[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    c[i] = e[i] = 0;
    if (s.row0 + i < p.N) {
      c[i] = *reinterpret_cast<const uint32_t*>(codes + (size_t)i * (KT * 64));
      e[i] = scale[16 * i];
    }
  }
  T* w = static_cast<T*>(p.w) + s.row0 * p.ldw + s.k0;
#pragma unroll
  for (int i = 0; i < U; ++i, w += p.ldw) {
    if (s.row0 + i >= p.N) break;
    const float f = mx_scale(e[i]);
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) f2_split(f2_mul(f2_of_e2m1x2(c[i] >> (8 * j)), f2(f, f)), v[2 * j], v[2 * j + 1]);
    store_row8(w, 0, 8, true, v);
  }
}

// early: the CTAs may come to their SMs before the kernel ahead in the stream
// has ended, and wait there.
cudaError_t launch(const void* k, dim3 grid, int threads, void** args, cudaStream_t st, bool early) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = early ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, k, args);
  if (e == cudaSuccess) ++g_launch_count;
  return e;
}

unsigned unit_blocks(long long rows, int K) {
  const long long n = (rows * ((K + 127) / 128) + 16 * kUnits - 1) / (16 * kUnits);
  return n <= 0x7fffffff ? (unsigned)n : 0;      // a grid of 0 is refused
}
// Strips of 256 columns and ``step`` rows, eight a CTA, counted in 31 bits.
bool strips_fit(long long rows, int K) { return rows * ((K + 255) / 256) < 0x7fff0000LL; }
unsigned strip_blocks(long long rows, int K, int step) {
  return (unsigned)(((rows + step - 1) / step * ((K + 255) / 256) + 7) / 8);
}

}  // namespace

cudaError_t launch_mx8_pack(const Mx8PackArgs& p, cudaStream_t st) {
  void* args[] = {const_cast<Mx8PackArgs*>(&p)};
  const bool vec = p.vec && p.K % 8 == 0 && strips_fit(p.T, p.K);
  const void* k = vec ? (p.x_bf16 ? (const void*)mx8_pack_vec_kernel<__nv_bfloat16> : (const void*)mx8_pack_vec_kernel<float>)
                      : (p.x_bf16 ? (const void*)mx8_pack_kernel<__nv_bfloat16> : (const void*)mx8_pack_kernel<float>);
  const int rows = p.x_bf16 ? kVecRows<__nv_bfloat16> : kVecRows<float>;
  return launch(k, dim3(vec ? strip_blocks(p.T, p.K, rows) : unit_blocks(p.T, p.K)), 256, args, st, true);
}

// Variants by type and, for aligned rows of up to 2,048 runs, runs a thread: one in
// a single warp; two, which halve what the sum over the CTA costs a value; four,
// where with two an SM would hold two CTAs only and wait for one's loads under the
// other's barriers (2,000 x 9,728 fp32 rows 63 -> 52 us).
template <typename TX, typename TR>
static const void* norm_kernel(int c) {
  return c == 1   ? (const void*)add_rmsnorm_mx8_vec_kernel<TX, TR, 1>
         : c == 2 ? (const void*)add_rmsnorm_mx8_vec_kernel<TX, TR, 2>
         : c == 4 ? (const void*)add_rmsnorm_mx8_vec_kernel<TX, TR, 4>
                  : (const void*)add_rmsnorm_mx8_kernel<TX, TR>;
}

cudaError_t launch_add_rmsnorm_mx8(const AddNormMx8Args& p, cudaStream_t st) {
  void* args[] = {const_cast<AddNormMx8Args*>(&p)};
  const int runs = (p.K + 127) / 128 * 16;
  const int c = !p.vec || !p.gain_vec || p.K % 8 ? 0 : runs <= 32 ? 1 : runs <= 512 ? 2 : runs <= 2048 ? 4 : 0;
  const int nt = c == 1 ? 128 : c ? ((runs + c - 1) / c + 31) / 32 * 32 : runs < 1024 ? (runs + 31) / 32 * 32 : 1024;
  const void* k = p.x_bf16 ? p.r_bf16 ? norm_kernel<__nv_bfloat16, __nv_bfloat16>(c) : norm_kernel<__nv_bfloat16, float>(c)
                  : p.r_bf16 ? norm_kernel<float, __nv_bfloat16>(c)
                             : norm_kernel<float, float>(c);
  return launch(k, dim3(c == 1 ? (p.T + 3) / 4 : p.T), nt, args, st, true);
}

cudaError_t launch_w4_pack(const W4PackArgs& p, cudaStream_t st) {
  void* args[] = {const_cast<W4PackArgs*>(&p)};
  const bool vec = p.vec && p.K % 8 == 0 && strips_fit(p.N, p.K);
  const void* k = vec ? (p.w_bf16 ? (const void*)w4_pack_vec_kernel<__nv_bfloat16> : (const void*)w4_pack_vec_kernel<float>)
                      : (p.w_bf16 ? (const void*)w4_pack_kernel<__nv_bfloat16> : (const void*)w4_pack_kernel<float>);
  const int rows = p.w_bf16 ? kVecRows<__nv_bfloat16> : kVecRows<float>;
  return launch(k, dim3(vec ? strip_blocks(p.N, p.K, rows) : unit_blocks(p.N, p.K)), 256, args, st, false);
}

cudaError_t launch_w4_unpack(const W4PackArgs& p, cudaStream_t st) {
  void* args[] = {const_cast<W4PackArgs*>(&p)};
  const bool vec = p.vec && p.K % 8 == 0 && strips_fit(p.N, p.K);
  const void* k =
      vec ? (p.w_bf16 ? (const void*)w4_unpack_vec_kernel<__nv_bfloat16> : (const void*)w4_unpack_vec_kernel<float>)
          : (p.w_bf16 ? (const void*)w4_unpack_kernel<__nv_bfloat16> : (const void*)w4_unpack_kernel<float>);
  return launch(k, dim3(vec ? strip_blocks(p.N, p.K, 4) : unit_blocks(p.N, p.K)), 256, args, st, false);
}

}  // namespace s2
