// Rounding of rows to 8-bit and 4-bit values with a power of two per 32 of
// them (mx_common.cuh): activations, the residual's addition with RMSNorm and
// such an output, weights, and weights back.
#include "mx_common.cuh"
#include "two_float.cuh"

namespace s2 {

namespace {

// Values k0 .. k0 + 7 of a row as floats, zeros from K on.  vec: rows start on
// 16-byte boundaries.
template <typename T>
S2_DEV void load_row8(const T* __restrict__ row, int k0, int K, bool vec, float (&v)[8]) {
  if (vec && k0 + 8 <= K) {
    load8(row + k0, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k0 + i < K ? to_f(row[k0 + i]) : 0.f;
  }
}
template <typename T>
S2_DEV void store_row8(T* __restrict__ row, int k0, int K, bool vec, const float (&v)[8]) {
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

// ---------------------------------------------------------------- rows to 8 bits

constexpr int kUnits = 4;   // (row, 128 values) of a half-warp, all loaded before the first is rounded

template <typename T>
__global__ void __launch_bounds__(256) mx8_pack_kernel(Mx8PackArgs p) {
  pdl_launch_next();
  pdl_wait();
  const int lane = threadIdx.x & 31, KT = (p.K + 127) / 128;
  const long long units = (long long)p.T * KT;
  const long long u0 = (long long)blockIdx.x * (16 * kUnits) + (threadIdx.x >> 4);
  float v[kUnits][8];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const long long u = u0 + 16 * i;
    const long long row = u / KT;
    const int k0 = (int)(u - row * KT) * 128 + (lane & 15) * 8;
    if (u < units) {
      load_row8(static_cast<const T*>(p.x) + row * p.ldx, k0, p.K, p.vec, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const long long u = u0 + 16 * i;
    const long long row = u / KT;
    const int kt = (int)(u - row * KT), k0 = kt * 128 + (lane & 15) * 8;
    uint32_t byte;
    const uint2 c = round8(v[i], (k0 & ~31) < p.K, byte);
    const uint32_t w = scale_word(byte, lane);
    if (u >= units) continue;
    store_codes8(p.y8 + row * p.ld8, k0, p.K, c);
    if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(p.scale + mx_scale_at(row, kt, KT)) = w;
  }
}

// ---------------------------------------------------------------- residual + RMSNorm to 8 bits

// One CTA per row: h = x + r (rounded to x's type and stored), then y = h /
// sqrt(mean h^2 + eps) * gain to e4m3 with scales.  The result is rounded to
// 8 bits at once, so it is computed to about 2^-44 (sum of squares, inverse
// root and products as unevaluated sums of two floats): the codes are those
// of the exact values whatever the order of the sum.  A thread holds its
// values in registers between the sum and the rounding (C runs of 8; C = 0:
// any length, h read back).  A row whose sum of squares leaves fp32's range
// is taken once more scaled by 2^-80 or 2^64 (2^120).  A row with a NaN or an
// infinity is NaN throughout.
template <typename TX, typename TR, int C>
__global__ void __launch_bounds__(1024) add_rmsnorm_mx8_kernel(AddNormMx8Args p) {
  __shared__ float part[2][32];
  pdl_launch_next();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
  const int KT = (p.K + 127) / 128;
  const long long row = blockIdx.x;
  const TX* x = static_cast<const TX*>(p.x) + row * p.ldx;
  const TR* r = p.r ? static_cast<const TR*>(p.r) + row * p.ldr : nullptr;
  TX* h = static_cast<TX*>(p.h) + row * p.ldh;
  const int runs = KT * 16;               // runs of 8 values, the row's padding included
  constexpr int CR = C ? C : 1;
  float v[CR][8];

  auto sum_up = [](const float (&a)[8], float f, Two& s) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const Two q = two_prod(a[i] * f, a[i] * f);
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
  auto total = [&](Two s) {                      // over the CTA, the same in every thread
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      s = add(s, Two{__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)});
    __syncthreads();
    if (lane == 0) {
      part[0][warp] = s.hi;
      part[1][warp] = s.lo;
    }
    __syncthreads();
    Two t = lane < nt / 32 ? Two{part[0][lane], part[1][lane]} : Two{0.f, 0.f};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      t = add(t, Two{__shfl_xor_sync(0xffffffffu, t.hi, o), __shfl_xor_sync(0xffffffffu, t.lo, o)});
    return t;
  };

  Two s;
  float f = 1.f, ef;
  for (int pass = 0;; ++pass) {
    s = {0.f, 0.f};
    if (C) {
#pragma unroll
      for (int c = 0; c < CR; ++c) {
        const int run = tid + c * nt;
        if (pass == 0) {
          if (run < runs) {
            joined(run * 8, v[c]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] = 0.f;
          }
        }
        sum_up(v[c], f, s);
      }
    } else {
      for (int run = tid; run < runs; run += nt) {
        if (pass == 0) joined(run * 8, v[0]);
        else load_row8(h, run * 8, p.K, p.vec, v[0]);
        sum_up(v[0], f, s);
      }
    }
    s = total(s);
    // fp32 holds the squares' sum to the last bits of two floats between about
    // 2^-79 a value and 2^120 in all
    ef = p.eps * f * f;
    if (pass == 0 && !(s.hi < 1.329e36f)) f = 8.2718061255302767e-25f;                       // 2^-80
    else if (pass < 2 && f >= 1.f && s.hi * p.inv_k.hi + ef < 1.654e-24f) f = pass ? 1.3292279957849159e36f   // 2^120
                                                                                   : 1.8446744073709552e19f;  // 2^64
    else break;
  }
  // 1 / sqrt(s / K + eps): a Newton step on the float one
  Two m = two_prod(s.hi, p.inv_k.hi);
  m.lo = __fmaf_rn(s.hi, p.inv_k.lo, __fmaf_rn(s.lo, p.inv_k.hi, m.lo));
  m = add(quick_two(m.hi, m.lo), Two{ef, 0.f});
  Two rs;
  if (m.hi < __uint_as_float(0x7f800000u) && m.hi > 0.f) {
    const float r0 = rsqrtf(m.hi);
    const Two q = two_prod(r0, r0);
    Two t = mul(m, q.hi);
    t.lo = __fmaf_rn(m.hi, q.lo, t.lo);
    const float d = __fsub_rn(__fsub_rn(1.f, t.hi), t.lo);
    rs = quick_two(r0, __fmul_rn(__fmul_rn(0.5f, r0), d));
  } else {
    rs = {__uint_as_float(0x7fffffffu), 0.f};   // a NaN or an infinity in the row, or nothing at all without eps
  }
  auto finish = [&](int run, float (&a)[8]) {
    const int k0 = run * 8, kt = run >> 4;
    float y[8], g[8];
    load_row8(p.gain, k0, p.K, p.gain_vec, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float af = a[i] * f;
      Two q = two_prod(af, rs.hi);
      q.lo = __fmaf_rn(af, rs.lo, q.lo);
      const Two t = two_prod(q.hi, g[i]);
      y[i] = round_odd(quick_two(t.hi, __fmaf_rn(q.lo, g[i], t.lo)));
    }
    if (k0 + 8 > p.K)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k0 + i >= p.K) y[i] = 0.f;
    uint32_t byte;
    const uint2 c = round8(y, (k0 & ~31) < p.K, byte);
    const uint32_t w = scale_word(byte, lane);
    if (run < runs) {
      store_codes8(p.y8 + row * p.ld8, k0, p.K, c);
      if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(p.scale + mx_scale_at(row, kt, KT)) = w;
    }
  };
  if (C) {
#pragma unroll
    for (int c = 0; c < CR; ++c) finish(tid + c * nt, v[c]);
  } else {
    for (int run0 = 0; run0 < runs; run0 += nt) {
      const int run = run0 + tid;
      load_row8(h, run * 8, run < runs ? p.K : 0, p.vec, v[0]);
      finish(run, v[0]);
    }
  }
}

// ---------------------------------------------------------------- weights to 4 bits and back

// As mx8_pack_kernel, eight values to a word of codes.  A group that holds a
// NaN or an infinity gets the scale NaN.
template <typename T>
__global__ void __launch_bounds__(256) w4_pack_kernel(W4PackArgs p) {
  const int lane = threadIdx.x & 31, KT = (p.K + 127) / 128;
  const long long units = (long long)p.N * KT;
  const long long u0 = (long long)blockIdx.x * (16 * kUnits) + (threadIdx.x >> 4);
  float v[kUnits][8];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const long long u = u0 + 16 * i;
    const long long row = u / KT;
    const int k0 = (int)(u - row * KT) * 128 + (lane & 15) * 8;
    if (u < units) {
      load_row8(static_cast<const T*>(p.w) + row * p.ldw, k0, p.K, p.vec, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const long long u = u0 + 16 * i;
    const long long row = u / KT;
    const int kt = (int)(u - row * KT), k0 = kt * 128 + (lane & 15) * 8;
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
    if (u >= units) continue;
    *reinterpret_cast<uint32_t*>(p.codes + (size_t)row * (KT * 64) + k0 / 2) = c;
    if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(p.scale + mx_scale_at(row, kt, KT)) = w;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) w4_unpack_kernel(W4PackArgs p) {
  const int lane = threadIdx.x & 31, KT = (p.K + 127) / 128;
  const long long units = (long long)p.N * KT;
  const long long u0 = (long long)blockIdx.x * (16 * kUnits) + (threadIdx.x >> 4);
  uint32_t c[kUnits], w[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const long long u = u0 + 16 * i;
    const long long row = u / KT;
    const int kt = (int)(u - row * KT), k0 = kt * 128 + (lane & 15) * 8;
    c[i] = w[i] = 0;
    if (u < units) {
      c[i] = *reinterpret_cast<const uint32_t*>(p.codes + (size_t)row * (KT * 64) + k0 / 2);
      w[i] = *reinterpret_cast<const uint32_t*>(p.scale + mx_scale_at(row, kt, KT));
    }
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const long long u = u0 + 16 * i;
    const long long row = u / KT;
    const int k0 = (int)(u - row * KT) * 128 + (lane & 15) * 8;
    if (u >= units) continue;
    const float s = mx_scale((w[i] >> (((lane >> 2) & 3) * 8)) & 255u);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = mx_e2m1((c[i] >> (4 * j)) & 15u) * s;
    store_row8(static_cast<T*>(p.w) + row * p.ldw, k0, p.K, p.vec, v);
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
  return (unsigned)((rows * ((K + 127) / 128) + 16 * kUnits - 1) / (16 * kUnits));
}

}  // namespace

cudaError_t launch_mx8_pack(const Mx8PackArgs& p, cudaStream_t st) {
  void* args[] = {const_cast<Mx8PackArgs*>(&p)};
  const void* k = p.x_bf16 ? (const void*)mx8_pack_kernel<__nv_bfloat16> : (const void*)mx8_pack_kernel<float>;
  return launch(k, dim3(unit_blocks(p.T, p.K)), 256, args, st, true);
}

template <int C>
static const void* norm_kernel(const AddNormMx8Args& p) {
  if (p.x_bf16)
    return p.r_bf16 ? (const void*)add_rmsnorm_mx8_kernel<__nv_bfloat16, __nv_bfloat16, C>
                    : (const void*)add_rmsnorm_mx8_kernel<__nv_bfloat16, float, C>;
  return p.r_bf16 ? (const void*)add_rmsnorm_mx8_kernel<float, __nv_bfloat16, C>
                  : (const void*)add_rmsnorm_mx8_kernel<float, float, C>;
}

cudaError_t launch_add_rmsnorm_mx8(const AddNormMx8Args& p, cudaStream_t st) {
  void* args[] = {const_cast<AddNormMx8Args*>(&p)};
  const int runs = (p.K + 127) / 128 * 16;
  // threads: a run of 8 each up to 512 of them, then two, then any number
  const int c = runs <= 512 ? 1 : runs <= 2048 ? 2 : 0;
  const int nt = c ? ((runs + c - 1) / c + 31) / 32 * 32 : 1024;
  const void* k = c == 1 ? norm_kernel<1>(p) : c == 2 ? norm_kernel<2>(p) : norm_kernel<0>(p);
  return launch(k, dim3(p.T), nt, args, st, true);
}

cudaError_t launch_w4_pack(const W4PackArgs& p, cudaStream_t st) {
  void* args[] = {const_cast<W4PackArgs*>(&p)};
  const void* k = p.w_bf16 ? (const void*)w4_pack_kernel<__nv_bfloat16> : (const void*)w4_pack_kernel<float>;
  return launch(k, dim3(unit_blocks(p.N, p.K)), 256, args, st, false);
}

cudaError_t launch_w4_unpack(const W4PackArgs& p, cudaStream_t st) {
  void* args[] = {const_cast<W4PackArgs*>(&p)};
  const void* k = p.w_bf16 ? (const void*)w4_unpack_kernel<__nv_bfloat16> : (const void*)w4_unpack_kernel<float>;
  return launch(k, dim3(unit_blocks(p.N, p.K)), 256, args, st, false);
}

}  // namespace s2
