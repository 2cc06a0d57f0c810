// Prompt attention over the 8-bit KV cache on tcgen05: ragged prompts behind
// cached pages, grouped queries, causal.
#include <algorithm>
#include <type_traits>

#include "kv8_common.cuh"
#include "tc_common.cuh"

namespace s2 {

namespace {

constexpr int kPreRows = 128;                 // rows of a query tile; two tiles a CTA
constexpr int kPreKeys = 128;                 // keys of a step
constexpr int kPrePages = kPreKeys / kKv8Page;
constexpr int kPreSmem = 227 * 1024;
constexpr int kPreTmem = 512;                 // S / P of two tiles, O of two tiles
// Weights carry 2^bias, and the running maximum may lag by ``lag``: they are 2^15 at
// most.  f16 pairs (an fp32 output) get the better resolution of a short lag, which
// costs more rescaling where scores are large (single f16, gains of 5: 607 us for
// 8,000 tokens with a lag of 4, 572 with 8).
template <int PLANES>
struct PreScale {
  static constexpr int kBias = PLANES == 1 ? 7 : 11, kLag = 15 - kBias;
};
// Binades by which the value scales of a step's pages may lie below the largest one
// met: the values then are f16 relative to the step's largest (exactly), and the
// step's weights carry that one.  The row's largest weight still stands at 2^-7
// (pairs: 2^-3) then, so that the others are good to 2^-18 (2^-22) of it.  A step
// with a page further down goes page by page (spread_step), which takes three
// times as long, and more where pages are added apart.
constexpr int kPreFar = 14;
constexpr int kPreStepBytes = 4;              // what is kept of each step

// Groups of four warps: two of softmax, one for keys and one for values (one
// for both with an fp32 output, where the products take twice the time), one
// for the products.  The launch's registers are shared out anew among them:
// with an fp32 output a softmax thread holds its row's output too.  The keys'
// and values' warps want theirs for loads ahead (8,000 tokens: 561 us with 72 a
// thread, 511 with 88).
template <int PLANES>
struct PreRoles {
  static constexpr int kWiden = PLANES == 1 ? 2 : 1, kGroups = 3 + kWiden, kThreads = kGroups * 128;
  static constexpr int kMma = 8 + 4 * kWiden;                 // first warp of the products' group
  static constexpr int kRegs = PLANES == 1 ? 96 : 128;        // a thread, at launch
  static constexpr int kRegsSoftmax = PLANES == 1 ? 128 : 192, kRegsWiden = 88, kRegsMma = PLANES == 1 ? 48 : 40;
  // the shares are no more than the launch has, and each moves the way of its instruction
  static_assert(2 * kRegsSoftmax + kWiden * kRegsWiden + kRegsMma <= kGroups * kRegs, "the launch's registers");
  static_assert(kRegsSoftmax >= kRegs && kRegsWiden <= kRegs && kRegsMma <= kRegs, "inc and dec");
};

template <int HD, int PLANES>
struct PreLayout {
  static constexpr int kTile = 128 * HD * 2;                  // bytes of 128 rows in f16
  static constexpr int kStages = PLANES == 1 ? 2 : 1;
  static constexpr int kQ = 0;                                // [tile][plane]
  static constexpr int kK = kQ + 2 * PLANES * kTile;          // [stage]
  static constexpr int kV = kK + kStages * kTile;
  static constexpr int kMeta = kV + kStages * kTile;
};

template <int PLANES> struct OutOf { using type = float; };
template <> struct OutOf<1> { using type = __nv_bfloat16; };

// ---------------------------------------------------------------- tcgen05 pieces

// kind::f16 with f16 A and B, fp32 D; B is K-major, or MN-major if b_mn.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, int b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
// Shared-memory operands as the two words of their descriptors; the lower one,
// with the address, is all that differs between products.  128-byte swizzle,
// 8-row atoms of 128-byte rows one after the other.  K-major: the rows are M or
// N.  MN-major: the rows are K, 64 values along MN each, the next 64 values
// ``block`` bytes on.
constexpr uint32_t kDescHi = (1024 >> 4) | 1u << 14 | 2u << 29;   // atom stride, version, swizzle
S2_DEV uint32_t desc_k(uint32_t saddr) { return saddr >> 4 | 1u << 16; }
S2_DEV uint32_t desc_mn(uint32_t saddr, uint32_t block) { return saddr >> 4 | (block >> 4) << 16; }
S2_DEV void umma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}"
      :: "r"(d), "r"(a), "r"(b), "r"(idesc), "r"(accum), "r"(kDescHi) : "memory");
}
S2_DEV void umma_ts(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}"
      :: "r"(d), "r"(a_tmem), "r"(b), "r"(idesc), "r"(accum), "r"(kDescHi) : "memory");
}
// One lane of a converged warp, chosen such that the compiler knows that it is
// one: the products' operands then go to uniform registers as they are, where
// a branch by lane number has each of them moved there in a loop over lanes.
S2_DEV bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}
S2_DEV void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};"
      :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
         "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 32 columns of this thread's lane: the load, and the wait that the values may
// be used after.
S2_DEV void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
S2_DEV void tmem_ld32_done(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :: "memory");
}
S2_DEV void tmem_put8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
S2_DEV void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr) : "memory");
}
S2_DEV void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

S2_DEV void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];" :: "l"(p)); }
S2_DEV void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" :: "l"(p)); }
// A barrier of the n threads that are softmax rows.
S2_DEV void softmax_sync(int n) { asm volatile("bar.sync 1, %0;" :: "r"(n) : "memory"); }
template <int N>
S2_DEV void more_regs() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N)); }
template <int N>
S2_DEV void fewer_regs() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N)); }
S2_DEV float ex2p(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool VEC>
S2_DEV void load4(const float* p, float* v) {
  const float4 x = VEC ? *reinterpret_cast<const float4*>(p) : make_float4(p[0], p[1], p[2], p[3]);
  v[0] = x.x;
  v[1] = x.y;
  v[2] = x.z;
  v[3] = x.w;
}

// Two e4m3 bytes (the low ones of w) as f16x2 times f.
S2_DEV uint32_t widen(uint32_t w, __half2 f) {
  uint32_t h = f16x2_of_e4m3((uint16_t)w);
  const __half2 p = __hmul2(*reinterpret_cast<__half2*>(&h), f);
  return *reinterpret_cast<const uint32_t*>(&p);
}
// Nonzero if one of the four bytes is a NaN (0x7f or 0xff).
S2_DEV uint32_t has_nan(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
// The bytes without their NaNs.  A NaN must not reach rows that do not see it
// through 0 * NaN: it is left out of the products, and the first key that has
// one in this dim noted for the epilogue.
__device__ __noinline__ uint4 without_nan(uint4 y, int* first, int* any, int key) {
  uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if ((w[i / 4] >> (8 * (i % 4)) & 0x7f) == 0x7f) {
      atomicMin(first + i, key);
      *any = 1;
      w[i / 4] &= ~(0xffu << (8 * (i % 4)));
    }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// What is kept of a step: the largest scale exponent of its pages' keys, which
// pages are there (a bit each), the largest and the smallest exponent of their
// values.  Whether it goes page by page; e_top is the largest exponent of values so far.
S2_DEV bool goes_by_page(const char4& step, int& e_top) {
  e_top = max(e_top, (int)step.z);
  return step.w < e_top - kPreFar;
}

// A step of one row page by page: the row's maximum and sum as new (m, l), its
// weights to where the products read them, each with its page's scale.  A scale
// bounds its block's values, and a row may see none of the large ones: a page whose
// largest weight x scale is more than kPreFar binades below the row's is added to
// O by fp32 arithmetic.  In a code of its own, since steps like it are rare.  last:
// the row's last key of the step, left: the keys of the step, table: its pages.
// Called by whole warps.
template <int HD, int PLANES>
__device__ __noinline__ float2 spread_step(uint32_t t_o, uint32_t t_s, float f, float m, float l, int e_top, int last,
                                           uint32_t there, const Kv8Args& a, const int* table, int left, int g) {
  const int lane = threadIdx.x & 31;
  int e_page = kKv8EMin;                                   // of page ``lane``
  if (lane < kPrePages && lane * kKv8Page < left && (there >> lane & 1))
    e_page = kv8_scale_exp(a.scale[((size_t)table[lane] * 2 + 1) * a.Hkv + g]);
  __syncwarp();
  float s[kPreKeys];
#pragma unroll
  for (int c = 0; c < kPreKeys; c += 16) {
    uint32_t r[16];
    tmem_ld16(t_s + c, r);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      s[c + i] = c + i <= last && (there >> (c / kKv8Page) & 1) ? __uint_as_float(r[i]) : -INFINITY;
  }
  auto top_of = [&](int q) {                               // its largest score + exponent
    float x = -INFINITY;
#pragma unroll
    for (int i = 0; i < kKv8Page; ++i) x = fmaxf(x, s[kKv8Page * q + i]);
    return fmaf(x, f, (float)__shfl_sync(0xffffffffu, e_page, q));
  };
  float mx = -INFINITY;
#pragma unroll 1
  for (int q = 0; q < kPrePages; ++q) mx = fmaxf(mx, top_of(q));
  if (__any_sync(0xffffffffu, mx > m + (float)PreScale<PLANES>::kLag)) {
    const float mn = fmaxf(m, mx), y = mn == -INFINITY ? 1.f : ex2p(m - mn);
    l *= y;
    m = mn;
#pragma unroll 1
    for (int c = 0; c < HD; c += 8) {
      float o[8];
      tmem_ld8(t_o + c, o);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] *= y;
      tmem_st8(t_o + c, o);
    }
  }
  const float base = (float)PreScale<PLANES>::kBias - (m == -INFINITY ? 0.f : m);
#pragma unroll 1
  for (int q = 0; q < kPrePages; ++q) {
    const int e = __shfl_sync(0xffffffffu, e_page, q);
    const float off = (float)e + base, x = top_of(q);
    float p[kKv8Page], sum = 0.f;
#pragma unroll
    for (int i = 0; i < kKv8Page; ++i) {
      p[i] = ex2p(fmaf(s[kKv8Page * q + i], f, off));
      sum += p[i];
    }
    l = fmaf(sum, pow2f(-e - PreScale<PLANES>::kBias), l);
    if (__any_sync(0xffffffffu, e < e_top - kPreFar && x > -INFINITY && m - x > (float)kPreFar)) {
      const uint8_t* v = a.kv + (((size_t)table[q] * 2 + 1) * a.Hkv + g) * (kKv8Page * HD);
#pragma unroll 1
      for (int c = 0; c < HD; c += 8) {
        float o[8];
        tmem_ld8(t_o + c, o);
#pragma unroll
        for (int k = 0; k < kKv8Page; ++k) {
          const uint2 w = *reinterpret_cast<const uint2*>(v + k * HD + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t h = f16x2_of_e4m3((uint16_t)((i < 2 ? w.x : w.y) >> (i & 1) * 16));
            const float2 y = __half22float2(*reinterpret_cast<__half2*>(&h));
            o[2 * i] += y.x == y.x ? p[k] * y.x : 0.f;           // NaN: see nan_s
            o[2 * i + 1] += y.y == y.y ? p[k] * y.y : 0.f;
          }
        }
        tmem_st8(t_o + c, o);
      }
#pragma unroll
      for (int i = 0; i < kKv8Page; ++i) p[i] = 0.f;
    }
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __half2 h = __floats2half2_rn(p[2 * i], p[2 * i + 1]);
      const float2 hf = __half22float2(h);
      const __half2 d = __floats2half2_rn(p[2 * i] - hf.x, p[2 * i + 1] - hf.y);
      hi[i] = *reinterpret_cast<const uint32_t*>(&h);
      lo[i] = *reinterpret_cast<const uint32_t*>(&d);
    }
    tmem_put8(t_s + (PLANES == 1 ? 64 : 0) + 8 * q, hi);
    if (PLANES == 2) tmem_put8(t_s + 64 + 8 * q, lo);
  }
  return make_float2(m, l);
}

// ---------------------------------------------------------------- the kernel

// Where a few rows stand behind many keys there are too few CTAs: the keys then
// are cut into up to kPreMaxSplits ranges of whole steps, at least kPreMinSteps
// each, a CTA for each, and the last one to arrive joins their rows in order.
constexpr int kPreMaxSplits = 16, kPreMinSteps = 3;
// A range's rows in the workspace, for each tile: [HD / 4][row] four values,
// then (maximum, sum) [row].
template <int HD>
__device__ constexpr size_t part_floats() { return (size_t)2 * kPreRows * (HD + 2); }

// One CTA: one kv head, two tiles of 128 / G tokens x the head's G query heads,
// every key up to its last token in steps of 128.
//   warps 0..7   prologue: the tiles' queries (norm, RoPE, f16) to shared
//                memory; then one row per thread: maximum, weights, row sum
//   warps 8..    e4m3 keys and values to f16 (exactly; the pages' scales
//                relative to the step's largest), in the swizzled layout
//   last group   S = Q K^T and O += P V, issued by one thread
// S and P share tensor memory (P is written over S as f16, and is the A operand
// from there), O stays in it; V is read as [key][dim], MN-major, so nothing is
// transposed.  While one tile's softmax runs, the other tile's products do.
// The value scale 2^e goes into the weights, and the running maximum is that of
// score + e: a weight in f16 is held against the largest weight x scale among the
// keys that its row sees.  With a maximum of the scores and another of e, rows lost
// bits to pages without weight, and weights of 2^-33 on values of 2^48 were lost.
// PLANES = 2 (fp32 output): Q and P as f16 pairs hi + lo, twice the products,
// the low ones first.  The tensor cores cut what they add to an accumulator
// off, toward zero; over a thousand steps that grows to 2^-16 of the output.
// So each step's P V starts from zero, and the row's thread adds it up, rounded
// to nearest, in registers (error against 64 bits behind 8,000 tokens: 1.7e-5
// with the sums in tensor memory, 3.0e-7 so).
// PLANES = 1 (bf16 output): Q and P as single f16.  P is rounded by at most 2^-11 of
// each weight, an eighth of the output's own rounding.  Q's rounding moves a score
// by up to 2^-11 of sum |q k|, so that its part grows with the scores: the error
// against 64 bits is 1.02 times that of the output's rounding alone with gains of
// 0.5 to 1.5, 1.06 times with query gains five times as large, 1.29 times with
// twenty.  Pairs would take 1,054 us for 8,000 tokens (as with an fp32 output).
//
// Bound on paper by the products (2,048 clocks a step for both tiles), in fact by
// the softmax threads' way through tensor memory and by issue slots: 4,400 clocks
// a step (issue slots 62 % taken, the tensor pipe 48 % busy).  With the append before it: 8,000 tokens, 32 query
// and 8 kv heads of 128, bf16: 509 us, 1,030 TFLOP/s, 53 % of what a bf16 matrix
// product reaches; 1,024, fp32: 58 us; 16 prompts of about 94 tokens behind 600 to
// 900 cached ones, bf16: 65 us, each CTA's start (12,500 clocks) over a quarter of it.
template <int HD, int PLANES, bool VEC>
__global__ void __launch_bounds__(PreRoles<PLANES>::kThreads, 1)
kv8_prefill_kernel(const __grid_constant__ Kv8Args a, int slots, int parts_off, int o_vec, unsigned inv_g) {
  // grid: slots, kv heads, ranges of keys
  using L = PreLayout<HD, PLANES>;
  using W = PreRoles<PLANES>;
  constexpr int kThreads = W::kThreads;
  constexpr int ST = L::kStages, kBlock = 128 * 128;   // a 64-dim block: 128 rows x 128 bytes
  extern __shared__ __align__(1024) uint8_t raw[];
  uint8_t* sm = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;
  __shared__ __align__(8) uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_half[2], p_full[2], o_full[2];
  __shared__ uint32_t tmem_s;
  __shared__ int nan_s[HD];
  __shared__ int nan_any, last_s, gave_up_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.H / a.Hkv, TT = kPreRows / G;                       // tokens of a tile
  const int g = blockIdx.y, slot = slots - 1 - (int)blockIdx.x;       // long rows first

  // this CTA's sequence: the last b whose slots start at or before ``slot``
  // (sequence b's start at row0[b] / (2 TT) + b)
  __shared__ int seq_s;
  if (warp == 0) {
    int n = 0;
    for (int b = lane; b < a.B; b += 32) {
      prefetch_l1(a.pos + b);                // wanted next
      n += (a.row0[b] / (2 * TT) + b <= slot) ? 1 : 0;
    }
    n = __reduce_add_sync(0xffffffffu, n) - 1;
    if (lane == 0) seq_s = n;
  }
  if (tid == 0) {
    mbar_init(&q_full, kThreads);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 128);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 128);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_half[i], 128);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_full[i], 1);
    }
    fence_mbar_init();
    nan_any = 0;
    gave_up_s = 0;
  }
  for (int i = tid; i < HD; i += kThreads) nan_s[i] = 0x7fffffff;
  __syncthreads();
  const int b = seq_s;
  if (b < 0) {
    pdl_wait();      // as every way out: this grid must not end before the one it follows
    return;
  }
  const int r0 = a.row0[b], rows = min(a.row0[b + 1], a.T) - r0, pos0 = a.pos[b];
  const int t0 = (slot - (r0 / (2 * TT) + b)) * 2 * TT;               // first token of tile 0
  if (r0 < 0 || t0 < 0 || t0 >= rows) {
    pdl_wait();
    return;
  }
  const int nt = t0 + TT < rows ? 2 : 1;                              // tiles with tokens
  if (pos0 < 0 || pos0 > a.max_pos - rows) {                          // left out: zeros
    const int cols = G * HD, n = min(rows - t0, 2 * TT);
    for (int i = tid; i < n * cols; i += kThreads) {
      const size_t at = (size_t)(r0 + t0 + i / cols) * a.o_ld + (size_t)g * cols + i % cols;
      if (a.o) a.o[at] = 0.f;
      else a.o16[at] = __float2bfloat16_rn(0.f);
    }
    pdl_wait();
    return;
  }
  const int keys = pos0 + min(rows, t0 + nt * TT);                    // keys that the last token sees
  const int all_steps = (keys + kPreKeys - 1) / kPreKeys;
  const int ranges = min((int)gridDim.z, max(all_steps / kPreMinSteps, 1));
  const int per = (all_steps + ranges - 1) / ranges, j0 = (int)blockIdx.z * per;   // this range's first step
  const int steps = min(all_steps - j0, per);
  if (steps <= 0) {
    pdl_wait();
    return;
  }
  const int splits = (all_steps + per - 1) / per;                     // ranges with steps
  const int* table = a.table + (size_t)b * a.table_ld;
  if (warp == W::kMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(&tmem_s)), "n"(kPreTmem) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  // queries (the rows that the append before this kernel reads too), four dims
  // and the four that they are rotated with a lane: norm, RoPE, log2(e) / sqrt(HD), and one power of two for the whole
  // launch: a normed row times the gains has no value above sqrt(HD) times the
  // largest gain, which goes to 2^9 .. 2^10 (its typical values then to 2^6: a
  // pair of f16 is good to 2^-22 of a value, and to 2^-34 of the largest)
  float qf;                                 // the power of two back
  {
    constexpr int LPR = HD / 8, TPW = 32 / LPR;                       // lanes of a row, tokens of a warp
    const int l = lane % LPR, d = 4 * l;
    // all rows on their way from memory at once (16 prompts behind cached tokens: 67 -> 66 us)
    for (int q = warp * TPW + lane / LPR; q < 2 * TT; q += kThreads / 32 * TPW)
      if (t0 + q < rows && l % 4 == 0)
#pragma unroll 1
        for (int h = 0; h < G; ++h)
          prefetch_l2(a.qkv + (size_t)(r0 + t0 + q) * a.qkv_ld + (g * G + h) * HD + 8 * l);
    float gain[8];
    load4<VEC>(a.q_gain + d, gain);
    load4<VEC>(a.q_gain + HD / 2 + d, gain + 4);
    float mx = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(gain[e]));
    mx = warp_max(mx) * 1.44269504f;        // log2(e); sqrt(HD) and 1 / sqrt(HD) cancel
    const int ex = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 100);
    qf = pow2f(ex - 9);
    const float up = pow2f(9 - ex);
#pragma unroll
    for (int e = 0; e < 8; ++e) gain[e] *= up * (HD == 128 ? 0.127517431f : 0.180336880f);
    // a token's heads one after the other, two in flight: its RoPE rows once
#pragma unroll 1
    for (int q0 = warp * TPW; q0 < 2 * TT; q0 += kThreads / 32 * TPW) {
      const int q = q0 + lane / LPR, tile = q >= TT ? 1 : 0, i0 = (q - tile * TT) * G;
      const bool live = q < 2 * TT && t0 + q < rows;
      const int tok = live ? t0 + q : t0;
      const float* x0 = a.qkv + (size_t)(r0 + tok) * a.qkv_ld + g * G * HD + d;
      uint8_t* q_hi = sm + L::kQ + tile * PLANES * L::kTile + (l & 1) * 8;
      float co[4], si[4];
      load4<VEC>(a.rope_cos + (size_t)(pos0 + tok) * (HD / 2) + d, co);
      load4<VEC>(a.rope_sin + (size_t)(pos0 + tok) * (HD / 2) + d, si);
#pragma unroll 1
      for (int h = 0; h < G; h += 2) {
        float x[2][8];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          load4<VEC>(x0 + min(h + k, G - 1) * HD, x[k]);
          load4<VEC>(x0 + min(h + k, G - 1) * HD + HD / 2, x[k] + 4);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss += x[k][e] * x[k][e];
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float f = live ? rsqrtf(ss * (1.f / HD) + a.eps) : 0.f;
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[k][e] = live ? x[k][e] * (f * gain[e]) : 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 2 * e % 4;
            const float u = e < 2 ? x[k][i] * co[i] - x[k][i + 4] * si[i] : x[k][i + 4] * co[i] + x[k][i] * si[i];
            const float v = e < 2 ? x[k][i + 1] * co[i + 1] - x[k][i + 5] * si[i + 1]
                                  : x[k][i + 5] * co[i + 1] + x[k][i + 1] * si[i + 1];
            const __half2 y = __floats2half2_rn(u, v);
            const float2 yf = __half22float2(y);
            const __half2 r = __floats2half2_rn(u - yf.x, v - yf.y);
            hi[e] = *reinterpret_cast<const uint32_t*>(&y);
            lo[e] = *reinterpret_cast<const uint32_t*>(&r);
          }
          if (q < 2 * TT && h + k < G) {
            uint8_t* to = q_hi + sw128_offset(i0 + h + k, l / 2);
            uint8_t* to2 = HD == 128 ? to + kBlock : q_hi + sw128_offset(i0 + h + k, 4 + l / 2);
            *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(to2) = make_uint2(hi[2], hi[3]);
            if (PLANES == 2) {
              *reinterpret_cast<uint2*>(to + L::kTile) = make_uint2(lo[0], lo[1]);
              *reinterpret_cast<uint2*>(to2 + L::kTile) = make_uint2(lo[2], lo[3]);
            }
          }
        }
      }
    }
    // rows of no token are zeros: the rows beside them must not depend on what
    // the memory held, not even by when their maximum is taken over
    for (int i = tid; i < (kPreRows - TT * G) * 2 * PLANES * (HD / 8); i += kThreads) {
      const int c = i % (HD / 8), row = TT * G + i / (HD / 8) / (2 * PLANES), at = i / (HD / 8) % (2 * PLANES);
      *reinterpret_cast<uint4*>(sm + L::kQ + at * L::kTile + c / 8 * kBlock + sw128_offset(row, c % 8)) =
          make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async();
    mbar_arrive(&q_full);
  }
  pdl_launch_next();
  pdl_wait();      // the new rows are in their pages

  char4* step_s = reinterpret_cast<char4*>(sm + L::kMeta);              // see goes_by_page
  {
    const int pages = (keys + kKv8Page - 1) / kKv8Page - j0 * kPrePages;   // of this range on
    for (int i0 = warp * 32; i0 < steps * kPrePages; i0 += kThreads) {
      const int i = i0 + lane, page = i < pages ? table[j0 * kPrePages + i] : -1;
      const bool in = page >= 0 && page < a.n_pages;
      int ek = kKv8EMin, hi = kKv8EMin, lo = kKv8EMax;
      if (in) {
        const float* s = a.scale + (size_t)page * 2 * a.Hkv + g;
        ek = kv8_scale_exp(s[0]);
        hi = lo = kv8_scale_exp(s[a.Hkv]);
      }
#pragma unroll
      for (int o = 1; o < kPrePages; o <<= 1) {
        ek = max(ek, __shfl_xor_sync(0xffffffffu, ek, o));
        hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      }
      const unsigned there = __ballot_sync(0xffffffffu, in || i >= pages) >> (lane & 24) & 0xff;
      if ((lane & 7) == 0 && i < steps * kPrePages)
        step_s[i / kPrePages] = make_char4((signed char)ek, (signed char)there, (signed char)hi, (signed char)lo);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_s;
  // A bounded wait.  A role whose wait has run out leaves its loop and arrives at no
  // barrier any more, so that nothing is made of what it did not wait for: the waits
  // for it run out too, up to the rows, which are NaN then.
  auto came = [&](uint64_t& bar, uint32_t parity) { return mbar_wait(&bar, parity, nullptr, a.polls); };

  if (warp >= W::kMma) {
    // ------------------------------------------------ products
    fewer_regs<W::kRegsMma>();
    if (warp == W::kMma && elect_one()) {
      constexpr uint32_t i_qk = idesc_f16(kPreRows, kPreKeys, 0), i_pv = idesc_f16(kPreRows, HD, 1);
      const uint32_t tm = tmem;
      const uint32_t q_d = desc_k(smem_u32(sm + L::kQ)), k_d = desc_k(smem_u32(sm + L::kK));
      const uint32_t v_d = desc_mn(smem_u32(sm + L::kV), kBlock);
      auto qk = [&](int t, int st) {
        const uint32_t qt = q_d + (t * PLANES * L::kTile >> 4), kt = k_d + (st * L::kTile >> 4);
#pragma unroll
        for (int p = PLANES - 1; p >= 0; --p)
#pragma unroll
          for (int ks = 0; ks < HD / 16; ++ks) {
            const uint32_t off = ((ks / 4) * kBlock + (ks % 4) * 32) >> 4;
            umma_ss(tm + t * 128, qt + (p * L::kTile >> 4) + off, kt + off, i_qk, p < PLANES - 1 || ks > 0);
          }
        umma_commit(&s_full[t]);
      };
      // keys 16 k0 .. 16 k1 - 1 of the step
      auto pv = [&](int t, int st, int k0, int k1, uint32_t acc) {
        const uint32_t vt = v_d + (st * L::kTile >> 4);
#pragma unroll
        for (int p = PLANES - 1; p >= 0; --p)
#pragma unroll
          for (int ks = k0; ks < k1; ++ks)
            umma_ts(tm + 256 + t * 128, tm + t * 128 + (PLANES == 1 ? 64 : p * 64) + ks * 8, vt + (ks * 2048 >> 4), i_pv,
                    p < PLANES - 1 || ks > k0 ? 1u : acc);
      };
      int left = nt;                                          // tiles whose last products are to come
      auto products = [&] {
        if (!came(q_full, 0) || !came(k_full[0], 0)) return;
        tc_fence_after();
        for (int t = 0; t < nt; ++t) qk(t, 0);
        umma_commit(&k_empty[0]);
#pragma unroll 1
        for (int j = 0; j < steps; ++j) {
          const int st = j % ST, sn = (j + 1) % ST;
          if (!came(v_full[st], (uint32_t)(j / ST) & 1u)) return;
#pragma unroll 1
          for (int t = 0; t < nt; ++t) {
            if (PLANES == 1) {
              if (!came(p_half[t], (uint32_t)j & 1u)) return;
              tc_fence_after();
              pv(t, st, 4, 8, 1u);
            }
            if (!came(p_full[t], (uint32_t)j & 1u)) return;
            tc_fence_after();
            if (PLANES == 1) pv(t, st, 0, 4, 1u);
            else pv(t, st, 0, 8, 0u);
            if (t == nt - 1) umma_commit(&v_empty[st]);
            if (j + 1 < steps) {
              if (t == 0) {
                if (!came(k_full[sn], (uint32_t)((j + 1) / ST) & 1u)) return;
                tc_fence_after();
              }
              qk(t, sn);
              if (t == nt - 1) umma_commit(&k_empty[sn]);
            } else {
              umma_commit(&o_full[t]);
              --left;
            }
          }
        }
      };
      products();
      if (left > 0) {        // a wait ran out: the rows wait for what was issued, and are told
        *static_cast<volatile int*>(&gave_up_s) = 1;
        __threadfence_block();
        for (int t = nt - left; t < nt; ++t) umma_commit(&o_full[t]);
      }
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ------------------------------------------------ e4m3 to f16
    fewer_regs<W::kRegsWiden>();
    // lane (row = lane / 8 + 4 it, unit = lane % 8) moves 16 bytes of a key's
    // row: 512 bytes in one piece per load (HD 64: lane / 4, 8 rows a load)
    constexpr int U = HD / 16, RP = 32 / U, N = 32 / RP;    // units of a row, rows per load, loads of a warp's 32 keys
    constexpr int KINDS = 3 - W::kWiden;                    // of this warp; kind 0: keys, 1: values
    const int first = KINDS == 1 ? warp / 4 - 2 : 0, w = warp % 4, u = lane % U, rr = lane / U;
    // the second block's lanes swap their stores: no bank twice
    const int odd = u / 4 & 1, c0 = u % 4 * 2 + odd, c1 = u % 4 * 2 + 1 - odd;
    const size_t half = (size_t)a.Hkv * (kKv8Page * HD);    // bytes of a page's keys
    const uint8_t* base = a.kv + first * half + (size_t)g * (kKv8Page * HD) + rr * HD + u * 16;
    const float* scales = a.scale + (size_t)first * a.Hkv + g;
    uint4 x[N];                                             // the step to come
    // this warp's two pages: ids two steps ahead of use, scales one, so that
    // neither is waited for
    int page[2], page_next[2];
    float sc[KINDS][2], sc_next[KINDS][2];
    auto load_ids = [&](int j, int (&p)[2]) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = (j0 + j) * kPrePages + w * 2 + i;
        p[i] = at * kKv8Page < keys ? table[at] : -1;
      }
    };
    auto load_scales = [&](int (&p)[2], float (&f)[KINDS][2]) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (p[i] >= a.n_pages) p[i] = -1;
#pragma unroll
        for (int k = 0; k < KINDS; ++k) f[k][i] = scales[((size_t)max(p[i], 0) * 2 + k) * a.Hkv];
      }
    };
    auto load = [&](int k, int j, const int (&p)[2]) {
      const int left = keys - (j0 + j) * kPreKeys - w * 32 - rr;   // rows of this lane that are keys: it * RP < left
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint8_t* from = base + ((size_t)max(p[i], 0) * 2 + k) * half;
        const int n = p[i] < 0 ? 0 : left;
#pragma unroll
        for (int it = i * (N / 2); it < (i + 1) * (N / 2); ++it) {
          x[it] = make_uint4(0, 0, 0, 0);
          if (it * RP < n) x[it] = *reinterpret_cast<const uint4*>(from + (it * RP % kKv8Page) * HD);
        }
      }
    };
    int e_top = kKv8EMin;
    load_ids(0, page);
    load_ids(1, page_next);
    load_scales(page, sc);
    load(0, 0, page);
#pragma unroll 1
    for (int j = 0; j < steps; ++j) {
      const int st = j % ST;
      int page_2[2];
      const char4 step = step_s[j];
      const bool by_page = goes_by_page(step, e_top);
      load_ids(j + 2, page_2);
      load_scales(page_next, sc_next);
#pragma unroll
      for (int k = 0; k < KINDS; ++k) {
        const int kind = first + k;
        // the two pages' scales over the step's largest one; values whose weights
        // carry the page's scale as they are
        __half2 by[2];
        const int top = kind ? step.z : step.x;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          by[i] = __float2half2_rn(page[i] < 0 ? 0.f
                                   : kind && by_page ? 1.f
                                                     : pow2f(max(kv8_scale_exp(sc[k][i]) - top, -60)));
        if (!came(kind ? v_empty[st] : k_empty[st], ((uint32_t)(j / ST) & 1u) ^ 1u)) goto left_off;
        uint8_t* to = sm + (kind ? L::kV : L::kK) + st * L::kTile + (u / 4) * kBlock;
        if (kind) {
          uint32_t nan = 0;
#pragma unroll
          for (int it = 0; it < N; ++it)
            nan |= has_nan(x[it].x) | has_nan(x[it].y) | has_nan(x[it].z) | has_nan(x[it].w);
          if (nan)
#pragma unroll
            for (int it = 0; it < N; ++it)
              x[it] = without_nan(x[it], nan_s + u * 16, &nan_any, (j0 + j) * kPreKeys + w * 32 + it * RP + rr);
        }
#pragma unroll
        for (int it = 0; it < N; ++it) {
          const int row = w * 32 + it * RP + rr;
          const __half2 f = by[it * RP / kKv8Page];
          const uint4 y = x[it];
          const uint4 one = make_uint4(widen(y.x, f), widen(y.x >> 16, f), widen(y.y, f), widen(y.y >> 16, f));
          const uint4 two = make_uint4(widen(y.z, f), widen(y.z >> 16, f), widen(y.w, f), widen(y.w >> 16, f));
          *reinterpret_cast<uint4*>(to + sw128_offset(row, c0)) = odd ? two : one;
          *reinterpret_cast<uint4*>(to + sw128_offset(row, c1)) = odd ? one : two;
        }
        fence_proxy_async();
        mbar_arrive(kind ? &v_full[st] : &k_full[st]);
        if (k + 1 < KINDS) load(k + 1, j, page);
        else load(0, j + 1, page_next);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        page[i] = page_next[i];
        page_next[i] = page_2[i];
#pragma unroll
        for (int k = 0; k < KINDS; ++k) sc[k][i] = sc_next[k][i];
      }
    }
  left_off:;
  } else {
    // ------------------------------------------------ softmax, a row per thread
    more_regs<W::kRegsSoftmax>();
    if (warp / 4 < nt) {
      const int tile = warp / 4, i = tid % kPreRows, tt = i * inv_g >> 16, t = t0 + tile * TT + tt;
      const bool on = tt < TT && t < rows;
      const int lim = on ? pos0 + t : -1;                    // last key of this row
      const int lim_min = pos0 + t0 + tile * TT;             // of the tile's first row
      const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
      const uint32_t ts = tmem + tile * 128 + lanes, to = tmem + 256 + tile * 128 + lanes;
      // m: the largest score + exponent of its value scale so far, or up to the lag
      // below; l sums 2^(score - m), the output 2^(score + exponent - m + bias) times
      // the e4m3 values
      float m = -INFINITY, l = 0.f;
      int e_top = kKv8EMin;
      float acc[PLANES == 2 ? HD : 1];                       // PLANES 2: the row's output so far
      auto clear_o = [&] {
        const float zero[8] = {};
#pragma unroll 1
        for (int c = 0; c < HD; c += 8) tmem_st8(to + c, zero);
      };
      auto add_step = [&] {                                  // the last step's P V to it
        if constexpr (PLANES == 2) {
#pragma unroll
          for (int c = 0; c < HD; c += 32) {
            uint32_t y[32];
            tmem_ld32_start(to + c, y);
            tmem_ld32_done(y);
#pragma unroll
            for (int e = 0; e < 32; ++e) acc[c + e] += __uint_as_float(y[e]);
          }
        }
      };
      if constexpr (PLANES == 1) clear_o();
      else
#pragma unroll
        for (int c = 0; c < HD; ++c) acc[c] = 0.f;
#pragma unroll 1
      for (int j = 0; j < steps; ++j) {
        const int k0 = (j0 + j) * kPreKeys;
        const char4 step_j = step_s[j];
        const int ev = step_j.z;
        const uint32_t there = (uint8_t)step_j.y;
        const bool by_page = goes_by_page(step_j, e_top);
        const bool masked = k0 + kPreKeys - 1 > lim_min || there != 0xff;
        const float f = qf * pow2f(step_j.x);
        if (!__all_sync(0xffffffffu, came(s_full[tile], (uint32_t)j & 1u))) {
          l = __int_as_float(0x7fffffff);
          break;
        }
        tc_fence_after();
        if (PLANES == 2 && j > 0) add_step();
        if (by_page) {
          if constexpr (PLANES == 2)       // the output so far over to O, free until the products of this step
#pragma unroll
            for (int c = 0; c < HD; c += 8) {
              float y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = acc[c + e];
              tmem_st8(to + c, y);
            }
          const float2 ml = spread_step<HD, PLANES>(to, ts, f, m, l, e_top, lim - k0, there, a,
                                                    table + (j0 + j) * kPrePages, keys - k0, g);
          if constexpr (PLANES == 2)
#pragma unroll
            for (int c = 0; c < HD; c += 8) {
              float y[8];
              tmem_ld8(to + c, y);
#pragma unroll
              for (int e = 0; e < 8; ++e) acc[c + e] = y[e];
            }
          m = ml.x;
          l = ml.y;
          tmem_wait_st();
          tc_fence_before();
          if (PLANES == 1) mbar_arrive(&p_half[tile]);
          mbar_arrive(&p_full[tile]);
          continue;
        }
        // keys of this row: bit e of word c of 32 keys
        uint32_t see[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
        if (masked) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int n = min(max(lim - (k0 + 32 * c) + 1, 0), 32);
            see[c] = n == 32 ? 0xffffffffu : (1u << n) - 1u;
            if (!(there >> (2 * c) & 1)) see[c] &= 0xffff0000u;
            if (!(there >> (2 * c + 1) & 1)) see[c] &= 0xffffu;
          }
        }
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        auto largest = [&](int c, const uint32_t (&s)[32]) {
          if (masked) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              mx4[e & 3] = fmaxf(mx4[e & 3], see[c] >> e & 1 ? __uint_as_float(s[e]) : -INFINITY);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) mx4[e & 3] = fmaxf(mx4[e & 3], __uint_as_float(s[e]));
          }
        };
        uint32_t s0[32], s1[32];               // 32 columns in use, 32 on their way (PLANES 2: no room)
        if constexpr (PLANES == 1) {
          tmem_ld32_start(ts, s0);
          tmem_ld32_done(s0);
          tmem_ld32_start(ts + 32, s1);
          largest(0, s0);
          tmem_ld32_done(s1);
          tmem_ld32_start(ts + 64, s0);
          largest(1, s1);
          tmem_ld32_done(s0);
          tmem_ld32_start(ts + 96, s1);
          largest(2, s0);
          tmem_ld32_done(s1);
          largest(3, s1);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_ld32_start(ts + 32 * c, s0);
            tmem_ld32_done(s0);
            largest(c, s0);
          }
        }
        float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        mx = fmaf(mx, f, (float)ev);
        if (__any_sync(0xffffffffu, mx > m + (float)PreScale<PLANES>::kLag)) {
          const float mn = fmaxf(m, mx);
          const float y = mn == -INFINITY ? 1.f : ex2p(m - mn);
          l *= y;
          if constexpr (PLANES == 2) {
#pragma unroll
            for (int c = 0; c < HD; ++c) acc[c] *= y;
          } else if (j > 0) {  // the products before this step's S are complete
#pragma unroll 1
            for (int c = 0; c < HD; c += 8) {
              float v[8];
              tmem_ld8(to + c, v);
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] *= y;
              tmem_st8(to + c, v);
            }
          }
          m = mn;
        }
        const int up = PreScale<PLANES>::kBias + ev;
        const float sub = (m == -INFINITY ? 0.f : m) - (float)up;
        float sum[4] = {};
        auto step = [&](auto masks) {
          // a weight, by its score and whether the row sees the key
          auto weight = [&](uint32_t r, bool sees) {
            const float p = ex2p(fmaf(__uint_as_float(r), f, -sub));
            return !decltype(masks)::value || sees ? p : 0.f;
          };
          if constexpr (PLANES == 1) {
            // 32 keys at a time into tensor memory as f16: the last 64, whose scores
            // are here still, first, and all over those scores' columns.  The
            // products of that half begin under the other's arithmetic.
            auto weights = [&](int c, const uint32_t (&r)[32]) {
              uint32_t hi[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float x = weight(r[2 * e], see[c] >> (2 * e) & 1);
                const float y = weight(r[2 * e + 1], see[c] >> (2 * e + 1) & 1);
                sum[e & 3] += x + y;
                const __half2 h = __floats2half2_rn(x, y);
                hi[e] = *reinterpret_cast<const uint32_t*>(&h);
              }
              tmem_st16(ts + 64 + 16 * c, hi);
            };
            weights(2, s0);
            tmem_ld32_start(ts, s0);
            weights(3, s1);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&p_half[tile]);
            tmem_ld32_done(s0);
            tmem_ld32_start(ts + 32, s1);
            weights(0, s0);
            tmem_ld32_done(s1);
            weights(1, s1);
          } else {
            // 16 keys at a time; the low parts of the first half are kept back
            // until the scores in their columns are read
            uint32_t lo[4][8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              uint32_t r[16], hi[8], rest[8];
              tmem_ld16(ts + 16 * c, r);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int k = 16 * c + 2 * e;
                const float x = weight(r[2 * e], see[k / 32] >> (k % 32) & 1);
                const float y = weight(r[2 * e + 1], see[k / 32] >> (k % 32 + 1) & 1);
                sum[e & 3] += x + y;
                const __half2 h = __floats2half2_rn(x, y);
                const float2 hf = __half22float2(h);
                const __half2 d = __floats2half2_rn(x - hf.x, y - hf.y);
                hi[e] = *reinterpret_cast<const uint32_t*>(&h);
                rest[e] = *reinterpret_cast<const uint32_t*>(&d);
              }
              tmem_put8(ts + 8 * c, hi);
              if (c < 4) {
#pragma unroll
                for (int e = 0; e < 8; ++e) lo[c][e] = rest[e];
              } else {
                // columns 16 c .. 16 c + 15 are free: two of the eight blocks of low parts
                if (c < 6) {
                  tmem_put8(ts + 16 * c, lo[2 * (c - 4)]);
                  tmem_put8(ts + 16 * c + 8, lo[2 * (c - 4) + 1]);
                } else if (c == 6) {
                  tmem_put8(ts + 96, lo[0]);
                  tmem_put8(ts + 104, lo[1]);
                }
                if (c == 7) {
                  tmem_put8(ts + 112, lo[2]);
                  tmem_put8(ts + 120, rest);
                } else {
#pragma unroll
                  for (int e = 0; e < 8; ++e) lo[c - 4][e] = rest[e];
                }
              }
            }
          }
        };
        if (masked) step(std::true_type());
        else step(std::false_type());
        l += ((sum[0] + sum[1]) + (sum[2] + sum[3])) * pow2f(-up);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[tile]);
      }
      // The products read shared memory and write tensor memory, which are given
      // back behind this wait: it has all its polls, and twice.
      if (!mbar_wait(&o_full[tile], 0, nullptr)) {
        mbar_wait(&o_full[tile], 0, nullptr);
        l = __int_as_float(0x7fffffff);
      }
      if (*static_cast<volatile int*>(&gave_up_s)) l = __int_as_float(0x7fffffff);
      tc_fence_after();
      add_step();
      const bool nans = nan_any != 0;
      // 32 dims of the row as it stands, times f
      auto own = [&](int c, float f, float (&y)[32]) {
        if constexpr (PLANES == 2) {
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = acc[(c + e) % HD];
        } else {
          tmem_ld32(to + c, y);
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          y[e] *= f;
          if (nans && nan_s[c + e] <= lim) y[e] = __int_as_float(0x7fffffff);
        }
      };
      float inv = l == 0.f ? 0.f : pow2f(-PreScale<PLANES>::kBias) / l;
      float weight[kPreMaxSplits];                            // of each range
      const float4* parts = nullptr;
      bool mine = true;
      if (splits > 1) {
        const size_t cta = (size_t)blockIdx.y * gridDim.x + blockIdx.x;
        unsigned* ticket = reinterpret_cast<unsigned*>(a.ws) + cta;
        float* part0 =
            reinterpret_cast<float*>(static_cast<char*>(a.ws) + parts_off) + cta * gridDim.z * part_floats<HD>();
        float* part = part0 + blockIdx.z * part_floats<HD>() + tile * (part_floats<HD>() / 2);
#pragma unroll
        for (int c = 0; c < HD; c += 32) {
          float y[32];
          own(c, pow2f(-PreScale<PLANES>::kBias), y);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            reinterpret_cast<float4*>(part)[(c / 4 + q) * kPreRows + i] =
                make_float4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
        }
        reinterpret_cast<float2*>(part + HD * kPreRows)[i] = make_float2(m, l);
        __threadfence();
        softmax_sync(nt * kPreRows);
        if (tid == 0) {
          const unsigned got = atomicAdd(ticket, 1u);
          last_s = got == (unsigned)(splits - 1);
          if (last_s) {
            __threadfence();
            *ticket = 0u;
          }
        }
        softmax_sync(nt * kPreRows);
        mine = last_s;
        if (mine) {
          __threadfence();
          const float* ml = part0 + tile * (part_floats<HD>() / 2) + HD * kPreRows;
          float top = -INFINITY, sum = 0.f;
#pragma unroll
          for (int z = 0; z < kPreMaxSplits; ++z)
            if (z < splits) top = fmaxf(top, __ldcg(reinterpret_cast<const float2*>(ml + z * part_floats<HD>()) + i).x);
#pragma unroll
          for (int z = 0; z < kPreMaxSplits; ++z) {
            weight[z] = 0.f;
            if (z < splits) {
              const float2 v = __ldcg(reinterpret_cast<const float2*>(ml + z * part_floats<HD>()) + i);
              weight[z] = v.x == -INFINITY ? (v.y == v.y ? 0.f : v.y) : ex2p(v.x - top);   // no keys; NaN stays
              sum += v.y * weight[z];
            }
          }
          inv = sum == 0.f ? 0.f : 1.f / sum;
          parts = reinterpret_cast<const float4*>(part0 + tile * (part_floats<HD>() / 2));
        }
      }
      if (mine) {
        // rows by threads to rows by warps, over the tile's queries, which nothing
        // reads any more: 16-byte units XORed with the row against bank conflicts
        using T = typename OutOf<PLANES>::type;
        constexpr int UE = 16 / sizeof(T), UR = HD / UE;        // values of a unit, units of a row
        uint8_t* rows_s = sm + L::kQ + tile * PLANES * L::kTile + (size_t)(i & ~31) * HD * sizeof(T);
#pragma unroll (PLANES == 2 ? 4 : 1)
        for (int c = 0; c < HD; c += 32) {
          float y[32];
          if (!parts) {
            own(c, inv, y);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = 0.f;
#pragma unroll
            for (int z = 0; z < kPreMaxSplits; ++z)
              if (z < splits)
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                  const float4 v = __ldcg(parts + z * (part_floats<HD>() / 4) + (c / 4 + q) * kPreRows + i);
                  y[4 * q] += v.x * weight[z];
                  y[4 * q + 1] += v.y * weight[z];
                  y[4 * q + 2] += v.z * weight[z];
                  y[4 * q + 3] += v.w * weight[z];
                }
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] *= inv;
          }
#pragma unroll
          for (int q = 0; q < 32 / UE; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (UE == 4) {
                w[e] = __float_as_uint(y[(4 * q + e) % 32]);
              } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(y[(8 * q + 2 * e) % 32], y[(8 * q + 2 * e + 1) % 32]);
                w[e] = *reinterpret_cast<const uint32_t*>(&h);
              }
            *reinterpret_cast<uint4*>(rows_s + (size_t)lane * HD * sizeof(T) + (((c / UE + q) ^ lane) % UR) * 16) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        __syncwarp();
        T* out = reinterpret_cast<T*>(PLANES == 2 ? static_cast<void*>(a.o) : static_cast<void*>(a.o16));
#pragma unroll 4
        for (int k = 0; k < UR; ++k) {                          // 32 units a step: 32 / UR rows
          const int row = (k * 32 + lane) / UR, q = lane % UR, ri = (i & ~31) + row, rt = ri * inv_g >> 16;
          const uint4 y = *reinterpret_cast<const uint4*>(rows_s + (size_t)row * HD * sizeof(T) + ((q ^ row) % UR) * 16);
          if (rt < TT && t0 + tile * TT + rt < rows) {
            T* p = out + (size_t)(r0 + t0 + tile * TT + rt) * a.o_ld + (size_t)(g * G + ri - rt * G) * HD + q * UE;
            if (o_vec) {
              *reinterpret_cast<uint4*>(p) = y;
            } else {
              const T* v = reinterpret_cast<const T*>(&y);
#pragma unroll
              for (int e = 0; e < UE; ++e) p[e] = v[e];
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W::kMma) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "n"(kPreTmem) : "memory");
  }
}

int pre_slots(int T, int B, int H, int Hkv) { return T / (2 * (kPreRows / (H / Hkv))) + B; }
// Ranges of keys: as many as one wave of CTAs holds.
int pre_splits(int slots, int Hkv) {
  const long long ctas = (long long)slots * Hkv;
  const int n = (int)(kv8_sms() / ctas);
  return n < 1 ? 1 : n > kPreMaxSplits ? kPreMaxSplits : n;
}

static_assert(1024 + PreLayout<128, 2>::kMeta + kPreStepBytes * (kKv8MaxPrompt / kPreKeys) <= kPreSmem - 2048 &&
                  1024 + PreLayout<128, 1>::kMeta + kPreStepBytes * (kKv8MaxPrompt / kPreKeys) <= kPreSmem - 2048,
              "the longest prompt's steps");

template <int HD, int PLANES, bool VEC>
cudaError_t launch(const Kv8Args& a, cudaStream_t st) {
  auto k = kv8_prefill_kernel<HD, PLANES, VEC>;
  static bool attr = false;
  if (!attr) {
    // all but what is static
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kPreSmem - 2048);
    if (e != cudaSuccess) return e;
    attr = true;
  }
  const int slots = pre_slots(a.T, a.B, a.H, a.Hkv);
  const uintptr_t o = reinterpret_cast<uintptr_t>(a.o) | reinterpret_cast<uintptr_t>(a.o16);
  const int o_vec = (o & 15) == 0 && a.o_ld % (PLANES == 2 ? 4 : 8) == 0;
  cudaLaunchConfig_t cfg = {};
  const int most = (a.max_pos + kPreKeys - 1) / kPreKeys / kPreMinSteps;     // ranges that the table has room for
  cfg.gridDim = dim3(slots, a.Hkv, std::max(1, std::min(pre_splits(slots, a.Hkv), most)));
  cfg.blockDim = dim3(PreRoles<PLANES>::kThreads);
  cfg.dynamicSmemBytes =
      1024 + PreLayout<HD, PLANES>::kMeta + kPreStepBytes * ((a.max_pos + kPreKeys - 1) / kPreKeys);
  cfg.stream = st;
  // runs its queries' part while the append before it ends
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const unsigned inv_g = 65536u / (a.H / a.Hkv) + 1;      // i / G = i * inv_g >> 16, i < 128
  return s2_launch(&cfg, k, a, slots, (int)kv8_ticket_bytes(kv8_sms()), o_vec, inv_g);
}
template <int HD, int PLANES>
cudaError_t launch(const Kv8Args& a, cudaStream_t st) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.qkv) | reinterpret_cast<uintptr_t>(a.q_gain) |
                       reinterpret_cast<uintptr_t>(a.rope_cos) | reinterpret_cast<uintptr_t>(a.rope_sin);
  return (at & 15) == 0 && a.qkv_ld % 4 == 0 ? launch<HD, PLANES, true>(a, st) : launch<HD, PLANES, false>(a, st);
}

}  // namespace

size_t kv8_prefill_ws_bytes(int hd) {   // the ranges of all slots and heads are one wave, an SM each
  const int sms = kv8_sms();
  return kv8_ticket_bytes(sms) + (size_t)sms * 2 * kPreRows * (hd + 2) * 4;
}

cudaError_t launch_kv8_prefill(const Kv8Args& a, cudaStream_t st) {
  if (a.hd == 128) return a.o ? launch<128, 2>(a, st) : launch<128, 1>(a, st);
  return a.o ? launch<64, 2>(a, st) : launch<64, 1>(a, st);
}

}  // namespace s2
