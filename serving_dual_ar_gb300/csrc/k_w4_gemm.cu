// Products of rows with 4-bit weights (mx_common.cuh) on the tensor cores:
//   Y[t, n] (op)= sum_k X[t, k] W[n, k].
//
// The weights are the M = 128 operand (e2m1), the rows the N = TN operand
// (e4m3), both K-major; tcgen05.mma kind::mxf8f6f4 multiplies them with their
// scales as they are held.  So no weight passes through a register: the TMA
// engine spreads a tile's 8 KB of codes to the 16 KB that the MMA reads, and
// scale tiles go from shared to tensor memory in the order that they have in
// memory.  A tile of 128 weights' k costs 8.7 KB of the memory stream and 4 MMAs
// of 32 k, so few rows are bound by memory and many by the tensor cores.
//
// Sums: the tensor core cuts what it adds below the last bit of its fp32 sum,
// which leans towards zero by about 2^-24 of the sum so far with each step of 32 k.
// So seven tiles (896 k) at most are summed there; these partial sums are added up
// in registers, rounded to nearest (two accumulators take turns).  Where CTAs stay
// and the output is bf16, up to 16,384 k (kWholeSum).
//
// One thread issues all copies and one all MMAs of a CTA: elected lanes (a branch
// by lane number moves each operand to a uniform register in a loop over lanes:
// 1,024 rows times 19,456 x 2,560 took 141 us, 91 with them) and stages by number
// (77), then CTAs that stay (39).
//
// Few rows do not have tiles for every SM: then K is cut into up to eight parts
// which form a thread-block cluster and add their sums in the order of the
// parts through distributed shared memory.  Clusters that wait for one another
// must not also wait for tensor memory that the other holds: each CTA of a cluster
// takes more than half of an SM's shared memory, so no two of them meet on one.
#include "kept_count.h"
#include "mx_common.cuh"
#include "tc_common.cuh"
#include "tma_map.h"

namespace s2 {

namespace {

// Warp 0: copies, warp 1: MMAs, then groups of four for sums and output, up to
// 64 columns each.
constexpr int w4_groups(int tn) { return (tn + 63) / 64; }
constexpr int w4_threads(int tn) { return (2 + 4 * w4_groups(tn)) * 32; }

struct W4Params {
  int N, T, K, KT, n_tiles, tiles, chunk, mode, y_bf16;
  const void* x;         // plain rows
  long long ldx;
  int x_vec;
  long long ldy;
  const uint8_t* codes;
  const uint8_t* w_scale;
  const uint8_t* x_scale;
  void* y;
  unsigned polls;
};

// A wait that ends when another one of the CTA gave up.
S2_DEV bool w4_wait(uint64_t* bar, uint32_t parity, unsigned polls, volatile int* fail) {
  for (unsigned i = 0; i < polls; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*fail) return false;
  }
  *fail = 1;
  return false;
}
// The same for a whole warp, with one outcome: what follows it (loads of tensor
// memory, shuffles) needs every lane, and lanes count their polls each for itself.
S2_DEV bool w4_wait_warp(uint64_t* bar, uint32_t parity, unsigned polls, volatile int* fail) {
  return __all_sync(0xffffffffu, w4_wait(bar, parity, polls, fail));
}

// 16 columns of this thread's tensor-memory lane, there after the next wait.
S2_DEV void tmem_issue16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
template <int N>
S2_DEV void tmem_ld_row(uint32_t taddr, float (&v)[N]) {   // N columns, one wait
  uint32_t r[N];
#pragma unroll
  for (int i = 0; i < N; i += 16) tmem_issue16(taddr + i, r + i);
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) {
    asm volatile("" : "+r"(r[i]));      // read behind the wait
    v[i] = __uint_as_float(r[i]);
  }
}

// A box of a tensor map, or a scale tile, to shared memory.
S2_DEV void w4_load_2d(uint32_t dst, uint64_t map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
S2_DEV void w4_load(uint32_t dst, const void* src, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(dst), "l"(src), "r"(kMxTile), "r"(bar) : "memory");
}

// Towards L2 alone; both a multiple of 16.
S2_DEV void w4_prefetch(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" :: "l"(src), "r"(bytes) : "memory");
}

constexpr int w4_stage_bytes(int tn) { return 128 * 128 + tn * 128 + (tn > 128 ? 2048 : 1024); }
constexpr int w4_tmem_cols(int need) {
  return need <= 32 ? 32 : need <= 64 ? 64 : need <= 128 ? 128 : need <= 256 ? 256 : 512;
}

S2_DEV float w4_inverse(float x) {      // to one unit, subnormal results included
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Where a warp's outputs go: feature n (32 of them) of consecutive rows.
template <int MODE, typename TY>
struct W4Out {
  TY* at;
  long long ldy;
  bool live;
  S2_DEV W4Out(const W4Params& p, int t, int n)
      : at(static_cast<TY*>(p.y) + t * p.ldy + (MODE == W4_SWIGLU ? n >> 1 : n)), ldy(p.ldy), live(n < p.N) {
    // gate and up lie in an even lane and the odd one beside it: the odd one
    // takes the second of two rows
    if (MODE == W4_SWIGLU && (n & 1)) at += p.ldy;
  }
  // What row's output is added to; asked for ahead of put, since a load behind
  // a store waits for it.
  S2_DEV float get(int row, bool there) const {
    return MODE == W4_ADD && live && there ? to_f(at[row * ldy]) : 0.f;
  }
  // SwiGLU of two rows: this lane's one of them.
  S2_DEV static float silu_mul(float v0, float v1) {
    const bool odd = threadIdx.x & 1;
    const float got = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
    const float g = odd ? got : v0, u = odd ? v1 : got;
    return g * w4_inverse(1.f + expf(-g)) * u;
  }
  S2_DEV void put_silu(int row, int n, float v) const {
    if (live && n > (int)(threadIdx.x & 1)) at[row * ldy] = from_f<TY>(v);
  }
  // Rows row and row + 1, n of them (none where n <= 0).
  S2_DEV void put(int row, int n, float v0, float v1, float before0, float before1) const {
    if (MODE == W4_SWIGLU) {
      put_silu(row, n, silu_mul(v0, v1));
    } else {
      if (live && n > 0) at[row * ldy] = from_f<TY>(MODE == W4_ADD ? before0 + v0 : v0);
      if (live && n > 1) at[(row + 1) * ldy] = from_f<TY>(MODE == W4_ADD ? before1 + v1 : v1);
    }
  }
  static constexpr bool kSilu = MODE == W4_SWIGLU;
};
template <typename F>
S2_DEV void w4_with_out(const W4Params& p, int t, int n, F f) {
  switch (p.mode * 2 + p.y_bf16) {
    case 0: f(W4Out<W4_STORE, float>(p, t, n)); break;
    case 1: f(W4Out<W4_STORE, __nv_bfloat16>(p, t, n)); break;
    case 2: f(W4Out<W4_ADD, float>(p, t, n)); break;
    case 3: f(W4Out<W4_ADD, __nv_bfloat16>(p, t, n)); break;
    case 4: f(W4Out<W4_SWIGLU, float>(p, t, n)); break;
    default: f(W4Out<W4_SWIGLU, __nv_bfloat16>(p, t, n)); break;
  }
}

// ``rows`` of a group's GB rows, 16 at a time: what they are added to is asked for
// together, and SwiGLU of all of them comes before the first store, or each would
// wait for its own (32 rows times 19,456 x 2,560 8.8 -> 8.2 us).
template <int GB, int N, typename OUT>
S2_DEV void w4_put_rows(const OUT& out, const float (&v)[N], int rows) {
  constexpr int Q = 16;
#pragma unroll
  for (int b = 0; b < GB; b += Q) {
    if constexpr (OUT::kSilu) {
      float r[Q / 2];
#pragma unroll
      for (int j = 0; j < Q; j += 2)
        if (b + j < GB) r[j / 2] = OUT::silu_mul(v[b + j], v[b + j + 1 < GB ? b + j + 1 : b + j]);
#pragma unroll
      for (int j = 0; j < Q; j += 2)
        if (b + j < GB) out.put_silu(b + j, rows - b - j, r[j / 2]);
    } else {
      float before[Q];
#pragma unroll
      for (int j = 0; j < Q; ++j) before[j] = b + j < GB ? out.get(b + j, b + j < rows) : 0.f;
#pragma unroll
      for (int j = 0; j < Q; j += 2)
        if (b + j < GB)
          out.put(b + j, rows - b - j, v[b + j], v[b + j + 1 < GB ? b + j + 1 : b + j], before[j], before[j + 1]);
    }
  }
}

// Four values into another CTA of the cluster, counted by its barrier; both
// addresses are this CTA's own of the same places.
S2_DEV void st_async4(uint32_t at, float x, float y, float z, float w, uint32_t bar, uint32_t rank) {
  asm volatile(
      "{\n\t.reg .b32 a, m;\n\tmapa.shared::cluster.u32 a, %0, %6;\n\tmapa.shared::cluster.u32 m, %5, %6;\n\t"
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [a], {%1, %2, %3, %4}, [m];\n\t}"
      :: "r"(at), "f"(x), "f"(y), "f"(z), "f"(w), "r"(bar), "r"(rank) : "memory");
}

// ---------------------------------------------------------------- plain rows as 8-bit parts

// A row of fp32 (bf16) values as P = 6 (3) rows of e4m3 values whose scales
// fall by 2^4 from one to the next: each takes four bits or more of what the
// ones before it left, exactly.  What remains is 2^-10 of the last row's scale at
// most, 2^-37 (2^-25) of the group's largest magnitude, and nothing of values
// within 2^13 (2^17) of that; no scale is below 2^-126, so 2^-136 may remain of any
// value.  NaN stays NaN, and e4m3 has nothing else for an infinity.
constexpr int kParts32 = 6, kParts16 = 3;
// Up to this many rows' parts are made by the CTAs that multiply them.  With 6,144
// x 2,560 weights 1, 2, 3 and 4 fp32 rows take 5.7, 6.4, 8.1 and 9.2 us that way, and
// 6.7 us with a kernel ahead that leaves them in memory; bf16 rows 5.5, 5.7, 6.7 and
// 7.3 against 6.2 to 6.3.  The border is the same at 2,560 x 4,096, 2,560 x 9,728,
// 19,456 x 2,560 and 40,000 x 1,024 (two rows 3 to 14 % faster in the CTAs, three 3 to
// 29 % slower, but for bf16 rows with the smallest of them, 5.2 for 5.5).
constexpr int kPlainRows = 2;

// Four values of a lane, 128 of a warp, as they lie in memory (vec: on 16 bytes;
// zeros from K on), and as floats.
template <typename T> struct Raw4;
template <> struct Raw4<float> {
  float4 q;
  S2_DEV void load(const float* row, int k0, int K, bool vec) {
    if (vec && k0 + 4 <= K)
      q = *reinterpret_cast<const float4*>(row + k0);
    else
      q = make_float4(k0 < K ? row[k0] : 0.f, k0 + 1 < K ? row[k0 + 1] : 0.f, k0 + 2 < K ? row[k0 + 2] : 0.f,
                      k0 + 3 < K ? row[k0 + 3] : 0.f);
  }
  S2_DEV void get(float (&v)[4]) const { v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w; }
};
template <> struct Raw4<__nv_bfloat16> {
  uint2 q;
  S2_DEV void load(const __nv_bfloat16* row, int k0, int K, bool vec) {
    const uint16_t* r = reinterpret_cast<const uint16_t*>(row) + k0;
    if (vec && k0 + 4 <= K)
      q = *reinterpret_cast<const uint2*>(r);
    else
      q = make_uint2((k0 < K ? r[0] : 0u) | (k0 + 1 < K ? (uint32_t)r[1] << 16 : 0u),
                     (k0 + 2 < K ? r[2] : 0u) | (k0 + 3 < K ? (uint32_t)r[3] << 16 : 0u));
  }
  S2_DEV void get(float (&v)[4]) const {
    v[0] = bf16lo(q.x), v[1] = bf16hi(q.x), v[2] = bf16lo(q.y), v[3] = bf16hi(q.y);
  }
};
// put(p, codes, scales): part p's four bytes of each lane, and the bytes of its
// four groups' scales as one word.
template <int P, typename F>
S2_DEV void parts_of(float (&v)[4], int lane, F put) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (!(fabsf(v[i]) <= 3.402823466e38f)) v[i] = __uint_as_float(0x7fffffffu);
    m = fmaxf(m, fabsf(v[i]));
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int e = mx8_exponent(m);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int ep = max(e - 4 * p, kMxEMin);
    const float f = mx_pow2(-ep), g = mx_pow2(ep);
    float q[4] = {v[0] * f, v[1] * f, v[2] * f, v[3] * f};
    if (p == 0 && e == kMxEMax) {      // the next code, 256 * 2^120, would be infinite as a sum of fp32
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = fabsf(q[i]) > 240.f ? copysignf(240.f, q[i]) : q[i];
    }
    const uint32_t c = mx_e4m3x2(q[0], q[1]) | (mx_e4m3x2(q[2], q[3]) << 16);
    if (p < P - 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = fabsf(v[i]) <= 3.402823466e38f ? fmaf(-mx_e4m3(c >> (8 * i)), g, v[i]) : 0.f;
    }
    uint32_t w = (uint32_t)(ep + 127) << (lane / 8 * 8);
    w |= __shfl_xor_sync(0xffffffffu, w, 8);
    w |= __shfl_xor_sync(0xffffffffu, w, 16);
    put(p, c, w);
  }
}

// ---------------------------------------------------------------- few rows

// One tile of 128 weights and TN rows a CTA, or one part of K of it.  A k-tile of
// the stream is 8.7 KB of weights; ten stages of 16 rows keep 87 KB an SM under way,
// which 6 TB/s need (1 row times 19,456 x 20,480: 36.2 us, 5.9 TB/s; five stages 41.9).
// Under the kernel ahead the first stages' weights are brought to L2 (4 bf16 rows
// times 2,560 x 9,728 7.4 us; without that 8.0); to shared memory they come behind
// it, as the rows do: it, or one before it, may have written them, and only its end
// makes that visible.
// P: rows of the operand per row of X (parts of its values, added up).  TX: the
// type of plain rows whose parts four warps of the CTA make, each every fourth
// k-tile's; uint8_t: rows of 8 bits in memory.
template <int TN, int STAGES, int P, bool CL, typename TX>
__global__ void __launch_bounds__(w4_threads(TN) + (sizeof(TX) > 1 ? 128 : 0))
w4_tc_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const W4Params p) {
  constexpr int STAGE = w4_stage_bytes(TN), B_AT = 128 * 128, SF_AT = B_AT + TN * 128;
  constexpr int CH = STAGES >= 8 ? STAGES / 2 : STAGES;   // k-tiles summed in tensor memory
  constexpr int SF_COLS = 2 * TN, TM_COLS = w4_tmem_cols(2 * TN + STAGES * 8);
  constexpr bool PLAIN = sizeof(TX) > 1;
  constexpr int OUT_WARPS = 2 + 4 * w4_groups(TN);      // behind them those that make parts
  constexpr int GN = TN / w4_groups(TN); // columns of a group of warps
  constexpr int GB = GN / P;             // rows of X in them
  static_assert(P == 1 || GN == TN, "parts of a row lie in one group");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  __shared__ __align__(8) uint64_t full[STAGES], made[STAGES], empty[STAGES], acc_full[2], acc_empty[2], drained, joined;
  __shared__ uint32_t tmem_base;
  __shared__ int s_fail;
  volatile int* fail = &s_fail;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_tile = blockIdx.x % p.n_tiles, n0 = n_tile * 128, t0 = blockIdx.x / p.n_tiles * TN;
  const int S = CL ? (int)gridDim.z : 1, split = CL ? (int)blockIdx.z : 0;
  const int kt0 = (int)((long long)split * p.KT / S);
  const int nk = (int)((long long)(split + 1) * p.KT / S) - kt0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      if (PLAIN) mbar_init(&made[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4 * w4_groups(TN));
    }
    mbar_init(&drained, 1);
    mbar_init(&joined, 1);
    s_fail = 0;
    fence_mbar_init();
    asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(&map_w)) : "memory");
    if (!PLAIN) asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(&map_x)) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(&tmem_base)), "r"(TM_COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  // Behind the allocation: CTAs of the next kernel may now take what is left.  Of the
  // kernel ahead, CTAs may still have to allocate; where one fits an SM's shared memory
  // together with this kernel's, the two ask for 288 of the 512 columns at most.
  pdl_launch_next();
  if (CL) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

  float acc[GN];
  if (warp == 0) {
    if (elect_one()) {
      const uint64_t mw = reinterpret_cast<uint64_t>(&map_w), mx = reinterpret_cast<uint64_t>(&map_x);
      const uint8_t* ws = p.w_scale + ((size_t)n_tile * p.KT + kt0) * kMxTile;
      const uint8_t* xs = p.x_scale + ((size_t)(t0 >> 7) * p.KT + kt0) * kMxTile;
      const uint32_t sm = smem_u32(smem);
      int k = kt0 * 128, left = nk;
      pdl_wait();     // nothing is read ahead of it
      bool ok = true;
      for (int r = 0; left > 0 && ok; ++r) {
#pragma unroll
        for (int i = 0; i < STAGES; ++i) {
          if (left <= 0 || (r > 0 && !(ok = w4_wait(&empty[i], (r + 1) & 1, p.polls, fail)))) break;
          // codes count as they lie in memory
          mbar_arrive_expect_tx(&full[i], 128 * 64 + kMxTile + (PLAIN ? 0 : TN * 128 + kMxTile));
          w4_load_2d(sm + i * STAGE, mw, k, n0, smem_u32(&full[i]));
          w4_load(sm + i * STAGE + SF_AT, ws, smem_u32(&full[i]));
          if (!PLAIN) {
            w4_load_2d(sm + i * STAGE + B_AT, mx, k, t0, smem_u32(&full[i]));
            w4_load(sm + i * STAGE + SF_AT + kMxTile, xs, smem_u32(&full[i]));
          }
          ws += kMxTile;
          xs += kMxTile;
          k += 128;
          --left;
        }
      }
      // behind a wait that gave up, copies may still be under way
      mbar_wait(&drained, 0, nullptr);
      for (int s = *fail ? max(nk - left - STAGES, 0) : nk; s < nk - left; ++s)
        mbar_wait(&full[s % STAGES], (s / STAGES) & 1, nullptr);
    }
  } else if (warp == 1) {
    pdl_wait();     // polls count from here on, however long the kernel ahead takes
    if (elect_one()) {
      const uint32_t st0 = desc_lo(smem_u32(smem)), sf0 = tmem + SF_COLS;
      const uint32_t sfb = 4 + ((t0 & 127) >> 5);      // a tile of 64 rows: the scale tile's first or second half
      int left = nk;
      bool ok = true;
      for (int r = 0; left > 0 && ok; ++r) {
#pragma unroll
        for (int i = 0; i < STAGES; ++i) {
          if (left <= 0) break;
          const int c = r * (STAGES / CH) + i / CH, buf = c & 1;
          if (i % CH == 0 && c >= 2 && !(ok = w4_wait(&acc_empty[buf], ((c >> 1) + 1) & 1, p.polls, fail))) break;
          if (!(ok = w4_wait(&full[i], r & 1, p.polls, fail))) break;
          if (PLAIN && !(ok = w4_wait(&made[i], r & 1, p.polls, fail))) break;
          tc_fence_after();
          const uint32_t st = st0 + (i * STAGE >> 4), sf = sf0 + i * 8;
          tmem_cp_scales(sf, st + (SF_AT >> 4));
          tmem_cp_scales(sf + 4, st + ((SF_AT + kMxTile) >> 4));
#pragma unroll
          for (int j = 0; j < 4; ++j)
            umma_mxf8f6f4(tmem + buf * TN, st + 2 * j, st + (B_AT >> 4) + 2 * j, idesc_e2m1_e4m3(128, TN, j), sf,
                          sf + sfb, i % CH + j > 0);
          umma_commit(&empty[i]);
          if (--left == 0 || i % CH == CH - 1) umma_commit(&acc_full[buf]);
        }
      }
      umma_commit(&drained);
    }
  } else if (PLAIN && warp >= OUT_WARPS) {
    if constexpr (PLAIN) {
      pdl_wait();
      constexpr int B = kPlainRows;
      // every row's values are asked for at once, and a tile ahead
      Raw4<TX> raw[B];
      auto load = [&](int s) {
#pragma unroll
        for (int b = 0; b < B; ++b)
          raw[b].load(static_cast<const TX*>(p.x) + min(b, p.T - 1) * p.ldx, (kt0 + s) * 128 + lane * 4, p.K, p.x_vec);
      };
      if (warp - OUT_WARPS < nk) load(warp - OUT_WARPS);
      for (int s = warp - OUT_WARPS; s < nk; s += 4) {
        const int slot = s % STAGES;
        float v[B][4];
#pragma unroll
        for (int b = 0; b < B; ++b) raw[b].get(v[b]);
        if (s + 4 < nk) load(s + 4);
        if (s >= STAGES && !w4_wait_warp(&empty[slot], (s / STAGES + 1) & 1, p.polls, fail)) break;
        uint8_t* rows8 = smem + slot * STAGE + B_AT;
#pragma unroll
        for (int b = 0; b < B; ++b)
          if (b < p.T)
            parts_of<P>(v[b], lane, [&](int i, uint32_t c, uint32_t w) {
              const int row = b * P + i;
              *reinterpret_cast<uint32_t*>(rows8 + sw128_offset(row, lane >> 2) + (lane & 3) * 4) = c;
              if (lane == 0) *reinterpret_cast<uint32_t*>(rows8 + TN * 128 + kMxTile + mx_scale_at(row, 0, 1)) = w;
            });
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&made[slot]);
      }
    }
  } else {
    // the first stages' weights towards L2, a row a thread of the first group
    const int first = min(nk, STAGES), row = (int)threadIdx.x - 64;
    if (row < 128 && n0 + row < p.N) w4_prefetch(p.codes + ((size_t)(n0 + row) * p.KT + kt0) * 64, first * 64);
    if (row == 0) w4_prefetch(p.w_scale + ((size_t)n_tile * p.KT + kt0) * kMxTile, first * kMxTile);
    pdl_wait();     // outputs and what they are added to
    const uint32_t from = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (warp - 2) / 4 * GN;
    const int chunks = (nk + CH - 1) / CH;
    for (int c = 0; c < chunks; ++c) {
      const int buf = c & 1;
      if (!w4_wait_warp(&acc_full[buf], (c >> 1) & 1, p.polls, fail)) break;
      tc_fence_after();
      if (c == 0) {
        tmem_ld_row<GN>(from, acc);
      } else {
        float v[GN];
        tmem_ld_row<GN>(from + buf * TN, v);
#pragma unroll
        for (int i = 0; i < GN; ++i) acc[i] += v[i];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[buf]);
    }
  }
  __syncwarp();
  // shared and tensor memory are used again and given back when products and
  // copies are done, behind a wait that gave up, too
  mbar_wait(&drained, 0, nullptr);
  __syncthreads();

  // this group's rows of X: b0 .. b0 + GB - 1 of the tile
  const bool writes = warp >= 2 && warp < OUT_WARPS;
  const int b0 = writes ? (warp - 2) / 4 * GB : 0;
  const int rows = min(GB, p.T - t0 - b0), f = (warp & 3) * 32 + lane, n = n0 + f;
  if (writes) {
#pragma unroll
    for (int b = 0; b < GB; ++b) {       // into the first GB, behind those still to be read
      float v = acc[b * P + P - 1];
#pragma unroll
      for (int i = P - 2; i >= 0; --i) v += acc[b * P + i];
      acc[b] = v;
    }
    if (*fail) {
#pragma unroll
      for (int b = 0; b < GB; ++b) acc[b] = __uint_as_float(0x7fffffffu);
    }
  }
  if (CL) {
    // Four rows of the tile (quad q) are joined by part q % S: every part stores
    // its sums straight into that one's shared memory, whose barrier counts the
    // bytes.
    constexpr int JOIN_AT = STAGES * STAGE;
    const int quads = (min(TN / P, p.T - t0) + 3) / 4, mine = split < quads ? (quads - split + S - 1) / S : 0;
    if (threadIdx.x == 0) mbar_arrive_expect_tx(&joined, mine * S * 2048);
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (writes) {
      const uint32_t slot = smem_u32(smem + JOIN_AT) + f * 16, bar = smem_u32(&joined);
      int to = b0 / 4 % S, at = b0 / 4 / S * S + split;
#pragma unroll
      for (int b = 0; b < GB; b += 4) {
        if (b < rows)
          st_async4(slot + at * 2048, acc[b], b + 1 < GB ? acc[b + 1] : 0.f, b + 2 < GB ? acc[b + 2] : 0.f,
                    b + 3 < GB ? acc[b + 3] : 0.f, bar, to);
        if (++to == S) {
          to = 0;
          at += S;
        }
      }
      w4_with_out(p, t0, n, [&](auto out) {
        constexpr int Q = 3;      // quads whose rows are asked for at once
        const int live = min(TN / P, p.T - t0);
        bool came = false;
        for (int i0 = (warp - 2) / 4; i0 < mine; i0 += Q * w4_groups(TN)) {
          float before[Q][4];
#pragma unroll
          for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int b = (split + (i0 + q * w4_groups(TN)) * S) * 4 + j;
              before[q][j] = out.get(b, b < live);
            }
          // far longer than a part may take to give up: none stores to a CTA that is gone
          came = came || mbar_wait(&joined, 0, nullptr, 32000000u);
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            const int i = i0 + q * w4_groups(TN), b = (split + i * S) * 4;
            if (i >= mine) break;
            const float4* from = reinterpret_cast<const float4*>(smem + JOIN_AT) + i * S * 128 + f;
            float4 v = from[0];
            for (int s = 1; s < S; ++s) {
              const float4 u = from[s * 128];
              v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
            }
            if (!came) v.x = v.y = v.z = v.w = __uint_as_float(0x7fffffffu);
            out.put(b, live - b, v.x, v.y, before[q][0], before[q][1]);
            out.put(b + 2, live - b - 2, v.z, v.w, before[q][2], before[q][3]);
          }
        }
      });
    }
  } else if (writes) {
    w4_with_out(p, t0 + b0, n, [&](auto out) { w4_put_rows<GB>(out, acc, rows); });
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(TM_COLS) : "memory");
  }
}

// ---------------------------------------------------------------- many rows

// As w4_tc_kernel for more tiles than SMs: a CTA stays and takes tile after
// tile; copies and MMAs of the next one run on while this one's sums are written
// out.  TN = 256: one accumulator, which the next tile may use as soon as it has
// been read to registers; below that two that take turns.  At 1,024 rows times 19,456
// x 2,560 (38.8 us, 2.6 PFLOP/s) a k-tile of 256 rows takes about 650 clocks, 512 of
// them MMAs; the first tile of a CTA, whose weights come from memory, 2 us more than
// the others, the start 3 us and the last tile's output 2 us.  Half of the rows'
// copies shared by two CTAs changed nothing; two tiles of weights against 128 rows
// took 40.7 us.
template <int TN, int STAGES>
__global__ void __launch_bounds__(w4_threads(TN))
w4_tc_rows_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                  const W4Params p) {
  constexpr int STAGE = w4_stage_bytes(TN), B_AT = 128 * 128, SF_AT = B_AT + TN * 128;
  constexpr int ST = (TN + 127) / 128, SFC = 4 + 4 * ST;       // tiles of row scales, scale columns of a stage
  constexpr int NB = TN > 192 ? 1 : 2, SF_COLS = NB * TN, TM_COLS = w4_tmem_cols(SF_COLS + STAGES * SFC);
  constexpr int GN = TN / w4_groups(TN);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  __shared__ __align__(8) uint64_t full[STAGES], empty[STAGES], acc_full[2], acc_empty[2], drained;
  __shared__ uint32_t tmem_base;
  __shared__ int s_fail;
  volatile int* fail = &s_fail;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int KT = p.KT, chunks = (KT + p.chunk - 1) / p.chunk;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4 * w4_groups(TN));
    }
    mbar_init(&drained, 1);
    s_fail = 0;
    fence_mbar_init();
    asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(&map_w)) : "memory");
    asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(&map_x)) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(&tmem_base)), "r"(TM_COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  pdl_launch_next();
  pdl_wait();

  if (warp == 0) {
    if (elect_one()) {
      const uint64_t mw = reinterpret_cast<uint64_t>(&map_w), mx = reinterpret_cast<uint64_t>(&map_x);
      const uint32_t sm = smem_u32(smem), full0 = smem_u32(full);
      const int row_tiles = (p.T + 127) >> 7;
      int tile = blockIdx.x, left = 0, done = 0, n0 = 0, t0 = 0, k = 0;
      const uint8_t *ws = nullptr, *xs = nullptr;
      size_t next = 0;
      // stages by number, so that their addresses are constants: what one thread
      // issues for a k-tile has to take less time than the tile's products
      for (uint32_t parity = 1; tile < p.tiles; parity ^= 1) {
#pragma unroll
        for (int i = 0; i < STAGES; ++i) {
          if (left == 0) {
            if (tile >= p.tiles) break;
            n0 = tile % p.n_tiles * 128;
            t0 = tile / p.n_tiles * TN;
            ws = p.w_scale + (size_t)(n0 >> 7) * KT * kMxTile;
            xs = p.x_scale + (size_t)(t0 >> 7) * KT * kMxTile;
            // behind the last rows there is no scale tile; another one's serves
            next = (t0 >> 7) + 1 < row_tiles ? (size_t)KT * kMxTile : 0;
            k = 0;
            left = KT;
          }
          if (!w4_wait(&empty[i], parity, p.polls, fail)) {
            tile = p.tiles;
            break;
          }
          const uint32_t st = sm + i * STAGE, bar = full0 + i * 8;
          mbar_arrive_expect_tx(&full[i], 128 * 64 + TN * 128 + (1 + ST) * kMxTile);
          w4_load_2d(st, mw, k, n0, bar);
          w4_load_2d(st + B_AT, mx, k, t0, bar);
          w4_load(st + SF_AT, ws, bar);
          w4_load(st + SF_AT + kMxTile, xs, bar);
          if (ST > 1) w4_load(st + SF_AT + 2 * kMxTile, xs + next, bar);
          ws += kMxTile;
          xs += kMxTile;
          k += 128;
          ++done;
          if (--left == 0) tile += gridDim.x;
        }
      }
      // behind a wait that gave up, copies may still be under way
      mbar_wait(&drained, 0, nullptr);
      for (int s = *fail ? max(done - STAGES, 0) : done; s < done; ++s)
        mbar_wait(&full[s % STAGES], (s / STAGES) & 1, nullptr);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t st0 = desc_lo(smem_u32(smem)), sf0 = tmem + SF_COLS;
      int tile = blockIdx.x, left = 0, chunk = 0, buf = 0;      // k-tiles of the tile, and of the sum under way
      uint32_t d = tmem, sfb = 4, acc_parity = 1, accum = 0;
      for (uint32_t parity = 0; tile < p.tiles; parity ^= 1) {
#pragma unroll
        for (int i = 0; i < STAGES; ++i) {
          if (chunk == 0) {
            if (tile >= p.tiles) break;
            if (left == 0) {
              left = KT;
              // a tile of 192 rows may begin in the middle of a scale tile, 32 rows a column
              sfb = 4 + (TN % 128 ? (tile / p.n_tiles * TN & 127) >> 5 : 0);
            }
            if (!w4_wait(&acc_empty[buf], acc_parity, p.polls, fail)) {
              tile = p.tiles;
              break;
            }
            chunk = min(left, p.chunk);
            d = tmem + buf * TN;
            accum = 0;
          }
          if (!w4_wait(&full[i], parity, p.polls, fail)) {
            tile = p.tiles;
            break;
          }
          tc_fence_after();
          const uint32_t st = st0 + (i * STAGE >> 4), sf = sf0 + i * SFC;
          tmem_cp_scales(sf, st + (SF_AT >> 4));
#pragma unroll
          for (int j = 0; j < ST; ++j) tmem_cp_scales(sf + 4 + 4 * j, st + ((SF_AT + (1 + j) * kMxTile) >> 4));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            umma_mxf8f6f4(d, st + 2 * j, st + (B_AT >> 4) + 2 * j, idesc_e2m1_e4m3(128, TN, j), sf, sf + sfb, accum);
            accum = 1;
          }
          umma_commit(&empty[i]);
          --left;
          if (--chunk == 0) {
            umma_commit(&acc_full[buf]);
            if (left == 0) tile += gridDim.x;
            if (++buf == NB) {
              buf = 0;
              acc_parity ^= 1;
            }
          }
        }
      }
      umma_commit(&drained);
    }
  } else {
    const int group = (warp - 2) / 4, f = (warp & 3) * 32 + lane;
    const uint32_t from = tmem + ((uint32_t)((warp & 3) * 32) << 16) + group * GN;
    int buf = 0;
    uint32_t parity = 0;
    bool ok = true;      // behind a wait that gave up all further tiles are NaN
    for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
      float acc[GN];
      for (int c = 0; c < chunks; ++c) {
        if (!ok || !(ok = w4_wait_warp(&acc_full[buf], parity, p.polls, fail))) break;
        tc_fence_after();
        if (c == 0) {
          tmem_ld_row<GN>(from + buf * TN, acc);
        } else if (TN <= 192) {      // one chunk otherwise
#pragma unroll
          for (int i = 0; i < GN; i += 32) {
            float v[32];
            tmem_ld_row<32>(from + buf * TN + i, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[i + j] += v[j];
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[buf]);
        if (++buf == NB) {
          buf = 0;
          parity ^= 1;
        }
      }
      if (!ok) {
#pragma unroll
        for (int i = 0; i < GN; ++i) acc[i] = __uint_as_float(0x7fffffffu);
      }
      const int t0 = tile / p.n_tiles * TN + group * GN;
      w4_with_out(p, t0, tile % p.n_tiles * 128 + f, [&](auto out) { w4_put_rows<GN>(out, acc, p.T - t0); });
    }
  }
  __syncwarp();
  mbar_wait(&drained, 0, nullptr);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(TM_COLS) : "memory");
  }
}

// The parts in memory, for rows that the product's own warps would not keep up with.
template <typename T, int P>
__global__ void __launch_bounds__(256) w4_parts_kernel(W4GemmArgs a, uint8_t* rows8, long long ld8, uint8_t* scale) {
  pdl_launch_next();
  pdl_wait();
  const int lane = threadIdx.x & 31, KT = (a.K + 127) / 128;
  const int u = blockIdx.x * 8 + (threadIdx.x >> 5);       // a warp: 128 values of a row, four a lane
  if (u >= a.T * KT) return;
  const int b = u / KT, kt = u % KT, k0 = kt * 128 + lane * 4;
  Raw4<T> raw;
  raw.load(static_cast<const T*>(a.x) + b * a.ldx, k0, a.K, a.vec);
  float v[4];
  raw.get(v);
  parts_of<P>(v, lane, [&](int p, uint32_t c, uint32_t w) {
    const long long row = (long long)b * P + p;
    *reinterpret_cast<uint32_t*>(rows8 + row * ld8 + k0) = c;
    if (lane == 0) *reinterpret_cast<uint32_t*>(scale + mx_scale_at(row, kt, KT)) = w;
  });
}

// ---------------------------------------------------------------- host side

// Stages, in clusters a tile's quads of rows from up to eight parts, and room to
// start on 1,024 bytes.
template <int TN, int STAGES, int P, bool CL>
constexpr int w4_smem() {
  return STAGES * w4_stage_bytes(TN) + (CL ? ((TN / P + 3) / 4 + 7) * 2048 : 0) + 1024;
}

template <int TN, int STAGES, int P, bool CL, typename TX>
cudaError_t launch_tc(const CUtensorMap& mw, const CUtensorMap& mx, const W4Params& p, dim3 grid, cudaStream_t st) {
  constexpr int SMEM = w4_smem<TN, STAGES, P, CL>();
  auto k = w4_tc_kernel<TN, STAGES, P, CL, TX>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(w4_threads(TN) + (sizeof(TX) > 1 ? 128 : 0));
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = grid.z;
  cfg.attrs = attr;
  cfg.numAttrs = CL ? 2 : 1;
  return s2_launch(&cfg, k, mw, mx, p);
}

// Clusters of S CTAs that are on the current device at once (kept per device).
template <int TN, int STAGES, int P, typename TX = uint8_t>
cudaError_t cluster_room(int S, int* n) {
  static KeptCounts<9> kept;
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  return kept.get(dev, S, n, [&](int* m) {
    constexpr int SMEM = w4_smem<TN, STAGES, P, true>();
    auto k = w4_tc_kernel<TN, STAGES, P, true, TX>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1, 1, S);
    cfg.blockDim = dim3(w4_threads(TN) + (sizeof(TX) > 1 ? 128 : 0));
    cfg.dynamicSmemBytes = SMEM;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = S;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(m, k, &cfg);
  });
}

// As many parts of K as have room on the SMs at once, two k-tiles each at least.
// An error of the device is passed on: another number of parts gives other bits.
template <int TN, int STAGES, int P, typename TX = uint8_t>
cudaError_t w4_parts(int KT, long long tiles, int* parts) {
  int S = KT / 2 < 8 ? KT / 2 : 8;
  for (; S > 1; --S) {
    int room = 0;
    const cudaError_t e = cluster_room<TN, STAGES, P, TX>(S, &room);
    if (e != cudaSuccess) return e;
    if (tiles <= room) break;
  }
  *parts = S > 1 ? S : 1;
  return cudaSuccess;
}

int w4_sms() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 1;
}

// Tensor maps and parameters; T * P rows in tiles of TN.
template <int TN, int P>
bool w4_fill(const W4GemmArgs& a, const uint8_t* rows8, long long ld8, const uint8_t* x_scale, CUtensorMap* mw,
             CUtensorMap* mx, W4Params* p) {
  p->N = a.N;
  p->T = a.T;
  p->KT = (a.K + 127) / 128;
  p->n_tiles = (a.N + 127) / 128;
  const long long tiles = (long long)p->n_tiles * (P > 1 ? 1 : (a.T + TN - 1) / TN);
  p->tiles = (int)tiles;
  p->chunk = 7;
  p->mode = a.mode;
  p->y_bf16 = a.y_bf16;
  p->ldy = a.ldy;
  p->codes = a.codes;
  p->w_scale = a.scale;
  p->x_scale = x_scale;
  p->y = a.y;
  p->polls = a.polls;
  p->K = a.K;
  p->x = a.x;
  p->ldx = a.ldx;
  p->x_vec = a.vec;
  return tiles <= 0x3fffffff && tma_map_w4(mw, a.codes, a.N, p->KT * 128) &&
         (!rows8 || tma_map_u8_2d(mx, rows8, (long long)a.T * P, a.K, ld8, TN));
}

// rows8: T * P rows of the operand (null: plain rows of TX).  SC: stages where
// parts of K are joined (32 rows times 2,560 x 9,728 in six parts 6.6 us; through
// loads from the parts' shared memory, between two cluster barriers, 9.3).
template <int TN, int STAGES, int P, int SC = STAGES, typename TX = uint8_t>
cudaError_t launch_tn(const W4GemmArgs& a, const uint8_t* rows8, long long ld8, const uint8_t* x_scale,
                      cudaStream_t st) {
  CUtensorMap mw, mx = {};
  W4Params p;
  if (!w4_fill<TN, P>(a, rows8, ld8, x_scale, &mw, &mx, &p)) return cudaErrorInvalidValue;
  int S = 1;
  const cudaError_t e = w4_parts<TN, SC, P, TX>(p.KT, p.tiles, &S);
  if (e != cudaSuccess) return e;
  if (S > 1) return launch_tc<TN, SC, P, true, TX>(mw, mx, p, dim3(p.tiles, 1, S), st);
  // More tiles than SMs: half the stages, so that two CTAs share an SM and one's
  // start and end lie under the other's products (1 row times 20,000 x 2,560 11.2 ->
  // 8.0 us, times 156,032 x 2,560 50.5 -> 41.5).
  if constexpr (TN <= 64) {
    if (p.tiles > w4_sms()) return launch_tc<TN, (STAGES + 1) / 2, P, false, TX>(mw, mx, p, dim3(p.tiles), st);
  }
  return launch_tc<TN, STAGES, P, false, TX>(mw, mx, p, dim3(p.tiles), st);
}

constexpr int kWholeSum = 128;      // k-tiles

template <int TN, int STAGES>
cudaError_t launch_rows(const W4GemmArgs& a, cudaStream_t st) {
  CUtensorMap mw, mx;
  W4Params p;
  if (!w4_fill<TN, 1>(a, a.x8, a.ld8, a.x_scale, &mw, &mx, &p)) return cudaErrorInvalidValue;
  // What the tensor core's sums lose over 16,384 k is about 2^-15 of sum |x w| at
  // most, 2^-7 of what an output of bf16 is rounded by unless the sum cancels; the
  // interface says so.  4,000 rows times 2,560 x 9,728 take 67.5 us, 70.3 with sums of
  // seven tiles; tiles of 256 rows have one accumulator, which must hold them all.
  if (a.y_bf16) p.chunk = min(p.KT, kWholeSum);
  constexpr int SMEM = STAGES * w4_stage_bytes(TN) + 1024;
  auto k = w4_tc_rows_kernel<TN, STAGES>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(min(p.tiles, w4_sms()));
  cfg.blockDim = dim3(w4_threads(TN));
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return s2_launch(&cfg, k, mw, mx, p);
}

}  // namespace

size_t w4_gemv_ws_bytes(int K, int B) {
  const size_t KT = (K + 127) / 128;
  return KT * kMxTile + (size_t)B * kParts32 * KT * 128;
}

cudaError_t launch_w4_gemv(const W4GemmArgs& a, cudaStream_t st) {
  const int KT = (a.K + 127) / 128, P = a.x_bf16 ? kParts16 : kParts32;
  if (a.T <= kPlainRows)
    return a.x_bf16 ? launch_tn<16, 10, kParts16, 10, __nv_bfloat16>(a, nullptr, 0, nullptr, st)
                    : launch_tn<16, 10, kParts32, 10, float>(a, nullptr, 0, nullptr, st);
  uint8_t* scale = static_cast<uint8_t*>(a.ws);
  uint8_t* rows8 = scale + (size_t)KT * kMxTile;
  const long long ld8 = KT * 128LL;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.T * KT + 7) / 8);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = a.x_bf16 ? s2_launch(&cfg, w4_parts_kernel<__nv_bfloat16, kParts16>, a, rows8, ld8, scale)
                                 : s2_launch(&cfg, w4_parts_kernel<float, kParts32>, a, rows8, ld8, scale);
  if (e != cudaSuccess) return e;
  W4GemmArgs q = a;
  q.K = (int)ld8;        // the parts' rows are padded with zeros
  if (a.x_bf16)
    return a.T * P <= 16 ? launch_tn<16, 10, kParts16>(q, rows8, ld8, scale, st)
                         : launch_tn<32, 8, kParts16>(q, rows8, ld8, scale, st);
  return a.T * P <= 32 ? launch_tn<32, 8, kParts32>(q, rows8, ld8, scale, st)
                       : launch_tn<48, 8, kParts32>(q, rows8, ld8, scale, st);
}

cudaError_t launch_w4_gemm(const W4GemmArgs& a, cudaStream_t st) {
  if (a.T <= 16) return launch_tn<16, 10, 1>(a, a.x8, a.ld8, a.x_scale, st);
  if (a.T <= 32) return launch_tn<32, 8, 1>(a, a.x8, a.ld8, a.x_scale, st);
  const int KT = (a.K + 127) / 128, n_tiles = (a.N + 127) / 128, sms = w4_sms();
  if (a.T <= 64) return launch_tn<64, 7, 1>(a, a.x8, a.ld8, a.x_scale, st);
  // up to 128 rows in two tiles of 64 where the SMs have room and K's parts do not
  // get long: what they send one another halves, but each takes in the weights for
  // itself.  128 rows times 6,144 x 2,560 10.1 -> 6.7 us, 2,560 x 4,096 7.9 -> 7.4, 4,096 x
  // 4,096 9.0 -> 9.1; 80 rows 8.7 -> 6.6, 6.8 -> 7.0, 7.8 -> 8.8.  Longer parts: 128 rows times
  // 4,096 x 8,192 11.5 -> 11.8 us, 2,560 x 9,728 10.2 -> 9.9; 80 rows 10.3 -> 11.5, 9.1 -> 9.6.
  if (a.T <= 128 && 2 * n_tiles <= sms) {
    int S = 1;
    const cudaError_t e = w4_parts<64, 7, 1>(KT, 2 * n_tiles, &S);
    if (e != cudaSuccess) return e;
    if ((KT + S - 1) / S <= 20) return launch_tn<64, 7, 1>(a, a.x8, a.ld8, a.x_scale, st);
  }
  if (a.T <= 128 && n_tiles <= sms) return launch_tn<128, 6, 1, 4>(a, a.x8, a.ld8, a.x_scale, st);
  // Tiles of 128, 192 or 256 rows by what a pass over the SMs would take, in
  // units of 10 ns: a k-tile 25, 32 or 45 (1,024 rows times 19,456 x 2,560: 44.6,
  // 42.2 and 38.9 us), a tile's end 60; or tiles of 128 with K in S parts.
  auto cost = [&](int tn, int k_tile) {
    const long long tiles = (long long)n_tiles * ((a.T + tn - 1) / tn);
    return (tiles + sms - 1) / sms * (KT * k_tile + 60);
  };
  const long long c128 = cost(128, 25), c192 = cost(192, 32), c256 = a.y_bf16 && KT <= kWholeSum ? cost(256, 45) : 1LL << 60;
  const long long best = c128 < c192 ? (c128 < c256 ? c128 : c256) : (c192 < c256 ? c192 : c256);
  const long long tiles = (long long)n_tiles * ((a.T + 127) / 128);
  int S = 1;
  const cudaError_t e = w4_parts<128, 4, 1>(KT, tiles, &S);
  if (e != cudaSuccess) return e;
  if (S > 1 && (KT + S - 1) / S * 27LL + 250 < best) return launch_tn<128, 6, 1, 4>(a, a.x8, a.ld8, a.x_scale, st);
  if (c256 == best) return launch_rows<256, 4>(a, st);
  return c192 == best ? launch_rows<192, 5>(a, st) : launch_rows<128, 6>(a, st);
}

}  // namespace s2
