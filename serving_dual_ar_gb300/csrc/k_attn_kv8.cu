// Decode attention over the 8-bit KV cache: q/k norm and RoPE, append of the
// new rows, attention of all rows of a (sequence, kv head), one launch.
#include <cuda.h>

#include "kv8_common.cuh"
#include "tc_common.cuh"
#include "tma_map.h"

namespace s2 {

namespace {

constexpr int kDecWarps = 8;
constexpr int kDecMaxDepth = 8;
constexpr int kDecSmem = 227 * 1024;

// Warps in use for U pages of work: at least kDecMinPages each.
constexpr int kDecMinPages = 2;

struct DecLayout {
  int depth;                       // pages in flight per warp
  int slot_off, meta_off;          // bytes
  int slot_floats;                 // one partial: R rows of HD values, then (m, l) of each
  int ctas;
  int vec;                         // query rows, gains and RoPE rows on 16-byte boundaries
};

S2_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
S2_DEV uint32_t f16x2(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// x, y as f16 pairs hi + lo
S2_DEV void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = f16x2(x - f.x, y - f.y);
}
S2_DEV void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
               "{%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
S2_DEV void tma_load_page(void* dst, const CUtensorMap* map, int g, int page, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %2, %3, %2, %4}], [%5];"
      :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(g), "r"(page), "r"(smem_u32(bar))
      : "memory");
}
// Byte offset of the 16-byte unit c of a block's row in the layout that the
// copy engine writes (128- or 64-byte swizzle, by the row's length).
template <int HD>
S2_DEV uint32_t unit_off(int row, int c) {
  return HD == 128 ? row * 128 + ((c ^ (row & 7)) << 4) : row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
}

template <int N>
S2_DEV void load_row(const float* p, bool vec, float (&v)[N]) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(p + i);
      v[i] = x.x;
      v[i + 1] = x.y;
      v[i + 2] = x.z;
      v[i + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = p[i];
  }
}

// Run ``i`` of the ``runs`` equal ones that U units are cut into starts at
// unit Cut::start(i); Cut::of(u) is the run that holds unit u.
struct Cut {
  unsigned base, more;    // every run has base units, the first ``more`` one more
  S2_DEV unsigned start(unsigned i) const { return i * base + min(i, more); }
  S2_DEV unsigned of(unsigned u) const {
    const unsigned big = more * (base + 1);
    return u < big ? u / (base + 1) : more + (u - big) / base;
  }
};

// What a warp knows of one page of work.
struct Unit {
  int page, seg, j, exps;   // page id (-1: not to be followed), b * Hkv + g, page of the sequence, K and V exponents
};

template <int HD>
struct DecState {           // one piece of a (sequence, kv head): all rows, log2 domain
  float o[HD / 8][4];       // tile t: dims n * HD/8 + t of column n; [0..1] hi part of row r, [2..3] lo part
  float m, l;               // row r = lane / 4 (l: this lane's keys)
  int E;                    // o counts in units of 2^(E - 14)
};

// One result row set into o: dims [c * HD/4, (c + 1) * HD/4) of row r.
template <int HD>
S2_DEV void store_rows(const Kv8Args& a, int seg, int r, int c, const float (&y)[HD / 4]) {
  const int G = a.H / a.Hkv;
  if (r >= a.m * G) return;
  const int b = seg / a.Hkv, g = seg % a.Hkv;
  const size_t at = (size_t)(b * a.m + r / G) * a.o_ld + (size_t)(g * G + r % G) * HD + c * (HD / 4);
  if (a.o) {
    float* p = a.o + at;
    if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
#pragma unroll
      for (int i = 0; i < HD / 4; i += 4)
        *reinterpret_cast<float4*>(p + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < HD / 4; ++i) p[i] = y[i];
    }
  } else {
    __nv_bfloat16* p = a.o16 + at;
    if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
#pragma unroll
      for (int i = 0; i < HD / 4; i += 8) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(y[i + 2 * k], y[i + 2 * k + 1]);
          w[k] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p + i) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < HD / 4; ++i) p[i] = __float2bfloat16_rn(y[i]);
    }
  }
}

// Joining of partials (rows of HD values relative to 2^m, and (m, l)).
template <int HD>
struct Join {
  float o[HD / 4], m = -INFINITY, l = 0.f;
  S2_DEV Join() {
#pragma unroll
    for (int i = 0; i < HD / 4; ++i) o[i] = 0.f;
  }
  // All of the partials slot(k), first <= k < last, in order: the largest
  // maximum first, so that the loads of the values wait for nothing.
  template <bool kGlobal, typename F>
  S2_DEV void take(F slot, int first, int last, int R, int r, int c) {
    if (r >= R) return;
#pragma unroll 4
    for (int k = first; k < last; ++k) {
      const float* p = slot(k);
      if (p) m = fmaxf(m, kGlobal ? __ldcg(p + R * HD + 2 * r) : p[R * HD + 2 * r]);
    }
#pragma unroll 2
    for (int k = first; k < last; ++k) {
      const float* p = slot(k);
      if (!p) continue;
      const float* ml = p + R * HD + 2 * r;
      const float m2 = kGlobal ? __ldcg(ml) : ml[0], l2 = kGlobal ? __ldcg(ml + 1) : ml[1];
      const float y = m2 == -INFINITY ? (l2 == l2 ? 0.f : l2) : ex2(m2 - m);   // no keys: nothing; NaN stays
      l += l2 * y;
      const float4* s = reinterpret_cast<const float4*>(p + r * HD + c * (HD / 4));
#pragma unroll
      for (int i = 0; i < HD / 16; ++i) {
        const float4 v = kGlobal ? __ldcg(s + i) : s[i];
        o[4 * i] += v.x * y;
        o[4 * i + 1] += v.y * y;
        o[4 * i + 2] += v.z * y;
        o[4 * i + 3] += v.w * y;
      }
    }
  }
  S2_DEV void put(float* slot, int R, int r, int c) const {
    if (r >= R) return;
    float4* s = reinterpret_cast<float4*>(slot + r * HD + c * (HD / 4));
#pragma unroll
    for (int i = 0; i < HD / 16; ++i) s[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    if (c == 0) {
      slot[R * HD + 2 * r] = m;
      slot[R * HD + 2 * r + 1] = l;
    }
  }
  S2_DEV void finish() {
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < HD / 4; ++i) o[i] *= inv;
  }
};

// The work is the list of all pages, in the order (sequence, kv head, page),
// cut into equal runs, one per warp of the grid: ragged lengths, one long
// sequence and many short ones all load every SM alike.  A warp streams its
// run through its own ring of shared-memory pages (one TMA copy brings a
// head's 16 keys and 16 values), with no barrier shared between warps.  A
// (sequence, kv head) that lies within one run is finished by its warp; one
// that is cut is joined from partials, first within the CTA, then, if its
// pages reach into other CTAs, by the last CTA to arrive, in order.
//
// Products: mma.sync m16n8k16 with the up to 8 query rows (new rows x heads
// of the kv head) as f16 hi parts in rows 0..7 and lo parts in rows 8..15, so
// the pair costs nothing; e4m3 bytes become f16 in registers.  The order of
// dims in Q K^T and of dims in the output is free, and is chosen such that
// each lane's bytes are contiguous: lane (n, c) takes dims c * HD/4 .. of key
// n, and dims n * HD/8 .. of the values of keys 2c, 2c + 1, 2c + 8, 2c + 9.
// The block scale of K multiplies the scores; the one of V goes into the
// weights, with the running exponent E handled like the running maximum.
template <int HD>
__global__ void __launch_bounds__(kDecWarps * 32, 1)
kv8_decode_kernel(const __grid_constant__ CUtensorMap map, Kv8Args a, DecLayout lay) {
  constexpr int NT = HD / 8;              // output tiles of 8 dims
  constexpr int KS = HD / 16;             // k-steps of the scores
  constexpr int UB = 2 * kKv8Page * HD;   // bytes of a unit
  extern __shared__ __align__(1024) uint8_t raw[];
  uint8_t* sm = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;
  __shared__ __align__(8) uint64_t bars[kDecWarps][kDecMaxDepth];
  __shared__ int scan_s[kDecWarps + 1];
  __shared__ int seg_s[2 * kDecWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, c = lane & 3;
  const int D = lay.depth, G = a.H / a.Hkv, R = a.m * G;
  int* first_s = reinterpret_cast<int*>(sm + lay.meta_off);   // pages before sequence b, B + 1 entries
  int* pos_s = first_s + a.B + 1;
  uint8_t* ring = sm + (size_t)warp * D * UB;
  float* slots = reinterpret_cast<float*>(sm + lay.slot_off) + (size_t)warp * 2 * lay.slot_floats;
  if (tid < kDecWarps * D) mbar_init(&bars[tid / D][tid % D], 1);
  if (tid < 2 * kDecWarps) seg_s[tid] = -1;
  fence_mbar_init();
  pdl_launch_next();
  pdl_wait();

  // pages of each sequence (none for one that is left out), and their sums
  {
    const int per = (a.B + kDecWarps * 32 - 1) / (kDecWarps * 32), b0 = tid * per;
    int own = 0;
    for (int b = b0; b < min(b0 + per, a.B); ++b) {
      const int p = a.pos[b];
      const bool in = p >= 0 && p <= a.max_pos - a.m;
      pos_s[b] = in ? p : -1;
      first_s[b] = own;
      own += in ? (p + a.m + kKv8Page - 1) / kKv8Page : 0;
    }
    int x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scan_s[warp + 1] = x;
    if (tid == 0) scan_s[0] = 0;
    __syncthreads();
    int before = x - own;
    for (int w = 0; w <= warp; ++w) before += scan_s[w];
    for (int b = b0; b < min(b0 + per, a.B); ++b) first_s[b] += before;
    if (tid == kDecWarps * 32 - 1) first_s[a.B] = before + own;
    __syncthreads();
  }
  for (int b = blockIdx.x; b < a.B; b += gridDim.x)
    if (pos_s[b] < 0)
      for (int i = tid; i < a.m * a.H * HD; i += kDecWarps * 32) {
        const size_t at = (size_t)(b * a.m + i / (a.H * HD)) * a.o_ld + i % (a.H * HD);
        if (a.o) a.o[at] = 0.f;
        else a.o16[at] = __float2bfloat16_rn(0.f);
      }
  // units fit 31 bits (the caller refuses more)
  const unsigned U = (unsigned)first_s[a.B] * a.Hkv;
  if (U == 0) return;
  const unsigned W = min(gridDim.x * kDecWarps, (U + kDecMinPages - 1) / kDecMinPages);
  if (blockIdx.x * kDecWarps >= W) return;
  const Cut cut{U / W, U % W};
  const unsigned wid = min(blockIdx.x * kDecWarps + warp, W);
  const unsigned u0 = cut.start(wid);
  const int n = wid < W ? (int)(cut.start(wid + 1) - u0) : 0;

  // the unit u0 + t, looked up by lane t % 32
  auto look_up = [&](int t) {
    Unit x{-1, -1, 0, 0};
    if (t >= n) return x;
    const unsigned u = u0 + t;
    int lo = 0, hi = a.B;                       // last b with first unit <= u
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((unsigned)first_s[mid] * a.Hkv <= u) lo = mid;
      else hi = mid;
    }
    const int pages = first_s[lo + 1] - first_s[lo];
    const int rem = (int)(u - (unsigned)first_s[lo] * a.Hkv), g = rem / pages;
    x.j = rem - g * pages;
    x.seg = lo * a.Hkv + g;
    const int p = a.table[(size_t)lo * a.table_ld + x.j];
    if (p >= 0 && p < a.n_pages) {
      x.page = p;
      const float* s = a.scale + (size_t)p * 2 * a.Hkv + g;
      x.exps = (kv8_scale_exp(s[0]) + 64) | ((kv8_scale_exp(s[a.Hkv]) + 64) << 8);
    }
    return x;
  };
  auto issue = [&](const Unit& x, int t) {      // by the lane that looked it up
    uint64_t* bar = &bars[warp][t % D];
    if (x.page < 0) mbar_arrive(bar);
    else {
      mbar_arrive_expect_tx(bar, UB);
      tma_load_page(ring + (size_t)(t % D) * UB, &map, x.seg % a.Hkv, x.page, bar);
    }
  };

  Unit cur = look_up(lane), nxt{-1, -1, 0, 0};
  if (lane < min(D, n)) issue(cur, lane);
  if (n > 32) nxt = look_up(32 + lane);

  uint32_t qa[KS][4];        // query fragments: {hi, lo} x {dims 4t, 4t+1 | 4t+2, 4t+3}
  float qf = 0.f;            // 2^-(exponent given to row r's query)
  DecState<HD> st;
  int seg = -1, pos = 0;
  bool nan_new = false;      // a new value row after the first holds a NaN

  auto begin = [&](int s) {
    seg = s;
    nan_new = false;
    const int b = s / a.Hkv, g = s % a.Hkv;
    pos = pos_s[b];
    st.m = -INFINITY;
    st.l = 0.f;
    st.E = kKv8EMin;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[t][e] = 0.f;
    // lane (r, c): dims c HD/4 .. of query row r, whose rotation partners lane
    // (r, c ^ 2) has; all loads at once
    float q[HD / 4], gain[HD / 4], co[HD / 4], si[HD / 4];
    const bool vec = lay.vec;
    if (r < R) {
      const int p = pos + r / G, half = (c & 1) * (HD / 4);
      load_row(a.qkv + (size_t)(b * a.m + r / G) * a.qkv_ld + (size_t)(g * G + r % G) * HD + c * (HD / 4), vec, q);
      load_row(a.q_gain + c * (HD / 4), vec, gain);
      load_row(a.rope_cos + (size_t)p * (HD / 2) + half, vec, co);
      load_row(a.rope_sin + (size_t)p * (HD / 2) + half, vec, si);
    } else {
#pragma unroll
      for (int i = 0; i < HD / 4; ++i) q[i] = gain[i] = co[i] = si[i] = 0.f;
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < HD / 4; ++i) ss += q[i] * q[i];
    ss += __shfl_xor_sync(0xffffffffu, ss, 1);
    ss += __shfl_xor_sync(0xffffffffu, ss, 2);
    // log2(e) / sqrt(HD): the softmax runs on powers of two
    const float f = rsqrtf(ss * (1.f / HD) + a.eps) * (HD == 128 ? 0.127517431f : 0.180336880f);
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < HD / 4; ++i) {
      q[i] *= f * gain[i];
      const float w = __shfl_xor_sync(0xffffffffu, q[i], 2);
      q[i] = q[i] * co[i] + (c < 2 ? -w : w) * si[i];
      mx = fmaxf(mx, fabsf(q[i]));
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // the row's largest magnitude to 2^12 .. 2^13: its pair then is good to
    // 2^-22 of each value and 2^-37 of the largest
    const int ex = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 100);
    const float up = pow2f(12 - ex);
    qf = pow2f(ex - 12);
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      split2(q[4 * t] * up, q[4 * t + 1] * up, qa[t][0], qa[t][1]);
      split2(q[4 * t + 2] * up, q[4 * t + 3] * up, qa[t][2], qa[t][3]);
    }
  };

  // The piece's rows relative to 2^m, as a Join: dims 2c NT + t and (2c + 1) NT + t.
  auto piece = [&](Join<HD>& x) {
    st.l += __shfl_xor_sync(0xffffffffu, st.l, 1);
    st.l += __shfl_xor_sync(0xffffffffu, st.l, 2);
    x.m = st.m;
    x.l = st.l;
    const float f = pow2f(st.E - 14);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      x.o[t] = (st.o[t][0] + st.o[t][2]) * f;
      x.o[NT + t] = (st.o[t][1] + st.o[t][3]) * f;
    }
    if (nan_new && r < R) {      // the rows that see it get it back
      const int b = seg / a.Hkv, g = seg % a.Hkv;
      for (int i = 0; i <= r / G; ++i) {
        const float* v = a.qkv + (size_t)(b * a.m + i) * a.qkv_ld + (size_t)(a.H + a.Hkv + g) * HD + c * (HD / 4);
        for (int k = 0; k < HD / 4; ++k)
          if (v[k] != v[k]) x.o[k] = v[k];
      }
    }
  };
  auto end = [&](int t_end) {    // piece of ``seg`` up to unit t_end of the run
    const int b = seg / a.Hkv, g = seg % a.Hkv, pages = first_s[b + 1] - first_s[b];
    const unsigned s0 = (unsigned)first_s[b] * a.Hkv + (unsigned)g * pages;
    Join<HD> x;
    piece(x);
    if (s0 >= u0 && s0 + pages <= u0 + t_end) {
      x.finish();
      store_rows<HD>(a, seg, r, c, x.o);
    } else {
      const int k = seg_s[2 * warp] < 0 ? 0 : 1;
      x.put(slots + k * lay.slot_floats, R, r, c);
      __syncwarp();
      if (lane == 0) seg_s[2 * warp + k] = seg;
      __syncwarp();
    }
  };

  // One new key (normed, rotated) and value, lane l taking dims l + 32 i.
  constexpr int N = HD / 32;
  float k[N], v[N];
  auto row = [&](int p) {
    const int b = seg / a.Hkv, g = seg % a.Hkv;
    const float* x = a.qkv + (size_t)(b * a.m + p - pos) * a.qkv_ld + (size_t)(a.H + g) * HD;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = x[(size_t)a.Hkv * HD + lane + 32 * i];
    kv8_key_row<HD>(x, a.k_gain, a.rope_cos + (size_t)p * (HD / 2), a.rope_sin + (size_t)p * (HD / 2), a.eps, lane, k);
  };
  // New rows of this page into its shared-memory copy and to the pool; the
  // page's last new row is in k, v already.
  auto append = [&](uint8_t* blk, int page, int j, int& ke, int& ve) {
    const int b = seg / a.Hkv, g = seg % a.Hkv;
    const int first = max(pos, j * kKv8Page), last = min(pos + a.m, (j + 1) * kKv8Page);
    const int had = first - j * kKv8Page, rows = last - j * kKv8Page;
    float mk = abs_max(k, 0.f), mv = abs_max(v, 0.f);
    for (int p = last - 2; p >= first; --p) {
      row(p);
      mk = abs_max(k, mk);
      mv = abs_max(v, mv);
    }
    const int ko = had ? ke : kKv8EMin, vo = had ? ve : kKv8EMin;
    ke = max(ko, kv8_exponent(warp_max(mk)));
    ve = max(vo, kv8_exponent(warp_max(mv)));
    const bool grew[2] = {had && ke > ko, had && ve > vo};
    const float by[2] = {pow2f(ko - ke), pow2f(vo - ve)};
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint8_t* x = blk + t * (kKv8Page * HD);
      if (grew[t])
        for (int i = lane; i < had * HD / 16; i += 32) {
          uint4* w = reinterpret_cast<uint4*>(x + unit_off<HD>(i / (HD / 16), i % (HD / 16)));
          uint4 y = *w;
          y.x = e4m3_rescale4(y.x, by[t]);
          y.y = e4m3_rescale4(y.y, by[t]);
          y.z = e4m3_rescale4(y.z, by[t]);
          y.w = e4m3_rescale4(y.w, by[t]);
          *w = y;
        }
    }
    uint8_t* xv = blk + kKv8Page * HD;
    for (int i = rows * HD / 16 + lane; i < HD; i += 32)   // rows behind the last one: their weight is 0, not their bytes
      *reinterpret_cast<uint4*>(xv + unit_off<HD>(i / (HD / 16), i % (HD / 16))) = make_uint4(0, 0, 0, 0);
    const float fk = pow2f(-ke), fv = pow2f(-ve);
    for (int p = first; p < last; ++p) {
      if (p != first) row(p);       // k, v: the first row, the last one computed
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int d = lane + 32 * i;
        const uint32_t at = unit_off<HD>(p % kKv8Page, d >> 4) + (d & 15);
        blk[at] = (uint8_t)e4m3x2(k[i] * fk, 0.f);
        xv[at] = (uint8_t)e4m3x2(v[i] * fv, 0.f);
      }
    }
    __syncwarp();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint8_t* out = a.kv + (((size_t)page * 2 + t) * a.Hkv + g) * (kKv8Page * HD);
      const uint8_t* x = blk + t * (kKv8Page * HD);
      for (int i = (grew[t] ? 0 : had) * HD / 16 + lane; i < rows * HD / 16; i += 32)
        *reinterpret_cast<uint4*>(out + (size_t)i * 16) =
            *reinterpret_cast<const uint4*>(x + unit_off<HD>(i / (HD / 16), i % (HD / 16)));
    }
    if (lane == 0) {
      float* s = a.scale + (size_t)page * 2 * a.Hkv + g;
      s[0] = pow2f(ke);
      s[a.Hkv] = pow2f(ve);
    }
    // A NaN among the new values must not reach the rows before it through
    // 0 * NaN: it leaves the copy, and ``piece`` gives it back to the others.
    if (a.m > 1) {
      __syncwarp();
      bool any = false;
      for (int p = first; p < last; ++p) {
        const float* x = a.qkv + (size_t)(b * a.m + p - pos) * a.qkv_ld + (size_t)(a.H + a.Hkv + g) * HD;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int d = lane + 32 * i;
          if (x[d] != x[d]) {
            any = true;
            xv[unit_off<HD>(p % kKv8Page, d >> 4) + (d & 15)] = 0;
          }
        }
      }
      nan_new = nan_new || __any_sync(0xffffffffu, any);
    }
    __syncwarp();
    fence_proxy_async();
  };

  for (int t = 0; t < n; ++t) {
    const int src = t & 31;
    const int page = __shfl_sync(0xffffffffu, cur.page, src), sg = __shfl_sync(0xffffffffu, cur.seg, src);
    const int j = __shfl_sync(0xffffffffu, cur.j, src), ex = __shfl_sync(0xffffffffu, cur.exps, src);
    if (sg != seg) {
      if (seg >= 0) end(t);
      begin(sg);
    }
    const bool tail = (j + 1) * kKv8Page > pos;
    if (tail) row(min(pos + a.m, (j + 1) * kKv8Page) - 1);
    bool ok = mbar_wait(&bars[warp][t % D], (uint32_t)(t / D) & 1u, nullptr);
    ok = __all_sync(0xffffffffu, ok) && page >= 0;
    if (ok) {
      uint8_t* blk = ring + (size_t)(t % D) * UB;
      int ke = (ex & 0xff) - 64, ve = (ex >> 8) - 64;
      if (tail) append(blk, page, j, ke, ve);

      // S = Q K^T for the page's two groups of 8 keys
      float s[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[h][e] = 0.f;
        const int key = h * 8 + r;
        uint32_t w[KS];
        if (HD == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(blk + unit_off<HD>(key, 2 * c));
          const uint4 y = *reinterpret_cast<const uint4*>(blk + unit_off<HD>(key, 2 * c + 1));
          w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
          w[KS - 4] = y.x; w[KS - 3] = y.y; w[KS - 2] = y.z; w[KS - 1] = y.w;
        } else {
          const uint4 x = *reinterpret_cast<const uint4*>(blk + unit_off<HD>(key, c));
          w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        }
#pragma unroll
        for (int k = 0; k < KS; ++k)
          mma_f16(s[h], qa[k], f16x2_of_e4m3((uint16_t)w[k]), f16x2_of_e4m3((uint16_t)(w[k] >> 16)));
      }
      const float f = qf * pow2f(ke);
      float p[4] = {(s[0][0] + s[0][2]) * f, (s[0][1] + s[0][3]) * f, (s[1][0] + s[1][2]) * f,
                    (s[1][1] + s[1][3]) * f};
      if (tail) {
        const int lim = pos + r / G - j * kKv8Page;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if ((e >> 1) * 8 + 2 * c + (e & 1) > lim) p[e] = -INFINITY;
      }
      float mx = fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(st.m, mx);
      const int En = max(st.E, ve);
      if (__any_sync(0xffffffffu, mn > st.m) || En > st.E) {
        const float x = mn == -INFINITY ? 1.f : ex2(st.m - mn), y = x * pow2f(st.E - En);
        st.l *= x;
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) st.o[q][e] *= y;
        st.m = mn;
        st.E = En;
      }
      // weights times 2^14 and the block's scale over 2^E: at most 2^14, a pair
      // of f16 then is good to 2^-22 of each and 2^-39 of the largest
      const float sub = (mn == -INFINITY ? 0.f : mn) - (float)(14 + ve - En);
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = ex2(p[e] - sub);
      st.l += ((p[0] + p[1]) + (p[2] + p[3])) * pow2f(En - ve - 14);
      uint32_t pa[4];
      split2(p[0], p[1], pa[0], pa[1]);
      split2(p[2], p[3], pa[2], pa[3]);

      // O += P V
      const uint8_t* xv = blk + kKv8Page * HD;
      uint32_t v[4][HD / 32];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = (e >> 1) * 8 + 2 * c + (e & 1);
        if (HD == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(xv + unit_off<HD>(key, r));
          v[e][0] = x.x; v[e][1] = x.y; v[e][HD / 32 - 2] = x.z; v[e][HD / 32 - 1] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(xv + unit_off<HD>(key, r >> 1) + (r & 1) * 8);
          v[e][0] = x.x; v[e][1] = x.y;
        }
      }
#pragma unroll
      for (int k = 0; k < HD / 32; ++k) {
        const uint32_t a01 = __byte_perm(v[0][k], v[1][k], 0x5140), a23 = __byte_perm(v[0][k], v[1][k], 0x7362);
        const uint32_t b01 = __byte_perm(v[2][k], v[3][k], 0x5140), b23 = __byte_perm(v[2][k], v[3][k], 0x7362);
        mma_f16(st.o[4 * k], pa, f16x2_of_e4m3((uint16_t)a01), f16x2_of_e4m3((uint16_t)b01));
        mma_f16(st.o[4 * k + 1], pa, f16x2_of_e4m3((uint16_t)(a01 >> 16)), f16x2_of_e4m3((uint16_t)(b01 >> 16)));
        mma_f16(st.o[4 * k + 2], pa, f16x2_of_e4m3((uint16_t)a23), f16x2_of_e4m3((uint16_t)b23));
        mma_f16(st.o[4 * k + 3], pa, f16x2_of_e4m3((uint16_t)(a23 >> 16)), f16x2_of_e4m3((uint16_t)(b23 >> 16)));
      }
    }
    __syncwarp();
    // the slot is free: the unit D further on
    const int ti = t + D;
    if (ti < n && lane == (ti & 31)) issue((ti >> 5) == (t >> 5) ? cur : nxt, ti);
    if (src == 31) {
      cur = nxt;
      nxt = look_up((t & ~31) + 64 + lane);
    }
  }
  if (seg >= 0) end(n);
  __syncthreads();

  // partials of this CTA's warps, each cut (sequence, kv head) by the warp of its first one
  const unsigned c0 = cut.start(blockIdx.x * kDecWarps), c1 = cut.start(min((blockIdx.x + 1) * kDecWarps, W));
  unsigned* tickets = reinterpret_cast<unsigned*>(a.ws);
  float* parts = reinterpret_cast<float*>(static_cast<char*>(a.ws) + ((size_t)a.B * a.Hkv * 4 + 255) / 256 * 256);
  const float* all = reinterpret_cast<const float*>(sm + lay.slot_off);
  int prev = -1;
  for (int e = 0; e < 2 * warp; ++e)
    if (seg_s[e] >= 0) prev = seg_s[e];
  for (int e = 2 * warp; e < 2 * warp + 2; ++e) {
    const int sg = seg_s[e];
    if (sg < 0 || sg == prev) continue;
    prev = sg;
    Join<HD> x;
    x.template take<false>(
        [&](int k) { return seg_s[k] == sg ? all + (size_t)k * lay.slot_floats : nullptr; }, e, 2 * kDecWarps, R, r, c);
    const int b = sg / a.Hkv, g = sg % a.Hkv, pages = first_s[b + 1] - first_s[b];
    const unsigned s0 = (unsigned)first_s[b] * a.Hkv + (unsigned)g * pages, s1 = s0 + pages;
    if (s0 >= c0 && s1 <= c1) {
      x.finish();
      store_rows<HD>(a, sg, r, c, x.o);
      continue;
    }
    // CTAs that share it: those of its first and of its last page
    const int f = (int)(cut.of(s0) / kDecWarps), l = (int)(cut.of(s1 - 1) / kDecWarps);
    x.put(parts + ((size_t)blockIdx.x * 2 + (s0 < c0 ? 0 : 1)) * lay.slot_floats, R, r, c);
    __threadfence();
    __syncwarp();
    unsigned got = 0;
    if (lane == 0) got = atomicAdd(&tickets[sg], 1u);
    got = __shfl_sync(0xffffffffu, got, 0);
    if (got != (unsigned)(l - f)) continue;
    __threadfence();
    Join<HD> y;
    y.template take<true>(
        [&](int k) { return parts + ((size_t)k * 2 + (k == f ? 1 : 0)) * lay.slot_floats; }, f, l + 1, R, r, c);
    y.finish();
    store_rows<HD>(a, sg, r, c, y.o);
    if (lane == 0) tickets[sg] = 0u;
  }
}

int num_sms() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 1;
}

DecLayout dec_layout(int B, int R, int hd) {
  DecLayout l;
  l.ctas = num_sms();
  l.slot_floats = R * hd + 2 * R + (2 * R) % 4;
  const int slot = kDecWarps * 2 * l.slot_floats * 4, meta = (2 * B + 1) * 4, unit = 2 * kKv8Page * hd;
  const int room = kDecSmem - 1024 - 2048 - slot - meta;   // alignment, static
  l.depth = room / (kDecWarps * unit);
  if (l.depth > kDecMaxDepth) l.depth = kDecMaxDepth;
  l.slot_off = kDecWarps * l.depth * unit;
  l.meta_off = l.slot_off + (slot + 15) / 16 * 16;
  return l;
}

}  // namespace

size_t kv8_decode_ws_bytes(int B, int m, int H, int Hkv, int hd) {
  const int R = m * (H / Hkv);
  const DecLayout l = dec_layout(B, R, hd);
  return ((size_t)B * Hkv * 4 + 255) / 256 * 256 + (size_t)l.ctas * 2 * l.slot_floats * 4;
}

cudaError_t launch_kv8_decode(const Kv8Args& a, cudaStream_t st) {
  CUtensorMap map;
  if (!tma_map_kv8(&map, a.kv, a.n_pages, a.Hkv, a.hd)) return cudaErrorNotSupported;
  DecLayout l = dec_layout(a.B, a.m * (a.H / a.Hkv), a.hd);
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.qkv) | reinterpret_cast<uintptr_t>(a.q_gain) |
                       reinterpret_cast<uintptr_t>(a.rope_cos) | reinterpret_cast<uintptr_t>(a.rope_sin);
  l.vec = (at & 15) == 0 && a.qkv_ld % 4 == 0;
  auto k = a.hd == 128 ? kv8_decode_kernel<128> : kv8_decode_kernel<64>;
  static bool attr[2] = {false, false};
  if (!attr[a.hd == 128]) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kDecSmem - 2048);
    if (e != cudaSuccess) return e;
    attr[a.hd == 128] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(l.ctas);
  cfg.blockDim = dim3(kDecWarps * 32);
  cfg.dynamicSmemBytes = l.meta_off + (2 * a.B + 1) * 4 + 1024;
  cfg.stream = st;
  // the kernel reads nothing before its wait on the launch before it
  cudaLaunchAttribute at1[1];
  at1[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at1[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at1;
  cfg.numAttrs = 1;
  return s2_launch(&cfg, k, map, a, l);
}

}  // namespace s2
