// Decode attention over the 8-bit KV cache: q/k norm and RoPE, append of the
// new rows, attention of all rows of a (sequence, kv head), one launch.
#include <cuda.h>

#include "kv8_common.cuh"
#include "tc_common.cuh"
#include "tma_map.h"

namespace s2 {

namespace {

constexpr int kDecWarps = 8;       // most warps of a CTA
constexpr int kDecMaxDepth = 8;
constexpr int kDecSmem = 227 * 1024;
// Pages of a run at least: a cut costs a joining, about as long as four pages.
constexpr int kDecMinPages = 4;
// Pieces that one warp joins; more are joined in two levels of about sqrt(n).
constexpr int kDecFlat = 12;

struct DecLayout {
  int groups, heads, slices;   // kv heads in groups of ``heads``; a CTA has heads x slices warps
  int depth;                   // pages in flight per warp
  int q_off, meta_off;         // bytes
  int slot_floats;             // one partial: R rows of HD values, then (m, l) of each
  int ctas;
  int vec;                     // query rows, gains and RoPE rows on 16-byte boundaries
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

S2_DEV float4 load4(const float* p, bool vec) {
  return vec ? *reinterpret_cast<const float4*>(p) : make_float4(p[0], p[1], p[2], p[3]);
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

// The key row as a call: it is rare, long and wanted at three places, and the
// kernel's other paths share the instruction cache with it.
template <int HD>
struct KeyRow {
  float v[HD / 32];
};
template <int HD>
__device__ __noinline__ KeyRow<HD> key_row_call(const float* x, const float* gain, const float* cs, const float* sn,
                                                float eps, int lane) {
  KeyRow<HD> y;
  kv8_key_row<HD>(x, gain, cs, sn, eps, lane, y.v);
  return y;
}

// What a warp knows of one page of work.
struct Unit {
  int page, seg, j;   // page id (-1: not to be followed), group * B + b, page of the sequence
  float ks, vs;       // the block scales
};

template <int HD>
struct DecState {           // one piece of a (sequence, kv head): all rows, log2 domain
  float o[HD / 8][4];       // tile t: dims n * HD/8 + t of column n; [0..1] hi part of row r, [2..3] lo part
  float m, l;               // row r = lane / 4 (l: this lane's keys)
  int E;                    // o counts in units of 2^(E - 14)
};

// One result row set into o: dims [c * HD/4, (c + 1) * HD/4) of row r.
template <int HD>
S2_DEV void store_rows(const Kv8Args& a, int b, int g, int r, int c, const float (&y)[HD / 4]) {
  const int G = a.H / a.Hkv;
  if (r >= a.m * G) return;
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
  // The partials slot(0) .. slot(n - 1), in order: the largest maximum first,
  // so that the loads of the values wait for nothing.
  template <typename F>
  S2_DEV void take(F slot, int n, int R, int r, int c) {
    if (r >= R) return;
#pragma unroll 4
    for (int k = 0; k < n; ++k) m = fmaxf(m, __ldcg(slot(k) + R * HD + 2 * r));
#pragma unroll 2
    for (int k = 0; k < n; ++k) {
      const float* p = slot(k);
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(p + R * HD + 2 * r));
      const float y = ml.x == -INFINITY ? (ml.y == ml.y ? 0.f : ml.y) : ex2(ml.x - m);   // no keys: nothing; NaN stays
      l += ml.y * y;
      const float4* s = reinterpret_cast<const float4*>(p + r * HD + c * (HD / 4));
#pragma unroll
      for (int i = 0; i < HD / 16; ++i) {
        const float4 v = __ldcg(s + i);
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

// The work is the list of all pages in the order (sequence, page), cut into
// equal runs: ragged lengths, one long sequence and many short ones load every
// SM alike.  A run is taken by as many warps as there are kv heads, one head
// each, side by side, so that a page is read whole at about one time (read
// head by head, with 2 KB here and there, the memory gives half: 26 us instead
// of 17 for 65 MB).  Each warp streams its head's part of the pages through
// its own ring in shared memory (one copy brings 16 keys and 16 values) and
// shares no barrier with another.  A sequence that a run holds whole is
// finished by it; one that is cut is joined by the last of its runs to arrive,
// in order, in two levels where there are many.
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
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = blockDim.x;
  const int r = lane >> 2, c = lane & 3;
  const int D = lay.depth, G = a.H / a.Hkv, R = a.m * G;
  const int h = warp % lay.heads;                                  // head within its group
  const unsigned run = blockIdx.x * lay.slices + warp / lay.heads;
  int* first_s = reinterpret_cast<int*>(sm + lay.meta_off);   // pages before sequence b, B + 1 entries
  int* pos_s = first_s + a.B + 1;
  uint8_t* ring = sm + (size_t)warp * D * UB;
  uint4* qst = reinterpret_cast<uint4*>(sm + lay.q_off) + (size_t)warp * R * (HD / 4);
  for (int i = tid; i < kDecWarps * D; i += threads) mbar_init(&bars[i / D][i % D], 1);
  fence_mbar_init();
  pdl_launch_next();
  pdl_wait();

  // pages of each sequence (none for one that is left out), and their sums
  {
    const int per = (a.B + threads - 1) / threads, b0 = tid * per;
    int own = 0;
#pragma unroll 1
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
#pragma unroll 1
    for (int w = 0; w <= warp; ++w) before += scan_s[w];
#pragma unroll 1
    for (int b = b0; b < min(b0 + per, a.B); ++b) first_s[b] += before;
    if (tid == threads - 1) first_s[a.B] = before + own;
    __syncthreads();
  }
#pragma unroll 1
  for (int b = blockIdx.x; b < a.B; b += gridDim.x)
    if (pos_s[b] < 0)
#pragma unroll 1
      for (int i = tid; i < a.m * a.H * HD; i += threads) {
        const size_t at = (size_t)(b * a.m + i / (a.H * HD)) * a.o_ld + i % (a.H * HD);
        if (a.o) a.o[at] = 0.f;
        else a.o16[at] = __float2bfloat16_rn(0.f);
      }
  // units fit 31 bits (the caller refuses more)
  const unsigned P = first_s[a.B], U = P * lay.groups;
  if (U == 0) return;
  const unsigned W = min(gridDim.x * lay.slices, (U + kDecMinPages - 1) / kDecMinPages);
  if (run >= W) return;
  const Cut cut{U / W, U % W};
  const unsigned u0 = cut.start(run);
  const int n = (int)(cut.start(run + 1) - u0);

  // (group, sequence) of unit u
  auto seg_of = [&](unsigned u) {
    const int group = lay.groups > 1 ? u / P : 0;
    u -= group * P;
    int lo = 0;                                 // last b with first page <= u
#pragma unroll 1
    for (int hi = a.B; hi - lo > 1;) {
      const int mid = (lo + hi) >> 1;
      if ((unsigned)first_s[mid] <= u) lo = mid;
      else hi = mid;
    }
    return group * a.B + lo;
  };
  auto seg_start = [&](int s) { return (unsigned)(s / a.B) * P + first_s[s % a.B]; };
  // the unit u0 + t, looked up by lane t % 32
  auto look_up = [&](int t) {
    Unit x{-1, -1, 0, 1.f, 1.f};
    if (t >= n) return x;
    x.seg = seg_of(u0 + t);
    x.j = (int)(u0 + t - seg_start(x.seg));
    const int p = a.table[(size_t)(x.seg % a.B) * a.table_ld + x.j], g = x.seg / a.B * lay.heads + h;
    if (p >= 0 && p < a.n_pages && g < a.Hkv) {
      x.page = p;
      const float* s = a.scale + (size_t)p * 2 * a.Hkv + g;
      x.ks = s[0];
      x.vs = s[a.Hkv];
    }
    return x;
  };
  auto issue = [&](const Unit& x, int t) {      // by the lane that looked it up
    uint64_t* bar = &bars[warp][t % D];
    if (x.page < 0) mbar_arrive(bar);
    else {
      mbar_arrive_expect_tx(bar, UB);
      tma_load_page(ring + (size_t)(t % D) * UB, &map, x.seg / a.B * lay.heads + h, x.page, bar);
    }
  };

  uint32_t qa[KS][4];        // query fragments: {hi, lo} x {dims 4t, 4t+1 | 4t+2, 4t+3}
  float qf = 0.f;            // 2^-(exponent given to row r's query)
  DecState<HD> st;
  int seg = -1, pos = 0, b = 0, g = 0;
  bool nan_new = false;      // a new value row after the first holds a NaN

  // HD/4 lanes take a row, four dims each (the rotation's partners are half
  // a row of lanes apart): whole rows by each load, and the loads of four
  // rows (or eight half ones) in flight at once.  What lane l holds of row i
  // is fragment t = l % KS of lane (i, l / KS); a warp's buffer, XORed
  // against bank conflicts, takes it there.
  constexpr int LPR = HD / 4, RPS = 32 / LPR, ST = 4;    // rows per load, loads at a time
  const int l = lane % LPR, d = 4 * l, dh = d % (HD / 2);
  const bool vec = lay.vec;
  float4 x[ST] = {}, co[ST] = {}, si[ST] = {};
  auto load_rows = [&](int s, int k0) {
    const int b = s % a.B, g = s / a.B * lay.heads + h;
    if (g >= a.Hkv) return;
#pragma unroll
    for (int k = 0; k < ST; ++k) {
      const int i = k0 + k * RPS + lane / LPR;
      x[k] = co[k] = si[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < R) {
        const int p = pos_s[b] + i / G;
        x[k] = load4(a.qkv + (size_t)(b * a.m + i / G) * a.qkv_ld + (size_t)(g * G + i % G) * HD + d, vec);
        co[k] = load4(a.rope_cos + (size_t)p * (HD / 2) + dh, vec);
        si[k] = load4(a.rope_sin + (size_t)p * (HD / 2) + dh, vec);
      }
    }
  };
  // the first rows' loads go ahead of the stream of pages
  load_rows(seg_of(u0), 0);
  Unit cur = look_up(lane);
  Unit nxt = cur;
  if (lane < min(D, n)) issue(cur, lane);

  // The query rows of (sequence, kv head) s; ``load_rows(s, 0)`` came before.
  auto begin = [&](int s) {
    seg = s;
    nan_new = false;
    b = s % a.B;
    g = s / a.B * lay.heads + h;
    pos = pos_s[b];
    st.m = -INFINITY;
    st.l = 0.f;
    st.E = kKv8EMin;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[t][e] = 0.f;
    const float4 gain = load4(a.q_gain + d, vec);
    const float sg = l < LPR / 2 ? -1.f : 1.f;
#pragma unroll 1
    for (int k0 = 0; k0 < R; k0 += ST * RPS) {
      float ss[ST];
      if (k0 > 0) load_rows(s, k0);
#pragma unroll
      for (int k = 0; k < ST; ++k) ss[k] = x[k].x * x[k].x + x[k].y * x[k].y + x[k].z * x[k].z + x[k].w * x[k].w;
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < ST; ++k) ss[k] += __shfl_xor_sync(0xffffffffu, ss[k], o);
#pragma unroll
      for (int k = 0; k < ST; ++k) {
        // log2(e) / sqrt(HD): the softmax runs on powers of two
        const float f = rsqrtf(ss[k] * (1.f / HD) + a.eps) * (HD == 128 ? 0.127517431f : 0.180336880f);
        float4 y = x[k];
        y.x *= f * gain.x;
        y.y *= f * gain.y;
        y.z *= f * gain.z;
        y.w *= f * gain.w;
        const float w0 = __shfl_xor_sync(0xffffffffu, y.x, LPR / 2) * sg;
        const float w1 = __shfl_xor_sync(0xffffffffu, y.y, LPR / 2) * sg;
        const float w2 = __shfl_xor_sync(0xffffffffu, y.z, LPR / 2) * sg;
        const float w3 = __shfl_xor_sync(0xffffffffu, y.w, LPR / 2) * sg;
        y.x = y.x * co[k].x + w0 * si[k].x;
        y.y = y.y * co[k].y + w1 * si[k].y;
        y.z = y.z * co[k].z + w2 * si[k].z;
        y.w = y.w * co[k].w + w3 * si[k].w;
        x[k] = y;
        ss[k] = fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w)));
      }
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < ST; ++k) ss[k] = fmaxf(ss[k], __shfl_xor_sync(0xffffffffu, ss[k], o));
#pragma unroll
      for (int k = 0; k < ST; ++k) {
        const int i = k0 + k * RPS + lane / LPR;
        // the row's largest magnitude to 2^12 .. 2^13: its pair then is good
        // to 2^-22 of each value and 2^-37 of the largest
        const int ex = min(max((int)(__float_as_uint(ss[k]) >> 23) - 127, -100), 100);
        const float up = pow2f(12 - ex);
        const int ex_r = __shfl_sync(0xffffffffu, ex, (r % RPS) * LPR);
        if (r / RPS == k0 / RPS + k) qf = pow2f(ex_r - 12);
        uint4 y;
        split2(x[k].x * up, x[k].y * up, y.x, y.y);
        split2(x[k].z * up, x[k].w * up, y.z, y.w);
        if (i < R) qst[i * LPR + (l ^ ((l / KS) | ((i & 1) << 2)))] = y;
      }
    }
    __syncwarp();
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      uint4 y = make_uint4(0, 0, 0, 0);
      if (r < R) y = qst[r * LPR + ((c * KS + t) ^ (c | ((r & 1) << 2)))];
      qa[t][0] = y.x;
      qa[t][1] = y.y;
      qa[t][2] = y.z;
      qa[t][3] = y.w;
    }
    __syncwarp();
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
#pragma unroll 1
      for (int i = 0; i <= r / G; ++i) {
        const float* v = a.qkv + (size_t)(b * a.m + i) * a.qkv_ld + (size_t)(a.H + a.Hkv + g) * HD + c * (HD / 4);
#pragma unroll
        for (int k = 0; k < HD / 4; ++k)
          if (v[k] != v[k]) x.o[k] = v[k];
      }
    }
  };
  // The end of a piece: stored if it is all of its sequence, else left for,
  // or joined with, the other runs' pieces.
  unsigned* tickets = reinterpret_cast<unsigned*>(a.ws);      // [level][run][2][warp of the run]
  float* parts = reinterpret_cast<float*>(tickets + (size_t)lay.ctas * lay.slices * 4 * lay.heads);
  auto end = [&] {
    if (g >= a.Hkv) return;
    const unsigned s0 = seg_start(seg);
    const int f = (int)cut.of(s0), n = (int)cut.of(s0 + first_s[b + 1] - first_s[b] - 1) - f + 1;
    Join<HD> x;
    piece(x);
    // piece i of the sequence is run f + i's: its last one if i = 0, else its first
    auto at = [&](int i) { return ((size_t)(f + i) * 2 + (i == 0)) * lay.heads + h; };
    int i = (int)run - f, step = 1, per = n;
    if (n > kDecFlat)
      for (per = 4; per * per < n;) ++per;
    while (n > 1) {
      x.put(parts + at(i) * lay.slot_floats, R, r, c);
      __threadfence();
      __syncwarp();
      const int i0 = i / per * per, count = (min(n - i0, per) + step - 1) / step;
      unsigned* ticket = tickets + (step == 1 ? 0 : (size_t)lay.ctas * lay.slices * 2 * lay.heads) + at(i0);
      unsigned got = 0;
      if (lane == 0) got = atomicAdd(ticket, 1u);
      got = __shfl_sync(0xffffffffu, got, 0);
      if (got != (unsigned)(count - 1)) return;
      __threadfence();
      if (lane == 0) *ticket = 0u;
      x = Join<HD>();
      x.take([&](int k) { return parts + at(i0 + k * step) * lay.slot_floats; }, count, R, r, c);
      if (per >= n) break;
      __syncwarp();          // all lanes have read the slot that is written next
      i = i0;
      step = per;
      per = n;
    }
    x.finish();
    store_rows<HD>(a, b, g, r, c, x.o);
  };

  // One new key (normed, rotated) and value, lane l taking dims l + 32 i.
  constexpr int N = HD / 32;
  float k[N], v[N];
  auto row = [&](int p) {
    const float* x = a.qkv + (size_t)(b * a.m + p - pos) * a.qkv_ld + (size_t)(a.H + g) * HD;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = x[(size_t)a.Hkv * HD + lane + 32 * i];
    const KeyRow<HD> y = key_row_call<HD>(x, a.k_gain, a.rope_cos + (size_t)p * (HD / 2),
                                          a.rope_sin + (size_t)p * (HD / 2), a.eps, lane);
#pragma unroll
    for (int i = 0; i < N; ++i) k[i] = y.v[i];
  };
  // New rows of this page into its shared-memory copy and to the pool; the
  // page's last new row is in k, v already.
  auto append = [&](uint8_t* blk, int page, int j, int& ke, int& ve) {
    const int first = max(pos, j * kKv8Page), last = min(pos + a.m, (j + 1) * kKv8Page);
    const int had = first - j * kKv8Page, rows = last - j * kKv8Page;
    float mk = abs_max(k, 0.f), mv = abs_max(v, 0.f);
#pragma unroll 1
    for (int p = last - 2; p >= first; --p) {
      row(p);
      mk = abs_max(k, mk);
      mv = abs_max(v, mv);
    }
    const int ko = had ? ke : kKv8EMin, vo = had ? ve : kKv8EMin;
    ke = max(ko, kv8_exponent(warp_max(mk)));
    ve = max(vo, kv8_exponent(warp_max(mv)));
    const bool grew_k = had && ke > ko, grew_v = had && ve > vo;
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
      uint8_t* x = blk + t * (kKv8Page * HD);
      const float by = t ? pow2f(vo - ve) : pow2f(ko - ke);
      if (t ? grew_v : grew_k)
#pragma unroll 1
        for (int i = lane; i < had * HD / 16; i += 32) {
          uint4* w = reinterpret_cast<uint4*>(x + unit_off<HD>(i / (HD / 16), i % (HD / 16)));
          uint4 y = *w;
          y.x = e4m3_rescale4(y.x, by);
          y.y = e4m3_rescale4(y.y, by);
          y.z = e4m3_rescale4(y.z, by);
          y.w = e4m3_rescale4(y.w, by);
          *w = y;
        }
    }
    uint8_t* xv = blk + kKv8Page * HD;
#pragma unroll 1
    for (int i = rows * HD / 16 + lane; i < HD; i += 32)   // rows behind the last one: their weight is 0, not their bytes
      *reinterpret_cast<uint4*>(xv + unit_off<HD>(i / (HD / 16), i % (HD / 16))) = make_uint4(0, 0, 0, 0);
    const float fk = pow2f(-ke), fv = pow2f(-ve);
#pragma unroll 1
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
    fence_proxy_async();     // before the stores below, so as not to wait for them
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
      uint8_t* out = a.kv + (((size_t)page * 2 + t) * a.Hkv + g) * (kKv8Page * HD);
      const uint8_t* x = blk + t * (kKv8Page * HD);
#pragma unroll 1
      for (int i = ((t ? grew_v : grew_k) ? 0 : had) * HD / 16 + lane; i < rows * HD / 16; i += 32)
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
#pragma unroll 1
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
      any = __any_sync(0xffffffffu, any);
      if (any) fence_proxy_async();
      nan_new = nan_new || any;
    }
    __syncwarp();
  };

#pragma unroll 1
  for (int t = 0;; ++t) {
    const int src = t & 31;
    if (src == 0 && t > 0) cur = nxt;
    if (src == 0 && t + 32 < n) nxt = look_up(t + 32 + lane);
    const int page = __shfl_sync(0xffffffffu, cur.page, src);
    const int sg = t < n ? __shfl_sync(0xffffffffu, cur.seg, src) : -1;
    const int j = __shfl_sync(0xffffffffu, cur.j, src);
    if (sg != seg) {
      if (seg >= 0) end();
      if (sg < 0) break;
      if (t > 0) load_rows(sg, 0);
      begin(sg);
    }
    if (sg < 0) break;
    const bool tail = (j + 1) * kKv8Page > pos;
    if (tail && page >= 0) row(min(pos + a.m, (j + 1) * kKv8Page) - 1);
    bool ok = mbar_wait(&bars[warp][t % D], (uint32_t)(t / D) & 1u, nullptr);
    ok = __all_sync(0xffffffffu, ok) && page >= 0;
    if (ok) {
      uint8_t* blk = ring + (size_t)(t % D) * UB;
      int ke = kv8_scale_exp(__shfl_sync(0xffffffffu, cur.ks, src));
      int ve = kv8_scale_exp(__shfl_sync(0xffffffffu, cur.vs, src));
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
  }
}

int num_sms() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 1;
}

DecLayout dec_layout(int B, int R, int Hkv, int hd) {
  DecLayout l;
  l.ctas = num_sms();
  l.groups = (Hkv + kDecWarps - 1) / kDecWarps;
  l.heads = (Hkv + l.groups - 1) / l.groups;
  l.slices = kDecWarps / l.heads;
  l.slot_floats = R * hd + 2 * R + (2 * R) % 4;
  const int warps = l.heads * l.slices, q = warps * R * hd * 4, unit = 2 * kKv8Page * hd;
  const int room = kDecSmem - 1024 - 2048 - q - (2 * B + 1) * 4;   // alignment, static
  l.depth = room / (warps * unit);
  if (l.depth > kDecMaxDepth) l.depth = kDecMaxDepth;
  l.q_off = warps * l.depth * unit;
  l.meta_off = l.q_off + q;
  l.vec = 0;
  return l;
}

}  // namespace

size_t kv8_decode_ws_bytes(int B, int m, int H, int Hkv, int hd) {
  const DecLayout l = dec_layout(B, m * (H / Hkv), Hkv, hd);
  return (size_t)l.ctas * l.slices * 2 * l.heads * (2 + l.slot_floats) * 4;
}

cudaError_t launch_kv8_decode(const Kv8Args& a, cudaStream_t st) {
  CUtensorMap map;
  if (!tma_map_kv8(&map, a.kv, a.n_pages, a.Hkv, a.hd)) return cudaErrorNotSupported;
  DecLayout l = dec_layout(a.B, a.m * (a.H / a.Hkv), a.Hkv, a.hd);
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
  cfg.blockDim = dim3(l.heads * l.slices * 32);
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
