// Decode attention over the 8-bit KV cache: q/k norm and RoPE, append of the
// new rows, attention of all rows of a (sequence, kv head), one launch.
#include <cuda.h>

#include <type_traits>

#include "kv8_common.cuh"
#include "tc_common.cuh"
#include "tma_map.h"

namespace s2 {

namespace {

constexpr int kDecWarps = 8;       // most warps of a CTA
constexpr int kDecMaxDepth = 8;
constexpr int kDecSmem = 227 * 1024;
constexpr int kDecFlight = 128 * 1024;
constexpr int kDecPages = 2;       // pages of a unit of work
// Units of a run at least: a cut costs a joining, about as long as a few units
// (one sequence of 1,090 tokens: 15.7 us with 3, 17.7 us with 6).
constexpr int kDecMinUnits = 3;
// What starting and ending a sequence costs, in units: the cut counts it (128
// sequences of up to 1,700 tokens: 57.8 us with 2, 56.0 us with 4; 32 of about
// 1,000: 27.6 and 25.9 us).
constexpr int kDecSeqUnits = 4;
// Pieces that are joined at once, one per lane; more are joined in two levels
// of about the square root each.
constexpr int kDecFlat = 32;
constexpr int kDecMaxRuns = kDecFlat * kDecFlat;

struct DecLayout {
  int groups, heads, slices;   // kv heads in groups of ``heads``; a CTA has heads x slices warps
  int depth;                   // units in flight per warp
  int buf_off, meta_off;       // bytes
  int buf;                     // a warp's buffer: its rows of HD floats, 4 at least
  int slot_floats;             // one partial: R rows of HD values, then (m, l) of each
  int ctas;
  int parts_off;               // of the partials in the workspace, bytes
  int o_vec;                   // rows of o on 16-byte (bf16: 8-byte) boundaries
  unsigned inv_g;              // i / G = i * inv_g >> 16 for rows i
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

// Four consecutive floats, on a 16-byte boundary if VEC.
template <bool VEC>
S2_DEV float4 load4(const float* p) {
  return VEC ? *reinterpret_cast<const float4*>(p) : make_float4(p[0], p[1], p[2], p[3]);
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

// What a warp knows of one unit: two pages of a sequence, for one kv head.
struct Unit {
  int seg, j;              // group * B + b, the sequence's page that comes first
  int page[kDecPages];     // page ids (-1: none, or not to be followed)
  float ks[kDecPages], vs[kDecPages];   // the block scales
};
// Flags that the pages are there, and the exponents + 64 of their scales.
struct UnitBits {
  uint32_t exps;           // K, V of the first page, K, V of the second
  uint32_t there;
};

// Weights carry 2^kDecBias, and the running maximum may lag by kDecLag, so that a
// weight of at most 2^14 fits f16 and the accumulators are rescaled rarely.  Over
// 2^20 keys the sums stay below 2^60 (l) and 2^43 (o), and l above 2^-32.
constexpr int kDecBias = 6, kDecLag = 8;
// A page whose value scale lies more than kDecFar binades below the largest one
// met is looked at row by row: where its largest weight x scale is that far below
// the row's, o is lifted for its products by up to 2^kDecLift (to 2^107 at most).
constexpr int kDecFar = 10, kDecLift = 64;

template <int HD>
struct DecState {           // one piece of a (sequence, kv head): all rows, log2 domain
  float o[HD / 8][4];       // tile t: dims n * HD/8 + t of column n; [0..1] hi part of row r, [2..3] lo part
  // Row r = lane / 4.  m: the largest score + exponent of its value block's scale
  // so far, or up to kDecLag below; l (this lane's keys) sums 2^(score - m), and o
  // 2^(score + exponent - m + kDecBias) times the e4m3 values.
  float m, l;
  int e;                    // largest exponent of a value scale so far
};

// The work is the list of all pages in the order (sequence, page), cut into
// equal runs: ragged lengths, one long sequence and many short ones load every
// SM alike.  A run is taken by as many warps as there are kv heads, one head
// each, side by side, so that a page is read whole at about one time (read
// head by head, with 2 KB here and there, the memory gives two thirds: the
// loop over 65 MB then took 26 us, and 17 side by side).  Each warp streams
// its head's part of the pages through its own ring in shared memory (one copy
// brings 16 keys and 16 values) and shares no barrier with another.  A
// sequence that a run holds whole is finished by it; one that is cut is joined
// by the last of its runs to arrive, in order, in two levels where there are
// many.
//
// Products: mma.sync m16n8k16 with the up to 8 query rows (new rows x heads
// of the kv head) as f16 hi parts in rows 0..7 and lo parts in rows 8..15, so
// the pair costs nothing; e4m3 bytes become f16 in registers.  The order of
// dims in Q K^T and of dims in the output is free, and is chosen such that
// each lane's bytes are contiguous: lane (n, c) takes dims c * HD/4 .. of key
// n, and dims n * HD/8 .. of the values of keys 2c, 2c + 1, 2c + 8, 2c + 9.
// The block scale of K multiplies the scores; the one of V, 2^e, goes into the
// weights, and the running maximum is that of score + e.  So a weight in f16 is
// held against the largest weight x scale among the keys that its row sees: a
// block of large values that has next to no weight takes no bits from the
// others, and keeps its own where weight x scale counts (with a maximum of the
// scores and another of e, weights of 2^-33 on values of 2^48 were lost).  A
// scale bounds its block's values, and a row may see none of the large ones:
// pages far below the largest scale are added with o lifted to them.
//
// Bound by memory where the keys are many: 128 sequences of 200 to 1,700 tokens,
// 8 heads of 128 (250 MB): 56.0 us, 4.5 TB/s over all, 6 TB/s in the loop; 32 of
// 900 to 1,090 (65 MB): 25.9 us, of which a start of 1.7 us and round trips of
// half a microsecond each (queries, append, ticket, join) with the tail of the
// joins are more than half.  mma.sync, not tcgen05: with at most 8 rows its tile of
// 128 would be empty, and the tensor pipe is 17 % busy as it is.
template <int HD, bool VEC>
__global__ void __launch_bounds__(kDecWarps * 32, 1)
kv8_decode_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ Kv8Args a,
                  const __grid_constant__ DecLayout lay) {
  constexpr int NT = HD / 8;              // output tiles of 8 dims
  constexpr int KS = HD / 16;             // k-steps of the scores
  constexpr int PB = 2 * kKv8Page * HD;   // bytes of a page's part: 16 keys, 16 values
  constexpr int UB = kDecPages * PB;
  extern __shared__ __align__(1024) uint8_t raw[];
  uint8_t* sm = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;
  __shared__ __align__(8) uint64_t bars[kDecWarps][kDecMaxDepth];
  __shared__ int scan_s[kDecWarps + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = blockDim.x;
  const int r = lane >> 2, c = lane & 3;
  const int D = lay.depth, G = a.H / a.Hkv, R = a.m * G, rt = r * lay.inv_g >> 16;   // row r: new row rt
  const int h = warp % lay.heads;                                  // head within its group
  const unsigned run = blockIdx.x * lay.slices + warp / lay.heads;
  int* first_s = reinterpret_cast<int*>(sm + lay.meta_off);   // units before sequence b, B + 1 entries
  int* pos_s = first_s + a.B + 1;
  uint8_t* ring = sm + (size_t)warp * D * UB;
  float* buf = reinterpret_cast<float*>(sm + lay.buf_off + warp * lay.buf);
  for (int i = tid; i < kDecWarps * D; i += threads) mbar_init(&bars[i / D][i % D], 1);
  fence_mbar_init();
  pdl_launch_next();
  pdl_wait();

  // units of each sequence (none for one that is left out; kDecSeqUnits more
  // than it has, which no page stands for), and their sums
  auto units_at = [&](int p) { return (p + a.m + kDecPages * kKv8Page - 1) / (kDecPages * kKv8Page); };
  {
    const int per = (a.B + threads - 1) / threads, b0 = tid * per;
    int own = 0;
#pragma unroll 1
    for (int b = b0; b < min(b0 + per, a.B); ++b) {
      const int p = a.pos[b];
      const bool in = p >= 0 && p <= a.max_pos - a.m;
      pos_s[b] = in ? p : -1;
      first_s[b] = own;
      own += in ? units_at(p) + kDecSeqUnits : 0;
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
      for (int t = 0; t < a.m; ++t)
#pragma unroll 1
        for (int i = tid; i < a.H * HD; i += threads) {
          const size_t at = (size_t)(b * a.m + t) * a.o_ld + i;
          if (a.o) a.o[at] = 0.f;
          else a.o16[at] = __float2bfloat16_rn(0.f);
        }
  // units fit 31 bits (the caller refuses more)
  const unsigned P = first_s[a.B], U = P * lay.groups;
  if (U == 0) return;
  const unsigned W = min(min(gridDim.x * lay.slices, kDecMaxRuns), (U + kDecMinUnits - 1) / kDecMinUnits);
  if (run >= W) return;
  const Cut cut{U / W, U % W};
  const unsigned u0 = cut.start(run);
  const int n = (int)(cut.start(run + 1) - u0);

  // A (group, sequence) is named by group << 16 | b.
  auto seg_start = [&](int s) { return (unsigned)(s >> 16) * P + first_s[s & 0xffff]; };
  auto head_of = [&](int s) { return (s >> 16) * lay.heads + h; };
  // the unit u0 + t, looked up by lane t % 32
  auto look_up = [&](int t) {
    // a page that is not there has the least scale, which no other is far below
    const float least = pow2f(kKv8EMin);
    Unit x{-1, 0, {-1, -1}, {least, least}, {least, least}};
    if (t >= n) return x;
    unsigned u = u0 + t;
    int group = 0, b = 0;                       // last b with first unit <= u
    for (; u >= P; u -= P) ++group;
#pragma unroll 1
    for (int hi = a.B; hi - b > 1;) {
      const int mid = (b + hi) >> 1;
      if ((unsigned)first_s[mid] <= u) b = mid;
      else hi = mid;
    }
    x.j = kDecPages * (int)(u - first_s[b]);
    if (x.j >= kDecPages * units_at(pos_s[b])) {
      x.seg = -2;                               // none
      return x;
    }
    x.seg = group << 16 | b;
    const int g = head_of(x.seg), pages = (pos_s[b] + a.m + kKv8Page - 1) / kKv8Page;
    const int* row = a.table + (size_t)b * a.table_ld + x.j;
#pragma unroll
    for (int i = 0; i < kDecPages; ++i) {
      const int p = x.j + i < pages ? row[i] : -1;
      x.page[i] = p >= 0 && p < a.n_pages && g < a.Hkv ? p : -1;
    }
#pragma unroll
    for (int i = 0; i < kDecPages; ++i)
      if (x.page[i] >= 0) {
        const float* s = a.scale + (size_t)x.page[i] * 2 * a.Hkv + g;
        x.ks[i] = s[0];
        x.vs[i] = s[a.Hkv];
      }
    return x;
  };
  auto bits_of = [&](const Unit& x) {           // waits for the scales
    return UnitBits{(uint32_t)(kv8_scale_exp(x.ks[0]) + 64) | (uint32_t)(kv8_scale_exp(x.vs[0]) + 64) << 8 |
                        (uint32_t)(kv8_scale_exp(x.ks[1]) + 64) << 16 | (uint32_t)(kv8_scale_exp(x.vs[1]) + 64) << 24,
                    (x.page[0] >= 0 ? 1u : 0u) | (x.page[1] >= 0 ? 2u : 0u)};
  };
  auto issue = [&](const Unit& x, int slot) {   // by the lane that looked it up
    uint64_t* bar = &bars[warp][slot];
    const int there = (x.page[0] >= 0) + (x.page[1] >= 0);
    if (!there) mbar_arrive(bar);
    else {
      mbar_arrive_expect_tx(bar, there * PB);
#pragma unroll
      for (int i = 0; i < kDecPages; ++i)
        if (x.page[i] >= 0) tma_load_page(ring + slot * UB + i * PB, &map, head_of(x.seg), x.page[i], bar);
    }
  };

  uint32_t qa[KS][4];        // query fragments: {hi, lo} x {dims 4t, 4t+1 | 4t+2, 4t+3}
  uint32_t polls = a.polls;  // of a wait; 1 after one that gave up
  float qf = 0.f;            // 2^-(exponent given to row r's query)
  DecState<HD> st;
  int seg = -1, pos = 0, b = 0, g = 0;
  bool nan_new = false;      // a new value row after the first holds a NaN

  // The query rows of (group, sequence) s.  HD/4 lanes take a row, four dims
  // each (the rotation's partners are half a row of lanes apart): whole rows by
  // each load, and the loads of four rows (or eight half ones) in flight at
  // once.  What lane l holds of row i is fragment t = l % KS of lane (i, l / KS);
  // a warp's buffer, XORed against bank conflicts, takes it there.
  auto begin = [&](int s) {
    seg = s;
    nan_new = false;
    b = s & 0xffff;
    g = head_of(s);
    pos = pos_s[b];
    st.m = -INFINITY;
    st.e = kKv8EMin;
    st.l = polls > 1 ? 0.f : __int_as_float(0x7fffffff);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[t][e] = 0.f;
#pragma unroll
    for (int t = 0; t < KS; ++t) qa[t][0] = qa[t][1] = qa[t][2] = qa[t][3] = 0u;
    if (g >= a.Hkv) return;
    constexpr int LPR = HD / 4, RPS = 32 / LPR, ST = 4;    // rows per load, loads at a time
    const int l = lane % LPR, d = 4 * l;
    const float4 gain = load4<VEC>(a.q_gain + d);
    const float sg = l < LPR / 2 ? -1.f : 1.f;
    const float* rows = a.qkv + (size_t)b * a.m * a.qkv_ld + (size_t)g * G * HD + d;
    const size_t turn = (size_t)pos * (HD / 2) + d % (HD / 2);
    uint4* qst = reinterpret_cast<uint4*>(buf);
    __syncwarp();
#pragma unroll 1
    for (int k0 = 0; k0 < R; k0 += ST * RPS) {
      float4 x[ST], co[ST], si[ST];
      float ss[ST];
#pragma unroll
      for (int k = 0; k < ST; ++k) {
        const int i = min(k0 + k * RPS + lane / LPR, R - 1), t = i * lay.inv_g >> 16;
        x[k] = load4<VEC>(rows + (size_t)t * a.qkv_ld + (i - t * G) * HD);
        co[k] = load4<VEC>(a.rope_cos + turn + t * (HD / 2));
        si[k] = load4<VEC>(a.rope_sin + turn + t * (HD / 2));
      }
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
        const int i = k * RPS + lane / LPR;
        // the row's largest magnitude to 2^12 .. 2^13: its pair then is good
        // to 2^-22 of each value and 2^-37 of the largest
        const int ex = min(max((int)(__float_as_uint(ss[k]) >> 23) - 127, -100), 100);
        const float up = pow2f(12 - ex);
        const int ex_r = __shfl_sync(0xffffffffu, ex, (r % RPS) * LPR);
        if (r / RPS == k0 / RPS + k) qf = pow2f(ex_r - 12);
        uint4 y;
        split2(x[k].x * up, x[k].y * up, y.x, y.y);
        split2(x[k].z * up, x[k].w * up, y.z, y.w);
        qst[i * LPR + (l ^ ((l / KS) | ((i & 1) << 2)))] = y;
      }
      __syncwarp();
      if (r >= k0 && r < min(k0 + ST * RPS, R))
#pragma unroll
        for (int t = 0; t < KS; ++t) {
          const uint4 y = qst[(r - k0) * LPR + ((c * KS + t) ^ (c | ((r & 1) << 2)))];
          qa[t][0] = y.x;
          qa[t][1] = y.y;
          qa[t][2] = y.z;
          qa[t][3] = y.w;
        }
      __syncwarp();
    }
  };

  // The end of a piece: into o if it is all of its sequence, else into the
  // run's slot 1 (a sequence's first piece) or 0 (any other) for the joining.
  unsigned* tickets = reinterpret_cast<unsigned*>(a.ws);      // [level][run][slot][warp of the run]
  float* parts = reinterpret_cast<float*>(static_cast<char*>(a.ws) + lay.parts_off);
  int open[2] = {-1, -1};
  // A sequence's pieces are those of the runs f .. f + n - 1; ``per`` of them are
  // joined at the first level.
  struct Pieces {
    int f, n, per;
  };
  auto pieces_of = [&](int s) {
    const unsigned s0 = seg_start(s), s1 = s0 + units_at(pos_s[s & 0xffff]);
    Pieces x;
    x.f = (int)cut.of(s0);
    x.per = x.n = (int)cut.of(s1 - 1) - x.f + 1;
    if (x.n > kDecFlat)
      for (x.per = 4; x.per * x.per < x.n;) ++x.per;
    return x;
  };
  // Slot (and ticket) of piece i: its run's slot 1 if it is the first one.
  auto at = [&](const Pieces& x, int i) { return ((size_t)(x.f + i) * 2 + (i == 0)) * lay.heads + h; };
  // The number (lane 0) of those that came to the first level's group before.
  unsigned came[2] = {0, 0};
  auto arrive = [&](int s) {
    __threadfence();
    __syncwarp();
    const Pieces x = pieces_of(s);
    const int i = (int)run - x.f;
    return lane == 0 ? atomicAdd(tickets + at(x, i - i % x.per), 1u) : 0u;
  };
  // Four values of row i of kv head g of sequence b, at dim d, to o or a slot.
  auto put = [&](float* slot, int b, int g, int i, int d, float4 y) {
    if (slot) {
      *reinterpret_cast<float4*>(slot + i * HD + d) = y;
      return;
    }
    const int t = i * lay.inv_g >> 16;
    const size_t at = (size_t)(b * a.m + t) * a.o_ld + (size_t)(g * G + i - t * G) * HD + d;
    if (a.o) {
      if (lay.o_vec) {
        *reinterpret_cast<float4*>(a.o + at) = y;
      } else {
        a.o[at] = y.x;
        a.o[at + 1] = y.y;
        a.o[at + 2] = y.z;
        a.o[at + 3] = y.w;
      }
    } else {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x, y.y), hi = __floats2bfloat162_rn(y.z, y.w);
      if (lay.o_vec) {
        *reinterpret_cast<uint2*>(a.o16 + at) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      } else {
        a.o16[at] = lo.x;
        a.o16[at + 1] = lo.y;
        a.o16[at + 2] = hi.x;
        a.o16[at + 3] = hi.y;
      }
    }
  };
  auto end = [&] {
    if (g >= a.Hkv) return;
    const unsigned s0 = seg_start(seg), s1 = s0 + units_at(pos);
    const bool whole = s0 >= u0 && s1 <= u0 + n;
    const int k = s0 >= u0;
    float* slot = whole ? nullptr : parts + (((size_t)run * 2 + k) * lay.heads + h) * lay.slot_floats;
    st.l += __shfl_xor_sync(0xffffffffu, st.l, 1);
    st.l += __shfl_xor_sync(0xffffffffu, st.l, 2);
    float f = pow2f(-kDecBias);
    if (whole) f = st.l == 0.f ? 0.f : f * (1.f / st.l);
    __syncwarp();
    if (r < R) {
      float4* y = reinterpret_cast<float4*>(buf + r * HD + c * (HD / 4));
#pragma unroll
      for (int t = 0; t < NT; t += 4) {
        y[t / 4] = make_float4((st.o[t][0] + st.o[t][2]) * f, (st.o[t + 1][0] + st.o[t + 1][2]) * f,
                               (st.o[t + 2][0] + st.o[t + 2][2]) * f, (st.o[t + 3][0] + st.o[t + 3][2]) * f);
        y[NT / 4 + t / 4] = make_float4((st.o[t][1] + st.o[t][3]) * f, (st.o[t + 1][1] + st.o[t + 1][3]) * f,
                                        (st.o[t + 2][1] + st.o[t + 2][3]) * f, (st.o[t + 3][1] + st.o[t + 3][3]) * f);
      }
      if (slot && c == 0) *reinterpret_cast<float2*>(slot + R * HD + 2 * r) = make_float2(st.m, st.l);
    }
    __syncwarp();
    if (nan_new) {        // the rows that see a new value's NaN get it back
#pragma unroll 1
      for (int i = lane; i < R * HD; i += 32)
#pragma unroll 1
        for (int t = 0; t <= (int)(i / HD * lay.inv_g >> 16); ++t) {
          const float v = a.qkv[(size_t)(b * a.m + t) * a.qkv_ld + (size_t)(a.H + a.Hkv + g) * HD + i % HD];
          if (v != v) buf[i] = v;
        }
      __syncwarp();
    }
#pragma unroll 1
    for (int q = 4 * lane; q < R * HD; q += 128)
      put(slot, b, g, q / HD, q % HD, *reinterpret_cast<const float4*>(buf + q));
    if (!whole) {
      // a ticket at once: what is asked of it is looked at after the run, when
      // the pieces before this one have come, most likely, and join
      const unsigned c = arrive(seg);
      if (k) {
        open[1] = seg;
        came[1] = c;
      } else {
        open[0] = seg;
        came[0] = c;
      }
    }
  };
  // After the run: of each open piece's group the last to arrive joins.
  auto join = [&] {
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
      const int s = k ? open[1] : open[0];
      if (s < 0) continue;
      const Pieces x = pieces_of(s);
      const int n = x.n;
      int per = x.per, step = 1, i0 = (int)run - x.f;
      unsigned got = k ? came[1] : came[0];
#pragma unroll 1
      for (;;) {
        i0 -= i0 % per;
        const int count = (min(n - i0, per) + step - 1) / step;
        unsigned* ticket = tickets + (step == 1 ? 0 : (size_t)lay.ctas * lay.slices * 2 * lay.heads) + at(x, i0);
        if (step > 1 && lane == 0) got = atomicAdd(ticket, 1u);
        if (__shfl_sync(0xffffffffu, got, 0) != (unsigned)(count - 1)) break;
        __threadfence();
        if (lane == 0) *ticket = 0u;
        const bool done = per >= n;
        float* slot = done ? nullptr : parts + at(x, i0) * lay.slot_floats;
        // 128 values a step (a row of 128, two of 64); all steps of four pieces,
        // and of eight if there are few rows, in flight at once, the first ones
        // together with the maxima: a round trip is half a microsecond
        auto gather = [&](auto steps, auto batch) {
          constexpr int ST = decltype(steps)::value, Q = decltype(batch)::value, RPS = 128 / HD, NR = ST * RPS;
          const int row = 4 * lane / HD;             // row within a step
          float4 v4[Q][ST], o[ST];
          auto load = [&](int q0) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
              const float* v = parts + at(x, i0 + min(q0 + q, count - 1) * step) * lay.slot_floats + 4 * lane;
#pragma unroll
              for (int i = 0; i < ST; ++i) {
                v4[q][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (q0 + q < count && i * RPS + row < R) v4[q][i] = __ldcg(reinterpret_cast<const float4*>(v + i * 128));
              }
            }
          };
          // piece q's maxima and sums in lane q, its weight for row i in w[i]
          float w[NR], inv[NR], m[NR];
          const float* ml = parts + at(x, i0 + min(lane, count - 1) * step) * lay.slot_floats + R * HD;
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            float2 v = make_float2(-INFINITY, 0.f);
            if (i < R && lane < count) v = __ldcg(reinterpret_cast<const float2*>(ml + 2 * i));
            m[i] = w[i] = v.x;
            inv[i] = v.y;
          }
          load(0);
#pragma unroll
          for (int k = 16; k > 0; k >>= 1)
#pragma unroll
            for (int i = 0; i < NR; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], k));
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            // no keys: nothing; NaN stays
            w[i] = w[i] == -INFINITY ? (inv[i] == inv[i] ? 0.f : inv[i]) : ex2(w[i] - m[i]);
            inv[i] *= w[i];
          }
#pragma unroll
          for (int k = 16; k > 0; k >>= 1)
#pragma unroll
            for (int i = 0; i < NR; ++i) inv[i] += __shfl_xor_sync(0xffffffffu, inv[i], k);
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            if (slot && lane == 0 && i < R) *reinterpret_cast<float2*>(slot + R * HD + 2 * i) = make_float2(m[i], inv[i]);
            inv[i] = !done ? 1.f : inv[i] == 0.f ? 0.f : 1.f / inv[i];
          }
#pragma unroll
          for (int i = 0; i < ST; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
          for (int q0 = 0;;) {
#pragma unroll
            for (int q = 0; q < Q; ++q)
#pragma unroll
              for (int i = 0; i < ST; ++i) {
                float y = __shfl_sync(0xffffffffu, w[i * RPS], (q0 + q) & 31);
                if (RPS == 2) {
                  const float y2 = __shfl_sync(0xffffffffu, w[i * RPS + RPS - 1], (q0 + q) & 31);
                  y = row ? y2 : y;
                }
                o[i].x += v4[q][i].x * y;
                o[i].y += v4[q][i].y * y;
                o[i].z += v4[q][i].z * y;
                o[i].w += v4[q][i].w * y;
              }
            q0 += Q;
            if (q0 >= count) break;
            load(q0);
          }
          __syncwarp();      // all lanes have read the slot that is written below
#pragma unroll
          for (int i = 0; i < ST; ++i) {
            const float y = row ? inv[i * RPS + RPS - 1] : inv[i * RPS];
            if (i * RPS + row < R)
              *reinterpret_cast<float4*>(buf + i * 128 + 4 * lane) =
                  make_float4(o[i].x * y, o[i].y * y, o[i].z * y, o[i].w * y);
          }
        };
        if (R * HD <= 512) gather(std::integral_constant<int, 4>(), std::integral_constant<int, 8>());
        else gather(std::integral_constant<int, 8 * HD / 128>(), std::integral_constant<int, 4>());
        __syncwarp();
#pragma unroll 1
        for (int q = 4 * lane; q < R * HD; q += 128)
          put(slot, s & 0xffff, head_of(s), q / HD, q % HD, *reinterpret_cast<const float4*>(buf + q));
        if (done) break;
        __threadfence();
        __syncwarp();
        step = per;
        per = n;
      }
    }
  };

  // New rows of this page into its shared-memory copy and to the pool.
  auto append = [&](uint8_t* blk, int page, int j, int& ke, int& ve) {
    constexpr int N = HD / 32;
    const int first = max(pos, j * kKv8Page), last = min(pos + a.m, (j + 1) * kKv8Page);
    const int had = first - j * kKv8Page, rows = last - j * kKv8Page, cnt = last - first;
    const int ko = had ? ke : kKv8EMin, vo = had ? ve : kKv8EMin;
    uint8_t* xv = blk + kKv8Page * HD;
    float k[N], v[N], mk = 0.f, mv = 0.f;
    bool grew_k = false, grew_v = false, nan = false;
    // two passes over the new rows, from the last to the first for their
    // largest magnitudes, and back to be rounded
#pragma unroll 1
    for (int it = 0; it < 2 * cnt; ++it) {
      const int p = it < cnt ? last - 1 - it : first + it - cnt;
      if (it != cnt) {
        const float* x = a.qkv + (size_t)(b * a.m + p - pos) * a.qkv_ld + (size_t)(a.H + g) * HD;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = x[(size_t)a.Hkv * HD + lane + 32 * i];
        kv8_key_row<HD>(x, a.k_gain, a.rope_cos + (size_t)p * (HD / 2), a.rope_sin + (size_t)p * (HD / 2), a.eps, lane,
                        k);
      }
      if (it < cnt) {
        mk = abs_max(k, mk);
        mv = abs_max(v, mv);
        continue;
      }
      if (it == cnt) {
        ke = max(ko, kv8_exponent(warp_max(mk)));
        ve = max(vo, kv8_exponent(warp_max(mv)));
        grew_k = had && ke > ko;
        grew_v = had && ve > vo;
#pragma unroll 1
        for (int t = 0; t < 2; ++t)
          if (t ? grew_v : grew_k) {
            const float by = t ? pow2f(vo - ve) : pow2f(ko - ke);
#pragma unroll 1
            for (int i = lane; i < had * HD / 4; i += 32) {
              uint32_t* w = reinterpret_cast<uint32_t*>(blk + t * (kKv8Page * HD) +
                                                        unit_off<HD>(i / (HD / 4), i % (HD / 4) / 4)) + i % 4;
              *w = e4m3_rescale4(*w, by);
            }
          }
        // rows behind the last one: their weight is 0, not their bytes
#pragma unroll 1
        for (int i = rows * HD / 16 + lane; i < HD; i += 32)
          *reinterpret_cast<uint4*>(xv + unit_off<HD>(i / (HD / 16), i % (HD / 16))) = make_uint4(0, 0, 0, 0);
      }
      const float fk = pow2f(-ke), fv = pow2f(-ve);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int d = lane + 32 * i;
        const uint32_t to = unit_off<HD>(p % kKv8Page, d >> 4) + (d & 15);
        blk[to] = (uint8_t)e4m3x2(k[i] * fk, 0.f);
        xv[to] = (uint8_t)e4m3x2(v[i] * fv, 0.f);
        nan = nan || v[i] != v[i];
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
    // A NaN among several new rows' values must not reach the rows before it
    // through 0 * NaN: it leaves the copy, and ``end`` gives it back.
    if (a.m > 1 && __any_sync(0xffffffffu, nan)) {
      nan_new = true;
#pragma unroll 1
      for (int i = had * HD + lane; i < rows * HD; i += 32) {
        uint8_t* w = xv + unit_off<HD>(i / HD, i % HD / 16) + i % 16;
        if ((*w & 0x7f) == 0x7f) *w = 0;
      }
      __syncwarp();
      fence_proxy_async();
    }
    __syncwarp();
  };

  auto lift_by = [&](int e) {
    const float y = pow2f(e);
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
      for (int k = 0; k < 4; ++k) st.o[q][k] *= y;
  };

  Unit cur = look_up(lane), nxt = cur;
  if (lane < min(D, n)) issue(cur, lane);
  UnitBits bits{0u, 0u};
  int slot = 0;
  uint32_t phase = 0;
  int issued = n;            // units that were copied, or will be
#pragma unroll 1
  for (int t = 0;; ++t) {
    const int src = t & 31;
    if (src == 0) {
      if (t > 0) cur = nxt;
      bits = bits_of(cur);
      if (t + 32 < n) nxt = look_up(t + 32 + lane);
    }
    const int sg = t < n ? __shfl_sync(0xffffffffu, cur.seg, src) : -1;
    if (sg != seg && sg != -2) {
      if (seg >= 0) end();
      if (sg >= 0) begin(sg);
    }
    if (t >= n) break;
    const int j = __shfl_sync(0xffffffffu, cur.j, src);   // a unit that is none has no pages either
    const uint32_t exps = __shfl_sync(0xffffffffu, bits.exps, src);
    const uint32_t there = __shfl_sync(0xffffffffu, bits.there, src);
    uint8_t* blk = ring + slot * UB;
    const bool came = __all_sync(0xffffffffu, mbar_wait(&bars[warp][slot], phase, nullptr, polls));
    if (!came) {              // gave up: no more copies, outputs from here on are NaN
      polls = 1;
      st.l = __int_as_float(0x7fffffff);
      issued = min(issued, t + D);
    }
    if (came && there) {
      int ke[kDecPages] = {(int)(exps & 0xff) - 64, (int)(exps >> 16 & 0xff) - 64};
      int ve[kDecPages] = {(int)(exps >> 8 & 0xff) - 64, (int)(exps >> 24) - 64};
      const bool tail = (j + kDecPages) * kKv8Page > pos || there != 3;
      if (tail) {
#pragma unroll 1
        for (int i = 0; i < kDecPages; ++i) {
          const int page = __shfl_sync(0xffffffffu, i ? cur.page[1] : cur.page[0], src);
          if (page < 0) {           // no such page: weights 0, and values that are numbers
#pragma unroll 1
            for (int k = lane; k < HD; k += 32)
              *reinterpret_cast<uint4*>(blk + i * PB + kKv8Page * HD + 16 * k) = make_uint4(0, 0, 0, 0);
            fence_proxy_async();
          } else if ((j + i + 1) * kKv8Page > pos) {
            int k2 = i ? ke[1] : ke[0], v2 = i ? ve[1] : ve[0];
            append(blk + i * PB, page, j + i, k2, v2);
            if (i) ke[1] = k2, ve[1] = v2;
            else ke[0] = k2, ve[0] = v2;
          }
        }
        __syncwarp();
      }

      // S = Q K^T: each page's two groups of 8 keys
      float s[2 * kDecPages][4];
#pragma unroll
      for (int q = 0; q < 2 * kDecPages; ++q) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[q][e] = 0.f;
        const uint8_t* xk = blk + q / 2 * PB;
        const int key = q % 2 * 8 + r;
        uint32_t w[KS];
        if (HD == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(xk + unit_off<HD>(key, 2 * c));
          const uint4 y = *reinterpret_cast<const uint4*>(xk + unit_off<HD>(key, 2 * c + 1));
          w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
          w[KS - 4] = y.x; w[KS - 3] = y.y; w[KS - 2] = y.z; w[KS - 1] = y.w;
        } else {
          const uint4 x = *reinterpret_cast<const uint4*>(xk + unit_off<HD>(key, c));
          w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        }
#pragma unroll
        for (int k = 0; k < KS; ++k)
          mma_f16(s[q], qa[k], f16x2_of_e4m3((uint16_t)w[k]), f16x2_of_e4m3((uint16_t)(w[k] >> 16)));
      }
      float p[4 * kDecPages];          // page i, keys 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
      for (int i = 0; i < kDecPages; ++i) {
        const float f = qf * pow2f(ke[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) p[4 * i + e] = (s[2 * i + e / 2][e & 1] + s[2 * i + e / 2][2 + (e & 1)]) * f;
      }
      if (tail) {
        const int lim = pos + rt - j * kKv8Page;
#pragma unroll
        for (int e = 0; e < 4 * kDecPages; ++e)
          if (e / 2 * 8 + 2 * c + (e & 1) > lim || !(there >> (e / 4) & 1)) p[e] = -INFINITY;
      }
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < kDecPages; ++i)
        mx = fmaxf(mx, fmaxf(fmaxf(p[4 * i], p[4 * i + 1]), fmaxf(p[4 * i + 2], p[4 * i + 3])) + (float)ve[i]);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if (__any_sync(0xffffffffu, mx > st.m + (float)kDecLag)) {
        const float mn = fmaxf(st.m, mx);
        const float x = mn == -INFINITY ? 1.f : ex2(st.m - mn);
        st.l *= x;
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) st.o[q][e] *= x;
        st.m = mn;
      }
      // weights times 2^kDecBias and the block's scale: at most 2^14, at least
      // 2^6 for the largest; a pair of f16 then is good to 2^-22 of each and
      // 2^-31 of the largest
      const float ref = st.m == -INFINITY ? 0.f : st.m;
      int lift[kDecPages] = {};
      bool lifted = false;
      st.e = max(st.e, max(ve[0], ve[1]));
      if (min(ve[0], ve[1]) < st.e - kDecFar) {
#pragma unroll
        for (int i = 0; i < kDecPages; ++i)
          if (ve[i] < st.e - kDecFar && (there >> i & 1)) {
            float x = fmaxf(fmaxf(p[4 * i], p[4 * i + 1]), fmaxf(p[4 * i + 2], p[4 * i + 3]));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            x = ref - (x + (float)ve[i]);            // infinity: no key is seen
            const bool far = x > (float)kDecFar && x < INFINITY;
            if (__any_sync(0xffffffffu, far && r < R)) {
              lifted = true;
              if (far) lift[i] = (int)fminf(x, (float)kDecLift);
            }
          }
      }
      uint32_t pa[kDecPages][4];
#pragma unroll
      for (int i = 0; i < kDecPages; ++i) {
        const int up = kDecBias + ve[i] + lift[i];
        const float sub = ref - (float)up;
#pragma unroll
        for (int e = 0; e < 4; ++e) p[4 * i + e] = ex2(p[4 * i + e] - sub);
        st.l += ((p[4 * i] + p[4 * i + 1]) + (p[4 * i + 2] + p[4 * i + 3])) * pow2f(-up);
        split2(p[4 * i], p[4 * i + 1], pa[i][0], pa[i][1]);
        split2(p[4 * i + 2], p[4 * i + 3], pa[i][2], pa[i][3]);
      }

      // O += P V
#pragma unroll
      for (int i = 0; i < kDecPages; ++i) {
        if (lifted) lift_by(lift[i] - (i ? lift[i - 1] : 0));
        const uint8_t* xv = blk + i * PB + kKv8Page * HD;
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
          mma_f16(st.o[4 * k], pa[i], f16x2_of_e4m3((uint16_t)a01), f16x2_of_e4m3((uint16_t)b01));
          mma_f16(st.o[4 * k + 1], pa[i], f16x2_of_e4m3((uint16_t)(a01 >> 16)), f16x2_of_e4m3((uint16_t)(b01 >> 16)));
          mma_f16(st.o[4 * k + 2], pa[i], f16x2_of_e4m3((uint16_t)a23), f16x2_of_e4m3((uint16_t)b23));
          mma_f16(st.o[4 * k + 3], pa[i], f16x2_of_e4m3((uint16_t)(a23 >> 16)), f16x2_of_e4m3((uint16_t)(b23 >> 16)));
        }
      }
      if (lifted) lift_by(-lift[kDecPages - 1]);
    }
    __syncwarp();
    // the slot is free: the unit D further on
    if (t + D < issued && lane == ((t + D) & 31)) issue(src + D < 32 ? cur : nxt, slot);
    if (++slot == D) {
      slot = 0;
      phase ^= 1;
    }
  }
  if (polls == 1)            // copies that were not seen to end are waited for once more
#pragma unroll 1
    for (int k = 0; k < min(D, n); ++k) mbar_wait(&bars[warp][k], (issued - 1 - k) / D & 1, nullptr);
  join();
}

DecLayout dec_layout(int B, int m, int H, int Hkv, int hd) {
  DecLayout l;
  const int G = H / Hkv, R = m * G;
  l.ctas = kv8_sms();
  l.parts_off = (int)kv8_ticket_bytes(l.ctas);
  l.groups = (Hkv + kDecWarps - 1) / kDecWarps;
  l.heads = (Hkv + l.groups - 1) / l.groups;
  l.slices = kDecWarps / l.heads;
  l.slot_floats = R * hd + 2 * R + (2 * R) % 4;
  l.inv_g = 65536 / G + 1;
  l.buf = (R > 512 / hd ? R : 512 / hd) * hd * 4;    // four rows of 128 (eight of 64) at a time in ``begin``
  const int warps = l.heads * l.slices, unit = kDecPages * 2 * kKv8Page * hd;
  const int room = kDecSmem - 1024 - 2048 - warps * l.buf - (2 * B + 1) * 4;   // alignment, static
  // 128 KB in flight per SM fill the memory; more only lengthens its queue
  l.depth = (room < kDecFlight ? room : kDecFlight) / (warps * unit);
  if (l.depth > kDecMaxDepth) l.depth = kDecMaxDepth;
  l.buf_off = warps * l.depth * unit;
  l.meta_off = l.buf_off + warps * l.buf;
  return l;
}

}  // namespace

size_t kv8_decode_ws_bytes(int B, int m, int H, int Hkv, int hd) {
  const DecLayout l = dec_layout(B, m, H, Hkv, hd);
  return kv8_ticket_bytes(l.ctas) + (size_t)l.ctas * l.slices * 2 * l.heads * l.slot_floats * 4;
}

cudaError_t launch_kv8_decode(const Kv8Args& a, cudaStream_t st) {
  CUtensorMap map;
  if (!tma_map_kv8(&map, a.kv, a.n_pages, a.Hkv, a.hd)) return cudaErrorNotSupported;
  DecLayout l = dec_layout(a.B, a.m, a.H, a.Hkv, a.hd);
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.qkv) | reinterpret_cast<uintptr_t>(a.q_gain) |
                       reinterpret_cast<uintptr_t>(a.rope_cos) | reinterpret_cast<uintptr_t>(a.rope_sin);
  const bool vec = (at & 15) == 0 && a.qkv_ld % 4 == 0;
  l.o_vec = a.o ? a.o_ld % 4 == 0 && !(reinterpret_cast<uintptr_t>(a.o) & 15)
                : a.o_ld % 4 == 0 && !(reinterpret_cast<uintptr_t>(a.o16) & 7);
  auto k = a.hd == 128 ? (vec ? kv8_decode_kernel<128, true> : kv8_decode_kernel<128, false>)
                       : (vec ? kv8_decode_kernel<64, true> : kv8_decode_kernel<64, false>);
  static bool attr[4] = {};
  if (!attr[(a.hd == 128) * 2 + vec]) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kDecSmem - 2048);
    if (e != cudaSuccess) return e;
    attr[(a.hd == 128) * 2 + vec] = true;
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
