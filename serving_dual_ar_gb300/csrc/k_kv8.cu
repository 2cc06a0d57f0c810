// The 8-bit KV cache outside the attention kernels: appending a prompt's
// keys and values to their pages, packing fp32 / bf16 pages and unpacking
// them, copying pages and rewriting page tables.
#include "kv8_common.cuh"

namespace s2 {

namespace {

// ---------------------------------------------------------------- append

// The sequence that owns slot ``t`` where sequence b owns the slots from
// (row0[b] / unit) + b * extra on: the last b whose first slot is <= t.  One
// warp, one round of loads per 32 sequences.
S2_DEV int owner_of_slot(const int* row0, int B, int unit, int extra, int t, int lane) {
  int n = 0;
  for (int b = lane; b < B; b += 32) n += (row0[b] / unit + b * extra <= t) ? 1 : 0;
  return __reduce_add_sync(0xffffffffu, n) - 1;
}

// One (touched page of a sequence, kv head): its new rows' keys (normed,
// rotated) and values, one scale each over old and new rows, and the page's
// old rows rescaled where the scale grew.  Four warps; warp w takes new rows
// w, w + 4, ...  Grid (slots, Hkv): T / 16 + 2 B slots, since a sequence with
// n rows touches at most n / 16 + 2 pages.  Bound by the two-float chain of a
// key row (four rows a warp, one after the other), then by memory; a kernel of
// its own because CTAs of the attention behind it read pages that others fill.
template <int HD>
__global__ void __launch_bounds__(128) kv8_append_kernel(Kv8Args a) {
  constexpr int N = HD / 32;
  __shared__ float x[2][kKv8Page][HD];
  __shared__ float amax_s[2][4];
  const int g = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the wait first: the attention behind may read qkv as soon as it starts
  pdl_wait();
  pdl_launch_next();
  const int b = owner_of_slot(a.row0, a.B, kKv8Page, 2, blockIdx.x, lane);
  if (b < 0) return;
  const int r0 = a.row0[b], n = min(a.row0[b + 1], a.T) - r0, pos0 = a.pos[b];
  if (r0 < 0 || n <= 0 || pos0 < 0 || pos0 > a.max_pos - n) return;
  const int j = pos0 / kKv8Page + (int)blockIdx.x - (r0 / kKv8Page + 2 * b);
  const int first = max(pos0, j * kKv8Page), end = min(pos0 + n, (j + 1) * kKv8Page);
  if (first >= end) return;
  const int page = a.table[(size_t)b * a.table_ld + j];
  if (page < 0 || page >= a.n_pages) return;

  float mk = 0.f, mv = 0.f;
  for (int p = first + warp; p < end; p += 4) {
    const float* row = a.qkv + (size_t)(r0 + p - pos0) * a.qkv_ld + (size_t)(a.H + g) * HD;
    float k[N], v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = row[(size_t)a.Hkv * HD + lane + 32 * i];
    kv8_key_row<HD>(row, a.k_gain, a.rope_cos + (size_t)p * (HD / 2), a.rope_sin + (size_t)p * (HD / 2), a.eps, lane,
                    k);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[0][p % kKv8Page][lane + 32 * i] = k[i];
      x[1][p % kKv8Page][lane + 32 * i] = v[i];
    }
    mk = abs_max(k, mk);
    mv = abs_max(v, mv);
  }
  mk = warp_max(mk);
  mv = warp_max(mv);
  if (lane == 0) {
    amax_s[0][warp] = mk;
    amax_s[1][warp] = mv;
  }
  __syncthreads();
  const int had = first - j * kKv8Page;   // rows of the page that came before
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const size_t blk = ((size_t)page * 2 + t) * a.Hkv + g;
    const float am = fmaxf(fmaxf(amax_s[t][0], amax_s[t][1]), fmaxf(amax_s[t][2], amax_s[t][3]));
    const int e_old = had ? kv8_scale_exp(a.scale[blk]) : kKv8EMin;
    const int e = max(e_old, kv8_exponent(am));
    uint32_t* out = reinterpret_cast<uint32_t*>(a.kv + blk * (kKv8Page * HD));
    if (had && e > e_old) {
      const float f = pow2f(e_old - e);
      for (int i = tid; i < had * HD / 4; i += 128) out[i] = e4m3_rescale4(out[i], f);
    }
    const float f = pow2f(-e);
    for (int i = tid; i < (end - first) * HD / 4; i += 128) {
      const float* s = &x[t][had][0] + 4 * i;
      out[had * HD / 4 + i] = e4m3x2(s[0] * f, s[1] * f) | (e4m3x2(s[2] * f, s[3] * f) << 16);
    }
    __syncthreads();   // every thread has read the scale
    if (tid == 0) a.scale[blk] = pow2f(e);
  }
}

// ---------------------------------------------------------------- pack / unpack

// One block (16 rows of one page, K or V, head) per warp: its 8 KB (fp32) are
// all in flight at once, the largest magnitude needs no barrier, and the
// values are rounded from the registers that they were loaded to.  Bound by
// memory: 2,052 fp32 pages of 8 heads x 128 (336 MB) take 53.6 us, 6.3 TB/s; a
// CTA per block with a barrier took 56.
template <typename T> struct Unit16;            // 16 bytes of an unpacked page
template <> struct Unit16<float> {
  static constexpr int kValues = 4;
  static S2_DEV void get(const uint4& u, float (&v)[4]) {
    v[0] = __uint_as_float(u.x);
    v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z);
    v[3] = __uint_as_float(u.w);
  }
  static S2_DEV uint4 put(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
template <> struct Unit16<__nv_bfloat16> {
  static constexpr int kValues = 8;
  static S2_DEV void get(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16lo(w[i]);
      v[2 * i + 1] = bf16hi(w[i]);
    }
  }
  static S2_DEV uint4 put(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <typename T, int HD>
__global__ void __launch_bounds__(128) kv8_pack_kernel(Kv8PackArgs p) {
  constexpr int V = Unit16<T>::kValues, N = kKv8Page * HD / (32 * V);     // values and units of a lane
  const int at = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int i = at / (2 * p.Hkv), blk = at % (2 * p.Hkv);
  if (i >= p.n) return;
  const int src = p.src[i], dst = p.dst[i];
  if (src < 0 || src >= p.n_src || dst < 0 || dst >= p.n_dst) return;
  const int rows = p.fill ? min(max(p.fill[i], 0), kKv8Page) : kKv8Page;
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const T*>(p.kv) +
                                                  ((size_t)src * 2 * p.Hkv + blk) * (kKv8Page * HD));
  uint4 u[N];
#pragma unroll
  for (int c = 0; c < N; ++c) u[c] = (c * 32 + lane) * V < rows * HD ? __ldcs(x + c * 32 + lane) : make_uint4(0, 0, 0, 0);
  float m = 0.f;
#pragma unroll
  for (int c = 0; c < N; ++c) {
    float v[V];
    Unit16<T>::get(u[c], v);
    m = abs_max(v, m);
  }
  const int e = kv8_exponent(warp_max(m));
  const float f = pow2f(-e);
  const size_t ob = (size_t)dst * 2 * p.Hkv + blk;
  uint32_t* out = reinterpret_cast<uint32_t*>(p.kv8 + ob * (kKv8Page * HD));
#pragma unroll
  for (int c = 0; c < N; ++c) {
    float v[V];
    Unit16<T>::get(u[c], v);
    uint32_t w[V / 4];
#pragma unroll
    for (int k = 0; k < V / 4; ++k)
      w[k] = e4m3x2(v[4 * k] * f, v[4 * k + 1] * f) | (e4m3x2(v[4 * k + 2] * f, v[4 * k + 3] * f) << 16);
    if constexpr (V == 4) out[c * 32 + lane] = w[0];
    else reinterpret_cast<uint2*>(out)[c * 32 + lane] = make_uint2(w[0], w[V / 4 - 1]);
  }
  if (lane == 0) p.scale[ob] = pow2f(e);
}

template <typename T, int HD>
__global__ void __launch_bounds__(128) kv8_unpack_kernel(Kv8PackArgs p) {
  constexpr int V = Unit16<T>::kValues, N = kKv8Page * HD / (32 * V);
  const int at = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int i = at / (2 * p.Hkv), blk = at % (2 * p.Hkv);
  if (i >= p.n) return;
  const int src = p.src[i], dst = p.dst[i];
  if (src < 0 || src >= p.n_src || dst < 0 || dst >= p.n_dst) return;
  const size_t ib = (size_t)src * 2 * p.Hkv + blk;
  const uint32_t* in = reinterpret_cast<const uint32_t*>(p.kv8 + ib * (kKv8Page * HD));
  uint32_t w[N][V / 4];
#pragma unroll
  for (int c = 0; c < N; ++c) {
    if constexpr (V == 4) {
      w[c][0] = in[c * 32 + lane];
    } else {
      const uint2 y = reinterpret_cast<const uint2*>(in)[c * 32 + lane];
      w[c][0] = y.x;
      w[c][V / 4 - 1] = y.y;
    }
  }
  const float f = pow2f(kv8_scale_exp(p.scale[ib]));
  uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(p.kv) + ((size_t)dst * 2 * p.Hkv + blk) * (kKv8Page * HD));
#pragma unroll
  for (int c = 0; c < N; ++c) {
    float v[V];
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      uint32_t h = f16x2_of_e4m3((uint16_t)(w[c][k / 2] >> (k & 1) * 16));
      const float2 x = __half22float2(*reinterpret_cast<__half2*>(&h));
      v[2 * k] = x.x * f;
      v[2 * k + 1] = x.y * f;
    }
    __stcs(out + c * 32 + lane, Unit16<T>::put(v));
  }
}

// ---------------------------------------------------------------- page copies

// One 16 KB chunk of one page in one layer per CTA, all of it in flight at
// once; the pairs are a kernel argument, of the smaller size where they fit (a
// launch with 16 KB of arguments costs the host more).  Bound by memory: 400
// pages of 32 KB in 36 layers (946 MB read and written) take 143 us, 6.6 TB/s;
// 32 pages (76 MB) 14.4 us, where the start counts.
constexpr int kCopyChunk = 16384;
template <int N>
struct Pairs {
  int src[N], dst[N];
};
template <int N>
__global__ void __launch_bounds__(256)
kv_copy_pages_kernel(uint8_t* kv, long long page_bytes, uint8_t* scale, int scale_bytes, int n_pages, int chunks,
                     const __grid_constant__ Pairs<N> pairs) {
  const int i = blockIdx.x / chunks, chunk = blockIdx.x % chunks, tid = threadIdx.x;
  const size_t base = (size_t)blockIdx.y * n_pages;
  const size_t s = base + pairs.src[i], d = base + pairs.dst[i];
  const uint4* from = reinterpret_cast<const uint4*>(kv + s * page_bytes) + (size_t)chunk * (kCopyChunk / 16);
  uint4* to = reinterpret_cast<uint4*>(kv + d * page_bytes) + (size_t)chunk * (kCopyChunk / 16);
  const long long left = page_bytes / 16 - (long long)chunk * (kCopyChunk / 16);
  uint4 x[kCopyChunk / 4096];
#pragma unroll
  for (int c = 0; c < kCopyChunk / 4096; ++c)
    if (c * 256 + tid < left) x[c] = __ldcs(from + c * 256 + tid);
#pragma unroll
  for (int c = 0; c < kCopyChunk / 4096; ++c)
    if (c * 256 + tid < left) __stcs(to + c * 256 + tid, x[c]);
  if (scale && chunk == 0)
    for (int c = tid; c < scale_bytes / 4; c += 256)
      reinterpret_cast<uint32_t*>(scale + d * scale_bytes)[c] =
          reinterpret_cast<const uint32_t*>(scale + s * scale_bytes)[c];
}

// Each table entry that is some pair's source becomes its destination (binary
// search among the sources in order; they are a kernel argument, read through
// the constant cache).  128 x 107 entries: latency alone, about 3 us.
__global__ void __launch_bounds__(256)
kv_remap_kernel(int* table, int rows, int table_ld, int cols, int n, const __grid_constant__ PagePairs pairs) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= (long long)rows * cols) return;
  int* e = table + i / cols * table_ld + i % cols;
  const int page = *e;
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pairs.src[mid] < page) lo = mid + 1;
    else hi = mid;
  }
  if (lo < n && pairs.src[lo] == page) *e = pairs.dst[lo];
}

cudaLaunchConfig_t config(dim3 grid, int threads, cudaStream_t st) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.stream = st;
  return c;
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8Args& a, cudaStream_t st) {
  const cudaLaunchConfig_t c = config(dim3(a.T / kKv8Page + 2 * a.B, a.Hkv), 128, st);
  return s2_launch(&c, a.hd == 128 ? kv8_append_kernel<128> : kv8_append_kernel<64>, a);
}

cudaError_t launch_kv8_pack(const Kv8PackArgs& p, cudaStream_t st) {
  const cudaLaunchConfig_t c = config(dim3((p.n * 2 * p.Hkv + 3) / 4), 128, st);
  auto k = p.kv_bf16 ? (p.hd == 128 ? kv8_pack_kernel<__nv_bfloat16, 128> : kv8_pack_kernel<__nv_bfloat16, 64>)
                     : (p.hd == 128 ? kv8_pack_kernel<float, 128> : kv8_pack_kernel<float, 64>);
  return s2_launch(&c, k, p);
}

cudaError_t launch_kv8_unpack(const Kv8PackArgs& p, cudaStream_t st) {
  const cudaLaunchConfig_t c = config(dim3((p.n * 2 * p.Hkv + 3) / 4), 128, st);
  auto k = p.kv_bf16 ? (p.hd == 128 ? kv8_unpack_kernel<__nv_bfloat16, 128> : kv8_unpack_kernel<__nv_bfloat16, 64>)
                     : (p.hd == 128 ? kv8_unpack_kernel<float, 128> : kv8_unpack_kernel<float, 64>);
  return s2_launch(&c, k, p);
}

template <int N>
static cudaError_t copy_pages(uint8_t* kv, long long page_bytes, uint8_t* scale, int scale_bytes, int n_pages,
                              int layers, const PagePairs& pairs, int n, cudaStream_t st) {
  Pairs<N> few;
  for (int i = 0; i < n; ++i) {
    few.src[i] = pairs.src[i];
    few.dst[i] = pairs.dst[i];
  }
  const int chunks = (int)((page_bytes + kCopyChunk - 1) / kCopyChunk);
  const cudaLaunchConfig_t c = config(dim3(n * chunks, layers), 256, st);
  return s2_launch(&c, kv_copy_pages_kernel<N>, kv, page_bytes, scale, scale_bytes, n_pages, chunks, few);
}

cudaError_t launch_kv_copy_pages(uint8_t* kv, long long page_bytes, uint8_t* scale, int scale_bytes, int n_pages,
                                 int layers, const PagePairs& pairs, int n, cudaStream_t st) {
  return (n <= 64 ? copy_pages<64> : copy_pages<kPagePairs>)(kv, page_bytes, scale, scale_bytes, n_pages, layers, pairs,
                                                             n, st);
}

cudaError_t launch_kv_remap(int* table, int rows, int table_ld, int cols, const PagePairs& pairs, int n,
                            cudaStream_t st) {
  const long long entries = (long long)rows * cols;
  const cudaLaunchConfig_t c = config(dim3((unsigned)((entries + 255) / 256)), 256, st);
  return s2_launch(&c, kv_remap_kernel, table, rows, table_ld, cols, n, pairs);
}

}  // namespace s2
