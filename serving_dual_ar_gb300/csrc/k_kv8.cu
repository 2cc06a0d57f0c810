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
// n rows touches at most n / 16 + 2 pages.
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

// One block (16 rows of one page, K or V, head) per CTA of 128 threads.
template <typename T, int HD>
__global__ void __launch_bounds__(128) kv8_pack_kernel(Kv8PackArgs p) {
  __shared__ float am_s[4];
  const int i = blockIdx.x / (2 * p.Hkv), blk = blockIdx.x % (2 * p.Hkv), tid = threadIdx.x;
  const int src = p.src[i], dst = p.dst[i];
  if (src < 0 || src >= p.n_src || dst < 0 || dst >= p.n_dst) return;
  const int rows = p.fill ? min(max(p.fill[i], 0), kKv8Page) : kKv8Page;
  const T* x = static_cast<const T*>(p.kv) + ((size_t)src * 2 * p.Hkv + blk) * (kKv8Page * HD);
  constexpr int W = kKv8Page * HD / 128;   // values of each thread
  float v[W], m = 0.f;
#pragma unroll
  for (int c = 0; c < W; c += 4)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int at = (c / 4 * 128 + tid) * 4 + e;
      v[c + e] = at < rows * HD ? to_f(x[at]) : 0.f;
      m = fmaxf(m, fabsf(v[c + e]));
    }
  m = warp_max(m);
  if ((tid & 31) == 0) am_s[tid >> 5] = m;
  __syncthreads();
  const int e = kv8_exponent(fmaxf(fmaxf(am_s[0], am_s[1]), fmaxf(am_s[2], am_s[3])));
  const float f = pow2f(-e);
  const size_t ob = (size_t)dst * 2 * p.Hkv + blk;
  uint32_t* out = reinterpret_cast<uint32_t*>(p.kv8 + ob * (kKv8Page * HD));
#pragma unroll
  for (int c = 0; c < W; c += 4)
    out[c / 4 * 128 + tid] = e4m3x2(v[c] * f, v[c + 1] * f) | (e4m3x2(v[c + 2] * f, v[c + 3] * f) << 16);
  if (tid == 0) p.scale[ob] = pow2f(e);
}

template <typename T, int HD>
__global__ void __launch_bounds__(128) kv8_unpack_kernel(Kv8PackArgs p) {
  const int i = blockIdx.x / (2 * p.Hkv), blk = blockIdx.x % (2 * p.Hkv), tid = threadIdx.x;
  const int src = p.src[i], dst = p.dst[i];
  if (src < 0 || src >= p.n_src || dst < 0 || dst >= p.n_dst) return;
  const size_t ib = (size_t)src * 2 * p.Hkv + blk;
  const uint32_t* in = reinterpret_cast<const uint32_t*>(p.kv8 + ib * (kKv8Page * HD));
  const float f = pow2f(kv8_scale_exp(p.scale[ib]));
  T* out = static_cast<T*>(p.kv) + ((size_t)dst * 2 * p.Hkv + blk) * (kKv8Page * HD);
  for (int c = tid; c < kKv8Page * HD / 4; c += 128) {
    const uint32_t w = in[c];
    uint32_t a = f16x2_of_e4m3((uint16_t)w), b = f16x2_of_e4m3((uint16_t)(w >> 16));
    const float2 x = __half22float2(*reinterpret_cast<__half2*>(&a));
    const float2 y = __half22float2(*reinterpret_cast<__half2*>(&b));
    out[4 * c] = from_f<T>(x.x * f);
    out[4 * c + 1] = from_f<T>(x.y * f);
    out[4 * c + 2] = from_f<T>(y.x * f);
    out[4 * c + 3] = from_f<T>(y.y * f);
  }
}

// ---------------------------------------------------------------- page copies

__global__ void __launch_bounds__(256)
kv_copy_pages_kernel(uint8_t* kv, long long page_bytes, uint8_t* scale, int scale_bytes, int n_pages,
                     const __grid_constant__ PagePairs pairs) {
  const int i = blockIdx.x;
  const size_t base = (size_t)blockIdx.y * n_pages;
  const size_t s = base + pairs.src[i], d = base + pairs.dst[i];
  const uint4* from = reinterpret_cast<const uint4*>(kv + s * page_bytes);
  uint4* to = reinterpret_cast<uint4*>(kv + d * page_bytes);
  for (long long c = threadIdx.x; c < page_bytes / 16; c += 256) to[c] = from[c];
  if (scale)
    for (int c = threadIdx.x; c < scale_bytes / 4; c += 256)
      reinterpret_cast<uint32_t*>(scale + d * scale_bytes)[c] =
          reinterpret_cast<const uint32_t*>(scale + s * scale_bytes)[c];
}

// Each table entry that is some pair's source becomes its destination (binary
// search among the sources in order).
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
  const cudaLaunchConfig_t c = config(dim3(p.n * 2 * p.Hkv), 128, st);
  auto k = p.kv_bf16 ? (p.hd == 128 ? kv8_pack_kernel<__nv_bfloat16, 128> : kv8_pack_kernel<__nv_bfloat16, 64>)
                     : (p.hd == 128 ? kv8_pack_kernel<float, 128> : kv8_pack_kernel<float, 64>);
  return s2_launch(&c, k, p);
}

cudaError_t launch_kv8_unpack(const Kv8PackArgs& p, cudaStream_t st) {
  const cudaLaunchConfig_t c = config(dim3(p.n * 2 * p.Hkv), 128, st);
  auto k = p.kv_bf16 ? (p.hd == 128 ? kv8_unpack_kernel<__nv_bfloat16, 128> : kv8_unpack_kernel<__nv_bfloat16, 64>)
                     : (p.hd == 128 ? kv8_unpack_kernel<float, 128> : kv8_unpack_kernel<float, 64>);
  return s2_launch(&c, k, p);
}

cudaError_t launch_kv_copy_pages(uint8_t* kv, long long page_bytes, uint8_t* scale, int scale_bytes, int n_pages,
                                 int layers, const PagePairs& pairs, int n, cudaStream_t st) {
  const cudaLaunchConfig_t c = config(dim3(n, layers), 256, st);
  return s2_launch(&c, kv_copy_pages_kernel, kv, page_bytes, scale, scale_bytes, n_pages, pairs);
}

cudaError_t launch_kv_remap(int* table, int rows, int table_ld, int cols, const PagePairs& pairs, int n,
                            cudaStream_t st) {
  const long long entries = (long long)rows * cols;
  const cudaLaunchConfig_t c = config(dim3((unsigned)((entries + 255) / 256)), 256, st);
  return s2_launch(&c, kv_remap_kernel, table, rows, table_ld, cols, n, pairs);
}

}  // namespace s2
