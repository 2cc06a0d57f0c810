// C ABI of the 8-bit KV cache and the page copies (include/s2_ops.h): checks
// of the arguments, then the launchers.
#include "s2.h"
#include "s2_ops.h"
#include "s2_kernels.h"

#include <algorithm>
#include <cstdlib>
#include <new>
#include <vector>

using namespace s2;

static int status(cudaError_t e) {
  if (e == cudaSuccess) return S2_OK;
  if (e == cudaErrorInvalidValue) {
    cudaGetLastError();
    return S2_EINVAL;
  }
  return S2_ECUDA;
}
static bool aligned(const void* p, uintptr_t n) { return !(reinterpret_cast<uintptr_t>(p) & (n - 1)); }

static bool shape_ok(int B, int H, int Hkv, int hd) {
  return B >= 1 && B <= kKv8MaxSeqs && Hkv >= 1 && Hkv <= 4096 && H >= Hkv && H % Hkv == 0 && H / Hkv <= 8 &&
         (hd == 64 || hd == 128);
}

// S2_FAULT_KV8_POLLS=n (read once): waits inside the attention kernels give up
// after n polls, for the tests of what they leave then.
static unsigned wait_polls() {
  static const unsigned n = [] {
    const char* e = std::getenv("S2_FAULT_KV8_POLLS");
    return e ? (unsigned)std::atoi(e) : Kv8Args().polls;
  }();
  return n;
}

// The arguments that both attention calls have; false if one of them is refused.
static bool fill_args(Kv8Args& a, const float* qkv, int qkv_ld, int B, int H, int Hkv, int hd, const float* q_gain,
                      const float* k_gain, float eps, const float* rope_cos, const float* rope_sin, int n_pos,
                      const int32_t* pos, void* kv8, float* kv_scale, int n_pages, const int32_t* table,
                      int table_ld, void* o, int o_bf16, int o_ld, void* workspace) {
  if (!qkv || !q_gain || !k_gain || !rope_cos || !rope_sin || !pos || !kv8 || !kv_scale || !table || !o ||
      !workspace)
    return false;
  if (!shape_ok(B, H, Hkv, hd) || n_pos < 1 || n_pages < 1 || table_ld < 1) return false;
  if (qkv_ld < (H + 2 * Hkv) * hd || o_ld < H * hd) return false;
  if (!aligned(kv8, 16) || !aligned(workspace, 16) || !aligned(qkv, 4) || !aligned(q_gain, 4) || !aligned(k_gain, 4) ||
      !aligned(rope_cos, 4) || !aligned(rope_sin, 4) || !aligned(pos, 4) || !aligned(kv_scale, 4) ||
      !aligned(table, 4) || !aligned(o, o_bf16 ? 2 : 4))
    return false;
  a.qkv = qkv;
  a.qkv_ld = qkv_ld;
  a.B = B;
  a.pos = pos;
  a.H = H;
  a.Hkv = Hkv;
  a.hd = hd;
  a.q_gain = q_gain;
  a.k_gain = k_gain;
  a.eps = eps;
  a.rope_cos = rope_cos;
  a.rope_sin = rope_sin;
  a.max_pos = (int)std::min<long long>(n_pos, 16LL * table_ld);
  a.kv = static_cast<uint8_t*>(kv8);
  a.scale = kv_scale;
  a.n_pages = n_pages;
  a.table = table;
  a.table_ld = table_ld;
  a.o = o_bf16 ? nullptr : static_cast<float*>(o);
  a.o16 = o_bf16 ? static_cast<__nv_bfloat16*>(o) : nullptr;
  a.o_ld = o_ld;
  a.ws = workspace;
  a.polls = wait_polls();
  return true;
}

extern "C" size_t s2op_attn_decode_kv8_workspace_bytes(int B, int m, int H, int Hkv, int hd) {
  if (!shape_ok(B, H, Hkv, hd) || m < 1 || (long long)m * (H / Hkv) > kKv8MaxRows) return 0;
  return kv8_decode_ws_bytes(B, m, H, Hkv, hd);
}

extern "C" int s2op_attn_decode_kv8(const float* qkv, int qkv_ld, int B, int m, int H, int Hkv, int hd,
                                    const float* q_gain, const float* k_gain, float eps, const float* rope_cos,
                                    const float* rope_sin, int n_pos, const int32_t* pos, void* kv8,
                                    float* kv_scale, int n_pages, const int32_t* table, int table_ld, void* o,
                                    int o_bf16, int o_ld, void* workspace, void* stream) {
  Kv8Args a;
  if (!fill_args(a, qkv, qkv_ld, B, H, Hkv, hd, q_gain, k_gain, eps, rope_cos, rope_sin, n_pos, pos, kv8, kv_scale,
                 n_pages, table, table_ld, o, o_bf16, o_ld, workspace))
    return S2_EINVAL;
  if (m < 1 || (long long)m * (H / Hkv) > kKv8MaxRows) return S2_EINVAL;
  if ((double)B * Hkv * table_ld >= 2147483648.0) return S2_EINVAL;   // pages to read, counted in 31 bits
  a.m = m;
  a.T = B * m;
  return status(launch_kv8_decode(a, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t s2op_attn_prefill_kv8_workspace_bytes(int T, int B, int H, int Hkv, int hd) {
  if (!shape_ok(B, H, Hkv, hd) || T < 1 || T > (1 << 24)) return 0;
  return kv8_prefill_ws_bytes(hd);
}

extern "C" int s2op_attn_prefill_kv8(const float* qkv, int qkv_ld, int T, int B, const int32_t* row0,
                                     const int32_t* pos0, int H, int Hkv, int hd, const float* q_gain,
                                     const float* k_gain, float eps, const float* rope_cos,
                                     const float* rope_sin, int n_pos, void* kv8, float* kv_scale, int n_pages,
                                     const int32_t* table, int table_ld, void* o, int o_bf16, int o_ld,
                                     void* workspace, void* stream) {
  Kv8Args a;
  if (!row0 || !aligned(row0, 4) || T < 1 || T > (1 << 24)) return S2_EINVAL;
  if (!fill_args(a, qkv, qkv_ld, B, H, Hkv, hd, q_gain, k_gain, eps, rope_cos, rope_sin, n_pos, pos0, kv8, kv_scale,
                 n_pages, table, table_ld, o, o_bf16, o_ld, workspace))
    return S2_EINVAL;
  a.T = T;
  a.row0 = row0;
  if (a.max_pos > kKv8MaxPrompt) a.max_pos = kKv8MaxPrompt;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_kv8_append(a, st);
  return status(e == cudaSuccess ? launch_kv8_prefill(a, st) : e);
}

static bool pack_ok(const void* kv, const void* kv8, const void* scale, const int32_t* src, const int32_t* dst,
                    int n_src, int n_dst, int n, int Hkv, int hd) {
  return kv && kv8 && scale && src && dst && n_src >= 1 && n_dst >= 1 && n >= 0 && Hkv >= 1 && Hkv <= 4096 &&
         (long long)n * 2 * Hkv <= 0x7ffffffcLL && (hd == 64 || hd == 128) && aligned(kv, 16) && aligned(kv8, 16) &&
         aligned(scale, 4) && aligned(src, 4) && aligned(dst, 4);
}

extern "C" int s2op_kv8_pack_pages(const void* kv, int kv_bf16, int n_src, const int32_t* src, const int32_t* fill,
                                   void* kv8, float* kv_scale, int n_dst, const int32_t* dst, int n, int Hkv, int hd,
                                   void* stream) {
  if (!pack_ok(kv, kv8, kv_scale, src, dst, n_src, n_dst, n, Hkv, hd) || !aligned(fill, 4)) return S2_EINVAL;
  if (n == 0) return S2_OK;
  Kv8PackArgs p;
  p.kv = const_cast<void*>(kv);
  p.kv_bf16 = kv_bf16 ? 1 : 0;
  p.kv8 = static_cast<uint8_t*>(kv8);
  p.scale = kv_scale;
  p.n_src = n_src;
  p.n_dst = n_dst;
  p.n = n;
  p.src = src;
  p.dst = dst;
  p.fill = fill;
  p.Hkv = Hkv;
  p.hd = hd;
  return status(launch_kv8_pack(p, static_cast<cudaStream_t>(stream)));
}

extern "C" int s2op_kv8_unpack_pages(const void* kv8, const float* kv_scale, int n_src, const int32_t* src, void* kv,
                                     int kv_bf16, int n_dst, const int32_t* dst, int n, int Hkv, int hd,
                                     void* stream) {
  if (!pack_ok(kv, kv8, kv_scale, src, dst, n_src, n_dst, n, Hkv, hd)) return S2_EINVAL;
  if (n == 0) return S2_OK;
  Kv8PackArgs p;
  p.kv = kv;
  p.kv_bf16 = kv_bf16 ? 1 : 0;
  p.kv8 = static_cast<uint8_t*>(const_cast<void*>(kv8));
  p.scale = const_cast<float*>(kv_scale);
  p.n_src = n_src;
  p.n_dst = n_dst;
  p.n = n;
  p.src = src;
  p.dst = dst;
  p.Hkv = Hkv;
  p.hd = hd;
  return status(launch_kv8_unpack(p, static_cast<cudaStream_t>(stream)));
}

// Page pairs in order of ``key`` if no key comes twice and no page is both a
// source and a destination; false otherwise.
static bool ordered_pairs(const int32_t* src, const int32_t* dst, int n, bool by_src,
                          std::vector<std::pair<int32_t, int32_t>>& out) {
  out.resize(n);
  for (int i = 0; i < n; ++i) {
    if (src[i] < 0 || dst[i] < 0) return false;
    out[i] = by_src ? std::make_pair(src[i], dst[i]) : std::make_pair(dst[i], src[i]);
  }
  std::sort(out.begin(), out.end());
  for (int i = 1; i < n; ++i)
    if (out[i].first == out[i - 1].first) return false;
  for (int i = 0; i < n; ++i) {
    const auto it = std::lower_bound(out.begin(), out.end(), std::make_pair(out[i].second, (int32_t)-1));
    if (it != out.end() && it->first == out[i].second) return false;
  }
  return true;
}

extern "C" int s2op_kv_copy_pages(void* kv, size_t page_bytes, void* scale, size_t scale_bytes, int n_pages,
                                  int layers, const int32_t* src, const int32_t* dst, int n, void* stream) {
  if (!kv || page_bytes == 0 || page_bytes % 16 || page_bytes > (1u << 30) || !aligned(kv, 16) || n_pages < 1 ||
      layers < 1 || layers > 65535 || n < 0 || (n > 0 && (!src || !dst)))
    return S2_EINVAL;
  if (scale && (scale_bytes == 0 || scale_bytes % 4 || scale_bytes > (1u << 30) || !aligned(scale, 4)))
    return S2_EINVAL;
  if (n == 0) return S2_OK;
  if (n > n_pages) return S2_EINVAL;   // destinations are distinct
  try {
    std::vector<std::pair<int32_t, int32_t>> by_dst;
    if (!ordered_pairs(src, dst, n, false, by_dst)) return S2_EINVAL;
    for (const auto& p : by_dst)
      if (p.first >= n_pages || p.second >= n_pages) return S2_EINVAL;
    PagePairs pairs;
    for (int at = 0; at < n; at += kPagePairs) {
      const int k = std::min(kPagePairs, n - at);
      for (int i = 0; i < k; ++i) {
        pairs.dst[i] = by_dst[at + i].first;
        pairs.src[i] = by_dst[at + i].second;
      }
      const int s = status(launch_kv_copy_pages(static_cast<uint8_t*>(kv), (long long)page_bytes,
                                                static_cast<uint8_t*>(scale), (int)scale_bytes, n_pages, layers, pairs,
                                                k, static_cast<cudaStream_t>(stream)));
      if (s) return s;
    }
  } catch (const std::bad_alloc&) {
    return S2_ENOMEM;
  }
  return S2_OK;
}

extern "C" int s2op_kv_remap_pages(int32_t* table, int rows, int cols, int table_ld, const int32_t* src,
                                   const int32_t* dst, int n, void* stream) {
  if (!table || !aligned(table, 4) || rows < 0 || cols < 0 || table_ld < cols || n < 0 || (n > 0 && (!src || !dst)) ||
      (long long)rows * cols > (1LL << 38))
    return S2_EINVAL;
  if (n == 0) return S2_OK;
  try {
    std::vector<std::pair<int32_t, int32_t>> by_src;
    if (!ordered_pairs(src, dst, n, true, by_src)) return S2_EINVAL;
    if (rows == 0 || cols == 0) return S2_OK;
    PagePairs pairs;
    for (int at = 0; at < n; at += kPagePairs) {
      const int k = std::min(kPagePairs, n - at);
      for (int i = 0; i < k; ++i) {
        pairs.src[i] = by_src[at + i].first;
        pairs.dst[i] = by_src[at + i].second;
      }
      const int s = status(launch_kv_remap(table, rows, table_ld, cols, pairs, k, static_cast<cudaStream_t>(stream)));
      if (s) return s;
    }
  } catch (const std::bad_alloc&) {
    return S2_ENOMEM;
  }
  return S2_OK;
}
