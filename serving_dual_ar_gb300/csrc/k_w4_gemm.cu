// Products of rows with 4-bit weights (mx_common.cuh):
//   Y[t, n] (op)= sum_k X[t, k] W[n, k].
#include "mx_common.cuh"

namespace s2 {

namespace {

S2_DEV float w4_silu_mul(float g, float u) { return g / (1.f + expf(-g)) * u; }

template <typename TY>
S2_DEV void w4_store(TY* y, float v, int mode) {
  *y = from_f<TY>(mode == W4_ADD ? to_f(*y) + v : v);
}

// Four consecutive values of row t from k on.
template <typename TX> S2_DEV void x_values(const W4GemmArgs& a, int t, int k, int KT, float (&v)[4]) {
  const TX* row = static_cast<const TX*>(a.x) + (long long)t * a.ldx;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = k + i < a.K ? to_f(row[k + i]) : 0.f;
}
template <> S2_DEV void x_values<uint8_t>(const W4GemmArgs& a, int t, int k, int KT, float (&v)[4]) {
  const uint8_t* row = a.x8 + (long long)t * a.ld8;
  const float s = mx_scale(a.x_scale[mx_scale_at(t, k / 128, KT) + (k / 32) % 4]);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = k + i < a.K ? mx_e4m3(row[k + i]) * s : 0.f;
}

// One warp per two features and four rows of X; a lane takes four of 128 k.
template <typename TX, typename TY>
__global__ void __launch_bounds__(128) w4_gemm_kernel(W4GemmArgs a) {
  const int lane = threadIdx.x & 31, KT = (a.K + 127) / 128;
  const int n0 = (blockIdx.x * 4 + (threadIdx.x >> 5)) * 2;
  if (n0 >= a.N) return;
  for (int t0 = blockIdx.y * 4; t0 < a.T; t0 += gridDim.y * 4) {
    float acc[2][4] = {};
    for (int kt = 0; kt < KT; ++kt) {
      const int k = kt * 128 + lane * 4;
      float w[2][4], x[4][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int n = min(n0 + j, a.N - 1);
        const uint32_t c = *reinterpret_cast<const uint16_t*>(a.codes + (size_t)n * (KT * 64) + k / 2);
        const float s = mx_scale(a.scale[mx_scale_at(n, kt, KT) + lane / 8]);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[j][i] = mx_e2m1((c >> (4 * i)) & 15u) * s;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) x_values<TX>(a, min(t0 + q, a.T - 1), k, KT, x[q]);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[j][q] = fmaf(w[j][i], x[q][i], acc[j][q]);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float y0 = warp_sum(acc[0][q]), y1 = warp_sum(acc[1][q]);
      if (lane || t0 + q >= a.T) continue;
      TY* y = static_cast<TY*>(a.y) + (long long)(t0 + q) * a.ldy;
      if (a.mode == W4_SWIGLU) {
        y[n0 / 2] = from_f<TY>(w4_silu_mul(y0, y1));
      } else {
        w4_store(y + n0, y0, a.mode);
        if (n0 + 1 < a.N) w4_store(y + n0 + 1, y1, a.mode);
      }
    }
  }
}

template <typename TX>
cudaError_t launch_simple(const W4GemmArgs& a, cudaStream_t st) {
  void* args[] = {const_cast<W4GemmArgs*>(&a)};
  const void* k = a.y_bf16 ? (const void*)w4_gemm_kernel<TX, __nv_bfloat16> : (const void*)w4_gemm_kernel<TX, float>;
  const dim3 grid((a.N + 7) / 8, min((a.T + 3) / 4, 65535));
  const cudaError_t e = cudaLaunchKernel(k, grid, dim3(128), args, 0, st);
  if (e == cudaSuccess) ++g_launch_count;
  return e;
}

}  // namespace

size_t w4_gemv_ws_bytes(int K, int B) { return 16; }

cudaError_t launch_w4_gemv(const W4GemmArgs& a, cudaStream_t st) {
  return a.x_bf16 ? launch_simple<__nv_bfloat16>(a, st) : launch_simple<float>(a, st);
}

cudaError_t launch_w4_gemm(const W4GemmArgs& a, cudaStream_t st) { return launch_simple<uint8_t>(a, st); }

}  // namespace s2
