// C ABI of the 4-bit weights and the 8-bit rows with scales (include/s2_ops.h):
// checks of the arguments, then the launchers.
#include "s2.h"
#include "s2_ops.h"
#include "s2_kernels.h"

#include <cfloat>
#include <cstdlib>

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

// Rows and columns that the kernels count in 31 bits.
static bool rows_ok(long long n) { return n >= 0 && n <= (1 << 24); }
static bool cols_ok(long long k) { return k >= 1 && k <= (1 << 20); }
// A matrix of fp32 (bf16 = 0) or bf16 rows.
static bool plain_ok(const void* p, int bf16, long long ld, long long cols) {
  return p && aligned(p, bf16 ? 2 : 4) && ld >= cols;
}
static bool vec_ok(const void* p, int bf16, long long ld) {
  return aligned(p, 16) && ld % (bf16 ? 8 : 4) == 0;
}
static bool rows8_ok(const void* y8, long long ld8, int K, const void* scale) {
  return y8 && scale && aligned(y8, 16) && ld8 >= K && ld8 % 16 == 0 && aligned(scale, 16);
}
static bool weights_ok(const void* codes, const void* scale) {
  return codes && scale && aligned(codes, 32) && aligned(scale, 16);
}

extern "C" size_t s2op_w4_code_bytes(int N, int K) {
  return rows_ok(N) && cols_ok(K) ? (size_t)N * ((K + 127) / 128) * 64 : 0;
}

extern "C" size_t s2op_mx_scale_bytes(int rows, int K) {
  return rows_ok(rows) && cols_ok(K) ? (size_t)((rows + 127) / 128) * ((K + 127) / 128) * 512 : 0;
}

static int w4_rows(bool pack, const void* codes, const void* scale, int N, int K, const void* W, int w_bf16, int ldw,
                   void* stream) {
  if (!rows_ok(N) || !cols_ok(K)) return S2_EINVAL;
  if (N == 0) return S2_OK;
  if (!weights_ok(codes, scale) || !plain_ok(W, w_bf16, ldw, K)) return S2_EINVAL;
  W4PackArgs p;
  p.w = const_cast<void*>(W);
  p.w_bf16 = w_bf16 ? 1 : 0;
  p.ldw = ldw;
  p.N = N;
  p.K = K;
  p.codes = static_cast<uint8_t*>(const_cast<void*>(codes));
  p.scale = static_cast<uint8_t*>(const_cast<void*>(scale));
  p.vec = vec_ok(W, w_bf16, ldw);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return status(pack ? launch_w4_pack(p, st) : launch_w4_unpack(p, st));
}

extern "C" int s2op_w4_pack(const void* W, int w_bf16, int N, int K, int ldw, void* codes, void* scale,
                            void* stream) {
  return w4_rows(true, codes, scale, N, K, W, w_bf16, ldw, stream);
}

extern "C" int s2op_w4_unpack(const void* codes, const void* scale, int N, int K, void* W, int w_bf16, int ldw,
                              void* stream) {
  return w4_rows(false, codes, scale, N, K, W, w_bf16, ldw, stream);
}

extern "C" int s2op_mx8_pack(const void* X, int x_bf16, int ldx, int T, int K, void* y8, int ld8, void* y_scale,
                             void* stream) {
  if (!rows_ok(T) || !cols_ok(K)) return S2_EINVAL;
  if (T == 0) return S2_OK;
  if (!plain_ok(X, x_bf16, ldx, K) || !rows8_ok(y8, ld8, K, y_scale)) return S2_EINVAL;
  Mx8PackArgs p;
  p.x = X;
  p.x_bf16 = x_bf16 ? 1 : 0;
  p.ldx = ldx;
  p.T = T;
  p.K = K;
  p.y8 = static_cast<uint8_t*>(y8);
  p.ld8 = ld8;
  p.scale = static_cast<uint8_t*>(y_scale);
  p.vec = vec_ok(X, x_bf16, ldx);
  return status(launch_mx8_pack(p, static_cast<cudaStream_t>(stream)));
}

extern "C" int s2op_add_rmsnorm_mx8(const void* X, int x_bf16, int ldx, const void* R, int r_bf16, int ldr, int T,
                                    int K, const float* gain, float eps, void* H, int ldh, void* y8, int ld8,
                                    void* y_scale, void* stream) {
  if (!rows_ok(T) || !cols_ok(K) || !(eps >= 0.f && eps <= FLT_MAX)) return S2_EINVAL;
  if (T == 0) return S2_OK;
  if (!plain_ok(X, x_bf16, ldx, K) || !gain || !aligned(gain, 4) || !rows8_ok(y8, ld8, K, y_scale)) return S2_EINVAL;
  if (R ? !plain_ok(R, r_bf16, ldr, K) || !H : false) return S2_EINVAL;
  if (H && !plain_ok(H, x_bf16, ldh, K)) return S2_EINVAL;
  // in place: each row onto itself
  if (H == X && ldh != ldx) return S2_EINVAL;
  if (H && H == R && (ldh != ldr || (x_bf16 != 0) != (r_bf16 != 0))) return S2_EINVAL;
  AddNormMx8Args p;
  p.x = X;
  p.x_bf16 = x_bf16 ? 1 : 0;
  p.ldx = ldx;
  p.r = R;
  p.r_bf16 = r_bf16 ? 1 : 0;
  p.ldr = ldr;
  p.h = H ? H : const_cast<void*>(X);
  p.ldh = H ? ldh : ldx;
  p.T = T;
  p.K = K;
  p.gain = gain;
  p.eps = eps;
  p.inv_k.hi = (float)(1.0 / K);
  p.inv_k.lo = (float)(1.0 / K - (double)p.inv_k.hi);
  p.y8 = static_cast<uint8_t*>(y8);
  p.ld8 = ld8;
  p.scale = static_cast<uint8_t*>(y_scale);
  p.vec = vec_ok(X, x_bf16, ldx) && vec_ok(p.h, x_bf16, p.ldh) && (!R || vec_ok(R, r_bf16, ldr));
  p.gain_vec = aligned(gain, 16);
  return status(launch_add_rmsnorm_mx8(p, static_cast<cudaStream_t>(stream)));
}

// S2_FAULT_W4_POLLS=n (read once): waits inside the products give up after n
// polls, for the tests of what they leave then.
static unsigned wait_polls() {
  static const unsigned n = [] {
    const char* e = std::getenv("S2_FAULT_W4_POLLS");
    return e ? (unsigned)std::atoi(e) : W4GemmArgs().polls;
  }();
  return n;
}

// What both products have; false if an argument is refused.
static bool fill_product(W4GemmArgs& a, const void* codes, const void* scale, int N, int K, int T, void* Y, int y_bf16,
                         int ldy, int mode) {
  if (!weights_ok(codes, scale) || !plain_ok(Y, y_bf16, ldy, mode == W4_SWIGLU ? N / 2 : N)) return false;
  a.codes = static_cast<const uint8_t*>(codes);
  a.scale = static_cast<const uint8_t*>(scale);
  a.N = N;
  a.K = K;
  a.T = T;
  a.y = Y;
  a.y_bf16 = y_bf16 ? 1 : 0;
  a.ldy = ldy;
  a.mode = mode;
  a.polls = wait_polls();
  return true;
}
static bool product_shape_ok(int N, int K, int mode) {
  return rows_ok(N) && cols_ok(K) && mode >= W4_STORE && mode <= W4_SWIGLU && !(mode == W4_SWIGLU && N % 2);
}

extern "C" size_t s2op_w4_gemv_workspace_bytes(int K, int B) {
  return cols_ok(K) && B >= 1 && B <= 8 ? w4_gemv_ws_bytes(K, B) : 0;
}

extern "C" int s2op_w4_gemv(const void* codes, const void* scale, int N, int K, const void* X, int x_bf16, int ldx,
                            int B, void* Y, int y_bf16, int ldy, int mode, void* workspace, void* stream) {
  if (!product_shape_ok(N, K, mode) || B < 1 || B > 8) return S2_EINVAL;
  if (N == 0) return S2_OK;
  W4GemmArgs a;
  if (!fill_product(a, codes, scale, N, K, B, Y, y_bf16, ldy, mode) || !plain_ok(X, x_bf16, ldx, K) || !workspace ||
      !aligned(workspace, 16))
    return S2_EINVAL;
  a.x = X;
  a.x_bf16 = x_bf16 ? 1 : 0;
  a.ldx = ldx;
  a.vec = vec_ok(X, x_bf16, ldx);
  a.ws = workspace;
  return status(launch_w4_gemv(a, static_cast<cudaStream_t>(stream)));
}

extern "C" int s2op_w4_gemm(const void* codes, const void* scale, int N, int K, const void* X8, int ld8,
                            const void* x_scale, int T, void* Y, int y_bf16, int ldy, int mode, void* stream) {
  if (!product_shape_ok(N, K, mode) || !rows_ok(T)) return S2_EINVAL;
  if (N == 0 || T == 0) return S2_OK;
  W4GemmArgs a;
  if (!fill_product(a, codes, scale, N, K, T, Y, y_bf16, ldy, mode) || !rows8_ok(X8, ld8, K, x_scale)) return S2_EINVAL;
  a.x8 = static_cast<const uint8_t*>(X8);
  a.ld8 = ld8;
  a.x_scale = static_cast<const uint8_t*>(x_scale);
  return status(launch_w4_gemm(a, static_cast<cudaStream_t>(stream)));
}
