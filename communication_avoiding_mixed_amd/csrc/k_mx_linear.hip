// Products of a low-precision linear layer, simplest form: 64 x 64 output
// tiles on the vector ALUs, each element of an operand read as float32 by an
// accessor, 16 steps of the summed index at a time through LDS.
//
//   linear       y[m][n]  = sum_k Q4(x)[m][k] W4[n][k]
//   grad input   dx[m][k] = sum_n dy[m][n] W4[n][k]
//   grad weight  dW[n][k] = sum_t dy[t][n] Q8(x)[t][k]
#include "casgd.h"
#include "casgd_internal.h"
#include "casgd_mx.h"
#include "casgd_mx_gemm.h"

namespace casgd {
namespace mx {
namespace {

constexpr int kTile = 64, kStep = 16, kThreads = 256;

template <int FMT>
__device__ __forceinline__ float code_value(const uint8_t* codes, const uint8_t* scales, int64_t ld, int64_t row, int64_t col) {
  const float s = scale_value(scales[row * (ld / kBlock) + col / kBlock]);
  if constexpr (FMT == kMx4) {
    const uint32_t c = (codes[row * (ld / 2) + (col >> 1)] >> (4 * (col & 1))) & 15u;
    return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0)[0] * s;
  } else {
    return e4m3_to_f32(codes[row * ld + col]) * s;
  }
}

// operand(i, k): element of output row (or column) i at summed index k
template <int FMT, bool ACROSS>
struct Coded {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t ld;
  __device__ float operator()(int64_t i, int64_t k) const {
    return ACROSS ? code_value<FMT>(codes, scales, ld, k, i) : code_value<FMT>(codes, scales, ld, i, k);
  }
};
template <int TY, bool ACROSS>
struct Plain {
  const typename Elem<TY>::type* p;
  int64_t stride;
  __device__ float operator()(int64_t i, int64_t k) const { return load1<TY>(ACROSS ? p + k * stride + i : p + i * stride + k); }
};

template <int OUT, typename A, typename B>
__global__ __launch_bounds__(kThreads) void product_kernel(A a, B b, int64_t rows, int64_t cols, int64_t depth,
                                                          typename Elem<OUT>::type* __restrict__ out, int64_t stride,
                                                          int accumulate) {
  __shared__ float As[kStep][kTile + 1], Bs[kStep][kTile + 1];
  const int64_t i0 = static_cast<int64_t>(blockIdx.y) * kTile, j0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < depth; k0 += kStep) {
    for (int e = threadIdx.x; e < kTile * kStep; e += kThreads) {
      const int i = e / kStep, k = e % kStep;
      As[k][i] = i0 + i < rows && k0 + k < depth ? a(i0 + i, k0 + k) : 0.f;
      Bs[k][i] = j0 + i < cols && k0 + k < depth ? b(j0 + i, k0 + k) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep; ++k)
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[u][q] = fmaf(As[k][ty * 4 + u], Bs[k][tx * 4 + q], acc[u][q]);
    __syncthreads();
  }
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t i = i0 + ty * 4 + u, j = j0 + tx * 4 + q;
      if (i < rows && j < cols) {
        auto* p = out + i * stride + j;
        store1<OUT>(p, accumulate ? load1<OUT>(p) + acc[u][q] : acc[u][q]);
      }
    }
}

template <int OUT, typename A, typename B>
hipError_t run_as(A a, B b, int64_t rows, int64_t cols, int64_t depth, void* out, int64_t stride, int accumulate,
                  hipStream_t stream) {
  if (rows == 0 || cols == 0) return hipSuccess;
  hipLaunchKernelGGL((product_kernel<OUT, A, B>), dim3((cols + kTile - 1) / kTile, (rows + kTile - 1) / kTile), dim3(kThreads),
                     0, stream, a, b, rows, cols, depth, static_cast<typename Elem<OUT>::type*>(out), stride, accumulate);
  return hipGetLastError();
}

template <typename A, typename B>
hipError_t run_product(int type, A a, B b, int64_t rows, int64_t cols, int64_t depth, void* out, int64_t stride,
                       int accumulate, hipStream_t stream) {
  if (type == kBF16) return run_as<kBF16>(a, b, rows, cols, depth, out, stride, accumulate, stream);
  if (type == kF16) return run_as<kF16>(a, b, rows, cols, depth, out, stride, accumulate, stream);
  return run_as<kF32>(a, b, rows, cols, depth, out, stride, accumulate, stream);
}

constexpr int kSkinnyRows = 128;
constexpr int64_t kMaxDepth = int64_t{1} << 24;  // 256 rows of codes stay below 2^32 bytes

// Rows of x up to which quantising them again in every workgroup costs less
// than a launch of its own
bool decodes(int64_t m, int64_t k, int64_t n) { return m <= 16 && n * k <= (int64_t{1} << 25); }

template <int OUT, int RX, int RW, int GM, int GN>
hipError_t gemm_as(const Mx4Operand& x, const Mx4Operand& w, int64_t ld, void* y, int64_t stride, hipStream_t stream) {
  constexpr int lds = gemm_lds_bytes<RX, RW>();
  auto* kernel = mx4_gemm_kernel<OUT, RX, RW, GM, GN>;
  static const hipError_t allowed =
      hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (allowed != hipSuccess) return allowed;
  const int64_t tm = (x.rows + RX - 1) / RX, tn = (w.rows + RW - 1) / RW;
  if (tm * tn > (int64_t{1} << 24) - 1) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(tm * tn)), dim3(64 * GM * GN), lds, stream, x, w, ld,
                     static_cast<typename Elem<OUT>::type*>(y), stride, static_cast<uint32_t>(tm), static_cast<uint32_t>(tn), 8u);
  return hipGetLastError();
}

template <int OUT>
hipError_t product_as(const Mx4Operand& x, const Mx4Operand& w, int64_t ld, void* y, int64_t stride, hipStream_t stream) {
  auto* out = static_cast<typename Elem<OUT>::type*>(y);
  const dim3 grid(static_cast<unsigned>((w.rows + 31) / 32)), block(512);
  if (x.rows <= 32)
    hipLaunchKernelGGL((mx4_skinny_kernel<OUT, 1>), grid, block, 0, stream, x, w, ld, out, stride);
  else if (x.rows <= 64)
    hipLaunchKernelGGL((mx4_skinny_kernel<OUT, 2>), grid, block, 0, stream, x, w, ld, out, stride);
  else if (x.rows <= kSkinnyRows)
    hipLaunchKernelGGL((mx4_skinny_kernel<OUT, 4>), grid, block, 0, stream, x, w, ld, out, stride);
  else if (((x.rows + 255) / 256) * ((w.rows + 255) / 256) >= 256)
    return gemm_as<OUT, 256, 256, 4, 2>(x, w, ld, y, stride, stream);
  else
    return gemm_as<OUT, 128, 128, 2, 2>(x, w, ld, y, stride, stream);
  return hipGetLastError();
}

hipError_t launch_product(int type, const Mx4Operand& x, const Mx4Operand& w, int64_t ld, void* y, int64_t stride,
                          hipStream_t stream) {
  if (type == kBF16) return product_as<kBF16>(x, w, ld, y, stride, stream);
  if (type == kF16) return product_as<kF16>(x, w, ld, y, stride, stream);
  return product_as<kF32>(x, w, ld, y, stride, stream);
}

template <int TY, int OUT>
hipError_t decode_as(const void* x, int64_t m, int64_t k, int64_t x_stride, const Mx4Operand& w, void* y, int64_t stride,
                     hipStream_t stream) {
  hipLaunchKernelGGL((mx4_decode_kernel<TY, OUT>), dim3(static_cast<unsigned>((w.rows + 15) / 16)), dim3(512), 0, stream,
                     static_cast<const typename Elem<TY>::type*>(x), m, k, x_stride, w, ld_of(k),
                     static_cast<typename Elem<OUT>::type*>(y), stride);
  return hipGetLastError();
}

template <int TY>
hipError_t decode_from(const void* x, int64_t m, int64_t k, int64_t x_stride, const Mx4Operand& w, void* y, int type,
                       int64_t stride, hipStream_t stream) {
  if (type == kBF16) return decode_as<TY, kBF16>(x, m, k, x_stride, w, y, stride, stream);
  if (type == kF16) return decode_as<TY, kF16>(x, m, k, x_stride, w, y, stride, stream);
  return decode_as<TY, kF32>(x, m, k, x_stride, w, y, stride, stream);
}

}  // namespace
}  // namespace mx
}  // namespace casgd

using namespace casgd;

extern "C" {

int64_t casgd_mx4_linear_workspace(int64_t m, int64_t k, int64_t n) {
  if (m < 0 || m > mx::kMaxDim || k < 1 || k > mx::kMaxDim || n < 0 || n > mx::kMaxDim) return -1;
  const int64_t ld = mx::ld_of(k);
  return m * (ld / 2 + ld / mx::kBlock);
}

int casgd_mx4_linear(const void* x, int x_type, int64_t m, int64_t k, int64_t x_stride, const uint8_t* w_codes,
                     const uint8_t* w_scales, int64_t n, void* y, int y_type, int64_t y_stride, void* workspace,
                     int64_t workspace_bytes, void* hip_stream) {
  if (const char* why = mx::bad_matrix(m, k, x_stride, x_type)) return api_fail(CASGD_EINVAL, why);
  if (const char* why = mx::bad_matrix(m, n, y_stride, y_type)) return api_fail(CASGD_EINVAL, why);
  if (const char* why = mx::bad_codes(w_codes, w_scales, n, mx::kMx4)) return api_fail(CASGD_EINVAL, why);
  if (k > mx::kMaxDepth) return api_fail(CASGD_EINVAL, "k exceeds 2^24");
  if (m == 0) return CASGD_OK;
  if (!x || !y || !workspace) return api_fail(CASGD_EINVAL, "NULL pointer");
  if (reinterpret_cast<uintptr_t>(workspace) % 16 != 0) return api_fail(CASGD_EINVAL, "workspace must be 16-byte aligned");
  if (workspace_bytes < casgd_mx4_linear_workspace(m, k, n)) return api_fail(CASGD_EINVAL, "workspace too small");
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  const int64_t ld = mx::ld_of(k);
  uint8_t* codes = static_cast<uint8_t*>(workspace);
  uint8_t* scales = codes + m * (ld / 2);
  const mx::Mx4Operand w{w_codes, w_scales, n};
  hipError_t e;
  if (mx::decodes(m, k, n)) {
    if (x_type == mx::kBF16)
      e = mx::decode_from<mx::kBF16>(x, m, k, x_stride, w, y, y_type, y_stride, stream);
    else if (x_type == mx::kF16)
      e = mx::decode_from<mx::kF16>(x, m, k, x_stride, w, y, y_type, y_stride, stream);
    else
      e = mx::decode_from<mx::kF32>(x, m, k, x_stride, w, y, y_type, y_stride, stream);
  } else {
    e = mx::launch_quantize(mx::kMx4, x_type, x, m, k, x_stride, codes, scales, stream);
    if (e == hipSuccess) e = mx::launch_product(y_type, {codes, scales, m}, w, ld, y, y_stride, stream);
  }
  return e == hipSuccess ? CASGD_OK : api_hip_fail(e, "linear launch");
}

int casgd_mx4_grad_input(const void* dy, int dy_type, int64_t m, int64_t n, int64_t dy_stride, const uint8_t* w_codes,
                         const uint8_t* w_scales, int64_t k, void* dx, int dx_type, int64_t dx_stride, void* hip_stream) {
  if (const char* why = mx::bad_matrix(m, n, dy_stride, dy_type)) return api_fail(CASGD_EINVAL, why);
  if (const char* why = mx::bad_matrix(m, k, dx_stride, dx_type)) return api_fail(CASGD_EINVAL, why);
  if (const char* why = mx::bad_codes(w_codes, w_scales, n, mx::kMx4)) return api_fail(CASGD_EINVAL, why);
  if (m == 0) return CASGD_OK;
  if (!dy || !dx) return api_fail(CASGD_EINVAL, "NULL pointer");
  const mx::Coded<mx::kMx4, true> w{w_codes, w_scales, mx::ld_of(k)};
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  hipError_t e;
  if (dy_type == mx::kBF16)
    e = mx::run_product(dx_type, mx::Plain<mx::kBF16, false>{static_cast<const uint16_t*>(dy), dy_stride}, w, m, k, n, dx,
                        dx_stride, 0, stream);
  else if (dy_type == mx::kF16)
    e = mx::run_product(dx_type, mx::Plain<mx::kF16, false>{static_cast<const uint16_t*>(dy), dy_stride}, w, m, k, n, dx,
                        dx_stride, 0, stream);
  else
    e = mx::run_product(dx_type, mx::Plain<mx::kF32, false>{static_cast<const float*>(dy), dy_stride}, w, m, k, n, dx,
                        dx_stride, 0, stream);
  return e == hipSuccess ? CASGD_OK : api_hip_fail(e, "input gradient launch");
}

int casgd_mx8_grad_weight(const void* dy, int dy_type, int64_t t, int64_t n, int64_t dy_stride, const uint8_t* x_codes,
                          const uint8_t* x_scales, int64_t k, void* dw, int dw_type, int64_t dw_stride, int accumulate,
                          void* hip_stream) {
  if (const char* why = mx::bad_matrix(t, n, dy_stride, dy_type)) return api_fail(CASGD_EINVAL, why);
  if (const char* why = mx::bad_matrix(n, k, dw_stride, dw_type)) return api_fail(CASGD_EINVAL, why);
  if (const char* why = mx::bad_codes(x_codes, x_scales, t, mx::kMx8)) return api_fail(CASGD_EINVAL, why);
  if (!dw || (t > 0 && !dy)) return api_fail(CASGD_EINVAL, "NULL pointer");
  const mx::Coded<mx::kMx8, true> x{x_codes, x_scales, mx::ld_of(k)};
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  hipError_t e;
  if (dy_type == mx::kBF16)
    e = mx::run_product(dw_type, mx::Plain<mx::kBF16, true>{static_cast<const uint16_t*>(dy), dy_stride}, x, n, k, t, dw,
                        dw_stride, accumulate, stream);
  else if (dy_type == mx::kF16)
    e = mx::run_product(dw_type, mx::Plain<mx::kF16, true>{static_cast<const uint16_t*>(dy), dy_stride}, x, n, k, t, dw,
                        dw_stride, accumulate, stream);
  else
    e = mx::run_product(dw_type, mx::Plain<mx::kF32, true>{static_cast<const float*>(dy), dy_stride}, x, n, k, t, dw,
                        dw_stride, accumulate, stream);
  return e == hipSuccess ? CASGD_OK : api_hip_fail(e, "weight gradient launch");
}

}  // extern "C"
