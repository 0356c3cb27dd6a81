// y = Q4(x) W4^T with its C entry point: which of the product's forms runs.
#include "casgd.h"
#include "casgd_internal.h"
#include "casgd_mx.h"
#include "casgd_mx_gemm.h"

namespace casgd {
namespace mx {
namespace {

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
  if (mx::decodes(m, k, n)) return 0;
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
  const int64_t need = casgd_mx4_linear_workspace(m, k, n);
  if (!x || !y || (need > 0 && !workspace)) return api_fail(CASGD_EINVAL, "NULL pointer");
  if (reinterpret_cast<uintptr_t>(workspace) % 16 != 0) return api_fail(CASGD_EINVAL, "workspace must be 16-byte aligned");
  if (workspace_bytes < need) return api_fail(CASGD_EINVAL, "workspace too small");
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

}  // extern "C"
