// Microscaled storage: rows of bf16, fp16 or float32 to MX4 / MX8 codes and
// scales, and back, with their C entry points.
//
// One lane holds 8 elements, four lanes a block of 32: the block's max |x|
// is two DPP moves, its scale is integer arithmetic on the max's bits, and
// the elements are converted once.  Both directions are one pass and bound
// by memory traffic (8192 x 8192 float32 to MX4 5.3 TB/s, back 6.2 TB/s; two or
// four loads of a lane in flight were no faster).
#include "casgd.h"
#include "casgd_internal.h"
#include "casgd_mx.h"

namespace casgd {
namespace mx {
namespace {

constexpr int kThreads = 256;

// (row, first column) of this thread's 8 elements.  The workgroup's start is
// divided once in 64 bits by scalar code, the lanes' part in 32 bits.
__device__ __forceinline__ void locate(uint32_t per_row, int64_t& row, uint32_t& chunk) {
  const int64_t start = static_cast<int64_t>(blockIdx.x) * kThreads;
  const int64_t r0 = start / per_row;
  const uint32_t at = static_cast<uint32_t>(start - r0 * per_row) + threadIdx.x;
  const uint32_t r = at / per_row;
  row = r0 + r;
  chunk = at - r * per_row;
}

template <int FMT, int TY, bool STREAM>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(const typename Elem<TY>::type* __restrict__ x, int64_t rows,
                                                              int64_t cols, int64_t stride, uint32_t per_row,
                                                              uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  int64_t row;
  uint32_t chunk;
  locate(per_row, row, chunk);
  if (row >= rows) return;  // whole blocks leave together: 4 divides per_row
  float v[8];
  load8<TY, STREAM>(x + row * stride, static_cast<int64_t>(chunk) * 8, cols, v);
  const uint32_t byte = scale_byte<FMT>(quad_max(amax_bits(v)));
  const int64_t at = row * per_row + chunk;
  if constexpr (FMT == kMx4)
    reinterpret_cast<uint32_t*>(codes)[at] = encode_mx4(v, byte);
  else
    reinterpret_cast<u32x2*>(codes)[at] = encode_mx8(v, byte);
  if ((threadIdx.x & 3) == 0) scales[at >> 2] = static_cast<uint8_t>(byte);
}

template <int FMT, int TY>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, int64_t rows,
                                                                int64_t cols, int64_t stride, uint32_t per_row,
                                                                typename Elem<TY>::type* __restrict__ out) {
  int64_t row;
  uint32_t chunk;
  locate(per_row, row, chunk);
  if (row >= rows) return;
  const int64_t at = row * per_row + chunk;
  const float scale = scale_value(scales[at >> 2]);
  float v[8];
  if constexpr (FMT == kMx4)
    decode_mx4(reinterpret_cast<const uint32_t*>(codes)[at], scale, v);
  else
    decode_mx8(reinterpret_cast<const u32x2*>(codes)[at], scale, v);
  store8<TY>(out + row * stride, static_cast<int64_t>(chunk) * 8, cols, v);
}

// a launch has fewer than 2^32 threads; one row is at most 2^28 chunks
int64_t rows_per_launch(int64_t per_row) { return (int64_t{1} << 31) / per_row; }

template <int FMT, int TY>
hipError_t quantize_as(const void* x, int64_t rows, int64_t cols, int64_t stride, uint8_t* codes, uint8_t* scales,
                       hipStream_t stream) {
  const uint32_t per_row = static_cast<uint32_t>(ld_of(cols) / 8);
  const int64_t step = rows_per_launch(per_row);
  const auto* src = static_cast<const typename Elem<TY>::type*>(x);
  // A matrix of more than half the 256 MB last-level cache is read past it
  // (8192 x 8192 float32 to MX4 58 us instead of 71, and reading the codes back
  // 49 instead of 60); a smaller one may still be there (5001 x 4100 fp16 to MX8
  // 13 us, past the cache 15).
  const bool large = rows * cols * static_cast<int64_t>(sizeof(*src)) > (int64_t{1} << 27);
  auto* kernel = large ? mx_quantize_kernel<FMT, TY, true> : mx_quantize_kernel<FMT, TY, false>;
  for (int64_t r = 0; r < rows; r += step) {
    const int64_t part = rows - r < step ? rows - r : step;
    const int64_t grid = (part * per_row + kThreads - 1) / kThreads;
    const int64_t at = r * per_row;  // in chunks of 8 codes
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream, src + r * stride, part, cols, stride, per_row, codes + at * (FMT == kMx4 ? 4 : 8), scales + at / 4);
  }
  return hipGetLastError();
}

template <int FMT, int TY>
hipError_t dequantize_as(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out, int64_t stride,
                         hipStream_t stream) {
  const uint32_t per_row = static_cast<uint32_t>(ld_of(cols) / 8);
  const int64_t step = rows_per_launch(per_row);
  auto* dst = static_cast<typename Elem<TY>::type*>(out);
  for (int64_t r = 0; r < rows; r += step) {
    const int64_t part = rows - r < step ? rows - r : step;
    const int64_t grid = (part * per_row + kThreads - 1) / kThreads;
    const int64_t at = r * per_row;
    hipLaunchKernelGGL((mx_dequantize_kernel<FMT, TY>), dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream,
                       codes + at * (FMT == kMx4 ? 4 : 8), scales + at / 4, part, cols, stride, per_row, dst + r * stride);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize(int format, int type, const void* x, int64_t rows, int64_t cols, int64_t stride, uint8_t* codes,
                           uint8_t* scales, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  if (format == kMx4) {
    if (type == kBF16) return quantize_as<kMx4, kBF16>(x, rows, cols, stride, codes, scales, stream);
    if (type == kF16) return quantize_as<kMx4, kF16>(x, rows, cols, stride, codes, scales, stream);
    return quantize_as<kMx4, kF32>(x, rows, cols, stride, codes, scales, stream);
  }
  if (type == kBF16) return quantize_as<kMx8, kBF16>(x, rows, cols, stride, codes, scales, stream);
  if (type == kF16) return quantize_as<kMx8, kF16>(x, rows, cols, stride, codes, scales, stream);
  return quantize_as<kMx8, kF32>(x, rows, cols, stride, codes, scales, stream);
}

hipError_t launch_dequantize(int format, int type, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                             void* out, int64_t stride, hipStream_t stream) {
  if (rows == 0) return hipSuccess;
  if (format == kMx4) {
    if (type == kBF16) return dequantize_as<kMx4, kBF16>(codes, scales, rows, cols, out, stride, stream);
    if (type == kF16) return dequantize_as<kMx4, kF16>(codes, scales, rows, cols, out, stride, stream);
    return dequantize_as<kMx4, kF32>(codes, scales, rows, cols, out, stride, stream);
  }
  if (type == kBF16) return dequantize_as<kMx8, kBF16>(codes, scales, rows, cols, out, stride, stream);
  if (type == kF16) return dequantize_as<kMx8, kF16>(codes, scales, rows, cols, out, stride, stream);
  return dequantize_as<kMx8, kF32>(codes, scales, rows, cols, out, stride, stream);
}

}  // namespace mx
}  // namespace casgd

using namespace casgd;

extern "C" {

int64_t casgd_mx_ld(int64_t cols) { return cols < 1 || cols > mx::kMaxDim ? -1 : mx::ld_of(cols); }

int casgd_mx_quantize(const void* x, int type, int64_t rows, int64_t cols, int64_t stride, int format, uint8_t* codes,
                      uint8_t* scales, void* hip_stream) {
  if (const char* why = mx::bad_matrix(rows, cols, stride, type)) return api_fail(CASGD_EINVAL, why);
  if (const char* why = mx::bad_codes(codes, scales, rows, format)) return api_fail(CASGD_EINVAL, why);
  if (rows > 0 && !x) return api_fail(CASGD_EINVAL, "NULL x");
  const hipError_t e = mx::launch_quantize(format, type, x, rows, cols, stride, codes, scales,
                                           static_cast<hipStream_t>(hip_stream));
  return e == hipSuccess ? CASGD_OK : api_hip_fail(e, "quantise launch");
}

int casgd_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int format, int64_t rows, int64_t cols, void* out,
                        int type, int64_t stride, void* hip_stream) {
  if (const char* why = mx::bad_matrix(rows, cols, stride, type)) return api_fail(CASGD_EINVAL, why);
  if (const char* why = mx::bad_codes(codes, scales, rows, format)) return api_fail(CASGD_EINVAL, why);
  if (rows > 0 && !out) return api_fail(CASGD_EINVAL, "NULL out");
  const hipError_t e = mx::launch_dequantize(format, type, codes, scales, rows, cols, out, stride,
                                             static_cast<hipStream_t>(hip_stream));
  return e == hipSuccess ? CASGD_OK : api_hip_fail(e, "dequantise launch");
}

}  // extern "C"
