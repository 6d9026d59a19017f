// MX4: 4-bit values in blocks of 32 along a row.  A block holds 32 e2m1 codes
// (sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to
// a byte with the even column in the low half, under one e8m0 scale byte b that
// stands for 2^(b - 127); b = 255 stands for NaN.
//
// Quantisation of a block with largest magnitude a:
//   b = max(floor(log2 a) - 2 + 127, 0),   code = round(v / 2^(b - 127)) to e2m1,
// to nearest, ties to the even code, magnitudes past 6 to 6 (a lies below 8 steps,
// so only values above 6 steps saturate).  b needs no logarithm: it is a's
// exponent field less 2.  Division by a power of two is exact, so codes and scales
// are the same in any precision.  A block with an infinity or a NaN gets b = 255
// and zero codes: e2m1 has neither.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "kernels.hpp"

namespace moelora {

static constexpr int kMxThreads = 256;

// 8 consecutive values per lane, so 4 lanes share a block
template <typename T>
__global__ void __launch_bounds__(kMxThreads)
mx4_quantize_kernel(int64_t num_rows, int64_t cols, const T* __restrict__ x,
                    const int32_t* __restrict__ rows_used, uint32_t* __restrict__ codes,
                    uint8_t* __restrict__ scales) {
  typedef T tx8 __attribute__((ext_vector_type(8)));
  const int64_t rows = rows_used ? min((int64_t)max(rows_used[0], 0), num_rows) : num_rows;
  const int64_t n = rows * cols / 8;
  const int64_t step = (int64_t)gridDim.x * kMxThreads;
  // n and step are multiples of 4: the four lanes of a block stay together
  for (int64_t i = (int64_t)blockIdx.x * kMxThreads + threadIdx.x; i < n; i += step) {
    const tx8 v = reinterpret_cast<const tx8*>(x)[i];
    // magnitudes compare as integers: finite < infinity < NaN
    uint32_t a = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q)
      a = max(a, __builtin_bit_cast(uint32_t, (float)v[q]) & 0x7FFFFFFFu);
    a = max(a, (uint32_t)__shfl_xor((int)a, 1, 64));
    a = max(a, (uint32_t)__shfl_xor((int)a, 2, 64));
    const uint32_t field = a >> 23;
    const uint32_t b = field == 255 ? 255u : field > 2 ? field - 2 : 0u;
    const float scale = __builtin_bit_cast(float, b << 23);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, (float)v[0], (float)v[1], scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, (float)v[2], (float)v[3], scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, (float)v[4], (float)v[5], scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, (float)v[6], (float)v[7], scale, 3);
    codes[i] = b == 255 ? 0u : c;
    if ((i & 3) == 0) scales[i >> 2] = (uint8_t)b;
  }
}

// 8 values (one word of codes) per lane
template <typename T>
__global__ void __launch_bounds__(kMxThreads)
mx4_dequantize_kernel(int64_t n, const uint32_t* __restrict__ codes,
                      const uint8_t* __restrict__ scales, T* __restrict__ out) {
  typedef T tx8 __attribute__((ext_vector_type(8)));
  const int64_t step = (int64_t)gridDim.x * kMxThreads;
  for (int64_t i = (int64_t)blockIdx.x * kMxThreads + threadIdx.x; i < n; i += step) {
    const uint32_t c = codes[i];
    const float scale = mx4_scale(scales[i >> 2]);
    tx8 v;
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = (T)(e2m1_value(c >> (4 * q)) * scale);
    reinterpret_cast<tx8*>(out)[i] = v;
  }
}

static unsigned mx4_grid(int64_t n) {
  return (unsigned)std::min<int64_t>(ceil_div(n, kMxThreads), 256 * 32);
}

hipError_t launch_mx4_quantize(bool x_f32, int64_t num_rows, int64_t cols, const void* x,
                               const int32_t* rows_used, uint8_t* codes, uint8_t* scales,
                               hipStream_t stream) {
  const dim3 grid(mx4_grid(num_rows * cols / 8)), block(kMxThreads);
  if (x_f32)
    hipLaunchKernelGGL(mx4_quantize_kernel<float>, grid, block, 0, stream, num_rows, cols,
                       static_cast<const float*>(x), rows_used, reinterpret_cast<uint32_t*>(codes),
                       scales);
  else
    hipLaunchKernelGGL(mx4_quantize_kernel<bf16_t>, grid, block, 0, stream, num_rows, cols,
                       static_cast<const bf16_t*>(x), rows_used, reinterpret_cast<uint32_t*>(codes),
                       scales);
  return hipGetLastError();
}

hipError_t launch_mx4_dequantize(bool out_f32, int64_t num_rows, int64_t cols,
                                 const uint8_t* codes, const uint8_t* scales, void* out,
                                 hipStream_t stream) {
  const int64_t n = num_rows * cols / 8;
  const dim3 grid(mx4_grid(n)), block(kMxThreads);
  if (out_f32)
    hipLaunchKernelGGL(mx4_dequantize_kernel<float>, grid, block, 0, stream, n,
                       reinterpret_cast<const uint32_t*>(codes), scales, static_cast<float*>(out));
  else
    hipLaunchKernelGGL(mx4_dequantize_kernel<bf16_t>, grid, block, 0, stream, n,
                       reinterpret_cast<const uint32_t*>(codes), scales, static_cast<bf16_t*>(out));
  return hipGetLastError();
}

}  // namespace moelora
