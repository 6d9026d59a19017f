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

// 8 consecutive values per lane, so 4 lanes share a block.  A thread takes kUnits such
// units kMxThreads apart, all loaded before the first is worked on: one where they would
// not fill the chip otherwise, four else.
template <typename T, int kUnits>
__global__ void __launch_bounds__(kMxThreads)
mx4_quantize_kernel(int64_t num_rows, int64_t cols, const T* __restrict__ x,
                    const int32_t* __restrict__ rows_used, uint32_t* __restrict__ codes,
                    uint8_t* __restrict__ scales) {
  typedef T tx8 __attribute__((ext_vector_type(8)));
  const int64_t rows = rows_used ? min((int64_t)max(rows_used[0], 0), num_rows) : num_rows;
  const int64_t n = rows * cols / 8;
  // n is a multiple of 4: the four lanes of a block stay together
  for (int64_t base = (int64_t)blockIdx.x * (kMxThreads * kUnits); base < n;
       base += (int64_t)gridDim.x * (kMxThreads * kUnits)) {
    tx8 v[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int64_t i = base + u * kMxThreads + threadIdx.x;
      if (i < n) v[u] = reinterpret_cast<const tx8*>(x)[i];
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int64_t i = base + u * kMxThreads + threadIdx.x;
      if (i >= n) break;
      float f[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] = (float)v[u][q];
      // magnitudes compare as integers: finite < infinity < NaN
      uint32_t a = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) a = max(a, __builtin_bit_cast(uint32_t, f[q]) & 0x7FFFFFFFu);
      a = max(a, (uint32_t)__shfl_xor((int)a, 1, 64));
      a = max(a, (uint32_t)__shfl_xor((int)a, 2, 64));
      const uint32_t field = a >> 23;
      const uint32_t b = field == 255 ? 255u : field > 2 ? field - 2 : 0u;
      const float scale = __builtin_bit_cast(float, b << 23);   // read by its exponent: 0 is 2^-127
      uint32_t c = 0;
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[0], f[1], scale, 0);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[2], f[3], scale, 1);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[4], f[5], scale, 2);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[6], f[7], scale, 3);
      codes[i] = b == 255 ? 0u : c;
      if ((i & 3) == 0) scales[i >> 2] = (uint8_t)b;
    }
  }
}

// 8 values (one word of codes) per lane
template <typename T, int kUnits>
__global__ void __launch_bounds__(kMxThreads)
mx4_dequantize_kernel(int64_t n, const uint32_t* __restrict__ codes,
                      const uint8_t* __restrict__ scales, T* __restrict__ out) {
  typedef T tx8 __attribute__((ext_vector_type(8)));
  for (int64_t base = (int64_t)blockIdx.x * (kMxThreads * kUnits); base < n;
       base += (int64_t)gridDim.x * (kMxThreads * kUnits)) {
    uint32_t c[kUnits], b[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int64_t i = base + u * kMxThreads + threadIdx.x;
      if (i < n) {
        c[u] = codes[i];
        b[u] = scales[i >> 2];
      }
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int64_t i = base + u * kMxThreads + threadIdx.x;
      if (i >= n) break;
      // read by its exponent: 0 is 2^-127, 255 NaN
      const float scale = __builtin_bit_cast(float, b[u] << 23);
      tx8 v;
      if constexpr (sizeof(T) == 2) {
        v = mx4_bf16x8(c[u], scale);
      } else {
        static_for<4>([&](auto Q) {
          constexpr int q = decltype(Q)::value;
          const auto two = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], scale, q);
          v[2 * q] = two[0];
          v[2 * q + 1] = two[1];
        });
      }
      reinterpret_cast<tx8*>(out)[i] = v;
    }
  }
}

// go(kernel of one or of four units, its blocks): all units at once up to 2^20 blocks
// (threads of a launch are counted in 32 bits), round by round behind that
template <typename F>
static void for_units(int64_t n, F&& go) {
  if (n < int64_t(4) * kMxThreads * 256 * 8) {
    go(std::integral_constant<int, 1>{}, dim3((unsigned)ceil_div(n, kMxThreads)));
  } else {
    go(std::integral_constant<int, 4>{},
       dim3((unsigned)std::min<int64_t>(ceil_div(n, 4 * kMxThreads), int64_t(1) << 20)));
  }
}

hipError_t launch_mx4_quantize(bool x_f32, int64_t num_rows, int64_t cols, const void* x,
                               const int32_t* rows_used, uint8_t* codes, uint8_t* scales,
                               hipStream_t stream) {
  for_units(num_rows * cols / 8, [&](auto units, dim3 grid) {
    constexpr int U = decltype(units)::value;
    uint32_t* c = reinterpret_cast<uint32_t*>(codes);
    if (x_f32)
      hipLaunchKernelGGL((mx4_quantize_kernel<float, U>), grid, dim3(kMxThreads), 0, stream, num_rows,
                         cols, static_cast<const float*>(x), rows_used, c, scales);
    else
      hipLaunchKernelGGL((mx4_quantize_kernel<bf16_t, U>), grid, dim3(kMxThreads), 0, stream,
                         num_rows, cols, static_cast<const bf16_t*>(x), rows_used, c, scales);
  });
  return hipGetLastError();
}

hipError_t launch_mx4_dequantize(bool out_f32, int64_t num_rows, int64_t cols,
                                 const uint8_t* codes, const uint8_t* scales, void* out,
                                 hipStream_t stream) {
  const int64_t n = num_rows * cols / 8;
  for_units(n, [&](auto units, dim3 grid) {
    constexpr int U = decltype(units)::value;
    const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
    if (out_f32)
      hipLaunchKernelGGL((mx4_dequantize_kernel<float, U>), grid, dim3(kMxThreads), 0, stream, n, c,
                         scales, static_cast<float*>(out));
    else
      hipLaunchKernelGGL((mx4_dequantize_kernel<bf16_t, U>), grid, dim3(kMxThreads), 0, stream, n, c,
                         scales, static_cast<bf16_t*>(out));
  });
  return hipGetLastError();
}

}  // namespace moelora
