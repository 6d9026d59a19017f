// 8-bit integers with one scale for each row, for the products of int8_gemm.hip:
//
//   quantize   s = max |v| / 127 rounded to fp32,  code = round(v / s), ties to even
//   dequantize code * s
//   norm       h = x + residual,  n = h * weight / sqrt(mean(h^2) + eps),  n quantized;
//              h and n themselves on request
//
// The integers are those of the formula to the bit: next to the border of two of them the
// quotient of fp32 values is not decided by an fp32 quotient, so from the sums of squares on
// all is fp64, whose units (half the fp32 rate) have time to spare under these kernels, which
// memory bounds.  A row with an infinity or a NaN gets the scale NaN and codes 0, a row of
// zeros (or one whose scale is below fp32) the scale 0 and codes 0.
//
// A row is read once: its threads keep it in registers between the maximum and the codes.  In
// the norm max |n| = max |h weight| / sqrt(..), so one exchange between the threads gives the
// sum of squares and the maximum together.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "kernels.hpp"
#include "vec.hpp"
#include "wave.hpp"

namespace moelora {

static constexpr double kCodes = 127.0;

// scale of a row with largest magnitude `top`, and what its values are multiplied by to become
// codes (0 where all codes are 0)
struct RowScale {
  float scale;
  double per;
  bool clamp;
};
__device__ __forceinline__ RowScale row_scale(double top) {
  RowScale s;
  s.scale = (float)(top / kCodes);
  s.per = s.scale > 0.0f ? 1.0 / (double)s.scale : 0.0;
  if (!(top < __builtin_inf())) s = {__builtin_nanf(""), 0.0, false};
  s.clamp = s.scale < 0x1p-126f;
  return s;
}

// Nearest integer of v * per, in the low bits of what is returned.  SNAP, for the quotient of two
// fp32 values by per = the rounded 1 / scale: that quotient is half an integer or at least 2^-27
// away from one, so rounded to multiples of 2^-36 first it is what the exact one would be.  The
// rounding is that of additions: ties to even.
template <bool SNAP>
__device__ __forceinline__ uint32_t code_of(double v, double per) {
  constexpr double kSnap = 1.5 * 65536.0;              // its last bit is 2^-36
  constexpr double kInt = 1.5 * 4503599627370496.0;    // its last bit is 1
  const double q = SNAP ? __builtin_fma(v, per, kSnap) + (kInt - kSnap) : __builtin_fma(v, per, kInt);
  return (uint32_t)__builtin_bit_cast(uint64_t, q);
}

// The codes of a piece.  A scale below fp32's normal numbers is that much off that codes past 127
// come out (clamp).
template <int V, typename F>
__device__ __forceinline__ void store_codes(int8_t* to, bool clamp, F&& code) {
  uint32_t c[V];
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = code(i);
  if (clamp) {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = (uint32_t)min(max((int32_t)c[i], -127), 127);
  }
  if constexpr (V == 1) {
    *to = (int8_t)c[0];
  } else {
    typedef uint32_t words __attribute__((ext_vector_type(V / 4), aligned(1)));
    words w;
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const uint32_t lo = __builtin_amdgcn_perm(c[4 * i + 1], c[4 * i], 0x0C0C0400);
      const uint32_t hi = __builtin_amdgcn_perm(c[4 * i + 3], c[4 * i + 2], 0x04000C0C);
      const uint32_t both = lo | hi;
      if constexpr (V == 4) w = both;
      else w[i] = both;
    }
    __builtin_memcpy(to, &w, V);
  }
}

// The largest of `top` and the sum of `sum` over the G threads of a row (over all waves of the
// workgroup if G is more than a wave).  `buf`: a set of two, taken in turn, so that one barrier a
// row is enough.
template <int G, typename M>
__device__ __forceinline__ void over_row(M& top, double& sum, bool with_sum, uint64_t (*buf)[2]) {
  top = wave_max(top, M(0));
  if (with_sum) sum = wave_sum(sum);
  if constexpr (G > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      buf[wave][0] = top;
      buf[wave][1] = __builtin_bit_cast(uint64_t, sum);
    }
    __syncthreads();
    top = (M)buf[0][0];
    sum = __builtin_bit_cast(double, buf[0][1]);
#pragma unroll
    for (int w = 1; w < G / 64; ++w) {
      top = max(top, (M)buf[w][0]);
      if (with_sum) sum += __builtin_bit_cast(double, buf[w][1]);
    }
  }
}

// What comes behind does not see through to where `v` was used before: it converts again what the
// compiler would otherwise keep as fp64 from the first use on (256 registers instead of 90).
template <typename P>
__device__ __forceinline__ void forget(P& v) {
  if constexpr (sizeof(P) == 16) {
    typedef uint32_t words __attribute__((ext_vector_type(4)));
    words b = __builtin_bit_cast(words, v);
    asm volatile("" : "+v"(b));
    v = __builtin_bit_cast(P, b);
  }
}

// G threads to a row of n elements, U pieces of V elements to a thread.
template <typename T, int V, int G, int U, bool NORM>
__global__ void __launch_bounds__(G > 256 ? G : 256)
int8_rows_kernel(Int8Rows p) {
  constexpr int kPer = (G > 256 ? G : 256) / G;   // rows of a workgroup
  __shared__ uint64_t buf[2][G / 64][2];
  // a row's base is uniform and its places are 32 bits: an address of 64 bits for each piece of
  // each array would cost half the waves
  const uint32_t n = (uint32_t)p.cols, lane = threadIdx.x % G;
  const int64_t rows = p.rows_used ? min((int64_t)max(p.rows_used[0], 0), p.num_rows) : p.num_rows;
  auto in_row = [&](int u) { return (lane + u * G) * V < n; };
  auto place = [&](int u) { return min((lane + u * G) * V, n - V); };
  auto elem = [](const typename Vec<T, V>::type& v, int i) -> float {
    if constexpr (V == 1) return (float)v;
    else return (float)v[i];
  };
  // every thread of a workgroup goes through the same rounds: there is a barrier in each
  int turn = 0;
  for (int64_t first = (int64_t)blockIdx.x * kPer; first < rows; first += (int64_t)gridDim.x * kPer, turn ^= 1) {
    const int64_t row = first + (kPer > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / G) : 0);
    if (kPer > 1 && row >= rows) return;   // a whole wave, and no barrier with G = 64
    const T* const x = static_cast<const T*>(p.x) + row * n;
    typename Vec<T, V>::type vx[U], vr[NORM ? U : 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (in_row(u)) vx[u] = load_vec<T, V>(x + place(u));
    }
    if constexpr (NORM) {
#pragma unroll
      for (int u = 0; u < U; ++u) vr[u] = {};
      if (p.residual) {
        const T* const res = static_cast<const T*>(p.residual) + row * n;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (in_row(u)) vr[u] = load_vec<T, V>(res + place(u));
        }
      }
    }
    auto h_of = [&](int u, int i) -> double {
      const double h = (double)elem(vx[u], i);
      if constexpr (NORM) return h + (double)elem(vr[u], i);
      return h;
    };
    // The weights stay in the L1: in registers over the rows they would cost waves.
    float w[V];
    uint32_t again = 0;   // for the second time: not known to be 0
    auto weights = [&](int u) {
      if constexpr (NORM) {
        if (p.weight_f32) load_floats<float, V>(static_cast<const float*>(p.weight) + (place(u) + again), w);
        else load_floats<bf16_t, V>(static_cast<const bf16_t*>(p.weight) + (place(u) + again), w);
      }
    };
    // what is quantized, but for the factor 1 / sqrt(..) of the row
    auto value = [&](int u, int i) -> double {
      if constexpr (NORM) return h_of(u, i) * (double)w[i];
      return h_of(u, i);
    };
    // magnitudes as integers: finite < infinity < NaN
    typename std::conditional<NORM, uint64_t, uint32_t>::type top = 0;
    double sum = 0.0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!in_row(u)) continue;
      weights(u);
      // elements that the last piece of a row repeats
      const int twice = (int)((lane + u * G) * V - place(u));
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (NORM) {
          top = max(top, __builtin_bit_cast(uint64_t, value(u, i)) & ~(uint64_t(1) << 63));
          const double h = h_of(u, i);
          if (V == 1 || i >= twice) sum = __builtin_fma(h, h, sum);
        } else {
          top = max(top, __builtin_bit_cast(uint32_t, elem(vx[u], i)) & 0x7FFFFFFFu);
        }
      }
    }
    over_row<G>(top, sum, NORM, buf[turn]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      forget(vx[u]);
      if constexpr (NORM) forget(vr[u]);
    }
    asm volatile("" : "+s"(again));
    double norm = 1.0;
    if constexpr (NORM) norm = 1.0 / __builtin_sqrt(sum / (double)n + p.eps);
    RowScale s;
    if constexpr (NORM) s = row_scale(__builtin_bit_cast(double, top) * norm);
    else s = row_scale((double)__builtin_bit_cast(float, top));
    const double per = NORM ? norm * s.per : s.per;
    if (lane == 0) p.scales[row] = s.scale;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!in_row(u)) continue;
      weights(u);
      store_codes<V>(p.codes + row * n + place(u), s.clamp, [&](int i) {
        return s.per > 0.0 ? code_of<!NORM>(value(u, i), per) : 0;
      });
      if constexpr (NORM) {
        float out[V];
        if (p.residual_out) {
#pragma unroll
          for (int i = 0; i < V; ++i) out[i] = elem(vx[u], i) + elem(vr[u], i);
          store_floats<T, V>(static_cast<T*>(p.residual_out) + row * n + place(u), out);
        }
        if (p.y) {
#pragma unroll
          for (int i = 0; i < V; ++i) out[i] = (float)(value(u, i) * norm);
          if (p.y_f32) store_floats<float, V>(static_cast<float*>(p.y) + row * n + place(u), out);
          else store_floats<bf16_t, V>(static_cast<bf16_t*>(p.y) + row * n + place(u), out);
        }
      }
    }
  }
}

// Rows that registers do not hold: read a second time for the codes.
template <typename T, int V>
__global__ void __launch_bounds__(1024) int8_long_rows_kernel(Int8Rows p) {
  __shared__ uint64_t buf[2][16][2];
  const int64_t n = p.cols, units = (n + V - 1) / V;
  const int64_t rows = p.rows_used ? min((int64_t)max(p.rows_used[0], 0), p.num_rows) : p.num_rows;
  const T* const x = static_cast<const T*>(p.x);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
    uint32_t top = 0;
    for (int64_t u = threadIdx.x; u < units; u += 1024) {
      float v[V];
      load_floats<T, V>(x + row * n + piece_at<V>(u, n), v);
#pragma unroll
      for (int i = 0; i < V; ++i) top = max(top, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
    }
    double none = 0.0;
    over_row<1024>(top, none, false, buf[turn]);
    const RowScale s = row_scale((double)__builtin_bit_cast(float, top));
    if (threadIdx.x == 0) p.scales[row] = s.scale;
    for (int64_t u = threadIdx.x; u < units; u += 1024) {
      const int64_t at = row * n + piece_at<V>(u, n);
      float v[V];
      load_floats<T, V>(x + at, v);
      store_codes<V>(p.codes + at, s.clamp,
                     [&](int i) { return s.per > 0.0 ? code_of<true>((double)v[i], s.per) : 0; });
    }
  }
}

// blocks of one launch: enough to fill the chip, so that a workgroup keeps the norm's weights
// over its rows
static unsigned row_blocks(int64_t num_rows, int per, int waves) {
  return (unsigned)std::min<int64_t>(ceil_div(num_rows, per), 256 * 32 / waves);
}

template <typename T, bool NORM>
static hipError_t launch_rows(const Int8Rows& p, hipStream_t stream) {
  constexpr int V = kWide<T>;
  auto go = [&](auto kernel, int threads, int per) {
    hipLaunchKernelGGL(kernel, dim3(row_blocks(p.num_rows, per, threads / 64)), dim3(threads), 0, stream, p);
    return hipGetLastError();
  };
  const int64_t units = ceil_div(p.cols, V);
  if (p.cols < V) return go(int8_rows_kernel<T, 1, 64, 1, NORM>, 256, 4);
  if (units <= 64) return go(int8_rows_kernel<T, V, 64, 1, NORM>, 256, 4);
  if (units <= 128) return go(int8_rows_kernel<T, V, 64, 2, NORM>, 256, 4);
  if (units <= 256) return go(int8_rows_kernel<T, V, 256, 1, NORM>, 256, 1);
  if (units <= 512) return go(int8_rows_kernel<T, V, 256, 2, NORM>, 256, 1);
  if (units <= 1024) return go(int8_rows_kernel<T, V, 256, 4, NORM>, 256, 1);
  if (units <= 4096) return go(int8_rows_kernel<T, V, 1024, 4, NORM>, 1024, 1);
  if constexpr (!NORM) return go(int8_long_rows_kernel<T, V>, 1024, 1);
  return hipErrorInvalidValue;
}

hipError_t launch_int8_rows(const Int8Rows& p, hipStream_t stream) {
  if (p.weight) return p.x_f32 ? launch_rows<float, true>(p, stream) : launch_rows<bf16_t, true>(p, stream);
  return p.x_f32 ? launch_rows<float, false>(p, stream) : launch_rows<bf16_t, false>(p, stream);
}

static constexpr int kFlatThreads = 256;

// V codes to a thread.  Threads of a launch lie `step` apart, step_rows rows and step_units
// pieces, so that only the first place takes a division.
template <typename T, int V>
__global__ void __launch_bounds__(kFlatThreads)
int8_dequantize_kernel(int64_t num_rows, int64_t n, int64_t units, int64_t step_rows, int64_t step_units,
                       const int8_t* __restrict__ codes, const float* __restrict__ scales,
                       T* __restrict__ out) {
  const int64_t first = (int64_t)blockIdx.x * kFlatThreads + threadIdx.x;
  int64_t row = first / units, unit = first - row * units;
  while (row < num_rows) {
    const int64_t at = row * n + piece_at<V>(unit, n);
    const float s = scales[row];
    float v[V];
    load_floats<int8_t, V>(codes + at, v);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] *= s;
    store_floats<T, V>(out + at, v);
    row += step_rows;
    unit += step_units;
    if (unit >= units) {
      unit -= units;
      ++row;
    }
  }
}

hipError_t launch_int8_dequantize(bool out_f32, int64_t num_rows, int64_t cols, const int8_t* codes,
                                  const float* scales, void* out, hipStream_t stream) {
  auto go = [&](auto kernel, auto* to, int V) {
    const int64_t units = ceil_div(cols, V);
    const int64_t blocks = std::min<int64_t>(ceil_div(num_rows * units, kFlatThreads), 256 * 32);
    const int64_t step = blocks * kFlatThreads;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kFlatThreads), 0, stream, num_rows, cols, units,
                       step / units, step % units, codes, scales, to);
    return hipGetLastError();
  };
  float* f = static_cast<float*>(out);
  bf16_t* b = static_cast<bf16_t*>(out);
  if (cols < 8) return out_f32 ? go(int8_dequantize_kernel<float, 1>, f, 1) : go(int8_dequantize_kernel<bf16_t, 1>, b, 1);
  return out_f32 ? go(int8_dequantize_kernel<float, 8>, f, 8) : go(int8_dequantize_kernel<bf16_t, 8>, b, 8);
}

}  // namespace moelora
