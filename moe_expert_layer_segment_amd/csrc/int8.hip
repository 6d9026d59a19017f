// 8-bit integers with one scale for each row, for the products of int8_gemm.hip:
//
//   quantize   s = max |v| / 127 rounded to fp32,  code = round(v / s), ties to even
//   dequantize code * s
//   norm       h = x + residual,  n = h * weight / sqrt(mean(h^2) + eps),  n quantized;
//              h and n themselves on request
//
// The integers of a quantisation are those of the formula to the bit: next to the border of two of
// them the quotient of fp32 values is not decided by an fp32 quotient.  The norm is not a quotient
// of fp32 values; its integers are those of the formula in fp64, but within 1e-9 of a border.  So all
// from the sums of squares on is fp64, whose units (half the fp32 rate) have time to spare under
// these kernels, which memory bounds.  What is stored as bf16 is rounded to fp32 first.  A row with an
// infinity or a NaN gets the scale NaN and codes 0, a row of zeros (or one whose scale is below fp32)
// the scale 0 and codes 0.
//
// A row is read once: its threads keep it in registers between the maximum and the codes.  In
// the norm max |n| = max |h weight| / sqrt(..), so one exchange between the threads gives the
// sum of squares and the maximum together.
//
// Memory bounds all three: 229376 x 4096 bf16 quantized in 495 us (5.7 TB/s) and dequantized in 587
// (4.8), the norm of 16384 x 7168 bf16 with its sum, h and n in 200 (5.3); the card copies at 5.1
// and adds two arrays into a third at 6.0.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "kernels.hpp"
#include "vec.hpp"
#include "wave.hpp"

namespace moelora {

// 1 / sqrt(v), as reciprocal of common.hpp.  (Every wave of a row works them out: as quotients and a
// root of fp64 they took 16384 x 7168 from 215 to 228 us.)
__device__ __forceinline__ double reciprocal_root(double v) {
  double r = __builtin_amdgcn_rsq(v);
#pragma unroll
  for (int i = 0; i < 2; ++i) r = __builtin_fma(__builtin_fma(-v * r, r, 1.0), 0.5 * r, r);
  return r;
}

// scale of a row, what its values are multiplied by to become codes (0 where all codes are 0),
// and whether codes past 127 may come out: a scale below fp32's normal numbers is that much off
struct RowScale {
  float scale;
  double per;
  bool clamp;
};
// of scale = largest magnitude / 127; not finite: `top` was not
__device__ __forceinline__ RowScale row_scale(float scale, bool finite) {
  RowScale s;
  s.scale = finite ? scale : __builtin_nanf("");
  s.per = s.scale > 0.0f ? reciprocal((double)s.scale) : 0.0;
  s.clamp = s.scale < 0x1p-126f;
  return s;
}
__device__ __forceinline__ RowScale row_scale_of(uint32_t top) {   // magnitude as an integer
  return row_scale(__builtin_bit_cast(float, top) / 127.0f, top < 0x7F800000u);
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

// The codes of a piece
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
    // every wave's, one to a lane: all of them in a thread are 64 registers of a large workgroup
    const int lane = threadIdx.x & 63;
    const bool in = lane < G / 64;
    top = wave_max(in ? (M)buf[lane % (G / 64)][0] : M(0), M(0));
    if (with_sum) sum = wave_sum(in ? __builtin_bit_cast(double, buf[lane % (G / 64)][1]) : 0.0);
  }
}

// What comes behind does not see through to where `v` was used before: bf16 is widened again where
// the compiler would keep it as fp32, in twice the registers, from the first use on (a row of 4096
// to a wave: 76 registers, and 667 us instead of 535 for 229376 rows).
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
template <typename T, int V, int G, int U>
__global__ void __launch_bounds__(G > 256 ? G : 256)
int8_rows_kernel(Int8Rows p) {
  constexpr int kPer = (G > 256 ? G : 256) / G;   // rows of a workgroup
  __shared__ uint64_t buf[2][G / 64][2];
  // a row's base is uniform and its places are 32 bits
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
    typename Vec<T, V>::type v[U];
    uint32_t top = 0;   // magnitudes as integers: finite < infinity < NaN
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (in_row(u)) v[u] = load_vec<T, V>(x + place(u));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!in_row(u)) continue;
#pragma unroll
      for (int i = 0; i < V; ++i) top = max(top, __builtin_bit_cast(uint32_t, elem(v[u], i)) & 0x7FFFFFFFu);
    }
    double none = 0.0;
    over_row<G>(top, none, false, buf[turn]);
#pragma unroll
    for (int u = 0; u < U; ++u) forget(v[u]);
    const RowScale s = row_scale_of(top);
    if (lane == 0) p.scales[row] = s.scale;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!in_row(u)) continue;
      store_codes<V>(p.codes + row * n + place(u), s.clamp,
                     [&](int i) { return s.per > 0.0 ? code_of<true>((double)elem(v[u], i), s.per) : 0; });
    }
  }
}

// The same of the norm.  h * weight stays in registers, as fp64, from the sums to the codes: made
// again from x and the residual it costs as much as all that follows (16384 x 7168: 247 -> 229 us).
template <typename T, int V, int G, int U>
__global__ void __launch_bounds__(G > 256 ? G : 256)
int8_norm_kernel(Int8Rows p) {
  constexpr int kPer = (G > 256 ? G : 256) / G;
  __shared__ uint64_t buf[2][G / 64][2];
  const uint32_t n = (uint32_t)p.cols, lane = threadIdx.x % G;
  auto in_row = [&](int u) { return (lane + u * G) * V < n; };
  auto place = [&](int u) { return min((lane + u * G) * V, n - V); };
  int turn = 0;
  for (int64_t first = (int64_t)blockIdx.x * kPer; first < p.num_rows;
       first += (int64_t)gridDim.x * kPer, turn ^= 1) {
    const int64_t row = first + (kPer > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / G) : 0);
    if (kPer > 1 && row >= p.num_rows) return;
    const T* const x = static_cast<const T*>(p.x) + row * n;
    typename Vec<T, V>::type vx[U], vr[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (in_row(u)) vx[u] = load_vec<T, V>(x + place(u));
#pragma unroll
    for (int u = 0; u < U; ++u) vr[u] = {};
    if (p.residual) {
      const T* const res = static_cast<const T*>(p.residual) + row * n;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (in_row(u)) vr[u] = load_vec<T, V>(res + place(u));
    }
    // Where residual_out is the residual (or x) the last piece of a row may repeat elements that
    // another wave is about to change.
    if (G > 64 && p.residual_out && n % V) __syncthreads();
    double value[U][V];   // what is quantized, but for the factor 1 / sqrt(..) of the row
    uint64_t top = 0;
    double sum = 0.0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!in_row(u)) continue;
      float fx[V], fr[V], w[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (V == 1) {
          fx[i] = (float)vx[u];
          fr[i] = (float)vr[u];
        } else {
          fx[i] = (float)vx[u][i];
          fr[i] = (float)vr[u][i];
        }
      }
      if (p.weight_f32) load_floats<float, V>(static_cast<const float*>(p.weight) + place(u), w);
      else load_floats<bf16_t, V>(static_cast<const bf16_t*>(p.weight) + place(u), w);
      // elements that the last piece of a row repeats
      const int twice = (int)((lane + u * G) * V - place(u));
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const double h = (double)fx[i] + (double)fr[i];
        value[u][i] = h * (double)w[i];
        top = max(top, __builtin_bit_cast(uint64_t, value[u][i]) & ~(uint64_t(1) << 63));
        if (V == 1 || i >= twice) sum = __builtin_fma(h, h, sum);
      }
      if (p.residual_out) {
#pragma unroll
        for (int i = 0; i < V; ++i) fx[i] += fr[i];
        store_floats<T, V>(static_cast<T*>(p.residual_out) + row * n + place(u), fx);
      }
      if constexpr (G * U > 2048) {   // 128 registers: piece after piece, and not all widened first
        for (int q = u + 1; q < U; ++q) {
          forget(vx[q]);
          forget(vr[q]);
        }
        asm volatile("" : "+v"(top), "+v"(sum));
      }
    }
    over_row<G>(top, sum, true, buf[turn]);
    const double square = sum * p.per_col + p.eps;
    // 0, infinite and NaN sums have no steps to take
    const double norm = square > 0.0 && square < __builtin_inf() ? reciprocal_root(square) : 1.0 / __builtin_sqrt(square);
    const double most = __builtin_bit_cast(double, top) * norm;
    const RowScale s = row_scale((float)(most * (1.0 / 127.0)), most < __builtin_inf());
    const double per = norm * s.per;
    if (lane == 0) p.scales[row] = s.scale;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!in_row(u)) continue;
      store_codes<V>(p.codes + row * n + place(u), s.clamp,
                     [&](int i) { return s.per > 0.0 ? code_of<false>(value[u][i], per) : 0; });
      if (p.y) {
        float out[V];
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = (float)(value[u][i] * norm);
        if (p.y_f32) store_floats<float, V>(static_cast<float*>(p.y) + row * n + place(u), out);
        else store_floats<bf16_t, V>(static_cast<bf16_t*>(p.y) + row * n + place(u), out);
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
    const RowScale s = row_scale_of(top);
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

// A workgroup to every row (or four), in their order: with as many as fill the chip, each taking
// every 2048th row, 229376 rows of 4096 took 539 us instead of 512.  Threads of a launch are
// counted in 32 bits, so past 2^20 workgroups they come round again.
static unsigned row_blocks(int64_t num_rows, int per) {
  return (unsigned)std::min<int64_t>(ceil_div(num_rows, per), int64_t(1) << 20);
}

template <typename K>
static hipError_t go_rows(K kernel, int threads, int per, const Int8Rows& p, hipStream_t stream) {
  hipLaunchKernelGGL(kernel, dim3(row_blocks(p.num_rows, per)), dim3(threads), 0, stream, p);
  return hipGetLastError();
}

template <typename T>
static hipError_t launch_rows(const Int8Rows& p, hipStream_t stream) {
  constexpr int V = kWide<T>;
  const int64_t units = ceil_div(p.cols, V);
  if (p.cols < V) return go_rows(int8_rows_kernel<T, 1, 64, 1>, 256, 4, p, stream);
  if (units <= 128) return go_rows(int8_rows_kernel<T, V, 64, 2>, 256, 4, p, stream);
  // a wave to a row, so no barrier (229376 rows of 4096: 585 us with 256 threads, 535)
  if (units <= 512) return go_rows(int8_rows_kernel<T, V, 64, 8>, 256, 4, p, stream);
  if (units <= 1024) return go_rows(int8_rows_kernel<T, V, 256, 4>, 256, 1, p, stream);
  if (units <= 4096) return go_rows(int8_rows_kernel<T, V, 1024, 4>, 1024, 1, p, stream);
  return go_rows(int8_long_rows_kernel<T, V>, 1024, 1, p, stream);
}

template <typename T>
static hipError_t launch_norm(const Int8Rows& p, hipStream_t stream) {
  constexpr int V = kWide<T>;
  const int64_t units = ceil_div(p.cols, V);   // 4096 at the most
  if (p.cols < V) return go_rows(int8_norm_kernel<T, 1, 64, 1>, 256, 4, p, stream);
  if (units <= 128) return go_rows(int8_norm_kernel<T, V, 64, 2>, 256, 4, p, stream);
  if (units <= 256) return go_rows(int8_norm_kernel<T, V, 256, 1>, 256, 1, p, stream);
  if (units <= 512) return go_rows(int8_norm_kernel<T, V, 256, 2>, 256, 1, p, stream);
  if (units <= 1024) return go_rows(int8_norm_kernel<T, V, 512, 2>, 512, 1, p, stream);
  if constexpr (V == 4) {   // eights are 2048 at the most
    if (units > 2048) return go_rows(int8_norm_kernel<T, V, 1024, 4>, 1024, 1, p, stream);
  }
  return go_rows(int8_norm_kernel<T, V, 1024, 2>, 1024, 1, p, stream);
}

hipError_t launch_int8_rows(const Int8Rows& p, hipStream_t stream) {
  if (p.weight) return p.x_f32 ? launch_norm<float>(p, stream) : launch_norm<bf16_t>(p, stream);
  return p.x_f32 ? launch_rows<float>(p, stream) : launch_rows<bf16_t>(p, stream);
}

static constexpr int kFlatThreads = 256;

// V codes to a unit, 16 bytes of values.  Threads lie step_rows rows and step_units units apart,
// so that only the first place takes a division.  (Four units at once to a thread: 61 -> 68 us for
// 16384 x 7168 to bf16.  Stores past the caches, which leave the codes in them: 61 -> 52.)
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
    store_floats<T, V, true>(out + at, v);
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
  if (out_f32) {
    if (cols < 4) return go(int8_dequantize_kernel<float, 1>, f, 1);
    return go(int8_dequantize_kernel<float, 4>, f, 4);
  }
  if (cols < 8) return go(int8_dequantize_kernel<bf16_t, 1>, b, 1);
  return go(int8_dequantize_kernel<bf16_t, 8>, b, 8);
}

}  // namespace moelora
