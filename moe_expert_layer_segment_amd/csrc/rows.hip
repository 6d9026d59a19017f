// Rows in expert order and back, for training and for serving.
//
//   permute            rows[r(t, j)] = x[t]
//   its gradient       dx[t] = sum_j d_rows[r(t, j)]
//   unpermute          y[t] = sum_j w_tj rows[r(t, j)]
//   its gradients      d_rows[r(t, j)] = w_tj dy[t],  dw_tj = dy[t] . rows[r(t, j)]
//
// r(t, j) = pair_rows[t k + j] is the row of pair (t, j) in the layout of
// align, -1 for a pair that has none (its expert lives on another rank).  Two
// directions are enough: tokens spread over rows (each token row is read once
// and written k times) and rows gathered into tokens (each pair's row is read
// once).  Nothing is added through memory, so there are no atomics and the
// order of every sum is fixed: j ascending, in fp32, rounded once at the end.
// All of it is bound by memory.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "kernels.hpp"

namespace moelora {

static constexpr int kRowThreads = 256;
static constexpr int kPadRows = 16;   // rows of the layout a pad block looks at, at a time
// blocks of one launch: its threads are counted in 32 bits, so tokens and pads
// past these are taken in further rounds of the same blocks
static constexpr int64_t kTokenBlocks = int64_t(1) << 22;
static constexpr int64_t kPadBlocks = int64_t(1) << 20;

template <typename T, int V> struct Vec { typedef T type __attribute__((ext_vector_type(V))); };
template <typename T> struct Vec<T, 1> { typedef T type; };

template <typename T, int V>
__device__ __forceinline__ void load_floats(const T* p, float (&v)[V]) {
  const typename Vec<T, V>::type x = *reinterpret_cast<const typename Vec<T, V>::type*>(p);
  if constexpr (V == 1) {
    v[0] = (float)x;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = (float)x[i];
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_floats(T* p, const float (&v)[V]) {
  typename Vec<T, V>::type x;
  if constexpr (V == 1) {
    x = (T)v[0];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = (T)v[i];
  }
  *reinterpret_cast<typename Vec<T, V>::type*>(p) = x;
}

// Zeroes units [u0, u1) of the pad rows: rows before *num_rows_padded whose entry
// names no pair, kPadRows rows of the layout per block at a time.  Rows behind it
// are not touched.
template <typename U>
__device__ __forceinline__ void zero_pads(const RowsLayout& l, int64_t block, int64_t blocks,
                                          int64_t units, int64_t u0, int64_t u1,
                                          U* __restrict__ rows) {
  const int64_t used = min((int64_t)l.num_rows_padded[0], l.num_rows);
  const int64_t pairs = (int64_t)l.T * l.k;
  constexpr int kPerWave = kPadRows / (kRowThreads / 64);
  for (int64_t r0 = block * kPadRows; r0 < used; r0 += blocks * kPadRows) {
    for (int i = 0; i < kPerWave; ++i) {
      const int64_t r = r0 + (threadIdx.x >> 6) * kPerWave + i;
      if (r >= used) break;
      const int32_t id = l.sorted_ids[r];
      if (id >= 0 && id < pairs) continue;
      for (int64_t u = u0 + (threadIdx.x & 63); u < u1; u += 64) rows[r * units + u] = U{};
    }
  }
}

static unsigned token_blocks(const RowsLayout& l) {
  return (unsigned)std::min<int64_t>(l.T, kTokenBlocks);
}
static unsigned pad_blocks(const RowsLayout& l) {
  return (unsigned)std::min<int64_t>(ceil_div(l.num_rows, kPadRows), kPadBlocks);
}

// Blocks [0, tblocks): a token each; blocks behind them: the pads.  blockIdx.y
// takes kRowThreads * PER units of the row.
template <typename U, int PER>
__global__ void __launch_bounds__(kRowThreads)
permute_kernel(RowsLayout l, unsigned tblocks, int64_t units, const U* __restrict__ x,
               U* __restrict__ rows) {
  const int64_t u0 = (int64_t)blockIdx.y * (kRowThreads * PER);
  if (blockIdx.x >= tblocks) {
    zero_pads<U>(l, blockIdx.x - tblocks, gridDim.x - tblocks, units, u0,
                 min(units, u0 + (int64_t)kRowThreads * PER), rows);
    return;
  }
  for (int64_t t = blockIdx.x; t < l.T; t += tblocks) {
    U v[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int64_t u = u0 + i * kRowThreads + threadIdx.x;
      v[i] = u < units ? x[t * units + u] : U{};
    }
    for (int j = 0; j < l.k; ++j) {
      const int64_t r = l.pair_rows[t * l.k + j];
      if (r < 0 || r >= l.num_rows) continue;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int64_t u = u0 + i * kRowThreads + threadIdx.x;
        if (u < units) rows[r * units + u] = v[i];
      }
    }
  }
}

// One unit of V columns per thread; a token's rows are loaded kRowsAtOnce at a
// time, all in flight before the first is added.
template <typename TR, typename TY, int V>
__global__ void __launch_bounds__(kRowThreads)
unpermute_kernel(RowsLayout l, int64_t hidden, const TR* __restrict__ rows,
                 const float* __restrict__ weights, TY* __restrict__ y) {
  constexpr int kRowsAtOnce = 8;
  const int64_t c = ((int64_t)blockIdx.y * kRowThreads + threadIdx.x) * V;
  if (c >= hidden) return;
  for (int64_t t = blockIdx.x; t < l.T; t += gridDim.x) {
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < l.k; j0 += kRowsAtOnce) {
      float z[kRowsAtOnce][V];
      float w[kRowsAtOnce];
      bool live[kRowsAtOnce];
#pragma unroll
      for (int q = 0; q < kRowsAtOnce; ++q) {
        live[q] = false;
        if (j0 + q < l.k) {
          const int64_t p = t * l.k + j0 + q;
          const int64_t r = l.pair_rows[p];
          live[q] = r >= 0 && r < l.num_rows;
          w[q] = weights ? weights[p] : 1.0f;
          if (live[q]) load_floats<TR, V>(rows + r * hidden + c, z[q]);
        }
      }
#pragma unroll
      for (int q = 0; q < kRowsAtOnce; ++q)
        if (live[q]) {
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] = fmaf(w[q], z[q][i], acc[i]);
        }
    }
    store_floats<TY, V>(y + t * hidden + c, acc);
  }
}

// Blocks [0, tblocks): a token each, its whole row; blocks behind them: the pads.
// Each block adds its threads' partial dots through LDS in a fixed order.
template <typename TR, typename TY, int V>
__global__ void __launch_bounds__(kRowThreads)
unpermute_backward_kernel(RowsLayout l, unsigned tblocks, int64_t hidden, const TY* __restrict__ dy,
                          const TR* __restrict__ rows, const float* __restrict__ weights,
                          TR* __restrict__ d_rows, float* __restrict__ d_weights) {
  constexpr int kRowsAtOnce = 4;
  constexpr int kWaves = kRowThreads / 64;
  __shared__ float part[kWaves][kRowsAtOnce];
  if (blockIdx.x >= tblocks) {
    zero_pads<typename Vec<TR, V>::type>(l, blockIdx.x - tblocks, gridDim.x - tblocks, hidden / V,
                                         0, hidden / V,
                                         reinterpret_cast<typename Vec<TR, V>::type*>(d_rows));
    return;
  }
  for (int64_t t = blockIdx.x; t < l.T; t += tblocks) {
    for (int j0 = 0; j0 < l.k; j0 += kRowsAtOnce) {
      int64_t at[kRowsAtOnce];
      float w[kRowsAtOnce], dot[kRowsAtOnce];
#pragma unroll
      for (int q = 0; q < kRowsAtOnce; ++q) {
        at[q] = -1;
        w[q] = 1.0f;
        dot[q] = 0.0f;
        if (j0 + q < l.k) {
          const int64_t p = t * l.k + j0 + q;
          const int64_t r = l.pair_rows[p];
          if (r >= 0 && r < l.num_rows) at[q] = r * hidden;
          if (weights) w[q] = weights[p];
        }
      }
      for (int64_t c = (int64_t)threadIdx.x * V; c < hidden; c += kRowThreads * V) {
        float g[V];
        load_floats<TY, V>(dy + t * hidden + c, g);
#pragma unroll
        for (int q = 0; q < kRowsAtOnce; ++q) {
          if (at[q] < 0) continue;
          if (d_weights) {
            float z[V];
            load_floats<TR, V>(rows + at[q] + c, z);
#pragma unroll
            for (int i = 0; i < V; ++i) dot[q] = fmaf(g[i], z[i], dot[q]);
          }
          float d[V];
#pragma unroll
          for (int i = 0; i < V; ++i) d[i] = w[q] * g[i];
          store_floats<TR, V>(d_rows + at[q] + c, d);
        }
      }
      if (!d_weights) continue;
#pragma unroll
      for (int q = 0; q < kRowsAtOnce; ++q) {
        float s = dot[q];
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off, 64);
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][q] = s;
      }
      __syncthreads();
      if (threadIdx.x < kRowsAtOnce && j0 + (int)threadIdx.x < l.k) {
        float s = 0.0f;
        for (int i = 0; i < kWaves; ++i) s += part[i][threadIdx.x];
        d_weights[t * l.k + j0 + threadIdx.x] = s;
      }
      __syncthreads();
    }
  }
}

static bool aligned(const void* p, int64_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0;
}

template <typename U>
static void permute_units(const RowsLayout& l, int64_t units, const void* x, void* rows,
                          hipStream_t stream) {
  constexpr int PER = 4;
  const dim3 grid(token_blocks(l) + pad_blocks(l), (unsigned)ceil_div(units, kRowThreads * PER));
  hipLaunchKernelGGL((permute_kernel<U, PER>), grid, dim3(kRowThreads), 0, stream, l,
                     token_blocks(l), units, static_cast<const U*>(x), static_cast<U*>(rows));
}

hipError_t launch_permute(const RowsLayout& l, int64_t row_bytes, const void* x, void* rows,
                          hipStream_t stream) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  if (row_bytes % 16 == 0 && aligned(x, 16) && aligned(rows, 16))
    permute_units<u32x4>(l, row_bytes / 16, x, rows, stream);
  else if (row_bytes % 4 == 0 && aligned(x, 4) && aligned(rows, 4))
    permute_units<uint32_t>(l, row_bytes / 4, x, rows, stream);
  else if (row_bytes % 2 == 0 && aligned(x, 2) && aligned(rows, 2))
    permute_units<uint16_t>(l, row_bytes / 2, x, rows, stream);
  else
    permute_units<uint8_t>(l, row_bytes, x, rows, stream);
  return hipGetLastError();
}

// f(TR{}, TY{}) for the element types of the rows and of the tokens
template <typename F>
static void for_types(bool rows_f32, bool y_f32, F&& f) {
  if (rows_f32) {
    if (y_f32) f(float{}, float{});
    else f(float{}, bf16_t{});
  } else {
    if (y_f32) f(bf16_t{}, float{});
    else f(bf16_t{}, bf16_t{});
  }
}

hipError_t launch_unpermute(const RowsLayout& l, int64_t hidden, bool rows_f32, bool y_f32,
                            const void* rows, const float* weights, void* y, hipStream_t stream) {
  const bool wide = hidden % 8 == 0 && aligned(rows, 16) && aligned(y, 16);
  for_types(rows_f32, y_f32, [&](auto tr, auto ty) {
    using TR = decltype(tr);
    using TY = decltype(ty);
    auto go = [&](auto v) {
      constexpr int V = decltype(v)::value;
      const dim3 grid(token_blocks(l), (unsigned)ceil_div(hidden, kRowThreads * V));
      hipLaunchKernelGGL((unpermute_kernel<TR, TY, V>), grid, dim3(kRowThreads), 0, stream, l,
                         hidden, static_cast<const TR*>(rows), weights, static_cast<TY*>(y));
    };
    if (wide) go(std::integral_constant<int, 8>{});
    else go(std::integral_constant<int, 1>{});
  });
  return hipGetLastError();
}

hipError_t launch_unpermute_backward(const RowsLayout& l, int64_t hidden, bool rows_f32,
                                     bool dy_f32, const void* dy, const void* rows,
                                     const float* weights, void* d_rows, float* d_weights,
                                     hipStream_t stream) {
  const bool wide = hidden % 8 == 0 && aligned(dy, 16) && aligned(d_rows, 16) &&
                    (!d_weights || aligned(rows, 16));
  for_types(rows_f32, dy_f32, [&](auto tr, auto ty) {
    using TR = decltype(tr);
    using TY = decltype(ty);
    auto go = [&](auto v) {
      constexpr int V = decltype(v)::value;
      const dim3 grid(token_blocks(l) + pad_blocks(l));
      hipLaunchKernelGGL((unpermute_backward_kernel<TR, TY, V>), grid, dim3(kRowThreads), 0, stream,
                         l, token_blocks(l), hidden, static_cast<const TY*>(dy),
                         static_cast<const TR*>(rows), weights, static_cast<TR*>(d_rows), d_weights);
    };
    if (wide) go(std::integral_constant<int, 8>{});
    else go(std::integral_constant<int, 1>{});
  });
  return hipGetLastError();
}

}  // namespace moelora
