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

// V elements at any address aligned to one of them: global memory is read and written
// 16 bytes at a time whatever the alignment, so rows of odd lengths go the same way.
// ONCE: what is touched once, the rows that unpermute reads and the tokens it writes,
// goes past the caches (fp32 rows of 8192 x 8 tokens, 2048 wide: 136 -> 93 us; the
// stores of the other direction gain nothing, its loads lose 10%).
template <typename T, int V> struct Vec {
  typedef T type __attribute__((ext_vector_type(V), aligned(sizeof(T))));
};
template <typename T> struct Vec<T, 1> { typedef T type; };

template <typename T, int V, bool ONCE = false>
__device__ __forceinline__ typename Vec<T, V>::type load_vec(const T* p) {
  const typename Vec<T, V>::type* from = reinterpret_cast<const typename Vec<T, V>::type*>(p);
  if constexpr (ONCE) return __builtin_nontemporal_load(from);
  else return *from;
}
template <typename T, int V, bool ONCE = false>
__device__ __forceinline__ void store_vec(T* p, typename Vec<T, V>::type v) {
  typename Vec<T, V>::type* to = reinterpret_cast<typename Vec<T, V>::type*>(p);
  if constexpr (ONCE) __builtin_nontemporal_store(v, to);
  else *to = v;
}
template <typename T, int V, bool ONCE = false>
__device__ __forceinline__ void load_floats(const T* p, float (&v)[V]) {
  const auto x = load_vec<T, V, ONCE>(p);
  if constexpr (V == 1) {
    v[0] = (float)x;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = (float)x[i];
  }
}
template <typename T, int V, bool ONCE = false>
__device__ __forceinline__ void store_floats(T* p, const float (&v)[V]) {
  typename Vec<T, V>::type x;
  if constexpr (V == 1) {
    x = (T)v[0];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = (T)v[i];
  }
  store_vec<T, V, ONCE>(p, x);
}
// 16 bytes of the rows to a thread; rows shorter than that, element by element
template <typename T> constexpr int kWide = 16 / (int)sizeof(T);

// A row of n elements is taken V at a time; the last piece of a row that V does not
// divide starts early, and repeats elements of the one before.
template <int V>
__device__ __forceinline__ int64_t piece_at(int64_t u, int64_t n) {
  return min(u * V, n - V);
}

// Zeroes pieces [u0, u1) of the pad rows: rows before *num_rows_padded whose entry
// names no pair, kPadRows rows of the layout per block at a time.  Rows behind it
// are not touched.
template <typename T, int V>
__device__ __forceinline__ void zero_pads(const RowsLayout& l, int64_t block, int64_t blocks,
                                          int64_t n, int64_t u0, int64_t u1, T* __restrict__ rows) {
  const int64_t used = min((int64_t)l.num_rows_padded[0], l.num_rows);
  const int64_t pairs = (int64_t)l.T * l.k;
  constexpr int kPerWave = kPadRows / (kRowThreads / 64);
  for (int64_t r0 = block * kPadRows; r0 < used; r0 += blocks * kPadRows) {
    bool pad[kPerWave];
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      const int64_t r = r0 + (threadIdx.x >> 6) * kPerWave + i;
      const int32_t id = l.sorted_ids[min(r, used - 1)];
      pad[i] = r < used && (id < 0 || id >= pairs);
    }
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      const int64_t r = r0 + (threadIdx.x >> 6) * kPerWave + i;
      if (!pad[i]) continue;
      for (int64_t u = u0 + (threadIdx.x & 63); u < u1; u += 64)
        store_vec<T, V>(rows + r * n + piece_at<V>(u, n), typename Vec<T, V>::type{});
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
// takes kRowThreads * PER pieces of the row.
template <typename T, int V, int PER>
__global__ void __launch_bounds__(kRowThreads)
permute_kernel(RowsLayout l, unsigned tblocks, int64_t n, const T* __restrict__ x,
               T* __restrict__ rows) {
  const int64_t units = (n + V - 1) / V;
  const int64_t u0 = (int64_t)blockIdx.y * (kRowThreads * PER);
  if (blockIdx.x >= tblocks) {
    zero_pads<T, V>(l, blockIdx.x - tblocks, gridDim.x - tblocks, n, u0,
                    min(units, u0 + (int64_t)kRowThreads * PER), rows);
    return;
  }
  for (int64_t t = blockIdx.x; t < l.T; t += tblocks) {
    typename Vec<T, V>::type v[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int64_t u = u0 + i * kRowThreads + threadIdx.x;
      v[i] = {};
      if (u < units) v[i] = load_vec<T, V>(x + t * n + piece_at<V>(u, n));
    }
    // the pairs' rows are read ahead of the stores: for all the compiler knows these could
    // change them, and each would wait for the one before
    constexpr int kRowsAtOnce = 8;
    for (int j0 = 0; j0 < l.k; j0 += kRowsAtOnce) {
      int64_t to[kRowsAtOnce];
#pragma unroll
      for (int q = 0; q < kRowsAtOnce; ++q) {
        const int64_t r = l.pair_rows[t * l.k + min(j0 + q, l.k - 1)];
        to[q] = j0 + q < l.k && r < l.num_rows ? r : -1;
      }
#pragma unroll
      for (int q = 0; q < kRowsAtOnce; ++q) {
        if (to[q] < 0) continue;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int64_t u = u0 + i * kRowThreads + threadIdx.x;
          if (u < units) store_vec<T, V>(rows + to[q] * n + piece_at<V>(u, n), v[i]);
        }
      }
    }
  }
}

// V columns per thread; a token's rows are loaded kRowsAtOnce at a time, all in flight
// before the first is added.
template <typename TR, typename TY, int V>
__global__ void __launch_bounds__(kRowThreads)
unpermute_kernel(RowsLayout l, int64_t hidden, const TR* __restrict__ rows,
                 const float* __restrict__ weights, TY* __restrict__ y) {
  constexpr int kRowsAtOnce = 8;
  int64_t c = ((int64_t)blockIdx.y * kRowThreads + threadIdx.x) * V;
  if (c >= hidden) return;
  c = min(c, hidden - V);   // the last piece of an odd row repeats columns
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
          if (live[q]) load_floats<TR, V, true>(rows + r * hidden + c, z[q]);
        }
      }
#pragma unroll
      for (int q = 0; q < kRowsAtOnce; ++q)
        if (live[q]) {
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] = fmaf(w[q], z[q][i], acc[i]);
        }
    }
    store_floats<TY, V, true>(y + t * hidden + c, acc);
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
    zero_pads<TR, V>(l, blockIdx.x - tblocks, gridDim.x - tblocks, hidden, 0, (hidden + V - 1) / V,
                     d_rows);
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
      for (int64_t c0 = (int64_t)threadIdx.x * V; c0 < hidden; c0 += kRowThreads * V) {
        const int64_t c = min(c0, hidden - V);
        float g[V], z[kRowsAtOnce][V];
        load_floats<TY, V>(dy + t * hidden + c, g);
        if (d_weights) {
#pragma unroll
          for (int q = 0; q < kRowsAtOnce; ++q)
            if (at[q] >= 0) load_floats<TR, V>(rows + at[q] + c, z[q]);
        }
#pragma unroll
        for (int q = 0; q < kRowsAtOnce; ++q) {
          if (at[q] < 0) continue;
          float d[V];
#pragma unroll
          for (int i = 0; i < V; ++i) d[i] = w[q] * g[i];
          store_floats<TR, V>(d_rows + at[q] + c, d);
          if (d_weights) {
            // columns that the last piece repeats are counted once
#pragma unroll
            for (int i = 0; i < V; ++i)
              if (V == 1 || c + i >= c0) dot[q] = fmaf(g[i], z[q][i], dot[q]);
          }
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

template <typename T>
static void permute_elements(const RowsLayout& l, int64_t n, const void* x, void* rows,
                             hipStream_t stream) {
  auto go = [&](auto v, auto per) {
    constexpr int V = decltype(v)::value, PER = decltype(per)::value;
    const dim3 grid(token_blocks(l) + pad_blocks(l), (unsigned)ceil_div(n, V * kRowThreads * PER));
    hipLaunchKernelGGL((permute_kernel<T, V, PER>), grid, dim3(kRowThreads), 0, stream, l,
                       token_blocks(l), n, static_cast<const T*>(x), static_cast<T*>(rows));
  };
  if (n >= kWide<T>) go(std::integral_constant<int, kWide<T>>{}, std::integral_constant<int, 4>{});
  else go(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
}

hipError_t launch_permute(const RowsLayout& l, int64_t hidden, int elem_bytes, const void* x,
                          void* rows, hipStream_t stream) {
  if (elem_bytes == 4) permute_elements<uint32_t>(l, hidden, x, rows, stream);
  else if (elem_bytes == 2) permute_elements<uint16_t>(l, hidden, x, rows, stream);
  else permute_elements<uint8_t>(l, hidden, x, rows, stream);
  return hipGetLastError();
}

// f(TR{}, TY{}, V) for the element types of the rows and of the tokens, and the columns
// that a thread takes
template <typename F>
static void for_types(bool rows_f32, bool y_f32, int64_t hidden, F&& f) {
  auto width = [&](auto tr, auto ty) {
    constexpr int V = kWide<decltype(tr)>;
    if (hidden >= V) f(tr, ty, std::integral_constant<int, V>{});
    else f(tr, ty, std::integral_constant<int, 1>{});
  };
  if (rows_f32) {
    if (y_f32) width(float{}, float{});
    else width(float{}, bf16_t{});
  } else {
    if (y_f32) width(bf16_t{}, float{});
    else width(bf16_t{}, bf16_t{});
  }
}

hipError_t launch_unpermute(const RowsLayout& l, int64_t hidden, bool rows_f32, bool y_f32,
                            const void* rows, const float* weights, void* y, hipStream_t stream) {
  for_types(rows_f32, y_f32, hidden, [&](auto tr, auto ty, auto v) {
    using TR = decltype(tr);
    using TY = decltype(ty);
    constexpr int V = decltype(v)::value;
    const dim3 grid(token_blocks(l), (unsigned)ceil_div(hidden, kRowThreads * V));
    hipLaunchKernelGGL((unpermute_kernel<TR, TY, V>), grid, dim3(kRowThreads), 0, stream, l, hidden,
                       static_cast<const TR*>(rows), weights, static_cast<TY*>(y));
  });
  return hipGetLastError();
}

hipError_t launch_unpermute_backward(const RowsLayout& l, int64_t hidden, bool rows_f32,
                                     bool dy_f32, const void* dy, const void* rows,
                                     const float* weights, void* d_rows, float* d_weights,
                                     hipStream_t stream) {
  for_types(rows_f32, dy_f32, hidden, [&](auto tr, auto ty, auto v) {
    using TR = decltype(tr);
    using TY = decltype(ty);
    constexpr int V = decltype(v)::value;
    const dim3 grid(token_blocks(l) + pad_blocks(l));
    hipLaunchKernelGGL((unpermute_backward_kernel<TR, TY, V>), grid, dim3(kRowThreads), 0, stream, l,
                       token_blocks(l), hidden, static_cast<const TY*>(dy),
                       static_cast<const TR*>(rows), weights, static_cast<TR*>(d_rows), d_weights);
  });
  return hipGetLastError();
}

}  // namespace moelora
