// Rows of elements in pieces of 16 bytes, at any alignment.
#pragma once

#include "common.hpp"

namespace moelora {

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

}  // namespace moelora
