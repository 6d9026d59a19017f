// Pairs per expert and the balance loss of a router, and its gradient for the logits.
//
// Over the n tokens that take part (all, or those of a mask), with p_t = softmax(logits_t):
//
//   counts_e = pairs of these tokens with id e,   P_e = sum_t p_te / n
//   loss     = E / (n k) sum_e counts_e P_e       (1 where both are even)
//   d loss / d logits_te = E / (n^2 k) p_te (counts_e - sum_i p_ti counts_i)
//
// counts are constants to the gradient.  A row of logits that are all -inf has p = 0, and with
// n = 0 everything is 0.  Logits of tokens outside the mask are never read.
//
// One wave per token, experts lane, lane + 64, .. in its registers.  p is fp32, from the
// difference to the largest logit with its rounding error (two fp32 numbers); a wave adds its
// tokens up in fp64 registers, a workgroup its waves through LDS, and the workgroups' sums go
// through memory to one more that adds them in order: no atomics but integer ones on LDS, so
// results do not change from run to run.  Few tokens are one workgroup, and one launch.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "kernels.hpp"

namespace moelora {

static constexpr int kBalThreads = 1024, kBalWaves = kBalThreads / 64;
static constexpr int kBalBlocks = 128;        // whose sums the last workgroup adds
static constexpr int kBalSingle = 256;        // tokens that one workgroup takes alone

struct BalanceWs {
  double* sums;       // [blocks][E]
  int32_t* counts;    // [blocks][E]
  int32_t* valid;     // [blocks]
};
static BalanceWs balance_ws(void* ws, int64_t E) {
  BalanceWs w;
  w.sums = static_cast<double*>(ws);
  w.counts = reinterpret_cast<int32_t*>(w.sums + kBalBlocks * E);
  w.valid = w.counts + kBalBlocks * E;
  return w;
}
size_t balance_ws_bytes(int64_t T, int64_t E) {
  return T <= kBalSingle ? 16 : (size_t)kBalBlocks * ((size_t)E * 12 + 4);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
  return v;
}
template <typename F>
__device__ __forceinline__ F wave_sum(F v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// v[i]: logit of expert lane + 64 i, -inf behind the last, to its probability
template <int V>
__device__ __forceinline__ void softmax(float (&v)[V]) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = fmaxf(m, v[i]);
  m = wave_max(m);
  if (m == -INFINITY) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = v[i] == -INFINITY ? 0.0f : v[i];   // NaN stays
    return;
  }
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    // z + lo = v - m exactly where both are finite
    const float z = v[i] - m;
    const float back = z + m;
    const float lo = (v[i] - back) - ((z - (back - m)));
    const float e = expf(z);
    v[i] = lo == lo ? __builtin_fmaf(e, lo, e) : e;
    sum += v[i];
  }
  sum = wave_sum(sum);
  const float per = 1.0f / sum;
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] *= per;
}

template <typename T, int V>
__device__ __forceinline__ void load_logits(const T* row, int E, float (&v)[V]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = lane + 64 * i < E ? (float)row[lane + 64 * i] : -INFINITY;
}

struct BalanceOut {
  float* loss;
  int32_t* counts;
  float* mean_probs;
  int32_t* num_valid;
};

// loss from the sums: every thread of the workgroup, experts threadIdx.x, + kBalThreads, ..
__device__ __forceinline__ void finish(int E, int k, int32_t n, const double* sums, const int32_t* counts,
                                       const BalanceOut& out, double (*part)) {
  double dot = 0.0;
  for (int e = threadIdx.x; e < E; e += kBalThreads) {
    const double mean = n > 0 ? sums[e] / (double)n : 0.0;
    out.mean_probs[e] = (float)mean;
    out.counts[e] = counts[e];
    dot += (double)counts[e] * mean;
  }
  dot = wave_sum(dot);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
  __syncthreads();
  if (threadIdx.x == 0) {
    double all = 0.0;
    for (int w = 0; w < kBalWaves; ++w) all += part[w];
    out.loss[0] = n > 0 ? (float)(all * (double)E / ((double)n * (double)k)) : 0.0f;
    out.num_valid[0] = n;
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kBalThreads)
balance_kernel(Balance b, BalanceWs ws, BalanceOut out) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int E = b.E, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double* const sums = reinterpret_cast<double*>(lds);              // [E]
  int32_t* const counts = reinterpret_cast<int32_t*>(sums + E);     // [E]
  __shared__ int32_t valid[kBalWaves];
  __shared__ double part[kBalWaves];
  for (int e = threadIdx.x; e < E; e += kBalThreads) {
    sums[e] = 0.0;
    counts[e] = 0;
  }
  __syncthreads();
  double acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0;
  int32_t n = 0;
  const int64_t waves = (int64_t)gridDim.x * kBalWaves;
  for (int64_t t = (int64_t)blockIdx.x * kBalWaves + wave; t < b.T; t += waves) {
    if (b.mask && !b.mask[t]) continue;
    ++n;
    for (int j = lane; j < b.k; j += 64) {
      const int32_t e = b.topk_ids[t * b.k + j];
      if (e >= 0 && e < E) atomicAdd(&counts[e], 1);
    }
    float v[V];
    load_logits<T, V>(static_cast<const T*>(b.logits) + t * E, E, v);
    softmax<V>(v);
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] += (double)v[i];
  }
  if (lane == 0) valid[wave] = n;
  // wave after wave: the order of the sums is fixed
  for (int w = 0; w < kBalWaves; ++w) {
    if (w == wave) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane + 64 * i < E) sums[lane + 64 * i] += acc[i];
    }
    __syncthreads();
  }
  n = 0;
  for (int w = 0; w < kBalWaves; ++w) n += valid[w];
  if (gridDim.x == 1) {
    finish(E, b.k, n, sums, counts, out, part);
    return;
  }
  for (int e = threadIdx.x; e < E; e += kBalThreads) {
    ws.sums[(int64_t)blockIdx.x * E + e] = sums[e];
    ws.counts[(int64_t)blockIdx.x * E + e] = counts[e];
  }
  if (threadIdx.x == 0) ws.valid[blockIdx.x] = n;
}

__global__ void __launch_bounds__(kBalThreads)
balance_finish_kernel(int E, int k, int blocks, BalanceWs ws, BalanceOut out) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  double* const sums = reinterpret_cast<double*>(lds);
  int32_t* const counts = reinterpret_cast<int32_t*>(sums + E);
  __shared__ double part[kBalWaves];
  for (int e = threadIdx.x; e < E; e += kBalThreads) {
    double s = 0.0;
    int32_t c = 0;
    for (int q = 0; q < blocks; ++q) {
      s += ws.sums[(int64_t)q * E + e];
      c += ws.counts[(int64_t)q * E + e];
    }
    sums[e] = s;
    counts[e] = c;
  }
  int32_t n = 0;
  for (int q = 0; q < blocks; ++q) n += ws.valid[q];
  __syncthreads();
  finish(E, k, n, sums, counts, out, part);
}

static constexpr int kBackThreads = 256, kBackWaves = kBackThreads / 64;

template <typename T, typename O, int V>
__global__ void __launch_bounds__(kBackThreads)
balance_backward_kernel(Balance b, const int32_t* __restrict__ counts, const int32_t* __restrict__ num_valid,
                        const float* __restrict__ d_loss, O* __restrict__ d_logits) {
  const int E = b.E, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t n = num_valid[0];
  const double g = n > 0 ? (d_loss ? (double)d_loss[0] : 1.0) * (double)E / ((double)n * (double)n * (double)b.k) : 0.0;
  float c[V];
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = lane + 64 * i < E ? (float)counts[lane + 64 * i] : 0.0f;
  const int64_t waves = (int64_t)gridDim.x * kBackWaves;
  for (int64_t t = (int64_t)blockIdx.x * kBackWaves + wave; t < b.T; t += waves) {
    O* const to = d_logits + t * E;
    if (b.mask && !b.mask[t]) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (lane + 64 * i < E) to[lane + 64 * i] = (O)0.0f;
      continue;
    }
    float p[V];
    load_logits<T, V>(static_cast<const T*>(b.logits) + t * E, E, p);
    softmax<V>(p);
    double dot = 0.0;
#pragma unroll
    for (int i = 0; i < V; ++i) dot = __builtin_fma((double)p[i], (double)c[i], dot);
    dot = wave_sum(dot);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (lane + 64 * i < E) to[lane + 64 * i] = (O)(float)(g * (double)p[i] * ((double)c[i] - dot));
  }
}

template <typename F>
static hipError_t for_experts(int E, F&& go) {
  if (E <= 64) return go(std::integral_constant<int, 1>{});
  if (E <= 128) return go(std::integral_constant<int, 2>{});
  if (E <= 256) return go(std::integral_constant<int, 4>{});
  if (E <= 512) return go(std::integral_constant<int, 8>{});
  return go(std::integral_constant<int, 16>{});
}

hipError_t launch_balance_loss(const Balance& b, float* loss, int32_t* counts, float* mean_probs,
                               int32_t* num_valid, void* workspace, hipStream_t stream) {
  const BalanceWs ws = balance_ws(workspace, b.E);
  const BalanceOut out = {loss, counts, mean_probs, num_valid};
  const int blocks = b.T <= kBalSingle ? 1 : (int)std::min<int64_t>(ceil_div(b.T, kBalWaves), kBalBlocks);
  const size_t lds = (size_t)b.E * 12;
  const hipError_t st = for_experts(b.E, [&](auto per) {
    constexpr int V = decltype(per)::value;
    if (b.logits_f32)
      hipLaunchKernelGGL((balance_kernel<float, V>), dim3(blocks), dim3(kBalThreads), lds, stream, b, ws, out);
    else
      hipLaunchKernelGGL((balance_kernel<bf16_t, V>), dim3(blocks), dim3(kBalThreads), lds, stream, b, ws, out);
    return hipGetLastError();
  });
  if (st != hipSuccess || blocks == 1) return st;
  hipLaunchKernelGGL(balance_finish_kernel, dim3(1), dim3(kBalThreads), lds, stream, b.E, b.k, blocks, ws, out);
  return hipGetLastError();
}

hipError_t launch_balance_loss_backward(const Balance& b, bool out_f32, const int32_t* counts,
                                        const int32_t* num_valid, const float* d_loss, void* d_logits,
                                        hipStream_t stream) {
  const unsigned blocks = (unsigned)std::min<int64_t>(ceil_div(b.T, kBackWaves), 256 * 8);
  return for_experts(b.E, [&](auto per) {
    constexpr int V = decltype(per)::value;
    auto go = [&](auto kernel, auto* to) {
      hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kBackThreads), 0, stream, b, counts, num_valid, d_loss, to);
    };
    float* f = static_cast<float*>(d_logits);
    bf16_t* h = static_cast<bf16_t*>(d_logits);
    if (b.logits_f32) {
      if (out_f32) go(balance_backward_kernel<float, float, V>, f);
      else go(balance_backward_kernel<float, bf16_t, V>, h);
    } else {
      if (out_f32) go(balance_backward_kernel<bf16_t, float, V>, f);
      else go(balance_backward_kernel<bf16_t, bf16_t, V>, h);
    }
    return hipGetLastError();
  });
}

}  // namespace moelora
