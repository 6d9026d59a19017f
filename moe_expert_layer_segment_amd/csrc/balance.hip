// Pairs per expert and the balance loss of a router, and its gradient for the logits.
//
// Over the n tokens that take part (all, or those of a mask), with p_t = softmax(logits_t):
//
//   counts_e = pairs of these tokens with id e,   P_e = sum_t p_te / n
//   loss     = E / (n k) sum_e counts_e P_e       (1 where both are even)
//   d loss / d logits_te = E / (n^2 k) p_te (counts_e - sum_i p_ti counts_i)
//
// counts are constants to the gradient.  A row of logits that are all -inf has p = 0, one with a NaN or
// +inf has p = NaN, and with n = 0 everything is 0.  Logits of tokens outside the mask are never read.
//
// One wave per token, V experts to a lane: neighbours where V divides their number, so that a
// load brings them all, else every 64th.  p is fp64, and holds more than fp32 would: the gradient is
// a difference, and an fp32 result lacks little but its own rounding.  A wave adds its tokens up in
// registers, a workgroup its waves through LDS, and the workgroups' sums go through memory to others
// that add them in order: no floating-point atomics, so results do not change from run to run.  Few
// tokens are one workgroup, and one launch.
//
// Latency bounds small batches, and the instructions of the softmax large ones: 16384 tokens of 256
// experts in fp32 take 11 us forward (17 MB: 3 at the rate of reading), 5.5 for the finish, and 12
// back (34 MB: 7).
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "kernels.hpp"
#include "vec.hpp"
#include "wave.hpp"

namespace moelora {

static constexpr int kBalThreads = 1024, kBalWaves = kBalThreads / 64;
static constexpr int kBalBlocks = 256;        // whose sums are added by the finish
static constexpr int kFinishWide = 32;        // experts of one of its workgroups
static constexpr int kFinishGroups = (int)kMaxBalanceExperts / kFinishWide;
// tokens that one workgroup takes alone, without a second launch and its workspace (of 128 experts
// in a graph: 64 tokens 7.3 us, by two launches 8.5; 96 tokens 9.3 and 8.6; 128 10.6 and 8.3; 192 13.9 and
// 8.8; calls made one by one take longer than that on the host, and more by two launches)
static constexpr int kBalSingle = 128;

struct BalanceWs {
  double* sums;       // [blocks][E]
  int32_t* counts;    // [blocks][E]
  int32_t* valid;     // [blocks]
  double* dots;       // [kFinishGroups] parts of sum_e counts_e P_e
  int32_t* done;      // workgroups that have written theirs
};
static BalanceWs balance_ws(void* ws, int64_t E) {
  BalanceWs w;
  w.sums = static_cast<double*>(ws);
  w.counts = reinterpret_cast<int32_t*>(w.sums + kBalBlocks * E);
  w.valid = w.counts + kBalBlocks * E;
  w.dots = reinterpret_cast<double*>(w.valid + kBalBlocks);
  w.done = reinterpret_cast<int32_t*>(w.dots + kFinishGroups);
  return w;
}
size_t balance_ws_bytes(int64_t T, int64_t E) {
  return T <= kBalSingle ? 0 : (size_t)kBalBlocks * ((size_t)E * 12 + 4) + kFinishGroups * 8 + 8;
}

// expert i of a lane
template <int V, bool NEXT>
__device__ __forceinline__ int expert_of(int i) {
  const int lane = threadIdx.x & 63;
  return NEXT ? lane * V + i : lane + 64 * i;
}

// e^z of z <= 0 (0 below -2000), to 2^-29 of its value: 2^n 2^f of z log2(e) = n + f, |f| <= 1/2, with
// the series of 2^f to f^8.  Its terms from f^3 on are fp32, rounded at 2^-28 of an eighth of the result,
// all else fp64.  (It takes no longer than the hardware's exponential with what makes its argument good,
// and gives 6 bits more.)
__device__ __forceinline__ double exp_of(double z) {
  constexpr double kLog2e = 1.4426950408889634;
  constexpr double kInt = 1.5 * 4503599627370496.0;   // its last bit is 1
  const double s = __builtin_fma(z, kLog2e, kInt);
  const double f = __builtin_fma(z, kLog2e, -(s - kInt));
  const float x = (float)f;
  float r = 1.3215487e-6f;                            // ln(2)^k / k!, from k = 8 down
  r = __builtin_fmaf(r, x, 1.5252734e-5f);
  r = __builtin_fmaf(r, x, 1.5403530e-4f);
  r = __builtin_fmaf(r, x, 1.3333558e-3f);
  r = __builtin_fmaf(r, x, 9.6181291e-3f);
  r = __builtin_fmaf(r, x, 5.5504109e-2f);
  double e = __builtin_fma(f, (double)r, 0.2402265069591007);
  e = __builtin_fma(f, e, 0.6931471805599453);
  e = __builtin_fma(f, e, 1.0);
  return __builtin_amdgcn_ldexp(e, (int32_t)(uint32_t)__builtin_bit_cast(uint64_t, s));
}

// logits of a lane, -inf behind the last, to e^(logit - the row's largest); all 0 where there is none
// but -inf.  The largest is that of the numbers, and a NaN stays one.
template <int V>
__device__ __forceinline__ void exponentials(const float (&v)[V], double (&e)[V]) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = fmaxf(m, v[i]);
  m = wave_max(m == m ? m : -INFINITY);
  const double base = m == -INFINITY ? 0.0 : (double)m;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const double z = (double)v[i] - base;
    e[i] = exp_of(z < -2000.0 ? -2000.0 : z);   // (for -inf; NaN stays)
  }
}

// what makes exponentials of this sum (at least 1, 0 or NaN) to probabilities
__device__ __forceinline__ double per_sum(double sum) { return sum == 0.0 ? 0.0 : reciprocal(sum); }

template <typename T, int V, bool NEXT>
__device__ __forceinline__ void load_logits(const T* row, int E, float (&v)[V]) {
  if constexpr (NEXT) {
    constexpr int W = V < kWide<T> ? V : kWide<T>;   // of one load
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = -INFINITY;
    if (expert_of<V, true>(0) < E) {
#pragma unroll
      for (int i = 0; i < V; i += W) {
        float part[W];
        load_floats<T, W>(row + expert_of<V, true>(i), part);
#pragma unroll
        for (int q = 0; q < W; ++q) v[i + q] = part[q];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = expert_of<V, false>(i) < E ? (float)row[expert_of<V, false>(i)] : -INFINITY;
  }
}
template <typename O, int V, bool NEXT>
__device__ __forceinline__ void store_logits(O* row, int E, const float (&v)[V]) {
  if constexpr (NEXT) {
    constexpr int W = V < kWide<O> ? V : kWide<O>;
    if (expert_of<V, true>(0) >= E) return;
#pragma unroll
    for (int i = 0; i < V; i += W) {
      float part[W];
#pragma unroll
      for (int q = 0; q < W; ++q) part[q] = v[i + q];
      store_floats<O, W>(row + expert_of<V, true>(i), part);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (expert_of<V, false>(i) < E) row[expert_of<V, false>(i)] = (O)v[i];
  }
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

template <typename T, int V, bool NEXT>
__global__ void __launch_bounds__(kBalThreads)
balance_kernel(Balance b, BalanceWs ws, BalanceOut out) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int E = b.E, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  double* const sums = reinterpret_cast<double*>(lds);              // [4][E]
  int32_t* const counts = reinterpret_cast<int32_t*>(sums + 4 * E); // [E]
  __shared__ int32_t valid[kBalWaves];
  __shared__ double part[kBalWaves];
  for (int e = threadIdx.x; e < E; e += kBalThreads) counts[e] = 0;
  __syncthreads();
  double acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0;
  int32_t n = 0;
  // U tokens of a wave at a time, all loaded before the first is worked on
  constexpr int U = V <= 4 ? 4 : V == 8 ? 2 : 1;
  const int64_t waves = (int64_t)gridDim.x * kBalWaves;
  for (int64_t t0 = (int64_t)blockIdx.x * kBalWaves + wave; t0 < b.T; t0 += waves * U) {
    bool live[U];
    float v[U][V];
    int32_t id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * waves;
      live[u] = t < b.T && (!b.mask || b.mask[t]);
      id[u] = -1;
      if (live[u]) {
        load_logits<T, V, NEXT>(static_cast<const T*>(b.logits) + t * E, E, v[u]);
        if (lane < b.k) id[u] = b.topk_ids[t * b.k + lane];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!live[u]) continue;
      ++n;
      if (id[u] >= 0 && id[u] < E) atomicAdd(&counts[id[u]], 1);
      for (int j = lane + 64; j < b.k; j += 64) {
        const int32_t e = b.topk_ids[(t0 + u * waves) * b.k + j];
        if (e >= 0 && e < E) atomicAdd(&counts[e], 1);
      }
      double e[V], sum = 0.0;
      exponentials<V>(v[u], e);
#pragma unroll
      for (int i = 0; i < V; ++i) sum += e[i];
      const double per = per_sum(wave_sum(sum));
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = __builtin_fma(e[i], per, acc[i]);
    }
  }
  if (lane == 0) valid[wave] = n;
  // the upper waves' sums to the lower ones, four waves at a time: their order is fixed
#pragma unroll
  for (int top = kBalWaves; top > 1; top = top > 4 ? top - 4 : top / 2) {
    const int from = top > 4 ? top - 4 : top / 2, many = top - from;
    if (wave >= from && wave < top) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (expert_of<V, NEXT>(i) < E) sums[(wave - from) * E + expert_of<V, NEXT>(i)] = acc[i];
    }
    __syncthreads();
    if (wave >= from - many && wave < from) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (expert_of<V, NEXT>(i) < E) acc[i] += sums[(wave - from + many) * E + expert_of<V, NEXT>(i)];
    }
    __syncthreads();
  }
  if (wave == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (expert_of<V, NEXT>(i) < E) sums[expert_of<V, NEXT>(i)] = acc[i];
  }
  __syncthreads();
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
  if (threadIdx.x == 0) {
    ws.valid[blockIdx.x] = n;
    if (blockIdx.x == 0) ws.done[0] = 0;
  }
}

// A workgroup adds up kFinishWide experts, thread (part, expert) the workgroups part, part + 32,
// ..: one alone, which fetches what 256 CUs wrote at the pace of one CU, took 17 us where these take
// 5.5 (16384 tokens, 256 experts).  The one that is done last adds the parts of the loss, in order.
__global__ void __launch_bounds__(kBalThreads)
balance_finish_kernel(int E, int k, int blocks, BalanceWs ws, BalanceOut out) {
  constexpr int kParts = kBalThreads / kFinishWide;
  __shared__ double sums[kParts][kFinishWide];
  __shared__ int32_t many[kParts][kFinishWide];
  __shared__ bool last;
  const int in = threadIdx.x % kFinishWide, part = threadIdx.x / kFinishWide;
  const int e = blockIdx.x * kFinishWide + in;
  double s = 0.0;
  int32_t c = 0;
  if (e < E) {
#pragma unroll 8
    for (int q = part; q < blocks; q += kParts) {
      s += ws.sums[(int64_t)q * E + e];
      c += ws.counts[(int64_t)q * E + e];
    }
  }
  sums[part][in] = s;
  many[part][in] = c;
  int32_t n = 0;
  for (int q = threadIdx.x & 63; q < blocks; q += 64) n += ws.valid[q];
  n = wave_sum(n);
  __syncthreads();
  if (threadIdx.x < 64) {   // the first wave: 32 experts, its other lanes nothing
    double dot = 0.0;
    if (part == 0 && e < E) {
      for (int q = 1; q < kParts; ++q) {
        s += sums[q][in];
        c += many[q][in];
      }
      const double mean = n > 0 ? s / (double)n : 0.0;
      out.mean_probs[e] = (float)mean;
      out.counts[e] = c;
      dot = (double)c * mean;
    }
    dot = wave_sum(dot);
    if (threadIdx.x == 0) {
      ws.dots[blockIdx.x] = dot;
      __threadfence();
      last = atomicAdd(ws.done, 1) == (int32_t)gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!last || threadIdx.x >= 64) return;
  __threadfence();
  double all = 0.0;
  for (int q = threadIdx.x; q < (int)gridDim.x; q += 64)
    all += __hip_atomic_load(&ws.dots[q], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  all = wave_sum(all);
  if (threadIdx.x == 0) {
    out.loss[0] = n > 0 ? (float)(all * (double)E / ((double)n * (double)k)) : 0.0f;
    out.num_valid[0] = n;
  }
}

static constexpr int kBackThreads = 256, kBackWaves = kBackThreads / 64;

template <typename T, typename O, int V, bool NEXT>
__global__ void __launch_bounds__(kBackThreads)
balance_backward_kernel(Balance b, const int32_t* __restrict__ counts, const int32_t* __restrict__ num_valid,
                        const float* __restrict__ d_loss, O* __restrict__ d_logits) {
  const int E = b.E, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t n = num_valid[0];
  const double g = n > 0 ? (d_loss ? (double)d_loss[0] : 1.0) * (double)E / ((double)n * (double)n * (double)b.k) : 0.0;
  double c[V];   // exactly: their differences may be below what fp32 holds of counts of many ranks
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = expert_of<V, NEXT>(i) < E ? (double)counts[expert_of<V, NEXT>(i)] : 0.0;
  constexpr int U = V <= 4 ? 2 : 1;
  const int64_t waves = (int64_t)gridDim.x * kBackWaves;
  for (int64_t t0 = (int64_t)blockIdx.x * kBackWaves + wave; t0 < b.T; t0 += waves * U) {
    bool live[U];
    float v[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * waves;
      live[u] = t < b.T && (!b.mask || b.mask[t]);
      if (live[u]) load_logits<T, V, NEXT>(static_cast<const T*>(b.logits) + t * E, E, v[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * waves;
      if (t >= b.T) break;
      float d[V];
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = 0.0f;
      if (live[u]) {
        // the sums of e_i and e_i c_i, so that probabilities add up to 1: in c_e - mean all of c would
        // stay of what they lack, beside differences that can be any part of it (every c the same: 0)
        double e[V], sum = 0.0, dot = 0.0;
        exponentials<V>(v[u], e);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          sum += e[i];
          dot = __builtin_fma(e[i], c[i], dot);
        }
        sum = wave_sum(sum);
        dot = wave_sum(dot);
        const double per = per_sum(sum), mean = dot * per, scale = g * per;
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = (float)(scale * e[i] * (c[i] - mean));
      }
      store_logits<O, V, NEXT>(d_logits + t * E, E, d);
    }
  }
}

// go(experts of a lane, whether they are neighbours)
template <typename F>
static hipError_t for_experts(int E, F&& go) {
  auto with = [&](auto per) {
    if (decltype(per)::value > 1 && E % decltype(per)::value == 0) return go(per, std::true_type{});
    return go(per, std::false_type{});
  };
  if (E <= 64) return go(std::integral_constant<int, 1>{}, std::false_type{});
  if (E <= 128) return with(std::integral_constant<int, 2>{});
  if (E <= 256) return with(std::integral_constant<int, 4>{});
  if (E <= 512) return with(std::integral_constant<int, 8>{});
  return with(std::integral_constant<int, 16>{});
}

hipError_t launch_balance_loss(const Balance& b, float* loss, int32_t* counts, float* mean_probs,
                               int32_t* num_valid, void* workspace, hipStream_t stream) {
  const BalanceWs ws = balance_ws(workspace, b.E);
  const BalanceOut out = {loss, counts, mean_probs, num_valid};
  const int blocks = b.T <= kBalSingle ? 1 : (int)std::min<int64_t>(ceil_div(b.T, kBalWaves), kBalBlocks);
  const size_t lds = (size_t)b.E * 36;
  const hipError_t st = for_experts(b.E, [&](auto per, auto next) {
    constexpr int V = decltype(per)::value;
    constexpr bool N = decltype(next)::value;
    if (b.logits_f32)
      hipLaunchKernelGGL((balance_kernel<float, V, N>), dim3(blocks), dim3(kBalThreads), lds, stream, b, ws, out);
    else
      hipLaunchKernelGGL((balance_kernel<bf16_t, V, N>), dim3(blocks), dim3(kBalThreads), lds, stream, b, ws, out);
    return hipGetLastError();
  });
  if (st != hipSuccess || blocks == 1) return st;
  hipLaunchKernelGGL(balance_finish_kernel, dim3((unsigned)ceil_div(b.E, kFinishWide)), dim3(kBalThreads), 0, stream,
                     b.E, b.k, blocks, ws, out);
  return hipGetLastError();
}

hipError_t launch_balance_loss_backward(const Balance& b, bool out_f32, const int32_t* counts,
                                        const int32_t* num_valid, const float* d_loss, void* d_logits,
                                        hipStream_t stream) {
  const unsigned blocks = (unsigned)std::min<int64_t>(ceil_div(b.T, kBackWaves), 256 * 8);
  return for_experts(b.E, [&](auto per, auto next) {
    constexpr int V = decltype(per)::value;
    constexpr bool N = decltype(next)::value;
    auto go = [&](auto kernel, auto* to) {
      hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kBackThreads), 0, stream, b, counts, num_valid, d_loss, to);
    };
    float* f = static_cast<float*>(d_logits);
    bf16_t* h = static_cast<bf16_t*>(d_logits);
    if (b.logits_f32) {
      if (out_f32) go(balance_backward_kernel<float, float, V, N>, f);
      else go(balance_backward_kernel<float, bf16_t, V, N>, h);
    } else {
      if (out_f32) go(balance_backward_kernel<bf16_t, float, V, N>, f);
      else go(balance_backward_kernel<bf16_t, bf16_t, V, N>, h);
    }
    return hipGetLastError();
  });
}

}  // namespace moelora
