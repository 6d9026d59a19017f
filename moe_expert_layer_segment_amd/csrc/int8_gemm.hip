// Products of 8-bit integers:  y[m, n] = (sum_k x[m, k] W_e[n, k]) * x_scale[m] * w_scale_e[n],
// with e the expert of row m's tile (tile_expert of align; one weight for all rows without
// it), optionally followed by out[m, i] = SiLU(y[m, i]) y[m, I + i] for N = 2 I.
//
// Sums are int32 and exact in any order (K < 2^17 products below 2^14 each), so however K is
// split the result is the same to the bit.  y is that integer rounded to fp32, times the two
// scales in fp32, and a store rounds once more to the type of out.
//
// The matrix cores take W as the A operand (its rows are the output columns) and x as the B
// operand, so a lane ends up with four consecutive columns of one row.  One
// v_mfma_i32_16x16x64_i8 wants, per lane, 16 neighbouring values of row l % 16; which four
// such chunks of a row make up its 64 is free as long as both operands agree.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "gemm_common.hpp"
#include "kernels.hpp"

namespace moelora {

typedef bf16_t bf16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int4v mfma_i8(int4v a, int4v b, int4v c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ void store_out(const Int8Gemm& p, int64_t at, floatx4 v) {
  if (p.out_f32) {
    *reinterpret_cast<floatx4*>(static_cast<float*>(p.out) + at) = v;
  } else {
    bf16x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (bf16_t)v[i];
    *reinterpret_cast<bf16x4*>(static_cast<bf16_t*>(p.out) + at) = o;
  }
}

// SiLU(v) as silu_f, with what rounding the exponent -v log2(e) to fp32 leaves made good: it
// would cost e^-v |v| 2^-25 of its value.
__device__ __forceinline__ float silu_near(float v) {
  const float kLog2e = 1.4426950408889634f, kRest = 1.925963033500887e-8f, kLn2 = 0.6931471805599453f;
  const float t = -v * kLog2e;
  const float lo = __builtin_fmaf(-v, kRest, __builtin_fmaf(-v, kLog2e, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  // behind the range of e the correction would be infinity times lo
  const float d = 1.0f + (e < 1e38f ? __builtin_fmaf(e, lo * kLn2, e) : e);
  return v * __builtin_amdgcn_rcpf(d);
}

// first weight row of 16-column block cb; with silu_mul even blocks are gate
// columns, odd ones the up columns beside them
__device__ __forceinline__ int64_t weight_row(const Int8Gemm& p, int64_t cb) {
  return p.silu_mul ? (cb & 1) * (p.N / 2) + (cb >> 1) * 16 : cb * 16;
}

// ---- few rows --------------------------------------------------------------
// The weights are streamed from memory into registers, once, and bound the kernel.  A workgroup
// holds 16 MB rows and 16 NB columns; its WV waves take every WV-th group of 128 values of K and
// add their sums through LDS.
template <int MB, int NB, int WV>
__global__ void __launch_bounds__(64 * WV, MB == 1 ? 4 : 2)
int8_stream_kernel(Int8Gemm p, int row_groups, int col_groups) {
  constexpr int H = 2;   // 64-value steps of a group
  __shared__ int4v sums[WV][MB * NB][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int row_group = (int)blockIdx.x / col_groups, col_group = (int)blockIdx.x % col_groups;
  const int64_t m0 = (int64_t)row_group * (16 * MB);
  const int64_t cb0 = (int64_t)col_group * NB, ncb = p.N / 16;
  int64_t e = 0;
  if (p.tile_expert) {
    e = __builtin_amdgcn_readfirstlane(p.tile_expert[(uint32_t)m0 / (uint32_t)p.BM]);
    if (e < 0 || e >= p.E) return;
  }
  // a lane's row of each 16-row block: whether it holds a pair, and where its x lies
  bool live[MB];
  int64_t src[MB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const int64_t m = min(m0 + mb * 16 + r, p.M - 1);
    src[mb] = m;
    live[mb] = true;
    if (p.row_ids) {
      const int32_t id = p.row_ids[m];
      live[mb] = id >= 0 && id < p.num_ids;
      if (p.top_k > 0) src[mb] = live[mb] ? (uint32_t)id / (uint32_t)p.top_k : 0;
    }
  }
  struct Group {
    int4v w[NB][H], x[MB][H];
  };
  const int chunks = (int)(p.K / 16);
  auto load = [&](Group& f, int s, auto end) {
    constexpr bool kEnd = decltype(end)::value;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int c = s * 4 * H + h * 4 + g;
      const bool in = !kEnd || c < chunks;   // zeros behind the row's end
      const int at = (in ? c : 0) * 16;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int64_t n = e * p.N + weight_row(p, min(cb0 + nb, ncb - 1));
        const int4v v = *reinterpret_cast<const int4v*>(p.w + n * p.K + (r * (uint32_t)p.K + at));
        f.w[nb][h] = in ? v : int4v{0, 0, 0, 0};
      }
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        f.x[mb][h] = int4v{0, 0, 0, 0};
        if (live[mb] && in) f.x[mb][h] = *reinterpret_cast<const int4v*>(p.x + src[mb] * p.K + at);
      }
    }
  };
  int4v acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = int4v{0, 0, 0, 0};
  auto multiply = [&](const Group& f) {
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) acc[mb][nb] = mfma_i8(f.w[nb][h], f.x[mb][h], acc[mb][nb]);
  };
  const int whole = chunks / (4 * H);
  Group f;
  int s = wave;
  for (; s < whole; s += WV) {
    load(f, s, std::false_type{});
    multiply(f);
  }
  if (s * 4 * H < chunks) {   // the wave whose turn it is takes the end of the rows
    load(f, s, std::true_type{});
    multiply(f);
  }
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) sums[wave][mb * NB + nb][lane] = acc[mb][nb];
  __syncthreads();
  // y of a block: columns 4 g.. of row r
  auto total = [&](int mb, int nb) {
    int4v t = sums[0][mb * NB + nb][lane];
#pragma unroll
    for (int w = 1; w < WV; ++w) t += sums[w][mb * NB + nb][lane];
    const float xs = p.x_scale[src[mb]];
    const float* ws = p.w_scale + e * p.N + weight_row(p, cb0 + nb) + 4 * g;
    floatx4 v;
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = live[mb] ? (float)t[q] * xs * ws[q] : 0.0f;
    return v;
  };
  static_for<MB>([&](auto I) {
    constexpr int mb = decltype(I)::value;
    const int64_t m = m0 + mb * 16 + r;
    if (p.silu_mul) {
      for (int nb = 0; nb < NB; nb += 2) {
        if ((mb * NB + nb) / 2 % WV != wave || cb0 + nb + 1 >= ncb || m >= p.M) continue;
        const floatx4 gate = total(mb, nb), up = total(mb, nb + 1);
        floatx4 v;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = silu_near(gate[q]) * up[q];
        store_out(p, m * (p.N / 2) + (cb0 + nb) / 2 * 16 + 4 * g, v);
      }
    } else {
      for (int nb = 0; nb < NB; ++nb) {
        if ((mb * NB + nb) % WV != wave || cb0 + nb >= ncb || m >= p.M) continue;
        store_out(p, m * p.N + (cb0 + nb) * 16 + 4 * g, total(mb, nb));
      }
    }
  });
}

template <int MB, int NB, int WV>
static hipError_t stream(const Int8Gemm& p, hipStream_t stream) {
  const int64_t col_groups = ceil_div(p.N / 16, NB), row_groups = ceil_div(p.M, 16 * MB);
  const auto kernel = int8_stream_kernel<MB, NB, WV>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(row_groups * col_groups)), dim3(64 * WV), 0, stream, p,
                     (int)row_groups, (int)col_groups);
  return hipGetLastError();
}

hipError_t launch_int8_gemm(const Int8Gemm& p, hipStream_t s) {
  // rows of a workgroup: within one tile_expert entry, or those there are
  const int64_t rows = p.tile_expert ? p.BM : p.M;
  auto takes = [&](int64_t n) { return p.tile_expert ? rows % n == 0 : rows > n / 2; };
  if (takes(64)) return stream<4, 2, 4>(p, s);
  if (takes(32)) return stream<2, 4, 4>(p, s);
  return stream<1, 4, 4>(p, s);
}

}  // namespace moelora
