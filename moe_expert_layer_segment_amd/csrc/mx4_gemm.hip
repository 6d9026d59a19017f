// Products with MX4 weights:  out[m, n] = sum_k x[m, k] W_e[n, k], with e the expert
// of row m's tile (tile_expert of align; one weight for all rows without it),
// optionally followed by out[m, i] = SiLU(y[m, i]) y[m, I + i] for N = 2 I.
//
// The matrix cores take W as the A operand (its rows are the output columns)
// and x as the B operand, so a lane ends up with four consecutive columns of one
// row.  One MFMA of 128 K values wants, per lane, the 32 values (16 bytes) of
// one block of one row and that block's scale: lane l holds row l % 16 and one of
// four blocks.  Which four blocks of a row make up a step is free as long as both
// operands agree; here lane group g = l / 16 takes blocks 2g and 2g + 1 of every 8
// (one 128-byte line of codes), so its two scale bytes are neighbours.
//
//   MX4 x:   v_mfma_scale_f32_16x16x128_f8f6f4 on the codes as they are.  Products
//            of codes are exact; the sums are fp32.
//   bf16 x:  the codes become bf16 times their scale, which is exact (2
//            significand bits, the exponent range of fp32), and go through four
//            v_mfma_f32_16x16x32_bf16: 8 consecutive values of the block each.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "kernels.hpp"

namespace moelora {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef bf16_t bf16x2 __attribute__((ext_vector_type(2)));
typedef bf16_t bf16x4 __attribute__((ext_vector_type(4)));

// the 8 values of one word of codes, times 2^(scale byte - 127)
__device__ __forceinline__ bf16x8 mx4_bf16x8(uint32_t w, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  bf16x8 v;
  v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1];
  v[4] = c[0]; v[5] = c[1]; v[6] = d[0]; v[7] = d[1];
  return v;
}

__device__ __forceinline__ floatx4 mfma_mx4(u32x4 a, int sa, u32x4 b, int sb, floatx4 c) {
  const i32x8 va = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 vb = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, c, 4, 4, 0, sa, 0, sb);
}

__device__ __forceinline__ void store_out(const Mx4Gemm& p, int64_t at, floatx4 v) {
  if (p.out_f32) {
    *reinterpret_cast<floatx4*>(static_cast<float*>(p.out) + at) = v;
  } else {
    bf16x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (bf16_t)v[i];
    *reinterpret_cast<bf16x4*>(static_cast<bf16_t*>(p.out) + at) = o;
  }
}

// first weight row of 16-column block cb; with silu_mul even blocks are gate
// columns, odd ones the up columns beside them
__device__ __forceinline__ int64_t weight_row(const Mx4Gemm& p, int64_t cb) {
  return p.silu_mul ? (cb & 1) * (p.N / 2) + (cb >> 1) * 16 : cb * 16;
}

// Few rows: the weights are streamed from memory into registers, once.  A workgroup
// holds 16 MB rows and 16 NB columns; its WV waves take every WV-th group of 8
// blocks (256 K values) and add their sums through LDS.
template <bool XMX, int MB, int NB, int WV>
__global__ void __launch_bounds__(64 * WV) mx4_stream_kernel(Mx4Gemm p, int col_groups) {
  extern __shared__ floatx4 sums[];   // [WV][MB * NB][64]
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int64_t m0 = (int64_t)(blockIdx.x / col_groups) * (16 * MB);
  const int64_t cb0 = (int64_t)(blockIdx.x % col_groups) * NB;
  const int64_t ncb = p.N / 16;
  int64_t e = 0;
  if (p.tile_expert) {
    e = p.tile_expert[m0 / p.BM];
    if (e < 0 || e >= p.E) return;
  }
  const int nblk = (int)(p.K / 32);
  const uint8_t *wc[NB], *ws[NB], *xc[MB], *xs[MB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int64_t n = e * p.N + weight_row(p, min(cb0 + nb, ncb - 1)) + r;
    wc[nb] = p.w + n * (p.K / 2);
    ws[nb] = p.w_scale + n * nblk;
  }
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const int64_t m = min(m0 + mb * 16 + r, p.M - 1);
    xc[mb] = static_cast<const uint8_t*>(p.x) + m * (XMX ? p.K / 2 : p.K * 2);
    xs[mb] = XMX ? p.x_scale + m * nblk : nullptr;
  }
  floatx4 acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

  for (int s = wave; s * 8 < nblk; s += WV) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      // blocks behind the row's end: zero codes under the scale of 1
      const int blk = s * 8 + 2 * g + b;
      const bool in = blk < nblk;
      const int at = in ? blk : 0;
      u32x4 wf[NB];
      int wsc[NB];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        wf[nb] = *reinterpret_cast<const u32x4*>(wc[nb] + at * 16);
        wsc[nb] = ws[nb][at];
        if (!in) {
          wf[nb] = u32x4{0, 0, 0, 0};
          wsc[nb] = 127;
        }
      }
      if constexpr (XMX) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          u32x4 xf = *reinterpret_cast<const u32x4*>(xc[mb] + at * 16);
          int xsc = xs[mb][at];
          if (!in) {
            xf = u32x4{0, 0, 0, 0};
            xsc = 127;
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            acc[mb][nb] = mfma_mx4(wf[nb], wsc[nb], xf, xsc, acc[mb][nb]);
        }
      } else {
        bf16x8 xf[MB][4];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            xf[mb][q] = *reinterpret_cast<const bf16x8*>(xc[mb] + at * 64 + q * 16);
            if (!in) xf[mb][q] = Elt<bf16_t>::zero();
          }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const float scale = mx4_scale((uint32_t)wsc[nb]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const bf16x8 a = mx4_bf16x8(wf[nb][q], scale);
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
              acc[mb][nb] = Elt<bf16_t>::mma(a, xf[mb][q], acc[mb][nb]);
          }
        }
      }
    }
  }

#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) sums[(wave * MB * NB + mb * NB + nb) * 64 + lane] = acc[mb][nb];
  __syncthreads();
  auto total = [&](int tile) {
    floatx4 v = sums[tile * 64 + lane];
    for (int w = 1; w < WV; ++w) v += sums[(w * MB * NB + tile) * 64 + lane];
    return v;
  };
  if (p.silu_mul) {
    for (int i = wave; i < MB * NB / 2; i += WV) {
      const int mb = i / (NB / 2), nb = 2 * (i % (NB / 2));
      const int64_t m = m0 + mb * 16 + r;
      if (cb0 + nb + 1 >= ncb || m >= p.M) continue;
      const floatx4 gate = total(mb * NB + nb), up = total(mb * NB + nb + 1);
      floatx4 v;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = silu_f(gate[q]) * up[q];
      store_out(p, m * (p.N / 2) + (cb0 + nb) / 2 * 16 + 4 * g, v);
    }
  } else {
    for (int i = wave; i < MB * NB; i += WV) {
      const int mb = i / NB, nb = i % NB;
      const int64_t m = m0 + mb * 16 + r;
      if (cb0 + nb >= ncb || m >= p.M) continue;
      store_out(p, m * p.N + (cb0 + nb) * 16 + 4 * g, total(i));
    }
  }
}

template <bool XMX, int MB, int NB, int WV>
static hipError_t stream(const Mx4Gemm& p, hipStream_t stream) {
  const int64_t col_groups = ceil_div(p.N / 16, NB);
  const int64_t blocks = ceil_div(p.M, 16 * MB) * col_groups;
  hipLaunchKernelGGL((mx4_stream_kernel<XMX, MB, NB, WV>), dim3((unsigned)blocks), dim3(64 * WV),
                     (size_t)WV * MB * NB * 64 * sizeof(floatx4), stream, p, (int)col_groups);
  return hipGetLastError();
}

hipError_t launch_mx4_gemm(const Mx4Gemm& p, hipStream_t s) {
  // rows of a workgroup: within one tile_expert entry
  const int64_t rows = p.tile_expert ? p.BM : p.M;
  const bool r64 = p.tile_expert ? rows % 64 == 0 : rows > 32;
  const bool r32 = p.tile_expert ? rows % 32 == 0 : rows > 16;
  if (p.x_mx4) {
    if (r64) return stream<true, 4, 2, 4>(p, s);
    if (r32) return stream<true, 2, 4, 4>(p, s);
    return stream<true, 1, 4, 4>(p, s);
  }
  if (r64) return stream<false, 4, 2, 4>(p, s);
  if (r32) return stream<false, 2, 4, 4>(p, s);
  return stream<false, 1, 4, 4>(p, s);
}

}  // namespace moelora
