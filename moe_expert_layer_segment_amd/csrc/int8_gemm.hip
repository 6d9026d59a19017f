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
// would cost e^-v |v| 2^-25 of its value.  The exponent is that of a v within [-126, 126], where
// it and its correction are finite: e^126 is infinite and e^-126 nothing beside 1, so a v beyond
// gives what it should, v itself (or its infinity) or -0.  Below -88, where SiLU is less than 1e-36,
// the result is -0.
__device__ __forceinline__ float silu_near(float v) {
  const float kLog2e = 1.4426950408889634f, kRest = 1.925963033500887e-8f, kLn2 = 0.6931471805599453f;
  const float x = -__builtin_amdgcn_fmed3f(v, -126.0f, 126.0f);
  const float t = x * kLog2e;
  const float lo = __builtin_fmaf(x, kRest, __builtin_fmaf(x, kLog2e, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  // (an infinite e stays one: times lo it would not)
  return v * __builtin_amdgcn_rcpf(1.0f + __builtin_fmaf(fminf(e, 1e38f), lo * kLn2, e));
}

// 4 outputs of SiLU(gate) * up
__device__ __forceinline__ floatx4 silu_mul(floatx4 gate, floatx4 up) {
  floatx4 v;
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = silu_near(gate[q]) * up[q];
  return v;
}

// first weight row of 16-column block cb; with silu_mul even blocks are gate
// columns, odd ones the up columns beside them
__device__ __forceinline__ int64_t weight_row(const Int8Gemm& p, int64_t cb) {
  return p.silu_mul ? (cb & 1) * (p.N / 2) + (cb >> 1) * 16 : cb * 16;
}

// ---- few rows --------------------------------------------------------------
// The weights are streamed from memory into registers, once for each 16 MB rows, and bound the kernel
// where that is once for an expert (64 tokens x 8 of 128 experts, 1536 x 2048 each: 74 us, 5.3 TB/s);
// with more rows the groups read them again, and x once for each of the columns' workgroups (2112 x
// 7168 with 17 rows 10.7 us, 64 19.4, 128 23.7).  A workgroup holds 16 MB rows and 16 NB
// columns; its WV waves take every WV-th group of 128 values of K and add their sums through LDS.
template <int MB, int NB, int WV>
__global__ void __launch_bounds__(64 * WV, MB == 1 ? 4 : 2)
int8_stream_kernel(Int8Gemm p, int col_groups) {
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
  // a group is fetched while the one before is multiplied
  const int whole = chunks / (4 * H);
  Group f[2];
  int s = wave;
  if (s < whole) load(f[0], s, std::false_type{});
  while (s < whole) {
    if (s + WV < whole) load(f[1], s + WV, std::false_type{});
    multiply(f[0]);
    s += WV;
    if (s >= whole) break;
    if (s + WV < whole) load(f[0], s + WV, std::false_type{});
    multiply(f[1]);
    s += WV;
  }
  if (s * 4 * H < chunks) {   // the wave whose turn it is takes the end of the rows
    load(f[0], s, std::true_type{});
    multiply(f[0]);
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
        store_out(p, m * (p.N / 2) + (cb0 + nb) / 2 * 16 + 4 * g, silu_mul(gate, up));
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
                     (int)col_groups);
  return hipGetLastError();
}

// ---- many rows -------------------------------------------------------------
// Tiles of TM rows x 256 weight rows, K in steps of 128 values: rows of 128 bytes in LDS, of x
// and of the weights alike, in two buffers.  Four waves, one to a SIMD, so that a wave has 512
// registers: 256 of them hold the sums of 128 x 128 outputs, and a step of 64 K values takes 16
// fragments (256 bytes a lane) for 64 MFMAs, half the LDS reads of eight waves with 128 x 64.
//
// A step multiplies one set of fragments while the other is read for the step that follows, the
// reads and the DMAs spread over the MFMAs.  Half way through the first step of a K tile all of it
// is in registers: a barrier there frees its buffer for the DMAs of the tile after the next, half
// of which go out in what is left of this step and half in the second.  A barrier between the
// steps, ahead of which every wave has waited for its DMAs of the next tile, admits that one.
// (With one barrier for both, behind the first step, DMAs had half a step less to arrive:
// 2048 x 4096 x 4128 52 us, so 46; 1000 x 4096 x 7168 50 and 44; 8192 rows of 32 experts x 8192 x
// 4096 425 and 402.)
//
// LDS rows are eight 16-byte chunks.  Lane group g takes chunk 2g + h of its row in step h, from
// place (2g + h) ^ (bits 3, 1, 2 of the row's number): no two of 16 lanes read one bank, and a
// DMA's lanes, which fill places in order, still read whole 64-byte pieces.
//
// 4096 x 4096 x 7168 takes 99 us (2.4e15 operations a second; 87 where all values are zero: the
// clock gives way to the power, from 2.1 GHz to 1.8 where the weights come from memory), of which
// about 11 are the start and the end of a tile: there is one workgroup to a CU, so nothing runs
// beside them.  Of 4096 x 4096 x 28672 (380 us, matrix units busy for 58% of its cycles) the DMAs
// cost a fourth and the LDS reads an eighth; without both they are busy for 81%.
constexpr int kTileN = 256;
constexpr int kStep = 128;   // bytes of K in an LDS row

// this wave's DMAs but its last N are done, then every wave's
template <int N>
__device__ __forceinline__ void wait_barrier() {
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}
// this wave's LDS reads are done, then every wave's
__device__ __forceinline__ void read_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// 8 neighbouring columns
__device__ __forceinline__ void store_out(const Int8Gemm& p, int64_t at, floatx4 v, floatx4 w) {
  if (p.out_f32) {
    store_out(p, at, v);
    store_out(p, at + 4, w);
  } else {
    bf16x8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (bf16_t)(i < 4 ? v[i] : w[i - 4]);
    *reinterpret_cast<bf16x8*>(static_cast<bf16_t*>(p.out) + at) = o;
  }
}

constexpr int tile_lds(int tm) { return 2 * (tm + kTileN) * kStep; }

// c += a * b, in place.  (As a builtin the compiler moves a quarter of the sums from registers to
// registers in every round of the K loop.)  It does not see that a matrix instruction's operands
// want two wait states behind another vector instruction that wrote them, and its sums more of
// them before they are read: the K loop's operands are written by LDS reads alone, and `settle`
// stands wherever else they, or the sums, change hands.
__device__ __forceinline__ void mfma_in_place(int4v& c, int4v a, int4v b) {
  asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
__device__ __forceinline__ void settle() { asm volatile("s_nop 15\n\ts_nop 2" ::: "memory"); }

// a uniform address, in scalar registers
__device__ __forceinline__ uint64_t uniform_address(const void* p) {
  const uint64_t g = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)g);   // (an int, which would extend its sign)
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(g >> 32));
  return (uint64_t)hi << 32 | lo;
}
// as dma16 from a uniform_address, without keeping M0, which nothing else here uses.  (s_nop: the
// base may come from a vector instruction, which wants five wait states ahead of the load.)
__device__ __forceinline__ void dma16_m0(uint64_t base, uint32_t goff, uint32_t lds_addr) {
  asm volatile(
      "s_mov_b32 m0, %[la]\n\t"
      "s_nop 3\n\t"
      "global_load_lds_dwordx4 %[go], %[gb]"
      :
      : [la] "s"(lds_addr), [go] "v"(goff), [gb] "s"(base)
      : "memory");
}

// rows [m0, m0 + TM) of expert e, weight rows from 16 cb0 on; rows from m0 + rows on do not exist.
// ids: with row_ids, those of rows lane, 64 + lane, ...
struct Ids { int32_t a, b, c, d; };
template <int TM>
__device__ __forceinline__ void int8_tile(const Int8Gemm& p, char* lds, int64_t m0, int64_t cb0,
                                          int64_t e, int rows, Ids ids) {
  constexpr int WN = TM == 64 ? 4 : 2, WM = 4 / WN;             // waves over columns and rows
  constexpr int MB = TM / WM / 16, NB = kTileN / WN / 16;       // 16-row blocks of a wave
  constexpr int XSEG = TM / 8 / 4, WSEG = kTileN / 8 / 4;       // a wave's DMAs of 8 rows for a K tile
  constexpr int XPART = TM * kStep, STAGE = XPART + kTileN * kStep;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int wm = wave / WN, wn = wave % WN;
  const int tiles = (int)((p.K + kStep - 1) / kStep);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds);
  auto swz = [](int row) { return (row >> 1 & 4) | (row & 2) | (row >> 2 & 1); };
  // LDS row n of the weights holds row spot(n) of the tile: rows 4q..4q + 3 of two blocks of 16
  // lie side by side, and so do the outputs that a lane has of the two
  auto spot = [](int n) { return n / 32 * 32 + n % 16 / 4 * 8 + n / 16 % 2 * 4 + n % 4; };
  // weight row of LDS row n; with silu_mul blocks of gate and of up rows alternate, and side by
  // side lie those of two gate or two up blocks.  What would lie behind the last column repeats
  // the last.
  const int out_cols = (int)(p.silu_mul ? p.N / 2 : p.N), col0 = (int)cb0 * (p.silu_mul ? 8 : 16);
  auto w_col = [&](int n) {
    const int col = p.silu_mul ? spot(n / 64 * 32 + n / 32 % 2 * 16 + n % 16) : spot(n);
    return min(col, out_cols - 1 - col0);
  };
  auto is_up = [&](int n) { return p.silu_mul && n / 16 % 2; };
  const int32_t id0 = ids.a, id1 = ids.b, id2 = ids.c, id3 = ids.d;
  auto ids_of = [=](int q) { return q == 0 ? id0 : q == 1 ? id1 : q == 2 ? id2 : id3; };
  // what the others read instead is not used
  auto token_of = [&](int32_t id) -> int64_t { return id >= 0 && id < p.num_ids ? (uint32_t)id / (uint32_t)p.top_k : 0; };

  // This lane's row in each of its DMAs: 8 rows of 128 bytes, lane l the chunk at place l % 8 of
  // row l / 8.  Offsets are 32 bits, of x from its start (where the rows of a pair's tokens lie
  // anywhere) or from the tile's first row, of the weights from the tile's first gate or up row.
  constexpr int DMAS = XSEG + WSEG;
  static_assert(XSEG % 2 == 0 && WSEG % 2 == 0, "even segments of 8 rows have one swizzle, odd ones the other");
  uint32_t off[DMAS];
  const uint64_t x_base = uniform_address(p.x + (p.top_k > 0 ? 0 : m0 * p.K));
  const uint64_t w_base = uniform_address(p.w + (e * p.N + col0) * p.K);
  const uint64_t up_base = w_base + (p.silu_mul ? out_cols * p.K : 0);
  auto lds_row = [&](int i) { return i < XSEG ? (wave * XSEG + i) * 8 : (wave * WSEG + i - XSEG) * 8; };
#pragma unroll
  for (int i = 0; i < DMAS; ++i) {
    const int row = lds_row(i) + lane / 8;
    int64_t src = i < XSEG ? min(row, rows - 1) : w_col(row);
    if (i < XSEG && p.top_k > 0) src = token_of(__builtin_amdgcn_ds_bpermute(4 * (row % 64), ids_of(wave * TM / 256)));
    off[i] = (uint32_t)(src * p.K);
  }
  // scale of row threadIdx.x (and whether it holds a pair) and of column threadIdx.x: they arrive
  // while the products are made
  float own_xs = 0.0f, own_ws;
  uint32_t own_holds = 1;
  {
    const int row = min((int)threadIdx.x, rows - 1), id = ids_of(min(wave, TM / 64 - 1));
    if (p.row_ids) own_holds = id >= 0 && id < p.num_ids;
    if ((int)threadIdx.x < TM) own_xs = p.x_scale[p.top_k > 0 ? token_of(id) : m0 + row];
    const int n = threadIdx.x;
    own_ws = p.w_scale[e * p.N + col0 + w_col(n) + (is_up(n) ? out_cols : 0)];
  }
  // its chunk of a K tile, in even and in odd segments
  const uint32_t chunk[2] = {(uint32_t)((lane % 8) ^ swz(lane / 8)) * 16, (uint32_t)((lane % 8) ^ swz(8 + lane / 8)) * 16};
#pragma unroll
  for (int i = 0; i < DMAS; ++i) off[i] += chunk[i % 2];
  // chunks of the last K tile that lie behind the rows' end: the rows' first ones instead, whose
  // products are left out
  auto last_tile = [&]() {
    const uint32_t at = (uint32_t)(tiles - 1) * kStep;
#pragma unroll
    for (int i = 0; i < DMAS; ++i) off[i] -= at + chunk[i % 2] < (uint32_t)p.K ? 0 : chunk[i % 2];
  };
  struct Bases { uint64_t x, w, up; };
  auto bases_of = [&](int t) {
    return Bases{x_base + (uint64_t)t * kStep, w_base + (uint64_t)t * kStep, up_base + (uint64_t)t * kStep};
  };
  auto issue = [&](const Bases& at, int place, int i) {
    const int row = lds_row(i);
    const uint32_t to = lds0 + place * STAGE + (i < XSEG ? 0 : XPART) + row * kStep;
    // a segment of 8 rows is gate or up as a whole
    dma16_m0(i < XSEG ? at.x : is_up(row) ? at.up : at.w, off[i], to);
  };

  int4v acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = int4v{0, 0, 0, 0};
  // places of this lane's row of a wave's first block; a block is 16 rows further
  const int x_at = (wm * MB * 16 + r) * kStep, w_at = XPART + (wn * NB * 16 + r) * kStep;
  const int c_at[2] = {((2 * g) ^ swz(r)) * 16, ((2 * g + 1) ^ swz(r)) * 16};
  int4v xf[2][MB], wf[2][NB];
  auto read_x = [&](int place, auto H, auto I) {
    constexpr int h = decltype(H)::value, i = decltype(I)::value;
    xf[h][i] = *reinterpret_cast<const int4v*>(lds + (place * STAGE + x_at + c_at[h]) + i * 16 * kStep);
  };
  auto read_w = [&](int place, auto H, auto J) {
    constexpr int h = decltype(H)::value, j = decltype(J)::value;
    wf[h][j] = *reinterpret_cast<const int4v*>(lds + (place * STAGE + w_at + c_at[h]) + j * 16 * kStep);
  };
  constexpr std::integral_constant<int, 0> first{};
  constexpr std::integral_constant<int, 1> second{};
  // The MFMAs of step H.  Between them the fragments of the other step are read from `place`: in the
  // second step at an even pace, in the first one behind each of the first MFMAs, and then(slot)
  // does what else there is.
  constexpr int SLOTS = MB * NB, READS = MB + NB, FREE = SLOTS / 2, EARLY = DMAS / 2;
  static_assert(READS <= FREE, "every fragment is read before the buffer is free");
  auto step = [&](auto H, int place, auto&& then) {
    constexpr int h = decltype(H)::value;
    std::integral_constant<int, 1 - h> other;
    static_for<SLOTS>([&](auto S) {
      constexpr int s = decltype(S)::value, i = s / NB, j = s % NB;
      mfma_in_place(acc[i][j], wf[h][j], xf[h][i]);
      // the n-th of READS lies behind MFMA n SPAN / READS; those of the weights come first
      constexpr int SPAN = h == 0 ? READS : SLOTS, n = (s * READS + SPAN - 1) / SPAN;
      if constexpr (n < READS && n * SPAN / READS == s) {
        if constexpr (n < NB) read_w(place, other, std::integral_constant<int, n < NB ? n : 0>{});
        else read_x(place, other, std::integral_constant<int, n < NB ? 0 : n - NB>{});
      }
      then(S);
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  static_for<DMAS>([&](auto D) {
    if (decltype(D)::value == 0 && tiles == 1) last_tile();
    issue(bases_of(0), 0, decltype(D)::value);
  });
  wait_barrier<0>();
  if (tiles > 1) {
    if (tiles == 2) last_tile();
    static_for<DMAS>([&](auto D) { issue(bases_of(1), 1, decltype(D)::value); });
  }
  static_for<MB>([&](auto I) { read_x(0, first, I); });
  static_for<NB>([&](auto J) { read_w(0, first, J); });
  // chunks of the last K tile that lie behind the end of the rows
  auto cut = [&](auto H) {
    constexpr int h = decltype(H)::value;
    const bool in = ((int64_t)(tiles - 1) * 8 + 2 * g + h) * 16 < p.K;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      wf[h][j] = in ? wf[h][j] : int4v{0, 0, 0, 0};
      asm volatile("" : "+v"(wf[h][j]));
    }
    settle();
  };
  settle();
  // one loop for every tile, the last ones too: where the sums pass from one piece of code to
  // another the compiler moves them.  (What the last tile reads ahead is not used.)
  constexpr std::integral_constant<int, EARLY> early{};
  constexpr std::integral_constant<int, DMAS> all{};
  int place = 0;
#pragma unroll 1
  for (int t = 0; t < tiles; ++t, place ^= 1) {
    if (t + 1 == tiles) cut(first);
    if (t + 3 == tiles) last_tile();
    const Bases at = bases_of(t + 2);
    const bool sends = t + 2 < tiles;
    // DMAs LO to HI - 1 behind the MFMAs from slot FROM on, at an even pace
    auto send = [&](auto S, auto FROM, auto LO, auto HI) {
      constexpr int s = decltype(S)::value - decltype(FROM)::value, span = SLOTS - decltype(FROM)::value;
      constexpr int lo = decltype(LO)::value, many = decltype(HI)::value - lo;
      constexpr int d = lo + s * many / span, end = lo + (s + 1) * many / span;
      static_for<end - d>([&](auto D) {
        if (sends) issue(at, place, d + decltype(D)::value);
      });
    };
    step(first, place, [&](auto S) {
      constexpr int s = decltype(S)::value;
      if constexpr (s == FREE) read_barrier();
      if constexpr (s >= FREE) send(S, std::integral_constant<int, FREE>{}, first, early);
    });
    if (sends) wait_barrier<EARLY>();
    else wait_barrier<0>();
    if (t + 1 == tiles) cut(second);
    step(second, place ^ 1, [&](auto S) { send(S, first, early, all); });
    // the last products are done before what follows reads them: here, since the compiler may move
    // the sums as soon as the loop ends
    settle();
  }
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) asm volatile("" : "+a"(acc[i][j]));

  // the scales go through LDS, where what is still read ahead there is not used
  struct Row { float scale; uint32_t holds; };
  Row* const row_lds = reinterpret_cast<Row*>(lds);
  float* const col_lds = reinterpret_cast<float*>(lds + TM * sizeof(Row));
  if ((int)threadIdx.x < TM) row_lds[threadIdx.x] = Row{own_xs, own_holds};
  col_lds[threadIdx.x] = own_ws;
  __syncthreads();
  float xs[MB];
  floatx4 ws[NB];
  uint32_t live = 0;
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const Row row = row_lds[(wm * MB + i) * 16 + r];
    live |= row.holds << i;
    xs[i] = row.scale;
  }
#pragma unroll
  for (int j = 0; j < NB; ++j) ws[j] = *reinterpret_cast<const floatx4*>(col_lds + (wn * NB + j) * 16 + 4 * g);

#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int row = (wm * MB + i) * 16 + r;
    if (row >= rows) continue;
    const bool holds = live >> i & 1;
    const int64_t at = (m0 + row) * out_cols + col0;
    auto y = [&](int j) {
      floatx4 v;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = holds ? (float)acc[i][j][q] * xs[i] * ws[j][q] : 0.0f;
      return v;
    };
    if (p.silu_mul) {
#pragma unroll
      for (int j = 0; j < NB; j += 4) {
        const int col = (wn * NB + j) * 8 + 8 * g;
        if (col0 + col >= out_cols) continue;
        store_out(p, at + col, silu_mul(y(j), y(j + 1)), silu_mul(y(j + 2), y(j + 3)));
      }
    } else {
#pragma unroll
      for (int j = 0; j < NB; j += 2) {
        const int col = (wn * NB + j) * 16 + 8 * g;
        if (col0 + col >= out_cols) continue;
        store_out(p, at + col, y(j), y(j + 1));
      }
    }
  }
}

// Tiles are numbered in bands of kBand rows of them, in patches of kBand x kPatch.  The XCD that
// workgroup b runs on, b % 8, takes 32 neighbours in that order at a time (one for each of its CUs),
// which share rows and weights in its L2.  Workgroups without a tile are the last ones alone: with
// those that the patches at the edges lack left empty, XCDs got unequal shares (65536 x 1536 x
// 2048 of 128 experts 403 us, so 320), and so did the parts of an XCD that consecutive workgroups
// go round (512 x 28672 x 4096, two tiles high, 113 us, so 65).  For the latter the tiles of a
// patch are numbered along its rows, too: rows differ in how many of them hold a pair.
//
// Workgroups of the last, incomplete round of 256 (one to a CU) take a half or a quarter of a
// tile's rows each, where that fills the round no more than once; a workgroup whose rows end
// early with padding takes a smaller tile.
constexpr int kRound = 256, kBand = 4, kPatch = 8;
constexpr int64_t kTailTiles = 16 * kRound;   // with more, a share of a round does not count

// An entry of tile_expert holds several tiles (for block_m = 80 one of 64 rows and one of 16), or
// (entries of 16, 32 or 48 rows: these are the m_tiles, then) a tile takes as many neighbours of
// one expert as it has room for, from the expert's first on; the workgroups of the others have
// nothing to do.
template <int TOP>
__global__ void __launch_bounds__(256, 1) int8_tile_kernel(Int8Gemm p, int m_tiles, int n_tiles, int tail) {
  __shared__ __attribute__((aligned(1024))) char lds[tile_lds(TOP)];
  const int lane = threadIdx.x & 63;
  const bool small = TOP == 64 && p.tile_expert && p.BM < TOP;
  const uint32_t per_entry = p.tile_expert ? ((uint32_t)p.BM + TOP - 1) / TOP : 1;
  uint32_t tile = blockIdx.x / 256 * 256 + blockIdx.x % 8 * 32 + blockIdx.x / 8 % 32;
  int used = m_tiles, whole = m_tiles, pieces = 1;   // tiles with rows; those taken whole
  if (tail) {
    if (p.tile_expert) {
      used = 0;   // from the end, where the entries without an expert are
      for (int t0 = (m_tiles - 1) / 64 * 64; t0 >= 0 && used == 0; t0 -= 64) {
        const int t = t0 + lane;
        const int te = t < m_tiles ? p.tile_expert[(uint32_t)t / per_entry] : -1;
        const uint64_t has = __ballot(te >= 0 && te < p.E);
        if (has) used = t0 + 64 - __clzll(has);
      }
      used = __builtin_amdgcn_readfirstlane(used);
    }
    whole = used * n_tiles / kRound * kRound / n_tiles;
    const int rest = (used - whole) * n_tiles;
    if (TOP == 256 && 4 * rest <= kRound) pieces = 4;
    else if (TOP >= 128 && 2 * rest <= kRound) pieces = 2;
    else whole = used;
  }
  const bool part = tile >= (uint32_t)(whole * n_tiles);
  if (part) tile -= (uint32_t)(whole * n_tiles);
  const uint32_t down = part ? (used - whole) * pieces : whole;
  if (tile >= down * n_tiles) return;
  const uint32_t band = tile / (kBand * n_tiles), high = min((uint32_t)kBand, down - band * kBand);
  tile -= band * kBand * n_tiles;
  const uint32_t patch = tile / (high * kPatch), wide = min((uint32_t)kPatch, n_tiles - patch * kPatch);
  tile -= patch * high * kPatch;
  const int mt = band * kBand + tile / wide, nt = patch * kPatch + tile % wide;
  const int span = part ? TOP / pieces : TOP;
  int64_t m0 = (int64_t)(part ? whole : mt) * TOP + (part ? mt * span : 0);
  int rows = (int)min((int64_t)span, p.M - m0);
  const int64_t cb0 = (int64_t)nt * (kTileN / 16);
  int64_t e = 0;
  if (p.tile_expert) {
    const uint32_t entry = (uint32_t)(part ? whole + mt / pieces : mt) / per_entry;
    e = __builtin_amdgcn_readfirstlane(p.tile_expert[entry]);
    if (e < 0 || e >= p.E) return;
    if (TOP == 64) {
      const int in_entry = (mt - (int)(entry * per_entry)) * TOP;
      m0 = (int64_t)entry * p.BM + in_entry;
      rows = min((int)p.BM - in_entry, TOP);
    }
  }
  if (small) {
    int before = 0;   // entries of this expert
    for (int at = mt - 1; at >= 0; at -= 64) {
      const uint64_t other = __ballot(at < lane || p.tile_expert[max(at - lane, 0)] != e);
      before += other ? __ffsll((unsigned long long)other) - 1 : 64;
      if (other) break;
    }
    const int room = TOP / (int)p.BM;
    if (before % room) return;
    int entries = 1;
    while (entries < room && mt + entries < m_tiles && p.tile_expert[mt + entries] == e) ++entries;
    rows = __builtin_amdgcn_readfirstlane(entries) * (int)p.BM;
  }
  if (rows <= 0) return;
  int live = rows;   // up to the last row that holds a pair
  Ids ids = {};
  if (p.row_ids) {
    live = 0;
    auto id_at = [&](int q) { return 64 * q < TOP ? p.row_ids[m0 + min(q * 64 + lane, rows - 1)] : -1; };
    ids = {id_at(0), id_at(1), id_at(2), id_at(3)};
    auto look = [&](int q, int32_t id) {
      const uint64_t has = __ballot(q * 64 + lane < rows && id >= 0 && id < p.num_ids);
      live = has ? q * 64 + 64 - __clzll(has) : live;
    };
    look(0, ids.a), look(1, ids.b), look(2, ids.c), look(3, ids.d);
    live = __builtin_amdgcn_readfirstlane(live);
  }
  const int done = live > 128 ? 256 : live > 64 ? 128 : live > 0 ? 64 : 0, some = min(rows, done);
  if (TOP == 256 && done == 256) int8_tile<TOP>(p, lds, m0, cb0, e, some, ids);
  else if (TOP >= 128 && done == 128) int8_tile<TOP >= 128 ? 128 : 64>(p, lds, m0, cb0, e, some, ids);
  else if (done == 64) int8_tile<64>(p, lds, m0, cb0, e, some, ids);
  // the rows behind the tile that these take hold no pair
  const int cols = (int)(p.silu_mul ? p.N / 2 : p.N), col0 = (int)cb0 * (p.silu_mul ? 8 : 16);
  const int width = min(p.silu_mul ? kTileN / 2 : kTileN, cols - col0);
  for (int row = done + threadIdx.x / 64; row < rows; row += 4)
    if (lane * 4 < width) store_out(p, (m0 + row) * cols + col0 + lane * 4, floatx4{0.0f, 0.0f, 0.0f, 0.0f});
}

template <int TM>
static hipError_t tiled(const Int8Gemm& p, hipStream_t stream) {
  const int64_t m_tiles = p.tile_expert ? p.M / p.BM * ceil_div(p.BM, TM) : ceil_div(p.M, TM);
  const int64_t n_tiles = ceil_div(p.N, kTileN);
  const bool tail = m_tiles * n_tiles <= kTailTiles;
  // where the last tiles are parted, a round of parts takes their place
  const int64_t blocks = std::max(m_tiles * n_tiles, tail ? (m_tiles - 1) * n_tiles + kRound : 0);
  hipLaunchKernelGGL(int8_tile_kernel<TM>, dim3((unsigned)(ceil_div(blocks, kRound) * kRound)), dim3(256), 0, stream, p,
                     (int)m_tiles, (int)n_tiles, (int)tail);
  return hipGetLastError();
}

// A workgroup of 4 waves and 16 NB columns, or, where those would not fill the chip, of WIDE
// waves and 16 columns (32 with silu_mul: a gate and an up block).  By 4 waves and by WIDE (us): a row x
// 2112 x 7168 16.3 and 9.4, x 8192 x 2048 (128 workgroups of 4) 9.9 and 9.4, x 16384 x 2048 (256)
// 10.8 and 12.0, x 28672 x 4096 23 and 28; 30 rows x 2112 x 7168 21.4 and 12.1; 40 rows x 4096 x 4096
// (128) 13.8 and 11.5, 128 rows x 2112 x 7168 (132) 23.5 and 35.6: more waves read x more often.
template <int MB, int NB, int WIDE>
static hipError_t few(const Int8Gemm& p, hipStream_t s) {
  if (ceil_div(p.M, 16 * MB) * ceil_div(p.N, 16 * NB) > (MB == 1 ? 255 : 128)) return stream<MB, NB, 4>(p, s);
  if (p.silu_mul) return stream<MB, 2, WIDE>(p, s);
  return stream<MB, 1, WIDE>(p, s);
}

// Workgroups of 64 rows, two to a CU, hide each other's beginning and end, those of 256 read less
// for each product.  16384 x 4096 x 256 51 us by 64 rows, 56 by 256; x 512 67 and 68; x 768 82
// and 80, x 2048 167 and 140.  384 x 20480 x 7168, 160 tiles of 256 rows: 67 and 97.
constexpr int64_t kShortK = 512;
// In blocks of 128 rows, by 64 rows and by 128: 65536 rows of 128 experts x 1536 x 2048 357 and 370
// us, 8192 of 32 x 8192 x 4096 486 and 511, x 4096 x 7168 475 and 447.
constexpr int64_t kLongK = 4096;

hipError_t launch_int8_gemm(const Int8Gemm& p, hipStream_t s) {
  // rows of a workgroup: within one tile_expert entry, or those there are
  const int64_t rows = p.tile_expert ? p.BM : p.M;
  auto takes = [&](int64_t n) { return p.tile_expert ? rows % n == 0 : rows > n / 2; };
  const int64_t n_tiles = ceil_div(p.N, kTileN), of64 = ceil_div(p.M, 64) * n_tiles;
  const bool many = p.tile_expert ? !int8_few_rows(p) : takes(64);
  // (64 workgroups of tiles and fewer: 64 rows x 8192 x 2048 20 us, streamed 11; 256 x 4096 x 4096,
  // with 64, 30 and 26; 256 x 8192 x 2048, with 128, 19 and 27)
  if (many && of64 > 64) {
    // one round of pairs of 64 rows, where those of 256 would be more than half a round, not parted
    const bool pairs = !p.tile_expert && of64 <= 2 * kRound && 2 * ceil_div(p.M, 256) * n_tiles > kRound;
    if (p.K > kShortK && !pairs) {
      if (takes(256)) return tiled<256>(p, s);
      if (p.K > kLongK && takes(128)) return tiled<128>(p, s);
    }
    return tiled<64>(p, s);
  }
  if (takes(64)) return few<4, 2, 8>(p, s);
  if (takes(32)) return few<2, 4, 8>(p, s);
  return few<1, 4, 16>(p, s);
}

}  // namespace moelora
