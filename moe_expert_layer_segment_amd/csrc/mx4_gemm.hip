// Products with MX4 weights:  out[m, n] = sum_k x[m, k] W_e[n, k], with e the expert
// of row m's tile (tile_expert of align; one weight for all rows without it),
// optionally followed by out[m, i] = SiLU(y[m, i]) y[m, I + i] for N = 2 I.
//
// The matrix cores take W as the A operand (its rows are the output columns)
// and x as the B operand, so a lane ends up with four consecutive columns of one
// row.  One MFMA of 128 K values wants, per lane, the 32 values (16 bytes) of
// one block of one row and that block's scale: lane l holds row l % 16 and one of
// four blocks.  Which four blocks of a row make up a step is free as long as both
// operands agree.
//
//   MX4 x:   v_mfma_scale_f32_16x16x128_f8f6f4 on the codes as they are.  Products
//            of codes are exact; the sums are fp32.
//   bf16 x:  the codes become bf16 times their scale, which is exact (2
//            significand bits, the exponent range of fp32), and go through four
//            v_mfma_f32_16x16x32_bf16: 8 consecutive values of the block each.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "gemm_common.hpp"
#include "kernels.hpp"

namespace moelora {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef bf16_t bf16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ floatx4 mfma_mx4(u32x4 a, int sa, u32x4 b, int sb, floatx4 c) {
  const i32x8 va = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 vb = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, c, 4, 4, 0, sa, 0, sb);
}

// t[q] of lane group g = w[g] of lane group q: a 4 x 4 transpose over the groups of
// 16 lanes, in four swaps
__device__ __forceinline__ u32x4 transpose_groups(u32x4 w) {
  const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], c[1], d[0], d[1]};
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

// 8 neighbouring columns
__device__ __forceinline__ void store_out(const Mx4Gemm& p, int64_t at, floatx4 v, floatx4 w) {
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

// first weight row of 16-column block cb; with silu_mul even blocks are gate
// columns, odd ones the up columns beside them
__device__ __forceinline__ int64_t weight_row(const Mx4Gemm& p, int64_t cb) {
  return p.silu_mul ? (cb & 1) * (p.N / 2) + (cb >> 1) * 16 : cb * 16;
}

// ---- few rows --------------------------------------------------------------
// The weights are streamed from memory into registers, once, and bound the kernel.
// A workgroup holds 16 MB rows and 16 NB columns; its WV waves take every WV-th
// group of four blocks and add their sums through LDS.  Longer groups cost the registers
// of another workgroup on the CU (7168 x 2048 of 32 experts, MX4 x, tiles of 32 rows:
// 97 us with eight blocks, 84 with four).
//
// Lane group g loads block g of the four, so the 16 bytes of neighbouring lane groups
// make up 64 bytes of a row; so do the bytes of bf16 x, of which lane group g loads
// 16 g..16 g + 15 of each block.  To match, the weights' words are exchanged between the
// lane groups: 4 x 4 words, in four swaps.
// (Loading x to match the weights instead, 16 bytes in 64, took 91 us where this took
// 64 on gate and up of 64 tokens x 8 of 128 experts, 1536 x 2048.)
//
// What the rows and the scales cost there, beside 36 us for the codes alone (5.9 TB/s):
// 16 us for x, whose padding rows (three in four) are therefore not read, and 10 us
// for scales loaded as they are used, 8 bytes of a row at a time.  The 16 rows of a
// block have their scales in one piece of memory, so a workgroup fetches them
// 16 bytes a lane into LDS first, up to K = kStageK.
constexpr int kStageK = 16384;

template <bool XMX, int MB, int NB, int WV>
__global__ void __launch_bounds__(64 * WV, MB == 1 ? 4 : 2)
mx4_stream_kernel(Mx4Gemm p, int row_groups, int col_groups, int spread) {
  constexpr int GB = 4;   // blocks of a group
  __shared__ floatx4 sums[WV][MB * NB][64];
  extern __shared__ __attribute__((aligned(16))) uint8_t staged[];   // [NB (+ MB)][16][nblk]
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  // With many row groups (spread) the column groups of two neighbouring ones run on one
  // XCD (workgroup b on XCD b % 8), in pairs: its L2 then holds their rows, and the
  // weights where the two are of one expert.
  int row_group, col_group;
  if (spread) {
    const int at = (int)(blockIdx.x / 8), two = 2 * col_groups;
    row_group = (at / two * 8 + (int)(blockIdx.x % 8)) * 2 + at % 2;
    col_group = at % two / 2;
  } else {
    row_group = (int)blockIdx.x / col_groups;
    col_group = (int)blockIdx.x % col_groups;
  }
  if (row_group >= row_groups) return;
  const int64_t m0 = (int64_t)row_group * (16 * MB);
  const int64_t cb0 = (int64_t)col_group * NB, ncb = p.N / 16;
  int32_t id[MB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const int64_t m = min(m0 + mb * 16 + r, p.M - 1);
    id[mb] = p.row_ids ? p.row_ids[m] : 0;
  }
  int64_t e = 0;
  if (p.tile_expert) {
    e = __builtin_amdgcn_readfirstlane(p.tile_expert[(uint32_t)m0 / (uint32_t)p.BM]);
    if (e < 0 || e >= p.E) return;
  }
  const int nblk = (int)(p.K / 32);
  // uniform bases and an offset per lane
  const int64_t w_row = p.K / 2, x_row = XMX ? p.K / 2 : p.K * 2;
  const uint8_t* const x_base = static_cast<const uint8_t*>(p.x) + m0 * x_row;
  const uint8_t* const xs_base = XMX ? p.x_scale + m0 * nblk : nullptr;
  uint32_t m_lane[MB];
  bool live[MB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    m_lane[mb] = (uint32_t)min((int64_t)mb * 16 + r, p.M - 1 - m0);
    live[mb] = !p.row_ids || (id[mb] >= 0 && id[mb] < p.num_ids);
  }
  // Scales on their way to LDS, in pieces of 16 bytes: nblk of a block's 16 rows.  The
  // first piece of a thread travels beside its first codes.
  const bool stage = p.K <= kStageK;
  const bool stage_x = XMX && stage && m0 + 16 * MB <= p.M;
  const int pieces = stage ? (NB + (stage_x ? MB : 0)) * nblk : 0;
  auto fetch = [&](int at) {
    const int blk = at / nblk, in = (at - blk * nblk) * 16;
    const uint8_t* src = p.w_scale + (e * p.N + weight_row(p, min(cb0 + blk, ncb - 1))) * nblk;
    if constexpr (XMX) {
      if (blk >= NB) src = xs_base + (int64_t)(blk - NB) * 16 * nblk;
    }
    u32x4 v;
    __builtin_memcpy(&v, src + in, 16);
    return v;
  };
  auto put = [&](int at, u32x4 v) { *reinterpret_cast<u32x4*>(staged + at * 16) = v; };
#pragma unroll 1
  for (int at = 64 * WV + (int)threadIdx.x; at < pieces; at += 64 * WV) put(at, fetch(at));
  u32x4 piece = {0, 0, 0, 0};
  if ((int)threadIdx.x < pieces) piece = fetch(threadIdx.x);

  struct Group {
    u32x4 w[NB], x[MB][XMX ? 1 : GB];
  };
  // the scales of group s, 2^0 behind the end and for padding rows (whose scales may be
  // anything, NaN too)
  uint32_t wsc[NB], xsc[XMX ? MB : 1];
  auto load_scales = [&](int s, auto end) {
    auto get = [&](uint32_t& v, const uint8_t* row) {
      if constexpr (!decltype(end)::value) {
        __builtin_memcpy(&v, row + s * GB, GB);
      } else {
        v = 0;
#pragma unroll
        for (int b = s * GB + GB - 1; b >= s * GB; --b) v = v << 8 | (b < nblk ? row[b] : 127);
      }
    };
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if (stage) {
        get(wsc[nb], staged + (nb * 16 + r) * nblk);
      } else {
        get(wsc[nb], p.w_scale + (e * p.N + weight_row(p, min(cb0 + nb, ncb - 1)) + r) * nblk);
      }
    }
    if constexpr (XMX) {
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        if (stage_x) {
          get(xsc[mb], staged + ((NB + mb) * 16 + r) * nblk);
        } else {
          get(xsc[mb], xs_base + (int64_t)m_lane[mb] * nblk);
        }
        if (!live[mb]) xsc[mb] = 0x7F7F7F7Fu;
      }
    }
  };
  auto load = [&](Group& f, int s, auto end) {
    constexpr bool kEnd = decltype(end)::value;
    // blocks behind the row's end: zero codes under the scale of 1
    auto codes = [&](const uint8_t* base, uint32_t row) {
      const int blk = s * GB + g;
      const bool in = !kEnd || blk < nblk;
      const u32x4 v = *reinterpret_cast<const u32x4*>(base + (row + (in ? blk : 0) * 16));
      return in ? v : u32x4{0, 0, 0, 0};
    };
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int64_t n = e * p.N + weight_row(p, min(cb0 + nb, ncb - 1));
      f.w[nb] = codes(p.w + n * w_row, r * (uint32_t)w_row);
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
#pragma unroll
      for (int q = 0; q < (XMX ? 1 : GB); ++q) f.x[mb][q] = u32x4{0, 0, 0, 0};
      if (live[mb]) {
        const uint32_t row = m_lane[mb] * (uint32_t)x_row;
        if constexpr (XMX) {
          f.x[mb][0] = codes(x_base, row);
        } else {
#pragma unroll
          for (int q = 0; q < GB; ++q)
            if (!kEnd || s * GB + q < nblk)
              f.x[mb][q] = *reinterpret_cast<const u32x4*>(x_base + (row + (s * GB + q) * 64 + g * 16));
        }
      }
    }
  };
  floatx4 acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](const Group& f) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if constexpr (XMX) {
        const int sw = (int)(wsc[nb] >> (8 * g));
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
          acc[mb][nb] = mfma_mx4(f.w[nb], sw, f.x[mb][0], (int)(xsc[mb] >> (8 * g)), acc[mb][nb]);
      } else {
        const u32x4 t = transpose_groups(f.w[nb]);
#pragma unroll
        for (int q = 0; q < GB; ++q) {
          // the scale byte as an exponent; the conversion reads 0 as 2^-127, 255 as NaN
          const uint32_t scale = (wsc[nb] >> (8 * q) & 255) << 23;
          const bf16x8 a = mx4_bf16x8(t[q], __builtin_bit_cast(float, scale));
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
            acc[mb][nb] = Elt<bf16_t>::mma(a, __builtin_bit_cast(bf16x8, f.x[mb][q]), acc[mb][nb]);
        }
      }
    }
  };
  Group f;
  int s = wave;
  const int whole = nblk / GB;
  if (s < whole) load(f, s, std::false_type{});
  if (stage) {
    if ((int)threadIdx.x < pieces) put(threadIdx.x, piece);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // the first loads stay in flight
  }
  while (s < whole) {
    load_scales(s, std::false_type{});
    multiply(f);
    s += WV;
    if (s < whole) load(f, s, std::false_type{});
  }
  if (s * GB < nblk) {   // the wave whose turn it is takes the end of the rows
    load(f, s, std::true_type{});
    load_scales(s, std::true_type{});
    multiply(f);
  }

  // padding rows give zeros: their x is, but zero times a NaN or infinite weight is not
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
      sums[wave][mb * NB + nb][lane] = live[mb] ? acc[mb][nb] : floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  __syncthreads();
  auto total = [&](int tile) {
    floatx4 v = sums[0][tile][lane];
#pragma unroll
    for (int w = 1; w < WV; ++w) v += sums[w][tile][lane];
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

// ---- many rows -------------------------------------------------------------
// Tiles of TM rows x 256 weight rows, K in steps of 128-byte LDS rows of x: 256
// values of MX4 x or 64 of bf16.  Eight waves as 2 x 4, each (TM / 2) x 64.
//
// Codes reach LDS by global -> LDS DMA, in a ring of RING K tiles: three of bf16 x
// (40 KB each; two took the prefill product of a 4096 x 14336 layer from 0.97 to
// 1.13 ms), two of MX4 x (64 KB; a ring of nine quarters, one of which stays in
// flight over each wait, was 8% slower).  What bounds both is the L1, which keeps
// about 64 lines in flight: 64 KB per 256 x 256 x 256 products, at that window over
// the latency of the L2.
//
// A K tile is two steps.  In a step a wave keeps its four weight fragments in
// registers and takes the 16-row blocks of x one after another, four MFMAs each,
// reading the block that comes kAhead later meanwhile.  When the last fragments of
// a tile have been read, a barrier admits the next tile; behind it the wave starts
// the DMA into the places just left and reads the next tile's first fragments under
// the MFMAs that remain.  Beside its K tiles (16384 rows of 4 experts, 4096 x 7168 of MX4
// x: 48 us of the 59 that 256 workgroups take) a workgroup spends 3 us before its first
// products and 2 on its stores, and 3 go by until the CU holds the next one.
//
// LDS rows of x (and of MX4 weights) are eight 16-byte chunks.  Lane group g wants
// chunk 2g + h in step h.  A fragment read serves 16 lanes at a time, rows of two
// neighbouring groups among them; without a bank met twice it reads a chunk either from
// place (4h + g) ^ (bits 3, 2, 1 of the row's number) or from place (2g + h) ^ (bits
// 3, 1, 2).  The first spreads the four lanes of a DMA that should share 64 bytes over
// 128, which costs MX4 x, whose two operands both come this way, 5%; bf16 x is 7%
// faster with it.
constexpr int kTileN = 256;

__device__ __attribute__((aligned(16))) uint32_t mx4_zeros[4];   // what lies behind a row's end

// as dma16, with an address per lane, of 16 or of 4 bytes a lane
template <int BYTES>
__device__ __forceinline__ void dma_lane(const void* p, uint32_t lds_addr) {
  const uint32_t la = __builtin_amdgcn_readfirstlane(lds_addr);
  uint32_t saved;
  if constexpr (BYTES == 16)
    asm volatile(
        "s_mov_b32 %[sv], m0\n\t"
        "s_mov_b32 m0, %[la]\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %[p], off\n\t"
        "s_mov_b32 m0, %[sv]"
        : [sv] "=&s"(saved)
        : [la] "s"(la), [p] "v"((uint64_t)(uintptr_t)p)
        : "memory");
  else
    asm volatile(
        "s_mov_b32 %[sv], m0\n\t"
        "s_mov_b32 m0, %[la]\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dword %[p], off\n\t"
        "s_mov_b32 m0, %[sv]"
        : [sv] "=&s"(saved)
        : [la] "s"(la), [p] "v"((uint64_t)(uintptr_t)p)
        : "memory");
}

// this wave's DMA but the newest N and its LDS accesses are done, then every wave's
template <int N>
__device__ __forceinline__ void wait_dma_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

constexpr int tile_ring(bool xmx) { return xmx ? 2 : 3; }
// LDS of a tile: the ring, and two buffers of scales
constexpr int tile_lds(bool xmx, int tm) {
  return tile_ring(xmx) * (tm * 128 + kTileN * (xmx ? 128 : 32)) +
         2 * ((xmx ? tm : 0) + kTileN) * (xmx ? 16 : 4);
}

// rows [m0, m0 + TM) of expert e, weight rows from 16 cb0 on; holds: a bit per row
// that holds a pair; DS: scales by DMA; rows before m0 + skip are left to another workgroup
struct Holds { uint64_t r0, r64, r128, r192; };   // not an array: those end in LDS

template <bool XMX, int TM, bool DS>
__device__ __forceinline__ void mx4_tile(const Mx4Gemm& p, char* lds, int64_t m0, int64_t cb0,
                                         int64_t e, Holds holds, int skip) {
  constexpr int WN = 4, NW = 8;
  constexpr int MB = TM / 32, NB = kTileN / 16 / WN;        // 16-row blocks of a wave
  constexpr int WROWB = XMX ? 128 : 32;                     // LDS bytes of a weight row
  constexpr int RING = tile_ring(XMX);
  constexpr int XPART = TM * 128, STAGE = XPART + kTileN * WROWB;
  constexpr int XSEG = XPART / 1024 / NW, WSEG = kTileN * WROWB / 1024 / NW;  // a wave's DMAs
  constexpr int SROWS = (XMX ? TM : 0) + kTileN;            // rows with scales; x's come first
  constexpr int KB = XMX ? 8 : 2;                           // blocks of 32 in a K tile
  constexpr int SB = 2 * KB;                                // scale bytes of a row for two K tiles
  constexpr int SCALES = RING * STAGE;                      // where the two scale buffers lie
  static_assert(SROWS <= 64 * NW && SROWS % 64 == 0, "one scale row per thread");
  static_assert(SCALES + 2 * SROWS * SB == tile_lds(XMX, TM), "the LDS of a tile");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int wm = wave / WN, wn = wave % WN;
  const int nblk = (int)(p.K / 32);
  const int tiles = (nblk + KB - 1) / KB;
  const int64_t x_row = XMX ? p.K / 2 : p.K * 2;
  const int m_last = (int)min((int64_t)TM, p.M - m0) - 1;
  const char* x_base = static_cast<const char*>(p.x) + m0 * x_row;
  const uint8_t* w_base = p.w + e * p.N * (p.K / 2);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  auto swz = [](int row) {
    return XMX ? (row >> 1 & 4) | (row & 2) | (row >> 2 & 1) : (row >> 1) & 7;
  };
  auto chunk_in = [](int place) { return XMX ? place : (place & 3) * 2 + (place >> 2); };
  // LDS row n holds row spot(n) of the tile: rows 4q..4q + 3 of two blocks of 16 lie side
  // by side, and so do the outputs that a lane has of the two
  auto spot = [](int n) { return n / 32 * 32 + n % 16 / 4 * 8 + n / 16 % 2 * 4 + n % 4; };
  // weight row of LDS row n; with silu_mul blocks of gate and of up rows alternate, and
  // side by side lie those of two gate or two up blocks.  What would lie behind the last
  // column repeats another, `room` rows of it.
  const int out_cols = (int)(p.silu_mul ? p.N / 2 : p.N), col0 = (int)cb0 * (p.silu_mul ? 8 : 16);
  auto w_row = [&](int n, int room) {
    const int col = p.silu_mul ? spot(n / 64 * 32 + n / 32 % 2 * 16 + n % 16) : spot(n);
    return min(col0 + col, out_cols - room) + (p.silu_mul ? n / 16 % 2 * out_cols : 0);
  };

  // One KB of LDS per DMA: 8 rows of x or MX4 weights, 32 of the weights beside
  // bf16 x.  The 8 rows of a segment lie at a uniform base, so an offset per lane
  // (one for even and one for odd segments: their swizzle differs) serves them all.
  // A tile behind the end of K or of M takes an address per lane instead, worked out
  // on the spot (kept over the loop, these would cost more registers than there are).
  static_assert((XSEG == 1 || XSEG % 2 == 0) && (!XMX || WSEG % 2 == 0), "even and odd segments");
  uint32_t lane_off[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    lane_off[h] = (uint32_t)(spot(lane / 8) * (int)x_row + chunk_in((lane % 8) ^ swz(h * 8 + lane / 8)) * 16);
  const uint32_t lane_off_one = wave % 2 ? lane_off[1] : lane_off[0];
  const bool all_rows = m_last == TM - 1;
  constexpr int DMAS = XSEG + WSEG;      // of a wave, for a tile
  // the i-th of them; fast: a whole tile of whole rows
  auto issue_one = [&](int t, int place, int i, auto fast) {
    constexpr bool kWhole = decltype(fast)::value;
    const uint32_t at = lds0 + place * STAGE;
    int l = lane;
    if constexpr (!kWhole) asm volatile("" : "+v"(l));
    if (i < XSEG) {
      const int seg = wave * XSEG + i;
      if constexpr (kWhole) {
        const uint32_t off = XSEG == 1 ? lane_off_one : lane_off[i % 2];
        dma16(x_base + spot(seg * 8) * x_row, off + t * 128, at + seg * 1024);
      } else {
        const int row = seg * 8 + l / 8, c = chunk_in((l % 8) ^ swz(row));
        // chunks of 16 bytes: a block of MX4, a quarter of one in bf16
        const bool in_row = t * KB + (XMX ? c : c / 4) < nblk;
        const char* src = x_base + min(spot(row), m_last) * x_row + t * 128 + c * 16;
        dma_lane<16>(in_row ? (const void*)src : (const void*)mx4_zeros, at + seg * 1024);
      }
    } else {
      const int seg = wave * WSEG + i - XSEG;
      const uint32_t to = at + XPART + seg * 1024;
      if constexpr (XMX && kWhole) {
        dma16(w_base + (int64_t)w_row(seg * 8, 12) * (p.K / 2), lane_off[(i - XSEG) % 2] + t * 128, to);
      } else {
        const int row = XMX ? seg * 8 + l / 8 : seg * 32 + l / 2;
        const int c = XMX ? chunk_in((l % 8) ^ swz(row)) : l % 2;
        const uint8_t* src = w_base + (int64_t)w_row(row, 1) * (p.K / 2) + t * WROWB + c * 16;
        const bool in_row = kWhole || t * KB + c < nblk;
        dma_lane<16>(in_row ? (const void*)src : (const void*)mx4_zeros, to);
      }
    }
  };
  auto issue = [&](int t, int place, int from, int to, auto fast) {
#pragma unroll
    for (int i = 0; i < DMAS; ++i)
      if (i >= from && i < to) issue_one(t, place, i, fast);
  };

  // Scales of tiles 2 grp and 2 grp + 1, a row per thread.  Beside bf16 x they take
  // the DMA (DS; 4 bytes a row) where rows of them are aligned to words.  Otherwise
  // they go through registers, loaded behind the barrier of an even tile and stored
  // ahead of that of the odd one, at the price of waiting there for the DMA of both
  // tiles ahead (2048 rows, 4096 x 4128: 73 us; 4096 x 4096 64 so and 67 through
  // registers, 94 with the address of each row worked out tile by tile).  MX4's 16 bytes
  // a row always do: by DMA they took a third more requests to the L2, and 347 instead of
  // 326 us.  So do those at the end of a row, with 2^0 behind it.
  // (a wave's 64 rows are all of x or all of the weights: a uniform base)
  const int s_lane = min(wave * 64 + lane, SROWS - 1);
  const bool s_of_x = XMX && wave < TM / 64;
  const uint8_t* const s_base = s_of_x ? p.x_scale + m0 * nblk : p.w_scale + e * p.N * nblk;
  const uint32_t s_off = (uint32_t)(s_of_x ? min(spot(s_lane), m_last) : w_row(s_lane - (XMX ? TM : 0), 1)) *
                         (uint32_t)nblk;
  struct Words { uint32_t w[SB / 4]; } s_val;
  auto scales_load = [&](int grp) {
    __builtin_memcpy(&s_val, s_base + grp * SB + s_off, SB);
  };
  // whether or not they are all in the row: the row's last SB bytes are shifted down
  auto scales_load_end = [&](int grp) {
    const int behind = (grp + 1) * SB - nblk;
    if (behind <= 0) {
      scales_load(grp);
    } else if (nblk >= SB) {
      __builtin_memcpy(&s_val, s_base + (nblk - SB) + s_off, SB);
      for (int b = 0; b < behind; ++b) {
#pragma unroll
        for (int w = 0; w < SB / 4; ++w)
          s_val.w[w] = __builtin_amdgcn_alignbyte(w + 1 < SB / 4 ? s_val.w[w + 1] : 127u, s_val.w[w], 1);
      }
    } else {
#pragma unroll
      for (int w = 0; w < SB / 4; ++w) {
        s_val.w[w] = 0;
#pragma unroll
        for (int b = 3; b >= 0; --b) {
          const int at = grp * SB + 4 * w + b;
          s_val.w[w] = s_val.w[w] << 8 | (at < nblk ? s_base[s_off + min(at, nblk - 1)] : 127);
        }
      }
    }
  };
  auto scales_store = [&](int grp) {
    if (SROWS == 64 * NW || (int)threadIdx.x < SROWS)
      __builtin_memcpy(lds + SCALES + ((grp & 1) * SROWS + threadIdx.x) * SB, &s_val, SB);
  };
  auto scales_dma = [&](int grp) {
    if (wave < SROWS / 64)
      dma_lane<SB>(s_base + grp * SB + s_off, lds0 + SCALES + ((grp & 1) * SROWS + wave * 64) * SB);
  };

  constexpr int kAhead = MB > 3 ? 3 : 1, kRing = kAhead + 1;
  static_assert((2 * MB) % kRing == 0 && MB > kAhead, "the ring starts each tile at its first place");
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  // of a K tile.  MX4: a word holds the bytes of both steps of two neighbouring
  // blocks; bf16 x: the weights' codes of both steps, and their scale bytes
  struct TileScales {
    int xs[XMX ? MB / 2 : 1], ws[XMX ? NB / 2 : NB];
    u32x2 codes[XMX ? 1 : NB];
  };
  // places of this lane's row of a wave's first block; a block is 16 rows further
  const int x_lane = (wm * MB * 16 + r) * 128, w_lane = XPART + (wn * NB * 16 + r) * WROWB;
  int c_at[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) c_at[h] = ((XMX ? 2 * g + h : 4 * h + g) ^ swz(r)) * 16;
  const int xs_at = SCALES + (wm * MB * 16 + r) * SB + 2 * g;
  const int ws_at = SCALES + ((XMX ? TM : 0) + wn * NB * 16 + r) * SB + (XMX ? 2 * g : g >> 1);
  auto read_x = [&](int place, int i, int step) {
    return *reinterpret_cast<const u32x4*>(lds + place * STAGE + x_lane + c_at[step] + i * 2048);
  };
  auto read_w = [&](int place, int j, int step) {
    return *reinterpret_cast<const u32x4*>(lds + place * STAGE + w_lane + c_at[step] + j * 2048);
  };
  auto read_scales = [&](TileScales& f, int place, int t) {
    const char* s = lds + ((t / 2) & 1) * SROWS * SB + (t & 1) * KB;
    if constexpr (XMX) {
      typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
      auto two = [&](const char* q) {
        u16x2 v;
        v[0] = *reinterpret_cast<const uint16_t*>(q);
        v[1] = *reinterpret_cast<const uint16_t*>(q + 16 * SB);
        return __builtin_bit_cast(int, v);
      };
#pragma unroll
      for (int i = 0; i < MB; i += 2) f.xs[i / 2] = two(s + xs_at + i * 16 * SB);
#pragma unroll
      for (int j = 0; j < NB; j += 2) f.ws[j / 2] = two(s + ws_at + j * 16 * SB);
    } else {
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        f.codes[j] = *reinterpret_cast<const u32x2*>(lds + place * STAGE + w_lane + g * 8 + j * 512);
        f.ws[j] = (int)*reinterpret_cast<const uint8_t*>(s + ws_at + j * 16 * SB);
      }
    }
  };
  // weight fragment of a step: codes, or their values times the scale (the
  // conversion reads scale byte 0 as 2^-127 and 255 as NaN)
  auto expand = [&](const TileScales& f, int j, int step) {
    return __builtin_bit_cast(
        u32x4, mx4_bf16x8(f.codes[j][step], __builtin_bit_cast(float, f.ws[j] << 23)));
  };

  floatx4 acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  // the products so far happen here: left to itself the compiler moves them behind
  // the barrier, where nothing is left to cover the reads
  auto pin = [&]() {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) asm volatile("" : "+v"(acc[i][j]));
  };

  u32x4 x[kRing], w0[NB], w1[NB];   // blocks of x, weights of the first and second step
  TileScales sc;
  auto multiply = [&](auto step, auto block, const u32x4 (&w)[NB]) {
    constexpr int S = decltype(step)::value, i = decltype(block)::value;
    const u32x4 xf = x[(S * MB + i) % kRing];
    static_for<NB>([&](auto J) {
      constexpr int j = decltype(J)::value;
      if constexpr (XMX) {
        const i32x8 a = {(int)w[j][0], (int)w[j][1], (int)w[j][2], (int)w[j][3], 0, 0, 0, 0};
        const i32x8 b = {(int)xf[0], (int)xf[1], (int)xf[2], (int)xf[3], 0, 0, 0, 0};
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            a, b, acc[i][j], 4, 4, 2 * (j % 2) + S, sc.ws[j / 2], 2 * (i % 2) + S, sc.xs[i / 2]);
      } else {
        acc[i][j] = Elt<bf16_t>::mma(__builtin_bit_cast(bf16x8, w[j]), __builtin_bit_cast(bf16x8, xf),
                                     acc[i][j]);
      }
    });
  };
  constexpr std::integral_constant<int, 0> first{};
  constexpr std::integral_constant<int, 1> second{};
  // first fragments of tile t, as far as they are read before its MFMAs
  auto read_first = [&](TileScales& f, int place, int t) {
    read_scales(f, place, t);
    if constexpr (XMX) {
#pragma unroll
      for (int j = 0; j < NB; ++j) w0[j] = read_w(place, j, 0);
    }
  };
  int where = 0;          // place of the present tile in the ring
  // kEven, kOdd: a tile of that number, with every tile and scale that it sends
  // for whole; kAny: any but the last
  enum { kEven, kOdd, kAny, kLast };
  // A wave's DMAs go out kPerBlock beside each block of x, the first kEarly of a tile
  // behind the barrier that empties its place, the others in the tile that follows:
  // one after another they hold the wave, and its MFMAs, at the L1's pace (bf16 x:
  // 0.96 instead of 0.93 ms).
  constexpr int kPerBlock = 2, kEarly = kAhead * kPerBlock < DMAS ? kAhead * kPerBlock : DMAS;
  static_assert(kEarly + MB * kPerBlock >= DMAS, "every DMA has its block");
  auto tile = [&](int t, auto mode) {
    constexpr int kMode = decltype(mode)::value;
    // in a ring of two an even tile lies in place 0: known, it costs no address sums
    constexpr bool kKnown = RING == 2 && (kMode == kEven || kMode == kOdd);
    const int place = kKnown ? kMode == kOdd : where;
    const int ahead = place + 1 == RING ? 0 : place + 1;
    if constexpr (!XMX) {
#pragma unroll
      for (int j = 0; j < NB; ++j) w0[j] = expand(sc, j, 0);
    }
    const int behind = place == 0 ? RING - 1 : place - 1;   // left by the tile before
    static_for<MB>([&](auto I) {
      constexpr int i = decltype(I)::value, q = i + kAhead;
      x[q % kRing] = q < MB ? read_x(place, q, 0) : read_x(place, q - MB, 1);
      static_for<NB>([&](auto J) {
        constexpr int j = decltype(J)::value;
        if constexpr (j % MB == i) w1[j] = XMX ? read_w(place, j, 1) : expand(sc, XMX ? 0 : j, 1);
      });
      constexpr int from = kEarly + i * kPerBlock;
      if constexpr (kMode == kAny) {
        if (t + RING - 1 < tiles) issue(t + RING - 1, behind, from, from + kPerBlock, std::false_type{});
      } else if constexpr (kMode != kLast) {
        issue(t + RING - 1, behind, from, from + kPerBlock, std::true_type{});
      }
      multiply(first, I, w0);
      __builtin_amdgcn_sched_barrier(0);
    });
    TileScales next;
    static_for<MB>([&](auto I) {
      constexpr int i = decltype(I)::value, q = MB + i + kAhead;
      if constexpr (i + kAhead < MB) {
        x[q % kRing] = read_x(place, i + kAhead, 1);
      } else if constexpr (kMode != kLast) {
        if constexpr (i + kAhead == MB) {
          pin();
          if constexpr (kMode == kAny) {
            if (t & 1) scales_store((t + 1) / 2);
            wait_dma_barrier<0>();
            if (!(t & 1) && t + 2 < tiles) scales_load_end(t / 2 + 1);
          } else {
            if constexpr (!DS && kMode == kOdd) scales_store((t + 1) / 2);
            wait_dma_barrier<(RING - 2) * DMAS>();
            if constexpr (DS && kMode == kEven) scales_dma(t / 2 + 1);
            if constexpr (!DS && kMode == kEven) scales_load(t / 2 + 1);
          }
          read_first(next, ahead, t + 1);
        }
        x[q % kRing] = read_x(ahead, i + kAhead - MB, 0);
        constexpr int from = (i + kAhead - MB) * kPerBlock;
        if constexpr (kMode != kAny) issue(t + RING, place, from, from + kPerBlock, std::true_type{});
        else if (t + RING < tiles) issue(t + RING, place, from, from + kPerBlock, std::false_type{});
      }
      multiply(second, I, w1);
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr (kMode != kLast) {
      sc = next;
      where = ahead;
    }
  };

  issue(0, 0, 0, DMAS, std::false_type{});
  scales_load_end(0);
  scales_store(0);
  wait_dma_barrier<0>();
#pragma unroll
  for (int j = 1; j < RING; ++j)
    if (j < tiles) issue(j, j, 0, j + 1 < RING ? DMAS : kEarly, std::false_type{});
  read_first(sc, 0, 0);
#pragma unroll
  for (int i = 0; i < kAhead; ++i) x[i] = read_x(0, i, 0);
  int t = 0;
  if (all_rows) {
    // tile t + 1 sends for tile t + 1 + RING, tile t for the scales of t + 2 and t + 3
    for (; (t + 2 + RING) * KB <= nblk; t += 2) {
      tile(t, std::integral_constant<int, kEven>{});
      tile(t + 1, std::integral_constant<int, kOdd>{});
    }
  }
  for (; t + 1 < tiles; ++t) tile(t, std::integral_constant<int, kAny>{});
  tile(t, std::integral_constant<int, kLast>{});

  const uint64_t mine[2] = {MB == 8 && wm ? holds.r128 : MB == 4 && wm ? holds.r64 : holds.r0,
                            MB == 8 && wm ? holds.r192 : holds.r64};   // of the wave's rows
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int row = spot((wm * MB + i) * 16 + r);
    if (row > m_last || row < skip) continue;
    const bool holds_pair = mine[i / 4] >> (row % 64) & 1;
    const int64_t at = (m0 + row) * out_cols;
    if (p.silu_mul) {
      const int col = col0 + wn * (NB / 2) * 16 + 8 * g;
      if (col >= out_cols) continue;
      floatx4 v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          v[h][q] = holds_pair ? silu_f(acc[i][2 * h][q]) * acc[i][2 * h + 1][q] : 0.0f;
      store_out(p, at + col, v[0], v[1]);
    } else {
#pragma unroll
      for (int j = 0; j < NB; j += 2) {
        const int col = col0 + (wn * NB + j) * 16 + 8 * g;
        if (col >= out_cols) continue;
        floatx4 v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int q = 0; q < 4; ++q) v[h][q] = holds_pair ? acc[i][j + h][q] : 0.0f;
        store_out(p, at + col, v[0], v[1]);
      }
    }
  }
}

// Workgroups of the last, incomplete round of 256 (one to a CU) take a half or a quarter
// of a tile's rows each, where that fills the round no more than once; a workgroup whose
// live rows fit a smaller tile takes the smaller one (padding closes the rows of an
// expert).  8192 rows of 8 experts, 4096 x 14336, bf16 x: 912 -> 793 us, 2.25 rounds
// having run as three; 16384 rows of 32 experts, 4096 x 7168, MX4 x: 345 -> 318 us.
//
// Patches of (32 / pn) x pn tiles go round the eight XCDs (workgroup b runs on XCD b % 8),
// so the 32 workgroups that an XCD holds share rows and weights in its L2.
constexpr int kRound = 256;
constexpr int64_t kTailTiles = 16 * kRound;   // with more, a share of a round does not count

// per_entry: tiles of an entry of tile_expert (three of 64 rows for block_m = 192)
template <bool XMX, int TOP, bool DS>
__global__ void __launch_bounds__(512) mx4_tile_kernel(Mx4Gemm p, int m_tiles, int n_tiles, int pn,
                                                       int n_patches, int per_entry, int tail) {
  __shared__ __attribute__((aligned(1024))) char lds[tile_lds(XMX, TOP)];
  const int lane = threadIdx.x & 63;
  const int pm = 32 / pn;
  int patch = (int)(blockIdx.x / 256) * 8 + (int)(blockIdx.x % 8);
  const int in = (int)(blockIdx.x / 8) % 32;
  int used = m_tiles, whole = m_tiles, pieces = 1;   // tiles with rows; those taken whole
  if (tail) {
    if (p.tile_expert) {
      used = 0;   // from the end, where the entries without an expert are
      for (int t0 = (m_tiles - 1) / 64 * 64; t0 >= 0 && used == 0; t0 -= 64) {
        const int t = t0 + lane;
        const int te = t < m_tiles ? p.tile_expert[(uint32_t)t / (uint32_t)per_entry] : -1;
        const uint64_t has = __ballot(te >= 0 && te < p.E);
        if (has) used = t0 + 64 - __clzll(has);
      }
      used = __builtin_amdgcn_readfirstlane(used);
    }
    whole = used * n_tiles / kRound * kRound / n_tiles / pm * pm;
    const int rest = (used - whole) * n_tiles;
    if (TOP == 256 && 4 * rest <= kRound) pieces = 4;
    else if (TOP >= 128 && 2 * rest <= kRound) pieces = 2;
    else whole = used;
  }
  const int whole_patches = (whole + pm - 1) / pm * n_patches;
  const bool part = patch >= whole_patches;
  if (part) patch -= whole_patches;
  const int mt = patch / n_patches * pm + in % pm, nt = patch % n_patches * pn + in / pm;
  if (nt >= n_tiles || mt >= (part ? (used - whole) * pieces : whole)) return;
  const int span = part ? TOP / pieces : TOP;
  const int64_t m0 = part ? (int64_t)whole * TOP + (int64_t)mt * span : (int64_t)mt * TOP;
  const int64_t cb0 = (int64_t)nt * (kTileN / 16);
  int64_t e = 0;
  if (p.tile_expert) {
    e = __builtin_amdgcn_readfirstlane(p.tile_expert[(uint32_t)(part ? whole + mt / pieces : mt) / (uint32_t)per_entry]);
    if (e < 0 || e >= p.E) return;
  }
  const int rows = (int)min((int64_t)span, p.M - m0);
  if (rows <= 0) return;
  int live = rows;   // up to the last row that holds a pair
  Holds holds = {~uint64_t(0), ~uint64_t(0), ~uint64_t(0), ~uint64_t(0)};
  if (p.row_ids) {
    auto id_at = [&](int i) { return p.row_ids[m0 + min(i * 64 + lane, rows - 1)]; };
    auto bits = [&](int i, int32_t id) {
      return (uint64_t)__ballot(i * 64 + lane < rows && id >= 0 && id < p.num_ids);
    };
    const int32_t id0 = id_at(0), id1 = TOP >= 128 ? id_at(1) : -1, id2 = TOP == 256 ? id_at(2) : -1,
                  id3 = TOP == 256 ? id_at(3) : -1;
    holds = {bits(0, id0), bits(1, id1), bits(2, id2), bits(3, id3)};
    live = holds.r192   ? 256 - __clzll(holds.r192)
           : holds.r128 ? 192 - __clzll(holds.r128)
           : holds.r64  ? 128 - __clzll(holds.r64)
           : holds.r0   ? 64 - __clzll(holds.r0)
                        : 0;
  }
  // the rows behind the tile that these take hold no pair
  const int done = live > 128 ? 256 : live > 64 ? 128 : live > 0 ? 64 : 0;
  const int blocks = (int)min((int64_t)kTileN / 16, p.N / 16 - cb0) / (p.silu_mul ? 2 : 1);
  const int64_t block0 = p.silu_mul ? cb0 / 2 : cb0, cols = p.silu_mul ? p.N / 2 : p.N;
  for (int row = done + threadIdx.x / 64; row < rows; row += 8)
    if (lane < blocks * 4) store_out(p, (m0 + row) * cols + block0 * 16 + lane * 4, floatx4{0.0f, 0.0f, 0.0f, 0.0f});
  // whole tiles of whole rows are the fast ones: where the rows end inside the last tile it
  // starts early (1000 rows, 8192 x 7168, MX4 x: 66 -> 45 us; bf16 x: 163 -> 112)
  const int early = !p.tile_expert && rows < done && p.M >= done ? done - rows : 0;
  const int64_t from = m0 - early;
  if (TOP == 256 && done == 256) mx4_tile<XMX, TOP, DS>(p, lds, from, cb0, e, holds, early);
  else if (TOP >= 128 && done == 128)
    mx4_tile<XMX, TOP >= 128 ? 128 : 64, DS>(p, lds, from, cb0, e, holds, early);
  else if (done == 64) mx4_tile<XMX, 64, DS>(p, lds, from, cb0, e, holds, early);
}

template <bool XMX, int TM>
static hipError_t tiled(const Mx4Gemm& p, hipStream_t stream) {
  const int64_t m_tiles = ceil_div(p.M, TM), n_tiles = ceil_div(p.N, kTileN);
  int pn = 8;
  while (pn > n_tiles) pn /= 2;
  const int64_t n_patches = ceil_div(n_tiles, pn);
  const bool tail = m_tiles * n_tiles <= kTailTiles;
  // parts of tiles fill a round at most: 16 patches, and one more for each part of the
  // columns in which their rows end
  const int64_t patches = ceil_div(m_tiles, 32 / pn) * n_patches + (tail ? 16 + 2 * n_patches : 0);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(ceil_div(patches, 8) * 256)), dim3(512), 0, stream, p,
                       (int)m_tiles, (int)n_tiles, pn, (int)n_patches,
                       (int)(p.tile_expert ? p.BM / TM : 1), (int)tail);
  };
  if constexpr (XMX) {
    go(mx4_tile_kernel<XMX, TM, false>);
  } else {
    const bool dma_scales = p.K % 128 == 0 && reinterpret_cast<uintptr_t>(p.w_scale) % 4 == 0;
    if (dma_scales) go(mx4_tile_kernel<XMX, TM, true>);
    else go(mx4_tile_kernel<XMX, TM, false>);
  }
  return hipGetLastError();
}

template <bool XMX, int MB, int NB, int WV>
static hipError_t stream(const Mx4Gemm& p, hipStream_t stream) {
  const int64_t col_groups = ceil_div(p.N / 16, NB), row_groups = ceil_div(p.M, 16 * MB);
  const bool spread = row_groups >= kSpreadGroups;
  const size_t staged = p.K <= kStageK ? (size_t)(NB + (XMX ? MB : 0)) * 16 * (p.K / 32) : 0;
  const auto kernel = mx4_stream_kernel<XMX, MB, NB, WV>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(mx4_stream_groups(row_groups) * col_groups)),
                     dim3(64 * WV), staged, stream, p, (int)row_groups, (int)col_groups, (int)spread);
  return hipGetLastError();
}

// A workgroup of 4 waves and 16 NB columns, or, where those would not fill the chip, of
// WIDE waves and 32 columns (2112 columns for one row: 13 us against 24).
template <bool XMX, int MB, int NB, int WIDE>
static hipError_t few(const Mx4Gemm& p, hipStream_t s) {
  if (ceil_div(p.M, 16 * MB) * ceil_div(p.N, 16 * NB) >= 512) return stream<XMX, MB, NB, 4>(p, s);
  return stream<XMX, MB, 2, WIDE>(p, s);
}

// With more than 64 tiles of 64 rows x 256 columns a workgroup takes a tile.  Below that the
// chip is filled by streaming 32 or 64 columns at a time past the same rows again: 4096 x
// 7168 for 64, 256 and 384 rows of MX4 15, 24 and 40 us streamed and 32, 34 and 34 in
// tiles, of bf16 31, 59 and 86 against 69, 74 and 73.
template <bool XMX>
static hipError_t product(const Mx4Gemm& p, hipStream_t s) {
  // rows of a workgroup: within one tile_expert entry, or those there are
  const int64_t rows = p.tile_expert ? p.BM : p.M;
  auto takes = [&](int64_t n) { return p.tile_expert ? rows % n == 0 : rows > n / 2; };
  if (takes(64)) {
    if (ceil_div(p.M, 64) * ceil_div(p.N, kTileN) <= 64) return few<XMX, 4, 2, 8>(p, s);
    if (takes(256)) return tiled<XMX, 256>(p, s);
    if (takes(128)) return tiled<XMX, 128>(p, s);
    return tiled<XMX, 64>(p, s);
  }
  if (takes(32)) return few<XMX, 2, 4, 8>(p, s);
  return few<XMX, 1, 4, 16>(p, s);
}

hipError_t launch_mx4_gemm(const Mx4Gemm& p, hipStream_t s) {
  return p.x_mx4 ? product<true>(p, s) : product<false>(p, s);
}

}  // namespace moelora
