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
#include "gemm_common.hpp"
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

// ---- many rows -------------------------------------------------------------
// Tiles of TM rows x 256 weight rows, K in steps of 128-byte LDS rows of x: 256
// values of MX4 x or 64 of bf16.  Codes reach LDS by global -> LDS DMA in a ring of
// two slots; scales take the long way through registers, because their rows need not be
// aligned.
// Eight waves as 2 x 4, each (TM / 2) x 64.
//
// A K tile is two steps.  In a step a wave keeps its four weight fragments in
// registers and takes the 16-row blocks of x one after another, four MFMAs each,
// reading the block that comes kAhead later meanwhile.  When the last fragments of
// a tile have been read, a barrier admits the next tile; behind it the wave starts
// the DMA of the tile after next into the slot just left and reads the next tile's
// first fragments under the MFMAs that remain.
//
// LDS rows of x (and of MX4 weights) are eight 16-byte chunks, chunk c of a row in
// place c ^ ((row >> 1) & 7): the 16 rows of a fragment read then fall on all banks.
constexpr int kTileN = 256;

__device__ __attribute__((aligned(16))) uint32_t mx4_zeros[4];   // what lies behind a row's end

// as dma16, with an address per lane
__device__ __forceinline__ void dma16_lane(const void* p, uint32_t lds_addr) {
  const uint32_t la = __builtin_amdgcn_readfirstlane(lds_addr);
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %[sv], m0\n\t"
      "s_mov_b32 m0, %[la]\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %[p], off\n\t"
      "s_mov_b32 m0, %[sv]"
      : [sv] "=&s"(saved)
      : [la] "s"(la), [p] "v"((uint64_t)(uintptr_t)p)
      : "memory");
}

// this wave's DMA and LDS accesses are done, then every wave's
__device__ __forceinline__ void wait_all_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// COUNT (4 or 16) scale bytes of a row from block b0 on
template <int COUNT> struct ScaleWords { typedef uint32_t type __attribute__((ext_vector_type(COUNT / 4))); };
template <> struct ScaleWords<4> { typedef uint32_t type; };
template <int COUNT>
__device__ __forceinline__ typename ScaleWords<COUNT>::type load_scales(const uint8_t* row, int b0) {
  typename ScaleWords<COUNT>::type v;
  __builtin_memcpy(&v, row + b0, COUNT);
  return v;
}

template <bool XMX, int TM>
__global__ void __launch_bounds__(512) mx4_tile_kernel(
    Mx4Gemm p, int m_tiles, int n_tiles, int pn, int n_patches) {
  constexpr int WM = 2, WN = 4, NW = WM * WN, NT = 64 * NW;
  constexpr int MB = TM / 16 / WM, NB = kTileN / 16 / WN;   // 16-row blocks of a wave
  constexpr int WROWB = XMX ? 128 : 32;                     // LDS bytes of a weight row
  constexpr int XSTAGE = TM * 128, STAGE = XSTAGE + kTileN * WROWB;
  constexpr int SROWS = (XMX ? TM : 0) + kTileN;            // rows with scales; x's come first
  constexpr int KB = XMX ? 8 : 2;                           // blocks of 32 in a K tile
  constexpr int SB = 2 * KB;                                // scale bytes of a row for two K tiles
  constexpr int SPT = (SROWS + NT - 1) / NT;                // scale rows of a thread
  __shared__ __attribute__((aligned(1024))) char lds[2 * STAGE + 2 * SROWS * SB];

  // patches of (32 / pn) x pn tiles go round the eight XCDs (workgroup b runs on
  // XCD b % 8), so the 32 workgroups that an XCD holds share rows and weights in its L2
  const int pm = 32 / pn;
  const int patch = (int)(blockIdx.x / 256) * 8 + (int)(blockIdx.x % 8);
  const int in = (int)(blockIdx.x / 8) % 32;
  const int mt = patch / n_patches * pm + in % pm, nt = patch % n_patches * pn + in / pm;
  if (mt >= m_tiles || nt >= n_tiles) return;
  const int64_t m0 = (int64_t)mt * TM;
  const int64_t cb0 = (int64_t)nt * (kTileN / 16), ncb = p.N / 16;
  int64_t e = 0;
  if (p.tile_expert) {
    e = __builtin_amdgcn_readfirstlane(p.tile_expert[m0 / p.BM]);
    if (e < 0 || e >= p.E) return;
  }
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
  auto swz = [](int row) { return (row >> 1) & 7; };
  // weight row of LDS row n (rows of column blocks behind the last repeat it)
  auto w_row = [&](int n) { return weight_row(p, min(cb0 + n / 16, ncb - 1)) + n % 16; };

  // One KB of LDS per DMA: 8 rows of x or MX4 weights, 32 of the weights beside
  // bf16 x.  The 8 rows of a segment lie at a uniform base, so two offsets per
  // lane (the swizzle of even and of odd segments) serve them all.  A tile behind
  // the end of K or of M takes an address per lane instead, worked out on the spot
  // (kept over the loop, the addresses would cost more registers than there are).
  constexpr int XSEG = XSTAGE / 1024 / NW, WSEG = kTileN * WROWB / 1024 / NW;
  static_assert(XSEG % 2 == 0 && (!XMX || WSEG % 2 == 0), "segments come in pairs");
  uint32_t lane_off[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    lane_off[h] = (uint32_t)(lane / 8 * (int)x_row + ((lane % 8) ^ swz(h * 8 + lane / 8)) * 16);
  const bool all_rows = m_last == TM - 1;
  auto issue = [&](int t, int slot, auto fast) {   // fast: a whole tile of whole rows
    const uint32_t at = lds0 + slot * STAGE;
    if constexpr (decltype(fast)::value) {
#pragma unroll
      for (int i = 0; i < XSEG; ++i) {
        const int seg = wave * XSEG + i;
        dma16(x_base + seg * 8 * x_row, lane_off[i % 2] + t * 128, at + seg * 1024);
      }
    } else {
      int l = lane;
      asm volatile("" : "+v"(l));
#pragma unroll
      for (int i = 0; i < XSEG; ++i) {
        const int seg = wave * XSEG + i, row = seg * 8 + l / 8, c = (l % 8) ^ swz(row);
        // chunks of 16 bytes: a block of MX4, a quarter of one in bf16
        const bool in_row = t * KB + (XMX ? c : c / 4) < nblk;
        const char* src = x_base + min(row, m_last) * x_row + t * 128 + c * 16;
        dma16_lane(in_row ? (const void*)src : (const void*)mx4_zeros, at + seg * 1024);
      }
    }
    if constexpr (XMX && decltype(fast)::value) {
#pragma unroll
      for (int i = 0; i < WSEG; ++i) {
        const int seg = wave * WSEG + i;
        dma16(w_base + w_row(seg * 8) * (p.K / 2), lane_off[i % 2] + t * 128,
              at + XSTAGE + seg * 1024);
      }
    } else {
      int l = lane;
      asm volatile("" : "+v"(l));
#pragma unroll
      for (int i = 0; i < WSEG; ++i) {
        const int seg = wave * WSEG + i;
        const int row = XMX ? seg * 8 + l / 8 : seg * 32 + l / 2;
        const int c = XMX ? (l % 8) ^ swz(row) : l % 2;
        const uint8_t* src = w_base + w_row(row) * (p.K / 2) + t * WROWB + c * 16;
        dma16_lane(t * KB + c < nblk ? (const void*)src : (const void*)mx4_zeros,
                   at + XSTAGE + seg * 1024);
      }
    }
  };

  // scale rows of this thread, and their way through registers into LDS
  const uint8_t* s_row[SPT];
  // The scales of tiles 2 grp and 2 grp + 1 go through registers into LDS: the load
  // behind the barrier of the even tile before them, the store ahead of that of
  // the odd one.
  typename ScaleWords<SB>::type s_val[SPT];
#pragma unroll
  for (int i = 0; i < SPT; ++i) {
    const int q = min((int)threadIdx.x + i * NT, SROWS - 1);
    if (XMX && q < TM) s_row[i] = p.x_scale + (m0 + min(q, m_last)) * nblk;
    else s_row[i] = p.w_scale + (e * p.N + w_row(q - (XMX ? TM : 0))) * nblk;
  }
  auto scales_load = [&](int grp, auto fast) {   // fast: both tiles are whole
#pragma unroll
    for (int i = 0; i < SPT; ++i) {
      if (decltype(fast)::value || (grp + 1) * SB <= nblk) {
        s_val[i] = load_scales<SB>(s_row[i], grp * SB);
      } else {
        // 2^0 behind the end of the row
        uint8_t bytes[SB];
#pragma unroll
        for (int b = 0; b < SB; ++b) bytes[b] = grp * SB + b < nblk ? s_row[i][grp * SB + b] : 127;
        __builtin_memcpy(&s_val[i], bytes, SB);
      }
    }
  };
  char* const s_lds = lds + 2 * STAGE;
  auto scales_store = [&](int grp) {
#pragma unroll
    for (int i = 0; i < SPT; ++i) {
      const int q = (int)threadIdx.x + i * NT;
      if (SROWS % NT == 0 || q < SROWS)
        __builtin_memcpy(s_lds + ((grp & 1) * SROWS + q) * SB, &s_val[i], SB);
    }
  };

  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  constexpr int kAhead = 3, kRing = 4;
  static_assert((2 * MB) % kRing == 0 && MB > kAhead, "the ring starts each tile at its first place");
  // of a K tile.  MX4: a word holds the bytes of both steps of two neighbouring
  // blocks; bf16 x: the weights' codes of both steps, and their scale bytes
  struct TileScales {
    int xs[XMX ? MB / 2 : 1], ws[XMX ? NB / 2 : NB];
    u32x2 codes[XMX ? 1 : NB];
  };
  // places of this lane's row of a wave's first block; a block is 16 rows further
  int x_at[2], w_at[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = ((2 * g + h) ^ swz(r)) * 16;
    x_at[h] = (wm * MB * 16 + r) * 128 + c;
    w_at[h] = XSTAGE + (wn * NB * 16 + r) * 128 + c;
  }
  const int codes_at = XSTAGE + (wn * NB * 16 + r) * 32 + g * 8;
  const int xs_at = 2 * STAGE + (wm * MB * 16 + r) * SB + 2 * g;
  const int ws_at = 2 * STAGE + ((XMX ? TM : 0) + wn * NB * 16 + r) * SB + (XMX ? 2 * g : g >> 1);
  auto read_x = [&](int slot, int i, int step) {
    return *reinterpret_cast<const u32x4*>(lds + slot * STAGE + x_at[step] + i * 2048);
  };
  auto read_w = [&](int slot, int j, int step) {
    return *reinterpret_cast<const u32x4*>(lds + slot * STAGE + w_at[step] + j * 2048);
  };
  auto read_scales = [&](TileScales& f, int slot, int t) {
    const char* s = lds + ((t / 2) & 1) * SROWS * SB + slot * KB;
    if constexpr (XMX) {
      typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
      auto two = [&](const char* at) {
        u16x2 v;
        v[0] = *reinterpret_cast<const uint16_t*>(at);
        v[1] = *reinterpret_cast<const uint16_t*>(at + 16 * SB);
        return __builtin_bit_cast(int, v);
      };
#pragma unroll
      for (int i = 0; i < MB; i += 2) f.xs[i / 2] = two(s + xs_at + i * 16 * SB);
#pragma unroll
      for (int j = 0; j < NB; j += 2) f.ws[j / 2] = two(s + ws_at + j * 16 * SB);
    } else {
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        f.codes[j] = *reinterpret_cast<const u32x2*>(lds + slot * STAGE + codes_at + j * 512);
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
  auto read_first = [&](TileScales& f, int t) {
    const int slot = t & 1;
    read_scales(f, slot, t);
    if constexpr (XMX) {
#pragma unroll
      for (int j = 0; j < NB; ++j) w0[j] = read_w(slot, j, 0);
    }
  };
  // kEven, kOdd: a tile of that number with two whole tiles of whole rows or more
  // behind the next; kAny: any but the last
  enum { kEven, kOdd, kAny, kLast };
  auto tile = [&](int t, auto mode) {
    constexpr int kMode = decltype(mode)::value;
    const int slot = t & 1;
    if constexpr (!XMX) {
#pragma unroll
      for (int j = 0; j < NB; ++j) w0[j] = expand(sc, j, 0);
    }
    static_for<MB>([&](auto I) {
      constexpr int i = decltype(I)::value, q = i + kAhead;
      x[q % kRing] = q < MB ? read_x(slot, q, 0) : read_x(slot, q - MB, 1);
      if constexpr (i < NB) w1[i] = XMX ? read_w(slot, i, 1) : expand(sc, XMX ? 0 : i, 1);
      multiply(first, I, w0);
      __builtin_amdgcn_sched_barrier(0);
    });
    TileScales next;
    static_for<MB>([&](auto I) {
      constexpr int i = decltype(I)::value, q = MB + i + kAhead;
      if constexpr (i + kAhead < MB) {
        x[q % kRing] = read_x(slot, i + kAhead, 1);
      } else if constexpr (kMode != kLast) {
        if constexpr (i + kAhead == MB) {
          pin();
          if (kMode == kOdd || (kMode == kAny && (t & 1))) scales_store((t + 1) / 2);
          wait_all_barrier();
          if constexpr (kMode != kAny) issue(t + 2, slot, std::true_type{});
          else if (t + 2 < tiles) issue(t + 2, slot, std::false_type{});
          if constexpr (kMode == kEven) scales_load(t / 2 + 1, std::true_type{});
          else if (kMode == kAny && !(t & 1) && t + 2 < tiles) scales_load(t / 2 + 1, std::false_type{});
          read_first(next, t + 1);
        }
        x[q % kRing] = read_x(slot ^ 1, i + kAhead - MB, 0);
      }
      multiply(second, I, w1);
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr (kMode != kLast) sc = next;
  };

  scales_load(0, std::false_type{});
  scales_store(0);
  issue(0, 0, std::false_type{});
  wait_all_barrier();
  if (tiles > 1) issue(1, 1, std::false_type{});
  read_first(sc, 0);
#pragma unroll
  for (int i = 0; i < kAhead; ++i) x[i] = read_x(0, i, 0);
  int t = 0;
  if (all_rows) {
    for (; (t + 4) * KB <= nblk; t += 2) {
      tile(t, std::integral_constant<int, kEven>{});
      tile(t + 1, std::integral_constant<int, kOdd>{});
    }
  }
  for (; t + 1 < tiles; ++t) tile(t, std::integral_constant<int, kAny>{});
  tile(t, std::integral_constant<int, kLast>{});

#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int row = (wm * MB + i) * 16 + r;
    if (row > m_last) continue;
    const int64_t m = m0 + row;
    if (p.silu_mul) {
#pragma unroll
      for (int j = 0; j < NB; j += 2) {
        const int64_t cb = cb0 + wn * NB + j;
        if (cb + 1 >= ncb) continue;
        floatx4 v;
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = silu_f(acc[i][j][q]) * acc[i][j + 1][q];
        store_out(p, m * (p.N / 2) + cb / 2 * 16 + 4 * g, v);
      }
    } else {
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int64_t cb = cb0 + wn * NB + j;
        if (cb < ncb) store_out(p, m * p.N + cb * 16 + 4 * g, acc[i][j]);
      }
    }
  }
}

template <bool XMX, int TM>
static hipError_t tiled(const Mx4Gemm& p, hipStream_t stream) {
  const int64_t m_tiles = ceil_div(p.M, TM), n_tiles = ceil_div(p.N, kTileN);
  int pn = 8;
  while (pn > n_tiles) pn /= 2;
  const int64_t n_patches = ceil_div(n_tiles, pn);
  const int64_t patches = ceil_div(m_tiles, 32 / pn) * n_patches;
  const auto kernel = mx4_tile_kernel<XMX, TM>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(ceil_div(patches, 8) * 256)), dim3(512), 0,
                     stream, p, (int)m_tiles, (int)n_tiles, pn, (int)n_patches);
  return hipGetLastError();
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
  // whole tiles of 128 rows and more
  const bool r256 = p.tile_expert ? rows % 256 == 0 : rows > 128;
  const bool r128 = p.tile_expert ? rows % 128 == 0 : rows > 64;
  if (p.x_mx4) {
    if (r256) return tiled<true, 256>(p, s);
    if (r128) return tiled<true, 128>(p, s);
    if (r64) return stream<true, 4, 2, 4>(p, s);
    if (r32) return stream<true, 2, 4, 4>(p, s);
    return stream<true, 1, 4, 4>(p, s);
  }
  if (r256) return tiled<false, 256>(p, s);
  if (r128) return tiled<false, 128>(p, s);
  if (r64) return stream<false, 4, 2, 4>(p, s);
  if (r32) return stream<false, 2, 4, 4>(p, s);
  return stream<false, 1, 4, 4>(p, s);
}

}  // namespace moelora
