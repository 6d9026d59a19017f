// Host-side launchers of the gfx950 MoE-LoRA kernels (internal to the library;
// the public surface is the C ABI in include/moe_lora.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moelora {

// ---- align -----------------------------------------------------------------
struct AlignWs {
  int64_t nchunks;
  size_t rank_off, cnt_off, bstart_off, btotal_off, bytes;
};
AlignWs align_ws_layout(int64_t num_pairs, int64_t num_keys);
int64_t align_chunk_pairs(int64_t num_pairs, int64_t num_keys);

// rows of the align outputs: P + min(P, E*(L+1)) * (BM - 1), rounded up to BM
inline int64_t align_capacity(int64_t P, int64_t E, int64_t L, int64_t BM) {
  int64_t K = E * (L + 1);
  int64_t nb = P < K ? P : K;
  int64_t rows = P + nb * (BM - 1);
  return (rows + BM - 1) / BM * BM;
}

// debug_word: the device flag word of MOE_LORA_DEBUG builds (null: no checks)
hipError_t launch_info(int32_t num_tokens, int32_t num_reqs, int32_t num_loras,
                       const int32_t* seg_indptr, const int32_t* weight_indices,
                       const int32_t* lora_ranks, int32_t* adapter_enabled,
                       int32_t* token_lora_mapping, uint32_t* debug_word, hipStream_t stream);

// The device flag word of this build on the current device (null in release
// builds), and reading / clearing it after a stream synchronisation.
uint32_t* debug_word();
hipError_t debug_word_read(uint32_t* flags, bool clear, hipStream_t stream);

int route_max_k();
hipError_t launch_route(int32_t T, int32_t E, int32_t k, const float* logits, int32_t* topk_ids,
                        float* topk_weights, hipStream_t stream);

hipError_t launch_align(int32_t T, int32_t k, int32_t E, int32_t L, int32_t BM,
                        const int32_t* topk_ids, const int32_t* mapping, const int32_t* enabled,
                        int32_t* sorted_ids, int32_t* tile_expert, int32_t* tile_lora,
                        int32_t* expert_tile_offsets, int32_t* num_rows_padded, int32_t* pair_rows,
                        void* workspace, uint32_t* debug_word, hipStream_t stream);

// ---- rows in expert order --------------------------------------------------
// The layout of align seen from both sides: sorted_ids[row] = pair (or >= P for a
// pad), pair_rows[pair] = row (or -1 for a pair without one).
struct RowsLayout {
  int32_t T, k;
  int64_t num_rows;                  // rows the buffers hold
  const int32_t *sorted_ids, *pair_rows, *num_rows_padded;
};
// rows[pair_rows[t k + j]] = x[t] (elements of 1, 2 or 4 bytes); pads are zeroed
hipError_t launch_permute(const RowsLayout& l, int64_t hidden, int elem_bytes, const void* x,
                          void* rows, hipStream_t stream);
// y[t] = sum_j weights[t k + j] rows[pair_rows[t k + j]] (weights null: ones)
hipError_t launch_unpermute(const RowsLayout& l, int64_t hidden, bool rows_f32, bool y_f32,
                            const void* rows, const float* weights, void* y, hipStream_t stream);
// d_rows[pair_rows[t k + j]] = weights[t k + j] dy[t], pads zeroed;
// d_weights[t k + j] = dy[t] . rows[pair_rows[t k + j]] (null: not computed)
hipError_t launch_unpermute_backward(const RowsLayout& l, int64_t hidden, bool rows_f32,
                                     bool dy_f32, const void* dy, const void* rows,
                                     const float* weights, void* d_rows, float* d_weights,
                                     hipStream_t stream);

// ---- MX4 -------------------------------------------------------------------
hipError_t launch_mx4_quantize(bool x_f32, int64_t num_rows, int64_t cols, const void* x,
                               const int32_t* rows_used, uint8_t* codes, uint8_t* scales,
                               hipStream_t stream);
hipError_t launch_mx4_dequantize(bool out_f32, int64_t num_rows, int64_t cols,
                                 const uint8_t* codes, const uint8_t* scales, void* out,
                                 hipStream_t stream);
struct Mx4Gemm {
  int64_t M, N, K, E, BM;            // BM: rows of a tile_expert entry
  bool x_mx4, out_f32, silu_mul;
  const void* x;                     // [M, K] bf16, or MX4 codes [M, K / 2]
  const uint8_t* x_scale;            // MX4 x: [M, K / 32]
  const uint8_t* w;                  // [E, N, K / 2]
  const uint8_t* w_scale;            // [E, N, K / 32]
  const int32_t* tile_expert;        // [M / BM], null: one weight for all rows
  const int32_t* row_ids;            // [M], null, or rows outside [0, num_ids) are pads
  int32_t num_ids;
  void* out;                         // [M, N], or [M, N / 2] with silu_mul
};
hipError_t launch_mx4_gemm(const Mx4Gemm& p, hipStream_t stream);
// groups of rows that the streaming kernel launches: from kSpreadGroups on they come in
// sixteens, two for each XCD
constexpr int64_t kSpreadGroups = 32;
inline int64_t mx4_stream_groups(int64_t groups) {
  return groups >= kSpreadGroups ? (groups + 15) / 16 * 16 : groups;
}
// its workgroups of 64 columns for blocks that 64 does not divide, 0 for the others (more
// than 64 tiles of 64 x 256 never go through it)
inline int64_t mx4_stream_blocks(int64_t num_rows, int64_t out_features, int32_t block_m) {
  if (block_m % 64 == 0) return 0;
  const int64_t rows = block_m % 32 ? 16 : 32;
  return mx4_stream_groups((num_rows + rows - 1) / rows) * ((out_features + 63) / 64);
}

// ---- 8-bit integers --------------------------------------------------------
struct Int8Rows {
  int64_t num_rows, cols;
  bool x_f32, weight_f32, y_f32;
  const void* x;                     // [num_rows, cols]
  const int32_t* rows_used;          // null, or rows from *rows_used on are skipped
  // the norm (weight null: x is quantized as it is)
  const void* weight;                // [cols]
  const void* residual;              // [num_rows, cols] or null
  double eps, per_col;               // per_col: 1 / cols
  void* residual_out;                // null, or x + residual
  void* y;                           // null, or the norm
  int8_t* codes;                     // [num_rows, cols]
  float* scales;                     // [num_rows]
};
constexpr int64_t kMaxNormCols = 16384;   // a row in the registers of a workgroup
hipError_t launch_int8_rows(const Int8Rows& p, hipStream_t stream);
hipError_t launch_int8_dequantize(bool out_f32, int64_t num_rows, int64_t cols, const int8_t* codes,
                                  const float* scales, void* out, hipStream_t stream);
struct Int8Gemm {
  int64_t M, N, K, E, BM;            // BM: rows of a tile_expert entry
  bool out_f32, silu_mul;
  const int8_t* x;                   // [M, K], or [T, K] with top_k
  const float* x_scale;              // [M] or [T]
  const int8_t* w;                   // [E, N, K]
  const float* w_scale;              // [E, N]
  const int32_t* tile_expert;        // [M / BM], null: one weight for all rows
  const int32_t* row_ids;            // [M], null, or rows outside [0, num_ids) are pads
  int32_t num_ids;
  int32_t top_k;                     // > 0: row m reads row row_ids[m] / top_k of x
  void* out;                         // [M, N], or [M, N / 2] with silu_mul
};
hipError_t launch_int8_gemm(const Int8Gemm& p, hipStream_t stream);
// In blocks of 16 rows with up to 14 rows an expert, and of 32 rows with up to 20, weights are streamed
// for each block; with more, a tile takes 64 rows of an expert.  Layers (run_int8_layer in a graph)
// streamed and by tiles, us, with 12, 16, 20, 24 and 32 rows an expert:
//   32 experts of 4096 x 2048   blocks of 16   225, 250, 283, 299, 354   246, 251, 253, 224, 255
//                               blocks of 32   213, 221, 228, 233, 281   234, 235, 236, 235, 262
//   128 experts of 2048 x 768   blocks of 16   180, 206, 229, 244, 283   168, 172, 179, 178, 195
//                               blocks of 32   191, 195, 201, 207, 243   175, 176, 177, 181, 202
//   16 experts of 4096 x 6144   blocks of 16   305, 354, 412, 438, 509   313, 316, 334, 333, 337
//                               blocks of 32   295, 307, 315, 321, 399   308, 307, 307, 309, 336
inline bool int8_few_rows(const Int8Gemm& p) {
  // rows that hold a pair, about: without their number half of the blocks' last rows do not
  const int64_t held = p.row_ids ? p.num_ids : p.M - p.E * p.BM / 2;
  return p.BM <= 32 && held <= (p.BM == 16 ? 14 : 20) * p.E;
}

// ---- balance loss ----------------------------------------------------------
struct Balance {
  int32_t T, E, k;
  bool logits_f32;
  const void* logits;                // [T, E]
  const int32_t* topk_ids;           // [T, k]
  const uint8_t* mask;               // [T] or null: nonzero takes part
};
constexpr int64_t kMaxBalanceExperts = 1024;   // 16 registers of a wave
size_t balance_ws_bytes(int64_t T, int64_t E);
hipError_t launch_balance_loss(const Balance& b, float* loss, int32_t* counts, float* mean_probs,
                               int32_t* num_valid, void* workspace, hipStream_t stream);
hipError_t launch_balance_loss_backward(const Balance& b, bool out_f32, const int32_t* counts,
                                        const int32_t* num_valid, const float* d_loss, void* d_logits,
                                        hipStream_t stream);

// ---- forward ---------------------------------------------------------------
// expert weights as fp8 e4m3 codes with 128 x 128 block scales (dtype bf16)
constexpr int kWeightFp8 = 2;

struct ForwardProblem {
  int dtype;  // 0 = fp32, 1 = bf16
  int wdtype = 0;  // dtype of the expert weights: dtype, or kWeightFp8
  const float* w_gate_up_scale = nullptr;   // fp8: [E, 2I/128, H/128]
  const float* w_down_scale = nullptr;      // fp8: [E, H/128, I/128]
  int64_t T, H, I, E, k, L, R, BM;
  const void* x;
  const float* topk_weights;
  const void *w_gate_up, *w_down;
  const void *a_gate, *a_up, *b_gate, *b_up, *a_down, *b_down;
  const int32_t* lora_ranks;
  const float* scaling;
  const int32_t *sorted_ids, *tile_expert, *tile_lora, *expert_tile_offsets, *num_rows_padded;
  void* y;
  int out_f32;  // y in fp32 instead of dtype
};

struct ForwardWs {
  int64_t cap, max_items, RP;
  int64_t n_tiles_gu = 0, n_tiles_dn = 0;   // column tiles (x K splits) of the two GEMMs
  size_t items_off, count_off, tab_gu_off, tab_dn_off, slot_rank_off, hgu_off, act_off, hd_off, z_off,
      part_off = 0, bytes;
  int64_t grid_gu = 0;             // workgroups of the general gate_up GEMM (0: tail split unused)
  int split_gu = 1, split_d = 1;   // K splits of the two shrinks
  bool shrink4 = false;            // shrinks share pool rows across 4 row groups
  int split_down_k = 1;            // K splits of the down GEMM (planes of z)
  bool big = false;                // the large-tile bf16 GEMMs (256-row items)
  int rows_per_item = 0;           // rows of a GEMM work item
};
ForwardWs forward_ws_layout(const ForwardProblem& p);
// stages of the forward, in launch order (index into the optional event pairs)
enum { kStagePlan = 0, kStageShrinkX, kStageGateUp, kStageShrinkA, kStageDown, kStageCombine,
       kNumStages };
hipError_t launch_forward(const ForwardProblem& p, void* workspace, hipStream_t stream,
                          hipEvent_t* events);

// The allocation-free forward's workspace: a static device array of this many
// bytes, one per device; noalloc_scratch returns the current device's address.
constexpr size_t kNoAllocScratchBytes = size_t(64) << 20;
hipError_t noalloc_scratch(void** ptr);

// A dense projection with per-request LoRA whose output is two column slices
// [0, N0) and [N0, N0 + N1), each with its own LoRA factors (N1 may be 0).
struct DenseProblem {
  int dtype;  // 0 = fp32, 1 = bf16
  int64_t T, H, N0, N1, L, R, BM;
  const void* x;                       // [T, H]
  const void* w;                       // [N0 + N1, H]
  const void *a0, *a1, *b0, *b1;       // [L, R, H] x2, [L, R, N0], [L, R, N1]
  const int32_t* lora_ranks;
  const float* scaling;
  const int32_t *sorted_ids, *tile_expert, *tile_lora, *expert_tile_offsets, *num_rows_padded;
  void* y;                             // [T, N0 + N1]
  int out_f32;
};
struct DenseWs {
  int64_t cap, max_items, RP;
  int npool = 1, split = 1, ksplit = 1;   // shrink pools / shrink K splits / GEMM K splits
  int64_t n_tiles = 0;                    // GEMM column tiles x K splits
  size_t items_off, count_off, tab_off, slot_rank_off, h_off, z_off, bytes;
};
DenseWs dense_ws_layout(const DenseProblem& p);
enum { kDenseStagePlan = 0, kDenseStageShrink, kDenseStageGemm, kDenseStageCombine, kDenseNumStages };
hipError_t launch_dense(const DenseProblem& p, void* workspace, hipStream_t stream, hipEvent_t* events);

}  // namespace moelora
