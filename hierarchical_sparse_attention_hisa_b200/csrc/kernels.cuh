// Launchers of the HISA kernels; called by the C ABI in api.cu.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "hsa.h"

namespace hsa {

// Counts kernel launches made by this library (see hsa_kernel_launches).
void count_launches(int n);

// Launches kern<<<grid, block, smem, s>>>(args...); with pdl set, as a
// programmatic dependent launch (the kernel must begin with griddep_wait()).
template <typename... KArgs, typename... Args>
inline void launch_kernel(bool pdl, void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                          Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = pdl ? 1 : 0;
  (void)cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// 2-D row-major bf16 [rows][cols] TMA map, box {64 columns, box_rows rows},
// 128-byte swizzle. False if the driver entry point or the encoding fails.
bool make_tmap_2d(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows);
int num_sms();

void launch_block_sums(const void* k_idx, int64_t Lk, int B, int d_idx, float* ksum,
                       cudaStream_t s);
void launch_select_blocks(RowMap rm, int64_t rows, const void* q_idx, const float* ksum,
                          int64_t ksum_seq_stride, int B, int m, int d_idx, int32_t* blocks,
                          int64_t max_cand, cudaStream_t s);
// max_cand: the most candidates any row can have (its keys are staged in shared memory)
void launch_select_tokens(RowMap rm, int64_t rows, const void* q_idx, const void* k_idx,
                          const int32_t* blocks, int B, int m, int k, int d_idx, int32_t* indices,
                          int64_t max_cand, cudaStream_t s);
// Tensor-core sparse attention (d = 64 or 128, any H: one launch per group of
// up to 64 heads); returns false if a launch attribute could not be set.
bool tc_attn_supported(int H, int d, int64_t Lq, int64_t Lk);
bool launch_sparse_attn_tc(int64_t Lq, const void* Q, const void* K, const void* V, const int32_t* idx,
                           int64_t Lk, int k, int H, int d, float scale, void* O, cudaStream_t s);
void launch_ksum_split(const float* ksum, int64_t n, void* split, cudaStream_t s);
bool launch_block_score_gemm(const void* q_idx, const void* bsplit, int64_t Lq, int64_t Lk, int B, int m,
                             int d_idx, int64_t nbc, uint32_t* out, int64_t ld, cudaStream_t s);
bool launch_token_score_gemm(const void* q_idx, const void* k_idx, int64_t Lq, int64_t Lk, int B, int m,
                             int d_idx, const int4* tiles, const int* ntiles, const uint32_t* pairs,
                             int64_t max_tiles, uint32_t* out, cudaStream_t s);
void launch_topm_from_keys(RowMap rm, int64_t rows, const uint32_t* bkeys, int64_t ld, int B, int m,
                           int64_t max_cand, int32_t* blocks, cudaStream_t s, bool pdl = false);
void launch_pair_lists(RowMap rm, int64_t rows, const int32_t* blocks, int B, int m, int k, int nbins,
                       int* cnt, int* off, int* cursor, int4* tiles, int* ntiles, uint32_t* pairs,
                       cudaStream_t s);
// Whether launch_topk_from_keys has a CTA with the whole row in shared memory for these sizes.
bool topk_rows_takes(int B, int m);
void launch_topk_from_keys(RowMap rm, int64_t rows, const int32_t* blocks, const uint32_t* tkeys, int B,
                           int m, int k, int32_t* indices, cudaStream_t s, bool pdl = false);
// (also appends each sequence's new token: k_idx/K/V rows and a completed block's sum)
void launch_decode_block_scores(int batch, int64_t capacity, const int32_t* ctx, int B, int m, int d_idx,
                                const void* q_new, const float* ksum_cache, uint32_t* bkeys, int64_t ld,
                                int d, void* k_idx_cache, void* K_cache, void* V_cache, float* ksum_w,
                                const void* k_idx_new, const void* K_new, const void* V_new, cudaStream_t s);
void launch_decode_token_scores(int batch, int64_t capacity, const int32_t* ctx, int B, int m, int d_idx,
                                const int32_t* blocks, const void* q_new, const void* k_idx_cache,
                                uint32_t* tkeys, cudaStream_t s);
// (also advances ctx: every sequence that took the step grows by one token)
void launch_decode_combine(int batch, int64_t capacity, int32_t* ctx, int H, int d, int parts,
                           const float* Opart, const float* mpart, const float* lpart, void* O, cudaStream_t s);
bool launch_sparse_attn_tc_split(int batch, const void* Q, const void* Kc, const void* Vc, const int32_t* idx,
                                 int64_t capacity, int k, int H, int d, float scale, int parts, float* Opart,
                                 float* mpart, float* lpart, cudaStream_t s, bool pdl = false);
// Per-head RMS norm and rotation of queries [L][H][d] and keys [L][d] (either may be null).
void launch_qk_norm_rope(int64_t L, int H, int d, const void* Q, int64_t q_stride, const void* K, int64_t k_stride,
                         const void* qw, const void* kw, float eps, const float* inv_freq, int rot, bool interleaved,
                         const int32_t* positions, int64_t pos0, void* Qo, void* Ko, cudaStream_t s);

// Drafted trees (tree_kernels.cu, tree_scores.cu): T nodes per sequence, row = sequence * T + node.
constexpr int kTreeMax = HSA_TREE_MAX;
struct TreeArgs {
  int T, B, m, k, d;
  int64_t capacity, ldb;           // ldb: row length of bkeys (kBkeys0 keys, then the blocks' from block 0 on)
  const int32_t *ctx, *positions, *paths;
  uint16_t *k_idx_cache, *K_cache, *V_cache;
  const float* ksum_cache;
  const uint16_t *q_new, *k_idx_new, *K_new, *V_new;
  int32_t* rowpos;                 // [rows] position of each node that takes part, else -1
  uint32_t *bkeys, *tailkeys, *tkeys;  // [rows][ldb], [rows][tail_ld], [rows][m][B]
  int tail_ld;
  const int32_t* blocks;           // [rows][m]
  uint32_t* pairs;                 // [rows * m]: node << 16 | slot
  int4* items;                     // (first key row, first pair, pairs | key rows << 16, sequence << 3 | 128-row piece)
  int* counters;                   // [3]: items, pairs, flagged rows
  // the attention's work: items (row, first tile | tiles << 8 | kept rows << 16, part or -1 to write O whole, -)
  // and each CTA's first; the rows that lie in several CTAs (row, first part, parts, -); and of each row the
  // groups of eight heads (bits) whose weights left the range of the fixed reference
  int4* attn_items;
  int* cta_items;                  // [kTreeAttnCtas + 1]
  int4* cut;                       // [kTreeAttnCtas], row -1 behind the last
  int *flags, *flagged;            // [rows] each: the bits, and a list of the rows that have any
  uint16_t* O;                     // [rows][H][d]
  int H;
};
constexpr int kTreeAttnCtas = 148;  // one per SM
constexpr int kBkeys0 = 3;          // so that block 1's key, the first candidate, is on 16 bytes
// A tree's top-k (launch_tree_topk: a wide CTA per row, which writes cache rows itself) against the prefill's
// selection and a mapping launch. The prefill's CTA of 256 threads with the row in shared memory, where it takes
// the row at all (topk_rows_takes), is the faster one with more than 1024 candidates and more rows than the wide
// CTAs, two to an SM, take in one wave. A whole step (us, wide / prefill's):
//   m * B          288 rows    320       512       1024      8192
//   1024           53 / 62*    65 / 74   75 / 84   107 / 118 593 / 659   (* 256 rows)
//   4096           102 / 109   119 / 123 157 / 162 270 / 264 1796 / 1741
//   8192           109 / 114   134 / 132 178 / 175 299 / 283 1960 / 1854
// Rows that it does not take go to selections for a few rows of any length or a warp per row, always slower here:
//   8000 (B = 100) 111 / 121*  131 / 226 172 / 267 302 / 380 2098 / 2319
//   16384          123 / 150   143 / 280 195 / 329 342 / 445 2376 / 2804
constexpr int kWideRows = 296, kWideKeys = 1024;
// Token candidates of a query at position t: all up to it, or those of its m kept blocks.
HSA_DEV int candidates(int t, int B, int m) { return t / B < m ? t + 1 : (m - 1) * B + t % B + 1; }
void launch_tree_plan(int batch, int T, int64_t capacity, const int32_t* ctx, const int32_t* n_nodes,
                      const int32_t* parents, int32_t* positions, int32_t* paths, cudaStream_t s);
// (also appends the drafted rows to the caches, scores every node's tail, and zeroes the O of nodes that take no part)
bool launch_tree_block_scores(const TreeArgs& a, int batch, int d_idx, cudaStream_t s);
// Whether the token scores are few enough to be made without lists (launch_tree_few_scores; else
// launch_tree_lists, then launch_tree_token_scores). Both also cut the attention's work.
bool tree_few_scores(const TreeArgs& a, int64_t rows, int d_idx);
void launch_tree_few_scores(const TreeArgs& a, int64_t rows, int d_idx, cudaStream_t s);
void launch_tree_lists(const TreeArgs& a, int batch, cudaStream_t s);
bool launch_tree_token_scores(const TreeArgs& a, int batch, int d_idx, int64_t max_items, cudaStream_t s);
void launch_tree_topm(const TreeArgs& a, int64_t rows, int32_t* blocks, cudaStream_t s);
// Whether launch_tree_topk takes these rows (else launch_topk_from_keys, then launch_tree_rows).
bool tree_topk_wide(const TreeArgs& a, int64_t rows);
void launch_tree_topk(const TreeArgs& a, int64_t rows, int32_t* idx, cudaStream_t s);
void launch_tree_rows(const TreeArgs& a, int64_t rows, int32_t* idx, cudaStream_t s);
bool launch_tree_attn(const TreeArgs& t, const void* Q, const int32_t* idx, float scale, float* Opart, float* mpart,
                      float* lpart, cudaStream_t s);
void launch_tree_combine(const TreeArgs& a, int64_t rows, const void* Q, const int32_t* idx, float scale,
                         const float* Opart, const float* mpart, const float* lpart, cudaStream_t s);
int tree_attn_wait_flag(bool reset);
bool tree_attn_set_inject(bool on);
void launch_tree_commit(int batch, int T, int64_t capacity, int B, int d_idx, int d, int32_t* ctx,
                        const int32_t* paths, const int32_t* accepted, void* k_idx_cache, void* K_cache,
                        void* V_cache, float* ksum_cache, cudaStream_t s);
int tree_wait_flag(bool reset);
bool tree_set_inject(bool on);

// Sticky per-device flags set by a bounded wait that gave up (1), read on the
// host with a synchronous copy and optionally cleared; -1 on a CUDA error.
int attn_wait_flag(bool reset);
// Test hook of the tensor-core kernels on the current device: short bounded
// waits and one lost producer arrival in the next launch of CTA 0.
bool attn_set_inject(bool on);
bool score_set_inject(bool on);
int score_wait_flag(bool reset);

}  // namespace hsa
