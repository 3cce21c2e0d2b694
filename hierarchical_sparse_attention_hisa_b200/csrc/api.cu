// C ABI of libhsa.so (declared in include/hsa.h): host-side argument checks,
// workspace layout and kernel launches. No allocation, no synchronisation.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "hsa.h"
#include "kernels.cuh"

namespace hsa {
static std::atomic<uint64_t> g_launches{0};
void count_launches(int n) { g_launches.fetch_add(uint64_t(n), std::memory_order_relaxed); }
}  // namespace hsa

namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Blocks of a sequence the block stage scores per query.
constexpr int64_t kMaxBlocks = 16384;
// Token candidates per query (kept blocks x B): the tensor-core token scoring
// with its key-stream top-k takes up to kMaxCandidates, the CUDA-core token
// scoring (block sizes the MMA cannot take) stages them in shared memory and
// takes up to kMaxCandidatesSmem.
constexpr int64_t kMaxCandidates = 65536;
constexpr int64_t kMaxCandidatesSmem = 16384;
constexpr int kMaxM = 512;  // kept blocks per query

int check_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return HSA_ERR_CUDA;
  thread_local int cached_dev = -1, cached_ok = 0;  // per host thread: no shared mutable state
  if (dev != cached_dev) {
    int major = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
      return HSA_ERR_CUDA;
    cached_ok = major == 10;
    cached_dev = dev;
  }
  return cached_ok ? HSA_OK : HSA_ERR_DEVICE;
}

int check_index_params(const hsa_params* p) {
  if (!p) return HSA_ERR_ARG;
  if (p->B < 1 || p->B > 1024) return HSA_ERR_ARG;
  if (p->m < 2 || p->m > kMaxM) return HSA_ERR_ARG;
  if (p->k < 1 || p->k > 8192) return HSA_ERR_ARG;
  if (p->d_idx != 64 && p->d_idx != 128) return HSA_ERR_ARG;
  const bool mma_tokens = p->B == 64 || p->B == 128 || p->B == 256;
  if (int64_t(p->m) * p->B > (mma_tokens ? kMaxCandidates : kMaxCandidatesSmem)) return HSA_ERR_ARG;
  return HSA_OK;
}

int check_attn_params(const hsa_params* p) {
  if (!p) return HSA_ERR_ARG;
  if (p->k < 1 || p->k > 8192) return HSA_ERR_ARG;
  if (p->H < 1 || p->H > 128) return HSA_ERR_ARG;
  if (p->d != 64 && p->d != 128) return HSA_ERR_ARG;
  if (!(p->scale >= 0.f) || std::isinf(p->scale)) return HSA_ERR_ARG;
  return HSA_OK;
}

float softmax_scale(const hsa_params* p) {
  return p->scale > 0.f ? p->scale : 1.0f / std::sqrt(float(p->d));
}

int check_lengths(const hsa_params* p, int64_t Lq, int64_t Lk) {
  if (Lq < 0 || Lk < 1 || Lq > Lk || Lq > (int64_t(1) << 31) - 1) return HSA_ERR_ARG;
  if (Lk > (int64_t(1) << 31) - 1) return HSA_ERR_ARG;
  if (Lk / p->B > kMaxBlocks) return HSA_ERR_ARG;
  return HSA_OK;
}

int launch_status() {
  return cudaGetLastError() == cudaSuccess ? HSA_OK : HSA_ERR_CUDA;
}

// Largest number of block candidates any query of [Lk-Lq, Lk) scores.
int64_t max_block_candidates(const hsa_params* p, int64_t Lk) {
  const int64_t nb = (Lk - 1) / p->B + 1;
  return nb > 2 ? nb - 2 : 1;
}

// Workspace of the indexer (all offsets 256-byte aligned):
//   ksum   [nbc][d_idx] fp32          block sums
//   bsplit [3][nbc][d_idx] bf16       hi/mid/lo planes of ksum
//   bkeys  [Lq][ldb] u32              block-score keys (ldb = nbc rounded to 64)
//   blocks [Lq][m] i32                kept blocks
//   cnt/cursor [nbins] i32            pairs per key block (nbins = ceil(Lk/B))
//   off [2][nbins] i32                first pair and first tile of each key block
//   ntiles i32, tiles [max_tiles] int4, pairs [Lq*m] u32
//   tkeys  [Lq][m][B] u32             token-score keys
struct IndexWs {
  size_t ksum, bsplit, bkeys, blocks, cnt, off, cursor, ntiles, tiles, pairs, tkeys, total;
  int64_t nbc, ldb, nbins, max_tiles;
};
IndexWs index_ws(const hsa_params* p, int64_t Lq, int64_t Lk) {
  IndexWs w{};
  w.nbc = Lk / p->B;
  w.ldb = (w.nbc + 63) / 64 * 64;
  w.nbins = (Lk + p->B - 1) / p->B;
  w.max_tiles = (Lq * p->m + 127) / 128 + w.nbins;
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o += align_up(bytes > 0 ? bytes : 1); return at; };
  w.ksum = take(size_t(w.nbc) * p->d_idx * 4);
  w.bsplit = take(size_t(3) * w.nbc * p->d_idx * 2);
  w.bkeys = take(size_t(Lq) * w.ldb * 4);
  w.blocks = take(size_t(Lq) * p->m * 4);
  w.cnt = take(size_t(w.nbins) * 4);
  w.off = take(size_t(w.nbins) * 8);
  w.cursor = take(size_t(w.nbins) * 4);
  w.ntiles = take(16);
  w.tiles = take(size_t(w.max_tiles) * 16);
  w.pairs = take(size_t(Lq) * p->m * 4);
  w.tkeys = take(size_t(Lq) * p->m * p->B * 4);
  w.total = o;
  return w;
}

// Tensor-core scoring covers d_idx in {64, 128}; block scoring needs a full
// 128-query tile and at least 64 rows of split block sums, token scoring a
// block size the MMA N dimension can take and one full key block.
bool block_gemm_ok(const hsa_params* p, int64_t Lq, int64_t Lk) {
  return Lq >= 128 && 3 * (Lk / p->B) >= 64;
}
bool token_gemm_ok(const hsa_params* p, int64_t Lq, int64_t Lk) {
  return (p->B == 64 || p->B == 128 || p->B == 256) && Lk >= p->B && Lq * int64_t(p->m) < (int64_t(1) << 32);
}

// Kept blocks for rows [0, Lq) from fp32 block sums.
void run_select_blocks(const hsa_params* p, int64_t Lq, int64_t Lk, const void* q_idx, const float* ksum,
                       int32_t* blocks, char* ws, const IndexWs& w, cudaStream_t s, bool* ok) {
  hsa::RowMap rm{Lq, Lk, nullptr, 0};
  const int64_t nb_last = (Lk - 1) / p->B + 1;
  if (nb_last > p->m && p->m > 2 && block_gemm_ok(p, Lq, Lk)) {
    void* bsplit = ws + w.bsplit;
    uint32_t* bkeys = reinterpret_cast<uint32_t*>(ws + w.bkeys);
    hsa::launch_ksum_split(ksum, w.nbc * p->d_idx, bsplit, s);
    if (!hsa::launch_block_score_gemm(q_idx, bsplit, Lq, Lk, p->B, p->m, p->d_idx, w.nbc, bkeys, w.ldb, s)) {
      *ok = false;
      return;
    }
    hsa::launch_topm_from_keys(rm, Lq, bkeys, w.ldb, p->B, p->m, max_block_candidates(p, Lk), blocks, s, true);
  } else {
    hsa::launch_select_blocks(rm, Lq, q_idx, ksum, 0, p->B, p->m, p->d_idx, blocks,
                              max_block_candidates(p, Lk), s);
  }
}

// Kept tokens for rows [0, Lq) from their kept blocks.
void run_select_tokens(const hsa_params* p, int64_t Lq, int64_t Lk, const void* q_idx, const void* k_idx,
                       const int32_t* blocks, int32_t* indices, char* ws, const IndexWs& w, cudaStream_t s,
                       bool* ok) {
  hsa::RowMap rm{Lq, Lk, nullptr, 0};
  if (token_gemm_ok(p, Lq, Lk)) {
    int* cnt = reinterpret_cast<int*>(ws + w.cnt);
    int* off = reinterpret_cast<int*>(ws + w.off);
    int* cursor = reinterpret_cast<int*>(ws + w.cursor);
    int* ntiles = reinterpret_cast<int*>(ws + w.ntiles);
    int4* tiles = reinterpret_cast<int4*>(ws + w.tiles);
    uint32_t* pairs = reinterpret_cast<uint32_t*>(ws + w.pairs);
    uint32_t* tkeys = reinterpret_cast<uint32_t*>(ws + w.tkeys);
    hsa::launch_pair_lists(rm, Lq, blocks, p->B, p->m, p->k, int(w.nbins), cnt, off, cursor, tiles, ntiles,
                           pairs, s);
    if (!hsa::launch_token_score_gemm(q_idx, k_idx, Lq, Lk, p->B, p->m, p->d_idx, tiles, ntiles, pairs,
                                      w.max_tiles, tkeys, s)) {
      *ok = false;
      return;
    }
    hsa::launch_topk_from_keys(rm, Lq, blocks, tkeys, p->B, p->m, p->k, indices, s, true);
  } else {
    // CUDA-core scoring: the row's candidates (at most m*B, at most Lk) in shared memory
    if (std::min<int64_t>(int64_t(p->m) * p->B, Lk) > kMaxCandidatesSmem) {
      *ok = false;
      return;
    }
    hsa::launch_select_tokens(rm, Lq, q_idx, k_idx, blocks, p->B, p->m, p->k, p->d_idx, indices,
                              std::min<int64_t>(int64_t(p->m) * p->B, Lk), s);
  }
}


}  // namespace

extern "C" {

uint64_t hsa_kernel_launches(void) { return hsa::g_launches.load(std::memory_order_relaxed); }

int hsa_device_status(int reset) {
  if (int e = check_device()) return e;
  if (cudaDeviceSynchronize() != cudaSuccess) return HSA_ERR_CUDA;
  const int a = hsa::attn_wait_flag(reset != 0);
  const int b = hsa::score_wait_flag(reset != 0);
  const int c = hsa::tree_wait_flag(reset != 0);
  const int d = hsa::tree_attn_wait_flag(reset != 0);
  if (a < 0 || b < 0 || c < 0 || d < 0) return HSA_ERR_CUDA;
  return a || b || c || d ? HSA_ERR_TIMEOUT : HSA_OK;
}

int hsa_debug_inject_lost_arrival(int on) {
  if (int e = check_device()) return e;
  if (!hsa::attn_set_inject(on != 0) || !hsa::score_set_inject(on != 0) || !hsa::tree_set_inject(on != 0) ||
      !hsa::tree_attn_set_inject(on != 0))
    return HSA_ERR_CUDA;
  return HSA_OK;
}

const char* hsa_status_string(int status) {
  switch (status) {
    case HSA_OK: return "ok";
    case HSA_ERR_ARG: return "invalid argument (null/misaligned pointer or unsupported size)";
    case HSA_ERR_WORKSPACE: return "workspace missing or too small";
    case HSA_ERR_CUDA: return "CUDA launch or runtime error";
    case HSA_ERR_TIMEOUT: return "bounded device wait gave up";
    case HSA_ERR_DEVICE: return "current device is not an sm_100 (B200-class) GPU";
    default: return "unknown status";
  }
}

int hsa_index_workspace_size(const hsa_params* p, int64_t Lq, int64_t Lk, size_t* bytes) {
  if (!bytes) return HSA_ERR_ARG;
  if (int e = check_index_params(p)) return e;
  if (int e = check_lengths(p, Lq, Lk)) return e;
  *bytes = index_ws(p, Lq, Lk).total;
  return HSA_OK;
}

int hsa_block_sums(const hsa_params* p, int64_t Lk, const hsa_bf16* k_idx, float* ksum,
                   cudaStream_t stream) {
  if (int e = check_index_params(p)) return e;
  if (Lk < 0) return HSA_ERR_ARG;
  if (Lk / p->B == 0) return HSA_OK;
  if (!aligned16(k_idx) || !aligned16(ksum)) return HSA_ERR_ARG;
  if (int e = check_device()) return e;
  hsa::launch_block_sums(k_idx, Lk, p->B, p->d_idx, ksum, stream);
  return launch_status();
}

int hsa_select_blocks(const hsa_params* p, int64_t Lq, int64_t Lk, const hsa_bf16* q_idx,
                      const float* ksum, int32_t* blocks, void* workspace,
                      size_t workspace_bytes, cudaStream_t stream) {
  if (int e = check_index_params(p)) return e;
  if (int e = check_lengths(p, Lq, Lk)) return e;
  if (Lq == 0) return HSA_OK;
  if (!aligned16(q_idx) || !aligned16(blocks) || (Lk / p->B > 0 && !aligned16(ksum)))
    return HSA_ERR_ARG;
  const IndexWs w = index_ws(p, Lq, Lk);
  if (!aligned16(workspace) || workspace_bytes < w.total) return HSA_ERR_WORKSPACE;
  if (int e = check_device()) return e;
  bool ok = true;
  run_select_blocks(p, Lq, Lk, q_idx, ksum, blocks, static_cast<char*>(workspace), w, stream, &ok);
  return ok ? launch_status() : HSA_ERR_CUDA;
}

int hsa_select_tokens(const hsa_params* p, int64_t Lq, int64_t Lk, const hsa_bf16* q_idx,
                      const hsa_bf16* k_idx, const int32_t* blocks, int32_t* indices,
                      void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (int e = check_index_params(p)) return e;
  if (int e = check_lengths(p, Lq, Lk)) return e;
  if (Lq == 0) return HSA_OK;
  if (!aligned16(q_idx) || !aligned16(k_idx) || !aligned16(blocks) || !aligned16(indices))
    return HSA_ERR_ARG;
  const IndexWs w = index_ws(p, Lq, Lk);
  if (!aligned16(workspace) || workspace_bytes < w.total) return HSA_ERR_WORKSPACE;
  if (int e = check_device()) return e;
  bool ok = true;
  run_select_tokens(p, Lq, Lk, q_idx, k_idx, blocks, indices, static_cast<char*>(workspace), w, stream, &ok);
  return ok ? launch_status() : HSA_ERR_CUDA;
}

int hsa_index(const hsa_params* p, int64_t Lq, int64_t Lk, const hsa_bf16* q_idx,
              const hsa_bf16* k_idx, int32_t* indices, void* workspace, size_t workspace_bytes,
              cudaStream_t stream) {
  if (int e = check_index_params(p)) return e;
  if (int e = check_lengths(p, Lq, Lk)) return e;
  if (Lq == 0) return HSA_OK;
  if (!aligned16(q_idx) || !aligned16(k_idx) || !aligned16(indices)) return HSA_ERR_ARG;
  const IndexWs w = index_ws(p, Lq, Lk);
  if (!aligned16(workspace) || workspace_bytes < w.total) return HSA_ERR_WORKSPACE;
  if (int e = check_device()) return e;
  char* ws = static_cast<char*>(workspace);
  float* ksum = reinterpret_cast<float*>(ws + w.ksum);
  int32_t* blocks = reinterpret_cast<int32_t*>(ws + w.blocks);
  bool ok = true;
  hsa::launch_block_sums(k_idx, Lk, p->B, p->d_idx, ksum, stream);
  run_select_blocks(p, Lq, Lk, q_idx, ksum, blocks, ws, w, stream, &ok);
  if (ok) run_select_tokens(p, Lq, Lk, q_idx, k_idx, blocks, indices, ws, w, stream, &ok);
  return ok ? launch_status() : HSA_ERR_CUDA;
}

int hsa_sparse_attn(const hsa_params* p, int64_t Lq, int64_t Lk, const hsa_bf16* Q,
                    const hsa_bf16* K, const hsa_bf16* V, const int32_t* indices, hsa_bf16* O,
                    cudaStream_t stream) {
  if (int e = check_attn_params(p)) return e;
  if (Lq < 0 || Lk < 1 || Lq > (int64_t(1) << 31) - 1 || Lk > (int64_t(1) << 31) - 1)
    return HSA_ERR_ARG;
  if (Lq == 0) return HSA_OK;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(indices) || !aligned16(O))
    return HSA_ERR_ARG;
  if (int e = check_device()) return e;
  if (!hsa::tc_attn_supported(p->H, p->d, Lq, Lk)) return HSA_ERR_ARG;
  if (!hsa::launch_sparse_attn_tc(Lq, Q, K, V, indices, Lk, p->k, p->H, p->d, softmax_scale(p), O, stream))
    return HSA_ERR_CUDA;
  return launch_status();
}

}  // extern "C"

namespace {

// Workspace of a decode step (256-byte aligned regions):
//   blocks [batch][m] i32, indices [batch][k] i32 (unless the caller takes them),
//   block-score keys [batch][capacity/B] u32, token-score keys [batch][m*B] u32,
//   attention parts: O [batch*parts][H][d] f32, maxima and row sums [batch*parts][H] f32.
struct DecodeWs {
  size_t blocks, idx, bkeys, tkeys, opart, mpart, lpart, total;
  int parts;
};
DecodeWs decode_ws(const hsa_params* p, int32_t batch, int64_t capacity) {
  DecodeWs w{};
  const int tiles = (p->k + 127) / 128;
  // enough parts per query to give every SM work at small batch, at most 16
  // (the combine kernel holds every part's values in registers)
  w.parts = batch > 0 ? std::max(1, std::min(std::min(tiles, 16), 128 / std::max(1, int(batch)))) : 1;
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o += align_up(bytes > 0 ? bytes : 1); return at; };
  w.blocks = take(size_t(batch) * p->m * 4);
  w.idx = take(size_t(batch) * p->k * 4);
  w.bkeys = take(size_t(batch) * (capacity / p->B) * 4);
  w.tkeys = take(size_t(batch) * p->m * p->B * 4);
  w.opart = take(size_t(batch) * w.parts * p->H * p->d * 4);
  w.mpart = take(size_t(batch) * w.parts * p->H * 4);
  w.lpart = take(size_t(batch) * w.parts * p->H * 4);
  w.total = o;
  return w;
}

}  // namespace

extern "C" {

int hsa_decode_workspace_size(const hsa_params* p, int32_t batch, int64_t capacity,
                              size_t* bytes) {
  if (!bytes) return HSA_ERR_ARG;
  if (int e = check_index_params(p)) return e;
  if (int e = check_attn_params(p)) return e;
  if (batch < 0 || capacity < p->B || capacity % p->B) return HSA_ERR_ARG;
  *bytes = decode_ws(p, batch, capacity).total;
  return HSA_OK;
}

int hsa_decode_step(const hsa_params* p, int32_t batch, int64_t capacity, int32_t* ctx_len,
                    hsa_bf16* k_idx_cache, hsa_bf16* K_cache, hsa_bf16* V_cache,
                    float* ksum_cache, const hsa_bf16* q_idx_new, const hsa_bf16* k_idx_new,
                    const hsa_bf16* Q_new, const hsa_bf16* K_new, const hsa_bf16* V_new,
                    hsa_bf16* O, int32_t* indices_out, void* workspace, size_t workspace_bytes,
                    cudaStream_t stream) {
  size_t need = 0;
  if (int e = hsa_decode_workspace_size(p, batch, capacity, &need)) return e;
  if (capacity / p->B > kMaxBlocks || capacity > (int64_t(1) << 31) - 1) return HSA_ERR_ARG;
  if (batch == 0) return HSA_OK;
  const void* ptrs[] = {k_idx_cache, K_cache, V_cache, ksum_cache, q_idx_new,
                        k_idx_new, Q_new, K_new, V_new, O};
  for (const void* q : ptrs)
    if (!aligned16(q)) return HSA_ERR_ARG;
  if (!ctx_len || (reinterpret_cast<uintptr_t>(ctx_len) & 3u)) return HSA_ERR_ARG;
  if (indices_out && !aligned16(indices_out)) return HSA_ERR_ARG;
  if (!aligned16(workspace) || workspace_bytes < need) return HSA_ERR_WORKSPACE;
  if (int e = check_device()) return e;
  const DecodeWs w = decode_ws(p, batch, capacity);
  char* ws = static_cast<char*>(workspace);
  int32_t* blocks = reinterpret_cast<int32_t*>(ws + w.blocks);
  int32_t* idx = indices_out ? indices_out : reinterpret_cast<int32_t*>(ws + w.idx);
  uint32_t* bkeys = reinterpret_cast<uint32_t*>(ws + w.bkeys);
  uint32_t* tkeys = reinterpret_cast<uint32_t*>(ws + w.tkeys);
  const int64_t nbc = capacity / p->B;
  hsa::RowMap rm{batch, capacity, ctx_len, capacity};
  // The step's kernels are programmatic dependent launches: each may begin
  // launching while its predecessor runs, and waits for it before touching
  // memory (griddepcontrol), which hides the launch gaps of a short step.
  // 1. append the new token (and the block sum of a block it completes), in
  //    the same kernel as 2. the block scores against the block-sum cache;
  //    top-m with the forced blocks
  hsa::launch_decode_block_scores(batch, capacity, ctx_len, p->B, p->m, p->d_idx, q_idx_new, ksum_cache,
                                  bkeys, nbc, p->d, k_idx_cache, K_cache, V_cache, ksum_cache, k_idx_new,
                                  K_new, V_new, stream);
  hsa::launch_topm_from_keys(rm, batch, bkeys, nbc, p->B, p->m, nbc > 2 ? nbc - 2 : 1, blocks, stream, true);
  // 3. token scores inside the kept blocks, top-k
  hsa::launch_decode_token_scores(batch, capacity, ctx_len, p->B, p->m, p->d_idx, blocks, q_idx_new,
                                  k_idx_cache, tkeys, stream);
  hsa::launch_topk_from_keys(rm, batch, blocks, tkeys, p->B, p->m, p->k, idx, stream, true);
  // 4. attention over the kept tokens: parts of each query on the tensor cores,
  //    then combined; 5. the combine also grows each sequence by one token
  if (!hsa::tc_attn_supported(p->H, p->d, batch, capacity)) return HSA_ERR_ARG;
  float* opart = reinterpret_cast<float*>(ws + w.opart);
  float* mpart = reinterpret_cast<float*>(ws + w.mpart);
  float* lpart = reinterpret_cast<float*>(ws + w.lpart);
  if (!hsa::launch_sparse_attn_tc_split(batch, Q_new, K_cache, V_cache, idx, capacity, p->k, p->H, p->d,
                                        softmax_scale(p), w.parts, opart, mpart, lpart, stream, true))
    return HSA_ERR_CUDA;
  hsa::launch_decode_combine(batch, capacity, ctx_len, p->H, p->d, w.parts, opart, mpart, lpart, O, stream);
  return launch_status();
}

}  // extern "C"

// ------------------------------------------------------------------ queries and keys from projections

extern "C" int hsa_qk_norm_rope(int64_t L, int32_t H, int32_t d, const hsa_bf16* Q, int64_t q_stride,
                                const hsa_bf16* K, int64_t k_stride, const hsa_bf16* q_weight,
                                const hsa_bf16* k_weight, float eps, const float* inv_freq, int32_t rot,
                                int32_t interleaved, const int32_t* positions, int64_t pos0, hsa_bf16* Q_out,
                                hsa_bf16* K_out, cudaStream_t stream) {
  constexpr int64_t kMax = (int64_t(1) << 31) - 1;
  if (L < 0 || L > kMax || H < 1 || H > 128 || (d != 64 && d != 128)) return HSA_ERR_ARG;
  if (rot < 0 || rot > d || rot % 16 || !(eps >= 0.f) || std::isinf(eps)) return HSA_ERR_ARG;
  if (interleaved != 0 && interleaved != 1) return HSA_ERR_ARG;
  if (!positions && (pos0 < 0 || pos0 > kMax - L)) return HSA_ERR_ARG;
  if (L == 0) return HSA_OK;
  if (!Q && !K) return HSA_ERR_ARG;
  auto rows_ok = [&](const hsa_bf16* in, const hsa_bf16* w, const hsa_bf16* out, int64_t stride, int64_t n) {
    return aligned16(in) && aligned16(out) && (!w || aligned16(w)) && stride >= n && stride % 8 == 0 &&
           stride <= (int64_t(1) << 62) / L && (in != out || stride == n || L == 1);  // in place: dense rows only
  };
  if (Q && !rows_ok(Q, q_weight, Q_out, q_stride, int64_t(H) * d)) return HSA_ERR_ARG;
  if (K && !rows_ok(K, k_weight, K_out, k_stride, d)) return HSA_ERR_ARG;
  const auto word = [](const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; };
  if ((rot > 0 && !word(inv_freq)) || (positions && !word(positions))) return HSA_ERR_ARG;
  if (int e = check_device()) return e;
  hsa::launch_qk_norm_rope(L, H, d, Q, q_stride, K, k_stride, q_weight, k_weight, eps, inv_freq, rot,
                           interleaved != 0, positions, pos0, Q_out, K_out, stream);
  return launch_status();
}

// ------------------------------------------------------------------ drafted trees

namespace {

// Workspace of a tree step (256-byte aligned regions), rows = batch * T:
//   counters [3] i32, rowpos [rows] i32, block-score keys [rows][ldb] u32, tail
//   keys [rows][tail_ld] u32, kept blocks [rows][m] i32, pairs [rows][m] u32,
//   items [max_items] int4, token-score keys [rows][m*B] u32, indices [rows][k]
//   i32 (unless the caller takes them), the attention's items, their CTAs' first
//   ones, the rows that are cut, the rows' flags, and the parts: O f32, maxima and row sums f32.
struct TreeWs {
  size_t counters, rowpos, bkeys, tail, blocks, pairs, items, tkeys, idx, aitems, cta, cut, flags, flagged, opart, mpart, lpart,
      total;
  int64_t rows, ldb, max_items;
  int tail_ld;
};
TreeWs tree_ws(const hsa_params* p, int32_t batch, int32_t T, int64_t capacity) {
  TreeWs w{};
  w.rows = int64_t(batch) * T;
  const int64_t blocks = capacity / p->B;
  w.ldb = (hsa::kBkeys0 + blocks + 3) / 4 * 4;
  w.tail_ld = (p->B - 1 + T + 3) / 4 * 4;
  w.max_items = batch * std::min<int64_t>(int64_t(T) * p->m, blocks) * ((p->B + 127) / 128);
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o += align_up(bytes > 0 ? bytes : 1); return at; };
  const size_t rows = size_t(w.rows);
  w.counters = take(12);
  w.rowpos = take(rows * 4);
  w.bkeys = take(rows * w.ldb * 4);
  w.tail = take(rows * w.tail_ld * 4);
  w.blocks = take(rows * p->m * 4);
  w.pairs = take(rows * p->m * 4);
  w.items = take(size_t(w.max_items) * 16);
  w.tkeys = take(rows * p->m * p->B * 4);
  w.idx = take(rows * p->k * 4);
  // a CTA's list has at most two rows that it shares with its neighbours
  const size_t parts = 2 * hsa::kTreeAttnCtas;
  w.aitems = take((rows + hsa::kTreeAttnCtas) * 16);
  w.cta = take((hsa::kTreeAttnCtas + 1) * 4);
  w.cut = take(hsa::kTreeAttnCtas * 16);
  w.flags = take(rows * 4);
  w.flagged = take(rows * 4);
  w.opart = take(parts * p->H * p->d * 4);
  w.mpart = take(parts * p->H * 4);
  w.lpart = take(parts * p->H * 4);
  w.total = o;
  return w;
}

int check_tree_sizes(const hsa_params* p, int32_t batch, int32_t T, int64_t capacity) {
  constexpr int64_t kMax = (int64_t(1) << 31) - 1;
  if (batch < 0 || T < 1 || T > HSA_TREE_MAX) return HSA_ERR_ARG;
  if (capacity < p->B || capacity % p->B || capacity / p->B > kMaxBlocks) return HSA_ERR_ARG;
  // cache rows and (node, slot) pairs are counted in 32 bits, sequences in 28
  if (batch > 0 && (capacity > kMax / batch || int64_t(batch) * T > kMax / p->m || batch >= (1 << 28)))
    return HSA_ERR_ARG;
  if (int64_t(batch) * T > kMax / std::max(p->H, 64)) return HSA_ERR_ARG;  // (also: at most 64 tiles per node)
  return HSA_OK;
}

bool aligned4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

extern "C" {

int hsa_tree_plan(int32_t batch, int32_t T, int64_t capacity, const int32_t* ctx_len, const int32_t* n_nodes,
                  const int32_t* parents, int32_t* positions, int32_t* paths, cudaStream_t stream) {
  if (batch < 0 || T < 1 || T > HSA_TREE_MAX || capacity < 1 || capacity > (int64_t(1) << 31) - 1) return HSA_ERR_ARG;
  if (batch == 0) return HSA_OK;
  if (!aligned4(ctx_len) || !aligned4(parents) || !aligned4(positions) || !aligned4(paths)) return HSA_ERR_ARG;
  if (n_nodes && !aligned4(n_nodes)) return HSA_ERR_ARG;
  if (int e = check_device()) return e;
  hsa::launch_tree_plan(batch, T, capacity, ctx_len, n_nodes, parents, positions, paths, stream);
  return launch_status();
}

int hsa_tree_workspace_size(const hsa_params* p, int32_t batch, int32_t T, int64_t capacity, size_t* bytes) {
  if (!bytes) return HSA_ERR_ARG;
  if (int e = check_index_params(p)) return e;
  if (int e = check_attn_params(p)) return e;
  if (int e = check_tree_sizes(p, batch, T, capacity)) return e;
  *bytes = tree_ws(p, batch, T, capacity).total;
  return HSA_OK;
}

int hsa_tree_step(const hsa_params* p, int32_t batch, int32_t T, int64_t capacity, const int32_t* ctx_len,
                  const int32_t* positions, const int32_t* paths, hsa_bf16* k_idx_cache, hsa_bf16* K_cache,
                  hsa_bf16* V_cache, const float* ksum_cache, const hsa_bf16* q_idx_new, const hsa_bf16* k_idx_new,
                  const hsa_bf16* Q_new, const hsa_bf16* K_new, const hsa_bf16* V_new, hsa_bf16* O,
                  int32_t* indices_out, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  size_t need = 0;
  if (int e = hsa_tree_workspace_size(p, batch, T, capacity, &need)) return e;
  if (batch == 0) return HSA_OK;
  const void* ptrs[] = {k_idx_cache, K_cache, V_cache, ksum_cache, q_idx_new, k_idx_new, Q_new, K_new, V_new, O};
  for (const void* q : ptrs)
    if (!aligned16(q)) return HSA_ERR_ARG;
  if (!aligned4(ctx_len) || !aligned4(positions) || !aligned4(paths)) return HSA_ERR_ARG;
  if (indices_out && !aligned16(indices_out)) return HSA_ERR_ARG;
  if (!aligned16(workspace) || workspace_bytes < need) return HSA_ERR_WORKSPACE;
  if (int e = check_device()) return e;
  const TreeWs w = tree_ws(p, batch, T, capacity);
  char* ws = static_cast<char*>(workspace);
  int32_t* blocks = reinterpret_cast<int32_t*>(ws + w.blocks);
  int32_t* idx = indices_out ? indices_out : reinterpret_cast<int32_t*>(ws + w.idx);
  hsa::TreeArgs a{};
  a.T = T; a.B = p->B; a.m = p->m; a.k = p->k; a.d = p->d;
  a.capacity = capacity; a.ldb = w.ldb;
  a.ctx = ctx_len; a.positions = positions; a.paths = paths;
  a.k_idx_cache = k_idx_cache; a.K_cache = K_cache; a.V_cache = V_cache; a.ksum_cache = ksum_cache;
  a.q_new = q_idx_new; a.k_idx_new = k_idx_new; a.K_new = K_new; a.V_new = V_new;
  a.rowpos = reinterpret_cast<int32_t*>(ws + w.rowpos);
  a.bkeys = reinterpret_cast<uint32_t*>(ws + w.bkeys);
  a.tailkeys = reinterpret_cast<uint32_t*>(ws + w.tail);
  a.tkeys = reinterpret_cast<uint32_t*>(ws + w.tkeys);
  a.tail_ld = w.tail_ld;
  a.blocks = blocks;
  a.pairs = reinterpret_cast<uint32_t*>(ws + w.pairs);
  a.items = reinterpret_cast<int4*>(ws + w.items);
  a.counters = reinterpret_cast<int*>(ws + w.counters);
  a.attn_items = reinterpret_cast<int4*>(ws + w.aitems);
  a.cta_items = reinterpret_cast<int*>(ws + w.cta);
  a.cut = reinterpret_cast<int4*>(ws + w.cut);
  a.O = O; a.H = p->H;
  a.flags = reinterpret_cast<int*>(ws + w.flags);
  a.flagged = reinterpret_cast<int*>(ws + w.flagged);
  // The kernels are programmatic dependent launches, as in a decode step.
  // 1. drafted rows appended, tails and cached blocks scored; top-m
  if (!hsa::launch_tree_block_scores(a, batch, p->d_idx, stream)) return HSA_ERR_CUDA;
  hsa::launch_tree_topm(a, w.rows, blocks, stream);
  // 2. token scores of the kept blocks, each cached block read once for all its nodes; top-k
  if (hsa::tree_few_scores(a, w.rows, p->d_idx)) {
    hsa::launch_tree_few_scores(a, w.rows, p->d_idx, stream);
  } else {
    hsa::launch_tree_lists(a, batch, stream);
    if (!hsa::launch_tree_token_scores(a, batch, p->d_idx, w.max_items, stream)) return HSA_ERR_CUDA;
  }
  if (hsa::tree_topk_wide(a, w.rows)) {
    hsa::launch_tree_topk(a, w.rows, idx, stream);
  } else {
    // a node's row of the selection is at the node's own position; a row that takes no part has position -1
    const hsa::RowMap rm{w.rows, capacity, a.rowpos, capacity};
    hsa::launch_topk_from_keys(rm, w.rows, blocks, a.tkeys, p->B, p->m, p->k, idx, stream, true);
    hsa::launch_tree_rows(a, w.rows, idx, stream);
  }
  // 3. attention over the kept rows, in equal shares of 128-key tiles per CTA
  float* opart = reinterpret_cast<float*>(ws + w.opart);
  float* mpart = reinterpret_cast<float*>(ws + w.mpart);
  float* lpart = reinterpret_cast<float*>(ws + w.lpart);
  if (!hsa::launch_tree_attn(a, Q_new, idx, softmax_scale(p), opart, mpart, lpart, stream)) return HSA_ERR_CUDA;
  hsa::launch_tree_combine(a, w.rows, Q_new, idx, softmax_scale(p), opart, mpart, lpart, stream);
  return launch_status();
}

int hsa_tree_commit(const hsa_params* p, int32_t batch, int32_t T, int64_t capacity, int32_t* ctx_len,
                    const int32_t* paths, const int32_t* accepted, hsa_bf16* k_idx_cache, hsa_bf16* K_cache,
                    hsa_bf16* V_cache, float* ksum_cache, cudaStream_t stream) {
  if (int e = check_index_params(p)) return e;
  if (int e = check_attn_params(p)) return e;
  if (int e = check_tree_sizes(p, batch, T, capacity)) return e;
  if (batch == 0) return HSA_OK;
  const void* ptrs[] = {k_idx_cache, K_cache, V_cache, ksum_cache};
  for (const void* q : ptrs)
    if (!aligned16(q)) return HSA_ERR_ARG;
  if (!aligned4(ctx_len) || !aligned4(paths) || !aligned4(accepted)) return HSA_ERR_ARG;
  if (int e = check_device()) return e;
  hsa::launch_tree_commit(batch, T, capacity, p->B, p->d_idx, p->d, ctx_len, paths, accepted, k_idx_cache, K_cache,
                          V_cache, ksum_cache, stream);
  return launch_status();
}

}  // extern "C"
