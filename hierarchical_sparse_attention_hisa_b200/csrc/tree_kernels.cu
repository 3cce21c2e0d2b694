// Verification of a tree of drafted tokens over the decode caches: node i of
// a sequence's tree is the query that a decode step would make had the tokens
// of its path (its ancestors, then itself) been appended one by one.
//
// The drafted rows live behind the cached ones, node j in cache row ctx + j,
// so along a node's path position p is row p below ctx and row
// ctx + path[p - ctx] from there on. Blocks wholly below f = floor(ctx / B)
// are the same for every node and go through the block-sum cache and the
// tensor cores (tree_scores.cu); the "tail", positions from f*B on, differs
// from node to node, is at most B - 1 + T rows long and is scored here. A
// tail block's score is the sum of its token scores: q . sum k = sum q . k.
#include <algorithm>

#include "kernels.cuh"

namespace hsa {
namespace {

// ---------------------------------------------------------------------------
// Positions and paths of the drafted nodes, one CTA per tree. A thread per
// node walks up its parents in shared memory (at most T steps; a parent must
// come before its child, so every walk ends), and the CTA writes the rows out
// coalesced.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) tree_plan_kernel(int T, int64_t capacity, const int32_t* __restrict__ ctx,
                                                        const int32_t* __restrict__ n_nodes,
                                                        const int32_t* __restrict__ parents,
                                                        int32_t* __restrict__ positions, int32_t* __restrict__ paths) {
  __shared__ int par[kTreeMax], dep[kTreeMax];
  __shared__ int8_t up[kTreeMax][kTreeMax + 4];  // up[i][s]: the node s steps above i
  griddep_wait();
  griddep_launch();
  const int64_t b = blockIdx.x;
  const int i = threadIdx.x;
  if (i < T) par[i] = parents[b * T + i];
  const int64_t c = ctx[b];
  const int n = n_nodes ? min(max(n_nodes[b], 0), T) : T;
  const bool fits = c >= 0 && c + n <= capacity;
  __syncthreads();
  if (i < T) {
    int d = -1;
    if (fits && i < n) {
      int j = i;
      for (int s = 0; s < T; ++s) {
        up[i][s] = int8_t(j);
        const int q = par[j];
        if (q == -1) { d = s; break; }
        if (q < -1 || q >= j) break;  // not a tree: the node takes no part
        j = q;
      }
    }
    dep[i] = d;
    positions[b * T + i] = d >= 0 ? int32_t(c + d) : -1;
  }
  __syncthreads();
  int32_t* out = paths + b * T * T;
  for (int e = threadIdx.x; e < T * T; e += 256) {
    const int r = e / T, s = e - r * T;
    out[e] = s <= dep[r] ? up[r][dep[r] - s] : -1;
  }
}

// ---------------------------------------------------------------------------
// Node block scores. Grid (sequence, part). The first `chunks` parts score 64
// cached whole blocks each against every node of the sequence:
// bkeys[row][blk] = key(q . ksum[blk]), fp32 products and sums. The other
// parts are one node each: append its drafted rows to the caches, score its
// tail, write the tail's keys and the scores of its whole tail blocks.
// ---------------------------------------------------------------------------
constexpr int kBlkChunk = 64;
constexpr int kNT = 256;

// Does the selection of a node at position t need token scores?
HSA_DEV bool needs_scores(int64_t t, int B, int m, int k) {
  const int64_t nb = t / B + 1;
  const int64_t n = nb <= m ? t + 1 : int64_t(m - 1) * B + t % B + 1;
  return n > k;
}

template <int DI>
HSA_DEV float dot8(const uint4& kv, const float (&q)[8]) {
  float acc = q[0] * bf16_lo(kv.x);
  acc = __fmaf_rn(q[1], bf16_hi(kv.x), acc);
  acc = __fmaf_rn(q[2], bf16_lo(kv.y), acc);
  acc = __fmaf_rn(q[3], bf16_hi(kv.y), acc);
  acc = __fmaf_rn(q[4], bf16_lo(kv.z), acc);
  acc = __fmaf_rn(q[5], bf16_hi(kv.z), acc);
  acc = __fmaf_rn(q[6], bf16_lo(kv.w), acc);
  acc = __fmaf_rn(q[7], bf16_hi(kv.w), acc);
  return acc;
}

template <int DI>
__device__ void node_tail(const TreeArgs& a, int64_t b, int i, float* sc) {
  const int64_t row = b * a.T + i;
  const int64_t c = a.ctx[b];
  const int64_t t = a.positions[row];
  // a plan made for other lengths must not reach outside the sequence's rows
  const bool ok = c >= 0 && t >= c && t - c <= i && c + i < a.capacity;
  if (threadIdx.x == 0) a.rowpos[row] = ok ? int32_t(t) : -1;
  if (!ok) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  {  // the drafted rows, node i in cache row c + i
    const int64_t at = b * a.capacity + c + i;
    const int ci = DI / 8, cd = a.d / 8;
    for (int e = tid; e < ci + 2 * cd; e += kNT) {
      if (e < ci)
        reinterpret_cast<uint4*>(a.k_idx_cache + at * DI)[e] = reinterpret_cast<const uint4*>(a.k_idx_new + row * DI)[e];
      else if (e < ci + cd)
        reinterpret_cast<uint4*>(a.K_cache + at * a.d)[e - ci] = reinterpret_cast<const uint4*>(a.K_new + row * a.d)[e - ci];
      else
        reinterpret_cast<uint4*>(a.V_cache + at * a.d)[e - ci - cd] =
            reinterpret_cast<const uint4*>(a.V_new + row * a.d)[e - ci - cd];
    }
  }
  const int64_t nb = t / a.B + 1;
  const int64_t f = c / a.B;
  const bool tokens = needs_scores(t, a.B, a.m, a.k);
  const bool blocks = nb > a.m && f < nb - 1;  // whole blocks in the tail
  if (!tokens && !blocks) return;
  // tail rows: cached ones from f*B, then the path
  const int head = int(c - f * a.B), n = head + int(t - c) + 1;
  constexpr int LPR = DI / 8, RPW = 32 / LPR;
  const int sub = lane % LPR, rsub = lane / LPR;
  float q[8];
  {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(a.q_new + row * DI) + sub);
    q[0] = bf16_lo(v.x); q[1] = bf16_hi(v.x); q[2] = bf16_lo(v.y); q[3] = bf16_hi(v.y);
    q[4] = bf16_lo(v.z); q[5] = bf16_hi(v.z); q[6] = bf16_lo(v.w); q[7] = bf16_hi(v.w);
  }
  const uint16_t* cached = a.k_idx_cache + (b * a.capacity + f * a.B) * DI;
  const int32_t* path = a.paths + row * a.T;
  uint32_t* keys = a.tailkeys + row * a.tail_ld;
  constexpr int U = 4;  // rows in flight per lane group
  for (int r0 = warp * RPW; r0 < n; r0 += (kNT / 32) * RPW * U) {
    uint4 kv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * (kNT / 32) * RPW + rsub;
      kv[u] = make_uint4(0, 0, 0, 0);
      if (r < head) {
        kv[u] = *(reinterpret_cast<const uint4*>(cached + int64_t(r) * DI) + sub);
      } else if (r < n) {
        const int j = min(max(path[r - head], 0), a.T - 1);
        kv[u] = __ldg(reinterpret_cast<const uint4*>(a.k_idx_new + (b * a.T + j) * DI) + sub);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * (kNT / 32) * RPW + rsub;
      float acc = dot8<DI>(kv[u], q);
#pragma unroll
      for (int o = LPR / 2; o >= 1; o >>= 1) acc += __shfl_xor_sync(kFull, acc, o);
      if (sub == 0 && r < n) {
        sc[r] = acc;
        keys[r] = score_key(acc);
      }
    }
  }
  if (!blocks) return;
  __syncthreads();
  for (int64_t blk = f + warp; blk < nb - 1; blk += kNT / 32) {
    float s = 0.f;
    for (int r = lane; r < a.B; r += 32) s += sc[(blk - f) * a.B + r];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    if (lane == 0) a.bkeys[row * a.ldb + blk] = score_key(s);
  }
}

// 64 blocks x TP nodes, DI summed in shared memory: a thread holds TP/16 nodes
// x 4 blocks. The operands are read as float4 along the summed axis.
template <int DI, int TP>
__device__ void cached_block_scores(const TreeArgs& a, int64_t b, int chunk, float* smem) {
  const int64_t c = a.ctx[b];
  if (c < 0 || c >= a.capacity) return;
  const int64_t f = c / a.B;
  const int64_t lo = int64_t(chunk) * kBlkChunk, hi = min(f, lo + kBlkChunk);
  if (lo >= hi) return;
  if ((c + a.T - 1) / a.B + 1 <= a.m) return;  // every node keeps all its blocks
  constexpr int LD = DI + 4;
  float* qs = smem;             // [TP][LD]
  float* ks = smem + TP * LD;   // [64][LD]
  const int tid = threadIdx.x;
  for (int e = tid; e < TP * (DI / 8); e += kNT) {
    const int n = e / (DI / 8), ch = e % (DI / 8);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (n < a.T) v = __ldg(reinterpret_cast<const uint4*>(a.q_new + (b * a.T + n) * DI) + ch);
    float4* o = reinterpret_cast<float4*>(qs + n * LD + 8 * ch);
    o[0] = make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
    o[1] = make_float4(bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w));
  }
  const float* src = a.ksum_cache + (b * (a.capacity / a.B) + lo) * DI;
  for (int e = tid; e < kBlkChunk * (DI / 4); e += kNT) {
    const int n = e / (DI / 4), ch = e % (DI / 4);
    const float4 v = lo + n < hi ? __ldg(reinterpret_cast<const float4*>(src + n * DI) + ch) : make_float4(0, 0, 0, 0);
    *reinterpret_cast<float4*>(ks + n * LD + 4 * ch) = v;
  }
  __syncthreads();
  constexpr int NN = TP / 16;
  const int bg = tid & 15, ng = tid >> 4;  // blocks bg + 16 j, nodes ng + 16 i
  float acc[NN][4] = {};
#pragma unroll 4
  for (int e = 0; e < DI; e += 4) {
    float4 kv[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(ks + (bg + 16 * j) * LD + e);
#pragma unroll
    for (int i = 0; i < NN; ++i) {
      const float4 qv = *reinterpret_cast<const float4*>(qs + (ng + 16 * i) * LD + e);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][j] = __fmaf_rn(qv.x, kv[j].x, acc[i][j]);
        acc[i][j] = __fmaf_rn(qv.y, kv[j].y, acc[i][j]);
        acc[i][j] = __fmaf_rn(qv.z, kv[j].z, acc[i][j]);
        acc[i][j] = __fmaf_rn(qv.w, kv[j].w, acc[i][j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NN; ++i) {
    const int n = ng + 16 * i;
    if (n >= a.T) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (lo + bg + 16 * j < hi) a.bkeys[(b * a.T + n) * a.ldb + lo + bg + 16 * j] = score_key(acc[i][j]);
  }
}

template <int DI, int TP>
__global__ void __launch_bounds__(kNT) tree_block_scores_kernel(const TreeArgs a, int chunks) {
  extern __shared__ __align__(16) float smem_f[];
  griddep_wait();
  griddep_launch();
  const int64_t b = blockIdx.x;
  if (b == 0 && blockIdx.y == 0 && threadIdx.x < 2) a.counters[threadIdx.x] = 0;
  if (int(blockIdx.y) < chunks)
    cached_block_scores<DI, TP>(a, b, blockIdx.y, smem_f);
  else
    node_tail<DI>(a, b, int(blockIdx.y) - chunks, smem_f);
}

// ---------------------------------------------------------------------------
// Work lists, one launch.
//
// Token scores: CTA (sequence, range of 512 cached blocks), a thread per block:
// the (node, slot) pairs of each kept block and an item per 128 rows of such a
// block. The order of items and of pairs inside one is not fixed (atomics);
// each writes its own keys, so results do not depend on it. Kept tail blocks
// take their keys from the tail's scores here.
//
// Attention: one more CTA cuts all rows' 128-key tiles, in row order, into
// kGivenItemCtas equal shares (what a row keeps follows from its position
// alone). A static row per CTA leaves most SMs idle when trees are ragged; with
// equal shares at most two rows of a CTA are cut, whose parts are combined.
// ---------------------------------------------------------------------------
constexpr int kListNT = 512;

HSA_DEV void attn_shares(const TreeArgs& a, int64_t rows, int* s_tmp) {
  const int tid = threadIdx.x;
  auto tiles_of = [&](int64_t row) -> int {
    if (row >= rows) return 0;
    const int64_t t = a.rowpos[row];
    if (t < 0) return 0;
    const int64_t nb = t / a.B + 1;
    const int64_t n = nb <= a.m ? t + 1 : int64_t(a.m - 1) * a.B + t % a.B + 1;
    return int((min(n, int64_t(a.k)) + 127) / 128);
  };
  int64_t total = 0;
  for (int64_t r0 = 0; r0 < rows; r0 += kListNT) {
    int sum;
    block_exclusive_scan<kListNT>(tiles_of(r0 + tid), s_tmp, &sum);
    total += sum;
  }
  const int64_t quota = max(int64_t(1), (total + kGivenItemCtas - 1) / kGivenItemCtas);
  int64_t tile0 = 0;
  int item0 = 0, part0 = 0;
  for (int64_t r0 = 0; r0 < rows; r0 += kListNT) {
    const int64_t row = r0 + tid;
    const int n = tiles_of(row);
    int sum, items, parts;
    const int64_t s = tile0 + block_exclusive_scan<kListNT>(n, s_tmp, &sum);
    const int64_t c0 = s / quota;
    const int pieces = n ? int((s + n - 1) / quota - c0) + 1 : 0;
    int at = item0 + block_exclusive_scan<kListNT>(pieces, s_tmp, &items);
    const int part = part0 + block_exclusive_scan<kListNT>(pieces > 1 ? pieces : 0, s_tmp, &parts);
    if (row < rows) a.row_parts[row] = make_int2(part, pieces);
    for (int j = 0; j < pieces; ++j, ++at) {
      const int64_t lo = max(s, (c0 + j) * quota), hi = min(s + n, (c0 + j + 1) * quota);
      a.attn_items[at] = make_int4(int(row), int(lo - s), int(hi - lo), pieces > 1 ? part + j : -1);
      if (lo == (c0 + j) * quota) a.cta_items[c0 + j] = at;  // the first item of CTA c0 + j
    }
    tile0 += sum;
    item0 += items;
    part0 += parts;
  }
  for (int64_t c = (total + quota - 1) / quota + tid; c <= kGivenItemCtas; c += kListNT) a.cta_items[c] = item0;
}

__global__ void __launch_bounds__(kListNT) tree_lists_kernel(const TreeArgs a, int64_t rows, int ranges) {
  __shared__ int hist[kListNT];  // pair counts of this range's blocks, then cursors
  __shared__ int s_tmp[kListNT / 32 + 1];
  __shared__ int s_base[2];
  __shared__ int pos_s[kTreeMax];
  griddep_wait();
  griddep_launch();
  if (blockIdx.x == gridDim.x - 1) {
    attn_shares(a, rows, s_tmp);
    return;
  }
  const int64_t b = blockIdx.x / ranges;
  const int range = int(blockIdx.x % ranges);
  const int64_t c = a.ctx[b];
  if (c < 0 || c >= a.capacity) return;
  const int f = int(c / a.B);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lo = range * kListNT, mine = lo + tid;  // this thread's block
  if (tid < a.T) {
    const int t = a.rowpos[b * a.T + tid];
    pos_s[tid] = t >= 0 && needs_scores(t, a.B, a.m, a.k) ? t : -1;
  }
  hist[tid] = 0;
  __syncthreads();
  const int32_t* blocks = a.blocks + b * a.T * a.m;
  const int entries = a.T * a.m;
  const int end = min(f, lo + kListNT);
  for (int e = tid; e < entries; e += kListNT) {
    const int blk = blocks[e];
    if (blk >= lo && blk < end && pos_s[e / a.m] >= 0) atomicAdd(&hist[blk - lo], 1);
  }
  // tail blocks: their keys, a warp per node, the nodes spread over the ranges
  for (int i = range + warp * ranges; i < a.T; i += kListNT / 32 * ranges) {
    const int t = pos_s[i];
    if (t < 0) continue;
    const int64_t row = b * a.T + i;
    const int n = t - f * a.B + 1;  // tail rows of the node
    const int nblk = min(a.m, t / a.B + 1);
    const uint32_t* src = a.tailkeys + row * a.tail_ld;
    for (int s = nblk - 1; s >= 0; --s) {
      const int blk = blocks[i * a.m + s];
      if (blk < f) break;
      const int r0 = (blk - f) * a.B;
      uint32_t* dst = a.tkeys + (row * a.m + s) * int64_t(a.B);
      for (int r = lane; r < a.B && r0 + r < n; r += 32) dst[r] = src[r0 + r];
    }
  }
  __syncthreads();
  // this range's items: `per` for each block with a pair
  const int per = (a.B + 127) / 128;
  const int cnt = hist[tid];
  int tot_p, tot_i;
  const int at_p = block_exclusive_scan<kListNT>(cnt, s_tmp, &tot_p);
  const int at_i = block_exclusive_scan<kListNT>(cnt > 0, s_tmp, &tot_i);
  if (tot_p == 0) return;
  if (tid == 0) s_base[0] = atomicAdd(a.counters, tot_i * per);
  if (tid == 32) s_base[1] = atomicAdd(a.counters + 1, tot_p);
  hist[tid] = at_p;
  __syncthreads();
  uint32_t* pairs = a.pairs + s_base[1];
  if (cnt)
    for (int ch = 0; ch < per; ++ch)
      a.items[s_base[0] + at_i * per + ch] =
          make_int4(int(b * a.capacity) + mine * a.B + 128 * ch, s_base[1] + at_p,
                    cnt | (min(128, a.B - 128 * ch) << 16), int(b << 3) | ch);
  for (int e = tid; e < entries; e += kListNT) {
    const int blk = blocks[e], i = e / a.m;
    if (blk >= lo && blk < end && pos_s[i] >= 0)
      pairs[atomicAdd(&hist[blk - lo], 1)] = uint32_t(i) << 16 | uint32_t(e - i * a.m);
  }
}

// Kept positions of each node -> rows of its sequence's cache, in place, a warp
// per node. Positions ascend, so the drafted ones are the last of the list: at
// most T, found from its end.
__global__ void __launch_bounds__(256) tree_rows_kernel(const TreeArgs a, int64_t rows, int32_t* __restrict__ idx) {
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int64_t t = a.rowpos[row];
  if (t < 0) return;  // no part: its entries are -1
  const int c = a.ctx[row / a.T];
  const int64_t nb = t / a.B + 1;
  const int64_t n = min(int64_t(a.k), nb <= a.m ? t + 1 : int64_t(a.m - 1) * a.B + t % a.B + 1);
  const int32_t* path = a.paths + row * a.T;
  int32_t* out = idx + row * a.k;
  for (int64_t e0 = n - 32; e0 > -32; e0 -= 32) {
    const int64_t e = e0 + lane;
    const int p = e >= 0 ? out[e] : -1;
    const bool late = p >= c;
    if (late) out[e] = c + min(max(path[min(p - c, a.T - 1)], 0), a.T - 1);
    if (!__all_sync(kFull, late)) break;
  }
}

// O of the rows that were cut (with M the largest part maximum, O = sum_p
// 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p in log2 units), and of the rows that
// keep nothing (zero). Grid (row, heads / HPC), a thread per four values.
template <int D>
__global__ void __launch_bounds__(256) tree_combine_kernel(const TreeArgs a, int H, const float* __restrict__ Opart,
                                                           const float* __restrict__ mpart,
                                                           const float* __restrict__ lpart, uint16_t* __restrict__ O) {
  constexpr int TPH = D / 4, HPC = 256 / TPH;  // threads per head, heads per CTA
  griddep_wait();
  griddep_launch();
  const int64_t row = blockIdx.x;
  const int2 rp = a.row_parts[row];
  if (rp.y == 1) return;  // written whole
  const int h = blockIdx.y * HPC + threadIdx.x / TPH, v = threadIdx.x % TPH;
  if (h >= H) return;
  float M = -INFINITY;
#pragma unroll 8
  for (int p = 0; p < rp.y; ++p) {
    const int64_t w = int64_t(rp.x + p) * H + h;
    if (lpart[w] > 0.f) M = fmaxf(M, mpart[w]);
  }
  float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
  float den = 0.f;
#pragma unroll 8
  for (int p = 0; p < rp.y; ++p) {
    const int64_t w = int64_t(rp.x + p) * H + h;
    const float l = lpart[w];
    if (!(l > 0.f)) continue;
    const float4 o = reinterpret_cast<const float4*>(Opart + w * D)[v];
    const float g = exp2f(mpart[w] - M);
    num.x = __fmaf_rn(g, o.x, num.x); num.y = __fmaf_rn(g, o.y, num.y);
    num.z = __fmaf_rn(g, o.z, num.z); num.w = __fmaf_rn(g, o.w, num.w);
    den = __fmaf_rn(g, l, den);
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
  reinterpret_cast<uint2*>(O + (row * H + h) * D)[v] =
      make_uint2(cvt_bf16x2(num.x * inv, num.y * inv), cvt_bf16x2(num.z * inv, num.w * inv));
}

// ---------------------------------------------------------------------------
// The accepted path's rows moved to ctx, ctx + 1, ..., one CTA per sequence
// (node path[j] >= j, so a row may be both source and target: every row is
// read before any is written), then the sums of the blocks they complete and
// the new length.
// ---------------------------------------------------------------------------
constexpr int kCommitNT = 512;

template <int DI>
__global__ void __launch_bounds__(kCommitNT) tree_commit_kernel(int T, int64_t capacity, int B, int d,
                                                                int32_t* __restrict__ ctx,
                                                                const int32_t* __restrict__ paths,
                                                                const int32_t* __restrict__ accepted,
                                                                uint16_t* k_idx_cache, uint16_t* K_cache,
                                                                uint16_t* V_cache, float* __restrict__ ksum_cache) {
  __shared__ int path[kTreeMax];
  __shared__ int s_n;
  constexpr int CG = DI / 8, RL = kCommitNT / CG;
  __shared__ float red[RL][DI + 1];
  griddep_wait();
  griddep_launch();
  const int64_t b = blockIdx.x;
  const int tid = threadIdx.x;
  const int64_t c = ctx[b];
  const int acc = accepted[b];
  if (acc < 0 || acc >= T || c < 0) return;
  if (tid < T) path[tid] = paths[(b * T + acc) * T + tid];
  __syncthreads();
  if (tid == 0) {
    int n = 0, last = -1;
    while (n < T && path[n] > last && path[n] < T) last = path[n++];
    s_n = last == acc && c + acc < capacity ? n : 0;  // else not a path of this plan
  }
  __syncthreads();
  const int n = s_n;
  if (n == 0) return;
  {
    // at most 64 rows of (d_idx + 2d) / 8 <= 48 chunks: six per thread, all
    // read before any is written
    constexpr int PER = kTreeMax * 48 / kCommitNT;
    const int ci = DI / 8, cd = d / 8, cr = ci + 2 * cd;
    uint4 v[PER];
    auto at = [&](int ch, int64_t row) -> uint4* {
      const int64_t r = b * capacity + c + row;
      if (ch < ci) return reinterpret_cast<uint4*>(k_idx_cache + r * DI) + ch;
      if (ch < ci + cd) return reinterpret_cast<uint4*>(K_cache + r * d) + (ch - ci);
      return reinterpret_cast<uint4*>(V_cache + r * d) + (ch - ci - cd);
    };
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int e = tid + u * kCommitNT, j = e / cr, ch = e - j * cr;
      if (j < n && path[j] != j) v[u] = *at(ch, path[j]);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int e = tid + u * kCommitNT, j = e / cr, ch = e - j * cr;
      if (j < n && path[j] != j) *at(ch, j) = v[u];
    }
  }
  __syncthreads();
  const int cg = tid % CG, rl = tid / CG;
  for (int64_t blk = c / B; blk < (c + n) / B; ++blk) {
    float s[8] = {};
    const uint4* rows = reinterpret_cast<const uint4*>(k_idx_cache + (b * capacity + blk * B) * DI) + cg;
#pragma unroll 4
    for (int r = rl; r < B; r += RL) {
      const uint4 x = rows[int64_t(r) * CG];
      s[0] += bf16_lo(x.x); s[1] += bf16_hi(x.x);
      s[2] += bf16_lo(x.y); s[3] += bf16_hi(x.y);
      s[4] += bf16_lo(x.z); s[5] += bf16_hi(x.z);
      s[6] += bf16_lo(x.w); s[7] += bf16_hi(x.w);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) red[rl][8 * cg + e] = s[e];
    __syncthreads();
    if (tid < DI) {
      float t = 0.f;
      const int used = min(RL, B);
      for (int l = 0; l < used; ++l) t += red[l][tid];
      ksum_cache[(b * (capacity / B) + blk) * DI + tid] = t;
    }
    __syncthreads();
  }
  if (tid == 0) ctx[b] = int32_t(c + n);
}

}  // namespace

void launch_tree_plan(int batch, int T, int64_t capacity, const int32_t* ctx, const int32_t* n_nodes,
                      const int32_t* parents, int32_t* positions, int32_t* paths, cudaStream_t s) {
  count_launches(1);
  launch_kernel(true, tree_plan_kernel, unsigned(batch), 256, 0, s, T, capacity, ctx, n_nodes, parents, positions,
                paths);
}

bool launch_tree_block_scores(const TreeArgs& a, int batch, int d_idx, cudaStream_t s) {
  const int chunks = int((a.capacity / a.B + kBlkChunk - 1) / kBlkChunk);
  const dim3 grid(unsigned(batch), unsigned(chunks + a.T));
  const int TP = a.T <= 16 ? 16 : a.T <= 32 ? 32 : 64;
  const size_t smem = std::max(size_t(TP + kBlkChunk) * (d_idx + 4) * 4, size_t(a.tail_ld) * 4);
  auto go = [&](auto kern) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess) return false;
    count_launches(1);
    launch_kernel(true, kern, grid, kNT, smem, s, a, chunks);
    return true;
  };
  if (d_idx == 128)
    return TP == 16 ? go(tree_block_scores_kernel<128, 16>)
           : TP == 32 ? go(tree_block_scores_kernel<128, 32>) : go(tree_block_scores_kernel<128, 64>);
  return TP == 16 ? go(tree_block_scores_kernel<64, 16>)
         : TP == 32 ? go(tree_block_scores_kernel<64, 32>) : go(tree_block_scores_kernel<64, 64>);
}

void launch_tree_lists(const TreeArgs& a, int batch, cudaStream_t s) {
  const int ranges = int((a.capacity / a.B + kListNT - 1) / kListNT);
  count_launches(1);
  launch_kernel(true, tree_lists_kernel, unsigned(batch * ranges + 1), kListNT, 0, s, a, int64_t(batch) * a.T, ranges);
}

void launch_tree_rows(const TreeArgs& a, int64_t rows, int32_t* idx, cudaStream_t s) {
  count_launches(1);
  launch_kernel(true, tree_rows_kernel, unsigned((rows + 7) / 8), 256, 0, s, a, rows, idx);
}

void launch_tree_combine(const TreeArgs& a, int64_t rows, int H, const float* Opart, const float* mpart,
                         const float* lpart, void* O, cudaStream_t s) {
  const int hpc = 1024 / a.d;
  const dim3 grid(unsigned(rows), unsigned((H + hpc - 1) / hpc));
  count_launches(1);
  launch_kernel(true, a.d == 128 ? tree_combine_kernel<128> : tree_combine_kernel<64>, grid, 256, 0, s, a, H, Opart,
                mpart, lpart, (uint16_t*)O);
}

void launch_tree_commit(int batch, int T, int64_t capacity, int B, int d_idx, int d, int32_t* ctx,
                        const int32_t* paths, const int32_t* accepted, void* k_idx_cache, void* K_cache,
                        void* V_cache, float* ksum_cache, cudaStream_t s) {
  count_launches(1);
  launch_kernel(true, d_idx == 128 ? tree_commit_kernel<128> : tree_commit_kernel<64>, unsigned(batch), kCommitNT, 0,
                s, T, capacity, B, d, ctx, paths, accepted, (uint16_t*)k_idx_cache, (uint16_t*)K_cache,
                (uint16_t*)V_cache, ksum_cache);
}

}  // namespace hsa
