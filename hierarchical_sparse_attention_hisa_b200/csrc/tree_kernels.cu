// Verification of a tree of drafted tokens over the decode caches: node i of
// a sequence's tree is the query that a decode step would make had the tokens
// of its path (its ancestors, then itself) been appended one by one.
//
// The drafted rows live behind the cached ones, node j in cache row ctx + j,
// so along a node's path position p is row p below ctx and row
// ctx + path[p - ctx] from there on. Blocks wholly below f = floor(ctx / B)
// are the same for every node and go through the block-sum cache and the
// tensor cores; the "tail", positions from f*B on, differs from node to node
// and is at most B - 1 + T rows long (tree_scores.cu for both).
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
// Work lists of the token scores, CTA (sequence, range of 512 cached blocks), a
// thread per block: the (node, slot) pairs of each kept block and an item per
// 128 rows of such a block. The order of items and of pairs inside one is not
// fixed (atomics); each writes its own keys, so results do not depend on it.
//
// Beside them, a warp per node gives the kept tail blocks their keys from the
// tail's scores, and one CTA cuts the attention's work.
// ---------------------------------------------------------------------------
constexpr int kListNT = 512;

// The attention's work: all rows' 128-key tiles, in row order, cut into
// kTreeAttnCtas equal shares (what a row keeps follows from its position
// alone). A row per CTA leaves most SMs idle when trees are ragged; with equal
// shares at most two rows of a CTA are cut, whose parts are combined.
template <int NT>
__device__ void attn_shares(const TreeArgs& a, int64_t rows, int* s_tmp) {
  const int tid = threadIdx.x;
  const int64_t per = (rows + NT - 1) / NT;  // a thread has `per` rows in a row, and looks at them three times
  const int64_t r0 = min(rows, tid * per), r1 = min(rows, r0 + per);
  auto kept_of = [&](int64_t row) -> int {
    const int t = a.rowpos[row];
    return t < 0 ? 0 : min(a.k, candidates(t, a.B, a.m));
  };
  const int kept0 = r0 < r1 ? kept_of(r0) : 0;  // (mostly the only one)
  int mine = (kept0 + 127) / 128, total;          // (at most 64 tiles per row, rows below 2^25)
  for (int64_t row = r0 + 1; row < r1; ++row) mine += (kept_of(row) + 127) / 128;
  const int tile0 = block_exclusive_scan<NT>(mine, s_tmp, &total);
  const int quota = max(1, (total + kTreeAttnCtas - 1) / kTreeAttnCtas);
  // f(row, kept rows, first tile, tiles, pieces): a row's tiles lie in `pieces` CTAs
  auto for_rows = [&](auto fn) {
    int s = tile0;
    for (int64_t row = r0; row < r1; ++row) {
      const int kept = row == r0 ? kept0 : kept_of(row), n = (kept + 127) / 128;
      fn(row, kept, s, n, n ? (s + n - 1) / quota - s / quota + 1 : 0);
      s += n;
    }
  };
  int items = 0, cuts = 0;  // cuts: pieces of cut rows << 16 | cut rows (at most 2 and 1 per CTA)
  for_rows([&](int64_t row, int, int, int, int pieces) {
    a.flags[row] = 0;
    items += pieces;
    cuts += pieces > 1 ? pieces << 16 | 1 : 0;
  });
  int all_items, all_cuts;
  int at = block_exclusive_scan<NT>(items, s_tmp, &all_items);
  const int before = block_exclusive_scan<NT>(cuts, s_tmp, &all_cuts);
  int part = before >> 16, cut = before & 0xffff;
  for_rows([&](int64_t row, int kept, int s, int n, int pieces) {
    if (pieces > 1) a.cut[cut++] = make_int4(int(row), part, pieces, 0);
    const int c0 = s / quota;
    for (int j = 0; j < pieces; ++j, ++at) {
      const int lo = max(s, (c0 + j) * quota), hi = min(s + n, (c0 + j + 1) * quota);
      a.attn_items[at] = make_int4(int(row), (lo - s) | (hi - lo) << 8 | kept << 16, pieces > 1 ? part++ : -1, 0);
      if (lo == (c0 + j) * quota) a.cta_items[c0 + j] = at;  // the first item of CTA c0 + j
    }
  });
  for (int c = (total + quota - 1) / quota + tid; c <= kTreeAttnCtas; c += NT) a.cta_items[c] = all_items;
  // (a cut lies between two CTAs, so fewer rows than CTAs are cut)
  for (int c = (all_cuts & 0xffff) + tid; c < kTreeAttnCtas; c += NT) a.cut[c] = make_int4(-1, 0, 0, 0);
}

__device__ void tail_keys(const TreeArgs& a, int64_t row) {  // a warp per node
  const int64_t c = a.ctx[row / a.T];
  const int t = a.rowpos[row];
  if (t < 0 || candidates(t, a.B, a.m) <= a.k) return;
  const int f = int(c / a.B), lane = threadIdx.x & 31;
  const int n = t - f * a.B + 1;  // the node's tail rows
  const uint32_t* src = a.tailkeys + row * a.tail_ld;
  // the kept tail blocks are the last of the list, 32 looked up at a time
  for (int s0 = min(a.m, t / a.B + 1) - 1; s0 >= 0; s0 -= 32) {
    const int mine = s0 - lane >= 0 ? a.blocks[row * a.m + s0 - lane] : -1;
    const int cnt = __popc(__ballot_sync(kFull, mine >= f));
    for (int u = 0; u < cnt; ++u) {
      const int r0 = (__shfl_sync(kFull, mine, u) - f) * a.B;
      uint32_t* dst = a.tkeys + (row * a.m + s0 - u) * int64_t(a.B);
      for (int r = lane; r < a.B && r0 + r < n; r += 32) dst[r] = src[r0 + r];
    }
    if (cnt < 32) break;
  }
}

__global__ void __launch_bounds__(kListNT) tree_lists_kernel(const TreeArgs a, int batch, int ranges) {
  __shared__ int hist[kListNT];  // pair counts of this range's blocks, then cursors
  __shared__ int s_tmp[kListNT / 32 + 1];
  __shared__ int s_base[2];
  __shared__ uint8_t need[kTreeMax];
  griddep_wait();
  griddep_launch();
  if (blockIdx.x == gridDim.x - 1) {
    attn_shares<kListNT>(a, int64_t(batch) * a.T, s_tmp);
    return;
  }
  if (int(blockIdx.x) >= batch * ranges) {
    const int64_t row = (int64_t(blockIdx.x) - int64_t(batch) * ranges) * (kListNT / 32) + (threadIdx.x >> 5);
    if (row < int64_t(batch) * a.T) tail_keys(a, row);
    return;
  }
  const int64_t b = blockIdx.x / ranges;
  const int tid = threadIdx.x, lo = int(blockIdx.x % ranges) * kListNT;
  const int32_t* blocks = a.blocks + b * a.T * a.m;
  const int entries = a.T * a.m;
  constexpr int U = 8;
  int first[U];  // this thread's first entries, loaded beside the lengths
#pragma unroll
  for (int u = 0; u < U; ++u) first[u] = tid + u * kListNT < entries ? blocks[tid + u * kListNT] : -1;
  const int64_t c = a.ctx[b];
  if (tid < a.T) {
    const int t = a.rowpos[b * a.T + tid];
    need[tid] = t >= 0 && candidates(t, a.B, a.m) > a.k;
  }
  hist[tid] = 0;
  if (c < 0 || c >= a.capacity) return;
  const int end = min(int(c / a.B), lo + kListNT);  // cached whole blocks of this range
  __syncthreads();
  // f(entry, block) for the entries of this range whose nodes need scores
  auto for_entries = [&](auto fn) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int e = tid + u * kListNT;
      if (first[u] >= lo && first[u] < end && need[e / a.m]) fn(e, first[u]);
    }
    for (int e = tid + U * kListNT; e < entries; e += kListNT) {
      const int blk = blocks[e];
      if (blk >= lo && blk < end && need[e / a.m]) fn(e, blk);
    }
  };
  for_entries([&](int, int blk) { atomicAdd(&hist[blk - lo], 1); });
  __syncthreads();
  // this range's items, `per` for each block with a pair, and pairs: one scan of
  // both counts (at most 512 blocks and 64 * 512 pairs)
  const int per = (a.B + 127) / 128;
  const int cnt = hist[tid];
  int total;
  const int at = block_exclusive_scan<kListNT>(cnt | int(cnt > 0) << 20, s_tmp, &total);
  const int at_p = at & 0xfffff, at_i = at >> 20;
  if (total == 0) return;
  if (tid == 0) s_base[0] = atomicAdd(a.counters, (total >> 20) * per);
  if (tid == 32) s_base[1] = atomicAdd(a.counters + 1, total & 0xfffff);
  hist[tid] = at_p;
  __syncthreads();
  uint32_t* pairs = a.pairs + s_base[1];
  if (cnt)
    for (int ch = 0; ch < per; ++ch)
      a.items[s_base[0] + at_i * per + ch] =
          make_int4(int(b * a.capacity) + (lo + tid) * a.B + 128 * ch, s_base[1] + at_p,
                    cnt | (min(128, a.B - 128 * ch) << 16), int(b << 3) | ch);
  for_entries([&](int e, int blk) {
    const int i = e / a.m;
    pairs[atomicAdd(&hist[blk - lo], 1)] = uint32_t(i) << 16 | uint32_t(e - i * a.m);
  });
}

// ---------------------------------------------------------------------------
// Token scores of few nodes without lists: grid (node, slot), a CTA per kept
// block of each node, on CUDA cores. A block that several nodes kept is read by
// each (from L2), but no list has to be made first: that launch costs more than
// the reading as long as there is little of it (see tree_few_scores).
// ---------------------------------------------------------------------------
constexpr int kFewNT = 128;

template <int DI>
__global__ void __launch_bounds__(kFewNT) tree_few_scores_kernel(const TreeArgs a, int64_t rows) {
  __shared__ int s_tmp[kFewNT / 32 + 1];
  griddep_wait();
  griddep_launch();
  if (int(blockIdx.y) == a.m) {
    if (blockIdx.x == 0) attn_shares<kFewNT>(a, rows, s_tmp);
    return;
  }
  const int64_t row = blockIdx.x, b = row / a.T;
  const int blk = a.blocks[row * a.m + blockIdx.y];
  const int t = a.rowpos[row], c = a.ctx[b];
  constexpr int LPR = DI / 8, RPC = kFewNT / LPR, U = 8;  // lanes per key row, rows per CTA at a time, turns in flight
  const int sub = threadIdx.x % LPR, r1 = threadIdx.x / LPR;
  const uint4 qv = __ldg(reinterpret_cast<const uint4*>(a.q_new + row * DI) + sub);
  if (t < 0 || blk < 0 || candidates(t, a.B, a.m) <= a.k) return;
  uint32_t* out = a.tkeys + (row * a.m + blockIdx.y) * int64_t(a.B);
  const int f = c / a.B;
  if (blk >= f) {  // a tail block
    const uint32_t* src = a.tailkeys + row * a.tail_ld + (blk - f) * a.B;
    const int n = min(a.B, t - blk * a.B + 1);
    for (int r = threadIdx.x; r < n; r += kFewNT) out[r] = src[r];
    return;
  }
  const uint4* kb = reinterpret_cast<const uint4*>(a.k_idx_cache + (b * a.capacity + int64_t(blk) * a.B) * DI) + sub;
  const uint32_t qw[4] = {qv.x, qv.y, qv.z, qv.w};
  for (int r0 = r1; r0 < a.B + r1; r0 += RPC * U) {  // (every lane of a warp takes part in the sums)
    uint4 kv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPC;
      kv[u] = r < a.B ? __ldg(kb + int64_t(r) * LPR) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t kw[4] = {kv[u].x, kv[u].y, kv[u].z, kv[u].w};
      float acc = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc = __fmaf_rn(bf16_lo(qw[e]), bf16_lo(kw[e]), acc);
        acc = __fmaf_rn(bf16_hi(qw[e]), bf16_hi(kw[e]), acc);
      }
#pragma unroll
      for (int o = LPR / 2; o >= 1; o >>= 1) acc += __shfl_xor_sync(kFull, acc, o);
      const int r = r0 + u * RPC;
      if (sub == 0 && r < a.B) out[r] = score_key(acc);
    }
  }
}

// ---------------------------------------------------------------------------
// Selections with a wide CTA per row: what a step's latency needs, where the
// prefill's kernels are made for many rows (a step of 8 nodes at 128K with 1024,
// 512 and 256 threads per top-k row: 34.8, 35.6 and 38.9 us).
//
// WideSelect picks the r largest of n keys (1 <= r < n <= 16384) held in
// registers, thread t positions t*KPT .. t*KPT + KPT - 1, ties to the lowest
// position. One histogram of 2048 bins linear in the score finds the bin of the
// r-th largest; its keys, if at most 64, are ranked pairwise. A crowded bin (or
// a range that is not finite) goes through RegSelect's rounds. Counts cross the
// CTA by one value per warp that every warp sums for itself: five barriers, or
// seven with a ranking, where the general selection takes some sixteen (top-k of
// 8192 keys with its loads: 7.0 us before).
// ---------------------------------------------------------------------------
template <int NT, int KPT>
struct __align__(16) WideSmem {
  uint32_t hist[RegSelect<NT, KPT>::kBins];
  uint32_t list[64];
  int warp[3][NT / 32];
  int pick[4];
  int scratch[NT / 32 + 8];
};

template <int NT, int KPT>
struct WideSelect {
  static constexpr int NW = NT / 32, kBins = RegSelect<NT, KPT>::kBins, BPT = kBins / NT;
  WideSmem<NT, KPT>& S;

  // before the keys are there: no barrier, the first one in select() covers it
  HSA_DEV void prepare() {
#pragma unroll
    for (int e = 0; e < BPT; ++e) S.hist[threadIdx.x * BPT + e] = 0;
    if (threadIdx.x == 0) S.pick[2] = 0;
  }

  // The thread's selected keys as bits, and how many are selected at lower positions.
  HSA_DEV uint32_t select(const uint32_t (&key)[KPT], int n, int r, int* before) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int have = max(0, min(KPT, n - int(threadIdx.x) * KPT));
    uint32_t lo = 0xffffffffu, hi = 0u;
#pragma unroll
    for (int j = 0; j < KPT; ++j)
      if (j < have) { lo = min(lo, key[j]); hi = max(hi, key[j]); }
    lo = __reduce_min_sync(kFull, lo);
    hi = __reduce_max_sync(kFull, hi);
    if (lane == 0) { S.warp[0][w] = int(lo); S.warp[1][w] = int(hi); }
    __syncthreads();
    lo = __reduce_min_sync(kFull, lane < NW ? uint32_t(S.warp[0][lane]) : 0xffffffffu);
    hi = __reduce_max_sync(kFull, lane < NW ? uint32_t(S.warp[1][lane]) : 0u);
    const float flo = key_score(lo), fhi = key_score(hi), c = float(kBins - 1) / (fhi - flo);
    // A bin never decreases as the score grows (every step is monotone), so it is a range of keys. Adding 2^23
    // leaves the rounded bin in the low bits: a conversion runs at a quarter of the rate.
    auto vbin = [&](uint32_t u) {
      return min(__float_as_uint(__fmaf_rn(key_score(u) - flo, c, 8388608.f)) - 0x4b000000u, uint32_t(kBins - 1));
    };
    // the r-th largest key, and how many of its equals are taken
    uint32_t T = 0;
    int take_eq = -1;
    if (flo < fhi && c > 0.f && c < INFINITY) {
#pragma unroll
      for (int j = 0; j < KPT; ++j)
        if (j < have) atomicAdd(&S.hist[vbin(key[j])], 1u);
      __syncthreads();
      int cnt[BPT], tot = 0;
#pragma unroll
      for (int e = 0; e < BPT; ++e) { cnt[e] = int(S.hist[threadIdx.x * BPT + e]); tot += cnt[e]; }
      int x = tot;  // over the warp's lanes from this one on
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_down_sync(kFull, x, o);
        if (lane + o < 32) x += y;
      }
      if (lane == 0) S.warp[2][w] = x;
      __syncthreads();
      int above = x - tot + int(__reduce_add_sync(kFull, lane < NW && lane > w ? unsigned(S.warp[2][lane]) : 0u));
      if (above < r && r <= above + tot) {
#pragma unroll
        for (int e = BPT - 1; e >= 0; --e) {
          if (above < r && r <= above + cnt[e]) { S.pick[0] = threadIdx.x * BPT + e; S.pick[1] = above; }
          above += cnt[e];
        }
      }
      __syncthreads();
      const uint32_t bin = uint32_t(S.pick[0]);
      const int rem = r - S.pick[1], in = int(S.hist[bin]);
      if (in <= 64) {
#pragma unroll
        for (int j = 0; j < KPT; ++j)
          if (j < have && vbin(key[j]) == bin) S.list[atomicAdd(&S.pick[2], 1)] = key[j];
        __syncthreads();
        if (int(threadIdx.x) < in) {
          const uint32_t u = S.list[threadIdx.x];
          int gt = 0, ge = 0;
#pragma unroll 8
          for (int q = 0; q < in; ++q) {
            const uint32_t y = S.list[q];
            gt += y > u;
            ge += y >= u;
          }
          if (gt < rem && rem <= ge) { S.pick[0] = int(u); S.pick[3] = rem - gt; }  // writers agree
        }
        __syncthreads();
        T = uint32_t(S.pick[0]);
        take_eq = S.pick[3];
      }
    }
    if (take_eq < 0) {  // (the whole CTA)
      __syncthreads();
      RegSelect<NT, KPT> rs{S.hist, S.scratch};
      rs.threshold(key, n, r, &T, &take_eq);
    }
    uint32_t gt = 0, eq = 0;
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      gt |= uint32_t(j < have && key[j] > T) << j;
      eq |= uint32_t(j < have && key[j] == T) << j;
    }
    const int mine = __popc(gt) << 16 | __popc(eq);  // (both counts stay below 2^15)
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) S.warp[0][w] = incl;
    __syncthreads();
    const int at = incl - mine + int(__reduce_add_sync(kFull, lane < w ? unsigned(S.warp[0][lane]) : 0u));
    const int gt_before = at >> 16, eq_before = at & 0xffff;
    *before = gt_before + min(eq_before, take_eq);
    for (int q = eq_before; eq && q < take_eq; eq &= eq - 1, ++q) gt |= eq & (0u - eq);
    return gt;
  }
};

// Top-m: candidate c is block c + 1 of 1 .. nb-2; bkeys rows start three keys
// in, so that block 1's key is on 16 bytes.
template <int NT, int KPT>
__global__ void __launch_bounds__(NT) tree_topm_kernel(const TreeArgs a, int32_t* __restrict__ blocks) {
  __shared__ WideSmem<NT, KPT> S;
  WideSelect<NT, KPT> sel{S};
  sel.prepare();
  griddep_wait();
  griddep_launch();
  const int64_t row = blockIdx.x;
  uint32_t key[KPT];  // (loaded beside the position: the row holds at least capacity / B - 1 keys)
  load_keys<KPT>(a.bkeys + row * a.ldb + kBkeys0 + 1, int(a.ldb) - kBkeys0 - 1, key);
  const int64_t t = a.rowpos[row];
  int32_t* out = blocks + row * a.m;
  const int64_t nb = t < 0 ? 0 : t / a.B + 1;
  if (nb <= a.m) {
    for (int s = threadIdx.x; s < a.m; s += NT) out[s] = s < nb ? s : -1;
    return;
  }
  if (threadIdx.x == 0) { out[0] = 0; out[a.m - 1] = int32_t(nb - 1); }
  if (a.m == 2) return;
  int at;
  uint32_t bits = sel.select(key, int(nb - 2), a.m - 2, &at);
  for (; bits; bits &= bits - 1) out[1 + at++] = threadIdx.x * KPT + __ffs(bits);
}

// Top-k of a node's candidates (the tokens of its kept blocks, ascending), and
// their positions as rows of the sequence's cache; up to 2048 are gathered over
// the histogram and written out whole. (A buffer of its own for more would keep
// the attention's CTA from being set up beside this one.)
template <int NT, int KPT>
__global__ void __launch_bounds__(NT, NT == 1024 && KPT <= 8 ? 2 : 1) tree_topk_kernel(const TreeArgs a,
                                                                                      int32_t* __restrict__ idx) {
  __shared__ WideSmem<NT, KPT> S;
  __shared__ int blk[512];
  __shared__ int path[kTreeMax];
  WideSelect<NT, KPT> sel{S};
  sel.prepare();
  griddep_wait();
  griddep_launch();
  const int64_t row = blockIdx.x;
  // every load at once; keys behind the row's candidates are not looked at
  uint32_t key[KPT];
  load_keys<KPT>(a.tkeys + row * int64_t(a.m) * a.B, a.m * a.B, key);
  const int t = a.rowpos[row], c0 = a.ctx[row / a.T];
  for (int s = threadIdx.x; s < a.m; s += NT) blk[s] = a.blocks[row * a.m + s];
  if (int(threadIdx.x) < a.T) path[threadIdx.x] = min(max(a.paths[row * a.T + threadIdx.x], 0), a.T - 1);
  int32_t* out = idx + row * a.k;
  if (t < 0) {
    for (int s = threadIdx.x; s < a.k; s += NT) out[s] = -1;
    return;
  }
  const int n = candidates(t, a.B, a.m);
  const bool pow2 = (a.B & (a.B - 1)) == 0;
  const int lb = 31 - __clz(a.B);
  auto row_of = [&](int c) -> int32_t {
    const int p = pow2 ? (blk[c >> lb] << lb) + (c & (a.B - 1)) : blk[c / a.B] * a.B + c % a.B;
    return p < c0 ? p : c0 + path[p - c0];
  };
  if (n <= a.k) {
    __syncthreads();
    for (int s = threadIdx.x; s < a.k; s += NT) out[s] = s < n ? row_of(s) : -1;
    return;
  }
  int at;
  uint32_t bits = sel.select(key, n, a.k, &at);
  int32_t* kept = a.k <= int(sizeof(S.hist) / 4) ? reinterpret_cast<int32_t*>(S.hist) : out;
  for (; bits; bits &= bits - 1) kept[at++] = row_of(threadIdx.x * KPT + __ffs(bits) - 1);
  if (kept == out) return;
  __syncthreads();
  if ((a.k & 3) == 0) {
    for (int e = threadIdx.x; e < a.k / 4; e += NT) reinterpret_cast<int4*>(out)[e] = reinterpret_cast<const int4*>(kept)[e];
  } else {
    for (int e = threadIdx.x; e < a.k; e += NT) out[e] = kept[e];
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
  const int n = min(a.k, candidates(int(t), a.B, a.m));
  const int32_t* path = a.paths + row * a.T;
  int32_t* out = idx + row * a.k;
  for (int e0 = n - 32; e0 > -32; e0 -= 32) {
    const int e = e0 + lane;
    const int p = e >= 0 ? out[e] : -1;
    const bool late = p >= c;
    if (late) out[e] = c + min(max(path[min(p - c, a.T - 1)], 0), a.T - 1);
    if (!__all_sync(kFull, late)) break;
  }
}

// One head of a row whose weights left the range that the attention's fixed
// reference covers, on CUDA cores with a running maximum, by a warp: 32 kept
// rows at a time, eight of them loaded at once, a lane holding D / 32 values of
// each. Weights are held times 2^-13, so that 8192 of them times the largest
// values stay in range. (Out of line: the registers it needs would halve the
// combination's CTAs.)
template <int D>
__device__ __noinline__ void attend_head(const uint16_t* K, const uint16_t* V, const int32_t* idx, int n,
                                         const uint16_t* q, float scale, uint16_t* out) {
  constexpr int W = D / 64;  // 32-bit words per lane and row
  const int lane = threadIdx.x & 31;
  float qv[2 * W], o[2 * W] = {};
#pragma unroll
  for (int e = 0; e < W; ++e) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(q)[lane * W + e];
    qv[2 * e] = bf16_lo(w);
    qv[2 * e + 1] = bf16_hi(w);
  }
  float M = -INFINITY, l = 0.f;
#pragma unroll 1
  for (int c0 = 0; c0 < n; c0 += 32) {
    const int j = max(idx[min(c0 + lane, n - 1)], 0);
    float x = -INFINITY;  // lane i: the score of row c0 + i
#pragma unroll 1
    for (int k0 = 0; k0 < 32; k0 += 8) {
      uint32_t w[8][W];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t* r = reinterpret_cast<const uint32_t*>(K + int64_t(__shfl_sync(kFull, j, k0 + i)) * D) + lane * W;
#pragma unroll
        for (int e = 0; e < W; ++e) w[i][e] = r[e];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float acc = 0.f;
#pragma unroll
        for (int e = 0; e < W; ++e) {
          acc = __fmaf_rn(qv[2 * e], bf16_lo(w[i][e]), acc);
          acc = __fmaf_rn(qv[2 * e + 1], bf16_hi(w[i][e]), acc);
        }
#pragma unroll
        for (int s = 16; s >= 1; s >>= 1) acc += __shfl_xor_sync(kFull, acc, s);
        if (lane == k0 + i && c0 + lane < n) x = acc * scale;
      }
    }
    float top = x;  // (the maximum leaves NaN out, the sum below does not)
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, s));
    const float Mn = fmaxf(M, top), ref = Mn == -INFINITY ? 0.f : Mn;
    const float g = M == -INFINITY ? 0.f : expf(M - ref), p = expf(x - ref) * 1.220703125e-4f;
    float add = p;
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) add += __shfl_xor_sync(kFull, add, s);
    l = l * g + add;
    M = Mn;
#pragma unroll
    for (int e = 0; e < 2 * W; ++e) o[e] *= g;
#pragma unroll 1
    for (int k0 = 0; k0 < 32; k0 += 8) {
      uint32_t w[8][W];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t* r = reinterpret_cast<const uint32_t*>(V + int64_t(__shfl_sync(kFull, j, k0 + i)) * D) + lane * W;
#pragma unroll
        for (int e = 0; e < W; ++e) w[i][e] = r[e];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float pi = __shfl_sync(kFull, p, k0 + i);
        if (c0 + k0 + i >= n) break;  // (rows past the list repeat its last one)
#pragma unroll
        for (int e = 0; e < W; ++e) {
          o[2 * e] = __fmaf_rn(pi, bf16_lo(w[i][e]), o[2 * e]);
          o[2 * e + 1] = __fmaf_rn(pi, bf16_hi(w[i][e]), o[2 * e + 1]);
        }
      }
    }
  }
  // (every score -inf: no weights at all, as a row that keeps nothing)
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < W; ++e)
    reinterpret_cast<uint32_t*>(out)[lane * W + e] = cvt_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
}

// O of the rows that were cut (with M the largest part maximum, O = sum_p
// 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p in log2 units), and of the flagged
// groups of eight heads (taken again). Grid (cut, head groups), a thread per four
// values; the parts come U at a time, every load of a group issued before any is
// used.
template <int D, int U>
__global__ void __launch_bounds__(256, U == 4 ? 6 : 2) tree_combine_kernel(const TreeArgs a,
                                                                          const uint16_t* __restrict__ Q,
                                                                          const int32_t* __restrict__ idx, float scale,
                                                                          const float* __restrict__ Opart,
                                                                          const float* __restrict__ mpart,
                                                                          const float* __restrict__ lpart) {
  constexpr int TPH = D / 4, HPC = 256 / TPH;  // threads per head, heads per CTA at a time
  griddep_wait();
  griddep_launch();
  const int H = a.H, v = threadIdx.x % TPH;
  const int4 cut = a.cut[blockIdx.x];
  const int flags = cut.x < 0 ? 0 : a.flags[cut.x];  // (its load is not waited for until a store)
  for (int h = blockIdx.y * HPC + threadIdx.x / TPH; cut.x >= 0 && h < H; h += gridDim.y * HPC) {
    float M = -INFINITY, den = 0.f;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < cut.z; p0 += U) {
      float l[U], m[U];
      float4 o[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool in = p0 + u < cut.z;
        const int64_t w = int64_t(cut.y + p0 + u) * H + h;
        l[u] = in ? lpart[w] : 0.f;
        m[u] = in ? mpart[w] : -INFINITY;
        o[u] = in ? reinterpret_cast<const float4*>(Opart + w * D)[v] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float top = M;
#pragma unroll
      for (int u = 0; u < U; ++u) top = fmaxf(top, m[u]);
      const float g = p0 > 0 ? exp2f(M - top) : 1.f;  // (a row not flagged has finite maxima)
      num.x *= g; num.y *= g; num.z *= g; num.w *= g;
      den *= g;
      M = top;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float f = exp2f(m[u] - M);
        num.x = __fmaf_rn(f, o[u].x, num.x); num.y = __fmaf_rn(f, o[u].y, num.y);
        num.z = __fmaf_rn(f, o[u].z, num.z); num.w = __fmaf_rn(f, o[u].w, num.w);
        den = __fmaf_rn(f, l[u], den);
      }
    }
    const float inv = 1.f / den;
    if (!(flags >> (h >> 3) & 1))
      reinterpret_cast<uint2*>(a.O + (int64_t(cut.x) * H + h) * D)[v] =
          make_uint2(cvt_bf16x2(num.x * inv, num.y * inv), cvt_bf16x2(num.z * inv, num.w * inv));
  }
  const int again = a.counters[2];
  for (int i = blockIdx.x; i < again; i += gridDim.x) {
    const int64_t row = a.flagged[i];
    const int64_t base = row / a.T * a.capacity * D;
    const int n = min(a.k, candidates(a.rowpos[row], a.B, a.m)), bits = a.flags[row];
    for (int h = blockIdx.y * 8 + threadIdx.x / 32; h < H; h += gridDim.y * 8)
      if (bits >> (h >> 3) & 1)
        attend_head<D>(a.K_cache + base, a.V_cache + base, idx + row * a.k, n, Q + (row * H + h) * D, scale,
                       a.O + (row * H + h) * D);
  }
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

void launch_tree_lists(const TreeArgs& a, int batch, cudaStream_t s) {
  const int ranges = int((a.capacity / a.B + kListNT - 1) / kListNT);
  count_launches(1);
  const unsigned tails = unsigned((int64_t(batch) * a.T + kListNT / 32 - 1) / (kListNT / 32));
  launch_kernel(true, tree_lists_kernel, unsigned(batch * ranges) + tails + 1, kListNT, 0, s, a, batch, ranges);
}

bool tree_few_scores(const TreeArgs& a, int64_t rows, int d_idx) {
  // by the bytes that all nodes' kept blocks have. A whole step with lists / without them: 42.2 / 37.2 us at
  // 16 MB (8 nodes, m = 64, B = 128), 51.4 / 49.2 at 64 MB (32 nodes), 55.0 / 53.8 at 128 MB (8 x 8 nodes),
  // 62.5 / 65.3 at 256 MB (16 x 8 nodes)
  return rows * a.m * a.B * int64_t(d_idx) * 2 <= int64_t(128) << 20;
}

void launch_tree_few_scores(const TreeArgs& a, int64_t rows, int d_idx, cudaStream_t s) {
  const dim3 grid{unsigned(rows), unsigned(a.m + 1)};
  count_launches(1);
  launch_kernel(true, d_idx == 128 ? tree_few_scores_kernel<128> : tree_few_scores_kernel<64>, grid, kFewNT, 0, s, a,
                rows);
}

void launch_tree_topm(const TreeArgs& a, int64_t rows, int32_t* blocks, cudaStream_t s) {
  const int64_t n = a.capacity / a.B;
  count_launches(1);
  auto go = [&](auto kern, int nt) { launch_kernel(true, kern, unsigned(rows), nt, 0, s, a, blocks); };
  if (n <= 256) go(tree_topm_kernel<256, 1>, 256);
  else if (n <= 1024) go(tree_topm_kernel<256, 4>, 256);
  else if (n <= 2048) go(tree_topm_kernel<512, 4>, 512);
  else if (n <= 4096) go(tree_topm_kernel<1024, 4>, 1024);
  else if (n <= 8192) go(tree_topm_kernel<1024, 8>, 1024);
  else go(tree_topm_kernel<1024, 16>, 1024);  // (at most 16384 blocks)
}

bool tree_topk_wide(const TreeArgs& a, int64_t rows) {
  const int64_t n = int64_t(a.m) * a.B;
  return n <= 16384 && (rows <= kWideRows || n <= kWideKeys || !topk_rows_takes(a.B, a.m));
}

void launch_tree_topk(const TreeArgs& a, int64_t rows, int32_t* idx, cudaStream_t s) {
  const int64_t n = int64_t(a.m) * a.B;
  count_launches(1);
  auto go = [&](auto kern, int nt) { launch_kernel(true, kern, unsigned(rows), nt, 0, s, a, idx); };
  if (n <= 256) go(tree_topk_kernel<256, 1>, 256);
  else if (n <= 1024) go(tree_topk_kernel<256, 4>, 256);
  else if (n <= 4096) go(tree_topk_kernel<1024, 4>, 1024);
  else if (n <= 8192) go(tree_topk_kernel<1024, 8>, 1024);
  else go(tree_topk_kernel<1024, 16>, 1024);
}

void launch_tree_rows(const TreeArgs& a, int64_t rows, int32_t* idx, cudaStream_t s) {
  count_launches(1);
  launch_kernel(true, tree_rows_kernel, unsigned((rows + 7) / 8), 256, 0, s, a, rows, idx);
}

void launch_tree_combine(const TreeArgs& a, int64_t rows, const void* Q, const int32_t* idx, float scale,
                         const float* Opart, const float* mpart, const float* lpart, cudaStream_t s) {
  const dim3 grid{unsigned(kTreeAttnCtas), unsigned((a.H * a.d + 1023) / 1024)};
  count_launches(1);
  // few rows are cut into many parts, many rows into two: there fewer registers put the grid into one wave. A
  // whole step (us, 16 parts at a time / 4): 1 row 36.9 / 38.9, 16 rows 41.9 / 43.0, 24 rows 49.1 / 49.2, 32 rows
  // 49.2 / 47.1 (of k = 512 and H = 8: 41.0 / 43.0), 64 rows 63.5 / 61.4, 256 rows 108.6 / 106.5 (k = 2048, H = 64)
  auto kern = rows <= 32 ? (a.d == 128 ? tree_combine_kernel<128, 16> : tree_combine_kernel<64, 16>)
                         : (a.d == 128 ? tree_combine_kernel<128, 4> : tree_combine_kernel<64, 4>);
  launch_kernel(true, kern, grid, 256, 0, s, a, (const uint16_t*)Q, idx, scale, Opart, mpart, lpart);
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
