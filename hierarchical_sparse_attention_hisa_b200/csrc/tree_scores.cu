// Scores of a drafted tree's nodes, on tcgen05 where nodes share what they
// score. In both kernels the scored rows are the MMA's M dimension and all of a
// sequence's nodes its N (16, 32 or 64 columns), so a row is read once whatever
// number of nodes it is scored for, and an accumulator column is one node's
// scores of 128 consecutive rows: 128 epilogue threads (TMEM lane = row) write
// it as 512 contiguous bytes. Every wait is bounded.
#include <algorithm>

#include "kernels.cuh"
#include "tc.cuh"

namespace hsa {

__device__ int g_tree_err;
__device__ int g_tree_inject;  // test hook: short waits and one item never produced

namespace {

using namespace tc;

constexpr long long kInjectWaitCycles = 1ll << 21;  // about a millisecond

HSA_DEV void tmem_ld1(uint32_t taddr, uint32_t& r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
}

// Bounded wait; the limit, the error flag and the test hook are slow to read, so
// they are looked at once in 64 probes.
HSA_DEV bool tw_wait(uint64_t* bar, uint32_t parity, bool& dead) {
  if (dead) return false;
  long long t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*(volatile int*)&g_tree_err) break;
      const long long t = clock64();
      if (t0 == 0) t0 = t;
      if (t - t0 > (*(volatile int*)&g_tree_inject ? kInjectWaitCycles : kWaitCycles)) {
        atomicExch(&g_tree_err, 1);
        break;
      }
    }
  }
  dead = true;
  return false;
}
// Every lane polls (a lane that polls for the others holds the warp up).
HSA_DEV bool tw_wait_warp(uint64_t* bar, uint32_t parity, bool& dead) {
  const bool ok = __all_sync(kFull, tw_wait(bar, parity, dead));
  dead = !ok;
  return ok;
}

// ---------------------------------------------------------------------------
// Block scores, grid (sequence, 128 cached whole blocks):
//   bkeys[row][blk] = key(q . ksum[blk]),  ksum = hi + mid + lo in bf16,
// three MMAs per 16 summed values (as the prefill's block scores: exact for
// sums of at most 24 significant bits). A CTA reads its fp32 sums once (HBM),
// splits them in registers and writes the planes straight into the swizzled
// layout the MMA reads. On CUDA cores the same tile is bound by shared memory
// (2.4 us per SM at 16 nodes, FMAs at 64).
//
// Tails, a launch of its own with four warps per node: append the node's
// drafted rows to the caches and score its tail, the rows of its path from f*B
// on. A tail block's score is the sum of its token scores: q . sum k =
// sum q . k.
//
// The two do not depend on one another, and the tails' CTAs are small, the
// blocks' (113 KB at d_idx = 128) two to an SM: as parts of one launch they ran
// as two waves (17 us for 32 x 16 nodes at 128K), as two they share the SMs.
// ---------------------------------------------------------------------------
constexpr int kBlkTile = 128;
constexpr int kNT = 256, kNodeNT = 128, kNodesPerCta = kNT / kNodeNT;

// Node i's position, or -1 if it takes no part. A plan made for other lengths
// must not reach outside the sequence's rows.
HSA_DEV int64_t node_position(const TreeArgs& a, int64_t b, int i) {
  const int64_t c = a.ctx[b], t = a.positions[b * a.T + i];
  return c >= 0 && t >= c && t - c <= i && c + i < a.capacity ? t : -1;
}

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

// tid: 0 .. kNodeNT-1 within the node's warps; bar: their named barrier; sc: tail_ld floats
template <int DI>
__device__ void node_tail(const TreeArgs& a, int64_t b, int i, int tid, int bar, float* sc) {
  const int64_t row = b * a.T + i;
  const int64_t c = a.ctx[b];
  const int64_t t = node_position(a, b, i);
  if (tid == 0) a.rowpos[row] = int32_t(t);
  if (t < 0) {
    uint4* o = reinterpret_cast<uint4*>(a.O + row * a.H * a.d);
    for (int e = tid; e < a.H * a.d / 8; e += kNodeNT) o[e] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int lane = tid & 31, warp = tid >> 5;
  {  // the drafted rows, node i in cache row c + i
    const int64_t at = b * a.capacity + c + i;
    const int ci = DI / 8, cd = a.d / 8;
    for (int e = tid; e < ci + 2 * cd; e += kNodeNT) {
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
  const bool tokens = candidates(int(t), a.B, a.m) > a.k;  // else all are kept, without scores
  const bool blocks = nb > a.m && f < nb - 1;  // whole blocks in the tail
  if (!tokens && !blocks) return;
  // tail rows: cached ones from f*B, then the path
  const int head = int(c - f * a.B), n = head + int(t - c) + 1;
  constexpr int LPR = DI / 8, RPW = 32 / LPR, NW = kNodeNT / 32;
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
  constexpr int U = 8;  // rows in flight per lane group
  for (int r0 = warp * RPW; r0 < n; r0 += NW * RPW * U) {
    uint4 kv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * NW * RPW + rsub;
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
      const int r = r0 + u * NW * RPW + rsub;
      float acc = dot8(kv[u], q);
#pragma unroll
      for (int o = LPR / 2; o >= 1; o >>= 1) acc += __shfl_xor_sync(kFull, acc, o);
      if (sub == 0 && r < n) {
        sc[r] = acc;
        keys[r] = score_key(acc);
      }
    }
  }
  if (!blocks) return;
  bar_sync(bar, kNodeNT);
  for (int64_t blk = f + warp; blk < nb - 1; blk += NW) {
    float s = 0.f;
    for (int r = lane; r < a.B; r += 32) s += sc[(blk - f) * a.B + r];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    if (lane == 0) a.bkeys[row * a.ldb + kBkeys0 + blk] = score_key(s);
  }
}

template <int DI, int N>
struct BS {
  static constexpr int PLANE = kBlkTile * DI * 2;  // one bf16 plane of the sums
  static constexpr int OFF_Q = 3 * PLANE;
  static constexpr int SMEM = OFF_Q + N * DI * 2 + 1024;
  static constexpr int TMEM_COLS = N < 32 ? 32 : N;
};

template <int DI, int N>
__device__ void cached_block_scores(const TreeArgs& a, int64_t b, int tile, uint8_t* sm, uint64_t* bar,
                                    uint32_t* tmem_base) {
  using C = BS<DI, N>;
  constexpr int CPR = DI / 8;  // eight-value chunks per row
  const int64_t c = __ldcg(a.ctx + b);  // (loads by L2 alone: see the kernel)
  if (c < 0 || c >= a.capacity) return;
  const int64_t f = c / a.B;
  const int64_t lo = int64_t(tile) * kBlkTile;
  const int n = int(min(int64_t(kBlkTile), f - lo));
  if (n <= 0) return;
  if ((c + a.T - 1) / a.B + 1 <= a.m) return;  // every node keeps all its blocks
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float4* src = reinterpret_cast<const float4*>(a.ksum_cache + (b * (a.capacity / a.B) + lo) * DI);
  constexpr int PER = kBlkTile * CPR / kNT;
  float4 x[PER][2];
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int e = tid + u * kNT;  // (row, chunk) = (e / CPR, e % CPR)
    x[u][0] = x[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (e / CPR < n) {
      x[u][0] = __ldcg(src + 2 * e);
      x[u][1] = __ldcg(src + 2 * e + 1);
    }
  }
  if (warp == 0) { tmem_alloc(tmem_base, C::TMEM_COLS); tmem_relinquish(); }
  if (tid == 0) { mbar_init(bar, 1); fence_barrier_init(); }
  for (int e = tid; e < a.T * CPR; e += kNT) {  // (columns past the nodes hold anything: nobody reads them)
    const int r = e / CPR, ch = e % CPR;
    *reinterpret_cast<uint4*>(sm + C::OFF_Q + (ch >> 3) * (N * 128) + swz_offset(r, ch & 7, 128)) =
        __ldcg(reinterpret_cast<const uint4*>(a.q_new + b * a.T * DI) + e);
  }
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int e = tid + u * kNT, r = e / CPR, ch = e % CPR;
    const float v[8] = {x[u][0].x, x[u][0].y, x[u][0].z, x[u][0].w, x[u][1].x, x[u][1].y, x[u][1].z, x[u][1].w};
    uint32_t w[3][4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      float r0 = v[2 * h], r1 = v[2 * h + 1];
#pragma unroll
      for (int pl = 0; pl < 3; ++pl) {
        w[pl][h] = cvt_bf16x2(r0, r1);
        r0 -= bf16_lo(w[pl][h]);
        r1 -= bf16_hi(w[pl][h]);
      }
    }
#pragma unroll
    for (int pl = 0; pl < 3; ++pl)
      *reinterpret_cast<uint4*>(sm + pl * C::PLANE + (ch >> 3) * (kBlkTile * 128) + swz_offset(r, ch & 7, 128)) =
          make_uint4(w[pl][0], w[pl][1], w[pl][2], w[pl][3]);
  }
  fence_proxy_async_smem();  // written by the generic proxy, read by the MMA
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_base;
  bool dead = false;
  if (tid == 0) {
    constexpr uint32_t idesc = idesc_bf16(128, N, false, false);
    const uint32_t a_s = smem_u32(sm), b_s = a_s + C::OFF_Q;
#pragma unroll
    for (int pl = 0; pl < 3; ++pl)
#pragma unroll
      for (int ks = 0; ks < DI / 16; ++ks) {
        const uint64_t da = smem_desc(a_s + pl * C::PLANE + (ks / 4) * kBlkTile * 128 + (ks % 4) * 32, 16, 1024, kSw128);
        const uint64_t db = smem_desc(b_s + (ks / 4) * N * 128 + (ks % 4) * 32, 16, 1024, kSw128);
        mma_bf16(tmem, da, db, idesc, pl + ks > 0);
      }
    mma_commit(bar);
  }
  __syncwarp();
  // warps 0-3 take the first half of the columns, warps 4-7 the second
  const bool ok = tw_wait_warp(bar, 0, dead);
  if (ok) {
    tc_fence_after();
    constexpr int NH = N / 2;
    const int r = (warp & 3) * 32 + lane, n0 = (warp >> 2) * NH;
    float v[NH];
    tmem_load_f32<NH>(tmem + (uint32_t((warp & 3) * 32) << 16) + n0, v);
    uint32_t* out = a.bkeys + b * a.T * a.ldb + kBkeys0 + lo + r;
    if (r < n) {
#pragma unroll
      for (int i = 0; i < NH; ++i)
        if (n0 + i < a.T) out[int64_t(n0 + i) * a.ldb] = score_key(v[i]);
    }
  } else if (tid == 0) {
    mbar_drain(bar, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int DI>
__global__ void __launch_bounds__(kNT) tree_tails_kernel(const TreeArgs a) {
  extern __shared__ __align__(16) float tail_smem[];
  griddep_wait();
  griddep_launch();
  const int64_t b = blockIdx.x;
  if (b == 0 && blockIdx.y == 0 && threadIdx.x < 3) a.counters[threadIdx.x] = 0;
  const int half = threadIdx.x / kNodeNT, i = int(blockIdx.y) * kNodesPerCta + half;
  if (i < a.T) node_tail<DI>(a, b, i, threadIdx.x % kNodeNT, 1 + half, tail_smem + half * a.tail_ld);
}

// Launched dependent on the tails and run beside them: its CTAs start once
// every tail CTA has passed its own wait for the work before it, which is all
// that the scores depend on. That work's writes are in L2 by then; with no wait
// of its own this kernel reads its inputs there (an L1 might hold older lines).
// The wait at the end makes the kernels after this one, which wait for it alone,
// wait for the tails too.
template <int DI, int N>
__global__ void __launch_bounds__(kNT) tree_block_scores_kernel(const TreeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar;
  __shared__ uint32_t tmem_base;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  griddep_launch();
  cached_block_scores<DI, N>(a, blockIdx.x, blockIdx.y, sm, &bar, &tmem_base);
  griddep_wait();
}

// ---------------------------------------------------------------------------
// Token scores inside the kept cached blocks:
//   S^T[key][node] = k_idx[row0 + key] . q_idx[node]
// for every (node, slot) pair that kept a block. An item is up to 128 rows of
// one block with the nodes that kept it.
//
// The keys are what bounds it: 2 * d_idx bytes a row from HBM (or L2) against
// 2 * N * d_idx FLOP, far below the tensor peak at N <= 64.
//
// Warp roles of the persistent kernel: warp 0 TMA producer (key rows and the
// sequence's query rows of an item), warp 1 MMA issuer (+ TMEM owner), warps
// 2-5 epilogue. The accumulator is two deep, so an item's epilogue overlaps
// the next one's MMAs.
// ---------------------------------------------------------------------------
template <int DK, int N>
struct TS {
  static constexpr int KB = DK / 64;              // 128-byte column blocks per row
  static constexpr int A_BYTES = 128 * DK * 2;    // key rows
  static constexpr int B_BYTES = N * DK * 2;      // query rows
  static constexpr int STAGE = A_BYTES + B_BYTES; // a multiple of 1024
  static constexpr int NS = (200 * 1024) / STAGE > 6 ? 6 : (200 * 1024) / STAGE;
  static constexpr int SMEM = NS * STAGE + 1024;
  static constexpr int TMEM_COLS = 2 * N;         // 32, 64 or 128
};

constexpr int kThreads = 192;

template <int DK, int N>
__global__ void __launch_bounds__(kThreads, 1) tree_token_scores_kernel(const __grid_constant__ CUtensorMap kmap,
                                                                        const __grid_constant__ CUtensorMap qmap,
                                                                        const TreeArgs a, int box_rows) {
  using C = TS<DK, N>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full[C::NS], empty[C::NS], tfull[2], tempty[2], done;
  __shared__ uint32_t tmem_base;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int b = 0; b < 2; ++b) { mbar_init(&tfull[b], 1); mbar_init(&tempty[b], 4); }
    mbar_init(&done, 1);
    fence_barrier_init();
  }
  if (warp == 1) { tmem_alloc(&tmem_base, C::TMEM_COLS); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  griddep_wait();
  griddep_launch();
  const int total = a.counters[0];
  const int g = int(gridDim.x);
  bool dead = false;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tmap(&kmap);
      prefetch_tmap(&qmap);
      // the boxes are box_rows x 64 and T x 64 elements; rows of a stage that
      // no box covers hold old data, whose lanes and columns nobody reads
      const uint32_t bytes = uint32_t(C::KB) * 128u * uint32_t(box_rows + a.T);
      uint32_t it = 0;
      int4 next = blockIdx.x < total ? a.items[blockIdx.x] : make_int4(0, 0, 0, 0);
      for (int t = blockIdx.x; t < total && !dead; t += g) {
        const int4 item = next;
        if (t + g < total) next = a.items[t + g];
        const int s = it % C::NS;
        if (!tw_wait(&empty[s], ((it / C::NS) & 1) ^ 1, dead)) break;
        // test hook: CTA 0 never produces its first item, so its consumer's wait runs out
        if (it == 0 && blockIdx.x == 0 && *(volatile int*)&g_tree_inject) { ++it; continue; }
        uint8_t* a_s = sm + s * C::STAGE;
        mbar_arrive_expect_tx(&full[s], bytes);
#pragma unroll
        for (int kb = 0; kb < C::KB; ++kb) {
          tma_load_2d(a_s + kb * 128 * 128, &kmap, &full[s], kb * 64, item.x);
          tma_load_2d(a_s + C::A_BYTES + kb * N * 128, &qmap, &full[s], kb * 64, (item.w >> 3) * a.T);
        }
        ++it;
      }
      for (uint32_t u = (it >= uint32_t(C::NS) ? it - C::NS : 0); u < it; ++u)
        mbar_drain(&full[u % C::NS], (u / C::NS) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16(128, N, false, false);
      uint32_t it = 0;
      for (int t = blockIdx.x; t < total && !dead; t += g) {
        const int s = it % C::NS, tb = it & 1;
        if (!tw_wait(&full[s], (it / C::NS) & 1, dead)) break;
        if (!tw_wait(&tempty[tb], ((it >> 1) & 1) ^ 1, dead)) break;
        tc_fence_after();
        const uint32_t a_s = smem_u32(sm + s * C::STAGE);
        const uint32_t b_s = a_s + C::A_BYTES;
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks) {
          const uint64_t da = smem_desc(a_s + (ks / 4) * 128 * 128 + (ks % 4) * 32, 16, 1024, kSw128);
          const uint64_t db = smem_desc(b_s + (ks / 4) * N * 128 + (ks % 4) * 32, 16, 1024, kSw128);
          mma_bf16(tmem + tb * N, da, db, idesc, ks > 0);
        }
        mma_commit(&empty[s]);
        mma_commit(&tfull[tb]);
        ++it;
      }
      mma_commit(&done);
      mbar_drain(&done, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lane_addr = uint32_t(quad * 32) << 16;
    uint32_t it = 0;
    // an item is fetched two ahead, its pairs one ahead
    auto item_of = [&](int tt) { return tt < total ? a.items[tt] : make_int4(0, 0, 0, 0); };
    auto pair_of = [&](const int4& d, int e) { return e < (d.z & 0xffff) ? a.pairs[d.y + e] : 0u; };
    int4 cur = item_of(blockIdx.x), next = item_of(blockIdx.x + g);
    uint32_t p0 = pair_of(cur, lane), p1 = pair_of(cur, lane + 32);
    for (int t = blockIdx.x; t < total && !dead; t += g) {
      const int4 item = cur;
      const uint32_t q0 = p0, q1 = p1;
      cur = next;
      next = item_of(t + 2 * g);
      p0 = pair_of(cur, lane);
      p1 = pair_of(cur, lane + 32);
      const int tb = it & 1, cnt = item.z & 0xffff;
      if (!tw_wait_warp(&tfull[tb], (it >> 1) & 1, dead)) break;
      tc_fence_after();
      const bool mine = r < (item.z >> 16);
      uint32_t* out = a.tkeys + int64_t(item.w >> 3) * a.T * a.m * a.B + 128 * (item.w & 7) + r;
      // a node's scores are one accumulator column: four pairs' at a time
      for (int e0 = 0; e0 < cnt; e0 += 4) {
        uint32_t v[4], pr[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int e = min(e0 + u, cnt - 1);
          pr[u] = __shfl_sync(kFull, e < 32 ? q0 : q1, e & 31);
          tmem_ld1(tmem + lane_addr + tb * N + (pr[u] >> 16), v[u]);
        }
        tmem_wait_ld();
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (mine && e0 + u < cnt)
            out[(int64_t(pr[u] >> 16) * a.m + (pr[u] & 0xffffu)) * a.B] = score_key(__uint_as_float(v[u]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[tb]);
      ++it;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int DK, int N>
bool launch_n(const CUtensorMap& km, const CUtensorMap& qm, const TreeArgs& a, int box_rows, int grid,
              cudaStream_t s) {
  using C = TS<DK, N>;
  auto kern = tree_token_scores_kernel<DK, N>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess) return false;
  count_launches(1);
  launch_kernel(true, kern, unsigned(grid), kThreads, C::SMEM, s, km, qm, a, box_rows);
  return true;
}

template <int DI, int N>
bool launch_bs(const TreeArgs& a, int batch, cudaStream_t s) {
  const int smem_t = kNodesPerCta * a.tail_ld * 4, smem_b = BS<DI, N>::SMEM;
  const int tiles = int((a.capacity / a.B + kBlkTile - 1) / kBlkTile);
  auto blocks = tree_block_scores_kernel<DI, N>;
  if (cudaFuncSetAttribute(blocks, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_b) != cudaSuccess) return false;
  count_launches(2);
  launch_kernel(true, tree_tails_kernel<DI>, dim3(unsigned(batch), unsigned((a.T + kNodesPerCta - 1) / kNodesPerCta)),
                kNT, size_t(smem_t), s, a);
  launch_kernel(true, blocks, dim3(unsigned(batch), unsigned(tiles)), kNT, size_t(smem_b), s, a);
  return true;
}

}  // namespace

bool launch_tree_block_scores(const TreeArgs& a, int batch, int d_idx, cudaStream_t s) {
  if (d_idx == 128)
    return a.T <= 16 ? launch_bs<128, 16>(a, batch, s)
           : a.T <= 32 ? launch_bs<128, 32>(a, batch, s) : launch_bs<128, 64>(a, batch, s);
  return a.T <= 16 ? launch_bs<64, 16>(a, batch, s)
         : a.T <= 32 ? launch_bs<64, 32>(a, batch, s) : launch_bs<64, 64>(a, batch, s);
}

bool launch_tree_token_scores(const TreeArgs& a, int batch, int d_idx, int64_t max_items, cudaStream_t s) {
  const int box_rows = a.B < 128 ? a.B : 128;
  CUtensorMap km, qm;
  if (!make_tmap_2d(&km, a.k_idx_cache, uint64_t(batch) * a.capacity, uint64_t(d_idx), box_rows) ||
      !make_tmap_2d(&qm, a.q_new, uint64_t(batch) * a.T, uint64_t(d_idx), a.T))
    return false;
  const int grid = int(max_items < num_sms() ? max_items : num_sms());
  if (d_idx == 128) {
    if (a.T <= 16) return launch_n<128, 16>(km, qm, a, box_rows, grid, s);
    if (a.T <= 32) return launch_n<128, 32>(km, qm, a, box_rows, grid, s);
    return launch_n<128, 64>(km, qm, a, box_rows, grid, s);
  }
  if (a.T <= 16) return launch_n<64, 16>(km, qm, a, box_rows, grid, s);
  if (a.T <= 32) return launch_n<64, 32>(km, qm, a, box_rows, grid, s);
  return launch_n<64, 64>(km, qm, a, box_rows, grid, s);
}

int tree_wait_flag(bool reset) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_tree_err, sizeof v) != cudaSuccess) return -1;
  if (reset && v) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_tree_err, &zero, sizeof zero) != cudaSuccess) return -1;
  }
  return v != 0;
}

bool tree_set_inject(bool on) {
  const int v = on ? 1 : 0;
  return cudaMemcpyToSymbol(g_tree_inject, &v, sizeof v) == cudaSuccess;
}

}  // namespace hsa
