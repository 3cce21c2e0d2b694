// Token scores of a drafted tree inside the kept cached blocks, on tcgen05:
//   S^T[key][node] = k_idx[row0 + key] . q_idx[node]
// for every (node, slot) pair that kept a block. An item is up to 128 rows of
// one block with the nodes that kept it. The keys are the MMA's M dimension
// and all of a sequence's nodes its N (16, 32 or 64 columns), so a block is
// read once whatever number of nodes kept it, nothing is gathered, and an
// accumulator column is one node's scores of 128 consecutive keys: the 128
// epilogue threads (TMEM lane = key) write it as 512 contiguous bytes.
//
// The keys are what bounds it: 2 * d_idx bytes a row from HBM (or L2) against
// 2 * N * d_idx FLOP, far below the tensor peak at N <= 64.
//
// Warp roles of the persistent kernel: warp 0 TMA producer (key rows and the
// sequence's query rows of an item), warp 1 MMA issuer (+ TMEM owner), warps
// 2-5 epilogue. The accumulator is two deep, so an item's epilogue overlaps
// the next one's MMAs. Every wait is bounded.
#include "kernels.cuh"
#include "tc.cuh"

namespace hsa {

__device__ int g_tree_err;
__device__ int g_tree_inject;  // test hook: short waits and one item never produced

namespace {

using namespace tc;

constexpr long long kInjectWaitCycles = 1ll << 21;  // about a millisecond

HSA_DEV bool tw_wait(uint64_t* bar, uint32_t parity, bool& dead) {
  if (dead) return false;
  if (mbar_try_wait(bar, parity)) return true;
  const long long lim = *(volatile int*)&g_tree_inject ? kInjectWaitCycles : kWaitCycles;
  if (mbar_wait_bounded(bar, parity, &g_tree_err, lim)) return true;
  dead = true;
  return false;
}
HSA_DEV bool tw_wait_warp(uint64_t* bar, uint32_t parity, bool& dead) {
  bool ok = false;
  if ((threadIdx.x & 31) == 0) ok = tw_wait(bar, parity, dead);
  ok = __shfl_sync(kFull, ok ? 1 : 0, 0) != 0;
  __syncwarp();
  dead = !ok;
  return ok;
}

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
      bool d2 = false;  // drain armed loads before the CTA may exit
      for (uint32_t u = (it >= uint32_t(C::NS) ? it - C::NS : 0); u < it; ++u)
        tw_wait(&full[u % C::NS], (u / C::NS) & 1, d2);
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
      bool d2 = false;
      tw_wait(&done, 0, d2);
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

}  // namespace

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
