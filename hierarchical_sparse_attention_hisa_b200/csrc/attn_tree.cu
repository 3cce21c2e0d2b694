// Attention of the drafted trees' nodes over their kept cache rows, on tcgen05:
// softmax(q K^T * scale) V with one list of kept rows per node, shared by its
// H heads. A launch takes up to 64 heads (HP = 16, 32 or 64 MMA columns).
//
// The kept rows are the MMA's M dimension, 128 at a time:
//   S^T[key][h] = Ktile[key][:] . Q[h][:]      (A = gathered K rows, K-major)
//   O^T[c][h]  += Vtile[key][c] . P^T[key][h]  (A = gathered V rows read MN-major)
// so every MMA has 128 rows whatever H is. With d = 64 the upper 64 rows of V^T
// are read from a zero tile.
//
// Work comes as a list per CTA (one CTA per SM) of items: a run of 128-row
// tiles of one node. A node that lies in one CTA is written whole, one that is
// cut between CTAs as parts for tree_combine_kernel. Ragged trees leave too few
// nodes for a node per CTA: 253 nodes of 16 tiles took 4 rounds and 133 us that
// way, equal shares of 28 tiles 64 us.
//
// A tile costs 768 cycles of MMA (N = 64), 512 of exponentials and 1024 of
// gather (64 KB at 64 B a cycle), but a chain of hand-offs: gather, S, softmax,
// P, PV. Three things keep tiles overlapped when a CTA has few of them:
//   - K and V rows come through separate producer warps, so a V stage that
//     waits for its PV does not hold up the next K, and V has three stages;
//   - S runs up to four tiles ahead of the softmax (four TMEM buffers);
//   - two softmax groups of eight warps take alternate tiles, one in its
//     exponentials while the other waits for its hand-offs.
//
// Softmax: the maximum of an item's first tile is the reference of all its
// tiles, no later tile looks for another. That is exact to rounding as long as
// nothing leaves the range of fp32 and bf16 exponents: weights may grow to 2^90
// times the first tile's largest (62 nats above its maximum), and their products
// with V to 2^119 (a row's 64 parts at that size still add up below 2^128). Where
// a head's sum passes 2^90, is not positive or not a number, or a value of its O
// passes 2^119 or is not a number, its group of eight heads is flagged, and taken
// again by tree_combine_kernel with a running maximum, at some 20 times the cost. P is
// rounded to bf16 for the second MMA (2^-9 of each weight, independent from key
// to key), everything else is fp32, O rounded once.
//
// Every mbarrier wait is bounded. A thread whose wait runs out goes on through
// its loops without waiting (and without storing), so that named barriers and
// arrivals stay in step and the CTA ends.
#include "kernels.cuh"
#include "tc.cuh"

namespace hsa {

__device__ int g_tattn_err;     // set when a bounded wait gives up
__device__ int g_tattn_inject;  // test hook: short waits and one lost arrival

namespace {

using namespace tc;

constexpr int TILE = 128;
constexpr long long kInjectWaitCycles = 1ll << 21;  // about a millisecond
constexpr int kSB = 4, kOB = 2;                     // S and O buffers in TMEM
constexpr float kMostWeight = 1.2379400392853803e27f;  // 2^90
constexpr uint32_t kMostOut = (127u + 119u) << 23;     // 2^119, as the bits of an fp32
constexpr int kIB = 4;                              // per-item scratch buffers
constexpr int kGroups = 2, kGroupWarps = 8;

template <int HP, int DH>
struct TA {
  // K and V stages: a K stage is free after its S, which runs ahead, a V stage only after its PV
  static constexpr int NSK = DH == 128 && HP >= 32 ? 2 : 3, NSV = 3;
  static constexpr int NP = 2;                               // P buffers
  static constexpr int NQ = HP == 64 && DH == 128 ? 1 : 2;   // Q buffers
  static constexpr int HPT = HP / 2;                // heads per softmax thread
  static constexpr int KV_BYTES = TILE * DH * 2;
  static constexpr int Q_BYTES = HP * DH * 2;
  static constexpr int P_ROW = HP * 2;
  static constexpr int P_BYTES = TILE * P_ROW;
  static constexpr int Z_BYTES = DH == 64 ? TILE * 128 : 0;
  static constexpr int CPR = DH / 8, RPI = 32 / CPR;  // 16-byte chunks per row, rows per warp-wide copy
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + NSK * KV_BYTES;
  static constexpr int OFF_Q = OFF_V + NSV * KV_BYTES;
  static constexpr int OFF_P = OFF_Q + NQ * Q_BYTES;
  static constexpr int OFF_Z = OFF_P + NP * P_BYTES;
  static constexpr int SMEM = OFF_Z + Z_BYTES + 1024;  // + alignment slack
  static constexpr int TMEM_COLS = (kSB + kOB) * HP > 256 ? 512 : (kSB + kOB) * HP > 128 ? 256 : 128;
  static constexpr uint32_t P_SWZ = P_ROW == 128 ? kSw128 : P_ROW == 64 ? kSw64 : kSw32;
  static constexpr int NWARPS = 4 + 2 + kGroups * kGroupWarps + 1;
};

struct Bars {
  uint64_t kfull[3], kempty[3], vfull[3], vempty[3];
  uint64_t qfull[2], qempty[2], sfull[kSB], sempty[kSB], pfull[2], pempty[2], ofull[kOB], oempty[kOB];
  uint64_t mfull[kIB], lfull[kIB];
  uint64_t done;
};

struct Args {
  const uint16_t *Q, *K, *V;
  const int32_t* idx;
  int T, k, H, h0, nh;
  float scale_log2;
  int64_t capacity;
  const int4* items;
  const int* cta_items;
  uint16_t* O;
  float *Opart, *mpart, *lpart;
  int *flags, *flagged, *n_flagged;
};

// A group of eight heads of a row is to be taken again; a row's first group lists it.
HSA_DEV void flag_heads(const Args& a, int row, int head) {
  if (atomicOr(a.flags + row, 1 << (head >> 3)) == 0) a.flagged[atomicAdd(a.n_flagged, 1)] = row;
}

// Bounded wait. A failed probe goes straight back to the barrier: the limit,
// the error flag and the test hook are global or slow to read, and a look at
// them between two probes (some 700 cycles) is a hand-off's latency several
// times over. So they are read once in 64 probes.
HSA_DEV bool wait_bar(uint64_t* bar, uint32_t parity, bool& dead) {
  if (dead) return false;
  long long t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*(volatile int*)&g_tattn_err) break;
      const long long t = clock64();
      if (t0 == 0) t0 = t;
      if (t - t0 > (*(volatile int*)&g_tattn_inject ? kInjectWaitCycles : kWaitCycles)) {
        atomicExch(&g_tattn_err, 1);
        break;
      }
    }
  }
  dead = true;
  return false;
}
// Every lane polls. (With lane 0 polling for the others, which wait for its
// answer at a shuffle, a warp that had waited long was then held up for about as
// long again: 270 us where this form takes 103, 64 tiles on every SM.)
HSA_DEV void wait_warp(uint64_t* bar, uint32_t parity, bool& dead) {
  const bool ok = wait_bar(bar, parity, dead);
  dead = !__all_sync(kFull, ok);
}

// Sum (or maximum) of v[0..N) over the 32 lanes by halving exchanges: lane l ends
// with that of element l / (32 / N) (N <= 32, a power of two).
template <int N, bool MAX = false>
HSA_DEV float lanes_sum(float (&v)[N]) {
  auto join = [](float x, float y) { return MAX ? fmaxf(x, y) : x + y; };
  const int lane = threadIdx.x & 31;
  int n = N;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    if (n > 1) {
      const bool hi = lane & o;
      n /= 2;
#pragma unroll
      for (int i = 0; i < N / 2; ++i)
        if (i < n) {
          const float send = hi ? v[i] : v[i + n], keep = hi ? v[i + n] : v[i];
          v[i] = join(keep, __shfl_xor_sync(kFull, send, o));
        }
    } else {
      v[0] = join(v[0], __shfl_xor_sync(kFull, v[0], o));
    }
  }
  return v[0];
}

struct Item { int row, t0, nt, kept, part; };
HSA_DEV Item read_item(const int4* items, int wi) {
  const int4 v = __ldg(items + wi);
  return {v.x, v.y & 0xff, (v.y >> 8) & 0xff, v.y >> 16, v.z};
}

// One side's rows (K or V), by two warps: warp `pw` the rows 64 pw .. 64 pw + 63
// of every tile. A row past the node's list repeats the list's last one: its
// weight is zero, and zero times a value that the node does not keep might not be.
template <int HP, int DH, bool IS_K>
HSA_DEV void produce(const Args& a, uint8_t* sm, Bars& bars, int pw, int w0, int w1) {
  using C = TA<HP, DH>;
  const int lane = threadIdx.x & 31, rsub = lane / C::CPR, cpk = lane % C::CPR;
  const uint32_t dbase = (cpk >> 3) * (TILE * 128) + (64 * pw + rsub) * 128;
  const bool inject = IS_K && *(volatile int*)&g_tattn_inject != 0;
  uint64_t* full = IS_K ? bars.kfull : bars.vfull;
  uint64_t* empty = IS_K ? bars.kempty : bars.vempty;
  constexpr int NS = IS_K ? C::NSK : C::NSV;
  bool dead = false;
  uint32_t g = 0;
  Item it = w0 < w1 ? read_item(a.items, w0) : Item{};
  auto rows_of = [&](const Item& x, int i, int (&j)[2]) {
    const int32_t* row = a.idx + int64_t(x.row) * a.k;
#pragma unroll
    for (int u = 0; u < 2; ++u) j[u] = __ldg(row + min((x.t0 + i) * TILE + 64 * pw + 32 * u + lane, x.kept - 1));
  };
  auto in_cache = [&](int j) { return j >= 0 && j < a.capacity ? j : 0; };
  int jn[2] = {0, 0};
  if (w0 < w1) rows_of(it, 0, jn);
  for (int wi = w0; wi < w1; ++wi) {
    const Item cur = it;
    if (wi + 1 < w1) it = read_item(a.items, wi + 1);
    const uint4* src = reinterpret_cast<const uint4*>((IS_K ? a.K : a.V) + int64_t(cur.row / a.T) * a.capacity * DH) + cpk;
    for (int i = 0; i < cur.nt; ++i, ++g) {
      const int s = g % NS, j0 = in_cache(jn[0]), j1 = in_cache(jn[1]);  // (loaded a tile ago)
      // the next tile's rows, this item's or the next one's
      if (i + 1 < cur.nt) rows_of(cur, i + 1, jn);
      else if (wi + 1 < w1) rows_of(it, 0, jn);
      wait_warp(&empty[s], ((g / NS) & 1) ^ 1, dead);
      const uint32_t dst = smem_u32(sm + (IS_K ? C::OFF_K : C::OFF_V) + s * C::KV_BYTES) + dbase;
#pragma unroll
      for (int u = 0; u < 64 / C::RPI; ++u) {
        const int rr = C::RPI * u + rsub;  // 0 .. 63
        const int j = __shfl_sync(kFull, C::RPI * u < 32 ? j0 : j1, rr & 31);
        cp_async16(dst + u * (C::RPI * 128) + ((uint32_t((cpk & 7) ^ (rr & 7))) << 4), src + int64_t(j) * C::CPR);
      }
      // test hook: one K arrival on the first tile of CTA 0 is lost
      if (!(inject && blockIdx.x == 0 && g == 0 && pw == 0 && lane == 0)) cp_async_arrive(&full[s]);
    }
  }
  cp_async_wait_all();  // every copy has landed before the CTA may exit
}

// The items' Q: HP head rows each (rows past the launch's nh heads: zeros). A
// warp of its own: in front of a K warp's first rows it cost them 0.9 us.
template <int HP, int DH>
HSA_DEV void produce_q(const Args& a, uint8_t* sm, Bars& bars, int w0, int w1) {
  using C = TA<HP, DH>;
  const int lane = threadIdx.x & 31;
  bool dead = false;
  uint32_t qn = 0;
  for (int wi = w0; wi < w1; ++wi, ++qn) {
    const int row = read_item(a.items, wi).row, qb = qn % C::NQ;
    const uint32_t qt = smem_u32(sm + C::OFF_Q + qb * C::Q_BYTES);
    const uint4* src = reinterpret_cast<const uint4*>(a.Q) + (int64_t(row) * a.H + a.h0) * C::CPR;
    wait_warp(&bars.qempty[qb], ((qn / C::NQ) & 1) ^ 1, dead);
#pragma unroll 8
    for (int e = lane; e < HP * C::CPR; e += 32) {
      const int h = e / C::CPR, c = e % C::CPR;
      const bool live = h < a.nh;
      cp_async16_zfill(qt + (c >> 3) * (HP * 128) + swz_offset(h, c & 7, 128), live ? src + e : src, live);
    }
    cp_async_arrive(&bars.qfull[qb]);
  }
  cp_async_wait_all();
}

template <int HP, int DH>
__global__ void __launch_bounds__(32 * TA<HP, DH>::NWARPS, 1) tree_attn_kernel(const Args a) {
  using C = TA<HP, DH>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) Bars bars;
  __shared__ uint32_t tmem_base;
  __shared__ float red[kGroups][4][HP];            // a group's per-warp maxima of an item's first tile
  __shared__ __align__(16) float neg_m[kIB][HP];   // the item's negated reference maxima (log2 units)
  __shared__ float lred[kIB][kGroups][4][HP];      // per-warp row sums
  __shared__ __align__(16) float linv[kGroups][HP];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 3; ++s) {
      mbar_init(&bars.kfull[s], 64); mbar_init(&bars.kempty[s], 1);
      mbar_init(&bars.vfull[s], 64); mbar_init(&bars.vempty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars.qfull[b], 32); mbar_init(&bars.qempty[b], 1);
      mbar_init(&bars.pfull[b], kGroupWarps); mbar_init(&bars.pempty[b], 1);
    }
    for (int b = 0; b < kSB; ++b) { mbar_init(&bars.sfull[b], 1); mbar_init(&bars.sempty[b], kGroupWarps); }
    for (int b = 0; b < kOB; ++b) { mbar_init(&bars.ofull[b], 1); mbar_init(&bars.oempty[b], kGroupWarps); }
    for (int b = 0; b < kIB; ++b) {
      mbar_init(&bars.mfull[b], kGroupWarps);
      mbar_init(&bars.lfull[b], kGroups * kGroupWarps);
    }
    mbar_init(&bars.done, 2);
    fence_barrier_init();
  }
  if (C::Z_BYTES > 0) {
    for (int e = threadIdx.x; e < C::Z_BYTES / 16; e += blockDim.x)
      reinterpret_cast<uint4*>(sm + C::OFF_Z)[e] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  if (warp == 4) { tmem_alloc(&tmem_base, C::TMEM_COLS); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  // the set-up above touches no global memory: it overlaps the previous kernel
  griddep_wait();
  griddep_launch();
  const int w0 = a.cta_items[blockIdx.x], w1 = a.cta_items[blockIdx.x + 1];
  bool dead = false;

  if (warp < 2) {
    produce<HP, DH, true>(a, sm, bars, warp, w0, w1);
  } else if (warp < 4) {
    produce<HP, DH, false>(a, sm, bars, warp - 2, w0, w1);
  } else if (warp == 4) {
    // ------------------------------------------------------------ S issuer
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_bf16(128, HP, false, false);
      uint32_t g = 0, qn = 0;
      for (int wi = w0; wi < w1; ++wi, ++qn) {
        const int nt = read_item(a.items, wi).nt, qb = qn % C::NQ;
        wait_bar(&bars.qfull[qb], (qn / C::NQ) & 1, dead);
        const uint64_t qd = smem_desc(smem_u32(sm + C::OFF_Q + qb * C::Q_BYTES), 16, 1024, kSw128);
        const uint32_t qlo = uint32_t(qd), qhi = uint32_t(qd >> 32);
        for (int i = 0; i < nt; ++i, ++g) {
          const int s = g % C::NSK, sb = g % kSB;
          wait_bar(&bars.sempty[sb], ((g / kSB) & 1) ^ 1, dead);
          wait_bar(&bars.kfull[s], (g / C::NSK) & 1, dead);
          fence_proxy_async_smem();  // K and Q rows landed by cp.async, read by the MMA
          tc_fence_after();
          const uint64_t kd = smem_desc(smem_u32(sm + C::OFF_K + s * C::KV_BYTES), 16, 1024, kSw128);
          const uint32_t klo = uint32_t(kd), khi = uint32_t(kd >> 32);
#pragma unroll
          for (int ks = 0; ks < DH / 16; ++ks)
            mma_bf16_split(tmem + sb * HP, klo + (((ks / 4) * TILE * 128 + (ks % 4) * 32) >> 4), khi,
                           qlo + (((ks / 4) * HP * 128 + (ks % 4) * 32) >> 4), qhi, id_s, ks > 0 ? 1u : 0u);
          mma_commit(&bars.sfull[sb]);
          mma_commit(&bars.kempty[s]);
          if (i == nt - 1) mma_commit(&bars.qempty[qb]);
        }
      }
      mma_commit(&bars.done);
      mbar_drain(&bars.done, 0);
    }
    __syncwarp();
  } else if (warp == 5) {
    // ------------------------------------------------------------ PV issuer
    if (lane == 0) {
      constexpr uint32_t id_o = idesc_bf16(128, HP, true, true);
      uint32_t g = 0, qn = 0;
      for (int wi = w0; wi < w1; ++wi, ++qn) {
        const int nt = read_item(a.items, wi).nt, ob = qn % kOB;
        wait_bar(&bars.oempty[ob], ((qn / kOB) & 1) ^ 1, dead);
        for (int i = 0; i < nt; ++i, ++g) {
          const int s = g % C::NSV, pb = g % C::NP;
          wait_bar(&bars.vfull[s], (g / C::NSV) & 1, dead);
          wait_bar(&bars.pfull[pb], (g / C::NP) & 1, dead);
          fence_proxy_async_smem();  // the V rows landed by cp.async, read by the MMA
          tc_fence_after();
          const uint32_t vs = smem_u32(sm + C::OFF_V + s * C::KV_BYTES);
          // the second 64 rows of V^T: the tile's upper half, or the zero tile when d = 64
          const uint32_t lbo = DH == 128 ? TILE * 128 : smem_u32(sm + C::OFF_Z) - vs;
          const uint64_t a0 = smem_desc(vs, lbo, 1024, kSw128);
          const uint64_t b0 = smem_desc(smem_u32(sm + C::OFF_P + pb * C::P_BYTES), 16384, 8 * C::P_ROW, C::P_SWZ);
          const uint32_t d = tmem + (kSB + ob) * HP;
          const uint32_t alo = uint32_t(a0), ahi = uint32_t(a0 >> 32), blo = uint32_t(b0), bhi = uint32_t(b0 >> 32);
#pragma unroll
          for (int ks = 0; ks < TILE / 16; ++ks)
            mma_bf16_split(d, alo + ((ks * 2048) >> 4), ahi, blo + ((ks * 16 * C::P_ROW) >> 4), bhi, id_o,
                           (i == 0 && ks == 0) ? 0u : 1u);
          mma_commit(&bars.pempty[pb]);
          mma_commit(&bars.vempty[s]);
          if (i == nt - 1) mma_commit(&bars.ofull[ob]);
        }
      }
      mma_commit(&bars.done);
      mbar_drain(&bars.done, 0);
    }
    __syncwarp();
  } else if (warp == C::NWARPS - 1) {
    produce_q<HP, DH>(a, sm, bars, w0, w1);
  } else {
    // ------------------------------------------------------------ softmax
    constexpr int HPT = C::HPT, CW = HPT < 16 ? HPT : 16;  // heads per thread, columns per TMEM load
    const int sg = (warp - 6) / kGroupWarps, half = ((warp - 6) % kGroupWarps) / 4;
    const int quad = warp & 3;          // TMEM lane quadrant this warp may access
    const int r = quad * 32 + lane;     // key row of the tile / dim row of O^T
    const int h0 = half * HPT;          // first head of this thread
    const uint32_t lane_addr = uint32_t(quad * 32) << 16;
    const int half_bar = 1 + 2 * sg + half, group_bar = 5 + sg;  // 128 and 256 threads
    auto load_cols = [&](uint32_t col, float (&x)[CW]) {
      uint32_t w[CW];
      if constexpr (CW == 16) tmem_ld16(tmem + lane_addr + col, w);
      else tmem_ld8(tmem + lane_addr + col, w);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < CW; ++e) x[e] = __uint_as_float(w[e]);
    };
    uint32_t base = 0, qn = 0;  // tiles and items before this one
    Item it = w0 < w1 ? read_item(a.items, w0) : Item{};
    for (int wi = w0; wi < w1; ++wi, ++qn) {
      const Item cur = it;
      if (wi + 1 < w1) it = read_item(a.items, wi + 1);
      const int ib = qn % kIB;
      const uint32_t ib_phase = (qn / kIB) & 1;
      float lp[HPT];
#pragma unroll
      for (int h = 0; h < HPT; ++h) lp[h] = 0.f;
      bool have_m = false;
      for (int i = int((base ^ uint32_t(sg)) & 1u); i < cur.nt; i += 2) {
        const uint32_t g = base + i;
        const int sb = g % kSB, pb = g % C::NP;
        const bool valid = (cur.t0 + i) * TILE + r < cur.kept;
        wait_warp(&bars.sfull[sb], (g / kSB) & 1, dead);
        tc_fence_after();
        if (i == 0) {
          // the reference maxima: over the tile's rows, each thread's own heads
#pragma unroll
          for (int c = 0; c < HPT; c += CW) {
            float x[CW];
            load_cols(sb * HP + h0 + c, x);
#pragma unroll
            for (int e = 0; e < CW; ++e) x[e] = valid ? x[e] * a.scale_log2 : -INFINITY;
            const float m = lanes_sum<CW, true>(x);
            if (lane % (32 / CW) == 0) red[sg][quad][h0 + c + lane / (32 / CW)] = m;
          }
          bar_sync(half_bar, 128);
          if (quad == 0 && lane < HPT) {
            const int h = h0 + lane;
            const float m = fmaxf(fmaxf(red[sg][0][h], red[sg][1][h]), fmaxf(red[sg][2][h], red[sg][3][h]));
            neg_m[ib][h] = fabsf(m) < INFINITY ? -m : 0.f;  // (no finite maximum: the row will be flagged)
          }
          bar_sync(half_bar, 128);
          if (lane == 0) mbar_arrive(&bars.mfull[ib]);
        } else if (!have_m) {
          wait_warp(&bars.mfull[ib], ib_phase, dead);
        }
        have_m = true;
        uint32_t w[HPT / 2];
#pragma unroll
        for (int c = 0; c < HPT; c += CW) {
          float x[CW];
          load_cols(sb * HP + h0 + c, x);
          if (c + CW == HPT) {  // the buffer has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.sempty[sb]);
          }
          const float4* nm = reinterpret_cast<const float4*>(&neg_m[ib][h0 + c]);
#pragma unroll
          for (int e = 0; e < CW; e += 4) {
            const float4 m = nm[e / 4];
            x[e] = ex2(__fmaf_rn(x[e], a.scale_log2, m.x));
            x[e + 1] = ex2(__fmaf_rn(x[e + 1], a.scale_log2, m.y));
            x[e + 2] = ex2(__fmaf_rn(x[e + 2], a.scale_log2, m.z));
            x[e + 3] = ex2(__fmaf_rn(x[e + 3], a.scale_log2, m.w));
          }
          if (!valid) {
#pragma unroll
            for (int e = 0; e < CW; ++e) x[e] = 0.f;
          }
#pragma unroll
          for (int e = 0; e < CW; e += 2) {
            lp[c + e] += x[e];
            lp[c + e + 1] += x[e + 1];
            w[(c + e) / 2] = cvt_bf16x2(x[e], x[e + 1]);
          }
        }
        wait_warp(&bars.pempty[pb], ((g / C::NP) & 1) ^ 1, dead);
        uint8_t* prow = sm + C::OFF_P + pb * C::P_BYTES;
#pragma unroll
        for (int c = 0; c < HPT / 8; ++c)
          *reinterpret_cast<uint4*>(prow + swz_offset(r, h0 / 8 + c, C::P_ROW)) =
              make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.pfull[pb]);
      }
      // this group's row sums of the item
      if (have_m) {
        const float l = lanes_sum<HPT>(lp);
        if (lane % (32 / HPT) == 0) lred[ib][sg][quad][h0 + lane / (32 / HPT)] = l;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.lfull[ib]);
      const uint32_t last = base + cur.nt - 1;
      base += cur.nt;
      if (int(last & 1u) != sg) continue;
      // ---- epilogue, by the group of the last tile: O^T of the node's heads, normalised, or a part
      const int ob = qn % kOB;
      wait_warp(&bars.lfull[ib], ib_phase, dead);
      if (half == 0 && r < HP) {
        float l = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          l += lred[ib][sg][q][r];
          if (cur.nt > 1) l += lred[ib][sg ^ 1][q][r];
        }
        linv[sg][r] = l > 0.f ? 1.f / l : 0.f;
        if (r < a.nh && !dead) {
          if (!(l > 0.f && l <= kMostWeight)) flag_heads(a, cur.row, a.h0 + r);
          if (cur.part >= 0) {
            a.mpart[int64_t(cur.part) * a.H + a.h0 + r] = -neg_m[ib][r];
            a.lpart[int64_t(cur.part) * a.H + a.h0 + r] = l;
          }
        }
      }
      bar_sync(group_bar, 32 * kGroupWarps);
      wait_warp(&bars.ofull[ob], (qn / kOB) & 1, dead);
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < HPT; c += CW) {
        float x[CW];
        load_cols((kSB + ob) * HP + h0 + c, x);
        if (c + CW == HPT) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.oempty[ob]);
        }
        if (r < DH && !dead) {
#pragma unroll
          for (int e = 0; e < CW; e += 8) {  // (as integers, magnitudes order with NaN above all)
            uint32_t most = 0;
#pragma unroll
            for (int z = 0; z < 8; ++z) most = max(most, __float_as_uint(x[e + z]) & 0x7fffffffu);
            if (most > kMostOut && h0 + c + e < a.nh) flag_heads(a, cur.row, a.h0 + h0 + c + e);
          }
          if (cur.part < 0) {
            uint16_t* o = a.O + (int64_t(cur.row) * a.H + a.h0 + h0 + c) * DH + r;
#pragma unroll
            for (int e = 0; e < CW; ++e)
              if (h0 + c + e < a.nh) o[e * DH] = cvt_bf16(x[e] * linv[sg][h0 + c + e]);
          } else {
            float* o = a.Opart + (int64_t(cur.part) * a.H + a.h0 + h0 + c) * DH + r;
#pragma unroll
            for (int e = 0; e < CW; ++e)
              if (h0 + c + e < a.nh) o[e * DH] = x[e];
          }
        }
      }
      bar_sync(group_bar, 32 * kGroupWarps);  // linv is free again
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int HP, int DH>
bool launch_hp(const Args& a, cudaStream_t s) {
  using C = TA<HP, DH>;
  auto kern = tree_attn_kernel<HP, DH>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess) return false;
  count_launches(1);
  launch_kernel(true, kern, kTreeAttnCtas, 32 * C::NWARPS, C::SMEM, s, a);
  return true;
}

template <int DH>
bool launch_d(const Args& a, cudaStream_t s) {
  return a.nh <= 16 ? launch_hp<16, DH>(a, s) : a.nh <= 32 ? launch_hp<32, DH>(a, s) : launch_hp<64, DH>(a, s);
}

}  // namespace

bool launch_tree_attn(const TreeArgs& t, const void* Q, const int32_t* idx, float scale, float* Opart, float* mpart,
                      float* lpart, cudaStream_t s) {
  Args a{};
  a.Q = static_cast<const uint16_t*>(Q);
  a.K = t.K_cache; a.V = t.V_cache;
  a.idx = idx; a.T = t.T; a.k = t.k; a.H = t.H;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.capacity = t.capacity;
  a.items = t.attn_items; a.cta_items = t.cta_items;
  a.O = t.O;
  a.Opart = Opart; a.mpart = mpart; a.lpart = lpart;
  a.flags = t.flags; a.flagged = t.flagged; a.n_flagged = t.counters + 2;
  for (int h0 = 0; h0 < t.H; h0 += 64) {
    a.h0 = h0;
    a.nh = t.H - h0 < 64 ? t.H - h0 : 64;
    if (!(t.d == 128 ? launch_d<128>(a, s) : launch_d<64>(a, s))) return false;
  }
  return true;
}

int tree_attn_wait_flag(bool reset) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_tattn_err, sizeof v) != cudaSuccess) return -1;
  if (reset && v) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_tattn_err, &zero, sizeof zero) != cudaSuccess) return -1;
  }
  return v != 0;
}

bool tree_attn_set_inject(bool on) {
  const int v = on ? 1 : 0;
  return cudaMemcpyToSymbol(g_tattn_inject, &v, sizeof v) == cudaSuccess;
}

}  // namespace hsa
