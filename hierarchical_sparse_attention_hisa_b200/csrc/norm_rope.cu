// Per-head RMS norm of queries and keys with the position rotation in the
// same pass: what turns a layer's projections (its own and its indexer's)
// into the Q / K (q_idx / k_idx) of the selection and the attention.
//
// For a row x of d values at position t:
//   y = x * w / sqrt(mean(x^2) + eps)
//   pairs (a, b) of the first `rot` values, (i, i + rot/2) or (2i, 2i+1):
//   (a cos u - b sin u, b cos u + a sin u),  u = t * inv_freq[i]
// in fp32, rounded once to bf16. The angle is taken in 64 bits: an fp32
// product t * inv_freq is off by up to t * 2^-24 turns' worth of radians,
// 0.06 at position 2^20, while the fp64 product keeps 2^-53 of it; reduced to
// (-1/2, 1/2] turns it fits fp32 without loss that a bf16 result could show.
//
// One read and one write of every value bound it (HBM). A row is d/16 lanes of
// two 16-byte chunks, chosen so that both values of every pair are the same
// lane's: the split layout's lane holds chunk l and its partner l + rot/16, so
// the rotation exchanges nothing and only the sum of squares crosses lanes.
// A lane keeps its eight pairs' coefficients w cos u, w sin u in registers over
// all heads of a token.
#include <algorithm>

#include "kernels.cuh"

namespace hsa {
namespace {

constexpr int kNT = 128;

struct NormRopeArgs {
  const uint16_t *Q, *K, *qw, *kw;
  int64_t q_stride, k_stride;
  const float* inv_freq;
  const int32_t* positions;
  int64_t pos0, L;
  uint16_t *Qo, *Ko;
  float eps;
  int H, rot;
  // work units, one warp each: nq of queries, then those of keys
  int64_t nq, units;
  int parts, heads;  // parts per token and heads per part; parts = 0: a group of lanes per token
};

HSA_DEV void unpack8(const uint4& v, float (&x)[8]) {
  x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x);
  x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z);
  x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
}

// (a, b) of the lane's eight pairs from its two chunks, and back.
template <bool INTER>
HSA_DEV void to_pairs(const float (&x)[8], const float (&y)[8], float (&a)[8], float (&b)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (INTER) {
      a[e] = e < 4 ? x[2 * e] : y[2 * e - 8];
      b[e] = e < 4 ? x[2 * e + 1] : y[2 * e - 7];
    } else {
      a[e] = x[e];
      b[e] = y[e];
    }
  }
}
template <bool INTER>
HSA_DEV void from_pairs(const float (&a)[8], const float (&b)[8], uint4& x, uint4& y) {
  if (INTER) {
    x = make_uint4(cvt_bf16x2(a[0], b[0]), cvt_bf16x2(a[1], b[1]), cvt_bf16x2(a[2], b[2]), cvt_bf16x2(a[3], b[3]));
    y = make_uint4(cvt_bf16x2(a[4], b[4]), cvt_bf16x2(a[5], b[5]), cvt_bf16x2(a[6], b[6]), cvt_bf16x2(a[7], b[7]));
  } else {
    x = make_uint4(cvt_bf16x2(a[0], a[1]), cvt_bf16x2(a[2], a[3]), cvt_bf16x2(a[4], a[5]), cvt_bf16x2(a[6], a[7]));
    y = make_uint4(cvt_bf16x2(b[0], b[1]), cvt_bf16x2(b[2], b[3]), cvt_bf16x2(b[4], b[5]), cvt_bf16x2(b[6], b[7]));
  }
}

HSA_DEV void angle(int64_t p, float f, float* c, float* s) {
  double turns = double(p) * double(f) * 0.15915494309189533577;
  turns -= rint(turns);
  sincospif(2.0f * float(turns), s, c);
}

// n rows of this lane's group (src, src + step, ...) at position p. SHARED:
// every group of the warp is at the same position, and each computes its
// share of the angles. All 32 lanes call; n may differ between groups.
template <int D, bool INTER, bool SHARED>
HSA_DEV void norm_rope_rows(const NormRopeArgs& a, const uint16_t* src, uint16_t* dst, int64_t step, int n, int n_max,
                            const uint16_t* w, int64_t p) {
  constexpr int LPR = D / 16, G = 32 / LPR, U = 4;
  const int lane = threadIdx.x & 31, l = lane % LPR, grp = lane / LPR;
  const int hr = a.rot / 2, hc = a.rot / 16;
  const int c0 = INTER ? l : l < hc ? l : 2 * l, c1 = INTER ? l + LPR : l < hc ? l + hc : 2 * l + 1;
  auto freq = [&](int e) { return INTER ? (e < 4 ? 4 * l + e : 4 * (l + LPR) + e - 4) : 8 * l + e; };
  uint4 v[U][2];
  auto load = [&](int i) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u < n) {
        const uint4* r = reinterpret_cast<const uint4*>(src + (i + u) * step);
        v[u][0] = r[c0];
        v[u][1] = r[c1];
      } else {
        v[u][0] = v[u][1] = make_uint4(0, 0, 0, 0);
      }
  };
  load(0);
  // P = wa cos, Q = wb sin, R = wb cos, S = wa sin of the lane's pairs
  float P[8], Q[8], R[8], S[8];
  {
    float wa[8], wb[8];
    if (w) {
      float x[8], y[8];
      unpack8(__ldg(reinterpret_cast<const uint4*>(w) + c0), x);
      unpack8(__ldg(reinterpret_cast<const uint4*>(w) + c1), y);
      to_pairs<INTER>(x, y, wa, wb);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) wa[e] = wb[e] = 1.f;
    }
    float mc[SHARED ? 8 / G : 8], ms[SHARED ? 8 / G : 8];
    constexpr int E = SHARED ? 8 / G : 8;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      // (the compile-time index keeps freq() in registers: e of the lane's share)
      int f = freq(e);
      if (SHARED) {
#pragma unroll
        for (int q = 1; q < G; ++q)
          if (grp == q) f = freq(q * E + e);
      }
      mc[e] = 1.f;
      ms[e] = 0.f;
      if (f < hr) angle(p, __ldg(a.inv_freq + f), &mc[e], &ms[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float c = SHARED ? __shfl_sync(kFull, mc[e % E], (e / E) * LPR + l) : mc[e];
      const float s = SHARED ? __shfl_sync(kFull, ms[e % E], (e / E) * LPR + l) : ms[e];
      P[e] = wa[e] * c; Q[e] = wb[e] * s; R[e] = wb[e] * c; S[e] = wa[e] * s;
    }
  }
  for (int i = 0; i < n_max; i += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[8], y[8], xa[8], xb[8];
      unpack8(v[u][0], x);
      unpack8(v[u][1], y);
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) { s0 = __fmaf_rn(x[e], x[e], s0); s1 = __fmaf_rn(y[e], y[e], s1); }
      float ss = s0 + s1;
#pragma unroll
      for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
      const float rs = rsqrtf(ss * (1.0f / D) + a.eps);
      to_pairs<INTER>(x, y, xa, xb);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // a value that is not turned must not meet an infinite neighbour
        const bool on = freq(e) < hr;
        const float ua = xa[e] * P[e] - (on ? xb[e] : xa[e]) * Q[e];
        const float ub = xb[e] * R[e] + (on ? xa[e] : xb[e]) * S[e];
        xa[e] = ua * rs;
        xb[e] = ub * rs;
      }
      if (i + u < n) {
        uint4* o = reinterpret_cast<uint4*>(dst + (i + u) * step);
        from_pairs<INTER>(xa, xb, v[u][0], v[u][1]);
        o[c0] = v[u][0];
        o[c1] = v[u][1];
      }
    }
    if (i + U < n_max) load(i + U);
  }
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kNT) qk_norm_rope_kernel(const NormRopeArgs a) {
  constexpr int LPR = D / 16, G = 32 / LPR;
  griddep_wait();
  griddep_launch();
  const int64_t unit = int64_t(blockIdx.x) * (kNT / 32) + (threadIdx.x >> 5);
  if (unit >= a.units) return;
  const int grp = (threadIdx.x & 31) / LPR;
  auto pos = [&](int64_t t) { return a.positions ? int64_t(a.positions[t]) : a.pos0 + t; };
  const bool keys = unit >= a.nq;
  if (!keys && a.parts > 0) {
    // the warp's groups take every G-th head of one token
    const int64_t t = unit / a.parts;
    const int h0 = int(unit - t * a.parts) * a.heads, nh = min(a.heads, a.H - h0);
    const int64_t p = pos(t);
    if (p < 0) return;
    const int n = (nh - grp + G - 1) / G;  // (zero for a group past the last head)
    norm_rope_rows<D, INTER, true>(a, a.Q + t * a.q_stride + (h0 + grp) * D, a.Qo + (t * a.H + h0 + grp) * D,
                                   int64_t(G) * D, n, (nh + G - 1) / G, a.qw, p);
  } else {
    // a token per group: its few heads, or its key
    const int64_t t = (keys ? unit - a.nq : unit) * G + grp;
    const int64_t p = t < a.L ? pos(t) : -1;
    const int rows = keys ? 1 : a.H;
    const int64_t ts = p < 0 ? 0 : t;
    norm_rope_rows<D, INTER, false>(a, keys ? a.K + ts * a.k_stride : a.Q + ts * a.q_stride,
                                    keys ? a.Ko + ts * D : a.Qo + ts * a.H * D, D, p < 0 ? 0 : rows, rows,
                                    keys ? a.kw : a.qw, p < 0 ? 0 : p);
  }
}

}  // namespace

void launch_qk_norm_rope(int64_t L, int H, int d, const void* Q, int64_t q_stride, const void* K, int64_t k_stride,
                         const void* qw, const void* kw, float eps, const float* inv_freq, int rot, bool interleaved,
                         const int32_t* positions, int64_t pos0, void* Qo, void* Ko, cudaStream_t s) {
  NormRopeArgs a{};
  a.Q = (const uint16_t*)Q; a.K = (const uint16_t*)K; a.qw = (const uint16_t*)qw; a.kw = (const uint16_t*)kw;
  a.q_stride = q_stride; a.k_stride = k_stride;
  a.inv_freq = inv_freq; a.positions = positions; a.pos0 = pos0; a.L = L;
  a.Qo = (uint16_t*)Qo; a.Ko = (uint16_t*)Ko;
  a.eps = eps; a.H = H; a.rot = rot;
  const int G = 512 / d;  // rows a warp takes at once
  const int64_t by_group = (L + G - 1) / G;
  if (Q && H < G) {
    a.nq = by_group;
  } else if (Q) {
    // few tokens: their heads over more warps, down to 4 rows per group
    const int most = std::max(1, H / (4 * G));
    const int64_t want = 16 * int64_t(num_sms()) / L;
    a.parts = int(std::max<int64_t>(1, std::min<int64_t>(most, want)));
    a.heads = (H + a.parts - 1) / a.parts;
    a.parts = (H + a.heads - 1) / a.heads;
    a.nq = L * a.parts;
  }
  a.units = a.nq + (K ? by_group : 0);
  const unsigned grid = unsigned((a.units + kNT / 32 - 1) / (kNT / 32));
  count_launches(1);
  if (d == 128)
    launch_kernel(true, interleaved ? qk_norm_rope_kernel<128, true> : qk_norm_rope_kernel<128, false>, grid, kNT, 0,
                  s, a);
  else
    launch_kernel(true, interleaved ? qk_norm_rope_kernel<64, true> : qk_norm_rope_kernel<64, false>, grid, kNT, 0, s,
                  a);
}

}  // namespace hsa
