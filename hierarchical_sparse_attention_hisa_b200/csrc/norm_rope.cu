// Per-head RMS norm of queries and keys with the position rotation in the
// same pass: what turns a layer's projections (its own and its indexer's)
// into the Q / K (q_idx / k_idx) of the selection and the attention.
//
// For a row x of d values at position t:
//   y = x * w / sqrt(mean(x^2) + eps)
//   pairs (a, b) of the first `rot` values, (i, i + rot/2) or (2i, 2i+1):
//   (a cos u - b sin u, b cos u + a sin u),  u = t * inv_freq[i]
// in fp32, rounded once to bf16. A position times a frequency is taken in 64
// bits: in fp32 the angle would be off by up to t * 2^-24 radians, 0.06 at
// position 2^20. Here inv_freq becomes a fraction of a turn in 64-bit fixed
// point, whose product with t wraps at whole turns by itself; its top 32 bits
// are the angle to 2^-32 of a turn.
//
// One read and one write of every value bound it (HBM). A row is d/16 lanes of
// two 16-byte chunks, chosen so that both values of every pair are the same
// lane's: the split layout's lane holds chunk l and its partner l + rot/16, so
// the rotation exchanges nothing and only the sum of squares crosses lanes. A
// lane keeps its eight pairs' coefficients w cos u, w sin u in registers over
// all heads of a token. Warps stay and take token after token, the next rows'
// loads issued before the present ones are worked on. Measured: 65,536 tokens of
// 64 heads of 128 in 341 us (6.4 TB/s, 0.97 of the measured copy rate), 16,384
// of 16 heads out of a fused projection in 29 us (4.9 TB/s). Four CTAs of 128
// threads per SM: three (no spills) take 374 us, five 421 us.
#include <algorithm>

#include "kernels.cuh"

namespace hsa {
namespace {

constexpr int kNT = 128, kWarps = kNT / 32, kCtasPerSm = 4;

// One tensor's rows: token t's are src + t * stride + h * D, h < H.
struct Side {
  const uint16_t *src, *w;
  uint16_t* dst;
  int64_t stride;
  int H;
  // a unit (one warp's turn): heads `heads` of a token in `parts` parts, or with
  // parts = 0 a token per group of lanes
  int parts, heads;
  int64_t units;
};
struct NormRopeArgs {
  Side q, k;
  int q_ctas;  // the first CTAs take the queries, the others the keys
  const float* inv_freq;
  const int32_t* positions;
  int64_t pos0, L;
  float eps;
  int rot;
};

// Two fp32 values in one 64-bit register pair (packed arithmetic).
typedef unsigned long long f2;
HSA_DEV f2 pack2(float x, float y) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
HSA_DEV void unpack2(f2 v, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
HSA_DEV f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
HSA_DEV f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
HSA_DEV uint32_t bf16x2_of(f2 v) {
  float x, y;
  unpack2(v, x, y);
  return cvt_bf16x2(x, y);
}

// (a, b) of the lane's eight pairs from its two chunks, two pairs to an f2, and back.
template <bool INTER>
HSA_DEV void to_pairs(const uint4& x, const uint4& y, f2 (&a)[4], f2 (&b)[4]) {
  if (INTER) {
    a[0] = pack2(bf16_lo(x.x), bf16_lo(x.y)); b[0] = pack2(bf16_hi(x.x), bf16_hi(x.y));
    a[1] = pack2(bf16_lo(x.z), bf16_lo(x.w)); b[1] = pack2(bf16_hi(x.z), bf16_hi(x.w));
    a[2] = pack2(bf16_lo(y.x), bf16_lo(y.y)); b[2] = pack2(bf16_hi(y.x), bf16_hi(y.y));
    a[3] = pack2(bf16_lo(y.z), bf16_lo(y.w)); b[3] = pack2(bf16_hi(y.z), bf16_hi(y.w));
  } else {
    a[0] = pack2(bf16_lo(x.x), bf16_hi(x.x)); b[0] = pack2(bf16_lo(y.x), bf16_hi(y.x));
    a[1] = pack2(bf16_lo(x.y), bf16_hi(x.y)); b[1] = pack2(bf16_lo(y.y), bf16_hi(y.y));
    a[2] = pack2(bf16_lo(x.z), bf16_hi(x.z)); b[2] = pack2(bf16_lo(y.z), bf16_hi(y.z));
    a[3] = pack2(bf16_lo(x.w), bf16_hi(x.w)); b[3] = pack2(bf16_lo(y.w), bf16_hi(y.w));
  }
}
template <bool INTER>
HSA_DEV void from_pairs(const f2 (&a)[4], const f2 (&b)[4], uint4& x, uint4& y) {
  if (INTER) {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a0, a1, b0, b1;
      unpack2(a[e], a0, a1);
      unpack2(b[e], b0, b1);
      w[2 * e] = cvt_bf16x2(a0, b0);
      w[2 * e + 1] = cvt_bf16x2(a1, b1);
    }
    x = make_uint4(w[0], w[1], w[2], w[3]);
    y = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
    x = make_uint4(bf16x2_of(a[0]), bf16x2_of(a[1]), bf16x2_of(a[2]), bf16x2_of(a[3]));
    y = make_uint4(bf16x2_of(b[0]), bf16x2_of(b[1]), bf16x2_of(b[2]), bf16x2_of(b[3]));
  }
}

// One side's units first, first + step, ... SHARED: a unit is a part of one
// token's heads, the warp's groups take every G-th, and each computes its share
// of the angles; otherwise every group of lanes has a token of its own.
template <int D, bool INTER, bool SHARED>
HSA_DEV void norm_rope_side(const NormRopeArgs& a, const Side& s, int64_t first, int64_t step) {
  constexpr int LPR = D / 16, G = 32 / LPR;  // lanes per row, rows per warp
  constexpr int U = 2;                       // rows per group at a time, as many again on their way
  constexpr int E = SHARED ? 8 / G : 8;      // angles per lane
  const int lane = threadIdx.x & 31, l = lane % LPR, grp = lane / LPR;
  const int hr = a.rot / 2, hc = a.rot / 16;
  const int c0 = INTER ? l : l < hc ? l : 2 * l, c1 = INTER ? l + LPR : l < hc ? l + hc : 2 * l + 1;
  // the lane's frequencies, in 2^-64 turns per position (0 turns: not rotated)
  unsigned long long turn[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int q = SHARED ? grp * E + e : e;  // the pair
    const int f = INTER ? (q < 4 ? 4 * l + q : 4 * (l + LPR) + q - 4) : 8 * l + q;
    double x = f < hr ? double(__ldg(a.inv_freq + f)) * 0.15915494309189533577 : 0.0;
    x -= floor(x);
    turn[e] = __double2ull_rz(x * 18446744073709551616.0);
  }
  uint4 wx = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u), wy = wx;  // bf16 ones
  if (s.w) {
    wx = __ldg(reinterpret_cast<const uint4*>(s.w) + c0);
    wy = __ldg(reinterpret_cast<const uint4*>(s.w) + c1);
  }
  // a unit's rows for this group: n rows `row_step` apart, at position p
  const int64_t row_step = SHARED ? int64_t(G) * D : D;
  struct Unit { int64_t in, out; int n, p; };
  auto unit_of = [&](int64_t u) {
    Unit r{0, 0, 0, -1};
    const int64_t t = SHARED ? u / s.parts : u * G + grp;
    if (u < s.units && t < a.L) {
      const int64_t p = a.positions ? int64_t(a.positions[t]) : a.pos0 + t;
      const int h0 = SHARED ? int(u - t * s.parts) * s.heads + grp : 0;
      const int h1 = SHARED ? min(s.H, h0 - grp + s.heads) : s.H;
      r.in = t * s.stride + int64_t(h0) * D;
      r.out = (t * s.H + h0) * D;
      r.p = int(p);
      r.n = p < 0 ? 0 : SHARED ? (h1 - h0 + G - 1) / G : h1;
    }
    return r;
  };
  // rows of a unit that some group of the warp has
  const int most = SHARED ? (s.heads + G - 1) / G : s.H;
  auto load = [&](uint4 (&v)[U][2], const Unit& x, int i) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u][0] = v[u][1] = make_uint4(0, 0, 0, 0);
      if (i + u < x.n) {
        const uint4* r = reinterpret_cast<const uint4*>(s.src + x.in + (i + u) * row_step);
        v[u][0] = r[c0];
        v[u][1] = r[c1];
      }
    }
  };
  uint4 v[U][2], vn[U][2];
  Unit cur = unit_of(first), next = unit_of(first + step);
  load(v, cur, 0);
  for (int64_t u0 = first; u0 < s.units; u0 += step) {
    // P = wa cos, Q = -wb sin, R = wb cos, S = wa sin of the lane's pairs
    f2 P[4], Q[4], R[4], S[4];
    {
      float mc[E], ms[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int at = int((turn[e] * (unsigned long long)(unsigned)cur.p) >> 32);  // signed: (-1/2, 1/2] turns
        const float u = float(at) * 1.46291807926715968e-9f;                      // 2 pi / 2^32
        mc[e] = __cosf(u);
        ms[e] = __sinf(u);
      }
      f2 wa[4], wb[4];
      to_pairs<INTER>(wx, wy, wa, wb);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float c[2], n[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int q = 2 * e + z;
          c[z] = SHARED ? __shfl_sync(kFull, mc[q % E], (q / E) * LPR + l) : mc[q];
          n[z] = SHARED ? __shfl_sync(kFull, ms[q % E], (q / E) * LPR + l) : ms[q];
        }
        const f2 co = pack2(c[0], c[1]), si = pack2(n[0], n[1]);
        P[e] = mul2(wa[e], co);
        R[e] = mul2(wb[e], co);
        S[e] = mul2(wa[e], si);
        Q[e] = mul2(wb[e], pack2(-n[0], -n[1]));
      }
    }
    const Unit now = cur;
    cur = next;
    next = unit_of(u0 + 2 * step);
    for (int i = 0; i < most; i += U) {
      if (i + U < most) load(vn, now, i + U);
      else load(vn, cur, 0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        f2 xa[4], xb[4], s2 = 0;
        to_pairs<INTER>(v[u][0], v[u][1], xa, xb);
#pragma unroll
        for (int e = 0; e < 4; ++e) s2 = fma2(xb[e], xb[e], fma2(xa[e], xa[e], s2));
        float ss, s1;
        unpack2(s2, ss, s1);
        ss += s1;
#pragma unroll
        for (int o = LPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
        const float rs = rsqrtf(ss * (1.0f / D) + a.eps);
        const f2 rs2 = pack2(rs, rs);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f2 ua = fma2(xa[e], P[e], mul2(xb[e], Q[e]));
          xb[e] = mul2(fma2(xb[e], R[e], mul2(xa[e], S[e])), rs2);
          xa[e] = mul2(ua, rs2);
        }
        if (i + u < now.n) {
          uint4* o = reinterpret_cast<uint4*>(s.dst + now.out + (i + u) * row_step);
          uint4 x, y;
          from_pairs<INTER>(xa, xb, x, y);
          o[c0] = x;
          o[c1] = y;
        }
        v[u][0] = vn[u][0];
        v[u][1] = vn[u][1];
      }
    }
  }
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kNT, kCtasPerSm) qk_norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  griddep_wait();
  griddep_launch();
  const int warp = threadIdx.x >> 5;
  if (int(blockIdx.x) < a.q_ctas) {
    const int64_t first = int64_t(blockIdx.x) * kWarps + warp, step = int64_t(a.q_ctas) * kWarps;
    if (a.q.parts > 0) norm_rope_side<D, INTER, true>(a, a.q, first, step);
    else norm_rope_side<D, INTER, false>(a, a.q, first, step);
  } else {
    const int64_t first = int64_t(blockIdx.x - a.q_ctas) * kWarps + warp;
    norm_rope_side<D, INTER, false>(a, a.k, first, int64_t(gridDim.x - a.q_ctas) * kWarps);
  }
}

}  // namespace

void launch_qk_norm_rope(int64_t L, int H, int d, const void* Q, int64_t q_stride, const void* K, int64_t k_stride,
                         const void* qw, const void* kw, float eps, const float* inv_freq, int rot, bool interleaved,
                         const int32_t* positions, int64_t pos0, void* Qo, void* Ko, cudaStream_t s) {
  NormRopeArgs a{};
  a.inv_freq = inv_freq; a.positions = positions; a.pos0 = pos0; a.L = L; a.eps = eps; a.rot = rot;
  const int G = 512 / d;  // rows a warp takes at once
  const int64_t by_group = (L + G - 1) / G;
  if (Q) {
    a.q = Side{(const uint16_t*)Q, (const uint16_t*)qw, (uint16_t*)Qo, q_stride, H, 0, 0, by_group};
    // A token to a warp (its angles computed once) from G heads on; with up to 1.5 G
    // its second step leaves groups idle, and many tokens are better one to each group:
    // 65,536 of 4 heads of 128 in 35.5 us (a warp each: 60), of 8 of 64 in 35 (52);
    // 512 tokens take 2.9 us (a warp each: 2.5). At 2 G: 58 to 60 us either way.
    if (H >= G && (2 * H > 3 * G || L < 16 * int64_t(num_sms()))) {
      // few tokens: their heads over more warps, down to 4 rows per group
      const int64_t want = std::min<int64_t>(std::max(1, H / (4 * G)), 16 * int64_t(num_sms()) / L);
      a.q.heads = (H + std::max<int64_t>(1, want) - 1) / std::max<int64_t>(1, want);
      a.q.parts = (H + a.q.heads - 1) / a.q.heads;
      a.q.units = L * a.q.parts;
    }
  }
  if (K) a.k = Side{(const uint16_t*)K, (const uint16_t*)kw, (uint16_t*)Ko, k_stride, 1, 0, 0, by_group};
  // the CTAs that the device holds at once, split as the work is: a token's key
  // costs about three rows (its angles are its own)
  const int64_t all = int64_t(kCtasPerSm) * num_sms();
  const int64_t q_need = (a.q.units + kWarps - 1) / kWarps, k_need = (a.k.units + kWarps - 1) / kWarps;
  const int64_t k_share = Q ? std::max<int64_t>(1, all * 3 / (H + 5)) : all;
  const int64_t k_ctas = std::min(k_need, k_share);
  a.q_ctas = int(std::min(q_need, std::max<int64_t>(1, all - k_ctas)));
  const unsigned grid = unsigned(a.q_ctas + k_ctas);
  count_launches(1);
  if (d == 128)
    launch_kernel(true, interleaved ? qk_norm_rope_kernel<128, true> : qk_norm_rope_kernel<128, false>, grid, kNT, 0,
                  s, a);
  else
    launch_kernel(true, interleaved ? qk_norm_rope_kernel<64, true> : qk_norm_rope_kernel<64, false>, grid, kNT, 0, s,
                  a);
}

}  // namespace hsa
