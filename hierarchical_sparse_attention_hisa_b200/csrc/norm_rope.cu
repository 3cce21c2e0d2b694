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
// One read and one write of every value bound it (HBM). A row is d/8 lanes of
// 16 bytes; its sum of squares is reduced across those lanes and the rotation
// partner of the split layout comes by shuffle, so a value never leaves
// registers. A CTA's tokens share one table of angles in shared memory.
#include "kernels.cuh"

namespace hsa {
namespace {

constexpr int kNT = 256;

struct NormRopeArgs {
  const uint16_t *Q, *K, *qw, *kw;
  int64_t q_stride, k_stride;
  const float* inv_freq;
  const int32_t* positions;
  int64_t pos0, L;
  uint16_t *Qo, *Ko;
  float eps;
  int HQ, rows, rot, toks;  // query heads, rows per token (queries, then the key), tokens per CTA
};

HSA_DEV void unpack8(const uint4& v, float (&x)[8]) {
  x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x);
  x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z);
  x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kNT) qk_norm_rope_kernel(const NormRopeArgs a) {
  constexpr int CH = D / 8, RPP = kNT / CH;  // chunks per row; rows per pass
  constexpr int U = 4;                                       // rows in flight per lane
  griddep_wait();
  griddep_launch();
  extern __shared__ __align__(16) float table[];  // [toks][2][rot/2]: cosines, sines
  const int hr = a.rot / 2;
  const int64_t t0 = int64_t(blockIdx.x) * a.toks;
  const int nt = int(a.L - t0 < a.toks ? a.L - t0 : a.toks);
  for (int e = threadIdx.x; e < nt * hr; e += kNT) {
    const int tk = e / hr, i = e - tk * hr;
    const int64_t p = a.positions ? int64_t(a.positions[t0 + tk]) : a.pos0 + t0 + tk;
    double turns = double(p) * double(a.inv_freq[i]) * 0.15915494309189533577;
    turns -= rint(turns);
    float s, c;
    sincospif(2.0f * float(turns), &s, &c);
    table[tk * a.rot + i] = c;
    table[tk * a.rot + hr + i] = s;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, c = lane % CH;
  const int hc = hr / 8;
  const int total = nt * a.rows;
  for (int r0 = threadIdx.x / CH; r0 < total; r0 += RPP * U) {
    uint4 v[U];
    int tk[U], h[U];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPP;
      on[u] = r < total;
      tk[u] = r / a.rows;
      h[u] = r - tk[u] * a.rows;
      if (on[u] && a.positions) on[u] = a.positions[t0 + tk[u]] >= 0;  // a row that takes no part
      v[u] = make_uint4(0, 0, 0, 0);
      if (on[u]) {
        const uint16_t* src = h[u] < a.HQ ? a.Q + (t0 + tk[u]) * a.q_stride + h[u] * D : a.K + (t0 + tk[u]) * a.k_stride;
        v[u] = *(reinterpret_cast<const uint4*>(src) + c);
      }
    }
    // (the lanes of a warp leave the outer loop together only when every row
    // of the warp is past the end; a warp's rows are adjacent, so shuffles
    // below are taken by the lanes of whole rows: their mask is the row's)
    const unsigned mask = (CH == 32 ? kFull : ((1u << CH) - 1u)) << (lane & ~(CH - 1));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[8];
      unpack8(v[u], x);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = __fmaf_rn(x[e], x[e], ss);
#pragma unroll
      for (int o = CH / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
      const float rs = rsqrtf(ss * (1.0f / D) + a.eps);
      const uint16_t* wp = h[u] < a.HQ ? a.qw : a.kw;
      float w[8];
      if (wp) unpack8(__ldg(reinterpret_cast<const uint4*>(wp) + c), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= wp ? rs * w[e] : rs;
      const float* cs = table + (on[u] ? tk[u] : 0) * a.rot;
      if (INTER) {
        if (c < 2 * hc) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float co = cs[4 * c + e], si = cs[hr + 4 * c + e];
            const float p = x[2 * e], q = x[2 * e + 1];
            x[2 * e] = p * co - q * si;
            x[2 * e + 1] = q * co + p * si;
          }
        }
      } else {
        const bool lo = c < hc, in = c < 2 * hc;
        const int src = (lane & ~(CH - 1)) + (lo ? c + hc : in ? c - hc : c);
        const int f0 = 8 * (lo ? c : in ? c - hc : 0);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float other = __shfl_sync(mask, x[e], src);
          if (in) {
            const float co = cs[f0 + e], si = cs[hr + f0 + e];
            x[e] = x[e] * co + (lo ? -other : other) * si;
          }
        }
      }
      if (on[u]) {
        uint16_t* dst = h[u] < a.HQ ? a.Qo + ((t0 + tk[u]) * a.HQ + h[u]) * D : a.Ko + (t0 + tk[u]) * D;
        *(reinterpret_cast<uint4*>(dst) + c) = make_uint4(cvt_bf16x2(x[0], x[1]), cvt_bf16x2(x[2], x[3]),
                                                          cvt_bf16x2(x[4], x[5]), cvt_bf16x2(x[6], x[7]));
      }
    }
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
  a.eps = eps;
  a.HQ = Q ? H : 0;
  a.rows = a.HQ + (K ? 1 : 0);
  a.rot = rot;
  // few rows per token: several tokens per CTA, so that every lane has one
  const int rpp = kNT / (d / 8);
  a.toks = a.rows >= 2 * rpp ? 1 : (2 * rpp + a.rows - 1) / a.rows;
  const unsigned grid = unsigned((L + a.toks - 1) / a.toks);
  const size_t smem = size_t(a.toks) * rot * 4;
  count_launches(1);
  if (d == 128)
    launch_kernel(true, interleaved ? qk_norm_rope_kernel<128, true> : qk_norm_rope_kernel<128, false>, grid, kNT,
                  smem, s, a);
  else
    launch_kernel(true, interleaved ? qk_norm_rope_kernel<64, true> : qk_norm_rope_kernel<64, false>, grid, kNT, smem,
                  s, a);
}

}  // namespace hsa
