// kp_rope_qk.cuh -- rotary positions with several axes (time, height, width,
// ...) on the heads of q and k, with the per-head RMS norm in front of them:
//
//   v = q / sqrt(mean(q^2) + eps) * w                    (w given; per head)
//   phi_p = pos[t, axis(p)] * theta^(-2 i_p / d_axis)    (pair p)
//   (e0, e1) -> (e0 cos phi - e1 sin phi, e0 sin phi + e1 cos phi)
//
// pairs (2p, 2p + 1), or (p, p + R/2) for the halves layout, R the rotated
// width; elements from R on keep v.  fp32 inside, rounded once.
//
// Bound by memory: every element is read once and written once.  The angle
// depends on the token alone, so a block takes a few whole tokens, computes
// their cosines and sines once into shared memory (while its first loads of
// q and k are in flight) and applies them to every head.  Angles are taken in
// turns in 64 bits and reduced there before the 32-bit sine and cosine, so a
// position of any int32 value keeps an angle error below 2^-23 turns.
#pragma once

#include <cstdint>

#include "kn_norm_gate.cuh"
#include "sm100_ptx.cuh"

namespace svdq {
namespace kp {

constexpr int THREADS = 256;
constexpr int MAX_D = 256;
constexpr int MAX_AXES = 4;
constexpr int MAX_TOKENS = 4;   // tokens of one block
constexpr int UNROLL = 4;       // 16-byte words of q / k in flight per thread

struct Params {
  const uint16_t *q, *k, *qw, *kw;
  uint16_t *qo, *ko;
  const int32_t* pos;             // [T, axes]
  int64_t qst, qsh, kst, ksh, qost, qosh, kost, kosh, ldpos;
  int T, Hq, Hk, D, half, axes;   // half = R / 2 pairs
  int tokens;                     // per block
  int lanes;                      // per head: a power of two >= D / 8, at most 32
  int pairs;                      // 1: (2p, 2p + 1); 0: (p, p + R / 2)
  float eps, inv_d;
  int first[MAX_AXES + 1];        // first pair of each axis
  double turns[MAX_D / 2];        // theta^(-2 i / d) / (2 pi) of each pair
};

template <bool BF16>
__global__ void __launch_bounds__(THREADS) rope_qk_kernel(const __grid_constant__ Params p) {
  // cos and sin of pair i of token t at [t][i].
  __shared__ __align__(16) float2 cs[MAX_TOKENS][MAX_D / 2];
  griddep_wait();
  griddep_launch_dependents();
  const int t0 = static_cast<int>(blockIdx.x) * p.tokens;
  const int nt = min(p.tokens, p.T - t0);
  const int H = p.Hq + p.Hk;
  const int j = static_cast<int>(threadIdx.x) & (p.lanes - 1);   // 8-element word of the head
  const int head0 = static_cast<int>(threadIdx.x) / p.lanes;
  const int heads = THREADS / p.lanes;                           // heads a pass covers
  const bool in = 8 * j < p.D;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);

  auto load = [&](int t, int h) -> uint4 {
    if (h >= H || !in) return zero;
    const uint16_t* src = h < p.Hq ? p.q + (t0 + t) * p.qst + h * p.qsh
                                   : p.k + (t0 + t) * p.kst + (h - p.Hq) * p.ksh;
    return ld_stream(src + 8 * j);
  };
  uint4 raw[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) raw[u] = load(0, head0 + u * heads);
  uint4 wq = zero, wk = zero;
  if (in && p.qw) wq = *reinterpret_cast<const uint4*>(p.qw + 8 * j);
  if (in && p.kw) wk = *reinterpret_cast<const uint4*>(p.kw + 8 * j);

  for (int i = threadIdx.x; i < nt * p.half; i += THREADS) {
    const int t = i / p.half, c = i - t * p.half;
    int a = 0;
#pragma unroll
    for (int b = 1; b < MAX_AXES; ++b) a += b < p.axes && c >= p.first[b] ? 1 : 0;
    const double turn = static_cast<double>(p.pos[(t0 + t) * p.ldpos + a]) * p.turns[c];
    float2 v;
    sincospif(2.f * static_cast<float>(turn - rint(turn)), &v.y, &v.x);
    cs[t][c] = v;
  }
  __syncthreads();

  // Lanes of this head, for its sum of squares.
  const uint32_t group = p.lanes == 32 ? 0xFFFFFFFFu
                                       : ((1u << p.lanes) - 1u) << (threadIdx.x & 31 & ~(p.lanes - 1));
  // The halves layout: the partner word, `words` up or down, is another lane's.
  const int words = p.half / 8;
  const bool low = j < words;
  const int from = (threadIdx.x & 31 & ~(p.lanes - 1)) + (low ? j + words : j < 2 * words ? j - words : j);
  const float sign = low ? -1.f : 1.f;

  for (int t = 0; t < nt; ++t) {
    // This lane's cosines and sines: the same for every head of the token.
    float c[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = p.pairs ? 4 * j + (e >> 1) : 8 * (low ? j : j - words) + e;
      const bool turned = p.pairs ? i < p.half : j < 2 * words;
      const float2 v = turned ? cs[t][i] : make_float2(1.f, 0.f);
      c[e] = v.x;
      sn[e] = p.pairs ? ((e & 1) ? v.y : -v.y) : sign * v.y;
    }
    for (int h0 = head0; h0 < H; h0 += UNROLL * heads) {
      uint4 cur[UNROLL];
      const bool next_token = h0 + UNROLL * heads >= H;
      const int nh = next_token ? head0 : h0 + UNROLL * heads;
      const int tn = next_token ? t + 1 : t;
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        cur[u] = raw[u];
        if (tn < nt) raw[u] = load(tn, nh + u * heads);
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int h = h0 + u * heads;
        if (h >= H) break;
        const bool is_q = h < p.Hq;
        float v[8];
        unpack8<BF16>(cur[u], v);
        if (is_q ? p.qw != nullptr : p.kw != nullptr) {
          float w[8];
          unpack8<BF16>(is_q ? wq : wk, w);
          uint64_t q2 = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint64_t x = pk(v[2 * e], v[2 * e + 1]);
            q2 = fma2(x, x, q2);
          }
          float lo, hi;
          upk(q2, lo, hi);
          float q = lo + hi;
          for (int o = p.lanes / 2; o > 0; o >>= 1) q += __shfl_xor_sync(group, q, o);
          const float r = rsqrtf(fmaf(q, p.inv_d, p.eps));
          const uint64_t r2 = pk(r, r);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            upk(mul2(mul2(pk(v[2 * e], v[2 * e + 1]), r2), pk(w[2 * e], w[2 * e + 1])), v[2 * e],
                v[2 * e + 1]);
        }
        float o[8];
        if (p.pairs) {
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = fmaf(v[e ^ 1], sn[e], v[e] * c[e]);
          // Past the rotated part: as it is, whatever the neighbour holds.
          if (4 * j + 4 > p.half) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (4 * j + (e >> 1) >= p.half) o[e] = v[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float other = __shfl_sync(group, v[e], from);
            o[e] = j < 2 * words ? fmaf(other, sn[e], v[e] * c[e]) : v[e];
          }
        }
        if (in) {
          uint16_t* dst = is_q ? p.qo + (t0 + t) * p.qost + h * p.qosh
                               : p.ko + (t0 + t) * p.kost + (h - p.Hq) * p.kosh;
          *reinterpret_cast<uint4*>(dst + 8 * j) = pack8<BF16>(o);
        }
      }
    }
  }
}

}  // namespace kp
}  // namespace svdq
