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

struct Params {
  const uint16_t *q, *k, *qw, *kw;
  uint16_t *qo, *ko;
  const int32_t* pos;             // [T, axes]
  int64_t qst, qsh, kst, ksh, qost, qosh, kost, kosh, ldpos;
  int T, Hq, Hk, D, half, axes;   // half = R / 2 pairs
  int tokens;                     // per block
  float eps, inv_d;
  int first[MAX_AXES + 1];        // first pair of each axis
  double turns[MAX_D / 2];        // theta^(-2 i / d) / (2 pi) of each pair
};

// LANES: threads of one head, one 8-element word each (8 LANES >= D).
// PAIRS: pairs (2p, 2p + 1), else (p, p + R / 2).
template <bool BF16, int LANES, bool PAIRS>
__global__ void __launch_bounds__(THREADS, 4) rope_qk_kernel(const __grid_constant__ Params p) {
  constexpr int HEADS = THREADS / LANES;   // heads a pass of the block covers
  constexpr int UNROLL = 2;                // words in flight per thread
  // cos and sin of pair i of token t at [t][i].
  __shared__ __align__(16) float2 cs[MAX_TOKENS][MAX_D / 2];
  griddep_wait();
  griddep_launch_dependents();
  const int t0 = static_cast<int>(blockIdx.x) * p.tokens;
  const int nt = min(p.tokens, p.T - t0);
  const int j = static_cast<int>(threadIdx.x) % LANES;   // word of the head
  const int head0 = static_cast<int>(threadIdx.x) / LANES;
  const bool in = 8 * j < p.D;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);

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

  // Lanes of this head, for its sum of squares and its other half.
  const uint32_t group = LANES == 32 ? 0xFFFFFFFFu
                                     : ((1u << (LANES & 31)) - 1u) << (threadIdx.x & 31 & ~(LANES - 1));
  // The halves layout: the partner word, `words` up or down, is another lane's.
  const int words = p.half / 8;
  const bool low = j < words;
  const bool turned = j < 2 * words;   // halves: a whole word is, or is not
  const int from = (threadIdx.x & 31 & ~(LANES - 1)) + (low ? j + words : turned ? j - words : j);
  const float sign = low ? -1.f : 1.f;

  // One tensor's heads of one token.
  auto rotate = [&](const uint16_t* src, int64_t sh, uint16_t* dst, int64_t dh, int H, bool norm,
                    const uint4& wv, const float (&c)[PAIRS ? 4 : 8], const float (&sn)[PAIRS ? 4 : 8]) {
    src += head0 * sh + 8 * j;
    dst += head0 * dh + 8 * j;
    for (int h = head0; h < H; h += UNROLL * HEADS) {
      uint4 raw[UNROLL];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        raw[u] = in && h + u * HEADS < H ? ld_stream(src) : zero;
        src += HEADS * sh;
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        if (h + u * HEADS >= H) return;
        float v[8];
        unpack8<BF16>(raw[u], v);
        if (norm) {
          float q = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) q = fmaf(v[e], v[e], q);
#pragma unroll
          for (int o = LANES / 2; o > 0; o >>= 1) q += __shfl_xor_sync(group, q, o);
          const float r = rsqrtf(fmaf(q, p.inv_d, p.eps));
          float w[8];
          unpack8<BF16>(wv, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = (v[e] * r) * w[e];
        }
        float o[8];
        if (PAIRS) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o[2 * e] = fmaf(-v[2 * e + 1], sn[e], v[2 * e] * c[e]);
            o[2 * e + 1] = fmaf(v[2 * e], sn[e], v[2 * e + 1] * c[e]);
          }
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
            o[e] = turned ? fmaf(other, sn[e % (PAIRS ? 4 : 8)], v[e] * c[e % (PAIRS ? 4 : 8)]) : v[e];
          }
        }
        if (in) *reinterpret_cast<uint4*>(dst) = pack8<BF16>(o);
        dst += HEADS * dh;
      }
    }
  };

  uint4 wq = zero, wk = zero;
  if (in && p.qw) wq = *reinterpret_cast<const uint4*>(p.qw + 8 * j);
  if (in && p.kw) wk = *reinterpret_cast<const uint4*>(p.kw + 8 * j);
  for (int t = 0; t < nt; ++t) {
    // This lane's cosines and sines: the same for every head of the token.
    float c[PAIRS ? 4 : 8], sn[PAIRS ? 4 : 8];
#pragma unroll
    for (int e = 0; e < (PAIRS ? 4 : 8); ++e) {
      const int i = PAIRS ? 4 * j + e : 8 * (low ? j : j - words) + e;
      const float2 v = (PAIRS ? i < p.half : turned) ? cs[t][i] : make_float2(1.f, 0.f);
      c[e] = v.x;
      sn[e] = PAIRS ? v.y : sign * v.y;
    }
    const int64_t row = t0 + t;
    rotate(p.q + row * p.qst, p.qsh, p.qo + row * p.qost, p.qosh, p.Hq, p.qw != nullptr, wq, c, sn);
    rotate(p.k + row * p.kst, p.ksh, p.ko + row * p.kost, p.kosh, p.Hk, p.kw != nullptr, wk, c, sn);
  }
}

}  // namespace kp
}  // namespace svdq
