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
  // cos and sin of pair i of token t at [t][i].
  __shared__ __align__(16) float2 cs[MAX_TOKENS][MAX_D / 2];
  griddep_wait();
  griddep_launch_dependents();
  const int t0 = static_cast<int>(blockIdx.x) * p.tokens;
  const int nt = min(p.tokens, p.T - t0);
  const int j = static_cast<int>(threadIdx.x) % LANES;   // word of the head
  const int head0 = static_cast<int>(threadIdx.x) / LANES;

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
  const uint32_t group = LANES == 32 ? 0xFFFFFFFFu
                                     : ((1u << (LANES & 31)) - 1u) << (threadIdx.x & 31 & ~(LANES - 1));
  // The lane's eight elements: pairs 4 j .. 4 j + 3, which are eight in a row,
  // or (halves) four in a row at `lo` and their partners at `hi`; from the
  // rotated part's end on, eight in a row.
  const bool turned = PAIRS || 4 * j < p.half;
  const int lo = PAIRS ? 8 * j : turned ? 4 * j : 2 * p.half + 8 * (j - p.half / 4);
  const int hi = PAIRS ? 8 * j + 4 : turned ? 4 * j + p.half : lo + 4;
  const bool in = lo < p.D;

  auto load = [&](const uint16_t* src) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (PAIRS) {
      v = ld_stream(src + lo);
    } else {
      const uint2 a = *reinterpret_cast<const uint2*>(src + lo), b = *reinterpret_cast<const uint2*>(src + hi);
      v = make_uint4(a.x, a.y, b.x, b.y);
    }
    return v;
  };

  // One head: its norm, its rotation, its store.
  auto rotate = [&](const uint4& raw, uint16_t* dst, bool norm, const uint4& wv, const float (&c)[4],
                    const float (&sn)[4]) {
    float v[8], o[8];
    unpack8<BF16>(raw, v);
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
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      constexpr int STEP = PAIRS ? 2 : 1, OTHER = PAIRS ? 1 : 4;
      const float e0 = v[STEP * e], e1 = v[STEP * e + OTHER];
      o[STEP * e] = fmaf(-e1, sn[e], e0 * c[e]);
      o[STEP * e + OTHER] = fmaf(e0, sn[e], e1 * c[e]);
    }
    // Past the rotated part: as it is, whatever the neighbour holds.
    if (4 * j + 4 > p.half) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (4 * j + (PAIRS ? e >> 1 : e & 3) >= p.half) o[e] = v[e];
    }
    if (!in) return;
    const uint4 w = pack8<BF16>(o);
    if (PAIRS) {
      *reinterpret_cast<uint4*>(dst + lo) = w;
    } else {
      *reinterpret_cast<uint2*>(dst + lo) = make_uint2(w.x, w.y);
      *reinterpret_cast<uint2*>(dst + hi) = make_uint2(w.z, w.w);
    }
  };

  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const uint4 wq = in && p.qw ? load(p.qw) : zero, wk = in && p.kw ? load(p.kw) : zero;
  for (int t = 0; t < nt; ++t) {
    // This lane's cosines and sines: the same for every head of the token.
    float c[4], sn[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 v = 4 * j + e < p.half ? cs[t][4 * j + e] : make_float2(1.f, 0.f);
      c[e] = v.x;
      sn[e] = v.y;
    }
    const int64_t row = t0 + t;
    const uint16_t* q = p.q + row * p.qst + head0 * p.qsh;
    const uint16_t* k = p.k + row * p.kst + head0 * p.ksh;
    uint16_t* qo = p.qo + row * p.qost + head0 * p.qosh;
    uint16_t* ko = p.ko + row * p.kost + head0 * p.kosh;
    // Two heads of q and two of k in flight.
    for (int h = head0; h < max(p.Hq, p.Hk); h += 2 * HEADS) {
      uint4 a[2], b[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        a[u] = in && h + u * HEADS < p.Hq ? load(q) : zero;
        b[u] = in && h + u * HEADS < p.Hk ? load(k) : zero;
        q += HEADS * p.qsh;
        k += HEADS * p.ksh;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (h + u * HEADS < p.Hq) {
          rotate(a[u], qo, p.qw != nullptr, wq, c, sn);
        }
        if (h + u * HEADS < p.Hk) {
          rotate(b[u], ko, p.kw != nullptr, wk, c, sn);
        }
        qo += HEADS * p.qosh;
        ko += HEADS * p.kosh;
      }
    }
  }
}

}  // namespace kp
}  // namespace svdq
