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
// Bound by memory: every element is read once and written once.  A warp works
// alone on a run of units (up to 4 KB of one tensor's heads of one token),
// which come by bulk copies into its own two slots of shared memory; no
// barrier ever joins the warps.  The angle depends on the token alone: the
// warp computes its cosines and sines when the token changes, and a lane,
// which always has the same place in the head, folds its four pairs of them
// with the norm's weights into sixteen registers for all heads of a unit.
// Angles are taken in turns in 64 bits and reduced there before the 32-bit
// sine and cosine, so a position of any int32 value keeps an angle error
// below 2^-22 turns.  Calls in a row: 4352 tokens x 60 heads of 128 (134 MB) 29.8
// us, 4.5 TB/s, 69% of a plain copy's rate; 9973 tokens x 40 heads in halves (204
// MB) 41.8 us, 4.9 TB/s, 76%; as a graph 28.2 and 40.5 us, one token 4.5.  Issue
// slots are 60% taken.  Three blocks an SM leave 80 registers a thread; ten of
// the twelve instances spill 4 to 20 bytes there (pairs of 128 and less 12,
// halves 20).  In short runs, 28.9 us then: a block per few tokens with a
// barrier for the angles 32.6 us, one with the whole block on a shared ring
// 34.1 (warps waiting for the two that compute angles), packed two-wide
// arithmetic 29.6 (half the instructions, at half the rate), units of 2 KB in
// rings of four 33.2; four passes unrolled gain 1.5% here and lose 3% at 17408
// tokens.
#pragma once

#include <cstdint>

#include "kn_norm_gate.cuh"
#include "sm100_ptx.cuh"

namespace svdq {
namespace kp {

constexpr int THREADS = 256;
constexpr int MAX_D = 256;
constexpr int MAX_AXES = 4;
constexpr int WARPS = THREADS / 32;
constexpr int RING = 2;                     // units on their way, per warp
constexpr uint32_t UNIT_BYTES = 4096;       // heads of one token that a unit takes, at most
constexpr uint32_t SMEM_BYTES = WARPS * RING * UNIT_BYTES;
constexpr uint32_t SITE_UNIT = 0x68;

struct Params {
  const uint16_t *q, *k, *qw, *kw;
  uint16_t *qo, *ko;
  const int32_t* pos;             // [T, axes]
  int64_t qst, qsh, kst, ksh, qost, qosh, kost, kosh, ldpos;
  int T, Hq, Hk, D, half, axes;   // half = R / 2 pairs
  int heads_q, heads_k;           // heads of a unit of q, of k
  int parts_q, parts;             // units of q, of both, per token
  int units_per_warp;
  float eps, inv_d;
  int first[MAX_AXES + 1];        // first pair of each axis
  double turns[MAX_D / 2];        // theta^(-2 i / d) / (2 pi) of each pair
};

// LANES: threads of one head, eight elements each (8 LANES >= D).
// PAIRS: pairs (2p, 2p + 1), else (p, p + R / 2).
template <bool BF16, int LANES, bool PAIRS>
__global__ void __launch_bounds__(THREADS, 3) rope_qk_kernel(const __grid_constant__ Params p) {
  constexpr int HEADS = 32 / LANES;   // heads a pass of the warp covers
  extern __shared__ __align__(128) uint8_t ring[];       // [WARPS][RING][UNIT_BYTES]
  __shared__ __align__(16) float2 cs_all[WARPS][MAX_D / 2];   // cos, sin of the warp's token
  __shared__ __align__(8) uint64_t bars[WARPS][RING];
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  const uint32_t head_bytes = 2u * p.D;
  const uint32_t ring_s = smem_u32(ring) + warp * (RING * UNIT_BYTES), bar = smem_u32(bars[warp]);
  float2* cs = cs_all[warp];
  if (lane == 0) {
    for (int i = 0; i < RING; ++i) mbar_init(bar + 8 * i, 1);
    fence_mbar_init();
  }
  __syncwarp();
  griddep_wait();
  griddep_launch_dependents();

  const int64_t total = static_cast<int64_t>(p.T) * p.parts;
  const int64_t u0 = (static_cast<int64_t>(blockIdx.x) * WARPS + warp) * p.units_per_warp;
  if (u0 >= total) return;
  const int units = static_cast<int>(min(static_cast<int64_t>(p.units_per_warp), total - u0));
  int t = static_cast<int>(u0 / p.parts), part = static_cast<int>(u0 % p.parts);

  // Requests units in order; (ft, fp) is the next one.
  int fetched = 0, ft = t, fp = part;
  auto fetch = [&]() {
    const bool is_q = fp < p.parts_q;
    const int h0 = is_q ? fp * p.heads_q : (fp - p.parts_q) * p.heads_k;
    const int n = is_q ? min(p.heads_q, p.Hq - h0) : min(p.heads_k, p.Hk - h0);
    const int64_t sh = is_q ? p.qsh : p.ksh;
    const uint16_t* src = (is_q ? p.q + ft * p.qst : p.k + ft * p.kst) + h0 * sh;
    const uint32_t b = bar + 8 * (fetched % RING), at = ring_s + (fetched % RING) * UNIT_BYTES;
    if (lane == 0) mbar_arrive_expect_tx(b, n * head_bytes);
    __syncwarp();
    if (sh == p.D) {
      if (lane == 0) bulk_load(at, src, n * head_bytes, b);
    } else {
      for (int h = lane; h < n; h += 32) bulk_load(at + h * head_bytes, src + h * sh, head_bytes, b);
    }
    ++fetched;
    if (++fp == p.parts) fp = 0, ++ft;
  };
  for (int i = 0; i < min(units, RING); ++i) fetch();

  const int j = lane % LANES;   // place in the head
  const int head0 = lane / LANES;
  // The lane's eight elements: pairs 4 j .. 4 j + 3, which are eight in a row,
  // or (halves) four in a row at `lo` and their partners at `hi`; from the
  // rotated part's end on, eight in a row.
  const bool turned = PAIRS || 4 * j < p.half;
  const int lo = PAIRS ? 8 * j : turned ? 4 * j : 2 * p.half + 8 * (j - p.half / 4);
  const int hi = PAIRS ? 8 * j + 4 : turned ? 4 * j + p.half : lo + 4;
  const bool in = lo < p.D;
  const bool straight = 4 * j + 4 > p.half;   // has elements past the rotated part
  auto word = [&](const uint16_t* w) {
    if (!w || !in) return make_uint4(0u, 0u, 0u, 0u);
    const uint2 a = *reinterpret_cast<const uint2*>(w + lo), b = *reinterpret_cast<const uint2*>(w + hi);
    return make_uint4(a.x, a.y, b.x, b.y);
  };
  const uint4 wq = word(p.qw), wk = word(p.kw);

  // Elements e0[e], e1[e] of pair e among the lane's eight.
  constexpr int STEP = PAIRS ? 2 : 1, OTHER = PAIRS ? 1 : 4;

  // The n heads of a unit.
  auto heads = [&](auto norm_tag, const uint4& wv, uint32_t src, uint16_t* dst, int64_t dh, int n) {
    constexpr bool NORM = decltype(norm_tag)::value;
    float w[8];
    unpack8<BF16>(wv, w);
    // e0' = a0 e0 - b1 e1, e1' = b0 e0 + a1 e1, the weights folded in
    float a0[4], a1[4], b0[4], b1[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 v = 4 * j + e < p.half ? cs[4 * j + e] : make_float2(1.f, 0.f);
      const float w0 = NORM ? w[STEP * e] : 1.f, w1 = NORM ? w[STEP * e + OTHER] : 1.f;
      a0[e] = v.x * w0;
      a1[e] = v.x * w1;
      b0[e] = v.y * w0;
      b1[e] = -v.y * w1;
    }
    src += head0 * head_bytes;
    dst += head0 * dh;
    dh *= HEADS;
#pragma unroll 2
    for (int h = head0; h < n + head0; h += HEADS) {   // whole passes: all lanes take part
      const bool here = in && h < n;
      uint4 raw = make_uint4(0u, 0u, 0u, 0u);
      if (here) {
        if (PAIRS) {
          ld_shared_v4(src + 2 * lo, raw.x, raw.y, raw.z, raw.w);
        } else {
          ld_shared_v2(src + 2 * lo, raw.x, raw.y);
          ld_shared_v2(src + 2 * hi, raw.z, raw.w);
        }
      }
      src += HEADS * head_bytes;
      float v[8], o[8];
      unpack8<BF16>(raw, v);
      if (NORM) {
        float q = 0.f, q1 = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          q = fmaf(v[e], v[e], q);
          q1 = fmaf(v[4 + e], v[4 + e], q1);
        }
        q += q1;
#pragma unroll
        for (int k = LANES / 2; k > 0; k >>= 1) q += __shfl_xor_sync(0xFFFFFFFFu, q, k);
        const float r = rsqrtf(fmaf(q, p.inv_d, p.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= r;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float e0 = v[STEP * e], e1 = v[STEP * e + OTHER];
        o[STEP * e] = fmaf(e1, b1[e], e0 * a0[e]);
        o[STEP * e + OTHER] = fmaf(e0, b0[e], e1 * a1[e]);
      }
      if (straight) {   // past the rotated part: whatever the neighbour holds
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (4 * j + (PAIRS ? e >> 1 : e & 3) >= p.half) o[e] = NORM ? v[e] * w[e] : v[e];
      }
      if (here) {
        const uint4 r = pack8<BF16>(o);
        if (PAIRS) {
          *reinterpret_cast<uint4*>(dst + lo) = r;
        } else {
          *reinterpret_cast<uint2*>(dst + lo) = make_uint2(r.x, r.y);
          *reinterpret_cast<uint2*>(dst + hi) = make_uint2(r.z, r.w);
        }
      }
      dst += dh;
    }
  };

  int have = -1;   // the token whose angles are in cs
  bool ok = true;
  for (int i = 0; i < units; ++i) {
    if (t != have) {
      have = t;
      for (int c = lane; c < p.half; c += 32) {
        int a = 0;
#pragma unroll
        for (int b = 1; b < MAX_AXES; ++b) a += b < p.axes && c >= p.first[b] ? 1 : 0;
        const double turn = static_cast<double>(p.pos[t * p.ldpos + a]) * p.turns[c];
        float2 v;
        sincospif(2.f * static_cast<float>(turn - rint(turn)), &v.y, &v.x);
        cs[c] = v;
      }
      __syncwarp();
    }
    ok = __all_sync(0xFFFFFFFFu, svdq_wait(bar + 8 * (i % RING), (i / RING) & 1u, SITE_UNIT));
    if (!ok) break;
    const uint32_t at = ring_s + (i % RING) * UNIT_BYTES;
    if (part < p.parts_q) {
      const int h0 = part * p.heads_q, n = min(p.heads_q, p.Hq - h0);
      uint16_t* dst = p.qo + t * p.qost + h0 * p.qosh;
      if (p.qw)
        heads(Tag<true>(), wq, at, dst, p.qosh, n);
      else
        heads(Tag<false>(), wq, at, dst, p.qosh, n);
    } else {
      const int h0 = (part - p.parts_q) * p.heads_k, n = min(p.heads_k, p.Hk - h0);
      uint16_t* dst = p.ko + t * p.kost + h0 * p.kosh;
      if (p.kw)
        heads(Tag<true>(), wk, at, dst, p.kosh, n);
      else
        heads(Tag<false>(), wk, at, dst, p.kosh, n);
    }
    __syncwarp();   // the slot and the angles have been read
    if (fetched < units) fetch();
    if (++part == p.parts) part = 0, ++t;
  }
  // After an error: what was requested lands before the block exits.
  for (int i = max(0, fetched - RING); i < fetched; ++i)
    drain_wait(bar + 8 * (i % RING), (i / RING) & 1u, 50000000ull);
}

}  // namespace kp
}  // namespace svdq
