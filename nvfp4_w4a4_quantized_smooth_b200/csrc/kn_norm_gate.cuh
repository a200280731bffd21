// kn_norm_gate.cuh -- the norms before and after a transformer block, fused
// with the block's gate and residual scale:
//
//   u = post(y)                             (post: none, RMS or layer norm)
//   h = a x + g u                           (g: 1, gate[s] or tanh(gate[s]))
//   n = pre(h) (1 + scale[s]) + shift[s]    (pre: none, RMS or layer norm)
//
// for every row of the packed sequences, s the row's sequence.  x, y, h and n
// are bf16 or fp16; everything between is fp32, n is computed from the
// unrounded h, and h and n are rounded once.
//
// Bound by memory: a row is read once (x, y) and written once (h, n).  One
// block owns a run of consecutive rows and keeps what belongs to the
// sequence (gate x weight, weight x (1 + scale), shift: fp32) in registers
// until the sequence changes, so that tanh and the modulation rows are read
// once per block and sequence instead of once per row; the next row's x and
// y are requested before the current row's statistics are summed.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sm100_ptx.cuh"

namespace svdq {

// Eight 16-bit elements (a 16-byte word) -> fp32.
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& w, float (&f)[8]) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      f[2 * i] = __uint_as_float(v[i] << 16);
      f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    } else {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
}

// The same as four packed pairs.
template <bool BF16>
__device__ __forceinline__ void unpack4x2(const uint4& w, uint64_t (&f)[4]) {
  float t[8];
  unpack8<BF16>(w, t);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = pk(t[2 * i], t[2 * i + 1]);
}

// Two fp32 -> a pair of 16-bit elements, nearest-even (lo in the low half).
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2<BF16>(f[0], f[1]), pack2<BF16>(f[2], f[3]), pack2<BF16>(f[4], f[5]),
                    pack2<BF16>(f[6], f[7]));
}

template <bool BF16>
__device__ __forceinline__ uint4 pack4x2(const uint64_t (&f)[4]) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    upk(f[i], lo, hi);
    r[i] = pack2<BF16>(lo, hi);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// 16 bytes that this kernel reads once (not kept in L1).  Plain loads, not
// the read-only path: the buffer may be the output's.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

namespace kn {

constexpr int MAX_THREADS = 512;
constexpr int MAX_VPT = 2;                        // 8-element words per thread
constexpr int MAX_C = MAX_THREADS * MAX_VPT * 8;  // 8192

enum Norm { NORM_NONE = 0, NORM_RMS = 1, NORM_LAYER = 2 };
enum Gate { GATE_NONE = 0, GATE_LINEAR = 1, GATE_TANH = 2 };

struct Params {
  const uint16_t *x, *y, *gate, *scale, *shift, *post_w, *pre_w;
  uint16_t *h, *n;
  const int32_t* cu;   // [S + 1] or NULL: one sequence of all rows
  int64_t ldx, ldy, ldh, ldn, ldg, lds, ldb;
  int T, C, S;
  int post, pre, gate_kind;
  float a, eps, inv_c;
  int rows_per_block;
};

// Sequence of `row`: the number of entries of cu[1..S] that are <= row
// (S if the row is behind the last sequence).  Whole warp, 32 probes a step;
// stays inside cu whatever it holds.
__device__ __forceinline__ int find_sequence(const int32_t* cu, int S, int row, int lane) {
  int lo = 0, hi = S;   // the answer is in [lo, hi]
  while (lo < hi) {
    const int span = hi - lo;
    const int step = (span + 31) / 32;
    const int at = lo + (lane + 1) * step;   // probe: are the first `at` ends all <= row?
    const bool past = at <= hi && cu[at] <= row;
    const int n = __popc(__ballot_sync(0xFFFFFFFFu, past));
    // ends are non-decreasing, so the lanes that say yes are the first n
    lo += n * step;
    hi = lo + step - 1 < hi ? lo + step - 1 : hi;
  }
  return lo;
}

// Sum over the block of one value per thread, the same in every thread and
// every run (fixed order).  `buf` alternates so that one barrier is enough;
// the words of absent warps hold zero.
__device__ __forceinline__ float block_sum(float v, float (*red)[16], int& buf, int warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (warps == 1) return v;
  float* r = red[buf];
  buf ^= 1;
  if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
  __syncthreads();
  const ulonglong2* r2 = reinterpret_cast<const ulonglong2*>(r);
  uint64_t s = add2(add2(r2[0].x, r2[0].y), add2(r2[1].x, r2[1].y));
  if (warps > 8) s = add2(s, add2(add2(r2[2].x, r2[2].y), add2(r2[3].x, r2[3].y)));
  float lo, hi;
  upk(s, lo, hi);
  return lo + hi;
}

template <bool BF16, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 256 : MAX_THREADS, VPT == 1 ? 4 : 1) norm_gate_kernel(const Params p) {
  __shared__ __align__(16) float red[2][16];
  const int lane = threadIdx.x & 31;
  const int warps = blockDim.x >> 5;
  int buf = 0;
  if (threadIdx.x < 32) red[threadIdx.x >> 4][threadIdx.x & 15] = 0.f;
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const int row0 = static_cast<int>(blockIdx.x) * p.rows_per_block;
  const int row1 = min(p.T, row0 + p.rows_per_block);
  if (row0 >= row1) return;

  int col[VPT];
  bool in[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    col[i] = 8 * (static_cast<int>(threadIdx.x) + i * static_cast<int>(blockDim.x));
    in[i] = col[i] < p.C;
  }
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const bool has_y = p.y != nullptr;

  // The sequence of the current row and its first and last row.
  int s = p.cu ? find_sequence(p.cu, p.S, row0, lane) : 0;
  int seq_end = p.cu ? (s < p.S ? p.cu[s + 1] : row0) : p.T;
  int seq_begin = p.cu && s < p.S ? p.cu[s] : 0;
  bool fresh = true;   // the sequence's vectors are not in registers yet

  // gate x post weight, pre weight x (1 + scale), shift
  uint64_t gw[VPT][4], sw[VPT][4], sb[VPT][4];
  uint4 xv[VPT], yv[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    xv[i] = in[i] ? ld_stream(p.x + row0 * p.ldx + col[i]) : zero;
    yv[i] = in[i] && has_y ? ld_stream(p.y + row0 * p.ldy + col[i]) : zero;
  }
  const uint64_t a2 = pk(p.a, p.a);

  // Takes the mean off (layer norm: two passes over the registers, so that a
  // large mean costs no digits) and returns 1 / sqrt(mean square + eps).
  auto normalize = [&](uint64_t (&v)[VPT][4], int kind) {
    if (kind == NORM_LAYER) {
      uint64_t t = 0;   // (0, 0); columns behind the last one hold zeros
#pragma unroll
      for (int i = 0; i < VPT; ++i) t = add2(t, add2(add2(v[i][0], v[i][1]), add2(v[i][2], v[i][3])));
      float lo, hi;
      upk(t, lo, hi);
      const float m = block_sum(lo + hi, red, buf, warps) * -p.inv_c;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const uint64_t m2 = in[i] ? pk(m, m) : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] = add2(v[i][e], m2);
      }
    }
    uint64_t q = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) q = fma2(v[i][e], v[i][e], q);
    float lo, hi;
    upk(q, lo, hi);
    return rsqrtf(fmaf(block_sum(lo + hi, red, buf, warps), p.inv_c, p.eps));
  };

  for (int row = row0; row < row1; ++row) {
    while (p.cu && s < p.S && row >= seq_end) {
      ++s;
      if (s < p.S) {
        seq_begin = p.cu[s];
        seq_end = p.cu[s + 1];
      }
      fresh = true;
    }
    uint64_t u[VPT][4], h[VPT][4];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      unpack4x2<BF16>(yv[i], u[i]);
      unpack4x2<BF16>(xv[i], h[i]);
    }
    if (row + 1 < row1) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (in[i]) {
          xv[i] = ld_stream(p.x + (row + 1) * p.ldx + col[i]);
          if (has_y) yv[i] = ld_stream(p.y + (row + 1) * p.ldy + col[i]);
        }
      }
    }
    if (s >= p.S) break;             // this row and all behind it: no sequence
    if (row < seq_begin) continue;   // in front of the first sequence
    if (fresh) {
      fresh = false;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        float g[8], w[8], b[8], t[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = 1.f, w[e] = 1.f, b[e] = 0.f;
        if (in[i]) {
          if (p.gate_kind != GATE_NONE) {
            unpack8<BF16>(*reinterpret_cast<const uint4*>(p.gate + s * p.ldg + col[i]), g);
            if (p.gate_kind == GATE_TANH) {
#pragma unroll
              for (int e = 0; e < 8; ++e) g[e] = tanhf(g[e]);
            }
          }
          if (p.post_w) {
            unpack8<BF16>(*reinterpret_cast<const uint4*>(p.post_w + col[i]), t);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] *= t[e];
          }
          if (p.scale) {
            unpack8<BF16>(*reinterpret_cast<const uint4*>(p.scale + s * p.lds + col[i]), t);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] += t[e];
          }
          if (p.pre_w) {
            unpack8<BF16>(*reinterpret_cast<const uint4*>(p.pre_w + col[i]), t);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] *= t[e];
          }
          if (p.shift) unpack8<BF16>(*reinterpret_cast<const uint4*>(p.shift + s * p.ldb + col[i]), b);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          gw[i][e] = pk(g[2 * e], g[2 * e + 1]);
          sw[i][e] = pk(w[2 * e], w[2 * e + 1]);
          sb[i][e] = pk(b[2 * e], b[2 * e + 1]);
        }
      }
    }

    if (has_y) {
      const float r = p.post == NORM_NONE ? 1.f : normalize(u, p.post);
      const uint64_t r2 = pk(r, r);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) h[i][e] = fma2(mul2(u[i][e], r2), gw[i][e], mul2(h[i][e], a2));
        if (in[i]) *reinterpret_cast<uint4*>(p.h + row * p.ldh + col[i]) = pack4x2<BF16>(h[i]);
      }
    }
    if (p.n) {
      const float r = p.pre == NORM_NONE ? 1.f : normalize(h, p.pre);
      const uint64_t r2 = pk(r, r);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (!in[i]) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[i][e] = fma2(mul2(h[i][e], r2), sw[i][e], sb[i][e]);
        *reinterpret_cast<uint4*>(p.n + row * p.ldn + col[i]) = pack4x2<BF16>(h[i]);
      }
    }
  }
}

}  // namespace kn
}  // namespace svdq
