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
// once per block and sequence instead of once per row.  Rows of x and y come
// by bulk copies into a ring in shared memory, four rows ahead, which takes
// no registers and no load instructions; the statistics of a row's branch
// are summed together with those of the previous row's h, so that a row
// costs one block barrier.  Calls in a row: 4352 rows x 3840 (134 MB) 27.0 us, 4.95
// TB/s, 77% of a plain copy's rate; 17408 rows with layer norm (two barriers a
// row) 98-99 us, 5.4 TB/s, 84%; as a graph 24.8 and 95 us.  In short runs, 26.3 us
// then: loads one row ahead into registers 29.6 us, a warp per row (no barrier,
// but 255 registers and spills) 38.
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

// A truth value as an argument's type.
template <bool B>
struct Tag {
  static constexpr bool value = B;
};

namespace kn {

constexpr int MAX_THREADS = 512;
constexpr int RING = 4;                           // rows of x and y on their way
constexpr int MAX_VPT = 2;                        // 8-element words per thread
constexpr int MAX_C = MAX_THREADS * MAX_VPT * 8;  // 8192

constexpr uint32_t SITE_ROW = 0x60;

enum Norm { NORM_NONE = 0, NORM_RMS = 1, NORM_LAYER = 2 };
enum Gate { GATE_NONE = 0, GATE_LINEAR = 1, GATE_TANH = 2 };

// Shared memory of the ring for C columns, with or without a branch.
constexpr size_t ring_bytes(int C, bool has_y) {
  return static_cast<size_t>(RING) * C * 2 * (has_y ? 2 : 1);
}

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

// Sums over the block of N values per thread, the same in every thread and
// every run (fixed order).  `buf` alternates so that one barrier is enough;
// the words of absent warps hold zero.
struct Red {
  float v[2][2][16];   // [buffer][value][warp]
};
__device__ __forceinline__ void block_sums(float& a, float& b, Red& red, int& buf, int warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
  }
  float (*r)[16] = red.v[buf];
  buf ^= 1;
  if ((threadIdx.x & 31) == 0) {
    r[0][threadIdx.x >> 5] = a;
    r[1][threadIdx.x >> 5] = b;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const ulonglong2* r2 = reinterpret_cast<const ulonglong2*>(r[k]);
    uint64_t s = add2(add2(r2[0].x, r2[0].y), add2(r2[1].x, r2[1].y));
    if (warps > 8) s = add2(s, add2(add2(r2[2].x, r2[2].y), add2(r2[3].x, r2[3].y)));
    float lo, hi;
    upk(s, lo, hi);
    (k ? b : a) = lo + hi;
  }
}

template <bool BF16, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 256 : MAX_THREADS, VPT == 1 ? 4 : 1)
    norm_gate_kernel(const Params p) {
  // [RING] rows of x, then of y; a row's slot is refilled RING rows later.
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(16) Red red;
  __shared__ __align__(8) uint64_t bars[RING];
  const int lane = threadIdx.x & 31;
  const int warps = blockDim.x >> 5;
  const bool has_y = p.y != nullptr;
  const uint32_t row_bytes = static_cast<uint32_t>(p.C) * 2u;
  const uint32_t x_s = smem_u32(ring), y_s = x_s + RING * row_bytes, bar = smem_u32(bars);
  int buf = 0;
  for (int i = threadIdx.x; i < 64; i += blockDim.x) red.v[i >> 5][(i >> 4) & 1][i & 15] = 0.f;
  if (threadIdx.x == 0) {
    for (int i = 0; i < RING; ++i) mbar_init(bar + 8 * i, 1);
    fence_mbar_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();

  const int row0 = static_cast<int>(blockIdx.x) * p.rows_per_block;
  const int row1 = min(p.T, row0 + p.rows_per_block);
  const int rows = row1 - row0;
  int fetched = 0;            // by thread 0
  auto fetch = [&]() {        // the next row, by thread 0
    const int i = fetched++;
    const uint32_t b = bar + 8 * (i % RING);
    mbar_arrive_expect_tx(b, has_y ? 2 * row_bytes : row_bytes);
    bulk_load(x_s + (i % RING) * row_bytes, p.x + (row0 + i) * p.ldx, row_bytes, b);
    if (has_y) bulk_load(y_s + (i % RING) * row_bytes, p.y + (row0 + i) * p.ldy, row_bytes, b);
  };
  if (threadIdx.x == 0)
    for (int i = 0; i < min(rows, RING); ++i) fetch();

  int col[VPT];
  bool in[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    col[i] = 8 * (static_cast<int>(threadIdx.x) + i * static_cast<int>(blockDim.x));
    in[i] = col[i] < p.C;
  }
  // The sequence of the current row and its first and last row.
  int s = p.cu ? find_sequence(p.cu, p.S, row0, lane) : 0;
  int seq_end = p.cu ? (s < p.S ? p.cu[s + 1] : row0) : p.T;
  int seq_begin = p.cu && s < p.S ? p.cu[s] : 0;
  bool fresh = false;   // another sequence's vectors are in the registers

  // gate x post weight, pre weight x (1 + scale), shift
  uint64_t gw[VPT][4], sw[VPT][4], sb[VPT][4];
  const uint64_t a2 = pk(p.a, p.a);
  const bool layer = p.pre == NORM_LAYER || p.post == NORM_LAYER;

  // All of a sequence's loads first, then what is made of them.
  auto load_vectors = [&]() {
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    uint4 vg[VPT], vp[VPT], vs[VPT], vq[VPT], vb[VPT];
    auto word = [&](const uint16_t* ptr, int64_t at, int k) {
      return ptr && in[k] ? *reinterpret_cast<const uint4*>(ptr + at + col[k]) : zero;
    };
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      vg[k] = word(p.gate, s * p.ldg, k);
      vp[k] = word(p.post_w, 0, k);
      vs[k] = word(p.scale, s * p.lds, k);
      vq[k] = word(p.pre_w, 0, k);
      vb[k] = word(p.shift, s * p.ldb, k);
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float g[8], w[8], b[8], t[8];
      unpack8<BF16>(vg[k], g);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        g[e] = p.gate_kind == GATE_NONE ? 1.f : p.gate_kind == GATE_TANH ? tanhf(g[e]) : g[e];
      if (p.post_w) {
        unpack8<BF16>(vp[k], t);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] *= t[e];
      }
      unpack8<BF16>(vs[k], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] += 1.f;
      if (p.pre_w) {
        unpack8<BF16>(vq[k], t);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] *= t[e];
      }
      unpack8<BF16>(vb[k], b);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        gw[k][e] = pk(g[2 * e], g[2 * e + 1]);
        sw[k][e] = pk(w[2 * e], w[2 * e + 1]);
        sb[k][e] = pk(b[2 * e], b[2 * e + 1]);
      }
    }
  };
  if (s < p.S) load_vectors();   // while the first rows are on their way

  auto row_words = [&](uint32_t at, uint64_t (&v)[VPT][4]) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (in[i]) ld_shared_v4(at + 2 * col[i], w.x, w.y, w.z, w.w);
      unpack4x2<BF16>(w, v[i]);
    }
  };
  auto sum = [&](const uint64_t (&v)[VPT][4]) {
    uint64_t t = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) t = add2(t, add2(add2(v[i][0], v[i][1]), add2(v[i][2], v[i][3])));
    float lo, hi;
    upk(t, lo, hi);
    return lo + hi;
  };
  auto squares = [&](const uint64_t (&v)[VPT][4]) {
    uint64_t t0 = 0, t1 = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      t0 = fma2(v[i][0], v[i][0], t0);
      t1 = fma2(v[i][1], v[i][1], t1);
      t0 = fma2(v[i][2], v[i][2], t0);
      t1 = fma2(v[i][3], v[i][3], t1);
    }
    float lo, hi;
    upk(add2(t0, t1), lo, hi);
    return lo + hi;
  };
  auto shift_by = [&](uint64_t (&v)[VPT][4], float m) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const uint64_t m2 = in[i] ? pk(m, m) : 0;   // columns behind the last stay zero
#pragma unroll
      for (int e = 0; e < 4; ++e) v[i][e] = add2(v[i][e], m2);
    }
  };
  // 1 / sqrt(mean square + eps) of h (pre) and of the next row's u (post), both
  // in one round of the block: a barrier per row, two with a layer norm
  // (whose mean is taken off first, so that a large one costs no digits).
  auto statistics = [&](uint64_t (&h)[VPT][4], uint64_t (&u)[VPT][4], float& rh, float& ru) {
    if (layer) {
      float a = p.pre == NORM_LAYER ? sum(h) : 0.f, b = p.post == NORM_LAYER ? sum(u) : 0.f;
      block_sums(a, b, red, buf, warps);
      if (p.pre == NORM_LAYER) shift_by(h, a * -p.inv_c);
      if (p.post == NORM_LAYER) shift_by(u, b * -p.inv_c);
    }
    float a = squares(h), b = squares(u);
    block_sums(a, b, red, buf, warps);
    rh = p.pre == NORM_NONE ? 1.f : rsqrtf(fmaf(a, p.inv_c, p.eps));
    ru = p.post == NORM_NONE ? 1.f : rsqrtf(fmaf(b, p.inv_c, p.eps));
  };
  auto landed = [&](int i) {
    return __all_sync(0xFFFFFFFFu, svdq_wait(bar + 8 * (i % RING), (i / RING) & 1u, SITE_ROW));
  };

  // u: the branch's row, its mean already off, one row ahead of h.
  uint64_t u[VPT][4], h[VPT][4];
  float rh = 1.f, ru = 1.f;
  bool ok = landed(0);
  if (ok && has_y) {
    row_words(y_s, u);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) h[i][e] = 0;
    if (p.post != NORM_NONE) statistics(h, u, rh, ru);
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) u[i][e] = 0;
  }
  for (int i = 0; ok && i < rows; ++i) {
    const int row = row0 + i;
    while (p.cu && s < p.S && row >= seq_end) {
      ++s;
      if (s < p.S) {
        seq_begin = p.cu[s];
        seq_end = p.cu[s + 1];
      }
      fresh = true;
    }
    if (s >= p.S) break;                    // this row and all behind it: no sequence
    const bool live = row >= seq_begin;     // not in front of the first sequence
    if (fresh) {
      fresh = false;
      load_vectors();
    }

    row_words(x_s + (i % RING) * row_bytes, h);
    if (has_y) {
      const uint64_t r2 = pk(ru, ru);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
#pragma unroll
        for (int e = 0; e < 4; ++e) h[k][e] = fma2(mul2(u[k][e], r2), gw[k][e], mul2(h[k][e], a2));
        if (in[k] && live) *reinterpret_cast<uint4*>(p.h + row * p.ldh + col[k]) = pack4x2<BF16>(h[k]);
      }
    }
    // The next row's branch, and the statistics of both.  Every thread has
    // read this row's slot before the barrier in there.
    if (i + 1 < rows) {
      ok = landed(i + 1);
      if (!ok) break;
      if (has_y) row_words(y_s + ((i + 1) % RING) * row_bytes, u);
    }
    statistics(h, u, rh, ru);
    if (threadIdx.x == 0 && fetched < rows) fetch();   // row i + RING, into this row's slot
    if (p.n) {
      const uint64_t r2 = pk(rh, rh);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
#pragma unroll
        for (int e = 0; e < 4; ++e) h[k][e] = fma2(mul2(h[k][e], r2), sw[k][e], sb[k][e]);
        if (in[k] && live) *reinterpret_cast<uint4*>(p.n + row * p.ldn + col[k]) = pack4x2<BF16>(h[k]);
      }
    }
  }
  // Rows fetched and not waited for (rows in no sequence, an error) land
  // before the block exits.
  if (threadIdx.x == 0)
    for (int i = max(0, fetched - RING); i < fetched; ++i)
      drain_wait(bar + 8 * (i % RING), (i / RING) & 1u, 50000000ull);
}

}  // namespace kn
}  // namespace svdq
