// ka_attention.cuh -- attention over whole packed sequences:
//
//   out_i = sum_j w_ij v_j,  w_ij = softmax_j(scale q_i . k_j),
//
// j over the keys of row i's sequence (full), or over j <= i (causal); query
// head h reads key / value head h / (Hq / Hk).
//
// One work item is 256 query rows of one head (two slots of 128 rows, the
// tensor core's row count) against all key tiles of 128 they attend.  Per
// key tile and slot: S = Q K^T into TMEM (fp32), one softmax step by the
// slot's four warps (one thread per row, so no shuffles), P back into the
// same TMEM columns as 16-bit values, O += P V with P read from TMEM.  Each
// slot has its own warp that issues its products, so that while one slot's
// warps work on their tile the tensor core runs the other slot's, and K and V
// tiles pass both slots from one ring in shared memory.
//
// The softmax keeps a running reference m (log2 units after the scale), sum
// and O relative to it.  O is rescaled only when a row's maximum has grown by
// more than 2^8 over its reference: until then the weights stay below 2^8
// times the reference's.  P is rounded to the input type for the tensor core;
// the sum is over the unrounded fp32 weights.  bf16 has fp32's exponents, so
// a weight is off by half a step (2^-8 of it) however small it is, and the
// reference weight is 1.  fp16 ends at 65504 and loses digits below 2^-14,
// everything at 2^-25: there the reference weight is 2^7, the largest one
// then 2^15, and a weight is off by 2^-11 of itself or, where that is less, by
// 2^-32 of the reference weight (with a reference of 1, 2^-25: weak keys
// beside a strong one lost a visible share of their mass).  The tensor core
// cuts O off at fp32's last place once per 16 keys, where the sum of the
// weights is rounded: values of one sign lose up to 2^-27 per key (measured at
// 65536 keys 0.0004, at 262144 0.0017).
//
// Keys that a row does not attend are replaced by -inf after the product, by
// selection, so what they hold does not matter.  Values need more, since a
// zero weight times inf or NaN is NaN: the tile behind a sequence's end
// holds other rows, and on the causal diagonal a tile holds values that some
// of its rows do not attend.  For these tiles alone a guard warp zeroes the
// rows behind the end (only up to the next multiple of 16; the product stops
// there) and, when causal, replaces non-finite values by zero and notes their
// keys; the epilogue adds a noted value back into the rows that do attend it.
//
// Bound: per key tile and 256 rows the tensor core has 2048 cycles of products
// (D = 128) and the special function units 2048 cycles of exponentials; a
// slot's tile is a chain of both (about 1350 cycles from S to P, 1500 from P
// to the next S), so two slots in turns need about 2800.  At 4352 rows x 30
// heads of 128: 280 us a call in runs of a second (1040 TFLOP/s, 62% of what a
// cuBLAS product of 8192^3 reaches alone), where the GPU is at its power limit
// and lowers the clock (cuBLAS then: 1403 TFLOP/s); 241 us in runs of some
// milliseconds.  What was
// tried against that: exponentials by a polynomial on the FMA units (1/8 of
// them: 307 us, more: slower still), handing over half of P first (286 against
// 250), five stages of the ring (1083 us against 974 at four times the rows).
//
// The outline is that of published work: the running maximum and sum of a
// softmax (Milakov and Gimelshein, 2018), both products tile by tile on the
// chip around it (Rabe and Staats, 2021; Dao et al., 2022), and for this
// GPU's tensor memory two query tiles in turns with rescaling only where a
// maximum has grown much.  The walk over the work items, the guard, the turns
// and the join are this file's own.
#pragma once

#include <climits>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kn_norm_gate.cuh"
#include "sm100_ptx.cuh"

namespace svdq {
namespace ka {

constexpr int ROWS = 128;               // query rows of a slot, keys of a tile
constexpr int ITEM_ROWS = 2 * ROWS;     // query rows of a work item
constexpr int MAX_D = 128;
constexpr int NUM_THREADS = 384;        // 2 x 4 softmax warps, 2 MMA, TMA, guard
constexpr int MMA_WARP = 8, TMA_WARP = 10, GUARD_WARP = 11;
constexpr uint32_t BOX_BYTES = ROWS * 128;   // 128 rows x 64 elements, 128-byte swizzle
constexpr uint32_t TMEM_COLS = 512;
constexpr int ITEMS = 4;                // work items that the warps are told in advance
constexpr uint32_t TM_S = 0;            // S / P of slot s at 128 s
constexpr uint32_t TM_O = 256;          // O of slot s at 256 + 128 s
constexpr int MIN_RUN = 6;               // places of a block's run, at least (split)
constexpr int P_STEPS = 6;              // 16-key steps of P that are handed over first
constexpr float RESCALE_LOG2 = 8.f;
// Of the weight of a key that scores a row's reference.
template <bool BF16>
constexpr float REF_LOG2 = BF16 ? 0.f : 7.f;
// Registers per thread of the softmax warps and of the others: all that the
// block has (384 x 168).  At 4352 x 30 heads, in short runs, 237 us, 250 with
// 216 / 72 or 224 / 56.
constexpr int SOFTMAX_REGS = 208, OTHER_REGS = 88;

// NB: 64-element boxes per row (1: D <= 64, 2: D <= 128).
template <int NB>
struct Shape {
  static constexpr uint32_t TILE_BYTES = NB * BOX_BYTES;
  static constexpr int STAGES = NB == 2 ? 4 : 8;
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_KV = 2 * TILE_BYTES;
  // A warp's 32 rows x 128 bytes on the way out.
  static constexpr uint32_t OFF_OUT = OFF_KV + STAGES * TILE_BYTES;
  static constexpr uint32_t OFF_BAR = OFF_OUT + 8 * 4096;
  // full, empty, guard_go, guard_done [STAGES], q_full, q_empty, s_full[2],
  // p_full[2], p_rest[2], o_full[2], flags_full[2], flags_free[2], final[2],
  // turn[2], item_full[ITEMS], item_empty[ITEMS]
  static constexpr int BARS = 4 * STAGES + 18 + 2 * ITEMS;
  // Notes of the guard, one bit per key: [item parity][8 words].
  static constexpr uint32_t OFF_FLAGS = OFF_BAR + 8 * BARS;
  static constexpr uint32_t OFF_TMEM = OFF_FLAGS + 2 * 8 * 4;
  static constexpr uint32_t OFF_ITEMS = OFF_TMEM + 16;   // 32 bytes each
  static constexpr uint32_t USED = OFF_ITEMS + 32 * ITEMS;
  static constexpr uint32_t SMEM_BYTES = USED + 1024;   // 1024-byte alignment of the boxes
};
static_assert(Shape<2>::SMEM_BYTES <= 232448 && Shape<1>::SMEM_BYTES <= 232448, "");

constexpr uint32_t SITE_TMA_Q = 0x50, SITE_TMA_KV = 0x51, SITE_MMA_Q = 0x52, SITE_MMA_KV = 0x53,
                   SITE_MMA_P = 0x54, SITE_MMA_GUARD = 0x55, SITE_SOFT_S = 0x56,
                   SITE_SOFT_O = 0x57, SITE_GUARD_V = 0x58, SITE_GUARD_FLAGS = 0x59,
                   SITE_SOFT_FLAGS = 0x5A, SITE_MMA_TURN = 0x5B, SITE_ITEM = 0x5C,
                   SITE_TMA_ITEM = 0x5D;

// What a block leaves of an item that it has only some key tiles of: a row's
// reference, sum and unscaled O in the workspace, and this.
struct Meta {
  int valid, last;          // last: up to the item's last key tile
  int begin, len, q0, head;
  int pad[2];
};

// Workspace of a launch of `blocks`: two partial results per block (an item
// begun by the block in front, an item left to the one behind).
struct Workspace {
  float* o;                 // [2 blocks][256][dp]
  float2* ml;               // [2 blocks][256]  reference, sum
  Meta* meta;               // [2 blocks]
  static constexpr size_t bytes(int blocks, int dp) {
    return static_cast<size_t>(2) * blocks * (ITEM_ROWS * (4u * dp + 8u) + sizeof(Meta));
  }
};

struct Params {
  const int32_t* cu;        // [S + 1] or NULL: one sequence of all T rows
  const uint16_t* v;        // for the non-finite values' way back
  uint16_t* out;
  int64_t vst, vsh, ost, osh;
  int T, S, Hq, group, D;
  int causal;
  float scale_log2;         // scale * log2(e)
  Workspace ws;             // items divided among the blocks
};

// One work item: rows [q0, q0 + 256) of the sequence [begin, begin + len),
// head h, and of its key tiles the range [ka, kb).
struct Item {
  int begin, len, q0, head, ka, kb;
  __device__ __forceinline__ int key_tiles() const { return (len + ROWS - 1) / ROWS; }
  // key tiles of slot s: it attends [0, tiles), and reads [ka, end) of them
  __device__ __forceinline__ int tiles(int s, int causal) const {
    if (q0 + s * ROWS >= len) return 0;
    const int n = key_tiles();
    return causal ? min(n, q0 / ROWS + s + 1) : n;
  }
  __device__ __forceinline__ int all_tiles(int causal) const {
    return max(tiles(0, causal), tiles(1, causal));
  }
  __device__ __forceinline__ int end(int s, int causal) const { return min(kb, tiles(s, causal)); }
  __device__ __forceinline__ bool whole(int causal) const { return ka == 0 && kb == all_tiles(causal); }
  // The first guarded value tile: the diagonal's (and all behind it), or the
  // last one where it ends inside 16 keys.
  __device__ __forceinline__ int guard_from(int causal) const {
    return max(ka, causal ? q0 / ROWS : len % 16 != 0 ? key_tiles() - 1 : INT_MAX);
  }
};

// Walks a block's work: one warp does and tells the others.  Sequence s is
// [e_s, e_s+1), e_s the largest of cu[0 .. s] clamped to [0, T]: offsets that
// do not fall are taken as they are, and whatever cu holds the sequences lie
// inside the tensors, do not meet, and have at most T rows together.
//
// Whole items: all items in a line, longest first (among the sequences of a
// group of 32), dealt to the blocks in rounds, every other round from the
// last block to the first, so that who had a longer item gets a shorter one
// next.  (Causal, in key tiles of the busiest SM, an item counted 1.5 more:
// 8192 rows x 8 heads 95 without the turning back, 66 with it, 60 if all were
// equal.)  Split: the items of all
// sequences lie in one line, each as long as its key tiles and one place more
// for what an item costs by itself, and the line is cut into equal runs, one
// per block.  (The host keeps the places below 2^31 and divides calls of at
// most 32 sequences, one group, in which places may be looked up in any order.)
template <bool SPLIT>
struct Items {
  int s0 = -32;                   // the present group of 32 sequences, one per lane:
  int begin_ = 0, len_ = 0;       //   its rows,
  int incl_ = 0, size_ = 0;       //   places up to its end (within the group), its places
  int base = 0, next_base = 0;    // places in front of the group, of the next
  int front = 0;                  // where the next group's rows begin, at least
  int class_ = 0, class_base = 0; // causal, whole: the item of a sequence that is being dealt
                                  //   out, places of the group in front of it
  int at = 0, end = 0;            // split: this block's run; whole: the round, and its direction

  // Of a sequence: items, or places of one head's items.
  static __device__ __forceinline__ int size(const Params& p, int len) {
    const int nt = (len + ITEM_ROWS - 1) / ITEM_ROWS;
    if (!SPLIT) return nt * p.Hq;
    const int nk = (len + ROWS - 1) / ROWS;
    // causal: 2, 4, 6, ... tiles, the last item one fewer where it has one slot
    return (p.causal ? nt * (nt + 2) - (2 * nt - nk) : nt * (nk + 1)) * p.Hq;
  }
  __device__ __forceinline__ bool next_group(const Params& p) {
    if (s0 + 32 >= p.S) return false;
    s0 += 32;
    base = next_base;
    const int lane = threadIdx.x & 31, s = s0 + lane;
    begin_ = 0;
    int stop = s < p.S && !p.cu ? p.T : 0;
    if (s < p.S && p.cu) {
      begin_ = min(max(p.cu[s], 0), p.T);
      stop = min(max(p.cu[s + 1], 0), p.T);
    }
    begin_ = max(begin_, front);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) begin_ = max(begin_, __shfl_up_sync(0xFFFFFFFFu, begin_, o));
    stop = max(stop, begin_);
    front = __shfl_sync(0xFFFFFFFFu, stop, 31);
    len_ = stop - begin_;
    if (!SPLIT && !p.causal && p.S > 1) longest_first(p);
    if (!SPLIT && p.causal) {
      class_base = 0;
      class_ = __reduce_max_sync(0xFFFFFFFFu, (len_ + ITEM_ROWS - 1) / ITEM_ROWS) - 1;
    }
    incl_ = size_ = size(p, len_);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xFFFFFFFFu, incl_, o);
      if (lane >= o) incl_ += t;
    }
    next_base = base + __shfl_sync(0xFFFFFFFFu, incl_, 31);
    return true;
  }
  // The group's sequences in order of their lengths, where there are more
  // items than blocks.
  __device__ __forceinline__ void longest_first(const Params& p) {
    const int lane = threadIdx.x & 31;
    if (__reduce_add_sync(0xFFFFFFFFu, size(p, len_)) <= static_cast<int>(gridDim.x)) return;
    int rank = 0;
    for (int s = 0; s < 32; ++s) {
      const int l = __shfl_sync(0xFFFFFFFFu, len_, s);
      rank += l > len_ || (l == len_ && s < lane);
    }
    int from = 0;
    for (int s = 0; s < 32; ++s)
      if (__shfl_sync(0xFFFFFFFFu, rank, s) == lane) from = s;
    begin_ = __shfl_sync(0xFFFFFFFFu, begin_, from);
    len_ = __shfl_sync(0xFFFFFFFFu, len_, from);
  }
  // The sequence that holds place w (which must not fall to an earlier group
  // from call to call): the place within it, -1 behind the last.
  __device__ __forceinline__ int find(const Params& p, int w, Item& it) {
    while (w >= next_base)
      if (!next_group(p)) return -1;
    const int src = __ffs(__ballot_sync(0xFFFFFFFFu, base + incl_ > w)) - 1;
    it.begin = __shfl_sync(0xFFFFFFFFu, begin_, src);
    it.len = __shfl_sync(0xFFFFFFFFu, len_, src);
    return w - base - __shfl_sync(0xFFFFFFFFu, incl_ - size_, src);
  }
  // Split: the item at place w, and w's place in it.
  __device__ __forceinline__ int locate(const Params& p, int w, Item& it) {
    const int r = find(p, w, it);
    if (r < 0) return -1;
    const int per = size(p, it.len) / p.Hq;
    it.head = r / per;
    const int r2 = r - it.head * per;
    if (p.causal) {
      // i (i + 2) places in front of item i
      int i = static_cast<int>(sqrtf(static_cast<float>(r2) + 1.f)) - 1;
      while (i > 0 && i * (i + 2) > r2) --i;
      while ((i + 1) * (i + 3) <= r2) ++i;
      it.q0 = i * ITEM_ROWS;
      return r2 - i * (i + 2);
    }
    const int n = it.key_tiles() + 1;
    it.q0 = r2 / n * ITEM_ROWS;
    return r2 % n;
  }
  // Where a run begins that should begin at w: at an item's edge where one is
  // near (two partial results less).  So no run begins at an item's last key
  // tile, and every part has one for each row of the item.
  __device__ __forceinline__ int edge(const Params& p, int w, int total, int run) {
    if (w >= total) return total;
    Item it;
    const int r = locate(p, w, it), n = it.all_tiles(p.causal) + 1;
    const int near = 1 + max(1, run / 16);
    return r <= near ? w - r : n - r < near ? w + n - r : w;
  }
  __device__ __forceinline__ void start(const Params& p) {
    if (!SPLIT) return;
    next_group(p);   // the only one
    const int total = next_base;
    const int run = max(MIN_RUN, (total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x));
    const int64_t w = static_cast<int64_t>(blockIdx.x) * run;
    end = edge(p, static_cast<int>(min(w + run, static_cast<int64_t>(total))), total, run);
    at = edge(p, static_cast<int>(min(w, static_cast<int64_t>(total))), total, run);
  }
  __device__ __forceinline__ bool get(const Params& p, Item& it) {
    if (SPLIT) {
      if (at >= end) return false;
      const int r = locate(p, at, it);
      if (r < 0) return false;
      const int n = it.all_tiles(p.causal);
      it.ka = max(0, r - 1);
      it.kb = min(n, end - at + r - 1);
      at += 1 + it.kb - r;
      return true;
    }
    // at: the round's first place; this block's is counted from either end
    const int G = static_cast<int>(gridDim.x), b = static_cast<int>(blockIdx.x);
    const int w = at + (end ? G - 1 - b : b);
    at += G;
    end ^= 1;
    if (p.causal) {
      // item i of every sequence that has one, then item i - 1, ...
      while (w >= next_base)
        if (!next_group(p)) return false;
      const int r = w - base;
      uint32_t has;
      int n;
      for (;;) {
        has = __ballot_sync(0xFFFFFFFFu, len_ > class_ * ITEM_ROWS);
        n = __popc(has) * p.Hq;
        if (r < class_base + n) break;
        class_base += n;
        --class_;
      }
      const int k = (r - class_base) / p.Hq;
      const int src = __fns(has, 0, k + 1);
      it.begin = __shfl_sync(0xFFFFFFFFu, begin_, src);
      it.len = __shfl_sync(0xFFFFFFFFu, len_, src);
      it.head = r - class_base - k * p.Hq;
      it.q0 = class_ * ITEM_ROWS;
    } else {   // the items of one head together: they read the same keys
      const int r = find(p, w, it);
      if (r < 0) return false;
      const int nt = (it.len + ITEM_ROWS - 1) / ITEM_ROWS;
      it.head = r / nt;
      it.q0 = (r % nt) * ITEM_ROWS;
    }
    it.ka = 0;
    it.kb = it.all_tiles(p.causal);
    return true;
  }
};

template <int N>
__device__ __forceinline__ void set_max_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_max_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <bool BF16>
__device__ __forceinline__ bool is_nonfinite16(uint32_t e) {
  constexpr uint32_t m = BF16 ? 0x7F80u : 0x7C00u;
  return (e & m) == m;
}

// The larger of a's halves and the magnitudes of b's, NaN if one is NaN.
template <bool BF16>
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  b &= 0x7FFF7FFFu;
  if (BF16)
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Replaces the non-finite values of the first `valid` rows of a tile by zero
// and notes their keys (it hardly ever runs).
template <bool BF16, int NB>
__device__ __forceinline__ void clean_tile(uint32_t tile, int valid, uint32_t* notes) {
  for (int b = 0; b < NB; ++b) {
    for (int c = threadIdx.x & 31; c < 8 * valid; c += 32) {
      const uint32_t at = tile + b * BOX_BYTES + 16 * c;
      uint32_t x[4];
      bool bad = false;
      ld_shared_v4(at, x[0], x[1], x[2], x[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (is_nonfinite16<BF16>(x[i])) x[i] &= 0xFFFF0000u, bad = true;
        if (is_nonfinite16<BF16>(x[i] >> 16)) x[i] &= 0x0000FFFFu, bad = true;
      }
      if (bad) {
        st_shared_v4(at, x[0], x[1], x[2], x[3]);
        atomicOr(notes + (c >> 8), 1u << ((c >> 3) & 31));
      }
    }
  }
}

template <bool BF16, int NB, bool SPLIT>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    attention_kernel(const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const Params p) {
  using S_ = Shape<NB>;
  constexpr int STAGES = S_::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  // (by shuffle: the compiler then knows it to be the same in all lanes)
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  auto bar = [&](int i) { return sb + S_::OFF_BAR + 8u * i; };
  auto full_bar = [&](uint32_t s) { return bar(s); };
  auto empty_bar = [&](uint32_t s) { return bar(STAGES + s); };
  // A guarded value tile goes TMA -> guards -> MMA.  Both steps have a
  // barrier per stage: a stage is not loaded again before the MMA has
  // passed, so its phases alternate one by one, however far ahead of one
  // another the three warps are with other stages.
  auto guard_go = [&](uint32_t s) { return bar(2 * STAGES + s); };
  auto guard_done = [&](uint32_t s) { return bar(3 * STAGES + s); };
  const uint32_t q_full = bar(4 * STAGES), q_empty = bar(4 * STAGES + 1);
  auto s_full = [&](int s) { return bar(4 * STAGES + 2 + s); };
  auto p_full = [&](int s) { return bar(4 * STAGES + 4 + s); };
  auto p_rest = [&](int s) { return bar(4 * STAGES + 6 + s); };
  auto o_full = [&](int s) { return bar(4 * STAGES + 8 + s); };
  auto flags_full = [&](int b) { return bar(4 * STAGES + 10 + b); };
  auto flags_free = [&](int b) { return bar(4 * STAGES + 12 + b); };
  const uint32_t final_bar = bar(4 * STAGES + 14);
  const uint32_t turn_bar = bar(4 * STAGES + 16);
  auto item_full = [&](uint32_t i) { return bar(4 * STAGES + 18 + i % ITEMS); };
  auto item_empty = [&](uint32_t i) { return bar(4 * STAGES + 18 + ITEMS + i % ITEMS); };
  const uint32_t s_items = sb + S_::OFF_ITEMS;
  auto s_q = [&](int s) { return sb + S_::OFF_Q + s * S_::TILE_BYTES; };
  auto s_kv = [&](uint32_t s) { return sb + S_::OFF_KV + s * S_::TILE_BYTES; };
  uint32_t* flags = reinterpret_cast<uint32_t*>(smem + S_::OFF_FLAGS);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 2);   // both slots' products have passed it
      mbar_init(guard_go(s), 1);
      mbar_init(guard_done(s), 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_full(s), 1);
      mbar_init(p_full(s), 4);
      mbar_init(p_rest(s), 4);
      mbar_init(o_full(s), 1);
      mbar_init(flags_full(s), 1);
      mbar_init(flags_free(s), 8);
    }
    mbar_init(final_bar, 1);
    mbar_init(final_bar + 8, 1);
    mbar_init(turn_bar, 1);
    mbar_init(turn_bar + 8, 1);
    for (int i = 0; i < ITEMS; ++i) {
      mbar_init(item_full(i), 1);
      mbar_init(item_empty(i), 11);   // every warp but the one that writes them
    }
    fence_mbar_init();
  }
  if (warp == MMA_WARP) {
    tmem_alloc(sb + S_::OFF_TMEM, TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == TMA_WARP && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem =
      __shfl_sync(0xFFFFFFFFu, *reinterpret_cast<volatile uint32_t*>(smem + S_::OFF_TMEM), 0);
  griddep_wait();
  griddep_launch_dependents();

  Item it = {};
  uint32_t n = 0;   // items so far
  // The next item, as the TMA warp has written it down; false behind the last.
  auto next_item = [&]() {
    if (!__all_sync(0xFFFFFFFFu, svdq_wait(item_full(n), (n / ITEMS) & 1u, SITE_ITEM))) return false;
    const uint32_t at = s_items + 32 * (n % ITEMS);
    uint32_t w[6];
    ld_shared_v4(at, w[0], w[1], w[2], w[3]);
    ld_shared_v2(at + 16, w[4], w[5]);
    // (by shuffle, as the warp's number: loops over them are then uniform)
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = __shfl_sync(0xFFFFFFFFu, w[i], 0);
    it.begin = w[0], it.len = w[1], it.q0 = w[2], it.head = w[3];
    it.ka = SPLIT ? w[4] : 0;
    it.kb = SPLIT ? w[5] : it.all_tiles(p.causal);
    if (lane == 0) mbar_arrive(item_empty(n));
    return it.len > 0;
  };
  if (warp >= MMA_WARP) {
    set_max_regs_down<OTHER_REGS>();
    if (warp == TMA_WARP) {
      // ------------------------------------------------------------ TMA --
      uint32_t kv = 0;   // ring uses
      bool ok = true;
      Items<SPLIT> items;
      items.start(p);
      for (bool more = true; more && ok; ++n) {
        more = items.get(p, it);
        ok = __all_sync(0xFFFFFFFFu, svdq_wait(item_empty(n), ((n / ITEMS) & 1u) ^ 1u, SITE_TMA_ITEM));
        if (!ok) break;
        if (lane == 0) {
          const uint32_t at = s_items + 32 * (n % ITEMS);
          st_shared_v4(at, it.begin, more ? it.len : 0, it.q0, it.head);
          st_shared_v4(at + 16, it.ka, it.kb, 0, 0);
          mbar_arrive(item_full(n));
        }
        if (!more) break;
        if (lane == 0) {
          const int kh = it.head / p.group;
          ok = svdq_wait(q_empty, (n & 1u) ^ 1u, SITE_TMA_Q);
          if (ok) {
            const int slots = it.q0 + ROWS < it.len ? 2 : 1;
            mbar_arrive_expect_tx(q_full, slots * S_::TILE_BYTES);
            for (int s = 0; s < slots; ++s)
              for (int b = 0; b < NB; ++b)
                tma_load_3d(s_q(s) + b * BOX_BYTES, &tm_q, 64 * b, it.head,
                            it.begin + it.q0 + s * ROWS, q_full);
          }
          for (int j = 2 * it.ka; ok && j < 2 * it.kb; ++j, ++kv) {
            const uint32_t st = kv % STAGES;
            ok = svdq_wait(empty_bar(st), ((kv / STAGES) & 1u) ^ 1u, SITE_TMA_KV);
            if (!ok) break;
            mbar_arrive_expect_tx(full_bar(st), S_::TILE_BYTES);
            for (int b = 0; b < NB; ++b)
              tma_load_3d(s_kv(st) + b * BOX_BYTES, (j & 1) ? &tm_v : &tm_k, 64 * b, kh,
                          it.begin + (j >> 1) * ROWS, full_bar(st));
            if ((j & 1) && (j >> 1) >= it.guard_from(p.causal)) mbar_arrive(guard_go(st));
          }
        }
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      }
      if (lane == 0) {
        // Every copy issued has landed before the block exits (after an
        // error nobody else may be waiting for them).
        for (uint32_t j = 0; j < min(kv, static_cast<uint32_t>(STAGES)); ++j) {
          const uint32_t u = kv - 1 - j;
          drain_wait(full_bar(u % STAGES), (u / STAGES) & 1u, 50000000ull);
        }
        if (n > 0) drain_wait(q_full, (n - 1) & 1u, 50000000ull);
      }
      __syncwarp();
    } else if (warp != GUARD_WARP) {
      // ------------------------------------------------------------ MMA --
      // A warp per slot; they take turns at the tensor core, a slot's P V and
      // next Q K^T at a time, the next turn beginning when these are done.
      // That keeps the slots half a period apart: left alone they fall into
      // step and want the same unit at the same time (4352 x 30 heads: 365
      // us), and with the turn handed on earlier one slot's last weights are
      // taken beside the other's first ones (278 us, against 252).
      // The warp stays together (one lane issues), so that descriptors are
      // uniform and an MMA costs an addition or two to issue: the tensor core
      // takes 64 cycles for one.
      const int s = warp - MMA_WARP;
      const uint32_t leader = elect_one();
      const uint32_t dn = (p.D + 15) / 16 * 16;   // columns of O, and k of Q K^T
      const int dk = dn / 16;
      const uint32_t id_o = BF16 ? idesc_bf16_f32(ROWS, dn, 0, 1) : idesc_f16_f32(ROWS, dn, 0, 1);
      const uint64_t desc_q = smem_desc(s_q(s), 16, 1024, kLayoutSwizzle128B);
      const uint64_t desc_k = smem_desc(s_kv(0), 16, 1024, kLayoutSwizzle128B);
      const uint64_t desc_v = smem_desc(s_kv(0), BOX_BYTES, 1024, kLayoutSwizzle128B);
      constexpr uint32_t TILE_16 = S_::TILE_BYTES / 16;
      const uint32_t tm_s = tmem + TM_S + ROWS * s, tm_o = tmem + TM_O + ROWS * s;
      const uint32_t b_s = s_full(s), b_p = p_full(s), b_rest = p_rest(s), b_o = o_full(s);
      uint32_t st = 0, ph = 0;          // next use of the ring: stage, parity
      uint32_t guards = 0;              // parity of the guarded uses, by stage
      uint32_t np = 0;                  // P tiles
      uint32_t turn = s ^ 1u;           // parity of the turns (slot 0 has the first)
      bool ok = true;
      auto wait = [&](uint32_t b, uint32_t parity, uint32_t site) {
        if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(b, parity)))
          ok = __all_sync(0xFFFFFFFFu, svdq_wait(b, parity, site)) && ok;
      };
      auto next = [&]() {
        if (++st == STAGES) st = 0, ph ^= 1u;
      };
      for (; ok && next_item(); ++n) {
        // (tiles by their number from ka on: loops from zero)
        const int tiles = it.kb - it.ka;
        const int mine = it.end(s, p.causal) - it.ka;   // this slot's
        const int last = it.key_tiles() - 1 - it.ka;    // the sequence's last
        const int last_steps = (it.len % ROWS + ROWS - 1) % ROWS / 16 + 1;   // 16-key steps of that one
        const int guard_from = it.guard_from(p.causal) - it.ka;
        // S of tile j from stage `at`; with `pass` the other slot's turn begins
        // when it is done.
        auto qk = [&](int j, uint32_t at, bool pass) {
          if (j < mine) {
            const uint32_t keys = j == last ? 16 * last_steps : ROWS;
            const uint32_t id = BF16 ? idesc_bf16_f32(ROWS, keys, 0, 0) : idesc_f16_f32(ROWS, keys, 0, 0);
            const uint64_t dkk = desc_k + TILE_16 * at;
#pragma unroll
            for (int c = 0; c < 4 * NB; ++c) {
              const uint64_t off = ((c >> 2) * BOX_BYTES + 32 * (c & 3)) / 16;
              if (c < dk) mma_f16_by(leader, tm_s, desc_q + off, dkk + off, id, c != 0);
            }
            tc_commit_by(leader, b_s);
            if (pass) tc_commit_by(leader, turn_bar + 8 * (s ^ 1));
          } else if (pass && leader) {
            mbar_arrive(turn_bar + 8 * (s ^ 1));
          }
          tc_commit_by(leader, empty_bar(at));
          if (j == tiles - 1) tc_commit_by(leader, q_empty);
        };
        wait(q_full, n & 1u, SITE_MMA_Q);
        wait(full_bar(st), ph, SITE_MMA_KV);
        tc_fence_after();
        if (!ok) break;
        qk(0, st, false);
        next();
        for (int j = 0; j < tiles; ++j) {
          // All that the turn's products need is there before it is taken.
          const uint32_t sv = st;
          const uint64_t dv = desc_v + TILE_16 * sv;
          const bool more = j + 1 < tiles;
          wait(full_bar(sv), ph, SITE_MMA_KV);
          if (j >= guard_from) {
            wait(guard_done(sv), (guards >> sv) & 1u, SITE_MMA_GUARD);
            guards ^= 1u << sv;
          }
          next();
          const uint32_t sk = st;
          if (more) {
            wait(full_bar(sk), ph, SITE_MMA_KV);
            next();
          }
          if (j < mine) wait(b_p, np & 1u, SITE_MMA_P);
          wait(turn_bar + 8 * s, turn, SITE_MMA_TURN);
          turn ^= 1u;
          tc_fence_after();
          if (!ok) break;
          if (j < mine) {
            const int steps = j == last ? last_steps : ROWS / 16;
            // The first keys of P are multiplied while the softmax warps are
            // at the rest.
#pragma unroll
            for (int c = 0; c < P_STEPS; ++c)
              if (c < steps)
                mma_f16_ts_by(leader, tm_o, tm_s + 8 * c, dv + 128 * c, id_o, c == 0 ? j != 0 : 1u);
            wait(b_rest, np++ & 1u, SITE_MMA_P);
            tc_fence_after();
            if (!ok) break;
#pragma unroll
            for (int c = P_STEPS; c < ROWS / 16; ++c)
              if (c < steps) mma_f16_ts_by(leader, tm_o, tm_s + 8 * c, dv + 128 * c, id_o, 1u);
            if (j == mine - 1) tc_commit_by(leader, b_o);
          }
          tc_commit_by(leader, empty_bar(sv));
          if (more)
            qk(j + 1, sk, true);
          else if (leader)
            mbar_arrive(turn_bar + 8 * (s ^ 1));
        }
      }
      // Every MMA issued completes before TMEM is released.
      tc_commit_by(leader, final_bar + 8 * s);
      drain_wait(final_bar + 8 * s, 0, 100000000ull);
      __syncwarp();
    } else {
      // ---------------------------------------------------------- guard --
      uint32_t kv = 0, phases = 0;
      if (SPLIT && lane < 2) p.ws.meta[2 * blockIdx.x + lane].valid = 0;   // no partial results yet
      __syncwarp();
      bool ok = true;
      for (; ok && next_item(); ++n) {
        uint32_t* f = flags + 8 * (n & 1);
        if (p.causal) {
          // the epilogues of the item before last have read these words
          if (n >= 2)
            ok = __all_sync(0xFFFFFFFFu, svdq_wait(flags_free(n & 1), ((n >> 1) & 1u) ^ 1u,
                                                   SITE_GUARD_FLAGS));
          if (!ok) break;
          if (lane < 8) f[lane] = 0u;
          __syncwarp();
        }
        for (int j = it.guard_from(p.causal); ok && j < it.kb; ++j) {
          const uint32_t u = kv + 2 * (j - it.ka) + 1;
          const uint32_t st = u % STAGES;
          ok = __all_sync(0xFFFFFFFFu, svdq_wait(guard_go(st), (phases >> st) & 1u, SITE_GUARD_V) &&
                                           svdq_wait(full_bar(st), (u / STAGES) & 1u, SITE_GUARD_V));
          if (!ok) break;
          phases ^= 1u << st;
          const int valid = min(ROWS, it.len - j * ROWS);
          uint32_t* fj = f + 4 * (j - it.q0 / ROWS);   // causal
          // 16-byte words of the tile's boxes: eight per row
          const int stop = (valid + 15) / 16 * 16;
          const uint32_t tile = s_kv(st);
          for (int b = 0; b < NB; ++b)
            for (int c = 8 * valid + lane; c < 8 * stop; c += 32)
              st_shared_v4(tile + b * BOX_BYTES + 16 * c, 0u, 0u, 0u, 0u);
          if (p.causal) {
            // First only whether there is a non-finite value at all: the
            // largest magnitude of each lane's words, NaN if there is one.
            uint32_t top = 0;
            for (int b = 0; b < NB; ++b) {
              const uint32_t box = tile + b * BOX_BYTES;
#pragma unroll 8
              for (int c = lane; c < 8 * valid; c += 32) {
                uint32_t x[4];
                ld_shared_v4(box + 16 * c, x[0], x[1], x[2], x[3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) top = max_abs2<BF16>(top, x[i]);
              }
            }
            const bool bad = is_nonfinite16<BF16>(top) || is_nonfinite16<BF16>(top >> 16);
            if (__any_sync(0xFFFFFFFFu, bad)) {
              clean_tile<BF16, NB>(tile, valid, fj);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(guard_done(st));
        }
        if (ok && p.causal && lane == 0) mbar_arrive(flags_full(n & 1));
        kv += 2 * (it.kb - it.ka);
        if (SPLIT && lane == 0 && !it.whole(p.causal)) {
          Meta& m = p.ws.meta[2 * blockIdx.x + (it.ka > 0 ? 0 : 1)];
          m.valid = 1;
          m.last = it.kb == it.all_tiles(p.causal);
          m.begin = it.begin, m.len = it.len, m.q0 = it.q0, m.head = it.head;
        }
      }
    }
  } else {
    // ----------------------------------------------------------- softmax --
    set_max_regs_up<SOFTMAX_REGS>();
    const int slot = warp >> 2;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t tm_s = lane_base + TM_S + ROWS * slot;
    const uint32_t tm_o = lane_base + TM_O + ROWS * slot;
    const int r = (warp & 3) * 32 + lane;   // row of the slot
    const float sc = p.scale_log2;
    uint32_t ns = 0, no = 0;                // S tiles, O tiles waited for
    bool ok = true;
    for (; ok && next_item(); ++n) {
      const int tiles = it.end(slot, p.causal) - it.ka;   // the slot's, from ka on
      const bool whole = !SPLIT || it.whole(p.causal);
      auto notes = [&]() {   // the guard has been through this item
        return __all_sync(0xFFFFFFFFu, svdq_wait(flags_full(n & 1), (n >> 1) & 1u, SITE_SOFT_FLAGS)) != 0;
      };
      const int row = it.q0 + slot * ROWS + r;   // of the sequence
      if (tiles > 0) {
        const int row_keys = (p.causal ? min(it.len, row + 1) : it.len) - it.ka * ROWS;   // from ka on
        float m = -INFINITY;     // reference of the row, raw units of S
        float off = REF_LOG2<BF16>;   // less m in log2 units, unless m is taken off first
        bool big = false;        // m is taken off first in a row of the warp
        uint64_t sum2 = 0;       // of the weights, even and odd keys
        for (int j = 0; j < tiles; ++j) {
          ok = __all_sync(0xFFFFFFFFu, svdq_wait(s_full(slot), ns++ & 1u, SITE_SOFT_S));
          if (!ok) break;
          tc_fence_after();
          uint32_t x[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(tm_s + 32 * c, x[c]);
          tmem_ld_wait();
          // keys at or behind `keys` are not this row's
          const int keys = row_keys - j * ROWS;
          if (__any_sync(0xFFFFFFFFu, keys < ROWS)) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (32 * c + e >= keys) x[c][e] = 0xFF800000u;   // -inf
          }
          // Weights 2^(x sc + off) of 32 keys, packed, and their sum.
          auto weights = [&](const uint32_t (&xc)[32], uint32_t (&w16)[16]) {
            const uint64_t sc2 = pk(sc, sc), off2 = pk(off, off);
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float a, b;
              upk(fma2(pk(__uint_as_float(xc[2 * e]), __uint_as_float(xc[2 * e + 1])), sc2, off2), a, b);
              a = ex2_approx_ftz(a);
              b = ex2_approx_ftz(b);
              sum[e & 1] = add2(sum[e & 1], pk(a, b));
              w16[e] = pack2<BF16>(a, b);
            }
            return add2(sum[0], sum[1]);
          };
          // The first weights are taken with the present reference, beside
          // the maximum that says whether it still holds: it nearly always
          // does, so the maximum is off the way from S to P.
          uint32_t w16[16];
          uint64_t part = weights(x[0], w16);
          float t[4] = {m, m, m, m};
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              t[(e >> 1) & 3] = max3(t[(e >> 1) & 3], __uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1]));
          const float top = fmaxf(max3(t[0], t[1], t[2]), t[3]);
          // The votes say whether the warp comes here; what happens to a row
          // is decided by its own maximum, so that rows which share a warp
          // (other queries, rows of another sequence) do not show in it.
          const bool grown = __any_sync(0xFFFFFFFFu, (top - m) * sc > RESCALE_LOG2);
          if (grown || big) {
            if (grown) {
              const float to = (top - m) * sc > RESCALE_LOG2 ? top : m;
              const float f = to == m ? 1.f : ex2_approx_ftz((m - to) * sc);
              m = to;
              sum2 = mul2(sum2, pk(f, f));
              if (j > 0) {
                // O is idle here: the commit behind s_full also covers this
                // slot's previous P V.
                for (int c = 0; c < p.D; c += 16) {
                  uint32_t o[16];
                  tmem_ld_32x32b_x16(tm_o + c, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                  tmem_st_32x32b_x16(tm_o + c, o);
                }
              }
              const float msc = m == -INFINITY ? 0.f : m * sc;
              off = REF_LOG2<BF16> - msc;
              big = __any_sync(0xFFFFFFFFu, fabsf(msc) > 4096.f);
            }
            // Exponents x sc - m sc come from one fma: the rounding of m sc,
            // 2^-24 of it, adds to the one S has anyway.  Where m sc is so
            // large that this would show (2^-12 and more), m is taken off
            // first.
            if (big) {
              const bool far = m != -INFINITY && fabsf(m * sc) > 4096.f;
              const float ref = far ? m : 0.f;
              off = far ? REF_LOG2<BF16> : off;
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 32; ++e) x[c][e] = __float_as_uint(__uint_as_float(x[c][e]) - ref);
            }
            part = weights(x[0], w16);
          }
          sum2 = add2(sum2, part);
          tmem_st_32x32b_x16(tm_s, w16);
#pragma unroll
          for (int c = 1; c < 4; ++c) {
            sum2 = add2(sum2, weights(x[c], w16));
            tmem_st_32x32b_x16(tm_s + 16 * c, w16);
            if (c >= 2) {   // P_STEPS steps of 16 keys are there, then the rest
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(c == 2 ? p_full(slot) : p_rest(slot));
            }
          }
        }
        if (!ok) break;
        // -------------------------------------------------------- epilogue --
        ok = __all_sync(0xFFFFFFFFu, svdq_wait(o_full(slot), no++ & 1u, SITE_SOFT_O));
        if (!ok) break;
        tc_fence_after();
        float l0, l1;
        upk(sum2, l0, l1);
        // A partial result stays unscaled, in fp32.
        const float inv = whole ? 1.f / (l0 + l1) : 1.f;
        const uint32_t* f = flags + 8 * (n & 1);
        uint32_t noted = 0;
        if (p.causal) {
          ok = notes();
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < 8; ++i) noted |= f[i];
        }
        // Out by way of shared memory, 128 bytes of each of the warp's rows at
        // a time, so that a store covers four whole lines instead of a piece
        // of 32 (straight from the registers an item's rows took 4000 cycles
        // of the memory pipe).  16-byte piece i of row k stands at i ^ (k & 7).
        const uint32_t stage = sb + S_::OFF_OUT + 4096 * warp;
        const int row0 = it.q0 + slot * ROWS + (warp & 3) * 32;   // the warp's first row
        const int prow = (2 * blockIdx.x + (it.ka > 0 ? 0 : 1)) * ITEM_ROWS + slot * ROWS + (warp & 3) * 32;
        const int dp = (p.D + 15) / 16 * 16;
        if (!whole) p.ws.ml[prow + lane] = make_float2(m, l0 + l1);
        const int width = whole ? 64 : 32;   // columns of 128 bytes
        for (int c0 = 0; c0 < p.D; c0 += width) {
          for (int c = c0; c < min(c0 + width, p.D); c += 16) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(tm_o + c, o);
            tmem_ld_wait();
            float v[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(o[e]) * inv;
            if (noted != 0u) {
              // Non-finite values of the diagonal tiles: into the rows that attend them.
              for (int i = 0; i < 8; ++i) {
                for (uint32_t b = f[i]; b != 0u; b &= b - 1) {
                  const int key = it.q0 + 32 * i + __ffs(b) - 1;
                  if (key > row) continue;
                  const uint16_t* src = p.v + static_cast<int64_t>(it.begin + key) * p.vst +
                                        (it.head / p.group) * p.vsh + c;
#pragma unroll
                  for (int e = 0; e < 16; ++e) {
                    if (c + e >= p.D) break;
                    const uint32_t u = src[e];
                    if (is_nonfinite16<BF16>(u))
                      v[e] += BF16 ? __uint_as_float(u << 16)
                                   : __half2float(__ushort_as_half(static_cast<unsigned short>(u)));
                  }
                }
              }
            }
            const uint32_t line = stage + 128 * lane;
            if (whole) {
              const int i = (c - c0) / 8;
#pragma unroll
              for (int k = 0; k < 2; ++k)
                st_shared_v4(line + 16 * ((i + k) ^ (lane & 7)), pack2<BF16>(v[8 * k], v[8 * k + 1]),
                             pack2<BF16>(v[8 * k + 2], v[8 * k + 3]), pack2<BF16>(v[8 * k + 4], v[8 * k + 5]),
                             pack2<BF16>(v[8 * k + 6], v[8 * k + 7]));
            } else {
              const int i = (c - c0) / 4;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                st_shared_v4(line + 16 * ((i + k) ^ (lane & 7)), __float_as_uint(v[4 * k]),
                             __float_as_uint(v[4 * k + 1]), __float_as_uint(v[4 * k + 2]),
                             __float_as_uint(v[4 * k + 3]));
            }
          }
          __syncwarp();
          const int i = lane & 7;   // eight lanes a row, four rows a store
          const bool in = whole ? c0 + 8 * i < p.D : c0 + 4 * i < dp;
#pragma unroll
          for (int k0 = 0; k0 < 32; k0 += 4) {
            const int k = k0 + (lane >> 3);
            uint4 w;
            ld_shared_v4(stage + 128 * k + 16 * (i ^ (k & 7)), w.x, w.y, w.z, w.w);
            if (!in) continue;
            if (whole) {
              if (row0 + k < it.len)
                *reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(it.begin + row0 + k) * p.ost +
                                          it.head * p.osh + c0 + 8 * i) = w;
            } else {
              *reinterpret_cast<uint4*>(p.ws.o + static_cast<size_t>(prow + k) * dp + c0 + 4 * i) = w;
            }
          }
          __syncwarp();
        }
        tc_fence_before();
      }
      if (p.causal) {
        // (also a slot that had nothing here waits for the notes: else it
        // would run ahead and arrive for a later item in this one's phase)
        if (tiles <= 0) ok = notes();
        __syncwarp();
        if (lane == 0) mbar_arrive(flags_free(n & 1));
      }
    }
  }

  // ----------------------------------------------------------- teardown --
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Joins the partial results of split items.  An item begins in block b's
// second one and goes on in the first ones of the blocks behind b, up to the
// one that has its last key tile: the rows' references are brought to the
// largest, sums and O added in that order, O divided by the sum.  Grid
// (blocks, JOIN_PARTS): each block 256 / JOIN_PARTS rows, a warp four of them
// at a time (it waits for memory once, not once a row).
constexpr int JOIN_PARTS = 8;
constexpr int JOIN_THREADS = 256;

template <bool BF16>
__global__ void __launch_bounds__(JOIN_THREADS) join_kernel(const Params p) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x, blocks = gridDim.x;
  const Meta first = p.ws.meta[2 * b + 1];
  if (!first.valid) return;
  int parts = 1;
  for (bool last = first.last; !last && b + parts < blocks; ++parts) {
    const Meta& m = p.ws.meta[2 * (b + parts)];
    if (!m.valid) break;
    last = m.last;
  }
  constexpr int R = ITEM_ROWS / JOIN_PARTS / (JOIN_THREADS / 32);   // rows of a warp
  const int lane = threadIdx.x & 31;
  const int r0 = blockIdx.y * (ITEM_ROWS / JOIN_PARTS) + (threadIdx.x >> 5) * R;
  if (first.q0 + r0 >= first.len) return;
  const int dp = (p.D + 15) / 16 * 16;
  const int col = 4 * lane;
  auto place = [&](int k) { return static_cast<size_t>(k == 0 ? 2 * b + 1 : 2 * (b + k)) * ITEM_ROWS + r0; };
  // (rows behind the sequence's end are computed too, from memory of the
  // workspace that may not have been written, and not stored)
  float top[R], l[R];
  float4 o[R];
#pragma unroll
  for (int i = 0; i < R; ++i) top[i] = -INFINITY, l[i] = 0.f, o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < parts; ++k) {
#pragma unroll
    for (int i = 0; i < R; ++i) top[i] = fmaxf(top[i], p.ws.ml[place(k) + i].x);
  }
#pragma unroll 2
  for (int k = 0; k < parts; ++k) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float2 ml = p.ws.ml[place(k) + i];
      const float f = ml.x == top[i] ? 1.f : ex2_approx_ftz((ml.x - top[i]) * p.scale_log2);
      l[i] = fmaf(ml.y, f, l[i]);
      if (col < dp) {
        const float4 v = *reinterpret_cast<const float4*>(p.ws.o + (place(k) + i) * dp + col);
        o[i].x = fmaf(v.x, f, o[i].x);
        o[i].y = fmaf(v.y, f, o[i].y);
        o[i].z = fmaf(v.z, f, o[i].z);
        o[i].w = fmaf(v.w, f, o[i].w);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = first.q0 + r0 + i;
    if (row >= first.len || col >= p.D) continue;
    const float inv = 1.f / l[i];
    uint16_t* dst = p.out + static_cast<int64_t>(first.begin + row) * p.ost + first.head * p.osh + col;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<BF16>(o[i].x * inv, o[i].y * inv),
                                                pack2<BF16>(o[i].z * inv, o[i].w * inv));
  }
}

}  // namespace ka
}  // namespace svdq
